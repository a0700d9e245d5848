"""moe_adapter_forward and moe_adapter_backward against their definitions in 64 bits.

Bounds: products of bf16 values are exact and each fp32 sum of n of them is off by at most
n 2^-23 of the sum of magnitudes (which covers an accumulator that truncates); the fp32
low-rank values enter further products as bf16 terms (two terms: off by 2^-16 at most, three:
2^-23); bf16 outputs are rounded once (2^-8)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, TWO = 2.0 ** -8, 2.0 ** -23, 2.0 ** -16


def make(T, d_in, d_out, L, r, seed, ids="mixed"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)

    inp = dict(x=normal(T, d_in), d_y=normal(T, d_out, std=0.1), w=normal(d_in, d_out, std=d_in ** -0.5),
               a=normal(L, d_in, r, std=d_in ** -0.5), b=normal(L, r, d_out, std=r ** -0.5),
               scale=torch.rand(L, generator=g, device="cuda") * 2 + 0.1)
    if ids == "mixed":  # any adapter, or none, in any row
        i = torch.randint(-1, L, (T,), generator=g, device="cuda")
    elif ids == "runs":  # a few requests of several rows
        cut = torch.randint(0, T, (max(1, T // 100),), generator=g, device="cuda")
        run = torch.zeros(T, dtype=torch.int64, device="cuda").index_fill_(0, cut, 1).cumsum(0)
        i = torch.randint(-1, L, (T + 1,), generator=g, device="cuda")[run]
    elif ids == "none":
        i = torch.full((T,), -1, device="cuda")
    else:  # the last adapter only
        i = torch.full((T,), L - 1, device="cuda")
    inp["ids"] = i.int()
    return inp


def low64(x, m, ids, scale):
    """scale_l x M_l by row, and the bound on its fp32 value."""
    low = torch.zeros(x.shape[0], m.shape[2], dtype=torch.float64, device="cuda")
    err = torch.zeros_like(low)
    for l in range(m.shape[0]):
        t = (ids == l).nonzero().squeeze(1)
        low[t] = scale[l].double() * (x[t] @ m[l])
        err[t] = scale[l].double() * (x.shape[1] + 4) * F32 * (x[t].abs() @ m[l].abs())
    return low, err


def through64(x, w, low, dlow, m, ids):
    """x W + low M_l by row, and its bound when low is off by dlow."""
    y = x @ w
    err = (x.shape[1] + 4) * F32 * (x.abs() @ w.abs())
    for l in range(m.shape[0]):
        t = (ids == l).nonzero().squeeze(1)
        y[t] += low[t] @ m[l]
        err[t] += (dlow[t] + (TWO + low.shape[1] * F32) * low[t].abs()) @ m[l].abs()
    return y, err + BF16 * (y.abs() + err) + 1e-30


def call_forward(tdr, inp, **kw):
    T, d_in = inp["x"].shape
    L, r, d_out = inp["b"].shape
    s = tdr.make_adapter_shape(T, d_in, d_out, L, r)
    return s, tdr.adapter_forward(s, inp["x"], inp["w"], inp["a"], inp["b"], inp["ids"],
                                  inp["scale"], **kw)


SHAPES = [  # T, d_in, d_out, L, r
    (1, 64, 64, 1, 8), (1, 4096, 4096, 8, 16), (2, 128, 320, 3, 24), (16, 2048, 192, 5, 128),
    (57, 2048, 2880, 32, 16), (127, 192, 1024, 256, 40), (128, 1024, 512, 7, 64),
    (129, 64, 64, 1, 8), (130, 320, 448, 3, 24), (255, 512, 64, 9, 32), (257, 2048, 768, 4, 8),
    (300, 192, 960, 256, 16), (1111, 2880, 320, 5, 40), (2049, 1024, 2880, 48, 24),
    (700, 256, 512, 6, 128),
]


@pytest.mark.parametrize("T,d_in,d_out,L,r", SHAPES)
@pytest.mark.parametrize("ids", ["mixed", "runs", "none", "one"])
def test_forward_matches_the_definition(cuda_lib, T, d_in, d_out, L, r, ids):
    tdr = cuda_lib
    inp = make(T, d_in, d_out, L, r, T + r, ids)
    out = torch.full((T, d_out), 7.0, dtype=torch.bfloat16, device="cuda")
    low = torch.full((T, r), 7.0, device="cuda")
    call_forward(tdr, inp, out=out, low=low)
    assert tdr.device_status() == 0
    x, w, a, b = (inp[k].double() for k in ("x", "w", "a", "b"))
    lref, lerr = low64(x, a, inp["ids"], inp["scale"])
    assert ((low.double() - lref).abs() <= lerr).all()
    y, err = through64(x, w, lref, lerr, b, inp["ids"])
    bad = (out.double() - y).abs() > err
    assert not bad.any(), (bad.sum().item(), ((out.double() - y).abs() / err).max().item())


@pytest.mark.parametrize("T,d_in,d_out,L,r", SHAPES + [(4100, 512, 128, 2, 16)])
@pytest.mark.parametrize("ids", ["mixed", "runs", "none", "one"])
def test_backward_matches_the_definition(cuda_lib, T, d_in, d_out, L, r, ids):
    tdr = cuda_lib
    inp = make(T, d_in, d_out, L, r, T + r + 1, ids)
    x, d_y, w, a, b = (inp[k].double() for k in ("x", "d_y", "w", "a", "b"))
    low = low64(x, a, inp["ids"], inp["scale"])[0].float()
    s = tdr.make_adapter_shape(T, d_in, d_out, L, r)
    d_x = torch.full((T, d_in), 7.0, dtype=torch.bfloat16, device="cuda")
    d_a = torch.full((L, d_in, r), 7.0, device="cuda")
    d_b = torch.full((L, r, d_out), 7.0, device="cuda")
    tdr.adapter_backward(s, inp["d_y"], inp["x"], inp["w"], inp["a"], inp["b"], inp["ids"],
                         inp["scale"], low, d_x=d_x, d_a=d_a, d_b=d_b)
    assert tdr.device_status() == 0
    dl, dlerr = low64(d_y, b.transpose(1, 2), inp["ids"], inp["scale"])
    ref, err = through64(d_y, w.t(), dl, dlerr, a.transpose(1, 2), inp["ids"])
    bad = (d_x.double() - ref).abs() > err
    assert not bad.any(), ("d_x", bad.sum().item(), ((d_x.double() - ref).abs() / err).max().item())
    for l in range(L):
        t = (inp["ids"] == l).nonzero().squeeze(1)
        n = t.numel() + 8
        ra, rb = x[t].t() @ dl[t], low[t].double().t() @ d_y[t]
        ea = x[t].abs().t() @ (dlerr[t] + n * F32 * dl[t].abs())
        eb = n * F32 * (low[t].double().abs().t() @ d_y[t].abs())
        assert ((d_a[l].double() - ra).abs() <= ea).all(), ("d_a", l)
        assert ((d_b[l].double() - rb).abs() <= eb).all(), ("d_b", l)
