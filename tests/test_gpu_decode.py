"""moe_decode, the layer for a few tokens, against the layer's definition in 64 bits.

The bound of each output value follows the kernel's roundings: products of bf16 values are
exact and summed in fp32 (each of n additions off by at most 2^-23 of the sum of magnitudes,
which covers an accumulator that truncates), silu(g) * u is taken to 2^-18 relative (fast
exponential and divide) and rounded to bf16 (2^-8), the second product is summed in fp32, and
the combined row is rounded to bf16 (2^-8)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = 2.0 ** -8, 2.0 ** -23


def make(T, d, E, K, n, seed, bias=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)

    inp = dict(x=normal(T, d), w_r=normal(d, E, std=d ** -0.5), w_gate=normal(E, d, n, std=d ** -0.5),
               w_up=normal(E, d, n, std=d ** -0.5), w_down=normal(E, n, d, std=n ** -0.5))
    inp["bias"] = None
    if bias:
        inp["bias"] = torch.empty(E, device="cuda").normal_(0, 1, generator=g)
    return inp


def logits_of(inp):
    lg = inp["x"].double() @ inp["w_r"].double()
    return lg if inp["bias"] is None else lg + inp["bias"].double()


def layer64(inp, logits, K, renorm=True, capacity=0.0):
    """The layer and the bound on the kernel's error, both [T, d] in 64 bits."""
    x = inp["x"].double()
    T, E = logits.shape
    d, n = inp["w_gate"].shape[1:]
    ids = torch.argsort(-logits, dim=1, stable=True)[:, :K]
    p = torch.softmax(logits, 1)
    w = torch.gather(p, 1, ids)
    if renorm:
        w = w / w.sum(1, keepdim=True)
    C = math.ceil(capacity * T * K / E) if capacity > 0 else T
    out, err = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(E):
        t, k = (ids == e).nonzero(as_tuple=True)
        t, k = t[:C], k[:C]
        if not t.numel():
            continue
        wg, wu, wd = (inp[m][e].double() for m in ("w_gate", "w_up", "w_down"))
        g, u = x[t] @ wg, x[t] @ wu
        s = torch.sigmoid(g)
        act = g * s * u
        dg, du = d * F32 * (x[t].abs() @ wg.abs()), d * F32 * (x[t].abs() @ wu.abs())
        # |d silu| <= 1.1; second-order terms are covered by the factors' slack
        dact = (BF16 + 2.0 ** -18) * act.abs() + 1.1 * dg * u.abs() + (g * s).abs() * du
        wt = w[t, k].unsqueeze(1)
        out[t] += wt * (act @ wd)
        err[t] += wt * (1.01 * dact @ wd.abs() + (n + 4) * F32 * (act.abs() @ wd.abs()))
    # the weights: fp32 logits (their error moves a weight by at most twice as much), softmax
    dl = (d + 8) * F32 * (x.abs() @ inp["w_r"].double().abs()).amax(1, keepdim=True)
    return out, err + (4 * dl + 2.0 ** -20) * (out.abs() + err) + BF16 * (out.abs() + err) + 1e-30


def settled(logits, K):
    """Rows whose top-K does not hang on the last bits of a logit."""
    v = logits.sort(1, descending=True).values
    gap = (v[:, :K] - v[:, 1:K + 1]).amin(1) if K < logits.shape[1] else \
        (v[:, :-1] - v[:, 1:]).amin(1) if K > 1 else torch.ones_like(v[:, 0])
    return gap > 1e-4


SHAPES = [  # T, d, E, K, n
    (1, 64, 1, 1, 64), (1, 256, 8, 2, 512), (1, 2048, 128, 8, 768), (2, 320, 7, 3, 192),
    (3, 128, 256, 32, 64), (7, 4096, 8, 2, 1024), (15, 2880, 32, 4, 2880), (16, 512, 16, 4, 448),
    (17, 192, 33, 5, 320), (33, 1024, 40, 8, 256), (64, 2048, 128, 8, 768), (65, 960, 12, 12, 704),
    (127, 448, 5, 2, 1344), (128, 1024, 64, 6, 512), (128, 256, 200, 20, 128),
]


@pytest.mark.parametrize("T,d,E,K,n", SHAPES)
@pytest.mark.parametrize("given", [False, True], ids=["routed", "given"])
def test_matches_the_definition(cuda_lib, T, d, E, K, n, given):
    tdr = cuda_lib
    inp = make(T, d, E, K, n, seed=T + d + E, bias=E % 2 == 0)
    lg = logits_of(inp)
    s = tdr.make_shape(T, d, E, K, n)
    out = torch.full((T, d), 7.0, dtype=torch.bfloat16, device="cuda")
    if given:
        lg = lg.float()
        tdr.decode(s, inp["x"], None, inp["w_gate"], inp["w_up"], inp["w_down"], logits_in=lg,
                   out=out)
    else:
        tdr.decode(s, inp["x"], inp["w_r"], inp["w_gate"], inp["w_up"], inp["w_down"],
                   bias=inp["bias"], out=out)
    assert tdr.device_status() == 0
    ref, tol = layer64(inp, lg.double(), K)
    ok = settled(lg, K) if not given else torch.ones(T, dtype=torch.bool, device="cuda")
    assert ok.float().mean() > 0.5
    bad = ((out.double() - ref).abs() > tol) & ok.unsqueeze(1)
    assert not bad.any(), (bad.sum().item(), ((out.double() - ref).abs() / tol)[ok].max().item())
