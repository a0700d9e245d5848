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


def check(tdr, inp, logits, K, out, **kw):
    ref, tol = layer64(inp, logits, K, **kw)
    ok = settled(logits, K)
    bad = ((out.double() - ref).abs() > tol) & ok.unsqueeze(1)
    assert not bad.any(), ((out.double() - ref).abs() / tol)[ok].max().item()


def run(tdr, s, inp, **kw):
    out, ws = tdr.decode(s, inp["x"], inp["w_r"], inp["w_gate"], inp["w_up"], inp["w_down"],
                         bias=inp["bias"], **kw)
    assert tdr.device_status() == 0
    return out


@pytest.mark.parametrize("T,E,K,capacity,renorm", [
    (37, 32, 4, 1.25, True), (128, 8, 2, 0.5, True), (64, 16, 4, 1e-3, False), (128, 8, 8, 1.0, True),
    (1, 8, 2, 1.0, False), (100, 48, 6, 1e30, False),
])
def test_capacity_and_plain_weights(cuda_lib, T, E, K, capacity, renorm):
    tdr = cuda_lib
    inp = make(T, 512, E, K, 384, seed=5, bias=True)
    inp["bias"] = 1.75 * torch.arange(1, E + 1, device="cuda").float().pow(-1.2)
    s = tdr.make_shape(T, 512, E, K, 384, capacity, renorm)
    lg = logits_of(inp)
    if not settled(lg, K).all():  # a token whose choice hangs on a rounding may displace others
        lg = lg.float().double()
        out, _ = tdr.decode(s, inp["x"], None, inp["w_gate"], inp["w_up"], inp["w_down"],
                            logits_in=lg.float())
    else:
        out = run(tdr, s, inp)
    check(tdr, inp, lg, K, out, renorm=renorm, capacity=capacity)


def test_given_ties_go_to_the_lowest_expert(cuda_lib):
    tdr = cuda_lib
    inp = make(5, 256, 9, 3, 128, seed=3)
    lg = torch.zeros(5, 9, device="cuda")
    lg[1, 4] = lg[1, 7] = 1.0
    lg[2] = -torch.inf
    lg[2, [8, 2, 5]] = 0.25
    s = tdr.make_shape(5, 256, 9, 3, 128)
    out, _ = tdr.decode(s, inp["x"], None, inp["w_gate"], inp["w_up"], inp["w_down"], logits_in=lg)
    ref, tol = layer64(inp, lg.double(), 3)
    assert ((out.double() - ref).abs() <= tol).all()


def test_nan_and_infinite_rows_stay_alone(cuda_lib):
    tdr = cuda_lib
    inp = make(33, 512, 16, 4, 256, seed=8)
    s = tdr.make_shape(33, 512, 16, 4, 256)
    clean = run(tdr, s, inp)
    sick = dict(inp, x=inp["x"].clone())
    sick["x"][3] = torch.nan
    sick["x"][17, 5] = torch.inf
    out = run(tdr, s, sick)
    assert out[3].isnan().all() and not out[17].isfinite().any()
    rest = [t for t in range(33) if t not in (3, 17)]
    assert torch.equal(out[rest], clean[rest])
    lg = logits_of(inp).float()
    lg[6] = torch.nan
    lg[9] = -torch.inf
    out, _ = tdr.decode(s, inp["x"], None, inp["w_gate"], inp["w_up"], inp["w_down"], logits_in=lg)
    assert out[6].isnan().all() and out[9].isnan().all()
    assert out[[t for t in range(33) if t not in (6, 9)]].isfinite().all()


@pytest.mark.parametrize("T,d,E,K,n", [(128, 1024, 64, 6, 512), (64, 2048, 32, 2, 320),
                                       (17, 448, 9, 3, 1344), (128, 256, 8, 2, 64)])
def test_a_broken_expert_reaches_its_own_tokens_only(cuda_lib, T, d, E, K, n):
    tdr = cuda_lib
    inp = make(T, d, E, K, n, seed=T + E)
    lg = logits_of(inp).float()
    s = tdr.make_shape(T, d, E, K, n)
    args = lambda i: (s, i["x"], None, i["w_gate"], i["w_up"], i["w_down"])  # noqa: E731
    clean, _ = tdr.decode(*args(inp), logits_in=lg)
    ids = torch.argsort(-lg.double(), dim=1, stable=True)[:, :K]
    for e, name in ((0, "w_down"), (E - 1, "w_down"), (E // 2, "w_gate"), (1, "w_up"), (2, "w_down")):
        sick = dict(inp, **{name: inp[name].clone()})
        sick[name][e] = torch.inf if e == 2 else torch.nan
        out, _ = tdr.decode(*args(sick), logits_in=lg)
        hit = (ids == e).any(1)
        assert torch.equal(out[~hit], clean[~hit]), (e, name)
        assert not out[hit].isfinite().any(), (e, name)


@pytest.mark.parametrize("T", [1, 19, 128])
def test_workspace_output_and_repetition(cuda_lib, T):
    tdr = cuda_lib
    inp = make(T, 704, 24, 4, 576, seed=T)
    s = tdr.make_shape(T, 704, 24, 4, 576)
    first = run(tdr, s, inp)
    ws = torch.full((tdr.decode_workspace_size(s),), 255, dtype=torch.uint8, device="cuda")  # NaN
    whole = torch.full((T + 2, 704), 3.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(5):
        out = run(tdr, s, inp, workspace=ws, out=whole[1:T + 1])
        assert torch.equal(out, first)
    assert (whole[0] == 3).all() and (whole[T + 1] == 3).all()


def test_streams_and_graphs(cuda_lib):
    tdr = cuda_lib
    sets = [make(T, 512, 16, 2, 512, seed=T) for T in (4, 70, 128)]
    shapes = [tdr.make_shape(i["x"].shape[0], 512, 16, 2, 512) for i in sets]
    ref = [run(tdr, s, i) for s, i in zip(shapes, sets)]
    # at the same time, a workspace each
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for st, s, i in zip(streams, shapes, sets):
            with torch.cuda.stream(st):
                outs.append(tdr.decode(s, i["x"], i["w_r"], i["w_gate"], i["w_up"], i["w_down"],
                                       bias=i["bias"]))
    torch.cuda.synchronize()
    for k, (o, _) in enumerate(outs):
        assert torch.equal(o, ref[k % 3])
    # two graphs that share a workspace, replayed in turn on changed inputs
    ws = torch.empty(max(tdr.decode_workspace_size(s) for s in shapes), dtype=torch.uint8,
                     device="cuda")
    graphs, res = [], []
    for s, i in zip(shapes, sets):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append(tdr.decode(s, i["x"], i["w_r"], i["w_gate"], i["w_up"], i["w_down"],
                                  bias=i["bias"], workspace=ws)[0])
        graphs.append(g)
    for _ in range(3):
        for k, g in enumerate(graphs):
            g.replay()
            assert torch.equal(res[k], ref[k])
    sets[1]["x"].copy_(sets[1]["x"].flip(0))
    for g in graphs:
        g.replay()
    assert torch.equal(res[1], ref[1].flip(0))
    assert torch.equal(res[2], ref[2])
    assert tdr.device_status() == 0


@pytest.mark.parametrize("T", [1, 40, 128])
def test_agrees_with_forward(cuda_lib, T):
    """moe_forward also rounds the expert outputs to bf16 before it combines them."""
    tdr = cuda_lib
    inp = make(T, 1024, 16, 4, 512, seed=2)
    s = tdr.make_shape(T, 1024, 16, 4, 512)
    out = run(tdr, s, inp)
    full, _ = tdr.forward(s, inp["x"], inp["w_r"], inp["w_gate"], inp["w_up"], inp["w_down"])
    lg = logits_of(inp)
    ref, tol = layer64(inp, lg, 4)
    ids = torch.argsort(-lg, dim=1, stable=True)[:, :4]
    parts = torch.zeros_like(ref)  # sum of |w y| over the experts: each y is off by 2^-8
    w = torch.softmax(torch.gather(lg, 1, ids), 1)
    for k in range(4):
        for t in range(T):
            e = int(ids[t, k])
            g, u = inp["x"][t].double() @ inp["w_gate"][e].double(), inp["x"][t].double() @ inp["w_up"][e].double()
            parts[t] += w[t, k] * ((g * torch.sigmoid(g) * u) @ inp["w_down"][e].double()).abs()
    ok = settled(lg, 4)
    assert (((out.double() - full.double()).abs() <= 2 * tol + BF16 * 1.01 * parts) | ~ok.unsqueeze(1)).all()


def test_weights_beyond_32_bit_offsets(cuda_lib):
    tdr = cuda_lib
    d, n, E = 4096, 4160, 132  # 2.25e9 values a matrix
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    inp = dict(x=torch.empty(3, d, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g))
    for name, shape in (("w_gate", (E, d, n)), ("w_up", (E, d, n)), ("w_down", (E, n, d))):
        inp[name] = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        for e in (0, 1, E // 2, E - 2, E - 1):
            inp[name][e].normal_(0, 0.015, generator=g)
    lg = torch.full((3, E), -30.0, device="cuda")
    lg[0, [E - 1, 0]] = torch.tensor([1.0, 0.5], device="cuda")
    lg[1, [E - 2, E // 2]] = torch.tensor([0.5, 1.0], device="cuda")
    lg[2, [E - 1, 1]] = torch.tensor([0.0, 1.0], device="cuda")
    inp["w_r"], inp["bias"] = torch.zeros(d, E, dtype=torch.bfloat16, device="cuda"), None
    s = tdr.make_shape(3, d, E, 2, n)
    out, _ = tdr.decode(s, inp["x"], None, inp["w_gate"], inp["w_up"], inp["w_down"], logits_in=lg)
    ref, tol = layer64(inp, lg.double(), 2)
    assert ((out.double() - ref).abs() <= tol).all()


def test_nothing_to_do_and_refusals(cuda_lib):
    tdr = cuda_lib
    inp = make(4, 256, 8, 2, 128, seed=1)
    w = (inp["w_r"], inp["w_gate"], inp["w_up"], inp["w_down"])
    z = tdr.make_shape(0, 256, 8, 2, 128)
    out, _ = tdr.decode(z, inp["x"][:0], *w)
    assert out.shape == (0, 256)
    s = tdr.make_shape(4, 256, 8, 2, 128)
    for kw in (dict(out=torch.empty(4, 256, device="cuda")),
               dict(out=torch.empty(4, 512, dtype=torch.bfloat16, device="cuda")[:, ::2]),
               dict(logits_in=torch.zeros(4, 9, device="cuda")),
               dict(bias=torch.zeros(8, dtype=torch.bfloat16, device="cuda")),
               dict(bias=torch.zeros(8))):
        with pytest.raises(ValueError):
            tdr.decode(s, inp["x"], *w, **kw)
    with pytest.raises(tdr.MoEError):
        tdr.decode(s, inp["x"], *w, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    odd = torch.empty(4 * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 256)
    with pytest.raises(tdr.MoEError):
        tdr.decode(s, odd, *w)
    with pytest.raises(tdr.MoEError):
        tdr.decode(tdr.make_shape(129, 256, 8, 2, 128), inp["x"], *w)
    assert tdr.device_status() == 0
