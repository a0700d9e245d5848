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


def backward(tdr, s, inp, low, **kw):
    return tdr.adapter_backward(s, inp["d_y"], inp["x"], inp["w"], inp["a"], inp["b"], inp["ids"],
                                inp["scale"], low, **kw)


@pytest.mark.parametrize("T", [5, 128, 300, 1000])
def test_a_broken_adapter_or_row_stays_alone(cuda_lib, T):
    """NaN and infinity in one adapter, or one row, reach its own rows and gradients only."""
    tdr = cuda_lib
    d_in, d_out, L, r = 512, 704, 7, 24
    inp = make(T, d_in, d_out, L, r, T)
    s, (y, low, _) = call_forward(tdr, inp)
    d_x, d_a, d_b = backward(tdr, s, inp, low)
    ids = inp["ids"]
    for l, name, value in ((0, "a", torch.nan), (L - 1, "b", torch.inf), (3, "b", torch.nan)):
        sick = dict(inp, **{name: inp[name].clone()})
        sick[name][l] = value
        _, (y2, low2, _) = call_forward(tdr, sick)
        own = ids == l
        assert torch.equal(y2[~own], y[~own]) and not y2[own].isfinite().any()
        x2, a2, b2 = backward(tdr, s, sick, low)
        assert torch.equal(x2[~own], d_x[~own]) and not x2[own].isfinite().any()
        keep = torch.arange(L, device="cuda") != l
        assert torch.equal(a2[keep], d_a[keep]) and torch.equal(b2, d_b)
    t = int((ids >= 0).nonzero()[0, 0])
    sick = dict(inp, x=inp["x"].clone(), d_y=inp["d_y"].clone())
    sick["x"][t], sick["d_y"][t] = torch.nan, torch.inf
    _, (y2, low2, _) = call_forward(tdr, sick)
    rest = torch.arange(T, device="cuda") != t
    assert torch.equal(y2[rest], y[rest]) and torch.equal(low2[rest], low[rest])
    assert y2[t].isnan().all()
    x2, a2, b2 = backward(tdr, s, sick, low)
    assert torch.equal(x2[rest], d_x[rest]) and not x2[t].isfinite().any()
    keep = torch.arange(L, device="cuda") != ids[t]
    assert torch.equal(a2[keep], d_a[keep]) and torch.equal(b2[keep], d_b[keep])


@pytest.mark.parametrize("T", [1, 77, 129, 2500])
def test_workspace_outputs_and_repetition(cuda_lib, T):
    tdr = cuda_lib
    inp = make(T, 576, 320, 9, 16, T, "runs")
    s, (y, low, _) = call_forward(tdr, inp)
    grads = backward(tdr, s, inp, low)
    ws = torch.full((tdr.adapter_workspace_size(s),), 255, dtype=torch.uint8, device="cuda")  # NaN
    whole = torch.full((T + 2, 320), 3.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(4):
        y2, low2, _ = call_forward(tdr, inp, workspace=ws, out=whole[1:T + 1])[1]
        assert torch.equal(y2, y) and torch.equal(low2, low)
        for p, q in zip(backward(tdr, s, inp, low, workspace=ws), grads):
            assert torch.equal(p, q)
        ws.fill_(255)
    assert (whole[0] == 3).all() and (whole[T + 1] == 3).all()
    d_x, d_a, d_b = backward(tdr, s, inp, low, want_d_x=False)
    assert d_x is None and torch.equal(d_a, grads[1]) and torch.equal(d_b, grads[2])
    assert tdr.device_status() == 0


@pytest.mark.parametrize("T", [100, 400])
def test_ids_out_of_range_count_as_none_and_are_reported(cuda_lib, T):
    tdr = cuda_lib
    inp = make(T, 128, 128, 4, 8, 1)
    none = dict(inp, ids=inp["ids"].clone())
    none["ids"][[3, 50]] = -1
    _, (y, low, _) = call_forward(tdr, none)
    assert tdr.device_status() == 0
    sick = dict(inp, ids=none["ids"].clone())
    sick["ids"][3], sick["ids"][50] = 4, -2
    _, (y2, low2, _) = call_forward(tdr, sick)
    assert tdr.device_status() == 6
    assert torch.equal(y2, y) and torch.equal(low2, low)


def test_streams_and_graphs(cuda_lib):
    tdr = cuda_lib
    sets = [make(T, 512, 448, 6, 16, T, "runs") for T in (9, 200, 1500)]
    ref = []
    for i in sets:
        s, (y, low, _) = call_forward(tdr, i)
        ref.append((s, y, low, backward(tdr, s, i, low)))
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        for st, i in zip(streams, sets):
            with torch.cuda.stream(st):
                s, (y, low, _) = call_forward(tdr, i)
                outs.append((y, low, backward(tdr, s, i, low)))
    torch.cuda.synchronize()
    for k, (y, low, grads) in enumerate(outs):
        _, ry, rlow, rg = ref[k % 3]
        assert torch.equal(y, ry) and torch.equal(low, rlow)
        assert all(torch.equal(p, q) for p, q in zip(grads, rg))
    ws = torch.empty(max(tdr.adapter_workspace_size(r[0]) for r in ref), dtype=torch.uint8,
                     device="cuda")
    graphs = []
    for i in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s, (y, low, _) = call_forward(tdr, i, workspace=ws)
            graphs.append((g, y, low, backward(tdr, s, i, low, workspace=ws)))
    for _ in range(3):
        for (g, y, low, grads), (_, ry, rlow, rg) in zip(graphs, ref):
            g.replay()
            assert torch.equal(y, ry) and torch.equal(low, rlow)
            assert all(torch.equal(p, q) for p, q in zip(grads, rg))
    assert tdr.device_status() == 0


def test_gradients_against_differences(cuda_lib):
    """<d, grad> against (f(v + h d) - f(v - h d)) / 2h of f = <y, d_y>, in 64 bits: f is linear in
    x, A and B each, so the difference is exact but for the outputs' rounding of f itself; the
    gradients are held to the bounds that their definition tests derive, summed over d."""
    tdr = cuda_lib
    T, d_in, d_out, L, r = 260, 192, 128, 3, 8
    inp = make(T, d_in, d_out, L, r, 4)
    s, (_, low, _) = call_forward(tdr, inp)
    d_x, d_a, d_b = backward(tdr, s, inp, low)
    v = {k: inp[k].double() for k in ("x", "w", "a", "b", "d_y")}

    def f(x, a, b):
        y = x @ v["w"]
        for l in range(L):
            t = (inp["ids"] == l).nonzero().squeeze(1)
            y[t] += inp["scale"][l].double() * (x[t] @ a[l]) @ b[l]
        return (y * v["d_y"]).sum()

    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    for k, grad, rel in (("x", d_x, BF16), ("a", d_a, 2.0 ** -12), ("b", d_b, 2.0 ** -12)):
        for _ in range(3):
            d = torch.empty_like(v[k]).normal_(0, 1, generator=g)
            at = dict(x=v["x"], a=v["a"], b=v["b"])
            up, down = dict(at, **{k: v[k] + d}), dict(at, **{k: v[k] - d})
            want = (f(**up) - f(**down)) / 2
            got = (grad.double() * d).sum()
            assert (got - want).abs() <= rel * (grad.double() * d).abs().sum() + 1e-9, k


def test_rows_beyond_32_bit_offsets(cuda_lib):
    tdr = cuda_lib
    T, d_in, d_out, L, r = 540672, 4096, 64, 5, 8  # 2.2e9 values of x
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.empty(T, d_in, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g)
    inp = make(2, d_in, d_out, L, r, 2)
    inp["x"] = x
    inp["ids"] = torch.randint(-1, L, (T,), generator=g, device="cuda").int()
    inp["d_y"] = torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda").normal_(0, 0.1, generator=g)
    s, (y, low, _) = call_forward(tdr, inp)
    d_x, d_a, d_b = backward(tdr, s, inp, low)
    assert tdr.device_status() == 0
    at = torch.cat([torch.arange(40), torch.arange(T // 2, T // 2 + 40), torch.arange(T - 300, T)]).cuda()
    xs, ds, ids = x[at].double(), inp["d_y"][at].double(), inp["ids"][at]
    w, a, b = (inp[k].double() for k in ("w", "a", "b"))
    lref, lerr = low64(xs, a, ids, inp["scale"])
    assert ((low[at].double() - lref).abs() <= lerr).all()
    ref, err = through64(xs, w, lref, lerr, b, ids)
    assert ((y[at].double() - ref).abs() <= err).all()
    dl, dlerr = low64(ds, b.transpose(1, 2), ids, inp["scale"])
    ref, err = through64(ds, w.t(), dl, dlerr, a.transpose(1, 2), ids)
    assert ((d_x[at].double() - ref).abs() <= err).all()
    for l in (0, L - 1):  # the sums over all rows, a slice of the columns
        t = (inp["ids"] == l).nonzero().squeeze(1)
        dy, xc = inp["d_y"][t].double(), x[t, -64:].double()
        dl = inp["scale"][l].double() * (dy @ b[l].t())
        n = t.numel() + 72
        assert ((d_a[l, -64:].double() - xc.t() @ dl).abs() <= n * F32 * (xc.abs().t() @ dl.abs())).all()
        lw = low[t].double()
        assert ((d_b[l].double() - lw.t() @ dy).abs() <= n * F32 * (lw.abs().t() @ dy.abs())).all()


def test_nothing_to_do_and_refusals(cuda_lib):
    tdr = cuda_lib
    inp = make(6, 128, 192, 3, 8, 1)
    z = tdr.make_adapter_shape(0, 128, 192, 3, 8)
    y, low, _ = tdr.adapter_forward(z, inp["x"][:0], inp["w"], inp["a"], inp["b"], inp["ids"][:0],
                                    inp["scale"])
    assert y.shape == (0, 192) and low.shape == (0, 8)
    d_a = torch.ones(3, 128, 8, device="cuda")
    _, d_a, d_b = tdr.adapter_backward(z, inp["d_y"][:0], inp["x"][:0], inp["w"], inp["a"], inp["b"],
                                       inp["ids"][:0], inp["scale"], low, d_a=d_a)
    assert (d_a == 0).all() and (d_b == 0).all()
    s = tdr.make_adapter_shape(6, 128, 192, 3, 8)
    names = ("x", "w", "a", "b", "ids", "scale")
    for key, value in (("ids", inp["ids"].long()), ("scale", inp["scale"].double()),
                       ("a", inp["a"].float()), ("b", inp["b"].transpose(1, 2)),
                       ("w", inp["w"].cpu()), ("w", inp["w"].t()), ("x", inp["x"][:5])):
        sick = dict(inp, **{key: value})
        with pytest.raises((TypeError, ValueError)):
            tdr.adapter_forward(s, *[sick[k] for k in names])
        with pytest.raises((TypeError, ValueError)):
            tdr.adapter_backward(s, inp["d_y"], *[sick[k] for k in names], low=torch.zeros_like(low))
    _, (y, low, _) = call_forward(tdr, inp)
    with pytest.raises((TypeError, ValueError)):
        backward(tdr, s, inp, low.cpu())
    with pytest.raises(ValueError):
        backward(tdr, s, inp, low, d_x=torch.empty_like(inp["x"]), want_d_x=False)
    with pytest.raises(tdr.MoEError):
        call_forward(tdr, inp, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tdr.MoEError):
        backward(tdr, s, inp, low, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    for bad in (tdr.make_adapter_shape(6, 100, 192, 3, 8), tdr.make_adapter_shape(6, 128, 192, 3, 12),
                tdr.make_adapter_shape(6, 128, 192, 3, 136), tdr.make_adapter_shape(6, 128, 192, 257, 8),
                tdr.make_adapter_shape(6, 128, 192, 3, 8, torch.float32)):
        with pytest.raises(tdr.MoEError):
            tdr.adapter_forward(bad, *[inp[k] for k in names])
    assert tdr.device_status() == 0


def test_a_decode_step_and_a_tuning_step(cuda_lib):
    """The calls as a program makes them: projection with adapters, then the layer; and the
    gradient of a loss through the layer into the adapters."""
    tdr = cuda_lib
    T, d, L, r, E, K, n = 48, 512, 5, 16, 16, 4, 384
    inp = make(T, 256, d, L, r, 3)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def normal(*shape, std):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)

    w_r, wg, wu = normal(d, E, std=0.05), normal(E, d, n, std=0.05), normal(E, d, n, std=0.05)
    wd = normal(E, n, d, std=0.05)
    s, (h, low, _) = call_forward(tdr, inp)
    layer = tdr.make_shape(T, d, E, K, n)
    out, _ = tdr.decode(layer, h, w_r, wg, wu, wd)
    full, ws, pre = tdr.forward_h(layer, h, w_r, wg, wu, wd)
    # two expert outputs' roundings apart, of the size of the row
    assert ((out.float() - full.float()).norm() / full.float().norm()) < 2 ** -6
    # captured: the same values on replay
    graph = torch.cuda.CUDAGraph()
    a_ws = torch.empty(tdr.adapter_workspace_size(s), dtype=torch.uint8, device="cuda")
    d_ws = torch.empty(tdr.decode_workspace_size(layer), dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        h2, _, _ = call_forward(tdr, inp, workspace=a_ws)[1]
        out2, _ = tdr.decode(layer, h2, w_r, wg, wu, wd, workspace=d_ws)
    graph.replay()
    assert torch.equal(out2, out)
    # tuning: d_out -> layer -> projection
    v = tdr.workspace_views(layer, ws)
    d_out = normal(T, d, std=0.1)
    d_h, d_w, d_in = tdr.backward(layer, d_out, v["topk_w"], v["offsets"], v["perm_to_assign"],
                                  v["assign_to_perm"], wd, pre, wg, wu, input_grad=True)
    tdr.backward_router(layer, h, w_r, v["topk_ids"], v["topk_w"], d_w, d_x=d_in)
    d_x, d_a, d_b = backward(tdr, s, dict(inp, d_y=d_in), low)
    assert tdr.device_status() == 0
    # autograd of the same chain in 64 bits, the layer's selection held fixed
    x, a, b = (inp[k].double().requires_grad_() for k in ("x", "a", "b"))
    parts = [x @ inp["w"].double()]
    for l in range(L):
        own = (inp["ids"] == l).double().unsqueeze(1)
        parts.append(own * inp["scale"][l].double() * ((x @ a[l]) @ b[l]))
    hh = sum(parts)
    ids = v["topk_ids"].long()
    wt = torch.softmax((hh @ w_r.double()).gather(1, ids), 1)
    y = torch.zeros_like(hh)
    for e in range(E):
        up, gate = hh @ wu[e].double(), hh @ wg[e].double()
        ye = (torch.nn.functional.silu(gate) * up) @ wd[e].double()
        y = y + ((ids == e) * wt).sum(1, keepdim=True) * ye
    (y * d_out.double()).sum().backward()
    for got, want in ((d_x, x.grad), (d_a, a.grad), (d_b, b.grad)):
        # bf16 roundings of h, the activations and the layer's input gradient: a few 2^-8
        assert ((got.double() - want).norm() / want.norm()) < 6 * BF16


def test_many_calls_on_several_streams(cuda_lib):
    """CTAs of several calls share SMs and their tensor memory, in pieces of several sizes: no call
    may hold some of it while it waits for another call, and results stay what they are alone."""
    tdr = cuda_lib
    shapes = [(300, 1024, 768, 4, 8), (513, 2048, 1024, 8, 64), (700, 256, 512, 6, 128),
              (2049, 960, 1024, 48, 24), (57, 1024, 960, 32, 16), (1500, 512, 512, 3, 16)]
    sets, ref = [], []
    for shape in shapes:
        inp = make(*shape, shape[0], "runs")
        s, (y, low, ws) = call_forward(tdr, inp)
        sets.append((s, inp, low, [torch.empty_like(ws) for _ in range(4)]))
        ref.append([t.clone() for t in (y, *backward(tdr, s, inp, low))])
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for turn in range(40):
        got = []
        for i in range(24):
            k, j = (7 * i + turn) % len(sets), i % 4
            s, inp, low, ws = sets[k]
            with torch.cuda.stream(streams[j]):
                y = call_forward(tdr, inp, workspace=ws[j])[1][0]
                g = backward(tdr, s, inp, low, workspace=ws[j], want_d_x=(i + turn) % 3 > 0)
                got.append((k, (y, *g)))
        torch.cuda.synchronize()
        for k, outs in got:
            for a, b in zip(outs, ref[k]):
                if a is not None:
                    wrong += (a != b).any()
        torch.cuda.synchronize()
    assert wrong.item() == 0 and tdr.device_status() == 0
