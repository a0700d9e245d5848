"""Adapter calls at sizes where the kernels' own choices change: clusters, CTAs an SM, whole and cut
tiles in one call. Against the definition in 64 bits, as in test_gpu_adapter.py."""
import pytest
import torch

from test_gpu_adapter import F32, backward, call_forward, low64, make, through64

pytestmark = pytest.mark.gpu


def check_forward(tdr, inp):
    _, (y, low, _) = call_forward(tdr, inp)
    assert tdr.device_status() == 0
    x, w, a, b = (inp[k].double() for k in ("x", "w", "a", "b"))
    lref, lerr = low64(x, a, inp["ids"], inp["scale"])
    assert ((low.double() - lref).abs() <= lerr).all()
    ref, err = through64(x, w, lref, lerr, b, inp["ids"])
    bad = (y.double() - ref).abs() > err
    assert not bad.any(), (bad.sum().item(), ((y.double() - ref).abs() / err).max().item())


@pytest.mark.parametrize("T,d_in,d_out,L,r", [
    (64, 512, 32768, 24, 80), (40, 192, 20480, 30, 128), (71, 1088, 8448, 5, 32),
    (70, 1024, 16896, 5, 32), (66, 1024, 16384, 8, 8), (33, 2048, 2880, 8, 72), (128, 64, 320, 30, 40),
    (127, 576, 17024, 9, 8), (128, 256, 192, 128, 128), (128, 2048, 1024, 128, 64),
    (100, 1024, 640, 256, 120),
])
def test_few_rows_through_wide_projections(cuda_lib, T, d_in, d_out, L, r):
    """Around the sizes where two CTAs no longer fit an SM, clusters shrink, tiles outnumber SMs."""
    check_forward(cuda_lib, make(T, d_in, d_out, L, r, T + r))


def check_backward(tdr, inp):
    x, d_y, w, a, b = (inp[k].double() for k in ("x", "d_y", "w", "a", "b"))
    low = low64(x, a, inp["ids"], inp["scale"])[0].float()
    s = tdr.make_adapter_shape(*inp["x"].shape, *(inp["b"].shape[i] for i in (2, 0, 1)))
    d_x, d_a, d_b = backward(tdr, s, inp, low)
    assert tdr.device_status() == 0
    dl, dlerr = low64(d_y, b.transpose(1, 2), inp["ids"], inp["scale"])
    ref, err = through64(d_y, w.t(), dl, dlerr, a.transpose(1, 2), inp["ids"])
    assert ((d_x.double() - ref).abs() <= err).all()
    for l in range(a.shape[0]):
        t = (inp["ids"] == l).nonzero().squeeze(1)
        n = t.numel() + 8
        ea = x[t].abs().t() @ (dlerr[t] + n * F32 * dl[t].abs())
        eb = n * F32 * (low[t].double().abs().t() @ d_y[t].abs())
        assert ((d_a[l].double() - x[t].t() @ dl[t]).abs() <= ea).all(), l
        assert ((d_b[l].double() - low[t].double().t() @ d_y[t]).abs() <= eb).all(), l


@pytest.mark.parametrize("T,wide,narrow,L,r", [
    (2049, 2880, 2880, 7, 24),  # 256 x 256 tiles: 9 x 12, 34 more than pairs of SMs; one row in the last
    (2600, 2880, 1856, 5, 16),  # 11 x 8, 14 more, cut in five; ragged both ways
    (4000, 2624, 1280, 9, 72),  # 16 x 5, 6 more, cut in eight
    (5000, 2880, 1984, 4, 8),   # 20 x 8: two whole rounds, 12 more
])
def test_whole_and_cut_tiles_in_one_call(cuda_lib, T, wide, narrow, L, r):
    """Tiles beyond a whole number of rounds are cut along the contraction and added by another
    kernel, where the contraction is long: `wide` forward, and again backward."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    tiles = -(-T // 256) * -(-narrow // 256)
    assert tiles > pairs and 2 <= pairs // (tiles % pairs), "sizes for 148 SMs"
    check_forward(cuda_lib, make(T, wide, narrow, L, r, T + r, "mixed"))
    check_backward(cuda_lib, make(T, narrow, wide, L, r, T + r + 1, "runs"))


@pytest.mark.parametrize("T", [20, 260, 600])
def test_gradients_against_differences_one_value_at_a_time(cuda_lib, T):
    """(f(v + e) - f(v - e)) / 2 of f = <y, d_y> for single elements e of x, A and B, in 64 bits (f is
    linear in each, so that it is the derivative but for the sums' rounding, below 1e-9). The bound
    is that of the element's own sums, from magnitudes in 64 bits."""
    tdr = cuda_lib
    d_in, d_out, L, r = 192, 128, 3, 8
    inp = make(T, d_in, d_out, L, r, T)
    s, (_, low, _) = call_forward(tdr, inp)
    grads = dict(zip(("x", "a", "b"), backward(tdr, s, inp, low)))
    v = {k: inp[k].double() for k in ("x", "w", "a", "b", "d_y")}
    own = [(inp["ids"] == l).nonzero().squeeze(1) for l in range(L)]

    def f(x, a, b):
        y = x @ v["w"]
        for l in range(L):
            y[own[l]] += inp["scale"][l].double() * (x[own[l]] @ a[l]) @ b[l]
        return (y * v["d_y"]).sum()

    dl, dlerr = low64(v["d_y"], v["b"].transpose(1, 2), inp["ids"], inp["scale"])
    lref, lerr = low64(v["x"], v["a"], inp["ids"], inp["scale"])
    _, ex = through64(v["d_y"], v["w"].t(), dl, dlerr, v["a"].transpose(1, 2), inp["ids"])
    ea, eb = torch.zeros_like(v["a"]), torch.zeros_like(v["b"])
    for l, t in enumerate(own):
        n = t.numel() + 8
        ea[l] = v["x"][t].abs().t() @ (dlerr[t] + n * F32 * dl[t].abs())
        eb[l] = (lerr[t] + n * F32 * (lref[t].abs() + lerr[t])).t() @ v["d_y"][t].abs()
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    for k, err in (("x", ex), ("a", ea), ("b", eb)):
        assert err.max() < 0.05 * grads[k].abs().max()  # a bound that can be missed
        for i in torch.randperm(v[k].numel(), generator=g, device="cuda")[:40].tolist():
            e = torch.zeros_like(v[k])
            e.view(-1)[i] = 1.0
            at = dict(x=v["x"], a=v["a"], b=v["b"])
            want = (f(**dict(at, **{k: v[k] + e})) - f(**dict(at, **{k: v[k] - e}))) / 2
            assert (grads[k].view(-1)[i].double() - want).abs() <= err.view(-1)[i] + 1e-9, (k, i)
