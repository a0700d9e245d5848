"""moe_adapter_forward and moe_adapter_backward where inputs are infinite or end in few bits: which
outputs are NaN, +inf and -inf is what the definition in 64 bits says, whatever the number of rows
(few rows add the adapter term in fp32, more rows take it through the tensor cores in bf16 terms)."""
import pytest
import torch

from test_gpu_adapter import backward, call_forward, low64, make

pytestmark = pytest.mark.gpu


def classes(v):
    """0 finite, 1 +inf, 2 -inf, 3 NaN."""
    return torch.where(v.isnan(), 3, torch.where(v.isinf(), torch.where(v > 0, 1, 2), 0))


def settled(v, err):
    """Values whose sign does not hang on a rounding (err 0: sums of zeros)."""
    return (v.abs() > err) | (err == 0) | ~v.isfinite()


def definition(inp, low):
    """y, its low, d_x, d_a, d_b in 64 bits (low: what the backward is given); and which values of
    low and d_low have a certain sign."""
    x, d_y, w, a, b = (inp[k].double() for k in ("x", "d_y", "w", "a", "b"))
    lref, lerr = low64(x, a, inp["ids"], inp["scale"])
    dl, dlerr = low64(d_y, b.transpose(1, 2), inp["ids"], inp["scale"])
    y, d_x = x @ w, d_y @ w.t()
    d_a, d_b = torch.zeros_like(a), torch.zeros_like(b)
    for l in range(a.shape[0]):
        t = (inp["ids"] == l).nonzero().squeeze(1)
        y[t] += lref[t] @ b[l]
        d_x[t] += dl[t] @ a[l].t()
        d_a[l] = x[t].t() @ dl[t]
        d_b[l] = low[t].double().t() @ d_y[t]
    return y, lref, d_x, d_a, d_b, settled(lref, lerr), settled(dl, dlerr)


def compare(tdr, inp):
    s, (y, low, _) = call_forward(tdr, inp)
    ry, rlow, rx, ra, rb, sure, dsure = definition(inp, low)
    d_x, d_a, d_b = backward(tdr, s, inp, low)
    assert tdr.device_status() == 0
    assert torch.equal(classes(low)[sure], classes(rlow)[sure])
    rows, drows = sure.all(1), dsure.all(1)
    assert rows.double().mean() >= 0.6 and drows.double().mean() >= 0.6
    assert torch.equal(classes(y)[rows], classes(ry)[rows])
    assert torch.equal(classes(d_x)[drows], classes(rx)[drows])
    for l in range(d_a.shape[0]):
        cols = dsure[inp["ids"] == l].all(0)
        assert torch.equal(classes(d_a[l])[:, cols], classes(ra[l])[:, cols]), l
        assert torch.equal(classes(d_b[l]), classes(rb[l])), l
    return ry, rx, ra, rb


SIZES = [(5, 24), (24, 80), (300, 8), (300, 72), (1000, 24)]  # the first two: few rows forward


@pytest.mark.parametrize("T,r", SIZES)
@pytest.mark.parametrize("name,sign", [("a", 1), ("a", -1), ("b", 1), ("b", -1)])
def test_an_infinity_in_an_adapter(cuda_lib, T, r, name, sign):
    inp = make(T, 512, 704, 5, r, T + r)
    inp["ids"][:5] = torch.arange(5, device="cuda").int()
    for l in range(4):  # one element each
        inp[name][l, (7 * l + 3) % inp[name].shape[1], (5 * l + 1) % inp[name].shape[2]] = \
            sign * torch.inf
    ry, rx, ra, rb = compare(cuda_lib, inp)
    assert ry.isinf().any() and rx.isinf().any()


@pytest.mark.parametrize("T,r", SIZES)
@pytest.mark.parametrize("sign", [1, -1])
def test_an_infinity_in_a_row(cuda_lib, T, r, sign):
    inp = make(T, 512, 704, 5, r, T + r)
    inp["ids"][:5] = torch.tensor([4, 2, 0, 1, -1], device="cuda").int()
    inp["x"][0, 100] = sign * torch.inf
    inp["d_y"][1, 37] = sign * torch.inf
    inp["x"][4, 5] = -sign * torch.inf  # a row without an adapter
    ry, rx, ra, rb = compare(cuda_lib, inp)
    assert ra[4].isinf().any() and rb[2].isinf().any()


@pytest.mark.parametrize("T,r", SIZES)
def test_low_rank_values_that_bf16_holds_beside_infinities(cuda_lib, T, r):
    """Rows that pick one row of A (or column of B) make low-rank values of few bits: none of their
    terms may be a zero that meets an infinity."""
    inp = make(T, 512, 704, 5, r, T + r)
    inp["ids"][:5] = torch.tensor([1, 2, 3, 0, -1], device="cuda").int()
    inp["scale"][:] = 1.0
    inp["x"][:4] = 0
    inp["d_y"][:4] = 0
    for t in range(4):
        inp["x"][t, 11 * t] = 1.0
        inp["d_y"][t, 13 * t] = -2.0
    inp["a"][:, :, 0] = inp["a"][:, :, 0].abs() + 0.5
    inp["b"][:, 0, :] = inp["b"][:, 0, :].abs() + 0.5
    inp["a"][2, 7, 0] = torch.inf
    inp["b"][1, 0, 8] = -torch.inf
    inp["b"][3, 0, 700] = torch.inf
    inp["x"][0, 300] = torch.inf
    compare(cuda_lib, inp)


@pytest.mark.parametrize("T,r", SIZES)
def test_low_rank_values_at_the_ends_of_the_range(cuda_lib, T, r):
    """Finite values next to the largest stay finite, and a value of any size keeps its bits: a
    power of two times the adapter scales low, d_low and what comes of them by that power."""
    tdr = cuda_lib
    inp = make(T, 512, 704, 5, r, T + r)
    inp["w"][:] = 0  # the adapter term alone
    s, (y, low, _) = call_forward(tdr, inp)
    grads = backward(tdr, s, inp, low)
    for p in (-60, 60):
        big = dict(inp, scale=inp["scale"] * 2.0 ** p)
        _, (y2, low2, _) = call_forward(tdr, big)
        assert torch.equal(low2, low * 2.0 ** p) and torch.equal(y2, y * 2.0 ** p)
        g2 = backward(tdr, s, big, low2)
        for got, want in zip(g2, grads):
            assert torch.equal(got, want * 2.0 ** p)
    top = torch.full_like(low, 3.4e38)  # rounded to bf16 it would be an infinity
    inp["d_y"][:] = 0
    inp["d_y"][:, 0] = 2.0 ** -20
    inp["ids"][:] = torch.arange(T, device="cuda").int() % 5
    _, d_a, d_b = backward(tdr, s, inp, top)
    assert d_b.isfinite().all()
    want = top[0, 0].double() * 2.0 ** -20 * torch.bincount(inp["ids"].long(), minlength=5).double()
    assert ((d_b[:, :, 0].double() - want[:, None]).abs() <= want[:, None] * T * 2.0 ** -23).all()
