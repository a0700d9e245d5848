"""Adapter calls at sizes where the kernels' own choices change: clusters, CTAs an SM, whole and cut
tiles in one call. Against the definition in 64 bits, as in test_gpu_adapter.py."""
import pytest
import torch

from test_gpu_adapter import call_forward, low64, make, through64

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
