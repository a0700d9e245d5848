"""Adapter calls beside kernels that take tensor memory before they wait for the kernel before
them: behind the gradients in one stream, and on several streams at once."""
import pytest
import torch

from test_gpu_adapter import backward, call_forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("r", [16, 64, 72, 128])  # above 64 the gradients take all of it
def test_a_router_behind_the_gradients(cuda_lib, r):
    tdr = cuda_lib
    inp = make(300, 512, 448, 6, r, r, "runs")  # no partial sums: the gradients come last
    s, (_, low, ws) = call_forward(tdr, inp)
    x = make(1024, 256, 64, 1, 8, 1)["x"]
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    w_row, w_col = (torch.empty(256, n, dtype=torch.bfloat16, device="cuda").normal_(0, 0.1, generator=g)
                    for n in (24, 40))
    o = tdr.make_omni_shape(1024, 256, 24, 40, 8)
    ref = [*backward(tdr, s, inp, low), *tdr.omni_route(o, x, w_row, w_col)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    spaces = [torch.empty(tdr.adapter_workspace_size(s), dtype=torch.uint8, device="cuda")
              for _ in streams]
    torch.cuda.synchronize()
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(40):
        got = []
        for _ in range(5):
            for st, w in zip(streams, spaces):
                with torch.cuda.stream(st):
                    got.append([*backward(tdr, s, inp, low, workspace=w),
                                *tdr.omni_route(o, x, w_row, w_col)])
        torch.cuda.synchronize()
        for outs in got:
            for p, q in zip(outs, ref):
                wrong += (p != q).any()
        torch.cuda.synchronize()
    assert wrong.item() == 0 and tdr.device_status() == 0
