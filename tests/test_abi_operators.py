"""moe_decode and moe_adapter_forward / _backward on a host without a GPU: sizes are host
arithmetic, and bad arguments are refused before any CUDA call is made."""
import ctypes

import pytest
import torch

import token_dispatch_router_b200 as tdr

DUMMY = ctypes.c_void_p(256)  # never dereferenced: every check fails first
ODD = ctypes.c_void_p(264)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    from token_dispatch_router_b200 import build
    build.build()
    return tdr.load_library()


@pytest.mark.parametrize("kw,code", [
    (dict(T=16, d=128, E=8, K=9, n=128), 1),                       # K > E
    (dict(T=16, d=100, E=8, K=2, n=128), 1),                       # d not a multiple of 64
    (dict(T=16, d=128, E=8, K=2, n=96), 1),                        # n not a multiple of 64
    (dict(T=-1, d=128, E=8, K=2, n=128), 1),                       # negative T
    (dict(T=16, d=128, E=300, K=2, n=128), 2),                     # E > 256
    (dict(T=129, d=128, E=8, K=2, n=128), 2),                      # more tokens than one tile
    (dict(T=16, d=128, E=8, K=2, n=128, tile_round=16), 2),        # rounding of kept counts
    (dict(T=16, d=128, E=8, K=2, n=128, dtype=torch.float32), 2),
])
def test_decode_shapes_refused(lib, kw, code):
    s = tdr.make_shape(**kw)
    assert lib.moe_decode_workspace_size(ctypes.byref(s)) == 0
    assert lib.moe_decode(ctypes.byref(s), *[DUMMY] * 9, BIG, None) == code
    with pytest.raises(tdr.MoEError):
        tdr.decode(s, None, None, None, None, None)


def test_decode_arguments_refused(lib):
    s = tdr.make_shape(16, 128, 8, 2, 128)
    need = lib.moe_decode_workspace_size(ctypes.byref(s))
    assert need > 0
    names = ("x", "w_r", "bias", "logits_in", "w_gate", "w_up", "w_down", "out", "workspace")

    def call(size=BIG, **kw):
        args = dict({k: DUMMY for k in names}, bias=None, logits_in=None)
        args.update(kw)
        return lib.moe_decode(ctypes.byref(s), *[args[k] for k in names], size, None)

    for k in ("x", "w_r", "w_gate", "w_up", "w_down", "out"):
        assert call(**{k: None}) == 1, k
        assert call(**{k: ODD}) == 1, k
    assert call(workspace=None) == 4 and call(need - 1) == 4
    assert call(workspace=ODD) == 1
    assert lib.moe_decode(None, *[DUMMY] * 9, BIG, None) == 1
    none = tdr.make_shape(0, 128, 8, 2, 128)  # no tokens: nothing to check or run
    assert lib.moe_decode(ctypes.byref(none), *[None] * 9, 0, None) == 0


@pytest.mark.parametrize("args,code", [
    ((-1, 128, 128, 1, 8), 1), ((16, 0, 128, 1, 8), 1), ((16, 128, 96, 1, 8), 1),
    ((16, 100, 128, 1, 8), 1), ((16, 128, 128, 0, 8), 1), ((16, 128, 128, 1, 0), 1),
    ((16, 128, 128, 1, 12), 1), ((16, 128, 128, 1, 136), 2), ((16, 128, 128, 257, 8), 2),
    (((1 << 24) + 1, 128, 128, 1, 8), 2), ((16, 128, 128, 1, 8, None), 2),
])
def test_adapter_shapes_refused(lib, args, code):
    s = tdr.make_adapter_shape(*args)
    assert lib.moe_adapter_workspace_size(ctypes.byref(s)) == 0
    assert lib.moe_adapter_forward(ctypes.byref(s), *[DUMMY] * 9, BIG, None) == code
    assert lib.moe_adapter_backward(ctypes.byref(s), *[DUMMY] * 12, BIG, None) == code
    with pytest.raises(tdr.MoEError):
        tdr.adapter_forward(s, None, None, None, None, None, None)


@pytest.mark.parametrize("T", [1, 128, 129, 1 << 24])
def test_adapter_arguments_refused(lib, T):
    s = tdr.make_adapter_shape(T, 128, 192, 4, 16)
    assert lib.moe_adapter_workspace_size(ctypes.byref(s)) > 0
    fwd = ("x", "w", "a", "b", "ids", "scale", "low", "y", "workspace")
    bwd = ("d_y", "x", "w", "a", "b", "ids", "scale", "low", "d_x", "d_a", "d_b", "workspace")
    for f, names in ((lib.moe_adapter_forward, fwd), (lib.moe_adapter_backward, bwd)):
        def call(size=BIG, **kw):
            args = {k: DUMMY for k in names}
            args.update(kw)
            return f(ctypes.byref(s), *[args[k] for k in names], size, None)

        for k in names[:-1]:
            if k != "d_x":  # may be left out
                assert call(**{k: None}) == 1, k
            if k not in ("ids", "scale"):
                assert call(**{k: ODD}) == 1, k
        assert call(workspace=None) == 4 and call(0) == 4
        assert call(workspace=ODD) == 1
        assert f(None, *[DUMMY] * len(names), BIG, None) == 1


def test_workspaces_grow_with_the_rows(lib):
    sizes = [tdr.adapter_workspace_size(tdr.make_adapter_shape(T, 2048, 2880, 32, 16))
             for T in (0, 1, 128, 129, 4096, 1 << 20, 1 << 24)]
    assert all(p > 0 for p in sizes) and sizes == sorted(sizes)
    sizes = [tdr.decode_workspace_size(tdr.make_shape(T, 2048, 64, 8, 1024)) for T in (0, 1, 8, 128)]
    assert all(p > 0 for p in sizes) and sizes == sorted(sizes)


def test_the_table_of_tiles_has_room_for_the_adapters_there_are(lib):
    """A 256-row tile lists at most n_adapters of them, 36 bytes each: 2^24 rows of one adapter do
    without 255 of 256 in 65536 tiles."""
    def size(n):
        return tdr.adapter_workspace_size(tdr.make_adapter_shape(1 << 24, 64, 64, n, 8))

    assert size(256) - size(1) >= 65536 * 252 * 36


def test_the_stream_of_a_call_without_torchs_own_shortcut(monkeypatch):
    """Every call passes the current stream's handle; the shortcut to it may go from torch."""
    import importlib.util
    import types

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    spec = importlib.util.spec_from_file_location("tdr_without_shortcut", tdr.__file__)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert mod._stream() == 77
