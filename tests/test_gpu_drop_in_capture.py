"""Handles that are dropped while a stream is being captured, as Python's collector may do at any time: the capture goes on. And
destruction waits for the device, as include/np.h says."""
import ctypes
import gc

import numpy as np
import pytest

from tests.harness import torch_mod

pytestmark = pytest.mark.gpu

torch = None


@pytest.fixture(autouse=True, scope="module")
def _torch():
    global torch
    torch = torch_mod()
    assert torch.cuda.is_available()


def rope():
    from delta_prefetched_ffn_amd import Rope
    return Rope(head_dim=64)


def w4(n_out=64, n_in=256):
    from delta_prefetched_ffn_amd import W4
    codes = torch.randint(0, 256, (n_out, n_in // 2), dtype=torch.uint8, device="cuda")
    scales = torch.ones((n_out, 2), device="cuda")
    return W4(n_out=n_out, n_in=n_in, group=n_in // 2, codes_ptr=codes.data_ptr(), scales_ptr=scales.data_ptr(), scale_dtype="f32")


def cache():
    from delta_prefetched_ffn_amd import KVCache, kv_bytes
    shape = dict(n_layers=1, n_heads=2, n_kv_heads=2, head_dim=64, page_tokens=16, n_pages=4)
    nc, ne = kv_bytes(**shape)
    codes, exps = torch.zeros(nc, dtype=torch.uint8, device="cuda"), torch.zeros(ne, dtype=torch.int8, device="cuda")
    return KVCache(**shape, max_seqs=2, max_pages=4, codes=codes.data_ptr(), exps=exps.data_ptr(), keepalive=(codes, exps))


def layer():
    from delta_prefetched_ffn_amd import MASK_UNION, Layer
    d, m, k, r = 256, 1024, 512, 3
    store = torch.zeros((m, r, d), dtype=torch.bfloat16, device="cuda")
    return Layer(d_model=d, d_ff=m, k_max=k, n_rows=r, masks=np.ones((2, 8, m // 64), np.uint64), mask_mode=MASK_UNION, row_store=store.data_ptr(), keepalive=store)


MAKE = {"rope": rope, "w4": w4, "cache": cache, "layer": layer}


def captured(body):
    """body(stream) captured (in the global mode, which forbids most) by the runtime's own calls, and replayed twice."""
    hip = ctypes.CDLL("libamdhip64.so.7")
    side, graph, ready = torch.cuda.Stream(), ctypes.c_void_p(), ctypes.c_void_p()
    stream = ctypes.c_void_p(side.cuda_stream)
    torch.cuda.synchronize()
    assert hip.hipStreamBeginCapture(stream, 0) == 0
    try:
        body(side.cuda_stream)
    finally:
        ended = hip.hipStreamEndCapture(stream, ctypes.byref(graph))
    assert ended == 0 and graph, ended
    assert hip.hipGraphInstantiate(ctypes.byref(ready), graph, None, None, 0) == 0
    for _ in range(2):
        assert hip.hipGraphLaunch(ready, stream) == 0
    side.synchronize()
    assert hip.hipGraphExecDestroy(ready) == 0 and hip.hipGraphDestroy(graph) == 0


@pytest.mark.parametrize("how", ["del", "collector", "close"])
@pytest.mark.parametrize("kind", list(MAKE))
def test_the_capture_goes_on(kind, how):
    kept = rope()
    x = torch.randn((3, 2, 64), device="cuda")
    y, z = torch.zeros_like(x), torch.zeros_like(x)
    want, twice = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.current_stream().cuda_stream
    kept.apply(3, x.data_ptr(), want.data_ptr(), 2, "f32", first=7, stream=s)
    kept.apply(3, want.data_ptr(), twice.data_ptr(), 2, "f32", first=-7, stream=s)
    gone = MAKE[kind]()
    gc.collect()

    def body(stream):
        nonlocal gone
        kept.apply(3, x.data_ptr(), y.data_ptr(), 2, "f32", first=7, stream=stream)
        if how == "close":
            gone.close()
        elif how == "collector":
            gone.itself = gone
        gone = None
        if how == "collector":
            gc.collect()
        kept.apply(3, y.data_ptr(), z.data_ptr(), 2, "f32", first=-7, stream=stream)

    captured(body)
    assert torch.equal(y, want) and torch.equal(z, twice)


@pytest.mark.parametrize("kind", list(MAKE))
def test_destruction_waits_for_the_device(kind):
    gone = MAKE[kind]()
    busy = w4(1 << 14, 1 << 13)
    x, y = torch.randn((64, 1 << 13), device="cuda"), torch.empty((64, 1 << 14), device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(100):
        busy.matvec(64, x.data_ptr(), "f32", y.data_ptr(), "f32", stream=side.cuda_stream)
    assert not side.query()
    gone.close()
    assert side.query()
