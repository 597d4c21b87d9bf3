"""The host side of the 8-bit key/value cache where something fails beneath it, on the CPU: np_kv.hip compiled together with
tests/kv_stub.cpp, which stands for the device (allocations, the current device and launches fail on demand there)."""
import ctypes
import importlib.util
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "delta_prefetched_ffn_amd", "csrc")


@pytest.fixture(scope="module")
def B(tmp_path_factory):
    """The binding over the stubbed library, with the stub's switches as B.stub."""
    so = str(tmp_path_factory.mktemp("kv") / "libkv_stub.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), "-x", "c++", os.path.join(CSRC, "np_kv.hip"),
                    os.path.join(ROOT, "tests", "kv_stub.cpp"), "-o", so], check=True, capture_output=True, text=True)
    spec = importlib.util.spec_from_file_location("kv_stubbed_binding", os.path.join(ROOT, "delta_prefetched_ffn_amd", "binding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    real, stub = m.lib(), ctypes.CDLL(so)
    for name in m.EXPORTS:
        if name.startswith("np_kv_"):
            getattr(stub, name).argtypes = getattr(real, name).argtypes
    stub.np_last_error.restype = ctypes.c_char_p
    stub.stub_fail_new.argtypes = [ctypes.c_long]
    stub.stub_launches.restype = stub.stub_wrong_device.restype = ctypes.c_long
    stub.stub_table.restype = ctypes.POINTER(ctypes.c_int32)
    m.lib = lambda: stub
    m.stub = stub
    return m


def cache(B, **kw):
    base = dict(n_layers=2, n_heads=8, n_kv_heads=4, head_dim=64, page_tokens=16, n_pages=40, max_seqs=6, max_pages=12, device=1,
                codes=1 << 20, exps=1 << 20)
    base.update(kw)
    return B.KVCache(**base)


def books(kv):
    return [(kv.pages(s).tolist(), kv.tokens(s)) for s in range(kv.max_seqs)], kv.info()


def prepared(B):
    """Sequences with shared, dropped, half-filled and reserved pages, and holes in the pool."""
    kv = cache(B)
    kv.extend([0, 1], [75, 40])
    kv.fork(0, 2, 70)
    kv.extend([1], [20])
    kv.evict(1, 16, 0)
    kv.adopt(3, [30, 31, 38], 20)
    kv.extend([0, 3], [0, 0])
    return kv


CALLS = {
    "extend": lambda kv: kv.extend([0, 2, 1, 4], [60, 100, 1, 33]),
    "extend_copies": lambda kv: kv.extend([2, 0], [1, 1]),
    "share": lambda kv: kv.fork(0, 4, 66),
    "copy": lambda kv: kv.fork(0, 4, 66, "copy"),
    "adopt": lambda kv: kv.adopt(4, [20, 21, 22, 23, 24], 70),
    "evict": lambda kv: kv.evict(0, 5, 0),
    "compact": lambda kv: kv.compact(),
    "trim": lambda kv: kv.trim(2, 3),
    "reset": lambda kv: kv.reset(),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_failed_allocations_change_nothing(B, name):
    call = CALLS[name]
    want = prepared(B)
    call(want)
    for after in range(200):
        kv = prepared(B)
        before = books(kv)
        B.stub.stub_fail_new(after)
        try:
            call(kv)
            failed = False
        except B.NPError as e:
            failed = True
            assert e.status == B.NP_ENOMEM
        finally:
            B.stub.stub_fail_new(-1)
        if failed:
            assert books(kv) == before, f"changed by a call that failed at allocation {after}"
            call(kv)
        assert books(kv) == books(want)
        # and the device's page table follows
        live = [s for s in range(kv.max_seqs) if kv.tokens(s) % 16]
        if live:
            kv.extend(live, [0] * len(live))
            for s in live:
                at = s * kv.max_pages
                assert B.stub.stub_table()[at:at + len(kv.pages(s))] == kv.pages(s).tolist(), s
        if not failed:
            return
    assert False, "never came through"


def test_an_error_is_reported_without_memory(tmp_path):
    # The text of an error is kept without an allocation: a throw from there would leave a C entry.
    src = tmp_path / "new.cpp"
    src.write_text("#include <cstdlib>\n#include <new>\nextern \"C\" { int no_memory = 0; }\n"
                   "void* operator new(size_t n) { if (no_memory) throw std::bad_alloc(); return std::malloc(n ? n : 1); }\n"
                   "void operator delete(void* p) noexcept { std::free(p); }\nvoid operator delete(void* p, size_t) noexcept { std::free(p); }\n")
    so = str(tmp_path / "libnew.so")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", str(src), "-o", so], check=True)
    script = ("import ctypes, sys\n"
              "L, new = ctypes.CDLL(sys.argv[1]), ctypes.CDLL(sys.argv[2])\n"
              "L.np_last_error.restype = ctypes.c_char_p\n"
              "off = ctypes.c_int.in_dll(new, 'no_memory')\n"
              "desc = (ctypes.c_int32 * 16)(1, 7, 3, 64, 16, 4, 1, 4, -1)\n"
              "h = ctypes.c_void_p()\n"
              "off.value = 1\n"
              "bad = L.np_kv_create(desc, ctypes.byref(h))\n"          # n_heads no multiple of n_kv_heads
              "desc[1] = 6\n"
              "none = L.np_kv_create(desc, ctypes.byref(h))\n"         # in order, but there is no memory for it
              "off.value = 0\n"
              "print(bad, none, L.np_last_error().decode())\n")
    env = dict(os.environ)
    env["LD_PRELOAD"] = so + (":" + env["LD_PRELOAD"] if env.get("LD_PRELOAD") else "")
    r = subprocess.run(["python3", "-c", script, os.path.join(ROOT, "delta_prefetched_ffn_amd", "libnp.so"), so],
                       env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip() == "1 3 host allocation failed"


STREAM_CALLS = {
    "extend": lambda kv: kv.extend([0, 2], [60, 1]),
    "append": lambda kv: kv.append(0, 4096, 4096, "bf16"),
    "attend": lambda kv: kv.attend(0, 4096, 4096, "bf16", scale=1.0),
    "copy": lambda kv: kv.fork(0, 4, 66, "copy"),
    "compact": lambda kv: kv.compact(),
    "read_tokens": lambda kv: kv.read_tokens(0, 3, 0, 0),
}


@pytest.mark.parametrize("name", list(STREAM_CALLS))
def test_a_device_that_cannot_be_made_current_is_reported(B, name):
    # The current device is another one (0); work for the cache's would go to it.
    kv = prepared(B)
    kv.extend([0, 1], [3, 2])
    before, wrong, launches = books(kv), B.stub.stub_wrong_device(), B.stub.stub_launches()
    B.stub.stub_fail_set_device(1)
    try:
        with pytest.raises(B.NPError) as e:
            STREAM_CALLS[name](kv)
    finally:
        B.stub.stub_fail_set_device(0)
    assert e.value.status == B.NP_EHIP and "hipSetDevice" in str(e.value)
    assert books(kv) == before and B.stub.stub_launches() == launches
    STREAM_CALLS[name](kv)
    assert B.stub.stub_wrong_device() == wrong and B.stub.stub_device() == 0


def test_a_failed_launch_asks_for_a_reset(B):
    for call in (lambda kv: kv.extend([0, 2], [60, 1]), lambda kv: kv.fork(0, 4, 66, "copy"), lambda kv: kv.compact()):
        kv = prepared(B)
        B.stub.stub_fail_launch(0)
        try:
            with pytest.raises(B.NPError) as e:
                call(kv)
        finally:
            B.stub.stub_fail_launch(-1)
        assert e.value.status == B.NP_EHIP
        for again in (lambda: kv.extend([0], [1]), lambda: kv.append(0, 4096, 4096, "f32"), lambda: kv.attend(0, 4096, 4096, "f32", scale=1.0),
                      lambda: kv.fork(0, 5, 1), lambda: kv.free(0), lambda: kv.adopt(5, [], 0), lambda: kv.compact()):
            with pytest.raises(B.NPError) as e:
                again()
            assert e.value.status == B.NP_ESTATE
        kv.reset()
        kv.extend([0], [17])
        assert B.stub.stub_table()[:2] == kv.pages(0).tolist() == [0, 1]


def test_calls_too_large_for_a_launch_are_refused_before_anything_is_enqueued(B):
    # 2^24 blocks of one append, 2^23 row tiles of one attend: a grid would pass 2^32 threads.
    kv = cache(B, n_heads=1024, n_kv_heads=1024, head_dim=8, n_pages=1 << 15, max_pages=1 << 15)
    kv.extend([0], [((1 << 14) - 1) * 16])
    kv.append(0, 4096, 4096, "bf16")
    kv.extend([0], [16 * ((1 << 14) - 1)])
    kv.append(0, 4096, 4096, "bf16")
    kv.free(0)
    kv.extend([0], [1 << 18])
    launches = B.stub.stub_launches()
    with pytest.raises(B.NPError) as e:
        kv.append(0, 4096, 4096, "bf16")
    assert e.value.status == B.NP_EINVAL
    kv = cache(B, n_heads=4096, n_kv_heads=1, head_dim=128, n_pages=1 << 14, max_pages=1 << 14, page_tokens=128)
    kv.extend([0], [(1 << 15) - 16])
    kv.attend(0, 4096, 4096, "f32", scale=1.0)
    assert B.stub.stub_launches() == launches + 2      # a table of at most 480 entries, the attention
    kv.extend([0], [1 << 15])
    launches = B.stub.stub_launches()
    with pytest.raises(B.NPError) as e:
        kv.attend(0, 4096, 4096, "f32", scale=1.0)
    assert e.value.status == B.NP_EINVAL
    kv.attend(0, 4096, 4096, "bf16", scale=1.0)        # large tiles: 256 rows a workgroup
    assert B.stub.stub_launches() == launches + 1


def test_exponents_at_an_odd_address_are_refused(B):
    # The attention reads a head's two exponents as one 16-bit number.
    for exps in ((1 << 20) + 1, (1 << 20) + 3):
        with pytest.raises(B.NPError) as e:
            cache(B, exps=exps)
        assert e.value.status == B.NP_EINVAL and "exps" in str(e.value)
    cache(B, exps=(1 << 20) + 2)
    cache(B, device=B.KV_HOST, codes=0, exps=0)
