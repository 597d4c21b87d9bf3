"""Host sides of the attention over shared pages, the rotary positions and the products with 4-bit weights, on the CPU: compiled
over tests/ops_stub.cpp, which stands for the device, so that plans can be looked at, and refusals and failures tried."""
import ctypes
import importlib.util
import os
import random
import subprocess

import numpy as np
import pytest

from tests import rope_reference as RR

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "delta_prefetched_ffn_amd", "csrc")
P = 1 << 20   # an aligned address, never followed here


@pytest.fixture(scope="module")
def B(tmp_path_factory):
    """The binding over the stubbed library, with the stub's switches as B.stub."""
    so = str(tmp_path_factory.mktemp("ops") / "libops_stub.so")
    srcs = [os.path.join(CSRC, f) for f in ("np_kv.hip", "np_prefix.hip", "np_rope.hip", "np_w4.hip")] + [os.path.join(ROOT, "tests", "ops_stub.cpp")]
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "tests"), "-x", "c++", *srcs, "-o", so],
                   check=True, capture_output=True, text=True)
    spec = importlib.util.spec_from_file_location("ops_stubbed_binding", os.path.join(ROOT, "delta_prefetched_ffn_amd", "binding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    real, stub = m.lib(), ctypes.CDLL(so)
    for name in m.EXPORTS:
        if name.startswith(("np_kv_", "np_attend_", "np_rope_", "np_w4_")):
            getattr(stub, name).argtypes = getattr(real, name).argtypes
    stub.np_last_error.restype = stub.stub_check_prefix.restype = ctypes.c_char_p
    stub.stub_fail_new.argtypes = [ctypes.c_long]
    stub.stub_launches.restype = stub.stub_wrong_device.restype = stub.stub_prefix_calls.restype = stub.stub_rope_items.restype = ctypes.c_long
    m.lib = lambda: stub
    m.stub = stub
    return m


def refused(B, status, f, *a, **kw):
    launches = B.stub.stub_launches()
    with pytest.raises(B.NPError) as e:
        f(*a, **kw)
    assert e.value.status == status, str(e.value)
    assert B.stub.stub_launches() == launches
    return str(e.value)


def cache(B, **kw):
    base = dict(n_layers=2, n_heads=32, n_kv_heads=32, head_dim=128, page_tokens=16, n_pages=1 << 14, max_seqs=140, max_pages=4000, device=1, codes=P, exps=P)
    base.update(kw)
    return B.KVCache(**base)


def shared(B, kv, dtype="bf16", **kw):
    """Whether a call shares; if so its plan is checked."""
    before = B.stub.stub_prefix_calls()
    kv.attend_shared(0, P, P, dtype, scale=1.0, **kw)
    if B.stub.stub_prefix_calls() == before:
        return False
    assert B.stub.stub_check_prefix() == b""
    return True


# ------------------------------------------------------------------------------------------- attention over shared pages

@pytest.mark.parametrize("seed", range(12))
def test_plans_of_random_families(B, seed):
    rng = random.Random(seed)
    pt = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([8, 16, 32])
    kv = cache(B, n_heads=kv_heads * rng.choice([1, 2, 4]), n_kv_heads=kv_heads, head_dim=rng.choice([40, 64, 128, 192, 256]), page_tokens=pt)
    made, at = [], 0
    for _ in range(rng.randint(1, 4)):
        kv.extend([at], [rng.randint(1500, 9000)])
        made.append(at)
        at += 1
    took = 0
    for _ in range(rng.randint(20, 100)):
        src = rng.choice(made)
        kv.fork(src, at, max(1, kv.tokens(src) - rng.choice([0, 0, 1, pt, rng.randint(0, 900)])))
        if rng.random() < 0.7:
            kv.extend([at], [rng.randint(1, 500)])
        made.append(at)
        at += 1
    for _ in range(6):
        some = rng.sample(made, rng.randint(2, min(len(made), 110)))
        same = rng.choice([0, 1, 1, 3])
        kv.extend(some, [same or rng.randint(0, 6) for _ in some])
        for dtype in ("bf16", "f32"):
            for kw in ({}, dict(window=rng.randint(1, 12000), sinks=rng.choice([0, 4, 300]))):
                took += shared(B, kv, dtype, **kw)
        took += shared(B, kv)      # the plan is kept
        if rng.random() < 0.3:
            kv.compact()
            took += shared(B, kv)
    assert took > 6


def test_the_gpu_tests_shapes_reach_the_shared_kernels(B):
    def family(heads, kvh, hd, page, prompt, tails, new, dtype="bf16", **kw):
        kv = cache(B, n_heads=heads, n_kv_heads=kvh, head_dim=hd, page_tokens=page)
        n = len(tails)
        kv.extend([0], [prompt])
        for i in range(n):
            kv.fork(0, i + 1, prompt)
        kv.extend(list(range(1, n + 1)), tails)
        kv.extend(list(range(1, n + 1)), new)
        return shared(B, kv, dtype, **kw)

    for dtype in ("f32", "bf16"):
        for heads, kvh, hd, page, prompt, n in ((16, 16, 64, 16, 4003, 24), (32, 8, 128, 64, 4003, 24), (28, 4, 80, 32, 5003, 40), (12, 12, 40, 128, 5401, 24), (16, 16, 256, 16, 1003, 24),
                                                (24, 12, 192, 64, 1903, 24), (40, 4, 128, 32, 4003, 40)):
            assert family(heads, kvh, hd, page, prompt, [70] * n, [1] * n, dtype), (heads, hd, dtype)
    kv = cache(B, n_heads=4, n_kv_heads=4, head_dim=64, page_tokens=64)
    kv.extend(list(range(40)), [3000 + 19 * i for i in range(40)])
    for i in range(40):
        kv.fork(i, 40 + i, 3000 + 19 * i - i % 5)
        kv.fork(i, 80 + i, 3000 + 19 * i - i % 7)
    kv.extend(list(range(120)), [1] * 120)
    assert shared(B, kv) and B.stub.stub_prefix_runs() == 32   # 40 families
    kv = cache(B, n_heads=16, n_kv_heads=16, head_dim=64)
    kv.extend([0], [2000])
    for i in range(40):
        kv.fork(i, i + 1, kv.tokens(i) // 16 * 16)
        kv.extend([i + 1], [80])
    kv.extend(list(range(41)), [1] * 41)
    assert shared(B, kv) and B.stub.stub_prefix_runs() == 32   # a chain of 40
    assert not family(4, 4, 64, 16, 300, [20] * 3, [1] * 3)                # too little
    assert not family(32, 8, 128, 64, 4003, [20] * 24, [1] * 23 + [64])    # a prompt among the tokens


def test_nothing_to_share_and_no_rows(B):
    kv = cache(B)
    kv.extend([0, 1], [4000, 4000])
    assert not shared(B, kv)
    kv.extend([0, 1], [0, 0])
    launches = B.stub.stub_launches()
    kv.attend_shared(0, P, P, "bf16", scale=1.0)
    assert B.stub.stub_launches() == launches
    # one sequence of the step only: its page is shared with one that is not in it
    kv.fork(0, 2, 4000)
    kv.extend([2], [1])
    assert not shared(B, kv)


def test_shared_attention_where_something_fails(B):
    def prepared():
        kv = cache(B)
        kv.extend([0], [3000])
        for i in range(1, 25):
            kv.fork(0, i, 3000)
        kv.extend(list(range(1, 25)), [1] * 24)
        return kv

    for after in range(200):
        kv = prepared()
        B.stub.stub_fail_new(after)
        try:
            kv.attend_shared(0, P, P, "bf16", scale=1.0)
            failed = False
        except B.NPError as e:
            failed = True
            assert e.status == B.NP_ENOMEM
        finally:
            B.stub.stub_fail_new(-1)
        assert shared(B, kv)
        if not failed:
            break
    else:
        assert False, "never came through"
    kv = prepared()
    B.stub.stub_fail_set_device(1)
    try:
        refused(B, B.NP_EHIP, kv.attend_shared, 0, P, P, "bf16", scale=1.0)
    finally:
        B.stub.stub_fail_set_device(0)
    wrong = B.stub.stub_wrong_device()
    assert shared(B, kv) and B.stub.stub_wrong_device() == wrong and B.stub.stub_device() == 0
    for a, kw in (((2, P, P, "bf16"), {}), ((0, P + 8, P, "bf16"), {}), ((0, P, P, "bf16", (4096, 128, 4096, 64)), {}), ((0, P, P, "bf16"), dict(window=-1)), ((0, P, P, "bf16"), dict(sinks=-1)),
                  ((0, P, P, "bf16"), dict(lse_ptr=P + 2)), ((0, P, P, "bf16", (4096, 128, -4096, 128)), {})):
        refused(B, B.NP_EINVAL, kv.attend_shared, *a, scale=1.0, **kw)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        refused(B, B.NP_EINVAL, kv.attend_shared, 0, P, P, "bf16", scale=scale)
    with pytest.raises(OverflowError):
        kv.attend_shared(0, P, P, "bf16", scale=1.0, window=1 << 32)
    kv.trim(3, 100)
    refused(B, B.NP_ESTATE, kv.attend_shared, 0, P, P, "bf16", scale=1.0)
    books = cache(B, device=B.KV_HOST, codes=0, exps=0)
    books.extend([0], [1])
    refused(B, B.NP_ESTATE, books.attend_shared, 0, P, P, "bf16", scale=1.0)


# ----------------------------------------------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("kw", [{}, dict(base=500000.0), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0), dict(scaling="blend", factor=16.0, context=4096, low=1.0, high=32.0),
                                dict(scaling="blend", factor=8.0, context=8192, low=1.0, high=4.0, base=500000.0), dict(scaling="blend", factor=2.0, context=100, low=-1.0, high=0.5)])
def test_frequencies(B, kw):
    for rot in (4, 20, 64, 128, 256):
        got = B.rope_freqs(head_dim=256, rot_dim=rot, **kw)
        np.testing.assert_allclose(got, RR.freqs(rot, **kw), rtol=1e-13)
    assert B.rope_freqs(head_dim=64, rot_dim=0).size == 0


def test_rope_refusals(B):
    good = dict(head_dim=64, device=1)
    for bad in (dict(head_dim=0), dict(head_dim=12), dict(head_dim=264), dict(rot_dim=-2), dict(rot_dim=3), dict(rot_dim=66), dict(amplitude=0.0), dict(amplitude=float("inf")), dict(base=0.0), dict(base=float("nan")),
                dict(scaling="linear", factor=0.0), dict(scaling="ntk", factor=2.0, rot_dim=2), dict(scaling="blend", factor=2.0), dict(scaling="blend", factor=2.0, context=10, low=2.0, high=1.0),
                dict(freqs=[float("inf")] * 32), dict(device=2), dict(device=-1), dict(base=1e-300, scaling="linear", factor=1e-200)):
        refused(B, B.NP_EINVAL, B.Rope, **{**good, **bad})
    with pytest.raises(ValueError):
        B.Rope(**good, freqs=[1.0])
    with pytest.raises(KeyError):
        B.Rope(**good, layout="other")
    r = B.Rope(**good)
    for a, kw in (((-1, P, P, 2, "f32"), {}), (((1 << 28) + 1, P, P, 2, "f32"), {}), ((4, P, P, 0, "f32"), {}), ((4, P, P, 4097, "f32"), {}), ((4, 0, P, 2, "f32"), {}), ((4, P, 0, 2, "f32"), {}), ((4, P + 4, P, 2, "f32"), {}),
                  ((4, P, P, 2, "f32"), dict(n_kv_heads=-1)), ((4, P, P, 2, "f32"), dict(n_kv_heads=1)), ((4, P, P, 2, "f32"), dict(k_ptr=P)), ((4, P, P, 2, "f32"), dict(first=2 ** 31 - 3)),
                  ((4, P, P, 2, "f32", (128, 64, 128, 32, 0, 0, 0, 0)), {}), ((4, P, P, 2, "f32", (128, 64, 64, 64, 0, 0, 0, 0)), {}), ((4, P, P, 2, "bf16", (128, 4, 128, 64, 0, 0, 0, 0)), {}),
                  ((1 << 28, P, P, 2, "f32", (128, 64, 0, 64, 0, 0, 0, 0)), {}), ((4, P, P, 2, "f32"), dict(eps=-1e-9)), ((4, P, P, 2, "f32"), dict(q_weight_ptr=P + 8))):
        refused(B, B.NP_EINVAL, r.apply, *a, **kw)
    r.apply(4, P, P, 2, "f32", first=2 ** 31 - 4)
    r.apply(1 << 25, P, P, 32, "f32")
    assert B.stub.stub_rope_items() == 1 << 25
    refused(B, B.NP_EINVAL, r.apply, (1 << 26) + 64, P, P, 2, "f32")
    r.apply(1, P, P, 32, "f32")
    assert B.stub.stub_rope_items() == 2           # 16 heads of 64 values a wave, each wave its own
    kv = cache(B, head_dim=64)
    refused(B, B.NP_ESTATE, r.append, kv, 0, P, P, P, P, "f32")
    kv.extend([0], [3])
    r.append(kv, 0, P, P, P, P, "f32")
    for a, kw in (((2, P, P, P, P, "f32"), {}), ((0, P, P, P + 4, P, "f32"), {}), ((0, P, P, P, 0, "f32"), {}), ((0, P, P, P, P, "f32", (2048, 64, 2048, 32, 2048, 64, 2048, 64)), {}),
                  ((0, P, P, P, P, "f32"), dict(eps=float("nan"))), ((0, P, P, P, P, "f32"), dict(k_weight_ptr=P + 4))):
        refused(B, B.NP_EINVAL, r.append, kv, *a, **kw)
    refused(B, B.NP_EINVAL, B.Rope(head_dim=64, device=0).append, kv, 0, P, P, P, P, "f32")
    refused(B, B.NP_EINVAL, B.Rope(head_dim=72, device=1).append, kv, 0, P, P, P, P, "f32")
    books = cache(B, device=B.KV_HOST, codes=0, exps=0, head_dim=64)
    books.extend([0], [1])
    refused(B, B.NP_ESTATE, r.append, books, 0, P, P, P, P, "f32")
    B.stub.stub_fail_set_device(1)
    try:
        refused(B, B.NP_EHIP, r.append, kv, 0, P, P, P, P, "f32")
        refused(B, B.NP_EHIP, r.apply, 4, P, P, 2, "f32")
        refused(B, B.NP_EHIP, B.Rope, **good)
    finally:
        B.stub.stub_fail_set_device(0)
    wrong = B.stub.stub_wrong_device()
    r.apply(4, P, P, 2, "f32")
    r.append(kv, 0, P, P, P, P, "f32")
    assert B.stub.stub_wrong_device() == wrong and B.stub.stub_device() == 0
    r.close()


def test_the_largest_prompts_fit_a_launch_or_are_refused(B):
    # Workgroups of up to 512 threads, of which a launch takes less than 2^32.
    for heads, kv, hd, page, pages in ((64, 64, 256, 128, 62000), (64, 64, 256, 128, 120000), (64, 64, 8, 16, 130000), (1, 1, 256, 128, 65000), (128, 128, 8, 16, 62000), (128, 128, 8, 16, 70000), (64, 64, 256, 128, 130000), (128, 128, 8, 16, 600000)):
        c = cache(B, n_heads=heads, n_kv_heads=kv, head_dim=hd, page_tokens=page, n_pages=pages, max_pages=pages, max_seqs=2)
        rope = B.Rope(head_dim=hd, device=1)
        c.extend([0], [pages * page])
        launches = B.stub.stub_launches()
        try:
            rope.append(c, 0, P, P << 22, P << 23, P << 24, "bf16")
        except B.NPError as e:
            assert e.status == B.NP_EINVAL and "too many" in str(e), (heads, hd, page, pages, str(e))
            assert B.stub.stub_launches() == launches
        else:
            assert B.stub.stub_launches() == launches + 1


def test_failed_allocations_reach_the_caller(B):
    for make in (lambda: B.Rope(head_dim=64, device=1), lambda: B.W4(n_out=16, n_in=128, group=128, codes_ptr=P, scales_ptr=P, scale_dtype="f16", device=1)):
        for after in range(20):
            B.stub.stub_fail_new(after)
            try:
                made = make()
                break
            except B.NPError as e:
                assert e.status == B.NP_ENOMEM
            finally:
                B.stub.stub_fail_new(-1)
        else:
            assert False, "never came through"
        made.close()


# --------------------------------------------------------------------------------------------------------- 4-bit weights

def test_w4_refusals(B):
    good = dict(n_out=16, n_in=128, group=128, codes_ptr=P, scales_ptr=P, scale_dtype="f16", device=1)
    for bad in (dict(n_out=0), dict(n_out=(1 << 20) + 1), dict(n_in=0), dict(n_in=4), dict(n_in=12), dict(n_in=(1 << 17) + 8), dict(group=0), dict(group=-64), dict(group=16), dict(group=96), dict(group=192),
                dict(group=1 << 18), dict(codes_ptr=0), dict(codes_ptr=P + 2), dict(scales_ptr=0), dict(scales_ptr=P + 1), dict(scales_ptr=P + 2, scale_dtype="f32"), dict(device=2), dict(device=-1)):
        refused(B, B.NP_EINVAL, B.W4, **{**good, **bad})
    w = B.W4(**good)
    Y = P + (1 << 16)
    for a, kw in (((-1, P, "f32", Y, "f32"), {}), (((1 << 20) + 1, P, "f32", Y, "f32"), {}), ((1, P + 4, "f32", Y, "f32"), {}), ((1, 0, "f32", Y, "f32"), {}), ((1, P, "f32", 0, "f32"), {}), ((1, P, "f32", Y + 2, "f32"), {}),
                  ((1, P, "f32", Y + 1, "bf16"), {}), ((1, P, "f32", P + 508, "f32"), {}), ((1, P, "f32", P - 60, "f32"), {}), ((2, P, "bf16", Y, "f32"), dict(x_stride=132)), ((2, P, "f32", Y, "f32"), dict(x_stride=-128)),
                  ((2, P, "f32", Y, "f32"), dict(x_stride=124)), ((2, P, "f32", Y, "f32"), dict(y_stride=15)), ((2, P, "f32", P + 4 * 120, "f32"), dict(x_stride=144, y_stride=144)),
                  ((2, P, "f32", P + 4 * 132, "f32"), dict(x_stride=144, y_stride=144)), ((3, P, "f32", P + 4 * 128, "f32"), dict(x_stride=144, y_stride=148))):
        refused(B, B.NP_EINVAL, w.matvec, *a, **kw)
    w.matvec(2, P, "f32", P + 4 * 128, "f32", x_stride=144, y_stride=144)
    w.matvec(2, P + 64, "f32", P, "f32", x_stride=144, y_stride=144)
    launches = B.stub.stub_launches()
    w.matvec(0, P, "f32", Y, "f32")
    assert B.stub.stub_launches() == launches
    with pytest.raises(OverflowError):
        w.matvec(1 << 63, P, "f32", Y, "f32")
    big = B.W4(**{**good, "n_out": 1 << 20, "n_in": 8})
    refused(B, B.NP_EINVAL, big.matvec, 1 << 20, P, "f32", 1 << 50, "f32")
    B.stub.stub_fail_set_device(1)
    try:
        refused(B, B.NP_EHIP, w.matvec, 1, P, "f32", Y, "f32")
        refused(B, B.NP_EHIP, B.W4, **good)
    finally:
        B.stub.stub_fail_set_device(0)
    wrong = B.stub.stub_wrong_device()
    w.matvec(1, P, "f32", Y, "f32")
    assert B.stub.stub_wrong_device() == wrong and B.stub.stub_device() == 0
    w.close()
