"""What a pair of rotary positions turns by per position, as the kernels get it: the fraction of a turn in 64 bits, from the host
side of np_rope_create over a stand-in for the device, against whole-number arithmetic."""
import ctypes
import importlib.util
import os
import random
import subprocess
from fractions import Fraction

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "delta_prefetched_ffn_amd", "csrc")
P = 1 << 20   # an aligned address, never followed here


def _arctan_of_one_over(x, one):
    term, n, total = one // x, 1, 0
    while term:
        total += term // n if n % 4 == 1 else -(term // n)
        term //= x * x
        n += 2
    return total


def turns_of(f):
    """f / (2 pi) to some 500 bits (pi by Machin's formula)."""
    one = 1 << 560
    pi = 4 * (4 * _arctan_of_one_over(5, one) - _arctan_of_one_over(239, one))
    return Fraction(f) * Fraction(one, 2 * pi)


@pytest.fixture(scope="module")
def B(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("rope") / "librope_stub.so")
    srcs = [os.path.join(CSRC, f) for f in ("np_kv.hip", "np_prefix.hip", "np_rope.hip", "np_w4.hip")] + [os.path.join(ROOT, "tests", "rope_stub.cpp")]
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "tests"), "-x", "c++", *srcs, "-o", so],
                   check=True, capture_output=True, text=True)
    spec = importlib.util.spec_from_file_location("rope_stubbed_binding", os.path.join(ROOT, "delta_prefetched_ffn_amd", "binding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    real, stub = m.lib(), ctypes.CDLL(so)
    for name in m.EXPORTS:
        if name.startswith(("np_kv_", "np_attend_", "np_rope_", "np_w4_")):
            getattr(stub, name).argtypes = getattr(real, name).argtypes
    stub.np_last_error.restype = ctypes.c_char_p
    stub.stub_turns.argtypes = [ctypes.c_void_p]
    m.lib = lambda: stub
    return m


def bits_of(B, freqs):
    rope = B.Rope(head_dim=256, rot_dim=2 * len(freqs), freqs=freqs, device=1)
    rope.apply(1, P, P, 1, "f32")
    got = np.zeros(128, np.uint64)
    assert B.lib().stub_turns(got.ctypes.data) == len(freqs)
    return [int(x) for x in got[:len(freqs)]]


def test_fractions_of_a_turn_to_the_nearest_64_bits(B):
    rng = random.Random(1)
    some = [0.0, 1.0, -1.0, 1e-30, -1e-30, 5e-324, 2.0 ** -60, -2.0 ** -60, 2 * np.pi, -2 * np.pi, np.nextafter(2 * np.pi, 0), np.pi / 4, 2.0 ** 40, -2.0 ** 40, 1e12, 123456.789]
    some += [rng.choice([-1, 1]) * 10.0 ** rng.uniform(-25, 12) for _ in range(300)] + [10000.0 ** (-i / 64) for i in range(64)]
    for at in range(0, len(some), 100):
        part = some[at:at + 100]
        for f, got in zip(part, bits_of(B, part)):
            off = (turns_of(f) * (1 << 64) - got) % (1 << 64)
            off = min(off, (1 << 64) - off)
            # to the nearest, but for what the last of 128 bits of 1 / (2 pi) leaves out of 2^38 turns
            assert off <= Fraction(1, 2) + Fraction(1, 1 << 20), (f, float(off))


def test_more_than_the_bits_hold_is_refused(B):
    for f in (np.nextafter(2.0 ** 40, np.inf), -1e13, 1e300, float("inf"), float("nan")):
        with pytest.raises(B.NPError) as e:
            B.Rope(head_dim=8, freqs=[1.0, f, 1.0, 1.0], device=1)
        assert e.value.status == B.NP_EINVAL
    for kw in (dict(base=1e-300), dict(base=1e-17), dict(scaling="linear", factor=1e-13)):
        with pytest.raises(B.NPError) as e:
            B.Rope(head_dim=64, device=1, **kw)
        assert e.value.status == B.NP_EINVAL
    B.Rope(head_dim=64, device=1, base=1e-9)
