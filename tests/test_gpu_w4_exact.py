"""Products with 4-bit weights whose sums are exact in fp32, so that every bit of x is seen: one input of a row is not zero, all 24 of
its bits set at random, codes are powers of two, scales too. With zero points besides, within a few steps of the true sums. Each kernel
that np_w4_matvec may take, by the name of the one that ran."""
import re

import numpy as np
import pytest

from tests import test_gpu_kv as K
from tests.harness import torch_mod

pytestmark = pytest.mark.gpu

torch = None


@pytest.fixture(autouse=True, scope="module")
def _torch():
    global torch
    torch = K.torch = torch_mod()
    assert torch.cuda.is_available()


def tdt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def kernel(w, rows, n_in, n_out, xd):
    """"staged" or "rows" with its row tiles, or "tile" with its waves."""
    x, y = torch.zeros((rows, n_in), dtype=tdt(xd), device="cuda"), torch.zeros((rows, n_out), device="cuda")
    names = [n for n in K.kernels_of(lambda s: w.matvec(rows, x.data_ptr(), xd, y.data_ptr(), "f32", stream=s)) if "k_w4" in n]
    got = set()
    for n in names:
        m = re.search(r"k_w4_rowsI\w+?Li(\d)ELi\dELi\dELb(\d)E", n)
        got.add(("staged" if m[2] == "1" else "rows", int(m[1])) if m else ("tile", 8 if "Li1ELi2ELi" in n else 4))
    assert len(got) == 1
    return got.pop()


def matrix(c, s, z, group, scales):
    from delta_prefetched_ffn_amd import W4
    codes = torch.from_numpy((c[:, 0::2] | c[:, 1::2] << 4).astype(np.uint8)).cuda()
    sd, zd = torch.from_numpy(s.astype(np.float32)).to(tdt(scales)).cuda(), torch.from_numpy(z.astype(np.uint8)).cuda()
    return W4(n_out=c.shape[0], n_in=c.shape[1], group=group, codes_ptr=codes.data_ptr(), scales_ptr=sd.data_ptr(), scale_dtype=scales, zeros_ptr=zd.data_ptr())


def one_a_row(rng, rows, n_in, xd):
    """x with one value a row, somewhere, all of whose type's bits count, between 2^-4 and 2^4."""
    bits = {"f32": 23, "bf16": 7, "f16": 10}[xd]
    x = np.zeros((rows, n_in))
    at = rng.integers(0, n_in, rows)
    x[np.arange(rows), at] = (1 + (rng.integers(0, 1 << bits, rows) | 1) * 2.0 ** -bits) * np.exp2(rng.integers(-4, 4, rows)) * rng.choice([-1, 1], rows)
    return x, at


CASES = [  # rows, n_out, n_in, x, the kernel
    (1, 70, 1160, "f32", ("staged", 1)), (16, 33, 520, "f32", ("staged", 1)), (16, 70, 1160, "f32", ("rows", 1)), (9, 70, 11008, "f32", ("rows", 1)), (27, 70, 1160, "f32", ("rows", 2)),
    (64, 70, 1160, "f32", ("rows", 4)), (130, 4100, 392, "f32", ("tile", 8)), (64, 8200, 264, "f32", ("tile", 8)), (130, 4100, 136, "f32", ("tile", 8)),
    (5, 70, 1160, "bf16", ("rows", 1)), (64, 70, 1160, "f16", ("rows", 4)), (260, 4100, 392, "f16", ("tile", 8)), (260, 4100, 392, "bf16", ("tile", 8)), (4100, 1100, 264, "f16", ("tile", 4)),
    (4100, 1100, 264, "bf16", ("tile", 4))]


@pytest.mark.parametrize("group,scales", [(32, "f32"), (64, "f16"), (128, "bf16"), (256, "f32")])
@pytest.mark.parametrize("rows,n_out,n_in,xd,takes", CASES)
def test_every_bit_of_x_counts(rows, n_out, n_in, xd, takes, group, scales):
    rng = np.random.default_rng(rows + n_out + group)
    groups = -(-n_in // group)
    c, z = 1 << rng.integers(0, 4, (n_out, n_in)), np.zeros((n_out, groups), np.int64)
    s = np.exp2(rng.integers(-3, 4, (n_out, groups)))
    w = matrix(c, s, z, group, scales)
    assert kernel(w, rows, n_in, n_out, xd) == takes
    x, at = one_a_row(rng, rows, n_in, xd)
    xt, y = torch.from_numpy(x.astype(np.float32)).to(tdt(xd)).cuda(), torch.empty((rows, n_out), device="cuda")
    assert np.array_equal(xt.double().cpu().numpy(), x)
    stream = torch.cuda.current_stream().cuda_stream
    w.matvec(rows, xt.data_ptr(), xd, y.data_ptr(), "f32", stream=stream)
    one = x[np.arange(rows), at][:, None]
    got, cx, sx = y.double().cpu().numpy(), c[:, at].T, s[:, at // group].T
    assert np.array_equal(got, one * cx * sx), f"{(got != one * cx * sx).sum()} of {got.size} differ"
    # With zero points: c x and z x have up to 28 bits. At most three additions for each of them, one step of 2^-23 of the sums so far each.
    c, z = rng.integers(0, 16, (n_out, n_in)), rng.integers(0, 16, (n_out, groups))
    matrix(c, s, z, group, scales).matvec(rows, xt.data_ptr(), xd, y.data_ptr(), "f32", stream=stream)
    cx, zx = c[:, at].T, z[:, at // group].T
    err, tol = np.abs(y.double().cpu().numpy() - one * (cx - zx) * sx), 6 * 2.0 ** -23 * np.abs(one) * (cx + zx) * sx
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} off, worst {(err[tol > 0] / tol[tol > 0]).max():.1f} bounds"


@pytest.mark.parametrize("rows,n_out,n_in,takes", [(3, 70, 264, ("rows", 1)), (20, 70, 264, ("rows", 2)), (60, 70, 264, ("rows", 4)), (260, 4100, 264, ("tile", 8)), (4100, 1100, 264, ("tile", 4))])
def test_subnormal_fp16_inputs(rows, n_out, n_in, takes):
    # fp16 numbers below 2^-14 are numbers like others: whole multiples of 2^-24, so all sums are exact.
    rng = np.random.default_rng(rows)
    groups = -(-n_in // 64)
    c, z = rng.integers(0, 16, (n_out, n_in)), rng.integers(0, 16, (n_out, groups))
    w = matrix(c, np.full((n_out, groups), 0.5), z, 64, "f16")
    assert kernel(w, rows, n_in, n_out, "f16") == takes
    x = rng.integers(-1023, 1024, (rows, n_in)) * 2.0 ** -24
    xt, y = torch.from_numpy(x).half().cuda(), torch.empty((rows, n_out), device="cuda")
    w.matvec(rows, xt.data_ptr(), "f16", y.data_ptr(), "f32", stream=torch.cuda.current_stream().cuda_stream)
    want = x @ ((c - np.repeat(z, 64, 1)[:, :n_in]) * 0.5).T
    assert np.array_equal(y.double().cpu().numpy(), want)


@pytest.mark.parametrize("rows,n_out,n_in,takes", [(3, 70, 264, ("rows", 1)), (60, 70, 264, ("rows", 4)), (260, 8200, 264, ("tile", 8)), (4100, 1100, 264, ("tile", 4))])
def test_tiny_inputs(rows, n_out, n_in, takes):
    # bf16 numbers below 2^-126, and fp32 ones down to where bf16 summands end (2^-133); large scales make them visible.
    rng = np.random.default_rng(rows)
    groups = -(-n_in // 64)
    c = 1 << rng.integers(0, 4, (n_out, n_in))
    w = matrix(c, np.full((n_out, groups), 2.0 ** 60), np.zeros((n_out, groups), np.int64), 64, "f32")
    assert kernel(w, rows, n_in, n_out, "bf16") == takes
    at = rng.integers(0, n_in, rows)
    for xd, lowest, bits in (("bf16", -133, 0), ("bf16", -130, 3), ("bf16", -126, 7), ("f32", -110, 23), ("f32", -120, 23)):
        x = np.zeros((rows, n_in))
        x[np.arange(rows), at] = ((1 << bits) + rng.integers(0, 1 << bits, rows)) * 2.0 ** (lowest - bits) * rng.choice([-1, 1], rows)
        xt, y = torch.from_numpy(x.astype(np.float32)).to(tdt(xd)).cuda(), torch.empty((rows, n_out), device="cuda")
        assert np.array_equal(xt.double().cpu().numpy(), x)
        w.matvec(rows, xt.data_ptr(), xd, y.data_ptr(), "f32", stream=torch.cuda.current_stream().cuda_stream)
        cx = c[:, at].T * 2.0 ** 60
        err = np.abs(y.double().cpu().numpy() - x[np.arange(rows), at][:, None] * cx)
        assert (err <= (2.0 ** -133 * cx if lowest < -110 and xd == "f32" else 0)).all(), (xd, lowest)
