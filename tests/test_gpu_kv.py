"""The 8-bit key/value cache on the GPU against the fp64 definitions in tests/kv_reference.py: appended codes and exponents
exactly, attention within bounds counted from its roundings."""
import ctypes
import math

import numpy as np
import pytest

from tests import kv_reference as R
from tests.harness import torch_mod

pytestmark = pytest.mark.gpu

torch = None


@pytest.fixture(autouse=True, scope="module")
def _torch():
    global torch
    torch = torch_mod()
    assert torch.cuda.is_available()


def tdt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


class Env:
    """A cache, its pool (every byte NaN codes to begin with, so that nothing unwritten may matter) and its reference."""

    def __init__(self, *, heads=4, kv=2, hd=64, page=16, pages=64, seqs=4, layers=1, max_pages=None, seed=0):
        from delta_prefetched_ffn_amd import KVCache, kv_bytes
        shape = dict(n_layers=layers, n_heads=heads, n_kv_heads=kv, head_dim=hd, page_tokens=page, n_pages=pages)
        nc, ne = kv_bytes(**shape)
        self.codes = torch.full((nc,), 0x7F, dtype=torch.uint8, device="cuda")
        self.exps = torch.full((ne,), 100, dtype=torch.int8, device="cuda")
        self.kv = KVCache(**shape, max_seqs=seqs, max_pages=max_pages or pages, codes=self.codes.data_ptr(), exps=self.exps.data_ptr(),
                          keepalive=(self.codes, self.exps))
        self.heads, self.nkv, self.hd, self.page, self.layers = heads, kv, hd, page, layers
        self.ref = [[R.RefSeq(kv, hd, page) for _ in range(seqs)] for _ in range(layers)]
        self.rng = np.random.default_rng(seed)
        self.current = []

    def stream(self):
        return torch.cuda.current_stream().cuda_stream

    def extend(self, seqs, new):
        self.kv.extend(seqs, new, self.stream())
        self.current = list(zip(seqs, new))

    def rand(self, rows, n, dtype, scale=1.0):
        x = torch.from_numpy((self.rng.standard_normal((rows, n, self.hd)) * scale).astype(np.float32)).to(tdt(dtype))
        return x, x.double().numpy()

    def append(self, k, v, dtype, layer=0, strides=None):
        """k, v: (device tensor, fp64 values)."""
        kd, vd = k[0].cuda(), v[0].cuda()
        self.kv.append(layer, kd.data_ptr(), vd.data_ptr(), dtype, strides, self.stream())
        row = 0
        for s, n in self.current:
            if n:
                self.ref[layer][s].append(k[1][row:row + n], v[1][row:row + n])
            row += n

    def step(self, seqs, new, dtype="f32", layer=0, scale=1.0):
        self.extend(seqs, new)
        rows = sum(new)
        if rows:
            self.append(self.rand(rows, self.nkv, dtype, scale), self.rand(rows, self.nkv, dtype, scale), dtype, layer)

    def check_tokens(self, seqs, layer=0):
        for s in seqs:
            k, v = self.kv.read_tokens(layer, s)
            rk, rv = self.ref[layer][s].values()
            np.testing.assert_array_equal(k, rk.astype(np.float32), err_msg=f"seq {s} K")
            np.testing.assert_array_equal(v, rv.astype(np.float32), err_msg=f"seq {s} V")

    def attend(self, dtype, layer=0, window=0, sinks=0, held=None, scale=None, q_scale=1.0, layout="plain", lse=True, q=None):
        rows = sum(n for _, n in self.current)
        scale = 1 / math.sqrt(self.hd) if scale is None else scale
        qt, q64 = self.rand(rows, self.heads, dtype, q_scale) if q is None else q
        H, hd = self.heads, self.hd
        if layout == "plain":
            qd, out, st = qt.cuda(), torch.full((rows, H, hd), 7.0, dtype=qt.dtype, device="cuda"), None
        elif layout == "fused":       # q inside a wider projection output; out padded
            wide = torch.zeros((rows, H + 3, hd), dtype=qt.dtype, device="cuda")
            wide[:, 1:1 + H] = qt.cuda()
            qd = wide[:, 1:1 + H]
            hold = torch.full((rows, H, hd + 8), 7.0, dtype=qt.dtype, device="cuda")
            out = hold[:, :, :hd]
            st = (qd.stride(0), qd.stride(1), out.stride(0), out.stride(1))
        else:                         # heads outermost
            qd = qt.cuda().transpose(0, 1).contiguous().transpose(0, 1)
            out = torch.full((H, rows, hd), 7.0, dtype=qt.dtype, device="cuda").transpose(0, 1)
            st = (qd.stride(0), qd.stride(1), out.stride(0), out.stride(1))
        ls = torch.full((rows, H), 7.0, device="cuda") if lse else None
        self.kv.attend(layer, qd.data_ptr(), out.data_ptr(), dtype, st, scale=scale, window=window, sinks=sinks,
                       lse_ptr=ls.data_ptr() if lse else 0, stream=self.stream())
        got = out.double().cpu().numpy()
        if layout == "fused":
            assert bool((hold[:, :, hd:] == 7.0).all()), "written past the head dimension"
        row = 0
        for s, n in self.current:
            k, v = self.ref[layer][s].values()
            want, wl, terms, mag = R.attention(q64[row:row + n], k, v, len(k) - n, scale, window, sinks, None if held is None else held.get(s))
            g = got[row:row + n]
            nan = np.isnan(want)
            assert np.array_equal(np.isnan(g), nan), f"seq {s}: NaN in other places ({np.isnan(g).sum()} and {nan.sum()})"
            tol = R.bound(want, terms, mag, len(k), hd, dtype)
            err = np.abs(g - want)
            bad = ~nan & ~(err <= tol)
            assert not bad.any(), f"seq {s}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.where(bad, err / tol, 0)):.2f} bounds at {np.argwhere(bad)[0]}"
            if lse:
                gl = ls.double().cpu().numpy()[row:row + n]
                fin = np.isfinite(wl)
                assert np.array_equal(np.isneginf(gl), np.isneginf(wl)), f"seq {s}: lse of empty rows"
                assert np.array_equal(np.isnan(gl), np.isnan(wl)), f"seq {s}: lse NaN"
                assert (np.abs(gl - wl)[fin] <= R.lse_bound(wl, mag, len(k), hd)[fin]).all(), f"seq {s}: lse"
            row += n
        return out


# ------------------------------------------------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hd,page,kv", [(64, 16, 2), (128, 64, 3), (40, 32, 1), (80, 128, 2), (256, 16, 1), (200, 64, 2)])
def test_append_is_exact(dtype, hd, page, kv):
    e = Env(hd=hd, page=page, kv=kv, heads=kv, seed=hd + page)
    # one token, a few, across pages, ragged batches with an empty member, ends at every place of a group of four
    for seqs, new in (([0], [1]), ([0, 1], [2, 5]), ([2, 0, 1], [3 * page + 1, 0, page - 5]), ([0, 2], [page, 1]), ([1, 0], [2, 3])):
        e.step(seqs, new, dtype, scale=float(e.rng.choice([0.01, 1.0, 300.0])))
        e.check_tokens([0, 1, 2])


def test_append_special_values():
    e = Env(hd=64, page=16, kv=1, heads=1)
    rng = e.rng

    def put(x, y):
        e.extend([0], [len(x)])
        t = [torch.from_numpy(a.astype(np.float32).reshape(-1, 1, 64)) for a in (x, y)]
        e.append((t[0], t[0].double().numpy()), (t[1], t[1].double().numpy()), "f32")
        e.check_tokens([0])

    z = np.zeros((1, 64))
    put(z, z)                                                # a block of zeros: exponent -120
    put(z + 1e-30, z - 1e-38)                                # tiny: codes of the smallest exponents
    put(z + 448.0, np.nextafter(np.float32(448.0), np.float32(1e9)) + z)  # on and just above the border
    x = rng.standard_normal((2, 64))
    x[0, 3], x[1, 7], x[1, 9] = np.inf, np.nan, -np.inf
    put(x, -x)
    big = rng.standard_normal((3, 64)) * 1e30
    put(big, z.repeat(3, 0))
    put(z + 3.3e38, z - 3.3e38)                              # the largest exponents
    # ties to even, borders between binades and subnormals at a known exponent (0)
    v = np.concatenate([[448.0], np.arange(1, 32) * 2.0 ** -10, 1 + np.arange(32) / 16])
    put(v.reshape(1, 64), -v.reshape(1, 64))


def test_append_strided_rows_and_second_call():
    e = Env(hd=80, page=32, kv=3, heads=3)
    e.step([0], [37], "bf16")
    e.extend([0, 1], [9, 40])
    wide = torch.from_numpy(e.rng.standard_normal((49, 8, 80)).astype(np.float32)).bfloat16()
    k, v = wide[:, 1:4], wide[:, 5:8]
    dev = wide.cuda()
    kd, vd = dev[:, 1:4], dev[:, 5:8]
    for _ in range(3):   # a repeated call stores the same
        e.kv.append(0, kd.data_ptr(), vd.data_ptr(), "bf16", (kd.stride(0), kd.stride(1), vd.stride(0), vd.stride(1)), e.stream())
    row = 0
    for s, n in e.current:
        e.ref[0][s].append(k[row:row + n].double().numpy(), v[row:row + n].double().numpy())
        row += n
    e.check_tokens([0, 1])


# ------------------------------------------------------------------------------------------------------------- attend

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kv,hd,page", [(4, 4, 64, 16), (8, 2, 128, 64), (7, 1, 80, 32), (6, 3, 40, 128), (4, 1, 256, 16), (2, 2, 192, 64), (40, 1, 128, 32)])
def test_attend_single_tokens(dtype, heads, kv, hd, page):
    e = Env(heads=heads, kv=kv, hd=hd, page=page, pages=96, seed=heads * hd)
    e.step([0, 1, 2], [1, page + 3, 300], dtype)
    e.step([0, 1, 2], [1, 1, 1], dtype)
    e.attend(dtype)
    e.step([2, 0], [1, 1], dtype)
    e.attend(dtype, layout="fused", q_scale=4.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kv,hd,page,new,before", [
    (4, 4, 64, 16, 33, 0), (4, 2, 128, 64, 200, 0), (6, 2, 128, 32, 97, 131), (7, 1, 80, 16, 64, 1), (2, 2, 40, 128, 150, 50),
    (2, 1, 256, 16, 70, 5), (2, 1, 192, 32, 129, 0)])
def test_attend_prompts(dtype, heads, kv, hd, page, new, before):
    e = Env(heads=heads, kv=kv, hd=hd, page=page, pages=64, seed=new)
    if before:
        e.step([0, 1], [before, before // 2], dtype)
    e.step([1, 0, 2], [new // 3, new, 0], dtype)
    e.attend(dtype)
    e.attend(dtype, layout="heads", q_scale=3.0, lse=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 0), (32, 4), (33, 33), (100, 16), (7, 200), (1000, 3), (64, 70)])
@pytest.mark.parametrize("new", [1, 3, 90])
def test_window_and_first_tokens(dtype, window, sinks, new):
    e = Env(heads=4, kv=2, hd=64, page=32, pages=64, seed=window)
    e.step([0, 1], [290, 20], dtype)
    e.step([0, 1, 2], [new, max(1, new // 2), new], dtype)
    e.attend(dtype, window=window, sinks=sinks)


def test_long_sequence_is_split_and_joined():
    e = Env(heads=2, kv=1, hd=128, page=64, pages=160, seqs=2)
    e.step([0, 1], [9000, 37], "bf16")
    e.step([0, 1], [1, 1], "bf16")
    a = e.attend("bf16")
    e.attend("bf16", window=4096, sinks=4)
    e.attend("f32", q_scale=8.0)
    q = e.rand(2, 2, "bf16")
    runs = [e.attend("bf16", q=q).clone() for _ in range(4)]
    assert all(torch.equal(r, runs[0]) for r in runs), "not the same from run to run"
    assert a.isfinite().all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_scales_of_blocks_far_apart(dtype):
    # Value blocks of very different magnitude, the large ones hardly weighted: the unit of the sums has to follow.
    for page in (16, 64):
        e = Env(heads=2, kv=1, hd=64, page=page, pages=32, seed=page)
        mags = [1.0, 2.0 ** 6, 2.0 ** -9, 2.0 ** 8, 1e-3, 0.0, 5.0, 2.0 ** -14]
        rows = page * len(mags)
        e.extend([0], [rows])
        k = e.rng.standard_normal((rows, 1, 64))
        k[:, 0, 0] = np.repeat([-40 if m > 10 else 5 for m in mags], page)   # the large blocks get weight e^-5 or so
        v = e.rng.standard_normal((rows, 1, 64)) * np.repeat(mags, page)[:, None, None]
        kt, vt = (torch.from_numpy(x.astype(np.float32)) for x in (k, v))
        e.append((kt, kt.double().numpy()), (vt, vt.double().numpy()), "f32")
        q = np.zeros((rows, 2, 64), np.float32)
        q[:, :, 0] = 1.0
        q[:, :, 1:] = e.rng.standard_normal((rows, 2, 63)) * 0.1
        qt = torch.from_numpy(q).to(tdt(dtype))
        e.attend(dtype, q=(qt, qt.double().numpy()))
        e.extend([0], [0])
        e.extend([0], [1])
        e.append(e.rand(1, 1, "f32"), e.rand(1, 1, "f32"), "f32")
        e.attend(dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_scores_with_large_spread(dtype):
    # The running maximum rises by more than the lazy step many times, and early tokens end with weight zero.
    e = Env(heads=2, kv=2, hd=64, page=16, pages=32)
    rows = 180
    e.extend([0], [rows])
    k = e.rng.standard_normal((rows, 2, 64)) * 0.1
    k[:, :, 0] = np.linspace(-60, 60, rows)[:, None]
    kt = torch.from_numpy(k.astype(np.float32))
    e.append((kt, kt.double().numpy()), e.rand(rows, 2, "f32"), "f32")
    q = e.rng.standard_normal((rows, 2, 64)).astype(np.float32)
    q[:, 0, 0], q[:, 1, 0] = 30.0, -30.0
    qt = torch.from_numpy(q).to(tdt(dtype))
    e.attend(dtype, q=(qt, qt.double().numpy()))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("page", [16, 64])
def test_nan_and_infinity_stay_with_the_rows_that_see_them(dtype, page):
    e = Env(heads=2, kv=1, hd=64, page=page, pages=32)
    e.step([0], [70], "f32")
    e.extend([0], [60])
    k, v = (e.rng.standard_normal((60, 1, 64)).astype(np.float32) for _ in range(2))
    v[20, 0, 5] = np.nan          # seen by rows 20 .. 20 + window - 1 only
    v[41, 0, 9] = -np.inf         # stored as the block's lowest value
    k[30, 0, 0] = np.nan          # rows that see it are NaN
    kt, vt = torch.from_numpy(k), torch.from_numpy(v)
    e.append((kt, kt.double().numpy()), (vt, vt.double().numpy()), "f32")
    e.check_tokens([0])
    e.attend(dtype, window=9)
    e.attend(dtype)
    e.attend(dtype, window=3, sinks=2)
    q = e.rand(60, 2, dtype)
    q[0][7, 1, 0] = float("inf")  # a row of its own: NaN or not by its own formula, the others untouched
    q[0][9, 0, 3] = float("nan")
    e.attend(dtype, window=20, q=(q[0], q[0].double().numpy()))


def test_dropped_pages_and_rows_that_see_nothing():
    e = Env(heads=4, kv=2, hd=64, page=16, pages=64)
    e.step([0, 1], [200, 200], "bf16")
    # a cache restored without its past: rows see only what is held
    pages = e.kv.pages(0)
    keep = 8
    gone = np.array([-1] * keep + pages[keep:].tolist(), np.int32)
    e.kv.free(0)
    e.kv.adopt(0, gone, 200, e.stream())
    held = {0: np.arange(1000) >= keep * 16}
    e.ref[0][0].codes[:keep * 16] = np.nan
    e.step([0, 1], [3, 2], "bf16")
    e.attend("bf16", held=held)
    e.attend("f32", held=held, window=130, sinks=20)
    # nothing held but the new tokens' page, and they are hidden: window 1 with every page dropped
    assert e.kv.evict(1, 16, 0, e.stream()) == 11
    held[1] = np.arange(1000) >= 11 * 16
    e.step([1], [1], "bf16")
    e.attend("bf16", held=held)
    # rows with no visible token at all
    e.kv.free(2)
    p = e.kv.pages(1)
    e.kv.free(1)
    e.kv.adopt(2, [-1] * len(p), len(p) * 16, e.stream())
    e.extend([2, 0], [2, 1])
    e.ref[0][2] = R.RefSeq(2, 64, 16)
    e.ref[0][2].codes = np.full((len(p) * 16, 2, 2, 64), np.nan)
    e.ref[0][2].exps = np.zeros((len(p), 2, 2), dtype=np.int64)
    e.append(e.rand(3, 2, "bf16"), e.rand(3, 2, "bf16"), "bf16")
    e.attend("bf16", held={2: np.arange(1000) >= len(p) * 16, 0: held[0]})


def test_empty_rows_are_zero():
    # adopt with every page dropped, then a step whose queries lie in the past: no visible token, output 0, lse -inf
    from delta_prefetched_ffn_amd import KVCache
    e = Env(heads=4, kv=2, hd=64, page=16, pages=8)
    e.step([0], [16], "bf16")
    e.kv.evict(0, 1, 0, e.stream())
    e.kv.extend([0], [0], e.stream())
    q = torch.zeros((1, 4, 64), device="cuda")
    e.kv.attend(0, q.data_ptr(), q.data_ptr(), "f32", scale=1.0, stream=e.stream())   # no rows: nothing to do
    # window 4 hides every held token of a page-wide gap: rows at the start of a page see only themselves
    e.step([0], [1], "bf16")
    e.attend("bf16", held={0: np.arange(17) >= 16})
    torch.cuda.synchronize()
    assert KVCache is not None


# --------------------------------------------------------------------------------------------------------- pages, order

@pytest.mark.parametrize("mode", ["share", "copy"])
def test_forks_keep_their_own_tokens(mode):
    e = Env(heads=4, kv=2, hd=80, page=32, pages=40, layers=3)

    def both(seqs, new):
        e.extend(seqs, new)
        for layer in range(3):
            e.append(e.rand(sum(new), 2, "f32"), e.rand(sum(new), 2, "f32"), "f32", layer)

    both([0], [75])
    for dst, n in ((1, 75), (2, 70), (3, 64)):
        e.kv.fork(0, dst, n, mode, e.stream())
        for layer in range(3):
            r = e.ref[layer][dst]
            r.codes, r.exps = e.ref[layer][0].codes[:n].copy(), e.ref[layer][0].exps[:-(-n // 32)].copy()
    both([1, 0, 2, 3], [4, 1, 3, 2])
    both([2, 3], [40, 1])
    for layer in range(3):
        e.check_tokens([0, 1, 2, 3], layer)
        e.attend("f32", layer)
    # shorter again, then packed: contents stay
    e.kv.trim(0, 40)
    e.kv.free(3)
    for layer in range(3):
        e.ref[layer][0].codes = e.ref[layer][0].codes[:40]
        e.ref[layer][0].exps = e.ref[layer][0].exps[:2]
    e.kv.compact(e.stream())
    used = sorted({int(p) for s in (0, 1, 2) for p in e.kv.pages(s)})
    assert used == list(range(len(used)))
    for layer in range(3):
        e.check_tokens([0, 1, 2], layer)
    both([0, 2], [30, 1])
    for layer in range(3):
        e.check_tokens([0, 1, 2], layer)
        e.attend("bf16", layer)


def test_compact_moves_many_pages():
    e = Env(heads=1, kv=1, hd=64, page=16, pages=1200, seqs=3, max_pages=600)
    for _ in range(20):   # pages of three sequences interleaved
        e.step([0, 1, 2], [480, 160, 7], "f16")
    e.kv.free(0)
    assert e.kv.compact(e.stream()) > 0
    e.ref[0][0] = R.RefSeq(1, 64, 16)
    e.check_tokens([1, 2])
    e.step([2, 1], [1, 1], "f16")
    e.attend("f16")


def test_offsets_past_32_bits():
    # A pool above 4 GiB whose last pages are the ones in use.
    e = Env(heads=2, kv=2, hd=128, page=64, pages=140000)
    assert e.codes.numel() > (1 << 32)
    e.kv.adopt(0, list(range(139999, 139990, -1)), 0, e.stream())
    e.step([0], [530], "bf16")
    e.check_tokens([0])
    e.step([0], [1], "bf16")
    e.attend("bf16")
    e.kv.fork(0, 1, 500, "copy", e.stream())
    assert e.kv.compact(e.stream()) == 9
    e.check_tokens([0])


def test_another_stream_and_graph_replays():
    e = Env(heads=4, kv=2, hd=128, page=32, pages=64)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        e.step([0, 1], [500, 90], "bf16")
        e.step([0, 1], [1, 1], "bf16")
        e.attend("bf16")
        e.check_tokens([0, 1])
        q = torch.randn((2, 4, 128), device="cuda").bfloat16()
        k, v = (torch.randn((2, 2, 128), device="cuda").bfloat16() for _ in range(2))
        out = torch.zeros_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st = torch.cuda.current_stream().cuda_stream
        e.kv.append(0, k.data_ptr(), v.data_ptr(), "bf16", None, st)
        e.kv.attend(0, q.data_ptr(), out.data_ptr(), "bf16", scale=0.1, stream=st)
    for i in range(4):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda"))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        e.kv.append(0, k.data_ptr(), v.data_ptr(), "bf16", None, e.stream())
        e.kv.attend(0, q.data_ptr(), out.data_ptr(), "bf16", scale=0.1, stream=e.stream())
        torch.cuda.synchronize()
        assert torch.equal(got, out), i


def test_refusals_with_a_device():
    from delta_prefetched_ffn_amd import KVCache, NPError
    from delta_prefetched_ffn_amd import binding as B
    e = Env()
    e.extend([0], [3])
    host = np.zeros(4096, np.float32)
    at = (host.ctypes.data + 15) // 16 * 16
    x = torch.zeros(4096, device="cuda")
    for call in (lambda: e.kv.append(0, at, x.data_ptr(), "f32"), lambda: e.kv.append(0, x.data_ptr(), at, "f32"),
                 lambda: e.kv.attend(0, at, x.data_ptr(), "f32", scale=1.0), lambda: e.kv.attend(0, x.data_ptr(), at, "f32", scale=1.0),
                 lambda: e.kv.attend(0, x.data_ptr(), x.data_ptr(), "f32", scale=1.0, lse_ptr=at),
                 lambda: KVCache(n_layers=1, n_heads=1, n_kv_heads=1, head_dim=64, page_tokens=16, n_pages=1, max_seqs=1, max_pages=1, codes=at, exps=x.data_ptr()),
                 lambda: KVCache(n_layers=1, n_heads=1, n_kv_heads=1, head_dim=64, page_tokens=16, n_pages=1, max_seqs=1, max_pages=1, codes=x.data_ptr(), exps=at),
                 lambda: KVCache(n_layers=1, n_heads=1, n_kv_heads=1, head_dim=64, page_tokens=16, n_pages=1, max_seqs=1, max_pages=1),
                 lambda: KVCache(n_layers=1, n_heads=1, n_kv_heads=1, head_dim=64, page_tokens=16, n_pages=1, max_seqs=1, max_pages=1, device=99, codes=x.data_ptr(), exps=x.data_ptr())):
        with pytest.raises(NPError) as err:
            call()
        assert err.value.status == B.NP_EINVAL
    e.append(e.rand(3, 2, "f32"), e.rand(3, 2, "f32"), "f32")   # still usable
    e.check_tokens([0])
    e.attend("f32")


# ------------------------------------------------------------------------------------------------- many rows, many heads
# Enough heads and rows that prompts run in large tiles (the tests above stay below: few workgroups).

TILES = [("bf16", 128), ("f16", 128), ("bf16", 64), ("f32", 64), ("f16", 80), ("bf16", 40), ("bf16", 192), ("f16", 256)]


@pytest.mark.parametrize("dtype,hd", TILES)
@pytest.mark.parametrize("group,new,before,window,sinks", [(1, 300, 0, 0, 0), (2, 170, 77, 0, 0), (1, 290, 0, 50, 3), (1, 257, 130, 64, 70), (3, 129, 5, 1, 0)])
def test_prompt_tiles(dtype, hd, group, new, before, window, sinks):
    e = Env(heads=64 * group, kv=64, hd=hd, page=32, pages=40, seqs=3, seed=new)
    if before:
        e.step([0, 1], [before, before // 3], dtype)
    e.step([0, 2, 1], [new, 0, 1], dtype)     # a prompt beside a single token: both kernels in one call
    e.attend(dtype, window=window, sinks=sinks, layout="fused")


@pytest.mark.parametrize("dtype,hd", TILES)
def test_prompt_tiles_nan_scales_and_dropped_pages(dtype, hd):
    # Value blocks of very different size, NaN values that only some rows see, NaN codes in every unwritten byte.
    e = Env(heads=64, kv=64, hd=hd, page=16, pages=40, seqs=2)
    rows = 260
    e.extend([0], [rows])
    mags = np.repeat([1.0, 2.0 ** 6, 2.0 ** -9, 2.0 ** 8, 1e-3, 0.0, 5.0, 2.0 ** -14, 1.0, 1.0, 2.0 ** -20, 30.0, 1.0, 1.0, 1.0, 1.0, 1.0], 16)[:rows]
    k = e.rng.standard_normal((rows, 64, hd)) * 0.3
    k[:, :, 0] = np.where(mags > 10, -40, 3)[:, None]
    v = e.rng.standard_normal((rows, 64, hd)) * mags[:, None, None]
    v[40, ::7, 5], v[201, 3, hd - 1], k[100, 9, 1] = np.nan, np.nan, np.nan
    v[150, 11, 2] = np.inf
    kt, vt = (torch.from_numpy(x.astype(np.float32)) for x in (k, v))
    e.append((kt, kt.double().numpy()), (vt, vt.double().numpy()), "f32")
    q = e.rng.standard_normal((rows, 64, hd)).astype(np.float32) * 0.3
    q[:, :, 0] = 1.0
    qt = torch.from_numpy(q).to(tdt(dtype))
    e.attend(dtype, q=(qt, qt.double().numpy()), window=23, sinks=2, scale=1.0)
    e.attend(dtype, q=(qt, qt.double().numpy()), scale=1.0)
    # restored without its first pages
    e.kv.free(0)
    e.kv.adopt(0, [-1] * 5 + list(range(20)), 80, e.stream())
    e.ref[0][0] = R.RefSeq(64, hd, 16)
    e.ref[0][0].codes, e.ref[0][0].exps = np.full((80, 2, 64, hd), np.nan), np.zeros((5, 2, 64), dtype=np.int64)
    e.step([0], [250], "f32")
    e.attend(dtype, held={0: np.arange(1000) >= 80}, window=100, sinks=10)
    e.attend(dtype, held={0: np.arange(1000) >= 80}, layout="heads")


def test_prompt_tiles_are_the_same_from_run_to_run():
    e = Env(heads=64, kv=64, hd=128, page=64, pages=12, seqs=1)
    e.step([0], [300], "bf16")
    q = e.rand(300, 64, "bf16")
    runs = [e.attend("bf16", q=q, lse=False).clone() for _ in range(3)]
    assert all(torch.equal(r, runs[0]) for r in runs)


@pytest.mark.parametrize("kv", [2, 64])
def test_windows_and_first_tokens_up_to_the_largest_number(kv):
    e = Env(heads=kv, kv=kv, hd=64, page=16, pages=24, seqs=1)
    e.step([0], [20], "bf16")
    e.step([0], [280], "bf16")
    q = e.rand(280, kv, "bf16")
    full = e.attend("bf16", q=q, lse=False).clone()
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 28, 1), (7, 2 ** 31 - 1), (300, 0)):
        assert torch.equal(e.attend("bf16", q=q, window=window, sinks=sinks, lse=False), full), (window, sinks)


# ---------------------------------------------------------------------------------------- pages that are not the sequence's
# Where a sequence holds no page (dropped, or past its last token) the kernels have page 0's address at hand. Nothing of it
# may matter: here it belongs to nobody or to another sequence, with finite codes at a scale far from the rows' own.

def page_zero_of_nobody(e):
    """Page 0 as an unwritten pool may hold it: the largest finite codes at the largest exponent, in no sequence."""
    assert e.layers == 1
    e.codes[:e.codes.numel() // e.kv.n_pages] = 0x7E
    e.exps[:2 * e.nkv] = 120


@pytest.mark.parametrize("dtype,hd", TILES)
@pytest.mark.parametrize("new", [260, 129])
def test_prompt_tiles_end_inside_a_step(dtype, hd, new):
    e = Env(heads=64, kv=64, hd=hd, page=16, pages=24, seqs=2, seed=new)
    page_zero_of_nobody(e)
    e.kv.adopt(0, list(range(1, 20)), 0, e.stream())
    e.step([0], [new], dtype)
    e.attend(dtype)
    e.attend(dtype, window=100, sinks=3)


@pytest.mark.parametrize("dtype,hd", TILES)
def test_prompt_tiles_with_values_of_zero(dtype, hd):
    # The last page's values are zero, and one head's everywhere: the unit of the sums goes far below page 0's scale.
    e = Env(heads=64, kv=64, hd=hd, page=16, pages=24, seqs=2)
    e.step([1], [16], "f32")             # another sequence's ordinary tokens in page 0
    assert e.kv.pages(1).tolist() == [0]
    e.extend([0], [260])
    k, v = (e.rng.standard_normal((260, 64, hd)).astype(np.float32) for _ in range(2))
    v[256:] = 0
    v[:, 5] = 0
    kt, vt = torch.from_numpy(k), torch.from_numpy(v)
    e.append((kt, kt.double().numpy()), (vt, vt.double().numpy()), "f32")
    e.attend(dtype)


@pytest.mark.parametrize("dtype,hd", TILES)
def test_prompt_tiles_behind_dropped_pages(dtype, hd):
    e = Env(heads=64, kv=64, hd=hd, page=16, pages=32, seqs=1)
    page_zero_of_nobody(e)
    e.kv.adopt(0, [-1] * 9 + list(range(1, 23)), 144, e.stream())
    e.ref[0][0].codes, e.ref[0][0].exps = np.full((144, 2, 64, hd), np.nan), np.zeros((9, 2, 64), dtype=np.int64)
    e.step([0], [330], "f32")
    held = {0: np.arange(1000) >= 144}
    e.attend(dtype, held=held)
    e.attend(dtype, held=held, window=300, sinks=70)


@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("f16", 128), ("f32", 64), ("f32", 128), ("bf16", 192), ("f16", 256)])
@pytest.mark.parametrize("page", [16, 64])
def test_tokens_behind_dropped_pages(dtype, hd, page):
    # Whole pieces of 32 tokens are not held, and no window hides them.
    e = Env(heads=4, kv=2, hd=hd, page=page, pages=32, seqs=1)
    page_zero_of_nobody(e)
    e.kv.adopt(0, [-1] * 9 + list(range(1, 20)), 9 * page, e.stream())
    e.ref[0][0].codes, e.ref[0][0].exps = np.full((9 * page, 2, 2, hd), np.nan), np.zeros((9, 2, 2), dtype=np.int64)
    held = {0: np.arange(2000) >= 9 * page}
    for new in (1, 3, 40):
        e.step([0], [new], dtype)
        e.attend(dtype, held=held)
        e.attend(dtype, held=held, window=8 * page, sinks=page + 3)
    # and pages dropped behind a window that the next call does not use
    gone = e.kv.evict(0, 16, 0, e.stream())
    held = {0: np.arange(2000) >= (9 + gone) * page}
    e.step([0], [1], dtype)
    e.attend(dtype, held=held)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,new", [(1, 1), (1, 20), (64, 400)])
def test_scores_of_minus_infinity_beside_finite_ones(dtype, heads, new):
    # q . k of most tokens overflows to -inf: their weight is 0, and the 32 tokens with finite scores make the row. The
    # reference leaves the others out (in 64 bits they weigh exp(-1e40) = 0).
    e = Env(heads=heads, kv=heads, hd=64, page=16, pages=48, seqs=1)
    total = 500
    k, v = (e.rng.standard_normal((total, heads, 64)).astype(np.float32) for _ in range(2))
    finite = (np.arange(2000) >= 96) & (np.arange(2000) < 128)
    k[:, :, 0] = np.where(finite[:total], 0.0, -224.0)[:, None]
    for lo, hi in ((0, total - new), (total - new, total)):
        e.extend([0], [hi - lo])
        kt, vt = torch.from_numpy(k[lo:hi]), torch.from_numpy(v[lo:hi])
        e.append((kt, kt.double().numpy()), (vt, vt.double().numpy()), "f32")
    q = e.rng.standard_normal((new, heads, 64)).astype(np.float32)
    q[:, :, 0] = 2.0 ** 126
    qt = torch.from_numpy(q).to(tdt(dtype))
    e.attend(dtype, q=(qt, qt.double().numpy()), held={0: finite}, scale=1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,new", [(1, 1), (64, 300)])
def test_a_row_whose_scores_are_all_minus_infinity_is_nan(dtype, heads, new):
    e = Env(heads=heads, kv=heads, hd=64, page=16, pages=48, seqs=1)
    e.extend([0], [100])
    k = np.abs(e.rng.standard_normal((300, heads, 64))).astype(np.float32) + 1
    kt = torch.from_numpy(k[:100])
    e.append((kt, kt.double().numpy()), e.rand(100, heads, "f32"), "f32")
    e.extend([0], [new])
    kt = torch.from_numpy(k[:new])
    e.append((kt, kt.double().numpy()), e.rand(new, heads, "f32"), "f32")
    q, _ = e.rand(new, heads, dtype)
    q[0, 0, 3] = -float("inf")
    out = e.attend(dtype, q=(q, q.double().numpy()))
    assert bool(out[0, 0].isnan().all()) and int(out.isnan().sum()) == 64


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("prompt", [True, False])
def test_small_weights_of_many_tokens_count(dtype, hd, prompt):
    # One dominant first token whose value is 0; each later token weighs 2^-25.6 of it, so together they make the output.
    # A 16-bit weight is off by 2^-11 of itself or, at the bottom of fp16's range, by 2^-32 of the running largest weight
    # (half of 2^-24, the weights being held times 2^7 at least).
    heads, n, seqs = (32, 4100, 1) if prompt else (64, 2000, 8)
    e = Env(heads=heads, kv=heads, hd=hd, page=64, pages=300, seqs=seqs)
    k, v = torch.zeros((n, heads, hd)), torch.rand((n, heads, hd), generator=torch.Generator().manual_seed(1)) + 0.5
    k[0, :, 0], v[0] = 16.0, 0.0
    kd, vd = k.cuda(), v.cuda()
    for s in range(seqs):
        e.kv.extend([s], [n], e.stream())
        e.kv.append(0, kd.data_ptr(), vd.data_ptr(), "f32", None, e.stream())
    new = n if prompt else seqs
    if not prompt:      # the rows' own tokens: another one of the kind
        e.kv.extend(list(range(seqs)), [1] * seqs, e.stream())
        own = kd[1:2].repeat(seqs, 1, 1), vd[1:2].repeat(seqs, 1, 1)
        e.kv.append(0, own[0].data_ptr(), own[1].data_ptr(), "f32", None, e.stream())
    scale, w = 25.6 * math.log(2) / 16, 2.0 ** -25.6
    q = torch.zeros((new, heads, hd))
    q[:, :, 0] = 1.0
    qd = q.to(tdt(dtype)).cuda()
    out = torch.empty_like(qd)
    e.kv.attend(0, qd.data_ptr(), out.data_ptr(), dtype, scale=scale, stream=e.stream())
    got = out.double().cpu().numpy()
    _, val = e.kv.read_tokens(0, 0)
    total = np.cumsum(val.astype(np.float64), axis=0)
    if not prompt:
        total = np.repeat(total[-1:], seqs, axis=0)
    count = np.arange(n)[:, None, None] if prompt else n
    want = w * total / (1 + w * count)
    tiny = 2.0 ** -24 if dtype == "f16" else 2.0 ** -126
    weights = 2.0 ** -24 if dtype == "f32" else 2.0 ** -11
    scores, sums = 16 * 26 * 2.0 ** -24, 2 * (n + 16) * 2.0 ** -24   # as in kv_reference.bound, one product a score
    bottom = 0 if dtype == "f32" else 2.0 ** -32
    tol = R.U[dtype] * np.abs(want) * 1.01 + 2 * (want * (weights + 2 * scores + sums) + bottom * total) + tiny
    err = np.abs(got - want)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.2f} bounds, {np.max(err[-1] / want[-1]):.3f} of the last row"


# ------------------------------------------------------------------------------------------------ which kernels are reached

class _KernelNode(ctypes.Structure):   # hipKernelNodeParams
    _fields_ = [("block", ctypes.c_uint32 * 3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", ctypes.c_uint32 * 3),
                ("args", ctypes.c_void_p), ("lds", ctypes.c_uint32)]


def kernels_of(call):
    """Names of the kernels that `call` launches: from a captured graph that is never run."""
    hip = ctypes.CDLL("libamdhip64.so.7")
    hip.hipKernelNameRefByPtr.restype = ctypes.c_char_p
    g = torch.cuda.CUDAGraph(keep_graph=True)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(torch.cuda.current_stream().cuda_stream)
    graph, n = ctypes.c_void_p(g.raw_cuda_graph()), ctypes.c_size_t()
    assert hip.hipGraphGetNodes(graph, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * n.value)()
    assert hip.hipGraphGetNodes(graph, nodes, ctypes.byref(n)) == 0
    names = []
    for node in nodes:
        p = _KernelNode()
        assert hip.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        names.append(hip.hipKernelNameRefByPtr(ctypes.c_void_p(p.func), None).decode())
    return names


def attention_kernels(heads, kv, hd, page, before, new, dtype, window=0, sinks=0):
    e = Env(heads=heads, kv=kv, hd=hd, page=page, pages=sum(-(-(b + n) // page) for b, n in zip(before, new)) + 1, seqs=len(new))
    seqs = list(range(len(new)))
    e.kv.extend(seqs, before, e.stream())
    e.kv.extend(seqs, new, e.stream())
    q = torch.empty((sum(new), heads, hd), dtype=tdt(dtype), device="cuda")
    names = kernels_of(lambda s: e.kv.attend(0, q.data_ptr(), q.data_ptr(), dtype, scale=1.0, window=window, sinks=sinks, stream=s))
    return ["tile" if "k_attn_tile" in n else "rows" if "k_attn_rows" in n else n for n in names]


@pytest.mark.parametrize("dtype,hd", TILES)
def test_prompt_tests_reach_the_large_tiles(dtype, hd):
    # The shapes of the tests above that are there for k_attn_tile, with single tokens beside a prompt in k_attn_rows.
    for group, new, before, window, sinks in ((1, 300, 0, 0, 0), (2, 170, 77, 0, 0), (1, 290, 0, 50, 3), (1, 257, 130, 64, 70), (3, 129, 5, 1, 0)):
        got = attention_kernels(64 * group, 64, hd, 32, [before, before // 3, 0], [new, 1, 0], dtype, window, sinks)
        assert got == ["tile", "rows"], (group, new, before, window)
    for before, new, window, sinks in ((0, 260, 0, 0), (0, 260, 100, 3), (0, 260, 23, 2), (144, 330, 0, 0), (144, 330, 300, 70), (100, 400, 0, 0),
                                       (100, 300, 0, 0), (80, 250, 100, 10)):
        assert attention_kernels(64, 64, hd, 16, [before], [new], dtype, window, sinks) == ["tile"], (before, new, window)


def test_few_rows_reach_the_row_tiles():
    for dtype in ("f32", "bf16", "f16"):
        assert attention_kernels(4, 2, 64, 16, [153], [40], dtype) == ["rows"]
        assert attention_kernels(64, 64, 128, 64, [2000] * 8, [1] * 8, dtype) == ["rows"]
    assert attention_kernels(32, 32, 128, 64, [0], [1024], "f32") == ["rows"]   # q's three summands leave no room for tiles


@pytest.mark.parametrize("dtype,hd", [("bf16", 128), ("f16", 64), ("f32", 64), ("bf16", 256)])
@pytest.mark.parametrize("heads,new,kernel", [(2, 32, "rows"), (64, 272, "tile")])
def test_rows_that_see_nothing(dtype, hd, heads, new, kernel):
    # A step's rows see their own tokens at least. A graph of it that is replayed after pages were dropped may have rows
    # that see none: 0, lse -inf. Here the first page only is left, and the window hides it from all but the first rows.
    e = Env(heads=heads, kv=heads, hd=hd, page=16, pages=24, seqs=2)
    page_zero_of_nobody(e)
    e.kv.adopt(0, list(range(1, 18)), 0, e.stream())
    e.step([0], [new], dtype)
    assert attention_kernels(heads, heads, hd, 16, [0], [new], dtype, 5) == [kernel]
    qt, q64 = e.rand(new, heads, dtype)
    q = qt.cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((new, heads), 7.0, device="cuda")

    def attend(window, sinks):
        e.kv.attend(0, q.data_ptr(), out.data_ptr(), dtype, scale=0.1, window=window, sinks=sinks, lse_ptr=lse.data_ptr(), stream=torch.cuda.current_stream().cuda_stream)

    attend(5, 0)
    torch.cuda.synchronize()
    graphs = []
    for window, sinks in ((5, 0), (0, 0), (5, 16)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            attend(window, sinks)
    k, v = e.ref[0][0].values()
    for sinks, held in ((16, np.arange(new) < 16), (0, np.zeros(new, bool))):
        e.kv.evict(0, 1, sinks)
        e.kv.extend([1], [1], e.stream())          # writes the page table
        for g, (window, first) in zip(graphs, ((5, 0), (0, 0), (5, 16))):
            want, wl, terms, mag = R.attention(q64, k, v, 0, 0.1, window, first, held)
            for _ in range(2):
                out.fill_(7.0)
                lse.fill_(7.0)
                g.replay()
                torch.cuda.synchronize()
                got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
                assert (np.abs(got - want) <= R.bound(want, terms, mag, new, hd, dtype)).all()
                assert np.array_equal(np.isneginf(gl), np.isneginf(wl)) and not np.isnan(gl).any()
                fin = np.isfinite(wl)
                assert (np.abs(gl[fin] - wl[fin]) <= R.lse_bound(wl, mag, new, hd)[fin]).all()
                assert (got[np.isneginf(wl)] == 0).all()
    assert np.isneginf(wl).all()                   # the last round: nothing held at all


@pytest.mark.parametrize("dtype,hd", [("f32", 64), ("bf16", 128), ("f16", 64), ("bf16", 256), ("f16", 192)])
@pytest.mark.parametrize("heads,new,kernel", [(2, 1, "rows"), (2, 3, "rows"), (64, 300, "tile")])
def test_values_that_no_row_sees_do_not_set_the_scale(dtype, hd, heads, new, kernel):
    # Behind the first tokens and before the window lie pages whose values are 2^80 larger; no row of the call sees them.
    e = Env(heads=heads, kv=heads, hd=hd, page=16, pages=34, seqs=1)
    assert attention_kernels(heads, heads, hd, 16, [200], [new], dtype, 89, 4) == [kernel]
    k, v = (e.rng.standard_normal((200 + new, heads, hd)).astype(np.float32) for _ in range(2))
    v[16:112] *= 2.0 ** 80                # row 200 sees tokens 112 on
    for lo, hi in ((0, 200), (200, 200 + new)):
        e.extend([0], [hi - lo])
        kt, vt = torch.from_numpy(k[lo:hi]), torch.from_numpy(v[lo:hi])
        e.append((kt, kt.double().numpy()), (vt, vt.double().numpy()), "f32")
    e.attend(dtype, window=89, sinks=4)


@pytest.mark.parametrize("dtype,hd", [("f32", 64), ("bf16", 128), ("f16", 64), ("bf16", 256), ("f16", 192)])
@pytest.mark.parametrize("heads,new,kernel", [(2, 150, "rows"), (64, 300, "tile")])
def test_later_values_of_another_scale_leave_earlier_rows_alone(dtype, hd, heads, new, kernel):
    # Rows 0 .. 95 share tiles with rows that see values 2^80 larger, and do not see them.
    e = Env(heads=heads, kv=heads, hd=hd, page=16, pages=24, seqs=1)
    assert attention_kernels(heads, heads, hd, 16, [0], [new], dtype) == [kernel]
    e.extend([0], [new])
    k, v = (e.rng.standard_normal((new, heads, hd)).astype(np.float32) for _ in range(2))
    v[96:130] *= 2.0 ** 80
    kt, vt = torch.from_numpy(k), torch.from_numpy(v)
    e.append((kt, kt.double().numpy()), (vt, vt.double().numpy()), "f32")
    q, q64 = e.rand(new, heads, dtype)
    out = torch.empty((new, heads, hd), dtype=tdt(dtype), device="cuda")
    qd = q.cuda()
    e.kv.attend(0, qd.data_ptr(), out.data_ptr(), dtype, scale=1 / math.sqrt(hd), stream=e.stream())
    rk, rv = e.ref[0][0].values()
    want, _, terms, mag = R.attention(q64[:96], rk[:96], rv[:96], 0, 1 / math.sqrt(hd))
    err = np.abs(out.double().cpu().numpy()[:96] - want)
    tol = R.bound(want, terms, mag, 96, hd, dtype)
    assert (err <= tol).all(), f"worst {np.max(err / tol):.2f} bounds"
