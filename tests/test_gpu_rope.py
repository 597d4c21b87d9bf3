"""Rotary positions, the norms of queries and keys in the same pass, and both on the way into the cache, on the GPU against the
fp64 definitions in tests/rope_reference.py."""
import ctypes

import numpy as np
import pytest

from tests import kv_reference as KR
from tests import rope_reference as R
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


def stream():
    return torch.cuda.current_stream().cuda_stream


def rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(tdt(dtype))


def weights(rng, hd):
    return (1 + 0.3 * rng.standard_normal(hd)).astype(np.float32)


def same(got, want, mag, dtype, what=""):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN in other places"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    fin = np.isfinite(want)
    err, tol = np.abs(got - want)[fin], R.bound(want, mag, dtype)[fin]
    assert (err <= tol).all(), f"{what}: {(err > tol).sum()} off, worst {(err / tol).max():.2f} bounds"


CASES = [  # heads, kv, hd, rot, layout
    (4, 4, 64, 64, "half"), (8, 2, 128, 128, "half"), (3, 1, 128, 128, "interleaved"), (5, 5, 128, 32, "half"), (6, 3, 80, 80, "half"),
    (7, 1, 40, 40, "half"), (2, 2, 40, 20, "half"), (4, 2, 96, 26, "half"), (9, 3, 256, 256, "half"), (1, 1, 256, 64, "interleaved"),
    (4, 4, 8, 8, "half"), (3, 3, 8, 2, "interleaved"), (33, 11, 24, 16, "half"), (2, 1, 200, 198, "half"), (2, 1, 72, 70, "interleaved"), (40, 8, 128, 64, "interleaved"),
    (2, 2, 128, 0, "half"), (16, 1, 48, 48, "half")]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kv,hd,rot,layout", CASES)
def test_rows_heads_and_layouts(dtype, heads, kv, hd, rot, layout):
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(heads * 1000 + hd + rot)
    rope = Rope(head_dim=hd, rot_dim=rot, layout=layout, amplitude=1.25)
    f = R.freqs(rot)
    for rows, norm_q, norm_k in ((1, True, True), (3, False, True), (17, True, False), (130, False, False), (1500, True, True)):
        q, k = rand(rng, (rows, heads, hd), dtype), rand(rng, (rows, kv, hd), dtype, 3.0)
        wq, wk = weights(rng, hd), weights(rng, hd)
        pos = rng.integers(0, 40000, rows).astype(np.int32)
        pos[0] = 0
        dq, dk, dp = q.cuda(), k.cuda(), torch.from_numpy(pos).cuda()
        dwq, dwk = torch.from_numpy(wq).cuda(), torch.from_numpy(wk).cuda()
        oq, ok = torch.full_like(dq, 7), torch.full_like(dk, 7)
        rope.apply(rows, dq.data_ptr(), oq.data_ptr(), heads, dtype, k_ptr=dk.data_ptr(), k_out_ptr=ok.data_ptr(), n_kv_heads=kv, positions_ptr=dp.data_ptr(),
                   q_weight_ptr=dwq.data_ptr() if norm_q else 0, k_weight_ptr=dwk.data_ptr() if norm_k else 0, eps=1e-5, stream=stream())
        eps = float(np.float32(1e-5))
        for o, x, w in ((oq, q, wq if norm_q else None), (ok, k, wk if norm_k else None)):
            want, mag = R.turned(x.double().numpy(), pos, f, layout, 1.25, None if w is None else w.astype(np.float64), eps)
            same(o, want, mag, dtype, f"{rows} rows")


@pytest.mark.parametrize("kw", [
    dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0, base=500000.0),
    dict(scaling="blend", factor=16.0, context=4096, low=1.0, high=32.0), dict(scaling="blend", factor=8.0, context=8192, low=1.0, high=4.0, base=500000.0)])
def test_scalings_at_far_positions(kw):
    from delta_prefetched_ffn_amd import Rope, rope_freqs
    f = R.freqs(128, **kw)
    np.testing.assert_allclose(rope_freqs(head_dim=128, **kw), f, rtol=1e-13)
    rng = np.random.default_rng(1)
    rope = Rope(head_dim=128, **kw)
    given = Rope(head_dim=128, freqs=f)
    pos = np.array([0, 1, 2, 4095, 4096, 131071, 1048575, 16777215, 16777217, -1, -77777], np.int32)
    q = rand(rng, (len(pos), 2, 128), "f32")
    dq, dp = q.cuda(), torch.from_numpy(pos).cuda()
    want, mag = R.turned(q.double().numpy(), pos, f)
    for r in (rope, given):
        out = torch.empty_like(dq)
        r.apply(len(pos), dq.data_ptr(), out.data_ptr(), 2, "f32", positions_ptr=dp.data_ptr(), stream=stream())
        # The frequency itself is a double: half a step of it, times the position.
        far = np.abs(pos)[:, None] * f * 2.0 ** -52
        same(out, want, mag * (1 + np.concatenate([far, far], 1)[:, None] * 2.0 ** 24), "f32")


def test_angles_of_the_largest_positions_are_exact():
    # Frequencies that are whole fractions of a turn: the angle is known exactly, whatever the position.
    from delta_prefetched_ffn_amd import Rope
    turn = np.array([1 / 8, 3 / 16, 1 / 1024, -1 / 4, 5 / 4, 0.0, 1 / 3, 1 / 2])
    rope = Rope(head_dim=16, freqs=2 * np.pi * turn)
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 0, 1, 12345679], np.int64)
    q = np.zeros((len(pos), 1, 16), np.float32)
    q[..., :8] = 1.0
    dq, out = torch.from_numpy(q).cuda(), torch.empty((len(pos), 1, 16), device="cuda")
    dp = torch.from_numpy(pos.astype(np.int32)).cuda()
    rope.apply(len(pos), dq.data_ptr(), out.data_ptr(), 1, "f32", positions_ptr=dp.data_ptr(), stream=stream())
    from fractions import Fraction
    got = out.double().cpu().numpy()[:, 0]
    for r, p in enumerate(pos):
        for i, t in enumerate([Fraction(1, 8), Fraction(3, 16), Fraction(1, 1024), Fraction(-1, 4), Fraction(5, 4), Fraction(0), Fraction(1, 3), Fraction(1, 2)]):
            a = float(Fraction(int(p)) * t % 1) * 2 * np.pi
            # 2 pi t as a double is off by 2^-53 of itself: at 2^31 positions 2^-22 of the angle's rate
            tol = 8 * 2.0 ** -24 + abs(int(p)) * abs(float(t)) * 2 * np.pi * 2.0 ** -52
            assert abs(got[r, i] - np.cos(a)) <= tol and abs(got[r, 8 + i] - np.sin(a)) <= tol, (p, t)


def test_first_position_in_place_strides_and_broadcast_rows():
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(2)
    rope = Rope(head_dim=80, rot_dim=64)
    f = R.freqs(64)
    # in place, inside a fused projection's output; what lies between stays
    both = rand(rng, (29, 12, 80), "bf16")
    dev = both.cuda()
    q, k = dev[:, :6], dev[:, 6:9]
    rope.apply(29, q.data_ptr(), q.data_ptr(), 6, "bf16", (960, 80, 960, 80, 960, 80, 960, 80), k_ptr=k.data_ptr(), k_out_ptr=k.data_ptr(), n_kv_heads=3,
               first=1000, stream=stream())
    want, mag = R.turned(both[:, :9].double().numpy(), 1000 + np.arange(29), f)
    same(dev[:, :9], want, mag, "bf16")
    assert torch.equal(dev[:, 9:].cpu(), both[:, 9:])
    # heads outermost in the result, one input row for all (stride 0), negative first positions
    one = rand(rng, (1, 4, 80), "f16")
    out = torch.full((4, 7, 88), 3.0, dtype=torch.float16, device="cuda")
    d = one.cuda()
    rope.apply(7, d.data_ptr(), out.data_ptr(), 4, "f16", (0, 80, 88, 7 * 88, 0, 0, 0, 0), first=-3, stream=stream())
    want, mag = R.turned(one.expand(7, 4, 80).double().numpy(), np.arange(-3, 4), f)
    same(out[:, :, :80].transpose(0, 1), want, mag, "f16")
    assert bool((out[:, :, 80:] == 3.0).all())
    rope.apply(0, d.data_ptr(), out.data_ptr(), 4, "f16", stream=stream())   # no rows
    rope.apply(3, d.data_ptr(), d.data_ptr(), 1, "f16", (80, 80, 80, 80, 0, 0, 0, 0), first=2 ** 31 - 3, stream=stream())


@pytest.mark.parametrize("layout,rot", [("half", 64), ("half", 20), ("interleaved", 64)])
def test_special_values_stay_in_their_head(layout, rot):
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(3)
    rope = Rope(head_dim=64, rot_dim=rot, layout=layout)
    q = rand(rng, (6, 3, 64), "f32")
    q[0, 1, 3], q[1, 2, 60], q[2, 0, 5], q[3, 1, 2] = float("nan"), float("nan"), float("inf"), -float("inf")
    q[4, 0] = 0.0
    q[5, 1] = 1e-30
    w = weights(rng, 64)
    dq, dw = q.cuda(), torch.from_numpy(w).cuda()
    for weight in (None, w):
        out = torch.empty_like(dq)
        rope.apply(6, dq.data_ptr(), out.data_ptr(), 3, "f32", first=5, q_weight_ptr=0 if weight is None else dw.data_ptr(), eps=1e-5, stream=stream())
        with np.errstate(invalid="ignore"):
            want, mag = R.turned(q.double().numpy(), 5 + np.arange(6), R.freqs(rot), layout, 1.0, weight, float(np.float32(1e-5)))
        same(out, want, mag, "f32")


def test_the_same_on_other_streams_and_in_graphs():
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(4)
    rope = Rope(head_dim=128)
    q = rand(rng, (64, 8, 128), "bf16").cuda()
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    want = torch.empty_like(q)
    rope.apply(64, q.data_ptr(), want.data_ptr(), 8, "bf16", positions_ptr=pos.data_ptr(), stream=stream())
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    rope.apply(64, q.data_ptr(), out.data_ptr(), 8, "bf16", positions_ptr=pos.data_ptr(), stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.apply(64, q.data_ptr(), out.data_ptr(), 8, "bf16", positions_ptr=pos.data_ptr(), stream=stream())
    for step in range(3):   # a replay takes the positions that are there
        pos += 100
        rope.apply(64, q.data_ptr(), want.data_ptr(), 8, "bf16", first=100 * (step + 1), stream=stream())
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    rope.close()


# ------------------------------------------------------------------------------------------------- into the cache

class Cache:
    def __init__(self, *, heads, kv, hd, page, pages=64, seqs=4, layers=1):
        from delta_prefetched_ffn_amd import KVCache, kv_bytes
        shape = dict(n_layers=layers, n_heads=heads, n_kv_heads=kv, head_dim=hd, page_tokens=page, n_pages=pages)
        nc, ne = kv_bytes(**shape)
        self.codes = torch.full((nc,), 0x7F, dtype=torch.uint8, device="cuda")
        self.exps = torch.full((ne,), 100, dtype=torch.int8, device="cuda")
        self.kv = KVCache(**shape, max_seqs=seqs, max_pages=pages, codes=self.codes.data_ptr(), exps=self.exps.data_ptr(), keepalive=(self.codes, self.exps))
        self.shape, self.pages_exps = shape, (layers, pages, kv, 2)

    def exp(self, page):
        return self.exps.view(self.pages_exps)[0, page].cpu().numpy()


def check_block(c, kv, seq, want, mag, before):
    """K of a sequence: each value within its rounding to the block's codes of what was appended last, the exponents as defined."""
    k, _ = kv.read_tokens(0, seq)
    pt, pages = kv.page_tokens, kv.pages(seq)
    new = want.shape[0]
    for p in range(before // pt, -(-(before + new) // pt)):
        lo, hi = max(before, p * pt), min(before + new, (p + 1) * pt)
        exps = c.exp(int(pages[p]))
        for h in range(kv.n_kv_heads):
            w, m = want[lo - before:hi - before, h], mag[lo - before:hi - before, h]
            slack = R.STEPS * 2.0 ** -24 * m * 1.01
            e = int(exps[h, 0])
            if lo == p * pt:
                assert e in {KR.exponent_for((np.abs(w) + s).max()) for s in (slack, -slack)}, (p, h)
            step = np.maximum(np.abs(w) * 2.0 ** -4, 2.0 ** (e - 10)) * (1 + 2.0 ** -18)
            assert (np.abs(k[lo:hi, h] - w) <= step + slack).all(), (p, h)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kv,hd,page,rot,layout,norm", [
    (4, 4, 64, 16, 64, "half", True), (8, 2, 128, 64, 128, "half", False), (6, 3, 128, 32, 64, "interleaved", True), (7, 1, 80, 32, 80, "half", True),
    (3, 1, 40, 128, 20, "half", True), (2, 2, 256, 128, 256, "half", True), (2, 1, 8, 16, 8, "interleaved", False), (2, 1, 200, 64, 198, "half", True)])
def test_append_is_rope_then_append(dtype, heads, kv, hd, page, rot, layout, norm):
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(hd + page + rot)
    rope = Rope(head_dim=hd, rot_dim=rot, layout=layout)
    c, plain = Cache(heads=heads, kv=kv, hd=hd, page=page), Cache(heads=heads, kv=kv, hd=hd, page=page)
    wq, wk = weights(rng, hd), weights(rng, hd)
    dwq, dwk = torch.from_numpy(wq).cuda(), torch.from_numpy(wk).cuda()
    f = R.freqs(rot)
    for seqs, new in (([0], [1]), ([0, 1], [2, 5]), ([2, 0, 1], [3 * page + 1, 0, page - 5]), ([1, 0, 2], [1, 1, 1])):
        before = [c.kv.tokens(s) for s in seqs]
        rows = sum(new)
        both = rand(rng, (rows, heads + 2 * kv, hd), dtype)
        dev = both.cuda()
        q, k, v = dev[:, :heads], dev[:, heads:heads + kv], dev[:, heads + kv:]
        out = torch.full((rows, heads, hd), 7.0, dtype=q.dtype, device="cuda")
        w = both.shape[1] * hd
        for x in (c, plain):
            x.kv.extend(seqs, new, stream())
        for _ in range(2):   # a second call stores the same
            rope.append(c.kv, 0, q.data_ptr(), out.data_ptr(), k.data_ptr(), v.data_ptr(), dtype, (w, hd, heads * hd, hd, w, hd, w, hd),
                        q_weight_ptr=dwq.data_ptr() if norm else 0, k_weight_ptr=dwk.data_ptr() if norm else 0, eps=1e-5, stream=stream())
        plain.kv.append(0, k.data_ptr(), v.data_ptr(), dtype, (w, hd, w, hd), stream())
        pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, new)])
        eps = float(np.float32(1e-5))
        x64 = both.double().numpy()
        want, mag = R.turned(x64[:, :heads], pos, f, layout, 1.0, wq.astype(np.float64) if norm else None, eps)
        same(out, want, mag, dtype, "q")
        want, mag = R.turned(x64[:, heads:heads + kv], pos, f, layout, 1.0, wk.astype(np.float64) if norm else None, eps)
        row = 0
        for s, n, b in zip(seqs, new, before):
            if n:
                check_block(c, c.kv, s, want[row:row + n], mag[row:row + n], b)
            row += n
            np.testing.assert_array_equal(c.kv.read_tokens(0, s)[1], plain.kv.read_tokens(0, s)[1], err_msg="V")


@pytest.mark.parametrize("kv,hd,page,rot,layout,dtype", [
    (17, 64, 128, 64, "half", "bf16"), (17, 40, 64, 40, "interleaved", "f16"), (17, 24, 32, 20, "half", "f32"), (17, 64, 16, 0, "half", "f32"), (5, 256, 128, 128, "half", "f16")])
def test_long_prompts_take_several_heads_at_once(kv, hd, page, rot, layout, dtype):
    # Two prompts that go on where small tokens lie in their pages already; infinities and NaN (rot 0) stay in their own block.
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(kv + hd + page)
    rope = Rope(head_dim=hd, rot_dim=rot, layout=layout)
    new = [50000 // kv, 7]
    pages = 2 * (new[0] // page + 4)
    c, plain = (Cache(heads=kv, kv=kv, hd=hd, page=page, pages=pages) for _ in range(2))
    w = weights(rng, hd) if rot else np.ones(hd, np.float32)
    dw = torch.from_numpy(w).cuda()
    for seqs, n, scale in (([1, 0], [9, page - 3], 1e-3), ([1, 0], new, 1.0)):
        before = [c.kv.tokens(s) for s in seqs]
        k, v = rand(rng, (sum(n), kv, hd), dtype, scale), rand(rng, (sum(n), kv, hd), dtype)
        if not rot:
            k[3, 1, 5], k[4, 2, 6], k[sum(n) - 1, 0, 7] = float("inf"), float("nan"), -float("inf")
        dk, dv, out = k.cuda(), v.cuda(), torch.empty_like(k, device="cuda")
        for x in (c, plain):
            x.kv.extend(seqs, n, stream())
        rope.append(c.kv, 0, dk.data_ptr(), out.data_ptr(), dk.data_ptr(), dv.data_ptr(), dtype, k_weight_ptr=dw.data_ptr() if rot else 0, eps=1e-5, stream=stream())
        plain.kv.append(0, dk.data_ptr(), dv.data_ptr(), dtype, stream=stream())
        torch.cuda.synchronize()
        if rot == 0:
            assert torch.equal(c.codes, plain.codes) and torch.equal(c.exps, plain.exps)
            continue
        pos = np.concatenate([np.arange(b, b + m) for b, m in zip(before, n)])
        want, mag = R.turned(k.double().numpy(), pos, R.freqs(rot), layout, 1.0, w.astype(np.float64), float(np.float32(1e-5)))
        row = 0
        for s, m, b in zip(seqs, n, before):
            if scale == 1.0 or b == 0:
                check_block(c, c.kv, s, want[row:row + m], mag[row:row + m], b)
            row += m
            np.testing.assert_array_equal(c.kv.read_tokens(0, s)[1], plain.kv.read_tokens(0, s)[1], err_msg="V")


def test_append_special_values_and_other_layers():
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(9)
    rope = Rope(head_dim=64, rot_dim=0)     # no turn: K goes in as it is, as np_kv_append's
    c, plain = Cache(heads=2, kv=2, hd=64, page=16, layers=2), Cache(heads=2, kv=2, hd=64, page=16, layers=2)
    k, v = rand(rng, (21, 2, 64), "f32"), rand(rng, (21, 2, 64), "f32", 1e20)
    k[3, 0, 5], k[4, 1, 6], k[5, 0, 7], v[9, 1, 1], v[2, 0, 3] = float("inf"), float("nan"), -float("inf"), float("nan"), -float("inf")
    k[16:, 1] = 0.0
    dk, dv = k.cuda(), v.cuda()
    out = torch.empty_like(dk)
    for x in (c, plain):
        x.kv.extend([0], [21], stream())
        x.codes.fill_(0x7F)
    rope.append(c.kv, 1, dk.data_ptr(), out.data_ptr(), dk.data_ptr(), dv.data_ptr(), "f32", stream=stream())
    plain.kv.append(1, dk.data_ptr(), dv.data_ptr(), "f32", stream=stream())
    torch.cuda.synchronize()
    assert torch.equal(c.codes, plain.codes) and torch.equal(c.exps, plain.exps)
    assert torch.equal(out.nan_to_num(5.0), dk.nan_to_num(5.0))


def test_append_in_graphs_and_with_attention():
    # A step of a decode loop, captured: rope.append and attend; replays are checked against eager calls on another cache.
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(5)
    rope = Rope(head_dim=128, scaling="ntk", factor=2.0)
    a, b = Cache(heads=8, kv=2, hd=128, page=32), Cache(heads=8, kv=2, hd=128, page=32)
    first = rand(rng, (70, 12, 128), "bf16").cuda()
    token = torch.empty((2, 12, 128), dtype=torch.bfloat16, device="cuda")
    out = [torch.zeros((70, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step(c, x, y):
        q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
        rope.append(c.kv, 0, q.data_ptr(), y.data_ptr(), k.data_ptr(), v.data_ptr(), "bf16", (1536, 128, 1024, 128, 1536, 128, 1536, 128), stream=stream())
        z = torch.empty_like(y)
        c.kv.attend(0, y.data_ptr(), z.data_ptr(), "bf16", scale=0.1, stream=stream())
        return z

    for c, y in ((a, out[0]), (b, out[1])):
        c.kv.extend([0, 1], [40, 30], stream())
        step(c, first, y)
        c.kv.extend([0, 1], [1, 1], stream())
    g = torch.cuda.CUDAGraph()
    token.copy_(rand(rng, (2, 12, 128), "bf16"))
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = step(a, token, out[0])
    for _ in range(3):
        token.copy_(rand(rng, (2, 12, 128), "bf16"))
        g.replay()
        want = step(b, token, out[1])
        torch.cuda.synchronize()
        assert torch.equal(got[:2], want[:2]) and torch.equal(a.codes, b.codes) and torch.equal(a.exps, b.exps)


def test_refusals():
    from delta_prefetched_ffn_amd import NPError, Rope
    from delta_prefetched_ffn_amd import binding as B
    x = torch.zeros((4, 2, 64), device="cuda")
    rope = Rope(head_dim=64)

    def refused(status, f, *a, **kw):
        with pytest.raises(NPError) as e:
            f(*a, **kw)
        assert e.value.status == status, str(e.value)

    p = x.data_ptr()
    host = torch.zeros((4, 2, 64))
    for a, kw in [((4, p + 4, p, 2, "f32"), {}), ((4, p, p + 8, 2, "f32"), {}), ((-1, p, p, 2, "f32"), {}), ((4, p, p, 0, "f32"), {}), ((4, 0, p, 2, "f32"), {}),
                  ((4, p, p, 2, "f32", (128, 64, 128, 32, 0, 0, 0, 0)), {}), ((4, p, p, 2, "f32", (128, 64, 2, 64, 0, 0, 0, 0)), {}),
                  ((4, p, p, 2, "f32", (128, 64, 64, 64, 0, 0, 0, 0)), {}), ((4, p, p, 2, "f32", (256, 64, 128, 64, 0, 0, 0, 0)), {}),
                  ((4, p, p, 2, "f32"), dict(k_ptr=p)), ((4, p, p, 2, "f32"), dict(eps=-1.0)), ((4, p, p, 2, "f32"), dict(eps=float("nan"))),
                  ((4, p, p, 2, "f32"), dict(first=2 ** 31 - 3)), ((4, p, p, 2, "f32"), dict(positions_ptr=p + 2)), ((4, p, p, 2, "f32"), dict(q_weight_ptr=p + 4)),
                  ((4, host.data_ptr() // 16 * 16, p, 2, "f32"), {}), ((4, p, p, 2, "f32"), dict(positions_ptr=host.data_ptr() // 16 * 16))]:
        refused(B.NP_EINVAL, rope.apply, *a, **kw)
    with pytest.raises(ValueError):
        rope.apply(4, p, p, 2, "f32", (1, 2, 3, 4))
    with pytest.raises(OverflowError):
        rope.apply(4, p, p, 2, "f32", first=2 ** 31)
    c = Cache(heads=2, kv=2, hd=64, page=16)
    refused(B.NP_ESTATE, rope.append, c.kv, 0, p, p, p, p, "f32")
    c.kv.extend([0], [4], stream())
    refused(B.NP_EINVAL, rope.append, c.kv, 1, p, p, p, p, "f32")
    refused(B.NP_EINVAL, Rope(head_dim=128).append, c.kv, 0, p, p, p, p, "f32")
    refused(B.NP_EINVAL, rope.append, c.kv, 0, p, p, p + 4, p, "f32")
    refused(B.NP_EINVAL, rope.append, c.kv, 0, p, p, p, p, "f32", k_weight_ptr=p + 4)
    torch.cuda.synchronize()
    assert bool((x == 0).all())
