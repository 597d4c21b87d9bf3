"""np_rope_append on pages that hold tokens already: the block's exponent never goes down and grows only as far as the new tokens ask,
the tokens before keep their values, rounded once more where it grew."""
import numpy as np
import pytest

from tests import kv_reference as KR
from tests import rope_reference as R
from tests import test_gpu_rope as T
from tests.harness import torch_mod

pytestmark = pytest.mark.gpu

torch = None


@pytest.fixture(autouse=True, scope="module")
def _torch():
    global torch
    torch = T.torch = torch_mod()
    assert torch.cuda.is_available()


def exponents(c, seq):
    """[pages][kv heads]: K's."""
    return np.array([c.exp(int(p))[:, 0] for p in c.kv.pages(seq)], np.int64).reshape(-1, c.kv.n_kv_heads)


def check_continued(c, seq, want, mag, before, k0, e0):
    """K of a sequence after its tokens from `before` on were taken up (values want, off by mag * 2^-24 * STEPS at most), which had
    values k0 [before, heads, hd] and exponents e0 [pages, heads]; how many blocks grew."""
    kv, pt, n = c.kv, c.kv.page_tokens, want.shape[0]
    k, _ = kv.read_tokens(0, seq)
    e1, grown = exponents(c, seq), 0
    slack = R.STEPS * 2.0 ** -24 * mag * 1.01
    for p in range(before // pt, -(-(before + n) // pt)):
        lo, hi = max(before, p * pt), min(before + n, (p + 1) * pt)
        for h in range(kv.n_kv_heads):
            w, s, e = want[lo - before:hi - before, h], slack[lo - before:hi - before, h], int(e1[p, h])
            asked = {KR.exponent_for(max(0.0, (np.abs(w) + sign * s).max())) for sign in (1, -1)}
            if lo > p * pt:
                asked = {max(int(e0[p, h]), x) for x in asked}
                old = k0[p * pt:lo, h].astype(np.float64)
                grown += e > int(e0[p, h])
                np.testing.assert_array_equal(k[p * pt:lo, h], KR.round_e4m3(old * 2.0 ** -e) * 2.0 ** e, err_msg=f"page {p}, head {h}: the tokens before")
            assert e in asked, (p, h, e, asked)
            # half a step: 2^-4 of the value, or of the smallest numbers' 2^-9
            step = np.maximum(np.abs(w) * 2.0 ** -4, 2.0 ** (e - 10)) * (1 + 2.0 ** -18)
            assert (np.abs(k[lo:hi, h] - w) <= step + s).all(), (p, h)
    if before % pt == 0:
        np.testing.assert_array_equal(k[:before], k0)
    else:
        np.testing.assert_array_equal(k[:before // pt * pt], k0[:before // pt * pt])
    return grown


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kv,hd,page,rot,layout", [
    (4, 4, 64, 16, 64, "half"), (8, 2, 128, 64, 128, "half"), (4, 4, 128, 128, 64, "interleaved"), (6, 3, 80, 32, 20, "half"), (3, 3, 200, 64, 198, "half"),
    (2, 2, 200, 128, 200, "interleaved"), (4, 2, 256, 64, 256, "half"), (2, 2, 256, 128, 256, "half"), (2, 2, 8, 128, 8, "half"), (5, 5, 40, 64, 40, "half"), (3, 3, 192, 32, 192, "half")])
def test_exponents_and_tokens_of_continued_pages(dtype, heads, kv, hd, page, rot, layout):
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(hd + page + rot)
    rope = Rope(head_dim=hd, rot_dim=rot, layout=layout)
    c = T.Cache(heads=heads, kv=kv, hd=hd, page=page)
    w = T.weights(rng, hd)
    dw = torch.from_numpy(w).cuda()
    f, eps, grown, kept = R.freqs(rot), float(np.float32(1e-5)), 0, 0
    state = {s: (np.zeros((0, kv, hd), np.float32), np.zeros((0, kv), np.int64)) for s in range(3)}
    #            tokens of each, and how large each head's values are (a power of two; without the norm, which would undo it)
    steps = [([0, 1, 2], [1, page - 2, page + 3]), ([0, 1, 2], [1, 1, 2]), ([2, 0], [1, 3]), ([1, 0, 2], [page + 2, 1, page - 1]), ([0, 1, 2], [2 * page, 1, 1]), ([0, 1, 2], [1, 1, 1])]
    for turn, (seqs, new) in enumerate(steps):
        norm, rows = turn == 4, sum(new)
        size = np.exp2(rng.integers(-9, 4, kv)).astype(np.float32)[:, None]
        size[turn % kv] = 2.0 ** (turn - 3)   # one head that grows with each step
        k = (torch.from_numpy(rng.standard_normal((rows, kv, hd)).astype(np.float32) * size)).to(T.tdt(dtype))
        q, v = T.rand(rng, (rows, heads, hd), dtype), T.rand(rng, (rows, kv, hd), dtype)
        dq, dk, dv, out = q.cuda(), k.cuda(), v.cuda(), torch.empty((rows, heads, hd), dtype=T.tdt(dtype), device="cuda")
        before = [c.kv.tokens(s) for s in seqs]
        c.kv.extend(seqs, new, T.stream())
        rope.append(c.kv, 0, dq.data_ptr(), out.data_ptr(), dk.data_ptr(), dv.data_ptr(), dtype, k_weight_ptr=dw.data_ptr() if norm else 0, eps=1e-5, stream=T.stream())
        torch.cuda.synchronize()
        pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, new)])
        want, mag = R.turned(k.double().numpy(), pos, f, layout, 1.0, w.astype(np.float64) if norm else None, eps)
        row = 0
        for s, n, b in zip(seqs, new, before):
            k0, e0 = state[s]
            g = check_continued(c, s, want[row:row + n], mag[row:row + n], b, k0, e0)
            grown, kept = grown + g, kept + (kv - g if b % page else 0)
            row += n
        for s in range(3):
            state[s] = c.kv.read_tokens(0, s)[0], exponents(c, s)
    assert grown >= 2 and kept >= 2


@pytest.mark.parametrize("kv,hd,page,dtype,new", [
    (3, 128, 64, "bf16", 5), (3, 128, 128, "f16", 70), (2, 200, 64, "f32", 3), (2, 200, 128, "bf16", 200), (2, 256, 64, "f16", 40), (2, 256, 128, "f32", 130), (3, 136, 128, "bf16", 9),
    (17, 128, 128, "bf16", 3000), (5, 200, 64, "f16", 10000), (17, 256, 128, "bf16", 2500), (9, 80, 128, "f32", 5000)])
def test_without_a_turn_the_bytes_are_appends_also_where_blocks_grow(kv, hd, page, dtype, new):
    from delta_prefetched_ffn_amd import Rope
    rng = np.random.default_rng(kv + hd + page)
    rope = Rope(head_dim=hd, rot_dim=0)
    pages = 2 * (new // page + 4)
    c, plain = (T.Cache(heads=kv, kv=kv, hd=hd, page=page, pages=pages, seqs=2) for _ in range(2))
    grown = 0
    for turn, n in enumerate(([page - 3, 6], [1, 1], [1, new], [new, page - 1], [2, 3])):
        before = [exponents(c, s) for s in (0, 1)]
        size = np.exp2(rng.integers(-6, 2, kv) + 2 * turn).astype(np.float32)[:, None]
        k, v = (torch.from_numpy(rng.standard_normal((sum(n), kv, hd)).astype(np.float32) * size).to(T.tdt(dtype)) for _ in range(2))
        dk, dv, out = k.cuda(), v.cuda(), torch.empty_like(k, device="cuda")
        for x in (c, plain):
            x.kv.extend([0, 1], n, T.stream())
        rope.append(c.kv, 0, dk.data_ptr(), out.data_ptr(), dk.data_ptr(), dv.data_ptr(), dtype, stream=T.stream())
        plain.kv.append(0, dk.data_ptr(), dv.data_ptr(), dtype, stream=T.stream())
        torch.cuda.synchronize()
        assert torch.equal(c.codes, plain.codes) and torch.equal(c.exps, plain.exps), turn
        grown += sum(int((exponents(c, s)[:len(b)] > b).sum()) for s, b in enumerate(before))
    assert grown >= 3
