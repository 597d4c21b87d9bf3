"""np_attend_shared on the GPU: sequences that share first pages, against the fp64 definition in tests/kv_reference.py (which
knows nothing of sharing)."""
import numpy as np
import pytest

from tests import kv_reference as R
from tests import test_gpu_kv as K
from tests.harness import torch_mod

pytestmark = pytest.mark.gpu

torch = None


@pytest.fixture(autouse=True, scope="module")
def _torch():
    global torch
    torch = K.torch = torch_mod()
    assert torch.cuda.is_available()


def attention(q, k, v, before, scale, window=0, sinks=0, held=None):
    """kv_reference.attention, a kv head's rows at a time (the same numbers, long sequences in less time)."""
    n, H, hd = q.shape
    Hk = k.shape[1]
    G = H // Hk
    out, terms, lse, mag = np.zeros((n, H, hd)), np.zeros((n, H, hd)), np.full((n, H), -np.inf), np.zeros((n, H))
    for i in range(n):
        pos = before + i
        j = np.arange(pos + 1)
        ok = np.ones(pos + 1, bool) if held is None else held[:pos + 1].copy()
        if window:
            ok &= (pos - j < window) | (j < sinks)
        j = j[ok]
        if not j.size:
            continue
        j = slice(None, pos + 1) if j.size == pos + 1 else j
        for h in range(Hk):
            kk, vv, g = k[j, h], v[j, h], slice(h * G, (h + 1) * G)
            with np.errstate(all="ignore"):
                s = q[i, g] @ kk.T * scale
                top = s.max(-1, keepdims=True)
                p = np.exp(s - top)
                l = p.sum(-1, keepdims=True)
                out[i, g], terms[i, g] = p @ vv / l, p @ np.abs(vv) / l
                lse[i, g] = np.log(l[:, 0]) + top[:, 0]
                mag[i, g] = (np.abs(q[i, g]) @ np.abs(kk).T).max(-1) * scale
    return out, lse, terms, mag


class Env(K.Env):
    """test_gpu_kv's, with attend() as attend_shared and forks that the reference follows."""

    def __init__(self, **kw):
        super().__init__(**kw)
        self.plain, self.kv.attend = self.kv.attend, self.kv.attend_shared

    def attend(self, *a, **kw):
        whole, R.attention = R.attention, attention
        try:
            return super().attend(*a, **kw)
        finally:
            R.attention = whole

    def fork(self, src, dst, n, mode="share"):
        self.kv.fork(src, dst, n, mode, self.stream())
        for layer in range(self.layers):
            r = R.RefSeq(self.nkv, self.hd, self.page)
            r.codes, r.exps = self.ref[layer][src].codes[:n].copy(), self.ref[layer][src].exps[:-(-n // self.page)].copy()
            self.ref[layer][dst] = r

    def shared(self, dtype, **kw):
        """Whether a call with these arguments takes the shared kernels."""
        rows = sum(n for _, n in self.current)
        q = torch.zeros((rows, self.heads, self.hd), dtype=K.tdt(dtype), device="cuda")
        names = K.kernels_of(lambda s: self.kv.attend_shared(0, q.data_ptr(), q.data_ptr(), dtype, scale=1.0, stream=s, **kw))
        kinds = {"k_prefix" in n for n in names}
        assert len(kinds) == 1
        return kinds.pop()


def batch(heads, kv, hd, page, prefix, tails, dtype="bf16", seed=0, new=None, pages=None):
    """Sequence 0 holds a prompt; 1, 2, ... go on from it by tails[i] tokens, then by new[i]."""
    n = len(tails)
    new = new or [1] * n
    pages = pages or -(-prefix // page) + sum(-(-(t + m) // page) + 2 for t, m in zip(tails, new)) + 2
    e = Env(heads=heads, kv=kv, hd=hd, page=page, pages=pages, seqs=n + 1, seed=seed)
    e.step([0], [prefix], dtype)
    for i in range(n):
        e.fork(0, i + 1, prefix)
    e.step(list(range(1, n + 1)), tails, dtype)
    e.step(list(range(1, n + 1)), new, dtype)
    return e


# Sharing takes calls of some 200 MB of keys and values in all (it pays from there on): 24 or 40 sequences, prompts of that length.

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kv,hd,page,prompt,n", [
    (16, 16, 64, 16, 4003, 24), (32, 8, 128, 64, 4003, 24), (28, 4, 80, 32, 5003, 40), (12, 12, 40, 128, 5401, 24), (16, 16, 256, 16, 1003, 24), (24, 12, 192, 64, 1903, 24), (40, 4, 128, 32, 4003, 40)])
def test_continuations_of_a_prompt(dtype, heads, kv, hd, page, prompt, n):
    rng = np.random.default_rng(heads + hd)
    tails = [0, 1, page, 2 * page - 1] + [int(x) for x in rng.integers(0, 150, n - 4)]
    e = batch(heads, kv, hd, page, prompt, tails, dtype)
    assert e.shared(dtype)
    e.attend(dtype)
    e.attend(dtype, layout="fused", q_scale=4.0)
    e.attend(dtype, layout="heads", lse=False)


def test_the_reference_of_long_sequences_is_the_reference():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 6, 8)), rng.standard_normal((40, 3, 8)), rng.standard_normal((40, 3, 8))
    v[5, 1, 2] = np.nan
    held = np.arange(40) != 7
    for kw in (dict(), dict(window=9, sinks=2), dict(held=held)):
        for a, b in zip(attention(q, k, v, 37, 0.3, **kw), R.attention(q, k, v, 37, 0.3, **kw)):
            np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,hd,prompt", [(24, 24, 64, 2500), (32, 4, 128, 4000), (24, 8, 256, 2500)])
def test_drafts_of_different_lengths(dtype, heads, kv, hd, prompt):
    new = [1, 5, 9, 2, 0, 3, 7, 1, 1, 12, 4, 6, 0, 2, 8, 3, 11, 10, 1, 1, 1, 14, 13, 2]
    tails = [0, 40, 3, 70, 20, 16, 1, 0, 33, 90, 5, 64, 2, 8, 31, 17, 11, 12, 13, 14, 15, 16, 17, 18]
    e = batch(heads, kv, hd, 16, prompt, tails, dtype, new=new, pages=-(-prompt // 16) + 24 * 10)
    assert e.shared(dtype)
    e.attend(dtype)
    # the same number for all
    e.step([3, 1, 2, 9, 14, 6, 7, 8, 4, 5, 10, 11, 20, 21, 22, 23, 24, 12], [4] * 18, dtype)
    assert e.shared(dtype)
    e.attend(dtype, q_scale=3.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_branches_families_and_strangers(dtype):
    # Two prompts; conversations forked from conversations; sequences of their own in between; all in mixed order.
    e = Env(heads=16, kv=16, hd=64, page=32, pages=600, seqs=60)
    e.step([0, 1, 2], [2900, 1700, 333], dtype)
    leaves, at = [2], 3
    for root, n in ((0, 2900), (1, 1700)):
        for b in range(4):
            e.fork(root, at, n - 37 * b)
            branch = at
            at += 1
            e.step([branch], [100 + 60 * b], dtype)
            for k in range(5):
                e.fork(branch, at, e.kv.tokens(branch) - 20 * k)
                leaves.append(at)
                at += 1
            leaves.append(branch)
    e.step([55, 56], [1, 40], dtype)
    leaves += [55, 56, 0]
    e.rng.shuffle(leaves)
    leaves = [int(x) for x in leaves]
    e.step(leaves, [int(x) for x in e.rng.integers(0, 40, len(leaves))], dtype)
    e.step(leaves, [1] * len(leaves), dtype)
    assert e.shared(dtype)
    e.attend(dtype)
    e.step(leaves, [int(x) for x in e.rng.integers(0, 4, len(leaves))], dtype)
    assert e.shared(dtype)
    e.attend(dtype)
    e.kv.compact(e.stream())   # the step goes on with other page numbers
    e.attend(dtype)


def test_more_runs_than_a_call_takes():
    # 40 families of three that share some 3,000 tokens each: the longest runs are shared, the others read by each.
    e = Env(heads=4, kv=4, hd=64, page=64, pages=2400, seqs=121, seed=5)
    e.step(list(range(40)), [3000 + 19 * i for i in range(40)], "bf16")
    for i in range(40):
        e.fork(i, 40 + i, 3000 + 19 * i - i % 5)
        e.fork(i, 80 + i, 3000 + 19 * i - i % 7)
    e.step(list(range(120)), [1] * 120, "bf16")
    assert e.shared("bf16")
    e.attend("bf16")
    # one chain: each continues the one before
    e = Env(heads=16, kv=16, hd=64, page=16, pages=900, seqs=41, seed=6)
    e.step([0], [2000], "bf16")
    for i in range(40):
        e.fork(i, i + 1, e.kv.tokens(i) // 16 * 16)
        e.step([i + 1], [80], "bf16")
    e.step(list(range(41)), [1] * 41, "bf16")
    assert e.shared("bf16")
    e.attend("bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (200, 0), (200, 70), (1700, 4), (2050, 40), (5000, 0), (300, 2000), (1600, 45)])
def test_windows_and_first_tokens(dtype, window, sinks):
    e = batch(32, 32, 64, 32, 2000, [0, 60, 3, 90, 20, 16, 1, 0, 33, 190, 5, 64, 2, 8, 31, 17, 40, 41, 42, 43, 1, 2, 3, 4], dtype, seed=window)
    e.attend(dtype, window=window, sinks=sinks)
    if window >= 1600 or sinks > 1600:
        assert e.shared(dtype, window=window, sinks=sinks)


def test_dropped_pages():
    # A window moved on: the shared first pages are gone but for the first tokens', those behind are still shared.
    e = batch(32, 32, 64, 16, 2600, [20 + 3 * i for i in range(24)], "bf16", seed=3)
    held = {}
    for s in range(1, 25):
        n = e.kv.tokens(s)
        gone = e.kv.evict(s, 2000, 5)
        assert gone > 0
        held[s] = np.ones(n + 10, bool)
        held[s][16:16 + 16 * gone] = False
    e.step(list(range(1, 25)), [1] * 24, "bf16")
    assert e.shared("bf16", window=2000, sinks=5) and e.shared("bf16")
    e.attend("bf16", window=2000, sinks=5, held=held)
    e.attend("bf16", held=held)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_nan_infinity_and_far_scales_in_the_shared_pages(dtype):
    e = Env(heads=32, kv=32, hd=64, page=16, pages=600, seqs=25, seed=11)
    rows = 2000
    e.extend([0], [rows])
    k, v = (e.rng.standard_normal((rows, 32, 64)).astype(np.float32) for _ in range(2))
    v *= np.repeat(2.0 ** e.rng.integers(-30, 8, (-(-rows // 16), 32)), 16, 0)[:rows, :, None].astype(np.float32)   # blocks of different magnitude
    v[20, 0, 5], v[300, 1, 7], v[640, 2, 0], k[400, 3, 3], k[401, 4, 4] = np.nan, np.inf, -np.inf, np.nan, np.inf
    kt, vt = torch.from_numpy(k), torch.from_numpy(v)
    e.append((kt, kt.double().numpy()), (vt, vt.double().numpy()), "f32")
    for i in range(1, 25):
        e.fork(0, i, rows - i % 3)
    e.step(list(range(1, 25)), [1 + 5 * i for i in range(24)], "f32")
    e.step(list(range(1, 25)), [1] * 24, "f32")
    assert e.shared(dtype)
    e.attend(dtype)
    assert e.shared(dtype, window=1700, sinks=30)
    e.attend(dtype, window=1700, sinks=30)
    q = e.rand(24, 32, dtype)
    q[0][3, 1, 0], q[0][9, 5, 3] = float("nan"), float("nan")   # rows of their own, the others untouched
    e.attend(dtype, q=(q[0], q[0].double().numpy()))


def test_the_same_from_run_to_run_on_streams_and_in_graphs():
    e = batch(32, 8, 128, 32, 6000, [50 + 7 * i for i in range(20)], "bf16", seed=2)
    assert e.shared("bf16") and e.shared("bf16", window=5500)
    q = e.rand(20, 32, "bf16")
    runs = [e.attend("bf16", q=q).clone() for _ in range(4)]
    assert all(torch.equal(r, runs[0]) for r in runs)
    qd, out = q[0].cuda(), torch.zeros((20, 32, 128), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = lambda s: e.kv.attend_shared(0, qd.data_ptr(), out.data_ptr(), "bf16", scale=1 / np.sqrt(128), stream=s)  # noqa: E731
    call(side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, runs[0])
    graphs = []
    for window in (0, 5500):   # two graphs that share the cache's workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            e.kv.attend_shared(0, qd.data_ptr(), out.data_ptr(), "bf16", scale=0.1, window=window, stream=torch.cuda.current_stream().cuda_stream)
        graphs.append(g)
    for turn in range(3):
        qd.copy_(e.rand(20, 32, "bf16")[0])
        for g, window in zip(graphs, (0, 5500)):
            out.zero_()
            g.replay()
            got = out.clone()
            e.kv.attend_shared(0, qd.data_ptr(), out.data_ptr(), "bf16", scale=0.1, window=window, stream=e.stream())
            torch.cuda.synchronize()
            assert torch.equal(got, out), (turn, window)


def test_what_does_not_share_or_pay_is_attend():
    e = batch(8, 8, 64, 16, 900, [200] + [3 * i for i in range(18)], "bf16", new=[150] + [1] * 18)   # a prompt among the tokens
    assert not e.shared("bf16")
    e.attend("bf16")
    e = Env(heads=8, kv=4, hd=64, page=16, pages=300, seqs=8)
    e.step([0, 1, 2, 3], [900, 800, 10, 40], "bf16")
    e.fork(0, 4, 40)          # too little
    e.fork(0, 5, 900, "copy")  # pages of its own
    e.step([0, 1, 2, 3, 4, 5], [1, 1, 1, 0, 1, 1], "bf16")
    assert not e.shared("bf16")
    e.attend("bf16")
    q = torch.zeros((5, 8, 64), device="cuda")
    K.torch = torch
    from delta_prefetched_ffn_amd import NPError
    from delta_prefetched_ffn_amd import binding as B
    p = q.data_ptr()
    for status, a, kw in ((B.NP_EINVAL, (0, p + 4, p, "f32"), dict(scale=1.0)), (B.NP_EINVAL, (1, p, p, "f32"), dict(scale=1.0)), (B.NP_EINVAL, (0, p, p, "f32"), dict(scale=0.0)),
                          (B.NP_EINVAL, (0, p, p, "f32"), dict(scale=1.0, window=-1)), (B.NP_EINVAL, (0, p, p, "f32", (512, 64, 512, 32)), dict(scale=1.0)),
                          (B.NP_EINVAL, (0, p, p, "f32"), dict(scale=1.0, lse_ptr=p + 2))):
        with pytest.raises(NPError) as err:
            e.kv.attend_shared(*a, **kw)
        assert err.value.status == status
    e.kv.reset()
    with pytest.raises(NPError) as err:
        e.kv.attend_shared(0, p, p, "f32", scale=1.0)
    assert err.value.status == B.NP_ESTATE


def test_offsets_past_4_gib():
    # The prompt's pages lie past 4 GiB of the pool.
    e = Env(heads=32, kv=32, hd=128, page=128, pages=4400, seqs=26, max_pages=4300, seed=4)
    e.kv.extend([25], [4200 * 128], e.stream())
    e.step([0], [1000], "bf16")
    assert int(min(e.kv.pages(0))) * 32 * 2 * 128 * 128 > 1 << 32
    for i in range(1, 25):
        e.fork(0, i, 1000)
    e.step(list(range(1, 25)), [1] * 24, "bf16")
    assert e.shared("bf16")
    e.attend("bf16")
