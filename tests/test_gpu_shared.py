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


class Env(K.Env):
    """test_gpu_kv's, with attend() as attend_shared and forks that the reference follows."""

    def __init__(self, **kw):
        super().__init__(**kw)
        self.plain, self.kv.attend = self.kv.attend, self.kv.attend_shared

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


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,kv,hd,page", [(8, 8, 64, 16), (32, 8, 128, 64), (28, 4, 80, 32), (6, 6, 40, 128), (8, 8, 256, 16), (12, 6, 192, 64), (64, 2, 128, 32), (4, 4, 128, 16)])
def test_continuations_of_a_prompt(dtype, heads, kv, hd, page):
    rng = np.random.default_rng(heads + hd)
    tails = [0, 1, page, 2 * page - 1] + [int(x) for x in rng.integers(0, 150, 20)]
    e = batch(heads, kv, hd, page, 1003, tails, dtype)
    assert e.shared(dtype)
    e.attend(dtype)
    e.attend(dtype, layout="fused", q_scale=4.0)
    e.attend(dtype, layout="heads", lse=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,hd", [(8, 8, 64), (32, 4, 128), (12, 4, 256)])
def test_drafts_of_different_lengths(dtype, heads, kv, hd):
    new = [1, 5, 9, 2, 0, 3, 7, 1, 1, 12, 4, 6, 0, 2, 8, 3]
    e = batch(heads, kv, hd, 16, 1100, [0, 40, 3, 70, 20, 16, 1, 0, 33, 90, 5, 64, 2, 8, 31, 17], dtype, new=new)
    assert e.shared(dtype)
    e.attend(dtype)
    # the same number for all
    e.step([3, 1, 2, 9, 14, 6, 7, 8, 4, 5, 10, 11], [4] * 12, dtype)
    e.attend(dtype, q_scale=3.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_branches_families_and_strangers(dtype):
    # Two prompts; conversations forked from conversations; sequences of their own in between; all in mixed order.
    e = Env(heads=8, kv=4, hd=64, page=32, pages=400, seqs=60)
    e.step([0, 1, 2], [900, 700, 333], dtype)
    leaves, at = [2], 3
    for root, n in ((0, 900), (1, 700)):
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
    # 45 pairs that share 300 to 700 tokens each: the longest runs are shared, the others read by each.
    e = Env(heads=4, kv=4, hd=64, page=16, pages=3200, seqs=91, seed=5)
    e.step(list(range(45)), [300 + 9 * i for i in range(45)], "bf16")
    for i in range(45):
        e.fork(i, 45 + i, 300 + 9 * i - i % 5)
    e.step(list(range(90)), [1] * 90, "bf16")
    assert e.shared("bf16")
    e.attend("bf16")
    # one chain: each continues the one before
    e = Env(heads=8, kv=8, hd=64, page=16, pages=900, seqs=41, seed=6)
    e.step([0], [200], "bf16")
    for i in range(40):
        e.fork(i, i + 1, e.kv.tokens(i) // 16 * 16)
        e.step([i + 1], [80], "bf16")
    e.step(list(range(41)), [1] * 41, "bf16")
    assert e.shared("bf16")
    e.attend("bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 3), (200, 0), (200, 70), (900, 4), (1100, 40), (5000, 0), (300, 2000)])
def test_windows_and_first_tokens(dtype, window, sinks):
    e = batch(16, 8, 64, 32, 1000, [0, 60, 3, 90, 20, 16, 1, 0, 33, 190, 5, 64, 2, 8, 31, 17, 40, 41, 42, 43], dtype, seed=window)
    e.attend(dtype, window=window, sinks=sinks)
    if window >= 900:
        assert e.shared(dtype, window=window, sinks=sinks)


def test_dropped_pages():
    # A window moved on: the shared first pages are gone but for the first tokens', those behind are still shared.
    e = batch(16, 8, 64, 16, 1200, [20 + 3 * i for i in range(20)], "bf16", seed=3)
    held = {}
    for s in range(1, 21):
        n = e.kv.tokens(s)
        gone = e.kv.evict(s, 1000, 5)
        assert gone > 0
        held[s] = np.ones(n + 10, bool)
        held[s][16:16 + 16 * gone] = False
    e.step(list(range(1, 21)), [1] * 20, "bf16")
    assert e.shared("bf16", window=1000, sinks=5) and e.shared("bf16")
    e.attend("bf16", window=1000, sinks=5, held=held)
    e.attend("bf16", held=held)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_nan_infinity_and_far_scales_in_the_shared_pages(dtype):
    e = Env(heads=8, kv=8, hd=64, page=16, pages=400, seqs=25, seed=11)
    rows = 1000
    e.extend([0], [rows])
    k, v = (e.rng.standard_normal((rows, 8, 64)).astype(np.float32) for _ in range(2))
    v *= np.repeat(2.0 ** e.rng.integers(-30, 8, (-(-rows // 16), 8)), 16, 0)[:rows, :, None].astype(np.float32)   # blocks of different magnitude
    v[20, 0, 5], v[300, 1, 7], v[640, 2, 0], k[400, 3, 3], k[401, 4, 4] = np.nan, np.inf, -np.inf, np.nan, np.inf
    kt, vt = torch.from_numpy(k), torch.from_numpy(v)
    e.append((kt, kt.double().numpy()), (vt, vt.double().numpy()), "f32")
    for i in range(1, 25):
        e.fork(0, i, rows - i % 3)
    e.step(list(range(1, 25)), [1 + 5 * i for i in range(24)], "f32")
    e.step(list(range(1, 25)), [1] * 24, "f32")
    assert e.shared(dtype)
    e.attend(dtype)
    e.attend(dtype, window=650, sinks=30)
    q = e.rand(24, 8, dtype)
    q[0][3, 1, 0], q[0][9, 5, 3] = float("nan"), float("nan")   # rows of their own, the others untouched
    e.attend(dtype, q=(q[0], q[0].double().numpy()))


def test_the_same_from_run_to_run_on_streams_and_in_graphs():
    e = batch(32, 8, 128, 32, 2000, [50 + 7 * i for i in range(20)], "bf16", seed=2)
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
    for window in (0, 1500):   # two graphs that share the cache's workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            e.kv.attend_shared(0, qd.data_ptr(), out.data_ptr(), "bf16", scale=0.1, window=window, stream=torch.cuda.current_stream().cuda_stream)
        graphs.append(g)
    for turn in range(3):
        qd.copy_(e.rand(20, 32, "bf16")[0])
        for g, window in zip(graphs, (0, 1500)):
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
    e = Env(heads=32, kv=32, hd=128, page=128, pages=4400, seqs=22, max_pages=4300, seed=4)
    e.kv.extend([21], [4200 * 128], e.stream())
    e.step([0], [1000], "bf16")
    assert int(min(e.kv.pages(0))) * 32 * 2 * 128 * 128 > 1 << 32
    for i in range(1, 21):
        e.fork(0, i, 1000)
    e.step(list(range(1, 21)), [1] * 20, "bf16")
    assert e.shared("bf16")
    e.attend("bf16")
