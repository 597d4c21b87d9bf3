"""Page bookkeeping and refusals of the 8-bit key/value cache, on the CPU: a cache with device KV_HOST keeps the same books
as one on a GPU, so every allocation rule and every refusal is checked here against a plain model."""
import ctypes
import random
import time

import numpy as np
import pytest

from delta_prefetched_ffn_amd import KVCache, NPError, kv_bytes
from delta_prefetched_ffn_amd import binding as B


def cache(**kw):
    base = dict(n_layers=2, n_heads=8, n_kv_heads=4, head_dim=64, page_tokens=16, n_pages=40, max_seqs=6, max_pages=12, device=B.KV_HOST)
    base.update(kw)
    return KVCache(**base)


def refused(status, f, *a, **kw):
    with pytest.raises(NPError) as e:
        f(*a, **kw)
    assert e.value.status == status, str(e.value)
    return str(e.value)


class Model:
    """Pages as lists, reference counts by counting."""

    def __init__(self, n_pages, max_seqs, pt, max_pages):
        self.n, self.pt, self.max_pages = n_pages, pt, max_pages
        self.seqs = [([], 0) for _ in range(max_seqs)]

    def refs(self, p):
        return sum(q.count(p) for q, _ in self.seqs)

    def free(self):
        used = {p for q, _ in self.seqs for p in q}
        return [p for p in range(self.n) if p not in used]

    def extend(self, seqs, new):
        trial = [(list(q), t) for q, t in self.seqs]
        saved, self.seqs = self.seqs, trial
        for s, n in zip(seqs, new):
            q, t = self.seqs[s]
            if -(-(t + n) // self.pt) > self.max_pages:
                self.seqs = saved
                return False
            if n and t % self.pt and self.refs(q[t // self.pt]) > 1:
                f = self.free()
                if not f:
                    self.seqs = saved
                    return False
                q[t // self.pt] = f[0]
            while len(q) < -(-(t + n) // self.pt):
                f = self.free()
                if not f:
                    self.seqs = saved
                    return False
                q.append(f[0])
            self.seqs[s] = (q, t + n)
        return True


def same(kv, m):
    for s, (q, t) in enumerate(m.seqs):
        assert kv.pages(s).tolist() == q, s
        assert kv.tokens(s) == t, s
    assert kv.info()["free"] == len(m.free())
    assert kv.info()["shared"] == sum(m.refs(p) > 1 for p in range(m.n))


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("pt", [16, 64])
def test_random_calls_against_a_plain_model(seed, pt):
    rng = random.Random(seed * 100 + pt)
    kv = cache(page_tokens=pt)
    m = Model(40, 6, pt, 12)
    for _ in range(400):
        op = rng.choice(["extend"] * 4 + ["fork", "copy", "trim", "free", "evict", "compact"])
        s = rng.randrange(6)
        q, t = m.seqs[s]
        if op == "extend":
            seqs = rng.sample(range(6), rng.randint(1, 3))
            new = [rng.choice([0, 1, 1, pt - 1, pt, 3 * pt + 5]) for _ in seqs]
            if m.extend(seqs, new):
                kv.extend(seqs, new)
            else:
                refused(B.NP_ECAPACITY, kv.extend, seqs, new)
        elif op in ("fork", "copy"):
            d = rng.randrange(6)
            n = rng.randint(0, t)
            if d == s or m.seqs[d][0]:
                refused(B.NP_EINVAL, kv.fork, s, d, n)
                continue
            pages = q[:-(-n // pt)]
            if n % pt and pages[-1] < 0:
                refused(B.NP_EINVAL, kv.fork, s, d, n)
                continue
            if op == "copy":
                free = m.free()
                if sum(p >= 0 for p in pages) > len(free):
                    refused(B.NP_ECAPACITY, kv.fork, s, d, n, "copy")
                    continue
                it = iter(free)
                pages = [next(it) if p >= 0 else -1 for p in pages]
            m.seqs[d] = (list(pages), n)
            kv.fork(s, d, n, "copy" if op == "copy" else "share")
        elif op == "trim":
            n = rng.randint(0, t)
            if n % pt and q[n // pt] < 0:
                refused(B.NP_EINVAL, kv.trim, s, n)
                continue
            m.seqs[s] = (q[:-(-n // pt)], n)
            kv.trim(s, n)
        elif op == "free":
            m.seqs[s] = ([], 0)
            kv.free(s)
        elif op == "evict":
            window, sinks = rng.randint(1, 4 * pt), rng.choice([0, 1, pt, pt + 1])
            gone = [i for i, p in enumerate(q) if p >= 0 and all(sinks <= j <= t - window for j in range(i * pt, (i + 1) * pt))]
            assert kv.evict(s, window, sinks) == len(gone)
            m.seqs[s] = ([-1 if i in gone else p for i, p in enumerate(q)], t)
        else:
            used = sorted({p for q, _ in m.seqs for p in q if p >= 0})
            holes = [p for p in range(len(used)) if p not in used]
            to = dict(zip([p for p in used if p >= len(used)], holes))
            assert kv.compact() == len(to)
            m.seqs = [([to.get(p, p) for p in q], t) for q, t in m.seqs]
        same(kv, m)
    kv.reset()
    assert kv.info() == {"n_pages": 40, "free": 40, "shared": 0, "current": 0}


def test_refused_extend_changes_nothing():
    kv = cache(n_pages=4)
    kv.extend([0, 1], [20, 16])
    before = [kv.pages(s).tolist() for s in range(6)]
    refused(B.NP_ECAPACITY, kv.extend, [2, 3], [16, 16])
    refused(B.NP_ECAPACITY, kv.extend, [0], [12 * 16])
    refused(B.NP_EINVAL, kv.extend, [0, 0], [1, 1])
    refused(B.NP_EINVAL, kv.extend, [6], [1])
    refused(B.NP_EINVAL, kv.extend, [-1], [1])
    refused(B.NP_EINVAL, kv.extend, [1], [-1])
    refused(B.NP_EINVAL, kv.extend, [], [])
    refused(B.NP_EINVAL, kv.extend, list(range(129)), [0] * 129)
    with pytest.raises(ValueError):
        kv.extend([0, 1], [1])
    assert [kv.pages(s).tolist() for s in range(6)] == before
    assert kv.info()["current"] == 2     # the step of the accepted extend is still current


def test_copies_on_write_are_counted_exactly():
    # 0 and 1 share a half-filled page; extending both needs one copy only: the second keeps the page.
    kv = cache(n_pages=2)
    kv.extend([0], [8])
    kv.fork(0, 1, 8)
    kv.extend([0, 1], [1, 1])
    assert kv.pages(0).tolist() == [1] and kv.pages(1).tolist() == [0]
    kv.free(0)
    kv.fork(1, 0, 9)
    kv.fork(1, 2, 9)
    refused(B.NP_ECAPACITY, kv.extend, [0, 1, 2], [1, 1, 1])   # two copies, one free page
    kv.extend([0], [1])
    assert kv.pages(0).tolist() == [1]


def test_adopt_refuses_pages_in_use_and_bad_pages():
    kv = cache()
    kv.adopt(0, [7, 3, 39], 33)
    for bad in ([7], [40], [-2], [5, 5], [1 << 30]):
        refused(B.NP_EINVAL, kv.adopt, 1, bad, 1)
    refused(B.NP_EINVAL, kv.adopt, 0, [1], 1)              # not empty
    refused(B.NP_EINVAL, kv.adopt, 1, [1], 17)             # too few pages
    refused(B.NP_EINVAL, kv.adopt, 1, [1], -1)
    refused(B.NP_EINVAL, kv.adopt, 1, list(range(13)), 0)  # max_pages
    refused(B.NP_EINVAL, kv.adopt, 1, [-1, 1], 8)          # the first page's tokens are not all past
    kv.adopt(1, [-1, 1], 20)                               # a dropped page
    assert kv.pages(1).tolist() == [-1, 1] and kv.tokens(1) == 20
    refused(B.NP_EINVAL, kv.trim, 1, 8)                    # would end inside the dropped page
    refused(B.NP_EINVAL, kv.fork, 1, 2, 8)
    kv.trim(1, 0)
    kv.adopt(2, [0, 1, 2], 0)                              # reserved pages, no tokens
    kv.extend([2], [40])
    assert kv.pages(2).tolist() == [0, 1, 2]


def test_current_tokens_end_with_their_sequence():
    kv = cache()
    kv.extend([0, 1], [20, 3])
    kv.fork(0, 2, 20)
    kv.compact()
    assert kv.info()["current"] == 2
    kv.trim(1, 2)
    assert kv.info()["current"] == 0
    refused(B.NP_ESTATE, kv.append, 0, 16, 16, "f32")
    refused(B.NP_ESTATE, kv.attend, 0, 16, 16, "f32", scale=1.0)


def test_append_and_attend_refusals():
    kv = cache()
    kv.extend([0, 1], [5, 2])
    good = 4096
    for layer in (-1, 2):
        refused(B.NP_EINVAL, kv.append, layer, good, good, "f32")
        refused(B.NP_EINVAL, kv.attend, layer, good, good, "f32", scale=1.0)
    L = B.lib()
    assert L.np_kv_append(kv.h, 0, good, good, 3, None, None) == B.NP_EINVAL
    assert L.np_kv_attend(kv.h, 0, good, good, None, -1, None, 1.0, 0, 0, None) == B.NP_EINVAL
    for bad in (0, 8, 4097):
        refused(B.NP_EINVAL, kv.append, 0, bad or None, good, "f32")
        refused(B.NP_EINVAL, kv.append, 0, good, bad or None, "bf16")
        refused(B.NP_EINVAL, kv.attend, 0, bad or None, good, "f16", scale=1.0)
        refused(B.NP_EINVAL, kv.attend, 0, good, bad or None, "f16", scale=1.0)
    for st in ((-256, 64, 256, 64), (256, 4, 256, 64), (258, 64, 256, 64), (256, 64, 1 << 50, 64)):
        refused(B.NP_EINVAL, kv.append, 0, good, good, "bf16", st)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        refused(B.NP_EINVAL, kv.attend, 0, good, good, "f32", scale=scale)
    refused(B.NP_EINVAL, kv.attend, 0, good, good, "f32", scale=1.0, window=-1)
    refused(B.NP_EINVAL, kv.attend, 0, good, good, "f32", scale=1.0, window=4, sinks=-1)
    refused(B.NP_EINVAL, kv.attend, 0, good, good, "f32", scale=1.0, lse_ptr=4098)
    for st in ((512, 64, 256, 64), (512, 64, 512, 32), (512, 64, 0, 64), (512, 64, 512, 0), (512, 64, 64, 256)):
        assert "overlap" in refused(B.NP_EINVAL, kv.attend, 0, good, good, "f32", st, scale=1.0)
    # everything in order: only the missing device is left to refuse
    for st in (None, (512, 64, 512, 64), (0, 0, 64, 7 * 64), (512, 64, 64, 448)):
        refused(B.NP_ESTATE, kv.attend, 0, good, good, "f32", st, scale=1.0)
    refused(B.NP_ESTATE, kv.append, 0, good, good, "f32", (0, 0, 256, 64))
    refused(B.NP_ESTATE, kv.read_tokens, 0, 0)
    refused(B.NP_EINVAL, kv.read_tokens, 0, 0, 1, 5)
    refused(B.NP_EINVAL, kv.read_tokens, 2, 0)
    refused(B.NP_EINVAL, kv.read_tokens, 0, 0, -1, 1)


def test_descriptors_out_of_range():
    ok = dict(n_layers=2, n_heads=8, n_kv_heads=4, head_dim=64, page_tokens=16, n_pages=40, max_seqs=6, max_pages=12)
    for k, bad in (("n_layers", (0, 1025)), ("n_heads", (0, 6, 4100)), ("n_kv_heads", (0, 3, 1025)), ("head_dim", (0, 4, 12, 264)),
                   ("page_tokens", (0, 8, 24, 256)), ("n_pages", (0, (1 << 24) + 1)), ("max_seqs", (0, 4097)),
                   ("max_pages", (0, (1 << 24) + 1))):
        for b in bad:
            refused(B.NP_EINVAL, cache, **{**ok, k: b})
    refused(B.NP_EINVAL, cache, **{**ok, "max_seqs": 4096, "max_pages": 1 << 17})
    assert kv_bytes(n_layers=3, n_heads=8, n_kv_heads=4, head_dim=80, page_tokens=32, n_pages=5) == (3 * 5 * 4 * 2 * 32 * 128, 3 * 5 * 4 * 2)
    L = B.lib()
    h = ctypes.c_void_p(1)
    assert L.np_kv_create(None, ctypes.byref(h)) == B.NP_EINVAL
    assert L.np_kv_bytes(None, None) == B.NP_EINVAL
    for f in ("np_kv_destroy", "np_kv_reset"):
        assert getattr(L, f)(None) == B.NP_EINVAL
    assert L.np_kv_extend(None, 1, None, None, None) == B.NP_EINVAL
    assert L.np_kv_trim(None, 0, 0) == B.NP_EINVAL
    assert L.np_kv_free(None, 0) == B.NP_EINVAL
    assert L.np_kv_fork(None, 0, 1, 0, 0, None) == B.NP_EINVAL
    assert L.np_kv_compact(None, None, None) == B.NP_EINVAL
    assert L.np_kv_info(None, None) == B.NP_EINVAL


def test_fork_trim_evict_refusals():
    kv = cache()
    kv.extend([0], [20])
    refused(B.NP_EINVAL, kv.fork, 0, 0, 3)
    refused(B.NP_EINVAL, kv.fork, 0, 1, 21)
    refused(B.NP_EINVAL, kv.fork, 0, 6, 1)
    refused(B.NP_EINVAL, kv.fork, 9, 1, 1)
    assert B.lib().np_kv_fork(kv.h, 0, 1, 1, 2, None) == B.NP_EINVAL
    refused(B.NP_EINVAL, kv.trim, 0, 21)
    refused(B.NP_EINVAL, kv.trim, 0, -1)
    refused(B.NP_EINVAL, kv.trim, 6, 0)
    refused(B.NP_EINVAL, kv.evict, 0, 0)
    refused(B.NP_EINVAL, kv.evict, 0, 4, -1)
    cap = np.zeros(1, np.int32)
    n = ctypes.c_int32()
    assert B.lib().np_kv_read_pages(kv.h, 0, cap.ctypes.data, 1, ctypes.byref(n), None) == B.NP_EINVAL


def test_strides_are_four_numbers():
    # A short tuple was filled up with zeros: every row of v the first one.
    kv = cache()
    kv.extend([0], [5])
    for bad in ((256, 64), (256, 64, 256), (), [256, 64], (256, 64, 256, 64, 1)):
        with pytest.raises(ValueError):
            kv.append(0, 4096, 4096, "f32", bad)
        with pytest.raises(ValueError):
            kv.attend(0, 4096, 4096, "f32", bad, scale=1.0)
    with pytest.raises(OverflowError):
        kv.append(0, 4096, 4096, "f32", (256, 64, 256, (1 << 64) + 64))
    for good in ((256, 64, 256, 64), [256, 64, 256, 64], np.array([256, 64, 256, 64])):
        for _ in range(2):
            refused(B.NP_ESTATE, kv.append, 0, 4096, 4096, "f32", good)   # only the missing device is left to refuse


def test_numbers_beyond_32_bits_are_refused():
    # They were cut to their lower 32 bits: a window of 2^32 + 5 became one of 5, a page 2^32 + 3 page 3.
    big = 1 << 32
    kv = cache()
    kv.extend([0], [40])
    before = kv.pages(0).tolist(), kv.tokens(0), kv.info()
    for call in (lambda: kv.extend([big + 1], [1]), lambda: kv.extend([1], [big + 1]), lambda: kv.append(big, 4096, 4096, "f32"),
                 lambda: kv.attend(big, 4096, 4096, "f32", scale=1.0), lambda: kv.attend(0, 4096, 4096, "f32", scale=1.0, window=big + 5),
                 lambda: kv.attend(0, 4096, 4096, "f32", scale=1.0, window=1 << 31), lambda: kv.attend(0, 4096, 4096, "f32", scale=1.0, window=7, sinks=big),
                 lambda: kv.trim(0, big), lambda: kv.trim(big, 0), lambda: kv.free(big), lambda: kv.fork(0, 1, big + 3), lambda: kv.fork(big, 1, 3),
                 lambda: kv.fork(0, big + 1, 3), lambda: kv.evict(0, big + 1), lambda: kv.evict(0, 1, big), lambda: kv.evict(big, 1),
                 lambda: kv.adopt(1, [big + 5], 1), lambda: kv.adopt(1, np.array([big + 5]), 1), lambda: kv.adopt(1, (big + 5,), 1),
                 lambda: kv.adopt(1, np.array([5, (1 << 63) + 9], np.uint64), 1), lambda: kv.adopt(1, [5], big + 1), lambda: kv.adopt(big + 1, [5], 1),
                 lambda: kv.pages(big), lambda: kv.tokens(big), lambda: kv.read_tokens(0, 0, 0, big), lambda: kv.read_tokens(big, 0),
                 lambda: cache(n_pages=big + 40), lambda: cache(max_seqs=(1 << 33) + 6),
                 lambda: kv_bytes(n_layers=big + 1, n_heads=8, n_kv_heads=4, head_dim=64, page_tokens=16, n_pages=5)):
        with pytest.raises(OverflowError):
            call()
    for pages in (np.array([5.0]), [5.0], np.array([[5, 6]])):
        with pytest.raises((TypeError, ValueError)):
            kv.adopt(1, pages, 1)
    assert before == (kv.pages(0).tolist(), kv.tokens(0), kv.info())
    for pages in ([20, 21], (20, 21), np.array([20, 21]), np.array([20, 21], np.uint8), np.array([20, 0, 21, 0], np.int32)[::2], np.array([20, 21], np.uint64)):
        kv.adopt(1, pages, 30)
        assert kv.pages(1).tolist() == [20, 21]
        kv.free(1)
    kv.adopt(1, [], 0)
    kv.adopt(1, np.array([], np.int32), 0)
    kv.extend(np.array([0, 1]), (np.int64(1), 2))
    assert kv.tokens(1) == 2


def test_taking_pages_does_not_search_the_pool_again():
    # 2^21 pages taken in one call, then the low half given back and taken again: each page's search began at page 0.
    kv = cache(n_layers=1, n_pages=1 << 21, max_pages=1 << 21)
    t = time.process_time()
    kv.extend([0], [1 << 24])
    kv.extend([1], [16 * (1 << 20)])
    t = time.process_time() - t
    assert kv.tokens(1) == 1 << 24
    kv.free(0)
    kv.extend([2], [1600])
    assert kv.pages(2).tolist() == list(range(100))
    kv.free(1)
    kv.compact()
    kv.extend([3], [16])
    assert kv.pages(3).tolist() == [100]
    kv.adopt(4, [101, 103], 20)
    kv.extend([5], [40])
    assert kv.pages(5).tolist() == [102, 104, 105]
    assert t < 2.0, f"{t:.1f} s for 2^21 pages"
