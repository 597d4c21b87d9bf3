"""examples/decode_attention.py: attention over the cache and the sparse FFN in one decode loop."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_decode_with_attention_and_sparse_ffn():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_attention.py")
    spec = importlib.util.spec_from_file_location("decode_attention", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    got = m.main()
    assert got["shared"] == 5                     # 77 tokens in pages of 16, all shared by the fork
    assert got["same"] and got["finite"]
    assert got["tokens"] == (81, 138)
    # sequence 1 had 137 tokens when it last dropped pages: tokens 16 .. 95 are gone (the first page holds the first tokens)
    assert got["dropped"] == 5
    assert got["moved"] >= 0 and got["free"] == 64 - (6 + 4 - 1)   # the first page is still shared


def test_the_example_packs_the_pages_that_its_calls_leave():
    # The same page calls on a cache without a device: the numbers that the example has to end with.
    import importlib.util as u
    from delta_prefetched_ffn_amd import KVCache
    from delta_prefetched_ffn_amd import binding as B
    kv = KVCache(n_layers=3, n_heads=4, n_kv_heads=4, head_dim=64, page_tokens=16, n_pages=64, max_seqs=3, max_pages=64, device=B.KV_HOST)
    kv.extend([0], [77])
    kv.fork(0, 1, 77)
    for _ in range(20):
        kv.extend([0, 1], [1, 1])
    dropped = 0
    for _ in range(40):
        kv.extend([1], [1])
        dropped += kv.evict(1, 32, 4)
    kv.trim(0, 80)
    moved = kv.compact()
    kv.extend([0, 1], [1, 1])
    assert moved > 0
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_attention.py")
    spec = u.spec_from_file_location("decode_attention", path)
    m = u.module_from_spec(spec)
    spec.loader.exec_module(m)
    got = m.main()
    assert (got["dropped"], got["moved"], got["tokens"], got["free"]) == (dropped, moved, (kv.tokens(0), kv.tokens(1)), kv.info()["free"])
