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
