"""Whole numbers that the C ABI's 32 bits cannot hold are refused by the binding, on either side: ctypes would cut them to other,
valid ones. Over the stand-in for the device of tests/test_ops_host.py."""
import pytest

from tests.test_ops_host import B, P, cache  # noqa: F401

CUT = [-(1 << 32), -(1 << 32) + 1, -(1 << 32) + 5, -(1 << 31) - 1, 1 << 31, 1 << 32, (1 << 32) + 1, -(1 << 70), 1 << 70]


@pytest.fixture
def calls(B):  # noqa: F811
    kv, rope = cache(B, head_dim=64), B.Rope(head_dim=64, device=1)
    kv.extend([0, 1], [700, 700])
    return {
        "append": lambda layer=0: kv.append(layer, P, P, "f32"),
        "attend": lambda layer=0, window=0, sinks=0: kv.attend(layer, P, P, "f32", scale=1.0, window=window, sinks=sinks),
        "attend_shared": lambda layer=0, window=0, sinks=0: kv.attend_shared(layer, P, P, "f32", scale=1.0, window=window, sinks=sinks),
        "rope.append": lambda layer=0: rope.append(kv, layer, P, P, P, P, "f32"),
        "rope.apply": lambda first=0, n_heads=2, n_kv_heads=0: rope.apply(4, P, P, n_heads, "f32", first=first, n_kv_heads=n_kv_heads),
    }


@pytest.mark.parametrize("x", CUT)
@pytest.mark.parametrize("call,names", [("append", ["layer"]), ("attend", ["layer", "window", "sinks"]), ("attend_shared", ["layer", "window", "sinks"]),
                                        ("rope.append", ["layer"]), ("rope.apply", ["first", "n_heads", "n_kv_heads"])])
def test_numbers_beyond_32_bits_are_refused(B, calls, call, names, x):  # noqa: F811
    calls[call]()
    for name in names:
        for other in ({}, {n: 1 for n in names if n != name and call != "rope.apply"}):
            launches = B.stub.stub_launches()
            with pytest.raises(OverflowError):
                calls[call](**{name: x}, **other)
            assert B.stub.stub_launches() == launches


@pytest.mark.parametrize("call,name", [("append", "layer"), ("attend", "layer"), ("attend", "window"), ("attend", "sinks"), ("attend_shared", "layer"),
                                       ("attend_shared", "window"), ("attend_shared", "sinks"), ("rope.append", "layer")])
def test_negative_numbers_that_fit_are_the_librarys_to_refuse(B, calls, call, name):  # noqa: F811
    for x in (-1, -(1 << 31)):
        with pytest.raises(B.NPError) as e:
            calls[call](**{name: x})
        assert e.value.status == B.NP_EINVAL
