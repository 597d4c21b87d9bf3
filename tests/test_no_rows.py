"""Calls without rows: they enqueue nothing, whatever their pointers are (an empty tensor has none), and refuse what is wrong besides.
Over the stand-in for the device of tests/test_ops_host.py."""
import pytest

from tests.test_ops_host import B, P, refused  # noqa: F401


def test_rope_apply(B):  # noqa: F811
    r = B.Rope(head_dim=64, device=1)
    launches = B.stub.stub_launches()
    for q, out, k, k_out in ((P, P, P, P), (0, 0, 0, 0), (P, 0, 0, P)):
        r.apply(0, q, out, 2, "bf16")
        r.apply(0, q, out, 2, "f32", k_ptr=k, k_out_ptr=k_out, n_kv_heads=1, first=2 ** 31 - 1)
        r.apply(0, q, out, 2, "f32", (128, 64, 128, 64, 0, 0, 0, 0), positions_ptr=P, q_weight_ptr=P)
    assert B.stub.stub_launches() == launches
    for a, kw in (((0, 0, 0, 0, "f32"), {}), ((0, 0, 0, 2, "f32"), dict(eps=-1.0)), ((0, 0, 0, 2, "f32"), dict(n_kv_heads=-1)), ((0, 0, 0, 2, "f32"), dict(k_ptr=P)),
                  ((0, 0, 0, 2, "f32"), dict(positions_ptr=P + 2)), ((0, 0, 0, 2, "bf16", (128, 4, 128, 64, 0, 0, 0, 0)), {}), ((1, 0, 0, 2, "f32"), {}), ((0, P + 4, P, 2, "f32"), {}), ((0, 0, 0, 2, "f32"), dict(q_weight_ptr=P + 8))):
        refused(B, B.NP_EINVAL, r.apply, *a, **kw)


def test_w4_matvec(B):  # noqa: F811
    w = B.W4(n_out=16, n_in=128, group=128, codes_ptr=P, scales_ptr=P, scale_dtype="f16", device=1)
    launches = B.stub.stub_launches()
    for x, y in ((P, P + 4096), (0, 0), (0, P), (P, 0), (P, P)):
        w.matvec(0, x, "bf16", y, "f32")
        w.matvec(0, x, "f32", y, "f16", x_stride=256, y_stride=100, accumulate=True)
    assert B.stub.stub_launches() == launches
    for a, kw in (((0, 0, "f32", 0, "f32"), dict(x_stride=130)), ((0, 0, "f32", 0, "f32"), dict(y_stride=15)), ((1, 0, "f32", P, "f32"), {}), ((1, P, "f32", 0, "f32"), {}), ((-1, 0, "f32", 0, "f32"), {}),
                  ((0, P + 4, "f32", 0, "f32"), {}), ((0, 0, "f32", P + 2, "f32"), {})):
        refused(B, B.NP_EINVAL, w.matvec, *a, **kw)


@pytest.mark.parametrize("status", ["NP_EHIP"])
def test_the_device_is_not_looked_for(B, status):  # noqa: F811
    r, w = B.Rope(head_dim=64, device=1), B.W4(n_out=16, n_in=128, group=128, codes_ptr=P, scales_ptr=P, scale_dtype="f16", device=1)
    B.stub.stub_fail_set_device(1)
    try:
        r.apply(0, 0, 0, 2, "f32")
        w.matvec(0, 0, "f32", 0, "f32")
        refused(B, getattr(B, status), r.apply, 1, P, P, 2, "f32")
    finally:
        B.stub.stub_fail_set_device(0)
