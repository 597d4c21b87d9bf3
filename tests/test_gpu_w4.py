"""Products with 4-bit weights on the GPU against the definition in fp64."""
import numpy as np
import pytest

from tests.harness import torch_mod

pytestmark = pytest.mark.gpu

torch = None
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative


@pytest.fixture(autouse=True, scope="module")
def _torch():
    global torch
    torch = torch_mod()
    assert torch.cuda.is_available()


def tdt(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def stream():
    return torch.cuda.current_stream().cuda_stream


class Matrix:
    def __init__(self, rng, n_out, n_in, group, scales="f16", zeros=True):
        from delta_prefetched_ffn_amd import W4
        groups = -(-n_in // group)
        self.c = rng.integers(0, 16, (n_out, n_in))
        self.z = rng.integers(0, 16, (n_out, groups)) if zeros else np.full((n_out, groups), 8)
        st = torch.from_numpy(((0.5 + rng.random((n_out, groups))) * np.where(rng.random((n_out, groups)) < 0.2, -0.01, 0.01)).astype(np.float32)).to(tdt(scales))
        self.s = st.double().numpy()
        codes = torch.from_numpy((self.c[:, 0::2] | self.c[:, 1::2] << 4).astype(np.uint8)).cuda()
        sd, zd = st.cuda(), torch.from_numpy((self.z | 0xA0).astype(np.uint8)).cuda()   # the zero points' upper bits do not count
        self.w = W4(n_out=n_out, n_in=n_in, group=group, codes_ptr=codes.data_ptr(), scales_ptr=sd.data_ptr(), scale_dtype=scales, zeros_ptr=zd.data_ptr() if zeros else 0)
        codes.fill_(0x55)   # read by create, not kept
        sd.fill_(9.0)
        self.n_out, self.n_in, self.group, self.groups = n_out, n_in, group, groups

    def product(self, x):
        """y, and what it may be off before its own rounding: per group at most one rounding a term (three for fp32's summands, counted always) in
        both sums, four more to join and scale, and one per group of the row and wave behind."""
        y, mag = np.zeros((len(x), self.n_out)), np.zeros((len(x), self.n_out))
        with np.errstate(invalid="ignore", over="ignore"):
            for g in range(self.groups):
                at = slice(g * self.group, min(self.n_in, (g + 1) * self.group))
                w = self.c[:, at] - self.z[:, g, None]
                y += x[:, at] @ (w * self.s[:, g, None]).T if np.isfinite(x).all() else (x[:, None, at] * (w * self.s[:, g, None])[None]).sum(-1)
                a = np.abs(x[:, at])
                mag += (a @ self.c[:, at].T + a.sum(-1, keepdims=True) * self.z[:, g]) * np.abs(self.s[:, g]) * (3 * min(self.group, 128) + 4 + -(-self.n_in // min(self.group, 128)) + 8)
        return y, mag * 2.0 ** -24


def check(got, want, slack, dtype):
    got = got.double().cpu().numpy()
    fin = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    tol = U[dtype] * np.abs(want) * 1.01 + slack + (2.0 ** -25 if dtype == "f16" else 2.0 ** -126)
    err = np.abs(got - want)[fin]
    assert (err <= tol[fin]).all(), f"{(err > tol[fin]).sum()} of {err.size} off, worst {(err / tol[fin]).max():.2f} bounds at {np.argwhere(fin)[(err / tol[fin]).argmax()]}"


def run(m, x, xd, yd, rows, accumulate=False, pad=0):
    xt = torch.from_numpy(x.astype(np.float32)).to(tdt(xd))
    dev = torch.full((rows, m.n_in + 8 * pad), float("nan"), dtype=xt.dtype, device="cuda")
    dev[:, :m.n_in] = xt.cuda()
    y = torch.full((rows, m.n_out + 3 * pad), 2.5, dtype=tdt(yd), device="cuda")
    m.w.matvec(rows, dev.data_ptr(), xd, y.data_ptr(), yd, x_stride=dev.stride(0) if pad else 0, y_stride=y.stride(0) if pad else 0, accumulate=accumulate, stream=stream())
    want, slack = m.product(xt.double().numpy())
    if accumulate:
        want = want + 2.5
        slack = slack + 2.0 ** -24 * np.abs(want)
    check(y[:, :m.n_out], want, slack, yd)
    assert not pad or bool((y[:, m.n_out:] == 2.5).all()), "written past the outputs"
    return y


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n_out,n_in,group,scales,zeros", [
    (16, 128, 128, "f16", True), (1, 8, 32, "f32", True), (17, 200, 64, "bf16", True), (100, 1000, 32, "f16", False), (130, 4104, 128, "f32", False),
    (33, 1544, 256, "bf16", True), (48, 640, 640, "f16", True), (257, 72, 64, "f32", True), (64, 2048, 131072, "f16", True)])
def test_shapes_groups_and_rows(xd, n_out, n_in, group, scales, zeros):
    rng = np.random.default_rng(n_out * 7 + n_in)
    m = Matrix(rng, n_out, n_in, group, scales, zeros)
    for rows in (1, 2, 5, 16, 17, 31, 33, 64, 65, 130):
        yd = ["f32", "bf16", "f16"][rows % 3]
        run(m, rng.standard_normal((rows, n_in)), xd, yd, rows, accumulate=rows % 2 == 1, pad=rows % 2)


@pytest.mark.parametrize("yd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
def test_types_and_accumulation(xd, yd):
    rng = np.random.default_rng(3)
    m = Matrix(rng, 90, 512, 128)
    for rows in (1, 20, 200):
        x = rng.standard_normal((rows, 512)) * 3
        run(m, x, xd, yd, rows)
        run(m, x, xd, yd, rows, accumulate=True)


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 16, 40, 150])
def test_infinities_and_nan_stay_in_their_row(xd, rows):
    rng = np.random.default_rng(rows)
    m = Matrix(rng, 70, 384, 64)
    m2 = Matrix(rng, 70, 384, 64, zeros=False)
    x = rng.standard_normal((rows, 384))
    x[0, 5] = np.inf
    if rows > 1:
        x[3, 7], x[4, 200], x[5, 0], x[5, 300], x[rows - 1, 383] = -np.inf, np.nan, np.inf, -np.inf, np.inf
        x[8] = 0.0
    for k in (m, m2):
        y = run(k, x, xd, "f32", rows)
        assert rows == 1 or bool((y[8] == 0).all())
    x = rng.standard_normal((rows, 384)) * (2.0 ** 12 if xd == "f16" else 2.0 ** 100)   # large, but within the sums' range
    run(m, x, xd, "f32", rows)


def kernel_of(m, xd, rows):
    from tests import test_gpu_kv as K
    K.torch = torch
    x, y = torch.zeros((rows, m.n_in), dtype=tdt(xd), device="cuda"), torch.zeros((rows, m.n_out), device="cuda")
    names = [n for n in K.kernels_of(lambda s: m.w.matvec(rows, x.data_ptr(), xd, y.data_ptr(), "f32", stream=s)) if "k_w4" in n]
    got = {"rows" if "k_w4_rows" in n else "eight waves" if "Li1ELi2ELi" in n else "four waves" for n in names}
    assert len(got) == 1
    return got.pop()


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n_out,n_in,group,scales", [(8190, 264, 32, "f16"), (8200, 520, 64, "f32"), (16400, 264, 128, "bf16"), (16390, 1032, 32, "f32")])
def test_many_outputs(xd, n_out, n_in, group, scales):
    # workgroups of one, two and four output tiles, the last of them in part past the outputs
    rng = np.random.default_rng(n_out)
    m = Matrix(rng, n_out, n_in, group, scales)
    for rows in (1, 7, 16, 18, 32, 49):
        run(m, rng.standard_normal((rows, n_in)), xd, ["bf16", "f32", "f16"][rows % 3], rows, accumulate=rows % 2 == 1, pad=rows % 2)


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n_out,rows,n_in,group,scales", [(130, 7301, 72, 32, "f16"), (1050, 1111, 264, 64, "f32"), (265, 4000, 392, 128, "bf16"), (16390, 129, 520, 256, "f16"), (2060, 640, 128, 32, "bf16"),
                                                            (1050, 3700, 72, 32, "f32"), (16390, 260, 392, 64, "f16"), (2060, 2000, 264, 128, "bf16")])
def test_many_rows_and_outputs(xd, n_out, rows, n_in, group, scales):
    rng = np.random.default_rng(rows)
    m = Matrix(rng, n_out, n_in, group, scales)
    many = -(-rows // 64) * -(-n_out // 128) > 512
    assert kernel_of(m, xd, rows) == ("four waves" if many and xd != "f32" else "eight waves")
    run(m, rng.standard_normal((rows, n_in)), xd, "f32", rows, accumulate=True)
    run(m, rng.standard_normal((rows, n_in)), xd, "bf16", rows, pad=1)


@pytest.mark.parametrize("xd", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n_out,rows,n_in,group", [(265, 3900, 200, 64), (20, 33000, 136, 32), (265, 3900, 264, 128)])
def test_infinities_and_nan_in_many_rows(xd, n_out, rows, n_in, group):
    rng = np.random.default_rng(11)
    m = Matrix(rng, n_out, n_in, group)
    x = rng.standard_normal((rows, n_in))
    x[3, 7], x[4, 130], x[5, 0], x[5, n_in - 1], x[rows - 1, n_in - 1], x[640, 64] = -np.inf, np.nan, np.inf, -np.inf, np.inf, np.inf
    x[8] = 0.0
    assert kernel_of(m, xd, rows) == ("four waves" if rows > 4000 and xd != "f32" else "eight waves")
    assert bool((run(m, x, xd, "f32", rows)[8] == 0).all())
    run(m, rng.standard_normal((rows, n_in)) * (2.0 ** 12 if xd == "f16" else 2.0 ** 100), xd, "f32", rows)


def test_small_values_and_exact_products():
    # x and scales that are powers of two: every sum is exact, so y is the nearest number of its type.
    rng = np.random.default_rng(8)
    m = Matrix(rng, 40, 256, 64)
    x = rng.integers(-8, 9, (70, 256)).astype(np.float64) * 2.0 ** -10
    from delta_prefetched_ffn_amd import W4
    one = torch.full((40, 4), 2.0 ** -3, device="cuda")
    codes = torch.from_numpy((m.c[:, 0::2] | m.c[:, 1::2] << 4).astype(np.uint8)).cuda()
    zd = torch.from_numpy(m.z.astype(np.uint8)).cuda()
    w = W4(n_out=40, n_in=256, group=64, codes_ptr=codes.data_ptr(), scales_ptr=one.data_ptr(), scale_dtype="f32", zeros_ptr=zd.data_ptr())
    want = x @ ((m.c - np.repeat(m.z, 64, 1)) * 2.0 ** -3).T
    for xd in ("f32", "bf16", "f16"):
        for rows in (1, 9, 30, 70):
            xt, y = torch.from_numpy(x[:rows].astype(np.float32)).to(tdt(xd)).cuda(), torch.empty((rows, 40), device="cuda")
            w.matvec(rows, xt.data_ptr(), xd, y.data_ptr(), "f32", stream=stream())
            assert np.array_equal(y.double().cpu().numpy(), want[:rows])
    full = (rng.standard_normal((1, 256)) * 1e3).astype(np.float32)   # all 24 bits of fp32 count: a basis row gives x back
    for rows in (1, 70):
        xt = torch.zeros((rows, 256), device="cuda")
        xt[0] = torch.from_numpy(full)
        c = np.full((256, 256), 8)
        c[np.arange(256), np.arange(256)] = 9
        codes = torch.from_numpy((c[:, 0::2] | c[:, 1::2] << 4).astype(np.uint8)).cuda()
        sc = torch.ones((256, 8), device="cuda")
        w = W4(n_out=256, n_in=256, group=32, codes_ptr=codes.data_ptr(), scales_ptr=sc.data_ptr(), scale_dtype="f32")
        y = torch.empty((rows, 256), device="cuda")
        w.matvec(rows, xt.data_ptr(), "f32", y.data_ptr(), "f32", stream=stream())
        # 9 x - 8 sum and the like: off by roundings of the group's sums only
        assert np.abs(y[0].double().cpu().numpy() - full[0]).max() <= 2.0 ** -24 * 200 * np.abs(full.reshape(8, 32)).sum(1).max()


def test_the_same_from_run_to_run_on_streams_and_in_graphs():
    rng = np.random.default_rng(4)
    m = Matrix(rng, 1000, 1024, 128)
    for rows in (1, 12, 64, 200, 1700, 5000):   # the last two take the tiles of many rows
        x = torch.from_numpy(rng.standard_normal((rows, 1024)).astype(np.float32)).bfloat16().cuda()
        want, y = torch.empty((rows, 1000), device="cuda"), torch.zeros((rows, 1000), device="cuda")
        m.w.matvec(rows, x.data_ptr(), "bf16", want.data_ptr(), "f32", stream=stream())
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        m.w.matvec(rows, x.data_ptr(), "bf16", y.data_ptr(), "f32", stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(y, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.w.matvec(rows, x.data_ptr(), "bf16", y.data_ptr(), "f32", accumulate=True, stream=stream())
        for n in range(3):   # y grows by each replay
            before = y.clone()
            x.mul_(0.5)
            g.replay()
            m.w.matvec(rows, x.data_ptr(), "bf16", before.data_ptr(), "f32", accumulate=True, stream=stream())
            torch.cuda.synchronize()
            assert torch.equal(y, before)


def test_columns_of_one_buffer_and_weights_past_4_gib_of_offsets():
    rng = np.random.default_rng(5)
    m = Matrix(rng, 64, 128, 32)
    both = torch.full((70, 200), 1.5, device="cuda")
    x = rng.standard_normal((70, 128)).astype(np.float32)
    both[:, :128] = torch.from_numpy(x)
    m.w.matvec(70, both.data_ptr(), "f32", both.data_ptr() + 4 * 130, "f32", x_stride=200, y_stride=200, stream=stream())
    want, slack = m.product(x.astype(np.float64))
    check(both[:, 130:194], want, slack, "f32")
    assert bool((both[:, 128:130] == 1.5).all()) and bool((both[:, 194:] == 1.5).all())
    # rows 2^29 elements apart: byte offsets past 32 bits
    far = torch.empty((3 << 29) + 128, dtype=torch.bfloat16, device="cuda")
    xs = rng.standard_normal((4, 128)).astype(np.float32)
    for r in range(4):
        far[r << 29:(r << 29) + 128] = torch.from_numpy(xs[r]).bfloat16()
    y = torch.empty((4, 64), device="cuda")
    m.w.matvec(4, far.data_ptr(), "bf16", y.data_ptr(), "f32", x_stride=1 << 29, stream=stream())
    want, slack = m.product(torch.from_numpy(xs).bfloat16().double().numpy())
    check(y, want, slack, "f32")


def test_weights_past_4_gib():
    # 2^20 outputs x 8,200 inputs: the last outputs' tiles lie past 2^32 bytes.
    from delta_prefetched_ffn_amd import W4
    n_out, n_in, last = 1 << 20, 8200, 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 256, (n_out, n_in // 2), dtype=torch.uint8, device="cuda", generator=gen)
    groups = -(-n_in // 4096)
    sc = (torch.rand((n_out, groups), device="cuda", generator=gen) + 0.5).bfloat16()
    w = W4(n_out=n_out, n_in=n_in, group=4096, codes_ptr=codes.data_ptr(), scales_ptr=sc.data_ptr(), scale_dtype="bf16")
    tail = codes[-last:].cpu().numpy().astype(np.int64)
    m = Matrix.__new__(Matrix)
    m.c = np.empty((last, n_in), np.int64)
    m.c[:, 0::2], m.c[:, 1::2] = tail & 15, tail >> 4
    m.z, m.s = np.full((last, groups), 8), sc[-last:].double().cpu().numpy()
    m.n_out, m.n_in, m.group, m.groups = last, n_in, 4096, groups
    del codes
    for rows in (1, 20, 70):
        x = torch.randn((rows, n_in), device="cuda", generator=gen).bfloat16()
        y = torch.empty((rows, n_out), device="cuda")
        w.matvec(rows, x.data_ptr(), "bf16", y.data_ptr(), "f32", stream=stream())
        want, slack = m.product(x.double().cpu().numpy())
        check(y[:, -last:], want, slack, "f32")
    w.close()


def test_refusals():
    from delta_prefetched_ffn_amd import W4, NPError
    from delta_prefetched_ffn_amd import binding as B
    buf = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = buf.data_ptr()
    good = dict(n_out=16, n_in=128, group=128, codes_ptr=p, scales_ptr=p, scale_dtype="f16")
    host = torch.zeros(64)
    for bad in (dict(n_out=0), dict(n_out=(1 << 20) + 1), dict(n_in=0), dict(n_in=12), dict(n_in=(1 << 17) + 8), dict(group=0), dict(group=16), dict(group=96), dict(group=192), dict(codes_ptr=0),
                dict(codes_ptr=p + 2), dict(scales_ptr=p + 1), dict(scales_ptr=0), dict(scales_ptr=p + 2, scale_dtype="f32"), dict(device=64), dict(codes_ptr=host.data_ptr()),
                dict(zeros_ptr=host.data_ptr())):
        with pytest.raises(NPError) as e:
            W4(**{**good, **bad})
        assert e.value.status == B.NP_EINVAL, bad
    w = W4(**good)
    for a, kw in [((-1, p, "f32", p + 4096, "f32"), {}), (((1 << 20) + 1, p, "f32", p + 4096, "f32"), {}), ((1, p + 4, "f32", p + 4096, "f32"), {}), ((1, 0, "f32", p + 4096, "f32"), {}),
                  ((1, p, "f32", p + 4098, "f32"), {}), ((1, p, "f32", p + 256, "f32"), {}), ((2, p, "f32", p + 4096, "f32"), dict(x_stride=130)), ((2, p, "f32", p + 4096, "f32"), dict(x_stride=64)),
                  ((2, p, "f32", p + 4096, "f32"), dict(y_stride=15)), ((2, p, "f32", p + 4 * 140, "f32"), dict(x_stride=144, y_stride=144)), ((1, host.data_ptr() // 16 * 16, "f32", p, "f32"), {}),
                  ((1, p, "f32", host.data_ptr(), "f32"), {}), ((2, p, "bf16", p + 4096, "f32"), dict(y_stride=-16))]:
        with pytest.raises(NPError) as e:
            w.matvec(*a, **kw)
        assert e.value.status == B.NP_EINVAL, (a, kw)
    w.matvec(0, p, "f32", p + 4096, "f32", stream=stream())
    torch.cuda.synchronize()
    assert bool((buf == 0).all())
    w.close()
