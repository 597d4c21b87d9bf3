"""An attention block of a language model with 4-bit weights: projection, rotary positions and norms on the way into the cache,
attention over the prompt that the sequences share, and the projection back onto the residual. Each stage is checked against its
definition in fp64, from what the stage before has really given it."""
import numpy as np
import pytest

from tests import kv_reference as KR
from tests import rope_reference as RR
from tests import test_gpu_kv as K
from tests import test_gpu_rope as T
from tests import test_gpu_shared as S
from tests import test_gpu_w4 as W
from tests.harness import torch_mod

pytestmark = pytest.mark.gpu

torch = None


@pytest.fixture(autouse=True, scope="module")
def _torch():
    global torch
    torch = K.torch = T.torch = S.torch = W.torch = torch_mod()
    assert torch.cuda.is_available()


class Block:
    def __init__(self, dtype, d=640, heads=32, kv=8, hd=128, page=64, pages=200, seqs=25, group=64):
        from delta_prefetched_ffn_amd import Rope
        rng = np.random.default_rng(1)
        self.dtype, self.d, self.heads, self.nkv, self.hd, self.group = dtype, d, heads, kv, hd, group
        self.wide = heads + 2 * kv
        self.qkv, self.back = W.Matrix(rng, self.wide * hd, d, group), W.Matrix(rng, d, heads * hd, group, scales="bf16")
        self.rope = Rope(head_dim=hd, base=500000.0)
        self.cache = T.Cache(heads=heads, kv=kv, hd=hd, page=page, pages=pages, seqs=seqs)
        self.kv = self.cache.kv
        self.wq, self.wk = T.weights(rng, hd), T.weights(rng, hd)
        self.dwq, self.dwk = torch.from_numpy(self.wq).cuda(), torch.from_numpy(self.wk).cuda()

    def run(self, x, h):
        """h (fp32) += the block of x."""
        s, rows, hd = torch.cuda.current_stream().cuda_stream, x.shape[0], self.hd
        qkv = torch.empty((rows, self.wide, hd), dtype=x.dtype, device="cuda")
        q, att = (torch.empty((rows, self.heads, hd), dtype=x.dtype, device="cuda") for _ in range(2))
        self.qkv.w.matvec(rows, x.data_ptr(), self.dtype, qkv.data_ptr(), self.dtype, stream=s)
        k, v = qkv[:, self.heads:], qkv[:, self.heads + self.nkv:]
        w = self.wide * hd
        self.rope.append(self.kv, 0, qkv.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), self.dtype, (w, hd, self.heads * hd, hd, w, hd, w, hd),
                         q_weight_ptr=self.dwq.data_ptr(), k_weight_ptr=self.dwk.data_ptr(), eps=1e-5, stream=s)
        self.kv.attend_shared(0, q.data_ptr(), att.data_ptr(), self.dtype, scale=hd ** -0.5, stream=s)
        self.back.w.matvec(rows, att.data_ptr(), self.dtype, h.data_ptr(), "f32", accumulate=True, stream=s)
        return qkv, q, att

    def check(self, seqs, new, x):
        rows, hd = x.shape[0], self.hd
        h0 = torch.randn((rows, self.d), device="cuda")
        h = h0.clone()
        qkv, q, att = self.run(x, h)
        torch.cuda.synchronize()
        want, slack = self.qkv.product(x.double().cpu().numpy())
        W.check(qkv.view(rows, -1), want, slack, self.dtype)
        x64, q64, a64 = (t.double().cpu().numpy() for t in (qkv, q, att))
        before = [self.kv.tokens(s) - n for s, n in zip(seqs, new)]
        pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, new)])
        f, eps = RR.freqs(hd, base=500000.0), float(np.float32(1e-5))
        want, mag = RR.turned(x64[:, :self.heads], pos, f, "half", 1.0, self.wq.astype(np.float64), eps)
        T.same(q, want, mag, self.dtype, "q")
        want, mag = RR.turned(x64[:, self.heads:self.heads + self.nkv], pos, f, "half", 1.0, self.wk.astype(np.float64), eps)
        row = 0
        for s, n, b in zip(seqs, new, before):
            T.check_block(self.cache, self.kv, s, want[row:row + n], mag[row:row + n], b)
            k, v = (t.astype(np.float64) for t in self.kv.read_tokens(0, s))
            some = range(n) if n < 4 else (0, 1, n // 2, n - 1)
            for i in some:
                y, _, terms, m = S.attention(q64[row + i:row + i + 1], k[:b + i + 1], v[:b + i + 1], b + i, hd ** -0.5)
                assert (np.abs(a64[row + i] - y[0]) <= KR.bound(y, terms, m, b + i + 1, hd, self.dtype)[0]).all(), f"seq {s}, token {i}"
            row += n
        want, slack = self.back.product(a64.reshape(rows, -1))
        want = want + h0.double().cpu().numpy()
        W.check(h, want, slack + 2.0 ** -24 * np.abs(want), "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_prompt_its_continuations_and_a_captured_step(dtype):
    b = Block(dtype)
    rng = np.random.default_rng(2)

    def x_of(rows):
        return torch.from_numpy(rng.standard_normal((rows, b.d)).astype(np.float32)).to(K.tdt(dtype)).cuda()

    s = torch.cuda.current_stream().cuda_stream
    b.kv.extend([0], [4003], s)
    b.check([0], [4003], x_of(4003))
    seqs = list(range(1, 25))
    for i in seqs:
        b.kv.fork(0, i, 4003)
    new = [1 + i % 3 for i in seqs]
    b.kv.extend(seqs, new, s)
    x = x_of(sum(new))
    b.check(seqs, new, x)
    b.kv.extend(seqs, [1] * 24, s)
    x = x_of(24)
    assert any("k_prefix" in n for n in K.kernels_of(lambda _: b.run(x, torch.zeros((24, b.d), device="cuda"))))
    b.check(seqs, [1] * 24, x)
    # The step as a graph: each replay against the same calls made after it.
    h, want = torch.zeros((24, b.d), device="cuda"), torch.zeros((24, b.d), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run(x, h)
    for _ in range(3):
        x.copy_(x_of(24))
        want.copy_(h)
        g.replay()
        b.run(x, want)
        torch.cuda.synchronize()
        assert torch.equal(h, want)
