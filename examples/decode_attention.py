"""A small activation-sparse decoder: attention over the 8-bit key/value cache next to the sparse FFN, as a decode loop
uses them. A prompt is taken up, two continuations share its pages, each token runs every layer's attention
(np_kv_append, np_kv_attend) and sparse FFN (np_delta_assign, np_sparse_ffn_acc), the second continuation drops the pages
its window no longer sees, and at the end the cache is packed.

    python examples/decode_attention.py

Weights are random; the point is the order of the calls. Both continuations are given the same tokens first, and must
agree exactly: they read the same pages.
"""
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Decoder:
    def __init__(self, torch, *, layers=3, d=256, heads=4, page=16, pages=64, seqs=3, seed=0):
        from delta_prefetched_ffn_amd import KVCache, kv_bytes
        from delta_prefetched_ffn_amd import binding as B
        from workload.gen import Workload, small_config
        self.torch, self.d, self.heads, self.hd = torch, d, heads, d // heads
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.w = [[(torch.randn((d, n), device="cuda", generator=gen) / d ** 0.5).bfloat16() for n in (3 * d, d)] for _ in range(layers)]
        shape = dict(n_layers=layers, n_heads=heads, n_kv_heads=heads, head_dim=self.hd, page_tokens=page, n_pages=pages)
        codes, exps = (torch.zeros(n, dtype=torch.uint8, device="cuda") for n in kv_bytes(**shape))
        self.kv = KVCache(**shape, max_seqs=seqs, max_pages=pages, codes=codes.data_ptr(), exps=exps.data_ptr(), keepalive=(codes, exps))
        # The sparse FFN of each layer, its row store in HBM.
        self.wl = Workload(small_config(4000, L=layers, d=d, M=700, K=260, C=8, mode="union", m=90, swap=12, T=64))
        c = self.wl.cfg
        self.ffn = []
        for l in range(layers):
            store = torch.from_numpy(self.wl.store(l).reshape(-1).view(np.int16)).cuda()
            self.ffn.append(B.Layer(d_model=c.d, d_ff=c.M, k_max=c.K, n_rows=c.R, masks=self.wl.masks(l), mask_mode=B.MODES[c.mode],
                                    row_store=store.data_ptr(), keepalive=store))

    def attention(self, l, x, window=0, sinks=0):
        """x += attention of the current tokens; x fp32 [rows][d]."""
        torch, stream = self.torch, self.torch.cuda.current_stream().cuda_stream
        qkv = (x.bfloat16() @ self.w[l][0]).view(-1, 3 * self.heads, self.hd)
        q, k, v = qkv[:, :self.heads], qkv[:, self.heads:2 * self.heads], qkv[:, 2 * self.heads:]
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        self.kv.append(l, k.data_ptr(), v.data_ptr(), "bf16", (k.stride(0), k.stride(1), v.stride(0), v.stride(1)), stream)
        self.kv.attend(l, q.data_ptr(), out.data_ptr(), "bf16", (q.stride(0), q.stride(1), out.stride(0), out.stride(1)),
                       scale=self.hd ** -0.5, window=window, sinks=sinks, stream=stream)
        x += (out.view(-1, self.d) @ self.w[l][1]).float()

    def step(self, seqs, x, token, window=0, sinks=0):
        """One token of each sequence (x fp32 [len(seqs)][d]); `token` picks the layers' active neurons."""
        stream = self.torch.cuda.current_stream().cuda_stream
        self.kv.extend(seqs, [1] * len(seqs), stream)
        for l, ffn in enumerate(self.ffn):
            self.attention(l, x, window, sinks)
            gate, up = (int(c) for c in self.wl.cids()[token, l])
            ffn.delta_assign(gate, up, stream)
            for r in range(len(seqs)):   # the FFN is a batch-1 kernel: rows share the predicted neurons
                h = x[r].clone()
                ffn.sparse_ffn_acc(h.data_ptr(), x[r].data_ptr(), stream)
        return x


def main() -> dict:
    import torch
    assert torch.cuda.is_available(), "this example needs cuda:0"
    m = Decoder(torch)
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randn((77, m.d), device="cuda", generator=gen)
    m.kv.extend([0], [len(prompt)], torch.cuda.current_stream().cuda_stream)
    x = prompt.clone()
    for l in range(len(m.ffn)):
        m.attention(l, x)
    m.kv.fork(0, 1, len(prompt))
    shared = m.kv.info()["shared"]
    same = True
    for t in range(20):   # the same tokens on both: the first step copies the page they share half full
        x = torch.randn((1, m.d), device="cuda", generator=gen).repeat(2, 1)
        y = m.step([0, 1], x, t)
        same = same and torch.equal(y[0], y[1])
    dropped = 0
    for t in range(20, 60):   # sequence 1 goes on alone with a window of 32 and four first tokens
        y = m.step([1], torch.randn((1, m.d), device="cuda", generator=gen), t, window=32, sinks=4)
        dropped += m.kv.evict(1, 32, 4)
    m.kv.trim(0, 80)
    moved = m.kv.compact(torch.cuda.current_stream().cuda_stream)
    y = m.step([0, 1], torch.randn((2, m.d), device="cuda", generator=gen), 60, window=32, sinks=4)
    got = dict(shared=shared, same=bool(same), dropped=dropped, moved=moved, finite=bool(torch.isfinite(y).all()),
               tokens=(m.kv.tokens(0), m.kv.tokens(1)), free=m.kv.info()["free"])
    for ffn in m.ffn:
        ffn.close()
    m.kv.close()
    return got


if __name__ == "__main__":
    print(main())
