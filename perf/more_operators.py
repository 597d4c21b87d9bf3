"""The operators around the attention of a decode loop, as cases to be measured: products with 4-bit weights, rotary positions
with the norms of queries and keys in the same pass, the same on the way into the 8-bit key/value cache, and attention over
that cache for sequences that share their first pages.

Each operator has a plain form here (elementary torch operations in 32 bits, angles in 64) and the framework's own call (`own`).

4-bit weights: code c of row o and column i (byte i // 2 of the row, its low 4 bits for an even i), in groups of `group`
columns: w[o, i] = scale[o, i // group] * (c - zero[o, i // group]), zero 8 where there are none; y = x w^T.

Rotary positions: of a head's first `rot` values, pair i (values i and i + rot / 2 in the "half" layout, 2 i and 2 i + 1 in the
"interleaved" one) turns by position * f_i: (a, b) -> amplitude * (a cos - b sin, a sin + b cos). f_i = base^(-2 i / rot), divided by
`factor` ("linear"), or of a larger base ("ntk": base * factor^(rot / (rot - 2))), or ("blend") divided by it where the pair makes
fewer than `low` turns over `context` positions, as it is above `high` turns, and in between in proportion. A norm before it:
x * weight / sqrt(mean(x^2) + eps) over the head.

The cache's format is that of perf/operators.py: `codes` uint8 [layers][pages][kv heads][2][page_tokens / 16][hd64 / 64][1024] of
e4m3 values, `exps` int8 [layers][pages][kv heads][2], value = code * 2^exp; for K, byte (16 g + t) * 16 + b of 16 tokens x 64 values is
token t, value 16 g + b; for V, byte (16 g + r) * 16 + 4 i + t is token 4 g + t, value 4 r + i.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    plain = dict(scaling="none", factor=1.0, context=0, low=0.0, high=0.0, amplitude=1.0)
    far = dict(scaling="blend", factor=16.0, context=4096, low=1.0, high=32.0, amplitude=1.2772588722239782)
    near = dict(scaling="blend", factor=8.0, context=8192, low=1.0, high=4.0, amplitude=1.0)
    return [
        # One decode token's output projection, d_model 4096: a call bound by its latency.
        dict(name="w4_token", op="w4", rows=1, n_in=4096, n_out=4096, group=128, zeros=False, scales="f16", x="bf16", y="bf16"),
        # One token through a projection as wide as the FFN (d_ff 11008 to d_model 4096), in the framework's own fp32 activations, small groups with zero points.
        dict(name="w4_token_wide", op="w4", rows=1, n_in=11008, n_out=4096, group=64, zeros=True, scales="f32", x="f32", y="f32"),
        # A small batch's scores over a vocabulary of 32,000: bound by the weights' bytes.
        dict(name="w4_batch", op="w4", rows=12, n_in=4096, n_out=32000, group=128, zeros=True, scales="f16", x="f16", y="f32"),
        # A prompt's fused projection to queries, keys and values (d_model 5120): bound by the matrix units.
        dict(name="w4_prompt", op="w4", rows=1500, n_in=5120, n_out=15360, group=128, zeros=False, scales="bf16", x="bf16", y="bf16"),
        # One decode token's queries and keys, normalised and turned, from the fused projection's output: latency.
        dict(name="rope_token", op="rope", rows=1, heads=32, kv_heads=32, hd=128, rot=128, layout="half", norm=True, base=10000.0, **plain, first=4097, spread=0, dtype="bf16", fused=True),
        # A long prompt, half of each head turned, for a context sixteen times the trained one; no norms.
        dict(name="rope_prompt", op="rope", rows=4099, heads=32, kv_heads=8, hd=128, rot=64, layout="interleaved", norm=False, base=10000.0, **far, first=0, spread=61000, dtype="f16", fused=False),
        # One decode token on its way into the cache: norms, turn, quantised keys and values in one call.
        dict(name="take_token", op="take", seqs=1, heads=32, kv_heads=32, hd=128, rot=128, layout="half", norm=True, base=10000.0, **plain, page=64, new=1, before=701, lens_seed=1, dtype="bf16", fused=True),
        # A serving step of many sequences, grouped heads, a longer context than the trained one.
        dict(name="take_batch", op="take", seqs=48, heads=32, kv_heads=8, hd=128, rot=128, layout="half", norm=False, base=500000.0, **near, page=32, new=1, before=20000, lens_seed=2, dtype="f16", fused=False),
        # A prompt taken up behind a short system prompt that ends inside a page.
        dict(name="take_prompt", op="take", seqs=1, heads=32, kv_heads=32, hd=128, rot=128, layout="half", norm=True, base=10000.0, **plain, page=64, new=4097, before=37, lens_seed=3, dtype="bf16", fused=True),
        # The smallest model (4 heads of 64), three continuations of one prompt: latency.
        dict(name="prefix_tiny", op="prefix", seqs=3, families=1, heads=4, kv_heads=4, hd=64, page=16, prefix=300, tail=20, new=1, lens_seed=4, dtype="f32", window=0, sinks=0),
        # A serving step of 32 conversations behind one system prompt of 8,011 tokens, grouped heads.
        dict(name="prefix_batch", op="prefix", seqs=32, families=1, heads=32, kv_heads=8, hd=128, page=64, prefix=8011, tail=600, new=1, lens_seed=5, dtype="bf16", window=0, sinks=0),
        # Ninety questions about two long documents, three drafted tokens each.
        dict(name="prefix_long", op="prefix", seqs=90, families=2, heads=32, kv_heads=8, hd=128, page=32, prefix=30001, tail=700, new=3, lens_seed=6, dtype="bf16", window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _draw_turn(rng, hd):
    layout = rng.choice(["half", "interleaved"])
    rot = rng.choice([hd, hd, hd // 2, 2 * rng.randint(1, hd // 2)])
    rot = max(4, rot - rot % 2)
    got = dict(rot=rot, layout=layout, norm=rng.random() < 0.6, base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=rng.choice(["none", "linear", "ntk", "blend"]),
               factor=1.0, context=0, low=0.0, high=0.0, amplitude=1.0)
    if got["scaling"] != "none":
        got["factor"] = rng.choice([2.0, 4.0, 8.0, 32.0])
    if got["scaling"] == "blend":
        got.update(context=rng.choice([2048, 4096, 8192]), low=1.0, high=rng.choice([4.0, 32.0]), amplitude=rng.choice([1.0, 0.1 * math.log(got["factor"]) + 1]))
    return got


def draw(rng):
    op = rng.choice(["w4", "w4", "rope", "take", "prefix", "prefix"])
    if op == "w4":
        rows = rng.choice([1, _log(rng, 1, 64), _log(rng, 1, 64), _log(rng, 65, 1500)])
        n_in, n_out = 8 * _log(rng, 8, 1376), _log(rng, 64, 32000)
        while rows * n_in * n_out > 1500 * 5120 * 15360:
            n_out //= 2
        return dict(op=op, rows=rows, n_in=n_in, n_out=n_out, group=rng.choice([32, 64, 128, 128]), zeros=rng.random() < 0.5, scales=rng.choice(["f32", "f16", "bf16"]),
                    x=rng.choice(["f32", "f16", "bf16"]), y=rng.choice(["f32", "f16", "bf16"]))
    hd, kv, group = rng.choice([64, 128, 128, 80, 96, 40, 256]), _log(rng, 1, 40), rng.choice([1, 1, 2, 4, 7, 8])
    while group * kv > 64:
        kv = (kv + 1) // 2
    case = dict(op=op, heads=group * kv, kv_heads=kv, hd=hd, dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "rope":
        return dict(case, rows=_log(rng, 1, 4099), **_draw_turn(rng, hd), first=_log(rng, 1, 100000) - 1, spread=rng.choice([0, 100, 200000]), fused=rng.random() < 0.5)
    case.update(page=rng.choice([16, 32, 64, 128]), lens_seed=rng.randint(0, 1 << 30))
    if op == "take":
        return dict(case, seqs=_log(rng, 1, 64), **_draw_turn(rng, hd), new=_log(rng, 1, 256), before=_log(rng, 1, 2000), fused=rng.random() < 0.5)
    case.update(seqs=_log(rng, 2, 90), prefix=_log(rng, 20, 30000), tail=_log(rng, 1, 700), new=rng.choice([1, 1, 1, 2, 5, 9]), window=0, sinks=0)
    case["families"] = min(case["seqs"], rng.choice([1, 1, 2, 5]))
    if rng.random() < 0.2:
        case.update(window=_log(rng, 1, 20000), sinks=rng.choice([0, 4, 64]))
    while case["seqs"] * case["new"] * case["heads"] * (case["prefix"] + case["tail"]) > 90 * 3 * 32 * 30701:
        case["prefix"] = max(20, case["prefix"] // 2)
    while case["seqs"] * case["kv_heads"] * (case["tail"] + case["page"]) * hd > 90 * 8 * 732 * 128 and case["seqs"] > 2:
        case["seqs"] = max(2, case["seqs"] // 2)
    case["families"] = min(case["families"], case["seqs"])
    return case


def _lengths(case):
    """Per sequence (tokens before the call, new tokens): the first takes the case's own figures, the others spread below them."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "take":
        got = [(case["before"], case["new"])]
        for _ in range(case["seqs"] - 1):
            got.append((rng.randint(case["before"] // 8, case["before"]), rng.randint(max(1, case["new"] // 3), case["new"])))
        return got
    prefix = [case["prefix"]] + [rng.randint(case["prefix"] // 2, case["prefix"]) for _ in range(case["families"] - 1)]
    tail = [case["tail"]] + [rng.randint(max(1, case["tail"] // 8), case["tail"]) for _ in range(case["seqs"] - 1)]
    return [(prefix[i % case["families"]], tail[i]) for i in range(case["seqs"])]


def _hd64(case):
    return -(-case["hd"] // 64) * 64


# --------------------------------------------------------------------------------------------------------------- inputs

def _pool(case, pages, gen):
    """Codes spread as a quantised block's are (its largest near 448 * 0.5..1), and exponents of values of about 0.4 to 3."""
    shape = (1, pages, case["kv_heads"], 2, case["page"] // 16, _hd64(case) // 64, 1024)
    codes = (torch.randn(shape, device="cuda", generator=gen) * 96).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    if case["hd"] != _hd64(case):
        slabs = (torch.arange(_hd64(case), device="cuda") >= case["hd"]).view(-1, 64)
        codes[:, :, :, 0].masked_fill_(slabs.view(-1, 4, 1, 16).expand(-1, 4, 16, 16).reshape(-1, 1024), 0)
        codes[:, :, :, 1].masked_fill_(slabs.view(-1, 1, 16, 4, 1).expand(-1, 4, 16, 4, 4).reshape(-1, 1024), 0)
    exps = torch.randint(-8, -5, (1, pages, case["kv_heads"], 2), device="cuda", generator=gen).to(torch.int8)
    return codes, exps


def _rows(case, rows, gen):
    """q, k, v [rows][heads][hd], about 0.75 in size: tensors of their own, or views of one fused projection output."""
    H, Hk, hd, t = case["heads"], case["kv_heads"], case["hd"], DTYPES[case["dtype"]]
    if case["fused"]:
        both = (torch.randn((rows, H + 2 * Hk, hd), device="cuda", generator=gen) * 0.75).to(t)
        return both[:, :H], both[:, H:H + Hk], both[:, H + Hk:]
    return tuple((torch.randn((rows, n, hd), device="cuda", generator=gen) * 0.75).to(t) for n in (H, Hk, Hk))


def _weights(case, s, gen):
    """The norms' weights of queries and keys, about 0.75."""
    s["wq"] = s["wk"] = None
    if case["norm"]:
        s["wq"], s["wk"] = (0.75 + 0.05 * torch.randn(case["hd"], device="cuda", generator=gen) for _ in range(2))


def _rope(case):
    from delta_prefetched_ffn_amd import Rope
    return Rope(head_dim=case["hd"], rot_dim=case["rot"], layout=case["layout"], base=case["base"], scaling=case["scaling"], factor=case["factor"], context=case["context"],
                low=case["low"], high=case["high"], amplitude=case["amplitude"])


def _cache(case, s, pages, seqs, per_seq):
    from delta_prefetched_ffn_amd import KVCache
    return KVCache(n_layers=1, n_heads=case["heads"], n_kv_heads=case["kv_heads"], head_dim=case["hd"], page_tokens=case["page"], n_pages=pages, max_seqs=seqs,
                   max_pages=per_seq, codes=s["codes"].data_ptr(), exps=s["exps"].data_ptr(), keepalive=(s["codes"], s["exps"]))


def _turns(case):
    """What each pair turns by per position, in radians (64 bits)."""
    i, rot, factor = np.arange(case["rot"] // 2, dtype=np.float64), case["rot"], case["factor"]
    base = case["base"] * factor ** (rot / (rot - 2)) if case["scaling"] == "ntk" else case["base"]
    f = base ** (-2 * i / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "blend":
        keep = np.clip((case["context"] * f / (2 * np.pi) - case["low"]) / (case["high"] - case["low"]), 0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    s = {"case": case}
    if case["op"] == "w4":
        n_out, n_in, groups = case["n_out"], case["n_in"], -(-case["n_in"] // case["group"])
        s["codes"] = torch.randint(0, 256, (n_out, n_in // 2), device="cuda", generator=gen, dtype=torch.uint8)
        s["scales"] = ((0.5 + torch.rand((n_out, groups), device="cuda", generator=gen)) * (0.25 / n_in ** 0.5)).to(DTYPES[case["scales"]])
        s["zeros"] = torch.randint(5, 11, (n_out, groups), device="cuda", generator=gen, dtype=torch.uint8) if case["zeros"] else None
        s["x"] = torch.randn((case["rows"], n_in), device="cuda", generator=gen).to(DTYPES[case["x"]])
        if own:
            from delta_prefetched_ffn_amd import W4
            s["w"] = W4(n_out=n_out, n_in=n_in, group=case["group"], codes_ptr=s["codes"].data_ptr(), scales_ptr=s["scales"].data_ptr(), scale_dtype=case["scales"],
                        zeros_ptr=s["zeros"].data_ptr() if case["zeros"] else 0)
        return s
    if case["op"] in ("rope", "take"):
        s["f"] = torch.from_numpy(_turns(case)).cuda()
    if case["op"] == "rope":
        _weights(case, s, gen)
        s["q"], s["k"], _ = _rows(case, case["rows"], gen)
        pos = torch.arange(case["rows"], device="cuda") + case["first"]
        if case["spread"]:
            pos = torch.randint(case["first"], case["first"] + case["spread"], (case["rows"],), device="cuda", generator=gen)
        s["pos"] = pos.to(torch.int32)
        if own:
            s["rope"] = _rope(case)
        return s
    page, lens = case["page"], _lengths(case)
    if case["op"] == "take":
        _weights(case, s, gen)
        held = [-(-(b + n) // page) for b, n in lens]
        pages = sum(held) + 3
        s["codes"], s["exps"] = _pool(case, pages, gen)
        order = host.sample(range(pages), sum(held))
        s["lens"], s["tables"] = lens, [order[sum(held[:i]):sum(held[:i + 1])] for i in range(len(lens))]
        s["q"], s["k"], s["v"] = _rows(case, sum(n for _, n in lens), gen)
        # The plain form's plan: the page table, the rows' positions, the pages that new tokens touch.
        table = np.zeros((len(lens), max(held)), np.int64)
        for i, t in enumerate(s["tables"]):
            table[i, :len(t)] = t
        s["table"] = torch.from_numpy(table).cuda()
        s["before"] = torch.tensor([b for b, _ in lens], device="cuda")
        s["new"] = torch.tensor([n for _, n in lens], device="cuda")
        s["row0"] = s["new"].cumsum(0) - s["new"]
        s["pos"] = torch.cat([torch.arange(b, b + n, device="cuda") for b, n in lens])
        s["touched"] = torch.tensor([(i, p) for i, (b, n) in enumerate(lens) for p in range(b // page, held[i])], device="cuda")
        if own:
            s["rope"] = _rope(case)
            s["kv"] = _cache(case, s, pages, len(lens), max(held))
            for i, (b, _) in enumerate(lens):
                s["kv"].adopt(i, s["tables"][i], b)
            s["kv"].extend(list(range(len(lens))), [n for _, n in lens])
        return s
    # Prompts, one for each family, that lie scattered in the pool; every sequence forks its family's, goes on by its tail (a copy
    # of the prompt's last page where that is not full, then the free pages with the lowest numbers), and then by the new tokens.
    n, new, families = len(lens), case["new"], case["families"]
    upto = [p + t + new for p, t in lens]
    pages = sum(-(-p // page) for p, _ in lens[:families]) + sum(-(-u // page) - p // page for u, (p, _) in zip(upto, lens)) + 3
    s["codes"], s["exps"] = _pool(case, pages, gen)
    left, s["prompts"] = set(range(pages)), []
    for p, _ in lens[:families]:
        s["prompts"].append(host.sample(sorted(left), -(-p // page)))
        left -= set(s["prompts"][-1])
    free = iter(sorted(left))
    tables, copies = [], []
    for i, (p, t) in enumerate(lens):
        prompt = s["prompts"][i % families]
        tables.append(prompt[:p // page] + [next(free) for _ in range(-(-(p + t) // page) - p // page)])
        if p % page:
            copies.append((prompt[-1], tables[-1][p // page]))
    for i, u in enumerate(upto):
        tables[i] += [next(free) for _ in range(-(-u // page) - len(tables[i]))]
    s["lens"], s["tables"] = lens, tables
    s["q"] = torch.randn((n * new, case["heads"], case["hd"]), device="cuda", generator=gen).to(DTYPES[case["dtype"]])
    if own:
        s["kv"] = _cache(case, s, pages, families + n, max(map(len, tables)))
        for f, prompt in enumerate(s["prompts"]):
            s["kv"].adopt(f, prompt, lens[f][0])
        for i, (p, _) in enumerate(lens):
            s["kv"].fork(i % families, families + i, p)
        stream = torch.cuda.current_stream().cuda_stream
        s["kv"].extend([families + i for i in range(n)], [t for _, t in lens], stream)
        s["kv"].extend([families + i for i in range(n)], [new] * n, stream)
    else:
        for a, b in copies:
            s["codes"][:, b], s["exps"][:, b] = s["codes"][:, a], s["exps"][:, a]
    # The plain form's plan: the pages of each family's shared part and of each sequence's own, and where a sequence stands in its family.
    whole = [p // page for p, _ in lens]
    shared = np.zeros((families, max(1, max(whole[:families]))), np.int64)
    for f in range(families):
        shared[f, :whole[f]] = s["prompts"][f][:whole[f]]
    rest = np.zeros((n, max(len(t) - w for t, w in zip(tables, whole))), np.int64)
    for i, (t, w) in enumerate(zip(tables, whole)):
        rest[i, :len(t) - w] = t[w:]
    s["shared"], s["rest"] = torch.from_numpy(shared).cuda(), torch.from_numpy(rest).cuda()
    s["whole"] = torch.tensor(whole, device="cuda") * page
    s["before"] = torch.tensor([p + t for p, t in lens], device="cuda")
    s["family"] = torch.tensor([i % families for i in range(n)], device="cuda")
    s["place"] = torch.tensor([i // families for i in range(n)], device="cuda")
    return s


# ----------------------------------------------------------------------------------------------------------- plain forms

def _w4(s):
    case = s["case"]
    c = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(case["n_out"], -1).float()
    zero = 8.0 if s["zeros"] is None else s["zeros"].float().repeat_interleave(case["group"], 1)[:, :case["n_in"]]
    w = (c - zero) * s["scales"].float().repeat_interleave(case["group"], 1)[:, :case["n_in"]]
    return torch.matmul(s["x"].float(), w.t()).to(DTYPES[case["y"]])


def _turned(case, x, pos, f, weight):
    """x [rows][heads][hd], normalised and turned, in fp32."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    angle = pos.double()[:, None] * f
    cos, sin = (angle.cos() * case["amplitude"]).float()[:, None], (angle.sin() * case["amplitude"]).float()[:, None]
    rot = case["rot"]
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat((a * cos - b * sin, a * sin + b * cos, x[..., rot:]), -1)
    a, b = x[..., :rot:2], x[..., 1:rot:2]
    return torch.cat((torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2), x[..., rot:]), -1)


def _k_plain(c):
    """[..., groups, slabs, 1024] K bytes -> [..., tokens, hd64]."""
    *a, G, S, _ = c.shape
    return c.reshape(*a, G, S, 4, 16, 16).movedim(-2, -4).reshape(*a, G * 16, S * 64)


def _v_plain(c):
    *a, G, S, _ = c.shape
    n = len(a)
    return c.reshape(*a, G, S, 4, 16, 4, 4).permute(*range(n), n, n + 2, n + 5, n + 1, n + 3, n + 4).reshape(*a, G * 16, S * 64)


def _k_tiles(x):
    """The inverse of _k_plain."""
    *a, T, D = x.shape
    return x.reshape(*a, T // 16, 16, D // 64, 4, 16).movedim(-4, -2).reshape(*a, T // 16, D // 64, 1024)


def _v_tiles(x):
    *a, T, D = x.shape
    n = len(a)
    return x.reshape(*a, T // 16, 4, 4, D // 64, 16, 4).permute(*range(n), n, n + 3, n + 1, n + 4, n + 5, n + 2).reshape(*a, T // 16, D // 64, 1024)


def _store(s, x, side, plain, tiles):
    """Quantises x [rows][kv heads][hd] into the pages that the rows touch: the smallest power of two as a block's scale, never less than the page had."""
    case, page = s["case"], s["case"]["page"]
    seq, p = s["touched"][:, 0], s["touched"][:, 1]
    at = s["table"][seq, p]
    j = p[:, None] * page + torch.arange(page, device="cuda")
    new = (j >= s["before"][seq, None]) & (j < (s["before"] + s["new"])[seq, None])
    row = torch.where(new, s["row0"][seq, None] + j - s["before"][seq, None], 0)
    val = x[row].float().masked_fill(~new[:, :, None, None], 0).transpose(1, 2)  # [touched][kv heads][page][hd]
    m, e = torch.frexp(val.abs().amax(dim=(2, 3)))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -120).clamp(-120, 120)
    was = s["exps"][0, at, :, side].int()
    old = (p * page < s["before"][seq])[:, None]
    e = torch.where(old, torch.maximum(e, was), e)
    codes = s["codes"][0, at, :, side]
    kept = plain(codes).view(torch.float8_e4m3fn).float() * torch.exp2((was - e).clamp(min=-160).float())[:, :, None, None]
    val = torch.nn.functional.pad(torch.ldexp(val, -e[:, :, None, None]), (0, _hd64(case) - case["hd"]))
    done = torch.where(new[:, None, :, None], val, kept).to(torch.float8_e4m3fn).view(torch.uint8)
    first = (j < s["before"][seq, None])[:, None, :, None]
    done = torch.where(new[:, None, :, None] | first, done, plain(codes))
    s["codes"][0, at, :, side] = tiles(done)
    s["exps"][0, at, :, side] = e.to(torch.int8)


def _take(s):
    case = s["case"]
    q = _turned(case, s["q"], s["pos"], s["f"], s["wq"]).to(s["q"].dtype)
    _store(s, _turned(case, s["k"], s["pos"], s["f"], s["wk"]), 0, _k_plain, _k_tiles)
    _store(s, s["v"], 1, _v_plain, _v_tiles)
    return q


def _tokens(s, table):
    """Keys and values of the pages in `table` [n][pages]: fp32 [n][kv heads][tokens][hd]."""
    hd = s["case"]["hd"]
    c, e = s["codes"][0, table], s["exps"][0, table].float()
    got = []
    for side, plain in ((0, _k_plain), (1, _v_plain)):
        x = plain(c[:, :, :, side]).view(torch.float8_e4m3fn).float() * torch.exp2(e[..., side])[..., None, None]
        got.append(x.transpose(1, 2).reshape(table.shape[0], x.shape[2], -1, x.shape[-1])[..., :hd].contiguous())
    return got


def _attend(s):
    """The scores and values of the shared tokens once for a family's rows, of the others for each sequence; one softmax over both."""
    case, hd, T = s["case"], s["case"]["hd"], s["case"]["new"]
    H, Hk, n, F = case["heads"], case["kv_heads"], len(s["lens"]), case["families"]
    G = H // Hk
    q = s["q"].float().view(n, T, Hk, G, hd).permute(0, 2, 3, 1, 4).reshape(n, Hk, G * T, hd)
    per = -(-n // F)
    qf = torch.zeros((F, per, Hk, G * T, hd), device="cuda")
    qf[s["family"], s["place"]] = q
    qf = qf.transpose(1, 2).reshape(F, Hk, per * G * T, hd)
    ks, vs = _tokens(s, s["shared"])
    kr, vr = _tokens(s, s["rest"])
    S, R = ks.shape[2], kr.shape[2]
    ws = torch.matmul(qf, ks.transpose(2, 3).contiguous()).view(F, Hk, per, G * T, S).transpose(1, 2)[s["family"], s["place"]]
    wr = torch.matmul(q, kr.transpose(2, 3).contiguous())
    w = torch.cat((ws, wr), -1).mul_(1 / math.sqrt(hd)).view(n, Hk, G, T, S + R)
    i = (s["before"][:, None] + torch.arange(T, device="cuda"))[:, :, None]
    j = torch.cat((torch.arange(S, device="cuda").expand(n, S), s["whole"][:, None] + torch.arange(R, device="cuda")), 1)[:, None]
    seen = (j <= i) & ((torch.arange(S + R, device="cuda") >= S) | (j < s["whole"][:, None, None]))
    if case["window"]:
        seen = seen & ((i - j < case["window"]) | (j < case["sinks"]))
    w = w.masked_fill_(~seen[:, None, None], -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    total = w.sum(-1)
    w = w.view(n, Hk, G * T, S + R)
    wf = torch.zeros((F, per, Hk, G * T, S), device="cuda")
    wf[s["family"], s["place"]] = w[..., :S]
    os_ = torch.matmul(wf.transpose(1, 2).reshape(F, Hk, per * G * T, S), vs).view(F, Hk, per, G * T, hd).transpose(1, 2)[s["family"], s["place"]]
    o = (os_ + torch.matmul(w[..., S:].contiguous(), vr)).view(n, Hk, G, T, hd) / total[..., None]
    return o.permute(0, 3, 1, 2, 4).reshape(n * T, H, hd).to(s["q"].dtype)


# ------------------------------------------------------------------------------------------------------------------ run

def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _own(s):
    case, stream = s["case"], torch.cuda.current_stream().cuda_stream
    if case["op"] == "w4":
        y = torch.empty((case["rows"], case["n_out"]), dtype=DTYPES[case["y"]], device="cuda")
        s["w"].matvec(case["rows"], s["x"].data_ptr(), case["x"], y.data_ptr(), case["y"], stream=stream)
        return y
    q = s["q"]
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    if case["op"] == "prefix":
        s["kv"].attend_shared(0, q.data_ptr(), out.data_ptr(), case["dtype"], scale=1 / math.sqrt(case["hd"]), window=case["window"], sinks=case["sinks"], stream=stream)
        return out
    k = s["k"]
    if case["op"] == "rope":
        turned = torch.empty(k.shape, dtype=k.dtype, device="cuda")
        s["rope"].apply(case["rows"], q.data_ptr(), out.data_ptr(), case["heads"], case["dtype"], (q.stride(0), q.stride(1), out.stride(0), out.stride(1), k.stride(0), k.stride(1), turned.stride(0), turned.stride(1)),
                        k_ptr=k.data_ptr(), k_out_ptr=turned.data_ptr(), n_kv_heads=case["kv_heads"], positions_ptr=s["pos"].data_ptr(), q_weight_ptr=_ptr(s["wq"]), k_weight_ptr=_ptr(s["wk"]), eps=EPS,
                        stream=stream)
        return {"q": out, "k": turned}
    v = s["v"]
    s["rope"].append(s["kv"], 0, q.data_ptr(), out.data_ptr(), k.data_ptr(), v.data_ptr(), case["dtype"], (q.stride(0), q.stride(1), out.stride(0), out.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1)),
                     q_weight_ptr=_ptr(s["wq"]), k_weight_ptr=_ptr(s["wk"]), eps=EPS, stream=stream)
    return out


def run(s):
    case = s["case"]
    if own:
        got = _own(s)
    elif case["op"] == "rope":
        got = {x: _turned(case, s[x], s["pos"], s["f"], s["w" + x]).to(s[x].dtype) for x in ("q", "k")}
    else:
        got = {"w4": _w4, "take": _take, "prefix": _attend}[case["op"]](s)
    if case["op"] == "take":
        return {"q": got, "codes": s["codes"].view(torch.float8_e4m3fn), "exps": s["exps"]}
    return got


# ----------------------------------------------------------------------------------------------------------------- work

def work(case):
    if case["op"] == "w4":
        weights = case["n_out"] * (case["n_in"] / 2 + -(-case["n_in"] // case["group"]) * (DTYPES[case["scales"]].itemsize + case["zeros"]))
        return {"bytes": weights + case["rows"] * (case["n_in"] * DTYPES[case["x"]].itemsize + case["n_out"] * DTYPES[case["y"]].itemsize), "flops": 2 * case["rows"] * case["n_in"] * case["n_out"]}
    H, Hk, hd, size = case["heads"], case["kv_heads"], case["hd"], DTYPES[case["dtype"]].itemsize
    if case["op"] == "rope":
        return {"bytes": case["rows"] * (2 * (H + Hk) * hd * size + 4), "flops": 0}
    if case["op"] == "take":
        return {"bytes": sum(n for _, n in _lengths(case)) * hd * (2 * H * size + 2 * Hk * (size + 1)), "flops": 0}
    lens, page, new, pairs, tokens = _lengths(case), case["page"], case["new"], 0, 0
    lowest = {}
    for i, (p, t) in enumerate(lens):
        pos = np.arange(p + t, p + t + new)
        lo = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros(new, np.int64)
        pairs += int((pos + 1 - lo + np.minimum(lo, case["sinks"])).sum())
        whole, first = p // page * page, int(lo[0])
        f = i % case["families"]
        lowest[f] = (min(first, lowest.get(f, (first, 0))[0]), whole)
        tokens += p + t + new - max(whole, first)
    for first, whole in lowest.values():
        tokens += max(0, whole - first) + min(case["sinks"], first, whole)
    return {"bytes": 2 * len(lens) * new * H * hd * size + tokens * Hk * 2 * (hd + 1 / page), "flops": 4 * hd * H * pairs}


# ---------------------------------------------------------------------------------------------------------------- exact

def _byte_values():
    """The 256 values of e4m3 by its definition: sign, 4 bits of exponent with bias 7, 3 bits of fraction, subnormals, no infinity."""
    b = np.arange(256)
    x, f = (b >> 3) & 15, b & 7
    v = np.where(x == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (x - 10.0))
    return np.where((b & 127) == 127, np.nan, v) * np.where(b > 127, -1.0, 1.0)


def _place(hd64):
    """Byte offset within a 16-token group of (token, value), for K and for V."""
    t, d = np.arange(16)[:, None], np.arange(hd64)[None]
    u = d % 64
    return 1024 * (d // 64) + (u // 16 * 16 + t) * 16 + u % 16, 1024 * (d // 64) + (t // 4 * 16 + u // 4) * 16 + u % 4 * 4 + t % 4


def _turned_exact(case, x, pos, weight):
    """As complex numbers: pair i times amplitude * e^(i position f_i)."""
    x = x.double()
    if weight is not None:
        x = weight.double() * x / (x.pow(2).sum(-1, keepdim=True) / case["hd"] + EPS).sqrt()
    half, rot = case["rot"] // 2, case["rot"]
    f = []
    for i in range(half):
        turn = math.exp(-2 * i / rot * math.log(case["base"]))
        if case["scaling"] == "linear":
            turn /= case["factor"]
        elif case["scaling"] == "ntk":
            turn = math.exp(-2 * i / rot * (math.log(case["base"]) + rot / (rot - 2) * math.log(case["factor"])))
        elif case["scaling"] == "blend":
            made = case["context"] * turn / (2 * math.pi)
            if made < case["low"]:
                turn /= case["factor"]
            elif made < case["high"]:
                part = (made - case["low"]) / (case["high"] - case["low"])
                turn = turn / case["factor"] + part * (turn - turn / case["factor"])
        f.append(turn)
    first, second = (torch.arange(half) * 2, torch.arange(half) * 2 + 1) if case["layout"] == "interleaved" else (torch.arange(half), torch.arange(half) + half)
    angle = torch.outer(pos.double(), torch.tensor(f, dtype=torch.float64, device=pos.device))
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.full_like(angle, case["amplitude"]), angle)[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "w4":
        w = torch.empty((case["n_out"], case["n_in"]), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = s["codes"] % 16, s["codes"] // 16
        for g in range(0, case["n_in"], case["group"]):
            at, k = slice(g, g + case["group"]), g // case["group"]
            w[:, at] = s["scales"][:, k, None].double() * (w[:, at] - (8 if s["zeros"] is None else s["zeros"][:, k, None].double()))
        return s["x"].double() @ w.T
    if case["op"] == "rope":
        return {"q": _turned_exact(case, s["q"], s["pos"], s["wq"]), "k": _turned_exact(case, s["k"], s["pos"], s["wk"])}
    values, place = _byte_values(), _place(_hd64(case))
    page, hd, Hk = case["page"], case["hd"], case["kv_heads"]
    if case["op"] == "take":
        q, k = _turned_exact(case, s["q"], s["pos"], s["wq"]), _turned_exact(case, s["k"], s["pos"], s["wk"])
        codes = s["codes"].cpu().numpy().reshape(-1, Hk, 2, page * _hd64(case))
        exps = s["exps"].cpu().numpy().reshape(-1, Hk, 2)
        state = values[codes]
        row = 0
        for i, (b, n) in enumerate(s["lens"]):
            for side, x in ((0, k), (1, s["v"])):
                x = x[row:row + n].double().cpu().numpy()
                off = (np.arange(page // 16)[:, None, None] * 16 * _hd64(case) + place[side]).reshape(page, -1)[:, :hd]
                for p in range(b // page, -(-(b + n) // page)):
                    at, lo, hi = s["tables"][i][p], max(0, b - p * page), min(page, b + n - p * page)
                    for h in range(Hk):
                        got = x[p * page + lo - b:p * page + hi - b, h]
                        top = np.abs(got).max()
                        e = max(-120, math.ceil(math.log2(top / 448))) if top else -120
                        e = max(e, int(exps[at, h, side])) if lo else e
                        old = values[codes[at, h, side]][off[:lo]] * 2.0 ** int(exps[at, h, side])
                        all_ = np.concatenate([old, got]) / 2.0 ** e
                        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(all_), 2.0 ** -6))) - 3)
                        state[at, h, side][off[:hi]] = np.rint(all_ / step) * step
            row += n
        return {"q": q, "codes": torch.from_numpy(state.reshape(tuple(s["codes"].shape))), "exps": None}
    G, new, out = case["heads"] // Hk, case["new"], torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    values = torch.from_numpy(values).cuda()
    place = [torch.from_numpy((np.arange(page // 16)[:, None, None] * 16 * _hd64(case) + p).reshape(page, -1)[:, :hd].copy()).cuda() for p in place]
    for i, (p, t) in enumerate(s["lens"]):
        at, b = torch.tensor(s["tables"][i], device="cuda"), p + t
        k, v = ((values[s["codes"][0, at, :, side].reshape(len(at), Hk, -1)[:, :, place[side]].long()] * torch.exp2(s["exps"][0, at, :, side].double())[:, :, None, None])
                .transpose(0, 1).reshape(Hk, -1, hd)[:, :b + new] for side in (0, 1))
        j, pos = torch.arange(b + new, device="cuda"), torch.arange(b, b + new, device="cuda")[:, None]
        hidden = j > pos
        if case["window"]:
            hidden |= (j <= pos - case["window"]) & (j >= case["sinks"])
        q = s["q"][i * new:(i + 1) * new].double().reshape(new, Hk, G, hd).permute(1, 2, 0, 3).reshape(Hk, G * new, hd)
        a = torch.bmm(q, k.transpose(1, 2).contiguous()).view(Hk, G, new, -1) / math.sqrt(hd)
        o = torch.bmm(torch.softmax(a.masked_fill(hidden, -math.inf), -1).view(Hk, G * new, -1), v.contiguous())
        out[i * new:(i + 1) * new] = o.view(Hk, G, new, hd).permute(2, 0, 1, 3).reshape(new, -1, hd)
    return out
