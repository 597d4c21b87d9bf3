"""The operators of the 8-bit key/value cache, as cases to be measured: appending tokens (quantised), attention over the
cache, attention with a sliding window and visible first tokens, and the copying, forking and compacting of pages.

Each operator has a plain form here (elementary torch operations in 32 bits) and the framework's own call (`own`).

The cache. `codes` is uint8 [layers][pages][kv heads][2][page_tokens / 16][hd64 / 64][1024] (index 0 of the fourth axis: K,
1: V; hd64 is the head dimension rounded up to a multiple of 64; positions past the head dimension are zero), each byte an
e4m3 value; `exps` is int8 [layers][pages][kv heads][2]; a stored value is code * 2^exp. The 1024 bytes hold 16 tokens x 64
values: for K, byte (16 g + t) * 16 + b is token t, value 16 g + b; for V, byte (16 g + r) * 16 + 4 i + t is token 4 g + t,
value 4 r + i. A sequence is a list of pages; its token j is in page j // page_tokens, place j % page_tokens.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # One decode token's keys and values of one layer: 32 heads of 128 (d_model 4096), a call bound by its latency.
        dict(name="append_token", op="append", seqs=1, heads=32, kv_heads=32, hd=128, page=64, new=1, before=701, lens_seed=1, dtype="bf16", fused=False),
        # A prompt taken up in one call, from the fused projection's output, behind a short system prompt that ends inside a page.
        dict(name="append_prompt", op="append", seqs=1, heads=32, kv_heads=32, hd=128, page=64, new=4097, before=37, lens_seed=2, dtype="bf16", fused=True),
        # A few requests' prompts together, in the framework's own fp32 activations, 40 heads of 128 (d_model 5120), small pages.
        dict(name="append_ragged", op="append", seqs=5, heads=40, kv_heads=40, hd=128, page=16, new=700, before=999, lens_seed=3, dtype="f32", fused=False),
        # The smallest model (d_model 256: 4 heads of 64), one token: latency.
        dict(name="attend_tiny", op="attend", seqs=1, heads=4, kv_heads=4, hd=64, page=16, new=1, before=300, lens_seed=4, dtype="f32", fused=False, window=0, sinks=0),
        # One decode token at batch 1, 32 heads of 128, a cache of 4 Ki tokens: the attention next to the sparse FFN's decode step.
        dict(name="attend_token", op="attend", seqs=1, heads=32, kv_heads=32, hd=128, page=64, new=1, before=4094, lens_seed=5, dtype="bf16", fused=True, window=0, sinks=0),
        # Many sequences of uneven lengths up to 32 Ki, grouped heads (32 over 8): a serving step bound by memory.
        dict(name="attend_batch", op="attend", seqs=24, heads=32, kv_heads=8, hd=128, page=32, new=1, before=32767, lens_seed=6, dtype="bf16", fused=False, window=0, sinks=0),
        # A few drafted tokens checked at once for several sequences (40 heads of 128), fp16.
        dict(name="attend_drafts", op="attend", seqs=4, heads=40, kv_heads=40, hd=128, page=64, new=5, before=2500, lens_seed=7, dtype="f16", fused=False, window=0, sinks=0),
        # A prompt's own attention: 4 Ki tokens, 32 heads of 128, bound by the matrix units.
        dict(name="attend_prompt", op="attend", seqs=1, heads=32, kv_heads=32, hd=128, page=64, new=4096, before=0, lens_seed=8, dtype="bf16", fused=True, window=0, sinks=0),
        # Long conversations of a model with a window of 4096 and four first tokens kept: only the window is read.
        dict(name="window_token", op="attend", seqs=8, heads=32, kv_heads=8, hd=128, page=64, new=1, before=60001, lens_seed=9, dtype="bf16", fused=False, window=4096, sinks=4),
        # A long prompt of the same model, fp16.
        dict(name="window_prompt", op="attend", seqs=1, heads=32, kv_heads=8, hd=128, page=32, new=8191, before=0, lens_seed=10, dtype="f16", fused=False, window=4096, sinks=4),
        # A prompt of 1,001 tokens continued in seven ways: the shared last page is copied for all 31 layers.
        dict(name="pages_fork", op="fork", layers=31, seqs=7, kv_heads=32, hd=128, page=64, before=1001),
        # A cache whose pages lie scattered after requests came and went, packed to the front of the pool.
        dict(name="pages_compact", op="compact", layers=8, seqs=6, kv_heads=8, hd=128, page=32, pool=512, live=200, lens_seed=11),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    hd = rng.choice([64, 128, 128, 80, 96, 40, 256])
    page = rng.choice([16, 32, 64, 128])
    kv = _log(rng, 1, 40)
    dtype = rng.choice(["bf16", "f16", "f32"])
    op = rng.choice(["append", "token", "drafts", "prompt", "window_token", "window_prompt", "fork", "compact"])
    if op == "fork":
        case = dict(op=op, layers=_log(rng, 1, 32), seqs=_log(rng, 1, 8), kv_heads=kv, hd=hd, page=page, before=page * _log(rng, 1, 8) + rng.randint(1, page - 1))
        case["layers"] = max(1, min(case["layers"], 130_000_000 // (_page_bytes(case) * (1 + case["seqs"]))))
        return case
    if op == "compact":
        pool = _log(rng, 24, 512)
        case = dict(op=op, layers=_log(rng, 1, 8), seqs=_log(rng, 1, 8), kv_heads=min(kv, 16), hd=hd, page=min(page, 64), pool=pool, live=rng.randint(9, max(9, pool // 2)), lens_seed=rng.randint(0, 1 << 30))
        case["layers"] = max(1, min(case["layers"], 60_000_000 // (_page_bytes(case) * case["live"])))
        return case
    group = rng.choice([1, 1, 2, 4, 7, 8])
    while group * kv > 64:
        kv = (kv + 1) // 2
    case = dict(op="append" if op == "append" else "attend", seqs=1, heads=group * kv, kv_heads=kv, hd=hd, page=page, lens_seed=rng.randint(0, 1 << 30), dtype=dtype, fused=rng.random() < 0.5)
    if op == "append":
        case.update(seqs=_log(rng, 1, 16), new=_log(rng, 1, 1024), before=_log(rng, 1, 2000))
        return case
    case.update(window=0, sinks=0)
    if op in ("token", "drafts"):
        case.update(seqs=_log(rng, 1, 32), new=1 if op == "token" else rng.randint(2, 24), before=_log(rng, 1, 16000))
        if case["seqs"] * case["before"] * case["kv_heads"] > 4_000_000:
            case["before"] = 4_000_000 // (case["seqs"] * case["kv_heads"])
    elif op == "prompt":
        case.update(seqs=rng.choice([1, 1, 2, 3]), new=_log(rng, 33, 2600), before=rng.choice([0, 0, 1, 100, 900]))
    else:
        case.update(window=_log(rng, 1, 5000), sinks=rng.choice([0, 1, 4, 16]))
        if op == "window_token":
            case.update(seqs=_log(rng, 1, 16), new=1, before=_log(rng, 10, 30000))
        else:
            case.update(new=_log(rng, 33, 5000), before=rng.choice([0, 0, 333]))
    if case["new"] * (case["new"] + case["before"]) * case["seqs"] * case["heads"] > 400_000_000:
        case["new"] = max(1, int(math.sqrt(400_000_000 / (case["seqs"] * case["heads"]))) - case["before"])
    return case


def _lengths(case):
    """Per sequence (tokens before the call, new tokens): the first takes the case's own figures, the others spread below them."""
    rng = random.Random(case["lens_seed"])
    got = [(case["before"], case["new"])]
    for _ in range(case["seqs"] - 1):
        got.append((rng.randint(case["before"] // 8, case["before"]), rng.randint(max(1, case["new"] // 3), case["new"])))
    return got


def _hd64(case):
    return -(-case["hd"] // 64) * 64


def _page_bytes(case):
    return case["kv_heads"] * 2 * case["page"] * _hd64(case)


# --------------------------------------------------------------------------------------------------------------- inputs

def _pool(case, layers, pages, gen):
    """Codes spread as a quantised block's are (its largest near 448 * 0.5..1), and exponents of values of about 0.4 to 3."""
    shape = (layers, pages, case["kv_heads"], 2, case["page"] // 16, _hd64(case) // 64, 1024)
    codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for layer in range(layers):
        codes[layer] = (torch.randn(shape[1:], device="cuda", generator=gen) * 96).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    dead = torch.arange(_hd64(case), device="cuda") >= case["hd"]
    if case["hd"] != _hd64(case):
        slabs = dead.view(-1, 64)
        k = slabs.view(-1, 4, 1, 16).expand(-1, 4, 16, 16).reshape(-1, 1024)
        v = slabs.view(-1, 1, 16, 4, 1).expand(-1, 4, 16, 4, 4).reshape(-1, 1024)
        codes[:, :, :, 0].masked_fill_(k, 0)
        codes[:, :, :, 1].masked_fill_(v, 0)
    exps = torch.randint(-8, -5, (layers, pages, case["kv_heads"], 2), device="cuda", generator=gen).to(torch.int8)
    return codes, exps


def _rows(case, rows, gen):
    """q, k, v [rows][heads][hd]: tensors of their own, or views of one fused projection output."""
    H, Hk, hd, t = case["heads"], case["kv_heads"], case["hd"], DTYPES[case["dtype"]]
    if case["fused"]:
        both = torch.randn((rows, H + 2 * Hk, hd), device="cuda", generator=gen).to(t)
        return both[:, :H], both[:, H:H + Hk], both[:, H + Hk:]
    return tuple(torch.randn((rows, n, hd), device="cuda", generator=gen).to(t) for n in (H, Hk, Hk))


def _handle(case, s, layers, pages, seqs, per_seq):
    from delta_prefetched_ffn_amd import KVCache
    return KVCache(n_layers=layers, n_heads=case.get("heads", case["kv_heads"]), n_kv_heads=case["kv_heads"], head_dim=case["hd"], page_tokens=case["page"], n_pages=pages,
                   max_seqs=seqs, max_pages=per_seq, codes=s["codes"].data_ptr(), exps=s["exps"].data_ptr(), keepalive=(s["codes"], s["exps"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = random.Random(seed)
    page = case["page"]
    s = {"case": case}
    if case["op"] == "fork":
        held = -(-case["before"] // page)
        pages = held + 2 * case["seqs"] + 1
        s["codes"], s["exps"] = _pool(case, case["layers"], pages, gen)
        s["table"] = host.sample(range(pages), held)
        if own:
            s["kv"] = _handle(case, s, case["layers"], pages, case["seqs"] + 1, held + 1)
            s["kv"].adopt(0, s["table"], case["before"])
        return s
    if case["op"] == "compact":
        s["codes"], s["exps"] = _pool(case, case["layers"], case["pool"], gen)
        live = host.sample(range(case["pool"]), case["live"])
        n = min(case["seqs"], case["live"])
        s["tables"] = [live[i * len(live) // n:(i + 1) * len(live) // n] for i in range(n)]
        if own:
            s["kv"] = _handle(case, s, case["layers"], case["pool"], n, max(map(len, s["tables"])))
        return s
    lens = _lengths(case)
    held = [-(-(b + n) // page) for b, n in lens]
    pages = sum(held) + 3
    s["codes"], s["exps"] = _pool(case, 1, pages, gen)
    order = host.sample(range(pages), sum(held))
    s["lens"], s["tables"] = lens, [order[sum(held[:i]):sum(held[:i + 1])] for i in range(len(lens))]
    s["q"], s["k"], s["v"] = _rows(case, sum(n for _, n in lens), gen)
    # The plain form's plan: the page table, and where each sequence's rows lie.
    table = np.zeros((len(lens), max(held)), np.int64)
    for i, t in enumerate(s["tables"]):
        table[i, :len(t)] = t
    s["table"] = torch.from_numpy(table).cuda()
    s["before"] = torch.tensor([b for b, _ in lens], device="cuda")
    s["new"] = torch.tensor([n for _, n in lens], device="cuda")
    s["row0"] = s["new"].cumsum(0) - s["new"]
    s["most"] = max(n for _, n in lens)
    if case["op"] == "append":
        s["touched"] = torch.tensor([(i, p) for i, (b, n) in enumerate(lens) for p in range(b // page, held[i])], device="cuda")
    if own:
        s["kv"] = _handle(case, s, 1, pages, len(lens), max(held))
        for i, (b, _) in enumerate(lens):
            s["kv"].adopt(i, s["tables"][i], b)
        s["kv"].extend(list(range(len(lens))), [n for _, n in lens])
    return s


# ----------------------------------------------------------------------------------------------------------- plain forms

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


def _append_one(s, x, side, plain, tiles):
    case, page = s["case"], s["case"]["page"]
    seq, p = s["touched"][:, 0], s["touched"][:, 1]
    at = s["table"][seq, p]
    # The row that fills each place of each touched page, where one does.
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


def _attend(s):
    case, page, hd = s["case"], s["case"]["page"], s["case"]["hd"]
    H, Hk, n, T = case["heads"], case["kv_heads"], len(s["lens"]), s["most"]
    P = s["table"].shape[1]
    c, e = s["codes"][0, s["table"]], s["exps"][0, s["table"]].float()  # [n][P][Hk][2]...
    k = (_k_plain(c[:, :, :, 0]).view(torch.float8_e4m3fn).float() * torch.exp2(e[..., 0])[..., None, None]).transpose(1, 2).reshape(n, Hk, P * page, -1)[..., :hd]
    v = (_v_plain(c[:, :, :, 1]).view(torch.float8_e4m3fn).float() * torch.exp2(e[..., 1])[..., None, None]).transpose(1, 2).reshape(n, Hk, P * page, -1)[..., :hd]
    t = torch.arange(T, device="cuda")
    real = t < s["new"][:, None]
    row = torch.where(real, s["row0"][:, None] + t, 0)
    q = s["q"][row].float().reshape(n, T, Hk, H // Hk, hd).permute(0, 2, 3, 1, 4).reshape(n, Hk, H // Hk * T, hd)
    w = (torch.matmul(q, k.transpose(2, 3).contiguous()) * (1 / math.sqrt(hd))).view(n, Hk, H // Hk, T, P * page)
    i, j = (s["before"][:, None] + t)[:, :, None], torch.arange(P * page, device="cuda")
    seen = j <= i
    if case["window"]:
        seen = seen & ((i - j < case["window"]) | (j < case["sinks"]))
    w = w.masked_fill_(~seen[:, None, None], -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    total = w.sum(-1)
    o = torch.matmul(w.view(n, Hk, -1, P * page), v.contiguous()).view(n, Hk, H // Hk, T, hd) / total[..., None]
    return o.permute(0, 3, 1, 2, 4).reshape(n, T, H, hd)[real].to(s["q"].dtype)


def _fork(s):
    case = s["case"]
    tail = s["table"][-1]
    free = sorted(set(range(s["codes"].shape[1])) - set(s["table"]))[:case["seqs"]]
    s["codes"][:, free] = s["codes"][:, tail].unsqueeze(1)
    s["exps"][:, free] = s["exps"][:, tail].unsqueeze(1)
    return np.array([s["table"][:-1] + [f] for f in free], np.int32)


def _compact(s):
    live = np.concatenate([np.array(t, np.int64) for t in s["tables"]])
    to = np.arange(s["codes"].shape[1])
    holes = np.setdiff1d(np.arange(live.size), live)
    high = np.sort(live[live >= live.size])
    to[high] = holes
    s["codes"][:, torch.from_numpy(holes).cuda()] = s["codes"][:, torch.from_numpy(high).cuda()]
    s["exps"][:, torch.from_numpy(holes).cuda()] = s["exps"][:, torch.from_numpy(high).cuda()]
    return to[live].astype(np.int32)


# ------------------------------------------------------------------------------------------------------------------ run

def _own(s):
    case, stream = s["case"], torch.cuda.current_stream().cuda_stream
    kv = s["kv"]
    if case["op"] == "append":
        k, v = s["k"], s["v"]
        kv.append(0, k.data_ptr(), v.data_ptr(), case["dtype"], (k.stride(0), k.stride(1), v.stride(0), v.stride(1)), stream)
    elif case["op"] == "attend":
        q = s["q"]
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        kv.attend(0, q.data_ptr(), out.data_ptr(), case["dtype"], (q.stride(0), q.stride(1), out.stride(0), out.stride(1)),
                  scale=1 / math.sqrt(case["hd"]), window=case["window"], sinks=case["sinks"], stream=stream)
        return out
    elif case["op"] == "fork":
        forks = list(range(1, case["seqs"] + 1))
        for f in forks:
            kv.fork(0, f, case["before"], stream=stream)
        kv.extend(forks, [1] * len(forks), stream)
        tables = np.stack([kv.pages(f) for f in forks])
        for f in forks:
            kv.free(f)
        return tables
    else:
        kv.reset()
        for i, t in enumerate(s["tables"]):
            kv.adopt(i, t, len(t) * case["page"], stream)
        kv.compact(stream)
        return np.concatenate([kv.pages(i) for i in range(len(s["tables"]))])


def run(s):
    op = s["case"]["op"]
    if own:
        got = _own(s)
    elif op == "append":
        got = _append_one(s, s["k"], 0, _k_plain, _k_tiles)
        got = _append_one(s, s["v"], 1, _v_plain, _v_tiles)
    else:
        got = {"attend": _attend, "fork": _fork, "compact": _compact}[op](s)
    if op == "attend":
        return got
    state = {"codes": s["codes"].view(torch.float8_e4m3fn), "exps": s["exps"]}
    return state if op == "append" else {**state, "pages": got}


# ----------------------------------------------------------------------------------------------------------------- work

def _seen(case):
    """Per sequence (tokens that some row sees, (row, token) pairs)."""
    got = []
    for b, n in _lengths(case):
        i = np.arange(b, b + n, dtype=np.int64)
        if not case["window"]:
            got.append((b + n, int((i + 1).sum())))
            continue
        lo = np.maximum(0, i - case["window"] + 1)
        got.append((b + n - int(lo[0]) + min(case["sinks"], int(lo[0])), int((i + 1 - lo + np.minimum(lo, case["sinks"])).sum())))
    return got


def work(case):
    Hk, hd, page = case["kv_heads"], case["hd"], case["page"]
    if case["op"] == "fork":
        one = case["layers"] * (_page_bytes(case) + 2 * Hk)
        return {"bytes": one * (1 + case["seqs"]), "flops": 0}
    if case["op"] == "compact":
        # On average the share of live pages that lies past the packed length moves.
        moved = case["live"] * (1 - case["live"] / case["pool"])
        return {"bytes": 2 * moved * case["layers"] * (_page_bytes(case) + 2 * Hk), "flops": 0}
    size = DTYPES[case["dtype"]].itemsize
    rows = sum(n for _, n in _lengths(case))
    if case["op"] == "append":
        return {"bytes": rows * Hk * hd * 2 * (size + 1), "flops": 0}
    seen = _seen(case)
    return {"bytes": 2 * rows * case["heads"] * hd * size + sum(t for t, _ in seen) * Hk * 2 * (hd + 1 / page),
            "flops": 4 * hd * case["heads"] * sum(p for _, p in seen)}


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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fork", "compact"):
        return None
    values, place = _byte_values(), _place(_hd64(case))
    page, hd, Hk = case["page"], case["hd"], case["kv_heads"]
    if case["op"] == "append":
        codes = s["codes"].cpu().numpy().reshape(-1, Hk, 2, page * _hd64(case))
        exps = s["exps"].cpu().numpy().reshape(-1, Hk, 2)
        state = values[codes]
        row = 0
        for i, (b, n) in enumerate(s["lens"]):
            for side, x in ((0, s["k"]), (1, s["v"])):
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
        return {"codes": torch.from_numpy(state.reshape(tuple(s["codes"].shape))), "exps": None}
    G, out, row = case["heads"] // Hk, torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    values = torch.from_numpy(values).cuda()
    place = [torch.from_numpy((np.arange(page // 16)[:, None, None] * 16 * _hd64(case) + p).reshape(page, -1)[:, :hd].copy()).cuda() for p in place]
    for i, (b, n) in enumerate(s["lens"]):
        at = torch.tensor(s["tables"][i], device="cuda")
        for h in range(Hk):
            k, v = ((values[s["codes"][0, at, h, side].reshape(len(at), -1)[:, place[side]].long()] * torch.exp2(s["exps"][0, at, h, side].double())[:, None, None]).reshape(-1, hd)[:b + n]
                    for side in (0, 1))
            j = torch.arange(b + n, device="cuda")
            pos = torch.arange(b, b + n, device="cuda")[:, None]
            hidden = j > pos
            if case["window"]:
                hidden |= (j <= pos - case["window"]) & (j >= case["sinks"])
            for g in range(h * G, (h + 1) * G):
                a = (s["q"][row:row + n, g].double() @ k.T / math.sqrt(hd)).masked_fill(hidden, -math.inf)
                out[row:row + n, g] = torch.softmax(a, -1) @ v
        row += n
    return out
