"""Cases of the key/value cache held in 8 bits: writing it (quantized as it is written), reading it
back, and attention over it.

The cache is paged. A page holds `page` tokens of every key/value head: K codes are E4M3
[pages, kv_heads, page, dim], V codes E4M3 [pages, kv_heads, dim, page] (each page's tokens
contiguous along the last axis), and each (page, head) block has one power-of-two scale, a byte
e + 127, for K and one for V. A batch is cu_tokens [seqs + 1] (how the rows of q, k and v belong to
sequences), context [seqs] (each sequence's tokens in the cache, the batch's own included) and
table [seqs, width] (each sequence's pages in order): row i of a sequence with n rows sits at
position context - n + i.

`own` chooses between the plain torch form of each operator (elementary operations in 32 bits) and
the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one user's single token written: pure latency
        dict(name="append_one_token", op="append", dtype="bf16", seqs=1, tokens=1, context=517, ragged=False,
             kv_heads=8, dim=128, page=32, rule="ceil"),
        # a decode step of a full batch: a token each into partly filled pages
        dict(name="append_decode_step", op="append", dtype="bf16", seqs=128, tokens=1, context=1000, ragged=True,
             kv_heads=8, dim=128, page=32, rule="ceil"),
        # two prompts of a Llama-7B-shaped layer (32 heads of 128): all of K and V written once
        dict(name="append_prompts", op="append", dtype="bf16", seqs=2, tokens=4096, context=4096, ragged=False,
             kv_heads=32, dim=128, page=32, rule="ceil"),
        # chunks of uneven lengths in fp32 behind uneven contexts, small pages, a head size off the powers of two
        dict(name="append_chunks_f32", op="append", dtype="f32", seqs=5, tokens=333, context=1500, ragged=True,
             kv_heads=4, dim=80, page=16, rule="floor"),
        # the contexts of a batch taken out of the cache (to another engine, or to host memory)
        dict(name="read_contexts", op="read", dtype="bf16", seqs=8, tokens=4096, context=4096, ragged=True,
             kv_heads=8, dim=128, page=64),
        # the last tokens of a few sequences in fp32, large pages
        dict(name="read_tails_f32", op="read", dtype="f32", seqs=3, tokens=100, context=700, ragged=True,
             kv_heads=2, dim=64, page=128),
        # one user's single token, a short conversation: latency
        dict(name="decode_one_short", op="attend", dtype="bf16", seqs=1, tokens=1, context=600, ragged=False,
             q_heads=32, kv_heads=8, dim=128, page=32, causal=True, window=0),
        # a full batch of single tokens over uneven contexts: the serving step, bound by the cache's bytes
        dict(name="decode_batch", op="attend", dtype="bf16", seqs=64, tokens=1, context=8192, ragged=True,
             q_heads=32, kv_heads=8, dim=128, page=32, causal=True, window=0),
        # two very long documents, few rows: the keys have to be split over the chip
        dict(name="decode_long", op="attend", dtype="bf16", seqs=2, tokens=1, context=131071, ragged=False,
             q_heads=64, kv_heads=8, dim=128, page=64, causal=True, window=0),
        # drafted tokens checked in fp32, five a sequence, five query heads to a key head, wide heads
        dict(name="verify_drafts_f32", op="attend", dtype="f32", seqs=8, tokens=5, context=2000, ragged=True,
             q_heads=20, kv_heads=4, dim=256, page=16, causal=True, window=0),
        # a whole prompt of a Llama-7B-shaped layer: bound by the matrix products
        dict(name="prompt_causal", op="attend", dtype="bf16", seqs=1, tokens=4096, context=4096, ragged=False,
             q_heads=32, kv_heads=32, dim=128, page=32, causal=True, window=0),
        # chunks of prompts over a sliding window, grouped heads, uneven lengths
        dict(name="chunks_window", op="attend", dtype="bf16", seqs=4, tokens=512, context=6000, ragged=True,
             q_heads=32, kv_heads=4, dim=64, page=64, causal=True, window=1024),
    ]


def spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    c = dict(op=rng.choice(["append", "read", "attend", "attend"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
             seqs=spread(rng, 1, 128), tokens=1, context=spread(rng, 1, 32768), ragged=rng.random() < 0.7,
             kv_heads=rng.choice([1, 2, 4, 8, 16, 32]), dim=rng.choice([64, 80, 112, 128, 256]),
             page=rng.choice([16, 32, 64, 128]))
    if c["op"] == "attend":
        kind = rng.choice(["decode", "drafts", "chunk", "prompt"])
        n = {"decode": 1, "drafts": rng.randint(2, 8), "chunk": spread(rng, 9, 1024), "prompt": c["context"]}[kind]
        c.update(tokens=min(n, c["context"]), causal=rng.random() < 0.85, window=0)
        c["q_heads"] = c["kv_heads"] * rng.choice([1, 2, 4, 5, 7, 8] if c["kv_heads"] <= 8 else [1, 2])
        if rng.random() < 0.25:
            c["window"] = spread(rng, 16, 4096)
    else:
        c["tokens"] = rng.choice([1, min(spread(rng, 2, 1000), c["context"]), c["context"]])
        if c["op"] == "append":
            c["rule"] = rng.choice(["ceil", "floor"])
    while cost(c) > 1:  # smaller until it costs no more than the largest listed cases do
        if c["seqs"] > 1:
            c["seqs"] = (c["seqs"] + 1) // 2
        else:
            c["context"] = (c["context"] + 1) // 2
            c["tokens"] = min(c["tokens"], c["context"])
    return c


def cost(c):
    """The drawn case's work over the largest listed case's, each kind of work for itself (with the
    plain form's padded scores and keys, which take memory)."""
    kv = c["seqs"] * c["context"] * c["kv_heads"] * c["dim"]
    if c["op"] != "attend":
        return max(work(c)["bytes"] / 2e8, kv / 1.4e8)
    scores = c["seqs"] * c["q_heads"] * c["tokens"] * c["context"]
    return max(scores / 5.4e8, kv / 5.4e8, work(c)["flops"] / 1.37e11, 1.5 * scores * c["dim"] / 1.37e11 / 1.3)


def lengths(case):
    """Each sequence's (tokens, context): the case's own, or spread from a few to the case's largest."""
    got = []
    for i in range(case["seqs"]):
        n, ctx = case["tokens"], case["context"]
        if case["ragged"] and i:
            share = (i * 0.6180339887) % 1.0
            ctx = max(1, round(ctx * share))
            if case["tokens"] == case["context"]:
                n = ctx
            else:
                n = min(ctx, max(1, round(n * ((i * 0.7548776662) % 1.0))))
        got.append((n, ctx))
    return got


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    seqs, page, heads, dim = case["seqs"], case["page"], case["kv_heads"], case["dim"]
    dtype = DTYPES[case["dtype"]]
    lens = lengths(case)
    need = [-(-ctx // page) for _, ctx in lens]
    width, used = max(need), sum(need)
    pages = used + 3
    order = torch.randperm(pages, generator=g, device=DEV)[:used].to(torch.int32)
    table = torch.zeros(seqs, width, dtype=torch.int32, device=DEV)
    filled = torch.arange(width, device=DEV) < torch.tensor(need, device=DEV)[:, None]
    table[filled] = order
    cu = torch.tensor([0] + [n for n, _ in lens], device=DEV).cumsum(0).to(torch.int32)
    context = torch.tensor([ctx for _, ctx in lens], dtype=torch.int32, device=DEV)
    rows = sum(n for n, _ in lens)

    def drawn(*shape, channel):
        """Normal values, a few channels 8 times as large, as keys have them."""
        x = torch.randn(*shape, generator=g, device=DEV)
        size = torch.ones(shape[channel], device=DEV)
        size[torch.randperm(shape[channel], generator=g, device=DEV)[: max(1, shape[channel] // 100)]] = 8.0
        return x.mul_(size if channel == len(shape) - 1 else size[:, None])

    s = dict(case=case, cu=cu, context=context, table=table)
    for name, shape, channel in (("k", (pages, heads, page, dim), 3), ("v", (pages, heads, dim, page), 2)):
        x = drawn(*shape, channel=channel)
        # pages of uneven magnitudes, so that scales differ
        x.mul_(torch.exp(0.5 * torch.randn(pages, heads, 1, 1, generator=g, device=DEV)))
        e = exponent(x.abs().amax((2, 3)), True)
        x.mul_(power(-e)[:, :, None, None])
        s[name + "_codes"] = x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        s[name + "_scales"] = (e + 127).to(torch.uint8)
        del x
    if case["op"] == "append":
        s["k"] = drawn(rows, heads, dim, channel=2).to(dtype)
        s["v"] = drawn(rows, heads, dim, channel=2).mul_(0.5).to(dtype)
    elif case["op"] == "attend":
        s["q"] = torch.randn(rows, case["q_heads"], dim, generator=g, device=DEV).to(dtype)
    s["rows"] = rows
    s["most"] = max(n for n, _ in lens)
    s["longest"] = max(ctx for _, ctx in lens)
    if own:  # the handles that a serving program keeps from step to step
        from bit_gemm_fwht_amd import kv

        s["cache"] = kv.KVCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        s["batch"] = kv.Batch(cu, context, table, max_tokens=s["most"], max_context=s["longest"])
    return s


def run(state):
    return (run_own if own else run_plain)(state)


def run_own(s):
    from bit_gemm_fwht_amd import kv

    case = s["case"]
    if case["op"] == "append":
        kv.append(s["cache"], s["k"], s["v"], s["batch"],
                  scale_mode=kv.SCALE_E8M0_CEIL if case["rule"] == "ceil" else kv.SCALE_E8M0_FLOOR)
        return cache_values(s)
    if case["op"] == "read":
        k, v = kv.read(s["cache"], s["batch"], s["rows"], dtype=DTYPES[case["dtype"]])
        return {"k": k, "v": v}
    return kv.attention(s["q"], s["cache"], s["batch"], causal=case["causal"], window=case["window"])


def run_plain(s):
    op = s["case"]["op"]
    return plain_append(s) if op == "append" else plain_read(s) if op == "read" else plain_attention(s)


def cache_values(s):
    """The whole cache: its elements as the 8-bit floating values they stand for, and its scales."""
    return {"k": s["k_codes"].view(torch.float8_e4m3fn), "v": s["v_codes"].view(torch.float8_e4m3fn),
            "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def exponent(amax, ceil):
    """The block exponent e: floor(log2 amax) - 8, and with `ceil` one more where 448 2^e is below amax."""
    m, ex = torch.frexp(amax)
    e = ex - 9
    if ceil:
        e = e + (m > 0.875)
    return torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)


def places(s):
    """Of each row of the batch: its sequence, its position in it, its page and its place in the page."""
    page = s["case"]["page"]
    row = torch.arange(s["rows"], device=DEV)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = s["context"].long()[seq] - cu[seq + 1] + row
    return seq, pos, s["table"][seq, pos // page].long(), pos % page


def power(e):
    """2^e in fp32, exact (0 for e = -127, which stands for blocks of zeros)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def plain_append(s):
    case = s["case"]
    page, ceil = case["page"], case["rule"] == "ceil"
    seq, pos, pid, slot = places(s)
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    first = s["context"].long() - n  # where each sequence's new tokens begin
    begun = first % page  # tokens that its page already holds
    part = s["table"][torch.arange(case["seqs"], device=DEV), first // page].long()
    where = (pid, slot, part, begun, page, ceil)
    write(s["k"].float(), s["k_codes"], s["k_scales"], False, *where)
    write(s["v"].float(), s["v_codes"], s["v_scales"], True, *where)
    return cache_values(s)


def write(x, codes, scales, transposed, pid, slot, part, begun, page, ceil):
    amax = torch.zeros(codes.shape[:2], device=DEV)
    amax.index_reduce_(0, pid, x.abs().amax(2), "amax")
    new = exponent(amax, ceil)
    old = torch.full_like(new, -127)
    held = scales[part].to(torch.int32) - 127
    old[part] = torch.where((begun > 0)[:, None], held, -127)
    e = torch.maximum(new, old)
    # the tokens that were there, under the block's new scale
    c = codes[part].view(torch.float8_e4m3fn).float() * power((held - e[part]).clamp(min=-127))[:, :, None, None]
    there = torch.arange(page, device=DEV) < begun[:, None]
    there = there[:, None, None, :] if transposed else there[:, None, :, None]
    codes[part] = torch.where(there, c.to(torch.float8_e4m3fn).view(torch.uint8), codes[part])
    scales[pid] = (e + 127).to(torch.uint8)[pid]
    y = (x * power(-e[pid])[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    if transposed:
        codes[pid, :, :, slot] = y
    else:
        codes[pid, :, slot] = y


def plain_read(s):
    dtype = DTYPES[s["case"]["dtype"]]
    _, _, pid, slot = places(s)
    k = s["k_codes"][pid, :, slot].view(torch.float8_e4m3fn).float()
    v = s["v_codes"][pid, :, :, slot].view(torch.float8_e4m3fn).float()
    return {"k": (k * power(s["k_scales"][pid].to(torch.int32) - 127)[:, :, None]).to(dtype),
            "v": (v * power(s["v_scales"][pid].to(torch.int32) - 127)[:, :, None]).to(dtype)}


def plain_attention(s):
    case = s["case"]
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    group, seqs, most = case["q_heads"] // heads, case["seqs"], s["most"]
    table = s["table"].long()
    k = s["k_codes"][table].view(torch.float8_e4m3fn).float()  # [seqs, width, heads, page, dim]
    k.mul_(power(s["k_scales"][table].to(torch.int32) - 127)[..., None, None])
    k = k.permute(0, 2, 4, 1, 3).reshape(seqs, heads, dim, -1)
    seq, pos, _, _ = places(s)
    row = torch.arange(s["rows"], device=DEV) - s["cu"].long()[seq]
    q = torch.zeros(seqs, most, case["q_heads"], dim, device=DEV)
    q[seq, row] = s["q"].float() * (1.0 / math.sqrt(dim))
    q = q.view(seqs, most, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, heads, group * most, dim)
    p = (q @ k).view(seqs, heads, group, most, -1)
    del k
    at = torch.arange(p.shape[-1], device=DEV)
    n = (s["cu"][1:] - s["cu"][:-1]).long()
    own_pos = (s["context"].long() - n)[:, None] + torch.arange(most, device=DEV)
    allowed = (at < s["context"].long()[:, None, None])
    if case["causal"]:
        allowed = allowed & (at <= own_pos[..., None])
    if case["window"]:
        allowed = allowed & (at > own_pos[..., None] - case["window"])
    p.masked_fill_(~allowed[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["v_codes"][table].view(torch.float8_e4m3fn).float()  # [seqs, width, heads, dim, page]
    v.mul_(power(s["v_scales"][table].to(torch.int32) - 127)[..., None, None])
    v = v.permute(0, 2, 1, 4, 3).reshape(seqs, heads, -1, dim)
    o = (p.view(seqs, heads, group * most, -1) @ v).view(seqs, heads, group, most, dim)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, most, case["q_heads"], dim)
    return o[seq, row].to(s["q"].dtype)


def pairs(case, n, ctx):
    """(query, key) pairs of one sequence that the masks allow, and the keys that any query needs."""
    w = case["window"]
    got = sum((p + 1 if case["causal"] else ctx) - (max(0, p - w + 1) if w else 0) for p in range(ctx - n, ctx))
    return got, ctx - (max(0, ctx - n - w + 1) if w else 0)


def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    lens = lengths(case)
    rows = sum(n for n, _ in lens)
    if case["op"] != "attend":
        blocks = sum((ctx - 1) // page - (ctx - n) // page + 1 for n, ctx in lens)
        return {"bytes": 2 * heads * (rows * dim * (esz + 1) + blocks) + 4 * blocks + 8 * case["seqs"],
                "flops": 2 * rows * heads * dim}
    flops, total = 0, 2 * rows * case["q_heads"] * dim * esz
    for n, ctx in lens:
        got, keys = pairs(case, n, ctx)
        flops += 4 * got * case["q_heads"] * dim
        total += 2 * heads * keys * dim + -(-keys // page) * (2 * heads + 4) + 8
    return {"bytes": total, "flops": flops}


# ---- the definitions in 64 bits, a sequence and a page or head at a time ----

def e4m3(x):
    """The E4M3 value nearest to x (ties to the even one), at most 448."""
    step = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6.0) - 3.0
    unit = torch.exp2(step)
    return (torch.round(x / unit) * unit).clamp(-448.0, 448.0)


def block_exponent(amax, rule):
    if amax == 0:
        return -127
    e = math.frexp(amax)[1] - 9
    return min(127, max(-127, e + 1 if rule == "ceil" and 448.0 * 2.0 ** e < amax else e))


def exact(case, seed):
    s = prepare(case, seed)
    op, page, dim, heads = case["op"], case["page"], case["dim"], case["kv_heads"]
    table = s["table"].tolist()
    lens, cu = lengths(case), s["cu"].tolist()
    values = {}
    for name in ("k", "v"):
        values[name] = s[name + "_codes"].view(torch.float8_e4m3fn)
        values[name + "_scales"] = s[name + "_scales"].long()
    if op == "append":
        for name in ("k", "v"):
            held, scales = values[name].double(), values[name + "_scales"].cpu()
            for i, (n, ctx) in enumerate(lens):
                x = s[name][cu[i]: cu[i + 1]].double()
                for j in range((ctx - n) // page, (ctx - 1) // page + 1):
                    lo, hi = max(j * page, ctx - n), min((j + 1) * page, ctx)
                    new = x[lo - (ctx - n): hi - (ctx - n)]  # [tokens, heads, dim]
                    amax, pid = new.abs().amax((0, 2)).tolist(), table[i][j]
                    es = [block_exponent(a, case["rule"]) for a in amax]
                    old = [int(v) - 127 for v in scales[pid]]
                    if lo > j * page:
                        es = [max(a, b) for a, b in zip(es, old)]
                        grow = torch.tensor([2.0 ** (b - a) for a, b in zip(es, old)], dtype=torch.float64, device=DEV)
                        t = lo - j * page
                        if name == "k":
                            held[pid, :, :t] = e4m3(held[pid, :, :t] * grow[:, None, None])
                        else:
                            held[pid, :, :, :t] = e4m3(held[pid, :, :, :t] * grow[:, None, None])
                    d = torch.tensor([2.0 ** -a for a in es], dtype=torch.float64, device=DEV)
                    y = e4m3(new * d[:, None])
                    if name == "k":
                        held[pid, :, lo - j * page: hi - j * page] = y.permute(1, 0, 2)
                    else:
                        held[pid, :, :, lo - j * page: hi - j * page] = y.permute(1, 2, 0)
                    scales[pid] = torch.tensor([a + 127 for a in es])
            values[name], values[name + "_scales"] = held, None
        return {k: values[k] for k in ("k", "v", "k_scales", "v_scales")}
    factor = {n: torch.exp2(values[n + "_scales"].double() - 127.0) for n in ("k", "v")}
    out = {"k": [], "v": []}
    o = torch.zeros(s["rows"], case.get("q_heads", 0), dim, dtype=torch.float64, device=DEV)
    for i, (n, ctx) in enumerate(lens):
        ids = torch.tensor(table[i][: -(-ctx // page)], device=DEV)
        k = s["k_codes"][ids].view(torch.float8_e4m3fn).double() * factor["k"][ids][:, :, None, None]
        v = s["v_codes"][ids].view(torch.float8_e4m3fn).double() * factor["v"][ids][:, :, None, None]
        k = k.permute(1, 0, 2, 3).reshape(heads, -1, dim)[:, :ctx]
        v = v.permute(1, 0, 3, 2).reshape(heads, -1, dim)[:, :ctx]
        if op == "read":
            out["k"].append(k[:, ctx - n:].permute(1, 0, 2))
            out["v"].append(v[:, ctx - n:].permute(1, 0, 2))
            continue
        p = torch.arange(ctx - n, ctx, device=DEV)[:, None]
        at = torch.arange(ctx, device=DEV)[None]
        gone = torch.zeros(n, ctx, dtype=torch.bool, device=DEV)
        if case["causal"]:
            gone |= at > p
        if case["window"]:
            gone |= at <= p - case["window"]
        for h in range(case["q_heads"]):
            kv_head = h // (case["q_heads"] // heads)
            x = s["q"][cu[i]: cu[i + 1], h].double() @ k[kv_head].T / math.sqrt(dim)
            o[cu[i]: cu[i + 1], h] = torch.softmax(x.masked_fill(gone, -math.inf), -1) @ v[kv_head]
    return o if op == "attend" else {n: torch.cat(out[n]) for n in ("k", "v")}
