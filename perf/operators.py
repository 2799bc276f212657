"""The paged-cache operators as a serving program calls them, beside their plain forms.

Three operators: the page plan of a step (block table, slot map, positions and
free list from request lengths), the write of new keys and values into a paged
cache, and the attention of new tokens over that cache. Lengths are a function
of the case alone; values, page order and cache contents come from the seed.
"""
import math

import torch

own = False

# Heads, widths and page sizes: 10 heads of 256 is a width of 2560, 16 heads of
# 128 the delta rule's 2048; the others are generic.
LISTED = [
    # one decode step of 64 running requests: one new token each, a page now and then
    dict(name="plan_decode_64", op="plan", n=64, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=8192, page=16, rollback=0, pad=0),
    # a step of 1024 requests: prompt chunks, rolled-back drafts (pages go back), a padded batch
    dict(name="plan_chunks_1024", op="plan", n=1024, new_lo=1, new_hi=128, ctx_lo=0, ctx_hi=4096, page=32, rollback=40,
         pad=777),
    # the keys and values of one decode step
    dict(name="write_decode_64", op="write", n=64, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=2048, page=16, kv_heads=8, dim=128,
         dtype="bf16", pad=0),
    # the keys and values of a step of prompt chunks, rows of a fused projection's output
    dict(name="write_chunks_16k", op="write", n=9, new_lo=1500, new_hi=2100, ctx_lo=0, ctx_hi=4000, page=64, kv_heads=8,
         dim=128, dtype="bf16", pad=100),
    # decode, four short requests, a local attention layer (the smallest call: latency)
    dict(name="decode_4_local", op="attn", n=4, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=700, page=16, q_heads=10, kv_heads=1,
         dim=256, window=2048, dtype="bf16", pad=0),
    # decode, 64 running requests of mixed age
    dict(name="decode_64", op="attn", n=64, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=8191, page=16, q_heads=32, kv_heads=8,
         dim=128, window=0, dtype="bf16", pad=0),
    # decode, two very long contexts: few rows, a long axis
    dict(name="decode_2_long", op="attn", n=2, new_lo=1, new_hi=1, ctx_lo=100000, ctx_hi=131000, page=64, q_heads=16,
         kv_heads=2, dim=128, window=0, dtype="bf16", pad=0),
    # verification of drafts: a few tokens of each request, one key head per query head
    dict(name="drafts_32", op="attn", n=32, new_lo=2, new_hi=6, ctx_lo=10, ctx_hi=4096, page=32, q_heads=16, kv_heads=16,
         dim=64, window=0, dtype="bf16", pad=5),
    # one long prompt, a later chunk of it
    dict(name="chunk_long", op="attn", n=1, new_lo=2048, new_hi=2048, ctx_lo=30011, ctx_hi=30011, page=128, q_heads=32,
         kv_heads=8, dim=128, window=0, dtype="bf16", pad=0),
    # whole prompts through a local attention layer, B=8 L=4096 W=2560
    dict(name="prompt_local", op="attn", n=8, new_lo=4096, new_hi=4096, ctx_lo=0, ctx_hi=0, page=64, q_heads=10, kv_heads=1,
         dim=256, window=2048, dtype="bf16", pad=0),
    # a continuous batch: one prompt chunk among running requests
    dict(name="mixed_48", op="attn", n=48, new_lo=1, new_hi=1, first_new=1000, ctx_lo=3, ctx_hi=4000, page=16, q_heads=16,
         kv_heads=4, dim=128, window=0, dtype="bf16", pad=24),
    # ragged chunks in float32
    dict(name="chunks_f32", op="attn", n=5, new_lo=37, new_hi=333, ctx_lo=0, ctx_hi=900, page=16, q_heads=8, kv_heads=4,
         dim=64, window=0, dtype="f32", pad=7),
]


def listed():
    return [dict(c) for c in LISTED]


def _spread(lo, hi, n, phase):
    """n whole numbers over [lo, hi], unordered: a fixed low-discrepancy sequence."""
    return [lo + int((hi - lo + 1) * math.modf(phase + 0.6180339887498949 * i)[0]) for i in range(n)]


def lengths(case):
    """(tokens in the cache before the step, new tokens) of every sequence."""
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["n"], 0.5)
    new = _spread(case["new_lo"], case["new_hi"], case["n"], 0.25)
    if "first_new" in case:
        new[0] = case["first_new"]
    return ctx, new


def _visible(ctx, new, window):
    """(pairs of a query and a key it sees, keys that some query sees) of one sequence."""
    if new == 0:
        return 0, 0
    first, last = ctx + 1, ctx + new   # keys seen by the first and the last query, without a window
    if not window or last <= window:
        return (first + last) * new // 2, last
    if first >= window:
        return new * window, min(last, window + new - 1)
    grow = window - first
    return (first + window - 1) * grow // 2 + (new - grow) * window, last


def work(case):
    ctx, new = lengths(case)
    tokens = sum(new)
    if case["op"] == "plan":
        rows = tokens + case["pad"]
        # lengths in and out, the slot map and positions, a table entry read or written for every page that new tokens touch
        pages = sum((c + m - 1) // case["page"] - c // case["page"] + 1 for c, m in zip(ctx, new) if m)
        return {"bytes": 4 * (4 * case["n"] + 2 * rows + 2 * pages), "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "write":
        return {"bytes": 4 * tokens * case["kv_heads"] * case["dim"] * e + 4 * (tokens + case["pad"]), "flops": 0}
    seen = [_visible(c, m, case["window"]) for c, m in zip(ctx, new)]
    d, hq, hk = case["dim"], case["q_heads"], case["kv_heads"]
    moved = 2 * tokens * hq * d * e + 4 * tokens * hq + 2 * hk * d * e * sum(k for _, k in seen)
    return {"bytes": moved + 4 * sum(-(-k // case["page"]) for _, k in seen), "flops": 4 * d * hq * sum(p for p, _ in seen)}


def _padded(case):
    """Elements of the plain form's padded scores and of its gathered keys."""
    ctx, new = lengths(case)
    total = max(c + m for c, m in zip(ctx, new))
    return case["n"] * case["q_heads"] * max(new) * total, case["n"] * case["kv_heads"] * total * case["dim"]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "attn", "attn", "attn", "attn"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    pad = rng.choice([0, 1, rng.randrange(2, 200)])
    if op == "plan":
        hi = _log(rng, 1, 256)
        n = _log(rng, 1, 1024 if hi <= 128 else 256)
        c = dict(op=op, n=n, new_lo=rng.randrange(0, hi) + (n == 1), new_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 1, 8192),
                 page=page, rollback=rng.choice([0, rng.randrange(1, 90)]), pad=pad)
        while work(c)["bytes"] > work(LISTED[1])["bytes"]:
            c["n"] = c["n"] * 3 // 4
        return c
    if op == "write":
        hi = _log(rng, 1, 1024)
        n = max(1, min(_log(rng, 1, 64), 16000 * 1024 // (hi * kv_heads * dim * (2 if dtype == "f32" else 1))))
        return dict(op=op, n=n, new_lo=rng.randrange(0, hi) + (n == 1), new_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 1, 4096),
                    page=page, kv_heads=kv_heads, dim=dim, dtype=dtype, pad=pad)
    group = rng.choice([1, 2, 4, 5, 8, 10, 16])
    hi = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 2, 2048), _log(rng, 2, 2048)])
    c = dict(op=op, n=_log(rng, 1, 64), new_lo=rng.randrange(1, hi + 1), new_hi=hi, ctx_lo=rng.choice([0, 5]),
             ctx_hi=_log(rng, 6, 32768), page=page, q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim,
             window=rng.choice([0, 0, _log(rng, 1, 4096)]), dtype=dtype, pad=pad)
    # no dearer than the listed ones: fewer sequences, then shorter contexts, then shorter chunks
    most = max(work(x)["flops"] for x in LISTED) // (16 if dtype == "f32" else 2)
    while (_padded(c)[0] > 1 << 30 or _padded(c)[1] > 1 << 29 or work(c)["flops"] > most
           or work(c)["bytes"] > 250 << 20):
        if c["n"] > 3:
            c["n"] = c["n"] * 2 // 3
        elif c["ctx_hi"] > 1000:
            c["ctx_hi"] = c["ctx_hi"] * 2 // 3
        else:
            c["new_hi"] = max(1, c["new_hi"] * 2 // 3)
            c["new_lo"] = min(c["new_lo"], c["new_hi"])
    return c


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ctx, new = lengths(case)
    n, page = case["n"], case["page"]
    tokens = sum(new)
    rows = tokens + case["pad"]
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    s = {"case": case, "tokens": tokens, "max_new": max(1, max(new)),
         "cu": torch.tensor(cu, dtype=torch.int32, device=dev)}
    width = max(1, max(-(-(c + m + case.get("rollback", 0)) // page) for c, m in zip(ctx, new)))
    n_pages = n * width + 3
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    if case["op"] == "plan":
        # what a running server holds: the pages of every request so far (some hold drafts since rejected), the
        # others in the free list
        held = [c + (case["rollback"] if i % 3 == 0 else 0) for i, c in enumerate(ctx)]
        have = [-(-h // page) for h in held]
        have_t = torch.tensor(have, device=dev)
        col = torch.arange(width, device=dev)
        mask = col[None, :] < have_t[:, None]
        start = torch.cumsum(have_t, 0) - have_t
        table = torch.where(mask, order[(start[:, None] + col[None, :]).clamp(max=n_pages - 1)], torch.zeros_like(order[:1]))
        used = sum(have)
        free = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        free[: n_pages - used] = order[used:]
        s.update(ctx=torch.tensor(ctx, dtype=torch.int32, device=dev), rows=rows, table=table.contiguous(), free=free,
                 held=torch.tensor(held, dtype=torch.int32, device=dev),
                 count=torch.tensor([n_pages - used], dtype=torch.int32, device=dev))
        return s
    io = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    hk, d = case["kv_heads"], case["dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=io)

    table = order[: n * width].view(n, width).contiguous()
    s["k_cache"], s["v_cache"] = normal(n_pages, hk, page, d), normal(n_pages, hk, page, d)
    if case["op"] == "write":
        pos = torch.cat([torch.arange(c, c + m, device=dev) for c, m in zip(ctx, new)])
        seq = torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(new, device=dev))
        slots = torch.full((rows,), -1, dtype=torch.int32, device=dev)
        slots[:tokens] = table[seq, pos // page] * page + (pos % page).to(torch.int32)
        fused = normal(rows, 2, hk, d)   # the projection's output: a row holds a token's keys, then its values
        s.update(k=fused[:, 0], v=fused[:, 1], slots=slots)
        return s
    s.update(table=table, kv_lens=torch.tensor([c + m for c, m in zip(ctx, new)], dtype=torch.int32, device=dev),
             q=normal(rows, case["q_heads"], d), o=torch.zeros(rows, case["q_heads"], d, dtype=io, device=dev),
             lse=torch.zeros(rows, case["q_heads"], dtype=torch.float32, device=dev), parts=[])
    for part in ([i for i in range(n) if new[i] == 1], [i for i in range(n) if new[i] > 1]):
        if part:
            most = max(new[i] for i in part)
            packed = [cu[i] + t for i in part for t in range(new[i])]
            padded = [k * most + t for k, i in enumerate(part) for t in range(new[i])]
            s["parts"].append((torch.tensor(part, device=dev), most, max(ctx[i] + new[i] for i in part),
                               torch.tensor(packed, device=dev), torch.tensor(padded, device=dev)))
    return s


def _plain_plan(s):
    page = s["case"]["page"]
    table, free, count = s["table"], s["free"], s["count"].long()
    n, width = table.shape
    cu, ctx = s["cu"].long(), s["ctx"].long()
    new = cu[1:] - cu[:-1]
    have = (s["held"].long() + page - 1) // page
    need = (ctx + new + page - 1) // page
    fits = need <= width
    rel = (have - need).clamp(min=0)
    take = torch.where(fits, (need - have).clamp(min=0), 0)
    col = torch.arange(width, device=table.device)
    # pages that go back onto the stack, in the order of sequences and columns
    back = (col >= need[:, None]) & (col < have[:, None])
    at = count + torch.cumsum(rel, 0)[:, None] - rel[:, None] + col - need[:, None]
    last = free.numel()
    stack = torch.cat([free, free.new_zeros(1)])
    stack.scatter_(0, torch.where(back, at, last).flatten(), table.flatten())
    avail = count + rel.sum()
    ends = torch.cumsum(take, 0)
    served = fits & ((take == 0) | (ends <= avail))
    taken = torch.where(served, ends, 0).max()
    t = ends[:, None] - take[:, None] + col - have[:, None]
    fresh = served[:, None] & (col >= have[:, None]) & (col < need[:, None])
    got = stack[(avail - 1 - t).clamp(0, last - 1)]
    table.copy_(torch.where(fresh, got, table))
    free.copy_(stack[:last])
    row = torch.arange(s["rows"], device=table.device)
    seq = torch.searchsorted(cu[1:].contiguous(), row, right=True).clamp(max=n - 1)
    live = (row < cu[-1]) & served[seq]
    pos = ctx[seq] + row - cu[seq]
    slot = table[seq, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    return (torch.where(live, slot, -1).int(), torch.where(live, pos, -1).int(),
            torch.where(served, ctx + new, ctx).int(),
            torch.where(served, ctx + new, s["held"].long()).int(), (avail - taken).int(), (~served).sum().int().view(1), table, free)


def _plain_write(s):
    page, t = s["case"]["page"], s["tokens"]
    slot = s["slots"][:t].long()
    s["k_cache"][slot // page, :, slot % page] = s["k"][:t]
    s["v_cache"][slot // page, :, slot % page] = s["v"][:t]
    return s["k_cache"], s["v_cache"]


def _attend(s, seqs, most, longest):
    """Output and log-sum-exp of the sequences `seqs`, padded to `most` new tokens and `longest` keys."""
    case = s["case"]
    page, hk, d, n = case["page"], case["kv_heads"], case["dim"], seqs.numel()
    g = case["q_heads"] // hk
    dev = s["q"].device
    cu, kv = s["cu"].long(), s["kv_lens"].long()[seqs]
    first, new = cu[seqs], cu[seqs + 1] - cu[seqs]
    # the pages of every sequence side by side
    at = s["table"][seqs, : -(-longest // page)].long()
    k = s["k_cache"][at].float().permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)[:, :, :longest]
    v = s["v_cache"][at].float().permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)[:, :, :longest]
    i = torch.arange(most, device=dev)
    row = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(n, most, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * most, d)
    sc = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(1.0 / math.sqrt(d)).view(n, hk, g, most, longest)
    j = torch.arange(longest, device=dev)
    p = (kv - new)[:, None] + i
    seen = j <= p[:, :, None]
    if case["window"]:
        seen &= j > p[:, :, None] - case["window"]
    sc = sc.masked_fill_(~seen[:, None, None], float("-inf"))
    top = sc.amax(-1, keepdim=True)
    sc = sc.sub_(top).exp_()
    total = sc.sum(-1, keepdim=True)
    out = torch.matmul(sc.view(n, hk, g * most, longest), v).view(n, hk, g, most, d).div_(total)
    out = out.permute(0, 3, 1, 2, 4).reshape(n * most, hk * g, d)
    return out, (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(n * most, hk * g)


def _plain_attn(s):
    # the requests that bring one token and the others apart, so that neither is padded to the other
    for seqs, most, longest, rows, src in s["parts"]:
        out, lse = _attend(s, seqs, most, longest)
        # back to packed rows; rows behind the last sequence stay as they were
        s["o"][rows] = out[src].to(s["o"].dtype)
        s["lse"][rows] = lse[src]
    return s["o"], s["lse"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "write": _plain_write, "attn": _plain_attn}[op](s)
    import gated_linear_recurrence_amd as glr
    if op == "plan":
        out = glr.rglru_page_plan(s["ctx"], s["cu"], s["table"], s["free"], s["count"], n_tokens=s["rows"],
                                  page_size=s["case"]["page"], held_lens=s["held"], max_new=s["max_new"])
        return (*out, s["table"], s["free"])
    if op == "write":
        glr.rglru_paged_kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
        return s["k_cache"], s["v_cache"]
    return glr.rglru_paged_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_lens"],
                                    max_new=s["max_new"], window=s["case"]["window"], o=s["o"], lse=s["lse"])


def exact(case, seed):
    """From the definition, a sequence and a key head at a time, in 64 bits."""
    s = prepare(case, seed)
    ctx, new = lengths(case)
    cu = s["cu"].tolist()
    if case["op"] == "plan":
        return None   # whole numbers only
    if case["op"] == "write":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for t, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                kc[slot // case["page"], :, slot % case["page"]] = s["k"][t].double()
                vc[slot // case["page"], :, slot % case["page"]] = s["v"][t].double()
        return kc, vc
    o, lse = s["o"].double(), s["lse"].double()
    d, hk = case["dim"], case["kv_heads"]
    g = case["q_heads"] // hk
    for b, (c, m) in enumerate(zip(ctx, new)):
        pages = s["table"][b, : -(-(c + m) // case["page"])].long()
        for h in range(hk):
            keys = s["k_cache"][pages, h].double().reshape(-1, d)[: c + m]
            values = s["v_cache"][pages, h].double().reshape(-1, d)[: c + m]
            for t0 in range(0, m, 512):
                t1 = min(m, t0 + 512)
                where = torch.arange(c + t0, c + t1, device=o.device)[:, None] - torch.arange(c + m, device=o.device)
                bad = where < 0
                if case["window"]:
                    bad |= where >= case["window"]
                rows = slice(cu[b] + t0, cu[b] + t1)
                for x in range(h * g, h * g + g):
                    z = (s["q"][rows, x].double() @ keys.T) / math.sqrt(d)
                    z[bad] = -math.inf
                    norm = torch.logsumexp(z, 1)
                    lse[rows, x] = norm
                    o[rows, x] = torch.exp(z - norm[:, None]) @ values
    return o, lse
