"""The 4-bit cache and the page pool as a serving program calls them, beside their plain forms.

Operators: the write of new keys and values into a paged cache of 4-bit blocks
(and the rows read back as the values they stand for), the attention of new
tokens over that cache, and the operations on a pool whose pages several
requests share: fork (a request goes on from another's context), free (requests
end or give tokens up) and compact (the pages in use move to the front of the
pool), the first and the last with the copies of page contents that they ask for.

A block is 32 elements of a head's row: one power of two (a byte b for
2^(b - 127), 255 for a block with an infinity or NaN) and 32 codes of 4 bits
(sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6; the even element of a pair in the low
half of a byte). The power is the smallest that takes the block's largest
magnitude to 6 or less, from 2^-126 to 2^125. Lengths are a function of the
case alone; values, page order and cache contents come from the seed.
"""
import math

import torch

own = False

LISTED = [
    # the keys and values of one decode step of 64 requests, and what the cache holds of them
    dict(name="write_decode_64", op="write", n=64, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=2048, page=16, kv_heads=8, dim=128,
         dtype="bf16", pad=0),
    # a step of prompt chunks: rows of a fused projection's output
    dict(name="write_chunks_16k", op="write", n=9, new_lo=1500, new_hi=2100, ctx_lo=0, ctx_hi=4000, page=64, kv_heads=8,
         dim=128, dtype="bf16", pad=100),
    # decode, four short requests, a local attention layer (the smallest call: latency)
    dict(name="attn_decode_4", op="attn", n=4, new_lo=1, new_hi=1, ctx_lo=100, ctx_hi=700, page=16, q_heads=10, kv_heads=1,
         dim=256, window=2048, dtype="bf16", pad=0),
    # decode, 64 running requests of mixed age: what a 4-bit cache is for
    dict(name="attn_decode_64", op="attn", n=64, new_lo=1, new_hi=1, ctx_lo=1, ctx_hi=16383, page=16, q_heads=32, kv_heads=8,
         dim=128, window=0, dtype="bf16", pad=0),
    # verification of drafts in float32: a few tokens of each request, one key head per query head
    dict(name="attn_drafts_f32", op="attn", n=32, new_lo=2, new_hi=6, ctx_lo=10, ctx_hi=4096, page=32, q_heads=16, kv_heads=16,
         dim=64, window=0, dtype="f32", pad=5),
    # one long prompt, a later chunk of it
    dict(name="attn_chunk_long", op="attn", n=1, new_lo=2048, new_hi=2048, ctx_lo=30011, ctx_hi=30011, page=128, q_heads=32,
         kv_heads=8, dim=128, window=0, dtype="bf16", pad=0),
    # 8 prompts, 8 answers each: 64 requests go on from the context of 8, over a 4-bit cache
    dict(name="fork_answers_64", op="fork", n=72, src=8, ctx_lo=100, ctx_hi=2000, page=16, kv_heads=8, dim=128, cache="q4"),
    # half of 512 rows go on from the other half, a row each, over a bf16 cache
    dict(name="fork_rows_512", op="fork", n=512, src=256, ctx_lo=1, ctx_hi=1024, page=32, kv_heads=4, dim=128, cache="bf16"),
    # a step's end with 64 requests: some are done, some give rejected tokens up
    dict(name="free_64", op="free", n=64, ctx_lo=0, ctx_hi=8192, page=16, rollback=40),
    # the same with 1024
    dict(name="free_1024", op="free", n=1024, ctx_lo=0, ctx_hi=8192, page=16, rollback=200),
    # a pool twice as large as what 64 requests hold shrinks to half, bf16
    dict(name="compact_64", op="compact", n=64, ctx_lo=0, ctx_hi=2048, page=16, kv_heads=1, dim=256, cache="bf16"),
    # the same with 192 requests and a 4-bit cache of 8 heads
    dict(name="compact_192", op="compact", n=192, ctx_lo=0, ctx_hi=2048, page=64, kv_heads=8, dim=128, cache="q4"),
]


def listed():
    return [dict(c) for c in LISTED]


def _spread(lo, hi, n, phase):
    """n whole numbers over [lo, hi], unordered: a fixed low-discrepancy sequence."""
    return [lo + int((hi - lo + 1) * math.modf(phase + 0.6180339887498949 * i)[0]) for i in range(n)]


def lengths(case):
    """(tokens in the cache before the step, new tokens) of every sequence."""
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["n"], 0.5)
    return ctx, _spread(case["new_lo"], case["new_hi"], case["n"], 0.25)


def _pool(case):
    """Tokens held by every row and, of its pages, how many it shares with the row before."""
    held = _spread(case["ctx_lo"], case["ctx_hi"], case["n"], 0.5)
    if case["op"] == "fork":
        return [h if i < case["src"] else 0 for i, h in enumerate(held)], [0] * case["n"]
    shared = [0] * case["n"]
    for i in range(2, case["n"], 3):   # every third row went on from half of the one before
        shared[i] = min(held[i - 1] // 2, held[i]) // case["page"]
    return held, shared


def _keep(case):
    """Tokens that every row keeps: a quarter are done, a quarter give some up."""
    held, _ = _pool(case)
    some = _spread(0, case["rollback"], case["n"], 0.1)
    return [0 if i % 4 == 0 else max(0, h - some[i]) if i % 4 == 1 else h for i, h in enumerate(held)]


def _page_bytes(case):
    """Bytes of a page in every array of the cache."""
    rows = case["page"] * case["kv_heads"]
    if case["cache"] == "bf16":
        return [rows * case["dim"] * 2] * 2
    return [rows * case["dim"] // 2, rows * case["dim"] // 32] * 2


def _sizes(case):
    """(pages of the pool, columns of the table, pages in use) of a pool's case."""
    held, shared = _pool(case)
    have = [-(-h // case["page"]) for h in held]
    used = sum(have) - sum(shared)
    spare = case["n"] + used // 8 + 3 if case["op"] != "compact" else used + 2
    return used + spare, max(1, max(have)), used


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
    op, page = case["op"], case["page"]
    if op in ("write", "attn"):
        ctx, new = lengths(case)
        tokens, d, hk = sum(new), case["dim"], case["kv_heads"]
        e = 2 if case["dtype"] == "bf16" else 4
        row = d // 2 + d // 32
        if op == "write":   # rows in, blocks written, rows out
            return {"bytes": tokens * hk * (4 * d * e + 2 * row) + 4 * (tokens + case["pad"]), "flops": 0}
        seen = [_visible(c, m, case["window"]) for c, m in zip(ctx, new)]
        hq = case["q_heads"]
        moved = 2 * tokens * hq * d * e + 4 * tokens * hq + 2 * hk * row * sum(k for _, k in seen)
        return {"bytes": moved + 4 * sum(-(-k // page) for _, k in seen), "flops": 4 * d * hq * sum(p for p, _ in seen)}
    held, shared = _pool(case)
    n_pages, width, used = _sizes(case)
    have = [-(-h // page) for h in held]
    if op == "free":   # table entries given up, counts of sharing read and written, pages pushed
        given = sum(h - -(-k // page) for h, k in zip(have, _keep(case)))
        return {"bytes": 16 * given + 16 * case["n"], "flops": 0}
    if op == "fork":   # table entries read and written, counts of sharing, and the pages that are copied
        src = [held[r % case["src"]] for r in range(case["src"], case["n"])]
        copied = sum(1 for s in src if s % page)
        return {"bytes": 16 * sum(-(-s // page) for s in src) + 32 * case["n"] + 2 * copied * sum(_page_bytes(case)), "flops": 0}
    # compact: the table, the counts of sharing and the free list in and out; about half of the pages in use move
    return {"bytes": 8 * sum(have) + 16 * n_pages + used * sum(_page_bytes(case)), "flops": 0}


def _padded(case):
    """Elements of the plain form's padded scores and of its gathered keys."""
    ctx, new = lengths(case)
    total = max(c + m for c, m in zip(ctx, new))
    return case["n"] * case["q_heads"] * max(new) * total, case["n"] * case["kv_heads"] * total * case["dim"]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "write", "attn", "attn", "attn", "attn", "attn", "fork", "free", "compact"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 16])
    pad = rng.choice([0, 1, rng.randrange(2, 200)])
    if op == "write":
        hi = _log(rng, 1, 1024)
        n = max(1, min(_log(rng, 1, 64), 16000 * 1024 // (hi * kv_heads * dim * (2 if dtype == "f32" else 1))))
        return dict(op=op, n=n, new_lo=rng.randrange(0, hi) + (n == 1), new_hi=hi, ctx_lo=0, ctx_hi=_log(rng, 1, 4096),
                    page=page, kv_heads=kv_heads, dim=dim, dtype=dtype, pad=pad)
    if op == "attn":
        group = rng.choice([1, 2, 4, 5, 8, 10, 16])
        hi = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 2, 2048), _log(rng, 2, 2048)])
        c = dict(op=op, n=_log(rng, 1, 64), new_lo=rng.randrange(1, hi + 1), new_hi=hi, ctx_lo=rng.choice([0, 5]),
                 ctx_hi=_log(rng, 6, 32768), page=page, q_heads=group * kv_heads, kv_heads=kv_heads, dim=dim,
                 window=rng.choice([0, 0, _log(rng, 1, 4096)]), dtype=dtype, pad=pad)
        # no dearer than the listed ones: fewer sequences, then shorter contexts, then shorter chunks
        most = max(work(x)["flops"] for x in LISTED) // (16 if dtype == "f32" else 2)
        while _padded(c)[0] > 1 << 30 or _padded(c)[1] > 1 << 29 or work(c)["flops"] > most or work(c)["bytes"] > 250 << 20:
            if c["n"] > 3:
                c["n"] = c["n"] * 2 // 3
            elif c["ctx_hi"] > 1000:
                c["ctx_hi"] = c["ctx_hi"] * 2 // 3
            else:
                c["new_hi"] = max(1, c["new_hi"] * 2 // 3)
                c["new_lo"] = min(c["new_lo"], c["new_hi"])
        return c
    n = _log(rng, 2, 1024)
    c = dict(op=op, n=n, ctx_lo=rng.choice([0, 1]), ctx_hi=_log(rng, 2, 8192), page=page)
    if op == "free":
        c["rollback"] = _log(rng, 1, 400)
        while work(c)["bytes"] > work(LISTED[9])["bytes"]:
            c["ctx_hi"] = c["ctx_hi"] * 2 // 3
        return c
    c.update(kv_heads=kv_heads, dim=dim, cache=rng.choice(["bf16", "q4"]))
    if op == "fork":
        c["src"] = rng.randrange(1, n)
    most = work(LISTED[7 if op == "fork" else 11])["bytes"]
    while work(c)["bytes"] > most or _sizes(c)[0] * sum(_page_bytes(c)) > 320 << 20:
        if c["ctx_hi"] > 100:
            c["ctx_hi"] = c["ctx_hi"] * 2 // 3
        elif c["n"] > 8:
            c["n"] = c["n"] * 2 // 3
            if op == "fork":
                c["src"] = min(c["src"], c["n"] - 1)
        elif c["kv_heads"] > 1:
            c["kv_heads"] = 1
        else:
            c["page"] //= 2
    return c


def _encode(x):
    """Rows [..., D] as codes [..., D / 2] and powers [..., D / 32] (uint8), in float32, where every step is exact."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    frac, exp = torch.frexp(top)   # top = frac 2^exp, frac in [0.5, 1): at most 6 2^e from e = exp - 3 on where frac <= 0.75
    e = (exp - 3 + (frac > 0.75)).clamp(-126, 125)
    odd = ~torch.isfinite(top)
    e = torch.where(odd | (top == 0), torch.full_like(e, -126), e)
    y = torch.where(odd[..., None], torch.zeros_like(b), torch.ldexp(b, -e[..., None]))
    a = y.abs()
    # halves go to the even code
    code = (a > 0.25).to(torch.uint8)
    for edge, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += a >= edge if even else a > edge
    code += torch.signbit(y).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, torch.where(odd, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _table(device, dtype):
    half = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(half + [-x for x in half], device=device, dtype=dtype)


def _decode(codes, powers):
    """The values of codes [..., D / 2] and powers [..., D / 32], in float32."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    p = powers.float() - 127.0
    p = torch.where(powers == 255, torch.full_like(p, float("nan")), torch.exp2(p))
    return (_table(codes.device, torch.float32)[both.int()].unflatten(-1, (-1, 32)) * p[..., None]).flatten(-2)


def _fill_pool(case, s, gen, dev):
    """A pool as a server holds it: a table, the tokens held, how many further rows share a page, the free list."""
    held, shared = _pool(case)
    n_pages, width, used = _sizes(case)
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    have = torch.tensor([-(-h // case["page"]) for h in held], device=dev)
    first = torch.tensor(shared, device=dev)
    col = torch.arange(width, device=dev)
    start = torch.cumsum(have - first, 0) - have
    mine = (col >= first[:, None]) & (col < have[:, None])
    table = torch.where(mine, order[(start[:, None] + col).clamp(0, n_pages - 1)], 0)
    theirs = col < first[:, None]
    table = torch.where(theirs, table.roll(1, 0), table)
    shares = torch.zeros(n_pages + 1, dtype=torch.int32, device=dev)
    shares.scatter_add_(0, torch.where(theirs, table, n_pages).long().flatten(), theirs.int().flatten())
    free = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
    free[: n_pages - used] = order[used:]
    s.update(table=table.contiguous(), held=torch.tensor(held, dtype=torch.int32, device=dev), shares=shares[:n_pages].clone(),
             free=free, count=torch.tensor([n_pages - used], dtype=torch.int32, device=dev))
    if "cache" in case:
        rows = (n_pages, case["kv_heads"], case["page"])
        if case["cache"] == "bf16":
            s["caches"] = [torch.randn(*rows, case["dim"], generator=gen, device=dev, dtype=torch.bfloat16) for _ in range(2)]
        else:
            s["caches"] = [torch.randint(0, 256 if c % 2 == 0 else 253, (*rows, case["dim"] // (32 if c % 2 else 2)),
                                         generator=gen, device=dev, dtype=torch.uint8) for c in range(4)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    page, n, op = case["page"], case["n"], case["op"]
    s = {"case": case}
    if op not in ("write", "attn"):
        _fill_pool(case, s, gen, dev)
        if op == "fork":
            s["from"] = torch.tensor([-1 if r < case["src"] else r % case["src"] for r in range(n)], dtype=torch.int32, device=dev)
        elif op == "free":
            s["keep"] = torch.tensor(_keep(case), dtype=torch.int32, device=dev)
        else:
            s["keep_pages"] = s["free"].numel() // 2
        return s
    ctx, new = lengths(case)
    tokens = sum(new)
    rows = tokens + case["pad"]
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    s.update(tokens=tokens, max_new=max(1, max(new)), cu=torch.tensor(cu, dtype=torch.int32, device=dev))
    width = max(1, max(-(-(c + m) // page) for c, m in zip(ctx, new)))
    n_pages = n * width + 3
    table = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)[: n * width].view(n, width).contiguous()
    io = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    hk, d = case["kv_heads"], case["dim"]
    # keys: some columns of a head are larger than others, the same ones for every token
    wide = torch.exp(0.5 * torch.randn(hk, d, generator=gen, device=dev))
    if op == "write":
        pos = torch.cat([torch.arange(c, c + m, device=dev) for c, m in zip(ctx, new)])
        seq = torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(new, device=dev))
        slots = torch.full((rows,), -1, dtype=torch.int32, device=dev)
        slots[:tokens] = table[seq, pos // page] * page + (pos % page).to(torch.int32)
        # the projection's output: a row holds a token's keys, then its values
        fused = torch.randn(rows, 2, hk, d, generator=gen, device=dev)
        fused[:, 0] *= wide
        fused = fused.to(io)
        s.update(k=fused[:, 0], v=fused[:, 1], slots=slots)
        shape = (n_pages, hk, page)
        s["cache"] = [torch.zeros(*shape, d // (32 if c % 2 else 2), dtype=torch.uint8, device=dev) for c in range(4)]
        return s
    parts = [[], [], [], []]
    for p in range(0, n_pages, max(1, (1 << 26) // (hk * page * d))):
        m = min(n_pages - p, max(1, (1 << 26) // (hk * page * d)))
        for i in range(2):
            x = torch.randn(m, hk, page, d, generator=gen, device=dev)
            for a, b in zip(parts[2 * i:], _encode(x * wide[:, None] if i == 0 else x)):
                a.append(b)
    s["cache"] = [torch.cat(p) for p in parts]
    s.update(table=table, kv_lens=torch.tensor([c + m for c, m in zip(ctx, new)], dtype=torch.int32, device=dev),
             q=torch.randn(rows, case["q_heads"], d, generator=gen, device=dev, dtype=io),
             o=torch.zeros(rows, case["q_heads"], d, dtype=io, device=dev),
             lse=torch.zeros(rows, case["q_heads"], dtype=torch.float32, device=dev), parts=[])
    for part in ([i for i in range(n) if new[i] == 1], [i for i in range(n) if new[i] > 1]):
        if part:
            most = max(new[i] for i in part)
            packed = [cu[i] + t for i in part for t in range(new[i])]
            padded = [k * most + t for k, i in enumerate(part) for t in range(new[i])]
            s["parts"].append((torch.tensor(part, device=dev), most, max(ctx[i] + new[i] for i in part),
                               torch.tensor(packed, device=dev), torch.tensor(padded, device=dev)))
    return s


def _plain_write(s):
    page, t, io = s["case"]["page"], s["tokens"], s["k"].dtype
    slot = s["slots"][:t].long()
    out = []
    for x, codes, powers in ((s["k"], *s["cache"][:2]), (s["v"], *s["cache"][2:])):
        c, p = _encode(x[:t])
        codes[slot // page, :, slot % page] = c
        powers[slot // page, :, slot % page] = p
        rows = torch.zeros_like(x, memory_format=torch.contiguous_format)
        rows[:t] = _decode(codes[slot // page, :, slot % page], powers[slot // page, :, slot % page]).to(io)
        out.append(rows)
    return tuple(out)


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
    k, v = (_decode(s["cache"][c][at], s["cache"][c + 1][at]).permute(0, 2, 1, 3, 4).reshape(n, hk, -1, d)[:, :, :longest]
            for c in (0, 2))
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


def _bits(s):
    """The caches, whose pages are copied bit by bit."""
    return [c if c.dtype == torch.uint8 else c.view(torch.int16) for c in s["caches"]]


def _plain_fork(s):
    page, table, held, shares = s["case"]["page"], s["table"], s["held"].long(), s["shares"]
    n_pages, (n, width) = s["free"].numel(), table.shape
    src = s["from"].long().clamp(0, n - 1)
    row = torch.arange(n, device=table.device)
    valid = (s["from"] >= 0) & (s["from"] < n) & (src != row) & (s["from"][src] < 0) & (held == 0)
    length = held[src]
    part = valid & (length % page != 0)
    rank = torch.cumsum(part, 0) - part.long()
    count = s["count"].long()
    served = valid & (~part | (rank < count))
    fresh = s["free"][(count - 1 - rank).clamp(0, n_pages - 1)]
    full = length // page
    col = torch.arange(width, device=table.device)
    shared = served[:, None] & (col < full[:, None])
    old = table[src]
    last = (full[:, None] == col) & (served & part)[:, None]
    pairs = torch.where((served & part)[:, None], torch.stack([old.gather(1, full.clamp(max=width - 1)[:, None])[:, 0], fresh], 1), -1)
    more = torch.zeros(n_pages + 1, dtype=torch.int32, device=table.device)
    more.scatter_add_(0, torch.where(shared, old, n_pages).long().flatten(), shared.int().flatten())
    shares += more[:n_pages]
    table.copy_(torch.where(shared, old, torch.where(last, fresh[:, None], table)))
    some = pairs[:, 0] >= 0
    first = pairs[some.int().argmax()].clamp(min=0)   # rows without a copy make the first one's again
    a, b = (torch.where(some, pairs[:, x], first[x]).long() for x in range(2))
    for c in s["caches"]:
        c[b] = c[a]
    lens = torch.where(served, length, held).int()
    return pairs.int(), lens, lens, (count - (served & part).sum()).int(), ((s["from"] >= 0) & ~served).sum().int().view(1), table, shares, *_bits(s)


def _plain_free(s):
    page, table, shares, free = s["case"]["page"], s["table"], s["shares"], s["free"]
    n_pages = free.numel()
    kept = torch.minimum(s["keep"], s["held"])
    have, stay = (s["held"].long() + page - 1) // page, (kept.long() + page - 1) // page
    col = torch.arange(table.shape[1], device=table.device)
    given = (col >= stay[:, None]) & (col < have[:, None])
    less = torch.zeros(n_pages + 1, dtype=torch.int32, device=table.device)
    less.scatter_add_(0, torch.where(given, table, n_pages).long().flatten(), given.int().flatten())
    shares -= less[:n_pages]
    gone = shares < 0
    shares.clamp_(min=0)
    count = s["count"].long()
    # the last page first, so that the first one is on top
    at = count + gone.flip(0).cumsum(0).flip(0) - 1
    stack = torch.cat([free, free.new_zeros(1)])
    stack.scatter_(0, torch.where(gone, at, n_pages), torch.arange(n_pages, device=table.device, dtype=torch.int32))
    free.copy_(stack[:n_pages])
    return kept, (count + gone.sum()).int(), shares, free


def _plain_compact(s):
    page, table, shares, free, keep = s["case"]["page"], s["table"], s["shares"], s["free"], s["keep_pages"]
    n_pages, dev = free.numel(), table.device
    most = min(keep, n_pages - keep)
    have = (s["held"].long() + page - 1) // page
    mine = torch.arange(table.shape[1], device=dev) < have[:, None]
    index = torch.arange(n_pages, device=dev)
    used, idle = (torch.zeros(n_pages + 1, dtype=torch.bool, device=dev) for _ in range(2))
    used.scatter_(0, torch.where(mine, table, n_pages).long().flatten(), True)
    idle.scatter_(0, torch.where(index < s["count"], free.long(), n_pages), True)
    used, idle = used[:n_pages], idle[:n_pages]
    go, to = used & (index >= keep), idle & ~used & (index < keep)
    rank, place = go.cumsum(0) - 1, to.cumsum(0) - 1
    moves = torch.minimum(go.sum(), to.sum())
    go &= rank < moves
    left = to & (place >= moves)
    to &= place < moves
    pairs = torch.full((most + 1, 2), -1, dtype=torch.int32, device=dev)
    pairs[torch.where(go, rank, most), 0] = index.int()
    pairs[torch.where(to, place, most), 1] = index.int()
    pairs = pairs[:most].contiguous()
    target = torch.where(go, pairs[rank.clamp(0, most - 1), 1].long(), index) if most else index
    table_out = torch.where(mine, target[table.long()].int(), table)
    shares_out = torch.cat([torch.where(go, 0, shares), shares.new_zeros(1)])
    shares_out.scatter_(0, torch.where(go, target, n_pages), shares)
    count = left.sum()
    free_out = torch.full((n_pages + 1,), -1, dtype=torch.int32, device=dev)
    free_out.scatter_(0, torch.where(left, count + moves - 1 - place, n_pages), index.int())
    for c in s["caches"]:
        a, b = (torch.where(pairs[:, x] >= 0, pairs[:, x], pairs[0, x]).long() for x in range(2))
        c[b] = c[a]
    return (table_out, shares_out[:n_pages], free_out[:n_pages], count.int().view(1), pairs, moves.int().view(1),
            (used & (index >= keep)).sum().int().view(1) - moves.int(), *_bits(s))


PLAIN = {"write": _plain_write, "attn": _plain_attn, "fork": _plain_fork, "free": _plain_free, "compact": _plain_compact}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    import gated_linear_recurrence_amd as glr
    if op == "write":
        glr.rglru_paged_kv_write_q4(s["k"], s["v"], *s["cache"], s["slots"])
        return glr.rglru_paged_kv_read_q4(*s["cache"], s["slots"], dtype=s["k"].dtype)
    if op == "attn":
        return glr.rglru_paged_attn_q4_fwd(s["q"], *s["cache"], s["table"], s["cu"], s["kv_lens"], max_new=s["max_new"],
                                           window=case["window"], o=s["o"], lse=s["lse"])
    pool = (s["held"], s["table"], s["shares"], s["free"], s["count"])
    if op == "fork":
        pairs, lens, held, count, unserved = glr.rglru_page_fork(s["from"], *pool, page_size=case["page"])
        glr.rglru_page_copy(pairs, s["caches"])
        return pairs, lens, held, count, unserved, s["table"], s["shares"], *_bits(s)
    if op == "free":
        kept, count = glr.rglru_page_free(s["keep"], *pool, page_size=case["page"])
        return kept, count, s["shares"], s["free"]
    table, shares, free, count, pairs, n_pairs, unmoved = glr.rglru_page_compact(*pool, page_size=case["page"],
                                                                                 keep_pages=s["keep_pages"])
    glr.rglru_page_copy(pairs, s["caches"], n_pairs=n_pairs)
    return table, shares, free, count, pairs, n_pairs, unmoved, *_bits(s)


def _values(codes, powers):
    """The values of a few rows of the cache, in 64 bits."""
    out = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    value = _table(codes.device, torch.float64)
    out[..., 0::2] = value[(codes % 16).long()]
    out[..., 1::2] = value[(codes // 16).long()]
    return out * torch.repeat_interleave(torch.pow(2.0, powers.double() - 127), 32, -1)


def _blocks(x):
    """What rows become as 4-bit blocks, from the definition: the nearest of a block's values, of two the one of even code."""
    b = x.double().unflatten(-1, (-1, 32))
    power = torch.full_like(b[..., :1], -126.0)
    for e in range(-126, 125):   # the smallest power that takes all to 6 or less
        power += (b.abs().amax(-1, keepdim=True) > 6 * 2.0 ** e).double()
    y = b.abs() / torch.pow(2.0, power)
    half = _table(x.device, torch.float64)[:8]
    gap = torch.stack([(y - h).abs() * 2 + (c % 2) * 1e-12 for c, h in enumerate(half.tolist())])
    return (half[gap.argmin(0)] * torch.pow(2.0, power) * torch.sign(b)).flatten(-2)


def exact(case, seed):
    """From the definition, a sequence and a key head at a time, in 64 bits."""
    if case["op"] not in ("write", "attn"):
        return None   # whole numbers and copies only
    s = prepare(case, seed)
    if case["op"] == "write":
        out = []
        for x in (s["k"], s["v"]):
            rows = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
            for t in range(0, s["tokens"], 1024):
                rows[t: min(t + 1024, s["tokens"])] = _blocks(x[t: min(t + 1024, s["tokens"])])
            out.append(rows)
        return tuple(out)
    ctx, new = lengths(case)
    cu = s["cu"].tolist()
    o, lse = s["o"].double(), s["lse"].double()
    d, hk = case["dim"], case["kv_heads"]
    g = case["q_heads"] // hk
    for b, (c, m) in enumerate(zip(ctx, new)):
        pages = s["table"][b, : -(-(c + m) // case["page"])].long()
        for h in range(hk):
            keys, values = (_values(s["cache"][x][pages, h], s["cache"][x + 1][pages, h]).reshape(-1, d)[: c + m] for x in (0, 2))
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
