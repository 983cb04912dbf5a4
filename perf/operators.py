"""The serving attention operators and how they are measured.

Three operators run one after another in every step of a served model:

  plan       block tables, slot maps and positions of a batch, built on the GPU
             from the requests' lengths and a pool of free pages;
  append     rotary positions on q and k, and the step's keys and values
             written into the paged cache;
  attention  a chunk of new tokens (or one) per request over the paged cache,
             causal, with an optional sliding window and first tokens that
             stay visible (sinks).

Each case is one call.  `own` chooses between the plain form, written with
elementary torch operations in 32 bits, and the framework's kernels.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
ROPE_BASE = 10000.0


# ---- lengths ---------------------------------------------------------------------------

def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], evenly spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lengths(case):
    """(tokens already in the cache, new tokens) of each request: fixed by the case."""
    rng = random.Random(case["pick"])
    ctx, new = [], []
    for _ in range(case["batch"]):
        c = _log_int(rng, case["ctx_lo"] + 1, case["ctx_hi"] + 1) - 1
        n = _log_int(rng, case["new_lo"], case["new_hi"])
        if case["op"] == "plan":
            if rng.random() < case["decode_share"]:
                n = 1
            if rng.random() < case["ended_share"]:
                n = -1
        ctx.append(c)
        new.append(n)
    return ctx, new


def _pages(tokens, page):
    return -(-tokens // page)


def _visible(pos, window, sinks):
    """How many keys the query at position `pos` sees."""
    if not window or pos < window:
        return pos + 1
    return window + min(sinks, pos + 1 - window)


# ---- cases -----------------------------------------------------------------------------

def listed():
    def plan(name, batch, pick, ctx_hi, new_hi, decode_share, ended_share, page):
        return {"name": name, "op": "plan", "batch": batch, "pick": pick, "ctx_lo": 0, "ctx_hi": ctx_hi, "new_lo": 1,
                "new_hi": new_hi, "decode_share": decode_share, "ended_share": ended_share, "page": page}

    def append(name, batch, pick, ctx_lo, ctx_hi, new_lo, new_hi, heads, kv_heads, head_dim, page, dtype):
        return {"name": name, "op": "append", "batch": batch, "pick": pick, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
                "new_lo": new_lo, "new_hi": new_hi, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
                "page": page, "dtype": dtype}

    def attend(name, batch, pick, ctx_lo, ctx_hi, new_lo, new_hi, heads, kv_heads, head_dim, page, dtype, window=0,
               sinks=0):
        return {"name": name, "op": "attention", "batch": batch, "pick": pick, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
                "new_lo": new_lo, "new_hi": new_hi, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
                "page": page, "dtype": dtype, "window": window, "sinks": sinks}

    return [
        # a small server's decode step: one token for each of 16 requests
        plan("plan_decode_16", 16, 1, 2000, 1, 1.0, 0.0, 16),
        # a full server's step: mostly decode, some prompts in chunks, some requests that have ended
        plan("plan_mixed_1000", 1000, 2, 30000, 2048, 0.93, 0.04, 16),
        # decode of 16 requests of the 65B layer (64 heads of 128)
        append("append_decode_16", 16, 3, 100, 2000, 1, 1, 64, 64, 128, 16, "bf16"),
        # prompts in chunks, heads in groups of four, far positions
        append("append_chunk_8k", 5, 4, 1000, 130000, 1500, 1800, 32, 8, 128, 64, "fp16"),
        # one user's decode step of the 7B layer: latency
        attend("decode_1", 1, 5, 500, 500, 1, 1, 32, 32, 128, 16, "bf16"),
        # decode of 16 long requests of the 65B layer: bandwidth
        attend("decode_16_65b", 16, 6, 3900, 4300, 1, 1, 64, 64, 128, 16, "bf16"),
        # decode of 64 requests of very unlike lengths, heads in groups of four
        attend("decode_64_ragged", 64, 7, 100, 16000, 1, 1, 32, 8, 128, 64, "fp16"),
        # one whole prompt of the 7B layer, nothing in the cache
        attend("prompt_4096", 1, 8, 0, 0, 4096, 4096, 32, 32, 128, 16, "bf16"),
        # chunks of several requests over their contexts, heads of 64 in groups of eight
        attend("chunk_ragged", 7, 9, 100, 8000, 100, 1000, 32, 4, 64, 32, "fp16"),
        # decode with a window of 1024 and four sinks over long contexts
        attend("window_decode_32", 32, 10, 2000, 16000, 1, 1, 32, 8, 128, 16, "bf16", 1024, 4),
        # chunks of four long prompts with the same window
        attend("window_chunk_4", 4, 11, 1000, 8000, 1500, 2048, 32, 32, 128, 64, "bf16", 1024, 4),
    ]


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "attention", "attention"])
    case = {"op": op, "pick": rng.randrange(1 << 30)}
    if op == "plan":
        batch = _log_int(rng, 1, 1000)
        return {**case, "batch": batch, "ctx_lo": 0, "ctx_hi": _log_int(rng, 100, 30000), "new_lo": 1,
                "new_hi": _log_int(rng, 1, 2048), "decode_share": rng.choice([0.0, 0.5, 0.9]) if batch <= 100 else 0.93,
                "ended_share": rng.choice([0.0, 0.04]), "page": rng.choice([16, 32, 64, 128])}
    kv_heads = rng.choice([1, 2, 4, 5, 8, 32])
    heads = kv_heads * (rng.choice([1, 2]) if kv_heads == 32 else rng.choice([1, 2, 4, 7, 8]))
    case |= {"heads": heads, "kv_heads": kv_heads, "head_dim": rng.choice([64, 128]),
             "page": rng.choice([16, 32, 64, 128]), "dtype": rng.choice(["bf16", "fp16"])}
    if op == "append":
        batch = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, 8192 // batch)
        return {**case, "batch": batch, "ctx_lo": 0, "ctx_hi": _log_int(rng, 100, 130000),
                "new_lo": _log_int(rng, 1, new), "new_hi": new}
    window, sinks = rng.choice([(0, 0), (0, 0), (_log_int(rng, 64, 4096), rng.choice([0, 1, 4, 16]))])
    case |= {"window": window, "sinks": sinks}
    if rng.random() < 0.5:  # decode: one token, or a few that were guessed ahead
        batch = _log_int(rng, 1, 64)
        new = rng.choice([1, 1, 1, 2, 5])
        ctx = _log_int(rng, 64, min(16000, 4_000_000 // (batch * kv_heads)))
        return {**case, "batch": batch, "ctx_lo": _log_int(rng, 16, ctx), "ctx_hi": ctx, "new_lo": new, "new_hi": new}
    batch = _log_int(rng, 1, 7)
    # no more products than a whole prompt of 4096 with 32 heads of 128 has
    pairs = 4096 * 2048 * 32 // (heads * batch)
    new = _log_int(rng, 16, min(4096, math.isqrt(2 * pairs)))
    ctx = _log_int(rng, 1, max(1, min(8000, pairs // new - new)))
    return {**case, "batch": batch, "ctx_lo": 0, "ctx_hi": ctx, "new_lo": _log_int(rng, 8, new), "new_hi": new}


# ---- inputs ----------------------------------------------------------------------------

def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "attention": _prepare_attention}[case["op"]](case, seed)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(gen, counts, num_pages, width):
    """Block tables of the given page counts over a shuffled pool, and the pages left over."""
    order = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    counts = torch.tensor(counts, device="cuda")
    at = torch.arange(width, device="cuda")
    held = at[None] < counts[:, None]
    first = torch.cumsum(counts, 0) - counts
    table = torch.where(held, order[(first[:, None] + at[None]).clamp(max=num_pages - 1)], -1)
    return table.to(torch.int32).contiguous(), order[int(counts.sum()):].contiguous()


def _prepare_plan(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    page = case["page"]
    ctx, new = _lengths(case)
    held = [_pages(c, page) for c in ctx]
    fresh = sum(_pages(c + max(n, 0), page) - h for c, n, h in zip(ctx, new, held))
    num_pages = sum(held) + fresh + 64
    width = max(_pages(c + max(n, 0), page) for c, n in zip(ctx, new))
    table, free = _tables(gen, held, num_pages, width)
    tokens = sum(max(n, 0) for n in new) + 8     # eight rows of padding, as a captured step has them
    pool = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    pool[:free.numel()] = free
    s = {"op": "plan", "page": page, "num_pages": num_pages, "tokens": tokens, "batch": case["batch"], "width": width,
         "table": table, "ctx": _int32(ctx), "new": _int32(new), "free_pages": pool,
         "free_count": _int32([free.numel()]), "free_count_out": _int32([0])}
    if own:
        import bit_nf4_quantized_16_b200 as q
        # what a server keeps: the batch's buffers.  The plan reads only the cache's page size and page count.
        s["kv"] = q.KVBatch(case["batch"], width, tokens, block_table=table)
    return s


def _prepare_step(case, seed):
    """What append and attention share: a batch that has been planned, with its cache."""
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype, page = DTYPES[case["dtype"]], case["page"]
    ctx, new = _lengths(case)
    total = [c + n for c, n in zip(ctx, new)]
    counts = [_pages(t, page) for t in total]
    width = max(counts)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    tokens = start[-1]
    request = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"), torch.tensor(new, device="cuda"))
    row = torch.arange(tokens, device="cuda") - torch.tensor(start, device="cuda")[request]
    positions = torch.tensor(ctx, device="cuda")[request] + row
    s = {"op": case["op"], "batch": case["batch"], "tokens": tokens, "width": width, "most_new": max(new), "page": page,
         "heads": case["heads"], "kv_heads": case["kv_heads"], "head_dim": case["head_dim"], "dtype": dtype,
         "cu_q": _int32(start), "kv_len": _int32(total), "positions": positions.to(torch.int32), "request": request,
         "row": row}

    def normal(*shape, std=1.0):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    return s, gen, normal, counts


def _prepare_append(case, seed):
    s, gen, normal, counts = _prepare_step(case, seed)
    # The cache holds just the pages that this step writes to: page ids are dense over them.
    page = s["page"]
    index = (s["request"] * s["width"] + s["positions"].long() // page).unique(return_inverse=True)[1]
    num_pages = int(index.max()) + 9
    order = torch.randperm(num_pages, generator=gen, device="cuda")
    s["slots"] = (order[index] * page + s["positions"].long() % page).to(torch.int32)
    shape = (num_pages, s["kv_heads"], page, s["head_dim"])
    s |= {"k_cache": torch.zeros(shape, dtype=s["dtype"], device="cuda"),
          "v_cache": torch.zeros(shape, dtype=s["dtype"], device="cuda"),
          "q": normal(s["tokens"], s["heads"], s["head_dim"]), "k": normal(s["tokens"], s["kv_heads"], s["head_dim"]),
          "v": normal(s["tokens"], s["kv_heads"], s["head_dim"])}
    s["q_out"] = torch.empty_like(s["q"])
    half = s["head_dim"] // 2
    s["frequencies"] = ROPE_BASE ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    if own:
        import bit_nf4_quantized_16_b200 as q
        s["cache"] = q.KVCache(s["k_cache"], s["v_cache"])
        s["kv"] = q.KVBatch(s["batch"], 1, s["tokens"], positions=s["positions"], slots=s["slots"])
        s["rope"] = q.qlora_build_rope(s["head_dim"], ROPE_BASE)
    return s


def _prepare_attention(case, seed):
    s, gen, normal, counts = _prepare_step(case, seed)
    num_pages = sum(counts) + 8
    s["table"], _ = _tables(gen, counts, num_pages, s["width"])
    shape = (num_pages, s["kv_heads"], s["page"], s["head_dim"])
    s |= {"k_cache": normal(*shape), "v_cache": normal(*shape), "window": case["window"], "sinks": case["sinks"],
          # queries of twice the keys' deviation: scores of deviation two
          "q": normal(s["tokens"], s["heads"], s["head_dim"], std=2.0), "scale": s["head_dim"] ** -0.5}
    s["out"] = torch.empty_like(s["q"])
    if own:
        import bit_nf4_quantized_16_b200 as q
        s["cache"] = q.KVCache(s["k_cache"], s["v_cache"])
        s["kv"] = q.KVBatch(s["batch"], s["width"], s["tokens"], max_q_len=s["most_new"], block_table=s["table"],
                            cu_q=s["cu_q"], kv_len=s["kv_len"])
        s["workspace"] = torch.empty(q.qlora_paged_attn_workspace_bytes(s["cache"], s["kv"], s["heads"]),
                                     dtype=torch.uint8, device="cuda")
    return s


# ---- one pass --------------------------------------------------------------------------

def run(s):
    if own:
        return {"plan": _own_plan, "append": _own_append, "attention": _own_attention}[s["op"]](s)
    return {"plan": _plain_plan, "append": _plain_append, "attention": _plain_attention}[s["op"]](s)


def _own_plan(s):
    import bit_nf4_quantized_16_b200 as q
    kv = s["kv"]
    q.qlora_kv_plan(kv, s["page"], s["num_pages"], s["ctx"], s["new"], s["free_pages"], s["free_count"],
                    s["free_count_out"])
    return {"block_table": kv.block_table, "cu_q": kv.cu_q, "kv_len": kv.kv_len, "positions": kv.positions,
            "slots": kv.slots, "free_pages": s["free_pages"], "free_count": s["free_count_out"]}


def _own_append(s):
    import bit_nf4_quantized_16_b200 as q
    q.qlora_kv_append(s["cache"], s["kv"], s["rope"], s["q"], s["k"], s["v"], s["q_out"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attention(s):
    import bit_nf4_quantized_16_b200 as q
    q.qlora_paged_attn_fwd(s["cache"], s["kv"], s["q"], s["out"], s["scale"], s["workspace"], window=s["window"],
                           sinks=s["sinks"])
    return s["out"]


def _plain_plan(s):
    page, width, tokens = s["page"], s["width"], s["tokens"]
    ctx, new, count = s["ctx"].long(), s["new"].long(), s["free_count"].long()
    live = new >= 0
    rows = torch.where(live, new, 0)
    ends = torch.cumsum(rows, 0)
    cu_q = torch.cat([torch.zeros_like(ends[:1]), ends]).clamp(max=tokens)
    held, total = (ctx + page - 1) // page, ctx + rows
    # the pages of requests that have ended go back on top of the pool
    back = torch.where(live, 0, held)
    back_ends = torch.cumsum(back, 0)
    at = torch.arange(s["num_pages"], device="cuda")
    j = at - count
    owner = torch.searchsorted(back_ends, j.contiguous(), right=True).clamp(max=s["batch"] - 1)
    theirs = s["table"].long()[owner, (j - (back_ends - back)[owner]).clamp(0, width - 1)]
    pool_size = count + back_ends[-1]
    pool = torch.where((j >= 0) & (at < pool_size), theirs, s["free_pages"].long())
    # pages are taken from the top, in the requests' order
    fits = live & (total <= width * page) & ((ends <= tokens) | (rows == 0))
    need = torch.where(fits, (total + page - 1) // page - held, 0)
    taken = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (taken <= pool_size))
    used = torch.where(granted, taken, 0).max()
    at = torch.arange(width, device="cuda")[None]
    fresh = granted[:, None] & (at >= held[:, None]) & (at < (held + need)[:, None])
    place = pool_size - 1 - ((taken - need)[:, None] + at - held[:, None])
    table = torch.where(fresh, pool[place.clamp(0, s["num_pages"] - 1)], s["table"].long())
    # positions and slots of the new tokens
    t = torch.arange(tokens, device="cuda")
    request = torch.searchsorted(cu_q[1:].contiguous(), t, right=True)
    inside = request < s["batch"]
    request = request.clamp(max=s["batch"] - 1)
    inside &= granted[request]
    position = torch.where(inside, ctx[request] + t - cu_q[request], -1)
    slot = table[request, position.clamp(min=0) // page] * page + position % page
    return {"block_table": table.int(), "cu_q": cu_q.int(), "kv_len": torch.where(granted, total, 0).int(),
            "positions": position.int(), "slots": torch.where(inside, slot, -1).int(), "free_pages": pool.int(),
            "free_count": (pool_size - used).int()}


def _plain_append(s):
    angles = s["positions"].double()[:, None] * s["frequencies"][None]
    cos, sin = angles.cos().float()[:, None], angles.sin().float()[:, None]

    def rotate(x):
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(s["dtype"])

    slots = s["slots"].long()
    where, offset = slots // s["page"], slots % s["page"]
    s["k_cache"][where, :, offset] = rotate(s["k"])
    s["v_cache"][where, :, offset] = s["v"]
    return {"q": rotate(s["q"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attention(s):
    batch, most, heads, kv_heads, dim = s["batch"], s["most_new"], s["heads"], s["kv_heads"], s["head_dim"]
    group, length = heads // kv_heads, s["width"] * s["page"]
    table = s["table"].long().clamp(min=0)
    # [batch, kv head, position, dim], each request padded to the longest
    k = s["k_cache"][table].transpose(1, 2).reshape(batch, kv_heads, length, dim).float()
    v = s["v_cache"][table].transpose(1, 2).reshape(batch, kv_heads, length, dim).float()
    cu, kv_len = s["cu_q"].long(), s["kv_len"].long()
    rows = torch.arange(most, device="cuda")
    q = s["q"][(cu[:-1, None] + rows).clamp(max=s["tokens"] - 1)].float()
    q = q.view(batch, most, kv_heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, kv_heads, group * most, dim)
    scores = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(batch, kv_heads, group, most, length)
    own_position = (kv_len - (cu[1:] - cu[:-1]))[:, None] + rows            # [batch, row]
    at = torch.arange(length, device="cuda")
    seen = at <= own_position[..., None]
    if s["window"]:
        seen &= (at > own_position[..., None] - s["window"]) | (at < s["sinks"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    scores.div_(scores.sum(-1, keepdim=True))
    out = scores.view(batch, kv_heads, group * most, length) @ v
    out = out.view(batch, kv_heads, group, most, dim).permute(0, 3, 1, 2, 4).reshape(batch, most, heads, dim)
    return out[s["request"], s["row"]].to(s["dtype"])


# ---- what each pass cannot do without -----------------------------------------------------

def work(case):
    ctx, new = _lengths(case)
    if case["op"] == "plan":
        tokens, page = sum(max(n, 0) for n in new) + 8, case["page"]
        fresh = sum(_pages(c + max(n, 0), page) - _pages(c, page) for c, n in zip(ctx, new))
        back = sum(_pages(c, page) for c, n in zip(ctx, new) if n < 0)
        pages = sum(-(-(c % page + n) // page) for c, n in zip(ctx, new) if n > 0)   # pages that hold new tokens
        return {"bytes": 4 * (4 * len(ctx) + 2 * tokens + 2 * (fresh + back) + pages), "flops": 0}
    tokens, dim = sum(new), case["head_dim"]
    row = 2 * case["head_dim"]
    if case["op"] == "append":
        # q and its rotated copy, k and v and their places in the cache, positions and slots
        return {"bytes": tokens * (row * (2 * case["heads"] + 4 * case["kv_heads"]) + 8),
                "flops": tokens * 3 * dim * (case["heads"] + case["kv_heads"])}
    window, sinks = case["window"], case["sinks"]
    keys = pairs = 0
    for c, n in zip(ctx, new):
        first = max(0, c - window + 1) if window else 0     # the first position in the first row's window
        keys += c + n - first + min(sinks, first)
        pairs += sum(_visible(p, window, sinks) for p in range(c, c + n))
    return {"bytes": row * (2 * tokens * case["heads"] + 2 * keys * case["kv_heads"])
            + 4 * (2 * len(ctx) + sum(_pages(c + n, case["page"]) for c, n in zip(ctx, new))),
            "flops": 4 * dim * case["heads"] * pairs}


# ---- the definition in 64 bits ------------------------------------------------------------

def exact(case, seed):
    if case["op"] == "plan":
        return None     # whole numbers
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    if case["op"] == "append":
        half = case["head_dim"] // 2
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           torch.outer(s["positions"].double(),
                                       torch.tensor([ROPE_BASE ** (-i / half) for i in range(half)],
                                                    dtype=torch.float64, device="cuda")))

        def rotated(x):
            z = torch.complex(x[..., :half].double(), x[..., half:].double()) * turn[:, None]
            return torch.cat([z.real, z.imag], -1)

        def placed(x):
            flat = torch.zeros(s["k_cache"].shape, dtype=torch.float64, device="cuda").transpose(1, 2).contiguous()
            flat.view(-1, case["kv_heads"], case["head_dim"]).index_copy_(0, s["slots"].long(), x)
            return flat.transpose(1, 2).contiguous()

        return {"q": rotated(s["q"]), "k_cache": placed(rotated(s["k"])), "v_cache": placed(s["v"].double())}
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, start = case["heads"] // case["kv_heads"], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        pages = s["table"][b, :_pages(c + n, case["page"])].long()
        own_position = torch.arange(c, c + n, device="cuda")[:, None]
        at = torch.arange(c + n, device="cuda")[None]
        hidden = at > own_position
        if case["window"]:
            hidden |= (at <= own_position - case["window"]) & (at >= case["sinks"])
        for h in range(case["kv_heads"]):
            k = s["k_cache"][pages, h].reshape(-1, case["head_dim"])[:c + n].double()
            v = s["v_cache"][pages, h].reshape(-1, case["head_dim"])[:c + n].double()
            mine = s["q"][start:start + n, h * group:(h + 1) * group].double()
            weight = torch.einsum("nge,le->gnl", mine, k) * case["head_dim"] ** -0.5
            weight = torch.softmax(weight.masked_fill(hidden, -math.inf), -1)
            out[start:start + n, h * group:(h + 1) * group] = torch.einsum("gnl,le->nge", weight, v)
        start += n
    return out
