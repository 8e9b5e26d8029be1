"""The paged key/value cache and its attention: cases, their plain forms and
the library's calls.

Three operators of a decoding step that run between the q/k/v and the output
projections:

* ``plan``: pages, slots, positions and tree masks of a step's new tokens from
  the requests' lengths (``kv_plan``);
* ``append``: the new tokens' key and value rows written into a paged cache,
  as bf16 or as int8 codes with a scale per (token, head) (``kv_append``);
* ``attend``: attention of a tree of drafted tokens (or of one token, or of a
  causal chunk) over such a cache (``tree_attention``).

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the library.
"""
from __future__ import annotations

import math

import torch

own = False

HEAD_DIM = 128


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # plan: eight requests decode one token each; what a small server pays per step
        dict(name="plan_decode_r8", op="plan", requests=8, ctx_lo=5, ctx_hi=2000, new_lo=1, new_hi=1, page=16,
             tree=False),
        # plan: a full server verifies drafted trees of up to 64 nodes
        dict(name="plan_tree_r256", op="plan", requests=256, ctx_lo=0, ctx_hi=8190, new_lo=1, new_hi=64, page=16,
             tree=True),
        # plan: a thousand prompts of odd lengths enter at once
        dict(name="plan_prompts_r1001", op="plan", requests=1001, ctx_lo=0, ctx_hi=0, new_lo=1, new_hi=1023, page=32,
             tree=False),
        # append: one decoded token of eight requests, rows as the projections leave them (fp32)
        dict(name="append_decode_bf16", op="append", tokens=8, kv_heads=8, page=16, cache="bf16", rows="f32",
             head_major=False),
        # append: a long prompt's rows, fp32 into a bf16 cache whose pages keep each head together
        dict(name="append_prompt_bf16", op="append", tokens=16384, kv_heads=8, page=64, cache="bf16", rows="f32",
             head_major=True),
        # append: an odd number of bf16 rows into an int8 cache
        dict(name="append_prompt_int8", op="append", tokens=8191, kv_heads=8, page=16, cache="s8", rows="bf16",
             head_major=False),
        # attend: one request, one token, a short context, the heads of the 0.6B projections: latency alone
        dict(name="decode_r1", op="attend", requests=1, ctx_lo=777, ctx_hi=777, new_lo=1, new_hi=1, heads=16,
             kv_heads=8, page=16, cache="bf16", head_major=False, tree=False),
        # attend: a batch of ordinary decode steps with contexts from a few tokens to 8k
        dict(name="decode_r64", op="attend", requests=64, ctx_lo=3, ctx_hi=8191, new_lo=1, new_hi=1, heads=32,
             kv_heads=8, page=16, cache="bf16", head_major=False, tree=False),
        # attend: small drafted trees of odd sizes over an int8 cache
        dict(name="tree_r8_int8", op="attend", requests=8, ctx_lo=500, ctx_hi=4097, new_lo=9, new_hi=25, heads=16,
             kv_heads=8, page=32, cache="s8", head_major=False, tree=True),
        # attend: one long context (a book) with eight drafted tokens, int8 cache
        dict(name="long_r1_int8", op="attend", requests=1, ctx_lo=200001, ctx_hi=200001, new_lo=8, new_hi=8, heads=32,
             kv_heads=8, page=16, cache="s8", head_major=True, tree=True),
        # attend: causal chunks of prompts (no tree), contexts of a few thousand tokens
        dict(name="chunk_r4", op="attend", requests=4, ctx_lo=0, ctx_hi=6000, new_lo=300, new_hi=512, heads=16,
             kv_heads=8, page=128, cache="bf16", head_major=False, tree=False),
        # attend: wide trees over 16k contexts, eight query heads to a key head: the largest
        dict(name="tree_r16_wide", op="attend", requests=16, ctx_lo=6000, ctx_hi=16383, new_lo=64, new_hi=64, heads=32,
             kv_heads=4, page=64, cache="bf16", head_major=True, tree=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attend", "attend"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        tree = rng.random() < 0.5
        r = _log(rng, 1, 1024)
        new_hi = _log(rng, 1, 64) if tree else _log(rng, 1, max(1, min(4096, 500000 // r)))
        return dict(op=op, requests=r, ctx_lo=0, ctx_hi=_log(rng, 1, 8192), new_lo=1, new_hi=new_hi, page=page,
                    tree=tree)
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 16384), kv_heads=rng.choice([1, 2, 4, 8]), page=page,
                    cache=rng.choice(["bf16", "s8"]), rows=rng.choice(["f32", "bf16"]),
                    head_major=rng.random() < 0.5)
    kv = rng.choice([1, 2, 4, 8])
    heads = kv * rng.choice([1, 2, 4, 8])
    kind = rng.choice(["decode", "tree", "chunk"])
    new_hi = {"decode": 1, "tree": _log(rng, 2, 64), "chunk": _log(rng, 65, 512)}[kind]
    r = _log(rng, 1, {"decode": 64, "tree": 16, "chunk": 4}[kind])
    # contexts so long that a pass costs no more than the largest listed one
    most = max(64, min(200000, int(1.5e8 / (r * heads * max(new_hi, 8)))))
    hi = _log(rng, 1, most)
    return dict(op=op, requests=r, ctx_lo=hi // 4, ctx_hi=hi, new_lo=max(1, new_hi // 2), new_hi=new_hi, heads=heads,
                kv_heads=kv, page=page, cache=rng.choice(["bf16", "s8"]), head_major=rng.random() < 0.5,
                tree=kind == "tree")


def _spread(n, lo, hi, phase):
    """n whole numbers over lo..hi, both ends among them from n = 2 on, in a scattered order."""
    if n == 1:
        return [hi]
    mid = [lo + int((hi - lo) * ((i * 0.6180339887 + phase) % 1.0)) for i in range(n - 2)]
    return [hi] + mid + [lo]


def _lengths(case):
    r = case["requests"]
    return (_spread(r, case["ctx_lo"], case["ctx_hi"], 0.137), _spread(r, case["new_lo"], case["new_hi"], 0.741))


def work(case):
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        p, tokens = case["page"], sum(new)
        taken = sum(-(-(c + n) // p) + (-c // p) for c, n in zip(ctx, new))
        words = -(-max(new) // 32) if case["tree"] else 0
        moved = 8 * len(ctx) + 4 * (len(ctx) + 1) + 12 * tokens + 8 * taken
        return {"bytes": moved + (4 * tokens * (1 + words) if case["tree"] else 0), "flops": 0}
    if case["op"] == "append":
        values = 2 * case["tokens"] * case["kv_heads"] * HEAD_DIM
        e = 4 if case["rows"] == "f32" else 2
        scales = 4 * values // HEAD_DIM if case["cache"] == "s8" else 0
        return {"bytes": values * (e + (1 if case["cache"] == "s8" else 2)) + scales + 8 * case["tokens"],
                "flops": 2 * values if case["cache"] == "s8" else 0}
    ctx, new = _lengths(case)
    kv, h = case["kv_heads"], case["heads"]
    row = HEAD_DIM + 4 if case["cache"] == "s8" else 2 * HEAD_DIM
    cached = 2 * kv * row * sum(c + n for c, n in zip(ctx, new))
    pairs = sum(n * (c + (n + 1) / 2) for c, n in zip(ctx, new))   # each token sees half of its step's
    return {"bytes": cached + 4 * h * HEAD_DIM * sum(new), "flops": 4 * HEAD_DIM * h * pairs}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _starts(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return cu


def _tree_parents(new, seed):
    """Parents within each request: the first node is a root, each other hangs
    below one of the eight nodes before it (a draft of some depth and breadth)."""
    g = _gen(seed, "cpu")
    cu = _starts(new)
    tokens = cu[-1]
    i = torch.arange(tokens) - torch.repeat_interleave(torch.tensor(cu[:-1]), torch.tensor(new))
    back = 1 + (torch.rand(tokens, generator=g) * torch.clamp(i, max=8)).long()
    return torch.clamp(i - back, min=-1).to(torch.int32)


def _masks(parents, new, words):
    """Bit j of row i: j is i or one of its ancestors (rows of `words` 32-bit words)."""
    out = []
    for start, n in zip(_starts(new), new):
        seen = []
        for i in range(n):
            p = int(parents[start + i])
            seen.append((seen[p] if p >= 0 else 0) | (1 << i))
        out += [[(b >> (32 * w)) & 0xFFFFFFFF for w in range(words)] for b in seen]
    m = torch.tensor(out, dtype=torch.int64)
    return torch.where(m >= 2 ** 31, m - 2 ** 32, m).to(torch.int32)


def _empty_cache(case, pages, dtype, fill):
    """[pages][page][kv_heads][HEAD_DIM] as the operators see it; a head-major
    cache keeps a page's rows of one head together in memory."""
    p, h = case["page"], case["kv_heads"]
    if case["head_major"]:
        return torch.full((pages, h, p, HEAD_DIM), fill, dtype=dtype, device="cuda").permute(0, 2, 1, 3)
    return torch.full((pages, p, h, HEAD_DIM), fill, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    dev = torch.device("cuda")
    s = {"case": case, "op": case["op"]}
    if case["op"] == "append":
        t, h = case["tokens"], case["kv_heads"]
        pages = -(-t // case["page"]) + 1
        dtype = torch.float32 if case["rows"] == "f32" else torch.bfloat16
        # q, k and v rows leave one projection side by side: strided views of it
        both = torch.randn((t, 2 * h, HEAD_DIM), generator=g, device=dev)
        both *= torch.exp(0.5 * torch.randn((t, 2 * h, 1), generator=g, device=dev))
        both = both.to(dtype)
        s["k"], s["v"] = both[:, :h], both[:, h:]
        order = torch.randperm(pages, generator=g, device=dev)
        at = torch.arange(t, device=dev)
        s["slots"] = order[at // case["page"]] * case["page"] + at % case["page"]
        q8 = case["cache"] == "s8"
        cache_type = torch.int8 if q8 else torch.bfloat16
        s["k_cache"], s["v_cache"] = (_empty_cache(case, pages, cache_type, 0) for _ in range(2))
        shape = (pages, h, case["page"])
        s["k_scale"], s["v_scale"] = (torch.zeros(shape, device=dev) if q8 else None for _ in range(2))
        s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        return s
    ctx, new = _lengths(case)
    r, page, tokens = case["requests"], case["page"], sum(new)
    as_i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    s["ctx"], s["new"], s["cu"] = as_i32(ctx), as_i32(new), as_i32(_starts(new))
    s["tokens"], s["max_new"], s["max_ctx"] = tokens, max(new), max(ctx)
    s["words"] = -(-max(new) // 32) if case["tree"] else 0
    parents = _tree_parents(new, seed) if case["tree"] else None
    blocks = max(-(-(c + n) // page) for c, n in zip(ctx, new))
    need = sum(-(-(c + n) // page) for c, n in zip(ctx, new))
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    pages = need + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    if case["op"] == "plan":
        held = [-(-c // page) for c in ctx]
        table = torch.full((r, blocks), -1, dtype=torch.int32)
        host, at = order.cpu(), 0
        for i, n in enumerate(held):
            table[i, :n] = host[at:at + n]
            at += n
        s["table"], s["free"] = table.to(dev), order[at:].contiguous()
        s["parents"] = parents.to(dev) if parents is not None else None
        # a server keeps these from step to step
        s["cu_new"] = torch.empty(r + 1, dtype=torch.int32, device=dev)
        s["slots"] = torch.empty(tokens, dtype=torch.int64, device=dev)
        s["positions"] = torch.empty(tokens, dtype=torch.int32, device=dev)
        s["mask"] = torch.empty((tokens, s["words"]), dtype=torch.int32, device=dev) if case["tree"] else None
        s["taken"] = torch.empty(1, dtype=torch.int32, device=dev)
        return s
    h, kv = case["heads"], case["kv_heads"]
    starts, table = 0, torch.zeros((r, blocks), dtype=torch.int32)
    host = order.cpu()
    for i, (c, n) in enumerate(zip(ctx, new)):
        m = -(-(c + n) // page)
        table[i, :m] = host[starts:starts + m]
        starts += m
    s["table"] = table.to(dev)
    s["q"] = torch.randn((tokens, h, HEAD_DIM), generator=g, device=dev).to(torch.bfloat16)
    s["mask"] = _masks(parents, new, s["words"]).to(dev) if case["tree"] else None
    s["k_scale"] = s["v_scale"] = None
    if case["cache"] == "s8":
        s["k_cache"], s["v_cache"] = (_empty_cache(case, pages, torch.int8, 0) for _ in range(2))
        for c in (s["k_cache"], s["v_cache"]):
            c.copy_(torch.randint(-127, 128, c.shape, generator=g, device=dev, dtype=torch.int8))
        # codes spread evenly over +-127 are 73 rms: scales that make rows of about unit rms
        s["k_scale"], s["v_scale"] = (torch.exp(0.3 * torch.randn((pages, kv, page), generator=g, device=dev)) / 73.0
                                      for _ in range(2))
    else:
        s["k_cache"], s["v_cache"] = (_empty_cache(case, pages, torch.bfloat16, 0.0) for _ in range(2))
        for c in (s["k_cache"], s["v_cache"]):
            c.copy_(torch.randn(c.shape, generator=g, device=dev, dtype=torch.bfloat16))
    s["out"] = torch.empty((tokens, h, HEAD_DIM), dtype=torch.bfloat16, device=dev)
    s["scale"] = 1.0 / math.sqrt(HEAD_DIM)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _cached_values(s):
    """The cache's rows as the values they stand for."""
    if s["k_scale"] is None:
        return s["k_cache"], s["v_cache"]
    return [c.float() * sc.permute(0, 2, 1)[..., None] for c, sc in
            ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]))]


def _own(s):
    import quantized_matmul_qmm_gb300.qmm as qmm
    case = s["case"]
    if s["op"] == "plan":
        qmm.kv_plan(s["ctx"], s["new"], s["free"], s["table"], case["page"], s["slots"], s["positions"],
                    cu_new=s["cu_new"], pages_taken=s["taken"], parents=s["parents"], mask=s["mask"],
                    dev_status=s["status"])
        return {"table": s["table"], "cu_new": s["cu_new"], "slots": s["slots"], "positions": s["positions"],
                "mask": s["mask"], "taken": s["taken"]}
    if s["op"] == "append":
        qmm.kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
                      v_scale=s["v_scale"], dev_status=s["status"])
        return _cached_values(s)
    if "workspace" not in s:   # scratch that a server keeps from step to step
        n = qmm.tree_attention_workspace_size(s["q"].shape[1], case["kv_heads"], HEAD_DIM, s["max_new"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return qmm.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["cu"], s["max_new"],
                              mask=s["mask"], scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                              out=s["out"], workspace=s["workspace"], dev_status=s["status"])


def _plan(s):
    page, tokens = s["case"]["page"], s["tokens"]
    ctx, new = s["ctx"].long(), s["new"].long()
    have, need = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    cu = torch.cat([ctx.new_zeros(1), torch.cumsum(new, 0)])
    ends = torch.cumsum(need - have, 0)
    base = ends - (need - have)
    col = torch.arange(s["table"].shape[1], device=ctx.device)[None, :]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    pick = torch.clamp(base[:, None] + col - have[:, None], 0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][pick], s["table"])
    at = torch.arange(tokens, device=ctx.device)
    req = torch.searchsorted(cu, at, right=True) - 1
    i = at - cu[req]
    p = ctx[req] + i
    slots = table[req, p // page].long() * page + p % page
    mask, depth = None, i
    if s["parents"] is not None:
        # each token's set of ancestors doubles its reach with every step
        words, up = s["words"], s["parents"].long()
        bits = torch.arange(32 * words, device=ctx.device)[None, :] == i[:, None]
        jump = torch.where(up >= 0, up + cu[req], tokens)   # `tokens`: above a root, an empty row
        bits = torch.cat([bits, bits.new_zeros((1, 32 * words))])
        jump = torch.cat([jump, jump.new_full((1,), tokens)])
        for _ in range(max(1, (s["max_new"] - 1).bit_length())):
            bits = bits | bits[jump]
            jump = jump[jump]
        depth = bits[:tokens].sum(1) - 1
        weight = torch.tensor([1 << b for b in range(31)] + [-2 ** 31], device=ctx.device)
        mask = (bits[:tokens].view(tokens, words, 32) * weight).sum(2).to(torch.int32)
    return {"table": table, "cu_new": cu.to(torch.int32), "slots": slots,
            "positions": (ctx[req] + depth).to(torch.int32), "mask": mask, "taken": ends[-1:].to(torch.int32)}


def _append(s):
    page = s["case"]["page"]
    pg, off = s["slots"] // page, s["slots"] % page
    if s["k_scale"] is None:
        s["k_cache"][pg, off] = s["k"].float().to(torch.bfloat16)
        s["v_cache"][pg, off] = s["v"].float().to(torch.bfloat16)
        return _cached_values(s)
    rows = torch.stack([s["k"], s["v"]]).float()
    amax = rows.abs().amax(-1)
    scale = amax / torch.full_like(amax, 127.0)   # a true division, not a product with 1 / 127
    codes = torch.where(scale[..., None] > 0, torch.clamp(torch.round(rows / scale[..., None]), -127, 127), 0.0)
    s["k_cache"][pg, off], s["v_cache"][pg, off] = codes.to(torch.int8).unbind(0)
    s["k_scale"].permute(0, 2, 1)[pg, off], s["v_scale"].permute(0, 2, 1)[pg, off] = scale.unbind(0)
    return _cached_values(s)


def _attend(s, dtype=torch.float32):
    case = s["case"]
    page, h, kv = case["page"], case["heads"], case["kv_heads"]
    r, n, length = case["requests"], s["max_new"], s["max_ctx"] + s["max_new"]
    dev = s["q"].device
    ctx, cu = s["ctx"].long(), s["cu"].long()
    j = torch.arange(length, device=dev)
    blk = torch.clamp(j // page, max=s["table"].shape[1] - 1)
    pg = s["table"].long()[:, blk]                                        # [r][length]
    off = (j % page).expand(r, length)
    k, v = s["k_cache"][pg, off].to(dtype), s["v_cache"][pg, off].to(dtype)   # [r][length][kv][d]
    if s["k_scale"] is not None:
        k = k * s["k_scale"].permute(0, 2, 1)[pg, off].to(dtype)[..., None]
        v = v * s["v_scale"].permute(0, 2, 1)[pg, off].to(dtype)[..., None]
    i = torch.arange(n, device=dev)
    new = cu[1:] - cu[:-1]
    tok = torch.clamp(cu[:-1, None] + i[None, :], max=s["tokens"] - 1)    # [r][n]
    q = s["q"][tok].to(dtype).view(r, n, kv, h // kv, HEAD_DIM).permute(0, 2, 3, 1, 4).reshape(r, kv, -1, HEAD_DIM)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]           # [r][kv][group * n][length]
    node = j[None, :] - ctx[:, None]                                      # place among the new tokens
    if s["mask"] is None:
        seen = node[:, None, :] <= i[None, :, None]
    else:
        at = torch.clamp(node, 0, 32 * s["words"] - 1)[:, None, :].expand(r, n, length)
        word = torch.gather(s["mask"][tok].long() & 0xFFFFFFFF, 2, at // 32)
        seen = (node < 0)[:, None, :] | (((word >> (at % 32)) & 1) > 0)
    seen = seen & (node < new[:, None])[:, None, :]
    seen = seen[:, None, None].expand(r, 1, h // kv, n, length).reshape(r, 1, -1, length)
    score = score.masked_fill_(~seen, -math.inf)
    top = torch.clamp(score.amax(-1, keepdim=True), min=-1e30)
    p = torch.exp_(score.sub_(top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    o = o.view(r, kv, h // kv, n, HEAD_DIM).permute(0, 3, 1, 2, 4).reshape(r * n, h, HEAD_DIM)
    keep = torch.searchsorted(cu, torch.arange(s["tokens"], device=dev), right=True) - 1
    return o[keep * n + torch.arange(s["tokens"], device=dev) - cu[keep]]


def run(state):
    if own:
        return _own(state)
    if state["op"] == "plan":
        return _plan(state)
    if state["op"] == "append":
        return _append(state)
    return _attend(state).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                                # whole numbers only
    if case["op"] == "append":
        page, out = case["page"], []
        for rows, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
            x = rows.double()
            if case["cache"] == "s8":              # the nearest of 255 evenly spaced values to each
                step = (x.abs().amax(-1, keepdim=True) / 127.0).float().double()
                x = torch.where(step > 0, torch.round(x / step).clamp(-127, 127) * step, 0.0)
            full = torch.zeros(cache.shape, dtype=torch.float64, device="cuda")
            full.view(-1, *full.shape[2:])[s["slots"]] = x
            out.append(full)
        return out
    ctx, new = _lengths(case)
    group, page = case["heads"] // case["kv_heads"], case["page"]
    table, out = s["table"].long(), torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        at = torch.arange(c + n, device="cuda")
        pg, off = table[r, at // page], at % page
        seen = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        if case["tree"]:
            w = s["mask"][start:start + n].long()
            b = torch.arange(n, device="cuda")
            seen[:, c:] = ((w[:, b // 32] >> (b % 32)[None, :]) & 1) > 0
        else:
            seen[:, c:] = torch.tril(seen[:, c:])
        for h in range(case["kv_heads"]):
            k, v = s["k_cache"][pg, off, h].double(), s["v_cache"][pg, off, h].double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][pg, h, off].double()[:, None], v * s["v_scale"][pg, h, off].double()[:, None]
            for e in range(h * group, (h + 1) * group):
                x = (s["q"][start:start + n, e].double() @ k.T) / math.sqrt(HEAD_DIM)
                x = x.masked_fill(~seen, -math.inf)
                x = torch.exp(x - x.amax(-1, keepdim=True))
                out[start:start + n, e] = (x @ v) / x.sum(-1, keepdim=True)
        start += n
    return out
