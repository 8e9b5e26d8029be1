"""The steps on either side of a projection: cases, their plain forms and the
library's calls.

Three operators that chain with the quantised projections of a decoder:

* ``norm``: a block's output joined to the residual stream (normalised, gated
  and scaled where the model does that) and the next block's normalised input
  made from the sum, as bf16 rows or as int8 codes with a scale per row
  (``block_norm``);
* ``lora``: low-rank adapters of many requests added to a shared projection's
  output (``lora_add``);
* ``logprobs``: log probabilities of given tokens, the entropy and the top
  alternatives of rows of logits (``token_logprobs``).

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the library.
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # norm: one decoded token of eight requests at the 0.6B projections' width: latency alone
        dict(name="norm_decode_r8", op="norm", rows=8, dim=1024, kind="rms", residual="f32", branch="f32", post=False,
             gate="none", out="bf16", scale=1.0),
        # norm: a batch of prompts, a norm after the block as well as before the next, scaled residual
        dict(name="norm_prompt_post", op="norm", rows=16384, dim=4096, kind="rms", residual="f32", branch="f32",
             post=True, gate="none", out="bf16", scale=0.22),
        # norm: a learned gate per channel, int8 codes for the exact int8 GEMM of width 4608, an odd number of rows
        dict(name="norm_gate_int8", op="norm", rows=2049, dim=4608, kind="rms", residual="f32", branch="f32", post=True,
             gate="channel", out="s8", scale=1.0),
        # norm: layer norms of an odd width over a bf16 stream, a gate for every token and channel
        dict(name="norm_layer_odd", op="norm", rows=5000, dim=1001, kind="layer", residual="bf16", branch="bf16",
             post=False, gate="token", out="bf16", scale=1.0),
        # lora: eight requests decode one token each, small adapters, the 0.6B q projection: latency
        dict(name="lora_decode_r8", op="lora", rows=8, k=1024, n=2048, adapters=5, rank_lo=16, rank_hi=16, prompt=False),
        # lora: a full decoding batch over many adapters of uneven ranks
        dict(name="lora_decode_r256", op="lora", rows=256, k=4096, n=4096, adapters=40, rank_lo=5, rank_hi=64,
             prompt=False),
        # lora: prompts of several requests, contiguous rows of one adapter each
        dict(name="lora_prompt", op="lora", rows=4097, k=4608, n=4608, adapters=6, rank_lo=8, rank_hi=64, prompt=True),
        # lora: large ranks beside a wide projection
        dict(name="lora_prompt_wide", op="lora", rows=2048, k=2048, n=12288, adapters=3, rank_lo=100, rank_hi=256,
             prompt=True),
        # logprobs: one decoded token, 20 alternatives, the 0.6B lm_head's logits
        dict(name="logprobs_decode_r1", op="logprobs", rows=1, vocab=151936, pad=0, type="f32", tokens=1, top=20,
             masked=0.0, scale=1.0),
        # logprobs: the nodes of drafted trees, with several children to score, at a temperature
        dict(name="logprobs_verify_r64", op="logprobs", rows=64, vocab=151936, pad=0, type="f32", tokens=4, top=5,
             masked=0.0, scale=1.25),
        # logprobs: constrained decoding over an odd vocabulary in rows padded to the projection's tiles
        dict(name="logprobs_masked_odd", op="logprobs", rows=300, vocab=50257, pad=15, type="bf16", tokens=1, top=8,
             masked=0.97, scale=1.0),
        # logprobs: a prompt's tokens scored, a chunk of 1024 rows: the largest
        dict(name="logprobs_score_r1024", op="logprobs", rows=1024, vocab=151936, pad=0, type="f32", tokens=1, top=1,
             masked=0.0, scale=1.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "lora", "logprobs"])
    if op == "norm":
        dim = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            dim = max(64, dim // 64 * 64)
        rows = _log(rng, 1, min(16384, 2 ** 26 // dim))
        return dict(op=op, rows=rows, dim=dim, kind=rng.choice(["rms", "rms", "layer"]),
                    residual=rng.choice(["f32", "bf16"]), branch=rng.choice(["f32", "bf16"]),
                    post=rng.random() < 0.5, gate=rng.choice(["none", "channel", "token"]),
                    out=rng.choice(["bf16", "bf16", "s8", "f32"]), scale=rng.choice([1.0, 0.22]))
    if op == "lora":
        k, n = 8 * _log(rng, 32, 1024), _log(rng, 256, 12288)
        hi = _log(rng, 1, 256)
        adapters = _log(rng, 1, 64)
        prompt = rng.random() < 0.5
        rows = _log(rng, 1, min(8192 if prompt else 512, 4097 * 46080 // (2 * k + 8 * n)))
        return dict(op=op, rows=rows, k=k, n=n, adapters=adapters, rank_lo=max(1, hi // 4), rank_hi=hi, prompt=prompt)
    vocab = _log(rng, 1000, 160000)
    return dict(op=op, rows=_log(rng, 1, min(4096, 1024 * 151936 // vocab)), vocab=vocab, pad=rng.choice([0, 0, 7, 32]),
                type=rng.choice(["f32", "f32", "bf16"]), tokens=rng.choice([1, 1, 2, 8]),
                top=rng.choice([0, 1, 5, 20, 32]), masked=rng.choice([0.0, 0.0, 0.9]), scale=rng.choice([1.0, 1.25, 0.5]))


def _ranks(case):
    """Adapters' ranks over rank_lo..rank_hi, the largest first, in a scattered order."""
    lo, hi, n = case["rank_lo"], case["rank_hi"], case["adapters"]
    return [hi] + [lo + int((hi - lo + 0.999) * ((i * 0.6180339887) % 1.0)) for i in range(1, n)]


def _counts(case):
    """Rows of each adapter, and at the end of the list those without one."""
    m, n = case["rows"], case["adapters"]
    if case["prompt"]:                       # uneven prompts; the last few rows have none
        weight, have = [1.0 + 3.0 * ((i * 0.7548776662) % 1.0) for i in range(n)], m - m // 50
    else:                                    # a tenth of the requests have none
        weight, have = [1.0] * n, m - m // 10
    ends = [int(have * sum(weight[:i + 1]) / sum(weight) + 0.5) for i in range(n)]
    got = [e - b for b, e in zip([0] + ends, ends)]
    return got + [m - sum(got)]


def work(case):
    m = case["rows"]
    if case["op"] == "norm":
        d, size = case["dim"], {"f32": 4, "bf16": 2, "s8": 1}
        weights = (2 + (case["kind"] == "layer")) if case["post"] else (1 + (case["kind"] == "layer"))
        gate = {"none": 0, "channel": 4 * d, "token": 2 * d * m}[case["gate"]]
        row = 2 * size[case["residual"]] + size[case["branch"]] + size[case["out"]]
        return {"bytes": m * d * row + 4 * weights * d + gate + (4 * m if case["out"] == "s8" else 0),
                "flops": 12 * m * d}
    if case["op"] == "lora":
        k, n, counts, ranks = case["k"], case["n"], _counts(case), _ranks(case)
        used = [(c, r) for c, r in zip(counts, ranks) if c]
        return {"bytes": 2 * k * sum(c for c, _ in used) + 8 * m * n + sum(2 * r * (k + n) for _, r in used) + 4 * m,
                "flops": sum(2 * c * r * (k + n) for c, r in used)}
    v, g, top = case["vocab"], case["tokens"], case["top"]
    return {"bytes": m * (v * (4 if case["type"] == "f32" else 2) + 8 * g + 4 + 8 * top), "flops": 5 * m * v}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "s8": torch.int8}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    m, s = case["rows"], {"case": case}
    normal = lambda *shape: torch.randn(shape, generator=g, device=dev)
    if case["op"] == "norm":
        d = case["dim"]
        # a residual stream has a few channels far above the others
        loud = torch.where(torch.rand((1, d), generator=g, device=dev) < 0.01, 20.0, 1.0)
        s["residual"] = (normal(m, d) * loud + 0.1).to(_TYPES[case["residual"]])
        s["branch"] = (normal(m, d) * torch.exp(0.5 * normal(m, 1))).to(_TYPES[case["branch"]])
        s["weight"], s["post_weight"] = 1.0 + 0.2 * normal(d), 0.5 + 0.1 * normal(d)
        s["bias"] = s["post_bias"] = None
        if case["kind"] == "layer":
            s["bias"], s["post_bias"] = 0.1 * normal(d), 0.1 * normal(d)
        s["gate"] = None
        if case["gate"] == "channel":
            s["gate"] = 0.5 * normal(d)
        elif case["gate"] == "token":
            s["gate"] = torch.sigmoid(normal(m, d)).to(torch.bfloat16)
        s["sum"] = torch.empty_like(s["residual"])
        # the int8 GEMM takes rows of whole 16 bytes
        width = -(-d // 16) * 16 if case["out"] == "s8" else d
        s["x"] = torch.empty((m, width), dtype=_TYPES[case["out"]], device=dev)[:, :d]
        if case["out"] == "s8":
            s["s_x"] = torch.empty(m, device=dev)
            s["values"] = torch.empty((m, d), dtype=torch.bfloat16, device=dev)
        return s
    if case["op"] == "lora":
        k, n, a, r = case["k"], case["n"], case["adapters"], case["rank_hi"]
        ids = torch.repeat_interleave(torch.tensor(list(range(a)) + [-1], dtype=torch.int32),
                                      torch.tensor(_counts(case)))
        cpu = torch.Generator().manual_seed(int(seed))
        if not case["prompt"]:
            ids = ids[torch.randperm(m, generator=cpu)]
        s["ids"] = ids.to(dev)
        s["x"] = normal(m, k).to(torch.bfloat16)
        # what lies behind an adapter's rank in its slot is another adapter's old content
        s["a"] = (normal(a, r, k) / math.sqrt(k)).to(torch.bfloat16)
        s["b"] = (normal(a, n, -(-r // 8) * 8) * 0.05).to(torch.bfloat16)[:, :, :r]
        s["ranks"] = torch.tensor(_ranks(case), dtype=torch.int32, device=dev)
        s["scales"] = 16.0 / torch.clamp(s["ranks"].float(), min=8.0)
        s["base"] = normal(m, n)
        s["out"] = torch.empty_like(s["base"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        return s
    v, t = case["vocab"], case["tokens"]
    x = torch.empty((m, v + case["pad"]), dtype=_TYPES[case["type"]], device=dev)
    top = torch.randint(0, v, (m,), generator=g, device=dev)
    for lo in range(0, m, 256):              # by chunks: the fp32 draws of 1024 rows would be another gigabyte
        part = 2.5 * normal(min(256, m - lo), v + case["pad"])
        part[torch.arange(part.shape[0], device=dev), top[lo:lo + 256]] += 4.0 + 12.0 * torch.rand(
            part.shape[0], generator=g, device=dev)
        if case["masked"]:
            part.masked_fill_(torch.rand(part.shape, generator=g, device=dev) < case["masked"], -math.inf)
        x[lo:lo + 256] = part.to(x.dtype)
    s["logits"] = x[:, :v]
    tokens = torch.randint(0, v, (m, t), generator=g, device=dev)
    tokens[:, 0] = torch.where(torch.rand(m, generator=g, device=dev) < 0.7, top, tokens[:, 0])
    s["tokens"] = tokens.to(torch.int32)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _own(s):
    import quantized_matmul_qmm_gb300.qmm as qmm
    case = s["case"]
    if case["op"] == "norm":
        post = dict(branch_norm=case["kind"], branch_weight=s["post_weight"], branch_bias=s["post_bias"]) \
            if case["post"] else {}
        qmm.block_norm(s["residual"], s["branch"], norm=case["kind"], weight=s["weight"], bias=s["bias"], eps=EPS,
                       gate=s["gate"], scale=case["scale"], residual_out=s["sum"], out=s["x"], s_x=s.get("s_x"), **post)
        return {"sum": s["sum"], "x": _values(s, s["x"], s.get("s_x"))}
    if case["op"] == "lora":
        if "workspace" not in s:   # scratch that a server keeps from step to step
            size = qmm.lora_add_workspace_size(case["rows"], case["k"], case["n"], s["a"].shape[0], s["a"].shape[1])
            s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        return qmm.lora_add(s["x"], s["ids"], s["a"], s["b"], base=s["base"], out=s["out"], ranks=s["ranks"],
                            scales=s["scales"], workspace=s["workspace"], dev_status=s["status"])
    logprobs, entropy, top_ids, top_logprobs = qmm.token_logprobs(
        s["logits"], s["tokens"], top_k=case["top"], scale=case["scale"], dev_status=s["status"])
    return {"logprobs": logprobs, "entropy": entropy, "top_ids": top_ids, "top_logprobs": top_logprobs}


def _values(s, x, s_x):
    """int8 codes as the values they stand for."""
    return x if s_x is None else torch.mul(x, s_x[:, None], out=s["values"])


def _normed(v, kind, weight, bias):
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * weight
    return v if bias is None else v + bias


def _norm(s):
    case = s["case"]
    u = s["branch"].float()
    if case["post"]:
        u = _normed(u, case["kind"], s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        u = u * s["gate"].float()
    total = s["residual"].float() + case["scale"] * u
    x = _normed(total, case["kind"], s["weight"], s["bias"])
    s_x = None
    if case["out"] == "s8":
        amax = x.abs().amax(-1)
        s_x = amax / torch.full_like(amax, 127.0)
        x = torch.where(s_x[:, None] > 0, torch.clamp(torch.round(x / s_x[:, None]), -127, 127), 0.0)
    return {"sum": total.to(s["sum"].dtype), "x": _values(s, x.to(s["x"].dtype), s_x)}


def _lora(s):
    """All adapters' products for all rows; those of other adapters, and what
    lies behind an adapter's rank, are cleared between the two products."""
    a, b = s["a"].float(), s["b"].float()
    n_a, r, k = a.shape
    h = torch.matmul(s["x"].float(), a.reshape(n_a * r, k).t()).view(-1, n_a, r)
    keep = (s["ids"][:, None, None] == torch.arange(n_a, device=a.device)[None, :, None]) & (
        torch.arange(r, device=a.device)[None, None, :] < s["ranks"][None, :, None])
    h = torch.where(keep, h * s["scales"][None, :, None], 0.0)
    return s["base"] + torch.matmul(h.view(-1, n_a * r), b.permute(0, 2, 1).reshape(n_a * r, -1))


def _logprobs(s):
    """Sums and logarithms in 64 bits: a token that holds nearly all of a row has
    a log probability next to zero, which 1 + rest in 32 bits would round away."""
    case = s["case"]
    x = s["logits"].float()
    x = (x - x.amax(-1, keepdim=True)) * case["scale"]
    p = torch.exp(x)
    total = p.sum(-1, keepdim=True, dtype=torch.float64)
    x = x.double() - torch.log(total)
    entropy = -(torch.where(p > 0, p * x, 0.0).sum(-1) / total[:, 0]).float()
    del p
    x = x.float()
    logprobs = torch.gather(x, 1, s["tokens"].long())
    if case["top"] == 0:
        return {"logprobs": logprobs, "entropy": entropy, "top_ids": None, "top_logprobs": None}
    # a stable sort: equal values keep the order of their indexes
    value, at = torch.sort(s["logits"], dim=-1, descending=True, stable=True)
    at = at[:, :case["top"]]
    at = torch.where(value[:, :case["top"]] > -math.inf, at, -1)
    best = torch.where(at >= 0, torch.gather(x, 1, torch.clamp(at, min=0)), -math.inf)
    return {"logprobs": logprobs, "entropy": entropy, "top_ids": at.to(torch.int32), "top_logprobs": best}


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm, "lora": _lora, "logprobs": _logprobs}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _exact_norm(v, kind, weight, bias):
    centre = v.mean(1, keepdim=True) if kind == "layer" else 0.0
    length = torch.linalg.vector_norm(v - centre, dim=1, keepdim=True) ** 2 / v.shape[1]
    out = (v - centre) * weight.double() * (length + EPS) ** -0.5
    return out if bias is None else out + bias.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        total, x = [], []
        for rows in torch.arange(case["rows"], device="cuda").split(2048):
            u = s["branch"][rows].double()
            if case["post"]:
                u = _exact_norm(u, case["kind"], s["post_weight"], s["post_bias"])
            if case["gate"] == "channel":
                u = u * s["gate"].double()
            elif case["gate"] == "token":
                u = u * s["gate"][rows].double()
            total.append(s["residual"][rows].double() + case["scale"] * u)
            v = _exact_norm(total[-1], case["kind"], s["weight"], s["bias"])
            if case["out"] == "s8":          # the nearest of 255 evenly spaced values to each
                step = v.abs().amax(1, keepdim=True) / 127.0
                v = torch.where(step > 0, torch.round(v / step) * step, 0.0)
            x.append(v)
        return {"sum": torch.cat(total), "x": torch.cat(x)}
    if case["op"] == "lora":
        out = s["base"].double()
        for a, r in enumerate(_ranks(case)):
            rows = torch.nonzero(s["ids"] == a).flatten()
            if rows.numel():
                h = s["x"][rows].double() @ s["a"][a, :r].double().t()
                out[rows] += float(s["scales"][a]) * (h @ s["b"][a, :, :r].double().t())
        return out
    got = {"logprobs": [], "entropy": [], "top_ids": None, "top_logprobs": []}
    for rows in torch.arange(case["rows"], device="cuda").split(128):
        x = s["logits"][rows].double() * case["scale"]
        lse = torch.logsumexp(x, 1, keepdim=True)
        q = x - lse
        got["logprobs"].append(torch.gather(q, 1, s["tokens"][rows].long()))
        got["entropy"].append(torch.special.entr(torch.exp(q)).sum(1))
        best = torch.topk(q, min(case["top"], case["vocab"]), dim=1).values
        got["top_logprobs"].append(best)
    got = {k: torch.cat(v) if isinstance(v, list) else v for k, v in got.items()}
    if case["top"] == 0:
        got["top_logprobs"] = None
    return got
