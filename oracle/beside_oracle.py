"""Plain CPU implementation of what runs beside the projections (test
infrastructure): block norms, low-rank adapters and token log probabilities in
fp64 numpy, with bounds on the error that fp32 arithmetic may add.  It shares no
code with the CUDA library."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24                      # half a step of fp32, relative
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step of a type, relative


def norm(v, kind, weight=None, bias=None, eps=0.0):
    """Rows of v normalised, in fp64."""
    v = np.asarray(v, np.float64)
    if kind == "layer":
        v = v - v.mean(-1, keepdims=True)
    z = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    if weight is not None:
        z = z * weight
    return z if bias is None else z + bias


def norm_bound(v, dv, kind, weight, bias, eps):
    """How far a norm of rows v, each value dv off, may be from the exact one.
    The sums of a row are trees of at most 64 roundings (32 values of a thread in
    turn, two shuffles of five steps, a division and what rounds each term), so a
    mean is within 64 U32 of the mean of magnitudes and a mean square within 64
    U32 of itself, its root within half of that; rsqrt is within 2 steps.  The
    norm's derivative is (d - z mean(z d)) / rms."""
    v = np.asarray(v, np.float64)
    dv = np.broadcast_to(dv, v.shape)
    if kind == "layer":
        dv = dv + dv.mean(-1, keepdims=True) + 64 * U32 * np.abs(v).mean(-1, keepdims=True) + U32 * np.abs(v)
        v = v - v.mean(-1, keepdims=True)
    rms = np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    z = np.abs(v / rms)
    w = 1.0 if weight is None else np.abs(weight)
    d = (dv + z * np.sqrt((dv * dv).mean(-1, keepdims=True))) / rms
    out = w * (d + z * (32 + 4 + 4) * U32)
    return out if bias is None else out + U32 * (np.abs(bias) + w * z)


def block(residual, branch, branch_norm, branch_weight, branch_bias, branch_eps, gate, scale, kind, weight, bias, eps):
    """(sum, bound, out, bound): exact values, and how far fp32 arithmetic may
    be from them before the rounding to the output type."""
    total, d = np.asarray(residual, np.float64), 0.0
    if branch is not None:
        u, du = np.asarray(branch, np.float64), 0.0
        if branch_norm is not None:
            du = norm_bound(u, 0.0, branch_norm, branch_weight, branch_bias, branch_eps)
            u = norm(u, branch_norm, branch_weight, branch_bias, branch_eps)
        g = 1.0 if gate is None else np.asarray(gate, np.float64)
        total = total + scale * g * u
        d = abs(scale) * np.abs(g) * (du + 2 * U32 * np.abs(u)) + U32 * np.abs(total)
    d = np.broadcast_to(d, total.shape)
    if kind is None:
        return total, d, total, d
    return total, d, norm(total, kind, weight, bias, eps), norm_bound(total, d, kind, weight, bias, eps)


def lora(X, ids, A, B, base, ranks, scales):
    """(out, bound) in fp64.  The first product: exact terms, at most K/16 + 8
    additions of an accumulator that may truncate (2 U32 of the sum of magnitudes
    each).  The second: the inner sums as two bf16 terms (2^-16), at most
    2 * 16 + 8 additions; then base."""
    X, A, B = (np.asarray(t, np.float64) for t in (X, A, B))
    M, K = X.shape
    n_adapters, max_rank, _ = A.shape
    out = np.zeros((M, B.shape[1])) if base is None else np.array(base, np.float64)
    bound = 2 * U32 * np.abs(out)
    for m in range(M):
        a = int(ids[m])
        r = max_rank if ranks is None else (int(ranks[a]) if 0 <= a < n_adapters else 0)
        if not 0 <= a < n_adapters or not 0 < r <= max_rank:
            continue
        s = 1.0 if scales is None else float(scales[a])
        h = A[a, :r] @ X[m]
        dh = (K / 16 + 8) * 2 * U32 * (np.abs(A[a, :r]) @ np.abs(X[m])) + 2.0 ** -16 * np.abs(h) + U32 * np.abs(h)
        add = s * (B[a, :, :r] @ h)
        size = abs(s) * (np.abs(B[a, :, :r]) @ np.abs(h))
        out[m] += add
        bound[m] += abs(s) * (np.abs(B[a, :, :r]) @ dh) + (2 * 16 + 8) * 2 * U32 * size + 2 * U32 * np.abs(out[m])
    return out, bound


def logprobs(x, tokens, k, scale):
    """Rows x (fp64 of the logits as stored): a dict of exact values and bounds.
    S = N + R: a term 2^t carries |t| * 3 U32 (two roundings of t, one of its
    factor) and the exponential's 4 U32; R is a sum of at most V / 512 + 64
    roundings in turn."""
    x = np.asarray(x, np.float64)
    M, V = x.shape
    G = tokens.shape[1] if tokens is not None else 0
    got = {"logprobs": np.full((M, G), np.nan), "entropy": np.full(M, np.nan), "ids": np.full((M, k), -1, np.int64),
           "top": np.full((M, k), np.nan)}
    tol = {"logprobs": np.zeros((M, G)), "entropy": np.zeros(M), "top": np.zeros((M, k))}
    for m in range(M):
        row = x[m]
        if np.isnan(row).any() or row.max() in (np.inf, -np.inf):
            continue
        t = (row - row.max()) * scale
        e = np.exp(t)
        N, R = float((t == 0).sum()), float(e[t < 0].sum())
        S = N + R
        log_s = np.log(N) + np.log1p(R / N)
        tf = np.where(e > 0, t, 0.0)
        spread = float((e * np.abs(tf)).sum())            # sum of |t| e
        rel = (4 + V / 512 + 64) * U32
        # a term below fp32's normal range is flushed: V of them are at most V 2^-126
        d_log = (rel * R + 3 * U32 * 1.4427 * spread) / S + 3 * U32 * log_s + V * 2.0 ** -126
        square = float((e * tf * tf).sum())
        got["entropy"][m] = log_s + spread / S
        tol["entropy"][m] = d_log + (rel * spread + 3 * U32 * 1.4427 * square + spread * d_log) / S \
            + 4 * U32 * got["entropy"][m]
        logp = t - log_s
        d_logp = d_log + 3 * U32 * np.abs(tf) + U32 * np.abs(np.where(np.isfinite(logp), logp, 0.0))
        for g in range(G):
            if 0 <= tokens[m, g] < V:
                got["logprobs"][m, g], tol["logprobs"][m, g] = logp[tokens[m, g]], d_logp[tokens[m, g]]
        if k:
            order = np.lexsort((np.arange(V), -row))[:k]  # falling value, then rising index
            order = order[row[order] > -np.inf]
            got["ids"][m, :len(order)] = order
            got["top"][m] = -np.inf
            got["top"][m, :len(order)] = logp[order]
            tol["top"][m, :len(order)] = d_logp[order]
    return got, tol
