"""Plain CPU implementation of the paged key/value cache (test infrastructure):
the plan of a step in Python integers, the append by the activation
quantiser's oracle, and tree attention in fp64 numpy.  It shares no code with
the CUDA library."""
from __future__ import annotations

import numpy as np

import oracle.qmm_oracle as O


def plan(ctx, new, free, table, page_size, capacity, parents=None, words=0):
    """The step's results as the C entry point documents them, for valid
    inputs: dict of table, cu_new, slots, positions, mask, taken."""
    table = np.array(table, dtype=np.int64)
    slots = np.full(capacity, -1, np.int64)
    positions = np.zeros(capacity, np.int64)
    mask = np.zeros((capacity, words), np.int64)
    cu, taken = [0], 0
    for r, (L, n) in enumerate(zip(ctx, new)):
        for col in range(-(-L // page_size), -(-(L + n) // page_size)):
            table[r, col] = free[taken]
            taken += 1
        rows = []
        for i in range(n):
            t = cu[-1] + i
            j = L + i
            slots[t] = table[r, j // page_size] * page_size + j % page_size
            depth = i
            if parents is not None:
                up = parents[t]
                rows.append((rows[up] if up >= 0 else set()) | {i})
                depth = len(rows[i]) - 1
                for a in rows[i]:
                    mask[t, a // 32] |= 1 << (a % 32)
            positions[t] = L + depth
        cu.append(cu[-1] + n)
    return {"table": table, "cu_new": np.array(cu), "slots": slots, "positions": positions, "mask": mask,
            "taken": taken}


def append_s8(x):
    """int8 codes and scales of fp32 rows [T][H][D]: (codes, scales [T][H])."""
    t, h, d = x.shape
    q, s = O.quantize_activations_f32(x.reshape(t * h, d), True)
    return q.reshape(t, h, d), s.reshape(t, h)


def visible(L, n, mask=None):
    """bool [n][L + n]; mask: int words [n][W] or None for a chain."""
    seen = np.ones((n, L + n), bool)
    for i in range(n):
        for j in range(n):
            seen[i, L + j] = j <= i if mask is None else bool((int(mask[i][j // 32]) >> (j % 32)) & 1)
    return seen


def attend(q, k, v, seen, scale):
    """q [n][Hq][D], k and v [len][H][D], seen [n][len]: (out, weight) with
    out = sum_j p_j v_j and weight = sum_j p_j |v_j| (what rounding errors of
    the p_j scale with), in fp64.  Hidden tokens are left out of the sums, not
    multiplied by zero."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    out, weight = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    with np.errstate(all="ignore"):
        for i in range(n):
            at = np.flatnonzero(seen[i])
            if not len(at):
                continue
            for h in range(hq):
                s = k[at, h // group].astype(np.float64) @ q[i, h].astype(np.float64) * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                vv = v[at, h // group].astype(np.float64)
                out[i, h] = p @ vv
                weight[i, h] = p @ np.abs(vv)
    return out, weight
