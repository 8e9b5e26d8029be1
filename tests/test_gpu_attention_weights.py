"""Which calls of qmm_tree_attention multiply the values by weights of two bf16
terms: requests of up to 64 query rows per key head in calls of up to 128, and
pages that are no multiple of 8 (the row kernel) whatever the rows.

Bound (test_gpu_attention.py has its parts): with A = sum_j p_j |v_j|,
|out - o| <= (2^-11 + 2^-13) A + 2^-8 (1 + 2^-10) |o| with two terms, and with
weights rounded once 2^-8 (1 + 2^-8) A more.  Few tokens are seen, so that the
roundings of single weights do not average out; each test shows that weights of
one term would miss the first bound on the same numbers.
"""
import numpy as np
import pytest
import torch

import oracle.kv_oracle as KV
from test_gpu_attention import build, call

pytestmark = pytest.mark.gpu


def bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def one_term(q, k, v, seen, scale):
    """Attention whose weights, against the row's maximum, are rounded to bf16 once."""
    group = q.shape[1] // k.shape[1]
    out = np.zeros(q.shape)
    for i in range(q.shape[0]):
        at = np.flatnonzero(seen[i])
        for h in range(q.shape[1]):
            s = k[at, h // group] @ q[i, h] * scale
            p = np.exp(s - s.max())
            out[i, h] = bf16(p) @ v[at, h // group] / p.sum()
    return out


@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctx,new,heads,page", [
    ([0, 3, 5, 1], [9, 16, 13, 11], 8, 16),       # 36 to 64 rows
    ([2, 0, 3, 1], [32, 16, 1, 9], 8, 16),        # one request of 128 rows beside smaller ones
    ([1, 2], [17, 16], 8, 64),                    # 68 rows and 64
    ([0, 2, 1], [40, 9, 1], 8, 20),               # pages for the row kernel
    ([0, 4], [8, 4], 8, 16),                      # 32 rows and 16
    ([0, 4], [4, 1], 8, 16),                      # the row kernel by the rows
])
def test_two_terms(qmm, cuda, ctx, new, heads, page, d, s8):
    kv = 2
    s = build(cuda, ctx, new, heads, kv, d, page, s8, tree=True, seed=sum(new) + d)
    out = call(qmm, cuda, s).double().cpu().numpy()
    q = s["q"].to(torch.bfloat16).double().numpy()
    apart = False
    for (c, n, first), (k, v, _, _) in zip(s["lens"], s["rows"]):
        m = [[int(w) & 0xFFFFFFFF for w in row] for row in s["mask"][first:first + n]]
        seen, qr, k, v = KV.visible(c, n, m), q[first:first + n], k.numpy(), v.numpy()
        ref, weight = KV.attend(qr, k, v, seen, s["scale"])
        tight = (2 ** -11 + 2 ** -13) * weight + 2 ** -8 * (1 + 2 ** -10) * np.abs(ref) + 1e-37
        rows = heads // kv
        two = page % 8 != 0 or (n * rows <= 64 and max(new) * rows <= 128)
        tol = tight if two else tight + 2 ** -8 * (1 + 2 ** -8) * weight
        err = np.abs(out[first:first + n] - ref)
        assert (err <= tol).all(), (c, n, (err - tol).max())
        apart |= two and (np.abs(bf16(one_term(qr, k, v, seen, s["scale"])) - ref) > tight).any()
    assert apart


@pytest.mark.parametrize("new,heads,page", [(6, 4, 16), (12, 8, 16), (20, 8, 16), (50, 16, 16), (20, 8, 20)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("place", ["cached", "new"])
@pytest.mark.parametrize("s8", [False, True])
def test_nonfinite_rows_that_are_seen(qmm, cuda, s8, place, side, bad, new, heads, page):
    """A row of the cache that is not finite makes exactly those outputs non-finite
    that the formula does: of the rows that see it, all elements (a key's NaN or
    +inf score), or the value's own."""
    if s8 and side == "k" and bad == bad:
        pytest.skip("an infinite key scale: codes of 0 decide, which the scores' sum does not see")
    s = build(cuda, [150], [new], heads, 2, 128, page, s8, tree=True, seed=2)
    s["mask"][:] &= ~8
    s["mask"][3] |= 8
    s["mask"][5] |= 8                             # of the new tokens rows 3 and 5 see token 3
    k, v, pg, off = s["rows"][0]
    x, t = (k if side == "k" else v), 153 if place == "new" else 77
    if s8:
        s["ks" if side == "k" else "vs"][pg[t], :, off[t]] = bad
        x[t] = s[side][pg[t], off[t]].cpu().double() * bad
    else:
        s[side][pg[t], off[t], :, 7] = bad
        x[t, :, 7] = bad
    out = call(qmm, cuda, s).double().cpu().numpy()
    m = [[int(w) & 0xFFFFFFFF for w in row] for row in s["mask"]]
    with np.errstate(all="ignore"):
        ref, _ = KV.attend(s["q"].double().numpy(), k.numpy(), v.numpy(), KV.visible(150, new, m), s["scale"])
    assert np.array_equal(np.isfinite(out), np.isfinite(ref))
