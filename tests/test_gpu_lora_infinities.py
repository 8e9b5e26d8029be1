"""Infinities in an adapter's B: out is what the formula gives, an infinity of the sign of
the inner sum times B's, or NaN where that sum is zero or infinities of both signs meet."""
import numpy as np
import pytest
import torch

import oracle.beside_oracle as O

pytestmark = pytest.mark.gpu
INF = float("inf")


def case(dev, M, K, N, adapters, rank, seed=0):
    g = torch.Generator().manual_seed(seed + M + 7 * rank)
    r = lambda *s: torch.randn(s, generator=g)
    ids = torch.randint(-1, adapters, (M,), generator=g)
    ranks = torch.randint(1, rank + 1, (adapters,), generator=g)
    ranks[0] = rank
    X = r(M, K)
    A, B = r(adapters, rank, K) / K ** 0.5, r(adapters, N, -(-rank // 8) * 8)
    ids[:4] = 0
    X[1] = 0                                  # inner sums of zero: 0 times an infinity
    X[2] = 0
    X[2, 3] = 1.0                             # inner sums that are bf16 values: nothing is left for a second term
    B[0, 3, 0] = INF
    B[0, 4, rank - 1] = -INF
    B[0, N - 1, rank // 2] = INF
    if rank > 1:
        B[0, N // 2, 0], B[0, N // 2, rank - 1] = INF, -INF
    if adapters > 1:
        B[1, :, 0] = INF
    for a in range(adapters):                 # what lies behind a rank is never used
        A[a, int(ranks[a]):], B[a, :, int(ranks[a]):] = float("nan"), INF
    scales = 0.1 + r(adapters).abs()
    scales[0] = 1.0
    b16 = torch.bfloat16
    return dict(X=X.to(b16).to(dev), ids=ids.to(torch.int32).to(dev), A=A.to(b16).to(dev),
                B=B.to(b16).to(dev)[:, :, :rank], base=r(M, N).to(dev), ranks=ranks.to(torch.int32).to(dev), scales=scales.to(dev))


def exact(a):
    """(out, bound): the formula in fp64, term by term; the oracle's bound where B is finite."""
    f = lambda t: t.double().cpu().numpy()
    X, A, B, base, scales = (f(a[k]) for k in ("X", "A", "B", "base", "scales"))
    ids, ranks = a["ids"].cpu().numpy(), a["ranks"].cpu().numpy()
    _, bound = O.lora(X, ids, np.nan_to_num(A), np.where(np.isfinite(B), B, 0.0), base, ranks, scales)
    out = base.copy()
    with np.errstate(invalid="ignore"):
        for m, i in enumerate(ids):
            if i >= 0:
                r = ranks[i]
                out[m] += (B[i, :, :r] * (scales[i] * (A[i, :r] @ X[m]))).sum(1)
    return out, bound


# few rows with ranks of each form, and rows routed to tiles of 128 with partly filled and full ones
@pytest.mark.parametrize("M,K,N,adapters,rank", [
    (5, 64, 48, 1, 1), (5, 64, 48, 2, 8), (40, 264, 100, 3, 24), (30, 128, 131, 3, 50), (60, 512, 260, 2, 100),
    (20, 96, 75, 2, 201), (300, 64, 257, 5, 16), (2000, 64, 48, 3, 8), (1600, 264, 131, 2, 40),
    (1700, 128, 300, 4, 150), (1540, 72, 129, 30, 17)])
@pytest.mark.parametrize("inplace", [False, True])
def test_infinities_in_b(qmm, cuda, M, K, N, adapters, rank, inplace):
    a = case(cuda, M, K, N, adapters, rank)
    want, bound = exact(a)
    assert np.isinf(want).any() and np.isnan(want).any()
    got = qmm.lora_add(**a, out=a["base"] if inplace else None).double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), np.argwhere(np.isnan(got) != np.isnan(want))[:8]
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(got), inf) and np.array_equal(got[inf], want[inf])
    fine = np.isfinite(want)
    assert (np.abs(got[fine] - want[fine]) <= bound[fine]).all()


@pytest.mark.parametrize("M", [6, 2000])
def test_infinities_in_both(qmm, cuda, M):
    a = case(cuda, M, 64, 48, 2, 8, seed=5)
    a["A"].nan_to_num_()
    a["X"][0, 5], a["X"][3, 9] = INF, float("nan")
    with np.errstate(invalid="ignore"):
        want, _ = exact(a)
    got = qmm.lora_add(**a).double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    assert np.array_equal(np.sign(got[np.isinf(want)]), np.sign(want[np.isinf(want)]))


@pytest.mark.parametrize("M", [6, 2000])
def test_inner_sums_next_to_the_largest_number(qmm, cuda, M):
    """Inner sums that are finite but above bf16's largest value: finite products, and
    zeros beside B's zeros."""
    K, N, rank = 64, 48, 3
    A = torch.zeros((1, rank, K))
    A[0, :, 0], A[0, :, 1] = (2.0 - 2.0 ** -7) * 2.0 ** 127, 2.0 ** 119   # half a step beyond it
    A[0, 1] *= -1.0
    B = torch.zeros((1, N, 8))
    B[0, ::2, 0], B[0, ::3, 1] = 2.0 ** -100, 2.0 ** -101
    X = torch.zeros((M, K))
    X[:, :2] = 1.0
    X[1, 1] = 0.0                                            # bf16's largest value itself
    b16 = torch.bfloat16
    got = qmm.lora_add(X.to(b16).to(cuda), torch.zeros(M, dtype=torch.int32, device=cuda), A.to(b16).to(cuda),
                       B.to(b16).to(cuda)[:, :, :rank])
    want = (X.double() @ A[0].double().t()) @ B[0, :, :rank].double().t()
    assert torch.isfinite(got).all() and (got.cpu()[want == 0] == 0).all()
    assert ((got.double().cpu() - want).abs() <= (2.0 ** -16 + 100 * O.U32) * 2 * want.abs().max()).all()
