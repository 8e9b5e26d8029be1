"""Where fp32 ends: rows whose squares add up to more than it holds, and to less than its
smallest normal number."""
import numpy as np
import pytest
import torch

import oracle.beside_oracle as O

pytestmark = pytest.mark.gpu
MAX, TINY = float(np.finfo(np.float32).max), float(np.finfo(np.float32).tiny)
ROWS = [(3, 64), (2, 4096), (3000, 1000), (700, 5000), (2, 1001), (1500, 1001), (3, 20000)]


def row_of(dev, T, D, squares, kind, seed=1):
    """Rows of which the squares (of the values less their mean) add up to `squares`."""
    g = torch.Generator().manual_seed(seed + T + D)
    v = torch.randn((T, D), generator=g, dtype=torch.float64)
    if kind == "layer":
        v -= v.mean(1, keepdim=True)
    v *= (squares / (v * v).sum(1, keepdim=True)).sqrt()
    return v.float().to(dev)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("T,D", ROWS)
def test_the_largest_rows(qmm, cuda, T, D, kind):
    """Up to the largest sum of squares a norm is one; beyond it is zeros and the bias."""
    w, b = 1.0 + 0.1 * torch.randn(D, device=cuda), torch.randn(D, device=cuda)
    n = lambda t: t.double().cpu().numpy()
    v = row_of(cuda, T, D, 0.99 * MAX, kind)
    out = n(qmm.block_norm(v, norm=kind, weight=w, bias=b, out_type="f32")[1])
    want = O.norm(n(v), kind, n(w), n(b), 1e-6)
    assert (np.abs(out - want) <= O.norm_bound(n(v), 0.0, kind, n(w), n(b), 1e-6) + O.U32 * np.abs(want)).all()
    v = row_of(cuda, T, D, 1.02 * MAX, kind)
    out = qmm.block_norm(v, norm=kind, weight=w, bias=b, out_type="f32")[1]
    assert torch.equal(out, b.expand(T, D))
    # the same of the norm behind the branch
    total = qmm.block_norm(torch.ones_like(v), v, branch_norm=kind, branch_weight=w, branch_bias=b, out=False)[0]
    assert torch.equal(total, 1.0 + b.expand(T, D))


@pytest.mark.parametrize("T,D", ROWS)
def test_the_smallest_rows(qmm, cuda, T, D):
    """Without eps a norm is one down to squares that are normal numbers."""
    n = lambda t: t.double().cpu().numpy()
    g = torch.Generator().manual_seed(T + D)
    v = (torch.where(torch.rand((T, D), generator=g) < 0.5, -1.0, 1.0) * (1.0 + torch.rand((T, D), generator=g))
         * TINY ** 0.5).to(cuda)
    out = n(qmm.block_norm(v, eps=0.0, out_type="f32")[1])
    want = O.norm(n(v), "rms", None, None, 0.0)
    assert (np.abs(out - want) <= O.norm_bound(n(v), 0.0, "rms", None, None, 0.0) + O.U32 * np.abs(want)).all()
