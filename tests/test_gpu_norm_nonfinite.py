"""Infinities and NaN in single weights and gates: the other values of a row are what
the formula gives, wherever the row ends in its block's threads."""
import pytest
import torch

pytestmark = pytest.mark.gpu
INF = float("inf")

# few rows, rows of one warp, rows of several that come ahead, many short rows; ends inside a warp and at one
ROWS = [(3, 132), (3, 128), (2, 1000), (1, 4100), (3000, 132), (5000, 260), (2000, 1000), (1500, 4100), (700, 5000),
        (33000, 516), (4, 8200), (400, 16388), (3, 131)]


def inputs(dev, T, D):
    g = torch.Generator(device=dev).manual_seed(T + D)
    r = lambda *s: torch.randn(s, generator=g, device=dev)
    return r(T, D), r(T, D), 1.0 + 0.1 * r(D)


@pytest.mark.parametrize("value", [INF, -INF, float("nan")])
@pytest.mark.parametrize("where", ["branch_weight", "gate"])
@pytest.mark.parametrize("T,D", ROWS)
def test_one_infinite_value(qmm, cuda, T, D, where, value):
    """The last channel's weight or gate is no number: the sum is one there alone; behind
    an rms norm an infinity makes the others zeros, a NaN all of them NaN."""
    res, branch, w = inputs(cuda, T, D)
    bad = w.clone()
    bad[-1] = value
    kw = dict(branch_norm="rms", branch_weight=bad if where == "branch_weight" else w,
              gate=bad if where == "gate" else None, residual_out=torch.empty_like(res))
    clean = qmm.block_norm(res, branch, branch_norm="rms", branch_weight=w, gate=w if where == "gate" else None,
                           residual_out=torch.empty_like(res), out=False)[0]
    total, out = qmm.block_norm(res, branch, norm="rms", weight=w, out_type="f32", **kw)
    assert torch.equal(total[:, :-1], clean[:, :-1])
    assert (torch.isnan(total[:, -1]) if value != value else torch.isinf(total[:, -1])).all()
    if value != value:
        assert torch.isnan(out).all()
    else:
        assert (out[:, :-1] == 0).all() and torch.isnan(out[:, -1]).all()


@pytest.mark.parametrize("T,D", ROWS)
def test_the_norm_before_the_projection(qmm, cuda, T, D):
    """Weights and biases of the norm that ends the row."""
    res, branch, w = inputs(cuda, T, D)
    bad = w.clone()
    bad[-1] = INF
    clean = qmm.block_norm(res, branch, weight=w, out_type="f32", residual_out=torch.empty_like(res))[1]
    for kw in (dict(weight=bad), dict(weight=w, bias=torch.where(torch.isinf(bad), bad, 0.0))):
        out = qmm.block_norm(res, branch, out_type="f32", residual_out=torch.empty_like(res), **kw)[1]
        assert torch.equal(out[:, :-1], clean[:, :-1]) and torch.isinf(out[:, -1]).all()
