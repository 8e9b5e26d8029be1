"""qmm_tree_attention at the largest lengths: token numbers just below 2^31, on a
block table whose entries all name one page (the page's 65536 places are the
cached tokens again and again).

Bound.  A block adds up some 2^31 / 152 tokens one step after another, in fp32.
Row kernel: steps of 64, of which a warp takes 16: 2^31 / 152 / 64 = 220,753
steps, in each of them two products onto the outputs and four additions to a
lane's sum.  Tile kernel: tiles of 128, two streams: 55,189 tiles, eight products
of 16 tokens each onto the outputs, 64 additions to a half of the sum.  Every
addition is off by one unit in the last place, 2^-23, at most (tensor cores cut
off): 883,012 of them for the sum (row kernel), 441,512 products and 3,532,096
additions (tile kernel).  Sums of rounded-to-nearest terms are off by half a
unit each and not all in one direction, but the bound does not count on it for
the products: with A = sum_j p_j |v_j|, the outputs are within 441,512 * 2^-23 =
0.053 A; the sum's roundings to nearest, independent of each other, within
8 * 2^-24 * sqrt(3,532,096) < 0.001 of itself; a score, a weight and the output
add less than 2^-7.  Together |out - o| <= 0.064 A.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

PAGE, D, MOST = 65536, 64, 2 ** 31 - 8193


def setup(dev, s8, new):
    g = torch.Generator(device=dev).manual_seed(new)
    if s8:
        k, v = (torch.randint(-127, 128, (1, PAGE, 1, D), generator=g, device=dev).to(torch.int8) for _ in range(2))
        scales = {n: torch.full((1, 1, PAGE), 1 / 73, device=dev) for n in ("k_scale", "v_scale")}
        kv = [x.double().cpu().numpy()[0, :, 0] * float(np.float32(1 / 73)) for x in (k, v)]
    else:
        k, v = (torch.randn((1, PAGE, 1, D), generator=g, device=dev).to(torch.bfloat16) for _ in range(2))
        scales = {}
        kv = [x.double().cpu().numpy()[0, :, 0] for x in (k, v)]
    table = torch.zeros((1, -(-2 ** 31 // PAGE)), dtype=torch.int32, device=dev)
    q = torch.randn((new, 1, D), generator=g, device=dev).to(torch.bfloat16)
    cu = torch.tensor([0, new], dtype=torch.int32, device=dev)
    return q, k, v, scales, table, cu, kv


def run(qmm, dev, s8, new, length):
    q, k, v, scales, table, cu, kv = setup(dev, s8, new)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out = torch.full((new, 1, D), 7.0, dtype=torch.bfloat16, device=dev)
    ctx = torch.tensor([length - new], dtype=torch.int32, device=dev)
    qmm.tree_attention(q, k, v, table, ctx, cu, new, out=out, dev_status=status, **scales)
    torch.cuda.synchronize()
    return status.item(), out, q, kv


@pytest.mark.parametrize("new", [1, 32])
@pytest.mark.parametrize("s8", [False, True])
def test_longest(qmm, cuda, s8, new):
    status, out, q, (k, v) = run(qmm, cuda, s8, new, MOST)
    assert status == 0
    q, out = q.double().cpu().numpy(), out.double().cpu().numpy()
    for i in range(new):
        seen = MOST - new + i + 1
        times = seen // PAGE + (np.arange(PAGE) < seen % PAGE)   # how often each place counts
        s = k @ q[i, 0] * D ** -0.5
        p = times * np.exp(s - s.max())
        p /= p.sum()
        assert (np.abs(out[i, 0] - p @ v) <= 0.064 * (p @ np.abs(v))).all()


@pytest.mark.parametrize("new", [1, 32])
@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("over", [1, 7000, 8192])
def test_longer_is_refused(qmm, cuda, over, s8, new):
    """Reported, and the rows left alone."""
    status, out, _, _ = run(qmm, cuda, s8, new, MOST + over)
    assert status == qmm.QMM_ERR_INVALID_ARG
    assert (out == 7).all()


@pytest.mark.parametrize("requests", [1, 40])
@pytest.mark.parametrize("page,heads,new", [(PAGE, 1024, 129), (PAGE - 1, 104, 20)])
def test_more_work_than_a_call_counts(qmm, cuda, page, heads, new, requests):
    """2^24 cached tiles of 128 tokens times 516 tiles of 256 rows, or 2^25 of 64
    times 65 of 32 rows (pages that TMA does not take): reported, nothing written,
    however many requests share the step."""
    length = MOST - 1000
    k = torch.zeros((1, page, 1, D), dtype=torch.bfloat16, device=cuda)
    q = torch.zeros((new, heads, D), dtype=torch.bfloat16, device=cuda)
    out = torch.full_like(q, 7.0)
    table = torch.zeros((requests, -(-length // page)), dtype=torch.int32, device=cuda)
    ctx = torch.full((requests,), length - new, dtype=torch.int32, device=cuda)
    cu = torch.full((requests + 1,), new, dtype=torch.int32, device=cuda)
    cu[0] = 0
    mask = torch.full((new, (new + 31) // 32), -1, dtype=torch.int32, device=cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    qmm.tree_attention(q, k, k, table, ctx, cu, new, mask=mask, out=out, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == qmm.QMM_ERR_INVALID_ARG
    assert (out == 7).all()
