"""GPU parity of the paged key/value cache (qmm_kv_plan, qmm_kv_append) against
the CPU oracle: whole numbers, codes, scales and bf16 roundings all equal."""
import numpy as np
import pytest
import torch

import oracle.kv_oracle as KV

pytestmark = pytest.mark.gpu


def draw_parents(g, new):
    out = []
    for n in new:
        for i in range(n):
            out.append(int(torch.randint(-1, i, (1,), generator=g)) if i and torch.rand(1, generator=g) < 0.9 else -1)
    return out


def run_plan(qmm, dev, ctx, new, page, capacity=None, parents=None, words=0, n_free=None, blocks=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    held = [-(-c // page) for c in ctx]
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    taken = sum(need) - sum(held)
    blocks = max(1, max(need)) if blocks is None else blocks
    pool = torch.randperm(sum(need) + 5, generator=g)
    table = torch.full((len(ctx), blocks + 3), -7, dtype=torch.int32)[:, :blocks]   # a strided view
    at = 0
    for r, n in enumerate(held):
        m = min(n, blocks)
        table[r, :m] = pool[at:at + m].to(torch.int32)
        at += n
    free = pool[at:].to(torch.int32)
    if n_free is not None:
        free = free[:n_free]
    tokens = sum(new)
    capacity = tokens if capacity is None else capacity
    dtab = torch.full((len(ctx), blocks + 3), -7, dtype=torch.int32, device=dev)[:, :blocks]
    dtab.copy_(table)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
    slots = torch.full((capacity,), 99, dtype=torch.int64, device=dev)
    positions = torch.full((capacity,), 99, dtype=torch.int32, device=dev)
    par = msk = None
    if parents is not None:
        par = torch.zeros(capacity, dtype=torch.int32)
        par[:min(tokens, capacity)] = torch.tensor(parents[:capacity], dtype=torch.int32)
        par = par.to(dev)
        msk = torch.full((capacity, words + 1), 99, dtype=torch.int32, device=dev)[:, :words]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    args = (i32(ctx), i32(new), free.to(dev), dtab, page, slots, positions)
    cu, tk = qmm.kv_plan(*args, parents=par, mask=msk, dev_status=status)
    first = [x.clone() for x in (dtab, cu, slots, positions, tk)]
    qmm.kv_plan(*args, parents=par, mask=msk, cu_new=cu, pages_taken=tk, dev_status=status)   # the same again
    torch.cuda.synchronize()
    for x, y in zip(first, (dtab, cu, slots, positions, tk)):
        assert torch.equal(x, y)
    got = {"table": dtab, "cu_new": cu, "slots": slots, "positions": positions, "taken": tk}
    got = {k: v.cpu().numpy().astype(np.int64) for k, v in got.items()}
    got["mask"] = np.zeros((capacity, 0), np.int64) if msk is None else msk.cpu().numpy().astype(np.int64) & 0xFFFFFFFF
    return got, int(status.item()), dict(table=table.numpy(), free=free.tolist(), taken=taken)


CASES = [
    # ctx, new, page
    ([0], [1], 16), ([15], [1], 16), ([16], [1], 16), ([17], [0], 16), ([0, 0, 0], [0, 0, 0], 4),
    ([5, 0, 31, 32, 33], [3, 0, 1, 1, 40], 16), ([100, 7, 0, 1], [1, 1, 1, 1], 1), ([3, 999], [130, 1], 7),
    ([0, 1, 2, 3], [513, 511, 1, 1200], 128),
]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("extra", [0, 5])
@pytest.mark.parametrize("ctx,new,page", CASES)
def test_plan(qmm, cuda, ctx, new, page, extra, tree):
    g = torch.Generator().manual_seed(len(ctx) + page)
    capacity = sum(new) + extra
    if capacity == 0 and tree:
        pytest.skip("no token, no tree")
    parents = draw_parents(g, new) if tree else None
    words = max(1, -(-max(new) // 32)) if tree else 0
    got, status, base = run_plan(qmm, cuda, ctx, new, page, capacity, parents, words)
    ref = KV.plan(ctx, new, base["free"], base["table"], page, capacity, parents, words)
    assert status == 0
    for k in ("table", "cu_new", "slots", "positions", "mask"):
        assert np.array_equal(got[k], ref[k]), k
    assert got["taken"][0] == ref["taken"] == base["taken"]


@pytest.mark.parametrize("R", [1, 31, 512, 513, 1500])
def test_plan_many_requests(qmm, cuda, R):
    g = torch.Generator().manual_seed(R)
    ctx = torch.randint(0, 200, (R,), generator=g).tolist()
    new = torch.randint(0, 40, (R,), generator=g).tolist()
    parents = draw_parents(g, new)
    got, status, base = run_plan(qmm, cuda, ctx, new, 16, None, parents, 2)
    ref = KV.plan(ctx, new, base["free"], base["table"], 16, sum(new), parents, 2)
    assert status == 0
    for k in ("table", "cu_new", "slots", "positions", "mask"):
        assert np.array_equal(got[k], ref[k]), k


def test_plan_chain_as_tree(qmm, cuda):
    """A tree without branches is the chain: every earlier token an ancestor."""
    n = 100
    got, status, _ = run_plan(qmm, cuda, [9], [n], 16, None, list(range(-1, n - 1)), 4)
    assert status == 0
    assert got["positions"].tolist() == list(range(9, 9 + n))
    for i in range(n):
        bits = sum(int(w) << (32 * k) for k, w in enumerate(got["mask"][i]))
        assert bits == (1 << (i + 1)) - 1


def test_plan_reports_what_does_not_fit(qmm, cuda):
    S = qmm
    # a free list one page short: the tokens of that page have no slot, all others do
    got, status, base = run_plan(qmm, cuda, [10, 10], [30, 30], 16, n_free=3)
    assert status == S.QMM_ERR_NO_PAGES and got["taken"][0] == base["taken"] == 4
    assert (got["slots"][:38] >= 0).all() or (got["slots"][:30] >= 0).all()
    assert (got["slots"][52:] == -1).all() and (got["slots"][30:52] >= 0).all()
    # a negative length: that request gets nothing, the others their slots
    got, status, _ = run_plan(qmm, cuda, [4, -1, 4], [2, 3, 2], 16, blocks=1, capacity=4)
    assert status == S.QMM_ERR_INVALID_ARG and got["cu_new"].tolist() == [0, 2, 2, 4] and (got["slots"] >= 0).all()
    # more tokens than rows; more pages than columns
    _, status, _ = run_plan(qmm, cuda, [4], [9], 16, capacity=8)
    assert status == S.QMM_ERR_INVALID_ARG
    got, status, _ = run_plan(qmm, cuda, [4], [60], 16, blocks=2)
    assert status == S.QMM_ERR_INVALID_ARG and (got["slots"][28:] == -1).all() and (got["slots"][:28] >= 0).all()
    # parents that are not earlier tokens, a token that the mask has no bit for
    for parents in ([-1, 1, 0], [0, 0, 0], [-1, -2, 0], [-1, 0, 5]):
        _, status, _ = run_plan(qmm, cuda, [4], [3], 16, parents=parents, words=1)
        assert status == S.QMM_ERR_INVALID_ARG, parents
    _, status, _ = run_plan(qmm, cuda, [4], [40], 16, parents=[-1] * 40, words=1)
    assert status == S.QMM_ERR_INVALID_ARG


def caches(dev, pages, page, heads, d, dtype, head_major, fill):
    if head_major:
        return [torch.full((pages, heads, page, d), fill, dtype=dtype, device=dev).permute(0, 2, 1, 3)
                for _ in range(2)]
    return [torch.full((pages, page, heads, d), fill, dtype=dtype, device=dev) for _ in range(2)]


@pytest.mark.parametrize("T,heads,page", [(1, 1, 1), (5, 3, 16), (70, 2, 7), (33, 8, 64)])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("rows", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_append(qmm, cuda, d, rows, s8, head_major, T, heads, page):
    g = torch.Generator().manual_seed(T * 100 + heads)
    pages = -(-T // page) + 2
    x = (torch.randn((T, 2 * heads, d), generator=g) * torch.exp(2 * torch.randn((T, 2 * heads, 1), generator=g)))
    x = x.to(rows)
    x[0, 0] = 0                                   # a zero row: scale 0, codes 0
    xd = x.to(cuda)                               # K and V are interleaved views of one buffer
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 2:
        slots[1] = -1
    kc, vc = caches(cuda, pages, page, heads, d, torch.int8 if s8 else torch.bfloat16, head_major, 77)
    ks = vs = None
    if s8:
        ks, vs = (torch.full((pages, heads, page), 55.0, device=cuda) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    qmm.kv_append(xd[:, 0::2], xd[:, 1::2], slots.to(cuda), kc, vc, k_scale=ks, v_scale=vs, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    for cache, scale, part in ((kc, ks, x[:, 0::2]), (vc, vs, x[:, 1::2])):
        want = torch.full((pages * page, heads, d), 77, dtype=cache.dtype)
        keep = slots >= 0
        if s8:
            q, sc = KV.append_s8(part.float().numpy())
            want[slots[keep]] = torch.from_numpy(q).to(torch.int8)[keep]
            wsc = torch.full((pages * page, heads), 55.0)
            wsc[slots[keep]] = torch.from_numpy(sc).float()[keep]
            assert torch.equal(scale.permute(0, 2, 1).reshape(-1, heads).cpu(), wsc)
        else:
            want[slots[keep]] = part.float().to(torch.bfloat16)[keep]
        assert torch.equal(cache.reshape(-1, heads, d).cpu(), want)


def test_append_ties_and_slot_out_of_range(qmm, cuda):
    x = torch.zeros((3, 1, 64))
    x[0, 0, :8] = torch.tensor([127.0, 2.5, 3.5, -2.5, 0.5, 1.5, -126.5, 126.5])
    x[1:] = 1.0
    kc, vc = caches(cuda, 2, 4, 1, 64, torch.int8, False, 9)
    ks, vs = (torch.full((2, 1, 4), 5.0, device=cuda) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    xd = x.to(cuda)
    qmm.kv_append(xd, xd, torch.tensor([3, 8, -2], device=cuda), kc, vc, k_scale=ks, v_scale=vs, dev_status=status)
    assert status.item() == qmm.QMM_ERR_INVALID_ARG
    assert kc[0, 3, 0, :8].tolist() == [127, 2, 4, -2, 0, 2, -126, 126] and ks[0, 0, 3] == 1
    assert (kc.reshape(8, 64)[[0, 1, 2, 4, 5, 6, 7]] == 9).all() and (ks.flatten()[[0, 1, 2, 4, 5, 6, 7]] == 5).all()


@pytest.mark.parametrize("rows", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("s8", [False, True])
def test_append_many_rows(qmm, cuda, s8, rows):
    """A long prompt: several (token, head) pairs per warp, the last warp short."""
    T, heads, d, page = 13007, 3, 64, 16
    g = torch.Generator().manual_seed(7)
    x = (torch.randn((T, heads, d), generator=g) * torch.exp(torch.randn((T, heads, 1), generator=g))).to(rows)
    pages = -(-T // page)
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[5::1000] = -1
    kc, vc = caches(cuda, pages, page, heads, d, torch.int8 if s8 else torch.bfloat16, True, 7)
    ks, vs = (torch.full((pages, heads, page), 5.0, device=cuda) if s8 else None for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    qmm.kv_append(x.to(cuda), -x.to(cuda), slots.to(cuda), kc, vc, k_scale=ks, v_scale=vs, dev_status=status)
    assert status.item() == 0
    keep = slots >= 0
    for cache, scale, part in ((kc, ks, x), (vc, vs, -x)):
        want = torch.full((pages * page, heads, d), 7, dtype=cache.dtype)
        if s8:
            q, sc = KV.append_s8(part.float().numpy())
            want[slots[keep]] = torch.from_numpy(q).to(torch.int8)[keep]
            wsc = torch.full((pages * page, heads), 5.0)
            wsc[slots[keep]] = torch.from_numpy(sc).float()[keep]
            assert torch.equal(scale.permute(0, 2, 1).reshape(-1, heads).cpu(), wsc)
        else:
            want[slots[keep]] = part.float().to(torch.bfloat16)[keep]
        assert torch.equal(cache.reshape(-1, heads, d).cpu(), want)


def test_append_codes_next_to_ties(qmm, cuda):
    """Quotients at and a few units in the last place around every half, at
    scales from subnormal to huge, against the oracle's division."""
    g = torch.Generator().manual_seed(3)
    T, heads, d = 400, 2, 128
    top = torch.exp2(torch.randint(-149, 127, (T, heads, 1), generator=g).float()) \
        * (1 + torch.rand((T, heads, 1), generator=g))
    half = torch.randint(-127, 127, (T, heads, d), generator=g) + 0.5
    x = (half.double() * (top.double() / 127)).float()
    bits = x.view(torch.int32) + torch.randint(-3, 4, x.shape, generator=g).int() * (x != 0)
    x = torch.minimum(torch.maximum(bits.view(torch.float32).nan_to_num(0, 0, 0), -top), top)
    x[..., :1] = top
    kc, vc = caches(cuda, 25, 16, heads, d, torch.int8, False, 7)
    ks, vs = (torch.full((25, heads, 16), 5.0, device=cuda) for _ in range(2))
    qmm.kv_append(x.to(cuda), x.flip(0).to(cuda), torch.arange(T, device=cuda), kc, vc, k_scale=ks, v_scale=vs)
    q, sc = KV.append_s8(x.numpy())
    for cache, scale, flip in ((kc, ks, False), (vc, vs, True)):
        got, gs = cache.reshape(T, heads, d).cpu(), scale.permute(0, 2, 1).reshape(T, heads).cpu()
        if flip:
            got, gs = got.flip(0), gs.flip(0)
        assert torch.equal(gs, torch.from_numpy(sc).float())
        assert torch.equal(got, torch.from_numpy(q).to(torch.int8))


def test_append_nothing(qmm, cuda):
    kc, vc = caches(cuda, 1, 4, 2, 64, torch.bfloat16, False, 3)
    e = torch.empty((0, 2, 64), device=cuda)
    qmm.kv_append(e, e, torch.empty(0, dtype=torch.int64, device=cuda), kc, vc)
    assert (kc == 3).all()


def test_append_past_four_gigabytes(qmm, cuda):
    """A page stride that carries the last pages past 2^32 bytes."""
    stride = (1 << 28) + 64                       # elements of bf16 between pages
    buf = torch.zeros(9 * stride, dtype=torch.bfloat16, device=cuda)
    kc = torch.as_strided(buf, (9, 2, 1, 64), (stride, 64, 64, 1))
    vc = torch.as_strided(buf, (9, 2, 1, 64), (stride, 64, 64, 1), 128)
    x = torch.randn((2, 1, 64), device=cuda)
    qmm.kv_append(x, -x, torch.tensor([17, 1], device=cuda), kc, vc)
    assert torch.equal(kc[8, 1], x[0].bfloat16()) and torch.equal(vc[8, 1], -x[0].bfloat16())
    assert torch.equal(kc[0, 1], x[1].bfloat16()) and not kc[1:8].any()
