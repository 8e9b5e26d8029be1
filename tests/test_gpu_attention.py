"""GPU parity of qmm_tree_attention against fp64 attention on the values that
the cache stands for.

Bound.  The kernels' inputs (bf16 q, bf16 or int8 cache with fp32 scales) are
exact in the oracle.  A score's fp32 sum over head_dim <= 128 products and its
scaling are within 128 * 2^-23 * scale * sum|q||k| plus 2^-22 |s|: for the
scores drawn here (sum|q||k| scale below 16, |s| below 16) at most 2.5e-4,
which changes a weight and the weights' sum by at most 2^-12 of themselves
each, 2^-11 together; the base-2 exponential and the fp32 sums add less than
2^-14.  The output is rounded to bf16 once, 2^-8 of itself.  With
A = sum_j p_j |v_j| >= |o|:
* up to 32 query rows per key head, the weights are two bf16 terms (2^-16):
  |out - o| <= (2^-11 + 2^-13) A + 2^-8 |o| (1 + 2^-10)
            <= (2^-9 + 2^-10) A + 2^-9 (1 + 2^-7) |o|;
* more rows, the weights are rounded to bf16 once, 2^-8 of each:
  |out - o| <= (2^-8 + 2^-11 + 2^-13) (1 + 2^-8) A + 2^-8 |o|
            <= (2^-8 + 2^-10) A + 2^-8 (1 + 2^-7) |o|.
"""
import numpy as np
import pytest
import torch

import oracle.kv_oracle as KV

pytestmark = pytest.mark.gpu


def build(dev, ctx, new, heads, kv, d, page, s8, head_major=False, tree=False, q_f32=False, seed=0, spare=1,
          stale=float("nan")):
    """A cache with the requests' rows at scattered pages; places that belong to
    no request hold `stale` (int8: extreme codes with `stale` scales)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g)
    blocks = max(need) + 1
    table = torch.full((len(ctx), blocks), -5, dtype=torch.int32)
    k = torch.full((pages, page, kv, d), stale)
    v = torch.full((pages, page, kv, d), stale)
    ks, vs = torch.full((2, pages, page, kv), stale)
    if s8:
        k.fill_(-128), v.fill_(-128)
    rows, at = [], 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        ids = order[at:at + need[r]]
        table[r, :need[r]] = ids.to(torch.int32)
        at += need[r]
        j = torch.arange(c + n)
        pg, off = ids[j // page] if c + n else j, j % page
        if s8:
            kr, vr = (torch.randint(-127, 128, (c + n, kv, d), generator=g).float() for _ in range(2))
            kc, vc = (torch.exp(0.3 * torch.randn((c + n, kv), generator=g)) / 73 for _ in range(2))
            ks[pg, off], vs[pg, off] = kc, vc
        else:
            kr, vr = (torch.randn((c + n, kv, d), generator=g).to(torch.bfloat16).float() for _ in range(2))
            kc = vc = torch.ones((c + n, kv))
        k[pg, off], v[pg, off] = kr, vr
        rows.append((kr.double() * kc.double()[..., None], vr.double() * vc.double()[..., None], pg, off))
    T = sum(new)
    q = torch.randn((T, heads, d), generator=g)
    if not q_f32:
        q = q.to(torch.bfloat16)
    mask = None
    if tree:
        W = -(-max(new) // 32)
        m = torch.zeros((T, W), dtype=torch.int64)
        t = 0
        for n in new:
            sets = []
            for i in range(n):
                up = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
                sets.append((sets[up] if up >= 0 else set()) | {i})
                for a in sets[i]:
                    m[t, a // 32] |= 1 << (a % 32)
                t += 1
        mask = torch.where(m >= 2 ** 31, m - 2 ** 32, m).to(torch.int32)
    dt = torch.int8 if s8 else torch.bfloat16

    def cache(x):
        x = x.to(dt)
        return x.permute(0, 2, 1, 3).contiguous().to(dev).permute(0, 2, 1, 3) if head_major else x.to(dev)

    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    scales = [x.permute(0, 2, 1).contiguous().to(dev) if s8 else None for x in (ks, vs)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    return dict(q=q, k=cache(k), v=cache(v), table=table.to(dev), ctx=i32(ctx), cu=i32(cu), mask=mask, ks=scales[0],
                vs=scales[1], rows=rows, lens=list(zip(ctx, new, cu)), max_new=max(1, max(new)), scale=d ** -0.5)


def call(qmm, dev, s, **over):
    a = dict(mask=None if s["mask"] is None else s["mask"].to(dev), scale=s["scale"], k_scale=s["ks"],
             v_scale=s["vs"], dev_status=torch.zeros(1, dtype=torch.int32, device=dev))
    a.update(over)
    out = qmm.tree_attention(over.pop("q", None) if "q" in over else s["q"].to(dev), s["k"], s["v"], s["table"],
                             s["ctx"], s["cu"], a.pop("max_new", s["max_new"]),
                             **{k: x for k, x in a.items() if k != "q"})
    torch.cuda.synchronize()
    assert a["dev_status"].item() == 0
    return out


def bound(s, ref, weight):
    rows = s["max_new"] * s["q"].shape[1] // s["k"].shape[2]
    u = 2 ** -9 if rows <= 32 else 2 ** -8
    return (u + 2 ** -10) * weight + u * (1 + 2 ** -7) * np.abs(ref) + 1e-37


def check(s, out):
    out = out.float().cpu().double().numpy()
    q = s["q"].to(torch.bfloat16).double().numpy()
    for (c, n, first), (k, v, _, _) in zip(s["lens"], s["rows"]):
        m = None if s["mask"] is None else [[int(w) & 0xFFFFFFFF for w in row] for row in s["mask"][first:first + n]]
        ref, weight = KV.attend(q[first:first + n], k.numpy(), v.numpy(), KV.visible(c, n, m), s["scale"])
        got = out[first:first + n]
        assert np.array_equal(np.isfinite(got), np.isfinite(ref))
        with np.errstate(invalid="ignore"):
            tol = bound(s, ref, weight)
            over = np.where(np.isfinite(ref), np.abs(got - ref) - tol, 0)
        assert (over <= 0).all(), (c, n, over.max())


LENS = [
    ([0], [1]), ([1], [1]), ([15], [1]), ([16], [1]), ([62], [1]), ([63], [1]), ([64], [1]), ([777], [1]),
    ([0, 5, 200, 63, 64], [3, 1, 0, 2, 7]), ([300, 0, 129], [4, 4, 4]), ([1000], [11]),
]


@pytest.mark.parametrize("ctx,new", LENS)
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths(qmm, cuda, d, s8, tree, ctx, new):
    s = build(cuda, ctx, new, 4, 2, d, 16, s8, tree=tree, seed=sum(ctx) + d)
    check(s, call(qmm, cuda, s))


@pytest.mark.parametrize("page", [1, 3, 16, 24, 48, 64, 100, 256])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("s8", [False, True])
def test_pages(qmm, cuda, s8, head_major, page):
    s = build(cuda, [130, 17, 255], [2, 9, 1], 6, 2, 128, page, s8, head_major, tree=True, seed=page)
    check(s, call(qmm, cuda, s))


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 3), (8, 1), (14, 2), (32, 8), (5, 1)])
@pytest.mark.parametrize("new", [1, 5, 33])
@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("q_f32", [False, True])
def test_heads(qmm, cuda, q_f32, s8, new, heads, kv):
    """From one query row per key head to several tiles of rows."""
    s = build(cuda, [90, 3], [new, max(1, new // 2)], heads, kv, 128, 16, s8, tree=True, q_f32=q_f32, seed=heads + new)
    check(s, call(qmm, cuda, s))


@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 40, 128])
@pytest.mark.parametrize("tree", [False, True])
def test_many_rows(qmm, cuda, tree, page, d, s8):
    """Hundreds of query rows per key head, tails of every kind."""
    s = build(cuda, [0, 500, 127, 128, 37], [64, 70, 1, 129, 60], 8, 2, d, page, s8, tree=tree, seed=page + d)
    check(s, call(qmm, cuda, s))


@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("heads,kv", [(2, 2), (6, 2), (10, 2), (16, 2)])
@pytest.mark.parametrize("page", [16, 20])
def test_prompts(qmm, cuda, page, heads, kv, s8):
    """Causal chunks over several row tiles, where later cached tiles are seen
    by the last rows only: row tiles that end inside a token's group, at empty
    caches and past them."""
    s = build(cuda, [0, 127, 300, 64], [519, 257, 1, 384], heads, kv, 64, page, s8, seed=heads)
    check(s, call(qmm, cuda, s))


def test_prompts_of_many_requests(qmm, cuda):
    """More requests than a warp's lanes, of every length."""
    new = [(37 * i) % 290 for i in range(41)]
    s = build(cuda, [(61 * i) % 200 for i in range(41)], new, 3, 1, 64, 32, False, seed=41)
    check(s, call(qmm, cuda, s))


@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("new,heads", [(1, 4), (8, 8), (40, 8)])
def test_long_context_split_between_blocks(qmm, cuda, s8, new, heads):
    s = build(cuda, [20011], [new], heads, 1, 128, 16, s8, tree=True, seed=new)
    a = call(qmm, cuda, s)
    check(s, a)
    assert torch.equal(a, call(qmm, cuda, s))    # fixed order of the sums


@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("heads,new", [(16, [33, 28, 22, 32, 26, 19, 30, 23]), (8, [9, 16, 5, 14, 12, 3, 10, 8])])
def test_many_items_in_a_block(qmm, cuda, s8, heads, new):
    """Requests of a few tiles each, of which every block walks several, with
    new tokens across tile boundaries (and, in the first, rows just past 128)."""
    ctx = [3819, 1346, 3117, 2022, 3793, 2699, 1604, 3375]
    s = build(cuda, ctx, new, heads, 4, 64, 32, s8, tree=True, seed=11)
    check(s, call(qmm, cuda, s))
    s = build(cuda, [120 + i % 16 for i in range(300)], [2 + i % 9 for i in range(300)], heads, 4, 64, 8, s8, tree=True,
              seed=12)
    check(s, call(qmm, cuda, s))


def test_many_requests(qmm, cuda):
    g = torch.Generator().manual_seed(3)
    ctx = torch.randint(0, 90, (333,), generator=g).tolist()
    new = torch.randint(0, 4, (333,), generator=g).tolist()
    s = build(cuda, ctx, new, 4, 2, 64, 16, False, tree=True, seed=4)
    check(s, call(qmm, cuda, s))


@pytest.mark.parametrize("new,heads", [(6, 4), (50, 16)])
@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("ctx", [0, 100])
def test_rows_that_see_little(qmm, cuda, ctx, s8, new, heads):
    """Mask rows without a bit: zeros without a context, the context's average
    with one; and a row that does not see itself."""
    s = build(cuda, [ctx], [new], heads, 2, 128, 16, s8, tree=True, seed=1)
    s["mask"][0] = 0
    s["mask"][new - 1] = 0
    s["mask"][2] = 2                              # only token 1
    out = call(qmm, cuda, s)
    if ctx == 0:
        assert not out[0].any() and not out[new - 1].any()
    check(s, out)


@pytest.mark.parametrize("new,heads", [(6, 4), (50, 16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("side", ["k", "v"])
@pytest.mark.parametrize("s8", [False, True])
def test_nonfinite_values_stay_hidden(qmm, cuda, s8, side, bad, new, heads):
    """A new token whose row is not finite reaches exactly the rows that see it."""
    s = build(cuda, [70], [new], heads, 2, 128, 16, s8, tree=True, seed=2)
    s["mask"][:] &= ~8
    s["mask"][3] |= 8
    s["mask"][5] |= 8                             # rows 3 and 5 see token 3, the others do not
    k, v, pg, off = s["rows"][0]
    t = 70 + 3
    if s8:
        s["ks" if side == "k" else "vs"][pg[t], :, off[t]] = bad
        x = k if side == "k" else v
        code = s["k" if side == "k" else "v"][pg[t], off[t]].cpu().double()
        x[t] = code * bad
    else:
        s["k" if side == "k" else "v"][pg[t], off[t], :, 7] = bad
        (k if side == "k" else v)[t, :, 7] = bad
    out = call(qmm, cuda, s).float().cpu()
    rows = [i for i in range(new) if i not in (3, 5)]
    clean = dict(s, rows=[(torch.nan_to_num(k, 0, 0, 0), torch.nan_to_num(v, 0, 0, 0), pg, off)])
    assert torch.isfinite(out[rows]).all()
    if side == "v" and not s8:
        assert (~torch.isfinite(out[[3, 5]])).sum() == 2 * heads    # one value of each row
        assert torch.equal(torch.isnan(out[3, :, 7]), torch.isnan(torch.full((heads,), bad)))
    ref, weight = KV.attend(s["q"].double().numpy(), clean["rows"][0][0].numpy(), clean["rows"][0][1].numpy(),
                            KV.visible(70, new, [[int(w) & 0xFFFFFFFF for w in r] for r in s["mask"]]), s["scale"])
    got = out.double().numpy()
    tol = bound(s, ref, weight)
    assert (np.abs(got - ref)[rows] <= tol[rows]).all()


@pytest.mark.parametrize("new", [1, 40])
def test_large_scores(qmm, cuda, new):
    """Scores of a few hundred: one token takes all the weight; no overflow."""
    s = build(cuda, [200], [new], 4, 2, 128, 16, False, seed=5)
    s["scale"] = 16.0
    out = call(qmm, cuda, s).float()
    assert torch.isfinite(out).all()
    # the largest score's value row, wherever it leads by 40 (the others' weights are below e^-40)
    k, v, _, _ = s["rows"][0]
    for i in range(new):
        for h in range(4):
            sc = (k[:200 + i + 1, h // 2] @ s["q"][i, h].double()) * 16.0
            top = sc.topk(2)
            if top.values[0] - top.values[1] > 40:
                want = v[top.indices[0], h // 2].float()
                assert torch.equal(out[i, h].cpu(), want)


def test_strided_views_and_padding_rows(qmm, cuda):
    """q and out inside wider buffers; rows past the step's tokens untouched."""
    s = build(cuda, [40, 9], [3, 2], 4, 2, 64, 16, False, tree=True, seed=6)
    T = 5
    wide = torch.randn((T + 3, 12, 64), device=cuda).to(torch.bfloat16)
    wide[:T, 2:10:2] = s["q"].to(cuda)
    out = torch.full((T + 3, 5, 96), 7.0, dtype=torch.bfloat16, device=cuda)
    m = torch.zeros((T + 3, 3), dtype=torch.int32, device=cuda)[:, :1]
    m[:T] = s["mask"].to(cuda)
    o = out[:, 1:, 16:80]
    call(qmm, cuda, s, q=wide[:, 2:10:2], out=o, mask=m)
    check(s, o[:T])
    assert (out[T:] == 7).all() and (out[:, 0] == 7).all() and (out[..., :16] == 7).all() and (out[..., 80:] == 7).all()


@pytest.mark.parametrize("new", [2, 64])
def test_cache_past_four_gigabytes(qmm, cuda, new):
    s = build(cuda, [100], [new], 4, 1, 64, 16, False, seed=7)
    n = s["k"].shape[0]
    stride = ((5 << 30) // (n - 1) // 2 + 64) // 64 * 64
    for x in "kv":
        buf = torch.empty(n * stride, dtype=torch.bfloat16, device=cuda)
        wide = torch.as_strided(buf, s[x].shape, (stride,) + s[x].stride()[1:])
        wide.copy_(s[x])
        s[x] = wide
    check(s, call(qmm, cuda, s))


@pytest.mark.parametrize("new", [1, 64])
def test_other_stream_and_graph(qmm, cuda, new):
    """Queued on a side stream, and captured once then replayed with lengths and
    tables that changed on the device."""
    s = build(cuda, [333], [new], 4, 2, 128, 16, False, seed=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros((new, 4, 128), dtype=torch.bfloat16, device=cuda)
    ws = torch.empty(qmm.tree_attention_workspace_size(4, 2, 128, new), dtype=torch.uint8, device=cuda)
    q = s["q"].to(cuda)
    with torch.cuda.stream(side):
        call(qmm, cuda, s, q=q, out=out, workspace=ws)
    torch.cuda.synchronize()
    check(s, out)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.tree_attention(q, s["k"], s["v"], s["table"], s["ctx"], s["cu"], new, scale=s["scale"], out=out,
                           workspace=ws, dev_status=status)
    s["ctx"].fill_(200)                           # a shorter context: the same pages, fewer tokens
    k, v, pg, off = s["rows"][0]
    s["rows"] = [(k[:200 + new], v[:200 + new], pg, off)]
    s["lens"] = [(200, new, 0)]
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert status.item() == 0
    check(s, out)


def test_lengths_that_do_not_fit(qmm, cuda):
    """Reported on the device; the other requests get their rows."""
    for what in ("ctx", "blocks", "new", "cu"):
        s = build(cuda, [40, 50], [2, 2], 4, 2, 64, 16, False, seed=9)
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        out = torch.full((4, 4, 64), 7.0, dtype=torch.bfloat16, device=cuda)
        max_new = 2
        if what == "ctx":
            s["ctx"][1] = -1
        elif what == "blocks":
            s["ctx"][1] = 16 * s["table"].shape[1]
        elif what == "new":
            s["cu"][2] = 4
            max_new = 1
        else:
            s["cu"][2] = 5
        qmm.tree_attention(s["q"].to(cuda), s["k"], s["v"], s["table"], s["ctx"], s["cu"], max_new, out=out,
                           dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == qmm.QMM_ERR_INVALID_ARG, what
        assert (out[2:] == 7).all()
        if what != "new":
            s["lens"], s["rows"] = s["lens"][:1], s["rows"][:1]
            check(s, out)


@pytest.mark.parametrize("page_id", [-1, 1000])
@pytest.mark.parametrize("new", [2, 64])
def test_bad_page_id(qmm, cuda, page_id, new):
    s = build(cuda, [40, 50], [2, new], 4, 2, 64, 16, False, seed=10)
    s["table"][1, 1] = page_id
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    out = qmm.tree_attention(s["q"].to(cuda), s["k"], s["v"], s["table"], s["ctx"], s["cu"], max(2, new),
                             dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == qmm.QMM_ERR_INVALID_ARG
    s["lens"], s["rows"] = s["lens"][:1], s["rows"][:1]
    check(s, out)


def test_no_tokens(qmm, cuda):
    s = build(cuda, [5], [1], 4, 2, 64, 16, False)
    out = qmm.tree_attention(torch.empty((0, 4, 64), dtype=torch.bfloat16, device=cuda), s["k"], s["v"], s["table"],
                             s["ctx"], s["cu"], 1)
    assert out.shape == (0, 4, 64)
    empty = build(cuda, [5, 7], [0, 0], 4, 2, 64, 16, False)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device=cuda)
    out = torch.full((3, 4, 64), 7.0, dtype=torch.bfloat16, device=cuda)
    qmm.tree_attention(q, empty["k"], empty["v"], empty["table"], empty["ctx"], empty["cu"], 1, out=out)
    torch.cuda.synchronize()
    assert (out == 7).all()
