"""GPU parity of what runs beside the projections (qmm_block_norm, qmm_lora_add,
qmm_token_logprobs) against the fp64 oracle, within its bounds on fp32 arithmetic
and half a step of the output type."""
import numpy as np
import pytest
import torch

import oracle.beside_oracle as O

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, bound, half, what):
    got = got.double().cpu().numpy()
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), what
    with np.errstate(invalid="ignore"):
        far = np.abs(got - want) - (bound * (1 + half) + half * np.abs(want))
    far = np.where(nan | (got == want), -1.0, far)
    assert far.max() <= 0, f"{what}: {(far > 0).sum()} of {far.size} too far, worst by {far.max():.3g}"


def wide(t, cols):
    """A view of t's values inside rows of `cols` elements."""
    out = torch.full((t.shape[0], cols), 7.0, dtype=t.dtype, device=t.device)[:, :t.shape[1]]
    return out.copy_(t)


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------

NORM_CASES = [
    # T, D, residual, branch, post, gate, kind, out
    (1, 1, "f32", "f32", "rms", None, "rms", "bf16"),
    (3, 8, "bf16", "f32", None, "channel", "layer", "f32"),
    (5, 24, "f32", "bf16", "layer", "token", "rms", "bf16"),
    (2, 100, "f32", "f32", None, None, None, "bf16"),
    (7, 255, "bf16", "bf16", "rms", "token", "layer", "bf16"),
    (4, 256, "f32", None, None, None, "rms", "bf16"),
    (9, 1000, "f32", "f32", "rms", "channel", "rms", "s8"),
    (6, 1001, "bf16", "bf16", "layer", "token", "layer", "s8"),
    (400, 1024, "f32", "f32", "rms", None, "rms", "bf16"),
    (1, 4096, "f32", "f32", "rms", "token", "rms", "s8"),
    (330, 4608, "f32", "f32", "rms", "channel", "rms", "s8"),
    (320, 2052, "bf16", "f32", None, "token", "layer", "f32"),
    (3, 8200, "f32", "bf16", "layer", None, "rms", "bf16"),
    (2, 8193, "f32", "f32", "rms", "token", "layer", "bf16"),
    (310, 16392, "bf16", "bf16", "rms", "channel", "rms", "bf16"),
    (2, 32768, "f32", "f32", "layer", "token", "layer", "f32"),
    (2, 32767, "bf16", "f32", "rms", None, "rms", "s8"),
]


def norm_case(dev, T, D, residual, branch, post, gate, kind, out, stride=0, seed=0):
    g = torch.Generator().manual_seed(seed + T + 31 * D)
    r = lambda *s: torch.randn(s, generator=g)
    loud = torch.where(torch.rand(D, generator=g) < 0.05, 30.0, 1.0)
    lay = (lambda t: wide(t, D + stride)) if stride else (lambda t: t)
    a = dict(residual=lay((r(T, D) * loud + 0.5).to(TYPES[residual]).to(dev)), norm=kind, scale=0.7, eps=1e-5)
    if kind is not None:
        a.update(weight=(1 + 0.3 * r(D)).to(dev))
        if kind == "layer" or D % 2:
            a.update(bias=(0.2 * r(D)).to(dev))
    if branch is not None:
        a.update(branch=lay((r(T, D) * torch.exp(r(T, 1))).to(TYPES[branch]).to(dev)))
    if post is not None:
        a.update(branch_norm=post, branch_weight=(1 + 0.3 * r(D)).to(dev), branch_eps=1e-6)
        if post == "layer":
            a.update(branch_bias=(0.2 * r(D)).to(dev))
    if gate == "channel":
        a.update(gate=r(D).to(dev))
    elif gate == "token":
        a.update(gate=lay(torch.sigmoid(r(T, D)).to(torch.bfloat16).to(dev)))
    return a, out


def norm_exact(a):
    return O.block(f64(a["residual"]), f64(a.get("branch")), a.get("branch_norm"), f64(a.get("branch_weight")),
                   f64(a.get("branch_bias")), a.get("branch_eps", 0.0), f64(a.get("gate")), np.float32(a["scale"]),
                   a["norm"], f64(a.get("weight")), f64(a.get("bias")), np.float32(a["eps"]))


def check_norm(a, out_type, got, half_sum):
    total, d_total, x, d_x = norm_exact(a)
    if a.get("branch") is not None:
        close(got[0], total, d_total, half_sum, "sum")
    if out_type != "s8":
        close(got[1], x, d_x, O.HALF[out_type], "out")
        return
    codes, s = got[1].double().cpu().numpy(), got[2].double().cpu().numpy()[:, None]
    amax = np.abs(x).max(1, keepdims=True)
    assert (np.abs(s * 127 - amax) <= d_x.max(1, keepdims=True) + 2 * O.U32 * amax).all()
    # a code is within half a step of the value, give or take the value's own error and two roundings
    assert (np.abs(codes * s - x) <= s * 0.5 * (1 + 256 * O.U32) + d_x + 4 * O.U32 * np.abs(x)).all()
    assert np.abs(codes).max() <= 127


@pytest.mark.parametrize("case", NORM_CASES, ids=lambda c: "-".join(map(str, c)))
def test_norm(qmm, cuda, case):
    a, out_type = norm_case(cuda, *case)
    kw = {k: v for k, v in a.items() if k not in ("residual", "branch")}
    if a.get("branch") is not None:
        kw["residual_out"] = torch.full_like(a["residual"], 9.0)
    before = a["residual"].clone()
    got = qmm.block_norm(a["residual"], a.get("branch"), out_type=out_type, **kw)
    again = qmm.block_norm(a["residual"], a.get("branch"), out_type=out_type, **kw)
    assert torch.equal(a["residual"], before)
    for x, y in zip(got[1:], again[1:]):
        assert torch.equal(x, y)
    check_norm(a, out_type, got, O.HALF[case[2]])


@pytest.mark.parametrize("stride", [8, 16, 1, 5])
@pytest.mark.parametrize("case", [NORM_CASES[i] for i in (4, 6, 7, 11, 12)], ids=lambda c: "-".join(map(str, c)))
def test_norm_strided_in_place(qmm, cuda, case, stride):
    """Rows inside wider ones, the sum over the residual itself: the same values
    as in rows laid out the same apart from it (in others the sums may be split
    otherwise), and nothing written between the rows."""
    a, out_type = norm_case(cuda, *case, stride=stride)
    T, D = a["residual"].shape
    kw = {k: v for k, v in a.items() if k not in ("residual", "branch")}
    store = torch.full((T, (D + 47) // 16 * 16), 5, dtype={"s8": torch.int8}.get(out_type, TYPES.get(out_type)),
                       device=cuda)
    apart = qmm.block_norm(a["residual"], a["branch"], residual_out=torch.empty_like(a["residual"]),
                           out=store[:, :D], **kw)
    check_norm(a, out_type, apart, O.HALF[case[2]])
    apart = qmm.block_norm(a["residual"], a["branch"], residual_out=wide(a["residual"], D + stride),
                           out=store[:, :D], **kw)
    check_norm(a, out_type, apart, O.HALF[case[2]])
    assert (store[:, D:] == 5).all()
    first = apart[1].clone()
    total = a["residual"]
    qmm.block_norm(total, a["branch"], out=store[:, :D], **kw)
    assert torch.equal(total, apart[0]) and torch.equal(store[:, :D], first)
    whole = torch.as_strided(total, (T - 1, stride), (D + stride, 1), total.storage_offset() + D)
    assert (whole == 7.0).all()


def test_norm_alone_and_sum_alone(qmm, cuda):
    a, _ = norm_case(cuda, 5, 72, "f32", "f32", "rms", None, "rms", "bf16")
    total, out = qmm.block_norm(a["residual"], norm="rms", weight=a["weight"], eps=1e-5)
    assert total is a["residual"]
    close(out, *O.block(f64(a["residual"]), None, None, None, None, 0, None, 1, "rms", f64(a["weight"]), None,
                        np.float32(1e-5))[2:], O.HALF["bf16"], "out")
    want = f64(a["residual"]) + f64(a["branch"])
    total, out = qmm.block_norm(a["residual"], a["branch"], out=False)
    assert out is None and total is a["residual"]
    close(total, want, O.U32 * np.abs(want), O.U32, "sum")


def test_norm_nonfinite_rows_stay_apart(qmm, cuda):
    a, _ = norm_case(cuda, 6, 512, "f32", "f32", "rms", None, "rms", "bf16")
    clean = qmm.block_norm(a["residual"], a["branch"], residual_out=torch.empty_like(a["residual"]),
                           **{k: v for k, v in a.items() if k not in ("residual", "branch")})
    a["branch"][2, 100], a["residual"][4, 7] = float("nan"), float("inf")
    got = qmm.block_norm(a["residual"], a["branch"], residual_out=torch.empty_like(a["residual"]),
                         **{k: v for k, v in a.items() if k not in ("residual", "branch")})
    rows = [0, 1, 3, 5]
    assert torch.equal(got[0][rows], clean[0][rows]) and torch.equal(got[1][rows], clean[1][rows])
    assert torch.isnan(got[1][2]).all() and torch.isnan(got[1][4, 7])


# widths where a row's threads, groups and their order of loading change, and enough rows to fill the GPU
@pytest.mark.parametrize("case", [
    (1300, 64, "f32", "f32", "rms", "token", "rms", "bf16"), (5000, 72, "bf16", "bf16", None, None, "layer", "s8"),
    (700, 1032, "f32", "bf16", "layer", "token", "rms", "s8"), (640, 3001, "f32", "f32", "rms", "token", "rms", "bf16"),
    (500, 8192, "bf16", "f32", "rms", "channel", "layer", "bf16"),
    (400, 12288, "f32", "f32", "rms", "token", "rms", "bf16"),
    (400, 12296, "f32", "f32", "layer", "token", "rms", "s8"),
    (330, 20000, "f32", "bf16", "rms", "token", "rms", "f32"),
    (5, 16384, "bf16", "f32", "rms", None, "layer", "bf16"), (320, 32768, "f32", "f32", None, "token", "rms", "bf16"),
    (310, 9999, "f32", "bf16", "rms", "channel", "layer", "bf16"),
], ids=lambda c: "-".join(map(str, c)))
def test_norm_many(qmm, cuda, case):
    test_norm(qmm, cuda, case)


@pytest.mark.parametrize("T,D", [(5, 96), (3, 101), (330, 4608), (310, 16384)])
def test_norm_gates_of_the_other_type(qmm, cuda, T, D):
    """A channel gate in bf16, a gate of rows in fp32."""
    a, out_type = norm_case(cuda, T, D, "f32", "f32", "rms", "channel", "rms", "bf16")
    for gate in (a["gate"].to(torch.bfloat16), torch.randn((T, D), device=cuda)):
        a["gate"] = gate
        kw = {k: v for k, v in a.items() if k not in ("residual", "branch")}
        check_norm(a, out_type, qmm.block_norm(a["residual"], a["branch"], residual_out=torch.empty_like(a["residual"]),
                                               **kw), 0.0)


def test_norm_zero_rows(qmm, cuda):
    z = torch.zeros((4, 640), device=cuda)
    total, out, s = qmm.block_norm(z, z.clone(), residual_out=torch.empty_like(z), out_type="s8", eps=1e-6)
    assert not total.any() and not out.any() and not s.any()
    total, out = qmm.block_norm(z[:0], z[:0])
    assert total.shape == out.shape == (0, 640)


def test_norm_rows_past_32_bits(qmm, cuda):
    """Element offsets beyond 2^31: rows far apart in memory."""
    D, T, ld = 64, 5, 1 << 29
    store = torch.zeros((T - 1) * ld + D, dtype=torch.bfloat16, device=cuda)
    res = torch.as_strided(store, (T, D), (ld, 1))
    want = torch.randn((T, D), device=cuda).to(torch.bfloat16)
    res.copy_(want)
    _, out = qmm.block_norm(res, norm=None, out_type="f32")
    assert torch.equal(out, want.float())


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------

LORA_CASES = [
    # M, K, N, adapters, max_rank, prompt
    (1, 8, 1, 1, 1, False), (1, 1024, 2048, 3, 16, False), (3, 40, 33, 2, 5, False), (16, 256, 100, 1, 8, False),
    (17, 512, 260, 4, 17, False), (64, 1000, 516, 20, 64, False), (65, 264, 130, 1, 33, True),
    (200, 2048, 1028, 5, 100, True), (256, 1024, 640, 300, 24, False), (300, 520, 257, 3, 256, True),
    (700, 320, 1200, 2, 200, True), (1025, 136, 96, 7, 12, False), (2500, 64, 64, 3, 8, True),
]


def lora_case(dev, M, K, N, adapters, rank, prompt, seed=0, none=0.1):
    g = torch.Generator().manual_seed(seed + M + K + N)
    r = lambda *s: torch.randn(s, generator=g)
    ids = torch.randint(0, adapters, (M,), generator=g)
    ids = torch.sort(ids).values if prompt else ids
    ids[torch.rand(M, generator=g) < none] = -1
    ranks = torch.randint(0, rank + 1, (adapters,), generator=g)
    ranks[0] = rank
    A = r(adapters, rank, K) / K ** 0.5
    B = r(adapters, N, -(-rank // 8) * 8)
    for a in range(adapters):           # what lies behind a rank is never used
        A[a, int(ranks[a]):] = float("nan")
        B[a, :, int(ranks[a]):] = float("nan")
    return dict(X=r(M, K).to(torch.bfloat16).to(dev), ids=ids.to(torch.int32).to(dev), A=A.to(torch.bfloat16).to(dev),
                B=B.to(torch.bfloat16).to(dev)[:, :, :rank], base=r(M, N).to(dev),
                ranks=ranks.to(torch.int32).to(dev), scales=(0.1 + r(adapters).abs()).to(dev))


def lora_exact(a, **over):
    a = {**a, **over}
    clean = lambda t: torch.nan_to_num(t.float(), nan=0.0)
    return O.lora(f64(a["X"]), a["ids"].cpu().numpy(), f64(clean(a["A"])), f64(clean(a["B"])), f64(a["base"]),
                  None if a["ranks"] is None else a["ranks"].cpu().numpy(),
                  None if a["scales"] is None else f64(a["scales"]))


@pytest.mark.parametrize("case", LORA_CASES, ids=lambda c: "-".join(map(str, c)))
def test_lora(qmm, cuda, case):
    a = lora_case(cuda, *case)
    want, bound = lora_exact(a)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    out = qmm.lora_add(**a, dev_status=status)
    close(out, want, bound, 0.0, "out")
    assert torch.equal(qmm.lora_add(**a), out)
    inplace = a["base"].clone()
    assert torch.equal(qmm.lora_add(**{**a, "base": inplace}, out=inplace), out)
    want0, bound0 = lora_exact(a, base=None)
    close(qmm.lora_add(**{**a, "base": None}), np.zeros(out.shape) if want0 is None else want0, bound0, 0.0, "no base")
    assert int(status) == 0


# many rows, ranks and adapters: rows routed to tiles of 128, and the limits on either side
@pytest.mark.parametrize("case", [
    (384, 264, 68, 5, 256, False), (385, 520, 130, 3, 256, False), (1536, 264, 100, 700, 8, False),
    (1537, 72, 40, 3000, 8, False), (1000, 64, 36, 8192, 5, False), (1700, 72, 36, 8192, 5, False),
    (1700, 328, 517, 5, 16, True), (2100, 512, 388, 40, 40, False), (600, 1024, 260, 2, 200, True),
    (5000, 128, 132, 1, 7, True), (1900, 1000, 65, 9, 64, True), (40, 4096, 33, 3, 250, False),
    (200, 520, 70, 7, 129, False), (4000, 2048, 300, 6, 65, True),
    (1600, 520, 130, 3, 256, False), (1600, 1032, 260, 2, 200, True), (2000, 256, 300, 60, 150, False),
    (1600, 128, 200, 70, 24, False), (1700, 72, 131, 40, 96, False), (1540, 64, 257, 1500, 70, False),
    (900, 4096, 2052, 2, 256, True), (300, 8192, 4100, 3, 256, True),
], ids=lambda c: "-".join(map(str, c)))
def test_lora_many(qmm, cuda, case):
    test_lora(qmm, cuda, case)


@pytest.mark.parametrize("M", [400, 2000])
def test_lora_many_rows_in_another_order(qmm, cuda, M):
    a = lora_case(cuda, M, 512, 300, 4, 40, True)
    out = qmm.lora_add(**a)
    order = torch.randperm(M, device=cuda)
    moved = qmm.lora_add(**{**a, "X": a["X"][order], "ids": a["ids"][order], "base": a["base"][order]})
    assert torch.equal(moved, out[order])
    X = a["X"].clone()
    X[77] = float("inf")
    got = qmm.lora_add(**{**a, "X": X})
    rows = torch.arange(M, device=cuda) != 77
    assert torch.equal(got[rows], out[rows])


def test_lora_many_rows_without_ranks_and_scales_strided(qmm, cuda):
    test_lora_without_ranks_and_scales_strided(qmm, cuda, 2000)


def test_lora_many_rows_bad_ids_and_ranks(qmm, cuda):
    test_lora_bad_ids_and_ranks(qmm, cuda, 2000)


@pytest.mark.parametrize("M", [500, 2000])
def test_lora_many_rows_nobody_has_an_adapter(qmm, cuda, M):
    a = lora_case(cuda, M, 64, 48, 2, 8, False, none=1.1)
    assert torch.equal(qmm.lora_add(**a), a["base"])
    assert not qmm.lora_add(**{**a, "base": None}).any()
    store = a["base"].clone()
    assert qmm.lora_add(**{**a, "base": store}, out=store) is store and torch.equal(store, a["base"])


@pytest.mark.parametrize("M", [3, 500, 2000])
def test_lora_infinities(qmm, cuda, M):
    """Infinities in rows of X reach out as the formula has them, beside an adapter's
    zeros as NaN."""
    a = lora_case(cuda, M, 64, 48, 3, 1, False, none=0.0)
    a["ranks"][:] = 1                       # adapters of rank 0 before: all zeros
    a["A"].nan_to_num_(), a["B"].nan_to_num_()
    a["ids"][1:3] = 0                       # one that is not
    a["X"][1, 3], a["X"][2, 60] = float("inf"), -float("inf")
    with np.errstate(invalid="ignore"):
        want, bound = lora_exact(a)
    assert np.isinf(want[1:3]).all()
    close(qmm.lora_add(**a), want, bound, 0.0, "out")


@pytest.mark.parametrize("M", [3, 500, 2000])
def test_lora_slots_past_32_bits(qmm, cuda, M):
    """Slots, and rows of X, base and out, far apart."""
    a = lora_case(cuda, M, 64, 48, 3, 8, False)
    want = qmm.lora_add(**a)
    slot = (1 << 31) + 8
    for name in ("A", "B"):
        t = a[name]
        store = torch.empty(2 * slot + t[0].numel() + 8 * t.shape[1], dtype=torch.bfloat16, device=cuda)
        far = torch.as_strided(store, t.shape, (slot, t.stride(1), 1))
        far.copy_(t)
        a[name] = far
    assert torch.equal(qmm.lora_add(**a), want)


def test_lora_rows_past_32_bits(qmm, cuda):
    a = lora_case(cuda, 3, 64, 48, 3, 8, False)
    want = qmm.lora_add(**a)
    ld = (1 << 30) + 8
    for name in ("X", "base"):
        t = a[name]
        far = torch.as_strided(torch.empty(2 * ld + 64, dtype=t.dtype, device=cuda), t.shape, (ld, 1))
        a[name] = far.copy_(t)
    assert torch.equal(qmm.lora_add(**a), want)
    assert qmm.lora_add(**a, out=a["base"]) is a["base"] and torch.equal(a["base"], want)


def test_lora_rows_do_not_depend_on_each_other(qmm, cuda):
    """A row's result is the same in another order of rows, and a row of NaN
    beside it changes nothing."""
    a = lora_case(cuda, 150, 512, 300, 4, 40, False)
    out = qmm.lora_add(**a)
    order = torch.randperm(150, device=cuda)
    moved = qmm.lora_add(**{**a, "X": a["X"][order], "ids": a["ids"][order], "base": a["base"][order]})
    assert torch.equal(moved, out[order])
    X = a["X"].clone()
    X[77] = float("nan")
    got = qmm.lora_add(**{**a, "X": X})
    rows = torch.arange(150, device=cuda) != 77
    assert torch.equal(got[rows], out[rows])


@pytest.mark.parametrize("M", [5, 70, 600])
def test_lora_without_ranks_and_scales_strided(qmm, cuda, M):
    a = lora_case(cuda, M, 128, 75, 3, 24, False)
    a["A"], a["B"] = torch.nan_to_num(a["A"]), torch.nan_to_num(a["B"])
    a["ranks"] = a["scales"] = None
    a["X"] = wide(a["X"], 136)
    a["base"] = wide(a["base"], 81)
    store = torch.full((M, 90), 3.0, device=cuda)
    want, bound = lora_exact(a)
    qmm.lora_add(**a, out=store[:, :75])
    close(store[:, :75], want, bound, 0.0, "out")
    assert (store[:, 75:] == 3.0).all()


@pytest.mark.parametrize("M", [9, 600])
def test_lora_bad_ids_and_ranks(qmm, cuda, M):
    a = lora_case(cuda, M, 64, 40, 4, 8, False, none=0.0)
    a["ids"][1], a["ids"][4] = 4, -2
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    out = qmm.lora_add(**a, dev_status=status)
    assert int(status) == qmm.QMM_ERR_INVALID_ARG
    close(out, *lora_exact(a), 0.0, "out")
    a["ids"][1] = a["ids"][4] = -1
    for bad in (9, -1):
        a["ranks"][2] = bad
        status.zero_()
        out = qmm.lora_add(**a, dev_status=status)
        assert int(status) == (qmm.QMM_ERR_INVALID_ARG if (a["ids"] == 2).any() else 0)
        close(out, *lora_exact(a), 0.0, "out")


def test_lora_nobody_has_an_adapter(qmm, cuda):
    a = lora_case(cuda, 90, 64, 48, 2, 8, False, none=1.1)
    assert torch.equal(qmm.lora_add(**a), a["base"])
    assert not qmm.lora_add(**{**a, "base": None}).any()
    assert qmm.lora_add(**{**a, "X": a["X"][:0], "ids": a["ids"][:0], "base": a["base"][:0]}).shape == (0, 48)


# ---------------------------------------------------------------------------
# log probabilities
# ---------------------------------------------------------------------------

def check_logprobs(qmm, x, tokens, k, scale, status=None):
    got = qmm.token_logprobs(x, tokens, top_k=k, scale=scale, dev_status=status)
    again = qmm.token_logprobs(x, tokens, top_k=k, scale=scale)
    want, tol = O.logprobs(f64(x), None if tokens is None else tokens.cpu().numpy(), k, float(np.float32(scale)))
    for a, b in zip(got, again):
        assert a is None and b is None or torch.equal(torch.nan_to_num(a, nan=1e9), torch.nan_to_num(b, nan=1e9))
    if tokens is not None:
        close(got[0], want["logprobs"], tol["logprobs"], 0.0, "logprobs")
    close(got[1], want["entropy"], tol["entropy"], 0.0, "entropy")
    if k:
        assert np.array_equal(got[2].cpu().numpy(), want["ids"])
        close(got[3], want["top"], tol["top"], 0.0, "top_logprobs")
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V,k,scale", [(1, 1, 1, 1.0), (2, 3, 5, 1.0), (3, 7, 0, 0.3), (5, 100, 32, 2.0),
                                         (1, 4096, 20, 1.0), (4, 4099, 7, 1.0), (2, 16384, 1, 1.0),
                                         (3, 16389, 20, 0.7), (1, 151936, 20, 1.0), (2, 151936, 32, 1.25),
                                         (310, 5001, 3, 1.0), (700, 300, 4, 1.0), (9, 70001, 11, 1.0)])
def test_logprobs(qmm, cuda, M, V, k, scale, dtype):
    g = torch.Generator().manual_seed(M + V)
    x = 3.0 * torch.randn((M, V), generator=g)
    x[torch.arange(M), torch.randint(0, V, (M,), generator=g)] += 8.0
    tokens = torch.randint(0, V, (M, 3), generator=g).to(torch.int32)
    tokens[:, 1] = x.argmax(1).to(torch.int32)
    check_logprobs(qmm, x.to(TYPES[dtype]).to(cuda), tokens.to(cuda), k, scale)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad", [1, 2, 3, 8])
def test_logprobs_rows_inside_wider_ones(qmm, cuda, pad, dtype):
    """What lies between the rows is not read; rows start at every alignment."""
    x = torch.full((9, 1237 + pad), float("nan"), dtype=TYPES[dtype], device=cuda)
    x[:, :1237] = torch.randn((9, 1237), device=cuda) * 2
    tokens = torch.randint(0, 1237, (9, 5), device=cuda, dtype=torch.int32)
    check_logprobs(qmm, x[:, :1237], tokens[:, 1:4], 6, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [50, 20000, 151936])
def test_logprobs_ties(qmm, cuda, V, dtype):
    """Equal logits fall by rising index; -0 equals 0; a whole row of one value."""
    x = torch.zeros((5, V))
    x[1] = torch.randint(0, 3, (V,)).float()
    x[2, ::2] = -0.0
    x[3] = torch.finfo(TYPES[dtype]).min
    x[4] = torch.finfo(TYPES[dtype]).min
    x[4, V // 2] = 1.0
    tokens = torch.tensor([[0, V - 1]] * 5, dtype=torch.int32)
    check_logprobs(qmm, x.to(TYPES[dtype]).to(cuda), tokens.to(cuda), 32, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,V,k", [(2, 600001, 32), (1, 1100003, 20), (1, 262144, 2), (3, 2048, 32), (5, 2052, 31),
                                   (930, 2500, 32), (930, 700, 1), (320, 16380, 20), (320, 17001, 20), (2, 33, 32)])
def test_logprobs_many(qmm, cuda, M, V, k, dtype):
    """Rows of several steps, and the limits between the blocks that take them."""
    test_logprobs(qmm, cuda, M, V, k, 1.0, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logprobs_many_long_rows(qmm, cuda, dtype):
    """More long rows than the GPU takes at once; a few of them against the oracle,
    the others against calls of few rows, whose alternatives are the same."""
    g = torch.Generator(device=cuda).manual_seed(3)
    x = torch.randn((1000, 140001), generator=g, device=cuda).to(TYPES[dtype])
    x[5] = -float("inf")
    x[7, :-3] = torch.finfo(TYPES[dtype]).min
    x[9] = 1.0
    tokens = torch.randint(0, 140001, (1000, 2), generator=g, device=cuda, dtype=torch.int32)
    got = qmm.token_logprobs(x, tokens, top_k=32)
    rows = torch.tensor([0, 5, 7, 9, 500, 999], device=cuda)
    want, tol = O.logprobs(f64(x[rows]), tokens[rows].cpu().numpy(), 32, 1.0)
    close(got[0][rows], want["logprobs"], tol["logprobs"], 0.0, "logprobs")
    close(got[1][rows], want["entropy"], tol["entropy"], 0.0, "entropy")
    assert np.array_equal(got[2][rows].cpu().numpy(), want["ids"])
    close(got[3][rows], want["top"], tol["top"], 0.0, "top_logprobs")
    few = torch.cat([qmm.token_logprobs(x[i:i + 200], top_k=32)[2] for i in range(0, 1000, 200)])
    assert torch.equal(got[2], few)


@pytest.mark.parametrize("order", ["rising", "falling"])
def test_logprobs_sorted_rows(qmm, cuda, order):
    """Rows in order of value: every tile replaces the alternatives, or none does."""
    x = torch.linspace(-20, 20, 120001)
    x = torch.stack([x if order == "rising" else x.flip(0)] * 170)     # one block per row
    check_logprobs(qmm, x[:3].to(cuda), None, 32, 1.0)
    got = qmm.token_logprobs(x.to(cuda), top_k=32)
    want = torch.arange(120000, 119968, -1) if order == "rising" else torch.arange(32)
    assert torch.equal(got[2].cpu(), want.to(torch.int32).expand(170, 32))


def test_logprobs_masked(qmm, cuda):
    inf = float("inf")
    x = torch.randn((8, 33000)) * 2
    x[0] = -inf
    x[1, 5:] = -inf
    x[2, :] = -inf
    x[2, 32999] = 1.0
    x[3, 7] = float("nan")
    x[4, 20000] = inf
    x[5, 100:32000] = -inf
    x[6, :16500] = -inf
    x[7, :] = -inf
    x[7, 4] = float("nan")
    tokens = torch.tensor([[0, 7, 32999]] * 8, dtype=torch.int32)
    got = check_logprobs(qmm, x.to(cuda), tokens.to(cuda), 9, 1.0)
    assert (got[2][[0, 3, 4, 7]] == -1).all() and torch.isnan(got[1][[0, 3, 4, 7]]).all()
    assert float(got[0][2, 2]) == 0.0 and float(got[1][2]) == 0.0 and float(got[0][2, 0]) == -inf


def test_logprobs_next_to_zero(qmm, cuda):
    """One token far above the rest: its log probability keeps its relative accuracy."""
    x = torch.randn((6, 40000))
    x[torch.arange(6), torch.arange(6) * 7000] += torch.tensor([20.0, 30.0, 40.0, 60.0, 80.0, 120.0])
    tokens = (torch.arange(6) * 7000).to(torch.int32)[:, None]
    got = check_logprobs(qmm, x.to(cuda), tokens.to(cuda), 2, 1.0)
    want, _ = O.logprobs(f64(x), tokens.numpy(), 0, 1.0)
    rel = np.abs(got[0].double().cpu().numpy() / want["logprobs"] - 1)[:5]
    assert rel.max() <= (4 + 40000 / 512 + 64 + 3 * 1.4427 * 90) * O.U32


def test_logprobs_skipped_and_bad_tokens(qmm, cuda):
    x = torch.randn((4, 500), device=cuda)
    tokens = torch.tensor([[3, -1], [-1, -1], [499, 0], [1, 2]], dtype=torch.int32, device=cuda)
    out = torch.full((4, 2), 55.0, device=cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    qmm.token_logprobs(x, tokens, logprobs=out, dev_status=status)
    assert int(status) == 0 and (out[tokens == -1] == 55.0).all() and (out[tokens != -1] < 0).all()
    for bad in (500, -2, 2 ** 31 - 1):
        tokens[3, 1] = bad
        out.fill_(55.0)
        status.zero_()
        qmm.token_logprobs(x, tokens, logprobs=out, dev_status=status)
        assert int(status) == qmm.QMM_ERR_INVALID_ARG and float(out[3, 1]) == 55.0 and float(out[3, 0]) < 0


def test_logprobs_many_rows_past_32_bits(qmm, cuda):
    ld = 1 << 30
    store = torch.empty(2 * ld + 300, dtype=torch.bfloat16, device=cuda)
    x = torch.as_strided(store, (3, 300), (ld, 1))
    x.copy_(torch.randn((3, 300), device=cuda))
    check_logprobs(qmm, x, torch.tensor([[1], [2], [299]], dtype=torch.int32, device=cuda), 4, 1.0)


# ---------------------------------------------------------------------------
# captured, on another stream, and together
# ---------------------------------------------------------------------------

def test_captured_and_replayed(qmm, cuda):
    """All three in one graph, replayed on new contents of the same buffers."""
    a, _ = norm_case(cuda, 30, 256, "f32", "f32", "rms", None, "rms", "bf16")
    kw = {k: v for k, v in a.items() if k not in ("residual", "branch")}
    b = lora_case(cuda, 30, 256, 520, 4, 16, False)
    total, x = torch.empty_like(a["residual"]), torch.empty((30, 256), dtype=torch.bfloat16, device=cuda)
    ws = torch.empty(qmm.lora_add_workspace_size(30, 256, 520, 4, 16), dtype=torch.uint8, device=cuda)
    out = torch.empty((30, 520), device=cuda)
    tokens = torch.randint(0, 520, (30, 2), device=cuda, dtype=torch.int32)
    lp, ent = torch.empty((30, 2), device=cuda), torch.empty(30, device=cuda)
    ids, top = torch.empty((30, 4), dtype=torch.int32, device=cuda), torch.empty((30, 4), device=cuda)

    def step():
        qmm.block_norm(a["residual"], a["branch"], residual_out=total, out=x, **kw)
        qmm.lora_add(x, b["ids"], b["A"], b["B"], base=b["base"], out=out, ranks=b["ranks"], scales=b["scales"],
                     workspace=ws)
        qmm.token_logprobs(out, tokens, top_k=4, logprobs=lp, entropy=ent, top_ids=ids, top_logprobs=top)
        return [t.clone() for t in (total, x, out, lp, ent, ids, top)]

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for seed in (5, 6):
        fresh, _ = norm_case(cuda, 30, 256, "f32", "f32", "rms", None, "rms", "bf16", seed=seed)
        a["residual"].copy_(fresh["residual"])
        a["branch"].copy_(fresh["branch"])
        b["ids"].copy_(torch.randint(-1, 4, (30,), device=cuda))
        want = step()
        for t in (total, x, out, lp, ent, ids, top):
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for w, t in zip(want, (total, x, out, lp, ent, ids, top)):
            assert torch.equal(w, t)


@pytest.mark.parametrize("M", [600, 1700])
def test_on_two_streams_at_once(qmm, cuda, M):
    """Calls on two streams, none of them the default, with a workspace each."""
    cases = [(lora_case(cuda, M, 512, 516, 4, 200, True, seed=i), lora_case(cuda, 90, 512, 516, 4, 30, False, seed=i),
              norm_case(cuda, 300, 1024, "f32", "f32", "rms", "token", "rms", "bf16", seed=i)[0]) for i in (0, 1)]

    def step(i):
        many, few, a = cases[i]
        kw = {k: v for k, v in a.items() if k not in ("residual", "branch")}
        x, y = qmm.lora_add(**many), qmm.lora_add(**few)
        z = qmm.block_norm(a["residual"], a["branch"], residual_out=torch.empty_like(a["residual"]), **kw)
        return [x, y, *z[:2], *qmm.token_logprobs(x, top_k=5)[1:]]

    want = [step(0), step(1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in (0, 1):
        for run in got[i]:
            for w, t in zip(want[i], run):
                assert torch.equal(w, t)


def test_two_graphs_share_a_workspace(qmm, cuda):
    """Two captured calls of different sizes in one workspace, replayed in turn."""
    cases = [lora_case(cuda, 2000, 512, 516, 6, 40, False), lora_case(cuda, 500, 256, 260, 3, 200, True)]
    ws = torch.empty(max(qmm.lora_add_workspace_size(2000, 512, 516, 6, 40),
                         qmm.lora_add_workspace_size(500, 256, 260, 3, 200)), dtype=torch.uint8, device=cuda)
    want = [qmm.lora_add(**a) for a in cases]
    outs, graphs = [torch.empty_like(w) for w in want], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for a, out in zip(cases, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                qmm.lora_add(**a, out=out, workspace=ws)
        graphs.append(graph)
    torch.cuda.current_stream().wait_stream(side)
    ws.fill_(0xFF)                           # nothing is expected of a workspace's contents
    for _ in range(4):
        for out in outs:
            out.fill_(0)
        for graph in graphs:
            graph.replay()
        for w, out in zip(want, outs):
            assert torch.equal(w, out)
