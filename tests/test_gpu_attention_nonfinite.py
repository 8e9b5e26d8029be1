"""Infinities and NaN among the values that a row sees reach its output element
whatever their weight, as in the formula (0 times infinity is not a number): in
every kernel, in whichever cached tile they lie.

The other elements are the same, bit for bit, as without them.
"""
import numpy as np
import pytest
import torch

import oracle.kv_oracle as KV
from test_gpu_attention import build, call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("s8", [False, True])
@pytest.mark.parametrize("new,heads", [(4, 4), (9, 4), (32, 4), (25, 8), (35, 8)])
def test_seen_values_of_no_weight(qmm, cuda, new, heads, s8, bad):
    """8 to 140 query rows per key head over contexts whose cached tiles lead and
    trail in turn by more than the exponential reaches (hundreds); a cached token
    of a trailing tile has a value (int8: a value scale) that is not finite.
    Requests enough that a block has several tiles of an item."""
    kv, d, page, R = 2, 64, 16, 60
    ctx = [500 + 7 * (r % 9) for r in range(R)]
    s = build(cuda, ctx, [new] * R, heads, kv, d, page, s8, seed=new)
    s["scale"] = 1.0
    s["q"][..., 0] = 200.0
    for r, (k, v, pg, off) in enumerate(s["rows"]):
        j = torch.arange(len(k))
        leads = (j // 128) % 2 == r % 2
        row = s["k"][pg, off].float().cpu()
        row[..., 0] = torch.where(leads, 127.0 if s8 else 1.75, 0.0)[:, None]
        s["k"][pg, off] = row.to(s["k"].dtype).to(cuda)
        scale = s["ks"][pg, :, off].double().cpu() if s8 else torch.ones((len(k), kv), dtype=torch.float64)
        k[:] = row.double() * scale[..., None]
        t = 128 * (1 - r % 2) + 3 + r              # of the first or second tile, the one that trails
        if s8:
            s["vs"][pg[t], 1, off[t]] = bad
            v[t, 1] = s["v"][pg[t], off[t], 1].double().cpu() * bad
        else:
            s["v"][pg[t], off[t], 1, 5] = bad
            v[t, 1, 5] = bad
    got = call(qmm, cuda, s)
    for r, (k, v, pg, off) in enumerate(s["rows"]):   # without: that value is 0
        t = 128 * (1 - r % 2) + 3 + r
        if s8:
            s["vs"][pg[t], 1, off[t]] = 0.0
        else:
            s["v"][pg[t], off[t], 1, 5] = 0.0
    clean = call(qmm, cuda, s)
    assert torch.isfinite(clean).all()
    hit = torch.zeros((heads, d), dtype=torch.bool, device=cuda)
    hit[heads // kv:, slice(None) if s8 else 5] = True    # the elements that have the value among theirs
    got_hit = ~torch.isfinite(got)
    for (c, n, first), (k, v, _, _) in zip(s["lens"], s["rows"]):
        q = s["q"][first:first + n].to(torch.bfloat16).double().numpy()
        with np.errstate(invalid="ignore"):
            ref, _ = KV.attend(q, k.numpy(), v.numpy(), KV.visible(c, n), s["scale"])
        assert np.array_equal(~np.isfinite(ref), hit.cpu().numpy()[None].repeat(n, 0))
        assert torch.equal(got_hit[first:first + n], hit[None].expand(n, heads, d)), (c, n)
    assert torch.equal(got[:, ~hit], clean[:, ~hit])


@pytest.mark.parametrize("s8", [False, True])
def test_many_row_tiles_of_one_token(qmm, cuda, s8):
    """A new token whose 4608 query heads per key head fill 18 tiles of rows, of
    requests that end with a cached tile: only the first tile of rows has tokens
    to clean in its cached tiles, and nothing holds that warp back in the next 17.
    The token's infinity is there for every row all the same."""
    R, kv, heads, d, page = 16, 14, 14 * 4608, 64, 32
    s = build(cuda, [127] * R, [1] * R, kv, kv, d, page, s8, seed=3)
    for _, _, pg, off in s["rows"]:
        if s8:
            s["vs"][pg[127], :, off[127]] = float("inf")
            code = s["v"][pg[127], off[127]]
            code[code == 0] = 1
            s["v"][pg[127], off[127]] = code
        else:
            s["v"][pg[127], off[127], :, 5] = float("inf")
    g = torch.Generator(device=cuda).manual_seed(4)
    s["q"] = torch.randn((R, heads, d), generator=g, device=cuda).to(torch.bfloat16)
    out = call(qmm, cuda, s)
    if s8:
        assert torch.isinf(out).all()
    else:
        assert (out[..., 5] == float("inf")).all()
        assert torch.isfinite(out[..., :5]).all() and torch.isfinite(out[..., 6:]).all()
