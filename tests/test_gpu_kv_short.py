"""qmm_kv_plan on a free list one page short: every token but those of the page
that is missing has the slot that a full list would give it."""
import numpy as np
import pytest

import oracle.kv_oracle as KV
from test_gpu_kv import run_plan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [False, True])
def test_plan_one_page_short(qmm, cuda, tree):
    ctx, new, page = [10, 10], [30, 30], 16       # two pages each; the second request gets one
    parents = [-1] + list(range(29)) if tree else None
    parents = parents * 2 if tree else None
    got, status, base = run_plan(qmm, cuda, ctx, new, page, n_free=3, parents=parents, words=int(tree))
    assert status == qmm.QMM_ERR_NO_PAGES and got["taken"][0] == base["taken"] == 4
    ref = KV.plan(ctx, new, base["free"] + [0], base["table"], page, 60, parents, int(tree))
    assert np.array_equal(got["slots"][:52], ref["slots"][:52])
    assert (got["slots"][52:] == -1).all()        # 6 tokens beside the cached ones, 16 on its page, then none
    assert np.array_equal(got["positions"], ref["positions"]) and np.array_equal(got["mask"], ref["mask"])
    assert np.array_equal(got["table"][0], ref["table"][0]) and np.array_equal(got["table"][1, :2], ref["table"][1, :2])
