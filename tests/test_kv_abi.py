"""CPU tests of the paged cache's entry points: bad arguments are refused on the
host before anything touches the GPU, and sizes."""
import ctypes

import pytest
import torch

P, U = 1 << 20, (1 << 20) + 2          # aligned and misaligned addresses, never dereferenced


def test_plan_refusals(qmm):
    base = dict(ctx=P, new=P, R=4, free=P, n_free=3, table=P, ld=8, blocks=8, page=16, parents=None, mask=None,
                ld_mask=0, words=0, tokens=10, cu=P, slots=P, pos=P, taken=P)

    def call(**over):
        a = {**base, **over}
        return qmm.lib.qmm_kv_plan(a["ctx"], a["new"], a["R"], a["free"], a["n_free"], a["table"], a["ld"],
                                   a["blocks"], a["page"], a["parents"], a["mask"], a["ld_mask"], a["words"],
                                   a["tokens"], a["cu"], a["slots"], a["pos"], a["taken"], None, None)

    tree = dict(parents=P, mask=P, ld_mask=2, words=2)
    for over in (dict(ctx=None), dict(new=None), dict(table=None), dict(cu=None), dict(slots=None), dict(pos=None),
                 dict(taken=None), dict(free=None), dict(R=0), dict(R=-1), dict(n_free=-1), dict(blocks=0),
                 dict(ld=7), dict(page=0), dict(tokens=-1), dict(ctx=U), dict(new=U), dict(table=U), dict(cu=U),
                 dict(pos=U), dict(taken=U), dict(free=U), dict(slots=P + 4),
                 dict(parents=P), dict(mask=P, ld_mask=2, words=2), {**tree, "words": 0}, {**tree, "ld_mask": 1},
                 {**tree, "parents": U}, {**tree, "mask": U}, dict(words=1)):
        assert call(**over) == qmm.QMM_ERR_INVALID_ARG, over
    for over in (dict(R=16385), dict(page=1 << 31), dict(tokens=1 << 31)):
        assert call(**over) == qmm.QMM_ERR_UNSUPPORTED, over


def cache(qmm, **over):
    a = dict(k=P, v=P, k_scale=None, v_scale=None, type=qmm.QMM_BF16, n_pages=4, page_size=16, n_heads=2,
             head_dim=128, stride_page=4096, stride_token=256, stride_head=128)
    a.update(over)
    return qmm.QmmKvCache(*a.values())


def bad_caches(qmm):
    I, N = qmm.QMM_ERR_INVALID_ARG, qmm.QMM_ERR_UNSUPPORTED
    return [(dict(k=None), I), (dict(v=None), I), (dict(k=P + 8), I), (dict(v=P + 8), I), (dict(type=qmm.QMM_F32), I),
            (dict(type=qmm.QMM_S8), I), (dict(type=qmm.QMM_S8, k_scale=P), I),
            (dict(type=qmm.QMM_S8, k_scale=P, v_scale=U), I), (dict(n_pages=0), I), (dict(page_size=0), I),
            (dict(n_heads=0), I), (dict(head_dim=96), N), (dict(head_dim=256), N), (dict(stride_page=4097), I),
            (dict(stride_token=252), I), (dict(stride_head=132), I), (dict(stride_token=-256), I),
            (dict(stride_head=64), I), (dict(stride_token=64), I), (dict(stride_page=64), I),
            (dict(page_size=1 << 30), N)]


def test_append_refusals(qmm):
    base = dict(K=P, kt=256, kh=128, V=P, vt=256, vh=128, type=qmm.QMM_BF16, T=5, slots=P)

    def call(c=None, **over):
        a = {**base, **over}
        c = cache(qmm) if c is None else c
        return qmm.lib.qmm_kv_append(a["K"], a["kt"], a["kh"], a["V"], a["vt"], a["vh"], a["type"], a["T"],
                                     a["slots"], ctypes.byref(c), None, None)

    for over in (dict(K=None), dict(V=None), dict(slots=None), dict(K=P + 8), dict(V=P + 8), dict(slots=P + 4),
                 dict(T=-1), dict(type=qmm.QMM_S8), dict(kt=252), dict(kh=132), dict(vt=252), dict(vh=132),
                 dict(kt=-256)):
        assert call(**over) == qmm.QMM_ERR_INVALID_ARG, over
    for over, status in bad_caches(qmm):
        assert call(cache(qmm, **over)) == status, over
    assert call(T=1 << 31) == qmm.QMM_ERR_UNSUPPORTED
    assert call(T=0) == qmm.QMM_OK and call(T=0, K=None, V=None, slots=None) == qmm.QMM_OK
    assert qmm.lib.qmm_kv_append(P, 256, 128, P, 256, 128, qmm.QMM_BF16, 5, P, None, None,
                                 None) == qmm.QMM_ERR_INVALID_ARG


def test_attention_refusals(qmm):
    need = qmm.tree_attention_workspace_size(4, 2, 128, 3)
    base = dict(q=P, q_type=qmm.QMM_BF16, qt=512, qh=128, heads=4, table=P, ld=8, blocks=8, ctx=P, cu=P, R=2, T=5,
                max_new=3, mask=None, ld_mask=0, scale=0.1, out=P, ot=512, oh=128, ws=P, ws_bytes=need)

    def call(c=None, **over):
        a = {**base, **over}
        c = cache(qmm) if c is None else c
        return qmm.lib.qmm_tree_attention(a["q"], a["q_type"], a["qt"], a["qh"], a["heads"], ctypes.byref(c),
                                          a["table"], a["ld"], a["blocks"], a["ctx"], a["cu"], a["R"], a["T"],
                                          a["max_new"], a["mask"], a["ld_mask"], a["scale"], a["out"], a["ot"],
                                          a["oh"], a["ws"], a["ws_bytes"], None, None)

    nan, inf = float("nan"), float("inf")
    for over in (dict(q=None), dict(table=None), dict(ctx=None), dict(cu=None), dict(out=None), dict(q=P + 8),
                 dict(out=P + 8), dict(table=U), dict(ctx=U), dict(cu=U), dict(mask=U, ld_mask=1), dict(heads=3),
                 dict(heads=0), dict(R=0), dict(T=-1), dict(max_new=0), dict(blocks=0), dict(ld=7), dict(scale=0.0),
                 dict(scale=-1.0), dict(scale=nan), dict(scale=inf), dict(q_type=qmm.QMM_S8), dict(qt=508),
                 dict(qh=130), dict(ot=508), dict(oh=130), dict(oh=64), dict(ot=64), dict(mask=P, ld_mask=0),
                 dict(mask=P, ld_mask=1, max_new=33), dict(qt=-512)):
        assert call(**over) == qmm.QMM_ERR_INVALID_ARG, over
    for over in (dict(ws=None), dict(ws=P + 128), dict(ws_bytes=need - 1), dict(ws_bytes=0)):
        assert call(**over) == qmm.QMM_ERR_WORKSPACE, over
    for over, status in bad_caches(qmm):
        assert call(cache(qmm, **over)) == status, over
    for over in (dict(R=1 << 30), dict(T=1 << 30), dict(max_new=1 << 30), dict(heads=1 << 17)):
        assert call(**over) == qmm.QMM_ERR_UNSUPPORTED, over
    assert call(T=0) == qmm.QMM_OK


def test_attention_workspace_size(qmm):
    sz = ctypes.c_size_t(0)
    f = lambda *a: qmm.lib.qmm_tree_attention_workspace_size(*a, ctypes.byref(sz))
    assert f(4, 2, 128, 1) == qmm.QMM_OK and sz.value > 0
    assert f(4, 3, 128, 1) == qmm.QMM_ERR_INVALID_ARG
    assert f(4, 0, 128, 1) == qmm.QMM_ERR_INVALID_ARG
    assert f(4, 2, 128, 0) == qmm.QMM_ERR_INVALID_ARG
    assert f(4, 2, 96, 1) == qmm.QMM_ERR_UNSUPPORTED
    assert qmm.lib.qmm_tree_attention_workspace_size(4, 2, 128, 1, None) == qmm.QMM_ERR_INVALID_ARG


def test_binding_checks_shapes(qmm):
    """Shapes that do not agree are refused in Python, before the call."""
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros((2, 4, 2, 64), dtype=bf)
    q = torch.zeros((3, 4, 64), dtype=bf)
    t, ctx, cu = torch.zeros((1, 2), dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(2, dtype=i32)
    for bad in (dict(v=torch.zeros((2, 4, 2, 64), dtype=torch.int8)), dict(v=k.permute(0, 2, 1, 3)),
                dict(cu=torch.zeros(3, dtype=i32)), dict(t=torch.zeros((2, 2), dtype=i32)),
                dict(q=torch.zeros((3, 4, 32), dtype=bf)), dict(mask=torch.zeros((2, 1), dtype=i32)),
                dict(out=torch.zeros((3, 4, 64)))):
        a = {**dict(q=q, k=k, v=k, t=t, ctx=ctx, cu=cu, mask=None, out=None), **bad}
        with pytest.raises(ValueError):
            qmm.tree_attention(a["q"], a["k"], a["v"], a["t"], a["ctx"], a["cu"], 3, mask=a["mask"], out=a["out"])
    k8 = k.to(torch.int8)
    rows, slots = torch.zeros((3, 2, 64)), torch.zeros(3, dtype=torch.int64)
    sc = torch.zeros((2, 2, 4))
    for bad in (dict(ks=None), dict(vs=torch.zeros((2, 4, 2))), dict(ks=sc.double()), dict(K=rows[:2]),
                dict(slots=slots[:2]), dict(K=torch.zeros((3, 2, 32)), V=torch.zeros((3, 2, 32)))):
        a = {**dict(K=rows, V=rows, slots=slots, ks=sc, vs=sc), **bad}
        with pytest.raises(ValueError):
            qmm.kv_append(a["K"], a["V"], a["slots"], k8, k8, k_scale=a["ks"], v_scale=a["vs"])
    with pytest.raises(ValueError):
        qmm.kv_plan(ctx, torch.zeros(2, dtype=i32), ctx, t, 4, slots, torch.zeros(3, dtype=i32))
