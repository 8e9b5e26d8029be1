"""CPU tests of what runs beside the projections: bad arguments are refused on the
host before anything touches the GPU, by the entry points and by their Python
wrappers."""
import ctypes

import pytest
import torch

P, U, H = 1 << 20, (1 << 20) + 2, (1 << 20) + 1   # aligned, off a word, off a half-word; never dereferenced
F, BF, I32 = torch.float32, torch.bfloat16, torch.int32


def norm(qmm, kind=1, eps=1e-6, weight=None, bias=None):
    return ctypes.byref(qmm.QmmNorm(kind, eps, weight, bias))


def test_norm_refusals(qmm):
    F32, B16, S8, I, N = qmm.QMM_F32, qmm.QMM_BF16, qmm.QMM_S8, qmm.QMM_ERR_INVALID_ARG, qmm.QMM_ERR_UNSUPPORTED
    base = dict(r=P, rt=F32, ldr=64, b=P + 4096, bt=F32, ldb=64, bn=norm(qmm), g=P, gt=B16, ldg=0, scale=1.0, s=P,
                lds=64, n=norm(qmm), o=P + 8192, ot=B16, ldo=64, s_x=None, T=4, D=64)

    def call(**over):
        a = {**base, **over}
        return qmm.lib.qmm_block_norm(*a.values(), None)

    nan, inf = float("nan"), float("inf")
    for over in (dict(r=None), dict(r=U), dict(rt=S8), dict(rt=0), dict(ldr=63), dict(ldr=-64), dict(ldr=1 << 60),
                 dict(b=U), dict(bt=S8), dict(ldb=63), dict(bn=norm(qmm, 0)), dict(bn=norm(qmm, 3)),
                 dict(bn=norm(qmm, eps=-1.0)), dict(bn=norm(qmm, eps=nan)), dict(bn=norm(qmm, eps=inf)),
                 dict(bn=norm(qmm, weight=U)), dict(bn=norm(qmm, bias=U)), dict(g=H), dict(gt=S8), dict(ldg=63),
                 dict(ldg=-1), dict(scale=nan), dict(scale=inf), dict(s=U), dict(lds=63), dict(s=None, o=None),
                 dict(ldr=64, lds=72), dict(n=norm(qmm, 7)), dict(o=H), dict(ot=qmm.QMM_S32), dict(ldo=63),
                 dict(o=P), dict(o=P + 4096), dict(ot=S8), dict(ot=S8, s_x=U), dict(ot=S8, s_x=P, ldo=72),
                 dict(ot=S8, s_x=P, o=P + 8200), dict(T=-1), dict(D=0)):
        assert call(**over) == I, over
    for over in (dict(D=32769, ldr=40000, ldb=40000, lds=40000, ldo=40000), dict(T=1 << 31)):
        assert call(**over) == N, over
    assert call(T=0) == qmm.QMM_OK and call(T=0, r=None, s=None, o=None, b=None) == qmm.QMM_OK


def lora_set(qmm, **over):
    a = dict(A=P, a_slot=1024, a_rank=64, B=P, b_slot=1600, b_row=16, ranks=P, scales=P, n=3, rank=16, K=64, N=100)
    a.update(over)
    return qmm.QmmLoraSet(*a.values())


def test_lora_refusals(qmm):
    I, N, W = qmm.QMM_ERR_INVALID_ARG, qmm.QMM_ERR_UNSUPPORTED, qmm.QMM_ERR_WORKSPACE
    need = qmm.lora_add_workspace_size(500, 64, 100, 3, 16)
    base = dict(X=P, ldx=64, ids=P, M=500, base=P, ldb=100, out=P, ldo=100, ws=P, ws_bytes=need)

    def call(s=None, **over):
        a = {**base, **over}
        s = lora_set(qmm) if s is None else s
        return qmm.lib.qmm_lora_add(ctypes.byref(s), *a.values(), None, None)

    for over in (dict(X=None), dict(X=P + 8), dict(ldx=60), dict(ldx=68), dict(ids=None), dict(ids=U), dict(M=-1),
                 dict(base=U), dict(ldb=99), dict(out=None), dict(out=U), dict(ldo=99), dict(ldb=104)):
        assert call(**over) == I, over
    for over in (dict(A=None), dict(A=P + 8), dict(a_slot=1028), dict(a_rank=60), dict(a_rank=56), dict(a_slot=-8),
                 dict(B=None), dict(B=P + 8), dict(b_slot=1604), dict(b_row=20), dict(b_row=8), dict(ranks=U),
                 dict(scales=U), dict(n=0), dict(rank=0), dict(K=0), dict(N=0)):
        assert call(lora_set(qmm, **over)) == I, over
    for over in (dict(K=60), dict(rank=257, b_row=264), dict(n=8193), dict(K=1 << 28, a_rank=1 << 28), dict(N=1 << 24)):
        assert call(lora_set(qmm, **over)) == N, over
    assert call(M=1 << 24) == N
    for over in (dict(ws=None), dict(ws=P + 128), dict(ws_bytes=need - 1)):
        assert call(**over) == W, over
    assert call(M=0) == qmm.QMM_OK and call(M=0, X=None, ids=None, out=None, base=None, ws=None) == qmm.QMM_OK
    assert qmm.lib.qmm_lora_add(None, *base.values(), None, None) == I
    size = ctypes.c_size_t(7)
    q = qmm.lib.qmm_lora_add_workspace_size
    assert q(0, 64, 100, 3, 16, ctypes.byref(size)) == qmm.QMM_OK and size.value == 0
    assert q(5, 64, 100, 3, 16, None) == I and q(5, 63, 100, 3, 16, ctypes.byref(size)) == N


def test_logprobs_refusals(qmm):
    I, N = qmm.QMM_ERR_INVALID_ARG, qmm.QMM_ERR_UNSUPPORTED
    base = dict(x=P, type=qmm.QMM_F32, M=3, V=50, ld=50, scale=1.0, tokens=P, ldt=2, G=2, lp=P, ent=P, k=4, ids=P, top=P)

    def call(**over):
        a = {**base, **over}
        return qmm.lib.qmm_token_logprobs(*a.values(), None, None)

    for over in (dict(x=None), dict(x=U), dict(type=qmm.QMM_S8), dict(M=-1), dict(V=0), dict(ld=49), dict(scale=0.0),
                 dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(tokens=None),
                 dict(tokens=U), dict(ldt=1), dict(G=-1), dict(lp=None), dict(lp=U), dict(ent=U), dict(k=-1),
                 dict(ids=None), dict(ids=U), dict(top=None), dict(top=U), dict(ent=None, G=0, k=0)):
        assert call(**over) == I, over
    for over in (dict(k=33), dict(V=(1 << 31) - 65536, ld=1 << 31), dict(G=1025, ldt=1025), dict(M=1 << 26)):
        assert call(**over) == N, over
    assert call(M=0) == qmm.QMM_OK
    assert call(M=0, x=None, tokens=None, lp=None, ent=None, ids=None, top=None, G=0, k=1) == qmm.QMM_OK


# ---------------------------------------------------------------------------
# the wrappers
# ---------------------------------------------------------------------------

@pytest.fixture
def calls(qmm, monkeypatch):
    """The arguments that reach the library; tensors of the host pass for the device's."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            def entry(*args):
                seen.append((name, args))
                return qmm.QMM_OK
            return entry

    monkeypatch.setattr(qmm, "lib", Lib())
    monkeypatch.setattr(qmm, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(qmm, "_current_device", lambda: -1)
    return seen


def z(*shape, dtype=F):
    return torch.zeros(shape, dtype=dtype)


def test_host_tensors_are_refused(qmm, calls, monkeypatch):
    monkeypatch.setattr(qmm, "_current_device", lambda: 0)
    for call in (lambda: qmm.block_norm(z(2, 8)), lambda: qmm.token_logprobs(z(2, 8)),
                 lambda: qmm.lora_add(z(2, 8, dtype=BF), z(2, dtype=I32), z(1, 8, 8, dtype=BF), z(1, 4, 8, dtype=BF))):
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
    assert not calls


def test_norm_wrapper(qmm, calls):
    r = z(4, 16)
    for bad in (dict(branch=z(4, 15)), dict(branch=z(3, 16)), dict(branch=z(4, 16, dtype=torch.float16)),
                dict(branch=z(16, 4).t()), dict(weight=z(15)), dict(weight=z(16, dtype=BF)), dict(weight=z(32)[::2]),
                dict(branch=z(4, 16), gate=z(15)), dict(branch=z(4, 16), gate=z(3, 16)),
                dict(branch=z(4, 16), residual_out=z(4, 16, dtype=BF)), dict(out=z(4, 8)), dict(out=z(4, 16, dtype=I32)),
                dict(out_type="s8", s_x=z(3)), dict(branch=z(4, 16), branch_norm="rms", branch_weight=z(17))):
        with pytest.raises(ValueError):
            qmm.block_norm(r, **bad)
    with pytest.raises(KeyError):
        qmm.block_norm(r, norm="batch")
    assert not calls
    total, out, s = qmm.block_norm(r, z(4, 16, dtype=BF), gate=z(16), out_type="s8", weight=z(16), bias=z(16))
    assert total is r and out.shape == (4, 16) and out.dtype == torch.int8 and s.shape == (4,)
    total, out = qmm.block_norm(z(4, 40)[:, 3:19], gate=z(4, 16))
    assert out.dtype == BF and len(calls) == 2
    args = calls[1][1]
    assert args[2] == 40 and args[3] is None and args[7] is None and args[11] is None


def test_lora_wrapper(qmm, calls):
    ok = dict(X=z(4, 16, dtype=BF), ids=z(4, dtype=I32), A=z(3, 8, 16, dtype=BF), B=z(3, 24, 8, dtype=BF),
              base=z(4, 24), ranks=z(3, dtype=I32), scales=z(3), workspace=z(64, dtype=torch.uint8))
    for bad in (dict(X=z(4, 16)), dict(X=z(4, 8, dtype=BF)), dict(X=z(16, 4, dtype=BF).t()), dict(ids=z(4, dtype=torch.int64)),
                dict(ids=z(5, dtype=I32)), dict(ids=z(8, dtype=I32)[::2]), dict(A=z(3, 8, 16)), dict(A=z(3, 8, 8, dtype=BF)),
                dict(B=z(3, 24, 16, dtype=BF)), dict(B=z(2, 24, 8, dtype=BF)), dict(B=z(3, 8, 24, dtype=BF).transpose(1, 2)),
                dict(base=z(4, 23)), dict(base=z(4, 24, dtype=BF)), dict(out=z(3, 24)), dict(ranks=z(4, dtype=I32)),
                dict(ranks=z(3)), dict(scales=z(2)), dict(dev_status=z(1))):
        with pytest.raises(ValueError):
            qmm.lora_add(**{**ok, **bad})
    assert not calls
    out = qmm.lora_add(**ok)
    assert out.shape == (4, 24) and out.dtype == F and len(calls) == 1
    assert qmm.lora_add(**ok, out=ok["base"]) is ok["base"]


def test_logprobs_wrapper(qmm, calls):
    x, t = z(4, 16), z(4, 2, dtype=I32)
    for bad in (dict(logits=z(4, 16, dtype=torch.float16)), dict(logits=z(16, 4).t()), dict(tokens=z(4, 2, dtype=torch.int64)),
                dict(tokens=z(3, 2, dtype=I32)), dict(tokens=z(2, 4, dtype=I32).t()), dict(logprobs=z(7)),
                dict(logprobs=z(8, dtype=BF)), dict(entropy=z(3)), dict(top_k=2, top_ids=z(4, 1, dtype=I32)),
                dict(top_k=2, top_logprobs=z(4, 3)), dict(dev_status=z(1))):
        with pytest.raises(ValueError):
            qmm.token_logprobs(**{"logits": x, "tokens": t, **bad})
    assert not calls
    lp, ent, ids, top = qmm.token_logprobs(x, t, top_k=3)
    assert lp.shape == (4, 2) and ent.shape == (4,) and ids.shape == top.shape == (4, 3) and ids.dtype == I32
    lp, ent, ids, top = qmm.token_logprobs(z(4, 20)[:, 1:17], z(4, dtype=I32), entropy=False)
    assert lp.shape == (4,) and ent is None and ids is None and top is None
    assert calls[1][1][4] == 20 and calls[1][1][10] is None
