"""CPU tests of the paged cache's documented limits: refused from there on, and
taken just below where a call of no tokens can show it (it launches nothing)."""
import ctypes

import pytest

P = 1 << 20                              # an aligned address, never dereferenced


def cache(qmm, **over):
    a = dict(k=P, v=P, k_scale=None, v_scale=None, type=qmm.QMM_BF16, n_pages=4, page_size=16, n_heads=2,
             head_dim=128, stride_page=1 << 40, stride_token=1 << 24, stride_head=128)
    a.update(over)
    return qmm.QmmKvCache(*a.values())


def append(qmm, T, c):
    return qmm.lib.qmm_kv_append(P, 1 << 24, 128, P, 1 << 24, 128, qmm.QMM_BF16, T, P, ctypes.byref(c), None, None)


def attend(qmm, T, c, heads=None, R=1, max_new=1):
    heads = c.n_heads if heads is None else heads
    return qmm.lib.qmm_tree_attention(P, qmm.QMM_BF16, 1 << 24, 128, heads, ctypes.byref(c), P, 1, 1, P, P, R, T,
                                      max_new, None, 0, 0.1, P, 1 << 24, 128, P, 0, None, None)


@pytest.mark.parametrize("name,most", [("page_size", (1 << 30) - 1), ("n_heads", 65535), ("n_pages", (1 << 31) - 1)])
def test_cache(qmm, name, most):
    for call in (append, attend):
        assert call(qmm, 0, cache(qmm, **{name: most})) == qmm.QMM_OK
        assert call(qmm, 0, cache(qmm, **{name: most + 1})) == qmm.QMM_ERR_UNSUPPORTED


def test_append(qmm):
    assert append(qmm, 1 << 31, cache(qmm, n_heads=1)) == qmm.QMM_ERR_UNSUPPORTED
    # T * n_heads = 8 * (2^31 - 1)
    assert append(qmm, (1 << 31) - 1, cache(qmm, n_heads=8)) == qmm.QMM_ERR_UNSUPPORTED


def test_attention(qmm):
    one = cache(qmm, n_heads=1)
    assert attend(qmm, 0, one, heads=65535) == qmm.QMM_OK
    assert attend(qmm, 0, one, heads=65536) == qmm.QMM_ERR_UNSUPPORTED
    assert attend(qmm, 0, one, R=(1 << 30) - 1) == qmm.QMM_OK
    assert attend(qmm, 0, one, R=1 << 30) == qmm.QMM_ERR_UNSUPPORTED
    assert attend(qmm, 1 << 30, one) == qmm.QMM_ERR_UNSUPPORTED
    for heads in (1, 7, 1000):
        edge = (1 << 30) // heads
        assert attend(qmm, 0, one, heads=heads, max_new=edge - 1) == qmm.QMM_OK
        assert attend(qmm, 0, one, heads=heads, max_new=edge) == qmm.QMM_ERR_UNSUPPORTED


def test_plan(qmm):
    def call(R=1, page=16, tokens=1, words=1):
        return qmm.lib.qmm_kv_plan(P, P, R, P, 1, P, 1, 1, page, P, P, words, words, tokens, P, P, P, P, None, None)

    for over in (dict(R=16385), dict(page=1 << 31), dict(tokens=(1 << 31) - 1), dict(words=(1 << 20) + 1)):
        assert call(**over) == qmm.QMM_ERR_UNSUPPORTED, over
