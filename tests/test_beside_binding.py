"""CPU tests of the binding of what runs beside the projections: what it makes itself
and what it says of a call that it or the library refuses."""
import math

import pytest
import torch

F, BF, I32 = torch.float32, torch.bfloat16, torch.int32
P = 1 << 20          # an aligned address that nothing reads


@pytest.fixture
def calls(qmm, monkeypatch):
    """The calls that reach the library; host tensors pass for the device's."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, args)) or qmm.QMM_OK

    monkeypatch.setattr(qmm, "lib", Lib())
    monkeypatch.setattr(qmm, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(qmm, "_current_device", lambda: -1)
    return seen


def test_log_probabilities_made_here_are_written_throughout(qmm, calls):
    """Skipped tokens' places are NaN where the binding makes them, not what the memory
    held, and as they were where they are given."""
    for tokens in (torch.full((64, 3), -1, dtype=I32), torch.full((64,), -1, dtype=I32)):
        lp = qmm.token_logprobs(torch.zeros(64, 16), tokens)[0]
        name, args = calls.pop()
        assert name == "qmm_token_logprobs_or" and math.isnan(args[15]) and args[9] == lp.data_ptr()
        given = torch.full(tokens.shape, 5.0)
        assert qmm.token_logprobs(torch.zeros(64, 16), tokens, logprobs=given)[0] is given
        assert calls.pop()[0] == "qmm_token_logprobs"
    qmm.token_logprobs(torch.zeros(64, 16), top_k=3)
    assert calls.pop()[0] == "qmm_token_logprobs"


def test_refusals_with_a_value_for_other_tokens(qmm):
    base = dict(x=P, type=qmm.QMM_F32, M=3, V=50, ld=50, scale=1.0, tokens=P, ldt=2, G=2, lp=P, ent=P, k=4, ids=P,
                top=P, status=None, other=math.nan)

    def call(**over):
        return qmm.lib.qmm_token_logprobs_or(*{**base, **over}.values(), None)

    for over in (dict(x=None), dict(type=qmm.QMM_S8), dict(ld=49), dict(scale=0.0), dict(tokens=None), dict(lp=P + 2),
                 dict(k=-1), dict(top=None), dict(ent=None, G=0, k=0)):
        assert call(**over) == qmm.QMM_ERR_INVALID_ARG, over
    assert call(k=33) == qmm.QMM_ERR_UNSUPPORTED and call(M=0) == qmm.QMM_OK


def test_scales_whose_product_with_log2_e_is_infinite(qmm):
    """0 times that product would be NaN for a row's largest logit."""
    def call(entry, scale, *more):
        return getattr(qmm.lib, entry)(P, qmm.QMM_F32, 0, 50, 50, scale, P, 2, 2, P, P, 4, P, P, None, *more, None)

    for scale in (1.702e38, 2.4e38, 3.4e38, math.inf):
        assert call("qmm_token_logprobs", scale) == qmm.QMM_ERR_INVALID_ARG
        assert call("qmm_token_logprobs_or", scale, 0.0) == qmm.QMM_ERR_INVALID_ARG
    for scale in (2.0 ** 127, 1e30, 1e-45):
        assert call("qmm_token_logprobs", scale) == qmm.QMM_OK


def test_adapters_off_the_16_bytes_are_named(qmm, monkeypatch):
    """The library refuses them; the binding says which tensor and why."""
    monkeypatch.setattr(qmm, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(qmm, "_current_device", lambda: -1)
    z = lambda *shape: torch.zeros(shape, dtype=BF)
    ok = dict(X=z(4, 16), ids=torch.zeros(4, dtype=I32), A=z(3, 5, 16), B=z(3, 24, 8)[:, :, :5])
    for name, bad in (("B", z(3, 24, 5)), ("B", z(3, 24, 12)[:, :, :5]), ("A", z(3, 5, 20)[:, :, :16]),
                      ("X", z(4, 20)[:, :16]), ("X", z(4, 32)[:, 3:19]), ("A", z(3, 5, 24)[:, :, 4:20])):
        with pytest.raises(ValueError, match=f"lora_add: {name} has to begin at 16 bytes"):
            qmm.lora_add(**{**ok, name: bad})
    with pytest.raises(qmm.QmmError, match="qmm_lora_add"):  # another reason keeps the library's own word
        qmm.lora_add(**ok, base=torch.zeros(1, 24).expand(4, 24))


def test_an_unknown_output_type_is_refused(qmm, calls):
    """As an unknown norm is; it gave fp32."""
    for name in ("fp32", "f16", "int8", None):
        with pytest.raises(KeyError):
            qmm.block_norm(torch.zeros(4, 16), out_type=name)
    assert not calls
    for name, dtype in (("bf16", BF), ("f32", F), ("s8", torch.int8)):
        assert qmm.block_norm(torch.zeros(4, 16), out_type=name)[1].dtype == dtype
