"""GPU tests of what the binding of the operators beside the projections makes itself."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_skipped_tokens_are_nan(qmm, cuda):
    x = torch.randn((40, 500), device=cuda)
    tokens = torch.randint(0, 500, (40, 3), device=cuda, dtype=torch.int32)
    want = qmm.token_logprobs(x, tokens)[0]
    assert torch.isfinite(want).all()
    skip = torch.rand((40, 3), device=cuda) < 0.4
    skip[0, 0] = True
    bad = torch.where(skip, -1, tokens)
    bad[1] = torch.tensor([500, -2, -1], device=cuda)
    skip[1] = True
    for _ in range(3):
        got = qmm.token_logprobs(x, bad.to(torch.int32))[0]
        assert torch.equal(torch.isnan(got), skip) and torch.equal(got[~skip], want[~skip])
        del got
        torch.zeros((40, 3), device=cuda)
    row = qmm.token_logprobs(x, bad[:, 1].to(torch.int32).contiguous())[0]
    assert torch.equal(torch.isnan(row), skip[:, 1])


def test_skipped_tokens_in_a_graph(qmm, cuda):
    """A captured call: its places are NaN again where the next tokens are skipped."""
    x = torch.randn((8, 500), device=cuda)
    tokens = torch.zeros((8, 2), dtype=torch.int32, device=cuda)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        qmm.token_logprobs(x, tokens)
        with torch.cuda.graph(graph, stream=side):
            got = qmm.token_logprobs(x, tokens)[0]
    torch.cuda.current_stream().wait_stream(side)
    for skipped in (0, 1):
        tokens[:, skipped], tokens[:, 1 - skipped] = -1, 3
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isnan(got[:, skipped]).all() and torch.isfinite(got[:, 1 - skipped]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5, 3001])
def test_the_largest_scale(qmm, cuda, V, dtype):
    """All of a row's probability at its largest logits, whatever lies between them."""
    x = torch.full((3, V), -2.0, dtype=dtype, device=cuda)
    x[0, 2] = x[1, 1] = x[1, 4] = 0.5
    x[2, 3] = -float("inf")
    tokens = torch.tensor([[2, 0], [4, 0], [0, 3]], dtype=torch.int32, device=cuda)
    lp, entropy, ids, top = qmm.token_logprobs(x, tokens, top_k=3, scale=2.0 ** 127)
    n = torch.tensor([1.0, 2.0, V - 1.0], device=cuda)
    torch.testing.assert_close(entropy, n.log(), rtol=1e-6, atol=0)
    torch.testing.assert_close(lp[:, 0], -n.log(), rtol=1e-6, atol=0)
    assert (lp[:, 1] == -float("inf")).all() and ids[0].tolist() == [2, 0, 1] and ids[1].tolist() == [1, 4, 0]
    assert float(top[0, 1]) == -float("inf") and ids[2].tolist() == [0, 1, 2]
