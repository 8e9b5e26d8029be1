"""Equal logits in rows that a warp reads in several steps per segment: pieces of a
segment then lie between one another's steps, and alternatives still fall by rising index."""
import pytest
import torch

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
K = 32


def check(qmm, dev, M, V, dtype, high, first, every, tops=(2, K)):
    """Row r: -5, logits of 3 at the places `high`, and 0 from first + every * r to the end: the
    alternatives are those places and then the run's, all by rising index."""
    start = (first + every * torch.arange(M, device=dev))[:, None]
    at = torch.arange(V, device=dev)[None]
    x = torch.empty((M, V), dtype=TYPES[dtype], device=dev)
    for r in range(0, M, 64):                # without M x V intermediates of eight bytes
        x[r:r + 64] = torch.where(at >= start[r:r + 64], 0.0, -5.0)
    assert max(high) < first and first + every * (M - 1) + K <= V
    x[:, list(high)] = 3.0
    want = torch.cat([torch.tensor(sorted(high), device=dev).expand(M, -1), start + torch.arange(K, device=dev)], 1)
    for k in tops:
        got = qmm.token_logprobs(x, entropy=False, top_k=k)[2]
        assert torch.equal(got.long(), want[:, :k]), (k, (got.long() != want[:, :k]).any(1).nonzero()[:5].flatten())


# one row per block of four warps: more than three times the rows that the long blocks take at once
@pytest.mark.parametrize("dtype,V", [("bf16", 530001), ("bf16", 600000), ("bf16", 600001), ("bf16", 1200000),
                                     ("f32", 270001), ("f32", 800001)])
@pytest.mark.parametrize("high", [(5,), (5, 1700), (40, 300, 1000, 2000)], ids=lambda h: f"{len(h)}high")
def test_many_rows(qmm, cuda, dtype, V, high):
    M = 6 * torch.cuda.get_device_properties(cuda).multi_processor_count + 18
    check(qmm, cuda, M, V, dtype, high, 2048, 128)


# one row per cluster of blocks of 16 warps
@pytest.mark.parametrize("dtype,V", [("f32", 1100003), ("f32", 4000003), ("bf16", 4000003), ("bf16", 8000000)])
@pytest.mark.parametrize("high", [(5,), (5, 9000, 20000)], ids=lambda h: f"{len(h)}high")
def test_few_rows(qmm, cuda, dtype, V, high):
    check(qmm, cuda, 40, V, dtype, high, 24000, 256)


def test_places_between_steps(qmm, cuda):
    """Lone logits in several pieces of a segment, and whole steps of equal ones of which
    the one in the later piece comes first."""
    M = 6 * torch.cuda.get_device_properties(cuda).multi_processor_count + 18
    V, unit, step = 600001, 256, 1024        # bf16: a piece's step, a segment's step
    x = torch.full((V,), -5.0)
    base = 2 * step                          # the second segment
    x[3 * unit + 7] = 5.0
    x[base + step:base + step + unit] = 5.0                   # its first piece, second step
    x[base + unit + 11] = x[base + 2 * unit + 3] = 5.0
    x[base + 3 * unit:base + 4 * unit] = 5.0                  # its last piece, first step
    want = torch.sort(x, descending=True, stable=True).indices[:K]
    got = qmm.token_logprobs(x.to(torch.bfloat16).to(cuda).expand(M, V).contiguous(), entropy=False, top_k=K)[2]
    assert torch.equal(got.cpu().long(), want.expand(M, K))
    got = qmm.token_logprobs(x.to(torch.bfloat16).to(cuda)[None], entropy=False, top_k=K)[2]
    assert torch.equal(got.cpu().long(), want[None])
