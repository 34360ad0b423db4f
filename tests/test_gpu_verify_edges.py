"""Draft verification over vocabularies so long that a part of a row is summed
in chunks of several steps."""

import pytest
import torch

from test_gpu_verify import check, inputs

pytestmark = pytest.mark.gpu
FP32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("reqs,vocab,dtype", [
    (1, 5000003, FP32),       # a cluster of 16, 611 steps a part, two a chunk
    (2, 9437184, BF16),       # 576 steps a part
    (1, 13000001, FP32),      # four steps a chunk, the last one short
    (310, 262145, FP32)])     # one CTA a request, 513 steps, two a chunk
def test_chunks_of_several_steps(mm, reqs, vocab, dtype, drafts):
    target, tokens, u, draft, _ = inputs(reqs, 1, vocab, dtype, drafts, vocab, spread=1.0)
    check(mm, target, tokens, u, draft)
    u[:, 0] = 0.0                                        # accepted: the bonus row
    check(mm, target, tokens, u, draft)


@pytest.mark.parametrize("dtype,step", [(FP32, 512), (BF16, 1024), (FP16, 1024)])
@pytest.mark.parametrize("reject", [True, False])
def test_draws_in_every_step_of_a_chunk(mm, dtype, step, reject):
    """A few likely tokens in the first, second and last steps of chunks and at a row's end; the
    refused token among them."""
    vocab = 5000 * step + 37
    at = sorted({0, 1, step - 1, step, step + 1, 2 * step - 1, 2 * step, 313 * step + 5,
                 4096 * step - 1, 4097 * step, vocab - 37, vocab - 2, vocab - 1})
    p = torch.zeros((1, 2, vocab), dtype=dtype, device="cuda")
    p[:, :, at] = 2.0 ** -4
    q = torch.zeros((1, 1, vocab), dtype=dtype, device="cuda")
    token = at[3]
    q[:, :, token] = 1.0
    tokens = torch.tensor([[token]], dtype=torch.int32, device="cuda")
    for k in range(2 * len(at)):
        u = torch.tensor([[0.9 if reject else 0.0, (k + 0.5) / (2 * len(at))]], device="cuda")
        out, accepted = check(mm, p, tokens, u, q)
        assert accepted.tolist() == [0 if reject else 1]
        assert int(out[0, 0 if reject else 1]) in at
        check(mm, p, tokens, u)
