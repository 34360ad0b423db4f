"""mm3idx_verify_drafts against the same rule in exact integers: every token
and count equal."""

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu
FP32, BF16, FP16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def inputs(reqs, k, vocab, dtype, drafts, seed, spread=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = spread * torch.randn((reqs, k + 1, vocab), generator=g, device="cuda")
    target = torch.softmax(logits, -1).to(dtype)
    low = logits[:, :k] + 0.8 * torch.randn((reqs, k, vocab), generator=g, device="cuda")
    draft = torch.softmax(low, -1).to(dtype) if drafts else None
    noise = -torch.log(-torch.log(torch.rand((reqs, k, vocab), generator=g, device="cuda")
                                  .clamp(1e-20, 1 - 1e-7)))
    tokens = (low + noise).argmax(-1).to(torch.int32) if k else \
        torch.zeros((reqs, 0), dtype=torch.int32, device="cuda")
    u = torch.rand((reqs, k + 1), generator=g, device="cuda")
    lens = torch.randint(0, k + 1, (reqs,), generator=g, device="cuda").to(torch.int32)
    return target, tokens, u, draft, lens


def check(mm, target, tokens, u, draft=None, lens=None, **kw):
    out, accepted = mm.verify_drafts(target, tokens, u, draft_probs=draft, draft_lens=lens, **kw)
    c = [None if t is None else t.cpu() for t in (target, tokens, u, draft, lens)]
    want, count = R.verify_ref(*c)
    assert accepted.tolist() == count
    assert out.tolist() == want
    return out, accepted


CASES = [
    # requests, drafts, vocab, type, draft probabilities
    (1, 1, 1, FP32, True),
    (3, 0, 100, FP32, False),
    (5, 3, 2, FP32, True),
    (64, 3, 1000, FP32, True),
    (64, 3, 1000, FP32, False),
    (7, 5, 32000, FP32, True),
    (9, 4, 50257, BF16, True),
    (9, 4, 50257, BF16, False),
    (6, 31, 513, FP16, True),
    (300, 2, 77, FP32, True),
    (2, 2, 200000, FP32, True),
    (3, 7, 131072, FP16, True),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"b{c[0]}k{c[1]}v{c[2]}" + str(c[3])[6:])
def test_verify_matches_exact_integers(mm, case):
    reqs, k, vocab, dtype, drafts = case
    for seed in (1, 2):
        target, tokens, u, draft, lens = inputs(reqs, k, vocab, dtype, drafts, seed * 100 + vocab)
        check(mm, target, tokens, u, draft)
        check(mm, target, tokens, u, draft, lens)
    assert mm.get_device_error() == 0


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("vocab", [4097, 4098, 4099, 4100, 4101, 4102, 4103, 4104, 2047, 65535])
def test_rows_of_odd_lengths(mm, dtype, vocab):
    """Target and draft rows that begin anywhere in 16 bytes, in every distance from each other."""
    target, tokens, u, draft, lens = inputs(12, 6, vocab, dtype, True, vocab, spread=4.0)
    check(mm, target, tokens, u, draft, lens)
    check(mm, target, tokens, u, draft)


def test_edges_of_the_random_numbers(mm):
    """u = 0 takes the first token with weight, u just below 1 the last one; a draft with u q = p
    is rejected."""
    target = torch.zeros((4, 2, 9), device="cuda")
    target[:, :, 2] = 0.25
    target[:, :, 5] = 0.5
    target[:, :, 7] = 0.25
    draft = torch.zeros((4, 1, 9), device="cuda")
    draft[:, :, 5] = 1.0
    tokens = torch.full((4, 1), 5, dtype=torch.int32, device="cuda")
    below = 1.0 - 2.0 ** -24
    u = torch.tensor([[0.5, 0.0], [0.5 - 2.0 ** -25, 0.0], [0.75, below], [0.1, below]],
                     device="cuda")
    out, accepted = check(mm, target, tokens, u, draft)
    assert accepted.tolist() == [0, 1, 0, 1]
    assert out.tolist() == [[2, -1], [5, 2], [7, -1], [5, 7]]
    # numbers outside [0, 1) and NaN are clamped: the draw stays in the vocabulary
    u = torch.tensor([[2.0, 1.0], [2.0, float("nan")], [-1.0, -3.0], [float("nan"), 5.0]],
                     device="cuda")
    out, accepted = mm.verify_drafts(target, tokens, u, draft_probs=draft)
    assert accepted.tolist() == [0, 0, 1, 0]
    assert out.tolist() == [[7, -1], [2, -1], [5, 2], [7, -1]]


def test_rows_without_weight_and_odd_values(mm):
    """p = q throughout (nothing is left: drawn from p), a row of zeros, NaN and infinities."""
    target = torch.zeros((4, 2, 6), device="cuda")
    target[0, 0] = torch.tensor([0.1, 0.2, 0.3, 0.4, 0.0, 0.0])
    draft = torch.zeros((4, 1, 6), device="cuda")
    draft[0, 0] = target[0, 0] * 2
    target[2, 0] = torch.tensor([float("nan"), 0.25, -1.0, 0.0, 0.25, 0.0])
    target[3, 0] = torch.tensor([0.0, float("inf"), 0.0, 1.0, 0.0, 0.0])
    draft[1:, :, 0] = 1.0
    tokens = torch.tensor([[1], [0], [0], [0]], dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.9, 0.35], [0.5, 0.5], [0.5, 0.6], [0.5, 0.5]], device="cuda")
    out, accepted = mm.verify_drafts(target, tokens, u, draft_probs=draft)
    assert accepted.tolist() == [0, 0, 0, 0]
    assert out.tolist() == [[2, -1], [5, -1], [4, -1], [3, -1]]


def test_drafted_tokens_outside_the_vocabulary(mm):
    target, tokens, u, draft, _ = inputs(4, 3, 50, FP32, True, 7)
    tokens[0, 0], tokens[2, 1] = -1, 50
    for d in (draft, None):
        check(mm, target, tokens, u, d)
        assert mm.get_device_error() & mm.DEV_BAD_TOKEN
    # behind a shorter draft nothing is read
    lens = torch.tensor([0, 3, 1, 3], dtype=torch.int32, device="cuda")
    check(mm, target, tokens, u, draft, lens)
    assert mm.get_device_error() == 0
    # lengths are clamped to 0..drafts
    lens = torch.tensor([-4, 9, 1, 3], dtype=torch.int32, device="cuda")
    check(mm, target, tokens, u, draft, lens)


def test_strides_alignment_stream_and_graph(mm):
    """Probabilities inside wider logits-sized buffers, rows that start at any element, outputs
    inside wider ones, on another stream and from a replayed graph."""
    target, tokens, u, draft, lens = inputs(5, 3, 1001, FP32, True, 8)
    wide_t = torch.zeros((5, 4, 1007), device="cuda")
    wide_t[:, :, 3:1004] = target
    wide_d = torch.zeros((5, 3, 1004), device="cuda")
    wide_d[:, :, 1:1002] = draft
    out = torch.full((5, 6), 9, dtype=torch.int32, device="cuda")
    want = check(mm, target, tokens, u, draft, lens)
    got = check(mm, wide_t[:, :, 3:1004], tokens, u, wide_d[:, :, 1:1002], lens, out=out[:, 1:5])
    assert torch.equal(got[0], want[0]) and (out[:, 0] == 9).all() and (out[:, 5] == 9).all()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = mm.verify_drafts(target, tokens, u, draft_probs=draft, draft_lens=lens, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    graph = torch.cuda.CUDAGraph()
    out, acc = torch.empty_like(want[0]), torch.empty_like(want[1])
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            mm.verify_drafts(target, tokens, u, draft_probs=draft, draft_lens=lens, out=out,
                             accepted=acc)
        for seed in (1, 2):
            u.uniform_(generator=torch.Generator(device="cuda").manual_seed(seed))
            graph.replay()
            side.synchronize()
            w = mm.verify_drafts(target, tokens, u, draft_probs=draft, draft_lens=lens)
            side.synchronize()
            assert torch.equal(out, w[0]) and torch.equal(acc, w[1])
    torch.cuda.synchronize()


def test_tail_of_small_probabilities(mm):
    """A likely token and 100000 unlikely ones: the draws inside the tail are exact too."""
    g = torch.Generator(device="cuda").manual_seed(9)
    p = torch.rand((64, 1, 100000), generator=g, device="cuda") * 1e-8
    p[:, :, 500] = 0.999
    tokens = torch.zeros((64, 0), dtype=torch.int32, device="cuda")
    u = 0.999 + 0.001 * torch.rand((64, 1), generator=g, device="cuda")
    check(mm, p, tokens, u.clamp(max=1 - 2.0 ** -24))


def test_empty_batch(mm):
    out, acc = mm.verify_drafts(torch.zeros((0, 3, 10), device="cuda"),
                                torch.zeros((0, 2), dtype=torch.int32, device="cuda"),
                                torch.zeros((0, 3), device="cuda"))
    assert out.shape == (0, 3) and acc.shape == (0,)
