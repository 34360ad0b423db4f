"""Eviction and the sum of weights at their edges: weights of -inf, sums next
to a rounding border, steps of selected blocks over wide tables."""

import itertools
from fractions import Fraction

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


@pytest.mark.parametrize("width", [200, 257, 1025, 4097, 8192, 8193])
@pytest.mark.parametrize("few", [1, 5, 200, 256, 257, 700])
def test_the_lowest_weights(mm, width, few):
    """Blocks of weight -inf and of the type's lowest values, and a budget that keeps some of them:
    the threshold lies in the lowest of all intervals, where forced blocks and the places behind a
    request's last block (most of them in the short requests) do not count."""
    g = torch.Generator().manual_seed(width + few)
    n = [width, width - 3, max(few + 20, width // 3), min(few + 50, width)]
    n = [min(x, width) for x in n]
    acc = torch.randn((4, width), generator=g)
    acc[1::2] = acc[1::2].abs()
    low = torch.tensor([-float("inf"), -3.4028235e38, -1.8e38])
    for i, x in enumerate(n):
        at = torch.randperm(x, generator=g)[:few]
        acc[i, at] = low[torch.randint(0, 3 if i < 2 else 1, (at.numel(),), generator=g)]
    lens = [128 * x for x in n]
    table = torch.arange(width, dtype=torch.int32).repeat(4, 1).cuda()
    for init, local, less in ((0, 1, 1), (1, 20, few // 2 + 1), (2, 3, few)):
        # the shortest request loses `less` blocks, the others more; then the longest does
        for m in (min(n), max(n)):
            budget = max(init + local, m - less)
            _, kept, out_lens = R.evict_ref(acc, lens, [], budget=budget, init=init, local=local,
                                            max_seq_len=128 * width)
            r = mm.evict_blocks(acc.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table,
                                budget=budget, init_blocks=init, local_blocks=local,
                                max_seq_len=128 * width)
            for i, stay in enumerate(kept):
                assert r.ids[i].tolist() == stay + [-1] * (budget - len(stay)), (i, budget)
                assert torch.equal(r.weights[i, :len(stay)].cpu(), acc[i, stay])
                gone = sorted(set(range(n[i])) - set(stay))
                assert r.freed[i].tolist() == gone + [-1] * (r.freed.shape[1] - len(gone))
            assert r.seq_lens.tolist() == out_lens
    assert mm.get_device_error() == 0


@pytest.mark.parametrize("sparse", [False, True])
def test_sums_next_to_a_rounding_border(mm, sparse):
    """Terms whose exact sum lies next to the middle between two fp32 numbers, in every order.  The
    second float takes up what each of the additions rounds off, at most k 2^-24 of the terms'
    magnitudes after k of them, and rounds itself by 2^-24 of that: 6 2^-48 for three terms, beside
    the half step of the one rounding at the end.  The same call gives the same."""
    terms = [[2.0 ** -24, 2.0 ** -48, 2.0 ** -48], [2.0 ** -24, -2.0 ** -48, 2.0 ** -50],
             [-2.0 ** -25, -2.0 ** -49, 2.0 ** -51], [2.0 ** -24, 2.0 ** -24, 2.0 ** -47],
             [3.0, -3.0, 2.0 ** -24], [0.1, 0.2, 0.3]]
    orders = [list(p) for t in terms for p in itertools.permutations(t)]
    w = torch.tensor(orders).T.contiguous()              # [rows, blocks]: a block an order
    n = w.shape[1]
    ids = torch.arange(n, dtype=torch.int32).repeat(3, 1).contiguous() if sparse else None
    true = [1 + sum(Fraction(float(x)) for x in col) for col in w.T]
    size = [1 + sum(abs(Fraction(float(x))) for x in col) for col in w.T]
    got = []
    for _ in range(2):
        acc = torch.ones((1, n)).cuda()
        mm.accumulate_weights(acc, w.cuda(), torch.tensor([128 * n], dtype=torch.int32).cuda(),
                              query_len=3, max_seq_len=128 * n,
                              ids=None if ids is None else ids.cuda())
        got.append(acc[0].cpu())
    assert torch.equal(*got)
    for x, t, a in zip(got[0], true, size):
        step = Fraction(float(torch.nextafter(x, torch.tensor(9.0)) - x))
        assert abs(Fraction(float(x)) - t) <= step / 2 + 6 * a / 2 ** 48


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("width", [257, 1025, 2049, 4097, 8192, 8193])
def test_selected_blocks_over_wide_tables(mm, width, in_place):
    """Steps of 4 rows x 32 ids, some given twice, some of no block, all over tables of 257 to 8193
    blocks, most of which the requests do not reach."""
    ql, topk = 4, 32
    g = torch.Generator().manual_seed(width)
    n = [width, width - 1, width // 2 + 1, 70, 1, 0]
    reqs = len(n)
    lens = torch.tensor([max(0, 128 * x - 5) for x in n], dtype=torch.int32)
    acc = torch.exp(torch.randn((reqs, width), generator=g))
    # a quarter of the ids next to the end of the table, the others anywhere, none's (-1), repeats
    ids = torch.randint(0, width, (reqs * ql, topk), generator=g, dtype=torch.int32)
    ids[:, ::4] = width - 1 - torch.randint(0, 40, (reqs * ql, topk // 4), generator=g,
                                            dtype=torch.int32)
    ids[:, 5], ids[:, 7], ids[1::ql, 9] = -1, ids[:, 6], ids[::ql, 9]
    w = 4 * torch.exp(torch.randn((reqs * ql, topk), generator=g))
    table = torch.randint(0, 10 ** 6, (reqs, width), generator=g, dtype=torch.int32)
    budget = width // 2
    new, kept, out_lens = R.evict_ref(acc, lens.tolist(), [], budget=budget, init=1, local=2,
                                      max_seq_len=128 * width, weights=w, ids=ids, ql=ql, decay=0.9)
    d = [t.cuda() for t in (acc, lens, table, w, ids)]
    kw = dict(budget=budget, init_blocks=1, local_blocks=2, max_seq_len=128 * width,
              block_weights=d[3], ids=d[4], query_len=ql, decay=0.9)
    r = mm.evict_blocks(d[0], d[1], d[2], in_place=in_place, **kw)
    for i, stay in enumerate(kept):
        m, gone = len(stay), sorted(set(range(n[i])) - set(stay))
        assert r.ids[i].tolist() == stay + [-1] * (budget - m)
        assert int(r.seq_lens[i]) == out_lens[i]
        assert torch.equal(r.weights[i, :m].cpu(), new[i][stay].float())
        assert (r.weights[i, m:] == 0).all()
        assert r.block_table[i, :budget].tolist() == table[i, stay].tolist() + [-1] * (budget - m)
        assert r.freed[i].tolist() == table[i, gone].tolist() + [-1] * (r.freed.shape[1] - len(gone))
    assert mm.get_device_error() == 0
