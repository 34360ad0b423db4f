"""mm3idx_accumulate_weights and mm3idx_evict_blocks against a plain form:
the sums rounded once, the kept ids, tables, freed entries and lengths exact."""

import math

import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def inputs(lens, *, ql, topk, seed, ties=False, max_seq_len=None):
    g = torch.Generator().manual_seed(seed)
    most = max_seq_len or max(max(lens), 1)
    width, reqs = R.cdiv(most, 128), len(lens)

    def mass(*shape):
        x = torch.exp(2 * torch.randn(*shape, generator=g))
        return torch.round(x).clamp(max=4) if ties else x

    acc = mass(reqs, width + 3)
    if topk:
        ids = torch.full((reqs * ql, topk), -1, dtype=torch.int32)
        for r in range(reqs * ql):
            n = R.cdiv(max(0, lens[r // ql]), 128)
            m = min(n, topk)
            if m:
                ids[r, :m] = torch.randperm(n, generator=g)[:m].sort().values.to(torch.int32)
        w = mass(reqs * ql, topk)
    else:
        ids, w = None, mass(reqs * ql, width + 1)
    tables = [torch.randint(0, 10 ** 6, (reqs, width + k), generator=g, dtype=torch.int32)
              for k in (0, 5)]
    return acc, ids, w, tables, width, most


CASES = [
    # lens, query_len, topk, budget, init, local, decay, ties
    ([1, 128, 129, 0, 5000, 4096], 1, 0, 8, 1, 2, 1.0, False),
    ([1, 128, 129, 0, 5000, 4096], 2, 4, 8, 1, 2, 0.9, False),
    ([4000, 300, 4000], 4, 16, 3, 1, 2, 1.0, False),            # only the forced blocks stay
    ([4000, 300, 4000], 1, 32, 100, 1, 2, 0.5, False),          # everything stays
    ([20000, 19999, 100, 12345], 3, 16, 40, 0, 1, 1.0, True),   # many equal weights
    ([20000, 19999, 100, 12345], 1, 0, 41, 3, 5, 0.0, True),
    ([128 * 5000, 128 * 1025 - 1, 128 * 1024], 1, 0, 1024, 4, 8, 0.99, False),
    ([128 * 9000 + 1, 77], 8, 32, 2050, 1, 2, 0.99, False),
    ([128 * 8200, 128 * 8193 - 5, 40], 2, 0, 700, 2, 3, 0.7, True),
    ([128 * 512, 128 * 513], 1, 0, 300, 1, 1, 1.0, True),
    ([128 * 512], 1, 8, 511, 1, 1, 1.0, False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"max{max(c[0])}q{c[1]}k{c[2]}b{c[3]}")
def test_evict_matches_plain_form(mm, case):
    lens, ql, topk, budget, init, local, decay, ties = case
    acc, ids, w, tables, width, most = inputs(lens, ql=ql, topk=topk, seed=sum(lens) + topk,
                                              ties=ties)
    new, kept, out_lens = R.evict_ref(acc, lens, tables, budget=budget, init=init, local=local,
                                      max_seq_len=most, weights=w, ids=ids, ql=ql, decay=decay)
    d = dict(acc=acc.cuda(), ids=None if ids is None else ids.cuda(), w=w.cuda(),
             lens=torch.tensor(lens, dtype=torch.int32).cuda(), t=[t.cuda() for t in tables])
    kw = dict(budget=budget, init_blocks=init, local_blocks=local, max_seq_len=most,
              block_weights=d["w"], ids=d["ids"], query_len=ql, decay=decay)

    # the sum alone, in place
    summed = mm.accumulate_weights(d["acc"].clone(), d["w"], d["lens"], query_len=ql,
                                   max_seq_len=most, ids=d["ids"], decay=decay).cpu()
    for i, n in enumerate(lens):
        n = R.cdiv(n, 128)
        assert torch.equal(summed[i, :n], new[i][:n].float())
        assert torch.equal(summed[i, n:], acc[i, n:])

    def expect(r, padded_to):
        for i, stay in enumerate(kept):
            n = R.cdiv(lens[i], 128)
            gone = [b for b in range(n) if b not in set(stay)]
            m = len(stay)
            assert r.ids[i].tolist() == stay + [-1] * (budget - m)
            assert int(r.seq_lens[i]) == out_lens[i]
            assert torch.equal(r.weights[i, :m].cpu(), new[i][stay].float())
            assert (r.weights[i, m:width] == 0).all()
            for table, got, freed in ((tables[0], r.block_table, r.freed),
                                      (tables[1], r.attention_block_table, r.attention_freed)):
                row = table[i].tolist()
                assert got[i, :budget].tolist() == [row[b] for b in stay] + [-1] * (budget - m)
                if padded_to:
                    assert got[i, budget:].tolist() == row[budget:]
                f = freed[i].tolist()
                assert f == [row[b] for b in gone] + [-1] * (len(f) - len(gone))

    r = mm.evict_blocks(d["acc"], d["lens"], d["t"][0], attention_block_table=d["t"][1], **kw)
    expect(r, False)
    assert torch.equal(d["acc"].cpu(), acc) and torch.equal(d["t"][0].cpu(), tables[0])
    assert d["lens"].tolist() == lens
    # into the same buffers, captured and replayed
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            mm.evict_blocks(d["acc"], d["lens"], d["t"][0], attention_block_table=d["t"][1],
                            out=r, **kw)
        for t in r:
            t.fill_(9)
        graph.replay()
        graph.replay()
    side.synchronize()
    expect(r, False)
    # in place (where the tables have the columns)
    if budget <= width:
        r = mm.evict_blocks(d["acc"], d["lens"], d["t"][0], attention_block_table=d["t"][1],
                            in_place=True, **kw)
        assert r.block_table is d["t"][0] and r.weights is d["acc"] and r.seq_lens is d["lens"]
        expect(r, True)
        assert torch.equal(d["acc"][:, width:].cpu(), acc[:, width:])
    assert mm.get_device_error() == 0


def test_without_new_weights_and_with_nan(mm):
    acc = torch.tensor([[5.0, 1.0, float("nan"), 3.0, -0.0, 0.0, float("inf"), 2.0]])
    lens = torch.tensor([8 * 128 - 3], dtype=torch.int32).cuda()
    table = torch.arange(10, 18, dtype=torch.int32)[None].cuda()
    r = mm.evict_blocks(acc.cuda(), lens, table, budget=5, init_blocks=0, local_blocks=1,
                        max_seq_len=1024)
    assert r.ids.tolist() == [[0, 2, 3, 6, 7]]
    assert r.freed.tolist() == [[11, 14, 15]]
    assert r.block_table.tolist() == [[10, 12, 13, 16, 17]]
    assert r.seq_lens.tolist() == [8 * 128 - 3 - 3 * 128]
    r = mm.evict_blocks(acc.cuda(), lens, table, budget=7, init_blocks=0, local_blocks=1,
                        max_seq_len=1024)
    assert r.ids.tolist() == [[0, 1, 2, 3, 4, 6, 7]]      # -0 and 0 are equal: the lower id stays
    assert r.attention_block_table is None


@pytest.mark.parametrize("n,budget", [(3000, 1500), (3000, 2990), (8000, 5), (1500, 700), (700, 350)])
@pytest.mark.parametrize("kind", ["equal", "two", "signs", "narrow", "steps"])
def test_thresholds_of_all_kinds(mm, n, budget, kind):
    """Weights that are all equal, of two values, of both signs, a few units apart or on a coarse
    grid: the search ends at every depth, with and without ties."""
    g = torch.Generator().manual_seed(n + budget)
    x = {"equal": torch.full((1, n), 0.37),
         "two": torch.randint(0, 2, (1, n), generator=g).float() * 3 + 1,
         "signs": torch.randn((1, n), generator=g) * 1e10 ** torch.rand((1, n), generator=g),
         "narrow": 1.0 + torch.randint(0, 900, (1, n), generator=g).float() * 2.0 ** -23,
         "steps": torch.exp2(torch.randint(-60, 60, (1, n), generator=g).float())}[kind]
    lens = [n * 128]
    new, kept, _ = R.evict_ref(x, lens, [], budget=budget, init=1, local=2, max_seq_len=n * 128)
    table = torch.arange(n, dtype=torch.int32)[None].cuda()
    r = mm.evict_blocks(x.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), table,
                        budget=budget, init_blocks=1, local_blocks=2, max_seq_len=n * 128)
    assert r.ids[0].tolist() == kept[0]
    assert torch.equal(r.weights[0, :budget].cpu(), x[0, kept[0]])


@pytest.mark.parametrize("width", [5, 33, 256, 257, 1024, 1025, 2048, 8192])
def test_thresholds_of_many_batches(mm, width):
    """24 requests of random lengths, budgets and weights: a cluster a few units wide between far
    outliers (the count goes over several levels), infinities, weights of 0 and below, ties."""
    g = torch.Generator().manual_seed(width)
    for budget in sorted({2, width // 3 + 2, width - 1}):
        lens = torch.randint(1, width * 128 + 1, (24,), generator=g)
        lens[0] = width * 128
        x = torch.rand((24, width), generator=g)
        x[::4] = 1.0 + torch.randint(0, 300, (6, width), generator=g).float() * 2.0 ** -23
        x[1::4] = torch.randint(0, 4, (6, width), generator=g).float()
        x[2::4] = torch.exp(3 * torch.randn((6, width), generator=g))
        far = torch.rand((24, width), generator=g)
        x = torch.where(far < 0.02, 1e30, torch.where(far > 0.98, -1e-30, x))
        x = torch.where((far > 0.5) & (far < 0.51), float("inf"), x)
        n = lens.tolist()
        _, kept, _ = R.evict_ref(x, n, [], budget=budget, init=1, local=1, max_seq_len=width * 128)
        table = torch.arange(width, dtype=torch.int32).repeat(24, 1).cuda()
        r = mm.evict_blocks(x.cuda(), lens.int().cuda(), table, budget=budget, init_blocks=1,
                            local_blocks=1, max_seq_len=width * 128)
        for i in range(24):
            ids = r.ids[i].tolist()
            m = len(kept[i])
            assert ids == kept[i] + [-1] * (budget - m), (budget, i)
            assert torch.equal(r.weights[i, :m].cpu(), x[i, kept[i]])
            gone = sorted(set(range((n[i] + 127) // 128)) - set(kept[i]))
            assert r.freed[i, :len(gone)].tolist() == gone


def test_ids_given_twice_and_outside(mm):
    acc = torch.ones((1, 4)).cuda()
    lens = torch.tensor([400], dtype=torch.int32).cuda()
    ids = torch.tensor([[2, 2, -1, 4, 3], [0, 2, 70000, -5, 1]], dtype=torch.int32).cuda()
    w = torch.arange(1.0, 11.0).view(2, 5).cuda()
    mm.accumulate_weights(acc, w, lens, query_len=2, max_seq_len=512, ids=ids, decay=0.5)
    assert acc.tolist() == [[6.5, 10.5, 10.5, 5.5]]
    assert mm.get_device_error() == 0
    # as many entries as there can be, all of one block but the last
    acc = torch.ones((1, 4)).cuda()
    ids = torch.full((32, 32), 1, dtype=torch.int32).cuda()
    ids[31, 31] = 3
    mm.accumulate_weights(acc, torch.full((32, 32), 2.0).cuda(), lens, query_len=32,
                          max_seq_len=512, ids=ids)
    assert acc.tolist() == [[1.0, 2047.0, 1.0, 3.0]]


def test_lengths_out_of_bounds_are_clamped(mm):
    acc = torch.arange(8.0).view(2, 4).cuda()
    lens = torch.tensor([900, -2], dtype=torch.int32).cuda()
    table = torch.arange(8, dtype=torch.int32).view(2, 4).cuda()
    r = mm.evict_blocks(acc, lens, table, budget=2, init_blocks=0, local_blocks=1,
                        max_seq_len=512)
    assert mm.get_device_error() == mm.DEV_SEQ_TOO_LONG | mm.DEV_SEQ_TOO_SHORT
    assert r.ids.tolist() == [[2, 3], [-1, -1]] and r.seq_lens.tolist() == [256, 0]
    assert r.freed.tolist() == [[0, 1], [-1, -1]]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_outputs_are_ordinary_tensors(mm, mode):
    """Parts of one allocation: contiguous, apart from each other, alive on their own, of use to
    every other operation."""
    with mode():
        acc = torch.arange(24.0).view(3, 8).cuda()
        lens = torch.tensor([1024, 300, 900], dtype=torch.int32).cuda()
        table = torch.arange(24, dtype=torch.int32).view(3, 8).cuda()
        args = dict(budget=3, init_blocks=1, local_blocks=1, max_seq_len=1024,
                    attention_block_table=table + 100)
        r = mm.evict_blocks(acc, lens, table, **args)
        want = [x.clone() for x in r]
        spans = sorted((x.data_ptr(), x.data_ptr() + x.nbytes) for x in r)
        assert all(x.is_contiguous() and x.data_ptr() % 256 == 0 for x in r)
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        ids = r.ids
        del r
        other = mm.evict_blocks(acc, lens, table, **args)
        assert torch.equal(ids, want[0]) and ids.data_ptr() != other.ids.data_ptr()
        other.weights.zero_()
        other.ids.add_(1)
        assert torch.equal(other.ids, want[0] + 1)
        assert all(torch.equal(x, y) for x, y in zip(other[3:], want[3:]))
        none = mm.evict_blocks(acc[:0], lens[:0], table[:0], budget=3, init_blocks=1,
                               local_blocks=1, max_seq_len=1024)
        assert none.ids.shape == (0, 3) and none.freed.shape == (0, 5)
