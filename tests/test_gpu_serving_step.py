"""The operators together, as a decode loop uses them: the indexer selects
blocks, attention reads them and reports their weights, the weights add up,
the lightest blocks leave both caches' tables, the indexer and the attention
go on over what is left, and drafted tokens are verified."""

import numpy as np
import pytest
import torch

import serving_ref as R
import workloads as W
from helpers import to_device

pytestmark = pytest.mark.gpu
BLOCK, TOPK, INIT, LOCAL, QL, P = 128, 8, 1, 2, 4, 2


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def test_decode_loop_with_eviction(mm):
    reqs, heads, kvh, budget = 5, 8, 2, 14
    wl = W.random_case(71, num_reqs=reqs, query_len=QL, heads=1, topk=TOPK, init_blocks=INIT,
                       local_blocks=LOCAL, min_len=900, max_len=4000)
    d = to_device(wl)
    most = wl.max_seq_len
    width = R.cdiv(most, BLOCK)
    attn = torch.from_numpy(W.attention_block_table(wl, 71)).cuda()
    g = torch.Generator(device="cuda").manual_seed(7)
    pool = torch.randn((int(attn.max() + 1) * 2 * P, BLOCK // P, kvh, 128), generator=g,
                       device="cuda").to(torch.bfloat16)
    k, v = pool[:-P], pool[P:]
    rows = reqs * QL
    st = torch.empty((rows, TOPK * P), dtype=torch.int32, device="cuda")
    ctx = torch.empty((rows,), dtype=torch.int32, device="cuda")
    acc = torch.zeros((reqs, width), device="cuda")
    step_w = torch.empty((rows, TOPK), device="cuda")
    ws = mm.new_workspace(mm.OP_DECODE, 1, reqs, QL, most, TOPK)
    aws = mm.new_attention_workspace(heads, kvh, 128, rows, 1, TOPK * BLOCK, block_weights=True)
    index_table, lens = d["table"].clone(), d["lens"].clone()
    # what the tables hold, by hand: the original block of every column
    origin = [list(range(R.cdiv(int(n), BLOCK))) for n in wl.seq_lens]
    total = [dict.fromkeys(o, 0.0) for o in origin]

    for step in range(3):
        ids = mm.decode_sparse_table(
            d["q"], d["cache"], index_table, lens, query_len=QL, max_seq_len=most, topk=TOPK,
            init_blocks=INIT, local_blocks=LOCAL, sm_scale=wl.sm_scale,
            attention_block_table=attn, sparse_block_table_out=st, sparse_context_lens_out=ctx,
            block_page_stride=2 * P, pages_per_block=P, workspace=ws)
        q = torch.randn((rows, heads, 128), generator=g, device="cuda").to(torch.bfloat16)
        out = mm.paged_attention(q, k, v, st, ctx, query_len=1, max_seq_len=TOPK * BLOCK,
                                 sm_scale=128 ** -0.5, block_weights=step_w, workspace=aws)
        s = dict(q=q, k=k, v=v, table=st, lens=ctx, ql=1, max_seq_len=TOPK * BLOCK,
                 sm_scale=128 ** -0.5)
        ref, _, mass, tol, ltol = R.attention_ref(s)
        assert ((out.double() - ref).abs() <= tol).all()
        assert ((step_w.double() - mass).abs() <= R.weights_bound(mass, ltol)).all()
        # each row's weights add up to its number of heads
        assert ((step_w.double().sum(1) - heads).abs() <= heads * 2.0 ** -16).all()
        idn, wn = ids[0].cpu().numpy(), step_w.cpu().numpy()
        now = lens.cpu().numpy()
        for r in range(rows):
            for c, b in enumerate(idn[r]):
                if b >= 0:
                    total[r // QL][origin[r // QL][b]] += float(wn[r, c])
        if step < 1:
            mm.accumulate_weights(acc, step_w, lens, query_len=QL, max_seq_len=most, ids=ids)
            continue
        e = mm.evict_blocks(acc, lens, index_table, attention_block_table=attn, budget=budget,
                            init_blocks=INIT, local_blocks=LOCAL, max_seq_len=most,
                            block_weights=step_w, ids=ids, query_len=QL, in_place=True)
        assert e.seq_lens is lens and e.weights is acc and e.block_table is index_table
        kept = e.ids.cpu().numpy()
        for i in range(reqs):
            n = len(origin[i])
            stay = [b for b in kept[i] if b >= 0]
            assert len(stay) == min(n, budget) and stay == sorted(set(stay))
            assert set(range(min(INIT, n))) | set(range(max(0, n - LOCAL), n)) <= set(stay)
            left = [total[i][origin[i][b]] for b in range(n) if b not in stay]
            free = [total[i][origin[i][b]] for b in stay if INIT <= b < n - LOCAL]
            # (sums of a few fp32 weights, added in another order here)
            if left and free:
                assert max(left) <= min(free) * (1 + 2.0 ** -20) + 1e-12
            assert int(lens[i]) == now[i] - BLOCK * (n - len(stay))
            origin[i] = [origin[i][b] for b in stay]
            got = acc[i, :len(stay)].cpu().numpy()
            np.testing.assert_allclose(got, [total[i][o] for o in origin[i]], rtol=2.0 ** -20,
                                       atol=1e-12)
            assert index_table[i, :len(stay)].tolist() == [int(wl.block_table[i, o])
                                                           for o in origin[i]]
    assert mm.get_device_error() == 0
    # the freed and the kept entries are the old table's
    assert all(len(o) <= budget for o in origin)


def test_step_as_one_graph(mm):
    """Selection, attention, accumulation, eviction (a copy) and verification captured once and
    replayed: the same as one call after another."""
    reqs, heads, kvh, budget, vocab = 6, 16, 1, 10, 3000
    wl = W.random_case(72, num_reqs=reqs, query_len=QL, heads=1, topk=TOPK, init_blocks=INIT,
                       local_blocks=LOCAL, min_len=500, max_len=6000)
    d = to_device(wl)
    most, rows = wl.max_seq_len, reqs * QL
    attn = torch.from_numpy(W.attention_block_table(wl, 72)).cuda()
    g = torch.Generator(device="cuda").manual_seed(8)
    pool = torch.randn((int(attn.max() + 1) * 2 * P, BLOCK // P, kvh, 64), generator=g,
                       device="cuda").to(torch.float16)
    k, v = pool[:-P], pool[P:]
    q = torch.randn((rows, heads, 64), generator=g, device="cuda").to(torch.float16)
    st = torch.empty((rows, TOPK * P), dtype=torch.int32, device="cuda")
    ctx = torch.empty((rows,), dtype=torch.int32, device="cuda")
    acc0 = torch.rand((reqs, R.cdiv(most, BLOCK)), generator=g, device="cuda")
    step_w = torch.empty((rows, TOPK), device="cuda")
    ws = mm.new_workspace(mm.OP_DECODE, 1, reqs, QL, most, TOPK)
    aws = mm.new_attention_workspace(heads, kvh, 64, rows, 1, TOPK * BLOCK, block_weights=True)
    target = torch.softmax(2 * torch.randn((reqs, QL, vocab), generator=g, device="cuda"), -1)
    draft = torch.softmax(2 * torch.randn((reqs, QL - 1, vocab), generator=g, device="cuda"), -1)
    tokens = torch.randint(0, vocab, (reqs, QL - 1), generator=g, device="cuda").to(torch.int32)
    u = torch.rand((reqs, QL), generator=g, device="cuda")

    def step():
        ids = mm.decode_sparse_table(
            d["q"], d["cache"], d["table"], d["lens"], query_len=QL, max_seq_len=most, topk=TOPK,
            init_blocks=INIT, local_blocks=LOCAL, sm_scale=wl.sm_scale,
            attention_block_table=attn, sparse_block_table_out=st, sparse_context_lens_out=ctx,
            block_page_stride=2 * P, pages_per_block=P, workspace=ws)
        out = mm.paged_attention(q, k, v, st, ctx, query_len=1, max_seq_len=TOPK * BLOCK,
                                 sm_scale=0.125, block_weights=step_w, workspace=aws)
        e = mm.evict_blocks(acc0, d["lens"], d["table"], attention_block_table=attn,
                            budget=budget, init_blocks=INIT, local_blocks=LOCAL, max_seq_len=most,
                            block_weights=step_w, ids=ids, query_len=QL, decay=0.5)
        t, n = mm.verify_drafts(target, tokens, u, draft_probs=draft)
        return [ids, out, *e, t, n]

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = step()
        for _ in range(3):
            for x in got:
                x.fill_(3)
            graph.replay()
            side.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, want))
    torch.cuda.synchronize()
    assert mm.get_device_error() == 0
    w, count = R.verify_ref(target.cpu(), tokens.cpu(), u.cpu(), draft.cpu())
    assert want[-2].tolist() == w and want[-1].tolist() == count
