"""A cache's pages from the first prompt to the last: allocation, prompts and
tokens appended in 8 bits, requests forked, attention with scales and block
weights, eviction, release, compaction, as a serving loop uses them together."""

import pytest
import torch

import pages_ref as P
import serving_ref as R

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
PAGE, KVH, GROUP, D = 128, 2, 4, 128


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def pages_in_use(table, lens):
    used = [0] * 1000
    for row, n in zip(table.tolist(), lens.tolist()):
        for p in row[:R.cdiv(n, PAGE)]:
            used[p] += 1
    return used


def test_a_cache_from_prompts_to_compaction(mm):
    g = torch.Generator(device="cuda").manual_seed(1)
    pool, width, slots = 64, 12, 6
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    table = torch.full((slots, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(slots, dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((pool, PAGE, KVH, D), dtype=torch.uint8, device="cuda").view(E4M3)
              for _ in range(2))
    ks, vs = (torch.zeros((pool, KVH), device="cuda") for _ in range(2))
    caches = [kc, vc, ks, vs]
    most = width * PAGE
    ws, aws = mm.new_pages_workspace(pool, slots), mm.new_attention_workspace(
        GROUP * KVH, KVH, D, slots, 1, most, block_weights=True)
    history = [[torch.zeros((0, KVH, D), device="cuda")] * 2 for _ in range(slots)]

    def new(n, size):
        x = torch.randn((n, KVH, D), generator=g, device="cuda") * size
        return x.to(BF16)

    def append(counts, size):
        """counts[i] new tokens of request i, in one ragged call."""
        for i, c in enumerate(counts):
            lens[i] += c
        ql = max(counts)
        cu = torch.tensor([sum(counts[:i]) for i in range(slots + 1)], dtype=torch.int32).cuda()
        mm.allocate_pages(refs, table, lens, query_len=ql, page_size=PAGE, workspace=ws)
        k, v = new(sum(counts), size), new(sum(counts), 1.0)
        mm.append_kv(k, v, kc, vc, table, lens, query_len=ql, max_seq_len=most, k_scales=ks,
                     v_scales=vs, cu_seqlens_q=cu)
        at = 0
        for i, c in enumerate(counts):
            history[i] = [torch.cat([h, x[at:at + c].float()]) for h, x in zip(history[i], (k, v))]
            at += c

    def check_cache():
        for i in range(slots):
            n = int(lens[i])
            ids = table[i, :R.cdiv(n, PAGE)].long()
            for c, s, h in zip((kc, vc), (ks, vs), history[i]):
                sc = s[ids].repeat_interleave(PAGE, 0)[:n, :, None]
                x = P.raw(c)[ids].flatten(0, 1)[:n].view(E4M3).float() * sc
                # half a step of e4m3: 2^-4 of the value, or of its subnormals, 2^-10 of the scale;
                # a scale that grew has rounded subnormals again, at most once a doubling: their half
                # steps add up to less than twice the last
                assert ((x - h).abs() <= 2.0 ** -4 * h.abs() + 2.0 ** -9 * sc).all(), i

    def attend():
        q = torch.randn((slots, GROUP * KVH, D), generator=g, device="cuda").to(BF16)
        w = torch.empty((slots, R.cdiv(most, 128)), device="cuda")
        out = mm.paged_attention(q, kc, vc, table, lens, query_len=1, max_seq_len=most,
                                 sm_scale=D ** -0.5, k_scales=ks, v_scales=vs, block_weights=w,
                                 workspace=aws)
        s = dict(q=q, k=kc, v=vc, table=table, lens=lens, ql=1, max_seq_len=most, sm_scale=D ** -0.5)
        ref, _, mass, tol, ltol = P.scaled_attention_ref(s, ks, vs)
        assert ((out.double() - ref).abs() <= tol).all()
        assert ((w.double() - mass).abs() <= R.weights_bound(mass, ltol)).all()
        return q, out, w

    def check_refs():
        want = pages_in_use(table, lens)[:pool]
        assert refs.tolist() == want

    # two prompts, an empty slot or two; pieces of prompts behind them
    append([300, 700, 0, 0, 0, 0], 1.0)
    append([0, 133, 0, 0, 0, 0], 2.0)
    check_cache()
    check_refs()
    attend()
    # the prompts continued by others in the free slots
    mm.fork_pages(refs, table[:2], lens[:2], torch.tensor([0, 1, 1, 0], dtype=torch.int32,
                                                          device="cuda"),
                  caches, page_size=PAGE, out=table[2:], out_lens=lens[2:], workspace=ws)
    for i, p in enumerate([0, 1, 1, 0]):
        history[2 + i] = list(history[p])
    check_cache()
    check_refs()
    for step in range(6):                      # every branch goes its own way, values growing
        append([1] * slots, 1.0 + 0.7 * step)
        attend()
    append([3, 5, 90, 1, 100, 2], 3.0)
    check_cache()
    check_refs()
    # two requests end; the lightest blocks of the others go
    q, out, w = attend()
    for i in (1, 5):
        mm.release_pages(refs, table[i:i + 1])
        table[i], lens[i], history[i] = -1, 0, [torch.zeros((0, KVH, D), device="cuda")] * 2
    check_refs()
    budget = 4
    e = mm.evict_blocks(w, lens, table, budget=budget, init_blocks=1, local_blocks=2,
                        max_seq_len=most, in_place=True)
    table[:, budget:] = -1
    mm.release_pages(refs, e.freed)
    for i in range(slots):
        keep = torch.cat([torch.arange(b * PAGE, (b + 1) * PAGE) for b in e.ids[i].tolist() if b >= 0]
                         or [torch.zeros(0, dtype=torch.int64)]).cuda()
        keep = keep[keep < history[i][0].shape[0]]
        history[i] = [h[keep] for h in history[i]]
    check_refs()
    check_cache()
    append([1, 0, 130, 1, 1, 0], 1.0)
    check_cache()
    check_refs()
    # what is left moves to the front: attention gives the same bits
    q, out, w = attend()
    c = mm.compact_pages(refs, table, caches, in_place=True, workspace=ws)
    live = int(c.live)
    assert (refs[:live] > 0).all() and (refs[live:] == 0).all()
    check_cache()
    check_refs()
    w2 = torch.empty_like(w)
    again = mm.paged_attention(q, kc, vc, table, lens, query_len=1, max_seq_len=most,
                               sm_scale=D ** -0.5, k_scales=ks, v_scales=vs, block_weights=w2,
                               workspace=aws)
    assert torch.equal(again, out) and torch.equal(w2, w)
    mm.release_pages(refs, table)
    assert refs.sum() == 0 and mm.get_device_error() == 0


def test_a_step_as_one_graph(mm):
    """Allocation, append, attention and eviction's release captured once and replayed while the
    lengths grow on the device: the same as one call after another."""
    pool, width, slots, ql = 40, 6, 3, 2
    most = width * PAGE
    g = torch.Generator(device="cuda").manual_seed(2)
    q = torch.randn((slots * ql, GROUP * KVH, D), generator=g, device="cuda").to(BF16)
    k, v = (torch.randn((slots * ql, KVH, D), generator=g, device="cuda").to(BF16) for _ in range(2))
    ws = mm.new_pages_workspace(pool)
    aws = mm.new_attention_workspace(GROUP * KVH, KVH, D, slots, ql, most)

    def state():
        return dict(refs=torch.zeros(pool, dtype=torch.int32, device="cuda"),
                    table=torch.full((slots, width), -1, dtype=torch.int32, device="cuda"),
                    lens=torch.tensor([0, 126, 400], dtype=torch.int32, device="cuda"),
                    kc=torch.zeros((pool, PAGE, KVH, D), dtype=torch.uint8, device="cuda").view(E4M3),
                    vc=torch.zeros((pool, PAGE, KVH, D), dtype=torch.uint8, device="cuda").view(E4M3),
                    ks=torch.ones((pool, KVH), device="cuda"), vs=torch.ones((pool, KVH), device="cuda"),
                    out=torch.zeros_like(q))

    def begin(s):
        mm.allocate_pages(s["refs"], s["table"], s["lens"], query_len=most, page_size=PAGE,
                          workspace=ws)

    def step(s):
        s["lens"] += ql
        mm.allocate_pages(s["refs"], s["table"], s["lens"], query_len=ql, page_size=PAGE, workspace=ws)
        mm.append_kv(k, v, s["kc"], s["vc"], s["table"], s["lens"], query_len=ql, max_seq_len=most,
                     k_scales=s["ks"], v_scales=s["vs"])
        mm.paged_attention(q, s["kc"], s["vc"], s["table"], s["lens"], query_len=ql, max_seq_len=most,
                           sm_scale=0.1, k_scales=s["ks"], v_scales=s["vs"], out=s["out"],
                           workspace=aws)

    one, two = state(), state()
    begin(one)
    begin(two)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(two)
        for _ in range(5):
            step(one)
            graph.replay()
            side.synchronize()
            for n in one:
                assert torch.equal(P.raw(one[n]), P.raw(two[n])), n
    torch.cuda.synchronize()
    assert mm.get_device_error() == 0
