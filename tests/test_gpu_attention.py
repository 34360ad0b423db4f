"""mm3idx_paged_attention against a plain form in 64 bits: types, head
layouts, page sizes and cache orders, lengths from an empty slot to long
contexts, masked places that hold NaN, bad pages, streams and graphs."""

import math

import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu
BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def call(mm, s, weights=True, **kw):
    rows, heads = s["q"].shape[:2]
    lse = torch.full((rows + 1, heads), 7.0, device="cuda")
    w = torch.full((rows + 1, R.cdiv(s["max_seq_len"], 128)), 7.0, device="cuda") \
        if weights else None
    out = mm.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], query_len=s["ql"],
                             max_seq_len=s["max_seq_len"], sm_scale=s["sm_scale"], lse=lse,
                             block_weights=w, **kw)
    assert (lse[rows] == 7.0).all() and (w is None or (w[rows] == 7.0).all())
    return out, lse[:rows], None if w is None else w[:rows]


def check(got, want):
    out, lse, w = got
    ref, rlse, mass, tol, ltol = want
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((out.double() - ref).abs() / tol).nan_to_num().max()))
    assert torch.isfinite(out).all()
    empty = torch.isinf(rlse)
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    assert ((lse.double() - rlse).abs()[~empty] <= ltol[~empty]).all()
    assert (out[empty] == 0).all()
    if w is not None:
        d = (w.double() - mass).abs()
        assert (d <= R.weights_bound(mass, ltol)).all(), float(d.max())


CASES = [
    # lens, query_len, group, kv heads, head_dim, page, type, cache type, order
    ([300, 700], 1, 8, 2, 128, 128, BF16, BF16, "nhd"),
    ([1], 1, 1, 1, 64, 16, BF16, BF16, "nhd"),
    ([0, 1, 2, 15, 16, 17, 0], 1, 4, 2, 128, 16, BF16, BF16, "nhd"),
    ([127, 128, 129, 0, 255, 256, 257], 1, 16, 1, 128, 64, FP16, FP16, "hnd"),
    ([4, 5, 130, 0, 1000], 4, 8, 2, 128, 32, BF16, BF16, "pair"),
    ([33, 8, 2049], 8, 8, 1, 64, 128, FP16, FP16, "pair"),
    ([5, 77, 640], 3, 5, 3, 128, 16, BF16, BF16, "hnd"),
    ([1500, 1, 0, 333], 1, 3, 4, 64, 32, BF16, BF16, "nhd"),
    ([2000, 31, 128], 1, 8, 2, 128, 64, BF16, E4M3, "nhd"),
    ([0, 1, 16, 515], 5, 6, 2, 128, 16, FP16, E4M3, "pair"),
    ([999, 2, 64], 2, 16, 2, 64, 128, BF16, E4M3, "hnd"),
    ([700, 128, 1], 1, 64, 1, 128, 128, BF16, BF16, "nhd"),      # one kv head, 64 query heads
    ([260, 90], 8, 16, 1, 128, 64, BF16, BF16, "nhd"),           # 128 query rows a kv head
    ([400, 90, 0], 7, 11, 2, 64, 32, FP16, E4M3, "nhd"),         # 77 rows
    ([20000, 17, 9000], 1, 4, 2, 128, 64, BF16, BF16, "nhd"),    # split over many CTAs
    ([30000], 4, 8, 1, 128, 128, FP16, FP16, "nhd"),
    ([1 + 37 * (i % 23) for i in range(300)], 1, 2, 2, 64, 16, BF16, BF16, "nhd"),
]


def case_id(c):
    return f"n{len(c[0])}max{max(c[0])}q{c[1]}g{c[2]}h{c[3]}d{c[4]}p{c[5]}{c[8]}" + \
        ("e4m3" if c[7] is E4M3 else "") + ("f16" if c[6] is FP16 else "")


@pytest.mark.parametrize("case", CASES, ids=case_id)
def test_attention_matches_64_bits(mm, case):
    lens, ql, group, kvh, d, page, dtype, kv, order = case
    s = R.make_attention(lens, ql=ql, group=group, kvh=kvh, d=d, page=page, dtype=dtype, kv=kv,
                         order=order, seed=len(lens) + max(lens))
    # lengths between 0 and query_len are reported, their early rows see nothing
    short = any(0 < n < ql for n in lens)
    scales = dict(k_scale=0.5, v_scale=1.5) if kv is E4M3 else {}
    got = call(mm, s, **scales)
    assert mm.get_device_error() == (mm.DEV_SEQ_TOO_SHORT if short else 0)
    check(got, R.attention_ref(s, **scales))
    # without the optional outputs, into a strided output: the same bits
    rows, heads, _ = s["q"].shape
    wide = torch.full((rows, heads + 1, d + 8), 3.0, dtype=dtype, device="cuda")
    mm.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], query_len=ql,
                       max_seq_len=s["max_seq_len"], sm_scale=s["sm_scale"],
                       out=wide[:, :heads, :d], **scales)
    assert torch.equal(wide[:, :heads, :d], got[0])
    assert (wide[:, heads:] == 3.0).all() and (wide[:, :, d:] == 3.0).all()
    mm.get_device_error()


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_a_later_query_tokens_keys_and_values_stay_out(mm, value):
    """Keys and values of drafted tokens that only later rows see may be anything: the earlier
    rows do not change by a bit, the later ones become NaN as the formula has it."""
    s = R.make_attention([300, 1029], ql=4, group=4, kvh=2, page=64, seed=3)
    base = call(mm, s)[0]
    for i, n in enumerate([300, 1029]):
        t = n - 2                                       # seen by rows 2 and 3 of the request
        p = int(s["table"][i, t // 64])
        s["v"][p, t % 64, :, 5] = value
        s["k"][p, t % 64, :, 9] = float("nan")
    got = call(mm, s)[0]
    for i in range(2):
        assert torch.equal(got[4 * i:4 * i + 2], base[4 * i:4 * i + 2])
        assert torch.isnan(got[4 * i + 2:4 * i + 4]).any()
    assert mm.get_device_error() == 0


def test_extreme_scores(mm):
    """Scores of several hundred, both signs, rising and falling along the context."""
    s = R.make_attention([3000, 900], ql=2, group=4, kvh=1, page=16, seed=4, q_scale=60.0)
    check(call(mm, s), R.attention_ref(s))
    ramp = torch.linspace(-4, 4, s["k"].shape[0], device="cuda").to(BF16)
    order = torch.empty(s["k"].shape[0], dtype=torch.long, device="cuda").fill_(0)
    first = s["table"][0].long()
    order[first] = torch.arange(first.numel(), device="cuda")
    for sign in (1, -1):
        t = {**s, "k": (s["k"].float() * 0.05).to(BF16)}
        t["k"][..., 0] = sign * ramp[order][:, None, None]
        t["k"] = torch.where(torch.isnan(s["k"]), s["k"], t["k"])
        check(call(mm, t), R.attention_ref(t))


@pytest.mark.parametrize("kv", [BF16, FP16, E4M3])
@pytest.mark.parametrize("where", [0, 1, -1])
def test_many_small_weights_next_to_a_large_one(mm, kv, where):
    """One token takes nearly all the weight and has values of 0: what is left is the sum of 4000
    weights of 2^-22 to 2^-26 each, the large one seen first, among them or last.  304 requests of
    the same tokens, so that a warp sees many of them after the large one."""
    n, reqs = 4000, 304
    s = R.make_attention([n], group=4, kvh=1, page=64, seed=12, dtype=FP16 if kv is FP16 else BF16,
                         kv=kv)
    k, v = torch.zeros(s["k"].shape, device="cuda"), torch.ones(s["v"].shape, device="cuda")
    t = {0: 0, 1: n // 3, -1: n - 1}[where]
    at = int(s["table"][0, t // 64])
    k[at, t % 64, :, 0] = 64.0
    v[at, t % 64] = 0.0
    q = torch.zeros(s["q"].shape, device="cuda")
    q[0, :, 0] = torch.tensor([15.25, 16.0, 17.0, 18.0]) * 128 ** 0.5 / 64.0
    s = {**s, "q": q.to(s["q"].dtype), "k": k.to(kv), "v": v.to(kv)}
    ref = R.attention_ref(s)
    many = {**s, **{x: s[x].repeat(reqs, *[1] * (s[x].dim() - 1)) for x in ("q", "table", "lens")}}
    check(call(mm, many), [x.repeat(reqs, *[1] * (x.dim() - 1)) for x in ref])


@pytest.mark.parametrize("reqs,kvh", [(31, 8), (38, 4), (39, 4), (153, 1), (305, 1), (77, 4),
                                      (1000, 2)])
def test_more_requests_than_multiprocessors(mm, reqs, kvh):
    """Requests are dealt out to CTAs in turns; every count of full turns and of the rest."""
    g = torch.Generator().manual_seed(reqs)
    lens = torch.randint(0, 300, (reqs,), generator=g).tolist()
    lens[reqs // 2] = 5000
    s = R.make_attention(lens, group=2, kvh=kvh, page=16, d=64, seed=reqs)
    check(call(mm, s), R.attention_ref(s))


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_pages_outside_the_cache_hold_nothing(mm, page, bad):
    s = R.make_attention([1000, 100, 2500], ql=2, group=8, kvh=2, page=page, seed=5)
    s["table"][0, 1] = bad
    s["table"][2, 2500 // page] = bad                   # the last page
    s["table"][1, :] = bad                              # a request with no page at all
    got = call(mm, s)
    assert mm.get_device_error() == mm.DEV_BAD_PAGE
    check(got, R.attention_ref(s, drop=(bad,)))


def test_lengths_out_of_bounds_are_clamped(mm):
    s = R.make_attention([500, 300, 64], ql=2, group=4, kvh=2, page=64, seed=6)
    s["lens"] = torch.tensor([700, -3, 64], dtype=torch.int32, device="cuda")
    got = call(mm, s)
    assert mm.get_device_error() == mm.DEV_SEQ_TOO_LONG | mm.DEV_SEQ_TOO_SHORT
    check(got, R.attention_ref(s))


def test_strided_queries_and_wide_bounds(mm):
    """Queries inside a wider projection, a table wider than needed, a bound far above the
    lengths, a workspace made for a larger batch and used by a smaller one."""
    s = R.make_attention([900, 40, 0, 129], ql=1, group=4, kvh=2, page=32, seed=7)
    check_base = call(mm, s)
    wide = torch.randn((4, 24, 128), device="cuda").to(BF16)
    wide[:, 8:16] = s["q"]
    t = {**s, "q": wide[:, 8:16], "max_seq_len": 5000}
    t["table"] = torch.nn.functional.pad(s["table"], (0, 157 - s["table"].shape[1] + 3),
                                         value=2 ** 30)[:, :157 + 1]
    ws = mm.new_attention_workspace(8, 2, 128, 9, 1, 5000, block_weights=True)
    for _ in range(3):
        got = call(mm, t, workspace=ws)
        assert torch.equal(got[0], check_base[0])
        assert torch.equal(got[2][:, :8], check_base[2]) and (got[2][:, 8:] == 0).all()
    check(got, R.attention_ref(t))


def test_one_workspace_for_batches_of_many_sizes(mm):
    """Small and large batches, with and without weights, take turns on a workspace made for the
    largest: what one leaves behind does not disturb the next."""
    lens = [[9000], [700 + 13 * i for i in range(400)], [5000, 20, 0, 3000], [64] * 300, [20000, 1]]
    ws = mm.new_attention_workspace(8, 2, 128, 400, 1, 20000, block_weights=True)
    made = [R.make_attention(n, group=4, kvh=2, page=64, seed=40 + k) for k, n in enumerate(lens)]
    want = [call(mm, s, weights=k % 2 == 0) for k, s in enumerate(made)]
    for _ in range(2):
        for k, s in enumerate(made):
            got = call(mm, s, weights=k % 2 == 0, workspace=ws)
            assert torch.equal(got[0], want[k][0])
            assert k % 2 or torch.equal(got[2], want[k][2])
    check(want[4], R.attention_ref(made[4]))
    assert mm.get_device_error() == 0


def test_two_calls_at_once(mm):
    """Calls on two streams, each with its own workspace, side by side."""
    made = [R.make_attention([3000, 17, 9000], ql=2, group=8, kvh=2, page=32, seed=60),
            R.make_attention([800] * 40, group=2, kvh=2, page=16, seed=61, kv=E4M3)]
    want = [call(mm, s, weights=False)[0] for s in made]
    streams = [torch.cuda.Stream() for _ in made]
    wss = [mm.new_attention_workspace(s["q"].shape[1], 2, 128, s["lens"].shape[0], s["ql"], 9000)
           for s in made]
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for s, stream, ws in zip(made, streams, wss):
            outs.append(mm.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"],
                                           query_len=s["ql"], max_seq_len=s["max_seq_len"],
                                           sm_scale=s["sm_scale"], workspace=ws, stream=stream))
    torch.cuda.synchronize()
    for k, out in enumerate(outs):
        assert torch.equal(out, want[k % 2])


def test_many_row_tiles_and_a_bound_far_above_the_lengths(mm):
    """130 64-row tiles a kv head, and a bound of 65533 blocks: a few requests whose work list the
    32-bit form cannot hold."""
    lens = [130, 400, 0, 150]
    s = R.make_attention(lens, ql=130, group=64, kvh=1, d=64, page=128, seed=33)
    want = R.attention_ref(s)
    check(call(mm, s), want)
    most = 65533 * 128
    table = torch.nn.functional.pad(s["table"], (0, 65533 - s["table"].shape[1]), value=2 ** 30)
    check(call(mm, {**s, "table": table, "max_seq_len": most}, weights=False), want)
    assert mm.get_device_error() == 0


def test_refusals_with_real_tensors(mm):
    s = R.make_attention([300], group=4, kvh=2, page=64, seed=62)
    ws = mm.new_attention_workspace(8, 2, 128, 1, 1, 300)

    def go(**kw):
        names = ("q", "k", "v", "table", "lens")
        a = {k: kw.pop(k, s[k]) for k in names}
        return mm.paged_attention(a["q"], a["k"], a["v"], a["table"], a["lens"],
                                  **{**dict(query_len=1, max_seq_len=300, sm_scale=1.0), **kw})

    for kw, status in [(dict(workspace=ws[:ws.numel() - 256]), -9), (dict(workspace=ws[8:]), -9),
                       (dict(max_seq_len=400), -4), (dict(sm_scale=0.0), -1),
                       (dict(q=s["q"][:, :7]), -13), (dict(max_seq_len=0), -6),
                       (dict(out=torch.empty((1, 8, 132), dtype=BF16, device="cuda")[:, :, :128]),
                        -14)]:
        with pytest.raises(mm.Mm3idxError) as e:
            go(**kw)
        assert e.value.status == status
    for kw in (dict(workspace=ws.cpu()), dict(lens=s["lens"].cpu()),
               dict(out=torch.empty_like(s["q"]).half()), dict(query_len=2),
               dict(lse=torch.empty((1, 7), device="cuda")),
               dict(block_weights=torch.empty((1, 2), device="cuda"))):
        with pytest.raises(ValueError):
            go(**kw)
    assert torch.isfinite(go(workspace=ws)).all()


def test_far_pages(mm):
    """Pages that lie more than 2^32 bytes into the cache."""
    pages, page = 2 ** 18 + 5, 128
    k = torch.empty((pages, page, 1, 128), dtype=BF16, device="cuda")
    v = torch.empty((pages, page, 1, 128), dtype=BF16, device="cuda")
    s = R.make_attention([400, 1200], group=8, kvh=1, page=page, seed=8)
    far = torch.arange(pages - s["k"].shape[0], pages, device="cuda")
    k[far], v[far] = s["k"], s["v"]
    t = {**s, "k": k, "v": v,
         "table": torch.where(s["table"] < 2 ** 29, s["table"] + int(far[0]), s["table"])}
    a, b = call(mm, s), call(mm, t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    assert mm.get_device_error() == 0


def test_results_do_not_depend_on_the_run(mm):
    s = R.make_attention([50000, 3, 12000, 700], ql=2, group=4, kvh=2, page=64, seed=9)
    first = call(mm, s)
    ws = mm.new_attention_workspace(8, 2, 128, 4, 2, s["max_seq_len"], block_weights=True)
    for _ in range(5):
        again = call(mm, s, workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(first, again))


def test_other_stream_and_graph_replay(mm):
    s = R.make_attention([9000, 0, 3, 640], ql=2, group=8, kvh=2, page=128, seed=10)
    want = call(mm, s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(mm, s, stream=side)                      # its own workspace, on that stream
    side.synchronize()
    assert torch.equal(got[0], want[0])
    ws = mm.new_attention_workspace(16, 2, 128, 4, 2, s["max_seq_len"], block_weights=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call(mm, s, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        out = torch.empty_like(s["q"])
        w = torch.empty((8, 71), device="cuda")
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            mm.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], query_len=2,
                               max_seq_len=9000, sm_scale=s["sm_scale"], out=out,
                               block_weights=w, workspace=ws)
        for lens in ([9000, 0, 3, 640], [10, 4000, 2, 0]):
            # the lengths change under the graph; pages that a length newly reaches are the first's
            s["lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            s["table"].copy_(torch.where(s["table"] >= 2 ** 29, s["table"][0], s["table"]))
            out.fill_(5.0)
            for _ in range(2):
                graph.replay()
            side.synchronize()
            fresh = call(mm, s)
            assert torch.equal(out, fresh[0]) and torch.equal(w, fresh[2])
    torch.cuda.synchronize()
    assert mm.get_device_error() == 0


def test_selected_blocks(mm):
    """Attention over the sparse page table that the decode writes, K and V pages of a block next
    to each other, against the plain form over the selected tokens."""
    import workloads as W
    from helpers import to_device
    wl = W.random_case(31, num_reqs=6, query_len=3, heads=1, topk=8, init_blocks=1,
                       local_blocks=2, min_len=3, max_len=4000)
    d = to_device(wl)
    P, rows = 2, wl.rows
    width = wl.block_table.shape[1]
    attn = torch.from_numpy(W.attention_block_table(wl, 31)).cuda()
    st = torch.empty((rows, 8 * P), dtype=torch.int32, device="cuda")
    ctx = torch.empty((rows,), dtype=torch.int32, device="cuda")
    ids = mm.decode_sparse_table(
        d["q"], d["cache"], d["table"], d["lens"], query_len=3, max_seq_len=wl.max_seq_len,
        topk=8, init_blocks=1, local_blocks=2, sm_scale=wl.sm_scale, attention_block_table=attn,
        sparse_block_table_out=st, sparse_context_lens_out=ctx, block_page_stride=2 * P,
        pages_per_block=P)
    blocks = int(attn.max()) + 1
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.randn((blocks * 2 * P, 64, 2, 128), generator=g, device="cuda").to(BF16)
    k, v = pool[:-P], pool[P:]
    q = torch.randn((rows, 8, 128), generator=g, device="cuda").to(BF16)
    s = dict(q=q, k=k, v=v, table=st, lens=ctx, ql=1, max_seq_len=8 * 128, sm_scale=128 ** -0.5)
    got = call(mm, s)
    assert mm.get_device_error() == 0
    check(got, R.attention_ref(s))
    # by the definition: tokens of the selected logical blocks up to the row's position
    lens, idn = wl.seq_lens, ids[0].cpu().numpy()
    for r in range(rows):
        i, pos = r // 3, int(lens[r // 3]) - 3 + r % 3
        toks = [t for b in idn[r] if b >= 0 for t in range(128 * b, min(128 * b + 128, pos + 1))]
        page = [int(attn[i, t // 128]) * 2 * P + (t % 128) // 64 for t in toks]
        kk = pool[page, [t % 64 for t in toks]].double()
        vv = pool[[x + P for x in page], [t % 64 for t in toks]].double()
        x = q[r].double().view(2, 4, 128)
        p = torch.softmax(torch.einsum("hgd,thd->hgt", x, kk) * 128 ** -0.5, -1)
        o = torch.einsum("hgt,thd->hgd", p, vv).reshape(8, 128)
        # the output's half step and the scores' and sums' fp32 roundings, as in R.attention_ref
        tol = 2.0 ** -8 * o.abs() + 2.0 ** -8 * 2.0 ** -4 * \
            torch.einsum("hgt,thd->hgd", p, vv.abs()).reshape(8, 128)
        assert ((got[0][r].double() - o).abs() <= tol).all()


def test_empty_batch(mm):
    s = R.make_attention([], group=4, kvh=2)
    out = mm.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], query_len=1,
                             max_seq_len=128, sm_scale=1.0)
    assert out.shape == (0, 8, 128)
