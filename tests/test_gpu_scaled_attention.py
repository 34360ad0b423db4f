"""mm3idx_paged_attention_scaled (e4m3 pages with a scale for each page and head)
against a plain form in 64 bits."""

import pytest
import torch

import pages_ref as P
import serving_ref as R
from test_gpu_attention import call, check

pytestmark = pytest.mark.gpu
BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def make_scales(s, seed, spread, power=False):
    """Scales of every page and head, about 2^(+-spread); pages that nothing uses hold NaN."""
    g = torch.Generator().manual_seed(seed)
    shape = (s["k"].shape[0], s["k"].shape[2])
    made = []
    for _ in range(2):
        x = torch.exp2(spread * (2 * torch.rand(shape, generator=g) - 1))
        x = torch.exp2(x.log2().round()) if power else x
        used = torch.zeros(shape[0], dtype=torch.bool)
        page = s["k"].shape[1]
        for i, n in enumerate(s["lens"].tolist()):
            used[s["table"][i, :R.cdiv(max(n, 0), page)].cpu().long()] = True
        x[~used] = float("nan")
        made.append(x.cuda())
    return made


CASES = [
    # lens, query_len, group, kv heads, head_dim, page, type, order, spread
    ([300, 700], 1, 8, 2, 128, 128, BF16, "nhd", 2),
    ([1], 1, 1, 1, 64, 16, BF16, "nhd", 2),
    ([0, 1, 2, 15, 16, 17, 0], 1, 4, 2, 128, 16, FP16, "nhd", 3),
    ([127, 128, 129, 0, 255, 256, 257], 1, 16, 1, 128, 64, BF16, "hnd", 1),
    ([4, 5, 130, 0, 1000], 4, 8, 2, 128, 32, BF16, "pair", 2),
    ([33, 8, 2049], 8, 8, 1, 64, 128, FP16, "pair", 2),
    ([5, 77, 640], 3, 5, 3, 128, 16, BF16, "hnd", 4),
    ([260, 90], 8, 16, 1, 128, 64, BF16, "nhd", 2),              # 128 query rows a kv head
    ([400, 90, 0], 7, 11, 2, 64, 32, FP16, "nhd", 2),
    ([20000, 17, 9000], 1, 4, 2, 128, 64, BF16, "nhd", 2),       # split over many CTAs
    ([30000], 4, 8, 1, 128, 16, FP16, "hnd", 2),
    ([1 + 37 * (i % 23) for i in range(300)], 1, 2, 2, 64, 16, BF16, "nhd", 2),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"n{len(c[0])}max{max(c[0])}q{c[1]}g{c[2]}"
                         f"h{c[3]}d{c[4]}p{c[5]}{c[7]}")
def test_scaled_attention_matches_64_bits(mm, case):
    lens, ql, group, kvh, d, page, dtype, order, spread = case
    s = R.make_attention(lens, ql=ql, group=group, kvh=kvh, d=d, page=page, dtype=dtype, kv=E4M3,
                         order=order, seed=len(lens) + max(lens))
    ks, vs = make_scales(s, 5 + max(lens), spread)
    short = any(0 < n < ql for n in lens)
    got = call(mm, s, k_scale=0.5, v_scale=1.5, k_scales=ks, v_scales=vs)
    assert mm.get_device_error() == (mm.DEV_SEQ_TOO_SHORT if short else 0)
    check(got, P.scaled_attention_ref(s, ks, vs, k_scale=0.5, v_scale=1.5))
    # strided scales, no optional outputs: the same bits
    ks2 = torch.full((ks.shape[1], 3 * ks.shape[0]), float("nan"), device="cuda")
    ks2[:, ::3] = ks.T
    out = call(mm, s, weights=False, k_scale=0.5, v_scale=1.5, k_scales=ks2[:, ::3].T,
               v_scales=vs.T.contiguous().T)[0]
    assert torch.equal(out, got[0])
    mm.get_device_error()


@pytest.mark.parametrize("dtype,d,page", [(BF16, 128, 64), (FP16, 64, 16), (BF16, 64, 128)])
def test_unit_scales(mm, dtype, d, page):
    """Scales of 1 give what no scales give, to the order of the weights' fp32 sums: with scales a
    slice of 16 tokens is summed by itself and then added, so a log-sum-exp may differ by the sums'
    rounding, which both bounds count, and an output by what that moves its own rounding."""
    s = R.make_attention([700, 0, 5000, 3], ql=2, group=4, kvh=2, d=d, page=page, dtype=dtype,
                         kv=E4M3, seed=11)
    one = torch.ones((s["k"].shape[0], 2), device="cuda")
    want = R.attention_ref(s)
    for kw in ({}, dict(k_scales=one, v_scales=one)):
        check(call(mm, s, **kw), want)
    assert mm.get_device_error() == 0


@pytest.mark.parametrize("dtype,group,d,page,ql", [(BF16, 8, 128, 64, 1), (FP16, 4, 64, 16, 2),
                                                   (BF16, 16, 128, 128, 4)])
def test_scales_that_lie_far_apart(mm, dtype, group, d, page, ql):
    """Pages' scales up to 2^60 apart, the same order for keys and values in one request and the
    opposite in another: what the pages with tiny values (or tiny scores) give must not drown."""
    lens = [3000, 2500, 40000]
    s = R.make_attention(lens, ql=ql, group=group, kvh=2, d=d, page=page, dtype=dtype, kv=E4M3,
                         seed=12)
    ks, vs = make_scales(s, 13, 30)
    # scores of the pages with large key scales stay finite: their queries are small
    s["q"] = s["q"] * 2.0 ** -10
    ks = (ks.log2() / 10).exp2()
    # in request 1 the weight lies on pages of small values: large keys there, none elsewhere
    ids = s["table"][1, :R.cdiv(lens[1], page)].long()
    vs[ids] = torch.exp2(torch.where(torch.arange(ids.numel(), device="cuda") % 2 == 0, -30.0, 30.0)
                         )[:, None]
    ks[ids] = torch.where(vs[ids] < 1, 64.0, 2.0 ** -20)
    got = call(mm, s, k_scales=ks, v_scales=vs)
    assert mm.get_device_error() == 0
    want = P.scaled_attention_ref(s, ks, vs)
    if dtype is FP16:
        # values of 2^30 leave fp16's range, whose last number is 65504: such outputs are infinite,
        # or next to its end; the others are compared
        far = want[0].abs() > 6e4
        assert far.any() and not far.all()
        assert (got[0][far].abs() > 5.9e4).all()
        assert torch.equal(got[0][far] > 0, want[0][far] > 0)
        got[0][far], want[0][far] = 0.0, 0.0
    check(got, want)


@pytest.mark.parametrize("bad", [0.0, -1.0, 1e-30, 1e30, float("inf"), float("nan")])
def test_scales_outside_their_range_are_clamped(mm, bad):
    s = R.make_attention([500, 70], group=4, kvh=2, d=128, page=16, kv=E4M3, seed=14)
    one = torch.ones((s["k"].shape[0], 2), device="cuda")
    at = int(s["table"][0, 3])
    ks, vs = one.clone(), one.clone()
    clamped = P.clamp_scale(bad)
    for x, which in ((ks, "k"), (vs, "v")):
        x[at, 1] = bad
        same = one.clone()
        same[at, 1] = float(clamped)
        a = dict(k_scales=one, v_scales=one) | {which + "_scales": x}
        b = dict(k_scales=one, v_scales=one) | {which + "_scales": same}
        for got, want in zip(call(mm, s, **a), call(mm, s, **b)):
            # (scores of 2^60 and more, rounded to 2^36, are not served: their rows may be NaN)
            assert torch.equal(P.raw(got.contiguous()), P.raw(want.contiguous()))
            assert not torch.isnan(got).any() or (which == "k" and clamped > 1)
        x[at, 1] = 1.0
    assert mm.get_device_error() == 0


def test_pages_outside_the_cache_have_no_scales(mm):
    s = R.make_attention([600, 300], ql=2, group=4, kvh=2, d=128, page=64, kv=E4M3, seed=15)
    ks, vs = make_scales(s, 16, 2)
    pool = s["k"].shape[0]
    s["table"][0, 2], s["table"][0, 5], s["table"][1, 0] = -1, pool, 2 ** 31 - 1
    got = call(mm, s, k_scales=ks, v_scales=vs)
    assert mm.get_device_error() == mm.DEV_BAD_PAGE
    check(got, P.scaled_attention_ref(s, ks, vs, drop=(-1, pool, 2 ** 31 - 1)))


def test_masked_tokens_of_scaled_pages(mm):
    """Codes behind a row's last token, NaN in their pages' scales where no row sees them."""
    s = R.make_attention([130, 257, 64], ql=4, group=4, kvh=1, d=64, page=16, kv=E4M3, seed=17)
    ks, vs = make_scales(s, 18, 2)
    base = call(mm, s, k_scales=ks, v_scales=vs)
    check(base, P.scaled_attention_ref(s, ks, vs))
    # the last token's page of request 1 is seen by its last row alone: NaN there stays there
    at = int(s["table"][1, 16])
    k = P.raw(s["k"]).clone()
    k[at] = 0x7f
    got = call(mm, {**s, "k": k.view(E4M3)}, k_scales=ks, v_scales=vs)
    assert torch.isnan(got[0][7]).all()
    keep = [r for r in range(12) if r != 7]
    for x, y in zip(got, base):
        assert torch.equal(x[keep], y[keep])
    mm.get_device_error()


def test_scaled_attention_on_streams_and_graphs(mm):
    s = R.make_attention([900, 4000, 0, 77], ql=2, group=8, kvh=2, d=128, page=32, kv=E4M3, seed=19)
    ks, vs = make_scales(s, 20, 2)
    want = call(mm, s, weights=False, k_scales=ks, v_scales=vs)[0]
    ws = mm.new_attention_workspace(16, 2, 128, 4, 2, s["max_seq_len"])
    out = torch.empty_like(s["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def run():
        return mm.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], query_len=2,
                                  max_seq_len=s["max_seq_len"], sm_scale=s["sm_scale"], k_scales=ks,
                                  v_scales=vs, out=out, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            run()
        for _ in range(3):
            out.fill_(9)
            graph.replay()
            side.synchronize()
            assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert mm.get_device_error() == 0
