"""mm3idx_paged_attention where its arithmetic or its bookkeeping meets an
edge: NaN in queries and keys of whole and split requests, a workspace that
problems of several shapes share, scales at the ends of fp32's range,
infinite scores, an empty request of very many rows, weights over e4m3 values."""

import pytest
import torch

import serving_ref as R
from test_gpu_attention import call, check

pytestmark = pytest.mark.gpu
BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


@pytest.mark.parametrize("dtype,kv,group,kvh,d,ql", [
    (BF16, BF16, 8, 2, 128, 2), (FP16, FP16, 1, 1, 64, 1), (BF16, E4M3, 8, 2, 128, 4),
    (FP16, E4M3, 4, 1, 64, 1), (BF16, BF16, 16, 1, 64, 4)])
def test_nan_in_a_query_head(mm, dtype, kv, group, kvh, d, ql):
    """One head of one row of a short request (a CTA has it whole) and of a long one (many share
    it) is NaN: its output and log-sum-exp are NaN and so are the row's weights, in every block that
    the row sees; the rest stays what it was."""
    lens = [300, 40000, 700]
    s = R.make_attention(lens, ql=ql, group=group, kvh=kvh, d=d, page=64, dtype=dtype, kv=kv,
                         seed=70)
    base, want = call(mm, s), R.attention_ref(s)
    check(base, want)
    bad = [(0, 0), (2 * ql - 1, group * kvh - 1)]
    t = {**s, "q": s["q"].clone()}
    for row, head in bad:
        t["q"][row, head, 5] = float("nan")
    out, lse, w = call(mm, t)
    assert mm.get_device_error() == 0
    for row, head in bad:
        assert torch.isnan(out[row, head]).all() and torch.isnan(lse[row, head])
        i = row // ql
        blocks = R.cdiv(lens[i] - ql + row % ql + 1, 128)
        assert torch.isnan(w[row, :blocks]).all() and (w[row, blocks:] == 0).all()
        out[row, head], lse[row, head], w[row] = want[0][row, head], want[1][row, head], want[2][row]
    check((out, lse, w), want)
    # the third request shares no row tile with them
    for got, was in zip((out, lse, w), base):
        assert torch.equal(got[2 * ql:], was[2 * ql:])


@pytest.mark.parametrize("dtype,kv,group,kvh,d", [
    (BF16, BF16, 1, 1, 64), (FP16, FP16, 32, 1, 64), (BF16, E4M3, 4, 2, 128),
    (FP16, E4M3, 16, 1, 128)])
@pytest.mark.parametrize("nan", [slice(0, 30000), slice(30000, 60000), slice(0, 60000)])
def test_nan_in_the_keys_of_many_shares(mm, dtype, kv, group, kvh, d, nan):
    """Whole shares of a long request hold keys of NaN and the others finite ones, in either
    order: the request is NaN, its neighbours are not."""
    s = R.make_attention([60000, 900], group=group, kvh=kvh, d=d, page=128, dtype=dtype, kv=kv,
                         seed=71)
    base = call(mm, s)
    raw = torch.uint8 if kv is E4M3 else torch.int16
    value = int(torch.tensor([float("nan")]).to(kv).view(raw)[0])
    ids = s["table"][0].long()
    k = s["k"].view(raw).clone()
    seen = torch.arange(469 * 128, device="cuda").view(469, 128)
    seen = (seen >= nan.start) & (seen < nan.stop)
    k[ids] = torch.where(seen[:, :, None, None], value, k[ids])
    out, lse, w = call(mm, {**s, "k": k.view(kv)})
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and torch.isnan(w[0]).all()
    for got, was in zip((out, lse, w), base):
        assert torch.equal(got[1], was[1])
    assert mm.get_device_error() == 0


def test_one_workspace_for_models_of_different_shapes(mm):
    """Calls of different head counts, head sizes and types take turns on one workspace, called and
    as two captured graphs: what one leaves in it does not disturb the next."""
    made = [R.make_attention([200 + 7 * (i % 90) for i in range(400)], group=2, kvh=8, d=64, page=16,
                             seed=73),
            R.make_attention([300, 0, 9000, 40000], ql=8, group=8, kvh=2, d=128, page=64, seed=74),
            R.make_attention([30000] * 3, group=32, kvh=1, d=128, page=128, kv=E4M3, seed=75)]
    sizes = [mm.attention_workspace_bytes(s["q"].shape[1], s["k"].shape[2], s["q"].shape[2],
                                          s["lens"].shape[0], s["ql"], s["max_seq_len"], k == 1)
             for k, s in enumerate(made)]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    want = [call(mm, s, weights=k == 1) for k, s in enumerate(made)]

    def same(got, k):
        assert torch.equal(got[0], want[k][0]) and torch.equal(got[1], want[k][1])
        assert k != 1 or torch.equal(got[2], want[k][2])

    for k in (0, 1, 0, 2, 1, 2, 0):
        same(call(mm, made[k], weights=k == 1, workspace=ws), k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for k, s in enumerate(made):
            rows, heads = s["q"].shape[:2]
            o = [torch.empty_like(s["q"]), torch.empty((rows, heads), device="cuda"),
                 torch.empty((rows, R.cdiv(s["max_seq_len"], 128)), device="cuda")]
            graphs.append(torch.cuda.CUDAGraph())
            side.synchronize()
            with torch.cuda.graph(graphs[k], stream=side):
                mm.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"],
                                   query_len=s["ql"], max_seq_len=s["max_seq_len"],
                                   sm_scale=s["sm_scale"], out=o[0], lse=o[1],
                                   block_weights=o[2] if k == 1 else None, workspace=ws)
            outs.append(o)
        for k in (0, 1, 0, 2, 0, 1, 2, 2, 1):
            for x in outs[k]:
                x.fill_(5)
            graphs[k].replay()
            side.synchronize()
            same(outs[k], k)
    torch.cuda.synchronize()
    assert mm.get_device_error() == 0


@pytest.mark.parametrize("dtype,kv,d", [(BF16, E4M3, 128), (FP16, E4M3, 64), (BF16, BF16, 128),
                                        (FP16, FP16, 64)])
def test_scales_beyond_the_range_of_their_product(mm, dtype, kv, d):
    """Queries and scales whose product leaves fp32's range at either end while the scores are 0
    or next to it: every visible token counts alike, and no masked one does."""
    small, large = torch.finfo(dtype).tiny, torch.finfo(dtype).max
    for size, sm_scale in ((small, 2.0 ** -120), (large / 2, 2.3e38)):
        s = R.make_attention([300, 5, 1000], ql=2, group=4, kvh=2, d=d, page=64, dtype=dtype, kv=kv,
                             seed=72)
        s["q"] = (torch.sign(s["q"].float()) * size).to(dtype)
        if size == large / 2:
            s["k"] = torch.where(torch.isnan(s["k"].float()), s["k"].float(), 0.0).to(kv)
        s["sm_scale"] = sm_scale
        got, want = call(mm, s), R.attention_ref(s)
        assert torch.isfinite(want[3]).all()
        check(got, want)
    assert mm.get_device_error() == 0


def test_an_empty_request_of_very_many_rows(mm):
    """An empty slot whose rows are 2^31 pieces of 16 bytes and more: zeros throughout."""
    rows, heads, d = 2 ** 20 + 1, 128, 128
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 48 GB")
    # queries of all rows lie over each other: 8 elements from one to the next
    q = torch.zeros(8 * (rows + heads) + d, dtype=BF16, device="cuda")
    q = q.as_strided((rows, heads, d), (8, 8, 1))
    cache = torch.zeros((1, 128, 1, d), dtype=BF16, device="cuda")
    out = torch.empty((rows, heads, d), dtype=BF16, device="cuda")
    lse = torch.zeros((rows, heads), device="cuda")
    at = [0, 1, 2 ** 18, 2 ** 19 - 1, 2 ** 19, 2 ** 20 - 1, 2 ** 20]
    out[at] = 3.0
    mm.paged_attention(q, cache, cache, torch.zeros((1, 8193), dtype=torch.int32, device="cuda"),
                       torch.zeros(1, dtype=torch.int32, device="cuda"), query_len=rows,
                       max_seq_len=rows, sm_scale=1.0, out=out, lse=lse)
    assert (out[at] == 0).all() and (lse == -float("inf")).all()
    assert mm.get_device_error() == 0
    del out
    torch.cuda.empty_cache()


def test_fp16_weights_over_e4m3_values_are_pairs(mm, monkeypatch):
    """fp16 output over e4m3 values: two tokens of opposite values, so that the output is the
    difference of two weights, which a single fp16 number each would miss by up to 2^-12."""
    monkeypatch.setitem(R.WEIGHT, E4M3, 2.0 ** -22)      # the square of half a step, as over fp16
    s = R.make_attention([2] * 200, group=16, kvh=2, d=64, page=16, dtype=FP16, kv=E4M3, seed=76,
                         q_scale=0.5)
    v = torch.ones(s["v"].shape, device="cuda")
    v[:, 1] = -1.0
    s["v"] = v.to(E4M3)
    check(call(mm, s), R.attention_ref(s))


@pytest.mark.parametrize("dtype,group,d", [(BF16, 4, 128), (FP16, 8, 64)])
def test_infinite_scores(mm, dtype, group, d):
    """A score of -inf weighs nothing, whether a CTA has the request or many share it; one of +inf
    makes NaN of the rows that see it, and of no other."""
    lens = [500, 30000, 200]
    s = R.make_attention(lens, ql=2, group=group, kvh=2, d=d, page=64, dtype=dtype, seed=77)
    s["q"][:, :, 0] = 1.0
    at = [(0, 100), (1, 20000), (1, 29999), (2, 199)]        # the last tokens: the later rows' alone

    def with_key(value):
        k = s["k"].clone()
        for i, t in at:
            k[int(s["table"][i, t // 64]), t % 64, :, 0] = value
        return call(mm, {**s, "k": k})

    low = with_key(-6e4)                                     # 2^-5000 of the others and less
    for x, y in zip(with_key(-float("inf")), low):
        assert torch.equal(x, y) and not torch.isnan(x).any()
    out, lse, w = with_key(float("inf"))
    want = R.attention_ref(s)
    assert mm.get_device_error() == 0
    for r in range(6):
        seen = any(i == r // 2 and t < lens[i] - 1 + r % 2 for i, t in at)
        blocks = R.cdiv(lens[r // 2] - 1 + r % 2, 128)
        if seen:
            assert torch.isnan(out[r]).all() and torch.isnan(lse[r]).all()
            assert torch.isnan(w[r, :blocks]).all() and (w[r, blocks:] == 0).all()
        else:
            assert ((out[r].double() - want[0][r]).abs() <= want[3][r]).all()
            assert ((lse[r].double() - want[1][r]).abs() <= want[4][r]).all()
