"""mm3idx_paged_attention where its arithmetic or its bookkeeping meets an
edge: NaN in queries and keys of whole and split requests."""

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
