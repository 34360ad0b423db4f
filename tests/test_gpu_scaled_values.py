"""Attention over scaled pages where the weight lies on pages whose values are tiny
next to those of the others: what they give is the output, or half of it.  Inputs
and bounds are made so that an attention without those pages' values does not pass,
which is tested on the CPU."""

import math

import pytest
import torch

import pages_ref as P
import serving_ref as R
from test_gpu_attention import call, check

BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
V_SCALE = 2.0 ** 20


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def make(lens, dtype, group, d, page, ql, apart, bits, device):
    """Every second page has values of about 2^-20, the others of 2^(apart - 20); the scores of the
    first ones are `bits` higher in base 2, so that a page of the second kind gives 2^(apart - bits)
    of what one of the first kind gives."""
    s = R.make_attention(lens, ql=ql, group=group, kvh=2, d=d, page=page, dtype=dtype, kv=E4M3,
                         seed=31 + page, device=device)
    g = torch.Generator().manual_seed(32)
    shape = (s["k"].shape[0], 2)
    ks = torch.exp2(0.05 * torch.rand(shape, generator=g))
    vs = torch.exp2(torch.rand(shape, generator=g) - 20.0)
    small = torch.ones(shape[0], dtype=torch.bool)
    table = s["table"].cpu()
    for i, n in enumerate(lens):
        small[table[i, 1:R.cdiv(n, page):2].long()] = False
    vs = torch.where(small[:, None], vs, vs * 2.0 ** apart)
    # one dimension of the keys tells the pages apart
    k = s["k"].float().cpu()
    k[..., 0] = torch.where(small, 8.0, -8.0)[:, None, None]
    raw = P.raw(k.to(E4M3)).to(device)
    q = s["q"].clone()
    q[..., 0] = bits * math.log(2.0) / (16.0 * s["sm_scale"])
    return dict(s, k=raw.view(E4M3), q=q), ks.to(device), vs.to(device), small.to(device)


def bounded_ref(s, ks, vs, small=None):
    """(out, bound) in 64 bits; `small`: pages whose values count as 0.  As
    pages_ref.scaled_attention_ref, but for the fp16 weights' last bits: they hold p vs (the weight
    times its page's scale), of which the largest is 2^11 at least, and are off by 2^-25, so by 2^-36
    of the largest p vs that the row sees, for every token."""
    q, lens, ql = s["q"], s["lens"].tolist(), s["ql"]
    page, dev = s["k"].shape[1], q.device
    rows, qh, d = q.shape
    group = qh // 2
    out = torch.zeros((rows, qh, d), dtype=torch.float64, device=dev)
    tol = torch.zeros_like(out)
    for i, n in enumerate(lens):
        ids = s["table"][i, :R.cdiv(n, page)].long()

        def tokens(x):
            return P.raw(x)[ids].flatten(0, 1)[:n].view(x.dtype).double()

        def scales(x):
            return x[ids].double().repeat_interleave(page, 0)[:n]

        kc, vc, kss, vss = tokens(s["k"]), tokens(s["v"]), scales(ks), scales(vs)
        if small is not None:
            vc = torch.where(small[ids].repeat_interleave(page)[:n, None, None], 0.0, vc)
        for j in range(ql):
            m, r = n - ql + j + 1, i * ql + j
            for h in range(2):
                hs = slice(h * group, (h + 1) * group)
                x, kh = q[r, hs].double(), kc[:m, h] * kss[:m, h, None]
                sc = x @ kh.T * s["sm_scale"]
                off = d * 2.0 ** -23 * (x.abs() @ kh.abs().T).amax(1) * s["sm_scale"]
                off += d * 2.0 ** -24 * s["sm_scale"] * x.abs().amax(1) * kh.abs().max()
                off += 2.0 ** -22 * (sc.abs().amax(1) + 16 + 3 * vss[:m, h].log2().abs().max())
                pv = torch.softmax(sc, -1) * vss[:m, h] * V_SCALE
                out[r, hs] = pv @ vc[:m, h]
                weight = 2.0 ** -11 if q.dtype == BF16 else 2.0 ** -22
                rel = 2 * weight + 2 * off[:, None] + 2 * (64 + m / 16) * 2.0 ** -23
                tol[r, hs] = (R.HALF[q.dtype] * out[r, hs].abs() + rel * (pv @ vc[:m, h].abs())
                              + 2.0 ** -36 * m * pv.amax(1, keepdim=True) * vc[:m, h].abs().max()
                              + (2.0 ** -25 if q.dtype == FP16 else 0.0))
    return out, tol


CASES = [
    # lens, type, group, head_dim, page, query_len, apart, bits
    ([3000, 2500], BF16, 8, 128, 64, 1, 76, 100),
    ([3000, 2500], BF16, 8, 128, 64, 1, 76, 76),
    ([3000, 257], BF16, 4, 64, 16, 3, 40, 60),
    ([700, 1025], FP16, 4, 64, 16, 2, 76, 96),
    ([700, 1025], FP16, 8, 128, 128, 4, 60, 60),
    ([20000], BF16, 16, 128, 128, 4, 76, 90),            # 64 rows, split over many CTAs
    ([20000], FP16, 2, 128, 32, 1, 76, 78),
]


def ids(c):
    return f"n{max(c[0])}{'f16' if c[1] is FP16 else 'bf16'}g{c[2]}d{c[3]}p{c[4]}q{c[5]}a{c[6]}b{c[7]}"


@pytest.mark.parametrize("case", CASES, ids=ids)
def test_the_bounds_see_lost_values(case):
    s, ks, vs, small = make(*case, "cpu")
    out, tol = bounded_ref(s, ks, vs)
    lost, _ = bounded_ref(s, ks, vs, small)
    assert ((out - lost).abs() > tol).double().mean() > 0.5       # most of the outputs leave them


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=ids)
def test_values_of_small_scales_stay(mm, case):
    s, ks, vs, _ = make(*case, "cuda")
    got = call(mm, s, v_scale=V_SCALE, k_scales=ks, v_scales=vs)
    assert mm.get_device_error() == 0
    out, tol = bounded_ref(s, ks, vs)
    _, lse, mass, _, ltol = P.scaled_attention_ref(s, ks, vs, v_scale=V_SCALE)
    check(got, (out, lse, mass, tol, ltol))
