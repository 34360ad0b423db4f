"""mm3idx_append_kv against a plain form: every code, scale and untouched byte."""

import math

import pytest
import torch

import pages_ref as P
import serving_ref as R

pytestmark = pytest.mark.gpu
BF16, FP16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def make(lens, counts, *, kvh=2, d=128, page=16, dtype=BF16, kv=E4M3, order="nhd", seed=0, spare=2,
         scaled=True):
    """Inputs on the CPU: caches of random bytes, new tokens of magnitudes from 2^-12 to 2^12, old
    scales powers of two."""
    g = torch.Generator().manual_seed(seed)
    need = [R.cdiv(max(0, n), page) for n in lens]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), 2 ** 30, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    first, rows = [], 0
    for c in counts:
        first.append(rows)
        rows += c

    def tokens():
        x = torch.randn((rows, kvh, d), generator=g)
        x *= torch.exp2(24 * torch.rand((rows, kvh, 1), generator=g) - 12)
        return x.to(dtype)

    def cache():
        x = torch.randn((pool, page, kvh, d), generator=g) * 60
        x = P.to_e4m3(x.numpy()) if kv is E4M3 else x.to(kv)
        if order == "hnd":
            x = P.raw(x).transpose(1, 2).contiguous().view(kv).transpose(1, 2)
        return x

    s = dict(k=tokens(), v=tokens(), kc=cache(), vc=cache(), table=table, lens=list(lens),
             counts=list(counts), first=first, page=page, most=max(1, max(lens), max(counts)))
    s["ks"], s["vs"] = ((torch.exp2((16 * torch.rand((pool, kvh), generator=g) - 8).round())
                         for _ in range(2)) if kv is E4M3 and scaled else (None, None))
    return s


def run(mm, s, ragged=False, k_scale=1.0, v_scale=1.0, **kw):
    """The caches and scales after the call, on the CPU, and the inputs on the GPU."""
    gpu = {n: None if s[n] is None else s[n].cuda() for n in ("k", "v", "table", "ks", "vs")}
    for n in ("kc", "vc"):
        x = P.raw(s[n])
        y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
        y.copy_(x)
        gpu[n] = y.view(s[n].dtype)
    ql = max(max(s["counts"]), 1) if s["counts"] else 1
    cu = torch.tensor(s["first"] + [s["k"].shape[0]], dtype=torch.int32).cuda() if ragged else None
    args = dict(query_len=ql, max_seq_len=s["most"], k_scale=k_scale, v_scale=v_scale,
                k_scales=gpu["ks"], v_scales=gpu["vs"], cu_seqlens_q=cu, **kw)
    lens = torch.tensor(s["lens"], dtype=torch.int32).cuda()
    mm.append_kv(gpu["k"], gpu["v"], gpu["kc"], gpu["vc"], gpu["table"], lens, **args)
    return gpu, args, lens


def check(s, gpu, k_scale=1.0, v_scale=1.0):
    for new, cache, scales, scale in (("k", "kc", "ks", k_scale), ("v", "vc", "vs", v_scale)):
        want = P.raw(s[cache]).clone().view(s[cache].dtype)
        wsc = None if s[scales] is None else s[scales].clone()
        wrote = P.append_ref(s[new], want, wsc, s["table"], s["lens"], s["counts"], s["first"],
                             s["page"], s["most"], scale)
        got = gpu[cache].cpu()
        if wsc is not None:
            assert torch.equal(P.raw(gpu[scales].cpu()), P.raw(wsc))     # (NaN too)
        x, y = got.float(), want.float()
        assert torch.equal(x.isnan(), y.isnan())
        assert torch.equal(x.nan_to_num(7.0), y.nan_to_num(7.0))
        # what was not written keeps its bits
        mark = torch.zeros(got.shape[:2], dtype=torch.bool)
        for p, t in wrote:
            mark[p, t] = True
        assert torch.equal(P.raw(got)[~mark], P.raw(s[cache])[~mark])


CASES = [
    # lens, new tokens, ragged, kv heads, head_dim, page, type, cache, scaled, order
    ([300, 700, 1], [1, 1, 1], False, 2, 128, 128, BF16, E4M3, True, "nhd"),
    ([16, 17, 1, 0, 33, 2], [1] * 6, False, 3, 64, 16, FP16, E4M3, True, "hnd"),
    ([4, 5, 130, 0, 1000, 2], [4] * 6, False, 2, 128, 32, BF16, E4M3, True, "nhd"),
    ([200, 131, 128], [128] * 3, False, 1, 128, 128, FP16, E4M3, True, "hnd"),
    ([257, 300], [257] * 2, False, 4, 64, 64, BF16, E4M3, True, "nhd"),
    ([1000], [1000], False, 2, 128, 16, BF16, E4M3, True, "nhd"),
    ([129, 64, 700, 0, 5], [1, 64, 300, 0, 5], True, 2, 128, 64, BF16, E4M3, True, "hnd"),
    ([50, 60, 70], [0, 60, 7], True, 1, 64, 32, FP16, E4M3, True, "nhd"),
    ([300, 0, 33], [9] * 3, False, 2, 128, 64, BF16, BF16, False, "hnd"),
    ([77, 200], [3, 150], True, 5, 64, 16, FP16, FP16, False, "nhd"),
    ([77, 200], [70] * 2, False, 2, 128, 128, BF16, E4M3, False, "nhd"),
    ([40 + i for i in range(200)], [2] * 200, False, 2, 64, 16, BF16, E4M3, True, "nhd"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"n{len(c[0])}max{max(c[0])}new{max(c[1])}"
                         f"h{c[3]}d{c[4]}p{c[5]}{c[9]}{'s' if c[8] else ''}")
def test_append_matches_the_plain_form(mm, case):
    lens, counts, ragged, kvh, d, page, dtype, kv, scaled, order = case
    s = make(lens, counts, kvh=kvh, d=d, page=page, dtype=dtype, kv=kv, scaled=scaled, order=order,
             seed=max(lens))
    gpu, args, dl = run(mm, s, ragged)
    assert mm.get_device_error() == 0
    check(s, gpu)
    # once more: the same bits (a scale that has grown is large enough)
    before = {n: gpu[n].clone() for n in ("kc", "vc", "ks", "vs") if gpu[n] is not None}
    mm.append_kv(gpu["k"], gpu["v"], gpu["kc"], gpu["vc"], gpu["table"], dl, **args)
    for n, x in before.items():
        assert torch.equal(P.raw(gpu[n]), P.raw(x))


@pytest.mark.parametrize("kv,scaled", [(E4M3, True), (E4M3, False), (FP16, False)])
@pytest.mark.parametrize("scale", [0.5, 3.0, 0.1])
def test_append_divides_by_the_tensors_scales(mm, kv, scaled, scale):
    s = make([50, 129, 20], [20] * 3, page=32, dtype=FP16, kv=kv, scaled=scaled, seed=3)
    gpu, _, _ = run(mm, s, k_scale=scale, v_scale=1 / scale)
    import numpy as np
    check(s, gpu, np.float32(scale), np.float32(1 / scale))
    assert mm.get_device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_values_at_the_ends(mm, dtype):
    """Zeros, subnormals, the largest numbers, infinities and NaN among the new tokens; codes of NaN
    and scales at or outside the ends of their range among the old ones."""
    big, small = torch.finfo(dtype).max, 2.0 ** (-133 if dtype is BF16 else -24)
    values = [0.0, -0.0, small, big, -big, math.inf, -math.inf, math.nan, 448.0, 449.0, 2.0 ** -60]
    lens, counts = [], []
    for _ in range(40):
        lens.append(16 * 2)
        counts.append(9)
    s = make(lens, counts, kvh=2, d=64, page=16, dtype=dtype, seed=4)
    g = torch.Generator().manual_seed(5)
    for i in range(40):                        # each request its own few values, one of them rare
        pick = torch.randint(0, len(values), (3,), generator=g)
        for n in ("k", "v"):
            x = torch.tensor([values[j] for j in pick])[torch.randint(0, 3, (9, 2, 64), generator=g)]
            x[:, 1] = values[int(pick[0])]     # a head with nothing else
            s[n][9 * i:9 * i + 9] = x.to(dtype)
    for n in ("ks", "vs"):
        ends = torch.tensor([2.0 ** -60, 2.0 ** 60, 0.0, 1e-30, math.inf, math.nan, -1.0, 0.3, 1.0])
        s[n] = ends[torch.randint(0, 9, s[n].shape, generator=g)]
    for n in ("kc", "vc"):
        P.raw(s[n])[:, 3, 0, 5] = 0x7f
    gpu, _, _ = run(mm, s)
    check(s, gpu)
    assert mm.get_device_error() == 0


def test_a_scale_that_grows_step_by_step(mm):
    """One token a step, each larger than the last: the older codes follow, subnormals rounded at
    every step as documented."""
    s = make([1, 40], [1, 1], kvh=2, d=64, page=64, seed=6)
    g = torch.Generator().manual_seed(7)
    gpu = None
    for step in range(30):
        new = (torch.randn((2, 2, 64), generator=g) * 2.0 ** (0.7 * step - 8)).to(BF16)
        s["k"], s["v"], s["lens"], s["most"] = new, new.flip(0).contiguous(), [1 + step, 40 + step], 128
        if step == 0:
            s["table"] = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32)
            for n in ("kc", "vc"):
                s[n] = P.raw(s[n])[:1].expand(4, -1, -1, -1).contiguous().view(E4M3)
            for n in ("ks", "vs"):
                s[n] = s[n][:1].expand(4, -1).contiguous()
        gpu, _, _ = run(mm, s)
        check(s, gpu)
        for n in ("kc", "vc", "ks", "vs"):
            s[n] = gpu[n].cpu()
    assert mm.get_device_error() == 0


def test_bad_pages_lengths_and_offsets(mm):
    s = make([100, 50, 64, 20], [40, 10, 33, 20], page=16, seed=8)
    pool = s["kc"].shape[0]
    s["table"][0, 5], s["table"][1, 3], s["table"][2, 2] = -1, pool, 2 ** 31 - 1
    gpu, _, _ = run(mm, s, ragged=True)
    assert mm.get_device_error() == mm.DEV_BAD_PAGE
    check(s, gpu)
    # a length above the bound: positions follow the bound
    s = make([100, 64], [40, 40], page=16, seed=9)
    s["most"], s["lens"] = 96, [100, 64]
    gpu, _, _ = run(mm, s)
    assert mm.get_device_error() == mm.DEV_SEQ_TOO_LONG
    check(s, gpu)
    # offsets that decrease, or pass the rows: the requests they belong to write nothing
    s = make([64, 64, 64], [8, 8, 8], page=16, seed=10)
    gpu, args, dl = run(mm, s, ragged=True)
    for cu in ([0, 8, 4, 24], [0, 8, 16, 25], [0, 30, 16, 24], [-5, 8, 16, 24]):
        args["cu_seqlens_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        mm.append_kv(gpu["k"], gpu["v"], gpu["kc"], gpu["vc"], gpu["table"], dl, **args)
        assert mm.get_device_error() == mm.DEV_BAD_ROWS


def test_strided_inputs_and_scales(mm):
    """New tokens as parts of one projection's output, heads outside of tokens, scales by head."""
    s = make([40, 90], [30, 30], kvh=2, d=64, page=32, seed=11)
    gpu, args, dl = run(mm, s)
    rows = s["k"].shape[0]
    both = torch.full((rows, 7, 64), math.nan, dtype=BF16, device="cuda")
    both[:, 2:4], both[:, 4:6] = gpu["k"], gpu["v"]
    heads = both[:, 4:6].transpose(0, 1).contiguous().transpose(0, 1)
    fresh = {n: s[n].cuda() for n in ("kc", "vc")}
    sc = {n: s[n].T.contiguous().cuda().T for n in ("ks", "vs")}
    mm.append_kv(both[:, 2:4], heads, fresh["kc"], fresh["vc"], gpu["table"], dl,
                 **{**args, "k_scales": sc["ks"], "v_scales": sc["vs"]})
    for n in ("kc", "vc"):
        assert torch.equal(P.raw(fresh[n]), P.raw(gpu[n]))
    for n in ("ks", "vs"):
        assert torch.equal(sc[n], gpu[n])
    assert mm.get_device_error() == 0


def test_append_behind_32_bits_of_offsets(mm):
    """Pages whose bytes lie 2^31 and 2^32 and more from the cache's start."""
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB")
    page, kvh, d = 128, 1, 128
    pool = (2 ** 32 + 2 ** 31) // (page * kvh * d)
    cache = torch.zeros((pool, page, kvh, d), dtype=torch.uint8, device="cuda").view(E4M3)
    vc = torch.zeros_like(cache.view(torch.uint8)).view(E4M3)
    ks, vs = torch.ones((pool, kvh), device="cuda"), torch.ones((pool, kvh), device="cuda")
    at = [pool - 1, 2 ** 31 // (page * d), 2 ** 32 // (page * d), 0]
    table = torch.tensor(at, dtype=torch.int32, device="cuda")[:, None]
    k = torch.randn((4, kvh, d), device="cuda").to(BF16)
    lens = torch.tensor([1, 128, 5, 64], dtype=torch.int32, device="cuda")
    mm.append_kv(k, k, cache, vc, table, lens, query_len=1, max_seq_len=128, k_scales=ks, v_scales=vs)
    for i, p in enumerate(at):
        t = int(lens[i]) - 1
        got = cache[p, t].float() * ks[p, :, None]
        assert ((got - k[i].float()).abs() <= 2.0 ** -4 * k[i].float().abs() + 2.0 ** -10 * ks[p, 0]).all()
        assert torch.equal(P.raw(cache[p, t]), P.raw(vc[p, t]))
    assert int((cache.view(torch.int64) != 0).sum()) <= 4 * d // 8
    assert mm.get_device_error() == 0


def test_append_on_streams_and_graphs(mm):
    s = make([40, 90, 0, 128], [20] * 4, page=32, seed=12)
    gpu, args, dl = run(mm, s)
    want = {n: gpu[n].clone() for n in ("kc", "vc", "ks", "vs")}
    side = torch.cuda.Stream()
    fresh = {n: s[n].cuda() for n in ("kc", "vc", "ks", "vs")}
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    call = lambda: mm.append_kv(gpu["k"], gpu["v"], fresh["kc"], fresh["vc"], gpu["table"], dl,  # noqa: E731
                                **{**args, "k_scales": fresh["ks"], "v_scales": fresh["vs"]})
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            call()
        for _ in range(2):
            for n in fresh:
                P.raw(fresh[n]).copy_(P.raw(s[n]))
            graph.replay()
            side.synchronize()
            assert all(torch.equal(P.raw(fresh[n]), P.raw(want[n])) for n in fresh)
    for n in fresh:
        P.raw(fresh[n]).copy_(P.raw(s[n]))
    torch.cuda.synchronize()
    mm.append_kv(gpu["k"], gpu["v"], fresh["kc"], fresh["vc"], gpu["table"], dl, stream=side,
                 **{**args, "k_scales": fresh["ks"], "v_scales": fresh["vs"]})
    side.synchronize()
    assert all(torch.equal(P.raw(fresh[n]), P.raw(want[n])) for n in fresh)
    assert mm.get_device_error() == 0


def test_nothing_to_append(mm):
    s = make([20, 30], [5, 5], seed=13)
    gpu, args, dl = run(mm, s)
    before = P.raw(gpu["kc"]).clone()
    none = torch.empty((0, 2, 128), dtype=BF16, device="cuda")
    mm.append_kv(none, none, gpu["kc"], gpu["vc"], gpu["table"][:0], dl[:0], **{**args})
    args["cu_seqlens_q"] = torch.zeros(3, dtype=torch.int32, device="cuda")
    mm.append_kv(none, none, gpu["kc"], gpu["vc"], gpu["table"], dl, **args)
    assert torch.equal(P.raw(gpu["kc"]), before) and mm.get_device_error() == 0
