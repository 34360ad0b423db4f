"""mm3idx_append_kv: where its scales may lie, and where they may not."""

import pytest
import torch

import pages_ref as P
from test_gpu_append import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def layouts(pages, heads):
    """(keys' scales, values' scales, of all that holds them) in one allocation each."""
    def new(*shape):
        return torch.full(shape, 7.0, device="cuda")
    t = new(pages, 2, heads)
    yield t[:, 0], t[:, 1], t
    t = new(pages, heads, 2)
    yield t[..., 1], t[..., 0], t
    t = new(2, heads, pages)
    yield t[0].T, t[1].T, t
    t = new(heads, 2, pages)
    yield t[:, 0].T, t[:, 1].T, t
    t = new(pages * 3, heads * 2)
    yield t[::3, :heads], t[1::3, heads:], t
    t = new(2 * pages * heads + 8)
    yield t[:pages * heads].view(pages, heads), t[pages * heads:2 * pages * heads].view(heads, pages).T, t


@pytest.mark.parametrize("kvh", [1, 3])
@pytest.mark.parametrize("pool", [1, 9])
def test_scales_of_both_sides_in_one_allocation(mm, pool, kvh):
    lens, counts = ([13], [6]) if pool == 1 else ([40, 33, 20], [20, 1, 20])
    s = make(lens, counts, kvh=kvh, d=64, page=16, seed=20 + kvh, spare=0 if pool == 1 else 1)
    assert s["kc"].shape[0] == pool
    gpu, args, dl = run(mm, s, ragged=True)
    check(s, gpu)
    for ks, vs, whole in layouts(pool, kvh):
        ks.copy_(s["ks"])
        vs.copy_(s["vs"])
        kc, vc = (P.raw(s[n]).cuda().view(s[n].dtype) for n in ("kc", "vc"))
        before = whole.clone()
        mm.append_kv(gpu["k"], gpu["v"], kc, vc, gpu["table"], dl,
                     **{**args, "k_scales": ks, "v_scales": vs})
        assert torch.equal(ks, gpu["ks"]) and torch.equal(vs, gpu["vs"])
        assert torch.equal(P.raw(kc), P.raw(gpu["kc"])) and torch.equal(P.raw(vc), P.raw(gpu["vc"]))
        ks.copy_(s["ks"])                       # and nothing else was written
        vs.copy_(s["vs"])
        assert torch.equal(whole, before)
    assert mm.get_device_error() == 0


def test_broadcast_scales_are_refused(mm):
    s = make([40, 33], [20, 20], kvh=2, d=64, page=16, seed=22)
    gpu, args, dl = run(mm, s)
    pages = s["kc"].shape[0]
    before = {n: P.raw(gpu[n]).clone() for n in ("kc", "vc", "ks", "vs")}
    one = torch.ones((pages, 2), device="cuda")
    for ks, vs in ((torch.ones((pages, 1), device="cuda").expand(pages, 2), gpu["vs"]),
                   (gpu["ks"], torch.ones((1, 2), device="cuda").expand(pages, 2)),
                   (torch.ones((), device="cuda").expand(pages, 2), gpu["vs"]),
                   (one, one), (one, one.flatten().as_strided((pages, 2), (2, 1)))):
        with pytest.raises(mm.Mm3idxError):
            mm.append_kv(gpu["k"], gpu["v"], gpu["kc"], gpu["vc"], gpu["table"], dl,
                         **{**args, "k_scales": ks, "v_scales": vs})
    with pytest.raises(mm.Mm3idxError):
        mm.append_kv(gpu["k"], gpu["v"], gpu["kc"], gpu["kc"], gpu["table"], dl, **args)
    assert all(torch.equal(P.raw(gpu[n]), x) for n, x in before.items())
    assert mm.get_device_error() == 0


def test_attention_over_broadcast_scales(mm):
    """Attention only reads scales: one for all heads, or for all pages, is what the same numbers
    written out give."""
    import serving_ref as R
    from test_gpu_attention import call
    s = R.make_attention([300, 90], group=4, kvh=2, d=64, page=16, kv=torch.float8_e4m3fn, seed=23)
    pages = s["k"].shape[0]
    ks = torch.exp2(torch.arange(pages, device="cuda") % 5 - 2.0)[:, None].expand(pages, 2)
    vs = torch.tensor([[0.5, 2.0]], device="cuda").expand(pages, 2)
    got = call(mm, s, k_scales=ks, v_scales=vs)
    want = call(mm, s, k_scales=ks.contiguous(), v_scales=vs.contiguous())
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert mm.get_device_error() == 0
