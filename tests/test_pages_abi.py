"""Refusals of the operators of a cache's pages, without a GPU: the library
rejects bad arguments with the documented codes before it touches the device,
and the binding rejects bad tensors before it calls the library."""

import ctypes
import os
import re

import pytest
import torch

import sparse_attention_block_paged_gb300 as mm
from test_serving_abi import FAKE, attention, fill

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIG = 1 << 40


def scales(**kw):
    return fill(mm.KvScales(), dict(k=FAKE, k_page_stride=2, k_head_stride=1, v=FAKE,
                                    v_page_stride=2, v_head_stride=1), kw)


def attend(sc=None, **kw):
    a = attention(**{**dict(kv_type=3, k_page_stride=32768, k_token_stride=256), **kw})
    sc = scales() if sc is None else sc
    return mm.lib.mm3idx_paged_attention_scaled(ctypes.byref(a), ctypes.byref(sc), FAKE, BIG, None)


@pytest.mark.parametrize("sc,kw,code", [
    ({}, dict(kv_type=0), -13), ({}, dict(q_type=1, kv_type=1), -13), ({}, dict(head_dim=96), -13),
    (dict(k=None), {}, -1), (dict(v=None), {}, -1), (dict(k=FAKE + 2), {}, -14),
    (dict(v=FAKE + 1), {}, -14), (dict(k_page_stride=-1), {}, -14), (dict(v_head_stride=-2), {}, -14),
    ({}, dict(query_len=0), -6), ({}, dict(sm_scale=0.0), -1), ({}, dict(table_width=3), -4)])
def test_scaled_attention_rejects(sc, kw, code):
    assert attend(scales(**sc), **kw) == code
    a = attention(kv_type=3)
    assert mm.lib.mm3idx_paged_attention_scaled(ctypes.byref(a), None, FAKE, BIG, None) == -1
    assert attend(num_reqs=0) == 0


def append(**kw):
    sub = kw.pop("scales", {})
    a = fill(mm.Append(), dict(
        k=FAKE, k_token_stride=256, k_head_stride=128, v=FAKE, v_token_stride=256, v_head_stride=128,
        type=0, kv_type=3, kv_heads=2, head_dim=128, k_cache=FAKE, k_page_stride=32768,
        k_page_token_stride=256, k_page_head_stride=128, v_cache=FAKE, v_page_stride=32768,
        v_page_token_stride=256, v_page_head_stride=128, k_scale=1.0, v_scale=1.0, num_pages=10,
        page_size=128, page_table=FAKE, table_stride=8, table_width=8, seq_lens=FAKE, num_reqs=3,
        query_len=2, max_seq_len=1000, cu_seqlens_q=None, total_q=6), kw)
    a.scales = scales(**sub)
    return a


def append_rc(**kw):
    return mm.lib.mm3idx_append_kv(ctypes.byref(append(**kw)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_reqs=-1), -1), (dict(query_len=0), -6), (dict(query_len=4, max_seq_len=3), -6),
    (dict(max_seq_len=0xFFFF * 128), -5), (dict(num_reqs=1 << 30, query_len=1, total_q=1 << 30), -1),
    (dict(num_reqs=1 << 20, query_len=1, total_q=1 << 20, kv_heads=1024), -1),
    (dict(k_scale=0.0), -1), (dict(v_scale=-1.0), -1), (dict(k_scale=1e-40), -1),
    (dict(v_scale=float("inf")), -1), (dict(k_scale=float("nan")), -1), (dict(type=2), -13),
    (dict(type=3), -13), (dict(kv_type=1), -13), (dict(kv_type=0), -13), (dict(kv_heads=0), -13),
    (dict(head_dim=96), -13), (dict(page_size=8), -13), (dict(page_size=256), -13),
    (dict(total_q=5), -1), (dict(total_q=-1, cu_seqlens_q=FAKE), -1),
    (dict(total_q=7, cu_seqlens_q=FAKE), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(k_cache=None), -1), (dict(v_cache=None), -1), (dict(page_table=None), -1),
    (dict(seq_lens=None), -1), (dict(scales=dict(k=None)), -1), (dict(scales=dict(v=None)), -1),
    (dict(seq_lens=FAKE + 2), -1), (dict(cu_seqlens_q=FAKE + 1), -1), (dict(page_table=FAKE + 2), -4),
    (dict(num_pages=0), -3), (dict(k=FAKE + 8), -14), (dict(v_cache=FAKE + 4), -14),
    (dict(k_token_stride=4), -14), (dict(v_head_stride=0), -14), (dict(k_page_stride=-16), -14),
    (dict(v_page_token_stride=8), -14), (dict(k_page_head_stride=24), -14),
    (dict(scales=dict(k=FAKE + 2)), -14), (dict(scales=dict(v_page_stride=-1)), -14),
    (dict(table_width=7), -4), (dict(page_size=64), -4), (dict(table_stride=4), -4)])
def test_append_rejects(kw, code):
    assert append_rc(**kw) == code
    assert mm.status_string(code) != "unknown status"


def test_append_accepts_nothing():
    assert append_rc(num_reqs=0, total_q=0, k=None, k_cache=None, seq_lens=None) == 0
    assert append_rc(total_q=0, cu_seqlens_q=FAKE, k=None, v=None) == 0
    assert mm.lib.mm3idx_append_kv(None, None) == -1


def pool(**kw):
    return fill(mm.Pool(), dict(refs=FAKE, num_pages=100, page_size=16, page_table=FAKE,
                                table_stride=8, table_width=8, seq_lens=FAKE, num_reqs=4), kw)


def cache(**kw):
    return fill(mm.Cache(), dict(data=FAKE, page_stride=64, page_bytes=64), kw)


def allocate(ql=1, ws=FAKE, n=BIG, **kw):
    return mm.lib.mm3idx_allocate_pages(ctypes.byref(pool(**kw)), ql, ws, n, None)


def release(**kw):
    return mm.lib.mm3idx_release_pages(ctypes.byref(pool(**kw)), None)


def fork(forks=2, parents=FAKE, out=FAKE, stride=8, lens=FAKE, caches=1, c=None, ws=FAKE, n=BIG,
         **kw):
    cs = (mm.Cache * 65)(*([c or cache()] * 65))
    return mm.lib.mm3idx_fork_pages(ctypes.byref(pool(**kw)), parents, forks, out, stride, lens, cs,
                                    caches, ws, n, None)


def compact(refs_out=FAKE, out=FAKE, stride=8, live=FAKE, caches=1, c=None, ws=FAKE, n=BIG, **kw):
    cs = (mm.Cache * 65)(*([c or cache()] * 65))
    return mm.lib.mm3idx_compact_pages(ctypes.byref(pool(**kw)), refs_out, out, stride, live, cs,
                                       caches, ws, n, None)


POOL = [(dict(num_reqs=-1), -1), (dict(num_reqs=(1 << 20) + 1), -1), (dict(num_pages=0), -17),
        (dict(num_pages=(1 << 30) + 1), -17), (dict(table_width=-1), -4), (dict(table_stride=7), -4),
        (dict(page_table=FAKE + 2), -4), (dict(refs=None), -1), (dict(refs=FAKE + 1), -1),
        (dict(page_table=None), -1)]
SIZED = [(dict(page_size=0), -17), (dict(page_size=1 << 28), -17), (dict(seq_lens=FAKE + 2), -1)]


@pytest.mark.parametrize("kw,code", POOL + SIZED + [
    (dict(seq_lens=None), -1), (dict(ql=0), -6), (dict(ws=None), -9), (dict(ws=FAKE + 128), -9),
    (dict(n=100), -9), (dict(num_reqs=1 << 20, ql=1 << 20, page_size=1, table_width=4096,
                             table_stride=4096), -1)])
def test_allocate_rejects(kw, code):
    assert allocate(**kw) == code


@pytest.mark.parametrize("kw,code", POOL + SIZED)
def test_release_rejects(kw, code):
    assert release(**kw) == code


CACHES = [(dict(caches=-1), -17), (dict(caches=65), -17), (dict(c=cache(data=None)), -1),
          (dict(c=cache(page_bytes=0)), -17), (dict(c=cache(page_stride=63)), -17),
          (dict(c=cache(page_bytes=(1 << 24) + 1, page_stride=1 << 30)), -17)]


@pytest.mark.parametrize("kw,code", POOL + SIZED + CACHES + [
    (dict(seq_lens=None), -1), (dict(forks=-1), -1), (dict(forks=(1 << 20) + 1), -1),
    (dict(parents=None), -1), (dict(parents=FAKE + 2), -1), (dict(lens=None), -1), (dict(out=None), -1),
    (dict(stride=7), -8), (dict(out=FAKE + 2), -8), (dict(lens=FAKE + 1), -8), (dict(ws=None), -9),
    (dict(ws=FAKE + 4), -9), (dict(n=1000), -9)])
def test_fork_rejects(kw, code):
    assert fork(**kw) == code


@pytest.mark.parametrize("kw,code", POOL + CACHES + [
    (dict(refs_out=None), -1), (dict(live=None), -1), (dict(out=None), -1), (dict(stride=7), -8),
    (dict(refs_out=FAKE + 2), -8), (dict(live=FAKE + 1), -8), (dict(stride=9), -8),
    (dict(ws=None), -9), (dict(n=1000), -9)])
def test_compact_rejects(kw, code):
    assert compact(**kw) == code


def test_copy_rejects():
    def copy(count=3, src=FAKE, dst=FAKE, caches=1, pages=10, c=None):
        cs = (mm.Cache * 65)(*([c or cache()] * 65))
        return mm.lib.mm3idx_copy_pages(cs, caches, pages, src, dst, count, None)
    assert copy(count=-1) == -1 and copy(src=None) == -1 and copy(dst=FAKE + 2) == -1
    assert copy(pages=0) == -17 and copy(caches=65) == -17 and copy(c=cache(page_bytes=0)) == -17
    assert copy(count=0, src=None) == 0 and copy(caches=0) == 0
    assert mm.lib.mm3idx_copy_pages(None, 1, 10, FAKE, FAKE, 1, None) == -1


def test_calls_with_nothing_to_do():
    assert allocate(num_reqs=0, ws=None) == 0 and allocate(table_width=0, page_table=None, ws=None) == 0
    assert release(num_reqs=0) == 0 and fork(forks=0, ws=None) == 0
    for f in (lambda p: mm.lib.mm3idx_allocate_pages(p, 1, FAKE, BIG, None),
              lambda p: mm.lib.mm3idx_release_pages(p, None)):
        assert f(None) == -1
    size, n = mm.lib.mm3idx_pages_workspace_bytes, ctypes.c_size_t()
    assert size(100, 7, None) == -1 and size(100, -1, ctypes.byref(n)) == -1
    assert size(0, 1, ctypes.byref(n)) == -17
    assert size(100, 7, ctypes.byref(n)) == 0 and n.value == 256 + 3 * 512 == mm.pages_workspace_bytes(100, 7)
    assert mm.pages_workspace_bytes(100, 1000) == 256 + 3 * 4096


def test_constants_match_the_header():
    text = open(os.path.join(ROOT, "include", "mm3idx.h")).read()
    for name, value in (("MAX_CACHES", mm.MAX_CACHES), ("DEV_NO_PAGES", mm.DEV_NO_PAGES),
                        ("DEV_NOT_HELD", mm.DEV_NOT_HELD)):
        assert int(re.search(rf"#define MM3IDX_{name}\s+(\d+)", text).group(1)) == value


def test_binding_refuses_tensors():
    i32 = torch.int32
    k = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    c = torch.zeros((5, 16, 2, 128), dtype=torch.bfloat16)
    t, lens = torch.zeros((4, 3), dtype=i32), torch.zeros(4, dtype=i32)
    kw = dict(query_len=1, max_seq_len=48)
    ones = torch.ones((5, 2))
    for bad in (dict(k=k.float()), dict(v=k[:3]), dict(k=k[..., ::2]), dict(kc=c.half()),
                dict(kc=c[:, :, :1]), dict(t=t.long()), dict(t=t[:3]), dict(lens=lens.long()),
                dict(ks=ones), dict(ks=ones, vs=ones), dict(cu=torch.zeros(4, dtype=i32)),
                dict(cu=torch.zeros(5)), dict()):          # the last: not on a GPU
        a = dict(k=k, v=k, kc=c, vc=c, t=t, lens=lens, ks=None, vs=None, cu=None) | bad
        with pytest.raises(ValueError):
            mm.append_kv(a["k"], a["v"], a["kc"], a["vc"], a["t"], a["lens"], k_scales=a["ks"],
                         v_scales=a["vs"], cu_seqlens_q=a["cu"], **kw)
    with pytest.raises(TypeError):
        mm.append_kv(k, k, c, c, t, None, **kw)
    refs = torch.zeros(5, dtype=i32)
    for f in (lambda **a: mm.allocate_pages(a["r"], a["t"], a["lens"], query_len=1, page_size=16),
              lambda **a: mm.release_pages(a["r"], a["t"], seq_lens=a["lens"], page_size=16),
              lambda **a: mm.fork_pages(a["r"], a["t"], a["lens"], a["p"], a["c"], page_size=16),
              lambda **a: mm.compact_pages(a["r"], a["t"], a["c"])):
        for bad in (dict(r=refs.long()), dict(r=refs[::2]), dict(t=t.float()), dict(t=t[0]),
                    dict(t=t.T), {}):
            with pytest.raises(ValueError):
                f(**(dict(r=refs, t=t, lens=lens, p=lens, c=[c]) | bad))
    with pytest.raises(ValueError, match="go together"):
        mm.release_pages(refs, t, seq_lens=lens)
    with pytest.raises(ValueError):
        mm.fork_pages(refs, t, lens, lens.long(), [c], page_size=16)
    with pytest.raises(ValueError):
        mm.copy_pages([c], lens.long(), lens)
