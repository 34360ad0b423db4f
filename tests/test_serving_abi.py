"""Refusals of the operators that use the selection, without a GPU: the
library rejects bad arguments with the documented codes before it touches the
device, and the binding rejects bad tensors before it calls the library."""

import ctypes

import pytest
import torch

import sparse_attention_block_paged_gb300 as mm

FAKE = 0x7f0000000000


def fill(struct, vals, kw):
    vals = dict(vals, **kw)
    for k, v in vals.items():
        setattr(struct, k, v)
    return struct


def attention(**kw):
    return fill(mm.Attention(), dict(
        q=FAKE, q_token_stride=1024, q_head_stride=128, q_heads=8, kv_heads=2, head_dim=128,
        q_type=0, kv_type=0, k_cache=FAKE, k_page_stride=32768, k_token_stride=256,
        k_head_stride=128, v_cache=FAKE, v_page_stride=32768, v_token_stride=256,
        v_head_stride=128, k_scale=1.0, v_scale=1.0, num_pages=10, page_size=128, page_table=FAKE,
        table_stride=8, table_width=8, seq_lens=FAKE, num_reqs=2, query_len=1, max_seq_len=1000,
        sm_scale=0.1, out=FAKE, out_token_stride=1024, out_head_stride=128), kw)


def attend(ws=FAKE, n=1 << 40, **kw):
    return mm.lib.mm3idx_paged_attention(ctypes.byref(attention(**kw)), ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(num_reqs=-1), -1), (dict(query_len=0), -6), (dict(max_seq_len=0), -6),
    (dict(query_len=4, max_seq_len=3), -6), (dict(num_reqs=1 << 30, query_len=2), -1),
    (dict(max_seq_len=0xFFFF * 128), -5), (dict(num_reqs=1 << 27, max_seq_len=1 << 20), -1),
    (dict(sm_scale=0.0), -1), (dict(sm_scale=float("nan")), -1), (dict(k_scale=0.0), -1),
    (dict(sm_scale=1e-30, k_scale=1e-10), -1), (dict(sm_scale=1e30, k_scale=1e30), -1),
    (dict(k_scale=float("inf")), -1), (dict(v_scale=float("nan")), -1),
    (dict(q_type=2), -13), (dict(q_type=3, kv_type=3), -13), (dict(kv_type=1), -13),
    (dict(kv_type=2), -13), (dict(q_heads=7), -13), (dict(kv_heads=0), -13),
    (dict(q_heads=1), -13), (dict(head_dim=96), -13), (dict(head_dim=256), -13),
    (dict(page_size=8), -13), (dict(page_size=48), -13), (dict(page_size=256), -13),
    (dict(q=None), -1), (dict(k_cache=None), -1), (dict(v_cache=None), -1),
    (dict(page_table=None), -1), (dict(seq_lens=None), -1), (dict(out=None), -1),
    (dict(num_pages=0), -3), (dict(q=FAKE + 8), -14), (dict(k_cache=FAKE + 2), -14),
    (dict(v_cache=FAKE + 8), -14), (dict(out=FAKE + 4), -14), (dict(q_token_stride=1028), -14),
    (dict(q_head_stride=0), -14), (dict(k_page_stride=32764), -14), (dict(k_token_stride=-256), -14),
    (dict(v_head_stride=4), -14), (dict(kv_type=3, k_head_stride=136), -14),
    (dict(out_token_stride=512), -14), (dict(out_head_stride=64), -14),
    (dict(lse=FAKE, lse_token_stride=7), -14),
    (dict(block_weights=FAKE, block_weights_stride=7), -14),
    (dict(table_width=7), -4), (dict(page_size=64), -4), (dict(table_stride=6), -4),
])
def test_attention_rejects(kw, code):
    assert attend(**kw) == code
    assert mm.status_string(code) != "unknown status"


def test_attention_accepts_an_empty_batch_and_null():
    assert attend(num_reqs=0, q=None, ws=None, n=0) == 0
    assert mm.lib.mm3idx_paged_attention(None, FAKE, 1 << 30, None) == -1
    size, n = mm.lib.mm3idx_attention_workspace_bytes, ctypes.c_size_t()
    assert size(7, 2, 128, 1, 1, 100, 0, ctypes.byref(n)) == -13
    assert size(8, 2, 100, 1, 1, 100, 0, ctypes.byref(n)) == -13
    assert size(8, 2, 128, -1, 1, 100, 0, ctypes.byref(n)) == -1
    assert size(8, 2, 128, 1, 0, 100, 0, ctypes.byref(n)) == -6
    assert size(8, 2, 128, 1, 1, 0, 0, ctypes.byref(n)) == -6
    assert size(8, 2, 128, 1, 1, 100, 0, None) == -1


def weights(**kw):
    return fill(mm.Weights(), dict(acc=FAKE, acc_stride=8, block_weights=FAKE, weights_stride=8,
                                   seq_lens=FAKE, num_reqs=2, query_len=2, max_seq_len=1000,
                                   decay=1.0), kw)


IDS = dict(ids=FAKE, ids_stride=4, topk=4)


@pytest.mark.parametrize("kw,code", [
    (dict(num_reqs=-1), -1), (dict(query_len=0), -6), (dict(max_seq_len=0), -6),
    (dict(decay=-0.1), -15), (dict(decay=1.5), -15), (dict(decay=float("nan")), -15),
    (dict(acc=None), -1), (dict(seq_lens=None), -1), (dict(acc_stride=7), -8),
    (dict(weights_stride=7), -4), (dict(topk=-1), -1), (dict(IDS, block_weights=None), -1),
    (dict(IDS, topk=0), -7), (dict(IDS, ids_stride=3), -4), (dict(IDS, weights_stride=3), -4),
    (dict(ids=FAKE, ids_stride=600, topk=513, weights_stride=600), -10),
    (dict(max_seq_len=0xFFFF * 128), -5),
])
def test_accumulate_and_evict_reject_weights(kw, code):
    w = weights(**kw)
    assert mm.lib.mm3idx_accumulate_weights(ctypes.byref(w), None) == code
    assert mm.lib.mm3idx_evict_blocks(ctypes.byref(w), ctypes.byref(eviction()), None) == code


def eviction(table=None, second=None, **kw):
    e = fill(mm.EvictionArgs(), dict(budget=4, init_blocks=1, local_blocks=2, ids=FAKE,
                                     ids_stride=4, acc_out=FAKE + 4096, acc_out_stride=8,
                                     seq_lens_out=FAKE), kw)
    fill(e.tables[0], dict(in_=FAKE, in_stride=8, out=FAKE + 4096, out_stride=4, freed=FAKE,
                           freed_stride=4), table or {})
    fill(e.tables[1], {}, second or {})
    return e


@pytest.mark.parametrize("kw,code", [
    (dict(budget=2), -15), (dict(init_blocks=-1), -15), (dict(local_blocks=0), -15),
    (dict(acc_out=None), -1), (dict(seq_lens_out=None), -1), (dict(acc_out_stride=7), -8),
    (dict(acc_out=FAKE, acc_out_stride=9), -8), (dict(ids_stride=3), -8),
    (dict(table=dict(out=None)), -1), (dict(table=dict(in_stride=7)), -4),
    (dict(table=dict(out_stride=3)), -8), (dict(table=dict(out=FAKE, out_stride=9)), -8),
    (dict(table=dict(freed_stride=3)), -8), (dict(second=dict(out=FAKE)), -1),
    (dict(second=dict(in_=FAKE, in_stride=8)), -1),
])
def test_evict_rejects(kw, code):
    e = eviction(**kw)
    assert mm.lib.mm3idx_evict_blocks(ctypes.byref(weights()), ctypes.byref(e), None) == code


def test_evict_accepts_an_empty_batch_and_null():
    assert mm.lib.mm3idx_evict_blocks(ctypes.byref(weights(num_reqs=0)),
                                      ctypes.byref(eviction()), None) == 0
    assert mm.lib.mm3idx_accumulate_weights(ctypes.byref(weights(num_reqs=0)), None) == 0
    assert mm.lib.mm3idx_accumulate_weights(None, None) == -1
    assert mm.lib.mm3idx_evict_blocks(ctypes.byref(weights()), None, None) == -1


def drafts(**kw):
    return fill(mm.Drafts(), dict(
        target=FAKE, target_req_stride=400, target_row_stride=100, draft=FAKE,
        draft_req_stride=300, draft_row_stride=100, type=2, tokens=FAKE, tokens_stride=3,
        uniforms=FAKE, uniforms_stride=4, num_reqs=2, drafts=3, vocab=100, out=FAKE, out_stride=4,
        accepted=FAKE), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(num_reqs=-1), -1), (dict(vocab=0), -16), (dict(vocab=(1 << 30) + 1), -16), (dict(drafts=-1), -16), (dict(drafts=32), -16),
    (dict(type=3), -1), (dict(target=None), -1), (dict(tokens=None), -1), (dict(uniforms=None), -1),
    (dict(out=None), -1), (dict(accepted=None), -1), (dict(target=FAKE + 2), -1),
    (dict(type=0, draft=FAKE + 1), -1), (dict(target_row_stride=99), -16),
    (dict(target_req_stride=10), -16), (dict(draft_row_stride=99), -16),
    (dict(draft_req_stride=-300), -16), (dict(tokens_stride=2), -4), (dict(uniforms_stride=3), -4),
    (dict(out_stride=3), -8),
])
def test_verify_rejects(kw, code):
    assert mm.lib.mm3idx_verify_drafts(ctypes.byref(drafts(**kw)), None) == code


def test_verify_accepts_an_empty_batch_and_null():
    assert mm.lib.mm3idx_verify_drafts(ctypes.byref(drafts(num_reqs=0, target=None)), None) == 0
    assert mm.lib.mm3idx_verify_drafts(None, None) == -1


def test_constants_match_the_header():
    import test_abi
    c = test_abi.header_constants()
    assert c["MM3IDX_DEV_BAD_TOKEN"] == mm.DEV_BAD_TOKEN
    assert c["MM3IDX_MAX_DRAFTS"] == mm.MAX_DRAFTS
    assert c["MM3IDX_MAX_WEIGHT_ENTRIES"] == mm.MAX_WEIGHT_ENTRIES
    assert {torch.bfloat16: c["MM3IDX_TYPE_BF16"], torch.float16: c["MM3IDX_TYPE_FP16"],
            torch.float32: c["MM3IDX_TYPE_FP32"],
            torch.float8_e4m3fn: c["MM3IDX_TYPE_E4M3"]} == mm.TYPES


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_attention_tensors():
    kw = dict(query_len=1, max_seq_len=128, sm_scale=1.0)
    q, k, t, n = bf(2, 8, 128), bf(4, 64, 2, 128), ints(2, 2), ints(2)
    for args, what in [
            ((q.float(), k, k, t, n), "queries"), ((bf(2, 128, 8).transpose(1, 2), k, k, t, n), "queries"),
            ((q, k.half(), k.half(), t, n), "caches"), ((q, k, bf(4, 64, 1, 128), t, n), "caches"),
            ((q, bf(4, 64, 2, 64), bf(4, 64, 2, 64), t, n), "caches"),
            ((q, k, k, t.long(), n), "page table"), ((q, k, k, t, n.long()), "page table"),
            ((q, k, k, t, n), "same GPU")]:
        with pytest.raises(ValueError, match=what):
            mm.paged_attention(*args, **kw)


def test_binding_refuses_eviction_and_draft_tensors():
    acc, n, t = torch.zeros(2, 8), ints(2), ints(2, 8)
    kw = dict(budget=4, init_blocks=1, local_blocks=1, max_seq_len=1024)
    for args, what in [((acc.double(), n, t), "fp32"), ((acc[:, :7], n, t), "fp32"),
                       ((acc, n.long(), t), "lengths"), ((acc, n, t), "same GPU")]:
        with pytest.raises(ValueError, match=what):
            mm.evict_blocks(*args, **kw)
    p, tok, u = torch.zeros(2, 4, 10), ints(2, 3), torch.zeros(2, 4)
    for args, more, what in [
            ((p.double(), tok, u), {}, "target_probs"), ((p, tok.long(), u), {}, "draft_tokens"),
            ((p, tok[:, :2], u), {}, "draft_tokens"), ((p, tok, u[:, :3]), {}, "uniforms"),
            ((p, tok, u), dict(draft_probs=p), "draft_probs"),
            ((p, tok, u), dict(draft_lens=ints(3)), "draft_lens"), ((p, tok, u), {}, "same GPU")]:
        with pytest.raises(ValueError, match=what):
            mm.verify_drafts(*args, **more)
