"""Refusals of the operators that use the selection, at the ends of ranges."""

import ctypes

import pytest

import sparse_attention_block_paged_gb300 as mm
from test_serving_abi import FAKE, IDS, attend, drafts, eviction, weights


@pytest.mark.parametrize("kw", [dict(sm_scale=2.4e38), dict(sm_scale=3e38),
                                dict(sm_scale=1e30, k_scale=3e8)])
def test_scales_whose_base_2_scores_overflow(kw):
    """Scores are taken to base 2: the scale times log2(e) has to be finite too."""
    assert attend(**kw) == -1
    # (the largest one gets past this check, to the table's)
    assert attend(sm_scale=2.3e38, table_width=7) == -4


@pytest.mark.parametrize("kw,code", [
    (dict(lse=FAKE + 2, lse_token_stride=8), -14),
    (dict(block_weights=FAKE + 1, block_weights_stride=8), -14), (dict(page_table=FAKE + 2), -4),
    (dict(seq_lens=FAKE + 3), -1)])
def test_attention_rejects_misaligned_arrays(kw, code):
    assert attend(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(acc=FAKE + 2), -8), (dict(block_weights=FAKE + 1), -4), (dict(IDS, ids=FAKE + 2), -4),
    (dict(seq_lens=FAKE + 1), -1)])
def test_accumulate_and_evict_reject_misaligned_weights(kw, code):
    w = weights(**kw)
    assert mm.lib.mm3idx_accumulate_weights(ctypes.byref(w), None) == code
    assert mm.lib.mm3idx_evict_blocks(ctypes.byref(w), ctypes.byref(eviction()), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ids=FAKE + 2), -8), (dict(acc_out=FAKE + 4098), -8), (dict(seq_lens_out=FAKE + 1), -8),
    (dict(table=dict(in_=FAKE + 2)), -4), (dict(table=dict(out=FAKE + 4097)), -8),
    (dict(second=dict(in_=FAKE, in_stride=8, out=FAKE + 4096, out_stride=4, freed=FAKE + 2,
                      freed_stride=4)), -8)])
def test_evict_rejects_misaligned_arrays(kw, code):
    e = eviction(**kw)
    assert mm.lib.mm3idx_evict_blocks(ctypes.byref(weights()), ctypes.byref(e), None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=FAKE + 2), -4), (dict(draft_lens=FAKE + 1), -4), (dict(uniforms=FAKE + 2), -4),
    (dict(out=FAKE + 2), -8), (dict(accepted=FAKE + 3), -8)])
def test_verify_rejects_misaligned_arrays(kw, code):
    assert mm.lib.mm3idx_verify_drafts(ctypes.byref(drafts(**kw)), None) == code
