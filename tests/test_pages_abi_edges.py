"""Scales that mm3idx_append_kv may not write: floats that several pages, heads or
sides have in common.  Refused before the device is touched, so no GPU is needed."""

import random

import pytest

from test_pages_abi import FAKE, append_rc, attend, scales

# of 10 pages and 2 heads, values right behind the keys
APART = dict(k_page_stride=2, k_head_stride=1, v_page_stride=2, v_head_stride=1, v=FAKE + 80)


def floats(at, ps, hs, pages, heads):
    return [at + 4 * (p * ps + h * hs) for p in range(pages) for h in range(heads)]


@pytest.mark.parametrize("sc", [
    dict(k_head_stride=0), dict(v_head_stride=0),              # one scale a page for all heads
    dict(k_page_stride=0), dict(v_page_stride=0),              # one a head for all pages
    dict(k_page_stride=0, k_head_stride=0),
    dict(k_page_stride=1), dict(v_page_stride=3, v_head_stride=3),
    dict(k_page_stride=3, k_head_stride=6), dict(k_page_stride=2, k_head_stride=18)])
def test_scales_that_pages_or_heads_share(sc):
    assert append_rc(scales={**APART, **sc}) == -14
    # attention only reads them (it goes on to its next check)
    assert attend(scales(**sc), table_width=3) == -4


def test_one_page_and_one_head():
    assert append_rc(scales={**APART, "k_head_stride": 0}, num_pages=1) == -14
    assert append_rc(scales={**APART, "v_page_stride": 0}, kv_heads=1) == -14
    # the stride that is not used may be 0 (they go on to the next check)
    assert append_rc(scales={**APART, "k_page_stride": 0}, num_pages=1, table_width=7) == -4
    assert append_rc(scales={**APART, "v_head_stride": 0}, kv_heads=1, table_width=7) == -4


@pytest.mark.parametrize("sc,kw", [
    (dict(v=FAKE), {}),                                                       # one tensor
    (dict(v=FAKE + 4), {}), (dict(v=FAKE - 8), {}), (dict(v=FAKE + 76), {}),  # parts of one
    (dict(k_page_stride=7, v_page_stride=7, v=FAKE + 29 * 4), {}),
    (dict(k_page_stride=1, v_page_stride=1, k_head_stride=10, v_head_stride=10, v=FAKE + 40), {}),
    (dict(k_page_stride=1, v_page_stride=1, k_head_stride=0, v_head_stride=5, v=FAKE + 36),
     dict(kv_heads=1)),
    (dict(k_page_stride=4, v_page_stride=9, v=FAKE + 36), {}),                # in turns, unlike
    (dict(v=FAKE), dict(num_pages=1, kv_heads=1))])
def test_scales_that_both_sides_share(sc, kw):
    assert append_rc(scales={**APART, **sc}, v_cache=FAKE + (1 << 20), **kw) == -14


def test_one_cache_for_both_sides():
    assert append_rc(scales=APART) == -14
    assert append_rc(scales=APART, num_reqs=0, total_q=0) == 0
    assert append_rc(scales=APART, total_q=0, cu_seqlens_q=FAKE) == 0


def test_strides_by_counting():
    """Every side whose pages and heads share a float is refused, and no other (those go on to the
    next check, of the table)."""
    rng = random.Random(1)
    met = set()
    for _ in range(3000):
        pages, heads = rng.randint(1, 9), rng.randint(1, 6)
        ps, hs = rng.randint(0, 12), rng.randint(0, 12)
        own = len(set(floats(0, ps, hs, pages, heads))) == pages * heads
        met.add(own)
        rc = append_rc(scales={**APART, "k_page_stride": ps, "k_head_stride": hs, "v_page_stride": 64,
                               "v_head_stride": 1}, num_pages=pages, kv_heads=heads, table_width=7)
        assert rc == (-4 if own else -14), (pages, heads, ps, hs)
    assert met == {True, False}
    # two sides with the same strides: refused where a float is one of both
    shared = 0
    for _ in range(3000):
        pages, heads = rng.randint(1, 9), rng.randint(1, 6)
        ps, hs, off = rng.randint(0, 12), rng.randint(0, 12), rng.randint(-40, 40)
        k, v = (floats(x, ps, hs, pages, heads) for x in (0, 4 * off))
        if len(set(k)) == len(k) and set(k) & set(v):
            shared += 1
            sc = dict(k_page_stride=ps, k_head_stride=hs, v_page_stride=ps, v_head_stride=hs,
                      v=FAKE + 4 * off)
            assert append_rc(scales=sc, num_pages=pages, kv_heads=heads, v_cache=FAKE + (1 << 20)) == -14
    assert shared > 300
