"""Refusals of the operators that use the selection, at the ends of ranges."""

import pytest

from test_serving_abi import attend


@pytest.mark.parametrize("kw", [dict(sm_scale=2.4e38), dict(sm_scale=3e38),
                                dict(sm_scale=1e30, k_scale=3e8)])
def test_scales_whose_base_2_scores_overflow(kw):
    """Scores are taken to base 2: the scale times log2(e) has to be finite too."""
    assert attend(**kw) == -1
    # (the largest one gets past this check, to the table's)
    assert attend(sm_scale=2.3e38, table_width=7) == -4
