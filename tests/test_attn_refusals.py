"""Host-side refusals of the attention entry points with options, through the
binding (no GPU)."""

import pytest

from bit_rotated_kv_block_b200 import kvq


def test_a_softcap_that_float32_cannot_hold_is_refused():
    for cap in (1e-50, -1e-60):
        with pytest.raises(ValueError):
            kvq.Score(softcap=cap)       # it would act as no cap
    assert kvq.Score(softcap=0.0).desc.softcap == 0.0
    assert kvq.Score(softcap=50.0).desc.softcap == 50.0
