"""Caches whose own tensors overlap are refused where they would be written.  No GPU."""
import pytest

from causal_scaled_dot_gb300.native import ATTN_ERR_INVALID_ARG
from tests.test_cache_cpu import T, cache, call_write


@pytest.mark.parametrize("kw", [
    dict(v=T), dict(v=T + 64 * 128 * 16), dict(k_scale=T + 4096), dict(v_scale=2 * T), dict(v_scale=3 * T), dict(v_scale=3 * T + 4),
    dict(block_table=T + 128), dict(block_table=4 * T), dict(seq_lens=3 * T + 796), dict(seq_lens=2 * T + 16),
])
def test_write_into_overlapping_tensors_is_refused(kw):
    assert call_write(cache(**kw)) == ATTN_ERR_INVALID_ARG
