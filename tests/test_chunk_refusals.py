"""Calls of the chunk operators that are refused before anything is launched (CPU only)."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def pa(built_library):
    from paged_kv_cache_341_b200 import pa as mod
    return mod


@pytest.fixture
def caches():
    return torch.zeros(16, 8, 1, 64), torch.zeros(16, 8, 1, 64)


@pytest.mark.parametrize("table", [
    torch.zeros(1, 8, dtype=torch.int32).expand(4, 8),            # one row four times
    torch.zeros(40, dtype=torch.int32).as_strided((4, 8), (3, 1)),
    torch.zeros(8, 4, dtype=torch.int32).t(),
    torch.zeros(32, dtype=torch.int32),
])
def test_moves_refuse_tables_whose_rows_overlap(pa, caches, table):
    """Rows are written `stride` apart: rows that overlap have no such stride."""
    k, v = caches
    with pytest.raises(ValueError):
        pa.pa_move_blocks([k], [v], torch.zeros(1, 2, dtype=torch.int32), table)


@pytest.mark.parametrize("table", [torch.zeros(4, 12, dtype=torch.int32)[:, :9], torch.zeros(1, 8, dtype=torch.int32),
                                   torch.zeros(3, 8, dtype=torch.int32)[1:2].expand(1, 8), torch.zeros(0, 8)])
def test_strided_and_single_rows_pass_the_shape_checks(pa, caches, table):
    """(CPU tensors: refused for that alone)"""
    k, v = caches
    with pytest.raises(TypeError):
        pa.pa_move_blocks([k], [v], torch.zeros(1, 2, dtype=torch.int32), table)


@pytest.mark.parametrize("scale,bad", [(2.4e38, True), (-2.4e38, True), (3.0e38, True), (float("-inf"), True),
                                       (2.3e38, False), (-2.3e38, False), (0.0, False)])
def test_scales_that_overflow_in_units_of_log2(pa, scale, bad):
    """The largest float32 is 3.403e38, 2.359e38 times log2(e): beyond it a zero score would be 0 * inf."""
    fake = ctypes.c_void_p(1 << 20)                               # never dereferenced: no workspace is given
    assert pa._lib.pa_prefill_attention(fake, fake, fake, 16, fake, 4, fake, fake, 10, 2, 4, 2, 64, 16, scale, 1, None,
                                        0, fake, pa.PA_BF16, None) == pa.PA_ERR_INVALID
    assert ("scale" if bad else "workspace") in pa.pa_last_error()
