"""Calls of the chunk operators that are refused before anything is launched (CPU only)."""

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
