"""Chunk steps and compactions that are refused leave the host and device state
as it was, and the same call put right then works (needs a B200)."""

import numpy as np
import pytest
import torch

from paged_kv_cache_341_b200 import workloads

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 4, 2, 64, 16


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_341_b200 import build
    build.ensure_built()
    from paged_kv_cache_341_b200 import pa as mod
    assert mod.pa_device_error(reset=True) == 0
    return mod


def shifted(x, elements=4):
    """A copy of ``x`` whose address is 8 bytes past a 16-byte boundary (two-byte elements)."""
    buf = torch.zeros(x.numel() + 8, dtype=x.dtype, device=x.device)
    y = buf[elements:elements + x.numel()].view_as(x)
    y.copy_(x)
    assert y.data_ptr() % 16 == 8
    return y


def filled(counts=(20, 3)):
    """A cache with a first chunk in it, one row shared, and the tensors of a second step."""
    from paged_kv_cache_341_b200.cache import PagedKVCache
    cache = PagedKVCache(12, BS, HKV, D, torch.bfloat16, 3, 4, fill=0.0)
    cache.upload_tables()
    freq = torch.ones(D // 2, device="cuda") / torch.arange(1, D // 2 + 1, device="cuda")
    t = sum(counts)
    q, k, v = (workloads.randn((t, h, D), "bf16", 50 + i).cuda() for i, h in enumerate((HQ, HKV, HKV)))
    cache.prefill_step(q, k, v, torch.empty_like(q), 0.1, counts, rows=slice(0, 2), inv_freq=freq)
    cache.share(0, 2)
    cache.upload_tables()
    q, k, v = (workloads.randn((30, h, D), "bf16", 60 + i).cuda() for i, h in enumerate((HQ, HKV, HKV)))
    return cache, q, k, v, freq


def state(cache):
    torch.cuda.synchronize()
    refs, free = cache.pool.pa_pool_export()
    return [cache.tables.copy(), cache.lens.copy(), refs, free] + [
        x.clone() for x in (cache.d_tables, cache.d_lens, cache.k_cache, cache.v_cache)]


def same(a, b):
    return all(torch.equal(x, y) if isinstance(x, torch.Tensor) else np.array_equal(x, y) for x, y in zip(a, b))


def strided(x):
    """The same values as a view of rows twice as wide."""
    wide = torch.zeros((x.shape[0], 2 * x.shape[1], x.shape[2]), dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def bad_steps(pa, q, k, v, freq):
    out = torch.zeros_like(q)
    need = pa.pa_prefill_workspace_size(30, 3, HQ, HKV, D, 4, BS)
    room = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    yield "short workspace", (q, k, v, out, 0.1), dict(workspace=room[:need - 1])
    yield "misaligned workspace", (q, k, v, out, 0.1), dict(workspace=room[16:])
    yield "workspace on the host", (q, k, v, out, 0.1), dict(workspace=room.cpu())
    yield "strided workspace", (q, k, v, out, 0.1), dict(
        workspace=torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2])
    for scale in (float("nan"), float("inf"), float("-inf"), 2.4e38, 1e39):
        yield "scale %g" % scale, (q, k, v, out, scale), {}
    for kw in ({}, dict(inv_freq=freq)):
        yield "misaligned out", (q, k, v, shifted(out), 0.1), kw
        yield "misaligned q", (shifted(q), k, v, out, 0.1), kw
        yield "misaligned k", (q, shifted(k), v, out, 0.1), kw
        yield "misaligned v", (q, k, shifted(v), out, 0.1), kw
        yield "a number as stream", (q, k, v, out, 0.1), dict(kw, stream=7)
    yield "k rows one over another", (q, k[:1].expand(30, HKV, D), v, out, 0.1), dict(inv_freq=freq)
    yield "misaligned q_out", (q, k, v, out, 0.1), dict(inv_freq=freq, q_out=shifted(q))
    wide = strided(q)
    yield "q_out over strided q", (wide, k, v, out, 0.1), dict(
        inv_freq=freq, q_out=wide.as_strided((30, HQ, D), (HQ * D, D, 1)))


def test_refused_steps_leave_the_state_as_it_was(pa):
    cache, q, k, v, freq = filled()
    before = state(cache)
    for name, args, kw in bad_steps(pa, q, k, v, freq):
        with pytest.raises((ValueError, TypeError, pa.PagedAttnError)):
            cache.prefill_step(*args, [10, 15, 5], **kw)
        assert same(state(cache), before), name
    assert pa.pa_device_error() == 0
    out = torch.empty_like(q)
    room = torch.empty(pa.pa_prefill_workspace_size(30, 3, HQ, HKV, D, 4, BS), dtype=torch.uint8, device="cuda")
    cache.prefill_step(q, strided(k), v, out, 0.1, [10, 15, 5], inv_freq=freq, workspace=room)
    other, q2, k2, v2, freq2 = filled()
    want = torch.empty_like(q)
    other.prefill_step(q2, k2, v2, want, 0.1, [10, 15, 5], inv_freq=freq2)
    assert torch.equal(out, want) and same(state(cache), state(other))


def test_a_failed_allocation_leaves_the_state_as_it_was(pa, monkeypatch):
    cache, q, k, v, freq = filled()
    before = state(cache)

    def no_memory(*args, **kw):
        raise torch.OutOfMemoryError("no memory")

    for kw in ({}, dict(inv_freq=freq)):
        with monkeypatch.context() as m:
            m.setattr(pa, "prefill_workspace", no_memory)
            with pytest.raises(torch.OutOfMemoryError):
                cache.prefill_step(q, k, v, torch.empty_like(q), 0.1, [10, 15, 5], **kw)
        assert same(state(cache), before)


def test_one_row_of_any_stride_and_steps_of_no_tokens(pa):
    """A single token's row stride says nothing; a step of no tokens changes nothing."""
    cache, q, k, v, freq = filled()
    before = state(cache)
    empty = [x[:0].contiguous() for x in (q, k, v)]
    for kw in ({}, dict(inv_freq=freq)):
        slots, pairs = cache.prefill_step(*empty, torch.empty_like(empty[0]), 0.1, [0, 0, 0], **kw)
        assert slots.size == 0 and len(pairs) == 0 and same(state(cache), before)
    out = torch.empty_like(q[:1])
    odd = k[:1].as_strided((1, HKV, D), (7, D, 1))
    cache.prefill_step(q[:1], odd, v[:1], out, 0.1, [0, 1, 0], inv_freq=freq)
    other = filled()[0]
    want = torch.empty_like(out)
    other.prefill_step(q[:1], k[:1], v[:1], want, 0.1, [0, 1, 0], inv_freq=freq)
    assert torch.equal(out, want) and same(state(cache), state(other))


def test_refused_compactions_leave_the_state_as_it_was(pa):
    cache, q, k, v, freq = filled()
    cache.release(0)
    cache.release(2)                                              # (row 0's sharer: now there is a block to move)
    cache.upload_tables()
    before = state(cache)
    shape = cache.k_cache
    other = [torch.randn_like(shape), torch.randn_like(shape)]
    bad = [dict(layers=[(shifted(other[0]), other[1])]), dict(layers=[(other[0], shifted(other[1]))]),
           dict(layers=[(other[0].cpu(), other[1].cpu())]), dict(layers=[(other[0], other[1], other[1])]),
           dict(layers=[(other[0],)]), dict(layers=[(other[0], other[0])]), dict(layers=[(shape, other[1])]),
           dict(layers=[(other[0].float(), other[1].float())]), dict(stream=7)]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, pa.PagedAttnError)):
            cache.compact(**kw)
        assert same(state(cache), before), str(kw)
    old = [c.clone() for c in other]
    moves = cache.compact(layers=iter([tuple(other)]))            # (any iterable of pairs)
    assert len(moves)
    for now, was in zip(other, old):
        assert torch.equal(now[moves[:, 1].tolist()], was[moves[:, 0].tolist()])
    assert np.array_equal(cache.d_tables.cpu().numpy(), cache.tables)
    assert pa.pa_device_error() == 0


def test_compaction_of_blocks_that_fill_no_16_bytes_is_refused(pa):
    from paged_kv_cache_341_b200.cache import PagedKVCache
    cache = PagedKVCache(6, 1, 1, 2, torch.float32, 2, 4, initial_free_order=[5, 4, 3, 2, 1, 0], fill=0.0)
    cache.allocate(0, 2)
    cache.upload_tables()
    before = state(cache)
    with pytest.raises((ValueError, pa.PagedAttnError)):
        cache.compact()
    assert same(state(cache), before)


@pytest.mark.parametrize("shape", [(2, 3), (4,), (3,), (2, 2, 1), (1, 4)])
def test_move_lists_that_are_not_pairs_are_refused(pa, shape):
    """A list laid out as all sources, then all destinations, would be taken for other pairs."""
    k, v = (workloads.randn((8, 8, 1, 64), "f32", i).cuda() for i in (1, 2))
    old = k.clone(), v.clone()
    moves = torch.arange(int(np.prod(shape)), dtype=torch.int32, device="cuda").reshape(shape)
    with pytest.raises(ValueError):
        pa.pa_move_blocks([k], [v], moves)
    torch.cuda.synchronize()
    assert torch.equal(k, old[0]) and torch.equal(v, old[1])
