"""Chunk steps in the forms a serving loop uses them: a range of rows, positions
of several axes, slices of one projection, every cache type, and a compaction
between an engine's steps (needs a B200)."""

import math

import numpy as np
import pytest
import torch

from gpu_cases import TORCH, assert_close
from oracle import oracle_prefill, oracle_rope
from paged_kv_cache_341_b200 import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_341_b200 import build
    build.ensure_built()
    from paged_kv_cache_341_b200 import pa as mod
    assert mod.pa_device_error(reset=True) == 0
    return mod


def history(cache, row):
    n = int(cache.lens[row])
    ids = torch.from_numpy(cache.tables[row, :-(-n // cache.block_size)].astype(np.int64)).cuda()
    return [c[ids].reshape(-1, cache.num_kv_heads, cache.head_dim)[:n].double().cpu().numpy()
            for c in (cache.k_cache, cache.v_cache)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,interleaved", [(64, True), (128, False)])
def test_ranges_of_rows_with_positions_of_three_axes(pa, dtype, d, interleaved):
    """Steps of rows 2..4 of 6 on a side stream, q, k and v slices of one projection; other rows stay as they were."""
    from paged_kv_cache_341_b200.cache import PagedKVCache
    hq, hkv, bs, scale = 8, 2, 16, 1 / math.sqrt(d)
    cache = PagedKVCache(90, bs, hkv, d, TORCH[dtype], 6, 12, initial_free_order=np.random.default_rng(1).permutation(90),
                         fill=float("nan"))
    cache.upload_tables()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    half = d // 2
    freq = (1e4 ** (-np.arange(half) / half)).astype(np.float32)
    axis = (np.arange(half) * 3 // half).astype(np.int32)
    dfreq, daxis = torch.from_numpy(freq).cuda(), torch.from_numpy(axis).cuda()
    rng = np.random.default_rng(2)
    u = torch.finfo(TORCH[dtype]).eps / 2
    for step, (rows, counts) in enumerate([(slice(2, 5), [30, 0, 100]), (slice(2, 5), [1, 17, 40]),
                                           (slice(4, 6), [3, 5]), (slice(0, 1), [20])]):
        t = sum(counts)
        qkv = workloads.randn((t, hq + 2 * hkv, d), dtype, 40 + step).cuda()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        pos = rng.integers(0, 100000, (3, t)).astype(np.int32)
        out = torch.full((t, hq, d), 5.0, dtype=TORCH[dtype], device="cuda")
        turned = torch.empty_like(out)
        dpos = torch.from_numpy(pos).cuda()
        before = [history(cache, r) for r in range(6)]
        torch.cuda.synchronize()
        cache.prefill_step(q, k, v, out, scale, counts, rows=rows, inv_freq=dfreq, positions=dpos, pair_axis=daxis,
                           interleaved=interleaved, q_out=turned, stream=side)
        side.synchronize()
        assert pa.pa_device_error() == 0
        assert np.array_equal(cache.d_tables.cpu().numpy(), cache.tables)
        assert np.array_equal(cache.d_lens.cpu().numpy(), cache.lens)
        rq = oracle_rope(q.double().cpu().numpy(), pos, freq, axis, interleaved)
        rk = oracle_rope(k.double().cpu().numpy(), pos, freq, axis, interleaved)
        # one rounding to the type, and the pair turned in 32 bits (as derived in test_gpu_chunk_ops)
        slack = 8 * 2.0 ** -24 * 2 * np.abs(qkv.double().cpu().numpy()).max() + 2.0 ** -25 * (dtype == "f16")
        assert (np.abs(turned.double().cpu().numpy() - rq) <= u * np.abs(rq) + slack).all()
        at = 0
        for r in range(6):
            got_k, got_v = history(cache, r)
            n = counts[r - rows.start] if rows.start <= r < rows.stop else 0
            assert np.array_equal(got_k[:len(before[r][0])], before[r][0])
            assert np.array_equal(got_v[:len(before[r][1])], before[r][1])
            if n == 0:
                assert len(got_k) == len(before[r][0])
                continue
            assert np.array_equal(got_v[-n:], v[at:at + n].double().cpu().numpy())
            assert (np.abs(got_k[-n:] - rk[at:at + n]) <= u * np.abs(rk[at:at + n]) + slack).all()
            tq = turned[at:at + n].double().cpu().numpy()
            ref = oracle_prefill(tq, got_k[None], got_v[None], [[0]], [len(got_k)], [0, n], scale)
            err = np.abs(out[at:at + n].double().cpu().numpy() - ref).max()
            # weights and output rounded once each (|out| <= max |V|), 2 ctx 2^-23 of the sums, and scores off by
            # (d + 16) 2^-23 of their largest term sum, twice
            b = (np.abs(tq).reshape(n * hq, d).sum(axis=1).max() * np.abs(got_k).max()) * scale
            bound = (2 * u * (dtype != "f32") + u + 2 * len(got_k) * 2.0 ** -23 + 2 * ((d + 16) * 2.0 ** -23 * b
                                                                                      + 2.0 ** -21))
            assert err <= bound * np.abs(got_v).max()
            at += n


def test_compaction_between_the_steps_of_an_engine(pa):
    """The engine works on the cache's tables and lengths: after a compaction its steps follow the new ids."""
    from paged_kv_cache_341_b200.cache import PagedKVCache
    hq, hkv, d, bs, scale = 8, 2, 128, 16, 0.09
    cache = PagedKVCache(60, bs, hkv, d, torch.bfloat16, 4, 8, initial_free_order=np.random.default_rng(3).permutation(60),
                         fill=float("nan"))
    cache.upload_tables()
    lens = [50, 16, 31, 90]
    t = sum(lens)
    q, k, v = (workloads.randn((t, h, d), "bf16", 80 + i).cuda() for i, h in enumerate((hq, hkv, hkv)))
    cache.prefill_step(q, k, v, torch.empty_like(q), scale, lens)
    cache.release(1)                                              # a hole, and a row that starts again
    engine = cache.engine(hq)
    for step in range(4):
        q1, k1, v1 = (workloads.randn((4, h, d), "bf16", 90 + 10 * step + i).pin_memory()
                       for i, h in enumerate((hq, hkv, hkv)))
        out = torch.zeros((4, hq, d), dtype=torch.bfloat16).pin_memory()
        engine.pa_engine_step(0, 4, q1, k1, v1, out, scale)
        engine.pa_engine_synchronize()
        assert pa.pa_device_error() == 0
        hist = [history(cache, r) for r in range(4)]
        for r in range(4):
            assert np.array_equal(hist[r][1][-1], v1[r].double().numpy())
        ref = np.concatenate([oracle_prefill(q1[r:r + 1].double().numpy(), hist[r][0][None], hist[r][1][None], [[0]],
                                             [len(hist[r][0])], [0, 1], scale) for r in range(4)])
        assert_close(out.float().numpy(), ref, "bf16", "engine step %d" % step)
        moves = cache.compact()
        assert len(moves) or step > 0
        live = 60 - cache.pool.pa_pool_num_free()
        assert cache.tables.max() < live and np.array_equal(cache.d_tables.cpu().numpy(), cache.tables)
        for r in range(4):
            for a, b in zip(history(cache, r), hist[r]):
                assert np.array_equal(a, b)
    engine.close()
