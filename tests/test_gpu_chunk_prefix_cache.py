"""A prefix-cached prompt brought into the cache in chunks: the row's own blocks
take its tokens, and attention reads the shared ones (needs a B200)."""

import numpy as np
import pytest
import torch

from paged_kv_cache_341_b200 import workloads

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 8, 2, 128, 16


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_341_b200 import build
    build.ensure_built()
    from paged_kv_cache_341_b200 import pa as mod
    assert mod.pa_device_error(reset=True) == 0
    return mod


def test_prefix_cached_prompt_in_chunks(pa):
    """Equal bits to the same prompts in blocks of their own, through ``prefill_step``."""
    from paged_kv_cache_341_b200.cache import PagedKVCache
    system, own = 48, (12, 30)
    freq = torch.from_numpy((1e4 ** (-np.arange(D // 2) / (D // 2))).astype(np.float32)).cuda()
    tokens = [list(range(system)) + [1000 * (r + 1) + i for i in range(own[r])] for r in range(2)]
    rows = [[workloads.randn((len(t), h, D), "bf16", 10 * r + i).cuda() for i, h in enumerate((HQ, HKV, HKV))]
            for r, t in enumerate(tokens)]
    for a, b in zip(rows[0], rows[1]):
        b[:system] = a[:system]                                   # the system prompt's rows are the same

    def cache_of():
        c = PagedKVCache(40, BS, HKV, D, torch.bfloat16, 2, 8, fill=float("nan"))
        c.upload_tables()
        return c

    plain, shared = cache_of(), cache_of()
    shared.pool.pa_pool_enable_prefix_cache()
    for r, (q, k, v) in enumerate(rows):
        cached = shared.pool.pa_seq_alloc_prompt(tokens[r], shared.tables[r])
        assert cached == (0, system)[r]
        with pytest.raises(pa.PagedAttnError):                    # the row holds its blocks
            shared.lens[r] = cached
            shared.prefill_step(q[cached:], k[cached:], v[cached:], torch.empty_like(q[cached:]), 0.09,
                                [len(q) - cached], rows=slice(r, r + 1), inv_freq=freq)
        n = len(tokens[r])
        shared.lens[r] = n
        shared.upload_tables()
        at = np.arange(cached, n)
        slots = torch.from_numpy(shared.tables[r][at // BS].astype(np.int64) * BS + at % BS).cuda()
        turned, out = torch.empty_like(q[cached:]), torch.empty_like(q[cached:])
        pa.pa_rope_append(q[cached:], k[cached:], v[cached:], torch.from_numpy(at.astype(np.int32)).cuda(), freq, slots,
                          shared.k_cache, shared.v_cache, turned)
        starts = torch.tensor([0, n - cached], dtype=torch.int32, device="cuda")
        shared.attend_chunks(turned, starts, out, 0.09, tables=shared.d_tables[r:r + 1], lens=shared.d_lens[r:r + 1])
        for lo, hi in ((0, cached), (cached, n)):
            want = torch.empty_like(q[lo:hi])
            plain.prefill_step(q[lo:hi], k[lo:hi], v[lo:hi], want, 0.09, [hi - lo], rows=slice(r, r + 1), inv_freq=freq)
        assert torch.equal(out, want)
    # both go on alike, in blocks of their own
    q, k, v = (workloads.randn((25, h, D), "bf16", 70 + i).cuda() for i, h in enumerate((HQ, HKV, HKV)))
    outs = [torch.empty_like(q) for _ in range(2)]
    for c, o in zip((plain, shared), outs):
        c.prefill_step(q, k, v, o, 0.09, [5, 20], inv_freq=freq)
    assert torch.equal(*outs)
    assert pa.pa_device_error() == 0
    for r in range(2):
        shared.release(r)
    assert shared.pool.pa_pool_num_free() == 40 and shared.pool.pa_pool_cached_blocks() == 0
