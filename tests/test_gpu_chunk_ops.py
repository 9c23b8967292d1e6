"""GPU parity of pa_rope_append, pa_move_blocks and the cache's chunk steps
against the oracle (needs a B200)."""

import math

import numpy as np
import pytest
import torch

from gpu_cases import TORCH
from oracle import OraclePool, oracle_append, oracle_copy_blocks, oracle_prefill, oracle_rope
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


def assert_turned(got, ref, x, dtype, where=""):
    """|got - ref| <= u |ref| (rounding to the type) + 8 2^-24 r, where r = the pair's length, at most the sum of
    the two elements' sizes: cos and sin are off by 2^-22 at most (the reduced turn is rounded once to 32 bits, and
    the function adds up to two units), each product and the sum are rounded once."""
    got, ref = got.double().cpu().numpy(), np.asarray(ref)
    u = torch.finfo(TORCH[dtype]).eps / 2
    r = np.abs(x).max(axis=-1, keepdims=True) * 2
    err = np.abs(got - ref) - u * np.abs(ref)
    assert (err <= 8 * 2.0 ** -24 * r + 2.0 ** -25 * (dtype == "f16")).all(), "%s: %g" % (where, err.max())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq,hkv,d,rotary", [(4, 2, 128, 128), (8, 8, 64, 32), (3, 1, 128, 22), (2, 2, 64, 6),
                                             (1, 1, 96, 96), (40, 8, 128, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [1, 3])
def test_rope_append_matches_oracle(pa, dtype, hq, hkv, d, rotary, interleaved, axes):
    rng = np.random.default_rng(d + rotary + axes)
    t, nb, bs = 37, 6, 16
    q, k, v = (workloads.randn((t, h, d), dtype, i) for i, h in enumerate((hq, hkv, hkv)))
    pos = rng.integers(-5000, 2000000, (axes, t)).astype(np.int32)
    freq = (1e4 ** (-np.arange(rotary // 2) / (rotary // 2))).astype(np.float32)
    axis = rng.integers(0, axes, rotary // 2).astype(np.int32) if axes > 1 else None
    slots = rng.permutation(nb * bs)[:t].astype(np.int64)
    slots[5] = -1
    slots[6] = -7
    kc, vc = workloads.randn((nb, bs, hkv, d), dtype, 7), workloads.randn((nb, bs, hkv, d), dtype, 8)
    dk, dv, dq = kc.cuda(), vc.cuda(), q.cuda()
    out = torch.full_like(dq, 9.0)
    pa.pa_rope_append(dq, k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(),
                      torch.from_numpy(slots).cuda(), dk, dv, out,
                      pair_axis=None if axis is None else torch.from_numpy(axis).cuda(), interleaved=interleaved)
    assert pa.pa_device_error() == 0
    qd, kd = q.double().numpy(), k.double().numpy()
    assert_turned(out, oracle_rope(qd, pos, freq, axis, interleaved), qd, dtype, "q")
    ek, ev = kc.double().numpy(), vc.double().numpy()
    oracle_append(ek, ev, oracle_rope(kd, pos, freq, axis, interleaved), v.double().numpy(), slots)
    assert np.array_equal(dv.double().cpu().numpy(), ev)
    rows = slots[slots >= 0]
    written = np.zeros(nb * bs, bool)
    written[rows] = True
    flat = dk.view(nb * bs, hkv, d)
    assert torch.equal(flat.cpu()[~torch.from_numpy(written)], kc.view(nb * bs, hkv, d)[~torch.from_numpy(written)])
    assert_turned(flat[torch.from_numpy(rows).cuda()], ek.reshape(nb * bs, hkv, d)[rows], kd[slots >= 0], dtype, "k")
    # elements behind the rotated width are copied bit for bit
    assert torch.equal(out[..., rotary:], dq[..., rotary:])
    # in place
    same = dq.clone()
    pa.pa_rope_append(same, k.cuda(), v.cuda(), torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(),
                      torch.from_numpy(slots).cuda(), dk, dv, same,
                      pair_axis=None if axis is None else torch.from_numpy(axis).cuda(), interleaved=interleaved)
    assert torch.equal(same, out)


@pytest.mark.parametrize("t", [1, 700])
def test_rope_append_takes_slices_of_one_projection(pa, t):
    """q, k and v as views of one [T, (Hq + 2 Hkv) D] product; large and small token counts."""
    hq, hkv, d, bs = 8, 2, 128, 16
    qkv = workloads.randn((t, hq + 2 * hkv, d), "bf16", 3).cuda()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    nb = -(-t // bs)
    kc, vc = (torch.zeros((nb, bs, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.arange(t, dtype=torch.int32, device="cuda")
    freq = torch.from_numpy((1e4 ** (-np.arange(64) / 64)).astype(np.float32)).cuda()
    out = torch.empty((t, hq, d), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_rope_append(q, k, v, pos, freq, pos.long(), kc, vc, out, stream=side)
    side.synchronize()
    p = pos.cpu().numpy()[None]
    for got, x in ((out, q), (kc.view(-1, hkv, d)[:t], k)):
        xd = x.double().cpu().numpy()
        assert_turned(got, oracle_rope(xd, p, freq.cpu().numpy()), xd, "bf16")
    assert torch.equal(vc.view(-1, hkv, d)[:t], v)
    with pytest.raises(ValueError):
        pa.pa_rope_append(qkv.transpose(1, 2)[:, :, :hq].transpose(1, 2)[:, ::2], k, v, pos, freq, pos.long(), kc, vc,
                          out)


def test_rope_append_reports_bad_slots_and_axes(pa):
    x = workloads.randn((2, 1, 64), "f32", 1).cuda()
    c = torch.zeros((2, 8, 1, 64), device="cuda")
    pos = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    freq = torch.ones(32, device="cuda")
    out = torch.empty_like(x)
    pa.pa_rope_append(x, x, x, pos, freq, torch.tensor([16, 3], device="cuda"), c, c.clone(), out)
    assert pa.pa_device_error() == 3
    assert torch.equal(c.view(16, 1, 64)[3], x[1]) and int((c != 0).any(dim=-1).sum()) == 1
    axis = torch.full((32,), 2, dtype=torch.int32, device="cuda")
    pa.pa_rope_append(x, x, x, pos, freq, torch.tensor([1, 3], device="cuda"), c, c.clone(), out, pair_axis=axis)
    assert pa.pa_device_error() == 6 and torch.equal(out, x)


@pytest.mark.parametrize("dtype,layers,nb,bs,hkv,d", [("bf16", 3, 50, 16, 2, 64), ("f32", 1, 7, 8, 1, 4),
                                                     ("f16", 70, 24, 16, 1, 64), ("bf16", 2, 300, 32, 8, 128)])
def test_moves_match_oracle(pa, dtype, layers, nb, bs, hkv, d):
    rng = np.random.default_rng(nb)
    pool = pa.Pool(nb, bs, rng.permutation(nb).astype(np.int32))
    tables = np.full((5, 9), -1, np.int32)
    for r in range(5):
        n = min(9, nb // 7)
        tables[r, :n] = pool.pa_pool_alloc(n)
    pool.pa_pool_fork(tables[1, :1])
    tables[0, 8] = tables[1, 0]
    kh = [workloads.randn((nb, bs, hkv, d), dtype, i) for i in range(layers)]
    vh = [workloads.randn((nb, bs, hkv, d), dtype, 100 + i) for i in range(layers)]
    dk, dv = [k.cuda() for k in kh], [v.cuda() for v in vh]
    wide = torch.full((5, 12), -5, dtype=torch.int32, device="cuda")
    dt = wide[:, :9]                                              # a strided view
    dt.copy_(torch.from_numpy(tables))
    moves = pool.pa_pool_compact(tables)
    assert len(moves)
    pa.pa_move_blocks(dk, dv, torch.from_numpy(moves).cuda(), dt)
    assert pa.pa_device_error() == 0
    assert np.array_equal(dt.cpu().numpy(), tables) and (wide[:, 9:] == -5).all()
    for i in range(layers):
        oracle_copy_blocks(kh[i], vh[i], moves)
        assert torch.equal(dk[i].cpu(), kh[i]) and torch.equal(dv[i].cpu(), vh[i])


def test_moves_report_bad_ids_and_order(pa):
    k = workloads.randn((6, 8, 1, 64), "f32", 1).cuda()
    v, before = k.clone() + 1, k.clone()
    pa.pa_move_blocks([k], [v], torch.tensor([[4, 1], [6, 0]], dtype=torch.int32, device="cuda"))
    assert pa.pa_device_error() == 4
    assert torch.equal(k[1], before[4]) and torch.equal(k[0], before[0])
    pa.pa_move_blocks([k], [v], torch.tensor([[5, 1], [4, 0]], dtype=torch.int32, device="cuda"))
    assert pa.pa_device_error() == 7
    pa.pa_move_blocks([k], [v], torch.zeros((0, 2), dtype=torch.int32, device="cuda"))
    assert pa.pa_device_error() == 0


def test_compaction_of_a_cache_with_several_layers(pa):
    """`PagedKVCache.compact` moves further layers that share its pool and tables."""
    from paged_kv_cache_341_b200.cache import PagedKVCache
    rng = np.random.default_rng(3)
    cache = PagedKVCache(30, 16, 2, 64, torch.float16, 3, 8, initial_free_order=rng.permutation(30), fill=0.0)
    layers = [tuple(workloads.randn((30, 16, 2, 64), "f16", 10 * i + j).cuda() for j in range(2)) for i in range(3)]
    for r in range(3):
        cache.allocate(r, 40 + 30 * r)
    cache.upload_tables()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids = [torch.from_numpy(cache.tables[r, :-(-int(cache.lens[r]) // 16)].astype(np.int64)) for r in range(3)]
    before = [[[c[i.cuda()].cpu() for i in ids] for c in pair] for pair in layers]
    moves = cache.compact(layers=layers, stream=side)
    side.synchronize()
    assert len(moves) and np.array_equal(cache.d_tables.cpu().numpy(), cache.tables)
    for pair, old in zip(layers, before):
        for c, rows in zip(pair, old):
            for r in range(3):
                now = torch.from_numpy(cache.tables[r, :len(ids[r])].astype(np.int64))
                assert torch.equal(c[now.cuda()].cpu(), rows[r])
    assert len(cache.compact(layers=layers)) == 0


def _rows(cache, row):
    n = int(cache.lens[row])
    ids = cache.tables[row, :-(-n // cache.block_size)]
    return (c[torch.from_numpy(ids.astype(np.int64)).cuda()].reshape(-1, cache.num_kv_heads, cache.head_dim)[:n]
            .double().cpu().numpy() for c in (cache.k_cache, cache.v_cache))


def test_prompts_in_chunks_fork_compact_and_decode(pa):
    """Prompts in ragged chunks with rotary positions, a fork, chunks after the fork (copy-on-write), a release and a
    compaction, then decode steps: every output against the oracle over a history kept in plain arrays."""
    from paged_kv_cache_341_b200.cache import PagedKVCache
    hq, hkv, d, bs, scale = 8, 2, 128, 16, 0.09
    rng = np.random.default_rng(12)
    cache = PagedKVCache(80, bs, hkv, d, torch.bfloat16, 4, 24, initial_free_order=rng.permutation(80),
                         fill=float("nan"))
    cache.upload_tables()
    freq = (1e4 ** (-np.arange(64) / 64)).astype(np.float32)
    dfreq = torch.from_numpy(freq).cuda()
    hist_k, hist_v = [np.zeros((0, hkv, d)) for _ in range(4)], [np.zeros((0, hkv, d)) for _ in range(4)]
    seed = 100

    def step(counts):
        nonlocal seed
        seed += 10
        t = sum(counts)
        q, k, v = (workloads.randn((t, h, d), "bf16", seed + i) for i, h in enumerate((hq, hkv, hkv)))
        lens0 = cache.lens.copy()
        out = torch.full((t, hq, d), 77.0, dtype=torch.bfloat16, device="cuda")
        cache.prefill_step(q.cuda(), k.cuda(), v.cuda(), out, scale, counts, inv_freq=dfreq)
        assert pa.pa_device_error() == 0
        assert np.array_equal(cache.d_tables.cpu().numpy(), cache.tables)
        assert np.array_equal(cache.d_lens.cpu().numpy(), cache.lens)
        at = 0
        for r, n in enumerate(counts):
            if n == 0:
                continue
            pos = (lens0[r] + np.arange(n))[None]
            rk = oracle_rope(k[at:at + n].double().numpy(), pos, freq)
            rq = oracle_rope(q[at:at + n].double().numpy(), pos, freq)
            rk = torch.from_numpy(rk).bfloat16().double().numpy()          # as the cache holds them
            rq = torch.from_numpy(rq).bfloat16().double().numpy()
            hist_k[r] = np.concatenate([hist_k[r], rk])
            hist_v[r] = np.concatenate([hist_v[r], v[at:at + n].double().numpy()])
            got_k, got_v = _rows(cache, r)
            assert np.array_equal(got_v, hist_v[r])
            assert np.abs(got_k - hist_k[r]).max() <= 2 ** -7 * np.abs(hist_k[r]).max()   # a rounding may fall either way
            ref = oracle_prefill(rq, got_k[None], got_v[None], [[0]], [len(got_k)], [0, n], scale)
            err = np.abs(out[at:at + n].double().cpu().numpy() - ref)
            # the output's and the weights' roundings (2^-8 each of values up to max |V|), and the queries' whose
            # last bit may differ from the oracle's
            assert (err <= 2 ** -6 * np.abs(got_v).max()).all(), err.max()
            at += n

    step([40, 7, 0, 100])
    step([1, 30, 0, 17])
    cache.share(0, 2)
    hist_k[2], hist_v[2] = hist_k[0].copy(), hist_v[0].copy()
    cache.upload_tables()
    step([3, 0, 5, 1])                                            # copy-on-write of the shared last block
    cache.release(3)
    hist_k[3], hist_v[3] = np.zeros((0, hkv, d)), np.zeros((0, hkv, d))
    cache.upload_tables()
    moves = cache.compact()
    live = 80 - cache.pool.pa_pool_num_free()
    assert len(moves) and cache.tables.max() < live
    assert np.array_equal(cache.d_tables.cpu().numpy(), cache.tables)
    for r in range(3):
        got_k, got_v = _rows(cache, r)
        assert np.array_equal(got_v, hist_v[r])
    step([1, 1, 1, 1])
    step([0, 64, 2, 20])
    # a decode step over the same rows
    q, k, v = (workloads.randn((4, h, d), "bf16", 900 + i).cuda() for i, h in enumerate((hq, hkv, hkv)))
    out = torch.empty((4, hq, d), dtype=torch.bfloat16, device="cuda")
    cache.decode_step(q, k, v, out, scale)
    for r in range(4):
        got_k, got_v = _rows(cache, r)
        ref = oracle_prefill(q[r:r + 1].double().cpu().numpy(), got_k[None], got_v[None], [[0]], [len(got_k)], [0, 1],
                             scale)
        assert np.abs(out[r:r + 1].double().cpu().numpy() - ref).max() <= 2 ** -6 * np.abs(got_v).max()


def test_cross_attention_over_a_cache_of_encoder_states(pa):
    from paged_kv_cache_341_b200.cache import PagedKVCache
    cache = PagedKVCache(40, 16, 4, 64, torch.float16, 3, 16)
    lens = [150, 33, 0]
    k, v = (workloads.randn((sum(lens), 4, 64), "f16", i) for i in (1, 2))
    slots, _, _ = cache.pool.pa_reserve_chunks(cache.tables, cache.lens, lens)
    cache.append(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda())
    cache.upload_tables()
    starts = torch.tensor([0, 5, 25, 30], dtype=torch.int32, device="cuda")
    q = workloads.randn((30, 4, 64), "f16", 3)
    out = torch.empty((30, 4, 64), dtype=torch.float16, device="cuda")
    cache.attend_chunks(q.cuda(), starts, out, 0.125, causal=False)
    kh, vh = cache.k_cache.double().cpu().numpy(), cache.v_cache.double().cpu().numpy()
    ref = oracle_prefill(q.double().numpy(), kh, vh, cache.tables, lens, starts.cpu().numpy(), 0.125, causal=False)
    # roundings of weights and output (2^-11 each, |out| <= max |V|), and 2 ctx 2^-23 of the float32 sums
    assert np.abs(out.double().cpu().numpy() - ref).max() <= (2 * 2 ** -11 + 300 * 2 ** -23) * np.abs(v.double().numpy()).max()
    assert (out[25:] == 0).all()


def test_prefill_step_refuses_before_it_reserves(pa):
    from paged_kv_cache_341_b200.cache import PagedKVCache
    cache = PagedKVCache(4, 16, 2, 64, torch.bfloat16, 2, 4)
    cache.upload_tables()
    q, k = (torch.zeros((5, h, 64), dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    for counts, args in (([3, 1], (q, k, k, q)), ([5], (q, k, k, q)), ([6, -1], (q, k, k, q)),
                         ([4, 1], (q, k, k[:4], q)), ([4, 1], (q, k, k, q[:4])),
                         ([4, 1], (k.new_zeros((5, 6, 64)), k, k, k.new_zeros((5, 6, 64))))):
        with pytest.raises(ValueError):
            cache.prefill_step(*args, 0.1, counts)
    with pytest.raises(TypeError):
        cache.prefill_step(q.float(), k, k, q, 0.1, [4, 1])
    freq = torch.ones(32, device="cuda")
    for kw in (dict(inv_freq=freq, positions=torch.zeros(4, dtype=torch.int32, device="cuda")),
               dict(inv_freq=torch.ones(33, device="cuda")),
               dict(inv_freq=freq, pair_axis=torch.zeros(31, dtype=torch.int32, device="cuda")),
               dict(inv_freq=freq, q_out=q[:4]), dict(inv_freq=freq, q_out=q.float())):
        with pytest.raises(ValueError):
            cache.prefill_step(q, k, k, q.clone(), 0.1, [4, 1], **kw)
    for kw in (dict(inv_freq=freq.double()), dict(inv_freq=freq, positions=torch.zeros(5, device="cuda"))):
        with pytest.raises(TypeError):
            cache.prefill_step(q, k, k, q.clone(), 0.1, [4, 1], **kw)
    wide = torch.zeros((5, 8, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):                                # strided rows need the rotary append
        cache.prefill_step(wide[:, :4], k, k, q.clone(), 0.1, [4, 1])
    with pytest.raises(ValueError):
        cache.compact(layers=[(cache.k_cache, cache.v_cache.clone())])
    with pytest.raises(ValueError):
        cache.compact(layers=[(cache.k_cache[:2], cache.v_cache.clone())])
    with pytest.raises(pa.PoolExhausted):
        big = torch.zeros((70, 4, 64), dtype=torch.bfloat16, device="cuda")
        kv = torch.zeros((70, 2, 64), dtype=torch.bfloat16, device="cuda")
        cache.prefill_step(big, kv, kv, big.clone(), 0.1, [35, 35])
    assert cache.lens.sum() == 0 and cache.pool.pa_pool_num_free() == 4 and (cache.tables == -1).all()
    assert math.isfinite(float(q.sum()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_beyond_32_bits(pa, dtype):
    """The last blocks of a cache of more than 2^31 elements: attention, append and moves give the bits that they
    give in a small cache."""
    hq, hkv, d, bs, nb = 8, 8, 128, 16, 140000
    t, ctx = 20, 300
    n = -(-ctx // bs)
    dt = TORCH[dtype]
    big = [torch.empty((nb, bs, hkv, d), dtype=dt, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 31
    small = [workloads.randn((n + 2, bs, hkv, d), dtype, i).cuda() for i in range(2)]
    high = nb - 1 - torch.arange(n + 2)                           # block i of the small cache is block high[i]
    for b, s in zip(big, small):
        b[high.cuda()] = s
    q, k, v = (workloads.randn((t, h, d), dtype, 10 + i).cuda() for i, h in enumerate((hq, hkv, hkv)))
    pos = torch.arange(ctx - t, ctx, dtype=torch.int32, device="cuda")
    freq = torch.ones(64, device="cuda") / torch.arange(1, 65, device="cuda")
    starts = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    lens = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    results = []
    for caches, ids in ((small, torch.arange(n + 2)), (big, high)):
        token = torch.arange(ctx - t, ctx)
        slots = (ids[token // bs].long() * bs + token % bs).cuda()
        q_out, out = torch.empty_like(q), torch.empty_like(q)
        table = ids[:n].to(torch.int32)[None].cuda()
        pa.pa_rope_append(q, k, v, pos, freq, slots, *caches, q_out)
        pa.pa_prefill_attention(q_out, *caches, table, lens, starts, 0.09, out)
        pair = sorted([int(ids[0]), int(ids[n])])                 # one block on to an unused one
        moves = torch.tensor([pair], dtype=torch.int32, device="cuda")
        pa.pa_move_blocks([caches[0]], [caches[1]], moves)
        assert pa.pa_device_error() == 0
        assert torch.equal(caches[0][pair[0]], caches[0][pair[1]])
        results.append((out, q_out, caches[0].view(-1, hkv, d)[slots], caches[1].view(-1, hkv, d)[slots]))
    for a, b in zip(*results):
        assert torch.equal(a, b)
