"""Host side of the chunk operators (CPU only): reservation of several tokens
per sequence and compaction of the pool against the oracle, and the argument
checks of the device entry points, which run before anything is launched."""

import ctypes
import random

import numpy as np
import pytest

from oracle import OraclePool, PoolExhausted


@pytest.fixture(scope="module")
def pa(built_library):
    from paged_kv_cache_341_b200 import pa as mod
    return mod


def same_state(lp, op):
    refs, free = lp.pa_pool_export()
    orefs, ofree = op.export()
    return list(refs) == orefs and list(free) == ofree


def test_chunk_reservations_match_the_oracle(pa):
    rng = random.Random(5)
    for _ in range(80):
        nb, bs, cap, s = rng.randint(4, 60), rng.choice([1, 4, 8, 16]), 40, rng.randint(1, 5)
        order = list(range(nb))
        rng.shuffle(order)
        lp, op = pa.Pool(nb, bs, order), OraclePool(nb, bs, order)
        tables, lens = np.full((s, cap), -1, np.int32), np.zeros(s, np.int32)
        otables, olens = [[] for _ in range(s)], [0] * s
        for _ in range(12):
            if rng.random() < 0.3 and s > 1:                      # a fork: copy-on-write at the next chunk
                a, b = rng.sample(range(s), 2)
                lp.pa_pool_free(tables[b, :len(otables[b])])
                op.free(otables[b])
                lp.pa_pool_fork(tables[a, :len(otables[a])])
                op.fork(otables[a])
                tables[b], lens[b] = tables[a], lens[a]
                otables[b], olens[b] = list(otables[a]), olens[a]
            counts = [rng.choice([0, 1, rng.randint(0, 3 * bs)]) for _ in range(s)]
            before = (tables.copy(), lens.copy(), lp.pa_pool_export())
            import copy
            trial, ttables, tlens = copy.deepcopy(op), copy.deepcopy(otables), list(olens)
            slots, pairs, failed = [], [], False
            try:
                for i in range(s):
                    got, tlens[i], p = trial.reserve_chunk(ttables[i], tlens[i], counts[i], cap)
                    slots += got
                    pairs += p
            except (PoolExhausted, ValueError):
                failed = True
            if failed:
                with pytest.raises(pa.PagedAttnError):
                    lp.pa_reserve_chunks(tables, lens, counts, row0=7)
                assert np.array_equal(tables, before[0]) and np.array_equal(lens, before[1])
                refs, free = lp.pa_pool_export()
                assert np.array_equal(refs, before[2][0]) and np.array_equal(free, before[2][1])
                continue
            old = tables.copy()
            lslots, lpairs, updates = lp.pa_reserve_chunks(tables, lens, counts, row0=7)
            op, otables, olens = trial, ttables, tlens
            assert list(lslots) == slots and [tuple(p) for p in lpairs] == pairs
            assert list(lens) == olens and same_state(lp, op)
            for i in range(s):
                assert list(tables[i, :len(otables[i])]) == otables[i]
            for row, col, block in updates:                       # the updates lead from the old tables to the new
                old[row - 7, col] = block
            assert np.array_equal(old, tables)


def test_chunk_reservation_refusals(pa):
    lp = pa.Pool(4, 4)
    tables, lens = np.full((1, 8), -1, np.int32), np.zeros(1, np.int32)
    with pytest.raises(ValueError):
        lp.pa_reserve_chunks(tables, lens, [-1])
    with pytest.raises(ValueError):
        lp.pa_reserve_chunks(tables, lens, [1, 2])
    with pytest.raises(pa.PoolExhausted):
        lp.pa_reserve_chunks(tables, lens, [17])
    assert lp.pa_pool_num_free() == 4 and lens[0] == 0 and (tables == -1).all()
    lp.pa_reserve_chunks(tables, lens, [16])
    assert lens[0] == 16 and lp.pa_pool_num_free() == 0
    slots, pairs, updates = lp.pa_reserve_chunks(tables, lens, [0])
    assert slots.size == 0 and len(pairs) == 0 and len(updates) == 0
    counts = np.array([-3], np.int32)
    n = ctypes.c_int32()
    p32, p64 = pa._p32, pa._p64
    out = np.zeros(4, np.int64)
    assert pa._lib.pa_reserve_chunks(lp._h, tables.ctypes.data_as(p32), 8, lens.ctypes.data_as(p32),
                                     counts.ctypes.data_as(p32), 1, 0, out.ctypes.data_as(p64),
                                     tables.ctypes.data_as(p32), ctypes.byref(n), None, None) == pa.PA_ERR_INVALID


def test_compaction_matches_the_oracle(pa):
    rng = random.Random(6)
    for trial in range(80):
        nb, bs = rng.randint(1, 60), rng.choice([2, 4])
        order = list(range(nb))
        rng.shuffle(order)
        lp, op = pa.Pool(nb, bs, order), OraclePool(nb, bs, order)
        cached = trial % 2 == 0
        if cached:
            lp.pa_pool_enable_prefix_cache()
            op.enable_prefix_cache()
        rows = []                                                 # (library row, oracle row)
        for _ in range(14):
            if rng.random() < 0.6:
                n = rng.randint(1, 4 * bs)
                row = np.full(8, -1, np.int32)
                if -(-n // bs) > op.num_free():
                    continue
                if cached:
                    toks = [rng.randint(0, 1) for _ in range(n)]
                    lp.pa_seq_alloc_prompt(toks, row)
                    orow, _ = op.alloc_prompt(toks)
                else:
                    orow = op.alloc(-(-n // bs))
                    row[:len(orow)] = lp.pa_pool_alloc(len(orow))
                rows.append((row, orow))
            elif rows:
                if rng.random() < 0.5:
                    row, orow = rng.choice(rows)
                    lp.pa_pool_fork(orow)
                    op.fork(orow)
                    rows.append((row.copy(), list(orow)))
                else:
                    row, orow = rows.pop(rng.randrange(len(rows)))
                    lp.pa_pool_free(orow)
                    op.free(orow)
            if rng.random() < 0.3:
                tables = np.stack([r for r, _ in rows]) if rows else np.zeros((0, 8), np.int32)
                moves = lp.pa_pool_compact(tables)
                omoves = op.compact()
                assert [tuple(m) for m in moves] == omoves and same_state(lp, op)
                to = dict(omoves)
                rows = [(tables[i], [to.get(b, b) for b in orow]) for i, (_, orow) in enumerate(rows)]
                for row, orow in rows:
                    assert list(row[:len(orow)]) == orow and (row[len(orow):] == -1).all()
                live = nb - op.num_free()
                assert all(b < live for _, orow in rows for b in orow)
                if cached:
                    assert lp.pa_pool_cached_blocks() == len(op.prefix_cache)
                assert len(lp.pa_pool_compact()) == 0             # compact already


def test_compaction_refusals(pa):
    lp = pa.Pool(4, 4, [3, 2, 1, 0])
    lp.pa_pool_alloc(1)
    n = ctypes.c_int32()
    assert pa._lib.pa_pool_compact(lp._h, None, 0, 0, None, ctypes.byref(n)) == pa.PA_ERR_INVALID
    assert lp.pa_pool_refcount(3) == 1                            # unchanged
    assert pa._lib.pa_pool_compact(None, None, 0, 0, None, ctypes.byref(n)) == pa.PA_ERR_INVALID
    with pytest.raises(TypeError):
        lp.pa_pool_compact(np.zeros((2, 2), np.int64))
    assert [tuple(m) for m in lp.pa_pool_compact()] == [(3, 0)]
    empty = pa.Pool(0, 4)
    assert len(empty.pa_pool_compact()) == 0


def test_prefill_rejects_bad_arguments_on_host(pa):
    lib = pa._lib
    fake = ctypes.c_void_p(1 << 20)                               # never dereferenced: validation fails first
    base = dict(q=fake, k=fake, v=fake, nb=16, tables=fake, mb=4, lens=fake, starts=fake, t=10, s=2, hq=4, hkv=2,
                d=64, bs=16, scale=0.125, causal=1, ws=fake, wsb=1 << 40, out=fake, dt=pa.PA_BF16)

    def call(**kw):
        a = dict(base, **kw)
        return lib.pa_prefill_attention(a["q"], a["k"], a["v"], a["nb"], a["tables"], a["mb"], a["lens"], a["starts"],
                                        a["t"], a["s"], a["hq"], a["hkv"], a["d"], a["bs"], a["scale"], a["causal"],
                                        a["ws"], a["wsb"], a["out"], a["dt"], None)

    for bad in (dict(hq=3), dict(hq=0), dict(dt=9), dict(nb=0), dict(mb=0), dict(t=-1), dict(s=-1), dict(q=None),
                dict(starts=None), dict(tables=None), dict(out=None), dict(ws=None), dict(wsb=100),
                dict(ws=ctypes.c_void_p((1 << 20) + 16)), dict(q=ctypes.c_void_p((1 << 20) + 8)),
                dict(out=ctypes.c_void_p((1 << 20) + 2)), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(nb=1 << 28), dict(mb=1 << 28), dict(t=1 << 30)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    for bad in (dict(d=96), dict(hq=6), dict(hq=32), dict(bs=24), dict(bs=4)):
        assert call(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    assert call(t=0) == pa.PA_OK and call(s=0) == pa.PA_OK        # nothing to do, nothing launched


def test_prefill_workspace_size(pa):
    size = pa.pa_prefill_workspace_size
    assert size(0, 1, 8, 8, 64, 4, 16) == 0 and size(4, 1, 6, 4, 64, 4, 16) == 0
    # contexts of one step of 128 tokens are never split: the work list only
    assert size(100, 2, 8, 2, 128, 8, 16) < 8192
    # the partials are bounded by the SM count, whatever the context
    a, b = size(16, 1, 64, 8, 128, 1 << 12, 32), size(16, 1, 64, 8, 128, 1 << 16, 32)
    assert a <= b < 200 << 20
    assert size(16, 1, 64, 8, 128, 1 << 20, 32) == b


def test_rope_append_rejects_bad_arguments_on_host(pa):
    lib = pa._lib
    fake = ctypes.c_void_p(1 << 20)
    base = dict(q=fake, qs=512, k=fake, ks=256, v=fake, vs=256, pos=fake, axes=1, freq=fake, axis=None, rot=128,
                inter=0, slots=fake, t=4, out=fake, kc=fake, vc=fake, nb=8, bs=16, hq=4, hkv=2, d=128, dt=pa.PA_BF16)

    def call(**kw):
        a = dict(base, **kw)
        return lib.pa_rope_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["axes"], a["freq"],
                                  a["axis"], a["rot"], a["inter"], a["slots"], a["t"], a["out"], a["kc"], a["vc"],
                                  a["nb"], a["bs"], a["hq"], a["hkv"], a["d"], a["dt"], None)

    for bad in (dict(rot=0), dict(rot=127), dict(rot=130), dict(axes=0), dict(t=-1), dict(hq=0), dict(q=None),
                dict(pos=None), dict(freq=None), dict(slots=None), dict(out=None), dict(qs=500), dict(ks=260),
                dict(vs=128), dict(dt=5), dict(q=ctypes.c_void_p((1 << 20) + 8)),
                dict(kc=ctypes.c_void_p((1 << 20) + 4)), dict(qs=1024, q=fake, out=fake)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    assert call(d=1024, rot=64, qs=1 << 20, ks=1 << 20, vs=1 << 20) == pa.PA_ERR_UNSUPPORTED
    assert call(d=40, rot=40) == pa.PA_ERR_UNSUPPORTED
    assert call(t=0) == pa.PA_OK


def test_move_blocks_rejects_bad_arguments_on_host(pa):
    lib = pa._lib
    fake = ctypes.c_void_p(1 << 20)
    caches = (ctypes.c_void_p * 2)(1 << 20, 1 << 21)
    odd = (ctypes.c_void_p * 2)(1 << 20, (1 << 21) + 8)
    null = (ctypes.c_void_p * 2)(1 << 20, None)

    def call(k=caches, v=caches, n=2, moves=fake, m=3, nb=8, bs=16, hkv=2, d=64, tables=fake, rows=2, cols=4, stride=4,
             dt=pa.PA_F16):
        return lib.pa_move_blocks(k, v, n, moves, m, nb, bs, hkv, d, tables, rows, cols, stride, dt, None)

    for bad in (dict(k=odd), dict(v=null), dict(k=None), dict(moves=None), dict(tables=None), dict(stride=3),
                dict(m=-1), dict(n=-1), dict(rows=-1), dict(dt=4), dict(moves=ctypes.c_void_p((1 << 20) + 4))):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    assert call(bs=1, hkv=1, d=4) == pa.PA_ERR_UNSUPPORTED
    assert call(m=0) == pa.PA_OK


def test_bindings_refuse_cpu_tensors_and_shapes(pa):
    import torch
    x = torch.zeros(4, 2, 64)
    c = torch.zeros(16, 16, 2, 64)
    i32 = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(TypeError):
        pa.pa_prefill_attention(x, c, c, i32, i32[:, 0], torch.zeros(3, dtype=torch.int32), 0.125, x.clone())
    with pytest.raises(ValueError):
        pa.pa_prefill_attention(x, c, c, i32, i32[:, 0], torch.zeros(2, dtype=torch.int32), 0.125, x.clone())
    with pytest.raises(TypeError):
        pa.pa_rope_append(x, x, x, torch.zeros(4, dtype=torch.int32), torch.ones(32), torch.zeros(4).long(), c, c,
                          x.clone())
    with pytest.raises(ValueError):
        pa.pa_rope_append(x, x, x, torch.zeros(3, dtype=torch.int32), torch.ones(32), torch.zeros(4).long(), c, c,
                          x.clone())
    with pytest.raises(ValueError):
        pa.pa_move_blocks([c], [c], i32)
    with pytest.raises(TypeError):
        pa.pa_move_blocks([c], [c.clone()], i32)
