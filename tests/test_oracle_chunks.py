"""Pins of the oracle's chunk functions (CPU only)."""

import numpy as np
import torch

from oracle import oracle_decode, oracle_prefill, oracle_rope


def _cache(rng, nb, bs, hkv, d):
    return rng.standard_normal((nb, bs, hkv, d)), rng.standard_normal((nb, bs, hkv, d))


def test_causal_chunk_matches_library_attention():
    rng = np.random.default_rng(1)
    k, v = _cache(rng, 9, 4, 2, 16)
    table, ctx, n = [5, 1, 7, 0, 3], 18, 6
    q = rng.standard_normal((n, 4, 16))
    got = oracle_prefill(q, k, v, [table], [ctx], [0, n], 0.25)
    keys = torch.from_numpy(k[table].reshape(-1, 2, 16)[:ctx]).permute(1, 0, 2)[None]
    values = torch.from_numpy(v[table].reshape(-1, 2, 16)[:ctx]).permute(1, 0, 2)[None]
    mask = torch.ones(n, ctx).tril(ctx - n).bool()
    for causal, m in ((True, mask), (False, None)):
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.from_numpy(q).permute(1, 0, 2)[None], keys, values, attn_mask=m, scale=0.25, enable_gqa=True)
        got = oracle_prefill(q, k, v, [table], [ctx], [0, n], 0.25, causal)
        assert np.allclose(got, want[0].permute(1, 0, 2).numpy(), atol=1e-12)


def test_chunk_of_one_token_is_decode_and_empty_rows_are_zero():
    rng = np.random.default_rng(2)
    k, v = _cache(rng, 6, 4, 2, 8)
    tables, lens = [[0, 3], [2, 5], [1, 4]], [7, 1, 0]
    q = rng.standard_normal((3, 2, 8))
    a = oracle_prefill(q, k, v, tables, lens, [0, 1, 2, 3], 0.3)
    assert np.allclose(a, oracle_decode(q, k, v, tables, lens, 0.3), atol=1e-14)
    b = oracle_prefill(q, k, v, [tables[0]], [2], [0, 3], 0.3)     # a chunk longer than its context
    assert (b[0] == 0).all() and (b[1] != 0).any()
    c = oracle_prefill(q, k, v, [tables[0]], [5], [1, 2], 0.3)     # rows of no sequence
    assert (c[0] == 0).all() and (c[2] == 0).all() and (c[1] != 0).any()


def test_rope_turns_pairs_by_their_angle():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 2, 12))
    pos = np.array([[0, 1, 2, 50000, 7], [3, 3, 3, 3, 3]])
    freq, axis = np.array([1.0, 0.5, 0.01], np.float32), [0, 1, 0]
    for inter in (False, True):
        y = oracle_rope(x, pos, freq, axis, inter)
        assert np.array_equal(y[..., 6:], x[..., 6:])
        a, b = (np.s_[0:6:2], np.s_[1:6:2]) if inter else (np.s_[0:3], np.s_[3:6])
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * np.stack([pos[axis[i]] * float(freq[i]) for i in range(3)],
                                                                1))[:, None, :]
        assert np.allclose(y[..., a], z.real, atol=1e-12) and np.allclose(y[..., b], z.imag, atol=1e-12)
    # the score of a turned query and key depends on the difference of their positions alone
    u = oracle_rope(x[:1], [[10]], freq) * oracle_rope(x[1:2], [[4]], freq)
    w = oracle_rope(x[:1], [[106]], freq) * oracle_rope(x[1:2], [[100]], freq)
    assert np.allclose(u[..., :6].sum(-1), w[..., :6].sum(-1), atol=1e-12)
