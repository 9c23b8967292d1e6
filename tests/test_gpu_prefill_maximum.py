"""Chunk attention where the running maximum moves late, and where visible
scores are not finite (needs a B200).

A row's reference maximum moves only when a score passes it by 2^8.  Keys whose
scores grow along the context make it move again and again in steps without a
masked token, after the step's first weights were worked out with the maximum
that stood before.

Tolerance: that of test_gpu_prefill (moving the maximum multiplies sum and
output by one factor, rounded once each: fewer roundings than the 2 ctx 2^-23
counted there for the additions), and for f16 the weights below 2^-14, which are
rounded to multiples of 2^-24: ctx 2^-25 max |V|, the sum of weights being at
least 1 (the token that set the maximum has weight 1).
"""

import math

import numpy as np
import pytest
import torch

from gpu_cases import TORCH, AsF64
from oracle import oracle_prefill
from test_gpu_prefill import Case

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


STEP = 128
RISES = [0, 0, 9, 0, 20, 0, 0, 0, 11]           # of each step's scores over the step before, units of log2


def growing(dtype, q_lens, ctx_lens, hq, hkv, d, seed, sign):
    """A case whose keys have a growing part along one direction; two of three query tokens have it too."""
    case = Case(dtype, q_lens, ctx_lens, hq, hkv, d, 16, seed)
    rng = np.random.default_rng(seed)
    u = torch.from_numpy(rng.choice([-1.0, 1.0], d)).float()
    longest = max(ctx_lens)
    rise = np.cumsum([RISES[i % len(RISES)] for i in range(longest // STEP + 1)])
    # score of query 2 u and key a u, over sqrt(d): 2 a sqrt(d) = rise ln 2
    a = torch.from_numpy(rise[np.arange(longest) // STEP] * math.log(2) / (2 * math.sqrt(d))).float()
    for s, c in enumerate(ctx_lens):
        for j in range(-(-c // 16)):
            n = min(16, c - j * 16)
            b = case.tables[s, j]
            x = case.k[b, :n].float() + a[j * 16:j * 16 + n, None, None] * u
            case.k[b, :n] = x.to(TORCH[dtype])
    q = case.q.float()
    q = q - (q @ u / d)[..., None] * u
    some = torch.arange(q.shape[0]) % 3 != 1
    q[some] += 2.0 * sign * u
    case.q = q.to(TORCH[dtype])
    return case


def moves_late(case, scale, causal):
    """Number of (row, step) pairs, steps 2 and on without a masked token, whose scores pass the ones before by 2^8."""
    count = 0
    for s, c in enumerate(case.ctx_lens):
        lo, hi = case.starts[s], case.starts[s + 1]
        if lo == hi:
            continue
        keys = np.concatenate([case.k[b].double().numpy() for b in case.tables[s, :-(-c // 16)]])[:c]
        first = c - (hi - lo) + 1 if causal else c
        full = min(first, c) // STEP
        if full < 4:
            continue
        x = np.einsum("td,jd->tj", case.q[lo:hi, 0].double().numpy(), keys[:full * STEP, 0]) * scale / math.log(2)
        top = x.reshape(hi - lo, full, STEP).max(axis=2)
        before = np.maximum.accumulate(top, axis=1)
        count += int((top[:, 2:] > before[:, 1:-1] + 8).sum())
    return count


SHAPES = {
    "tiles of 256 rows": ([300, 70], [1500, 1300], 8, 2),
    "rows dealt by steps": ([1, 2, 3] * 14, [1100 + 37 * i for i in range(42)], 8, 4),
    "split": ([16], [9000], 16, 2),
    "split, one head per group": ([40], [5000], 2, 2),
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_scores_that_grow_along_the_context(pa, dtype, d, sign, causal, shape):
    q_lens, ctx, hq, hkv = SHAPES[shape]
    scale = sign / math.sqrt(d)
    case = growing(dtype, q_lens, ctx, hq, hkv, d, 5 + d, sign)
    assert moves_late(case, scale, causal) > 3 * sum(q_lens) // 2     # two of three tokens, several steps each
    case.device()
    out = case.call(pa, scale, causal).double().cpu().numpy()
    ref, tol = case.expect(scale, causal)
    if dtype == "f16":
        tol = tol + max(ctx) * 2.0 ** -25 * float(np.nanmax(case.v.double().abs().numpy()))
    assert np.isfinite(out).all()
    over = np.abs(out - ref) / tol
    assert over.max() <= 1.0, "%.3g of the tolerance at %s" % (over.max(), np.unravel_index(over.argmax(), over.shape))
    assert pa.pa_device_error() == 0


def _slot(case, s, j):
    return int(case.tables[s, j // case.bs]), j % case.bs


def reference(case, v, scale):
    with np.errstate(invalid="ignore"):
        return oracle_prefill(case.q.double().numpy(), AsF64(case.k), AsF64(v), case.tables, case.ctx_lens, case.starts,
                              scale, True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("q_lens,ctx,at", [([200, 3], [600, 90], 130), ([2, 3], [1700, 90], 1300), ([4], [6000], 17)])
def test_visible_keys_and_values_that_are_not_finite(pa, dtype, q_lens, ctx, at):
    """A row that sees a NaN score, or an infinite one, is NaN; a score of -inf has weight zero; a value that is not
    finite spoils its own element.  Other heads and sequences keep their bits."""
    hq, hkv, d, scale = 8, 2, 128, 0.09
    clean = Case(dtype, q_lens, ctx, hq, hkv, d, 16, seed=31).device()
    good = clean.call(pa, scale, True)
    n = q_lens[0]
    extra = ctx[0] * 2.0 ** -25 * float(np.nanmax(clean.v.double().abs().numpy()))
    for place, value in (("k", float("nan")), ("k", float("inf")), ("k", float("-inf")), ("v", float("nan")),
                         ("v", float("inf"))):
        case = Case(dtype, q_lens, ctx, hq, hkv, d, 16, seed=31)
        b, r = _slot(case, 0, at)
        (case.k if place == "k" else case.v)[b, r, 1, 5] = value
        case.device()
        out = case.call(pa, scale, True)
        assert torch.equal(out[n:], good[n:]) and torch.equal(out[:, :4], good[:, :4])
        mine = out[:n, 4:].double().cpu().numpy()
        if place == "v":
            bad = mine[..., 5]
            assert np.isnan(bad).all() if math.isnan(value) else (np.isposinf(bad) | np.isnan(bad)).all()
            keep = np.arange(d) != 5
            assert np.array_equal(mine[..., keep], good[:n, 4:].double().cpu().numpy()[..., keep])
            continue
        score = case.q[:n, 4:, 5].double().numpy() * value
        spoilt = ~(score == -np.inf)
        assert np.isnan(mine[spoilt]).all() and (math.isnan(value) or (~spoilt).any())
        # rows in which the score is -inf are those of a context without that token.  The bound is A times a factor
        # that is no less than u, plus u |out|, |out| <= A: with A' in the place of A at most 2 max(1, A' / A) as much
        ref = reference(case, case.v, scale)[:n, 4:]
        a, a2 = (reference(c, c.v.abs(), scale)[:n, 4:] for c in (clean, case))
        _, tol = clean.expect(scale, True)
        tol = 2 * tol[:n, 4:] * np.maximum(1, a2 / a) + extra * (dtype == "f16")
        ok = np.abs(mine - ref) <= tol
        assert ok[~spoilt].all()
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_whose_every_visible_score_is_minus_infinity_are_zero(pa, dtype):
    case = Case(dtype, [1, 40], [1, 200], 2, 2, 64, 16, seed=33)
    b, r = _slot(case, 0, 0)
    case.k[b, r, :, 3] = float("inf")
    case.q[0, :, 3] = -1.0
    case.device()
    out = case.call(pa, 0.125, True)
    assert (out[0] == 0).all() and torch.isfinite(out).all()
    assert pa.pa_device_error() == 0
