"""GPU parity of pa_prefill_attention against the float64 oracle (needs a B200).

Tolerance, per output element, from the roundings of the kernels.  With
p_j the softmax weights and A = sum_j p_j |V_j| (so |out| <= A):

* the output is rounded to its type: u |out|, u = eps / 2;
* 16-bit caches: each weight is rounded to the type for the product with V (u A);
* float32 sums over the context, numerator and denominator: at most
  2 ctx 2^-23 A (each addition off by one unit at most; the tensor cores'
  may truncate);
* the score of a row is off by at most e = (D + 16) 2^-23 B, where B =
  max_j scale sum_d |q_d K_jd| (a dot product of D terms, its scaling, the
  subtraction of the maximum and the rounding of the exponent's argument,
  each at most one unit of a term that B bounds), and the exponential itself
  by 2^-21; a weight moves by that, and so does the sum: 2 (e + 2^-21) A.
"""

import math

import numpy as np
import pytest
import torch

from gpu_cases import TORCH, AsF64
from oracle import oracle_prefill
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


class Case:
    """A paged cache whose slots behind every context hold NaN, and the chunks' queries."""

    def __init__(self, dtype, q_lens, ctx_lens, hq, hkv, d, bs, seed, q_scale=1.0, extra=0):
        rng = np.random.default_rng(seed)
        self.dtype, self.q_lens, self.ctx_lens, self.d, self.bs = dtype, list(q_lens), list(ctx_lens), d, bs
        need = [-(-c // bs) for c in ctx_lens]
        nb, mb = sum(need) + 3, max(need + [1]) + 1
        order = rng.permutation(nb)
        self.tables = np.full((len(need), mb), -1, np.int32)
        at = 0
        for i, n in enumerate(need):
            self.tables[i, :n] = order[at:at + n]
            at += n
        self.k = torch.full((nb, bs, hkv, d), float("nan"), dtype=TORCH[dtype])
        self.v = torch.full((nb, bs, hkv, d), float("nan"), dtype=TORCH[dtype])
        for i, c in enumerate(ctx_lens):
            x = workloads.randn((2, max(c, 1), hkv, d), dtype, seed + 10 + i)
            for j in range(need[i]):
                n = min(bs, c - j * bs)
                self.k[self.tables[i, j], :n] = x[0, j * bs:j * bs + n]
                self.v[self.tables[i, j], :n] = x[1, j * bs:j * bs + n]
        self.starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        t = int(self.starts[-1]) + extra
        self.q = (workloads.randn((t, hq, d), "f32", seed + 1) * q_scale).to(TORCH[dtype])
        self.hq, self.hkv = hq, hkv

    def device(self):
        self.dk, self.dv, self.dq = self.k.cuda(), self.v.cuda(), self.q.cuda()
        self.dt = torch.from_numpy(self.tables).cuda()
        self.dl = torch.tensor(self.ctx_lens, dtype=torch.int32, device="cuda")
        self.ds = torch.from_numpy(self.starts).cuda()
        return self

    def call(self, pa, scale, causal, out=None, **kw):
        out = torch.full_like(self.dq, 77.0) if out is None else out
        pa.pa_prefill_attention(self.dq, self.dk, self.dv, self.dt, self.dl, self.ds, scale, out, causal=causal, **kw)
        return out

    def expect(self, scale, causal):
        q = self.q.double().numpy()
        args = (self.tables, self.ctx_lens, self.starts)
        k, v = AsF64(self.k), AsF64(self.v)
        ref = oracle_prefill(q, k, v, *args, scale, causal)
        a = oracle_prefill(q, k, AsF64(self.v.abs()), *args, scale, causal)
        b = np.zeros(q.shape[:2] + (1,))
        n_ctx = np.zeros(q.shape[0])
        for s, c in enumerate(self.ctx_lens):
            lo, hi = self.starts[s], self.starts[s + 1]
            if c == 0 or lo == hi:
                continue
            keys = np.concatenate([self.k[x].double().abs().numpy() for x in self.tables[s, :-(-c // self.bs)]])[:c]
            for h in range(self.hq):
                kv = h // (self.hq // self.hkv)
                b[lo:hi, h, 0] = (np.abs(q[lo:hi, h]) @ keys[:, kv].T).max(axis=1) * abs(scale)
            n_ctx[lo:hi] = c
        u = torch.finfo(TORCH[self.dtype]).eps / 2
        tol = 2 * n_ctx[:, None, None] * 2.0 ** -23 * a + 2 * ((self.d + 16) * 2.0 ** -23 * b + 2.0 ** -21) * a
        tol = tol + u * np.abs(ref) + (0 if self.dtype == "f32" else u) * a
        return ref, tol + 1e-30

    def check(self, out, scale, causal, where=""):
        ref, tol = self.expect(scale, causal)
        got = out.double().cpu().numpy()
        lo, hi = self.starts[0], self.starts[-1]
        assert np.isfinite(got[lo:hi]).all(), where
        over = np.abs(got - ref)[lo:hi] / tol[lo:hi]
        assert over.max(initial=0.0) <= 1.0, "%s: %.3g of the tolerance at %s" % (
            where, over.max(), np.unravel_index(over.argmax(), over.shape))
        assert (got[hi:] == 77.0).all() and (got[:lo] == 77.0).all()     # rows of no sequence stay as they were


Q_LENS = [1, 0, 5, 17, 64, 130, 33, 2]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("bs", [8, 16, 48, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_matches_oracle(pa, dtype, d, hq, hkv, bs, causal):
    cached = [0, 40, 300, 127, 128, 129, 0, 511]
    ctx = [n + c if causal else c + 1 for n, c in zip(Q_LENS, cached)]
    case = Case(dtype, Q_LENS, ctx, hq, hkv, d, bs, seed=hq * 3 + hkv + d + bs, extra=3).device()
    out = case.call(pa, 1 / math.sqrt(d), causal)
    assert pa.pa_device_error() == 0
    case.check(out, 1 / math.sqrt(d), causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(pa, dtype, causal):
    """Contexts of zero tokens, and chunks longer than their context."""
    q_lens, ctx = [3, 70, 300, 1, 200, 4], [0, 20, 130, 0, 1, 2]
    case = Case(dtype, q_lens, ctx, 4, 1, 128, 16, seed=3).device()
    out = case.call(pa, 0.09, causal)
    case.check(out, 0.09, causal)
    assert (out[0:3] == 0).all() and (out[373] == 0).all()
    if causal:
        assert (out[3:53] == 0).all() and (out[73:243] == 0).all()
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("dtype,q_lens,ctx,hq,hkv,d,bs,causal", [
    ("bf16", [16], [9001], 16, 2, 128, 32, True),                 # few rows, long context: split
    ("f16", [1, 3, 2], [5000, 17, 2500], 8, 8, 64, 16, True),
    ("bf16", [300], [4097], 4, 4, 128, 16, False),
    ("f32", [9], [3001], 8, 2, 64, 16, True),
    ("f16", [1200], [1200], 2, 1, 128, 64, True),
    ("bf16", [700, 1, 1, 1], [1900, 700, 1400, 3], 8, 1, 64, 16, True),
])
def test_long_and_split_contexts(pa, dtype, q_lens, ctx, hq, hkv, d, bs, causal):
    case = Case(dtype, q_lens, ctx, hq, hkv, d, bs, seed=41).device()
    case.check(case.call(pa, 1 / math.sqrt(d), causal), 1 / math.sqrt(d), causal)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale,q_scale", [(-0.125, 1.0), (0.0, 1.0), (0.125, 30.0), (1e-30, 1.0)])
def test_scales(pa, dtype, scale, q_scale):
    case = Case(dtype, [40, 3], [170, 260], 4, 2, 64, 16, seed=8, q_scale=q_scale).device()
    case.check(case.call(pa, scale, True), scale, True)


def test_many_sequences(pa):
    """More sequences than the planner has threads."""
    rng = np.random.default_rng(4)
    q_lens = [int(x) for x in rng.integers(0, 4, 1500)]
    ctx = [n + int(x) for n, x in zip(q_lens, rng.integers(0, 40, 1500))]
    case = Case("bf16", q_lens, ctx, 2, 1, 64, 16, seed=5).device()
    case.check(case.call(pa, 0.125, True), 0.125, True)


def test_more_tiles_than_planner_threads(pa):
    case = Case("f16", [100] * 400, [100 + 7 * (i % 5) for i in range(400)], 8, 1, 64, 16, seed=15).device()
    case.check(case.call(pa, 0.125, True), 0.125, True)


def test_calls_on_two_streams_at_once(pa):
    """Each with its own workspace, in flight together, over and over."""
    cases = [Case("bf16", [300, 7], [900, 3000], 8, 2, 128, 16, seed=16).device(),
             Case("f16", [40, 1, 1], [2500, 800, 64], 4, 4, 64, 16, seed=17).device()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [pa.prefill_workspace(c.dq.shape[0], len(c.q_lens), c.hq, c.hkv, c.d, c.tables.shape[1], c.bs) for c in cases]
    outs = [torch.full_like(c.dq, 77.0) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, o, w, st in zip(cases, outs, ws, streams):
            c.call(pa, 0.1, True, out=o, workspace=w, stream=st)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(o, 0.1, True)
    assert pa.pa_device_error() == 0


def test_infinite_keys_in_masked_places(pa):
    """Later tokens' keys may be anything; their weight is zero."""
    case = Case("bf16", [64], [200], 4, 1, 128, 16, seed=6)
    last = case.tables[0, 199 // 16]
    ref, tol = case.expect(0.09, True)                             # (the bound of a key that is not finite is not)
    for value in (float("inf"), float("nan"), float("-inf"), 3e38):
        case.k[last, 199 % 16] = value
        case.device()
        out = case.call(pa, 0.09, True)
        got = out.double().cpu().numpy()
        assert (np.abs(got - ref) <= tol)[:63].all()


def test_repeats_give_the_same_bits(pa):
    case = Case("bf16", [16, 200], [4000, 900], 8, 2, 128, 16, seed=9).device()
    first = case.call(pa, 0.09, True)
    for _ in range(5):
        assert torch.equal(case.call(pa, 0.09, True), first)


def test_one_token_chunks_agree_with_decode(pa):
    ctx = [1, 16, 100, 2000]
    case = Case("bf16", [1] * 4, ctx, 8, 2, 128, 16, seed=10).device()
    out = case.call(pa, 0.09, True)
    ref = torch.empty_like(out)
    pa.pa_decode_attention(case.dq, case.dk, case.dv, case.dt.clamp(min=0), case.dl, 0.09, ref, 0,
                           pa.decode_workspace(4, 8, 128, case.tables.shape[1], 16, 0))
    # both are within one bound of the same value
    _, tol = case.expect(0.09, True)
    assert (np.abs((out.double() - ref.double()).cpu().numpy()) <= 2 * tol).all()


def test_queries_and_outputs_that_are_only_16_byte_aligned(pa):
    case = Case("f16", [50], [90], 2, 2, 64, 16, seed=11).device()
    buf = torch.full((case.dq.numel() + 8,), 5.0, dtype=torch.float16, device="cuda")
    out = buf[8:].view_as(case.dq)
    case.check(case.call(pa, 0.125, True, out=out), 0.125, True)
    assert (buf[:8] == 5.0).all()


def test_shared_workspace_back_to_back_and_streams(pa):
    """Calls queued without a wait between them on one workspace; and on another stream than the tensors' own."""
    cases = [Case("bf16", q, c, 8, 2, 128, 16, seed=20 + i).device()
             for i, (q, c) in enumerate([([16], [5000]), ([300, 20], [300, 2000]), ([1, 1, 1], [900, 30, 1]),
                                         ([64], [64])])]
    ws = torch.empty(max(pa.pa_prefill_workspace_size(c.dq.shape[0], len(c.q_lens), 8, 2, 128, c.tables.shape[1], 16)
                         for c in cases), dtype=torch.uint8, device="cuda")
    outs = [c.call(pa, 0.09, True, workspace=ws) for c in cases]
    for c, o in zip(cases, outs):
        c.check(o, 0.09, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.full_like(c.dq, 77.0) for c in cases]
    side.wait_stream(torch.cuda.current_stream())
    for c, o in zip(cases, outs):
        c.call(pa, 0.09, True, out=o, stream=side)
    side.synchronize()
    for c, o in zip(cases, outs):
        c.check(o, 0.09, True)
    assert pa.pa_device_error() == 0


def test_captured_and_replayed_with_other_lengths(pa):
    """The plan is made on the device: a graph follows the lengths, starts and tables it finds."""
    a = Case("bf16", [40, 24], [2000, 100], 8, 2, 128, 16, seed=30).device()
    b = Case("bf16", [9, 55], [700, 2050], 8, 2, 128, 16, seed=31).device()
    nb, mb = max(a.dk.shape[0], b.dk.shape[0]), max(a.tables.shape[1], b.tables.shape[1])
    k = torch.zeros((nb, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    v, q = torch.zeros_like(k), torch.zeros((64, 8, 128), dtype=torch.bfloat16, device="cuda")
    tables = torch.zeros((2, mb), dtype=torch.int32, device="cuda")
    lens, starts = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = pa.prefill_workspace(64, 2, 8, 2, 128, mb, 16)

    def load(c):
        k[:c.dk.shape[0]] = c.dk
        v[:c.dv.shape[0]] = c.dv
        tables[:, :c.tables.shape[1]] = c.dt
        q.copy_(c.dq)
        lens.copy_(c.dl)
        starts.copy_(c.ds)
        out.fill_(77.0)

    load(a)
    pa.pa_prefill_attention(q, k, v, tables, lens, starts, 0.09, out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_prefill_attention(q, k, v, tables, lens, starts, 0.09, out, workspace=ws)
    for c in (b, a, b):
        load(c)
        g.replay()
        torch.cuda.synchronize()
        c.check(out, 0.09, True)


def test_bad_tables_and_lengths_set_the_device_error(pa):
    case = Case("bf16", [20], [60], 4, 2, 64, 16, seed=12).device()
    for dtype in ("bf16", "f32"):
        c = Case(dtype, [20], [60], 4, 2, 64, 16, seed=12).device()
        c.dt[0, 1] = 10 ** 6
        c.call(pa, 0.125, True)
        assert pa.pa_device_error() == 1
        c = Case(dtype, [20], [60], 4, 2, 64, 16, seed=12).device()
        c.dl[0] = 10 ** 6                                          # beyond the table: clamped
        c.dt.clamp_(min=0)
        c.call(pa, 0.125, True)
        assert pa.pa_device_error() == 2
    for starts in ([0, 21], [-1, 20], [5, 3]):                     # 21 rows of 20 tokens, and so on
        case.ds.copy_(torch.tensor(starts, dtype=torch.int32))
        out = torch.full_like(case.dq, 77.0)
        case.call(pa, 0.125, True, out=out)
        assert pa.pa_device_error() == 2
        if starts == [5, 3]:
            assert (out == 77.0).all()
    # overlapping chunks would overfill the work list: they are cut off
    two = Case("bf16", [600, 600, 600], [600] * 3, 8, 1, 64, 16, seed=13).device()
    two.ds.copy_(torch.tensor([0, 1800, 0, 1800], dtype=torch.int32))
    two.call(pa, 0.125, False)
    assert pa.pa_device_error() == 2
    two.ds.copy_(torch.from_numpy(two.starts))
    two.check(two.call(pa, 0.125, True), 0.125, True)
    assert pa.pa_device_error() == 0
