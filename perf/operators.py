"""Cases, plain forms and work counts of the chunk (prompt) operators.

Four operators that bring a run of new tokens into a paged KV cache and attend
over it:

prefill   attention of a chunk of new tokens per sequence over the paged cache
          (causal: token i of a chunk of n sees the first ctx - n + i + 1
          tokens of its sequence's context)
cross     the same call without the causal mask: decoder tokens over an
          encoder's states of another length, kept in a paged cache
rope      rotary positions with one or several axes (time, height, width)
          for queries and keys, and the write of keys and values into their slots
compact   live blocks moved to the front of the pool in every layer's cache,
          with the block tables rewritten

Formulas (kv = h // (Hq / Hkv); a slot x is row x % bs of block x // bs):

prefill, cross   out[t][h] = sum_j softmax_j(scale q[t][h].K[j][kv]) V[j][kv]
                 over the tokens j the mask leaves; a zero row if it leaves none
rope             angle[t][i] = positions[axis[i]][t] * inv_freq[i]; element i
                 and its partner (i + R/2, or 2i and 2i + 1 when interleaved)
                 are turned by that angle; elements from R on stay
compact          block dst of every cache := block src; table entries src -> dst

``run`` computes the plain forms in 32 bits with elementary torch operations
(angles in 64 bits), or calls the library when ``own`` is set.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(str(int(v)) for v in values)


def _attention(name, kind, q_lens, ctx_lens, hq, hkv, d, bs, dtype):
    case = {"kind": kind, "q_lens": _text(q_lens), "ctx_lens": _text(ctx_lens), "hq": hq, "hkv": hkv, "d": d,
            "bs": bs, "dtype": dtype}
    return dict(case, name=name) if name else case


def _rope(name, tokens, hq, hkv, d, rotary, axes, interleaved, bs, far, dtype):
    case = {"kind": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rotary": rotary, "axes": axes,
            "interleaved": interleaved, "bs": bs, "far": far, "dtype": dtype}
    return dict(case, name=name) if name else case


def _compact(name, layers, blocks, moves, rows, cols, hkv, d, bs, dtype):
    case = {"kind": "compact", "layers": layers, "blocks": blocks, "moves": moves, "rows": rows, "cols": cols,
            "hkv": hkv, "d": d, "bs": bs, "dtype": dtype}
    return dict(case, name=name) if name else case


def listed():
    return [
        # a chunk of a long prompt whose first half is cached (32/8 heads, block 16)
        _attention("prefill_chunk_8k_of_16k", "prefill", [8192], [16384], 32, 8, 128, 16, "bf16"),
        # whole prompts of mixed lengths arriving together, nothing cached
        _attention("prefill_ragged_prompts", "prefill", [4001, 1023, 517, 2048, 130, 77, 1500, 16],
                   [4001, 1023, 517, 2048, 130, 77, 1500, 16], 32, 32, 128, 16, "f16"),
        # a scheduler's mixed step: one prompt chunk beside decoding sequences (one token each)
        _attention("prefill_mixed_step", "prefill", [512] + [1] * 48,
                   [2560] + [300 + 97 * i for i in range(48)], 32, 8, 128, 16, "bf16"),
        # a few speculated tokens on one long context (64/8 heads, block 32): few rows, long axis
        _attention("prefill_16_on_32k", "prefill", [16], [32701], 64, 8, 128, 32, "bf16"),
        # the toy-sized float32 cache (2/2 heads, head_dim 64)
        _attention("prefill_tiny_f32", "prefill", [1, 16, 17, 45], [1, 16, 40, 300], 2, 2, 64, 16, "f32"),
        # decoder prompts over an encoder's 1,500 states
        _attention("cross_prompts_1500", "cross", [224] * 16, [1500] * 16, 16, 16, 64, 16, "f16"),
        # a few decoder tokens per sequence over encoder states of odd lengths
        _attention("cross_few_tokens", "cross", [4, 1, 3, 4, 2, 4, 4, 1], [1500, 700, 33, 1499, 1, 910, 1024, 250],
                   32, 8, 128, 16, "bf16"),
        # a multimodal prompt: three axes, 32/8 heads
        _rope("rope_three_axes_16k", 16384, 32, 8, 128, 128, 3, False, 16, 32768, "bf16"),
        # one decode step of 64 sequences, far positions, one axis
        _rope("rope_decode_64", 64, 32, 32, 128, 128, 1, False, 16, 1000000, "f16"),
        # all layers of a cache: the live blocks of a quarter of the pool move
        _compact("compact_32_layers", 32, 512, 128, 64, 64, 8, 128, 16, "bf16"),
        # one layer of a float32 cache, a handful of blocks
        _compact("compact_one_layer_f32", 1, 64, 9, 8, 16, 2, 64, 16, "f32"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "cross", "rope", "compact"])
    dtype = rng.choice(["bf16", "f16", "bf16", "f16", "f32"])
    d = rng.choice([64, 128])
    group = rng.choice([1, 2, 4, 8])
    hkv = rng.choice([1, 2, 4, 8])
    bs = rng.choice([8, 16, 32, 48, 64])
    if kind in ("prefill", "cross"):
        tokens = _log_int(rng, 1, 512 if dtype == "f32" else 8192)
        seqs = _log_int(rng, 1, 64)
        most = min(32768, 131072 // seqs) // (8 if dtype == "f32" else 1)
        q_lens = [_log_int(rng, 1, max(2, 2 * tokens // seqs)) for _ in range(seqs)]
        ctx_lens = [_log_int(rng, 1, most) for _ in range(seqs)]
        if kind == "prefill":                                    # the context ends with the chunk itself
            ctx_lens = [n + rng.choice([0, c]) for n, c in zip(q_lens, ctx_lens)]
        elif seqs > 1:                                           # some without tokens, some without states
            q_lens = [q_lens[0]] + [rng.choice([n, n, n, 0]) for n in q_lens[1:]]
            ctx_lens = [ctx_lens[0]] + [rng.choice([c, c, c, 0]) for c in ctx_lens[1:]]
        while 4 * sum(n * c for n, c in zip(q_lens, ctx_lens)) * hkv * group * d > 1.6e12:
            q_lens = [(n + 1) // 2 for n in q_lens]
        return _attention(None, kind, q_lens, ctx_lens, hkv * group, hkv, d, bs, dtype)
    if kind == "rope":
        rotary = rng.choice([d, d, d // 2, 2 * rng.randint(3, d // 2)])
        return _rope(None, _log_int(rng, 1, 16000), hkv * group, hkv, d, rotary, rng.choice([1, 2, 3, 4]),
                     rng.random() < 0.3, bs, _log_int(rng, 1000, 2000000), dtype)
    blocks = _log_int(rng, 8, 500)
    return _compact(None, _log_int(rng, 1, 32), blocks, rng.randint(1, max(1, blocks // 3)), rng.randint(1, 64),
                    rng.randint(1, 64), hkv, d, rng.choice([8, 16]), dtype)


def _pairs_of(case):
    """Number of (query token, context token) pairs the mask leaves."""
    total = 0
    for n, ctx in zip(_ints(case["q_lens"]), _ints(case["ctx_lens"])):
        if case["kind"] == "cross":
            total += n * ctx
        else:
            first = ctx - n + 1                       # tokens the first row sees (may be <= 0)
            skip = min(n, max(0, 1 - first))
            rows = n - skip
            total += rows * (first + skip) + rows * (rows - 1) // 2 if rows > 0 else 0
    return total


def work(case):
    e = _BYTES[case["dtype"]]
    if case["kind"] in ("prefill", "cross"):
        q_lens, ctx_lens = _ints(case["q_lens"]), _ints(case["ctx_lens"])
        rows = 2 * sum(q_lens) * case["hq"] * case["d"] * e
        seen = sum(c for n, c in zip(q_lens, ctx_lens) if n > 0)
        return {"bytes": rows + 2 * seen * case["hkv"] * case["d"] * e,
                "flops": 4 * _pairs_of(case) * case["hq"] * case["d"]}
    if case["kind"] == "rope":
        t, d = case["tokens"], case["d"]
        moved = 2 * t * (case["hq"] + 2 * case["hkv"]) * d * e
        return {"bytes": moved + t * (4 * case["axes"] + 8),
                "flops": 3 * t * (case["hq"] + case["hkv"]) * case["rotary"]}
    block = case["bs"] * case["hkv"] * case["d"] * e
    return {"bytes": 4 * case["layers"] * case["moves"] * block + 8 * case["rows"] * case["cols"] + 8 * case["moves"],
            "flops": 0}


def _randn(gen, shape, dtype, times=1.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * times).to(DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    st = {"case": case}
    if case["kind"] in ("prefill", "cross"):
        q_lens, ctx_lens = _ints(case["q_lens"]), _ints(case["ctx_lens"])
        bs, hq, hkv, d, dt = case["bs"], case["hq"], case["hkv"], case["d"], case["dtype"]
        s = len(q_lens)
        need = [-(-c // bs) for c in ctx_lens]
        nb, mb = sum(need) + 2, max(need) + 1
        order = rng.permutation(nb)
        tables = np.zeros((s, mb), np.int32)
        at = 0
        for i, n in enumerate(need):
            tables[i, :n] = order[at:at + n]
            at += n
        st["q"] = _randn(gen, (sum(q_lens), hq, d), dt, 2.0)     # scores spread by about 2, as in trained layers
        st["k_cache"] = _randn(gen, (nb, bs, hkv, d), dt)
        st["v_cache"] = _randn(gen, (nb, bs, hkv, d), dt)
        for c in ("k_cache", "v_cache"):                         # slots no token was written to hold anything
            flat = st[c].view(nb * bs, hkv, d)
            for b in order[at:]:
                flat[int(b) * bs:(int(b) + 1) * bs] = float("nan")
            for i, n in enumerate(ctx_lens):
                if n % bs:
                    base = int(tables[i, n // bs]) * bs
                    flat[base + n % bs:base + bs] = float("nan")
        st["tables"] = torch.from_numpy(tables).cuda()
        st["ctx"] = torch.tensor(ctx_lens, dtype=torch.int32, device="cuda")
        st["q_starts"] = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32, device="cuda")
        st["out"] = torch.empty_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(d)
        st["lists"] = (q_lens, ctx_lens)
        if own:
            from paged_kv_cache_341_b200 import pa
            st["pa"] = pa
            st["workspace"] = pa.prefill_workspace(st["q"].shape[0], s, hq, hkv, d, mb, bs)
        return st
    if case["kind"] == "rope":
        t, bs, hq, hkv, d, dt = case["tokens"], case["bs"], case["hq"], case["hkv"], case["d"], case["dtype"]
        nb = -(-t // bs) + 3
        half = case["rotary"] // 2
        st["q"] = _randn(gen, (t, hq, d), dt)
        st["k"] = _randn(gen, (t, hkv, d), dt)
        st["v"] = _randn(gen, (t, hkv, d), dt)
        st["positions"] = torch.from_numpy(rng.integers(0, case["far"], (case["axes"], t)).astype(np.int32)).cuda()
        st["inv_freq"] = torch.from_numpy((1e4 ** (-np.arange(half) / half)).astype(np.float32)).cuda()
        # runs of pairs per axis, as in the models with a (time, height, width) position
        st["axis"] = torch.from_numpy((np.arange(half) * case["axes"] // half).astype(np.int32)).cuda()
        blocks = rng.permutation(nb)[:-(-t // bs)]
        i = np.arange(t)
        st["slots"] = torch.from_numpy(blocks[i // bs].astype(np.int64) * bs + i % bs).cuda()
        st["k_cache"] = _randn(gen, (nb, bs, hkv, d), dt)
        st["v_cache"] = _randn(gen, (nb, bs, hkv, d), dt)
        st["q_out"] = torch.empty_like(st["q"])
    else:
        nb, bs, hkv, d, dt = case["blocks"], case["bs"], case["hkv"], case["d"], case["dtype"]
        shape = (nb, bs, hkv, d)
        st["caches"] = torch.stack([torch.stack([_randn(gen, shape, dt) for _ in range(case["layers"])])
                                    for _ in range(2)])          # K and V of all layers, one allocation
        st["k_caches"], st["v_caches"] = list(st["caches"][0]), list(st["caches"][1])
        # `moves` live blocks behind the front of the pool go to as many free ones in the front
        live = nb - max(case["moves"], nb // 4)
        moves = min(case["moves"], live)
        dst = np.sort(rng.permutation(live)[:moves])
        src = np.sort(live + rng.permutation(nb - live)[:moves])
        st["moves"] = torch.from_numpy(np.stack([src, dst], 1).astype(np.int32)).cuda()
        used = np.concatenate([np.setdiff1d(np.arange(live), dst), src])
        st["tables"] = torch.from_numpy(
            used[rng.integers(0, len(used), (case["rows"], case["cols"]))].astype(np.int32)).cuda()
    if own:
        from paged_kv_cache_341_b200 import pa
        st["pa"] = pa
    return st


def _plain_attention(st):
    case = st["case"]
    q_lens, ctx_lens = st["lists"]
    hq, hkv, d, bs = case["hq"], case["hkv"], case["d"], case["bs"]
    g = hq // hkv
    out = torch.zeros_like(st["q"])
    at = 0
    for i, (n, ctx) in enumerate(zip(q_lens, ctx_lens)):
        if n == 0:
            continue
        if ctx > 0:
            ids = st["tables"][i, :-(-ctx // bs)].long()
            k = st["k_cache"][ids].reshape(-1, hkv, d)[:ctx].permute(1, 2, 0).float()          # [Hkv, D, ctx]
            v = st["v_cache"][ids].reshape(-1, hkv, d)[:ctx].permute(1, 0, 2).float()          # [Hkv, ctx, D]
            step = max(1, min(n, (1 << 28) // (hq * ctx)))
            for t0 in range(0, n, step):
                m = min(step, n - t0)
                q = st["q"][at + t0:at + t0 + m].float().view(m, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, m * g, d)
                s = torch.matmul(q, k) * st["scale"]
                if case["kind"] == "prefill":
                    row = torch.arange(t0, t0 + m, device="cuda").repeat_interleave(g)[None, :, None]
                    s = s.masked_fill(torch.arange(ctx, device="cuda")[None, None, :] > ctx - n + row, -math.inf)
                top = s.max(dim=2, keepdim=True).values
                p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
                total = p.sum(dim=2, keepdim=True)
                o = torch.matmul(p, v) / torch.where(total == 0, torch.ones_like(total), total)
                out[at + t0:at + t0 + m] = o.view(hkv, m, g, d).permute(1, 0, 2, 3).reshape(m, hq, d).to(out.dtype)
        at += n
    return out


def _turn(x, cos, sin, rotary, interleaved):
    half = rotary // 2
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
        y[..., 0:rotary:2], y[..., 1:rotary:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:rotary]
        y[..., :half], y[..., half:rotary] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(st):
    case = st["case"]
    angle = st["positions"].double()[st["axis"].long()].t() * st["inv_freq"].double()      # [T, R/2]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    dt = st["q"].dtype
    st["q_out"].copy_(_turn(st["q"].float(), cos, sin, case["rotary"], case["interleaved"]).to(dt))
    rows = (-1, case["hkv"], case["d"])
    st["k_cache"].view(rows)[st["slots"]] = _turn(st["k"].float(), cos, sin, case["rotary"], case["interleaved"]).to(dt)
    st["v_cache"].view(rows)[st["slots"]] = st["v"]
    return st["q_out"], st["k_cache"], st["v_cache"]


def _plain_compact(st):
    src, dst = st["moves"][:, 0].long(), st["moves"][:, 1].long()
    for c in st["k_caches"] + st["v_caches"]:
        c[dst] = c[src]
    to = torch.arange(st["case"]["blocks"], dtype=torch.int32, device="cuda")
    to[src] = st["moves"][:, 1]
    st["tables"].copy_(to[st["tables"].long()])
    return st["caches"], st["tables"]


def run(state):
    kind = state["case"]["kind"]
    if own:
        pa = state["pa"]
        if kind in ("prefill", "cross"):
            pa.pa_prefill_attention(state["q"], state["k_cache"], state["v_cache"], state["tables"], state["ctx"],
                                    state["q_starts"], state["scale"], state["out"], causal=kind == "prefill",
                                    workspace=state["workspace"])
            return state["out"]
        if kind == "rope":
            pa.pa_rope_append(state["q"], state["k"], state["v"], state["positions"], state["inv_freq"],
                              state["slots"], state["k_cache"], state["v_cache"], state["q_out"],
                              pair_axis=state["axis"], interleaved=state["case"]["interleaved"])
            return state["q_out"], state["k_cache"], state["v_cache"]
        pa.pa_move_blocks(state["k_caches"], state["v_caches"], state["moves"], state["tables"])
        return state["caches"], state["tables"]
    if kind in ("prefill", "cross"):
        return _plain_attention(state)
    return _plain_rope(state) if kind == "rope" else _plain_compact(state)


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] in ("prefill", "cross"):
        n_of, c_of = _ints(case["q_lens"]), _ints(case["ctx_lens"])
        hkv, bs, group = case["hkv"], case["bs"], case["hq"] // case["hkv"]
        result = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        starts = np.concatenate([[0], np.cumsum(n_of)])
        for i in range(len(n_of)):
            if n_of[i] == 0 or c_of[i] == 0:
                continue
            slot = torch.arange(c_of[i], device="cuda")
            slot = st["tables"][i].long()[slot // bs] * bs + slot % bs
            for h in range(case["hq"]):
                keys = st["k_cache"].view(-1, hkv, case["d"])[slot, h // group].double()
                values = st["v_cache"].view(-1, hkv, case["d"])[slot, h // group].double()
                for a in range(0, n_of[i], 2048):
                    b = min(n_of[i], a + 2048)
                    scores = st["q"][starts[i] + a:starts[i] + b, h].double() @ keys.t() * st["scale"]
                    last = torch.arange(a, b, device="cuda") + (c_of[i] - n_of[i])          # last token seen
                    if case["kind"] == "prefill":
                        hidden = torch.arange(c_of[i], device="cuda")[None, :] > last[:, None]
                        scores[hidden] = -math.inf
                    weights = torch.softmax(scores, dim=1)
                    if case["kind"] == "prefill":
                        weights[last < 0] = 0.0
                    result[starts[i] + a:starts[i] + b, h] = weights @ values
        return result
    if case["kind"] == "rope":
        half = case["rotary"] // 2
        i = torch.arange(half, device="cuda")
        first = 2 * i if case["interleaved"] else i
        second = 2 * i + 1 if case["interleaved"] else i + half
        angle = torch.stack([st["positions"][int(a)].double() for a in st["axis"].tolist()], 1) * st["inv_freq"].double()
        turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]

        def turned(x):
            y = x.double()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y[..., first], y[..., second] = z.real, z.imag
            return y

        k, v = st["k_cache"].double(), st["v_cache"].double()
        block, row = st["slots"] // case["bs"], st["slots"] % case["bs"]
        k[block, row] = turned(st["k"])
        v[block, row] = st["v"].double()
        return turned(st["q"]), k, v
    caches = st["caches"].double()
    tables = st["tables"].cpu().numpy()
    renamed = tables.copy()
    for src, dst in st["moves"].tolist():
        caches[:, :, dst] = caches[:, :, src]
        renamed[tables == src] = dst
    return caches, torch.from_numpy(renamed).cuda()
