"""The chunk attention planner, run from its own source on the CPU (g++): a
block of fibers in a chosen order stands in for the GPU's warps, and shared
memory keeps what the plan before left in it.  Every plan has to cover each row
and context step exactly once, whatever the order of the warps."""

import os
import random
import subprocess

import pytest

from conftest import ROOT

HERE = os.path.join(ROOT, "tests", "cpu_emulation")
CSRC = os.path.join(ROOT, "paged_kv_cache_341_b200", "csrc")
STEP, CTAS, SPLIT_UNITS, ROWS16 = 128, 148, 2, 256
FORWARDS, BACKWARDS = 0, 1                      # other numbers: shuffled by that seed


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    work = tmp_path_factory.mktemp("plan")
    with open(os.path.join(CSRC, "prefill_plan.cuh")) as f:
        text = f.read()
    body = text[:text.index("struct PrefillMergeParams")] + "\n}  // namespace pa\n#endif\n"
    lines = [x for x in body.splitlines() if not x.startswith("#include")]
    (work / "plan_source.h").write_text("\n".join(lines) + "\n")
    exe = str(work / "plan")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", str(work), "-I", HERE, os.path.join(HERE, "plan_main.cpp"),
                    "-o", exe], check=True)
    return exe


class Call:
    def __init__(self, q_lens, ctx_lens, heads=2, group=4, rows=ROWS16, causal=True, cap=None, order=FORWARDS,
                 starts=None, tokens=None):
        self.q_lens, self.ctx, self.heads, self.group, self.rows = list(q_lens), list(ctx_lens), heads, group, rows
        self.causal, self.order = causal, order
        self.starts = [sum(self.q_lens[:i]) for i in range(len(self.q_lens) + 1)] if starts is None else list(starts)
        self.tokens = self.starts[-1] if tokens is None else tokens
        self.cap = max(self.ctx + [1]) if cap is None else cap
        s, t = len(self.ctx), self.tokens
        # the capacities of a call's workspace
        tiles = min(t, s) + t * group // rows
        steps = -(-self.cap // STEP)
        pieces = min(SPLIT_UNITS * CTAS * (ROWS16 // rows) // heads, tiles * steps)
        self.max_tiles = tiles
        self.max_slots = pieces if steps > (2 if rows == ROWS16 else 1) and pieces >= 2 else 0
        self.max_merges = self.max_slots // 2

    def text(self):
        head = [self.order, len(self.ctx), self.tokens, self.heads, self.group, self.rows, int(self.causal), self.cap,
                CTAS, self.max_tiles, self.max_merges, self.max_slots]
        return " ".join(map(str, head + self.starts + self.ctx)) + "\n"

    def check(self, entries, merges):
        """Every tile of every chunk once, its steps covered once, the pieces of a split in the merge list."""
        per = self.rows // self.group
        want = {}
        for s, (n, c) in enumerate(zip(self.q_lens, self.ctx)):
            for t0 in range(0, n, per):
                m = min(per, n - t0)
                lim0 = c - n + t0 + 1 if self.causal else c
                last = min(c, lim0 + m - 1) if self.causal else c
                want[self.starts[s] + t0] = (s, m, c, lim0, -(-last // STEP) if last > 0 else 0)
        got, lengths = {}, []
        for seq, tok0, ntok, step0, step1, ctx, lim0, slot in entries:
            assert want[tok0][:4] == (seq, ntok, ctx, lim0)
            got.setdefault(tok0, []).append((step0, step1, slot))
            lengths.append(tok0)
        assert got.keys() == want.keys()
        # longest first, by the length of a tile's first piece (a bucket per length below 1,024 steps)
        first = {t: max(b - a for a, b, _ in p) for t, p in got.items()}
        lengths = [first[t] for t in lengths]
        assert lengths == sorted(lengths, reverse=True)
        by_tok = {m[0]: m for m in merges}
        assert len(by_tok) == len(merges)
        used = set()
        for tok0, pieces in got.items():
            pieces.sort(key=lambda p: p[2])
            at = 0
            for step0, step1, _ in pieces:
                assert step0 == at and step1 >= step0
                at = step1
            assert at == want[tok0][4]
            if len(pieces) == 1 and pieces[0][2] < 0:
                assert tok0 not in by_tok
                continue
            _, ntok, slot0, count = by_tok[tok0]
            assert ntok == want[tok0][1] and count == len(pieces) > 1
            assert [p[2] for p in pieces] == list(range(slot0, slot0 + count)) and slot0 + count <= self.max_slots
            assert not used & set(range(slot0, slot0 + count))
            used |= set(range(slot0, slot0 + count))


def plan(exe, calls):
    """[(error, entries, merges)] of the calls, planned one after another in one process."""
    r = subprocess.run([exe], input="".join(c.text() for c in calls), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, "planner ended with %d (3: wrote out of range, 4: dead wait)" % r.returncode
    rows = iter(r.stdout.splitlines())
    out = []
    for _ in calls:
        err, ne, nm = map(int, next(rows).split())
        out.append((err, [tuple(map(int, next(rows).split())) for _ in range(ne)],
                    [tuple(map(int, next(rows).split())) for _ in range(nm)]))
    return out


def some_calls(rng, order):
    for seqs in (1, 2, 33, 40, 100, 1024, 1500):
        n = [rng.choice([0, 1, 3, 70, 300]) if seqs <= 100 else rng.randint(0, 3) for _ in range(seqs)]
        n[rng.randrange(seqs)] = 5
        ctx = [a + rng.choice([0, 1, 127, 900, 5000]) for a in n]
        yield Call(n, ctx, heads=rng.choice([1, 2, 8]), group=rng.choice([1, 4, 8]), rows=rng.choice([256, 32]),
                   causal=rng.random() < 0.6, order=order)


@pytest.mark.parametrize("order", [FORWARDS, BACKWARDS, 2, 3])
def test_plans_one_after_another(planner, order):
    """Each plan starts from the shared memory that the one before left."""
    calls = list(some_calls(random.Random(7 + order), order))
    calls = calls + calls[::-1]
    for call, (err, entries, merges) in zip(calls, plan(planner, calls)):
        assert err == 0
        call.check(entries, merges)


@pytest.mark.parametrize("order", [FORWARDS, BACKWARDS, 2])
def test_a_bad_length_is_reported_whatever_the_order(planner, order):
    """Of a sequence of the last warp, the first, and one in between."""
    for at in (0, 45, 1023):
        good = Call([1] * 1024, [9] * 1024, order=order)
        bad = Call([1] * 1024, [9] * at + [10] + [9] * (1023 - at), cap=9, order=order)
        assert [r[0] for r in plan(planner, [good, bad, good])] == [0, 2, 0]


@pytest.mark.parametrize("group,rows", [(1, 256), (8, 32), (4, 256), (2, 32)])
def test_long_contexts_are_split_and_covered(planner, group, rows):
    calls = [Call([16], [32701], heads=8, group=group, rows=rows, order=BACKWARDS),
             Call([512] + [1] * 48, [2560] + [300 + 97 * i for i in range(48)], heads=8, group=group, rows=rows),
             Call([9, 0, 70], [0, 4000, 9000], group=group, rows=rows, causal=False, order=BACKWARDS)]
    results = plan(planner, calls)
    for call, (err, entries, merges) in zip(calls, results):
        assert err == 0
        call.check(entries, merges)
    assert results[0][2]                                          # 16 tokens on 32,701: split
