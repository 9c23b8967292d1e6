// Work list of the chunk attention kernels and the merge of split contexts.
//
// A tile is `rows` query rows of one KV head: the rows of a sequence's chunk
// are its (token, query head of the group) pairs, token-major, so that the G
// query heads that share a KV head share every K/V tile, and a causal tile
// spans only rows / G tokens.  Row r of tile i is token (i * rows + r) / G,
// head r % G.  Along the context a tile needs the K/V steps of kStepTokens
// tokens up to the last token its last row may see.  An entry of the list is
// a tile with a range of its steps; every KV head is one unit of each entry.
#ifndef PAGEDATTN_PREFILL_PLAN_CUH
#define PAGEDATTN_PREFILL_PLAN_CUH

#include <cstdint>

#include "decode.cuh"
#include "dtype.cuh"
#include "ptx.cuh"

namespace pa {

constexpr int kStepTokens = 128;               // context tokens per K/V step
constexpr int kPrefillRows16 = 256;            // rows per tile, 16-bit caches (two MMA tiles of 128)
constexpr int kPrefillRows32 = 32;             // rows per tile, float32 caches
constexpr int kSplitUnits = 2;                 // pieces of 256 rows per CTA that the workspace has room for
constexpr int kPrefillPlanThreads = 1024;
constexpr int kPrefillBuckets = 1024;

struct __align__(16) PrefillEntry {
  int seq;
  int tok0, ntok;              // first query token (of the packed array) and tokens of the tile
  int step0, step1;            // K/V steps [step0, step1)
  int ctx;                     // context length of the sequence
  int lim0;                    // context tokens the tile's first token may see (may be <= 0)
  int slot;                    // partial slot of this piece, or -1: the whole range, written to out
};
static_assert(sizeof(PrefillEntry) == 32, "two 16-byte loads");

struct PrefillMerge {
  int tok0, ntok;
  int slot0, pieces;
};

struct PrefillHeader {
  int num_entries, num_merges;
};

// How long the attention kernel takes for a work list, in K/V steps, from sums
// over its pieces: every piece costs its steps and `piece` for its start and
// end, a piece of a split context also `partial` for its partial result; C
// CTAs take the pieces longest first, so that no schedule beats the average,
// and pieces of more than half of the longest share no CTA unless they fill
// more than one round; a split call pays `merge` for the merge.
struct PlanCost {
  int min_steps;                 // a piece of a split context is at least about this long
  float piece, partial, merge;   // in steps, as above
};
// (a step takes about 1.5 us with tensor cores, and 4 to 8 us without, of a CTA that has its SM to itself)
constexpr PlanCost kPlanCost16{2, 2.f, 1.5f, 3.f};
constexpr PlanCost kPlanCost32{1, 0.5f, 0.2f, 0.7f};

struct PrefillPlanParams {
  const int32_t* q_starts;       // [S + 1]
  const int32_t* context_lens;   // [S]
  PrefillHeader* header;
  int* tile_ends;                // [S]: tiles of sequences 0..s
  PrefillEntry* entries;
  PrefillMerge* merges;
  int num_seqs, num_tokens, num_kv_heads, group, rows;
  int causal, cap;               // cap: tokens a table row can hold
  int ctas;                      // what the estimate spreads the pieces over: one per SM (the float32 kernel
                                 // runs several CTAs on an SM, which then share its rate)
  int max_tiles, max_merges, max_slots;        // capacities; slots are per KV head
  int* tile_steps;               // [max_tiles]
  PlanCost cost;
};

// Chunk of sequence s, clamped into the arrays: tokens [lo, lo + n), context.
__device__ __forceinline__ void prefill_seq(const PrefillPlanParams& p, int s, int* lo, int* n, int* ctx, bool* bad) {
  const int a = p.q_starts[s], b = p.q_starts[s + 1], c = p.context_lens[s];
  *lo = min(max(a, 0), p.num_tokens);
  *n = max(min(b, p.num_tokens) - *lo, 0);
  *ctx = min(max(c, 0), p.cap);
  *bad = *lo != a || *lo + *n != b || *ctx != c;
}

// One CTA lists the work of a call, longest pieces first (a counting sort on
// their steps), and decides where contexts are split: 32 limits on the steps of
// a piece (the longest context over 1, 2, .. 16, and over the numbers that make
// 1 to 16 full rounds of the CTAs) are weighed by the estimate above, one per
// warp, and the cheapest is taken, so that few rows over a long context fill
// the GPU while calls with plenty of tiles are not split at all.  The order of
// entries within a bucket and of the partial slots depends on the order of
// atomics; no result does (each piece has its own slot, and a merge reads its
// pieces in order).  Bound by the latency of its few dependent loads.
__global__ void __launch_bounds__(kPrefillPlanThreads) prefill_plan_kernel(const PrefillPlanParams p) {
  __shared__ int s_warp[32];
  __shared__ int s_hist[kPrefillBuckets];
  __shared__ float s_est[32];
  __shared__ int s_limit[32];
  __shared__ int s_base, s_max, s_slots, s_merges, s_bad;
  // of up to kPrefillPlanThreads sequences and tiles, kept here (else in the workspace)
  __shared__ int s_end[kPrefillPlanThreads], s_steps[kPrefillPlanThreads];
  __shared__ int4 s_seq[kPrefillPlanThreads];   // first token, tokens, context
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  allow_dependent_launch();
  if (tid == 0) s_base = s_max = s_slots = s_merges = s_bad = 0;
  s_hist[tid] = 0;
  static_assert(kPrefillBuckets == kPrefillPlanThreads, "one bucket per thread");
  wait_prerequisite_grids();
  __syncthreads();                              // every warp sees the zeroes (the wait orders no warps)

  // inclusive scan of one int per thread over the CTA; *total = the sum
  auto scan = [&](int v, int* total) {
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    if (warp == 0) {
      int w = s_warp[lane];
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
      }
      s_warp[lane] = w;
    }
    __syncthreads();
    const int r = v + (warp > 0 ? s_warp[warp - 1] : 0);
    *total = s_warp[31];
    __syncthreads();
    return r;
  };

  const bool near_seqs = p.num_seqs <= kPrefillPlanThreads;
  const int* ends = near_seqs ? s_end : p.tile_ends;

  // tiles of sequences 0 .. s
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPrefillPlanThreads) {
    const int s = s0 + tid;
    int tiles = 0;
    if (s < p.num_seqs) {
      int lo, n, ctx;
      bool bad;
      prefill_seq(p, s, &lo, &n, &ctx, &bad);
      if (bad) s_bad = 1;
      tiles = static_cast<int>((static_cast<long long>(n) * p.group + p.rows - 1) / p.rows);
      if (near_seqs) s_seq[s] = make_int4(lo, n, ctx, 0);
    }
    int total;
    const int before = s_base;
    const int incl = scan(tiles, &total) + before;
    if (s < p.num_seqs) (near_seqs ? s_end : p.tile_ends)[s] = incl;
    if (tid == 0) s_base = before + total;
    __syncthreads();
  }
  // disjoint chunks fill the list exactly; overlapping ones (an error) are cut off
  const int tiles = min(s_base, p.max_tiles);
  int* steps = tiles <= kPrefillPlanThreads ? s_steps : p.tile_steps;

  // tile i of the call: its entry without a split
  auto tile_entry = [&](int i) {
    int lo_s = 0, hi_s = p.num_seqs - 1;
    while (lo_s < hi_s) {
      const int mid = (lo_s + hi_s) >> 1;
      if (ends[mid] <= i) lo_s = mid + 1;
      else hi_s = mid;
    }
    const int first = lo_s > 0 ? ends[lo_s - 1] : 0;
    int lo, n, ctx;
    bool bad;
    if (near_seqs) {
      lo = s_seq[lo_s].x;
      n = s_seq[lo_s].y;
      ctx = s_seq[lo_s].z;
    } else {
      prefill_seq(p, lo_s, &lo, &n, &ctx, &bad);
    }
    const int per = p.rows / p.group;           // tokens of a tile
    const int t0 = (i - first) * per;
    PrefillEntry e;
    e.seq = lo_s;
    e.tok0 = lo + t0;
    e.ntok = min(per, n - t0);
    e.ctx = ctx;
    e.lim0 = p.causal ? ctx - n + t0 + 1 : ctx;
    const int last = p.causal ? min(ctx, e.lim0 + e.ntok - 1) : ctx;
    e.step0 = 0;
    e.step1 = last > 0 ? (last + kStepTokens - 1) / kStepTokens : 0;
    e.slot = -1;
    return e;
  };

  PrefillEntry mine;                            // of tile tid, kept for the listing
  mine.step1 = 0;
  int longest = 0;
  for (int i = tid; i < tiles; i += kPrefillPlanThreads) {
    const PrefillEntry e = tile_entry(i);
    if (i == tid) mine = e;
    steps[i] = e.step1;
    longest = max(longest, e.step1);
  }
  for (int o = 16; o > 0; o >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  if (lane == 0) atomicMax(&s_max, longest);
  __syncthreads();
  const int top = s_max;

  // pieces of a tile of n steps under a limit
  auto pieces_of = [](int n, int limit) { return n > limit ? (n + limit - 1) / limit : 1; };
  {
    const int units = max(1, tiles * p.num_kv_heads);
    const int cut = warp < 16 ? warp + 1 : max(1, (warp - 15) * p.ctas / units);
    const int limit = p.max_slots > 0 ? max(min(top, p.cost.min_steps), (top + cut - 1) / cut) : max(top, 1);
    const float big = 0.5f * min(top, limit);
    float work = 0.f, big_work = 0.f;
    int bigs = 0, slots = 0, merges = 0;
    for (int i = lane; i < tiles; i += 32) {
      const int n = steps[i];
      const int k = pieces_of(n, max(limit, 1));
      const float each = (k > 1 ? static_cast<float>((n + k - 1) / k) + p.cost.partial : static_cast<float>(n)) + p.cost.piece;
      work += k * each;
      if (each > big + p.cost.piece) {
        bigs += k;
        big_work += k * each;
      }
      if (k > 1) {
        slots += k;
        ++merges;
      }
    }
    for (int o = 16; o > 0; o >>= 1) {
      work += __shfl_xor_sync(0xffffffffu, work, o);
      big_work += __shfl_xor_sync(0xffffffffu, big_work, o);
      bigs += __shfl_xor_sync(0xffffffffu, bigs, o);
      slots += __shfl_xor_sync(0xffffffffu, slots, o);
      merges += __shfl_xor_sync(0xffffffffu, merges, o);
    }
    if (lane == 0) {
      const float h = static_cast<float>(p.num_kv_heads), c = static_cast<float>(p.ctas);
      float est = work * h / c;
      if (bigs > 0) est = fmaxf(est, ceilf(bigs * h / c) * (big_work / bigs));
      if (merges > 0) est += p.cost.merge;
      const bool fits = slots <= p.max_slots && merges <= p.max_merges;
      s_est[warp] = fits || warp == 0 ? est : INFINITY;
      s_limit[warp] = max(limit, 1);
    }
  }
  __syncthreads();
  int best = 0;                                 // (warp 0's limit is the longest context: no split)
  for (int w = 1; w < 32; ++w)
    if (s_est[w] < s_est[best]) best = w;
  const int limit = s_limit[best];

  auto bucket_of = [&](int n) {                 // 0 = longest
    return kPrefillBuckets - 1 -
           (top < kPrefillBuckets ? n : static_cast<int>(static_cast<long long>(n) * (kPrefillBuckets - 1) / top));
  };
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = tid; i < tiles; i += kPrefillPlanThreads) {
      const int n = i == tid ? mine.step1 : steps[i];
      const int k = pieces_of(n, limit);
      const int len = (n + k - 1) / k;
      const int bucket = bucket_of(len);
      if (pass == 0) {
        atomicAdd(&s_hist[bucket], k);
        continue;
      }
      PrefillEntry e = i == tid ? mine : tile_entry(i);
      int at = atomicAdd(&s_hist[bucket], k);   // (the bucket's next index)
      int slot = -1;
      if (k > 1) {
        slot = atomicAdd(&s_slots, k);          // (fits: weighed above)
        p.merges[atomicAdd(&s_merges, 1)] = PrefillMerge{e.tok0, e.ntok, slot, k};
      }
      for (int j = 0; j < k; ++j, ++at) {
        e.step0 = min(n, j * len);
        e.step1 = min(n, (j + 1) * len);
        e.slot = k > 1 ? slot + j : -1;
        p.entries[at] = e;
      }
    }
    __syncthreads();
    if (pass == 0) {
      int total;
      const int own = s_hist[tid];
      const int incl = scan(own, &total);
      s_hist[tid] = incl - own;
      if (tid == 0) p.header->num_entries = total;
      __syncthreads();
    }
  }
  if (tid == 0) {
    p.header->num_merges = s_merges;
    if (s_bad || s_base > p.max_tiles) set_device_error(DEVERR_BAD_LENGTH);
  }
}

struct PrefillMergeParams {
  const PrefillHeader* header;
  const PrefillMerge* merges;
  const float* part_acc;         // [slot][Hkv][rows][D]
  const float2* part_ml;         // [slot][Hkv][rows]
  void* out;                     // [T][Hq][D]
  int num_kv_heads, group, rows;
};

constexpr int kPrefillMergeWarps = 8;

// out row = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p over the pieces of a
// split context, in piece order; one warp per row.  Bound by the reads of the
// partials (mostly in L2, where the attention kernel has just put them): the
// weights of 32 pieces are worked out at once, one per lane, and the rows of
// eight pieces are in flight at a time.
template <typename T, int D>
__global__ void __launch_bounds__(kPrefillMergeWarps * 32) prefill_merge_kernel(const PrefillMergeParams p) {
  constexpr int C = D / 32;                     // columns per lane
  const int lane = threadIdx.x & 31;
  allow_dependent_launch();
  wait_prerequisite_grids();
  const int per = p.num_kv_heads * p.rows;
  const int total = p.header->num_merges * per;
  for (int w = blockIdx.x * kPrefillMergeWarps + (threadIdx.x >> 5); w < total; w += gridDim.x * kPrefillMergeWarps) {
    const int i = w / per, hr = w - i * per;
    const int h = hr / p.rows, row = hr - h * p.rows;
    const PrefillMerge m = p.merges[i];
    const int tok = row / p.group;
    if (tok >= m.ntok) continue;
    const int64_t at0 = (static_cast<int64_t>(m.slot0) * p.num_kv_heads + h) * p.rows + row;
    const float* acc0 = p.part_acc + at0 * D + lane * C;
    float top = -INFINITY;
    float2 ml = make_float2(-INFINITY, 0.f);
    for (int k = lane; k < m.pieces; k += 32) {
      ml = p.part_ml[at0 + static_cast<int64_t>(k) * per];
      top = fmaxf(top, ml.x);
    }
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    float l = 0.f;
    for (int k0 = 0; k0 < m.pieces; k0 += 32) {
      const int n = min(32, m.pieces - k0);
      if (m.pieces > 32) ml = lane < n ? p.part_ml[at0 + static_cast<int64_t>(k0 + lane) * per] : make_float2(0.f, 0.f);
      // (a piece in which nothing is visible has l = 0: its weight is zero, whatever its row holds)
      const float f = ml.y == 0.f ? 0.f : exp2f(ml.x - top);
      l += f * ml.y;
#pragma unroll 8
      for (int k = 0; k < n; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k);
        const float* o = acc0 + static_cast<int64_t>(k0 + k) * per * D;
        float v[C];
        if constexpr (C == 4) {
          *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(o);
        } else {
          *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] += fk == 0.f ? 0.f : fk * v[c];
      }
    }
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* dst = static_cast<T*>(p.out) +
             (static_cast<int64_t>(m.tok0 + tok) * p.num_kv_heads * p.group + h * p.group + row % p.group) * D +
             lane * C;
    T t[C];
#pragma unroll
    for (int c = 0; c < C; ++c) t[c] = static_cast<T>(acc[c] * inv);
    if constexpr (sizeof(T) * C == 16) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<uint4*>(t);
    else if constexpr (sizeof(T) * C == 8) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(t);
    else *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<uint32_t*>(t);
  }
}

}  // namespace pa

#endif
