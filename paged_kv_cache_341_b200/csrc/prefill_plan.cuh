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
constexpr int kPrefillRows32 = 64;             // rows per tile, float32 caches
constexpr int kMinSplitSteps = 4;              // a piece of a split context is at least this long
constexpr int kSplitUnits = 2;                 // pieces aimed at per CTA where contexts are split
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

struct PrefillPlanParams {
  const int32_t* q_starts;       // [S + 1]
  const int32_t* context_lens;   // [S]
  PrefillHeader* header;
  int* tile_ends;                // [S]: tiles of sequences 0..s
  PrefillEntry* entries;
  PrefillMerge* merges;
  int num_seqs, num_tokens, num_kv_heads, group, rows;
  int causal, cap;               // cap: tokens a table row can hold
  int ctas;                      // CTAs of the attention grid
  int max_entries, max_merges, max_slots;      // slots are per KV head
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
// their steps), and decides where contexts are split: with W steps over all
// heads and C CTAs, a tile of more than W / (kSplitUnits C) steps is cut into
// equal pieces of at most that many (and at least kMinSplitSteps), so that few
// rows over a long context still fill the GPU, while calls with plenty of
// tiles are not split at all.  The order of entries within a bucket and of the
// partial slots depends on the order of atomics; no result does (each piece
// has its own slot, and a merge reads its pieces in order).
__global__ void __launch_bounds__(kPrefillPlanThreads) prefill_plan_kernel(const PrefillPlanParams p) {
  __shared__ int s_warp[32];
  __shared__ int s_hist[kPrefillBuckets];
  __shared__ unsigned long long s_work;
  __shared__ int s_base, s_max, s_slots, s_merges, s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  allow_dependent_launch();
  wait_prerequisite_grids();

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

  if (tid == 0) {
    s_work = 0;
    s_base = s_max = s_slots = s_merges = s_bad = 0;
  }
  for (int i = tid; i < kPrefillBuckets; i += kPrefillPlanThreads) s_hist[i] = 0;
  __syncthreads();

  // tiles of the sequences before each one
  for (int s0 = 0; s0 < p.num_seqs; s0 += kPrefillPlanThreads) {
    const int s = s0 + tid;
    int tiles = 0;
    if (s < p.num_seqs) {
      int lo, n, ctx;
      bool bad;
      prefill_seq(p, s, &lo, &n, &ctx, &bad);
      if (bad) s_bad = 1;
      tiles = static_cast<int>((static_cast<long long>(n) * p.group + p.rows - 1) / p.rows);
    }
    int total;
    const int incl = scan(tiles, &total) + s_base;
    if (s < p.num_seqs) p.tile_ends[s] = incl;
    __syncthreads();
    if (tid == 0) s_base += total;
    __syncthreads();
  }
  // disjoint chunks fill the list exactly; overlapping ones (an error) are cut off
  if (s_base > p.max_entries) s_bad = 1;
  const int tiles = min(s_base, p.max_entries);

  // tile i of the call: its entry without a split
  auto tile_entry = [&](int i) {
    int lo_s = 0, hi_s = p.num_seqs - 1;
    while (lo_s < hi_s) {
      const int mid = (lo_s + hi_s) >> 1;
      if (p.tile_ends[mid] <= i) lo_s = mid + 1;
      else hi_s = mid;
    }
    const int first = lo_s > 0 ? p.tile_ends[lo_s - 1] : 0;
    int lo, n, ctx;
    bool bad;
    prefill_seq(p, lo_s, &lo, &n, &ctx, &bad);
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

  unsigned long long work = 0;
  int longest = 0;
  for (int i = tid; i < tiles; i += kPrefillPlanThreads) {
    const int n = tile_entry(i).step1;
    work += n;
    longest = max(longest, n);
  }
  for (int o = 16; o > 0; o >>= 1) {
    work += __shfl_xor_sync(0xffffffffu, work, o);
    longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  }
  if (lane == 0) {
    atomicAdd(&s_work, work);
    atomicMax(&s_max, longest);
  }
  __syncthreads();
  const long long target = static_cast<long long>(kSplitUnits) * p.ctas;
  const int limit = max(kMinSplitSteps,
                        static_cast<int>((static_cast<long long>(s_work) * p.num_kv_heads + target - 1) / target));
  const int top = s_max;
  // pieces of a tile of n steps; a tile is left whole when the lists are full
  auto pieces_of = [&](int n) { return n > limit ? (n + limit - 1) / limit : 1; };
  auto bucket_of = [&](int n) {                 // 0 = longest
    return kPrefillBuckets - 1 -
           (top < kPrefillBuckets ? n : static_cast<int>(static_cast<long long>(n) * (kPrefillBuckets - 1) / top));
  };

  for (int pass = 0; pass < 2; ++pass) {
    for (int i = tid; i < tiles; i += kPrefillPlanThreads) {
      PrefillEntry e = tile_entry(i);
      const int n = e.step1;
      const int k = pieces_of(n);
      const int len = (n + k - 1) / k;
      const int bucket = bucket_of(len);
      if (pass == 0) {
        atomicAdd(&s_hist[bucket], k);
        continue;
      }
      int at = atomicAdd(&s_hist[bucket], k);   // (now the bucket's first index)
      int slot = -1;
      if (k > 1) {
        slot = atomicAdd(&s_slots, k);
        const int m = atomicAdd(&s_merges, 1);
        if (m < p.max_merges && slot + k <= p.max_slots)
          p.merges[m] = PrefillMerge{e.tok0, e.ntok, slot, k};
        else
          s_bad = 1;                            // (cannot happen: the lists are sized for the rule above)
      }
      for (int j = 0; j < k; ++j, ++at) {
        e.step0 = min(n, j * len);
        e.step1 = min(n, (j + 1) * len);
        e.slot = k > 1 ? min(slot + j, p.max_slots - 1) : -1;
        if (at < p.max_entries) p.entries[at] = e;
      }
    }
    __syncthreads();
    if (pass == 0) {
      int total;
      static_assert(kPrefillBuckets == kPrefillPlanThreads, "one bucket per thread");
      const int own = s_hist[tid];
      const int incl = scan(own, &total);
      s_hist[tid] = incl - own;
      if (tid == 0) s_base = total;
      __syncthreads();
    }
  }
  if (tid == 0) {
    if (s_base > p.max_entries) s_bad = 1;
    p.header->num_entries = min(s_base, p.max_entries);
    p.header->num_merges = min(s_merges, p.max_merges);
    if (s_bad) set_device_error(DEVERR_BAD_LENGTH);
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
// partials (mostly in L2, where the attention kernel has just put them).
template <typename T, int D>
__global__ void __launch_bounds__(kPrefillMergeWarps * 32) prefill_merge_kernel(const PrefillMergeParams p) {
  constexpr int C = D / 32;                     // columns per lane
  const int lane = threadIdx.x & 31;
  allow_dependent_launch();
  wait_prerequisite_grids();
  const long long total = static_cast<long long>(p.header->num_merges) * p.num_kv_heads * p.rows;
  const long long step = static_cast<long long>(gridDim.x) * kPrefillMergeWarps;
  for (long long w = static_cast<long long>(blockIdx.x) * kPrefillMergeWarps + (threadIdx.x >> 5); w < total;
       w += step) {
    const int row = static_cast<int>(w % p.rows);
    const long long mh = w / p.rows;
    const int h = static_cast<int>(mh % p.num_kv_heads);
    const PrefillMerge m = p.merges[mh / p.num_kv_heads];
    const int tok = row / p.group;
    if (tok >= m.ntok) continue;
    float top = -INFINITY;
    for (int k = lane; k < m.pieces; k += 32)
      top = fmaxf(top, p.part_ml[(static_cast<long long>(m.slot0 + k) * p.num_kv_heads + h) * p.rows + row].x);
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    float l = 0.f;
#pragma unroll 4
    for (int k = 0; k < m.pieces; ++k) {
      const long long at = (static_cast<long long>(m.slot0 + k) * p.num_kv_heads + h) * p.rows + row;
      const float2 ml = p.part_ml[at];
      if (ml.y == 0.f) continue;                // nothing visible in this piece: no output was written
      const float f = exp2f(ml.x - top);
      l += f * ml.y;
      const float* o = p.part_acc + at * D + lane * C;
      if constexpr (C == 4) {
        const float4 v = *reinterpret_cast<const float4*>(o);
        acc[0] += f * v.x;
        acc[1] += f * v.y;
        acc[2] += f * v.z;
        acc[3] += f * v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(o);
        acc[0] += f * v.x;
        acc[1] += f * v.y;
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* dst = static_cast<T*>(p.out) +
             (static_cast<long long>(m.tok0 + tok) * p.num_kv_heads * p.group + h * p.group + row % p.group) * D +
             lane * C;
#pragma unroll
    for (int c = 0; c < C; ++c) dst[c] = static_cast<T>(acc[c] * inv);
  }
}

}  // namespace pa

#endif
