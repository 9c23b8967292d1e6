// Chunk attention on the fifth-generation tensor cores (tcgen05 + tensor
// memory), 16-bit caches.
//
// out[t][h] = sum_j softmax_j(scale q[t][h] . K[j]) V[j] over the context
// tokens j < lim(t), in one pass over the context: per step of 128 tokens
// S = Q K^T, m = running row maximum, P = 2^(S scale log2(e) - m), O += P V,
// l += sum P; out = O / l.
//
// One CTA per SM (it holds all the tensor memory) takes units of the work list
// (prefill_plan.cuh): 256 query rows of one KV head as two tiles of 128, and a
// range of context steps.  Every K/V tile serves both query tiles.
//
// Roles (320 threads):
//   warps 0-7   softmax, four warps per query tile, one thread per row (=
//               tensor-memory lane): the whole row of 128 scores is read into
//               registers, so that the row maximum needs no exchange; P is
//               rounded to the cache's type and written over S.  (Sixteen warps,
//               four threads per row, were no faster: 1.45 against 1.31 ms.)
//   warp 8      TMA producer: Q tiles, then K and V tiles alternately through
//               one ring.  A piece of a cache block (8, 16, ... 128 tokens) is
//               one box of a 5-D view of the cache that puts the D/64 column
//               panels of 8 tokens behind one another (1024-byte atoms,
//               128-byte swizzled), so a tile of 128 tokens is 8 copies for
//               blocks of 16, issued by as many lanes at once.  (One elected
//               lane issuing them in turn took 1,000 cycles for a tile of 8
//               beside the softmax warps, against 600 to 800, and held up the
//               products: 1,300 -> 1,400 us.)
//   warp 9      issues the MMAs: the whole warp runs the loop and one elected
//               lane issues, so that the operands stay in uniform registers
//               (from a single thread's branch a product was issued every 90
//               to 100 cycles beside the busy softmax warps, and the tensor
//               core takes 64 for one: 1,056 -> 1,289 TFLOP/s).
// Tensor memory: query tile g owns columns 256 g..: S (and P over it) 0..127,
// O 128...  Products issued by one thread complete in order, so S_g(t+1) may
// overwrite P_g(t) once PV_g(t) is issued before it, and when S_g(t) is
// reported ready, PV_g(t-1) has completed and O may be rescaled.  While one
// query tile's softmax runs, the tensor core works for the other.  P is handed
// over in two halves, so that PV starts before the second half is written.
//
// The reference maximum of a row moves only when a score passes it by 2^kTau
// (then the thread rescales its row of O), which the final division undoes
// exactly; weights stay below 2^kTau, far from overflow.  Since it rarely moves,
// a step's first weights are worked out with the maximum as it stands while the
// step's own maximum is still being found (exponentials and comparisons use
// different pipes), and done again where it does: 1.32 -> 1.21 ms.  S, O and
// the statistics are float32; P is rounded to the cache's type for the second
// product (its sum is taken before the rounding, whose errors are unbiased).
//
// Measured, in short bursts as all times in this file: 8,192 tokens on a
// 16,384-token context (32/8 heads of 128, bf16, blocks of 16) 1.21 ms = 1,367
// TFLOP/s, 0.83 of the measured bf16 burst peak.  As a call among others it runs
// into the power limit: 1.41 ms = 1,170 TFLOP/s, 0.84 of the sustained peak.
// With head_dim 64 that call takes 1.07 ms = 769 TFLOP/s, its exponentials alone
// 0.69 ms.  What bounds the burst is the chain S -> softmax -> PV -> next S of a query tile
// (about 3,000 cycles for the two tiles' 2,048 of products): exponentials 1,100
// to 1,300, reading S and the maximum 200, and 200 to 300 for each hand-over
// between the softmax warps and the tensor core.  Sharing one S buffer between
// the tiles and giving P its own columns, so that S(t+1) does not wait for P(t),
// measured no faster, nor did exponentials as polynomials on the FMA pipe (2 or
// 4 of 16: 1.28 and 1.32 ms) or 208 registers per softmax thread (1.54 ms).
//
// Between units a query tile waits for the other tile's last products and for
// its Q (about 8,000 cycles from one unit's last score to the next one's first).
// Issuing the next unit's first S with this one's last products measured no
// faster: the longer issue loop lost what the shorter gap gained (1.23 against
// 1.19 ms; prompts of 1,300 units 237 against 221 us).
//
// Masks are compared only in steps that hold a masked token for some row of
// the tile; such tokens get weight zero whatever K holds.  V rows behind the
// context's end are zeroed in shared memory (a weight of zero would not undo
// a NaN there).  Every wait is bounded in time.
#ifndef PAGEDATTN_PREFILL_TC_CUH
#define PAGEDATTN_PREFILL_TC_CUH

#include <cuda.h>
#include <cstdint>
#include <type_traits>

#include "prefill.cuh"
#include "prefill_plan.cuh"
#include "prefix_tc.cuh"
#include "tcgen05.cuh"

namespace pa {

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_addr(bar))
      : "memory");
}

// One lane of the (converged) warp: 1 in it, 0 in the others.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
// Products and commits issued by the lane with `one` set, in code that the whole
// warp runs: operands stay in uniform registers.
template <bool kAcc>
__device__ __forceinline__ void mma_ss_one(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(one), "n"(kAcc ? 1 : 0)
      : "memory");
}
__device__ __forceinline__ void mma_ts_one(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 q, %4, 0;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(one), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t one, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(one)
      : "memory");
}

// 32 bytes to global memory: one store when `wide` (the address is then 32-byte
// aligned), else two of 16 bytes.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

constexpr int kChunkThreads = 320;
// K/V tiles in flight: as many as fit with head_dim 128 (32 KB each); with 64 more
// than 6 gain nothing (8,192 tokens on 16,384: 1.49 ms with 6, 1.51 with 5, 1.57
// with 11)
template <int D>
constexpr int kChunkStages = D == 128 ? 5 : 6;
constexpr int kChunkGroupBars = 6;

template <int D>
__host__ __device__ constexpr size_t prefill_umma_smem_bytes() {
  const size_t n = 1024 + 2 * static_cast<size_t>(D / 64) * 128 * 128            // Q tiles
                   + kChunkStages<D> * static_cast<size_t>(D / 64) * 128 * 128      // K/V ring
                   + 1024 + 512;                                                 // (m, l) of a row, barriers
  return n < kUmmaMinSmem ? kUmmaMinSmem : n;
}

// How the two softmax groups share a unit.  Normally group g has query tile g
// and every step.  A unit whose rows fit one tile (a chunk of few tokens, a
// decoding sequence) is dealt by steps instead: both groups hold the same rows,
// group g takes steps step0 + g, + 2, ..., and group 0 combines the two partial
// outputs at the end; a lone group would leave half of the softmax warps idle and
// wait for its own products (48 decoding sequences beside a 512-token chunk,
// 32/8 heads: 156 -> 137 us; 16 tokens on a 32k context, 64/8 heads: 36 -> 28 us
// of the kernel).
__device__ __forceinline__ int chunk_steps(const PrefillEntry& e, int g, int group, int causal) {
  const int per = 128 / group;
  const int last = min(e.ntok, (g + 1) * per) - 1;         // its last token
  if (last < g * per) return 0;
  const int lim = causal ? min(e.ctx, e.lim0 + last) : e.ctx;
  const int end = min(e.step1, (max(lim, 0) + kStepTokens - 1) / kStepTokens);
  return max(0, end - e.step0);
}
__device__ __forceinline__ bool chunk_dual(const PrefillEntry& e, int group, int steps) {
  return e.ntok * group <= 128 && steps >= 2;
}

template <typename T, int D>
__global__ void __launch_bounds__(kChunkThreads, 1)
    prefill_umma_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_q, const PrefillParams prm, const int piece_rows) {
  static_assert(sizeof(T) == 2 && (D == 64 || D == 128), "16-bit caches, head_dim 64 or 128");
  constexpr int kHalves = D / 64;
  constexpr uint32_t kAtomRow = kHalves * 1024;          // 8 tokens, all panels
  constexpr uint32_t kTileBytes = 16 * kAtomRow;         // 128 tokens
  constexpr uint32_t kQPanel = 128 * 128;
  constexpr uint32_t kQBytes = kHalves * kQPanel;
  constexpr int NS = kChunkStages<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  using M = MmaType<T>;

  extern __shared__ __align__(1024) unsigned char smem[];
  const uintptr_t base = (reinterpret_cast<uintptr_t>(smem) + 1023) & ~static_cast<uintptr_t>(1023);
  unsigned char* s_q = reinterpret_cast<unsigned char*>(base);          // [tile][panel][128 rows][128 B]
  unsigned char* s_kv = s_q + 2 * kQBytes;                              // [stage][token / 8][panel][8][128 B]
  float2* s_ml = reinterpret_cast<float2*>(s_kv + NS * static_cast<size_t>(kTileBytes));    // [128 rows], dual units
  uint64_t* full = reinterpret_cast<uint64_t*>(s_ml + 128);
  uint64_t* empty = full + NS;
  uint64_t* grp = empty + NS;
  auto s_full = [&](int g) { return grp + kChunkGroupBars * g; };       // S ready
  auto p_half = [&](int g) { return grp + kChunkGroupBars * g + 1; };   // P of the first 64 tokens ready, O rescaled
  auto p_full = [&](int g) { return grp + kChunkGroupBars * g + 2; };   // the rest of P
  auto o_done = [&](int g) { return grp + kChunkGroupBars * g + 3; };   // a unit's last PV
  auto o_free = [&](int g) { return grp + kChunkGroupBars * g + 4; };   // O read out
  uint64_t* q_full = grp + kChunkGroupBars * 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* tail = q_full + 2;
  uint64_t* drain = q_full + 3;
  uint64_t* ml_full = q_full + 4;                // group 1's (m, l) of a dual unit
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int G = prm.group;
  allow_dependent_launch();

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(s_full(g), 1);
      mbar_init(p_half(g), 4);                   // one arrival per softmax warp
      mbar_init(p_full(g), 4);
      mbar_init(o_done(g), 1);
      mbar_init(o_free(g), 4);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(tail, 1);
    mbar_init(drain, 1);
    mbar_init(ml_full, 4);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(tmem_slot, kUmmaTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  wait_prerequisite_grids();
  const long long units = static_cast<long long>(prm.header->num_entries) * prm.num_kv_heads;
  // unit of round r, -1 past the last
  auto unit_of = [&](int r) {
    const long long u = prefill_snake(r, blockIdx.x, gridDim.x);
    return u < units ? static_cast<int>(u) : -1;
  };
  const int rounds = static_cast<int>((units + gridDim.x - 1) / gridDim.x);

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
      prefetch_tensormap(&tm_q);
    }
    const int BS = prm.block_size;
    const int pieces = kStepTokens / piece_rows;           // 1..16 copies per tile
    int st = 0;
    uint32_t ph = 0;
    int armed = 0;                                         // tiles whose copies were issued
    int loaded = 0;                                        // units whose Q was loaded
    int tails = 0;
    bool ok = true;
    for (int r = 0; ok && r < rounds; ++r) {
      const int u = unit_of(r);
      if (u < 0) continue;
      int h;
      const PrefillEntry en = prefill_unit(prm, u, &h);
      const int n0 = chunk_steps(en, 0, G, prm.causal), n1 = chunk_steps(en, 1, G, prm.causal);
      const int steps = max(n0, n1);
      if (steps == 0) continue;
      const bool dual = chunk_dual(en, G, steps);
      const int ahead = dual ? 2 : 1;
      const int32_t* table = prm.block_tables + static_cast<int64_t>(en.seq) * prm.max_blocks;
      // first cache row / 8 of this lane's piece of step t
      auto piece_row = [&](int t) {
        const int tok = t * kStepTokens + lane * piece_rows;
        if (lane >= pieces || tok >= en.ctx) return 0;
        const int b = tok / BS;
        int phys = table[b];                     // (not through the read-only path: it may be newer than this grid)
        if (phys < 0 || phys >= prm.num_blocks) {
          set_device_error(DEVERR_BAD_BLOCK_ID);
          phys = 0;
        }
        return (phys * BS + (tok - b * BS)) >> 3;
      };
      // one K or V tile: step t, its pieces' rows in row8 of each lane
      auto load = [&](bool is_v, int t, int row8) {
        const int ntok = min(kStepTokens, en.ctx - t * kStepTokens);      // >= 1
        const int n = (ntok + piece_rows - 1) / piece_rows;
        const uint32_t tx = static_cast<uint32_t>(n) * (piece_rows / 8) * kAtomRow;
        if (!__all_sync(0xffffffffu, mbar_wait(&empty[st], ph ^ 1, abort_flag))) return false;
        unsigned char* dst = s_kv + static_cast<size_t>(st) * kTileBytes;
        // the last V tile of a context lands on a barrier of its own first:
        // the rows behind the context's end are zeroed before it is handed on
        const bool fix = is_v && ntok < kStepTokens;
        uint64_t* bar = fix ? tail : &full[st];
        if (lane == 0) mbar_arrive_expect_tx(bar, tx);
        __syncwarp();
        if (lane < n)
          tma_load_5d(dst + lane * (piece_rows / 8) * kAtomRow, is_v ? &tm_v : &tm_k, bar, 0, 0, 0, row8, h);
        bool fine = true;
        if (fix) {
          // (the copies are in flight whatever happens to the other warps: wait for them alone)
          fine = __all_sync(0xffffffffu, mbar_wait_drain(tail, tails & 1));
          ++tails;
          // 16-byte chunks of rows ntok..127: atom row, panel, row, chunk
          for (int i = lane; i < (kStepTokens - ntok) * kHalves * 8; i += 32) {
            const int row = ntok + i / (kHalves * 8), c = i % (kHalves * 8);
            *reinterpret_cast<uint4*>(dst + (row >> 3) * kAtomRow + (c >> 3) * 1024 + (row & 7) * 128 +
                                      (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[st]);
        }
        ++armed;
        if (++st == NS) {
          st = 0;
          ph ^= 1;
        }
        return fine;
      };
      // K of the first `ahead` steps, then V(i), K(i + ahead): the order of their
      // use; the rows of steps i, i + 1, i + 2 are at hand, read once per step
      auto rows_at = [&](int i) { return i < steps ? piece_row(en.step0 + i) : 0; };
      int ra = rows_at(0), rb = rows_at(1), rc = rows_at(2);
      ok = load(false, en.step0, ra) && (!dual || load(false, en.step0 + 1, rb));
      if (!ok) break;
      // Q, once the last S of the unit before has completed (the first K tiles are
      // on their way by then)
      if (!__all_sync(0xffffffffu, mbar_wait(q_empty, (loaded & 1) ^ 1, abort_flag))) {
        ok = false;
        break;
      }
      if (lane == 0) {
        const int copies = dual || n1 > 0 ? 2 : 1;
        mbar_arrive_expect_tx(q_full, copies * kQBytes);
        for (int g = 0; g < copies; ++g)
          for (int hf = 0; hf < kHalves; ++hf)
            tma_load_4d(s_q + g * kQBytes + hf * kQPanel, &tm_q, q_full, 0, hf, h * G, en.tok0 + (dual ? 0 : g * (128 / G)));
      }
      __syncwarp();
      ++loaded;
      for (int i = 0; ok && i < steps; ++i) {
        const int rv = ra, rk = dual ? rc : rb;
        ra = rb;
        rb = rc;
        rc = rows_at(i + 3);
        ok = load(true, en.step0 + i, rv) && (i + ahead >= steps || load(false, en.step0 + i + ahead, rk));
      }
    }
    // copies still in flight must land before the CTA may exit
    if (lane == 0) {
      for (int k = 0; k < min(armed, NS); ++k) {
        if (--st < 0) {
          st = NS - 1;
          ph ^= 1;
        }
        mbar_wait_drain(&full[st], ph);
      }
      if (loaded > 0) mbar_wait_drain(q_full, (loaded - 1) & 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // --------------------------------------------------------- MMA issuer
    {
      const uint32_t one = elect_lane();
      constexpr uint32_t idesc_s = tc::idesc_f16<kBf16>(128, 128, false, false);
      constexpr uint32_t idesc_o = tc::idesc_f16<kBf16>(128, D, false, true);
      const uint64_t q_desc = tc::smem_desc_sw128(smem_addr(s_q), 16, 1024);
      const uint64_t k_desc = tc::smem_desc_sw128(smem_addr(s_kv), 16, kAtomRow);
      const uint64_t v_desc = tc::smem_desc_sw128(smem_addr(s_kv), 1024, kAtomRow);
      bool ok = true;
      int st = 0;
      uint32_t ph = 0;
      int units_g[2] = {0, 0}, tiles_g[2] = {0, 0};
      int loaded = 0;
      auto issue_s = [&](int g, int ks) {
        const uint64_t kb = k_desc + ((ks * kTileBytes) >> 4);
        const uint64_t qb = q_desc + ((g * kQBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t qk = qb + (((kk >> 2) * kQPanel + (kk & 3) * 32) >> 4);
          const uint64_t kk_ = kb + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4);
          if (kk == 0) mma_ss_one<false>(one, tmem + g * kUmmaGroupCols + kSCol, qk, kk_, idesc_s);
          else mma_ss_one<true>(one, tmem + g * kUmmaGroupCols + kSCol, qk, kk_, idesc_s);
        }
        commit_one(one, s_full(g));
      };
      auto issue_pv = [&](int g, int vs, int half, bool first) {
        const uint64_t vb = v_desc + ((vs * kTileBytes) >> 4);
        const uint32_t col = tmem + g * kUmmaGroupCols;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int kk = half * 4 + k;
          mma_ts_one(one, col + kOCol, col + kSCol + kk * 8, vb + ((kk * 2 * kAtomRow) >> 4), idesc_o, !first || k > 0);
        }
      };
      auto advance = [&]() {
        if (++st == NS) {
          st = 0;
          ph ^= 1;
        }
      };
      for (int r = 0; ok && r < rounds; ++r) {
        const int u = unit_of(r);
        if (u < 0) continue;
        int h;
        const PrefillEntry en = prefill_unit(prm, u, &h);
        int ends[2];
        ends[0] = en.step0 + chunk_steps(en, 0, G, prm.causal);
        ends[1] = en.step0 + chunk_steps(en, 1, G, prm.causal);
        const int end = max(ends[0], ends[1]);
        if (end <= en.step0) continue;
        if (chunk_dual(en, G, end - en.step0)) {
          // the groups take the steps in turn: PV(i), S(i + 2) of group i % 2
          const int n = end - en.step0;
          ok = mbar_wait(q_full, loaded & 1, abort_flag);
          ++loaded;
          for (int i = -2; ok && i < n; ++i) {
            const int g = i & 1, vs = st;
            if (i >= 0) {
              ok = mbar_wait(&full[vs], ph, abort_flag) && mbar_wait(p_half(g), tiles_g[g] & 1, abort_flag) &&
                   (i >= 2 || units_g[g] == 0 || mbar_wait(o_free(g), (units_g[g] - 1) & 1, abort_flag));
              if (!ok) break;
              advance();
              tc::fence_after_sync();
              issue_pv(g, vs, 0, i < 2);
              ok = mbar_wait(p_full(g), tiles_g[g] & 1, abort_flag);
              if (!ok) break;
              ++tiles_g[g];
              tc::fence_after_sync();
              issue_pv(g, vs, 1, false);
            }
            if (i + 2 < n) {
              ok = mbar_wait(&full[st], ph, abort_flag);
              if (!ok) break;
              tc::fence_after_sync();
              issue_s(g, st);
            } else {
              commit_one(one, o_done(g));
              ++units_g[g];
            }
            if (i >= 0) commit_one(one, &empty[vs]);
            if (i + 2 < n) {
              commit_one(one, &empty[st]);
              advance();
              if (i + 3 == n) commit_one(one, q_empty);    // the unit's last S was issued
            }
          }
          continue;
        }
        ok = mbar_wait(q_full, loaded & 1, abort_flag) && mbar_wait(&full[st], ph, abort_flag);
        if (!ok) break;
        ++loaded;
        tc::fence_after_sync();
        for (int g = 0; g < 2; ++g)
          if (ends[g] > en.step0) issue_s(g, st);
        commit_one(one, &empty[st]);
        advance();
        if (end == en.step0 + 1) commit_one(one, q_empty);
        for (int t = en.step0; ok && t < end; ++t) {
          const bool more = t + 1 < end;
          const int vs = st;
          ok = mbar_wait(&full[vs], ph, abort_flag);
          if (!ok) break;
          advance();
          bool k_ready = false;
          for (int g = 0; g < 2; ++g) {
            if (t >= ends[g]) continue;
            // the first product of a unit overwrites O: the unit before has read it out
            ok = mbar_wait(p_half(g), tiles_g[g] & 1, abort_flag) &&
                 (t > en.step0 || units_g[g] == 0 || mbar_wait(o_free(g), (units_g[g] - 1) & 1, abort_flag));
            if (!ok) break;
            tc::fence_after_sync();
            issue_pv(g, vs, 0, t == en.step0);
            ok = mbar_wait(p_full(g), tiles_g[g] & 1, abort_flag);
            if (!ok) break;
            ++tiles_g[g];
            tc::fence_after_sync();
            issue_pv(g, vs, 1, false);
            if (t + 1 < ends[g]) {
              if (!k_ready) {
                ok = mbar_wait(&full[st], ph, abort_flag);
                if (!ok) break;
                k_ready = true;
                tc::fence_after_sync();
              }
              issue_s(g, st);                    // overwrites P_g(t) after PV_g(t), in issue order
            } else {
              commit_one(one, o_done(g));
              ++units_g[g];
            }
          }
          if (!ok) break;
          commit_one(one, &empty[vs]);
          if (more) {
            commit_one(one, &empty[st]);
            advance();
            if (t + 2 == end) commit_one(one, q_empty);         // the unit's last S was issued
          }
        }
      }
      // every product issued above completes before the tensor memory goes
      commit_one(one, drain);
      mbar_wait_drain(drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    const int g = warp >> 2;                               // query tile
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;                   // tensor-memory lane = row of the tile
    const uint32_t t_lane = tmem + g * kUmmaGroupCols + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t s_col = t_lane + kSCol, p_col = s_col, o_col = t_lane + kOCol;
    const bool negative = prm.qk_scale < 0.f;
    // (never zero, so that a masked -inf stays one: the least float32 times any
    // finite score is no more than 2^-21, whose exponential is 1 to float32)
    const float qk = fmaxf(fabsf(prm.qk_scale), 1.4e-45f);
    const bool wide = (reinterpret_cast<uintptr_t>(prm.out) & 31) == 0;
    const float2 qk2 = make_float2(qk, qk);
    // the row's 128 scores (of -q for a negative scale)
    auto read_scores = [&](uint32_t(&x)[128]) {
      tc::tmem_ld32_at<0>(s_col, x);
      tc::tmem_ld32_at<32>(s_col + 32, x);
      tc::tmem_ld32_at<64>(s_col + 64, x);
      tc::tmem_ld32_at<96>(s_col + 96, x);
      tc::tmem_wait_ld();
      if (negative) {
#pragma unroll
        for (int j = 0; j < 128; ++j) x[j] ^= 0x80000000u;
      }
    };
    // the P written so far may be read by the tensor core
    auto hand_over = [&](uint64_t* bar) {
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int tiles = 0, done = 0, duals = 0;
    bool ok = true;
    for (int r = 0; ok && r < rounds; ++r) {
      const int u = unit_of(r);
      if (u < 0) continue;
      int h;
      const PrefillEntry en = prefill_unit(prm, u, &h);
      const int n0 = chunk_steps(en, 0, G, prm.causal), n1 = chunk_steps(en, 1, G, prm.causal);
      const bool dual = chunk_dual(en, G, max(n0, n1));
      const int tok0 = dual ? 0 : g * 128 / G;          // first token of this group's rows in the unit
      const int tok = tok0 + row / G;                      // token of this row
      const int head = row % G;
      const bool valid = tok < en.ntok;
      const int begin = en.step0 + (dual ? g : 0);
      const int end = en.step0 + (dual ? max(n0, n1) : g ? n1 : n0);
      const int stride = dual ? 2 : 1;
      const int lim_first = prm.causal ? min(en.ctx, en.lim0 + tok0) : en.ctx;
      const int lim = prm.causal ? min(en.ctx, en.lim0 + min(tok, en.ntok - 1)) : en.ctx;
      float m = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      for (int t = begin; t < end; t += stride, ++tiles) {
        if (!__all_sync(0xffffffffu, mbar_wait(s_full(g), tiles & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const bool masked = lim_first < (t + 1) * kStepTokens;          // uniform over the tile
        bool moved = masked || t == begin;                 // the reference maximum may have to move
        if (!moved) {
          // Nothing masked: the weights of the first half are worked out with the
          // maximum as it stands while the step's own maximum is found beside them
          // (different pipes); only if that passes the threshold is this undone.
          uint32_t x[128];
          read_scores(x);
          const float2 nm2 = make_float2(-m, -m);
          float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          float cm[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) cm[k] = fmaxf(__uint_as_float(x[64 + k]), __uint_as_float(x[68 + k]));
          // 32 scores from j0 into 16 packed weights; with `top`, their maximum and
          // that of the 32 scores 64 further on is taken along
          auto weights = [&](auto tag, int j0, uint32_t(&w)[16]) {
            constexpr bool kTop = decltype(tag)::value;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int j = j0 + 2 * i;
              if constexpr (kTop) {
                cm[i & 3] = fmax3(cm[i & 3], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                cm[(i + 2) & 3] = fmax3(cm[(i + 2) & 3], __uint_as_float(x[j + 64]), __uint_as_float(x[j + 65]));
              }
              float2 v = nm2;
              ffma2(v, make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), qk2);
              v.x = exp2_approx(v.x);
              v.y = exp2_approx(v.y);
              w[i] = M::pack(v.x, v.y);
              fadd2(ls[i & 1], v);
            }
          };
          uint32_t w0[16], w1[16];
          weights(std::true_type{}, 0, w0);
          weights(std::true_type{}, 32, w1);
          const float c = fmaxf(fmax3(cm[0], cm[1], cm[2]), cm[3]) * qk;
          moved = __any_sync(0xffffffffu, !(c <= m + kTau && m > -INFINITY));
          if (!moved) {
            tc::tmem_st16(p_col, w0);
            tc::tmem_st16(p_col + 16, w1);
            hand_over(p_half(g));
            weights(std::false_type{}, 64, w0);
            tc::tmem_st16(p_col + 32, w0);
            weights(std::false_type{}, 96, w1);
            tc::tmem_st16(p_col + 48, w1);
            hand_over(p_full(g));
            fadd2(l2, ls[0]);
            fadd2(l2, ls[1]);
          }
        }
        if (moved) {
          // The first steps of a row, and steps with masked tokens: 32 scores at a
          // time, read twice (P over S stays behind the scores still to be read).
          const int nv = lim - t * kStepTokens;            // tokens of this step the row sees
          auto scores = [&](int q, uint32_t(&x)[32]) {
            tc::tmem_ld32(s_col + 32 * q, x);
            tc::tmem_wait_ld();
            if (negative) {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] ^= 0x80000000u;
            }
            if (masked) {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = j < nv - 32 * q ? x[j] : 0xff800000u;
            }
          };
          float ext = -INFINITY;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t x[32];
            scores(q, x);
#pragma unroll
            for (int j = 0; j < 32; j += 2) ext = fmax3(ext, __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
          }
          const float c = ext * qk;
          const float mn = c > m + kTau ? c : m;
          const float f = mn != m ? exp2_approx(m - mn) : 1.f;     // 0 when m was -inf
          if (t > begin && __any_sync(0xffffffffu, mn != m)) {
#pragma unroll 1
            for (int ob = 0; ob < D / 16; ++ob) {
              uint32_t o[16];
              tc::tmem_ld16(o_col + ob * 16, o);
              tc::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tc::tmem_st16(o_col + ob * 16, o);
            }
          }
          l2.x *= f;
          l2.y *= f;
          m = mn;
          const float mu = m == -INFINITY ? 0.f : m;       // nothing visible yet: every weight is 2^-inf
          const float2 nm2 = make_float2(-mu, -mu);
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t x[32], w[16];
            scores(q, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 v = nm2;
              ffma2(v, make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), qk2);
              v.x = exp2_approx(v.x);                      // (exact zeros for masked scores)
              v.y = exp2_approx(v.y);
              w[i] = M::pack(v.x, v.y);
              fadd2(l2, v);
            }
            tc::tmem_st16(p_col + 16 * q, w);
            if (q & 1) hand_over(q == 1 ? p_half(g) : p_full(g));
          }
        }
      }
      if (!ok) break;
      float l = l2.x + l2.y;
      const bool have = end > begin;                       // O holds this unit's product
      if (have) {
        if (!__all_sync(0xffffffffu, mbar_wait(o_done(g), done & 1, abort_flag))) {
          ok = false;
          break;
        }
        ++done;
        tc::fence_after_sync();
      }
      float f0 = 1.f, f1 = 0.f;                            // weights of the two groups' outputs
      if (dual) {
        if (g == 1) {
          s_ml[row] = make_float2(m, l);
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(ml_full);
          continue;                                        // (group 0 reads both and frees both)
        }
        if (!__all_sync(0xffffffffu, mbar_wait(ml_full, duals & 1, abort_flag))) {
          ok = false;
          break;
        }
        ++duals;
        tc::fence_after_sync();
        const float2 other = s_ml[row];
        const float top = fmaxf(m, other.x);
        f0 = l == 0.f ? 0.f : exp2_approx(m - top);
        f1 = other.y == 0.f ? 0.f : exp2_approx(other.x - top);
        l = f0 * l + f1 * other.y;
        m = top;
      }
      const int64_t at = (static_cast<int64_t>(en.slot) * prm.num_kv_heads + h) * kPrefillRows16 +
                         (dual ? 0 : g * 128) + row;
      T* dst = static_cast<T*>(prm.out) +
               (static_cast<int64_t>(en.tok0 + tok) * prm.num_kv_heads * G + h * G + head) * D;
      const float inv = l == 0.f ? 0.f : 1.f / l;          // a row that sees nothing is zero
      if (en.slot >= 0 && valid) prm.part_ml[at] = make_float2(m, l);
#pragma unroll 1
      for (int cb = 0; cb < D / 32; ++cb) {
        uint32_t o[32];
        if (have) {
          tc::tmem_ld32(o_col + cb * 32, o);
          tc::tmem_wait_ld();
          if (dual) {
            uint32_t o1[32];
            tc::tmem_ld32(o_col + kUmmaGroupCols + cb * 32, o1);
            tc::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = __float_as_uint(f0 * __uint_as_float(o[j]) + f1 * __uint_as_float(o1[j]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0u;
        }
        // (no divergence past this iteration: the tensor-memory loads take the whole warp)
        if (valid && en.slot >= 0) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            const uint32_t w[8] = {o[j], o[j + 1], o[j + 2], o[j + 3], o[j + 4], o[j + 5], o[j + 6], o[j + 7]};
            store32(prm.part_acc + at * D + cb * 32 + j, w, true);
          }
        } else if (valid) {
#pragma unroll
          for (int j = 0; j < 32; j += 16) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              w[i] = M::pack(__uint_as_float(o[j + 2 * i]) * inv, __uint_as_float(o[j + 2 * i + 1]) * inv);
            store32(dst + cb * 32 + j, w, wide);
          }
        }
        __syncwarp();
      }
      if (have) {
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(o_free(g));
          if (dual) mbar_arrive(o_free(1));
        }
      }
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kUmmaTmemCols);
  }
}

}  // namespace pa

#endif
