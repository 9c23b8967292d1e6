// Cache kernels of a chunk of new tokens (HBM-bound): rotary positions fused
// with the append of K/V into their slots, and the move of whole blocks in
// every layer's cache with the rewrite of the block tables.
#ifndef PAGEDATTN_CHUNK_OPS_CUH
#define PAGEDATTN_CHUNK_OPS_CUH

#include <cstdint>

#include "dtype.cuh"
#include "ptx.cuh"

namespace pa {

// More codes of the device error word (the first five are in ptx.cuh).
constexpr int DEVERR_BAD_AXIS = 6;     // axis of a rotary pair outside the positions (axis 0 used)
constexpr int DEVERR_MOVE_ORDER = 7;   // sources of a move list not in increasing order

struct RopeParams {
  const void* q;                 // [T] rows of Hq heads, q_stride elements apart
  const void* k_new;             // [T] rows of Hkv heads, k_stride elements apart
  const void* v_new;
  const int32_t* positions;      // [axes][T]
  const float* inv_freq;         // [half]
  const int32_t* pair_axis;      // [half], or nullptr (all axis 0)
  const int64_t* slots;          // [T]
  void* q_out;                   // [T][Hq][D]
  void* k_cache;
  void* v_cache;
  int64_t q_stride, k_stride, v_stride;
  int64_t num_slots;
  int num_tokens, num_axes, half;              // half = rotated pairs per head
  int num_q_heads, num_kv_heads, head_dim;
};

// Small CTAs with few loads per thread keep more of them in flight: 16,384 tokens
// of 32/8 heads of 128 (bf16) take 66.9 us in a captured graph with 64 threads of
// two items (6.02 TB/s), 75.6 with 128 of three, 90 with 256 of two; a call among
// others takes 69.9 us (5.77 TB/s).
constexpr int kRopeThreads = 64;
constexpr int kRopeMaxHalf = 256;              // pairs a CTA's table holds (head_dim up to 512)

// One pair turned by the angle whose (cos, sin) is cs.
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float x = a, y = b;
  a = x * cs.x - y * cs.y;
  b = y * cs.x + x * cs.y;
}

// Rotary positions + append: for every token t and pair i the angle is
// positions[axis(i)][t] * inv_freq[i]; q goes to q_out and k to its slot with
// every head's pairs turned by it, v to its slot unchanged.
//
// Bound by HBM: each row of q, k and v is read and written once.  A CTA takes
// one token (blockIdx.x) and a share of its heads (blockIdx.y: few tokens are
// spread over more CTAs); the angles are worked out once per CTA, while the
// first rows of q, k and v are on their way.  The angle is held in turns in
// 64 bits (position x frequency has up to 55 significant bits, and far
// positions lose all of their low ones in 32), reduced to [-1/2, 1/2] there
// and handed to sincospif in 32 bits.  The pairs are turned in 32 bits and
// rounded once.
//
// kVec: 16-byte chunks.  An item is two chunks of one head: the elements i..
// and their partners i + half.. (or, interleaved, 2i.. of neighbouring pairs),
// so a thread that reads an item writes the same elements and q_out may be q.
// Otherwise (the rotated width does not fill chunks) a thread takes one pair
// of elements at a time: the same tokens with 90 of 128 elements turned take 246
// us (interleaved 239), 1.64 TB/s, bound by loads and stores of 2 bytes; with 64
// turned, which fill chunks, 65.9 us.
template <typename T, bool kInterleaved, bool kVec>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams prm) {
  __shared__ float2 s_cs[kRopeMaxHalf];
  constexpr int E = Chunk<T>::kElems;
  const int t = blockIdx.x;
  const int D = prm.head_dim, half = prm.half, rot = 2 * half;
  const int heads = prm.num_q_heads + 2 * prm.num_kv_heads;
  allow_dependent_launch();
  wait_prerequisite_grids();
  const int64_t slot = prm.slots[t];
  const bool keep = slot >= 0 && slot < prm.num_slots;
  if (slot >= prm.num_slots && threadIdx.x == 0 && blockIdx.y == 0) set_device_error(DEVERR_BAD_SLOT);

  // source and destination rows of one head; false when the head is not written
  auto rows_of = [&](int h, const T** src, T** dst) {
    if (h < prm.num_q_heads) {
      *src = static_cast<const T*>(prm.q) + t * prm.q_stride + static_cast<int64_t>(h) * D;
      *dst = static_cast<T*>(prm.q_out) + (static_cast<int64_t>(t) * prm.num_q_heads + h) * D;
      return true;
    }
    h -= prm.num_q_heads;
    const bool is_v = h >= prm.num_kv_heads;
    if (is_v) h -= prm.num_kv_heads;
    const int64_t at = (slot * prm.num_kv_heads + h) * D;
    *src = (is_v ? static_cast<const T*>(prm.v_new) + t * prm.v_stride
                 : static_cast<const T*>(prm.k_new) + t * prm.k_stride) + static_cast<int64_t>(h) * D;
    *dst = static_cast<T*>(is_v ? prm.v_cache : prm.k_cache) + at;
    return keep;
  };
  auto angles = [&]() {
    for (int i = threadIdx.x; i < half; i += kRopeThreads) {
      int axis = prm.pair_axis ? prm.pair_axis[i] : 0;
      if (axis < 0 || axis >= prm.num_axes) {
        set_device_error(DEVERR_BAD_AXIS);
        axis = 0;
      }
      const double p = static_cast<double>(prm.positions[static_cast<int64_t>(axis) * prm.num_tokens + t]);
      const double turns = p * static_cast<double>(prm.inv_freq[i]) * 0.15915494309189533577;   // / (2 pi)
      const float r = static_cast<float>(turns - rint(turns));
      float2 cs;
      sincospif(2.f * r, &cs.y, &cs.x);
      s_cs[i] = cs;
    }
    __syncthreads();
  };

  if constexpr (kVec) {
    constexpr int kRound = 2;                  // items in flight per thread
    const int per_head = D / (2 * E);          // items of a head: D is a multiple of 2 chunks
    const int rot_items = rot / (2 * E);
    // (a value head's items, and those behind the rotated width, are copies)
    const int total = heads * per_head;
    const int step = kRopeThreads * gridDim.y;
    bool first = true;
    for (int base = blockIdx.y * kRopeThreads + threadIdx.x; first || base < total; base += kRound * step) {
      uint4 a[kRound], b[kRound];
      T* pa_[kRound];
      T* pb_[kRound];
      int pair[kRound];
      bool w[kRound];
#pragma unroll
      for (int r = 0; r < kRound; ++r) {
        const int item = base + r * step;
        w[r] = false;
        if (item < total) {
          const int h = item / per_head, j = item - h * per_head;
          const T* src;
          T* dst;
          const bool kept = rows_of(h, &src, &dst);
          w[r] = true;
          const bool turned = j < rot_items && h < prm.num_q_heads + prm.num_kv_heads;
          const int oa = turned && !kInterleaved ? j * E : j * 2 * E;
          const int ob = turned && !kInterleaved ? oa + half : oa + E;
          pair[r] = turned ? j * E : -1;
          // (read whatever the slot is: the reads do not wait for it)
          a[r] = *reinterpret_cast<const uint4*>(src + oa);
          b[r] = *reinterpret_cast<const uint4*>(src + ob);
          pa_[r] = kept ? dst + oa : nullptr;
          pb_[r] = dst + ob;
        }
      }
      if (first) angles();
      first = false;
#pragma unroll
      for (int r = 0; r < kRound; ++r) {
        if (!w[r] || pa_[r] == nullptr) continue;
        if (pair[r] >= 0) {
          float2 x[E / 2], y[E / 2];
          Chunk<T>::load(&a[r], x);
          Chunk<T>::load(&b[r], y);
          const float2* cs = s_cs + pair[r];
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            if constexpr (kInterleaved) {      // (2i, 2i + 1): E / 2 pairs in each chunk
              turn(x[e].x, x[e].y, cs[e]);
              turn(y[e].x, y[e].y, cs[E / 2 + e]);
            } else {
              turn(x[e].x, y[e].x, cs[2 * e]);
              turn(x[e].y, y[e].y, cs[2 * e + 1]);
            }
          }
          Chunk<T>::store(&a[r], x);
          Chunk<T>::store(&b[r], y);
        }
        *reinterpret_cast<uint4*>(pa_[r]) = a[r];
        *reinterpret_cast<uint4*>(pb_[r]) = b[r];
      }
    }
  } else {
    angles();
    // items of a head: its pairs, then the single elements behind them
    const int per_head = half + (D - rot);
    const int total = heads * per_head;
    for (int item = blockIdx.y * kRopeThreads + threadIdx.x; item < total; item += kRopeThreads * gridDim.y) {
      const int h = item / per_head, j = item - h * per_head;
      const T* src;
      T* dst;
      if (!rows_of(h, &src, &dst)) continue;
      if (j >= half) {
        dst[rot + j - half] = src[rot + j - half];
        continue;
      }
      const int oa = kInterleaved ? 2 * j : j, ob = kInterleaved ? 2 * j + 1 : j + half;
      if (h >= prm.num_q_heads + prm.num_kv_heads) {
        dst[oa] = src[oa];
        dst[ob] = src[ob];
        continue;
      }
      float x = static_cast<float>(src[oa]), y = static_cast<float>(src[ob]);
      turn(x, y, s_cs[j]);
      dst[oa] = static_cast<T>(x);
      dst[ob] = static_cast<T>(y);
    }
  }
}

// ---- block moves ------------------------------------------------------------

constexpr int kMoveMaxLayers = 64;             // layers of one launch (their pointers are kernel arguments)
constexpr int kMoveThreads = 256;
constexpr int kMoveVecs = 4;                   // 16-byte chunks in flight per thread
constexpr int kMoveSliceVecs = kMoveThreads * kMoveVecs;   // 16 KB of a block per CTA
constexpr int kRemapEntries = kMoveThreads * 4;            // table entries per CTA

struct MoveParams {
  uint4* cache[2 * kMoveMaxLayers];            // K of layer 0.., then V of layer 0..
  const int2* moves;                           // (source, destination), sources increasing
  int32_t* tables;
  int64_t table_entries;
  int64_t copy_ctas;                           // CTAs that copy; the rest rewrite table entries
  int num_caches, num_moves, num_blocks, block_vecs, slices;
  int table_cols, table_stride;
};

// Copies block moves[i].x to block moves[i].y in every cache, and rewrites each
// table entry that names a source.  Bound by HBM (every byte read and written
// once): a CTA copies one 16 KB slice with all of its loads in flight before
// the first store, one launch covers every layer, and the table entries are
// looked up in the (sorted) list by bisection in CTAs of their own behind the
// copies.
__global__ void __launch_bounds__(kMoveThreads) move_blocks_kernel(const __grid_constant__ MoveParams prm) {
  const int64_t cta = blockIdx.x;
  if (cta < prm.copy_ctas) {
    // caches outermost, so that neighbouring CTAs read neighbouring slices of one block
    const int slice = static_cast<int>(cta % prm.slices);
    const int64_t rest = cta / prm.slices;
    const int i = static_cast<int>(rest % prm.num_moves);
    const int c = static_cast<int>(rest / prm.num_moves);
    const int2 mv = prm.moves[i];
    if (mv.x < 0 || mv.x >= prm.num_blocks || mv.y < 0 || mv.y >= prm.num_blocks) {
      if (threadIdx.x == 0) set_device_error(DEVERR_BAD_PAIR);
      return;
    }
    if (c == 0 && slice == 0 && threadIdx.x == 0 && i > 0 && prm.moves[i - 1].x >= mv.x)
      set_device_error(DEVERR_MOVE_ORDER);
    uint4* base = prm.cache[c];
    const uint4* src = base + static_cast<int64_t>(mv.x) * prm.block_vecs;
    uint4* dst = base + static_cast<int64_t>(mv.y) * prm.block_vecs;
    const int begin = slice * kMoveSliceVecs + threadIdx.x;
    uint4 v[kMoveVecs];
#pragma unroll
    for (int k = 0; k < kMoveVecs; ++k) {
      const int j = begin + k * kMoveThreads;
      if (j < prm.block_vecs) v[k] = src[j];
    }
#pragma unroll
    for (int k = 0; k < kMoveVecs; ++k) {
      const int j = begin + k * kMoveThreads;
      if (j < prm.block_vecs) dst[j] = v[k];
    }
    return;
  }
  const int64_t base = (cta - prm.copy_ctas) * kRemapEntries + threadIdx.x;
#pragma unroll
  for (int k = 0; k < kRemapEntries / kMoveThreads; ++k) {
    const int64_t e = base + k * kMoveThreads;
    if (e >= prm.table_entries) return;
    int32_t* p = prm.tables + e / prm.table_cols * prm.table_stride + e % prm.table_cols;
    const int32_t id = *p;
    int lo = 0, hi = prm.num_moves;             // first source >= id
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (prm.moves[mid].x < id) lo = mid + 1;
      else hi = mid;
    }
    if (lo < prm.num_moves) {
      const int2 mv = prm.moves[lo];
      if (mv.x == id && mv.y >= 0 && mv.y < prm.num_blocks) *p = mv.y;
    }
  }
}

}  // namespace pa

#endif
