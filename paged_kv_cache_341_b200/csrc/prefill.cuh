// Chunk attention on the CUDA cores: the path of float32 caches (the tensor
// cores take no float32 operands without rounding them).
//
// out[t][h] = sum_j softmax_j(scale q[t][h] . K[j]) V[j] over the context
// tokens j < lim(t), one pass over the context with a running maximum and sum
// per row in float32.
//
// One CTA of 16 x 8 threads takes one unit (prefill_plan.cuh): 32 query rows of
// a KV head and a range of its context, 32 tokens at a time.  Q, K, V and the
// weights P are float32 in shared memory; each thread holds a 4 x 2 piece of
// S = Q K^T (rows 4 ty.., columns tx + 16 j: neighbouring threads read
// neighbouring K rows, whose stride of D + 4 floats keeps 16-byte reads free of
// bank conflicts) and a 4 x D/16 piece of O; the next tile's K and V wait in
// registers.  Bound by the FMA pipe and the shared-memory reads that feed it.
// Small tiles, several CTAs per SM: tiles of 64 rows x 64 tokens with 256
// threads took 10 us each for a handful of rows (4 sequences of up to 45 tokens
// on 300, head_dim 64: 43 us for the kernel, 13 in this form).  With many rows
// the six shared-memory reads for 32 products of a thread set the pace: 512 tokens
// on a 4,096-token context, 32/8 heads, take 1.52 ms (head_dim 128) and 0.80 ms
// (64), 21 and 20 TFLOP/s, 0.28 of the 74 TFLOP/s that 148 SMs multiply and add
// at 1.965 GHz.
#ifndef PAGEDATTN_PREFILL_CUH
#define PAGEDATTN_PREFILL_CUH

#include <cstdint>

#include "decode.cuh"
#include "dtype.cuh"
#include "prefill_plan.cuh"
#include "ptx.cuh"

namespace pa {

constexpr float kLog2e = 1.4426950408889634f;

struct PrefillParams {
  const void* q;                 // [T][Hq][D]
  const void* k_cache;           // [num_blocks][block_size][Hkv][D]
  const void* v_cache;
  const int32_t* block_tables;   // [S][max_blocks]
  const PrefillHeader* header;
  const PrefillEntry* entries;
  float* part_acc;               // [slot][Hkv][rows][D]
  float2* part_ml;               // [slot][Hkv][rows], m in units of log2
  void* out;                     // [T][Hq][D]
  int num_kv_heads, group;
  int max_blocks, block_size, num_blocks;
  int causal;
  float qk_scale;                // scale * log2(e)
};

// Entry of unit u and its KV head; heads of an entry are neighbouring units.
__device__ __forceinline__ PrefillEntry prefill_unit(const PrefillParams& prm, int u, int* head) {
  const int e = u / prm.num_kv_heads;
  *head = u - e * prm.num_kv_heads;
  PrefillEntry r;
  const int4* src = reinterpret_cast<const int4*>(prm.entries + e);
  reinterpret_cast<int4*>(&r)[0] = src[0];
  reinterpret_cast<int4*>(&r)[1] = src[1];
  return r;
}

// Unit of round r of CTA b in a grid of g: the list runs longest first, and the
// CTAs take it forwards and backwards in turn, so that each gets a fair share.
__device__ __forceinline__ long long prefill_snake(int r, int b, int g) {
  return static_cast<long long>(r) * g + (r & 1 ? g - 1 - b : b);
}

constexpr int kPrefillTile32 = 32;               // context tokens per tile
constexpr int kPrefillThreads32 = 4 * kPrefillRows32;

template <int D>
__host__ __device__ constexpr size_t prefill_f32_smem_bytes() {
  return sizeof(float) * (kPrefillRows32 * (D + 4) + kPrefillTile32 * (2 * D + 4) + kPrefillRows32 * (kPrefillTile32 + 4));
}

template <typename T, int D>
__global__ void __launch_bounds__(kPrefillThreads32) prefill_f32_kernel(const PrefillParams prm) {
  constexpr int R = kPrefillRows32, N = kPrefillTile32, LD = D + 4, LP = N + 4, NT = kPrefillThreads32;
  constexpr int J = N / 16;                      // columns of S per thread
  constexpr int E = Chunk<T>::kElems;
  constexpr int CPR = D / E;                     // 16-byte chunks per row
  constexpr int NC = N * CPR / NT;              // chunks of K (and of V) per thread and tile
  constexpr int OC = D / 64;                     // float4 output pieces per thread and row
  extern __shared__ __align__(16) float smem_f[];
  float* s_q = smem_f;
  float* s_k = s_q + R * LD;
  float* s_v = s_k + N * LD;
  float* s_p = s_v + N * D;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int G = prm.group, Hkv = prm.num_kv_heads, BS = prm.block_size;
  allow_dependent_launch();
  wait_prerequisite_grids();
  const long long units = static_cast<long long>(prm.header->num_entries) * Hkv;

  auto widen = [](const void* p, float* o) {
    float2 x[E / 2];
    Chunk<T>::load(p, x);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      o[2 * e] = x[e].x;
      o[2 * e + 1] = x[e].y;
    }
  };

  for (int round = 0;; ++round) {
    const long long u = prefill_snake(round, blockIdx.x, gridDim.x);
    if (static_cast<long long>(round) * gridDim.x >= units) break;
    if (u >= units) continue;
    int h;
    const PrefillEntry en = prefill_unit(prm, static_cast<int>(u), &h);
    const int32_t* table = prm.block_tables + static_cast<int64_t>(en.seq) * prm.max_blocks;
    const int rows = en.ntok * G;
    __syncthreads();                             // the previous unit's readers of shared memory
    for (int i = tid; i < R * CPR; i += NT) {
      const int r = i / CPR, c = i % CPR;
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = 0.f;
      if (r < rows)
        widen(static_cast<const T*>(prm.q) +
                  (static_cast<int64_t>(en.tok0 + r / G) * Hkv * G + h * G + r % G) * D + c * E, x);
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(s_q + r * LD + c * E + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
    }
    float m[4], l[4];
    int lim[4];
    float4 o[4][OC];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      const int tok = min(4 * ty + i, rows - 1) / G;
      lim[i] = prm.causal ? min(en.ctx, en.lim0 + tok) : en.ctx;
#pragma unroll
      for (int c = 0; c < OC; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int tok_lo = en.step0 * kStepTokens;
    const int tok_hi = min(en.ctx, en.step1 * kStepTokens);
    // the next tile's chunks, read into registers while this one is worked on:
    // first the blocks, then K and V, all in flight together
    uint4 rk[NC], rv[NC];
    auto fetch = [&](int t0) {
      int64_t at[NC];
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int i = tid + NT * k, r = i / CPR, c = i % CPR, tok = t0 + r;
        at[k] = -1;
        if (tok < tok_hi) {
          const int b = tok / BS, phys = table[b];
          if (phys < 0 || phys >= prm.num_blocks)
            set_device_error(DEVERR_BAD_BLOCK_ID);
          else
            at[k] = ((static_cast<int64_t>(phys) * BS + (tok - b * BS)) * Hkv + h) * D + c * E;
        }
      }
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        rk[k] = rv[k] = make_uint4(0, 0, 0, 0);
        if (at[k] >= 0) {
          rk[k] = *reinterpret_cast<const uint4*>(static_cast<const T*>(prm.k_cache) + at[k]);
          rv[k] = *reinterpret_cast<const uint4*>(static_cast<const T*>(prm.v_cache) + at[k]);
        }
      }
    };
    if (tok_lo < tok_hi) fetch(tok_lo);
    for (int t0 = tok_lo; t0 < tok_hi; t0 += N) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NC; ++k) {
        const int i = tid + NT * k, r = i / CPR, c = i % CPR;
        float x[E], y[E];
        widen(&rk[k], x);
        widen(&rv[k], y);
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          *reinterpret_cast<float4*>(s_k + r * LD + c * E + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          *reinterpret_cast<float4*>(s_v + r * D + c * E + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
        }
      }
      __syncthreads();
      if (t0 + N < tok_hi) fetch(t0 + N);
      float s[4][J];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 a[4], b[J];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(s_q + (4 * ty + i) * LD + d);
#pragma unroll
        for (int j = 0; j < J; ++j) b[j] = *reinterpret_cast<const float4*>(s_k + (tx + 16 * j) * LD + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < J; ++j)
            s[i][j] = fmaf(a[i].w, b[j].w, fmaf(a[i].z, b[j].z, fmaf(a[i].y, b[j].y, fmaf(a[i].x, b[j].x, s[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float c = -INFINITY;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          s[i][j] = t0 + tx + 16 * j < lim[i] ? s[i][j] * prm.qk_scale : -INFINITY;
          c = fmaxf(c, s[i][j]);
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, w));
        const float mn = fmaxf(m[i], c);
        const float mu = mn == -INFINITY ? 0.f : mn;     // nothing visible yet: every weight is 2^-inf
        const float f = exp2f(m[i] - mu);
        m[i] = mn;
        l[i] *= f;
#pragma unroll
        for (int k = 0; k < OC; ++k) {
          o[i][k].x *= f;
          o[i][k].y *= f;
          o[i][k].z *= f;
          o[i][k].w *= f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float w = exp2f(s[i][j] - mu);
          l[i] += w;
          s_p[(4 * ty + i) * LP + tx + 16 * j] = w;
        }
      }
      __syncwarp();                              // (a row of P is written and read by the same warp)
#pragma unroll 2
      for (int j = 0; j < N; j += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(s_p + (4 * ty + i) * LP + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
          for (int k = 0; k < OC; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(s_v + (j + jj) * D + tx * 4 + 64 * k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = jj == 0 ? w[i].x : jj == 1 ? w[i].y : jj == 2 ? w[i].z : w[i].w;
              o[i][k].x = fmaf(x, v.x, o[i][k].x);
              o[i][k].y = fmaf(x, v.y, o[i][k].y);
              o[i][k].z = fmaf(x, v.z, o[i][k].z);
              o[i][k].w = fmaf(x, v.w, o[i][k].w);
            }
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
      const int r = 4 * ty + i;
      if (r >= rows) continue;
      if (en.slot >= 0) {
        const int64_t at = (static_cast<int64_t>(en.slot) * Hkv + h) * R + r;
        if (tx == 0) prm.part_ml[at] = make_float2(m[i], l[i]);
#pragma unroll
        for (int k = 0; k < OC; ++k) *reinterpret_cast<float4*>(prm.part_acc + at * D + tx * 4 + 64 * k) = o[i][k];
      } else {
        // (a NaN sum stays NaN; a row that sees nothing is zero)
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        T* dst = static_cast<T*>(prm.out) +
                 (static_cast<int64_t>(en.tok0 + r / G) * Hkv * G + h * G + r % G) * D + tx * 4;
#pragma unroll
        for (int k = 0; k < OC; ++k) {
          dst[64 * k] = static_cast<T>(o[i][k].x * inv);
          dst[64 * k + 1] = static_cast<T>(o[i][k].y * inv);
          dst[64 * k + 2] = static_cast<T>(o[i][k].z * inv);
          dst[64 * k + 3] = static_cast<T>(o[i][k].w * inv);
        }
      }
    }
  }
}

}  // namespace pa

#endif
