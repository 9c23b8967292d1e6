// Host-side launch of the chunk attention kernels (included by pa_device.cu
// only): workspace layout, tensor maps, and the planner / attention / merge
// sequence.
#ifndef PAGEDATTN_LAUNCH_PREFILL_CUH
#define PAGEDATTN_LAUNCH_PREFILL_CUH

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <string>

#include "launch_decode.cuh"
#include "prefill.cuh"
#include "prefill_plan.cuh"
#include "prefill_tc.cuh"

namespace {

struct PrefillArgs {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  int num_blocks;
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* context_lens;
  const int32_t* q_starts;
  int T, S, Hq, Hkv, D, BS;
  float scale;
  int causal;
  void* workspace;
  void* out;
  cudaStream_t stream;
};

// The plan is made for at most this many CTAs, so that the workspace size is a
// function of the arguments alone (a B200 has 148 SMs); the grid of the 16-bit
// kernel, one CTA per SM, is bounded by it too.
constexpr int kPrefillMaxCtas = 148;

// Workspace: [header 256 B][tile ends][tile steps][entries][merges][partial (m, l)][partial outputs].
// There is room for kSplitUnits pieces of 256 rows per CTA (over all heads); the planner leaves contexts whole rather than take more.
struct PrefillLayout {
  size_t ends, steps, entries, merges, ml, acc, total;
  int max_tiles, max_entries, max_merges, max_slots;
};

PrefillLayout prefill_layout(long long T, long long S, long long Hq, long long Hkv, long long D, long long cap,
                             int rows) {
  const long long G = Hq / Hkv;
  const long long tiles = std::min(T, S) + T * G / rows;                  // every non-empty chunk may end in a part tile
  const long long steps = (cap + pa::kStepTokens - 1) / pa::kStepTokens;
  const long long room = static_cast<long long>(pa::kSplitUnits) * kPrefillMaxCtas * (pa::kPrefillRows16 / rows);
  const long long pieces = std::min(room / Hkv, tiles * steps);
  const pa::PlanCost& cost = rows == pa::kPrefillRows16 ? pa::kPlanCost16 : pa::kPlanCost32;
  const bool split = steps > cost.min_steps && pieces >= 2;
  PrefillLayout L;
  L.max_tiles = static_cast<int>(tiles);
  L.max_slots = split ? static_cast<int>(pieces) : 0;
  L.max_merges = L.max_slots / 2;                                         // a split context has two pieces at least
  L.max_entries = L.max_tiles + L.max_slots;
  L.ends = 256;
  L.steps = L.ends + round256(static_cast<size_t>(S) * sizeof(int));
  L.entries = L.steps + round256(static_cast<size_t>(L.max_tiles) * sizeof(int));
  L.merges = L.entries + round256(static_cast<size_t>(L.max_entries) * sizeof(pa::PrefillEntry));
  L.ml = L.merges + round256(static_cast<size_t>(L.max_merges) * sizeof(pa::PrefillMerge));
  const size_t slot_rows = static_cast<size_t>(L.max_slots) * Hkv * rows;
  L.acc = L.ml + round256(slot_rows * sizeof(float2));
  L.total = L.acc + round256(slot_rows * D * sizeof(float));
  return L;
}

// One cache viewed as [Hkv][rows / 8][D / 64 panels][8 rows][64 elements] (the
// last index fastest), 128-byte swizzled, box (64, 8, D / 64, piece / 8, 1): a
// piece of `piece` tokens of one head lands as 1024-byte atoms of 8 tokens x 64
// elements, the panels of 8 tokens behind one another.
template <typename T>
pa_status make_piece_map(CUtensorMap* map, const void* base, int D, int Hkv, long long rows, int piece) {
  auto encode = tensor_map_encoder();
  if (!encode) return pa::fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(Hkv) * D * sizeof(T);
  const cuuint64_t dims[5] = {64, 8, static_cast<cuuint64_t>(D / 64), static_cast<cuuint64_t>(rows / 8),
                              static_cast<cuuint64_t>(Hkv)};
  const cuuint64_t strides[4] = {row_bytes, 128, 8 * row_bytes, static_cast<cuuint64_t>(D) * sizeof(T)};
  const cuuint32_t box[5] = {64, 8, static_cast<cuuint32_t>(D / 64), static_cast<cuuint32_t>(piece / 8), 1};
  const cuuint32_t elem_strides[5] = {1, 1, 1, 1, 1};
  CUresult r = encode(map, map_type<T>(), 5, const_cast<void*>(base), dims, strides, box, elem_strides,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return pa::fail(PA_ERR_CUDA, "cuTensorMapEncodeTiled (cache pieces) failed (" + std::to_string(r) + ")");
  return PA_OK;
}

// The largest power of two that divides the block size, at most a step: pieces
// of that many tokens never cross a block, and fill a step exactly.
int piece_tokens(int block_size) { return std::min(block_size & -block_size, pa::kStepTokens); }

template <typename T, int D>
pa_status launch_prefill(const PrefillArgs& a) {
  DeviceInfo dev;
  pa_status st = device_info(&dev);
  if (st != PA_OK) return st;
  constexpr bool kTensor = sizeof(T) == 2;
  constexpr int kRows = kTensor ? pa::kPrefillRows16 : pa::kPrefillRows32;
  const PrefillLayout L = prefill_layout(a.T, a.S, a.Hq, a.Hkv, a.D, static_cast<long long>(a.max_blocks) * a.BS, kRows);
  char* ws = static_cast<char*>(a.workspace);

  pa::PrefillParams prm;
  prm.q = a.q;
  prm.k_cache = a.k_cache;
  prm.v_cache = a.v_cache;
  prm.block_tables = a.block_tables;
  prm.header = reinterpret_cast<const pa::PrefillHeader*>(ws);
  prm.entries = reinterpret_cast<const pa::PrefillEntry*>(ws + L.entries);
  prm.part_ml = reinterpret_cast<float2*>(ws + L.ml);
  prm.part_acc = reinterpret_cast<float*>(ws + L.acc);
  prm.out = a.out;
  prm.num_kv_heads = a.Hkv;
  prm.group = a.Hq / a.Hkv;
  prm.max_blocks = a.max_blocks;
  prm.block_size = a.BS;
  prm.num_blocks = a.num_blocks;
  prm.causal = a.causal;
  prm.qk_scale = a.scale * pa::kLog2e;

  // every kernel is a programmatic dependent of the one before it: it is set up
  // early, and reads nothing before its wait
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = a.stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;

  pa::PrefillPlanParams pp;
  pp.q_starts = a.q_starts;
  pp.context_lens = a.context_lens;
  pp.header = reinterpret_cast<pa::PrefillHeader*>(ws);
  pp.tile_ends = reinterpret_cast<int*>(ws + L.ends);
  pp.entries = reinterpret_cast<pa::PrefillEntry*>(ws + L.entries);
  pp.merges = reinterpret_cast<pa::PrefillMerge*>(ws + L.merges);
  pp.num_seqs = a.S;
  pp.num_tokens = a.T;
  pp.num_kv_heads = a.Hkv;
  pp.group = prm.group;
  pp.rows = kRows;
  pp.causal = a.causal;
  pp.cap = a.max_blocks * a.BS;
  pp.ctas = std::min(dev.sms, kPrefillMaxCtas);
  pp.max_tiles = L.max_tiles;
  pp.cost = kTensor ? pa::kPlanCost16 : pa::kPlanCost32;
  pp.tile_steps = reinterpret_cast<int*>(ws + L.steps);
  pp.max_merges = L.max_merges;
  pp.max_slots = L.max_slots;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(pa::kPrefillPlanThreads);
  cudaError_t e = cudaLaunchKernelEx(&cfg, pa::prefill_plan_kernel, pp);
  if (e != cudaSuccess) return cuda_fail(e, "prefill_plan_kernel launch");

  const long long units = static_cast<long long>(L.max_entries) * a.Hkv;
  if constexpr (kTensor) {
    const size_t smem = pa::prefill_umma_smem_bytes<D>();
    auto kern = pa::prefill_umma_kernel<T, D>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(prefill umma)");
    CUtensorMap tm_k, tm_v, tm_q;
    const int piece = piece_tokens(a.BS);
    const long long rows = static_cast<long long>(a.num_blocks) * a.BS;
    st = make_piece_map<T>(&tm_k, a.k_cache, D, a.Hkv, rows, piece);
    if (st != PA_OK) return st;
    st = make_piece_map<T>(&tm_v, a.v_cache, D, a.Hkv, rows, piece);
    if (st != PA_OK) return st;
    st = make_query_map<T>(&tm_q, a.q, a.T, a.Hq, D, prm.group);
    if (st != PA_OK) return st;
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(units, pp.ctas)));
    cfg.blockDim = dim3(pa::kChunkThreads);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, tm_q, prm, piece);
    if (e != cudaSuccess) return cuda_fail(e, "prefill_umma_kernel launch");
  } else {
    const size_t smem = pa::prefill_f32_smem_bytes<D>();
    auto kern = pa::prefill_f32_kernel<T, D>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(prefill f32)");
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, pa::kPrefillThreads32, smem);
    if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor(prefill f32)");
    if (per_sm < 1) return pa::fail(PA_ERR_UNSUPPORTED, "pa_prefill_attention: kernel does not fit on an SM");
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(units, static_cast<long long>(per_sm) * dev.sms)));
    cfg.blockDim = dim3(pa::kPrefillThreads32);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, kern, prm);
    if (e != cudaSuccess) return cuda_fail(e, "prefill_f32_kernel launch");
  }

  if (L.max_merges > 0) {
    pa::PrefillMergeParams mp;
    mp.header = prm.header;
    mp.merges = pp.merges;
    mp.part_acc = prm.part_acc;
    mp.part_ml = prm.part_ml;
    mp.out = a.out;
    mp.num_kv_heads = a.Hkv;
    mp.group = prm.group;
    mp.rows = kRows;
    const long long rows = static_cast<long long>(L.max_merges) * a.Hkv * kRows;
    const long long need = (rows + pa::kPrefillMergeWarps - 1) / pa::kPrefillMergeWarps;
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(need, 8ll * dev.sms)));
    cfg.blockDim = dim3(pa::kPrefillMergeWarps * 32);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, pa::prefill_merge_kernel<T, D>, mp);
    if (e != cudaSuccess) return cuda_fail(e, "prefill_merge_kernel launch");
  }
  return pa::ok();
}

template <typename T>
pa_status dispatch_prefill(const PrefillArgs& a) {
  switch (a.D) {
    case 64: return launch_prefill<T, 64>(a);
    case 128: return launch_prefill<T, 128>(a);
    default: return pa::fail(PA_ERR_UNSUPPORTED, "pa_prefill_attention: head_dim must be 64 or 128");
  }
}

}  // namespace

#endif
