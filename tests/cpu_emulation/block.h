// One CUDA thread block on the CPU: every thread is a fiber, and fibers run in a
// chosen order from one barrier or warp exchange to the next.  Shared memory is
// static, so it holds what the block before left in it, as on the GPU.
#pragma once

#include <ucontext.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <numeric>
#include <random>
#include <vector>

#define __global__
#define __device__
#define __host__
#define __forceinline__ inline
#define __launch_bounds__(...)
#define __align__(n) alignas(n)
#define __shared__ static

using std::max;
using std::min;

struct int4 {
  int x, y, z, w;
};
inline int4 make_int4(int x, int y, int z, int w) { return int4{x, y, z, w}; }

namespace emu {

constexpr size_t kStack = 64 * 1024;

struct Fiber {
  ucontext_t ctx;
  std::vector<char> stack;
  bool done = false;
  int block_gen = 0, warp_gen = 0;
};

struct Warp {
  int gen = 0, arrived = 0;
  unsigned char box[2][32][8];
};

inline std::vector<Fiber> fibers;
inline std::vector<Warp> warps;
inline ucontext_t scheduler;
inline std::function<void()> body;
inline int block_gen = 0, block_arrived = 0, current = 0, device_error = 0;

inline void yield() {
  const int me = current;
  swapcontext(&fibers[me].ctx, &scheduler);
}

inline void trampoline() {
  body();
  fibers[current].done = true;
  swapcontext(&fibers[current].ctx, &scheduler);
}

inline void sync_threads() {
  const int gen = block_gen;
  if (++block_arrived == static_cast<int>(fibers.size())) {
    block_arrived = 0;
    ++block_gen;
    return;
  }
  while (block_gen == gen) yield();
}

// lane `from` of this warp's value
template <typename T>
T exchange(T v, int from) {
  Warp& w = warps[current / 32];
  const int lane = current % 32, gen = w.gen;
  std::memcpy(w.box[gen & 1][lane], &v, sizeof(T));
  if (++w.arrived == 32) {
    w.arrived = 0;
    ++w.gen;
  }
  while (w.gen == gen) yield();
  T r;
  std::memcpy(&r, w.box[gen & 1][from], sizeof(T));
  return r;
}

// Runs `f` on `threads` threads in `order`; false when they wait for one another for good.
inline bool run(int threads, const std::vector<int>& order, std::function<void()> f) {
  body = std::move(f);
  if (static_cast<int>(fibers.size()) != threads) fibers = std::vector<Fiber>(threads);
  warps = std::vector<Warp>(threads / 32);
  block_arrived = 0;
  for (Fiber& x : fibers) {
    x.stack.resize(kStack);
    x.done = false;
    getcontext(&x.ctx);
    x.ctx.uc_stack.ss_sp = x.stack.data();
    x.ctx.uc_stack.ss_size = kStack;
    x.ctx.uc_link = &scheduler;
    makecontext(&x.ctx, trampoline, 0);
  }
  for (int idle = 0, left = threads; left > 0;) {
    const int before_gen = block_gen, before_left = left;
    int warp_gens = 0;
    for (const Warp& w : warps) warp_gens += w.gen;
    for (int i : order) {
      if (fibers[i].done) continue;
      current = i;
      swapcontext(&scheduler, &fibers[i].ctx);
      if (fibers[i].done) --left;
    }
    int after = 0;
    for (const Warp& w : warps) after += w.gen;
    idle = block_gen == before_gen && left == before_left && after == warp_gens ? idle + 1 : 0;
    if (idle > 2) return false;
  }
  return true;
}

inline std::vector<int> order_of(int threads, int kind) {
  std::vector<int> o(threads);
  std::iota(o.begin(), o.end(), 0);
  if (kind == 1) std::reverse(o.begin(), o.end());
  if (kind >= 2) std::shuffle(o.begin(), o.end(), std::mt19937(kind));
  return o;
}

struct ThreadIdx {
  struct X {
    operator int() const { return current; }
  } x;
};

}  // namespace emu

static emu::ThreadIdx threadIdx;

inline void __syncthreads() { emu::sync_threads(); }
template <typename T>
T __shfl_up_sync(unsigned, T v, int d) {
  const int lane = emu::current % 32;
  return emu::exchange(v, lane >= d ? lane - d : lane);
}
template <typename T>
T __shfl_xor_sync(unsigned, T v, int m) {
  const int lane = emu::current % 32;
  return emu::exchange(v, lane ^ m);
}
inline int atomicAdd(int* p, int v) {
  const int r = *p;
  *p += v;
  return r;
}
inline int atomicMax(int* p, int v) {
  const int r = *p;
  *p = max(*p, v);
  return r;
}

namespace pa {
constexpr int DEVERR_BAD_LENGTH = 2;
inline void set_device_error(int code) {
  if (emu::device_error == 0) emu::device_error = code;
}
inline void allow_dependent_launch() {}
inline void wait_prerequisite_grids() {}
}  // namespace pa
