// Geometry of sliding-window attention, shared by its forward, backward and decode kernels.
//
// Query t sees key j iff j <= t and (t - j < W or j < ns): the last W tokens and the first ns ones
// (the sinks).  A run of queries t0 .. t1 of one sequence therefore needs the keys [0, ns) and
// [t0 - W + 1, t1].  They are walked as one virtual sequence of 128-key tiles: the sinks rounded up
// to a multiple of eight (nsp; eight rows are one swizzle atom of a tile), then the window's keys
// from wherever they start.  So the sinks share a tile with the first window keys instead of taking
// 128-key blocks of their own, and the window starts at the tile row where it has to.  Where the
// two ranges meet, the walk is simply 0 .. t1.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace msa {

struct KeyRun {
  int ws;   // first key of the window part
  int nsp;  // virtual rows of the sink part (0: the parts meet, the walk starts at key 0)
  int len;  // virtual keys
  int nb;   // 128-key tiles
};
__device__ __forceinline__ KeyRun key_run(const WinDims& d, int t0, int t1) {
  KeyRun r;
  r.ws = t0 - d.W + 1 > 0 ? t0 - d.W + 1 : 0;
  r.nsp = d.nsp;
  if (r.ws <= r.nsp) r.ws = r.nsp = 0;
  r.len = r.nsp + t1 + 1 - r.ws;
  r.nb = (r.len + kBlock - 1) / kBlock;
  return r;
}

// Visible columns of tile n for query t: bit c of word c / 32 of `m`.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi, int q) {  // columns lo .. hi of word q
  const int a = lo - 32 * q > 0 ? lo - 32 * q : 0, z = hi - 32 * q < 31 ? hi - 32 * q : 31;
  return a > z ? 0u : (0xffffffffu >> (31 - z)) & (0xffffffffu << a);
}
__device__ __forceinline__ void visible_cols(const WinDims& d, const KeyRun& r, int n, int t,
                                             uint32_t (&m)[4]) {
  const int v0 = n * kBlock;
  const int sc = (t + 1 < d.ns ? t + 1 : d.ns) - v0;  // sink keys: columns 0 .. sc - 1
  int lo = t - d.W + 1 - r.ws + r.nsp;                // window keys
  if (lo < r.nsp) lo = r.nsp;
  const int hi = t - r.ws + r.nsp;
#pragma unroll
  for (int q = 0; q < 4; ++q) m[q] = bit_range(0, sc - 1, q) | bit_range(lo - v0, hi - v0, q);
}

// Tensor maps of K or V [B, S, Hkv, 128]: boxes of a whole tile's rows, of the sink rows of a tile
// shared by both parts, and of that tile's window rows.
struct KeyMaps {
  CUtensorMap full, sink, rest;
};
bool make_key_maps(const WinDims& d, const void* base, KeyMaps* m);  // win_fwd.cu

__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* tm, int col, int head,
                                              int row, int b, uint64_t* mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3, %4, %5}], [%6];\n" ::"r"(smem_u32(dst)),
      "l"(tm), "r"(col), "r"(head), "r"(row), "r"(b), "r"(smem_u32(mbar))
      : "memory");
}
__device__ __forceinline__ void tma_store_rows(const CUtensorMap* tm, uint32_t src, int col, int head,
                                               int row, int b) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];\n" ::"l"(tm),
      "r"(col), "r"(head), "r"(row), "r"(b), "r"(src)
      : "memory");
}
__device__ __forceinline__ void bulk_store_commit() {
  asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
}
__device__ __forceinline__ void bulk_store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
  asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
}

// Tile n of a key run into dst (two SW128 panels of 128 rows); rows past the sequence are zeros.
// The barrier has been told to expect the whole tile.
__device__ __forceinline__ void load_key_tile(uint8_t* dst, const KeyMaps& m, const KeyRun& r, int n,
                                              int head, int b, uint64_t* mbar) {
  constexpr int kPanel = kBlock * 128;
  const int v0 = n * kBlock;
  if (v0 >= r.nsp || v0 + kBlock <= r.nsp) {
    const int row = v0 >= r.nsp ? r.ws + v0 - r.nsp : v0;
    tma_load_rows(dst, &m.full, 0, head, row, b, mbar);
    tma_load_rows(dst + kPanel, &m.full, 64, head, row, b, mbar);
  } else {
    const int a = r.nsp - v0;  // = nsp mod 128, the box height of m.sink; a multiple of eight
    tma_load_rows(dst, &m.sink, 0, head, v0, b, mbar);
    tma_load_rows(dst + kPanel, &m.sink, 64, head, v0, b, mbar);
    tma_load_rows(dst + a * 128, &m.rest, 0, head, r.ws, b, mbar);
    tma_load_rows(dst + kPanel + a * 128, &m.rest, 64, head, r.ws, b, mbar);
  }
}

__device__ __forceinline__ uint32_t phase_of(long long k) { return (uint32_t)(k & 1); }
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace msa
