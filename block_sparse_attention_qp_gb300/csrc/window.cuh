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

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace msa {

struct KeyRun {
  int ws;   // first key of the window part
  int nsp;  // virtual rows of the sink part (0: the parts meet, the walk starts at key 0)
  int len;  // virtual keys
  int nb;   // 128-key tiles
  __device__ __forceinline__ int keys(int n) const { return len - n * kBlock; }  // of tile n and behind
  int f0, f1;  // tiles f0 .. f1 (none if f0 > f1) are seen whole by every query of the run
};
__device__ __forceinline__ KeyRun key_run(const WinDims& d, int t0, int t1) {
  KeyRun r;
  r.ws = t0 - d.W + 1 > 0 ? t0 - d.W + 1 : 0;
  r.nsp = d.nsp;
  if (r.ws <= r.nsp) r.ws = r.nsp = 0;
  r.len = r.nsp + t1 + 1 - r.ws;
  r.nb = (r.len + kBlock - 1) / kBlock;
  const int off = r.nsp - r.ws;  // virtual position of a window key: key + off
  const int lo = t1 - d.W + 1 + off > r.nsp ? t1 - d.W + 1 + off : r.nsp;  // first key of the last query
  r.f0 = (lo + kBlock - 1) / kBlock;
  r.f1 = (t0 + off + 1) / kBlock - 1;
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

// Tensor maps of K or V [B, S, Hkv, 128]: boxes of a whole tile's rows (head: of sinks only), of the sink
// rows of a tile shared by both parts, and of that tile's window rows.
struct KeyMaps {
  CUtensorMap full, head, sink, rest;
};
bool make_key_maps(const WinDims& d, const void* base, KeyMaps* m);  // win_fwd.cu

// The status area is cleared by the first block of the call's first kernel that uses it (in the backward
// win_dq_kernel, behind the row data) instead of a memset in front of it: a flag another block sets (a wait that gave up) is set 200 ms later at the earliest.
__device__ __forceinline__ void clear_status(unsigned* status) {
  if (blockIdx.x == 0 && threadIdx.x < 32) status[threadIdx.x] = 0u;
}

// Lets a kernel use `bytes` of dynamic shared memory: once per kernel and device (the attribute
// belongs to the device's context; a repeated call costs a microsecond of every launch).
template <auto* Kernel>
void allow_smem(size_t bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return;
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return;
  if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess)
    done.fetch_or(bit, std::memory_order_relaxed);
}

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

// Tile n of a key run into dst (two SW128 panels of 128 rows); rows past the sequence, and past the
// sinks in their part, are zeros.
// The barrier has been told to expect the whole tile.
__device__ __forceinline__ void load_key_tile(uint8_t* dst, const KeyMaps& m, const KeyRun& r, int n,
                                              int head, int b, uint64_t* mbar) {
  constexpr int kPanel = kBlock * 128;
  const int v0 = n * kBlock;
  if (v0 >= r.nsp || v0 + kBlock <= r.nsp) {
    const CUtensorMap* tm = v0 >= r.nsp ? &m.full : &m.head;
    const int row = v0 >= r.nsp ? r.ws + v0 - r.nsp : v0;
    tma_load_rows(dst, tm, 0, head, row, b, mbar);
    tma_load_rows(dst + kPanel, tm, 64, head, row, b, mbar);
  } else {
    const int a = r.nsp - v0;  // = nsp mod 128, the box height of m.sink; a multiple of eight
    tma_load_rows(dst, &m.sink, 0, head, v0, b, mbar);
    tma_load_rows(dst + kPanel, &m.sink, 64, head, v0, b, mbar);
    tma_load_rows(dst + a * 128, &m.rest, 0, head, r.ws, b, mbar);
    tma_load_rows(dst + kPanel + a * 128, &m.rest, 64, head, r.ws, b, mbar);
  }
}

// One 128 x 128 x 128 product is eight tcgen05.mma of K = 16.  One thread issues every product of a
// block, so the instructions between two MMAs count: issued by "lane 0" of a divergent branch, with a
// descriptor built for each, an MMA took 83 cycles alone and about 120 beside the softmax warps,
// whatever its N up to 128; the tensor core needs 64.  So the whole warp runs the issue code converged
// and elect.sync inside the instruction sequence picks the thread (the same one every time), which
// keeps the operands in uniform registers; the descriptors' upper half is one constant and each step
// adds a constant to the lower half (all tiles are 128 rows: a K-major operand moves 32 bytes a step
// and to its second panel after four, an MN-major one 16 rows).  64 to 67 cycles an MMA, measured
// with one block per SM on GB300.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride 1024, version, SW128
__device__ __forceinline__ uint32_t desc_lo_k(uint32_t tile) { return (tile >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_lo_mn(uint32_t tile) { return (tile >> 4) | ((128u * 128u >> 4) << 16); }
__device__ __forceinline__ constexpr uint32_t step_k(int ks) { return (ks >> 2) * (128 * 128 >> 4) + (ks & 3) * 2; }
__device__ __forceinline__ constexpr uint32_t step_mn(int ks) { return ks * (16 * 128 >> 4); }
__device__ __forceinline__ void warp_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 da, db;\n.reg .b32 el;\nsetp.ne.b32 p, %4, 0;\n"
      "mov.b64 da, {%1, %5};\nmov.b64 db, {%2, %5};\nelect.sync el|q, 0xffffffff;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void warp_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n.reg .pred p, q;\n.reg .b64 db;\n.reg .b32 el;\nsetp.ne.b32 p, %4, 0;\n"
      "mov.b64 db, {%2, %5};\nelect.sync el|q, 0xffffffff;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(kDescHi)
      : "memory");
}
// Arrive on an mbarrier once every MMA the warp issued so far has completed.
__device__ __forceinline__ void warp_mma_commit(uint64_t* mbar) {
  asm volatile(
      "{\n.reg .pred q;\n.reg .b32 el;\nelect.sync el|q, 0xffffffff;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(mbar))
      : "memory");
}
// D (+)= A B^T, both K-major tiles in shared memory.
__device__ __forceinline__ void mma_kk(uint32_t d, uint32_t a_tile, uint32_t b_tile, bool acc) {
  constexpr uint32_t id = sm100::idesc_bf16(128, 128, false, false);
  const uint32_t a = desc_lo_k(a_tile), b = desc_lo_k(b_tile);
  warp_mma_ss(d, a, b, id, acc);
#pragma unroll
  for (int ks = 1; ks < 8; ++ks) warp_mma_ss(d, a + step_k(ks), b + step_k(ks), id, true);
}
// D (+)= A B, A a K-major, B an MN-major tile in shared memory.
__device__ __forceinline__ void mma_kn(uint32_t d, uint32_t a_tile, uint32_t b_tile, bool acc) {
  constexpr uint32_t id = sm100::idesc_bf16(128, 128, false, true);
  const uint32_t a = desc_lo_k(a_tile), b = desc_lo_mn(b_tile);
  warp_mma_ss(d, a, b, id, acc);
#pragma unroll
  for (int ks = 1; ks < 8; ++ks) warp_mma_ss(d, a + step_k(ks), b + step_mn(ks), id, true);
}
// D (+)= A B, A in tensor memory (16 K values are 8 columns; runs of kRun steps start kPitch columns
// apart), B an MN-major tile in shared memory.
template <int kRun, int kPitch>
__device__ __forceinline__ void mma_tn(uint32_t d, uint32_t a, uint32_t b_tile, bool acc) {
  constexpr uint32_t id = sm100::idesc_bf16(128, 128, false, true);
  const uint32_t b = desc_lo_mn(b_tile);
  warp_mma_ts(d, a, b, id, acc);
#pragma unroll
  for (int ks = 1; ks < 8; ++ks)
    warp_mma_ts(d, a + (ks / kRun) * kPitch + (ks % kRun) * 8, b + step_mn(ks), id, true);
}
// The same for a tile of `keys` < 128: N of the scores and K of the other product rounded up to 16.
// (A run's keys seldom fill its last tile: at window 512 and 8 heads a group 23 or 39 of 128.)
__device__ __forceinline__ void mma_kk_part(uint32_t d, uint32_t a_tile, uint32_t b_tile, int keys) {
  constexpr uint32_t id = sm100::idesc_bf16(128, 0, false, false);
  const uint32_t a = desc_lo_k(a_tile), b = desc_lo_k(b_tile), idn = id | (uint32_t)((keys + 15) / 16 * 2) << 17;
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) warp_mma_ss(d, a + step_k(ks), b + step_k(ks), idn, ks > 0);
}
template <int kRun, int kPitch>
__device__ __forceinline__ void mma_tn_part(uint32_t d, uint32_t a, uint32_t b_tile, bool acc, int keys) {
  constexpr uint32_t id = sm100::idesc_bf16(128, 128, false, true);
  const uint32_t b = desc_lo_mn(b_tile);
  warp_mma_ts(d, a, b, id, acc);
#pragma unroll
  for (int ks = 1; ks < 8; ++ks)
    if (16 * ks < keys) warp_mma_ts(d, a + (ks / kRun) * kPitch + (ks % kRun) * 8, b + step_mn(ks), id, true);
}
// This thread's warp number, as a value the compiler knows to be the same in the whole warp.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xffffffffu, threadIdx.x / 32, 0); }

// Position in a ring of N slots: the slot and the phase of its barriers' current use.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t phase = 0;
  bool wrapped = false;  // the slot has been used before (its empty barrier has to be waited for)
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1;
      wrapped = true;
    }
  }
};

// Named barrier over `n` threads that also ORs a predicate across them.
__device__ __forceinline__ bool bar_or(int id, int n, bool p) {
  uint32_t r;
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %3, 0;\nbar.red.or.pred q, %1, %2, p;\nselp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((int)p)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t phase_of(long long k) { return (uint32_t)(k & 1); }
__device__ __forceinline__ float exp2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace msa
