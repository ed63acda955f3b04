// Attention of single new tokens over caches in 4 bits (format: q4.cuh), and the rows of such a cache as bf16.
//
// A block takes one sequence and attention group (the up to 16 query heads that share a KV head and see the same keys) and
// a run of the group's 128-key tiles: those of a window and the first tokens, or the key blocks that the
// proxy selected.  With codes c, scales s and the rows' exponents e (K) and f (V):
//   S[j, h] = 2^e_j sum_d (s c)[j, d] q[h, d]          x = scale log2(e) S,  masked keys -inf
//   m_h >= max_j (x + f) - 8,  l_h = sum_j 2^(x - m),  O[h, :] = sum_j 2^(x + f - m) (s c)[j, :] / l_h
// The exponents of V are folded into the weights, and the products' V operand s c is exact in fp16, as K's is; q, its head's
// largest element brought to 2^14 by a power of two, is exact there down to 2^-31 of that element, and off by at most 2^-39 of it
// below (to 1 instead: 2^-17, 2^-25).  The other roundings are those of the weights to fp16 and of O.  m is a whole number and the
// weights are taken 2^7 times as large: at most 2^15, the largest at least 2^6, so that they keep 11 bits down to 2^-20 of the
// largest of their warp's keys and are off by at most 2^-31 of it below.  (With the largest kept as 1, 16384 keys of 2^-26 of the first
// one's weight lost a quarter of what they add to O: all of those of the first one's warp.)
//
// Bound by memory, 73 bytes a key, head and tensor (bf16: 256), as long as the codes become operands with few
// instructions: 47 values a cycle and SM at 7 TB/s.  So no operand passes through shared memory as 16-bit values:
// the raw blocks arrive there by bulk copies, and each thread turns what it needs into fragments of warp-level
// products (m16n8k16, fp16, fp32 sums) in registers, K^T and V^T as the 16-row operands, the heads as the 8 columns.
// (As tiles for tcgen05 they would be written to and read from shared memory at 512 bytes a key, four times
// what its bandwidth allows at this rate; the tensor work itself is small, 2 x 8 products for 16 keys.)
// Which dims and keys a fragment's places stand for is free as long as both operands agree, so that
//   K: a thread's 32 values of a row are 32 consecutive dims, one 16-byte load and two scales;
//   V: a thread's 16 values of a row are one scale's dims, one 8-byte load; keys are dealt such that 32 lanes
//      read consecutive bytes, and the score rows are dealt alike.
// A tile's four warps take 32 keys each with sums of their own, joined at the end; a fifth keeps a ring of tiles
// loading.  Few (sequence, group) pairs or long ones: their tiles are split over blocks and joined by a second kernel.
//
// A call of a replayed graph of 20, 64 / 8 heads, us.  One wave of resident blocks over 16384 keys each (456 pairs): 188, 5.8 TB/s,
// 0.85 of a copy; 128 sequences of 4096 keys (2.25 waves): 122, 5.0 TB/s (118 in their order, launch_q4); the same with
// lengths of 2048 to 4096: 98, 4.8 TB/s (110 in their order); one sequence of 65536 keys: 23 with its join (alone, caches cold, 23
// and 8); 64 sequences of 4096 keys and 16 heads a group (twice the products and weights): 105; 32 sequences with 16 of 64
// blocks selected, 256 pairs on 152 SMs: 25, 2.8 TB/s (alone, cold).  340 instructions a run of 16 keys are issued in
// 66 % of the cycles; the pipes are busy at half that or less.  Measured on the way (128 sequences of 4096, among single calls): codes by
// shifts and masks and keys paired by byte permutations 260 us (660 instructions); both as below 149; tile data by the
// loading warp, full tiles without masks 123.  Tried and not kept: four blocks an SM with three stages (123) or with more
// (156, spills); the P of even and odd dims as two halves of the 16 rows, half of the multiplications and 24 instead of 16
// products (130); two chains of K products (121); the tiles of all pairs dealt out evenly (134 and 16 of joining).
#include <math.h>

#include <type_traits>

#include "q4.cuh"
#include "window.cuh"

namespace msa {
namespace {

constexpr int kStages = 4;
constexpr int kStageBytes = 2 * kQ4Block;  // K, V
constexpr int kQ4Threads = 160;            // warps 0-3 products, 4 loads
constexpr int kSorted = 512, kSteps = 16;  // sequences that are sorted by length at most, and steps of it
// log2 of the largest weight when the maximum is moved, and of how much larger one may be without moving it: 2^15 in all,
// within fp16.
constexpr float kLift = 7.f, kSlack = 8.f;
// The row sum is kept in units of 2^(m + kSlack + kShift), m the maximum of x + f.  A key of zero values adds 2^(100 + m) to it
// (f = -100), one of a row that no call has written, zero bytes, 2^(127 + m), and 2^23 of them have to stay in range.  At the
// other end, f = 90, the heaviest key adds 2^(m - 90), 2^-116 units: keys of a 2^10-th of its weight still count, and of a 2^24-th
// where V's rows are below 2^83.  The shift is free: x is made by a multiply-add, and V's exponent has an offset as it is.
constexpr float kShift = 18.f;

struct Q4Args {
  const uint8_t *k, *v;
  const bf16* q;
  const int32_t* seq_len;
  const int32_t* list;  // [B][Hp][top_k] key blocks; NULL: window and sinks
  bf16* o;
  float* lse;
  float *opart, *lpart;  // [split][B][Hq][128], [split][B][Hq] (log2 units)
  unsigned* status;
  int B, cap, blocks, Hq, Hkv, Hp, groups, G;
  int W, ns, top_k;
  float scale;
  int nsplit, tiles;
  bool own_status;  // this kernel writes the status word
  float steps;      // sorted by length: kSteps / tiles of the longest possible
};
struct Q4Tile {
  int block, r0, r1;  // rows r0 .. r1 - 1 of the block hold every visible key
  int full;           // and all 128 are
};
struct Q4Shared {
  uint64_t full[kStages], empty[kStages];
  Q4Tile tile[kStages];
  float m[4][16], l[4][16];
};
// The tiles of a sequence of n keys.
struct Q4Walk {
  int t, ws, ns, sink_tiles, first, count;
};
__device__ __forceinline__ Q4Walk q4_walk(const Q4Args& A, int n) {
  Q4Walk w;
  w.t = n - 1;
  const int last = w.t / kBlock;
  if (A.list) {
    w.ws = w.ns = w.sink_tiles = w.first = 0;
    w.count = min(A.top_k, last + 1);
    return w;
  }
  w.ws = max(0, n - A.W);
  w.ns = min(A.ns, w.ws);
  w.first = w.ws / kBlock;
  w.sink_tiles = min((w.ns + kBlock - 1) / kBlock, w.first);
  w.count = w.sink_tiles + last - w.first + 1;
  return w;
}
__device__ __forceinline__ Q4Tile q4_tile(const Q4Args& A, const Q4Walk& w, int listed, int i) {
  Q4Tile x;
  if (A.list) {
    x.block = listed;
    x.r0 = 0;
    if (x.block < 0 || x.block > w.t / kBlock) x.block = -1;  // (msa_decode's selection has none)
  } else {
    x.block = i < w.sink_tiles ? i : w.first + i - w.sink_tiles;
    x.r0 = x.block * kBlock < w.ns ? 0 : max(0, w.ws - x.block * kBlock);
  }
  x.r1 = i < w.sink_tiles ? w.ns - x.block * kBlock : w.t + 1 - x.block * kBlock;
  x.r1 = x.block < 0 ? 0 : min(kBlock, x.r1);
  x.full = x.r0 == 0 && x.r1 == kBlock && x.block * kBlock >= w.ws;
  return x;
}
// The sequence at place `at` when they are sorted by their tiles, most first, in kSteps steps and in order within one: every warp
// finds it for itself, the step bit by bit by ballots.  (Loops of few instructions: unrolled they cost more than they do, in
// fetching them.)
__device__ __forceinline__ int q4_by_length(const Q4Args& A, int at, uint8_t* step) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x % 32, chunks = (A.B + 31) / 32;
#pragma unroll 1
  for (int b = threadIdx.x; b < 32 * chunks; b += kQ4Threads) {
    const int n = b < A.B ? __ldg(A.seq_len + b) : 0;
    const int tiles = n < 1 || n > A.cap ? 0 : q4_walk(A, n).count;
    step[b] = b < A.B ? kSteps - 1 - min(kSteps - 1, (int)((float)tiles * A.steps)) : kSteps;
  }
  __syncthreads();
  int t = 0, behind = at;
#pragma unroll 1
  for (int bit = kSteps / 2; bit > 0; bit >>= 1) {
    int n = 0;  // in steps before t + bit
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) n += __popc(__ballot_sync(kAll, step[32 * c + lane] < t + bit));
    if (n <= at) {
      t += bit;
      behind = at - n;
    }
  }
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    const bool here = step[32 * c + lane] == t;
    const unsigned all = __ballot_sync(kAll, here);
    const unsigned hit = __ballot_sync(kAll, here && __popc(all & ((1u << lane) - 1u)) == behind);
    if (hit) return 32 * c + __ffs(hit) - 1;
    behind -= __popc(all);
  }
  return 0;  // (not reached)
}
__device__ __forceinline__ bool q4_visible(const Q4Walk& w, int j) { return j <= w.t && (j >= w.ws || j < w.ns); }

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // of an 8 x 8 matrix of 16-bit values
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Half kHalf of x times s (s, 0) plus that of y times t (0, t): no rounding.
template <int kHalf>
__device__ __forceinline__ uint32_t pair_of(uint32_t x, uint32_t s, uint32_t y, uint32_t t) {
  const __half2 hx = *reinterpret_cast<const __half2*>(&x), hy = *reinterpret_cast<const __half2*>(&y);
  const __half2 r = __hfma2(kHalf ? __high2half2(hy) : __low2half2(hy), *reinterpret_cast<const __half2*>(&t),
                            __hmul2(kHalf ? __high2half2(hx) : __low2half2(hx), *reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace

// NT: runs of eight heads.
template <int NT, bool kSort>
__global__ void __launch_bounds__(kQ4Threads, NT == 1 ? 3 : 2) q4_decode_kernel(const __grid_constant__ Q4Args A) {
  using namespace sm100;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ Q4Shared sh;
  __shared__ uint8_t step[kSort ? kSorted : 1];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int split = blockIdx.x % A.nsplit, bg = blockIdx.x / A.nsplit;
  const int grp = bg % A.groups;
  int b = bg / A.groups;
  if constexpr (kSort) b = __reduce_max_sync(0xffffffffu, q4_by_length(A, b, step));  // (a uniform register again)
  let_next();
  if (tid / 32 == 4) wait_before();  // (the selected blocks; all else is older)
  if (A.own_status && blockIdx.x == 0) {  // the status word whole: clear, or a length out of range
    int bad = 0;
    for (int x = tid; x < A.B; x += kQ4Threads) bad |= A.seq_len[x] < 1 || A.seq_len[x] > A.cap;
    bad = __syncthreads_or(bad);
    if (tid < 32) A.status[tid] = tid == 0 && bad ? kStatusBadIndex : 0u;
  }
  const int len = A.seq_len[b];
  if (len < 1 || len > A.cap) return;
  const Q4Walk w = q4_walk(A, len);
  const int n0 = split * A.tiles, ntile = min(A.tiles, w.count - n0);
  const long long row0 = (long long)b * A.Hq + (long long)grp * A.G;  // first query head of the group
  const long long part0 = (long long)split * A.B * A.Hq + row0;
  if (ntile <= 0) {  // a sequence with fewer tiles than the longest possible
    if (tid < A.G) A.lpart[part0 + tid] = -INFINITY;
    return;
  }
  const int32_t* list = A.list ? A.list + ((long long)b * A.Hp + (long long)grp * A.Hp / A.groups) * A.top_k : nullptr;
  if (tid == 0) {
    for (int x = 0; x < kStages; ++x) {
      mbar_init(&sh.full[x], 1);
      mbar_init(&sh.empty[x], 4);
    }
    mbar_fence_init();
  }
  __syncthreads();

  if (warp == 4) {
    // ---------------------------------------------------------------- loads
    // (the selected blocks first, two a lane: read one by one they cost their latency at every tile)
    const int at0 = n0 + lane, at1 = at0 + 32;
    const int e0 = list && at0 < w.count ? __ldcg(list + at0) : -1, e1 = list && at1 < w.count ? __ldcg(list + at1) : -1;
    const long long head = ((long long)b * A.Hkv + (long long)grp * A.Hkv / A.groups) * A.blocks;
    int i = 0;
    for (; i < ntile; ++i) {
      const int s = i % kStages;
      if (i >= kStages && !mbar_wait_warp(&sh.empty[s], phase_of(i / kStages - 1), A.status)) break;
      const Q4Tile x = q4_tile(A, w, __shfl_sync(0xffffffffu, i < 32 ? e0 : e1, i & 31), n0 + i);
      // rows in units of 16: every piece then starts and ends on 16 bytes
      const int r0 = x.r0 & ~15, rows = (x.r1 + 15 & ~15) - r0;
      const long long at = (head + max(x.block, 0)) * (long long)kQ4Block;
      uint8_t* dst = ring + s * kStageBytes;
      if (lane == 0) {
        sh.tile[s] = x;
        mbar_expect_tx(&sh.full[s], 2 * rows * (kQ4Codes + kQ4Scales + 1));
        if (rows == kBlock) {
          bulk_load(dst, A.k + at, kQ4Block, &sh.full[s]);
          bulk_load(dst + kQ4Block, A.v + at, kQ4Block, &sh.full[s]);
        } else if (rows > 0) {
          for (int y = 0; y < 2; ++y) {
            const uint8_t* src = (y ? A.v : A.k) + at;
            uint8_t* to = dst + y * kQ4Block;
            bulk_load(to + r0 * kQ4Codes, src + r0 * kQ4Codes, rows * kQ4Codes, &sh.full[s]);
            bulk_load(to + kQ4ScaleAt + r0 * kQ4Scales, src + kQ4ScaleAt + r0 * kQ4Scales, rows * kQ4Scales, &sh.full[s]);
            bulk_load(to + kQ4ExpAt + r0, src + kQ4ExpAt + r0, rows, &sh.full[s]);
          }
        }
      }
      __syncwarp();
    }
    // no copy may still be landing when the block exits
    for (int x = i > kStages ? i - kStages : 0; x < i; ++x) mbar_wait_warp(&sh.full[x % kStages], phase_of(x / kStages), A.status);
  }
  const int g = lane >> 2, q4 = lane & 3;
  float m[NT][2], top[NT][2], l[NT][2], acc[NT][8][4];  // m: the maximum less kLift; top: the maximum and kSlack
  if (warp < 4) {
    // ---------------------------------------------------------------- queries: column g of run y, dims 32 q4 ..
    uint32_t qf[NT][8][2];
    float qs[NT][2];  // scale log2(e) 2^f of heads 2 q4, 2 q4 + 1
#pragma unroll
    for (int y = 0; y < NT; ++y) {
      const int h = 8 * y + g;
      uint4 v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[c] = h < A.G ? __ldg(reinterpret_cast<const uint4*>(A.q + (row0 + h) * kD + 32 * q4) + c) : make_uint4(0u, 0u, 0u, 0u);
      uint32_t big = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        big = __vmaxu2(big, q4_top(v[c]));
      big = max(big & 0xffffu, big >> 16);
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // the head's largest element to 2^14 .. 2^15 (pow2f: -126 .. 127)
      const int f = max((int)(big >> 7) - 127 - 14, -126);
      const float down = pow2f(-f), up = A.scale * kLog2e * pow2f(f);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t wd[4] = {v[ks >> 1].x, v[ks >> 1].y, v[ks >> 1].z, v[ks >> 1].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t u = wd[2 * (ks & 1) + e];
          qf[y][ks][e] = pack_half(__uint_as_float(u << 16) * down, __uint_as_float(u & 0xffff0000u) * down);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qs[y][e] = __shfl_sync(0xffffffffu, up, 4 * (2 * q4 + e));
        m[y][e] = top[y][e] = -INFINITY;
        l[y][e] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[y][mt][e] = 0.f;
    }
    const int krow = 4 * (g & 1) + (g >> 1);  // key of score row g of a run of 16; row g + 8: 8 more
    // Two runs of 16 keys, rows r0 .. r0 + 31 of a tile; kFull: every key of the tile is visible.
    auto keys32 = [&](auto full, const uint8_t* sk, int r0, int block) {
      constexpr bool kFull = decltype(full)::value;
      const uint8_t* sv = sk + kQ4Block;
      float x2[2][NT][4], xv[2][NT][4];  // scores of two runs of 16 keys, less kShift, and with V's exponent
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int ra = r0 + 16 * c + krow, rb = ra + 8;
        const uint4 ka = *reinterpret_cast<const uint4*>(sk + ra * kQ4Codes + 16 * q4);
        const uint4 kb = *reinterpret_cast<const uint4*>(sk + rb * kQ4Codes + 16 * q4);
        const uint32_t fa = q4_scales(*reinterpret_cast<const uint16_t*>(sk + kQ4ScaleAt + ra * kQ4Scales + 2 * q4));
        const uint32_t fb = q4_scales(*reinterpret_cast<const uint16_t*>(sk + kQ4ScaleAt + rb * kQ4Scales + 2 * q4));
        const uint32_t fa0 = __byte_perm(fa, 0, 0x1010), fa1 = __byte_perm(fa, 0, 0x3232);
        const uint32_t fb0 = __byte_perm(fb, 0, 0x1010), fb1 = __byte_perm(fb, 0, 0x3232);
        float sc[NT][4];
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int k2 = 0; k2 < 4; ++k2) {  // two steps of 16 dims
          uint32_t ca[4], cb[4];
          q4_codes(wa[k2], ca);
          q4_codes(wb[k2], cb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ca[e] = hmul2(ca[e], k2 < 2 ? fa0 : fa1);
            cb[e] = hmul2(cb[e], k2 < 2 ? fb0 : fb1);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int y = 0; y < NT; ++y) {
              const uint32_t b0 = qf[y][2 * k2 + e][0], b1 = qf[y][2 * k2 + e][1];
              if (k2 + e == 0) mma16816_first(sc[y], ca[0], cb[0], ca[1], cb[1], b0, b1);
              else mma16816(sc[y], ca[2 * e], cb[2 * e], ca[2 * e + 1], cb[2 * e + 1], b0, b1);
            }
        }
        const float ea = __uint_as_float((uint32_t)sk[kQ4ExpAt + ra] << 23), eb = __uint_as_float((uint32_t)sk[kQ4ExpAt + rb] << 23);
        const float va = (float)((int)sv[kQ4ExpAt + ra] - 127 + (int)kShift), vb = (float)((int)sv[kQ4ExpAt + rb] - 127 + (int)kShift);
        const bool vis_a = kFull || q4_visible(w, block * kBlock + ra), vis_b = kFull || q4_visible(w, block * kBlock + rb);
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool vis = e < 2 ? vis_a : vis_b;
            const float z = fmaf(sc[y][e], (e < 2 ? ea : eb) * qs[y][e & 1], -kShift);
            x2[c][y][e] = vis ? z : -INFINITY;
            xv[c][y][e] = vis ? z + (e < 2 ? va : vb) : -INFINITY;
          }
      }
      // ---- the running maxima, moved only where a weight would pass 2^15
      bool up = false;
#pragma unroll
      for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          up |= fmax3(xv[0][y][e], xv[0][y][e + 2], fmaxf(xv[1][y][e], xv[1][y][e + 2])) > top[y][e];
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int y = 0; y < NT; ++y)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmax3(xv[0][y][e], xv[0][y][e + 2], fmaxf(xv[1][y][e], xv[1][y][e + 2]));
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            mx = fmaxf(ceilf(mx) - kLift, m[y][e]);
            // 2^(m - mx) as a square: V's exponents, -100 to 90, can move m by more than 126 at once, and the row sum,
            // which leaves them out, may still be large by as much: taken in two steps it is not flushed.  (0 at the first keys)
            const float root = mx == m[y][e] ? 1.f : exp2_ftz(0.5f * (m[y][e] - mx)), alpha = root * root;
            m[y][e] = mx;
            top[y][e] = mx + kLift + kSlack;
            l[y][e] = l[y][e] * root * root;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              acc[y][mt][e] *= alpha;
              acc[y][mt][e + 2] *= alpha;
            }
          }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int y = 0; y < NT; ++y) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool none = !kFull && m[y][e & 1] == -INFINITY;
            l[y][e & 1] += exp2_ftz(x2[c][y][e] - (none ? 0.f : top[y][e & 1]));
            p[e] = exp2_ftz(xv[c][y][e] - (none ? 0.f : m[y][e & 1]));
          }
          pb[y][0] = transpose8(pack_half(p[0], p[1]));
          pb[y][1] = transpose8(pack_half(p[2], p[3]));
        }
        // ---- V: keys 4 i + q4 of the run, dims 16 g .. 16 g + 15
        uint2 v[4];
        uint32_t fs[4];  // of even keys (s, 0), of odd ones (0, s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = r0 + 16 * c + 4 * e + q4;
          v[e] = *reinterpret_cast<const uint2*>(sv + r * kQ4Codes + 8 * g);
          uint32_t sb = sv[kQ4ScaleAt + r * kQ4Scales + g];
          if (!kFull && !q4_visible(w, block * kBlock + r)) sb = 0;  // whatever an unseen row holds
          fs[e] = q4_scales(e & 1 ? sb << 8 : sb);
        }
        // Pairs of keys from pairs of dims: the transposition is in the scales' products (a pair of keys is
        // (s, 0) d + (0, s') d'), on the pipe that has room.  (With byte permutations the conversions' pipe had 79 %
        // of its slots taken at a third of the bandwidth.)
#pragma unroll
        for (int m4 = 0; m4 < 2; ++m4) {
          uint32_t c4[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) q4_codes(m4 ? v[e].y : v[e].x, c4[e]);
#pragma unroll
          for (int mm = 0; mm < 4; ++mm) {
            const uint32_t a0 = pair_of<0>(c4[0][mm], fs[0], c4[1][mm], fs[1]), a1 = pair_of<1>(c4[0][mm], fs[0], c4[1][mm], fs[1]);
            const uint32_t a2 = pair_of<0>(c4[2][mm], fs[2], c4[3][mm], fs[3]), a3 = pair_of<1>(c4[2][mm], fs[2], c4[3][mm], fs[3]);
#pragma unroll
            for (int y = 0; y < NT; ++y) mma16816(acc[y][4 * m4 + mm], a0, a1, a2, a3, pb[y][0], pb[y][1]);
          }
        }
      }
    };
    int s = 0;
    uint32_t phase = 0;
    const int r0 = 32 * warp;
    for (int i = 0; i < ntile; ++i) {
      if (!mbar_wait_warp(&sh.full[s], phase, A.status)) break;
      const Q4Tile x = sh.tile[s];
      const uint8_t* sk = ring + s * kStageBytes;
      if (x.full) keys32(std::true_type{}, sk, r0, x.block);
      else if (r0 < x.r1 && r0 + 32 > x.r0) keys32(std::false_type{}, sk, r0, x.block);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[s]);
      if (++s == kStages) {
        s = 0;
        phase ^= 1;
      }
    }
#pragma unroll
    for (int y = 0; y < NT; ++y)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[y][e] += __shfl_xor_sync(0xffffffffu, l[y][e], off);
        if (g == 0) {
          sh.m[warp][8 * y + 2 * q4 + e] = m[y][e];
          sh.l[warp][8 * y + 2 * q4 + e] = l[y][e];
        }
      }
  }
  // ---- the warps' sums: [warp][head][128 dims] over the ring, which every copy has reached and every warp has read
  __syncthreads();
  float* sums = reinterpret_cast<float*>(ring);
  if (warp < 4) {
#pragma unroll
    for (int y = 0; y < NT; ++y)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* to = sums + ((warp * NT * 8) + 8 * y + 2 * q4 + e) * kD + 16 * g;
#pragma unroll
        for (int mt = 0; mt < 8; mt += 2)
          *reinterpret_cast<float4*>(to + 2 * mt) = make_float4(acc[y][mt][e], acc[y][mt][e + 2], acc[y][mt + 1][e], acc[y][mt + 1][e + 2]);
      }
  }
  __syncthreads();
  if (tid < kD) {
    for (int h = 0; h < A.G; ++h) {
      const float mx = fmaxf(fmaxf(sh.m[0][h], sh.m[1][h]), fmaxf(sh.m[2][h], sh.m[3][h]));
      float sum = 0.f, y = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float root = sh.m[k][h] == -INFINITY ? 0.f : exp2_ftz(0.5f * (sh.m[k][h] - mx));  // (as above)
        sum = fmaf(root * sh.l[k][h], root, sum);
        y = fmaf(root * root, sums[(k * NT * 8 + h) * kD + tid], y);
      }
      y = y * exp2f(-kLift - kSlack - kShift) / sum;  // (the sum itself may be too large for the factor)
      const float ls = mx + kLift + kSlack + kShift + log2f(sum);
      if (A.nsplit == 1) {
        A.o[(row0 + h) * kD + tid] = __float2bfloat16_rn(y);
        if (tid == 0) A.lse[row0 + h] = ls * kLn2;
      } else {
        A.opart[(part0 + h) * kD + tid] = y;
        if (tid == 0) A.lpart[part0 + h] = ls;
      }
    }
  }
}

// Rows first .. first + count - 1 of every sequence and head as the bf16 values they stand for.  A warp takes 16 tokens of
// a head, which lie together in the cache: four at a time, 8 lanes a row, all loads before the first store.
__global__ void __launch_bounds__(256) q4_read_kernel(const uint8_t* cache, int H, int blocks, int first, int count, long long units, bf16* out) {
  const int lane = threadIdx.x % 32, l8 = lane & 7, runs = (count + 15) / 16;
  for (long long u = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / 32; u < units; u += (long long)gridDim.x * blockDim.x / 32) {
    const int h = (int)(u % H), n0 = (int)(u / H % runs) * 16 + (lane >> 3);
    const long long b = u / H / runs;
    uint2 code[4];
    uint32_t sb[4], eb[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int n = first + min(n0 + 4 * k, count - 1), row = n % kBlock;
      const uint8_t* block = cache + ((b * H + h) * blocks + n / kBlock) * (long long)kQ4Block;
      code[k] = __ldg(reinterpret_cast<const uint2*>(block + row * kQ4Codes + 8 * l8));
      sb[k] = __ldg(block + kQ4ScaleAt + row * kQ4Scales + l8);
      eb[k] = __ldg(block + kQ4ExpAt + row);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t s2 = q4_scales(sb[k]);
      const float s = __half2float(*reinterpret_cast<const __half*>(&s2)) * __uint_as_float(eb[k] << 23);
      uint32_t w[2][4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t c[4];
        q4_codes(x ? code[k].y : code[k].x, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&c[i]));
          w[x][i] = pack_bf16(f.x * s, f.y * s);  // exact
        }
      }
      if (n0 + 4 * k >= count) continue;
      uint4* to = reinterpret_cast<uint4*>(out + ((b * count + n0 + 4 * k) * H + h) * kD) + 2 * l8;
      to[0] = make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
      to[1] = make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
    }
  }
}

void launch_q4_read(const void* cache, int B, int H, int cap, int first, int count, void* out, cudaStream_t st) {
  const long long units = (long long)B * ((count + 15) / 16) * H, g = (units + 7) / 8, most = (long long)num_sms() * 16;
  q4_read_kernel<<<(int)(g < most ? g : most), 256, 0, st>>>((const uint8_t*)cache, H, cap / kBlock, first, count, units, (bf16*)out);
}

// Splits of a pair's tiles: as many as fill the resident blocks, of at least four tiles (a part's start, end and share of
// the join cost about as much as three).  Where several sequences share the blocks, up to four times as many of 32 tiles:
// one wave of parts as long as the longest sequence's leaves blocks idle beside it, and lengths are known on the device
// only.  One wave / parts of 32, us (as above), all of the capacity, of 1 .. capacity, most of them short, 64 / 8 heads: 40
// sequences of 8192 97 / 93, 66 / 58, 54 / 37; of 16384 188 / 157, 145 / 103, 99 / 63; 16 of 65536 251 / 228,
// 245 / 148, 201 / 110; 8 of 65536 116 / 123, 115 / 97, 101 / 58: what it loses is 7 % where a few sequences are all full.
// (Among single calls, of 48 tiles the second line's last is 94 for 65, twice as many parts at most the third's second 198 for
// 167; with more pairs than blocks 64 of 8192 106 for 85.)
WinSplit q4_split(int B, long long groups, int tiles, int G) {
  WinSplit w;
  const long long pairs = B * groups, room = (long long)num_sms() * (G > 8 ? 2 : 3);
  long long n = room / pairs;
  if (B > 1 && pairs < room) {
    const long long more = tiles / 32 < 4 * room / pairs ? tiles / 32 : 4 * room / pairs;
    if (n < more) n = more;
  }
  if (n > (tiles + 3) / 4) n = (tiles + 3) / 4;
  if (n < 1) n = 1;
  w.tiles = (int)((tiles + n - 1) / n);
  w.nsplit = (tiles + w.tiles - 1) / w.tiles;
  return w;
}
WinSplit q4_window_split(const WinDims& d) {
  // sinks, and a window that may begin inside a block
  const long long keys = (long long)(d.ns + kBlock - 1) / kBlock * kBlock + d.W + kBlock - 1;
  const long long most = (d.S + kBlock - 1) / kBlock, n = (keys + kBlock - 1) / kBlock;
  return q4_split(d.B, d.Hkv, (int)(n < most ? n : most), d.G);
}
WinSplit q4_sparse_split(const Dims& d) {
  const int blocks = d.S / kBlock;
  return q4_split(d.B, d.Hp * d.R, d.top_k < blocks ? d.top_k : blocks, d.G);
}

template <int NT, bool kSort>
static void q4_launch(int grid, size_t smem, const Q4Args& a, cudaStream_t st) {
  allow_smem<q4_decode_kernel<NT, kSort>>(smem);
  if (a.list) launch_behind(q4_decode_kernel<NT, kSort>, grid, kQ4Threads, smem, st, a);
  else q4_decode_kernel<NT, kSort><<<grid, kQ4Threads, smem, st>>>(a);
}
static void launch_q4(Q4Args& a, const WinSplit& w, cudaStream_t st) {
  a.nsplit = w.nsplit;
  a.tiles = w.tiles;
  const int grid = a.B * a.groups * w.nsplit;
  constexpr size_t smem = (size_t)kStages * kStageBytes;
  // Long sequences first, where blocks wait for a place: the last ones are then short.  Each block sorts for itself, which is
  // worth it while B times the waves of blocks is a small multiple of a sequence's tiles.  Unsorted / sorted, us (as above), 64 / 8
  // heads but for the last: 128 sequences of 4096 keys 118 / 122, of 2048 .. 4096 110 / 98, of 1 .. 4096 81 / 67, most
  // of them short 57 / 40; 64 of 1 .. 8192 83 / 79; 512 of 1 .. 8192, 8 / 1 heads, 92 / 78 (all of 8192 135 / 142: equal lengths
  // lose 3 to 6 %).  Outside the rule: 300 of 1 .. 2048, 32 / 4 heads, 58 / 58; 512 of 1 .. 1536, 32 / 8 heads, 121 / 159.
  const long long room = (long long)num_sms() * (a.G > 8 ? 2 : 3);
  const bool sort = a.B > 1 && a.B <= kSorted && grid > room && (long long)grid * a.B <= 12 * room * w.tiles;
  a.steps = (float)kSteps / ((float)w.tiles * w.nsplit);
  if (a.G > 8) sort ? q4_launch<2, true>(grid, smem, a, st) : q4_launch<2, false>(grid, smem, a, st);
  else sort ? q4_launch<1, true>(grid, smem, a, st) : q4_launch<1, false>(grid, smem, a, st);
  if (w.nsplit > 1) launch_decode_join(a.B, a.Hq, a.cap, w.nsplit, a.seq_len, a.opart, a.lpart, a.o, a.lse, st);
}

void launch_q4_window(const WinDims& d, const void* q, const void* k, const void* v, const int32_t* seq_len, void* o,
                      float* lse, float* opart, float* lpart, unsigned* status, cudaStream_t st) {
  Q4Args a{};
  a.k = (const uint8_t*)k;
  a.v = (const uint8_t*)v;
  a.q = (const bf16*)q;
  a.seq_len = seq_len;
  a.o = (bf16*)o;
  a.lse = lse;
  a.opart = opart;
  a.lpart = lpart;
  a.status = status;
  a.B = d.B;
  a.cap = d.S;
  a.blocks = d.S / kBlock;
  a.Hq = d.Hq;
  a.Hkv = a.groups = d.Hkv;
  a.Hp = 1;
  a.G = d.G;
  a.W = d.W;
  a.ns = d.ns;
  a.scale = d.scale;
  a.own_status = true;
  launch_q4(a, q4_window_split(d), st);
}

void launch_q4_sparse(const Dims& d, const void* q, const void* k, const void* v, const int32_t* seq_len,
                      const int32_t* block_idx, void* o, float* lse, float* opart, float* lpart, unsigned* status,
                      cudaStream_t st) {
  Q4Args a{};
  a.k = (const uint8_t*)k;
  a.v = (const uint8_t*)v;
  a.q = (const bf16*)q;
  a.seq_len = seq_len;
  a.list = block_idx;
  a.o = (bf16*)o;
  a.lse = lse;
  a.opart = opart;
  a.lpart = lpart;
  a.status = status;
  a.B = d.B;
  a.cap = d.S;
  a.blocks = d.S / kBlock;
  a.Hq = d.Hq;
  a.Hkv = d.Hkv;
  a.Hp = d.Hp;
  a.groups = d.Hp * d.R;
  a.G = d.G;
  a.top_k = d.top_k;
  a.scale = d.scale;
  launch_q4(a, q4_sparse_split(d), st);
}

}  // namespace msa
