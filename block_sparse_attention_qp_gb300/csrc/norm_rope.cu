// Per-head RMS norm with the position rotation in the same pass, its gradient, and the serving form
// that writes the new tokens' rows straight into the caches.
//
// A row is one head of one token, x in R^128 (bf16).  With w the part's norm weight (fp32):
//   r = (mean x^2 + eps)^-1/2,  u = w x r,  y = R(pos) u            (forward; one rounding, of y)
// R rotates the first `rot` elements in pairs -- (i, i + rot/2), or (2 i, 2 i + 1) interleaved -- by
// the angle pos * inv_freq[i].  Backward, from x and dy alone (r is cheaper to recompute than to keep):
//   g = R(-pos) dy,  dw = sum over rows of g x r,  h = g w,  dx = r h - x r^3 mean(h x).
// A part without a weight is not normed, one without the rotate flag not rotated, one with neither
// copied (the values of a packed projection).  Positions of several axes (time, height, width): pair i turns by the position of
// its own axis.  An append may leave a part's rows in 4 bits (q4.cuh).
//
// Angles: pos * inv_freq grows to millions of radians at far positions, where fp32 has lost the
// angle.  The frequency in turns, inv_freq / 2 pi, is kept as a 64-bit fraction of a turn F; the low
// 64 bits of pos * F are then the angle's exact fraction of a turn (whole turns wrap away, also for
// negative positions), whose upper 32 bits go to sincospif.  F is the nearest 2^-64 turns (from two
// doubles, for |inv_freq| up to 2^40): the angle is off by at most |pos| 2^-64 turns plus fp32 rounding.
//
// Work: 16 lanes hold a row (16 bytes a lane), a warp two tokens at a time, and walks the token's
// heads with its angles in registers, so they are computed once a token and part list, not once a
// head.  Bound by memory: forward reads and writes 256 bytes a row (6.0 TB/s at 64K tokens x 89 heads, 494
// us), backward reads 512 (256 where a part has no weight) and writes 256 (5.7 TB/s, 768 us with the join of
// dw); a copy runs at 6.7.  Over three axes, 32768 tokens x 57 heads: forward 175 us (5.5 TB/s), backward 253 and 10 of joining
// (5.3 TB/s).
// Few tokens: the heads of a token are split over warps so that a decode step still spreads over SMs.
// dw: per-warp sums in shared memory, one partial per block, then a second kernel adds the blocks'
// partials in a fixed order: no atomics, the same bits every time.
#include "common.cuh"
#include "kernels.h"
#include "q4.cuh"

namespace msa {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kRows = 4;  // rows in flight per half-warp (forward): 4 x 16 bytes a lane

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // bf16 is the upper half of an fp32
    f[2 * i] = __uint_as_float(p[i] << 16);
    f[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ float sum16(float s) {  // over the 16 lanes of a row
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}
__device__ __forceinline__ void load_w(const float* w, int l, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w) + 2 * l);
  const float4 b = __ldg(reinterpret_cast<const float4*>(w) + 2 * l + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// The block's frequencies as 64-bit fractions of a turn (and the pairs' axes).
template <bool kAxes>
__device__ __forceinline__ void load_freqs(const RopeArgs& A, unsigned long long* sF, uint8_t* sA) {
  const int i = threadIdx.x;
  if (kAxes && i < 64) sA[i] = A.axis[i];
  if (i < A.rot / 2) {
    // |f| / 2 pi as a sum of doubles t + lo: the product with the constant's upper half exact (a fused
    // multiply-add gives its rounding error), its lower half's added.  Whole turns go from t exactly.
    const double f = (double)A.inv_freq[i], w = fabs(f), up64 = 18446744073709551616.0;
    const double hi = 0.15915494309189535, t = w * hi;
    double lo = fma(w, -9.839338337591243e-18, fma(w, hi, -t));
    lo -= rint(lo);
    const double a = (t - floor(t)) * up64;
    const unsigned long long F =
        (unsigned long long)a + (unsigned long long)__double2ll_rn((a - floor(a)) + lo * up64);
    sF[i] = f < 0.0 ? 0ull - F : F;
  }
  __syncthreads();
}

// This lane's eight elements 8 l .. 8 l + 7 of the rotation at position pos: y = u c + partner s,
// the partner being element e +- rot/2 (or e +- 1), s signed accordingly (dir -1: the inverse).
struct Turn {
  float c[8], s[8];
};
template <bool kInter, bool kAxes>
__device__ __forceinline__ void make_turn(const RopeArgs& A, const unsigned long long* sF, const uint8_t* sA, int l,
                                          int pos, long long tok, float dir, Turn& t) {
  const int half = A.rot / 2;
  const bool in = 8 * l < A.rot;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = 1.f;
    t.s[i] = 0.f;
  }
  if (!in) return;
  int at[kRopeAxes];
  if (kAxes && A.naxes) {
#pragma unroll
    for (int x = 0; x < kRopeAxes; ++x) at[x] = __ldg(A.positions + (x < A.naxes ? x : 0) * ((long long)A.B * A.N) + tok);
  }
#pragma unroll
  for (int i = 0; i < (kInter ? 4 : 8); ++i) {
    const int e = kInter ? 4 * l + i : (8 * l < half ? 8 * l + i : 8 * l + i - half);
    if (kAxes && A.naxes) {
      const int x = sA[e];
      pos = x == 0 ? at[0] : x == 1 ? at[1] : x == 2 ? at[2] : at[3];
    }
    const unsigned long long a = (unsigned long long)(long long)pos * sF[e];
    const int turn = (int)(a >> 32);  // in 2^-32 turns, -1/2 .. 1/2
    float sn, cs;
    sincospif((float)turn * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: turns to half turns
    if (kInter) {
      t.c[2 * i] = t.c[2 * i + 1] = cs;
      t.s[2 * i] = -sn * dir;
      t.s[2 * i + 1] = sn * dir;
    } else {
      t.c[i] = cs;
      t.s[i] = (8 * l < half ? -sn : sn) * dir;
    }
  }
}
template <bool kInter>
__device__ __forceinline__ void turn_row(const Turn& t, int partner, float (&u)[8]) {
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = kInter ? u[i ^ 1] : __shfl_sync(0xffffffffu, u[i], partner, 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = fmaf(o[i], t.s[i], u[i] * t.c[i]);
}

// The walk shared by both kernels: warp-unit `wu` is two tokens (one per half-warp) and one run of
// the token's heads.  Warp-uniform but for the token; a half-warp past the last token repeats it
// (its loads are valid) and stores nothing.
struct Unit {
  long long tok;
  int b, i, pos, r0, r1;  // pos: with axes a cache's row only
  bool live;
};
__device__ __forceinline__ Unit rope_unit(const RopeArgs& A, long long wu, int hw) {
  Unit u;
  const long long T = (long long)A.B * A.N, pairs = (T + 1) / 2;
  const int chunk = (int)(wu / pairs);
  long long tok = (wu % pairs) * 2 + hw;
  u.live = tok < T;
  if (!u.live) tok = T - 1;
  u.tok = tok;
  u.b = (int)(tok / A.N);
  u.i = (int)(tok % A.N);
  u.r0 = chunk * A.rows_chunk;
  u.r1 = u.r0 + A.rows_chunk < A.rows ? u.r0 + A.rows_chunk : A.rows;
  if (A.seq_len) {
    const int len = A.seq_len[u.b];
    u.pos = len - A.N + u.i;
    if (len < A.N || len > A.cap) {  // flagged by the block that writes the status word
      u.live = false;
      u.pos = 0;
    }
  } else {
    u.pos = A.positions && !A.naxes ? A.positions[tok] : u.i;
  }
  return u;
}

}  // namespace

// kAxes: positions of several axes, or an append's own; kQ4: parts that go to caches in 4 bits (with kAxes).  Each has
// instances of its own: with the code of the caches in one the forward over three axes ran two blocks an SM of the
// three that it is launched with (271 us for 956 MB at 32768 tokens x 57 heads; 178 without).
template <bool kInter, bool kAxes, bool kQ4>
__global__ void __launch_bounds__(32 * kRopeWarps, kAxes ? 3 : 0) norm_rope_fwd_kernel(RopeArgs A) {
  constexpr int kR = kQ4 ? 2 : kRows;
  __shared__ unsigned long long sF[64];
  __shared__ uint8_t sA[64];
  load_freqs<kAxes>(A, sF, sA);
  const int lane = threadIdx.x % 32, l = lane % 16, hw = lane / 16;
  const int half8 = A.rot / 16;  // lanes per half of the rotated elements
  const int partner = 8 * l >= A.rot ? l : (l < half8 ? l + half8 : l - half8);
  const long long nwu = ((long long)A.B * A.N + 1) / 2 * A.chunks;
  if (A.status && blockIdx.x == 0) {
    // the whole word, by one block: clear, or a sequence length that does not fit its cache
    int bad = 0;
    for (int b = threadIdx.x; b < A.B; b += blockDim.x) bad |= A.seq_len[b] < A.N || A.seq_len[b] > A.cap;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *A.status = bad ? kStatusBadIndex : 0u;
  }
  for (long long wu = (long long)blockIdx.x * kRopeWarps + threadIdx.x / 32; wu < nwu;
       wu += (long long)gridDim.x * kRopeWarps) {
    const Unit u = rope_unit(A, wu, hw);
    Turn t;
    make_turn<kInter, kAxes>(A, sF, sA, l, u.pos, u.tok, 1.f, t);
    int base = 0;
    for (int p = 0; p < A.nparts; ++p) {
      const RopePart& P = A.p[p];
      const int h0 = max(u.r0 - base, 0), h1 = min(u.r1 - base, P.H);
      base += P.H;
      if (h0 >= h1) continue;
      const bf16* x = P.x + (long long)u.b * P.xb + (long long)u.i * P.xt + 8 * l;
      // the row of a cache is the token's position, of a plain output its index
      bf16* y = P.y + (long long)u.b * P.yb + (long long)(P.flags & kRopeCache ? u.pos : u.i) * P.yt + 8 * l;
      float w[8];
      const bool norm = P.w != nullptr, turn = (P.flags & kRopeRotate) != 0;
      uint8_t* cache = nullptr;  // in 4 bits: the block of the token's row of head h is head_blocks * h behind it
      long long head_blocks = 0;
      if (kQ4 && (P.flags & kRopeQ4)) {
        head_blocks = (long long)(A.cap / kBlock) * kQ4Block;
        cache = reinterpret_cast<uint8_t*>(P.y) + (long long)u.b * P.H * head_blocks + (long long)(u.pos / kBlock) * kQ4Block;
        if (!norm && !turn) {
          // rows as they are: eight lanes a row, two heads of the half-warp's token at a time, two of them in flight
          const int l8 = lane & 7, second = lane >> 3 & 1;
          for (int h = h0; h < h1; h += 4) {
            uint4 a[2], b[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint4* from = reinterpret_cast<const uint4*>(x - 8 * l + (long long)min(h + 2 * k + second, h1 - 1) * kD + 16 * l8);
              a[k] = from[0];
              b[k] = from[1];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int hh = h + 2 * k + second;
              q4_store_row8(a[k], b[k], cache + hh * head_blocks, u.pos % kBlock, l8, u.live && hh < h1);
            }
          }
          continue;
        }
      }
      if (norm) load_w(P.w, l, w);
      for (int h = h0; h < h1; h += kR) {
        uint4 v[kR];
#pragma unroll
        for (int k = 0; k < kR; ++k)
          if (h + k < h1) v[k] = *reinterpret_cast<const uint4*>(x + (long long)(h + k) * kD);
#pragma unroll
        for (int k = 0; k < kR; ++k) {
          if (h + k < h1) {
            if (norm || turn) {
              float f[8];
              unpack8(v[k], f);
              if (norm) {
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
                const float r = rsqrtf(fmaf(sum16(s), 1.f / kD, A.eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i];
              }
              if (turn) turn_row<kInter>(t, partner, f);
              v[k] = pack8(f);
            }
            if (kQ4 && cache) {
              q4_store_row(v[k], cache + (h + k) * head_blocks, u.pos % kBlock, l, u.live);
            } else if (u.live) {
              *reinterpret_cast<uint4*>(y + (long long)(h + k) * kD) = v[k];
            }
          }
        }
      }
    }
  }
}

// An append whose parts all go to caches in 4 bits as they are (a prompt's rows that its attention has used, new
// tokens rotated elsewhere): eight lanes a row, a warp eight rows of a token at a time.  Two prompts of 8192 tokens, 16 rows
// each: 20 us (3.3 TB/s of x), the kernel above 29; bound by its instructions and the latency of two waves of blocks.
__global__ void __launch_bounds__(32 * kRopeWarps) q4_store_kernel(RopeArgs A) {
  if (blockIdx.x == 0 && blockIdx.y == 0) {  // as above
    int bad = 0;
    for (int b = threadIdx.x; b < A.B; b += blockDim.x) bad |= A.seq_len[b] < A.N || A.seq_len[b] > A.cap;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *A.status = bad ? kStatusBadIndex : 0u;
  }
  const int lane = threadIdx.x % 32, l8 = lane & 7, h0 = (int)blockIdx.y * 8 + (lane >> 3);
  const long long head_blocks = (long long)(A.cap / kBlock) * kQ4Block;
  // this lane's two heads: of the eight of the block
  const bf16* from[2];
  uint8_t* to[2];
  long long xb[2], xt[2], yb[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    int h = h0 + 4 * k < A.rows ? h0 + 4 * k : A.rows - 1, p = 0;  // (behind the last one: loaded, not stored)
    while (h >= A.p[p].H) h -= A.p[p++].H;
    from[k] = A.p[p].x + (long long)h * kD + 16 * l8;
    to[k] = reinterpret_cast<uint8_t*>(A.p[p].y) + h * head_blocks;
    xb[k] = A.p[p].xb;
    xt[k] = A.p[p].xt;
    yb[k] = A.p[p].H * head_blocks;
  }
  const unsigned tokens = (unsigned)A.B * A.N, step = gridDim.x * kRopeWarps;
  for (unsigned tok = blockIdx.x * kRopeWarps + threadIdx.x / 32; tok < tokens; tok += step) {
    const int b = (int)(tok / A.N), i = (int)(tok % A.N);
    uint4 x[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4* at = reinterpret_cast<const uint4*>(from[k] + b * xb[k] + i * xt[k]);
      x[k][0] = at[0];
      x[k][1] = at[1];
    }
    const int len = __ldg(A.seq_len + b);
    const bool live = len >= A.N && len <= A.cap;
    const int pos = live ? len - A.N + i : 0;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      q4_store_row8(x[k][0], x[k][1], to[k] + b * yb[k] + (long long)(pos / kBlock) * kQ4Block, pos % kBlock, l8, live && h0 + 4 * k < A.rows);
  }
}

template <bool kInter, bool kAxes>
__global__ void __launch_bounds__(32 * kRopeWarps) norm_rope_bwd_kernel(RopeArgs A) {
  __shared__ unsigned long long sF[64];
  __shared__ uint8_t sA[64];
  extern __shared__ float sw[];  // [warps][parts][128]: the warps' shares of dw
  for (int i = threadIdx.x; i < kRopeWarps * A.nparts * kD; i += blockDim.x) sw[i] = 0.f;
  load_freqs<kAxes>(A, sF, sA);  // also the barrier behind the zeroes
  if (blockIdx.x == 0 && threadIdx.x == 0) *A.status = 0u;
  const int lane = threadIdx.x % 32, l = lane % 16, hw = lane / 16, warp = threadIdx.x / 32;
  const int half8 = A.rot / 16;
  const int partner = 8 * l >= A.rot ? l : (l < half8 ? l + half8 : l - half8);
  const long long nwu = ((long long)A.B * A.N + 1) / 2 * A.chunks;
  // rows in flight, x and dy of each: 4 read at 5.7 TB/s at 64K tokens x 89 heads (2: 4.8), with two
  // blocks of 126 registers a thread; three blocks spill
  constexpr int kR = 4;
  for (long long wu = (long long)blockIdx.x * kRopeWarps + warp; wu < nwu;
       wu += (long long)gridDim.x * kRopeWarps) {
    const Unit u = rope_unit(A, wu, hw);
    Turn t;
    make_turn<kInter, kAxes>(A, sF, sA, l, u.pos, u.tok, -1.f, t);
    int base = 0;
    for (int p = 0; p < A.nparts; ++p) {
      const RopePart& P = A.p[p];
      const int h0 = max(u.r0 - base, 0), h1 = min(u.r1 - base, P.H);
      base += P.H;
      if (h0 >= h1) continue;
      const bf16* x = P.x + (long long)u.b * P.xb + (long long)u.i * P.xt + 8 * l;
      const bf16* dy = P.y + (long long)u.b * P.yb + (long long)u.i * P.yt + 8 * l;
      bf16* dx = P.dx + (long long)u.b * P.dxb + (long long)u.i * P.dxt + 8 * l;
      const bool norm = P.w != nullptr, turn = (P.flags & kRopeRotate) != 0;
      float w[8], acc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      if (norm) load_w(P.w, l, w);
      for (int h = h0; h < h1; h += kR) {
        uint4 vx[kR], vg[kR];
#pragma unroll
        for (int k = 0; k < kR; ++k) {
          if (h + k < h1) {
            vg[k] = *reinterpret_cast<const uint4*>(dy + (long long)(h + k) * kD);
            if (norm) vx[k] = *reinterpret_cast<const uint4*>(x + (long long)(h + k) * kD);
          }
        }
#pragma unroll
        for (int k = 0; k < kR; ++k) {
          if (h + k < h1) {
            if (norm || turn) {
              float g[8];
              unpack8(vg[k], g);
              if (turn) turn_row<kInter>(t, partner, g);
              if (norm) {
                float f[8], s = 0.f, q = 0.f;
                unpack8(vx[k], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  s = fmaf(f[i], f[i], s);
                  q = fmaf(g[i] * w[i], f[i], q);
                }
                const float r = rsqrtf(fmaf(sum16(s), 1.f / kD, A.eps));
                const float m = sum16(q) * (1.f / kD) * r * r * r;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  if (u.live) acc[i] = fmaf(g[i], f[i] * r, acc[i]);
                  g[i] = fmaf(g[i] * w[i], r, -f[i] * m);
                }
              }
              vg[k] = pack8(g);
            }
            if (u.live) *reinterpret_cast<uint4*>(dx + (long long)(h + k) * kD) = vg[k];
          }
        }
      }
      if (norm) {  // both half-warps' rows of this part into the warp's own sums
        float* s = sw + (warp * A.nparts + p) * kD + 8 * l;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = acc[i] + __shfl_xor_sync(0xffffffffu, acc[i], 16);
          if (hw == 0) s[i] += a;
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < A.nparts * kD; i += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kRopeWarps; ++k) s += sw[k * A.nparts * kD + i];
    A.partial[(long long)blockIdx.x * A.nparts * kD + i] = s;
  }
}

// x += y with the rounding error of the sum kept in c (the error-free transformation of two terms).
__device__ __forceinline__ void add_exact(float& x, float& c, float y) {
  const float s = __fadd_rn(x, y), b = __fsub_rn(s, x);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(x, __fsub_rn(s, b)), __fsub_rn(y, b)));
  x = s;
}

// dw of part blockIdx.x: the blocks' partials, 32 interleaved runs (a warp each, four elements a lane)
// and then the runs in order.  Compensated fp32 sums: as good as fp64 here, whose few units took 17 us
// for 188 blocks' partials (this: 7).
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(RopeArgs A, int nblocks) {
  __shared__ float s[32][kD], e[32][kD];
  const int lane = threadIdx.x % 32, run = threadIdx.x / 32, p = blockIdx.x;
  if (!A.p[p].dw) return;
  float a[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = run; k < nblocks; k += 32) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(A.partial + ((long long)k * A.nparts + p) * kD) + lane);
    add_exact(a[0], c[0], v.x);
    add_exact(a[1], c[1], v.y);
    add_exact(a[2], c[2], v.z);
    add_exact(a[3], c[3], v.w);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s[run][4 * lane + i] = a[i];
    e[run][4 * lane + i] = c[i];
  }
  __syncthreads();
  if (threadIdx.x < kD) {
    float t = 0.f, u = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      add_exact(t, u, s[k][threadIdx.x]);
      u += e[k][threadIdx.x];
    }
    A.p[p].dw[threadIdx.x] = t + u;
  }
}

// Heads of a token per warp: all of them while the token pairs alone give every SM its warps, else
// runs of at least kRows rows.
static void split_rows(RopeArgs& A, int warps_wanted) {
  const long long pairs = ((long long)A.B * A.N + 1) / 2;
  long long want = (warps_wanted + pairs - 1) / pairs;
  const long long most = (A.rows + kRows - 1) / kRows;
  if (want > most) want = most;
  A.rows_chunk = (int)((A.rows + want - 1) / want);
  A.rows_chunk = (A.rows_chunk + kRows - 1) / kRows * kRows;
  A.chunks = (A.rows + A.rows_chunk - 1) / A.rows_chunk;
}
static int rope_grid(const RopeArgs& A, int per_sm) {
  const long long nwu = ((long long)A.B * A.N + 1) / 2 * A.chunks;
  const long long g = (nwu + kRopeWarps - 1) / kRopeWarps, most = (long long)num_sms() * per_sm;
  return (int)(g < most ? g : most);
}

constexpr int kRopeFwdBlocks = 3, kRopeBwdBlocks = 2;  // blocks per SM

int rope_partials() { return num_sms() * kRopeBwdBlocks; }

void launch_norm_rope_fwd(RopeArgs A, cudaStream_t st) {
  bool q4 = false, stored = true;  // any part in 4 bits, all of them as they are
  for (int p = 0; p < A.nparts; ++p) {
    q4 |= (A.p[p].flags & kRopeQ4) != 0;
    stored &= A.p[p].flags == kRopeQ4 && !A.p[p].w;
  }
  if (stored) {
    const unsigned blocks = ((unsigned)A.B * A.N + kRopeWarps - 1) / kRopeWarps, chunks = (A.rows + 7) / 8;
    const unsigned most = (num_sms() * 8 + chunks - 1) / chunks;
    q4_store_kernel<<<dim3(blocks < most ? blocks : most, chunks), 32 * kRopeWarps, 0, st>>>(A);
    return;
  }
  // (two blocks' warps per SM: 3 x 999 tokens x 15 heads in 11.3 us, with one block's 13.7)
  split_rows(A, num_sms() * 2 * kRopeWarps);
  const int g = rope_grid(A, kRopeFwdBlocks);
  auto launch = [&](auto kernel) { kernel<<<g, 32 * kRopeWarps, 0, st>>>(A); };
  if (q4) launch(A.inter ? norm_rope_fwd_kernel<true, true, true> : norm_rope_fwd_kernel<false, true, true>);
  else if (A.naxes) launch(A.inter ? norm_rope_fwd_kernel<true, true, false> : norm_rope_fwd_kernel<false, true, false>);
  else launch(A.inter ? norm_rope_fwd_kernel<true, false, false> : norm_rope_fwd_kernel<false, false, false>);
}

void launch_norm_rope_bwd(RopeArgs A, cudaStream_t st) {
  split_rows(A, num_sms() * kRopeWarps);
  const int g = rope_grid(A, kRopeBwdBlocks);
  const size_t smem = (size_t)kRopeWarps * A.nparts * kD * sizeof(float);  // at most 32 KB
  if (A.naxes) {
    if (A.inter) norm_rope_bwd_kernel<true, true><<<g, 32 * kRopeWarps, smem, st>>>(A);
    else norm_rope_bwd_kernel<false, true><<<g, 32 * kRopeWarps, smem, st>>>(A);
  } else {
    if (A.inter) norm_rope_bwd_kernel<true, false><<<g, 32 * kRopeWarps, smem, st>>>(A);
    else norm_rope_bwd_kernel<false, false><<<g, 32 * kRopeWarps, smem, st>>>(A);
  }
  bool any = false;
  for (int p = 0; p < A.nparts; ++p) any |= A.p[p].dw != nullptr;
  if (any) norm_rope_dw_kernel<<<A.nparts, 1024, 0, st>>>(A, g);
}

}  // namespace msa
