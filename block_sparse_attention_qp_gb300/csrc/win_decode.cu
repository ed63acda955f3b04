// Decode step of sliding-window attention (geometry: window.cuh): one new token per sequence, at
// position t = seq_len[b] - 1 of caches that already hold it, against the last W keys and the sinks.
//
// Bound by memory: the visible K and V rows are read once, 512 bytes a key and KV head.  A block takes
// one (b, KV head) and a run of 128-key tiles of the virtual walk; per tile
//   S^T = K_n Q^T        (tensor core, 128 keys x 16: the G query heads, the rest zero)
//   thread = key: tile maximum per head (warp reductions, then four values through shared memory),
//   P = 2^(sl2 S - m) -> bf16, [16 heads][128 keys] in shared memory; row sums per thread.  The rows that
//   a group of up to eight heads leaves over take P's rounding errors as a second bf16, in the same
//   product: O then has its own rounding only (relative error 1.7e-3; one bf16 P, as groups of 16 heads
//   have it, 2.2e-3)
//   O_n^T = V_n^T P^T    (tensor core, 128 dims x 16), added to the running O (thread = dim)
// 128 sequences with windows of 1024, 64 / 8 heads: 100 us, 595 MB read (5.95 TB/s) for the 535
// that are visible, the rest being the ninth tiles' other keys.
// 73 KB of shared memory leave three blocks to an SM: the loads of two run behind the chain of the
// third, and a block's next K tile is loaded as soon as S^T is there, its next V after O_n^T.
// Keys that no head may see (behind the sequence's end, before the window, between the sinks and the
// window) are masked out of S, and their V rows are zeroed in shared memory, so that whatever the
// caches hold there (also NaN) reaches nothing.
// Few (b, KV head) pairs: the tiles are split over blocks (fp32 O / l and log-sum-exps to the
// workspace) and win_decode_join_kernel merges the splits.
#include <math.h>

#include "tmap.h"
#include "window.cuh"

namespace msa {
namespace {

constexpr int kTile = 128 * 128 * 2;
constexpr int kNH = 16;           // MMA N: the group's heads, padded
constexpr int kDecThreads = 192;  // warps 0-3 softmax, 4 TMA, 5 MMA
constexpr int kDecBlocks = 3;     // blocks per SM

struct DecArgs {
  WinDims d;  // S: the caches' capacity
  KeyMaps k, v;
  const bf16* q;
  const int32_t* seq_len;
  bf16* o;
  float* lse;
  float *opart, *lpart;  // [split][B][Hq][128], [split][B][Hq] (log2 units)
  unsigned* status;
  int nsplit, tiles;  // splits, and key tiles per split
};
struct DecShared {
  uint64_t k_full, v_full, k_empty, v_empty, s_full, p_full, o_full, mma_done;
  uint32_t tmem;
  float wmax[2][4][kNH], wsum[4][kNH];
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

}  // namespace

template <int G>
__global__ void __launch_bounds__(kDecThreads, kDecBlocks) win_decode_kernel(const __grid_constant__ DecArgs A) {
  using namespace sm100;
  const WinDims& d = A.d;
  extern __shared__ uint8_t smem_raw[];
  DecShared* sh = reinterpret_cast<DecShared*>(smem_raw);
  uint8_t* sK = align1024(smem_raw + sizeof(DecShared));
  uint8_t* sV = sK + kTile;
  uint8_t* sQ = sV + kTile;        // [16 heads][128 d], K-major
  uint8_t* sP = sQ + kNH * kD * 2;  // [16 heads][128 keys], K-major
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int split = blockIdx.x % A.nsplit, bg = blockIdx.x / A.nsplit;
  const int b = bg / d.Hkv, g = bg % d.Hkv;
  if (blockIdx.x == 0) {  // the status word whole (see clear_status): clear, or a length out of range
    int bad = 0;
    for (int x = tid; x < d.B; x += kDecThreads) bad |= A.seq_len[x] < 1 || A.seq_len[x] > d.S;
    bad = __syncthreads_or(bad);
    if (tid < 32) A.status[tid] = tid == 0 && bad ? kStatusBadIndex : 0u;
  }
  const int len = A.seq_len[b];
  if (len < 1 || len > d.S) return;
  const int t = len - 1;
  const KeyRun run = key_run(d, t, t);
  const int n0 = split * A.tiles, n1 = min(n0 + A.tiles, run.nb), ntile = n1 - n0;
  const long long row0 = (long long)b * d.Hq + g * G;  // first query head of the group
  const long long part0 = ((long long)split * d.B * d.Hq + row0);
  if (ntile <= 0) {  // a sequence with fewer tiles than the longest possible
    if (tid < G) A.lpart[part0 + tid] = -INFINITY;
    return;
  }

  if (tid == 0) {
    mbar_init(&sh->k_full, 1);
    mbar_init(&sh->v_full, 1);
    mbar_init(&sh->k_empty, 1);
    mbar_init(&sh->v_empty, 1);
    mbar_init(&sh->s_full, 1);
    mbar_init(&sh->p_full, 4);
    mbar_init(&sh->o_full, 1);
    mbar_init(&sh->mma_done, 1);
    mbar_fence_init();
  }
  if (warp == 0) {
    __syncwarp();  // lane 0 initialised the barriers alone; the allocation is warp-collective
    tmem_alloc(&sh->tmem, 32);  // S^T: columns 0-15, O^T: 16-31
    tmem_relinquish();
  }
  // Q rows of the group (rows >= G zero) and P zeroed, as SW128 K-major tiles
  for (int x = tid; x < kNH * 16; x += kDecThreads) {
    const int r = x >> 4, ch = x & 15;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < G) v = *reinterpret_cast<const uint4*>(A.q + (row0 + r) * kD + ch * 8);
    const uint32_t off = (ch >> 3) * (kNH * 128) + sw128_chunk(r, ch & 7);
    *reinterpret_cast<uint4*>(sQ + off) = v;
    *reinterpret_cast<uint4*>(sP + off) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_async_smem();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tS = sh->tmem, tO = tS + 16;

  if (warp == 4) {
    // ---------------------------------------------------------------- TMA loads
    if (lane == 0) {
      for (int i = 0; i < ntile; ++i) {
        if (i > 0 && !mbar_wait(&sh->k_empty, phase_of(i - 1), A.status)) break;
        mbar_expect_tx(&sh->k_full, kTile);
        load_key_tile(sK, A.k, run, n0 + i, g, b, &sh->k_full);
        if (i > 0 && !mbar_wait(&sh->v_empty, phase_of(i - 1), A.status)) {
          mbar_wait(&sh->k_full, phase_of(i), A.status);
          break;
        }
        mbar_expect_tx(&sh->v_full, kTile);
        load_key_tile(sV, A.v, run, n0 + i, g, b, &sh->v_full);
        if (i + 1 == ntile) {  // no copy may still be landing when the block exits
          mbar_wait(&sh->k_full, phase_of(i), A.status);
          mbar_wait(&sh->v_full, phase_of(i), A.status);
        }
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issue
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_bf16(128, kNH, false, false);  // S^T = K Q^T
      constexpr uint32_t id_o = idesc_bf16(128, kNH, true, false);   // O^T = V^T P^T
      const uint32_t aQ = smem_u32(sQ), aP = smem_u32(sP), aK = smem_u32(sK), aV = smem_u32(sV);
      auto mma_s = [&](int i) -> bool {
        if (!mbar_wait(&sh->k_full, phase_of(i), A.status)) return false;
        fence_after_sync();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ss(tS, desc_kmajor(aK, 128, ks), desc_kmajor(aQ, kNH, ks), id_s, ks > 0);
        mma_commit(&sh->s_full);
        mma_commit(&sh->k_empty);
        return true;
      };
      bool ok = mma_s(0);
      for (int i = 0; ok && i < ntile; ++i) {
        // S^T of tile i has been read, its P written, O^T of tile i - 1 read, V rows masked
        if (!mbar_wait(&sh->p_full, phase_of(i), A.status)) break;
        fence_after_sync();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          mma_ss(tO, desc_mnmajor(aV, 128, ks), desc_kmajor(aP, kNH, ks), id_o, ks > 0);
        mma_commit(&sh->o_full);
        mma_commit(&sh->v_empty);
        if (i + 1 < ntile) ok = mma_s(i + 1);
      }
      mma_commit(&sh->mma_done);
      mbar_wait(&sh->mma_done, 0, A.status);  // no product may still write tensor memory
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax, accumulation
    constexpr bool kResidual = 2 * G <= kNH;
    const int kr = tid;  // key row of S^T; head dimension of O^T (tensor-memory lane)
    const uint32_t lrow = static_cast<uint32_t>(warp * 32) << 16;
    const float sl2 = d.scale * kLog2e;
    // visible virtual keys: [0, sc) and [lo, hi]
    const int sc = min(t + 1, d.ns), lo = max(run.nsp, t - d.W + 1 - run.ws + run.nsp), hi = t - run.ws + run.nsp;
    float m[G], l[G], acc[G];
#pragma unroll
    for (int h = 0; h < G; ++h) {
      m[h] = -INFINITY;
      l[h] = acc[h] = 0.f;
    }
    // The four warps pass the same named barriers in every tile whatever happens: a wait that gives
    // up only clears `ok` (warp-uniform), which skips the later waits and tensor-memory reads.
    bool ok = true;
    for (int i = 0; i < ntile; ++i) {
      const int v = (n0 + i) * kBlock + kr;
      const bool vis = v < sc || (v >= lo && v <= hi);
      if (ok) ok = mbar_wait_warp(&sh->s_full, phase_of(i), A.status);
      fence_after_sync();
      uint32_t s[16];
#pragma unroll
      for (int h = 0; h < 16; ++h) s[h] = 0u;
      if (ok) {
        tmem_ld16(tS + lrow, s);
        tmem_wait_ld();
      }
      float x[G];
#pragma unroll
      for (int h = 0; h < G; ++h) {
        x[h] = vis ? __uint_as_float(s[h]) * sl2 : -INFINITY;
        const float mx = warp_max(x[h]);
        if (lane == 0) sh->wmax[i & 1][warp][h] = mx;
      }
      fence_before_sync();
      bar_sync(1, 128);
      fence_after_sync();
      float alpha[G];
      const uint32_t prow = (uint32_t)(kr >> 6) * (kNH * 128);
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float(*wm)[kNH] = sh->wmax[i & 1];
        // every tile of a run holds a visible key: finite
        const float mn = fmaxf(fmaxf(fmaxf(wm[0][h], wm[1][h]), fmaxf(wm[2][h], wm[3][h])), m[h]);
        alpha[h] = exp2_ftz(m[h] - mn);  // 0 on the first tile
        m[h] = mn;
        const float p = exp2_ftz(x[h] - mn);  // masked: 2^-inf = 0
        l[h] = l[h] * alpha[h] + p;
        const bf16 hi = __float2bfloat16_rn(p);
        *reinterpret_cast<bf16*>(sP + prow + sw128_offset(h, kr & 63)) = hi;
        if (kResidual)
          *reinterpret_cast<bf16*>(sP + prow + sw128_offset(G + h, kr & 63)) = __float2bfloat16_rn(p - __bfloat162float(hi));
      }
      if (ok) ok = mbar_wait_warp(&sh->v_full, phase_of(i), A.status);
      if (!vis) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<uint4*>(sV + (c >> 3) * (kTile / 2) + sw128_chunk(kr, c & 7)) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_async_smem();  // P and zeroed rows (generic-proxy stores) before the tensor core's reads
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_full);
      if (ok) ok = mbar_wait_warp(&sh->o_full, phase_of(i), A.status);
      fence_after_sync();
      if (ok) {
        tmem_ld16(tO + lrow, s);
        tmem_wait_ld();
      }
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float y = __uint_as_float(s[h]);
        acc[h] = fmaf(acc[h], alpha[h], kResidual ? y + __uint_as_float(s[(G + h) % 16]) : y);
      }
      fence_before_sync();
    }
#pragma unroll
    for (int h = 0; h < G; ++h) {
      const float sum = warp_sum(l[h]);
      if (lane == 0) sh->wsum[warp][h] = sum;
    }
    bar_sync(1, 128);
    if (ok) {
#pragma unroll
      for (int h = 0; h < G; ++h) {
        const float sum = (sh->wsum[0][h] + sh->wsum[1][h]) + (sh->wsum[2][h] + sh->wsum[3][h]);
        const float y = acc[h] / sum, ls = m[h] + log2f(sum);
        if (A.nsplit == 1) {
          A.o[(row0 + h) * kD + kr] = __float2bfloat16_rn(y);
          if (kr == 0) A.lse[row0 + h] = ls * kLn2;
        } else {
          A.opart[(part0 + h) * kD + kr] = y;
          if (kr == 0) A.lpart[part0 + h] = ls;
        }
      }
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 0) tmem_dealloc(sh->tmem, 32);
}

// Merges the splits of every (b, head): one block each.  The splits' weights first, one thread a split;
// then eight runs of splits at once, 32 threads of four dims each, so that a thread's loads do not wait
// for one another.
constexpr int kJoinRuns = 8, kJoinThreads = 32 * kJoinRuns;
__global__ void __launch_bounds__(kJoinThreads) win_decode_join_kernel(int B, int Hq, int S, int nsplit,
                                                                       const int32_t* seq_len, const float* opart,
                                                                       const float* lpart, bf16* o, float* lse) {
  extern __shared__ float w[];  // [nsplit] weights
  wait_before();
  __shared__ float red[kJoinRuns];
  __shared__ float4 acc[kJoinRuns][32];
  const long long row = blockIdx.x, rows = (long long)B * Hq;
  const int len = seq_len[row / Hq], lane = threadIdx.x % 32, run = threadIdx.x / 32;
  if (len < 1 || len > S) return;  // flagged by win_decode_kernel
  float mx = -INFINITY;
  for (int s = threadIdx.x; s < nsplit; s += kJoinThreads) {
    w[s] = __ldcg(lpart + s * rows + row);
    mx = fmaxf(mx, w[s]);
  }
  mx = warp_max(mx);
  if (lane == 0) red[run] = mx;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kJoinRuns; ++k) mx = fmaxf(mx, red[k]);
  float sum = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = run; s < nsplit; s += kJoinRuns) {
    const float ls = w[s], p = exp2_ftz(ls - mx);
    if (ls == -INFINITY) continue;  // an empty split wrote no rows
    const float4 v = __ldcg(reinterpret_cast<const float4*>(opart + (s * rows + row) * kD) + lane);
    sum += p;
    a.x = fmaf(p, v.x, a.x);
    a.y = fmaf(p, v.y, a.y);
    a.z = fmaf(p, v.z, a.z);
    a.w = fmaf(p, v.w, a.w);
  }
  __syncthreads();  // everyone has read the maxima
  if (lane == 0) red[run] = sum;
  acc[run][lane] = a;
  __syncthreads();
  if (run > 0) return;
  sum = red[0];
#pragma unroll
  for (int k = 1; k < kJoinRuns; ++k) {
    const float4 v = acc[k][lane];
    sum += red[k];
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
  }
  const float inv = 1.f / sum;
  *reinterpret_cast<uint2*>(o + row * kD + 4 * lane) =
      make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
  if (lane == 0) lse[row] = (mx + log2f(sum)) * kLn2;
}

// Splits of the key tiles: as many as fill the resident blocks, one where the (b, KV head) pairs do (1024
// pairs of nine tiles, 2.25 waves: 100 us whole, 117 in two parts, 119 in three or four; 8 pairs of 257 tiles
// in 52 parts: 29 us and 8 of joining, while whole they would use 8 SMs).  Pairs that fill half of the
// resident blocks already stay whole: fewer blocks an SM have the bandwidth (64 tiles a pair: 224 pairs in two
// parts 6.2 TB/s, 232 whole 6.6, 456 whole 6.7); just above all of them a second wave costs a fifth (464 pairs:
// 5.3 TB/s, 608: 6.6).
WinSplit win_decode_split(const WinDims& d) {
  WinSplit w;
  const long long keys = (long long)d.W + d.nsp < d.S ? (long long)d.W + d.nsp : d.S;
  const int nb = (int)((keys + kBlock - 1) / kBlock);
  const long long pairs = (long long)d.B * d.Hkv, room = (long long)num_sms() * kDecBlocks;
  long long n = room / pairs;
  if (n < 1) n = 1;
  if (n > nb) n = nb;
  w.tiles = (int)((nb + n - 1) / n);
  w.nsplit = (nb + w.tiles - 1) / w.tiles;
  return w;
}

template <int G>
static void win_decode_g(const DecArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(DecShared) + 1024 + 2 * (size_t)kTile + 2 * (size_t)kNH * kD * 2;
  allow_smem<win_decode_kernel<G>>(smem);
  win_decode_kernel<G><<<a.d.B * a.d.Hkv * a.nsplit, kDecThreads, smem, st>>>(a);
}

bool launch_win_decode(const WinDims& d, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* seq_len, void* o, float* lse, float* opart, float* lpart,
                       unsigned* status, cudaStream_t st) {
  DecArgs a;
  if (!make_key_maps(d, k_cache, &a.k) || !make_key_maps(d, v_cache, &a.v)) return false;
  const WinSplit w = win_decode_split(d);
  a.d = d;
  a.q = (const bf16*)q;
  a.seq_len = seq_len;
  a.o = (bf16*)o;
  a.lse = lse;
  a.opart = opart;
  a.lpart = lpart;
  a.status = status;
  a.nsplit = w.nsplit;
  a.tiles = w.tiles;
  switch (d.G) {
    case 1: win_decode_g<1>(a, st); break;
    case 2: win_decode_g<2>(a, st); break;
    case 4: win_decode_g<4>(a, st); break;
    case 8: win_decode_g<8>(a, st); break;
    case 16: win_decode_g<16>(a, st); break;
    default: return false;
  }
  if (w.nsplit > 1) launch_decode_join(d.B, d.Hq, d.S, w.nsplit, seq_len, opart, lpart, o, lse, st);
  return true;
}

void launch_decode_join(int B, int Hq, int cap, int nsplit, const int32_t* seq_len, const float* opart,
                        const float* lpart, void* o, float* lse, cudaStream_t st) {
  launch_behind(win_decode_join_kernel, B * Hq, kJoinThreads, nsplit * sizeof(float), st, B, Hq, cap, nsplit, seq_len, opart, lpart, (bf16*)o, lse);
}

}  // namespace msa
