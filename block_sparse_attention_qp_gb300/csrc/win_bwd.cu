// Backward of causal attention over a sliding window and the first tokens (geometry: window.cuh), on
// the tcgen05 tensor cores.  With P = exp(scale QK^T - LSE) over the visible pairs, dP = dO V^T and
// D = rowsum(dO O) (rowdot_kernel in bwd.cu), for rows of few keys sum P dP (see win_dq_kernel):
//   dS = scale P (dP - D),  dV = P^T dO,  dK = dS^T Q,  dQ = dS K.
//
// Two kernels, each with its sums in tensor memory and no atomics, so a gradient has the same bits
// every time and nothing is accumulated in memory; the price is S and dP computed twice (7 products
// a tile pair instead of 5):
//   win_dkv_kernel  key-outer: an item is one 128-key block and up to `chunk` of the 128-row query
//                   tiles that see it (a tile: 128/G consecutive tokens x G heads).  A block with one
//                   chunk writes its dK and dV rows; the chunks of a longer list (a sink block is
//                   seen by the whole sequence) write fp32 partials that win_join_kernel adds in order.
//   win_dq_kernel   query-outer over the key tiles of the forward's virtual walk.
// Both split the softmax of a tile in two phases, so that the tensor core works through each of them:
//   A  P from S alone, as soon as S is there (kept in fp32 registers for phase B)
//   B  dS from P and dP.
// win_dkv: ... S(i+1) | dV(i) dK(i) dP(i+1) ...: S(i+1) is issued once S(i) is in registers, the rest
// after phase B of tile i, running behind phase A of tile i+1.  P^T and dS^T (bf16) take dP^T's columns
// in tensor memory and are the products' A operands from there; P^T over S^T, with dV(i) before S(i+1),
// made phase A, dV and S one chain (2.09 ms at 64K tokens, and 1.87 once P^T had moved).
// win_dq:  ... S(n+1) | dP(n+1) dQ(n) ...: S(n+1) is issued once S(n) is in registers, the pair after
// phase B of tile n, which leaves dS in columns of its own (two buffers), so that dP(n+1) need not
// wait for dQ(n).
// P and dS are rounded to bf16 for their products (2^-9 relative each), the softmax scale is folded
// into dS, everything else is fp32.  32 (dkv) and 24 (dq) instructions of 128 x 128 x 16 a tile pair, 64
// to 67 cycles each: at 64K tokens, 64 / 8 heads, window 512 dkv takes 1.90 ms (1,160 TFLOP/s of its four
// products over visible pairs) and dq 1.62 ms (1,020 of its three).
//
// Roles of both (640 threads): warp 0 TMA loads, warp 1 MMA issue (two issuing warps interleaved the
// products of a chain with the other's and were slower), warp 2 the tile's row data (dkv) or the TMA
// stores of dQ (dq), warps 4-19 softmax and epilogue: four per tensor-memory lane quarter,
// one per 32 of the tile's columns (with two, a phase was bound by the latencies of a warp's loads and
// exponentials).  Every wait is bounded.
#include <math.h>

#include "tmap.h"
#include "window.cuh"

namespace msa {
namespace {

constexpr int kTile = 128 * 128 * 2;  // 128 rows x 128 bf16, two SW128 panels
constexpr int kItemRing = 4, kMetaRing = 2, kQRing = 3;
constexpr int kSoft = 16;        // softmax / epilogue warps
constexpr int kBwdThreads = 640;  // 4 + kSoft warps

struct DkvArgs {
  WinDims d;
  CUtensorMap q, dout, k, v;
  const float2* rowm;  // {LSE log2 e, D} per query row [B, S, Hq]
  bf16 *dk, *dv;
  float* part;  // [slot][2: dV, dK][128 keys][128]
  unsigned* status;
  int* sched;
  WinItems it;
  PackedTables p;  // packed form only; d.S is then the number of tokens
};
struct DkvShared {
  float nlse2[kMetaRing][128], ndrow[kMetaRing][128];  // -(LSE log2 e), -(D scale) per tile row
  int it_ring[kItemRing];
  uint64_t k_full, v_full, kv_empty, q_full[kQRing], q_empty[kQRing], do_full[2], do_empty[2], m_full[kMetaRing],
      m_empty[kMetaRing], s_full, dp_full, sa, pb, acc_full, acc_free, it_full[kItemRing],
      it_empty[kItemRing], mma_done;
  uint32_t tmem;
};

// Item number -> key block n of (b, g) and its query tiles [i0, i1) (empty: i0 >= i1); slot: where its
// partial goes, -1 when the block has no other item.
struct DkvItem {
  int b, g, n, i0, i1, slot;
  int tfull;  // queries below it see the block's first key
};
template <int G>
__device__ __forceinline__ int block_tiles(const WinDims& d, int n) {  // query tiles that see block n
  const int k0 = n * kBlock;
  long long last = (long long)k0 + kBlock - 1 + d.W - 1;  // the last query of the block's last key
  if (k0 < d.ns || last >= d.S) last = d.S - 1;
  return (int)((last - k0) / (128 / G)) + 1;
}
template <int G, bool kPacked>
__device__ __forceinline__ DkvItem dkv_item(const DkvArgs& A, int it) {
  const WinDims& d = A.d;
  const WinItems& w = A.it;
  DkvItem x;
  if (kPacked) {
    const int4 e = __ldg(A.p.items + 2 * (it / d.Hkv)), f = __ldg(A.p.items + 2 * (it / d.Hkv) + 1);
    x.b = 0;
    x.g = it % d.Hkv;
    x.n = e.x;
    x.i0 = e.y;
    x.i1 = e.z;
    x.slot = e.w < 0 ? -1 : e.w * d.Hkv + x.g;
    x.tfull = f.x + 1;
    return x;
  }
  const int per = d.B * d.Hkv;
  int c, chunk, bh;
  if (it < w.sink_items) {  // chunk-major: concurrent items share query tiles
    c = it / (w.sink_blocks * per);
    const int rem = it % (w.sink_blocks * per);
    x.n = rem / per;
    bh = rem % per;
    chunk = w.sink_chunk;
  } else {
    const int j = it - w.sink_items;
    x.n = w.sink_blocks + j / (w.win_split * per);
    c = j / per % w.win_split;
    bh = j % per;
    chunk = w.win_chunk;
  }
  x.b = bh / d.Hkv;
  x.g = bh % d.Hkv;
  const int nt = block_tiles<G>(d, x.n);
  x.i0 = c * chunk;
  x.i1 = x.i0 + chunk < nt ? x.i0 + chunk : nt;
  x.slot = nt > chunk ? it : -1;
  const int k0 = x.n * kBlock;
  x.tfull = k0 + kBlock <= d.ns || k0 + d.W >= d.S ? d.S : k0 + d.W;
  return x;
}

}  // namespace

template <int G, bool kPacked>
__global__ void __launch_bounds__(kBwdThreads, 1) win_dkv_kernel(const __grid_constant__ DkvArgs A) {
  using namespace sm100;
  constexpr int TT = 128 / G;
  const WinDims& d = A.d;
  extern __shared__ __align__(1024) uint8_t smem_tiles[];
  uint8_t* sK = smem_tiles;
  uint8_t* sV = sK + kTile;
  uint8_t* sQ = sV + kTile;           // [kQRing] query tiles
  uint8_t* sD = sQ + kQRing * kTile;  // [2] dO tiles
  DkvShared* sh = reinterpret_cast<DkvShared*>(sD + 2 * kTile);
  const uint32_t aK = smem_u32(sK), aV = smem_u32(sV), aQ = smem_u32(sQ), aD = smem_u32(sD);
  const int tid = threadIdx.x, lane = tid % 32, warp = warp_number();
  const int total = A.it.items;
  if (aK & 1023u) {  // the swizzled operand layout needs 1024-byte atoms
    if (tid == 0) atomicOr(A.status, kStatusInternal);
    return;
  }

  if (tid == 0) {
    mbar_init(&sh->k_full, 1);
    mbar_init(&sh->v_full, 1);
    mbar_init(&sh->kv_empty, 1);
    for (int x = 0; x < kQRing; ++x) {
      mbar_init(&sh->q_full[x], 1);
      mbar_init(&sh->q_empty[x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh->do_full[x], 1);
      mbar_init(&sh->do_empty[x], 1);
    }
    for (int x = 0; x < kMetaRing; ++x) {
      mbar_init(&sh->m_full[x], 1);
      mbar_init(&sh->m_empty[x], kSoft);
    }
    for (int x = 0; x < kItemRing; ++x) {
      mbar_init(&sh->it_full[x], 1);
      mbar_init(&sh->it_empty[x], 2 + kSoft);  // MMA, row data, softmax warps
    }
    mbar_init(&sh->s_full, 1);
    mbar_init(&sh->dp_full, 1);
    mbar_init(&sh->sa, kSoft);
    mbar_init(&sh->pb, kSoft);
    mbar_init(&sh->acc_full, 1);
    mbar_init(&sh->acc_free, kSoft);
    mbar_init(&sh->mma_done, 1);
    mbar_fence_init();
  }
  if (warp == 0) {
    __syncwarp();  // lane 0 initialised the barriers alone; the allocation is warp-collective
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t SB = sh->tmem, DB = SB + 128, RV = SB + 256, RK = SB + 384;
  // item number k of this block (handed out in list order to whichever block asks next)
  auto takew = [&](long long k, int& v) -> bool {
    const int x = (int)(k % kItemRing);
    if (!mbar_wait_warp(&sh->it_full[x], phase_of(k / kItemRing), A.status)) return false;
    v = sh->it_ring[x];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->it_empty[x]);
    return true;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- items + TMA loads
    if (lane == 0) {
      long long nk = 0, i = 0, nq = 0;  // items with tiles, tiles, query tiles asked for
      Ring<kQRing> q;
      bool ok = true;
      for (long long k = 0; ok; ++k) {
        const int x = (int)(k % kItemRing);
        if (k >= kItemRing && !mbar_wait(&sh->it_empty[x], phase_of(k / kItemRing - 1), A.status)) break;
        const int v = atomicAdd(A.sched, 1);
        sh->it_ring[x] = v;
        mbar_arrive(&sh->it_full[x]);
        if (v >= total) break;
        const DkvItem t = dkv_item<G, kPacked>(A, v);
        if (t.i0 >= t.i1) continue;
        if (nk > 0 && !mbar_wait(&sh->kv_empty, phase_of(nk - 1), A.status)) break;
        ++nk;
        mbar_expect_tx(&sh->k_full, kTile);
        mbar_expect_tx(&sh->v_full, kTile);
        for (int c = 0; c < 2; ++c)
          tma_load_rows(sK + c * (kTile / 2), &A.k, 64 * c, t.g, t.n * kBlock, t.b, &sh->k_full);
        for (int c = 0; c < 2; ++c)
          tma_load_rows(sV + c * (kTile / 2), &A.v, 64 * c, t.g, t.n * kBlock, t.b, &sh->v_full);
        for (int tl = t.i0; tl < t.i1; ++tl, ++i, q.next()) {
          const int s = (int)(i & 1), tok = t.n * kBlock + tl * TT;
          if (q.wrapped && !mbar_wait(&sh->q_empty[q.slot], q.phase ^ 1, A.status)) { ok = false; break; }
          mbar_expect_tx(&sh->q_full[q.slot], kTile);
          for (int c = 0; c < 2; ++c)
            tma_load_rows(sQ + q.slot * kTile + c * (kTile / 2), &A.q, 64 * c, t.g * G, tok, t.b, &sh->q_full[q.slot]);
          ++nq;
          if (i >= 2 && !mbar_wait(&sh->do_empty[s], phase_of(i / 2 - 1), A.status)) { ok = false; break; }
          mbar_expect_tx(&sh->do_full[s], kTile);
          for (int c = 0; c < 2; ++c)
            tma_load_rows(sD + s * kTile + c * (kTile / 2), &A.dout, 64 * c, t.g * G, tok, t.b, &sh->do_full[s]);
        }
      }
      // no copy may still be landing in shared memory when the block exits
      if (nk > 0) {
        mbar_wait(&sh->k_full, phase_of(nk - 1), A.status);
        mbar_wait(&sh->v_full, phase_of(nk - 1), A.status);
      }
      for (long long x = nq >= kQRing ? nq - kQRing : 0; x < nq; ++x)
        mbar_wait(&sh->q_full[x % kQRing], phase_of(x / kQRing), A.status);
      for (long long x = i >= 2 ? i - 2 : 0; x < i; ++x) mbar_wait(&sh->do_full[x & 1], phase_of(x >> 1), A.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issue
    int nk = 0, i = 0;
    Ring<kQRing> q;
    bool ok = true;
    auto mma_dp = [&](int j) -> bool {  // dP^T = V dO^T
      const int s = j & 1;
      if (!mbar_wait_warp(&sh->do_full[s], phase_of(j >> 1), A.status)) return false;
      fence_after_sync();
      mma_kk(DB, aV, aD + s * kTile, false);
      warp_mma_commit(&sh->dp_full);
      return true;
    };
    auto mma_s = [&](const Ring<kQRing>& x) -> bool {  // S^T = K Q^T
      if (!mbar_wait_warp(&sh->q_full[x.slot], x.phase, A.status)) return false;
      fence_after_sync();
      mma_kk(SB, aK, aQ + x.slot * kTile, false);
      warp_mma_commit(&sh->s_full);
      return true;
    };
    for (long long k = 0; ok; ++k) {
      int v;
      if (!takew(k, v) || v >= total) break;
      const DkvItem t = dkv_item<G, kPacked>(A, v);
      if (t.i0 >= t.i1) continue;
      // (the previous item's last S^T, dS^T and P^T were read before its last products were issued, or
      // by them)
      if (!mbar_wait_warp(&sh->k_full, phase_of(nk), A.status) || !mma_s(q) ||
          !mbar_wait_warp(&sh->v_full, phase_of(nk), A.status) || !mma_dp(i))
        break;
      for (int tl = t.i0; tl < t.i1; ++tl, ++i) {
        const bool first = tl == t.i0, more = tl + 1 < t.i1;
        const int s = i & 1, qs = q.slot;
        q.next();
        // S^T is in registers: the next one can be computed behind phase A
        if (more && (!mbar_wait_warp(&sh->sa, phase_of(i), A.status) || !mma_s(q))) { ok = false; break; }
        // phase B has written dS^T and P^T over dP^T
        if ((first && nk > 0 && !mbar_wait_warp(&sh->acc_free, phase_of(nk - 1), A.status)) ||
            !mbar_wait_warp(&sh->pb, phase_of(i), A.status)) {
          ok = false;
          break;
        }
        fence_after_sync();
        // rows 32 p .. 32 p + 31: dS^T in columns 32 p .. 32 p + 15, P^T in 32 p + 16 .. 32 p + 31
        mma_tn<2, 32>(RV, DB + 16, aD + s * kTile, !first);  // dV += P^T dO
        warp_mma_commit(&sh->do_empty[s]);
        mma_tn<2, 32>(RK, DB, aQ + qs * kTile, !first);  // dK += dS^T Q
        warp_mma_commit(&sh->q_empty[qs]);
        if (more && !mma_dp(i + 1)) { ok = false; break; }
      }
      if (!ok) break;
      warp_mma_commit(&sh->acc_full);
      warp_mma_commit(&sh->kv_empty);
      ++nk;
    }
    warp_mma_commit(&sh->mma_done);
    mbar_wait_warp(&sh->mma_done, 0, A.status);  // no product may still write tensor memory
  } else if (warp == 2) {
    // ---------------------------------------------------------------- row data of the tiles
    Ring<kMetaRing> meta;
    bool ok = true;
    for (long long k = 0; ok; ++k) {
      int v;
      if (!takew(k, v) || v >= total) break;
      const DkvItem t = dkv_item<G, kPacked>(A, v);
      for (int tl = t.i0; tl < t.i1; ++tl, meta.next()) {
        const int s = meta.slot, tok = t.n * kBlock + tl * TT;
        float2 m[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = lane + 32 * e, q = tok + r / G;
          m[e] = q < d.S ? __ldg(A.rowm + ((long long)t.b * d.S + q) * d.Hq + t.g * G + r % G)
                         : make_float2(0.f, 0.f);
        }
        if (meta.wrapped && !mbar_wait_warp(&sh->m_empty[s], meta.phase ^ 1, A.status)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sh->nlse2[s][lane + 32 * e] = -m[e].x;
          sh->ndrow[s][lane + 32 * e] = -m[e].y * d.scale;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->m_full[s]);
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax (thread = key)
    const int part = (warp - 4) >> 2;  // rows 32 part .. 32 part + 31 of the tile
    const int quad = warp & 3;
    const int kr = quad * 32 + lane;  // key row = tensor-memory lane
    const uint32_t lb = static_cast<uint32_t>(quad * 32) << 16;
    const float sl2 = d.scale * kLog2e;
    const float2 sl2x2 = make_float2(sl2, sl2), sc2 = make_float2(d.scale, d.scale);
    const uint32_t Sx = SB + lb + 32 * part, Dx = DB + lb + 32 * part;
    int nk = 0, i = 0;
    Ring<kMetaRing> meta;
    bool ok = true;
    for (long long k = 0; ok; ++k) {
      int v;
      if (!takew(k, v) || v >= total) break;
      const DkvItem t = dkv_item<G, kPacked>(A, v);
      if (t.i0 >= t.i1) continue;
      const int j = t.n * kBlock + kr;  // this thread's key
      // queries that see it: j .. tmax
      const int tmax = j >= d.S ? -1 : kPacked ? __ldg(A.p.hi + j) : j < d.ns || j + d.W - 1 >= d.S ? d.S - 1 : j + d.W - 1;
      const int k0 = t.n * kBlock;
      for (int tl = t.i0; tl < t.i1; ++tl, ++i, meta.next()) {
        const int s = meta.slot, tok = t.n * kBlock + tl * TT;
        // the whole block behind every query of the tile, and inside its window?
        const bool full = tok >= k0 + kBlock - 1 && tok + TT <= t.tfull;
        uint32_t vis = 0xffffffffu;  // else the visible rows of this part, as a mask
        if (!full) vis = bit_range((j - tok) * G - 32 * part, (tmax - tok + 1) * G - 1 - 32 * part, 0);
        if (!mbar_wait_warp(&sh->m_full[s], meta.phase, A.status) ||
            !mbar_wait_warp(&sh->s_full, phase_of(i), A.status)) {
          ok = false;
          break;
        }
        fence_after_sync();
        // ---- phase A: P^T of this key and 32 rows, kept in registers
        float p[32];
        {
          uint32_t rs[32];
          tmem_ld32(Sx, rs);
          tmem_wait_ld();
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->sa);
          const float4* l4 = reinterpret_cast<const float4*>(sh->nlse2[s] + 32 * part);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 nl = l4[e];
            const float2 x0 = ffma2(make_float2(__uint_as_float(rs[4 * e]), __uint_as_float(rs[4 * e + 1])),
                                    sl2x2, make_float2(nl.x, nl.y));
            const float2 x1 = ffma2(make_float2(__uint_as_float(rs[4 * e + 2]), __uint_as_float(rs[4 * e + 3])),
                                    sl2x2, make_float2(nl.z, nl.w));
            float* pe = p + 4 * e;
            pe[0] = exp2_ftz(x0.x);
            pe[1] = exp2_ftz(x0.y);
            pe[2] = exp2_ftz(x1.x);
            pe[3] = exp2_ftz(x1.y);
            if (!full) {
#pragma unroll
              for (int u = 0; u < 4; ++u) pe[u] = (vis >> (4 * e + u)) & 1u ? pe[u] : 0.f;
            }
          }
        }
        // ---- phase B: dS^T = P^T (scale dP^T - scale D); both to tensor memory as bf16
        if (!mbar_wait_warp(&sh->dp_full, phase_of(i), A.status)) { ok = false; break; }
        fence_after_sync();
        {
          uint32_t rp[32], dw[16], pw[16];
          tmem_ld32(Dx, rp);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) pw[e] = pack_bf16(p[2 * e], p[2 * e + 1]);
          tmem_st16(Dx + 16, pw);  // over columns of dP^T this warp has read
          const float4* d4 = reinterpret_cast<const float4*>(sh->ndrow[s] + 32 * part);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 nd = d4[e];
            float2 y0 = ffma2(make_float2(__uint_as_float(rp[4 * e]), __uint_as_float(rp[4 * e + 1])), sc2,
                              make_float2(nd.x, nd.y));
            float2 y1 = ffma2(make_float2(__uint_as_float(rp[4 * e + 2]), __uint_as_float(rp[4 * e + 3])), sc2,
                              make_float2(nd.z, nd.w));
            y0 = fmul2(y0, make_float2(p[4 * e], p[4 * e + 1]));
            y1 = fmul2(y1, make_float2(p[4 * e + 2], p[4 * e + 3]));
            dw[2 * e] = pack_bf16(y0.x, y0.y);
            dw[2 * e + 1] = pack_bf16(y1.x, y1.y);
          }
          tmem_st16(Dx, dw);
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh->pb);
          mbar_arrive(&sh->m_empty[s]);
        }
      }
      if (!ok) break;
      // ---- item end: parts 0, 1 take the two halves of this key's dV row, parts 2, 3 of its dK row
      if (!mbar_wait_warp(&sh->acc_full, phase_of(nk), A.status)) break;
      ++nk;
      fence_after_sync();
      const int which = part >> 1, col = 64 * (part & 1);
      const uint32_t acc = (which == 0 ? RV : RK) + lb + col;
      bf16* dst = (which == 0 ? A.dv : A.dk) + (((long long)t.b * d.S + j) * d.Hkv + t.g) * kD + col;
      float* pdst = A.part + ((long long)t.slot * 2 + which) * (kBlock * kD) + (long long)kr * kD + col;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        tmem_ld32(acc + c * 32, r);
        tmem_wait_ld();
        if (t.slot >= 0) {
#pragma unroll
          for (int u = 0; u < 8; ++u)
            reinterpret_cast<uint4*>(pdst + c * 32)[u] = make_uint4(r[4 * u], r[4 * u + 1], r[4 * u + 2], r[4 * u + 3]);
        } else if (j < d.S) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint4 w;
            w.x = pack_bf16(__uint_as_float(r[8 * u]), __uint_as_float(r[8 * u + 1]));
            w.y = pack_bf16(__uint_as_float(r[8 * u + 2]), __uint_as_float(r[8 * u + 3]));
            w.z = pack_bf16(__uint_as_float(r[8 * u + 4]), __uint_as_float(r[8 * u + 5]));
            w.w = pack_bf16(__uint_as_float(r[8 * u + 6]), __uint_as_float(r[8 * u + 7]));
            reinterpret_cast<uint4*>(dst + c * 32)[u] = w;
          }
        }
        __syncwarp();
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->acc_free);
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 0) tmem_dealloc(sh->tmem, 512);
}

// Helpers of the row data kernels below: 16 dims a lane, eight lanes a row.
struct Dims16 {
  float f[16];
};
__device__ __forceinline__ Dims16 load16(const bf16* x, long long row, int c) {  // dims 8 c .. and 64 + 8 c ..
  Dims16 r;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const uint4 w = *reinterpret_cast<const uint4*>(x + row * kD + 64 * y + 8 * c);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r.f[8 * y + 2 * e] = __uint_as_float(u[e] << 16);
      r.f[8 * y + 2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  }
  return r;
}
__device__ __forceinline__ float dot16(const Dims16& a, const Dims16& b) {  // over the row's eight lanes
  float s = 0.f, t = 0.f;
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    s = fmaf(a.f[e], b.f[e], s);
    t = fmaf(a.f[e + 1], b.f[e + 1], t);
  }
  s += t;
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return s;
}
// D = sum_j P_j dP_j of one query row over a few keys (key_of(0) .. key_of(keys - 1): their rows of k and v), by a whole
// warp: four keys at a time, eight lanes a key.
template <typename F>
__device__ __forceinline__ float row_sum(const WinDims& d, const bf16* q, const bf16* k, const bf16* v, const bf16* dout, long long r,
                                         float l2, int keys, F&& key_of) {
  const int lane = threadIdx.x % 32, c = lane % 8, kk = lane / 8;
  const Dims16 fq = load16(q, r, c), fo = load16(dout, r, c);
  float sum = 0.f;
  for (int x0 = 0; x0 < keys; x0 += 4) {
    const long long key = key_of(x0 + kk < keys ? x0 + kk : keys - 1);  // past the end: the last key, not counted
    const Dims16 fk = load16(k, key, c), fv = load16(v, key, c);
    const float p = exp2_ftz(dot16(fq, fk) * d.scale * kLog2e - l2), dp = dot16(fo, fv);
    if (x0 + kk < keys) sum = fmaf(p, dp, sum);
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 8);
  return sum + __shfl_xor_sync(0xffffffffu, sum, 16);
}

// Row data {LSE log2 e, D} of windows of a few keys where a group is one head (a query tile is then 128
// tokens and spans two key tiles): one warp per query row.
__global__ void win_rowdata_kernel(WinDims d, const bf16* __restrict__ q, const bf16* __restrict__ k,
                                   const bf16* __restrict__ v, const bf16* __restrict__ dout,
                                   const float* __restrict__ lse, float2* __restrict__ rowm) {
  const long long rows = (long long)d.B * d.S * d.Hq, step = (long long)gridDim.x * blockDim.x / 32;
  for (long long r = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / 32; r < rows; r += step) {
    const int h = (int)(r % d.Hq), t = (int)(r / d.Hq % d.S), b = (int)(r / d.Hq / d.S);
    const float l2 = lse[((long long)b * d.Hq + h) * d.S + t] * kLog2e;
    const int w0 = t - d.W + 1 > 0 ? t - d.W + 1 : 0, far = d.ns < w0 ? d.ns : w0;  // sinks before the window
    const float sum = row_sum(d, q, k, v, dout, r, l2, far + t - w0 + 1, [&](int x) {
      return ((long long)b * d.S + (x < far ? x : w0 + x - far)) * d.Hkv + h / d.G;
    });
    if (threadIdx.x % 32 == 0) rowm[r] = make_float2(l2, sum);
  }
}

// Row data of packed sequences (and zeros for the gradients' rows behind the last one): D = rowsum(dO O), four rows a warp; but rows of a few keys -- the first ones of every
// sequence -- whose query tile spans several key tiles (win_dq_kernel leaves D of the others) have it from P and dP.
__global__ void __launch_bounds__(256, 4) packed_rowdata_kernel(WinDims d, PackedTables p, const bf16* __restrict__ q, const bf16* __restrict__ k,
                                                             const bf16* __restrict__ v, const bf16* __restrict__ o,
                                                             const bf16* __restrict__ dout, const float* __restrict__ lse,
                                                             float2* __restrict__ rowm, bf16* dq, bf16* dk, bf16* dv) {
  for (int x = 0; x < 3; ++x) {
    const int heads = x ? d.Hkv : d.Hq;
    uint4* to = reinterpret_cast<uint4*>((x == 0 ? dq : x == 1 ? dk : dv) + (long long)d.S * heads * kD);
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < (p.rows - d.S) * heads * (kD / 8); i += (long long)gridDim.x * blockDim.x)
      to[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  const unsigned rows = (unsigned)d.S * d.Hq, step = gridDim.x * blockDim.x / 32;  // (below 2^31)
  const int lane = threadIdx.x % 32, c = lane % 8, part = lane / 8, tt = kBlock / d.G;
  // (a warp's rows a quarter of the tensor apart: the rows of a few keys lie together, and four of them in turn by one
  // warp were a tail of 35 us)
  const unsigned quarter = (rows + 3) / 4;
  for (unsigned w = (blockIdx.x * blockDim.x + threadIdx.x) / 32; w < quarter; w += step) {
    const unsigned r = w + part * quarter < rows ? w + part * quarter : rows - 1;
    const int t = (int)(r / (unsigned)d.Hq), h = (int)(r % (unsigned)d.Hq), lo = __ldg(p.lo + t);
    float sum = dot16(load16(o, r, c), load16(dout, r, c));
    const float l2 = __ldg(lse + h * p.rows + t) * kLog2e;
    bool few = t - lo < kFewKeys;
    if (few) {
      const int t0 = t / tt * tt, t1 = t0 + tt - 1 < d.S ? t0 + tt - 1 : d.S - 1;
      few = t1 - __ldg(p.lo + t0) >= kBlock;
    }
    const unsigned which = __ballot_sync(0xffffffffu, few);
    for (int x = 0; x < 4; ++x) {
      if (!(which >> (8 * x) & 1u)) continue;
      const unsigned rx = __shfl_sync(0xffffffffu, r, 8 * x);
      const int first = __shfl_sync(0xffffffffu, lo, 8 * x), keys = __shfl_sync(0xffffffffu, t, 8 * x) - first + 1;
      const int g = __shfl_sync(0xffffffffu, h, 8 * x) / d.G;
      const float s = row_sum(d, q, k, v, dout, rx, __shfl_sync(0xffffffffu, l2, 8 * x), keys,
                              [&](int y) { return (long long)(first + y) * d.Hkv + g; });
      if (part == x) sum = s;
    }
    if (c == 0) rowm[r] = make_float2(l2, sum);
  }
}

// dK and dV rows of the key blocks whose query tiles were split: their partials added in order.  One
// block per 8 rows of (key block, b, g) and tensor; 32 threads a row, four values each.
template <int G, bool kPacked>
__global__ void __launch_bounds__(256) win_join_kernel(WinDims d, WinItems w, PackedTables p, const float* part, bf16* dk, bf16* dv) {
  const int per = d.B * d.Hkv;
  const int unit = blockIdx.x / 16, row = (blockIdx.x % 16) * 8 + threadIdx.x / 32, c = threadIdx.x % 32;
  const int4 e = kPacked ? __ldg(p.joins + unit / per) : make_int4(0, 0, 0, 0);
  const int n = kPacked ? e.x : unit / per, bh = unit % per, b = bh / d.Hkv, g = bh % d.Hkv;
  const int hf = blockIdx.y;  // 0: dV, 1: dK
  const bool sink = n < w.sink_blocks;
  const int chunk = sink ? w.sink_chunk : w.win_chunk;
  const int nt = kPacked ? 0 : block_tiles<G>(d, n), nc = kPacked ? e.z : (nt + chunk - 1) / chunk, j = n * kBlock + row;
  if (nc == 1 || j >= d.S) return;
  const long long first = kPacked ? (long long)e.y * per + bh : sink ? (long long)n * per + bh
                               : w.sink_items + ((long long)(n - w.sink_blocks) * w.win_split) * per + bh;
  const long long step = !kPacked && sink ? (long long)w.sink_blocks * per : per;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int x = 0; x < nc; ++x) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(
        part + ((first + x * step) * 2 + hf) * (kBlock * kD) + (long long)row * kD + 4 * c));
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  bf16* dst = (hf == 0 ? dv : dk) + (((long long)b * d.S + j) * d.Hkv + g) * kD + 4 * c;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
}

// ========================================================================================== dQ
namespace {
constexpr int kRingQ = 5;  // shared-memory tiles of win_dq_kernel beside Q and dO

struct DqArgs {
  WinDims d;
  KeyMaps k, v;
  CUtensorMap q, dout, dq;
  float2* rowm;
  unsigned* status;
  unsigned long long unit_ns;  // win_unit_wait_ns
  int units;  // one 128-row tile each
  PackedTables p;  // packed form only; d.S is then the number of tokens
};
struct DqShared {
  uint64_t q_full, q_empty, do_full, do_empty, kv_full[kRingQ], kv_empty[kRingQ], s_full, dp_full, pa, pb,
      d_full, dq_full, dq_free, st_full, mma_done;
  uint32_t tmem;
};
struct DqUnit {
  int b, g, t0;
  KeyRun run;
};
template <int G, bool kPacked>
__device__ __forceinline__ DqUnit dq_unit(const DqArgs& A, int u) {
  const WinDims& d = A.d;
  constexpr int TT = 128 / G;
  if (kPacked) {
    const int4 e = __ldg(A.p.dq + u / d.Hkv);
    const int t1 = e.x + TT - 1;
    return DqUnit{0, u % d.Hkv, e.x, packed_run(e.x, t1 < d.S ? t1 : d.S - 1, e.y, e.z)};
  }
  const int per = d.B * d.Hkv;
  DqUnit x;
  const int rem = u % per;
  x.b = rem / d.Hkv;
  x.g = rem % d.Hkv;
  x.t0 = u / per * TT;
  x.run = key_run(d, x.t0, x.t0 + TT - 1 < d.S ? x.t0 + TT - 1 : d.S - 1);
  return x;
}
}  // namespace

// D of rows of few keys: taken from the stored O it carries the roundings of P and of O, 2^-9 of
// |dO| |O| each, which raises the relative error of dQ and dK by about sqrt(1 + 2.7 / n) for n keys (1.10
// at 12, 1.05 at 24) over that of rounding dS and the result.  A unit whose keys fit one tile therefore
// takes D from P and dP, which it holds anyway, and leaves it for win_dkv_kernel: every row of up to 32
// keys in groups of two heads and more, and the first 128 / G tokens of every sequence.
//
// One unit is one 128-row query tile.  The ring holds, in this order, K_0 V_0 K_1 V_1 .. of a unit and
// then one tile without a load, through which the unit's dQ leaves.  Q and dO have one buffer each:
// the next unit's Q is loaded once the last S product has read it, its dO after the last dP product,
// both a step before the unit ends.
template <int G, bool kPacked>
__global__ void __launch_bounds__(kBwdThreads, 1) win_dq_kernel(const __grid_constant__ DqArgs A) {
  using namespace sm100;
  const WinDims& d = A.d;
  extern __shared__ uint8_t smem_raw[];
  DqShared* sh = reinterpret_cast<DqShared*>(smem_raw);
  uint8_t* sQ = align1024(smem_raw + sizeof(DqShared));
  uint8_t* sD = sQ + kTile;
  uint8_t* sR = sD + kTile;
  const uint32_t aQ = smem_u32(sQ), aD = smem_u32(sD), aR = smem_u32(sR);
  const int tid = threadIdx.x, lane = tid % 32, warp = warp_number();
  clear_status(A.status);  // also the item counter of win_dkv_kernel, which runs behind this kernel

  if (tid == 0) {
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    mbar_init(&sh->do_full, 1);
    mbar_init(&sh->do_empty, 1);
    for (int x = 0; x < kRingQ; ++x) {
      mbar_init(&sh->kv_full[x], 1);
      mbar_init(&sh->kv_empty[x], 1);
    }
    mbar_init(&sh->s_full, 1);
    mbar_init(&sh->dp_full, 1);
    mbar_init(&sh->pa, kSoft);
    mbar_init(&sh->pb, kSoft);
    mbar_init(&sh->d_full, kSoft);
    mbar_init(&sh->dq_full, 1);
    mbar_init(&sh->dq_free, kSoft);
    mbar_init(&sh->st_full, kSoft);
    mbar_init(&sh->mma_done, 1);
    mbar_fence_init();
  }
  if (warp == 0) {
    __syncwarp();  // lane 0 initialised the barriers alone; the allocation is warp-collective
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  // dS of step i: DS + 64 (i & 1)
  const uint32_t SB = sh->tmem, DP = SB + 128, DS = SB + 256, RQ = SB + 384;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA loads
    if (lane == 0) {
      long long nl = 0, nu = 0, nq = 0, nd = 0;  // ring entries, units, loads of Q and dO
      Ring<kRingQ> ring;
      auto taken = [&]() -> bool {  // the next ring slot is free
        return !ring.wrapped || mbar_wait(&sh->kv_empty[ring.slot], ring.phase ^ 1, A.status);
      };
      auto load = [&](const KeyMaps& m, const DqUnit& x, int n) -> bool {
        if (!taken()) return false;
        mbar_expect_tx(&sh->kv_full[ring.slot], kTile);
        load_key_tile(sR + ring.slot * kTile, m, x.run, n, x.g, x.b, &sh->kv_full[ring.slot]);
        ring.next();
        ++nl;
        return true;
      };
      bool ok = true;
      for (int u = blockIdx.x; u < A.units && ok; u = unit_at<kPacked>((int)++nu)) {
        const DqUnit x = dq_unit<G, kPacked>(A, u);
        if (nu > 0 && !mbar_wait(&sh->q_empty, phase_of(nu - 1), A.status)) { ok = false; break; }
        mbar_expect_tx(&sh->q_full, kTile);
        for (int c = 0; c < 2; ++c)
          tma_load_rows(sQ + c * (kTile / 2), &A.q, 64 * c, x.g * G, x.t0, x.b, &sh->q_full);
        ++nq;
        for (int n = 0; n < x.run.nb && ok; ++n) {
          if (!(ok = load(A.k, x, n))) break;
          if (n == 0) {
            if (nu > 0 && !mbar_wait(&sh->do_empty, phase_of(nu - 1), A.status)) { ok = false; break; }
            mbar_expect_tx(&sh->do_full, kTile);
            for (int c = 0; c < 2; ++c)
              tma_load_rows(sD + c * (kTile / 2), &A.dout, 64 * c, x.g * G, x.t0, x.b, &sh->do_full);
            ++nd;
          }
          ok = load(A.v, x, n);
        }
        if (!ok || !(ok = taken())) break;
        mbar_arrive(&sh->kv_full[ring.slot]);  // the tile dQ leaves through: nothing to load
        ring.next();
        ++nl;
      }
      // no copy may still be landing in shared memory when the block exits
      for (long long x = nl >= kRingQ ? nl - kRingQ : 0; x < nl; ++x)
        mbar_wait(&sh->kv_full[x % kRingQ], phase_of(x / kRingQ), A.status);
      if (nq > 0) mbar_wait(&sh->q_full, phase_of(nq - 1), A.status);
      if (nd > 0) mbar_wait(&sh->do_full, phase_of(nd - 1), A.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issue
    {
      // step i: key tile n of unit nu, whose K is in ring slot k (its V in the one after)
      Ring<kRingQ> k;
      auto mma_s = [&](const Ring<kRingQ>& k, bool first, bool last, int nu, int keys) -> bool {
        if (first && !mbar_wait_warp(&sh->q_full, phase_of(nu), A.status)) return false;
        if (!mbar_wait_warp(&sh->kv_full[k.slot], k.phase, A.status)) return false;
        fence_after_sync();
        if (keys >= kBlock) mma_kk(SB, aQ, aR + k.slot * kTile, false);  // S = Q K^T
        else mma_kk_part(SB, aQ, aR + k.slot * kTile, keys);
        warp_mma_commit(&sh->s_full);
        if (last) warp_mma_commit(&sh->q_empty);
        return true;
      };
      // (V's slot is freed by the softmax, which sees dP first: a commit less)
      auto mma_dp = [&](Ring<kRingQ> k, bool first, bool last, int nu, int keys) -> bool {
        k.next();
        if (first && !mbar_wait_warp(&sh->do_full, phase_of(nu), A.status)) return false;
        if (!mbar_wait_warp(&sh->kv_full[k.slot], k.phase, A.status)) return false;
        fence_after_sync();
        if (keys >= kBlock) mma_kk(DP, aD, aR + k.slot * kTile, false);  // dP = dO V^T
        else mma_kk_part(DP, aD, aR + k.slot * kTile, keys);
        warp_mma_commit(&sh->dp_full);
        if (last) warp_mma_commit(&sh->do_empty);
        return true;
      };
      int u = blockIdx.x;
      int len = dq_unit<G, kPacked>(A, u).run.len, nb = (len + kBlock - 1) / kBlock, i = 0;
      bool ok = mma_s(k, true, nb == 1, 0, len) && mma_dp(k, true, nb == 1, 0, len);
      for (int nu = 0; ok && nb > 0; ++nu) {
        u = unit_at<kPacked>(nu + 1);
        const int len2 = u < A.units ? dq_unit<G, kPacked>(A, u).run.len : 0;  // of the next unit (0: none)
        const int nb2 = (len2 + kBlock - 1) / kBlock;
        for (int n = 0; n < nb; ++n, ++i) {
          const bool last = n + 1 == nb;
          Ring<kRingQ> k2 = k;
          k2.next();
          k2.next();
          if (last) k2.next();  // the tile dQ leaves through
          const bool more = !last || nb2 > 0, last2 = last ? nb2 == 1 : n + 2 == nb;
          const int keys = len - n * kBlock, keys2 = last ? len2 : keys - kBlock;  // from this tile, the next on
          // phase A has read S
          if (!mbar_wait_warp(&sh->pa, phase_of(i), A.status) || (more && !mma_s(k2, last, last2, nu + 1, keys2))) {
            ok = false;
            break;
          }
          // phase B has read dP and written dS: dP of the next step first, dQ behind it (dS of step
          // i + 2 is written only after dP of step i + 2, issued after this product, is there)
          if (!mbar_wait_warp(&sh->pb, phase_of(i), A.status) || (more && !mma_dp(k2, last, last2, nu + 1, keys2)) ||
              // (the epilogue of the previous unit has read its dQ: it comes before phase B of this one)
              (n == 0 && nu >= 1 && !mbar_wait_warp(&sh->dq_free, phase_of(nu - 1), A.status))) {
            ok = false;
            break;
          }
          fence_after_sync();
          if (keys >= kBlock) mma_tn<8, 0>(RQ, DS + 64 * (i & 1), aR + k.slot * kTile, n > 0);  // dQ += dS K
          else mma_tn_part<8, 0>(RQ, DS + 64 * (i & 1), aR + k.slot * kTile, n > 0, keys);
          warp_mma_commit(&sh->kv_empty[k.slot]);
          if (last) warp_mma_commit(&sh->dq_full);
          k = k2;
        }
        nb = nb2;
        len = len2;
      }
      warp_mma_commit(&sh->mma_done);
      mbar_wait_warp(&sh->mma_done, 0, A.status);  // no product may still write tensor memory
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------------------------- TMA stores of dQ
    if (lane == 0) {
      long long nu = 0;
      int slot = 0;
      for (int u = blockIdx.x; u < A.units; u = unit_at<kPacked>((int)++nu), slot = (slot + 1) % kRingQ) {
        const DqUnit x = dq_unit<G, kPacked>(A, u);
        slot = (slot + 2 * x.run.nb) % kRingQ;  // the unit's last ring entry
        if (!mbar_wait(&sh->st_full, phase_of(nu), A.status, A.unit_ns)) break;
        tma_store_rows(&A.dq, aR + slot * kTile, 0, x.g * G, x.t0, x.b);
        tma_store_rows(&A.dq, aR + slot * kTile + kTile / 2, 64, x.g * G, x.t0, x.b);
        bulk_store_commit();
        bulk_store_wait_read();
        mbar_arrive(&sh->kv_empty[slot]);
      }
      bulk_store_wait();
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax (thread = row)
    const int part = (warp - 4) >> 2;  // keys 32 part .. 32 part + 31 of the tile
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // tile row = tensor-memory lane
    const uint32_t lb = static_cast<uint32_t>(quad * 32) << 16;
    const float sl2 = d.scale * kLog2e;
    const float2 sl2x2 = make_float2(sl2, sl2), sc2 = make_float2(d.scale, d.scale);
    auto row_data = [&](int u) -> float2 {
      if (u >= A.units) return make_float2(0.f, 0.f);
      const DqUnit x = dq_unit<G, kPacked>(A, u);
      const int t = x.t0 + r / G;
      // (a plain load: the kernel itself replaces the D of other rows of it)
      return t < d.S ? A.rowm[((long long)x.b * d.S + t) * d.Hq + x.g * G + r % G] : make_float2(0.f, 0.f);
    };
    // dQ of unit number `nu` (ring entry `nl`): tensor memory -> bf16 rows of the swizzled tile
    auto epilogue = [&](int nu, long long nl) -> bool {
      const int slot = (int)(nl % kRingQ);
      if (!mbar_wait_warp(&sh->dq_full, phase_of(nu), A.status) ||
          !mbar_wait_warp(&sh->kv_full[slot], phase_of(nl / kRingQ), A.status))
        return false;
      fence_after_sync();
      const uint32_t dst = aR + slot * kTile + (part >> 1) * (kTile / 2);
      uint32_t v[32];
      tmem_ld32(RQ + lb + 32 * part, v);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
          w[y] = pack_bf16(__uint_as_float(v[8 * e + 2 * y]), __uint_as_float(v[8 * e + 2 * y + 1]));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(dst + sw128_chunk(r, 4 * (part & 1) + e)),
                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
      }
      fence_before_sync();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh->dq_free);
        mbar_arrive(&sh->st_full);
      }
      return true;
    };
    long long nl = 0, pending = -1;  // pending: ring entry of the last unit's dQ
    int i = 0, nu = 0, v_slot = 1, singles = 0;  // singles: units of one key tile
    float2 m = row_data(blockIdx.x);
    bool ok = true;
    for (int u = blockIdx.x; u < A.units && ok; u = unit_at<kPacked>(++nu)) {
      const DqUnit x = dq_unit<G, kPacked>(A, u);
      const float2 mnext = row_data(unit_at<kPacked>(nu + 1));
      const int t = x.t0 + r / G;
      const int t_lo = kPacked ? __ldg(A.p.lo + (t < d.S ? t : d.S - 1)) : 0;
      const float2 nl2 = make_float2(-m.x, -m.x);
      float2 nd2 = make_float2(-m.y * d.scale, -m.y * d.scale);
      for (int n = 0; n < x.run.nb; ++n, ++i) {
        if (n > 0 && x.run.keys(n) <= 32 * part) {  // a run's last tile that ends before this part
          if (!mbar_wait_warp(&sh->s_full, phase_of(i), A.status)) { ok = false; break; }
          if (lane == 0) mbar_arrive(&sh->pa);
          if (!mbar_wait_warp(&sh->dp_full, phase_of(i), A.status)) { ok = false; break; }
          if (lane == 0) mbar_arrive(&sh->pb);
          continue;
        }
        const bool full = n >= x.run.f0 && n <= x.run.f1;
        uint32_t vis = 0xffffffffu;
        if (!full) {
          uint32_t vis4[4];
          if (kPacked) visible_cols_packed(x.run, n, t, t_lo, vis4);
          else visible_cols(d, x.run, n, t, vis4);
          vis = part == 0 ? vis4[0] : part == 1 ? vis4[1] : part == 2 ? vis4[2] : vis4[3];
        }
        if (!mbar_wait_warp(&sh->s_full, phase_of(i), A.status)) { ok = false; break; }
        fence_after_sync();
        // ---- phase A
        float p[32];
        {
          uint32_t rs[32];
          tmem_ld32(SB + lb + 32 * part, rs);
          tmem_wait_ld();
          fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->pa);  // S is in registers
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = ffma2(make_float2(__uint_as_float(rs[2 * e]), __uint_as_float(rs[2 * e + 1])), sl2x2, nl2);
            p[2 * e] = exp2_ftz(y.x);
            p[2 * e + 1] = exp2_ftz(y.y);
            if (!full) {
              p[2 * e] = (vis >> (2 * e)) & 1u ? p[2 * e] : 0.f;
              p[2 * e + 1] = (vis >> (2 * e + 1)) & 1u ? p[2 * e + 1] : 0.f;
            }
          }
        }
        if (n == 0 && pending >= 0 && !epilogue(nu - 1, pending)) { ok = false; break; }
        // ---- phase B
        if (!mbar_wait_warp(&sh->dp_full, phase_of(i), A.status)) { ok = false; break; }
        fence_after_sync();
        if (warp == 4 && lane == 0) mbar_arrive(&sh->kv_empty[v_slot]);  // V has been read
        v_slot += n + 1 < x.run.nb ? 2 : 3;  // (a unit ends with the tile dQ leaves through)
        v_slot -= v_slot >= kRingQ ? kRingQ : 0;
        {
          uint32_t rp[32], dw[16];
          tmem_ld32(DP + lb + 32 * part, rp);
          tmem_wait_ld();
          if (x.run.nb == 1) {
            // D = sum P dP, here and for win_dkv_kernel: the row's four threads meet in columns of dP
            // that their own warps have read.  Columns behind the run's keys hold anything (the products
            // leave them out), so the sum picks those with a P; a factor of 0 would not silence a NaN.
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              s0 = fmaf(p[e], p[e] > 0.f ? __uint_as_float(rp[e]) : 0.f, s0);
              s1 = fmaf(p[e + 1], p[e + 1] > 0.f ? __uint_as_float(rp[e + 1]) : 0.f, s1);
            }
            tmem_st1(DP + lb + 32 * part, __float_as_uint(s0 + s1));
            tmem_wait_st();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->d_full);
            if (!mbar_wait_warp(&sh->d_full, phase_of(singles++), A.status)) { ok = false; break; }
            fence_after_sync();
            uint32_t c4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) c4[c] = tmem_ld1(DP + lb + 32 * c);
            tmem_wait_ld();
            const float dd = (__uint_as_float(c4[0]) + __uint_as_float(c4[1])) +
                             (__uint_as_float(c4[2]) + __uint_as_float(c4[3]));
            if (part == 0 && t < d.S)
              A.rowm[((long long)x.b * d.S + t) * d.Hq + x.g * G + r % G] = make_float2(m.x, dd);
            nd2 = make_float2(-dd * d.scale, -dd * d.scale);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = fmul2(
                ffma2(make_float2(__uint_as_float(rp[2 * e]), __uint_as_float(rp[2 * e + 1])), sc2, nd2),
                make_float2(p[2 * e], p[2 * e + 1]));
            dw[e] = pack_bf16(y.x, y.y);
          }
          tmem_st16(DS + 64 * (i & 1) + lb + 16 * part, dw);
        }
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->pb);
      }
      if (!ok) break;
      nl += 2 * x.run.nb;
      pending = nl++;
      m = mnext;
    }
    if (ok && pending >= 0) epilogue(nu - 1, pending);
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 0) tmem_dealloc(sh->tmem, 512);
}

// ========================================================================================== host
// Key blocks and query tiles are cut so that the key-outer items number about eight per SM, in
// chunks of at least four tiles.  Window blocks stay whole from four per SM on: their partials cost
// more than the last items' imbalance (2 x 8192 tokens, 8 KV heads, window 1024, 6.7 blocks per SM: 68 us
// of joining and 30 us of writing partials when split in two).
WinItems win_items(const WinDims& d) {
  WinItems w;
  const int tt = kBlock / d.G, nblk = (d.S + kBlock - 1) / kBlock, per = d.B * d.Hkv;
  w.sink_blocks = (d.ns + kBlock - 1) / kBlock;
  const long long span = (long long)kBlock + d.W - 1 < d.S ? (long long)kBlock + d.W - 1 : d.S;
  const long long win_tiles = (span + tt - 1) / tt, all_tiles = (d.S + tt - 1) / tt;
  const long long win_blocks = (long long)(nblk - w.sink_blocks) * per;
  const long long total = w.sink_blocks * all_tiles * per + win_blocks * win_tiles;
  long long c = (total + 8ll * num_sms() - 1) / (8ll * num_sms());
  if (c < 4) c = 4;
  w.sink_chunk = (int)(c < all_tiles ? c : all_tiles);
  w.win_chunk = (int)(c < win_tiles && win_blocks < 4ll * num_sms() ? c : win_tiles);
  w.win_split = (int)((win_tiles + w.win_chunk - 1) / w.win_chunk);
  const int sink_split = (int)((all_tiles + w.sink_chunk - 1) / w.sink_chunk);
  w.sink_items = w.sink_blocks * sink_split * per;
  w.items = w.sink_items + (nblk - w.sink_blocks) * w.win_split * per;
  // partials are indexed by item; without split window blocks only the sink items have any
  w.partials = w.win_split > 1 ? w.items : sink_split > 1 ? w.sink_items : 0;
  w.join_blocks = w.win_split > 1 ? nblk : sink_split > 1 ? w.sink_blocks : 0;
  return w;
}

#define MSA_BY_GROUP(G_, CALL) \
  switch (G_) {                \
    case 1: CALL(1); break;    \
    case 2: CALL(2); break;    \
    case 4: CALL(4); break;    \
    case 8: CALL(8); break;    \
    case 16: CALL(16); break;  \
    default: return false;     \
  }

void launch_win_rowdata(const WinDims& d, const void* q, const void* k, const void* v, const void* dout,
                        const float* lse, float2* rowm, cudaStream_t st) {
  const long long blocks = ((long long)d.B * d.S * d.Hq + 7) / 8, most = (long long)num_sms() * 8;
  win_rowdata_kernel<<<(int)(blocks < most ? blocks : most), 256, 0, st>>>(
      d, (const bf16*)q, (const bf16*)k, (const bf16*)v, (const bf16*)dout, lse, rowm);
}

static void dkv_args(DkvArgs& a, const WinDims& d, const float2* rowm, void* dk, void* dv, float* part, unsigned* status) {
  a.d = d;
  a.rowm = rowm;
  a.dk = (bf16*)dk;
  a.dv = (bf16*)dv;
  a.part = part;
  a.status = status;
  a.sched = reinterpret_cast<int*>(status + kSchedWinDkv);
}
template <bool kPacked>
static bool dkv_any(DkvArgs& a, const void* q, const void* k, const void* v, const void* dout, cudaStream_t st) {
  const WinDims& d = a.d;
  const int tt = kBlock / d.G, n = num_sms();
  if (!make_tmap_rows(&a.q, q, d.B, d.S, d.Hq, d.G, tt) || !make_tmap_rows(&a.dout, dout, d.B, d.S, d.Hq, d.G, tt) ||
      !make_tmap_rows(&a.k, k, d.B, d.S, d.Hkv, 1, kBlock) || !make_tmap_rows(&a.v, v, d.B, d.S, d.Hkv, 1, kBlock))
    return false;
  const size_t smem = sizeof(DkvShared) + 7 * (size_t)kTile;
#define MSA_CALL(G)                             \
  allow_smem<win_dkv_kernel<G, kPacked>>(smem); \
  win_dkv_kernel<G, kPacked><<<a.it.items < n ? a.it.items : n, kBwdThreads, smem, st>>>(a)
  MSA_BY_GROUP(d.G, MSA_CALL)
#undef MSA_CALL
  return true;
}
bool launch_win_dkv(const WinDims& d, const void* q, const void* k, const void* v, const void* dout,
                    const float2* rowm, void* dk, void* dv, float* part, unsigned* status, cudaStream_t st) {
  DkvArgs a{};
  dkv_args(a, d, rowm, dk, dv, part, status);
  a.it = win_items(d);
  return dkv_any<false>(a, q, k, v, dout, st);
}
void launch_packed_rowdata(const PackedDims& x, const PackedTables& p, const void* q, const void* k, const void* v, const void* o,
                           const void* dout, const float* lse, float2* rowm, void* dq, void* dk, void* dv, cudaStream_t st) {
  const long long blocks = ((long long)x.d.S * x.d.Hq + 31) / 32, most = (long long)num_sms() * 16;
  packed_rowdata_kernel<<<(int)(blocks < most ? blocks : most), 256, 0, st>>>(
      x.d, p, (const bf16*)q, (const bf16*)k, (const bf16*)v, (const bf16*)o, (const bf16*)dout, lse, rowm, (bf16*)dq, (bf16*)dk, (bf16*)dv);
}
bool launch_packed_dkv(const PackedDims& x, const PackedTables& p, const void* q, const void* k, const void* v, const void* dout,
                       const float2* rowm, void* dk, void* dv, float* part, unsigned* status, cudaStream_t st) {
  DkvArgs a{};
  dkv_args(a, x.d, rowm, dk, dv, part, status);
  a.p = p;
  a.it.items = x.items * x.d.Hkv;
  return dkv_any<true>(a, q, k, v, dout, st);
}

template <bool kPacked>
static bool dq_any(DqArgs& a, const void* q, const void* k, const void* v, const void* dout, void* dq, cudaStream_t st) {
  const WinDims& d = a.d;
  const int tt = kBlock / d.G, n = num_sms();
  if (!make_tmap_rows(&a.q, q, d.B, d.S, d.Hq, d.G, tt) || !make_tmap_rows(&a.dout, dout, d.B, d.S, d.Hq, d.G, tt) ||
      !make_tmap_rows(&a.dq, dq, d.B, d.S, d.Hq, d.G, tt) || !make_key_maps(d, k, &a.k) || !make_key_maps(d, v, &a.v))
    return false;
  a.unit_ns = win_unit_wait_ns(d);
  const size_t smem = sizeof(DqShared) + 1024 + (2 + kRingQ) * (size_t)kTile;
#define MSA_CALL(G)                            \
  allow_smem<win_dq_kernel<G, kPacked>>(smem); \
  win_dq_kernel<G, kPacked><<<a.units < n ? a.units : n, kBwdThreads, smem, st>>>(a)
  MSA_BY_GROUP(d.G, MSA_CALL)
#undef MSA_CALL
  return true;
}
bool launch_win_dq(const WinDims& d, const void* q, const void* k, const void* v, const void* dout,
                   float2* rowm, void* dq, unsigned* status, cudaStream_t st) {
  DqArgs a{};
  a.d = d;
  a.rowm = rowm;
  a.status = status;
  const int tt = kBlock / d.G;
  a.units = (d.S + tt - 1) / tt * d.B * d.Hkv;
  return dq_any<false>(a, q, k, v, dout, dq, st);
}
bool launch_packed_dq(const PackedDims& x, const PackedTables& p, const void* q, const void* k, const void* v, const void* dout,
                      float2* rowm, void* dq, unsigned* status, cudaStream_t st) {
  DqArgs a{};
  a.d = x.d;
  a.p = p;
  a.rowm = rowm;
  a.status = status;
  a.units = x.dq_units * x.d.Hkv;
  return dq_any<true>(a, q, k, v, dout, dq, st);
}

template <bool kPacked>
static bool join_any(const WinDims& d, const WinItems& w, const PackedTables& p, const float* part, void* dk, void* dv, cudaStream_t st) {
  const dim3 grid(w.join_blocks * d.B * d.Hkv * 16, 2);
#define MSA_CALL(G) win_join_kernel<G, kPacked><<<grid, 256, 0, st>>>(d, w, p, part, (bf16*)dk, (bf16*)dv)
  MSA_BY_GROUP(d.G, MSA_CALL)
#undef MSA_CALL
  return true;
}
bool launch_win_join(const WinDims& d, const float* part, void* dk, void* dv, cudaStream_t st) {
  const WinItems w = win_items(d);
  return !w.join_blocks || join_any<false>(d, w, PackedTables{}, part, dk, dv, st);
}
bool launch_packed_join(const PackedDims& x, const PackedTables& p, const float* part, void* dk, void* dv, cudaStream_t st) {
  WinItems w{};
  w.join_blocks = x.joins;
  return !w.join_blocks || join_any<true>(x.d, w, p, part, dk, dv, st);
}
#undef MSA_BY_GROUP

}  // namespace msa
