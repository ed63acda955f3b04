// Forward of causal attention over a sliding window and the first tokens (window.cuh has the
// geometry): O = softmax(scale Q K^T) V over each query's visible keys, and the log-sum-exp of every
// row, on the tcgen05 tensor cores.
//
// Query-outer: a unit is two 128-row tiles of one (b, KV head) -- a tile is 128/G consecutive tokens
// x the G query heads of the group -- whose queries share every key tile of their joint run (one
// tile per unit when pairs would leave SMs idle).  Per key tile n and query tile X:
//   S_X = Q_X K_n^T                (tensor memory, 128 x 128 fp32)
//   P = 2^(sl2 (S - mr)), l += row sum  (thread = row; P in bf16 over S in tensor memory); the
//       running maximum mr moves only when the tile's maximum exceeds it by more than 8 / sl2, and
//       then O_X and l are rescaled first (O_X's last product was issued before S_X, so it is done)
//   O_X += P V_n
// P is rounded to bf16 for its product: relative 2^-9 a key, which averages out to less than the
// rounding of O itself; the row sum l is taken from the fp32 values.  Keys outside a row's window get
// P = 0 exactly; a V row that is not finite and that only some of a tile's queries see is taken care of by
// mend_rows.  A row may see nothing of a tile (its maximum then stays -inf until it does).
//
// 4 x 128 flops a visible pair, and the tiles cost about (W + 256/G + 128) / W of that; K and V come
// through L2.  1,420 TFLOP/s of visible pairs at 32K tokens, 32 / 8 heads, window 2048 (754 us), 1,030 at 64K
// tokens, 64 / 8 heads, window 512 (1.07 ms), where the tiles hold 1.2 times the visible pairs.  Bound by
// the hand-offs of the chain S, softmax, P V of a tile: without exponentials, loads and seven of eight
// products an earlier form took 690 of its 840 us.  The order of products is
// O_A(n-1) S_A(n) O_B(n-1) S_B(n), so the softmax of one tile runs behind the products of the other.
// Q has two buffers, so a unit's loads and first products overlap the previous unit's end; O leaves
// through the unit's own Q buffer by TMA stores, which also drop the rows past the sequence.
//
// Roles (640 threads): warp 0 TMA loads, warp 1 MMA issue, warps 2 / 3 the TMA stores of tile A / B,
// warps 4-11 / 12-19 softmax and epilogue of tile A / B: a row belongs to two threads, one per half of
// the columns, so that a tile's softmax fits behind the other tile's products (one thread a row: 1,126 us
// at 32K tokens, two: 1,012, both before the later steps).  The two share the row maximum: a barrier that ORs
// "my half exceeds it" across them, and an exchange through shared memory in the rare case it does.
// Tensor memory: S_A, S_B, O_A, O_B (512 columns).  Units are dealt in turn, tokens outermost, so that concurrent
// units share K and V: equal costs where the window is short beside the sequence.  Where it is not, costs rise
// along the sequence and the longest units come last (dense, 32 / 8 heads: 690 TFLOP/s at 2K tokens, 1,090 at 4K,
// 1,490 at 32K), and few heads leave SMs idle, since a unit's keys are not split (dense, 4K tokens, one
// head: 32 units, 51 us).  Every wait is bounded:
// by 200 ms, and where a warp sits out a whole unit by win_unit_wait_ns.
#include <limits.h>
#include <math.h>

#include "tmap.h"
#include "window.cuh"

namespace msa {
namespace {

constexpr int kTile = 128 * 128 * 2;  // 128 rows x 128 bf16, two SW128 panels
constexpr int kRing = 3;              // K / V ring slots (loads alternate K, V)
constexpr float kSlack = 8.f;         // log2 of the largest P kept without moving the row maximum

struct FwdArgs {
  WinDims d;
  KeyMaps k, v;
  CUtensorMap q, o;
  const bf16 *qp, *kp, *vp;  // the same tensors by address (mend_rows)
  bf16* op;
  float* lse;
  unsigned* status;
  int tiles;        // query tiles per unit, 1 or 2
  int nseg;         // units along a sequence
  int units;  // nseg B Hkv
  unsigned long long unit_ns;  // win_unit_wait_ns
  PackedTables p;              // packed form only; d.S is then the number of tokens
};
constexpr int kFwdThreads = 640;
struct FwdShared {
  float half[2][2][128];  // per tile, half and row: the half's maximum, later its row sum
  uint64_t q_full[2], q_empty[2], kv_full[kRing], kv_empty[kRing], s_full[2], p_full[2], o_full[2],
      o_free[2], st_full[2], mma_done;
  uint32_t tmem;
  int bad0, bad1;  // the block's first and last unit with an O that is not finite
};
struct FwdUnit {
  int b, g, t0;
  bool two;  // the second tile has a token
  KeyRun run;
};
template <int G, bool kPacked>
__device__ __forceinline__ FwdUnit fwd_unit(const FwdArgs& A, int u) {
  constexpr int TT = 128 / G;
  const WinDims& d = A.d;
  FwdUnit x;
  if (kPacked) {
    const int4 e = __ldg(A.p.fwd + u / d.Hkv);
    x.b = 0;
    x.g = u % d.Hkv;
    x.t0 = e.x;
    x.two = A.tiles == 2 && x.t0 + TT < d.S;
    const int t1 = x.t0 + TT * A.tiles - 1;
    x.run = packed_run(x.t0, t1 < d.S ? t1 : d.S - 1, e.y, e.z);
    return x;
  }
  const int per = d.B * d.Hkv;
  const int seg = u / per, rem = u % per;
  x.b = rem / d.Hkv;
  x.g = rem % d.Hkv;
  x.t0 = seg * TT * A.tiles;
  x.two = A.tiles == 2 && x.t0 + TT < d.S;
  const int t1 = x.t0 + TT * A.tiles - 1;
  x.run = key_run(d, x.t0, t1 < d.S ? t1 : d.S - 1);
  return x;
}

__device__ __forceinline__ bool finite4(uint2 w) {  // four bf16
  auto bad = [](uint32_t x) { return (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u; };
  return !(bad(w.x) || bad(w.y));
}
__device__ __forceinline__ float4 widen4(uint2 w) {
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}

// O rows again that an infinity or NaN has reached through a V row which the query does not see: a
// product of the tensor core takes whole tiles, and P = 0 times NaN is NaN.  A warp takes a token and
// its group's heads, four dims a lane, and adds up the visible keys alone.  Only rows with an LSE (masked
// scores never enter it: without one the row's own scores are not finite), with such a V row among the few
// that their tiles hold unseen, and with none that they see are computed again; the others stay as they
// are, so a run that has diverged costs a look at its rows.  Runs behind the block's last store and only
// where an epilogue met a value that is not finite: 754 us at 32K tokens with it, 748 without, 1,069 and 1,096
// at 64K, 217 and 219 at 2 x 8192 (inlined; as a function call 760, 1,081 and 221).
template <int G, bool kPacked>
__device__ __forceinline__ void mend_rows(const FwdArgs& A, int u) {
  constexpr int TT = 128 / G;
  const WinDims& d = A.d;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const FwdUnit unit = fwd_unit<G, kPacked>(A, u);
  const int b = unit.b, g = unit.g, t0 = unit.t0;
  const float sl2 = d.scale * kLog2e;
  const long long seq = (long long)b * d.S, lse_rows = kPacked ? A.p.rows : d.S;
  const int t1 = t0 + TT * A.tiles - 1 < d.S ? t0 + TT * A.tiles - 1 : d.S - 1;
  const KeyRun run = unit.run;
  auto kv_row = [&](const bf16* x, int key) {
    return __ldg(reinterpret_cast<const uint2*>(x + ((seq + key) * d.Hkv + g) * kD) + lane);
  };
  auto v_finite = [&](auto key_of, int n) {  // V rows key_of(0) .. key_of(n - 1), four at a time
    for (int x = 0; x < n; x += 4) {
      bool ok = true;
#pragma unroll
      for (int e = 0; e < 4; ++e) ok &= finite4(kv_row(A.vp, key_of(x + e < n ? x + e : n - 1)));
      if (!__all_sync(0xffffffffu, ok)) return false;
    }
    return true;
  };
  for (int t = t0 + warp; t <= t1; t += kFwdThreads / 32) {
    const int w0 = kPacked ? A.p.lo[t] : t - d.W + 1 > 0 ? t - d.W + 1 : 0;
    const int far = kPacked ? 0 : d.ns < w0 ? d.ns : w0;  // sinks before the window
    const int keys = far + t - w0 + 1;
    auto key_of = [&](int x) { return x < far ? x : w0 + x - far; };
    // unseen in the unit's tiles: in front of the window (sinks are zero-filled to eight, see make_key_maps), and
    // behind the token up to the last tile's end
    const int c0 = kPacked || run.ws ? run.ws : d.ns, n0 = w0 - c0, n1 = (t1 + kBlock < d.S ? t1 + kBlock : d.S) - t - 1;
    bool look = true;
    for (int h = g * G; h < g * G + G; ++h) {
      const long long row = ((seq + t) * d.Hq + h) * kD;
      if (__all_sync(0xffffffffu, finite4(__ldcg(reinterpret_cast<const uint2*>(A.op + row) + lane)))) continue;
      if (!isfinite(__ldcg(A.lse + ((long long)b * d.Hq + h) * lse_rows + t))) continue;
      if (look && ((v_finite([&](int x) { return c0 + x; }, n0) && v_finite([&](int x) { return t + 1 + x; }, n1)) ||
                   !v_finite(key_of, keys)))
        break;  // for every head of the group
      look = false;
      {
        const float4 q = widen4(__ldg(reinterpret_cast<const uint2*>(A.qp + row) + lane));
        float m = -INFINITY, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int x = 0; x < keys; x += 4) {
          float s[4];
          uint2 v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key_of(x + e < keys ? x + e : keys - 1);
            const float4 k = widen4(kv_row(A.kp, key));
            v[e] = kv_row(A.vp, key);
            s[e] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)));
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] += __shfl_xor_sync(0xffffffffu, s[e], off);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[e] = x + e < keys ? s[e] * sl2 : -INFINITY;
          const float mn = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), m), alpha = exp2_ftz(m - mn);
          m = mn;
          l *= alpha;
          acc.x *= alpha;
          acc.y *= alpha;
          acc.z *= alpha;
          acc.w *= alpha;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = exp2_ftz(s[e] - mn);
            const float4 f = widen4(v[e]);
            l += p;
            acc.x = fmaf(p, f.x, acc.x);
            acc.y = fmaf(p, f.y, acc.y);
            acc.z = fmaf(p, f.z, acc.z);
            acc.w = fmaf(p, f.w, acc.w);
          }
        }
        const float sc = 1.f / l;
        reinterpret_cast<uint2*>(A.op + row)[lane] =
            make_uint2(pack_bf16(acc.x * sc, acc.y * sc), pack_bf16(acc.z * sc, acc.w * sc));
      }
    }
  }
}

}  // namespace

template <int G, bool kPacked>
__global__ void __launch_bounds__(kFwdThreads, 1) win_fwd_kernel(const __grid_constant__ FwdArgs A) {
  using namespace sm100;
  constexpr int TT = 128 / G;
  const WinDims& d = A.d;
  extern __shared__ __align__(1024) uint8_t smem_tiles[];
  uint8_t* sQ = smem_tiles;      // [2 units][2 tiles][128 rows][128 d]
  uint8_t* sR = sQ + 4 * kTile;  // K / V ring
  FwdShared* sh = reinterpret_cast<FwdShared*>(sR + kRing * kTile);
  const uint32_t aQ = smem_u32(sQ), aR = smem_u32(sR);
  const int tid = threadIdx.x, lane = tid % 32, warp = warp_number();
  const float sl2 = d.scale * kLog2e;
  clear_status(A.status);
  if (aQ & 1023u) {  // the swizzled operand layout needs 1024-byte atoms
    if (tid == 0) atomicOr(A.status, kStatusInternal);
    return;
  }

  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sh->q_full[x], 1);
      mbar_init(&sh->q_empty[x], 2);  // the store warps of both tiles
      mbar_init(&sh->s_full[x], 1);
      mbar_init(&sh->p_full[x], 8);
      mbar_init(&sh->o_full[x], 1);
      mbar_init(&sh->o_free[x], 8);
      mbar_init(&sh->st_full[x], 8);
    }
    for (int x = 0; x < kRing; ++x) {
      mbar_init(&sh->kv_full[x], 1);
      mbar_init(&sh->kv_empty[x], 1);
    }
    mbar_init(&sh->mma_done, 1);
    sh->bad0 = INT_MAX;
    sh->bad1 = -1;
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
  const uint32_t tmem = sh->tmem;
  const uint32_t S0 = tmem, O0 = tmem + 256;  // S_X = S0 + 128 X, O_X = O0 + 128 X

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA loads
    if (lane == 0) {
      bool ok = true;
      long long nl = 0, nu = 0, nq = 0;  // K / V loads, units, units whose Q was asked for
      Ring<kRing> kv;
      for (int u = blockIdx.x; u < A.units && ok; u = unit_at<kPacked>((int)++nu)) {
        const FwdUnit x = fwd_unit<G, kPacked>(A, u);
        const int qs = (int)(nu & 1);
        if (nu >= 2 && !mbar_wait(&sh->q_empty[qs], phase_of(nu / 2 - 1), A.status)) break;
        uint8_t* dq = sQ + qs * 2 * kTile;
        mbar_expect_tx(&sh->q_full[qs], (x.two ? 2 : 1) * kTile);
        for (int X = 0; X < (x.two ? 2 : 1); ++X)
          for (int c = 0; c < 2; ++c)
            tma_load_rows(dq + X * kTile + c * (kTile / 2), &A.q, 64 * c, x.g * G, x.t0 + X * TT, x.b,
                          &sh->q_full[qs]);
        ++nq;
        for (int n = 0; n < x.run.nb && ok; ++n)
          for (int w = 0; w < 2; ++w, ++nl, kv.next()) {  // K_n, then V_n
            if (kv.wrapped && !mbar_wait(&sh->kv_empty[kv.slot], kv.phase ^ 1, A.status)) {
              ok = false;
              break;
            }
            mbar_expect_tx(&sh->kv_full[kv.slot], kTile);
            load_key_tile(sR + kv.slot * kTile, w ? A.v : A.k, x.run, n, x.g, x.b, &sh->kv_full[kv.slot]);
          }
      }
      // no copy may still be landing in shared memory when the block exits
      for (long long x = nl >= kRing ? nl - kRing : 0; x < nl; ++x)
        mbar_wait(&sh->kv_full[x % kRing], phase_of(x / kRing), A.status);
      for (long long x = nq >= 2 ? nq - 2 : 0; x < nq; ++x)
        mbar_wait(&sh->q_full[x & 1], phase_of(x >> 1), A.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issue
    {
      int cs[2] = {0, 0};  // S products issued per tile
      int cu[2] = {0, 0};  // units begun per tile (o_free phases)
      Ring<kRing> kv;
      int v_slot = 0;  // the last V and its phase
      uint32_t v_phase = 0;
      bool ok = true;
      // O_X += P_X V for the last S product of tile X
      auto mma_o = [&](int X, bool first, bool last, bool free_v, int keys) -> bool {
        if (!mbar_wait_warp(&sh->p_full[X], phase_of(cs[X] - 1), A.status)) return false;
        if (first) {
          if (cu[X] > 0 && !mbar_wait_warp(&sh->o_free[X], phase_of(cu[X] - 1), A.status)) return false;
          ++cu[X];
        }
        if (!mbar_wait_warp(&sh->kv_full[v_slot], v_phase, A.status)) return false;
        fence_after_sync();
        if (keys >= kBlock) mma_tn<4, 64>(O0 + 128 * X, S0 + 128 * X, aR + v_slot * kTile, !first);
        else mma_tn_part<4, 64>(O0 + 128 * X, S0 + 128 * X, aR + v_slot * kTile, !first, keys);
        if (last) warp_mma_commit(&sh->o_full[X]);
        if (free_v) warp_mma_commit(&sh->kv_empty[v_slot]);
        return true;
      };
      auto mma_s = [&](int X, uint32_t q, int kslot, bool free_k, int keys) {
        fence_after_sync();
        if (keys >= kBlock) mma_kk(S0 + 128 * X, q + X * kTile, aR + kslot * kTile, false);  // S = Q K^T
        else mma_kk_part(S0 + 128 * X, q + X * kTile, aR + kslot * kTile, keys);
        warp_mma_commit(&sh->s_full[X]);
        if (free_k) warp_mma_commit(&sh->kv_empty[kslot]);
        ++cs[X];
      };
      int nu = 0;
      for (int u = blockIdx.x; u < A.units && ok; u = unit_at<kPacked>(++nu)) {
        const FwdUnit x = fwd_unit<G, kPacked>(A, u);
        const int qs = nu & 1;
        const uint32_t q = aQ + qs * 2 * kTile;
        if (!mbar_wait_warp(&sh->q_full[qs], phase_of(nu >> 1), A.status)) break;
        for (int n = 0; n < x.run.nb; ++n) {
          const int kslot = kv.slot, keys = x.run.keys(n);
          if (n > 0 && !mma_o(0, n == 1, false, !x.two, kBlock)) { ok = false; break; }
          // (K_n is waited for behind O_A(n-1): its load began when O_B(n-2) freed a slot)
          if (!mbar_wait_warp(&sh->kv_full[kslot], kv.phase, A.status)) { ok = false; break; }
          mma_s(0, q, kslot, !x.two, keys);
          if (x.two) {
            if (n > 0 && !mma_o(1, n == 1, false, true, kBlock)) { ok = false; break; }
            mma_s(1, q, kslot, true, keys);
          }
          kv.next();
          v_slot = kv.slot;
          v_phase = kv.phase;
          kv.next();
        }
        if (!ok) break;
        const int rest = x.run.keys(x.run.nb - 1);
        ok = mma_o(0, x.run.nb == 1, true, !x.two, rest) && (!x.two || mma_o(1, x.run.nb == 1, true, true, rest));
      }
      warp_mma_commit(&sh->mma_done);
      mbar_wait_warp(&sh->mma_done, 0, A.status);  // no product may still write tensor memory
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---------------------------------------------------------------- TMA stores of O
    if (lane == 0) {
      const int X = warp - 2;
      long long nu = 0, ns = 0;
      for (int u = blockIdx.x; u < A.units; u = unit_at<kPacked>((int)++nu)) {
        const FwdUnit x = fwd_unit<G, kPacked>(A, u);
        const int qs = (int)(nu & 1);
        if (X == 0 || x.two) {
          if (!mbar_wait(&sh->st_full[X], phase_of(ns++), A.status, A.unit_ns)) break;
          const uint32_t src = aQ + (qs * 2 + X) * kTile;
          tma_store_rows(&A.o, src, 0, x.g * G, x.t0 + X * TT, x.b);
          tma_store_rows(&A.o, src + kTile / 2, 64, x.g * G, x.t0 + X * TT, x.b);
          bulk_store_commit();
          bulk_store_wait_read();
        } else if (!mbar_wait(&sh->q_full[qs], phase_of(nu >> 1), A.status, A.unit_ns)) {
          break;  // (waited for only so that this arrival cannot run ahead into a later phase)
        }
        mbar_arrive(&sh->q_empty[qs]);
      }
      bulk_store_wait();
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax + epilogue
    const int X = (warp - 4) >> 3;         // tile A (warps 4-11) or B (warps 12-19)
    const int hf = ((warp - 4) >> 2) & 1;  // columns 64 hf .. 64 hf + 63
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // tile row = tensor-memory lane
    const uint32_t lb = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t Sx = S0 + 128 * X + 64 * hf + lb, Ox = O0 + 128 * X + 64 * hf + lb;
    const float2 sl2x2 = make_float2(sl2, sl2);
    const int bar = 1 + X * 4 + quad;  // named barrier of the two warps that share these rows
    float* mine = &sh->half[X][hf][r];
    const float* other = &sh->half[X][hf ^ 1][r];
    int cs = 0, nu = 0, nt = 0;  // S products, units, units with this tile
    // Both warps of a pair pass the same barriers whatever happens: a wait that gives up only clears
    // `ok` (warp-uniform), which skips the later waits.
    bool ok = true;
    for (int u = blockIdx.x; u < A.units; u = unit_at<kPacked>(++nu)) {
      const FwdUnit x = fwd_unit<G, kPacked>(A, u);
      if (X == 1 && !x.two) continue;
      const int t = x.t0 + X * TT + r / G;  // this row's token
      const int t_lo = kPacked ? __ldg(A.p.lo + (t < d.S ? t : d.S - 1)) : 0;
      float mr = -INFINITY, l = 0.f;
      for (int n = 0; n < x.run.nb; ++n, ++cs) {
        // (the masks cost about as many instructions as the exponentials: only where a tile needs them)
        const bool full = n >= x.run.f0 && n <= x.run.f1;
        uint32_t v0 = 0xffffffffu, v1 = v0;
        if (!full) {
          uint32_t vis[4];
          if (kPacked) visible_cols_packed(x.run, n, t, t_lo, vis);
          else visible_cols(d, x.run, n, t, vis);
          v0 = hf ? vis[2] : vis[0];
          v1 = hf ? vis[3] : vis[1];
        }
        if (ok) ok = mbar_wait_warp(&sh->s_full[X], phase_of(cs), A.status);
        fence_after_sync();
        uint32_t s0[32], s1[32];
        tmem_ld32(Sx, s0);
        tmem_ld32(Sx + 32, s1);
        tmem_wait_ld();
        float mx = -INFINITY;
        if (full) {
#pragma unroll
          for (int c = 0; c < 32; ++c) mx = fmax3(mx, __uint_as_float(s0[c]), __uint_as_float(s1[c]));
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            mx = fmax3(mx, (v0 >> c) & 1u ? __uint_as_float(s0[c]) : -INFINITY,
                       (v1 >> c) & 1u ? __uint_as_float(s1[c]) : -INFINITY);
        }
        if (bar_or(bar, 64, (mx - mr) * sl2 > kSlack || n == 0)) {  // (both -inf: NaN, no)
          *mine = mx;
          bar_sync(bar, 64);
          mx = fmaxf(mx, *other);
          if (n == 0) {
            mr = mx;
          } else if (__any_sync(0xffffffffu, (mx - mr) * sl2 > kSlack)) {
            // rescale this half of O and l of the rows that need it
            const bool need = (mx - mr) * sl2 > kSlack;
            const float alpha = need ? exp2_ftz((mr - mx) * sl2) : 1.f;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t v[16];
              tmem_ld16(Ox + q * 16, v);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * alpha);
              tmem_st16(Ox + q * 16, v);
            }
            l *= alpha;
            if (need) mr = mx;
          }
        }
        const float mb = mr == -INFINITY ? 0.f : mr * sl2;
        const float2 nmb = make_float2(-mb, -mb);
        float2 la = make_float2(0.f, 0.f);
        auto exps = [&](const uint32_t (&s)[32], uint32_t vw, uint32_t at) {
          uint32_t pw[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float2 e = ffma2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2x2, nmb);
            float2 p = make_float2(exp2_ftz(e.x), exp2_ftz(e.y));
            if (!full) {
              p.x = (vw >> (2 * c)) & 1u ? p.x : 0.f;
              p.y = (vw >> (2 * c + 1)) & 1u ? p.y : 0.f;
            }
            la = fadd2(la, p);
            pw[c] = pack_bf16(p.x, p.y);
          }
          tmem_st16(at, pw);
        };
        exps(s0, v0, Sx);
        // the second 32 columns again: kept in registers all along, they made the compiler spill
        tmem_ld32(Sx + 32, s1);
        tmem_wait_ld();
        exps(s1, v1, Sx + 16);
        l += la.x + la.y;
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->p_full[X]);
      }
      // ---- unit end: O / l into the tile's own Q rows (every S product has read them), as the
      // swizzled tile its TMA store expects; then the LSE
      if (ok) ok = mbar_wait_warp(&sh->o_full[X], phase_of(nt), A.status);
      ++nt;
      *mine = l;  // (the other warp has read this thread's last maximum: O is there)
      bar_sync(bar, 64);
      l += *other;
      fence_after_sync();
      const float sc = __fdividef(1.f, l);
      const uint32_t dst = aQ + ((nu & 1) * 2 + X) * kTile + hf * (kTile / 2);
      uint32_t v0[32], v1[32];
      tmem_ld32(Ox, v0);
      tmem_ld32(Ox + 32, v1);
      tmem_wait_ld();
      fence_before_sync();  // O_X may now take the next unit's products
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->o_free[X]);
      float nf = 0.f;  // NaN where a value is not finite
#pragma unroll
      for (int c = 0; c < 32; ++c) nf = fmaf(__uint_as_float(v0[c]), 0.f, fmaf(__uint_as_float(v1[c]), 0.f, nf));
      if (nf != 0.f) {
        atomicMin(&sh->bad0, nu);
        atomicMax(&sh->bad1, nu);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const uint32_t(&v)[32] = c < 4 ? v0 : v1;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_bf16(__uint_as_float(v[8 * (c & 3) + 2 * e]) * sc, __uint_as_float(v[8 * (c & 3) + 2 * e + 1]) * sc);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(dst + sw128_chunk(r, c)), "r"(w[0]),
                     "r"(w[1]), "r"(w[2]), "r"(w[3])
                     : "memory");
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->st_full[X]);
      if (hf == 0 && t < d.S)
        A.lse[((long long)x.b * d.Hq + x.g * G + r % G) * (kPacked ? A.p.rows : d.S) + t] = (mr * sl2 + __log2f(l)) * kLn2;
    }
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, 512);
  if (kPacked && A.p.rows > d.S) {  // the rows behind the last sequence
    const long long pad = A.p.rows - d.S, at = (long long)blockIdx.x * kFwdThreads + tid, step = (long long)gridDim.x * kFwdThreads;
    uint4* o = reinterpret_cast<uint4*>(A.op + (long long)d.S * d.Hq * kD);
    for (long long i = at; i < pad * d.Hq * (kD / 8); i += step) o[i] = make_uint4(0u, 0u, 0u, 0u);
    for (long long i = at; i < pad * d.Hq; i += step) A.lse[i / pad * A.p.rows + d.S + i % pad] = -INFINITY;
  }
  for (int nu = sh->bad0; nu <= sh->bad1; ++nu) mend_rows<G, kPacked>(A, unit_at<kPacked>(nu));
}

// The maps of K or V.  Those of sinks end at the last one, so that the rows up to a multiple of eight, which
// most queries do not see, are zeros.  nsp mod 128 rows of the shared tile are sinks (0: there is no
// such tile, and its two maps are not used).
bool make_key_maps(const WinDims& d, const void* base, KeyMaps* m) {
  const int a = d.nsp % kBlock;
  if (!make_tmap_rows(&m->full, base, d.B, d.S, d.Hkv, 1, kBlock)) return false;
  m->head = m->sink = m->rest = m->full;
  return (d.nsp < kBlock || make_tmap_rows(&m->head, base, d.B, d.S, d.Hkv, 1, kBlock, d.ns)) &&
         (a == 0 || (make_tmap_rows(&m->sink, base, d.B, d.S, d.Hkv, 1, a, d.ns) &&
                     make_tmap_rows(&m->rest, base, d.B, d.S, d.Hkv, 1, kBlock - a)));
}

// A unit's walk grows with the window: 65536 tiles at S = 2^23, 1.6 us each at 2,070 MHz and 2.2 at 1,507,
// so a warp that waits for the end of one gets 25 us a tile beside the 200 ms of every wait.
unsigned long long win_unit_wait_ns(const WinDims& d) {
  const long long keys = (long long)d.nsp + d.W + 2 * kBlock < d.S ? (long long)d.nsp + d.W + 2 * kBlock : d.S;
  return 200000000ull + 25000ull * (unsigned long long)(keys / kBlock + 1);
}

template <int G, bool kPacked>
static void win_fwd_g(const FwdArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(FwdShared) + (4 + kRing) * (size_t)kTile;
  allow_smem<win_fwd_kernel<G, kPacked>>(smem);
  const int n = num_sms();
  win_fwd_kernel<G, kPacked><<<a.units < n ? a.units : n, kFwdThreads, smem, st>>>(a);
}

template <bool kPacked>
static bool win_fwd_any(const FwdArgs& a, cudaStream_t st) {
  switch (a.d.G) {
    case 1: win_fwd_g<1, kPacked>(a, st); break;
    case 2: win_fwd_g<2, kPacked>(a, st); break;
    case 4: win_fwd_g<4, kPacked>(a, st); break;
    case 8: win_fwd_g<8, kPacked>(a, st); break;
    case 16: win_fwd_g<16, kPacked>(a, st); break;
    default: return false;
  }
  return true;
}

bool launch_win_fwd(const WinDims& d, const void* q, const void* k, const void* v, void* o,
                    float* lse, unsigned* status, cudaStream_t st) {
  FwdArgs a;
  if (!make_key_maps(d, k, &a.k) || !make_key_maps(d, v, &a.v) ||
      !make_tmap_rows(&a.q, q, d.B, d.S, d.Hq, d.G, kBlock / d.G) ||
      !make_tmap_rows(&a.o, o, d.B, d.S, d.Hq, d.G, kBlock / d.G))
    return false;
  a.d = d;
  a.qp = (const bf16*)q;
  a.kp = (const bf16*)k;
  a.vp = (const bf16*)v;
  a.op = (bf16*)o;
  a.lse = lse;
  a.status = status;
  a.unit_ns = win_unit_wait_ns(d);
  const int tt = kBlock / d.G;
  const long long per = (long long)d.B * d.Hkv;
  a.tiles = (d.S + 2 * tt - 1) / (2 * tt) * per < num_sms() ? 1 : 2;
  a.nseg = (d.S + tt * a.tiles - 1) / (tt * a.tiles);
  a.units = (int)(a.nseg * per);
  return win_fwd_any<false>(a, st);
}

bool launch_packed_fwd(const PackedDims& x, const PackedTables& p, const void* q, const void* k, const void* v, void* o,
                       float* lse, unsigned* status, cudaStream_t st) {
  const WinDims& d = x.d;
  FwdArgs a{};
  // (maps that end with the last sequence: rows behind it read as zeros and are not written)
  if (!make_key_maps(d, k, &a.k) || !make_key_maps(d, v, &a.v) ||
      !make_tmap_rows(&a.q, q, 1, d.S, d.Hq, d.G, kBlock / d.G) || !make_tmap_rows(&a.o, o, 1, d.S, d.Hq, d.G, kBlock / d.G))
    return false;
  a.d = d;
  a.p = p;
  a.qp = (const bf16*)q;
  a.kp = (const bf16*)k;
  a.vp = (const bf16*)v;
  a.op = (bf16*)o;
  a.lse = lse;
  a.status = status;
  a.unit_ns = win_unit_wait_ns(d);
  a.tiles = x.fwd_tiles;
  a.units = x.fwd_units * d.Hkv;
  return win_fwd_any<true>(a, st);
}

}  // namespace msa
