// The plan of packed sequences: which keys every token sees, and the work units of the packed forward and backward
// (window.cuh) in the order that they are dealt in.
//
// The lengths are known on the host and travel to the device as kernel arguments, so a plan needs no copy from
// host memory and no wait, and a captured graph holds the lengths it was captured with.  packed_plan_kernel, one launch
// for up to kSeqs sequences, writes lo(t) and hi(t); three blocks of the last launch cut the units and sort them by the
// length of their walks (a counting sort in shared memory): costs differ from unit to unit by the sequences' lengths, and
// the longest must not come last.  They find lo and hi of the tokens that they look at for themselves where all sequences
// are in their launch, and else in the tables of the launches before.  Bound by latency: 7 us for 20 sequences of 700
// tokens as for 30 of 16384.
//
// The attention kernels themselves (win_fwd.cu, win_bwd.cu), 16347 tokens of 30 sequences up to 4096, 32 / 8 heads, visible
// pairs: forward 230 us (1,190 TFLOP/s), dQ 315 (1,300 of its three products), dK/dV 375 (1,460 of its four), row data 65.
// Sequences of one length L at 16384 tokens, forward / dQ / dK and dV in us: L = 64: 67 / 109 / 99, 512: 95 / 142 / 152,
// 1024: 135 / 206 / 224, 2048: 214 / 325 / 367, 4096: 379 / 585 / 661, 8192: 739 / 1157 / 1272 (1,490 / 1,430 / 1,730 TFLOP/s).
// A unit costs 3.4 us beside its key tiles (1.46 us each for two query tiles): its first tile's chain, masks, epilogue.
// Tried and not kept: the next unit's first products between the last ones (230), the epilogue behind the next unit's first
// tile (236: its Q buffer is then free too late).
#include "window.cuh"

namespace msa {
namespace {

constexpr int kSeqs = 960;  // sequences of one launch: 3.8 KB of arguments
struct Starts {
  int n, at[kSeqs + 1];
};
constexpr int kBins = 1024;

struct UnitArgs {
  PackedDims x;
  const int32_t *lo, *hi;
  int4 *fwd, *dq, *items, *joins;
  int* first;
  int shift, shift2;  // of the costs of units (key tiles) and items (query tiles), to fit the bins
};

// {lo, hi} of token t, one of the n sequences that begin at at[0] .. at[n - 1].
__device__ __forceinline__ int2 seen(const int* at, int n, int W, int t) {
  int a = 0, z = n;  // at[a] <= t < at[z]
  while (z - a > 1) {
    const int m = (a + z) / 2;
    if (at[m] <= t) a = m;
    else z = m;
  }
  const int t0 = at[a], t1 = at[a + 1];
  return make_int2(t - t0 >= W ? t - W + 1 : t0, t1 - t > W ? t + W - 1 : t1 - 1);
}

// Items of a key block that nt query tiles see, of equal length; one up to a quarter above the aim.
__host__ __device__ inline int packed_pieces(int nt, int chunk) {
  return nt <= chunk + chunk / 4 ? 1 : (nt + chunk - 1) / chunk;
}

// Sorts by descending cost: f(i, emit) calls emit(cost, write) for every entry of source i.  The order among equal
// costs is free (no result depends on it).
template <typename F>
__device__ __forceinline__ void deal(int n, int shift, int* bins, F&& f) {
  const int tid = threadIdx.x;
  for (int b = tid; b < kBins; b += blockDim.x) bins[b] = 0;
  __syncthreads();
  auto bin = [&](int cost) {
    const int c = cost >> shift;
    return kBins - 1 - (c < kBins ? c : kBins - 1);
  };
  for (int i = tid; i < n; i += blockDim.x) f(i, [&](int cost, auto&&) { atomicAdd(&bins[bin(cost)], 1); });
  __syncthreads();
  // exclusive sum over the bins: blockDim.x = kBins, a thread a bin
  __shared__ int sums[32];
  const int own = bins[tid];
  int s = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, off);
    if (tid % 32 >= off) s += y;
  }
  if (tid % 32 == 31) sums[tid / 32] = s;
  __syncthreads();
  if (tid < 32) {
    int v = sums[tid];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, off);
      if (tid >= off) v += y;
    }
    sums[tid] = v;
  }
  __syncthreads();
  bins[tid] = s - own + (tid >= 32 ? sums[tid / 32 - 1] : 0);
  __syncthreads();
  for (int i = tid; i < n; i += blockDim.x) f(i, [&](int cost, auto&& write) { write(atomicAdd(&bins[bin(cost)], 1)); });
  __syncthreads();
}

// units: with block 0 for the forward's, 1 for dQ's, 2 for the key-outer items (one: the launch has all sequences, s.n of
// them); the other blocks write the tokens' tables.
__global__ void __launch_bounds__(kBins) packed_plan_kernel(const __grid_constant__ UnitArgs A, const __grid_constant__ Starts s,
                                                            bool units, bool one, int32_t* to_lo, int32_t* to_hi) {
  __shared__ int bins[kBins], slots, joins, at[kSeqs + 1];
  const WinDims& d = A.x.d;
  const int tt = kBlock / d.G;
  if (one || !units)
    for (int i = threadIdx.x; i <= s.n; i += kBins) at[i] = s.at[i];
  __syncthreads();
  if (!units || blockIdx.x >= 3) {
    const int first = units ? 3 : 0, step = ((int)gridDim.x - first) * kBins;
    for (int t = at[0] + ((int)blockIdx.x - first) * kBins + (int)threadIdx.x; t < at[s.n]; t += step) {
      const int2 e = seen(at, s.n, d.W, t);
      to_lo[t] = e.x;
      to_hi[t] = e.y;
    }
    return;
  }
  auto lo_of = [&](int t) { return one ? seen(at, s.n, d.W, t).x : A.lo[t]; };
  auto hi_of = [&](int t) { return one ? seen(at, s.n, d.W, t).y : A.hi[t]; };
  if (threadIdx.x == 0) slots = joins = 0;
  if (blockIdx.x < 2) {
    const int per = blockIdx.x == 0 ? tt * A.x.fwd_tiles : tt;
    int4* out = blockIdx.x == 0 ? A.fwd : A.dq;
    deal((d.S + per - 1) / per, A.shift, bins, [&](int i, auto&& emit) {
      const int t0 = i * per, t1 = min(t0 + per, d.S) - 1, lo = lo_of(t0);
      emit((t1 - lo) / kBlock, [&](int at) { out[at] = make_int4(t0, lo, lo_of(t1), 0); });
    });
    return;
  }
  const int nblk = (d.S + kBlock - 1) / kBlock;
  int* first = A.first;  // slot of a split block's first item
  __syncthreads();
  for (int n = threadIdx.x; n < nblk; n += blockDim.x) {
    const int k0 = n * kBlock, nt = (hi_of(min(k0 + kBlock, d.S) - 1) - k0) / tt + 1, nc = packed_pieces(nt, A.x.chunk);
    if (nc == 1) continue;
    first[n] = atomicAdd(&slots, nc);
    A.joins[atomicAdd(&joins, 1)] = make_int4(n, first[n], nc, 0);
  }
  __syncthreads();
  deal(nblk, A.shift2, bins, [&](int n, auto&& emit) {
    const int k0 = n * kBlock, hi0 = hi_of(k0), nt = (hi_of(min(k0 + kBlock, d.S) - 1) - k0) / tt + 1;
    const int nc = packed_pieces(nt, A.x.chunk), step = (nt + nc - 1) / nc, s0 = nc > 1 ? first[n] : -1;
    for (int c = 0; c < nc; ++c) {
      const int i0 = min(c * step, nt), i1 = min(i0 + step, nt);
      emit(i1 - i0, [&](int at) {
        A.items[2 * at] = make_int4(n, i0, i1, nc > 1 ? s0 + c : -1);
        A.items[2 * at + 1] = make_int4(hi0, 0, 0, 0);
      });
    }
  });
}

struct Layout {
  size_t lo, hi, fwd, dq, items, joins, first, bytes;
};
Layout layout(const PackedDims& x) {
  Layout l;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t a = at;
    at += (n + 255) / 256 * 256;
    return a;
  };
  l.lo = take((size_t)x.d.S * 4);
  l.hi = take((size_t)x.d.S * 4);
  l.fwd = take((size_t)x.fwd_units * sizeof(int4));
  l.dq = take((size_t)x.dq_units * sizeof(int4));
  l.items = take((size_t)x.items * 2 * sizeof(int4));
  l.joins = take((size_t)x.joins * sizeof(int4));
  l.first = take((size_t)((x.d.S + kBlock - 1) / kBlock) * 4);
  l.bytes = at;
  return l;
}

// The rows behind the last sequence: zeros, and -inf in lse (launched where there is no sequence at all).
struct PadArgs {
  uint4* rows[3];    // from the first such row on
  long long n[3];    // 16-byte pieces
  float* lse;        // [Hq, rows] or NULL
  int Hq, tokens;
  long long stride;
};
__global__ void __launch_bounds__(256) packed_pad_kernel(const __grid_constant__ PadArgs A) {
  const long long at = (long long)blockIdx.x * 256 + threadIdx.x, step = (long long)gridDim.x * 256;
#pragma unroll
  for (int x = 0; x < 3; ++x)
    for (long long i = at; i < A.n[x]; i += step) A.rows[x][i] = make_uint4(0u, 0u, 0u, 0u);
  if (!A.lse) return;
  const long long pad = A.stride - A.tokens;
  for (long long i = at; i < pad * A.Hq; i += step) A.lse[i / pad * A.stride + A.tokens + i % pad] = -INFINITY;
}

}  // namespace

// a, b, c: tensors of `heads` rows of 128 a token, NULL: none.
void launch_packed_pad(const PackedDims& x, void* a, int ha, void* b, int hb, void* c, int hc, float* lse, cudaStream_t st) {
  void* t[3] = {a, b, c};
  const int h[3] = {ha, hb, hc};
  PadArgs p{};
  long long most = 1;
  for (int i = 0; i < 3; ++i) {
    p.rows[i] = static_cast<uint4*>(t[i]) + (t[i] ? (long long)x.d.S * h[i] * (kD / 8) : 0);
    p.n[i] = t[i] ? (x.rows - x.d.S) * h[i] * (kD / 8) : 0;
    most = p.n[i] > most ? p.n[i] : most;
  }
  p.lse = lse;
  p.Hq = x.d.Hq;
  p.tokens = x.d.S;
  p.stride = x.rows;
  const long long g = (most + 255) / 256, cap = (long long)num_sms() * 8;
  packed_pad_kernel<<<(int)(g < cap ? g : cap), 256, 0, st>>>(p);
}

// The key-outer items are cut such that none has more than half of an SM's share of all query tiles: dealt longest
// first, they then even out, and few blocks leave partials (128 KB a slot and KV head, written and read).
void packed_count(const int32_t* lengths, int n, PackedDims* x) {
  const WinDims& d = x->d;
  const int tt = kBlock / d.G, nblk = (d.S + kBlock - 1) / kBlock;
  const long long pairs = (d.S + 2 * tt - 1) / (2 * tt);
  x->fwd_tiles = pairs * d.Hkv < num_sms() ? 1 : 2;
  x->fwd_units = (int)((d.S + tt * x->fwd_tiles - 1) / (tt * x->fwd_tiles));
  x->dq_units = (d.S + tt - 1) / tt;
  auto blocks = [&](auto&& f) {  // f(query tiles) of every key block
    long long start = 0;
    int i = 0;
    for (int b = 0; b < nblk; ++b) {
      const long long last = (long long)(b + 1) * kBlock < d.S ? (long long)(b + 1) * kBlock - 1 : d.S - 1;
      while (start + lengths[i] <= last) start += lengths[i++];  // the sequence of the block's last key
      const long long end = start + lengths[i] - 1;
      const long long hi = last + d.W - 1 < end ? last + d.W - 1 : end;
      f((hi - (long long)b * kBlock) / tt + 1);
    }
  };
  long long total = 0;
  blocks([&](long long nt) { total += nt; });
  const long long share = total * d.Hkv / (2ll * num_sms());
  x->chunk = (int)(share < 4 ? 4 : share);
  x->items = x->slots = x->joins = 0;
  blocks([&](long long nt) {
    const int nc = packed_pieces((int)nt, x->chunk);
    x->items += nc;
    x->slots += nc > 1 ? nc : 0;
    x->joins += nc > 1;
  });
}

size_t packed_table_bytes(const PackedDims& x) { return layout(x).bytes; }

PackedTables packed_tables(const PackedDims& x, const void* table) {
  const Layout l = layout(x);
  const char* p = static_cast<const char*>(table);
  PackedTables t;
  t.lo = reinterpret_cast<const int32_t*>(p + l.lo);
  t.hi = reinterpret_cast<const int32_t*>(p + l.hi);
  t.fwd = reinterpret_cast<const int4*>(p + l.fwd);
  t.dq = reinterpret_cast<const int4*>(p + l.dq);
  t.items = reinterpret_cast<const int4*>(p + l.items);
  t.joins = reinterpret_cast<const int4*>(p + l.joins);
  t.rows = x.rows;
  return t;
}

// (of n sequences, empty ones not counted)
int packed_launches(int n) { return n <= kSeqs ? 1 : (n + kSeqs - 1) / kSeqs + 1; }

void launch_packed_plan(const PackedDims& x, const int32_t* lengths, int n, void* table, cudaStream_t st) {
  const PackedTables p = packed_tables(x, table);
  UnitArgs a;
  a.x = x;
  a.lo = p.lo;
  a.hi = p.hi;
  a.fwd = const_cast<int4*>(p.fwd);
  a.dq = const_cast<int4*>(p.dq);
  a.items = const_cast<int4*>(p.items);
  a.joins = const_cast<int4*>(p.joins);
  a.first = reinterpret_cast<int*>(static_cast<char*>(table) + layout(x).first);
  a.shift = a.shift2 = 0;
  while ((x.d.S / kBlock + 1) >> a.shift >= kBins) ++a.shift;
  while (x.dq_units >> a.shift2 >= kBins) ++a.shift2;
  int32_t *lo = const_cast<int32_t*>(p.lo), *hi = const_cast<int32_t*>(p.hi);
  Starts s;
  int at = 0, filled = 0;
  for (int i = 0; i < n; ++i) filled += lengths[i] > 0;
  const bool one = filled <= kSeqs;
  for (int i = 0; i < n && at < x.d.S;) {
    s.n = 0;
    s.at[0] = at;
    for (; s.n < kSeqs && i < n; ++i) {
      if (lengths[i] == 0) continue;
      at += lengths[i];
      s.at[++s.n] = at;
    }
    const int tokens = at - s.at[0], g = (tokens + kBins - 1) / kBins, most = num_sms() * 2;
    packed_plan_kernel<<<(g < most ? g : most) + (one ? 3 : 0), kBins, 0, st>>>(a, s, one, one, lo, hi);
  }
  s.n = 0;
  if (!one) packed_plan_kernel<<<3, kBins, 0, st>>>(a, s, true, false, lo, hi);
}

}  // namespace msa
