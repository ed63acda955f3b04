// Internal interface between the C-ABI layer (api.cu) and the kernel files.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace msa {

// Head mapping (the MSA group is the proxy head): proxy head p selects key blocks for its Hq / Hp
// query heads.  An attention group is a set of G query heads that share one selection row and
// one KV head: G = Hq / max(Hp, Hkv), and proxy head p has R = max(1, Hkv / Hp) of them,
// a = p R + r (r < R), on KV head kv_of(a).  Hp == Hkv: a = p = the GQA group, R = 1.
struct Dims {
  int B, S, Hq, Hkv, Hp, G, top_k, nblk;
  float scale;
  int chunk;   // token-list chunk: a list holds the tokens of one (b, p, n) in one chunk of the
  int nchunk;  // sequence [c * chunk, (c+1) * chunk); lists are ordered chunk-major
  int R = 1;   // attention groups per proxy head
  __host__ __device__ long long nseg() const { return (long long)B * Hp * nblk; }  // (b, p, n)
  __host__ __device__ long long nlist() const { return nseg() * nchunk; }           // (c, b, p, n)
  __host__ __device__ int kv_of(int a) const { return a / (Hp * R / Hkv); }
  __host__ __device__ int Gp() const { return G * R; }  // query heads per proxy head
};

// A unit of attention work: `count` tokens of list `seg` (= c * nseg + (b * Hp + p) * nblk + n)
// starting at list position `first`, for attention group p R + sub; `base` = the list's offset +
// first, i.e. the position of the item's first entry in the packed entry array.
struct Item {
  int seg, first, count, base, sub;
};

// Shape of one work list: tiles of `tile_tokens` tokens, `chunk_tiles` tiles per item, and
// `nsub` items (attention groups r = 0 .. nsub-1) for each such run of tokens.
struct ItemSpec {
  int tile_tokens, chunk_tiles, nsub;
};

// ---------------------------------------------------------------- index kernels (index.cu)
// Count block references per (c, b, g, n) list (validating every index against its row).
void launch_count(const Dims& d, const int32_t* idx, int* seg_count, unsigned* status,
                  cudaStream_t st);
// Exclusive scans: list offsets (sparse only) and item offsets for up to two item specs.
// dense: list lengths are the tokens t >= 128 n of the chunk instead of seg_count.
// tile_tmp: scan_tiles(d.nlist()) x 3 long longs of scratch.  scan_kernels: how many kernels
// one scan launches (one block for few lists, three passes over every SM otherwise).
long long scan_tiles(long long nlists);
int scan_kernels(long long nlists);
void launch_scan(const Dims& d, bool dense, const int* seg_count, int* seg_offset,
                 const ItemSpec* specs, int nspecs, int* item_offset0, int* item_offset1,
                 int* totals, long long* tile_tmp, cudaStream_t st);
// Scatter (t << 8 | slot) into the lists; order inside a list is unspecified.
void launch_fill(const Dims& d, const int32_t* idx, const int* seg_offset, int* seg_cursor,
                 int* entries, unsigned* status, cudaStream_t st);
void launch_items(const Dims& d, bool dense, const int* seg_count, const int* seg_offset,
                  const ItemSpec& spec, const int* item_offset, Item* items, long long max_items,
                  unsigned* status, cudaStream_t st);

// Row data of every entry e of the sparse lists, in entry order: lpxe[e] = LSE_px of e's token
// x log2(e); emeta[e Gp + h] = rowm of e's token and head g Gp + h.  (Dense lists need no copy:
// their tokens are consecutive, and the dense kernels read rowm and LSE_px by token.)
void launch_entry_meta(const Dims& d, const int* seg_count, const int* seg_offset,
                       const int* entries, const float* lse_px, const float2* rowm, float* lpxe,
                       float2* emeta, cudaStream_t st);

// ---------------------------------------------------------------- proxy top-k (topk.cu)
// Returns false if the TMA tensor maps could not be created (driver entry point missing).
bool launch_proxy_topk(const Dims& d, const void* qp, const void* kp, int32_t* idx,
                       unsigned* status, cudaStream_t st);
// Dense proxy normaliser (warmup): lse_px[(b Hp + g) S + t] = log sum_{j <= t} exp(scale qp.kp).
bool launch_proxy_lse_dense(const Dims& d, const void* qp, const void* kp, float* lse_px,
                            unsigned* status, cudaStream_t st);

// ---------------------------------------------------------------- forward (fwd.cu)
// Sparse main-attention partials (attn_fwd.cu): for every list entry (t, slot) and query head h
// of the group, the block's normalised output (bf16, opart[(t, h, slot)][128]) and its natural
// log-sum-exp (lpart).  Returns false for an unsupported group size or if the TMA tensor maps
// cannot be created.
// One pass takes the items [*item_lo, *item_hi) (NULL: 0 / all) -- the lists of a range of
// sequence chunks -- and indexes its partials from token pass_t0 ((b pass_tokens + t - pass_t0)
// Hq + h) top_k + slot.
bool launch_attn_fwd(const Dims& d, const void* q, const void* k, const void* v,
                     const int* seg_offset, const int* entries, const Item* items,
                     const int* n_items, long long max_items, const int* item_lo,
                     const int* item_hi, int pass_t0, int pass_tokens, void* opart, float* lpart,
                     unsigned* status, cudaStream_t st);
int fwd_item_tiles();  // 128-row tiles per sparse-forward work item
// Merges the partials of every (b, t, h) with t in [t0, t0 + tn) (partials indexed as the pass
// with pass_tokens = tp wrote them); a partial is valid iff its log-sum-exp is not NaN (the
// caller fills lpart with NaN bytes before the partial pass).
void launch_combine(const Dims& d, const void* opart, const float* lpart, void* o, float* lse,
                    int t0, int tn, int tp, cudaStream_t st);
// Dense causal forward of the warmup mode (dense_fwd.cu).  Returns false for an unsupported group
// size or if the TMA tensor maps cannot be created.
bool launch_dense_fwd(const Dims& d, const void* q, const void* k, const void* v, void* o,
                      float* lse, unsigned* status, cudaStream_t st);

// ---------------------------------------------------------------- backward (bwd.cu)
// rowm[(b S + t) Hq + h] = {LSE(b, h, t) log2 e, rowsum(dO * O)(b, t, h)}
void launch_bwd_rowdot(const Dims& d, const void* o, const void* dout, const float* lse,
                       float2* rowm, cudaStream_t st);
// Sparse proxy normaliser, first pass (attn_fwd.cu, proxy mode): lpx_part[((b S + t) Hp + g) top_k
// + slot] = log-sum-exp of scale qp.kp over the visible keys of that slot's block; slots no list
// entry reaches are left as they were (the caller fills lpx_part with NaN bytes first).
bool launch_proxy_lse_sparse(const Dims& d, const void* qp, const void* kp, const int* seg_offset,
                             const int* entries, const Item* items, const int* n_items,
                             long long max_items, float* lpx_part, unsigned* status,
                             cudaStream_t st);
// Second pass: lse_px[(b Hp + g) S + t] from the written (non-NaN) partials of each row.
void launch_proxy_lse_combine(const Dims& d, const float* lpx_part, float* lse_px, cudaStream_t st);

// Main-attention backward (dQ, dK, dV into fp32 accumulators) and the teacher pbar
// ([list entry - *entry_lo][128 keys] fp16) of one pass: the items [*item_lo, *item_hi) (NULL:
// 0 / all; entry_lo NULL: 0).  rowdata: {LSE log2 e, D} per list entry and head (emeta, sparse)
// or per query row (rowm [B, S, Hq], dense).  Returns false for an unsupported group size or if
// the TMA tensor maps cannot be created.
bool launch_attn_bwd(const Dims& d, bool dense, const void* q, const void* k, const void* v,
                     const void* dout, const float2* rowdata, const int* seg_offset,
                     const int* entries, const Item* items, const int* n_items, long long max_items,
                     const int* item_lo, const int* item_hi, const int* entry_lo,
                     float* dq_acc, float* dk_acc, float* dv_acc, void* pbar, unsigned* status,
                     cudaStream_t st);
// Proxy gradients (dQp, dKp into fp32 accumulators) of the KL term from pbar, scaled by kl_grad,
// or by *kl_grad_dev (read on the device) when that is not NULL.  kl_acc: NULL, or
// a zeroed double that receives sum over the visited (token, key) pairs of
// pbar (ln pbar - ln p_student), i.e. B S Hp times the KL value.
// lpx: LSE_px x log2 e per list entry (lpxe, sparse) or LSE_px per proxy row (lse_px
// [B, Hp, S], dense).
bool launch_proxy_bwd(const Dims& d, bool dense, const void* qp, const void* kp,
                      const float* lpx, const void* pbar, float kl_grad,
                      const float* kl_grad_dev, const int* seg_offset,
                      const int* entries, const Item* items, const int* n_items,
                      long long max_items, const int* item_lo, const int* item_hi,
                      const int* entry_lo, float* dqp_acc, float* dkp_acc, double* kl_acc,
                      unsigned* status, cudaStream_t st);  // one pass, as launch_attn_bwd
// kl_out[0] = kl_acc[0] / (B S Hp)  (one thread)
void launch_kl_finalize(const Dims& d, const double* kl_acc, float* kl_out, cudaStream_t st);
int bwd_item_tokens();   // tokens per fused-backward work item
int bwd_group_tokens();  // tokens per proxy-gradient flush group
void launch_convert(const float* src, void* dst, long long n, cudaStream_t st);

// ---------------------------------------------------------------- decode (decode.cu)
// One new token per sequence against its cache, in three launches: proxy block scores (scores
// [B, Hp, nblk] fp32), selection (block_idx [B, Hp, top_k]) and sparse attention (o [B, Hq, 128],
// lse [B, Hq]).
bool launch_decode_scores(const Dims& d, const void* qp, const void* kp_cache,
                          const int32_t* seq_len, float* scores, unsigned* status,
                          cudaStream_t st);  // false: the tensor map could not be made
void launch_decode_select(const Dims& d, const float* scores, const int32_t* seq_len,
                          int32_t* block_idx, cudaStream_t st);
bool launch_decode_attn(const Dims& d, const void* q, const void* k_cache, const void* v_cache,
                        const int32_t* seq_len, const int32_t* block_idx, void* o, float* lse,
                        unsigned* status, cudaStream_t st);  // false: no tensor map

// ------------------------------------------- norm and rotation of the heads (norm_rope.cu)
constexpr int kRopeRotate = 1, kRopeCache = 2, kRopeQ4 = 8;  // RopePart::flags
constexpr int kRopeAxes = 4;                    // axes of positions at most
constexpr int kRopeParts = 8;                   // parts of one call at most
// One part: H consecutive heads (128 elements apart) of every token, with its own norm weight.
struct RopePart {
  const __nv_bfloat16* x;  // [B][N][H][128], batch and token strides in elements
  long long xb, xt;
  __nv_bfloat16* y;  // forward: the output (kRopeCache: its rows by position; kRopeQ4: a cache in 4 bits,
                     // without strides); backward: dy (read)
  long long yb, yt;
  __nv_bfloat16* dx;
  long long dxb, dxt;
  const float* w;  // [128], NULL: not normed
  float* dw;       // [128] or NULL
  int H, flags;
};
struct RopeArgs {
  int B, N, rot, inter, nparts, rows;  // rows: heads of all parts
  int cap;                             // append: rows of a cache
  float eps;
  const int32_t* positions;  // [B][N] or NULL: 0 .. N - 1; with axes [naxes][B][N]
  const int32_t* seq_len;    // append: [B], the new tokens are the last N of it
  const float* inv_freq;     // [rot / 2]
  unsigned* status;          // append, backward: written whole by the call
  float* partial;            // backward: [rope_partials()][nparts][128]
  int rows_chunk, chunks;    // set by the launch
  int naxes;                 // 0: positions as above, in an append those of the cache rows
  uint8_t axis[64];          // of each of the rot / 2 pairs
  RopePart p[kRopeParts];
};
int rope_partials();
void launch_norm_rope_fwd(RopeArgs a, cudaStream_t st);
void launch_norm_rope_bwd(RopeArgs a, cudaStream_t st);  // two kernels

// ------------------------------------------- sliding-window attention (window.cuh, win_*.cu)
struct WinDims {
  int B, S, Hq, Hkv, G;
  int W, ns, nsp;  // window and sinks, at most S; nsp: the sinks rounded up to a multiple of 8
  float scale;
};
// Causal attention over the window and the sinks; q, o [B, S, Hq, 128], k, v [B, S, Hkv, 128], lse
// [B, Hq, S].  The launches return false if a tensor map could not be made.
bool launch_win_fwd(const WinDims& d, const void* q, const void* k, const void* v, void* o,
                    float* lse, unsigned* status, cudaStream_t st);

// Packed sequences (packed.cu, window.cuh): tokens of sequences of different lengths one behind the other.
struct PackedDims {
  WinDims d;                 // B 1, S the tokens of all sequences, W the window; no sinks
  int fwd_tiles, fwd_units;  // query tiles per unit of the forward, units along the tokens
  int dq_units;              // query tiles
  int chunk;                 // query tiles of an item of the key-outer backward at most
  int items, slots, joins;   // its items along the tokens, those that leave partials, the blocks these belong to
  long long rows;            // of the tensors, at least S
};
struct PackedTables;
// Counts the work of sequences of these lengths (host); d, rows filled.
void packed_count(const int32_t* lengths, int n, PackedDims* x);
size_t packed_table_bytes(const PackedDims& x);
PackedTables packed_tables(const PackedDims& x, const void* table);
int packed_launches(int n);
void launch_packed_plan(const PackedDims& x, const int32_t* lengths, int n, void* table, cudaStream_t st);
bool launch_packed_fwd(const PackedDims& x, const PackedTables& p, const void* q, const void* k, const void* v, void* o,
                       float* lse, unsigned* status, cudaStream_t st);
void launch_packed_rowdata(const PackedDims& x, const PackedTables& p, const void* q, const void* k, const void* v,
                           const void* o, const void* dout, const float* lse, float2* rowm, void* dq, void* dk, void* dv,
                           cudaStream_t st);
bool launch_packed_dq(const PackedDims& x, const PackedTables& p, const void* q, const void* k, const void* v,
                      const void* dout, float2* rowm, void* dq, unsigned* status, cudaStream_t st);
bool launch_packed_dkv(const PackedDims& x, const PackedTables& p, const void* q, const void* k, const void* v,
                       const void* dout, const float2* rowm, void* dk, void* dv, float* part, unsigned* status, cudaStream_t st);
// Zeros (and -inf) where there is no sequence at all; else the forward and the row data write the rows behind the last one.
void launch_packed_pad(const PackedDims& x, void* a, int ha, void* b, int hb, void* c, int hc, float* lse, cudaStream_t st);
bool launch_packed_join(const PackedDims& x, const PackedTables& p, const float* part, void* dk, void* dv, cudaStream_t st);

// Limit of the waits that last a whole unit, its rows leaving only at its end (win_fwd.cu).
unsigned long long win_unit_wait_ns(const WinDims& d);

// Work items of the key-outer backward: first the sink blocks' chunks, then the window blocks'.
struct WinItems {
  int sink_blocks, sink_chunk, sink_items;  // key blocks that hold sinks; query tiles per item
  int win_chunk, win_split;                 // window blocks: tiles per item, items per block
  int items, partials, join_blocks;         // partial slots (2 x 128 x 128 fp32); blocks to join
};
WinItems win_items(const WinDims& d);
// Row data of one-head groups' windows of at most kFewKeys keys and sinks, in place of
// launch_bwd_rowdot (larger groups' rows of a few keys lie in one key tile: launch_win_dq).
constexpr int kFewKeys = 32;
void launch_win_rowdata(const WinDims& d, const void* q, const void* k, const void* v, const void* dout,
                        const float* lse, float2* rowm, cudaStream_t st);
// dk, dv and dq from rowm (launch_bwd_rowdot); dk, dv of split key blocks go to `part`
// (win_items(d).partials slots) and are added by the join.
bool launch_win_dkv(const WinDims& d, const void* q, const void* k, const void* v, const void* dout,
                    const float2* rowm, void* dk, void* dv, float* part, unsigned* status, cudaStream_t st);
// (launch_win_dq comes first: where a query tile's keys fit one key tile it replaces D in rowm.)
bool launch_win_dq(const WinDims& d, const void* q, const void* k, const void* v, const void* dout,
                   float2* rowm, void* dq, unsigned* status, cudaStream_t st);
bool launch_win_join(const WinDims& d, const float* part, void* dk, void* dv, cudaStream_t st);

// Decode step over caches of capacity d.S: key tiles per split and splits; opart [nsplit][B][Hq][128],
// lpart [nsplit][B][Hq] (used when nsplit > 1).
struct WinSplit {
  int nsplit, tiles;
};
WinSplit win_decode_split(const WinDims& d);
bool launch_win_decode(const WinDims& d, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* seq_len, void* o, float* lse, float* opart, float* lpart,
                       unsigned* status, cudaStream_t st);

// Joins the splits of a decode step (win_decode.cu): opart [nsplit][B][Hq][128] normalised, lpart
// [nsplit][B][Hq] in log2 units, -inf for an empty split; sequences whose length is not in 1 .. cap are skipped.
void launch_decode_join(int B, int Hq, int cap, int nsplit, const int32_t* seq_len, const float* opart,
                        const float* lpart, void* o, float* lse, cudaStream_t st);

// ------------------------------------------- caches in 4 bits (q4.cuh, q4.cu)
// Decode steps over K and V caches [B][Hkv][capacity / 128][9344 bytes]; d.S is the capacity.
WinSplit q4_window_split(const WinDims& d);
WinSplit q4_sparse_split(const Dims& d);
void launch_q4_window(const WinDims& d, const void* q, const void* k, const void* v, const int32_t* seq_len, void* o,
                      float* lse, float* opart, float* lpart, unsigned* status, cudaStream_t st);
// Over the key blocks block_idx [B, Hp, top_k] of launch_decode_select.
void launch_q4_sparse(const Dims& d, const void* q, const void* k, const void* v, const int32_t* seq_len,
                      const int32_t* block_idx, void* o, float* lse, float* opart, float* lpart, unsigned* status,
                      cudaStream_t st);
// Rows first .. first + count - 1 of every sequence and head: out [B, count, H, 128] bf16.
void launch_q4_read(const void* cache, int B, int H, int cap, int first, int count, void* out, cudaStream_t st);

int num_sms();
void set_api_error(const char* what);

}  // namespace msa
