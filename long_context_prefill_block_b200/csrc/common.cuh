// Shared device helpers and the launch interface between the C ABI (api.cu)
// and the kernels. Nothing here is visible outside libmoba.so.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moba {

constexpr int kBF16 = 0;
constexpr int kF32 = 1;

// Device status codes (same values as moba_status).
constexpr int kStInvalidArg = -1;
constexpr int kStTimeout = -4;
constexpr int kStBadIndices = -6;
constexpr int kStCheck = -7;

// Sizes of one call, validated on the host.
struct Dims {
  int batch;       // sequences
  int T;           // total tokens
  int max_seqlen;  // bound on every sequence length
  int Hq, Hkv;     // heads
  int d;           // head dim
  int B;           // block size
  int topk;        // k
  int nb;          // blocks reserved per sequence = ceil(max_seqlen / B)
  int dtype;       // kBF16 / kF32
  int shared;      // 1: a kv head's query heads share the blocks of their mean score
  int prefix;      // 1: the own block is scored by its prefix mean instead of forced
  int kv_hm;       // 1: k and v are head-major [Hkv][T][d] (decode caches), else [T][Hkv][d]
};

// Element offset of row t of kv head g in k or v.
__host__ __device__ __forceinline__ int64_t kv_row(const Dims& dm, int64_t t, int g) {
  return (dm.kv_hm ? (int64_t)g * dm.T + t : t * dm.Hkv + g) * dm.d;
}

// History slots an index row can hold: k - 1 beside the forced own block,
// all k when the own block competes for its slot.
__host__ __device__ inline int hist_slots(const Dims& dm) { return dm.prefix ? dm.topk : dm.topk - 1; }

// The prefix-mean own-block scores are built from per-chunk key sums: a
// block is split into chunks of kOwnChunkRows rows.
constexpr int kOwnChunkRows = 32;
__host__ __device__ inline int own_chunks_per_block(const Dims& dm) {
  return (dm.B + kOwnChunkRows - 1) / kOwnChunkRows;
}

// Whether query row `row` (k entries) reads its own block c: always when the
// own block is forced, else when the row names it.
__device__ __forceinline__ bool reads_own(const Dims& dm, const int32_t* row, int c) {
  if (!dm.prefix) return true;
  bool on = false;
  for (int r = 0; r < dm.topk; ++r) on |= row[r] == c;
  return on;
}

// Work of one pass over a group of kv heads [g0, g0 + ng): its q heads are
// [g0 * grp, (g0 + ng) * grp). Partial results are indexed by
// prow = ((t * nq) + h_local) * topk + slot, nq = ng * grp.
struct Chunk {
  int g0, ng;      // kv heads of this pass
  int h0, nq;      // q heads of this pass
  int n_lists;     // batch * ng * nb regroup lists
  int tile_m;      // query rows per history tile
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// 16-byte vector of elements widened to fp32.
template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  __device__ __forceinline__ static void load(const float* p, float* out) {
    const float4 r = __ldg(reinterpret_cast<const float4*>(p));
    out[0] = r.x; out[1] = r.y; out[2] = r.z; out[3] = r.w;
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void load(const __nv_bfloat16* p, float* out) {
    const uint4 r = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[2 * i] = __uint_as_float(w[i] << 16);
      out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// First error wins.
__device__ __forceinline__ void set_status(int* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// Checked build (MOBA_CHECKED defined: libmoba_checked.so): index and
// bounds checks at the kernels' computed global accesses. A failed check
// records kStCheck in the status word and the access is skipped; nothing
// traps. In the ordinary build MOBA_CHECK(cond, status) is the constant
// true and costs nothing.
#ifdef MOBA_CHECKED
__device__ __forceinline__ bool check_or_flag(bool ok, int* status) {
  if (!ok) set_status(status, kStCheck);
  return ok;
}
#define MOBA_CHECK(cond, status) (::moba::check_or_flag((cond), (status)))
#else
#define MOBA_CHECK(cond, status) (true)
#endif

// Sequence bounds with a device-side check against max_seqlen.
__device__ __forceinline__ bool seq_bounds(const Dims& dm, const int32_t* cu, int b, int64_t& start,
                                           int& len, int* status) {
  start = cu[b];
  len = cu[b + 1] - cu[b];
  if (len < 0 || len > dm.max_seqlen) {
    set_status(status, kStInvalidArg);
    return false;
  }
  return true;
}

// Largest r in [0, batch] with cu[r] <= i (cu: batch + 1 rising offsets).
__device__ __forceinline__ int find_request(const int32_t* __restrict__ cu, int batch, int i) {
  int lo = 0, hi = batch;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The same for one i by a whole warp: 32 offsets a round instead of one, two
// rounds of dependent loads for up to 1023 requests.
__device__ __forceinline__ int find_request_warp(const int32_t* __restrict__ cu, int batch, int i) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch + 1;  // the answer is in [lo, lo + n), cu[lo] <= i (or nothing is)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, lane * step < n && cu[at] <= i);
    const int k = le ? 31 - __clz(le) : 0;
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

// Place x of a launch over the tiles (of ROWS rows) of every sequence, for each
// of `heads` heads: tile_slots() x heads places. Every sequence has `slots` of
// them a head, at least as many as tiles, and takes rest in [0, slots * heads).
// By whole warps. slots == 0: no such place, or a sequence that has_place() says no
// to (which is for the caller to report).
//
// Lengths that are about even: each sequence has as many slots as the longest one
// may have tiles, and the place follows from x. Else, when those would be over
// twice the tiles that there can be, sequence b has the slots from cu[b] / ROWS + b
// on, which costs a search (one round of loads for up to 31 sequences): the
// gradient of 692 + 88 + 6 + 10 + 40 tokens, 24 on 8 heads, 68 -> 58 us without the
// empty CTAs, that of 4 x 8192 tokens, 16 heads, 3.64 -> 3.70 ms with the search.
struct TilePlace {
  int start, len, slots, rest;
};
// A sequence of a length in [0, max_seqlen] whose rows are all among the call's;
// a negative start or length is past every bound.
__device__ __forceinline__ bool has_place(const Dims& dm, uint32_t start, uint32_t len) {
  return len <= (uint32_t)min(dm.max_seqlen, dm.T) && start <= (uint32_t)dm.T - len;
}
template <int ROWS>
__host__ __device__ inline bool even_lengths(const Dims& dm) {
  return ((int64_t)dm.max_seqlen + ROWS - 1) / ROWS * dm.batch <=
         2 * ((int64_t)(dm.T / ROWS) + dm.batch);
}
template <int ROWS>
__host__ __device__ inline int64_t tile_slots(const Dims& dm) {
  return even_lengths<ROWS>(dm) ? ((int64_t)dm.max_seqlen + ROWS - 1) / ROWS * dm.batch
                                : (int64_t)(dm.T / ROWS) + dm.batch;
}
// TILE_MAJOR: with even lengths tile 0 of every sequence comes first, then tile
// 1; else one sequence after the other.
template <int ROWS, bool TILE_MAJOR>
__device__ __forceinline__ TilePlace find_tile(const Dims& dm, const int32_t* __restrict__ cu,
                                               int heads, int x) {
  int b, slots, rest;
  if (even_lengths<ROWS>(dm)) {
    slots = (int)(((int64_t)dm.max_seqlen + ROWS - 1) / ROWS);
    if (TILE_MAJOR) {
      b = x / heads % dm.batch;
      rest = x / heads / dm.batch * heads + x % heads;
    } else {
      b = x / (slots * heads);
      rest = x % (slots * heads);
    }
  } else {
    const int lane = threadIdx.x & 31, slot = x / heads;
    b = 0;  // the largest with cu[b] / ROWS + b <= slot
    for (int n = dm.batch + 1; n > 1;) {
      const int step = (n + 31) / 32, at = b + lane * step;
      const uint32_t le = __ballot_sync(0xffffffffu, lane * step < n && cu[at] / ROWS + at <= slot);
      const int k = le ? 31 - __clz(le) : 0;
      n = min(step, n - k * step);
      b += k * step;
    }
    if (b >= dm.batch) return {0, 0, 0, 0};
    const int base = cu[b] / ROWS + b;
    slots = cu[b + 1] / ROWS + b + 1 - base;
    rest = x - base * heads;
    if (rest < 0 || rest >= slots * heads) return {0, 0, 0, 0};  // offsets that fall
  }
  const uint32_t start = cu[b], len = (uint32_t)cu[b + 1] - start;
  if (!has_place(dm, start, len)) return {0, 0, 0, 0};
  return {(int)start, (int)len, slots, rest};
}

// Request r and cache position of row i of a call on a paged cache: request
// r's rows cu[r] .. cu[r+1]-1 stand at the last positions of its seqlens[r].
// False for a row that no request owns (a padded batch), and, with a status
// code, for a request whose length does not hold its rows or passes max_len, or
// whose rows are not all among the call's `rows`.
// whole_warp: every lane of the warp asks for the same i.
__device__ __forceinline__ bool tail_position(const int32_t* __restrict__ cu,
                                              const int32_t* __restrict__ seqlens, int batch,
                                              int rows, int max_len, int i, int& r, int& pos,
                                              int& len, int* status, bool whole_warp = false) {
  r = whole_warp ? find_request_warp(cu, batch, i) : find_request(cu, batch, i);
  if (r >= batch || i < cu[r]) return false;
  const int n = cu[r + 1] - cu[r];
  len = seqlens[r];
  if (len < n || len > max_len || cu[r] < 0 || cu[r + 1] > rows) {
    set_status(status, kStInvalidArg);
    return false;
  }
  pos = len - n + (i - cu[r]);
  return true;
}

// A paged 8-bit cache: codes [pages][Hkv][page][d] in e4m3 and one scale
// byte (e8m0: 2^(byte - 127), 255 = NaN) per row [pages][Hkv][page], for K
// and for V. Request r's position p is in page table[r][p / page].
struct Cache {
  uint8_t* k;
  uint8_t* v;
  uint8_t* ks;
  uint8_t* vs;
  const int32_t* table;  // [batch][max_pages]
  const int32_t* lens;   // [batch]
  int pages, page_log2, max_pages;
};

// Positions a request can have: what its pages hold and what the caller's
// max_seqlen allows, up to 2^31 - 4096: kernels step past a request's end by up to
// 2048 positions before they compare, in 32 bits.
__host__ __device__ __forceinline__ int max_positions(const Dims& dm, const Cache& c) {
  const int64_t held = (int64_t)c.max_pages << c.page_log2;
  const int most = dm.max_seqlen < INT32_MAX - 4095 ? dm.max_seqlen : INT32_MAX - 4095;
  return held < most ? (int)held : most;
}

// Row index of page slot `page` (an entry of the table) for kv head g, or -1
// for an entry that names no page.
__device__ __forceinline__ int64_t cache_page_row(const Cache& c, int Hkv, int page, int g) {
  if (page < 0 || page >= c.pages) return -1;
  return ((int64_t)page * Hkv + g) << c.page_log2;
}

// Whether a row index is one of the cache's (for the checked build).
__device__ __forceinline__ bool cache_holds(const Cache& c, int Hkv, int64_t row) {
  return row >= 0 && row < ((int64_t)c.pages * Hkv) << c.page_log2;
}

// The value of a scale byte.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
}

}  // namespace moba

// ---- launchers (host), one per kernel family -------------------------------
namespace moba {

cudaError_t launch_meanpool(const Dims& dm, const void* k, const int32_t* cu, float* kbar,
                            int* status, cudaStream_t st);
// Block means of only the blocks holding each sequence's last
// cu_new[b+1] - cu_new[b] positions (max_new: the largest such count).
cudaError_t launch_meanpool_update(const Dims& dm, const void* k, const int32_t* cu,
                                   const int32_t* cu_new, int max_new, float* kbar, int* status,
                                   cudaStream_t st);
// Decode step (decode.cu): gate into idx, split-K attention into partials
// [decode_partial_rows] x (d + 1) merged by the last split of each row into
// out / lse; arrivals: n_queries * Hq ints of scratch (zeroed by the gate).
size_t decode_partial_rows(const Dims& dm, int n_queries);
cudaError_t launch_decode(const Dims& dm, int n_queries, const void* q, const void* k,
                          const void* v, const int32_t* cu, const int32_t* cu_q, const float* kbar,
                          int32_t* idx, float* part_o, float* part_lse, int* arrivals, void* out,
                          float* lse, int* status, cudaStream_t st);
// Tensor-core gate (bf16, d = 128, at most 256 blocks per sequence).
bool gate_tc_supported(const Dims& dm);
// Its sorting-network form for 5 to 15 history slots and the forced own
// block (gate_net.cu); launch_gate_tc hands such calls to it.
bool gate_net_supported(const Dims& dm);
cudaError_t launch_gate_net(const Dims& dm, const void* q, const float* kbar, const int32_t* cu,
                            int32_t* idx, int* status, cudaStream_t st);
cudaError_t launch_gate_tc(const Dims& dm, const void* q, const float* kbar, const float* own,
                           const int32_t* cu, int32_t* idx, int* status, cudaStream_t st);
// own: with dm.prefix, the own-block scores [T][Hq] (launch_own_score); else unused.
cudaError_t launch_gate(const Dims& dm, const void* q, const float* kbar, const float* own,
                        const int32_t* cu, int32_t* idx, int* status, cudaStream_t st);
// Own-block scores by prefix mean: own[t][h] = q_{t,h} . mean(k_{cB..p}) (fp32).
// csum: scratch for the chunk key sums, batch * nb * own_chunks_per_block * Hkv * d floats.
cudaError_t launch_own_score(const Dims& dm, const void* q, const void* k, const int32_t* cu,
                             float* own, float* csum, int* status, cudaStream_t st);

// Regrouping of (query, head, slot) by the history block it chose.
struct Regroup {
  int32_t* counts;     // [n_lists]
  int32_t* cursor;     // [n_lists]
  int32_t* list_off;   // [n_lists + 1]
  int32_t* tile_off;   // [n_lists + 1]; tile_off[n_lists] = number of tiles
  int32_t* pairs;      // [max pairs] partial-row ids grouped by list
  int4* tiles;         // [max tiles] (list, first row in list, list size, list's first entry):
                       // a work unit's description in one 16-byte load
  int64_t max_tiles;
};
cudaError_t launch_regroup(const Dims& dm, const Chunk& ch, const int32_t* idx, const int32_t* cu,
                           const Regroup& rg, int* status, cudaStream_t st);

// Partial attention results of one pass.
struct Partials {
  void* o;     // part_rows(T, nq * topk) rows of d values in the input dtype (layout below)
  float* lse;  // part_rows(T, nq * topk)
};

// A partial result o_j = u_j / l_j (normalised, so |o_j| <= max |v|) is
// stored in the input dtype -- bf16 for bf16 inputs, as merge-state kernels
// commonly keep it -- and merged in fp32; its lse stays fp32.
//
// Partial results of a pass are stored interleaved over 32 consecutive
// tokens. For partial row prow = (t * nq + h_local) * k + slot (nr = nq * k
// rows per token) the 32-byte piece c of the row sits at piece
// (tile * npc + c) * 32 + t % 32 (npc = the row's 32-byte pieces) with
// tile = (t / 32) * nr + prow % nr, and its lse at tile * 32 + t % 32. A
// warp holding 32 consecutive tokens of one head -- the own-block kernel's
// merge -- then reads each piece of its rows' partials as one contiguous
// 1 KB access instead of 32 scattered ones.
struct PartRow {
  int64_t tile;
  int lane;
};
__host__ __device__ inline PartRow part_row(int64_t prow, int64_t nr) {
  const int64_t t = prow / nr;
  return {(t >> 5) * nr + (prow - t * nr), (int)(t & 31)};
}
template <typename P>
__host__ __device__ inline P* part_piece(void* o, const PartRow& r, int d, int c) {
  const int npc = d * (int)sizeof(P) / 32;
  return reinterpret_cast<P*>(static_cast<char*>(o) + ((r.tile * npc + c) * 32 + r.lane) * 32);
}
template <typename P>
__host__ __device__ inline const P* part_piece(const void* o, const PartRow& r, int d, int c) {
  const int npc = d * (int)sizeof(P) / 32;
  return reinterpret_cast<const P*>(static_cast<const char*>(o) + ((r.tile * npc + c) * 32 + r.lane) * 32);
}
__host__ __device__ inline int64_t part_lse_at(const PartRow& r) { return r.tile * 32 + r.lane; }
// Storage rows of a pass: T rounded up to whole 32-token tiles.
inline size_t part_rows(int64_t T, int64_t nr) { return (size_t)((T + 31) / 32) * 32 * (size_t)nr; }

// Portable SIMT kernels (fp32 or bf16 inputs, any block size).
cudaError_t launch_history_simt(const Dims& dm, const Chunk& ch, const void* q, const void* k,
                                const void* v, const int32_t* cu, const Regroup& rg,
                                const Partials& pt, cudaStream_t st);
cudaError_t launch_current_simt(const Dims& dm, const Chunk& ch, const void* q, const void* k,
                                const void* v, const int32_t* cu, const int32_t* idx,
                                const Partials& pt, cudaStream_t st);
cudaError_t launch_dense_simt(const Dims& dm, const void* q, const void* k, const void* v,
                              const int32_t* cu, void* out, float* lse, cudaStream_t st);
// Backward (bwd.cu): dq, dk, dv (fp32, zeroed by the caller) of the whole
// batch; `ch` covers every head in one pass; Dsum [T * Hq] is scratch.
cudaError_t launch_bwd_dot(const Dims& dm, const void* out, const void* dout, float* Dsum,
                           cudaStream_t st);
cudaError_t launch_backward(const Dims& dm, const Chunk& ch, const void* q, const void* k,
                            const void* v, const void* dout, const float* lse, const float* Dsum,
                            const int32_t* cu, const int32_t* idx, const Regroup& rg, float* dq,
                            float* dk, float* dv, int* status, cudaStream_t st);
// Tensor-core backward (bf16, d = 128, B % 128 == 0).
bool bwd_tc_supported(const Dims& dm);
cudaError_t launch_backward_tc(const Dims& dm, const Chunk& ch, const void* q, const void* k,
                               const void* v, const void* dout, const float* lse,
                               const float* Dsum, const int32_t* cu, const int32_t* idx,
                               const Regroup& rg, float* dq, float* dk, float* dv, int* status,
                               cudaStream_t st);
constexpr int kSimtTileM = 32;

// Gradient of dense causal attention. stat: 2 * Hq * T floats of scratch,
// filled by launch_dense_bwd_stat, which also zeroes the gradients of rows
// that no sequence owns; the gradients have the inputs' type.
cudaError_t launch_dense_bwd_stat(const Dims& dm, const void* out, const void* dout,
                                  const float* lse, const int32_t* cu, float* stat, void* dq,
                                  void* dk, void* dv, int* status, cudaStream_t st);
// CTAs that share a tile (a power of two up to `most`) of the gradient's passes,
// of `at_once` that run together: what takes least by a rough account in items
// (a tile of queries against a tile of keys), the longest tile's share or the
// mean of all, and `start` items for each round of CTAs. The number of CTAs sets
// the order of the sums, so T counts as the next power of two: a batch's padding
// seldom changes its bits.
template <int ROWS>
inline int cluster_for(Dims dm, int64_t at_once, int most, int start) {
  int T = 1;
  while (T < dm.T && T < 1 << 30) T *= 2;
  dm.T = T;
  const int64_t top = dm.max_seqlen < T ? dm.max_seqlen : T;  // the bound may be generous
  const int64_t tiles = (top + ROWS - 1) / ROWS, longest = tiles * (dm.Hq / dm.Hkv);
  const int64_t clusters = tile_slots<ROWS>(dm) * (dm.Hq + dm.Hkv);
  const int64_t all = (int64_t)(dm.T / ROWS + 1) * dm.Hq * (tiles + 1);  // sequences of max_seqlen
  int best = 1;
  int64_t least = INT64_MAX;
  for (int cs = 1; cs <= most; cs *= 2) {
    const int64_t share = (longest + cs - 1) / cs, mean = all / at_once;
    const int64_t t = (share > mean ? share : mean) + start * ((clusters * cs + at_once - 1) / at_once);
    if (t < least) least = t, best = cs;
  }
  return best;
}
// bf16 inputs (dense_bwd_tc.cu), then fp32 inputs.
cudaError_t launch_dense_bwd_tc(const Dims& dm, const void* q, const void* k, const void* v,
                                const void* dout, const float* stat, const int32_t* cu, void* dq,
                                void* dk, void* dv, int* status, cudaStream_t st);
cudaError_t launch_dense_bwd_simt(const Dims& dm, const void* q, const void* k, const void* v,
                                  const void* dout, const float* stat, const int32_t* cu, void* dq,
                                  void* dk, void* dv, int* status, cudaStream_t st);

// Paged 8-bit cache (cache.cu, decode_cache.cu); dm.T: the call's rows.
// sums: scratch of cache_sums_floats (or nullptr), from which launch_cache_means
// then makes the means of the blocks that the new rows complete.
size_t cache_sums_floats(const Dims& dm);
cudaError_t launch_cache_write(const Dims& dm, const Cache& c, const void* k, const void* v,
                               const int32_t* cu_new, float* sums, int* status, cudaStream_t st);
cudaError_t launch_cache_means(const Dims& dm, const Cache& c, const int32_t* cu_new,
                               const float* sums, float* kbar, int* status, cudaStream_t st);
cudaError_t launch_cache_read(const Dims& dm, const Cache& c, const int32_t* cu_rows, void* k,
                              void* v, int* status, cudaStream_t st);
// The decode gate with cache lengths in place of packed offsets (decode.cu).
cudaError_t launch_cache_gate(const Dims& dm, const void* q, const float* kbar,
                              const int32_t* seqlens, const int32_t* cu_q, int32_t* idx,
                              int max_len, int* status, cudaStream_t st);
// Decode over the cache: gate into idx, split attention into partials
// [decode_cache_partial_rows] x (d + 1), their merge into out and lse.
size_t decode_cache_partial_rows(const Dims& dm);
cudaError_t launch_decode_cache(const Dims& dm, const Cache& c, const void* q, const float* kbar,
                                const int32_t* cu_q, int32_t* idx, float* part_o, float* part_lse,
                                void* out, float* lse, int* status, cudaStream_t st);

cudaError_t launch_merge(const Dims& dm, const Chunk& ch, const int32_t* idx, const int32_t* cu,
                         const Partials& pt, void* out, float* lse, cudaStream_t st);

}  // namespace moba
