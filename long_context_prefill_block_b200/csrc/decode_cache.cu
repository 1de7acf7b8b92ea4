// Decode step over the paged 8-bit cache (cache.cu): PaperTrace "2.1.3 MoBA",
// section 5.4. A query at position p reads the blocks that the gate chose and
// its own block up to p, as one softmax (eq. 4-8); a key's scale multiplies
// its logit and a value's scale its weight, so codes are widened once and
// never rescaled.
//
//   cache_gate_kernel  scores and top-k, a cluster of CTAs per (query, kv head),
//                      where there are many blocks to choose from
//   cache_attn_tc      bf16 queries: split over the chosen keys, codes by TMA
//                      into each warp's own ring, products on the tensor core
//   cache_attn_kernel  fp32 queries: the same split, fp32 FMA
//
//   cache_merge_kernel joins the splits' partials of each row, where it has more
//                      than one
//
// Bound by the bytes of the chosen rows: 2 (d + 1) a key.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <climits>
#include <cmath>
#include <type_traits>

#include "tc_ptx.cuh"

namespace moba {
namespace {

constexpr int kSMs = 148;       // of a B200: what splits are sized by
constexpr int kMaxKeys = 2048;  // keys of a split at most
constexpr int kMaxSlots = 16;   // blocks of a split at most
constexpr int kMaxPages = kMaxKeys / 16 + 2 * kMaxSlots;
constexpr float kLog2e = 1.4426950408889634f;

// How a row's keys are divided. Its slots are the topk - 1 places for chosen
// earlier blocks (no more than there can be such blocks) and, last, the own
// block, which with shared routing is one slot among them and else is read apart,
// once for all heads of a group. Split x: of group x / parts of `slots` slots,
// part x % parts of each block (parts > 1 only where a group is one slot).
struct Split {
  int keys;    // of a part
  int parts;   // of a block
  int slots;   // of a group
  int own;     // the own block's slot
  int groups;  // before the own block's
  int per_row;
};

// Splits long enough that a CTA's start (about 5 us, most of it dependent
// loads) is small beside its keys, while two CTAs an SM are left: large blocks
// in parts of up to 2048 keys, small ones together. 48 x 32768 tokens, three
// shared blocks of 512: 54 us with a block a CTA, 41 with all three (which
// also need no merge). No slots for blocks that cannot exist: 8 requests of 778
// tokens, four queries, blocks of 2048, topk 3: 33 us with them, 17.5 without.
// fp32 queries have a CTA per q head with shared routing too (40 on 8 heads, d = 64,
// eight of 282 blocks: 101 us when counted by kv heads, 40). No parts of a block behind
// max_seqlen either: 4 requests of 200 tokens with blocks of 4096 had 32 a row, two
// of them with keys. The rule asks for the call's sizes alone, so that the workspace
// does not depend on the device that is current.
Split split_of(const Dims& dm) {
  const int64_t B = dm.B < dm.max_seqlen ? dm.B : dm.max_seqlen > 1 ? dm.max_seqlen : 1;
  // fp32 queries have a CTA per q head in either case
  const int64_t units = (int64_t)dm.T * (dm.shared && dm.dtype == kBF16 ? dm.Hkv : dm.Hq);
  const int64_t least = 2 * kSMs;
  const int k = dm.nb < 1 ? 1 : dm.topk < dm.nb ? dm.topk : dm.nb;
  const int listed = dm.shared ? k : k - 1;
  Split s{128, 1, 1, k - 1, 0, 0};
  while (s.keys < kMaxKeys && s.keys < B &&
         units * k * ((B + 2 * s.keys - 1) / (2 * s.keys)) >= 2 * least)
    s.keys *= 2;
  if (s.keys > B) s.keys = (int)B;
  s.parts = (int)((B + s.keys - 1) / s.keys);
  if (s.parts == 1)
    while (s.slots < kMaxSlots && s.slots < listed && (s.slots + 1) * B <= kMaxKeys &&
           units * ((listed + s.slots) / (s.slots + 1)) >= least)
      ++s.slots;
  s.groups = listed > 0 ? (listed + s.slots - 1) / s.slots : 0;
  s.per_row = (s.groups + (dm.shared ? 0 : 1)) * s.parts;
  return s;
}

// A call's fixed facts, and where a query's row stands.
struct Step {
  Dims dm;
  Cache c;
  Split sp;
  const int32_t* cu_q;
  const float* kbar;
  int32_t* idx;
  bool gated;       // idx comes from a launch of its own; else each CTA chooses
  float* part_o;    // [row][split][d], normalised
  float* part_lse;  // [row][split], base 2
  int max_len;
  int* status;
};

// Slots [first, last) of split x.
__device__ __forceinline__ void split_slots(const Step& a, int x, int& first, int& last) {
  const int group = x / a.sp.parts, own = a.sp.own, listed = a.dm.shared ? own + 1 : own;
  first = group < a.sp.groups ? group * a.sp.slots : own;
  last = group < a.sp.groups ? min(first + a.sp.slots, listed) : own + 1;
}

// Keys [lo, hi) of one slot of split x, for a row at position p (empty: lo >= hi).
// An index row lists the chosen earlier blocks, then the own block; the last
// slot stands for the own block wherever it is listed.
__device__ __forceinline__ void slot_range(const Step& a, const int32_t* list, int x, int slot,
                                           int p, int& lo, int& hi) {
  const int B = a.dm.B, own = p / B;
  lo = hi = 0;
  if (!MOBA_CHECK(slot <= a.sp.own && a.sp.own < a.dm.topk, a.status)) return;
  const int e = slot == a.sp.own ? own : list[slot];
  if (slot == a.sp.own || (e >= 0 && e < own)) {
    // counted inside the block: where its last parts would begin need not be a position
    const int n = e < own ? B : p - own * B + 1, from = x % a.sp.parts * a.sp.keys;
    if (from < n) {
      lo = e * B + from;
      hi = lo + min(a.sp.keys, n - from);
    }
  }
}

// First rows of the pages that hold keys [lo, hi) of request r, kv head g: -1
// (and a status code) where the table names no page. room: entries of page_row.
template <int kThreads>
__device__ __forceinline__ void load_pages(const Step& a, int r, int g, int lo, int hi,
                                           int* page_row, int room) {
  const Cache& c = a.c;
  const int p0 = lo >> c.page_log2, np = lo < hi ? ((hi - 1) >> c.page_log2) - p0 + 1 : 0;
  for (int i = threadIdx.x; i < np; i += kThreads) {
    if (!MOBA_CHECK(i < room && p0 + i < c.max_pages, a.status)) break;
    const int64_t row =
        cache_page_row(c, a.dm.Hkv, c.table[(int64_t)r * c.max_pages + p0 + i], g);
    page_row[i] = (int)row;  // rows of a cache fit 31 bits (checked on the host)
    if (row < 0) set_status(a.status, kStBadIndices);
  }
}

// ---- gate --------------------------------------------------------------------
// Scores of the complete earlier blocks by their means, and the best k - 1 of
// them (ties to the lower index, a NaN score never), in ascending order, then
// the own block, then -1.
//
// One cluster per (query, kv head): its CTAs take equal ranges of the blocks, a
// warp reads a mean as 16 bytes a lane and forms its product with every q row
// of the group (one row, their sum, with shared routing), and the scores meet
// in the first CTA's shared memory, where a warp a row picks the best by rounds
// of arg-max. A mean is read once for the group's rows, not once a row, and no
// thread walks a list alone: 39 -> 16 us for four queries at the million-token
// cache (1 MB of means: latency, not bandwidth).
//
// With at most kOwnGate blocks there is no such launch: every split chooses for
// its row itself (choose_blocks), which costs it less than the launch and the
// wait for it would. us in a graph, chosen by a launch -> by each split: 48 requests,
// two of 32, 48, 64 blocks of 512, shared, 53.7 -> 35.9, 54.7 -> 37.6, 54.7 -> 38.2; 4
// requests, 11 of 64, 54.3 -> 45.8; 4 short ones, two of 64 blocks of 128, 15.6 -> 10.6.
// 64 is what two words of a warp's flags hold. With four words the split's own choice
// was still the quicker one at 65 and 128 blocks (54.2 -> 38.1 and 56.2 -> 41.2; 53.6 ->
// 45.5 and 55.5 -> 49.4): it is not taken that far yet.
constexpr int kGateThreads = 256;
constexpr int kGateRows = 16;       // q rows of a group at a time, at most
constexpr int kGateScores = 49152;  // scores that fit: 192 KB, rows times blocks

constexpr int kOwnGate = 64;

// The index row of heads h0 .. h0 + n - 1 taken together (n > 1: shared
// routing), by a whole CTA into shared memory.
struct OwnGate {
  float score[kOwnGate];
  int32_t list[32];
};
template <typename T, int D, int kThreads>
__device__ __forceinline__ void choose_blocks(const Step& a, const T* __restrict__ q, int qi, int r,
                                              int h0, int n, int p, float* qs, OwnGate& og) {
  const Dims& dm = a.dm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = h0 / (dm.Hq / dm.Hkv), c = p / dm.B;
  int need = min(dm.topk - 1, c);
  if (need > 0 && !MOBA_CHECK(c <= kOwnGate && c < dm.nb && r < dm.batch, a.status)) need = 0;
  for (int x = tid; x < D; x += kThreads) {
    float s = 0.f;
    for (int j = 0; j < n; ++j) s += to_f32(q[((int64_t)qi * dm.Hq + h0 + j) * D + x]);
    qs[x] = s;
  }
  __syncthreads();
  constexpr int LPB = D / 4, BPW = 32 / LPB, U = 4, stride = kThreads / 32 * BPW;
  const int sub = lane % LPB, i_first = warp * BPW + lane / LPB;
  const float4 qv = reinterpret_cast<const float4*>(qs)[sub];
  for (int i0 = i_first; need > 0 && __any_sync(0xffffffffu, i0 < c); i0 += stride * U) {
    float4 kv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * stride;
      kv[u] = i < c ? __ldg(reinterpret_cast<const float4*>(
                                a.kbar + (((int64_t)r * dm.nb + i) * dm.Hkv + g) * D) + sub)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float acc = fmaf(kv[u].w, qv.w, fmaf(kv[u].z, qv.z, fmaf(kv[u].y, qv.y, kv[u].x * qv.x)));
#pragma unroll
      for (int off = LPB / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
      if (sub == 0 && i0 + u * stride < c) og.score[i0 + u * stride] = acc;
    }
  }
  __syncthreads();
  if (warp == 0) {
    float v[2] = {lane < c ? og.score[lane] : NAN, lane + 32 < c ? og.score[lane + 32] : NAN};
    uint32_t f[2] = {0u, 0u};  // chosen among blocks 0 .. 31 and 32 .. 63
    int taken = 0;
    for (; taken < need; ++taken) {
      float bs = -INFINITY;
      int bi = INT_MAX;
#pragma unroll
      for (int z = 0; z < 2; ++z)
        if (v[z] > bs || (v[z] == bs && lane + 32 * z < bi)) {
          bs = v[z];
          bi = lane + 32 * z;
        }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        const float os = __shfl_xor_sync(0xffffffffu, bs, off);
        const int oi = __shfl_xor_sync(0xffffffffu, bi, off);
        if (os > bs || (os == bs && oi < bi)) {
          bs = os;
          bi = oi;
        }
      }
      if (bi == INT_MAX) break;  // only NaN scores are left
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        if (bi == lane + 32 * z) v[z] = NAN;
        if (bi / 32 == z) f[z] |= 1u << (bi & 31);
      }
    }
    const uint32_t below = (1u << lane) - 1;
    if (f[0] >> lane & 1) og.list[__popc(f[0] & below)] = lane;
    if (f[1] >> lane & 1) og.list[__popc(f[0]) + __popc(f[1] & below)] = lane + 32;
    if (taken + lane < dm.topk) og.list[taken + lane] = lane == 0 ? c : -1;
  }
  __syncthreads();
}

template <typename T, int D>
__global__ void __launch_bounds__(kGateThreads)
cache_gate_kernel(const Step a, const T* __restrict__ q, const int cs, const int max_rows) {
  extern __shared__ __align__(16) float score[];  // [rows][c], then flags [rows][c / 32]
  __shared__ __align__(16) float qs[kGateRows][D];
  tc::grid_let_next();
  const Dims& dm = a.dm;
  const int grp = dm.Hq / dm.Hkv, chunks = dm.shared ? 1 : (grp + max_rows - 1) / max_rows;
  const int rank = blockIdx.x % cs, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int unit = blockIdx.x / cs;
  const int h_first = unit % chunks * max_rows;
  unit /= chunks;
  const int g = unit % dm.Hkv, qi = unit / dm.Hkv;
  const int h0 = g * grp + h_first;
  const int rows = dm.shared ? 1 : min(max_rows, grp - h_first);
  for (int e = tid; e < rows * D; e += kGateThreads) {
    const T* src = q + ((int64_t)qi * dm.Hq + h0 + e / D) * D + e % D;
    float s = to_f32(*src);
    if (dm.shared)
      for (int j = 1; j < grp; ++j) s += to_f32(src[j * D]);
    qs[e / D][e % D] = s;
  }
  int r, len, p;
  if (!tail_position(a.cu_q, a.c.lens, dm.batch, dm.T, a.max_len, qi, r, p, len, a.status,
                     true))
    return;
  const int c = p / dm.B, need = min(dm.topk - 1, c);
  if (!MOBA_CHECK(c < dm.nb && rows * c <= kGateScores && r < dm.batch, a.status)) return;
  if (need > 0) {
    tc::cluster_sync();  // also: CTA 0 runs, so its shared memory can be written
    constexpr int LPB = D / 4, BPW = 32 / LPB, U = 8;  // lanes a mean, means a warp, steps in flight
    const int sub = lane % LPB, per = (c + cs - 1) / cs;
    const int first = rank * per, end = min(c, first + per), stride = kGateThreads / 32 * BPW;
    for (int i0 = first + warp * BPW + lane / LPB; __any_sync(0xffffffffu, i0 < end);
         i0 += stride * U) {
      float4 kv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * stride;
        kv[u] = i < end ? __ldg(reinterpret_cast<const float4*>(
                                    a.kbar + (((int64_t)r * dm.nb + i) * dm.Hkv + g) * D) + sub)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      for (int j = 0; j < rows; ++j) {
        const float4 qv = reinterpret_cast<const float4*>(qs[j])[sub];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float acc = fmaf(kv[u].w, qv.w, fmaf(kv[u].z, qv.z, fmaf(kv[u].y, qv.y, kv[u].x * qv.x)));
#pragma unroll
          for (int off = LPB / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
          if (sub == 0 && i0 + u * stride < end)
            tc::store_first(&score[j * c + i0 + u * stride], acc);
        }
      }
    }
  }
  tc::cluster_sync();
  if (rank != 0) return;
  const int words = (c + 31) / 32;
  for (int j = warp; j < rows; j += kGateThreads / 32) {
    uint32_t* flags = reinterpret_cast<uint32_t*>(score + (int64_t)rows * c) + j * words;
    for (int w = lane; w < words; w += 32) flags[w] = 0;
    __syncwarp();
    float* sc = score + j * c;
    // a lane keeps the best of its blocks, lane, lane + 32, ...; when it is
    // taken the whole warp looks that lane's blocks through again
    auto best = [&](float s, int i, float& bs, int& bi) {
      if (s > bs || (s == bs && i < bi)) {
        bs = s;
        bi = i;
      }
    };
    auto over_lanes = [&](float& bs, int& bi) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
        best(__shfl_xor_sync(0xffffffffu, bs, off), __shfl_xor_sync(0xffffffffu, bi, off), bs, bi);
    };
    float ms = -INFINITY;
    int mi = INT_MAX, n = 0;
    if (need > 0)
      for (int i = lane; i < c; i += 32) best(sc[i], i, ms, mi);
    for (; n < need; ++n) {
      float bs = ms;
      int bi = mi;
      over_lanes(bs, bi);
      if (bi == INT_MAX) break;  // only NaN scores are left
      const int owner = bi & 31;
      if (lane == owner) {
        sc[bi] = NAN;
        flags[bi / 32] |= 1u << owner;
      }
      __syncwarp();
      float ts = -INFINITY;
      int ti = INT_MAX;
      for (int i = owner + 32 * lane; i < c; i += 1024) best(sc[i], i, ts, ti);
      over_lanes(ts, ti);
      if (lane == owner) {
        ms = ts;
        mi = ti;
      }
    }
    __syncwarp();
    const int copies = dm.shared ? grp : 1;
    int32_t* row = a.idx + ((int64_t)qi * dm.Hq + h0 + (dm.shared ? 0 : j)) * dm.topk;
    int done = 0;  // ascending: 32 words of flags at a time, one a lane
    for (int w0 = 0; w0 < words && n > 0; w0 += 32) {
      const uint32_t f = w0 + lane < words ? flags[w0 + lane] : 0u;
      int at = __popc(f);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, at, off);
        if (lane >= off) at += o;
      }
      const int total = __shfl_sync(0xffffffffu, at, 31);
      for (int x = 0; x < copies; ++x) {
        int o = done + at - __popc(f);
        for (uint32_t m = f; m; m &= m - 1)
          row[(int64_t)x * dm.topk + o++] = (w0 + lane) * 32 + __ffs(m) - 1;
      }
      done += total;
    }
    for (int x = 0; x < copies; ++x)
      if (n + lane < dm.topk) row[(int64_t)x * dm.topk + n + lane] = lane == 0 ? c : -1;
  }
}

// The exponent that takes a q row whose largest magnitude is `top` into [1, 2),
// as far as 2^-e and 2^e are normal numbers; 0 for one that is infinite or zero.
// A logit is (q 2^-e . codes) (2^e key scale): the sum cannot overflow, and where
// the large query meets a small scale neither does the factor (q . codes taken
// first gave infinities for queries of 2^120 on keys of 2^-118).
__device__ __forceinline__ int q_exponent(float top) {
  const int e = (int)(__float_as_uint(top) >> 23) - 127;
  return e == 128 || top == 0.f ? 0 : min(max(e, -126), 126);
}
__device__ __forceinline__ float power_of_two(int e) {  // e in [-126, 127]
  return __uint_as_float((uint32_t)(127 + e) << 23);
}

// ---- bf16 queries ------------------------------------------------------------
// One CTA per split: of one head for the chosen blocks (each head has its own),
// of up to 8 heads of a kv head for the own block, which they share, and for
// every block with shared routing. A warp owns steps of 32 keys, w, w + 4, ...;
// codes come by TMA in tiles of 16 rows (never across a page: pages are 16 or
// more, tiles are aligned to 16 positions) into the warp's ring of two
// steps, so the bytes in flight do not cost registers.
//
// The products run on m16n8k16 f16 instructions: e4m3 widens to f16 exactly in
// one conversion for two values, half of what fp32 FMA needs with its second
// widening, and the 8 columns take the group's heads at no cost. (A tcgen05
// product would want 64 or 128 query rows; a step here has 1 to 8.)
//   S^T = K Q^T   A: 16 keys; a lane's 16-byte pieces of two rows are its A
//                 registers as they come, d being permuted alike in Q
//   O^T = V^T P^T A: 16 dims; pairs of keys interleaved by byte permutes; P
//                 reaches the B layout by two 8 x 8 transposes
// q is scaled to [1, 2) by a power of two a head, since f16 has a narrower
// range than bf16: what drops out is 2^-24 of the largest entry. Weights times
// value scales are rounded to f16 (half a step of 2^-11) relative to a
// reference that the warp raises, with its sums, when one passes it by 2^8;
// sums of weights stay fp32.
//
// Four queries on a million-token cache (32 heads, 12 of 256 blocks of 4096,
// 1.44 GB of rows): 237 us, 6.1 TB/s; the same loop with fp32 FMA and loads to
// registers, 462. What it took: the conversion instruction written out in place of
// the toolkit's function (396 -> 325), references raised
// only when passed and whole steps without masks, two-step rings for three CTAs
// an SM instead of three-step ones for two (325 -> 236).
constexpr int kW = 4;        // warps
constexpr int kStages = 2;   // steps in a warp's ring: three CTAs an SM, 192 KB in flight
constexpr int kStep = 32;    // keys a step
constexpr int kHeads = 8;    // columns

template <int D>
struct Ring {
  static constexpr int kTile = 16 * D;             // 16 rows of codes
  static constexpr int kStage = 4 * kTile;         // K and V of a step
  static constexpr int kBytes = kW * kStages * kStage;
};

// Four e4m3 values as two pairs of f16 (exact).
__device__ __forceinline__ void widen4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float max_over_keys(float x) {  // over the 8 lanes of a column
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
template <int D>
__global__ void __launch_bounds__(kW * 32, 3)
cache_attn_tc(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
              const Step a, const __nv_bfloat16* __restrict__ q, __nv_bfloat16* __restrict__ out,
              float* __restrict__ lse_out) {
  extern __shared__ __align__(1024) uint8_t ring[];
  __shared__ uint64_t full[kW][kStages];
  __shared__ __align__(16) uint8_t scales[kW][kStages][2][kStep];
  __shared__ int page_row[kMaxPages];
  __shared__ float wm[kW][kHeads], wo[kW][kHeads], wl[kW][kHeads];
  __shared__ __align__(16) float qs[D];
  __shared__ OwnGate og;
  __shared__ int abort_flag;
  constexpr int NC = D / 64;  // 16-byte pieces of a row a lane holds
  using R = Ring<D>;
  tc::grid_let_next();
  const Dims& dm = a.dm;
  const Cache& cc = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r8 = lane >> 2, c4 = lane & 3;
  if (warp == 0 && lane < 2) tc::prefetch_map(lane ? &tmv : &tmk);
  // ---- which split, of which heads
  const int grp = dm.Hq / dm.Hkv, hc = (grp + kHeads - 1) / kHeads;
  const int n_hist = dm.shared ? 0 : dm.Hq * a.sp.groups * a.sp.parts;
  const int per = dm.shared ? a.sp.per_row : a.sp.parts;  // splits that a group's heads share
  const int n_group = dm.Hkv * hc * per;
  const int qi = blockIdx.x / (n_hist + n_group);
  int u = blockIdx.x % (n_hist + n_group), h0, nh, s;
  if (u < n_group) {
    s = u % per + (a.sp.per_row - per);
    u /= per;
    h0 = u / hc * grp + u % hc * kHeads;
    nh = min(kHeads, grp - u % hc * kHeads);
  } else {
    u -= n_group;
    s = u % (a.sp.groups * a.sp.parts);
    h0 = u / (a.sp.groups * a.sp.parts);
    nh = 1;
  }
  const int g = h0 / grp;
  const int64_t row0 = (int64_t)qi * dm.Hq + h0;
  // ---- q of head r8: this lane's pieces, f16, scaled into [1, 2)
  uint32_t qf[NC * 8];
  float qe = 0.f;  // what head r8's logits are multiplied by
  {
    float x[NC * 16], top = 0.f;
#pragma unroll
    for (int m = 0; m < NC; ++m) {
      const __nv_bfloat16* src = q + (row0 + (r8 < nh ? r8 : 0)) * D + (c4 * NC + m) * 16;
      Vec16<__nv_bfloat16>::load(src, x + m * 16);
      Vec16<__nv_bfloat16>::load(src + 8, x + m * 16 + 8);
    }
#pragma unroll
    for (int i = 0; i < NC * 16; ++i) {
      if (r8 >= nh) x[i] = 0.f;
      top = fmaxf(top, fabsf(x[i]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = q_exponent(top);
    const float f = power_of_two(-e);
    qe = power_of_two(e) * (kLog2e * rsqrtf((float)D));
#pragma unroll
    for (int i = 0; i < NC * 8; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i] * f, x[2 * i + 1] * f);
      qf[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  // of this lane's two columns
  const float qe0 = __shfl_sync(0xffffffffu, qe, c4 * 8), qe1 = __shfl_sync(0xffffffffu, qe, c4 * 8 + 4);
  if (lane == 0)
    for (int i = 0; i < kStages; ++i) tc::mbar_init(&full[warp][i], 1);
  if (tid == 0) abort_flag = 0;
  tc::mbar_fence_init();
  int r, len, p;
  const bool valid =
      tail_position(a.cu_q, cc.lens, dm.batch, dm.T, a.max_len, qi, r, p, len,
                    a.gated ? nullptr : a.status, true);
  // a split of own blocks alone needs no choice, and the merge waits for others
  // that did wait
  if (s < a.sp.groups * a.sp.parts || a.sp.groups == 0) tc::grid_wait();
  if (!valid) return;
  const int32_t* list = a.idx + row0 * dm.topk;
  if (!a.gated && a.sp.groups > 0 && s < a.sp.groups * a.sp.parts) {
    choose_blocks<__nv_bfloat16, D, kW * 32>(a, q, qi, r, dm.shared ? g * grp : h0,
                                             dm.shared ? grp : 1, p, qs, og);
    list = og.list;
  }
  if (!a.gated && s == 0)
    for (int e = tid; e < nh * dm.topk; e += kW * 32)
      a.idx[row0 * dm.topk + e] = a.sp.groups > 0 ? og.list[e % dm.topk]
                                              : e % dm.topk == 0 ? p / dm.B : -1;
  const int page = 1 << cc.page_log2;
  // lane x of every warp: slot x of the split, its keys, steps and page entries
  int my_lo = 0, my_hi = 0, my_step, my_page;  // step: one past the slot's last; page: its first
  {
    int first, last;
    split_slots(a, s, first, last);
    if (first + lane < last) slot_range(a, list, s, first + lane, p, my_lo, my_hi);
    const int t0 = my_lo & ~15, np = my_lo < my_hi ? ((my_hi - 1) / page - t0 / page) + 1 : 0;
    my_step = my_lo < my_hi ? (my_hi - t0 + kStep - 1) / kStep : 0;
    my_page = np;
#pragma unroll
    for (int off = 1; off < kMaxSlots; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, my_step, off);
      const int y = __shfl_up_sync(0xffffffffu, my_page, off);
      if (lane >= off) {
        my_step += x;
        my_page += y;
      }
    }
    my_page -= np;
  }
  const int n_steps = __shfl_sync(0xffffffffu, my_step, kMaxSlots - 1);
  if (n_steps == 0) {  // no keys (uniform over the CTA; never the only split of a row)
    if (tid < nh && MOBA_CHECK(row0 + tid < (int64_t)dm.T * dm.Hq && s < a.sp.per_row, a.status))
      a.part_lse[(row0 + tid) * a.sp.per_row + s] = -INFINITY;
    return;
  }
  // A walk over the steps: the slot of the current one.
  struct Walk {
    int slot, lo, hi, step, end, page;
  };
  auto enter = [&](Walk& w, int x) {
    w.slot = x;
    w.lo = __shfl_sync(0xffffffffu, my_lo, x);
    w.hi = __shfl_sync(0xffffffffu, my_hi, x);
    w.end = __shfl_sync(0xffffffffu, my_step, x);
    w.step = x ? __shfl_sync(0xffffffffu, my_step, x ? x - 1 : 0) : 0;
    w.page = __shfl_sync(0xffffffffu, my_page, x) - (w.lo >> cc.page_log2);
  };
  Walk wr, wc;  // of the requests, of the computation
  enter(wr, 0);
  for (int x = 0;; enter(wr, ++x)) {
    const int at = wr.page + (wr.lo >> cc.page_log2);
    load_pages<kW * 32>(a, r, g, wr.lo & ~15, wr.hi, page_row + at, kMaxPages - at);
    if (wr.end == n_steps) break;
  }
  enter(wr, 0);
  enter(wc, 0);
  __syncthreads();
  const uint32_t base = tc::smem_u32(ring) + warp * kStages * R::kStage;
  // moves a walk to step i (its slots rise); the step's first position
  auto locate = [&](Walk& w, int i) {
    while (i >= w.end) enter(w, w.slot + 1);
    return (w.lo & ~15) + (i - w.step) * kStep;
  };
  // the cache row that 16 keys from pos begin at, or -1: nothing to read
  auto tile_row = [&](const Walk& w, int pos) {
    if (pos >= w.hi) return -1;
    const int pr = page_row[w.page + (pos >> cc.page_log2)], row = pr + (pos & (page - 1));
    return pr < 0 || !MOBA_CHECK(cache_holds(cc, dm.Hkv, (int64_t)row + 15), a.status) ? -1 : row;
  };
  // the loads of step i, one lane a copy: tile lane / 4, then K, V and their scales
  auto request = [&](int i, int st) {
    const int t = lane >> 2 & 1, what = lane & 3;
    const int pos = locate(wr, i), at = tile_row(wr, pos + t * 16);
    uint64_t* bar = &full[warp][st];
    const uint32_t there = __ballot_sync(0xffffffffu, at >= 0);
    if (lane == 0)
      tc::mbar_expect_tx(bar, ((there & 1) + (there >> 4 & 1)) * (2 * R::kTile + 32));
    __syncwarp();
    if (lane < 8 && at >= 0) {
      if (what < 2)
        tc::tma_load_2d(base + st * R::kStage + (what * 2 + t) * R::kTile, what ? &tmv : &tmk, bar,
                        0, at);
      else
        tc::bulk_load(tc::smem_u32(&scales[warp][st][what - 2][t * 16]),
                      (what == 2 ? cc.ks : cc.vs) + at, 16, bar);
    }
  };
  for (int x = 0; x < kStages && warp + x * kW < n_steps; ++x) request(warp + x * kW, x);
  volatile int* abort = &abort_flag;
  // columns 2 c4 and 2 c4 + 1: references of the logits and of logit plus
  // value exponent, and the sum of weights
  float mr[2] = {-INFINITY, -INFINITY}, mo[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float qc[2] = {qe0, qe1};
  float acc[D / 16][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[i][x] = 0.f;

  // One step of 32 keys whose codes are in stage st. `one`: only column 0 of
  // lane column 0 is a head, so the second column is left out. `whole`: every
  // key counts.
  auto step = [&](auto one_t, auto whole_t, int from, int st) {
    constexpr int NCOL = decltype(one_t)::value ? 1 : 2;
    constexpr bool whole = decltype(whole_t)::value;
    const int lo = wc.lo, hi = wc.hi;
    const uint32_t sK = base + st * R::kStage, sV = sK + 2 * R::kTile;
    float x[2][2][NCOL], ev[2][2];
    bool on[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      float sc[4] = {0.f, 0.f, 0.f, 0.f};
      uint4 k0[NC], k1[NC];
#pragma unroll
      for (int m = 0; m < NC; ++m) {
        const int piece = c4 * NC + m;
        const uint32_t at = sK + t * R::kTile + r8 * D +
                            ((D == 128 ? piece ^ r8 : piece ^ (r8 >> 1 & 3)) << 4);
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(k0[m].x), "=r"(k0[m].y), "=r"(k0[m].z), "=r"(k0[m].w)
                     : "r"(at));
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(k1[m].x), "=r"(k1[m].y), "=r"(k1[m].z), "=r"(k1[m].w)
                     : "r"(at + 8 * D));
      }
#pragma unroll
      for (int m = 0; m < NC; ++m) {
        const uint32_t w0[4] = {k0[m].x, k0[m].y, k0[m].z, k0[m].w};
        const uint32_t w1[4] = {k1[m].x, k1[m].y, k1[m].z, k1[m].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t fa[4];
          widen4(w0[w], fa[0], fa[2]);
          widen4(w1[w], fa[1], fa[3]);
          mma16816(sc, fa, qf[m * 8 + w * 2], qf[m * 8 + w * 2 + 1]);
        }
      }
      const int pos = from + t * 16;
      const bool there = whole || tile_row(wc, pos) >= 0;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int kp = pos + r8 + 8 * y;
        on[t][y] = whole || (there && kp >= lo && kp < hi);
        const float ks = e8m0_value(scales[warp][st][0][t * 16 + r8 + 8 * y]);
        const uint32_t vb = scales[warp][st][1][t * 16 + r8 + 8 * y];
        ev[t][y] = vb == 255 ? NAN : (float)((int)vb - 127);
#pragma unroll
        for (int z = 0; z < NCOL; ++z)
          x[t][y][z] = on[t][y] ? sc[2 * y + z] * (qc[z] * ks) : -INFINITY;
      }
    }
    // ---- references: raised when a value passes one by 2^8 (the first always does)
    bool up = false;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int z = 0; z < NCOL; ++z)
          up = up || x[t][y][z] > mr[z] + 8.f || (on[t][y] && x[t][y][z] + ev[t][y] > mo[z] + 8.f);
    if (__any_sync(0xffffffffu, up)) {
      float f[2] = {1.f, 1.f};
#pragma unroll
      for (int z = 0; z < NCOL; ++z) {
        float a0 = mr[z], a1 = mo[z];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            a0 = fmaxf(a0, x[t][y][z]);
            if (on[t][y]) a1 = fmaxf(a1, x[t][y][z] + ev[t][y]);
          }
        a0 = max_over_keys(a0);
        a1 = max_over_keys(a1);
        if (mr[z] != -INFINITY) l[z] *= tc::ex2(mr[z] - a0);
        if (mo[z] != -INFINITY) f[z] = tc::ex2(mo[z] - a1);
        mr[z] = a0;
        mo[z] = a1;
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        acc[d][0] *= f[0];
        acc[d][2] *= f[0];
        acc[d][1] *= f[1];
        acc[d][3] *= f[1];
      }
    }
    // ---- weights, and their products with the values
    float rm[2], ro[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      rm[z] = mr[z] == -INFINITY ? 0.f : mr[z];
      ro[z] = mo[z] == -INFINITY ? 0.f : mo[z];
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint32_t b[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float po[2] = {0.f, 0.f};
#pragma unroll
        for (int z = 0; z < NCOL; ++z) {
          const float pw = tc::ex2(x[t][y][z] - rm[z]);
          const float ow = tc::ex2(x[t][y][z] + ev[t][y] - ro[z]);
          l[z] += on[t][y] ? pw : 0.f;
          po[z] = on[t][y] ? ow : 0.f;
        }
        const __half2 h = __floats2half2_rn(po[0], po[1]);
        b[y] = transpose8(*reinterpret_cast<const uint32_t*>(&h));
      }
      // keys 2 c4, 2 c4 + 1 and 8 further; dims r8 * D / 8 ..
      uint32_t v[4][NC * 2];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int key = 2 * c4 + (y & 1) + (y >> 1) * 8;
        const uint32_t at = sV + t * R::kTile + key * D;
        if constexpr (D == 128)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v[y][0]), "=r"(v[y][1]), "=r"(v[y][2]), "=r"(v[y][3])
                       : "r"(at + ((r8 ^ (key & 7)) << 4)));
        else
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                       : "=r"(v[y][0]), "=r"(v[y][1])
                       : "r"(at + (((r8 >> 1) ^ (key >> 1 & 3)) << 4) + (r8 & 1) * 8));
        if (!whole) {  // zero weights do not silence NaN codes behind a request
          const int kp = from + t * 16 + key;
          const bool in = kp >= lo && kp < hi && tile_row(wc, from + t * 16) >= 0;
#pragma unroll
          for (int w = 0; w < NC * 2; ++w) v[y][w] = in ? v[y][w] : 0u;
        }
      }
#pragma unroll
      for (int w = 0; w < NC * 2; ++w) {
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const uint32_t pick = z ? 0x7362u : 0x5140u;
          uint32_t fa[4];
          widen4(__byte_perm(v[0][w], v[1][w], pick), fa[0], fa[1]);
          widen4(__byte_perm(v[2][w], v[3][w], pick), fa[2], fa[3]);
          mma16816(acc[w * 2 + z], fa, b[0], b[1]);
        }
      }
    }
  };
  int n = 0;  // steps of this warp so far
  bool ok = true;
  for (int i = warp; i < n_steps; i += kW, ++n) {
    const int st = n % kStages;
    ok = tc::mbar_wait(&full[warp][st], n / kStages & 1, abort, a.status);
    if (!__all_sync(0xffffffffu, ok)) {
      ok = false;
      break;
    }
    const int pos = locate(wc, i);
    const bool whole = pos >= wc.lo && pos + kStep <= wc.hi && tile_row(wc, pos) >= 0 &&
                       tile_row(wc, pos + 16) >= 0;
    if (whole) {
      if (nh == 1)
        step(std::true_type{}, std::true_type{}, pos, st);
      else
        step(std::false_type{}, std::true_type{}, pos, st);
    } else {
      step(std::false_type{}, std::false_type{}, pos, st);
    }
    __syncwarp();  // the step's buffers are free
    if (i + kStages * kW < n_steps) request(i + kStages * kW, st);
  }
  if (!ok) {  // let the copies already issued land before the CTA exits
    for (int x = 0; x < kStages; ++x)
      if (warp + (n + x) * kW < n_steps)
        tc::mbar_drain(&full[warp][(n + x) % kStages], (n + x) / kStages & 1);
  }
  // ---- the warps' results, in their own rings
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
    l[1] += __shfl_xor_sync(0xffffffffu, l[1], off);
  }
  float* res = reinterpret_cast<float*>(ring + warp * kStages * R::kStage);  // [head][D]
#pragma unroll
  for (int d = 0; d < D / 16; ++d) {
    const int dim = r8 * (D / 8) + 2 * d;
    if (2 * c4 < nh)
      *reinterpret_cast<float2*>(res + 2 * c4 * D + dim) = make_float2(acc[d][0], acc[d][2]);
    if (2 * c4 + 1 < nh)
      *reinterpret_cast<float2*>(res + (2 * c4 + 1) * D + dim) = make_float2(acc[d][1], acc[d][3]);
  }
  if (r8 == 0) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      wm[warp][2 * c4 + z] = mr[z];
      wo[warp][2 * c4 + z] = mo[z];
      wl[warp][2 * c4 + z] = l[z];
    }
  }
  __syncthreads();
  if (*abort) return;
  for (int e = tid; e < nh * (D / 4); e += kW * 32) {
    const int h = e / (D / 4), d4 = e % (D / 4);
    if (!MOBA_CHECK(row0 + h < (int64_t)dm.T * dm.Hq && s < a.sp.per_row, a.status)) break;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kW; ++w) M = fmaxf(M, wm[w][h]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      // a warp without keys has sums 0 (or NaN, which has to show)
      L += wl[w][h] * (wm[w][h] == -INFINITY ? 1.f : tc::ex2(wm[w][h] - M));
      const float f = wo[w][h] == -INFINITY ? 1.f : exp2f(wo[w][h] - M);
      const float4 v = reinterpret_cast<const float4*>(
          ring + w * kStages * R::kStage)[h * (D / 4) + d4];
      o.x = fmaf(v.x, f, o.x);
      o.y = fmaf(v.y, f, o.y);
      o.z = fmaf(v.z, f, o.z);
      o.w = fmaf(v.w, f, o.w);
    }
    const int64_t at = (row0 + h) * a.sp.per_row + s;
    const bool none = M == -INFINITY && L == 0.f;  // bad pages only
    const float inv = 1.f / L;
    if (a.sp.per_row == 1) {  // the row's only split: this is the result
      *reinterpret_cast<uint2*>(out + (row0 + h) * D + d4 * 4) =
          none ? make_uint2(0, 0)
               : make_uint2(tc::pack_bf16x2(o.x * inv, o.y * inv),
                            tc::pack_bf16x2(o.z * inv, o.w * inv));
      if (d4 == 0 && lse_out)
        lse_out[row0 + h] = none ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
      continue;
    }
    if (!none)
      reinterpret_cast<float4*>(a.part_o + at * D)[d4] =
          make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    if (d4 == 0) a.part_lse[at] = none ? -INFINITY : L != L ? L : M + log2f(L);
  }
}

// ---- fp32 queries ------------------------------------------------------------
// One CTA per (query, q head, split), a row's 16 codes a lane, fp32 FMA.
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void decode16(const uint4& r, float (&x)[16]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * u)),
                                                       __NV_E4M3);
      const float2 f = __half22float2(__half2(h));
      x[4 * i + 2 * u] = f.x;
      x[4 * i + 2 * u + 1] = f.y;
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads)
cache_attn_kernel(const Step a, const float* __restrict__ q) {
  constexpr int LPK = D / 16, GPW = 32 / LPK, G = GPW * kWarps, U = 4;
  __shared__ float wm[kWarps], wl[kWarps];
  __shared__ __align__(16) float wo[kWarps][D];
  __shared__ int page_row[kMaxPages];
  __shared__ OwnGate og;
  tc::grid_let_next();
  const Dims& dm = a.dm;
  const Cache& c = a.c;
  const int S = a.sp.per_row;
  const int s = (int)(blockIdx.x % S), qi = (int)(blockIdx.x / S), h = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = (int64_t)qi * dm.Hq + h, prow = row * S + s;
  int r, len, p;
  const bool valid = tail_position(a.cu_q, c.lens, dm.batch, dm.T, a.max_len, qi, r, p, len,
                                   a.gated ? nullptr : a.status, true);
  tc::grid_wait();  // the chosen blocks
  if (!valid) return;
  const int grp = dm.Hq / dm.Hkv, g = h / grp;
  const int32_t* list = a.idx + row * dm.topk;
  if (!a.gated && a.sp.groups > 0 && s < a.sp.groups * a.sp.parts) {
    choose_blocks<float, D, kThreads>(a, q, qi, r, dm.shared ? g * grp : h, dm.shared ? grp : 1, p,
                                      &wo[0][0], og);
    list = og.list;
  }
  if (!MOBA_CHECK(prow < (int64_t)dm.T * dm.Hq * S, a.status)) return;
  if (!a.gated && s == 0)
    for (int e = tid; e < dm.topk; e += kThreads)
      a.idx[row * dm.topk + e] = a.sp.groups > 0 ? og.list[e] : e == 0 ? p / dm.B : -1;
  const int grp_id = warp * GPW + lane / LPK, sub = lane % LPK;
  float qv[16], top = 0.f;
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    qv[x] = q[row * D + sub * 16 + x];
    top = fmaxf(top, fabsf(qv[x]));
  }
#pragma unroll
  for (int off = LPK / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  const int qx = q_exponent(top);
  const float qe = power_of_two(qx) * (kLog2e * rsqrtf((float)D));
#pragma unroll
  for (int x = 0; x < 16; ++x) qv[x] *= power_of_two(-qx);
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) o[x] = 0.f;
  const int mask = (1 << c.page_log2) - 1;
  int first, last;
  split_slots(a, s, first, last);
  for (int slot = first; slot < last; ++slot) {
  int lo, hi;
  slot_range(a, list, s, slot, p, lo, hi);
  const int p0 = lo >> c.page_log2;
  __syncthreads();
  load_pages<kThreads>(a, r, g, lo, hi, page_row, kMaxPages);
  __syncthreads();
  for (int base = lo; base < hi; base += U * G) {
    uint4 kr[U], vr[U];
    float ks[U], vs[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = base + grp_id + u * G;
      const int jj = j < hi ? j : lo;
      const int pr = page_row[(jj >> c.page_log2) - p0];
      const bool there = pr >= 0 && MOBA_CHECK(cache_holds(c, dm.Hkv, pr + (jj & mask)), a.status);
      on[u] = j < hi && there;
      const int64_t at = there ? pr + (jj & mask) : 0;
      kr[u] = __ldg(reinterpret_cast<const uint4*>(c.k + at * D + sub * 16));
      vr[u] = __ldg(reinterpret_cast<const uint4*>(c.v + at * D + sub * 16));
      ks[u] = e8m0_value(__ldg(c.ks + at));
      vs[u] = e8m0_value(__ldg(c.vs + at));
    }
    float d[U], mn = m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[16];
      decode16(kr[u], x);
      float acc = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) acc = fmaf(qv[i], x[i], acc);
#pragma unroll
      for (int off = LPK / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
      d[u] = on[u] ? acc * (qe * ks[u]) : -INFINITY;
      mn = fmaxf(mn, d[u]);
    }
    if (mn == -INFINITY) {
      // nothing to weigh in this step, but a NaN logit must not be lost
#pragma unroll
      for (int u = 0; u < U; ++u) l += on[u] && d[u] != d[u] ? d[u] : 0.f;
      continue;
    }
    const float corr = exp2f(m - mn);
    l *= corr;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= corr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = on[u] ? exp2f(d[u] - mn) : 0.f;
      l += w;
      const float wv = on[u] ? w * vs[u] : 0.f;
      float x[16];
      decode16(vr[u], x);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = on[u] ? fmaf(wv, x[i], o[i]) : o[i];
    }
    m = mn;
  }
  }
  // merge the lane groups of the warp, then the warps
#pragma unroll
  for (int off = LPK; off < 32; off <<= 1) {
    const float mo = __shfl_xor_sync(0xffffffffu, m, off);
    const float lo2 = __shfl_xor_sync(0xffffffffu, l, off);
    const float mn = fmaxf(m, mo);
    const float fa = m == -INFINITY ? 1.f : exp2f(m - mn);
    const float fb = mo == -INFINITY ? 1.f : exp2f(mo - mn);
    l = l * fa + lo2 * fb;
#pragma unroll
    for (int x = 0; x < 16; ++x) o[x] = o[x] * fa + __shfl_xor_sync(0xffffffffu, o[x], off) * fb;
    m = mn;
  }
  if (lane < LPK) {
#pragma unroll
    for (int x = 0; x < 16; ++x) wo[warp][sub * 16 + x] = o[x];
    if (lane == 0) {
      wm[warp] = m;
      wl[warp] = l;
    }
  }
  __syncthreads();
  float M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w]);
  float L = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) L += wl[w] * (wm[w] == -INFINITY ? 1.f : exp2f(wm[w] - M));
  // a split without keys, or with bad pages only, leaves no partial;
  // one with a NaN logit leaves NaN
  const bool none = M == -INFINITY && L == 0.f;
  for (int x = tid; x < D && !none; x += kThreads) {
    float acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      acc = fmaf(wo[w][x], wm[w] == -INFINITY ? 1.f : exp2f(wm[w] - M), acc);
    a.part_o[prow * D + x] = acc / L;
  }
  if (tid == 0) a.part_lse[prow] = none ? -INFINITY : L != L ? L : M + log2f(L);
}

// ---- a row's partials --------------------------------------------------------
// Eq. (7)-(8) written with lse: w_s = 2^(lse_s - max), o = sum w_s o_s / sum w_s,
// in a fixed order. One CTA per row; warp w takes splits w, w + 4, ...
constexpr int kMergeWarps = 4;

template <typename T, int D>
__global__ void __launch_bounds__(kMergeWarps * 32)
cache_merge_kernel(const Step a, T* __restrict__ out, float* __restrict__ lse_out) {
  __shared__ float wl[kMergeWarps];
  __shared__ __align__(16) float wo[kMergeWarps][D];
  constexpr int E = D / 32;
  const int64_t row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = a.sp.per_row;
  int r, len, p;
  const bool valid = tail_position(a.cu_q, a.c.lens, a.dm.batch, a.dm.T, a.max_len,
                                   (int)(row / a.dm.Hq), r, p, len, nullptr, true);
  tc::grid_wait();  // the partials
  if (!valid) return;
  const float* ls = a.part_lse + row * S;
  float M = -INFINITY;
  for (int s = lane; s < S; s += 32) M = fmaxf(M, ls[s]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  float acc[E], L = 0.f;
#pragma unroll
  for (int x = 0; x < E; ++x) acc[x] = 0.f;
#pragma unroll 4
  for (int s = warp; s < S; s += kMergeWarps) {
    const float lv = ls[s];
    if (lv == -INFINITY) continue;  // its partial was never written; NaN counts: it has to show
    const float w = exp2f(lv - M);
    L += w;
    const float* src = a.part_o + (row * S + s) * D + lane * E;
#pragma unroll
    for (int x = 0; x < E; ++x) acc[x] = fmaf(w, src[x], acc[x]);
  }
#pragma unroll
  for (int x = 0; x < E; ++x) wo[warp][lane * E + x] = acc[x];
  if (lane == 0) wl[warp] = L;
  __syncthreads();
  for (int x = threadIdx.x; x < D; x += kMergeWarps * 32) {
    float O = 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      O += wo[w][x];
      sum += wl[w];
    }
    // sum == 0: every page of the row was bad; zeros and -inf, not 0 / 0
    out[row * D + x] = from_f32<T>(sum == 0.f ? 0.f : O / sum);
    if (x == 0 && lse_out)
      lse_out[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
  }
}

template <typename T, int D>
cudaError_t run_gate(const Step& a, const void* q, cudaStream_t st) {
  const Dims& dm = a.dm;
  const int grp = dm.Hq / dm.Hkv;
  int rows = dm.shared ? 1 : grp < kGateRows ? grp : kGateRows;
  if (rows > kGateScores / dm.nb) rows = kGateScores / dm.nb;
  const int chunks = dm.shared ? 1 : (grp + rows - 1) / rows;
  // CTAs a cluster: eight shorten the scoring of one request's many blocks (4 queries, 32
  // heads; four CTAs, eight: 256 blocks 55.0, 54.4 us, 512 blocks 61.6, 56.4), four leave
  // more clusters room at once (48 requests, shared: 128 blocks 31.0, 45.7; above the limit
  // too, 256 blocks 33.3, 49.5).
  const int cs = dm.nb > 128 ? 8 : 4;
  const int64_t grid = (int64_t)dm.T * dm.Hkv * chunks * cs;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const size_t smem = sizeof(float) * rows * ((size_t)dm.nb + (dm.nb + 31) / 32);
  cudaError_t e;
  static std::atomic<bool> ready[tc::kMaxDevices];
  if ((e = tc::allow_smem(cache_gate_kernel<T, D>,
                          (int)sizeof(float) * (kGateScores + kGateScores / 32 + kGateRows), ready)))
    return e;
  return tc::launch_cluster(cache_gate_kernel<T, D>, dim3((unsigned)grid), kGateThreads, smem, st, cs,
                            a, static_cast<const T*>(q), cs, rows);
}

template <typename T, int D>
cudaError_t run(const Step& a, const void* q, void* out, float* lse, cudaStream_t st) {
  const Dims& dm = a.dm;
  cudaError_t e = cudaSuccess;
  if (a.gated && dm.nb <= kGateScores)
    e = run_gate<T, D>(a, q, st);
  else if (a.gated)  // lists in registers instead of all scores in shared memory
    e = launch_cache_gate(dm, q, a.kbar, a.c.lens, a.cu_q, a.idx, a.max_len, a.status, st);
  if (e != cudaSuccess) return e;
  const int64_t rows = (int64_t)dm.T * dm.Hq;
  if constexpr (sizeof(T) == 2) {
    CUtensorMap mk, mv;
    const int64_t cache_rows = ((int64_t)a.c.pages * dm.Hkv) << a.c.page_log2;
    if ((e = tc::make_rows_map(&mk, a.c.k, cache_rows, D, 16))) return e;
    if ((e = tc::make_rows_map(&mv, a.c.v, cache_rows, D, 16))) return e;
    static std::atomic<bool> ready[tc::kMaxDevices];
    if ((e = tc::allow_smem(cache_attn_tc<D>, Ring<D>::kBytes, ready))) return e;
    const int hc = (dm.Hq / dm.Hkv + kHeads - 1) / kHeads;
    const int64_t per = dm.shared ? (int64_t)dm.Hkv * hc * a.sp.per_row
                                  : (int64_t)dm.Hkv * hc * a.sp.parts +
                                        (int64_t)dm.Hq * a.sp.groups * a.sp.parts;
    if (per * dm.T > INT32_MAX || rows > INT32_MAX) return cudaErrorInvalidValue;
    e = tc::launch_with(a.gated, cache_attn_tc<D>, dim3((unsigned)(per * dm.T)), kW * 32,
                        Ring<D>::kBytes, st, 1, mk, mv, a, static_cast<const __nv_bfloat16*>(q),
                          static_cast<__nv_bfloat16*>(out), lse);
    if (e != cudaSuccess || a.sp.per_row == 1) return e;
  } else {
    const int64_t x = (int64_t)a.sp.per_row * dm.T;
    if (x > INT32_MAX || rows > INT32_MAX) return cudaErrorInvalidValue;
    e = tc::launch_with(a.gated, cache_attn_kernel<D>, dim3((unsigned)x, (unsigned)dm.Hq), kThreads,
                        0, st, 1, a, static_cast<const float*>(q));
  }
  if (e != cudaSuccess) return e;
  return tc::launch_beside(cache_merge_kernel<T, D>, dim3((unsigned)rows), kMergeWarps * 32, 0, st, 1, a,
                       static_cast<T*>(out), lse);
}

}  // namespace

size_t decode_cache_partial_rows(const Dims& dm) {
  return (size_t)dm.T * dm.Hq * split_of(dm).per_row;
}

cudaError_t launch_decode_cache(const Dims& dm, const Cache& c, const void* q, const float* kbar,
                                const int32_t* cu_q, int32_t* idx, float* part_o, float* part_lse,
                                void* out, float* lse, int* status, cudaStream_t st) {
  Step a{};
  a.dm = dm;
  a.c = c;
  a.sp = split_of(dm);
  a.cu_q = cu_q;
  a.kbar = kbar;
  a.idx = idx;
  a.gated = dm.nb > kOwnGate && dm.topk > 1;
  a.part_o = part_o;
  a.part_lse = part_lse;
  a.max_len = max_positions(dm, c);
  a.status = status;
  if (dm.dtype == kBF16)
    return dm.d == 128 ? run<__nv_bfloat16, 128>(a, q, out, lse, st)
                       : run<__nv_bfloat16, 64>(a, q, out, lse, st);
  return dm.d == 128 ? run<float, 128>(a, q, out, lse, st)
                     : run<float, 64>(a, q, out, lse, st);
}

}  // namespace moba
