// A paged KV cache in 8 bits: rows are quantised as they are written, and
// read back. It holds what the decode step of PaperTrace "2.1.3 MoBA",
// section 5.4 reads (the bound there is the KV bytes: 1 + 1/d bytes a value
// here against 2) and keeps the block means of section 5.1.
//
// One row x of K or V (one token, one kv head) is kept as e4m3 codes c and a
// power of two 2^e, x ~ c * 2^e:
//   e = the smallest integer with max|x| <= 448 * 2^e, at least -127;
//   c = x * 2^-e rounded once to e4m3 (ties to even).
// A power of two scales without rounding, and e4m3 keeps its relative step
// over 15 binades, so a free scale would not be closer except below them.
// From e = 120 on (max|x| > 1.75 * 2^127) codes stop at 240, so that reading
// back stays finite. A row that holds an infinity or a NaN gets the scale
// NaN (byte 255): it reads back as NaN rather than as numbers.
#include <cuda_fp8.h>

#include "tc_ptx.cuh"

namespace moba {
namespace {

constexpr int kThreads = 128;  // write and read: four warps that share nothing
constexpr int kMeanThreads = 256;
constexpr int kMaxCluster = 8;
// SMs of a B200: what the work of a warp is sized by. A constant, so that the size of
// the write's workspace follows from the call alone and not from the device that is
// current when it is asked for.
constexpr int kSMs = 148;

// Exponent of a row whose largest magnitude has the fp32 bits `top` (finite).
__device__ __forceinline__ int row_exponent(uint32_t top) {
  // top = 1.man * 2^(ex - 127), 448 = 1.75 * 2^8; below 2^-126, 2^-127 holds it
  const int e = (int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return top < 0x00800000u || e < -127 ? -127 : e;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t c;
  asm("max.u16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
  return c;
}

// 16 bytes of a row: as they are, their largest magnitude as fp32 bits, and
// as fp32 values.
__device__ __forceinline__ uint32_t top_of(const uint4& r, __nv_bfloat16) {
  const uint32_t a = max_u16x2(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu);
  const uint32_t b = max_u16x2(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu);
  const uint32_t c = max_u16x2(a, b);
  return max(c << 16, c & 0xffff0000u);
}
__device__ __forceinline__ uint32_t top_of(const uint4& r, float) {
  return max(max(r.x & 0x7fffffffu, r.y & 0x7fffffffu), max(r.z & 0x7fffffffu, r.w & 0x7fffffffu));
}
// 16 bytes of a row times 2^-e, e in [-127, 120] (so a normal number), as fp32.
// For bf16 one multiply-add of mixed precision a value (exact), which spares
// the integer pipe two unpacking instructions: it is the busier one here.
__device__ __forceinline__ void scaled(const uint4& r, int e, float (&x)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  const uint16_t f = (uint16_t)((127 - e) << 7);  // bf16
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "fma.rn.f32.bf16 %0, l, %3, %4;\n\tfma.rn.f32.bf16 %1, h, %3, %4;\n\t}"
        : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
        : "r"(w[i]), "h"(f), "f"(0.f));
}
__device__ __forceinline__ void scaled(const uint4& r, int e, float (&x)[4]) {
  const float f = __uint_as_float((uint32_t)(127 - e) << 23);
  x[0] = __uint_as_float(r.x) * f;
  x[1] = __uint_as_float(r.y) * f;
  x[2] = __uint_as_float(r.z) * f;
  x[3] = __uint_as_float(r.w) * f;
}

// Scaled values, |x| <= 448, as e4m3 bytes.
template <int N>
__device__ __forceinline__ void encode(const float (&x)[N], uint32_t (&w)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N; i += 4)
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
        : "=r"(w[i / 4])
        : "f"(x[i]), "f"(x[i + 1]), "f"(x[i + 2]), "f"(x[i + 3]));
}

__device__ __forceinline__ void decode4(uint32_t four, float* x) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}
__device__ __forceinline__ void decode16(const uint4& r, float (&x)[16]) {
  decode4(r.x, x);
  decode4(r.y, x + 4);
  decode4(r.z, x + 8);
  decode4(r.w, x + 12);
}

// Row index in the cache of position pos of request r and kv head g, or -1
// (and a status code) where the page table names no page.
__device__ __forceinline__ int64_t cache_row(const Cache& c, int Hkv, int r, int pos, int g,
                                             int* status) {
  if (!MOBA_CHECK(pos >= 0 && (pos >> c.page_log2) < c.max_pages, status)) return -1;
  const int page = c.table[(int64_t)r * c.max_pages + (pos >> c.page_log2)];
  const int64_t first = cache_page_row(c, Hkv, page, g);
  if (first < 0) {
    set_status(status, kStBadIndices);
    return -1;
  }
  const int64_t row = first + (pos & ((1 << c.page_log2) - 1));
  return MOBA_CHECK(cache_holds(c, Hkv, row), status) ? row : -1;
}

// Warp of a write or read: head and tokens it takes. blockIdx.y: K or V.
// A warp takes `tpw` consecutive tokens of one head, so that their rows are
// neighbours in a page; lane t looks token t's row up (-1: none) while the
// rows are on their way.
struct WarpPlace {
  int g, t0, n;  // head, first token, tokens
  int row;       // lane t: cache row of token t0 + t
};
__device__ __forceinline__ WarpPlace warp_place(const Dims& dm, int tpw) {
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  WarpPlace p;
  p.g = (int)(w % dm.Hkv);
  const int64_t t0 = w / dm.Hkv * tpw;
  p.t0 = (int)(t0 < dm.T ? t0 : dm.T);
  p.n = min(tpw, dm.T - p.t0);
  p.row = -1;
  return p;
}
__device__ __forceinline__ int token_row(const Dims& dm, const Cache& c,
                                         const int32_t* __restrict__ cu, const WarpPlace& p,
                                         int* status) {
  const int lane = threadIdx.x & 31;
  int r, pos, len;
  if (lane >= p.n ||
      !tail_position(cu, c.lens, dm.batch, dm.T, max_positions(dm, c), p.t0 + lane, r, pos, len,
                     status))
    return -1;
  return (int)cache_row(c, dm.Hkv, r, pos, p.g, status);
}

// Quantise and store: a row is held by LPR lanes of 16 bytes, which share its
// maximum (as integers: an infinity or NaN is above every number). U rows' loads
// a lane are in flight. Bound by HBM: d * sizeof(T) bytes in, d + 1 out. (A lane
// group a row of any head, with a table look-up before each store and one-byte
// scale stores, took 663 us for 262144 tokens of 8 heads, bf16, d = 128.)
//
// sums: with 32 tokens a warp, also the sum of each warp's rows of K as stored,
// [token / 32][head][d], which the block means are made of. With them that call
// takes 285 us (5.7 TB/s) and the integer pipe is two thirds busy; without, 257,
// but the means then read all codes again: 325 in all, against 287.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
cache_write_kernel(Dims dm, Cache c, const T* __restrict__ k, const T* __restrict__ v,
                   const int32_t* __restrict__ cu_new, int tpw, float* __restrict__ sums,
                   int* status) {
  constexpr int VEC = Vec16<T>::N, LPR = D / VEC, RPS = 32 / LPR, U = 8;  // rows a step
  tc::grid_let_next();
  const int lane = threadIdx.x & 31, sub = lane % LPR, sel = lane / LPR;
  const T* __restrict__ src = blockIdx.y ? v : k;
  uint8_t* __restrict__ codes = blockIdx.y ? c.v : c.k;
  uint8_t* __restrict__ scales = blockIdx.y ? c.vs : c.ks;
  WarpPlace p = warp_place(dm, tpw);
  if (p.n <= 0) return;
  const T* base = src + ((int64_t)p.t0 * dm.Hkv + p.g) * D + sub * VEC;
  uint32_t mine = 255;  // lane t: scale byte of token t
  const bool add = sums && blockIdx.y == 0;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
  for (int s0 = 0; s0 < p.n; s0 += RPS * U) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = s0 + u * RPS + sel;
      x[u] = t < p.n ? __ldg(reinterpret_cast<const uint4*>(base + (int64_t)t * dm.Hkv * D))
                     : make_uint4(0, 0, 0, 0);
    }
    if (s0 == 0) p.row = token_row(dm, c, cu_new, p, status);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = s0 + u * RPS + sel;
      uint32_t top = top_of(x[u], T{});
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
      const bool fine = top < 0x7f800000u;
      const int e = row_exponent(top);
      float y[VEC];
      scaled(x[u], e, y);
      uint32_t w[VEC / 4];
      encode<VEC>(y, w);
      // rare, so behind a branch of the whole warp: rows that are not finite,
      // and codes above 240 (0x77) from e = 120 on
      if (__any_sync(0xffffffffu, top >= 0x7e800000u)) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
          if (e >= 120) w[i] = (w[i] & 0x80808080u) | __vminu4(w[i] & 0x7f7f7f7fu, 0x77777777u);
          if (!fine) w[i] = 0;
        }
      }
      const int row = __shfl_sync(0xffffffffu, p.row, t & 31);
      if (t < p.n && row >= 0) {
        uint8_t* dst = codes + (int64_t)row * D + sub * VEC;
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(dst) = w[0];
      }
      const uint32_t byte = fine ? (uint32_t)(e + 127) : 255u;
      if (add && t < p.n && row >= 0) {
        const float f = e8m0_value(byte);
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
          float z[4];
          decode4(w[i], z);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[4 * i + q] = fmaf(z[q], f, acc[4 * i + q]);
        }
      }
      // lane t takes token t's byte from the lanes that hold its row
      const uint32_t b = __shfl_sync(0xffffffffu, byte, lane % RPS * LPR);
      if (lane / RPS == s0 / RPS + u) mine = b;
    }
  }
  if (lane < p.n && p.row >= 0) scales[p.row] = (uint8_t)mine;
  if (add) {
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], off);
    float* dst = sums + ((int64_t)(p.t0 / 32) * dm.Hkv + p.g) * D + sub * VEC;
    if (sel == 0 && MOBA_CHECK(p.t0 / 32 < (dm.T + 31) / 32, status)) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        *reinterpret_cast<float4*>(dst + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    }
  }
}

// Which block a slot stands for. Request r's completed blocks have slots from
// cu_new[r] / B + r on (n / B + 1 of them at most). A request that the write
// skipped has none; one whose rows are not all among the call's is reported here
// too, since the write sees none of a request behind them. Called by whole warps.
struct Slot {
  int r, blk;       // blk: -1 for none
  int begin, row0;  // position and packed row of the request's first new row
};
__device__ __forceinline__ Slot find_slot(const Dims& dm, const Cache& c,
                                          const int32_t* __restrict__ cu_new, int slot,
                                          int* status) {
  const int B = dm.B;
  Slot s{0, -1, 0, 0};
  int r = 0;  // the largest with cu_new[r] / B + r <= slot, 32 requests a round
  for (int n = dm.batch + 1; n > 1;) {
    const int lane = threadIdx.x & 31, step = (n + 31) / 32, at = r + lane * step;
    const uint32_t le =
        __ballot_sync(0xffffffffu, lane * step < n && cu_new[at] / B + at <= slot);
    const int k = le ? 31 - __clz(le) : 0;
    n = min(step, n - k * step);
    r += k * step;
  }
  if (r < dm.batch) {
    const int n = cu_new[r + 1] - cu_new[r], len = c.lens[r];
    if (n > 0 && (cu_new[r] < 0 || cu_new[r + 1] > dm.T)) {
      set_status(status, kStInvalidArg);
    } else if (n > 0 && len >= n && len <= max_positions(dm, c)) {
      s.begin = len - n;
      s.row0 = cu_new[r];
      s.blk = s.begin / B + slot - (s.row0 / B + r);
      if (s.blk >= len / B || s.blk >= dm.nb) s.blk = -1;
    }
  }
  s.r = r;
  return s;
}

// Mean of each block that the new rows complete, over the rows as the cache
// holds them. One cluster per (slot, kv head), its CTAs taking equal parts of the block. Where the write
// left sums of 32 packed rows, those inside a part are added up (1/8 of the
// codes' bytes); the other rows are read: LPR lanes of 16 bytes a row, fp32 sums
// of every G-th row, then the lane groups' sums and the CTAs' sums in order.
// 11 us for 64 blocks of 4096 and 8 heads.
//
// Both kernels of the means begin beside the write, which still stores codes,
// scales and sums then: they read these by ordinary loads, after the wait.
constexpr int kMeanPages = 2048 / 16 + 1;  // pages looked up at a time

template <int D>
__global__ void __launch_bounds__(kMeanThreads, 4)
cache_means_kernel(Dims dm, Cache c, const int32_t* __restrict__ cu_new,
                   const float* sums, float* __restrict__ kbar, int cs, int* status) {
  constexpr int LPR = D / 16, G = kMeanThreads / LPR, U = 8;
  constexpr int LPS = D / 4, GS = kMeanThreads / LPS;  // lanes and streams of sums
  __shared__ __align__(16) float sum[G + GS][D + 4];
  __shared__ float part[kMaxCluster][D];
  __shared__ int page_row[kMeanPages];
  const int g = blockIdx.y, B = dm.B, rank = blockIdx.x % cs;
  const Slot at = find_slot(dm, c, cu_new, blockIdx.x / cs, status);
  const int r = at.r, blk = at.blk, begin = at.begin, row0 = at.row0;
  tc::grid_wait();  // the rows
  if (blk < 0) return;  // the whole cluster
  const int per = (B + cs - 1) / cs, first = blk * B + min(rank * per, B);
  const int last = blk * B + min(rank * per + per, B);
  const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR, mask = (1 << c.page_log2) - 1;
  // groups of 32 packed rows that lie inside [first, last): [g0, g1)
  int g0 = 0, g1 = 0, lo = last, hi = last;  // rows outside them: [first, lo), [hi, last)
  if (sums && last > begin) {
    g0 = (row0 + max(first, begin) - begin + 31) / 32;
    g1 = (row0 + last - begin) / 32;
    if (!MOBA_CHECK(g0 >= 0 && g1 <= (dm.T + 31) / 32, status)) g0 = g1 = 0;
    if (g1 > g0) {
      lo = begin + g0 * 32 - row0;
      hi = begin + g1 * 32 - row0;
    }
  }
  float acc[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) acc[x] = 0.f;
  auto add_rows = [&](int from, int to) {
    for (int c0 = from; c0 < to; c0 += 2048) {
      const int c1 = min(c0 + 2048, to), p0 = c0 >> c.page_log2;
      __syncthreads();
      for (int i = threadIdx.x; i <= ((c1 - 1) >> c.page_log2) - p0; i += kMeanThreads) {
        if (!MOBA_CHECK(i < kMeanPages && p0 + i < c.max_pages, status)) break;
        const int64_t row =
            cache_page_row(c, dm.Hkv, c.table[(int64_t)r * c.max_pages + p0 + i], g);
        page_row[i] = (int)row;
        if (row < 0) set_status(status, kStBadIndices);
      }
      __syncthreads();
      for (int j0 = c0 + grp; j0 < c1; j0 += G * U) {
        uint4 w[U];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = j0 + u * G;
          const int pr = j < c1 ? page_row[(j >> c.page_log2) - p0] : -1;
          w[u] = make_uint4(0, 0, 0, 0);
          s[u] = 0.f;
          if (pr >= 0 && MOBA_CHECK(cache_holds(c, dm.Hkv, pr + (j & mask)), status)) {
            const int64_t row = pr + (j & mask);
            w[u] = *reinterpret_cast<const uint4*>(c.k + row * D + sub * 16);
            s[u] = e8m0_value(c.ks[row]);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[16];
          decode16(w[u], x);
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[e] = fmaf(x[e], s[u], acc[e]);
        }
      }
    }
  };
  add_rows(first, lo);
  add_rows(hi, last);
#pragma unroll
  for (int x = 0; x < 16; ++x) sum[grp][sub * 16 + x] = acc[x];
  {
    const int ss = threadIdx.x % LPS, sg = threadIdx.x / LPS;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = g0 + sg; i < g1; i += GS) {
      const float4 v =
          reinterpret_cast<const float4*>(sums + ((int64_t)i * dm.Hkv + g) * D)[ss];
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
    *reinterpret_cast<float4*>(&sum[G + sg][ss * 4]) = t;
  }
  tc::cluster_sync();
  for (int x = threadIdx.x; x < D; x += kMeanThreads) {
    float t = 0.f;
    for (int i = 0; i < G + GS; ++i) t += sum[i][x];
    tc::store_first(&part[rank][x], t);
  }
  tc::cluster_sync();
  if (rank != 0 || !MOBA_CHECK(r < dm.batch && blk < dm.nb, status)) return;
  for (int x = threadIdx.x; x < D; x += kMeanThreads) {
    float t = 0.f;
    for (int i = 0; i < cs; ++i) t += part[i][x];
    kbar[(((int64_t)r * dm.nb + blk) * dm.Hkv + g) * D + x] = t / (float)B;
  }
}

// The same for blocks of up to kSmallBlock rows, one warp per (slot, kv head):
// their work is too little for a CTA's start and its two barriers. Write and
// means of 262144 rows of 8 heads in blocks of 64: 487 us with a CTA, 308 with a
// warp; 8192 rows after 1000 old ones in each of 4 requests: 91, 49. A warp is the
// slower one where a few requests each end one block of old rows: 8 requests of
// 200 rows, blocks of 128: 11 us with a CTA, 13 with a warp.
constexpr int kSmallBlock = 256;
constexpr int kSmallWarps = 4;

template <int D>
__global__ void __launch_bounds__(kSmallWarps * 32)
cache_small_means_kernel(Dims dm, Cache c, const int32_t* __restrict__ cu_new,
                         const float* sums, float* __restrict__ kbar, int* status) {
  constexpr int LPR = D / 16, G = 32 / LPR, U = 4;  // lanes of a row of codes, rows a load
  constexpr int LPS = D / 4, GS = 32 / LPS;         // the same for sums
  const int lane = threadIdx.x & 31, B = dm.B;
  const int64_t w = (int64_t)blockIdx.x * kSmallWarps + (threadIdx.x >> 5);
  const int64_t slot = w / dm.Hkv;
  const int g = (int)(w % dm.Hkv);
  Slot at{0, -1, 0, 0};
  if (slot < (int64_t)dm.T / B + dm.batch) at = find_slot(dm, c, cu_new, (int)slot, status);
  const int blk = at.blk, first = blk * B, last = first + B;
  // the block's pages, at most 17: lane x looks page x up
  int pages = -1;
  const int p0 = first >> c.page_log2;
  if (blk >= 0 && lane <= ((last - 1) >> c.page_log2) - p0 &&
      MOBA_CHECK(p0 + lane < c.max_pages, status)) {
    const int64_t row =
        cache_page_row(c, dm.Hkv, c.table[(int64_t)at.r * c.max_pages + p0 + lane], g);
    pages = (int)row;
    if (row < 0) set_status(status, kStBadIndices);
  }
  tc::grid_wait();  // the rows
  if (blk < 0) return;
  // groups of 32 packed rows inside the block: [g0, g1); rows outside them are read
  int g0 = 0, g1 = 0, lo = last, hi = last;
  if (sums && last > at.begin) {
    g0 = (at.row0 + max(first, at.begin) - at.begin + 31) / 32;
    g1 = (at.row0 + last - at.begin) / 32;
    if (!MOBA_CHECK(g0 >= 0 && g1 <= (dm.T + 31) / 32, status)) g0 = g1 = 0;
    if (g1 > g0) {
      lo = at.begin + g0 * 32 - at.row0;
      hi = at.begin + g1 * 32 - at.row0;
    }
  }
  float t[4] = {0.f, 0.f, 0.f, 0.f};  // dims ss * 4 .. + 3
  const int ss = lane % LPS, sg = lane / LPS;
#pragma unroll 4
  for (int i = g0 + sg; i < g1; i += GS) {
    const float4 v =
        reinterpret_cast<const float4*>(sums + ((int64_t)i * dm.Hkv + g) * D)[ss];
    t[0] += v.x;
    t[1] += v.y;
    t[2] += v.z;
    t[3] += v.w;
  }
  if (GS == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] += __shfl_xor_sync(0xffffffffu, t[e], 16);
  }
  const int rest = lo - first + last - hi;  // row x of them: first + x, or hi + x - (lo - first)
  if (rest > 0) {
    const int sub = lane % LPR, grp = lane / LPR, mask = (1 << c.page_log2) - 1;
    float acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    for (int x0 = 0; x0 < rest; x0 += G * U) {
      uint4 q[U];
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = x0 + u * G + grp;
        const int j = x < lo - first ? first + x : hi + x - (lo - first);
        const int pr = __shfl_sync(0xffffffffu, pages, ((j >> c.page_log2) - p0) & 31);
        q[u] = make_uint4(0, 0, 0, 0);
        s[u] = 0.f;
        if (x < rest && pr >= 0 && MOBA_CHECK(cache_holds(c, dm.Hkv, pr + (j & mask)), status)) {
          const int64_t row = pr + (j & mask);
          q[u] = *reinterpret_cast<const uint4*>(c.k + row * D + sub * 16);
          s[u] = e8m0_value(c.ks[row]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float y[16];
        decode16(q[u], y);
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = fmaf(y[e], s[u], acc[e]);
      }
    }
    // lane l has the dims 16 (l % LPR) .. of every G-th row, and wants 4 (l % LPS) ..
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int off = LPR; off < 32; off *= 2) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], off);
      const float v = __shfl_sync(0xffffffffu, acc[e], ss / 4);
      if (ss % 4 == e / 4) t[e % 4] += v;
    }
  }
  if (sg == 0 && MOBA_CHECK(at.r < dm.batch && blk < dm.nb, status)) {
    float* o = kbar + (((int64_t)at.r * dm.nb + blk) * dm.Hkv + g) * D + ss * 4;
    const float n = (float)B;
    *reinterpret_cast<float4*>(o) = make_float4(t[0] / n, t[1] / n, t[2] / n, t[3] / n);
  }
}

// 16 values, rounded once, in stores of 32 bytes (whole sectors).
__device__ __forceinline__ void store16(float* dst, const float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(x[8 * h + i]);
    tc::st_global_v8_b32(dst + 8 * h, w);
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  tc::st_global_v8_b32(dst, w);
}

// Read back: 16 codes a lane, widened, scaled and rounded once to the output
// type (exact for bf16 and fp32 but below their normal range). Bound by HBM: 262144
// rows of 8 heads to bf16, 250 us, 6.45 TB/s (the plain copy runs at 6.55). Four
// rows a lane in flight leave registers for more warps than eight do: 282 -> 252;
// stores of whole sectors: 252 -> 250.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(Dims dm, Cache c, const int32_t* __restrict__ cu_rows, T* __restrict__ k,
                  T* __restrict__ v, int tpw, int* status) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, U = 4;
  const int lane = threadIdx.x & 31, sub = lane % LPR, sel = lane / LPR;
  T* __restrict__ dst = blockIdx.y ? v : k;
  const uint8_t* __restrict__ codes = blockIdx.y ? c.v : c.k;
  const uint8_t* __restrict__ scales = blockIdx.y ? c.vs : c.ks;
  WarpPlace p = warp_place(dm, tpw);
  if (p.n <= 0) return;
  p.row = token_row(dm, c, cu_rows, p, status);
  const float scale = p.row >= 0 ? e8m0_value(scales[p.row]) : 0.f;
  T* base = dst + ((int64_t)p.t0 * dm.Hkv + p.g) * D + sub * 16;
  for (int s0 = 0; s0 < p.n; s0 += RPS * U) {
    uint4 w[U];
    int row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = s0 + u * RPS + sel;
      row[u] = __shfl_sync(0xffffffffu, p.row, t & 31);
      if (t >= p.n) row[u] = -1;
      if (row[u] >= 0)
        w[u] = *reinterpret_cast<const uint4*>(codes + (int64_t)row[u] * D + sub * 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = s0 + u * RPS + sel;
      const float f = __shfl_sync(0xffffffffu, scale, t & 31);
      if (row[u] < 0) continue;
      float x[16];
      decode16(w[u], x);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= f;
      store16(base + (int64_t)t * dm.Hkv * D, x);
    }
  }
}

// Tokens a warp takes: 32, or 8 where that leaves SMs with fewer than 16 warps
// (64 tokens of 8 heads: 9.4 -> 6.8 us).
int tokens_per_warp(const Dims& dm) {
  return (int64_t)dm.T * dm.Hkv < (int64_t)32 * 16 * kSMs ? 8 : 32;
}
dim3 warp_grid(const Dims& dm, int tpw) {
  const int64_t warps = (int64_t)((dm.T + tpw - 1) / tpw) * dm.Hkv;
  return dim3((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)), 2);
}

template <typename T, int D>
cudaError_t run_write(const Dims& dm, const Cache& c, const void* k, const void* v,
                      const int32_t* cu_new, float* sums, int* status, cudaStream_t st) {
  const int tpw = tokens_per_warp(dm);
  cache_write_kernel<T, D><<<warp_grid(dm, tpw), kThreads, 0, st>>>(
      dm, c, static_cast<const T*>(k), static_cast<const T*>(v), cu_new, tpw, sums, status);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t run_read(const Dims& dm, const Cache& c, const int32_t* cu_rows, void* k, void* v,
                     int* status, cudaStream_t st) {
  const int tpw = tokens_per_warp(dm);
  cache_read_kernel<T, D><<<warp_grid(dm, tpw), kThreads, 0, st>>>(
      dm, c, cu_rows, static_cast<T*>(k), static_cast<T*>(v), tpw, status);
  return cudaGetLastError();
}

}  // namespace

size_t cache_sums_floats(const Dims& dm) {
  return tokens_per_warp(dm) == 32 ? (size_t)((dm.T + 31) / 32) * dm.Hkv * dm.d : 0;
}

cudaError_t launch_cache_write(const Dims& dm, const Cache& c, const void* k, const void* v,
                               const int32_t* cu_new, float* sums, int* status, cudaStream_t st) {
  if (dm.dtype == kBF16)
    return dm.d == 128 ? run_write<__nv_bfloat16, 128>(dm, c, k, v, cu_new, sums, status, st)
                       : run_write<__nv_bfloat16, 64>(dm, c, k, v, cu_new, sums, status, st);
  return dm.d == 128 ? run_write<float, 128>(dm, c, k, v, cu_new, sums, status, st)
                     : run_write<float, 64>(dm, c, k, v, cu_new, sums, status, st);
}

cudaError_t launch_cache_means(const Dims& dm, const Cache& c, const int32_t* cu_new,
                               const float* sums, float* kbar, int* status, cudaStream_t st) {
  const int64_t slots = (int64_t)dm.T / dm.B + dm.batch;
  // Four CTAs a block where blocks are long and few, which pays where their rows have
  // to be read (one CTA, four): 4096 rows, too few for sums, in blocks of 1024 28.4 ->
  // 17.8 us, one row each for 4 requests that ends a block of 4096 41.3 -> 15.1. Where
  // sums are there it hardly matters: 16384 rows in blocks of 1024 25.2, 25.8; 65536 in
  // blocks of 4096 80.9, 79.4; 32768 in blocks of 1024, the last below the limit, 44.8,
  // 48.9. Above it: 65536 rows in blocks of 1024 79.6, 90.3, but one row each for 64
  // requests that ends a block of 4096 44.4, 21.0.
  const int cs = dm.B >= 1024 && slots * dm.Hkv < 2 * kSMs ? 4 : 1;
  if (slots * cs > INT32_MAX) return cudaErrorInvalidValue;
  if (dm.B <= kSmallBlock) {
    const int64_t x = (slots * dm.Hkv + kSmallWarps - 1) / kSmallWarps;
    if (x > INT32_MAX) return cudaErrorInvalidValue;
    const auto kernel = dm.d == 128 ? cache_small_means_kernel<128> : cache_small_means_kernel<64>;
    return tc::launch_beside(kernel, dim3((unsigned)x), kSmallWarps * 32, 0, st, 1, dm, c, cu_new, sums,
                             kbar, status);
  }
  const dim3 grid((unsigned)(slots * cs), (unsigned)dm.Hkv);
  const auto kernel = dm.d == 128 ? cache_means_kernel<128> : cache_means_kernel<64>;
  return tc::launch_beside(kernel, grid, kMeanThreads, 0, st, cs, dm, c, cu_new, sums, kbar, cs, status);
}

cudaError_t launch_cache_read(const Dims& dm, const Cache& c, const int32_t* cu_rows, void* k,
                              void* v, int* status, cudaStream_t st) {
  if (dm.dtype == kBF16)
    return dm.d == 128 ? run_read<__nv_bfloat16, 128>(dm, c, cu_rows, k, v, status, st)
                       : run_read<__nv_bfloat16, 64>(dm, c, cu_rows, k, v, status, st);
  return dm.d == 128 ? run_read<float, 128>(dm, c, cu_rows, k, v, status, st)
                     : run_read<float, 64>(dm, c, cu_rows, k, v, status, st);
}

}  // namespace moba
