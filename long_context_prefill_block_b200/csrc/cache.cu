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

#include "common.cuh"

namespace moba {
namespace {

constexpr int kThreads = 256;

// The largest e4m3 code value for scale 2^e, and 2^-e in two exact factors.
__device__ __forceinline__ int row_exponent(float top) {
  if (top == 0.f) return -127;
  const uint32_t u = __float_as_uint(top);
  int ex = (int)(u >> 23);
  uint32_t man = u & 0x7fffffu;
  if (ex == 0) {  // a number below 2^-126: 448 * 2^-127 holds it
    return -127;
  }
  // top = 1.man * 2^(ex - 127); 448 = 1.75 * 2^8
  const int e = ex - 127 - 8 + (man > 0x600000u ? 1 : 0);
  return e < -127 ? -127 : e;
}

// Values x[0 .. N) of a row as N e4m3 bytes.
template <int N>
__device__ __forceinline__ void encode(const float (&x)[N], int e, uint32_t (&w)[N / 4]) {
  // 2^-e = 2^h * 2^(-e-h): each a normal number for e in [-127, 120]
  const int h = (-e) >> 1;
  const float f0 = __uint_as_float((uint32_t)(h + 127) << 23);
  const float f1 = __uint_as_float((uint32_t)(-e - h + 127) << 23);
  const float lim = e >= 120 ? 240.f : 448.f;
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    float y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) y[u] = fminf(fmaxf(x[i + u] * f0 * f1, -lim), lim);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2], y[3]), __NV_SATFINITE, __NV_E4M3);
    w[i / 4] = lo | hi << 16;
  }
}

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

// Row index in the cache of position pos of request r and kv head g, or -1
// (and a status code) where the page table names no page.
__device__ __forceinline__ int64_t cache_row(const Cache& c, int Hkv, int r, int pos, int g,
                                             int* status) {
  const int page = c.table[(int64_t)r * c.max_pages + (pos >> c.page_log2)];
  const int64_t row = cache_page_row(c, Hkv, page, g);
  if (row < 0) {
    set_status(status, kStBadIndices);
    return -1;
  }
  return row + (pos & ((1 << c.page_log2) - 1));
}

// Positions a request can have: what its pages hold, and what the caller's
// max_seqlen allows.
__device__ __forceinline__ int max_positions(const Dims& dm, const Cache& c) {
  const int64_t held = (int64_t)c.max_pages << c.page_log2;
  return held < dm.max_seqlen ? (int)held : dm.max_seqlen;
}

// Quantise and store. Row i = token * Hkv + head of the packed new rows; a
// row is held by LPR lanes of 16 bytes, which share its maximum by shuffles;
// blockIdx.y: K or V. Bound by HBM: d * sizeof(T) bytes in, d + 1 out.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
cache_write_kernel(Dims dm, Cache c, const T* __restrict__ k, const T* __restrict__ v,
                   const int32_t* __restrict__ cu_new, int* status) {
  constexpr int VEC = Vec16<T>::N, LPR = D / VEC, G = kThreads / LPR, U = 4;
  const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const T* __restrict__ src = blockIdx.y ? v : k;
  uint8_t* __restrict__ codes = blockIdx.y ? c.v : c.k;
  uint8_t* __restrict__ scales = blockIdx.y ? c.vs : c.ks;
  const int64_t rows = (int64_t)dm.T * dm.Hkv, i0 = (int64_t)blockIdx.x * (G * U) + grp;
  const int max_len = max_positions(dm, c);
  float x[U][VEC];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * G;
    if (i < rows) Vec16<T>::load(src + i * D + sub * VEC, x[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * G;
    float top = 0.f;
    bool fine = true;
    if (i < rows) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        top = fmaxf(top, fabsf(x[u][e]));
        fine = fine && fabsf(x[u][e]) <= 3.4028234663852886e38f;
      }
    }
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      fine = __shfl_xor_sync(0xffffffffu, (int)fine, off) && fine;
    }
    if (i >= rows) continue;
    int r, pos, len;
    if (!tail_position(cu_new, c.lens, dm.batch, max_len, (int)(i / dm.Hkv), r, pos, len, status))
      continue;
    const int64_t row = cache_row(c, dm.Hkv, r, pos, (int)(i % dm.Hkv), status);
    if (row < 0) continue;
    uint32_t w[VEC / 4];
    const int e = row_exponent(fine ? top : 0.f);
    if (!fine) {
#pragma unroll
      for (int q = 0; q < VEC; ++q) x[u][q] = 0.f;
    }
    encode<VEC>(x[u], e, w);
    uint8_t* dst = codes + row * D + sub * VEC;
    if constexpr (VEC == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(dst) = w[0];
    if (sub == 0) scales[row] = (uint8_t)(fine ? e + 127 : 255);
  }
}

// Mean of each block that the new rows complete, over the rows as the cache
// holds them. Slot j of the grid: request r's completed blocks have slots
// from cu_new[r] / B + r on (n / B + 1 of them at most). One CTA per (slot,
// kv head): LPR lanes of 16 bytes a row, fp32 sums of every G-th row, then
// the groups' sums in order.
template <int D>
__global__ void __launch_bounds__(kThreads)
cache_means_kernel(Dims dm, Cache c, const int32_t* __restrict__ cu_new,
                   float* __restrict__ kbar, int* status) {
  constexpr int LPR = D / 16, G = kThreads / LPR, U = 4;
  __shared__ float sum[G][D + 4];
  const int g = blockIdx.y, B = dm.B;
  int lo = 0, hi = dm.batch;  // largest r with cu_new[r] / B + r <= slot
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu_new[mid] / B + mid <= (int)blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const int r = lo;
  if (r >= dm.batch) return;
  const int n = cu_new[r + 1] - cu_new[r], len = c.lens[r];
  if (n <= 0 || len < n || len > max_positions(dm, c)) return;
  const int blk = (len - n) / B + (int)blockIdx.x - (cu_new[r] / B + r);
  if (blk < 0 || blk >= len / B || blk >= dm.nb) return;
  const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  float acc[16];
#pragma unroll
  for (int x = 0; x < 16; ++x) acc[x] = 0.f;
  for (int j0 = grp; j0 < B; j0 += G * U) {
    uint4 w[U];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * G;
      w[u] = make_uint4(0, 0, 0, 0);
      s[u] = 0.f;
      if (j < B) {
        const int64_t row = cache_row(c, dm.Hkv, r, blk * B + j, g, status);
        if (row >= 0) {
          w[u] = *reinterpret_cast<const uint4*>(c.k + row * D + sub * 16);
          s[u] = e8m0_value(c.ks[row]);
        }
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
#pragma unroll
  for (int x = 0; x < 16; ++x) sum[grp][sub * 16 + x] = acc[x];
  __syncthreads();
  for (int x = threadIdx.x; x < D; x += kThreads) {
    float t = 0.f;
    for (int i = 0; i < G; ++i) t += sum[i][x];
    kbar[(((int64_t)r * dm.nb + blk) * dm.Hkv + g) * D + x] = t / (float)B;
  }
}

__device__ __forceinline__ void store16(float* dst, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Read back: 16 codes a lane, widened, scaled and rounded once to the output
// type (exact for bf16 and fp32 but below their normal range).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
cache_read_kernel(Dims dm, Cache c, const int32_t* __restrict__ cu_rows, T* __restrict__ k,
                  T* __restrict__ v, int* status) {
  constexpr int LPR = D / 16, G = kThreads / LPR, U = 4;
  const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  T* __restrict__ dst = blockIdx.y ? v : k;
  const uint8_t* __restrict__ codes = blockIdx.y ? c.v : c.k;
  const uint8_t* __restrict__ scales = blockIdx.y ? c.vs : c.ks;
  const int64_t rows = (int64_t)dm.T * dm.Hkv, i0 = (int64_t)blockIdx.x * (G * U) + grp;
  const int max_len = max_positions(dm, c);
  uint4 w[U];
  float s[U];
  bool on[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t i = i0 + u * G;
    int r, pos, len;
    on[u] = false;
    if (i < rows &&
        tail_position(cu_rows, c.lens, dm.batch, max_len, (int)(i / dm.Hkv), r, pos, len, status)) {
      const int64_t row = cache_row(c, dm.Hkv, r, pos, (int)(i % dm.Hkv), status);
      if (row >= 0) {
        on[u] = true;
        w[u] = *reinterpret_cast<const uint4*>(codes + row * D + sub * 16);
        s[u] = e8m0_value(scales[row]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!on[u]) continue;
    float x[16];
    decode16(w[u], x);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= s[u];
    store16(dst + (i0 + u * G) * D + sub * 16, x);
  }
}

template <typename T, int D>
cudaError_t run_write(const Dims& dm, const Cache& c, const void* k, const void* v,
                      const int32_t* cu_new, int* status, cudaStream_t st) {
  constexpr int per = kThreads / (D / Vec16<T>::N) * 4;
  const int64_t rows = (int64_t)dm.T * dm.Hkv;
  cache_write_kernel<T, D><<<dim3((unsigned)((rows + per - 1) / per), 2), kThreads, 0, st>>>(
      dm, c, static_cast<const T*>(k), static_cast<const T*>(v), cu_new, status);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t run_read(const Dims& dm, const Cache& c, const int32_t* cu_rows, void* k, void* v,
                     int* status, cudaStream_t st) {
  constexpr int per = kThreads / (D / 16) * 4;
  const int64_t rows = (int64_t)dm.T * dm.Hkv;
  cache_read_kernel<T, D><<<dim3((unsigned)((rows + per - 1) / per), 2), kThreads, 0, st>>>(
      dm, c, cu_rows, static_cast<T*>(k), static_cast<T*>(v), status);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const Dims& dm, const Cache& c, const void* k, const void* v,
                               const int32_t* cu_new, int* status, cudaStream_t st) {
  if (dm.dtype == kBF16)
    return dm.d == 128 ? run_write<__nv_bfloat16, 128>(dm, c, k, v, cu_new, status, st)
                       : run_write<__nv_bfloat16, 64>(dm, c, k, v, cu_new, status, st);
  return dm.d == 128 ? run_write<float, 128>(dm, c, k, v, cu_new, status, st)
                     : run_write<float, 64>(dm, c, k, v, cu_new, status, st);
}

cudaError_t launch_cache_means(const Dims& dm, const Cache& c, const int32_t* cu_new, float* kbar,
                               int* status, cudaStream_t st) {
  const dim3 grid((unsigned)(dm.T / dm.B + dm.batch), (unsigned)dm.Hkv);
  if (dm.d == 128)
    cache_means_kernel<128><<<grid, kThreads, 0, st>>>(dm, c, cu_new, kbar, status);
  else
    cache_means_kernel<64><<<grid, kThreads, 0, st>>>(dm, c, cu_new, kbar, status);
  return cudaGetLastError();
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
