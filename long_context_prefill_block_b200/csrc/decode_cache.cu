// Decode attention over the paged 8-bit cache (cache.cu): the decode step of
// PaperTrace "2.1.3 MoBA", section 5.4, for the blocks that the gate chose
// (launch_cache_gate). A query at position p reads the chosen earlier blocks
// whole and its own block up to p, as one softmax (eq. 4-8); a key's scale
// multiplies its logit and a value's scale its weight, so codes are widened
// once and never rescaled.
//
// Split over the chosen keys: one CTA per (query, q head, chosen block, chunk
// of at most 512 keys); the last split of a row to finish merges the row's
// partials (no CTA waits for another).
#include <cuda_fp8.h>

#include <cmath>

#include "common.cuh"

namespace moba {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSplit = 512;  // keys per split at most
constexpr int kMaxPages = kSplit / 16 + 1;
constexpr float kLog2e = 1.4426950408889634f;

__host__ __device__ inline int split_keys(const Dims& dm) { return dm.B < kSplit ? dm.B : kSplit; }
__host__ __device__ inline int splits_per_block(const Dims& dm) {
  return (dm.B + split_keys(dm) - 1) / split_keys(dm);
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

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
cache_attn_kernel(Dims dm, Cache c, const T* __restrict__ q, const int32_t* __restrict__ cu_q,
                  const int32_t* __restrict__ idx, float* __restrict__ part_o,
                  float* __restrict__ part_lse, int* __restrict__ arrivals, T* __restrict__ out,
                  float* __restrict__ lse_out, int* status) {
  constexpr int LPK = D / 16, GPW = 32 / LPK, G = GPW * kWarps, U = 4;
  __shared__ float wm[kWarps], wl[kWarps];
  __shared__ __align__(16) float wo[kWarps][D];
  __shared__ int64_t page_row[kMaxPages];
  __shared__ int last;
  const int spb = splits_per_block(dm), S = dm.topk * spb;
  const int s = (int)(blockIdx.x % S), qi = (int)(blockIdx.x / S), h = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t row = (int64_t)qi * dm.Hq + h, prow = row * S + s;
  const int64_t held = (int64_t)c.max_pages << c.page_log2;
  const int max_len = held < dm.max_seqlen ? (int)held : dm.max_seqlen;
  int r, len, p;
  if (!tail_position(cu_q, c.lens, dm.batch, max_len, qi, r, p, len, status)) return;
  const int g = h / (dm.Hq / dm.Hkv), own = p / dm.B;
  int lo = 0, hi = 0;
  const int e = idx[row * dm.topk + s / spb];
  if (e >= 0 && e <= own) {
    lo = e * dm.B + (s % spb) * split_keys(dm);
    hi = min(min(lo + split_keys(dm), (e + 1) * dm.B), p + 1);
  }
  if (lo >= hi) {
    if (tid == 0) part_lse[prow] = -INFINITY;
  } else {
    const int p0 = lo >> c.page_log2, np = ((hi - 1) >> c.page_log2) - p0 + 1;
    for (int i = tid; i < np; i += kThreads) {
      page_row[i] = cache_page_row(c, dm.Hkv, c.table[(int64_t)r * c.max_pages + p0 + i], g);
      if (page_row[i] < 0) set_status(status, kStBadIndices);
    }
    const int grp_id = warp * GPW + lane / LPK, sub = lane % LPK;
    const float sl2 = kLog2e * rsqrtf((float)D);
    float qv[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) qv[x] = to_f32(q[row * D + sub * 16 + x]) * sl2;
    float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) o[x] = 0.f;
    const int mask = (1 << c.page_log2) - 1;
    __syncthreads();
    for (int base = lo; base < hi; base += U * G) {
      uint4 kr[U], vr[U];
      float ks[U], vs[U];
      bool on[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = base + grp_id + u * G;
        const int jj = j < hi ? j : lo;
        const int64_t pr = page_row[(jj >> c.page_log2) - p0];
        on[u] = j < hi && pr >= 0;
        const int64_t at = pr < 0 ? 0 : pr + (jj & mask);
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
        d[u] = on[u] ? acc * ks[u] : -INFINITY;
        mn = fmaxf(mn, d[u]);
      }
      if (mn == -INFINITY) {
        // nothing to weigh in this step, but a NaN logit must not be lost
        float bad = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) bad += on[u] && d[u] != d[u] ? d[u] : 0.f;
        l += bad;
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
        for (int i = 0; i < 16; ++i) o[i] = fmaf(wv, x[i], o[i]);
      }
      m = mn;
    }
    // merge the lane groups of the warp, then the warps
#pragma unroll
    for (int off = LPK; off < 32; off <<= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m, off);
      const float lo2 = __shfl_xor_sync(0xffffffffu, l, off);
      const float mn = fmaxf(m, mo);
      const float a = m == -INFINITY ? 1.f : exp2f(m - mn);
      const float b = mo == -INFINITY ? 1.f : exp2f(mo - mn);
      l = l * a + lo2 * b;
#pragma unroll
      for (int x = 0; x < 16; ++x) o[x] = o[x] * a + __shfl_xor_sync(0xffffffffu, o[x], off) * b;
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
    // a split all of whose keys weigh nothing (bad pages) leaves no partial;
    // one with a NaN logit leaves NaN
    const bool none = M == -INFINITY && L == 0.f;
    for (int x = tid; x < D && !none; x += kThreads) {
      float acc = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        acc = fmaf(wo[w][x], wm[w] == -INFINITY ? 1.f : exp2f(wm[w] - M), acc);
      part_o[prow * D + x] = acc / L;
    }
    if (tid == 0)
      part_lse[prow] = none ? -INFINITY : L != L ? L : (M + log2f(L)) * 0.6931471805599453f;
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(&arrivals[row], 1) == S - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // the row's partials by eq. (7)-(8): w_s = exp(lse_s - max), in split order
  const float* ls = part_lse + row * S;
  float M = -INFINITY;
  for (int s2 = tid; s2 < S; s2 += kThreads) M = fmaxf(M, __ldcg(ls + s2));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  if (lane == 0) wm[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float Lw = 0.f;
  const bool cols = lane * 4 < D;
#pragma unroll 4
  for (int s2 = warp; s2 < S; s2 += kWarps) {
    const float lv = __ldcg(ls + s2);
    const bool on = lv != -INFINITY;  // NaN counts: it has to show
    const float w = on ? expf(lv - M) : 0.f;
    Lw += w;
    if (cols) {
      const float4 ov = __ldcg(reinterpret_cast<const float4*>(part_o + (row * S + s2) * D) + lane);
      acc.x += on ? w * ov.x : 0.f;
      acc.y += on ? w * ov.y : 0.f;
      acc.z += on ? w * ov.z : 0.f;
      acc.w += on ? w * ov.w : 0.f;
    }
  }
  __syncthreads();
  if (cols) *reinterpret_cast<float4*>(&wo[warp][lane * 4]) = acc;
  if (lane == 0) wl[warp] = Lw;
  __syncthreads();
  for (int x = tid; x < D; x += kThreads) {
    float O = 0.f, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      O += wo[w][x];
      L += wl[w];
    }
    // L == 0: every page of the row was bad; zeros and -inf, not 0 / 0
    out[row * D + x] = from_f32<T>(L == 0.f ? 0.f : O / L);
    if (x == 0 && lse_out) lse_out[row] = L == 0.f ? -INFINITY : M + logf(L);
  }
}

template <typename T, int D>
cudaError_t run(const Dims& dm, const Cache& c, const void* q, const int32_t* cu_q,
                const int32_t* idx, float* part_o, float* part_lse, int* arrivals, void* out,
                float* lse, int* status, cudaStream_t st) {
  const int64_t x = (int64_t)dm.topk * splits_per_block(dm) * dm.T;
  if (x > INT32_MAX) return cudaErrorInvalidValue;
  cache_attn_kernel<T, D><<<dim3((unsigned)x, (unsigned)dm.Hq), kThreads, 0, st>>>(
      dm, c, static_cast<const T*>(q), cu_q, idx, part_o, part_lse, arrivals,
      static_cast<T*>(out), lse, status);
  return cudaGetLastError();
}

}  // namespace

size_t decode_cache_partial_rows(const Dims& dm) {
  return (size_t)dm.T * dm.Hq * dm.topk * splits_per_block(dm);
}

cudaError_t launch_cache_attn(const Dims& dm, const Cache& c, const void* q, const int32_t* cu_q,
                              const int32_t* idx, float* part_o, float* part_lse, int* arrivals,
                              void* out, float* lse, int* status, cudaStream_t st) {
  if (dm.dtype == kBF16)
    return dm.d == 128 ? run<__nv_bfloat16, 128>(dm, c, q, cu_q, idx, part_o, part_lse, arrivals,
                                                 out, lse, status, st)
                       : run<__nv_bfloat16, 64>(dm, c, q, cu_q, idx, part_o, part_lse, arrivals,
                                                out, lse, status, st);
  return dm.d == 128
             ? run<float, 128>(dm, c, q, cu_q, idx, part_o, part_lse, arrivals, out, lse, status, st)
             : run<float, 64>(dm, c, q, cu_q, idx, part_o, part_lse, arrivals, out, lse, status, st);
}

}  // namespace moba
