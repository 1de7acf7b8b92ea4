// Gradient of dense causal attention (PaperTrace "2.1.3 MoBA", section 1
// eq. (1) with a causal mask; the layers of a hybrid stack that keep full
// attention). With logits s_ij = q_i . k_j / sqrt(d) over j <= i of one
// sequence and the forward's lse_i, out_i:
//   P_ij = exp(s_ij - lse_i)          (recomputed, never stored)
//   D_i  = dO_i . out_i,  dS_ij = P_ij (dO_i . v_j - D_i)
//   dq_i = sum_j dS_ij k_j / sqrt(d),  dk_j = sum_i dS_ij q_i / sqrt(d),
//   dv_j = sum_i P_ij dO_i            (i over every q head of the kv head)
//
// Two passes over the tiles, one that owns keys (dk, dv) and one that owns
// queries (dq). Each result row is summed by one CTA, or by one cluster in the
// order of its ranks, so equal calls give equal bits and nothing is added
// atomically; the price is seven products per tile instead of five (S and
// dO V^T are formed twice).
//
// This file: the row statistics both passes read, and the passes for fp32
// inputs in fp32 FMA. bf16 inputs take dense_bwd_tc.cu.
#include "tc_ptx.cuh"

namespace moba {
namespace {

constexpr int kThreads = 256;
constexpr int BR = 64;  // queries per tile
constexpr int BK = 64;  // keys per tile
constexpr int LP = BK + 4;

constexpr float kLog2e = 1.4426950408889634f;

// stat[0][h][t] = lse * log2(e), stat[1][h][t] = D = dO . out, laid out head
// by head so that a tile of one head's queries reads contiguous floats. Also
// writes the gradients of rows that no sequence owns (a padded batch) or that
// stand in a sequence that is skipped (longer than max_seqlen, or with rows that
// are not all among the call's): zeros.
// One CTA: 32 tokens of one head; 16 bytes of a row per lane.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
dense_bwd_stat_kernel(Dims dm, const T* __restrict__ out, const T* __restrict__ dout,
                      const float* __restrict__ lse, const int32_t* __restrict__ cu,
                      float* __restrict__ stat, T* __restrict__ dq, T* __restrict__ dk,
                      T* __restrict__ dv, int* status) {
  constexpr int VEC = Vec16<T>::N, LPR = D / VEC, RPS = kThreads / LPR;  // rows per step
  __shared__ float ds[32];
  __shared__ bool owned[32];
  // the tensor-core passes may begin: they wait for this launch where they
  // read the statistics
  tc::grid_let_next();
  const int h = blockIdx.y, t0 = blockIdx.x * 32;
  if (h == 0 && t0 == 0) {  // every sequence, those that get no tile too
    for (int b = threadIdx.x; b < dm.batch; b += kThreads)
      if (!has_place(dm, cu[b], (uint32_t)cu[b + 1] - cu[b])) set_status(status, kStInvalidArg);
  }
  const int sub = threadIdx.x % LPR, rr = threadIdx.x / LPR;
  for (int r = rr; r < 32; r += RPS) {
    const int t = t0 + r;
    float acc = 0.f;
    if (t < dm.T) {
      const int64_t at = ((int64_t)t * dm.Hq + h) * D + sub * VEC;
      float a[VEC], b[VEC];
      Vec16<T>::load(out + at, a);
      Vec16<T>::load(dout + at, b);
#pragma unroll
      for (int x = 0; x < VEC; ++x) acc = fmaf(a[x], b[x], acc);
    }
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (sub == 0) ds[r] = acc;
  }
  __syncthreads();
  const int t = t0 + threadIdx.x;
  if (threadIdx.x < 32) {
    bool mine = false;
    if (t < dm.T) {
      stat[(int64_t)h * dm.T + t] = lse[(int64_t)t * dm.Hq + h] * kLog2e;
      stat[((int64_t)dm.Hq + h) * dm.T + t] = ds[threadIdx.x];
      const int b = find_request(cu, dm.batch, t);
      mine = b < dm.batch && t >= cu[b] && has_place(dm, cu[b], (uint32_t)cu[b + 1] - cu[b]);
    }
    owned[threadIdx.x] = mine;
  }
  if (__syncthreads_and(threadIdx.x >= 32 || owned[threadIdx.x & 31])) return;
  const T zero = from_f32<T>(0.f);
  for (int e = threadIdx.x; e < 32 * D; e += kThreads) {
    const int64_t row = t0 + e / D;
    if (row >= dm.T || owned[e / D]) continue;
    dq[(row * dm.Hq + h) * D + e % D] = zero;
    if (h < dm.Hkv) {
      dk[(row * dm.Hkv + h) * D + e % D] = zero;
      dv[(row * dm.Hkv + h) * D + e % D] = zero;
    }
  }
}

struct Args {
  Dims dm;
  const float* q;
  const float* k;
  const float* v;
  const float* dout;
  const float* stat;
  const int32_t* cu;
  float* dq;
  float* dk;
  float* dv;
  int* status;
  int cs;  // CTAs a cluster
};

// 64 rows of one head (row stride in elements) into shared memory, rows at
// or past n as zeros.
template <int D>
__device__ __forceinline__ void load_tile(float (*dst)[D + 4], const float* src, int64_t stride,
                                          int n) {
  for (int e = threadIdx.x; e < 64 * (D / 4); e += kThreads) {
    const int r = e / (D / 4), c = e % (D / 4);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < n) x = __ldg(reinterpret_cast<const float4*>(src + r * stride) + c);
    *reinterpret_cast<float4*>(&dst[r][c * 4]) = x;
  }
}

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

template <int D>
struct Smem {
  float K[BK][D + 4], V[BK][D + 4], Q[BR][D + 4], O[BR][D + 4];
  float P[BR][LP], S[BK][LP];  // P [query][key]; dS [query][key], or [key][query] for dq
  float lse2[BR], D_[BR];
};

// P and dS of the 64 x 64 tile of queries q0.. and keys k0.. (positions in a
// sequence of length len) into shared memory. Thread (ty, tx): queries
// ty * 4 .. + 3, keys tx + 16 u: rows are read 16 bytes at a time along d and
// the padded stride puts 8 consecutive key rows into distinct bank groups.
template <int D, bool kTransposed>
__device__ __forceinline__ void tile_ps(Smem<D>& sm, int q0, int k0, int len) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float s[4][4], dp[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) s[a][b] = dp[a][b] = 0.f;
#pragma unroll 2
  for (int x = 0; x < D; x += 4) {
    float4 q4[4], o4[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      q4[a] = *reinterpret_cast<const float4*>(&sm.Q[ty * 4 + a][x]);
      o4[a] = *reinterpret_cast<const float4*>(&sm.O[ty * 4 + a][x]);
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float4 k4 = *reinterpret_cast<const float4*>(&sm.K[tx + 16 * b][x]);
      const float4 v4 = *reinterpret_cast<const float4*>(&sm.V[tx + 16 * b][x]);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        s[a][b] = fmaf(q4[a].x, k4.x, s[a][b]);
        s[a][b] = fmaf(q4[a].y, k4.y, s[a][b]);
        s[a][b] = fmaf(q4[a].z, k4.z, s[a][b]);
        s[a][b] = fmaf(q4[a].w, k4.w, s[a][b]);
        dp[a][b] = fmaf(o4[a].x, v4.x, dp[a][b]);
        dp[a][b] = fmaf(o4[a].y, v4.y, dp[a][b]);
        dp[a][b] = fmaf(o4[a].z, v4.z, dp[a][b]);
        dp[a][b] = fmaf(o4[a].w, v4.w, dp[a][b]);
      }
    }
  }
  const float sl2 = rsqrtf((float)D) * kLog2e;
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int qi = ty * 4 + a;
    const float l2 = sm.lse2[qi], dd = sm.D_[qi];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int kj = tx + 16 * b;
      // masked places get zeros by selection: whatever their rows hold
      const bool vis = q0 + qi < len && k0 + kj <= q0 + qi;
      const float p = vis ? exp2f(fmaf(s[a][b], sl2, -l2)) : 0.f;
      const float ds = vis ? p * (dp[a][b] - dd) : 0.f;
      if (kTransposed) {
        sm.S[kj][qi] = ds;
      } else {
        sm.P[qi][kj] = p;
        sm.S[qi][kj] = ds;
      }
    }
  }
}

// Rows of the query tile: q, dO and the statistics.
template <int D>
__device__ __forceinline__ void load_queries(const Args& a, Smem<D>& sm, int64_t start, int q0,
                                             int len, int h) {
  const int n = min(BR, len - q0);
  const int64_t row = (start + q0) * a.dm.Hq + h;
  load_tile<D>(sm.Q, a.q + row * D, (int64_t)a.dm.Hq * D, n);
  load_tile<D>(sm.O, a.dout + row * D, (int64_t)a.dm.Hq * D, n);
  if (threadIdx.x < BR) {
    const int r = threadIdx.x;
    const float* st = a.stat + (int64_t)h * a.dm.T + start + q0 + r;
    sm.lse2[r] = r < n ? st[0] : 0.f;
    sm.D_[r] = r < n ? st[(int64_t)a.dm.Hq * a.dm.T] : 0.f;
  }
}

// Writes accumulators acc[i][4 w + u] (row ty * 4 + i, column tx * 4 + 64 w + u)
// times f to rows of `out` (n of them, row stride in elements). In a cluster
// they are left in `tile` first, and each CTA sums and writes 1/cs of the rows.
template <int D>
__device__ __forceinline__ void store_rows(const float (&acc)[4][D / 16], float (*tile)[D + 4],
                                           int rank, int cs, float f, float* out, int64_t stride,
                                           int n) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  if (cs == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ty * 4 + i >= n) continue;
#pragma unroll
      for (int w = 0; w < D / 64; ++w)
        store4(out + (ty * 4 + i) * stride + tx * 4 + 64 * w, acc[i][4 * w] * f,
               acc[i][4 * w + 1] * f, acc[i][4 * w + 2] * f, acc[i][4 * w + 3] * f);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int w = 0; w < D / 64; ++w)
      store4(&tile[ty * 4 + i][tx * 4 + 64 * w], acc[i][4 * w], acc[i][4 * w + 1],
             acc[i][4 * w + 2], acc[i][4 * w + 3]);
  tc::cluster_sync();
  const int rows = 64 / cs;
  for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
    const int row = rank * rows + e / (D / 4), c = e % (D / 4) * 4;
    if (row >= n) continue;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < cs; ++k) {
      const float4 v = tc::load_rank(tc::smem_u32(&tile[row][c]), k);
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
    store4(out + row * stride + c, t.x * f, t.y * f, t.z * f, t.w * f);
  }
  tc::cluster_sync();  // the others' reads of this tile
}

// dk, dv of 64 keys of one kv head: every later query tile of every q head
// of the group. Every item is loaded, waited for and then used, with one CTA (d =
// 128) or two (d = 64) an SM to cover that: 1024 + 777 tokens, 4 heads, d = 64 take
// 139 us, where the seven products of their tiles (3.3 GFLOP) are 45 at a nominal
// 74 TFLOP/s of fp32 FMA. (Two CTAs an SM leave 128 registers a thread, and 92
// bytes of them spill.)
template <int D>
__device__ __forceinline__ void kv_pass(const Args& a, Smem<D>& sm, int x, int rank) {
  const Dims& dm = a.dm;
  const TilePlace at = find_tile<BK, true>(dm, a.cu, dm.Hkv, x);
  if (at.slots == 0) return;
  const int64_t start = at.start;
  const int len = at.len, g = at.rest % dm.Hkv;  // the longest tiles of a sequence first
  if (!MOBA_CHECK(start + len <= dm.T, a.status)) return;
  const int k0 = at.rest / dm.Hkv * BK;
  if (k0 >= len) return;
  const int nk = min(BK, len - k0);
  const int64_t krow = (start + k0) * dm.Hkv + g;
  load_tile<D>(sm.K, a.k + krow * D, (int64_t)dm.Hkv * D, nk);
  load_tile<D>(sm.V, a.v + krow * D, (int64_t)dm.Hkv * D, nk);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // keys ty * 4 .., dims tx * 4 + 64 w
  constexpr int NW = D / 64;
  float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int x = 0; x < 4 * NW; ++x) dk[i][x] = dv[i][x] = 0.f;
  const int grp = dm.Hq / dm.Hkv;
  int item = 0;
  for (int h = g * grp; h < (g + 1) * grp; ++h) {
    for (int q0 = k0; q0 < len; q0 += BR) {
      if (item++ % a.cs != rank) continue;  // dealt to the cluster's CTAs
      __syncthreads();
      load_queries<D>(a, sm, start, q0, len, h);
      __syncthreads();
      tile_ps<D, false>(sm, q0, k0, len);
      __syncthreads();
#pragma unroll 2
      for (int r = 0; r < BR; ++r) {
        const float4 p4 = *reinterpret_cast<const float4*>(&sm.P[r][ty * 4]);
        const float4 s4 = *reinterpret_cast<const float4*>(&sm.S[r][ty * 4]);
        const float p[4] = {p4.x, p4.y, p4.z, p4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float4 o4 = *reinterpret_cast<const float4*>(&sm.O[r][tx * 4 + 64 * w]);
          const float4 q4 = *reinterpret_cast<const float4*>(&sm.Q[r][tx * 4 + 64 * w]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            dv[i][4 * w + 0] = fmaf(p[i], o4.x, dv[i][4 * w + 0]);
            dv[i][4 * w + 1] = fmaf(p[i], o4.y, dv[i][4 * w + 1]);
            dv[i][4 * w + 2] = fmaf(p[i], o4.z, dv[i][4 * w + 2]);
            dv[i][4 * w + 3] = fmaf(p[i], o4.w, dv[i][4 * w + 3]);
            dk[i][4 * w + 0] = fmaf(s[i], q4.x, dk[i][4 * w + 0]);
            dk[i][4 * w + 1] = fmaf(s[i], q4.y, dk[i][4 * w + 1]);
            dk[i][4 * w + 2] = fmaf(s[i], q4.z, dk[i][4 * w + 2]);
            dk[i][4 * w + 3] = fmaf(s[i], q4.w, dk[i][4 * w + 3]);
          }
        }
      }
    }
  }
  __syncthreads();
  const int64_t stride = (int64_t)dm.Hkv * D;
  store_rows<D>(dk, sm.Q, rank, a.cs, rsqrtf((float)D), a.dk + krow * D, stride, nk);
  store_rows<D>(dv, sm.O, rank, a.cs, 1.f, a.dv + krow * D, stride, nk);
}

// dq of 64 queries of one head: every key tile up to the diagonal. Blocks
// are numbered last tile first, the longest work.
template <int D>
__device__ __forceinline__ void q_pass(const Args& a, Smem<D>& sm, int x, int rank) {
  const Dims& dm = a.dm;
  const TilePlace at = find_tile<BR, true>(dm, a.cu, dm.Hq, x);
  if (at.slots == 0) return;
  const int64_t start = at.start;
  const int len = at.len, h = at.rest % dm.Hq, g = h / (dm.Hq / dm.Hkv);
  if (!MOBA_CHECK(start + len <= dm.T, a.status)) return;
  const int q0 = ((len + BR - 1) / BR - 1 - at.rest / dm.Hq) * BR;
  if (q0 < 0) return;
  load_queries<D>(a, sm, start, q0, len, h);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // queries ty * 4 .., dims tx * 4 + 64 w
  constexpr int NW = D / 64;
  float dq[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int x = 0; x < 4 * NW; ++x) dq[i][x] = 0.f;
  for (int k0 = rank * BK; k0 <= q0; k0 += a.cs * BK) {
    const int64_t krow = (start + k0) * dm.Hkv + g;
    __syncthreads();
    load_tile<D>(sm.K, a.k + krow * D, (int64_t)dm.Hkv * D, min(BK, len - k0));
    load_tile<D>(sm.V, a.v + krow * D, (int64_t)dm.Hkv * D, min(BK, len - k0));
    __syncthreads();
    tile_ps<D, true>(sm, q0, k0, len);
    __syncthreads();
#pragma unroll 2
    for (int j = 0; j < BK; ++j) {
      const float4 s4 = *reinterpret_cast<const float4*>(&sm.S[j][ty * 4]);
      const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float4 k4 = *reinterpret_cast<const float4*>(&sm.K[j][tx * 4 + 64 * w]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dq[i][4 * w + 0] = fmaf(s[i], k4.x, dq[i][4 * w + 0]);
          dq[i][4 * w + 1] = fmaf(s[i], k4.y, dq[i][4 * w + 1]);
          dq[i][4 * w + 2] = fmaf(s[i], k4.z, dq[i][4 * w + 2]);
          dq[i][4 * w + 3] = fmaf(s[i], k4.w, dq[i][4 * w + 3]);
        }
      }
    }
  }
  __syncthreads();
  store_rows<D>(dq, sm.K, rank, a.cs, rsqrtf((float)D), a.dq + ((start + q0) * dm.Hq + h) * D,
                (int64_t)dm.Hq * D, min(BR, len - q0));
}

// Both passes in one launch of clusters: the first n_kv own keys, the others
// queries. With few tiles the other side's tiles are dealt to the cs CTAs of a
// cluster, which sum their results in the order of the ranks.
template <int D>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
dense_bwd_kernel(const Args a, const int n_kv) {
  extern __shared__ __align__(16) uint8_t raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
  const int x = (int)blockIdx.x / a.cs, rank = (int)blockIdx.x % a.cs;
  if (x < n_kv)
    kv_pass<D>(a, sm, x, rank);
  else
    q_pass<D>(a, sm, x - n_kv, rank);
}

template <typename T, int D>
cudaError_t run_stat(const Dims& dm, const void* out, const void* dout, const float* lse,
                     const int32_t* cu, float* stat, void* dq, void* dk, void* dv, int* status,
                     cudaStream_t st) {
  dense_bwd_stat_kernel<T, D><<<dim3((unsigned)((dm.T + 31) / 32), (unsigned)dm.Hq), kThreads, 0,
                                st>>>(dm, static_cast<const T*>(out), static_cast<const T*>(dout),
                                      lse, cu, stat, static_cast<T*>(dq), static_cast<T*>(dk),
                                      static_cast<T*>(dv), status);
  return cudaGetLastError();
}

template <int D>
cudaError_t run_simt(Args a, cudaStream_t st) {
  const Dims& dm = a.dm;
  cudaError_t e;
  constexpr int smem = (int)sizeof(Smem<D>);
  static std::atomic<bool> ready[tc::kMaxDevices];
  if ((e = tc::allow_smem(dense_bwd_kernel<D>, smem, ready))) return e;
  static_assert(BK == BR, "one number of slots for both passes");
  const int64_t nt = tile_slots<BK>(dm), clusters = nt * (dm.Hq + dm.Hkv);
  // 109 + 13 + 64 + 1 tokens, 8 on 2 heads, d = 128: 137 us with one CTA a tile, 46
  // with four, 80 with eight; 1024 + 777, 4 heads, d = 64: 222 with one, 148 with two
  // or four. A start costs about as much as an item.
  a.cs = cluster_for<BK>(dm, tc::sm_count() * (D == 64 ? 2 : 1), 8, 1);
  if (clusters * a.cs > INT32_MAX) return cudaErrorInvalidValue;
  return tc::launch_cluster(dense_bwd_kernel<D>, dim3((unsigned)(clusters * a.cs)), kThreads, smem, st,
                            a.cs, a, (int)(nt * dm.Hkv));
}

}  // namespace

cudaError_t launch_dense_bwd_stat(const Dims& dm, const void* out, const void* dout,
                                  const float* lse, const int32_t* cu, float* stat, void* dq,
                                  void* dk, void* dv, int* status, cudaStream_t st) {
  if (dm.dtype == kBF16)
    return dm.d == 128
               ? run_stat<__nv_bfloat16, 128>(dm, out, dout, lse, cu, stat, dq, dk, dv, status, st)
               : run_stat<__nv_bfloat16, 64>(dm, out, dout, lse, cu, stat, dq, dk, dv, status, st);
  return dm.d == 128 ? run_stat<float, 128>(dm, out, dout, lse, cu, stat, dq, dk, dv, status, st)
                     : run_stat<float, 64>(dm, out, dout, lse, cu, stat, dq, dk, dv, status, st);
}

cudaError_t launch_dense_bwd_simt(const Dims& dm, const void* q, const void* k, const void* v,
                                  const void* dout, const float* stat, const int32_t* cu, void* dq,
                                  void* dk, void* dv, int* status, cudaStream_t st) {
  if (dm.batch == 0 || dm.max_seqlen == 0) return cudaSuccess;
  const Args a{dm,
               static_cast<const float*>(q),
               static_cast<const float*>(k),
               static_cast<const float*>(v),
               static_cast<const float*>(dout),
               stat,
               cu,
               static_cast<float*>(dq),
               static_cast<float*>(dk),
               static_cast<float*>(dv),
               status,
               1};
  return dm.d == 128 ? run_simt<128>(a, st) : run_simt<64>(a, st);
}

}  // namespace moba
