// Tensor-core gradient of dense causal attention, bf16 inputs (formulas and
// the choice of two passes: dense_bwd.cu). 128 x 128 tiles of (keys, queries),
// tcgen05 products with fp32 accumulators in TMEM, operands by TMA.
//
//   kv pass  one CTA per (128 keys, kv head): per item (q head of the group,
//            128 queries at or after the keys)
//              S^T = K Q^T, dP^T = V dO^T        (K, V stay in shared memory)
//              P^T = exp2(S^T * c - lse2), dS^T = P^T (dP^T - D)
//              dV += P^T dO, dK += dS^T Q         (A operands from TMEM)
//   q pass   one CTA per (128 queries, q head): per 128 keys up to the diagonal
//              S = Q K^T, dP = dO V^T, dS as above, dQ += dS K
//
// P^T and dS^T come out of the products with the lanes (keys, or queries in
// the q pass) that the next product's A operand needs, so they go from
// registers straight back to TMEM as bf16 and never through shared memory.
// Shared-memory reads of the products bound the kv pass: 64 KB for each of S
// and dP (two operands), 32 KB for each of dV and dK (one), 64 KB of TMA
// writes, at 128 B/clock 2048 clocks an item, exactly the 2048 clocks of its
// four products.
//
// Roles (20 warps): warp 0 loads tiles by TMA; one lane of warp 1 issues
// the products; warp 2 brings the row statistics (kv pass). Rows of a last,
// partial tile that lie behind the sequence are cleared in shared memory (by
// warp 2, or warp 0 in the q pass): they are summed over, and zeros of P or
// dS would not silence an infinity or NaN in them. Warps 4 to 19 do the
// element-wise work, four threads a TMEM lane with 32 columns each.
// The products of one thread run in issue order, which is what lets S of the
// next item overwrite P of this one as soon as dV has been issued.
//
// 4 x 8192 tokens, 16 heads, d = 128: 3.1 ms a call while the clock holds (890
// TFLOP/s counting five products, 1240 counting the seven that run), 3.65 ms in
// a row under the power cap. Of the steps, only the issue of the products
// mattered much (see mma_ss_on): 4.0 -> 3.65; 8 or 16 element-wise warps, a
// part of the exponentials on the FMA pipes and two teams of warps on
// alternate items did not.
//
// Every wait is bounded (tc::mbar_wait); on expiry the CTA records kStTimeout,
// drains the copies and products it issued, frees its TMEM and exits.
#include "tc_ptx.cuh"

namespace moba {
namespace {

using namespace tc;

constexpr int TT = 128;  // keys and queries per tile
constexpr int kWarpsE = 16;                   // element-wise warps, four threads a TMEM lane
constexpr int kThreads = 128 + kWarpsE * 32;
constexpr int CW = TT * 4 / kWarpsE;          // columns of a tile per element-wise thread
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kHalf = 128 * 128;  // bytes of one 64-column half of a tile
constexpr uint32_t kTmemCols = 512;
constexpr int NA = 3;  // ring of the tiles used first and last in an item (Q; K in the q pass)
constexpr int NB = 2;  // ring of the others (dO; V)

template <int D>
struct Cfg {
  static constexpr int NH = D / 64;
  static constexpr uint32_t kTile = NH * kHalf;
  static constexpr uint32_t kSmem = (2 + NA + NB) * kTile;
  static constexpr uint32_t kIdescNN = idesc_bf16(TT, TT, false, false);
  static constexpr uint32_t kIdescTN = idesc_bf16(TT, D, false, true);  // A in TMEM, B N-major
};

struct Args {
  Dims dm;
  const float* stat;
  const int32_t* cu;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int* status;
};

struct Maps {
  const CUtensorMap *q, *k, *v, *o;
};

// Static shared memory, padded so that the dynamic part starts on a
// 1024-byte boundary (the swizzle's period).
struct alignas(1024) Shared {
  float lse2[2][TT], D[2][TT];
  uint64_t fixed_full;           // the resident pair of tiles
  uint64_t a_full[NA], a_empty[NA], b_full[NB], b_empty[NB];
  uint64_t clear_full[2];        // a partial tile's rows are cleared
  uint64_t stat_full[2], stat_empty[2];
  uint64_t s_full[2], p_ready, dp_full, ds_ready, acc_full, drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Shared) % 1024 == 0, "static shared memory");

// One 128-row tile of one head, from token z.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                          int head, int z) {
#pragma unroll
  for (int x = 0; x < Cfg<D>::NH; ++x) tma_load_3d(dst + x * kHalf, map, bar, x * 64, head, z);
}

// D[tmem] = A B^T over d: two tiles in shared memory, both K-major.
template <int D>
__device__ __forceinline__ void mma_nn(uint32_t on, uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
    mma_ss_on(on, d, desc_sw128(a + off, 16, 1024), desc_sw128(b + off, 16, 1024),
              Cfg<D>::kIdescNN, kk > 0 ? 1u : 0u);
  }
}

// D[tmem] += A B over the tile's 128 rows: A as bf16 pairs in TMEM, every CW
// rows' pairs at the columns their fp32 values had (each element-wise thread
// writes where it read), B a tile in shared memory, N-major.
template <int D>
__device__ __forceinline__ void mma_tn(uint32_t on, uint32_t d, uint32_t a, uint32_t b,
                                       bool add) {
#pragma unroll
  for (int kk = 0; kk < TT / 16; ++kk)
    mma_ts_on(on, d, a + kk * 16 / CW * CW + kk * 16 % CW / 2,
              desc_sw128(b + kk * 16 * 128, kHalf, 1024), Cfg<D>::kIdescTN,
              (add || kk > 0) ? 1u : 0u);
}

// Zeros rows n .. 127 of a tile (a warp's lanes together).
template <int D>
__device__ __forceinline__ void clear_rows(uint32_t tile, int n) {
  const int lane = threadIdx.x & 31;
  for (int e = n * 8 + lane; e < TT * 8; e += 32)
#pragma unroll
    for (int x = 0; x < Cfg<D>::NH; ++x)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + x * kHalf + e * 16),
                   "r"(0)
                   : "memory");
}

// One warp's arrival, after every lane's work.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void finish(Shared& sh) {
  fence_before_sync();
  __syncthreads();
  if ((threadIdx.x >> 5) == 1) {
    fence_after_sync();
    tmem_dealloc(sh.tmem_base, kTmemCols);
  }
}

// Barriers and TMEM. A CTA has the SM's tensor memory to itself and takes all
// of it, so its columns start at 0, which the kernels use as a constant.
__device__ __forceinline__ bool init_shared(Shared& sh, int* status) {
  if (threadIdx.x == 0) {
    mbar_init(&sh.fixed_full, 1);
    for (int i = 0; i < NA; ++i) {
      mbar_init(&sh.a_full[i], 1);
      mbar_init(&sh.a_empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&sh.b_full[i], 1);
      mbar_init(&sh.b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.clear_full[i], 1);
      mbar_init(&sh.stat_full[i], 1);
      mbar_init(&sh.stat_empty[i], kWarpsE);
      mbar_init(&sh.s_full[i], 1);
    }
    mbar_init(&sh.p_ready, kWarpsE);
    mbar_init(&sh.dp_full, 1);
    mbar_init(&sh.ds_ready, kWarpsE);
    mbar_init(&sh.acc_full, 1);
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    mbar_fence_init();
  }
  if ((threadIdx.x >> 5) == 1) {
    tmem_alloc(&sh.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (sh.tmem_base == 0) return true;
  if (threadIdx.x == 0) set_status(status, kStCheck);
  finish(sh);
  return false;
}

// 32 columns of an accumulator, times f, rounded to bf16, to 32 elements of a row.
__device__ __forceinline__ void store_cols(__nv_bfloat16* dst, uint32_t taddr, float f, bool on) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_wait_ld();
  if (!on) return;
#pragma unroll
  for (int x = 0; x < 32; x += 16) {
    uint32_t w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      w[u] = pack_bf16x2(__uint_as_float(r[x + 2 * u]) * f, __uint_as_float(r[x + 2 * u + 1]) * f);
    st_global_v8_b32(dst + x, w);
  }
}

// ---- sums over a cluster
// With few tiles the items of one tile are dealt to the cs CTAs of a cluster
// (item x to CTA x % cs); each leaves its accumulators in its shared memory, as
// fp32 rows whose 16-byte pieces are permuted by the row, and sums and writes
// 1/cs of the rows of all of them, in the order of the ranks.
template <int D>
__device__ __forceinline__ uint32_t sum_at(uint32_t mat, int row, int piece) {
  return mat + (uint32_t)row * D * 4 + (((uint32_t)(piece ^ row) & (D / 4 - 1)) << 4);
}
// 32 columns from c of an accumulator row (zeros: a CTA without items).
template <int D>
__device__ __forceinline__ void leave_cols(uint32_t mat, int row, int c, uint32_t taddr, bool some) {
  uint32_t r[32];
  tmem_ld32(taddr, r);
  tmem_wait_ld();
#pragma unroll
  for (int x = 0; x < 32; x += 4)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sum_at<D>(mat, row, (c + x) / 4)),
                 "r"(some ? r[x] : 0u), "r"(some ? r[x + 1] : 0u), "r"(some ? r[x + 2] : 0u),
                 "r"(some ? r[x + 3] : 0u)
                 : "memory");
}
// Sums rows of this CTA's share of a matrix, times f, to rows of `out` (row
// stride in elements), n of them.
template <int D>
__device__ __forceinline__ void sum_rows(uint32_t mat, int rank, int cs, float f,
                                         __nv_bfloat16* out, int64_t stride, int n) {
  const int rows = TT / cs;
  for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
    const int row = rank * rows + e / (D / 4), piece = e % (D / 4);
    if (row >= n) continue;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < cs; ++k) {
      const float4 v = load_rank(sum_at<D>(mat, row, piece), k);
      t.x += v.x;
      t.y += v.y;
      t.z += v.z;
      t.w += v.w;
    }
    *reinterpret_cast<uint2*>(out + row * stride + piece * 4) =
        make_uint2(pack_bf16x2(t.x * f, t.y * f), pack_bf16x2(t.z * f, t.w * f));
  }
}

template <int D>
__device__ __forceinline__ void kv_pass(Shared& sh, const uint32_t sb, const int cta, const int rank,
                                        const int cs, const Maps& m, const Args& a) {
  constexpr uint32_t kTile = Cfg<D>::kTile;
  const Dims& dm = a.dm;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // heads outermost: the CTAs that run together read the same Q and dO, and
  // within a head the tiles with the most queries come first
  const TilePlace at = find_tile<TT, false>(dm, a.cu, dm.Hkv, cta);
  if (at.slots == 0) return;
  const int64_t start = at.start;
  const int len = at.len, kt = at.rest % at.slots, g = at.rest / at.slots;
  if (!MOBA_CHECK(start + len <= dm.T, a.status)) return;
  const int k0 = kt * TT;
  if (k0 >= len) return;
  const uint32_t sK = sb, sV = sb + kTile, sQ = sb + 2 * kTile, sO = sQ + NA * kTile;
  const int grp = dm.Hq / dm.Hkv, per = (len - k0 + TT - 1) / TT;
  const int n_items = (grp * per - rank + cs - 1) / cs;  // of this CTA; 0 is possible
  // item it: q head h, query tile kt + i; the next item's by advance()
  const int h_first = g * grp + rank / per, i_first = rank % per;
  auto advance = [&](int& h, int& i) {
    for (i += cs; i >= per; i -= per) ++h;
  };
  const int last_rows = len - (k0 + (per - 1) * TT);  // queries of each head's last tile
  if (!init_shared(sh, a.status)) {
    if (cs > 1) cluster_sync(), cluster_sync();
    return;
  }
  constexpr uint32_t tS = 0, tP = 128, tV = 256, tK = 256 + D;  // TMEM columns
  volatile int* abort = &sh.abort;
  int* status = a.status;

  if (warp == 0) {
    if (lane == 0) {
      mbar_expect_tx(&sh.fixed_full, 2 * kTile);
      load_tile<D>(sK, m.k, &sh.fixed_full, g, (int)start + k0);
      load_tile<D>(sV, m.v, &sh.fixed_full, g, (int)start + k0);
      int na = 0, nb = 0;
      bool ok = true;
      for (int it = 0, h = h_first, i = i_first; it < n_items; ++it, advance(h, i)) {
        const int z = (int)start + k0 + i * TT;
        if (it >= NA && !(ok = mbar_wait(&sh.a_empty[it % NA], (it / NA - 1) & 1, abort, status)))
          break;
        mbar_expect_tx(&sh.a_full[it % NA], kTile);
        load_tile<D>(sQ + it % NA * kTile, m.q, &sh.a_full[it % NA], h, z);
        ++na;
        if (it >= NB && !(ok = mbar_wait(&sh.b_empty[it % NB], (it / NB - 1) & 1, abort, status)))
          break;
        mbar_expect_tx(&sh.b_full[it % NB], kTile);
        load_tile<D>(sO + it % NB * kTile, m.o, &sh.b_full[it % NB], h, z);
        ++nb;
      }
      if (!ok || *abort) {  // let the copies already issued land before the CTA exits
        mbar_drain(&sh.fixed_full, 0);
        for (int x = na > NA ? na - NA : 0; x < na; ++x) mbar_drain(&sh.a_full[x % NA], x / NA & 1);
        for (int x = nb > NB ? nb - NB : 0; x < nb; ++x) mbar_drain(&sh.b_full[x % NB], x / NB & 1);
      }
    }
  } else if (warp == 1) {
    const uint32_t on = elect_one();
    int cleared = 0, hn = h_first, in = i_first;  // of the next item to land
    // a wait of the whole warp; false in every lane if one gave up
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status)) != 0;
    };
    bool ok = wait(&sh.fixed_full, 0);
    // Q and dO of an item are in shared memory, and cleared where partial
    auto landed = [&](int it) {
      bool w = wait(&sh.a_full[it % NA], it / NA & 1);
      if (w && last_rows < TT && in == per - 1) {
        w = wait(&sh.clear_full[cleared & 1], cleared / 2 & 1);
        ++cleared;
      }
      advance(hn, in);
      return w;
    };
    if (ok && n_items > 0) ok = landed(0);
    if (ok && n_items > 0) {
      mma_nn<D>(on, tS, sK, sQ);
      commit_on(on, &sh.s_full[0]);
      ok = wait(&sh.b_full[0], 0);
    }
    if (ok && n_items > 0) {
      mma_nn<D>(on, tP, sV, sO);
      commit_on(on, &sh.dp_full);
    }
    for (int it = 0; ok && it < n_items; ++it) {
      const uint32_t q = sQ + it % NA * kTile, o = sO + it % NB * kTile;
      if (!(ok = wait(&sh.p_ready, it & 1))) break;
      fence_after_sync();
      mma_tn<D>(on, tV, tS, o, it > 0);
      commit_on(on, &sh.b_empty[it % NB]);
      if (it + 1 < n_items) {
        if (!(ok = landed(it + 1))) break;
        mma_nn<D>(on, tS, sK, sQ + (it + 1) % NA * kTile);
        commit_on(on, &sh.s_full[0]);
      }
      if (!(ok = wait(&sh.ds_ready, it & 1))) break;
      fence_after_sync();
      mma_tn<D>(on, tK, tP, q, it > 0);
      commit_on(on, &sh.a_empty[it % NA]);
      if (it + 1 < n_items) {
        if (!(ok = wait(&sh.b_full[(it + 1) % NB], (it + 1) / NB & 1))) break;
        mma_nn<D>(on, tP, sV, sO + (it + 1) % NB * kTile);
        commit_on(on, &sh.dp_full);
      }
    }
    if (ok) {
      commit_on(on, &sh.acc_full);
    } else {  // wait until every product issued has finished
      commit_on(on, &sh.drain);
      mbar_drain(&sh.drain, 0);
    }
  } else if (warp == 2) {
    // clear_full has two slots: dO of item it + 2 lands only after dV of item
    // it, so this warp is at most one partial tile ahead of the issuer
    const float* st = a.stat + start + k0;
    int cleared = 0;
    grid_wait();  // the statistics are the launch before this one
    for (int it = 0, h = h_first, i = i_first; it < n_items; ++it, advance(h, i)) {
      const int s = it & 1, n = i == per - 1 ? last_rows : TT;
      bool ok = it < 2 || mbar_wait(&sh.stat_empty[s], (it / 2 - 1) & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      // ordinary loads: the launch that writes these may run beside this one, so
      // they are not read-only for it
      const float* src = st + (int64_t)h * dm.T + i * TT;
      float l2[TT / 32], dd[TT / 32];
#pragma unroll
      for (int x = 0; x < TT / 32; ++x) {
        const int r = lane + 32 * x;
        l2[x] = r < n ? src[r] : 0.f;
        dd[x] = r < n ? src[(int64_t)dm.Hq * dm.T + r] : 0.f;
      }
#pragma unroll
      for (int x = 0; x < TT / 32; ++x) {
        sh.lse2[s][lane + 32 * x] = l2[x];
        sh.D[s][lane + 32 * x] = dd[x];
      }
      warp_arrive(&sh.stat_full[s]);
      if (n < TT) {
        ok = mbar_wait(&sh.a_full[it % NA], it / NA & 1, abort, status) &&
             mbar_wait(&sh.b_full[it % NB], it / NB & 1, abort, status);
        if (!__all_sync(0xffffffffu, ok)) break;
        clear_rows<D>(sQ + it % NA * kTile, n);
        clear_rows<D>(sO + it % NB * kTile, n);
        fence_proxy_async_smem();
        warp_arrive(&sh.clear_full[cleared++ & 1]);
      }
    }
  } else if (warp >= 4) {
    const int c0 = ((warp - 4) >> 2) * CW, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16, at = lanes + c0;
    const float sl2 = rsqrtf((float)D) * kLog2e;
    bool ok = true;
    for (int it = 0, h = h_first, i = i_first; it < n_items; ++it, advance(h, i)) {
      const int s = it & 1;
      // keys after a query and queries behind the sequence: only in each
      // head's first and last tile. Column x is visible in [lo, hi).
      const bool masked = i == 0 || (i == per - 1 && last_rows < TT);
      const int lo = (i == 0 ? r : 0) - c0;
      const int hi = (i == per - 1 ? last_rows : TT) - c0;
      ok = mbar_wait(&sh.stat_full[s], it / 2 & 1, abort, status) &&
           mbar_wait(&sh.s_full[0], it & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after_sync();
      float p[CW];
      {
        uint32_t v[CW];
        tmem_ld32(tS + at, v);
        tmem_wait_ld();
        const float4* l4 = reinterpret_cast<const float4*>(&sh.lse2[s][c0]);
#pragma unroll
        for (int x = 0; x < CW; x += 4) {
          const float4 l = l4[x / 4];
          p[x] = ex2(fmaf(__uint_as_float(v[x]), sl2, -l.x));
          p[x + 1] = ex2(fmaf(__uint_as_float(v[x + 1]), sl2, -l.y));
          p[x + 2] = ex2(fmaf(__uint_as_float(v[x + 2]), sl2, -l.z));
          p[x + 3] = ex2(fmaf(__uint_as_float(v[x + 3]), sl2, -l.w));
        }
      }
      if (masked) {
#pragma unroll
        for (int x = 0; x < CW; ++x) p[x] = x >= lo && x < hi ? p[x] : 0.f;
      }
      {
        // P in bf16 (half a step of 2^-8: the weights of dV's sum); the
        // products of dS keep the unrounded P
        uint32_t w[CW / 2];
#pragma unroll
        for (int x = 0; x < CW / 2; ++x) w[x] = pack_bf16x2(p[2 * x], p[2 * x + 1]);
        tmem_st16(tS + at, w);
      }
      tmem_wait_st();
      fence_before_sync();
      warp_arrive(&sh.p_ready);
      ok = mbar_wait(&sh.dp_full, it & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after_sync();
      uint32_t v[CW], w[CW / 2];
      tmem_ld32(tP + at, v);
      tmem_wait_ld();
      const float4* d4 = reinterpret_cast<const float4*>(&sh.D[s][c0]);
#pragma unroll
      for (int x = 0; x < CW; x += 4) {
        const float4 dd = d4[x / 4];
        float ds[4] = {p[x] * (__uint_as_float(v[x]) - dd.x),
                       p[x + 1] * (__uint_as_float(v[x + 1]) - dd.y),
                       p[x + 2] * (__uint_as_float(v[x + 2]) - dd.z),
                       p[x + 3] * (__uint_as_float(v[x + 3]) - dd.w)};
        if (masked) {
#pragma unroll
          for (int u = 0; u < 4; ++u) ds[u] = x + u >= lo && x + u < hi ? ds[u] : 0.f;
        }
        w[x / 2] = pack_bf16x2(ds[0], ds[1]);
        w[x / 2 + 1] = pack_bf16x2(ds[2], ds[3]);
      }
      tmem_st16(tP + at, w);
      tmem_wait_st();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.stat_empty[s]);
        mbar_arrive(&sh.ds_ready);
      }
    }
    // dK (the first half of the warps) and dV of key r, 32 columns at a time
    if (ok) ok = mbar_wait(&sh.acc_full, 0, abort, status);
    if (__all_sync(0xffffffffu, ok) && cs > 1) {
      fence_after_sync();
#pragma unroll 1
      for (int c = c0; c < 2 * D; c += TT)
        leave_cols<D>(sb + c / D * TT * D * 4, r, c % D, tK + lanes - (c < D ? 0 : 2 * D) + c,
                      n_items > 0);
    } else if (__all_sync(0xffffffffu, ok)) {
      fence_after_sync();
      const bool on = k0 + r < len;
      const int64_t row = ((start + k0 + (on ? r : 0)) * dm.Hkv + g) * D;
#pragma unroll 1
      for (int c = c0; c < 2 * D; c += TT) {
        const bool is_v = c >= D;
        store_cols((is_v ? a.dv - D : a.dk) + row + c, (is_v ? tV - D : tK) + lanes + c,
                   is_v ? 1.f : rsqrtf((float)D), on);
      }
    }
  }
  if (cs > 1) {
    __syncwarp();
    cluster_sync();
    const int64_t row = ((start + k0) * dm.Hkv + g) * D, stride = (int64_t)dm.Hkv * D;
    sum_rows<D>(sb, rank, cs, rsqrtf((float)D), a.dk + row, stride, min(TT, len - k0));
    sum_rows<D>(sb + TT * D * 4, rank, cs, 1.f, a.dv + row, stride, min(TT, len - k0));
    cluster_sync();
  }
  finish(sh);
}

template <int D>
__device__ __forceinline__ void q_pass(Shared& sh, const uint32_t sb, const int cta, const int rank,
                                       const int cs, const Maps& m, const Args& a) {
  constexpr uint32_t kTile = Cfg<D>::kTile;
  const Dims& dm = a.dm;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // the heads of a group outermost but one: CTAs that run together read the
  // same K and V; the longest tiles of a head come first
  const TilePlace at = find_tile<TT, false>(dm, a.cu, dm.Hq, cta);
  if (at.slots == 0) return;
  const int64_t start = at.start;
  const int len = at.len, h = at.rest / at.slots;
  if (!MOBA_CHECK(start + len <= dm.T, a.status)) return;
  const int qt = (len + TT - 1) / TT - 1 - at.rest % at.slots, q0 = qt * TT;
  if (qt < 0) return;
  const int g = h / (dm.Hq / dm.Hkv);
  const int n_items = (qt + 1 - rank + cs - 1) / cs;  // key tiles rank, rank + cs, ..; 0 is possible
  const bool diagonal = rank == qt % cs;              // the last of them is the diagonal
  const int last_keys = min(len - q0, TT);  // keys of the diagonal tile
  const uint32_t sQ = sb, sO = sb + kTile, sK = sb + 2 * kTile, sV = sK + NA * kTile;
  if (!init_shared(sh, a.status)) {
    if (cs > 1) cluster_sync(), cluster_sync();
    return;
  }
  constexpr uint32_t tP = 256, tQ = 384;  // TMEM columns; S at 0 and 128
  volatile int* abort = &sh.abort;
  int* status = a.status;

  if (warp == 0) {
    bool ok = true;
    if (lane == 0) {
      mbar_expect_tx(&sh.fixed_full, 2 * kTile);
      load_tile<D>(sQ, m.q, &sh.fixed_full, h, (int)start + q0);
      load_tile<D>(sO, m.o, &sh.fixed_full, h, (int)start + q0);
      int na = 0, nb = 0;
      for (int j = 0; j < n_items; ++j) {
        const int z = (int)start + (rank + j * cs) * TT;
        if (j >= NA && !(ok = mbar_wait(&sh.a_empty[j % NA], (j / NA - 1) & 1, abort, status)))
          break;
        mbar_expect_tx(&sh.a_full[j % NA], kTile);
        load_tile<D>(sK + j % NA * kTile, m.k, &sh.a_full[j % NA], g, z);
        ++na;
        if (j >= NB && !(ok = mbar_wait(&sh.b_empty[j % NB], (j / NB - 1) & 1, abort, status)))
          break;
        mbar_expect_tx(&sh.b_full[j % NB], kTile);
        load_tile<D>(sV + j % NB * kTile, m.v, &sh.b_full[j % NB], g, z);
        ++nb;
      }
      if (!ok || *abort) {
        mbar_drain(&sh.fixed_full, 0);
        for (int x = na > NA ? na - NA : 0; x < na; ++x) mbar_drain(&sh.a_full[x % NA], x / NA & 1);
        for (int x = nb > NB ? nb - NB : 0; x < nb; ++x) mbar_drain(&sh.b_full[x % NB], x / NB & 1);
      }
    }
    if (diagonal && last_keys < TT) {  // the diagonal tile's keys behind the sequence
      const int j = n_items - 1;
      if (lane == 0 && ok) ok = mbar_wait(&sh.a_full[j % NA], j / NA & 1, abort, status);
      if (__all_sync(0xffffffffu, ok)) {
        clear_rows<D>(sK + j % NA * kTile, last_keys);
        fence_proxy_async_smem();
        warp_arrive(&sh.clear_full[0]);
      }
    }
  } else if (warp == 1) {
    const uint32_t on = elect_one();
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status)) != 0;
    };
    bool ok = wait(&sh.fixed_full, 0);
    auto s_product = [&](int j) {
      if (!wait(&sh.a_full[j % NA], j / NA & 1)) return false;
      if (diagonal && j == n_items - 1 && last_keys < TT && !wait(&sh.clear_full[0], 0)) return false;
      mma_nn<D>(on, (j & 1) * 128, sQ, sK + j % NA * kTile);
      commit_on(on, &sh.s_full[j & 1]);
      return true;
    };
    auto dp_product = [&](int j) {
      if (!wait(&sh.b_full[j % NB], j / NB & 1)) return false;
      mma_nn<D>(on, tP, sO, sV + j % NB * kTile);
      commit_on(on, &sh.dp_full);
      commit_on(on, &sh.b_empty[j % NB]);
      return true;
    };
    ok = ok && (n_items == 0 || (s_product(0) && dp_product(0)));
    for (int j = 0; ok && j < n_items; ++j) {
      // S of the next keys goes into the other buffer, whose dS the last
      // dQ product has been issued for
      if (j + 1 < n_items && !(ok = s_product(j + 1))) break;
      if (!(ok = wait(&sh.ds_ready, j & 1))) break;
      fence_after_sync();
      if (j + 1 < n_items && !(ok = dp_product(j + 1))) break;
      mma_tn<D>(on, tQ, (j & 1) * 128, sK + j % NA * kTile, j > 0);
      commit_on(on, &sh.a_empty[j % NA]);
    }
    if (ok) {
      commit_on(on, &sh.acc_full);
    } else {
      commit_on(on, &sh.drain);
      mbar_drain(&sh.drain, 0);
    }
  } else if (warp >= 4) {
    const int c0 = ((warp - 4) >> 2) * CW, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16, at = lanes + c0;
    const float sl2 = rsqrtf((float)D) * kLog2e;
    const bool on = q0 + r < len;
    float l2 = 0.f, dd = 0.f;
    grid_wait();  // the statistics are the launch before this one
    if (on) {
      const float* st = a.stat + (int64_t)h * dm.T + start + q0 + r;
      l2 = st[0];  // ordinary loads, as in the key pass
      dd = st[(int64_t)dm.Hq * dm.T];
    }
    bool ok = true;
    for (int j = 0; j < n_items; ++j) {
      const uint32_t tS = (j & 1) * 128 + at;
      ok = mbar_wait(&sh.s_full[j & 1], j / 2 & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after_sync();
      float p[CW];
      {
        uint32_t v[CW];
        tmem_ld32(tS, v);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < CW; ++x) p[x] = ex2(fmaf(__uint_as_float(v[x]), sl2, -l2));
      }
      ok = mbar_wait(&sh.dp_full, j & 1, abort, status);
      if (!__all_sync(0xffffffffu, ok)) break;
      fence_after_sync();
      const bool masked = diagonal && j == n_items - 1;  // the diagonal: keys up to the query
      const int hi = min(r + 1, last_keys) - c0;
      uint32_t v[CW], w[CW / 2];
      tmem_ld32(tP + at, v);
      tmem_wait_ld();
#pragma unroll
      for (int x = 0; x < CW; x += 2) {
        float ds[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          ds[u] = p[x + u] * (__uint_as_float(v[x + u]) - dd);
          if (masked) ds[u] = x + u < hi ? ds[u] : 0.f;
        }
        w[x / 2] = pack_bf16x2(ds[0], ds[1]);
      }
      tmem_st16(tS, w);
      tmem_wait_st();
      fence_before_sync();
      warp_arrive(&sh.ds_ready);
    }
    if (ok) ok = mbar_wait(&sh.acc_full, 0, abort, status);
    if (__all_sync(0xffffffffu, ok) && cs > 1) {
      fence_after_sync();
      if (c0 < D) leave_cols<D>(sb, r, c0, tQ + lanes + c0, n_items > 0);
    } else if (__all_sync(0xffffffffu, ok)) {
      fence_after_sync();
      const int64_t row = ((start + q0 + (on ? r : 0)) * dm.Hq + h) * D;
      if (c0 < D) store_cols(a.dq + row + c0, tQ + lanes + c0, rsqrtf((float)D), on);
    }
  }
  if (cs > 1) {
    __syncwarp();
    cluster_sync();
    sum_rows<D>(sb, rank, cs, rsqrtf((float)D), a.dq + ((start + q0) * dm.Hq + h) * D,
                (int64_t)dm.Hq * D, min(TT, len - q0));
    cluster_sync();
  }
  finish(sh);
}

// Both passes in one launch: the first n_kv clusters own keys, the others
// queries, so that the second pass fills the SMs that the first one's end
// leaves idle.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
dense_bwd_tc(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
             const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmo,
             const Args a, const int n_kv, const int cs) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Shared sh;
  const uint32_t sb = smem_u32(smem);
  if (sb & 1023u) {  // the layout above did not hold: nothing can be right
    if (threadIdx.x == 0) set_status(a.status, kStCheck);
    return;
  }
  if (threadIdx.x < 4)
    prefetch_map(threadIdx.x == 0 ? &tmq : threadIdx.x == 1 ? &tmk : threadIdx.x == 2 ? &tmv : &tmo);
  const Maps m{&tmq, &tmk, &tmv, &tmo};
  const int cta = (int)blockIdx.x / cs, rank = (int)blockIdx.x % cs;
  if (cta < n_kv)
    kv_pass<D>(sh, sb, cta, rank, cs, m, a);
  else
    q_pass<D>(sh, sb, cta - n_kv, rank, cs, m, a);
  grid_wait();  // a CTA without work too: what follows this launch follows the last one
}

template <int D>
cudaError_t run(const Args& a, const void* q, const void* k, const void* v, const void* dout,
                cudaStream_t st) {
  const Dims& dm = a.dm;
  CUtensorMap mq, mk, mv, mo;
  cudaError_t e;
  if ((e = make_head_map(&mq, q, dm.T, dm.Hq, TT, D))) return e;
  if ((e = make_head_map(&mk, k, dm.T, dm.Hkv, TT, D))) return e;
  if ((e = make_head_map(&mv, v, dm.T, dm.Hkv, TT, D))) return e;
  if ((e = make_head_map(&mo, dout, dm.T, dm.Hq, TT, D))) return e;
  constexpr int smem = (int)Cfg<D>::kSmem;
  static std::atomic<bool> ready[kMaxDevices];
  if ((e = allow_smem(dense_bwd_tc<D>, smem, ready))) return e;
  // 300 + 212 tokens, 4 on 2 heads: 21 us with one CTA a tile, 15 with four; 692 +
  // 88 + 6 + 10 + 40, 24 on 8 heads: 44 with one, 58 with two; 8191, 4 on 1 head: 436
  // with one, 222 with two, 274 with four. Clusters of eight leave SMs without one.
  const int64_t nt = tile_slots<TT>(dm), clusters = nt * (dm.Hq + dm.Hkv);
  const int cs = cluster_for<TT>(dm, sm_count(), 4, 5);  // a start costs as much as five items
  if (clusters * cs > INT32_MAX) return cudaErrorInvalidValue;
  return launch_beside(dense_bwd_tc<D>, dim3((unsigned)(clusters * cs)), kThreads, smem,
                       st, cs, mq, mk, mv, mo, a, (int)(nt * dm.Hkv), cs);
}

}  // namespace

cudaError_t launch_dense_bwd_tc(const Dims& dm, const void* q, const void* k, const void* v,
                                const void* dout, const float* stat, const int32_t* cu, void* dq,
                                void* dk, void* dv, int* status, cudaStream_t st) {
  if (dm.batch == 0 || dm.max_seqlen == 0) return cudaSuccess;
  const Args a{dm, stat, cu, static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk),
               static_cast<__nv_bfloat16*>(dv), status};
  return dm.d == 128 ? run<128>(a, q, k, v, dout, st) : run<64>(a, q, k, v, dout, st);
}

}  // namespace moba
