// The many-adapter forward of a few rows (a decode step), bf16.
//
// Y [M, N] = X W0^T + the rows' own updates, M small: every byte of W0 is read once, which bounds it.  So the
// product is turned around: 128 rows of W0 are the M side of the tcgen05 MMA and the batch's rows its N side
// (16, 32 or 64, zero-filled), and K is shared by the CTAs of a cluster, each with its own stretch of W0, so that
// some 300 CTAs, two an SM, keep their copies in flight.  The partial accumulators meet through distributed
// shared memory, in the order of the ranks.  Measured (rank 16): one row of 4096 x 4096 10.1 us (W0 alone at the rate of
// a long copy: 5.0), 64 rows 18.5, 19 rows of 4096 x 11008 at rank 64 24.1 (15.0): a first read of 67 MB takes 16 us with
// nothing but loads, and a decode step is not long enough to get past that start.  The rank-r part is computed on the
// side:
//   multi_few_down   z_i = x_i A_a^T, one cluster a row, its CTAs sharing K;
//   multi_few        while W0 streams in, eight more warps form s z B_a^T.
// The second kernel starts while the first one runs (programmatic launch): it touches nothing that the first
// one writes before its wait, and what came before the first one is complete when that lets it start.
#include "common.cuh"
#include "multi.h"
#include "vec.cuh"

namespace lg {

namespace {

constexpr int kStretch = 512;     // columns of x that a CTA of multi_few_down takes at a time
constexpr int kRowsW = 128, kBK = 64;
constexpr int kDownCtas = 4;      // of multi_few_down on an SM
constexpr int kUpdate = 256;       // threads of the update; four of their warps read the accumulator
constexpr int kThreads = 64 + kUpdate;   // copies, MMA
constexpr int64_t kInFlight = 16 << 20;   // bytes of W0 and x on their way
constexpr int kAhead = 4;         // pieces of the factor that a thread asks for at a time, twice

struct FewArgs {
  CUtensorMap tmW, tmX;
  int M, N, r, nk, stages;
  const int32_t* ids;
  const bf16 *X, *A, *B, *bias;
  float one;
  const float* each;
  float* sz;                      // [M, r] s z
  bf16 *Y, *Z;
  int64_t K;
  uint32_t* err;
  uint64_t timeout_ns;
};

// sz[i] = s_a x_i A_a^T and Z[i] = x_i A_a^T, zeros for a row without adapter.  A CTA has its rank's share of K, in
// stretches of 512; of each the rows of A_a come by asynchronous copies, 16 at a time, up to four such blocks on
// their way: in flight in shared memory they need few registers and threads, and multi_few's CTAs find room beside
// these.  A warp takes four rows of a block.
constexpr int kBlock = 16 * (2 * kStretch + 16);      // bytes of a block of 16 rows
__global__ void __launch_bounds__(128) multi_few_down(const __grid_constant__ FewArgs a) {
  extern __shared__ __align__(16) uint8_t smem_down[];
  __shared__ float sum[128];
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int i = (int)(blockIdx.x / ranks), lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = a.r;
  const int ad = a.ids[i];
  const int64_t to = (int64_t)i * r;
  if (ad < 0) {                   // the whole cluster
    for (int j = threadIdx.x; rank == 0 && j < r; j += 128) {
      a.sz[to + j] = 0.f;
      if (a.Z) a.Z[to + j] = __float2bfloat16_rn(0.f);
    }
    return;
  }
  const bf16* u = a.A + (int64_t)ad * r * a.K;
  const int64_t all = (a.K + kStretch - 1) / kStretch;
  const int s0 = (int)(all * rank / ranks), s1 = (int)(all * (rank + 1) / ranks);
  const int each = (r + 15) / 16, blocks = (s1 - s0) * each;   // block b: stretch s0 + b / each, rows 16 (b % each) and on
  auto load = [&](int b, int s, int j0) {
    if (b < blocks) {
      uint8_t* to_block = smem_down + (b & 3) * kBlock;
      const int64_t k0 = (int64_t)s * kStretch;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int j = warp * 4 + (q >> 1), c = lane + 32 * (q & 1);     // 64 pieces of 16 bytes a row
        const bool on = j0 + j < r && k0 + c * 8 < a.K;
        cp_async16(to_block + j * (2 * kStretch + 16) + c * 16, on ? u + (int64_t)(j0 + j) * a.K + k0 + c * 8 : u, on);
      }
    }
    cp_async_commit();
  };
  int ls = s0, lj = 0;            // the block to load next
  auto step = [&](int& s, int& j) {
    j += 16;
    if (j >= r) j = 0, ++s;
  };
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    load(b, ls, lj);
    step(ls, lj);
  }
  const uint4 none = make_uint4(0, 0, 0, 0);
  Raw8<bf16> x[2];
  int s = s0, j0 = 0;
  for (int b = 0; b < blocks; ++b) {
    if (j0 == 0)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = (int64_t)s * kStretch + h * 256 + lane * 8;
        x[h].v = k < a.K ? __ldg(reinterpret_cast<const uint4*>(a.X + i * a.K + k)) : none;
      }
    cp_async_wait<3>();
    __syncwarp();                 // a warp reads what its own lanes have copied
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      F2 t = f2(0.f);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        F2 f[4], g[4];
        load4x2(reinterpret_cast<const bf16*>(smem_down + (b & 3) * kBlock + (warp * 4 + j) * (2 * kStretch + 16) +
                                              (lane + 32 * h) * 16), f);
        x[h].get(g);
#pragma unroll
        for (int q = 0; q < 4; ++q) t = fma2(f[q], g[q], t);
      }
      v[j] = sum2(t);
    }
    __syncwarp();
    load(b + 4, ls, lj);
    step(ls, lj);
    const float t = warp_sums_of<4>(v);
    const int j = j0 + warp * 4 + lane / 8;
    if (lane % 8 == 0 && j < r) sum[j] = s > s0 ? sum[j] + t : t;
    step(s, j0);
  }
  cluster_sync_all();
  if (rank == 0) {
    const float f = a.each ? __ldg(a.each + ad) : a.one;
    for (int j = threadIdx.x; j < r; j += 128) {
      float p[8], z = 0.f;
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q) {
        p[q] = 0.f;
        if (q < ranks)
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p[q]) : "r"(mapa_shared(smem_u32(sum + j), q)));
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) z += p[q];
      a.sz[to + j] = z * f;
      if (a.Z) a.Z[to + j] = __float2bfloat16_rn(z);
    }
  }
  cluster_sync_all();             // no CTA leaves while another reads its sums
}

template <int T>
struct Few {
  static constexpr int STAGE = kRowsW * 128 + T * 128;
  static constexpr int PITCH = kRowsW + 4;                          // floats of a row of partial outputs
  static constexpr int OUT = T * PITCH * 4;
  static constexpr int COLS = T < 32 ? 32 : T;                      // TMEM columns
};
// shared memory: the ring (later the partial outputs), the update [T, 128 / ranks], s z [T, r], the rows'
// adapters and units, the bias, barriers
template <int T>
__host__ __device__ constexpr int few_ring(int stages) {
  return stages * Few<T>::STAGE > Few<T>::OUT ? stages * Few<T>::STAGE : Few<T>::OUT;
}
template <int T>
__host__ __device__ constexpr int few_smem(int stages, int ranks, int r, bool own) {
  return 1024 + few_ring<T>(stages) + T * (kRowsW / ranks) * 4 + (own ? 2 : 1) * T * r * 4 + T * 12 + 16 + kRowsW * 4 +
         8 * (2 * stages + 2) + 32;
}

// zp[t][j] = sum over K-steps k0 .. k1 - 1 of x[t] A_a[j]: a warp takes every eighth group of four j of a row
template <int T>
__device__ __forceinline__ void own_z(const FewArgs& a, const int* ids, int rows, int m0, int warp, int lane, int k0, int k1,
                                      float* zp) {
  const int quads = a.r / 4;
  const int64_t end = min(a.K, (int64_t)k1 * kBK);
  const uint4 none = make_uint4(0, 0, 0, 0);
  for (int g = warp; g < rows * quads; g += kUpdate / 32) {
    const int t = g / quads, j0 = (g - t * quads) * 4, ad = ids[t];
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (ad >= 0) {
      const bf16 *x = a.X + (int64_t)(m0 + t) * a.K, *u = a.A + ((int64_t)ad * a.r + j0) * a.K;
      F2 s[4] = {f2(0.f), f2(0.f), f2(0.f), f2(0.f)};
      for (int64_t k = (int64_t)k0 * kBK + lane * 8; k < end; k += 512) {
        Raw8<bf16> xr[2], ur[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool on = k + 256 * h < end;
          xr[h].v = on ? __ldg(reinterpret_cast<const uint4*>(x + k + 256 * h)) : none;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            ur[h][j].v = on ? __ldg(reinterpret_cast<const uint4*>(u + j * a.K + k + 256 * h)) : none;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          F2 p[4];
          xr[h].get(p);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            F2 q[4];
            ur[h][j].get(q);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[j] = fma2(p[i], q[i], s[j]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = sum2(s[j]);
    }
    const float z = warp_sums_of<4>(v);
    if (lane % 8 == 0) zp[t * a.r + j0 + lane / 8] = z;
  }
}

// OWN: no multi_few_down before it; every cluster computes the z of all (few) rows itself, each CTA over its
// stretch of K.
template <int T, bool OWN>
__global__ void __launch_bounds__(kThreads, 2) multi_few(const __grid_constant__ FewArgs a) {
  using F = Few<T>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int own = kRowsW / (int)ranks;                              // output columns that this CTA finishes
  float* update = reinterpret_cast<float*>(smem + few_ring<T>(a.stages));   // [T, own]
  uint32_t* szh = reinterpret_cast<uint32_t*>(update + T * own);    // [T, r / 2] s z, pairs
  uint32_t* szl = szh + T * a.r / 2;    // what their rounding left; OWN: then [T, r] z of this CTA's K
  int* ids = reinterpret_cast<int*>(szl + T * a.r / 2 + (OWN ? T * a.r : 0));   // [T]
  uint32_t* leaders = reinterpret_cast<uint32_t*>(ids + T);         // rows that begin a unit; two more words unused
  float* bias = reinterpret_cast<float*>(leaders + 4);              // [128] of this CTA's columns
  uint8_t* units = reinterpret_cast<uint8_t*>(bias + kRowsW);       // [T, 8] rows, 255: none
  uint64_t* full = reinterpret_cast<uint64_t*>(units + 8 * T);
  uint64_t* empty = full + a.stages;
  uint64_t* done = empty + a.stages;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = (int)(blockIdx.x / ranks) * kRowsW, m0 = (int)blockIdx.y * T;
  const int rows = min(T, a.M - m0);
  const int k0 = (int)((int64_t)a.nk * rank / ranks), k1 = (int)((int64_t)a.nk * (rank + 1) / ranks);

  auto copy = [&](int i) {      // K-step k0 + i of this CTA
    const int s = i % a.stages;
    uint8_t* st = smem + s * F::STAGE;
    mbar_expect_tx(&full[s], F::STAGE);
    tma_load_2d(st, &a.tmW, &full[s], (k0 + i) * kBK, n0);
    tma_load_2d(st + kRowsW * 128, &a.tmX, &full[s], (k0 + i) * kBK, m0);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_fence_init();
    if (!OWN)                   // what came before multi_few_down is complete: these set off while the rest is set up
      for (int i = 0; i < min(a.stages, k1 - k0); ++i) copy(i);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, F::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (OWN) pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  if (OWN && threadIdx.x == 0)
    for (int i = 0; i < min(a.stages, k1 - k0); ++i) copy(i);
  if (OWN && warp < 2) cluster_arrive();   // the update's warps exchange their z once; these wait below

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int last = min(a.stages, k1 - k0);
      for (int i = last; i < k1 - k0; ++i) {
        if (!mbar_wait(&empty[i % a.stages], (uint32_t)(i / a.stages + 1) & 1, a.timeout_ns, abort_flag, a.err, 0x401)) {
          ok = false;
          break;
        }
        copy(i);
        last = i + 1;
      }
      if (!ok)                  // unwind: what is on its way lands before the CTA goes on
        for (int i = last > a.stages ? last - a.stages : 0; i < last; ++i)
          mbar_wait_drain(&full[i % a.stages], (uint32_t)(i / a.stages) & 1, 20000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = umma_idesc_bf16(kRowsW, T, 0, 0);
      for (int ks = k0; ks < k1; ++ks) {
        const int i = ks - k0, s = i % a.stages;
        if (!mbar_wait(&full[s], (uint32_t)(i / a.stages) & 1, a.timeout_ns, abort_flag, a.err, 0x402)) break;
        tc_fence_after();
        const uint32_t w = smem_u32(smem + s * F::STAGE), x = w + kRowsW * 128;
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
          umma_bf16(tmem, umma_smem_desc(w + kk * 32, 16, 1024), umma_smem_desc(x + kk * 32, 16, 1024), idesc,
                    (i > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&empty[s]);
      }
      umma_commit(done);
      mbar_wait_drain(done, 0, 20000000ull);
    }
    __syncwarp();
  } else {
    // the update of this CTA's own columns, while W0 streams in.  Up to eight rows of one adapter are a unit, the N side
    // of a warp MMA whose M side is 16 columns of the factor
    const int e = threadIdx.x - 64;
    if (e < T) {
      ids[e] = e < rows ? __ldg(a.ids + m0 + e) : -2;
      reinterpret_cast<uint2*>(units)[e] = make_uint2(0xffffffffu, 0xffffffffu);
    }
    named_bar_sync(1, kUpdate);
    float* zp = reinterpret_cast<float*>(szl + T * a.r / 2);   // OWN: [T, r] z of this CTA's stretch of K
    if (OWN) {
      own_z<T>(a, ids, rows, m0, e >> 5, lane, k0, k1, zp);
      cluster_arrive();
    }
    int place = 0, lead = 0;                           // among the rows of its adapter; the first row of its unit
    if (e < T) {
      const int ad = ids[e];
#pragma unroll
      for (int t = 0; t < T; ++t)
        if (ids[t] == ad && t <= e) {
          if ((place & 7) == 0) lead = t;
          ++place;
        }
    }
    if (e < (T + 31) / 32 * 32) {
      const uint32_t leads = __ballot_sync(0xffffffffu, e < rows && lead == e);
      if (lane == 0) leaders[e >> 5] = leads;
    }
    named_bar_sync(1, kUpdate);
    const uint32_t l0 = leaders[0], l1 = T > 32 ? leaders[1] : 0u;
    const int n_units = __popc(l0) + __popc(l1);
    if (e < rows) {
      const int at = lead < 32 ? __popc(l0 & ((1u << lead) - 1)) : __popc(l0) + __popc(l1 & ((1u << (lead - 32)) - 1));
      units[at * 8 + ((place - 1) & 7)] = (uint8_t)e;
    }
    named_bar_sync(1, kUpdate);
    // A piece is 16 columns of the factor and 16 of the rank.  Lane (g, q) reads 16 bytes: eight numbers of row g (q < 2) or
    // g + 8; lanes q and q + 2 exchange halves, and each has four numbers of both rows, which go into the MMA as
    // they lie, and s z by the same order: a sum over the rank may run in any.  A warp has every eighth (unit, 16
    // columns), kAhead of its pieces on their way, the first ones before z is there.  s z comes in two bf16 parts,
    // the second what the first one's rounding left.
    const int n = n0 + (int)rank * own, groups = own / 16, items = n_units * groups, uw = e >> 5;
    const int g = lane >> 2, q8 = (lane & 1) * 8, q4 = q8 + (lane & 2) * 2;   // what it reads of the 16, what it keeps
    if (e < own) bias[e] = a.bias && n + e < a.N ? __bfloat162float(a.bias[n + e]) : 0.f;   // read behind a barrier
    uint4 w[2][kAhead];
    int fi = uw, fj = 0;
    // first where all of them lie, then the loads: a wait for one shared-memory access between them would be one for
    // the loads before it, too (64 rows: 5 us until all were asked for)
    auto fetch = [&](uint4 (&x)[kAhead]) {
      const bf16* from[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int u = fi / groups, c = n + (fi - u * groups) * 16 + g + (lane & 2) * 4;
        const int ad = fi < items && fj + q8 < a.r && c < a.N ? ids[units[u * 8]] : -1;
        from[i] = ad >= 0 ? a.B + ((int64_t)ad * a.N + c) * a.r + fj + q8 : nullptr;
        fj += 16;
        if (fj >= a.r) fj = 0, fi += kUpdate / 32;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        x[i] = from[i] ? __ldg(reinterpret_cast<const uint4*>(from[i])) : make_uint4(0, 0, 0, 0);
    };
    fetch(w[0]);
    fetch(w[1]);
    // s z, two words: hi and lo of a pair
    auto put_z = [&](int i, float z0, float z1) { split_bf16x2(z0, z1, szh[i / 2], szl[i / 2]); };
    if (OWN) {
      cluster_wait();
      for (int i = e * 2; i < rows * a.r; i += kUpdate * 2) {
        float2 p[8];
        float z0 = 0.f, z1 = 0.f;
#pragma unroll
        for (uint32_t s = 0; s < 8; ++s) {
          p[s] = make_float2(0.f, 0.f);
          if (s < ranks)
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                         : "=f"(p[s].x), "=f"(p[s].y)
                         : "r"(mapa_shared(smem_u32(zp + i), s)));
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) z0 += p[s].x, z1 += p[s].y;
        if (a.Z && blockIdx.x == 0) *reinterpret_cast<uint32_t*>(a.Z + (int64_t)m0 * a.r + i) = pack_bf16x2(z0, z1);
        const int ad = ids[i / a.r];
        const float f = ad < 0 ? 0.f : a.each ? __ldg(a.each + ad) : a.one;
        put_z(i, z0 * f, z1 * f);
      }
    } else {
      pdl_wait();
#pragma unroll 4
      for (int i = e * 2; i < rows * a.r; i += kUpdate * 2) {
        const float2 z = __ldcg(reinterpret_cast<const float2*>(a.sz + (int64_t)m0 * a.r + i));
        put_z(i, z.x, z.y);
      }
    }
    named_bar_sync(1, kUpdate);
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    int it = uw, j = 0;
    auto use = [&](const uint4 (&x)[kAhead]) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (it >= items) break;
        const int u = it / groups, c = (it - u * groups) * 16;
        const uint2 rows8 = *reinterpret_cast<const uint2*>(units + u * 8);
        const uint32_t half = lane & 16 ? rows8.y : rows8.x;
        const int row = (half >> (8 * (g & 3))) & 255;
        uint2 hi = make_uint2(0, 0), lo = hi;
        if (row != 255 && j + q4 < a.r) {
          hi = *reinterpret_cast<const uint2*>(szh + (row * a.r + j + q4) / 2);
          lo = *reinterpret_cast<const uint2*>(szl + (row * a.r + j + q4) / 2);
        }
        const bool up = lane & 2;
        const uint32_t r0 = __shfl_xor_sync(0xffffffffu, up ? x[i].x : x[i].z, 2),
                       r1 = __shfl_xor_sync(0xffffffffu, up ? x[i].y : x[i].w, 2);
        const uint32_t m[4] = {up ? r0 : x[i].x, up ? x[i].z : r0, up ? r1 : x[i].y, up ? x[i].w : r1};
        const uint32_t f[4] = {finite_bf16x2(m[0]), finite_bf16x2(m[1]), finite_bf16x2(m[2]), finite_bf16x2(m[3])};
        mma_bf16_16816(d, m, hi.x, hi.y);
        mma_bf16_16816(d, f, lo.x, lo.y);
        j += 16;
        if (j >= a.r) {
          const uint32_t pair = ((lane & 2 ? rows8.y : rows8.x) >> (16 * (lane & 1))) & 0xffffu;
#pragma unroll
          for (int k = 0; k < 4; ++k) {                // columns g and g + 8, the unit's rows 2 (lane % 4) and + 1
            const int t = (pair >> (8 * (k & 1))) & 255, at = c + g + (k >> 1) * 8;
            if (t != 255) update[t * own + at] = d[k] + bias[at];
            d[k] = 0.f;
          }
          j = 0;
          it += kUpdate / 32;
        }
      }
    };
    while (it < items) {
      use(w[0]);
      if (it >= items) break;
      fetch(w[0]);
      use(w[1]);
      fetch(w[1]);
    }
    // the accumulator, once every MMA is done: the ring is free then
    const int q = warp & 3;
    const bool ok = warp >= 6 || mbar_wait(done, 0, a.timeout_ns, abort_flag, a.err, 0x403);
    tc_fence_after();
    float* out = reinterpret_cast<float*>(smem);
    if (warp < 6 && __all_sync(0xffffffffu, ok)) {
#pragma unroll
      for (int c0 = 0; c0 < T; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tmem + ((uint32_t)(32 * q) << 16) + c0, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) out[(c0 + i) * F::PITCH + 32 * q + lane] = __uint_as_float(v[i]);
      }
    }
    tc_fence_before();
  }
  if (OWN && warp < 2) cluster_wait();
  cluster_sync_all();
  tc_fence_after();
  // this CTA's columns: the ranks' partial sums in their order, and the update
  const uint32_t mine = smem_u32(smem);
  const int quads = own / 4;
  for (int i = threadIdx.x; i < rows * quads; i += kThreads) {
    const int t = i / quads, f = (i - t * quads) * 4, c = n0 + (int)rank * own + f;
    float4 p[8], v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (uint32_t s = 0; s < 8; ++s) {
      p[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < ranks)
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(p[s].x), "=f"(p[s].y), "=f"(p[s].z), "=f"(p[s].w)
                     : "r"(mapa_shared(mine + (t * F::PITCH + (int)rank * own + f) * 4, s)));
    }
#pragma unroll
    for (int s = 0; s < 8; ++s) v.x += p[s].x, v.y += p[s].y, v.z += p[s].z, v.w += p[s].w;
    const float4 u = *reinterpret_cast<const float4*>(update + t * own + f);
    if (c < a.N)                // N is a multiple of 8
      *reinterpret_cast<uint2*>(a.Y + (int64_t)(m0 + t) * a.N + c) =
          make_uint2(pack_bf16x2(v.x + u.x, v.y + u.y), pack_bf16x2(v.z + u.z, v.w + u.w));
  }
  cluster_sync_all();           // no CTA leaves while another reads its sums
  if (warp == 1) tmem_dealloc(tmem, F::COLS);
}

// beside: shared memory that multi_few_down's CTAs hold on an SM
template <int T, bool OWN>
cudaError_t few_launch(FewArgs& a, int beside, cudaStream_t st) {
  constexpr int kMost = 200 * 1024, kSm = 227 * 1024;
  const int tiles = (a.N + kRowsW - 1) / kRowsW, groups = (a.M + T - 1) / T;
  const int slots = 2 * num_sms_current();
  int ranks = 1;
  while (ranks < 8 && tiles * groups * ranks * 2 <= slots && a.nk >= ranks * 2 * 2) ranks *= 2;
  // what is on its way beyond the bytes that the memory needs only queues up, and the update's loads behind it
  const int each = a.nk / ranks + (a.nk % ranks != 0);
  int stages = (int)(kInFlight / ((int64_t)tiles * groups * ranks * Few<T>::STAGE));
  if (stages < 3) stages = 3;
  if (stages > 12) stages = 12;
  if (stages > each) stages = each;
  // two CTAs an SM, from the start: those that came after multi_few_down had ended decided the time
  while (stages > 2 && 2 * (few_smem<T>(stages, ranks, a.r, OWN) + 1024) + beside > kSm) --stages;
  a.stages = stages;
  const cudaError_t e = allow_smem<multi_few<T, OWN>>(kMost);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(tiles * ranks, groups, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = few_smem<T>(stages, ranks, a.r, OWN);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + pdl_attr(&attr[1]);
  const cudaError_t l = cudaLaunchKernelEx(&cfg, multi_few<T, OWN>, a);
  count_launch();
  return l != cudaSuccess ? l : cudaGetLastError();
}

cudaError_t down_launch(const FewArgs& a, int* beside, cudaStream_t st) {
  const int64_t stretches = (a.K + kStretch - 1) / kStretch, ctas = (int64_t)kDownCtas * num_sms_current();
  int ranks = 1;
  while (ranks < 8 && ranks * 2 <= stretches && (int64_t)a.M * ranks * 2 <= ctas) ranks *= 2;
  const int64_t blocks = (stretches + ranks - 1) / ranks * ((a.r + 15) / 16);
  const cudaError_t s = allow_smem<multi_few_down>(4 * kBlock);
  if (s != cudaSuccess) return s;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(a.M * ranks, 1, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.dynamicSmemBytes = (size_t)(blocks < 4 ? blocks : 4) * kBlock;
  *beside = (a.M * ranks + num_sms_current() - 1) / num_sms_current() * ((int)cfg.dynamicSmemBytes + 2048);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + pdl_attr(&attr[1]);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, multi_few_down, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Measured against the GEMM of 256-row tiles (K = 4096, us here and there): N 4096, 64 rows: 17.6, 29.6; 128: 20.4,
// 30.1; 192: 29.4, 30.1; N 11008, 64: 30.5, 33.2; 128: 48.6, 34.2; 256 rows, N 1024: 23.8, 28.4; 2048: 24.7, 29.9;
// 512 rows, N 1024: 31, 28.  Up to 128 rows while two CTAs share K, more only where four do: 256 rows up to N 2432,
// 192 up to 3200, 128 up to 9728, 64 up to 19456.  These figures are of 16 adapters at rank 16.  What the rule does
// not see is the GEMM's tail, 0.2 us for each adapter of a tile and 16 of the rank: behind its border a batch with an
// adapter for every row is slow (4096 x 4096, rank 16: 128 rows 29 us, 129 rows 69, 256 rows 102, at rank 64 271;
// with eight adapters 21, 29, 29, 34), and so is a single row of more than 19456 columns (28672: 83 us for 35 of
// reads).
bool multi_few_fits(int64_t M, int64_t N) {
  const int64_t groups = (M + 63) / 64, ctas = (N + kRowsW - 1) / kRowsW * groups;
  return M <= kFewRows && ctas * (groups <= 2 ? 2 : 4) <= 2 * num_sms_current();
}

cudaError_t multi_few_fwd(const MultiPlan& p, int64_t N, int64_t K, int r, const bf16* X, const bf16* W0,
                          const bf16* A, const bf16* B, const bf16* bias, float one, const float* each, float* sz,
                          bf16* Y, bf16* Z, uint32_t* err, uint64_t timeout_ns, cudaStream_t st) {
  FewArgs a;
  memset(&a, 0, sizeof(a));
  a.M = (int)p.M;
  a.N = (int)N;
  a.r = r;
  a.K = K;
  a.nk = (int)((K + kBK - 1) / kBK);
  a.ids = p.ids;
  a.X = X;
  a.A = A;
  a.B = B;
  a.bias = bias;
  a.one = one;
  a.each = each;
  a.sz = sz;
  a.Y = Y;
  a.Z = Z;
  a.err = err;
  a.timeout_ns = timeout_ns;
  const int T = a.M <= 16 ? 16 : a.M <= 32 ? 32 : 64;
  if (!make_tmap_bf16(&a.tmW, W0, K, N, K, kBK, kRowsW, 128) || !make_tmap_bf16(&a.tmX, X, K, p.M, K, kBK, T, 128))
    return cudaErrorInvalidValue;
  // with few sums its z costs a cluster less than the kernel before it: A_a is read at most half as often as W0
  if (a.M <= 16 && a.M * r <= kRowsW / 2) return few_launch<16, true>(a, 0, st);
  int beside = 0;
  const cudaError_t e = down_launch(a, &beside, st);
  if (e != cudaSuccess) return e;
  return T == 16 ? few_launch<16, false>(a, beside, st) : T == 32 ? few_launch<32, false>(a, beside, st)
                                                                  : few_launch<64, false>(a, beside, st);
}

}  // namespace lg
