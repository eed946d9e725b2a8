// The many-adapter forward of a few rows (a decode step), bf16.
//
// Y [M, N] = X W0^T + the rows' own updates, M small: every byte of W0 is read once, which bounds it.  So the
// product is turned around: 128 rows of W0 are the M side of the tcgen05 MMA and the batch's rows its N side
// (16, 32 or 64, zero-filled), and K is shared by the CTAs of a cluster, each with its own stretch of W0, so that
// some 300 CTAs, two an SM, keep their copies in flight.  The partial accumulators meet through distributed
// shared memory, in the order of the ranks.  The rank-r part is computed on the side:
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
constexpr int kUpdate = 256;       // threads of the update; four of their warps read the accumulator
constexpr int kThreads = 64 + kUpdate;   // copies, MMA
constexpr int kAhead = 6;         // pieces of the factor that a thread has on their way

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
// stretches of 512; of each a warp takes every W-th group of J rows of A_a, all of their loads on their way at once.
template <int J, int W>
__global__ void __launch_bounds__(32 * W) multi_few_down(const __grid_constant__ FewArgs a) {
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
    for (int j = threadIdx.x; rank == 0 && j < r; j += 32 * W) {
      a.sz[to + j] = 0.f;
      if (a.Z) a.Z[to + j] = __float2bfloat16_rn(0.f);
    }
    return;
  }
  const bf16* u = a.A + (int64_t)ad * r * a.K;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const int64_t all = (a.K + kStretch - 1) / kStretch;
  const int s0 = (int)(all * rank / ranks), s1 = (int)(all * (rank + 1) / ranks);
  for (int st = s0; st < s1; ++st) {
    int64_t k[2];
    bool on[2];
    Raw8<bf16> x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      k[h] = (int64_t)st * kStretch + h * 256 + lane * 8;
      on[h] = k[h] < a.K;
      x[h].v = on[h] ? __ldg(reinterpret_cast<const uint4*>(a.X + i * a.K + k[h])) : none;
    }
    for (int j0 = warp * J; j0 < r; j0 += W * J) {
      Raw8<bf16> w[J][2];
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[j][h].v = on[h] ? __ldg(reinterpret_cast<const uint4*>(u + (int64_t)(j0 + j) * a.K + k[h])) : none;
      float s[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        F2 t = f2(0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          F2 f[4], g[4];
          w[j][h].get(f);
          x[h].get(g);
#pragma unroll
          for (int q = 0; q < 4; ++q) t = fma2(f[q], g[q], t);
        }
        s[j] = sum2(t);
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
      if (lane == 0)
#pragma unroll
        for (int j = 0; j < J; ++j) sum[j0 + j] = st > s0 ? sum[j0 + j] + s[j] : s[j];
    }
  }
  cluster_sync_all();
  if (rank == 0) {
    const float f = a.each ? __ldg(a.each + ad) : a.one;
    for (int j = threadIdx.x; j < r; j += 32 * W) {
      float p[8], z = 0.f;
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q) {
        p[q] = 0.f;
        if (q < ranks) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(p[q]) : "r"(mapa_shared(smem_u32(sum + j), q)));
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
// adapters, barriers
template <int T>
__host__ __device__ constexpr int few_ring(int stages) {
  return stages * Few<T>::STAGE > Few<T>::OUT ? stages * Few<T>::STAGE : Few<T>::OUT;
}
template <int T>
__host__ __device__ constexpr int few_smem(int stages, int ranks, int r) {
  return 1024 + few_ring<T>(stages) + T * (kRowsW / ranks) * 4 + T * r * 4 + T * 4 + 8 * (2 * stages + 2) + 32;
}

template <int T>
__global__ void __launch_bounds__(kThreads) multi_few(const __grid_constant__ FewArgs a) {
  using F = Few<T>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int own = kRowsW / (int)ranks;                              // output columns that this CTA finishes
  float* update = reinterpret_cast<float*>(smem + few_ring<T>(a.stages));   // [T, own]
  float* sz = update + T * own;                                     // [T, r]
  int* ids = reinterpret_cast<int*>(sz + T * a.r);                  // [T]
  uint64_t* full = reinterpret_cast<uint64_t*>(ids + T);
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
    for (int i = 0; i < min(a.stages, k1 - k0); ++i) copy(i);   // on their way while the rest is set up
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, F::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (threadIdx.x == 0) pdl_trigger();

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
    // the update of this CTA's own columns, while W0 streams in
    const int e = threadIdx.x - 64;
    if (e < T) ids[e] = e < rows ? __ldg(a.ids + m0 + e) : -1;
    named_bar_sync(1, kUpdate);
    const int f = e % own, c = n0 + (int)rank * own + f, step = kUpdate / own;
    const float b = a.bias && c < a.N ? __bfloat162float(a.bias[c]) : 0.f;
    // this thread's rows are e / own, + step, ..; it takes their factor's row by 16 columns at a time, kAhead of these on
    // their way, the first ones before z is there
    uint4 w[kAhead][2];
    int ft = e / own, fj = 0;
    auto fetch = [&](uint4 (&x)[2]) {
      const int ad = ft < rows && c < a.N ? ids[ft] : -1;
      const bf16* u = a.B + ((int64_t)max(ad, 0) * a.N + c) * a.r + fj;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        x[h] = ad >= 0 && fj + 8 * h < a.r ? __ldg(reinterpret_cast<const uint4*>(u + 8 * h)) : make_uint4(0, 0, 0, 0);
      fj += 16;
      if (fj >= a.r) fj = 0, ft += step;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(w[i]);
    pdl_wait();
    for (int i = e * 4; i < rows * a.r; i += kUpdate * 4)
      *reinterpret_cast<float4*>(sz + i) = __ldcg(reinterpret_cast<const float4*>(a.sz + (int64_t)m0 * a.r + i));
    named_bar_sync(1, kUpdate);
    float v = b;
    for (int t = e / own, j = 0; t < rows;) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (t >= rows) break;
        const float* z = sz + t * a.r + j;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (j + 8 * h < a.r) {
            const uint32_t x[4] = {w[i][h].x, w[i][h].y, w[i][h].z, w[i][h].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 p = unpack_bf16x2(x[q]), s = *reinterpret_cast<const float2*>(z + 8 * h + 2 * q);
              v = fmaf(p.x, s.x, fmaf(p.y, s.y, v));
            }
          }
        fetch(w[i]);
        j += 16;
        if (j >= a.r) {
          update[t * own + f] = v;
          v = b;
          j = 0;
          t += step;
        }
      }
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
  cluster_sync_all();
  tc_fence_after();
  // this CTA's columns: the ranks' partial sums in their order, and the update
  const uint32_t mine = smem_u32(smem);
  const int pairs = own / 2;
  for (int i = threadIdx.x; i < rows * pairs; i += kThreads) {
    const int t = i / pairs, f = i % pairs * 2, c = n0 + (int)rank * own + f;
    float p[8][2], v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (uint32_t s = 0; s < 8; ++s) {
      p[s][0] = p[s][1] = 0.f;
      if (s < ranks)
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                     : "=f"(p[s][0]), "=f"(p[s][1])
                     : "r"(mapa_shared(mine + (t * F::PITCH + (int)rank * own + f) * 4, s)));
    }
#pragma unroll
    for (int s = 0; s < 8; ++s) v0 += p[s][0], v1 += p[s][1];
    if (c < a.N)
      *reinterpret_cast<uint32_t*>(a.Y + (int64_t)(m0 + t) * a.N + c) =
          pack_bf16x2(v0 + update[t * own + f], v1 + update[t * own + f + 1]);
  }
  cluster_sync_all();           // no CTA leaves while another reads its sums
  if (warp == 1) tmem_dealloc(tmem, F::COLS);
}

template <int T>
cudaError_t few_launch(FewArgs& a, cudaStream_t st) {
  constexpr int kMost = 200 * 1024;
  const int tiles = (a.N + kRowsW - 1) / kRowsW, groups = (a.M + T - 1) / T;
  const int slots = 2 * num_sms_current();
  int ranks = 1;
  while (ranks < 8 && tiles * groups * ranks * 2 <= slots && a.nk >= ranks * 2 * 2) ranks *= 2;
  // two CTAs an SM where their rings are at least four stages deep so
  int stages = 12;
  const int each = a.nk / ranks + (a.nk % ranks != 0);
  if (stages > each) stages = each;
  while (stages > 4 && few_smem<T>(stages, ranks, a.r) > 112 * 1024) --stages;
  while (stages > 2 && few_smem<T>(stages, ranks, a.r) > kMost) --stages;
  a.stages = stages;
  const cudaError_t e = allow_smem<multi_few<T>>(kMost);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(tiles * ranks, groups, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = few_smem<T>(stages, ranks, a.r);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + pdl_attr(&attr[1]);
  const cudaError_t l = cudaLaunchKernelEx(&cfg, multi_few<T>, a);
  count_launch();
  return l != cudaSuccess ? l : cudaGetLastError();
}

template <int J, int W>
cudaError_t down_launch(const FewArgs& a, cudaStream_t st) {
  const int64_t stretches = (a.K + kStretch - 1) / kStretch;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)(stretches < 8 ? stretches : 8);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(a.M * attr[0].val.clusterDim.x, 1, 1);
  cfg.blockDim = dim3(32 * W, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + pdl_attr(&attr[1]);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, multi_few_down<J, W>, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

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
  const cudaError_t e = r <= 16   ? down_launch<2, 8>(a, st)
                        : r <= 32 ? down_launch<4, 8>(a, st)
                                  : down_launch<4, 16>(a, st);
  if (e != cudaSuccess) return e;
  return T == 16 ? few_launch<16>(a, st) : T == 32 ? few_launch<32>(a, st) : few_launch<64>(a, st);
}

}  // namespace lg
