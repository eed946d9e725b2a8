// The many-adapter projection in fp32: FMA tiles, no reduced-precision tensor math, as everywhere here for fp32.
//
// Sums over long axes are taken in shares that are added up afterwards, so that their rounding grows with the share:
// those over rows in shares of a fixed length, the product's over K in one for each group of warps and CTA of a cluster.
#include "common.cuh"
#include "multi.h"
#include "vec.cuh"

namespace lg {

namespace {

__device__ __forceinline__ float scale_of(float one, const float* each, int a) { return each ? __ldg(each + a) : one; }

// ------------------------------------------------------------------ rank-r products of rows
// A CTA has eight rows of an item, all j of their adapter and its cluster rank's share of K; the rows pass through
// shared memory 1024 columns at a time, so a factor is read once for eight rows.  Up to eight warps take the j of
// U_a [r, K] in turn; of U_a [K, r] (KR) a thread keeps one j, and the threads' shares of k meet in shared memory.
// Latency: 10 us for 509 x 1000, rank 12, as for 300 x 1376, rank 8.
constexpr int kCols = 1024, kRows = 8;   // kItemRows is a multiple of kRows

struct F32Proj {
  MultiPlan p;
  int64_t K;
  int r;
  const float *S, *U;
  float one;
  const float* each;
  float *plain, *scaled;          // [M, r] T and s_a T; either may be null
};

template <bool KR>
__global__ void __launch_bounds__(256) f32_proj_kernel(const __grid_constant__ F32Proj a) {
  __shared__ float x[kRows][kCols];
  __shared__ float sum[kRows][128];
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int sub = (int)(blockIdx.x / ranks);
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int4 item = a.p.items[sub / (kItemRows / kRows)];   // there is room for as many as the grid has
  const int r = a.r, with = a.p.head[kHeadRows], items = a.p.head[kHeadItems];
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (a.p.M - with) * r; i += (int64_t)gridDim.x * 256) {
    const int64_t at = (int64_t)a.p.order[with + i / r] * r + i % r;     // rows without adapter
    if (a.plain) a.plain[at] = 0.f;
    if (a.scaled) a.scaled[at] = 0.f;
  }
  if (sub / (kItemRows / kRows) >= items) return;                  // the whole cluster
  const int first = sub % (kItemRows / kRows) * kRows, rows = min(kRows, item.z - first);
  if (rows <= 0) return;
  const int64_t begin = a.K / 8 * rank / ranks * 8, end = a.K / 8 * (rank + 1) / ranks * 8;   // K is a multiple of 8
  const int32_t* order = a.p.order + item.y + first;
  const float* u = a.U + (int64_t)item.x * r * a.K;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kRows * 128; i += 256) (&sum[0][0])[i] = 0.f;
  for (int64_t k0 = begin; k0 < end; k0 += kCols) {
    const int cols = (int)min((int64_t)kCols, end - k0);
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kCols / 4; i += 256) {
      const int m = i / (kCols / 4), c = i % (kCols / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (m < rows && c < cols) v = __ldg(reinterpret_cast<const float4*>(a.S + (int64_t)order[m] * a.K + k0 + c));
      *reinterpret_cast<float4*>(&x[m][c]) = v;
    }
    __syncthreads();
    if (!KR) {
      for (int j = warp; j < r; j += 8) {
        float t[kRows] = {};
        const float* w = u + (int64_t)j * a.K + k0;
#pragma unroll 4
        for (int c = lane * 4; c < cols; c += 128) {
          const float4 b = __ldg(reinterpret_cast<const float4*>(w + c));
#pragma unroll
          for (int m = 0; m < kRows; ++m) {
            const float4 v = *reinterpret_cast<const float4*>(&x[m][c]);
            t[m] = fmaf(v.x, b.x, fmaf(v.y, b.y, fmaf(v.z, b.z, fmaf(v.w, b.w, t[m]))));
          }
        }
        const float s = warp_sums_of<8>(t);
        if (lane % 4 == 0) sum[lane / 4][j] += s;      // this warp's j alone
      }
    } else {
      const int shares = 256 / r, j = threadIdx.x % r, k = threadIdx.x / r;
      float t[kRows] = {};
      if (k < shares) {
#pragma unroll 8
        for (int c = k; c < cols; c += shares) {
          const float b = __ldg(u + (k0 + c) * r + j);
#pragma unroll
          for (int m = 0; m < kRows; ++m) t[m] = fmaf(x[m][c], b, t[m]);
        }
      }
      __syncthreads();                                 // the rows have been read: their place takes the shares
      float* red = &x[0][0];
      if (k < shares)
#pragma unroll
        for (int m = 0; m < kRows; ++m) red[(k * kRows + m) * r + j] = t[m];
      __syncthreads();
      for (int i = threadIdx.x; i < kRows * r; i += 256) {
        float s = 0.f;
        for (int q = 0; q < shares; ++q) s += red[q * kRows * r + i];
        sum[i / r][i % r] += s;
      }
    }
  }
  cluster_sync_all();
  const float f = scale_of(a.one, a.each, item.x);
  for (int i = (int)rank * 256 + threadIdx.x; i < rows * r; i += 256 * (int)ranks) {
    const int64_t at = (int64_t)order[i / r] * r + i % r;
    float v = 0.f;
    for (uint32_t q = 0; q < ranks; ++q) {
      float s;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(s) : "r"(mapa_shared(smem_u32(&sum[i / r][i % r]), q)));
      v += s;
    }
    if (a.plain) a.plain[at] = v;
    if (a.scaled) a.scaled[at] = v * f;
  }
  cluster_sync_all();           // no CTA leaves while another reads its sums
}

// ------------------------------------------------------------------ shared product and rank-r update
// 64 x 64 outputs a CTA, 8 x 8 a thread, K in slabs of 16, of which each of two groups of two warps takes eight.
// Operands come by asynchronous copies, three slabs ahead, and lie as they do in memory: rows of 16 k (80 bytes apart,
// so that eight rows' 16 bytes fall into different banks), W [K, N] by k.  A thread reads four k of a row at once.
// What counts is warps: with two a scheduler it issues every second cycle (8 x 16 a thread: 60 us at 509 x 1000 x
// 1496, the FMA units 38% busy), so 128 registers and four CTAs an SM: 55 us, 28 TFLOP/s.  Two products an
// instruction (fma.rn.f32x2) do not help: a 16-byte read of shared memory takes four cycles of an SM, 16 of these
// feed 256 FMA, and the pairs of k they come in would need twice the accumulators (4 x 8 a thread: 5 us more).  The CTAs
// of a cluster share K and add their sums through distributed shared memory, each finishing its share of the rows.
// There a thread has one column, and takes its adapter's factor anew only where the next row has another one.  A tile
// computes 64 rows whatever the batch has: one row of 4096 x 4096 takes 80 us, 64 take 92.
constexpr int kTileM = 64, kTileN = 64, kSlab = 16, kGroups = 2, kGemmThreads = 64 * kGroups, kSlabs = 4;
constexpr int kRowPitch = kSlab + 4, kColPitch = kTileN + 4;          // floats
constexpr int kSlabA = kTileM * kRowPitch, kSlabB = kTileN * kRowPitch;
static_assert(kSlab * kColPitch <= kSlabB, "a slab of W [K, N] fits as well");
constexpr int kGemmSmem = kSlabs * (kSlabA + kSlabB) * 4;
static_assert(kGemmSmem >= kTileM * (kTileN + 4) * 4, "the sums take the slabs' place");

struct F32Gemm {
  MultiPlan p;
  int64_t N, K;
  int r;
  const float *S, *W, *P, *U, *bias;
  float one;
  const float* each;
  bool scaled;                    // the update takes s_a
  float* out;
  // The rank-r pass before this kernel gives P alone, and what came before that pass is complete when this kernel
  // starts: its sums may begin beside that pass.  Half way they wait for it, so that the kernels behind this one start
  // beside the rest (a quarter earlier or later: the same).  With one or two CTAs an SM (us without and with: backward of
  // 300 x 512 -> 1376 41.7, 40.1; 16 x 1024 -> 1024 20.0, 16.4, backward 22.8, 19.1); more are spread unevenly around that
  // pass's: 509 x 1000 -> 1496 60.4, 63.5, elsewhere up to a tenth is left (1 x 4096 -> 4096 80.1, 72.7; 200 x 1000 ->
  // 1000 33.9, 31.4; 1000 x 2048 -> 2048 261.7, 252.1; 1024 x 4096 -> 4096 834, 822).
  bool ahead;
};

template <bool MN>
__global__ void __launch_bounds__(kGemmThreads, 4) f32_gemm_kernel(const __grid_constant__ F32Gemm a) {
  constexpr int kPitch = kTileN + 4;
  extern __shared__ __align__(16) float pool[];
  __shared__ float ps[8 * kGroups][8];                // P of eight rows of each group and eight j
  __shared__ int ids[kTileM];
  float (*part)[kPitch] = reinterpret_cast<float (*)[kPitch]>(pool);
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  // rows ty + 8 i and columns tx + 8 j of a K-major W, 4 tx + 32 h and on of W [K, N]
  const int tid = threadIdx.x, group = tid >> 6, tx = tid & 7, ty = (tid >> 3) & 7;
  const int64_t K = a.K, N = a.N;
  const int tile = (int)(blockIdx.x / ranks), wide = (int)((N + kTileN - 1) / kTileN);
  const int64_t m0 = (int64_t)(tile / wide) * kTileM, n0 = (int64_t)(tile % wide) * kTileN;
  const int slabs = (int)((K + kSlab - 1) / kSlab), s0 = (int)((int64_t)slabs * rank / ranks),
            s1 = (int)((int64_t)slabs * (rank + 1) / ranks);
  // a thread brings four k of two rows of S and of W [N, K], four lanes a row; of W [K, N] four columns of every eighth k
  const int lr = tid >> 2, lk = (tid & 3) * 4, lc = (tid & 15) * 4;
  auto load = [&](int s) {
    if (s < s1) {
      float* A = pool + (s - s0) % kSlabs * (kSlabA + kSlabB);
      float* B = A + kSlabA;
      const int64_t k = (int64_t)s * kSlab + lk;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool on = k < K && m0 + lr + 32 * i < a.p.M;
        cp_async16(A + (lr + 32 * i) * kRowPitch + lk, on ? a.S + (m0 + lr + 32 * i) * K + k : a.S, on);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (MN) {
          const int kk = (tid >> 4) + 8 * i;
          const int64_t row = (int64_t)s * kSlab + kk;
          const bool on = row < K && n0 + lc < N;
          cp_async16(B + kk * kColPitch + lc, on ? a.W + row * N + n0 + lc : a.W, on);
        } else {
          const bool on = k < K && n0 + lr + 32 * i < N;
          cp_async16(B + (lr + 32 * i) * kRowPitch + lk, on ? a.W + (n0 + lr + 32 * i) * K + k : a.W, on);
        }
    }
    cp_async_commit();
  };
  float run[8][8] = {};
  const int wait_at = a.ahead ? (s0 + s1) / 2 : s1;
  if (!a.ahead) {
    pdl_wait();
    if (threadIdx.x == 0) pdl_trigger();
  }
#pragma unroll
  for (int s = 0; s < kSlabs - 1; ++s) load(s0 + s);
  for (int s = s0; s < s1; ++s) {
    if (s == wait_at) {
      pdl_wait();
      if (threadIdx.x == 0) pdl_trigger();
    }
    cp_async_wait<kSlabs - 2>();
    __syncthreads();              // slab s is there, and all are done with the one that is loaded next
    load(s + kSlabs - 1);
    const float* A = pool + (s - s0) % kSlabs * (kSlabA + kSlabB) + ty * kRowPitch + group * 8;
    const float* B = pool + (s - s0) % kSlabs * (kSlabA + kSlabB) + kSlabA;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float p[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 u = *reinterpret_cast<const float4*>(A + 8 * i * kRowPitch + 4 * q);
        p[i][0] = u.x, p[i][1] = u.y, p[i][2] = u.z, p[i][3] = u.w;
      }
      if (MN) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 v = *reinterpret_cast<const float4*>(B + (group * 8 + 4 * q + k) * kColPitch + 32 * h + 4 * tx);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              run[i][4 * h] = fmaf(p[i][k], v.x, run[i][4 * h]);
              run[i][4 * h + 1] = fmaf(p[i][k], v.y, run[i][4 * h + 1]);
              run[i][4 * h + 2] = fmaf(p[i][k], v.z, run[i][4 * h + 2]);
              run[i][4 * h + 3] = fmaf(p[i][k], v.w, run[i][4 * h + 3]);
            }
          }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 v = *reinterpret_cast<const float4*>(B + (tx + 8 * j) * kRowPitch + group * 8 + 4 * q);
#pragma unroll
          for (int i = 0; i < 8; ++i) run[i][j] = fmaf(p[i][0], v.x, run[i][j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) run[i][j] = fmaf(p[i][1], v.y, run[i][j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) run[i][j] = fmaf(p[i][2], v.z, run[i][j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) run[i][j] = fmaf(p[i][3], v.w, run[i][j]);
        }
      }
    }
  }
  cp_async_wait<0>();
  // the groups' sums one after another
  for (int q = 0; q < kGroups; ++q) {
    __syncthreads();
    if (group == q)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float* at = &part[ty + 8 * i][MN ? 32 * (j >> 2) + 4 * tx + (j & 3) : tx + 8 * j];
          *at = q == 0 ? run[i][j] : *at + run[i][j];
        }
  }
  if (tid < kTileM) ids[tid] = m0 + tid < a.p.M ? a.p.ids[m0 + tid] : -1;
  cluster_sync_all();
  // this thread's column of its group's half of this CTA's share of the rows, eight rows at a time
  const int c = tid & 63, part_of = (int)rank * kGroups + group, parts = (int)ranks * kGroups;
  const int r0 = kTileM * part_of / parts, r1 = kTileM * (part_of + 1) / parts;
  const int rounds = ((kTileM + parts - 1) / parts + 7) / 8;          // of the longest share
  const uint32_t mine = smem_u32(&part[0][0]);
  const float bias = a.bias && n0 + c < N ? __ldg(a.bias + n0 + c) : 0.f;
  for (int round = 0; round < rounds; ++round) {
    const int e0 = r0 + 8 * round;
    float v[8], t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = t[i] = 0.f;
    for (uint32_t q = 0; q < ranks; ++q) {
      const uint32_t from = mapa_shared(mine + (e0 * kPitch + c) * 4, q);
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[i] = 0.f;
        if (e0 + i < r1) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f[i]) : "r"(from + i * kPitch * 4));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += f[i];
    }
    for (int j0 = 0; j0 < a.r; j0 += 8) {
      __syncthreads();
      {
        const int m = e0 + (c >> 3), j = j0 + (c & 7);
        ps[group * 8 + (c >> 3)][c & 7] = m < r1 && ids[m] >= 0 && j < a.r ? a.P[(m0 + m) * a.r + j] : 0.f;
      }
      __syncthreads();
      if (n0 + c < N) {
        int have = -1;
        float u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (e0 + i >= r1) break;
          const int ad = ids[e0 + i];
          if (ad < 0) continue;
          if (ad != have) {
            have = ad;
            const float* f = a.U + (int64_t)ad * a.r * N;
            if (!MN && (a.r & 3) == 0) {              // a row of the factor by 16 bytes
#pragma unroll
              for (int q = 0; q < 8; q += 4) {
                const float4 x = j0 + q < a.r ? __ldg(reinterpret_cast<const float4*>(f + (n0 + c) * a.r + j0 + q))
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
                u[q] = x.x, u[q + 1] = x.y, u[q + 2] = x.z, u[q + 3] = x.w;
              }
            } else {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                u[q] = j0 + q < a.r ? __ldg(MN ? f + (int64_t)(j0 + q) * N + n0 + c : f + (n0 + c) * a.r + j0 + q) : 0.f;
            }
          }
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (j0 + q < a.r) t[i] = fmaf(ps[group * 8 + i][q], u[q], t[i]);
        }
      }
    }
    if (n0 + c < N)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (e0 + i >= r1 || m0 + e0 + i >= a.p.M) break;
        const int ad = ids[e0 + i];
        float y = v[i];
        if (ad >= 0) y += a.scaled ? scale_of(a.one, a.each, ad) * t[i] : t[i];
        a.out[(m0 + e0 + i) * N + n0 + c] = y + bias;
      }
  }
  cluster_sync_all();           // no CTA leaves while another reads its sums
}

// ------------------------------------------------------------------ gradients of the adapters
// out_a(j, k) = f_a sum over its rows T[i][j] S[i][k]: a CTA has 32 columns and 16 of the j of one adapter, its
// eight warps every eighth row, four at a time, asked for a round ahead; their T passes through shared memory.  Every
// 1024 rows a thread adds its sums, of 128 rows then, to those before.  Both stacks in one launch; zeros for an adapter
// without rows.  Latency: 9.7 us for 300 rows of three adapters, 512 and 1376 columns; with the pass for g 28.6 us for
// 1000 of four, 2048 and 2048 (T by uniform loads and nothing ahead: 31 more).  The rows of one adapter are not shared
// by CTAs: few adapters with many rows are slow (with the pass for g: 8192 rows of one, 4096 and 4096 columns, rank 64:
// 960 us; of four, 1024 and 1024, rank 16: 94).
constexpr int kShareRows = 1024;
struct F32Reduce {
  MultiPlan p;
  int r;
  int64_t K[2];                   // columns of S: dA (out [r, K]) and dB (out [K, r], times s_a)
  const float *S[2], *T[2];
  float* out[2];
  float one;
  const float* each;
  int blocks0;                    // column blocks of the first
  bool early;                     // see PdlEarly
};

__global__ void __launch_bounds__(256) f32_reduce_kernel(const __grid_constant__ F32Reduce a) {
  __shared__ float red[8][16][33];
  __shared__ __align__(16) float ts[2][32][16];        // T of 32 rows, zeros past the last row and j
  const PdlEarly order(a.early, blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1);
  const int which = (int)blockIdx.x >= a.blocks0, ad = blockIdx.y, j0 = blockIdx.z * 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = a.r;
  const int64_t K = a.K[which], k0 = (int64_t)((int)blockIdx.x - (which ? a.blocks0 : 0)) * 32, k = k0 + lane;
  const float *S = a.S[which], *T = a.T[which];
  const int first = a.p.start[ad], last = a.p.start[ad + 1];
  const int tr = threadIdx.x >> 3, tj = (threadIdx.x & 7) * 2;       // the row and the two j of T that a thread brings
  int64_t row[4], trow;                                // of the 32 rows that are loaded next
  float x[4], t[2];
  auto rows = [&](int i0) {
#pragma unroll
    for (int q = 0; q < 4; ++q) row[q] = i0 + warp + 8 * q < last ? a.p.order[i0 + warp + 8 * q] : -1;
    trow = i0 + tr < last ? a.p.order[i0 + tr] : -1;
  };
  auto load = [&] {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = row[q] >= 0 && k < K ? __ldg(S + row[q] * K + k) : 0.f;
#pragma unroll
    for (int q = 0; q < 2; ++q) t[q] = trow >= 0 && j0 + tj + q < r ? __ldg(T + trow * r + j0 + tj + q) : 0.f;
  };
  float acc[16] = {};
  rows(first);
  load();
  rows(first + 32);
  int i0 = first, flip = 0;
  do {
    const int end = min(last, i0 + kShareRows);
    const bool more = i0 > first;
#pragma unroll 2
    for (; i0 < end; i0 += 32, flip ^= 1) {
      *reinterpret_cast<float2*>(&ts[flip][tr][tj]) = make_float2(t[0], t[1]);
      float now[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) now[q] = x[q];
      __syncthreads();          // T is there, and all are done with the half that is written next
      load();
      rows(i0 + 64);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 u = *reinterpret_cast<const float4*>(&ts[flip][warp + 8 * q][j]);
          acc[j] = fmaf(u.x, now[q], acc[j]);
          acc[j + 1] = fmaf(u.y, now[q], acc[j + 1]);
          acc[j + 2] = fmaf(u.z, now[q], acc[j + 2]);
          acc[j + 3] = fmaf(u.w, now[q], acc[j + 3]);
        }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) {                     // a thread meets its own places alone
      red[warp][j][lane] = more ? red[warp][j][lane] + acc[j] : acc[j];
      acc[j] = 0.f;
    }
  } while (i0 < last);
  __syncthreads();
  // without rows the gradient is zero, whatever the slot's scale
  const float f = which && first < last ? scale_of(a.one, a.each, ad) : 1.f;
  float* out = a.out[which] + (int64_t)ad * r * K;
  for (int i = threadIdx.x; i < 512; i += 256) {
    // neighbouring threads write neighbouring elements: columns of dA, j of dB
    const int c = which ? i >> 4 : i & 31, j = which ? i & 15 : i >> 5;
    if (k0 + c >= K || j0 + j >= r) continue;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += red[w][j][c];
    out[which ? (k0 + c) * r + j0 + j : (int64_t)(j0 + j) * K + k0 + c] = s * f;
  }
}

// sums of all rows, 32 columns a cluster, whose CTAs have a stretch of the rows each and their warps every eighth of it;
// added up through distributed shared memory, in the order of the ranks.  1000 x 2048: 9 us, 36 by one CTA for all rows.
__global__ void __launch_bounds__(256) f32_colsum_kernel(int64_t M, int64_t K, const float* S, float* out) {
  __shared__ float red[8][32];
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const PdlEarly order(true, blockIdx.x == gridDim.x - 1);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k = (int64_t)(blockIdx.x / ranks) * 32 + lane, m0 = M * rank / ranks, m1 = M * (rank + 1) / ranks;
  float total = 0.f;
  for (int64_t b = m0 + warp; b < m1; b += 8 * 256) {
    float t = 0.f;
#pragma unroll 8
    for (int64_t m = b; m < min(m1, b + 8 * 256); m += 8)
      if (k < K) t += __ldg(S + m * K + k);
    total += t;
  }
  red[warp][lane] = total;
  __syncthreads();
  if (warp == 0) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) t += red[w][lane];
    red[0][lane] = t;         // read by this warp alone until the cluster meets
  }
  cluster_sync_all();
  if (warp == 0 && rank == 0 && k < K) {
    float t = 0.f;
    for (uint32_t q = 0; q < ranks; ++q) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&red[0][lane]), q)));
      t += v;
    }
    out[k] = t;
  }
  cluster_sync_all();         // no CTA leaves while another reads its sums
}

unsigned blocks(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }

template <bool MN>
cudaError_t gemm(F32Gemm a, cudaStream_t st) {
  const int64_t tiles = (int64_t)blocks(a.N, kTileN) * blocks(a.p.M, kTileM), slabs = blocks(a.K, kSlab),
                sms = num_sms_current();
  const cudaError_t allowed = allow_smem<f32_gemm_kernel<MN>>(kGemmSmem);
  if (allowed != cudaSuccess) return allowed;
  // the share of K that finishes soonest: what the fullest SM has, by how busy so many CTAs keep it (1 CTA 0.3 of
  // four's rate, 2 0.55, 3 0.75), and what a cluster costs.  Measured, us with 1 to 8 shares and what this takes: 300
  // x 512 -> 1376 74 41 36 29 28 39 38 36: 4; 509 x 1000 -> 1496 140 81 62 75 73 76 79 76: 3; 256 x 4096 -> 1024 362
  // 239 166 125 114 99 88 87: 7; 1000 x 2048 -> 2048 264 234 263 249 263 261 275 265: 5; 700 x 768 -> 3000 109 100
  // 115 112 123 124 134 132: 2; 1 x 4096 -> 4096 163 86 96 80 84 74 80 72: 7.  Backward, furthest from the best: 509
  // x 1000 -> 1496 140 107 85 66 87 84 82 77: 7.
  int ranks = 1;
  double best = 0;
  for (int s = 1; s <= 8; ++s) {
    if (s > 1 && slabs < 8 * s) break;
    const int64_t n = (tiles * s + sms - 1) / sms;
    const double t = (double)n / s / (n == 1 ? 0.3 : n == 2 ? 0.55 : n == 3 ? 0.75 : 0.9) + 0.02 * (s - 1);
    if (s == 1 || t < best) best = t, ranks = s;
  }
  a.ahead = tiles * ranks <= 2 * sms;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(tiles * ranks), 1, 1);
  cfg.blockDim = dim3(kGemmThreads, 1, 1);
  cfg.dynamicSmemBytes = kGemmSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + pdl_attr(&attr[1]);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, f32_gemm_kernel<MN>, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t multi_f32_proj(const MultiPlan& p, int64_t K, int r, const float* S, const float* U, bool kr, float one,
                           const float* each, float* plain, float* scaled, cudaStream_t st) {
  const F32Proj a{p, K, r, S, U, one, each, plain, scaled};
  const int64_t n = multi_items(p.M, p.n) * (kItemRows / kRows), slots = 3 * num_sms_current();
  int ranks = 1;                // shares of at least 128 columns, while there is room for their CTAs
  while (ranks < 8 && n * ranks * 2 <= slots && K >= ranks * 2 * 128) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(n * ranks), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + pdl_attr(&attr[1]);
  const cudaError_t e = kr ? cudaLaunchKernelEx(&cfg, f32_proj_kernel<true>, a)
                           : cudaLaunchKernelEx(&cfg, f32_proj_kernel<false>, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t multi_f32_gemm(const MultiPlan& p, int64_t N, int64_t K, int r, const float* S, const float* W, bool mn,
                           const float* P, const float* U, const float* bias, bool scaled, float one, const float* each,
                           float* out, cudaStream_t st) {
  const F32Gemm a{p, N, K, r, S, W, P, U, bias, one, each, scaled, out, false};
  return mn ? gemm<true>(a, st) : gemm<false>(a, st);
}

cudaError_t multi_f32_reduce(const MultiPlan& p, int r, int64_t in, const float* X, const float* G, float* dA, int64_t out,
                             const float* dY, const float* Z, float* dB, float one, const float* each, bool early,
                             cudaStream_t st) {
  const int b0 = (int)blocks(in, 32);
  const F32Reduce a{p, r, {in, out}, {X, dY}, {G, Z}, {dA, dB}, one, each, b0, early};
  return launch_pdl(f32_reduce_kernel, dim3(b0 + blocks(out, 32), (unsigned)p.n, blocks(r, 16)), dim3(256), 0, st, a);
}

cudaError_t multi_f32_colsum(int64_t M, int64_t K, const float* S, float* out, cudaStream_t st) {
  const int64_t columns = blocks(K, 32);
  int ranks = 1;                // stretches of at least 64 rows, while there is room for their CTAs
  while (ranks < 8 && M >= ranks * 2 * 64 && columns * ranks * 2 <= 4 * num_sms_current()) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(columns * ranks), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + pdl_attr(&attr[1]);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, f32_colsum_kernel, M, K, S, out);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace lg
