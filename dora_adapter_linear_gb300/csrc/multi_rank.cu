// Rank-r passes of the many-adapter projection, bf16: products of each row with its own adapter's factor, and
// the sums over each adapter's rows that are its gradients.  Warp MMAs, fp32 sums; rows are gathered through
// the plan's order, so any order of the batch costs the same.  Bound by memory: every element of a large
// operand is read once and takes part in 2 r operations.
#include "common.cuh"
#include "multi.h"

namespace lg {

namespace {

// ------------------------------------------------------------------ products of rows
// T = S U_a^T of one item (64 rows of one adapter), R columns of U_a [r, K], or (KR) [K, r].  The CTAs of a cluster
// share K and add their sums through distributed shared memory, in the order of the ranks, so that few items
// still fill the device; 64 rows to a CTA halve the reads of U_a through L2 against 32.  Stages of 128 columns by
// 16-byte asynchronous copies, three ahead of the one in use; a warp has 32 of the rows and every fourth pair of
// k16 steps.  8192 x 4096, rank 16: 20 us, 3.4 TB/s; [K, r] 8192 x 11008, rank 32: 42 us, 4.3 TB/s; small passes wait for
// the first two stages (3001 x 2568, rank 24: 12.5 us).  The form without shared memory, each warp feeding its MMAs from
// registers so that the product could begin beside it, waited for U_a at every block: 41 and 118 us.
template <int R, bool KR>
struct Proj {
  static constexpr int NT = R / 8;
  static constexpr int XP = 256 + 16, UP = KR ? 2 * R + 16 : 256 + 16;   // bytes of a row, in different banks
  static constexpr int STAGE = kItemRows * XP + (KR ? 128 : R) * UP;
  static constexpr int NST = 4 * STAGE <= 112 * 1024 ? 4 : 3;
  static constexpr int RED = 4 * kItemRows * R * 4;                      // the warps' sums
  static constexpr int RING = NST * STAGE > RED ? NST * STAGE : RED;
  static constexpr int SMEM = RING + kItemRows * 4;
};

struct ProjArgs {
  MultiPlan p;
  int64_t K;
  const bf16 *S, *U;
  float one;
  const float* each;
  bf16 *plain, *scaled, *rest;   // [M, r] T, s_a T and what its rounding leaves; each may be null
  int r, j0;                     // the rank, and the first of the R columns
};

template <int R, bool KR>
__global__ void __launch_bounds__(256) multi_proj_mma(const __grid_constant__ ProjArgs a) {
  using C = Proj<R, KR>;
  constexpr int NT = C::NT;
  extern __shared__ __align__(16) uint8_t smem[];
  int32_t* rows = reinterpret_cast<int32_t*>(smem + C::RING);
  uint32_t rank, ranks;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int mine = (int)(blockIdx.x / ranks);
  pdl_wait();
  if (tid == 0) pdl_trigger();
  const int4 item = a.p.items[mine];               // there is room for as many as there are CTAs
  const int items = a.p.head[kHeadItems], with = a.p.head[kHeadRows];
  if (a.plain) {              // rows without adapter: zeros
    for (int64_t i = (int64_t)blockIdx.x * 256 + tid; i < (a.p.M - with) * NT; i += (int64_t)gridDim.x * 256)
      *reinterpret_cast<uint4*>(a.plain + (int64_t)a.p.order[with + i / NT] * a.r + a.j0 + i % NT * 8) =
          make_uint4(0, 0, 0, 0);
  }
  if (mine >= items) return;  // the whole cluster
  const int64_t K = a.K;
  const bf16* U = a.U + (int64_t)item.x * a.r * K + (KR ? a.j0 : a.j0 * K);
  if (tid < kItemRows) rows[tid] = a.p.order[item.y + min(tid, item.z - 1)];   // past its end its last row, not used
  __syncthreads();
  const int steps = (int)((K + 127) / 128), s0 = (int)((int64_t)steps * rank / ranks),
            s1 = (int)((int64_t)steps * (rank + 1) / ranks);
  const int c = tid & 15, r0 = tid >> 4;           // 16 threads a row of 128 columns
  const bf16* x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = a.S + (int64_t)rows[r0 + 16 * i] * K + c * 8;
  auto load = [&](int s) {
    if (s < s1) {
      uint8_t* st = smem + (s - s0) % C::NST * C::STAGE;
      const int64_t k0 = (int64_t)s * 128;
      const bool on = k0 + c * 8 < K;
#pragma unroll
      for (int i = 0; i < 4; ++i) cp_async16(st + (r0 + 16 * i) * C::XP + c * 16, on ? x[i] + k0 : a.S, on);
      st += kItemRows * C::XP;
      if (KR) {
        for (int i = tid; i < 128 * NT; i += 256) {
          const int k = i / NT, q = i % NT;
          const bool in = k0 + k < K;
          cp_async16(st + k * C::UP + q * 16, in ? U + (k0 + k) * a.r + q * 8 : a.U, in);
        }
      } else {
#pragma unroll
        for (int j = 0; j < R; j += 16)
          if (j + r0 < R) cp_async16(st + (j + r0) * C::UP + c * 16, on ? U + (int64_t)(j + r0) * K + k0 + c * 8 : a.U, on);
      }
    }
    cp_async_commit();
  };
  const int mh = warp & 1, kq = warp >> 1;
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
#pragma unroll
  for (int s = 0; s < C::NST - 1; ++s) load(s0 + s);
  for (int s = s0; s < s1; ++s) {
    cp_async_wait<C::NST - 2>();
    __syncthreads();          // stage s is there, and all are done with the one that is loaded next
    load(s + C::NST - 1);
    const uint32_t X = smem_u32(smem + (s - s0) % C::NST * C::STAGE), W = X + kItemRows * C::XP;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kk = kq * 2 + h;
      uint32_t f[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
        ldsm_x4(f[m][0], f[m][1], f[m][2], f[m][3],
                X + (mh * 32 + m * 16 + (lane & 15)) * C::XP + (kk * 2 + (lane >> 4)) * 16);
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t b0, b1, b2 = 0, b3 = 0;
        if (KR) {
          const uint32_t at = W + (kk * 16 + (lane & 15)) * C::UP + n * 16;
          if (n + 1 < NT) ldsm_x4_t(b0, b1, b2, b3, at + (lane >> 4) * 16);
          else ldsm_x2_t(b0, b1, at);
        } else {
          const uint32_t at = W + (n * 8 + (lane & 7)) * C::UP + (kk * 2 + ((lane >> 3) & 1)) * 16;
          if (n + 1 < NT) ldsm_x4(b0, b1, b2, b3, at + (lane >> 4) * 8 * C::UP);
          else ldsm_x2(b0, b1, at);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          mma_bf16_16816(acc[m][n], f[m], b0, b1);
          if (n + 1 < NT) mma_bf16_16816(acc[m][n + 1 < NT ? n + 1 : n], f[m], b2, b3);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();            // the sums go where the stages were: [4][64][R]
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(red + (kq * kItemRows + mh * 32 + m * 16 + g + 8 * h) * R + n * 8 + 2 * t) =
            make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
  __syncthreads();
  if (ranks > 1) {            // this CTA's sums into the first quarter
    for (int i = tid; i < kItemRows * R / 2; i += 256) {
      float2 v = *reinterpret_cast<const float2*>(red + 2 * i);
#pragma unroll
      for (int w = 1; w < 4; ++w) {
        const float2 q = *reinterpret_cast<const float2*>(red + w * kItemRows * R + 2 * i);
        v.x += q.x;
        v.y += q.y;
      }
      *reinterpret_cast<float2*>(red + 2 * i) = v;
    }
    cluster_sync_all();
  }
  const float s = a.each ? __ldg(a.each + item.x) : a.one;
  const int pairs = item.z * R / 2, p0 = (int)((int64_t)pairs * rank / ranks),
            p1 = (int)((int64_t)pairs * (rank + 1) / ranks);
  for (int i = p0 + tid; i < p1; i += 256) {
    float2 q[8];
    if (ranks > 1) {
#pragma unroll
      for (uint32_t w = 0; w < 8; ++w)
        if (w < ranks)
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                       : "=f"(q[w].x), "=f"(q[w].y)
                       : "r"(mapa_shared(smem_u32(red + 2 * i), w)));
        else q[w] = make_float2(0.f, 0.f);
    } else {
#pragma unroll
      for (int w = 0; w < 8; ++w)
        q[w] = w < 4 ? *reinterpret_cast<const float2*>(red + w * kItemRows * R + 2 * i) : make_float2(0.f, 0.f);
    }
    float2 v = q[0];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      v.x += q[w].x;
      v.y += q[w].y;
    }
    const int64_t to = (int64_t)rows[2 * i / R] * a.r + a.j0 + 2 * i % R;
    if (a.plain) *reinterpret_cast<uint32_t*>(a.plain + to) = pack_bf16x2(v.x, v.y);
    uint32_t hi, lo;
    split_bf16x2(v.x * s, v.y * s, hi, lo);
    if (a.scaled) *reinterpret_cast<uint32_t*>(a.scaled + to) = hi;
    if (a.rest) *reinterpret_cast<uint32_t*>(a.rest + to) = lo;
  }
  if (ranks > 1) cluster_sync_all();   // no CTA leaves while another reads its sums
}

// ------------------------------------------------------------------ sums over an adapter's rows
// out[k][j] = f_a sum over the piece's rows S[row][k] T[row][j], of 128 columns k a CTA (a warp 32 of them).  Stages
// of 32 rows, gathered by 16-byte asynchronous copies; both factors are turned by ldmatrix.  Beside a product that fills
// the device two stages are enough, and fit what the product leaves of shared memory: training 8192 x 11008 took 535 us with
// the sums of dB in front of the product and 512 with both behind it; alone, four are faster (1999 x 2568: 38 us the
// whole backward, 43 with two).  8192 x 11008, rank 32, alone: 46 us, 3.9 TB/s.  An adapter's only
// piece gives the gradient itself, others fp32 partials, added by multi_sum in their order.
template <int R, bool TWO>
struct Reduce {
  static constexpr int NT = R / 8, PARTS = TWO ? 2 : 1;
  static constexpr int SP = 256 + 16, TP = 2 * R + 16;
  static constexpr int STAGE = 32 * (SP + PARTS * TP);
  static constexpr int NST = STAGE <= 14 * 1024 ? 4 : 3;     // stages, or two
  static constexpr int smem(int stages) { return stages * STAGE + kPieceRows * 4; }
};

struct ReduceArgs {
  MultiPlan p;
  int64_t K;
  const bf16 *S, *T, *T2;     // T2: what a rounding has left of T, added to it (TWO)
  float one;
  const float* each;          // with scaled: f_a = s_a
  bool scaled, kr;            // kr: out_a [K, R], else [R, K]
  bf16* out;
  float* part;                // [partials] x [K, R] or [R, K]
  bool early;                 // see PdlEarly
  int stages;                 // NST, or two
};

template <int R, bool TWO>
__global__ void __launch_bounds__(128) multi_reduce_mma(const __grid_constant__ ReduceArgs a) {
  using C = Reduce<R, TWO>;
  constexpr int NT = C::NT;
  extern __shared__ __align__(16) uint8_t smem[];
  const int nst = a.stages;
  int32_t* rows = reinterpret_cast<int32_t*>(smem + nst * C::STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t K = a.K;
  const int groups = (int)((K + 127) / 128);
  const PdlEarly order(a.early, blockIdx.x == gridDim.x - 1);
  const int mine = (int)blockIdx.x / groups, group = (int)blockIdx.x - mine * groups;
  const int4 piece = a.p.pieces[mine];             // there is room for as many as the grid has
  if (mine >= a.p.head[kHeadPieces]) return;
  const int64_t k0 = (int64_t)group * 128;
  for (int i = threadIdx.x; i < piece.z; i += 128) rows[i] = a.p.order[piece.y + i];
  __syncthreads();
  const int stages = (piece.z + 31) / 32;
  const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;     // 16 threads a row of S
  const bool in = k0 + c * 8 < K;
  auto load = [&](int s, int at_stage) {
    if (s < stages) {
      uint8_t* st = smem + at_stage * C::STAGE;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 8 * i;
        const bool on = in && s * 32 + r < piece.z;
        cp_async16(st + r * C::SP + c * 16, on ? a.S + (int64_t)rows[s * 32 + r] * K + k0 + c * 8 : a.S, on);
      }
      for (int i = threadIdx.x; i < 32 * NT; i += 128) {
        const int r = i / NT, q = i % NT;
        const bool on = s * 32 + r < piece.z;
        const int64_t at = on ? (int64_t)rows[s * 32 + r] * R + q * 8 : 0;
        cp_async16(st + 32 * C::SP + r * C::TP + q * 16, a.T + at, on);
        if (TWO) cp_async16(st + 32 * (C::SP + C::TP) + r * C::TP + q * 16, a.T2 + at, on);
      }
    }
    cp_async_commit();
  };
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
  for (int s = 0; s < nst - 1; ++s) load(s, s);
  for (int s = 0, now = 0; s < stages; ++s) {
    if (nst == 2) cp_async_wait<0>();
    else cp_async_wait<C::NST - 2>();
    __syncthreads();          // stage s is there, and all are done with the one that is loaded next
    load(s + nst - 1, now == 0 ? nst - 1 : now - 1);
    const uint32_t S = smem_u32(smem + now * C::STAGE), T = S + 32 * C::SP;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint32_t x[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
        ldsm_x4_t(x[m][0], x[m][1], x[m][2], x[m][3],
                  S + (kk * 16 + (lane & 7) + ((lane >> 4) << 3)) * C::SP +
                      (warp * 32 + m * 16 + ((lane >> 3) & 1) * 8) * 2);
#pragma unroll
      for (int w = 0; w < C::PARTS; ++w) {
        if (w == 1)
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[m][i] = finite_bf16x2(x[m][i]);
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          const uint32_t at = T + w * 32 * C::TP + (kk * 16 + (lane & 15)) * C::TP + n * 16;
          uint32_t b0, b1, b2 = 0, b3 = 0;
          if (n + 1 < NT) ldsm_x4_t(b0, b1, b2, b3, at + (lane >> 4) * 16);
          else ldsm_x2_t(b0, b1, at);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma_bf16_16816(acc[m][n], x[m], b0, b1);
            if (n + 1 < NT) mma_bf16_16816(acc[m][n + 1 < NT ? n + 1 : n], x[m], b2, b3);
          }
        }
      }
    }
    if (++now == nst) now = 0;
  }
  cp_async_wait<0>();
  const float f = !a.scaled ? 1.f : a.each ? __ldg(a.each + piece.x) : a.one;
  const bool whole = piece.w < 0;
  bf16* out = a.out + (int64_t)piece.x * R * K;
  float* part = a.part + (int64_t)(whole ? 0 : piece.w) * R * K;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = k0 + warp * 32 + m * 16 + g + 8 * h;
        const int j = n * 8 + 2 * t;
        if (k >= K) continue;
        const float v0 = acc[m][n][2 * h] * f, v1 = acc[m][n][2 * h + 1] * f;
        if (a.kr) {
          if (whole) *reinterpret_cast<uint32_t*>(out + k * R + j) = pack_bf16x2(v0, v1);
          else *reinterpret_cast<float2*>(part + k * R + j) = make_float2(v0, v1);
        } else if (whole) {
          out[(int64_t)j * K + k] = __float2bfloat16_rn(v0);
          out[(int64_t)(j + 1) * K + k] = __float2bfloat16_rn(v1);
        } else {
          part[(int64_t)j * K + k] = v0;
          part[(int64_t)(j + 1) * K + k] = v1;
        }
      }
}

// The gradients of adapters with several pieces, and zeros for those without rows; eight elements a thread.
// Both of a backward's stacks in one launch, and the column sums of dY.  9 us for eight adapters of 8192 rows, rank 32,
// d_in 4096, d_out 11008 (37 MB of partials and results), 5 us where there are none: latency.
struct SumArgs {
  MultiPlan p;
  int64_t size[2];            // elements of one adapter
  const float* part[2];
  bf16* out[2];
  int splits;                 // of the column sums; 0: none
  int64_t K;
  const float* csum;
  bf16* sums;
};
__global__ void __launch_bounds__(256) multi_sum_kernel(const __grid_constant__ SumArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int ad = blockIdx.y, which = blockIdx.z;
  if (ad == 0 && which == 0 && a.splits)
    for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < a.K; k += (int64_t)gridDim.x * 256) {
      float t = 0.f;
#pragma unroll 8
      for (int s = 0; s < a.splits; ++s) t += a.csum[s * a.K + k];
      a.sums[k] = __float2bfloat16_rn(t);
    }
  const int first = a.p.pstart[ad], count = a.p.pstart[ad + 1] - first;
  if (count == 1) return;
  const int64_t size = a.size[which];
  const int slot = count ? a.p.pieces[first].w : 0;
  bf16* out = a.out[which] + ad * size;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < size; i += (int64_t)gridDim.x * 2048) {
    float v[8] = {};
    const float* p = a.part[which] + slot * size + i;
    for (int k = 0; k < count; ++k, p += size) {
      const float4 lo = *reinterpret_cast<const float4*>(p), hi = *reinterpret_cast<const float4*>(p + 4);
      v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w;
      v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
    }
    *reinterpret_cast<uint4*>(out + i) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                    pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// column sums of 64 columns and one split of the rows a CTA: part [splits, K].  1999 x 2568: 8.5 us alone, most of it
// behind the product.
__global__ void __launch_bounds__(256) multi_colsum_kernel(int64_t M, int64_t K, int rows, const bf16* S, float* part) {
  __shared__ float red[32][64];
  const PdlEarly order(true, blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1);
  const int c = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const int64_t k = (int64_t)blockIdx.x * 64 + c * 8, m1 = min(M, (int64_t)(blockIdx.y + 1) * rows);
  float v[8] = {};
  if (k < K)
#pragma unroll 4
    for (int64_t m = (int64_t)blockIdx.y * rows + r0; m < m1; m += 32) {
      const uint4 x = __ldcs(reinterpret_cast<const uint4*>(S + m * K + k));
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack_bf16x2(w[i]);
        v[2 * i] += f.x;
        v[2 * i + 1] += f.y;
      }
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[r0][c * 8 + i] = v[i];
  __syncthreads();
  if (threadIdx.x < 64 && (int64_t)blockIdx.x * 64 + threadIdx.x < K) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += red[i][threadIdx.x];
    part[blockIdx.y * K + blockIdx.x * 64 + threadIdx.x] = t;
  }
}

// Rows of an odd multiple of 16 bytes slow the product's copies by a third (each 128 bytes of them lie across two lines),
// so a product that reads them often enough takes copies in rows of whole lines, made beside the pass before it.
struct PadArgs {
  const bf16* from[2];
  bf16* to[2];
  int64_t rows[2], K[2], ld[2];
};
__global__ void __launch_bounds__(256) multi_pad_kernel(const __grid_constant__ PadArgs a) {
  const PdlEarly order(true, blockIdx.x == gridDim.x - 1);
  const int lane = threadIdx.x & 31, warps = (int)gridDim.x * 8;
#pragma unroll
  for (int w = 0; w < 2; ++w)
    for (int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); row < a.rows[w]; row += warps) {   // a warp a row
      const uint4* from = reinterpret_cast<const uint4*>(a.from[w] + row * a.K[w]);
      uint4* to = reinterpret_cast<uint4*>(a.to[w] + row * a.ld[w]);
      const int all = (int)(a.K[w] / 8);
      for (int c = lane; c < all; c += 256) {
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (c + 32 * q < all) v[q] = __ldg(from + c + 32 * q);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (c + 32 * q < all) to[c + 32 * q] = v[q];
      }
    }
}

// as many CTAs to a cluster as two an SM have room for (about half of the adapters end in a part of an item).  Before
// a product that needs all multiprocessors a CTA has four stages at least, before a smaller one six: that one begins
// on multiprocessors that have none of these CTAs.  Whole calls with four and with six, us (adapters' rows behind one
// another):
//   smaller: 600 x 4096 -> 4096 33.0, 28.7, backward 40.4, 39.3; 1000 rows 33.2, 33.6, 42.4, 41.6; 1999 x 2568 -> 1000
//     28.9, 30.0; backward of 1999 x 1000 -> 2568 34.8, 36.7 (another batch 41.7, 37.7)
//   all: 2048 x 4096 -> 4096 55.8, 56.4, backward 65.1, 64.8; 3001 x 2568 -> 2568 57.0, 54.6, 70.0, 68.1 (another batch
//     61.2, 62.9); 4000 x 2048 -> 4096 59.9, 54.2, 68.8, 68.9; 3001 x 4096 and 1500 x 11008 -> 4096 the same
// It is a matter of a tenth either way, and of the batch.
template <int R, bool KR>
int proj_ranks(const MultiPlan& p, int64_t K, bool all) {
  const int64_t steps = (K + 127) / 128, slots = 2 * num_sms_current(), items = p.M / kItemRows + (p.n + 1) / 2;
  int ranks = 1;
  while (ranks < 8 && items * ranks * 2 <= slots && steps >= ranks * 2 * (all ? 4 : 6)) ranks *= 2;
  return ranks;
}
template <int R, bool KR>
cudaError_t proj_launch(const ProjArgs& a, int64_t items, bool all, cudaStream_t st) {
  using C = Proj<R, KR>;
  const cudaError_t e = allow_smem<multi_proj_mma<R, KR>>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int ranks = proj_ranks<R, KR>(a.p, a.K, all);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(items * ranks), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1 + pdl_attr(&attr[1]);
  const cudaError_t l = cudaLaunchKernelEx(&cfg, multi_proj_mma<R, KR>, a);
  count_launch();
  return l != cudaSuccess ? l : cudaGetLastError();
}
template <int R, bool TWO>
cudaError_t reduce_launch(ReduceArgs a, int64_t pieces, cudaStream_t st) {
  using C = Reduce<R, TWO>;
  const cudaError_t e = allow_smem<multi_reduce_mma<R, TWO>>(C::smem(C::NST));
  if (e != cudaSuccess) return e;
  if (a.stages == 0) a.stages = C::NST;
  return launch_pdl(multi_reduce_mma<R, TWO>, dim3((unsigned)((a.K + 127) / 128 * pieces)), dim3(128), C::smem(a.stages),
                    st, a);
}

}  // namespace

#define RANKS(CASE) CASE(8) CASE(16) CASE(24) CASE(32) CASE(40) CASE(48) CASE(56) CASE(64)
#define MORE_RANKS(CASE) CASE(72) CASE(80) CASE(88) CASE(96) CASE(104) CASE(112) CASE(120) CASE(128)

cudaError_t multi_proj(const MultiPlan& p, int64_t K, int r, const bf16* S, const bf16* U, bool kr, float one,
                       const float* each, bf16* plain, bf16* scaled, bf16* rest, bool all,
                       cudaStream_t st) {
  const int64_t items = multi_items(p.M, p.n);
  for (int j0 = 0; j0 < r; j0 += 64) {   // ranks above 64 take a second pass: their sums do not fit the registers
    const ProjArgs a{p, K, S, U, one, each, plain, scaled, rest, r, j0};
    cudaError_t e = cudaErrorInvalidValue;
    switch (r - j0 < 64 ? r - j0 : 64) {
#define CASE(R) \
  case R: e = kr ? proj_launch<R, true>(a, items, all, st) : proj_launch<R, false>(a, items, all, st); break;
      RANKS(CASE)
#undef CASE
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t multi_reduce(const MultiPlan& p, int64_t K, int r, const bf16* S, const bf16* T, const bf16* T2, bool kr,
                         bool scaled, float one, const float* each, float* part, bf16* out, bool early, bool beside,
                         cudaStream_t st) {
  const int64_t pieces = multi_pieces(p.M, p.n);
  const ReduceArgs a{p, K, S, T, T2, one, each, scaled, kr, out, part, early, beside ? 2 : 0};
  switch (r) {
#define CASE(R) \
  case R: return T2 ? reduce_launch<R, true>(a, pieces, st) : reduce_launch<R, false>(a, pieces, st);
    RANKS(CASE)
    MORE_RANKS(CASE)
#undef CASE
  }
  return cudaErrorInvalidValue;
}

cudaError_t multi_sum(const MultiPlan& p, int64_t size0, const float* part0, bf16* out0, int64_t size1, const float* part1,
                      bf16* out1, int64_t K, const float* csum, bf16* sums, cudaStream_t st) {
  const SumArgs a{p, {size0, size1}, {part0, part1}, {out0, out1}, sums ? multi_colsum_splits(p.M) : 0, K, csum, sums};
  const int64_t most = size0 > size1 ? size0 : size1, blocks = (most + 2047) / 2048;
  return launch_pdl(multi_sum_kernel, dim3((unsigned)(blocks < 256 ? blocks : 256), (unsigned)p.n, 2), dim3(256), 0, st, a);
}

cudaError_t multi_pad(const MultiPad& S, const MultiPad& W, cudaStream_t st) {
  const PadArgs a{{S.from, W.from}, {S.to, W.to}, {S.to ? S.rows : 0, W.to ? W.rows : 0}, {S.K, W.K},
                  {multi_pad_ld(S.K), multi_pad_ld(W.K)}};
  return launch_pdl(multi_pad_kernel, dim3((unsigned)(2 * num_sms_current())), dim3(256), 0, st, a);
}

int multi_colsum_splits(int64_t M) {
  const int64_t n = (M + 255) / 256;
  return (int)(n < 64 ? n : 64);
}
cudaError_t multi_colsum(int64_t M, int64_t K, const bf16* S, float* part, cudaStream_t st) {
  const int splits = multi_colsum_splits(M), rows = (int)((M + splits - 1) / splits);
  return launch_pdl(multi_colsum_kernel, dim3((unsigned)((K + 63) / 64), (unsigned)splits), dim3(256), 0, st, M, K, rows, S,
                    part);
}

}  // namespace lg
