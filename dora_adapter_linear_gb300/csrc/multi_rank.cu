// Rank-r passes of the many-adapter projection, bf16: products of each row with its own adapter's factor, and
// the sums over each adapter's rows that are its gradients.  Warp MMAs, fp32 sums; rows are gathered through
// the plan's order, so any order of the batch costs the same.  Bound by memory: every element of a large
// operand is read once and takes part in 2 r operations.
#include "common.cuh"
#include "multi.h"

namespace lg {

namespace {

// ------------------------------------------------------------------ products of rows
// T = S U_a^T of one item (32 rows of one adapter), R columns of U_a [r, K], or (KR) [K, r].  The eight warps share K in
// stretches of 64 columns and add their sums at the end, in their order.  A lane reads 16 bytes of a row at a
// time: of 32 columns it holds 8 t .. 8 t + 7 (t = lane % 4), and as a sum over k may run in any order, its
// words go into the MMA operands as they are, for both factors alike.  U_a [K, R] is turned by ldmatrix: a warp
// stages 32 rows k at a time, row 8 t + 2 m + e of them as row 8 m + 2 t + e, which gives the same order.
template <int R, bool KR>
struct Proj {
  static constexpr int NT = R / 8;
  static constexpr int PITCH = 2 * R + 16;                     // bytes: eight rows of 16 bytes in different banks
  static constexpr int STAGE = KR ? 32 * PITCH : 0;
  static constexpr int SMEM = 8 * (2 * STAGE > 32 * R * 4 ? 2 * STAGE : 32 * R * 4);
};

struct ProjArgs {
  MultiPlan p;
  int64_t K;
  const bf16 *S, *U;
  float one;
  const float* each;
  bf16 *plain, *scaled;       // [M, r] T and s_a T; either may be null
  int r, j0;                  // the rank, and the first of the R columns
};

template <int R, bool KR>
__global__ void __launch_bounds__(256) multi_proj_mma(const __grid_constant__ ProjArgs a) {
  using C = Proj<R, KR>;
  constexpr int NT = C::NT;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int items = a.p.head[kHeadItems], with = a.p.head[kHeadRows];
  if (a.plain) {              // rows without adapter: zeros
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (a.p.M - with) * NT; i += (int64_t)gridDim.x * 256)
      *reinterpret_cast<uint4*>(a.plain + (int64_t)a.p.order[with + i / NT] * a.r + a.j0 + i % NT * 8) = make_uint4(0, 0, 0, 0);
  }
  if ((int)blockIdx.x >= items) return;
  const int4 item = a.p.items[blockIdx.x];
  const bf16* U = a.U + (int64_t)item.x * a.r * a.K + (KR ? a.j0 : a.j0 * a.K);
  const bf16* row[4];         // rows g, g + 8, g + 16, g + 24 of the item; past its end its first row, not used
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = g + 8 * i;
    row[i] = a.S + (int64_t)a.p.order[item.y + (k < item.z ? k : 0)] * a.K;
  }
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;

  const int64_t K = a.K;
  const int halves = (int)((K + 31) / 32);                     // stretches of 32 columns; a warp takes two of 16
  const uint4 none = make_uint4(0, 0, 0, 0);
  auto load_rows = [&](int h, uint4 (&x)[4]) {
    const int64_t k = (int64_t)h * 32 + 8 * t;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = k < K ? __ldcs(reinterpret_cast<const uint4*>(row[i] + k)) : none;
  };
  auto mma = [&](const uint4 (&x)[4], int n, uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint32_t lo[4] = {x[2 * m].x, x[2 * m + 1].x, x[2 * m].y, x[2 * m + 1].y};
      const uint32_t hi[4] = {x[2 * m].z, x[2 * m + 1].z, x[2 * m].w, x[2 * m + 1].w};
      mma_bf16_16816(acc[m][n], lo, b0, b1);
      mma_bf16_16816(acc[m][n], hi, b2, b3);
    }
  };
  uint8_t* mine = smem + warp * 2 * C::STAGE;
  auto stage = [&](int h, int buf) {                           // 32 rows of U_a [K, R]; zeros past K
    if (h < halves)
      for (int i = lane; i < 32 * NT; i += 32) {
        const int k = i / NT, c = i % NT, at = 8 * ((k & 7) >> 1) + 2 * (k >> 3) + (k & 1);
        const int64_t kk = (int64_t)h * 32 + k;
        cp_async16(mine + buf * C::STAGE + at * C::PITCH + c * 16, U + (kk < K ? kk * a.r + c * 8 : 0), kk < K);
      }
    cp_async_commit();
  };
  auto work = [&](int h, int buf, const uint4 (&x)[4]) {
    if constexpr (KR) {
      const uint32_t base = smem_u32(mine + buf * C::STAGE) + lane * C::PITCH;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(b0, b1, b2, b3, base + n * 16);
        mma(x, n, b0, b1, b2, b3);
      }
    } else {
      const int64_t k = (int64_t)h * 32 + 8 * t;
#pragma unroll
      for (int n0 = 0; n0 < NT; n0 += 4) {
        uint4 u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < NT) u[i] = k < K ? __ldg(reinterpret_cast<const uint4*>(U + (int64_t)((n0 + i) * 8 + g) * K + k)) : none;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < NT) mma(x, n0 + i, u[i].x, u[i].y, u[i].z, u[i].w);
      }
    }
  };
  // stretch j of this warp: the j % 2 half of its 64-column run
  auto nth = [&](int j) { return (warp + (j >> 1) * 8) * 2 + (j & 1); };
  uint4 x0[4], x1[4];
  load_rows(nth(0), x0);
  load_rows(nth(1), x1);
  if (KR) {
    stage(nth(0), 0);
    stage(nth(1), 1);
  }
  for (int j = 0; nth(j) < halves; j += 2) {
    if (KR) {
      cp_async_wait<1>();
      __syncwarp();
    }
    work(nth(j), 0, x0);
    load_rows(nth(j + 2), x0);
    if (KR) {
      __syncwarp();
      stage(nth(j + 2), 0);
      cp_async_wait<1>();
      __syncwarp();
    }
    if (nth(j + 1) < halves) work(nth(j + 1), 1, x1);
    load_rows(nth(j + 3), x1);
    if (KR) {
      __syncwarp();
      stage(nth(j + 3), 1);
    }
  }
  if (KR) cp_async_wait<0>();
  __syncthreads();            // the sums go where the stages were
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(red + (warp * 32 + m * 16 + g + 8 * h) * R + n * 8 + 2 * t) =
            make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
  __syncthreads();
  const float s = a.each ? __ldg(a.each + item.x) : a.one;
  for (int i = threadIdx.x; i < item.z * R / 2; i += 256) {
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float2 q = *reinterpret_cast<const float2*>(red + w * 32 * R + 2 * i);
      v.x += q.x;
      v.y += q.y;
    }
    const int64_t to = (int64_t)a.p.order[item.y + 2 * i / R] * a.r + a.j0 + 2 * i % R;
    if (a.plain) *reinterpret_cast<uint32_t*>(a.plain + to) = pack_bf16x2(v.x, v.y);
    if (a.scaled) *reinterpret_cast<uint32_t*>(a.scaled + to) = pack_bf16x2(v.x * s, v.y * s);
  }
}

// ------------------------------------------------------------------ sums over an adapter's rows
// out[k][j] = f_a sum over the piece's rows S[row][k] T[row][j], of 128 columns k a CTA (a warp 32 of them).  Stages
// of 32 rows, gathered by 16-byte asynchronous copies; both factors are turned by ldmatrix.  An adapter's only
// piece gives the gradient itself, others fp32 partials, added by multi_sum in their order.
template <int R>
struct Reduce {
  static constexpr int NT = R / 8;
  static constexpr int SP = 256 + 16, TP = 2 * R + 16;
  static constexpr int STAGE = 32 * (SP + TP);
  static constexpr int NST = R <= 64 ? 4 : 3;
  static constexpr int SMEM = NST * STAGE;
};

struct ReduceArgs {
  MultiPlan p;
  int64_t K;
  const bf16 *S, *T;
  float one;
  const float* each;          // with scaled: f_a = s_a
  bool scaled, kr;            // kr: out_a [K, R], else [R, K]
  bf16* out;
  float* part;                // [partials] x [K, R] or [R, K]
};

template <int R>
__global__ void __launch_bounds__(128) multi_reduce_mma(const __grid_constant__ ReduceArgs a) {
  using C = Reduce<R>;
  constexpr int NT = C::NT;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int64_t K = a.K;
  const int groups = (int)((K + 127) / 128), mine = (int)blockIdx.x / groups;
  if (mine >= a.p.head[kHeadPieces]) return;
  const int4 piece = a.p.pieces[mine];
  const int64_t k0 = (int64_t)((int)blockIdx.x - mine * groups) * 128;
  const int32_t* order = a.p.order + piece.y;
  const int stages = (piece.z + 31) / 32;
  auto load = [&](int s) {
    if (s < stages) {
      uint8_t* st = smem + s % C::NST * C::STAGE;
      // 16 threads a row of S: rows threadIdx / 16 + 8 i
      const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = r0 + 8 * i;
        const bool on = s * 32 + r < piece.z && k0 + c * 8 < K;
        const int64_t row = on ? order[s * 32 + r] : 0;
        cp_async16(st + r * C::SP + c * 16, a.S + (on ? row * K + k0 + c * 8 : 0), on);
      }
      for (int i = threadIdx.x; i < 32 * NT; i += 128) {
        const int r = i / NT, q = i % NT;
        const bool on = s * 32 + r < piece.z;
        const int64_t row = on ? order[s * 32 + r] : 0;
        cp_async16(st + 32 * C::SP + r * C::TP + q * 16, a.T + row * R + q * 8, on);
      }
    }
    cp_async_commit();
  };
  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
#pragma unroll
  for (int s = 0; s < C::NST - 1; ++s) load(s);
  for (int s = 0; s < stages; ++s) {
    cp_async_wait<C::NST - 2>();
    __syncthreads();          // stage s is there, and all are done with the one that is loaded next
    load(s + C::NST - 1);
    const uint32_t S = smem_u32(smem + s % C::NST * C::STAGE), T = S + 32 * C::SP;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint32_t x[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
        ldsm_x4_t(x[m][0], x[m][1], x[m][2], x[m][3],
                  S + (kk * 16 + (lane & 7) + ((lane >> 4) << 3)) * C::SP + (warp * 32 + m * 16 + ((lane >> 3) & 1) * 8) * 2);
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        const uint32_t at = T + (kk * 16 + (lane & 15)) * C::TP + n * 16;
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
// Both of a backward's stacks in one launch.
struct SumArgs {
  MultiPlan p;
  int64_t size[2];            // elements of one adapter
  const float* part[2];
  bf16* out[2];
};
__global__ void __launch_bounds__(256) multi_sum_kernel(const __grid_constant__ SumArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int ad = blockIdx.y, which = blockIdx.z;
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

// column sums of 64 columns and one split of the rows a CTA: part [splits, K]
__global__ void __launch_bounds__(256) multi_colsum_kernel(int64_t M, int64_t K, int rows, const bf16* S, float* part) {
  __shared__ float red[32][64];
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
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

template <int R, bool KR>
cudaError_t proj_launch(const ProjArgs& a, int64_t ctas, cudaStream_t st) {
  using C = Proj<R, KR>;
  const cudaError_t e = allow_smem<multi_proj_mma<R, KR>>(C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(multi_proj_mma<R, KR>, dim3((unsigned)ctas), dim3(256), C::SMEM, st, a);
}
template <int R>
cudaError_t reduce_launch(const ReduceArgs& a, int64_t pieces, cudaStream_t st) {
  using C = Reduce<R>;
  const cudaError_t e = allow_smem<multi_reduce_mma<R>>(C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl(multi_reduce_mma<R>, dim3((unsigned)((a.K + 127) / 128 * pieces)), dim3(128), C::SMEM, st, a);
}

}  // namespace

#define RANKS(CASE) CASE(8) CASE(16) CASE(24) CASE(32) CASE(40) CASE(48) CASE(56) CASE(64)
#define MORE_RANKS(CASE) CASE(72) CASE(80) CASE(88) CASE(96) CASE(104) CASE(112) CASE(120) CASE(128)

cudaError_t multi_proj(const MultiPlan& p, int64_t K, int r, const bf16* S, const bf16* U, bool kr, float one,
                       const float* each, bf16* plain, bf16* scaled, cudaStream_t st) {
  // at least one CTA: with no row that has an adapter the others are still set to zero
  int64_t ctas = multi_items(p.M, p.n);
  if (ctas < 1) ctas = 1;
  for (int j0 = 0; j0 < r; j0 += 64) {   // ranks above 64 take a second pass: their sums do not fit the registers
    const ProjArgs a{p, K, S, U, one, each, plain, scaled, r, j0};
    cudaError_t e = cudaErrorInvalidValue;
    switch (r - j0 < 64 ? r - j0 : 64) {
#define CASE(R) \
  case R: e = kr ? proj_launch<R, true>(a, ctas, st) : proj_launch<R, false>(a, ctas, st); break;
      RANKS(CASE)
#undef CASE
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t multi_reduce(const MultiPlan& p, int64_t K, int r, const bf16* S, const bf16* T, bool kr, bool scaled,
                         float one, const float* each, float* part, bf16* out, cudaStream_t st) {
  const ReduceArgs a{p, K, S, T, one, each, scaled, kr, out, part};
  switch (r) {
#define CASE(R) \
  case R: return reduce_launch<R>(a, multi_pieces(p.M, p.n), st);
    RANKS(CASE) MORE_RANKS(CASE)
#undef CASE
  }
  return cudaErrorInvalidValue;
}

cudaError_t multi_sum(const MultiPlan& p, int64_t size0, const float* part0, bf16* out0, int64_t size1, const float* part1,
                      bf16* out1, cudaStream_t st) {
  const SumArgs a{p, {size0, size1}, {part0, part1}, {out0, out1}};
  const int64_t most = size0 > size1 ? size0 : size1, blocks = (most + 2047) / 2048;
  return launch_pdl(multi_sum_kernel, dim3((unsigned)(blocks < 256 ? blocks : 256), (unsigned)p.n, 2), dim3(256), 0, st, a);
}

int multi_colsum_splits(int64_t M) {
  const int64_t n = (M + 255) / 256;
  return (int)(n < 64 ? n : 64);
}
cudaError_t multi_colsum(int64_t M, int64_t K, const bf16* S, float* part, bf16* out, cudaStream_t st) {
  const int splits = multi_colsum_splits(M), rows = (int)((M + splits - 1) / splits);
  const cudaError_t e = launch_pdl(multi_colsum_kernel, dim3((unsigned)((K + 63) / 64), (unsigned)splits), dim3(256), 0, st,
                                   M, K, rows, S, part);
  return e != cudaSuccess ? e : sum_splits<bf16>(part, splits, K, nullptr, out, st);
}

}  // namespace lg
