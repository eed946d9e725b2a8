// Many adapters beside one projection: row i of a batch has adapter a = ids[i], or none.
//
//   forward   z_i = x_i A_a^T,  y_i = x_i W0^T + s_a z_i B_a^T (+ bias)
//   backward  g_i = s_a dy_i B_a,  dx_i = dy_i W0 + g_i A_a,
//             dA_a = sum over its rows g_i^T x_i,  dB_a = s_a sum dy_i^T z_i,  dbias = sum dy_i
//
// The plan (multi_plan.cu) gives the rows of each adapter.  A row meets no other adapter's numbers, so
// what is not finite in one adapter or row stays there.
#include <math.h>

#include "common.cuh"
#include "multi.h"

namespace lg {

namespace {

struct Scale {          // s_a: one number, or one for each adapter
  float one;
  const float* each;
  __device__ __forceinline__ float of(int a) const { return each ? __ldg(each + a) : one; }
};

// ------------------------------------------------------------------ rank-r products of rows
// P[i][j] = (scaled) sum_k S[i][k] U_a(j, k), U_a [r, K] or (KR) [K, r]; zeros for a row without adapter.  A
// warp takes every fourth j of its CTA's row.
template <typename T, bool KR>
__global__ void __launch_bounds__(128) multi_proj_kernel(MultiPlan p, int64_t K, int r, const T* S, const T* U, Scale s,
                                                         bool scaled, float* P, T* Z) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int64_t i = blockIdx.x;
  const int a = p.ids[i], lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* x = S + i * K;
  const T* u = U + (int64_t)max(a, 0) * r * K;
  const float f = a >= 0 && scaled ? s.of(a) : 1.f;
  for (int j = warp; j < r; j += 4) {
    float t = 0.f;
    if (a >= 0)
      for (int64_t k = lane; k < K; k += 32) t = fmaf(to_f(x[k]), to_f(KR ? u[k * r + j] : u[(int64_t)j * K + k]), t);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lane == 0) {
      if (P) P[i * r + j] = t * f;
      if (Z) Z[i * r + j] = from_f<T>(t);
    }
  }
}

// ------------------------------------------------------------------ shared product and rank-r update
// out[i][c] = sum_k S[i][k] W(c, k) + f_a sum_j P[i][j] U_a(c, j) + bias[c].  W [N, K] and U_a [N, r], or (MN)
// W [K, N] and U_a [r, N]; f_a = s_a when `scaled`, else 1.
template <typename T, bool MN>
__global__ void __launch_bounds__(256) multi_gemm_kernel(MultiPlan p, int64_t N, int64_t K, int r, const T* S, const T* W,
                                                         const float* P, const T* U, Scale s, bool scaled, const T* bias,
                                                         T* out) {
  constexpr int TT = 64, TK = 16;
  __shared__ float As[TK][TT + 4];
  __shared__ float Bs[TK][TT + 4];
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * TT, n0 = (int64_t)blockIdx.x * TT;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += TK) {
    for (int i = threadIdx.x; i < TT * TK; i += 256) {
      const int kk = i % TK, mm = i / TK;
      const int64_t m = m0 + mm, k = k0 + kk;
      As[kk][mm] = m < p.M && k < K ? to_f(S[m * K + k]) : 0.f;
    }
    for (int i = threadIdx.x; i < TT * TK; i += 256) {
      const int kk = MN ? i / TT : i % TK, nn = MN ? i % TT : i / TK;
      const int64_t c = n0 + nn, k = k0 + kk;
      Bs[kk][nn] = c < N && k < K ? to_f(MN ? W[k * N + c] : W[c * K + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < TK; ++kk) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = As[kk][ty * 4 + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = Bs[kk][tx * 4 + j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
    if (m >= p.M) continue;
    const int a = p.ids[m];
    const float f = a >= 0 && scaled ? s.of(a) : 1.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = n0 + tx * 4 + j;
      if (c >= N) continue;
      float v = acc[i][j];
      if (a >= 0) {
        const T* u = U + (int64_t)a * r * N;
        float t = 0.f;
        for (int q = 0; q < r; ++q) t = fmaf(P[m * r + q], to_f(MN ? u[(int64_t)q * N + c] : u[c * r + q]), t);
        v = fmaf(f, t, v);
      }
      if (bias) v += to_f(bias[c]);
      out[m * N + c] = from_f<T>(v);
    }
  }
}

// ------------------------------------------------------------------ gradients of the adapters
// out_a(j, k) = f_a sum over its rows P[i][j] S[i][k], out_a [r, K] or (KR) [K, r]; f_a = s_a when `scaled`.  P
// fp32 or of the rows' type.  A CTA has 64 columns of one adapter, a thread every fourth j of one; rows in
// the plan's order.  Zeros for an adapter without rows.
template <typename T, typename TP, bool KR>
__global__ void __launch_bounds__(256) multi_reduce_kernel(MultiPlan p, int64_t K, int r, const T* S, const TP* P, Scale s,
                                                           bool scaled, T* out) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int a = blockIdx.y;
  const int64_t k = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int j0 = threadIdx.x >> 6;
  if (k >= K) return;
  float acc[32] = {};
  for (int i = p.start[a]; i < p.start[a + 1]; ++i) {
    const int64_t row = p.order[i];
    const float x = to_f(S[row * K + k]);
#pragma unroll
    for (int q = 0; q < 32; ++q)
      if (j0 + 4 * q < r) acc[q] = fmaf(to_f(P[row * r + j0 + 4 * q]), x, acc[q]);
  }
  const float f = scaled ? s.of(a) : 1.f;
  T* o = out + (int64_t)a * r * K;
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    const int j = j0 + 4 * q;
    if (j < r) o[KR ? k * r + j : (int64_t)j * K + k] = from_f<T>(acc[q] * f);
  }
}

__global__ void __launch_bounds__(128) colsum_f32_kernel(int64_t M, int64_t K, const float* S, float* out) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int64_t k = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (k >= K) return;
  float t = 0.f;
  for (int64_t i = 0; i < M; ++i) t += S[i * K + k];
  out[k] = t;
}

// ------------------------------------------------------------------ launch sequences
struct MultiWs {
  uint32_t* err;
  void* P;                    // [M, r] z or s g; bf16: s z or s g
  void* Z;                    // [M, r] z recomputed by the backward
  float *pa, *pb, *csum;      // bf16 backward: partials of dA and dB, column sums
};
size_t carve(const lora_multi_shape& sh, bool bwd, char* base, MultiWs* w) {
  Carve c{base};
  const bool bf = sh.dtype == LORA_BF16;
  const size_t rank = (size_t)sh.M * sh.r * (bf ? 2 : 4), parts = (size_t)multi_partials(sh.M) * sh.r;
  w->err = c.take<uint32_t>(kErrBytes / 4);
  w->P = c.take<char>(rank);
  w->Z = bwd ? c.take<char>(rank) : nullptr;
  w->pa = bwd && bf ? c.take<float>(parts * sh.d_in) : nullptr;
  w->pb = bwd && bf ? c.take<float>(parts * sh.d_out) : nullptr;
  w->csum = bwd && bf ? c.take<float>((size_t)multi_colsum_splits(sh.M) * sh.d_out) : nullptr;
  return c.off;
}

unsigned blocks(int64_t n, int64_t per) { return (unsigned)((n + per - 1) / per); }

cudaError_t forward(const lora_multi_shape& sh, const MultiPlan& p, const MultiWs& w, const float* X, const float* W0,
                    const float* A, const float* B, const float* bias, Scale s, float* Y, float* Z, cudaStream_t st) {
  const int r = (int)sh.r;
  float* P = static_cast<float*>(w.P);
  const cudaError_t e = launch_pdl(multi_proj_kernel<float, false>, dim3((unsigned)sh.M), dim3(128), 0, st, p, sh.d_in, r,
                                   X, A, s, false, P, Z);
  if (e != cudaSuccess) return e;
  return launch_pdl(multi_gemm_kernel<float, false>, dim3(blocks(sh.d_out, 64), blocks(sh.M, 64)), dim3(256), 0, st, p,
                    sh.d_out, sh.d_in, r, X, W0, (const float*)P, B, s, true, bias, Y);
}

// out [M, N] = S [M, K] W (+ bias) and, for each row, T U_a: the GEMM with the tile's adapters as its tail
TcGemmDesc gemm(const MultiPlan& p, int mode, int64_t N, int64_t K, int r, int64_t n, const bf16* S, const bf16* W,
                const bf16* T, const bf16* U, const bf16* bias, bf16* out, uint32_t* err) {
  TcGemmDesc d;
  d.mode = mode;
  d.b0_mn = d.b1_mn = mode == TC_BWD_DX;
  d.M = (int)p.M;
  d.N = (int)N;
  d.K0 = (int)K;
  d.A0 = S;
  d.lda0 = K;
  d.B0 = W;
  d.ldb0 = d.b0_mn ? N : K;
  d.b0_rows = d.b0_mn ? (int)K : 0;
  d.has_tail = true;
  d.A1 = T;
  d.lda1 = r;
  d.K1 = d.K1_a = r;
  d.B1 = U;
  d.ad_count = p.tcount;
  d.ad_list = p.tlist;
  d.ad_mask = p.tmask;
  d.ad_total = (int)n;
  d.out[0] = out;
  d.ldo = N;
  d.bias = bias;
  d.err = err;
  d.timeout_ns = wait_timeout_ns();
  return d;
}

cudaError_t forward(const lora_multi_shape& sh, const MultiPlan& p, const MultiWs& w, const bf16* X, const bf16* W0,
                    const bf16* A, const bf16* B, const bf16* bias, Scale s, bf16* Y, bf16* Z, cudaStream_t st) {
  const int r = (int)sh.r;
  bf16* T = static_cast<bf16*>(w.P);
  const cudaError_t e = multi_proj(p, sh.d_in, r, X, A, false, s.one, s.each, Z, T, st);
  if (e != cudaSuccess) return e;
  return tc_gemm(gemm(p, TC_FWD, sh.d_out, sh.d_in, r, sh.n, X, W0, T, B, bias, Y, w.err), st);
}

cudaError_t backward(const lora_multi_shape& sh, const MultiPlan& p, const MultiWs& w, const float* X, const float* W0,
                     const float* A, const float* B, const float* Z, const float* dY, Scale s, float* dX, float* dA,
                     float* dB, float* dbias, cudaStream_t st) {
  const int r = (int)sh.r;
  float* P = static_cast<float*>(w.P);
  cudaError_t e;
  if (!Z) {
    e = launch_pdl(multi_proj_kernel<float, false>, dim3((unsigned)sh.M), dim3(128), 0, st, p, sh.d_in, r, X, A, s, false,
                   (float*)nullptr, (float*)w.Z);
    if (e != cudaSuccess) return e;
    Z = static_cast<const float*>(w.Z);
  }
  e = launch_pdl(multi_proj_kernel<float, true>, dim3((unsigned)sh.M), dim3(128), 0, st, p, sh.d_out, r, dY, B, s, true, P,
                 (float*)nullptr);
  if (e != cudaSuccess) return e;
  if (dX) {
    e = launch_pdl(multi_gemm_kernel<float, true>, dim3(blocks(sh.d_in, 64), blocks(sh.M, 64)), dim3(256), 0, st, p,
                   sh.d_in, sh.d_out, r, dY, W0, (const float*)P, A, s, false, (const float*)nullptr, dX);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(multi_reduce_kernel<float, float, false>, dim3(blocks(sh.d_in, 64), (unsigned)sh.n), dim3(256), 0, st, p,
                 sh.d_in, r, X, (const float*)P, s, false, dA);
  if (e != cudaSuccess) return e;
  e = launch_pdl(multi_reduce_kernel<float, float, true>, dim3(blocks(sh.d_out, 64), (unsigned)sh.n), dim3(256), 0, st, p,
                 sh.d_out, r, dY, Z, s, true, dB);
  if (e != cudaSuccess || !dbias) return e;
  return launch_pdl(colsum_f32_kernel, dim3(blocks(sh.d_out, 128)), dim3(128), 0, st, sh.M, sh.d_out, dY, dbias);
}

cudaError_t backward(const lora_multi_shape& sh, const MultiPlan& p, const MultiWs& w, const bf16* X, const bf16* W0,
                     const bf16* A, const bf16* B, const bf16* Z, const bf16* dY, Scale s, bf16* dX, bf16* dA, bf16* dB,
                     bf16* dbias, cudaStream_t st) {
  const int r = (int)sh.r;
  bf16* G = static_cast<bf16*>(w.P);
  cudaError_t e;
  if (!Z) {
    if ((e = multi_proj(p, sh.d_in, r, X, A, false, s.one, s.each, (bf16*)w.Z, nullptr, st)) != cudaSuccess) return e;
    Z = static_cast<const bf16*>(w.Z);
  }
  if ((e = multi_proj(p, sh.d_out, r, dY, B, true, s.one, s.each, nullptr, G, st)) != cudaSuccess) return e;
  if (dX && (e = tc_gemm(gemm(p, TC_BWD_DX, sh.d_in, sh.d_out, r, sh.n, dY, W0, G, A, nullptr, dX, w.err), st)) != cudaSuccess)
    return e;
  if ((e = multi_reduce(p, sh.d_in, r, X, G, false, false, 1.f, nullptr, w.pa, dA, st)) != cudaSuccess) return e;
  if ((e = multi_reduce(p, sh.d_out, r, dY, Z, true, true, s.one, s.each, w.pb, dB, st)) != cudaSuccess) return e;
  if ((e = multi_sum(p, sh.r * sh.d_in, w.pa, dA, sh.r * sh.d_out, w.pb, dB, st)) != cudaSuccess || !dbias) return e;
  return multi_colsum(sh.M, sh.d_out, dY, w.csum, dbias, st);
}

lora_status check(const lora_multi_shape* sh) {
  if (!sh) return LORA_ERR_INVALID_ARG;
  if (sh->M < 0 || sh->d_in <= 0 || sh->d_out <= 0 || sh->r <= 0 || sh->n <= 0) return LORA_ERR_INVALID_ARG;
  if (sh->dtype != LORA_F32 && sh->dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (sh->d_in % 8 || sh->d_out % 8 || sh->r > 128 || (sh->dtype == LORA_BF16 && sh->r % 8)) return LORA_ERR_UNSUPPORTED;
  constexpr int64_t top = (1LL << 31) - 1;
  // rows and columns are counted in 32 bits; 2^24 rows are 2^16 tiles, a launch's limit in its second dimension
  if (sh->M > 1 << 24 || sh->n > 65535 || sh->d_in > top - 512 || sh->d_out > top - 512) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

lora_status check_plan(const lora_multi_shape& sh, const void* plan, MultiPlan* p) {
  REQ(plan);
  if (reinterpret_cast<uintptr_t>(plan) & 255) return LORA_ERR_MISALIGNED;
  multi_plan_layout(sh.M, sh.n, static_cast<char*>(const_cast<void*>(plan)), p);
  return LORA_OK;
}

}  // namespace

}  // namespace lg

using namespace lg;

extern "C" {

size_t lora_multi_plan_bytes(int64_t M, int64_t n) {
  if (M < 0 || M > 1 << 24 || n < 1 || n > 65535) return 0;
  MultiPlan p;
  return multi_plan_layout(M, n, nullptr, &p);
}

lora_status lora_multi_plan(int64_t M, int64_t n, const void* ids, int id_bits, void* plan, size_t plan_bytes,
                            void* stream) {
  const size_t need = lora_multi_plan_bytes(M, n);
  if (need == 0) return M < 0 || n < 1 ? LORA_ERR_INVALID_ARG : LORA_ERR_UNSUPPORTED;
  if (id_bits != 32 && id_bits != 64) return LORA_ERR_INVALID_ARG;
  REQM(M, ids);
  if (reinterpret_cast<uintptr_t>(ids) % (id_bits / 8)) return LORA_ERR_MISALIGNED;
  const lora_status e = check_ws(plan, plan_bytes, need);
  if (e != LORA_OK) return e;
  if (M == 0) return LORA_OK;
  MultiPlan p;
  multi_plan_layout(M, n, static_cast<char*>(plan), &p);
  CK(multi_plan(p, ids, id_bits, (cudaStream_t)stream));
  return LORA_OK;
}

size_t lora_multi_workspace_bytes(int backward, const lora_multi_shape* sh) {
  if (check(sh) != LORA_OK) return 0;
  MultiWs w;
  return carve(*sh, backward != 0, nullptr, &w);
}

lora_status lora_multi_fwd(const lora_multi_shape* sh, const void* X, const void* W0, const void* A, const void* B,
                           const void* bias, float s, const float* s_each, const void* plan, void* Y, void* Z_save,
                           void* ws, size_t ws_bytes, void* stream) {
  lora_status e = check(sh);
  if (e != LORA_OK) return e;
  REQM(sh->M, X); REQ(W0); REQ(A); REQ(B); REQM(sh->M, Y);
  ALN(X); ALN(W0); ALN(A); ALN(B); ALN(bias); ALN(Y); ALN(Z_save);
  if (!s_each && !isfinite(s)) return LORA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(s_each) & 3) return LORA_ERR_MISALIGNED;
  MultiPlan p;
  if ((e = check_plan(*sh, plan, &p)) != LORA_OK) return e;
  MultiWs w;
  if ((e = check_ws(ws, ws_bytes, carve(*sh, false, nullptr, &w))) != LORA_OK) return e;
  carve(*sh, false, static_cast<char*>(ws), &w);
  if (sh->M == 0) return LORA_OK;
  cudaStream_t st = (cudaStream_t)stream;
  const Scale sc{s, s_each};
  if (sh->dtype == LORA_BF16)
    CK(forward(*sh, p, w, (const bf16*)X, (const bf16*)W0, (const bf16*)A, (const bf16*)B, (const bf16*)bias, sc, (bf16*)Y,
               (bf16*)Z_save, st));
  else
    CK(forward(*sh, p, w, (const float*)X, (const float*)W0, (const float*)A, (const float*)B, (const float*)bias, sc,
               (float*)Y, (float*)Z_save, st));
  return LORA_OK;
}

lora_status lora_multi_bwd(const lora_multi_shape* sh, const void* X, const void* W0, const void* A, const void* B,
                           const void* Z_saved, const void* dY, float s, const float* s_each, const void* plan, void* dX,
                           void* dA, void* dB, void* dbias, void* ws, size_t ws_bytes, void* stream) {
  lora_status e = check(sh);
  if (e != LORA_OK) return e;
  REQM(sh->M, X); REQ(W0); REQ(A); REQ(B); REQM(sh->M, dY); REQ(dA); REQ(dB);
  ALN(X); ALN(W0); ALN(A); ALN(B); ALN(Z_saved); ALN(dY); ALN(dX); ALN(dA); ALN(dB); ALN(dbias);
  if (!s_each && !isfinite(s)) return LORA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(s_each) & 3) return LORA_ERR_MISALIGNED;
  MultiPlan p;
  if ((e = check_plan(*sh, plan, &p)) != LORA_OK) return e;
  MultiWs w;
  if ((e = check_ws(ws, ws_bytes, carve(*sh, true, nullptr, &w))) != LORA_OK) return e;
  carve(*sh, true, static_cast<char*>(ws), &w);
  cudaStream_t st = (cudaStream_t)stream;
  const size_t es = sh->dtype == LORA_BF16 ? 2 : 4;
  if (sh->M == 0) {
    CK(cudaMemsetAsync(dA, 0, (size_t)sh->n * sh->r * sh->d_in * es, st));
    CK(cudaMemsetAsync(dB, 0, (size_t)sh->n * sh->r * sh->d_out * es, st));
    if (dbias) CK(cudaMemsetAsync(dbias, 0, (size_t)sh->d_out * es, st));
    return LORA_OK;
  }
  const Scale sc{s, s_each};
  if (sh->dtype == LORA_BF16)
    CK(backward(*sh, p, w, (const bf16*)X, (const bf16*)W0, (const bf16*)A, (const bf16*)B, (const bf16*)Z_saved,
                (const bf16*)dY, sc, (bf16*)dX, (bf16*)dA, (bf16*)dB, (bf16*)dbias, st));
  else
    CK(backward(*sh, p, w, (const float*)X, (const float*)W0, (const float*)A, (const float*)B, (const float*)Z_saved,
                (const float*)dY, sc, (float*)dX, (float*)dA, (float*)dB, (float*)dbias, st));
  return LORA_OK;
}

}  // extern "C"
