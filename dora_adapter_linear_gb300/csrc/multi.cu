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
};

// ------------------------------------------------------------------ launch sequences
struct MultiWs {
  uint32_t* err;
  void* P;                    // [M, r] z or s g; bf16: s z or s g
  void* P2;                   // bf16 backward: what the rounding of s g leaves
  void* Z;                    // [M, r] z recomputed by the backward
  float* few;                 // forward of a few bf16 rows: s z in fp32
  float *pa, *pb, *csum;      // bf16 backward: partials of dA and dB, column sums
  bf16 *S, *W;                // copies of X and W0, or of dY, in longer rows, where these are odd multiples of 16 bytes
};
// Whether copies of operands in longer rows pay.  Measured (rank 16, us without and with): forward 3001 x 2568 x 2568 58.3,
// 54.6, 8192 x 4104 x 4104 291, 240, 1999 x 2568 -> 1000 35.2, 32.2, but 1999 x 1000 -> 2568 27.6, 29.2, 600 x 2568 x 2568
// 28.4, 30.5; backward, dY alone, 3001 x 2568 x 2568 71.2, 68.8, 1000 x 4104 x 4104 59.8, 53.2, 600 x 2568 x 2568 33.1,
// 35.2 (W0 [K, N] as well: 74.3, 60.3, 36.3).  So: with some steps for a pair of multiprocessors, of 1000 rows or so.
// 76 pairs are written down here: a workspace is sized on hosts without a device as well.
bool pads(const lora_multi_shape& sh, bool bwd) {
  const int64_t mt = (sh.M + 255) / 256, tiles = mt * (((bwd ? sh.d_in : sh.d_out) + 255) / 256),
                steps = ((bwd ? sh.d_out : sh.d_in) + 63) / 64;
  return mt >= 4 && (tiles + 75) / 76 * steps >= 40;
}
size_t carve(const lora_multi_shape& sh, bool bwd, char* base, MultiWs* w) {
  Carve c{base};
  const bool bf = sh.dtype == LORA_BF16;
  const size_t rank = (size_t)sh.M * sh.r * (bf ? 2 : 4), parts = (size_t)multi_partials(sh.M) * sh.r;
  w->err = c.take<uint32_t>(kErrBytes / 4);
  w->P = c.take<char>(rank);
  w->Z = bwd ? c.take<char>(rank) : nullptr;
  w->P2 = bwd && bf ? c.take<char>(rank) : nullptr;
  w->few = !bwd && bf && sh.M <= kFewRows ? c.take<float>((size_t)sh.M * sh.r) : nullptr;
  w->pa = bwd && bf ? c.take<float>(parts * sh.d_in) : nullptr;
  w->pb = bwd && bf ? c.take<float>(parts * sh.d_out) : nullptr;
  const int64_t len = bwd ? sh.d_out : sh.d_in;
  const bool pad = bf && multi_pad_odd(len) && pads(sh, bwd);
  w->S = pad ? c.take<bf16>((size_t)sh.M * multi_pad_ld(len)) : nullptr;
  w->W = pad && !bwd ? c.take<bf16>((size_t)sh.d_out * multi_pad_ld(sh.d_in)) : nullptr;
  w->csum = bwd && bf ? c.take<float>((size_t)multi_colsum_splits(sh.M) * sh.d_out) : nullptr;
  return c.off;
}

cudaError_t forward(const lora_multi_shape& sh, const MultiPlan& p, const MultiWs& w, const float* X, const float* W0,
                    const float* A, const float* B, const float* bias, Scale s, float* Y, float* Z, cudaStream_t st) {
  const int r = (int)sh.r;
  if (!Z) Z = static_cast<float*>(w.P);
  const cudaError_t e = multi_f32_proj(p, sh.d_in, r, X, A, false, s.one, s.each, Z, nullptr, st);
  if (e != cudaSuccess) return e;
  return multi_f32_gemm(p, sh.d_out, sh.d_in, r, X, W0, false, Z, B, bias, true, s.one, s.each, Y, st);
}

cudaError_t backward(const lora_multi_shape& sh, const MultiPlan& p, const MultiWs& w, const float* X, const float* W0,
                     const float* A, const float* B, const float* Z, const float* dY, Scale s, float* dX, float* dA,
                     float* dB, float* dbias, cudaStream_t st) {
  const int r = (int)sh.r;
  float* G = static_cast<float*>(w.P);
  cudaError_t e;
  if (!Z) {
    if ((e = multi_f32_proj(p, sh.d_in, r, X, A, false, s.one, s.each, (float*)w.Z, nullptr, st)) != cudaSuccess) return e;
    Z = static_cast<const float*>(w.Z);
  }
  if ((e = multi_f32_proj(p, sh.d_out, r, dY, B, true, s.one, s.each, nullptr, G, st)) != cudaSuccess) return e;
  if (dX && (e = multi_f32_gemm(p, sh.d_in, sh.d_out, r, dY, W0, true, G, A, nullptr, false, 1.f, nullptr, dX, st)) !=
                cudaSuccess)
    return e;
  e = multi_f32_reduce(p, r, sh.d_in, X, G, dA, sh.d_out, dY, Z, dB, s.one, s.each, dX != nullptr, st);
  if (e != cudaSuccess || !dbias) return e;
  return multi_f32_colsum(sh.M, sh.d_out, dY, dbias, st);
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

// the product's operands in longer rows, where there is room for these
cudaError_t pad(const lora_multi_shape& sh, const MultiWs& w, const bf16* S, int64_t len, const bf16* W0, TcGemmDesc* d,
                cudaStream_t st) {
  if (!w.S && !w.W) return cudaSuccess;
  if (w.S) d->A0 = w.S, d->lda0 = multi_pad_ld(len);
  if (w.W) d->B0 = w.W, d->ldb0 = multi_pad_ld(sh.d_in);
  d->ad_wait = true;
  return multi_pad({S, w.S, sh.M, len}, {W0, w.W, sh.d_out, sh.d_in}, st);
}

// whether a product [M, N] has a tile for every pair of multiprocessors
bool fills(int64_t M, int64_t N) { return (M + 255) / 256 * ((N + 255) / 256) >= num_sms_current() / 2; }

cudaError_t forward(const lora_multi_shape& sh, const MultiPlan& p, const MultiWs& w, const bf16* X, const bf16* W0,
                    const bf16* A, const bf16* B, const bf16* bias, Scale s, bf16* Y, bf16* Z, cudaStream_t st) {
  const int r = (int)sh.r;
  if (multi_few_fits(sh.M, sh.d_out))
    return multi_few_fwd(p, sh.d_out, sh.d_in, r, X, W0, A, B, bias, s.one, s.each, w.few, Y, Z, w.err,
                         wait_timeout_ns(), st);
  bf16* T = static_cast<bf16*>(w.P);
  cudaError_t e = multi_proj(p, sh.d_in, r, X, A, false, s.one, s.each, Z, T, nullptr, fills(sh.M, sh.d_out), st);
  if (e != cudaSuccess) return e;
  TcGemmDesc d = gemm(p, TC_FWD, sh.d_out, sh.d_in, r, sh.n, X, W0, T, B, bias, Y, w.err);
  if ((e = pad(sh, w, X, sh.d_in, W0, &d, st)) != cudaSuccess) return e;
  return tc_gemm(d, st);
}

cudaError_t backward(const lora_multi_shape& sh, const MultiPlan& p, const MultiWs& w, const bf16* X, const bf16* W0,
                     const bf16* A, const bf16* B, const bf16* Z, const bf16* dY, Scale s, bf16* dX, bf16* dA, bf16* dB,
                     bf16* dbias, cudaStream_t st) {
  const int r = (int)sh.r;
  bf16* G = static_cast<bf16*>(w.P);
  cudaError_t e;
  if (!Z) {
    // as the forward has it where that takes the GEMM; multi_few sums in another order, and its z may be rounded the
    // other way
    if ((e = multi_proj(p, sh.d_in, r, X, A, false, s.one, s.each, (bf16*)w.Z, nullptr, nullptr, fills(sh.M, sh.d_out),
                        st)) != cudaSuccess)
      return e;
    Z = static_cast<const bf16*>(w.Z);
  }
  const bool beside = dX && fills(sh.M, sh.d_in);
  // s g enters dX rounded, like s z the output: a half step of the update, as the one-adapter layer has it (the
  // output's error beside its own rounding: 4% more at rank 16, where the update is 28% of the output, 12% at rank
  // 64, where it is half); a second part would double the tail's MMAs, 0.2 us for each adapter of a tile and 16 of
  // the rank.  As a factor of dA it comes with the rest of its rounding, which would otherwise add as much to dA's
  // error as dA's own rounding
  bf16* rest = static_cast<bf16*>(w.P2);
  if ((e = multi_proj(p, sh.d_out, r, dY, B, true, s.one, s.each, nullptr, G, rest, beside, st)) != cudaSuccess) return e;
  if (dX) {
    TcGemmDesc d = gemm(p, TC_BWD_DX, sh.d_in, sh.d_out, r, sh.n, dY, W0, G, A, nullptr, dX, w.err);
    if ((e = pad(sh, w, dY, sh.d_out, W0, &d, st)) != cudaSuccess || (e = tc_gemm(d, st)) != cudaSuccess) return e;
  }
  // the sums need nothing of that product: they run beside it, or where it leaves multiprocessors free
  e = multi_reduce(p, sh.d_out, r, dY, Z, nullptr, true, true, s.one, s.each, w.pb, dB, true, beside, st);
  if (e != cudaSuccess) return e;
  e = multi_reduce(p, sh.d_in, r, X, G, rest, false, false, 1.f, nullptr, w.pa, dA, dX != nullptr, beside, st);
  if (e == cudaSuccess && dbias) e = multi_colsum(sh.M, sh.d_out, dY, w.csum, st);
  if (e != cudaSuccess) return e;
  return multi_sum(p, sh.r * sh.d_in, w.pa, dA, sh.r * sh.d_out, w.pb, dB, sh.d_out, w.csum, dbias, st);
}

lora_status check(const lora_multi_shape* sh) {
  if (!sh) return LORA_ERR_INVALID_ARG;
  if (sh->M < 0 || sh->d_in <= 0 || sh->d_out <= 0 || sh->r <= 0 || sh->n <= 0) return LORA_ERR_INVALID_ARG;
  if (sh->dtype != LORA_F32 && sh->dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (sh->d_in % 8 || sh->d_out % 8 || sh->r > 128 || (sh->dtype == LORA_BF16 && sh->r % 8)) return LORA_ERR_UNSUPPORTED;
  // the launches' grids are counted for these
  if (sh->M > 1 << 24 || sh->n > 65535 || sh->d_in > 1 << 20 || sh->d_out > 1 << 20) return LORA_ERR_UNSUPPORTED;
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
