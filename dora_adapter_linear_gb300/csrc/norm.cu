// The norms before and after a block, fused with the block's gate and residual scale.
//
// Row i of M, D columns, gate row i / rows_per_gate, off = w_offset:
//   r_y = (mean(y^2) + eps)^-1/2,  p = y r_y (w_post + off)      (p = y without the post norm)
//   z   = x + alpha g o p                                        (z = x without a block output)
//   r_z = (mean(z^2) + eps)^-1/2,  h = z r_z (w_pre + off)
// and with c = r_z^3 / D sum(w_z dh z), w_z = w_pre + off, w_p = w_post + off:
//   dz = dz_in + r_z w_z dh - c z,   dx = dz,   dp = alpha g dz,   dg = sum_rows alpha p dz
//   dy = r_y w_p dp - y r_y^3 / D sum(w_p dp y)                  (dy = dp without the post norm)
//   dw_pre = sum_rows dh z r_z,   dw_post = sum_rows dp y r_y.
// Everything between a load and the one rounding of a store is fp32; h is formed from the unrounded
// z.  Bound by memory: the forward moves 4 M D elements, the backward 6 M D.
#include <math.h>

#include "checks.h"
#include "vec.cuh"

namespace lg {

namespace {

struct NormArgs {
  int64_t M, D, rpg;            // rpg: rows that share a gate row
  int64_t ldx, ldy, ldh, ldo;   // row strides of x (or z), y, dh, dz_in
  const void *x, *y, *w_pre, *w_post, *gate;
  float alpha, eps, off;
  int post;
  // forward outputs
  void *z_out, *h_out;
  float *r_pre, *r_post;
  // backward
  const void *dh, *dzi;
  void *dx, *dy;
  void* dgate_rows;             // [M, D] when every row has its own gate
  float* crow;                  // [M]: c of each row, for the column pass
  int64_t rp;                   // rows of a part of the column pass
  int parts;
  float *pw, *pp, *pg;          // partials [parts, D], [parts, D], [parts, 2, D]
  void *dw_pre, *dw_post, *dgate;
};

template <typename T>
__device__ __forceinline__ void weight8(const void* w, int64_t c, float off, float (&f)[8]) {
  if (w) {
    load8(static_cast<const T*>(w) + c, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] += off;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  }
}
// alpha times the gate of the row
template <typename T>
__device__ __forceinline__ void gate8(const NormArgs& a, const T* gate, int64_t c, float (&g)[8]) {
  if (gate) {
    load8(gate + c, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] *= a.alpha;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = a.alpha;
  }
}

// ------------------------------------------------------------------ forward, one CTA per row
// The row is read again for each of its steps (it is in L1 or L2 by then), so D has no limit.
template <typename T>
__device__ __forceinline__ void z8(const NormArgs& a, const T* x, const T* y, const T* gate, int64_t c, float r_y,
                                   float (&z)[8]) {
  load8(x + c, z);
  if (!y) return;
  float p[8], w[8], g[8];
  load8(y + c, p);
  gate8<T>(a, gate, c, g);
  if (a.post) {
    weight8<T>(a.w_post, c, a.off, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] *= r_y * w[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = fmaf(g[i], p[i], z[i]);
}

template <typename T>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  __shared__ float red[2 * 32];
  const int64_t row = blockIdx.x, step = (int64_t)blockDim.x * 8;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* y = a.y ? static_cast<const T*>(a.y) + row * a.ldy : nullptr;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + row / a.rpg * a.D : nullptr;
  const int64_t c0 = (int64_t)threadIdx.x * 8;
  float v[8], r_y = 1.f, ss[1];
  if (y && a.post) {
    ss[0] = 0.f;
    for (int64_t c = c0; c < a.D; c += step) {
      load8(y + c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = fmaf(v[i], v[i], ss[0]);
    }
    block_sums<1>(ss, red, 0);
    r_y = rsqrtf(ss[0] / (float)a.D + a.eps);
    if (threadIdx.x == 0 && a.r_post) a.r_post[row] = r_y;
  }
  float r_z = 1.f;
  if (a.h_out) {
    ss[0] = 0.f;
    for (int64_t c = c0; c < a.D; c += step) {
      z8<T>(a, x, y, gate, c, r_y, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss[0] = fmaf(v[i], v[i], ss[0]);
    }
    block_sums<1>(ss, red, 1);
    r_z = rsqrtf(ss[0] / (float)a.D + a.eps);
    if (threadIdx.x == 0 && a.r_pre) a.r_pre[row] = r_z;
  }
  // a thread writes only the columns that it alone has read, so z may replace x and h may replace y
  for (int64_t c = c0; c < a.D; c += step) {
    z8<T>(a, x, y, gate, c, r_y, v);
    if (a.z_out) store8(static_cast<T*>(a.z_out) + row * a.D + c, v);
    if (a.h_out) {
      float w[8];
      weight8<T>(a.w_pre, c, a.off, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= r_z * w[i];
      store8(static_cast<T*>(a.h_out) + row * a.D + c, v);
    }
  }
}

// ------------------------------------------------------------------ backward, rows: dx, dy, c
template <typename T>
__device__ __forceinline__ void opt8(const T* p, int64_t c, float (&f)[8]) {
  if (p) load8(p + c, f);
  else
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
}

template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_rows_kernel(const NormArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  __shared__ float red[2 * 32 * 3];
  const int64_t row = blockIdx.x, step = (int64_t)blockDim.x * 8;
  const T* z = static_cast<const T*>(a.x) + row * a.ldx;
  const T* y = a.y ? static_cast<const T*>(a.y) + row * a.ldy : nullptr;
  const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.ldh : nullptr;
  const T* dzi = a.dzi ? static_cast<const T*>(a.dzi) + row * a.ldo : nullptr;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + row / a.rpg * a.D : nullptr;
  const int64_t c0 = (int64_t)threadIdx.x * 8;
  const bool post = y && a.post;
  const float r_z = dh ? a.r_pre[row] : 0.f, r_y = post ? a.r_post[row] : 1.f;
  float zv[8], yv[8], hv[8], ov[8], wz[8], wp[8], g[8];
  // with u = alpha g w_p: S1 = sum(w_z dh z), S2 = sum(u y (dz_in + r_z w_z dh)), S3 = sum(u y z);
  // then sum(w_p dp y) = S2 - c S3, so one block reduction serves both norms
  float s[3] = {0.f, 0.f, 0.f};
  if (dh || post) {
    for (int64_t c = c0; c < a.D; c += step) {
      load8(z + c, zv);
      opt8<T>(dh, c, hv);
      weight8<T>(a.w_pre, c, a.off, wz);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hv[i] *= wz[i];
        s[0] = fmaf(hv[i], zv[i], s[0]);
      }
      if (!post) continue;
      load8(y + c, yv);
      opt8<T>(dzi, c, ov);
      weight8<T>(a.w_post, c, a.off, wp);
      gate8<T>(a, gate, c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float uy = g[i] * wp[i] * yv[i];
        s[1] = fmaf(uy, fmaf(r_z, hv[i], ov[i]), s[1]);
        s[2] = fmaf(uy, zv[i], s[2]);
      }
    }
    block_sums<3>(s, red, 0);
  }
  const float cz = dh ? r_z * r_z * r_z * (s[0] / (float)a.D) : 0.f;
  const float cy = post ? r_y * r_y * r_y * ((s[1] - cz * s[2]) / (float)a.D) : 0.f;
  if (threadIdx.x == 0 && a.crow) a.crow[row] = cz;
  for (int64_t c = c0; c < a.D; c += step) {
    load8(z + c, zv);
    opt8<T>(dh, c, hv);
    opt8<T>(dzi, c, ov);
    weight8<T>(a.w_pre, c, a.off, wz);
#pragma unroll
    for (int i = 0; i < 8; ++i) ov[i] = fmaf(r_z * wz[i], hv[i], ov[i]) - cz * zv[i];
    if (a.dx) store8(static_cast<T*>(a.dx) + row * a.D + c, ov);
    if (!y) continue;
    opt8<T>(y, c, yv);
    gate8<T>(a, gate, c, g);
    weight8<T>(post ? a.w_post : nullptr, c, a.off, wp);
    if (a.dgate_rows) {
      float dg[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) dg[i] = a.alpha * ov[i] * yv[i] * (r_y * wp[i]);
      store8(static_cast<T*>(a.dgate_rows) + row * a.D + c, dg);
    }
    if (a.dy) {
#pragma unroll
      for (int i = 0; i < 8; ++i) ov[i] = r_y * wp[i] * (g[i] * ov[i]) - cy * yv[i];
      store8(static_cast<T*>(a.dy) + row * a.D + c, ov);
    }
  }
}

// ------------------------------------------------------------------ backward, columns: dw, dgate
// Part b takes rows [b rp, (b + 1) rp); CTA (t, b) their columns [256 t, 256 t + 256), lane l of
// each of its 8 warps columns 8 l .. 8 l + 7 and warp w every 8th row.  dz is formed again from its
// inputs and the row's c, unrounded.  Inside a part the rows of one gate row are one segment; a
// segment that holds all rows of its gate row writes dgate itself, any other one writes its partial
// sum into slot 0 (the part's first segment) or 1 (its last).
constexpr int kColWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kColWarps) norm_bwd_cols_kernel(const NormArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  __shared__ float acc[kColWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 256 + lane * 8, part = blockIdx.y;
  const bool in = c < a.D;
  const int64_t r0 = part * a.rp, r1 = min(a.M, r0 + a.rp);
  const bool post = a.y && a.post;
  float wz[8], wp[8], dw[8], dp[8], dg[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = dp[i] = 0.f;
  if (in) {
    weight8<T>(a.w_pre, c, a.off, wz);
    weight8<T>(post ? a.w_post : nullptr, c, a.off, wp);
  }
  // adds the warps' sums in order and gives thread t column 256 blockIdx.x + t
  auto total = [&](const float (&v)[8]) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[warp][lane * 8 + i] = v[i];
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kColWarps; ++w) t += acc[w][threadIdx.x];
    return t;
  };
  const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t s0 = r0; s0 < r1;) {
    const int64_t grp = s0 / a.rpg, s1 = min(r1, (grp + 1) * a.rpg);
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[i] = 0.f;
    if (in) {
      float g[8];
      gate8<T>(a, a.gate ? static_cast<const T*>(a.gate) + grp * a.D : nullptr, c, g);
      for (int64_t row = s0 + warp; row < s1; row += kColWarps) {
        float zv[8], hv[8], ov[8], yv[8];
        load8(static_cast<const T*>(a.x) + row * a.ldx + c, zv);
        opt8<T>(a.dh ? static_cast<const T*>(a.dh) + row * a.ldh : nullptr, c, hv);
        const float r_z = a.dh ? a.r_pre[row] : 0.f, r_y = post ? a.r_post[row] : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] = fmaf(hv[i] * r_z, zv[i], dw[i]);
        if (!a.pp && !a.dgate) continue;
        const float cz = a.crow[row];
        opt8<T>(a.dzi ? static_cast<const T*>(a.dzi) + row * a.ldo : nullptr, c, ov);
        load8(static_cast<const T*>(a.y) + row * a.ldy + c, yv);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = (fmaf(r_z * wz[i], hv[i], ov[i]) - cz * zv[i]) * yv[i] * r_y;   // dz y r_y
          dp[i] = fmaf(g[i], n, dp[i]);
          dg[i] = fmaf(wp[i], n, dg[i]);
        }
      }
    }
    if (a.dgate) {
      const float t = a.alpha * total(dg);
      if (col < a.D) {
        const int64_t g0 = grp * a.rpg, g1 = min(a.M, g0 + a.rpg);
        if (g0 >= r0 && g1 <= r1) static_cast<T*>(a.dgate)[grp * a.D + col] = from_f<T>(t);
        else a.pg[(part * 2 + (s0 == r0 ? 0 : 1)) * a.D + col] = t;
      }
    }
    s0 = s1;
  }
  if (a.pw) {
    const float t = total(dw);
    if (col < a.D) a.pw[part * a.D + col] = t;
  }
  if (a.pp) {
    const float t = total(dp);
    if (col < a.D) a.pp[part * a.D + col] = t;
  }
}

// ------------------------------------------------------------------ backward: sums of the partials
// CTA (t, j): columns 32 t .. 32 t + 31, one per lane; the warps share the parts.  j = 0: dw_pre,
// 1: dw_post, 2 + k: the gate row that crosses the boundary before part k + 1, if that is its first.
template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_finish_kernel(const NormArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const int job = blockIdx.y;
  int first = 0, last = a.parts - 1;
  T* out = nullptr;
  int64_t grp = 0;
  if (job == 0) out = static_cast<T*>(a.dw_pre);
  else if (job == 1) out = static_cast<T*>(a.dw_post);
  else if (a.dgate) {
    const int64_t b = (int64_t)(job - 1) * a.rp;   // the boundary's row
    grp = b / a.rpg;
    const int64_t g0 = grp * a.rpg, g1 = min(a.M, g0 + a.rpg);
    first = (int)(g0 / a.rp);
    last = (int)((g1 - 1) / a.rp);
    if (g0 < b && first == job - 2) out = static_cast<T*>(a.dgate) + grp * a.D;
  }
  if (!out) return;
  float t = 0.f;
  if (col < a.D) {
    for (int p = first + warp; p <= last; p += 32) {
      if (job == 0) t += a.pw[p * a.D + col];
      else if (job == 1) t += a.pp[p * a.D + col];
      else t += a.pg[((int64_t)p * 2 + ((int64_t)p * a.rp / a.rpg == grp ? 0 : 1)) * a.D + col];
    }
  }
  acc[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && col < a.D) {
    t = 0.f;
    for (int w = 0; w < 32; ++w) t += acc[w][lane];
    out[col] = from_f<T>(t);
  }
}

int row_threads(int64_t D) {
  const int64_t n = (D / 8 + 31) / 32 * 32;
  return (int)(n > 1024 ? 1024 : n);
}

lora_status check_norm(const lora_norm_shape* sh) {
  if (!sh) return LORA_ERR_INVALID_ARG;
  if (sh->M < 0 || sh->D <= 0 || sh->rows_per_gate < 0) return LORA_ERR_INVALID_ARG;
  if (sh->dtype != LORA_F32 && sh->dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (!isfinite(sh->alpha) || !isfinite(sh->w_offset) || !(sh->eps > 0.f) || !isfinite(sh->eps))
    return LORA_ERR_INVALID_ARG;
  if (sh->D % 8 || sh->M > (1LL << 31) - 1 || sh->D > (1LL << 31) - 1) return LORA_ERR_UNSUPPORTED;
  const int64_t per16 = sh->dtype == LORA_BF16 ? 8 : 4;
  for (int64_t ld : {sh->ldx, sh->ldy, sh->lddh, sh->lddz}) {
    if (ld < sh->D) return LORA_ERR_INVALID_ARG;
    if (ld % per16) return LORA_ERR_MISALIGNED;
  }
  return LORA_OK;
}

// Row parts of the column sums: two CTAs per SM over all column tiles, at least 32 rows each.
void norm_parts(const lora_norm_shape& sh, int64_t* rp, int* parts) {
  const int64_t tiles = (sh.D + 255) / 256;
  int64_t want = (4LL * num_sms_current() + tiles - 1) / tiles;
  if (want > (sh.M + 31) / 32) want = (sh.M + 31) / 32;
  if (want < 1) want = 1;
  *rp = (sh.M + want - 1) / want;
  if (*rp < 1) *rp = 1;
  *parts = (int)((sh.M + *rp - 1) / *rp);
}

struct NormBwdWs {
  float *crow, *pw, *pp, *pg;
};
size_t plan_norm_bwd(const lora_norm_shape& sh, char* base, NormBwdWs* w) {
  int64_t rp;
  int parts;
  norm_parts(sh, &rp, &parts);
  Carve c{base};
  c.take<char>(kErrBytes);
  w->crow = c.take<float>((size_t)sh.M);
  w->pw = c.take<float>((size_t)parts * sh.D);
  w->pp = c.take<float>((size_t)parts * sh.D);
  w->pg = c.take<float>((size_t)parts * 2 * sh.D);
  return c.off;
}

NormArgs norm_args(const lora_norm_shape& sh, const void* x, const void* y, const void* w_pre, const void* w_post,
                   const void* gate) {
  NormArgs a = {};
  a.M = sh.M, a.D = sh.D;
  a.rpg = gate ? sh.rows_per_gate : (sh.M > 0 ? sh.M : 1);
  a.ldx = sh.ldx, a.ldy = sh.ldy, a.ldh = sh.lddh, a.ldo = sh.lddz;
  a.x = x, a.y = y, a.w_pre = w_pre, a.w_post = w_post, a.gate = gate;
  a.alpha = sh.alpha, a.eps = sh.eps, a.off = sh.w_offset, a.post = sh.post_norm != 0;
  return a;
}

template <typename T>
lora_status norm_bwd(NormArgs& a, cudaStream_t st) {
  const dim3 row_cta(row_threads(a.D));
  if (a.M > 0) CK(launch_pdl(norm_bwd_rows_kernel<T>, dim3((unsigned)a.M), row_cta, 0, st, a));
  if (!a.dw_pre && !a.dw_post && !a.dgate) return LORA_OK;
  if (a.parts > 0)
    CK(launch_pdl(norm_bwd_cols_kernel<T>, dim3((unsigned)((a.D + 255) / 256), (unsigned)a.parts),
                  dim3(32 * kColWarps), 0, st, a));
  const int jobs = a.dgate && a.parts > 1 ? 2 + a.parts - 1 : 2;
  CK(launch_pdl(norm_bwd_finish_kernel<T>, dim3((unsigned)((a.D + 31) / 32), (unsigned)jobs), dim3(1024), 0, st, a));
  return LORA_OK;
}

}  // namespace

}  // namespace lg

using namespace lg;

extern "C" {

lora_status block_norm_fwd(const lora_norm_shape* sh, const void* X, const void* Y, const void* w_pre,
                           const void* w_post, const void* gate, void* Xout, void* H, float* r_pre, float* r_post,
                           void* stream) {
  const lora_status e = check_norm(sh);
  if (e != LORA_OK) return e;
  REQM(sh->M, X);
  if (sh->M > 0) {
    if (Y && !Xout) return LORA_ERR_INVALID_ARG;
    if (!Y && (Xout || gate || sh->post_norm || !H)) return LORA_ERR_INVALID_ARG;   // only the pre norm is left
    if (w_pre && !H) return LORA_ERR_INVALID_ARG;
  }
  if (w_post && !sh->post_norm) return LORA_ERR_INVALID_ARG;
  if (gate && sh->rows_per_gate < 1) return LORA_ERR_INVALID_ARG;
  if ((Xout == X && X && sh->ldx != sh->D) || (H == Y && Y && sh->ldy != sh->D)) return LORA_ERR_INVALID_ARG;
  for (const void* p : {X, Y, w_pre, w_post, gate, (const void*)Xout, (const void*)H, (const void*)r_pre,
                        (const void*)r_post})
    ALN(p);
  if (sh->M == 0) return LORA_OK;
  NormArgs a = norm_args(*sh, X, Y, w_pre, w_post, gate);
  a.z_out = Xout, a.h_out = H, a.r_pre = r_pre, a.r_post = r_post;
  const dim3 grid((unsigned)sh->M), cta(row_threads(sh->D));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (sh->dtype == LORA_BF16) CK(launch_pdl(norm_fwd_kernel<bf16>, grid, cta, 0, st, a));
  else CK(launch_pdl(norm_fwd_kernel<float>, grid, cta, 0, st, a));
  return LORA_OK;
}

size_t block_norm_bwd_workspace_bytes(const lora_norm_shape* sh) {
  NormBwdWs w;
  return check_norm(sh) == LORA_OK ? plan_norm_bwd(*sh, nullptr, &w) : 0;
}

lora_status block_norm_bwd(const lora_norm_shape* sh, const void* Xout, const void* Y, const void* w_pre,
                           const void* w_post, const void* gate, const float* r_pre, const float* r_post,
                           const void* dH, const void* dXout, void* dX, void* dY, void* dw_pre, void* dw_post,
                           void* dgate, void* ws, size_t ws_bytes, void* stream) {
  const lora_status e = check_norm(sh);
  if (e != LORA_OK) return e;
  REQM(sh->M, Xout);
  if (sh->M > 0 && !dH && !dXout) return LORA_ERR_INVALID_ARG;
  if (dH) REQM(sh->M, r_pre);
  if (!Y && sh->M > 0 && (gate || sh->post_norm || dY)) return LORA_ERR_INVALID_ARG;
  if (Y && sh->post_norm) REQM(sh->M, r_post);
  if (w_post && !sh->post_norm) return LORA_ERR_INVALID_ARG;
  if ((dw_pre && !w_pre) || (dw_post && !w_post) || (dgate && !gate)) return LORA_ERR_INVALID_ARG;
  if (gate && sh->rows_per_gate < 1) return LORA_ERR_INVALID_ARG;
  for (const void* o : {(const void*)dX, (const void*)dY})
    for (const void* i : {Xout, Y, dH, dXout})
      if (o && o == i) return LORA_ERR_INVALID_ARG;   // an input is read again after an output row is written
  for (const void* p : {Xout, Y, w_pre, w_post, gate, (const void*)r_pre, (const void*)r_post, dH, dXout,
                        (const void*)dX, (const void*)dY, (const void*)dw_pre, (const void*)dw_post,
                        (const void*)dgate})
    ALN(p);
  NormBwdWs w;
  const lora_status ew = check_ws(ws, ws_bytes, plan_norm_bwd(*sh, static_cast<char*>(ws), &w));
  if (ew != LORA_OK) return ew;
  NormArgs a = norm_args(*sh, Xout, Y, w_pre, w_post, gate);
  norm_parts(*sh, &a.rp, &a.parts);
  a.r_pre = const_cast<float*>(r_pre), a.r_post = const_cast<float*>(r_post);
  a.dh = dH, a.dzi = dXout, a.dx = dX, a.dy = dY;
  a.dw_pre = dw_pre, a.dw_post = dw_post;
  a.crow = w.crow;
  if (gate && sh->rows_per_gate == 1) {
    a.dgate_rows = dgate;   // a gate row per row: its gradient is an output of the row pass
  } else {
    a.dgate = dgate;
  }
  a.pw = dw_pre ? w.pw : nullptr;
  a.pp = dw_post ? w.pp : nullptr;
  a.pg = w.pg;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return sh->dtype == LORA_BF16 ? norm_bwd<bf16>(a, st) : norm_bwd<float>(a, st);
}

}  // extern "C"
