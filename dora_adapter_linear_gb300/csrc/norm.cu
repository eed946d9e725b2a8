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

constexpr int kSmSmem = 227 * 1024, kRingStatic = 3 * 1024;   // of an SM; what a CTA has beside its dynamic part
// asked for by every kernel with a dynamic part: up to 48 KB go without, but a kernel's own arrays count among them
constexpr int kDynamicSmem = kSmSmem - kRingStatic;

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
  uint32_t* err;                // device error word and limit of the bounded waits
  uint64_t timeout_ns;
};

// threads of a CTA that takes one row
int row_threads(int64_t D) {
  const int64_t n = (D / 8 + 31) / 32 * 32;
  return (int)(n > 1024 ? 1024 : n);
}

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

template <typename T>
__device__ __forceinline__ void weight4x2(const void* w, int64_t c, float off, F2 (&f)[4]) {
  if (w) load4x2(static_cast<const T*>(w) + c, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = w ? add2(f[i], f2(off)) : f2(1.f);
}
template <typename T>
__device__ __forceinline__ void gate4x2(const T* gate, int64_t c, float alpha, F2 (&g)[4]) {
  if (gate) load4x2(gate + c, g);
#pragma unroll
  for (int i = 0; i < 4; ++i) g[i] = gate ? mul2(g[i], f2(alpha)) : f2(alpha);
}

// what a launch has of a block output: none, one, one behind a post norm, or either of the last two
enum { NO_Y = 0, PLAIN_Y = 1, POST_Y = 2, ANY_Y = 3 };

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

// ------------------------------------------------------------------ forward, the row in registers
// A thread holds K vectors of 8 columns, so x and y are read once and all their loads are in flight
// together.  G lanes of a warp share a row, or a whole CTA (G = 0).
// The post norm would put a second block sum in the row's way, behind the first.  With q = alpha g w_p o y
// the sum of z^2 is sum x^2 + 2 r_y sum x q + r_y^2 sum q^2, so one block sum of four values serves both
// norms; a row where those terms cancel to less than a quarter of their size (their rounding would be
// more than four times that of the plain sum) takes the plain sum after all, and so does one where they
// overflow (sum q^2 can without sum z^2 doing so).
template <typename T, int K, int G, int Y>
__global__ void __launch_bounds__(G ? 256 : 1024) norm_fwd_held_kernel(const NormArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  __shared__ __align__(16) float red[G ? 1 : 2 * 4 * 32];
  const int t = G ? threadIdx.x % G : threadIdx.x, group = G ? G : blockDim.x, D = (int)a.D;
  const int64_t at = G ? (int64_t)blockIdx.x * (256 / G) + threadIdx.x / G : blockIdx.x;
  const bool mine = !G || at < a.M;   // a group past the last row goes along for its warp's shuffles
  const int64_t row = mine ? at : 0;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* y = Y ? static_cast<const T*>(a.y) + row * a.ldy : nullptr;
  const T* gate = Y && a.gate ? static_cast<const T*>(a.gate) + row / a.rpg * D : nullptr;
  const auto col = [&](int k) { return mine ? (k * group + t) * 8 : D; };
  Raw8<T> xr[K], yr[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (col(k) >= D) continue;
    if (Y) stream8(y + col(k), yr[k]);
    stream8(x + col(k), xr[k]);
  }
  auto row_sums = [&](float (&v)[4], int flip) {
    if (G) spread<4, G ? G : 32>(warp_sums_of<4, G ? G : 32>(v), v);
    else block_sums_of<4, 32>(v, red, flip);
  };
  F2 q[K][4], p[4], w[4];   // q: what r_y times is added to x; later z
  F2 xx = f2(0.f), xq = f2(0.f), qq = f2(0.f), yy = f2(0.f);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (col(k) >= D) continue;
    xr[k].get(w);
    if (!Y) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[k][i] = w[i];
        xx = fma2(w[i], w[i], xx);
      }
      continue;
    }
    yr[k].get(q[k]);
    if (Y == POST_Y) {
      weight4x2<T>(a.w_post, col(k), a.off, p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        yy = fma2(q[k][i], q[k][i], yy);
        q[k][i] = mul2(q[k][i], p[i]);
      }
    }
    gate4x2<T>(gate, col(k), a.alpha, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (Y == POST_Y) {
        q[k][i] = mul2(q[k][i], p[i]);
        xx = fma2(w[i], w[i], xx);
        xq = fma2(w[i], q[k][i], xq);
        qq = fma2(q[k][i], q[k][i], qq);
      } else {
        q[k][i] = fma2(p[i], q[k][i], w[i]);
        xx = fma2(q[k][i], q[k][i], xx);
      }
    }
    if (Y == PLAIN_Y) store4x2(static_cast<T*>(a.z_out) + row * D + col(k), q[k]);
  }
  if (Y != POST_Y && !a.h_out) return;
  float s[4] = {sum2(xx), sum2(xq), sum2(qq), sum2(yy)};
  row_sums(s, 0);
  float zz = s[0];
  if (Y == POST_Y) {
    const float r_y = rsqrtf(s[3] / (float)D + a.eps), size = fmaf(r_y * r_y, s[2], s[0]);
    if (t == 0 && mine && a.r_post) a.r_post[row] = r_y;
    xx = f2(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (col(k) >= D) continue;
      xr[k].get(w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q[k][i] = fma2(f2(r_y), q[k][i], w[i]);
        xx = fma2(q[k][i], q[k][i], xx);
      }
      store4x2(static_cast<T*>(a.z_out) + row * D + col(k), q[k]);
    }
    if (!a.h_out) return;
    zz = fmaf(2.f * r_y, s[1], size);
    const bool plain = !(zz >= 0.25f * size) || isinf(size);   // the same for the whole row
    if (G && G < 32 ? __any_sync(0xffffffffu, plain) : plain) {
      s[0] = sum2(xx), s[1] = s[2] = s[3] = 0.f;
      row_sums(s, 1);
      if (plain) zz = s[0];
    }
  }
  const float r_z = rsqrtf(zz / (float)D + a.eps);
  if (t == 0 && mine && a.r_pre) a.r_pre[row] = r_z;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (col(k) >= D) continue;
    weight4x2<T>(a.w_pre, col(k), a.off, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = mul2(q[k][i], mul2(w[i], f2(r_z)));
    store4x2(static_cast<T*>(a.h_out) + row * D + col(k), w);
  }
}

template <typename T, int K, int G>
cudaError_t launch_held(const NormArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)(G ? (a.M + 256 / (G ? G : 1) - 1) / (256 / (G ? G : 1)) : a.M));
  const dim3 cta((unsigned)(G ? 256 : (a.D / 8 + 32 * K - 1) / (32 * K) * 32));
  if (!a.y) return launch_pdl(norm_fwd_held_kernel<T, K, G, NO_Y>, grid, cta, 0, st, a);
  if (!a.post) return launch_pdl(norm_fwd_held_kernel<T, K, G, PLAIN_Y>, grid, cta, 0, st, a);
  return launch_pdl(norm_fwd_held_kernel<T, K, G, POST_Y>, grid, cta, 0, st, a);
}

// ------------------------------------------------------------------ forward with a post norm, many rows
// A CTA walks over every gridDim-th row with the weights in registers, two vectors a thread, the sums as
// above.  Each thread keeps its own columns of the next row (x, y and, with a gate row per row, the gate)
// on their way into shared memory: no thread reads another's, so the copies need no barrier.  bf16, 16384 x
// 4096: 83 us (85 with a gate per sequence, 107 per row; floors 79, 79, 99) against 87 (101, 140) of the held
// kernel, which loads and unpacks the weights for every row.  Two rows of a CTA in flight are faster than
// three or four (83 against 94 and 96 us) and neighbouring rows at a time than a part of its own for each CTA.
constexpr int kWalkThreads = 512;   // an SM's, at 128 registers

template <typename T, bool TOKEN>
__global__ void __launch_bounds__(kWalkThreads) norm_fwd_walk_kernel(const NormArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  constexpr int A = TOKEN ? 3 : 2, K = 2, S = 2;   // arrays of a stage, vectors of a thread, stages
  extern __shared__ __align__(16) char stages[];
  __shared__ __align__(16) float red[2 * 4 * 16];
  const int D = (int)a.D, c0 = (int)threadIdx.x * 8, hop = (int)blockDim.x * 8;   // columns c0 + k hop
  const int64_t r0 = blockIdx.x, stride = gridDim.x;
  const T* gate = static_cast<const T*>(a.gate);
  T* const ring = reinterpret_cast<T*>(stages) + c0;
  T *fill = ring, *use = ring, *const ring_end = ring + S * A * D;
  // what moves from row to row is a pointer that is stepped
  const T* src[A];
  src[0] = static_cast<const T*>(a.x) + r0 * a.ldx + c0;
  src[1] = static_cast<const T*>(a.y) + r0 * a.ldy + c0;
  if (TOKEN) src[A - 1] = gate + r0 * D + c0;
  auto issue = [&](bool more) {   // this thread's columns of the next row; a group even past the end
    if (more) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (c0 + k * hop >= D) continue;
#pragma unroll
        for (int i = 0; i < A; ++i)
#pragma unroll
          for (int e = 0; e < 8; e += 16 / (int)sizeof(T)) cp_async16(fill + i * D + k * hop + e, src[i] + k * hop + e, true);
      }
      src[0] += stride * a.ldx;
      src[1] += stride * a.ldy;
      if (TOKEN) src[A - 1] += stride * D;
    }
    cp_async_commit();
    fill += A * D;
    if (fill == ring_end) fill = ring;
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(r0 + i * stride < a.M);
  F2 wz[K][4], u[K][4];   // u = alpha g w_p (TOKEN: alpha w_p)
  auto group_weights = [&](const T* g) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (c0 + k * hop >= D) continue;
      F2 w[4];
      gate4x2<T>(g, c0 + k * hop, a.alpha, w);
      weight4x2<T>(a.w_post, c0 + k * hop, a.off, u[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[k][i] = mul2(u[k][i], w[i]);
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (c0 + k * hop < D) weight4x2<T>(a.w_pre, c0 + k * hop, a.off, wz[k]);
  if (TOKEN || !gate) group_weights(nullptr);
  const float inv_d = 1.f / (float)D;
  T* zo = static_cast<T*>(a.z_out) + r0 * D + c0;
  T* ho = a.h_out ? static_cast<T*>(a.h_out) + r0 * D + c0 : nullptr;
  int64_t grp = -1;
  int flip = 0;
  for (int64_t row = r0; row < a.M; row += stride) {
    if (!TOKEN && gate && row >= (grp + 1) * a.rpg) {   // uniform over the CTA
      grp = row / a.rpg;
      group_weights(gate + grp * D);
    }
    issue(row + (S - 1) * stride < a.M);   // into the stage that the last row left
    cp_async_wait<S - 1>();
    F2 x[K][4], q[K][4], g[4], xx = f2(0.f), xq = f2(0.f), qq = f2(0.f), yy = f2(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (c0 + k * hop >= D) continue;
      load4x2(use + k * hop, x[k]);
      load4x2(use + D + k * hop, q[k]);
      if (TOKEN) load4x2(use + 2 * D + k * hop, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        yy = fma2(q[k][i], q[k][i], yy);
        q[k][i] = mul2(q[k][i], TOKEN ? mul2(u[k][i], g[i]) : u[k][i]);
        xx = fma2(x[k][i], x[k][i], xx);
        xq = fma2(x[k][i], q[k][i], xq);
        qq = fma2(q[k][i], q[k][i], qq);
      }
    }
    use += A * D;
    if (use == ring_end) use = ring;
    float s[4] = {sum2(xx), sum2(xq), sum2(qq), sum2(yy)};
    block_sums_of<4, 16>(s, red, flip);
    flip ^= 1;
    const float r_y = rsqrtf(fmaf(s[3], inv_d, a.eps)), size = fmaf(r_y * r_y, s[2], s[0]);
    if (threadIdx.x == 0 && a.r_post) a.r_post[row] = r_y;
    xx = f2(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (c0 + k * hop >= D) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[k][i] = fma2(f2(r_y), q[k][i], x[k][i]);
        xx = fma2(x[k][i], x[k][i], xx);
      }
      store4x2(zo + k * hop, x[k]);
    }
    zo += stride * D;
    if (!ho) continue;
    float zz = fmaf(2.f * r_y, s[1], size);
    if (!(zz >= 0.25f * size) || isinf(size)) {   // the same for the whole row
      s[0] = sum2(xx), s[1] = s[2] = s[3] = 0.f;
      block_sums_of<4, 16>(s, red, flip);
      flip ^= 1;
      zz = s[0];
    }
    const float r_z = rsqrtf(fmaf(zz, inv_d, a.eps));
    if (threadIdx.x == 0 && a.r_pre) a.r_pre[row] = r_z;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (c0 + k * hop >= D) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[k][i] = mul2(x[k][i], mul2(wz[k][i], f2(r_z)));
      store4x2(ho + k * hop, x[k]);
    }
    ho += stride * D;
  }
}

template <typename T>
cudaError_t launch_walk(const NormArgs& a, cudaStream_t st) {
  const int threads = (int)((a.D / 8 + 63) / 64 * 32);
  const int64_t most = (int64_t)(kWalkThreads / threads) * num_sms_current();
  const bool token = a.gate && a.rpg == 1;
  const size_t smem = 2 * (size_t)(token ? 3 : 2) * a.D * sizeof(T);   // at most 96 KB
  const cudaError_t allowed = token ? allow_smem<norm_fwd_walk_kernel<T, true>>(kDynamicSmem)
                                    : allow_smem<norm_fwd_walk_kernel<T, false>>(kDynamicSmem);
  if (allowed != cudaSuccess) return allowed;
  return launch_pdl(token ? norm_fwd_walk_kernel<T, true> : norm_fwd_walk_kernel<T, false>,
                    dim3((unsigned)(a.M < most ? a.M : most)), dim3((unsigned)threads), smem, st, a);
}

// Rows that are all resident at once (half the threads of the SMs) want the shortest chain: one vector a
// thread (1 x 4096 bf16: 2.4 against 2.7 us with two; at 512 rows 5.7 against 4.7).  Beyond that:
//   up to 256 columns a warp a row (16384 x 256 bf16: 7.6 us), up to 128 and 64 a half and a quarter of one
//   (131072 x 128 25 us against 44 with a warp, x 64 13 against 43); two vectors a lane for bf16 up to 512 (16384 x
//   512 without a post norm: 12.5 against 17 us) and fp32 up to 384 (11274 x 264: 9.8 against 12.1, x 384: 11.6
//   against 12.3, x 504: 15.2 against 14.0);
//   bf16 with a post norm the walk from 512 to 8192 columns (16384 x 512: 11.5 against 12.5 us with a warp a
//   row, x 2048: 43 against 47, x 8192: 85 per 8192 rows against 97);
//   fp32 one vector up to 2048 columns (8192 x 1024: 20 us against 21 with the walk and 28 with two vectors),
//   then two (8192 x 4096: 86 against 94 with one or the walk);
//   bf16 without a post norm two vectors (16384 x 4096: 79 us, the floor).
template <typename T>
cudaError_t norm_fwd(const NormArgs& a, cudaStream_t st) {
  constexpr bool narrow = sizeof(T) == 2;
  const int64_t vecs = a.D / 8;
  if (vecs <= 8) return launch_held<T, 1, 8>(a, st);
  if (vecs <= 16) return launch_held<T, 1, 16>(a, st);
  if (vecs <= 32) return launch_held<T, 1, 32>(a, st);
  if (vecs <= 1024 && a.M * vecs <= 1024LL * num_sms_current()) return launch_held<T, 1, 0>(a, st);
  if (vecs < (narrow ? 64 + !(a.y && a.post) : 49)) return launch_held<T, 2, 32>(a, st);
  if (narrow && a.y && a.post && vecs >= 64 && vecs <= 1024) return launch_walk<bf16>(a, st);
  if (!narrow && vecs <= 256) return launch_held<T, 1, 0>(a, st);
  if (vecs <= 2048) return launch_held<T, 2, 0>(a, st);
  return launch_pdl(norm_fwd_kernel<T>, dim3((unsigned)a.M), dim3((unsigned)row_threads(a.D)), 0, st, a);
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

// ------------------------------------------------------------------ backward in one pass
// One CTA takes the rows of a part in order, a thread always the same 8 columns: the column sums stay
// in its registers for the whole part, the weights too, and every input is read once.  The rows
// arrive by bulk copies in a ring of stages (z, y, dh, dz_in and, with a gate row per row, the gate).
// A row's stage is refilled after the next row's barrier: no thread can still be reading it then.
// While the gate row stays the same only N = sum dz y r_y is kept: dw_post += alpha g N and dgate =
// alpha w_p N at the segment's end (the segments and their partials as in the column kernel above).
struct RingPlan {
  int threads, stages, ctas;          // ctas: per SM
  int vectors, rows;                  // of 8 columns a thread, and rows a barrier
  int arrays, half;                   // input rows a row; where a pair of CTAs splits it (0: one takes it all)
  uint32_t stage_bytes;
};
constexpr int kMaxStages = 6, kRingThreads = 512;   // 16384 x 4096 bf16: 4 stages 172 us, 6 and more 128

// The column sums are formed also for a call that asks for none (16384 x 4096 bf16, frozen weights: 122.6 us, and
// 126.6 with both weights' gradients; floor 118).
// FULL: both gradients come in and dx and dy go out, so nothing of that is asked in the loop (126
// against 140 us at 16384 x 4096 bf16).
// K vectors of 8 columns a thread, R rows a barrier.  pl.half != 0: a cluster of two CTAs shares a row, the
// first takes its columns up to half; each adds the other's sums to its own, which they leave in each other's
// shared memory (4096 x 8192 fp32: 179 us against 290 with a pass over rows and one over columns; the cluster
// barrier is about 1 us a row).
template <typename T, int K, int R, int Y, bool TOKEN, bool FULL>
__global__ void __launch_bounds__(kRingThreads) norm_bwd_ring_kernel(const NormArgs a, const RingPlan pl) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  constexpr int N = R == 1 ? 4 : 8;   // three sums a row, rounded up
  constexpr bool HAS_Y = Y != NO_Y;
  extern __shared__ __align__(128) char ring[];
  __shared__ __align__(8) uint64_t full[kMaxStages];
  __shared__ __align__(16) float red[2 * 16 * N];
  __shared__ int abort_flag;
  __shared__ float other[2][N + 1];   // the other CTA's sums, and whether it has to stop
  const int rank = pl.half ? (int)cluster_ctarank() : 0, part = pl.half ? blockIdx.x >> 1 : blockIdx.x, S = pl.stages;
  const int D = (int)a.D, base = rank ? pl.half : 0, mine = !pl.half ? D : rank ? D - pl.half : pl.half;
  const int64_t r0 = part * a.rp, r1 = min(a.M, r0 + a.rp);
  const bool post = Y == POST_Y || (Y == ANY_Y && a.post);
  const bool has_dh = FULL || a.dh, has_dzi = FULL || a.dzi, has_dx = FULL || a.dx, has_dy = FULL || a.dy;
  const T* gate = static_cast<const T*>(a.gate);

  auto issue = [&](int64_t row, int s) {   // thread 0: the row's copies into stage s
    if (row >= r1) return;
    char* dst = ring + (size_t)s * pl.stage_bytes;
    const uint32_t bytes = (uint32_t)mine * sizeof(T);
    mbar_expect_tx(&full[s], pl.arrays * bytes);
    auto copy = [&](const void* src, int64_t ld) {
      bulk_load(dst, static_cast<const T*>(src) + row * ld + base, bytes, &full[s]);
      dst += bytes;
    };
    copy(a.x, a.ldx);
    if (has_dh) copy(a.dh, a.ldh);
    if (has_dzi) copy(a.dzi, a.ldo);
    if (HAS_Y) copy(a.y, a.ldy);
    if (TOKEN) copy(a.gate, a.D);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    mbar_fence_init();
    abort_flag = 0;
    for (int i = 0; i < S; ++i) issue(r0 + i, i);
  }
  __syncthreads();
  if (R == 1 && pl.half) cluster_sync_all();   // before anything is left in the other CTA it has to run

  // column of this thread's k-th vector among the CTA's, past `mine` nothing is read or written; and in the row
  const auto col = [&](int k) { return (k * (int)blockDim.x + (int)threadIdx.x) * 8; };
  const auto gcol = [&](int k) { return base + col(k); };
  F2 wz[K][4], u[K][4], dw[K][4], acc[K][4];   // u = alpha g w_p (TOKEN: alpha w_p); acc: N (TOKEN: dw_post)
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[k][i] = acc[k][i] = wz[k][i] = u[k][i] = f2(0.f);
    if (col(k) >= mine) continue;
    weight4x2<T>(a.w_pre, gcol(k), a.off, wz[k]);
    if (TOKEN) {
      weight4x2<T>(post ? a.w_post : nullptr, gcol(k), a.off, u[k]);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[k][i] = mul2(u[k][i], f2(a.alpha));
    }
  }
  auto begin_segment = [&](int64_t grp) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (col(k) >= mine) continue;
      F2 w[4];
      gate4x2<T>(gate ? gate + grp * D : nullptr, gcol(k), a.alpha, u[k]);
      weight4x2<T>(post ? a.w_post : nullptr, gcol(k), a.off, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[k][i] = mul2(u[k][i], w[i]);
    }
  };
  auto end_segment = [&](int64_t seg0, int64_t grp) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (col(k) >= mine) continue;
      F2 w[4];
      if (a.dgate) {
        weight4x2<T>(post ? a.w_post : nullptr, gcol(k), a.off, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = mul2(mul2(w[i], f2(a.alpha)), acc[k][i]);
        const int64_t g0 = grp * a.rpg, g1 = min(a.M, g0 + a.rpg);
        if (g0 >= r0 && g1 <= r1) store4x2(static_cast<T*>(a.dgate) + grp * D + gcol(k), w);
        else store4x2(a.pg + ((int64_t)part * 2 + (seg0 == r0 ? 0 : 1)) * D + gcol(k), w);
      }
      if (a.pp) {   // the part's own partial sum grows by a segment; no one else touches it
        float* pp = a.pp + (int64_t)part * D + gcol(k);
        F2 sum[4];
        if (seg0 != r0) load4x2(pp, sum);
        gate4x2<T>(gate ? gate + grp * D : nullptr, gcol(k), a.alpha, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = fma2(w[i], acc[k][i], seg0 != r0 ? sum[i] : f2(0.f));
        store4x2(pp, sum);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[k][i] = f2(0.f);
    }
  };

  // the arrays of a stage, in the order of the copies
  const int at_o = 1 + has_dh, at_y = at_o + has_dzi;
  const float inv_d = 1.f / (float)D;
  float r_z[R], r_y[R], r_z2[R], r_y2[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t at = min(r0 + r, r1 - 1);
    r_z2[r] = has_dh ? a.r_pre[at] : 0.f;
    r_y2[r] = post ? a.r_post[at] : 1.f;
  }
  int s = 0, flip = 0, refill = 0;   // refill (thread 0): the stage of the next row to ask for, `next`
  uint32_t parity = 0;
  int64_t next = r0 + S;
  int64_t row = r0, seg0 = r0, seg_end = r0, grp = 0;
  int rows = 0;
  for (; row < r1; row += rows) {
    if (HAS_Y && !TOKEN && row == seg_end) {   // uniform over the CTA
      if (row > r0) end_segment(seg0, grp);
      grp = row / a.rpg;
      seg0 = row;
      seg_end = min(r1, (grp + 1) * a.rpg);
      begin_segment(grp);
    }
    rows = (int)min((int64_t)R, (HAS_Y && !TOKEN ? seg_end : r1) - row);
    bool bad = false;
    float sums[N];   // of row r at 3 r: S1, S2, S3 of the row kernel above
#pragma unroll
    for (int i = 0; i < N; ++i) sums[i] = 0.f;
    F2 z[4], t[R][4], y[4], g[4];
    const T* st[R] = {};
    // z, t = dz_in + r_z w_z dh and y of a vector; the first time also what the sums need of dh
    auto load_zty = [&](int r, int k, F2* s0) {
      load4x2(st[r] + col(k), z);
      if (has_dzi) load4x2(st[r] + at_o * mine + col(k), t[r]);
      if (has_dh) {
        F2 h[4];
        load4x2(st[r] + mine + col(k), h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 rh = mul2(h[i], f2(r_z[r])), wh = mul2(rh, wz[k][i]);
          if (s0) {
            *s0 = fma2(wh, z[i], *s0);
            dw[k][i] = fma2(rh, z[i], dw[k][i]);
          }
          t[r][i] = has_dzi ? add2(t[r][i], wh) : wh;
        }
      }
      if (HAS_Y) load4x2(st[r] + at_y * mine + col(k), y);
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
      r_z[r] = r_z2[r], r_y[r] = r_y2[r];
      const int64_t at = min(row + rows + r, r1 - 1);
      r_z2[r] = has_dh ? a.r_pre[at] : 0.f;
      r_y2[r] = post ? a.r_post[at] : 1.f;
      const int sr = s + r < S ? s + r : s + r - S;
      st[r] = reinterpret_cast<const T*>(ring + (size_t)sr * pl.stage_bytes);
      if (r >= rows) continue;
      bad |= !mbar_wait(&full[sr], s + r < S ? parity : parity ^ 1, a.timeout_ns, &abort_flag, a.err, 40);
      if (bad) continue;
      F2 s0 = f2(0.f), s1 = f2(0.f), s2 = f2(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (col(k) >= mine) continue;
        load_zty(r, k, &s0);
        if (!post) continue;
        if (TOKEN) load4x2(st[r] + (at_y + 1) * mine + col(k), g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 uy = mul2(TOKEN ? mul2(u[k][i], g[i]) : u[k][i], y[i]);
          s1 = fma2(uy, t[r][i], s1);
          s2 = fma2(uy, z[i], s2);
        }
      }
      sums[3 * r] = sum2(s0);
      sums[3 * r + 1] = sum2(s1);
      sums[3 * r + 2] = sum2(s2);
    }
    bool stop = block_sums_of<N, 16>(sums, red, flip, bad);
    if (R == 1 && pl.half) {   // uniform over the cluster; only the variants with one row a barrier come in pairs
      if (threadIdx.x == 0) {
        const uint32_t to = mapa_shared(smem_u32(other[flip]), rank ^ 1);
#pragma unroll
        for (int i = 0; i <= N; ++i)
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * i), "f"(i < N ? sums[i] : stop ? 1.f : 0.f)
                       : "memory");
      }
      __syncwarp();
      cluster_sync_all();
#pragma unroll
      for (int i = 0; i < N; ++i) sums[i] += other[flip][i];
      stop |= other[flip][N] != 0.f;
    }
    flip ^= 1;
    if (stop) break;
    if (threadIdx.x == 0)   // the stages of all rows before `row` are free now
      for (; next < row + S; ++next) {
        issue(next, refill);
        refill = refill + 1 < S ? refill + 1 : 0;
      }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) continue;
      // s0 was summed over r_z w_z dh z
      const float cz = r_z[r] * r_z[r] * (sums[3 * r] * inv_d);
      const float cy = post ? r_y[r] * r_y[r] * r_y[r] * ((sums[3 * r + 1] - cz * sums[3 * r + 2]) * inv_d) : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (col(k) >= mine) continue;
        if (K > 1) {
          load_zty(r, k, nullptr);
        } else if (R > 1) {   // t stays in registers, z and y come from the stage again
          load4x2(st[r] + col(k), z);
          if (HAS_Y) load4x2(st[r] + at_y * mine + col(k), y);
        }
        const int64_t at = (row + r) * D + gcol(k);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[r][i] = fma2(f2(-cz), z[i], t[r][i]);
        if (has_dx) store4x2(static_cast<T*>(a.dx) + at, t[r]);
        if (!HAS_Y) continue;
        if (TOKEN) load4x2(st[r] + (at_y + 1) * mine + col(k), g);
        if (TOKEN && a.dgate_rows) {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = mul2(u[k][i], mul2(mul2(t[r][i], f2(r_y[r])), y[i]));
          store4x2(static_cast<T*>(a.dgate_rows) + at, z);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F2 e = mul2(t[r][i], f2(r_y[r]));
          if (TOKEN) acc[k][i] = fma2(mul2(mul2(g[i], f2(a.alpha)), e), y[i], acc[k][i]);
          else acc[k][i] = fma2(e, y[i], acc[k][i]);
          y[i] = fma2(TOKEN ? mul2(u[k][i], g[i]) : u[k][i], e, mul2(f2(-cy), y[i]));
        }
        if (has_dy) store4x2(static_cast<T*>(a.dy) + at, y);
      }
    }
    s += rows;
    if (s >= S) {
      s -= S;
      parity ^= 1;
    }
  }
  if (row < r1) {   // a wait ran out (every thread is here): let the copies in flight land, then leave
    if (threadIdx.x == 0)
      for (int64_t k = row; k < min(r1, next); ++k)
        mbar_wait_drain(&full[(k - r0) % S], (uint32_t)((k - r0) / S) & 1, 100000000ull);
    __syncthreads();
    if (R == 1 && pl.half) cluster_sync_all();
    return;
  }
  __syncthreads();
  if (R == 1 && pl.half) cluster_sync_all();   // the other CTA may still write here
  if (HAS_Y && !TOKEN) end_segment(seg0, grp);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (col(k) >= mine) continue;
    if (a.pw) store4x2(a.pw + (int64_t)part * D + gcol(k), dw[k]);
    if (TOKEN && a.pp) store4x2(a.pp + (int64_t)part * D + gcol(k), acc[k]);
  }
}

// ------------------------------------------------------------------ backward in one pass, short rows
// G lanes take a row, so its sums need no barrier, or one among the warps of a group; the L groups of a CTA's
// eight warps take every L-th row of its part.  Each lane keeps its own columns of its next rows on their way into
// shared memory, as the walk of the forward does.  The column sums stay in registers and are added over the groups
// when the gate row changes (N, as above) and at the end, so a CTA leaves one partial.  Against the ring, whose
// CTAs are many for short rows and leave a partial each: bf16, 131072 x 64 22 against 78 us, x 128 39 against 79,
// 16384 x 256 13 against 25, x 512 20 against 29, x 1024 38 against 41, 2000 x 256 with a gate per row 5.4 against
// 10.8; fp32 16384 x 256 19 against 26, x 512 36 against 40.  Bound by memory where rows are many (65536 x 512: 6.2
// TB/s).  A whole warp for 128 columns takes 59 us at 131072 rows, one for 512 (two vectors a lane, registers
// spilled) 25 at 16384; three CTAs an SM spill registers.  The groups of four warps (520 columns on) spill 16 to 32 bytes as they
// are, but with a gate row per row.  FULL as above (16384 x 256: 13.2 against 14.7 us).  The column sums are formed
// also for a call that asks for none of them (16384 x 256: 9.6 us then, 12.4 with them and the second launch).
constexpr int kShortThreads = 256;
template <typename T, bool TOKEN>
constexpr int short_stages() { return sizeof(T) == 2 ? 4 : TOKEN ? 2 : 3; }
template <typename T, int G, bool TOKEN>
size_t short_smem(int64_t D) {
  return kShortThreads / G * D * (short_stages<T, TOKEN>() * (TOKEN ? 5 : 4) * sizeof(T) + sizeof(float));
}

template <typename T, int G, bool TOKEN, bool FULL>
__global__ void __launch_bounds__(kShortThreads, 2) norm_bwd_short_kernel(const NormArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  constexpr int L = kShortThreads / G, Q = G > 32 ? G / 32 : 1;   // groups; columns a thread adds over them
  constexpr int S = short_stages<T, TOKEN>(), A = TOKEN ? 5 : 4;   // z, dh, dz_in, y, gate
  extern __shared__ __align__(16) char stages[];
  __shared__ __align__(16) float4 red[2][kShortThreads / 32];   // of a warp, for groups of several
  const int D = (int)a.D, lane = threadIdx.x % G, group = threadIdx.x / G, c = lane * 8;   // c: this lane's columns
  const bool in = c < D;
  const int64_t part = blockIdx.x, r0 = part * a.rp, r1 = min(a.M, r0 + a.rp);
  const bool has_y = FULL || a.y, has_dh = FULL || a.dh, has_dzi = FULL || a.dzi;
  const bool has_dx = FULL || a.dx, has_dy = FULL || a.dy;
  const bool post = has_y && a.post;
  const T* gate = static_cast<const T*>(a.gate);
  float* const sums = reinterpret_cast<float*>(stages + (size_t)L * S * A * D * sizeof(T));   // [L][D]
  T* const ring = reinterpret_cast<T*>(stages) + group * S * A * D + c;
  int fill = 0, used = 0;   // where in the ring the next row goes, and the row in hand is
  auto issue = [&](int64_t row) {   // this lane's columns of a row; a group even past the end
    if (row < r1 && in) {
      auto copy = [&](int at, const void* src, int64_t ld) {
        const T* from = static_cast<const T*>(src) + row * ld + c;
#pragma unroll
        for (int e = 0; e < 8; e += 16 / (int)sizeof(T)) cp_async16(ring + fill + at * D + e, from + e, true);
      };
      copy(0, a.x, a.ldx);
      if (has_dh) copy(1, a.dh, a.ldh);
      if (has_dzi) copy(2, a.dzi, a.ldo);
      if (has_y) copy(3, a.y, a.ldy);
      if (TOKEN) copy(4, a.gate, a.D);
    }
    cp_async_commit();
    fill += A * D;
    if (fill == S * A * D) fill = 0;
  };
  int64_t row = r0 + group;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(row + i * L);
  F2 wz[4], u[4], dw[4], acc[4];   // u = alpha g w_p (TOKEN: alpha w_p); acc: N (TOKEN: dw_post)
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[i] = acc[i] = f2(0.f);
  if (in) weight4x2<T>(a.w_pre, c, a.off, wz);
  // thread t: the sums over the groups of columns t, t + 256, ..
  auto over_groups = [&](F2 (&v)[4], float (&t)[Q]) {
    if (in) store4x2(sums + group * D + c, v);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int col = q * kShortThreads + (int)threadIdx.x;
      t[q] = 0.f;
      if (col < D)
#pragma unroll 8
        for (int l = 0; l < L; ++l) t[q] += sums[l * D + col];
    }
    __syncthreads();
  };
  const float inv_d = 1.f / (float)D;
  float dpost[Q], t1[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) dpost[q] = 0.f;
  int flip = 0;
  const auto factor = [&](const float* r, bool has, float other, int64_t at) { return has ? r[min(at, r1 - 1)] : other; };
  float r_z2 = factor(a.r_pre, has_dh, 0.f, row), r_y2 = factor(a.r_post, post, 1.f, row);
  for (int64_t seg0 = r0, seg_end; seg0 < r1; seg0 = seg_end) {   // rows of one gate row, uniform over the CTA
    const int64_t grp = TOKEN ? 0 : seg0 / a.rpg;
    seg_end = TOKEN ? r1 : min(r1, (grp + 1) * a.rpg);
    if (in) {
      F2 w[4];
      weight4x2<T>(post ? a.w_post : nullptr, c, a.off, u);
      gate4x2<T>(!TOKEN && gate ? gate + grp * D : nullptr, c, a.alpha, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = mul2(u[i], w[i]);
    }
    // a warp stays while one of its groups has a row
    for (bool mine; mine = row < seg_end, G >= 32 ? mine : __any_sync(0xffffffffu, mine);) {
      const float r_z = r_z2, r_y = r_y2;
      const T* use = ring + used;
      if (mine) {
        issue(row + (S - 1) * L);   // into the stage that the last row left
        r_z2 = factor(a.r_pre, has_dh, 0.f, row + L), r_y2 = factor(a.r_post, post, 1.f, row + L);
        cp_async_wait<S - 1>();
      }
      F2 z[4], y[4], g[4], t[4], s0 = f2(0.f), s1 = f2(0.f), s2 = f2(0.f);   // t = dz_in + r_z w_z dh
      if (mine && in) {
        load4x2(use, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = f2(0.f);
        if (has_dzi) load4x2(use + 2 * D, t);
        if (has_dh) {
          load4x2(use + D, g);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const F2 rh = mul2(g[i], f2(r_z)), wh = mul2(rh, wz[i]);
            s0 = fma2(wh, z[i], s0);
            dw[i] = fma2(rh, z[i], dw[i]);
            t[i] = add2(t[i], wh);
          }
        }
        if (has_y) load4x2(use + 3 * D, y);
        if (TOKEN) load4x2(use + 4 * D, g);
        if (post)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const F2 uy = mul2(TOKEN ? mul2(u[i], g[i]) : u[i], y[i]);
            s1 = fma2(uy, t[i], s1);
            s2 = fma2(uy, z[i], s2);
          }
      }
      float s[4] = {sum2(s0), sum2(s1), sum2(s2), 0.f};
      if (G <= 32) {
        spread<4, G <= 32 ? G : 32>(warp_sums_of<4, G <= 32 ? G : 32>(s), s);
      } else {   // one barrier a row of the group's warps: a warp that runs ahead writes the other half
        spread<4>(warp_sums_of<4>(s), s);
        if ((threadIdx.x & 31) == 0) red[flip][threadIdx.x >> 5] = make_float4(s[0], s[1], s[2], 0.f);
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(G) : "memory");
        s[0] = s[1] = s[2] = 0.f;
#pragma unroll
        for (int w = 0; w < Q; ++w) {
          const float4 o = red[flip][group * Q + w];
          s[0] += o.x, s[1] += o.y, s[2] += o.z;
        }
        flip ^= 1;
      }
      if (!mine) continue;
      const float cz = r_z * r_z * (s[0] * inv_d);   // s0 was summed over r_z w_z dh z
      const float cy = post ? r_y * r_y * r_y * ((s[1] - cz * s[2]) * inv_d) : 0.f;
      if (in) {
        const int64_t at = row * D + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = fma2(f2(-cz), z[i], t[i]);
        if (has_dx) store4x2(static_cast<T*>(a.dx) + at, t);
        if (TOKEN && a.dgate_rows) {
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = mul2(u[i], mul2(mul2(t[i], f2(r_y)), y[i]));
          store4x2(static_cast<T*>(a.dgate_rows) + at, z);
        }
        if (has_y) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const F2 e = mul2(t[i], f2(r_y));
            if (TOKEN) acc[i] = fma2(mul2(mul2(g[i], f2(a.alpha)), e), y[i], acc[i]);
            else acc[i] = fma2(e, y[i], acc[i]);
            y[i] = fma2(TOKEN ? mul2(u[i], g[i]) : u[i], e, mul2(f2(-cy), y[i]));
          }
          if (has_dy) store4x2(static_cast<T*>(a.dy) + at, y);
        }
      }
      row += L;
      used += A * D;
      if (used == S * A * D) used = 0;
    }
    if (TOKEN || !(a.dgate || a.pp)) continue;
    over_groups(acc, t1);
    const int64_t g0 = grp * a.rpg, g1 = min(a.M, g0 + a.rpg);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f2(0.f);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int col = q * kShortThreads + (int)threadIdx.x;
      if (col >= D) continue;
      const float gc = gate ? to_f<T>(gate[grp * D + col]) : 1.f;
      dpost[q] = fmaf(a.alpha * gc, t1[q], dpost[q]);
      if (!a.dgate) continue;
      const float wp = post && a.w_post ? to_f<T>(static_cast<const T*>(a.w_post)[col]) + a.off : 1.f;
      const float dg = a.alpha * wp * t1[q];
      if (g0 >= r0 && g1 <= r1) static_cast<T*>(a.dgate)[grp * D + col] = from_f<T>(dg);
      else a.pg[(part * 2 + (seg0 == r0 ? 0 : 1)) * D + col] = dg;
    }
  }
  auto leave = [&](float* to, const float (&v)[Q]) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int col = q * kShortThreads + (int)threadIdx.x;
      if (col < D) to[part * D + col] = v[q];
    }
  };
  if (a.pp) {
    if (TOKEN) over_groups(acc, dpost);
    leave(a.pp, dpost);
  }
  if (a.pw) {
    over_groups(dw, t1);
    leave(a.pw, t1);
  }
}

// ------------------------------------------------------------------ backward: sums of the partials
// CTA (t, j): columns 32 t .. 32 t + 31, one per lane.  j = 0: dw_pre, 1: dw_post, the warps sharing
// the parts.  Past that the gate rows that more than one part has rows of: GATE_CTA one a CTA in the same way
// (few gate rows, many parts each), GATE_WARP one a warp, GATE_BOUND (more gate rows than boundaries between
// parts) a warp takes the gate row that crosses a boundary, if that boundary is its first.
enum { GATE_NONE = 0, GATE_CTA = 1, GATE_WARP = 2, GATE_BOUND = 3 };

template <typename T, int HOW>
__global__ void __launch_bounds__(1024) norm_bwd_finish_kernel(const NormArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  const int job = (int)blockIdx.y - 2;
  // partials first, first + step, .. last of this warp, ten loads at a time, so that 32 warps have 320 on their
  // way (304 parts: 24.6 against 25.4 us with eight, 4096 x 2048); slot(p) is where part p keeps this sum
  auto add = [&](int first, int last, int step, auto slot) {
    float t = 0.f;
    if (col < a.D)
      for (int p = first; p <= last; p += 10 * step) {
        float v[10];
#pragma unroll
        for (int j = 0; j < 10; ++j) v[j] = p + j * step <= last ? slot(p + j * step)[col] : 0.f;
#pragma unroll
        for (int j = 0; j < 10; ++j) t += v[j];
      }
    return t;
  };
  auto parts_of = [&](int64_t grp, int& first, int& last) {
    const int64_t g0 = grp * a.rpg, g1 = min(a.M, g0 + a.rpg);
    first = (int)(g0 / a.rp);
    last = (int)((g1 - 1) / a.rp);
  };
  // its first part keeps a gate row in slot 1 unless it begins with it, the others begin with it
  auto gate_slot = [&](int64_t grp, int first) {
    const int late = grp * a.rpg > (int64_t)first * a.rp;
    return [&a, first, late](int p) { return a.pg + ((int64_t)p * 2 + (p == first ? late : 0)) * a.D; };
  };
  T* out;
  float t;
  if (HOW == GATE_NONE || job < 0) {
    const float* src = job == -2 ? a.pw : a.pp;
    out = static_cast<T*>(job == -2 ? a.dw_pre : a.dw_post);
    if (!out) return;
    t = add(warp, a.parts - 1, warps, [&](int p) { return src + (int64_t)p * a.D; });
  } else if (HOW == GATE_CTA) {
    int first, last;
    parts_of(job, first, last);
    if (first == last) return;   // written by its one part
    out = static_cast<T*>(a.dgate) + (int64_t)job * a.D;
    t = add(first + warp, last, warps, gate_slot(job, first));
  } else {
    const int64_t item = (int64_t)job * warps + warp, b = (item + 1) * a.rp;   // b: the first row of part item + 1
    const int64_t grp = HOW == GATE_WARP ? item : b / a.rpg;
    if (grp * a.rpg >= a.M || (HOW == GATE_BOUND && item + 1 >= a.parts)) return;
    int first, last;
    parts_of(grp, first, last);
    if (first == last || (HOW == GATE_BOUND && first != item)) return;
    t = add(first, last, 1, gate_slot(grp, first));
    if (col < a.D) static_cast<T*>(a.dgate)[grp * a.D + col] = from_f<T>(t);
    return;
  }
  acc[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && col < a.D) {
    t = 0.f;
    for (int w = 0; w < warps; ++w) t += acc[w][lane];
    out[col] = from_f<T>(t);
  }
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

// Ring plan of the one-pass backward with n input rows a row, or threads == 0 where no variant holds
// them: those take the row and column kernels.  Small rows get several CTAs an SM (the 128 registers a
// thread allow 512 threads), rows too long for one CTA a pair of them.  Two rows a barrier take four
// stages, one row three.
RingPlan ring_plan(const lora_norm_shape& sh, int n) {
  const bool narrow = sh.dtype == LORA_BF16;
  const int64_t es = narrow ? 2 : 4;
  const auto budget = [](int ctas) { return (int64_t)(kSmSmem / ctas - kRingStatic); };
  for (int pair = 0; pair < 2; ++pair) {
    const int64_t vecs = pair ? (sh.D / 8 + 1) / 2 : sh.D / 8, stage = n * vecs * 8 * es;
    RingPlan p = {};
    p.vectors = vecs <= kRingThreads && !(pair && narrow) ? 1 : 2;
    if (p.vectors == 2 && !narrow) continue;   // three stages of fp32 do not fit then
    p.threads = (int)((vecs + 32 * p.vectors - 1) / (32 * p.vectors) * 32);
    if (p.threads > kRingThreads) continue;
    p.ctas = pair ? 1 : (int)(kRingThreads / p.threads < 16 ? kRingThreads / p.threads : 16);
    while (p.ctas > 1 && 4 * stage > budget(p.ctas)) --p.ctas;
    const int64_t fit = budget(p.ctas) / stage;
    p.rows = p.vectors == 1 && fit >= 4 && !pair ? 2 : 1;
    if (fit < 3) continue;
    p.stages = (int)(fit < kMaxStages ? fit : kMaxStages);
    p.arrays = n;
    p.half = pair ? (int)vecs * 8 : 0;
    p.stage_bytes = (uint32_t)stage;
    return p;
  }
  return RingPlan{};
}

// Whether the rows are short (rpg: rows that share a gate row, 0 without a gate): half a CTA holds one, and a gate
// row's rows are all, or enough that the sum over the groups at its end costs less than it saves (16384 x 1024 bf16
// with 16 rows a gate 48 against 50 us with the ring, with 8 53 against 53; x 256 20 against 27, with 4 34 against 29).
// Five fp32 arrays of more than 512 columns leave too few rows on their way (16384 x 1024: 93 against 87 us).
bool short_rows(const lora_norm_shape& sh, int64_t rpg) {
  if (sh.D > (sh.dtype == LORA_F32 && rpg == 1 ? 512 : 1024)) return false;
  return rpg <= 1 || rpg >= 16 || rpg >= sh.M;
}

// Row parts of the column sums: one a resident CTA in the one-pass backwards; for the column kernel
// four CTAs per SM over all column tiles, at least 32 rows each.
void norm_parts(const lora_norm_shape& sh, bool brief, const RingPlan& ring, int64_t* rp, int* parts) {
  int64_t want;
  if (brief) {
    want = 2 * num_sms_current();
    // least rows of a part (300 x 1024: 5.3 us with 2 and 4, 6.4 with 8; 2000 x 512: 7.4 with 4, 6.8 with 8)
    const int64_t least = sh.D > 512 ? 4 : 8;
    if (want > (sh.M + least - 1) / least) want = (sh.M + least - 1) / least;
  } else if (ring.threads) {
    want = (int64_t)ring.ctas * num_sms_current() / (ring.half ? 2 : 1);
    if (want > sh.M) want = sh.M;
  } else {
    const int64_t tiles = (sh.D + 255) / 256;
    want = (4LL * num_sms_current() + tiles - 1) / tiles;
    if (want > (sh.M + 31) / 32) want = (sh.M + 31) / 32;
  }
  if (want < 1) want = 1;
  *rp = (sh.M + want - 1) / want;
  if (*rp < 1) *rp = 1;
  *parts = (int)((sh.M + *rp - 1) / *rp);
}

struct NormBwdWs {
  uint32_t* err;
  float *crow, *pw, *pp, *pg;
};
size_t plan_norm_bwd(const lora_norm_shape& sh, char* base, int parts, NormBwdWs* w) {
  Carve c{base};
  w->err = c.take<uint32_t>(kErrBytes / 4);
  w->crow = c.take<float>((size_t)sh.M);
  w->pw = c.take<float>((size_t)parts * sh.D);
  w->pp = c.take<float>((size_t)parts * sh.D);
  w->pg = c.take<float>((size_t)parts * 2 * sh.D);
  return c.off;
}
// over the variants that a call may take: they depend on its inputs
int most_parts(const lora_norm_shape& sh) {
  int most = 0;
  for (int n = 0; n <= 5; ++n) {
    int64_t rp;
    int parts;
    norm_parts(sh, n == 0 && short_rows(sh, 0), n ? ring_plan(sh, n) : RingPlan{}, &rp, &parts);
    if (parts > most) most = parts;
  }
  return most;
}

NormArgs norm_args(const lora_norm_shape& sh, const void* x, const void* y, const void* w_pre, const void* w_post,
                   const void* gate) {
  NormArgs a = {};
  a.M = sh.M, a.D = sh.D;
  a.rpg = sh.M > 0 ? sh.M : 1;   // more rows a gate row than there are rows are all of them
  if (gate && sh.rows_per_gate < a.rpg) a.rpg = sh.rows_per_gate;
  a.ldx = sh.ldx, a.ldy = sh.ldy, a.ldh = sh.lddh, a.ldo = sh.lddz;
  a.x = x, a.y = y, a.w_pre = w_pre, a.w_post = w_post, a.gate = gate;
  a.alpha = sh.alpha, a.eps = sh.eps, a.off = sh.w_offset, a.post = sh.post_norm != 0;
  return a;
}

template <typename T, int K, int R, int Y, bool TOKEN, bool FULL>
cudaError_t launch_ring(const NormArgs& a, const RingPlan& p, cudaStream_t st) {
  const cudaError_t allowed = allow_smem<norm_bwd_ring_kernel<T, K, R, Y, TOKEN, FULL>>(kDynamicSmem);
  if (allowed != cudaSuccess) return allowed;
  const size_t smem = (size_t)p.stages * p.stage_bytes;
  if (!p.half)
    return launch_pdl(norm_bwd_ring_kernel<T, K, R, Y, TOKEN, FULL>, dim3((unsigned)a.parts), dim3((unsigned)p.threads),
                      smem, st, a, p);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(2 * (unsigned)a.parts);
  cfg.blockDim = dim3((unsigned)p.threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.numAttrs = 1 + pdl_attr(&attr[1]);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_bwd_ring_kernel<T, K, R, Y, TOKEN, FULL>, a, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename T, int K, int R>
cudaError_t launch_ring(const NormArgs& a, const RingPlan& p, cudaStream_t st) {
  const bool token = a.gate && a.rpg == 1;
  if (!a.y) return launch_ring<T, K, R, NO_Y, false, false>(a, p, st);
  if (!(a.dh && a.dzi && a.dx && a.dy))
    return token ? launch_ring<T, K, R, ANY_Y, true, false>(a, p, st) : launch_ring<T, K, R, ANY_Y, false, false>(a, p, st);
  if (a.post)
    return token ? launch_ring<T, K, R, POST_Y, true, true>(a, p, st) : launch_ring<T, K, R, POST_Y, false, true>(a, p, st);
  return token ? launch_ring<T, K, R, PLAIN_Y, true, true>(a, p, st) : launch_ring<T, K, R, PLAIN_Y, false, true>(a, p, st);
}
// The variants that ring_plan can ask for: bf16 rows always fit four stages up to 4096 columns (one vector a
// thread) and come in pairs above 8192, with all five inputs (a gate row per row) above 7640; fp32 ones above 4096 and
// 3816.  Beyond 16384 (15280) bf16 or 8192 (7632) fp32 columns there is none.
inline cudaError_t launch_plan(const NormArgs& a, const RingPlan& p, cudaStream_t st, bf16) {
  return p.vectors == 2 ? launch_ring<bf16, 2, 1>(a, p, st) : launch_ring<bf16, 1, 2>(a, p, st);
}
inline cudaError_t launch_plan(const NormArgs& a, const RingPlan& p, cudaStream_t st, float) {
  return p.rows == 2 ? launch_ring<float, 1, 2>(a, p, st) : launch_ring<float, 1, 1>(a, p, st);
}

template <typename T, int G, bool TOKEN, bool FULL>
cudaError_t launch_short(const NormArgs& a, cudaStream_t st) {
  const size_t smem = short_smem<T, G, TOKEN>(a.D);
  const auto kernel = norm_bwd_short_kernel<T, G, TOKEN, FULL>;
  const cudaError_t allowed = allow_smem<norm_bwd_short_kernel<T, G, TOKEN, FULL>>(kDynamicSmem);
  if (allowed != cudaSuccess) return allowed;
  return launch_pdl(kernel, dim3((unsigned)a.parts), dim3(kShortThreads), smem, st, a);
}
template <typename T, int G>
cudaError_t launch_short(const NormArgs& a, cudaStream_t st) {
  const bool token = a.gate && a.rpg == 1;
  if (a.y && a.dh && a.dzi && a.dx && a.dy)
    return token ? launch_short<T, G, true, true>(a, st) : launch_short<T, G, false, true>(a, st);
  return token ? launch_short<T, G, true, false>(a, st) : launch_short<T, G, false, false>(a, st);
}
template <typename T>
cudaError_t launch_short(const NormArgs& a, cudaStream_t st) {
  if (a.D <= 64) return launch_short<T, 8>(a, st);
  if (a.D <= 128) return launch_short<T, 16>(a, st);
  if (a.D <= 256) return launch_short<T, 32>(a, st);
  if (a.D <= 512) return launch_short<T, 64>(a, st);
  return launch_short<T, 128>(a, st);
}

template <typename T>
lora_status norm_bwd(NormArgs& a, bool brief, const RingPlan& ring, cudaStream_t st) {
  const bool sums = a.dw_pre || a.dw_post || a.dgate;
  if (a.M > 0 && brief) {
    CK(launch_short<T>(a, st));
  } else if (a.M > 0 && ring.threads) {
    CK(launch_plan(a, ring, st, T{}));
  } else if (a.M > 0) {
    CK(launch_pdl(norm_bwd_rows_kernel<T>, dim3((unsigned)a.M), dim3((unsigned)row_threads(a.D)), 0, st, a));
    if (sums)
      CK(launch_pdl(norm_bwd_cols_kernel<T>, dim3((unsigned)((a.D + 255) / 256), (unsigned)a.parts),
                    dim3(32 * kColWarps), 0, st, a));
  }
  if (!sums) return LORA_OK;
  int warps = (a.parts + 9) / 10;   // ten partials a warp
  warps = warps < 4 ? 4 : warps > 32 ? 32 : warps;
  const int64_t groups = a.dgate && a.parts > 1 ? (a.M + a.rpg - 1) / a.rpg : 0, bounds = a.parts - 1;
  int how = GATE_NONE;
  int64_t jobs = 2;
  if (groups > 0) {
    // with 64 parts a gate row a warp takes longer than the CTAs do to come and go (2000 x 256, 4 gate rows: 11.1
    // against 7.4 us), with 38 not (16384 x 4096: 130.6 against 131.5)
    how = groups > bounds ? GATE_BOUND : a.parts / groups > 48 ? GATE_CTA : GATE_WARP;
    jobs += how == GATE_CTA ? groups : ((how == GATE_BOUND ? bounds : groups) + warps - 1) / warps;
  }
  auto finish = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)((a.D + 31) / 32), (unsigned)jobs), dim3(32 * warps), 0, st, a);
  };
  cudaError_t e;
  if (how == GATE_NONE) e = finish(norm_bwd_finish_kernel<T, GATE_NONE>);
  else if (how == GATE_CTA) e = finish(norm_bwd_finish_kernel<T, GATE_CTA>);
  else if (how == GATE_WARP) e = finish(norm_bwd_finish_kernel<T, GATE_WARP>);
  else e = finish(norm_bwd_finish_kernel<T, GATE_BOUND>);
  CK(e);
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
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  CK(sh->dtype == LORA_BF16 ? norm_fwd<bf16>(a, st) : norm_fwd<float>(a, st));
  return LORA_OK;
}

size_t block_norm_bwd_workspace_bytes(const lora_norm_shape* sh) {
  NormBwdWs w;
  return check_norm(sh) == LORA_OK ? plan_norm_bwd(*sh, nullptr, most_parts(*sh), &w) : 0;
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
  const lora_status ew = check_ws(ws, ws_bytes, plan_norm_bwd(*sh, static_cast<char*>(ws), most_parts(*sh), &w));
  if (ew != LORA_OK) return ew;
  NormArgs a = norm_args(*sh, Xout, Y, w_pre, w_post, gate);
  const bool token = gate && a.rpg == 1;
  const RingPlan ring = ring_plan(*sh, 1 + (Y != nullptr) + (dH != nullptr) + (dXout != nullptr) + token);
  const bool brief = short_rows(*sh, gate ? a.rpg : 0);
  norm_parts(*sh, brief, ring, &a.rp, &a.parts);
  a.r_pre = const_cast<float*>(r_pre), a.r_post = const_cast<float*>(r_post);
  a.dh = dH, a.dzi = dXout, a.dx = dX, a.dy = dY;
  a.dw_pre = dw_pre, a.dw_post = dw_post;
  a.crow = w.crow;
  if (token) a.dgate_rows = dgate;   // a gate row per row: its gradient is an output of the row pass
  else a.dgate = dgate;
  a.err = w.err, a.timeout_ns = wait_timeout_ns();
  a.pw = dw_pre ? w.pw : nullptr;
  a.pp = dw_post ? w.pp : nullptr;
  a.pg = w.pg;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return sh->dtype == LORA_BF16 ? norm_bwd<bf16>(a, brief, ring, st) : norm_bwd<float>(a, brief, ring, st);
}

}  // extern "C"
