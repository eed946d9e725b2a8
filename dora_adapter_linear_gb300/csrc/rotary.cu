// Rotary positions: pair j < rot / 2 of every head of token i turns by t = pos[i] theta_j,
//   (a, b) -> scale (a cos t - b sin t, b cos t + a sin t),
// the backward by -t (the transpose).  A pair is (j, j + rot / 2) of the head in the half layout and
// (2 j, 2 j + 1) in the interleaved one; the rest of a head passes unchanged.
//
// The angle is kept in turns: freq[j] = theta_j / (2 pi) as a 64-bit binary fraction, so the low 64
// bits of pos freq[j] are the fraction of a turn, without a rounding of the product (an fp32 one
// would be off by 2^-24 of the angle: 0.008 rad at position 131072).  Its upper 32 bits, as a signed
// half-turn in [-1, 1), go to sincospif: the angle is within pi 2^-25 of pos times the one that freq[j]
// stands for.  What freq[j] itself is off by grows with the position: from fp64 arithmetic 1.5 2^-53 theta_j (2^-30
// rad at position 2^22, as much as pi 2^-25 at 2^29) and half a unit of the fraction, pi 2^-64.
// Bound by memory: each rotated element is read and written once.
#include <math.h>

#include "checks.h"
#include "vec.cuh"

namespace lg {

namespace {

struct RotArgs {
  int64_t M;
  int H, half, rest;            // heads, pairs of a head, elements past them to copy (0 in place)
  int64_t xt, xh, yt, yh;       // token and head strides of x and y, in elements
  const void *x, *pos;
  const uint64_t* freq;
  void* y;
  float scale;
  int pos64, inverse;
  int tokens;                   // of a CTA
};

// B bytes as they lie in memory, and as fp32
template <int B>
struct Bytes {
  uint32_t w[B < 4 ? 1 : B / 4];
};
template <int B, typename T>
__device__ __forceinline__ void load_b(const T* p, Bytes<B>& r) {
  if constexpr (B == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else if constexpr (B == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else if constexpr (B == 4) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}
template <int B, typename T>
__device__ __forceinline__ void store_b(T* p, const Bytes<B>& r) {
  if constexpr (B == 16) *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  else if constexpr (B == 8) *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
  else if constexpr (B == 4) *reinterpret_cast<uint32_t*>(p) = r.w[0];
  else *reinterpret_cast<uint16_t*>(p) = (uint16_t)r.w[0];
}
template <int B, typename T>
__device__ __forceinline__ void open_b(const Bytes<B>& r, float (&f)[B / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) f[i] = __uint_as_float(r.w[i]);
  } else if constexpr (B == 2) {
    f[0] = __uint_as_float(r.w[0] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) {
      const float2 t = unpack_bf16x2(r.w[i]);
      f[2 * i] = t.x, f[2 * i + 1] = t.y;
    }
  }
}
template <int B, typename T>
__device__ __forceinline__ void close_b(const float (&f)[B / sizeof(T)], Bytes<B>& r) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) r.w[i] = __float_as_uint(f[i]);
  } else if constexpr (B == 2) {
    r.w[0] = pack_bf16x2(f[0], 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < B / 4; ++i) r.w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  }
}

// A CTA takes `tokens` tokens: their angles, one sincospif for each pair of a token whatever the number of
// heads, go to shared memory; its threads walk over the items (token, head, vector).  An item is P pairs:
// two accesses of B bytes in the half layout, one in the interleaved one (two where B is a single
// element); the vectors of the passed part (RB bytes) follow them.  A thread has U items on their way, the first of
// them while the angles are formed.
template <typename T, int B, bool INTER, int RB>
__global__ void __launch_bounds__(512) rotary_kernel(const RotArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  constexpr int E = B / sizeof(T), ER = RB / sizeof(T);
  constexpr bool TWO = !INTER || E == 1;          // an item's pairs lie in two accesses
  constexpr int P = TWO ? E : E / 2, U = 2;
  extern __shared__ __align__(16) float2 cs[];    // [token][pair of the item][vector]: neighbours at neighbours
  const int nv = a.half / P, per = nv + a.rest / ER;
  const int64_t tok0 = (int64_t)blockIdx.x * a.tokens;
  const int toks = (int)min((int64_t)a.tokens, a.M - tok0);
  // this thread's items: every blockDim-th, as (token, head, vector) with carries instead of divisions
  const int all = toks * a.H * per, rows = a.H * per;
  int i = threadIdx.x;
  int t = i / rows, h = (i - t * rows) / per, v = i - t * rows - h * per;
  const int st = blockDim.x / rows, sh = (blockDim.x - st * rows) / per, sv = blockDim.x - st * rows - sh * per;
  const T* x = static_cast<const T*>(a.x) + tok0 * a.xt;
  T* y = static_cast<T*>(a.y) + tok0 * a.yt;
  static_assert(RB == B || RB == 2 * B, "the passed part is as wide or twice as wide");
  Bytes<RB> p[U];
  Bytes<B> q[U];
  T* out[U];
  int at[U];              // where the item's angles begin; -1: a vector that passes, -2: none
  auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = -2;
      if (i < all) {
        const bool turned = v < nv;
        const int c = turned ? (INTER ? 2 * P * v : P * v) : 2 * a.half + (v - nv) * ER;
        const T* in = x + t * a.xt + h * a.xh + c;
        out[u] = y + t * a.yt + h * a.yh + c;
        if (RB == B || !turned) load_b<RB, T>(in, p[u]);
        else load_b<B, T>(in, reinterpret_cast<Bytes<B>&>(p[u]));   // the first part of it
        if (TWO && turned) load_b<B, T>(in + (INTER ? 1 : a.half), q[u]);
        at[u] = turned ? t * a.half + v : -1;
      }
      i += blockDim.x;
      v += sv;
      if (v >= per) v -= per, ++h;
      h += sh;
      if (h >= a.H) h -= a.H, ++t;
      t += st;
    }
  };
  fetch();
  for (int k = threadIdx.x; k < toks * a.half; k += blockDim.x) {
    const int tk = k / a.half, j = k - tk * a.half;
    const int64_t pos = a.pos64 ? static_cast<const int64_t*>(a.pos)[tok0 + tk] : static_cast<const int32_t*>(a.pos)[tok0 + tk];
    const int32_t turn = (int32_t)(((uint64_t)pos * a.freq[j]) >> 32);   // 2 x the fraction of a turn, x 2^31, signed
    float s, c;
    sincospif((float)turn * 0x1p-31f, &s, &c);
    s *= a.scale;
    cs[tk * a.half + (j % P) * nv + j / P] = make_float2(c * a.scale, a.inverse ? -s : s);
  }
  __syncthreads();
  while (at[0] != -2) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at[u] == -2) continue;
      if (at[u] >= 0) {
        Bytes<B>& first = reinterpret_cast<Bytes<B>&>(p[u]);
        float f[E], g[E];
        open_b<B, T>(first, f);
        if (TWO) open_b<B, T>(q[u], g);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 r = cs[at[u] + e * nv];
          float& m = TWO ? f[e] : f[2 * e];
          float& n = TWO ? g[e] : f[(2 * e + 1) % E];
          const float m0 = m;
          // written out: the same bits whatever the variant
          m = fmaf(m0, r.x, -(n * r.y));
          n = fmaf(n, r.x, m0 * r.y);
        }
        close_b<B, T>(f, first);
        if (TWO) {
          close_b<B, T>(g, q[u]);
          store_b<B, T>(out[u] + (INTER ? 1 : a.half), q[u]);
        }
        store_b<B, T>(out[u], first);
      } else {
        store_b<RB, T>(out[u], p[u]);
      }
    }
    fetch();
  }
}

template <typename T, int B, bool INTER, int RB>
cudaError_t launch(const RotArgs& a, cudaStream_t st) {
  constexpr int E = B / (int)sizeof(T), ER = RB / (int)sizeof(T), P = INTER && E > 1 ? E / 2 : E;
  const int64_t items = (int64_t)a.H * (a.half / P + a.rest / ER);   // of a token
  // A CTA reads about 40 KB (16384 x 40 heads of 128, bf16: 50 us in the half layout with 40 KB, 51 with 20 and
  // 55 with 160; 54 us in the interleaved one with 40 KB, 58 with 20), but rather there are two for every SM.
  RotArgs r = a;
  int64_t tokens = 40960 / (items * B * (INTER && E > 1 ? 1 : 2));
  const int64_t fit = 16384 / (a.half * (int64_t)sizeof(float2)), spread = a.M / (2 * num_sms_current());
  if (tokens > fit) tokens = fit;
  if (tokens > spread) tokens = spread;
  r.tokens = (int)(tokens < 1 ? 1 : tokens);
  const int64_t mine = items * r.tokens;
  const int threads = mine >= 512 ? 256 : (int)((mine + 31) / 32 * 32);
  const dim3 grid((unsigned)((a.M + r.tokens - 1) / r.tokens));
  const size_t smem = (size_t)r.tokens * a.half * sizeof(float2);
  return launch_pdl(rotary_kernel<T, B, INTER, RB>, grid, dim3((unsigned)threads), smem, st, r);
}
// heads: what the passed part's accesses have to divide.  It begins at twice a half, so where a half keeps
// its accesses below 16 bytes the passed part may take twice as much (8192 x 12 heads of 72, 18 turned: 18.5
// against 33 us).
template <typename T, int B>
cudaError_t launch(const RotArgs& a, bool inter, uintptr_t heads, cudaStream_t st) {
  if (inter) return launch<T, B, true, B>(a, st);
  if constexpr (B < 16)
    if (a.rest && heads % (2 * B) == 0) return launch<T, B, false, 2 * B>(a, st);
  return launch<T, B, false, B>(a, st);
}

// Whether a head of x and one of y, which begins d elements after x, share an element.  A head is hd consecutive
// elements, and y's heads are apart: o is the dimension of its larger stride, i the other.  A head of x at p, counted
// from y's begin, can only meet y's rows (over o) at p / stride and at the next one.  With the same outer stride in
// both, as columns of one packed projection have, all rows of x are alike and one stands for them; with the same
// inner one as well, so are all heads of a row.
struct Dim {
  int64_t n, stride;
};
bool heads_meet(Dim xo, Dim xi, Dim yo, Dim yi, int64_t hd, int64_t d) {
  typedef __int128 wide;    // a caller's strides are not bounded
  for (Dim* t : {&xo, &xi})
    if (t->stride == 0) t->n = 1;         // the same head again and again
  for (Dim* t : {&xo, &xi, &yo, &yi})
    if (t->n == 1) t->stride = INT64_MAX;   // of no use: 0 is its only index
  const auto span = [](Dim t) { return (wide)(t.n - 1) * (t.n == 1 ? 0 : t.stride); };
  if (d >= span(xo) + span(xi) + hd || d + span(yo) + span(yi) + hd <= 0) return false;
  const bool alike = xo.n == yo.n && xo.stride == yo.stride, all_alike = alike && xi.n == yi.n && xi.stride == yi.stride;
  const auto floor_div = [](wide a, wide b) { return a >= 0 ? a / b : -((b - 1 - a) / b); };
  const auto row_meets = [&](wide p) {   // a head at p and the heads of y's row that begins at 0
    if (p + hd <= 0) return false;
    wide j = (p + hd - 1) / yi.stride;   // the last one that begins before the head ends
    if (j > yi.n - 1) j = yi.n - 1;
    return j * yi.stride + hd > p;
  };
  if (all_alike) {   // m heads and k rows between two that meet
    const wide rows = floor_div(-(wide)d, yo.stride);
    for (wide k = rows - 1; k <= rows + 1; ++k) {
      const wide r = -d - k * yo.stride, heads = floor_div(-r, yi.stride);
      for (wide m = heads; m <= heads + 1; ++m)
        if (k > -yo.n && k < yo.n && m > -yi.n && m < yi.n && m * yi.stride + r < hd && m * yi.stride + r > -hd) return true;
    }
    return false;
  }
  for (int64_t a = 0; a < (alike ? 1 : xo.n); ++a)
    for (int64_t b = 0; b < xi.n; ++b) {
      const wide p = (wide)a * xo.stride + (wide)b * xi.stride - d, first = floor_div(p, yo.stride);
      for (wide k = first; k <= first + 1; ++k)
        if ((alike ? k > -yo.n && k < yo.n : k >= 0 && k < yo.n) && row_meets(p - k * yo.stride)) return true;
    }
  return false;
}

lora_status rotary(const lora_rotary_shape* sh, const void* X, const void* pos, const uint64_t* freq, void* Y,
                   bool inverse, void* stream) {
  if (!sh) return LORA_ERR_INVALID_ARG;
  if (sh->M < 0 || sh->H < 1 || sh->rot_dim < 2 || sh->rot_dim > sh->head_dim || sh->rot_dim % 2)
    return LORA_ERR_INVALID_ARG;
  if (sh->dtype != LORA_F32 && sh->dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
  if (sh->layout != LORA_ROTARY_HALF && sh->layout != LORA_ROTARY_INTERLEAVED) return LORA_ERR_INVALID_ARG;
  if (sh->pos_bits != 32 && sh->pos_bits != 64) return LORA_ERR_INVALID_ARG;
  if (!isfinite(sh->scale)) return LORA_ERR_INVALID_ARG;
  if (sh->M > (1LL << 31) - 1 || sh->head_dim > (1 << 12) || sh->H > (1LL << 30) / sh->head_dim)
    return LORA_ERR_UNSUPPORTED;
  REQ(freq);
  if (sh->M > 0 && (!X || !pos || !Y)) return LORA_ERR_INVALID_ARG;
  // no two elements of y at one address (x may repeat a head or a token); in place: the same layout
  const auto apart = [](int64_t n, int64_t s, int64_t inner) { return n <= 1 || s >= inner; };
  const int64_t hd = sh->head_dim, M = sh->M, H = sh->H;
  if (sh->x_token < 0 || sh->x_head < 0 || sh->y_token < 0 || sh->y_head < 0) return LORA_ERR_INVALID_ARG;
  const bool token_outer = apart(H, sh->y_head, hd) && apart(M, sh->y_token, (H - 1) * sh->y_head + hd);
  if (!token_outer &&
      !(apart(M, sh->y_token, hd) && apart(H, sh->y_head, (M - 1) * sh->y_token + hd)))
    return LORA_ERR_INVALID_ARG;
  if (X == Y && ((M > 1 && sh->x_token != sh->y_token) || (H > 1 && sh->x_head != sh->y_head)))
    return LORA_ERR_INVALID_ARG;
  const uintptr_t es = sh->dtype == LORA_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(X) % es || reinterpret_cast<uintptr_t>(Y) % es ||
      reinterpret_cast<uintptr_t>(freq) % 8 || reinterpret_cast<uintptr_t>(pos) % (sh->pos_bits / 8))
    return LORA_ERR_MISALIGNED;
  if (M == 0) return LORA_OK;
  if (X != Y) {
    const int64_t d = (int64_t)((uintptr_t)Y - (uintptr_t)X) / (int64_t)es;
    const Dim xt{M, sh->x_token}, xh{H, sh->x_head}, yt{M, sh->y_token}, yh{H, sh->y_head};
    if (token_outer ? heads_meet(xt, xh, yt, yh, hd, d) : heads_meet(xh, xt, yh, yt, hd, d)) return LORA_ERR_INVALID_ARG;
  }
  RotArgs a = {};
  a.M = M, a.H = (int)H, a.half = (int)(sh->rot_dim / 2), a.rest = X != Y ? (int)(hd - sh->rot_dim) : 0;
  a.xt = sh->x_token, a.xh = sh->x_head, a.yt = sh->y_token, a.yh = sh->y_head;
  a.x = X, a.pos = pos, a.freq = freq, a.y = Y, a.scale = sh->scale;
  a.pos64 = sh->pos_bits == 64, a.inverse = inverse;
  const bool inter = sh->layout == LORA_ROTARY_INTERLEAVED;
  // the widest access that every address of a vector is a multiple of
  uintptr_t heads = reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(Y) | (uintptr_t)a.rest * es;
  if (M > 1) heads |= (uintptr_t)(a.xt | a.yt) * es;
  if (H > 1) heads |= (uintptr_t)(a.xh | a.yh) * es;
  const uintptr_t bits = heads | (uintptr_t)(inter ? sh->rot_dim : sh->rot_dim / 2) * es;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (sh->dtype == LORA_BF16) {
    if (bits % 16 == 0) e = launch<bf16, 16>(a, inter, heads, st);
    else if (bits % 8 == 0) e = launch<bf16, 8>(a, inter, heads, st);
    else if (bits % 4 == 0) e = launch<bf16, 4>(a, inter, heads, st);
    else e = launch<bf16, 2>(a, inter, heads, st);
  } else {
    if (bits % 16 == 0) e = launch<float, 16>(a, inter, heads, st);
    else if (bits % 8 == 0) e = launch<float, 8>(a, inter, heads, st);
    else e = launch<float, 4>(a, inter, heads, st);
  }
  CK(e);
  return LORA_OK;
}

}  // namespace

}  // namespace lg

extern "C" {

lora_status rotary_fwd(const lora_rotary_shape* sh, const void* X, const void* pos, const uint64_t* freq, void* Y,
                       void* stream) {
  return lg::rotary(sh, X, pos, freq, Y, false, stream);
}

lora_status rotary_bwd(const lora_rotary_shape* sh, const void* dY, const void* pos, const uint64_t* freq, void* dX,
                       void* stream) {
  return lg::rotary(sh, dY, pos, freq, dX, true, stream);
}

}  // extern "C"
