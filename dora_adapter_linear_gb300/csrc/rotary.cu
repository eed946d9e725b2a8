// Rotary positions: pair j < rot / 2 of every head of token i turns by t = pos[i] theta_j,
//   (a, b) -> scale (a cos t - b sin t, b cos t + a sin t),
// the backward by -t (the transpose).  A pair is (j, j + rot / 2) of the head in the half layout and
// (2 j, 2 j + 1) in the interleaved one; the rest of a head passes unchanged.
//
// The angle is kept in turns: freq[j] = theta_j / (2 pi) as a 64-bit binary fraction, so the low 64
// bits of pos freq[j] are the fraction of a turn, exact for every 64-bit position (an fp32 product
// would be off by 2^-24 of the angle: 0.008 rad at position 131072).  Its upper 32 bits, as a signed
// half-turn in [-1, 1), go to sincospif: the angle is within pi 2^-25 of the true one.
// Bound by memory: each rotated element is read and written once.
#include <math.h>

#include "checks.h"
#include "vec.cuh"

namespace lg {

namespace {

struct RotArgs {
  int64_t M, H, hd, rot;
  int64_t xt, xh, yt, yh;       // token and head strides of x and y, in elements
  const void *x, *pos;
  const uint64_t* freq;
  void* y;
  float scale;
  int interleaved, pos64, inverse, copy_rest;
};

// scale cos t and scale sin t of one pair
__device__ __forceinline__ float2 turn(const RotArgs& a, int64_t pos, int j) {
  const int32_t half = (int32_t)(((uint64_t)pos * a.freq[j]) >> 32);   // 2 x the fraction, x 2^31, signed
  float s, c;
  sincospif((float)half * 0x1p-31f, &s, &c);
  s *= a.scale;
  return make_float2(c * a.scale, a.inverse ? -s : s);
}

// ------------------------------------------------------------------ any size and alignment
// One CTA per token: the token's angles in shared memory, then a pair (or a passed element) a thread.
template <typename T>
__global__ void __launch_bounds__(256) rotary_kernel(const RotArgs a) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  extern __shared__ float2 cs[];
  const int64_t tok = blockIdx.x;
  const int64_t pos = a.pos64 ? static_cast<const int64_t*>(a.pos)[tok] : static_cast<const int32_t*>(a.pos)[tok];
  const int half = (int)a.rot / 2, rest = a.copy_rest ? (int)(a.hd - a.rot) : 0, per = half + rest;
  for (int j = threadIdx.x; j < half; j += blockDim.x) cs[j] = turn(a, pos, j);
  __syncthreads();
  const T* x = static_cast<const T*>(a.x) + tok * a.xt;
  T* y = static_cast<T*>(a.y) + tok * a.yt;
  for (int64_t i = threadIdx.x; i < a.H * per; i += blockDim.x) {
    const int64_t h = i / per;
    const int j = (int)(i - h * per);
    const T* xh = x + h * a.xh;
    T* yh = y + h * a.yh;
    if (j >= half) {
      yh[a.rot + j - half] = xh[a.rot + j - half];
      continue;
    }
    const int ia = a.interleaved ? 2 * j : j, ib = a.interleaved ? 2 * j + 1 : j + half;
    const float u = to_f<T>(xh[ia]), v = to_f<T>(xh[ib]);
    yh[ia] = from_f<T>(u * cs[j].x - v * cs[j].y);
    yh[ib] = from_f<T>(v * cs[j].x + u * cs[j].y);
  }
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
  if (sh->M > (1LL << 31) - 1 || sh->H > (1 << 20) || sh->head_dim > (1 << 12)) return LORA_ERR_UNSUPPORTED;
  REQ(freq);
  if (sh->M > 0 && (!X || !pos || !Y)) return LORA_ERR_INVALID_ARG;
  // no two elements of y at one address (x may repeat a head or a token); in place: the same layout
  const auto apart = [](int64_t n, int64_t s, int64_t inner) { return n <= 1 || s >= inner; };
  const int64_t hd = sh->head_dim, M = sh->M, H = sh->H;
  if (sh->x_token < 0 || sh->x_head < 0 || sh->y_token < 0 || sh->y_head < 0) return LORA_ERR_INVALID_ARG;
  if (!(apart(H, sh->y_head, hd) && apart(M, sh->y_token, (H - 1) * sh->y_head + hd)) &&
      !(apart(M, sh->y_token, hd) && apart(H, sh->y_head, (M - 1) * sh->y_token + hd)))
    return LORA_ERR_INVALID_ARG;
  if (X == Y && ((M > 1 && sh->x_token != sh->y_token) || (H > 1 && sh->x_head != sh->y_head)))
    return LORA_ERR_INVALID_ARG;
  const uintptr_t es = sh->dtype == LORA_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(X) % es || reinterpret_cast<uintptr_t>(Y) % es ||
      reinterpret_cast<uintptr_t>(freq) % 8 || reinterpret_cast<uintptr_t>(pos) % (sh->pos_bits / 8))
    return LORA_ERR_MISALIGNED;
  if (M == 0) return LORA_OK;
  RotArgs a = {};
  a.M = M, a.H = H, a.hd = hd, a.rot = sh->rot_dim;
  a.xt = sh->x_token, a.xh = sh->x_head, a.yt = sh->y_token, a.yh = sh->y_head;
  a.x = X, a.pos = pos, a.freq = freq, a.y = Y, a.scale = sh->scale;
  a.interleaved = sh->layout == LORA_ROTARY_INTERLEAVED, a.pos64 = sh->pos_bits == 64;
  a.inverse = inverse, a.copy_rest = X != Y;
  const size_t smem = (size_t)sh->rot_dim / 2 * sizeof(float2);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (sh->dtype == LORA_BF16) CK(launch_pdl(rotary_kernel<bf16>, dim3((unsigned)M), dim3(256), smem, st, a));
  else CK(launch_pdl(rotary_kernel<float>, dim3((unsigned)M), dim3(256), smem, st, a));
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
