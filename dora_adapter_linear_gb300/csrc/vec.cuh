// Eight consecutive elements of a row as one (bf16) or two (fp32) 16-byte accesses, and the block
// sums of the row kernels.
#pragma once

#include "common.cuh"

namespace lg {

__device__ __forceinline__ void load8(const bf16* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack_bf16x2(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void store8(bf16* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// Pairs of fp32 in one 64-bit register: sm_100 and later multiply and add two at a time.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 unpack(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ float sum2(F2 a) {
  const float2 t = unpack(a);
  return t.x + t.y;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// The same eight elements as they lie in memory, for rows that wait in registers: bf16 takes half the
// registers of fp32 until it is unpacked.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16> {
  uint4 v;
  __device__ __forceinline__ void get(F2 (&f)[4]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void get(F2 (&f)[4]) const {
    f[0] = f2(a.x, a.y), f[1] = f2(a.z, a.w), f[2] = f2(b.x, b.y), f[3] = f2(b.z, b.w);
  }
};
// streaming loads: a row that is read once does not push out what is kept in L1
__device__ __forceinline__ void stream8(const bf16* p, Raw8<bf16>& r) { r.v = __ldcs(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void stream8(const float* p, Raw8<float>& r) {
  r.a = __ldcs(reinterpret_cast<const float4*>(p));
  r.b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
}

// Sums of N values over the block (a multiple of 32 threads, at most 1024), given to every thread
// in a fixed order.  `red` holds 2 x 32 x N floats and `flip` alternates from call to call, so that
// one barrier a call is enough: a warp that runs ahead into the next call writes the other half.
// Returns whether any thread came with `bad`, the same answer for all.
template <int N>
__device__ __forceinline__ bool block_sums(float (&v)[N], float* red, int flip, bool bad = false) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  float* r = red + flip * 32 * N;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) r[warp * N + i] = v[i];
  const bool any = __syncthreads_or(bad);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < warps ? r[lane * N + i] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  return any;
}

// eight elements as four pairs
__device__ __forceinline__ void load4x2(const bf16* p, F2 (&f)[4]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void load4x2(const float* p, F2 (&f)[4]) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *(reinterpret_cast<const ulonglong2*>(p) + 1);
  f[0].v = a.x, f[1].v = a.y, f[2].v = b.x, f[3].v = b.y;
}
__device__ __forceinline__ void store4x2(bf16* p, const F2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack(f[i]);
    w[i] = pack_bf16x2(t.x, t.y);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store4x2(float* p, const F2 (&f)[4]) {
  *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(f[0].v, f[1].v);
  *(reinterpret_cast<ulonglong2*>(p) + 1) = make_ulonglong2(f[2].v, f[3].v);
}

// Sums of N (4 or 8) values over each G neighbouring lanes of a warp: value i ends up in their lanes i Q ..
// i Q + Q - 1, Q = G / N.  Each of the first steps halves the values that a lane still carries: 9 shuffles for
// 8 values of a warp, not 40.
template <int N, int G = 32>
__device__ __forceinline__ float warp_sums_of(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = N / 2, o = G / 2; n >= 1; n /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  float t = v[0];
#pragma unroll
  for (int o = G / 2 / N; o >= 1; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}
template <int N, int G = 32>
__device__ __forceinline__ void spread(float t, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, t, i * (G / N), G);
}

// Sums of N (4 or 8) values over a block of at most W warps (16 or 32), all of them given to every
// thread, in a fixed order.  `red`: 2 N W floats, 16-byte aligned; flip and the answer as in block_sums.
template <int N, int W>
__device__ __forceinline__ bool block_sums_of(float (&v)[N], float* red, int flip, bool bad = false) {
  constexpr int Q = 32 / N, E = W / Q;   // lanes of a value, and warps that each of them adds
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
  float t = warp_sums_of<N>(v);
  float* r = red + flip * N * W + lane / Q * W;
  if (lane % Q == 0) r[warp] = t;
  const bool any = __syncthreads_or(bad);
  float e[E];
  if (E == 2) {
    const float2 p = *reinterpret_cast<const float2*>(r + lane % Q * E);
    e[0] = p.x, e[1] = p.y;
  } else {
    const float4 p = *reinterpret_cast<const float4*>(r + lane % Q * E);
    e[0] = p.x, e[1] = p.y, e[E - 2] = p.z, e[E - 1] = p.w;
  }
  t = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) t += lane % Q * E + i < warps ? e[i] : 0.f;
#pragma unroll
  for (int o = Q / 2; o >= 1; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
  spread<N>(t, v);
  return any;
}

}  // namespace lg
