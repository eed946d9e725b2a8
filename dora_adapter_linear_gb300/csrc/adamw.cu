// AdamW over a set of tensors at once, and the global norm of their gradients.
//
// Step t (kept on the device), gradient scaled to g' = c g (c: the caller's scale times the clip):
//   m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2
//   p = p - lr_i wd_i p - lr_i (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps),   lr_i = lr lr_mul_i.
//
// The state of all tensors is one array of blocks of 256 elements; tensor i begins at a block of its
// own, the rest of its last block holds zeros.  A warp takes a block, a lane 8 of its elements.  With
// 8-bit states a block keeps m and sqrt(v) as e4m3 codes times absmax / 448, the new values before
// their rounding make this step's update, and a sqrt(v) above zero is never stored as zero (an
// element whose v vanished would be divided by eps alone).  sqrt(v) instead of v halves the range
// that the 4 exponent bits have to span; the rounding is at most 2^-4 of a normal value.
// Bound by memory: 28 bytes an element (bf16, fp32 master and states), 16 with 8-bit states.
//
// The table of tensors travels in the launch's parameters (up to 32 KB), so a step copies nothing and
// is captured by a CUDA graph as it is.
#include <cuda_fp8.h>
#include <math.h>

#include "checks.h"
#include "vec.cuh"

namespace lg {

namespace {

constexpr int kBlock = 256;           // elements of a state block
constexpr int kSmallTable = 64, kTable = 640;
constexpr int kNormCtas = 608;        // gradient-norm CTAs of one launch, 4 per SM of a 152-SM part
constexpr float kMinTop = 0x1p-110f;  // a block whose largest value is below this is stored as zeros

struct AdamEntry {
  void* p;
  const void* g;
  int64_t n;
  int32_t first;                      // its first block among those of the launch
  int32_t state;                      // and among those of the state
  int32_t dtype;
  float lr_mul, decay;
};
struct AdamArgs {
  int count;                          // tensors in this launch's table
  int32_t blocks;                     // their blocks
  int advance;                        // the step's last launch: counts the step
  int bits;
  void *m, *v;
  float *m_scale, *v_scale, *master;
  int32_t* ctl;                       // {steps done, ticket}
  const float* norm_coef;             // {norm, factor of the gradients} or null
  const float* lr_dev;
  float lr, b1, b2, c1, c2, ln_b1, ln_b2, eps, grad_scale;
  // gradient norm
  float* parts;
  int part0, part_total;              // first partial of this launch, partials of all launches
  uint32_t* ticket;
  float* norm_out;
  float max_norm;
};
template <int N>
struct AdamTable {
  AdamEntry e[N];
};

// the table entry that holds block b of the launch
template <int N>
__device__ __forceinline__ int find_entry(const AdamTable<N>& t, int count, int32_t b) {
  int lo = 0, hi = count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].first <= b) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// 8 elements at i of an array of n, zeros past its end; whole aligned groups as 16-byte loads
template <typename T>
__device__ __forceinline__ void load8_of(const void* base, int64_t i, int64_t n, float (&f)[8]) {
  const T* p = static_cast<const T*>(base) + i;
  if (i + 8 <= n && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    load8(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = i + k < n ? to_f<T>(p[k]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8_of(void* base, int64_t i, int64_t n, const float (&f)[8]) {
  T* p = static_cast<T*>(base) + i;
  if (i + 8 <= n && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    store8(p, f);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) p[k] = from_f<T>(f[k]);
  }
}
__device__ __forceinline__ void load8_dt(const void* p, int dtype, int64_t i, int64_t n, float (&f)[8]) {
  if (dtype == LORA_BF16) load8_of<bf16>(p, i, n, f);
  else load8_of<float>(p, i, n, f);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ void decode8(const uint8_t* p, float scale, float (&f)[8]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 t = __half22float2(__half2(h));
    f[2 * i] = t.x * scale;
    f[2 * i + 1] = t.y * scale;
  }
}
__device__ __forceinline__ void encode8(uint8_t* p, const float (&f)[8]) {
  uint32_t u[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3)
                 << (16 * (i & 1));
  *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
}
// codes and scale of one block from its values (8 a lane); low: the least code of a value above zero
__device__ __forceinline__ void encode_block(uint8_t* codes, float* scale, const float (&f)[8], float low, int lane) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
  top = warp_max(top);
  const float inv = top >= kMinTop ? __fmul_rn(1.f / top, 448.f) : 0.f;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = f[i] * inv;
    if (f[i] > 0.f && inv > 0.f) q[i] = fmaxf(q[i], low);
  }
  encode8(codes, q);
  if (lane == 0) *scale = inv > 0.f ? __fmul_rn(top, 1.f / 448.f) : 0.f;
}

// b s + t, each operation rounded on its own: whether the compiler contracts a product into a sum does
// not decide on which side of a rounding boundary an 8-bit state falls
__device__ __forceinline__ float ema(float b, float s, float t) { return __fadd_rn(__fmul_rn(b, s), t); }

// ------------------------------------------------------------------ the step
template <int N>
__global__ void __launch_bounds__(256) adamw_kernel(const __grid_constant__ AdamArgs a,
                                                    const __grid_constant__ AdamTable<N> table) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int steps = a.ctl[0];
  const float coef = a.norm_coef ? a.norm_coef[1] : a.grad_scale;
  const bool go = isfinite(coef);       // gradients that are not finite leave everything as it was
  if (go && w < a.blocks) {
    const AdamEntry& e = table.e[find_entry(table, a.count, (int32_t)w)];
    const int32_t k0 = (int32_t)w - e.first, b = e.state + k0;
    const int64_t i = (int64_t)k0 * kBlock + lane * 8, si = (int64_t)b * kBlock + lane * 8;
    const float t = (float)(steps + 1);
    // 1 - b^t = -expm1(t ln b): no cancellation for b near 1
    const float i1 = -1.f / expm1f(t * a.ln_b1), i2 = rsqrtf(-expm1f(t * a.ln_b2));
    const float lr = (a.lr_dev ? *a.lr_dev : a.lr) * e.lr_mul;
    float g[8], m[8], v[8], p[8];
    load8_dt(e.g, e.dtype, i, e.n, g);
    if (a.bits == 8) {
      decode8(static_cast<const uint8_t*>(a.m) + si, a.m_scale[b], m);
      decode8(static_cast<const uint8_t*>(a.v) + si, a.v_scale[b], v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= v[k];
    } else {
      load8(static_cast<const float*>(a.m) + si, m);
      load8(static_cast<const float*>(a.v) + si, v);
    }
    const bool master = a.master && e.dtype == LORA_BF16;
    if (master) load8(a.master + si, p);
    else load8_dt(e.p, e.dtype, i, e.n, p);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float gs = g[k] * coef;
      m[k] = ema(a.b1, m[k], __fmul_rn(a.c1, gs));
      v[k] = ema(a.b2, v[k], __fmul_rn(__fmul_rn(a.c2, gs), gs));
      g[k] = sqrtf(v[k]);
      p[k] -= lr * e.decay * p[k] + lr * ((m[k] * i1) / fmaf(g[k], i2, a.eps));
    }
    if (master) store8(a.master + si, p);
    if (e.dtype == LORA_BF16) store8_of<bf16>(e.p, i, e.n, p);
    else store8_of<float>(e.p, i, e.n, p);
    if (a.bits == 8) {
      encode_block(static_cast<uint8_t*>(a.m) + si, a.m_scale + b, m, -448.f, lane);
      encode_block(static_cast<uint8_t*>(a.v) + si, a.v_scale + b, g, 0x1p-9f, lane);
    } else {
      store8(static_cast<float*>(a.m) + si, m);
      store8(static_cast<float*>(a.v) + si, v);
    }
  }
  // the last CTA of the step's last launch counts the step: every CTA has read the count by then
  if (a.advance) {
    __syncthreads();
    if (threadIdx.x == 0 && atomicAdd(a.ctl + 1, 1) == (int)gridDim.x - 1) {
      a.ctl[1] = 0;
      if (go) a.ctl[0] = steps + 1;
    }
  }
}

// ------------------------------------------------------------------ gradient norm
// Each CTA sums the squares of its share in a fixed order; the last one of the last launch adds the
// partial sums (fp64) and forms the factor.
template <int N>
__global__ void __launch_bounds__(256) adamw_norm_kernel(const __grid_constant__ AdamArgs a,
                                                         const __grid_constant__ AdamTable<N> table) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  __shared__ float red[2 * 32];
  __shared__ double tot[256];
  __shared__ int last;
  const int lane = threadIdx.x & 31;
  float s[1] = {0.f};
  for (int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < a.blocks; w += (int64_t)gridDim.x * 8) {
    const AdamEntry& e = table.e[find_entry(table, a.count, (int32_t)w)];
    float g[8];
    load8_dt(e.g, e.dtype, (int64_t)((int32_t)w - e.first) * kBlock + lane * 8, e.n, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[0] = fmaf(g[k], g[k], s[0]);
  }
  block_sums<1>(s, red, 0);
  if (threadIdx.x == 0) {
    a.parts[a.part0 + blockIdx.x] = s[0];
    last = 0;
    if (a.advance) {
      __threadfence();
      if (atomicAdd(a.ticket, 1u) == gridDim.x - 1) {
        last = 1;
        *a.ticket = 0;
        __threadfence();
      }
    }
  }
  __syncthreads();
  if (!last) return;
  double t = 0.0;
  for (int i = threadIdx.x; i < a.part_total; i += 256) t += (double)__ldcg(a.parts + i);
  tot[threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    t = 0.0;
    for (int i = 0; i < 256; ++i) t += tot[i];
    const float norm = (float)(sqrt(t) * fabs((double)a.grad_scale));
    a.norm_out[0] = norm;
    const float clip = a.max_norm > 0.f ? fminf(1.f, a.max_norm / (norm + 1e-6f)) : 1.f;
    a.norm_out[1] = isfinite(norm) ? a.grad_scale * clip : nanf("");
  }
}

lora_status check_table(const lora_adamw_tensor* t, const void* const* grads, int64_t count, int64_t* used) {
  if (count < 0 || (count > 0 && (!t || !grads))) return LORA_ERR_INVALID_ARG;
  int64_t b = 0, u = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n < 0) return LORA_ERR_INVALID_ARG;
    if (t[i].dtype != LORA_F32 && t[i].dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
    if (!isfinite(t[i].lr_mul) || !isfinite(t[i].weight_decay)) return LORA_ERR_INVALID_ARG;
    b += (t[i].n + kBlock - 1) / kBlock;
    if (b > (1LL << 31) - 1) return LORA_ERR_UNSUPPORTED;
    if (t[i].n == 0 || !grads[i]) continue;
    if (!t[i].p) return LORA_ERR_INVALID_ARG;
    const uintptr_t es = t[i].dtype == LORA_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(t[i].p) % es || reinterpret_cast<uintptr_t>(grads[i]) % es)
      return LORA_ERR_MISALIGNED;
    ++u;
  }
  *used = u;
  return LORA_OK;
}

// Runs `launch(args, table)` over the tensors that have a gradient, as many a launch as its table holds.
template <int N, typename F>
lora_status over_table(const lora_adamw_tensor* t, const void* const* grads, int64_t count, int64_t used, AdamArgs a,
                       F launch) {
  AdamTable<N> table;
  int32_t state = 0;
  int64_t i = 0, left = used;
  while (left > 0) {
    a.count = 0;
    a.blocks = 0;
    for (; i < count && a.count < N; ++i) {
      const int32_t nb = (int32_t)((t[i].n + kBlock - 1) / kBlock);
      if (nb > 0 && grads[i]) {
        table.e[a.count++] =
            AdamEntry{t[i].p, grads[i], t[i].n, a.blocks, state, t[i].dtype, t[i].lr_mul, t[i].weight_decay};
        a.blocks += nb;
      }
      state += nb;
    }
    left -= a.count;
    a.advance = left == 0;
    const lora_status e = launch(a, table);
    if (e != LORA_OK) return e;
  }
  return LORA_OK;
}

inline int norm_ctas(int64_t blocks) {
  const int64_t n = (blocks + 7) / 8;
  return (int)(n < kNormCtas ? n : kNormCtas);
}

}  // namespace

}  // namespace lg

using namespace lg;

extern "C" {

int64_t adamw_state_blocks(const lora_adamw_tensor* tensors, int64_t count) {
  int64_t b = 0;
  if (count < 0 || (count > 0 && !tensors)) return -1;
  for (int64_t i = 0; i < count; ++i) {
    if (tensors[i].n < 0) return -1;
    b += (tensors[i].n + kBlock - 1) / kBlock;
  }
  return b;
}

size_t adamw_norm_workspace_bytes(int64_t count) {
  if (count < 0) return 0;
  return kErrBytes + al256((size_t)((count + kSmallTable - 1) / kSmallTable + 1) * kNormCtas * sizeof(float));
}

lora_status adamw_grad_norm(const lora_adamw_tensor* tensors, const void* const* grads, int64_t count,
                            float grad_scale, float max_norm, float* norm_coef, void* ws, size_t ws_bytes,
                            void* stream) {
  int64_t used;
  const lora_status e = check_table(tensors, grads, count, &used);
  if (e != LORA_OK) return e;
  REQ(norm_coef);
  if (!isfinite(grad_scale) || isnan(max_norm)) return LORA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(norm_coef) % 8) return LORA_ERR_MISALIGNED;
  const lora_status ew = check_ws(ws, ws_bytes, adamw_norm_workspace_bytes(count));
  if (ew != LORA_OK) return ew;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  AdamArgs a = {};
  a.grad_scale = grad_scale, a.max_norm = max_norm, a.norm_out = norm_coef;
  a.ticket = static_cast<uint32_t*>(ws) + 16;   // in the cleared header, past the error word
  a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + kErrBytes);
  const auto run = [&](auto kernel, AdamArgs& b, const auto& table) {
    const int ctas = norm_ctas(b.blocks);
    b.part0 = a.part_total;
    a.part_total += ctas;
    b.part_total = a.part_total;
    CK(launch_pdl(kernel, dim3((unsigned)ctas), dim3(256), 0, st, b, table));
    return LORA_OK;
  };
  if (used == 0) {
    AdamTable<kSmallTable> none = {};
    a.advance = 1, a.part_total = 1;
    CK(launch_pdl(adamw_norm_kernel<kSmallTable>, dim3(1), dim3(256), 0, st, a, none));
    return LORA_OK;
  }
  if (used <= kSmallTable)
    return over_table<kSmallTable>(tensors, grads, count, used, a, [&](AdamArgs& b, const AdamTable<kSmallTable>& t) {
      return run(adamw_norm_kernel<kSmallTable>, b, t);
    });
  return over_table<kTable>(tensors, grads, count, used, a, [&](AdamArgs& b, const AdamTable<kTable>& t) {
    return run(adamw_norm_kernel<kTable>, b, t);
  });
}

lora_status adamw_step(const lora_adamw_tensor* tensors, const void* const* grads, int64_t count,
                       const lora_adamw_state* state, const lora_adamw_hyper* hyper, const float* norm_coef,
                       void* stream) {
  int64_t used;
  const lora_status e = check_table(tensors, grads, count, &used);
  if (e != LORA_OK) return e;
  REQ(state);
  REQ(hyper);
  const lora_adamw_hyper& h = *hyper;
  if (state->bits != 8 && state->bits != 32) return LORA_ERR_INVALID_ARG;
  REQ(state->ctl);
  if (used > 0) {
    REQ(state->m);
    REQ(state->v);
    if (state->bits == 8 && (!state->m_scale || !state->v_scale)) return LORA_ERR_INVALID_ARG;
  }
  if (!(h.beta1 >= 0.0 && h.beta1 < 1.0) || !(h.beta2 >= 0.0 && h.beta2 < 1.0)) return LORA_ERR_INVALID_ARG;
  if (!(h.eps > 0.0) || !isfinite(h.eps) || !isfinite(h.lr) || !isfinite(h.grad_scale)) return LORA_ERR_INVALID_ARG;
  for (const void* p : {(const void*)state->m, (const void*)state->v, (const void*)state->m_scale,
                        (const void*)state->v_scale, (const void*)state->master})
    ALN(p);
  if (reinterpret_cast<uintptr_t>(state->ctl) % 8 || reinterpret_cast<uintptr_t>(norm_coef) % 8 ||
      reinterpret_cast<uintptr_t>(h.lr_device) % 4)
    return LORA_ERR_MISALIGNED;
  if (used == 0) return LORA_OK;
  AdamArgs a = {};
  a.bits = state->bits;
  a.m = state->m, a.v = state->v, a.m_scale = state->m_scale, a.v_scale = state->v_scale, a.master = state->master;
  a.ctl = state->ctl;
  a.norm_coef = norm_coef;
  a.lr_dev = h.lr_device;
  a.lr = (float)h.lr, a.b1 = (float)h.beta1, a.b2 = (float)h.beta2;
  a.c1 = (float)(1.0 - h.beta1), a.c2 = (float)(1.0 - h.beta2);
  a.ln_b1 = (float)log(h.beta1), a.ln_b2 = (float)log(h.beta2);
  a.eps = (float)h.eps, a.grad_scale = (float)h.grad_scale;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto run = [&](auto kernel, AdamArgs& b, const auto& table) {
    CK(launch_pdl(kernel, dim3((unsigned)((b.blocks + 7) / 8)), dim3(256), 0, st, b, table));
    return LORA_OK;
  };
  if (used <= kSmallTable)
    return over_table<kSmallTable>(tensors, grads, count, used, a, [&](AdamArgs& b, const AdamTable<kSmallTable>& t) {
      return run(adamw_kernel<kSmallTable>, b, t);
    });
  return over_table<kTable>(tensors, grads, count, used, a, [&](AdamArgs& b, const AdamTable<kTable>& t) {
    return run(adamw_kernel<kTable>, b, t);
  });
}

}  // extern "C"
