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
// 28 bytes an element (bf16, fp32 master and states), 16 with 8-bit states.  32-bit states are bound by memory:
// 42 M bf16 elements 174 to 177 us, 6.7 TB/s.
//
// The table of tensors travels in the launch's parameters (up to 32 KB), so a step copies nothing and
// is captured by a CUDA graph as it is.
#include <cuda_fp8.h>
#include <float.h>
#include <math.h>

#include <type_traits>

#include "checks.h"
#include "vec.cuh"

namespace lg {

namespace {

constexpr int kBlock = 256;           // elements of a state block
constexpr int kSmallTable = 64, kTable = 640;
constexpr int kNormCtas = 608;        // gradient-norm CTAs of one launch, 4 per SM of a 152-SM part
constexpr int kStepCtas = 4;          // step CTAs of an SM: 64 registers a thread
constexpr int kStep8Ctas = 2, kPair = 2;   // with 8-bit states; blocks that a warp takes at a time
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
  int32_t blocks, rounds;             // their blocks; rounds of a chunk
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

// 8 elements as they lie in memory (bf16 takes the first half): a load that does not wait for its value
struct Eight {
  uint4 lo, hi;
};
// What a launch's tensors are, where that is known for all of them: bf16 with masters (KIND_BF16), fp32,
// or either, asked for each.  The last spills 40 bytes with 32-bit states and waits at its branches with 8-bit ones
// (42 M elements: half bf16 with masters 177 us of 173 and 125 of 99, bf16 without masters 145 of 136 and 129 of 62;
// all bf16 with masters 176 and 111).
enum { KIND_ANY = 0, KIND_BF16 = 1, KIND_F32 = 2 };
template <int KIND>
__device__ __forceinline__ int type_of(const AdamEntry& e) {
  return KIND == KIND_BF16 ? (int)LORA_BF16 : KIND == KIND_F32 ? (int)LORA_F32 : e.dtype;
}
template <int KIND>
__device__ __forceinline__ bool has_master(const AdamArgs& a, int dtype) {
  return KIND == KIND_BF16 || (KIND == KIND_ANY && a.master && dtype == LORA_BF16);
}
__device__ __forceinline__ void take(const void* base, int dtype, int64_t i, Eight& r) {
  if (dtype == LORA_BF16) {
    r.lo = __ldcs(reinterpret_cast<const uint4*>(static_cast<const bf16*>(base) + i));
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + i);
    r.lo = __ldcs(p);
    r.hi = __ldcs(p + 1);
  }
}
// the same element by element, zeros past the end of the array of n
template <typename T>
__device__ __forceinline__ void take_each(const void* base, int64_t i, int64_t n, Eight& r) {
  const T* p = static_cast<const T*>(base) + i;
  uint32_t w[8];
  float f[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = i + k < n ? to_f<T>(p[k]) : 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k)
    w[k] = sizeof(T) == 4 ? __float_as_uint(f[k]) : k < 4 ? pack_bf16x2(f[2 * k & 7], f[(2 * k + 1) & 7]) : 0u;
  r.lo = make_uint4(w[0], w[1], w[2], w[3]);
  r.hi = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void open8(const Eight& r, int dtype, F2 (&f)[4]) {
  const uint32_t a[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w}, b[4] = {r.hi.x, r.hi.y, r.hi.z, r.hi.w};
  if (dtype == LORA_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(a[i] << 16), __uint_as_float(a[i] & 0xffff0000u));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[i] = f2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
      f[i + 2] = f2(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1]));
    }
  }
}
template <typename T>
__device__ __forceinline__ void put_each(void* base, int64_t i, int64_t n, const F2 (&f)[4]) {
  T* p = static_cast<T*>(base) + i;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = unpack(f[k]);
    if (i + 2 * k < n) p[2 * k] = from_f<T>(t.x);
    if (i + 2 * k + 1 < n) p[2 * k + 1] = from_f<T>(t.y);
  }
}
// whether the block of 256 elements from i on lies within the array of n, which begins at 16 bytes
__device__ __forceinline__ bool whole(const void* base, int64_t i, int64_t n) {
  return i + kBlock <= n && (reinterpret_cast<uintptr_t>(base) & 15) == 0;
}

// eight e4m3 codes times their block's scale
__device__ __forceinline__ void decode8(uint2 w, float scale, F2 (&f)[4]) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
    const float2 t = __half22float2(__half2(h));
    f[i] = mul2(f2(t.x, t.y), f2(scale));
  }
}
// Codes and scale of one block from its values (8 a lane).  ROOT: values that are not negative, of which
// none above zero may become the code 0.  The largest absolute value is found on the bit patterns, whose
// order as integers is that of the numbers, with a NaN on top: a block with one becomes NaN as a whole.
template <bool ROOT>
__device__ __forceinline__ void encode_block(uint8_t* codes, float* scale, const F2 (&f)[4], int lane) {
  float x[8];
  uint32_t top_bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack(f[i]);
    x[2 * i] = t.x, x[2 * i + 1] = t.y;
    top_bits = max(top_bits, max(__float_as_uint(t.x) & 0x7fffffffu, __float_as_uint(t.y) & 0x7fffffffu));
  }
  const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, top_bits));
  const bool none = top < kMinTop;
  const float inv = none ? 0.f : __fmul_rn(1.f / top, 448.f), low = none ? 0.f : 0x1p-9f;
  uint32_t u[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 q = unpack(mul2(f[i], f2(inv)));
    if (ROOT) {
      if (x[2 * i] > 0.f) q.x = fmaxf(q.x, low);
      if (x[2 * i + 1] > 0.f) q.y = fmaxf(q.y, low);
    }
    u[i >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3) << (16 * (i & 1));
  }
  *reinterpret_cast<uint2*>(codes) = make_uint2(u[0], u[1]);
  if (lane == 0) *scale = none ? 0.f : __fmul_rn(top, 1.f / 448.f);
}

// b s + t, each operation rounded on its own: whether the compiler contracts a product into a sum does
// not decide on which side of a rounding boundary an 8-bit state falls
__device__ __forceinline__ F2 ema(float b, F2 s, F2 t) {
  const float2 x = unpack(s), y = unpack(t);
  return f2(__fadd_rn(__fmul_rn(b, x.x), y.x), __fadd_rn(__fmul_rn(b, x.y), y.y));
}

// ------------------------------------------------------------------ the step
// What a launch's steps have in common.  It is loaded first and formed once per thread; with 8-bit states when the
// first block's loads are on their way too, which its use before them would hold back (14 tensors of 40 k elements:
// 3.8 us against 4.2, 14 of 3.1 M behind a norm 18.9 against 19.4).
struct StepFactors {
  float coef, lr;           // of the gradients; lr
  int steps;
  float i1, i2;             // 1 / (1 - b1^t), (1 - b2^t)^-1/2
  bool formed, go;          // gradients that are not finite leave everything as it was
  __device__ __forceinline__ explicit StepFactors(const AdamArgs& a) : formed(false) {
    steps = a.ctl[0];
    coef = a.norm_coef ? a.norm_coef[1] : a.grad_scale;
    lr = a.lr_dev ? *a.lr_dev : a.lr;
  }
  // whether there is a step to do
  __device__ __forceinline__ bool form(const AdamArgs& a) {
    if (formed) return go;
    formed = true;
    go = isfinite(coef);
    // 1 - b^t = -expm1(t ln b): no cancellation for b near 1
    const float t = (float)(steps + 1);
    i1 = -1.f / expm1f(t * a.ln_b1);
    i2 = rsqrtf(-expm1f(t * a.ln_b2));
    return go;
  }
};
// the last CTA of the step's last launch counts the step: every CTA has read the count by then
__device__ __forceinline__ void count_step(const AdamArgs& a, StepFactors& f) {
  if (!a.advance) return;
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(a.ctl + 1, 1) == (int)gridDim.x - 1) {
    a.ctl[1] = 0;
    if (f.form(a)) a.ctl[0] = f.steps + 1;
  }
}
// m, v and p of eight elements; root becomes sqrt(v)
__device__ __forceinline__ void update8(const AdamArgs& a, const StepFactors& f, const AdamEntry& e, const F2 (&g)[4],
                                        F2 (&m)[4], F2 (&v)[4], F2 (&root)[4], F2 (&p)[4]) {
  const float lr = f.lr * e.lr_mul, step = lr * f.i1;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const F2 gs = mul2(g[j], f2(f.coef));
    m[j] = ema(a.b1, m[j], mul2(f2(a.c1), gs));
    v[j] = ema(a.b2, v[j], mul2(mul2(f2(a.c2), gs), gs));
    const float2 vv = unpack(v[j]);
    root[j] = f2(sqrtf(vv.x), sqrtf(vv.y));
    // the quotient within 2 ulp: it is lr times smaller than what it is added to
    const float2 den = unpack(fma2(root[j], f2(f.i2), f2(a.eps))), num = unpack(mul2(m[j], f2(step)));
    p[j] = fma2(f2(-lr * e.decay), p[j], p[j]);
    p[j] = add2(p[j], f2(-__fdividef(num.x, den.x), -__fdividef(num.y, den.y)));
  }
}
// the gradient and the parameter's exact value (master, or the parameter itself)
__device__ __forceinline__ void take_gp(const AdamArgs& a, const AdamEntry& e, int dtype, bool full, bool master,
                                        int64_t i, int64_t si, Eight& ge, Eight& pe) {
  if (full) take(e.g, dtype, i, ge);
  else if (dtype == LORA_BF16) take_each<bf16>(e.g, i, e.n, ge);
  else take_each<float>(e.g, i, e.n, ge);
  if (master) take(a.master, LORA_F32, si, pe);
  else if (full) take(e.p, dtype, i, pe);
  else if (dtype == LORA_BF16) take_each<bf16>(e.p, i, e.n, pe);
  else take_each<float>(e.p, i, e.n, pe);
}
__device__ __forceinline__ void put_p(const AdamArgs& a, const AdamEntry& e, int dtype, bool full, bool master, int64_t i,
                                      int64_t si, const F2 (&p)[4]) {
  if (master) store4x2(a.master + si, p);
  if (dtype == LORA_BF16) {
    if (full) store4x2(static_cast<bf16*>(e.p) + i, p);
    else put_each<bf16>(e.p, i, e.n, p);
  } else {
    if (full) store4x2(static_cast<float*>(e.p) + i, p);
    else put_each<float>(e.p, i, e.n, p);
  }
}
// A warp's way through its blocks: chunks of 8 `rounds` consecutive blocks, every gridDim-th chunk for a
// CTA; in a round each of its 8 warps has one, so a CTA touches 2048 neighbouring elements of every array.
// The tensor is looked up once per chunk.
template <int N>
struct Walk {
  const AdamArgs& a;
  const AdamTable<N>& table;
  int64_t c0;
  int32_t w, w1, end;
  int k;
  __device__ __forceinline__ Walk(const AdamArgs& args, const AdamTable<N>& t) : a(args), table(t) {
    c0 = (int64_t)blockIdx.x * 8 * a.rounds;
    begin();
  }
  __device__ __forceinline__ bool valid() const { return w < w1; }
  __device__ __forceinline__ void begin() {
    w = (int32_t)min(c0, (int64_t)a.blocks) + (int32_t)(threadIdx.x >> 5);   // at most 2^30 blocks
    w1 = (int32_t)min((int64_t)a.blocks, c0 + 8 * a.rounds);
    if (!valid()) return;
    k = find_entry(table, a.count, w);
    end = k + 1 < a.count ? table.e[k + 1].first : a.blocks;
  }
  __device__ __forceinline__ void next() {
    w += 8;
    if (w >= w1) {
      c0 += (int64_t)gridDim.x * 8 * a.rounds;
      begin();
      return;
    }
    while (w >= end) {
      ++k;
      end = k + 1 < a.count ? table.e[k + 1].first : a.blocks;
    }
  }
};

template <int N, int KIND>
__global__ void __launch_bounds__(256, kStepCtas) adamw_kernel(const __grid_constant__ AdamArgs a,
                                                       const __grid_constant__ AdamTable<N> table) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  const int lane = threadIdx.x & 31;
  StepFactors f(a);
  const bool go = f.form(a);   // within the loop it would cost spilled registers and bring nothing here
  for (Walk<N> at(a, table); go && at.valid(); at.next()) {
    const AdamEntry& e = table.e[at.k];
    const int32_t b0 = at.w - e.first;
    const int64_t i0 = (int64_t)b0 * kBlock, i = i0 + lane * 8, si = (int64_t)(e.state + b0) * kBlock + lane * 8;
    const int dtype = type_of<KIND>(e);
    const bool master = has_master<KIND>(a, dtype);
    const bool full = whole(e.g, i0, e.n) && whole(e.p, i0, e.n);   // the same for the warp
    Eight ge, pe;   // every load is on its way before the first value is opened
    F2 g[4], m[4], v[4], p[4];
    take_gp(a, e, dtype, full, master, i, si, ge, pe);
    load4x2(static_cast<const float*>(a.m) + si, m);
    load4x2(static_cast<const float*>(a.v) + si, v);
    open8(ge, dtype, g);
    open8(pe, master ? (int)LORA_F32 : dtype, p);
    update8(a, f, e, g, m, v, g, p);
    put_p(a, e, dtype, full, master, i, si, p);
    store4x2(static_cast<float*>(a.m) + si, m);
    store4x2(static_cast<float*>(a.v) + si, v);
  }
  count_step(a, f);
}

// ------------------------------------------------------------------ masters from the parameters
template <int N>
__global__ void __launch_bounds__(256) adamw_master_kernel(const __grid_constant__ AdamArgs a,
                                                           const __grid_constant__ AdamTable<N> table) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  const int lane = threadIdx.x & 31;
  for (Walk<N> at(a, table); at.valid(); at.next()) {
    const AdamEntry& e = table.e[at.k];
    if (e.dtype != LORA_BF16) continue;
    const int32_t b0 = at.w - e.first;
    const int64_t i0 = (int64_t)b0 * kBlock, i = i0 + lane * 8;
    Eight r;
    F2 f[4];
    if (whole(e.p, i0, e.n)) take(e.p, LORA_BF16, i, r);
    else take_each<bf16>(e.p, i, e.n, r);
    open8(r, LORA_BF16, f);
    store4x2(a.master + (int64_t)(e.state + b0) * kBlock + lane * 8, f);
  }
}

// ------------------------------------------------------------------ the step with 8-bit states
// A block's arithmetic (square roots, quotients, two block maxima, the codes both ways) takes about as long
// as its 4 KB take from memory, so nothing may stand between a warp and its next values: it takes two
// blocks of a tensor at a time, all loads before the first use, and has asked L2 for the next two by then.
// 168 M bf16 elements with masters: 414 us, 6.5 TB/s.  With one block at a time 617 us on two CTAs an SM and
// 473 on four, with three or four 441 and 451, with two on three CTAs 463 (80 registers spill); one block
// without the prefetch 570, one by asynchronous copies into shared memory 690.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// a block's values as they are loaded
struct Raw8Bit {
  Eight g, p;
  uint2 m, v;
  float ms, vs;
};

template <int N, int KIND>
__global__ void __launch_bounds__(256, kStep8Ctas) adamw8_kernel(const __grid_constant__ AdamArgs a,
                                                                 const __grid_constant__ AdamTable<N> table) {
  pdl_wait();   // inputs may come from the previous kernel in the stream
  if (threadIdx.x == 0) pdl_trigger();
  const int lane = threadIdx.x & 31;
  StepFactors f(a);
  uint8_t *const mc = static_cast<uint8_t*>(a.m), *const vc = static_cast<uint8_t*>(a.v);
  // one block: i its lane's first element in the tensor, b its place in the state
  auto load = [&](const AdamEntry& e, int dtype, bool full, int64_t i, int64_t b, Raw8Bit& r) {
    const int64_t si = b * kBlock + lane * 8;
    take_gp(a, e, dtype, full, has_master<KIND>(a, dtype), i, si, r.g, r.p);
    r.m = *reinterpret_cast<const uint2*>(mc + si);
    r.v = *reinterpret_cast<const uint2*>(vc + si);
    r.ms = a.m_scale[b], r.vs = a.v_scale[b];
  };
  auto step = [&](const AdamEntry& e, int dtype, bool full, int64_t i, int64_t b, const Raw8Bit& r) {
    const int64_t si = b * kBlock + lane * 8;
    const bool master = has_master<KIND>(a, dtype);
    F2 g[4], m[4], v[4], p[4];
    open8(r.g, dtype, g);
    open8(r.p, master ? (int)LORA_F32 : dtype, p);
    decode8(r.m, r.ms, m);
    decode8(r.v, r.vs, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], v[j]);
    update8(a, f, e, g, m, v, g, p);
    put_p(a, e, dtype, full, master, i, si, p);
    encode_block<false>(mc + si, a.m_scale + b, m, lane);
    encode_block<true>(vc + si, a.v_scale + b, g, lane);
  };
  for (Walk<N> at(a, table); at.valid();) {
    const AdamEntry& e = table.e[at.k];
    const int dtype = type_of<KIND>(e);
    const int64_t i0 = (int64_t)(at.w - e.first) * (kPair * kBlock), i = i0 + lane * 8;
    const int64_t b = e.state + (int64_t)(at.w - e.first) * kPair;
    at.next();
    // both blocks; the same for the warp
    if (whole(e.g, i0 + (kPair - 1) * kBlock, e.n) && whole(e.p, i0 + (kPair - 1) * kBlock, e.n)) {
      Raw8Bit r[kPair];   // every load is on its way before the first value is opened
#pragma unroll
      for (int h = 0; h < kPair; ++h) load(e, dtype, true, i + h * kBlock, b + h, r[h]);
      if (at.valid() && lane < 4) {
        const AdamEntry& n = table.e[at.k];
        const int ntype = type_of<KIND>(n), es = ntype == LORA_BF16 ? 2 : 4;
        const int64_t n0 = (int64_t)(at.w - n.first) * (kPair * kBlock), ns = (int64_t)n.state * kBlock + n0;
        if (whole(n.g, n0 + (kPair - 1) * kBlock, n.n)) {
          if (lane == 0) prefetch_l2(mc + ns, kPair * kBlock);
          else if (lane == 1) prefetch_l2(vc + ns, kPair * kBlock);
          else if (lane == 2 && has_master<KIND>(a, ntype)) prefetch_l2(a.master + ns, kPair * kBlock * 4);
          else if (lane == 3) prefetch_l2(static_cast<const char*>(n.g) + n0 * es, kPair * kBlock * es);
        }
      }
      if (!f.form(a)) break;
#pragma unroll
      for (int h = 0; h < kPair; ++h) step(e, dtype, true, i + h * kBlock, b + h, r[h]);
    } else {
      if (!f.form(a)) break;
      for (int h = 0; h < kPair && i0 + h * kBlock < e.n; ++h) {
        Raw8Bit r;
        const bool full = whole(e.g, i0 + h * kBlock, e.n) && whole(e.p, i0 + h * kBlock, e.n);
        load(e, dtype, full, i + h * kBlock, b + h, r);
        step(e, dtype, full, i + h * kBlock, b + h, r);
      }
    }
  }
  count_step(a, f);
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
  __shared__ double tot[8];
  __shared__ int last;
  const int lane = threadIdx.x & 31;
  // a warp has a run of consecutive blocks and keeps four of them on their way
  const int64_t warps = (int64_t)gridDim.x * 8, id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  int32_t w = (int32_t)(id * a.blocks / warps);
  const int32_t w1 = (int32_t)((id + 1) * a.blocks / warps);
  float s[1] = {0.f};
  for (int k = w < w1 ? find_entry(table, a.count, w) : 0; w < w1; ++k) {
    const AdamEntry& e = table.e[k];
    const int32_t end = min(w1, k + 1 < a.count ? table.e[k + 1].first : a.blocks);
    int64_t i = (int64_t)(w - e.first) * kBlock + lane * 8;
    auto sum = [&](auto one) {
      using T = decltype(one);
      const T* p = static_cast<const T*>(e.g) + i;
      if ((reinterpret_cast<uintptr_t>(p) & 15) == 0)
        for (; w + 4 <= end && i - lane * 8 + 4 * kBlock <= e.n; w += 4, i += 4 * kBlock, p += 4 * kBlock) {
          Raw8<T> r[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) stream8(p + u * kBlock, r[u]);
          F2 q = f2(0.f);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            F2 f[4];
            r[u].get(f);
#pragma unroll
            for (int j = 0; j < 4; ++j) q = fma2(f[j], f[j], q);
          }
          s[0] += sum2(q);
        }
      for (; w < end; ++w, i += kBlock) {
        Eight r;
        F2 f[4], q = f2(0.f);
        if (whole(e.g, i - lane * 8, e.n)) take(e.g, e.dtype, i, r);
        else take_each<T>(e.g, i, e.n, r);
        open8(r, e.dtype, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) q = fma2(f[j], f[j], q);
        s[0] += sum2(q);
      }
    };
    if (e.dtype == LORA_BF16) sum(bf16{});
    else sum(float{});
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
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if (lane == 0) tot[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    t = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += tot[i];
    const float norm = sqrtf((float)t) * fabsf(a.grad_scale);
    a.norm_out[0] = norm;
    const float clip = a.max_norm > 0.f ? fminf(1.f, a.max_norm / (norm + 1e-6f)) : 1.f;
    a.norm_out[1] = isfinite(norm) ? a.grad_scale * clip : nanf("");
  }
}

inline bool t_used(const lora_adamw_tensor& t, const void* grad) { return t.n > 0 && grad; }

lora_status check_table(const lora_adamw_tensor* t, const void* const* grads, int64_t count, int64_t* used) {
  if (count < 0 || (count > 0 && (!t || !grads))) return LORA_ERR_INVALID_ARG;
  int64_t b = 0, u = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n < 0) return LORA_ERR_INVALID_ARG;
    if (t[i].dtype != LORA_F32 && t[i].dtype != LORA_BF16) return LORA_ERR_INVALID_ARG;
    if (!isfinite(t[i].lr_mul) || !isfinite(t[i].weight_decay)) return LORA_ERR_INVALID_ARG;
    b += (t[i].n + kBlock - 1) / kBlock;
    if (b > 1LL << 30) return LORA_ERR_UNSUPPORTED;
    if (!t_used(t[i], grads[i])) continue;
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
// The launch's own numbering goes by `unit` blocks, the last of a tensor may be part of one.
template <int N, typename F>
lora_status over_table(const lora_adamw_tensor* t, const void* const* grads, int64_t count, int64_t used, AdamArgs a,
                       int unit, F launch) {
  AdamTable<N> table;
  int32_t state = 0;
  int64_t i = 0, left = used;
  while (left > 0) {
    a.count = 0;
    a.blocks = 0;
    for (; i < count && a.count < N; ++i) {
      const int32_t nb = (int32_t)((t[i].n + kBlock - 1) / kBlock);
      if (t_used(t[i], grads[i])) {
        table.e[a.count++] =
            AdamEntry{t[i].p, grads[i], t[i].n, a.blocks, state, t[i].dtype, t[i].lr_mul, t[i].weight_decay};
        a.blocks += (nb + unit - 1) / unit;
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

lora_status adamw_fill_master(const lora_adamw_tensor* tensors, int64_t count, float* master, void* stream) {
  if (count < 0 || (count > 0 && !tensors)) return LORA_ERR_INVALID_ARG;
  // every tensor counts here: its own pointer stands in for a gradient
  const void** self = static_cast<const void**>(malloc((size_t)(count > 0 ? count : 1) * sizeof(void*)));
  if (!self) return LORA_ERR_INVALID_ARG;
  for (int64_t i = 0; i < count; ++i) self[i] = tensors[i].p;
  int64_t used = 0;
  lora_status e = check_table(tensors, self, count, &used);
  for (int64_t i = 0; e == LORA_OK && i < count; ++i)
    if (tensors[i].n > 0 && !tensors[i].p) e = LORA_ERR_INVALID_ARG;
  if (e == LORA_OK && used > 0 && !master) e = LORA_ERR_INVALID_ARG;
  if (e == LORA_OK && !al16(master)) e = LORA_ERR_MISALIGNED;
  if (e == LORA_OK && used > 0) {
    AdamArgs a = {};
    a.master = master;
    e = over_table<kTable>(tensors, self, count, used, a, 1, [&](AdamArgs& b, const AdamTable<kTable>& t) {
      b.rounds = 1;
      CK(launch_pdl(adamw_master_kernel<kTable>, dim3((unsigned)((b.blocks + 7) / 8)), dim3(256), 0,
                    static_cast<cudaStream_t>(stream), b, t));
      return LORA_OK;
    });
  }
  free(self);
  return e;
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
    return over_table<kSmallTable>(tensors, grads, count, used, a, 1, [&](AdamArgs& b, const AdamTable<kSmallTable>& t) {
      return run(adamw_norm_kernel<kSmallTable>, b, t);
    });
  return over_table<kTable>(tensors, grads, count, used, a, 1, [&](AdamArgs& b, const AdamTable<kTable>& t) {
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
  // as the kernels have them; an eps below the normal numbers leaves elements without a gradient 0 / 0
  if (!((float)h.eps >= FLT_MIN) || !isfinite((float)h.eps) || !isfinite((float)h.lr) || !isfinite((float)h.grad_scale))
    return LORA_ERR_INVALID_ARG;
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
  // Two rounds a chunk; with 32-bit states a CTA for each chunk (448 tensors of 42 M elements, bf16: 174 us;
  // with one round 180, four 181, eight 188), with 8-bit ones as many CTAs as are resident, which know their
  // next blocks (168 M elements, one block at a time: 473 us against 630).
  const auto run = [&](auto kernel, AdamArgs& b, const auto& table, bool stay) {
    const int64_t slots = (stay ? kStep8Ctas : kStepCtas) * (int64_t)num_sms_current(), eights = (b.blocks + 7) / 8;
    b.rounds = eights >= 2 * slots ? 2 : 1;
    const int64_t chunks = (eights + b.rounds - 1) / b.rounds;
    CK(launch_pdl(kernel, dim3((unsigned)(stay && chunks > slots ? slots : chunks)), dim3(256), 0, st, b, table));
    return LORA_OK;
  };
  int kind = a.master ? KIND_BF16 : KIND_ANY;
  int64_t narrow = 0;
  for (int64_t i = 0; i < count; ++i) narrow += t_used(tensors[i], grads[i]) && tensors[i].dtype == LORA_BF16;
  if (narrow == 0) kind = KIND_F32;
  else if (narrow != used) kind = KIND_ANY;
  const auto step = [&](auto size, auto which) {
    constexpr int N = decltype(size)::value, K = decltype(which)::value;
    return over_table<N>(tensors, grads, count, used, a, a.bits == 8 ? kPair : 1, [&](AdamArgs& b, const AdamTable<N>& t) {
      return b.bits == 8 ? run(adamw8_kernel<N, K>, b, t, true) : run(adamw_kernel<N, K>, b, t, false);
    });
  };
  const auto sized = [&](auto which) {
    if (used <= kSmallTable) return step(std::integral_constant<int, kSmallTable>{}, which);
    return step(std::integral_constant<int, kTable>{}, which);
  };
  if (kind == KIND_BF16) return sized(std::integral_constant<int, KIND_BF16>{});
  if (kind == KIND_F32) return sized(std::integral_constant<int, KIND_F32>{});
  return sized(std::integral_constant<int, KIND_ANY>{});
}

}  // extern "C"
