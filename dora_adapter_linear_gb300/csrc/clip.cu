// Norms of grouped gradients over many tensors, and clipping in place: one group for each adapter that is
// trained in a batch with others.
//
//   norm_g = sqrt(sum over the group's elements x^2),  x = x min(1, max_norm / (norm_g + 1e-6)),
// and x = 0 throughout a group whose norm is not finite.
//
// Three launches.  A CTA of the first sums the squares of one unit (16384 elements of one tensor and group,
// all its loads on their way at once) in a fixed order; a CTA of the second adds the units' sums of one
// group (fp64); the third scales the groups whose factor is not 1, last units first, while their elements
// are still in L2.  Bytes bound large sets: every element read, those above the limit read again and written.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <vector>

#include "checks.h"
#include "vec.cuh"

namespace lg {

namespace {

constexpr int kUnit = 16384;          // elements of a unit
constexpr int kSmallTable = 64, kTable = 640;

struct ClipEntry {
  void* g;
  int64_t n;                          // elements of each group
  int32_t first;                      // its first unit in this launch
  int32_t units;                      // units of each group
  int32_t at;                         // the first of their sums (stacks: of group 0)
  int32_t group;                      // -1: a stack, one entry of it for each group
  int32_t sums;                       // sums of the group, on the group's first tensor; 0 elsewhere
  int32_t dtype;
};
struct ClipArgs {
  int count;
  int32_t units, per_group;           // of this launch; sums of each group of stacks
  float* parts;
  int32_t *gfirst, *gsums;            // where a group's sums begin and how many there are (lists)
  const float* factor;                // of each group: 0 a group that is not finite
};
template <int N>
struct ClipTable {
  ClipEntry e[N];
};

struct Unit {
  void* p;                            // its first element
  int n;                              // elements, at most kUnit
  int group, at, bf;
  bool leads;                         // the first unit of its group's first tensor
  int sums;
};
template <int N>
__device__ __forceinline__ Unit unit_of(const ClipArgs& a, const ClipTable<N>& t, int i) {
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.e[mid].first <= i) lo = mid;
    else hi = mid;
  }
  const ClipEntry& e = t.e[lo];
  const int v = i - e.first, k = e.group < 0 ? v / e.units : 0, u = v - k * e.units;
  const int64_t off = (int64_t)u * kUnit;
  Unit r;
  r.bf = e.dtype == LORA_BF16;
  r.p = static_cast<char*>(e.g) + (k * e.n + off) * (r.bf ? 2 : 4);
  r.n = (int)(e.n - off < kUnit ? e.n - off : kUnit);
  r.group = e.group < 0 ? k : e.group;
  r.at = e.at + k * a.per_group + u;
  r.leads = v == 0 && e.sums > 0;
  r.sums = e.sums;
  return r;
}

template <typename T>
__device__ __forceinline__ float squares(const T* p, int n) {
  float s = 0.f;
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    Raw8<T> r[kUnit / 2048];
#pragma unroll
    for (int i = 0; i < kUnit / 2048; ++i) {
      const int at = (i * 256 + threadIdx.x) * 8;
      if (at + 8 <= n) r[i] = *reinterpret_cast<const Raw8<T>*>(p + at);
    }
    F2 q = f2(0.f);
#pragma unroll
    for (int i = 0; i < kUnit / 2048; ++i)
      if ((i * 256 + (int)threadIdx.x) * 8 + 8 <= n) {
        F2 f[4];
        r[i].get(f);
#pragma unroll
        for (int j = 0; j < 4; ++j) q = fma2(f[j], f[j], q);
      }
    s = sum2(q);
    const int at = (n & ~7) + (int)threadIdx.x;
    if (at < n) s = fmaf(to_f(p[at]), to_f(p[at]), s);
  } else {
    for (int at = threadIdx.x; at < n; at += 256) s = fmaf(to_f(p[at]), to_f(p[at]), s);
  }
  return s;
}

template <int N>
__global__ void __launch_bounds__(256) clip_norm_kernel(const __grid_constant__ ClipArgs a,
                                                        const __grid_constant__ ClipTable<N> table) {
  __shared__ float red[2 * 32];
  const Unit u = unit_of(a, table, blockIdx.x);
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  float s[1] = {u.bf ? squares(static_cast<const bf16*>(u.p), u.n) : squares(static_cast<const float*>(u.p), u.n)};
  block_sums<1>(s, red, 0);
  if (threadIdx.x == 0) {
    a.parts[u.at] = s[0];
    if (a.gfirst && u.leads) {
      a.gfirst[u.group] = u.at;
      a.gsums[u.group] = u.sums;
    }
  }
}

__global__ void __launch_bounds__(256) clip_factor_kernel(const float* parts, const int32_t* gfirst, const int32_t* gsums,
                                                          int per_group, float max_norm, float* norms, float* factor) {
  __shared__ double tot[8];
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int g = blockIdx.x;
  const int first = gfirst ? gfirst[g] : g * per_group, sums = gfirst ? gsums[g] : per_group;
  double t = 0.0;
  for (int i = threadIdx.x; i < sums; i += 256) t += (double)parts[first + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  if ((threadIdx.x & 31) == 0) tot[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    t = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += tot[i];
    const float norm = sqrtf((float)t);
    norms[g] = norm;
    factor[g] = isfinite(norm) ? fminf(1.f, max_norm / (norm + 1e-6f)) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void scale(T* p, int n, float f, bool zero) {
  auto one = [&](int at) { p[at] = from_f<T>(zero ? 0.f : to_f(p[at]) * f); };
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const F2 f2f = f2(f);
    F2 x[kUnit / 4096][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < kUnit / 4096; ++i) {
        const int at = ((h * (kUnit / 4096) + i) * 256 + threadIdx.x) * 8;
        if (at + 8 <= n) load4x2(p + at, x[i]);
      }
#pragma unroll
      for (int i = 0; i < kUnit / 4096; ++i) {
        const int at = ((h * (kUnit / 4096) + i) * 256 + threadIdx.x) * 8;
        if (at + 8 <= n) {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[i][j] = zero ? f2(0.f) : mul2(x[i][j], f2f);
          store4x2(p + at, x[i]);
        }
      }
    }
    const int at = (n & ~7) + (int)threadIdx.x;
    if (at < n) one(at);
  } else {
    for (int at = threadIdx.x; at < n; at += 256) one(at);
  }
}

template <int N>
__global__ void __launch_bounds__(256) clip_scale_kernel(const __grid_constant__ ClipArgs a,
                                                         const __grid_constant__ ClipTable<N> table) {
  const Unit u = unit_of(a, table, a.units - 1 - (int)blockIdx.x);
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const float f = a.factor[u.group];
  if (f == 1.f) return;
  // a factor of an infinite max_norm's finite group is 1; 0 stands for a group that is not finite
  if (u.bf) scale(static_cast<bf16*>(u.p), u.n, f, f == 0.f);
  else scale(static_cast<float*>(u.p), u.n, f, f == 0.f);
}

int64_t units_of(int64_t n) { return (n + kUnit - 1) / kUnit; }

struct ClipWs {
  float *parts, *factor;
  int32_t* group;                     // [2, groups] of lists
};
size_t carve(int64_t sums, int64_t groups, bool stacked, char* base, ClipWs* w) {
  Carve c{base};
  w->parts = c.take<float>(sums);
  w->factor = c.take<float>(groups);
  w->group = stacked ? nullptr : c.take<int32_t>(2 * groups);
  return c.off;
}

// Sums of all units, or an error: negative.  Units are counted in 31 bits.
int64_t check_tensors(const lora_grad_tensor* t, int64_t count, int64_t groups, int stacked) {
  if (count < 0 || groups < 1 || (count > 0 && !t)) return -LORA_ERR_INVALID_ARG;
  if (groups > 65535) return -LORA_ERR_UNSUPPORTED;
  int64_t sums = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n < 0 || (t[i].dtype != LORA_F32 && t[i].dtype != LORA_BF16)) return -LORA_ERR_INVALID_ARG;
    if (!stacked && (t[i].group < 0 || t[i].group >= groups)) return -LORA_ERR_INVALID_ARG;
    if (t[i].n > 0 && !t[i].g) return -LORA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(t[i].g) % (t[i].dtype == LORA_BF16 ? 2 : 4)) return -LORA_ERR_MISALIGNED;
    const int64_t u = units_of(t[i].n);
    if (u > 0x7fffffff) return -LORA_ERR_UNSUPPORTED;
    sums += u * (stacked ? groups : 1);
    if (sums > 0x7fffffff) return -LORA_ERR_UNSUPPORTED;
  }
  return sums;
}

// whether two tensors share an element: it would be scaled under the other's hands
bool overlap(const lora_grad_tensor* t, int64_t count, int64_t each) {
  typedef std::pair<uintptr_t, uintptr_t> Span;
  std::vector<Span> s;
  s.reserve(count);
  bool ordered = true;
  for (int64_t i = 0; i < count; ++i) {
    if (t[i].n == 0) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(t[i].g);
    s.push_back(Span(p, p + (uintptr_t)t[i].n * each * (t[i].dtype == LORA_BF16 ? 2 : 4)));
    ordered = ordered && (s.size() < 2 || s[s.size() - 2].second <= p);
  }
  if (ordered) return false;
  std::sort(s.begin(), s.end());
  for (size_t i = 1; i < s.size(); ++i)
    if (s[i - 1].second > s[i].first) return true;
  return false;
}

template <int N, typename F>
cudaError_t over_table(const lora_grad_tensor* t, int64_t count, int64_t groups, bool stacked, ClipArgs a,
                       const std::vector<int32_t>& at, const std::vector<int32_t>& sums, F launch) {
  ClipTable<N> table;
  int64_t i = 0;
  while (i < count) {
    a.count = 0;
    a.units = 0;
    for (; i < count && a.count < N; ++i) {
      const int32_t u = (int32_t)units_of(t[i].n);
      if (u == 0) continue;
      table.e[a.count++] = ClipEntry{t[i].g, t[i].n, a.units, u, at[i], stacked ? -1 : t[i].group, sums[i], t[i].dtype};
      a.units += (int32_t)(u * (stacked ? groups : 1));
    }
    if (a.count == 0) break;
    const cudaError_t e = launch(a, table);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int N>
cudaError_t run(const lora_grad_tensor* t, int64_t count, int64_t groups, bool stacked, float max_norm, float* norms,
                ClipArgs a, const ClipWs& w, const std::vector<int32_t>& at, const std::vector<int32_t>& sums,
                cudaStream_t st) {
  cudaError_t e = over_table<N>(t, count, groups, stacked, a, at, sums, [&](const ClipArgs& b, const ClipTable<N>& table) {
    return launch_pdl(clip_norm_kernel<N>, dim3((unsigned)b.units), dim3(256), 0, st, b, table);
  });
  if (e != cudaSuccess) return e;
  e = launch_pdl(clip_factor_kernel, dim3((unsigned)groups), dim3(256), 0, st, (const float*)w.parts,
                 (const int32_t*)a.gfirst, (const int32_t*)a.gsums, (int)a.per_group, max_norm, norms, w.factor);
  if (e != cudaSuccess || !(max_norm > 0.f)) return e;
  return over_table<N>(t, count, groups, stacked, a, at, sums, [&](const ClipArgs& b, const ClipTable<N>& table) {
    return launch_pdl(clip_scale_kernel<N>, dim3((unsigned)b.units), dim3(256), 0, st, b, table);
  });
}

}  // namespace

}  // namespace lg

using namespace lg;

extern "C" {

size_t grad_clip_workspace_bytes(const lora_grad_tensor* tensors, int64_t count, int64_t groups, int stacked) {
  const int64_t sums = check_tensors(tensors, count, groups, stacked);
  ClipWs w;
  return sums < 0 ? 0 : carve(sums, groups, stacked != 0, nullptr, &w);
}

lora_status grad_clip(const lora_grad_tensor* tensors, int64_t count, int64_t groups, int stacked, float max_norm,
                      float* norms, void* ws, size_t ws_bytes, void* stream) {
  const int64_t total = check_tensors(tensors, count, groups, stacked);
  if (total < 0) return (lora_status)-total;
  REQ(norms);
  if (reinterpret_cast<uintptr_t>(norms) & 3) return LORA_ERR_MISALIGNED;
  if (isnan(max_norm)) return LORA_ERR_INVALID_ARG;
  try {
    if (overlap(tensors, count, stacked ? groups : 1)) return LORA_ERR_INVALID_ARG;
    ClipWs w;
    const lora_status e = check_ws(ws, ws_bytes, carve(total, groups, stacked != 0, nullptr, &w));
    if (e != LORA_OK) return e;
    carve(total, groups, stacked != 0, static_cast<char*>(ws), &w);
    cudaStream_t st = (cudaStream_t)stream;
    ClipArgs a = {};
    a.parts = w.parts;
    a.factor = w.factor;
    // where the sums of each tensor begin, those of a group behind one another
    std::vector<int32_t> at(count), sums(count, 0);
    if (stacked) {
      int32_t n = 0;
      for (int64_t i = 0; i < count; ++i) at[i] = n, n += (int32_t)units_of(tensors[i].n);
      a.per_group = n;
    } else {
      a.gfirst = w.group;
      a.gsums = w.group + groups;
      std::vector<int32_t> next(groups, 0), lead(groups, -1);
      for (int64_t i = 0; i < count; ++i) {
        const int32_t u = (int32_t)units_of(tensors[i].n), g = tensors[i].group;
        if (u > 0 && lead[g] < 0) lead[g] = (int32_t)i;
        next[g] += u;
      }
      int32_t n = 0;
      for (int64_t g = 0; g < groups; ++g) {
        if (lead[g] >= 0) sums[lead[g]] = next[g];
        const int32_t k = next[g];
        next[g] = n;
        n += k;
      }
      for (int64_t i = 0; i < count; ++i) at[i] = next[tensors[i].group], next[tensors[i].group] += (int32_t)units_of(tensors[i].n);
      CK(cudaMemsetAsync(w.group, 0, 2 * groups * sizeof(int32_t), st));   // groups without tensors
    }
    if (count <= kSmallTable) CK(run<kSmallTable>(tensors, count, groups, stacked, max_norm, norms, a, w, at, sums, st));
    else CK(run<kTable>(tensors, count, groups, stacked, max_norm, norms, a, w, at, sums, st));
  } catch (...) {                     // no memory on the host
    return LORA_ERR_WORKSPACE;
  }
  return LORA_OK;
}

}  // extern "C"
