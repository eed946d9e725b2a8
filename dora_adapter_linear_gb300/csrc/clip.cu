// Norms of grouped gradients over many tensors, and clipping in place: one group for each adapter that is
// trained in a batch with others.
//
//   norm_g = sqrt(sum over the group's elements x^2),  x = x min(1, max_norm / (norm_g + 1e-6)),
// and x = 0 throughout a group whose norm is not finite.
//
// A CTA of the first launch sums the squares of one unit (16384 elements of one tensor and group, all its loads on
// their way at once) in a fixed order.  A CTA of the last one scales a unit whose group's factor is not 1, last
// units first, while their elements are still in L2.  The units' sums of a group are added by one CTA for each
// group in a launch between, or, where a group has up to 512, by every CTA of the last launch for itself
// (three adapters of one small block: 3.4 us on the device, 9.2 a call, 12 with the launch between).  Bytes bound large
// sets: every element read, those above the limit read again and written.  168 M bf16 elements, half of them scaled: norms
// 53 us (6.3 TB/s), scaling 44, together 100 us of 74 at the rate of a long copy.
#include <float.h>
#include <math.h>

#include <algorithm>
#include <vector>

#include "checks.h"
#include "vec.cuh"

namespace lg {

namespace {

constexpr int kUnit = 16384;          // elements of a unit
constexpr int kSmallTable = 64, kMidTable = 192, kTable = 640;
constexpr int kFew = 512;              // sums of a group that every CTA adds for itself
constexpr int kGroups = 2048;          // groups of one launch's table of sums

struct ClipEntry {
  void* g;
  int64_t n;                          // elements of each group
  int32_t first;                      // its first unit in this launch
  int32_t units;                      // units of each group
  int32_t at;                         // the first of their sums (stacks: of group 0)
  int32_t group;                      // -1: a stack, one entry of it for each group
  int32_t gfirst, gsums;              // where the group's sums begin, and how many they are (stacks: of group 0)
  int16_t dtype, leads;               // leads: the group's first tensor
};
struct ClipArgs {
  int count;
  int32_t units;                      // of this launch
  float* parts;
  float max_norm;
  float* norms;
  float* factor;                      // of each group: 0 a group that is not finite
};
template <int N>
struct ClipTable {
  ClipEntry e[N];
};

struct Unit {
  void* p;                            // its first element
  int n;                              // elements, at most kUnit
  int group, at, gfirst, gsums;
  bool bf, leads;                     // leads: the first unit of its group
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
  r.gsums = e.gsums;
  r.gfirst = e.gfirst + k * e.gsums;
  r.at = e.at + k * e.gsums + u;
  r.leads = u == 0 && e.leads;
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
__global__ void __launch_bounds__(256, 4) clip_norm_kernel(const __grid_constant__ ClipArgs a,
                                                        const __grid_constant__ ClipTable<N> table) {
  __shared__ float red[2 * 32];
  const Unit u = unit_of(a, table, blockIdx.x);
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  float s[1] = {u.bf ? squares(static_cast<const bf16*>(u.p), u.n) : squares(static_cast<const float*>(u.p), u.n)};
  block_sums<1>(s, red, 0);
  if (threadIdx.x == 0) a.parts[u.at] = s[0];
}

// The norm of the group whose sums are parts[0 .. sums - 1], in every thread of a block of 256.  Eight at a time in
// fp32, longer runs of these in fp64, whose units are few: with each sum in fp64, as AdamW's one norm has them in a launch
// of its own, this took 4 us of every CTA.  A small fp32 set's norm is off by 4.7e-8 instead of 3.4e-8.
__device__ __forceinline__ float norm_of(const float* parts, int sums, float* tot) {
  auto eight = [&](int i) {
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = i + 256 * q < sums ? parts[i + 256 * q] : 0.f;
    return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
  };
  float s = eight(threadIdx.x);
  if (sums > 2048) {
    double t = (double)s;
    for (int i = threadIdx.x + 2048; i < sums; i += 2048) t += (double)eight(i);
    s = (float)t;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) tot[threadIdx.x >> 5] = s;
  __syncthreads();
  s = ((tot[0] + tot[1]) + (tot[2] + tot[3])) + ((tot[4] + tot[5]) + (tot[6] + tot[7]));
  return sqrtf(s);
}
__device__ __forceinline__ float factor_of(float norm, float max_norm) {
  return isfinite(norm) ? fminf(1.f, max_norm / (norm + 1e-6f)) : 0.f;
}

// where the sums of a launch's groups begin and how many they are: of stacks the same number for each
template <int N>
struct Sums {
  int32_t group0, each;
  int32_t first[N], sums[N];
};
template <int N>
__global__ void __launch_bounds__(256) clip_factor_kernel(const __grid_constant__ ClipArgs a,
                                                          const __grid_constant__ Sums<N> table) {
  __shared__ float tot[8];
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int k = blockIdx.x, g = table.group0 + k;
  const float norm = N > 1 ? norm_of(a.parts + table.first[N > 1 ? k : 0], table.sums[N > 1 ? k : 0], tot)
                           : norm_of(a.parts + (int64_t)g * table.each, table.each, tot);
  if (threadIdx.x == 0) {
    a.norms[g] = norm;
    a.factor[g] = factor_of(norm, a.max_norm);
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

template <int N, bool FEW>
__global__ void __launch_bounds__(256) clip_scale_kernel(const __grid_constant__ ClipArgs a,
                                                         const __grid_constant__ ClipTable<N> table) {
  __shared__ float tot[8];
  const Unit u = unit_of(a, table, a.units - 1 - (int)blockIdx.x);
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  float f;
  if (FEW) {
    const float norm = norm_of(a.parts + u.gfirst, u.gsums, tot);
    if (u.leads && threadIdx.x == 0) a.norms[u.group] = norm;
    f = factor_of(norm, a.max_norm);
  } else {
    f = a.factor[u.group];
  }
  if (f == 1.f) return;
  // a factor of an infinite max_norm's finite group is 1; 0 stands for a group that is not finite
  if (u.bf) scale(static_cast<bf16*>(u.p), u.n, f, f == 0.f);
  else scale(static_cast<float*>(u.p), u.n, f, f == 0.f);
}

int64_t units_of(int64_t n) { return (n + kUnit - 1) / kUnit; }

struct ClipWs {
  float *parts, *factor;
};
size_t carve(int64_t sums, int64_t groups, char* base, ClipWs* w) {
  Carve c{base};
  w->parts = c.take<float>(sums);
  w->factor = c.take<float>(groups);
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

// Where the sums lie: those of a group behind one another, in the order of its tensors.
struct Place {
  std::vector<int32_t> at;              // of each tensor's units (stacks: of group 0)
  std::vector<int32_t> gfirst, gsums;   // of each group; stacks: of group 0 alone
  std::vector<char> leads;              // the tensor is its group's first
  int32_t most = 0;                     // sums of the largest group
  bool none = false;                    // there is a group without elements
};
Place place(const lora_grad_tensor* t, int64_t count, int64_t groups, bool stacked) {
  Place p;
  const int64_t n = stacked ? 1 : groups;
  p.at.resize(count);
  p.leads.assign(count, 0);
  p.gfirst.assign(n, 0);
  p.gsums.assign(n, 0);
  auto group = [&](int64_t i) { return stacked ? 0 : t[i].group; };
  for (int64_t i = 0; i < count; ++i) {
    const int32_t u = (int32_t)units_of(t[i].n);
    p.at[i] = p.gsums[group(i)];
    p.leads[i] = u > 0 && p.at[i] == 0;
    p.gsums[group(i)] += u;
  }
  int32_t sum = 0;
  for (int64_t g = 0; g < n; ++g) {
    p.gfirst[g] = sum;
    sum += p.gsums[g];
    if (p.gsums[g] > p.most) p.most = p.gsums[g];
    if (p.gsums[g] == 0) p.none = true;
  }
  for (int64_t i = 0; i < count; ++i) p.at[i] += p.gfirst[group(i)];
  return p;
}

template <int N, typename F>
cudaError_t over_table(const lora_grad_tensor* t, int64_t count, int64_t groups, bool stacked, ClipArgs a, const Place& p,
                       F launch) {
  ClipTable<N> table;
  int64_t i = 0;
  while (i < count) {
    a.count = 0;
    a.units = 0;
    for (; i < count && a.count < N; ++i) {
      const int32_t u = (int32_t)units_of(t[i].n), g = stacked ? 0 : t[i].group;
      if (u == 0) continue;
      table.e[a.count++] = ClipEntry{t[i].g, t[i].n, a.units, u, p.at[i], stacked ? -1 : g, p.gfirst[g], p.gsums[g],
                                     (int16_t)t[i].dtype, (int16_t)p.leads[i]};
      a.units += (int32_t)(u * (stacked ? groups : 1));
    }
    if (a.count == 0) break;
    const cudaError_t e = launch(a, table);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int N>
cudaError_t factors_of(const ClipArgs& a, const Place& p, int64_t groups, cudaStream_t st) {
  Sums<N> s;
  for (int64_t g0 = 0; g0 < groups; g0 += N) {
    const int64_t n = groups - g0 < N ? groups - g0 : N;
    s.group0 = (int32_t)g0;
    s.each = 0;
    for (int64_t g = 0; g < n; ++g) s.first[g] = p.gfirst[g0 + g], s.sums[g] = p.gsums[g0 + g];
    const cudaError_t e = launch_pdl(clip_factor_kernel<N>, dim3((unsigned)n), dim3(256), 0, st, a, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int N>
cudaError_t run(const lora_grad_tensor* t, int64_t count, int64_t groups, bool stacked, const ClipArgs& a, const Place& p,
                cudaStream_t st) {
  cudaError_t e = over_table<N>(t, count, groups, stacked, a, p, [&](const ClipArgs& b, const ClipTable<N>& table) {
    return launch_pdl(clip_norm_kernel<N>, dim3((unsigned)b.units), dim3(256), 0, st, b, table);
  });
  if (e != cudaSuccess) return e;
  const bool scales = a.max_norm > 0.f, few = scales && !p.none && p.most <= kFew;
  if (!few) {
    if (stacked) {
      const Sums<1> s{0, p.gsums[0], {0}, {0}};
      e = launch_pdl(clip_factor_kernel<1>, dim3((unsigned)groups), dim3(256), 0, st, a, s);
    } else {
      e = groups <= 64 ? factors_of<64>(a, p, groups, st) : factors_of<kGroups>(a, p, groups, st);
    }
    if (e != cudaSuccess || !scales) return e;
  }
  return over_table<N>(t, count, groups, stacked, a, p, [&](const ClipArgs& b, const ClipTable<N>& table) {
    if (few) return launch_pdl(clip_scale_kernel<N, true>, dim3((unsigned)b.units), dim3(256), 0, st, b, table);
    return launch_pdl(clip_scale_kernel<N, false>, dim3((unsigned)b.units), dim3(256), 0, st, b, table);
  });
}

}  // namespace

}  // namespace lg

using namespace lg;

extern "C" {

size_t grad_clip_workspace_bytes(const lora_grad_tensor* tensors, int64_t count, int64_t groups, int stacked) {
  const int64_t sums = check_tensors(tensors, count, groups, stacked);
  ClipWs w;
  return sums < 0 ? 0 : carve(sums, groups, nullptr, &w);
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
    const lora_status e = check_ws(ws, ws_bytes, carve(total, groups, nullptr, &w));
    if (e != LORA_OK) return e;
    carve(total, groups, static_cast<char*>(ws), &w);
    cudaStream_t st = (cudaStream_t)stream;
    const Place p = place(tensors, count, groups, stacked != 0);
    const ClipArgs a{0, 0, w.parts, max_norm, norms, w.factor};
    if (count <= kSmallTable) CK(run<kSmallTable>(tensors, count, groups, stacked != 0, a, p, st));
    else if (count <= kMidTable) CK(run<kMidTable>(tensors, count, groups, stacked != 0, a, p, st));
    else CK(run<kTable>(tensors, count, groups, stacked != 0, a, p, st));
  } catch (...) {                     // no memory on the host
    return LORA_ERR_WORKSPACE;
  }
  return LORA_OK;
}

}  // extern "C"
