// The plan of a batch whose rows have different adapters: rows sorted by adapter, work items, and for
// every GEMM tile the adapters among its rows.
//
// One launch.  Block 0 sorts: a counting sort by 8 bits of the adapter's number a pass (one pass up to
// 255 adapters), stable, so that every sum over an adapter's rows has one fixed order.  Each warp counts
// and places a run of consecutive rows; rows of equal digit within 32 find their order by a warp match.
// The other blocks take four tiles each.  Once for all projections of a batch, bound by latency: 6 us for a row of eight
// adapters, 15 for 8192 rows of eight, 34 of 256 in any order (two passes).  One block sorts and lists whatever the sizes
// are: 106 us for 65536 rows of eight adapters, 1.6 ms for 2^20, 41 ms for 2^24 (104 of 65535 adapters); and one thread
// writes where the adapters between two neighbouring numbers begin: 211 us for a row of one of 65535.
#include "common.cuh"
#include "multi.h"

namespace lg {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

__device__ __forceinline__ int id_of(const void* ids, int bits, int64_t row, int n) {
  if (bits == 64) {
    const int64_t v = static_cast<const int64_t*>(ids)[row];
    return v >= 0 && v < n ? (int)v : -1;
  }
  const int32_t v = static_cast<const int32_t*>(ids)[row];
  return v >= 0 && v < n ? v : -1;
}

// exclusive prefix sums of one value a thread over the block; *total: the sum of all
__device__ int block_prefix(int v, int32_t* red, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31) red[warp] = s;
  __syncthreads();
  int w = lane < kWarps ? red[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  __syncthreads();
  return s - v + (warp ? before : 0);
}

// the last adapter whose first entry is at or before i (start[0] = 0 <= i < start[n])
__device__ __forceinline__ int owner_of(const int32_t* start, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ void sort_rows(const MultiPlan& p, const void* ids, int bits, int32_t (*count)[256], int32_t* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = p.n;
  const int64_t M = p.M;
  auto key = [&](int64_t row) {      // n for rows without an adapter: behind all others
    const int a = id_of(ids, bits, row, n);
    return a < 0 ? n : a;
  };
  int passes = 1;
  while (n >> (8 * passes)) ++passes;
  const int64_t per = ((M + kWarps - 1) / kWarps + 31) & ~int64_t(31);
  const int64_t r0 = min(M, per * warp), r1 = min(M, r0 + per);
  // the last pass writes p.order
  for (int pass = 0; pass < passes; ++pass) {
    int32_t* dst = (passes - pass) & 1 ? p.order : p.other;
    const int32_t* src = pass == 0 ? nullptr : dst == p.order ? p.other : p.order;
    for (int i = threadIdx.x; i < kWarps * 256; i += kThreads) (&count[0][0])[i] = 0;
    __syncthreads();
    for (int64_t i = r0; i < r1; i += 32) {
      const bool on = i + lane < r1;
      const int64_t row = on ? (src ? src[i + lane] : i + lane) : 0;
      const int d = on ? (key(row) >> (8 * pass)) & 255 : 256 + lane;
      const uint32_t same = __match_any_sync(0xffffffffu, d);
      if (on && (same & ((1u << lane) - 1)) == 0) count[warp][d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    int sum = 0;
    if (threadIdx.x < 256)
      for (int w = 0; w < kWarps; ++w) sum += count[w][threadIdx.x];
    int total;
    int at = block_prefix(sum, red, &total);
    if (threadIdx.x < 256)
      for (int w = 0; w < kWarps; ++w) {
        const int c = count[w][threadIdx.x];
        count[w][threadIdx.x] = at;
        at += c;
      }
    __syncthreads();
    for (int64_t i = r0; i < r1; i += 32) {
      const bool on = i + lane < r1;
      const int64_t row = on ? (src ? src[i + lane] : i + lane) : 0;
      const int d = on ? (key(row) >> (8 * pass)) & 255 : 256 + lane;
      const uint32_t same = __match_any_sync(0xffffffffu, d), before = same & ((1u << lane) - 1);
      if (on) dst[count[warp][d] + __popc(before)] = (int32_t)row;
      __syncwarp();
      if (on && before == 0) count[warp][d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
  }
  // where each adapter's rows begin: position i begins all adapters after its predecessor's
  for (int64_t i = threadIdx.x; i <= M; i += kThreads) {
    const int a = i < M ? key(p.order[i]) : n, b = i > 0 ? key(p.order[i - 1]) : -1;
    for (int k = b + 1; k <= a; ++k) p.start[k] = (int32_t)i;
  }
  __syncthreads();
  int items = 0, pieces = 0;
  for (int a0 = 0; a0 < n; a0 += kThreads) {
    const int a = a0 + threadIdx.x;
    const int rows = a < n ? p.start[a + 1] - p.start[a] : 0;
    int t;
    const int i = block_prefix((rows + kItemRows - 1) / kItemRows, red, &t);
    if (a < n) p.istart[a] = items + i;
    items += t;
    const int j = block_prefix((rows + kPieceRows - 1) / kPieceRows, red, &t);
    if (a < n) p.pstart[a] = pieces + j;
    pieces += t;
  }
  if (threadIdx.x == 0) {
    p.istart[n] = p.head[kHeadItems] = items;
    p.pstart[n] = p.head[kHeadPieces] = pieces;
    p.head[kHeadRows] = p.start[n];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < items; i += kThreads) {
    const int a = owner_of(p.istart, n, i), first = p.start[a] + (i - p.istart[a]) * kItemRows;
    p.items[i] = make_int4(a, first, min(kItemRows, p.start[a + 1] - first), 0);
  }
  for (int i = threadIdx.x; i < pieces; i += kThreads) {
    const int a = owner_of(p.pstart, n, i), first = p.start[a] + (i - p.pstart[a]) * kPieceRows;
    p.pieces[i] = make_int4(a, first, min(kPieceRows, p.start[a + 1] - first), p.pstart[a + 1] - p.pstart[a] > 1);
  }
  __syncthreads();
  // partials are numbered among the pieces that have one
  int slots = 0;
  for (int i0 = 0; i0 < pieces; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const int own = i < pieces ? p.pieces[i].w : 0;
    int t;
    const int at = block_prefix(own, red, &t);
    if (i < pieces) p.pieces[i].w = own ? slots + at : -1;
    slots += t;
  }
}

__global__ void __launch_bounds__(kThreads) multi_plan_kernel(MultiPlan p, const void* ids, int bits) {
  __shared__ int32_t count[kWarps][256];
  __shared__ int32_t red[kWarps];
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  if (blockIdx.x == 0) {
    sort_rows(p, ids, bits, count, red);
    return;
  }
  // four tiles, 256 threads each
  const int q = threadIdx.x >> 8, t = threadIdx.x & 255, lane = t & 31, w = t >> 5;
  const int64_t tile = (int64_t)(blockIdx.x - 1) * 4 + q, row = tile * kTileRows + t;
  int32_t* id = count[4 * q];                                       // [256]
  int32_t* slot = count[4 * q + 1];                                 // [256]
  const int a = row < p.M ? id_of(ids, bits, row, p.n) : -1;
  if (row < p.M) p.ids[row] = a;
  id[t] = a;
  __syncthreads();
  int first = t;                                                     // the first row of the same adapter
  for (int j = 0; j < t; ++j)
    if (id[j] == a) {
      first = j;
      break;
    }
  const uint32_t firsts = __ballot_sync(0xffffffffu, a >= 0 && first == t);
  if (lane == 0) red[8 * q + w] = __popc(firsts);
  __syncthreads();
  int at = __popc(firsts & ((1u << lane) - 1)), all = 0;
  for (int j = 0; j < 8; ++j) {
    const int c = red[8 * q + j];
    if (j < w) at += c;
    all += c;
  }
  slot[t] = at;
  __syncthreads();
  if (tile * kTileRows >= p.M) return;
  if (t == 0) p.tcount[tile] = all;
  if (a >= 0 && first == t) p.tlist[tile * kTileRows + at] = a;
  const int mine = a >= 0 ? slot[first] : -1;
  // word w of an adapter's mask: the rows 32 w .. 32 w + 31 that are not its own
  for (int s = 0; s < all; ++s) {
    const uint32_t not_mine = __ballot_sync(0xffffffffu, mine != s);
    if (lane == 0) p.tmask[(tile * kTileRows + s) * 8 + w] = not_mine;
  }
}

}  // namespace

cudaError_t multi_plan(const MultiPlan& p, const void* ids, int id_bits, cudaStream_t st) {
  const unsigned blocks = 1 + (unsigned)((multi_tiles(p.M) + 3) / 4);
  return launch_pdl(multi_plan_kernel, dim3(blocks), dim3(kThreads), 0, st, p, ids, id_bits);
}

}  // namespace lg
