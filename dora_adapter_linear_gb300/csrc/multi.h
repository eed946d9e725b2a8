// Layout of an adapter plan and the launches that use it (not part of the ABI).
#pragma once

#include "checks.h"

namespace lg {

constexpr int kItemRows = 64;     // rows of an item: consecutive rows of one adapter in the plan's order
// rows of a piece, the share of one adapter's gradients that is summed at once; the partial sums of adapters with several
// are up to M / 256 of [r, d_in + d_out] in fp32 in the backward's workspace
constexpr int kPieceRows = 512;
constexpr int kTileRows = 256;    // rows of a tile, whose adapters and row masks the GEMMs take

enum { kHeadItems = 0, kHeadPieces = 1, kHeadRows = 2, kHeadWords = 64 };

// An adapter plan of M rows and n adapters: int32 words on the device.
struct MultiPlan {
  int64_t M = 0;
  int n = 0;
  int32_t* head = nullptr;     // kHead*: items, pieces, rows that have an adapter
  int32_t* ids = nullptr;      // [M] the row's adapter, -1 for none
  int32_t* order = nullptr;    // [M] rows by adapter, in their own order within one; those without one last
  int32_t* other = nullptr;    // [M] the sort's second buffer
  int32_t* start = nullptr;    // [n + 1] where an adapter's rows begin in `order`
  int32_t* istart = nullptr;   // [n + 1] its first item
  int32_t* pstart = nullptr;   // [n + 1] its first piece
  int4* items = nullptr;       // {adapter, first of its rows in `order`, their count, 0}
  int4* pieces = nullptr;      // {adapter, first, count, partial or -1: the adapter's only piece}
  int32_t* tcount = nullptr;   // [tiles] adapters among a tile's rows
  int32_t* tlist = nullptr;    // [tiles, kTileRows] which, by their first row
  uint32_t* tmask = nullptr;   // [tiles, kTileRows, 8] the tile's rows that are NOT this adapter's
};
inline int64_t multi_tiles(int64_t M) { return (M + kTileRows - 1) / kTileRows; }
inline int64_t multi_used(int64_t M, int64_t n) { return M < n ? M : n; }   // adapters that may have rows
inline int64_t multi_items(int64_t M, int64_t n) { return M / kItemRows + multi_used(M, n); }
inline int64_t multi_pieces(int64_t M, int64_t n) { return M / kPieceRows + multi_used(M, n); }
// pieces that are not their adapter's only one: at most twice the whole pieces that there are
inline int64_t multi_partials(int64_t M) { return 2 * (M / kPieceRows); }

inline size_t multi_plan_layout(int64_t M, int64_t n, char* base, MultiPlan* p) {
  Carve c{base};
  p->M = M;
  p->n = (int)n;
  p->head = c.take<int32_t>(kHeadWords);
  p->ids = c.take<int32_t>(M);
  p->order = c.take<int32_t>(M);
  p->other = c.take<int32_t>(M);
  p->start = c.take<int32_t>(n + 1);
  p->istart = c.take<int32_t>(n + 1);
  p->pstart = c.take<int32_t>(n + 1);
  p->items = c.take<int4>(multi_items(M, n));
  p->pieces = c.take<int4>(multi_pieces(M, n));
  p->tcount = c.take<int32_t>(multi_tiles(M));
  p->tlist = c.take<int32_t>(multi_tiles(M) * kTileRows);
  p->tmask = c.take<uint32_t>(multi_tiles(M) * kTileRows * 8);
  return c.off;
}

cudaError_t multi_plan(const MultiPlan& p, const void* ids, int id_bits, cudaStream_t st);

// bf16 rank-r passes (multi_rank.cu); s_a is each[a], or `one` when each is null.
// T_i = S_i U_a^T (U_a [r, K], or kr: [K, r]): plain = T, scaled = s_a T, rest = what scaled's rounding left of s_a T,
// [M, r], each may be null.  Rows without adapter: zeros in plain, nothing in the others.
// all: the product that follows has tiles for all multiprocessors
cudaError_t multi_proj(const MultiPlan& p, int64_t K, int r, const bf16* S, const bf16* U, bool kr, float one,
                       const float* each, bf16* plain, bf16* scaled, bf16* rest, bool all, cudaStream_t st);
// out_a(j, k) = sum over its rows S[i][k] T[i][j] (scaled: times s_a), out_a [r, K], or kr: [K, r]; T + T2 where T2 is
// given; adapters with several pieces leave part [multi_partials, ...] for multi_sum, which also sets those without rows
// to zero
// early: see PdlEarly; beside: with little shared memory, to run on the multiprocessors of a large product
cudaError_t multi_reduce(const MultiPlan& p, int64_t K, int r, const bf16* S, const bf16* T, const bf16* T2, bool kr,
                         bool scaled, float one, const float* each, float* part, bf16* out, bool early, bool beside,
                         cudaStream_t st);
// copies of matrices [rows, K] in rows of multi_pad_ld(K) elements, `to` null: none; beside the kernel before it
struct MultiPad {
  const bf16* from;
  bf16* to;
  int64_t rows, K;
};
inline bool multi_pad_odd(int64_t K) { return K % 16 == 8; }
inline int64_t multi_pad_ld(int64_t K) { return (K + 63) / 64 * 64; }
cudaError_t multi_pad(const MultiPad& S, const MultiPad& W, cudaStream_t st);
// sums [K]: the column sums from multi_colsum, or null
cudaError_t multi_sum(const MultiPlan& p, int64_t size0, const float* part0, bf16* out0, int64_t size1, const float* part1,
                      bf16* out1, int64_t K, const float* csum, bf16* sums, cudaStream_t st);
// The whole bf16 forward of a few rows (multi_few.cu); sz: fp32 [M, r]
constexpr int kFewRows = 256;                        // the most that it takes
bool multi_few_fits(int64_t M, int64_t N);           // whether it is the faster way
cudaError_t multi_few_fwd(const MultiPlan& p, int64_t N, int64_t K, int r, const bf16* X, const bf16* W0,
                          const bf16* A, const bf16* B, const bf16* bias, float one, const float* each, float* sz,
                          bf16* Y, bf16* Z, uint32_t* err, uint64_t timeout_ns, cudaStream_t st);
// part [multi_colsum_splits, K]: column sums of all rows of S by stretches of rows (starts early)
int multi_colsum_splits(int64_t M);
cudaError_t multi_colsum(int64_t M, int64_t K, const bf16* S, float* part, cudaStream_t st);


// fp32 (multi_f32.cu)
cudaError_t multi_f32_proj(const MultiPlan& p, int64_t K, int r, const float* S, const float* U, bool kr, float one,
                           const float* each, float* plain, float* scaled, cudaStream_t st);
// out [M, N] = S [M, K] W (W [N, K], or mn: [K, N]) + (scaled: s_a) P_i U_a (U_a [N, r], or mn: [r, N]) (+ bias)
cudaError_t multi_f32_gemm(const MultiPlan& p, int64_t N, int64_t K, int r, const float* S, const float* W, bool mn,
                           const float* P, const float* U, const float* bias, bool scaled, float one, const float* each,
                           float* out, cudaStream_t st);
// dA_a = sum G_i^T X_i, dB_a = s_a sum dY_i^T Z_i
cudaError_t multi_f32_reduce(const MultiPlan& p, int r, int64_t in, const float* X, const float* G, float* dA, int64_t out,
                             const float* dY, const float* Z, float* dB, float one, const float* each, bool early,
                             cudaStream_t st);
cudaError_t multi_f32_colsum(int64_t M, int64_t K, const float* S, float* out, cudaStream_t st);

}  // namespace lg
