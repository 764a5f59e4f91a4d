// Pieces shared by the attention kernels over packed prompt rows: which request a row tile
// belongs to, and what its rows see.
#pragma once

#include "d2f_internal.cuh"

namespace d2f {

// Row tiles of the packed requests, tile_q queries each, without a prefix sum over their tile
// counts: request b's tiles are numbered from S_b = row_start[b] / tile_q + b. Since
// row_start[b+1] / tile_q - row_start[b] / tile_q + 1 >= ceil(n_b / tile_q), the numbers do not
// overlap; the few that no tile takes are empty items. S_b grows with b, so the request of a
// tile is found by search.
struct SeqTile {
  int b, q0, n, C, tile;  // request, its first row, rows, cached tokens; tile within the request
  bool live;              // the tile has rows and the request's lengths are consistent
  bool bad;               // they are not
};

// The request whose tiles hold number t (the last b with S_b <= t); all 32 lanes call this with
// the same t. Each step probes 32 places between the bounds.
__device__ __forceinline__ int seq_find(const int32_t *row_start, int batch, int tile_q, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;  // S_lo <= t (S_0 = 0 where row_start is consistent), S_hi > t
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33;
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && (long long)(__ldg(row_start + at) / tile_q) + at <= t;
    // (a row_start that does not grow gives some request here; its rows are checked after)
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
}

__device__ __forceinline__ SeqTile seq_tile(const PromptArgs &a, int t) {
  SeqTile s;
  s.b = seq_find(a.row_start, a.batch, a.tile_q, t);
  s.q0 = __ldg(a.row_start + s.b);
  const int q1 = __ldg(a.row_start + s.b + 1);
  s.C = a.ctx_len ? __ldg(a.ctx_len + s.b) : 0;
  s.n = q1 - s.q0;
  s.bad = !(s.q0 >= 0 && q1 >= s.q0 && q1 <= a.rows && s.C >= 0 &&
            (long long)s.C <= (long long)a.max_pages_per_seq * a.block_size);
  s.tile = t - (s.q0 / a.tile_q + s.b);
  s.live = !s.bad && s.tile >= 0 && (long long)s.tile * a.tile_q < s.n;
  return s;
}

// New rows that row i of a request of n rows sees: [0, seq_limit).
__device__ __forceinline__ int seq_limit(int i, int n, int mask_block) {
  return min(n, (i / mask_block + 1) * mask_block);  // (mask_block <= rows + 1, checked on the host)
}

// Whether row_start and ctx_len are consistent for every request; called by one warp of the
// launch, which reports what it finds (a request that owns no tile would go unreported).
__device__ __forceinline__ void seq_report(const PromptArgs &a) {
  bool bad = false;
  for (int b = threadIdx.x & 31; b < a.batch; b += 32) {
    const int q0 = __ldg(a.row_start + b), q1 = __ldg(a.row_start + b + 1);
    const int C = a.ctx_len ? __ldg(a.ctx_len + b) : 0;
    bad |= q0 < 0 || q1 < q0 || q1 > a.rows || (b == 0 && q0 != 0) || C < 0 ||
           (long long)C > (long long)a.max_pages_per_seq * a.block_size;
  }
  if (bad) set_err(a.err, D2F_ERR_INVALID_ARG);
}

}  // namespace d2f
