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

// Splits of the keys for `grid` items: S_b = ceil(T_b / L) a row tile of request b, T_b the
// key tiles that its last rows see, with the smallest L for which the items are no more than that (and no
// item has more than L key tiles, whatever the requests' lengths). All 32 lanes call this; a lane
// holds the requests lane, lane + 32, .. Returns the row tile of item c and its place among the S
// splits and the KV heads; the splits of every request are written to `counts` (NULL: not).
constexpr int kSplitLeast = 4;  // key tiles
__device__ __forceinline__ SeqTile seq_even(const PromptArgs &a, int c, int grid, int keys, int &S, int &split,
                                            int &g, int32_t *counts) {
  constexpr int K = kPromptSplitBatch / 32;
  const int lane = threadIdx.x & 31, Hk = a.num_heads_kv;
  int t[K], T[K];  // row tiles and key tiles of a request
  long long work = 0;
  int items = 0, longest = 1;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int b = 32 * k + lane;
    t[k] = T[k] = 0;
    if (b < a.batch) {
      const int q0 = __ldg(a.row_start + b), q1 = __ldg(a.row_start + b + 1);
      const int C = a.ctx_len ? __ldg(a.ctx_len + b) : 0;
      if (q0 >= 0 && q1 > q0 && q1 <= a.rows && C >= 0 &&
          (long long)C <= (long long)a.max_pages_per_seq * a.block_size) {
        t[k] = (q1 - q0 + a.tile_q - 1) / a.tile_q;
        T[k] = (C + keys - 1) / keys + (q1 - q0 + keys - 1) / keys;
      }
    }
    work += (long long)t[k] * T[k];
    items += t[k];
    longest = max(longest, T[k]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
  work *= Hk;
  items = __reduce_add_sync(0xffffffffu, items) * Hk;
  longest = __reduce_max_sync(0xffffffffu, longest);
  auto splits_of = [&](int k, int L) { return t[k] ? (T[k] + L - 1) / L : 0; };
  auto fits = [&](int L) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) n += t[k] * splits_of(k, L);
    return __reduce_add_sync(0xffffffffu, n) * Hk <= grid;
  };
  // (sum t ceil(T / L) <= work / L + items, which bounds L from above)
  int lo = max(kSplitLeast, (longest + a.num_splits - 1) / a.num_splits);
  lo = max(lo, (int)((work + grid - 1) / grid));
  int hi = items < grid ? (int)(work / (grid - items)) + 1 : longest;
  hi = max(lo, min(hi, longest));
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (fits(mid)) hi = mid;
    else lo = mid + 1;
  }
  // Worth it? In key tiles: an item costs 3 beside its own (queries, partials), the second launch 6.
  // Whole row tiles end with the longest, or in a second round; pieces end together.
  const int sms = min(grid, a.sms), mean = (int)(work / sms);
  const int whole = items <= sms ? longest : max(longest, mean + longest / 2);
  const int cut = grid <= sms ? lo + 9 : mean + lo / 2 + 3 * (grid / sms) + 6;
  if (cut >= whole) lo = longest;
  SeqTile s{};
  S = 1;
  split = g = 0;
  int base = 0;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int mine = splits_of(k, lo);
    if (counts && 32 * k + lane < a.batch) counts[32 * k + lane] = mine;
    const int x = t[k] * mine * Hk;
    int upto = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const int at = c - (base + upto - x);  // place among the items of this lane's request
    const uint32_t who = __ballot_sync(0xffffffffu, at >= 0 && at < x);
    if (who) {
      const int src = __ffs(who) - 1;
      const int rest = __shfl_sync(0xffffffffu, at, src);
      S = __shfl_sync(0xffffffffu, mine, src);
      s.b = 32 * k + src;
      split = rest % S;
      g = rest / S % Hk;
      s.tile = rest / S / Hk;
      s.q0 = __ldg(a.row_start + s.b);
      s.n = __ldg(a.row_start + s.b + 1) - s.q0;
      s.C = a.ctx_len ? __ldg(a.ctx_len + s.b) : 0;
      s.live = true;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
  }
  return s;
}

// New rows that row i of a request of n rows sees: [0, seq_limit).
__device__ __forceinline__ int seq_limit(int i, int n, int mask_block) {
  return min(n, (i / mask_block + 1) * mask_block);  // (mask_block <= rows, set on the host)
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
