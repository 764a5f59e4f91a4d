// Tensor-core path of d2f_prompt_attn (bf16, head_dim 64 or 128, up to 128 query heads a KV
// head, pages of 8 to 128 tokens).
//
// Source of the mask: "D2F: 확산 언어 모델이 KV 캐시를 얻고 자기회귀 모델보다 2.5배 빨라지는
// 방법", §블록 단위 인과 어텐션 (bidirectional inside a block, causal between blocks).
//
// Per row: x = scale <q, k>, out = sum 2^(x' - m) v / sum 2^(x' - m) with x' = x log2 e, one pass
// over the keys. m is a reference that follows the row's maximum: it moves only when a tile's
// maximum lies more than 2^8 above it, so the accumulator is rarely rescaled. Scores, weights,
// sums and both accumulators are float. The weights enter the product with V as bf16 (2^-8 of
// each, the type of the MMA's operands; the sum keeps the unrounded ones).
//
// Work. An item is a pair of row tiles of 128 rows of one (request, KV head) (neighbours, or from
// both ends of the request: `fold`), times a split of its keys. The G = Hq / Hkv query heads of the
// KV head are packed into the rows (row r = query r / G, head r % G, 128 / G queries a tile), so a
// K/V tile that is read once serves all of them. A CTA keeps an SM (its two row tiles, a ring of K
// and V tiles of 128 keys) and takes further items from the launch's own grid (cluster launch
// control: a CTA that has loaded its item's last tile cancels one that has not started and does its
// work), so that the next item's queries and keys load while the last one computes, and unequal
// items even out. Items of a request's last rows, which see the most keys, come first. Where row
// tiles are few, or long prefixes uneven, the keys are cut into even pieces and a second launch
// composes them (seq_even, prompt_merge_kernel).
//
// What bounds it. A pair of 128 x 128 tiles is 4 * 512 cycles of products for D = 128 (8192 operations
// a cycle) and 2 * 512 of exponentials, half of them a softmax warpgroup's. 16,384 causal rows, 28
// heads on 4: 1224 us at full clocks, 1570 TFLOP/s (81 % of the measured product rate; 1300 to 1320 us
// in a row of calls, where the power cap holds the clock at some 1.6 GHz). Without the weights'
// arithmetic the same loop takes 1141 us: S's operands, both from shared memory, fill its bandwidth.
// 16 requests of 251 to 4096 rows, 32 heads on 8: 775 us; the short rows' tiles that the mask cuts
// cost the difference. D = 64: 1091 us for the long case, 880 TFLOP/s, bound by the exponentials and
// their chain, which are the same for half the products.
//
// Roles of a CTA's warps:
//   0        producer: which request an item belongs to, tensor copies of the queries and of the
//            K and V tiles (of the pages for cached keys, a copy a page and 64 columns; a warp
//            issues one only every 100 cycles or so, so warp 3 takes half of a tile's pages)
//   1        MMA issuer (one lane): S = Q K^T, then O += P V with P in TMEM over S, the row tiles
//            in turn, so that one tile's products run while the other's weights are computed
//   2        V tiles that the mask cuts, or that pages do not fill (below)
//   3        half of a cached tile's pages, half of a new V tile's rows for warp 2
//   4 - 11   softmax: a warpgroup a row tile, a thread a row
// TMEM columns: S / P of tile 0 and 1 (128 each), O of tile 0 and 1 (D each).
//
// What a row does not see. Scores of keys past a row's limit are replaced by -inf, whatever they
// were. V of keys that no row sees (rows of another request, slots past the context) is zeroed in
// shared memory before the product. V of keys that only some rows of the tile see has to be
// finite for the product (0 * infinity is not 0): where the mask cuts through a tile a warp
// looks, and a tile with an infinity or NaN is multiplied by the softmax threads, each with the
// keys that its row sees.
//
// Every wait is bounded; a CTA whose wait ran out records D2F_ERR_TIMEOUT, drains its copies and
// MMAs, frees TMEM and returns.
#include <stdio.h>

#include <mutex>

#include "attn_common.cuh"
#include "seq_attn.cuh"
#include "tensor_map.cuh"

namespace d2f {
namespace {

constexpr int kKeys = 128;  // keys of a tile
constexpr int kThreads = 384;
// Registers: 168 a thread at launch (3 * 128 threads); the producer's and issuers' warpgroup
// gives up what the softmax warpgroups take (a row's 128 scores).
constexpr int kRegLaunch = 168, kRegCtl = 104, kRegSoft = 200;
static_assert(kRegCtl + 2 * kRegSoft <= 3 * kRegLaunch, "register split within the launch's allocation");
constexpr float kMove = 8.f;         // the reference moves when a score is 2^kMove above it
constexpr float kNothing = -3.402823466e38f;  // reference of a row that has seen no key: the lowest float
constexpr float kFar = 268435456.f;  // references of 2^28 and more take the far path (far_scores)

struct Item {
  int b, q0, n, C;      // request, its first row, rows, cached tokens (b < 0: no more items)
  int i0[2];            // first query of each row tile
  int g, split, splits; // KV head, split of the keys
  int t0, t1, Tc;       // key tiles of this item, tiles of the cached keys
  int tw[2];            // end of each row tile's key tiles
};

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * 128 * 128;  // bytes of 128 rows: 64-column halves, 128-byte rows
  static constexpr int kEntries = D == 128 ? 3 : 8;  // ring entries, K and V tiles in turn
  static constexpr int kRing = 4 * kTile;            // (two pairs of Q tiles come first)
  static constexpr int kBars = kRing + kEntries * kTile;
  static constexpr uint32_t kTmO = 256;              // TMEM column of O
};

struct Bars {
  // The u-th tile of the CTA (K and V in turn) lies in entry u % kEntries. Its landing has a barrier by
  // its number, not by its entry: a warp that waits for the V tiles only must neither be two phases
  // late nor find the phase of a K tile in its entry.
  uint64_t full[16];                    // u % 16
  uint64_t empty[8];                    // ring entry
  uint64_t clean[8];                    // V tile (number % 8) looked at, and zeroed where nobody sees it
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2], drain;
  uint64_t slot_full[2], slot_empty[2], clc;
  __align__(16) uint32_t clc_answer[4];
  Item slot[2];
  int bad[8];                           // ring entry: pages of the tile are missing
  int odd[2][8];                        // V tile's halves: an infinity or NaN that not every row sees
  int skip[2];                          // the threads have done this tile's product with V
  int abort;
  uint32_t tmem;
};
template <int D>
constexpr int smem_bytes() {
  return Cfg<D>::kBars + (int)sizeof(Bars) + 1024;  // (1024: the base is aligned by hand)
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory per CTA");

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0,
                                            int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// K or V of one page (the i-th of its tile) and KV head, a copy a 64 columns.
template <int D>
__device__ __forceinline__ void load_page(uint32_t tile, const CUtensorMap *map, uint32_t bar, int i,
                                          const PromptArgs &a, int page, int g) {
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
    tma_load_3d(tile + h * 16384 + i * a.block_size * 128, map, bar, h * 64, 0, page * a.num_heads_kv + g);
}
// Ask for a CTA of this grid that has not started; the answer lands at `answer`.
__device__ __forceinline__ void clc_ask(uint32_t answer, uint32_t bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          answer),
      "r"(bar)
      : "memory");
}
// The index of the CTA whose work came with the answer, or -1.
__device__ __forceinline__ int clc_read(uint32_t answer) {
  uint32_t ok, x = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(answer)
      : "memory");
  return ok ? (int)x : -1;
}
// Whether the phase is over, at once (a try_wait may suspend the thread for a while).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag, int32_t *err,
                                       long long budget) {
  return mbar_wait(bar, parity, abort_flag, err, budget);
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// One lane of a converged warp. (The compiler knows that elect.sync picks a single lane, so it
// does not wrap every tcgen05 instruction in a loop over the active lanes.)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r)
               : "r"(taddr)
               : "memory");
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, "
      "%9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
        "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
        "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_zero(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

// 128 bytes of each of a warp's 32 rows to memory, by way of shared memory so that a store covers
// whole lines (a thread that stores its own row touches a line with every 16 bytes: 32 lines an
// instruction, one a cycle for the SM). `row`: the thread's row in the tile, `hr` its place in
// memory (negative: none), a place every `row_bytes` bytes from `dst` on.
__device__ __forceinline__ void stage_rows(uint32_t stage, int row, const uint32_t (&y)[32], int64_t hr, char *dst,
                                        int row_bytes) {
  const int lane = row & 31;
#pragma unroll
  for (int c = 0; c < 8; ++c)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(stage + row * 128 + ((c ^ (row & 7)) << 4)),
                 "r"(y[4 * c]), "r"(y[4 * c + 1]), "r"(y[4 * c + 2]), "r"(y[4 * c + 3])
                 : "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (lane >> 3), c = lane & 7;  // four rows at a time, eight lanes a row
    const int64_t at = __shfl_sync(0xffffffffu, hr, r);
    const uint4 v = ld_shared_v4(stage + (row - lane + r) * 128 + ((c ^ (r & 7)) << 4));
    if (at >= 0) *reinterpret_cast<uint4 *>(dst + at * row_bytes + c * 16) = v;
  }
  __syncwarp();
}

// A row's output and the weights of its tile's first half times alpha.
template <int D>
__device__ __noinline__ void scale_o(uint32_t o, float alpha) {
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t x[16];
    tmem_ld16(o + c, x);
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * alpha);
    tmem_st16(o + c, x);
  }
}
__device__ __noinline__ void scale_p(uint32_t p, float alpha) {
#pragma unroll 1
  for (int c = 0; c < 32; c += 16) {
    uint32_t x[16];
    tmem_ld16(p + c, x);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      x[j] = pack_bf16x2(__uint_as_float(x[j] << 16) * alpha, __uint_as_float(x[j] & 0xffff0000u) * alpha);
    tmem_st16(p + c, x);
  }
}

// 64 scores of a row whose reference m is far from 0, made relative to it: y / scale with y = x' - m,
// the product x' = x scale rounded first as m was. (One fma a score, as for other references, would
// give the reference's own key the rounding error of m for its exponent, which from 2^31 on is above
// what a weight holds.) Other rows of the warp keep theirs.
__device__ __noinline__ void far_scores(uint32_t s, float scale, float m, bool far) {
#pragma unroll 1
  for (int c = 0; c < 64; c += 16) {
    uint32_t x[16];
    tmem_ld16(s + c, x);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (far) x[j] = __float_as_uint((__fmul_rn(__uint_as_float(x[j]), scale) - m) / scale);
    tmem_st16(s + c, x);
  }
  tmem_wait_st();
}

// The product with V of one tile by the threads: each row adds the keys below its limit.
// `p`: TMEM columns of the row's weights, `o` of its output (taken as 0 when `first`).
template <int D>
__device__ __noinline__ void slow_pv(uint32_t p, uint32_t o, uint32_t v, uint4 sees, bool first) {
  for (int dc = 0; dc < D / 32; ++dc) {
    uint32_t acc[32];
    if (first) {
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[j] = 0;
    } else {
      tmem_ld32(o + dc * 32, acc);
    }
    for (int c = 0; c < kKeys / 2; ++c) {
      const uint32_t w = tmem_ld1(p + c);
      const uint32_t word = c < 16 ? sees.x : c < 32 ? sees.y : c < 48 ? sees.z : sees.w;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = 2 * c + e;
        if (!(word >> (key & 31) & 1u)) continue;
        const float x = e ? __uint_as_float(w & 0xffff0000u) : __uint_as_float(w << 16);
        const uint32_t row = v + (dc >> 1) * (128 * 128) + key * 128;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint4 y = ld_shared_v4(row + ((((dc & 1) * 4 + q) ^ (key & 7)) << 4));
          const uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float &a0 = reinterpret_cast<float &>(acc[q * 8 + 2 * j]);
            float &a1 = reinterpret_cast<float &>(acc[q * 8 + 2 * j + 1]);
            a0 = fmaf(x, __uint_as_float(z[j] << 16), a0);
            a1 = fmaf(x, __uint_as_float(z[j] & 0xffff0000u), a1);
          }
        }
      }
      __syncwarp();
    }
    tmem_st32(o + dc * 32, acc);
  }
  tmem_wait_st();
}

// acc += 0 y, two bf16.
__device__ __forceinline__ void zero_times(uint32_t &acc, uint32_t y) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(y), "r"(0));
}
// Whether cached key `key` lies in a page of the pool.
__device__ __forceinline__ bool page_good(const PromptArgs &a, const Item &x, int key) {
  if (key >= x.C) return false;
  const int page = __ldg(a.page_table + (int64_t)x.b * a.max_pages_per_seq + key / a.block_size);
  return page >= 0 && page < a.num_pages;
}
// Rows r0 .. r1 - 1 of a tile of V in shared memory: rows that no query sees become zeros; whether the
// others hold an infinity or NaN, where the mask cuts through the tile (`cut`).
template <int D>
__device__ __noinline__ bool clean_v(const PromptArgs &a, const Item &x, uint32_t v, int r0, int r1, int base,
                                     int valid, bool cut, bool bad) {
  const int lane = threadIdx.x & 31;
  uint32_t hit[4] = {};  // sums of 0 y: NaN where a y is not finite, else 0
#pragma unroll 1
  for (int row = r0 + lane; row < r1; row += 32) {
    const uint32_t at = v + row * 128;
    if (row >= valid || (bad && !page_good(a, x, base + row))) {
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int c = 0; c < 8; ++c) st_shared_zero(at + h * 16384 + c * 16);
    } else if (cut) {
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 y = ld_shared_v4(at + h * 16384 + (((c + lane) & 7) << 4));
          zero_times(hit[0], y.x);
          zero_times(hit[1], y.y);
          zero_times(hit[2], y.z);
          zero_times(hit[3], y.w);
        }
    }
  }
  fence_proxy_async_smem();  // the zeros, before the MMA reads V
  return __any_sync(0xffffffffu, ((hit[0] | hit[1] | hit[2] | hit[3]) & 0x7fff7fffu) != 0);
}

// (Out of line and at the producer's end: inlined behind the item, it cost the long prompt 2 %.)
__device__ __noinline__ void report_lengths(const PromptArgs &a) { seq_report(a); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_tc_kernel(const PromptArgs a, const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_kp,
                     const __grid_constant__ CUtensorMap tm_vp) {
  using L = Cfg<D>;
  constexpr int NE = L::kEntries;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t sb = (smem_u32(smem_raw) + 1023u) & ~1023u;
  Bars *bars = reinterpret_cast<Bars *>(smem_raw + (sb - smem_u32(smem_raw)) + L::kBars);
  volatile int *abort_flag = &bars->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.group, QI = a.tile_q / 2;  // queries of a row tile

  if (warp == 0 && lane == 0) {
    for (int i = 0; i < NE; ++i) mbar_init(smem_u32(&bars->empty[i]), 1);
    for (int i = 0; i < 16; ++i) mbar_init(smem_u32(&bars->full[i]), 1);
    for (int i = 0; i < 8; ++i) mbar_init(smem_u32(&bars->clean[i]), 2);  // warps 2 and 3
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars->q_full[i]), 1);
      mbar_init(smem_u32(&bars->q_empty[i]), 8);  // the softmax warps
    }
    mbar_init(smem_u32(&bars->drain), 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&bars->s_full[w]), 1);
      mbar_init(smem_u32(&bars->p_full[w]), 4);  // the warps of a softmax warpgroup
      mbar_init(smem_u32(&bars->o_full[w]), 1);
      mbar_init(smem_u32(&bars->o_empty[w]), 4);
      mbar_init(smem_u32(&bars->slot_full[w]), 1);
      mbar_init(smem_u32(&bars->slot_empty[w]), 11);  // every warp but the producer
      bars->skip[w] = 0;
    }
    mbar_init(smem_u32(&bars->clc), 1);
    bars->abort = 0;
    mbar_fence_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  grid_dependency_wait();  // (what is above reads nothing that the kernel before may write)

  if (warp < 4) {
    reg_dec<kRegCtl>();
    if (warp == 0) {
      // ============ producer ====================================================
      uint32_t e = 0, items = 0, asked = 0;
      bool ok = true, had0 = false;
      int it = blockIdx.x;
      const int pages = kKeys / a.block_size;  // pages of a tile (cached keys)
      while (true) {
        Item w;
        w.splits = 1;
        had0 |= it == 0;
        SeqTile s;
        if (a.split_count) {
          s = seq_even(a, it, a.grid, kKeys, w.splits, w.split, w.g, it == 0 ? a.split_count : nullptr);
        } else {
          w.split = 0;
          w.g = it % a.num_heads_kv;
          s = seq_tile(a, a.tiles - 1 - it / a.num_heads_kv);
        }
        w.t0 = w.t1 = 0;
        bool asking = false;
        auto ask = [&] {  // (at most one question at a time, none after a "no")
          asking = true;
          if (lane == 0) {
            fence_proxy_async_smem();  // the last answer has been read
            mbar_arrive_expect_tx(smem_u32(&bars->clc), 16);
            clc_ask(smem_u32(bars->clc_answer), smem_u32(&bars->clc));
          }
        };
        if (s.live) {
          w.b = s.b;
          w.q0 = s.q0;
          w.n = s.n;
          w.C = s.C;
          w.i0[0] = s.tile * (a.fold ? QI : a.tile_q);
          w.i0[1] = w.i0[0] + QI;
          if (a.fold) {
            const int other = (s.n + QI - 1) / QI - 1 - s.tile;
            w.i0[1] = other > s.tile ? other * QI : s.n;  // (s.n: the middle one is alone)
          }
          w.Tc = (s.C + kKeys - 1) / kKeys;
          int T = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int first = w.i0[i], end = min(first + QI, s.n);
            w.tw[i] = first >= s.n ? 0 : w.Tc + (seq_limit(end - 1, s.n, a.mask_block) + kKeys - 1) / kKeys;
            T = max(T, w.tw[i]);
          }
          int s_eff;
          if (!split_range(T, w.splits, w.split, w.t0, w.t1, s_eff)) w.t0 = w.t1 = 0;
          const int sl = items & 1;
          ok = mbar_wait(smem_u32(&bars->slot_empty[sl]), ((items >> 1) & 1) ^ 1, abort_flag, a.err,
                         a.wait_cycles);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            bars->slot[sl] = w;
            mbar_arrive(smem_u32(&bars->slot_full[sl]));
          }
          ok = mbar_wait(smem_u32(&bars->q_empty[sl]), ((items >> 1) & 1) ^ 1, abort_flag, a.err, a.wait_cycles);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++items;
          if (lane == 0) {
            const uint32_t bar = smem_u32(&bars->q_full[sl]);
            mbar_arrive_expect_tx(bar, 2 * L::kHalves * QI * G * 128);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int h = 0; h < L::kHalves; ++h)
                tma_load_3d(sb + (2 * sl + i) * L::kTile + h * 16384, &tm_q, bar, h * 64, w.g * G,
                            w.q0 + w.i0[i]);
          }
          // page ids of the next cached tile, one a lane
          const int32_t *table = a.page_table + (int64_t)w.b * a.max_pages_per_seq;
          auto page_of = [&](int t) {
            const int at = t * pages + lane;
            return lane < pages && t < w.Tc && at * a.block_size < w.C ? __ldg(table + at) : 0;
          };
          int page = w.t0 < w.Tc ? page_of(w.t0) : 0;
          for (int t = w.t0; t < w.t1 && ok; ++t) {
            if (t == max(w.t0, w.t1 - 4)) ask();
            const bool cached = t < w.Tc;
            const bool need = cached && lane < pages && (t * pages + lane) * a.block_size < w.C;
            const bool good = need && page >= 0 && page < a.num_pages;
            const int next = t + 1 < w.Tc ? page_of(t + 1) : 0;
            const uint32_t n_good = __popc(__ballot_sync(0xffffffffu, good));
            const bool bad = __any_sync(0xffffffffu, need && !good);
            if (bad && lane == 0) set_err(a.err, D2F_ERR_BAD_INDEX);
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              const int ent = e % NE;
              ok = mbar_wait(smem_u32(&bars->empty[ent]), ((e / NE) & 1) ^ 1, abort_flag, a.err,
                             a.wait_cycles);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              const uint32_t bar = smem_u32(&bars->full[e & 15]), dst = sb + L::kRing + ent * L::kTile;
              if (cached) {
                if (lane == 0) {
                  bars->bad[ent] = bad;
                  mbar_arrive_expect_tx(bar, n_good * a.block_size * 128 * L::kHalves);
                }
                __syncwarp();
                if (good && lane < (pages + 1) / 2) load_page<D>(dst, kv ? &tm_vp : &tm_kp, bar, lane, a, page, w.g);
              } else if (elect_one()) {
                mbar_arrive_expect_tx(bar, L::kTile);
#pragma unroll
                for (int h = 0; h < L::kHalves; ++h)
                  tma_load_3d(dst + h * 16384, kv ? &tm_v : &tm_k, bar, h * 64, w.g,
                              w.q0 + (t - w.Tc) * kKeys);
              }
              __syncwarp();
              ++e;
            }
            page = next;
          }
          if (!ok) {
            asked += asking;
            break;
          }
        }
        if (!asking) ask();
        ok = mbar_wait(smem_u32(&bars->clc), asked & 1, abort_flag, a.err, a.wait_cycles);
        ok = __all_sync(0xffffffffu, ok);
        ++asked;
        if (!ok) break;
        it = clc_read(smem_u32(bars->clc_answer));
        __syncwarp();
        if (it < 0) break;
      }
      if (ok) {  // no more items
        const int sl = items & 1;
        ok = mbar_wait(smem_u32(&bars->slot_empty[sl]), ((items >> 1) & 1) ^ 1, abort_flag, a.err,
                       a.wait_cycles);
        if (ok && lane == 0) {
          bars->slot[sl].b = -1;
          mbar_arrive(smem_u32(&bars->slot_full[sl]));
        }
      }
      if (had0) report_lengths(a);  // (whichever CTA took item 0: its own may never start)
      // Drain: what was asked for has landed before the CTA ends.
      if (lane == 0) {
        volatile int no_abort = 0;
        for (uint32_t u = items > 2 ? items - 2 : 0; u < items; ++u)
          mbar_wait(smem_u32(&bars->q_full[u & 1]), (u >> 1) & 1, &no_abort, a.err, kDrainCycles);
        for (uint32_t u = e > (uint32_t)NE ? e - NE : 0; u < e; ++u)
          mbar_wait(smem_u32(&bars->full[u & 15]), (u >> 4) & 1, &no_abort, a.err, kDrainCycles);
        if (asked) mbar_wait(smem_u32(&bars->clc), (asked - 1) & 1, &no_abort, a.err, kDrainCycles);
      }
    } else if (warp == 1 && elect_one()) {
      // ============ MMA issuer =================================================
      // One thread for both row tiles: P V of a tile's last keys and S of its next ones, then the
      // same of the other row tile, so that one tile's softmax has the time of the other's products.
      // (Two issuers, a row tile each, fell into step: both tiles in the softmax at a time.)
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kKeys, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t q_desc = smem_desc_sw128(sb, 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(sb + L::kRing, 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(sb + L::kRing, 16384, 1024);
      // (Elected, not lane 0: 16,384 causal rows of 28 on 4 heads 1777 -> 1343 us.)
      const uint32_t full = smem_u32(bars->full), empty = smem_u32(bars->empty), clean = smem_u32(bars->clean);
      uint32_t sk = 0;                // ring entry of the next K
      uint32_t vt = 0;                // tiles whose S has been issued; the one before it is vt - 1
      uint32_t p_par = 0, o_par = 3;  // parities, a bit a row tile: p_full, o_empty
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort_flag, a.err, a.wait_cycles);
      };
      // The item in work and its next tile; the tile before it, whose products with V are still to come
      // (they stay so over the change of items where the next one's operands have landed).
      uint32_t item = 0;
      int t = 0, t0 = 0, t1 = 0, tw0 = 0, tw1 = 0;
      uint32_t sv = 0, todo = 0, last = 0, more = 0, qs = 0;  // todo, last: a bit a row tile
      bool behind = false;
      while (true) {
        bool score = t < t1;
        if (!score) {
          const uint32_t sl = item & 1, par = (item >> 1) & 1;
          bool ready = mbar_test(smem_u32(&bars->slot_full[sl]), par);
          if (!ready && !behind) {
            if (!wait(smem_u32(&bars->slot_full[sl]), par)) break;
            ready = true;
          }
          if (ready) {
            const bool end = bars->slot[sl].b < 0;
            if (end && !behind) break;
            if (!end && (!behind || (mbar_test(smem_u32(&bars->q_full[sl]), par) && mbar_test(full + 16 * (vt & 7), (vt >> 3) & 1)))) {
              t0 = t = bars->slot[sl].t0;
              t1 = bars->slot[sl].t1;
              tw0 = min(t1, bars->slot[sl].tw[0]);
              tw1 = min(t1, bars->slot[sl].tw[1]);
              mbar_arrive(smem_u32(&bars->slot_empty[sl]));
              ++item;
              if (!wait(smem_u32(&bars->q_full[sl]), par)) break;
              qs = 2 * sl;
              score = t < t1;
              if (!score) continue;  // (a split without keys)
            }
          }
        }
        bool ok = true;
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          const uint32_t ts = tmem + w * 128, to = tmem + L::kTmO + w * D;
          if (todo >> w & 1u) {
            ok = wait(clean + 8 * ((vt - 1) & 7), ((vt - 1) >> 3) & 1);
            if (ok && !more) {
              ok = wait(smem_u32(&bars->o_empty[w]), (o_par >> w) & 1);
              o_par ^= 1u << w;
            }
            ok = ok && wait(smem_u32(&bars->p_full[w]), (p_par >> w) & 1);
            if (!ok) break;
            p_par ^= 1u << w;
            tc_fence_after();
            if (!*(volatile int *)&bars->skip[w]) {
              const uint64_t vd = smem_desc_advance(v_desc, sv * L::kTile);
#pragma unroll
              for (int ks = 0; ks < kKeys / 16; ++ks)
                umma_bf16_tmem_a(to, ts + ks * 8, smem_desc_advance(vd, ks * 2048), idesc_pv, ks > 0 ? 1u : more);
            }
            if (last >> w & 1u) umma_commit(smem_u32(&bars->o_full[w]));
          }
          if (w && behind) umma_commit(empty + 8 * sv);
          if (score && t < (w ? tw1 : tw0)) {
            ok = wait(full + 16 * (vt & 7), (vt >> 3) & 1);
            if (!ok) break;
            tc_fence_after();
            const uint64_t qd = smem_desc_advance(q_desc, (qs + w) * L::kTile);
            const uint64_t kd = smem_desc_advance(k_desc, sk * L::kTile);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t at = (k >> 2) * 16384 + (k & 3) * 32;
              umma_bf16(ts, smem_desc_advance(qd, at), smem_desc_advance(kd, at), idesc_qk, k ? 1u : 0u);
            }
            umma_commit(smem_u32(&bars->s_full[w]));
          }
        }
        if (!ok) break;
        behind = score;
        todo = 0;
        if (score) {
          umma_commit(empty + 8 * sk);
          todo = (t < tw0 ? 1u : 0u) | (t < tw1 ? 2u : 0u);
          last = (t == tw0 - 1 ? 1u : 0u) | (t == tw1 - 1 ? 2u : 0u);
          more = t > t0 ? 1u : 0u;
          sv = sk + 1 == NE ? 0 : sk + 1;
          ++vt;
          sk += 2;
          if (sk >= NE) sk -= NE;
          ++t;
        }
      }
      umma_commit(smem_u32(&bars->drain));
      volatile int no_abort = 0;
      mbar_wait(smem_u32(&bars->drain), 0, &no_abort, a.err, kDrainCycles);
    } else if (warp == 2) {
      // ============ V of tiles that the mask cuts =================================
      uint32_t e = 0;
      auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        const uint32_t at = smem_u32(bar);
        const bool x = mbar_try_wait(at, parity) || wait_long(at, parity, abort_flag, a.err, a.wait_cycles);
        return __all_sync(0xffffffffu, x);
      };
      bool ok = true;
      for (uint32_t item = 0; ok; ++item) {
        const int sl = item & 1;
        if (!wait(&bars->slot_full[sl], (item >> 1) & 1)) break;
        const Item x = bars->slot[sl];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->slot_empty[sl]));
        if (x.b < 0) break;
        const int first[2] = {seq_limit(min(x.i0[0], x.n - 1), x.n, a.mask_block),  // (the first rows')
                              seq_limit(min(x.i0[1], x.n - 1), x.n, a.mask_block)};
#pragma unroll 1
        for (int t = x.t0; t < x.t1; ++t, e += 2) {  // K and V tiles in turn
          const uint32_t ent = (e + 1) % NE, vt = e >> 1;
          ok = wait(&bars->full[(e + 1) & 15], (e >> 4) & 1);
          if (!ok) break;
          const bool cached = t < x.Tc;
          const int base = (cached ? t : t - x.Tc) * kKeys, valid = (cached ? x.C : x.n) - base;
          const bool cut = !cached && ((t < x.tw[0] && first[0] - base < min(kKeys, valid)) ||
                                       (t < x.tw[1] && first[1] - base < min(kKeys, valid)));
          const bool bad = cached && *(volatile int *)&bars->bad[ent] != 0;
          bool odd = false;
          if (bad || cut || valid < kKeys)  // (of a cached tile all rows: warp 3 has copies to issue)
            odd = clean_v<D>(a, x, sb + L::kRing + ent * L::kTile, 0, cached ? kKeys : kKeys / 2, base, valid, cut, bad);
          __syncwarp();
          if (lane == 0) {
            *(volatile int *)&bars->odd[0][vt & 7] = odd;
            mbar_arrive(smem_u32(&bars->clean[vt & 7]));
          }
        }
      }
    } else if (warp == 3) {
      // ============ second producer of cached tiles: half of their pages; half of the new V =======
      const int pages = kKeys / a.block_size, mine = (pages + 1) / 2;
      uint32_t e = 0, issued = 0;
      bool ok = true;
      for (uint32_t item = 0; ok; ++item) {
        const int sl = item & 1;
        ok = mbar_wait(smem_u32(&bars->slot_full[sl]), (item >> 1) & 1, abort_flag, a.err, a.wait_cycles);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const Item x = bars->slot[sl];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->slot_empty[sl]));
        if (x.b < 0) break;
        const int32_t *table = a.page_table + (int64_t)x.b * a.max_pages_per_seq;
        auto page_of = [&](int t) {
          const int at = t * pages + lane;
          return lane >= mine && lane < pages && t < x.Tc && at * a.block_size < x.C ? __ldg(table + at) : -1;
        };
        const int end = min(x.t1, x.Tc);
        int page = x.t0 < end ? page_of(x.t0) : -1;
        auto done = [&](uint32_t vt, bool odd) {
          __syncwarp();
          if (lane == 0) {
            *(volatile int *)&bars->odd[1][vt & 7] = odd;
            mbar_arrive(smem_u32(&bars->clean[vt & 7]));
          }
        };
        auto landed = [&](uint32_t u) -> bool {
          const bool y = mbar_wait(smem_u32(&bars->full[u & 15]), (u >> 4) & 1, abort_flag, a.err, a.wait_cycles);
          return __all_sync(0xffffffffu, y);
        };
        for (int t = x.t0; t < end && ok; ++t) {
          const int next = t + 1 < end ? page_of(t + 1) : -1;
          const bool good = page >= 0 && page < a.num_pages;
          const uint32_t u0 = e + 2 * (t - x.t0);
          // (A wait may be for a phase that cannot be followed by another before this warp has done its
          // part: entries that it copies to, else the V tile, which is not used before `done`.)
          if (__any_sync(0xffffffffu, good)) {
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              const uint32_t u = u0 + kv, ent = u % NE;
              ok = mbar_wait(smem_u32(&bars->empty[ent]), ((u / NE) & 1) ^ 1, abort_flag, a.err, a.wait_cycles);
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              if (good)
                load_page<D>(sb + L::kRing + ent * L::kTile, kv ? &tm_vp : &tm_kp, smem_u32(&bars->full[u & 15]), lane, a,
                             page, x.g);
              issued = u + 1;
            }
          } else {
            ok = landed(u0 + 1);
          }
          page = next;
          if (ok) done(u0 >> 1, false);
        }
        const int first[2] = {seq_limit(min(x.i0[0], x.n - 1), x.n, a.mask_block),
                              seq_limit(min(x.i0[1], x.n - 1), x.n, a.mask_block)};
#pragma unroll 1
        for (int t = max(end, x.t0); t < x.t1 && ok; ++t) {
          const uint32_t u = e + 2 * (t - x.t0) + 1;
          ok = landed(u);
          if (!ok) break;
          const int base = (t - x.Tc) * kKeys, valid = x.n - base;
          const bool cut = (t < x.tw[0] && first[0] - base < min(kKeys, valid)) ||
                           (t < x.tw[1] && first[1] - base < min(kKeys, valid));
          bool odd = false;
          if (cut || valid < kKeys)
            odd = clean_v<D>(a, x, sb + L::kRing + u % NE * L::kTile, kKeys / 2, kKeys, base, valid, cut, false);
          done(u >> 1, odd);
        }
        e += 2 * (x.t1 - x.t0);
      }
      if (!ok && lane == 0) {  // what was asked for has landed before the CTA ends
        volatile int no_abort = 0;
        for (uint32_t u = issued > (uint32_t)NE ? issued - NE : 0; u < issued; ++u)
          mbar_wait(smem_u32(&bars->full[u & 15]), (u >> 4) & 1, &no_abort, a.err, kDrainCycles);
      }
    }
  } else {
    // ============ softmax: warpgroup w, a thread a row ==========================
    reg_inc<kRegSoft>();
    const int w = (warp >> 2) - 1;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
    const uint32_t ts = tmem + lane_base + w * 128, to = tmem + lane_base + L::kTmO + w * D;
    const int qi = row / G, qh = row % G;
    const int64_t n_hr = (int64_t)a.rows * a.num_heads_q;
    const float sl2 = a.scale_log2;
    uint32_t e = 0, tiles = 0, outs = 0;
    int was_odd = 0;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
      const bool x = mbar_wait(smem_u32(bar), parity, abort_flag, a.err, a.wait_cycles);
      return __all_sync(0xffffffffu, x);
    };
    for (uint32_t item = 0;; ++item) {
      const int sl = item & 1;
      if (!wait(&bars->slot_full[sl], (item >> 1) & 1)) break;
      const Item x = bars->slot[sl];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->slot_empty[sl]));
      if (x.b < 0) break;
      const int i = x.i0[w] + qi;                      // query of the row
      const bool rv = qi < QI && i < x.n;
      const int limit = rv ? seq_limit(i, x.n, a.mask_block) : 0;  // new rows it sees
      const int tw = min(x.t1, x.tw[w]);
      // new rows that every row of the tile sees: the first row's
      const int first_limit = seq_limit(min(x.i0[w], x.n - 1), x.n, a.mask_block);
      // The reference, and what a score has to be above to move it; with a reference from kFar on the
      // limit is -infinity, every 64 keys with a score take the rare path, and m_ref is 0.
      float m_ref = kNothing, m_far = kNothing, limit_up = rv ? kNothing : INFINITY, l = 0.f;
      bool ok = true;
      for (int t = x.t0; t < tw; ++t) {
        const uint32_t ev = e + 2 * (t - x.t0) + 1;
        const bool cached = t < x.Tc;
        const int base = (cached ? t : t - x.Tc) * kKeys;
        bool look = base + kKeys > (cached ? x.C : first_limit);  // some row does not see some key
        uint4 sees;
        bool odd = false;
        if (__builtin_expect(look || cached, 0)) {
          // (With S of an item's first tile there the issuer is past the V tile that had this barrier
          // before, even where the other row tile of the item before had more tiles than this one.)
          if (t == x.t0) ok = wait(&bars->s_full[w], tiles & 1);
          ok = ok && wait(&bars->clean[(ev >> 1) & 7], (ev >> 4) & 1);
          if (!ok) break;
          const volatile Bars *vb = bars;
          const bool bad = cached && vb->bad[ev % NE];
          look = look || bad;
          if (look) {
            odd = (vb->odd[0][(ev >> 1) & 7] | vb->odd[1][(ev >> 1) & 7]) != 0;
            const int lim = cached ? x.C - base : limit - base;
            uint32_t word[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int y = lim - 32 * k;
              word[k] = y >= 32 ? ~0u : y <= 0 ? 0u : (1u << y) - 1u;
            }
            if (bad)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                word[k] &= __ballot_sync(0xffffffffu, page_good(a, x, base + 32 * k + lane));
            sees = make_uint4(word[0], word[1], word[2], word[3]);
          }
        }
        ok = wait(&bars->s_full[w], tiles & 1);
        if (!ok) break;
        tc_fence_after();
        const bool first = t == x.t0;
        // 64 keys at a time
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          float sum[4], mx[4];
          uint32_t p[32];
          // Weights with the reference as it is, the largest score beside them; where that is too far
          // above the reference (seldom, and not a second time), the reference moves and the weights
          // are computed again.
          bool again = false;
          while (true) {
            uint32_t r[64];
            tmem_ld64(ts + c * 64, r);
            if (__builtin_expect(look, 0)) {
              const uint32_t w0 = c ? sees.z : sees.x, w1 = c ? sees.w : sees.y;
#pragma unroll
              for (int j = 0; j < 64; ++j)
                if (!((j < 32 ? w0 : w1) >> (j & 31) & 1u)) r[j] = 0xff800000u;
            }
            // Pairs of keys in three steps, apart so that the exponentials, which bound this loop (four
            // cycles each a warp), do not wait: argument; exponentials; sum and rounding.
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              sum[k] = 0.f;
              mx[k] = -INFINITY;
            }
            if (__builtin_expect(first && c == 0 && m_ref == kNothing, 0)) {  // an item's first scores
#pragma unroll
              for (int j = 0; j < 32; ++j)
                mx[j & 3] = fmax3(mx[j & 3], __uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
              const float m = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2, kNothing);
              const bool far = fabsf(m) >= kFar && m != kNothing;
              if (!far) m_ref = m;
              if (rv) limit_up = far ? -INFINITY : m + kMove;
            }
            // (One fma a score: the reference's own key has the rounding error of m_ref for its exponent,
            // up to 2^4 with references below kFar.)
            const float neg = -m_ref;
            constexpr int kA = 2, kB = 6;
#pragma unroll
            for (int j = 0; j < 32 + kA + kB; ++j) {
              if (j < 32) {
                const float x0 = __uint_as_float(r[2 * j]), x1 = __uint_as_float(r[2 * j + 1]);
                float y0, y1;
                mx[j & 3] = fmax3(mx[j & 3], x0, x1);
                fma2_bc(y0, y1, x0, x1, sl2, neg);
                r[2 * j] = __float_as_uint(y0);
                r[2 * j + 1] = __float_as_uint(y1);
              }
              if (j >= kA && j < 32 + kA) {
                const int k = 2 * (j - kA);
                r[k] = __float_as_uint(fast_exp2(__uint_as_float(r[k])));
                r[k + 1] = __float_as_uint(fast_exp2(__uint_as_float(r[k + 1])));
              }
              if (j >= kA + kB) {
                const int k = j - kA - kB;
                const float x0 = __uint_as_float(r[2 * k]), x1 = __uint_as_float(r[2 * k + 1]);
                add2(sum[2 * (k & 1)], sum[2 * (k & 1) + 1], sum[2 * (k & 1)], sum[2 * (k & 1) + 1], x0, x1);
                p[k] = pack_bf16x2(x0, x1);
              }
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
            const bool move = top > limit_up;
            if (__builtin_expect(!__any_sync(0xffffffffu, move) || again, 1)) break;
            // By a whole number of powers of two, so that weights of this tile's first half which are
            // stored already keep their bits; the first time, and by more than 126, to the score itself.
            float alpha = 1.f;
            bool far = limit_up == -INFINITY;
            if (move) {
              far |= fabsf(top) >= kFar;
              if (far) {
                const float old = limit_up == -INFINITY ? m_far : m_ref;
                m_far = fmaxf(old, top);
                alpha = fast_exp2(old - m_far);
                m_ref = 0.f;
                limit_up = -INFINITY;
              } else {
                const float up = ceilf(top - m_ref);
                const bool small = up <= 126.f;
                alpha = small ? __uint_as_float((uint32_t)(127 - (int)up) << 23) : 0.f;
                m_ref = small ? m_ref + up : top;
                limit_up = m_ref + kMove;
              }
            }
            l *= alpha;
            // (What the tile's first half stored is loaded here: a load does not wait for a store.)
            tmem_wait_st();
            if (c == 1) scale_p(ts, alpha);
            // (P V of the tile before is complete: S of this one came after it)
            if (!first) scale_o<D>(to, alpha);
            again = __any_sync(0xffffffffu, far);
            if (again) far_scores(ts + c * 64, sl2, m_far, far);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st32(ts + c * 32, p);
        }
        tmem_wait_st();
        if (__builtin_expect(odd || was_odd, 0)) {
          if (odd) slow_pv<D>(ts, to, sb + L::kRing + (ev % NE) * L::kTile, sees, first);
          if (warp % 4 == 0 && lane == 0) *(volatile int *)&bars->skip[w] = odd;
          was_odd = odd;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->p_full[w]));
        ++tiles;
      }
      if (!ok) break;
      e += 2 * (x.t1 - x.t0);
      const int64_t hr = rv ? (int64_t)(x.q0 + i) * a.num_heads_q + x.g * G + qh : -1;
      const uint32_t stage = sb + (2 * sl + w) * L::kTile;  // the queries' place: S is done with them
      if (tw > x.t0) {
        if (!wait(&bars->o_full[w], outs & 1)) break;
        ++outs;
        tc_fence_after();
        const float inv = 1.0f / l;
        const bool none = l == 0.f;  // every score is -inf (the product may be 0 * infinity)
        const bool parts = x.splits > 1;
        char *dst = parts ? reinterpret_cast<char *>(a.ws_o + x.split * n_hr * D) : static_cast<char *>(a.out);
        // 128 bytes of every row at a time: bf16 outputs of 64 columns, or float parts of 32
        const int chunks = parts ? D / 32 : D / 64, row_bytes = chunks * 128;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          uint32_t y[32];
          if (parts) {
            tmem_ld32(to + c * 32, y);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t o[32];
              tmem_ld32(to + c * 64 + h * 32, o);
#pragma unroll
              for (int j = 0; j < 16; ++j)
                y[h * 16 + j] = none ? 0u : pack_bf16x2(__uint_as_float(o[2 * j]) * inv,
                                                        __uint_as_float(o[2 * j + 1]) * inv);
            }
          }
          stage_rows(stage, row, y, hr, dst + c * 128, row_bytes);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->o_empty[w]));
        fence_proxy_async_smem();  // (the next queries come by a tensor copy)
      } else if (!wait(&bars->q_full[sl], (item >> 1) & 1)) {
        break;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->q_empty[sl]));
      if (limit_up == -INFINITY) m_ref = m_far;
      if (rv && x.splits > 1)
        a.ws_ml[x.split * n_hr + hr] = make_float2(m_ref == kNothing ? -INFINITY : m_ref, l);
      else if (rv && a.lse_out)
        a.lse_out[hr] = (m_ref + __log2f(l)) * 0.6931471805599453f;
    }
  }

  // ---- teardown ---------------------------------------------------------------
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_d(const PromptArgs &a, cudaStream_t s, char *why, size_t why_len) {
  constexpr int bytes = smem_bytes<D>();
  cudaFuncAttributes fa;
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncGetAttributes(&fa, prompt_tc_kernel<D>);
      if (e != cudaSuccess) return e;
      if (fa.numRegs != kRegLaunch) {  // the register split counts on it
        snprintf(why, why_len, "%d registers a thread, the kernel expects %d", fa.numRegs, kRegLaunch);
        return cudaErrorInvalidConfiguration;
      }
      e = cudaFuncSetAttribute(prompt_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  // Rows of 64 columns (128 bytes, swizzled), `box` of them a copy.
  const cuuint64_t rowb = (cuuint64_t)D * 2;
  auto map = [&](CUtensorMap *m, const void *base, cuuint64_t d1, cuuint64_t d2, cuuint64_t s1, cuuint64_t s2,
                 cuuint32_t b1, cuuint32_t b2) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, d1, d2}, strides[2] = {s1, s2};
    const cuuint32_t box[3] = {64, b1, b2};
    return encode_bf16_sw128(m, base, 3, dims, strides, box);
  };
  const int Hq = a.num_heads_q, Hk = a.num_heads_kv, B = a.block_size;
  CUtensorMap q, k, v, kp, vp;
  bool ok = map(&q, a.q, Hq, a.rows, rowb, Hq * rowb, a.group, a.tile_q / 2) &&
            map(&k, a.k, Hk, a.rows, rowb, Hk * rowb, 1, kKeys) &&
            map(&v, a.v, Hk, a.rows, rowb, Hk * rowb, 1, kKeys);
  if (a.ctx_len && a.num_pages > 0) {
    const cuuint64_t tiles = (cuuint64_t)a.num_pages * Hk;
    ok = ok && map(&kp, a.k_pool, B, tiles, rowb, B * rowb, B, 1) &&
         map(&vp, a.v_pool, B, tiles, rowb, B * rowb, B, 1);
  } else {  // (no cached key is read)
    kp = k;
    vp = v;
  }
  if (!ok) {
    snprintf(why, why_len, "cuTensorMapEncodeTiled is missing or rejected a tensor (alignment or size)");
    return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, prompt_tc_kernel<D>, a, q, k, v, kp, vp);
}

}  // namespace

cudaError_t launch_prompt_tc(const PromptArgs &a, cudaStream_t s, char *why, size_t why_len) {
  return a.head_dim == 128 ? launch_d<128>(a, s, why, why_len) : launch_d<64>(a, s, why, why_len);
}

}  // namespace d2f
