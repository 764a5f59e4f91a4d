// Tensor-core path of d2f_block_attn_kv4 (bf16 queries and window, 4-bit cached
// tokens; layout and conversions of the cache: kv4.cuh).
//
// Source of the computation: "D2F: 확산 언어 모델이 KV 캐시를 얻고 자기회귀
// 모델보다 2.5배 빨라지는 방법", §블록 단위 인과 어텐션 (bidirectional inside a
// block, causal between blocks, finished blocks in a KV cache) and §운영 관점
// (paged cache, one block per page); "확산 언어 모델(Diffusion LLM)이란 무엇인가",
// §FlashBlock (attention parts recombined in log space).
//
// Orientation. A window has few query rows and a cache many keys, so the products
// put keys and head dims on the 128 rows of the MMA and the queries on its columns:
//   S^T [128 keys x rows] = K [128 keys x D] Q^T,
//   O^T [D x rows]       += V^T [D x 128 keys] P^T.
// K and V^T are then the A operands, which tcgen05 reads from tensor memory: a
// thread dequantises the codes of one key (or one dim) in registers and stores them
// to its own TMEM lane. Dequantised tiles never pass through shared memory, whose
// bandwidth would bound the kernel (4x the bytes that the cache read brings), and
// the MMA's time follows the real number of rows in steps of 16.
//
// Types. Stored values are exact in fp16, so cached tiles multiply in fp16: Q is
// scaled per row by a power of two so that its largest element is in [2^14, 2^15)
// (8 significant bits stay exact down to 2^-28 of it), P is rounded to fp16 (2^-11).
// Window tiles keep bf16 K, V and Q; fp16 could not hold every V. P is then a pair of
// bf16, its value rounded and what that left (2^-16 together), each multiplied with V^T:
// one bf16 (2^-8) would be the largest error of a short context's output beside the
// output's own rounding. Sums, references and both accumulators are float.
//
// Work. A row tile holds up to NT = 64 of the group * n query rows of a (sequence, KV
// head): row r = query r / group, head r % group. Its key tiles (128 cached tokens each,
// then 128 window rows each) are units of work; what a row tile costs beside them counts
// as kSegmentTiles units more. All units of the launch are one line, cut into equal
// shares, one CTA a share: every SM gets the same work whatever the batch looks like. A row tile whose units lie in several shares is put together by the CTA that
// arrives last at its counter, from float partials in the workspace, in the order of the
// line (the result does not depend on who is last). No CTA waits on another. The counter is
// that of the share which holds the row tile's first key tile: a share has one end, so it
// cuts off one row tile at most, and the counters are as many as CTAs whatever the batch is.
//
// Roles of a CTA's warps:
//   0        producer: page ids -> one bulk copy per page (K and V of a head are one
//            contiguous piece) into a ring of five tiles
//   1        MMA issuer (one elected lane); 2 and 3 are spare
//   4 - 15   a warpgroup dequantises K (thread = key), two V^T (thread = dim, 64 keys each)
//   16 - 31  four softmax warpgroups of 16 columns each, thread = key. A column's
//            reference moves only when its scores leave a wide range round it: a tile
//            takes no maximum over the lanes, only a vote on whether some column
//            has to move. With 16 columns a thread stays within 72 registers, which lets
//            16 warps run side by side (32 columns a thread: 8 warps, and spills).
//
// Measured (B = 16, D = 128, in a CUDA graph, L2 flushed; in brackets the bf16 cache's
// kernel on the same lengths, which reads 3.6 times the bytes). 32 heads: 4 sequences of
// 32,768 cached tokens and 64 window rows 243 us (336), 2.5 TB/s of 4-bit cache; 16
// sequences of 251 to 4096 tokens 101 us (126); one sequence of 1024, 4096 and 8192
// tokens and 48 rows 17.6, 23 and 30 us (12, 19 and 31). 28 query heads on 4 KV heads, 8
// sequences of 8192 tokens and 48 rows 105 us (65): each of its six row tiles
// dequantises the cache again. A CTA takes some 14 us once, 1.0 us (about 1900 cycles) a
// key tile, and 7 us for each row tile that it begins beside the first. Of the 14 us, 4
// are the start (sequence metadata, work line, first page ids), 1 the queries, 2 the first
// tile, 2 the window tile, 2 the part and its arrival, 3 the composition: straight code
// that runs once, much of it instruction fetches. A tile is bound by the hand-overs between
// its roles, each of which takes 300 to 1000 cycles: when the longest contexts took 259 us,
// they still needed 225 with all conversions and exponentials taken out (without K's
// conversion 244, V's 248, the exponentials 253). The tensor pipe is active 24 % of the
// cycles, the ALU, which converts the codes, 54 %, the issue slots 71 %, DRAM 32 %. What
// shortened the chain: one issuer whose order stands for two waits (272 -> 259), V^T on
// two warpgroups (285 -> 272), polling warps on different schedulers (259 -> 249), small
// code (the hot loops of all roles share the instruction cache: V^T's loop unrolled by two
// costs 10 %, the window's second products in a loop of their own 2 %). What did not: a
// deeper ring, a third K buffer, a K chunk in a V^T warpgroup, polls that sleep, polls by
// every warp.
#include <atomic>

#include "kv4.cuh"

namespace d2f {
namespace {

constexpr int kKeys = 128;                 // keys per tile (UMMA M of S^T, K extent of O^T)
// References. P is fp16, whose numbers end at 2^16 and whose steps are 2^-24 below 2^-14,
// so a column's largest weight should lie near the top of that range: a weight errs by
// 2^-11 of itself and by 2^-25 at most (one below that is lost to the output, while the
// float sum holds it). The largest weight is at least 2^kLow = 2^6, so the second part is
// 2^-31 of it: N cached tokens lose N 2^-31 of the sum at most, 2^-11 at a million. A
// reference moves when a score rises 2^15 above it, and then to 2^kLift = 2^10 below that
// score. A column starts with the reference 2^-kStart (scores in log2 units, plus 7) and
// keeps it if its first tile has a score in [2^-1, 2^8], which saves most row tiles the
// search for a maximum over the lanes (columns without a query have scores of 1).
constexpr float kHigh = 15.0f, kLow = 6.0f, kLift = 10.0f, kStart = 7.0f;
constexpr int kMaxBatch = kKv4MaxBatch;
// What a row tile costs beside its key tiles (its queries, the pipeline's start, its
// output: about 7 us, against 1.0 us a key tile), in key tiles.
constexpr int kSegmentTiles = 6;

constexpr int NT = 64;                     // rows (columns of S^T and O^T) per row tile

template <int D>
struct Cfg {
  static constexpr int kDq = 3;                       // dequantising warpgroups: K, two of V^T
  static constexpr int kSw = NT / 16;                 // softmax warpgroups, 16 columns each
  static constexpr int kThreads = 128 * (1 + kDq + kSw);
  // named barriers: 1 .. kSw a softmax warpgroup each, then all of them, then K, V^T
  static constexpr int kBarSoft = 1, kBarAll = kBarSoft + kSw, kBarK = kBarAll + 1;
  static constexpr int kRegLaunch = 64;               // registers per thread at launch
  // (68 bytes of spill stores and 92 of loads; 80 for the softmax warps and 48 for the
  // others: no spills, but 2 to 8 % slower)
  static constexpr int kRegCtl = 40, kRegDq = 56, kRegSoft = 72;
  static_assert(kRegCtl + kDq * kRegDq + kSw * kRegSoft <= (1 + kDq + kSw) * kRegLaunch,
                "register split within the launch's allocation");
  static constexpr int kBuf = 2;                      // K and V^T operand buffers in TMEM
  static constexpr int kStages = 5;
  // TMEM columns: two S buffers, O, then the K and V^T operands (two halves a column)
  static constexpr uint32_t kTmS = 0, kTmO = 2 * NT, kTmK = 3 * NT, kTmV = kTmK + kBuf * (D / 2);
  static_assert(kTmV + kBuf * (kKeys / 2) <= 512, "TMEM columns");
  // shared memory: Q in fp16 and in bf16, two P buffers, one for the second half of a window
  // tile's P, the ring, the small arrays
  static constexpr int kQBytes = NT * D * 2;
  static constexpr int kPBytes = kKeys * NT * 2;
  static constexpr int kStage = kKeys * D * 9 / 8;
  static constexpr int kQ16 = 0, kQbf = kQBytes, kP = 2 * kQBytes, kPlo = kP + 2 * kPBytes,
                       kRing = kPlo + kPBytes;
  static constexpr int kMisc = kRing + kStages * kStage;
  static constexpr int kPSbo = 1024;                  // bytes between 8-key groups of P
};

struct SeqMeta {
  int q0, n, C, items;  // items: row tiles of the sequences before it
  int tiles, rows;      // row tiles of a KV head (of `rows` rows)
};
struct Seg {      // the part of one row tile that lies in a CTA's share
  int q0, n, C;   // sequence: first window row, window rows, cached tokens
  int b, g;
  int r0, nrows;  // rows of the tile
  int t0, len;    // key tiles [t0, t0 + len) of T (may be none); the first Tc are cached
  int T, Tc;
  int units;      // units of the line that the segment covers
  long long w0;   // first unit of the row tile on the line
};

template <int D>
struct Misc {
  using C = Cfg<D>;
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t k_full[2], v_full[2];
  // (s_full: S^T is there, its K operand buffer free, and P of two tiles before; p_full:
  // P is there, and S^T read; pv_done: O^T is up to date, the V^T operand buffer free)
  uint64_t s_full[2], p_full[2], pv_done[2], q_full, drain;
  uint32_t tmem_base;
  int abort_flag;
  int last, slot, c0, c1, second; // composition: the last to arrive; the row tile's shares
  long long W, wb, we;            // units of the line, and this CTA's share of them
  int n_cta, k0;                  // CTAs with a share; units of a row tile before its tiles
  alignas(16) float c[NT];        // cached tiles: factor of a score, log2 units
  alignas(16) float nm[NT];       // minus the column's reference
  alignas(16) int blk[NT];        // window block of the column's query (no row: sees all)
  alignas(16) long long hr[NT];   // output row (window row * heads + head) of the column
  Seg seg;                        // the softmax warps' current segment
  Seg dseg[4 * C::kDq];           // the dequantising warps' current segments
  float red[C::kSw][4][16];
  unsigned near[C::kSw][4];       // reductions over a warpgroup's warps
  uint32_t vmask[4][4];           // valid keys of a tile (by tile index mod 4, warp)
  uint8_t pvalid[C::kStages][16]; // valid tokens of a stage's pages
  bool ragged[C::kStages];        // ... some page has fewer than a full one
  // Per dim: first window block whose V is not finite, the value, and the first block at
  // which the sum of such values is NaN. By segment mod 4: V^T tiles run up to two
  // segments ahead of the epilogue that reads them.
  int nf_blk[2][4][128], nf_nan[2][4][128];
  float nf_val[2][4][128];
  // per sequence, [batch] (each array runs on behind the struct): units before it, then
  // its first window row, window rows and cached tokens
  alignas(16) long long pre[2];
};

// ---- small device helpers ----------------------------------------------------
// Paths that a steady tile does not take, out of the way of its instructions.
__device__ __forceinline__ bool rare(bool x) { return __builtin_expect(x, 0); }

template <int N>
__device__ __forceinline__ void set_regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// (d0, d1) = (a0, a1) * (b0, b1) + (c0, c1)
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b0, float b1,
                                     float c0, float c1) {
  asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ bool named_sync_or(int id, int count, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}
// One lane of a converged warp. (The compiler knows that elect.sync picks a single
// thread: an MMA issued under it takes its operands from uniform registers and issues
// at the tensor pipe's rate, 24 cycles for 48 columns, where `lane == 0` takes 45.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r));
  return r != 0;
}
// 16 consecutive 32-bit TMEM columns of this thread's lane as floats, waited for.
__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]),
        "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]),
        "=f"(r[14]), "=f"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16f(uint32_t taddr, const float (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]),
      "f"(r[8]), "f"(r[9]), "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                   taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// kind::f16 instruction descriptor: as idesc_bf16_f32, for fp16 (bf = 0) or bf16 operands.
__device__ __forceinline__ uint32_t idesc(int bf, int n, int b_mn) {
  return (1u << 4) | ((uint32_t)bf << 7) | ((uint32_t)bf << 10) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kKeys >> 4) << 24);
}

// Largest (or sum) over the 32 lanes of each of 16 registers: lanes j and j + 16 get
// column j's.
template <bool SUM>
__device__ __forceinline__ float transpose_reduce(const float (&v)[16], int lane) {
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool up = lane & 8;
    const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 8], 8);
    const float mine = up ? v[i + 8] : v[i];
    w[i] = SUM ? mine + got : fmaxf(mine, got);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float got = __shfl_xor_sync(0xffffffffu, up ? w[i] : w[i + o], o);
      const float mine = up ? w[i + o] : w[i];
      w[i] = SUM ? mine + got : fmaxf(mine, got);
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, w[0], 16);
  return SUM ? w[0] + got : fmaxf(w[0], got);
}

// Wait for a phase of an mbarrier. Every 64 polls (wait_polls) it looks whether another
// thread of the CTA gave up, and gives up itself after `wait_cycles`; the kernel's end
// reports that. (Fifteen copies of this are inlined: a report in each, or a second loop of
// polls before the clock is read, costs the instruction cache 3 to 5 % of the time.)
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                           const AttnArgs &a) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  do {
#pragma unroll 1
    for (int i = 0; i < a.wait_polls; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  } while (clock64() - t0 <= a.wait_cycles);
  *abort_flag = 1;
  return false;
}
// Arrive on an mbarrier from the warp's first lane (the warp's earlier accesses ordered
// before it), without a branch.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(lane)
      : "memory");
}

// ---- work line -----------------------------------------------------------------
// x / n, by 32-bit division where that does (64-bit ones take hundreds of cycles).
__device__ __forceinline__ long long share(long long x, long long n) {
  if ((x | n) >> 32 == 0) return (uint32_t)x / (uint32_t)n;
  return x / n;
}

// Row tiles of a sequence: `tiles` of `rows` rows each (a multiple of 16, the last
// one shorter), as equal as 16 rows allow.
struct RowTiles {
  int tiles, rows;
};
__device__ __forceinline__ RowTiles row_tiles(int total) {
  if (total <= NT) return {total > 0, (total + 15) & ~15};
  const unsigned t = (unsigned)(total + NT - 1) / NT, rows = (((unsigned)total + t - 1) / t + 15) & ~15;
  return {(int)(((unsigned)total + rows - 1) / rows), (int)rows};
}

// The segment that starts at unit w of the line (w < w1: end of the share). A row tile
// is k0 units without work, then one per key tile.
__device__ __forceinline__ Seg segment(const AttnArgs &a, const long long *pre, int k0, long long w,
                                       long long w1) {
  const SeqMeta *meta = reinterpret_cast<const SeqMeta *>(pre + ((a.batch + 1) & ~1));
  int lo = 0, hi = a.batch - 1;  // largest b with pre[b] <= w
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= w) lo = mid; else hi = mid - 1;
  }
  Seg s;
  s.b = lo;
  s.q0 = meta[lo].q0;
  s.n = meta[lo].n;
  s.C = meta[lo].C;
  const unsigned tiles = meta[lo].tiles;
  s.Tc = (s.C + kKeys - 1) / kKeys;
  s.T = s.Tc + (s.n + kKeys - 1) / kKeys;
  const int units = s.T + k0;
  const uint32_t local = (uint32_t)(w - pre[lo]);  // (the host checks: below 2^31 a sequence)
  const int it = (int)(local / (uint32_t)units), off = (int)(local - (uint32_t)it * units);
  s.w0 = w - off;
  s.units = (int)min((long long)(units - off), w1 - w);
  s.t0 = max(0, off - k0);
  s.len = max(0, off + s.units - k0) - s.t0;
  s.g = (unsigned)it / tiles;
  const int m = it - s.g * tiles;
  s.r0 = m * meta[lo].rows;
  s.nrows = min(meta[lo].rows, a.group * s.n - s.r0);
  return s;
}

// Four parts of a column into the running composition: o, l in units of 2^-m. A part
// without weight (reference -inf) may hold anything.
__device__ __forceinline__ void fold_parts(float4 &o, float &m, float &l, const float4 (&v)[4],
                                           const float2 (&ml)[4]) {
  const float top = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), m);
  if (top == -INFINITY) return;
  const float keep = m == -INFINITY ? 0.f : m == top ? 1.f : fast_exp2(m - top);
  o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
  l *= keep;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (ml[k].x == -INFINITY) continue;
    const float w = ml[k].x == top ? 1.f : fast_exp2(ml[k].x - top);
    o = make_float4(fmaf(w, v[k].x, o.x), fmaf(w, v[k].y, o.y), fmaf(w, v[k].z, o.z),
                    fmaf(w, v[k].w, o.w));
    l = fmaf(w, ml[k].y, l);
  }
  m = top;
}

// ---- dequantisation ---------------------------------------------------------------
// The eight codes of a word as packed halves. (Byte-wise conversions straight from the
// word: one ALU instruction per pair of codes, no shifts or masks.)
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t *out) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
      : "r"(w));
}
// The four e4m3 scales of a word as two packed pairs of halves.
__device__ __forceinline__ void scales_to_half(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// The 32 dims of one 16-byte piece of a K row, scales s0 (first 16) and s1.
__device__ __forceinline__ void dq_k32(uint4 w, uint32_t s0, uint32_t s1, uint32_t *out) {
  codes_to_half(w.x, out);
  codes_to_half(w.y, out + 4);
  codes_to_half(w.z, out + 8);
  codes_to_half(w.w, out + 12);
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] = hmul2(out[i], s0);
#pragma unroll
  for (int i = 8; i < 16; ++i) out[i] = hmul2(out[i], s1);
}

// Scale bytes of tokens 0-3 / 4-7 of which the first `valid` count: the others become 0.
__device__ __forceinline__ uint32_t keep_bytes(uint32_t w, int valid) {
  return valid >= 4 ? w : valid <= 0 ? 0u : w & ((1u << (8 * valid)) - 1);
}

// 32 keys (quarter h of the tile) of dim d: out[i] holds keys 2i and 2i + 1. `ragged`:
// some page holds fewer than B valid tokens (the others give 0 whatever their bytes).
template <int D, int B>
__device__ __forceinline__ void dq_v(uint32_t stage, const uint8_t *pvalid, bool ragged, int d,
                                     int h, uint32_t (&out)[16]) {
  constexpr int kPage = B * D + B * D / 8, kPages = 32 / B;
  uint32_t w[4], sc[8];  // the quarter's codes and scale bytes, every load before any use
  const uint32_t ca = stage + h * kPages * kPage + B * D / 2 + d * (B / 2);
  const uint32_t sa = stage + h * kPages * kPage + B * D + B * D / 16 + (d >> 4) * B;
#pragma unroll
  for (int p = 0; p < kPages; ++p) {
    if constexpr (B == 8) {
      w[p] = lds32(ca + p * kPage);
      const uint2 v = lds64(sa + p * kPage);
      sc[2 * p] = v.x;
      sc[2 * p + 1] = v.y;
    } else {
      if constexpr (B == 16) {
        const uint2 v = lds64(ca + p * kPage);
        w[2 * p] = v.x;
        w[2 * p + 1] = v.y;
      } else {
        const uint4 v = lds128(ca + p * kPage);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
      }
#pragma unroll
      for (int q = 0; q < B / 16; ++q) {
        const uint4 v = lds128(sa + p * kPage + 16 * q);
        const int i = p * (B / 4) + 4 * q;
        sc[i] = v.x;
        sc[i + 1] = v.y;
        sc[i + 2] = v.z;
        sc[i + 3] = v.w;
      }
    }
  }
  if (ragged) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sc[i] = keep_bytes(sc[i], (int)pvalid[h * kPages + 4 * i / B] - (4 * i) % B);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t s0, s1, s2, s3;
    scales_to_half(sc[2 * i], s0, s1);
    scales_to_half(sc[2 * i + 1], s2, s3);
    codes_to_half(w[i], out + 4 * i);
    out[4 * i] = hmul2(out[4 * i], s0);
    out[4 * i + 1] = hmul2(out[4 * i + 1], s1);
    out[4 * i + 2] = hmul2(out[4 * i + 2], s2);
    out[4 * i + 3] = hmul2(out[4 * i + 3], s3);
  }
}

// The warps that fill the K and V^T operands: thread = key of the K tile, dim of the
// V^T tile.
template <int D, int B>
__device__ __forceinline__ void dequant_role(const AttnArgs &a, Misc<D> *ms, uint32_t sb,
                                             uint32_t tmem) {
  using C = Cfg<D>;
  constexpr int kPage = B * D + B * D / 8;
  volatile int *abort_flag = &ms->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3;
  const int row = quad * 32 + lane;
  const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
  const int dq = (warp >> 2) - 1;  // the warpgroup
  const bool do_k = dq == 0;
  const int vhalf = dq - 1;        // V^T warpgroup: its 64 keys of a tile
  int u = 0, cu = 0, sg = 0;
  bool ok = true;
#pragma unroll 1
  for (long long w = ms->wb; w < ms->we && ok;) {
    int t, t_end, Tc;  // what the tile loop needs of the segment
    {
      const Seg s = segment(a, ms->pre, ms->k0, w, ms->we);
      w += s.units;
      if (s.len == 0) continue;
      t = s.t0;
      t_end = s.t0 + s.len;
      Tc = s.Tc;
      // (read back for window tiles)
      Seg &keep = ms->dseg[warp - 4];
      if (lane == 0) keep = s;
      __syncwarp();
      // The first window tile's rows to L1: the tile loads them in four steps, each of which
      // waits for its loads (one short context 19 -> 17 us, the ragged batch 109 -> 105).
      if (s.t0 + s.len > s.Tc) {
        constexpr int kLines = D / 64;  // 128-byte lines of a row
        const int first = max(s.t0 - s.Tc, 0) * kKeys;
        const char *base = static_cast<const char *>(do_k ? a.k_win : a.v_win);
#pragma unroll
        for (int c = 0; c < (do_k ? kLines : 1); ++c) {
          const int key = do_k ? row : 64 * vhalf + row / kLines, line = do_k ? c : row % kLines;
          if (first + key < s.n && (do_k || row < 64 * kLines))
            asm volatile("prefetch.global.L1 [%0];" ::"l"(
                base + ((int64_t)(s.q0 + first + key) * a.num_heads_kv + s.g) * (2 * D) + 128 * line));
        }
      }
    }
    const Seg &s = ms->dseg[warp - 4];
    int nf_blk = 0x7fffffff, nf_nan = 0x7fffffff;  // see Misc
    float nf_val = 0.f;
#pragma unroll 1
    for (; t < t_end && ok; ++t, ++u) {
      const int kb = u % C::kBuf;
      const bool reuse = u >= C::kBuf;  // the operand buffer held tile u - kBuf
      const uint32_t free_ph = (u / C::kBuf - 1) & 1;
      const bool win = t >= Tc;
      const int st = cu % C::kStages;
      const uint32_t stage = sb + C::kRing + st * C::kStage;
      // One warp of the warpgroup polls, for the tile's bytes and for the operand buffer
      // (not beside the producer or the issuer, warps 0 and 1); the others wait in the
      // named barrier, which takes no issue slots.
      if (quad == 2 + (dq == 2)) {
        if (!win)
          ok = wait_phase(smem_u32(&ms->full[st]), (cu / C::kStages) & 1, abort_flag, a);
        if (reuse)
          ok = wait_phase(smem_u32(do_k ? &ms->s_full[kb] : &ms->pv_done[kb]), free_ph, abort_flag, a) && ok;
      }
      ok = named_sync_and(C::kBarK + dq, 128, ok);
      if (rare(!ok)) break;
      tc_fence_after();
      const bool ragged = !win && ms->ragged[st];
      if (do_k) {
        const uint32_t ka = lane_base + C::kTmK + kb * (D / 2);
        if (!rare(win)) {
          const uint32_t tile = stage + (row / B) * kPage;
          const int o = row % B;
          unsigned m = 0xffffffffu;
          if (rare(ragged)) m = __ballot_sync(0xffffffffu, o < (int)ms->pvalid[st][row / B]);
          if (lane == 0) ms->vmask[u & 3][quad] = m;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            uint32_t x[16];
            const uint32_t sc = lds32(tile + B * D + o * (D / 16) + 4 * (i >> 1));
            uint32_t s0, s1;  // every scale in both halves of its pair
            scales_to_half(__byte_perm(sc, 0, i & 1 ? 0x3322 : 0x1100), s0, s1);
            dq_k32(lds128(tile + (i * B + o) * 16), s0, s1, x);
            __syncwarp();
            tmem_st16(ka + i * 16, x);
          }
        } else {
          const int wr = (t - Tc) * kKeys + row, n = s.n;  // window row
          const uint4 *src = reinterpret_cast<const uint4 *>(
              static_cast<const uint16_t *>(a.k_win) +
              ((int64_t)(s.q0 + wr) * a.num_heads_kv + s.g) * D);
#pragma unroll 1
          for (int h = 0; h < D / 32; ++h) {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 v = wr < n ? __ldg(src + 4 * h + i) : make_uint4(0, 0, 0, 0);
              x[4 * i] = v.x;
              x[4 * i + 1] = v.y;
              x[4 * i + 2] = v.z;
              x[4 * i + 3] = v.w;
            }
            __syncwarp();
            tmem_st16(ka + h * 16, x);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(smem_u32(&ms->k_full[kb]), lane);
      }
      if (!do_k) {
        if (D == 128 || row < 64) {  // (lanes past the head dim: their output is never read)
          const uint32_t va = lane_base + C::kTmV + kb * (kKeys / 2);
          if (!rare(win)) {
#pragma unroll 1
            for (int h = 2 * vhalf; h < 2 * vhalf + 2; ++h) {
              uint32_t x[16];
              dq_v<D, B>(stage, ms->pvalid[st], ragged, row, h, x);
              __syncwarp();
              tmem_st16(va + h * 16, x);
            }
          } else {
            const int64_t step = (int64_t)a.num_heads_kv * D;
#pragma unroll 1
            for (int w0 = 64 * vhalf; w0 < 64 * vhalf + 64; w0 += 16) {  // 16 keys at a time
              const int k0 = (t - Tc) * kKeys + w0;
              const int left = s.n - k0;  // window rows from here on
              const uint16_t *src = static_cast<const uint16_t *>(a.v_win) +
                                    ((int64_t)(s.q0 + k0) * a.num_heads_kv + s.g) * D + row;
              uint32_t x[8];
              bool odd = false;  // a value is not finite
#pragma unroll
              for (int i = 0; i < 8; ++i) {  // every load before any use
                const uint32_t e0 = 2 * i < left ? (uint32_t)__ldg(src + 2 * i * step) : 0u;
                const uint32_t e1 = 2 * i + 1 < left ? (uint32_t)__ldg(src + (2 * i + 1) * step) : 0u;
                x[i] = e0 | (e1 << 16);
              }
#pragma unroll
              for (int i = 0; i < 8; ++i)
                odd = odd || (x[i] & 0x7f80u) == 0x7f80u || (x[i] & 0x7f800000u) == 0x7f800000u;
              if (odd) {
                // infinite or NaN: out of the product (a hidden key's P is 0, and
                // 0 * infinity is not), into the sums of the rows that see it
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                  for (int j = 0; j < 2; ++j) {
                    const uint32_t e = (x[i] >> (16 * j)) & 0xffffu;
                    if ((e & 0x7f80u) != 0x7f80u) continue;
                    const float v = bf16_bits_to_float(e);
                    const int blk = (k0 + 2 * i + j) / B;
                    if (nf_blk == 0x7fffffff) {
                      nf_blk = blk;
                      nf_val = v;
                    } else {
                      const float z = nf_val + v;
                      if (z != z && nf_nan == 0x7fffffff) nf_nan = blk;
                    }
                    x[i] &= j ? 0x0000ffffu : 0xffff0000u;
                  }
              }
              __syncwarp();
              tmem_st8(va + w0 / 2, x);
            }
          }
          tmem_wait_st();
        }
        if (t == t_end - 1) {  // read by the epilogue, which follows this tile's product
          ms->nf_blk[vhalf][sg & 3][row] = nf_blk;
          ms->nf_nan[vhalf][sg & 3][row] = nf_nan;
          ms->nf_val[vhalf][sg & 3][row] = nf_val;
        }
        tc_fence_before();
        warp_arrive(smem_u32(&ms->v_full[kb]), lane);
      }
      if (!win) {
        warp_arrive(smem_u32(&ms->empty[st]), lane);
        ++cu;
      }
    }
    ++sg;
  }
}

// ---- the kernel ---------------------------------------------------------------------
template <int D, int B>
__global__ void __launch_bounds__((Cfg<D>::kThreads), 1) attn_kv4_kernel(const AttnArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  Misc<D> *ms = reinterpret_cast<Misc<D> *>(smem + C::kMisc);
  volatile int *abort_flag = &ms->abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (sb & 1023) {  // the swizzled tiles need the alignment that the declaration asks for
    if (tid == 0) set_err(a.err, D2F_ERR_UNSUPPORTED);
    return;
  }

  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&ms->full[i]), 1);
      mbar_init(smem_u32(&ms->empty[i]), 4 * C::kDq);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&ms->k_full[i]), 4);
      mbar_init(smem_u32(&ms->v_full[i]), 8);
      mbar_init(smem_u32(&ms->s_full[i]), 1);
      mbar_init(smem_u32(&ms->p_full[i]), 4 * C::kSw);
      mbar_init(smem_u32(&ms->pv_done[i]), 1);
    }
    mbar_init(smem_u32(&ms->q_full), 4 * C::kSw);
    mbar_init(smem_u32(&ms->drain), 1);
    ms->abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ms->tmem_base), 512);
    tmem_relinquish();
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- the line of work: units before each sequence -----------------------------
  long long *pre = ms->pre;
  SeqMeta *meta = reinterpret_cast<SeqMeta *>(pre + ((a.batch + 1) & ~1));
  if (warp == 0) {
    long long tiles = 0;  // key tiles and row tiles of the sequences so far
    int items = 0, longest = 0;
#pragma unroll 1
    for (int base = 0; base < a.batch; base += 32) {
      const int b = base + lane;
      long long u = 0;
      int it = 0;
      if (b < a.batch) {
        int q0, n, ctx;
        if (load_seq_meta(a, b, q0, n, ctx)) {
          const int T = (int)((ctx + kKeys - 1LL) / kKeys) + (n + kKeys - 1) / kKeys;
          const RowTiles rt = row_tiles(a.group * n);
          it = a.num_heads_kv * rt.tiles;
          u = (long long)T * it;
          if (it > 0) longest = max(longest, T);
          meta[b] = SeqMeta{q0, n, ctx, 0, rt.tiles, rt.rows};
        } else if (blockIdx.x == 0) {
          set_err(a.err, D2F_ERR_INVALID_ARG);
        }
      }
      long long inc = u;
      int inc_it = it;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, inc, o);
        const int y = __shfl_up_sync(0xffffffffu, inc_it, o);
        if (lane >= o) {
          inc += x;
          inc_it += y;
        }
      }
      if (b < a.batch) {
        pre[b] = tiles + inc - u;
        meta[b].items = items + inc_it - it;
      }
      tiles += __shfl_sync(0xffffffffu, inc, 31);
      items += __shfl_sync(0xffffffffu, inc_it, 31);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    // At least two key tiles a share: a smaller one costs more than it saves. Where all
    // row tiles are alike and there are no more of them than CTAs, each is cut into the
    // same number of shares, unless that leaves a share more than kSegmentTiles longer
    // than an even cut of the whole line (whose shares straddle row tiles, each a segment
    // of its own).
    long long n = max(1LL, min((long long)gridDim.x, max((long long)items, tiles / 2)));
    int k0 = kSegmentTiles;
    if (items > 0 && items <= n && (long long)longest * items == tiles) {
      const int k = (int)n / items;
      if ((longest + k - 1) / k <= share(tiles, n) + kSegmentTiles) {
        n = (long long)items * k;
        k0 = 0;
      }
    }
    __syncwarp();
    for (int b = lane; b < a.batch; b += 32) pre[b] += (long long)k0 * meta[b].items;
    if (lane == 0) {
      const long long W = tiles + (long long)k0 * items, c = blockIdx.x;
      ms->W = W;
      ms->n_cta = (int)n;
      ms->k0 = k0;
      ms->wb = c < n ? share(W * c, n) : 0;
      ms->we = c < n ? share(W * (c + 1), n) : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem_base;
  constexpr int page_bytes = B * D + B * D / 8;

  // Registers: what the control and dequantising warps do not need goes to the softmax
  // warps (the sum over the warpgroups stays under the launch's allocation).
  if (warp < 4) {
    set_regs_dec<C::kRegCtl>();
    if (warp == 0) {
      // ============================ producer =======================================
      constexpr int ppt = kKeys / B;
      int cu = 0;  // cached tiles so far: stage cu % kStages
      bool ok = true;
#pragma unroll 1
      for (long long w = ms->wb; w < ms->we && ok;) {
        const Seg s = segment(a, pre, ms->k0, w, ms->we);
        w += s.units;
        const int32_t *pt = a.page_table + (int64_t)s.b * a.max_pages_per_seq;
        const int t1 = min(s.t0 + s.len, s.Tc);
        auto fetch = [&](int t) -> int {  // page id of this lane's slot of tile t
          return t < t1 && lane < ppt && (int64_t)t * kKeys + lane * B < s.C
                     ? __ldg(pt + (int64_t)t * ppt + lane) : -1;
        };
        int id = fetch(s.t0);
#pragma unroll 1
        for (int t = s.t0; t < t1; ++t, ++cu) {
          const int next = fetch(t + 1);
          const int st = cu % C::kStages;
          if (cu >= C::kStages) {
            ok = wait_phase(smem_u32(&ms->empty[st]), (cu / C::kStages - 1) & 1, abort_flag, a);
            ok = __all_sync(0xffffffffu, ok);
            if (rare(!ok)) break;
          }
          const int first = t * kKeys + lane * B;  // first token of the slot
          int valid = lane < ppt ? min(max(s.C - first, 0), B) : 0;
          if (valid > 0 && (id < 0 || id >= a.num_pages)) {
            set_err(a.err, D2F_ERR_BAD_INDEX);
            valid = 0;
          }
          if (lane < 16) ms->pvalid[st][lane] = (uint8_t)valid;
          const unsigned have = __ballot_sync(0xffffffffu, valid > 0);
          const bool whole = __all_sync(0xffffffffu, lane >= ppt || valid == B);
          if (lane == 0) ms->ragged[st] = !whole;
          const uint32_t full = smem_u32(&ms->full[st]);
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(full, __popc(have) * (uint32_t)page_bytes);
          __syncwarp();
          if (valid > 0)
            bulk_load(sb + C::kRing + st * C::kStage + lane * page_bytes,
                      a.kv4_pool + ((int64_t)id * a.num_heads_kv + s.g) * page_bytes, page_bytes, full);
          id = next;
        }
      }
      if (lane == 0) {  // every copy issued must have landed before the CTA ends
#pragma unroll 1
        for (int i = max(0, cu - C::kStages); i < cu; ++i) {
          volatile int no_abort = 0;
          mbar_wait(smem_u32(&ms->full[i % C::kStages]), (i / C::kStages) & 1, &no_abort, a.err, kDrainCycles);
        }
      }
    } else if (warp == 1) {
      // ============================ MMA issuer =======================================
      // S^T of tile u, then O^T += of tile u - 1. One thread issues both, so S^T of tile u
      // follows the O^T product of tile u - 2: it may overwrite that tile's S^T (whose
      // readers have handed over P), and its commit tells the softmax warps that the
      // P buffer is free too.
      if (elect_one()) {
        bool ok = true;
        int u = 0, sg = 0;
        const uint64_t q_desc = smem_desc_sw128(sb + C::kQ16, 16, 1024);
        const uint64_t p_desc = smem_desc_sw128(sb + C::kP, 1024, C::kPSbo);
#pragma unroll 1
        for (long long w = ms->wb; w < ms->we && ok;) {
          const Seg s = segment(a, pre, ms->k0, w, ms->we);
          w += s.units;
          if (s.len == 0) continue;
          const int ncols = (s.nrows + 15) & ~15, t_end = s.t0 + s.len;
          ok = wait_phase(smem_u32(&ms->q_full), sg & 1, abort_flag, a);
          ++sg;
#pragma unroll 1
          for (int t = s.t0; ok; ++t) {
            if (t < t_end) {
              const int bf = t >= s.Tc;  // window tiles are bf16
              ok = wait_phase(smem_u32(&ms->k_full[u & 1]), (u >> 1) & 1, abort_flag, a);
              if (rare(!ok)) break;
              tc_fence_after();
              const uint32_t id = idesc(bf, ncols, 0);
              const uint64_t qd = smem_desc_advance(q_desc, bf ? C::kQbf - C::kQ16 : 0);
              const uint32_t sd = tmem + C::kTmS + (u & 1) * NT;
              const uint32_t ka = tmem + C::kTmK + (u & 1) * (D / 2);
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                umma_bf16_tmem_a(sd, ka + k * 8,
                                 smem_desc_advance(qd, (k >> 2) * (NT * 128) + (k & 3) * 32), id, k > 0);
              umma_commit(smem_u32(&ms->s_full[u & 1]));
              ++u;
            }
            if (t > s.t0) {
              const int v = t < t_end ? u - 2 : u - 1;  // the tile before
              ok = wait_phase(smem_u32(&ms->v_full[v & 1]), (v >> 1) & 1, abort_flag, a) &&
                   wait_phase(smem_u32(&ms->p_full[v & 1]), (v >> 1) & 1, abort_flag, a);
              if (rare(!ok)) break;
              tc_fence_after();
              const bool win = t > s.Tc;
              const uint32_t id = idesc(win, ncols, 1);
              uint64_t pd = smem_desc_advance(p_desc, (v & 1) * C::kPBytes);
              const uint32_t va = tmem + C::kTmV + (v & 1) * (kKeys / 2);
              // (a window tile's P is a pair: the same products again for its second halves)
#pragma unroll 1
              for (bool again = false;; again = true) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                  umma_bf16_tmem_a(tmem + C::kTmO, va + k * 8,
                                   smem_desc_advance(pd, k * 2 * C::kPSbo), id,
                                   again || t > s.t0 + 1 || k > 0);
                if (!win || again) break;
                pd = smem_desc_advance(p_desc, C::kPlo - C::kP);
              }
              umma_commit(smem_u32(&ms->pv_done[v & 1]));
              if (t == t_end) break;
            }
          }
        }
        umma_commit(smem_u32(&ms->drain));
        volatile int no_abort = 0;
        mbar_wait(smem_u32(&ms->drain), 0, &no_abort, a.err, kDrainCycles);
      }
    }
  } else if (warp < 4 + 4 * C::kDq) {
    set_regs_dec<C::kRegDq>();
    dequant_role<D, B>(a, ms, sb, tmem);
  } else {
    set_regs_inc<C::kRegSoft>();
    // ============================ softmax ============================================
    const int wg = (warp - 4 - 4 * C::kDq) >> 2;  // columns col0 .. col0 + 15
    const int col0 = 16 * wg;
    const int quad = warp & 3, col = lane & 15;
    const int row = quad * 32 + lane;             // key of the tile, later dim of O^T
    const int bar = C::kBarSoft + wg, bar_all = C::kBarAll;
    const int stid = tid - 128 * (1 + C::kDq);    // thread among the softmax threads
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t o_addr = lane_base + C::kTmO + col0;
    const int G = a.group, H = a.num_heads_q;
    const float win_unit = 1.0f / a.v_mul;        // O is in units of 2^v_exp
    int u = 0, sg = -1;
    bool ok = true;
#pragma unroll 1
    for (long long w = ms->wb; w < ms->we && ok;) {
      int t, t_end, Tc, n;  // what the tile loop needs of the segment
      bool idle;            // (warpgroup-uniform) no row in these columns

      // ---- Q: eight threads per row; bf16 as it is, fp16 scaled by a power of two -----
      {
        const Seg s = segment(a, pre, ms->k0, w, ms->we);
        w += s.units;
        if (s.len == 0) continue;
        ++sg;
        t = s.t0;
        t_end = s.t0 + s.len;
        Tc = s.Tc;
        n = s.n;
        idle = col0 >= s.nrows;
        const int qr = stid >> 3, part = stid & 7;
        constexpr int kV = D / 64;  // 16-byte pieces of a thread
        const int r = s.r0 + qr;
        const int64_t hr = (int64_t)(s.q0 + r / G) * H + s.g * G + r % G;
        const uint4 *src =
            reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + hr * D) + part * kV;
        uint4 v[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = qr < s.nrows ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        uint32_t top = 0;  // largest magnitude's bits, of both halves of the words at once
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const uint32_t t4 = __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                       __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
          top = __vmaxu2(top, t4);
        }
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int e = top ? min(max((int)(top >> 7) - 127 - 14, -126), 112) : 0;
        const float down = __int_as_float((127 - e) << 23);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          uint4 h;
          h.x = pack_half2(__uint_as_float(v[i].x << 16) * down, __uint_as_float(v[i].x & 0xffff0000u) * down);
          h.y = pack_half2(__uint_as_float(v[i].y << 16) * down, __uint_as_float(v[i].y & 0xffff0000u) * down);
          h.z = pack_half2(__uint_as_float(v[i].z << 16) * down, __uint_as_float(v[i].z & 0xffff0000u) * down);
          h.w = pack_half2(__uint_as_float(v[i].w << 16) * down, __uint_as_float(v[i].w & 0xffff0000u) * down);
          const int c = part * kV + i;
          const uint32_t off = (c >> 3) * (NT * 128) + (qr >> 3) * 1024 + (qr & 7) * 128 +
                               (((c & 7) ^ (qr & 7)) << 4);
          sts128(sb + C::kQ16 + off, h);
          sts128(sb + C::kQbf + off, v[i]);
        }
        // (the other warpgroups are done with the previous segment's arrays)
        named_sync(bar_all, 128 * C::kSw);
        if (stid == 0) {  // (read back by the epilogue)
          ms->seg = s;
          // Shares that hold key tiles of this row tile: unit w is in share ((w + 1) n - 1) / W.
          // A share's first segment has the CTA's first slot, any other the second: the
          // first share's part is in its second slot if the share starts before the row tile.
          const long long W = ms->W, nc = ms->n_cta, first = s.w0 + ms->k0;
          ms->c0 = (int)share((first + 1) * nc - 1, W);
          ms->c1 = (int)share((first + s.T) * nc - 1, W);
          ms->second = share(W * ms->c0, nc) < s.w0;
          ms->slot = w - s.units == ms->wb ? 0 : 1;
        }
        if (part == 0) {
          const float up = __int_as_float((127 + e) << 23);
          ms->c[qr] = a.scale_log2 * a.k_mul * up;
          ms->nm[qr] = kStart;
          ms->hr[qr] = hr;
          ms->blk[qr] = qr < s.nrows ? (r / G) / B : 0x7fffffff;
        }
        fence_proxy_async_smem();
        warp_arrive(smem_u32(&ms->q_full), lane);
        named_sync(bar_all, 128 * C::kSw);  // c, nm, hr and blk of every column
      }

      float l[16];  // this key lane's share of the columns' sums
#pragma unroll
      for (int j = 0; j < 16; ++j) l[j] = 0.f;
      float m_col = -kStart;  // reference of column `col`
      bool settled = false;  // every column has had a score near its reference
      unsigned seen_mask = 0;  // columns that have seen a key (kept while not settled)
      const int t_first = t;
#pragma unroll 1
      for (; t < t_end; ++t, ++u) {
        const int sbuf = u & 1;
        // One warp of the warpgroup polls, another scheduler's for every warpgroup (all on
        // one: 4 % slower); the others wait in the named barrier, which takes no issue slots.
        if (quad == (wg & 3)) ok = wait_phase(smem_u32(&ms->s_full[sbuf]), (u >> 1) & 1, abort_flag, a);
        ok = named_sync_and(bar, 128, ok);
        if (rare(!ok)) break;
        tc_fence_after();
        if (idle) {
          warp_arrive(smem_u32(&ms->p_full[sbuf]), lane);
          continue;
        }
        const bool win = t >= Tc;
        // scores in log2 units against the columns' references
        float x[16];
        const unsigned keys = win ? 0u : ms->vmask[u & 3][quad];
        tmem_ld16f(lane_base + C::kTmS + sbuf * NT + col0, x);
        if (keys == 0xffffffffu) {  // a cached tile of whole pages: every column sees every key
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(&ms->c[col0 + j]);
            const float4 n = *reinterpret_cast<const float4 *>(&ms->nm[col0 + j]);
            fma2(x[j], x[j + 1], x[j], x[j + 1], c.x, c.y, n.x, n.y);
            fma2(x[j + 2], x[j + 3], x[j + 2], x[j + 3], c.z, c.w, n.z, n.w);
          }
        } else {
          const int kw = (t - Tc) * kKeys + row;  // window key
          const bool none = win ? kw >= n : !((keys >> lane) & 1);
          const int kblk = win ? kw / B : -1;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            x[j] = fmaf(x[j], win ? a.scale_log2 : ms->c[col0 + j], ms->nm[col0 + j]);
            if (none || ms->blk[col0 + j] < kblk) x[j] = -INFINITY;
          }
        }
        const float top =
            fmax3(fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmax3(x[6], x[7], x[8])),
                  fmax3(fmax3(x[9], x[10], x[11]), x[12], x[13]), fmaxf(x[14], x[15]));
        bool move_any = top > kHigh;
        if (!settled) {
          // columns with a score above kLow, over the warpgroup's keys of this tile
          unsigned near = 0;
#pragma unroll
          for (int j = 0; j < 16; ++j) near |= x[j] > kLow ? 1u << j : 0u;
          near = __reduce_or_sync(0xffffffffu, near);
          if (lane == 0) ms->near[wg][quad] = near;
          named_sync(bar, 128);
          settled = (ms->near[wg][0] | ms->near[wg][1] | ms->near[wg][2] | ms->near[wg][3]) == 0xffffu;
          if (settled) seen_mask = 0xffffu;
          move_any = move_any || !settled;
        }
        if (rare(named_sync_or(bar, 128, move_any))) {
          // ---- move references: the columns' maxima over the tile ------------------
          // every P.V product so far must have landed in O before O is rescaled
          if (t > t_first)
            ok = wait_phase(smem_u32(&ms->pv_done[sbuf ^ 1]), ((u - 1) >> 1) & 1, abort_flag, a) && ok;
          __syncwarp();
          tc_fence_after();
          ms->red[wg][quad][col] = transpose_reduce<false>(x, lane);
          ok = named_sync_and(bar, 128, ok);
          if (rare(!ok)) break;
          // column `col`: its largest score against the reference. Without a visible key
          // (-inf) there is nothing to move to; the column settles with a later tile.
          const float rise = fmaxf(fmaxf(ms->red[wg][0][col], ms->red[wg][1][col]),
                                   fmaxf(ms->red[wg][2][col], ms->red[wg][3][col]));
          const bool seen = rise > -INFINITY;
          const bool move = seen && (rise > kHigh || (!settled && rise < kLow && !(seen_mask >> col & 1)));
          const float d_col = move ? rise - kLift : 0.f;
          // (a column that has seen no key yet has nothing to rescale)
          const float a_col = !move ? 1.f : !(seen_mask >> col & 1) ? 0.f : fast_exp2(-d_col);
          m_col += d_col;
          seen_mask |= __ballot_sync(0xffffffffu, seen) & 0xffffu;
          settled = seen_mask == 0xffffu;
          if (quad == 0 && lane < 16) ms->nm[col0 + lane] -= d_col;
          float o[16];
          if (t > t_first) tmem_ld16f(o_addr, o);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float al = __shfl_sync(0xffffffffu, a_col, j);
            x[j] -= __shfl_sync(0xffffffffu, d_col, j);
            l[j] *= al;
            o[j] *= al;
          }
          if (t > t_first) {
            tmem_st16f(o_addr, o);
            tmem_wait_st();
          }
          named_sync(bar, 128);  // nm is written, and red may be written again
        }
        // ---- P = 2^x; the row sums take the unrounded values ------------------------
        const uint32_t pb = sb + C::kP + sbuf * C::kPBytes + row * 128;
        float p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) p[j] = fast_exp2(x[j]);
#pragma unroll
        for (int j = 0; j < 16; j += 2) add2(l[j], l[j + 1], l[j], l[j + 1], p[j], p[j + 1]);
        uint32_t h[8];
        if (win) {
          const uint32_t lo = sb + C::kPlo + row * 128;
          // (the one buffer of second halves: the window tile before must be done with it)
          if (rare(t > max(t_first, Tc))) {
            ok = wait_phase(smem_u32(&ms->pv_done[sbuf ^ 1]), ((u - 1) >> 1) & 1, abort_flag, a);
            ok = named_sync_and(bar, 128, ok);
            if (rare(!ok)) break;
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t r[4];
#pragma unroll
            for (int j = 4 * i; j < 4 * i + 4; ++j) {
              const float x0 = p[2 * j] * win_unit, x1 = p[2 * j + 1] * win_unit;
              h[j] = pack_bf16x2(x0, x1);
              r[j - 4 * i] = pack_bf16x2(x0 - __uint_as_float(h[j] << 16),
                                         x1 - __uint_as_float(h[j] & 0xffff0000u));
            }
            sts128(lo + (((2 * wg + i) ^ (row & 7)) << 4), make_uint4(r[0], r[1], r[2], r[3]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) h[j] = pack_half2(p[2 * j], p[2 * j + 1]);
        }
        sts128(pb + (((2 * wg) ^ (row & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
        sts128(pb + (((2 * wg + 1) ^ (row & 7)) << 4), make_uint4(h[4], h[5], h[6], h[7]));
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(smem_u32(&ms->p_full[sbuf]), lane);
      }

      // ---- epilogue of the segment (a warpgroup that gave up joins the vote) ----------
      const int last = u - 1;
      ok = ok && wait_phase(smem_u32(&ms->pv_done[last & 1]), (last >> 1) & 1, abort_flag, a);
      __syncwarp();
      ms->red[wg][quad][col] = transpose_reduce<true>(l, lane);
      ok = named_sync_and(bar_all, 128 * C::kSw, ok);
      if (rare(!ok)) break;
      tc_fence_after();
      // sum of column `col` (the same in the four warps)
      float L = (ms->red[wg][0][col] + ms->red[wg][1][col]) +
                (ms->red[wg][2][col] + ms->red[wg][3][col]);
      float M = L > 0.f || L != L ? m_col : -INFINITY;  // (no key seen: no reference)
      float f = a.v_mul / L;
      const Seg s = ms->seg;
      const int live = min(16, s.nrows - col0);  // columns with a row (none or fewer: idle)
      const bool dim_on = D == 128 || row < D, whole = s.len == s.T;
      const bool odd = s.t0 + s.len > s.Tc && min(ms->nf_blk[0][sg & 3][row], ms->nf_blk[1][sg & 3][row]) != 0x7fffffff;
      uint16_t *outp = static_cast<uint16_t *>(a.out) + row;
      constexpr int kSlotFloats = NT * D + 2 * NT;
      float *slot = a.ws_o + ((int64_t)2 * blockIdx.x + ms->slot) * kSlotFloats;
      float o[16];
      tmem_ld16f(o_addr, o);
      tc_fence_before();
      if (rare(odd)) {  // infinite or NaN window values of this dim, for the rows that see them
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int nb = ms->nf_blk[h][sg & 3][row], nn = ms->nf_nan[h][sg & 3][row];
          const float nv = ms->nf_val[h][sg & 3][row];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int bj = ms->blk[col0 + j];
            if (nb != 0x7fffffff && bj >= nb) o[j] += bj >= nn ? NAN : nv;
          }
        }
      }
      if (whole) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float y = o[j] * __shfl_sync(0xffffffffu, f, j);
          if (j < live && dim_on) outp[ms->hr[col0 + j] * D] = float_to_bf16_bits(y);
        }
        if (quad == 0 && lane < live && a.lse_out)
          a.lse_out[ms->hr[col0 + lane]] = (M + __log2f(L)) * 0.6931471805599453f;
        continue;
      }
      // ---- a part of the row tile: to the workspace; the last to arrive composes --------
      if (dim_on) {
        float *so = slot + col0 * D + row;
#pragma unroll
        for (int j = 0; j < 16; ++j) __stcg(so + j * D, o[j]);  // (columns without a row too)
      }
      if (quad == 0 && lane < 16)
        __stcg(reinterpret_cast<float2 *>(slot + NT * D) + col0 + lane, make_float2(M, L));
      named_sync(bar_all, 128 * C::kSw);
      if (stid == 0) {
        // (release and acquire at once: the barrier ordered the others' stores before it,
        // and the next one orders their loads behind it)
        int32_t *counter = a.counters + ms->c0;
        const bool is_last = atomic_add_acq_rel(counter, 1) == ms->c1 - ms->c0;
        if (is_last) *counter = 0;
        ms->last = is_last;
      }
      named_sync(bar_all, 128 * C::kSw);
      if (!ms->last) continue;  // (written again only after the next segment's first barrier)
      const int c0 = ms->c0, parts = ms->c1 - c0 + 1;
      auto part = [&](int c) -> const float * {
        return a.ws_o + ((int64_t)2 * (c0 + c) + (c == 0 ? ms->second : 0)) * kSlotFloats;
      };
      // The composition, over the whole CTA's columns: a thread owns four dims of a column
      // at a time, reads four parts at once and keeps the running (reference, sum) of the
      // column beside its outputs.
      constexpr int kD4 = D / 4, kStep = 128 * C::kSw / kD4;  // threads a column, columns a pass
      const int d4 = 4 * (stid % kD4);
#pragma unroll 1
      for (int cl = stid / kD4; cl < s.nrows; cl += kStep) {
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        float My = -INFINITY, Ly = 0.f;
#pragma unroll 1
        for (int c = 0; c < parts; c += 4) {
          float4 v[4];
          float2 ml[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float *p = part(min(c + k, parts - 1));
            v[k] = __ldcg(reinterpret_cast<const float4 *>(p + cl * D + d4));
            ml[k] = __ldcg(reinterpret_cast<const float2 *>(p + NT * D) + cl);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (c + k >= parts) ml[k].x = -INFINITY;  // (no part: no weight)
          fold_parts(y, My, Ly, v, ml);
        }
        const float g = a.v_mul / Ly;
        const int64_t at = ms->hr[cl];
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at * D + d4) =
            make_uint2(pack_bf16x2(y.x * g, y.y * g), pack_bf16x2(y.z * g, y.w * g));
        if (d4 == 0 && a.lse_out) a.lse_out[at] = (My + __log2f(Ly)) * 0.6931471805599453f;
      }
    }
  }

  tc_fence_before();
  __syncwarp();
  __syncthreads();  // every role is done, every copy and MMA complete
  tc_fence_after();
  if (tid == 0 && ms->abort_flag) set_err(a.err, D2F_ERR_TIMEOUT);
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D>
constexpr int smem_bytes(int batch) {
  return Cfg<D>::kMisc + (int)sizeof(Misc<D>) + 8 * (batch + 2) + (int)sizeof(SeqMeta) * batch;
}

template <int D, int B>
cudaError_t launch(const AttnArgs &a, cudaStream_t s) {
  static_assert(smem_bytes<D>(kMaxBatch) <= 232448, "shared memory of a CTA");
  static std::atomic<bool> opted[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !opted[dev]) {
    e = cudaFuncSetAttribute(attn_kv4_kernel<D, B>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_bytes<D>(kMaxBatch));
    if (e != cudaSuccess) return e;
    if (dev < 64) opted[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.num_splits);
  cfg.blockDim = dim3(Cfg<D>::kThreads);
  cfg.dynamicSmemBytes = smem_bytes<D>(a.batch);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, attn_kv4_kernel<D, B>, a);
}

template <int D>
cudaError_t launch_d(const AttnArgs &a, cudaStream_t s) {
  switch (a.block_size) {
    case 8: return launch<D, 8>(a, s);
    case 16: return launch<D, 16>(a, s);
    default: return launch<D, 32>(a, s);
  }
}

}  // namespace

cudaError_t launch_attn_kv4(const AttnArgs &a, cudaStream_t s) {
  return a.head_dim == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace d2f
