// Tensor-core path of d2f_token_attn: bf16, head_dim 64 or 128.
//
// Source of the computation: "D2F: 확산 언어 모델이 KV 캐시를 얻고 자기회귀 모델보다 2.5배
// 빨라지는 방법", §운영 관점 (paged cache, one block a page); "확산 언어 모델(Diffusion
// LLM)이란 무엇인가", §FlashBlock (attention parts recombined in log space).
//
// A read of the cache bounds it: every K and V element is used for the G query heads of its group
// and no more. So the products take the small tensor instructions (mma.sync m16n8k16), whose
// operands are registers:
//   S^T [16 keys x 8 heads] = K [16 keys x D] Q^T,  O^T [D x 8 heads] += V^T [D x 16 keys] P^T.
// The sums over D and over keys may run in any order, so a thread's operand elements are chosen
// for its loads: 16 bytes (8 dims) of K of two keys per 32 dims, and 16 bytes of V of four keys
// per 64 dims, whose pairs of keys are put together by byte permutes. P^T's layout comes from
// S^T's by 8 x 8 transposes in registers.
//
// A warp takes 16 keys at a time (a chunk: 8 KB with head_dim 128) through a ring of its own in
// shared memory, filled by 16-byte asynchronous copies, so it waits for nobody but its copies.
// The copies run ahead across everything that the warp does, 128 KB an SM are always on the
// way. (With K and V loaded to registers, 4 to 8 KB a warp: 4 x 32,768 tokens of 32 heads 392 us.)
// Rows lie in shared memory with their 16-byte pieces permuted (place()), so that the stores and
// both operands' loads meet no bank twice.
//
// All chunks of the launch, (sequence, KV head, 8 or 16 heads, chunk), are one line, cut into runs:
// three quarters of it one run a warp, the rest two smaller runs a warp, handed out on arrival
// (SMs differ in bandwidth by some 15 %). Every SM reads what it can whatever the lengths
// are, and no warp waits for another. What of a (sequence, KV head) lies within a run is written
// out; the parts of a cut one go to the workspace, and a second launch composes them in the
// order of the line. (With the warps of a CTA on the same chunks in turn, a barrier for each
// (sequence, KV head) and the composition by the CTA that came last, 16 x 251 to 4096 tokens of 32
// heads took 130 us.)
//
// Both launches in a graph, L2 flushed: 4 x 32,768 tokens of 32 heads 337 us, 6.4 TB/s; 64 x 8192 of 28
// heads on 4 200 us, 13 of them the composition, 5.4 TB/s; 16 x 251 to 4096 of 32 heads 101 us, 4.5 TB/s
// (4 us for the places on the line and the first copies, 4 the composition). In a row of calls, which
// overlap and find part of the cache in L2, 314, 180 and 84. head_dim 64: 255, 149 and 75 us, 4.2, 3.6
// and 3.0 TB/s (a chunk of 16 keys has half the bytes).
//
// Softmax in log2 units with a reference a head and warp, which moves only when a score is more
// than 2^8 above it. Weights enter the product with V as bf16 (2^-8 of each; the sum keeps the
// unrounded ones); scores, sums and outputs are float.
#include "attn_common.cuh"

namespace d2f {
namespace {

constexpr float kMove = 8.f;
constexpr float kNothing = -3.402823466e38f;  // reference of a head that has seen no key: the lowest float

// 16 bytes to shared memory, or 16 zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// Piece x of token t of a chunk lies at x ^ place(t). Eight lanes that load 16 bytes together hold
// K of tokens 2 i, 2 i + 1 (four pieces of each: bit 2 of the two places differs) or V of tokens
// e, e + 2, e + 4, e + 6 (two pieces of each: bits 1 and 2 of the four differ).
__device__ __forceinline__ uint32_t place(uint32_t t) {
  return ((t & 1) << 2) ^ (t & 2) ^ ((t & 4) ? 5u : 0u);
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int D, int NQ>
struct Cfg {
  static constexpr int W = kTokenWarps;
  static constexpr int kThreads = 32 * W;
  static constexpr int HQ = 8 * NQ;            // heads of a run's warp
  static constexpr int kRow = 2 * D;           // bytes of a token's K or V
  static constexpr int kChunk = 2 * 16 * kRow;
  static constexpr int S = D == 64 ? 6 : 3;    // chunks of a warp's ring
  // shared memory: the rings, the sequences' places on the line and lengths, the chunks' headers
  static constexpr int kPre = W * S * kChunk;
  static constexpr int kCtx = kPre + (kTokenScanBatch + 1) * 8;
  static constexpr int kMeta = (kCtx + kTokenScanBatch * 4 + 15) / 16 * 16;
  static constexpr int kBytes = kMeta + W * S * 32;
  static_assert(kBytes <= 232448 - 1024, "shared memory per CTA");
};

// The line of `total` chunks and its runs: n1 runs of the first `a` chunks, n2 of the rest.
struct Runs {
  int64_t total, a, n1, n2;
  __device__ Runs(int64_t total, int warps) : total(total) {
    // (shorter lines: one run a warp, of a chunk at least. Cut from 16 chunks a warp on, 16 x 8192 tokens,
    // 28 heads on 4, took 77 us against 68, 4 x 32,768 90 against 70.)
    const bool two = total >= 32LL * warps;
    a = two ? total - total / 4 : total;
    n1 = min((int64_t)warps, total);
    n2 = two ? 2 * warps : 0;
  }
  __device__ int64_t begin(int64_t x) const {
    return x <= n1 ? x * a / n1 : a + (x - n1) * (total - a) / n2;
  }
  __device__ int64_t of(int64_t u) const {  // the run that holds chunk u
    return u < a ? ((u + 1) * n1 - 1) / a : n1 + ((u - a + 1) * n2 - 1) / (total - a);
  }
};

// Chunks of a sequence of C cached tokens; a negative C takes no part.
__device__ __forceinline__ int chunks_of(int C, int fresh) {
  return C < 0 ? 0 : max(1, (C + fresh + 15) / 16);
}
// The length of sequence b, negative where it takes no part.
__device__ __forceinline__ int length_of(const TokenArgs &a, int b, bool report) {
  const int C = __ldg(a.ctx_len + b);
  if ((long long)C > (long long)a.max_pages_per_seq * a.block_size) {
    if (report) set_err(a.err, D2F_ERR_INVALID_ARG);
    return -1;
  }
  return C;
}

struct Seg {       // chunks u0 .. u1 - 1 of the T of a (sequence, KV head, head chunk)
  int b, pair, C, u0, u1, T;  // pair: KV head * chunks + head chunk
  int64_t first;   // place of chunk 0 on the line
};
struct Meta {      // a chunk in the ring
  uint32_t keys;   // bits 0 .. 15: the tokens exist; flags
  int b, pair, u, C, run;
  int pad[2];
};
constexpr uint32_t kFirst = 1u << 16, kLast = 1u << 17;  // of the segment
constexpr uint32_t kWhole = 1u << 18;  // the segment is all of the pair's chunks
constexpr uint32_t kHead = 1u << 19;   // the segment holds the pair's first chunk

// Weight of a part with maximum x and sum l among parts with the maximum top. (A part whose scores
// are all NaN has no maximum and a NaN sum; a part without keys has the weight 0.)
__device__ __forceinline__ float weight(float x, float l, float top) {
  return x == kNothing && l == 0.f ? 0.f : fast_exp2(x - top);
}

template <int D, int NQ>
__global__ void __launch_bounds__(Cfg<D, NQ>::kThreads, 1) token_tc_kernel(const TokenArgs a) {
  using L = Cfg<D, NQ>;
  constexpr int W = L::W, HQ = L::HQ, NT = L::kThreads, KB = D / 32, VB = D / 64, S = L::S;
  extern __shared__ __align__(128) uint8_t sm[];
  int64_t *pre_s = reinterpret_cast<int64_t *>(sm + L::kPre);
  int *ctx_s = reinterpret_cast<int *>(sm + L::kCtx);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  if (tid == 0) D2F_TRACE_MARK(4, 0);
  const int Hk = a.num_heads_kv, B = a.block_size, fresh = a.k_new ? 1 : 0;
  const int pairs = Hk * a.chunks;  // of a sequence
  const bool line = a.line;
  const int warps = gridDim.x * W, me = warp * gridDim.x + blockIdx.x;
  grid_dependency_wait();
  if (line) {
    for (int b = tid; b < a.batch; b += NT) ctx_s[b] = length_of(a, b, blockIdx.x == 0);
    __syncthreads();
    if (warp == 0) {  // places of the sequences on the line
      int64_t carry = 0;
      for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        const int64_t x = b < a.batch ? (int64_t)chunks_of(ctx_s[b], fresh) * pairs : 0;
        int64_t upto = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        if (b < a.batch) pre_s[b] = carry + upto - x;
        carry += __shfl_sync(0xffffffffu, upto, 31);
      }
      if (lane == 0) pre_s[a.batch] = carry;
    }
    __syncthreads();
  }
  const Runs runs(line ? pre_s[a.batch] : 0, warps);
  if (tid == 0) D2F_TRACE_MARK(4, 1);

  // ---- the ring: the place of the copies, chunk fu of segment f of run x, which ends at `end` ----
  const uint32_t ring = smem_u32(sm) + warp * (S * L::kChunk);
  volatile Meta *meta = reinterpret_cast<volatile Meta *>(sm + L::kMeta) + warp * S;
  Seg f{};
  int fu = 0, p0 = 0, ids0 = 0, ids1 = 0;  // ids0, ids1: page-table entries p0 + lane and p0 + 32 + lane
  int64_t x = me, x_next = 0, end = 0;
  bool more = true;  // f is a segment
  auto ids_at = [&](int p) -> int {
    return p < (f.C + B - 1) / B ? __ldg(a.page_table + (int64_t)f.b * a.max_pages_per_seq + p) : 0;
  };
  auto enter_seg = [&] {
    f.u1 = (int)min((int64_t)f.T, end - f.first);
    fu = f.u0;
    p0 = 16 * fu / B;
    ids0 = ids_at(p0 + lane);
    ids1 = ids_at(p0 + 32 + lane);
  };
  auto ask = [&] {  // (the answer is used when this run ends)
    if (lane == 0) x_next = (line ? runs.n1 : warps) + atomicAdd(a.counters, 1);
  };
  auto enter_run = [&] {
    if (line) {
      more = x < runs.n1 + runs.n2;
      if (!more) return;
      if (runs.n2) ask();
      const int64_t at = runs.begin(x);
      end = runs.begin(x + 1);
      int lo = 0, hi = a.batch;  // pre_s[lo] <= at < pre_s[hi], lo the last such
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre_s[mid] <= at) lo = mid;
        else hi = mid;
      }
      f.b = lo;
      f.C = ctx_s[lo];
      f.T = chunks_of(f.C, fresh);
      const int64_t in = at - pre_s[lo];
      f.pair = (int)(in / f.T);
      f.u0 = (int)(in - (int64_t)f.pair * f.T);
      f.first = at - f.u0;
    } else {  // a run a (sequence, KV head, head chunk)
      while (true) {
        more = x < (int64_t)a.batch * pairs;
        if (!more) return;
        ask();
        f.b = (int)(x / pairs);
        f.pair = (int)(x % pairs);
        f.C = length_of(a, f.b, lane == 0);
        f.T = chunks_of(f.C, fresh);
        if (f.T > 0) break;
        x = __shfl_sync(0xffffffffu, x_next, 0);
      }
      f.u0 = 0;
      f.first = 0;
      end = f.T;
    }
    enter_seg();
  };
  enter_run();
  uint32_t filled = 0;
  auto fill = [&](int stage) {
    if (more) {
      if (16 * fu / B >= p0 + 32) {
        p0 += 32;
        ids0 = ids1;
        ids1 = ids_at(p0 + 32 + lane);
      }
      const int key = 16 * fu + (lane & 15), entry = key / B, g = f.pair / a.chunks;
      const int lo = __shfl_sync(0xffffffffu, ids0, entry - p0), hi = __shfl_sync(0xffffffffu, ids1, entry - p0);
      const int page = entry - p0 < 32 ? lo : hi;
      int64_t row = -1;  // of the pool's rows, -1: no key, -2: the new token's
      if (key < f.C) {
        if (page >= 0 && page < a.num_pages) row = ((int64_t)page * Hk + g) * B + (key - entry * B);
        else set_err(a.err, D2F_ERR_BAD_INDEX);
      } else if (key == f.C && fresh) {
        row = -2;
      }
      const uint32_t keys = __ballot_sync(0xffffffffu, row != -1) & 0xffffu;
      if (lane == 0) {
        meta[stage].keys = keys | (fu == f.u0 ? kFirst : 0) | (fu + 1 == f.u1 ? kLast : 0) |
                           (f.u0 == 0 ? kHead : 0) | (f.u0 == 0 && f.u1 == f.T ? kWhole : 0);
        meta[stage].b = f.b;
        meta[stage].pair = f.pair;
        meta[stage].u = fu;
        meta[stage].C = f.C;
        meta[stage].run = (int)x;
      }
      const uint32_t dst = ring + stage * L::kChunk;
      const int64_t new_at = ((int64_t)f.b * Hk + g) * L::kRow;
      constexpr int P = D / 8, per = 32 / P;  // pieces of a row, tokens a step
      const int piece = lane % P, sub = lane / P;
#pragma unroll
      for (int i = 0; i < 16 / per; ++i) {
        const int t = i * per + sub;
        const int64_t y = __shfl_sync(0xffffffffu, row, t);
        const uint32_t to = dst + t * L::kRow + ((piece ^ place(t & 7)) << 4);
        const int64_t from = (y == -2 ? new_at : y < 0 ? 0 : y * L::kRow) + piece * 16;
        copy16(to, static_cast<const char *>(y == -2 ? a.k_new : a.k_pool) + from, y != -1);
        copy16(to + 16 * L::kRow, static_cast<const char *>(y == -2 ? a.v_new : a.v_pool) + from, y != -1);
      }
      ++filled;
      if (++fu == f.u1) {
        const int64_t next = f.first + f.T;
        if (line && next < end) {  // the run goes on
          f.first = next;
          f.u0 = 0;
          if (++f.pair == pairs) {
            f.pair = 0;
            do ++f.b;
            while (ctx_s[f.b] < 0);  // (a sequence with chunks follows: next < end)
            f.C = ctx_s[f.b];
            f.T = chunks_of(f.C, fresh);
          }
          enter_seg();
        } else {
          x = line && !runs.n2 ? runs.n1 : __shfl_sync(0xffffffffu, x_next, 0);
          enter_run();
        }
      }
    }
    copy_commit();
  };
  uint4 q[NQ][KB], qn[NQ][KB];
  auto load_q = [&](int b, int pair) {
    const int g = pair / a.chunks, hc = pair % a.chunks;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int h = hc * HQ + n * 8 + r;  // head of the group
      const char *src = static_cast<const char *>(a.q) +
                        ((int64_t)b * a.num_heads_q + g * a.group + h) * L::kRow + c * 16;
#pragma unroll
      for (int k = 0; k < KB; ++k)
        qn[n][k] = h < a.group ? __ldg(reinterpret_cast<const uint4 *>(src + k * 64)) : make_uint4(0, 0, 0, 0);
    }
  };
  if (more) load_q(f.b, f.pair);
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fill(i);
  if (tid == 0) D2F_TRACE_MARK(4, 2);

  int stage = 0;
  const uint32_t k_at = r * L::kRow + ((c ^ place(r)) << 4);                         // ^ kb << 6
  const uint32_t v_at = 16 * L::kRow + 2 * c * L::kRow + ((r ^ place(2 * c)) << 4);  // token 2 c, ^ j << 7
  float m[NQ][2], l[NQ][2], o[NQ][VB][4][4];
  for (uint32_t done = 0; done < filled; ++done) {
    copy_wait<S - 2>();
    __syncwarp();  // this chunk has landed, and every lane is done with the one before
    fill(stage == 0 ? S - 1 : stage - 1);
    __syncwarp();
    const uint32_t at = ring + stage * L::kChunk;
    Meta mt;
    mt.keys = meta[stage].keys;
    mt.b = meta[stage].b;
    mt.pair = meta[stage].pair;
    mt.u = meta[stage].u;
    mt.C = meta[stage].C;
    mt.run = meta[stage].run;
    stage = stage + 1 == S ? 0 : stage + 1;
    const int g = mt.pair / a.chunks, hc = mt.pair % a.chunks;
    if (mt.keys & kFirst) {
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
#pragma unroll
        for (int k = 0; k < KB; ++k) q[i][k] = qn[i][k];
        m[i][0] = m[i][1] = kNothing;
        l[i][0] = l[i][1] = 0.f;
#pragma unroll
        for (int j = 0; j < VB; ++j)
#pragma unroll
          for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][j][w][e] = 0.f;
      }
    }
    if (done + 1 < filled && (meta[stage].keys & kFirst)) load_q(meta[stage].b, meta[stage].pair);
    if (fresh && hc == 0 && mt.C >= 16 * mt.u && mt.C < 16 * mt.u + 16) {
      // the new token to its slot, which no CTA reads in this call
      const int pg = mt.C / B < a.max_pages_per_seq
                         ? __ldg(a.page_table + (int64_t)mt.b * a.max_pages_per_seq + mt.C / B) : -1;
      if (pg < 0 || pg >= a.num_pages) {
        if (lane == 0) set_err(a.err, D2F_ERR_BAD_INDEX);
      } else if ((lane & 15) < D / 8) {
        const int64_t from = ((int64_t)mt.b * Hk + g) * (D / 8) + (lane & 15);
        const int64_t to = (((int64_t)pg * Hk + g) * B + mt.C % B) * (D / 8) + (lane & 15);
        if (lane < 16)
          static_cast<uint4 *>(a.k_pool)[to] = static_cast<const uint4 *>(a.k_new)[from];
        else
          static_cast<uint4 *>(a.v_pool)[to] = static_cast<const uint4 *>(a.v_new)[from];
      }
    }
    float x[NQ][4];
#pragma unroll
    for (int i = 0; i < NQ; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const uint4 k0 = ld_shared_v4(at + (k_at ^ (k << 6))), k1 = ld_shared_v4(at + (k_at ^ (k << 6)) + 8 * L::kRow);
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        mma_bf16(x[i], k0.x, k1.x, k0.y, k1.y, q[i][k].x, q[i][k].y);
        mma_bf16(x[i], k0.z, k1.z, k0.w, k1.w, q[i][k].z, q[i][k].w);
      }
    }
    uint32_t p[NQ][2];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      bool move = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[i][e] = (mt.keys >> (r + 8 * (e >> 1)) & 1u) ? x[i][e] * a.scale_log2 : -INFINITY;
        move |= x[i][e] > m[i][e & 1] + kMove;
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = fmaxf(x[i][e], x[i][e + 2]);
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          top = fmaxf(top, m[i][e]);
          const float alpha = fast_exp2(m[i][e] - top);
          m[i][e] = top;
          l[i][e] *= alpha;
#pragma unroll
          for (int j = 0; j < VB; ++j)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              o[i][j][w][e] *= alpha;
              o[i][j][w][e + 2] *= alpha;
            }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[i][e] = fast_exp2(x[i][e] - m[i][e & 1]);
        l[i][e & 1] += x[i][e];
      }
      p[i][0] = transpose8(pack_bf16x2(x[i][0], x[i][1]));
      p[i][1] = transpose8(pack_bf16x2(x[i][2], x[i][3]));
    }
#pragma unroll
    for (int j = 0; j < VB; ++j) {
      uint32_t v[4][4];  // tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 y = ld_shared_v4(at + (v_at ^ (j << 7) ^ ((e & 1) << 6)) + ((e & 1) + 8 * (e >> 1)) * L::kRow);
        v[e][0] = y.x;
        v[e][1] = y.y;
        v[e][2] = y.z;
        v[e][3] = y.w;
      }
#pragma unroll
      for (int w = 0; w < 4; ++w) {  // dims 64 j + 8 r + 2 w and + 1
        const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5410), a1 = __byte_perm(v[0][w], v[1][w], 0x7632);
        const uint32_t a2 = __byte_perm(v[2][w], v[3][w], 0x5410), a3 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
        for (int i = 0; i < NQ; ++i) mma_bf16(o[i][j][w], a0, a1, a2, a3, p[i][0], p[i][1]);
      }
    }
    if (!(mt.keys & kLast)) continue;

    // ---- the segment's outputs, or its part ----
    const int heads = min(HQ, a.group - hc * HQ);
    const int64_t hr0 = (int64_t)mt.b * a.num_heads_q + g * a.group + hc * HQ;
    const int slot_heads = min(HQ, a.group);
    float *slot = a.partial + (2 * (int64_t)mt.run + (mt.keys & kHead ? 1 : 0)) * (slot_heads * (D + 4));
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[i][e];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const int h = 8 * i + 2 * c + e;
        if (h >= heads) continue;
        const bool none = sum == 0.f;  // no key, or every score is -inf
        if (mt.keys & kWhole) {
          const float inv = 1.0f / sum;
          if (r == 0 && a.lse_out)
            a.lse_out[hr0 + h] = none ? -INFINITY : (m[i][e] + __log2f(sum)) * 0.6931471805599453f;
#pragma unroll
          for (int j = 0; j < VB; ++j) {
            uint32_t y[4];
#pragma unroll
            for (int w = 0; w < 4; ++w)
              y[w] = none ? 0u : pack_bf16x2(o[i][j][w][e] * inv, o[i][j][w][e + 2] * inv);
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + (hr0 + h) * D + 64 * j + 8 * r) =
                make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
          if (r == 0) *reinterpret_cast<float2 *>(slot + slot_heads * D + 2 * h) = make_float2(m[i][e], sum);
#pragma unroll
          for (int j = 0; j < VB; ++j) {
            float4 *dst = reinterpret_cast<float4 *>(slot + h * D + 64 * j + 8 * r);
            dst[0] = make_float4(o[i][j][0][e], o[i][j][0][e + 2], o[i][j][1][e], o[i][j][1][e + 2]);
            dst[1] = make_float4(o[i][j][2][e], o[i][j][2][e + 2], o[i][j][3][e], o[i][j][3][e + 2]);
          }
        }
      }
  }
  if (tid == 0) D2F_TRACE_MARK(4, 3);
  // (The composition waits for this grid's end. Started from the first, its CTAs wait beside warps that
  // still work: 1024 tokens of 32 heads 21.7 us in a graph against 17.5.)
  grid_launch_dependents();
  // the last warp of the launch leaves the counters as they were
  if (lane == 0 && atomic_add_acq_rel(a.counters + 1, 1) == warps - 1) a.counters[0] = a.counters[1] = 0;
}

// Composition of the pairs whose chunks lie in several runs, a CTA a (sequence, KV head, query head).
// Its warps share the parts.
constexpr int kMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) token_merge_kernel(const TokenArgs a, int warps, int hq) {
  constexpr int MW = kMergeThreads / 32, VL = D / 32, N = 8;  // (a warp asks for N parts at a time)
  __shared__ int64_t sum_s[MW][2];
  __shared__ float acc_s[MW][D];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) D2F_TRACE_MARK(4, 8);
  const int pairs = a.num_heads_kv * a.chunks, fresh = a.k_new ? 1 : 0;
  const int b = blockIdx.x / a.num_heads_q, head = blockIdx.x % a.num_heads_q;
  const int in_group = head % a.group, hc = in_group / hq, h = in_group % hq;
  const int pair = head / a.group * a.chunks + hc;
  const int C = length_of(a, b, false), T = chunks_of(C, fresh);
  // the line's length, and the place of sequence b
  int64_t all = 0, before = 0;
  for (int i = tid; i < a.batch; i += kMergeThreads) {
    const int64_t x = (int64_t)chunks_of(length_of(a, i, false), fresh) * pairs;
    all += x;
    if (i < b) before += x;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) {
    sum_s[warp][0] = all;
    sum_s[warp][1] = before;
  }
  __syncthreads();
  all = before = 0;
#pragma unroll
  for (int i = 0; i < MW; ++i) {
    all += sum_s[i][0];
    before += sum_s[i][1];
  }
  // The parts. (Before any return: the grid behind this one relies on the one before it too.)
  if (tid == 0) D2F_TRACE_MARK(4, 9);
  grid_dependency_wait();
  if (tid == 0) D2F_TRACE_MARK(4, 10);
  if (T == 0) return;
  const Runs runs(all, warps);
  const int64_t first = before + (int64_t)pair * T, r0 = runs.of(first), r1 = runs.of(first + T - 1);
  if (r0 == r1) return;  // (written by its run)
  const int parts = (int)(r1 - r0) + 1, slot_heads = min(hq, a.group);
  // part i: run r0 + i, whose segment holds the pair's first chunk where i == 0
  auto slot_of = [&](int i) { return a.partial + (2 * (r0 + i) + (i == 0 ? 1 : 0)) * (slot_heads * (D + 4)); };
  auto ml_of = [&](int i) {
    return __ldcg(reinterpret_cast<const float2 *>(slot_of(i) + slot_heads * D + 2 * h));
  };
  // The outputs of this warp's first parts are asked for together with every part's (maximum, sum).
  float2 ml[N];
  float y[N][VL];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + k * MW;
      ml[k] = make_float2(kNothing, 0.f);
#pragma unroll
      for (int j = 0; j < VL; ++j) y[k][j] = 0.f;
      if (i < parts) {
        ml[k] = ml_of(i);
        const float *src = slot_of(i) + h * D + lane * VL;
        if constexpr (VL == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4 *>(src));
          y[k][0] = v.x, y[k][1] = v.y, y[k][2] = v.z, y[k][3] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2 *>(src));
          y[k][0] = v.x, y[k][1] = v.y;
        }
      }
    }
  };
  load(warp);
  // of the parts lane, lane + 32, ..: the running maximum and the sum beside it
  float mine = kNothing, sum = 0.f, acc[VL] = {};
  for (int i = lane; i < parts; i += 32) {
    const float2 x = ml_of(i);
    const float t = fmaxf(mine, x.x);
    sum = weight(mine, sum, t) * sum + weight(x.x, x.y, t) * x.y;
    mine = t;
  }
  float top = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  sum *= weight(mine, sum, top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  for (int i0 = warp; i0 < parts; i0 += MW * N) {
    if (i0 != warp) load(i0);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float w = weight(ml[k].x, ml[k].y, top);
#pragma unroll
      for (int j = 0; j < VL; ++j) acc[j] = fmaf(w, y[k][j], acc[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < VL; ++j) acc_s[warp][lane * VL + j] = acc[j];
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int k = 1; k < MW; ++k)
#pragma unroll
    for (int j = 0; j < VL; ++j) acc[j] += acc_s[k][lane * VL + j];
  const int64_t hr = (int64_t)b * a.num_heads_q + head;
  const bool none = sum == 0.f;  // no key, or every score is -inf
  const float inv = 1.0f / sum;
  uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + hr * D + lane * VL);
#pragma unroll
  for (int j = 0; j < VL / 2; ++j) dst[j] = none ? 0u : pack_bf16x2(acc[2 * j] * inv, acc[2 * j + 1] * inv);
  if (lane == 0 && a.lse_out) a.lse_out[hr] = none ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
  if (tid == 0) D2F_TRACE_MARK(4, 11);
}

// (a partial slot: an output of D floats a head, then (maximum, sum) a head, padded to 16 bytes)
template <int D, int NQ>
cudaError_t launch_t(const TokenArgs &a, cudaStream_t s) {
  using L = Cfg<D, NQ>;
  cudaError_t e = allow_smem_once<&token_tc_kernel<D, NQ>>(L::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  cfg.stream = s;
  cfg.gridDim = dim3((unsigned)a.grid);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  e = cudaLaunchKernelEx(&cfg, token_tc_kernel<D, NQ>, a);
  if (e != cudaSuccess || !a.line) return e;
  cfg.dynamicSmemBytes = 0;
  cfg.gridDim = dim3((unsigned)(a.batch * a.num_heads_q));
  cfg.blockDim = dim3(kMergeThreads);
  return cudaLaunchKernelEx(&cfg, token_merge_kernel<D>, a, a.grid * L::W, (int)L::HQ);
}

}  // namespace

cudaError_t launch_token_tc(const TokenArgs &a, cudaStream_t s) {
  if (a.head_dim == 128) return a.head_chunk == 8 ? launch_t<128, 1>(a, s) : launch_t<128, 2>(a, s);
  return a.head_chunk == 8 ? launch_t<64, 1>(a, s) : launch_t<64, 2>(a, s);
}

#ifdef D2F_TRACE
D2F_TRACE_COPY_FN(d2f_trace_copy_token)
#endif

}  // namespace d2f
