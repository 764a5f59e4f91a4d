// Tensor-core path of d2f_token_attn: bf16, head_dim 64 or 128.
//
// Source of the computation: "D2F: 확산 언어 모델이 KV 캐시를 얻고 자기회귀 모델보다 2.5배
// 빨라지는 방법", §운영 관점 (paged cache, one block a page); "확산 언어 모델(Diffusion
// LLM)이란 무엇인가", §FlashBlock (attention parts recombined in log space).
//
// A read of the cache bounds it: every K and V element is used for the G query heads of its group
// and no more. So the products take the small tensor instructions (mma.sync m16n8k16), whose
// operands are registers, and K and V go from memory to registers and nowhere else:
//   S^T [16 keys x 8 heads] = K [16 keys x D] Q^T,  O^T [D x 8 heads] += V^T [D x 16 keys] P^T.
// The sums over D and over keys may run in any order, so a thread's operand elements are chosen
// for its loads: 16 bytes (8 dims) of K of two keys per 32 dims, and 16 bytes of V of four keys
// per 64 dims, whose pairs of keys are put together by byte permutes. P^T's layout comes from
// S^T's by 8 x 8 transposes in registers.
//
// A warp takes 16 keys at a time: V of these keys is requested before S is computed, K of the next
// ones right after, so a warp always has 4 to 8 KB on the way. 12 warps a CTA (16 with
// head_dim 64, 8 with more than eight heads a group), a CTA an SM.
//
// All chunks of 16 keys of the launch, (sequence, KV head, 16 heads, chunk), are one line cut into
// equal shares, one CTA a share: every SM reads the same number of bytes whatever the lengths.
// The warps of a CTA compose their parts of a (sequence, KV head) in shared memory; where it lies
// in several shares, the CTA that arrives last composes the parts from the workspace, in the
// order of the line. The arrival counter is that of the share with the first chunk: a share cuts
// off one at its end at most. No CTA waits on another.
//
// Softmax in log2 units with a reference a head and warp, which moves only when a score is more
// than 2^8 above it. Weights enter the product with V as bf16 (2^-8 of each; the sum keeps the
// unrounded ones); scores, sums and outputs are float.
#include "attn_common.cuh"

namespace d2f {
namespace {

constexpr uint32_t kNoKey = 0xffffffffu;   // row of a key that does not exist
constexpr uint32_t kNewKey = 0xfffffffeu;  // the new token's
constexpr float kMove = 8.f;
constexpr float kNothing = -1e30f;         // reference of a head that has seen no key
constexpr int kMaxGrid = kTokenMaxGrid;
constexpr int kMinChunks = 8;              // chunks of a share at least

// Pages hold fewer than 2^32 - 2 token rows of a head (128 bytes or more each).
__device__ __forceinline__ uint4 load_row(const void *pool, const void *fresh, uint32_t row, int row_bytes,
                                          int at) {
  const char *p = row == kNewKey ? static_cast<const char *>(fresh)
                                 : static_cast<const char *>(pool) + (int64_t)row * row_bytes;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (row != kNoKey)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p + at));
  return v;
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
  static constexpr int W = NQ == 2 ? 8 : D == 64 ? 16 : 12;  // warps: what the registers allow
  static constexpr int kThreads = 32 * W;
  static constexpr int HQ = 8 * NQ;            // heads of a CTA
  static constexpr int kPitch = D + 4;
  // shared memory: the warps' outputs (later the weights of a composition's parts and its
  // reduction), then their (maximum, sum), then the sequences
  static constexpr int kO = 0;
  static constexpr int kRed = kMaxGrid * HQ * 8;
  static constexpr int kMl = kO + (W * HQ * kPitch * 4 > kRed + kThreads * 16 ? W * HQ * kPitch * 4
                                                                             : kRed + kThreads * 16);
  static constexpr int kPre = kMl + W * HQ * 8;
  static constexpr int kCtx = kPre + (kTokenScanBatch + 1) * 8;
  static constexpr int kBytes = kCtx + kTokenScanBatch * 4;
};

struct Seg {       // chunks u0 .. u1 - 1 of the T of a (sequence, KV head, head chunk)
  int b, g, hc, C, u0, u1, T;
  int64_t first;   // place of chunk 0 on the line
  bool ok;
};

template <int D, int NQ>
__global__ void __launch_bounds__(Cfg<D, NQ>::kThreads, 1) token_tc_kernel(const TokenArgs a) {
  using L = Cfg<D, NQ>;
  constexpr int W = L::W, HQ = L::HQ, NT = L::kThreads, KB = D / 32, VB = D / 64;
  extern __shared__ __align__(16) uint8_t sm[];
  float *o_s = reinterpret_cast<float *>(sm + L::kO);
  float2 *ml_s = reinterpret_cast<float2 *>(sm + L::kMl);
  int64_t *pre_s = reinterpret_cast<int64_t *>(sm + L::kPre);
  int *ctx_s = reinterpret_cast<int *>(sm + L::kCtx);
  __shared__ int is_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  const int Hk = a.num_heads_kv, B = a.block_size, fresh = a.k_new ? 1 : 0;
  const int heads_b = Hk * a.chunks;  // (KV head, head chunk) pairs of a sequence
  const bool line = a.batch <= kTokenScanBatch;
  auto chunks_of = [&](int C) -> int { return C < 0 ? 0 : max(1, (C + fresh + 15) / 16); };
  // the length of a sequence: negative where it takes no part
  auto length = [&](int b, bool report) -> int {
    const int C = __ldg(a.ctx_len + b);
    if ((long long)C > (long long)a.max_pages_per_seq * B) {
      if (report) set_err(a.err, D2F_ERR_INVALID_ARG);
      return -1;
    }
    return C;
  };

  Seg s;
  int64_t total = 0, grid = gridDim.x, end = 0;  // places on the line; this share ends at `end`
  if (line) {
    for (int b = tid; b < a.batch; b += NT) ctx_s[b] = length(b, blockIdx.x == 0);
    __syncthreads();
    if (warp == 0) {
      int64_t carry = 0;
      for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        int64_t x = b < a.batch ? (int64_t)chunks_of(ctx_s[b]) * heads_b : 0, sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        if (b < a.batch) pre_s[b] = carry + sum - x;
        carry += __shfl_sync(0xffffffffu, sum, 31);
      }
      if (lane == 0) pre_s[a.batch] = carry;
    }
    __syncthreads();
    total = pre_s[a.batch];
    grid = max((int64_t)1, min(grid, (total + kMinChunks - 1) / kMinChunks));
    if (total == 0 || blockIdx.x >= grid) return;
    const int64_t at = blockIdx.x * total / grid;
    end = (blockIdx.x + 1) * total / grid;
    int lo = 0, hi = a.batch;  // pre_s[lo] <= at < pre_s[hi], lo the last such
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre_s[mid] <= at) lo = mid;
      else hi = mid;
    }
    s.b = lo;
    s.C = ctx_s[lo];
    s.T = chunks_of(s.C);
    const int64_t in = at - pre_s[lo];
    const int pair = (int)(in / s.T);
    s.g = pair / a.chunks;
    s.hc = pair % a.chunks;
    s.u0 = (int)(in - (int64_t)pair * s.T);
    s.first = at - s.u0;
    s.u1 = (int)min((int64_t)s.T, end - s.first);
    s.ok = true;
  } else {  // a (sequence, KV head, head chunk) a CTA
    s.b = blockIdx.x / heads_b;
    const int pair = blockIdx.x % heads_b;
    s.g = pair / a.chunks;
    s.hc = pair % a.chunks;
    s.C = length(s.b, tid == 0);
    s.T = chunks_of(s.C);
    if (s.T == 0) return;
    s.u0 = 0;
    s.u1 = s.T;
    s.first = 0;
    s.ok = true;
  }
  auto next_seg = [&](const Seg &p) -> Seg {
    Seg n = p;
    n.first = p.first + p.T;
    n.ok = line && n.first < end;
    if (!n.ok) return n;
    if (++n.hc == a.chunks) {
      n.hc = 0;
      if (++n.g == Hk) {
        n.g = 0;
        do ++n.b;
        while (ctx_s[n.b] < 0);  // (a sequence with chunks follows: first < end)
        n.C = ctx_s[n.b];
        n.T = chunks_of(n.C);
      }
    }
    n.u0 = 0;
    n.u1 = (int)min((int64_t)n.T, end - n.first);
    return n;
  };
  // page id of this lane's key of chunk u (lanes 16 .. 31: as lanes 0 .. 15), then its token row
  auto page_of = [&](const Seg &p, int u) -> int {
    const int key = 16 * u + (lane & 15);
    return u < p.u1 && key < p.C ? __ldg(a.page_table + (int64_t)p.b * a.max_pages_per_seq + key / B) : 0;
  };
  auto row_of = [&](const Seg &p, int u, int page) -> uint32_t {
    const int key = 16 * u + (lane & 15);
    if (key >= p.C) return key == p.C && fresh ? kNewKey : kNoKey;
    if (page < 0 || page >= a.num_pages) {
      set_err(a.err, D2F_ERR_BAD_INDEX);
      return kNoKey;
    }
    return (uint32_t)(((int64_t)page * Hk + p.g) * B + key % B);
  };

  uint4 q[NQ][KB], kx[2][KB], vx[4][VB];
  uint32_t k_ok = 0;  // bits 0, 1: keys r and r + 8 of the loaded K exist
  auto load_q = [&](const Seg &p) {
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int h = p.hc * HQ + n * 8 + r;  // head of the group
      const char *src = static_cast<const char *>(a.q) +
                        ((int64_t)p.b * a.num_heads_q + p.g * a.group + h) * (D * 2) + c * 16;
#pragma unroll
      for (int k = 0; k < KB; ++k)
        q[n][k] = h < a.group ? __ldg(reinterpret_cast<const uint4 *>(src + k * 64)) : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_k = [&](const Seg &p, uint32_t row) {
    const void *fr = static_cast<const char *>(a.k_new) + ((int64_t)p.b * Hk + p.g) * (D * 2);
    k_ok = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = __shfl_sync(0xffffffffu, row, r + 8 * i);
      if (x != kNoKey) k_ok |= 1u << i;
#pragma unroll
      for (int k = 0; k < KB; ++k) kx[i][k] = load_row(a.k_pool, fr, x, D * 2, k * 64 + c * 16);
    }
  };

  uint32_t row = kNoKey;
  int page = page_of(s, s.u0 + warp), page_next = 0;
  load_q(s);
  if (s.u0 + warp < s.u1) {
    row = row_of(s, s.u0 + warp, page);
    load_k(s, row);
    page_next = page_of(s, s.u0 + warp + W);
  }
  while (true) {
    const Seg n = next_seg(s);
    const bool n_mine = n.ok && n.u0 + warp < n.u1;
    page = n_mine ? page_of(n, n.u0 + warp) : 0;
    auto enter_next = [&] {  // the next segment's first loads
      load_q(n);
      row = row_of(n, n.u0 + warp, page);
      load_k(n, row);
      page_next = page_of(n, n.u0 + warp + W);
    };
    float m[NQ][2], l[NQ][2], o[NQ][VB][4][4];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      m[i][0] = m[i][1] = kNothing;
      l[i][0] = l[i][1] = 0.f;
#pragma unroll
      for (int j = 0; j < VB; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[i][j][w][x] = 0.f;
    }
    for (int u = s.u0 + warp; u < s.u1; u += W) {
      const void *fv = static_cast<const char *>(a.v_new) + ((int64_t)s.b * Hk + s.g) * (D * 2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x = __shfl_sync(0xffffffffu, row, 2 * c + (i & 1) + 8 * (i >> 1));
#pragma unroll
        for (int j = 0; j < VB; ++j) vx[i][j] = load_row(a.v_pool, fv, x, D * 2, j * 128 + r * 16);
      }
      if (fresh && s.hc == 0 && s.C >= 16 * u && s.C < 16 * u + 16) {
        // the new token to its slot, which no CTA reads in this call
        const int pg = s.C / B < a.max_pages_per_seq
                           ? __ldg(a.page_table + (int64_t)s.b * a.max_pages_per_seq + s.C / B) : -1;
        if (pg < 0 || pg >= a.num_pages) {
          if (lane == 0) set_err(a.err, D2F_ERR_BAD_INDEX);
        } else if ((lane & 15) < D / 8) {
          const int64_t from = ((int64_t)s.b * Hk + s.g) * (D / 8) + (lane & 15);
          const int64_t to = (((int64_t)pg * Hk + s.g) * B + s.C % B) * (D / 8) + (lane & 15);
          if (lane < 16)
            static_cast<uint4 *>(a.k_pool)[to] = static_cast<const uint4 *>(a.k_new)[from];
          else
            static_cast<uint4 *>(a.v_pool)[to] = static_cast<const uint4 *>(a.v_new)[from];
        }
      }
      float x[NQ][4];
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          mma_bf16(x[i], kx[0][k].x, kx[1][k].x, kx[0][k].y, kx[1][k].y, q[i][k].x, q[i][k].y);
          mma_bf16(x[i], kx[0][k].z, kx[1][k].z, kx[0][k].w, kx[1][k].w, q[i][k].z, q[i][k].w);
        }
      }
      const uint32_t ok = k_ok;
      if (u + W < s.u1) {
        row = row_of(s, u + W, page_next);
        load_k(s, row);
        page_next = page_of(s, u + 2 * W);
      } else if (n_mine) {
        enter_next();
      }
      uint32_t p[NQ][2];
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        bool move = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[i][e] = (ok >> (e >> 1) & 1u) ? x[i][e] * a.scale_log2 : -INFINITY;
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
        const uint32_t v[4][4] = {{vx[0][j].x, vx[0][j].y, vx[0][j].z, vx[0][j].w},
                                  {vx[1][j].x, vx[1][j].y, vx[1][j].z, vx[1][j].w},
                                  {vx[2][j].x, vx[2][j].y, vx[2][j].z, vx[2][j].w},
                                  {vx[3][j].x, vx[3][j].y, vx[3][j].z, vx[3][j].w}};
#pragma unroll
        for (int w = 0; w < 4; ++w) {  // dims 64 j + 8 r + 2 w and + 1
          const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5410), a1 = __byte_perm(v[0][w], v[1][w], 0x7632);
          const uint32_t a2 = __byte_perm(v[2][w], v[3][w], 0x5410), a3 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
          for (int i = 0; i < NQ; ++i) mma_bf16(o[i][j][w], a0, a1, a2, a3, p[i][0], p[i][1]);
        }
      }
    }
    if (n_mine && s.u0 + warp >= s.u1) enter_next();

    // ---- the warps' parts of this segment ----
    const int parts_w = min(W, s.u1 - s.u0);
    const int heads = min(HQ, a.group - s.hc * HQ);
    if (warp < parts_w) {
#pragma unroll
      for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[i][e];
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          const int h = 8 * i + 2 * c + e;
          if (r == 0) ml_s[warp * HQ + h] = make_float2(m[i][e], sum);
          if (h < heads) {
            float *dst = o_s + (warp * HQ + h) * L::kPitch + 8 * r;
#pragma unroll
            for (int j = 0; j < VB; ++j) {
              *reinterpret_cast<float4 *>(dst + 64 * j) =
                  make_float4(o[i][j][0][e], o[i][j][0][e + 2], o[i][j][1][e], o[i][j][1][e + 2]);
              *reinterpret_cast<float4 *>(dst + 64 * j + 4) =
                  make_float4(o[i][j][2][e], o[i][j][2][e + 2], o[i][j][3][e], o[i][j][3][e + 2]);
            }
          }
        }
    }
    __syncthreads();
    const bool whole = s.u0 == 0 && s.u1 == s.T;
    const int64_t hr0 = (int64_t)s.b * a.num_heads_q + s.g * a.group + s.hc * HQ;
    auto put = [&](int h, int d, float4 v, float top, float sum) {  // four outputs and, once, the lse
      const bool none = top == kNothing && sum == 0.f;  // no key
      const float inv = none ? 0.f : 1.0f / sum;
      uint2 y;
      y.x = none ? 0u : pack_bf16x2(v.x * inv, v.y * inv);
      y.y = none ? 0u : pack_bf16x2(v.z * inv, v.w * inv);
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + (hr0 + h) * D + d) = y;
      if (d == 0 && a.lse_out)
        a.lse_out[hr0 + h] = none ? -INFINITY : (top + __log2f(sum)) * 0.6931471805599453f;
    };
    // partial slots: (maximum, sum) [HQ], outputs [HQ][D]; two a CTA
    constexpr int kSlot = HQ * (D + 2);
    float *slots = a.partial;
    float *slot = slots + (2 * (int64_t)blockIdx.x + (s.u0 == 0 ? 1 : 0)) * kSlot;
    for (int e = tid; e < heads * (D / 4); e += NT) {
      const int h = e / (D / 4), d = (e % (D / 4)) * 4;
      float top = kNothing, sum = 0.f;
      for (int w = 0; w < parts_w; ++w) top = fmaxf(top, ml_s[w * HQ + h].x);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < parts_w; ++w) {
        const float2 x = ml_s[w * HQ + h];
        // (a part whose scores are all NaN has a NaN sum and no maximum)
        const float wt = x.x == kNothing && x.y == 0.f ? 0.f : fast_exp2(x.x - top);
        const float4 y = *reinterpret_cast<float4 *>(o_s + (w * HQ + h) * L::kPitch + d);
        sum = fmaf(wt, x.y, sum);
        acc.x = fmaf(wt, y.x, acc.x);
        acc.y = fmaf(wt, y.y, acc.y);
        acc.z = fmaf(wt, y.z, acc.z);
        acc.w = fmaf(wt, y.w, acc.w);
      }
      if (whole) {
        put(h, d, acc, top, sum);
      } else {
        *reinterpret_cast<float4 *>(slot + 2 * HQ + h * D + d) = acc;
        if (d == 0) reinterpret_cast<float2 *>(slot)[h] = make_float2(top, sum);
      }
    }
    if (!whole) {
      // shares that hold chunks of this pair: c0 .. c1, c0 with the first chunk
      const int64_t c0 = ((s.first + 1) * grid - 1) / total, c1 = ((s.first + s.T) * grid - 1) / total;
      const int parts = (int)(c1 - c0) + 1;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        is_last = atomic_add_acq_rel(a.counters + c0, 1) == parts - 1;
        if (is_last) a.counters[c0] = 0;
      }
      __syncthreads();
      if (is_last) {
        __threadfence();
        // weights of the parts, in shared memory over the warps' outputs
        float2 *wt = reinterpret_cast<float2 *>(o_s);  // [parts][HQ]
        auto slot_of = [&](int i) { return slots + (2 * (c0 + i) + (i == 0 ? 1 : 0)) * kSlot; };
        for (int e = tid; e < parts * heads; e += NT) {
          const int i = e / heads, h = e - i * heads;
          wt[i * HQ + h] = __ldcg(reinterpret_cast<const float2 *>(slot_of(i)) + h);
        }
        __syncthreads();
        for (int h = warp; h < heads; h += W) {
          float top = kNothing, sum = 0.f;
          for (int i = lane; i < parts; i += 32) top = fmaxf(top, wt[i * HQ + h].x);
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          for (int i = lane; i < parts; i += 32) {
            const float2 x = wt[i * HQ + h];
            const float y = x.x == kNothing && x.y == 0.f ? 0.f : fast_exp2(x.x - top);
            sum = fmaf(y, x.y, sum);
            wt[i * HQ + h].x = y;
          }
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          __syncwarp();
          if (lane == 0) ml_s[h] = make_float2(top, sum);
        }
        __syncthreads();
        // each output by `groups` threads, a share of the parts each
        const int outs = heads * (D / 4), groups = max(1, NT / outs);
        float4 *red = reinterpret_cast<float4 *>(sm + L::kRed);
        for (int e0 = 0; e0 < outs; e0 += NT) {
          const int e = e0 + (groups > 1 ? tid % outs : tid), gi = groups > 1 ? tid / outs : 0;
          const int h = e / (D / 4), d = (e % (D / 4)) * 4;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          if (e < outs && gi < groups) {
#pragma unroll 8
            for (int i = gi; i < parts; i += groups) {
              const float y = wt[i * HQ + h].x;
              const float4 x = __ldcg(reinterpret_cast<const float4 *>(slot_of(i) + 2 * HQ + h * D + d));
              acc.x = fmaf(y, x.x, acc.x);
              acc.y = fmaf(y, x.y, acc.y);
              acc.z = fmaf(y, x.z, acc.z);
              acc.w = fmaf(y, x.w, acc.w);
            }
          }
          if (groups > 1) {
            red[tid] = acc;
            __syncthreads();
            if (tid < outs) {
              for (int k = 1; k < groups; ++k) {
                const float4 x = red[k * outs + tid];
                acc.x += x.x;
                acc.y += x.y;
                acc.z += x.z;
                acc.w += x.w;
              }
              put(h, d, acc, ml_s[h].x, ml_s[h].y);
            }
          } else if (e < outs) {
            put(h, d, acc, ml_s[h].x, ml_s[h].y);
          }
        }
      }
    }
    if (!n.ok) break;
    __syncthreads();  // the shared arrays are free for the next segment
    s = n;
  }
}

template <int D, int NQ>
cudaError_t launch_t(const TokenArgs &a, cudaStream_t s) {
  using L = Cfg<D, NQ>;
  // (per device; every call sets the same value)
  const cudaError_t e = cudaFuncSetAttribute(token_tc_kernel<D, NQ>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  const int64_t pairs = (int64_t)a.batch * a.num_heads_kv * a.chunks;
  const unsigned grid = a.batch <= kTokenScanBatch ? (unsigned)a.grid : (unsigned)pairs;
  token_tc_kernel<D, NQ><<<grid, L::kThreads, L::kBytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_token_tc(const TokenArgs &a, cudaStream_t s) {
  if (a.head_dim == 128) return a.head_chunk == 8 ? launch_t<128, 1>(a, s) : launch_t<128, 2>(a, s);
  return a.head_chunk == 8 ? launch_t<64, 1>(a, s) : launch_t<64, 2>(a, s);
}

}  // namespace d2f
