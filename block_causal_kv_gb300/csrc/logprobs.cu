// d2f_token_logprobs kernel: one streaming pass over the logits of every row that
// has a token: log probability of the token, entropy, and the k largest logits.
//
// Source: "확산 언어 모델(Diffusion LLM)이란 무엇인가", §토큰 순서의 이론 (largest
// probabilities and entropy of a position's prediction).
//
// With m = max l, S = sum exp(l - m), E = sum exp(l - m)(l - m):
//   log p_t = l_t - m - ln S,  H = ln S - E / S.
// Grid (slices, rows) as in the commit kernel: CTA (s, r) reduces vocabulary slice s
// of row r; the CTA that arrives last at a row's counter composes the slices. Bound
// by the logits' bytes; the arithmetic per logit (one exponential, five fused
// operations) stays under what the loads of an SM take.
//
// The k largest are kept per warp as a sorted list, lane i holding the i-th, of
// 64-bit keys that order by (logit descending, index ascending). A logit enters a
// warp's candidate buffer only if it reaches the warp's bound, the k-th largest
// known so far (first the k-th largest of the lanes' maxima, then the list's last
// entry, or another warp's if that is larger). Full buffers are sorted and merged
// 32 at a time, so the work behind the rare candidates is a few sorts a warp.
#include "d2f_internal.cuh"

namespace d2f {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr float kLog2e = 1.4426950408889634f;

// ---- ordered keys ------------------------------------------------------------
// Larger key = larger logit, or the same logit at a lower index. 0 is below every key.
__device__ __forceinline__ uint64_t make_key(float x, int idx) {
  uint32_t u = __float_as_uint(x + 0.0f);  // -0 and 0 are the same logit
  u = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
  return ((uint64_t)u << 32) | (uint32_t)~(uint32_t)idx;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ int key_index(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ uint64_t umax64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t umin64(uint64_t a, uint64_t b) { return a > b ? b : a; }

// Lanes hold a bitonic sequence: sort it descending.
__device__ __forceinline__ uint64_t bitonic_merge(uint64_t v, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    v = (lane & o) ? umin64(v, w) : umax64(v, w);
  }
  return v;
}
__device__ __forceinline__ uint64_t bitonic_sort(uint64_t v, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
      const bool desc = (lane & size) == 0 || size == 32;
      v = (((lane & o) == 0) == desc) ? umax64(v, w) : umin64(v, w);
    }
  }
  return v;
}
// The 32 largest of two descending lists, descending.
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - lane);
  return bitonic_merge(umax64(a, r), lane);
}

// ---- softmax terms -----------------------------------------------------------
struct Terms {
  float m, s, e;  // maximum, sum of exp(l - m), sum of exp(l - m)(l - m)
};

__device__ __forceinline__ Terms combine(const Terms &a, const Terms &b) {
  // a part without any finite term has s = 0 and e = 0; NaN sums stay NaN
  Terms r;
  r.m = fmaxf(a.m, b.m);
  const float da = a.m == r.m ? 0.f : fmaxf(a.m - r.m, -1e30f);
  const float db = b.m == r.m ? 0.f : fmaxf(b.m - r.m, -1e30f);
  const float wa = fast_exp2(da * kLog2e), wb = fast_exp2(db * kLog2e);
  r.s = a.s * wa + b.s * wb;
  r.e = wa * fmaf(da, a.s, a.e) + wb * fmaf(db, b.s, b.e);
  return r;
}

__device__ __forceinline__ Terms warp_combine(Terms v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Terms w;
    w.m = __shfl_xor_sync(0xffffffffu, v.m, o);
    w.s = __shfl_xor_sync(0xffffffffu, v.s, o);
    w.e = __shfl_xor_sync(0xffffffffu, v.e, o);
    v = combine(v, w);
  }
  return v;
}

template <int DT>
__device__ __forceinline__ void unpack(const uint4 raw, float (&x)[DT == D2F_BF16 ? 8 : 4]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  if constexpr (DT == D2F_BF16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(w[j]);
  }
}
template <int DT>
__device__ __forceinline__ float load_scalar(const void *base, int64_t i) {
  if constexpr (DT == D2F_BF16) return bf16_bits_to_float(((const uint16_t *)base)[i]);
  else return ((const float *)base)[i];
}

// Per-warp list of the largest keys and its candidate buffer (shared memory, 64 keys).
struct TopList {
  uint64_t key;    // lane i: i-th largest so far, 0 if none
  uint64_t bound;  // keys at or below it cannot enter (warp-uniform)
  float bound_x;   // logits below it cannot (warp-uniform)
  uint64_t *buf;
  int cnt;         // candidates in buf (warp-uniform)
  int k;

  __device__ __forceinline__ void init(uint64_t *b, int top) {
    key = 0;
    bound = 0;
    bound_x = -INFINITY;
    buf = b;
    cnt = 0;
    k = top;
  }
  __device__ __forceinline__ void flush(int lane) {
    const int take = min(cnt, 32);
    uint64_t v = lane < take ? buf[lane] : 0;
    v = bitonic_sort(v, lane);
    key = merge_lists(key, v, lane);
    const uint64_t rest = 32 + lane < cnt ? buf[32 + lane] : 0;
    __syncwarp();
    if (32 + lane < cnt) buf[lane] = rest;
    __syncwarp();
    cnt -= take;
    raise(__shfl_sync(0xffffffffu, key, k - 1));
  }
  __device__ __forceinline__ void raise(uint64_t b) {
    if (b > bound) {
      bound = b;
      bound_x = fmaxf(bound_x, key_value(b));
    }
  }
  // every lane offers one logit (warp-converged)
  __device__ __forceinline__ void offer(float x, int idx, bool on, int lane) {
    uint64_t c = 0;
    bool in = on && x >= bound_x;  // NaN never enters
    if (in) {
      c = make_key(x, idx);
      in = c > bound;
    }
    const unsigned who = __ballot_sync(0xffffffffu, in);
    if (!who) return;
    if (in) buf[cnt + __popc(who & ((1u << lane) - 1))] = c;
    cnt += __popc(who);
    __syncwarp();
    if (cnt >= 32) flush(lane);
  }
};

template <int DT, int PATH, bool TOP>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobsArgs a) {
  constexpr int VEC = PATH == 1 ? (DT == D2F_BF16 ? 8 : 4) : 1;
  __shared__ Terms terms_s[kWarps];
  __shared__ uint64_t buf_s[TOP ? kWarps * 64 : 1];
  __shared__ unsigned long long shared_bound;
  __shared__ int last_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.y, split = blockIdx.x;
  if (TOP && tid == 0) shared_bound = 0;
  grid_dependency_wait();
  const int tok = a.tokens[r];
  const int lr = a.logit_row ? a.logit_row[r] : r;
  const bool bad = tok >= a.vocab || (tok >= 0 && (lr < 0 || lr >= a.num_logit_rows));
  if (tok < 0 || bad) {  // no token here (or an index that is none): the row is not read
    if (split == 0) {
      if (tid == 0) {
        if (bad) set_err(a.err, D2F_ERR_BAD_INDEX);
        a.logprob[r] = 0.f;
        if (a.entropy) a.entropy[r] = 0.f;
      }
      for (int i = tid; i < a.top_k; i += kThreads) {
        a.top_id[(int64_t)r * a.top_k + i] = -1;
        a.top_logprob[(int64_t)r * a.top_k + i] = 0.f;
      }
    }
    return;
  }
  if (TOP) __syncthreads();  // shared_bound
  const int elt = DT == D2F_BF16 ? 2 : 4;
  const char *row = (const char *)a.logits + (int64_t)lr * a.row_stride * elt;
  const int v0 = split * a.chunk, v1 = min(a.vocab, v0 + a.chunk);

  float m = -INFINITY, e = 0.f, acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
  TopList top;
  if (TOP) top.init(buf_s + warp * 64, a.top_k);

  auto fold = [&](const float (&x)[VEC]) {
    float vm = x[0];
#pragma unroll
    for (int j = 1; j < VEC; ++j) vm = fmaxf(vm, x[j]);
    if (vm > m) {
      const float d = fmaxf(m - vm, -1e30f);
      const float w = fast_exp2(d * kLog2e);
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += acc[j];
      e = w * fmaf(d, s, e);
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] *= w;
      m = vm;
    }
    // a logit of -inf adds nothing (also while no finite one has come: m = -inf)
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float raw = x[j] - ref;
      const float d = raw < -1e30f ? -1e30f : raw;  // keeps NaN
      const float t = fast_exp2(d * kLog2e);
      acc[j] += t;
      e = fmaf(t, d, e);
    }
  };

  // ---- stream the slice --------------------------------------------------------
  constexpr int STEP = kThreads * VEC;       // logits of one vector per thread
  const int n_full = (v1 - v0) / VEC * VEC;  // whole vectors
  bool first = true;
  for (int base = v0; base < v0 + n_full; base += STEP * kUnroll) {  // CTA-uniform
    float x[kUnroll][VEC];
    bool on[kUnroll];
    if constexpr (PATH == 1) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = base + u * STEP + tid * VEC;
        on[u] = v < v0 + n_full;
        raw[u] = on[u] ? __ldcs(reinterpret_cast<const uint4 *>(row + (int64_t)v * elt))
                       : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) unpack<DT>(raw[u], x[u]);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = base + u * STEP + tid;
        on[u] = v < v0 + n_full;
        x[u][0] = on[u] ? load_scalar<DT>(row, v) : 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (on[u]) fold(x[u]);
    if (TOP) {
      if (first) {
        // first bound: the k-th largest of the lanes' maxima (at least k logits
        // reach it); a lane without logits, or without one that compares, has -inf
        const uint64_t lm = bitonic_sort(make_key(m, 0), lane);
        const float b = key_value(__shfl_sync(0xffffffffu, lm, top.k - 1));
        top.bound_x = fmaxf(top.bound_x, b);
      }
      first = false;
      top.raise(*(volatile unsigned long long *)&shared_bound);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float vm = -INFINITY;
#pragma unroll
        for (int j = 0; j < VEC; ++j) vm = fmaxf(vm, x[u][j]);
        if (!__any_sync(0xffffffffu, on[u] && vm >= top.bound_x)) continue;
        const uint64_t before = top.bound;
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          top.offer(x[u][j], base + u * STEP + tid * VEC + j, on[u], lane);
        if (top.bound > before && lane == 0)
          atomicMax(&shared_bound, (unsigned long long)top.bound);
      }
    }
  }
  {  // the slice's last elements, fewer than one vector
    const int v = v0 + n_full + tid;
    if (VEC > 1 && v0 + n_full < v1) {  // CTA-uniform
      const bool on = v < v1;
      const float x = on ? load_scalar<DT>(row, v) : 0.f;
      if (on) {
        float one[VEC];
        one[0] = x;
#pragma unroll
        for (int j = 1; j < VEC; ++j) one[j] = -INFINITY;
        fold(one);
      }
      if (TOP) top.offer(x, v, on, lane);
    }
  }

  // ---- reduce over the CTA -----------------------------------------------------
  Terms t;
  t.m = m;
  t.s = 0.f;
#pragma unroll
  for (int j = 0; j < VEC; ++j) t.s += acc[j];
  t.e = e;
  t = warp_combine(t);
  if (lane == 0) terms_s[warp] = t;
  if (TOP) {
    while (top.cnt > 0) top.flush(lane);
    __syncwarp();
    buf_s[warp * 64 + lane] = top.key;
  }
  __syncthreads();
  if (TOP) {
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) {
      if (warp < o) {
        top.key = merge_lists(top.key, buf_s[(warp + o) * 64 + lane], lane);
        buf_s[warp * 64 + lane] = top.key;
      }
      __syncthreads();
    }
  }
  if (warp == 0) {
    t = lane < kWarps ? terms_s[lane] : Terms{-INFINITY, 0.f, 0.f};
    t = warp_combine(t);
  }
  if (a.splits > 1) {
    const int64_t at = (int64_t)r * a.splits + split;
    if (warp == 0) {
      if (lane == 0) a.partial[at] = make_float4(t.m, t.s, t.e, 0.f);
      if (TOP && lane < a.top_k) a.top_part[at * a.top_k + lane] = top.key;
      __threadfence();
      __syncwarp();
      if (lane == 0) last_s = atomic_add_acq_rel(a.row_cnt + r, 1) == a.splits - 1;
    }
    __syncthreads();
    if (!last_s) return;
    // ---- the last CTA of the row composes the slices ----------------------------
    __threadfence();
    if (tid == 0) a.row_cnt[r] = 0;
    if (warp == 0) {
      t = Terms{-INFINITY, 0.f, 0.f};
      for (int s = lane; s < a.splits; s += 32) {
        const float4 p = __ldcg(a.partial + (int64_t)r * a.splits + s);
        t = combine(t, Terms{p.x, p.y, p.z});
      }
      t = warp_combine(t);
    }
    if (TOP) {
      uint64_t key = 0;
      for (int s = warp; s < a.splits; s += kWarps) {
        const uint64_t o = lane < a.top_k
            ? __ldcg((const unsigned long long *)a.top_part +
                     ((int64_t)r * a.splits + s) * a.top_k + lane) : 0;
        key = merge_lists(key, o, lane);
      }
      buf_s[warp * 64 + lane] = key;
      __syncthreads();
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        if (warp < o) {
          key = merge_lists(key, buf_s[(warp + o) * 64 + lane], lane);
          buf_s[warp * 64 + lane] = key;
        }
        __syncthreads();
      }
      top.key = key;
    }
  }
  if (warp == 0) {
    const float ln_s = logf(t.s);
    if (lane == 0) {
      a.logprob[r] = load_scalar<DT>(row, tok) - t.m - ln_s;
      if (a.entropy) a.entropy[r] = ln_s - t.e / t.s;
    }
    if (TOP && lane < a.top_k) {
      const bool have = top.key != 0;
      a.top_id[(int64_t)r * a.top_k + lane] = have ? key_index(top.key) : -1;
      a.top_logprob[(int64_t)r * a.top_k + lane] = have ? key_value(top.key) - t.m - ln_s : 0.f;
    }
  }
}

template <int DT, int PATH>
cudaError_t launch(const LogprobsArgs &a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.splits, a.n);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return a.top_k > 0 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, PATH, true>, a)
                     : cudaLaunchKernelEx(&cfg, logprobs_kernel<DT, PATH, false>, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsArgs &a, int dtype, int path, cudaStream_t s) {
  if (dtype == D2F_BF16)
    return path ? launch<D2F_BF16, 1>(a, s) : launch<D2F_BF16, 0>(a, s);
  return path ? launch<D2F_F32, 1>(a, s) : launch<D2F_F32, 0>(a, s);
}

}  // namespace d2f
