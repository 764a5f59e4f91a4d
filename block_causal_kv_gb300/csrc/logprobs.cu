// d2f_token_logprobs kernel: one streaming pass over the logits of every row that
// has a token: log probability of the token, entropy, and the k largest logits.
//
// Source: "확산 언어 모델(Diffusion LLM)이란 무엇인가", §토큰 순서의 이론 (largest
// probabilities and entropy of a position's prediction).
//
// With m = max l, s = sum exp(l - m) over all logits but one that is m, and
// E = sum exp(l - m)(l - m):
//   log p_t = l_t - m - ln(1 + s),  H = ln(1 + s) - E / (1 + s).
// The 1 stays out of the sum: where one token has nearly all the probability, its log
// probability is -s, which 1 + s would keep only to 2^-24 of 1.
// Grid (slices, rows) as in the commit kernel: CTA (s, r) reduces vocabulary slice s
// of row r; the CTA that arrives last at a row's counter composes the slices.
// Measured (in a CUDA graph, L2 flushed): 384 rows of 152,064 bf16 logits, half of them
// with a token, 20 alternatives: 31 us, 2.0 TB/s (22 us without alternatives); 48 rows of
// 126,464 and 5 alternatives 16 us (10 without). 1 to 16 rows take 7 us without
// alternatives, 12 with 5, 14 with 20 (float32 8, 12 and 13): one CTA's chain. The bytes
// alone would take 9 and 2 us; the rest is the chain of a CTA (stream, reduce, second look, compose), at
// about 60 % of the issue slots on the former. Keeping the maximum's 1 out of the sum is 3
// and 1 us of it; four vectors at a time (one by one: 41 and 18 us; with a reference of
// the whole warp, which moves less often: 35 and 18 us).
//
// The k largest logits of a slice come from a second look at few of its elements. In the
// pass every thread keeps the largest of its own logits and where it was. The k-th
// largest of the 256 threads' maxima bounds the k-th largest logit from below, and only
// the threads whose maximum reaches it (k of them) hold anything above it: a warp reads
// each such thread's elements once more, from L2, a vector per lane, and sorts the few
// that reach the bound. Everything is ordered by 64-bit keys (logit descending, index
// ascending), so ties and constant rows stay as cheap. (Filtering the stream against a
// running k-th largest instead cost 3 to 6 times the pass without alternatives: 74 us
// against 25 at k = 1 for 192 rows of 152,064 logits.)
#include "d2f_internal.cuh"

namespace d2f {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr float kLog2e = 1.4426950408889634f;
// Logits further below the maximum than this count as this far (their weight is 0 in any case):
// times 2^30 of them it still is a finite float, so that the weight makes the product 0.
constexpr float kFar = -1e28f;

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
  // maximum; sum of exp(l - m) but for one that is m (none yet: m = -inf); sum of
  // exp(l - m)(l - m)
  float m, s, e;
};

__device__ __forceinline__ Terms combine(const Terms &x, const Terms &y) {
  const bool first = x.m >= y.m;
  const Terms a = first ? x : y, b = first ? y : x;  // b's maximum becomes a logit like others
  const float bs = b.s + (b.m > -INFINITY ? 1.f : 0.f);
  const float d = b.m == a.m ? 0.f : fmaxf(b.m - a.m, kFar);
  const float w = fast_exp2(d * kLog2e);
  // a part without any finite term has s = 0 and e = 0; NaN sums stay NaN
  return Terms{a.m, fmaf(bs, w, a.s), fmaf(w, fmaf(d, bs, b.e), a.e)};
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
  uint64_t key = 0;  // lane i: i-th largest so far, 0 if none
  uint64_t bound;    // keys below it cannot enter (warp-uniform)
  uint64_t *buf;
  int cnt = 0;       // candidates in buf (warp-uniform)

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
  }
  // every lane offers one logit (warp-converged); NaN never enters
  __device__ __forceinline__ void offer(float x, int idx, bool on, int lane) {
    const uint64_t c = make_key(x, idx);
    const bool in = on && x == x && c >= bound;
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
  __shared__ uint64_t bound_s;
  __shared__ int last_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = blockIdx.y, split = blockIdx.x;
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
  const int elt = DT == D2F_BF16 ? 2 : 4;
  const char *row = (const char *)a.logits + (int64_t)lr * a.row_stride * elt;
  const int v0 = split * a.chunk, v1 = min(a.vocab, v0 + a.chunk);

  float m = -INFINITY, e = 0.f, acc[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
  int idx = 0;  // (TOP) where m is
  TopList top;

  // NV vectors at once, from v on every STEP: in a warp one of 32 maxima moves for most
  // vectors of a row, and so moves once for all of them.
  constexpr int STEP = kThreads * VEC;  // logits of one vector per thread
  auto fold = [&](auto &x, int v) {
    constexpr int NV = sizeof(x) / sizeof(x[0]);
    float vm = x[0][0];
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int j = 0; j < VEC; ++j) vm = fmaxf(vm, x[u][j]);
    if (vm > m) {
      // the old maximum joins the sums, the new one stays out of them
      const float w = fast_exp2(fmaxf(m - vm, kFar) * kLog2e);
      float s = m > -INFINITY ? 1.f : 0.f;
      const float old = s * w;
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += acc[j];
      e = w * fmaf(fmaxf(m - vm, kFar), s, e);
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] *= w;
      acc[0] += vm == INFINITY ? NAN : old;  // (infinity: the row's sums are NaN)
      m = vm;
      bool out = false;
#pragma unroll
      for (int u = 0; u < NV; ++u)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const bool here = !out && x[u][j] == vm;
          out = out || here;
          if (here) x[u][j] = -INFINITY;
          if (TOP && here) idx = v + u * STEP + j;
        }
    }
    // a logit of -inf adds nothing (also while no finite one has come: m = -inf)
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float raw = x[u][j] - ref;
        const float d = raw < kFar ? kFar : raw;  // keeps NaN
        const float t = fast_exp2(d * kLog2e);
        acc[j] += t;
        e = fmaf(t, d, e);
      }
  };

  // ---- stream the slice --------------------------------------------------------
  const int n_full = (v1 - v0) / VEC * VEC;  // whole vectors
  for (int base = v0; base < v0 + n_full; base += STEP * kUnroll) {  // CTA-uniform
    float x[kUnroll][VEC];
    if constexpr (PATH == 1) {
      constexpr uint32_t kNone = DT == D2F_BF16 ? 0xff80ff80u : 0xff800000u;  // -inf
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = base + u * STEP + tid * VEC;
        const uint4 *p = reinterpret_cast<const uint4 *>(row + (int64_t)v * elt);
        raw[u] = v < v0 + n_full ? (TOP ? __ldg(p) : __ldcs(p)) : make_uint4(kNone, kNone, kNone, kNone);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) unpack<DT>(raw[u], x[u]);
    } else {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = base + u * STEP + tid;
        x[u][0] = v < v0 + n_full ? load_scalar<DT>(row, v) : -INFINITY;
      }
    }
    fold(x, base + tid * VEC);
  }
  // the slice's last elements, fewer than one vector
  const int v_tail = v0 + n_full + tid;
  const bool tail_on = VEC > 1 && v_tail < v1;
  float x_tail = 0.f;
  if (tail_on) {
    x_tail = load_scalar<DT>(row, v_tail);
    float one[1][VEC];
    one[0][0] = x_tail;
#pragma unroll
    for (int j = 1; j < VEC; ++j) one[0][j] = -INFINITY;
    fold(one, v_tail);
  }

  // The CTA's 32 largest of every warp's descending list, in warp 0.
  auto cta_merge = [&](uint64_t key) -> uint64_t {
    __syncthreads();
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
    return key;
  };
  if constexpr (TOP) {
    // A thread without a logit above -inf offers the first of its -inf ones; one whose
    // logits are all NaN has nothing to offer (its key would count as one of the k).
    bool any = m > -INFINITY;
    if (!any) {
      for (int v = v0 + tid * VEC; v < v0 + n_full && !any; v += STEP)
        for (int j = 0; j < VEC && !any; ++j) {
          const float x = load_scalar<DT>(row, v + j);
          any = x == x;
          idx = v + j;
        }
      if (!any && tail_on) {
        any = x_tail == x_tail;
        idx = v_tail;
      }
    }
    const uint64_t mine = any ? make_key(m, idx) : 0;
    uint64_t key = cta_merge(bitonic_sort(mine, lane));
    if (tid == a.top_k - 1) bound_s = key;  // (top_k <= 32: a lane of warp 0)
    __syncthreads();
    top.bound = bound_s;  // 0: fewer than k threads have a logit
    top.buf = buf_s + warp * 64;
    unsigned who = __ballot_sync(0xffffffffu, mine != 0 && mine >= top.bound);
    __syncthreads();  // buf_s becomes the candidate buffers
    while (who) {
      const int owner = warp * 32 + __ffs(who) - 1;  // its vectors, one per lane
      who &= who - 1;
      for (int v = v0 + owner * VEC; v < v0 + n_full; v += STEP * 32) {
        const int at = v + lane * STEP;
        const bool on = at < v0 + n_full;
        float x[VEC];
        if constexpr (PATH == 1) {
          const uint4 raw = on ? __ldg(reinterpret_cast<const uint4 *>(row + (int64_t)at * elt))
                               : make_uint4(0, 0, 0, 0);
          unpack<DT>(raw, x);
        } else {
          x[0] = on ? load_scalar<DT>(row, at) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) top.offer(x[j], at + j, on, lane);
      }
    }
    if (warp == 0) top.offer(x_tail, v_tail, tail_on, lane);  // (VEC <= 32)
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
  if constexpr (TOP) {
    while (top.cnt > 0) top.flush(lane);
    top.key = cta_merge(top.key);
  }
  __syncthreads();
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
    if constexpr (TOP) {
      uint64_t key = 0;
      for (int s = warp; s < a.splits; s += kWarps) {
        const uint64_t o = lane < a.top_k
            ? __ldcg((const unsigned long long *)a.top_part +
                     ((int64_t)r * a.splits + s) * a.top_k + lane) : 0;
        key = merge_lists(key, o, lane);
      }
      top.key = cta_merge(key);
    }
  }
  if (warp == 0) {
    const float ln_s = log1pf(t.s);
    if (lane == 0) {  // (a row without a logit above -inf: -inf + inf)
      a.logprob[r] = load_scalar<DT>(row, tok) - t.m - ln_s;
      if (a.entropy) a.entropy[r] = t.m == -INFINITY ? NAN : ln_s - t.e / (1.f + t.s);
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
