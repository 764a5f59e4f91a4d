// CUDA-core path of d2f_token_attn: float32 operands, and the bf16 shapes that the
// tensor-core path does not take.
//
// Source of the computation: "D2F: 확산 언어 모델이 KV 캐시를 얻고 자기회귀 모델보다 2.5배
// 빨라지는 방법", §운영 관점 (paged cache, one block a page); "확산 언어 모델(Diffusion
// LLM)이란 무엇인가", §FlashBlock (attention parts recombined in log space).
//
// A CTA takes up to HC = 1, 2 or 4 query heads of a (sequence, KV head) and one split of its keys.
// Eight lanes hold a key: each reads D / 8 of its dims in 16-byte pieces, the dot products are
// summed over the eight, and every group of eight lanes keeps a softmax state (maximum, sum,
// output) of its own, so that a key costs three shuffles a head and nothing else crosses lanes
// until the end. The states of the CTA's groups are composed in log space, then those of
// the splits by the CTA that arrives last. Split 0 takes the new token's key too and, for the
// first chunk of heads, writes its K and V to their slot, which no CTA reads in this call.
//
// A CTA has as many heads as the group, up to four, so that K and V are read once for them. float32,
// D = 128: 16 x 4096 tokens of 32 heads 331 us, 6.5 TB/s (577 with room for four heads in every CTA
// and a key at a time); of 32 heads on 8 150 us, 3.6 TB/s (165 with one key
// at a time): two CTAs an SM, whose registers four heads fill, wait for their loads. Groups of five and
// more read K and V once for every four heads: 28 heads on 4 138 us, 1.9 TB/s of the cache's bytes, 5 on 1
// 48 us, 1.4. bf16 with head_dim 32: 4 x 32,768 tokens of 32 heads 308 us, 1.7 TB/s, 64 x 8192 of 28
// on 4 558, 0.5.
#include "attn_common.cuh"

namespace d2f {
namespace {

constexpr int kThreads = 128;
constexpr int kGroups = kThreads / 8;

// N elements (8 or 16 bytes) as floats
template <typename T, int N>
__device__ __forceinline__ void load_n(const T *p, float (&x)[N]) {
  if constexpr (sizeof(T) == 4) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    uint32_t w[N / 2];
    if constexpr (N == 8) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      w[0] = v.x;
      w[1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      x[2 * i] = bf16_bits_to_float(w[i] & 0xffffu);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename T, int D, int HC>
__global__ void __launch_bounds__(kThreads) token_simt_kernel(const TokenArgs a) {
  constexpr int VEC = (D / 8 < 16 / (int)sizeof(T)) ? D / 8 : 16 / (int)sizeof(T);
  constexpr int NJ = D / 8 / VEC;  // pieces of a lane: dims (8 j + lane) VEC ..
  __shared__ float o_s[kGroups][HC][D];
  __shared__ float m_s[kGroups][HC], l_s[kGroups][HC];
  __shared__ int is_last;
  const int tid = threadIdx.x, grp = tid >> 3, ln = tid & 7;
  int pair = blockIdx.x / a.num_splits;
  const int split = blockIdx.x % a.num_splits;
  const int chunk = pair % a.chunks, bg = pair / a.chunks;
  const int b = bg / a.num_heads_kv, g = bg % a.num_heads_kv;
  const int Hk = a.num_heads_kv, B = a.block_size;
  const int C = a.ctx_len[b];
  if (C < 0) return;  // no token here: nothing is read or written
  if ((long long)C > (long long)a.max_pages_per_seq * B) {
    if (tid == 0) set_err(a.err, D2F_ERR_INVALID_ARG);
    return;
  }
  const int h0 = chunk * HC, heads = min(HC, a.group - h0);
  const int32_t *table = a.page_table + (int64_t)b * a.max_pages_per_seq;
  const T *Kp = static_cast<const T *>(a.k_pool), *Vp = static_cast<const T *>(a.v_pool);

  if (split == 0 && a.k_new && chunk == 0) {
    const int page = C / B < a.max_pages_per_seq ? table[C / B] : -1;
    if (page < 0 || page >= a.num_pages) {
      if (tid == 0) set_err(a.err, D2F_ERR_BAD_INDEX);
    } else {
      const int64_t to = (((int64_t)page * Hk + g) * B + C % B) * D, from = ((int64_t)b * Hk + g) * D;
      for (int d = tid; d < D; d += kThreads) {
        static_cast<T *>(a.k_pool)[to + d] = static_cast<const T *>(a.k_new)[from + d];
        static_cast<T *>(a.v_pool)[to + d] = static_cast<const T *>(a.v_new)[from + d];
      }
    }
  }

  float q[HC][NJ][VEC], o[HC][NJ][VEC], m[HC], l[HC];
#pragma unroll
  for (int h = 0; h < HC; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int c = 0; c < VEC; ++c) q[h][j][c] = o[h][j][c] = 0.f;
      if (h < heads)
        load_n<T, VEC>(static_cast<const T *>(a.q) +
                       ((int64_t)b * a.num_heads_q + g * a.group + h0 + h) * D + (8 * j + ln) * VEC,
                       q[h][j]);
#pragma unroll
      for (int c = 0; c < VEC; ++c) q[h][j][c] *= a.scale_log2;
    }
  }
  auto load = [&](const T *kp, const T *vp, float (&kx)[NJ][VEC], float (&vx)[NJ][VEC]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) load_n<T, VEC>(kp + (8 * j + ln) * VEC, kx[j]);
#pragma unroll
    for (int j = 0; j < NJ; ++j) load_n<T, VEC>(vp + (8 * j + ln) * VEC, vx[j]);
  };
  auto key = [&](const float (&kx)[NJ][VEC], const float (&vx)[NJ][VEC]) {
    const uint32_t mine = 0xffu << (tid & 24);  // the eight lanes of this key
#pragma unroll
    for (int h = 0; h < HC; ++h) {
      float x = 0.f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int c = 0; c < VEC; ++c) x = fmaf(q[h][j][c], kx[j][c], x);
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) x += __shfl_xor_sync(mine, x, off);
      const float m_new = fmaxf(m[h], x);
      const float base = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = fast_exp2(m[h] - base), p = fast_exp2(x - base);
      m[h] = m_new;
      l[h] = fmaf(l[h], alpha, p);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int c = 0; c < VEC; ++c) o[h][j][c] = fmaf(p, vx[j][c], o[h][j][c] * alpha);
    }
  };
  const int share = (C + a.num_splits - 1) / a.num_splits;
  const int begin = min(C, split * share), end = min(C, begin + share);
  // U keys at a time: their loads go out together. (Two heads: 235 us with two keys, 204 with four, 16 x
  // 4096 tokens of 32 heads on 16; one head 336 and 388, four heads 143 and, with three, 157.)
  constexpr int U = HC == 2 ? 4 : 2;
  int page[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int n = begin + grp + i * kGroups;
    page[i] = n < end ? table[n / B] : 0;
  }
  for (int t = begin + grp; t < end; t += U * kGroups) {
    int next[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int n = t + (U + i) * kGroups;
      next[i] = n < end ? table[n / B] : 0;
    }
    float kx[U][NJ][VEC], vx[U][NJ][VEC];
    bool ok[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int n = t + i * kGroups;
      ok[i] = n < end && page[i] >= 0 && page[i] < a.num_pages;
      if (n < end && !ok[i]) set_err(a.err, D2F_ERR_BAD_INDEX);
      if (ok[i]) {
        const int64_t at = (((int64_t)page[i] * Hk + g) * B + n % B) * D;
        load(Kp + at, Vp + at, kx[i], vx[i]);
      }
      page[i] = next[i];
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (ok[i]) key(kx[i], vx[i]);
  }
  if (split == 0 && grp == 0 && a.k_new) {
    const int64_t at = ((int64_t)b * Hk + g) * D;
    float kx[NJ][VEC], vx[NJ][VEC];
    load(static_cast<const T *>(a.k_new) + at, static_cast<const T *>(a.v_new) + at, kx, vx);
    key(kx, vx);
  }

  // ---- the CTA's groups, then the splits ----
#pragma unroll
  for (int h = 0; h < HC; ++h) {
    if (ln == 0) {
      m_s[grp][h] = m[h];
      l_s[grp][h] = l[h];
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int c = 0; c < VEC; ++c) o_s[grp][h][(8 * j + ln) * VEC + c] = o[h][j][c];
  }
  __syncthreads();
  // weight of a part whose maximum is x among parts with the maximum top (a part without keys: 0;
  // one whose scores are all NaN keeps its NaN sum)
  auto weight = [](float x, float top) { return x == -INFINITY ? (top == -INFINITY ? 1.f : 0.f)
                                                                : fast_exp2(x - top); };
  // partials: [pair][split][HC][D] outputs, then [pair][split][HC] (maximum, sum)
  const int64_t pairs = (int64_t)a.batch * Hk * a.chunks;
  float2 *ml = reinterpret_cast<float2 *>(a.partial + pairs * a.num_splits * HC * D);
  for (int e = tid; e < heads * D; e += kThreads) {
    const int h = e / D, d = e % D;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
    for (int i = 0; i < kGroups; ++i) top = fmaxf(top, m_s[i][h]);
    for (int i = 0; i < kGroups; ++i) {
      const float w = weight(m_s[i][h], top);
      sum = fmaf(w, l_s[i][h], sum);
      acc = fmaf(w, o_s[i][h][d], acc);
    }
    if (a.num_splits > 1) {
      const int64_t at = ((int64_t)pair * a.num_splits + split) * HC + h;
      a.partial[at * D + d] = acc;
      if (d == 0) ml[at] = make_float2(top, sum);
    } else {
      const int64_t hr = (int64_t)b * a.num_heads_q + g * a.group + h0 + h;
      const bool none = sum == 0.f;  // no key, or every score is -inf
      store_out<T>(static_cast<T *>(a.out) + hr * D + d, none ? 0.f : acc / sum);
      if (d == 0 && a.lse_out) a.lse_out[hr] = (top + __log2f(sum)) * 0.6931471805599453f;
    }
  }
  if (a.num_splits == 1) return;
  __threadfence();
  __syncthreads();
  if (tid == 0) is_last = atomic_add_acq_rel(a.counters + pair, 1) == a.num_splits - 1;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  for (int e = tid; e < heads * D; e += kThreads) {
    const int h = e / D, d = e % D;
    const int64_t at = (int64_t)pair * a.num_splits * HC + h;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
    for (int i = 0; i < a.num_splits; ++i) top = fmaxf(top, __ldcg(&ml[at + (int64_t)i * HC]).x);
    for (int i = 0; i < a.num_splits; ++i) {
      const float2 x = __ldcg(&ml[at + (int64_t)i * HC]);
      const float w = weight(x.x, top);
      sum = fmaf(w, x.y, sum);
      acc = fmaf(w, __ldcg(a.partial + (at + (int64_t)i * HC) * D + d), acc);
    }
    const int64_t hr = (int64_t)b * a.num_heads_q + g * a.group + h0 + h;
    const bool none = sum == 0.f;  // no key, or every score is -inf
    store_out<T>(static_cast<T *>(a.out) + hr * D + d, none ? 0.f : acc / sum);
    if (d == 0 && a.lse_out) a.lse_out[hr] = (top + __log2f(sum)) * 0.6931471805599453f;
  }
  if (tid == 0) a.counters[pair] = 0;
}

template <typename T, int D>
cudaError_t launch_d(const TokenArgs &a, cudaStream_t s) {
  const int64_t ctas = (int64_t)a.batch * a.num_heads_kv * a.chunks * a.num_splits;
  if (a.head_chunk == 1) token_simt_kernel<T, D, 1><<<(unsigned)ctas, kThreads, 0, s>>>(a);
  else if (a.head_chunk == 2) token_simt_kernel<T, D, 2><<<(unsigned)ctas, kThreads, 0, s>>>(a);
  else token_simt_kernel<T, D, 4><<<(unsigned)ctas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_t(const TokenArgs &a, cudaStream_t s) {
  switch (a.head_dim) {
    case 32: return launch_d<T, 32>(a, s);
    case 64: return launch_d<T, 64>(a, s);
    case 128: return launch_d<T, 128>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_token_simt(const TokenArgs &a, int dtype, cudaStream_t s) {
  return dtype == D2F_BF16 ? launch_t<uint16_t>(a, s) : launch_t<float>(a, s);
}

}  // namespace d2f
