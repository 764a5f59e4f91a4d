// CUDA-core path of d2f_prompt_attn: float32 operands, and the bf16 shapes that the
// tensor-core path does not take. The composition of key splits, for both paths, is here too.
//
// Source of the mask: "D2F: 확산 언어 모델이 KV 캐시를 얻고 자기회귀 모델보다 2.5배 빨라지는
// 방법", §블록 단위 인과 어텐션 (bidirectional inside a block, causal between blocks; a block
// of one row is the causal mask, one block of all rows the bidirectional one).
//
// A CTA holds R packed rows (row r = query r / head_chunk, head r % head_chunk) of
// one KV head and walks their key tiles of KT keys, the cached prefix first: S = Q K^T with R / 16
// rows and four keys a thread, the online softmax in log2 units over the 16 threads of a row, P
// through shared memory (over K, which is done with), O += P V with R / 16 rows and D / 16 columns a
// thread. Multiply-adds are made in pairs, which halves their issue (4096 causal rows of 32 heads on 8,
// D = 128, float32: 3440 -> 3166 us, 43 TFLOP/s); shared memory's reads bound it, eight 16-byte loads
// for 32 pairs. Operands are float in shared memory; rows are padded by four floats so that 16 keys a
// quarter apart fall on different banks. bf16 shapes run at the same rate or less: 16 x 251 to 4096 rows
// of 32 heads on 8 with head_dim 32 10.1 ms, 25 TFLOP/s; 1024 rows of 130 heads on 1, D = 128, 1.3 ms, 28;
// 2 x 40 to 77 rows of 28 heads on 4 behind 20,000 to 32,768 tokens in pages of 5 or 48 1.6 ms, 30 (in
// pages of 16, on the tensor cores, 80 us).
#include "attn_common.cuh"
#include "seq_attn.cuh"

namespace d2f {
namespace {

constexpr int kThreads = 256;
constexpr int KT = 64;

template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
  return __ldg(reinterpret_cast<const float4 *>(p));
}
template <>
__device__ __forceinline__ float4 load4<uint16_t>(const uint16_t *p) {
  const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
  return make_float4(bf16_bits_to_float(v.x & 0xffffu), bf16_bits_to_float(v.x >> 16),
                     bf16_bits_to_float(v.y & 0xffffu), bf16_bits_to_float(v.y >> 16));
}

// Pairs of floats in one register pair: d += a b, an instruction for both.
using Pair = unsigned long long;
__device__ __forceinline__ void fma2(Pair &d, Pair a, Pair b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ Pair twice(float x) {
  Pair p;
  asm("mov.b64 %0, {%1, %1};" : "=l"(p) : "f"(x));
  return p;
}
__device__ __forceinline__ float sum_of(Pair p) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
  return x + y;
}

template <int D, int R>
struct Smem {
  static constexpr int kPitch = D + 4;
  static constexpr int kPPitch = KT + 4;
  float q[R][kPitch];
  float k[KT][kPitch];  // P [R][kPPitch] after S is computed
  float v[KT][D];
  int page[KT];         // page of a cached key, -1: no key
  static_assert(R * kPPitch <= KT * kPitch || D < 64, "P fits K's place");
};
template <int D, int R>
constexpr size_t smem_bytes() {
  // (with D = 32 P is larger than K and gets its own place behind the struct)
  return sizeof(Smem<D, R>) + (D < 64 ? R * (KT + 4) * sizeof(float) : 0);
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads, 2) prompt_simt_kernel(const PromptArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  using S = Smem<D, R>;
  S &sm = *reinterpret_cast<S *>(smem_raw);
  float *p_s = D < 64 ? reinterpret_cast<float *>(smem_raw + sizeof(S)) : &sm.k[0][0];
  constexpr int PP = S::kPPitch, RT = R / 16;  // rows a thread
  const int tid = threadIdx.x;
  const int rg = tid >> 4, cg = tid & 15;  // rows RT rg ..; keys cg + 16 j; columns 4 cg + 64 j
  if (blockIdx.x == 0 && tid < 32) seq_report(a);

  int64_t item = blockIdx.x;
  const int split = (int)(item % a.num_splits);
  item /= a.num_splits;
  const int chunk = (int)(item % a.chunks);
  item /= a.chunks;
  const int g = (int)(item % a.num_heads_kv);
  // the last tiles of a request see the most keys: they come first
  const SeqTile s = seq_tile(a, a.tiles - 1 - (int)(item / a.num_heads_kv));
  if (!s.live) return;
  const int HC = a.head_chunk, H = a.num_heads_q, Hk = a.num_heads_kv;
  const int h0 = chunk * HC, heads = min(HC, a.group - h0);
  const int i0 = s.tile * a.tile_q, ni = min(a.tile_q, s.n - i0);
  const int last = seq_limit(i0 + ni - 1, s.n, a.mask_block);
  const int Tc = (s.C + KT - 1) / KT;
  int t0, t1, s_eff;
  if (!split_range(Tc + (last + KT - 1) / KT, a.num_splits, split, t0, t1, s_eff)) t0 = t1 = 0;

  const T *Q = static_cast<const T *>(a.q);
  for (int e = tid; e < R * (D / 4); e += kThreads) {
    const int r = e / (D / 4), d = (e % (D / 4)) * 4;
    const int i = r / HC, h = r % HC;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < ni && h < heads)
      x = load4<T>(Q + ((int64_t)(s.q0 + i0 + i) * H + g * a.group + h0 + h) * D + d);
    x.x *= a.scale_log2;
    x.y *= a.scale_log2;
    x.z *= a.scale_log2;
    x.w *= a.scale_log2;
    *reinterpret_cast<float4 *>(&sm.q[r][d]) = x;
  }

  constexpr int CJ = D / 64 > 0 ? D / 64 : 1;  // groups of four columns a thread
  const bool cols = D >= 64 || cg < D / 4;     // (D = 32: eight threads of a row hold columns)
  float m[RT], l[RT];
  union Out {  // four columns
    Pair p[2];
    float f[4];
  } o[RT][CJ];
  int lim[RT];  // new rows that the row sees
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    m[x] = -INFINITY;
    l[x] = 0.f;
    lim[x] = seq_limit(min(i0 + (RT * rg + x) / HC, s.n - 1), s.n, a.mask_block);
#pragma unroll
    for (int j = 0; j < CJ; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[x][j].f[c] = 0.f;
  }

  for (int t = t0; t < t1; ++t) {
    __syncthreads();
    const bool cached = t < Tc;
    const int k0 = (cached ? t : t - Tc) * KT;
    if (tid < KT) {
      int page = -1;
      if (cached && k0 + tid < s.C) {
        page = __ldg(a.page_table + (int64_t)s.b * a.max_pages_per_seq + (k0 + tid) / a.block_size);
        if (page < 0 || page >= a.num_pages) {
          page = -1;
          set_err(a.err, D2F_ERR_BAD_INDEX);
        }
      }
      sm.page[tid] = page;
    }
    __syncthreads();
    bool odd = false;  // an infinite or NaN V
    for (int e = tid; e < KT * (D / 4); e += kThreads) {
      const int c = e / (D / 4), d = (e % (D / 4)) * 4;
      float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
      if (cached) {
        if (sm.page[c] >= 0) {
          const int64_t at = (((int64_t)sm.page[c] * Hk + g) * a.block_size +
                              (k0 + c) % a.block_size) * D + d;
          kx = load4<T>(static_cast<const T *>(a.k_pool) + at);
          vx = load4<T>(static_cast<const T *>(a.v_pool) + at);
        }
      } else if (k0 + c < last) {
        const int64_t at = ((int64_t)(s.q0 + k0 + c) * Hk + g) * D + d;
        kx = load4<T>(static_cast<const T *>(a.k) + at);
        vx = load4<T>(static_cast<const T *>(a.v) + at);
      }
      // (0 * x is NaN for these x and 0 for the others)
      odd |= !(0.f * vx.x + 0.f * vx.y + 0.f * vx.z + 0.f * vx.w == 0.f);
      *reinterpret_cast<float4 *>(&sm.k[c][d]) = kx;
      *reinterpret_cast<float4 *>(&sm.v[c][d]) = vx;
    }
    odd = __syncthreads_or(odd);

    float sc[RT][4];
    {
      Pair sum[RT][4] = {};  // of the even and of the odd dims
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        ulonglong2 qx[RT], kx[4];
#pragma unroll
        for (int x = 0; x < RT; ++x) qx[x] = *reinterpret_cast<ulonglong2 *>(&sm.q[RT * rg + x][d]);
#pragma unroll
        for (int j = 0; j < 4; ++j) kx[j] = *reinterpret_cast<ulonglong2 *>(&sm.k[cg + 16 * j][d]);
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            fma2(sum[x][j], qx[x].x, kx[j].x);
            fma2(sum[x][j], qx[x].y, kx[j].y);
          }
      }
#pragma unroll
      for (int x = 0; x < RT; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[x][j] = sum_of(sum[x][j]);
    }
    uint32_t seen = 0;  // bit 4 x + j
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = cg + 16 * j;
      const bool key = cached ? sm.page[c] >= 0 : true;
#pragma unroll
      for (int x = 0; x < RT; ++x)
        if (key && (cached || k0 + c < lim[x])) seen |= 1u << (4 * x + j);
    }
    __syncthreads();  // K is done with: P takes its place
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!(seen >> (4 * x + j) & 1u)) sc[x][j] = -INFINITY;
        top = fmaxf(top, sc[x][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      const float m_new = fmaxf(m[x], top);
      const float base = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: all weights 0
      const float alpha = fast_exp2(m[x] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = (seen >> (4 * x + j) & 1u) ? fast_exp2(sc[x][j] - base) : 0.f;
        sum += p;
        p_s[(RT * rg + x) * PP + cg + 16 * j] = p;
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      l[x] = l[x] * alpha + sum;
      m[x] = m_new;
#pragma unroll
      for (int j = 0; j < CJ; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[x][j].f[c] *= alpha;
    }
    __syncthreads();
    if (cols) {
      if (!odd) {
#pragma unroll 2
        for (int c = 0; c < KT; c += 4) {
          float4 px[RT];
#pragma unroll
          for (int x = 0; x < RT; ++x)
            px[x] = *reinterpret_cast<const float4 *>(&p_s[(RT * rg + x) * PP + c]);
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            Pair p[RT];
#pragma unroll
            for (int x = 0; x < RT; ++x)
              p[x] = twice(cc == 0 ? px[x].x : cc == 1 ? px[x].y : cc == 2 ? px[x].z : px[x].w);
#pragma unroll
            for (int j = 0; j < CJ; ++j) {
              const ulonglong2 vx = *reinterpret_cast<const ulonglong2 *>(&sm.v[c + cc][4 * cg + 64 * j]);
#pragma unroll
              for (int x = 0; x < RT; ++x) {
                fma2(o[x][j].p[0], p[x], vx.x);
                fma2(o[x][j].p[1], p[x], vx.y);
              }
            }
          }
        }
      } else {  // a row takes the keys it sees only: 0 * infinity is not 0
        for (int c = 0; c < KT; ++c) {
          const bool key = !cached || sm.page[c] >= 0;
#pragma unroll
          for (int x = 0; x < RT; ++x) {
            if (!key || (!cached && k0 + c >= lim[x])) continue;
            const float p = p_s[(RT * rg + x) * PP + c];
#pragma unroll
            for (int j = 0; j < CJ; ++j)
#pragma unroll
              for (int d = 0; d < 4; ++d)
                o[x][j].f[d] = fmaf(p, sm.v[c][4 * cg + 64 * j + d], o[x][j].f[d]);
          }
        }
      }
    }
  }

  const int64_t n_hr = (int64_t)a.rows * H;
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int r = RT * rg + x, i = r / HC, h = r % HC;
    if (i >= ni || h >= heads) continue;
    const int64_t hr = (int64_t)(s.q0 + i0 + i) * H + g * a.group + h0 + h;
    if (a.num_splits > 1) {
      if (cg == 0) a.ws_ml[split * n_hr + hr] = make_float2(m[x], l[x]);
      float *dst = a.ws_o + (split * n_hr + hr) * D;
      if (cols)
#pragma unroll
        for (int j = 0; j < CJ; ++j)
          *reinterpret_cast<float4 *>(dst + 4 * cg + 64 * j) =
              make_float4(o[x][j].f[0], o[x][j].f[1], o[x][j].f[2], o[x][j].f[3]);
      continue;
    }
    if (cg == 0 && a.lse_out) a.lse_out[hr] = (m[x] + __log2f(l[x])) * 0.6931471805599453f;
    const float inv = 1.0f / l[x];
    const bool none = l[x] == 0.f;  // every score is -inf (the product may be 0 * infinity)
    T *dst = static_cast<T *>(a.out) + hr * D;
    if (cols)
#pragma unroll
      for (int j = 0; j < CJ; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          store_out<T>(dst + 4 * cg + 64 * j + c, none ? 0.f : o[x][j].f[c] * inv);
  }
}

// Composition of the splits, one warp a (row, head): rows behind the last request and rows of
// a request with inconsistent lengths have no partials and are left as they are.
template <typename T, int D>
__global__ void __launch_bounds__(256) prompt_merge_kernel(const PromptArgs a) {
  const int64_t hr = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t n_hr = (int64_t)a.rows * a.num_heads_q;
  if (hr >= n_hr) return;
  const int row = (int)(hr / a.num_heads_q);
  // the request that holds the row: the last b with row_start[b] <= row
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33, at = lo + (lane + 1) * step;
    const int k = __popc(__ballot_sync(0xffffffffu, at < hi && __ldg(a.row_start + at) <= row));
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  const int q0 = __ldg(a.row_start + lo), q1 = __ldg(a.row_start + lo + 1);
  const int C = a.ctx_len ? __ldg(a.ctx_len + lo) : 0;
  if (q0 < 0 || q1 > a.rows || row < q0 || row >= q1 || C < 0 ||
      (long long)C > (long long)a.max_pages_per_seq * a.block_size)
    return;
  // (After a wait that ran out the counts may not have been written: no more than there are parts.)
  const int splits = a.split_count ? min(__ldcg(a.split_count + lo), a.num_splits) : a.num_splits;
  if (splits <= 1) return;  // (written by its only item)
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < splits) ml = __ldcg(&a.ws_ml[lane * n_hr + hr]);
  float M = ml.x;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
  const float w = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
  // (a split that saw nothing: weight 0; one whose sum is NaN keeps it)
  float L = ml.x == -INFINITY ? ml.y : w * ml.y;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
  constexpr int V = D / 32;
  float acc[V] = {};
  // eight parts at a time, whose loads go out together
  constexpr int N = 8;
  for (int sp0 = 0; sp0 < splits; sp0 += N) {
    float y[N][V], ws[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      ws[k] = __shfl_sync(0xffffffffu, w, (sp0 + k) & 31);
#pragma unroll
      for (int j = 0; j < V; ++j) y[k][j] = 0.f;
      if (sp0 + k < splits && ws[k] != 0.f) {  // (a part without weight may not have been written)
        const float *src = a.ws_o + ((int64_t)(sp0 + k) * n_hr + hr) * D + lane * V;
        if constexpr (V == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4 *>(src));
          y[k][0] = x.x, y[k][1] = x.y, y[k][2] = x.z, y[k][3] = x.w;
        } else if constexpr (V == 2) {
          const float2 x = __ldcg(reinterpret_cast<const float2 *>(src));
          y[k][0] = x.x, y[k][1] = x.y;
        } else {
          y[k][0] = __ldcg(src);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = fmaf(ws[k], y[k][j], acc[j]);
  }
  const float inv = L == 0.f ? 0.f : 1.0f / L;
  T *dst = static_cast<T *>(a.out) + hr * D + lane * V;
#pragma unroll
  for (int j = 0; j < V; ++j) store_out<T>(dst + j, acc[j] * inv);
  if (lane == 0 && a.lse_out) a.lse_out[hr] = (M + __log2f(L)) * 0.6931471805599453f;
}

template <typename T, int D, int R>
cudaError_t launch_r(const PromptArgs &a, cudaStream_t s) {
  constexpr size_t bytes = smem_bytes<D, R>();
  const cudaError_t e = allow_smem_once<&prompt_simt_kernel<T, D, R>>((int)bytes);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)a.tiles * a.num_heads_kv * a.chunks * a.num_splits;
  prompt_simt_kernel<T, D, R><<<(unsigned)items, kThreads, bytes, s>>>(a);
  return cudaGetLastError();
}
template <typename T, int D>
cudaError_t launch_d(const PromptArgs &a, cudaStream_t s) {
  return a.simt_rows == 64 ? launch_r<T, D, 64>(a, s)
         : a.simt_rows == 32 ? launch_r<T, D, 32>(a, s) : launch_r<T, D, 16>(a, s);
}

template <typename T, int D>
cudaError_t merge_d(const PromptArgs &a, cudaStream_t s) {
  const int64_t n_hr = (int64_t)a.rows * a.num_heads_q;
  // (an ordinary launch: started early, its CTAs cost the few that still work more than they save)
  prompt_merge_kernel<T, D><<<(unsigned)((n_hr + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const PromptArgs &a, cudaStream_t s) {
  switch (a.head_dim) {
    case 32: return launch_d<T, 32>(a, s);
    case 64: return launch_d<T, 64>(a, s);
    case 128: return launch_d<T, 128>(a, s);
    default: return cudaErrorInvalidValue;
  }
}
template <typename T>
cudaError_t merge_t(const PromptArgs &a, cudaStream_t s) {
  switch (a.head_dim) {
    case 32: return merge_d<T, 32>(a, s);
    case 64: return merge_d<T, 64>(a, s);
    case 128: return merge_d<T, 128>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_prompt_simt(const PromptArgs &a, int dtype, cudaStream_t s) {
  return dtype == D2F_BF16 ? launch_t<uint16_t>(a, s) : launch_t<float>(a, s);
}

cudaError_t launch_prompt_merge(const PromptArgs &a, int dtype, cudaStream_t s) {
  return dtype == D2F_BF16 ? merge_t<uint16_t>(a, s) : merge_t<float>(a, s);
}

}  // namespace d2f
