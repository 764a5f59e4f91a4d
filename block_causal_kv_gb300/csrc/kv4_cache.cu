// d2f_kv4_append and d2f_kv4_read: writing finished blocks into the 4-bit cache and
// reading tokens of it back (layout and arithmetic: kv4.cuh).
//
// Source: "D2F: 확산 언어 모델이 KV 캐시를 얻고 자기회귀 모델보다 2.5배 빨라지는
// 방법", §블록 단위 인과 어텐션 and §운영 관점 (a completed block's K/V are final
// and persisted; a page holds one block).
#include "kv4.cuh"

namespace d2f {
namespace {

constexpr int kThreads = 256;

// Sixteen consecutive elements as floats.
template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]);
template <>
__device__ __forceinline__ void load16<uint16_t>(const uint16_t *p, float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + h);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * h + 2 * j] = __uint_as_float(w[j] << 16);
      x[8 * h + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
template <>
__device__ __forceinline__ void load16<float>(const float *p, float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const float4 v = __ldcs(reinterpret_cast<const float4 *>(p) + h);
    x[4 * h] = v.x;
    x[4 * h + 1] = v.y;
    x[4 * h + 2] = v.z;
    x[4 * h + 3] = v.w;
  }
}

// Scale bits and the sixteen codes (two words, element 0 in the lowest nibble) of one group.
template <typename T>
__device__ __forceinline__ uint32_t encode16(const float (&x)[16], float mul, uint32_t (&code)[2]) {
  float y[16], amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    y[j] = x[j] * mul;
    amax = fmax_nan(amax, fabsf(y[j]));
  }
  const uint32_t sb = e4m3_bits(__fdiv_rn(amax, 6.0f));
  const float s = e4m3_value(sb);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = y[8 * w + 2 * j], b = y[8 * w + 2 * j + 1];
      const float qa = s == 0.f ? 0.f : __fdiv_rn(a, s), qb = s == 0.f ? 0.f : __fdiv_rn(b, s);
      c |= e2m1x2_bits(qa, qb) << (8 * j);
    }
    code[w] = c;
  }
  return sb;
}

// One CTA per (append entry, KV head): the page is put together in shared memory and
// stored 16 bytes at a time. A thread owns one group of 16 elements.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) append_kernel(const Kv4AppendArgs a) {
  constexpr int NG = D / 16;
  extern __shared__ uint4 tile4[];
  uint8_t *tile = reinterpret_cast<uint8_t *>(tile4);
  grid_dependency_wait();
  const int ap = blockIdx.x / a.num_heads_kv;
  const int g = blockIdx.x % a.num_heads_kv;
  if (a.n_dev != nullptr && ap >= min(max(*a.n_dev, 0), a.n_append)) return;
  const int B = a.block_size;
  const int src = a.src_row[ap], dst = a.dst_page[ap];
  const int rows = a.n_rows ? a.n_rows[ap] : B;
  if (src < 0 || rows < 0 || rows > B || (int64_t)src + rows > a.total_q || dst < 0 ||
      dst >= a.num_pages) {
    if (threadIdx.x == 0 && g == 0) set_err(a.err, D2F_ERR_BAD_INDEX);
    return;
  }
  const Kv4Layout L{D, B};
  const int per = B * NG;  // groups of one tensor (a multiple of 32)
  for (int i = threadIdx.x; i < 2 * per; i += kThreads) {
    const int which = i / per, t = (i % per) / NG, grp = i % NG;
    float x[16];
    if (t < rows) {
      load16<T>(reinterpret_cast<const T *>(which ? a.v_win : a.k_win) +
                    ((int64_t)(src + t) * a.num_heads_kv + g) * D + grp * 16, x);
    } else {  // slots past the block's rows hold zeros
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = 0.f;
    }
    uint32_t code[2];
    const uint32_t sb = encode16<T>(x, which ? a.v_mul : a.k_mul, code);
    if (which == 0) {
      *reinterpret_cast<uint2 *>(tile + ((grp >> 1) * B + t) * 16 + (grp & 1) * 8) =
          make_uint2(code[0], code[1]);
      tile[L.k_scales() + t * NG + grp] = (uint8_t)sb;
    } else {
      // token t and its neighbour t ^ 1 (the lane NG away) share bytes: each of the
      // two threads takes half of the dims and writes both tokens' nibbles
      const uint32_t other0 = __shfl_xor_sync(0xffffffffu, code[0], NG);
      const uint32_t other1 = __shfl_xor_sync(0xffffffffu, code[1], NG);
      const bool odd = t & 1;
      const uint32_t mine = odd ? code[1] : code[0], theirs = odd ? other1 : other0;
      const uint32_t lo = odd ? theirs : mine, hi = odd ? mine : theirs;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int d = grp * 16 + odd * 8 + j;
        tile[L.v_codes() + d * (B / 2) + (t >> 1)] =
            (uint8_t)(((lo >> (4 * j)) & 15u) | (((hi >> (4 * j)) & 15u) << 4));
      }
      tile[L.v_scales() + grp * B + t] = (uint8_t)sb;
    }
  }
  __syncthreads();
  uint4 *out = reinterpret_cast<uint4 *>(a.pool + ((int64_t)dst * a.num_heads_kv + g) *
                                                      L.page_bytes());
  for (int i = threadIdx.x; i < L.page_bytes() / 16; i += kThreads) out[i] = tile4[i];
}

template <typename T>
__device__ __forceinline__ void store16(T *p, const float (&x)[16]);
template <>
__device__ __forceinline__ void store16<uint16_t>(uint16_t *p, const float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    reinterpret_cast<uint4 *>(p)[h] =
        make_uint4(pack_bf16x2(x[8 * h], x[8 * h + 1]), pack_bf16x2(x[8 * h + 2], x[8 * h + 3]),
                   pack_bf16x2(x[8 * h + 4], x[8 * h + 5]), pack_bf16x2(x[8 * h + 6], x[8 * h + 7]));
}
template <>
__device__ __forceinline__ void store16<float>(float *p, const float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 4; ++h)
    reinterpret_cast<float4 *>(p)[h] =
        make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
}

// A thread owns one group of 16 elements of one (token, KV head), K and V.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const Kv4ReadArgs a) {
  constexpr int NG = D / 16;
  grid_dependency_wait();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int grp = (int)(i % NG);
  const int64_t th = i / NG;
  const int g = (int)(th % a.num_heads_kv);
  const int64_t t = th / a.num_heads_kv;
  if (t >= a.n) return;
  const int B = a.block_size;
  const Kv4Layout L{D, B};
  const int64_t slot = a.slot[t];
  float k[16], v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) k[j] = v[j] = 0.f;
  if (slot >= 0 && slot < (int64_t)a.num_pages * B) {
    const int64_t page = slot / B;
    const int o = (int)(slot % B);
    const uint8_t *tile = a.pool + (page * a.num_heads_kv + g) * L.page_bytes();
    const uint2 kc = *reinterpret_cast<const uint2 *>(tile + ((grp >> 1) * B + o) * 16 + (grp & 1) * 8);
    const float ks = e4m3_value(tile[L.k_scales() + o * NG + grp]) * a.k_mul;
    const float vs = e4m3_value(tile[L.v_scales() + grp * B + o]) * a.v_mul;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      k[j] = e2m1_value((j < 8 ? kc.x : kc.y) >> (4 * (j & 7))) * ks;
      const uint32_t vb = tile[L.v_codes() + (grp * 16 + j) * (B / 2) + (o >> 1)];
      v[j] = e2m1_value(vb >> (4 * (o & 1))) * vs;
    }
  } else if (slot != -1 && grp == 0 && g == 0) {
    set_err(a.err, D2F_ERR_BAD_INDEX);
  }
  const int64_t off = (t * a.num_heads_kv + g) * D + grp * 16;
  store16<T>(reinterpret_cast<T *>(a.k_out) + off, k);
  store16<T>(reinterpret_cast<T *>(a.v_out) + off, v);
}

template <typename Kernel, typename Args>
cudaError_t launch(Kernel kernel, unsigned grid, size_t smem, const Args &a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs &a, int dtype, int D, cudaStream_t s) {
  const unsigned grid = (unsigned)a.n_append * a.num_heads_kv;
  const size_t smem = (size_t)Kv4Layout{D, a.block_size}.page_bytes();
  if (dtype == D2F_BF16)
    return D == 64 ? launch(append_kernel<uint16_t, 64>, grid, smem, a, s)
                   : launch(append_kernel<uint16_t, 128>, grid, smem, a, s);
  return D == 64 ? launch(append_kernel<float, 64>, grid, smem, a, s)
                 : launch(append_kernel<float, 128>, grid, smem, a, s);
}

cudaError_t launch_kv4_read(const Kv4ReadArgs &a, int dtype, int D, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.n * a.num_heads_kv * (D / 16) + kThreads - 1) / kThreads);
  if (dtype == D2F_BF16)
    return D == 64 ? launch(read_kernel<uint16_t, 64>, grid, 0, a, s)
                   : launch(read_kernel<uint16_t, 128>, grid, 0, a, s);
  return D == 64 ? launch(read_kernel<float, 64>, grid, 0, a, s)
                 : launch(read_kernel<float, 128>, grid, 0, a, s);
}

}  // namespace d2f
