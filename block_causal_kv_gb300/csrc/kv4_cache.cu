// d2f_kv4_append and d2f_kv4_read: writing finished blocks into the 4-bit cache and
// reading tokens of it back (layout and arithmetic: kv4.cuh).
//
// Source: "D2F: 확산 언어 모델이 KV 캐시를 얻고 자기회귀 모델보다 2.5배 빨라지는
// 방법", §블록 단위 인과 어텐션 and §운영 관점 (a completed block's K/V are final
// and persisted; a page holds one block).
//
// Both move bytes once: an append reads 2 D elements a token and head and writes 9/16 of
// that many bytes, a read the reverse. Measured (16 prompts of 251 to 4096 tokens, 30,000
// tokens, 32 heads, D = 128, B = 16, bf16): append 121 us and read 105 us, 5.2 and 6.0 TB/s;
// float32, twice the elements' bytes: 215 and 187 us, 5.2 and 6.0 TB/s (its append makes the
// definition's divisions, 17 a group, beside twice the loads).
// Neither is quite at the memory's rate: the conversions keep the issue slots 70 % and 73 %
// busy (ALU 63 % and 60 %), and every warp waits for its loads once. A step's 8 blocks of 4
// heads take 6 us for both, which is launches.
#include "kv4.cuh"

namespace d2f {
namespace {

constexpr int kThreads = 256;

// Sixteen consecutive elements.
template <typename T>
struct Group;
template <>
struct Group<uint16_t> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const uint16_t *p) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + h);
      w[4 * h] = v.x;
      w[4 * h + 1] = v.y;
      w[4 * h + 2] = v.z;
      w[4 * h + 3] = v.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0;
  }
};
template <>
struct Group<float> {
  float x[16];
  __device__ __forceinline__ void load(const float *p) {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float4 v = __ldcs(reinterpret_cast<const float4 *>(p) + h);
      x[4 * h] = v.x;
      x[4 * h + 1] = v.y;
      x[4 * h + 2] = v.z;
      x[4 * h + 3] = v.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = 0.f;
  }
};

// Scale bits and the sixteen codes (two words, element 0 in the lowest nibble) of one group.
//
// The definition's quotient is the float y / s with y = x * mul. With bf16 elements the
// code can be had from x * (mul / s) instead (mul is a power of two): y has 8 significant
// bits and a midpoint between two codes times s has at most 7, so a quotient that is not
// a midpoint is at least 2^-8 (relative) away from it; rounded to fp16 (error 2^-11, the
// product's own error 2^-23 beside it) it stays on its side, and an exact midpoint comes
// out as itself, also with a reciprocal that is a step off. The scale's quotient by 6 goes
// the same way (a midpoint between two e4m3 values has at most 5 bits, times 6 at most 7;
// what fp16 cannot hold is above 448 or rounds to 0). Eighteen divisions a group would make
// the kernel compute-bound (35,000 tokens x 32 heads: 440 us with them). The largest
// magnitude is that of the bits, two halves at a time (a NaN's are above infinity's).
__device__ __forceinline__ uint32_t encode16(const Group<uint16_t> &g, float mul,
                                             uint32_t (&code)[2]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __vmaxu2(top, g.w[j] & 0x7fff7fffu);
  const float amax = __uint_as_float(max(top << 16, top & 0xffff0000u)) * mul;
  uint32_t sb;
  asm("{\n\t.reg .b32 h;\n\t.reg .b16 t;\n\tcvt.rn.f16x2.f32 h, %1, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 t, h;\n\tcvt.u32.u16 %0, t;\n\t}"
      : "=r"(sb)
      : "f"(amax * (1.0f / 6.0f)));
  sb &= 0xffu;
  const float s = e4m3_value(sb);
  float inv;
  asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const float f = s == 0.f ? 0.f : mul * inv;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = g.w[4 * w + j];
      float a = __uint_as_float(x << 16), b = __uint_as_float(x & 0xffff0000u);
      mul2(a, b, f);
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(b), "f"(a));
    }
    const uint32_t c = half8_to_codes(h);
    code[w] = s == 0.f ? 0u : c;  // (no negative zeros in a group without a scale)
  }
  return sb;
}
__device__ __forceinline__ uint32_t encode16(const Group<float> &g, float mul,
                                             uint32_t (&code)[2]) {
  float y[16], amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    y[j] = g.x[j] * mul;
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
      c |= e2m1x2_bits(s == 0.f ? 0.f : __fdiv_rn(a, s), s == 0.f ? 0.f : __fdiv_rn(b, s)) << (8 * j);
    }
    code[w] = s == 0.f ? 0u : c;
  }
  return sb;
}

// 8 x 8 nibbles: o[d] gets nibble d of r[0] .. r[7], in that order.
__device__ __forceinline__ void transpose_nibbles(uint32_t (&r)[8]) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {  // halves of words, four apart
    const uint32_t a = r[t], b = r[t + 4];
    r[t] = __byte_perm(a, b, 0x5410);
    r[t + 4] = __byte_perm(a, b, 0x7632);
  }
#pragma unroll
  for (int t = 0; t < 8; t += t & 1 ? 3 : 1) {  // bytes, two apart: t = 0, 1, 4, 5
    const uint32_t a = r[t], b = r[t + 2];
    r[t] = __byte_perm(a, b, 0x6240);
    r[t + 2] = __byte_perm(a, b, 0x7351);
  }
#pragma unroll
  for (int t = 0; t < 8; t += 2) {  // nibbles
    const uint32_t a = r[t], b = r[t + 1];
    r[t] = (a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u);
    r[t + 1] = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
  }
}

// One CTA per (append entry, KV head). A thread owns one group of 16 elements of one
// token; the page is put together in shared memory and written in 16-byte pieces. V's
// codes are transposed there by one thread per eight dims, 8 tokens x 8 dims at a time
// in registers (a thread per dim that collects its nibbles: 130 us against 125).
template <typename T, int D, int B>
__global__ void __launch_bounds__(kThreads) append_kernel(const Kv4AppendArgs a) {
  constexpr int NG = D / 16;
  constexpr Kv4Layout L{D, B};
  // V codes of a (group, token); a row more than the tokens, against bank conflicts
  __shared__ uint2 v_s[NG][B + 1];
  __shared__ uint4 page_s[B * D * 9 / 128];
  grid_dependency_wait();
  const int ap = blockIdx.x / a.num_heads_kv;
  const int g = blockIdx.x % a.num_heads_kv;
  if (a.n_dev != nullptr && ap >= min(max(*a.n_dev, 0), a.n_append)) return;
  const int src = a.src_row[ap], dst = a.dst_page[ap];
  const int rows = a.n_rows ? a.n_rows[ap] : B;
  if (src < 0 || rows < 0 || rows > B || (int64_t)src + rows > a.total_q || dst < 0 ||
      dst >= a.num_pages) {
    if (threadIdx.x == 0 && g == 0) set_err(a.err, D2F_ERR_BAD_INDEX);
    return;
  }
  uint8_t *image = reinterpret_cast<uint8_t *>(page_s);
  constexpr int per = B * NG;  // groups of one tensor
#pragma unroll
  for (int i = threadIdx.x; i < 2 * per; i += kThreads) {
    const int which = i / per, t = (i % per) / NG, grp = i % NG;
    Group<T> x;
    if (t < rows)
      x.load(reinterpret_cast<const T *>(which ? a.v_win : a.k_win) +
             ((int64_t)(src + t) * a.num_heads_kv + g) * D + grp * 16);
    else
      x.zero();  // slots past the block's rows hold zeros
    uint32_t code[2];
    const uint32_t sb = encode16(x, which ? a.v_mul : a.k_mul, code);
    if (which == 0) {
      *reinterpret_cast<uint2 *>(image + ((grp >> 1) * B + t) * 16 + (grp & 1) * 8) =
          make_uint2(code[0], code[1]);
      image[L.k_scales() + t * NG + grp] = (uint8_t)sb;
    } else {
      v_s[grp][t] = make_uint2(code[0], code[1]);
      image[L.v_scales() + grp * B + t] = (uint8_t)sb;
    }
  }
  __syncthreads();
  if (threadIdx.x < D / 8) {
    const int d8 = threadIdx.x;  // dims 8 d8 .. 8 d8 + 7
    uint32_t out[B];             // word w of dim i: out[i * (B / 8) + w]
#pragma unroll
    for (int w = 0; w < B / 8; ++w) {
      uint32_t r[8];
#pragma unroll
      for (int t = 0; t < 8; ++t)
        r[t] = reinterpret_cast<const uint32_t *>(&v_s[d8 >> 1][8 * w + t])[d8 & 1];
      transpose_nibbles(r);
#pragma unroll
      for (int i = 0; i < 8; ++i) out[i * (B / 8) + w] = r[i];
    }
    uint4 *p = reinterpret_cast<uint4 *>(image + L.v_codes() + d8 * 4 * B);
#pragma unroll
    for (int i = 0; i < B / 4; ++i)
      p[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
  }
  __syncthreads();
  uint4 *page = reinterpret_cast<uint4 *>(a.pool + ((int64_t)dst * a.num_heads_kv + g) * L.page_bytes());
  for (int i = threadIdx.x; i < L.page_bytes() / 16; i += kThreads) page[i] = page_s[i];
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

// One CTA per (64 tokens of the list, KV head). K: a thread owns a group of 16 elements of
// one token. V: the list is cut into runs of consecutive slots of one page; a warp owns
// 64 dims of a run, a lane two of them, whose codes of the whole page are one coalesced
// read, so a page of V is read once a run and written a token (128 bytes a warp) at a
// time. (Gathering V element by element took twice as long: eight cache lines a load.)
constexpr int kReadRows = 64;
template <typename T, int D, int B>
// CTAs an SM: eight where 32 registers do without spills (B = 16: 228 us for the append and
// read of 30,000 tokens, 237 without a bound), five else.
__global__ void __launch_bounds__(kThreads, (B <= 16 ? 8 : 5)) read_kernel(const Kv4ReadArgs a) {
  constexpr int NG = D / 16;
  constexpr Kv4Layout L{D, B};
  __shared__ int64_t slot_s[kReadRows];  // -1: none
  __shared__ uint8_t run_s[kReadRows + 1];
  __shared__ int runs0_s, nruns_s;
  grid_dependency_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.x % a.num_heads_kv;
  const int64_t i0 = (int64_t)(blockIdx.x / a.num_heads_kv) * kReadRows;
  const int n = (int)min((int64_t)kReadRows, a.n - i0);
  if (warp < 2) {
    int64_t slot = -1;
    if (tid < n) {
      slot = a.slot[i0 + tid];
      if (slot < 0 || slot >= (int64_t)a.num_pages * B) {
        if (slot != -1 && g == 0) set_err(a.err, D2F_ERR_BAD_INDEX);
        slot = -1;
      }
    }
    slot_s[tid] = slot;
    // a run starts where the slot does not follow its predecessor within a page
    const int64_t prev = __shfl_up_sync(0xffffffffu, slot, 1);
    const bool start = tid < n && (lane == 0 || slot < 0 || slot != prev + 1 || slot % B == 0);
    const unsigned m = __ballot_sync(0xffffffffu, start);
    if (warp == 0 && lane == 0) runs0_s = __popc(m);
    if (warp == 0 && start) run_s[__popc(m & ((1u << lane) - 1))] = (uint8_t)tid;
    asm volatile("bar.sync 1, 64;" ::: "memory");
    if (warp == 1) {
      const int at = runs0_s;
      if (start) run_s[at + __popc(m & ((1u << lane) - 1))] = (uint8_t)tid;
      if (lane == 0) {
        nruns_s = at + __popc(m);
        run_s[at + __popc(m)] = (uint8_t)n;
      }
    }
  }
  __syncthreads();
  T *k_out = reinterpret_cast<T *>(a.k_out), *v_out = reinterpret_cast<T *>(a.v_out);
  constexpr int kK = 2;  // groups of a thread at once: every load before any use
  for (int i0k = tid; i0k < n * NG; i0k += kK * kThreads) {
    uint2 w[kK];
    uint32_t sc[kK];
#pragma unroll
    for (int q = 0; q < kK; ++q) {
      const int i = i0k + q * kThreads, t = i / NG, grp = i % NG;
      const int64_t slot = i < n * NG ? slot_s[t] : -1;
      w[q] = make_uint2(0, 0);
      sc[q] = 0;
      if (slot >= 0) {
        const int o = (int)(slot % B);
        const uint8_t *page = a.pool + (slot / B * a.num_heads_kv + g) * L.page_bytes();
        w[q] = __ldg(reinterpret_cast<const uint2 *>(page + ((grp >> 1) * B + o) * 16 + (grp & 1) * 8));
        sc[q] = __ldg(page + L.k_scales() + o * NG + grp);
      }
    }
#pragma unroll
    for (int q = 0; q < kK; ++q) {
      const int i = i0k + q * kThreads, t = i / NG, grp = i % NG;
      if (i >= n * NG) break;
      const float s = e4m3_value(sc[q]) * a.k_mul;
      float k[16];
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const uint32_t h = e2m1x2_to_half2(((j < 8 ? w[q].x : w[q].y) >> (4 * (j & 7))) & 0xffu);
        k[j] = half_lo(h);
        k[j + 1] = half_hi(h);
        mul2(k[j], k[j + 1], s);
      }
      store16<T>(k_out + ((i0 + t) * a.num_heads_kv + g) * D + grp * 16, k);
    }
  }
  constexpr int kHalves = D / 64;  // warps a run
  const int d = 64 * (warp % kHalves) + 2 * lane;
  for (int r = warp / kHalves; r < nruns_s; r += (kThreads / 32) / kHalves) {
    const int t0 = run_s[r], t1 = run_s[r + 1];
    const int64_t slot = slot_s[t0];
    const int o0 = slot < 0 ? 0 : (int)(slot % B);  // (a run of no slot is one token long)
    uint32_t w0[B / 8], w1[B / 8], sc[B / 4];  // both dims' codes, the group's scale bytes
#pragma unroll
    for (int i = 0; i < B / 8; ++i) w0[i] = w1[i] = 0;
#pragma unroll
    for (int i = 0; i < B / 4; ++i) sc[i] = 0;
    if (slot >= 0) {
      const uint8_t *page = a.pool + (slot / B * a.num_heads_kv + g) * L.page_bytes();
      const uint32_t *c = reinterpret_cast<const uint32_t *>(page + L.v_codes() + d * (B / 2));
      const uint32_t *s = reinterpret_cast<const uint32_t *>(page + L.v_scales() + (d >> 4) * B);
#pragma unroll
      for (int i = 0; i < B / 8; ++i) {
        w0[i] = __ldg(c + i);
        w1[i] = __ldg(c + B / 8 + i);
      }
#pragma unroll
      for (int i = 0; i < B / 4; ++i) sc[i] = __ldg(s + i);
    }
    T *out = v_out + ((i0 + t0 - o0) * a.num_heads_kv + g) * D + d;  // of token 0 of the page
    const int64_t step = (int64_t)a.num_heads_kv * D;
    const int n_run = t1 - t0;
#pragma unroll
    for (int q = 0; q < B / 8; ++q) {
      // both dims' codes of a token in one byte: tokens 0, 2, 4, 6 and 1, 3, 5, 7
      const uint32_t even = (w0[q] & 0x0f0f0f0fu) | ((w1[q] << 4) & 0xf0f0f0f0u);
      const uint32_t odd = ((w0[q] >> 4) & 0x0f0f0f0fu) | (w1[q] & 0xf0f0f0f0u);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t s2 = e4m3x2_to_half2(sc[2 * q + p / 2] >> (16 * (p & 1)));  // two tokens'
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int o = 8 * q + 2 * p + k;
          if ((unsigned)(o - o0) >= (unsigned)n_run) continue;
          const uint32_t h = e2m1x2_to_half2((k ? odd : even) >> (8 * p));
          const float s = (k ? half_hi(s2) : half_lo(s2)) * a.v_mul;
          float x = half_lo(h), y = half_hi(h);
          mul2(x, y, s);
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint32_t *>(out + o * step) = pack_bf16x2(x, y);
          else
            *reinterpret_cast<float2 *>(out + o * step) = make_float2(x, y);
        }
      }
    }
  }
}

template <typename Kernel, typename Args>
cudaError_t launch(Kernel kernel, unsigned grid, const Args &a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, int B>
cudaError_t launch_append(const Kv4AppendArgs &a, int dtype, cudaStream_t s) {
  const unsigned grid = (unsigned)a.n_append * a.num_heads_kv;
  return dtype == D2F_BF16 ? launch(append_kernel<uint16_t, D, B>, grid, a, s)
                           : launch(append_kernel<float, D, B>, grid, a, s);
}
template <int D, int B>
cudaError_t launch_read(const Kv4ReadArgs &a, int dtype, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.n + kReadRows - 1) / kReadRows * a.num_heads_kv);
  return dtype == D2F_BF16 ? launch(read_kernel<uint16_t, D, B>, grid, a, s)
                           : launch(read_kernel<float, D, B>, grid, a, s);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs &a, int dtype, int D, cudaStream_t s) {
  switch (a.block_size * 1000 + D) {
    case 8064: return launch_append<64, 8>(a, dtype, s);
    case 16064: return launch_append<64, 16>(a, dtype, s);
    case 32064: return launch_append<64, 32>(a, dtype, s);
    case 8128: return launch_append<128, 8>(a, dtype, s);
    case 16128: return launch_append<128, 16>(a, dtype, s);
    default: return launch_append<128, 32>(a, dtype, s);
  }
}

cudaError_t launch_kv4_read(const Kv4ReadArgs &a, int dtype, int D, cudaStream_t s) {
  switch (a.block_size * 1000 + D) {
    case 8064: return launch_read<64, 8>(a, dtype, s);
    case 16064: return launch_read<64, 16>(a, dtype, s);
    case 32064: return launch_read<64, 32>(a, dtype, s);
    case 8128: return launch_read<128, 8>(a, dtype, s);
    case 16128: return launch_read<128, 16>(a, dtype, s);
    default: return launch_read<128, 32>(a, dtype, s);
  }
}

}  // namespace d2f
