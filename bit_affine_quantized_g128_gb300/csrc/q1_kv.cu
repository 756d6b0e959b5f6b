// The 4-bit cache: K and V rows quantised into its pages, and read back.
//
// Per token, head and group of 64 or 128 channels, x = scale q + bias with q in
// -8..7: bias is the value that lets the codes -8 and 7 meet the least and the
// largest x, rounded to bf16, and scale the least that reaches both from there,
// rounded to bf16 (include/q1.h has the formula; every step is one fp32 operation,
// so the codes are the same everywhere).
//
// Both kernels are streams.  A thread owns a code word: 8 channels of a row, one or
// two 16-byte pieces of the dense row.  A group is 8 or 16 neighbouring threads, which
// find its least and largest value by shuffles.  A warp stays with one token, so
// that finding its sequence and page is the warp's work, not each thread's.
#include <cuda_bf16.h>

#include <type_traits>

#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kThreads = 256;
constexpr float kLimit = 32768.f;               // larger magnitudes are stored as this
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100: smaller scales are stored as 0

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = meta_f32(w[i], std::is_same<T, __nv_bfloat16>::value);
      f[2 * i + 1] = meta_f32(w[i] >> 16, std::is_same<T, __nv_bfloat16>::value);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The sequence of row t, the same for a whole warp: the last b with cu[b] <= t, 32
// candidates at a time.  -1: none (t lies before the first).
__device__ __forceinline__ int64_t sequence_of(const KvView &c, int64_t t, int lane) {
  if (!c.cu) return t / (c.T / c.B);
  int64_t lo = 0, n = c.B;  // the answer lies in [lo, lo + n), or is lo - 1 where lo = 0
  while (n > 0) {
    const int64_t step = (n + 31) / 32, at = lo + step * lane;
    const unsigned below = __ballot_sync(0xffffffffu, step * lane < n && c.cu[min(at, c.B - 1)] <= t);
    // cu ascends, so the lanes that vote are the first ones
    const int votes = __popc(below);
    if (votes == 0) return lo - 1;
    if (step == 1) return lo + votes - 1;
    const int64_t from = step * (votes - 1);
    lo += from;
    n = min(step, n - from);
  }
  return lo - 1;
}

// Where row t of the call goes: its page and position, page -1 where it has none.
struct Place {
  int page, pos;
};
__device__ __forceinline__ Place place_of(const KvView &c, int64_t t, int lane) {
  const int64_t b = sequence_of(c, t, lane);
  if (b < 0) return Place{-1, 0};
  int64_t t0, t1;
  c.range(b, t0, t1);
  if (t >= t1) return Place{-1, 0};
  const int pos = max(c.lengths[b], 0) - (int)(t1 - t);
  return Place{pos < 0 ? -1 : c.page(b, pos), max(pos, 0)};
}

// Word w (channels 8w .. 8w+7) of token t in a block's K or V codes.
__device__ __forceinline__ int k_word(int t, int w, int D) {
  return t * (D / 8) + (D == 64 ? 2 * (w & 3) + (w >> 2) : (w & ~15) + 4 * (w & 3) + ((w & 15) >> 2));
}
__device__ __forceinline__ int v_word(int t, int w) { return w * 16 + 4 * ((t >> 1) & 3) + (t & 1) + 2 * (t >> 3); }

// A warp's part of a token: threads of both tensors' words, K first.
__device__ __forceinline__ bool part_of(const KvView &c, int i, int &v, int &h, int &w) {
  const int words = c.D / 8, row = i / words;
  w = i % words;
  v = row >= c.HK;
  h = row - v * c.HK;
  return row < 2 * c.HK;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_store_kernel(const KvView c, const T *__restrict__ k, int64_t k_stride,
                                                            const T *__restrict__ v, int64_t v_stride, int parts) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), t = unit / parts;
  if (t >= c.T) return;
  const int per = c.gs / 8;  // threads of a group
  int is_v, h, w;
  const bool mine = part_of(c, (int)(unit - t * parts) * 32 + lane, is_v, h, w);
  float x[8] = {};
  if (mine) load8(is_v ? v + t * v_stride + (int64_t)h * c.D + 8 * w : k + t * k_stride + (int64_t)h * c.D + 8 * w, x);
  const Place at = place_of(c, t, lane);
  if (at.page < 0) return;
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
  for (int o = 1; o < per; o <<= 1) {
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!mine) return;
  lo = min_nan(max_nan(lo, -kLimit), kLimit);
  hi = min_nan(max_nan(hi, -kLimit), kLimit);
  const float s0 = __fmul_rn(__fsub_rn(hi, lo), (float)(1.0 / 15.0));
  const __nv_bfloat16 b16 = __float2bfloat16_rn(__fadd_rn(lo, 8.f * s0));
  const float b = __bfloat162float(b16);
  __nv_bfloat16 s16 = __float2bfloat16_rn(fmaxf(__fmul_rn(__fsub_rn(hi, b), (float)(1.0 / 7.0)), __fmul_rn(__fsub_rn(b, lo), 0.125f)));
  float s = __bfloat162float(s16);
  if (s < kTiny) s = 0.f;
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float xc = fminf(fmaxf(x[i], -kLimit), kLimit);
    const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(xc, b), inv), -8.f), 7.f);
    word |= (uint32_t)(__float2int_rn(q) + 8) << (4 * i);
  }
  uint32_t meta = __float_as_uint(b) & 0xFFFF0000u | (__float_as_uint(s) >> 16);
  if (lo != lo) {  // a NaN among them
    meta = 0x7FC07FC0u;
    word = 0x88888888u;
  }
  uint32_t *block = reinterpret_cast<uint32_t *>(c.block(at.page, h, at.pos));
  const int tok = at.pos & 15, G = c.D / c.gs, section = is_v ? 2 * c.D + 16 * G : 0;
  block[section + (is_v ? v_word(tok, w) : k_word(tok, w, c.D))] = word;
  if (w % per == 0) block[section + 2 * c.D + tok * G + w / per] = meta;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) kv_load_kernel(const KvView c, T *__restrict__ k, int64_t k_stride, T *__restrict__ v,
                                                           int64_t v_stride, int parts) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), t = unit / parts;
  if (t >= c.T) return;
  const Place at = place_of(c, t, lane);
  int is_v, h, w;
  if (!part_of(c, (int)(unit - t * parts) * 32 + lane, is_v, h, w)) return;
  float x[8] = {};
  if (at.page >= 0) {
    const uint32_t *block = reinterpret_cast<const uint32_t *>(c.block(at.page, h, at.pos));
    const int tok = at.pos & 15, G = c.D / c.gs, section = is_v ? 2 * c.D + 16 * G : 0;
    const uint32_t word = __ldg(block + section + (is_v ? v_word(tok, w) : k_word(tok, w, c.D)));
    const uint32_t meta = __ldg(block + section + 2 * c.D + tok * G + w / (c.gs / 8));
    const float s = meta_f32(meta, true), b = __uint_as_float(meta & 0xFFFF0000u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf((float)((int)((word >> (4 * i)) & 15u) - 8), s, b);  // the product is exact
  }
  store8(is_v ? v + t * v_stride + (int64_t)h * c.D + 8 * w : k + t * k_stride + (int64_t)h * c.D + 8 * w, x);
}

// warps per token
inline int parts_of(const KvView &c) { return (2 * c.HK * (c.D / 8) + 31) / 32; }

template <typename T>
cudaError_t store_t(const KvView &c, const void *k, int64_t ks, const void *v, int64_t vs, cudaStream_t st) {
  const int parts = parts_of(c);
  const int64_t blocks = (c.T * parts + kThreads / 32 - 1) / (kThreads / 32);
  kv_store_kernel<T><<<(unsigned)blocks, kThreads, 0, st>>>(c, static_cast<const T *>(k), ks, static_cast<const T *>(v), vs, parts);
  return cudaGetLastError();
}
template <typename T>
cudaError_t load_t(const KvView &c, void *k, int64_t ks, void *v, int64_t vs, cudaStream_t st) {
  const int parts = parts_of(c);
  const int64_t blocks = (c.T * parts + kThreads / 32 - 1) / (kThreads / 32);
  kv_load_kernel<T><<<(unsigned)blocks, kThreads, 0, st>>>(c, static_cast<T *>(k), ks, static_cast<T *>(v), vs, parts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_store(const KvView &c, const void *k, int64_t ks, const void *v, int64_t vs, q1_dtype t, cudaStream_t st) {
  if (t == Q1_BF16) return store_t<__nv_bfloat16>(c, k, ks, v, vs, st);
  if (t == Q1_F16) return store_t<__half>(c, k, ks, v, vs, st);
  return store_t<float>(c, k, ks, v, vs, st);
}
cudaError_t launch_kv_load(const KvView &c, void *k, int64_t ks, void *v, int64_t vs, q1_dtype t, cudaStream_t st) {
  if (t == Q1_BF16) return load_t<__nv_bfloat16>(c, k, ks, v, vs, st);
  if (t == Q1_F16) return load_t<__half>(c, k, ks, v, vs, st);
  return load_t<float>(c, k, ks, v, vs, st);
}

}  // namespace q1
