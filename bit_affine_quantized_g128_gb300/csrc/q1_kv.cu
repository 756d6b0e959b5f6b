// The 4-bit cache: K and V rows quantised into its pages, and read back.
//
// Per token, head and group of 64 or 128 channels, x = scale q + bias with q in
// -8..7: bias is the value that lets the codes -8 and 7 meet the least and the
// largest x, rounded to bf16, and scale the least that reaches both from there,
// rounded to bf16 (include/q1.h has the formula; every step is one fp32 operation,
// so the codes are the same everywhere).
//
// Both directions are streams, in two forms.  Few rows per sequence (decode): a thread
// owns a code word, 8 channels of a row; a group is 8 or 16 neighbouring threads, which
// find its least and largest value by shuffles; a warp stays with one token, so
// that finding its sequence and page is the warp's work, not each thread's.
// Many rows: a warp owns a block of 16 tokens of a head.  Four lanes share a token, lane t
// of them has channels 32 j + 8 t .. + 7, so a group is found in two shuffles, K's codes leave
// in the order in which they lie, 512 bytes per store, and V's go through shared memory,
// where words of a token become words of a channel.  Measured: 65536 tokens of 8 heads of 128 loaded in 55 us, 92 % of the copy
// rate (191 us by words); a prompt of 8192 stored and loaded again in 24 us, two launches (58 us by words); one token of a
// sequence 5.8 us, two launches.
#include <cuda_bf16.h>

#include <climits>
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

// The metadata word of a group with least and largest value lo, hi; its bias and the reciprocal of its scale.
__device__ __forceinline__ uint32_t group_meta(float lo, float hi, float &b, float &inv) {
  const bool bad = lo != lo;  // a NaN among them
  lo = min_nan(max_nan(lo, -kLimit), kLimit);
  hi = min_nan(max_nan(hi, -kLimit), kLimit);
  const float s0 = __fmul_rn(__fsub_rn(hi, lo), (float)(1.0 / 15.0));
  b = __bfloat162float(__float2bfloat16_rn(__fadd_rn(lo, 8.f * s0)));
  float s = __bfloat162float(__float2bfloat16_rn(
      fmaxf(__fmul_rn(__fsub_rn(hi, b), (float)(1.0 / 7.0)), __fmul_rn(__fsub_rn(b, lo), 0.125f))));
  if (s < kTiny) s = 0.f;
  inv = s > 0.f ? __frcp_rn(s) : 0.f;
  return bad ? 0x7FC07FC0u : (__float_as_uint(b) & 0xFFFF0000u) | (__float_as_uint(s) >> 16);
}
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], float b, float inv) {
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float xc = fminf(fmaxf(x[i], -kLimit), kLimit);
    const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(xc, b), inv), -8.f), 7.f);
    word |= (uint32_t)(__float2int_rn(q) + 8) << (4 * i);
  }
  return word;
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
  float b, inv;
  const uint32_t meta = group_meta(lo, hi, b, inv), word = lo != lo ? 0x88888888u : codes8(x, b, inv);
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

// ---- many rows: a warp per block of 16 tokens and head
// The block of a work item: sequence b's blocks are items t0 / 16 + 2 b and on, t0 its first row, which leaves room for
// each sequence's partial blocks without a sum over those before it.
struct BlockOf {
  int64_t t0;             // the sequence's first row, which stands for position pos0
  int pos0, end, page, p; // positions of the sequence end there; page (or -1) and first position (may be negative) of the block
};
__device__ __forceinline__ bool block_of(const KvView &c, int64_t item, int lane, BlockOf &k) {
  int64_t b;
  if (c.cu) {
    int64_t lo = 0, n = c.B;
    b = -1;
    while (n > 0) {
      const int64_t step = (n + 31) / 32, at = min(lo + step * lane, c.B - 1);
      const unsigned below =
          __ballot_sync(0xffffffffu, step * lane < n && min(max((int64_t)c.cu[at], (int64_t)0), c.T) / 16 + 2 * at <= item);
      const int votes = __popc(below);
      if (votes == 0) break;
      b = lo + step * (votes - 1);
      n = step == 1 ? 0 : min(step, n - step * (votes - 1));
      lo = b;
    }
    if (b < 0) return false;
  } else {
    const int64_t L = c.T / c.B;
    b = min(item * 16 / (L + 32), c.B - 1);
    while (b + 1 < c.B && (b + 1) * L / 16 + 2 * (b + 1) <= item) ++b;
    while (b > 0 && b * L / 16 + 2 * b > item) --b;
  }
  int64_t t1;
  c.range(b, k.t0, t1);
  k.end = max(c.lengths[b], 0);
  k.pos0 = k.end - (int)(t1 - k.t0);
  const int64_t block = (k.pos0 >> 4) + (item - (k.t0 / 16 + 2 * b));
  if (block < (k.pos0 >> 4) || block * 16 >= k.end) return false;
  k.p = (int)(block * 16);
  k.page = k.p < 0 ? -1 : c.page(b, k.p);
  return true;
}

template <int D, int GS>
struct Tile {
  static constexpr int G = D / GS, J = D / 32;  // groups; words of a token per lane
};

// Eight codes and a group's scale and bias -> values
__device__ __forceinline__ void values8(uint32_t word, uint32_t meta, float (&x)[8]) {
  const float s = meta_f32(meta, true), b = __uint_as_float(meta & 0xFFFF0000u);
#pragma unroll
  for (int i = 0; i < 8; ++i)  // 2^23 + q + 8 as bits; the difference and the product are exact
    x[i] = fmaf(__uint_as_float(0x4B000000u | ((word >> (4 * i)) & 15u)) - 8388616.f, s, b);
}

// The codes and metadata of one token's words (lane t of its four: channels 32 j + 8 t ..)
template <int D, int GS>
__device__ __forceinline__ void quantise(const float (&x)[D / 32][8], uint32_t (&word)[D / 32], uint32_t (&meta)[D / GS]) {
  constexpr int G = D / GS, JG = GS / 32;  // words of a group per lane
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float lo = x[g * JG][0], hi = lo;
#pragma unroll
    for (int j = g * JG; j < (g + 1) * JG; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo = min_nan(lo, x[j][i]);
        hi = max_nan(hi, x[j][i]);
      }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    float b, inv;
    meta[g] = group_meta(lo, hi, b, inv);
#pragma unroll
    for (int j = g * JG; j < (g + 1) * JG; ++j) word[j] = lo != lo ? 0x88888888u : codes8(x[j], b, inv);
  }
}

// APART: a warp for a block's K, one for its V.
template <typename T, int D, int GS, bool APART>
__global__ void __launch_bounds__(kThreads) kv_store_blocks_kernel(const KvView c, const T *__restrict__ k, int64_t k_stride,
                                                                   const T *__restrict__ v, int64_t v_stride, int64_t items) {
  constexpr int G = Tile<D, GS>::G, J = Tile<D, GS>::J;
  __shared__ uint32_t turn[kThreads / 32][2 * D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, t = lane & 3;
  const int64_t unit = ((int64_t)blockIdx.x * (kThreads / 32) + warp) >> APART, item = unit / c.HK;
  const int h = (int)(unit - item * c.HK);
  BlockOf at;
  if (item >= items || !block_of(c, item, lane, at) || at.page < 0) return;
  uint32_t *block = reinterpret_cast<uint32_t *>(c.block(at.page, h, at.p));
  const bool all = at.p >= at.pos0 && at.p + 16 <= at.end;  // every token of the block is among the rows
  auto section_of = [&](const int is_v) {
    const T *src = is_v ? v : k;
    const int64_t stride = is_v ? v_stride : k_stride;
    uint32_t *section = block + is_v * (2 * D + 16 * G);
    float x[2][J][8];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int p = at.p + 8 * half + (lane >> 2);
      const bool mine = p >= at.pos0 && p < at.end;
      const T *row = src + (at.t0 + (mine ? p - at.pos0 : 0)) * stride + (int64_t)h * D + 8 * t;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (mine) {
          load8(row + 32 * j, x[half][j]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[half][j][i] = 0.f;
        }
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int tok = 8 * half + (lane >> 2), p = at.p + tok;
      const bool mine = p >= at.pos0 && p < at.end;
      uint32_t word[J], meta[G];
      quantise<D, GS>(x[half], word, meta);
      if (mine && t < G) {
        uint32_t m = meta[0];
#pragma unroll
        for (int g = 1; g < G; ++g) m = t == g ? meta[g] : m;
        section[2 * D + tok * G + t] = m;
      }
      if (!is_v) {
        if (mine) {
          if constexpr (J == 2) {
            *reinterpret_cast<uint2 *>(section + tok * 8 + 2 * t) = make_uint2(word[0], word[1]);
          } else {
#pragma unroll
            for (int j = 0; j < J; j += 4)
              *reinterpret_cast<uint4 *>(section + tok * (D / 8) + 4 * j + 4 * t) =
                  make_uint4(word[j], word[j + 1], word[j + 2], word[j + 3]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int w = v_word(tok, 4 * j + t);
          if (all) turn[warp][w] = word[j];
          else if (mine) section[w] = word[j];
        }
      }
    }
    if (is_v && all) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
        reinterpret_cast<uint4 *>(section)[32 * i + lane] = reinterpret_cast<const uint4 *>(turn[warp])[32 * i + lane];
    }
  };
  if constexpr (APART) {
    section_of(warp & 1);
  } else {
    section_of(0);
    section_of(1);
  }
}

// Rows before the first sequence and behind the last, which no block has: zeros, by the call's warps in turn.
template <typename T>
__device__ __forceinline__ void zero_rest(const KvView &c, T *k, int64_t k_stride, T *v, int64_t v_stride, int64_t warp, int lane) {
  if (!c.cu) return;
  int64_t first, last, skip;
  c.range(0, first, skip);
  c.range(c.B - 1, skip, last);
  last = max(last, first);
  const int64_t n = first + (c.T - last), warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t i = warp; i < n; i += warps) {
    const int64_t t = i < first ? i : last + (i - first);
    for (int w = lane; w < c.HK * c.D / 8; w += 32) {
      const float none[8] = {};
      store8(k + t * k_stride + 8 * w, none);
      store8(v + t * v_stride + 8 * w, none);
    }
  }
}

// A block's rows, its K, its V or both
template <typename T, int D, int GS>
__device__ __forceinline__ void load_block(const KvView &c, const BlockOf &at, int h, int lane, bool of_k, bool of_v, T *k, int64_t k_stride,
                                           T *v, int64_t v_stride) {
  constexpr int G = Tile<D, GS>::G, J = Tile<D, GS>::J;
  const int t = lane & 3;
  const bool have = at.page >= 0;
  const uint32_t *block = reinterpret_cast<const uint32_t *>(c.block(max(at.page, 0), h, max(at.p, 0)));
  // K: a token for four lanes, as above
  uint32_t word[2][J], meta[2][G];
  uint4 vw[D / 64];
  uint32_t vm[4][G];
  const int w = lane >> 2;  // V: word w (and w + 8, ..) of tokens 2t, 2t + 1, 2t + 8, 2t + 9
  if (have && of_k) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int tok = 8 * half + w;
      if constexpr (J == 2) {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(block + tok * 8 + 2 * t));
        word[half][0] = u.x, word[half][1] = u.y;
      } else {
#pragma unroll
        for (int j = 0; j < J; j += 4) {
          const uint4 u = __ldg(reinterpret_cast<const uint4 *>(block + tok * (D / 8) + 4 * j + 4 * t));
          word[half][j] = u.x, word[half][j + 1] = u.y, word[half][j + 2] = u.z, word[half][j + 3] = u.w;
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) meta[half][g] = __ldg(block + 2 * D + tok * G + g);
    }
  }
  if (have && of_v) {
    const uint32_t *section = block + 2 * D + 16 * G;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) vw[i] = __ldg(reinterpret_cast<const uint4 *>(section) + (w + 8 * i) * 4 + t);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int g = 0; g < G; ++g) vm[j][g] = __ldg(section + 2 * D + (2 * t + (j & 1) + 8 * (j >> 1)) * G + g);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int p = at.p + 8 * half + w;
    if (!of_k || p < at.pos0 || p >= at.end) continue;
    T *row = k + (at.t0 + p - at.pos0) * k_stride + (int64_t)h * D + 8 * t;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float x[8] = {};
      if (have) values8(word[half][j], meta[half][32 * j / GS], x);
      store8(row + 32 * j, x);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int p = at.p + 2 * t + (j & 1) + 8 * (j >> 1);
    if (!of_v || p < at.pos0 || p >= at.end) continue;
    T *row = v + (at.t0 + p - at.pos0) * v_stride + (int64_t)h * D + 8 * w;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      float x[8] = {};
      if (have) values8(j == 0 ? vw[i].x : j == 1 ? vw[i].y : j == 2 ? vw[i].z : vw[i].w, vm[j][64 * i / GS], x);
      store8(row + 64 * i, x);
    }
  }
}

template <typename T, int D, int GS, bool APART>
__global__ void __launch_bounds__(kThreads, D == 256 ? 3 : 4) kv_load_blocks_kernel(const KvView c, T *__restrict__ k, int64_t k_stride, T *__restrict__ v,
                                                                  int64_t v_stride, int64_t items) {
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), unit = warp >> APART, item = unit / c.HK;
  BlockOf at;
  if (item < items && block_of(c, item, lane, at))
    load_block<T, D, GS>(c, at, (int)(unit - item * c.HK), lane, !APART || (warp & 1) == 0, !APART || (warp & 1) == 1, k, k_stride, v, v_stride);
  zero_rest(c, k, k_stride, v, v_stride, warp, lane);
}

// warps per token
inline int parts_of(const KvView &c) { return (2 * c.HK * (c.D / 8) + 31) / 32; }
// Blocks where sequences bring eight rows or more on average: below, most of a block's lanes would idle.
inline bool by_blocks(const KvView &c) { return c.T >= 8 * c.B; }

template <typename T, int D, int GS, bool LOAD, bool APART, typename P>
cudaError_t blocks_run(const KvView &c, int64_t items, P *k, int64_t ks, P *v, int64_t vs, cudaStream_t st) {
  const int64_t ctas = ((items * c.HK << APART) + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  if constexpr (LOAD)
    kv_load_blocks_kernel<T, D, GS, APART><<<(unsigned)ctas, kThreads, 0, st>>>(c, static_cast<T *>(k), ks, static_cast<T *>(v), vs, items);
  else
    kv_store_blocks_kernel<T, D, GS, APART>
        <<<(unsigned)ctas, kThreads, 0, st>>>(c, static_cast<const T *>(k), ks, static_cast<const T *>(v), vs, items);
  return cudaGetLastError();
}
// K and V by a warp each where warps are few, up to 10 of blocks per SM: what one does is then most of the call's time.  Store and
// load, us, by one warp and by two: 100 tokens of 8 heads of 128 in fp32 12.9 and 8.8, 1000 of 4 of 256 15.0 and 10.1, of 12 of 64
// 8.2 and 7.7; 8192 tokens of 4 of 256 (14 per SM) 26.3 and 28.5, of 12 of 64 (41) 19.0 and 21.2.
template <typename T, int D, int GS, bool LOAD, typename P>
cudaError_t blocks_t(const KvView &c, P *k, int64_t ks, P *v, int64_t vs, cudaStream_t st) {
  const int64_t items = c.T / 16 + 2 * c.B;
  return items * c.HK <= 10 * 152 ? blocks_run<T, D, GS, LOAD, true>(c, items, k, ks, v, vs, st)
                                  : blocks_run<T, D, GS, LOAD, false>(c, items, k, ks, v, vs, st);
}
template <typename T, bool LOAD, typename P>
cudaError_t run_t(const KvView &c, P *k, int64_t ks, P *v, int64_t vs, cudaStream_t st) {
  if (by_blocks(c)) {
    if (c.D == 64) return blocks_t<T, 64, 64, LOAD>(c, k, ks, v, vs, st);
    if (c.D == 128) return c.gs == 64 ? blocks_t<T, 128, 64, LOAD>(c, k, ks, v, vs, st) : blocks_t<T, 128, 128, LOAD>(c, k, ks, v, vs, st);
    return c.gs == 64 ? blocks_t<T, 256, 64, LOAD>(c, k, ks, v, vs, st) : blocks_t<T, 256, 128, LOAD>(c, k, ks, v, vs, st);
  }
  const int parts = parts_of(c);
  const int64_t ctas = (c.T * parts + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  if constexpr (LOAD) kv_load_kernel<T><<<(unsigned)ctas, kThreads, 0, st>>>(c, static_cast<T *>(k), ks, static_cast<T *>(v), vs, parts);
  else kv_store_kernel<T><<<(unsigned)ctas, kThreads, 0, st>>>(c, static_cast<const T *>(k), ks, static_cast<const T *>(v), vs, parts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_store(const KvView &c, const void *k, int64_t ks, const void *v, int64_t vs, q1_dtype t, cudaStream_t st) {
  if (t == Q1_BF16) return run_t<__nv_bfloat16, false>(c, k, ks, v, vs, st);
  if (t == Q1_F16) return run_t<__half, false>(c, k, ks, v, vs, st);
  return run_t<float, false>(c, k, ks, v, vs, st);
}
cudaError_t launch_kv_load(const KvView &c, void *k, int64_t ks, void *v, int64_t vs, q1_dtype t, cudaStream_t st) {
  if (t == Q1_BF16) return run_t<__nv_bfloat16, true>(c, k, ks, v, vs, st);
  if (t == Q1_F16) return run_t<__half, true>(c, k, ks, v, vs, st);
  return run_t<float, true>(c, k, ks, v, vs, st);
}

}  // namespace q1
