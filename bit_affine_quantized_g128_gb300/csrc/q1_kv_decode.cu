// Attention over the 4-bit cache for few query rows (single tokens, verifier
// windows; any number of rows in fp32).
//
// The rows that share a key head (its HQ / HK query heads times the sequence's new
// tokens) are the N = 8 columns of mma.sync tiles, 16 cached tokens its M rows:
//   S^T = K q^T,   O^T = V^T P^T.
// K's codes enter as fp16 integers, and scale and bias of a token's group are
// applied to the products: S = sum_groups (scale (codes . q) + bias sum q), so a
// cached value is exact however large its scale.  V's scale goes into P instead,
// O = sum_groups codes^T (P scale) + sum P bias.  The blocks' layout is what the
// fragments want: a lane reads its codes as 16-byte pieces, two neighbouring codes
// of a register are four bits apart from those of the next, and and-or with the
// exponent of 1024 (or 64) and a subtraction make them fp16 pairs.
//
// Each warp walks blocks of 16 tokens by itself, with its own running maximum, sum
// and accumulators (one pass); a context is split over the warps of a CTA and over
// CTAs, and joined in a fixed order.  The maximum is a reference that moves only when
// a logit exceeds it by more than 8 octaves, so most blocks need no reduction.
//
// What bounds it: issue.  A block of 16 tokens of 128 channels takes a warp 380 instructions (144 to expand the codes, 16 to 18
// MMAs, the rest softmax, scales and copies); 64 sequences of 8000 tokens, 40 heads over 8 of 128: 158 us, 3.7 TB/s, 55 % of the
// measured copy rate, 0.67 issued per scheduler and clock (0.83 on the busiest SM, as lengths differ), the pipe of the logic
// instructions the fullest.  One sequence of 200000, 24 heads over 4 of 256: 60 us, 55 %, 0.49 issued, as registers leave 8 warps
// on an SM.  One of 4096: 8.7 us, of which the launch and one CTA's chain of loads, blocks
// and join are most.
//
// Precision: q in bf16 or fp16 is one fp16 value scaled by a power of two per row
// (exact down to 2^-28 of the row's largest), fp32 a sum of two.  P scale is one fp16
// value for bf16 outputs (2^-11), a sum of two for fp16 and fp32 ones, with a power
// of two that follows the largest scale seen (of which it keeps 2^-30).  Sums are fp32.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kWarps = 8;      // of a CTA
constexpr int kStages = 4;     // blocks in flight per warp
constexpr float kNone = -3.0e38f;  // a maximum over nothing
constexpr float kSlack = 8.f;  // octaves by which a logit may exceed the reference
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// N words
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a) : "memory");
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = lds4(a + 4 * i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
}
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the 8 x 8 matrix of 16-bit values that the warp holds, transposed
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 half2_floats(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// Eight codes -> fp16 pairs (q_i, q_{i+4}), i = 0..3: an and-or puts the four bits
// under the exponent of 1024 (bits 0..3 count 1 there) or of 64 (bits 4..7 do).  The exponents come in registers: with
// both constants in the instruction it takes two.
struct Exponents {
  uint32_t a, b;
  __device__ __forceinline__ Exponents() {
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(a));
    asm volatile("mov.b32 %0, 0x54005400;" : "=r"(b));
  }
};
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t x) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(x));
  return r;
}
__device__ __forceinline__ void expand(uint32_t w, const Exponents &x, uint32_t (&h)[4]) {
  h[0] = hsub2(and_or<0x000F000Fu>(w, x.a), 0x64086408u);  // 1024 + u - 1032
  h[1] = hsub2(and_or<0x00F000F0u>(w, x.b), 0x54805480u);  // 64 + u - 72
  w >>= 8;
  h[2] = hsub2(and_or<0x000F000Fu>(w, x.a), 0x64086408u);
  h[3] = hsub2(and_or<0x00F000F0u>(w, x.b), 0x54805480u);
}
__device__ __forceinline__ float meta_scale(uint32_t m) { return __uint_as_float(m << 16); }
__device__ __forceinline__ float meta_bias(uint32_t m) { return __uint_as_float(m & 0xFFFF0000u); }

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
__device__ __forceinline__ void store4(T *p, float4 f) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4 *>(p) = f;
  } else if constexpr (std::is_same<T, __half>::value) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(half2_bits(f.x, f.y), half2_bits(f.z, f.w));
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f.x, f.y), b = __floats2bfloat162_rn(f.z, f.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
  }
}

// How a launch shares the work: row tiles and splits per sequence and head, and
// blocks of 16 tokens per chunk.  Split s does chunks s, s + splits, ... of its
// tile's context.  Up to kCluster splits are the CTAs of a cluster, which join through their shared
// memory; more go through the workspace and a second kernel.
struct Split {
  int tiles, splits, chunk;
  bool cluster; // the splits of a tile are a cluster
  float *part;  // [B][HK][tiles][splits][8 NT][D + 4]: unnormalised rows, then maximum and sum
};
constexpr int kCluster = 8;

__device__ __forceinline__ float4 load_shared_of(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [a];\n}\n"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// What a tile of rows sees: blocks [first, first + count) of the sequence.
struct Span {
  int64_t t0;    // the sequence's first row
  int rows, len, pos0, first, count;  // its rows (tokens times heads per key head), tokens, and first row's position
  template <int ROWS>
  __device__ __forceinline__ bool set(const KvView &c, const KvAttention &a, int64_t b, int tile) {
    int64_t t1;
    c.range(b, t0, t1);
    const int r = a.HQ / c.HK, n = (int)(t1 - t0);
    const int64_t all = (int64_t)n * r;
    if ((int64_t)tile * ROWS >= all) return false;
    rows = (int)all;
    len = max(c.lengths[b], 0);
    pos0 = len - n;
    const int row0 = tile * ROWS, row1 = min(row0 + ROWS, rows) - 1;
    const int64_t there = c.table_width << c.page_shift;
    int end = a.causal ? pos0 + row1 / r + 1 : (pos0 + row1 / r < 0 ? 0 : len);  // positions below it are seen
    end = (int)min((int64_t)end, there);
    const int begin = a.window ? (int)max((int64_t)pos0 + row0 / r - a.window + 1, (int64_t)0) : 0;
    first = begin >> 4;
    count = end > begin ? ((end + 15) >> 4) - first : 0;
    return true;
  }
};

template <typename T, int D, int GS, int NT>
struct Decode {
  static constexpr int kRows = 8 * NT, G = D / GS, kBlock = 16 * (D + 8 * G);
  static constexpr int QP = sizeof(T) == 4 ? 2 : 1;                                  // fp16 parts of q
  static constexpr int PP = std::is_same<T, __nv_bfloat16>::value ? 1 : 2;           // and of P scale
  static constexpr bool kQShared = NT * QP * D / 8 > 32;                             // q's fragments do not fit registers
  static constexpr int kQBytes = kQShared ? NT * QP * (D / 32) * 512 : 0;
  static constexpr int kStride = D + 8;                                              // floats of a joined row in shared memory
  static constexpr int kRing = kWarps * kStages * kBlock, kJoin = kWarps * kRows * kStride * 4;
  static constexpr int kOwn = kRows * (D + 4) * 4;                                    // this CTA's rows, for its cluster
  static constexpr int kSmem = kQBytes + (kRing > kJoin ? kRing : kJoin) + kOwn + kWarps * kRows * 8;
  static constexpr int kCtas = kSmem * 2 <= 220 * 1024 && NT * D <= 128 && QP == 1 ? 2 : 1;
};

template <typename T, int D, int GS, int NT, bool CLUSTER>
__global__ void __launch_bounds__(kWarps * 32, (Decode<T, D, GS, NT>::kCtas)) kv_decode_kernel(const KvView c, const KvAttention a,
                                                                                               const Split sp) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the joining kernel, where there is one
  using C = Decode<T, D, GS, NT>;
  constexpr int G = C::G, QP = C::QP, PP = C::PP, J = D / 32, H = D / 64, kRows = C::kRows;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), g = lane >> 2, t = lane & 3;
  const int split = (int)(blockIdx.x % sp.splits);
  int64_t id = blockIdx.x / sp.splits;
  const int64_t slot = id;
  const int tile0 = (int)(id % sp.tiles);
  id /= sp.tiles;
  const int hk = (int)(id % c.HK);
  const int64_t b = id / c.HK;
  const int r = a.HQ / c.HK;
  const uint32_t qs = smem_u32(smem), ring = qs + C::kQBytes + warp * (kStages * C::kBlock);
  float *join = reinterpret_cast<float *>(smem + C::kQBytes);
  float *sm_m = reinterpret_cast<float *>(smem + C::kSmem - kWarps * kRows * 8), *sm_l = sm_m + kWarps * kRows;
  float *own = sm_m - C::kOwn / 4;

  const Exponents exps;
  Span s{};
  // (tiles beyond those that the hint max_q foresaw are done whole by split 0)
  for (int tile = tile0; s.set<C::kRows>(c, a, b, tile); tile += sp.tiles) {
    const bool alone = sp.splits == 1 || tile != tile0;
    const int splits = alone ? 1 : sp.splits;
    if (alone && split > 0) return;
    const int chunks = (s.count + sp.chunk - 1) / sp.chunk;
    if (!(CLUSTER && !alone) && split >= chunks && split > 0) return;  // the joining kernel knows

    // ---- q: fragments, and per group the sum of its channels
    uint32_t q[C::kQShared ? 1 : NT][QP][C::kQShared ? 1 : J][4];
    float qsum[NT][G][2], f[NT][2];
    int hi[NT][2], lo[NT][2];  // positions lo < j <= hi are seen
    if constexpr (C::kQShared) __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = min(tile * kRows + 8 * nt + g, s.rows - 1);  // rows past the last repeat it
      const T *src = static_cast<const T *>(a.q) + (s.t0 + row / r) * a.q_stride + (int64_t)(hk * r + row % r) * D + 8 * t;
      float big = 0.f, sum[G] = {};
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float x[8];
        load8(src + 32 * j, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          big = fmaxf(big, fabsf(x[i]));
          sum[32 * j / GS] += x[i];
        }
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // the power of two that brings the largest into [2^14, 2^15)
      const int be = (int)(__float_as_uint(big) >> 23);
      const int e = be == 0 || be == 255 ? 0 : min(14 - (be - 127), 126);
      const float up = a.scale < 0.f ? -pow2f(e) : pow2f(e);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        sum[i] *= up;
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float x[8];
        load8(src + 32 * j, x);
        uint32_t w[QP][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = x[i] * up, v = x[i + 4] * up;
          w[0][i] = half2_bits(u, v);
          if constexpr (QP == 2) {
            const float2 h = half2_floats(w[0][i]);
            w[1][i] = half2_bits(u - h.x, v - h.y);
          }
        }
#pragma unroll
        for (int p = 0; p < QP; ++p) {
          if constexpr (C::kQShared) {
            if (warp == 0)
              *reinterpret_cast<uint4 *>(smem + ((nt * QP + p) * J + j) * 512 + lane * 16) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) q[nt][p][j][i] = w[p][i];
          }
        }
      }
      // this lane's columns 2t and 2t + 1 belong to the lanes of rows 2t and 2t + 1
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int from = 4 * (2 * t + k);
#pragma unroll
        for (int i = 0; i < G; ++i) qsum[nt][i][k] = __shfl_sync(0xffffffffu, sum[i], from);
        f[nt][k] = fmaxf(__shfl_sync(0xffffffffu, pow2f(-e), from) * (fabsf(a.scale) * kLog2e), 1e-30f);
        const int pos = s.pos0 + min(tile * kRows + 8 * nt + 2 * t + k, s.rows - 1) / r;
        hi[nt][k] = pos < 0 ? -1 : a.causal ? pos : s.len - 1;
        lo[nt][k] = a.window ? max(pos, 0) - a.window : -1;
      }
    }
    if constexpr (C::kQShared) __syncthreads();
    int hi_all = hi[0][0], lo_all = lo[0][0];  // positions lo_all < j <= hi_all are seen by every row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        hi_all = min(hi_all, hi[nt][k]);
        lo_all = max(lo_all, lo[nt][k]);
      }
    hi_all = __reduce_min_sync(0xffffffffu, hi_all);
    lo_all = __reduce_max_sync(0xffffffffu, lo_all);

    float O[NT][H][4][4] = {};         // [tile of 64 channels][channel mod 4]: channels 8g + i, 8g + i + 4 of two rows
    float M[NT][2], L[NT][2] = {}, bias[NT][G][2] = {};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) M[nt][0] = M[nt][1] = kNone;
    float vfac = pow2f(100);           // V's scales times this stay below 2^6

    // ---- the blocks of this warp: every kWarps-th of a chunk, kStages - 1 ahead
    const int page_blocks = c.page_shift - 4, mask = (1 << page_blocks) - 1, pages = (int)min(c.n_pages, (int64_t)INT32_MAX),
              width = (int)min(c.table_width, (int64_t)INT32_MAX);
    const int32_t *table = c.table + b * c.table_stride;
    const int64_t page_bytes = (int64_t)c.HK * C::kBlock << page_blocks;
    const unsigned char *data = c.data + ((int64_t)hk * C::kBlock << page_blocks) + lane * 16;
#pragma unroll 1
    for (int chunk = split; chunk < chunks; chunk += splits) {
    const int j0 = s.first + chunk * sp.chunk + warp;    // the first, in the sequence
    const int n = max(0, (s.first + min((chunk + 1) * sp.chunk, s.count) - j0 + kWarps - 1) / kWarps);
    int there = 0;                     // a bit per stage: its page exists
    int ahead = j0, page = n > 0 && (ahead >> page_blocks) < width ? table[ahead >> page_blocks] : -1;
    const int j1 = j0 + n * kWarps;
    auto fetch = [&](int stage) {
      const bool have = (unsigned)page < (unsigned)pages;
      there = (there & ~(1 << stage)) | (int)have << stage;
      if (have) {
        const unsigned char *src = data + page * page_bytes + (ahead & mask) * C::kBlock;
        const uint32_t dst = ring + stage * C::kBlock + lane * 16;
#pragma unroll
        for (int o = 0; o < C::kBlock; o += 512)
          if (o + 512 <= C::kBlock || o + lane * 16 < C::kBlock) copy16(dst + o, src + o);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      ahead += kWarps;
      page = ahead < j1 && (ahead >> page_blocks) < width ? table[ahead >> page_blocks] : -1;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    int stage = 0;
#pragma unroll 1
    for (int j = j0; j < j1; j += kWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();  // every lane's part is there, and every lane is done with the stage that is filled next
      fetch((stage + kStages - 1) & (kStages - 1));
      const bool have = there >> stage & 1;
      const uint32_t at = ring + stage * C::kBlock;
      const int p0 = (j << 4) + g;  // this lane's tokens: p0 and p0 + 8
      const bool whole = (j << 4) > lo_all && (j << 4) + 15 <= hi_all;
      stage = (stage + 1) & (kStages - 1);
      if (!__any_sync(0xffffffffu, have)) continue;  // (a vote: a branch of the whole warp)
      // S^T
      float x[NT][4] = {};
      {
        uint32_t k0[J], k1[J], m0[G], m1[G];
        if constexpr (J == 2) {
          lds_words(at + g * (D / 2) + 8 * t, k0);
          lds_words(at + (g + 8) * (D / 2) + 8 * t, k1);
        } else {
#pragma unroll
          for (int h = 0; h < J / 4; ++h) {
            const uint4 u = lds4(at + g * (D / 2) + 64 * h + 16 * t), v = lds4(at + (g + 8) * (D / 2) + 64 * h + 16 * t);
            k0[4 * h] = u.x, k0[4 * h + 1] = u.y, k0[4 * h + 2] = u.z, k0[4 * h + 3] = u.w;
            k1[4 * h] = v.x, k1[4 * h + 1] = v.y, k1[4 * h + 2] = v.z, k1[4 * h + 3] = v.w;
          }
        }
        lds_words(at + 8 * D + g * G * 4, m0);
        lds_words(at + 8 * D + (g + 8) * G * 4, m1);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          float acc[NT][4] = {};
#pragma unroll
          for (int j = i * GS / 32; j < (i + 1) * GS / 32; ++j) {
            uint32_t u[4], v[4];
            expand(k0[j], exps, u);
            expand(k1[j], exps, v);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int p = 0; p < QP; ++p) {
                if constexpr (C::kQShared) {
                  const uint4 w = lds4(qs + ((nt * QP + p) * J + j) * 512 + lane * 16);
                  mma16(acc[nt], u[0], v[0], u[1], v[1], w.x, w.y);
                  mma16(acc[nt], u[2], v[2], u[3], v[3], w.z, w.w);
                } else {
                  mma16(acc[nt], u[0], v[0], u[1], v[1], q[nt][p][j][0], q[nt][p][j][1]);
                  mma16(acc[nt], u[2], v[2], u[3], v[3], q[nt][p][j][2], q[nt][p][j][3]);
                }
              }
          }
          const float s0 = meta_scale(m0[i]), s1 = meta_scale(m1[i]), b0 = meta_bias(m0[i]), b1 = meta_bias(m1[i]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            x[nt][0] = fmaf(s0, acc[nt][0], fmaf(b0, qsum[nt][i][0], x[nt][0]));
            x[nt][1] = fmaf(s0, acc[nt][1], fmaf(b0, qsum[nt][i][1], x[nt][1]));
            x[nt][2] = fmaf(s1, acc[nt][2], fmaf(b1, qsum[nt][i][0], x[nt][2]));
            x[nt][3] = fmaf(s1, acc[nt][3], fmaf(b1, qsum[nt][i][1], x[nt][3]));
          }
        }
      }
      // the softmax's numerators; what some row does not see may hold anything
      uint32_t m0[G], m1[G];  // V's
      lds_words(at + 16 * D + 64 * G + g * G * 4, m0);
      lds_words(at + 16 * D + 64 * G + (g + 8) * G * 4, m1);
      uint32_t see = 0;  // a bit per value of x, where the block is not whole
      if (!whole) {
        bool seen0 = false, seen1 = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const bool v0 = p0 > lo[nt][k] && p0 <= hi[nt][k], v1 = p0 + 8 > lo[nt][k] && p0 + 8 <= hi[nt][k];
            x[nt][k] = v0 ? x[nt][k] : -INFINITY;
            x[nt][k + 2] = v1 ? x[nt][k + 2] : -INFINITY;
            see |= (uint32_t)v0 << (4 * nt + k) | (uint32_t)v1 << (4 * nt + k + 2);
            seen0 |= v0;
            seen1 |= v1;
          }
        // (the other lanes' rows see the same tokens)
        const unsigned any0 = __ballot_sync(0xffffffffu, seen0), any1 = __ballot_sync(0xffffffffu, seen1);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          m0[i] = (any0 >> (lane & 28) & 15u) ? m0[i] : 0u;
          m1[i] = (any1 >> (lane & 28) & 15u) ? m1[i] : 0u;
        }
      }
      float y[NT][4], over = kNone, top = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[nt][k] = fmaf(x[nt][k], f[nt][k & 1], -M[nt][k & 1]);
        over = max3(max3(over, y[nt][0], y[nt][1]), y[nt][2], y[nt][3]);
      }
#pragma unroll
      for (int i = 0; i < G; ++i) top = max3(top, fabsf(meta_scale(m0[i])), fabsf(meta_scale(m1[i])));
      if (__any_sync(0xffffffffu, over > kSlack || top * vfac > 64.f)) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float keep = 1.f;
        if (top * vfac > 64.f) {  // its exponent to [2^5, 2^6)
          const float next = pow2f(max(min(5 - ((int)(__float_as_uint(top) >> 23) - 127), 100), -100));
          keep = next * (1.f / vfac);
          vfac = next;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx = fmaxf(x[nt][k], x[nt][k + 2]);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = fmaxf(mx * f[nt][k], M[nt][k]);
            const float down = ex2(M[nt][k] - mx);
            M[nt][k] = mx;
            L[nt][k] *= down;
            y[nt][k] = fmaf(x[nt][k], f[nt][k], -mx);
            y[nt][k + 2] = fmaf(x[nt][k + 2], f[nt][k], -mx);
#pragma unroll
            for (int i = 0; i < G; ++i) bias[nt][i][k] *= down;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                O[nt][h][i][k] *= down * keep;
                O[nt][h][i][k + 2] *= down * keep;
              }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          x[nt][k] = ex2(y[nt][k]);
          x[nt][k + 2] = ex2(y[nt][k + 2]);
          L[nt][k] += x[nt][k] + x[nt][k + 2];
        }
      // O^T
      uint32_t pb[NT][G][PP][2];
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const float s0 = meta_scale(m0[i]) * vfac, s1 = meta_scale(m1[i]) * vfac, b0 = meta_bias(m0[i]), b1 = meta_bias(m1[i]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float y[4] = {x[nt][0] * s0, x[nt][1] * s0, x[nt][2] * s1, x[nt][3] * s1};
          if (whole) {
#pragma unroll
            for (int k = 0; k < 2; ++k) bias[nt][i][k] = fmaf(b0, x[nt][k], fmaf(b1, x[nt][k + 2], bias[nt][i][k]));
          } else {  // a token that other rows see may have a NaN; one that this row sees shows it whatever its weight
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = see >> (4 * nt + k) & 1u ? y[k] : 0.f;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              bias[nt][i][k] += (see >> (4 * nt + k) & 1u ? x[nt][k] * b0 : 0.f) + (see >> (4 * nt + k + 2) & 1u ? x[nt][k + 2] * b1 : 0.f);
          }
          const uint32_t h0 = half2_bits(y[0], y[1]), h1 = half2_bits(y[2], y[3]);
          pb[nt][i][0][0] = movmatrix(h0);
          pb[nt][i][0][1] = movmatrix(h1);
          if constexpr (PP == 2) {
            const float2 u0 = half2_floats(h0), u1 = half2_floats(h1);
            pb[nt][i][1][0] = movmatrix(half2_bits(y[0] - u0.x, y[1] - u0.y));
            pb[nt][i][1][1] = movmatrix(half2_bits(y[2] - u1.x, y[3] - u1.y));
          }
        }
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const uint4 w = lds4(at + 8 * D + 64 * G + (g + 8 * h) * 64 + 16 * t);
        // tokens 2t, 2t + 1 and 2t + 8, 2t + 9: channels 0..3 of the word, and 4..7
        uint32_t x01[4], x89[4], y01[4], y89[4];
        expand(__byte_perm(w.x, w.y, 0x5410), exps, x01);
        expand(__byte_perm(w.x, w.y, 0x7632), exps, y01);
        expand(__byte_perm(w.z, w.w, 0x5410), exps, x89);
        expand(__byte_perm(w.z, w.w, 0x7632), exps, y89);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            // fp32: a block at a time, as the tensor cores cut their sums (not round them), which adds up over a long context
            float sum[4] = {};
            float(&to)[4] = sizeof(T) == 4 ? sum : O[nt][h][i];
#pragma unroll
            for (int p = 0; p < PP; ++p)
              mma16(to, x01[i], y01[i], x89[i], y89[i], pb[nt][64 * h / GS][p][0], pb[nt][64 * h / GS][p][1]);
            if constexpr (sizeof(T) == 4)
#pragma unroll
              for (int k = 0; k < 4; ++k) O[nt][h][i][k] += sum[k];
          }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    }

    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) {
          L[nt][k] += __shfl_xor_sync(0xffffffffu, L[nt][k], o);
#pragma unroll
          for (int i = 0; i < G; ++i) bias[nt][i][k] += __shfl_xor_sync(0xffffffffu, bias[nt][i][k], o);
        }
      }
    __syncthreads();  // the ring becomes the join's buffer
    const float back = 1.f / vfac;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = 8 * nt + 2 * t + k;
        if (g == 0) {
          sm_m[warp * kRows + row] = M[nt][k];
          sm_l[warp * kRows + row] = L[nt][k];
        }
        float *dst = join + (warp * kRows + row) * C::kStride + 8 * g;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float bv = bias[nt][64 * h / GS][k];
#pragma unroll
          for (int u = 0; u < 2; ++u)
            *reinterpret_cast<float4 *>(dst + 64 * h + 4 * u) =
                make_float4(fmaf(O[nt][h][0][k + 2 * u], back, bv), fmaf(O[nt][h][1][k + 2 * u], back, bv),
                            fmaf(O[nt][h][2][k + 2 * u], back, bv), fmaf(O[nt][h][3][k + 2 * u], back, bv));
        }
      }
    __syncthreads();
    const int valid = min(kRows, s.rows - tile * kRows);
    for (int i = threadIdx.x; i < valid * (D / 4); i += kWarps * 32) {
      const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
      float m = kNone, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm_m[w * kRows + row]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float z = ex2(sm_m[w * kRows + row] - m);
        const float4 v = *reinterpret_cast<const float4 *>(join + (w * kRows + row) * C::kStride + d);
        l = fmaf(z, sm_l[w * kRows + row], l);
        o.x = fmaf(z, v.x, o.x);
        o.y = fmaf(z, v.y, o.y);
        o.z = fmaf(z, v.z, o.z);
        o.w = fmaf(z, v.w, o.w);
      }
      if (alone) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int all = tile * kRows + row, head = hk * r + all % r;
        const int64_t tok = s.t0 + all / r;
        store4(static_cast<T *>(a.o) + tok * a.o_stride + (int64_t)head * D + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (d == 0 && a.lse) a.lse[tok * a.HQ + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      } else if constexpr (CLUSTER) {
        *reinterpret_cast<float4 *>(own + row * (D + 4) + d) = o;
        if (d == 0) *reinterpret_cast<float2 *>(own + row * (D + 4) + D) = make_float2(m, l);
      } else {
        float *dst = sp.part + ((slot * splits + split) * kRows + row) * (D + 4);
        *reinterpret_cast<float4 *>(dst + d) = o;
        if (d == 0) *reinterpret_cast<float2 *>(dst + D) = make_float2(m, l);
      }
    }
    if constexpr (CLUSTER) {
      if (!alone) {
        // the cluster's CTAs share the rows' values among them
        cluster_sync();
        const uint32_t base = smem_u32(own);
        for (int i = split * kWarps * 32 + threadIdx.x; i < valid * (D / 4); i += splits * kWarps * 32) {
          const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
          float m = kNone, l = 0.f, ms[kCluster], ls[kCluster];
#pragma unroll
          for (int k = 0; k < kCluster; ++k)
            if (k < splits) {
              const float4 v = load_shared_of(base + (row * (D + 4) + D) * 4, k);
              ms[k] = v.x;
              ls[k] = v.y;
              m = fmaxf(m, v.x);
            }
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kCluster; ++k)
            if (k < splits) {
              const float z = ex2(ms[k] - m);
              const float4 v = load_shared_of(base + (row * (D + 4) + d) * 4, k);
              l = fmaf(z, ls[k], l);
              o.x = fmaf(z, v.x, o.x);
              o.y = fmaf(z, v.y, o.y);
              o.z = fmaf(z, v.z, o.z);
              o.w = fmaf(z, v.w, o.w);
            }
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int all = tile * kRows + row, head = hk * r + all % r;
          const int64_t tok = s.t0 + all / r;
          store4(static_cast<T *>(a.o) + tok * a.o_stride + (int64_t)head * D + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
          if (d == 0 && a.lse) a.lse[tok * a.HQ + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
        cluster_sync();  // no CTA leaves while another reads its rows
      }
    }
    __syncthreads();  // before the next tile's blocks come
  }
}

// Joins the splits of a row; a CTA per row, its threads in groups that take every so many-th split.
constexpr int kJoinThreads = 256;
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) kv_join_kernel(const KvView c, const KvAttention a, const Split sp) {
  constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
  __shared__ float4 part[kGroups][kLanes];
  __shared__ float2 ml[kGroups];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t slot = blockIdx.x / ROWS;
  const int row = (int)(blockIdx.x - slot * ROWS), tile = (int)(slot % sp.tiles);
  const int64_t id = slot / sp.tiles, b = id / c.HK;
  const int hk = (int)(id - b * c.HK), r = a.HQ / c.HK, group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
  Span s{};
  if (!s.set<ROWS>(c, a, b, tile) || tile * ROWS + row >= s.rows) return;
  const int n = max(1, min(sp.splits, (s.count + sp.chunk - 1) / sp.chunk));
  const float *src = sp.part + (slot * sp.splits * ROWS + row) * (D + 4);
  const int64_t step = (int64_t)ROWS * (D + 4);
  float m = kNone, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float m2, float l2, float4 v) {
    const float mx = fmaxf(m, m2), z = ex2(m - mx), z2 = ex2(m2 - mx);
    m = mx;
    l = fmaf(z, l, z2 * l2);
    o.x = fmaf(z, o.x, z2 * v.x);
    o.y = fmaf(z, o.y, z2 * v.y);
    o.z = fmaf(z, o.z, z2 * v.z);
    o.w = fmaf(z, o.w, z2 * v.w);
  };
  for (int i = group; i < n; i += 4 * kGroups) {
    float2 q[4];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * kGroups < n) {
        q[k] = *reinterpret_cast<const float2 *>(src + (i + k * kGroups) * step + D);
        v[k] = *reinterpret_cast<const float4 *>(src + (i + k * kGroups) * step + 4 * lane);
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * kGroups < n) add(q[k].x, q[k].y, v[k]);
  }
  part[group][lane] = o;
  if (lane == 0) ml[group] = make_float2(m, l);
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k)
    if (k < n) add(ml[k].x, ml[k].y, part[k][lane]);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int all = tile * ROWS + row, head = hk * r + all % r;
  const int64_t tok = s.t0 + all / r;
  store4(static_cast<T *>(a.o) + tok * a.o_stride + (int64_t)head * D + 4 * lane, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (lane == 0 && a.lse) a.lse[tok * a.HQ + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Rows per tile: 8 where the rows of a key head fit it, else 16 (a block's codes
// are expanded once for both halves).
inline int rows_of(const KvView &c, const KvAttention &a) { return std::max<int64_t>(a.max_q, 1) * (a.HQ / c.HK) <= 8 ? 8 : 16; }

Split plan(const KvView &c, const KvAttention &a, q1_dtype t) {
  const bool fp32 = t == Q1_F32;
  const int rows = rows_of(c, a), r = a.HQ / c.HK;
  Split s;
  s.tiles = (int)kv_tiles_of_grid(c, (std::min(std::max<int64_t>(a.max_q, 1), c.T) * r + rows - 1) / rows, c.T * r, rows);
  int64_t seen = std::max<int64_t>(a.max_len, 1);
  if (a.window) seen = std::min<int64_t>(seen, (int64_t)a.window + rows + 15);
  const int64_t blocks = (seen + 15) / 16, work = c.B * c.HK * s.tiles;
  // CTAs for one, two or four rounds of the GPU: the more, the better ragged batches even out, as long as each has 16, 64
  // or 128 blocks to do.
  // (as Decode::kCtas has it: fp32 rows and large tiles take an SM for a CTA)
  const int64_t slots = 152 * (!fp32 && c.D * rows <= 128 * 8 ? 2 : 1);
  int64_t want = std::min(slots / work, blocks / 16);
  if (blocks / std::max<int64_t>(2 * slots / work, 1) >= 64) want = 2 * slots / work;
  if (blocks / std::max<int64_t>(4 * slots / work, 1) >= 128) want = 4 * slots / work;
  // The tensor cores cut what they add to O instead of rounding it, fp16 rows' two parts of P at 2^-27 of O per token of a warp, where
  // all are of one sign: so a CTA's warps have at most 2^18 tokens (a quarter of a step).  Half a step of bf16 is more than 2^21
  // tokens lose with one part, and fp32 rows have their sums added up apart.
  want = std::max(want, std::min<int64_t>((blocks - 1) >> (t == Q1_F16 ? 14 : 17), 63) + 1);
  // Heads of 64: 9 to 16 splits are rather 8, in a cluster, whose join saves more than twice the blocks cost (12 heads over 4096
  // tokens 7.1 us, 8.4 with 16; heads of 128 and 256: 9.1 and 11.0, 8.4 and 9.4 with 16; clusters of 16 were slower yet).
  if (c.D == 64 && want > kCluster && want <= 2 * kCluster && work * kCluster <= slots) want = kCluster;
  s.chunk = (int)(((blocks + std::max<int64_t>(want, 1) - 1) / std::max<int64_t>(want, 1) + kWarps - 1) / kWarps * kWarps);
  s.splits = (int)((blocks + s.chunk - 1) / s.chunk);
  // (only where all run at once: a CTA whose split has no tokens would hold its place until the others are done)
  s.cluster = s.splits > 1 && s.splits <= kCluster && work * s.splits <= slots;
  s.part = nullptr;
  return s;
}

template <typename T, int D, int GS, int NT, bool CLUSTER>
cudaError_t run_c(const KvView &c, const KvAttention &a, const Split &s, cudaStream_t st) {
  using C = Decode<T, D, GS, NT>;
  static std::atomic<uint64_t> ready{0};
  const int dev = current_device();
  if (not_done(ready, dev)) {
    const cudaError_t e = cudaFuncSetAttribute(kv_decode_kernel<T, D, GS, NT, CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    mark_done(ready, dev);
  }
  const int64_t tiles = c.B * c.HK * s.tiles, ctas = tiles * s.splits;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(kWarps * 32, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  if (CLUSTER) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)s.splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_decode_kernel<T, D, GS, NT, CLUSTER>, c, a, s);
  if (e != cudaSuccess || CLUSTER || s.splits == 1) return e;
  if (tiles * 8 * NT > INT32_MAX) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3((unsigned)(tiles * 8 * NT), 1, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<T, D, 8 * NT>, c, a, s);
}

template <typename T, int D, int GS, int NT>
cudaError_t run(const KvView &c, const KvAttention &a, const Split &s, cudaStream_t st) {
  return s.cluster ? run_c<T, D, GS, NT, true>(c, a, s, st) : run_c<T, D, GS, NT, false>(c, a, s, st);
}
template <typename T, int D, int GS>
cudaError_t run_rows(const KvView &c, const KvAttention &a, const Split &s, cudaStream_t st) {
  return rows_of(c, a) == 8 ? run<T, D, GS, 1>(c, a, s, st) : run<T, D, GS, 2>(c, a, s, st);
}
template <typename T>
cudaError_t run_t(const KvView &c, const KvAttention &a, const Split &s, cudaStream_t st) {
  if (c.D == 64) return run_rows<T, 64, 64>(c, a, s, st);
  if (c.D == 128) return c.gs == 64 ? run_rows<T, 128, 64>(c, a, s, st) : run_rows<T, 128, 128>(c, a, s, st);
  return c.gs == 64 ? run_rows<T, 256, 64>(c, a, s, st) : run_rows<T, 256, 128>(c, a, s, st);
}

}  // namespace

size_t kv_decode_workspace_bytes(const KvView &c, const KvAttention &a, q1_dtype t) {
  const Split s = plan(c, a, t);
  if (s.splits == 1 || s.cluster) return 0;
  return (size_t)(c.B * c.HK) * s.tiles * s.splits * rows_of(c, a) * (c.D + 4) * sizeof(float);
}

cudaError_t launch_kv_decode(const KvView &c, const KvAttention &a, q1_dtype t, void *workspace, cudaStream_t st) {
  Split s = plan(c, a, t);
  s.part = static_cast<float *>(workspace);
  if (t == Q1_BF16) return run_t<__nv_bfloat16>(c, a, s, st);
  if (t == Q1_F16) return run_t<__half>(c, a, s, st);
  return run_t<float>(c, a, s, st);
}

}  // namespace q1
