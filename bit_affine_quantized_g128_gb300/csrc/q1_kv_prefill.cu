// Attention over the 4-bit cache for many query rows (prompts and pieces of
// prompts), on the tcgen05 tensor cores.
//
// A CTA owns 256 rows (two tiles of 128; one for heads of 256) of a key head: row i of
// a sequence is its new token i / r, query head i mod r of the r that share the key
// head, so K and V are expanded once for all of them.  Tiles of 128 cached tokens (64)
// go by:
//   S = Q K^T                      both operands in shared memory, S in tensor memory
//   P = 2^(f S - M + 7) as fp16    a thread per row, back into S's columns
//   O += P V                       P from tensor memory, O stays in tensor memory
//
// Roles: warps 0-3 and 4-7 the softmax of a row tile each (heads of 256: 0-3, and 4-7
// expand K); warps 8-11 expand K and V; warp 12 issues the MMAs.
//
// Exactness.  K enters as scale q, which fp16 holds exactly (8 bits of scale, 4 of
// code), and the biases through one more k16 step: columns bias_g (twice per
// group) of K against the high and low fp16 half of the sum of Q's channels in group g.
// So S is exact up to fp32 sums.  Q is fp16, scaled by a power of two per row so that its
// largest value lies in [2^7, 2^8): bf16 and fp16 inputs are exact down to 2^-22 of
// that.  A 17th column of K is -inf where a token's page is missing, against 1 in Q.
// V is scale q + bias rounded to fp16 (2^-12), P is rounded to fp16 (2^-12); the sum
// of P is fp32 of the unrounded values.  M is a reference that moves when a logit exceeds it
// by more than 8 octaves; 2^7 keeps all of P that matters among fp16's normal values.
//
// The channels of a group of 8 are stored in the order 0 4 1 5 2 6 3 7, as a code word
// expands: in Q and K alike, where their order does not matter, and in O's columns, which
// the last step puts back.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "q1_internal.h"

namespace q1 {

__device__ unsigned int g_kv_err = 0;
__constant__ unsigned long long c_kv_wait_ns = 2000000000ull;
__constant__ int c_kv_stall = 0;

namespace {

constexpr float kNone = -3.0e38f;  // a maximum over nothing
constexpr float kSlack = 8.f;      // octaves by which a logit may exceed the reference
constexpr float kShift = 7.f;      // P is 2^kShift times the softmax's numerator
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512;

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint64_t *b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

struct Bars {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_ready[2], o_done[2], q_full, drain;
  uint32_t tmem_base;
  volatile int abort_flag, bad_v;  // a wait ran out; V has values beyond fp16
};

// Whether a wait gives up: its limit has run out, or another role has given up.
__device__ __noinline__ bool give_up(Bars *bars, unsigned long long since) {
  if (bars->abort_flag) return true;
  if (global_ns() - since <= c_kv_wait_ns) return false;
  bars->abort_flag = 1;
  atomicOr(&g_kv_err, 1u);
  return true;
}
// Bounded wait of a whole warp; one verdict for all its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *b, uint32_t parity, Bars *bars) {
  bool ok = mbar_try(b, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  const unsigned long long since = global_ns();
  for (uint32_t i = 1;; ++i) {
    ok = ok || mbar_try(b, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    if ((i & 31u) == 0 && __any_sync(0xffffffffu, give_up(bars, since))) return false;
  }
}
// the same for one thread
__device__ __forceinline__ bool wait_one(uint64_t *b, uint32_t parity, Bars *bars) {
  if (mbar_try(b, parity)) return true;
  const unsigned long long since = global_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try(b, parity)) return true;
    if ((i & 31u) == 0 && give_up(bars, since)) return false;
  }
}

// Operands of 128-byte rows, the 16-byte pieces of row r exchanged by XOR with r mod 8,
// 8-row groups 1024 bytes apart: rows along M or N, contraction along the row
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// or rows along the contraction, 64 columns of N per row, 64-column boxes `box` bytes apart
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t box) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(box >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
__device__ __forceinline__ uint32_t swz(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4)); }
// fp16 x fp16 -> fp32; bit 16: B with its rows along the contraction
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes, a lane per thread
__device__ __forceinline__ void tm_ld32(uint32_t t, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
        "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]),
        "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t t, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
      "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
      "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
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
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
__device__ __forceinline__ __half2 half2_of(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }
__device__ __forceinline__ uint32_t half2_bits(float a, float b) { return bits(__floats2half2_rn(a, b)); }

// Eight codes -> fp16 pairs (q_i, q_{i+4}), i = 0..3: an and-or puts the four bits
// under the exponent of 1024 (bits 0..3 count 1 there) or of 64 (bits 4..7 do).
__device__ __forceinline__ void expand(uint32_t w, __half2 (&h)[4]) {
  h[0] = __hsub2(half2_of((w & 0x000F000Fu) | 0x64006400u), half2_of(0x64086408u));  // 1024 + u - 1032
  h[1] = __hsub2(half2_of((w & 0x00F000F0u) | 0x54005400u), half2_of(0x54805480u));  // 64 + u - 72
  w >>= 8;
  h[2] = __hsub2(half2_of((w & 0x000F000Fu) | 0x64006400u), half2_of(0x64086408u));
  h[3] = __hsub2(half2_of((w & 0x00F000F0u) | 0x54005400u), half2_of(0x54805480u));
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// whether a group of V has a value that fp16 does not hold (none that was stored does, but for a NaN)
__device__ __forceinline__ bool beyond_fp16(uint32_t meta) {
  return !(fmaf(8.f, fabsf(__uint_as_float(meta << 16)), fabsf(__uint_as_float(meta & 0xFFFF0000u))) <= 65504.f);
}
template <int N>
__device__ __forceinline__ void ldg_words(const unsigned char *p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
  } else if constexpr (N == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i / 4);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
}

template <int D, int GS>
struct Prefill {
  static constexpr int G = D / GS, kBlock = 16 * (D + 8 * G);
  static constexpr int QT = D <= 128 ? 2 : 1, kRows = 128 * QT;  // row tiles of a CTA
  static constexpr int BN = D <= 128 ? 128 : 64;                 // cached tokens of a tile
  static constexpr int kQTile = (D / 64) * 128 * 128, kBox = BN * 128, kStage = (D / 64) * kBox;
  static constexpr int kHeader = 1024;
  static constexpr int kQ = kHeader, kK = kQ + QT * kQTile, kV = kK + 2 * kStage, kX = kV + 2 * kStage;
  // kX: the extra k16 step, 32 bytes of each row: K's stages 0 and 1, then Q's tiles
  static constexpr int kSmem = kX + 128 * 128 + 1024;
  static constexpr int kMajorWarps = QT == 2 ? 8 : 4;            // of the softmax
  // registers per thread after the split: softmax, expansion, MMAs (heads of 256 keep 128 each)
  static constexpr int kRegS = 192, kRegD = 88, kRegM = 40;
};
static_assert(sizeof(Bars) <= 1024, "header");

// A CTA's rows: those of `tile` of sequence b, and the positions that any of them sees.
struct Rows {
  int64_t t0;
  int rows, len, pos0, first, tiles;  // rows of the sequence, its tokens, position of its first row; first position, number of tiles
  template <int ROWS, int BN>
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
    int end = a.causal ? pos0 + row1 / r + 1 : (pos0 + row1 / r < 0 ? 0 : len);
    end = (int)min((int64_t)end, c.table_width << c.page_shift);
    const int begin = a.window ? (int)max((int64_t)pos0 + row0 / r - a.window + 1, (int64_t)0) : 0;
    first = begin / BN * BN;
    tiles = end > begin ? (end - first + BN - 1) / BN : 0;
    return true;
  }
};

// K and V of a tile for one warp of the four that expand it: BN / 64 blocks of 16 tokens.
template <int D, int GS>
struct Expander {
  using C = Prefill<D, GS>;
  static constexpr int G = C::G, W = C::BN / 64, KW = D / 32, VM = D / 64;
  struct KRegs {
    uint32_t code[W][2][KW], meta[W][2][G];
    int page[W];
  };
  struct VRegs {
    uint4 code[W][VM];
    uint32_t meta[W][4][G];
    int page[W];
  };
  const KvView &c;
  int64_t b;
  int hk, warp, lane;
  __device__ __forceinline__ int pos(int n0, int i) const { return n0 + 16 * (W * warp + i); }
  __device__ __forceinline__ int page_of(int n0, int i) const { return c.page(b, pos(n0, i)); }
  __device__ __forceinline__ const unsigned char *block(int page, int p) const {
    const int per = 1 << (c.page_shift - 4);
    return c.data + (((int64_t)page * c.HK + hk) * per + ((p >> 4) & (per - 1))) * C::kBlock;
  }
  // token of a half block whose 8 lanes of a quarter warp fall into different banks
  __device__ __forceinline__ int k_token(int half) const { return 8 * half + (lane >> 3) + (lane & 4); }
  __device__ __forceinline__ void fetch_k(int n0, const int (&page)[W], KRegs &r) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      r.page[i] = page[i];
      if (page[i] < 0) continue;
      const unsigned char *p = block(page[i], pos(n0, i));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = k_token(h);
        if constexpr (D == 64) {
          ldg_words(p + t * 32 + 8 * (lane & 3), r.code[i][h]);
        } else {
#pragma unroll
          for (int k = 0; k < D / 128; ++k) {
            uint32_t w[4];
            ldg_words(p + t * (D / 2) + 64 * k + 16 * (lane & 3), w);
#pragma unroll
            for (int j = 0; j < 4; ++j) r.code[i][h][4 * k + j] = w[j];
          }
        }
        ldg_words(p + 8 * D + t * G * 4, r.meta[i][h]);
      }
    }
  }
  // scale q into the tile at `dst`, the biases (twice) into the extra columns
  __device__ __forceinline__ void put_k(const KRegs &r, uint32_t dst, uint32_t extra, int stage) const {
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * (W * warp + i) + k_token(h);
        const bool have = r.page[i] >= 0;
        __half2 s[G];
        uint32_t bias[4] = {0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < G; ++k) {
          const uint32_t m = have ? r.meta[i][h][k] : 0u;
          s[k] = __float2half2_rn(__uint_as_float(m << 16));
          bias[k] = bits(__float2half2_rn(__uint_as_float(m & 0xFFFF0000u)));
        }
#pragma unroll
        for (int j = 0; j < KW; ++j) {
          __half2 v[4];
          expand(r.code[i][h][j], v);
          const __half2 f = s[32 * j / GS];
          sts4(dst + (j >> 1) * C::kBox + swz(row, 4 * (j & 1) + (lane & 3)), bits(__hmul2(v[0], f)), bits(__hmul2(v[1], f)),
               bits(__hmul2(v[2], f)), bits(__hmul2(v[3], f)));
        }
        if ((lane & 3) == 0) sts4(extra + swz(row, 2 * stage), bias[0], bias[1], bias[2], bias[3]);
        if ((lane & 3) == 1) sts4(extra + swz(row, 2 * stage + 1), have ? 0u : 0x0000FC00u, 0u, 0u, 0u);  // -inf
      }
  }
  __device__ __forceinline__ void fetch_v(int n0, const int (&page)[W], VRegs &r) const {
    const int w = lane & 7, t = lane >> 3;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      r.page[i] = page[i];
      if (page[i] < 0) continue;
      const unsigned char *p = block(page[i], pos(n0, i)) + 8 * D + 64 * G;
#pragma unroll
      for (int m = 0; m < VM; ++m) r.code[i][m] = __ldg(reinterpret_cast<const uint4 *>(p + (8 * m + w) * 64 + 16 * t));
#pragma unroll
      for (int k = 0; k < 4; ++k) ldg_words(p + 8 * D + (2 * t + (k & 1) + 8 * (k >> 1)) * G * 4, r.meta[i][k]);
    }
  }
  // scale q + bias; tokens with values beyond fp16 become 0, which no P of 0 turns into NaN, and are reported if they are
  // among the first `left` of the tile, the sequence's own
  __device__ __forceinline__ bool put_v(const VRegs &r, uint32_t dst, int left) const {
    const int w = lane & 7, t = lane >> 3;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 16 * (W * warp + i) + 2 * t + (k & 1) + 8 * (k >> 1);
        bool here = false;
#pragma unroll
        for (int n = 0; n < G; ++n) here |= beyond_fp16(r.meta[i][k][n]);
        const bool use = r.page[i] >= 0 && !here;
        bad |= here && r.page[i] >= 0 && row < left;
        __half2 s[G], o[G];
#pragma unroll
        for (int n = 0; n < G; ++n) {
          const uint32_t m = use ? r.meta[i][k][n] : 0u;
          s[n] = __float2half2_rn(__uint_as_float(m << 16));
          o[n] = __float2half2_rn(__uint_as_float(m & 0xFFFF0000u));
        }
#pragma unroll
        for (int m = 0; m < VM; ++m) {
          __half2 v[4];
          expand(k == 0 ? r.code[i][m].x : k == 1 ? r.code[i][m].y : k == 2 ? r.code[i][m].z : r.code[i][m].w, v);
          const int n = 64 * m / GS;
          sts4(dst + m * C::kBox + swz(row, w), bits(__hfma2(v[0], s[n], o[n])), bits(__hfma2(v[1], s[n], o[n])),
               bits(__hfma2(v[2], s[n], o[n])), bits(__hfma2(v[3], s[n], o[n])));
        }
      }
    return bad;
  }
};

// shared-memory stores of this warp, to the MMAs
__device__ __forceinline__ void publish_smem(uint64_t *bar, int lane) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

template <typename T, int D, int GS>
__global__ void __launch_bounds__(kThreads, 1) kv_prefill_kernel(const KvView c, const KvAttention a, int tiles) {
  using C = Prefill<D, GS>;
  using X = Expander<D, GS>;
  constexpr int G = C::G, QT = C::QT, BN = C::BN;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Bars *bars = reinterpret_cast<Bars *>(base);
  const uint32_t sm = smem_u32(base);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // the last tiles first: they see the most
  int64_t id = blockIdx.x;
  const int64_t heads = c.B * c.HK;
  const int tile0 = tiles - 1 - (int)(id / heads);
  id %= heads;
  const int hk = (int)(id % c.HK), r = a.HQ / c.HK;
  const int64_t b = id / c.HK;
  Rows rows;
  if (!rows.set<C::kRows, BN>(c, a, b, tile0)) return;

  auto init = [&](bool again) {
    if (tid == 0) {
      if (again)
        for (uint64_t *bar = bars->k_full; bar <= &bars->drain; ++bar)
          asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
      for (int s = 0; s < 2; ++s) {
        mbar_init(&bars->k_full[s], 4);
        mbar_init(&bars->v_full[s], 4);
        mbar_init(&bars->k_empty[s], 1);
        mbar_init(&bars->v_empty[s], 1);
        mbar_init(&bars->s_full[s], 1);
        mbar_init(&bars->p_ready[s], 4);
        mbar_init(&bars->o_done[s], 1);
      }
      mbar_init(&bars->q_full, C::kMajorWarps);
      mbar_init(&bars->drain, 1);
      bars->bad_v = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  };
  if (tid == 0) bars->abort_flag = 0;
  init(false);
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);

  // Every role goes through the CTA's tiles (one, unless the hint max_q was too small)
  // and meets the others at the end of each; false: no other tile.
  auto next = [&](int &tile) -> bool {
    fence_before();
    __syncthreads();
    fence_after();
    tile += tiles;
    if (bars->abort_flag || !rows.set<C::kRows, BN>(c, a, b, tile)) return false;
    init(true);
    __syncthreads();
    return true;
  };

  if (warp < C::kMajorWarps) {
    // ---------------- softmax: a row per thread
    if constexpr (QT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegS));
    const int q = warp >> 2, quarter = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16), to = tl + 256 + D * q;
    int tile = tile0;
    do {
      const int mine = tile * C::kRows + 128 * q + 32 * quarter + lane, row = min(mine, rows.rows - 1);
      const int64_t tok = rows.t0 + row / r;
      const int head = hk * r + row % r, pos = rows.pos0 + row / r;
      const int hi = pos < 0 ? -1 : a.causal ? pos : rows.len - 1, lo = a.window ? max(pos, 0) - a.window : -1;  // lo < j <= hi is seen
      const int hi_all = __reduce_min_sync(0xffffffffu, hi), lo_all = __reduce_max_sync(0xffffffffu, lo);
      float f;
      {
        const T *src = static_cast<const T *>(a.q) + tok * a.q_stride + (int64_t)head * D;
        float big = 0.f, sum[G] = {};
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll 4
          for (int i = g * GS / 8; i < (g + 1) * GS / 8; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float x = meta_f32(w[k], std::is_same<T, __nv_bfloat16>::value), y = meta_f32(w[k] >> 16, std::is_same<T, __nv_bfloat16>::value);
              big = fmaxf(big, fmaxf(fabsf(x), fabsf(y)));
              sum[g] += x + y;
            }
          }
        // the power of two that brings the largest into [2^7, 2^8)
        const int be = (int)(__float_as_uint(big) >> 23);
        const int e = be == 0 || be == 255 ? 0 : min(max(7 - (be - 127), -100), 100);
        const float up = a.scale < 0.f ? -pow2f(e) : pow2f(e);
        f = fmaxf(fabsf(a.scale) * kLog2e * pow2f(-e), 1e-30f);
        const uint32_t dst = sm + C::kQ + q * C::kQTile;
        const int rr = 32 * quarter + lane;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + i);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          float x[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[2 * k] = up * meta_f32(w[k], std::is_same<T, __nv_bfloat16>::value);
            x[2 * k + 1] = up * meta_f32(w[k] >> 16, std::is_same<T, __nv_bfloat16>::value);
          }
          sts4(dst + (i >> 3) * (128 * 128) + swz(rr, i & 7), half2_bits(x[0], x[4]), half2_bits(x[1], x[5]), half2_bits(x[2], x[6]),
               half2_bits(x[3], x[7]));
        }
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float x = up * sum[g];
          w[g] = half2_bits(x, x - __half2float(__float2half_rn(x)));
        }
        sts4(sm + C::kX + swz(rr, 4 + 2 * q), w[0], w[1], w[2], w[3]);
        sts4(sm + C::kX + swz(rr, 5 + 2 * q), 0x00003C00u, 0u, 0u, 0u);  // 1, against what is -inf for a missing token
        publish_smem(&bars->q_full, lane);
      }
      float M = kNone, L = 0.f;
      bool ok = true;
      for (int i = 0; i < rows.tiles; ++i) {
        const int buf = QT == 2 ? q : i & 1;
        const uint32_t ph = QT == 2 ? i & 1 : (i >> 1) & 1, ts = tl + 128 * buf;
        if (!(ok = wait_warp(&bars->s_full[buf], ph, bars))) break;
        fence_after();
        float x[BN];
#pragma unroll
        for (int k = 0; k < BN; k += 32) tm_ld32(ts + k, x + k);
        wait_ld();
        const int n0 = rows.first + i * BN;
        if (n0 <= lo_all || n0 + BN - 1 > hi_all) {
          const int h = hi - n0, l = lo - n0;
#pragma unroll
          for (int k = 0; k < BN; ++k) x[k] = k > l && k <= h ? x[k] : -INFINITY;
        }
        float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int k = 4; k < BN; k += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j) m4[j] = k + 4 + j < BN ? max3(m4[j], x[k + j], x[k + 4 + j]) : fmaxf(m4[j], x[k + j]);
        const float top = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * f;
        const bool grow = top > M + kSlack;
        if (__any_sync(0xffffffffu, grow)) {
          const float down = grow ? ex2(M - top) : 1.f;
          M = grow ? top : M;
          L *= down;
          if (i > 0) {
            // O's product of the tile before (the one before that is complete, for S followed it); the next waits for P
            if (!(ok = wait_warp(&bars->o_done[q], (i - 1) & 1, bars))) break;
            fence_after();
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
              float o[32];
              tm_ld32(to + k, o);
              wait_ld();
              uint32_t w[32];
#pragma unroll
              for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(o[j] * down);
              tm_st32(to + k, w);
            }
          }
        }
        const float neg = kShift - M;
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < BN; k += 64) {
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float u = ex2(fmaf(x[k + 2 * j], f, neg)), v = ex2(fmaf(x[k + 2 * j + 1], f, neg));
            s4[j & 1] += u;
            s4[2 + (j & 1)] += v;
            w[j] = half2_bits(u, v);
          }
          tm_st32(ts + k / 2, w);
        }
        L += (s4[0] + s4[1]) + (s4[2] + s4[3]);
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_ready[buf]);
      }
      // O's last product.  With one row tile the last two may be open (S of a tile only says that the product two tiles
      // before is complete), and o_done's parity cannot tell them apart: all MMAs, then.
      if (ok && rows.tiles > 0) ok = QT == 2 ? wait_warp(&bars->o_done[q], (rows.tiles - 1) & 1, bars) : wait_warp(&bars->drain, 0, bars);
      fence_after();
      float inv = L == 0.f ? 0.f : 1.f / L;
      if (ok && bars->bad_v) {
        // rows that see such a token become NaN
        for (int p = max(lo + 1, 0); p <= min(hi, (int)min((int64_t)rows.len, c.table_width << c.page_shift) - 1); ++p) {
          const int page = c.page(b, p);
          if (page < 0) continue;
          const unsigned char *blk = c.block(page, hk, p) + 16 * D + 64 * G + (p & 15) * G * 4;
          for (int g = 0; g < G; ++g)
            if (beyond_fp16(__ldg(reinterpret_cast<const uint32_t *>(blk) + g))) inv = __int_as_float(0x7fc00000);
        }
      }
      __syncwarp();
      const bool write = ok && mine < rows.rows;
      T *dst = static_cast<T *>(a.o) + tok * a.o_stride + (int64_t)head * D;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        float o[32];
        if (rows.tiles > 0) {
          tm_ld32(to + k, o);
          wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = inv == 0.f ? 0.f : o[j] * inv;
        if (write) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            // columns hold channels 0 4 1 5 2 6 3 7
            uint32_t w[4];
            if constexpr (std::is_same<T, __half>::value) {
              w[0] = half2_bits(o[j], o[j + 2]), w[1] = half2_bits(o[j + 4], o[j + 6]);
              w[2] = half2_bits(o[j + 1], o[j + 3]), w[3] = half2_bits(o[j + 5], o[j + 7]);
            } else {
              const __nv_bfloat162 h[4] = {__floats2bfloat162_rn(o[j], o[j + 2]), __floats2bfloat162_rn(o[j + 4], o[j + 6]),
                                           __floats2bfloat162_rn(o[j + 1], o[j + 3]), __floats2bfloat162_rn(o[j + 5], o[j + 7])};
#pragma unroll
              for (int n = 0; n < 4; ++n) w[n] = *reinterpret_cast<const uint32_t *>(&h[n]);
            }
            *reinterpret_cast<uint4 *>(dst + k + j) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (write && a.lse) a.lse[tok * a.HQ + head] = L == 0.f ? -INFINITY : (M + log2f(L) - kShift) * kLn2;
    } while (next(tile));
  } else if (warp < 12) {
    // ---------------- expansion of K and V
    if constexpr (QT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegD));
    const X x{c, b, hk, warp & 3, lane};
    int tile = tile0;
    do {
      typename X::KRegs kr;
      typename X::VRegs vr;
      const bool has_k = QT == 2 || warp < 8, has_v = QT == 2 || warp >= 8;
      int page[X::W], ahead[X::W];
      const int n = c_kv_stall ? 0 : rows.tiles;
#pragma unroll
      for (int i = 0; i < X::W; ++i) page[i] = n > 0 ? x.page_of(rows.first, i) : -1;
      if (n > 0) {
        if (has_k) x.fetch_k(rows.first, page, kr);
        if (has_v) x.fetch_v(rows.first, page, vr);
      }
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const int n0 = rows.first + i * BN, s = i & 1;
        const uint32_t ph = ((i >> 1) & 1) ^ 1;
#pragma unroll
        for (int k = 0; k < X::W; ++k) ahead[k] = i + 1 < n ? x.page_of(n0 + BN, k) : -1;
        if (has_k) {
          if (!wait_warp(&bars->k_empty[s], ph, bars)) break;
          x.put_k(kr, sm + C::kK + s * C::kStage, sm + C::kX, s);
          publish_smem(&bars->k_full[s], lane);
          x.fetch_k(n0 + BN, ahead, kr);
        }
        if (has_v) {
          if (!wait_warp(&bars->v_empty[s], ph, bars)) break;
          if (x.put_v(vr, sm + C::kV + s * C::kStage, rows.len - n0)) bars->bad_v = 1;
          publish_smem(&bars->v_full[s], lane);
          x.fetch_v(n0 + BN, ahead, vr);
        }
      }
    } while (next(tile));
  } else {
    if constexpr (QT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegM));
    int tile = tile0;
    do {
      if (warp == 12) {
        // ---------------- the MMAs, in units: row tile u mod QT of tile u / QT, S in buffer u mod 2
        if (elect_one()) {
          const int units = rows.tiles * QT;
          const uint32_t kq = sm + C::kQ, kx = sm + C::kX;
          bool ok = wait_one(&bars->q_full, 0, bars);
          auto scores = [&](int u) {
            const int i = u / QT, q = u % QT, s = i & 1;
            if (q == 0 && !wait_one(&bars->k_full[s], (i >> 1) & 1, bars)) return false;
            fence_after();
            const uint32_t d = tmem + 128 * (u & 1), ka = kq + q * C::kQTile, kb = sm + C::kK + s * C::kStage;
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              umma_ss(d, desc_k(ka + (k >> 2) * (128 * 128) + (k & 3) * 32), desc_k(kb + (k >> 2) * C::kBox + (k & 3) * 32),
                      idesc(128, BN, false), k > 0);
            umma_ss(d, desc_k(kx + 64 + 32 * q), desc_k(kx + 32 * s), idesc(128, BN, false), true);
            umma_commit(&bars->s_full[u & 1]);
            if (q == QT - 1) umma_commit(&bars->k_empty[s]);
            return true;
          };
          for (int u = 0; ok && u < 2 && u < units; ++u) ok = scores(u);
          for (int u = 0; ok && u < units; ++u) {
            const int i = u / QT, q = u % QT, s = i & 1;
            if (q == 0 && !(ok = wait_one(&bars->v_full[s], (i >> 1) & 1, bars))) break;
            if (!(ok = wait_one(&bars->p_ready[u & 1], (u >> 1) & 1, bars))) break;
            fence_after();
            const uint32_t vb = sm + C::kV + s * C::kStage, p = tmem + 128 * (u & 1);
#pragma unroll
            for (int k = 0; k < BN / 16; ++k)
              umma_ts(tmem + 256 + D * q, p + 8 * k, desc_mn(vb + k * 2048, C::kBox), idesc(128, D, true), i > 0 || k > 0);
            umma_commit(&bars->o_done[q]);
            if (q == QT - 1) umma_commit(&bars->v_empty[s]);
            if (u + 2 < units) ok = scores(u + 2);
          }
          umma_commit(&bars->drain);  // every MMA issued, complete before their memory is used again
        }
        __syncwarp();
        const unsigned long long since = global_ns();
        while (!mbar_try(&bars->drain, 0) && global_ns() - since < c_kv_wait_ns) {
        }
      }
    } while (next(tile));
  }
  if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

template <typename T, int D, int GS>
cudaError_t run(const KvView &c, const KvAttention &a, cudaStream_t st) {
  using C = Prefill<D, GS>;
  static std::atomic<uint64_t> ready{0};
  const int dev = current_device();
  if (not_done(ready, dev)) {
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, kv_prefill_kernel<T, D, GS>);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv_prefill_kernel<T, D, GS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    // the warps' shares come out of what the block was launched with
    if (e == cudaSuccess && C::QT == 2 && at.numRegs * 4 < 2 * C::kRegS + C::kRegD + C::kRegM) e = cudaErrorInvalidConfiguration;
    if (e != cudaSuccess) return e;
    mark_done(ready, dev);
  }
  const int r = a.HQ / c.HK;
  const int64_t tiles = (std::min(std::max<int64_t>(a.max_q, 1), c.T) * r + C::kRows - 1) / C::kRows, ctas = tiles * c.B * c.HK;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  kv_prefill_kernel<T, D, GS><<<(unsigned)ctas, kThreads, C::kSmem, st>>>(c, a, (int)tiles);
  return cudaGetLastError();
}
template <typename T>
cudaError_t run_t(const KvView &c, const KvAttention &a, cudaStream_t st) {
  if (c.D == 64) return run<T, 64, 64>(c, a, st);
  if (c.D == 128) return c.gs == 64 ? run<T, 128, 64>(c, a, st) : run<T, 128, 128>(c, a, st);
  return c.gs == 64 ? run<T, 256, 64>(c, a, st) : run<T, 256, 128>(c, a, st);
}

}  // namespace

cudaError_t launch_kv_prefill(const KvView &c, const KvAttention &a, q1_dtype t, cudaStream_t st) {
  return t == Q1_BF16 ? run_t<__nv_bfloat16>(c, a, st) : run_t<__half>(c, a, st);
}

cudaError_t set_kv_diagnostics(unsigned long long wait_ns, int stall) {
  cudaError_t e = cudaMemcpyToSymbol(c_kv_wait_ns, &wait_ns, sizeof(wait_ns));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(c_kv_stall, &stall, sizeof(stall));
  return e;
}

unsigned int read_and_clear_kv_errors(cudaStream_t st, cudaError_t *err) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_kv_err, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_kv_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess && v) e = cudaStreamSynchronize(st);
  *err = e;
  return v;
}

}  // namespace q1
