// Gated delta rule in chunks of 64 tokens (prefill).
//
// With G the inclusive sum of g inside a chunk, gamma = exp(G), the tokens of a
// chunk that starts from the state S satisfy, all at once,
//   A_ij = beta_i exp(G_i - G_j) (k_i . k_j)  (i > j),  T = (I + A)^-1 diag(beta)
//   R    = V - diag(gamma) K S                          [64][DV]
//   U    = T R
//   O    = scale (diag(gamma) Q S + P U),   P_ij = exp(G_i - G_j) (q_i . k_j)  (i >= j)
//   S   <- gamma_C S + K^T diag(exp(G_C - G)) U
// and P U = (P T) R.  T and P' = scale P T depend on the keys, queries and
// gates only: a first kernel computes them for all chunks at once, and a second
// one, a CTA per sequence and head, walks the chunks with matrix products only.
//
// Operand precision.  The state is fp32 and goes through one product per
// chunk, so operands rounded to 16 bits once would leave it 2^-9 or 2^-12 off.
// Nor is o served by them, though it is rounded to 16 bits in the end: where a
// token overwrites what the state held under its key, Q S and P' R cancel, and what
// is left can be any number of times smaller than both.  So every fp32 operand
// (S, R, the scaled U, T, P') is a sum of two fp16 values, high and low, 22
// bits of each value together, scaled by a power of two (per row of the operand,
// or per tile) so that the largest lies in [2^14, 2^15); what lies 2^-17 or
// more below it keeps fewer bits, down to 2^-39 of it.  Products are exact in fp32
// up to its own rounding; those of two low parts are left out (2^-21).  Keys and
// queries enter as single fp16 values, scaled per row: bf16 and fp16 inputs are exact
// in them down to 2^-28 of the row's largest value.
#include <cuda_bf16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "q1_internal.h"

namespace q1 {

__device__ unsigned int g_delta_err = 0;
__constant__ unsigned long long c_delta_wait_ns = 2000000000ull;
__constant__ int c_delta_stall = 0;

namespace {

constexpr int kC = 64;                       // tokens of a chunk
constexpr int kTile = kC * kC * 2;           // bytes of a 64 x 64 fp16 tile
constexpr int kScalars = 3 * kC + 16;        // floats: a, c, b, then gamma_C and P's scale
constexpr int kScalarBytes = kScalars * 4;
constexpr int kTiles = 4 * kTile;            // T high, T low, P' high, P' low

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

// A chunk's place in the workspace: sequence b's chunks start at
// cu[b] / 64 + b.  That leaves room for each sequence's last partial chunk
// without a sum over the sequences before it, and stays below T / 64 + B + 1.
__device__ __forceinline__ int64_t chunk_base(int64_t t0, int64_t b) { return t0 / kC + b; }

struct ChunkPlaces {
  unsigned char *kq;  // [chunks][HK] K tile, Q tile: 64 x DK fp16 each
  unsigned char *tp;  // [chunks][HV] T high, T low, P' high, P' low: 64 x 64 fp16 each
  float *sc;          // [chunks][HV][kScalars]
  // between slabs, where there are any (batches that the chain does not sort):
  // the states [B][HV][DK][DV], and per 16 state columns [B][HV][DV / 16]
  // whether a wait for them ran out
  float *carry;
  int *failed;
};
// The chunks [first, end) of every sequence, which one launch of each kernel
// does; more: another slab follows, whose chunk kernel may run beside this one's
// chain.
struct Slab {
  int first, end, more;
};
__host__ __device__ inline int64_t chunk_places(int64_t T, int64_t B) { return T / kC + B + 1; }

// Tiles are stored as the products read them from shared memory: rows of 128
// bytes (64 values), the 16-byte pieces of row r exchanged by XOR with r mod 8;
// wider tiles are 64-column boxes one after another.
__device__ __forceinline__ uint32_t swz(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4)); }

// 2^e as a float, and the e that brings a value of size mx into [2^14, 2^15), at
// most 60 either way (sums of two stay exponents of fp32 values).  Infinite and NaN
// sizes take e = 0.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ int scale_exp(float mx) {
  const int e = (int)((__float_as_uint(mx) >> 23) & 0xFF);
  return e == 255 ? 0 : min(max(14 - (e - 127), -60), 60);
}

// The e that brings the root of a sum of squares into [2^13, 2^15)
__device__ __forceinline__ int root_exp(float ss) {
  const int e = (int)((__float_as_uint(ss) >> 23) & 0xFF);
  if (e == 0 || e == 255) return 0;
  return 14 - ((e - 126) >> 1);
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// (a, b) as fp16 high parts, and what they leave as fp16 low parts
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = half2_bits(a - f.x, b - f.y);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---- pairs of fp32 values: neighbouring columns of a fragment (plain fp32
// instructions: the two-wide ones took 3.6 clocks a warp, a single one 1.2)
struct f2 {
  float a, b;
};
__device__ __forceinline__ f2 pk(float a, float b) { return f2{a, b}; }
__device__ __forceinline__ void upk(f2 v, float &a, float &b) {
  a = v.a;
  b = v.b;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) { return f2{fmaf(a.a, b.a, c.a), fmaf(a.b, b.b, c.b)}; }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) { return f2{__fmul_rn(a.a, b.a), __fmul_rn(a.b, b.b)}; }
__device__ __forceinline__ f2 add2(f2 a, f2 b) { return f2{__fadd_rn(a.a, b.a), __fadd_rn(a.b, b.b)}; }
__device__ __forceinline__ uint32_t half2_of(f2 v) {
  float a, b;
  upk(v, a, b);
  return half2_bits(a, b);
}

// ======================================================================
// Per chunk and key head: the fp16 K and Q tiles, and for each of its value
// heads T, P' and the per-token factors.  Four warps; warp w owns rows
// 16w .. 16w+15 of all 64 x 64 matrices, in the fragment form of mma.sync:
// K K^T and Q K^T stay in its registers while the value heads are gone
// through, and A and P are made from them in place.  With D the 16 x 16 blocks
// on the diagonal of (I + A)^-1 (forward substitution, a lane per column) and
// Y = D A (all block rows at once),
//   T_Ic = -sum_{c <= m < I} Y_Im T_mc          block row after block row,
// which carries diag(beta) and the tile's scale along in T_cc.  All products
// are mma.sync on fp16 pairs (three products each).
//
// 199 us for 16384 tokens of 32 heads, of which the bytes are 80 us at a plain
// copy's rate: bound by the latency of the block rows' chain and its barriers.  Four CTAs a SM: three take as long, five or six spill more
// and take 3 to 12 % longer.
//
// Scales are powers of two from bounds, so that nothing is searched for on the
// way (searches for the largest value of each block row made this kernel 20 %
// slower).  With |k| the keys' norms after their factors, a token multiplies
// what lies before it by at most e^g max(1, |1 - beta |k|^2|): at most 1 with
// g <= 0 and beta |k|^2 <= 2, and otherwise grow, the product over the chunk of
// those above 1.  Then, entry by entry,
//   |A| <= X = max(beta |k|) max |k|          (times the growth of the gates)
//   |(I + A)^-1| <= grow max(1, X), |Y| <= grow X, |T| <= grow max(1, X) max beta
//   |P| <= max |q| max |k|                    (times the growth of the gates)
//   |P'| <= grow max |q| max |k| max beta
// and each is scaled so that its bound lies in [2^14, 2^15).  grow counts up to
// 2^kGrow: one fp16 pair reaches over 39 octaves, and what the bound takes of them the
// ordinary values lack.  A chunk that grows the state by more overflows.
constexpr float kGrow = 16.f;
constexpr int kPrepT = 128;

// Exponents of the scales of a value head's operands: A, (I + A)^-1, Y, T, P and P'
struct Scales {
  int a, d, y, t, p, x;
};

struct PrepShared {
  float D[4][16][20];          // per warp: the diagonal block of A, then its inverse
  float rk[kC], rq[kC];        // factors of the fp16 rows: norm, scale and 2^-e
  // of up to four value heads, a warp each
  float Gh[4][kC], Gl[4][kC];  // log2(e) G = Gh + Gl
  float beta[4][kC];
  Scales scales[4];
  float kn[kC];                // the keys' norms, after their factors
  float size[4];               // the largest of them (warps 0, 1), and of the scaled queries' (2, 3)
};

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, f2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
      f[i] = pk(t.x, t.y);
    } else {
      f[i] = pk(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
  }
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 2^(G 2^-40): the whole octaves go into the exponent, so that the rest is small
// enough for fp32 whatever G is
__device__ __forceinline__ float ex2_fixed(long long G) {
  const int n = (int)(G >> 40);
  const float f = (float)(G & ((1ll << 40) - 1)) * 9.094947017729282e-13f;
  return n < -126 ? 0.f : n > 127 ? __int_as_float(0x7f800000) : ex2(f) * pow2f(n);
}
// the 8 x 8 matrix of 16-bit values that the warp holds, transposed
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ f2 lds_pair(const float *p) {
  const float2 v = *reinterpret_cast<const float2 *>(p);
  return f2{v.x, v.y};
}
// d += (ah + al)(bh + bl) without the product of the low parts
__device__ __forceinline__ void mma3(float (&d)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], uint32_t bh0, uint32_t bh1,
                                     uint32_t bl0, uint32_t bl1) {
  mma16(d, al, bh0, bh1);
  mma16(d, ah, bl0, bl1);
  mma16(d, ah, bh0, bh1);
}
// a 16 x 16 block of fragments, times a power of two, as the pair operand of the next product
__device__ __forceinline__ void pair_operand(const f2 (&c)[2][2], float scale, uint32_t (&h)[4], uint32_t (&l)[4]) {
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const f2 v = mul2(c[n][e], pk(scale, scale));
      split2(v.a, v.b, h[2 * n + e], l[2 * n + e]);
    }
}

template <typename T, int DK>
__global__ void __launch_bounds__(kPrepT, 4) delta_prep_kernel(const DeltaView a, const ChunkPlaces ws, const Slab slab, int heads) {
  constexpr int kKq = kC * DK * 2;  // bytes of a K or Q tile
  constexpr int kArea = 2 * kKq > kTiles ? 2 * kKq : kTiles;
  __shared__ __align__(128) unsigned char area[kArea];  // K, Q tiles; later T and P' (as in the workspace)
  __shared__ PrepShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t place = blockIdx.x;
  const int hk = blockIdx.y;
  // the sequence whose places include this one: the last that begins at or before it
  int64_t t0, t1;
  int64_t seq = 0;
  for (int64_t end = a.B, step; end - seq > 1; end = min(end, seq + step)) {  // 32 places at once
    step = (end - seq + 31) / 32;
    const int64_t b = seq + lane * step;
    bool at_or_before = false;
    if (b < end) {
      a.range(b, t0, t1);
      at_or_before = chunk_base(t0, b) <= place;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, at_or_before);
    seq += m ? (31 - __clz(m)) * step : 0;
  }
  a.range(seq, t0, t1);
  const int64_t nth = place - chunk_base(t0, seq);
  t0 += nth * kC;
  // A later slab's grid starts beside the chain of the slab before it and writes
  // only what that chain does not touch; one of its CTAs ends after that chain,
  // so that the next chain, which follows this grid, follows both.
  auto leave = [&] {
    if (slab.first > 0 && blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1)
      asm volatile("griddepcontrol.wait;" ::: "memory");
  };
  if (nth < slab.first || nth >= slab.end || t0 >= t1) {
    leave();
    return;
  }
  const int len = (int)min((int64_t)kC, t1 - t0);
  const int group = a.HV / a.HK;
  const int of0 = blockIdx.z * heads, of1 = min(group, of0 + heads);  // this CTA's value heads of the group
  // this warp's gates, two tokens per lane, of one of them
  float gate_g[2], gate_b[2];
  auto load_gates = [&](int of) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int t = 2 * lane + x;
      const bool in = t < len && of < of1;
      gate_g[x] = in ? a.g[(t0 + t) * a.g_stride + hk * group + of] : 0.f;
      gate_b[x] = in ? a.beta[(t0 + t) * a.beta_stride + hk * group + of] : 0.f;
    }
  };
  load_gates(of0 + warp);

  // ---- K and Q rows -> fp16 tiles; DK/8 lanes per row.  A row's scale brings
  // its norm, and so every value, below 2^15
  constexpr int LPR = DK / 8, RPI = kPrepT / LPR, NI = kC / RPI;
  const int piece = tid % LPR;
  uint4 raw[2][NI];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int64_t stride = which ? a.q_stride : a.k_stride;
    const T *src = static_cast<const T *>(which ? a.q : a.k) + (t0 + tid / LPR) * stride + (int64_t)hk * DK + piece * 8;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      raw[which][i] =
          tid / LPR + i * RPI < len ? __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)(i * RPI) * stride)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    unsigned char *out = ws.kq + ((place * a.HK + hk) * 2 + which) * (int64_t)kKq;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = tid / LPR + i * RPI;
      f2 f[4], s2 = pk(0.f, 0.f);
      unpack8<T>(raw[which][i], f);
#pragma unroll
      for (int e = 0; e < 4; ++e) s2 = fma2(f[e], f[e], s2);
      float ss, sy;
      upk(s2, ss, sy);
      ss += sy;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const int e = root_exp(ss);
      const f2 sc = pk(pow2f(e), pow2f(e));
      uint4 h;
      h.x = half2_of(mul2(f[0], sc));
      h.y = half2_of(mul2(f[1], sc));
      h.z = half2_of(mul2(f[2], sc));
      h.w = half2_of(mul2(f[3], sc));
      const uint32_t at = (uint32_t)(piece >> 3) * (kC * 128) + swz(r, piece & 7);
      *reinterpret_cast<uint4 *>(area + which * kKq + at) = h;
      if (of0 == 0) *reinterpret_cast<uint4 *>(out + at) = h;
      if (piece == 0) (which ? sh.rq : sh.rk)[r] = ss;
    }
  }
  __syncthreads();
  {  // the rows' factors, a thread per row: keys by warps 0 and 1, queries by 2 and 3
    const int which = tid >> 6;
    float &slot = (which ? sh.rq : sh.rk)[tid & 63];
    const float ss = slot;
    const float n = (a.l2norm ? rsqrtf(ss + kDeltaEps) : 1.f) * (which ? a.scale : 1.f);
    slot = n * pow2f(-root_exp(ss));
    float size = fabsf(n) * sqrtf(ss);
    if (!which) sh.kn[tid & 63] = size;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) size = fmaxf(size, __shfl_xor_sync(0xffffffffu, size, o));
    if (lane == 0) sh.size[warp] = size;
  }

  // ---- K K^T and Q K^T, columns up to this warp's rows
  float kk[4][2][4] = {}, qk[4][2][4] = {};
  const uint32_t kt32 = smem_u32(area), qt32 = kt32 + kKq;
#pragma unroll
  for (int s = 0; s < DK / 16; ++s) {
    const uint32_t box = (uint32_t)(s >> 2) * (kC * 128);
    const int p0 = (s & 3) * 2;
    uint32_t ak[4], aq[4];
    const int ar = 16 * warp + (lane & 15);
    ldsm4(kt32 + box + swz(ar, p0 + (lane >> 4)), ak);
    ldsm4(qt32 + box + swz(ar, p0 + (lane >> 4)), aq);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j <= warp) {
        uint32_t b[4];
        ldsm4(kt32 + box + swz(16 * j + (lane & 7) + ((lane >> 4) << 3), p0 + ((lane >> 3) & 1)), b);
        mma16(kk[j][0], ak, b[0], b[1]);
        mma16(kk[j][1], ak, b[2], b[3]);
        mma16(qk[j][0], aq, b[0], b[1]);
        mma16(qk[j][1], aq, b[2], b[3]);
      }
  }
  __syncthreads();  // the tiles' area is free
  const float kmax = fmaxf(sh.size[0], sh.size[1]), qmax = fmaxf(sh.size[2], sh.size[3]);
  const uint32_t th = smem_u32(area), tl = th + kTile, ph = th + 2 * kTile, pl = th + 3 * kTile;
  // the blocks above the diagonal stay zero
  for (int i = tid; i < kTiles / 16; i += kPrepT) reinterpret_cast<uint4 *>(area)[i] = make_uint4(0, 0, 0, 0);

  const int fr = lane >> 2, fc = 2 * (lane & 3);  // fragment rows fr, fr + 8 of the block; columns 8n + fc, + 1
  // a fragment word (row, columns 8 piece + fc, + 1) of a tile
  auto word_at = [&](uint32_t tile, int row, int pc) { return tile + swz(row, pc) + (uint32_t)fc * 2; };
  auto put = [](uint32_t addr, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory"); };
  // the gates of value head `of` (this warp's): G in fixed point (2^-40), exact
  // sums whose differences are taken later; the factors of the chain go out
  auto gates = [&](int of) {
    float *sc = ws.sc + (place * a.HV + hk * group + of) * kScalars;
    const uint32_t nan0 = __ballot_sync(0xffffffffu, gate_g[0] != gate_g[0]), nan1 = __ballot_sync(0xffffffffu, gate_g[1] != gate_g[1]);
    float up = 0.f, over = 0.f, bmax = 0.f, bk = 0.f;  // log2 of what gates and corrections grow by; largest beta, beta |k|
    long long gi[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      // exp(-200) is 0 in fp32 already
      const float g = fminf(fmaxf(gate_g[x], -200.f), 200.f), l = g * 1.44269504f;
      // the product's own rounding, and log2(e) beyond fp32, are part of the sum
      const float rest = fmaf(g, 1.925963e-8f, fmaf(g, 1.44269504f, -l));
      up += fmaxf(l, 0.f);
      gi[x] = __float2ll_rn(l * 1099511627776.f) + __float2ll_rn(rest * 1099511627776.f);
      const float b = fabsf(gate_b[x]), kn = sh.kn[2 * lane + x];
      bmax = fmaxf(bmax, b);
      bk = fmaxf(bk, b * kn);
      over += __log2f(fmaxf(1.f, fabsf(1.f - gate_b[x] * kn * kn)));
    }
    long long sum = gi[0] + gi[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long z = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += z;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      up += __shfl_xor_sync(0xffffffffu, up, o);
      over += __shfl_xor_sync(0xffffffffu, over, o);
    }
    bmax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(bmax)));
    bk = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(bk)));
    const float by_gates = exp2f(fminf(up, kGrow)), grow = exp2f(fminf(up + over, kGrow)), X = bk * kmax;
    const Scales e = {scale_exp(X * by_gates), scale_exp(grow * fmaxf(1.f, X)), scale_exp(X * grow),
                      scale_exp(grow * fmaxf(1.f, X) * bmax), scale_exp(qmax * kmax * by_gates), scale_exp(grow * qmax * kmax * bmax)};
    const long long all = __shfl_sync(0xffffffffu, sum, 31);
    const long long G[2] = {sum - gi[1], sum};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int t = 2 * lane + x;
      // tokens from the first NaN on
      const bool bad = (nan0 & ((2u << lane) - 1u)) || (nan1 & (x ? (2u << lane) - 1u : (1u << lane) - 1u));
      float gh = (float)G[x];
      const float gl = (float)(G[x] - (long long)gh) * 9.094947017729282e-13f;
      gh *= 9.094947017729282e-13f;
      if (bad) gh = __int_as_float(0x7fc00000);
      sh.Gh[warp][t] = gh;
      sh.Gl[warp][t] = gl;
      sh.beta[warp][t] = gate_b[x];
      const float gam = bad ? gh : ex2_fixed(G[x]);
      const float tail = ex2_fixed(all - G[x]);
      sc[t] = gam * sh.rk[t];
      sc[kC + t] = ((nan0 | nan1) ? __int_as_float(0x7fc00000) : tail) * sh.rk[t] * pow2f(-e.t);
      sc[2 * kC + t] = gam * sh.rq[t];
      if (t == kC - 1) {
        sc[3 * kC] = gam;
        sc[3 * kC + 1] = pow2f(-e.x);
      }
    }
    if (lane == 0) sh.scales[warp] = e;
  };
  for (int of = of0; of < of1; ++of) {
    const int at = (of - of0) & 3, hv = hk * group + of;
    if (at == 0) {
      if (of > of0) load_gates(of + warp);
      if (of + warp < of1) gates(of + warp);
    }
    __syncthreads();  // the gates are there; the last head's tiles have been copied out
    const float *Gh = sh.Gh[at], *Gl = sh.Gl[at], *beta = sh.beta[at];
    const Scales e = sh.scales[at];
    const float ps = pow2f(e.p);
    // ---- A and P in place of the products' fragments
    f2 A[4][2][2];
    uint32_t Ph[4][4], Pl[4][4];
    {
      const int i0 = 16 * warp + fr;
      const f2 gh[2] = {pk(Gh[i0], Gh[i0]), pk(Gh[i0 + 8], Gh[i0 + 8])};
      const f2 gl[2] = {pk(Gl[i0], Gl[i0]), pk(Gl[i0 + 8], Gl[i0 + 8])};
      const float b0 = beta[i0] * sh.rk[i0], b1 = beta[i0 + 8] * sh.rk[i0 + 8];
      const float q0 = sh.rq[i0] * ps, q1 = sh.rq[i0 + 8] * ps;
      const f2 ba[2] = {pk(b0, b0), pk(b1, b1)}, rq[2] = {pk(q0, q0), pk(q1, q1)}, neg = pk(-1.f, -1.f);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= warp) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const int c = 16 * j + 8 * n + fc;
            const f2 ch = lds_pair(&Gh[c]), cl = lds_pair(&Gl[c]);
            const f2 rk = lds_pair(&sh.rk[c]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x, y;
              upk(add2(fma2(ch, neg, gh[e]), fma2(cl, neg, gl[e])), x, y);
              const f2 w = mul2(pk(ex2(x), ex2(y)), rk);
              f2 av = mul2(mul2(w, ba[e]), pk(kk[j][n][2 * e], kk[j][n][2 * e + 1]));
              f2 pv = mul2(mul2(w, rq[e]), pk(qk[j][n][2 * e], qk[j][n][2 * e + 1]));
              if (j == warp) {  // the block on the diagonal
                const int i = fr + 8 * e, cc = 8 * n + fc;
                float u0, u1, v0, v1;
                upk(av, u0, u1);
                upk(pv, v0, v1);
                av = pk(cc < i ? u0 : 0.f, cc + 1 < i ? u1 : 0.f);
                pv = pk(cc <= i ? v0 : 0.f, cc + 1 <= i ? v1 : 0.f);
                *reinterpret_cast<float2 *>(&sh.D[warp][i][cc]) = make_float2(av.a, av.b);
              }
              A[j][n][e] = av;
              split2(pv.a, pv.b, Ph[j][2 * n + e], Pl[j][2 * n + e]);
            }
          }
        }
    }
    __syncwarp();
    // ---- the diagonal block's inverse: lane c (and c + 16, the same) solves for column c
    {
      float x[16];
      const int c = lane & 15;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s0 = i == c ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
        for (int m = 0; m < i; m += 4) {
          const float4 av = *reinterpret_cast<const float4 *>(&sh.D[warp][i][m]);
          s0 = fmaf(-av.x, x[m], s0);
          if (m + 1 < i) s1 = fmaf(-av.y, x[m + 1], s1);
          if (m + 2 < i) s0 = fmaf(-av.z, x[m + 2], s0);
          if (m + 3 < i) s1 = fmaf(-av.w, x[m + 3], s1);
        }
        x[i] = s0 + s1;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((i >> 3) == (lane >> 4)) sh.D[warp][i][c] = x[i];
      __syncwarp();
    }
    // its fragments: T's block (with beta), and the operand of Y
    uint32_t dh[4], dl[4];
    {
      f2 d[2][2];
      const float ts = pow2f(e.t);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const f2 be = mul2(lds_pair(&beta[16 * warp + 8 * n + fc]), pk(ts, ts));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          d[n][i] = lds_pair(&sh.D[warp][fr + 8 * i][8 * n + fc]);
          const f2 x = mul2(d[n][i], be);
          uint32_t h, l;
          split2(x.a, x.b, h, l);
          const int row = 16 * warp + fr + 8 * i, pc = 2 * warp + n;
          put(word_at(th, row, pc), h);
          put(word_at(tl, row, pc), l);
        }
      }
      pair_operand(d, pow2f(e.d), dh, dl);
    }
    // ---- Y = D A, the blocks left of the diagonal (kept as pairs)
    uint32_t yh[3][4], yl[3][4];
    const float as = pow2f(e.a), ys = -pow2f(max(e.y - e.a - e.d, -126));
#pragma unroll
    for (int m = 0; m < 3; ++m)
      if (m < warp) {
        uint32_t ah[4], al[4];
        pair_operand(A[m], as, ah, al);
        f2 y[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float d[4] = {};
          mma3(d, dh, dl, movmatrix(ah[2 * n]), movmatrix(ah[2 * n + 1]), movmatrix(al[2 * n]), movmatrix(al[2 * n + 1]));
          y[n][0] = pk(d[0], d[1]);
          y[n][1] = pk(d[2], d[3]);
        }
        pair_operand(y, ys, yh[m], yl[m]);
      }
    // the operand pair of block (m, c) of T, as rows along the contraction
    auto t_block = [&](int m, int c, uint32_t (&bh)[4], uint32_t (&bl)[4]) {
      const uint32_t at = swz(16 * m + (lane & 7) + (((lane >> 3) & 1) << 3), 2 * c + (lane >> 4));
      ldsm4t(th + at, bh);
      ldsm4t(tl + at, bl);
    };
    // ---- T, block row after block row
    {
      float tv[3][2][4] = {};
      const float tvs = pow2f(-e.y);
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        __syncthreads();  // block row m is complete
        if (m < warp) {
#pragma unroll
          for (int c = 0; c <= m; ++c) {
            uint32_t bh[4], bl[4];
            t_block(m, c, bh, bl);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma3(tv[c][n], yh[m], yl[m], bh[2 * n], bh[2 * n + 1], bl[2 * n], bl[2 * n + 1]);
          }
        }
        if (m + 1 == warp) {  // this warp's block row is next
#pragma unroll
          for (int c = 0; c <= m; ++c)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t h, l;
                split2(tv[c][n][2 * i] * tvs, tv[c][n][2 * i + 1] * tvs, h, l);
                const int row = 16 * warp + fr + 8 * i, pc = 2 * c + n;
                put(word_at(th, row, pc), h);
                put(word_at(tl, row, pc), l);
              }
        }
      }
    }
    __syncthreads();
    // ---- P' = P T
    const float xs = pow2f(max(e.x - e.p - e.t, -126));
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c <= warp) {
        float pp[2][4] = {};
#pragma unroll
        for (int m = c; m < 4; ++m)
          if (m <= warp) {
            uint32_t bh[4], bl[4];
            t_block(m, c, bh, bl);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma3(pp[n], Ph[m], Pl[m], bh[2 * n], bh[2 * n + 1], bl[2 * n], bl[2 * n + 1]);
          }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t h, l;
            split2(pp[n][2 * i] * xs, pp[n][2 * i + 1] * xs, h, l);
            put(word_at(ph, 16 * warp + fr + 8 * i, 2 * c + n), h);
            put(word_at(pl, 16 * warp + fr + 8 * i, 2 * c + n), l);
          }
      }
    __syncthreads();
    uint4 *dst = reinterpret_cast<uint4 *>(ws.tp + (place * a.HV + hv) * (int64_t)kTiles);
#pragma unroll
    for (int i = 0; i < kTiles / 16 / kPrepT; ++i) dst[tid + i * kPrepT] = reinterpret_cast<const uint4 *>(area)[tid + i * kPrepT];
  }
  leave();
}

// ======================================================================
// The walk over a sequence's chunks, one CTA per sequence and value head.
// All products are in the transposed form, a value column per lane of tensor
// memory, so that the operand made from registers is the MMA's A operand in
// tensor memory (M = 128 lanes) and K, Q, T and P' are its B operands as they
// lie in shared memory.  The first 8 (or 4) warps, the chain, own 16 lanes (state columns) each, in
// the fragment form of tensor memory loads (16x256b): a thread holds two rows
// (columns lane/4 and lane/4 + 8 of the warp's 16) and pairs of neighbouring
// tokens or key entries, which are also the pairs of an fp16 operand word and
// of the two-wide fp32 instructions.  A row's size, for its scale, is then a
// matter of four lanes.  Per chunk:
//     1  S -> high, low                     MMA: KS = S^T K^T, QS = S^T Q^T
//     2  R = V - a KS -> high, low          MMA: U = R^T T^T, O2 = R^T P'^T
//     3  c U -> high, low                   MMA: D = (c U)^T K
//     o = b QS + O2 while D is computed; then S = gamma_C S + D
//   next warp: copies of the next chunk's tiles, factors and V rows (two stages)
//   next: tensor memory; issues the MMAs from the thread that elect.sync picks
//     (17 clocks per MMA, against 44 behind an `if (lane == 0)`, whose operands
//     leave the uniform registers)
//   last: the chunk's rows of o from shared memory, where the chain stages them
// One chunk is a chain of three dependent products; the time is the latency of
// that chain, not the rate of any unit: 2.6 us a chunk on half heads, 3.0 us on
// whole ones (1024 tokens of 32 heads, both kernels: 62 us on half heads, 69 us
// on whole ones; of 96 heads 131 and 101 us).  The low parts in o cost it 1 to 2 %:
// their products run while the next operand is made.
// Tensor memory columns: S high [0, 64), low [64, 128), and D over both;
// KS [128, 192); QS [192, 256); R [256, 320); U [320, 384); O2 [384, 448);
// c U [448, 512).
constexpr uint32_t kColS = 0, kColD = 0, kColKS = 128, kColQS = 192, kColR = 256, kColU = 320, kColO = 384, kColW = 448;

struct ChainBars {
  uint64_t full[2], empty[2];
  // halves: of the key entries (S, D), of the tokens (R, c U)
  uint64_t s_ready[2], r_ready[2], w_ready[2], d_done[2];
  uint64_t ks_done, u_done, o_done, o_ready, o_free, drain;
  uint32_t tmem_base;
  volatile int abort_flag;
};
constexpr int kSortMax = 256;  // sequences that are taken longest first
constexpr int kChainHeader = 2048;
static_assert(sizeof(ChainBars) + kSortMax * 4 <= kChainHeader, "header");

// M: the state columns of a CTA.  128 is one head; 64 gives half a head to a
// CTA (tensor memory lanes 0-15 of each quarter), which halves the work per
// chunk of the chain warps and so shortens the chain, on twice the SMs.
template <int DK, int M>
struct ChainStage {
  static constexpr int kWarps = M / 16, kThreads = 32 * (kWarps + 3);
  static constexpr int kRow = M * 2 + 16;  // bytes of a staged row of V or o: 8 rows at one column fall into different banks
  static constexpr int kKq = 2 * kC * DK * 2;
  static constexpr int kTp = kKq, kV = kTp + kTiles, kSc = kV + kC * kRow;
  static constexpr int kBytes = (kSc + kScalarBytes + 1023) / 1024 * 1024;
};
template <int DK, int M>
constexpr size_t chain_smem() {
  return 1024 + kChainHeader + 2 * (size_t)ChainStage<DK, M>::kBytes + kC * ChainStage<DK, M>::kRow;
}

__device__ __forceinline__ void mbar_init(uint64_t *b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
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
// Whether a wait gives up: its limit has run out, or another role has given up.
__device__ __noinline__ bool give_up(ChainBars *bars, unsigned long long since) {
  if (bars->abort_flag) return true;
  if (global_ns() - since <= c_delta_wait_ns) return false;
  bars->abort_flag = 1;
  atomicOr(&g_delta_err, 1u);
  return true;
}
// Bounded wait of a whole warp; one verdict for all its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *b, uint32_t parity, ChainBars *bars) {
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
__device__ __forceinline__ bool wait_one(uint64_t *b, uint32_t parity, ChainBars *bars) {
  if (mbar_try(b, parity)) return true;
  const unsigned long long since = global_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try(b, parity)) return true;
    if ((i & 31u) == 0 && give_up(bars, since)) return false;
  }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// 16 bytes, or zeros where !have
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have ? 16 : 0) : "memory");
}

// K-major operand, rows of 128 bytes, 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// The same bytes read with the rows as the contraction index: 64 values of N
// per row, 8-row groups 1024 bytes apart, 64-column boxes of 64 rows one after another.
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(kC * 128 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp16 x fp16 -> fp32; bit 16: B with its rows along the contraction
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn = false) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void umma(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool acc) {
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
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 64 columns of this warp's 16 lanes: v[2g + h] = row lane/4 + 8h, columns 8g + 2 (lane % 4) and the next
__device__ __forceinline__ void tm_ld(uint32_t t, f2 (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0].a), "=f"(v[0].b), "=f"(v[1].a), "=f"(v[1].b), "=f"(v[2].a), "=f"(v[2].b), "=f"(v[3].a), "=f"(v[3].b), "=f"(v[4].a), "=f"(v[4].b), "=f"(v[5].a), "=f"(v[5].b), "=f"(v[6].a), "=f"(v[6].b), "=f"(v[7].a), "=f"(v[7].b), "=f"(v[8].a), "=f"(v[8].b), "=f"(v[9].a), "=f"(v[9].b), "=f"(v[10].a), "=f"(v[10].b), "=f"(v[11].a), "=f"(v[11].b), "=f"(v[12].a), "=f"(v[12].b), "=f"(v[13].a), "=f"(v[13].b), "=f"(v[14].a), "=f"(v[14].b), "=f"(v[15].a), "=f"(v[15].b)
      : "r"(t)
      : "memory");
}
// 16 columns of operand words: w[2g + h] = row lane/4 + 8h, column 4g + lane % 4
__device__ __forceinline__ void tm_st(uint32_t t, const uint32_t (&w)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The exponents that scale two rows: of the largest absolute values in v[0],
// v[2], ... and v[1], v[3], ..., over the four lanes that share the rows
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int N>
__device__ __forceinline__ void row_max(const f2 *v, float (&m)[4]) {
#pragma unroll
  for (int i = 0; i < N; ++i) m[i & 3] = max3(m[i & 3], v[i].a, v[i].b);
}
// 2^e that brings the rows' sizes (m, over the four lanes that share them) into
// [2^14, 2^15), and 2^-e: from the exponent bits.  Sizes below 2^-100 count as that.
__device__ __forceinline__ void row_scales(const float (&m)[4], float (&up)[2], float (&dn)[2]) {
  float x[2] = {fmaxf(m[0], m[2]), fmaxf(m[1], m[3])};
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    const float x2 = __shfl_xor_sync(0xffffffffu, x[0], o), y2 = __shfl_xor_sync(0xffffffffu, x[1], o);
    x[0] = fmaxf(x[0], x2);
    x[1] = fmaxf(x[1], y2);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t e = __float_as_uint(fmaxf(x[h], 7.8886090522101181e-31f)) & 0x7F800000u;
    up[h] = __uint_as_float((268u << 23) - e);  // 127 + 14 - (e - 127)
    dn[h] = __uint_as_float(e - (14u << 23));
  }
}
// v (N pairs of values, two rows) times its rows' scales: the first 11 bits of
// each as fp16 at column hi, the first 11 of what they leave at column lo.  Cut
// off, not rounded: a mask, where a conversion to fp16 and back made a chunk 5 %
// longer (8192 tokens of 32 heads: 354 and 373 us), for one bit of the 23.
template <int N>
__device__ __forceinline__ void split_store(const f2 *v, const float (&scale)[2], uint32_t hi, uint32_t lo) {
#pragma unroll
  for (int k = 0; k < N; k += 8) {
    uint32_t h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = __fmul_rn(v[k + i].a, scale[i & 1]), y = __fmul_rn(v[k + i].b, scale[i & 1]);
      const float xh = __uint_as_float(__float_as_uint(x) & 0xFFFFE000u), yh = __uint_as_float(__float_as_uint(y) & 0xFFFFE000u);
      h[i] = half2_bits(xh, yh);
      l[i] = half2_bits(x - xh, y - yh);
    }
    tm_st(hi + 2 * k, h);
    tm_st(lo + 2 * k, l);
  }
}

// two 16-bit values (low half first) as a pair of fp32, and back
template <typename T>
__device__ __forceinline__ f2 pair_of(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return pk(t.x, t.y);
  } else {
    return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
}
template <typename T>
__device__ __forceinline__ uint32_t word_of(f2 v) {
  float a, b;
  upk(v, a, b);
  if constexpr (std::is_same<T, __half>::value) {
    return half2_bits(a, b);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}
__device__ __forceinline__ f2 lds2(uint32_t addr) {
  f2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.a), "=f"(v.b) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float lds1(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <typename T, int DK, int M>
__global__ void __launch_bounds__((ChainStage<DK, M>::kThreads), 1) delta_chain_kernel(const DeltaView a, const ChunkPlaces ws, const Slab slab, int sort) {
  if (slab.more) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ unsigned char smem_raw[];
  unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  using St = ChainStage<DK, M>;
  constexpr int NW = St::kWarps, kRow = St::kRow;  // chain warps; then the copies, the MMAs and the stores
  ChainBars *bars = reinterpret_cast<ChainBars *>(base);
  const uint32_t stages = smem_u32(base) + kChainHeader, o_tile = stages + 2 * St::kBytes;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int parts = a.DV / M;
  int64_t b = blockIdx.x / (a.HV * parts);
  const int item = (int)(blockIdx.x - b * (a.HV * parts)), hv = item / parts, hk = hv / (a.HV / a.HK);
  const int dv0 = (item - hv * parts) * M;  // this CTA's first state column
  if (sort) {
    // more CTAs than fit at once: the longest sequences first, so that the
    // last CTAs to start are short
    int *len = reinterpret_cast<int *>(base + kChainHeader - kSortMax * 4);
    __shared__ int pick;
    int64_t x0, x1;
    for (int i = tid; i < (int)a.B; i += St::kThreads) {
      a.range(i, x0, x1);
      len[i] = (int)(x1 - x0);
    }
    __syncthreads();
    for (int i = tid; i < (int)a.B; i += St::kThreads) {
      int rank = 0;
      for (int j = 0; j < (int)a.B; ++j) rank += len[j] > len[i] || (len[j] == len[i] && j < i);
      if (rank == (int)b) pick = i;
    }
    __syncthreads();
    b = pick;
  }
  int64_t t0, t1;
  a.range(b, t0, t1);
  const int64_t place0 = chunk_base(t0, b) + slab.first;
  t0 = min(t0 + (int64_t)slab.first * kC, t1);
  const int chunks = (int)min((t1 - t0 + kC - 1) / kC, (int64_t)slab.end - slab.first);

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->full[s], 1 + 32);  // bulk copies, and the producer's lanes (their zeros)
      mbar_init(&bars->empty[s], 1 + NW);
      mbar_init(&bars->s_ready[s], NW);
      mbar_init(&bars->r_ready[s], NW);
      mbar_init(&bars->w_ready[s], NW);
      mbar_init(&bars->d_done[s], 1);
    }
    mbar_init(&bars->ks_done, 1);
    mbar_init(&bars->u_done, 1);
    mbar_init(&bars->o_done, 1);
    mbar_init(&bars->o_ready, NW);
    mbar_init(&bars->o_free, 1);
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == NW + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);

  if (warp < NW) {
    // first of this warp's 16 columns in the CTA's M, and of its lanes
    const int L0 = M == 128 ? 32 * (warp & 3) + 16 * (warp >> 2) : 16 * warp;
    const int q = lane & 3, c = dv0 + L0 + (lane >> 2);  // this thread's columns c and c + 8 of the state
    const uint32_t tl = tmem + ((uint32_t)(M == 128 ? L0 : 32 * warp) << 16);
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool have = slot >= 0 && slot < a.n_slots;
    const int64_t mine = (int64_t)(2 * q) * a.DV + c;
    float *state = a.state + ((have ? slot : 0) * a.HV + hv) * (int64_t)DK * a.DV + mine;
    constexpr int NS = DK / 4;  // pairs of state values per thread: S[2g + h] = key entries 8g + 2q, + 1 of column c + 8h
    f2 S[NS];
    const bool load = slab.first > 0 || (have && !(a.fresh && a.fresh[b]));
    const float *from = slab.first > 0 ? ws.carry + (int64_t)(blockIdx.x / parts) * DK * a.DV + mine : state;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float *p = from + (int64_t)(8 * (i >> 1)) * a.DV + 8 * (i & 1);
      S[i] = load ? pk(p[0], p[a.DV]) : pk(0.f, 0.f);
    }
    float big[4] = {};
    row_max<NS>(S, big);
    auto publish = [&](uint64_t *bar) {  // tensor-memory stores of this warp, to the MMAs
      wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    bool ok = true;
    for (int n = 0; n < chunks; ++n) {
      const uint32_t ph = n & 1, s = n & 1, sph = (n >> 1) & 1;
      const uint32_t st = stages + s * St::kBytes, sc = st + St::kSc + 8 * q;
      // 1: the state as the operand of K S and Q S
      float f[2], is[2], ir[2], iu[2];  // a scale of the rows; the reciprocals of S's, R's and c U's
      row_scales(big, f, is);
      {
        split_store<NS / 2>(S, f, tl + kColS, tl + kColS + 64);
        publish(&bars->s_ready[0]);
        split_store<NS / 2>(S + NS / 2, f, tl + kColS + NS, tl + kColS + 64 + NS);
        publish(&bars->s_ready[1]);
      }
      // 2: R; V's pairs of tokens come transposed from its rows
      if (!(ok = wait_warp(&bars->full[s], sph, bars))) break;
      uint32_t v[16];
      f2 fac[8];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t w[4];
        ldsm4t(st + St::kV + (uint32_t)(16 * g + ((lane >> 4) << 3) + (lane & 7)) * kRow + (L0 + (((lane >> 3) & 1) << 3)) * 2, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * g + i] = w[i];
      }
#pragma unroll
      for (int g = 0; g < 8; ++g) fac[g] = lds2(sc + 32 * g);
      if (!(ok = wait_warp(&bars->ks_done, ph, bars))) break;
      fence_after();
      f2 R[16];
      tm_ld(tl + kColKS, R);
      {
        const f2 ni[2] = {pk(-is[0], -is[0]), pk(-is[1], -is[1])};
#pragma unroll
        for (int i = 0; i < 16; ++i) R[i] = fma2(mul2(fac[i >> 1], ni[i & 1]), R[i], pair_of<T>(v[i]));
      }
      {
        float m[4] = {};
        row_max<16>(R, m);
        row_scales(m, f, ir);
      }
      {
        split_store<8>(R, f, tl + kColR, tl + kColR + 32);
        publish(&bars->r_ready[0]);
        split_store<8>(R + 8, f, tl + kColR + 16, tl + kColR + 48);
        publish(&bars->r_ready[1]);
      }
      // 3: the scaled U
#pragma unroll
      for (int g = 0; g < 8; ++g) fac[g] = lds2(sc + 4 * kC + 32 * g);
      if (!(ok = wait_warp(&bars->u_done, ph, bars))) break;
      fence_after();
      tm_ld(tl + kColU, R);
#pragma unroll
      for (int i = 0; i < 16; ++i) R[i] = mul2(R[i], fac[i >> 1]);
      {
        float m[4] = {};
        row_max<16>(R, m);
        row_scales(m, f, iu);
      }
      {
        split_store<8>(R, f, tl + kColW, tl + kColW + 32);
        // D overwrites S's operand, which the products with Q read
        if (!(ok = wait_warp(&bars->o_done, ph, bars))) break;
        fence_after();
        publish(&bars->w_ready[0]);
        split_store<8>(R + 8, f, tl + kColW + 16, tl + kColW + 48);
        publish(&bars->w_ready[1]);
      }
      // o while D is computed
      {
        const float ps = lds1(st + St::kSc + (3 * kC + 1) * 4);
        f2 O[16];
        tm_ld(tl + kColQS, R);
        tm_ld(tl + kColO, O);
        const f2 is2[2] = {pk(is[0], is[0]), pk(is[1], is[1])}, ir2[2] = {pk(ir[0] * ps, ir[0] * ps), pk(ir[1] * ps, ir[1] * ps)};
        if (n > 0 && !(ok = wait_warp(&bars->o_free, ph ^ 1u, bars))) break;
#pragma unroll
        for (int g = 0; g < 8; g += 2) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = 2 * g + i;
            const f2 fb = lds2(sc + 8 * kC + 32 * (at >> 1));
            w[i] = word_of<T>(fma2(mul2(fb, is2[i & 1]), R[at], mul2(O[at], ir2[i & 1])));
          }
          // four 8 x 8 blocks (tokens 8g and 8g + 8, columns L0 and L0 + 8), transposed into rows of tokens
          const uint32_t at = o_tile + (uint32_t)(8 * g + ((lane >> 4) << 3) + (lane & 7)) * kRow + (L0 + (((lane >> 3) & 1) << 3)) * 2;
          asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w[0]), "r"(w[1]),
                       "r"(w[2]), "r"(w[3])
                       : "memory");
        }
      }
      const float gc = lds1(st + St::kSc + 3 * kC * 4);
      const float fd[2] = {iu[0] * ir[0], iu[1] * ir[1]};
      fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars->o_ready);
        mbar_arrive(&bars->empty[s]);  // this warp is done with V and the factors
      }
      // the state, 64 key entries at a time
      const f2 gc2 = pk(gc, gc), fd2[2] = {pk(fd[0], fd[0]), pk(fd[1], fd[1])};
      big[0] = big[1] = big[2] = big[3] = 0.f;
#pragma unroll
      for (int h = 0; h < DK / 64; ++h) {
        if (!(ok = wait_warp(&bars->d_done[h], ph, bars))) break;
        fence_after();
        f2 D[16];
        tm_ld(tl + kColD + 64 * h, D);
#pragma unroll
        for (int i = 0; i < 16; ++i) S[16 * h + i] = fma2(gc2, S[16 * h + i], mul2(D[i], fd2[i & 1]));
        row_max<16>(S + 16 * h, big);
      }
      if (!ok) break;
    }
    int *failed = ws.failed + ((int64_t)(blockIdx.x / parts) * a.DV + dv0 + L0) / 16;
    // these columns keep their value (others of the sequence may have advanced)
    if (slab.first > 0 && *failed) ok = false;
    __syncwarp();
    if (slab.more || (ok && have)) {
      // (not kept over the walk: its registers are worth 1 %)
      float *to = slab.more ? ws.carry + ((int64_t)(blockIdx.x / parts) * DK + 2 * q) * a.DV + c : state;
      if (slab.more && lane == 0) *failed = !ok;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        float *p = to + (int64_t)(8 * (i >> 1)) * a.DV + 8 * (i & 1);
        p[0] = S[i].a;
        p[a.DV] = S[i].b;
      }
    }
  } else if (warp == NW) {
    if (!c_delta_stall) {
      constexpr int pshift = M == 128 ? 4 : 3, per = 1 << pshift;  // 16-byte pieces of a row of V
      const T *v0 = static_cast<const T *>(a.v);
      int n = 0;
      for (; n < chunks; ++n) {
        const uint32_t s = n & 1, sph = (n >> 1) & 1;
        if (!wait_warp(&bars->empty[s], sph ^ 1u, bars)) break;
        const uint32_t st = stages + s * St::kBytes;
        const int64_t place = place0 + n, t = t0 + (int64_t)n * kC;
        const int len = (int)min((int64_t)kC, t1 - t);
        if (lane == 0) {
          mbar_expect(&bars->full[s], St::kKq + kTiles + kScalarBytes);
          bulk_load(st, ws.kq + (place * a.HK + hk) * (int64_t)St::kKq, St::kKq, &bars->full[s]);
          bulk_load(st + St::kTp, ws.tp + (place * a.HV + hv) * (int64_t)kTiles, kTiles, &bars->full[s]);
          bulk_load(st + St::kSc, ws.sc + (place * a.HV + hv) * kScalars, kScalarBytes, &bars->full[s]);
        }
        // V's rows in pieces of 16 bytes, zeros past the sequence's end (a bulk
        // copy per row took the warp about 50 clocks each)
        const T *v = static_cast<const T *>(a.v) + (t + (lane >> pshift)) * a.v_stride + (int64_t)hv * a.DV + dv0 + (lane & (per - 1)) * 8;
        const uint32_t dst = st + St::kV + (uint32_t)(lane >> pshift) * kRow + (lane & (per - 1)) * 16;
        constexpr int rows = 32 >> pshift;
#pragma unroll 8
        for (int r = 0; r < kC; r += rows) {
          const bool in = r + (lane >> pshift) < len;
          copy16(dst + r * kRow, in ? v + (int64_t)r * a.v_stride : v0, in);
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&bars->full[s])) : "memory");
      }
      // no copy is in flight when the CTA ends
      asm volatile("cp.async.wait_all;" ::: "memory");
      for (int m = n > 2 ? n - 2 : 0; m < n; ++m) {
        const unsigned long long since = global_ns();
        while (!mbar_try(&bars->full[m & 1], (m >> 1) & 1) && global_ns() - since < c_delta_wait_ns) {
        }
      }
    }
  } else if (warp == NW + 1) {
    if (elect_one()) {
      for (int n = 0; n < chunks; ++n) {
        const uint32_t ph = n & 1, s = n & 1, sph = (n >> 1) & 1;
        const uint32_t kt = stages + s * St::kBytes, qt = kt + St::kKq / 2, tp = kt + St::kTp;
        bool ok = wait_one(&bars->full[s], sph, bars);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || !(ok = wait_one(&bars->s_ready[h], ph, bars))) break;
          fence_after();
#pragma unroll
          for (int i = 0; i < DK / 32; ++i) {
            const int k = h * (DK / 32) + i;
            const uint64_t bd = desc_k(kt + (k >> 2) * (kC * 128) + (k & 3) * 32);
            umma(tmem + kColKS, tmem + kColS + 64 + 8 * k, bd, idesc(M, 64), k > 0);
            umma(tmem + kColKS, tmem + kColS + 8 * k, bd, idesc(M, 64), true);
          }
          if (h == 1) {
            umma_commit(&bars->ks_done);
#pragma unroll
            for (int k = 0; k < DK / 16; ++k) {
              const uint64_t bd = desc_k(qt + (k >> 2) * (kC * 128) + (k & 3) * 32);
              umma(tmem + kColQS, tmem + kColS + 64 + 8 * k, bd, idesc(M, 64), k > 0);
              umma(tmem + kColQS, tmem + kColS + 8 * k, bd, idesc(M, 64), true);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || !(ok = wait_one(&bars->r_ready[h], ph, bars))) break;
          fence_after();
#pragma unroll
          for (int k = 2 * h; k < 2 * h + 2; ++k) {
            const uint64_t th = desc_k(tp + k * 32), tl = desc_k(tp + kTile + k * 32);
            umma(tmem + kColU, tmem + kColR + 32 + 8 * k, th, idesc(M, 64), k > 0);
            umma(tmem + kColU, tmem + kColR + 8 * k, tl, idesc(M, 64), true);
            umma(tmem + kColU, tmem + kColR + 8 * k, th, idesc(M, 64), true);
          }
          if (h == 1) {
            umma_commit(&bars->u_done);
#pragma unroll
            for (int k = 0; k < kC / 16; ++k) {
              const uint64_t ph = desc_k(tp + 2 * kTile + k * 32), pl = desc_k(tp + 3 * kTile + k * 32);
              umma(tmem + kColO, tmem + kColR + 32 + 8 * k, ph, idesc(M, 64), k > 0);
              umma(tmem + kColO, tmem + kColR + 8 * k, pl, idesc(M, 64), true);
              umma(tmem + kColO, tmem + kColR + 8 * k, ph, idesc(M, 64), true);
            }
            umma_commit(&bars->o_done);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || !(ok = wait_one(&bars->w_ready[h], ph, bars))) break;
          fence_after();
#pragma unroll
          for (int d = 0; d < DK / 64; ++d) {
#pragma unroll
            for (int k = 2 * h; k < 2 * h + 2; ++k) {
              const uint64_t bd = desc_mn(kt + d * (kC * 128) + k * 2048);
              umma(tmem + kColD + 64 * d, tmem + kColW + 32 + 8 * k, bd, idesc(M, 64, true), k > 0);
              umma(tmem + kColD + 64 * d, tmem + kColW + 8 * k, bd, idesc(M, 64, true), true);
            }
            if (h == 1) umma_commit(&bars->d_done[d]);
          }
          if (h == 1) umma_commit(&bars->empty[s]);
        }
        if (!ok) break;
      }
      // every MMA issued, complete before the memory it uses is released
      umma_commit(&bars->drain);
    }
    __syncwarp();
    const unsigned long long since = global_ns();
    while (!mbar_try(&bars->drain, 0) && global_ns() - since < c_delta_wait_ns) {
    }
  } else {
    constexpr int pshift = M == 128 ? 4 : 3, per = 1 << pshift, rows = 32 >> pshift;
    const int r0 = lane >> pshift, at = (lane & (per - 1)) * 8;
    T *o = static_cast<T *>(a.o) + (t0 + r0) * a.o_stride + (int64_t)hv * a.DV + dv0 + at;
    for (int n = 0; n < chunks; ++n) {
      if (!wait_warp(&bars->o_ready, n & 1, bars)) break;
      const int len = (int)min((int64_t)kC, t1 - t0 - (int64_t)n * kC);
#pragma unroll 8
      for (int r = 0; r < kC; r += rows) {
        uint4 w;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(o_tile + (r + r0) * kRow + at * 2) : "memory");
        if (r + r0 < len) *reinterpret_cast<uint4 *>(o + (int64_t)r * a.o_stride) = w;
      }
      o += (int64_t)kC * a.o_stride;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->o_free);
    }
  }
  fence_before();
  __syncthreads();
  if (warp == NW + 1) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

constexpr int64_t kSlabCtas = 76;  // half of the 152 SMs
// Half a head per CTA: heads of 64 columns, or while all of them run at once.
bool half_heads(const DeltaView &a, int64_t sms) { return a.DV == 64 || 2 * a.B * a.HV <= sms; }
// Whether the chain leaves half of the SMs idle, on which the chunk kernel of a
// later slab then runs.
bool can_slab(const DeltaView &a) { return a.B * a.HV * (a.DV / 64) <= kSlabCtas; }

ChunkPlaces places(const DeltaView &a, void *ws, size_t *total) {
  const size_t n = (size_t)chunk_places(a.T, a.B);
  const size_t kq = up256(n * a.HK * (size_t)(2 * kC * a.DK * 2)), tp = up256(n * a.HV * (size_t)kTiles);
  unsigned char *p = static_cast<unsigned char *>(ws);
  const size_t sc = up256(n * a.HV * (size_t)kScalarBytes), st = (size_t)(a.B * a.HV) * a.DK * a.DV * 4;
  if (total) *total = kq + tp + sc + (can_slab(a) ? st + (size_t)(a.B * a.HV) * (a.DV / 16) * 4 : 0);
  unsigned char *carry = p + kq + tp + sc;
  return ChunkPlaces{p, p + kq, reinterpret_cast<float *>(p + kq + tp), reinterpret_cast<float *>(carry),
                     reinterpret_cast<int *>(carry + st)};
}

template <typename T, int DK, int M>
cudaError_t chain_t(const DeltaView &a, const ChunkPlaces &ws, const Slab &slab, int64_t sms, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  const int dev = current_device();
  if (not_done(ready, dev)) {
    cudaError_t e = cudaFuncSetAttribute(delta_chain_kernel<T, DK, M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)chain_smem<DK, M>());
    if (e != cudaSuccess) return e;
    mark_done(ready, dev);
  }
  const int64_t ctas = a.B * a.HV * (a.DV / M);
  const int sort = a.cu && a.B > 1 && a.B <= kSortMax && ctas > sms;
  delta_chain_kernel<T, DK, M><<<(unsigned)ctas, ChainStage<DK, M>::kThreads, chain_smem<DK, M>(), st>>>(a, ws, slab, sort);
  return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t chunks_t(const DeltaView &a, void *workspace, cudaStream_t st) {
  static std::atomic<int> sm_count[kMaxDevices];
  const int dev = current_device();
  int sms = dev < kMaxDevices ? sm_count[dev].load(std::memory_order_relaxed) : 0;
  if (!sms) {
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) sm_count[dev].store(sms, std::memory_order_relaxed);
  }
  const ChunkPlaces ws = places(a, workspace, nullptr);
  // a CTA takes the value heads of a key head one after another, unless that
  // leaves SMs idle: then a CTA per value head
  const int64_t n = chunk_places(a.T, a.B);
  const int group = a.HV / a.HK, heads = n * a.HK <= 2 * sms ? 1 : group;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)n, (unsigned)a.HK, (unsigned)((group + heads - 1) / heads));
  cfg.blockDim = dim3(kPrepT);
  cfg.stream = st;
  cudaLaunchAttribute beside;
  beside.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  beside.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &beside;  // of the later slabs' launches
  // Slabs of 1, 2, 4, ... parts: only the first one's chunk kernel is waited for,
  // and the others', on the half of the SMs that the chain leaves, keep ahead of
  // it.  A further slab costs 9 us (two launches, the state out and in), so their
  // number goes by the chunk kernel's work, in chunks times heads.  Times in us
  // with 1, 2, 3, 4 slabs (bf16, heads of 128 x 128):
  //   16 heads,  4096 tokens (1024)    177   177   182   191
  //   32 heads,  2048 tokens (1024)    112   113   126   142
  //   32 heads,  4096 tokens (2048)    216   196   201   218
  //   32 heads,  8192 tokens (4096)    422   373   364   375
  //   32 heads, 32768 tokens (16384)  1637  1437  1366  1361
  // Heads of 64 columns or key entries gain in the same places (32 heads of 64 x 64,
  // 4096 tokens: 176 in one, 159 by this rule; 8192 tokens: 343 and 292).
  const int64_t chunks = (std::min(a.max_len, a.T) + kC - 1) / kC;
  const int64_t work = std::min(chunks * a.B, n) * a.HV;
  const int slabs = !can_slab(a) || 2 * kSlabCtas > sms || work <= 1024 ? 1 : work <= 2600 ? 2 : work <= 6400 ? 3 : 4;
  const int parts = (1 << slabs) - 1;
  Slab slab = {0, 0, 0};
  for (int i = 0; i < slabs; ++i) {
    slab.first = slab.end;
    slab.more = i + 1 < slabs;
    slab.end = slab.more ? (int)(chunks * ((2 << i) - 1) / parts) : INT_MAX;
    cfg.numAttrs = i > 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, delta_prep_kernel<T, DK>, a, ws, slab, heads);
    if (e != cudaSuccess) return e;
    // half a head per CTA while all of them run at once
    e = half_heads(a, sms) ? chain_t<T, DK, 64>(a, ws, slab, sms, st) : chain_t<T, DK, 128>(a, ws, slab, sms, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t delta_chunk_workspace_bytes(const DeltaView &a) {
  size_t n;
  places(a, nullptr, &n);
  return n;
}

cudaError_t launch_delta_chunks(const DeltaView &a, q1_dtype t, void *workspace, cudaStream_t st) {
  if (t == Q1_BF16) return a.DK == 128 ? chunks_t<__nv_bfloat16, 128>(a, workspace, st) : chunks_t<__nv_bfloat16, 64>(a, workspace, st);
  return a.DK == 128 ? chunks_t<__half, 128>(a, workspace, st) : chunks_t<__half, 64>(a, workspace, st);
}

cudaError_t set_delta_diagnostics(unsigned long long wait_ns, int stall) {
  cudaError_t e = cudaMemcpyToSymbol(c_delta_wait_ns, &wait_ns, sizeof(wait_ns));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(c_delta_stall, &stall, sizeof(stall));
  return e;
}

unsigned int read_and_clear_delta_errors(cudaStream_t st, cudaError_t *err) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_delta_err, sizeof(v), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_delta_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
  if (e == cudaSuccess && v) e = cudaStreamSynchronize(st);
  *err = e;
  return v;
}

}  // namespace q1
