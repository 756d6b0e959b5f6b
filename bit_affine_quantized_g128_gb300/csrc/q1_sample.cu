// Sampling: one token per row of logits from a given uniform number, with
// temperature, top-k, top-p and min-p.
//
// A cluster of 1 to 16 CTAs takes one row.  Each CTA reads its slice of the row
// once, into shared memory; everything after that (maximum, weights, the
// truncations' thresholds, the draw) runs on chip, and the CTAs exchange a few
// words through distributed shared memory.
//
// Exactness.  The token is the answer to comparisons between sums over up to
// V weights, and with tens of thousands of small weights an fp32 sum is off by
// more than one of them.  The weights are therefore fixed-point integers,
// w = 2^44 exp((l - max) / temperature), relative error about 2^-34: integer
// sums are exact and the same in any order (so atomics and any split over
// threads give one answer).  The tokens are ordered by the 64-bit value
// (order-preserving bits of l, ~index), so "before" is one compare and ties
// fall to the lowest index.
//
// Truncations.  The end of top-k is found in rounds of 8 buckets of log2(weight)
// (a row of buckets per thread, no atomics): with small k the first round ends
// it.  The end of top-p takes one pass that counts the tokens in bins of 1/32
// octave, one shared atomic per token (17 clocks of the SM per warp: as much as
// its exact weight costs): since a bin's weights lie between its edges, the counts
// give the few bins in which top-p must end.  Should those hold too many tokens,
// rounds with fp32 weights narrow them.  If all tokens that can be kept are few,
// one CTA finishes the row from a list of them; otherwise a pass with exact
// weights sums those above the bins in question and lists the tokens in them,
// which are sorted for the last one kept.
//
// Bound by latency for few rows (one row of a large vocabulary: 15 us, ten
// dependent steps over 16 CTAs; top-k near 1000 with top-p: 43 us).  For many rows
// by its steps in a row: 28 us for 64 rows (48 instructions per token, 31 of them
// the exact weight: 13 us of full issue), 51 us for 301 rows of 32003 tokens (108
// per token).  Load, maximum, count, weights and sort lie between barriers, all CTAs
// of the single wave go through them together, and half of the issue slots stay
// empty (0.52 and 0.58 per scheduler and clock).
#include <cuda_bf16.h>

#include <type_traits>

#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kOctaves = 46;         // range of log2(weight) in use: below it a weight rounds to zero
constexpr int kRange = 1024 * kOctaves + 1;  // in steps of 1/1024
constexpr int kPer = 3;              // bins per thread when scanned
constexpr int kBins = kPer * kThreads;
static_assert(32 * kBins >= kRange, "bins");
constexpr int kBuckets = 8;          // of a search round
constexpr int kFirstShift = 12;      // the first round's buckets are 4 octaves wide (the last takes the rest)
constexpr float kMargin = 1e-4f;     // above the relative errors of the rounds' fp32 weights (5e-6) and sums (2e-5)
constexpr int kList = 1024;          // at most this many tokens are sorted; a fuller bucket is bisected
constexpr int kRuns = 4;             // a warp's tokens are summed in this many runs
constexpr float kMagic = 12582912.f; // 1.5 * 2^23: adding it leaves the nearest integer in the low bits
constexpr int kMagicBits = 0x4B400000;
constexpr float kDead = kMagic - 1024.f * kOctaves;  // keys below have no weight

typedef unsigned long long u64;

// 2^(i/1024) = hi + lo, the two nearest fp32 values.
struct Exp2Table {
  float2 v[1024];
};
constexpr Exp2Table make_table() {
  Exp2Table t{};
  for (int i = 0; i < 1024; ++i) {
    const double x = (double)i * (0.693147180559945309417232121458 / 1024.0);
    double s = 1.0, term = 1.0;
    for (int n = 1; n < 24; ++n) {
      term = term * x / n;
      s += term;
    }
    const float hi = (float)s;
    t.v[i].x = hi;
    t.v[i].y = (float)(s - (double)hi);
  }
  return t;
}
__device__ const Exp2Table g_exp2 = make_table();

// A row's weights: w(l) = 2^((l - m) c), c = log2(e) / temperature.
struct RowScale {
  float m;            // the largest logit
  float c_hi, c_lo;   // c
  float K, A0, a1;    // m c = A0 + a1 with A0 a multiple of 1/1024; K = kMagic - 1024 A0
  int wide;           // m c is too large for that, or m infinite
  u64 top, least;     // the weight of m, and the least that min-p keeps
};

struct alignas(16) SampleShared {
  float2 exp2[1024];
  union {
    unsigned int count[kBins];
    struct {                        // a search round: a row of buckets per thread
      float sum[kBuckets][kThreads];
      unsigned char cnt[kBuckets][kThreads];
    } own;
    struct {                        // rank 0, after the rounds
      u64 list[kList];              // collected tokens
      u64 weight[kList];            // theirs
    } few;
  };
  // written by the CTAs of the cluster (index: their rank)
  u64 part_sum[2][kMaxCluster];
  u64 part_rest[kMaxCluster];
  float part_max[kMaxCluster];
  int part_idx[kMaxCluster];
  float bucket_sum[2][kMaxCluster][kBuckets];
  unsigned int bucket_cnt[2][kMaxCluster][kBuckets];
  // written by rank 0 into every CTA
  int picked[4];                    // the bins in which top-p ends, the tokens before them and down to their end
  u64 threshold[2];                 // tokens with a smaller order value are not kept: by top-k, by top-p
  unsigned int list_n;              // rank 0: collected tokens
  // this CTA's own
  RowScale rs;
  u64 warp_sum[kWarps];
  u64 run_sum[kWarps][kRuns];       // kept weight of a warp's runs of tokens
  float warp_max[kWarps];
  int warp_idx[kWarps];
  u64 found;
  int pick[4];
};

// The generic address of p's counterpart in CTA `rank` of the cluster.
template <typename P>
__device__ __forceinline__ P *peer(P *p, uint32_t rank) {
  u64 out;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"((u64)p), "r"(rank));
  return reinterpret_cast<P *>(out);
}
__device__ __forceinline__ void cluster_sync(int cs) {
  if (cs == 1) __syncthreads();
  else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T minus_inf();
template <>
__device__ __forceinline__ float minus_inf<float>() { return __int_as_float(0xff800000); }
template <>
__device__ __forceinline__ __half minus_inf<__half>() { return __ushort_as_half(0xfc00); }
template <>
__device__ __forceinline__ __nv_bfloat16 minus_inf<__nv_bfloat16>() { return __ushort_as_bfloat16(0xff80); }

// Larger for an earlier place in the order: larger logit, then lower index.
__device__ __forceinline__ u64 order_value(float l, uint32_t index) {
  const uint32_t b = __float_as_uint(l + 0.f);  // -0 and +0 are equal
  const uint32_t key = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((u64)key << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float order_logit(u64 v) {
  const uint32_t key = (uint32_t)(v >> 32);
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

// A weight 2^44 w as hi 2^22 + lo: two 32-bit sums per thread instead of one of 64 bits
struct Weight {
  uint32_t hi;
  int32_t lo;
  __device__ __forceinline__ u64 whole() const { return ((u64)hi << 22) + (u64)(long long)lo; }
};

// kMagic + rint(1024 log2 w), monotone in l; below kDead, or NaN, where the
// weight is zero.  (Infinite m: the infinities share the weight.)
template <bool WIDE>
__device__ __forceinline__ float key_of(const RowScale &rs, float l) {
  if (!WIDE) return fmaf(l, 1024.f * rs.c_hi, rs.K);
  if (l == rs.m) return kMagic;
  return fmaf(fmaxf((l - rs.m) * rs.c_hi, -1e6f), 1024.f, kMagic) - (l != l ? __int_as_float(0x7fc00000) : 0.f);
}
// 2^44 2^((l - m) c) as an integer, for t = key_of(l) >= kDead: with i + 1024 n =
// t's integer, 2^n 2^(i/1024) 2^r, |r| <= 2^-10 and a little (2^-11 from the key's
// rounding, as much from a1).
template <bool WIDE>
__device__ __forceinline__ Weight weight_of(const RowScale &rs, const float2 *exp2, float l, float t) {
  const float ti = t - kMagic;
  float r;
  if (!WIDE) {
    // l c_hi - (A0 + ti/1024): the bracket is exact, the difference rounded once
    r = fmaf(l, rs.c_hi, -fmaf(ti, 1.f / 1024.f, rs.A0));
    r = fmaf(l, rs.c_lo, r - rs.a1);
  } else if (l == rs.m) {
    r = 0.f;
  } else {
    // l - m = s + e exactly (two-sum)
    const float s = l - rs.m, bb = s - l, e = (l - (s - bb)) - (rs.m + bb), y = s * rs.c_hi;
    r = fmaf(ti, -1.f / 1024.f, y) + (fmaf(s, rs.c_hi, -y) + fmaf(s, rs.c_lo, e * rs.c_hi));
  }
  // 2^r - 1 = r (ln2 + r (ln2^2 / 2 + r ln2^3 / 6))
  const float x = r * fmaf(r, fmaf(r, 0.0555041087f, 0.2402265070f), 0.6931471806f);
  const int tb = __float_as_int(t);
  const float2 h = exp2[tb & 1023];
  const float c = fmaf(h.x, x, h.y);
  const float scale = __int_as_float(((tb << 13) & (int)0xFF800000u) + ((127 + 22) << 23));  // 2^(n + 22)
  const float v = h.x * scale;                          // exact
  const float t1 = fmaf(c, scale, v) + kMagic;          // the nearest integer, or one beside it
  const float rem = fmaf(c, scale, v - (t1 - kMagic));  // at most 3/4; one rounding
  const float t2 = fmaf(rem, 4194304.f, kMagic);
  return Weight{(uint32_t)(__float_as_int(t1) - kMagicBits), __float_as_int(t2) - kMagicBits};
}

// the same where the row's case is not known at compile time
__device__ __forceinline__ float key_any(const RowScale &rs, float l) { return rs.wide ? key_of<true>(rs, l) : key_of<false>(rs, l); }
__device__ __forceinline__ u64 weight_any(const RowScale &rs, const float2 *exp2, float l) {
  return rs.wide ? weight_of<true>(rs, exp2, l, key_of<true>(rs, l)).whole()
                 : weight_of<false>(rs, exp2, l, key_of<false>(rs, l)).whole();
}

__device__ __forceinline__ u64 warp_total(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// inclusive prefix sum over the lanes
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}
// exclusive prefix sum over the block's threads, and the total
__device__ __forceinline__ u64 block_scan(SampleShared &sh, u64 v, u64 &all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const u64 incl = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) sh.warp_sum[warp] = incl;
  __syncthreads();
  u64 before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const u64 x = sh.warp_sum[w];
    if (w < warp) before += x;
    all += x;
  }
  return before + incl - v;
}
// This CTA's sum of v, written to slot `rank` of part_sum[par] in every CTA
__device__ __forceinline__ void send_sum(SampleShared &sh, u64 v, int par, uint32_t rank, int cs) {
  v = warp_total(v);
  if ((threadIdx.x & 31) == 0) sh.warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  if ((int)threadIdx.x < cs) {
    u64 all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += sh.warp_sum[w];
    *peer(&sh.part_sum[par][rank], threadIdx.x) = all;
  }
}
// floor(x 2^64) for x in [0, 1)
__device__ __forceinline__ u64 fraction(float x) {
  if (!(x > 0.f)) return 0;
  const int b = __float_as_int(x), e = (b >> 23) - 86;  // x 2^64 = significand 2^e
  const u64 sig = (u64)((b & 0x7FFFFF) | (b >= 0x800000 ? 0x800000 : 0));
  return e >= 0 ? sig << e : (e > -24 ? sig >> -e : 0);
}
// ceil(x w) for x in [0, 1]
__device__ __forceinline__ u64 part_up(float x, u64 w) {
  if (x >= 1.f) return w;
  const u64 f = fraction(x);
  return __umul64hi(f, w) + (f * w != 0 ? 1 : 0);
}
// floor(u total), within [0, total)
__device__ __forceinline__ u64 draw_target(float u, u64 total) {
  const u64 t = u < 1.f ? __umul64hi(fraction(u), total) : (u >= 1.f ? total - 1 : 0);
  return t < total ? t : total - 1;
}

template <typename T>
struct Slice {
  static constexpr int E = 16 / (int)sizeof(T);
  const T *data;   // shared memory, vectors of 16 bytes; places outside the slice hold -inf
  int nv, first;   // vectors, and the row index of the first element of vector 0
  __device__ __forceinline__ float at(int j) const { return to_f32(data[j]); }
  __device__ __forceinline__ int size() const { return nv * E; }
};

// Ascending (or descending) bitonic sort of n2 (a power of two, at most 1024)
// values in shared memory by the block.  A warp holds 64 neighbouring places in
// registers, two per lane, for the steps up to 32.
__device__ __forceinline__ u64 shuffle_xor(u64 v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ uint32_t shuffle_xor(uint32_t v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
template <typename V>
__device__ __forceinline__ void block_sort(V *v, int n2, bool descending) {
  const int lane = threadIdx.x & 31, base = (threadIdx.x >> 5) * 64;
  __syncthreads();
  for (int size = 2; size <= n2; size <<= 1) {
    for (int step = size >> 1; step >= 64; step >>= 1) {
      const int i = threadIdx.x;
      if (i < n2 / 2) {
        const int x = 2 * i - (i & (step - 1)), z = x + step;
        const V p = v[x], q = v[z];
        if ((p < q) == (((x & size) == 0) == descending)) {
          v[x] = q;
          v[z] = p;
        }
      }
      __syncthreads();
    }
    // all sizes up to 64 in one go
    if (size < 64 && size < n2) continue;
    if (base < n2) {
      const int at0 = base + lane, at1 = at0 + 32;
      V r0 = at0 < n2 ? v[at0] : V(0), r1 = at1 < n2 ? v[at1] : V(0);
      for (int sz = size <= 64 ? 2 : size; sz <= size; sz <<= 1) {
        if (sz >= 64 && n2 > 32) {
          if ((r0 < r1) == (((at0 & sz) == 0) == descending)) {
            const V t = r0;
            r0 = r1;
            r1 = t;
          }
        }
        for (int step = min(sz >> 1, 16); step > 0; step >>= 1) {
          const V p0 = shuffle_xor(r0, step), p1 = shuffle_xor(r1, step);
          // the lower place of a pair keeps the larger value where its run descends
          const bool low = (lane & step) == 0;
          const bool big0 = low == (((at0 & sz) == 0) == descending), big1 = low == (((at1 & sz) == 0) == descending);
          r0 = (r0 < p0) == big0 ? p0 : r0;
          r1 = (r1 < p1) == big1 ? p1 : r1;
        }
      }
      if (at0 < n2) v[at0] = r0;
      if (at1 < n2) v[at1] = r1;
    }
    __syncthreads();
  }
  __syncthreads();
}
__device__ __forceinline__ int power_of_two(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

constexpr int kMine = kList / kThreads;  // collected tokens per thread

// Rank 0, all threads: sorts the collected tokens; sh.found is the order value
// of the need-th of them (by_sum = 0), or of the first at which their weights reach need.
__device__ void find_in_list(SampleShared &sh, const RowScale &rs, int by_sum, u64 need) {
  const int tid = threadIdx.x, n = (int)min(sh.list_n, (unsigned int)kList), n2 = power_of_two(n);
  for (int i = n + tid; i < n2; i += kThreads) sh.few.list[i] = 0;
  block_sort(sh.few.list, n2, true);
  u64 w[kMine], s = 0, all;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int at = tid * kMine + i;
    w[i] = 0;
    if (at < n) {
      const float l = order_logit(sh.few.list[at]);
      w[i] = weight_any(rs, sh.exp2, l);
    }
    s += w[i];
  }
  s = block_scan(sh, s, all);
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int at = tid * kMine + i;
    if (at < n && (by_sum ? (s < need && need <= s + w[i]) : (u64)(at + 1) == need)) sh.found = sh.few.list[at];
    s += w[i];
  }
  __syncthreads();
}

// Rank 0, all threads: every token that can be kept is collected.  Truncates
// the sorted list and draws from what is left, in the order of the indices.
// want: the weight that top-p keeps, or 0 where the list holds all that top-k
// leaves and so tells it.
__device__ void draw_from_list(SampleShared &sh, const RowScale &rs, int top_k, float top_p, u64 want, float u, int32_t *token,
                               float *prob) {
  const int tid = threadIdx.x, n = (int)min(sh.list_n, (unsigned int)kList), n2 = power_of_two(n);
  for (int i = n + tid; i < n2; i += kThreads) sh.few.list[i] = 0;
  block_sort(sh.few.list, n2, true);
  u64 w[kMine], s = 0, total;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int at = tid * kMine + i;
    w[i] = 0;
    if (at < n && (top_k <= 0 || at < top_k)) {
      const float l = order_logit(sh.few.list[at]);
      w[i] = weight_any(rs, sh.exp2, l);
    }
    s += w[i];
  }
  if (top_p < 1.f) {
    u64 before = block_scan(sh, s, total);
    if (!want) want = part_up(top_p, total);
    want = want ? want : 1;  // the first always stays
    s = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const u64 x = w[i];
      if (before >= want) w[i] = 0;
      before += x;
      s += w[i];
    }
  }
  s = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (w[i] < rs.least) w[i] = 0;
    s += w[i];
    if (tid * kMine + i < n2) sh.few.weight[tid * kMine + i] = w[i];
  }
  block_scan(sh, s, total);  // its barriers publish the weights
  // the places of the tokens by index: (index, place) in 32 bits
  uint32_t *by_index = reinterpret_cast<uint32_t *>(sh.exp2);
  for (int i = tid; i < n2; i += kThreads) by_index[i] = i < n ? ((uint32_t)~(uint32_t)sh.few.list[i] << 10) | (uint32_t)i : 0xFFFFFFFFu;
  block_sort(by_index, n2, false);
  uint32_t at[kMine];
  s = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int j = tid * kMine + i;
    at[i] = j < n ? by_index[j] : 0u;
    w[i] = j < n ? sh.few.weight[at[i] & (kList - 1)] : 0;
    s += w[i];
  }
  u64 all;
  s = block_scan(sh, s, all);
  const u64 target = draw_target(u, total);
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (target >= s && target - s < w[i]) {
      *token = (int32_t)(at[i] >> 10);
      if (prob) *prob = (float)((double)w[i] / (double)total);
    }
    s += w[i];
  }
}

// The same for a list of at most kShort tokens, without sorting: four threads
// per token go through the list, once for what lies before it in the order, once
// for what lies before it by index.
constexpr int kShort = kThreads / 2;
__device__ void draw_from_short_list(SampleShared &sh, const RowScale &rs, int top_k, float top_p, u64 want, float u,
                                     int32_t *token, float *prob) {
  const int tid = threadIdx.x, n = (int)sh.list_n, part = tid & 3;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const float l = order_logit(sh.few.list[i]);
    sh.few.weight[i] = weight_any(rs, sh.exp2, l);
  }
  __syncthreads();
  constexpr int R = kShort / (kThreads / 4);  // tokens per thread
  u64 mine[R], w[R], before[R], s = 0, total;
  int ahead[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (tid >> 2) + r * (kThreads / 4);
    before[r] = 0;
    ahead[r] = 0;
    mine[r] = i < n ? sh.few.list[i] : 0;
    w[r] = i < n ? sh.few.weight[i] : 0;
    if (i < n) {
      for (int j = part; j < n; j += 4)
        if (sh.few.list[j] > mine[r]) {
          ++ahead[r];
          before[r] += sh.few.weight[j];
        }
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
      ahead[r] += __shfl_xor_sync(0xffffffffu, ahead[r], o);
      before[r] += __shfl_xor_sync(0xffffffffu, before[r], o);
    }
    if (top_k > 0 && ahead[r] >= top_k) w[r] = 0;
    if (part == 0) s += w[r];
  }
  if (top_p < 1.f) {
    if (!want) {
      block_scan(sh, s, total);
      want = part_up(top_p, total);
      want = want ? want : 1;
    }
  } else {
    want = ~0ull;
  }
  s = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (tid >> 2) + r * (kThreads / 4);
    if (before[r] >= want || w[r] < rs.least) w[r] = 0;
    if (part == 0) {
      s += w[r];
      if (i < n) sh.few.weight[i] = w[r];
    }
  }
  block_scan(sh, s, total);  // its barriers publish the weights
  const u64 target = draw_target(u, total);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (tid >> 2) + r * (kThreads / 4);
    u64 c = 0;
    if (i < n) {
      for (int j = part; j < n; j += 4)
        if ((uint32_t)sh.few.list[j] > (uint32_t)mine[r]) c += sh.few.weight[j];  // ~index: larger is earlier
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (i < n && part == 0 && target >= c && target - c < w[r]) {
      *token = (int32_t)~(uint32_t)mine[r];
      if (prob) *prob = (float)((double)w[r] / (double)total);
    }
  }
}

// The whole cluster, where too many tokens are left for a list: bit by bit, the
// largest order value with enough tokens (or weight) at or above it.  Bits
// 31..18 are set in every value (indices are below 2^18).  It writes both slots of
// part_sum: what the caller read of them has to lie behind a barrier of the
// cluster.  Its last round reads slot 1, so slot 0 may be written after it.
template <typename T>
__device__ u64 bisect(SampleShared &sh, const Slice<T> &slice, const RowScale &rs, uint32_t rank, int cs, u64 from, bool by_sum,
                      u64 need) {
  u64 t = 0xFFFC0000ull;
  int par = 0;
  for (int bit = 63; bit >= 0; --bit) {
    if (bit >= 18 && bit < 32) continue;
    const u64 cand = t | (1ull << bit);
    u64 acc = 0;
    for (int j = threadIdx.x; j < slice.size(); j += kThreads) {
      const float l = slice.at(j);
      const u64 value = order_value(l, (uint32_t)(slice.first + j));
      if (key_any(rs, l) >= kDead && value >= cand && value >= from) acc += by_sum ? weight_any(rs, sh.exp2, l) : 1ull;
    }
    send_sum(sh, acc, par, rank, cs);
    cluster_sync(cs);
    u64 all = 0;
    for (int r = 0; r < cs; ++r) all += sh.part_sum[par][r];
    if (all >= need) t = cand;
    par ^= 1;
  }
  return t;
}

// The window of a search: steps [d0, d1) of 1/1024 octave below the largest
// logit, with what lies above it and in it.
struct Window {
  int d0, d1;
  unsigned int above, in;  // tokens
  float above_sum;
};

// The whole cluster: the bins in which the end of the share `share` of the weight
// lies, from counts of the tokens of order value `from` on.
template <typename T, bool WIDE>
__device__ Window count_bins(SampleShared &sh, const Slice<T> &slice, const RowScale &rs, uint32_t rank, int cs, u64 from, float share) {
  const int tid = threadIdx.x;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i) sh.count[tid + i * kThreads] = 0;
  __syncthreads();
#pragma unroll 4
  for (int j = tid; j < slice.size(); j += kThreads) {
    const float l = slice.at(j), t = key_of<WIDE>(rs, l);
    if (t >= kDead && (!from || order_value(l, (uint32_t)(slice.first + j)) >= from))
      atomicAdd(&sh.count[(kMagicBits - __float_as_int(t)) >> 5], 1u);
  }
  cluster_sync(cs);
  if (rank == 0) {
    unsigned int c[kPer] = {};
#pragma unroll 4
    for (int r = 0; r < cs; ++r) {
      const unsigned int *h = peer(&sh.count[kPer * tid], (uint32_t)r);
#pragma unroll
      for (int i = 0; i < kPer; ++i) c[i] += h[i];
    }
    // prefixes: tokens, and weights by the bins' upper and lower edges (the keys
    // in them are rounded), in units of 2^-40 of the largest weight
    u64 up[kPer], dn[kPer], cn = 0, un = 0, ln = 0, all, up_all, dn_all;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float e = exp2f(40.f - (float)(kPer * tid + i) * (1.f / 32.f));
      up[i] = (u64)c[i] * ((u64)(e * 1.0005f) + 1);
      dn[i] = (u64)c[i] * (u64)(e * 0.9787f);  // 2^(-31.5/1024) = 0.97890
      cn += c[i];
      un += up[i];
      ln += dn[i];
    }
    cn = block_scan(sh, cn, all);
    un = block_scan(sh, un, up_all);
    ln = block_scan(sh, ln, dn_all);
    if (tid == 0) sh.pick[0] = sh.pick[1] = kBins - 1;
    __syncthreads();
    // The share of the weight down to the end of a bin is at most un / (un + the
    // lower edges of the rest) and at least ln / (ln + the upper edges of the
    // rest): the first bins at which these reach `share` enclose the end.
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      un += up[i];
      ln += dn[i];
      if (c[i]) {
        if ((float)un * (1.f - share) * 1.00001f >= share * (float)(dn_all - ln)) atomicMin(&sh.pick[0], kPer * tid + i);
        if ((float)ln * (1.f - share) >= share * (float)(up_all - un) * 1.00001f) atomicMin(&sh.pick[1], kPer * tid + i);
      }
    }
    __syncthreads();
    const int lo = sh.pick[0], hi = max(lo, sh.pick[1]);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int bin = kPer * tid + i;
      if (bin == lo) sh.pick[2] = (int)cn;
      cn += c[i];
      if (bin == hi) sh.pick[3] = (int)cn;
    }
    __syncthreads();
    if (tid < cs * 4) {
      SampleShared *d = peer(&sh, (uint32_t)(tid >> 2));
      d->picked[tid & 3] = (tid & 3) == 1 ? max(lo, sh.pick[1]) : sh.pick[tid & 3];
    }
  }
  cluster_sync(cs);
  const unsigned int above = (unsigned int)sh.picked[2];
  return Window{32 * sh.picked[0], min(kRange, 32 * (sh.picked[1] + 1)), above, (unsigned int)sh.picked[3] - above, 0.f};
}

// The whole cluster: rounds of kBuckets until the want-th token, or (SUMS) the end
// of the share `share` of the weight, is among few tokens.  Only tokens from
// order value `from` on count.  An empty window (d1 < 0): fewer than wanted.
template <typename T, bool WIDE, bool SUMS>
__device__ Window search(SampleShared &sh, const Slice<T> &slice, const RowScale &rs, uint32_t rank, int cs, u64 from, unsigned int want,
                         float share, int &par) {

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Window win{0, kRange, 0, 0, 0.f};
  int shift = kFirstShift;
  float goal = 0.f;
  for (bool first = true;; first = false) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBuckets; ++i) {
      if (SUMS) sh.own.sum[i][tid] = 0.f;
      sh.own.cnt[i][tid] = 0;
    }
    const int d_span = win.d1 - win.d0;
    const float mc = fmaf(rs.m, rs.c_hi, 0.f);
#pragma unroll 4
    for (int j = tid; j < slice.size(); j += kThreads) {
      const float l = slice.at(j), t = key_of<WIDE>(rs, l);
      const int d = kMagicBits - __float_as_int(t) - win.d0;
      if (t >= kDead && (unsigned int)d < (unsigned int)d_span && (!from || order_value(l, (uint32_t)(slice.first + j)) >= from)) {
        const int i = min(d >> shift, kBuckets - 1);
        sh.own.cnt[i][tid] += 1;
        if (SUMS) {
          const float y = WIDE ? (l - rs.m) * rs.c_hi : fmaf(l, rs.c_hi, -mc);
          float w;
          asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(WIDE && l == rs.m ? 0.f : y));
          sh.own.sum[i][tid] += w;
        }
      }
    }
    __syncthreads();
    // two warps per bucket: its sums over the threads
    {
      const int i = warp >> 1;
      unsigned int c = 0;
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < kThreads / 64; ++k) {
        const int at = (warp & 1) * 32 + lane + 64 * k;
        c += sh.own.cnt[i][at];
        if (SUMS) x += sh.own.sum[i][at];
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        c += __shfl_xor_sync(0xffffffffu, c, o);
        if (SUMS) x += __shfl_xor_sync(0xffffffffu, x, o);
      }
      if (lane == 0) {
        sh.warp_idx[warp] = (int)c;
        sh.warp_max[warp] = x;
      }
    }
    __syncthreads();
    if (tid < kBuckets * cs) {
      const int i = tid % kBuckets, to = tid / kBuckets;
      SampleShared *d = peer(&sh, (uint32_t)to);
      d->bucket_cnt[par][rank][i] = (unsigned int)(sh.warp_idx[2 * i] + sh.warp_idx[2 * i + 1]);
      if (SUMS) d->bucket_sum[par][rank][i] = sh.warp_max[2 * i] + sh.warp_max[2 * i + 1];
    }
    cluster_sync(cs);
    unsigned int c[kBuckets];
    float x[kBuckets], all = 0.f;
#pragma unroll
    for (int i = 0; i < kBuckets; ++i) {
      c[i] = 0;
      x[i] = 0.f;
      for (int r = 0; r < cs; ++r) {
        c[i] += sh.bucket_cnt[par][r][i];
        if (SUMS) x[i] += sh.bucket_sum[par][r][i];
      }
      all += x[i];
    }
    par ^= 1;
    if (SUMS && first) goal = share * all;
    // the buckets in which the end lies: one, or (sums) those within the margin
    int b0 = -1, b1 = -1;
    unsigned int n = win.above, n0 = win.above, n1 = 0;
    float s = win.above_sum, s0 = win.above_sum;
#pragma unroll
    for (int i = 0; i < kBuckets; ++i) {
      const unsigned int n_in = n + c[i];
      const float s_in = s + x[i];
      if (b0 < 0 && (SUMS ? s_in >= goal * (1.f - kMargin) : n_in >= want)) {
        b0 = i;
        n0 = n;
        s0 = s;
      }
      if (b1 < 0 && (SUMS ? s_in >= goal * (1.f + kMargin) : n_in >= want)) {
        b1 = i;
        n1 = n_in;
      }
      n = n_in;
      s = s_in;
    }
    if (b0 < 0) {
      if (!SUMS) return Window{0, -1, 0, 0, 0.f};
      b0 = kBuckets - 1;
      n0 = n - c[kBuckets - 1];
      s0 = s - x[kBuckets - 1];
    }
    if (b1 < 0) {
      b1 = kBuckets - 1;
      n1 = n;
    }
    const int d1 = b1 == kBuckets - 1 ? win.d1 : win.d0 + ((b1 + 1) << shift);
    win = Window{win.d0 + (b0 << shift), d1, n0, n1 - n0, s0};
    if (win.in <= (unsigned int)kList || shift == 0) return win;
    // the next round's buckets cover the window (the last one taking the rest of
    // a wide one); where a round could not narrow it, no other would
    const int last_shift = shift;
    while (shift > 0 && (kBuckets << (shift - 1)) >= win.d1 - win.d0) --shift;
    if (shift == last_shift && win.d1 - win.d0 >= d_span) return win;
  }
}

// Exact weights over the slice, in runs of each warp.  LIST: sh.run_sum gets those
// of tokens above key t_hi, the result is this thread's weight at or below it, and
// tokens with keys in [t_lo, t_hi] go to rank 0's list.  Otherwise sh.run_sum gets
// all.  TESTS: tokens before order value `from` or with less weight than `least`
// do not count.
template <typename T, bool WIDE, bool TESTS, bool LIST>
__device__ u64 exact_pass(SampleShared &sh, const Slice<T> &slice, const RowScale &rs, u64 from, u64 least, float t_lo, float t_hi) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_run = ((slice.size() + kWarps * kRuns - 1) / (kWarps * kRuns) + 31) & ~31;
  SampleShared *lead = peer(&sh, 0);
  Weight rest{0, 0};
  for (int run = 0; run < kRuns; ++run) {
    const int j0 = (warp * kRuns + run) * per_run, j1 = min(slice.size(), j0 + per_run);
    Weight above{0, 0};
#pragma unroll 4
    for (int j = j0 + lane; j < j1; j += 32) {
      const float l = slice.at(j), t = key_of<WIDE>(rs, l);
      const Weight w = weight_of<WIDE>(rs, sh.exp2, l, t);
      bool live = t >= kDead;
      if (TESTS) live = live && w.whole() >= least && order_value(l, (uint32_t)(slice.first + j)) >= from;
      const bool up = LIST ? live && t > t_hi : live;
      above.hi += up ? w.hi : 0;
      above.lo += up ? w.lo : 0;
      if (LIST) {
        const bool down = live && !up;
        rest.hi += down ? w.hi : 0;
        rest.lo += down ? w.lo : 0;
        if (down && t >= t_lo) {
          const unsigned int at = atomicAdd(&lead->list_n, 1u);
          if (at < kList) lead->few.list[at] = order_value(l, (uint32_t)(slice.first + j));
        }
      }
    }
    const u64 all = warp_total(above.whole());
    if (lane == 0) sh.run_sum[warp][run] = all;
  }
  return rest.whole();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const q1_sample_args a, int per, int cs) {
  extern __shared__ __align__(16) unsigned char dyn[];
  SampleShared &sh = *reinterpret_cast<SampleShared *>(dyn);
  T *data = reinterpret_cast<T *>(dyn + sizeof(SampleShared));
  constexpr int E = Slice<T>::E;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x / (unsigned)cs;
  const uint32_t rank = blockIdx.x - (uint32_t)b * cs;
  if (cs > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // peers may write once all have arrived
  const float temp = a.temperature ? a.temperature[b] : a.temperature_value;
  const int top_k = a.top_k ? a.top_k[b] : a.top_k_value;
  const float top_p = a.top_p ? a.top_p[b] : a.top_p_value;
  const float u = a.u[b];
  const bool greedy = !(temp > 0.f), has_p = top_p < 1.f;
  bool has_k = top_k > 0 && top_k < a.V;

  // ---- this CTA's slice into shared memory, and its maximum
  const int64_t i0 = min((int64_t)rank * per, a.V);
  const int n = (int)(min(i0 + per, a.V) - i0);
  const T *src = static_cast<const T *>(a.logits) + b * a.row_stride + i0;
  const int phase = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
  const Slice<T> slice{data, (phase + n + E - 1) / E, (int)i0 - phase};
  float mx = __int_as_float(0xff800000);
#pragma unroll 4
  for (int j = tid; j < slice.nv; j += kThreads) {
    const int lo = j * E - phase;
    uint4 v;
    T *e = reinterpret_cast<T *>(&v);
    if (lo >= 0 && lo + E <= n) {
      v = __ldcs(reinterpret_cast<const uint4 *>(src + lo));
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) e[i] = lo + i >= 0 && lo + i < n ? src[lo + i] : minus_inf<T>();
    }
    reinterpret_cast<uint4 *>(data)[j] = v;
#pragma unroll
    for (int i = 0; i < E; ++i) mx = fmaxf(mx, to_f32(e[i]));  // a NaN is passed over
  }
  if (!greedy) {
#pragma unroll
    for (int i = 0; i < 1024 / kThreads; ++i) sh.exp2[tid + i * kThreads] = g_exp2.v[tid + i * kThreads];
  }
  if (tid == 0) {
    // small enough that its products stay finite
    const double c = fmin(1.4426950408889634 / (double)temp, 1.2676506002282294e30);
    sh.rs.c_hi = (float)c;
    sh.rs.c_lo = (float)(c - (double)sh.rs.c_hi);
    sh.rs.top = 0;
    sh.rs.least = 0;
    sh.threshold[0] = sh.threshold[1] = 0;
    sh.list_n = 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) sh.warp_max[warp] = mx;
  __syncthreads();
  if (cs > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid < cs) {
    float m = sh.warp_max[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sh.warp_max[w]);
    *peer(&sh.part_max[rank], (uint32_t)tid) = m;
  }
  cluster_sync(cs);
  float m = sh.part_max[0];
  for (int r = 1; r < cs; ++r) m = fmaxf(m, sh.part_max[r]);
  if (!(m > __int_as_float(0xff800000))) {  // nothing to keep
    if (rank == 0 && tid == 0) {
      a.token[b] = -1;
      if (a.prob) a.prob[b] = 0.f;
    }
    return;
  }
  if (greedy) {
    int best = 0x7fffffff;
    for (int j = tid; j < slice.size(); j += kThreads)
      if (slice.at(j) == m) {
        best = slice.first + j;
        break;
      }
    best = __reduce_min_sync(0xffffffffu, best);
    if (lane == 0) sh.warp_idx[warp] = best;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) best = min(best, sh.warp_idx[w]);
      *peer(&sh.part_idx[rank], 0) = best;
    }
    cluster_sync(cs);
    if (rank == 0 && tid == 0) {
      for (int r = 0; r < cs; ++r) best = min(best, sh.part_idx[r]);
      a.token[b] = best;
      if (a.prob) a.prob[b] = 1.f;
    }
    return;
  }
  if (tid == 0) {
    RowScale rs = sh.rs;
    rs.m = m;
    const double mc = (double)m * (double)rs.c_hi;  // exact
    rs.wide = !(fabs(mc) < 4096.0);
    rs.K = rs.A0 = rs.a1 = 0.f;
    if (!rs.wide) {
      // rounded as key_of rounds (|m c_hi| 1024 is below 2^22), so that m's key is
      // kMagic and no key exceeds it
      const float grid = fmaf(m, 1024.f * rs.c_hi, kMagic) - kMagic;
      rs.A0 = grid * (1.f / 1024.f);
      rs.K = kMagic - grid;
      rs.a1 = fmaf(m, rs.c_lo, fmaf(m, rs.c_hi, -rs.A0));
    }
    const float mp = a.min_p ? a.min_p[b] : a.min_p_value;
    if (mp > 0.f) {
      rs.top = weight_any(rs, sh.exp2, m);
      rs.least = part_up(mp, rs.top);
    }
    sh.rs = rs;
  }
  __syncthreads();
  const RowScale rs = sh.rs;

  // ---- the truncations
  u64 thr = 0;            // tokens with a smaller order value are not kept
  bool summed = false;    // sh.run_sum holds the kept weights
  int par = 0;
  auto run_search = [&](bool sums, unsigned int want, float share) -> Window {
    if (!sums) return rs.wide ? search<T, true, false>(sh, slice, rs, rank, cs, thr, want, share, par)
                              : search<T, false, false>(sh, slice, rs, rank, cs, thr, want, share, par);
    const Window w = rs.wide ? count_bins<T, true>(sh, slice, rs, rank, cs, thr, share)
                             : count_bins<T, false>(sh, slice, rs, rank, cs, thr, share);
    if (w.in <= (unsigned int)kList) return w;
    return rs.wide ? search<T, true, true>(sh, slice, rs, rank, cs, thr, want, share, par)
                   : search<T, false, true>(sh, slice, rs, rank, cs, thr, want, share, par);
  };
  auto run_exact = [&](u64 from, float t_lo, float t_hi) -> u64 {  // top-p's: with a list
    if (rs.wide) return exact_pass<T, true, true, true>(sh, slice, rs, from, 0, t_lo, t_hi);
    if (from) return exact_pass<T, false, true, true>(sh, slice, rs, from, 0, t_lo, t_hi);
    return exact_pass<T, false, false, true>(sh, slice, rs, 0, 0, t_lo, t_hi);
  };
  auto run_kept = [&](u64 from) {
    if (rs.wide) exact_pass<T, true, true, false>(sh, slice, rs, from, rs.least, 0.f, 0.f);
    else if (from || rs.least) exact_pass<T, false, true, false>(sh, slice, rs, from, rs.least, 0.f, 0.f);
    else exact_pass<T, false, false, false>(sh, slice, rs, 0, 0, 0.f, 0.f);
  };
  auto key_at = [&](int d) { return __int_as_float(kMagicBits - d); };
  auto draw = [&](int k, u64 want) {  // rank 0
    float *prob = a.prob ? a.prob + b : nullptr;
    if (sh.list_n <= kShort) draw_from_short_list(sh, rs, k, top_p, want, u, a.token + b, prob);
    else draw_from_list(sh, rs, k, top_p, want, u, a.token + b, prob);
  };
  auto announce = [&](int which, u64 value) {  // rank 0's value to everyone
    if (rank == 0 && tid < cs) peer(&sh, (uint32_t)tid)->threshold[which] = value;
    cluster_sync(cs);
    return sh.threshold[which];
  };
  if (has_k) {
    const Window w = run_search(false, (unsigned int)top_k, 0.f);
    has_k = w.d1 > 0;  // a top_k beyond the tokens that have a weight keeps them all
    if (has_k) {
      const bool few = w.above + w.in <= (unsigned int)kList;
      if (few || w.in <= (unsigned int)kList) {
        const float t_lo = key_at(w.d1 - 1), t_hi = few ? kMagic : key_at(w.d0);
        SampleShared *lead = peer(&sh, 0);
        auto collect = [&](auto wide) {
#pragma unroll 4
          for (int j = tid; j < slice.size(); j += kThreads) {
            const float l = slice.at(j), t = key_of<decltype(wide)::value>(rs, l);
            if (t >= t_lo && t <= t_hi) {
              const unsigned int at = atomicAdd(&lead->list_n, 1u);
              if (at < kList) lead->few.list[at] = order_value(l, (uint32_t)(slice.first + j));
            }
          }
        };
        if (rs.wide) collect(std::true_type{});
        else collect(std::false_type{});
        cluster_sync(cs);
        if (few) {
          if (rank == 0) draw(top_k, 0);
          return;
        }
        if (rank == 0) {
          find_in_list(sh, rs, 0, (u64)top_k - w.above);
          if (tid == 0) sh.list_n = 0;
        }
        thr = announce(0, sh.found);
      } else {
        thr = bisect(sh, slice, rs, rank, cs, 0, false, (u64)top_k);
      }
    }
  }
  if (has_p) {
    const Window w = run_search(true, 0, top_p);
    const bool few = w.above + w.in <= (unsigned int)kList, many = !few && w.in > (unsigned int)kList;
    const float t_lo = many ? 2.f * kMagic : key_at(w.d1 - 1), t_hi = few || many ? 2.f * kMagic : key_at(w.d0);
    const u64 rest = run_exact(thr, t_lo, t_hi);
    // the weight above the window, and the rest
    u64 mine = 0;
    __syncwarp();
    if (lane < kRuns) mine = sh.run_sum[warp][lane];
    send_sum(sh, mine, 0, rank, cs);
    __syncthreads();
    {
      const u64 r = warp_total(rest);
      if (lane == 0) sh.warp_sum[warp] = r;
      __syncthreads();
      if (tid < cs) {
        u64 all = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) all += sh.warp_sum[i];
        peer(&sh, (uint32_t)tid)->part_rest[rank] = all;
      }
    }
    cluster_sync(cs);
    u64 above = 0, total = 0;
    for (int r = 0; r < cs; ++r) {
      above += sh.part_sum[0][r];
      total += sh.part_rest[r];
    }
    total += above;
    // kept: less than ceil(top_p * weight) before it; the first always is
    u64 want = part_up(top_p, total);
    want = want ? want : 1;
    if (few) {
      if (rank == 0) draw(has_k ? top_k : 0, want);
      return;
    }
    u64 last = 0;
    if (!many) {
      if (rank == 0) {
        if (tid == 0) sh.found = 0;
        if (want > above) find_in_list(sh, rs, 1, want - above);
      }
      __syncthreads();
      last = announce(1, sh.found);
      if (last && !rs.least) {
        // the list's kept tokens join the sums of their runs
        if (rank == 0) {
          const int n_list = (int)min(sh.list_n, (unsigned int)kList);
          for (int i = tid; i < n_list; i += kThreads) {
            const u64 value = sh.few.list[i];
            if (value >= last) {
              const int index = (int)~(uint32_t)value, r = index / per;
              // that CTA's slice: its first vector may begin before its first token
              const int f0 = r * per, ph = (int)((reinterpret_cast<uintptr_t>(static_cast<const T *>(a.logits) + b * a.row_stride + f0) & 15) / sizeof(T));
              const int len = (int)(min((int64_t)f0 + per, a.V) - f0), size = (ph + len + E - 1) / E * E;
              const int per_run = ((size + kWarps * kRuns - 1) / (kWarps * kRuns) + 31) & ~31;
              const int run = (index - f0 + ph) / per_run;
              atomicAdd(&peer(&sh, (uint32_t)r)->run_sum[run / kRuns][run % kRuns], weight_any(rs, sh.exp2, order_logit(value)));
            }
          }
        }
        cluster_sync(cs);
        summed = true;
      }
    }
    if (!last) {
      cluster_sync(cs);  // every CTA has read the sums above
      last = bisect(sh, slice, rs, rank, cs, thr, true, want);
    }
    thr = max(thr, last);
  }

  // ---- the kept weight by warp and run, and the draw
  if (!summed) run_kept(thr);
  __syncwarp();
  send_sum(sh, lane < kRuns ? sh.run_sum[warp][lane] : 0, 0, rank, cs);
  cluster_sync(cs);
  u64 total = 0, before = 0;
  for (int r = 0; r < cs; ++r) {
    if (r < (int)rank) before += sh.part_sum[0][r];
    total += sh.part_sum[0][r];
  }
  const u64 target = draw_target(u, total);
  for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
  if (target < before || target - before >= sh.warp_sum[warp]) return;
  int run = 0;
  while (target - before >= sh.run_sum[warp][run]) before += sh.run_sum[warp][run++];
  const int per_run = ((slice.size() + kWarps * kRuns - 1) / (kWarps * kRuns) + 31) & ~31;
  const int j1 = min(slice.size(), (warp * kRuns + run + 1) * per_run);
  for (int j0 = (warp * kRuns + run) * per_run; j0 < j1; j0 += 32) {
    const int j = j0 + lane;
    u64 w = 0;
    if (j < j1) {
      const float l = slice.at(j);
      if (key_any(rs, l) >= kDead && order_value(l, (uint32_t)(slice.first + j)) >= thr) w = weight_any(rs, sh.exp2, l);
      if (w < rs.least) w = 0;
    }
    const u64 incl = warp_scan(w, lane);
    const u64 step = __shfl_sync(0xffffffffu, incl, 31);
    if (target - before < step) {
      const u64 c = before + incl - w;
      if (target >= c && target - c < w) {
        a.token[b] = slice.first + j;
        if (a.prob) a.prob[b] = (float)((double)w / (double)total);
      }
      return;
    }
    before += step;
  }
}

template <typename T>
cudaError_t sample_t(const q1_sample_args &a, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  static std::atomic<int> largest[kMaxDevices];  // clusters of so many CTAs can be had
  constexpr int E = Slice<T>::E;
  const int dev = current_device();
  constexpr size_t kMost = 227 * 1024;  // shared memory of a CTA
  constexpr int64_t kSliceMax = (int64_t)((kMost - sizeof(SampleShared)) / sizeof(T)) - 2 * E - 8;
  int most = dev < kMaxDevices ? largest[dev].load(std::memory_order_relaxed) : 0;
  if (not_done(ready, dev) || !most) {
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    cudaLaunchConfig_t full{};
    full.gridDim = dim3(kMaxCluster);
    full.blockDim = dim3(kThreads);
    full.dynamicSmemBytes = kMost;
    if (e == cudaSuccess) e = cudaOccupancyMaxPotentialClusterSize(&most, sample_kernel<T>, &full);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) largest[dev].store(most, std::memory_order_relaxed);
    mark_done(ready, dev);
  }
  // as many CTAs per row as keep two per SM busy, and as the row needs: with 16
  // instead of 8, one row of 152064 logits took 16.5 us instead of 20.0; 64 rows
  // on 4 each 28 us
  int cs = most >= 16 ? 16 : 8;
  while (cs > 1 && a.B * cs > 2 * 152 && (a.V + cs / 2 - 1) / (cs / 2) <= kSliceMax) cs /= 2;
  const int per = (int)((a.V + cs - 1) / cs + 7) & ~7;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * cs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(SampleShared) + ((size_t)per + 2 * E) * sizeof(T);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cs;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, per, cs);
}

}  // namespace

cudaError_t launch_sample(const q1_sample_args &a, cudaStream_t st) {
  if (a.dtype == Q1_BF16) return sample_t<__nv_bfloat16>(a, st);
  if (a.dtype == Q1_F16) return sample_t<__half>(a, st);
  return sample_t<float>(a, st);
}

}  // namespace q1
