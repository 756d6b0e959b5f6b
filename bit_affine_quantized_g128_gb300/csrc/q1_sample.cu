// Sampling: one token per row of logits from a given uniform number, with
// temperature, top-k, top-p and min-p.
//
// A cluster of 1 to 8 CTAs takes one row.  Each CTA reads its slice of the row
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
// Truncations.  One pass counts the tokens by log2(weight) in bins 1.6 % wide;
// counts alone (32-bit atomics, no weights) give the bin in which top-k ends
// and, since a bin's weights lie between its edges, the few bins in which
// top-p must end.  A second pass sums the exact weights above those bins in
// registers and collects their tokens, which are sorted.
#include <cuda_bf16.h>

#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kPer = 4;              // histogram bins per thread when scanned
constexpr int kBins = kPer * kThreads;
constexpr int kList = 2048;          // at most this many tokens are sorted; a fuller bin is bisected
constexpr int kFrac = 44;            // fractional bits of a weight
constexpr float kRange = 46.f;       // log2 range of the histogram: below it a weight rounds to zero

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

struct alignas(16) SampleShared {
  float2 exp2[1024];
  union {                      // rank 0:
    u64 list[kList];           // the collected tokens, or
    u64 sum[kBins];            // weights of the bins in question, where they hold too many tokens to sort
  };
  unsigned int cnt[kBins];
  // written by the CTAs of the cluster (index: their rank)
  u64 part_sum[2][kMaxCluster];
  float part_max[kMaxCluster];
  int part_idx[kMaxCluster];
  // written by rank 0 into every CTA, a slot per stage (a CTA may read one after
  // rank 0 has begun the next): 0 top-k, 1 top-p's bins, 2 top-p's one bin
  struct Find {
    int lo, hi;                // the bins in question, lo > hi: none
    int many;                  // they hold more than kList tokens
    u64 need;                  // the count (top-k) or weight wanted
  } find[3];
  u64 threshold;               // tokens with a smaller order value are not kept
  // this CTA's own
  unsigned int list_n;
  u64 warp_sum[kWarps], warp_cnt[kWarps];
  float warp_max[kWarps];
  int warp_idx[kWarps];
  u64 found, found_sum;
  int pick[2];
  float c_hi, c_lo;            // log2(e) / temperature
  u64 w_min;
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
  __device__ __forceinline__ void add(const Weight &w) {
    hi += w.hi;
    lo += w.lo;
  }
};

struct RowScale {
  float m, c_hi, c_lo;
  const float2 *exp2;
  // log2 of the weight, rounded (monotone in l); NaN for a NaN logit
  __device__ __forceinline__ float log2w(float l) const {
    if (m == __int_as_float(0x7f800000)) return l == m ? 0.f : -2.f * kRange;
    return (l - m) * c_hi;
  }
  __device__ __forceinline__ int bin(float y) const { return min(kBins - 1, (int)(-y * ((float)kBins / kRange))); }
  // 2^44 exp((l - m) / temperature) as an integer, for y = log2w(l) > -kRange.
  // Adding 1.5 * 2^23 to a number below 2^22 leaves its nearest integer in the
  // low bits of the sum.
  __device__ __forceinline__ Weight weight(float l, float y) const {
    if (y == 0.f) return Weight{1u << 22, 0};
    constexpr float kMagic = 12582912.f;
    constexpr int kMagicBits = 0x4B400000;
    // l - m = s + e exactly (two-sum), times c_hi + c_lo = y + lo
    const float s = l - m, bb = s - l;
    const float e = (l - (s - bb)) - (m + bb);
    const float lo = fmaf(s, c_hi, -y) + fmaf(s, c_lo, e * c_hi);
    const float t = fmaf(y, 1024.f, kMagic);
    const int tb = __float_as_int(t);                       // 2^y = 2^n 2^(i/1024) 2^r
    const float r = fmaf(t - kMagic, -1.f / 1024.f, y) + lo;  // |r| <= 2^-11; the difference is exact
    const float p = r * 0.693147180559945f;
    const float x = fmaf(p * p, fmaf(p, 1.f / 6.f, 0.5f), p);  // e^p - 1
    const float2 h = exp2[tb & 1023];
    const int n = (tb - kMagicBits) >> 10;                  // -46 .. 0
    const float scale = __int_as_float((n + 127 + 22) << 23);
    const float v = h.x * scale;                            // exact
    const float c = fmaf(h.x, x, h.y);
    const float t1 = fmaf(c, scale, v) + kMagic;
    const float rem = fmaf(c, scale, v - (t1 - kMagic));    // at most 3/4; one rounding
    const float t2 = fmaf(rem, 4194304.f, kMagic);
    return Weight{(uint32_t)(__float_as_int(t1) - kMagicBits), __float_as_int(t2) - kMagicBits};
  }
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
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
__device__ __forceinline__ u64 block_scan(u64 *scratch, u64 v, u64 &all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const u64 incl = warp_scan(v, lane);
  __syncthreads();
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  u64 before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const u64 x = scratch[w];
    if (w < warp) before += x;
    all += x;
  }
  return before + incl - v;
}
// This CTA's sum of v, written to slot `rank` of part_sum[par] in CTA `to`, or in all (to < 0)
__device__ __forceinline__ void send_sum(SampleShared &sh, u64 v, int par, uint32_t rank, int cs, int to) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) sh.warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  if ((int)threadIdx.x < cs && (to < 0 || to == (int)threadIdx.x)) {
    u64 all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) all += sh.warp_sum[w];
    *peer(&sh.part_sum[par][rank], threadIdx.x) = all;
  }
}

// floor(x 2^64) for x in [0, 1)
__device__ __forceinline__ u64 fraction(float x) {
  return x > 0.f ? __double2ull_rd((double)x * 18446744073709551616.0) : 0ull;
}

template <typename T>
struct Slice {
  static constexpr int E = 16 / (int)sizeof(T);
  const T *data;   // shared memory, vectors of 16 bytes; places outside the slice hold -inf
  int nv, first;   // vectors, and the row index of the first element of vector 0
  __device__ __forceinline__ void get(int j, float (&f)[E]) const {
    const uint4 v = reinterpret_cast<const uint4 *>(data)[j];
    const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = to_f32(e[i]);
  }
  template <typename F>
  __device__ __forceinline__ void each(F fn) const {  // fn(logit, index)
    for (int j = threadIdx.x; j < nv; j += kThreads) {
      float f[E];
      get(j, f);
#pragma unroll
      for (int i = 0; i < E; ++i) fn(f[i], (uint32_t)(first + j * E + i));
    }
  }
};

// Rank 0, all threads: sorts the collected tokens and finds the last one kept:
// the need-th (by_sum = 0), or the first at which their weights reach need.
// sh.found is its order value, sh.found_sum the weight of the tokens up to it.
__device__ void sort_and_find(SampleShared &sh, const RowScale &rs, int by_sum, u64 need) {
  const int tid = threadIdx.x;
  const int n = (int)min(sh.list_n, (unsigned int)kList);
  int n2 = 1;
  while (n2 < n) n2 <<= 1;
  for (int i = n + tid; i < n2; i += kThreads) sh.list[i] = 0;
  __syncthreads();
  for (int size = 2; size <= n2; size <<= 1)
    for (int step = size >> 1; step > 0; step >>= 1) {  // bitonic sort, descending
      for (int i = tid; i < n2 / 2; i += kThreads) {
        const int x = 2 * i - (i & (step - 1)), z = x + step;
        const u64 p = sh.list[x], q = sh.list[z];
        if ((p < q) == ((x & size) == 0)) {
          sh.list[x] = q;
          sh.list[z] = p;
        }
      }
      // up to step 32 a warp's pairs lie in 64 places of its own
      if (step > 32 || (step == 1 && size > 32)) __syncthreads();
      else __syncwarp();
    }
  constexpr int P = kList / kThreads;
  u64 w[P], s = 0, all;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int at = tid * P + i;
    w[i] = 0;
    if (at < n) {
      const float l = order_logit(sh.list[at]);
      w[i] = rs.weight(l, rs.log2w(l)).whole();
    }
    s += w[i];
  }
  s = block_scan(sh.warp_cnt, s, all);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int at = tid * P + i;
    const bool last = by_sum ? (s < need && need <= s + w[i]) : (u64)(at + 1) == need;
    s += w[i];
    if (at < n && last) {
      sh.found = sh.list[at];
      sh.found_sum = s;
    }
  }
  __syncthreads();
}

// The whole cluster: the last token kept of a bin that holds too many to sort,
// bit by bit: the largest order value with enough tokens (or weight) of the bin
// at or above it.  Bits 31..18 are set in every value (indices are below 2^18).
// In rank 0, sh.found and sh.found_sum as above.
template <typename T>
__device__ void bisect(SampleShared &sh, const Slice<T> &slice, const RowScale &rs, uint32_t rank, int cs, int bin, int by_sum,
                       u64 need) {
  u64 t = 0xFFFC0000ull;
  int par = 0;
  for (int bit = 63; bit >= -1; --bit) {
    if (bit >= 18 && bit < 32) continue;
    const u64 cand = bit >= 0 ? t | (1ull << bit) : t;  // the last round: the weight at or above t
    u64 acc = 0;
    slice.each([&](float l, uint32_t idx) {
      const float y = rs.log2w(l);
      if (y > -kRange && rs.bin(y) == bin && order_value(l, idx) >= cand) acc += by_sum || bit < 0 ? rs.weight(l, y).whole() : 1ull;
    });
    send_sum(sh, acc, par, rank, cs, -1);
    cluster_sync(cs);
    u64 all = 0;
    for (int r = 0; r < cs; ++r) all += sh.part_sum[par][r];
    if (bit < 0) {
      if (threadIdx.x == 0) {
        sh.found = t;
        sh.found_sum = all;
      }
    } else if (all >= need) {
      t = cand;
    }
    par ^= 1;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const q1_sample_args a, int per, int cs) {
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
  const bool greedy = !(temp > 0.f), has_k = top_k > 0 && top_k < a.V, has_p = top_p < 1.f;

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
  if (!greedy)
    for (int i = tid; i < 1024; i += kThreads) sh.exp2[i] = g_exp2.v[i];
  if (has_k || has_p) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) sh.cnt[tid + i * kThreads] = 0;
  }
  if (tid == 0) {
    // log2(e) / temperature in two fp32 parts, small enough to stay finite
    const double c = fmin(1.4426950408889634 / (double)temp, 1.2676506002282294e30);
    sh.c_hi = (float)c;
    sh.c_lo = (float)(c - (double)sh.c_hi);
    const float mp = a.min_p ? a.min_p[b] : a.min_p_value;
    sh.w_min = mp > 0.f ? (u64)ceil((double)fminf(mp, 1.f) * (double)(1ull << kFrac)) : 0;
    sh.threshold = 0;
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
    slice.each([&](float l, uint32_t idx) {
      if (l == m) best = min(best, (int)idx);
    });
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
  const RowScale rs{m, sh.c_hi, sh.c_lo, sh.exp2};

  // ---- the truncations' threshold
  if (has_k || has_p) {
    Weight acc{0, 0};  // all weights, which top-p needs where top-k leaves all
    const bool all = !has_k;
    slice.each([&](float l, uint32_t) {
      const float y = rs.log2w(l);
      if (y > -kRange) {
        atomicAdd(&sh.cnt[rs.bin(y)], 1u);
        if (all) acc.add(rs.weight(l, y));
      }
    });
    send_sum(sh, acc.whole(), 0, rank, cs, 0);
    cluster_sync(cs);
    // rank 0 holds the cluster's counts, kPer bins per thread, and their prefix
    unsigned int c4[kPer] = {};
    u64 c_before = 0, c_all = 0, total = 0, thr = 0;
    if (rank == 0) {
      for (int r = 0; r < cs; ++r) {
        const uint4 c = *reinterpret_cast<const uint4 *>(peer(&sh.cnt[kPer * tid], (uint32_t)r));
        c4[0] += c.x, c4[1] += c.y, c4[2] += c.z, c4[3] += c.w;
        total += sh.part_sum[0][r];
      }
      c_before = block_scan(sh.warp_cnt, (u64)c4[0] + c4[1] + c4[2] + c4[3], c_all);
    }
    auto announce = [&](int stage) {  // rank 0: its find[stage] to the others
      __syncthreads();
      if (tid >= 1 && tid < cs) peer(&sh, (uint32_t)tid)->find[stage] = sh.find[stage];
    };
    // the tokens of bins lo..hi to rank 0's list (or, with `many`, their weights
    // by bin), and the weight of the bins above to its part_sum[1]
    auto collect = [&](int stage) {
      const auto f = sh.find[stage];
      SampleShared *lead = peer(&sh, 0);
      Weight above{0, 0};
      slice.each([&](float l, uint32_t idx) {
        const float y = rs.log2w(l);
        if (!(y > -kRange)) return;
        const int i = rs.bin(y);
        if (i < f.lo) {
          above.add(rs.weight(l, y));
        } else if (i <= f.hi) {
          if (f.many) {
            atomicAdd(&lead->sum[i], rs.weight(l, y).whole());
          } else {
            const unsigned int at = atomicAdd(&lead->list_n, 1u);
            if (at < kList) lead->list[at] = order_value(l, idx);
          }
        }
      });
      send_sum(sh, above.whole(), 1, rank, cs, 0);
      cluster_sync(cs);
    };
    auto above_all = [&]() {
      u64 v = 0;
      for (int r = 0; r < cs; ++r) v += sh.part_sum[1][r];
      return v;
    };
    if (has_k) {
      if (rank == 0) {
        if (tid == 0) {
          sh.find[0] = {1, 0, 0, 0};
          sh.list_n = 0;
        }
        __syncthreads();
        u64 c = c_before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (c < (u64)top_k && (u64)top_k <= c + c4[i])
            sh.find[0] = {kPer * tid + i, kPer * tid + i, c4[i] > kList, (u64)top_k - c};
          c += c4[i];
        }
        announce(0);
      }
      cluster_sync(cs);
      // a top_k beyond the tokens that have a weight keeps them all
      if (sh.find[0].lo > sh.find[0].hi) {
        if (has_p) {  // their weight, which the first pass did not sum
          Weight w{0, 0};
          slice.each([&](float l, uint32_t) {
            const float y = rs.log2w(l);
            if (y > -kRange) w.add(rs.weight(l, y));
          });
          send_sum(sh, w.whole(), 1, rank, cs, 0);
          cluster_sync(cs);
          if (rank == 0) total = above_all();
        }
      } else {
        collect(0);
        const u64 above = rank == 0 ? above_all() : 0;
        if (sh.find[0].many) bisect(sh, slice, rs, rank, cs, sh.find[0].lo, 0, sh.find[0].need);
        else if (rank == 0) sort_and_find(sh, rs, 0, sh.find[0].need);
        if (rank == 0) {
          thr = sh.found;
          total = above + sh.found_sum;
        }
      }
    }
    if (has_p) {
      u64 want = 0;
      if (rank == 0) {
        // kept: less than ceil(top_p * total) before it; the first always is
        const u64 p = fraction(top_p);
        want = __umul64hi(p, total) + (p * total != 0 ? 1 : 0);
        want = want ? want : 1;
        // between the sums that the bins' upper and lower edges give (with a
        // margin for the rounding of bins and weights) lies the end of top-p
        constexpr float kStep = kRange / kBins;
        const int k_bin = has_k && thr ? sh.find[0].hi : kBins - 1;
        u64 up[kPer], dn[kPer], us = 0, ds = 0, any;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const float e = exp2f(44.f - kStep * (float)(kPer * tid + i));
          up[i] = (u64)c4[i] * ((u64)(e * 1.0001f) + 1);
          dn[i] = (u64)c4[i] * (u64)(e * (exp2f(-kStep) * 0.9999f));
          us += up[i];
          ds += dn[i];
        }
        us = block_scan(sh.warp_cnt, us, any);
        ds = block_scan(sh.warp_cnt, ds, any);
        if (tid == 0) {
          sh.pick[0] = k_bin;
          sh.pick[1] = k_bin;
          sh.list_n = 0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (us < want && want <= us + up[i]) atomicMin(&sh.pick[0], kPer * tid + i);
          if (ds < want && want <= ds + dn[i]) atomicMin(&sh.pick[1], kPer * tid + i);
          us += up[i];
          ds += dn[i];
        }
        __syncthreads();
        const int lo = sh.pick[0], hi = max(sh.pick[1], lo);
        u64 in = 0, c_in;
#pragma unroll
        for (int i = 0; i < kPer; ++i) in += kPer * tid + i >= lo && kPer * tid + i <= hi ? c4[i] : 0;
        block_scan(sh.warp_cnt, in, c_in);
        if (tid == 0) sh.find[1] = {lo, hi, c_in > kList, want};
        if (c_in > kList) {
#pragma unroll
          for (int i = 0; i < kPer; ++i) sh.sum[tid + i * kThreads] = 0;
        }
        announce(1);
      }
      cluster_sync(cs);
      collect(1);
      u64 above = 0;
      if (rank == 0) above = above_all();
      if (!sh.find[1].many) {
        if (rank == 0) sort_and_find(sh, rs, 1, want - above);
      } else {
        // their weights by bin tell the bin; then its tokens
        if (rank == 0) {
          u64 w4[kPer], s = 0, any;
          const int lo = sh.find[1].lo, hi = sh.find[1].hi;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            w4[i] = kPer * tid + i >= lo && kPer * tid + i <= hi ? sh.sum[kPer * tid + i] : 0;
            s += w4[i];
          }
          s = above + block_scan(sh.warp_cnt, s, any);
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            if (s < want && want <= s + w4[i]) sh.find[2] = {kPer * tid + i, kPer * tid + i, c4[i] > kList, want - s};
            s += w4[i];
          }
          if (tid == 0) sh.list_n = 0;
          announce(2);
        }
        cluster_sync(cs);
        if (sh.find[2].many) {
          bisect(sh, slice, rs, rank, cs, sh.find[2].lo, 1, sh.find[2].need);
        } else {
          collect(2);
          if (rank == 0) sort_and_find(sh, rs, 1, sh.find[2].need);
        }
      }
      if (rank == 0) thr = thr > sh.found ? thr : sh.found;
    }
    if (rank == 0 && tid < cs) peer(&sh, (uint32_t)tid)->threshold = thr;
    cluster_sync(cs);
  }

  // ---- the kept weight: warp w of a CTA sums a contiguous run of vectors
  const u64 thr = sh.threshold, w_min = sh.w_min;
  const int vw = ((slice.nv + kWarps - 1) / kWarps + 31) & ~31;
  const int v0 = warp * vw, v1 = min(slice.nv, v0 + vw);
  auto kept = [&](float l, uint32_t idx) -> Weight {
    const float y = rs.log2w(l);
    if (!(y > -kRange) || (thr && order_value(l, idx) < thr)) return Weight{0, 0};
    const Weight w = rs.weight(l, y);
    return w_min && w.whole() < w_min ? Weight{0, 0} : w;
  };
  Weight acc{0, 0};
  for (int j = v0 + lane; j < v1; j += 32) {
    float f[E];
    slice.get(j, f);
#pragma unroll
    for (int i = 0; i < E; ++i) acc.add(kept(f[i], (uint32_t)(slice.first + j * E + i)));
  }
  send_sum(sh, acc.whole(), 0, rank, cs, -1);
  cluster_sync(cs);
  u64 total = 0, before = 0;
  for (int r = 0; r < cs; ++r) {
    if (r < (int)rank) before += sh.part_sum[0][r];
    total += sh.part_sum[0][r];
  }
  const float u = a.u[b];
  u64 target = u < 1.f ? __umul64hi(fraction(u), total) : (u >= 1.f ? total - 1 : 0);
  target = target < total ? target : total - 1;
  // ---- the draw: the warp whose run holds the target-th unit of weight
  for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
  if (target < before || target - before >= sh.warp_sum[warp]) return;
  for (int j0 = v0; j0 < v1; j0 += 32) {
    const int j = j0 + lane;
    float f[E];
    u64 w[E], s = 0;
    if (j < v1) slice.get(j, f);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      w[i] = j < v1 ? kept(f[i], (uint32_t)(slice.first + j * E + i)).whole() : 0;
      s += w[i];
    }
    const u64 incl = warp_scan(s, lane);
    const u64 step = __shfl_sync(0xffffffffu, incl, 31);
    if (target - before < step) {
      u64 c = before + incl - s;
      if (target >= c && target < c + s) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          if (target >= c && target < c + w[i]) {
            a.token[b] = slice.first + j * E + i;
            if (a.prob) a.prob[b] = (float)((double)w[i] / (double)total);
          }
          c += w[i];
        }
      }
      return;
    }
    before += step;
  }
}

template <typename T>
cudaError_t sample_t(const q1_sample_args &a, cudaStream_t st) {
  static std::atomic<uint64_t> ready{0};
  constexpr int E = Slice<T>::E;
  const int dev = current_device();
  constexpr size_t kMost = 227 * 1024;  // shared memory of a CTA
  constexpr int64_t kSliceMax = (int64_t)((kMost - sizeof(SampleShared)) / sizeof(T)) - 2 * E - 8;
  if (not_done(ready, dev)) {
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess) return e;
    mark_done(ready, dev);
  }
  // as many CTAs per row as keep two per SM busy, and as the row needs
  int cs = kMaxCluster;
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
