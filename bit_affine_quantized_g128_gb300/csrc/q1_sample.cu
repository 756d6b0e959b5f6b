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
// Truncations.  One pass makes a histogram over log2(weight), in bins of 1/32:
// counts for top-k (no weights computed), counts and exact weights for top-p.
// It gives the bin in which the kept tokens end, exactly.  If few tokens lie
// down to that bin, they go to one CTA, which sorts them and does the rest
// with that list.  Otherwise the tokens of that one bin are sorted for the
// order value of the last kept token, and a pass over the row sums the kept
// weights by warp, which leads to the token.
#include <cuda_bf16.h>

#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kOctaves = 46;         // range of log2(weight) in use: below it a weight rounds to zero
constexpr int kPer = 3;              // histogram bins per thread when scanned
constexpr int kBins = kPer * kThreads;
static_assert(kBins >= 32 * kOctaves, "bins");
constexpr int kList = 1024;          // at most this many tokens are sorted; a fuller bin is bisected
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
    struct {
      unsigned int cnt[kBins];      // tokens per bin
      unsigned int sum[3][kBins];   // their weights in pieces of 15 bits
    } hist;
    struct {                        // rank 0, once the histograms are read:
      u64 list[kList];              // collected tokens
      u64 weight[kList];            // theirs, in order
    } few;
  };
  // written by the CTAs of the cluster (index: their rank)
  u64 part_sum[2][kMaxCluster];
  float part_max[kMaxCluster];
  int part_idx[kMaxCluster];
  // written by rank 0 into every CTA, a slot per search (a CTA may read one
  // after rank 0 has begun the next)
  struct Find {
    int lo, hi;                     // bins whose tokens are collected; lo > hi: nothing to find
    int few;                        // all tokens that can be kept are among them
    int many;                       // more than kList tokens
    u64 need;                       // the count or weight wanted from bin hi
  } find[2];
  u64 threshold;                    // tokens with a smaller order value are not kept
  unsigned int list_n;              // rank 0: collected tokens
  // this CTA's own
  RowScale rs;
  double c;
  u64 warp_sum[kWarps];
  float warp_max[kWarps];
  int warp_idx[kWarps];
  u64 found;
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

// kMagic + rint(1024 log2 w), monotone in l; below kDead, or NaN, where the
// weight is zero.  (Infinite m: the infinities share the weight.)
__device__ __forceinline__ float key_of(const RowScale &rs, float l) {
  if (!rs.wide) return fmaf(l, 1024.f * rs.c_hi, rs.K);
  if (l == rs.m) return kMagic;
  return fmaf(fmaxf((l - rs.m) * rs.c_hi, -1e6f), 1024.f, kMagic) - (l != l ? __int_as_float(0x7fc00000) : 0.f);
}
__device__ __forceinline__ int bin_of(float t) { return (kMagicBits - __float_as_int(t)) >> 5; }
// 2^44 2^((l - m) c) as an integer, for t = key_of(l) >= kDead: with i + 1024 n =
// t's integer, 2^n 2^(i/1024) 2^r, |r| <= 2^-11 and a little.
__device__ __forceinline__ Weight weight_of(const RowScale &rs, const float2 *exp2, float l, float t) {
  const float ti = t - kMagic;
  float r;
  if (!rs.wide) {
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
  return x > 0.f ? __double2ull_rd((double)x * 18446744073709551616.0) : 0ull;
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
  __device__ __forceinline__ void get(int j, float (&f)[E]) const {
    const uint4 v = reinterpret_cast<const uint4 *>(data)[j];
    const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = to_f32(e[i]);
  }
  // fn(logit, key, index) for the tokens with a key of at least t_min
  template <typename F>
  __device__ __forceinline__ void each(const RowScale &rs, float t_min, F fn) const {
    for (int j = threadIdx.x; j < nv; j += kThreads) {
      float f[E], t[E], most = -1e30f;
      get(j, f);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        t[i] = key_of(rs, f[i]);
        most = fmaxf(most, t[i]);  // a NaN is passed over
      }
      if (most >= t_min) {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (t[i] >= t_min) fn(f[i], t[i], (uint32_t)(first + j * E + i));
      }
    }
  }
};

// Ascending (or descending) bitonic sort of n2 (a power of two) values in
// shared memory by the block.  Up to step 32 a warp's pairs lie in 64 places of
// its own.
template <typename V>
__device__ __forceinline__ void block_sort(V *v, int n2, bool descending) {
  __syncthreads();
  for (int size = 2; size <= n2; size <<= 1)
    for (int step = size >> 1; step > 0; step >>= 1) {
      for (int i = threadIdx.x; i < n2 / 2; i += kThreads) {
        const int x = 2 * i - (i & (step - 1)), z = x + step;
        const V p = v[x], q = v[z];
        if ((p < q) == (((x & size) == 0) == descending)) {
          v[x] = q;
          v[z] = p;
        }
      }
      if (step > 32 || (step == 1 && size > 32)) __syncthreads();
      else __syncwarp();
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
      w[i] = weight_of(rs, sh.exp2, l, key_of(rs, l)).whole();
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
      w[i] = weight_of(rs, sh.exp2, l, key_of(rs, l)).whole();
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

// The whole cluster: the last token kept of a bin that holds too many to sort,
// bit by bit: the largest order value with enough tokens (or weight) of the bin
// at or above it.  Bits 31..18 are set in every value (indices are below 2^18).
template <typename T>
__device__ u64 bisect(SampleShared &sh, const Slice<T> &slice, const RowScale &rs, uint32_t rank, int cs, int bin, int by_sum,
                      u64 need) {
  u64 t = 0xFFFC0000ull;
  int par = 0;
  for (int bit = 63; bit >= 0; --bit) {
    if (bit >= 18 && bit < 32) continue;
    const u64 cand = t | (1ull << bit);
    u64 acc = 0;
    slice.each(rs, kDead, [&](float l, float k, uint32_t idx) {
      if (bin_of(k) == bin && order_value(l, idx) >= cand) acc += by_sum ? weight_of(rs, sh.exp2, l, k).whole() : 1ull;
    });
    send_sum(sh, acc, par, rank, cs);
    cluster_sync(cs);
    u64 all = 0;
    for (int r = 0; r < cs; ++r) all += sh.part_sum[par][r];
    if (all >= need) t = cand;
    par ^= 1;
  }
  return t;
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
  auto clear_hist = [&]() {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      sh.hist.cnt[tid + i * kThreads] = 0;
#pragma unroll
      for (int x = 0; x < 3; ++x) sh.hist.sum[x][tid + i * kThreads] = 0;
    }
  };
  if (!greedy) {
#pragma unroll
    for (int i = 0; i < 1024 / kThreads; ++i) sh.exp2[tid + i * kThreads] = g_exp2.v[tid + i * kThreads];
  }
  if (has_k || has_p) clear_hist();
  if (tid == 0) {
    // small enough that its products stay finite
    sh.c = fmin(1.4426950408889634 / (double)temp, 1.2676506002282294e30);
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
    for (int j = tid; j < slice.nv; j += kThreads) {
      float f[E];
      slice.get(j, f);
#pragma unroll
      for (int i = E - 1; i >= 0; --i)
        if (f[i] == m) best = min(best, slice.first + j * E + i);
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
    RowScale rs;
    rs.m = m;
    rs.c_hi = (float)sh.c;
    rs.c_lo = (float)(sh.c - (double)rs.c_hi);
    const double mc = (double)m * (double)rs.c_hi;  // exact
    rs.wide = !(fabs(mc) < 4096.0);
    rs.K = rs.A0 = rs.a1 = 0.f;
    if (!rs.wide) {
      const double grid = rint(mc * 1024.0);
      rs.A0 = (float)(grid * (1.0 / 1024.0));
      rs.K = (float)(12582912.0 - grid);
      rs.a1 = (float)((mc - grid * (1.0 / 1024.0)) + (double)m * (double)rs.c_lo);
    }
    rs.top = weight_of(rs, sh.exp2, m, key_of(rs, m)).whole();
    const float mp = a.min_p ? a.min_p[b] : a.min_p_value;
    rs.least = mp > 0.f ? part_up(mp, rs.top) : 0;
    sh.rs = rs;
  }
  __syncthreads();
  const RowScale rs = sh.rs;

  // ---- the truncations
  if (has_k || has_p) {
    // rank 0: the cluster's histogram, kPer bins per thread, with the prefixes
    unsigned int c3[kPer];
    u64 s3[kPer], c_before = 0, s_before = 0, c_all = 0, s_all = 0;
    // counts (and weights) by bin of the tokens from order value `from` on
    auto histogram = [&](bool sums, u64 from) {
      slice.each(rs, kDead, [&](float l, float t, uint32_t idx) {
        if (from && order_value(l, idx) < from) return;
        const int i = bin_of(t);
        atomicAdd(&sh.hist.cnt[i], 1u);
        if (sums) {
          const u64 w = weight_of(rs, sh.exp2, l, t).whole();
          const uint32_t p0 = (uint32_t)w & 0x7FFFu, p1 = (uint32_t)(w >> 15) & 0x7FFFu, p2 = (uint32_t)(w >> 30);
          atomicAdd(&sh.hist.sum[0][i], p0);
          if (p1) atomicAdd(&sh.hist.sum[1][i], p1);
          if (p2) atomicAdd(&sh.hist.sum[2][i], p2);
        }
      });
      cluster_sync(cs);
      if (rank == 0) {
        u64 c = 0, s = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          c3[i] = 0;
          s3[i] = 0;
        }
#pragma unroll 4
        for (int r = 0; r < cs; ++r) {
          const auto *h = &peer(&sh, (uint32_t)r)->hist;
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const int at = kPer * tid + i;
            c3[i] += h->cnt[at];
            if (sums) s3[i] += (u64)h->sum[0][at] + ((u64)h->sum[1][at] << 15) + ((u64)h->sum[2][at] << 30);
          }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          c += c3[i];
          s += s3[i];
        }
        c_before = block_scan(sh, c, c_all);
        s_before = block_scan(sh, s, s_all);
      }
    };
    // rank 0: the bin at which the count (by_sum = 0) or the weight reaches want, to everyone
    auto locate = [&](int by_sum, u64 want) {
      if (rank == 0) {
        if (tid == 0) {
          sh.find[by_sum] = {1, 0, 0, 0, 0};
          sh.list_n = 0;
        }
        __syncthreads();
        u64 c = c_before, s = s_before;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const u64 x = by_sum ? s : c, dx = by_sum ? s3[i] : c3[i];
          if (x < want && want <= x + dx) {
            const int bin = kPer * tid + i, few = c + c3[i] <= kList;
            sh.find[by_sum] = {few ? 0 : bin, bin, few, !few && c3[i] > kList, want - x};
          }
          c += c3[i];
          s += s3[i];
        }
        __syncthreads();
        if (tid >= 1 && tid < cs) peer(&sh, (uint32_t)tid)->find[by_sum] = sh.find[by_sum];
      }
      cluster_sync(cs);
    };
    u64 thr = 0;
    // the tokens of find[which]'s bins, from thr on, to rank 0's list
    auto collect = [&](int which) {
      const int lo = sh.find[which].lo, hi = sh.find[which].hi;
      SampleShared *lead = peer(&sh, 0);
      slice.each(rs, __int_as_float(kMagicBits - (32 * hi + 31)), [&](float l, float t, uint32_t idx) {
        const u64 value = order_value(l, idx);
        if (bin_of(t) < lo || value < thr) return;
        const unsigned int at = atomicAdd(&lead->list_n, 1u);
        if (at < kList) lead->few.list[at] = value;
      });
      cluster_sync(cs);
    };
    if (has_k) {
      histogram(false, 0);
      locate(0, (u64)top_k);
      const auto f = sh.find[0];
      has_k = f.lo <= f.hi;  // a top_k beyond the tokens that have a weight keeps them all
      if (has_k && f.few) {
        collect(0);
        if (rank == 0) draw_from_list(sh, rs, top_k, top_p, 0, u, a.token + b, a.prob ? a.prob + b : nullptr);
        return;
      }
      if (has_k) {
        if (f.many) {
          thr = bisect(sh, slice, rs, rank, cs, f.hi, 0, f.need);
        } else {
          collect(0);
          if (rank == 0) {
            find_in_list(sh, rs, 0, f.need);
            if (tid < cs) peer(&sh, (uint32_t)tid)->threshold = sh.found;
          }
          cluster_sync(cs);
          thr = sh.threshold;
        }
      }
      if (has_p) {  // the histogram again, with weights
        clear_hist();
        cluster_sync(cs);
      }
    }
    if (has_p) {
      histogram(true, thr);
      u64 want = 0;
      if (rank == 0) {
        // kept: less than ceil(top_p * weight) before it; the first always is
        want = part_up(top_p, s_all);
        want = want ? want : 1;
      }
      locate(1, want);
      const auto f = sh.find[1];
      if (f.few) {
        collect(1);
        if (rank == 0) draw_from_list(sh, rs, has_k ? top_k : 0, top_p, want, u, a.token + b, a.prob ? a.prob + b : nullptr);
        return;
      }
      if (f.many) {
        thr = max(thr, bisect(sh, slice, rs, rank, cs, f.hi, 1, f.need));
      } else {
        collect(1);
        if (rank == 0) {
          find_in_list(sh, rs, 1, f.need);
          if (tid < cs) peer(&sh, (uint32_t)tid)->threshold = sh.found;
        }
        cluster_sync(cs);
        thr = max(thr, sh.threshold);
      }
    }
    if (tid == 0) sh.threshold = thr;
    __syncthreads();
  }

  // ---- the kept weight: warp w of a CTA sums a contiguous run of vectors
  const u64 thr = sh.threshold;
  const float t_min = thr ? key_of(rs, order_logit(thr)) : kDead;
  const int vw = ((slice.nv + kWarps - 1) / kWarps + 31) & ~31;
  const int v0 = warp * vw, v1 = min(slice.nv, v0 + vw);
  const bool tests = thr != 0 || rs.least != 0;
  auto kept = [&](float l, uint32_t idx) -> Weight {
    const float t = key_of(rs, l);
    if (!(t >= t_min)) return Weight{0, 0};
    const Weight w = weight_of(rs, sh.exp2, l, t);
    if (tests && (order_value(l, idx) < thr || w.whole() < rs.least)) return Weight{0, 0};
    return w;
  };
  Weight acc{0, 0};
  for (int j = v0 + lane; j < v1; j += 32) {
    float f[E];
    slice.get(j, f);
#pragma unroll
    for (int i = 0; i < E; ++i) acc.add(kept(f[i], (uint32_t)(slice.first + j * E + i)));
  }
  send_sum(sh, acc.whole(), 0, rank, cs);
  cluster_sync(cs);
  u64 total = 0, before = 0;
  for (int r = 0; r < cs; ++r) {
    if (r < (int)rank) before += sh.part_sum[0][r];
    total += sh.part_sum[0][r];
  }
  const u64 target = draw_target(u, total);
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
