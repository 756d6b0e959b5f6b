// Sampling: one token per row of logits from a given uniform number, with
// temperature, top-k, top-p and min-p.
//
// A cluster of 8 CTAs takes one row.  Each CTA reads its slice of the row
// once, into shared memory; everything after that (maximum, weights, the
// truncations' thresholds, the draw) runs on chip, and the CTAs exchange a few
// words through distributed shared memory.
//
// Exactness.  The token is the answer to comparisons between sums over up to
// V weights, and with tens of thousands of small weights an fp32 sum is off by
// more than one of them.  The weights are therefore fixed-point integers,
// w = 2^44 exp((l - max) / temperature), relative error about 2^-34: integer
// sums are exact and the same in any order (so shared-memory atomics and any
// split over threads give one answer).  The tokens are ordered by the 64-bit
// value (order-preserving bits of l, ~index), so "before" is one compare and
// ties fall to the lowest index.
#include <cuda_bf16.h>

#include "q1_internal.h"

namespace q1 {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kBins = 2 * kThreads;  // histogram over log2(weight), two bins per thread when scanned
constexpr int kList = 2048;          // a bin of at most this many tokens is sorted; a fuller one is bisected
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
  u64 sum[kBins];
  u64 list[kList];
  unsigned int cnt[kBins];
  // written by the CTAs of the cluster (index: their rank)
  u64 part_sum[2][kCluster];
  float part_max[kCluster];
  int part_idx[kCluster];
  // written by rank 0 into every CTA; [0] for top-k, [1] for top-p (a slot of
  // its own each: a CTA may read the first after rank 0 has begun the second)
  struct Find {
    u64 need;             // the count (top-k) or weight (top-p) wanted from the bin
    int bin;              // the bin to resolve, -1: none
    unsigned int in_bin;  // tokens in it
  } find[2];
  u64 threshold;          // tokens with a smaller order value are not kept
  // this CTA's own
  unsigned int list_n;
  u64 warp_sum[kWarps], warp_cnt[kWarps];
  float warp_max[kWarps];
  int warp_idx[kWarps];
  u64 found, found_sum;
  float c_hi, c_lo;     // log2(e) / temperature
  u64 w_min;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t rank_in_cluster() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The generic address of p's counterpart in CTA `rank` of the cluster.
template <typename P>
__device__ __forceinline__ P *peer(P *p, uint32_t rank) {
  u64 out;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(out) : "l"((u64)p), "r"(rank));
  return reinterpret_cast<P *>(out);
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
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

struct RowScale {
  float m, c_hi, c_lo;
  const float2 *exp2;
  // log2 of the weight, rounded (monotone in l); NaN for a NaN logit
  __device__ __forceinline__ float log2w(float l) const {
    if (m == __int_as_float(0x7f800000)) return l == m ? 0.f : -2.f * kRange;
    return (l - m) * c_hi;
  }
  __device__ __forceinline__ int bin(float y) const { return min(kBins - 1, (int)(-y * ((float)kBins / kRange))); }
  // 2^44 exp((l - m) / temperature) as an integer; y = log2w(l)
  __device__ __forceinline__ u64 weight(float l, float y) const {
    if (!(y > -kRange)) return 0;
    float lo = 0.f;
    if (l != m) {
      // l - m = s + e exactly (two-sum), times c_hi + c_lo
      const float s = l - m, bb = s - l;
      const float e = (l - (s - bb)) - (m + bb);
      lo = fmaf(s, c_hi, -y) + fmaf(s, c_lo, e * c_hi);
    }
    const float t = rintf(y * 1024.f);
    const float r = fmaf(t, -1.f / 1024.f, y) + lo;  // |r| <= 2^-11; the difference is exact
    const float p = r * 0.693147180559945f;
    const float x = fmaf(p * p, fmaf(p, 1.f / 6.f, 0.5f), p);  // e^p - 1
    const int ti = (int)t, i = ti & 1023, n = ti >> 10;      // n <= 0
    const float2 h = exp2[i];
    // 2^(i/1024) e^p with 40 fractional bits: hi's 24-bit significand plus a small correction
    const long long mant = (long long)((__float_as_uint(h.x) & 0x7FFFFFu) | 0x800000u) << 17;
    const long long v = mant + (long long)__float2int_rn(fmaf(h.x, x, h.y) * 1099511627776.f);
    const int sh = n + (kFrac - 40);
    if (sh >= 0) return (u64)v << sh;
    return ((u64)v + (1ull << (-sh - 1))) >> -sh;
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
// exclusive prefix sums of (c, s) over the block's threads, and the totals
__device__ __forceinline__ void block_scan(SampleShared &sh, u64 &c, u64 &s, u64 &c_all, u64 &s_all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const u64 ci = warp_scan(c, lane), si = warp_scan(s, lane);
  __syncthreads();
  if (lane == 31) {
    sh.warp_cnt[warp] = ci;
    sh.warp_sum[warp] = si;
  }
  __syncthreads();
  u64 cb = 0, sb = 0;
  c_all = s_all = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) {
      cb += sh.warp_cnt[w];
      sb += sh.warp_sum[w];
    }
    c_all += sh.warp_cnt[w];
    s_all += sh.warp_sum[w];
  }
  c = cb + ci - c;
  s = sb + si - s;
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

// The last token kept in the bin sh.find[by_sum].bin, found by the whole
// cluster: with the bin's tokens in order, the need-th one (by_sum = 0), or the
// first at which the weights of the bin reach need (by_sum = 1).  In rank 0, sh.found is its order
// value and sh.found_sum the weight of the bin's tokens up to it.
template <typename T>
__device__ void resolve_bin(SampleShared &sh, const Slice<T> &slice, const RowScale &rs, uint32_t rank,
                            int by_sum) {
  const int tid = threadIdx.x;
  const int bin = sh.find[by_sum].bin;
  const u64 need = sh.find[by_sum].need;
  if (sh.find[by_sum].in_bin <= kList) {
    SampleShared *lead = peer(&sh, 0);
    slice.each([&](float l, uint32_t idx) {
      const float y = rs.log2w(l);
      if (y > -kRange && rs.bin(y) == bin && rs.weight(l, y) != 0) {
        const unsigned int at = atomicAdd(&lead->list_n, 1u);
        if (at < kList) lead->list[at] = order_value(l, idx);
      }
    });
    cluster_sync();
    if (rank == 0) {
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
          __syncthreads();
        }
      constexpr int P = kList / kThreads;
      u64 w[P], c = 0, s = 0, ca, sa;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int at = tid * P + i;
        w[i] = 0;
        if (at < n) {
          const float l = order_logit(sh.list[at]);
          w[i] = rs.weight(l, rs.log2w(l));
        }
        s += w[i];
      }
      block_scan(sh, c, s, ca, sa);
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
    return;
  }
  // Bit by bit, the largest order value with enough tokens (or weight) at or
  // above it.  Bits 31..18 are set in every value (indices are below 2^18).
  u64 t = 0xFFFC0000ull;
  int par = 0;
  for (int bit = 63; bit >= 0; --bit) {
    if (bit >= 18 && bit < 32) continue;
    const u64 cand = t | (1ull << bit);
    u64 acc = 0;
    slice.each([&](float l, uint32_t idx) {
      const float y = rs.log2w(l);
      if (y > -kRange && rs.bin(y) == bin && order_value(l, idx) >= cand) {
        const u64 w = rs.weight(l, y);
        acc += by_sum ? w : (u64)(w != 0);
      }
    });
    acc = warp_sum(acc);
    if ((tid & 31) == 0) sh.warp_sum[tid >> 5] = acc;
    __syncthreads();
    if (tid < kCluster) {
      u64 v = 0;
      for (int w = 0; w < kWarps; ++w) v += sh.warp_sum[w];
      *peer(&sh.part_sum[par][rank], (uint32_t)tid) = v;
    }
    cluster_sync();
    u64 all = 0;
    for (int r = 0; r < kCluster; ++r) all += sh.part_sum[par][r];
    if (all >= need) t = cand;
    par ^= 1;
  }
  // the weight at or above t
  u64 acc = 0;
  slice.each([&](float l, uint32_t idx) {
    const float y = rs.log2w(l);
    if (y > -kRange && rs.bin(y) == bin && order_value(l, idx) >= t) acc += rs.weight(l, y);
  });
  acc = warp_sum(acc);
  if ((tid & 31) == 0) sh.warp_sum[tid >> 5] = acc;
  __syncthreads();
  if (tid == 0) {
    u64 v = 0;
    for (int w = 0; w < kWarps; ++w) v += sh.warp_sum[w];
    *peer(&sh.part_sum[par][rank], 0) = v;
  }
  cluster_sync();
  if (rank == 0 && tid == 0) {
    u64 v = 0;
    for (int r = 0; r < kCluster; ++r) v += sh.part_sum[par][r];
    sh.found = t;
    sh.found_sum = v;
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const q1_sample_args a, int per) {
  extern __shared__ __align__(16) unsigned char dyn[];
  SampleShared &sh = *reinterpret_cast<SampleShared *>(dyn);
  T *data = reinterpret_cast<T *>(dyn + sizeof(SampleShared));
  constexpr int E = Slice<T>::E;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = rank_in_cluster();
  const int64_t b = blockIdx.x / kCluster;
  cluster_arrive();  // peers' shared memory may be written once all have arrived
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
  for (int i = tid; i < 1024; i += kThreads) sh.exp2[i] = g_exp2.v[i];
  for (int i = tid; i < kBins; i += kThreads) {
    sh.sum[i] = 0;
    sh.cnt[i] = 0;
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
  cluster_wait();
  if (tid < kCluster) {
    float m = sh.warp_max[0];
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sh.warp_max[w]);
    *peer(&sh.part_max[rank], (uint32_t)tid) = m;
  }
  cluster_sync();
  float m = sh.part_max[0];
#pragma unroll
  for (int r = 1; r < kCluster; ++r) m = fmaxf(m, sh.part_max[r]);
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
    cluster_sync();
    if (rank == 0 && tid == 0) {
      for (int r = 0; r < kCluster; ++r) best = min(best, sh.part_idx[r]);
      a.token[b] = best;
      if (a.prob) a.prob[b] = 1.f;
    }
    return;
  }
  const RowScale rs{m, sh.c_hi, sh.c_lo, sh.exp2};

  // ---- the truncations' threshold: a histogram over log2(weight) finds the bin
  // in which top-k ends, and then the bin in which top-p ends
  if (has_k || has_p) {
    slice.each([&](float l, uint32_t) {
      const float y = rs.log2w(l);
      const u64 w = rs.weight(l, y);
      if (w) {
        const int i = rs.bin(y);
        atomicAdd(&sh.cnt[i], 1u);
        atomicAdd(&sh.sum[i], w);
      }
    });
    cluster_sync();
    u64 c2[2] = {0, 0}, s2[2] = {0, 0}, c_before = 0, s_before = 0, c_all = 0, s_all = 0;
    if (rank == 0) {  // the cluster's histogram: two bins per thread
      for (int r = 0; r < kCluster; ++r) {
        const uint2 c = *reinterpret_cast<const uint2 *>(peer(&sh.cnt[2 * tid], (uint32_t)r));
        const ulonglong2 s = *reinterpret_cast<const ulonglong2 *>(peer(&sh.sum[2 * tid], (uint32_t)r));
        c2[0] += c.x, c2[1] += c.y;
        s2[0] += s.x, s2[1] += s.y;
      }
      c_before = c2[0] + c2[1];
      s_before = s2[0] + s2[1];
      block_scan(sh, c_before, s_before, c_all, s_all);
    }
    u64 total = s_all, thr = 0;  // rank 0: the weight that top-k leaves
    for (int stage = has_k ? 0 : 1; stage < (has_p ? 2 : 1); ++stage) {
      if (rank == 0) {
        if (tid == 0) {
          sh.find[stage].bin = -1;
          sh.list_n = 0;
        }
        u64 want = (u64)top_k;
        if (stage == 1) {
          // kept: less than ceil(top_p * total) before it; the first always is
          const u64 p = fraction(top_p);
          want = __umul64hi(p, total) + (p * total != 0 ? 1 : 0);
          want = want ? want : 1;
        }
        __syncthreads();
        u64 c = c_before, s = s_before;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const u64 x = stage ? s : c, dx = stage ? s2[i] : c2[i];
          if (x < want && want <= x + dx) {
            sh.find[stage] = {want - x, 2 * tid + i, (unsigned int)c2[i]};
            sh.found_sum = s;  // the weight before the bin
          }
          c += c2[i];
          s += s2[i];
        }
        __syncthreads();
        if (tid >= 1 && tid < kCluster) peer(&sh, (uint32_t)tid)->find[stage] = sh.find[stage];
      }
      cluster_sync();
      if (sh.find[stage].bin >= 0) {
        const u64 before = sh.found_sum;
        __syncthreads();
        resolve_bin(sh, slice, rs, rank, stage);
        if (rank == 0) {
          total = before + sh.found_sum;
          thr = thr > sh.found ? thr : sh.found;
        }
      }
      __syncthreads();
    }
    if (rank == 0 && tid < kCluster) peer(&sh, (uint32_t)tid)->threshold = thr;
    cluster_sync();
  }

  // ---- the kept weight: warp w of a CTA sums a contiguous run of vectors
  const u64 thr = sh.threshold, w_min = sh.w_min;
  const int vw = ((slice.nv + kWarps - 1) / kWarps + 31) & ~31;
  const int v0 = warp * vw, v1 = min(slice.nv, v0 + vw);
  auto kept = [&](float l, uint32_t idx) -> u64 {
    const float y = rs.log2w(l);
    if (!(y > -kRange) || (thr && order_value(l, idx) < thr)) return 0;
    const u64 w = rs.weight(l, y);
    return w >= w_min ? w : 0;
  };
  u64 acc = 0;
  for (int j = v0 + lane; j < v1; j += 32) {
    float f[E];
    slice.get(j, f);
#pragma unroll
    for (int i = 0; i < E; ++i) acc += kept(f[i], (uint32_t)(slice.first + j * E + i));
  }
  acc = warp_sum(acc);
  if (lane == 0) sh.warp_sum[warp] = acc;
  __syncthreads();
  if (tid < kCluster) {
    u64 v = 0;
    for (int w = 0; w < kWarps; ++w) v += sh.warp_sum[w];
    *peer(&sh.part_sum[0][rank], (uint32_t)tid) = v;
  }
  cluster_sync();
  u64 total = 0, before = 0;
  for (int r = 0; r < kCluster; ++r) {
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
      w[i] = j < v1 ? kept(f[i], (uint32_t)(slice.first + j * E + i)) : 0;
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
  const int per = (int)((a.V + kCluster - 1) / kCluster + 7) & ~7;
  const size_t smem = sizeof(SampleShared) + ((size_t)per + 2 * E) * sizeof(T);
  if (not_done(ready, dev)) {
    const size_t most = sizeof(SampleShared) + ((size_t)(1 << 18) / kCluster + 2 * E) * sizeof(T);
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    mark_done(ready, dev);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(a.B * kCluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kCluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, per);
}

}  // namespace

cudaError_t launch_sample(const q1_sample_args &a, cudaStream_t st) {
  if (a.dtype == Q1_BF16) return sample_t<__nv_bfloat16>(a, st);
  if (a.dtype == Q1_F16) return sample_t<__half>(a, st);
  return sample_t<float>(a, st);
}

}  // namespace q1
