// Gated delta rule, token by token (the form for decode, and for any length).
//
// Per sequence and value head, with the state S [DK][DV] in fp32:
//   S~  = exp(g_t) S_{t-1}
//   d_t = beta_t (v_t - S~^T k_t)
//   S_t = S~ + k_t d_t^T,   o_t = scale S_t^T q_t
// Both reductions over DK run on the state as it was before the token:
//   S~^T k = alpha (S^T k),   S_t^T q = alpha (S^T q) + (k . q) d_t,
// so one pass over the state, and one reduction, serve a token.  The
// norms of k and q are sums over DK too and join the same reduction: the raw
// rows are used, and their scales multiply the reduced values.
#include <cuda_bf16.h>

#include "q1_internal.h"

namespace q1 {
namespace {

// A warp owns 16 columns (DV) of one head's state and keeps them in registers
// over the tokens: lane (group, quad) holds rows group*R .. group*R+R-1 of 8
// groups over DK and columns 4*quad .. 4*quad+3 (64 values at DK = 128), so the
// reductions over DK are three shuffle levels and no warp waits for another.
// The state is kept as S = Gamma St, with Gamma the product of the decays since
// it was last folded in: a token then costs one multiply-add per state value
// for the update, as for each of the two reductions.  CTAs are two warps (32
// columns), so that one sequence of 32 heads spreads over 128 SMs.
//
// Bound by the state's bytes for one token: 64 sequences of 32 heads (128 x 128)
// move 270 MB in 44.4 us, 6.1 TB/s, 90 % of a plain copy; one sequence takes 2.8
// us, the launch.  Windows of several tokens: 8 sequences of 48 heads and 8 tokens
// take 18.6 us (29 us with barriers between warps).  Of these the state's bytes are
// 7.7 us and the instructions 11 us of full issue (the multiply-adds 4 us; the rest
// are the reductions, and the norms, which every warp of a head forms again), and
// three warps per scheduler overlap little of it (0.58 issued per clock).  Few
// sequences: latency, 0.35 us a token, in which the shuffles, roots, exponential and
// division stand one behind another.
constexpr int kStepThreads = 64;
constexpr int kStepCols = 32;
constexpr int kStepGroups = 8;

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen<float>(float x) { return x; }
template <>
__device__ __forceinline__ float widen<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// N consecutive elements (N * sizeof(T) a multiple of 8 bytes, so aligned) as stored
template <typename T, int N>
struct Raw {
  static constexpr int kWords = N * (int)sizeof(T) / 8;
  uint2 w[kWords];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (kWords % 2 == 0) {
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
        w[2 * i] = make_uint2(v.x, v.y);
        w[2 * i + 1] = make_uint2(v.z, v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint2 *>(p) + i);
    }
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    const T *e = reinterpret_cast<const T *>(w);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = widen<T>(e[i]);
  }
};

template <typename T, int DK>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const DeltaView a) {
  constexpr int R = DK / kStepGroups;  // state rows per thread
  constexpr int P = R / 4;             // of them, the rows of this lane's share of the products of k and q
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane & 3, group = lane >> 2;
  const int h = blockIdx.y, b = blockIdx.x, col = blockIdx.z * kStepCols + 16 * warp + 4 * quad;
  const int hk = h / (a.HV / a.HK);
  int64_t t0, t1;
  a.range(b, t0, t1);
  const int64_t slot = a.slots ? a.slots[b] : b;
  const bool have = slot >= 0 && slot < a.n_slots;
  float *state = a.state + ((have ? slot : 0) * a.HV + h) * DK * a.DV + (int64_t)group * R * a.DV + col;
  float S[R][4];
  if (have && !(a.fresh && a.fresh[b])) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 s = *reinterpret_cast<const float4 *>(state + (int64_t)r * a.DV);
      S[r][0] = s.x, S[r][1] = s.y, S[r][2] = s.z, S[r][3] = s.w;
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) S[r][0] = S[r][1] = S[r][2] = S[r][3] = 0.f;
  }
  float gamma = 1.f;  // the state is gamma * S
  const T *qp = static_cast<const T *>(a.q) + (int64_t)hk * DK + group * R;
  const T *kp = static_cast<const T *>(a.k) + (int64_t)hk * DK + group * R;
  const T *vp = static_cast<const T *>(a.v) + (int64_t)h * a.DV + col;
  T *op = static_cast<T *>(a.o) + (int64_t)h * a.DV + col;
  Raw<T, R> qr, kr;
  Raw<T, 4> vr;
  float gr = 0.f, br = 0.f;
  auto fetch = [&](int64_t t) {
    qr.load(qp + t * a.q_stride);
    kr.load(kp + t * a.k_stride);
    vr.load(vp + t * a.v_stride);
    gr = __ldg(a.g + t * a.g_stride + h);
    br = __ldg(a.beta + t * a.beta_stride + h);
  };
  if (t0 < t1) fetch(t0);
  for (int64_t t = t0; t < t1; ++t) {
    float q[R], k[R], v[4];
    qr.get(q);
    kr.get(k);
    vr.get(v);
    const float alpha = expf(gr), beta = br;
    if (t + 1 < t1) fetch(t + 1);
    float kv[4] = {0.f, 0.f, 0.f, 0.f}, qv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        kv[c] = fmaf(k[r], S[r][c], kv[c]);
        qv[c] = fmaf(q[r], S[r][c], qv[c]);
      }
    // k.k, q.q and k.q: the four lanes of a group take a quarter of its rows each
    float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      float x = k[j], y = q[j];
#pragma unroll
      for (int c = 1; c < 4; ++c) {
        x = quad == c ? k[c * P + j] : x;
        y = quad == c ? q[c * P + j] : y;
      }
      kk = fmaf(x, x, kk);
      qq = fmaf(y, y, qq);
      kq = fmaf(x, y, kq);
    }
#pragma unroll
    for (int o = 1; o <= 16; o <<= 1) {
      kk += __shfl_xor_sync(0xffffffffu, kk, o);
      qq += __shfl_xor_sync(0xffffffffu, qq, o);
      kq += __shfl_xor_sync(0xffffffffu, kq, o);
      if (o >= 4) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          kv[c] += __shfl_xor_sync(0xffffffffu, kv[c], o);
          qv[c] += __shfl_xor_sync(0xffffffffu, qv[c], o);
        }
      }
    }
    const float rk = a.l2norm ? rsqrtf(kk + kDeltaEps) : 1.f;
    const float rq = a.l2norm ? rsqrtf(qq + kDeltaEps) : 1.f;
    // S~^T k and S~^T q carry the decay of this token too
    float next = gamma * alpha;
    float d[4], out[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      d[c] = beta * (v[c] - next * (rk * kv[c]));
      out[c] = a.scale * rq * fmaf(next, qv[c], rk * kq * d[c]);
    }
    // fold Gamma in before its reciprocal, or what it multiplies, can leave fp32
    if (!(next >= 9.5367431640625e-7f && next <= 1048576.f)) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) S[r][c] *= next;
      next = 1.f;
    }
    const float w = rk / next;
#pragma unroll
    for (int c = 0; c < 4; ++c) d[c] *= w;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[r][c] = fmaf(k[r], d[c], S[r][c]);
    gamma = next;
    if (group == 0) {
      T *dst = op + t * a.o_stride;
      Raw<T, 4> o4;
      T *e = reinterpret_cast<T *>(o4.w);
#pragma unroll
      for (int c = 0; c < 4; ++c) e[c] = narrow<T>(out[c]);
#pragma unroll
      for (int i = 0; i < Raw<T, 4>::kWords; ++i) reinterpret_cast<uint2 *>(dst)[i] = o4.w[i];
    }
  }
  if (have) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      *reinterpret_cast<float4 *>(state + (int64_t)r * a.DV) =
          make_float4(gamma * S[r][0], gamma * S[r][1], gamma * S[r][2], gamma * S[r][3]);
  }
}

template <typename T>
cudaError_t step_t(const DeltaView &a, cudaStream_t st) {
  const dim3 grid((unsigned)a.B, (unsigned)a.HV, (unsigned)(a.DV / kStepCols));
  if (a.DK == 128) delta_step_kernel<T, 128><<<grid, kStepThreads, 0, st>>>(a);
  else delta_step_kernel<T, 64><<<grid, kStepThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_step(const DeltaView &a, q1_dtype t, cudaStream_t st) {
  if (t == Q1_BF16) return step_t<__nv_bfloat16>(a, st);
  if (t == Q1_F16) return step_t<__half>(a, st);
  return step_t<float>(a, st);
}

}  // namespace q1
