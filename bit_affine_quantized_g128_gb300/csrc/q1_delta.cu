// Gated delta rule, token by token (the form for decode, and for any length).
//
// Per sequence and value head, with the state S [DK][DV] in fp32:
//   S~  = exp(g_t) S_{t-1}
//   d_t = beta_t (v_t - S~^T k_t)
//   S_t = S~ + k_t d_t^T,   o_t = scale S_t^T q_t
// Both reductions over DK run on the state as it was before the token:
//   S~^T k = alpha (S^T k),   S_t^T q = alpha (S^T q) + (k . q) d_t,
// so one pass over the state, and one block reduction, serve a token.  The
// norms of k and q are sums over DK too and join the same reduction: the raw
// rows are used, and their scales multiply the reduced values.
#include <cuda_bf16.h>

#include "q1_internal.h"

namespace q1 {
namespace {

// One CTA: 32 columns (DV) of one head's state.  Thread (group, quad): rows
// group*R .. group*R+R-1 of the state (16 groups over DK), columns
// 4*quad .. 4*quad+3, held in registers over the tokens.  A warp's load of the
// state covers 4 rows x 128 bytes.  The slice of 32 columns gives 4 CTAs per
// 128-wide head, so that one sequence of 32 heads spreads over 128 SMs.
constexpr int kStepThreads = 128;
constexpr int kStepCols = 32;
constexpr int kStepGroups = kStepThreads / (kStepCols / 4);  // 16

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

struct StepShared {
  float kv[2][kStepThreads / 32][kStepCols];
  float qv[2][kStepThreads / 32][kStepCols];
  float dot[2][kStepThreads / 32][4];  // k.k, q.q, k.q
};

template <typename T, int DK>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const DeltaView a) {
  constexpr int R = DK / kStepGroups;  // state rows per thread
  __shared__ StepShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = lane & 7, group = warp * 4 + (lane >> 3);
  const int h = blockIdx.y, b = blockIdx.x, col = blockIdx.z * kStepCols + 4 * quad;
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
    const int par = (int)(t - t0) & 1;  // two reduction buffers: one barrier per token
    float q[R], k[R], v[4];
    qr.get(q);
    kr.get(k);
    vr.get(v);
    const float alpha = expf(gr), beta = br;
    if (t + 1 < t1) fetch(t + 1);
    float kv[4] = {0.f, 0.f, 0.f, 0.f}, qv[4] = {0.f, 0.f, 0.f, 0.f}, kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        kv[c] = fmaf(k[r], S[r][c], kv[c]);
        qv[c] = fmaf(q[r], S[r][c], qv[c]);
      }
      kk = fmaf(k[r], k[r], kk);
      qq = fmaf(q[r], q[r], qq);
      kq = fmaf(k[r], q[r], kq);
    }
#pragma unroll
    for (int o = 8; o <= 16; o <<= 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        kv[c] += __shfl_xor_sync(0xffffffffu, kv[c], o);
        qv[c] += __shfl_xor_sync(0xffffffffu, qv[c], o);
      }
      kk += __shfl_xor_sync(0xffffffffu, kk, o);
      qq += __shfl_xor_sync(0xffffffffu, qq, o);
      kq += __shfl_xor_sync(0xffffffffu, kq, o);
    }
    if (lane < 8) {
      *reinterpret_cast<float4 *>(&sh.kv[par][warp][4 * quad]) = make_float4(kv[0], kv[1], kv[2], kv[3]);
      *reinterpret_cast<float4 *>(&sh.qv[par][warp][4 * quad]) = make_float4(qv[0], qv[1], qv[2], qv[3]);
      if (lane == 0) *reinterpret_cast<float4 *>(&sh.dot[par][warp][0]) = make_float4(kk, qq, kq, 0.f);
    }
    __syncthreads();
    kk = qq = kq = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) kv[c] = qv[c] = 0.f;
#pragma unroll
    for (int w = 0; w < kStepThreads / 32; ++w) {
      const float4 x = *reinterpret_cast<const float4 *>(&sh.kv[par][w][4 * quad]);
      const float4 y = *reinterpret_cast<const float4 *>(&sh.qv[par][w][4 * quad]);
      const float4 z = *reinterpret_cast<const float4 *>(&sh.dot[par][w][0]);
      kv[0] += x.x, kv[1] += x.y, kv[2] += x.z, kv[3] += x.w;
      qv[0] += y.x, qv[1] += y.y, qv[2] += y.z, qv[3] += y.w;
      kk += z.x, qq += z.y, kq += z.z;
    }
    const float rk = a.l2norm ? 1.f / sqrtf(kk + kDeltaEps) : 1.f;
    const float rq = a.l2norm ? 1.f / sqrtf(qq + kDeltaEps) : 1.f;
    float d[4], out[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      d[c] = beta * (v[c] - alpha * (rk * kv[c]));
      out[c] = a.scale * rq * fmaf(alpha, qv[c], rk * kq * d[c]);
      d[c] *= rk;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) S[r][c] = fmaf(alpha, S[r][c], k[r] * d[c]);
    if (group == 0) {
      T *dst = op + t * a.o_stride;
      Raw<T, 4> w;
      T *e = reinterpret_cast<T *>(w.w);
#pragma unroll
      for (int c = 0; c < 4; ++c) e[c] = narrow<T>(out[c]);
#pragma unroll
      for (int i = 0; i < Raw<T, 4>::kWords; ++i) reinterpret_cast<uint2 *>(dst)[i] = w.w[i];
    }
  }
  if (have) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      *reinterpret_cast<float4 *>(state + (int64_t)r * a.DV) = make_float4(S[r][0], S[r][1], S[r][2], S[r][3]);
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
