// C ABI entry points of libq1 (declared in include/q1.h): host-side argument
// validation, dispatch between the narrow and wide matmul paths, and launch
// chaining.  No device memory is allocated here; scratch (the prefill path's
// fp16 activation rows, the fused FFN's intermediate) comes from the caller's
// workspace.
#include <algorithm>
#include <atomic>
#include <cstdlib>
#include <cstring>

#include "q1_internal.h"

namespace {

using q1::WeightView;

std::atomic<int> g_max_rows{[] {
  const char *e = std::getenv("Q1_QMM_MAX_ROWS");
  if (!e) return 8;
  int v = std::atoi(e);
  return v < 0 ? 0 : (v > 8 ? 8 : v);
}()};

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

q1_status cuda_status(cudaError_t e) { return e == cudaSuccess ? Q1_OK : Q1_ERR_CUDA; }

// The kernels use tcgen05 / sm_103a features: refuse other devices loudly.
q1_status check_device() {
  static thread_local int checked_dev = -1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return Q1_ERR_CUDA;
  if (dev == checked_dev) return Q1_OK;
  int major = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return Q1_ERR_CUDA;
  if (major != 10) return Q1_ERR_DEVICE;
  checked_dev = dev;
  return Q1_OK;
}

q1_status check_weight(const q1_weight *W) {
  if (!W || !W->w || !W->scales) return Q1_ERR_NULL;
  if (W->group_size != 32 && W->group_size != 64 && W->group_size != 128) return Q1_ERR_GROUP;
  if (W->meta_dtype != Q1_META_F16 && W->meta_dtype != Q1_META_BF16) return Q1_ERR_DTYPE;
  if (W->N < 1 || W->K < 128 || W->K % 128 != 0) return Q1_ERR_SHAPE;
  if (W->K > (int64_t)1 << 24 || W->N > ((int64_t)1 << 31) - 1) return Q1_ERR_SHAPE;
  if (!aligned(W->w, 16) || !aligned(W->scales, 2) || (W->biases && !aligned(W->biases, 2)))
    return Q1_ERR_ALIGN;
  return Q1_OK;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

q1_status check_ws(const void *ws, size_t have, size_t need) {
  if (need == 0) return Q1_OK;
  if (!ws) return Q1_ERR_WORKSPACE;
  if (have < need || !aligned(ws, 256)) return Q1_ERR_WORKSPACE;
  return Q1_OK;
}

q1_status matmul_common(const q1_weight *W, const void *x, int64_t M, q1_dtype dtype,
                        const void *y) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  s = check_weight(W);
  if (s != Q1_OK) return s;
  if (!x || !y) return Q1_ERR_NULL;
  if (dtype != Q1_BF16 && dtype != Q1_F16 && dtype != Q1_F32) return Q1_ERR_DTYPE;
  if (M < 1 || M > ((int64_t)1 << 24)) return Q1_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16)) return Q1_ERR_ALIGN;
  return Q1_OK;
}

}  // namespace

extern "C" {

const char *q1_status_string(q1_status s) {
  switch (s) {
    case Q1_OK: return "ok";
    case Q1_ERR_NULL: return "a required pointer is NULL";
    case Q1_ERR_SHAPE: return "invalid shape (need N>=1, K>=128, K%128==0, M in range)";
    case Q1_ERR_ALIGN: return "pointer misaligned (packed words, x, y, out: 16 bytes)";
    case Q1_ERR_DTYPE: return "unsupported dtype for this call";
    case Q1_ERR_GROUP: return "group_size must be 32, 64 or 128 (gate and up of one FFN: the same)";
    case Q1_ERR_WORKSPACE: return "workspace missing, too small or not 256-byte aligned";
    case Q1_ERR_CUDA: return "CUDA runtime error";
    case Q1_ERR_TIMEOUT: return "a bounded device-side wait ran out";
    case Q1_ERR_DEVICE: return "current device is not a compute capability 10.x (Blackwell) GPU";
  }
  return "unknown status";
}

void q1_set_qmm_max_rows(int rows) { g_max_rows.store(rows < 0 ? 0 : (rows > 8 ? 8 : rows)); }
int q1_get_qmm_max_rows(void) { return g_max_rows.load(); }
void q1_set_prefill_plan(int token_tile, int split) { q1::set_pair_plan(token_tile, split); }

q1_status q1_pack(const uint8_t *bits, int64_t N, int64_t K, uint32_t *w, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if (!bits || !w) return Q1_ERR_NULL;
  if (N < 1 || K < 32 || K % 32 != 0) return Q1_ERR_SHAPE;
  if (!aligned(bits, 16) || !aligned(w, 16)) return Q1_ERR_ALIGN;
  return cuda_status(q1::launch_pack(bits, N, K, w, (cudaStream_t)stream));
}

q1_status q1_unpack(const uint32_t *w, int64_t N, int64_t K, uint8_t *bits, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if (!bits || !w) return Q1_ERR_NULL;
  if (N < 1 || K < 32 || K % 32 != 0) return Q1_ERR_SHAPE;
  if (!aligned(bits, 16) || !aligned(w, 16)) return Q1_ERR_ALIGN;
  return cuda_status(q1::launch_unpack(w, N, K, bits, (cudaStream_t)stream));
}

q1_status q1_dequantize(const q1_weight *W, q1_dtype out_t, void *out, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  s = check_weight(W);
  if (s != Q1_OK) return s;
  if (!out) return Q1_ERR_NULL;
  if (out_t != Q1_BF16 && out_t != Q1_F16 && out_t != Q1_F32) return Q1_ERR_DTYPE;
  if (!aligned(out, 16)) return Q1_ERR_ALIGN;
  return cuda_status(q1::launch_dequantize(q1::view(W), out_t, out, (cudaStream_t)stream));
}

q1_status q1_qmv(const q1_weight *W, const void *x, q1_dtype dtype, void *y, q1_stream stream) {
  q1_status s = matmul_common(W, x, 1, dtype, y);
  if (s != Q1_OK) return s;
  if (W->K > q1::kNarrowMaxK) return Q1_ERR_SHAPE;
  return cuda_status(q1::launch_narrow(q1::view(W), x, 1, y, (cudaStream_t)stream, true, dtype, dtype));
}

q1_status q1_qmm_narrow(const q1_weight *W, const void *x, int64_t M, q1_dtype dtype, void *y,
                        q1_stream stream) {
  q1_status s = matmul_common(W, x, M, dtype, y);
  if (s != Q1_OK) return s;
  if (M > q1::kNarrowMaxM || W->K > q1::kNarrowMaxK) return Q1_ERR_SHAPE;
  return cuda_status(q1::launch_narrow(q1::view(W), x, M, y, (cudaStream_t)stream, true, dtype, dtype));
}

size_t q1_qmm_workspace_size(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || K < 128 || K % 128) return 0;
  return q1::wide_workspace_bytes(M, N, K);
}

q1_status q1_qmm(const q1_weight *W, const void *x, int64_t M, q1_dtype dtype, void *y,
                 void *workspace, size_t workspace_bytes, q1_stream stream) {
  q1_status s = matmul_common(W, x, M, dtype, y);
  if (s != Q1_OK) return s;
  const int rows = g_max_rows.load();
  if (M <= rows && W->K <= q1::kNarrowMaxK)
    return cuda_status(q1::launch_narrow(q1::view(W), x, M, y, (cudaStream_t)stream, true, dtype, dtype));
  if (rows == q1::kNarrowMaxM && M <= 2 * q1::kNarrowMaxM && W->K <= q1::kNarrowMaxK) {
    // 9..16 rows at the default threshold: two narrow launches of 8 rows and
    // M - 8 rows, the second chained with PDL (it streams its weights while
    // the first drains).  Twice the weight traffic costs less than the
    // prefill path here, whose MMAs take as long for 16 tokens as for 256.
    const size_t es = dtype == Q1_F32 ? 4 : 2;
    const int64_t m0 = q1::kNarrowMaxM;
    cudaError_t e = q1::launch_narrow(q1::view(W), x, m0, y, (cudaStream_t)stream, true, dtype, dtype);
    if (e == cudaSuccess)
      e = q1::launch_narrow(q1::view(W), static_cast<const char *>(x) + (size_t)m0 * W->K * es, M - m0,
                            static_cast<char *>(y) + (size_t)m0 * W->N * es, (cudaStream_t)stream, true, dtype,
                            dtype);
    return cuda_status(e);
  }
  s = check_ws(workspace, workspace_bytes, q1::wide_workspace_bytes(M, W->N, W->K));
  if (s != Q1_OK) return s;
  return cuda_status(q1::launch_wide(q1::view(W), x, M, y, workspace, workspace_bytes, (cudaStream_t)stream, dtype));
}

q1_status q1_embed_gather(const q1_weight *E, const int32_t *ids, int64_t T, q1_dtype out_t,
                          void *out, int32_t *d_bad_count, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  s = check_weight(E);
  if (s != Q1_OK) return s;
  if (T < 0) return Q1_ERR_SHAPE;
  if (T == 0) return Q1_OK;
  if (!ids || !out) return Q1_ERR_NULL;
  if (out_t != Q1_BF16 && out_t != Q1_F16 && out_t != Q1_F32) return Q1_ERR_DTYPE;
  if (!aligned(out, 16) || !aligned(ids, 4) || (d_bad_count && !aligned(d_bad_count, 4)))
    return Q1_ERR_ALIGN;
  return cuda_status(q1::launch_gather(q1::view(E), ids, T, out_t, out, d_bad_count,
                                       (cudaStream_t)stream));
}

size_t q1_ffn_workspace_size(int64_t M, int64_t D, int64_t F) {
  if (M < 1 || M > 8 || D < 128 || F < 128 || D % 128 || F % 128) return 0;
  return align256((size_t)(M * F * 2));  // h [M][F] bf16
}

q1_status q1_ffn_fused(const q1_weight *gate, const q1_weight *up, const q1_weight *down,
                       const void *x, int64_t M, q1_dtype dtype, void *y, void *workspace,
                       size_t workspace_bytes, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if ((s = check_weight(gate)) != Q1_OK || (s = check_weight(up)) != Q1_OK ||
      (s = check_weight(down)) != Q1_OK)
    return s;
  // gate and up run in one launch with one group size; down may differ
  if (gate->group_size != up->group_size) return Q1_ERR_GROUP;
  if (!x || !y) return Q1_ERR_NULL;
  if (dtype != Q1_BF16 && dtype != Q1_F16 && dtype != Q1_F32) return Q1_ERR_DTYPE;
  if (M < 1 || M > q1::kNarrowMaxM) return Q1_ERR_SHAPE;
  const int64_t D = gate->K, F = gate->N;
  if (up->K != D || up->N != F || down->K != F || down->N != D) return Q1_ERR_SHAPE;
  if (D > q1::kNarrowMaxK || F > q1::kNarrowMaxK) return Q1_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(y, 16)) return Q1_ERR_ALIGN;
  s = check_ws(workspace, workspace_bytes, q1_ffn_workspace_size(M, D, F));
  if (s != Q1_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  void *h = workspace;
  // two launches chained with programmatic dependent launch: the down
  // projection starts streaming its weights while gate/up drains, and waits
  // for h only before reading it
  cudaError_t e = q1::launch_narrow_gate_up(q1::view(gate), q1::view(up), x, M, h, st, true, dtype);
  if (e == cudaSuccess) e = q1::launch_narrow(q1::view(down), h, M, y, st, true, Q1_BF16, dtype);
  return cuda_status(e);
}

size_t q1_decode_chain_workspace_size(int64_t M, int64_t D, int64_t F_max) {
  if (M < 1 || M > 8 || D < 128 || F_max < 128 || D % 128 || F_max % 128) return 0;
  // a [M][D], the current h [M][D], the FFN intermediate [M][F_max], all bf16
  return 2 * align256((size_t)(M * D * 2)) + align256((size_t)(M * F_max * 2));
}

q1_status q1_decode_chain(const q1_decode_layer *layers, int32_t n_layers, const void *x,
                          int64_t M, q1_dtype dtype, void *y, void *workspace,
                          size_t workspace_bytes, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if (!layers || !x || !y) return Q1_ERR_NULL;
  if (n_layers < 1) return Q1_ERR_SHAPE;
  if (dtype != Q1_BF16) return Q1_ERR_DTYPE;
  if (M < 1 || M > q1::kNarrowMaxM) return Q1_ERR_SHAPE;
  const int64_t D = layers[0].attn.N;
  int64_t F_max = 0;
  for (int32_t l = 0; l < n_layers; ++l) {
    const q1_decode_layer &L = layers[l];
    if ((s = check_weight(&L.attn)) != Q1_OK || (s = check_weight(&L.gate)) != Q1_OK ||
        (s = check_weight(&L.up)) != Q1_OK || (s = check_weight(&L.down)) != Q1_OK)
      return s;
    if (L.gate.group_size != L.up.group_size) return Q1_ERR_GROUP;
    const int64_t F = L.gate.N;
    if (L.attn.N != D || L.attn.K != D || L.gate.K != D || L.up.K != D || L.up.N != F ||
        L.down.K != F || L.down.N != D)
      return Q1_ERR_SHAPE;
    if (D > q1::kNarrowMaxK || F > q1::kNarrowMaxK) return Q1_ERR_SHAPE;
    F_max = F > F_max ? F : F_max;
  }
  if (!aligned(x, 16) || !aligned(y, 16)) return Q1_ERR_ALIGN;
  s = check_ws(workspace, workspace_bytes, q1_decode_chain_workspace_size(M, D, F_max));
  if (s != Q1_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  char *ws = static_cast<char *>(workspace);
  void *a = ws;
  void *hb = ws + align256((size_t)(M * D * 2));
  void *fh = ws + 2 * align256((size_t)(M * D * 2));
  cudaError_t e = cudaSuccess;
  for (int32_t l = 0; l < n_layers && e == cudaSuccess; ++l) {
    const q1_decode_layer &L = layers[l];
    const void *in = l == 0 ? x : hb;
    void *out = l == n_layers - 1 ? y : hb;
    // every kernel reads its input only after its predecessor has completed
    // (griddepcontrol.wait), and each predecessor completed only after its own
    // predecessor: the down projection overwrites hb after the attention
    // product that read it is done
    e = q1::launch_narrow(q1::view(&L.attn), in, M, a, st, true);
    if (e == cudaSuccess) e = q1::launch_narrow_gate_up(q1::view(&L.gate), q1::view(&L.up), a, M, fh, st, true);
    if (e == cudaSuccess) e = q1::launch_narrow(q1::view(&L.down), fh, M, out, st, true);
  }
  return cuda_status(e);
}

q1_status q1_pack_from_dense(const void *dense, q1_dtype in_t, int64_t N, int64_t K, uint32_t *w,
                             uint16_t *scales, uint16_t *biases, int32_t *d_bad_groups,
                             q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if (!dense || !w || !scales || !d_bad_groups) return Q1_ERR_NULL;
  if (in_t != Q1_BF16 && in_t != Q1_F16 && in_t != Q1_F32) return Q1_ERR_DTYPE;
  if (N < 1 || K < 128 || K % 128 != 0 || K > (int64_t)1 << 24 || N > ((int64_t)1 << 31) - 1)
    return Q1_ERR_SHAPE;
  if (!aligned(dense, 16) || !aligned(w, 16) || !aligned(scales, 2) || (biases && !aligned(biases, 2)) ||
      !aligned(d_bad_groups, 4))
    return Q1_ERR_ALIGN;
  return cuda_status(q1::launch_pack_from_dense(dense, in_t, N, K, w, scales, biases, d_bad_groups,
                                                (cudaStream_t)stream));
}

namespace {
// types and sizes: all that the workspace's size goes by
q1_status check_delta_sizes(const q1_delta_args *a) {
  if (!a) return Q1_ERR_NULL;
  if (a->dtype != Q1_BF16 && a->dtype != Q1_F16 && a->dtype != Q1_F32) return Q1_ERR_DTYPE;
  if ((a->DK != 64 && a->DK != 128) || (a->DV != 64 && a->DV != 128)) return Q1_ERR_SHAPE;
  if (a->HK < 1 || a->HV < 1 || a->HV % a->HK != 0 || a->HV > 65535) return Q1_ERR_SHAPE;
  if (a->T < 0 || a->T > ((int64_t)1 << 31) - 1 || a->B < 1 || a->B > (int64_t)1 << 24 ||
      a->B * a->HV > (int64_t)1 << 29 || a->n_slots < 0 || a->max_len < 0)
    return Q1_ERR_SHAPE;
  return Q1_OK;
}

q1_status check_delta(const q1_delta_args *a) {
  const q1_status s = check_delta_sizes(a);
  if (s != Q1_OK) return s;
  if (!a->cu_seqlens && a->T % a->B != 0) return Q1_ERR_SHAPE;
  if (!a->slots && a->n_slots < a->B) return Q1_ERR_SHAPE;
  if (!a->state) return Q1_ERR_NULL;
  if (!aligned(a->state, 16)) return Q1_ERR_ALIGN;
  if ((a->cu_seqlens && !aligned(a->cu_seqlens, 4)) || (a->slots && !aligned(a->slots, 4)) ||
      (a->fresh && !aligned(a->fresh, 4)))
    return Q1_ERR_ALIGN;
  if (a->T == 0) return Q1_OK;  // no rows to read: the states only
  if (!a->q || !a->k || !a->v || !a->o || !a->g || !a->beta) return Q1_ERR_NULL;
  const int64_t per16 = a->dtype == Q1_F32 ? 4 : 8;  // elements in 16 bytes
  if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->o, 16) || a->q_stride % per16 ||
      a->k_stride % per16 || a->v_stride % per16 || a->o_stride % per16 || !aligned(a->g, 4) || !aligned(a->beta, 4))
    return Q1_ERR_ALIGN;
  const int64_t qk = (int64_t)a->HK * a->DK, vo = (int64_t)a->HV * a->DV;
  if (a->T > 1 && (a->q_stride < qk || a->k_stride < qk || a->v_stride < vo || a->o_stride < vo ||
                   a->g_stride < a->HV || a->beta_stride < a->HV))
    return Q1_ERR_SHAPE;
  return Q1_OK;
}

q1::DeltaView delta_view(const q1_delta_args *a) {
  return q1::DeltaView{a->q, a->k, a->v, a->o, a->g, a->beta, a->state, a->cu_seqlens, a->slots, a->fresh,
                       a->q_stride, a->k_stride, a->v_stride, a->o_stride, a->g_stride, a->beta_stride,
                       a->T, a->B, a->n_slots, a->max_len, a->HK, a->HV, a->DK, a->DV, a->qk_l2norm != 0, a->scale};
}
}  // namespace

namespace {
// Short sequences go token by token, as do fp32 activations (the chunked form's
// operands hold 16-bit inputs exactly, not fp32 ones).  A token costs the first form
// the state's size once the heads fill the GPU, the second one next to nothing up
// to 64 tokens.  Where the two meet, bf16, in us token by token / in chunks:
//   1 sequence of 32 heads     128 x 128  16.7 / 17.9 at 36, 18.4 / 18.1 at 40
//                              64 x 64    14.2 / 16.0 at 36, 15.7 / 16.0 at 40
//   8 sequences of 48 heads    128 x 128  41.5 / 43.1 at 20, 48.7 / 43.3 at 24
//                              64 x 128   33.2 / 35.1 at 24, 38.1 / 35.2 at 28
//                              128 x 64   33.8 / 36.0 at 32, 37.5 / 36.8 at 36
//                              64 x 64    27.9 / 31.6 at 40, 32.9 / 32.3 at 48
//   32 sequences of 32 heads   95 / 91 at 20, 74 / 74 at 24, 76 / 77 at 32, 61 / 66 at 40
bool delta_in_chunks(const q1_delta_args *a) {
  const int filled = a->DV == 64 ? (a->DK == 64 ? 40 : 32) : (a->DK == 64 ? 24 : 20);
  return a->max_len > (a->B * a->HV <= 152 ? 36 : filled) && a->dtype != Q1_F32 && a->T > 0;
}
}  // namespace

size_t q1_gated_delta_workspace_size(const q1_delta_args *a) {
  if (check_delta_sizes(a) != Q1_OK || !delta_in_chunks(a)) return 0;
  return q1::delta_chunk_workspace_bytes(delta_view(a));
}

q1_status q1_gated_delta(const q1_delta_args *a, void *workspace, size_t workspace_bytes, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if ((s = check_delta(a)) != Q1_OK) return s;
  const q1::DeltaView v = delta_view(a);
  if (!delta_in_chunks(a)) return cuda_status(q1::launch_delta_step(v, (q1_dtype)a->dtype, (cudaStream_t)stream));
  if ((s = check_ws(workspace, workspace_bytes, q1::delta_chunk_workspace_bytes(v))) != Q1_OK) return s;
  return cuda_status(q1::launch_delta_chunks(v, (q1_dtype)a->dtype, workspace, (cudaStream_t)stream));
}

q1_status q1_sample(const q1_sample_args *a, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if (!a) return Q1_ERR_NULL;
  if (a->dtype != Q1_BF16 && a->dtype != Q1_F16 && a->dtype != Q1_F32) return Q1_ERR_DTYPE;
  if (a->B < 0 || a->B > (int64_t)1 << 24 || a->V < 1 || a->V > (int64_t)1 << 18 || (a->B > 1 && a->row_stride < a->V))
    return Q1_ERR_SHAPE;
  if (a->B == 0) return Q1_OK;
  if (!a->logits || !a->u || !a->token) return Q1_ERR_NULL;
  if (!aligned(a->logits, a->dtype == Q1_F32 ? 4 : 2) || !aligned(a->u, 4) || !aligned(a->token, 4) ||
      !aligned(a->prob, 4) || !aligned(a->temperature, 4) || !aligned(a->top_p, 4) || !aligned(a->min_p, 4) ||
      !aligned(a->top_k, 4))
    return Q1_ERR_ALIGN;
  return cuda_status(q1::launch_sample(*a, (cudaStream_t)stream));
}

namespace {
q1_status check_kv_sizes(const q1_kv_cache *c) {
  if (!c) return Q1_ERR_NULL;
  if (c->D != 64 && c->D != 128 && c->D != 256) return Q1_ERR_SHAPE;
  if ((c->group_size != 64 && c->group_size != 128) || c->group_size > c->D) return Q1_ERR_GROUP;
  if (c->page_size < 16 || c->page_size > 65536 || (c->page_size & (c->page_size - 1))) return Q1_ERR_SHAPE;
  if (c->HK < 1 || c->HK > 65535 || c->T < 0 || c->T > ((int64_t)1 << 31) - 1 || c->B < 1 || c->B > (int64_t)1 << 24 ||
      c->n_pages < 0 || c->n_pages > ((int64_t)1 << 31) - 1 || c->table_width < 0 ||
      c->table_width > (int64_t)1 << 31 || c->table_width * c->page_size > ((int64_t)1 << 31) - 65536 || c->T * c->HK * c->D > (int64_t)1 << 40)
    return Q1_ERR_SHAPE;
  return Q1_OK;
}

q1_status check_kv(const q1_kv_cache *c) {
  const q1_status s = check_kv_sizes(c);
  if (s != Q1_OK) return s;
  if (!c->cu_seqlens && c->T % c->B != 0) return Q1_ERR_SHAPE;
  if (c->B > 1 && c->table_stride < c->table_width) return Q1_ERR_SHAPE;
  if (c->T == 0) return Q1_OK;
  if (!c->lengths || (c->n_pages > 0 && !c->data) || (c->table_width > 0 && !c->block_table)) return Q1_ERR_NULL;
  if (!aligned(c->data, 16) || !aligned(c->block_table, 4) || !aligned(c->lengths, 4) || !aligned(c->cu_seqlens, 4))
    return Q1_ERR_ALIGN;
  return Q1_OK;
}

// rows of `heads` heads of c->D elements
q1_status check_kv_rows(const q1_kv_cache *c, const void *p, int64_t stride, int64_t heads, q1_dtype t) {
  if (!p) return Q1_ERR_NULL;
  if (!aligned(p, 16) || stride % (t == Q1_F32 ? 4 : 8)) return Q1_ERR_ALIGN;
  return c->T > 1 && stride < heads * c->D ? Q1_ERR_SHAPE : Q1_OK;
}

q1_status check_kv_attention_sizes(const q1_kv_cache *c, const q1_kv_attention_args *a) {
  const q1_status s = check_kv_sizes(c);
  if (s != Q1_OK) return s;
  if (!a) return Q1_ERR_NULL;
  if (a->dtype != Q1_BF16 && a->dtype != Q1_F16 && a->dtype != Q1_F32) return Q1_ERR_DTYPE;
  if (a->HQ < 1 || a->HQ > 65535 || a->HQ % c->HK != 0 || a->max_q < 0 || a->max_len < 0 || a->window < 0 ||
      (a->window > 0 && !a->causal) || c->T * a->HQ > ((int64_t)1 << 31) - 1 || c->B * c->HK > (int64_t)1 << 24)
    return Q1_ERR_SHAPE;
  return Q1_OK;
}

q1::KvView kv_view(const q1_kv_cache *c) {
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  return q1::KvView{static_cast<unsigned char *>(c->data), c->block_table, c->lengths, c->cu_seqlens, c->n_pages,
                    c->table_width, c->table_stride, c->T, c->B, c->HK, c->D, c->group_size, shift};
}

q1::KvAttention kv_attention_view(const q1_kv_attention_args *a) {
  // no sequence is longer than lengths can say: the plans count in 32 bits
  const int64_t max_len = std::min<int64_t>(a->max_len, INT32_MAX);
  return q1::KvAttention{a->q, a->o, a->lse, a->q_stride, a->o_stride, a->max_q, max_len, a->HQ, a->causal != 0, a->window,
                         a->scale};
}
}  // namespace

q1_status q1_kv_store(const q1_kv_cache *c, const void *k, int64_t k_stride, const void *v, int64_t v_stride, q1_dtype t,
                      q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if ((s = check_kv(c)) != Q1_OK) return s;
  if (t != Q1_BF16 && t != Q1_F16 && t != Q1_F32) return Q1_ERR_DTYPE;
  if (c->T == 0) return Q1_OK;
  if ((s = check_kv_rows(c, k, k_stride, c->HK, t)) != Q1_OK) return s;
  if ((s = check_kv_rows(c, v, v_stride, c->HK, t)) != Q1_OK) return s;
  return cuda_status(q1::launch_kv_store(kv_view(c), k, k_stride, v, v_stride, t, (cudaStream_t)stream));
}

q1_status q1_kv_load(const q1_kv_cache *c, void *k, int64_t k_stride, void *v, int64_t v_stride, q1_dtype t, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if ((s = check_kv(c)) != Q1_OK) return s;
  if (t != Q1_BF16 && t != Q1_F16 && t != Q1_F32) return Q1_ERR_DTYPE;
  if (c->T == 0) return Q1_OK;
  if ((s = check_kv_rows(c, k, k_stride, c->HK, t)) != Q1_OK) return s;
  if ((s = check_kv_rows(c, v, v_stride, c->HK, t)) != Q1_OK) return s;
  return cuda_status(q1::launch_kv_load(kv_view(c), k, k_stride, v, v_stride, t, (cudaStream_t)stream));
}

size_t q1_kv_attention_workspace_size(const q1_kv_cache *c, const q1_kv_attention_args *a) {
  if (check_kv_attention_sizes(c, a) != Q1_OK || c->T == 0) return 0;
  const q1::KvView v = kv_view(c);
  const q1::KvAttention at = kv_attention_view(a);
  const int splits = q1::kv_tiles_splits(v, at, (q1_dtype)a->dtype);
  return splits ? q1::kv_tiles_workspace_bytes(v, at, splits) : q1::kv_decode_workspace_bytes(v, at, (q1_dtype)a->dtype);
}

int32_t q1_kv_attention_parts(const q1_kv_cache *c, const q1_kv_attention_args *a) {
  if (check_kv_attention_sizes(c, a) != Q1_OK) return -1;
  return c->T == 0 ? 0 : q1::kv_tiles_splits(kv_view(c), kv_attention_view(a), (q1_dtype)a->dtype);
}

q1_status q1_kv_attention(const q1_kv_cache *c, const q1_kv_attention_args *a, void *workspace, size_t workspace_bytes,
                          q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  if ((s = check_kv_attention_sizes(c, a)) != Q1_OK) return s;
  if ((s = check_kv(c)) != Q1_OK) return s;
  if (c->T == 0) return Q1_OK;
  const q1_dtype t = (q1_dtype)a->dtype;
  if ((s = check_kv_rows(c, a->q, a->q_stride, a->HQ, t)) != Q1_OK) return s;
  if ((s = check_kv_rows(c, a->o, a->o_stride, a->HQ, t)) != Q1_OK) return s;
  if (!aligned(a->lse, 4)) return Q1_ERR_ALIGN;
  const q1::KvView v = kv_view(c);
  const q1::KvAttention at = kv_attention_view(a);
  const int splits = q1::kv_tiles_splits(v, at, t);
  const size_t need = splits ? q1::kv_tiles_workspace_bytes(v, at, splits) : q1::kv_decode_workspace_bytes(v, at, t);
  if (need && (s = check_ws(workspace, workspace_bytes, need)) != Q1_OK) return s;
  if (splits) return cuda_status(q1::launch_kv_prefill(v, at, t, splits, workspace, (cudaStream_t)stream));
  return cuda_status(q1::launch_kv_decode(v, at, t, workspace, (cudaStream_t)stream));
}

q1_status q1_check_symmetric(const q1_weight *W, int32_t *d_is_symmetric, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  s = check_weight(W);
  if (s != Q1_OK) return s;
  if (!W->biases || !d_is_symmetric) return Q1_ERR_NULL;
  if (!aligned(d_is_symmetric, 4)) return Q1_ERR_ALIGN;
  return cuda_status(q1::launch_check_symmetric(q1::view(W), d_is_symmetric, (cudaStream_t)stream));
}

namespace {
std::atomic<unsigned long long> g_wait_ns{2000000000ull};
std::atomic<int> g_stall{0};
q1_status push_diagnostics() {
  const unsigned long long ns = g_wait_ns.load();
  const int stall = g_stall.load();
  cudaError_t e = q1::set_narrow_diagnostics(ns, stall);
  if (e == cudaSuccess) e = q1::set_wide_diagnostics(ns, stall);
  if (e == cudaSuccess) e = q1::set_delta_diagnostics(ns, stall);
  if (e == cudaSuccess) e = q1::set_kv_diagnostics(ns, stall);
  return cuda_status(e);
}
}  // namespace

q1_status q1_set_wait_limit_ns(uint64_t ns) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  g_wait_ns.store(ns ? (unsigned long long)ns : 2000000000ull);
  return push_diagnostics();
}

q1_status q1_set_stalled_producers(int stall) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  g_stall.store(stall ? 1 : 0);
  return push_diagnostics();
}

q1_status q1_device_errors(unsigned int *flags, q1_stream stream) {
  q1_status s = check_device();
  if (s != Q1_OK) return s;
  cudaError_t e1 = cudaSuccess, e2 = cudaSuccess, e3 = cudaSuccess, e4 = cudaSuccess;
  unsigned int v = q1::read_and_clear_wide_errors((cudaStream_t)stream, &e1);
  v |= q1::read_and_clear_narrow_errors((cudaStream_t)stream, &e2) << 1;
  v |= q1::read_and_clear_delta_errors((cudaStream_t)stream, &e3) << 2;
  v |= q1::read_and_clear_kv_errors((cudaStream_t)stream, &e4) << 3;
  if (flags) *flags = v;
  if (e1 != cudaSuccess || e2 != cudaSuccess || e3 != cudaSuccess || e4 != cudaSuccess) return Q1_ERR_CUDA;
  return v ? Q1_ERR_TIMEOUT : Q1_OK;
}

}  // extern "C"
