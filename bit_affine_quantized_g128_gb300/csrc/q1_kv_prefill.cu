// Attention over the 4-bit cache for many query rows (prompts and pieces of
// prompts), on the tcgen05 tensor cores.
//
// A pair of CTAs owns 512 rows (two tiles of 128 each; one for heads of 256) of a key head: row i of
// a sequence is its new token i / r, query head i mod r of the r that share the key
// head.  Each expands half of K's tokens and half of V's channels, and the MMAs (cta_group::2) read both halves: with a
// CTA on its own, the MMAs' operands and the expansions' stores took all of shared memory's bandwidth (a prompt of 8192 tokens
// 561 us, 550 by pairs; heads of 64, whose operands are half as large, stay with one CTA).  Where tiles are few, their context is
// split over CTAs, whose fp32 parts a second kernel joins.  Tiles of 64 cached tokens (128 for heads of 64) go by:
//   S = Q K^T                      both operands in shared memory, S in tensor memory
//   P = 2^(f S - M + 7) as fp16    a thread per row, back into S's columns
//   O += P V                       P from tensor memory, O stays in tensor memory
//
// Roles, in groups of four warps: the softmax of a row tile each; K's expansion; V's; the
// MMAs (a thread per row tile).  Five roles share each scheduler and its instruction cache, so their loops
// are kept short (a few KB each): with the same loops unrolled twice as far the kernel took
// 1.5 times as long, though it issued fewer instructions.
//
// What bounds it.  8192 tokens, 32 heads over 8 of 128 channels: 486 us, 1130 TFLOP/s, 60 % of the measured bf16 peak; 1000 rows
// over 15000 tokens, 24 heads over 4 of 256, fp16: 376 us, 53 %.  A tile of 64 tokens takes a CTA 1800 clocks for 1266 of MMAs (an MMA
// of 256 x 64 x 16 takes 43 clocks with both operands in shared memory, 32 with Q in tensor memory; of 256 x 128 x 16 64): the two row
// tiles' softmax warps on a scheduler go through a tile in step, 600 clocks per 32 columns, and wait 450 for barriers and tensor
// memory.  Neither the other roles' traffic nor the fences slow the MMAs (633 clocks per row tile and 64 tokens beside all of it).
//
// Exactness.  K enters as scale q, which fp16 holds exactly (8 bits of scale, 4 of
// code), and the biases through one more k16 step: columns bias_g (twice per
// group) of K against the high and low fp16 half of the sum of Q's channels in group g.
// So S is exact up to fp32 sums, as far as fp16 reaches: K and V are multiplied with a power of
// two that brings the largest scale or bias that a tile's rows see to 2^-2 or more, so that
// scales and biases are exact down to 2^-15 of the largest and off by at most 2^-23 of it below.  It is a fixed one, and a tile
// that it turns out not to suit is done once more with one that does (a prompt of 8192 tokens 486 us, 481 without the
// search for the largest, 925 done twice).  Q is fp16, scaled by a power of two per row so that its
// largest value lies in [2^7, 2^8): bf16 and fp16 inputs are exact down to 2^-22 of
// that.  A 17th column of K is -inf where a token's page is missing, against 1 in Q.
// V is scale q + bias rounded to fp16 (2^-11) for bf16 outputs; for fp16 ones, whose own rounding is as small, scale q and bias are
// two operands, exact like K's, and O has two products (1000 rows over 15000 tokens 376 us and 2.9e-4 off, 354 and
// 3.2e-4 with one; their output's rounding is 2.1e-4).  P is rounded to fp16 (2^-11): its low part in a third product took 461 us, for
// 2.2e-4.  The sum of P is fp32 of the unrounded values.  M is a reference that moves when a tile's P would
// overflow fp16; 2^7 keeps all of P that matters among fp16's normal values.
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
constexpr float kShift = 7.f;      // P is 2^kShift times the softmax's numerator
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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
// the same without letting the thread sleep for a while where the phase is not complete
__device__ __forceinline__ bool mbar_test(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// A CTA's rows: those of `tile` of sequence b, and the positions that any of them sees, or a part of these.
struct Rows {
  int64_t t0;
  int rows, len, pos0, first, tiles;  // rows of the sequence, its tokens, position of its first row; first position, number of tiles
  int begin, end;                     // what any of the CTA's rows sees
  template <int ROWS, int BN>
  __device__ __forceinline__ bool set(const KvView &c, const KvAttention &a, int64_t b, int tile, int split, int splits) {
    int64_t t1;
    c.range(b, t0, t1);
    const int r = a.HQ / c.HK, n = (int)(t1 - t0);
    const int64_t all = (int64_t)n * r;
    if ((int64_t)tile * ROWS >= all) return false;
    rows = (int)all;
    len = max(c.lengths[b], 0);
    pos0 = len - n;
    const int row0 = tile * ROWS, row1 = min(row0 + ROWS, rows) - 1;
    end = a.causal ? pos0 + row1 / r + 1 : (pos0 + row1 / r < 0 ? 0 : len);
    end = (int)min((int64_t)end, c.table_width << c.page_shift);
    begin = a.window ? (int)max((int64_t)pos0 + row0 / r - a.window + 1, (int64_t)0) : 0;
    first = begin / BN * BN;
    tiles = end > begin ? (end - first + BN - 1) / BN : 0;
    const int64_t all_tiles = tiles;
    const int from = (int)(all_tiles * split / splits);
    first += from * BN;
    tiles = (int)(all_tiles * (split + 1) / splits) - from;
    return true;
  }
  __device__ __forceinline__ void put(const Rows &x) volatile {
    t0 = x.t0, rows = x.rows, len = x.len, pos0 = x.pos0, first = x.first, tiles = x.tiles, begin = x.begin, end = x.end;
  }
  __device__ __forceinline__ Rows get() const volatile { return {t0, rows, len, pos0, first, tiles, begin, end}; }
};

struct Bars {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[4], p_ready[4], o_done[2], q_full, drain;
  uint32_t tmem_base;
  volatile Rows rows;              // here, as no role has registers to keep all of it
  volatile int tile;
  volatile int abort_flag, bad_v;  // a wait ran out; V has a NaN or an infinity
  // K and V are multiplied with 2^up_k and 2^up_v; the largest scale or bias of those that rows of the pair see (bits of an fp32);
  // whether this is the second time that the CTA does its tile
  volatile int up_k, up_v, second;
  uint32_t top_k, top_v;
};
// Before scales, biases and values are rounded to fp16 their sizes are brought into its range, by a power of two that O and the
// logits' factor give back.  It starts at 2^kUpK and 2^kUpV, which suits a largest scale or bias in [2^-6, 2^8) for K and [2^-9,
// 2^5) for V; where a CTA finds another one it does its tile a second time, with that one brought into [2^11, 2^12) (9 times that,
// the largest value, is below fp16's).
constexpr int kUpK = 4, kUpV = 7, kLowK = -2, kLowV = -2, kHigh = 12;
__device__ __forceinline__ int octave(uint32_t bits) { return (int)(bits >> 23) - 127; }
__device__ __forceinline__ bool unsuited(uint32_t top, int up, int low) {
  return top != 0 && (octave(top) + up < low || octave(top) + up >= kHigh);
}
__device__ __forceinline__ bool once_more(const Bars *bars) {
  return !bars->second && (unsuited(bars->top_k, bars->up_k, kLowK) || unsuited(bars->top_v, bars->up_v, kLowV));
}

// Whether a wait gives up: its limit has run out, or another role has given up.  The clock is read on every 64th try only (a
// read takes hundreds of cycles), the first time to start it.
__device__ __noinline__ bool give_up(Bars *bars, unsigned long long since, unsigned long long now) {
  if (bars->abort_flag) return true;
  if (now - since <= c_kv_wait_ns) return false;
  bars->abort_flag = 1;
  atomicOr(&g_kv_err, 1u);
  return true;
}
// Bounded wait of a whole warp; one verdict for all its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *b, uint32_t parity, Bars *bars) {
  bool ok = mbar_try(b, parity);
  unsigned long long since = 0;
  for (uint32_t i = 1; !__all_sync(0xffffffffu, ok); ++i) {
    ok = ok || mbar_try(b, parity);
    if ((i & 63u) == 0) {
      const unsigned long long now = global_ns();
      if (i == 64) since = now;
      if (__any_sync(0xffffffffu, give_up(bars, since, now))) return false;
    }
  }
  return true;
}
// the same for one thread
__device__ __forceinline__ bool wait_one(uint64_t *b, uint32_t parity, Bars *bars) {
  unsigned long long since = 0;
  for (uint32_t i = 1; !mbar_try(b, parity); ++i)
    if ((i & 63u) == 0) {
      const unsigned long long now = global_ns();
      if (i == 64) since = now;
      if (give_up(bars, since, now)) return false;
    }
  return true;
}
// Operands of 128-byte rows, the 16-byte pieces of row r exchanged by XOR with r mod 8,
// 8-row groups 1024 bytes apart: the low word of a descriptor, with rows along M or N and the contraction
// along the row, or with rows along the contraction and 64-column boxes `box` bytes apart
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return ((saddr >> 4) & 0x3FFFu) | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t box) { return ((saddr >> 4) & 0x3FFFu) | (box >> 4) << 16; }
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;  // stride of the 8-row groups, version, 128-byte swizzle
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
template <int CG>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %5, 0;\n mov.b64 a, {%1, %4};\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::%6.kind::f16 [%0], a, b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(kDescHigh), "r"((uint32_t)acc), "n"(CG)
      : "memory");
}
template <int CG>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %5, 0;\n mov.b64 b, {%2, %4};\n"
      " tcgen05.mma.cta_group::%6.kind::f16 [%0], [%1], b, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(kDescHigh), "r"((uint32_t)acc), "n"(CG)
      : "memory");
}
// arrives on the barrier (of both CTAs of a pair) once every MMA issued so far by this thread has completed
template <int CG>
__device__ __forceinline__ void umma_commit(uint64_t *bar) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}
__device__ __forceinline__ uint32_t of_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Arrives on the barrier of the CTA that issues the MMAs (rank 0).  The default semantics (release at CTA scope) do: what
// the arrival publishes is complete before it, tensor-memory stores by tcgen05.wait::st, shared-memory stores by the proxy
// fence.  A release at cluster scope would wait for the loads in flight as well.
template <int CG>
__device__ __forceinline__ void arrive_lead(uint64_t *bar, int rank) {
  if (CG == 1 || rank == 0) mbar_arrive(bar);
  else asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(of_rank(smem_u32(bar), 0)) : "memory");
}
template <int CG>
__device__ __forceinline__ void sync_all() {
  __syncwarp();
  if constexpr (CG == 1) __syncthreads();
  else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// an int of any CTA of the pair, set by one of its roles before the last sync_all
template <int CG>
__device__ __forceinline__ int any_flag(const volatile int *flag) {
  if constexpr (CG == 1) return *flag;
  int x, y;
  const uint32_t a = smem_u32(const_cast<const int *>(flag));
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(x) : "r"(of_rank(a, 0)) : "memory");
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(y) : "r"(of_rank(a, 1)) : "memory");
  return x | y;
}
// raises a word of every CTA of the pair to the largest of the warp's values (none negative)
template <int CG>
__device__ __forceinline__ void raise(uint32_t *word, float x, int lane) {
  const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(x));
  if (lane != 0 || top == 0) return;
  if constexpr (CG == 1) {
    atomicMax(word, top);
  } else {
#pragma unroll
    for (uint32_t k = 0; k < CG; ++k)
      asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(of_rank(smem_u32(word), k)), "r"(top) : "memory");
  }
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// waits for the loads of this warp, v's 32 values the last of them
__device__ __forceinline__ void wait_ld32(float *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]),
                 "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]),
                 "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
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

__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t), "r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
      "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t t, uint32_t *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(t)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// two fp32 at once
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
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
__device__ __forceinline__ __half2 and_or(uint32_t w, uint32_t x) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(x));
  return half2_of(r);
}
__device__ __forceinline__ void expand(uint32_t w, const Exponents &x, __half2 (&h)[4]) {
  h[0] = __hsub2(and_or<0x000F000Fu>(w, x.a), half2_of(0x64086408u));  // 1024 + u - 1032
  h[1] = __hsub2(and_or<0x00F000F0u>(w, x.b), half2_of(0x54805480u));  // 64 + u - 72
  w >>= 8;
  h[2] = __hsub2(and_or<0x000F000Fu>(w, x.a), half2_of(0x64086408u));
  h[3] = __hsub2(and_or<0x00F000F0u>(w, x.b), half2_of(0x54805480u));
}
__device__ __forceinline__ void sts4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// the larger of a group's scale and bias, by size; NaN or infinite where one of them is (of those that were stored, NaN)
__device__ __forceinline__ float meta_size(uint32_t meta) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(__uint_as_float(meta << 16))), "f"(fabsf(__uint_as_float(meta & 0xFFFF0000u))));
  return r;
}
// scale and bias of a metadata word, times up, as fp16, twice each
__device__ __forceinline__ void split_meta(uint32_t meta, float up, __half2 &s, __half2 &o) {
  const uint32_t h = half2_bits(up * __uint_as_float(meta << 16), up * __uint_as_float(meta & 0xFFFF0000u));
  s = half2_of(__byte_perm(h, h, 0x1010));
  o = half2_of(__byte_perm(h, h, 0x3232));
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

template <typename T, int D, int GS>
struct Prefill {
  static constexpr int G = D / GS, kBlock = 16 * (D + 8 * G);
  static constexpr int CG = D == 64 ? 1 : 2;                     // CTAs that work together
  static constexpr int QT = D <= 128 ? 2 : 1, kRows = 128 * QT;  // row tiles of a CTA
  static constexpr int BN = D == 64 ? 128 : 64;                  // cached tokens of a tile
  static constexpr int BK = BN / CG, DV = D / CG;                // of them this CTA's tokens of K and channels of V
  static constexpr int NB = D == 128 ? 4 : 2;                    // buffers of S
  static constexpr bool kQTmem = D == 256;                       // Q as the MMA's operand in tensor memory
  static constexpr int kQTile = kQTmem ? 0 : (D / 64) * 128 * 128;
  static constexpr int kBoxK = BK * 128, kStageK = (D / 64) * kBoxK, kBoxV = BN * 128, kPartV = (DV / 64) * kBoxV;
  static constexpr int VP = std::is_same<T, __half>::value ? 2 : 1, kStageV = VP * kPartV;  // operands that add up to V
  static constexpr int NST = D == 64 ? 2 : 4;                    // stages of K, and of V
  static constexpr int kHeader = 2048;  // barriers, and from byte 1024 on the rows' factors
  static constexpr int kQ = kHeader, kK = kQ + QT * kQTile, kV = kK + NST * kStageK, kX = kV + NST * kStageV;
  // kX: the extra k16 step, 32 bytes of each of 128 rows: K's stages in the first two columns, Q's tiles in the others
  static constexpr int kSmem = kX + 128 * 128 + 1024;
  static_assert(kSmem <= 227 * 1024 && NST * BK <= 256, "shared memory");
  static_assert(!kQTmem || NST * kStageK >= 128 * D * 2, "room for a tile of o");
  // 16-byte pieces and rows of a stage's extra columns
  static constexpr int x_piece(int stage) { return 2 * (stage / (128 / BK)); }
  static constexpr int x_row(int stage) { return BK * (stage % (128 / BK)); }
  static constexpr int kFirstK = 4 * QT, kFirstV = kFirstK + 4, kMma = kFirstV + 4;  // the roles' first warps
  static constexpr int kThreads = 32 * (kMma + 4);
  // registers per thread: what a block of kThreads gets, and after the split the
  // softmax's, the expansions' and the MMAs' (they add up to the first one's)
  static constexpr int kRegs = QT == 2 ? 96 : 128;
  static constexpr int kRegS = QT == 2 ? 128 : 128, kRegX = QT == 2 ? 80 : 128, kRegM = QT == 2 ? 64 : 128;
  static_assert(QT * kRegS + 2 * kRegX + kRegM <= (QT + 3) * kRegs, "registers");
  // Pieces of S that the softmax's loop has at a time, the next loading meanwhile: heads of 128 gain from two (480 us for a
  // prompt of 8192 tokens, 501 with one), the others lose by the longer code (64: 46 us for six prompts of 650, 43 with one;
  // 256: 392 us for 1000 rows over 15000 tokens, 390 with one).
  static constexpr int kPieces = D == 128 ? 2 : 1;
  // tensor memory: S (and P) in NB times kS columns, O in 256 + D q; Q of heads of 256 in 128
  static constexpr int kS = BN;
};
static_assert(sizeof(Bars) <= 1024, "header");

// shared-memory stores of this warp, to the MMAs
template <int CG>
__device__ __forceinline__ void publish_smem(uint64_t *bar, int lane, int rank) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) arrive_lead<CG>(bar, rank);
}

// One warp's share of the expansion of K or V, in units numbered through all tiles.
template <typename T, int D, int GS>
struct Expander {
  using C = Prefill<T, D, GS>;
  static constexpr int G = C::G, KW = D / 32;
  const KvView &c;
  int64_t b;
  int hk, warp, lane, rank, first, tiles, begin, end;
  float up;  // what K or V is multiplied with
  Exponents exps;
  __device__ __forceinline__ bool seen(int p) const { return (unsigned)(p - begin) < (unsigned)(end - begin); }
  __device__ __forceinline__ int page_of(int p, bool in) const { return in ? c.page(b, p) : -1; }
  __device__ __forceinline__ const unsigned char *block(int page, int p) const {
    const int per = 1 << (c.page_shift - 4);
    return c.data + (((int64_t)page * c.HK + hk) * per + ((p >> 4) & (per - 1))) * C::kBlock;
  }

  // ---- K: half a block at a time, HK of them per tile and warp; a token for four lanes: lane t mod 4 has channels
  // 32 j + 8 t .. + 7 of token lane / 8 + (lane & 4), so that 8 lanes store to 8 different banks
  static constexpr int HK = C::BK / 32;
  struct KHalf {
    uint32_t code[KW], meta[G];
    bool have;
  };
  __device__ __forceinline__ int token() const { return (lane >> 3) + (lane & 4); }
  __device__ __forceinline__ int k_half(int v) const { return HK * warp + v % HK; }  // of this CTA's in the tile
  __device__ __forceinline__ int k_pos(int v) const { return first + v / HK * C::BN + rank * C::BK + (k_half(v) & ~1) * 8; }
  __device__ __forceinline__ void fetch_k(int v, int page, KHalf &r) const {
    r.have = page >= 0;
    if (!r.have) return;
    const unsigned char *p = block(page, k_pos(v));
    const int t = token() + 8 * (k_half(v) & 1);
    if constexpr (D == 64) {
      ldg_words(p + t * 32 + 8 * (lane & 3), r.code);
    } else {
#pragma unroll
      for (int k = 0; k < D / 128; ++k) {
        uint32_t w[4];
        ldg_words(p + t * (D / 2) + 64 * k + 16 * (lane & 3), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) r.code[4 * k + j] = w[j];
      }
    }
    ldg_words(p + 8 * D + t * G * 4, r.meta);
  }
  // scale q into the tile, the biases (twice) into the extra columns; both addresses are this lane's
  __device__ __forceinline__ void put_k(const KHalf &r, uint32_t dst, uint32_t extra, bool in_sight, float &top) const {
    __half2 s[G], o[G];
    uint32_t e[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < G; ++k) {
      const uint32_t meta = r.have ? r.meta[k] : 0u;
      const float size = meta_size(meta);
      if (in_sight && size < INFINITY) top = fmaxf(top, size);
      split_meta(meta, up, s[k], o[k]);
      e[k] = bits(o[k]);
    }
#pragma unroll
    for (int j = 0; j < KW; ++j) {
      __half2 v[4];
      expand(r.code[j], exps, v);
      const __half2 f = s[32 * j / GS];
      sts4((j & 1 ? dst ^ 64 : dst) + (j >> 1) * C::kBoxK, bits(__hmul2(v[0], f)), bits(__hmul2(v[1], f)), bits(__hmul2(v[2], f)),
           bits(__hmul2(v[3], f)));
    }
    // lane 0 of a token the biases, lane 1 the 17th column: -inf for a token without a page
    if (lane & 1) {
      e[0] = r.have ? 0u : 0x0000FC00u;
      e[1] = e[2] = e[3] = 0u;
    }
    if ((lane & 2) == 0) sts4(extra, e[0], e[1], e[2], e[3]);
  }
  __device__ __forceinline__ void run_k(Bars *bars, uint32_t sm) const {
    KHalf r0, r1;
    float top = 0.f;
    const int units = tiles * HK;
    auto page = [&](int v) { return page_of(k_pos(v), v < units); };
    fetch_k(0, page(0), r0);
    fetch_k(1, page(1), r1);
    int ahead = page(2);
    uint32_t s = 0, ph = 1;
    auto step = [&](int v, KHalf &r) {
      if (v % HK == 0 && !wait_warp(&bars->k_empty[s], ph, bars)) return false;
      const int row = 8 * k_half(v) + token();
      put_k(r, sm + C::kK + s * C::kStageK + swz(row, lane & 3), sm + C::kX + swz(C::x_row(s) + row, C::x_piece(s) + (lane & 1)),
            seen(k_pos(v) + 8 * (k_half(v) & 1) + token()), top);
      const int next = ahead;
      ahead = page(v + 3);
      if (v % HK == HK - 1) {
        publish_smem<C::CG>(&bars->k_full[s], lane, rank);
        if (++s == C::NST) {
          s = 0;
          ph ^= 1;
        }
      }
      fetch_k(v + 2, next, r);
      return true;
    };
#pragma unroll 1
    for (int v = 0; v < units; v += 2)
      if (!step(v, r0) || (v + 1 < units && !step(v + 1, r1))) break;
    raise<C::CG>(&bars->top_k, top, lane);
  }

  // ---- V: 64 channels of a block, VI of them per tile and warp.  Where there are two, a half warp has one each, words
  // 2 (l mod 4) and the next of tokens 2t, 2t + 1, 2t + 8, 2t + 9, t = l / 4 mod 4, and where t is odd the words change places,
  // again for the banks; else lane l has word l mod 8, t = l / 8.
  static constexpr int VI = C::BN / 16 * (C::DV / 64) / 4, VW = VI;
  static_assert(VI == 1 || VI == 2, "parts of V");
  struct VPart {
    uint4 code[VW];
    uint32_t meta[4];
    bool have;
  };
  __device__ __forceinline__ int v_block() const { return C::DV == 64 ? VI * warp + (VI == 2 ? lane >> 4 : 0) : warp; }
  __device__ __forceinline__ int v_group() const { return C::DV == 64 ? 0 : lane >> 4; }  // of this CTA's 64 channels
  __device__ __forceinline__ int v_time() const { return VI == 2 ? (lane >> 2) & 3 : lane >> 3; }
  __device__ __forceinline__ int v_piece(int w) const { return VI == 2 ? 2 * (lane & 3) + (w ^ ((lane >> 2) & 1)) : lane & 7; }
  __device__ __forceinline__ int v_pos(int i) const { return first + i * C::BN + 16 * v_block(); }
  __device__ __forceinline__ void fetch_v(int i, int page, VPart &r) const {
    r.have = page >= 0;
    if (!r.have) return;
    const int g = rank * (C::DV / 64) + v_group(), t = v_time();
    const unsigned char *p = block(page, v_pos(i)) + 8 * D + 64 * G;
#pragma unroll
    for (int w = 0; w < VW; ++w) r.code[w] = __ldg(reinterpret_cast<const uint4 *>(p + (8 * g + v_piece(w)) * 64 + 16 * t));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r.meta[j] = __ldg(reinterpret_cast<const uint32_t *>(p + 8 * D) + (2 * t + (j & 1) + 8 * (j >> 1)) * G + 64 * g / GS);
  }
  // scale q + bias; tokens with values beyond fp16 become 0, which no P of 0 turns into NaN: those that no row sees, and
  // else NaN and infinities, which are reported (or what the second time brings into range)
  __device__ __forceinline__ bool put_v(const VPart &r, uint32_t dst, int pos, float &top) const {
    const int row0 = 16 * v_block() + 2 * v_time();
    dst += v_group() * C::kBoxV;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = row0 + (j & 1) + 8 * (j >> 1);
      const float size = meta_size(r.meta[j]);
      const bool finite = size < INFINITY, in_sight = r.have && seen(pos + row);
      bad |= in_sight && !finite;
      if (in_sight && finite) top = fmaxf(top, size);
      __half2 s, o;
      split_meta(r.have && size * up < (float)(1 << kHigh) ? r.meta[j] : 0u, up, s, o);
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint4 &u = r.code[w];
        __half2 h[4];
        expand(j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w, exps, h);
        if constexpr (C::VP == 1) {
          sts4(dst + swz(row, v_piece(w)), bits(__hfma2(h[0], s, o)), bits(__hfma2(h[1], s, o)), bits(__hfma2(h[2], s, o)),
               bits(__hfma2(h[3], s, o)));
        } else {
          sts4(dst + swz(row, v_piece(w)), bits(__hmul2(h[0], s)), bits(__hmul2(h[1], s)), bits(__hmul2(h[2], s)), bits(__hmul2(h[3], s)));
          sts4(dst + C::kPartV + swz(row, v_piece(w)), bits(o), bits(o), bits(o), bits(o));
        }
      }
    }
    return bad;
  }
  __device__ __forceinline__ void run_v(Bars *bars, uint32_t sm) const {
    VPart r0, r1;
    float top = 0.f;
    auto page = [&](int i) { return page_of(v_pos(i), i < tiles); };
    fetch_v(0, page(0), r0);
    fetch_v(1, page(1), r1);
    int ahead = page(2);
    uint32_t s = 0, ph = 1;
    auto step = [&](int i, VPart &r) {
      if (!wait_warp(&bars->v_empty[s], ph, bars)) return false;
      if (put_v(r, sm + C::kV + s * C::kStageV, first + i * C::BN, top)) bars->bad_v = 1;
      const int next = ahead;
      ahead = page(i + 3);
      publish_smem<C::CG>(&bars->v_full[s], lane, rank);
      if (++s == C::NST) {
        s = 0;
        ph ^= 1;
      }
      fetch_v(i + 2, next, r);
      return true;
    };
#pragma unroll 1
    for (int i = 0; i < tiles; i += 2)
      if (!step(i, r0) || (i + 1 < tiles && !step(i + 1, r1))) break;
    raise<C::CG>(&bars->top_v, top, lane);
  }
};

// The power of two that brings a row's largest value into [2^7, 2^8), as the factor of Q (a negative scale goes with
// it), and what S is multiplied with to give logits in octaves.
__device__ __forceinline__ float2 q_factors(float big, float scale) {
  const int be = (int)(__float_as_uint(big) >> 23);
  const int e = be == 0 || be == 255 ? 0 : min(7 - (be - 127), 126);
  return make_float2(scale < 0.f ? -pow2f(e) : pow2f(e), fmaxf(fabsf(scale) * kLog2e * pow2f(-e), 1e-30f));
}
template <typename T>
__device__ __forceinline__ void widen8(const uint4 &v, float (&x)[8]) {
  constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[2 * k] = meta_f32(w[k], bf);
    x[2 * k + 1] = meta_f32(w[k] >> 16, bf);
  }
}
// the high and low fp16 half of x
__device__ __forceinline__ uint32_t high_low(float x) { return half2_bits(x, x - __half2float(__float2half_rn(x))); }

// A warp's 32 rows of Q (from row `first` of the sequence, `at` of the row tile q), scaled, to where the MMAs read them,
// with the extra columns; returns the factor of this lane's row.
template <typename T, int D, int GS>
__device__ __forceinline__ float load_q(const KvAttention &a, const Rows &rows, uint32_t sm, uint32_t tl, int first, int hk, int r, int q,
                                        int at, int lane) {
  using C = Prefill<T, D, GS>;
  constexpr int G = C::G;
  auto row_of = [&](int i) {
    const int row = min(first + i, rows.rows - 1);  // rows past the last repeat it
    return static_cast<const T *>(a.q) + (rows.t0 + row / r) * a.q_stride + (int64_t)(hk * r + row % r) * D;
  };
  if constexpr (C::kQTmem) {
    // a row per lane, in two passes of 64 channels at a time
    const T *src = row_of(lane);
    float big = 0.f, sum[G] = {};
#pragma unroll 1
    for (int k = 0; k < D / 64; ++k) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(src) + 8 * k + i);
      float all = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[8];
        widen8<T>(v[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          big = fmaxf(big, fabsf(x[j]));
          all += x[j];
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) sum[g] += g == 64 * k / GS ? all : 0.f;
    }
    const float2 f = q_factors(big, a.scale);
#pragma unroll 1
    for (int k = 0; k < D / 64; ++k) {
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(src) + 8 * k + i);
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x[8];
        widen8<T>(v[i], x);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = half2_bits(f.x * x[j], f.x * x[j + 4]);
      }
      tm_st32(tl + 128 + 32 * k, w);
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int g = 0; g < G; ++g) w[g] = high_low(f.x * sum[g]);
    sts4(sm + C::kX + swz(at + lane, 4 + 2 * q), w[0], w[1], w[2], w[3]);
    sts4(sm + C::kX + swz(at + lane, 5 + 2 * q), 0x00003C00u, 0u, 0u, 0u);  // 1, against what is -inf for a missing token
    return f.y;
  } else {
    // whole rows by neighbouring lanes, 16 bytes each
    constexpr int kPieces = D / 8, kRowsAtOnce = 32 / kPieces;
    const int piece = lane % kPieces;
    const uint32_t dst = sm + C::kQ + q * C::kQTile + (piece >> 3) * (128 * 128), fac = sm + 1024 + (128 * q + at) * 4;
    const long long own = reinterpret_cast<long long>(row_of(lane));  // (a division, once per lane)
#pragma unroll 1
    for (int n0 = 0; n0 < kPieces; n0 += 4) {
      uint4 v[4];  // loads before the first store
#pragma unroll
      for (int n = 0; n < 4; ++n)
        v[n] = __ldg(reinterpret_cast<const uint4 *>(__shfl_sync(0xffffffffu, own, (n0 + n) * kRowsAtOnce + lane / kPieces)) + piece);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int i = (n0 + n) * kRowsAtOnce + lane / kPieces;
        float x[8];
        widen8<T>(v[n], x);
        float big = 0.f, sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          big = fmaxf(big, fabsf(x[j]));
          sum += x[j];
        }
#pragma unroll
        for (int o = 1; o < kPieces; o <<= 1) {
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
          if (o < GS / 8) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        const float2 f = q_factors(big, a.scale);
        sts4(dst + swz(at + i, piece & 7), half2_bits(f.x * x[0], f.x * x[4]), half2_bits(f.x * x[1], f.x * x[5]),
             half2_bits(f.x * x[2], f.x * x[6]), half2_bits(f.x * x[3], f.x * x[7]));
        auto sts1 = [](uint32_t to, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(v) : "memory"); };
        const uint32_t extra = sm + C::kX + swz(at + i, 4 + 2 * q), one = sm + C::kX + swz(at + i, 5 + 2 * q);
        if (piece % (GS / 8) == 0) sts1(extra + 4 * (piece / (GS / 8)), high_low(f.x * sum));
        if (piece > 0 && piece < 4 && piece >= G) sts1(extra + 4 * piece, 0u);
        if (piece >= 4 && piece < 8) sts1(one + 4 * (piece - 4), piece == 4 ? 0x00003C00u : 0u);  // 1, against what is -inf for a missing token
        if (piece == 0) sts1(fac + 4 * i, __float_as_uint(f.y));
      }
    }
    __syncwarp();
    uint32_t f;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(f) : "r"(fac + 4 * lane) : "memory");
    return __uint_as_float(f);
  }
}

template <typename T, int D, int GS>
__global__ void __launch_bounds__((Prefill<T, D, GS>::kThreads), 1) kv_prefill_kernel(const KvView c, const KvAttention a, int tiles, int splits,
                                                                                      float *part) {
  using C = Prefill<T, D, GS>;
  using X = Expander<T, D, GS>;
  constexpr int G = C::G, QT = C::QT, BN = C::BN, CG = C::CG;
  extern __shared__ unsigned char smem_raw[];
  unsigned char *base = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Bars *bars = reinterpret_cast<Bars *>(base);
  const uint32_t sm = smem_u32(base);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  // the last tiles first: they see the most
  const int rank = blockIdx.x % CG;  // in the pair
  int64_t id = blockIdx.x / CG;
  const int split = (int)(id % splits);
  id /= splits;
  const int64_t heads = c.B * c.HK;
  const int tile0 = tiles - 1 - (int)(id / heads);
  id %= heads;
  const int hk = (int)(id % c.HK), r = a.HQ / c.HK;
  const int64_t b = id / c.HK;
  Rows rows0;
  if (!rows0.set<CG * C::kRows, BN>(c, a, b, tile0, split, splits)) return;

  auto init = [&](bool again, const Rows &rows, int tile, int up_k, int up_v, bool second) {
    if (tid == 0) {
      bars->rows.put(rows);
      bars->tile = tile;
      bars->up_k = up_k, bars->up_v = up_v, bars->second = second;
      bars->top_k = bars->top_v = 0;
      if (again)
        for (uint64_t *bar = bars->k_full; bar <= &bars->drain; ++bar)
          asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
      for (int s = 0; s < 4; ++s) {
        mbar_init(&bars->k_full[s], 4 * CG);
        mbar_init(&bars->v_full[s], 4 * CG);
        mbar_init(&bars->k_empty[s], QT);
        mbar_init(&bars->v_empty[s], QT);
        mbar_init(&bars->s_full[s], 1);
        mbar_init(&bars->p_ready[s], 4 * CG);
      }
      mbar_init(&bars->o_done[0], 1);
      mbar_init(&bars->o_done[1], 1);
      mbar_init(&bars->q_full, 4 * QT * CG);
      mbar_init(&bars->drain, QT);
      bars->bad_v = 0;
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  };
  if (tid == 0) bars->abort_flag = 0;
  init(false, rows0, tile0, kUpK, kUpV, false);
  if (warp == C::kMma) {
    asm volatile("tcgen05.alloc.cta_group::%2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bars->tmem_base)), "r"(512),
                 "n"(CG)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::%0.sync.aligned;" ::"n"(CG) : "memory");
  }
  fence_before();
  sync_all<CG>();
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);

  // Every role goes through the CTA's tiles (one, unless the hint max_q was too small; twice, where the sizes of K or V turn out
  // not to suit) and meets the others at the end of each; false: no other tile.
  auto next = [&]() -> bool {
    fence_before();
    sync_all<CG>();
    fence_after();
    Rows rows;
    const bool second = once_more(bars);
    const uint32_t top_k = bars->top_k, top_v = bars->top_v;
    int up_k = bars->up_k, up_v = bars->up_v;
    if (second && unsuited(top_k, up_k, kLowK)) up_k = min(kHigh - 1 - octave(top_k), 100);
    if (second && unsuited(top_v, up_v, kLowV)) up_v = min(kHigh - 1 - octave(top_v), 100);
    const int tile = bars->tile + (second ? 0 : tiles);
    const bool more = !any_flag<CG>(&bars->abort_flag) && rows.set<CG * C::kRows, BN>(c, a, b, tile, split, splits);
    sync_all<CG>();  // (each has read what the other's may change)
    if (!more) return false;
    init(true, rows, tile, up_k, up_v, second);
    sync_all<CG>();
    return true;
  };

  if (warp < C::kFirstK) {
    // ---------------- softmax: a row per thread
    if constexpr (C::kRegS > C::kRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegS));
    const int q = warp >> 2, quarter = warp & 3;
    const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16), to = tl + 256 + D * q;
    do {
      Rows rows = bars->rows.get();
      const int row0 = CG * (bars->tile * C::kRows + 128 * q) + 128 * rank + 32 * quarter;  // this warp's rows
      const int pos = rows.pos0 + min(row0 + lane, rows.rows - 1) / r;
      const int hi = pos < 0 ? -1 : a.causal ? pos : rows.len - 1, lo = a.window ? max(pos, 0) - a.window : -1;  // lo < j <= hi is seen
      const int hi_all = __reduce_min_sync(0xffffffffu, hi), lo_all = __reduce_max_sync(0xffffffffu, lo);
      const float f = fmaxf(load_q<T, D, GS>(a, rows, sm, tl, row0, hk, r, q, 32 * quarter, lane) * pow2f(-bars->up_k), 1e-30f);
      if constexpr (C::kQTmem) {
        wait_st();
        fence_before();
      }
      publish_smem<CG>(&bars->q_full, lane, rank);
      float M = kNone, L = 0.f;
      bool ok = true;
      const int n = rows.tiles, first = rows.first;
      for (int i = 0; i < n; ++i) {
        const int buf = (QT * i + q) % C::NB;
        const uint32_t ph = (QT * i + q) / C::NB & 1, ts = tl + C::kS * buf;
        if (!(ok = wait_warp(&bars->s_full[buf], ph, bars))) break;
        fence_after();
        const int n0 = first + i * BN, h = hi - n0, l = lo - n0;
        const bool masked = n0 <= lo_all || n0 + BN - 1 > hi_all;
        auto mask = [&](float(&x)[32], int k) {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = k + j > l && k + j <= h ? x[j] : -INFINITY;
        };
        float sum = 0.f;
        // P of 32 columns, into the 16 that its part of S leaves free
        auto piece = [&](float(&x)[32], int k) {
          if (masked) mask(x, k);
          uint32_t w[16];
          float s4[4];
#pragma unroll 1
          for (bool again = false;; again = true) {
            const uint64_t f2 = pair(f, f), neg2 = pair(kShift - M, kShift - M);
            uint64_t s2[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float u, v;
              unpair(fma2(pair(x[2 * j], x[2 * j + 1]), f2, neg2), u, v);
              u = ex2(u), v = ex2(v);
              s2[j & 1] = add2(s2[j & 1], pair(u, v));
              w[j] = half2_bits(u, v);
            }
            unpair(s2[0], s4[0], s4[1]);
            unpair(s2[1], s4[2], s4[3]);
            s4[0] = (s4[0] + s4[1]) + (s4[2] + s4[3]);
          // What sums to no more than fp16's largest value has no part beyond it.  Else (on the first piece, and seldom
          // again) the reference moves to the largest logit that is left in the tile, in whole octaves, so that what
          // is there already, O, L and P, is scaled exactly.
          if (again || !__any_sync(0xffffffffu, !(s4[0] <= 65504.f))) break;
            float top = kNone;
#pragma unroll 1
            for (int n = k; n < BN; n += 32) {
              float y[32];
              tm_ld32(ts + n, y);
              wait_ld32(y);
              if (masked) mask(y, n);
#pragma unroll
              for (int j = 0; j < 32; j += 2) top = max3(top, y[j], y[j + 1]);
            }
            // (a load of tensor memory is not ordered behind this thread's stores: P of earlier pieces, O of an earlier move)
            wait_st();
            const float next = top > kNone ? fmaxf(M, ceilf(top * f)) : M, move = M - next;
            const float down = move >= 0.f ? 1.f : move > -126.f ? pow2f((int)move) : 0.f;
            M = next;
            L *= down;
            sum *= down;
            const __half2 d2 = __float2half2_rn(down);
#pragma unroll 1
            for (int n = 0; n < k; n += 32) {
              uint32_t y[16];
              tm_ld16(ts + n / 2, y);
#pragma unroll
              for (int j = 0; j < 16; ++j) y[j] = bits(__hmul2(half2_of(y[j]), d2));
              tm_st16(ts + n / 2, y);
            }
            if (i > 0) {
              // O's product of the tile before (the one before that is complete, for S followed it or one later); the next
              // waits for P
              ok = wait_warp(&bars->o_done[q], (i - 1) & 1, bars) && ok;
              fence_after();
#pragma unroll 1
              for (int n = 0; n < D; n += 32) {
                float o[32];
                tm_ld32(to + n, o);
                wait_ld32(o);
                uint32_t v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(o[j] * down);
                tm_st32(to + n, v);
              }
            }
          }
          sum += s4[0];
          tm_st16(ts + k / 2, w);
        };
#pragma unroll 1
        for (int k = 0; k < BN; k += 32 * C::kPieces) {
          float x[C::kPieces][32];
          tm_ld32(ts + k, x[0]);
#pragma unroll
          for (int h = 0; h < C::kPieces; ++h) {
            wait_ld32(x[h]);
            if (h + 1 < C::kPieces) tm_ld32(ts + k + 32 * (h + 1), x[h + 1]);
            piece(x[h], k + 32 * h);
          }
        }
        if (!ok) break;
        L += sum;
        wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) arrive_lead<CG>(&bars->p_ready[buf], rank);
      }
      rows = bars->rows.get();
      // O's last product.  With two buffers of S per row tile the last two may be open (S of a tile only says that the
      // product two tiles before is complete), and o_done's parity cannot tell them apart: all MMAs, then.
      if (ok && rows.tiles > 0) ok = C::NB == QT ? wait_warp(&bars->o_done[q], (rows.tiles - 1) & 1, bars) : wait_warp(&bars->drain, 0, bars);
      // every role meets here: what the expansions found, in both CTAs, is final, and seen
      fence_before();
      sync_all<CG>();
      fence_after();
      if (once_more(bars)) continue;
      const float back = pow2f(-bars->up_v), inv = splits > 1 ? back : L == 0.f ? 0.f : back / L;
      uint32_t nan = 0;  // a bit per group of channels
      if (ok && any_flag<CG>(&bars->bad_v)) {
        // rows that see such a token become NaN in its group's channels
        for (int p = max(lo + 1, 0); p <= min(hi, (int)min((int64_t)rows.len, c.table_width << c.page_shift) - 1); ++p) {
          const int page = c.page(b, p);
          if (page < 0) continue;
          const unsigned char *blk = c.block(page, hk, p) + 16 * D + 64 * G + (p & 15) * G * 4;
          for (int g = 0; g < G; ++g) nan |= (uint32_t)!(meta_size(__ldg(reinterpret_cast<const uint32_t *>(blk) + g)) < INFINITY) << g;
        }
      }
      auto factor = [&](int k) { return nan >> (k / GS) & 1u ? __int_as_float(0x7fc00000) : inv; };  // of channel k and the others of its group
      __syncwarp();
      // rows of o through shared memory (Q's tile; K's stages for heads of 256: no MMA reads them any more), so that a
      // warp stores whole rows
      const uint32_t stage = sm + (C::kQTmem ? C::kK : C::kQ + q * C::kQTile) + quarter * (32 * D * 2);
      auto lds4 = [](uint32_t from) {
        uint4 w;
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(from) : "memory");
        return w;
      };
      const int mine = row0 + lane;
      constexpr int kPieces = D / 8;
      if (splits > 1) {
        // a part: o as it is, fp32, 32 channels at a time, its reference and its sum
        const int64_t step = (int64_t)splits * (D + 4);
        auto part_of = [&](int row) { return part + ((rows.t0 + row / r) * a.HQ + hk * r + row % r) * step + (int64_t)split * (D + 4); };
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          float o[32];
          if (rows.tiles > 0) {
            tm_ld32(to + k, o);
            wait_ld32(o);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0.f;
          }
          const float by = factor(k);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            // columns hold channels 0 4 1 5 2 6 3 7
            const int at = j & ~7, odd = (j >> 2) & 1;
            sts4(stage + lane * 128 + (((j >> 2) ^ (lane & 7)) << 4), __float_as_uint(o[at + odd] * by), __float_as_uint(o[at + odd + 2] * by),
                 __float_as_uint(o[at + odd + 4] * by), __float_as_uint(o[at + odd + 6] * by));
          }
          __syncwarp();
#pragma unroll 1
          for (int n = 0; n < 8; ++n) {
            const int from = 4 * n + (lane >> 3), piece = lane & 7;
            const uint4 w = lds4(stage + from * 128 + ((piece ^ (from & 7)) << 4));
            if (ok && row0 + from < rows.rows) reinterpret_cast<uint4 *>(part_of(row0 + from) + k)[piece] = w;
          }
        }
        if (ok && mine < rows.rows) *reinterpret_cast<float2 *>(part_of(mine) + D) = make_float2(M - kShift, L);
        continue;
      }
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        float o[32];
        if (rows.tiles > 0) {
          tm_ld32(to + k, o);
          wait_ld32(o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0.f;
        }
        const float by = factor(k);
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = by == 0.f ? 0.f : o[j] * by;
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
          const int piece = (k + j) / 8;
          sts4(stage + lane * (D * 2) + (((piece & ~7) | ((piece ^ lane) & 7)) << 4), w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
#pragma unroll 4
      for (int n = 0; n < kPieces; ++n) {
        const int from = n * (32 / kPieces) + lane / kPieces, piece = lane % kPieces;  // row of the warp, piece of the row
        const int other = row0 + from;
        const uint4 w = lds4(stage + from * (D * 2) + (((piece & ~7) | ((piece ^ from) & 7)) << 4));
        if (ok && other < rows.rows)
          reinterpret_cast<uint4 *>(static_cast<T *>(a.o) + (rows.t0 + other / r) * a.o_stride + (int64_t)(hk * r + other % r) * D)[piece] = w;
      }
      if (ok && a.lse && mine < rows.rows) a.lse[(rows.t0 + mine / r) * a.HQ + hk * r + mine % r] = L == 0.f ? -INFINITY : (M + log2f(L) - kShift) * kLn2;
    } while (next());
  } else if (warp < C::kMma) {
    // ---------------- expansion of K, or of V
    if constexpr (C::kRegX < C::kRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegX));
    do {
      const Rows rows = bars->rows.get();
      const bool of_k = warp < C::kFirstV;
      const X x{c, b, hk, warp & 3, lane, rank, rows.first, c_kv_stall ? 0 : rows.tiles, rows.begin, rows.end, pow2f(of_k ? bars->up_k : bars->up_v)};
      if (of_k) x.run_k(bars, sm);
      else x.run_v(bars, sm);
      sync_all<CG>();  // (the softmax's, before it looks at what was found)
    } while (next());
  } else {
    if constexpr (C::kRegM < C::kRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegM));
    do {
      const int q = warp - C::kMma;
      if (q < QT) {
        // ---------------- the MMAs of row tile q: S over the tile i, O of it.  A thread per row tile: an issue takes 20 to
        // 40 clocks and a wait on a barrier 80 to 180, also where it holds already, so that one thread for both kept the
        // tensor cores waiting.
        if (rank == 0 && elect_one()) {
          const int n = bars->rows.tiles;
          bool ok = wait_one(&bars->q_full, 0, bars);
          const uint32_t q0 = C::kQTmem ? tmem + 128 : desc_k(sm + C::kQ + q * C::kQTile), k0 = desc_k(sm + C::kK),
                         v0 = desc_mn(sm + C::kV, C::kBoxV), x0 = desc_k(sm + C::kX), o = tmem + 256 + D * q;
          constexpr int kAhead = C::NB / QT;  // buffers of S of a row tile
          auto k_ready = [&](int i) { return mbar_test(&bars->k_full[i % C::NST], i / C::NST & 1); };
          auto scores = [&](int i, bool ready) {
            const int s = i % C::NST, buf = QT * (i % kAhead) + q;
            if (!ready && !wait_one(&bars->k_full[s], i / C::NST & 1, bars)) return false;
            fence_after();
            const uint32_t d = tmem + C::kS * buf;
            uint32_t qa = q0, kb = k0 + s * (C::kStageK / 16);
#pragma unroll 1
            for (int k = 0; k < D / 64; ++k, qa += C::kQTmem ? 32 : 128 * 128 / 16, kb += C::kBoxK / 16)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if constexpr (C::kQTmem) umma_ts<CG>(d, qa + 8 * j, kb + 2 * j, idesc(128 * CG, BN, false), k > 0 || j > 0);
                else umma_ss<CG>(d, qa + 2 * j, kb + 2 * j, idesc(128 * CG, BN, false), k > 0 || j > 0);
              }
            umma_ss<CG>(d, x0 + 4 + 2 * q, x0 + C::x_row(s) * 8 + C::x_piece(s), idesc(128 * CG, BN, false), true);
            umma_commit<CG>(&bars->s_full[buf]);
            umma_commit<CG>(&bars->k_empty[s]);
            return true;
          };
          for (int i = 0; ok && i < kAhead && i < n; ++i) ok = scores(i, false);
#pragma unroll 1
          for (int i = 0; ok && i < n; ++i) {
            const int s = i % C::NST, buf = QT * (i % kAhead) + q;
            // the three that this tile waits for, asked at once: the answers take a while
            const bool v = mbar_test(&bars->v_full[s], i / C::NST & 1), pr = mbar_test(&bars->p_ready[buf], i / kAhead & 1),
                       k = k_ready(i + kAhead);
            if (!(ok = v || wait_one(&bars->v_full[s], i / C::NST & 1, bars))) break;
            if (!(ok = pr || wait_one(&bars->p_ready[buf], i / kAhead & 1, bars))) break;
            fence_after();
            uint32_t p = tmem + C::kS * buf, vb = v0 + s * (C::kStageV / 16);
#pragma unroll 1
            for (int h = 0; h < BN / 64; ++h, p += 32, vb += 4 * 2048 / 16)
#pragma unroll
              for (int j = 0; j < 4 * C::VP; ++j)
                umma_ts<CG>(o, p + 8 * (j & 3), vb + (j & 3) * (2048 / 16) + (j >> 2) * (C::kPartV / 16), idesc(128 * CG, D, true),
                            i > 0 || h > 0 || j > 0);
            umma_commit<CG>(&bars->o_done[q]);
            umma_commit<CG>(&bars->v_empty[s]);
            // P's place is free for other scores
            if (i + kAhead < n) ok = scores(i + kAhead, k);
          }
          umma_commit<CG>(&bars->drain);  // every MMA issued, complete before their memory is used again
        }
        __syncwarp();
        const unsigned long long since = global_ns();
        while (!mbar_try(&bars->drain, 0) && global_ns() - since < c_kv_wait_ns) {
        }
      }
      fence_before();
      sync_all<CG>();
      fence_after();
    } while (next());
  }
  if (warp == C::kMma) asm volatile("tcgen05.dealloc.cta_group::%2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512), "n"(CG));
}

// Joins the parts of a row: D / 4 threads per row, four channels each.
constexpr int kJoinThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) kv_join_parts_kernel(const KvView c, const KvAttention a, int splits, const float *part) {
  constexpr int kLanes = D / 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t id = (int64_t)blockIdx.x * (kJoinThreads / kLanes) + threadIdx.x / kLanes, tok = id / a.HQ;
  const int lane = threadIdx.x % kLanes;
  int64_t first, last, skip;
  c.range(0, first, skip);
  c.range(c.B - 1, skip, last);
  if (tok < first || tok >= last) return;  // (a row of no sequence)
  const float *src = part + id * splits * (D + 4);
  float m = kNone, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < splits; i += 4) {
    float2 q[4];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < splits) {
        q[k] = __ldcs(reinterpret_cast<const float2 *>(src + (i + k) * (D + 4) + D));
        v[k] = __ldcs(reinterpret_cast<const float4 *>(src + (i + k) * (D + 4)) + lane);
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < splits) {
        const float top = fmaxf(m, q[k].x), z = ex2(m - top), z2 = ex2(q[k].x - top);
        m = top;
        l = fmaf(z, l, z2 * q[k].y);
        o.x = fmaf(z, o.x, z2 * v[k].x);
        o.y = fmaf(z, o.y, z2 * v[k].y);
        o.z = fmaf(z, o.z, z2 * v[k].z);
        o.w = fmaf(z, o.w, z2 * v[k].w);
      }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T *dst = static_cast<T *>(a.o) + tok * a.o_stride + (id - tok * a.HQ) * D + 4 * lane;
  uint2 w;
  if constexpr (std::is_same<T, __half>::value) {
    w = make_uint2(half2_bits(o.x * inv, o.y * inv), half2_bits(o.z * inv, o.w * inv));
  } else {
    const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(o.x * inv, o.y * inv), __floats2bfloat162_rn(o.z * inv, o.w * inv)};
    w = make_uint2(*reinterpret_cast<const uint32_t *>(&h[0]), *reinterpret_cast<const uint32_t *>(&h[1]));
  }
  *reinterpret_cast<uint2 *>(dst) = w;
  if (lane == 0 && a.lse) a.lse[id] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

struct Shape {
  int64_t rows, tiles, units, slots;  // rows of a tile of a CTA or pair; tiles that the longest sequence has; of all; how many run at once
};
Shape shape(const KvView &c, const KvAttention &a) {
  const int r = a.HQ / c.HK, cg = c.D == 64 ? 1 : 2;
  Shape s;
  s.rows = c.D == 128 ? 512 : 256;
  s.tiles = (std::min(std::max<int64_t>(a.max_q, 1), c.T) * r + s.rows - 1) / s.rows;
  s.units = std::min(s.tiles * c.B, c.T * r / s.rows + c.B) * c.HK;
  s.slots = 152 / cg;
  return s;
}

template <typename T, int D, int GS>
cudaError_t run(const KvView &c, const KvAttention &a, int splits, float *part, cudaStream_t st) {
  using C = Prefill<T, D, GS>;
  static std::atomic<uint64_t> ready{0};
  const int dev = current_device();
  if (not_done(ready, dev)) {
    cudaFuncAttributes at;
    cudaError_t e = cudaFuncGetAttributes(&at, kv_prefill_kernel<T, D, GS>);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kv_prefill_kernel<T, D, GS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    // the warps' shares come out of what the block was launched with
    if (e == cudaSuccess && C::kRegS > C::kRegs && at.numRegs != C::kRegs) e = cudaErrorInvalidConfiguration;
    if (e != cudaSuccess) return e;
    mark_done(ready, dev);
  }
  const Shape s = shape(c, a);
  const int64_t tiles = kv_tiles_of_grid(c, s.tiles, c.T * (a.HQ / c.HK), s.rows), ctas = tiles * c.B * c.HK * C::CG * splits;
  const int64_t joins = (c.T * a.HQ * (D / 4) + kJoinThreads - 1) / kJoinThreads;
  if (ctas > INT32_MAX || joins > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C::CG;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = C::CG > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_prefill_kernel<T, D, GS>, c, a, (int)tiles, splits, part);
  if (e != cudaSuccess || splits == 1) return e;
  cfg.gridDim = dim3((unsigned)joins, 1, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_join_parts_kernel<T, D>, c, a, splits, const_cast<const float *>(part));
}
template <typename T>
cudaError_t run_t(const KvView &c, const KvAttention &a, int splits, float *part, cudaStream_t st) {
  if (c.D == 64) return run<T, 64, 64>(c, a, splits, part, st);
  if (c.D == 128) return c.gs == 64 ? run<T, 128, 64>(c, a, splits, part, st) : run<T, 128, 128>(c, a, splits, part, st);
  return c.gs == 64 ? run<T, 256, 64>(c, a, splits, part, st) : run<T, 256, 128>(c, a, splits, part, st);
}

}  // namespace

// Costs in units of what a tile of rows takes per cached token, 12 to 14 ns for each size of heads.  A tile's CTAs cost 1050
// of them besides (14 us: start, Q, O); its tokens may be split over several, which costs the join's launch (230) and
// the parts' traffic.  Few rows at a time take 2^-19 per row, channel and token (3.2 ps per row of 128 channels), 0.001 per row and
// channel (128 at most) for their CTAs' starts, 400 for the call.  Both sides measured, in us, few rows / tiles in one part / as
// chosen here, 32 query heads over 8 of 128 channels:
//   16 new tokens over 60000           104 / 806 / 112
//   64                                 401 / 807 / 112
//   128 over 4000                       81 /  69 /  30
//   12 of 16 sequences over 4000        92 / 134 /  92
//   24                                 181 / 134 / 136
//   128 alone                           12 /  15 /  12
int kv_tiles_splits(const KvView &c, const KvAttention &a, q1_dtype t) {
  if (t == Q1_F32) return 0;
  const Shape s = shape(c, a);
  int64_t seen = std::max<int64_t>(a.max_len, 1);
  if (a.window) seen = std::min<int64_t>(seen, (int64_t)a.window + s.rows / (a.HQ / c.HK));
  const double values = (double)c.T * a.HQ * c.D;
  // The tensor cores cut what they add to O instead of rounding it: 2^-27.5 of O per token and product, where all are of one sign
  // (200000 tokens 1.0e-3).  So a part has at most 2^15 tokens of fp16 outputs (two products), 2^18 of bf16, which stays below half
  // a step of these.
  const int least = (int)std::min<int64_t>((seen - 1) >> (t == Q1_F16 ? 15 : 18), 31) + 1;
  double best = values / (1 << 19) * (double)seen + 0.001 * values / c.D * std::min(c.D, 128) + 400;
  int splits = 0;
  for (int n = least; n <= 32 && (n == least || seen / n >= 128); ++n) {
    const double rounds = (double)((s.units * n + s.slots - 1) / s.slots);
    const double cost = rounds * (1050 + (double)seen / n) + (n > 1 ? 230 + 9e-5 * n * values : 0);
    if (cost < best) best = cost, splits = n;
  }
  return splits;
}
size_t kv_tiles_workspace_bytes(const KvView &c, const KvAttention &a, int splits) {
  return splits > 1 ? (size_t)c.T * a.HQ * splits * (c.D + 4) * sizeof(float) : 0;
}

cudaError_t launch_kv_prefill(const KvView &c, const KvAttention &a, q1_dtype t, int splits, void *workspace, cudaStream_t st) {
  float *part = static_cast<float *>(workspace);
  return t == Q1_BF16 ? run_t<__nv_bfloat16>(c, a, splits, part, st) : run_t<__half>(c, a, splits, part, st);
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
