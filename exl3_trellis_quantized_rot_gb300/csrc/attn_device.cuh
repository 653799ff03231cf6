// Device helpers shared by the attention kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>

#include "attn_internal.h"
#include "exl3_kernels.cuh"

namespace tfx {

// 5-D tensor copy: (value within a 64-value column block, token, column block, head, page).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t* b) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];" ::"r"(dst),
      "l"(tm), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(s_addr(b))
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* tm, int c0, int c1, int c2, int c3, int c4,
                                            uint64_t* b) {
  tma_load_5d(s_addr(dst), tm, c0, c1, c2, c3, c4, b);
}

// A map's descriptor on its way, ahead of the first copy by it.
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* tm) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(tm) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two values as T, rounded; beyond its range its largest, a NaN stays. For what 8-bit codes stand for, which
// can be beyond it where no appended value was: 65,504 of FP16 is code 64 under the I8 scale 2^10.
template <typename T>
__device__ __forceinline__ uint32_t pack2_finite(float lo, float hi) {
  uint32_t r;
  if constexpr (__is_same(T, __half))
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The largest probability is 2^kShift: FP16 has no normal numbers below 2^-14,
// and a shift of 7 keeps 11 bits down to 2^-21 of the row's largest term. BF16
// has the range of FP32 and needs none.
template <typename T>
struct Exponent;
template <>
struct Exponent<__half> {
  static constexpr float kShift = 7.f;
};
template <>
struct Exponent<__nv_bfloat16> {
  static constexpr float kShift = 0.f;
};

// 32 consecutive TMEM columns of this warp's 32 lanes; the registers are valid after tmem_loaded.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}

__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
               : "memory");
}
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- pairs of CTAs (cta_group::2): the even one issues the MMAs of both ------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Both CTAs come together, and nothing more: barriers are made visible by their own
// fence, and a release here waits for every store under way (about 1,300 cycles
// at a kernel's end, measured).
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// This CTA's shared address `a` in the CTA of the given rank.
__device__ __forceinline__ uint32_t peer_addr(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
// Arrivals on a barrier of either CTA. Without a release at cluster scope, which
// made a warp wait about 1,100 cycles for everything it had stored (measured): what
// they hand over is in tensor memory, or is read by the asynchronous proxy after
// a proxy fence. Nothing orders such an arrival before the pair's closing
// barrier, so none may be left that nobody waits for: the commits' arrivals (commit2)
// too, which warp 11 sees out at the end.
__device__ __forceinline__ void arrive_at(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void expect_tx_at(uint32_t cluster_bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(cluster_bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void store_at(uint32_t cluster_addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}
// A copy into this CTA's shared memory that counts on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap* tm, int c0, int c1, int c2, int c3, int c4,
                                                 uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
      "%5, %6}], [%7];" ::"r"(dst),
      "l"(tm), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(cluster_bar)
      : "memory");
}
// D[tmem] (+)= A[smem] B[smem] and D[tmem] (+)= A[tmem] B[smem], over the pair.
__device__ __forceinline__ void mma2_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
      "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma2_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
      "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives on the barrier at this shared address in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit2(uint64_t* b) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(s_addr(b)),
      "h"((uint16_t)3)
      : "memory");
}

// Shared-memory operands with the 128-byte swizzle: rows of 64 values (128 bytes),
// atoms of 8 rows (1 KB). `lead`: bytes between column blocks of 64 values of an
// operand whose columns are its M or N index (unused where they are its K index).
__host__ __device__ constexpr uint64_t operand_bits(uint32_t lead) {
  return ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t operand(uint32_t saddr, uint64_t bits) { return bits | ((saddr & 0x3FFFF) >> 4); }

// Two FP32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void parts_of(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Where a warp is in a ring of N barriers, and the parity it waits for there.
template <int N>
struct Turn {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      parity ^= 1;
    }
  }
};

// A CTA whose warps wait for one another: one that gives up takes the others along.
struct Ctx {
  volatile int* abort_flag;
  int* err;
  long long spin;
};

// The whole warp waits, its lanes together, as the warp-wide instructions that
// follow want them: after a timeout too. Warps that have time to spare sleep NAP
// ns between polls and leave issue slots and the shared-memory pipe to the softmax
// warps beside them (48/8 heads of 128: 299 -> 288 us).
template <int NAP>
__device__ __forceinline__ bool wait_warp(const Ctx& c, uint64_t* bar, uint32_t parity) {
  if (__all_sync(~0u, mbar_poll(bar, parity))) return true;
  const long long t0 = clock64();
  while (true) {
    for (int i = 0; i < 8; i++) {
      if (NAP) __nanosleep(NAP);
      if (__all_sync(~0u, mbar_poll(bar, parity))) return true;
    }
    const bool late = clock64() - t0 > c.spin;
    if (late && (threadIdx.x & 31) == 0) {
      *c.abort_flag = 1;
      atomicExch(c.err, 1);
    }
    if (__any_sync(~0u, late || *c.abort_flag)) return false;
  }
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// Tokens that sequence i of a decode batch holds; 0 for a slot out of range.
__device__ __forceinline__ int seq_len(const DecodeAttnArgs& a, int i) {
  const int s = a.seqs[i];
  if (s < 0 || s >= a.slots) return 0;
  return min(max(a.lens[s], 0), (int)min((long long)a.width << a.page_shift, (long long)INT_MAX));
}
// The page table that the shared prefix is read through: the first sequence's that
// holds all of it (the first one's, where the batch is what it says), else the longest's.
__device__ __forceinline__ const int* prefix_table(const DecodeAttnArgs& a) {
  int best = 0, most = -1;
  for (int i = 0; i < a.batch && most < a.shared; i++) {
    const int len = seq_len(a, i);
    if (len > most) {
      most = len;
      best = i;
    }
  }
  const int s = a.seqs[best];
  return a.tables + (long long)(s >= 0 && s < a.slots ? s : 0) * a.width;
}

}  // namespace tfx
