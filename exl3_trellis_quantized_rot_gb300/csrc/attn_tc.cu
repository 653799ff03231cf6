// Attention on the tensor cores: tiles of 2 x 128 rows against 128 keys at a
// time, two CTAs a tile (cta_group::2).
//
// The mathematics is that of attn_warp.cu, with one difference: the reference
// of the exponents follows the running maximum only when the maximum has passed
// it by more than 2^8. Numerator and denominator share the reference, so the
// result is the same, and the accumulator is rescaled a few times a row instead
// of once a tile. Probabilities reach 2^(kShift + 8) <= 2^15.
//
// A row is a (token, head) pair: the query heads of one K/V head lie next to
// each other in a tile, so a K/V tile is read once for all of them and a short
// prompt fills more of its tile. Each CTA holds 128 of the rows (Q in shared
// memory, S, P and O in its tensor memory) and half of K and V: 64 of a tile's
// keys of K, dim/2 columns of V. The pair's MMAs (M = 256) read both halves, so
// each byte of K and V is fetched from L2 once for 256 rows, and the two SMs'
// shared memories deliver half of it each.
//
// Tensor memory (512 columns): O 0..dim-1, two score buffers of 128 columns
// from 256 on. A buffer's first 64 columns take the probabilities (two 16-bit
// values a column), the A operand of P V. Order of the MMAs, one issuing
// thread: S0, [S1, P0 V0], [S2, P1 V1], ...: S(j+1) goes to the buffer whose
// probabilities P(j-1) V(j-1) has read before it.
//
// Warps of a CTA: 0..3 softmax (thread = row) and epilogue; 4 issues the MMAs
// (in the even CTA); 5 asks for K, V and Q; 6 and 7 look after V where a tile
// has keys that some row must not see: 0 * inf and 0 * NaN are NaN, so V's rows
// past the sequence become zeros, and later tokens' values that are not finite
// too; the epilogue gives the latter to the rows that do see them.
//
// Every wait is bounded (see exl3_tc.cuh); on a timeout all roles of the CTA
// leave at their next wait, copies and MMAs in flight get time to land, and the
// pair meets at its closing barrier.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_device.cuh"
#include "attn_internal.h"

namespace tfx {
namespace {

constexpr int kThreads = 256;
constexpr int kTileKeys = 128;
constexpr float kSlack = 8.f;  // log2 by which a row's maximum may pass its reference
constexpr uint32_t kScoreCol = 256;

template <int D>
struct Geom {
  static constexpr int kStages = D == 256 ? 2 : 4;
  static constexpr int kQ = 128 * D * 2;       // bytes of Q in a CTA
  static constexpr int kKV = 64 * D * 2;       // bytes of K, or of V, of a stage in a CTA
  static constexpr size_t kSmem = (size_t)kQ + 2 * kStages * kKV + 1024;
};

struct Barriers {
  uint64_t q_full;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t v_edge[4];    // V tiles that warps 6 and 7 look at before the MMAs may
  uint64_t s_full[2];    // scores are in tensor memory
  uint64_t p_full[2];    // probabilities of both CTAs are
  uint64_t pv_done;      // P V of a tile is added
};

struct Ctx {
  Barriers* b;
  volatile int* abort_flag;
  int* err;
  long long spin;
};

__device__ __forceinline__ bool wait(const Ctx& c, uint64_t* bar, uint32_t parity) {
  if (mbar_poll_cluster(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_poll_cluster(bar, parity)) {
    if (*c.abort_flag) return false;
    if (clock64() - t0 > c.spin) {
      *c.abort_flag = 1;
      atomicExch(c.err, 1);
      return false;
    }
  }
  return true;
}

// For a whole warp: one lane waits, so that the lanes are together again for the
// warp-wide instructions that follow, after a timeout too.
__device__ __forceinline__ bool wait_warp(const Ctx& c, uint64_t* bar, uint32_t parity) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = wait(c, bar, parity);
  ok = __shfl_sync(~0u, ok, 0);
  __syncwarp();
  return ok != 0;
}

template <typename T>
struct Bits;
template <>
struct Bits<__half> {
  static constexpr uint32_t kFormat = 0, kExp = 0x7C007C00u, kOne = 0x04000400u;
};
template <>
struct Bits<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1, kExp = 0x7F807F80u, kOne = 0x00800080u;
};
// Bit 15 of each 16-bit half: the half is infinite or NaN (all exponent bits set; adding one carries into bit 15).
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & Bits<T>::kExp) + Bits<T>::kOne) & 0x80008000u;
}
template <typename T>
__device__ __forceinline__ float value_of(uint32_t w, int half);
template <>
__device__ __forceinline__ float value_of<__half>(uint32_t w, int half) {
  return __half2float(__ushort_as_half((unsigned short)(w >> (16 * half))));
}
template <>
__device__ __forceinline__ float value_of<__nv_bfloat16>(uint32_t w, int half) {
  return __uint_as_float(half ? w & 0xFFFF0000u : w << 16);
}

// kind::f16, FP32 accumulator, M = 256 over the pair, A K-major; `mn`: B's columns are its N index.
template <typename T>
__host__ __device__ constexpr uint32_t idesc(int N, bool mn) {
  return (1u << 4) | (Bits<T>::kFormat << 7) | (Bits<T>::kFormat << 10) | ((uint32_t)mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(256 >> 4) << 24);
}

// What one pair of CTAs does.
struct Item {
  int row0;        // first token row of the sequence in q, k, v, out
  int t0;          // first token of the tile within the sequence
  int end;         // tokens of the sequence
  int tiles;       // key tiles
  int edge;        // first key tile with keys that some row must not see
  int kvh, head0;  // K/V head; first query head
};

__device__ __forceinline__ Item prompt_item(const PromptArgs& a) {
  const int sub = a.group / a.per_tile, hg = a.heads_kv * sub;
  const int pair = blockIdx.x >> 1, i = pair / hg, h = pair % hg;
  // the sequences by tiles, most first; a.before[s]: tiles of the list before
  // the first s+1 sequences are all in play at tile count a.count[s]
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.before[mid] <= i) lo = mid; else hi = mid - 1;
  }
  const int r = i - a.before[lo], tile = a.count[lo] - 1 - r / (lo + 1), s = r % (lo + 1);
  Item it;
  it.row0 = a.begin[s];
  it.end = a.len[s];
  it.t0 = tile * 2 * a.tokens;
  const int last = min(it.end, it.t0 + 2 * a.tokens) - 1;
  it.tiles = last / kTileKeys + 1;
  it.edge = (it.t0 + 1) / kTileKeys;
  it.kvh = h / sub;
  it.head0 = it.kvh * a.group + h % sub * a.per_tile;
  return it;
}

template <typename T, int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) prompt_tc_kernel(const __grid_constant__ PromptArgs a) {
  using G = Geom<D>;
  constexpr int ST = G::kStages;
  extern __shared__ uint8_t dyn[];
  __shared__ Barriers bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ uint32_t fix;  // V values that were not finite were taken out of a tile
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  const uint32_t base = s_addr(dyn) + ((1024u - (s_addr(dyn) & 1023u)) & 1023u);
  const uint32_t sq = base, sk = base + G::kQ, sv = sk + ST * G::kKV;
  Ctx c = {&bars, &abort_flag, a.err, a.spin};

  if (threadIdx.x == 0) {
    abort_flag = 0;
    fix = 0;
    mbar_init(&bars.q_full, 2);
    for (int i = 0; i < 4; i++) {
      mbar_init(&bars.k_full[i], 2);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 2);
      mbar_init(&bars.v_empty[i], 1);
      mbar_init(&bars.v_edge[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 8);
    }
    mbar_init(&bars.pv_done, 1);
    fence_mbar_init();
  }
  if (warp == 4) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(s_addr(&tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  fence_after_sync();
  const uint32_t tm = *(volatile uint32_t*)&tmem_slot;
  const Item it = prompt_item(a);
  const int n = it.tiles;

  if (warp == 5) {
    // ---- copies: this CTA's rows of Q, its 64 keys of K, its dim/2 columns of V
    if (lane == 0) {
      auto lead = [&](uint64_t* bar) { return peer_addr(s_addr(bar), 0); };
      const int t = it.t0 + (int)rank * a.tokens;
      expect_tx_at(lead(&bars.q_full), a.tokens * a.per_tile * D * 2);
      for (int ch = 0; ch < D / 64; ch++)
        tma_load_5d_pair(sq + ch * 16384, &a.qmap, 0, it.head0, it.row0 + t, ch, 0, lead(&bars.q_full));
      int edges = 0;
      for (int j = 0; j < n; j++) {
        const int st = j % ST;
        const uint32_t par = ((j / ST) & 1) ^ 1;
        if (!wait(c, &bars.k_empty[st], par)) break;
        expect_tx_at(lead(&bars.k_full[st]), G::kKV);
        tma_load_5d_pair(sk + st * G::kKV, &a.k, 0, it.row0 + j * kTileKeys + 64 * (int)rank, 0, it.kvh, 0,
                         lead(&bars.k_full[st]));
        if (!wait(c, &bars.v_empty[st], par)) break;
        uint32_t bar = lead(&bars.v_full[st]);
        if (j >= it.edge) {
          bar = s_addr(&bars.v_edge[edges++ % 4]);
          bar = peer_addr(bar, rank);
        }
        expect_tx_at(bar, G::kKV);
        tma_load_5d_pair(sv + st * G::kKV, &a.v, 0, it.row0 + j * kTileKeys, (int)rank * (D / 128), it.kvh, 0, bar);
      }
    }
  } else if (warp == 4) {
    // ---- MMAs
    if (rank == 0 && lane == 0) {
      constexpr uint32_t is = idesc<T>(kTileKeys, false), ip = idesc<T>(D, true);
      constexpr uint64_t kmaj = operand_bits(16), vmaj = operand_bits(kTileKeys * 128);
      auto scores = [&](int j) -> bool {
        const int st = j % ST;
        if (!wait(c, &bars.k_full[st], (j / ST) & 1)) return false;
        fence_after_sync();
        const uint64_t qd = operand(sq, kmaj), kd = operand(sk + st * G::kKV, kmaj);
        const uint32_t d = tm + kScoreCol + (j & 1) * 128;
#pragma unroll
        for (int k = 0; k < D / 16; k++)
          mma2_ss(d, qd + (((k >> 2) * 16384 + (k & 3) * 32) >> 4), kd + (((k >> 2) * 8192 + (k & 3) * 32) >> 4), is, k > 0);
        commit2(&bars.s_full[j & 1]);
        commit2(&bars.k_empty[st]);
        return true;
      };
      bool ok = wait(c, &bars.q_full, 0) && scores(0);
      for (int j = 0; ok && j < n; j++) {
        if (j + 1 < n && !scores(j + 1)) break;
        const int st = j % ST;
        if (!wait(c, &bars.v_full[st], (j / ST) & 1)) break;
        if (!wait(c, &bars.p_full[j & 1], (j >> 1) & 1)) break;
        fence_after_sync();
        const uint64_t vd = operand(sv + st * G::kKV, vmaj);
        const uint32_t p = tm + kScoreCol + (j & 1) * 128;
#pragma unroll
        for (int k = 0; k < kTileKeys / 16; k++) mma2_ts(tm, p + k * 8, vd + ((k * 2048) >> 4), ip, j > 0 || k > 0);
        commit2(&bars.v_empty[st]);
        commit2(&bars.pv_done);
      }
    }
  } else if (warp >= 6) {
    // ---- V tiles with keys that some row must not see
    int edges = 0;
    for (int j = it.edge; j < n; j++, edges++) {
      const int st = j % ST;
      // both warps meet at the barrier below for every tile, also after a timeout;
      // then nothing is handed on: v_full may still be in an earlier tile's
      // phase, which takes that tile's two arrivals and no more
      const bool ok = wait_warp(c, &bars.v_edge[edges % 4], (edges / 4) & 1);
      const int from = max(it.t0 + 1 - j * kTileKeys, 0);
      constexpr int kPieces = D / 16;  // 16-byte pieces of a row in this CTA
      bool found = false;
      for (int x = threadIdx.x - 192; ok && x < (kTileKeys - from) * kPieces; x += 64) {
        const int r = from + x / kPieces, p = x % kPieces;
        const uint32_t at = sv + st * G::kKV + (p >> 3) * (kTileKeys * 128) + r * 128 + (p & 7) * 16;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (j * kTileKeys + r < it.end) {
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at));
          const uint32_t m[4] = {not_finite<T>(w.x), not_finite<T>(w.y), not_finite<T>(w.z), not_finite<T>(w.w)};
          if (!(m[0] | m[1] | m[2] | m[3])) continue;
          found = true;
          // 0xFFFF where bit 15 of the half is set
          w.x &= ~((m[0] >> 15) * 0xFFFFu);
          w.y &= ~((m[1] >> 15) * 0xFFFFu);
          w.z &= ~((m[2] >> 15) * 0xFFFFu);
          w.w &= ~((m[3] >> 15) * 0xFFFFu);
        }
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
      }
      if (found) {
        store_at(peer_addr(s_addr(&fix), 0), 1);
        store_at(peer_addr(s_addr(&fix), 1), 1);
      }
      fence_async_smem();
      asm volatile("bar.sync 1, 64;" ::: "memory");
      if (threadIdx.x == 192 && ok && !*c.abort_flag) arrive_at(peer_addr(s_addr(&bars.v_full[st]), 0));
    }
  } else {
    // ---- softmax: thread = row
    const int row = threadIdx.x;
    const int tok = it.t0 + (int)rank * a.tokens + row / a.per_tile;
    const bool live = row < a.tokens * a.per_tile && tok < it.end;
    const int hi = live ? tok + 1 : 0;  // keys the row sees
    const uint32_t tw = tm + ((uint32_t)warp << 21);
    const float cs = a.scale_log2;
    float ref = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; j++) {
      if (!(ok = wait_warp(c, &bars.s_full[j & 1], (j >> 1) & 1))) break;
      fence_after_sync();
      const uint32_t ts = tw + kScoreCol + (j & 1) * 128;
      float s[128];
#pragma unroll
      for (int i = 0; i < 4; i++) tmem_ld32(ts + 32 * i, s + 32 * i);
      tmem_wait_ld_();
      const int left = hi - j * kTileKeys;
      if (left < kTileKeys) {
#pragma unroll
        for (int i = 0; i < 128; i++)
          if (i >= left) s[i] = -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int i = 4; i < 128; i++) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
      const float want = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs - Exponent<T>::kShift;
      const bool move = want > ref + kSlack;  // never for a row that sees nothing; always for its first keys
      if (__any_sync(~0u, move)) {
        const float f = move ? exp2_fast(ref - want) : 1.f;
        if (move) ref = want;
        l *= f;
        if (j > 0) {
          if (!(ok = wait_warp(c, &bars.pv_done, (j - 1) & 1))) break;
          fence_after_sync();
          const uint64_t ff = pair_of(f, f);
#pragma unroll 1
          for (int i = 0; i < D; i += 32) {
            float o[32];
            tmem_ld32(tw + i, o);
            tmem_wait_ld_();
            uint32_t u[32];
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float x, y;
              parts_of(mul2(pair_of(o[k], o[k + 1]), ff), x, y);
              u[k] = __float_as_uint(x);
              u[k + 1] = __float_as_uint(y);
            }
            tmem_st32(tw + i, u);
          }
        }
      }
      const float off = ref == -INFINITY ? 0.f : -ref;
      const uint64_t c2 = pair_of(cs, cs), o2 = pair_of(off, off);
      uint64_t sum2[2] = {0, 0};
#pragma unroll
      for (int h = 0; h < 2; h++) {
        uint32_t p[32];
#pragma unroll
        for (int i = 0; i < 32; i++) {
          float x, y;
          parts_of(fma2(pair_of(s[h * 64 + 2 * i], s[h * 64 + 2 * i + 1]), c2, o2), x, y);
          x = exp2_fast(x);
          y = exp2_fast(y);
          sum2[i & 1] = add2(sum2[i & 1], pair_of(x, y));
          p[i] = pack2<T>(x, y);  // matrix operands of the inputs' type; their sum stays FP32
        }
        tmem_st32(ts + h * 32, p);
      }
      tmem_wait_st_();
      fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_at(peer_addr(s_addr(&bars.p_full[j & 1]), 0));
      float x, y;
      parts_of(add2(sum2[0], sum2[1]), x, y);
      l += x + y;
    }
    // the last two: a parity says nothing of a phase that has yet to begin
    if (ok && (n < 2 || wait_warp(c, &bars.pv_done, (n - 2) & 1)) && wait_warp(c, &bars.pv_done, (n - 1) & 1)) {
      fence_after_sync();
      const float inv = 1.f / l;
      const bool mend = *(volatile uint32_t*)&fix != 0;
      T* out = reinterpret_cast<T*>(a.out) + (it.row0 + (long long)tok) * a.ldo + (long long)(it.head0 + row % a.per_tile) * D;
      const T* v = reinterpret_cast<const T*>(a.vbase) + (long long)it.row0 * a.ldv + (long long)it.kvh * D;
#pragma unroll 1
      for (int i = 0; i < D; i += 32) {
        float o[32];
        tmem_ld32(tw + i, o);
        tmem_wait_ld_();
        if (live) {
          if (mend)
            for (int key = it.t0 + 1; key < hi; key++) {
              const uint32_t* w = reinterpret_cast<const uint32_t*>(v + (long long)key * a.ldv + i);
  #pragma unroll
              for (int k = 0; k < 16; k++) {
                const uint32_t x = w[k], m = not_finite<T>(x);
                if (m & 0x8000u) o[2 * k] += value_of<T>(x, 0);
                if (m & 0x80000000u) o[2 * k + 1] += value_of<T>(x, 1);
              }
            }
  #pragma unroll
          for (int k = 0; k < 4; k++) {
            uint4 w;
            w.x = pack2<T>(o[8 * k] * inv, o[8 * k + 1] * inv);
            w.y = pack2<T>(o[8 * k + 2] * inv, o[8 * k + 3] * inv);
            w.z = pack2<T>(o[8 * k + 4] * inv, o[8 * k + 5] * inv);
            w.w = pack2<T>(o[8 * k + 6] * inv, o[8 * k + 7] * inv);
            *reinterpret_cast<uint4*>(out + i + 8 * k) = w;
          }
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  if (*c.abort_flag) {
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) {
    }
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();
  if (warp == 4) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  }
}

template <typename T, int D>
int prompt_of(const PromptArgs& a, int pairs, cudaStream_t s) {
  const void* fn = (const void*)prompt_tc_kernel<T, D>;
  const int rc = opt_in_smem(fn, Geom<D>::kSmem);
  if (rc) return rc;
  return launch_kernel(fn, dim3(2u * (unsigned)pairs), dim3(kThreads), Geom<D>::kSmem, s, const_cast<PromptArgs*>(&a), false, 1);
}

}  // namespace

int launch_prompt(const PromptArgs& a, int act, int dim, int pairs, cudaStream_t s) {
  if (act == TFX_F16) return dim == 128 ? prompt_of<__half, 128>(a, pairs, s) : prompt_of<__half, 256>(a, pairs, s);
  return dim == 128 ? prompt_of<__nv_bfloat16, 128>(a, pairs, s) : prompt_of<__nv_bfloat16, 256>(a, pairs, s);
}

}  // namespace tfx
