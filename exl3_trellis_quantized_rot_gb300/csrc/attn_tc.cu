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
// Tensor memory (512 columns): O in 0..dim-1, then B score buffers of 128 columns,
// two at dim 256, three at 128. A buffer's first 64 columns take the probabilities
// (two 16-bit values a column), the A operand of P V. Order of the MMAs, from one
// warp: S0 .. S(B-1), P0 V0, SB, P1 V1, S(B+1), ...: S(j+B) goes to the buffer whose
// probabilities P(j) V(j) has read before it.
//
// What bounds it (GB300): at dim 256 the tensor pipe, 2,063 cycles a tile of 256
// rows x 128 keys against the MMAs' 2,048 (16,384 tokens of 24/4 heads: 1.82 ms on the
// GPU, 1.88 as a call among others, 1,810 and 1,755 TFLOP/s). At dim 128 two chains of nearly one length: the softmax, about 1,425
// cycles a tile (its exponentials take 800, where the unit's rate allows 512; the rest is
// the way from scores to maximum and back, which two warps of a scheduler walk together),
// and the MMAs, about 1,300 where their rate allows 1,024. With either one's work halved
// the other still takes nearly the whole time. Tried there and slower: four warps of 32
// columns a row, two warps taking turns at whole tiles, two sets of warps taking turns.
// Between two items about 5,000 cycles at dim 256: the last product 900, the store of 64
// KB beside the next item's copies 3,500, the first softmax 1,700.
//
// Warps of a CTA: 0..7 softmax and results; 8 issues the MMAs (in the even CTA);
// 9 asks for K and Q, 10 for V; 11 looks after V where a tile has keys that some
// row must not see: 0 * inf and 0 * NaN are NaN, so V's rows past the sequence
// become zeros, and later tokens' values that are not finite too; the rows that
// do see the latter get them when the result is stored.
//
// A pair walks its items (a tile of rows and its key tiles) without a stop: K, V
// and the next Q are asked for as soon as their memory is free, and the next
// item's first scores are computed while the last one's result is stored.
//
// Every wait is bounded (see exl3_tc.cuh); on a timeout all roles of the CTA
// leave at their next wait, copies and MMAs in flight get time to land, and the
// pair meets at its closing barrier.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "attn_device.cuh"
#include "attn_internal.h"

namespace tfx {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8, kKWarp = 9, kVWarp = 10, kEdgeWarp = 11;  // 0..7 softmax
constexpr int kTileKeys = 128;
constexpr float kSlack = 8.f;  // log2 by which a row's maximum may pass its reference
constexpr int kEdgeBars = 4, kFixes = 8;

template <int D>
struct Geom {
  static constexpr int kStages = D == 256 ? 2 : 4;
  static constexpr int kScores = D == 256 ? 2 : 3;  // score buffers: what O leaves of the 512 columns, at most 3
  static constexpr int kQ = 128 * D * 2;       // bytes of Q in a CTA
  static constexpr int kKV = 64 * D * 2;       // bytes of K, or of V, of a stage in a CTA
  static constexpr size_t kSmem = (size_t)kQ + 2 * kStages * kKV + 1024;
};

struct Barriers {
  uint64_t q_full, q_empty;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t v_edge[kEdgeBars];  // V tiles that warp 11 looks at before the MMAs may
  uint64_t s_full[3];          // scores are in tensor memory
  uint64_t p_full[3];          // probabilities of both CTAs are
  // P V of a tile is added. One a score buffer, like the two above: a parity tells
  // two phases apart, and a tile's scores come after the addition SB tiles before.
  uint64_t pv_done[3];
  uint64_t o_empty;            // both CTAs have read an item's result
};

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

struct Ctx {
  Barriers* b;
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

// The two warps that share rows meet at their named barrier.
__device__ __forceinline__ void bar_meet(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
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
__device__ __forceinline__ uint4 ld_shared16(uint32_t at) {
  uint4 w;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
  return w;
}
__device__ __forceinline__ void st_shared16(uint32_t at, uint4 w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}
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

// 256 rows against some key tiles. The rows are those of `per_tile` heads of
// 2 * tokens consecutive "tokens": of a prompt, or, for the shared prefix of a
// decode batch, the batch's sequences (one token each).
struct Item {
  int row0;        // row of q of the tile's first token
  int end_row;     // tokens of the tile before this one exist
  int key_row;     // row of key 0 in k and v (prompt)
  int t0;          // position of the first token in its sequence (prompt)
  int first;       // first key tile
  int tiles;       // key tiles
  int seen;        // keys from here on are seen by no row
  int hidden;      // first key that some row must not see
  int kvh, head0;  // K/V head; first query head
  int split;       // which share of the prefix
};

__device__ __forceinline__ Item item_of(const PromptArgs& a, int x) {
  const int i = x / a.hg, h = x - i * a.hg, sub = a.sub;
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.before[mid] <= i) lo = mid; else hi = mid - 1;
  }
  const int r = i - a.before[lo], tile = a.count[lo] - 1 - r / (lo + 1), s = r % (lo + 1);
  Item it;
  it.key_row = a.begin[s];
  it.t0 = tile * 2 * a.tokens;
  it.row0 = it.key_row + it.t0;
  it.end_row = it.key_row + a.len[s];
  it.first = 0;
  it.seen = min(a.len[s], it.t0 + 2 * a.tokens);
  it.tiles = (it.seen - 1) / kTileKeys + 1;
  it.hidden = it.t0 + 1;
  it.kvh = h / sub;
  it.head0 = it.kvh * a.group + h % sub * a.per_tile;
  it.split = 0;
  return it;
}

__device__ __forceinline__ Item item_of(const DecodeAttnArgs& a, int x) {
  const int y = x / a.hg, h = x - y * a.hg, sub = a.sub;
  const unsigned all = (unsigned)(a.shared + kTileKeys - 1) / kTileKeys, splits = (unsigned)a.pre_splits;
  Item it;
  it.split = y / a.mt;
  it.row0 = (y - it.split * a.mt) * 2 * a.tokens;
  it.end_row = a.batch;
  it.key_row = it.t0 = 0;
  // the tiles evenly: the first all % splits shares have one more
  const unsigned each = all / splits, more = all - each * splits, n = (unsigned)it.split;
  it.first = (int)(each * n + min(n, more));
  it.tiles = (int)(each + (n < more));
  it.seen = it.hidden = a.shared;
  it.kvh = h / sub;
  it.head0 = it.kvh * a.group + h % sub * a.per_tile;
  return it;
}

// The x-th item of a pair of CTAs, or -1: rounds over the pairs, to and fro, so
// that the sizes (most keys first) even out.
template <typename A>
__device__ __forceinline__ int nth(const A& a, int r) {
  const int pairs = gridDim.x >> 1, p = blockIdx.x >> 1;
  const long long x = (long long)r * pairs + (r & 1 ? pairs - 1 - p : p);
  return x < a.items ? (int)x : -1;
}

// Keys that row `tok` (a token of the tile) sees.
__device__ __forceinline__ int sees(const PromptArgs&, const Item& it, int tok) { return it.t0 + tok + 1; }
__device__ __forceinline__ int sees(const DecodeAttnArgs& a, const Item& it, int tok) {
  return min(a.shared, seq_len(a, it.row0 + tok));
}

// The copies of K's 64 keys and V's 128 keys of a tile, by a warp. Each lane holds
// the page of one block of 16 keys: four tiles' blocks at a time, and the next
// four's are on their way.
struct Pages {
  const int* table;  // the shared prefix's
  int tile;          // first of the four
  int page, next;
};
__device__ __forceinline__ void look_up(const PromptArgs&, Pages&, int, int) {}
__device__ __forceinline__ int page_ahead(const DecodeAttnArgs& a, const Pages& pg, int tile, int lane) {
  const int p = (tile * kTileKeys + lane * 16) >> a.page_shift;
  return p < a.width ? __ldg(pg.table + p) : -1;
}
// Makes the window hold `tile`: called for each tile in order, and at an item's first.
__device__ __forceinline__ void look_up(const DecodeAttnArgs& a, Pages& pg, int tile, int lane) {
  if (tile == pg.tile + 4) {
    pg.page = pg.next;
  } else if (tile < pg.tile || tile > pg.tile + 4) {
    pg.page = page_ahead(a, pg, tile, lane);
  } else {
    return;
  }
  pg.tile = tile;
  pg.next = page_ahead(a, pg, tile + 4, lane);
}
__device__ __forceinline__ void first_pages(const PromptArgs&, Pages&, int, int) {}
__device__ __forceinline__ void first_pages(const DecodeAttnArgs& a, Pages& pg, int tile, int lane) {
  // the first sequence's, asked for beside its length; another's if that says so
  const int s = a.seqs[0];
  pg.table = a.tables + (long long)((unsigned)s < (unsigned)a.slots ? s : 0) * a.width;
  pg.page = page_ahead(a, pg, tile, lane);
  pg.next = page_ahead(a, pg, tile + 4, lane);
  if (seq_len(a, 0) < a.shared) {
    pg.table = prefix_table(a);
    pg.page = page_ahead(a, pg, tile, lane);
    pg.next = page_ahead(a, pg, tile + 4, lane);
  }
  pg.tile = tile;
}
template <int D>
__device__ __forceinline__ void copy_k(const PromptArgs& a, const Item& it, const Pages&, int j, int rank, uint32_t dst,
                                       uint32_t bar, int lane) {
  if (lane == 0) tma_load_5d_pair(dst, &a.k, 0, it.key_row + j * kTileKeys + 64 * rank, 0, it.kvh, 0, bar);
}
template <int D>
__device__ __forceinline__ void copy_v(const PromptArgs& a, const Item& it, const Pages&, int j, int rank, uint32_t dst,
                                       uint32_t bar, int lane) {
  if (lane == 0) tma_load_5d_pair(dst, &a.v, 0, it.key_row + j * kTileKeys, rank * (D / 128), it.kvh, 0, bar);
}
// Pages: boxes of up to 64 tokens of one page and one column block of 64 values;
// a page out of range becomes -1, out of the map's range: zeros.
template <int D>
__device__ __forceinline__ void copy_k(const DecodeAttnArgs& a, const Item& it, const Pages& pg, int j, int rank, uint32_t dst,
                                       uint32_t bar, int lane) {
  const int shift = min(a.page_shift, 6), key0 = (it.first + j) * kTileKeys;
  const int page = (unsigned)pg.page < (unsigned)a.pages ? pg.page : -1;
#pragma unroll
  for (int x0 = 0; x0 < 4 * (D / 64); x0 += 32) {
    const int x = x0 + lane, b = x / (D / 64), ch = x % (D / 64), key = 64 * rank + (b << shift);
    const int pid = __shfl_sync(~0u, page, (it.first + j - pg.tile) * 8 + ((key >> 4) & 7));
    if (x < (64 >> shift) * (D / 64))
      tma_load_5d_pair(dst + ch * 8192 + (b << shift) * 128, &a.kt, 0, (key0 + key) & (a.page_size - 1), ch, it.kvh, pid, bar);
  }
}
template <int D>
__device__ __forceinline__ void copy_v(const DecodeAttnArgs& a, const Item& it, const Pages& pg, int j, int rank, uint32_t dst,
                                       uint32_t bar, int lane) {
  const int shift = min(a.page_shift, 6), key0 = (it.first + j) * kTileKeys;
  const int page = (unsigned)pg.page < (unsigned)a.pages ? pg.page : -1;
#pragma unroll
  for (int x0 = 0; x0 < 8 * (D / 128); x0 += 32) {
    const int x = x0 + lane, b = x / (D / 128), ch = x % (D / 128), key = b << shift;
    const int pid = __shfl_sync(~0u, page, (it.first + j - pg.tile) * 8 + ((key >> 4) & 7));
    if (x < (128 >> shift) * (D / 128))
      tma_load_5d_pair(dst + ch * 16384 + (b << shift) * 128, &a.vt, 0, (key0 + key) & (a.page_size - 1), rank * (D / 128) + ch,
                       it.kvh, pid, bar);
  }
}

// N columns of a row's result, from column `col` on: o is the accumulator's, inv = 1
// / sum. All lanes call it. 32 columns at a time go through shared memory, so that
// neighbouring lanes store neighbouring pieces of a row: as 16 bytes of 32 rows an
// instruction they took longer.
template <typename T, int D, int N>
__device__ __forceinline__ void store_row(const PromptArgs& a, const Item& it, int tok, int head, int col, float (&o)[N],
                                          float inv, bool live, bool mend, uint4* stage) {
  if (mend && live) {  // values that were taken out of V: this row's own
    const T* v = reinterpret_cast<const T*>(a.vbase) + (long long)it.key_row * a.ldv + (long long)it.kvh * D + col;
    for (int key = it.hidden; key <= it.t0 + tok; key++) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(v + (long long)key * a.ldv);
#pragma unroll
      for (int k = 0; k < N / 2; k++) {
        const uint32_t x = w[k], m = not_finite<T>(x);
        if (m & 0x8000u) o[2 * k] += value_of<T>(x, 0);
        if (m & 0x80000000u) o[2 * k + 1] += value_of<T>(x, 1);
      }
    }
  }
  const int lane = threadIdx.x & 31, p = lane & 3;
  T* out = live ? reinterpret_cast<T*>(a.out) + (long long)(it.row0 + tok) * a.ldo + (long long)head * D + col : nullptr;
  T* to[4];  // the rows that this lane stores a piece of: four lanes a row's 64 bytes
#pragma unroll
  for (int k = 0; k < 4; k++)
    to[k] = reinterpret_cast<T*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(out), k * 8 + (lane >> 2)));
#pragma unroll
  for (int c = 0; c < N; c += 32) {
#pragma unroll
    for (int k = 0; k < 4; k++) {  // 8 lanes' pieces in 8 different columns of banks
      const float* x = o + c + 8 * k;
      stage[lane * 4 + (k ^ ((lane >> 1) & 3))] = make_uint4(pack2<T>(x[0] * inv, x[1] * inv), pack2<T>(x[2] * inv, x[3] * inv),
                                                             pack2<T>(x[4] * inv, x[5] * inv), pack2<T>(x[6] * inv, x[7] * inv));
    }
    __syncwarp();
    uint4 w[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const int r = k * 8 + (lane >> 2);
      w[k] = stage[r * 4 + (p ^ ((r >> 1) & 3))];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; k++)
      if (to[k]) *reinterpret_cast<uint4*>(to[k] + c + p * 8) = w[k];
  }
}
// A share of the prefix: the sums as they are, 16 rows at a time, eight lanes a row's 128 bytes.
template <typename T, int D, int N>
__device__ __forceinline__ void store_row(const DecodeAttnArgs& a, const Item& it, int tok, int head, int col, float (&o)[N],
                                          float, bool live, bool, uint4* stage) {
  const int lane = threadIdx.x & 31, p = lane & 7;
  float* po = live ? a.pre_o + (((long long)it.split * a.batch + it.row0 + tok) * a.heads_q + head) * D + col : nullptr;
  float* to[8];
#pragma unroll
  for (int k = 0; k < 8; k++)
    to[k] = reinterpret_cast<float*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(po), k * 4 + (lane >> 3)));
#pragma unroll
  for (int c = 0; c < N; c += 32)
#pragma unroll
    for (int h = 0; h < 2; h++) {
      if ((lane >> 4) == h)
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const float* x = o + c + 4 * k;
          stage[(lane & 15) * 8 + (k ^ (lane & 7))] =
              make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        }
      __syncwarp();
      uint4 w[4];
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const int r = k * 4 + (lane >> 3);
        w[k] = stage[r * 8 + (p ^ (r & 7))];
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; k++)
        if (to[h * 4 + k]) *reinterpret_cast<uint4*>(to[h * 4 + k] + c + p * 4) = w[k];
    }
}
__device__ __forceinline__ void store_sum(const PromptArgs&, const Item&, int, int, float, float) {}
__device__ __forceinline__ void store_sum(const DecodeAttnArgs& a, const Item& it, int tok, int head, float ref, float l) {
  a.pre_ml[((long long)it.split * a.batch + it.row0 + tok) * a.heads_q + head] = make_float2(ref, l);
}

template <typename T, int D, typename A>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ A a) {
  using G = Geom<D>;
  constexpr int ST = G::kStages, SB = G::kScores;
  extern __shared__ uint8_t dyn[];
  __shared__ Barriers bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int walked[2];    // tiles and items of this pair
  __shared__ int fix[kFixes];  // round + 1 of the item whose V had values that were not finite taken out
  __shared__ float shared_max[2][2][128], shared_sum[2][128];
  __shared__ uint4 stage[8][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  const uint32_t base = s_addr(dyn) + ((1024u - (s_addr(dyn) & 1023u)) & 1023u);
  const uint32_t sq = base, sk = base + G::kQ, sv = sk + ST * G::kKV;
  Ctx c = {&bars, &abort_flag, a.err, a.spin};

  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bars.q_full, 2);
    mbar_init(&bars.q_empty, 1);
    for (int i = 0; i < 4; i++) {
      mbar_init(&bars.k_full[i], 2);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 2);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int i = 0; i < kEdgeBars; i++) mbar_init(&bars.v_edge[i], 1);
    for (int i = 0; i < kFixes; i++) fix[i] = 0;
    for (int i = 0; i < 3; i++) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 16);
      mbar_init(&bars.pv_done[i], 1);
    }
    mbar_init(&bars.o_empty, 16);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(s_addr(&tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  // the first pages are looked up while the pair comes together
  Pages pg = {};
  const int x0 = nth(a, 0);
  Item it0 = {};
  if (x0 >= 0) it0 = item_of(a, x0);
  if ((warp == kKWarp || warp == kVWarp) && x0 >= 0) {
    griddep_wait();
    first_pages(a, pg, it0.first, lane);
  }
  // rows of Q that no copy writes
  for (int x = a.tokens * a.per_tile * 8 + threadIdx.x; x < 128 * 8; x += kThreads)
    for (int ch = 0; ch < D / 64; ch++)
      asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(sq + ch * 16384 + x * 16), "r"(0u) : "memory");
  fence_async_smem();
  fence_before_sync();
  __syncthreads();
  pair_sync();
  fence_after_sync();
  const uint32_t tm = *(volatile uint32_t*)&tmem_slot;
  griddep_wait();
  griddep_launch();  // what follows waits for this grid before it reads what it wrote
  // registers: 384 x 168 at launch; 256 x 208 + 128 x 80 = 63,488 of those 64,512 from here on
  if (warp >= kMmaWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");

  auto lead = [&](uint64_t* bar) { return peer_addr(s_addr(bar), 0); };
  if (warp == kKWarp) {
    // ---- copies: this CTA's 64 keys of K and its rows of Q; an item's first K
    // need not wait until the last one's Q has been read
    Turn<ST> t;
    bool ok = true;
    for (int r = 0, x; ok && (x = nth(a, r)) >= 0; r++) {
      const Item it = r ? item_of(a, x) : it0;
      for (int j = 0; ok && j < it.tiles; j++) {
        look_up(a, pg, it.first + j, lane);
        if (!(ok = wait_warp<30>(c, &bars.k_empty[t.i], t.parity ^ 1))) break;
        const uint32_t bar = lead(&bars.k_full[t.i]);
        if (lane == 0) expect_tx_at(bar, G::kKV);
        __syncwarp();
        copy_k<D>(a, it, pg, j, (int)rank, sk + t.i * G::kKV, bar, lane);
        t.next();
        if (j > 0) continue;
        if (!(ok = wait_warp<30>(c, &bars.q_empty, (r & 1) ^ 1))) break;
        if (lane == 0) {
          expect_tx_at(lead(&bars.q_full), a.tokens * a.per_tile * D * 2);
          for (int ch = 0; ch < D / 64; ch++)
            tma_load_5d_pair(sq + ch * 16384, &a.qmap, 0, it.head0, it.row0 + (int)rank * a.tokens, ch, 0, lead(&bars.q_full));
        }
        __syncwarp();
      }
    }
  } else if (warp == kVWarp) {
    // ---- copies: its dim/2 columns of V
    Turn<ST> t;
    int edges = 0;
    bool ok = true;
    for (int r = 0, x; ok && (x = nth(a, r)) >= 0; r++) {
      const Item it = r ? item_of(a, x) : it0;
      for (int j = 0; j < it.tiles; j++, t.next()) {
        look_up(a, pg, it.first + j, lane);
        if (!(ok = wait_warp<30>(c, &bars.v_empty[t.i], t.parity ^ 1))) break;
        const bool edge = (it.first + j + 1) * kTileKeys > it.hidden;
        const uint32_t bar = edge ? peer_addr(s_addr(&bars.v_edge[edges % kEdgeBars]), rank) : lead(&bars.v_full[t.i]);
        edges += edge;
        if (lane == 0) expect_tx_at(bar, G::kKV);
        __syncwarp();
        copy_v<D>(a, it, pg, j, (int)rank, sv + t.i * G::kKV, bar, lane);
      }
    }
  } else if (warp == kMmaWarp) {
    // ---- MMAs
    if (rank == 0) {
      constexpr uint32_t is = idesc<T>(kTileKeys, false), ip = idesc<T>(D, true);
      constexpr uint64_t kmaj = operand_bits(16), vmaj = operand_bits(kTileKeys * 128);
      const uint64_t qd = operand(sq, kmaj), kd0 = operand(sk, kmaj), vd0 = operand(sv, vmaj);
      Turn<ST> kt, vt;  // K and V stages
      Turn<SB> st, pt;  // score buffers, of the scores and of the products with V
      bool ok = true;
      auto scores = [&](bool last) -> bool {
        if (!wait_warp<10>(c, &bars.k_full[kt.i], kt.parity)) return false;
        fence_after_sync();
        const uint64_t kd = kd0 + kt.i * (G::kKV >> 4);
        const uint32_t d = tm + D + st.i * 128;
        if (elected()) {
#pragma unroll
          for (int k = 0; k < D / 16; k++)
            mma2_ss(d, qd + (((k >> 2) * 16384 + (k & 3) * 32) >> 4), kd + (((k >> 2) * 8192 + (k & 3) * 32) >> 4), is, k > 0);
          commit2(&bars.s_full[st.i]);
          commit2(&bars.k_empty[kt.i]);
          if (last) commit2(&bars.q_empty);
        }
        __syncwarp();
        kt.next();
        st.next();
        return true;
      };
      for (int r = 0, x; ok && (x = nth(a, r)) >= 0; r++) {
        const Item it = r ? item_of(a, x) : it0;
        const int n = it.tiles, last_steps = (min(it.seen - (it.first + n - 1) * kTileKeys, kTileKeys) + 15) >> 4;
        if (!(ok = wait_warp<10>(c, &bars.q_full, r & 1))) break;
        int ahead = 0;  // scores of the item's tiles issued: up to SB - 1 more than the products with V
        for (int j = 0; j < n; j++) {
          for (; ok && ahead < n && ahead < j + SB; ahead++) ok = scores(ahead + 1 == n);
          if (!ok || !(ok = wait_warp<10>(c, &bars.p_full[pt.i], pt.parity) && wait_warp<10>(c, &bars.v_full[vt.i], vt.parity))) break;
          if (j == 0 && r > 0 && !(ok = wait_warp<10>(c, &bars.o_empty, (r - 1) & 1))) break;
          fence_after_sync();
          const uint64_t vd = vd0 + vt.i * (G::kKV >> 4);
          const uint32_t p = tm + D + pt.i * 128;
          if (elected()) {
            const int steps = j + 1 < n ? kTileKeys / 16 : last_steps;
#pragma unroll
            for (int k = 0; k < kTileKeys / 16; k++)
              if (k < steps) mma2_ts(tm, p + k * 8, vd + ((k * 2048) >> 4), ip, j > 0 || k > 0);
            commit2(&bars.v_empty[vt.i]);
            commit2(&bars.pv_done[pt.i]);
          }
          __syncwarp();
          vt.next();
          pt.next();
        }
      }
    }
  } else if (warp == kEdgeWarp) {
    // ---- V tiles with keys that some row must not see
    Turn<ST> t;
    int edges = 0, tiles = 0, r = 0;
    bool ok = true;
    for (int x; (x = nth(a, r)) >= 0; r++) {
      const Item it = r ? item_of(a, x) : it0;
      tiles += it.tiles;
      for (int j = 0; j < it.tiles; j++, t.next()) {
        const int key0 = (it.first + j) * kTileKeys;
        if (key0 + kTileKeys <= it.hidden) continue;
        const int st = t.i;
        // after a timeout nothing is handed on: v_full may still be in an earlier
        // tile's phase, which takes that tile's two arrivals and no more
        ok = ok && wait_warp<100>(c, &bars.v_edge[edges % kEdgeBars], (edges / kEdgeBars) & 1);
        edges++;
        const int from = max(it.hidden - key0, 0), end = min(it.seen - key0, kTileKeys);
        const int till = min((it.seen - key0 + 15) & ~15, kTileKeys);  // the product takes 16 keys at a time, and no more
        // A lane looks at one 16-byte piece of every kRows-th row (which of a row's, the
        // swizzle decides), eight loads at a time, and only a piece that has something to
        // mend goes round again: mended as they were read, four at a time, they took up to
        // 3,000 cycles longer than the softmax of the item's last tile, and the product
        // waited for them (eight prompts of 1 to 2,049 tokens: 61.5 -> 57.9 us).
        constexpr int kPieces = D / 16, kRows = 32 / kPieces;
        const int r0 = lane / kPieces, piece = lane % kPieces;
        const uint32_t at = sv + st * G::kKV + (piece >> 3) * (kTileKeys * 128) + (piece & 7) * 16;
        uint32_t bad = 0;
        for (int r1 = from + r0; ok && r1 < end; r1 += 8 * kRows) {
          uint4 w[8];
#pragma unroll
          for (int k = 0; k < 8; k++)
            w[k] = r1 + k * kRows < end ? ld_shared16(at + (r1 + k * kRows) * 128) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int k = 0; k < 8; k++)
            bad |= not_finite<T>(w[k].x) | not_finite<T>(w[k].y) | not_finite<T>(w[k].z) | not_finite<T>(w[k].w);
        }
        for (int x = end + r0; ok && x < till; x += kRows) st_shared16(at + x * 128, make_uint4(0, 0, 0, 0));
        if (bad) {
          for (int x = from + r0; x < end; x += kRows) {
            uint4 w = ld_shared16(at + x * 128);
            // 0xFFFF where bit 15 of the half is set
            w.x &= ~((not_finite<T>(w.x) >> 15) * 0xFFFFu);
            w.y &= ~((not_finite<T>(w.y) >> 15) * 0xFFFFu);
            w.z &= ~((not_finite<T>(w.z) >> 15) * 0xFFFFu);
            w.w &= ~((not_finite<T>(w.w) >> 15) * 0xFFFFu);
            st_shared16(at + x * 128, w);
          }
          store_at(peer_addr(s_addr(&fix[r % kFixes]), 0), r + 1);
          store_at(peer_addr(s_addr(&fix[r % kFixes]), 1), r + 1);
          asm volatile("fence.acq_rel.cluster;" ::: "memory");
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && ok) arrive_at(peer_addr(s_addr(&bars.v_full[st]), 0));
      }
    }
    if (lane == 0) {
      walked[0] = tiles;
      walked[1] = r;
    }
  } else {
    // ---- softmax: warps w and w + 4 share 32 rows (thread = row), and halve their
    // columns. A wait that gave up changes only what is handed on: the two warps
    // go on meeting at their barrier.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int q4 = warp & 3, half = warp >> 2, row = q4 * 32 + lane;
    const uint32_t tw = tm + ((uint32_t)q4 << 21);
    const float cs = a.scale_log2;
    const int my_tok = row / a.per_tile, my_head = row % a.per_tile;
    Turn<SB> t, before;  // this tile's score buffer, and the one before it
    int even = 0;
    const uint32_t p_full = peer_addr(s_addr(&bars.p_full[0]), 0);
    bool ok = true;
    const int tok = (int)rank * a.tokens + my_tok;
    int x = x0;
    Item it = it0, next = {};
    for (int r = 0; x >= 0; r++, it = next) {
      const bool live = my_tok < a.tokens && it.row0 + tok < it.end_row;
      // A decode batch may leave whole warps without a row: they only hand on. (The
      // same in both warps. Prompts fill their tiles; the test alone cost 4 % there.)
      const bool some = !A::kFewRows || __any_sync(~0u, live);
      const int hi = live ? sees(a, it, tok) : INT_MAX;  // keys the row sees; a row that is no token's is not stored
      float ref = -INFINITY, l = 0.f;
      for (int j = 0; j < it.tiles; j++, before = t, t.next(), even ^= 1) {
        ok = wait_warp<0>(c, &bars.s_full[t.i], t.parity) && ok;
        if (!some) {
          if (lane == 0 && ok) arrive_at(p_full + 8 * t.i);
          continue;
        }
        fence_after_sync();
        const uint32_t buf = tw + D + t.i * 128;
        float s[64];
        tmem_ld32(buf + half * 64, s);
        tmem_ld32(buf + half * 64 + 32, s + 32);
        tmem_loaded();
        const int left = hi - (it.first + j) * kTileKeys - half * 64;
        if (__any_sync(~0u, left < 64)) {
          asm volatile("");  // keeps this a branch: as 64 selects in every tile it took a third of the time
#pragma unroll
          for (int i = 0; i < 64; i++)
            if (i >= left) s[i] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 60; i += 8)
#pragma unroll
          for (int k = 0; k < 4; k++) mx[k] = max3(mx[k], s[i + k], s[i + k + 4]);
#pragma unroll
        for (int k = 0; k < 4; k++) mx[k] = fmaxf(mx[k], s[60 + k]);
        const float mine = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
        shared_max[even][half][row] = mine;
        bar_meet(1 + q4);  // also: both warps hold their scores, whose columns the probabilities overwrite
        const float want = fmaxf(mine, shared_max[even][half ^ 1][row]) * cs - Exponent<T>::kShift;
        const bool move = want > ref + kSlack;  // never for a row that sees nothing; always for its first keys
        if (__any_sync(~0u, move)) {
          const float f = move ? exp2_fast(ref - want) : 1.f;
          if (move) ref = want;
          l *= f;
          if (j > 0) {
            ok = wait_warp<0>(c, &bars.pv_done[before.i], before.parity) && ok;
            fence_after_sync();
            const uint64_t ff = pair_of(f, f);
#pragma unroll 1
            for (int i = half * (D / 2); i < (half + 1) * (D / 2); i += 32) {
              float o[32];
              tmem_ld32(tw + i, o);
              tmem_loaded();
              uint32_t u[32];
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                float y0, y1;
                parts_of(mul2(pair_of(o[k], o[k + 1]), ff), y0, y1);
                u[k] = __float_as_uint(y0);
                u[k + 1] = __float_as_uint(y1);
              }
              tmem_st32(tw + i, u);
            }
          }
        }
        const float off = ref == -INFINITY ? 0.f : -ref;
        const uint64_t c2 = pair_of(cs, cs), o2 = pair_of(off, off);
        uint64_t sum2[2] = {0, 0};
        const uint32_t tp = buf + half * 32;
#pragma unroll
        for (int h = 0; h < 2; h++) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; i++) {
            float y0, y1;
            parts_of(fma2(pair_of(s[h * 32 + 2 * i], s[h * 32 + 2 * i + 1]), c2, o2), y0, y1);
            y0 = exp2_fast(y0);
            y1 = exp2_fast(y1);
            sum2[i & 1] = add2(sum2[i & 1], pair_of(y0, y1));
            p[i] = pack2<T>(y0, y1);  // matrix operands of the inputs' type; their sum stays FP32
          }
          tmem_st16u(tp + h * 16, p);
        }
        tmem_stored();
        fence_before_sync();
        __syncwarp();
        if (lane == 0 && ok) arrive_at(p_full + 8 * t.i);
        float y0, y1;
        parts_of(add2(sum2[0], sum2[1]), y0, y1);
        l += y0 + y1;
      }
      shared_sum[half][row] = l;
      x = nth(a, r + 1);  // while the last product runs
      if (x >= 0) next = item_of(a, x);
      bar_meet(1 + q4);
      l += shared_sum[half ^ 1][row];
      ok = wait_warp<0>(c, &bars.pv_done[before.i], before.parity) && ok;
      fence_after_sync();
      const float inv = 1.f / l;
      const bool mend = *(volatile int*)&fix[r % kFixes] == r + 1;
      if (live && ok && half == 0) store_sum(a, it, tok, it.head0 + my_head, ref, l);
      float o[D / 2];
#pragma unroll
      for (int i = 0; i < D / 2; i += 32) tmem_ld32(tw + half * (D / 2) + i, o + i);
      tmem_loaded();
      fence_before_sync();
      __syncwarp();
      // only where another item follows: see arrive_at
      if (lane == 0 && ok && x >= 0) arrive_at(peer_addr(s_addr(&bars.o_empty), 0));
      store_row<T, D>(a, it, tok, it.head0 + my_head, half * (D / 2), o, inv, live && ok, mend, stage[warp]);
      __syncwarp();
      bar_meet(1 + q4);  // shared_sum may be written again
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
  // The MMAs' last commits arrive in both CTAs, and nothing has waited for some of them
  // (no copy is left that would; the softmax wants the last product's alone): none may
  // still be on its way when a CTA leaves. All MMAs are done here, so each barrier is in its
  // last phase or past it, and a parity tells which. A lane each.
  if (warp == kEdgeWarp && !*c.abort_flag) {
    const int i = lane & 3, tiles = walked[0];
    uint64_t* bar = &bars.q_empty;
    int use = walked[1] - 1;  // the barrier's last, from 0; -1 where it has none: such a wait returns at once
    if (lane < 8 && i < ST) {
      bar = lane < 4 ? &bars.k_empty[i] : &bars.v_empty[i];
      use = tiles > i ? (tiles - 1 - i) / ST : -1;
    } else if (lane >= 8 && lane < 12 && i < SB) {
      bar = &bars.pv_done[i];
      use = tiles > i ? (tiles - 1 - i) / SB : -1;
    }
    wait_warp<0>(c, bar, (uint32_t)use & 1);
  }
  __syncwarp();
  pair_sync();
  if (warp == kMmaWarp) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  }
}

template <typename T, int D, typename A>
int launch_of(const A& a, cudaStream_t s) {
  const void* fn = (const void*)attn_tc_kernel<T, D, A>;
  const int rc = opt_in_smem(fn, Geom<D>::kSmem);
  if (rc) return rc;
  const int pairs = std::min(a.items, multiprocessors() / 2);
  return launch_kernel(fn, dim3(2u * (unsigned)pairs), dim3(kThreads), Geom<D>::kSmem, s, const_cast<A*>(&a),
                       dependent_launches(), 1);
}
template <typename A>
int launch_any(const A& a, int act, int dim, cudaStream_t s) {
  if (act == TFX_F16) return dim == 128 ? launch_of<__half, 128>(a, s) : launch_of<__half, 256>(a, s);
  return dim == 128 ? launch_of<__nv_bfloat16, 128>(a, s) : launch_of<__nv_bfloat16, 256>(a, s);
}

}  // namespace

int launch_prompt(const PromptArgs& a, int act, int dim, cudaStream_t s) { return launch_any(a, act, dim, s); }
int launch_prefix(const DecodeAttnArgs& a, int act, int dim, cudaStream_t s) { return launch_any(a, act, dim, s); }

}  // namespace tfx
