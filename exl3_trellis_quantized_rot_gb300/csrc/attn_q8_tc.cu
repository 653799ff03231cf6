// The shared prefix of a decode batch of many rows, over a cache of 8-bit codes, on the
// tensor cores: tiles of 128 rows against 64 keys at a time, a CTA a tile and share of the keys.
//
// The mathematics is attn_q8.cu's: codes become FP16 operands exactly, K's scale is a factor
// of a block's scores, V's goes into the weights, w_j = p_j vs(j), which have a reference of
// their own. Here that one follows the running maximum only when it is passed by more than
// 2^8 (weights reach 2^15), and a weight is p_j times one factor a block and row, except where
// that factor would leave FP32's range: there the exponent is taken again.
//
// A row is a (sequence, query head) pair of one K/V head; 128 of them fill a tile however the
// heads are grouped. Warps of a CTA: 0-7 softmax, and Q before it: warps w and w + 4 share 32
// rows (a thread a row) and halve their columns; 8-15 turn codes into operands, 16 at a time as
// two 16-byte pieces into the 128-byte swizzle; 16 issues the MMAs; 17 asks for codes and
// scales. Warps 0-15 store the result; 18 and 19 only fill the last four of the register split.
// Codes as registers of the converting warps
// instead of tensor copies made a tile take 3,400 cycles, most of it in issuing the loads.
// Bound: the converting warps, busy in all of a tile's 2,440 cycles (dim 256), of which its MMAs take
// 1,100 beside them. 64 sequences behind 16,384 tokens (24/4 heads of 256): 37 us, issue slots 47 %,
// behind 65,536 with up to 2,048 tokens of their own: 146 for the whole step; over 16-bit pages, whose
// tiles need no conversion, 131 to 133. Each tile of 128 rows converts for itself, so that the same codes are
// converted three times for the 384 rows of a K/V head here. Fewer CTAs here, so that decode_q8_kernel runs beside
// them, were no faster.
// Order of the MMAs: S0, S1, P0 V0, S2, P1 V1, ... Tensor memory: O in columns 0..dim-1, two
// buffers of 64 columns for scores, whose first 32 take the weights.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_device.cuh"
#include "codes.cuh"

namespace tfx {
namespace {

constexpr int kSoft = 8, kConvert = 8;  // warps
constexpr int kMmaWarp = kSoft + kConvert, kFetchWarp = kMmaWarp + 1;
constexpr int kWarps = kMmaWarp + 4;  // whole groups of four, for the register split
constexpr int kThreads = kWarps * 32;
constexpr int kKeys = 64, kRows = 128;
constexpr int kBlocks = kKeys / 16;
constexpr int kScaleTiles = 8;  // tiles whose scales are kept: as many as may be under way, and more
constexpr float kShift = 7.f, kSlack = 8.f;
constexpr float kMostFactor = 100.f;  // log2 of a block's factor, at most

template <int D>
struct Geom {
  static constexpr int kStages = D == 256 ? 1 : 2;  // of operands
  static constexpr int kSlots = D == 256 ? 5 : 8;   // of codes: a tile's K and V are one each
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kKV = kKeys * D * 2;  // bytes of K, or of V, of a stage
  static constexpr int kCodes = kKeys * D;   // bytes of a slot
  static constexpr size_t kSmem = (size_t)kQ + 2 * kStages * kKV + kSlots * kCodes + 1024;
};

struct Barriers {
  uint64_t codes_full[8], codes_empty[8];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2];   // scores are in tensor memory
  uint64_t p_full[2];   // weights are
  uint64_t pv_done[2];  // P V of a tile is added
  uint64_t scales_full[kScaleTiles];
  uint64_t q_full;     // Q is in shared memory
  uint64_t ends_full;  // factors of the rows' results are
};

// The two warps that share rows meet at their named barrier.
__device__ __forceinline__ void bar_meet(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ uint4 load16(uint32_t at) {
  uint4 w;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
  return w;
}

// kind::f16 on FP16, FP32 accumulator, M = 128, A K-major; `mn`: B's columns are its N index.
__host__ __device__ constexpr uint32_t idesc(int N, bool mn) {
  return (1u << 4) | ((uint32_t)mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
// Operands by the low halves of their descriptors: the high ones are the same for all here, and
// 32 whole ones, kept for the steps of a product, took registers that this warp does not have.
constexpr uint32_t kHigh = (uint32_t)(operand_bits(0) >> 32);
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 x, y; setp.ne.b32 p, %4, 0; mov.b64 x, {%1, %5}; mov.b64 y, {%2, %5}; "
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p; }" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 y; setp.ne.b32 p, %4, 0; mov.b64 y, {%2, %5}; "
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p; }" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kHigh)
      : "memory");
}
__device__ __forceinline__ uint32_t low_of(uint32_t saddr, uint64_t bits) { return (uint32_t)operand(saddr, bits); }
__device__ __forceinline__ void commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(s_addr(b)) : "memory");
}
__device__ __forceinline__ void store16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// The CTA's rows and key tiles.
struct Item {
  int head, row0, rows;     // K/V head; rows of the batch's batch * group
  int split, first, tiles;  // share of the prefix; its key tiles
};
__device__ __forceinline__ Item item_of(const DecodeAttnArgs& a) {
  const int x = blockIdx.x, y = x / a.heads_kv;
  Item it;
  it.head = x - y * a.heads_kv;
  it.split = y / a.mt;
  it.row0 = (y - it.split * a.mt) * kRows;
  it.rows = min(kRows, a.batch * a.group - it.row0);
  // the tiles evenly: the first all % splits shares have one more
  const int all = (a.shared + kKeys - 1) / kKeys, each = all / a.pre_splits, more = all - each * a.pre_splits;
  it.first = each * it.split + min(more, it.split);
  it.tiles = each + (it.split < more);
  return it;
}

// Pages of the blocks of 16 keys: a lane's block, eight tiles at a time.
__device__ __forceinline__ int page_of(const DecodeAttnArgs& a, const int* table, int tile, int lane) {
  const int p = (tile * kKeys + lane * 16) >> a.page_shift;
  return p < a.width ? __ldg(table + p) : -1;
}

// A tile's codes as FP16 rows of keys, in column blocks of 64 values. A lane takes 16 codes of a
// key, whose two pieces go to one column block; every other four lanes begin with the second, so
// that eight lanes meet all banks. Codes lie as their copies left them: 16 keys of dim bytes each,
// in column blocks of 128, swizzled.
template <int Store, int D>
struct Convert {
  static constexpr int kLanes = D / 16;     // of a key
  static constexpr int kPer = 32 / kLanes;  // keys of a load
  static constexpr int kLoads = kKeys / (kConvert * kPer);
  uint4 x[kLoads];
  __device__ __forceinline__ static int key_of(int i, int warp, int lane) { return (i * kConvert + warp) * kPer + lane / kLanes; }
  __device__ __forceinline__ void load(uint32_t src, int warp, int lane) {
    const int l = lane % kLanes;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int key = key_of(i, warp, lane), k = key & 15;
      x[i] = load16(src + (key >> 4) * (16 * D) + (l >> 3) * 2048 + k * 128 + (((l & 7) ^ (k & 7)) << 4));
    }
  }
  __device__ __forceinline__ void store(uint32_t dst, int warp, int lane) const {
    const int l = lane % kLanes, swap = (l >> 2) & 1;
#pragma unroll
    for (int i = 0; i < kLoads; i++) {
      const int key = key_of(i, warp, lane);
      // the lane's first piece, and its second
      uint32_t h[8];
      halves<Store, false>(swap ? x[i].z : x[i].x, h[0], h[1]);
      halves<Store, false>(swap ? x[i].w : x[i].y, h[2], h[3]);
      halves<Store, false>(swap ? x[i].x : x[i].z, h[4], h[5]);
      halves<Store, false>(swap ? x[i].y : x[i].w, h[6], h[7]);
      const uint32_t at = dst + (l >> 2) * (kKeys * 128) + key * 128;
      const int p = (l & 3) * 2 + swap;
      store16(at + ((p ^ (key & 7)) << 4), h[0], h[1], h[2], h[3]);
      store16(at + ((p ^ 1 ^ (key & 7)) << 4), h[4], h[5], h[6], h[7]);
    }
  }
};

template <typename T, int Store, int D>
__global__ void __launch_bounds__(kThreads, 1) prefix_q8_kernel(const __grid_constant__ DecodeAttnArgs a) {
  using G = Geom<D>;
  constexpr int ST = G::kStages, SL = G::kSlots;
  extern __shared__ uint8_t dyn[];
  __shared__ Barriers bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ float scales[kScaleTiles][2 * kBlocks];
  __shared__ float row_by[kRows];   // factor of a row's scores
  __shared__ float row_end[kRows];  // of its result
  __shared__ float shared_top[2][2][kRows][2], shared_sum[2][kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t base = s_addr(dyn) + ((1024u - (s_addr(dyn) & 1023u)) & 1023u);
  const uint32_t sq = base, sk = base + G::kQ, sv = sk + ST * G::kKV, sc = sv + ST * G::kKV;
  const Ctx c = {&abort_flag, a.err, a.spin};
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < SL; i++) {
      mbar_init(&bars.codes_full[i], 1 + kBlocks);  // the copies' bytes, and each block's scale
      mbar_init(&bars.codes_empty[i], kConvert);
    }
    for (int i = 0; i < ST; i++) {
      mbar_init(&bars.k_full[i], kConvert);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], kConvert);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], kSoft);
      mbar_init(&bars.pv_done[i], 1);
    }
    for (int i = 0; i < kScaleTiles; i++) mbar_init(&bars.scales_full[i], 1);
    mbar_init(&bars.q_full, kSoft);
    mbar_init(&bars.ends_full, kSoft / 2);
    fence_mbar_init();
    tma_prefetch(&a.k);
    tma_prefetch(&a.v);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(s_addr(&tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const Item it = item_of(a);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tm = *(volatile uint32_t*)&tmem_slot;
  griddep_wait();
  griddep_launch();  // what follows waits for this grid before it reads what it wrote

  // Q: a row by D/8 lanes, two rows at a time where that is half of them. A lane works out where
  // one of the warp's 16 rows is.
  auto load_q = [&](int helper) {
    constexpr int kLanes = D / 8, kPer = 32 / kLanes, kSteps = kRows / kPer / kSoft;
    const int l = lane % kLanes;
    const int my_r = (lane & 15) / kPer * (kSoft * kPer) + helper * kPer + (lane & 15) % kPer, my_row = it.row0 + my_r;
    const int my_seq = my_row / a.group;
    const long long my_at = my_r < it.rows ? my_seq * a.ldq + (long long)(it.head * a.group + my_row - my_seq * a.group) * D : -1;
    uint4 x[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; k++) {
      const long long at = __shfl_sync(~0u, my_at, k * kPer + lane / kLanes);
      x[k] = make_uint4(0, 0, 0, 0);
      if (at >= 0) x[k] = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + at + l * 8);
    }
#pragma unroll
    for (int k = 0; k < kSteps; k++) {
      const int r = (k * kSoft + helper) * kPer + lane / kLanes;
      uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      float by = a.scale_log2;
      if constexpr (!__is_same(T, __half)) {
        uint32_t top = 0;
#pragma unroll
        for (int n = 0; n < 4; n++) top = __vmaxu2(top, w[n] & 0x7fff7fffu);
        top = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int d = kLanes / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
        const float up = brings_up(top);
#pragma unroll
        for (int n = 0; n < 4; n++) {
          const float2 f = pair_to_float(w[n], T());
          w[n] = pack2<__half>(f.x * up, f.y * up);
        }
        by *= inverse_of(up);
      }
      store16(sq + (l >> 3) * (kRows * 128) + r * 128 + (((l & 7) ^ (r & 7)) << 4), w[0], w[1], w[2], w[3]);
      if (l == 0) row_by[r] = by;
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.q_full);
  };
  // The result's columns, 32 at a time: every fourth run of them by a warp, of the 32 rows whose
  // tensor memory it reaches. 16 rows at a time go through shared memory, eight lanes a row's 128 bytes.
  auto store_result = [&](bool ok) {
    const int quarter = warp & 3, r = quarter * 32 + lane, row = it.row0 + r;
    const bool stored = ok && r < it.rows;
    const int seq = stored ? row / a.group : 0, head = it.head * a.group + (stored ? row % a.group : 0);
    float* po = stored ? a.pre_o + (((long long)it.split * a.batch + seq) * a.heads_q + head) * D : nullptr;
    float* to[8];
#pragma unroll
    for (int k = 0; k < 8; k++)
      to[k] = reinterpret_cast<float*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(po), k * 4 + (lane >> 3)));
    const float scale = row_end[r];
    // 2 KB a warp of Q's memory, which nothing reads any more
    static_assert((kSoft + kConvert) * 2048 <= G::kQ && kSoft + kConvert == 16, "sixteen warps store the result");
    const uint32_t mine = sq + warp * 2048;
    const int q = lane & 7;
#pragma unroll 1
    for (int i = (warp >> 2) * 32; i < D; i += 128) {
      float o[32];
      tmem_ld32(tm + ((uint32_t)quarter << 21) + i, o);
      tmem_loaded();
#pragma unroll
      for (int h = 0; h < 2; h++) {
        if ((lane >> 4) == h)
#pragma unroll
          for (int k = 0; k < 8; k++) {
            uint32_t u[4];
#pragma unroll
            for (int n = 0; n < 4; n++) u[n] = __float_as_uint(o[4 * k + n] * 0.0078125f * scale);  // 2^-kShift
            store16(mine + ((lane & 15) * 8 + (k ^ q)) * 16, u[0], u[1], u[2], u[3]);
          }
        __syncwarp();
        uint4 w[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const int x = k * 4 + (lane >> 3);
          w[k] = load16(mine + (x * 8 + (q ^ (x & 7))) * 16);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; k++)
          if (to[h * 4 + k]) *reinterpret_cast<uint4*>(to[h * 4 + k] + i + q * 4) = w[k];
      }
    }
  };

  // registers: 640 x 96 at launch; 256 x 128 + 256 x 88 + 128 x 48 are as many from here on
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (warp == kFetchWarp) {
      // ---- codes and scales, a lane a block of 16 keys: K0, K1, V0, K2, V1, ...
      const int* table = prefix_table(a);
      int page = page_of(a, table, it.first, lane), next = 0;
      Turn<SL> t;
      bool ok = true;
      auto ask = [&](const CUtensorMap* map, int at, int got) -> uint64_t* {
        if (!(ok = wait_warp<30>(c, &bars.codes_empty[t.i], t.parity ^ 1))) return nullptr;
        uint64_t* bar = &bars.codes_full[t.i];
        if (lane == 0) mbar_expect_tx(bar, G::kCodes);
        __syncwarp();
        if (lane < kBlocks) tma_load_5d(sc + t.i * G::kCodes + lane * 16 * D, map, 0, at, 0, it.head, got, bar);
        t.next();
        return bar;
      };
      int v_at = 0, v_page = 0;
      for (int j = 0; ok && j <= it.tiles; j++) {
        int at = 0, got = 0;
        if (j < it.tiles) {
          if ((j & 7) == 0) {
            if (j) page = next;
            next = page_of(a, table, it.first + j + 8, lane);
          }
          const int key = (it.first + j) * kKeys + (lane & 3) * 16;
          at = key & (a.page_size - 1);
          got = __shfl_sync(~0u, page, (j & 7) * kBlocks + (lane & 3));
          // what is not there or not shared: -1, out of the map's range, that is zeros
          if (key >= a.shared || (unsigned)got >= (unsigned)a.pages) got = -1;
          uint64_t* bar = ask(&a.k, at, got);
          if (bar && lane < kBlocks) {
            float* to = &scales[j % kScaleTiles][lane];
            if (got >= 0) {
              const long long x = ((long long)got * (a.page_size / 16) + at / 16) * a.heads_kv + it.head;
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_addr(to)), "l"(a.k_scale + x) : "memory");
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_addr(to + kBlocks)), "l"(a.v_scale + x) : "memory");
              asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(s_addr(bar)) : "memory");
            } else {
              to[0] = to[kBlocks] = 1.f;
              mbar_arrive(bar);
            }
          }
          __syncwarp();
        }
        if (ok && j > 0) {
          uint64_t* bar = ask(&a.v, v_at, v_page);
          if (bar && lane < kBlocks) mbar_arrive(bar);
          __syncwarp();
        }
        v_at = at;
        v_page = got;
      }
    } else if (warp == kMmaWarp) {
      // ---- MMAs
      constexpr uint32_t is = idesc(kKeys, false), ip = idesc(D, true);
      constexpr uint64_t kmaj = operand_bits(16), vmaj = operand_bits(kKeys * 128);
      const uint32_t qd = low_of(sq, kmaj), kd0 = low_of(sk, kmaj), vd0 = low_of(sv, vmaj);
      Turn<ST> kt, vt;
      Turn<2> st, pt;
      auto scores = [&]() -> bool {
        if (!wait_warp<10>(c, &bars.k_full[kt.i], kt.parity)) return false;
        fence_after_sync();
        const uint32_t kd = kd0 + kt.i * (G::kKV >> 4);
        const uint32_t d = tm + D + st.i * kKeys;
        if (elected()) {
#pragma unroll 1
          for (int b = 0; b < D / 64; b++)  // column blocks of 64
#pragma unroll
            for (int k = 0; k < 4; k++)
              mma_ss(d, qd + ((b * (kRows * 128) + k * 32) >> 4), kd + ((b * (kKeys * 128) + k * 32) >> 4), is, b + k > 0);
          commit(&bars.s_full[st.i]);
          commit(&bars.k_empty[kt.i]);
        }
        __syncwarp();
        kt.next();
        st.next();
        return true;
      };
      bool ok = wait_warp<10>(c, &bars.q_full, 0);
      int issued = 0;
      for (int j = 0; ok && j < it.tiles; j++) {
        for (; ok && issued < it.tiles && issued < j + 2; issued++) ok = scores();
        if (!ok || !(ok = wait_warp<10>(c, &bars.p_full[pt.i], pt.parity) && wait_warp<10>(c, &bars.v_full[vt.i], vt.parity))) break;
        fence_after_sync();
        const uint32_t vd = vd0 + vt.i * (G::kKV >> 4);
        const uint32_t p = tm + D + pt.i * kKeys;
        if (elected()) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; k++) mma_ts(tm, p + k * 8, vd + ((k * 2048) >> 4), ip, j > 0 || k > 0);
          commit(&bars.v_empty[vt.i]);
          commit(&bars.pv_done[pt.i]);
        }
        __syncwarp();
        vt.next();
        pt.next();
      }
      // the last commits that nothing else waits for: none may be on its way when the CTA leaves
      for (int i = 0; i < ST && ok; i++) {
        const int use = it.tiles > i ? (it.tiles - 1 - i) / ST : -1;
        ok = wait_warp<0>(c, &bars.k_empty[i], (uint32_t)use & 1) && wait_warp<0>(c, &bars.v_empty[i], (uint32_t)use & 1);
      }
    }
  } else if (warp >= kSoft) {
    // ---- codes to operands
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int conv = warp - kSoft;
    Turn<ST> kt, vt;
    Turn<SL> from;
    Convert<Store, D> x;
    bool ok = true;
    auto step = [&](uint64_t* empty, uint64_t* full, const Turn<ST>& t, uint32_t dst, int tile) {
      if (!(ok = wait_warp<10>(c, &bars.codes_full[from.i], from.parity))) return;
      x.load(sc + from.i * G::kCodes, conv, lane);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bars.codes_empty[from.i]);
        if (conv == 0 && tile >= 0) mbar_arrive(&bars.scales_full[tile % kScaleTiles]);
      }
      from.next();
      if (!(ok = wait_warp<10>(c, empty + t.i, t.parity ^ 1))) return;
      x.store(dst + t.i * G::kKV, conv, lane);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(full + t.i);
    };
    // in the order of the copies: a tile's V waits for the product before it, the next K does not
    for (int j = 0; ok && j <= it.tiles; j++) {
      if (j < it.tiles) {
        step(bars.k_empty, bars.k_full, kt, sk, j);
        kt.next();
      }
      if (ok && j > 0) {
        step(bars.v_empty, bars.v_full, vt, sv, -1);
        vt.next();
      }
    }
    // the last product is added, and the rows' factors are there
    const int last = it.tiles - 1;
    ok = ok && wait_warp<100>(c, &bars.ends_full, 0) && wait_warp<30>(c, &bars.pv_done[last & 1], (last >> 1) & 1);
    fence_after_sync();
    store_result(ok);
  } else {
    // ---- softmax: a thread a row. A wait that gave up changes only what is handed on.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    load_q(warp);
    const int q4 = warp & 3, half = warp >> 2, r = q4 * 32 + lane, row = it.row0 + r;
    const uint32_t tw = tm + ((uint32_t)q4 << 21);
    const bool live = r < it.rows;
    const int seq = live ? row / a.group : 0, head = it.head * a.group + (live ? row % a.group : 0);
    const int hi = live ? min(a.shared, seq_len(a, seq)) : INT_MAX;  // keys the row sees
    bool ok = wait_warp<0>(c, &bars.q_full, 0);
    const float by = row_by[r];
    constexpr int kMine = kKeys / 2, kMyBlocks = kBlocks / 2;
    Turn<2> t, before;
    float m = -INFINITY, ref = -INFINITY, l = 0.f;
    for (int j = 0; j < it.tiles; j++, before = t, t.next()) {
      ok = wait_warp<0>(c, &bars.scales_full[j % kScaleTiles], (j / kScaleTiles) & 1) && ok;
      const float* mine = scales[j % kScaleTiles] + half * kMyBlocks;
      float ks[kMyBlocks], off[kMyBlocks];
#pragma unroll
      for (int b = 0; b < kMyBlocks; b++) {
        ks[b] = by * mine[b];
        off[b] = log2_scale(mine[kBlocks + b]);
      }
      ok = wait_warp<0>(c, &bars.s_full[t.i], t.parity) && ok;
      fence_after_sync();
      const uint32_t buf = tw + D + t.i * kKeys;
      float s[kMine];
      tmem_ld32(buf + half * kMine, s);
      tmem_loaded();
#pragma unroll
      for (int b = 0; b < kMyBlocks; b++) {
        const uint64_t f2 = pair_of(ks[b], ks[b]);
#pragma unroll
        for (int i = 16 * b; i < 16 * b + 16; i += 2) parts_of(mul2(pair_of(s[i], s[i + 1]), f2), s[i], s[i + 1]);
      }
      const int left = hi - (it.first + j) * kKeys - half * kMine;
      if (__any_sync(~0u, left < kMine)) {
        asm volatile("");  // a branch, not selects in every tile
#pragma unroll
        for (int i = 0; i < kMine; i++)
          if (i >= left) s[i] = -INFINITY;
      }
      float want = -INFINITY, top = -INFINITY;
#pragma unroll
      for (int b = 0; b < kMyBlocks; b++) {
        const float* x = s + 16 * b;
        float mx = max3(max3(x[0], x[1], x[2]), x[3], x[4]), my = max3(max3(x[5], x[6], x[7]), x[8], x[9]);
        mx = max3(max3(mx, my, x[10]), max3(x[11], x[12], x[13]), fmaxf(x[14], x[15]));
        // a block of which the row sees nothing may have any scale
        if (mx == -INFINITY) off[b] = 0.f;
        want = fmaxf(want, mx + off[b]);
        top = fmaxf(top, mx);
      }
      *reinterpret_cast<float2*>(shared_top[t.i][half][r]) = make_float2(top, want);
      bar_meet(1 + q4);  // also: both warps hold their scores, whose columns the weights overwrite
      const float2 other = *reinterpret_cast<const float2*>(shared_top[t.i][half ^ 1][r]);
      top = max3(top, other.x, m);
      want = fmaxf(want, other.y) - kShift;
      const float m0 = top == -INFINITY ? 0.f : top;
      l *= exp2_fast(m - m0);
      m = top;
      const bool move = want > ref + kSlack;  // never for a row that sees nothing; always for its first keys
      if (__any_sync(~0u, move)) {
        const float f = move ? exp2_fast(ref - want) : 1.f;
        if (move) ref = want;
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
      const float ref0 = ref == -INFINITY ? 0.f : ref;
      bool wide = false;
#pragma unroll
      for (int b = 0; b < kMyBlocks; b++) {
        off[b] -= ref0;
        wide = wide || off[b] + m0 > kMostFactor;
      }
      uint64_t sum2[2] = {0, 0};
      uint32_t p[kMine / 2];
      if (__any_sync(~0u, wide)) {
#pragma unroll
        for (int i = 0; i < kMine / 2; i++) {
          const float x = s[2 * i], y = s[2 * i + 1], o = off[i / 8];
          sum2[0] = add2(sum2[0], pair_of(exp2_fast(x - m0), exp2_fast(y - m0)));
          p[i] = pack2<__half>(exp2_fast(x + o), exp2_fast(y + o));
        }
      } else {
        const uint64_t m2 = pair_of(-m0, -m0);
#pragma unroll
        for (int b = 0; b < kMyBlocks; b++) {
          const float f = exp2_fast(off[b] + m0);
          const uint64_t f2 = pair_of(f, f);
#pragma unroll
          for (int i = 8 * b; i < 8 * b + 8; i++) {
            float x, y;
            parts_of(add2(pair_of(s[2 * i], s[2 * i + 1]), m2), x, y);
            const uint64_t e = pair_of(exp2_fast(x), exp2_fast(y));
            sum2[i & 1] = add2(sum2[i & 1], e);
            parts_of(mul2(e, f2), x, y);
            p[i] = pack2<__half>(x, y);  // FP16 matrix operands; the sum stays FP32
          }
        }
      }
      tmem_st16u(buf + half * (kMine / 2), p);
      tmem_stored();
      fence_before_sync();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&bars.p_full[t.i]);
      float y0, y1;
      parts_of(add2(sum2[0], sum2[1]), y0, y1);
      l += y0 + y1;
    }
    shared_sum[half][r] = l;
    bar_meet(1 + q4);
    l += shared_sum[half ^ 1][r];
    // o relative to m, in two steps that stay in FP32's range: see store_result
    if (half == 0) {
      row_end[r] = m == -INFINITY ? 0.f : exp2_fast(ref + kShift - m);
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&bars.ends_full);
    }
    ok = wait_warp<0>(c, &bars.ends_full, 0) && ok;
    ok = wait_warp<0>(c, &bars.pv_done[before.i], before.parity) && ok;
    fence_after_sync();
    if (live && ok && half == 0) a.pre_ml[((long long)it.split * a.batch + seq) * a.heads_q + head] = make_float2(m, l);
    store_result(ok);
  }
  __syncwarp();
  if (*c.abort_flag) {  // MMAs in flight land
    const long long t0 = clock64();
    while (clock64() - t0 < 2000000) {
    }
    __syncwarp();
  }
  fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm) : "memory");
  }
}

template <typename T, int Store, int D>
int prefix_of(const DecodeAttnArgs& a, cudaStream_t s) {
  const void* fn = (const void*)prefix_q8_kernel<T, Store, D>;
  const int rc = opt_in_smem(fn, Geom<D>::kSmem);
  if (rc) return rc;
  return launch_kernel(fn, dim3((unsigned)a.items), dim3(kThreads), Geom<D>::kSmem, s, const_cast<DecodeAttnArgs*>(&a),
                       dependent_launches(), 1);
}
template <typename T>
int prefix_of(const DecodeAttnArgs& a, int store, int dim, cudaStream_t s) {
  if (store == TFX_STORE_I8) return dim == 128 ? prefix_of<T, TFX_STORE_I8, 128>(a, s) : prefix_of<T, TFX_STORE_I8, 256>(a, s);
  return dim == 128 ? prefix_of<T, TFX_STORE_E4M3, 128>(a, s) : prefix_of<T, TFX_STORE_E4M3, 256>(a, s);
}

}  // namespace

int prefix_q8_rows() { return kRows; }
int prefix_q8_tiles(int shared) { return (shared + kKeys - 1) / kKeys; }

int launch_prefix_q8(const DecodeAttnArgs& a, int act, int store, int dim, cudaStream_t s) {
  return act == TFX_F16 ? prefix_of<__half>(a, store, dim, s) : prefix_of<__nv_bfloat16>(a, store, dim, s);
}

}  // namespace tfx
