// Attention of single tokens over a cache of 8-bit codes.
//
//   s_j = scale log2(e) q . c_j ks(j),  p_j = 2^(s_j - m),  l = sum_j p_j,
//   o = sum_j p_j vs(j) d_j / l,
// c_j, d_j the codes of K and V, ks and vs the scales of their blocks of 16 tokens, one
// pass over the keys. Codes become FP16 exactly, and FP16 MMAs take them: the scale of K is a
// factor of a block's scores, that of V goes into the other operand,
//   w_j = p_j vs(j) = 2^(s_j + log2 vs(j) - M),
// with a running reference M of its own (the largest s_j + log2 vs(j)), so that blocks of any
// size of V, zeros too, leave w in FP16's range; o is brought to m where a partial result is
// stored. l sums the p_j in FP32.
//
// The keys are the MMAs' 16 rows and the query rows their 8 columns, S^T = K Q^T and
// O^T = V^T W^T: the 6 rows of a K/V head of a 24/4 layout cost half of what 16 rows by 8
// keys would, in MMAs and in registers of O. A contraction may take its index in any order, so
// a lane's four consecutive bytes of K stand for k = 2t, 2t+1, 2t+8, 2t+9 of the fragment, and
// q is loaded to match; transposed 16-bit matrix loads of V give a lane two dims of two keys,
// which the conversion to FP16 takes apart: even dims are rows 0-7 of V^T, odd ones 8-15.
//
// A warp owns its rows, its slices (8 KB of K and V of one K/V head: 16 keys of 256, 32 of
// 128) and a ring of two of them, which it fills itself, a slice as soon as one is done.
// Every warp gets the same number of slices, as in attn_warp.cu; decode_join_kernel joins. A
// long prefix that many sequences share is attn_q8_tc.cu's; here keys begin behind it.
//
// Bound: the codes' bytes. 64 sequences of up to 8,192 tokens (553 MB of codes and scales, 24/4 heads of 256)
// take 95 us with the join, 262,144 tokens of one (538 MB, 48/8 of 128) 99: 5.8 and 5.4 TB/s. About 15 us do
// not grow with the tokens (the first loads, the join, SMs that end apart: those of the fullest
// parts of the chip are 10 us behind the others). One sequence of 1,000 tokens: 8 us, the latency of two
// launches and of their loads.
// The fewer bytes are asked for at a time, the faster the memory gives them, down to what its latency
// takes: 7 warps of 2 slices (112 KB an SM) 95 and 99 us, 8 of 2 96 and 99 to 103, 8 of 3 101 and 108, 6 of 2
// 98 and 105, 10 of 2 100 and 110; slices of 4 KB at dim 128 (8 warps of 2, 3 and 4, 12 of 2) 104, 103, 104,
// 100. A barrier a slice, so that a CTA's heads are read together, was no faster.
// One query head to a K/V head: 102 us for 554 MB (16/16 heads of 128), 173 for 1,103 (8/8 of 256). Groups of 9 to 16 take
// the variant of 16 rows (at dim 256 255 registers and 120 to 172 bytes of spills), larger ones walk the codes
// again for every 16: 64 sequences of up to 8,192 tokens, one K/V head of 256, 8, 16, 32, 64 and 128 query heads
// 37, 49, 74, 133 and 246 us (of up to 16,384, heads of 128: 36, 42, 69, 120, 227).
#include <cuda_fp16.h>

#include "attn_split.cuh"
#include "codes.cuh"

namespace tfx {
namespace {

constexpr int kThreads = kCodedWarps * 32;
constexpr int kStages = 2;     // of a warp's ring: see above
constexpr int kFewest = 1;     // slices a warp takes at least (one sequence of 1,000 tokens: 8.0 us, with two 9.0)
// A weight at its reference is 2^kShift, so the largest is between that and 2^15: 11 bits down to
// 2^-21 of it, or further.
constexpr float kShift = 7.f, kSlack = 8.f;

template <int D>
struct Slice {
  static constexpr int kKeys = 4096 / D;  // 16 (D = 256) or 32 (D = 128)
  static constexpr int kBlocks = kKeys / 16;
  static constexpr int kHalf = 4096;      // bytes of K (or V)
  static constexpr int kBlock = 16 * D;   // bytes of one copy of 16 tokens
  static constexpr int kStage = 2 * kHalf;
};
constexpr size_t kSmem = kCodedWarps * kStages * 8192 + 1024;

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8x8 matrix of 16-bit values over the warp, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// 8 * NT rows of a warp; a lane has columns 2t and 2t + 1 of each 8.
template <int NT, int D>
struct Rows {
  uint32_t q[NT][D / 16][2];  // m16n8k16 B fragments
  float o[NT][D / 16][4];     // O^T: dims 16 i + 2 g (elements 0, 1) and + 1 (2, 3)
  float m[NT][2], M[NT][2], l[NT][2];
  float by[NT][2];  // factor of the scores

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < NT; n++) {
#pragma unroll
      for (int i = 0; i < D / 16; i++)
#pragma unroll
        for (int c = 0; c < 4; c++) o[n][i][c] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; c++) {
        m[n][c] = M[n][c] = -INFINITY;
        l[n][c] = 0.f;
      }
    }
  }
  // Row g of 8 rows; null: zeros.
  template <typename T>
  __device__ __forceinline__ void fetch(int n, const T* row, int lane) {
#pragma unroll
    for (int i = 0; i < D / 16; i++) {
      const uint2 x = row ? *reinterpret_cast<const uint2*>(row + 16 * i + 4 * (lane & 3)) : make_uint2(0, 0);
      q[n][i][0] = x.x;
      q[n][i][1] = x.y;
    }
  }
  // BF16 rows become FP16 under a power of two that brings their largest magnitude to [2^14, 2^15).
  template <typename T>
  __device__ __forceinline__ void finish(int n, float scale, int lane) {
    by[n][0] = by[n][1] = scale;
    if constexpr (sizeof(T) == 2 && !__is_same(T, __half)) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 16; i++)
#pragma unroll
        for (int c = 0; c < 2; c++)
          top = max(top, max(q[n][i][c] & 0x7fffu, q[n][i][c] >> 16 & 0x7fffu));
      top = max(top, __shfl_xor_sync(~0u, top, 1));
      top = max(top, __shfl_xor_sync(~0u, top, 2));
      const float up = brings_up(top);
#pragma unroll
      for (int i = 0; i < D / 16; i++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
          const float2 f = pair_to_float(q[n][i][c], T());
          q[n][i][c] = pack2<__half>(f.x * up, f.y * up);
        }
      const float back = inverse_of(up);
#pragma unroll
      for (int c = 0; c < 2; c++) by[n][c] *= __shfl_sync(~0u, back, 4 * (2 * (lane & 3) + c));
    }
  }
};

// A warp's ring, and what of its slices is asked for.
template <int D, int NT>
struct Ring {
  static constexpr int Rows = 8 * NT, NB = Slice<D>::kBlocks;
  uint8_t* buf;
  uint64_t* full;
  float* scales;    // [kStages][K, V][NB]
  int got = 0;      // slices taken so far: stage got % kStages, phase got / kStages
  int asked = 0;    // slices asked for
  long long x, end;
  int s, s1, head;  // the next one to ask for
  const int* table;
  int base, page, next;  // pages of the blocks base + lane, and of 32 further on

  __device__ __forceinline__ int page_of(const DecodeAttnArgs& a, int block) const {
    const int p = (block * 16) >> a.page_shift;
    return p < a.width ? __ldg(table + p) : -1;
  }
  __device__ __forceinline__ void begin(const DecodeAttnArgs& a, const Segment& g, int lane) {
    s = g.s0;
    s1 = g.s1;
    head = g.head;
    table = g.table;
    base = s * NB;
    page = page_of(a, base + lane);
    next = page_of(a, base + 32 + lane);
  }
  // The next slice into its stage, whose last reads are behind the warp.
  __device__ __forceinline__ void ask(const DecodeAttnArgs& a, const Walk& w, const int* starts, int lane) {
    if (x >= end) return;
    const int st = asked % kStages;
    if (s * NB - base >= 32) {
      base += 32;
      page = next;
      next = page_of(a, base + 32 + lane);
    }
    // a lane a block of K or of V: its copy and its scale
    const int b = lane % NB, got = __shfl_sync(~0u, page, s * NB - base + b);
    uint64_t* bar = full + st;
    if (lane == 0) mbar_expect_tx(bar, Slice<D>::kStage);
    __syncwarp();
    if (lane < 2 * NB) {
      const bool value = lane >= NB, in = (unsigned)got < (unsigned)a.pages;
      const int at = (s * Slice<D>::kKeys + 16 * b) & (a.page_size - 1), p = in ? got : -1;  // -1 is out of the map's range: zeros
      tma_load_5d(buf + st * Slice<D>::kStage + lane * Slice<D>::kBlock, value ? &a.v : &a.k, 0, at, 0, head, p, bar);
      float* to = scales + st * 2 * NB + lane;
      if (in) {
        copy4(to, (value ? a.v_scale : a.k_scale) + ((long long)p * (a.page_size / 16) + at / 16) * a.heads_kv + head);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(s_addr(bar)) : "memory");
      } else {
        *to = 1.f;
        mbar_arrive(bar);
      }
    }
    asked++;
    x++;
    if (++s == s1 && x < end) begin(a, segment_at<Slice<D>::kKeys, Rows>(a, w, starts, x, end), lane);
  }
  static __device__ __forceinline__ void copy4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(s_addr(dst)), "l"(src) : "memory");
  }
};

// The rows against slices [s0, s1) of a sequence's keys lo <= key < hi. False: a wait gave up.
template <int Store, int NT, int D>
__device__ __forceinline__ bool attend(Rows<NT, D>& R, Ring<D, NT>& rg, const DecodeAttnArgs& a, const Walk& w,
                                       const int* starts, int s0, int s1, int lo, int hi, int lane) {
  constexpr int KS = Slice<D>::kKeys, NB = Slice<D>::kBlocks;
  const int g = lane >> 2, mi = lane >> 3, mr = lane & 7;
  // 16-byte column c of a key's 8: where the copies' 128-byte swizzle put it
  const int key = (mi & 1) * 8 + mr;
  auto at = [&](int block, int c) {
    return block * Slice<D>::kBlock + (c >> 3) * 2048 + key * 128 + (((c & 7) ^ (key & 7)) << 4);
  };
  for (int s = s0; s < s1; s++) {
    const int st = rg.got % kStages;
    // the warp gives up together: what follows wants all its lanes
    if (!__all_sync(~0u, mbar_wait_bounded(rg.full + st, (rg.got / kStages) & 1, a.spin))) return false;
    uint8_t* kb = rg.buf + st * Slice<D>::kStage;
    uint8_t* vb = kb + Slice<D>::kHalf;
    const float* sc = rg.scales + st * 2 * NB;
    const int k0 = s * KS;
    const bool edge = k0 < lo || k0 + KS > hi;
    // what no row may see: 0 * NaN would be NaN in the product, so V's codes there become zeros
    if (edge) {
      for (int r = 0; r < KS; r++)
        if (k0 + r < lo || k0 + r >= hi)
          for (int c = lane; c < D / 16; c += 32)
            *reinterpret_cast<uint4*>(vb + (r >> 4) * Slice<D>::kBlock + (c >> 3) * 2048 + (r & 15) * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
      fence_async_smem();  // ordinary stores to memory that a later copy writes
      __syncwarp();
    }
    float sx[NB][NT][4];
#pragma unroll
    for (int b = 0; b < NB; b++) {
      float s2[NT][4];
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < 4; c++) sx[b][n][c] = s2[n][c] = 0.f;
      uint32_t r[2][4];  // a step's codes are asked for a step ahead
      ldsm4(r[0], s_addr(kb) + at(b, mi >> 1));
#pragma unroll
      for (int i = 0; i < D / 32; i++) {
        uint32_t x[4][2];
        if (i + 1 < D / 32) ldsm4(r[(i + 1) & 1], s_addr(kb) + at(b, 2 * (i + 1) + (mi >> 1)));
#pragma unroll
        for (int j = 0; j < 4; j++) halves<Store, false>(r[i & 1][j], x[j][0], x[j][1]);
#pragma unroll
        for (int n = 0; n < NT; n++) {
          mma(sx[b][n], x[0][0], x[1][0], x[0][1], x[1][1], R.q[n][2 * i][0], R.q[n][2 * i][1]);
          mma(s2[n], x[2][0], x[3][0], x[2][1], x[3][1], R.q[n][2 * i + 1][0], R.q[n][2 * i + 1][1]);
        }
      }
      const float ks = sc[b];
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < 4; c++) sx[b][n][c] = (sx[b][n][c] + s2[n][c]) * (R.by[n][c & 1] * ks);
      if (edge) {
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int c = 0; c < 4; c++) {
            const int k = k0 + b * 16 + g + (c >> 1) * 8;
            if (k < lo || k >= hi) sx[b][n][c] = -INFINITY;
          }
      }
    }
    // The references follow the maxima where one is passed by more than 2^kSlack, which few slices
    // do: the exchange between lanes that the maxima take is left out of the others.
    float off[NB][NT][2];
    bool over = edge;
#pragma unroll
    for (int b = 0; b < NB; b++) {
      const float lv = log2_scale(sc[NB + b]);
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
          const float mx = fmaxf(sx[b][n][c], sx[b][n][c + 2]);
          over = over || mx > R.m[n][c] + kSlack || mx + lv > R.M[n][c] + kSlack;
          off[b][n][c] = lv + (kShift - (R.M[n][c] == -INFINITY ? 0.f : R.M[n][c]));
        }
    }
    if (__any_sync(~0u, over)) {
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
          float mn = R.m[n][c], Mn = R.M[n][c];
#pragma unroll
          for (int b = 0; b < NB; b++) {
            float mx = fmaxf(sx[b][n][c], sx[b][n][c + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, d));
            mn = fmaxf(mn, mx);
            // a block of which the row sees nothing may have any scale
            off[b][n][c] = mx == -INFINITY ? 0.f : log2_scale(sc[NB + b]);
            Mn = fmaxf(Mn, mx + off[b][n][c]);
          }
          const float Ref = Mn == -INFINITY ? 0.f : Mn, keep = exp2_fast(R.M[n][c] - Ref);
          R.l[n][c] *= exp2_fast(R.m[n][c] - (mn == -INFINITY ? 0.f : mn));
          R.m[n][c] = mn;
          R.M[n][c] = Mn;
#pragma unroll
          for (int b = 0; b < NB; b++) off[b][n][c] += kShift - Ref;
#pragma unroll
          for (int i = 0; i < D / 16; i++) {
            R.o[n][i][c] *= keep;
            R.o[n][i][c + 2] *= keep;
          }
        }
    }
    uint32_t p[NB][NT][2];  // W^T: m16n8k16 B fragments
#pragma unroll
    for (int n = 0; n < NT; n++) {
      float ref[2];
#pragma unroll
      for (int c = 0; c < 2; c++) ref[c] = R.m[n][c] == -INFINITY ? 0.f : R.m[n][c];
#pragma unroll
      for (int b = 0; b < NB; b++) {
        float e[4];
#pragma unroll
        for (int c = 0; c < 4; c++) {
          R.l[n][c & 1] += exp2_fast(sx[b][n][c] - ref[c & 1]);
          e[c] = exp2_fast(sx[b][n][c] + off[b][n][c & 1]);
        }
        // The weights become matrix operands of FP16, 11 bits of each, as TF32 operands would have at half the rate;
        // two operands each would double the product's MMAs. Outputs in FP16 are off by 0.00024 of their
        // size instead of 0.00021 with weights of FP32, nearly all of it their own rounding.
        p[b][n][0] = transposed(pack2<__half>(e[0], e[1]));
        p[b][n][1] = transposed(pack2<__half>(e[2], e[3]));
      }
    }
#pragma unroll
    for (int b = 0; b < NB; b++) {
      uint32_t r[2][4];
      ldsm4t(r[0], s_addr(vb) + at(b, mi >> 1));
#pragma unroll
      for (int i = 0; i < D / 32; i++) {
        uint32_t x[4][2];
        if (i + 1 < D / 32) ldsm4t(r[(i + 1) & 1], s_addr(vb) + at(b, 2 * (i + 1) + (mi >> 1)));
#pragma unroll
        for (int j = 0; j < 4; j++) halves<Store, true>(r[i & 1][j], x[j][0], x[j][1]);
#pragma unroll
        for (int n = 0; n < NT; n++) {
          mma(R.o[n][2 * i], x[0][0], x[0][1], x[1][0], x[1][1], p[b][n][0], p[b][n][1]);
          mma(R.o[n][2 * i + 1], x[2][0], x[2][1], x[3][0], x[3][1], p[b][n][0], p[b][n][1]);
        }
      }
    }
    __syncwarp();
    rg.got++;
    rg.ask(a, w, starts, lane);
  }
#pragma unroll
  for (int n = 0; n < NT; n++)
#pragma unroll
    for (int c = 0; c < 2; c++)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) R.l[n][c] += __shfl_xor_sync(~0u, R.l[n][c], d);
  return true;
}

template <typename T, int Store, int NT, int D>
__global__ void __launch_bounds__(kThreads, 1) decode_q8_kernel(const __grid_constant__ DecodeAttnArgs a) {
  constexpr int KS = Slice<D>::kKeys, NB = Slice<D>::kBlocks, kWarps = kCodedWarps;
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ float scales[kWarps][kStages * 2 * NB];
  __shared__ int starts[TFX_ATTN_MAX_BATCH + 1];
  __shared__ int wsum[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    // a slice's bytes, and its scales
    for (int i = 0; i < kWarps * kStages; i++) mbar_init(&full[0][0] + i, 1 + 2 * NB);
    fence_mbar_init();
    tma_prefetch(&a.k);
    tma_prefetch(&a.v);
  }
  // after the tensor-core kernel, this one starts where that leaves room: see attn_warp.cu
  if (!a.pre_splits) griddep_wait();
  const Walk w = walk_of<KS, 8 * NT>(a, sequence_starts<KS, kWarps>(a, starts, wsum));
  const long long per = max((w.total + a.warps - 1) / a.warps, (long long)kFewest);
  // neighbouring runs go to neighbouring CTAs: few runs still use every SM
  const int me = warp * gridDim.x + blockIdx.x;
  Ring<D, NT> rg;
  rg.buf = dyn + ((1024u - (s_addr(dyn) & 1023u)) & 1023u) + warp * kStages * Slice<D>::kStage;
  rg.full = full[warp];
  rg.scales = scales[warp];
  rg.x = me * per;
  rg.end = min(rg.x + per, w.total);
  long long x = rg.x;
  const long long end = rg.end;
  const T* q = reinterpret_cast<const T*>(a.q);
  Rows<NT, D> R;
  Segment g;
  auto begin = [&]() {  // the segment at x: its rows of q are asked for
    g = segment_at<KS, 8 * NT>(a, w, starts, x, end);
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const int r = 8 * n + (lane >> 2), head = g.head * a.group + g.row0 + r;
      R.fetch(n, r < g.rows ? q + (long long)g.seq * a.ldq + (long long)head * D : nullptr, lane);
    }
  };
  if (x < end) {
    begin();
    rg.begin(a, g, lane);
  }
  for (int i = 0; i < kStages; i++) rg.ask(a, w, starts, lane);
  note_runs(a, w, starts, per);
  griddep_launch();
  bool ok = true;
  while (ok && x < end) {
#pragma unroll
    for (int n = 0; n < NT; n++) R.template finish<T>(n, a.scale_log2, lane);
    R.reset();
    ok = attend<Store>(R, rg, a, w, starts, g.s0, g.s1, a.shared, seq_len(a, g.seq), lane);
    if (!ok) break;
    const long long slot = me + g.group;
    float* po = a.own_o + slot * a.own_rows * D;
    float2* pml = a.own_ml + slot * a.own_rows;
    const int rows = g.rows;
    x += g.s1 - g.s0;
    if (x < end) begin();  // the next segment's q is on its way while this one's result is stored
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int c = 0; c < 2; c++) {
        const int r = 8 * n + 2 * (lane & 3) + c;
        if (r >= rows) continue;
        if (lane < 4) pml[r] = make_float2(R.m[n][c], R.l[n][c]);
        // o relative to m, in two steps that stay in FP32's range
        const float by = R.m[n][c] == -INFINITY ? 0.f : exp2_fast(R.M[n][c] - R.m[n][c]);
#pragma unroll
        for (int i = 0; i < D / 16; i++)
          *reinterpret_cast<float2*>(po + (long long)r * D + i * 16 + 2 * (lane >> 2)) =
              make_float2(R.o[n][i][c] * 0.0078125f * by, R.o[n][i][c + 2] * 0.0078125f * by);  // 2^-kShift
      }
  }
  if (!ok) gave_up(a.err);
  if (a.pre_splits) griddep_wait();  // this grid's end says to the next that both are done
}

template <typename T, int Store, int NT, int D>
int run_of(const DecodeAttnArgs& a, cudaStream_t s) {
  const void* fn = (const void*)decode_q8_kernel<T, Store, NT, D>;
  const int rc = opt_in_smem(fn, kSmem);
  if (rc) return rc;
  return launch_kernel(fn, dim3((unsigned)multiprocessors()), dim3(kThreads), kSmem, s, const_cast<DecodeAttnArgs*>(&a),
                       dependent_launches(), 1);
}
template <typename T, int Store>
int run_of(const DecodeAttnArgs& a, int dim, cudaStream_t s) {
  const bool few = a.group <= 8;
  if (dim == 128) return few ? run_of<T, Store, 1, 128>(a, s) : run_of<T, Store, 2, 128>(a, s);
  return few ? run_of<T, Store, 1, 256>(a, s) : run_of<T, Store, 2, 256>(a, s);
}

}  // namespace

int launch_decode_q8(const DecodeAttnArgs& a, int act, int store, int dim, cudaStream_t s) {
  int rc;
  if (store == TFX_STORE_I8)
    rc = act == TFX_F16 ? run_of<__half, TFX_STORE_I8>(a, dim, s) : run_of<__nv_bfloat16, TFX_STORE_I8>(a, dim, s);
  else
    rc = act == TFX_F16 ? run_of<__half, TFX_STORE_E4M3>(a, dim, s) : run_of<__nv_bfloat16, TFX_STORE_E4M3>(a, dim, s);
  // where few rows have all the warps' partial results, a row's are joined by four times the warps
  const bool wide = a.batch * a.heads_kv * 24LL < a.warps;
  return rc ? rc : launch_join(a, act, dim, wide, s);
}

}  // namespace tfx
