// Attention by single warps: 16 rows against slices of keys, m16n8k16 MMAs.
//
//   m' = max(m, max_j s_j),  p_j = 2^(s_j - m'),  l' = l 2^(m - m') + sum_j p_j,
//   o' = o 2^(m - m') + sum_j p_j v_j,            s_j = scale log2(e) q . k_j,
// one pass over the keys; the row's result is o / l. A warp owns its rows, its
// slices and its own ring of shared-memory stages, so the four of a CTA never
// wait for one another; a fifth warp asks for their slices, one lane a ring, and
// runs on into the next segment while the last one's result is stored. Partial
// results (o, m, l) of several warps are joined by decode_join_kernel in slot order.
//
// A slice is 16 KB of K and V of one K/V head (16 keys of 256, 32 of 128),
// fetched by two to four tensor copies of 16 tokens each with the 128-byte
// swizzle, so that the 8x8 matrix loads of K (rows = keys) and V (transposed)
// meet no bank twice.
//
// What bounds it (GB300): the memory where there is enough to read (64 sequences of
// 1 to 2,048 tokens, 24/4 heads of 256, 268 MB: 39 us from the first slice to the
// median warp's last, 6.8 TB/s; the arithmetic of a slice takes a warp about 1,400
// cycles, a third of that time), latency where there is not (1,000 tokens of one
// sequence: 5 us). Every warp gets the same number of slices, at least two, and not
// whole sequences: with one warp a sequence and head the longest would be waited for.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_device.cuh"
#include "attn_internal.h"
#include "attn_split.cuh"

namespace tfx {
namespace {

constexpr int kWarps = 4;  // that compute; one more asks for their slices
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kStages = 3;
constexpr int kFewest = 2;  // slices a warp takes at least

template <int D>
struct Slice {
  static constexpr int kKeys = 4096 / D;           // 16 (D = 256) or 32 (D = 128)
  static constexpr int kHalf = kKeys * D * 2;      // bytes of K (or V) of a slice
  static constexpr int kBlock = 16 * D * 2;        // bytes of one 16-token copy
  static constexpr int kStage = 2 * kHalf;
};
template <int D>
constexpr size_t warp_smem() {
  return (size_t)kWarps * kStages * Slice<D>::kStage + 1024;
}

template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two rows of a warp's 16 as one lane sees them: row lane/4 and row lane/4 + 8.
template <typename T, int D>
struct Rows {
  uint32_t q[D / 16][4];  // m16n8k16 A fragments
  float o[D / 8][4];
  float m[2], l[2];  // reference of the exponents (log2 units) and sum
  int hi[2];         // keys the row sees end here

  __device__ __forceinline__ void load(const T* r0, const T* r1, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int i = 0; i < D / 16; i++) {
      const int c = i * 16 + 2 * t;
      q[i][0] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + c) : 0u;
      q[i][1] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + c) : 0u;
      q[i][2] = r0 ? *reinterpret_cast<const uint32_t*>(r0 + c + 8) : 0u;
      q[i][3] = r1 ? *reinterpret_cast<const uint32_t*>(r1 + c + 8) : 0u;
    }
  }
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int i = 0; i < D / 8; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) o[i][j] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }
};

// The ring of one warp: stages of one slice each.
struct Ring {
  uint8_t* buf;
  uint64_t *full, *empty;
  int it = 0;  // slices so far: stage it % kStages, phase it / kStages
};

// One lane: the slices [x, end) into a ring, in order.
template <int D>
__device__ __forceinline__ bool feed(const DecodeAttnArgs& a, const Walk& w, const int* starts, Ring& rg, long long x,
                                     long long end) {
  constexpr int KS = Slice<D>::kKeys;
  auto page_at = [&](const int* table, int token) {
    const int p = token >> a.page_shift;
    return p < a.width ? __ldg(table + p) : -1;
  };
  while (x < end) {
    const Segment g = segment_at<Slice<D>::kKeys, 16>(a, w, starts, x, end);
    int next = page_at(g.table, g.s0 * KS);
    for (int s = g.s0; s < g.s1; s++) {
      const int page0 = next, st = rg.it % kStages;
      if (s + 1 < g.s1) next = page_at(g.table, (s + 1) * KS);
      if (!mbar_wait_bounded(rg.empty + st, ((rg.it / kStages) & 1) ^ 1, a.spin)) return false;
      uint8_t* dst = rg.buf + st * Slice<D>::kStage;
      uint64_t* bar = rg.full + st;
      mbar_expect_tx(bar, Slice<D>::kStage);
#pragma unroll
      for (int b = 0; b < KS / 16; b++) {
        const int token = s * KS + 16 * b;
        // a page of 16 ends inside a slice of 32 keys: its second half has an entry of its own
        const int p = b == 0 ? page0 : page_at(g.table, token);
        const int page = (unsigned)p < (unsigned)a.pages ? p : -1;  // -1 is out of the map's range: zeros
        const int at = token & (a.page_size - 1);
        tma_load_5d(dst + b * Slice<D>::kBlock, &a.k, 0, at, 0, g.head, page, bar);
        tma_load_5d(dst + Slice<D>::kHalf + b * Slice<D>::kBlock, &a.v, 0, at, 0, g.head, page, bar);
      }
      rg.it++;
    }
    x += g.s1 - g.s0;
  }
  return true;
}

// The rows against slices [s0, s1) of the keys lo <= key < hi. False: a wait gave up.
template <typename T, int D>
__device__ __forceinline__ bool attend(Rows<T, D>& R, Ring& rg, int s0, int s1, int lo, float scale, int lane,
                                       long long spin) {
  constexpr int KS = Slice<D>::kKeys, NB = KS / 16;
  const int t = lane & 3, mi = lane >> 3, mr = lane & 7;
  int hmin = min(R.hi[0], R.hi[1]), hmax = max(R.hi[0], R.hi[1]);
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    hmin = min(hmin, __shfl_xor_sync(~0u, hmin, d));
    hmax = max(hmax, __shfl_xor_sync(~0u, hmax, d));
  }
  for (int s = s0; s < s1; s++) {
    const int st = rg.it % kStages;
    // the warp gives up together: what follows wants all its lanes
    if (!__all_sync(~0u, mbar_wait_bounded(rg.full + st, (rg.it / kStages) & 1, spin))) return false;
    uint8_t* kb = rg.buf + st * Slice<D>::kStage;
    uint8_t* vb = kb + Slice<D>::kHalf;
    const int k0 = s * KS;
    // what no row may see: 0 * inf would be NaN in the product, so V's rows there become zeros
    const bool edge = k0 < lo || k0 + KS > hmin;
    if (k0 < lo || k0 + KS > hmax) {
      for (int r = 0; r < KS; r++)
        if (k0 + r < lo || k0 + r >= hmax)
          for (int c = lane; c < D / 8; c += 32)
            *reinterpret_cast<uint4*>(vb + (r >> 4) * Slice<D>::kBlock + (c >> 3) * 2048 + (r & 15) * 128 +
                                      (c & 7) * 16) = make_uint4(0, 0, 0, 0);
      fence_async_smem();  // ordinary stores to memory that a later copy writes
      __syncwarp();
    }
    // S = Q K^T; two chains per tile of 8 keys, each step's K a step ahead
    float sc[KS / 8][4];
    {
      float s2[KS / 8][4];
#pragma unroll
      for (int j = 0; j < KS / 8; j++)
#pragma unroll
        for (int c = 0; c < 4; c++) sc[j][c] = s2[j][c] = 0.f;
      const int key = (mi >> 1) * 8 + mr;
      uint32_t f[2][NB][4];
      auto load = [&](int i) {
        const int c = i * 2 + (mi & 1);  // 16-byte column of 8 values
#pragma unroll
        for (int b = 0; b < NB; b++)
          ldsm4(f[i & 1][b], s_addr(kb) + b * Slice<D>::kBlock + (c >> 3) * 2048 + key * 128 + (((c & 7) ^ (key & 7)) << 4));
      };
      load(0);
#pragma unroll
      for (int i = 0; i < D / 16; i++) {
        if (i + 1 < D / 16) load(i + 1);
#pragma unroll
        for (int b = 0; b < NB; b++) {
          const uint32_t(&x)[4] = f[i & 1][b];
          mma<T>(i & 1 ? s2[2 * b] : sc[2 * b], R.q[i], x[0], x[1]);
          mma<T>(i & 1 ? s2[2 * b + 1] : sc[2 * b + 1], R.q[i], x[2], x[3]);
        }
      }
#pragma unroll
      for (int j = 0; j < KS / 8; j++)
#pragma unroll
        for (int c = 0; c < 4; c++) sc[j][c] = (sc[j][c] + s2[j][c]) * scale;
    }
    if (edge) {
#pragma unroll
      for (int j = 0; j < KS / 8; j++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
          const int key = k0 + j * 8 + 2 * t + (c & 1);
          if (key < lo || key >= R.hi[c >> 1]) sc[j][c] = -INFINITY;
        }
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < KS / 8; j++)
#pragma unroll
      for (int c = 0; c < 4; c++) mx[c >> 1] = fmaxf(mx[c >> 1], sc[j][c]);
    float ref[2], keep[2];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(~0u, mx[h], 2));
      // the exponents' reference: kShift below the running maximum; a row that has seen no key keeps 0
      const float mn = fmaxf(R.m[h], mx[h] - Exponent<T>::kShift);
      ref[h] = mn == -INFINITY ? 0.f : mn;
      keep[h] = exp2_fast(R.m[h] - ref[h]);
      R.m[h] = mn;
      R.l[h] *= keep[h];
    }
    if (__any_sync(~0u, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 8; i++)
#pragma unroll
        for (int c = 0; c < 4; c++) R.o[i][c] *= keep[c >> 1];
    }
    uint32_t p[NB][4];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
      for (int j = 0; j < 2; j++) {
        float e[4];
#pragma unroll
        for (int c = 0; c < 4; c++) {
          e[c] = exp2_fast(sc[2 * b + j][c] - ref[c >> 1]);
          R.l[c >> 1] += e[c];
        }
        // the probabilities become matrix operands of the inputs' type; their sum stays FP32
        p[b][2 * j] = pack2<T>(e[0], e[1]);
        p[b][2 * j + 1] = pack2<T>(e[2], e[3]);
      }
    const int vkey = (mi & 1) * 8 + mr;
    {
      uint32_t f[2][NB][4];
      auto load = [&](int i) {
        const int c = i * 2 + (mi >> 1);
#pragma unroll
        for (int b = 0; b < NB; b++)
          ldsm4t(f[i & 1][b],
                 s_addr(vb) + b * Slice<D>::kBlock + (c >> 3) * 2048 + vkey * 128 + (((c & 7) ^ (vkey & 7)) << 4));
      };
      load(0);
#pragma unroll
      for (int i = 0; i < D / 16; i++) {
        if (i + 1 < D / 16) load(i + 1);
#pragma unroll
        for (int b = 0; b < NB; b++) {
          mma<T>(R.o[2 * i], p[b], f[i & 1][b][0], f[i & 1][b][1]);
          mma<T>(R.o[2 * i + 1], p[b], f[i & 1][b][2], f[i & 1][b][3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(rg.empty + st);
    rg.it++;
  }
#pragma unroll
  for (int h = 0; h < 2; h++) {
    R.l[h] += __shfl_xor_sync(~0u, R.l[h], 1);
    R.l[h] += __shfl_xor_sync(~0u, R.l[h], 2);
  }
  return true;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) decode_warp_kernel(const __grid_constant__ DecodeAttnArgs a) {
  constexpr int KS = Slice<D>::kKeys;
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t full[kWarps][kStages], empty[kWarps][kStages];
  __shared__ int starts[TFX_ATTN_MAX_BATCH + 1];
  __shared__ int wsum[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWarps * kStages; i++) {
      mbar_init(&full[0][0] + i, 1);
      mbar_init(&empty[0][0] + i, 1);
    }
    fence_mbar_init();
  }
  // after the tensor-core kernel, this one starts where that leaves room: they
  // share no memory that is written, and that one lets this one start only when
  // all that came before has ended
  if (!a.pre_splits) griddep_wait();
  const Walk w = walk_of<KS, 16>(a, sequence_starts<KS, kWarps>(a, starts, wsum));
  const long long per = max((w.total + a.warps - 1) / a.warps, (long long)kFewest);
  note_runs(a, w, starts, per);
  griddep_launch();
  uint8_t* base = dyn + ((1024u - (s_addr(dyn) & 1023u)) & 1023u);
  auto ring_of = [&](int r) {
    Ring rg;
    rg.buf = base + r * kStages * Slice<D>::kStage;
    rg.full = full[r];
    rg.empty = empty[r];
    return rg;
  };
  bool ok = true;
  if (warp == kWarps) {
    if (lane < kWarps) {
      Ring rg = ring_of(lane);
      const long long x = ((long long)lane * gridDim.x + blockIdx.x) * per;
      ok = feed<D>(a, w, starts, rg, x, min(x + per, w.total));
    }
  } else {
    Ring rg = ring_of(warp);
    // neighbouring runs go to neighbouring CTAs: few runs still use every SM
    const int me = warp * gridDim.x + blockIdx.x;
    long long x = me * per;
    const long long end = min(x + per, w.total);
    const T* q = reinterpret_cast<const T*>(a.q);
    Rows<T, D> R;
    Segment g;
    auto begin = [&]() {  // the segment at x: its rows of q are asked for
      g = segment_at<Slice<D>::kKeys, 16>(a, w, starts, x, end);
      const T* rp[2];
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int r = (lane >> 2) + 8 * h;
        const bool in = r < g.rows;
        const int row = in ? g.row0 + r : g.row0, i = g.prefix ? row / a.group : g.seq;
        const int head = g.head * a.group + (g.prefix ? row % a.group : row);
        rp[h] = in ? q + (long long)i * a.ldq + (long long)head * D : nullptr;
        const int len = seq_len(a, i);
        R.hi[h] = !g.prefix ? len : in ? min(a.shared, len) : 0;
      }
      R.load(rp[0], rp[1], lane);
    };
    if (x < end) begin();
    while (ok && x < end) {
      R.reset();
      ok = attend<T, D>(R, rg, g.s0, g.s1, g.prefix ? 0 : a.shared, a.scale_log2, lane, a.spin);
      if (!ok) break;
      const long long slot = me + g.group;
      float* po = g.prefix ? a.pre_o + slot * 16 * D : a.own_o + slot * a.own_rows * D;
      float2* pml = g.prefix ? a.pre_ml + slot * 16 : a.own_ml + slot * a.own_rows;
      const int rows = g.rows;
      x += g.s1 - g.s0;
      if (x < end) begin();  // the next segment's q is on its way while this one's result is stored
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int r = (lane >> 2) + 8 * h;
        if (r >= rows) continue;
        if ((lane & 3) == 0) pml[r] = make_float2(R.m[h], R.l[h]);
#pragma unroll
        for (int i = 0; i < D / 8; i++)
          *reinterpret_cast<float2*>(po + (long long)r * D + i * 8 + 2 * (lane & 3)) =
              make_float2(R.o[i][2 * h], R.o[i][2 * h + 1]);
      }
      __syncwarp();
    }
  }
  if (!ok) gave_up(a.err);
  if (a.pre_splits) griddep_wait();  // this grid's end says to the next that both are done
}

// One CTA per (sequence, query head): the row's partial results, prefix first,
// in slot order. Each of W warps joins every W-th one, then theirs are joined.
template <typename T, int D, int W>
__global__ void __launch_bounds__(W * 32) decode_join_kernel(const __grid_constant__ DecodeAttnArgs a) {
  constexpr int V = D / 32;  // values of a row per lane, as V/4 runs of 4
  constexpr int kBatch = 6;  // partial results in flight a warp
  __shared__ float so[W][D];
  __shared__ float2 sml[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x / a.heads_q, head = blockIdx.x - i * a.heads_q;
  const int kvh = head / a.group, gh = head % a.group, r = i * a.group + gh;
  const int tiles = (a.group + 15) / 16, ptiles = (a.batch * a.group + 15) / 16;
  const int hr = kvh * tiles + gh / 16, grp = kvh * ptiles + r / 16;
  const bool pre = a.shared > 0 && !a.pre_splits;
  const int len = seq_len(a, i);  // nothing since the launch before the last one writes lengths
  griddep_wait();
  const int2 own = a.runs[(pre ? a.heads_kv * ptiles : 0) + hr * a.batch + i];
  const int2 first = pre ? a.runs[grp] : make_int2(0, 0);
  float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int c = 0; c < V; c++) o[c] = 0.f;
  // the row's partial results: shares of the prefix, runs of the prefix, runs of its own tokens
  const int shares = a.pre_splits, all = shares + first.y + own.y;
  const long long pre0 = (long long)(first.x + grp) * 16 + r % 16;
  const long long own0 = ((long long)own.x + (long long)hr * a.batch + i) * a.own_rows + gh % 16;
  for (int z0 = warp; z0 < all; z0 += W * kBatch) {
    float2 ml[kBatch];
    float4 x[kBatch][V / 4];
#pragma unroll
    for (int k = 0; k < kBatch; k++) {
      const int z = min(z0 + k * W, all - 1), y = z - shares;
      const bool mine = y >= first.y;
      const long long row = y < 0    ? (long long)z * a.batch * a.heads_q + blockIdx.x
                            : mine ? own0 + (long long)(y - first.y) * a.own_rows
                                   : pre0 + y * 16;
      ml[k] = (mine ? a.own_ml : a.pre_ml)[row];
      const float* po = (mine ? a.own_o : a.pre_o) + row * D + lane * 4;
#pragma unroll
      for (int c = 0; c < V / 4; c++) x[k][c] = *reinterpret_cast<const float4*>(po + c * 128);
      if (z0 + k * W >= all) ml[k] = make_float2(-INFINITY, 0.f);  // past the end: no weight
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < kBatch; k++) mn = fmaxf(mn, ml[k].x);
    const float ref = mn == -INFINITY ? 0.f : mn, f = exp2_fast(m - ref);
    l *= f;
#pragma unroll
    for (int c = 0; c < V; c++) o[c] *= f;
#pragma unroll
    for (int k = 0; k < kBatch; k++) {
      if (z0 + k * W >= all) break;
      const float g = exp2_fast(ml[k].x - ref);
      l += ml[k].y * g;
#pragma unroll
      for (int c = 0; c < V / 4; c++) {
        o[c * 4] += x[k][c].x * g;
        o[c * 4 + 1] += x[k][c].y * g;
        o[c * 4 + 2] += x[k][c].z * g;
        o[c * 4 + 3] += x[k][c].w * g;
      }
    }
    m = mn;
  }
  griddep_launch();
#pragma unroll
  for (int c = 0; c < V; c++) so[warp][(c >> 2) * 128 + lane * 4 + (c & 3)] = o[c];
  if (lane == 0) sml[warp] = make_float2(m, l);
  __syncthreads();
  float mn = -INFINITY, sum = 0.f, f[W];
  for (int k = 0; k < W; k++) mn = fmaxf(mn, sml[k].x);
  const float ref = mn == -INFINITY ? 0.f : mn;
#pragma unroll
  for (int k = 0; k < W; k++) {
    f[k] = exp2_fast(sml[k].x - ref);
    sum += sml[k].y * f[k];
  }
  const float inv = 1.f / sum;
  T* out = reinterpret_cast<T*>(a.out) + (long long)i * a.ldo + (long long)head * D;
  for (int c = threadIdx.x * 2; c < D; c += W * 64) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int k = 0; k < W; k++) {
      x += so[k][c] * f[k];
      y += so[k][c + 1] * f[k];
    }
    // a mean of values of 8-bit codes can be beyond FP16; of BF16's only where FP32 sums overflow, which shows as infinity
    const uint32_t w = __is_same(T, __half) && a.k_scale ? pack2_finite<T>(x * inv, y * inv) : pack2<T>(x * inv, y * inv);
    // a sequence without tokens: zeros
    *reinterpret_cast<uint32_t*>(out + c) = len == 0 ? 0u : w;
  }
}

template <typename T, int D, int W = kWarps>
int join_of(const DecodeAttnArgs& a, cudaStream_t s) {
  return launch_kernel((const void*)decode_join_kernel<T, D, W>, dim3((unsigned)(a.batch * a.heads_q)), dim3(W * 32), 0, s,
                       const_cast<DecodeAttnArgs*>(&a), dependent_launches(), 1);
}

template <typename T, int D>
int decode_of(const DecodeAttnArgs& a, cudaStream_t s) {
  const void* fn = (const void*)decode_warp_kernel<T, D>;
  int rc = opt_in_smem(fn, warp_smem<D>());
  if (rc) return rc;
  rc = launch_kernel(fn, dim3((unsigned)(a.warps / kWarps)), dim3(kThreads), warp_smem<D>(), s,
                     const_cast<DecodeAttnArgs*>(&a), dependent_launches(), 1);
  return rc ? rc : join_of<T, D>(a, s);
}

}  // namespace

int launch_join(const DecodeAttnArgs& a, int act, int dim, bool wide, cudaStream_t s) {
  if (wide) {
    if (act == TFX_F16) return dim == 128 ? join_of<__half, 128, 16>(a, s) : join_of<__half, 256, 16>(a, s);
    return dim == 128 ? join_of<__nv_bfloat16, 128, 16>(a, s) : join_of<__nv_bfloat16, 256, 16>(a, s);
  }
  if (act == TFX_F16) return dim == 128 ? join_of<__half, 128>(a, s) : join_of<__half, 256>(a, s);
  return dim == 128 ? join_of<__nv_bfloat16, 128>(a, s) : join_of<__nv_bfloat16, 256>(a, s);
}

int launch_decode(const DecodeAttnArgs& a, int act, int dim, cudaStream_t s) {
  if (act == TFX_F16) return dim == 128 ? decode_of<__half, 128>(a, s) : decode_of<__half, 256>(a, s);
  return dim == 128 ? decode_of<__nv_bfloat16, 128>(a, s) : decode_of<__nv_bfloat16, 256>(a, s);
}

}  // namespace tfx
