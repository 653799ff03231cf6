// Attention by single warps: 16 rows against slices of keys, m16n8k16 MMAs.
//
//   m' = max(m, max_j s_j),  p_j = 2^(s_j - m'),  l' = l 2^(m - m') + sum_j p_j,
//   o' = o 2^(m - m') + sum_j p_j v_j,            s_j = scale log2(e) q . k_j,
// one pass over the keys; the row's result is o / l. A warp owns its rows, its
// slices and its own ring of shared-memory stages, so warps never wait for
// one another. Partial results (o, m, l) of several warps are joined by
// decode_join_kernel in slot order.
//
// A slice is 16 KB of K and V of one K/V head (16 keys of 256, 32 of 128),
// fetched by two to four tensor copies of 16 tokens each with the 128-byte
// swizzle, so that the 8x8 matrix loads of K (rows = keys) and V (transposed)
// meet no bank twice.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_device.cuh"
#include "attn_internal.h"

namespace tfx {
namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;

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

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
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
#pragma unroll
    for (int i = 0; i < D / 8; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) o[i][j] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }
};

// The ring of one warp: stages of one slice each, refilled by lane 0.
struct Ring {
  uint8_t* buf;
  uint64_t* full;
  int it = 0;  // slices consumed so far: stage it % kStages, phase it / kStages
};

// Where the tokens are: token t of a paged sequence is in page table[t / page_size];
// without a table the tokens are rows base, base + 1, ... of one long "page".
struct Keys {
  const CUtensorMap *k, *v;
  const int* table;
  int page_shift, pages, width;
  int base, head;
};

template <int D>
__device__ __forceinline__ void fetch(const Keys& ks, Ring& rg, int stage, int token, int entry) {
  uint8_t* dst = rg.buf + stage * Slice<D>::kStage;
  uint64_t* bar = rg.full + stage;
  mbar_expect_tx(bar, Slice<D>::kStage);
#pragma unroll
  for (int b = 0; b < Slice<D>::kKeys / 16; b++) {
    int page = 0, at = ks.base + token + 16 * b;
    if (ks.table) {
      const int p = (token + 16 * b) >> ks.page_shift;
      // a page can end inside a slice of 32 keys: its second half has an entry of its own
      page = b == 0 ? entry : p < ks.width ? __ldg(ks.table + p) : -1;
      page = page >= 0 && page < ks.pages ? page : -1;  // -1 is out of the map's range: zeros
      at = (token + 16 * b) & ((1 << ks.page_shift) - 1);
    }
    tma_load_5d(dst + b * Slice<D>::kBlock, ks.k, 0, at, 0, ks.head, page, bar);
    tma_load_5d(dst + Slice<D>::kHalf + b * Slice<D>::kBlock, ks.v, 0, at, 0, ks.head, page, bar);
  }
}

// The rows against slices [s0, s1) of the keys lo <= key < hi. False: a wait gave up.
template <typename T, int D>
__device__ __forceinline__ bool attend(Rows<T, D>& R, const Keys& ks, Ring& rg, int s0, int s1, int lo, float scale,
                                       int lane, long long spin) {
  constexpr int KS = Slice<D>::kKeys;
  const int g = lane >> 2, t = lane & 3, mi = lane >> 3, mr = lane & 7;
  int hmin = min(R.hi[0], R.hi[1]), hmax = max(R.hi[0], R.hi[1]);
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    hmin = min(hmin, __shfl_xor_sync(~0u, hmin, d));
    hmax = max(hmax, __shfl_xor_sync(~0u, hmax, d));
  }
  // page-table entries of the slices ahead, one per lane
  int tb = -1, held = 0;
  auto entry_of = [&](int token) -> int {
    if (!ks.table) return 0;
    const int p = token >> ks.page_shift;
    if (tb < 0 || p >= tb + 32) {
      tb = p;
      held = p + lane < ks.width ? __ldg(ks.table + p + lane) : -1;
    }
    return __shfl_sync(~0u, held, p - tb);
  };
  const int it0 = rg.it;
  for (int i = 0; i < kStages && s0 + i < s1; i++) {
    const int e = entry_of((s0 + i) * KS);
    if (lane == 0) fetch<D>(ks, rg, (it0 + i) % kStages, (s0 + i) * KS, e);
  }
  for (int s = s0; s < s1; s++) {
    const int st = rg.it % kStages;
    if (!mbar_wait_bounded(rg.full + st, (rg.it / kStages) & 1, spin)) return false;
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
      __syncwarp();
    }
    // S = Q K^T; two chains per tile of 8 keys
    float sc[KS / 8][4];
    {
      float s2[KS / 8][4];
#pragma unroll
      for (int j = 0; j < KS / 8; j++)
#pragma unroll
        for (int c = 0; c < 4; c++) sc[j][c] = s2[j][c] = 0.f;
      const int key = (mi >> 1) * 8 + mr;
#pragma unroll
      for (int i = 0; i < D / 16; i++) {
        const int c = i * 2 + (mi & 1);  // 16-byte column of 8 values
#pragma unroll
        for (int b = 0; b < KS / 16; b++) {
          uint32_t f[4];
          ldsm4(f, s_addr(kb) + b * Slice<D>::kBlock + (c >> 3) * 2048 + key * 128 + (((c & 7) ^ (key & 7)) << 4));
          if (i & 1) {
            mma<T>(s2[2 * b], R.q[i], f[0], f[1]);
            mma<T>(s2[2 * b + 1], R.q[i], f[2], f[3]);
          } else {
            mma<T>(sc[2 * b], R.q[i], f[0], f[1]);
            mma<T>(sc[2 * b + 1], R.q[i], f[2], f[3]);
          }
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
    uint32_t p[KS / 16][4];
#pragma unroll
    for (int b = 0; b < KS / 16; b++)
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
#pragma unroll
    for (int b = 0; b < KS / 16; b++)
#pragma unroll
      for (int i = 0; i < D / 16; i++) {
        const int c = i * 2 + (mi >> 1);
        uint32_t f[4];
        ldsm4t(f, s_addr(vb) + b * Slice<D>::kBlock + (c >> 3) * 2048 + vkey * 128 + (((c & 7) ^ (vkey & 7)) << 4));
        mma<T>(R.o[2 * i], p[b], f[0], f[1]);
        mma<T>(R.o[2 * i + 1], p[b], f[2], f[3]);
      }
    fence_async_smem();  // zeroed rows are ordinary stores to memory that the next copy writes
    __syncwarp();
    if (s + kStages < s1) {
      const int e = entry_of((s + kStages) * KS);
      if (lane == 0) fetch<D>(ks, rg, st, (s + kStages) * KS, e);
    }
    rg.it++;
  }
#pragma unroll
  for (int h = 0; h < 2; h++) {
    R.l[h] += __shfl_xor_sync(~0u, R.l[h], 1);
    R.l[h] += __shfl_xor_sync(~0u, R.l[h], 2);
  }
  return true;
}

// Shared memory of this warp and its barriers; every thread of the CTA calls it.
template <int D>
__device__ __forceinline__ Ring make_ring(uint8_t* dyn, uint64_t (*full)[kStages], int warp, int lane) {
  uint8_t* base = dyn + ((1024u - (s_addr(dyn) & 1023u)) & 1023u);
  if (lane == 0) {
    for (int i = 0; i < kStages; i++) mbar_init(&full[warp][i], 1);
    fence_mbar_init();
  }
  __syncthreads();
  Ring r;
  r.buf = base + warp * kStages * Slice<D>::kStage;
  r.full = full[warp];
  return r;
}

// After a wait that gave up: the error word, and time for the copies in flight to land.
__device__ __forceinline__ void gave_up(int* err, int lane) {
  if (lane == 0) atomicExch(err, 1);
  const long long t0 = clock64();
  while (clock64() - t0 < 2000000) __nanosleep(1000);
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) decode_warp_kernel(const __grid_constant__ DecodeAttnArgs a) {
  constexpr int KS = Slice<D>::kKeys;
  extern __shared__ uint8_t dyn[];
  __shared__ uint64_t full[kWarps][kStages];
  __shared__ int starts[TFX_ATTN_MAX_BATCH + 1];
  __shared__ int wsum[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // after the tensor-core kernel, this one starts where that leaves room: they
  // share no memory that is written, and that one began after all that came before
  if (!a.pre_splits) griddep_wait();
  Ring rg = make_ring<D>(dyn, full, warp, lane);
  // own slices before each sequence
  int carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kWarps * 32) {
    const int i = b0 + threadIdx.x;
    const int len = i < a.batch ? seq_len(a, i) : 0;
    const int mine = len > a.shared ? (len + KS - 1) / KS - a.shared / KS : 0;
    int x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int before = carry, all = carry;
    for (int w = 0; w < kWarps; w++) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    if (i < a.batch) starts[i + 1] = before + x;
    carry = all;
    __syncthreads();
  }
  if (threadIdx.x == 0) starts[0] = 0;
  __syncthreads();
  const int own = starts[a.batch];
  const int tiles = (a.group + 15) / 16, ptiles = (a.batch * a.group + 15) / 16;
  const int sp = a.pre_splits ? 0 : (a.shared + KS - 1) / KS;
  const long long pre_total = (long long)a.heads_kv * ptiles * sp;
  const long long total = pre_total + (long long)a.heads_kv * tiles * own;
  const long long per = max((total + a.warps - 1) / a.warps, 4LL);
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= a.batch; i += kWarps * 32) a.starts[i] = starts[i];
    if (threadIdx.x == 0) a.starts[a.batch + 1] = (int)per;
  }
  griddep_launch();
  const int w = blockIdx.x * kWarps + warp;
  long long x = w * per;
  const long long end = min(x + per, total);
  const T* q = reinterpret_cast<const T*>(a.q);
  while (x < end) {
    Rows<T, D> R;
    const T* rp[2] = {nullptr, nullptr};
    Keys ks = {&a.k, &a.v, nullptr, a.page_shift, a.pages, a.width, 0, 0};
    int s0, s1, lo, rows;
    float* po;
    float2* pml;
    if (x < pre_total) {
      const int grp = (int)(x / sp), tile = grp % ptiles;
      s0 = (int)(x % sp);
      s1 = (int)min((long long)sp, s0 + (end - x));
      lo = 0;
      ks.head = grp / ptiles;
      const int s = a.seqs[0];
      ks.table = a.tables + (long long)(s >= 0 && s < a.slots ? s : 0) * a.width;
      rows = min(16, a.batch * a.group - tile * 16);
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int r = tile * 16 + (lane >> 2) + 8 * h;
        const bool in = r < a.batch * a.group;
        const int i = in ? r / a.group : 0;
        rp[h] = in ? q + (long long)i * a.ldq + (long long)(ks.head * a.group + r % a.group) * D : nullptr;
        R.hi[h] = in ? min(a.shared, seq_len(a, i)) : 0;
      }
      po = a.pre_o + ((long long)w + grp) * 16 * D;
      pml = a.pre_ml + ((long long)w + grp) * 16;
    } else {
      const long long y = x - pre_total;
      const int hr = (int)(y / own), z = (int)(y % own), tile = hr % tiles;
      int lo_i = 0, hi_i = a.batch - 1;  // the sequence that slice z belongs to
      while (lo_i < hi_i) {
        const int mid = (lo_i + hi_i) >> 1;
        if (starts[mid + 1] > z) hi_i = mid; else lo_i = mid + 1;
      }
      const int i = lo_i, off = a.shared / KS;
      s0 = z - starts[i] + off;
      s1 = (int)min((long long)(starts[i + 1] - starts[i] + off), s0 + (end - x));
      lo = a.shared;
      ks.head = hr / tiles;
      ks.table = a.tables + (long long)a.seqs[i] * a.width;
      rows = min(16, a.group - tile * 16);
      const int len = seq_len(a, i);
#pragma unroll
      for (int h = 0; h < 2; h++) {
        const int r = tile * 16 + (lane >> 2) + 8 * h;
        const bool in = r < a.group;
        rp[h] = in ? q + (long long)i * a.ldq + (long long)(ks.head * a.group + r) * D : nullptr;
        R.hi[h] = len;
      }
      const long long slot = (long long)w + (long long)hr * a.batch + i;
      po = a.own_o + slot * a.own_rows * D;
      pml = a.own_ml + slot * a.own_rows;
    }
    R.load(rp[0], rp[1], lane);
    if (!attend<T, D>(R, ks, rg, s0, s1, lo, a.scale_log2, lane, a.spin)) {
      gave_up(a.err, lane);
      return;
    }
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
    x += s1 - s0;
  }
  if (a.pre_splits) griddep_wait();  // this grid's end says to the next that both are done
}

// One CTA per (sequence, query head): the row's partial results, prefix first,
// in slot order. Each warp joins every fourth one, then the four are joined.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) decode_join_kernel(const __grid_constant__ DecodeAttnArgs a) {
  constexpr int KS = Slice<D>::kKeys;
  constexpr int V = D / 32;  // values of a row per lane, as V/4 runs of 4
  __shared__ float so[kWarps][D];
  __shared__ float2 sml[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_wait();
  const int i = blockIdx.x / a.heads_q, head = blockIdx.x % a.heads_q;
  const int kvh = head / a.group, gh = head % a.group;
  const int tiles = (a.group + 15) / 16, ptiles = (a.batch * a.group + 15) / 16;
  const int sp = a.pre_splits ? 0 : (a.shared + KS - 1) / KS, own = a.starts[a.batch];
  const long long per = a.starts[a.batch + 1];
  const long long pre_total = (long long)a.heads_kv * ptiles * sp;
  float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int c = 0; c < V; c++) o[c] = 0.f;
  auto take = [&](const float* po, float2 ml) {
    const float mn = fmaxf(m, ml.x), ref = mn == -INFINITY ? 0.f : mn;
    const float f = exp2_fast(m - ref), g = exp2_fast(ml.x - ref);
    l = l * f + ml.y * g;
#pragma unroll
    for (int c = 0; c < V / 4; c++) {
      const float4 x = *reinterpret_cast<const float4*>(po + c * 128 + lane * 4);
      o[c * 4] = o[c * 4] * f + x.x * g;
      o[c * 4 + 1] = o[c * 4 + 1] * f + x.y * g;
      o[c * 4 + 2] = o[c * 4 + 2] * f + x.z * g;
      o[c * 4 + 3] = o[c * 4 + 3] * f + x.w * g;
    }
    m = mn;
  };
  for (int z = warp; z < a.pre_splits; z += kWarps) {
    const long long row = (long long)z * a.batch * a.heads_q + blockIdx.x;
    take(a.pre_o + row * D, a.pre_ml[row]);
  }
  if (sp) {
    const int r = i * a.group + gh, grp = kvh * ptiles + r / 16;
    const long long x0 = (long long)grp * sp, x1 = x0 + sp;
    for (long long w = x0 / per + warp; w <= (x1 - 1) / per; w += kWarps) {
      const long long row = (w + grp) * 16 + r % 16;
      take(a.pre_o + row * D, a.pre_ml[row]);
    }
  }
  const int n = a.starts[i + 1] - a.starts[i];
  if (n) {
    const int hr = kvh * tiles + gh / 16;
    const long long x0 = pre_total + (long long)hr * own + a.starts[i], x1 = x0 + n;
    for (long long w = x0 / per + warp; w <= (x1 - 1) / per; w += kWarps) {
      const long long row = (w + (long long)hr * a.batch + i) * a.own_rows + gh % 16;
      take(a.own_o + row * D, a.own_ml[row]);
    }
  }
  griddep_launch();
#pragma unroll
  for (int c = 0; c < V; c++) so[warp][(c >> 2) * 128 + lane * 4 + (c & 3)] = o[c];
  if (lane == 0) sml[warp] = make_float2(m, l);
  __syncthreads();
  float mn = -INFINITY, sum = 0.f, f[kWarps];
  for (int w = 0; w < kWarps; w++) mn = fmaxf(mn, sml[w].x);
  const float ref = mn == -INFINITY ? 0.f : mn;
#pragma unroll
  for (int w = 0; w < kWarps; w++) {
    f[w] = exp2_fast(sml[w].x - ref);
    sum += sml[w].y * f[w];
  }
  const bool none = seq_len(a, i) == 0;  // a sequence without tokens: zeros
  const float inv = 1.f / sum;
  T* out = reinterpret_cast<T*>(a.out) + (long long)i * a.ldo + (long long)head * D;
  for (int c = threadIdx.x * 2; c < D; c += kWarps * 64) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      x += so[w][c] * f[w];
      y += so[w][c + 1] * f[w];
    }
    *reinterpret_cast<uint32_t*>(out + c) = none ? 0u : pack2<T>(x * inv, y * inv);
  }
}

template <typename T, int D>
int decode_of(const DecodeAttnArgs& a, cudaStream_t s) {
  const void* fn = (const void*)decode_warp_kernel<T, D>;
  int rc = opt_in_smem(fn, warp_smem<D>());
  if (rc) return rc;
  rc = launch_kernel(fn, dim3((unsigned)(a.warps / kWarps)), dim3(kWarps * 32), warp_smem<D>(), s,
                     const_cast<DecodeAttnArgs*>(&a), a.pre_splits > 0, 1);
  if (rc) return rc;
  return launch_kernel((const void*)decode_join_kernel<T, D>, dim3((unsigned)(a.batch * a.heads_q)), dim3(kWarps * 32), 0,
                       s, const_cast<DecodeAttnArgs*>(&a), true, 1);
}

}  // namespace

int launch_decode(const DecodeAttnArgs& a, int act, int dim, cudaStream_t s) {
  if (act == TFX_F16) return dim == 128 ? decode_of<__half, 128>(a, s) : decode_of<__half, 256>(a, s);
  return dim == 128 ? decode_of<__nv_bfloat16, 128>(a, s) : decode_of<__nv_bfloat16, 256>(a, s);
}

}  // namespace tfx
