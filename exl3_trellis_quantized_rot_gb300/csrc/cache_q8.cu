// Keys and values quantised as they are appended, and rows read back.
//
// A block is 16 tokens of one head of K or V under one scale (codes.cuh). An append
// touches a block's bytes once: a warp takes the block's new values, their largest
// magnitude, and with it the scale; codes that the block holds already are rounded again
// only where the scale grows.
//
// Bound: memory at large sizes: three prompts of 32,001 tokens (8 heads of 128) are appended in 39 us (131 MB
// read, 66 written; DRAM busy half the time, issue slots 41 %), 43,695 tokens (4 heads of 256) read back
// in 46 us (268 MB, 5.8 TB/s), out of 16-bit pages in 58 to 61 (358 MB, 5.8 to 6.2 TB/s). 64 single tokens: 3.4 us,
// 300 rows read: 3.1 us, the latency of lists, table, scale and codes one after another. It stands in front of the
// 3.7 us that the bytes of 4,096 tokens take, too (7.2 us, a window a CTA: nothing hides the first look-up). Two CTAs an SM hold a block in registers (128 a
// thread); copies into shared memory for eight warps an SM took 60 us where this took 46.
#include <cuda_runtime.h>

#include <type_traits>

#include "attn_device.cuh"
#include "cache_device.cuh"
#include "codes.cuh"
#include "exl3_kernels.cuh"

namespace tfx {
namespace {

constexpr int kBlock = TFX_CACHE_BLOCK;
constexpr int kMostRows = 32;  // rows of the list that are looked at together: a lane each
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Loads that stay where they are written: beside a test of their own the compiler moved them
// to the values' use, one wait after another (a read of 43,695 tokens: 68 us instead of 48).
__device__ __forceinline__ void load_here(uint2& x, const uint2* p) {
  asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "l"(p));
}
__device__ __forceinline__ void load_here(uint4& x, const uint4* p) {
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(p));
}

// The next of a window's tasks, for a warp.
__device__ __forceinline__ int take(int* taken) {
  int it = 0;
  if ((threadIdx.x & 31) == 0) it = atomicAdd(taken, 1);
  return __shfl_sync(~0u, it, 0);
}

template <typename T>
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b);  // of magnitudes; a NaN stays
template <>
__device__ __forceinline__ uint32_t larger2<__half>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{ .reg .b32 x; abs.f16x2 x, %2; max.NaN.f16x2 %0, %1, x; }" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <>
__device__ __forceinline__ uint32_t larger2<__nv_bfloat16>(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{ .reg .b32 x; abs.bf16x2 x, %2; max.NaN.bf16x2 %0, %1, x; }" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The blocks of a window of rows of a list: first row, first token of the pool (-1: none), and
// rows, up to 16 of one block.
struct Blocks {
  int first[kMostRows], rows[kMostRows];
  long long to[kMostRows];
  int n, taken;

  // By a warp, a lane a row: those that stand for a block.
  __device__ __forceinline__ void list(bool stands, int row, long long token, int count) {
    const int lane = threadIdx.x & 31;
    const unsigned all = __ballot_sync(~0u, stands);
    if (stands) {
      const int i = __popc(all & ((1u << lane) - 1));
      first[i] = row;
      to[i] = token;
      rows[i] = count;
    }
    if (lane == 0) {
      n = __popc(all);
      taken = kWarps;  // a warp's first one goes by its number
    }
  }
};

// A task's place: a lane has 8 values of each of up to 16 tokens. D: values of a head.
struct Task {
  int t, n, at, in;
  long long to, block;
  bool value, mine;
};
__device__ __forceinline__ Task task_of(const Blocks& w, int it, int parts, int row) {
  Task k;
  const int i = it / (2 * parts), rest = it - i * 2 * parts;
  k.value = rest >= parts;
  k.at = (k.value ? rest - parts : rest) * 256 + (threadIdx.x & 31) * 8;
  k.mine = k.at < row;
  k.t = w.first[i];
  k.n = w.rows[i];
  k.to = w.to[i];
  k.in = (int)(k.to & (kBlock - 1));
  k.block = k.to / kBlock;
  return k;
}

// Windows of a.per rows of the list. A row that is the first of its block's new tokens stands
// for the block, also where the block's tokens go on past the window. The first warp of a CTA
// looks up the next window's blocks while the others do this one's: the way from the lists to a
// page is five loads that wait for one another. A task is 256 values of a block's tokens: one
// head of 256 or two of 128.
template <typename T, int Store, int D>
__global__ void __launch_bounds__(kThreads, 2) append_q8_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ Blocks ring[2];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = a.heads * D, parts = (row + 255) / 256, step = row / 8;  // step: words of 8 values
  const int windows = (int)(((long long)a.rows + a.per - 1) / a.per);
  auto look_up = [&](int window, Blocks& w) {
    const int t0 = window * a.per, t = t0 + lane;
    const Place at = places_of(a, t0, min(a.per, a.rows - t0));
    const int in = at.pos % kBlock;
    w.list(at.to >= 0 && (t == at.begin || in == 0), t, at.to, min(min(kBlock - in, at.end - t), a.rows - t));
  };
  // Of up to `most` new tokens, or (whole) of 16. One token has code of its own: what is laid out
  // for 16 takes a warp that runs through it once longer to fetch than to run.
  auto run = [&](const Task& k, auto most_of, auto whole) {
    constexpr int kMost = decltype(most_of)::value;
    constexpr bool kWhole = decltype(whole)::value;
    const long long ld = k.value ? a.ldv : a.ldk;  // words of 8 values
    const uint4* src = reinterpret_cast<const uint4*>(k.value ? a.v_new : a.k_new) + k.t * ld + k.at / 8;
    uint2* codes = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(k.value ? a.v : a.k) + k.block * kBlock * row + k.at);
    float* scales = (k.value ? a.v_scale : a.k_scale) + k.block * a.heads + k.at / D;
    uint4 x[kMost];
#pragma unroll
    for (int j = 0; j < kMost; j++) {
      x[j] = make_uint4(0, 0, 0, 0);
      if (k.mine && (kWhole || j < k.n)) load_here(x[j], src + j * ld);
    }
    const float before = !kWhole && k.mine && k.in ? *scales : 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kMost; j++)
      top = larger2<T>(larger2<T>(larger2<T>(larger2<T>(top, x[j].x), x[j].y), x[j].z), x[j].w);
    // magnitudes as the type's bits: their order is that of the values, and NaN is above all
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int d = D / 16; d; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
    const float2 most = pair_to_float(top, T());
    const float scale = larger_scale(before, scale_for<Store>(__float_as_uint(most.x)));
    const float inv = inverse_of(scale);
    // a block of scale NaN holds zeros: rows that see nothing of it multiply its codes by 0
    const uint32_t keep = scale == scale ? ~0u : 0u;
    if (!kWhole && k.mine && k.in && scale != before) {
      const float by = before * inv;
      for (int j = 0; j < k.in; j++) {
        uint2 c = codes[j * step];
        float f[4], g[4];
        values4<Store>(c.x, f);
        values4<Store>(c.y, g);
        c.x = code4<Store>(f[0], f[1], f[2], f[3], by) & keep;
        c.y = code4<Store>(g[0], g[1], g[2], g[3], by) & keep;
        codes[j * step] = c;
      }
    }
    uint2* out = codes + (kWhole ? 0 : k.in * step);
#pragma unroll
    for (int j = 0; j < kMost; j++)
      if (k.mine && (kWhole || j < k.n)) {
        const float2 p = pair_to_float(x[j].x, T()), q = pair_to_float(x[j].y, T());
        const float2 r = pair_to_float(x[j].z, T()), s = pair_to_float(x[j].w, T());
        out[j * step] = make_uint2(code4<Store>(p.x, p.y, q.x, q.y, inv) & keep, code4<Store>(r.x, r.y, s.x, s.y, inv) & keep);
      }
    if (k.mine && k.at % D == 0) *scales = scale;
  };
  if (warp == 0) look_up(blockIdx.x, ring[0]);
  __syncthreads();
  int b = 0;
  for (int window = blockIdx.x; window < windows; window += gridDim.x, b ^= 1, __syncthreads()) {
    if (warp == 0 && window + (int)gridDim.x < windows) look_up(window + gridDim.x, ring[b ^ 1]);
    const int all = ring[b].n * 2 * parts;
    for (int it = warp; it < all; it = take(&ring[b].taken)) {
      const Task k = task_of(ring[b], it, parts, row);
      if (k.n == kBlock) run(k, std::integral_constant<int, kBlock>(), std::true_type());
      else if (k.n == 1) run(k, std::integral_constant<int, 1>(), std::false_type());
      else run(k, std::integral_constant<int, kBlock>(), std::false_type());
    }
  }
}

constexpr int read_ctas(int store) { return store == TFX_STORE_ACT ? 4 : 6; }  // of an SM
// Tokens that a lane of a read has asked for. 43,695 rows of 4 heads of 256 (us on the GPU): 8 tokens 47.6
// (E4M3 49.1), 4 45.8 to 46.3, 2 47.6; 4 of eight CTAs an SM 50.4, 8 of five and four 51 and 61.
constexpr int kAhead = 4;

// The same for rows that are read, a.span tokens of a block at a time: they lie together and
// have its scale.
// A row whose sequence does not hold its token stands for itself.
template <typename T, int Store, int D>
__global__ void __launch_bounds__(kThreads, read_ctas(Store)) read_kernel(const __grid_constant__ ReadArgs a) {
  using Word = typename std::conditional<Store == TFX_STORE_ACT, uint4, uint2>::type;  // 8 values
  __shared__ Blocks ring[2];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = a.heads * D, parts = (row + 255) / 256, step = row / 8;
  const int windows = (int)(((long long)a.rows + a.per - 1) / a.per);
  auto look_up = [&](int window, Blocks& w) {
    const int t0 = window * a.per, rows = min(a.per, a.rows - t0);
    const int i = entries_of(a.offsets, a.n, t0, rows), t = t0 + lane;
    const int begin = a.offsets[i], end = a.offsets[i + 1], s = a.seqs[i];
    const bool listed = lane < rows && t >= begin && t < end;
    const long long pos = (long long)a.starts[i] + (t - begin);
    int page = -1, len = 0;
    const long long column = pos >> a.page_shift;
    if (listed && (unsigned)s < (unsigned)a.slots && pos >= 0 && column < a.width) {
      len = a.lens[s];  // both at once
      page = a.table[(long long)s * a.width + column];
      if (pos >= len) page = -1;
    }
    const bool there = page >= 0 && page < a.pages;
    if (listed && !there) atomicOr(&a.book[0], TFX_CACHE_BAD);
    const int in = (int)(pos & (kBlock - 1));
    w.list(listed && (!there || t == begin || in % a.span == 0), t, there ? ((long long)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1)) : -1,
           there ? (int)min((long long)min(min(a.span - in % a.span, end - t), a.rows - t), len - pos) : 1);
  };
  if (warp == 0) look_up(blockIdx.x, ring[0]);
  __syncthreads();
  int b = 0;
  for (int window = blockIdx.x; window < windows; window += gridDim.x, b ^= 1, __syncthreads()) {
    if (warp == 0 && window + (int)gridDim.x < windows) look_up(window + gridDim.x, ring[b ^ 1]);
    const int all = ring[b].n * 2 * parts;
    for (int it = warp; it < all; it = take(&ring[b].taken)) {
      const Task k = task_of(ring[b], it, parts, row);
      if (!k.mine) continue;
      const long long ld = (k.value ? a.ldv : a.ldk) / 8;
      const Word* src = reinterpret_cast<const Word*>(k.value ? a.v : a.k) + k.to * step + k.at / 8;
      uint4* out = reinterpret_cast<uint4*>(k.value ? a.v_out : a.k_out) + k.t * ld + k.at / 8;
      const bool there = k.to >= 0;
      const float scale = Store != TFX_STORE_ACT && there ? (k.value ? a.v_scale : a.k_scale)[k.block * a.heads + k.at / D] : 0.f;
#pragma unroll 1
      for (int j0 = 0; j0 < k.n; j0 += kAhead, src += kAhead * step, out += kAhead * ld) {
        const int n = k.n - j0;
        Word x[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
          x[j] = Word{};
          if (there && j < n) load_here(x[j], src + j * step);
        }
#pragma unroll
        for (int j = 0; j < kAhead; j++)
          if (j < n) {
            if constexpr (Store == TFX_STORE_ACT) {
              __stcs(out + j * ld, x[j]);
            } else {
              float f[4], g[4];
              values4<Store>(x[j].x, f);
              values4<Store>(x[j].y, g);
              __stcs(out + j * ld, make_uint4(pack2_finite<T>(f[0] * scale, f[1] * scale), pack2_finite<T>(f[2] * scale, f[3] * scale),
                                              pack2_finite<T>(g[0] * scale, g[1] * scale), pack2_finite<T>(g[2] * scale, g[3] * scale)));
            }
          }
      }
    }
  }
}

template <typename T, int Store>
const void* read_of(int dim) {
  return dim == 128 ? (const void*)read_kernel<T, Store, 128> : (const void*)read_kernel<T, Store, 256>;
}
template <typename T, int Store>
const void* append_of(int dim) {
  return dim == 128 ? (const void*)append_q8_kernel<T, Store, 128> : (const void*)append_q8_kernel<T, Store, 256>;
}

// Rows of a window, where `ctas` CTAs share them, and the CTAs that have any.
int rows_per_window(long long rows, int ctas, int most) {
  const long long per = (rows + ctas - 1) / ctas;
  return (int)(per > most ? most : per);
}
unsigned ctas_of(long long rows, int per, int ctas) {
  const long long windows = (rows + per - 1) / per;
  return (unsigned)(windows < ctas ? windows : ctas);
}

}  // namespace

int launch_append_q8(AppendArgs& a, int act, int store, int dim, cudaStream_t s) {
  const int ctas = 2 * multiprocessors();
  a.per = rows_per_window(a.rows, ctas, kMostRows);
  const void* fn = store == TFX_STORE_I8
                       ? act == TFX_F16 ? append_of<__half, TFX_STORE_I8>(dim) : append_of<__nv_bfloat16, TFX_STORE_I8>(dim)
                   : act == TFX_F16 ? append_of<__half, TFX_STORE_E4M3>(dim)
                                    : append_of<__nv_bfloat16, TFX_STORE_E4M3>(dim);
  return launch_kernel(fn, dim3(ctas_of(a.rows, a.per, ctas)), dim3(kThreads), 0, s, &a, dependent_launches(), 1);
}

int launch_read(ReadArgs& a, int act, int store, cudaStream_t s) {
  const int ctas = read_ctas(store) * multiprocessors();
  a.per = rows_per_window(a.rows, ctas, kMostRows / 2);
  // Tokens of a task: as few as keep the SMs' first warps busy. Measured with 2, 4, 8, 16 tokens, 4
  // heads of 256 (us on the GPU, with 8 tokens asked for): 300 rows 3.2, 3.3, 3.9, 4.1; 2,000 rows 6.4,
  // 4.9, 5.6, 7.2; 4,096 rows 9.0, 7.2, 6.8, 8.8; 16,000 rows 28.0, 23.0, 21.3, 21.3; 43,695 rows 61.4,
  // 46.6, 48.3, 48.0. With 4, of 4, 8 and 16 tokens: 2,000 rows 5.2, 5.1, 5.2; 4,096 rows 7.0, 7.0, 9.3;
  // 16,000 rows 22.7, 22.6, 22.5; 43,695 rows 48.8, 46.3, 46.2.
  const long long warps = (long long)multiprocessors() * kWarps, parts = 2 * (((long long)a.heads * a.dim + 255) / 256);
  a.span = a.rows * parts < 4 * warps ? 2 : a.rows * parts < 24 * warps ? 4 : 8;
  const void* fn;
  if (store == TFX_STORE_ACT)  // 16 bits either way
    fn = read_of<__half, TFX_STORE_ACT>(a.dim);
  else if (store == TFX_STORE_I8)
    fn = act == TFX_F16 ? read_of<__half, TFX_STORE_I8>(a.dim) : read_of<__nv_bfloat16, TFX_STORE_I8>(a.dim);
  else
    fn = act == TFX_F16 ? read_of<__half, TFX_STORE_E4M3>(a.dim) : read_of<__nv_bfloat16, TFX_STORE_E4M3>(a.dim);
  return launch_kernel(fn, dim3(ctas_of(a.rows, a.per, ctas)), dim3(kThreads), 0, s, &a, dependent_launches(), 1);
}

}  // namespace tfx
