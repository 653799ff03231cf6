// Keys and values quantised as they are appended, and rows read back.
//
// A block is 16 tokens of one head of K or V under one scale (codes.cuh). An append
// touches a block's bytes once: a warp takes the block's new values, their largest
// magnitude, and with it the scale; codes that the block holds already are rounded again
// only where the scale grows.
#include <cuda_runtime.h>

#include "attn_device.cuh"
#include "cache_device.cuh"
#include "codes.cuh"
#include "exl3_kernels.cuh"

namespace tfx {
namespace {

constexpr int kBlock = TFX_CACHE_BLOCK;
constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kMostRows = 16;  // rows of the list that a CTA looks at

// A CTA looks at a.per rows of the list. A row that is the first of its block's new tokens
// stands for the block, also where the block's tokens go on past the CTA's rows. A warp takes
// 256 values of a block's tokens (a lane 8 of each token): one head of 256 or two of 128.
template <typename T, int Store, int D>
__global__ void __launch_bounds__(kAppendThreads, 2) append_q8_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ int first[kMostRows], to[kMostRows], fresh[kMostRows], blocks;
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * a.per, rows = min(a.per, a.rows - t0);
  if (threadIdx.x == 0) blocks = 0;
  __syncthreads();
  for (int r = warp; r < rows; r += kAppendWarps) {
    const Place at = place_of(a, t0 + r);
    const int in = at.pos % kBlock;
    if (lane == 0 && at.to >= 0 && (t0 + r == at.begin || in == 0)) {
      const int i = atomicAdd(&blocks, 1);  // in any order
      first[i] = t0 + r;
      to[i] = at.to;
      fresh[i] = min(min(kBlock - in, at.end - t0 - r), a.rows - t0 - r);
    }
  }
  __syncthreads();
  const int row = a.heads * D, parts = (row + 255) / 256;
  for (int it = warp; it < blocks * 2 * parts; it += kAppendWarps) {
    const int i = it / (2 * parts), rest = it - i * 2 * parts;
    const bool value = rest >= parts;
    const int at = (value ? rest - parts : rest) * 256 + lane * 8;
    const bool mine = at < row;
    const int t = first[i], n = fresh[i], in = to[i] % kBlock;
    const long long block = to[i] / kBlock;
    const long long ld = value ? a.ldv : a.ldk;  // words of 8 values
    const uint4* src = reinterpret_cast<const uint4*>(value ? a.v_new : a.k_new) + t * ld + at / 8;
    uint2* codes = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(value ? a.v : a.k) + block * kBlock * row + at);
    float* scales = (value ? a.v_scale : a.k_scale) + block * a.heads + at / D;
    uint4 x[kBlock];
#pragma unroll
    for (int j = 0; j < kBlock; j++) x[j] = mine && j < n ? __ldcs(src + j * ld) : make_uint4(0, 0, 0, 0);
    const float before = mine && in ? *scales : 0.f;
    // magnitudes as the type's bits: their order is that of the values, and NaN is above all
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kBlock; j++) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int k = 0; k < 4; k++) top = __vmaxu2(top, w[k] & 0x7fff7fffu);
    }
    top = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int d = D / 16; d; d >>= 1) top = max(top, __shfl_xor_sync(~0u, top, d));
    const float2 most = pair_to_float(top, T());
    const float scale = larger_scale(before, scale_for<Store>(__float_as_uint(most.x)));
    const float inv = inverse_of(scale);
    if (mine && in && scale != before) {
      const float by = before * inv;
      for (int j = 0; j < in; j++) {
        uint2 c = codes[(long long)j * row / 8];
        float f[4], g[4];
        values4<Store>(c.x, f);
        values4<Store>(c.y, g);
        c.x = code4<Store>(f[0] * by, f[1] * by, f[2] * by, f[3] * by);
        c.y = code4<Store>(g[0] * by, g[1] * by, g[2] * by, g[3] * by);
        codes[(long long)j * row / 8] = c;
      }
    }
#pragma unroll
    for (int j = 0; j < kBlock; j++)
      if (mine && j < n) {
        const float2 p = pair_to_float(x[j].x, T()), q = pair_to_float(x[j].y, T());
        const float2 r = pair_to_float(x[j].z, T()), s = pair_to_float(x[j].w, T());
        codes[(long long)(in + j) * row / 8] = make_uint2(code4<Store>(p.x * inv, p.y * inv, q.x * inv, q.y * inv),
                                                          code4<Store>(r.x * inv, r.y * inv, s.x * inv, s.y * inv));
      }
    if (mine && at % D == 0) *scales = scale;
  }
}

constexpr int kReadThreads = 256;

// A CTA does a.per rows: a warp finds one row's place, then all threads take 16 bytes of a row
// of K or V at a time, four of them in flight.
template <typename T, int Store>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int kValues = Store == TFX_STORE_ACT ? 8 : 16;  // in 16 bytes
  __shared__ long long to[kMostRows];  // a token of the pool; -1: none, -2: the row is in no list
  griddep_wait();
  griddep_launch();
  const int t0 = blockIdx.x * a.per, rows = min(a.per, a.rows - t0);
  for (int r = threadIdx.x >> 5; r < rows; r += kReadThreads / 32) {
    const int t = t0 + r, i = entry_of(a.offsets, a.n, t);
    const int begin = a.offsets[i], end = a.offsets[i + 1], s = a.seqs[i];
    const long long pos = (long long)a.starts[i] + (t - begin);
    int page = -1;
    if ((unsigned)s < (unsigned)a.slots && pos >= 0 && pos < a.lens[s] && pos / a.page_size < a.width)
      page = a.table[(long long)s * a.width + pos / a.page_size];
    if (threadIdx.x % 32 == 0) {
      const bool listed = t >= begin && t < end, there = page >= 0 && page < a.pages;
      to[r] = !listed ? -2 : there ? (long long)page * a.page_size + pos % a.page_size : -1;
      if (listed && !there) atomicOr(&a.book[0], TFX_CACHE_BAD);
    }
  }
  __syncthreads();
  const int words = a.heads * a.dim / kValues, all = rows * 2 * words;
  constexpr int kAhead = 4;
  for (int c0 = threadIdx.x; c0 < all; c0 += kReadThreads * kAhead) {
    uint4 x[kAhead];
    float scale[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      const int c = c0 + j * kReadThreads, r = c / (2 * words), rest = c - r * 2 * words;
      const bool value = rest >= words;
      const int w = value ? rest - words : rest;
      const long long from = c < all ? to[r] : -2;
      x[j] = make_uint4(0, 0, 0, 0);
      scale[j] = 0.f;
      if (from < 0) continue;
      x[j] = __ldcs(reinterpret_cast<const uint4*>(value ? a.v : a.k) + from * words + w);
      if (Store != TFX_STORE_ACT) scale[j] = (value ? a.v_scale : a.k_scale)[from / kBlock * a.heads + w * kValues / a.dim];
    }
#pragma unroll
    for (int j = 0; j < kAhead; j++) {
      const int c = c0 + j * kReadThreads, r = c / (2 * words), rest = c - r * 2 * words;
      const bool value = rest >= words;
      const int w = value ? rest - words : rest;
      if (c >= all || to[r] == -2) continue;
      uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<T*>(value ? a.v_out : a.k_out) +
                                            (long long)(t0 + r) * (value ? a.ldv : a.ldk) + w * kValues);
      if constexpr (Store == TFX_STORE_ACT) {
        __stcs(out, x[j]);
      } else {
        const uint32_t code[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 4; k++) {
          float f[4];
          values4<Store>(code[k], f);
          y[2 * k] = pack2<T>(f[0] * scale[j], f[1] * scale[j]);
          y[2 * k + 1] = pack2<T>(f[2] * scale[j], f[3] * scale[j]);
        }
        __stcs(out, make_uint4(y[0], y[1], y[2], y[3]));
        __stcs(out + 1, make_uint4(y[4], y[5], y[6], y[7]));
      }
    }
  }
}

template <typename T, int Store>
const void* append_of(int dim) {
  return dim == 128 ? (const void*)append_q8_kernel<T, Store, 128> : (const void*)append_q8_kernel<T, Store, 256>;
}

}  // namespace

// Rows that a CTA does: one where that leaves every SM `most` CTAs at most, else so many more.
static int rows_per_cta(long long rows, int most) {
  const long long per = (rows + multiprocessors() * most - 1) / (multiprocessors() * most);
  return (int)(per < 1 ? 1 : per > kMostRows ? kMostRows : per);
}

int launch_append_q8(AppendArgs& a, int act, int store, int dim, cudaStream_t s) {
  a.per = rows_per_cta(a.rows, 2);
  const void* fn = store == TFX_STORE_I8
                       ? act == TFX_F16 ? append_of<__half, TFX_STORE_I8>(dim) : append_of<__nv_bfloat16, TFX_STORE_I8>(dim)
                   : act == TFX_F16 ? append_of<__half, TFX_STORE_E4M3>(dim)
                                    : append_of<__nv_bfloat16, TFX_STORE_E4M3>(dim);
  return launch_kernel(fn, dim3((unsigned)((a.rows + a.per - 1) / a.per)), dim3(kAppendThreads), 0, s, &a,
                       dependent_launches(), 1);
}

int launch_read(ReadArgs& a, int act, int store, cudaStream_t s) {
  a.per = rows_per_cta(a.rows, 8);
  const void* fn;
  if (store == TFX_STORE_ACT)  // 16 bits either way
    fn = (const void*)read_kernel<__half, TFX_STORE_ACT>;
  else if (store == TFX_STORE_I8)
    fn = act == TFX_F16 ? (const void*)read_kernel<__half, TFX_STORE_I8> : (const void*)read_kernel<__nv_bfloat16, TFX_STORE_I8>;
  else
    fn = act == TFX_F16 ? (const void*)read_kernel<__half, TFX_STORE_E4M3>
                        : (const void*)read_kernel<__nv_bfloat16, TFX_STORE_E4M3>;
  return launch_kernel(fn, dim3((unsigned)((a.rows + (long long)a.per - 1) / a.per)), dim3(kReadThreads), 0, s, &a,
                       dependent_launches(), 1);
}

}  // namespace tfx
