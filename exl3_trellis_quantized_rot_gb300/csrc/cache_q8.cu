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
constexpr int kAppendWarps = 8;

// One CTA per row of the list; the row that is the first of a block's new tokens does
// the block. A warp a head of K or V; a lane holds D/32 values of a token.
template <typename T, int Store, int D>
__global__ void __launch_bounds__(kAppendWarps * 32) append_q8_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int V = D / 32, W = V / 2;  // values and words of a lane
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x;
  const Place at = place_of(a, t);
  const int in = at.pos % kBlock;
  if (at.to < 0 || (t != at.begin && in)) return;
  const int fresh = min(min(kBlock - in, at.end - t), a.rows - t);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = a.heads * D;
  const long long block = at.to / kBlock;
  for (int it = warp; it < 2 * a.heads; it += kAppendWarps) {
    const bool value = it >= a.heads;
    const int head = value ? it - a.heads : it;
    const T* src = reinterpret_cast<const T*>(value ? a.v_new : a.k_new) + (long long)t * (value ? a.ldv : a.ldk) * 8 +
                   head * D + lane * V;
    uint8_t* codes = reinterpret_cast<uint8_t*>(value ? a.v : a.k) + block * kBlock * row + head * D + lane * V;
    float* scales = (value ? a.v_scale : a.k_scale) + block * a.heads + head;
    const long long ld = (value ? a.ldv : a.ldk) * 8;
    uint32_t x[kBlock][W];
#pragma unroll
    for (int i = 0; i < kBlock; i++)
      if (i < fresh) {
        if constexpr (W == 4)
          *reinterpret_cast<uint4*>(x[i]) = *reinterpret_cast<const uint4*>(src + i * ld);
        else
          *reinterpret_cast<uint2*>(x[i]) = *reinterpret_cast<const uint2*>(src + i * ld);
      }
    const float before = in ? *scales : 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kBlock; i++)
      if (i < fresh)
#pragma unroll
        for (int w = 0; w < W; w++) {
          const float2 f = pair_to_float(x[i][w], T());
          top = max(top, max(__float_as_uint(fabsf(f.x)), __float_as_uint(fabsf(f.y))));
        }
    const float scale = larger_scale(before, scale_for<Store>(__reduce_max_sync(~0u, top)));
    const float inv = inverse_of(scale);
    if (in && scale != before) {
      const float by = before * inv;
      for (int i = 0; i < in; i++) {
        uint32_t* c = reinterpret_cast<uint32_t*>(codes + (long long)i * row);
#pragma unroll
        for (int w = 0; w < W / 2; w++) {
          float f[4];
          values4<Store>(c[w], f);
          c[w] = code4<Store>(f[0] * by, f[1] * by, f[2] * by, f[3] * by);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBlock; i++)
      if (i < fresh) {
        uint32_t* c = reinterpret_cast<uint32_t*>(codes + (long long)(in + i) * row);
#pragma unroll
        for (int w = 0; w < W / 2; w++) {
          const float2 f = pair_to_float(x[i][2 * w], T()), g = pair_to_float(x[i][2 * w + 1], T());
          c[w] = code4<Store>(f.x * inv, f.y * inv, g.x * inv, g.y * inv);
        }
      }
    if (lane == 0) *scales = scale;
  }
}

constexpr int kReadThreads = 128;

// One CTA per row.
template <typename T, int Store>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadArgs a) {
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x;
  const int i = entry_of(a.offsets, a.n, t);
  const int begin = a.offsets[i], s = a.seqs[i];
  if (t < begin || t >= a.offsets[i + 1]) return;
  const long long pos = (long long)a.starts[i] + (t - begin);
  int page = -1;
  if ((unsigned)s < (unsigned)a.slots && pos >= 0 && pos < a.lens[s] && pos / a.page_size < a.width)
    page = a.table[(long long)s * a.width + pos / a.page_size];
  const bool there = page >= 0 && page < a.pages;
  if (!there && threadIdx.x == 0) atomicOr(&a.book[0], TFX_CACHE_BAD);
  const int row = a.heads * a.dim, words = row / 8;  // words of 8 values
  const long long to = there ? (long long)page * a.page_size + pos % a.page_size : 0;
  for (int c = threadIdx.x; c < 2 * words; c += kReadThreads) {
    const bool value = c >= words;
    const int w = value ? c - words : c;
    uint4 y = make_uint4(0, 0, 0, 0);
    if (there) {
      const void* pool = value ? a.v : a.k;
      if constexpr (Store == TFX_STORE_ACT) {
        y = reinterpret_cast<const uint4*>(pool)[to * words + w];
      } else {
        const uint2 x = reinterpret_cast<const uint2*>(pool)[to * words + w];
        const float scale = (value ? a.v_scale : a.k_scale)[to / kBlock * a.heads + w * 8 / a.dim];
        float f[4], g[4];
        values4<Store>(x.x, f);
        values4<Store>(x.y, g);
        y = make_uint4(pack2<T>(f[0] * scale, f[1] * scale), pack2<T>(f[2] * scale, f[3] * scale),
                       pack2<T>(g[0] * scale, g[1] * scale), pack2<T>(g[2] * scale, g[3] * scale));
      }
    }
    T* out = reinterpret_cast<T*>(value ? a.v_out : a.k_out) + (long long)t * (value ? a.ldv : a.ldk);
    reinterpret_cast<uint4*>(out)[w] = y;
  }
}

template <typename T, int Store>
const void* append_of(int dim) {
  return dim == 128 ? (const void*)append_q8_kernel<T, Store, 128> : (const void*)append_q8_kernel<T, Store, 256>;
}

}  // namespace

int launch_append_q8(const AppendArgs& a, int act, int store, int dim, int rows, cudaStream_t s) {
  const void* fn = store == TFX_STORE_I8
                       ? act == TFX_F16 ? append_of<__half, TFX_STORE_I8>(dim) : append_of<__nv_bfloat16, TFX_STORE_I8>(dim)
                   : act == TFX_F16 ? append_of<__half, TFX_STORE_E4M3>(dim)
                                    : append_of<__nv_bfloat16, TFX_STORE_E4M3>(dim);
  return launch_kernel(fn, dim3((unsigned)rows), dim3(kAppendWarps * 32), 0, s, const_cast<AppendArgs*>(&a),
                       dependent_launches(), 1);
}

int launch_read(const ReadArgs& a, int act, int store, cudaStream_t s) {
  const void* fn;
  if (store == TFX_STORE_ACT)  // 16 bits either way
    fn = (const void*)read_kernel<__half, TFX_STORE_ACT>;
  else if (store == TFX_STORE_I8)
    fn = act == TFX_F16 ? (const void*)read_kernel<__half, TFX_STORE_I8> : (const void*)read_kernel<__nv_bfloat16, TFX_STORE_I8>;
  else
    fn = act == TFX_F16 ? (const void*)read_kernel<__half, TFX_STORE_E4M3>
                        : (const void*)read_kernel<__nv_bfloat16, TFX_STORE_E4M3>;
  return launch_kernel(fn, dim3((unsigned)a.rows), dim3(kReadThreads), 0, s, const_cast<ReadArgs*>(&a), dependent_launches(), 1);
}

}  // namespace tfx
