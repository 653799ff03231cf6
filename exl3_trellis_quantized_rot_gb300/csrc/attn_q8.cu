// Attention of single tokens over a cache of 8-bit codes.
//
//   s_j = scale q . c_j ks(j),  p = softmax(s),  o = sum_j p_j vs(j) d_j,
// c_j, d_j the codes of K and V, ks and vs the scales of their blocks of 16 tokens.
#include <cuda_runtime.h>

#include "attn_device.cuh"
#include "codes.cuh"

namespace tfx {
namespace {

constexpr int kWarps = 4;

// One CTA per (sequence, query head): a warp every fourth token, a lane D/32 values.
template <typename T, int Store, int D>
__global__ void __launch_bounds__(kWarps * 32) decode_q8_kernel(const __grid_constant__ DecodeAttnArgs a) {
  constexpr int V = D / 32;
  __shared__ float so[kWarps][D];
  __shared__ float2 sml[kWarps];
  griddep_wait();
  griddep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x / a.heads_q, head = blockIdx.x - i * a.heads_q, kvh = head / a.group;
  const int len = seq_len(a, i);
  const int* shared_table = prefix_table(a);
  const int* table = len ? a.tables + (long long)a.seqs[i] * a.width : shared_table;
  const T* qr = reinterpret_cast<const T*>(a.q) + (long long)i * a.ldq + (long long)head * D + lane * V;
  float q[V], o[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < V; c++) {
    q[c] = (float)qr[c] * a.scale_log2;
    o[c] = 0.f;
  }
  for (int j = warp; j < len; j += kWarps) {
    const int page = (j < a.shared ? shared_table : table)[j >> a.page_shift];
    if ((unsigned)page >= (unsigned)a.pages) continue;
    const long long tok = ((long long)page << a.page_shift) + (j & (a.page_size - 1));
    const long long at = (tok * a.heads_kv + kvh) * D + lane * V;
    const float ks = a.k_scale[tok / 16 * a.heads_kv + kvh], vs = a.v_scale[tok / 16 * a.heads_kv + kvh];
    float dot = 0.f;
#pragma unroll
    for (int w = 0; w < V / 4; w++) {
      float f[4];
      values4<Store>(*reinterpret_cast<const uint32_t*>(a.codes_k + at + 4 * w), f);
#pragma unroll
      for (int c = 0; c < 4; c++) dot += q[4 * w + c] * f[c];
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(~0u, dot, d);
    const float s = dot * ks, mn = fmaxf(m, s), keep = exp2_fast(m - mn), p = exp2_fast(s - mn);
    m = mn;
    l = l * keep + p;
#pragma unroll
    for (int w = 0; w < V / 4; w++) {
      float f[4];
      values4<Store>(*reinterpret_cast<const uint32_t*>(a.codes_v + at + 4 * w), f);
#pragma unroll
      for (int c = 0; c < 4; c++) o[4 * w + c] = o[4 * w + c] * keep + p * vs * f[c];
    }
  }
#pragma unroll
  for (int c = 0; c < V; c++) so[warp][lane * V + c] = o[c];
  if (lane == 0) sml[warp] = make_float2(m, l);
  __syncthreads();
  float mn = -INFINITY, sum = 0.f;
  for (int k = 0; k < kWarps; k++) mn = fmaxf(mn, sml[k].x);
  const float ref = mn == -INFINITY ? 0.f : mn;
  for (int k = 0; k < kWarps; k++) sum += sml[k].y * exp2_fast(sml[k].x - ref);
  T* out = reinterpret_cast<T*>(a.out) + (long long)i * a.ldo + (long long)head * D;
  for (int c = threadIdx.x * 2; c < D; c += kWarps * 64) {
    float x = 0.f, y = 0.f;
    for (int k = 0; k < kWarps; k++) {
      const float f = exp2_fast(sml[k].x - ref);
      x += so[k][c] * f;
      y += so[k][c + 1] * f;
    }
    // a sequence without tokens: zeros
    *reinterpret_cast<uint32_t*>(out + c) = len == 0 ? 0u : pack2<T>(x / sum, y / sum);
  }
}

template <typename T, int Store>
const void* kernel_of(int dim) {
  return dim == 128 ? (const void*)decode_q8_kernel<T, Store, 128> : (const void*)decode_q8_kernel<T, Store, 256>;
}

}  // namespace

int launch_decode_q8(const DecodeAttnArgs& a, int act, int store, int dim, cudaStream_t s) {
  const void* fn = store == TFX_STORE_I8
                       ? act == TFX_F16 ? kernel_of<__half, TFX_STORE_I8>(dim) : kernel_of<__nv_bfloat16, TFX_STORE_I8>(dim)
                   : act == TFX_F16 ? kernel_of<__half, TFX_STORE_E4M3>(dim)
                                    : kernel_of<__nv_bfloat16, TFX_STORE_E4M3>(dim);
  return launch_kernel(fn, dim3((unsigned)(a.batch * a.heads_q)), dim3(kWarps * 32), 0, s, const_cast<DecodeAttnArgs*>(&a),
                       dependent_launches(), 1);
}

}  // namespace tfx
