// Rotary positions of packed rows.
//
//   (a, b) -> g (a cos w - b sin w, b cos w + a sin w),  w = n f_i.
// An angle is held as a fraction of a turn in 64 bits: f_i / 2 pi as F_i / 2^64, so
// n F_i mod 2^64 is the angle without its whole turns, exactly but for F_i's own rounding.
// Its top 32 bits, as a signed number of half turns, go to sincospi.
//
// Bound: memory at large sizes: 16,384 rows of 24 + 4 heads of 256 (470 MB) take 76.7 us, 6.1 TB/s, 4,097 rows of
// 48 + 8 of 128 (118 MB, partly in L2) 22.3. 64 rows: 2.4 us, position, frequency and sine one after
// another. A row a CTA: CTAs that go from row to row took 29 us where this took 22.7.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/tfx_rope.h"
#include "attn_device.cuh"
#include "codes.cuh"

namespace tfx {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4;  // of an SM: five and six keep fewer words in registers and are slower (16,384 rows: 76.8, 78.3, 79.3 us)
constexpr int kMostRotary = 2048;
constexpr uint32_t kSide = 1u << 31;
constexpr int kCopies = 3;  // words that a thread copies at a time

struct RopeArgs {
  const uint64_t* table;
  const void* in[2];  // q, k
  void* out[2];
  long long ld_in[2], ld_out[2];
  const int* positions;
  int heads[2];
  int dim, rotary, rows;
  float gain, sine;  // factors of cosine and sine
  int copy;          // whether the values behind the rotated ones are written
};

// One CTA per row. Items of a head: rotary/16 pairs of 16-byte words (half) or rotary/8 words
// (interleaved). A thread asks for its first items, and copies what is only copied, before it
// works out its share of the row's sines.
template <typename T, bool Interleaved>
__global__ void __launch_bounds__(kThreads, kCtas) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kAhead = Interleaved ? 4 : 2;
  __shared__ __align__(16) float cosine[kMostRotary / 2], sine[kMostRotary / 2];
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x, half = a.rotary / 2;
  const int turned = Interleaved ? a.rotary / 8 : a.rotary / 16;
  const int all = (a.heads[0] + a.heads[1]) * turned;
  const T* in[2];
  T* out[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    in[i] = reinterpret_cast<const T*>(a.in[i]) + t * a.ld_in[i];
    out[i] = reinterpret_cast<T*>(a.out[i]) + t * a.ld_out[i];
  }
  uint4 x[kAhead], y[Interleaved ? 1 : kAhead];
  uint32_t place[kAhead];  // the first value's number in the row, and whether it is k's
  // Item or word `it` of `per` a head: its place where a head's first is at `at0`.
  auto place_of = [&](int it, int per, int at0) {
    const int h = it / per, side = h >= a.heads[0];
    return (uint32_t)((side ? h - a.heads[0] : h) * a.dim + at0 + (it - h * per) * 8) | (side ? kSide : 0u);
  };
  auto ask = [&](int it0) {
#pragma unroll
    for (int n = 0; n < kAhead; n++) {
      const int it = it0 + n * kThreads;
      if (it >= all) break;
      place[n] = place_of(it, turned, 0);
      const T* from = (place[n] & kSide ? in[1] : in[0]) + (place[n] & ~kSide);
      x[n] = *reinterpret_cast<const uint4*>(from);
      if (!Interleaved) y[Interleaved ? 0 : n] = *reinterpret_cast<const uint4*>(from + half);
    }
  };
  ask(threadIdx.x);
  if (a.copy) {
    const int rest = (a.dim - a.rotary) / 8, words = (a.heads[0] + a.heads[1]) * rest;
    for (int c0 = threadIdx.x; c0 < words; c0 += kThreads * kCopies) {
      uint4 w[kCopies];
      uint32_t at[kCopies];
#pragma unroll
      for (int n = 0; n < kCopies; n++)
        if (c0 + n * kThreads < words) {
          at[n] = place_of(c0 + n * kThreads, rest, a.rotary);
          w[n] = *reinterpret_cast<const uint4*>((at[n] & kSide ? in[1] : in[0]) + (at[n] & ~kSide));
        }
#pragma unroll
      for (int n = 0; n < kCopies; n++)
        if (c0 + n * kThreads < words) *reinterpret_cast<uint4*>((at[n] & kSide ? out[1] : out[0]) + (at[n] & ~kSide)) = w[n];
    }
  }
  const long long position = a.positions[t];
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const uint64_t turn = (uint64_t)position * a.table[i];
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31
    cosine[i] = c * a.gain;
    sine[i] = s * a.sine;
  }
  __syncthreads();
  for (int it0 = threadIdx.x; it0 < all; it0 += kThreads * kAhead) {
    if (it0 != threadIdx.x) ask(it0);
#pragma unroll
    for (int n = 0; n < kAhead; n++) {
      if (it0 + n * kThreads >= all) break;
      const int at = (int)(place[n] & ~kSide), word = at % a.dim / 8;
      T* to = (place[n] & kSide ? out[1] : out[0]) + at;
      uint32_t v[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
      if constexpr (Interleaved) {
        const float4 c = *reinterpret_cast<const float4*>(cosine + word * 4);
        const float4 s = *reinterpret_cast<const float4*>(sine + word * 4);
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float2 f = pair_to_float(v[k], T());
          v[k] = pack2<T>(f.x * cs[k] - f.y * sn[k], f.y * cs[k] + f.x * sn[k]);
        }
      } else {
        uint32_t u[4] = {y[n].x, y[n].y, y[n].z, y[n].w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const float2 f = pair_to_float(v[k], T()), g = pair_to_float(u[k], T());
          const float2 c = *reinterpret_cast<const float2*>(cosine + word * 8 + 2 * k);
          const float2 s = *reinterpret_cast<const float2*>(sine + word * 8 + 2 * k);
          v[k] = pack2<T>(f.x * c.x - g.x * s.x, f.y * c.y - g.y * s.y);
          u[k] = pack2<T>(g.x * c.x + f.x * s.x, g.y * c.y + f.y * s.y);
        }
        *reinterpret_cast<uint4*>(to + half) = make_uint4(u[0], u[1], u[2], u[3]);
      }
      *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

}  // namespace
}  // namespace tfx

namespace {

using tfx::fail_with;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_side(const char* what, const void* p, int64_t ld, const void* out, int64_t ldo, int64_t width) {
  if (!p || !out) return fail_with(TFX_EINVAL, "null %s or its output", what);
  if (ld < width || ldo < width)
    return fail_with(TFX_EINVAL, "pitches %lld and %lld of %s below its %lld values", (long long)ld, (long long)ldo, what,
                     (long long)width);
  if (ld > (1LL << 36) || ldo > (1LL << 36)) return fail_with(TFX_EINVAL, "pitch %lld or %lld of %s", (long long)ld, (long long)ldo, what);
  if (ld % 8 || ldo % 8 || !aligned16(p) || !aligned16(out))
    return fail_with(TFX_EALIGN, "%s and its output: 16-byte aligned pointers and pitches of whole 8 values", what);
  if (p == out && ld != ldo) return fail_with(TFX_EINVAL, "%s in place with two pitches", what);
  return 0;
}

}  // namespace

extern "C" {

int tfx_rope_table(const double* freqs, int n, uint64_t* table) {
  if (n < 0 || (n && (!freqs || !table))) return fail_with(TFX_EINVAL, "n=%d, or a null list", n);
  for (int i = 0; i < n; i++)
    if (!std::isfinite(freqs[i])) return fail_with(TFX_EINVAL, "freqs[%d] is not finite", i);
  for (int i = 0; i < n; i++) {
    const double turns = freqs[i] / 6.283185307179586;
    const double part = turns - std::floor(turns);  // [0, 1], 1 where a tiny negative one is rounded up
    table[i] = part < 1.0 ? (uint64_t)std::ldexp(part, 64) : 0;
  }
  return 0;
}

int tfx_rope_apply(const tfx_rope* r, int act, int dim, const void* q, int64_t ldq, int heads_q, void* q_out, int64_t ldqo,
                   const void* k, int64_t ldk, int heads_k, void* k_out, int64_t ldko, const int32_t* positions, int rows,
                   int inverse, cudaStream_t stream) {
  if (!r || !r->table) return fail_with(TFX_EINVAL, "null rope or table");
  if (act != TFX_F16 && act != TFX_BF16) return fail_with(TFX_EINVAL, "act=%d", act);
  if (dim < 16 || dim > 65536) return fail_with(TFX_EINVAL, "dim=%d outside 16..65536", dim);
  if (dim % 8) return fail_with(TFX_EALIGN, "dim=%d is not a multiple of 8", dim);
  if (r->rotary < 16 || r->rotary % 16 || r->rotary > dim || r->rotary > tfx::kMostRotary)
    return fail_with(TFX_EUNSUPPORTED, "rotary=%d of dim=%d: a multiple of 16, at most %d", r->rotary, dim, tfx::kMostRotary);
  if (!std::isfinite(r->gain)) return fail_with(TFX_EINVAL, "gain=%g", (double)r->gain);
  if (heads_q < 1 || heads_k < 0 || heads_q > 65535 || heads_k > 65535 || ((int64_t)heads_q + heads_k) * dim > (1 << 30))
    return fail_with(TFX_EINVAL, "heads_q=%d, heads_k=%d of %d values", heads_q, heads_k, dim);
  if (rows < 0) return fail_with(TFX_EINVAL, "rows=%d", rows);
  if (!rows) return 0;
  int rc = check_side("q", q, ldq, q_out, ldqo, (int64_t)heads_q * dim);
  if (rc) return rc;
  if (heads_k && (rc = check_side("k", k, ldk, k_out, ldko, (int64_t)heads_k * dim))) return rc;
  // a row's items are written while others are still read
  if (heads_k && (q_out == k || k_out == q || k_out == q_out))
    return fail_with(TFX_EINVAL, "an output is the other one, or the other's input");
  if (!positions) return fail_with(TFX_EINVAL, "null positions");
  if (reinterpret_cast<uintptr_t>(positions) & 3u || reinterpret_cast<uintptr_t>(r->table) & 7u)
    return fail_with(TFX_EALIGN, "positions or table is not aligned");
  tfx::RopeArgs a = {};
  a.table = r->table;
  a.in[0] = q;
  a.in[1] = k;
  a.out[0] = q_out;
  a.out[1] = k_out;
  a.ld_in[0] = ldq;
  a.ld_in[1] = ldk;
  a.ld_out[0] = ldqo;
  a.ld_out[1] = ldko;
  a.positions = positions;
  a.heads[0] = heads_q;
  a.heads[1] = heads_k;
  a.dim = dim;
  a.rotary = r->rotary;
  a.rows = rows;
  a.gain = r->gain;
  a.sine = inverse ? -r->gain : r->gain;
  a.copy = q != q_out || (heads_k && k != k_out);
  const void* fn = r->interleaved ? act == TFX_F16 ? (const void*)tfx::rope_kernel<__half, true>
                                                   : (const void*)tfx::rope_kernel<__nv_bfloat16, true>
                   : act == TFX_F16 ? (const void*)tfx::rope_kernel<__half, false>
                                    : (const void*)tfx::rope_kernel<__nv_bfloat16, false>;
  return tfx::launch_kernel(fn, dim3((unsigned)rows), dim3(tfx::kThreads), 0, stream, &a, tfx::dependent_launches(), 1);
}

}  // extern "C"
