// Device helpers shared by the cache kernels.
#pragma once
#include "attn_internal.h"

namespace tfx {

// The entry of a list of n > 0 (offsets not decreasing) that row t is of, by a warp:
// 32 entries a step. Whether the row is in it at all is the caller's to look at.
__device__ __forceinline__ int entry_of(const int* offsets, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32, x = lane * step;
    const int k = max(__popc(__ballot_sync(~0u, x < len && offsets[lo + x] <= t)) - 1, 0);
    lo += k * step;
    len = min(step, len - k * step);
  }
  return lo;
}

// Where row t of an append goes: the number of its token in the layer's pool, -1 where
// it has no place; its position, and the end of its list entry's rows. By a warp. A row of a
// slot that its extend refused has said so; any other without a place leaves a status bit.
struct Place {
  int to, pos, begin, end;
};
__device__ __forceinline__ Place place_of(const AppendArgs& a, int t) {
  const int n = a.seqs ? a.n : *a.grown.n;
  const int* offsets = a.seqs ? a.offsets : a.grown.offsets;
  Place x = {-1, 0, 0, 0};
  if (n < 1) return x;
  const int i = entry_of(offsets, n, t);
  x.begin = offsets[i];
  x.end = offsets[i + 1];
  const int s = (a.seqs ? a.seqs : a.grown.seqs)[i];
  if (t < x.begin || t >= x.end) return x;
  const int2 mark = (unsigned)s < (unsigned)a.slots ? a.grown.mark[s] : make_int2(0, 0);
  if (mark.y < 0) return x;
  int page = -1;
  x.pos = mark.x + (t - x.begin);
  if (mark.y == x.end - x.begin && x.pos / a.page_size < a.width)
    page = a.table[(long long)s * a.width + x.pos / a.page_size];
  if (page < 0 || page >= a.pages) {
    if ((threadIdx.x & 31) == 0) atomicOr(&a.book[0], TFX_CACHE_BAD);
    return x;
  }
  x.to = page * a.page_size + x.pos % a.page_size;
  return x;
}

}  // namespace tfx
