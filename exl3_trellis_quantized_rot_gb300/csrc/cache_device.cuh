// Device helpers shared by the cache kernels.
#pragma once
#include <climits>

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

// The same for the rows t0 .. t0 + rows - 1 (up to 32), a lane a row: the entries from the
// first row's on are looked at together, in a short list all of them.
__device__ __forceinline__ int entries_of(const int* offsets, int n, int t0, int rows) {
  const int lane = threadIdx.x & 31;
  const int i0 = n <= 32 ? 0 : entry_of(offsets, n, t0);
  if (rows == 1 && n > 32) return i0;
  const int ends = i0 + 1 + lane < n ? offsets[i0 + 1 + lane] : INT_MAX;
  int mine = i0;
  for (int r = 0; r < rows; r++) {
    const int k = __popc(__ballot_sync(~0u, ends <= t0 + r));
    const int i = k < 32 ? i0 + k : entry_of(offsets, n, t0 + r);  // behind 32 empty entries or more
    if (lane == r) mine = i;
  }
  return mine;
}

// Where row t of an append goes: the number of its token in the layer's pool, -1 where
// it has no place; its position, and its list entry's rows (an end of -1: there should be a
// place). A row of a slot that its extend refused has said so; any other without a place
// leaves a status bit.
struct Place {
  int to, pos, begin, end;
};
__device__ __forceinline__ Place place_in(const AppendArgs& a, const int* offsets, int i, int t) {
  Place x = {-1, 0, offsets[i], offsets[i + 1]};
  const int s = (a.seqs ? a.seqs : a.grown.seqs)[i];
  if (t < x.begin || t >= x.end) return x;
  const int2 mark = (unsigned)s < (unsigned)a.slots ? a.grown.mark[s] : make_int2(0, 0);
  if (mark.y < 0) return x;
  int page = -1;
  x.pos = mark.x + (t - x.begin);
  if (mark.y == x.end - x.begin && x.pos / a.page_size < a.width)
    page = a.table[(long long)s * a.width + x.pos / a.page_size];
  if (page >= 0 && page < a.pages) x.to = page * a.page_size + x.pos % a.page_size;
  else x.end = -1;
  return x;
}
__device__ __forceinline__ Place place_of(const AppendArgs& a, int t) {
  const int n = a.seqs ? a.n : *a.grown.n;
  const int* offsets = a.seqs ? a.offsets : a.grown.offsets;
  if (n < 1) return {-1, 0, 0, 0};
  const Place x = place_in(a, offsets, entry_of(offsets, n, t), t);
  if (x.end < 0 && (threadIdx.x & 31) == 0) atomicOr(&a.book[0], TFX_CACHE_BAD);
  return x;
}
// A lane a row, t0 .. t0 + rows - 1, up to 32.
__device__ __forceinline__ Place places_of(const AppendArgs& a, int t0, int rows) {
  const int n = a.seqs ? a.n : *a.grown.n;
  const int* offsets = a.seqs ? a.offsets : a.grown.offsets;
  if (n < 1) return {-1, 0, 0, 0};
  const int i = entries_of(offsets, n, t0, rows), r = threadIdx.x & 31;
  if (r >= rows) return {-1, 0, 0, 0};
  const Place x = place_in(a, offsets, i, t0 + r);
  if (x.end < 0) atomicOr(&a.book[0], TFX_CACHE_BAD);
  return x;
}

}  // namespace tfx
