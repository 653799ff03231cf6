// Page operations of the K/V cache.
//
// A step is a book kernel (one CTA: who gets which page; the free pages in
// order are a running count over the reference counts) followed, where page
// contents move, by a copy kernel over all layers that reads the list of moves
// from the scratch. Appends work out for themselves where their rows go (extend and
// append of 4,096 rows: 12.0 us on the GPU, against 14.4 with a map made by extend's one
// CTA). Contents move at the memory's rate: 16-byte accesses, eight in flight a
// thread. Counts are integers, so the atomics on them give the same values in every order.
#include <cuda_runtime.h>

#include <climits>

#include "attn_internal.h"
#include "exl3_kernels.cuh"

namespace tfx {

namespace {

constexpr int kBookThreads = 1024;
constexpr int kPerThread = 8;  // pages a thread looks at in one round of the free-page scan
constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 8;

// Exclusive sum of v over the CTA's threads; *total is the whole sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int ws[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(~0u, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) ws[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = ws[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int z = __shfl_up_sync(~0u, y, d);
      if (lane >= d) y += z;
    }
    ws[lane] = y;
  }
  __syncthreads();
  *total = ws[31];
  return x - v + (warp ? ws[warp - 1] : 0);
}

// Lists the first `want` pages of reference count 0; returns how many there are (at most want).
__device__ __forceinline__ int list_free(const int* refs, int pages, int want, int* out) {
  int found = 0;
  for (int p0 = 0; p0 < pages && found < want; p0 += kBookThreads * kPerThread) {
    int r[kPerThread], n = 0;
    const int mine = p0 + threadIdx.x * kPerThread;
#pragma unroll
    for (int j = 0; j < kPerThread; j++) {
      r[j] = mine + j < pages ? refs[mine + j] : 1;
      n += r[j] == 0;
    }
    int all;
    int at = found + block_scan(n, &all);
#pragma unroll
    for (int j = 0; j < kPerThread; j++)
      if (r[j] == 0) {
        if (at < want) out[at] = mine + j;
        at++;
      }
    found += all;
  }
  __syncthreads();
  return min(found, want);
}

__device__ __forceinline__ int pages_for(const BookArgs& a, int tokens) {
  return (int)(((long long)tokens + a.page_size - 1) / a.page_size);
}
// A slot's length, -1 where slot or length is out of range.
__device__ __forceinline__ int held(const BookArgs& a, int s) {
  if (s < 0 || s >= a.slots) return -1;
  const int len = a.lens[s];
  return len >= 0 && pages_for(a, len) <= a.width ? len : -1;
}
// Tokens that entry i of a growth list adds to the `old` ones of its slot, and
// the pages that takes; a status bit where it cannot be done.
__device__ __forceinline__ int growth(const BookArgs& a, int i, int* slot, int* old, int* add, int* cnt) {
  const int b = a.list1[i], e = a.list1[i + 1];
  *slot = a.list0[i];
  *old = held(a, *slot);
  *add = e - b;
  *cnt = 0;
  if (*old < 0 || b < 0 || e < b || e > a.row_cap) return TFX_CACHE_BAD;
  if (*add > INT_MAX - *old || pages_for(a, *old + *add) > a.width) return TFX_CACHE_TABLE_FULL;
  *cnt = pages_for(a, *old + *add) - pages_for(a, *old);
  return 0;
}

__global__ void __launch_bounds__(kBookThreads) extend_kernel(const __grid_constant__ BookArgs a) {
  __shared__ int status, asked;
  griddep_wait();
  if (threadIdx.x == 0) status = asked = 0;
  __syncthreads();
  // pages that the list asks for
  int mine = 0;
  for (int i = threadIdx.x; i < a.n; i += kBookThreads) {
    int s, old, add, cnt;
    growth(a, i, &s, &old, &add, &cnt);
    mine += cnt;
  }
  atomicAdd(&asked, mine);
  __syncthreads();
  const int have = list_free(a.refs, a.pages, asked, a.free_list);
  int carry = 0;
  for (int i0 = 0; i0 < a.n; i0 += kBookThreads) {
    const int i = i0 + threadIdx.x;
    int s = 0, old = 0, add = 0, cnt = 0, bad = 0;
    if (i < a.n) bad = growth(a, i, &s, &old, &add, &cnt);
    int all;
    const int first = carry + block_scan(cnt, &all);
    if (cnt && first + cnt > have) bad = TFX_CACHE_FULL;
    if (i < a.n) {
      if (!bad) {
        int* row = a.tables + (long long)s * a.width + pages_for(a, old);
        for (int c = 0; c < cnt; c++) {
          const int p = a.free_list[first + c];
          row[c] = p;
          a.refs[p] = 1;
        }
        a.lens[s] = old + add;
      }
      // for the appends; a slot that asks for nothing keeps what it has
      if (s >= 0 && s < a.slots && (bad || add)) a.grown.mark[s] = bad ? make_int2(0, -1) : make_int2(old, add);
      a.grown.seqs[i] = s;
      a.grown.offsets[i] = a.list1[i];
    }
    if (bad) atomicOr(&status, bad);
    carry += all;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    *a.grown.n = a.n;
    a.grown.offsets[a.n] = a.n ? a.list1[a.n] : 0;
    if (status) a.book[0] |= status;
  }
  griddep_launch();
}

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

// One CTA per token: its K row and its V row. Where they go follows from the lists,
// the marks that extends left and the tables as they are now, so that other calls may come
// between an extend and its appends.
__global__ void __launch_bounds__(128) append_kernel(const __grid_constant__ AppendArgs a) {
  griddep_wait();
  griddep_launch();
  const int t = blockIdx.x;
  const int n = a.seqs ? a.n : *a.grown.n;
  const int* offsets = a.seqs ? a.offsets : a.grown.offsets;
  if (n < 1) return;
  const int i = entry_of(offsets, n, t);
  const int begin = offsets[i], end = offsets[i + 1], s = (a.seqs ? a.seqs : a.grown.seqs)[i];
  if (t < begin || t >= end) return;
  const int2 mark = (unsigned)s < (unsigned)a.slots ? a.grown.mark[s] : make_int2(0, 0);
  if (mark.y < 0) return;  // refused by its extend, which said so
  int page = -1;
  const int pos = mark.x + (t - begin);
  if (mark.y == end - begin && pos / a.page_size < a.width)
    page = a.table[(long long)s * a.width + pos / a.page_size];
  if (page < 0 || page >= a.pages) {
    if (threadIdx.x == 0) atomicOr(&a.book[0], TFX_CACHE_BAD);
    return;
  }
  const int to = page * a.page_size + pos % a.page_size;
  const uint4* ks = reinterpret_cast<const uint4*>(a.k_new) + (long long)t * a.ldk;
  const uint4* vs = reinterpret_cast<const uint4*>(a.v_new) + (long long)t * a.ldv;
  uint4* kd = reinterpret_cast<uint4*>(a.k) + (long long)to * a.row;
  uint4* vd = reinterpret_cast<uint4*>(a.v) + (long long)to * a.row;
  for (int c = threadIdx.x; c < a.row; c += 128) {
    const uint4 x = ks[c], y = vs[c];
    kd[c] = x;
    vd[c] = y;
  }
}

// Which free page each fork's partial page goes to; the new lengths.
__global__ void __launch_bounds__(kBookThreads) fork_book_kernel(const __grid_constant__ BookArgs a) {
  __shared__ int status, asked;
  griddep_wait();
  if (threadIdx.x == 0) status = asked = 0;
  __syncthreads();
  auto valid = [&](int i, int* s, int* d) {
    *s = a.list0[i];
    *d = a.list1[i];
    return *s != *d && held(a, *s) >= 0 && held(a, *d) == 0;
  };
  int mine = 0;
  for (int i = threadIdx.x; i < a.n; i += kBookThreads) {
    int s, d;
    if (valid(i, &s, &d)) mine += a.lens[s] % a.page_size != 0;
  }
  atomicAdd(&asked, mine);
  __syncthreads();
  const int have = list_free(a.refs, a.pages, asked, a.free_list);
  int carry = 0;
  for (int i0 = 0; i0 < a.n; i0 += kBookThreads) {
    const int i = i0 + threadIdx.x;
    int s = 0, d = 0, cnt = 0, len = 0, bad = 0;
    bool ok = false;
    if (i < a.n) {
      ok = valid(i, &s, &d);
      if (ok) {
        len = a.lens[s];
        cnt = len % a.page_size != 0;
      } else {
        bad = TFX_CACHE_BAD;
      }
    }
    int all;
    const int first = carry + block_scan(cnt, &all);  // the scan's barriers: every slot is read before one is written
    if (cnt && first + cnt > have) {
      ok = false;
      bad = TFX_CACHE_FULL;
    }
    if (i < a.n) {
      int from = -1, to = -1;
      if (ok) {
        if (cnt) {
          from = a.tables[(long long)s * a.width + len / a.page_size];
          to = a.free_list[first];
          a.refs[to] = 1;
          if (from < 0 || from >= a.pages) from = -1;
        }
        a.lens[d] = len;
        a.grown.mark[d] = make_int2(0, 0);
      }
      a.move_src[i] = from;
      a.move_dst[i] = to;
      a.start[i] = ok ? len : -1;
    }
    if (bad) atomicOr(&status, bad);
    carry += all;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    *a.count = a.n;
    if (status) a.book[0] |= status;
  }
  griddep_launch();
}

// Pages to the front: the moves, the counts, and where each page is afterwards.
// A count below zero is a caller's mistake and a free page: there are as many holes as movers.
__global__ void __launch_bounds__(kBookThreads) compact_book_kernel(const __grid_constant__ BookArgs a) {
  griddep_wait();
  int live = 0;
  for (int p = threadIdx.x; p < a.pages; p += kBookThreads) live += a.refs[p] > 0;
  int used;
  block_scan(live, &used);
  int holes = 0, movers = 0;
  for (int p0 = 0; p0 < a.pages; p0 += kBookThreads * kPerThread) {
    int r[kPerThread], h = 0, m = 0;
    const int mine = p0 + threadIdx.x * kPerThread;
#pragma unroll
    for (int j = 0; j < kPerThread; j++) {
      const int p = mine + j;
      r[j] = p < a.pages ? a.refs[p] : -1;
      h += r[j] <= 0 && p < used;
      m += r[j] > 0 && p >= used;
    }
    int hall, mall;
    int hat = holes + block_scan(h, &hall);
    int mat = movers + block_scan(m, &mall);
#pragma unroll
    for (int j = 0; j < kPerThread; j++) {
      const int p = mine + j;
      if (p >= a.pages) break;
      a.map[p] = p;
      if (r[j] <= 0 && p < used) a.move_dst[hat++] = p;
      if (r[j] > 0 && p >= used) a.move_src[mat++] = p;
    }
    holes += hall;
    movers += mall;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < movers; i += kBookThreads) {
    const int s = a.move_src[i], d = a.move_dst[i];
    a.map[s] = d;
    a.refs[d] = a.refs[s];
    a.refs[s] = 0;
  }
  if (threadIdx.x == 0) {
    *a.count = movers;
    a.book[1] = movers;
  }
  griddep_launch();
}

// One CTA per sequence. The exchange makes a slot that is listed twice give its pages back once.
__global__ void __launch_bounds__(256) free_kernel(const __grid_constant__ BookArgs a) {
  __shared__ int len;
  griddep_wait();
  griddep_launch();
  const int s = a.list0[blockIdx.x];
  if (s < 0 || s >= a.slots) {
    if (threadIdx.x == 0) atomicOr(&a.book[0], TFX_CACHE_BAD);
    return;
  }
  if (threadIdx.x == 0) {
    len = atomicExch(&a.lens[s], 0);
    a.grown.mark[s] = make_int2(0, 0);
  }
  __syncthreads();
  int* row = a.tables + (long long)s * a.width;
  const int n = (int)min((long long)a.width, ((long long)len + a.page_size - 1) / a.page_size);
  for (int c = threadIdx.x; c < n; c += 256) {
    const int p = row[c];
    if (p >= 0 && p < a.pages) atomicSub(&a.refs[p], 1);
    row[c] = -1;
  }
}

// Moves pages (an item is kCopyThreads * kCopyVec 16-byte words of one page, one
// layer, K or V), and does what of the tables takes more than one CTA:
// a fork's shared pages, or the renumbering after a compact.
__global__ void __launch_bounds__(kCopyThreads) move_kernel(const __grid_constant__ MoveArgs a) {
  griddep_wait();
  griddep_launch();
  const long long tid = (long long)blockIdx.x * kCopyThreads + threadIdx.x, nt = (long long)gridDim.x * kCopyThreads;
  if (a.tables == kTablesFork) {
    for (long long x = tid; x < (long long)a.n * a.width; x += nt) {
      const int i = (int)(x / a.width), c = (int)(x % a.width), len = a.start[i];
      if (len < 0) continue;
      int p = -1;
      if (c < len / a.page_size) {
        p = a.table[(long long)a.list0[i] * a.width + c];
        if (p >= 0 && p < a.pages) atomicAdd(&a.refs[p], 1);
      } else if (c == len / a.page_size) {
        p = a.move_dst[i];
      }
      a.table[(long long)a.list1[i] * a.width + c] = p;
    }
  } else if (a.tables == kTablesCompact) {
    for (long long x = tid; x < (long long)a.slots * a.width; x += nt) {
      const int p = a.table[x];
      if (p >= 0 && p < a.pages) a.table[x] = a.map[p];
    }
  }
  const int moves = a.count ? *a.count : a.n;
  const long long parts = (a.page_words + kCopyThreads * kCopyVec - 1) / (kCopyThreads * kCopyVec);
  const long long per_move = 2LL * a.layers * parts, items = per_move * moves;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int mv = (int)(it / per_move);
    const int s = a.move_src[mv], d = a.move_dst[mv];
    if (s < 0 || s >= a.pages || d < 0 || d >= a.pages) {
      // a fork without a partial page has none to move; a listed page out of range is an error
      if (a.tables == kTablesNone && threadIdx.x == 0) atomicOr(&a.book[0], TFX_CACHE_BAD);
      continue;
    }
    const long long rest = it % per_move, part = rest % parts, lk = rest / parts;
    uint4* pool = reinterpret_cast<uint4*>(lk & 1 ? a.v : a.k);
    const long long layer = (lk >> 1) * a.pages;
    const uint4* src = pool + (layer + s) * a.page_words;
    uint4* dst = pool + (layer + d) * a.page_words;
    const long long c0 = part * kCopyThreads * kCopyVec + threadIdx.x;
    uint4 x[kCopyVec];
#pragma unroll
    for (int j = 0; j < kCopyVec; j++)
      if (c0 + j * kCopyThreads < a.page_words) x[j] = __ldcs(src + c0 + j * kCopyThreads);
#pragma unroll
    for (int j = 0; j < kCopyVec; j++)
      if (c0 + j * kCopyThreads < a.page_words) __stcs(dst + c0 + j * kCopyThreads, x[j]);
  }
}

}  // namespace

int launch_extend(const BookArgs& a, cudaStream_t s) {
  return launch_kernel((const void*)extend_kernel, dim3(1), dim3(kBookThreads), 0, s, const_cast<BookArgs*>(&a),
                       dependent_launches(), 1);
}
int launch_append(const AppendArgs& a, int rows, cudaStream_t s) {
  return launch_kernel((const void*)append_kernel, dim3((unsigned)rows), dim3(128), 0, s, const_cast<AppendArgs*>(&a),
                       dependent_launches(), 1);
}
int launch_free(const BookArgs& a, cudaStream_t s) {
  return launch_kernel((const void*)free_kernel, dim3((unsigned)a.n), dim3(256), 0, s, const_cast<BookArgs*>(&a),
                       dependent_launches(), 1);
}
int launch_move(const BookArgs* book, bool compact, const MoveArgs& m, cudaStream_t s) {
  if (book) {
    const int rc = launch_kernel(compact ? (const void*)compact_book_kernel : (const void*)fork_book_kernel, dim3(1),
                                 dim3(kBookThreads), 0, s, const_cast<BookArgs*>(book), dependent_launches(), 1);
    if (rc) return rc;
  }
  const unsigned ctas = (unsigned)multiprocessors() * 8;  // eight CTAs of 256 threads fill an SM
  return launch_kernel((const void*)move_kernel, dim3(ctas), dim3(kCopyThreads), 0, s, const_cast<MoveArgs*>(&m),
                       dependent_launches(), 1);
}

}  // namespace tfx
