// How a decode step's work is cut among warps, and what the kernels that do it share.
// KS: keys of a slice; Rows: rows of a tile.
#pragma once
#include "attn_device.cuh"

namespace tfx {

// A run of slices of one group: a tile of rows of one K/V head against keys of one sequence.
struct Segment {
  bool prefix;
  int s0, s1;    // slices, from the sequence's first token
  int head;      // K/V head
  int seq;       // of the batch; -1: the shared prefix
  int row0;      // first row of the tile: of the batch's rows (prefix) or of the group's heads
  int rows;
  long long group;  // number of the group in its list
  const int* table;
};

struct Walk {
  long long pre_total, total;
  int own, sp, tiles, ptiles;
};
template <int KS, int Rows>
__device__ __forceinline__ Walk walk_of(const DecodeAttnArgs& a, int own) {
  Walk w;
  w.own = own;
  w.sp = a.pre_splits ? 0 : (a.shared + KS - 1) / KS;
  w.tiles = (a.group + Rows - 1) / Rows;
  w.ptiles = (a.batch * a.group + Rows - 1) / Rows;
  w.pre_total = (long long)a.heads_kv * w.ptiles * w.sp;
  w.total = w.pre_total + (long long)a.heads_kv * w.tiles * own;
  return w;
}

// The segment that begins with slice x of those before `end`.
template <int KS, int Rows>
__device__ __forceinline__ Segment segment_at(const DecodeAttnArgs& a, const Walk& w, const int* starts, long long x,
                                              long long end) {
  Segment g;
  g.prefix = x < w.pre_total;
  if (g.prefix) {
    const int grp = (int)(x / w.sp);
    g.group = grp;
    g.s0 = (int)(x % w.sp);
    g.s1 = (int)min((long long)w.sp, g.s0 + (end - x));
    g.head = grp / w.ptiles;
    g.seq = -1;
    g.row0 = grp % w.ptiles * Rows;
    g.rows = min(Rows, a.batch * a.group - g.row0);
    g.table = prefix_table(a);
  } else {
    const long long y = x - w.pre_total;
    const int hr = (int)(y / w.own), z = (int)(y % w.own);
    int lo = 0, hi = a.batch - 1;  // the sequence that slice z belongs to
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid + 1] > z) hi = mid; else lo = mid + 1;
    }
    const int off = a.shared / KS;
    g.seq = lo;
    g.group = (long long)hr * a.batch + lo;
    g.s0 = z - starts[lo] + off;
    g.s1 = (int)min((long long)(starts[lo + 1] - starts[lo] + off), g.s0 + (end - x));
    g.head = hr / w.tiles;
    g.row0 = hr % w.tiles * Rows;
    g.rows = min(Rows, a.group - g.row0);
    g.table = a.tables + (long long)a.seqs[lo] * a.width;  // it has slices, so its slot is in range
  }
  return g;
}

// Number of the batch's own slices of K and V, and in starts[0 .. batch] how many come
// before each sequence. All threads call; the first Warps warps count.
template <int KS, int Warps>
__device__ __forceinline__ int sequence_starts(const DecodeAttnArgs& a, int* starts, int* wsum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) starts[0] = 0;
  int carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += Warps * 32) {
    const int i = b0 + threadIdx.x;
    const int len = warp < Warps && i < a.batch ? seq_len(a, i) : 0;
    int x = len > a.shared ? (len + KS - 1) / KS - a.shared / KS : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(~0u, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31 && warp < Warps) wsum[warp] = x;
    __syncthreads();
    int before = carry, all = carry;
    for (int w = 0; w < Warps; w++) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    if (warp < Warps && i < a.batch) starts[i + 1] = before + x;
    carry = all;
    __syncthreads();
  }
  return carry;
}

// For the join: the runs of `per` slices that hold a part of each group.
__device__ __forceinline__ void note_runs(const DecodeAttnArgs& a, const Walk& w, const int* starts, long long per) {
  const int pre = a.heads_kv * w.ptiles * (w.sp > 0), own = a.heads_kv * w.tiles * a.batch;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < pre + own; i += gridDim.x * blockDim.x) {
    const int y = i - pre, hr = y / a.batch, seq = y - hr * a.batch;
    const long long x0 = i < pre ? (long long)i * w.sp : w.pre_total + (long long)hr * w.own + starts[seq];
    const int n = i < pre ? w.sp : starts[seq + 1] - starts[seq];
    const int first = (int)(x0 / per);
    a.runs[i] = make_int2(first, n ? (int)((x0 + n - 1) / per) - first + 1 : 0);
  }
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
// After a wait that gave up: the error word, and time for the copies in flight to land.
__device__ __forceinline__ void gave_up(int* err) {
  atomicExch(err, 1);
  const long long t0 = clock64();
  while (clock64() - t0 < 2000000) {
  }
}

}  // namespace tfx
