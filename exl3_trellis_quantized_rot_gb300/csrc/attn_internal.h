// Internal interface between the attention and cache translation units (not installed).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tfx_attn.h"
#include "exl3_internal.h"

namespace tfx {

constexpr int kAttnMaxSeqs = 512;  // sequences of one prompt launch (longer lists take several launches)

// Work of one prompt launch, in the kernel's parameters: nothing is copied to
// the device and a captured launch keeps it. A tile is 2 x `tokens` tokens of
// per_tile query heads that share a K/V head. The sequences are ordered by their
// number of tiles, most first, and tiles are started from the last (the most
// keys) to the first: level by level, at each the sequences that have it.
// before[s] is the number of tiles that come before level count[s] - 1.
struct PromptArgs {
  static constexpr bool kFewRows = false;
  CUtensorMap qmap, k, v;
  const void* vbase;
  void* out;
  long long ldv, ldo;
  float scale_log2;  // scale * log2(e)
  int heads_kv, group, per_tile, tokens;
  int sub, hg;  // tiles of a group's heads; of all heads
  int n, items;
  int* err;
  long long spin;
  int begin[kAttnMaxSeqs];  // first row of a sequence
  int len[kAttnMaxSeqs];
  int count[kAttnMaxSeqs];   // its tiles
  int before[kAttnMaxSeqs];
};

// A decode call. The shared prefix goes to the tensor-core kernel where the
// batch has enough rows (pre_splits > 0: the prefix in that many shares, each
// with its own partial result); the rest is cut into slices of 16 KB of K and V,
// numbered through: first those of the prefix where it was not taken (for each
// K/V head and 16-row tile of the batch's rows), then the sequences' own (for
// each K/V head and 16-row tile of a sequence's heads, sequence after sequence).
// Warp w takes the slices [w*per, (w+1)*per); a run of them inside one group is
// a segment with its own partial result, in slot w + (number of the group).
struct DecodeAttnArgs {
  static constexpr bool kFewRows = true;
  CUtensorMap k, v;           // boxes of 16 tokens, all of a head's values
  CUtensorMap qmap, kt, vt;   // tensor-core kernel: tiles of Q; boxes of up to 64 tokens of 64 values
  const void* q;
  void* out;
  long long ldq, ldo;
  const int* seqs;
  const int* lens;
  const int* tables;
  float scale_log2;
  int heads_q, heads_kv, group, batch, shared;
  int page_size, page_shift, pages, slots, width;
  // tensor-core kernel: as above, and tiles of the batch's rows
  int per_tile, tokens, sub, hg, mt, pre_splits, items;
  int warps;          // NW
  int own_rows;       // rows of an own slot: min(16, group)
  int2* runs;         // [prefix groups + own groups]: the first warp that has a part of a group, and how many have
  float* own_o;       // [NW + groups][own_rows][dim]
  float2* own_ml;     // [NW + groups][own_rows]: (reference of the exponents, sum)
  float* pre_o;       // [NW + prefix groups][16][dim], or [pre_splits][batch][heads_q][dim]
  float2* pre_ml;
  int* err;
  long long spin;
};

// What appends need to know of the extends before them. Only an extend writes it,
// except that a slot which is freed, or becomes a fork, loses its mark.
struct Grown {
  int2* mark;    // of each slot: the position its last new tokens begin at, and how many they are; y 0: none, -1: refused
  int* n;        // the last extend's lists
  int* seqs;     // [slots]
  int* offsets;  // [slots + 1]
};

// One-CTA book kernels of the page operations.
struct BookArgs {
  int *book, *lens, *refs, *tables;
  const int *list0, *list1;  // seqs / sources; offsets / targets
  int n, slots, width, pages, page_size, row_cap;
  // scratch: free pages in order; moves; where a page is after a compact; the
  // length that each fork takes over (-1: left alone); moves counted
  int *free_list, *move_src, *move_dst, *map, *start, *count;
  Grown grown;
};

struct AppendArgs {
  const void *k_new, *v_new;
  void *k, *v;         // the layer's pages
  long long ldk, ldv;  // 16-byte words
  int row;             // 16-byte words of a token's K (or V)
  const int *seqs, *offsets;  // null: the last extend's, in `grown`
  int n;
  int* book;
  const int* table;
  int slots, width, pages, page_size;
  Grown grown;
};

enum Tables { kTablesNone = 0, kTablesFork = 1, kTablesCompact = 2 };
struct MoveArgs {
  void *k, *v;
  int *book, *refs, *table;
  const int *list0, *list1, *move_src, *move_dst, *map, *start;
  const int* count;  // moves (null: n)
  int n, layers, pages, slots, width, page_size;
  long long page_words;  // 16-byte words of one page of one layer
  Tables tables;
};

int launch_extend(const BookArgs& a, cudaStream_t s);
int launch_append(const AppendArgs& a, int rows, cudaStream_t s);
int launch_free(const BookArgs& a, cudaStream_t s);
int launch_move(const BookArgs* book, bool compact, const MoveArgs& m, cudaStream_t s);

int launch_prompt(const PromptArgs& a, int act, int dim, cudaStream_t s);
int launch_prefix(const DecodeAttnArgs& a, int act, int dim, cudaStream_t s);
int launch_decode(const DecodeAttnArgs& a, int act, int dim, cudaStream_t s);

// exl3_host.cu
tfx_exl3_driver driver_hooks();
bool driver_is_runtime();
long long spin_limit();
int multiprocessors();
int current_device();  // -1 where there is none
// Whether launches may carry the programmatic dependency (tfx_exl3_set_pdl: not
// where it is off). Every attention and cache kernel waits for the launches before
// it (griddepcontrol.wait) ahead of its first access to memory that they may use.
bool dependent_launches();
int launch_kernel(const void* fn, dim3 grid, dim3 block, size_t smem, cudaStream_t s, void* arg, bool pdl, int cluster);
int opt_in_smem(const void* fn, size_t smem);
int fail_with(int code, const char* fmt, ...);
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled tensor_map_encoder();

}  // namespace tfx
