// Host side of the attention and cache C ABI: validation, tensor maps, scratch,
// launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "attn_internal.h"
#include "per_device.h"

namespace tfx {
__device__ int g_attn_error = 0;  // device error word: a bounded wait gave up
}

namespace {

using tfx::fail_with;

constexpr int kRowTile = 16;  // rows of a warp
// Tokens of one sequence: kernels round positions up to whole tiles and look up pages
// of up to 1,008 tokens past the last, in 32 bits.
constexpr int64_t kMostTokens = INT32_MAX - 2047;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct CachePriv {
  int* pages = nullptr;  // page-call scratch
  size_t pages_bytes = 0;
  char* part = nullptr;  // decode partial results
  size_t part_bytes = 0;
  int max_batch = 0, heads_q = 0;
};

// The current device's own.
int* error_word() {
  static thread_local tfx::PerDevice<int*> words;
  return words.of(tfx::current_device(), []() -> int* {
    void* q = nullptr;
    if (cudaGetSymbolAddress(&q, tfx::g_attn_error) == cudaSuccess) return static_cast<int*>(q);
    cudaGetLastError();
    return nullptr;
  });
}

int check_heads(const tfx_attn_heads* h) {
  if (!h) return fail_with(TFX_EINVAL, "null heads");
  if (h->heads_q < 1 || h->heads_kv < 1 || h->heads_q % h->heads_kv || h->heads_q / h->heads_kv > 128)
    return fail_with(TFX_EINVAL, "heads_q=%d, heads_kv=%d: heads_kv divides heads_q, at most 128 to one", h->heads_q,
                     h->heads_kv);
  if (h->heads_kv > 65535) return fail_with(TFX_EINVAL, "heads_kv=%d above 65535", h->heads_kv);
  if (h->act != TFX_F16 && h->act != TFX_BF16) return fail_with(TFX_EINVAL, "act=%d", h->act);
  if (h->dim != 128 && h->dim != 256) return fail_with(TFX_EUNSUPPORTED, "dim=%d (128 or 256)", h->dim);
  if (!(h->scale > 0.f) || !std::isfinite(h->scale)) return fail_with(TFX_EINVAL, "scale=%g", (double)h->scale);
  return 0;
}

int check_rows(const char* what, const void* p, int64_t ld, int64_t width) {
  if (!p) return fail_with(TFX_EINVAL, "null %s", what);
  if (ld < width) return fail_with(TFX_EINVAL, "pitch %lld of %s below its %lld values", (long long)ld, what, (long long)width);
  if (ld % 8 || !aligned16(p)) return fail_with(TFX_EALIGN, "%s: a 16-byte aligned pointer and a pitch of whole 8 values", what);
  if (ld > (1LL << 36)) return fail_with(TFX_EINVAL, "pitch %lld of %s", (long long)ld, what);
  return 0;
}

int encode_map(CUtensorMap* tm, const void* base, CUtensorMapDataType type, const cuuint64_t (&dims)[5],
               const cuuint64_t (&strides)[4], const cuuint32_t (&box)[5],
               CUtensorMapL2promotion promotion = CU_TENSOR_MAP_L2_PROMOTION_L2_256B) {
  const tfx::EncodeTiled enc = tfx::tensor_map_encoder();
  if (!enc) return fail_with(TFX_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = enc(tm, type, 5, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, promotion, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail_with(TFX_ECUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return 0;
}

CUtensorMapDataType type_of(int act) {
  return act == TFX_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// K or V as (64 values, tokens, dim/64 column blocks, heads, pages), in boxes of
// some tokens of some column blocks of one head.
int make_map(CUtensorMap* tm, const void* base, int act, int dim, int heads, int64_t tokens, int64_t ld, int64_t pages,
             int64_t page_pitch, int box_tokens, int box_blocks) {
  const cuuint64_t dims[5] = {64, (cuuint64_t)tokens, (cuuint64_t)dim / 64, (cuuint64_t)heads, (cuuint64_t)pages};
  const cuuint64_t strides[4] = {(cuuint64_t)ld * 2, 128, (cuuint64_t)dim * 2, (cuuint64_t)page_pitch * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)box_tokens, (cuuint32_t)box_blocks, 1, 1};
  return encode_map(tm, base, type_of(act), dims, strides, box);
}

// Pages of 8-bit codes as (128 codes, tokens, dim/128 column blocks, heads, pages), in boxes
// of 16 tokens of one head.
int make_code_map(CUtensorMap* tm, const void* base, const tfx_cache* c) {
  const cuuint64_t row = (cuuint64_t)c->heads_kv * c->dim;
  const cuuint64_t dims[5] = {128, (cuuint64_t)c->page_size, (cuuint64_t)c->dim / 128, (cuuint64_t)c->heads_kv, (cuuint64_t)c->pages};
  const cuuint64_t strides[4] = {row, 128, (cuuint64_t)c->dim, row * c->page_size};
  const cuuint32_t box[5] = {128, TFX_CACHE_BLOCK, (cuuint32_t)c->dim / 128, 1, 1};
  // a head's codes of a token are 128 or 256 bytes, and what lies beside them is another head's
  return encode_map(tm, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, dims, strides, box,
                    c->dim == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Q as (64 values, heads, tokens, dim/64 column blocks), in boxes of one column
// block of some heads of some tokens: the rows of a tile in order.
int make_q_map(CUtensorMap* tm, const void* base, int act, int dim, int heads, int64_t tokens, int64_t ld, int box_heads,
               int box_tokens) {
  const cuuint64_t dims[5] = {64, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)dim / 64, 1};
  const cuuint64_t strides[4] = {(cuuint64_t)dim * 2, (cuuint64_t)ld * 2, 128, 16};
  const cuuint32_t box[5] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens, 1, 1};
  return encode_map(tm, base, type_of(act), dims, strides, box);
}

// Query heads of one K/V head that share a 128-row tile: the most that divide
// the group and leave at most one row in 16 of the tile empty.
int heads_per_tile(int group) {
  int g = group;
  while (group % g || 128 / g * g < 120) g--;
  return g;
}

int check_cache(const tfx_cache* c) {
  if (!c) return fail_with(TFX_EINVAL, "null cache");
  if (!c->k || !c->v || !c->book) return fail_with(TFX_EINVAL, "null k, v or book");
  if (c->layers < 1 || c->pages < 1 || c->heads_kv < 1 || c->slots < 1 || c->width < 1)
    return fail_with(TFX_EINVAL, "layers=%d, pages=%d, heads_kv=%d, slots=%d, width=%d: all at least 1", c->layers, c->pages,
                     c->heads_kv, c->slots, c->width);
  if (c->act != TFX_F16 && c->act != TFX_BF16) return fail_with(TFX_EINVAL, "act=%d", c->act);
  if (c->dim != 128 && c->dim != 256) return fail_with(TFX_EUNSUPPORTED, "dim=%d (128 or 256)", c->dim);
  if ((int64_t)c->heads_kv * c->dim > (1 << 30))
    return fail_with(TFX_EUNSUPPORTED, "heads_kv=%d of dim=%d: a token has more than 2^30 values", c->heads_kv, c->dim);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return fail_with(TFX_EUNSUPPORTED, "page_size=%d (16, 32, 64 or 128)", c->page_size);
  if ((int64_t)c->pages * c->page_size > INT32_MAX || (int64_t)c->width * c->page_size > kMostTokens)
    return fail_with(TFX_EUNSUPPORTED, "2^31 tokens or more in the pool, or above %lld in a table", (long long)kMostTokens);
  // an extend adds up what a list of at most `slots` entries asks for
  if ((int64_t)c->slots * c->width > INT32_MAX) return fail_with(TFX_EUNSUPPORTED, "2^31 table entries or more");
  if (!aligned16(c->k) || !aligned16(c->v)) return fail_with(TFX_EALIGN, "k or v is not 16-byte aligned");
  if (c->store != TFX_STORE_ACT) {
    if (c->store != TFX_STORE_I8 && c->store != TFX_STORE_E4M3) return fail_with(TFX_EINVAL, "store=%d", c->store);
    if (!c->k_scale || !c->v_scale) return fail_with(TFX_EINVAL, "null k_scale or v_scale");
    if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3u)
      return fail_with(TFX_EALIGN, "k_scale or v_scale is not 4-byte aligned");
  }
  if (reinterpret_cast<uintptr_t>(c->book) & 3u) return fail_with(TFX_EALIGN, "book is not 4-byte aligned");
  return 0;
}

int check_reserved(const tfx_cache* c) {
  const CachePriv* pv = static_cast<const CachePriv*>(c->priv);
  return pv && pv->pages ? 0 : fail_with(TFX_ENOTRESERVED, "cache not reserved");
}

int check_list(const tfx_cache* c, int n, const void* p, const void* q) {
  int rc = check_cache(c);
  if (rc) return rc;
  if (n < 0) return fail_with(TFX_EINVAL, "n=%d", n);
  if (n && (!p || !q)) return fail_with(TFX_EINVAL, "null list");
  return check_reserved(c);
}

int grow(void** p, size_t* have, size_t want, cudaStream_t s) {
  if (want <= *have) return 0;
  void* np = nullptr;
  const tfx_exl3_driver d = tfx::driver_hooks();
  if (d.alloc(&np, want, s) != 0 || !np) return fail_with(TFX_ECUDA, "allocation of %zu bytes failed", want);
  if (*p) d.free(*p, s);
  *p = np;
  *have = want;
  return 0;
}

int* lens_of(const tfx_cache* c) { return c->book + 4; }
int* refs_of(const tfx_cache* c) { return lens_of(c) + c->slots; }
int* tables_of(const tfx_cache* c) { return refs_of(c) + c->pages; }
int64_t page_values(const tfx_cache* c) { return (int64_t)c->page_size * c->heads_kv * c->dim; }
int page_shift(const tfx_cache* c) { return c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7; }
int value_bytes(const tfx_cache* c) { return c->store == TFX_STORE_ACT ? 2 : 1; }
int64_t page_scales(const tfx_cache* c) { return (int64_t)(c->page_size / TFX_CACHE_BLOCK) * c->heads_kv; }
// A layer's pages and scales.
template <typename P>
P* layer_of(const tfx_cache* c, void* pool, int layer) {
  return reinterpret_cast<P*>(static_cast<char*>(pool) + (int64_t)layer * c->pages * page_values(c) * value_bytes(c));
}
float* scales_of(const tfx_cache* c, float* scales, int layer) {
  return c->store == TFX_STORE_ACT ? nullptr : scales + (int64_t)layer * c->pages * page_scales(c);
}

// Page-call scratch: a counter and the list length that an append uses, what
// extends leave for the appends (a mark and a list entry of each slot), and five
// lists of `slots`-or-`pages` entries (a call lists at most that many).
int64_t list_cap(const tfx_cache* c) { return c->slots > c->pages ? c->slots : c->pages; }
size_t page_scratch_ints(const tfx_cache* c) { return 4 + 4 * (size_t)c->slots + 1 + 5 * (size_t)list_cap(c); }

tfx::BookArgs book_args(const tfx_cache* c, const int32_t* l0, const int32_t* l1, int n) {
  const CachePriv* pv = static_cast<const CachePriv*>(c->priv);
  tfx::BookArgs a = {};
  a.book = c->book;
  a.lens = lens_of(c);
  a.refs = refs_of(c);
  a.tables = tables_of(c);
  a.list0 = l0;
  a.list1 = l1;
  a.n = n;
  a.slots = c->slots;
  a.width = c->width;
  a.pages = c->pages;
  a.page_size = c->page_size;
  a.row_cap = c->pages * c->page_size;
  const int64_t cap = list_cap(c);
  int* p = pv->pages;
  a.count = p;
  a.grown.n = p + 1;
  a.grown.mark = reinterpret_cast<int2*>(p + 4);
  a.grown.seqs = p + 4 + 2 * (int64_t)c->slots;
  a.grown.offsets = a.grown.seqs + c->slots;
  a.free_list = a.grown.offsets + c->slots + 1;
  a.move_src = a.free_list + cap;
  a.move_dst = a.move_src + cap;
  a.map = a.move_dst + cap;
  a.start = a.map + cap;
  return a;
}

tfx::MoveArgs move_args(const tfx_cache* c, const tfx::BookArgs& b, tfx::Tables tables) {
  tfx::MoveArgs m = {};
  m.k = c->k;
  m.v = c->v;
  m.book = c->book;
  m.refs = b.refs;
  m.table = b.tables;
  m.list0 = b.list0;
  m.list1 = b.list1;
  m.move_src = b.move_src;
  m.move_dst = b.move_dst;
  m.map = b.map;
  m.start = b.start;
  m.count = b.count;
  m.n = b.n;
  m.layers = c->layers;
  m.pages = c->pages;
  m.slots = c->slots;
  m.width = c->width;
  m.page_size = c->page_size;
  m.page_words = page_values(c) * value_bytes(c) / 16;
  if (c->store != TFX_STORE_ACT) {
    m.k_scale = c->k_scale;
    m.v_scale = c->v_scale;
    m.page_scales = (int)page_scales(c);
  }
  m.tables = tables;
  return m;
}

// The shared prefix on the tensor cores: in so many shares that the items
// (heads, 256-row tiles of the batch's rows, shares) fill the pairs of SMs once.
int prefix_splits(int batch, int heads_q, int heads_kv, int shared) {
  const int group = heads_q / heads_kv, per = heads_per_tile(group), seqs = 2 * (128 / per);
  const int64_t rest = (int64_t)heads_kv * (group / per) * ((batch + seqs - 1) / seqs);
  const int64_t fill = tfx::multiprocessors() / 2 / rest, tiles = (shared + 127) / 128;
  return (int)(fill < 1 ? 1 : fill > tiles ? tiles : fill);
}
// Rows of one K/V head from which on the shared prefix goes to the tensor cores, where
// it has 256 tokens or more: a tile costs the same there for 1 row as for 256, while the
// warps read K and V again for every 16. Measured, a step on the tensor cores / by warps
// (us; 24/4 heads of 256, 6 rows a sequence, 100 own tokens, pages of 64): prefix of
// 65,536 and 2 sequences 55 / 63, 4: 56 / 99, 6: 57 / 89, 16: 59 / 232; of 8,192 and
// 4: 20.5 / 20.3, 6: 21.0 / 21.5, 16: 21.9 / 29.3; of 1,024 and 6: 12.5 / 12.7, 16: 17.4 /
// 12.7, 64: 23.5 / 23.5; of 256 and 64: 21.4 / 17.4. So the rule is right for many rows
// or long prefixes, gives away 40 us with 17 to 32 rows of a very long one, and 5 us with
// 96 rows of a short one.
bool many_rows(int64_t batch, int64_t group) { return batch * group > 32; }
// Partial results that the prefix's shares leave, at most: batch * heads_q times
// the shares, which are one, or as many as give each pair of SMs an item of 256 rows.
// It grows with both counts, as a reservation for more than is used must.
int64_t prefix_rows(int64_t batch, int64_t heads_q, int64_t heads_kv) {
  if (!many_rows(batch, heads_q / heads_kv)) return 0;
  return std::max(batch * heads_q, (int64_t)tfx::multiprocessors() / 2 * 256);
}

// Over 8-bit codes, the tokens of a prefix that the tensor cores read once; 0: each sequence
// reads it as its own. That takes the warps as long as reading the prefix `batch` times, from L2
// where it fits, and once more for every further 16 heads of a group. The rule leaves those out: it is
// measured with groups of 6 and 1, and late for those above 16. The other kernel begins with 8 us.
// Measured, the tensor cores / as their own (us;
// 100 own tokens): 24/4 heads of 256, 8,192 tokens and 2 sequences 18.1 / 15.3, 4: 18.7 / 17.7, 6: 19.2 /
// 21.2, 16: 23.8 / 41.0; of 2,048 and 6: 16.0 / 11.9, 16: 19.8 / 17.2; of 32,768 and 2: 31.9 / 28.8, 3: 32.0 /
// 35.2; 8/8 heads of 128, 8,192 and 4: 18.5 / 16.8, 8: 20.0 / 26.3; of 32,768 and 4: 39.5 / 44.9.
// Wide groups just above / below 64 MiB, one K/V head of 256: 16 sequences of 32 heads behind 8,300 / 8,000
// tokens 31.3 / 46.7, of 64 heads 42.1 / 77.6, of 128 heads 65.0 / 138.
constexpr int kFewSequences = 2;  // batches up to this never go there, and reserve nothing for it
int coded_prefix(const tfx_cache* c, int batch, int shared) {
  shared = shared / TFX_CACHE_BLOCK * TFX_CACHE_BLOCK;
  return batch > kFewSequences && (int64_t)batch * shared * c->heads_kv * c->dim * 2 > (64LL << 20) ? shared : 0;
}
// Partial results of that kernel's shares, at most: as prefix_rows, in tiles of its own.
int64_t coded_prefix_rows(int64_t batch, int64_t heads_q) {
  if (batch <= kFewSequences) return 0;
  return std::max(batch * heads_q, (int64_t)tfx::multiprocessors() * tfx::prefix_q8_rows());
}

int decode_warps(const tfx_cache* c) { return tfx::multiprocessors() * (c->store == TFX_STORE_ACT ? 4 : tfx::kCodedWarps); }
// Decode scratch for `batch` sequences: byte offsets of its parts. No part shrinks with batch or heads.
struct DecodeScratch {
  size_t runs, own_ml, pre_ml, own_o, pre_o, bytes;
};
DecodeScratch decode_scratch(const tfx_cache* c, int batch, int heads_q) {
  const int heads_kv = c->heads_kv, dim = c->dim, warps = decode_warps(c);
  const int64_t group = heads_q / heads_kv, tiles = (group + kRowTile - 1) / kRowTile;
  const int64_t ptiles = (batch * group + kRowTile - 1) / kRowTile;
  const int64_t own_rows = group < kRowTile ? group : kRowTile;
  const int64_t own = (warps + heads_kv * tiles * batch) * own_rows;
  const int64_t few = (warps + heads_kv * ptiles) * kRowTile, many = prefix_rows(batch, heads_q, heads_kv);
  const int64_t pre = c->store != TFX_STORE_ACT ? coded_prefix_rows(batch, heads_q) : few > many ? few : many;
  auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
  DecodeScratch d;
  int64_t at = 0;
  d.runs = at;
  at += up(heads_kv * (ptiles + tiles * batch) * 8);
  d.own_ml = at;
  at += up(own * 8);
  d.pre_ml = at;
  at += up(pre * 8);
  d.own_o = at;
  at += up(own * dim * 4);
  d.pre_o = at;
  at += up(pre * dim * 4);
  d.bytes = (size_t)at;
  return d;
}

// Rows of the given lists (null: the last extend's).
int append_rows(tfx_cache* c, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv, int rows,
                const int32_t* seqs, const int32_t* offsets, int n, cudaStream_t stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  if (layer < 0 || layer >= c->layers) return fail_with(TFX_EINVAL, "layer %d of %d", layer, c->layers);
  if (rows < 0 || rows > c->pages * c->page_size)
    return fail_with(TFX_EINVAL, "rows=%d outside 0..%d", rows, c->pages * c->page_size);
  if ((rc = check_reserved(c))) return rc;
  if (!rows) return 0;
  if ((rc = check_rows("k", k, ldk, (int64_t)c->heads_kv * c->dim))) return rc;
  if ((rc = check_rows("v", v, ldv, (int64_t)c->heads_kv * c->dim))) return rc;
  const tfx::BookArgs b = book_args(c, nullptr, nullptr, 0);
  tfx::AppendArgs a = {};
  a.k_new = k;
  a.v_new = v;
  a.k = layer_of<void>(c, c->k, layer);
  a.v = layer_of<void>(c, c->v, layer);
  a.ldk = ldk / 8;
  a.ldv = ldv / 8;
  a.row = c->heads_kv * c->dim / 8;
  a.seqs = seqs;
  a.offsets = offsets;
  a.n = n;
  a.book = c->book;
  a.table = b.tables;
  a.slots = c->slots;
  a.width = c->width;
  a.pages = c->pages;
  a.page_size = c->page_size;
  a.grown = b.grown;
  if (c->store == TFX_STORE_ACT) return tfx::launch_append(a, rows, stream);
  a.k_scale = scales_of(c, c->k_scale, layer);
  a.v_scale = scales_of(c, c->v_scale, layer);
  a.heads = c->heads_kv;
  a.rows = rows;
  return tfx::launch_append_q8(a, c->act, c->store, c->dim, stream);
}

}  // namespace

extern "C" {

int tfx_attn_prompt(const tfx_attn_heads* h, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                    int64_t ldv, const int32_t* offsets, int n, void* out, int64_t ldo, cudaStream_t stream) {
  int rc = check_heads(h);
  if (rc) return rc;
  if (n < 0) return fail_with(TFX_EINVAL, "n=%d", n);
  if (n && !offsets) return fail_with(TFX_EINVAL, "null offsets");
  if (n && offsets[0] < 0) return fail_with(TFX_EINVAL, "offsets[0]=%d", offsets[0]);
  for (int i = 0; i < n; i++)
    if (offsets[i + 1] < offsets[i]) return fail_with(TFX_EINVAL, "offsets[%d]=%d below offsets[%d]", i + 1, offsets[i + 1], i);
  if (!n || offsets[n] == offsets[0]) return 0;
  if ((rc = check_rows("q", q, ldq, (int64_t)h->heads_q * h->dim))) return rc;
  if ((rc = check_rows("k", k, ldk, (int64_t)h->heads_kv * h->dim))) return rc;
  if ((rc = check_rows("v", v, ldv, (int64_t)h->heads_kv * h->dim))) return rc;
  if ((rc = check_rows("out", out, ldo, (int64_t)h->heads_q * h->dim))) return rc;
  tfx::PromptArgs a;
  const int64_t rows = offsets[n];
  a.heads_kv = h->heads_kv;
  a.group = h->heads_q / h->heads_kv;
  a.per_tile = heads_per_tile(a.group);
  a.tokens = 128 / a.per_tile;
  if ((rc = make_q_map(&a.qmap, q, h->act, h->dim, h->heads_q, rows, ldq, a.per_tile, a.tokens))) return rc;
  if ((rc = make_map(&a.k, k, h->act, h->dim, h->heads_kv, rows, ldk, 1, 8, 64, h->dim / 64))) return rc;
  if ((rc = make_map(&a.v, v, h->act, h->dim, h->heads_kv, rows, ldv, 1, 8, 128, h->dim / 128))) return rc;
  a.vbase = v;
  a.out = out;
  a.ldv = ldv;
  a.ldo = ldo;
  a.scale_log2 = h->scale * 1.4426950408889634f;
  a.err = error_word();
  a.spin = tfx::spin_limit();
  if (!a.err) return fail_with(TFX_ECUDA, "no device error word");
  a.sub = a.group / a.per_tile;
  a.hg = a.heads_kv * a.sub;
  const int tile = 2 * a.tokens, per_token_tile = a.hg;
  for (int i = 0; i < n;) {
    struct Seq {
      int begin, len;
    } seqs[tfx::kAttnMaxSeqs];
    for (a.n = 0; i < n && a.n < tfx::kAttnMaxSeqs; i++)
      if (offsets[i + 1] > offsets[i]) seqs[a.n++] = {offsets[i], offsets[i + 1] - offsets[i]};
    if (!a.n) break;
    std::stable_sort(seqs, seqs + a.n, [](const Seq& x, const Seq& y) { return x.len > y.len; });
    int64_t total = 0;
    for (int s = 0; s < a.n; s++) {
      a.begin[s] = seqs[s].begin;
      a.len[s] = seqs[s].len;
      a.count[s] = (seqs[s].len + tile - 1) / tile;
      total += a.count[s];
      a.before[s] = (int)(total - (int64_t)a.count[s] * (s + 1));
    }
    if (total * per_token_tile > (1 << 30)) return fail_with(TFX_EUNSUPPORTED, "%lld tiles", (long long)(total * per_token_tile));
    a.items = (int)total * per_token_tile;
    if ((rc = tfx::launch_prompt(a, h->act, h->dim, stream))) return rc;
  }
  return 0;
}

int64_t tfx_cache_book_ints(const tfx_cache* c) {
  return c ? 4 + (int64_t)c->slots + c->pages + (int64_t)c->slots * c->width : 0;
}

int tfx_cache_reserve(tfx_cache* c, int max_batch, int heads_q, cudaStream_t stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  if (max_batch < 1 || max_batch > TFX_ATTN_MAX_BATCH)
    return fail_with(TFX_EINVAL, "max_batch=%d outside 1..%d", max_batch, TFX_ATTN_MAX_BATCH);
  if (heads_q < 1 || heads_q % c->heads_kv || heads_q / c->heads_kv > 128)
    return fail_with(TFX_EINVAL, "heads_q=%d over heads_kv=%d", heads_q, c->heads_kv);
  CachePriv* pv = static_cast<CachePriv*>(c->priv);
  if (!pv) {
    pv = new (std::nothrow) CachePriv();
    if (!pv) return fail_with(TFX_ECUDA, "no host memory");
    c->priv = pv;
  }
  const size_t had = pv->pages_bytes;
  if ((rc = grow(reinterpret_cast<void**>(&pv->pages), &pv->pages_bytes, page_scratch_ints(c) * 4, stream))) return rc;
  if (pv->pages_bytes > had && tfx::driver_hooks().memset0(pv->pages, pv->pages_bytes, stream) != 0) {  // no slot has a mark
    tfx::driver_hooks().free(pv->pages, stream);
    pv->pages = nullptr;
    pv->pages_bytes = 0;
    return fail_with(TFX_ECUDA, "clearing %zu bytes failed", page_scratch_ints(c) * 4);
  }
  const int b = max_batch > pv->max_batch ? max_batch : pv->max_batch, hq = heads_q > pv->heads_q ? heads_q : pv->heads_q;
  const size_t part = decode_scratch(c, b, hq).bytes;
  if ((rc = grow(reinterpret_cast<void**>(&pv->part), &pv->part_bytes, part, stream))) return rc;
  pv->max_batch = b;
  pv->heads_q = hq;
  return 0;
}

int tfx_cache_release(tfx_cache* c) {
  if (!c) return fail_with(TFX_EINVAL, "null cache");
  CachePriv* pv = static_cast<CachePriv*>(c->priv);
  if (!pv) return 0;
  const tfx_exl3_driver d = tfx::driver_hooks();
  if (tfx::driver_is_runtime()) cudaDeviceSynchronize();
  if (pv->pages) d.free(pv->pages, nullptr);
  if (pv->part) d.free(pv->part, nullptr);
  if (tfx::driver_is_runtime()) cudaDeviceSynchronize();
  delete pv;
  c->priv = nullptr;
  return 0;
}

int tfx_cache_extend(tfx_cache* c, const int32_t* seqs, const int32_t* offsets, int n, cudaStream_t stream) {
  const int rc = check_list(c, n, seqs, offsets);
  if (rc) return rc;
  if (n > c->slots) return fail_with(TFX_EINVAL, "%d sequences, %d slots", n, c->slots);
  return tfx::launch_extend(book_args(c, seqs, offsets, n), stream);
}

int tfx_cache_append(tfx_cache* c, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv, int rows,
                     cudaStream_t stream) {
  return append_rows(c, layer, k, ldk, v, ldv, rows, nullptr, nullptr, 0, stream);
}

int tfx_cache_append_listed(tfx_cache* c, int layer, const void* k, int64_t ldk, const void* v, int64_t ldv, int rows,
                            const int32_t* seqs, const int32_t* offsets, int n, cudaStream_t stream) {
  const int rc = check_list(c, n, seqs, offsets);
  if (rc) return rc;
  if (n > c->slots) return fail_with(TFX_EINVAL, "%d sequences, %d slots", n, c->slots);
  return append_rows(c, layer, k, ldk, v, ldv, n ? rows : 0, seqs, offsets, n, stream);
}

int tfx_cache_read(tfx_cache* c, int layer, const int32_t* seqs, const int32_t* starts, const int32_t* offsets, int n,
                   int rows, void* k, int64_t ldk, void* v, int64_t ldv, cudaStream_t stream) {
  int rc = check_list(c, n, seqs, offsets);
  if (rc) return rc;
  if (n && !starts) return fail_with(TFX_EINVAL, "null starts");
  if (layer < 0 || layer >= c->layers) return fail_with(TFX_EINVAL, "layer %d of %d", layer, c->layers);
  if (rows < 0) return fail_with(TFX_EINVAL, "rows=%d", rows);
  if (!n || !rows) return 0;
  if ((rc = check_rows("k", k, ldk, (int64_t)c->heads_kv * c->dim))) return rc;
  if ((rc = check_rows("v", v, ldv, (int64_t)c->heads_kv * c->dim))) return rc;
  if (k == v) return fail_with(TFX_EINVAL, "k and v are one tensor");
  tfx::ReadArgs a = {};
  a.k = layer_of<const void>(c, c->k, layer);
  a.v = layer_of<const void>(c, c->v, layer);
  a.k_scale = scales_of(c, c->k_scale, layer);
  a.v_scale = scales_of(c, c->v_scale, layer);
  a.k_out = k;
  a.v_out = v;
  a.ldk = ldk;
  a.ldv = ldv;
  a.seqs = seqs;
  a.starts = starts;
  a.offsets = offsets;
  a.n = n;
  a.rows = rows;
  a.book = c->book;
  a.lens = lens_of(c);
  a.table = tables_of(c);
  a.slots = c->slots;
  a.width = c->width;
  a.pages = c->pages;
  a.page_shift = page_shift(c);
  a.heads = c->heads_kv;
  a.dim = c->dim;
  return tfx::launch_read(a, c->act, c->store, stream);
}

int tfx_cache_fork(tfx_cache* c, const int32_t* src, const int32_t* dst, int n, cudaStream_t stream) {
  const int rc = check_list(c, n, src, dst);
  if (rc) return rc;
  if (n > c->slots) return fail_with(TFX_EINVAL, "%d forks, %d slots", n, c->slots);
  if (!n) return 0;
  const tfx::BookArgs b = book_args(c, src, dst, n);
  return tfx::launch_move(&b, false, move_args(c, b, tfx::kTablesFork), stream);
}

int tfx_cache_free(tfx_cache* c, const int32_t* seqs, int n, cudaStream_t stream) {
  const int rc = check_list(c, n, seqs, seqs);
  if (rc) return rc;
  if (n > c->slots) return fail_with(TFX_EINVAL, "%d sequences, %d slots", n, c->slots);
  if (!n) return 0;
  return tfx::launch_free(book_args(c, seqs, nullptr, n), stream);
}

int tfx_cache_compact(tfx_cache* c, cudaStream_t stream) {
  const int rc = check_list(c, 0, nullptr, nullptr);
  if (rc) return rc;
  const tfx::BookArgs b = book_args(c, nullptr, nullptr, 0);
  return tfx::launch_move(&b, true, move_args(c, b, tfx::kTablesCompact), stream);
}

int tfx_cache_copy(tfx_cache* c, const int32_t* src, const int32_t* dst, int n, cudaStream_t stream) {
  const int rc = check_list(c, n, src, dst);
  if (rc) return rc;
  if (n > c->pages) return fail_with(TFX_EINVAL, "%d copies, %d pages", n, c->pages);
  if (!n) return 0;
  tfx::MoveArgs m = move_args(c, book_args(c, nullptr, nullptr, n), tfx::kTablesNone);
  m.move_src = src;
  m.move_dst = dst;
  m.count = nullptr;
  return tfx::launch_move(nullptr, false, m, stream);
}

int tfx_attn_decode(tfx_cache* c, int layer, const tfx_attn_heads* h, const void* q, int64_t ldq, const int32_t* seqs,
                    int batch, int shared, void* out, int64_t ldo, cudaStream_t stream) {
  int rc = check_cache(c);
  if (rc || (rc = check_heads(h))) return rc;
  if (h->heads_kv != c->heads_kv || h->dim != c->dim || h->act != c->act)
    return fail_with(TFX_EINVAL, "heads_kv, dim and act must be the cache's");
  if (layer < 0 || layer >= c->layers) return fail_with(TFX_EINVAL, "layer %d of %d", layer, c->layers);
  if (batch < 0) return fail_with(TFX_EINVAL, "batch=%d", batch);
  if (shared < 0 || shared > c->width * c->page_size)
    return fail_with(TFX_EINVAL, "shared=%d outside 0..%d", shared, c->width * c->page_size);
  if ((rc = check_reserved(c))) return rc;
  const CachePriv* pv = static_cast<const CachePriv*>(c->priv);
  // the kernel numbers the slices of the batch's own tokens, 4,096 / dim each, in 32 bits
  const int64_t slices = ((int64_t)c->width * c->page_size) / (4096 / c->dim) + 1;
  if (batch * slices > INT32_MAX)
    return fail_with(TFX_EUNSUPPORTED, "batch=%d sequences of up to %lld tokens", batch, (long long)c->width * c->page_size);
  if (batch > pv->max_batch || h->heads_q > pv->heads_q)
    return fail_with(TFX_ENOTRESERVED, "reserved for %d sequences of %d heads, called with %d of %d", pv->max_batch,
                     pv->heads_q, batch, h->heads_q);
  if (!batch) return 0;
  if (!seqs) return fail_with(TFX_EINVAL, "null seqs");
  if ((rc = check_rows("q", q, ldq, (int64_t)h->heads_q * h->dim))) return rc;
  if ((rc = check_rows("out", out, ldo, (int64_t)h->heads_q * h->dim))) return rc;
  tfx::DecodeAttnArgs a = {};
  const bool coded = c->store != TFX_STORE_ACT;
  const int64_t ld = (int64_t)c->heads_kv * c->dim;
  const void *kl = layer_of<const void>(c, c->k, layer), *vl = layer_of<const void>(c, c->v, layer);
  if (coded) {
    if ((rc = make_code_map(&a.k, kl, c)) || (rc = make_code_map(&a.v, vl, c))) return rc;
    a.k_scale = scales_of(c, c->k_scale, layer);
    a.v_scale = scales_of(c, c->v_scale, layer);
  } else {
    if ((rc = make_map(&a.k, kl, c->act, c->dim, c->heads_kv, c->page_size, ld, c->pages, page_values(c), 16, c->dim / 64))) return rc;
    if ((rc = make_map(&a.v, vl, c->act, c->dim, c->heads_kv, c->page_size, ld, c->pages, page_values(c), 16, c->dim / 64))) return rc;
  }
  a.q = q;
  a.out = out;
  a.ldq = ldq;
  a.ldo = ldo;
  a.seqs = seqs;
  a.lens = lens_of(c);
  a.tables = tables_of(c);
  a.scale_log2 = h->scale * 1.4426950408889634f;
  a.heads_q = h->heads_q;
  a.heads_kv = h->heads_kv;
  a.group = h->heads_q / h->heads_kv;
  a.batch = batch;
  a.shared = coded ? coded_prefix(c, batch, shared) : shared;
  a.page_size = c->page_size;
  a.page_shift = page_shift(c);
  a.pages = c->pages;
  a.slots = c->slots;
  a.width = c->width;
  if (coded && a.shared) {
    const int64_t rows = (int64_t)batch * a.group, per = tfx::prefix_q8_rows();
    a.mt = (int)((rows + per - 1) / per);
    const int64_t rest = (int64_t)c->heads_kv * a.mt, fill = tfx::multiprocessors() / rest, tiles = tfx::prefix_q8_tiles(a.shared);
    // of the most tiles that a share must have then, as few shares: each leaves partial results
    const int64_t most = fill < 1 ? tiles : (tiles + fill - 1) / fill;
    a.pre_splits = (int)((tiles + most - 1) / most);
    if (rest * a.pre_splits > INT32_MAX) return fail_with(TFX_EUNSUPPORTED, "%lld tiles of rows", (long long)rest);
    a.items = (int)(rest * a.pre_splits);
  }
  if (!coded && many_rows(batch, a.group) && shared >= 256) {
    a.per_tile = heads_per_tile(a.group);
    a.tokens = 128 / a.per_tile;
    const int most = 2 * a.tokens, tiles = (batch + most - 1) / most;
    a.tokens = (batch + 2 * tiles - 1) / (2 * tiles);  // the sequences spread evenly over the tiles' CTAs
    a.pre_splits = prefix_splits(batch, h->heads_q, h->heads_kv, shared);
    a.sub = a.group / a.per_tile;
    a.hg = a.heads_kv * a.sub;
    a.mt = (batch + 2 * a.tokens - 1) / (2 * a.tokens);
    a.items = a.hg * a.mt * a.pre_splits;
    const int box = c->page_size < 64 ? c->page_size : 64;
    if ((rc = make_q_map(&a.qmap, q, c->act, c->dim, h->heads_q, batch, ldq, a.per_tile, a.tokens))) return rc;
    if ((rc = make_map(&a.kt, kl, c->act, c->dim, c->heads_kv, c->page_size, ld, c->pages, page_values(c), box, 1))) return rc;
    if ((rc = make_map(&a.vt, vl, c->act, c->dim, c->heads_kv, c->page_size, ld, c->pages, page_values(c), box, 1))) return rc;
  }
  a.warps = decode_warps(c);
  a.own_rows = a.group < kRowTile ? a.group : kRowTile;
  const DecodeScratch d = decode_scratch(c, batch, h->heads_q);
  if (d.bytes > pv->part_bytes)
    return fail_with(TFX_ENOTRESERVED, "%d sequences of %d heads take more scratch than was reserved", batch, h->heads_q);
  a.runs = reinterpret_cast<int2*>(pv->part + d.runs);
  a.own_ml = reinterpret_cast<float2*>(pv->part + d.own_ml);
  a.pre_ml = reinterpret_cast<float2*>(pv->part + d.pre_ml);
  a.own_o = reinterpret_cast<float*>(pv->part + d.own_o);
  a.pre_o = reinterpret_cast<float*>(pv->part + d.pre_o);
  a.err = error_word();
  a.spin = tfx::spin_limit();
  if (!a.err) return fail_with(TFX_ECUDA, "no device error word");
  if (a.pre_splits && (rc = coded ? tfx::launch_prefix_q8(a, c->act, c->store, c->dim, stream)
                                  : tfx::launch_prefix(a, c->act, c->dim, stream)))
    return rc;
  return coded ? tfx::launch_decode_q8(a, c->act, c->store, c->dim, stream) : tfx::launch_decode(a, c->act, c->dim, stream);
}

int tfx_attn_debug_error(int* device_error) {
  if (!device_error) return fail_with(TFX_EINVAL, "null argument");
  const int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(device_error, tfx::g_attn_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(tfx::g_attn_error, &zero, sizeof(int));
  return e == cudaSuccess ? 0 : fail_with(TFX_ECUDA, "reading the device error word: %s", cudaGetErrorString(e));
}

}  // extern "C"
