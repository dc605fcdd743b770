// C-ABI of the attention half of a block: argument checks of the key-value
// cache's operators.  The kernels are in kv_cache.hip and kv_attention.hip.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "kernels.hpp"
#include "kv_cache.hpp"
#include "moe_layout.hpp"

namespace nvfp4 {

namespace {

int64_t value_bytes(int32_t dtype) { return dtype == MOE_F32 ? 4 : dtype == MOE_BF16 || dtype == MOE_F16 ? 2 : 0; }

struct Range {
  const void* p;
  int64_t bytes;
};

// Whether `x` overlaps one of the others.
bool meets(Range x, std::initializer_list<Range> others) {
  for (const Range& o : others)
    if (x.p && o.p && x.bytes > 0 && o.bytes > 0 && overlap(x.p, x.bytes, o.p, o.bytes)) return true;
  return false;
}

int64_t product(std::initializer_list<int64_t> f) {
  __int128 n = 1;
  for (const int64_t v : f) {
    n *= v;
    if (n > INT64_MAX) return INT64_MAX;
  }
  return static_cast<int64_t>(n);
}

// Bytes from the first to the last element of [tokens, heads, D] with these strides.
int64_t strided(int64_t tokens, int64_t ld, int64_t heads, int64_t ld_head, int64_t D, int64_t bytes) {
  const __int128 n = (static_cast<__int128>(tokens - 1) * ld + static_cast<__int128>(heads - 1) * ld_head + D) * bytes;
  return n > INT64_MAX ? INT64_MAX : static_cast<int64_t>(n);
}

struct CacheRanges {
  Range codes, scales, tails, tail_scales;
};

CacheRanges ranges(const kv_cache& c) {
  const int64_t heads = 2 * int64_t{c.kv_heads}, page = int64_t{c.page_size} * c.head_dim;
  return {{c.codes_dev, product({c.num_pages, heads, page})},
          {c.scales_dev, product({c.num_pages, heads, 4})},
          {c.tails_dev, product({c.num_slots, heads, page, 2})},
          {c.tail_scales_dev, product({c.num_slots, heads, c.page_size, 4})}};
}

int check_sizes(const kv_cache* c, const kv_batch* b) {
  if (!c || !b) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL cache or batch");
  if (c->num_pages < 1 || c->num_pages > INT32_MAX || c->num_slots < 1 || c->num_slots > INT32_MAX)
    return api_fail(NVFP4_ERR_INVALID_ARG, "num_pages and num_slots must be in [1, 2^31) (got %lld, %lld)",
                    (long long)c->num_pages, (long long)c->num_slots);
  if (c->kv_heads < 1 || c->kv_heads > 1024)
    return api_fail(NVFP4_ERR_INVALID_ARG, "kv_heads must be in [1, 1024] (got %d)", c->kv_heads);
  if (c->head_dim < 64 || c->head_dim > 256 || c->head_dim % 64 != 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "head_dim must be 64, 128, 192 or 256 (got %d)", c->head_dim);
  if (c->page_size < 16 || c->page_size > 128 || (c->page_size & (c->page_size - 1)) != 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "page_size must be 16, 32, 64 or 128 (got %d)", c->page_size);
  if (b->entries < 0 || b->tokens < 0 || b->entries > INT32_MAX - 1 || b->tokens > INT32_MAX)
    return api_fail(NVFP4_ERR_INVALID_ARG, "entries and tokens must be in [0, 2^31) (got %lld, %lld)",
                    (long long)b->entries, (long long)b->tokens);
  if (!b->cu_dev && b->tokens != b->entries)
    return api_fail(NVFP4_ERR_INVALID_ARG, "without cu every entry has one token (got %lld entries, %lld tokens)",
                    (long long)b->entries, (long long)b->tokens);
  if (b->table_width < 1 || b->table_width > (int64_t{1} << 30) / c->page_size)
    return api_fail(NVFP4_ERR_INVALID_ARG, "table_width must be >= 1, table_width * page_size <= 2^30 (got %lld)",
                    (long long)b->table_width);
  if (b->ld_table < b->table_width || b->ld_table > (int64_t{1} << 31))
    return api_fail(NVFP4_ERR_INVALID_ARG, "ld_table must be in [table_width, 2^31] (got %lld)", (long long)b->ld_table);
  return NVFP4_OK;
}

int check_pointers(const kv_cache& c, const kv_batch& b) {
  if (!c.codes_dev || !c.scales_dev || !c.tails_dev || !c.tail_scales_dev || !b.table_dev || !b.lens_dev || !b.slots_dev)
    return api_fail(NVFP4_ERR_INVALID_ARG, "NULL pointer in the cache or the batch");
  if (!aligned(c.codes_dev, 16) || !aligned(c.scales_dev, 16) || !aligned(c.tails_dev, 16) ||
      !aligned(c.tail_scales_dev, 16))
    return api_fail(NVFP4_ERR_INVALID_ARG, "the cache's memory must be 16-byte aligned");
  if (!aligned(b.table_dev, 4) || !aligned(b.lens_dev, 4) || !aligned(b.slots_dev, 4) || !aligned(b.cu_dev, 4))
    return api_fail(NVFP4_ERR_INVALID_ARG, "table, lens, slots and cu must be aligned to their element");
  return NVFP4_OK;
}

// A tensor [tokens, heads, D] of 16-byte pieces.
int check_rows(const char* name, const void* p, int64_t ld, int64_t ld_head) {
  if (!p) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL %s", name);
  if (ld % 8 != 0 || ld_head % 8 != 0 || ld < 0 || ld_head < 0 || ld > (int64_t{1} << 31) || ld_head > (int64_t{1} << 31))
    return api_fail(NVFP4_ERR_INVALID_ARG, "%s: strides of tokens and heads must be multiples of 8 in [0, 2^31] (got %lld, %lld)",
                    name, (long long)ld, (long long)ld_head);
  if (!aligned(p, 16)) return api_fail(NVFP4_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  return NVFP4_OK;
}

Range table_range(const kv_batch& b) {
  return {b.table_dev, product({(b.entries - 1) * b.ld_table + b.table_width, 4})};
}
Range lens_range(const kv_batch& b) { return {b.lens_dev, b.entries * 4}; }
Range slots_range(const kv_batch& b) { return {b.slots_dev, b.entries * 4}; }
Range cu_range(const kv_batch& b) { return {b.cu_dev, (b.entries + 1) * 4}; }

KvParams params(const kv_cache& c, const kv_batch& b) {
  KvParams p{};
  p.codes = static_cast<uint8_t*>(c.codes_dev);
  p.scales = c.scales_dev;
  p.tails = static_cast<_Float16*>(c.tails_dev);
  p.tail_scales = c.tail_scales_dev;
  p.pages = c.num_pages;
  p.slots = c.num_slots;
  p.table = b.table_dev;
  p.lens = b.lens_dev;
  p.slot = b.slots_dev;
  p.cu = b.cu_dev;
  p.ld_table = b.ld_table;
  p.width = static_cast<int>(b.table_width);
  p.entries = static_cast<int>(b.entries);
  p.tokens = static_cast<int>(b.tokens);
  p.heads = c.kv_heads;
  p.D = c.head_dim;
  p.P = c.page_size;
  p.shift = __builtin_ctz(static_cast<unsigned>(c.page_size));
  return p;
}

constexpr int64_t kMostBlocks = INT32_MAX;

int check_blocks(int64_t blocks) {
  if (blocks > kMostBlocks)
    return api_fail(NVFP4_ERR_INVALID_ARG, "the batch needs %lld blocks, more than one launch has", (long long)blocks);
  return NVFP4_OK;
}

int check_heads(const kv_cache& c, const kv_batch& b, int32_t heads) {
  if (heads < 1 || heads % c.kv_heads != 0 || heads / c.kv_heads > 64)
    return api_fail(NVFP4_ERR_INVALID_ARG, "heads must be a multiple of kv_heads, at most 64 times as many (got %d of %d)",
                    heads, c.kv_heads);
  if (b.tokens * (heads / c.kv_heads) > (int64_t{1} << 28))
    return api_fail(NVFP4_ERR_INVALID_ARG, "tokens * heads / kv_heads must be <= 2^28");
  return NVFP4_OK;
}

}  // namespace

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int kv_append(const kv_cache* cache, const kv_batch* batch, const void* k_dev, int64_t ld_k, int64_t ld_k_head,
              const void* v_dev, int64_t ld_v, int64_t ld_v_head, int32_t dtype, void* stream) {
  int st = check_sizes(cache, batch);
  if (st != NVFP4_OK) return st;
  if (dtype != MOE_BF16 && dtype != MOE_F16)
    return api_fail(NVFP4_ERR_INVALID_ARG, "keys and values must be bf16 or fp16 (got dtype %d)", dtype);
  const kv_cache& c = *cache;
  const kv_batch& b = *batch;
  if (b.entries == 0 || b.tokens == 0) return api_ok();
  st = check_pointers(c, b);
  if (st == NVFP4_OK) st = check_rows("k", k_dev, ld_k, ld_k_head);
  if (st == NVFP4_OK) st = check_rows("v", v_dev, ld_v, ld_v_head);
  const KvParams p = params(c, b);
  if (st == NVFP4_OK) st = check_blocks(kv_page_blocks(p));
  if (st != NVFP4_OK) return st;
  const Range k{k_dev, strided(b.tokens, ld_k, c.kv_heads, ld_k_head, c.head_dim, 2)};
  const Range v{v_dev, strided(b.tokens, ld_v, c.kv_heads, ld_v_head, c.head_dim, 2)};
  const CacheRanges r = ranges(c);
  for (const Range& own : {r.codes, r.scales, r.tails, r.tail_scales})
    if (meets(own, {k, v, table_range(b), lens_range(b), slots_range(b), cu_range(b)}))
      return api_fail(NVFP4_ERR_ALIAS, "the cache overlaps an input");
  const hipError_t e = launch_kv_append(p, k_dev, ld_k, ld_k_head, v_dev, ld_v, ld_v_head, dtype,
                                        static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "kv_append launch");
  return api_ok();
}

int kv_attention_workspace(const kv_cache* cache, const kv_batch* batch, int32_t heads, int64_t* bytes) {
  if (!bytes) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL output");
  int st = check_sizes(cache, batch);
  if (st == NVFP4_OK) st = check_heads(*cache, *batch, heads);
  if (st != NVFP4_OK) return st;
  *bytes = 0;
  if (batch->entries == 0 || batch->tokens == 0) return api_ok();
  int64_t blocks = 0;
  *bytes = kv_attention_bytes(params(*cache, *batch), heads / cache->kv_heads, &blocks);
  return api_ok();
}

int kv_attention(const kv_cache* cache, const kv_batch* batch, const void* q_dev, int64_t ld_q, int64_t ld_q_head,
                 int32_t heads, int32_t dtype, float scale, int64_t window, void* workspace_dev, int64_t workspace_bytes,
                 void* out_dev, int64_t ld_out, int64_t ld_out_head, void* stream) {
  int st = check_sizes(cache, batch);
  if (st == NVFP4_OK) st = check_heads(*cache, *batch, heads);
  if (st != NVFP4_OK) return st;
  if (dtype != MOE_BF16 && dtype != MOE_F16)
    return api_fail(NVFP4_ERR_INVALID_ARG, "queries must be bf16 or fp16 (got dtype %d)", dtype);
  if (!std::isfinite(scale)) return api_fail(NVFP4_ERR_INVALID_ARG, "scale must be finite");
  if (window < 0) return api_fail(NVFP4_ERR_INVALID_ARG, "window must be >= 0 (got %lld)", (long long)window);
  const kv_cache& c = *cache;
  const kv_batch& b = *batch;
  if (b.entries == 0 || b.tokens == 0) return api_ok();
  st = check_pointers(c, b);
  if (st == NVFP4_OK) st = check_rows("q", q_dev, ld_q, ld_q_head);
  if (st == NVFP4_OK) st = check_rows("out", out_dev, ld_out, ld_out_head);
  if (st != NVFP4_OK) return st;
  const int64_t D = c.head_dim, row = heads > 1 ? (heads - 1) * ld_out_head + D : D;
  const int64_t column = b.tokens > 1 ? (b.tokens - 1) * ld_out + D : D;
  if (!((heads == 1 || ld_out_head >= D) && (b.tokens == 1 || ld_out >= row)) &&
      !((b.tokens == 1 || ld_out >= D) && (heads == 1 || ld_out_head >= column)))
    return api_fail(NVFP4_ERR_INVALID_ARG, "out: its rows overlap (strides %lld, %lld)", (long long)ld_out,
                    (long long)ld_out_head);
  KvAttention k{};
  k.c = params(c, b);
  k.group = heads / c.kv_heads;
  int64_t blocks = 0;
  const int64_t need = kv_attention_bytes(k.c, k.group, &blocks);
  st = check_blocks(blocks);
  if (st != NVFP4_OK) return st;
  if (need > 0 && (!workspace_dev || !aligned(workspace_dev, 16) || workspace_bytes < need))
    return api_fail(NVFP4_ERR_INVALID_ARG, "workspace must be 16-byte aligned, of at least %lld bytes (got %lld)",
                    (long long)need, (long long)workspace_bytes);
  const Range q{q_dev, strided(b.tokens, ld_q, heads, ld_q_head, c.head_dim, 2)};
  const Range out{out_dev, strided(b.tokens, ld_out, heads, ld_out_head, c.head_dim, 2)};
  const Range ws{workspace_dev, need};
  const CacheRanges r = ranges(c);
  for (const Range& own : {out, ws})
    if (meets(own, {q, r.codes, r.scales, r.tails, r.tail_scales, table_range(b), lens_range(b), slots_range(b),
                    cu_range(b)}))
      return api_fail(NVFP4_ERR_ALIAS, "out or the workspace overlaps an input");
  if (meets(out, {ws})) return api_fail(NVFP4_ERR_ALIAS, "out overlaps the workspace");
  k.q = q_dev;
  k.out = out_dev;
  k.ldq = ld_q;
  k.ldq_head = ld_q_head;
  k.ldo = ld_out;
  k.ldo_head = ld_out_head;
  k.scale = scale;
  // (no sequence is longer than 2^30)
  k.window = static_cast<int>(window < (int64_t{1} << 30) ? window : 0);
  k.dtype = dtype;
  const hipError_t e = launch_kv_attention(k, workspace_dev, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "kv_attention launch");
  return api_ok();
}

int kv_read(const kv_cache* cache, const kv_batch* batch, void* k_out_dev, void* v_out_dev, int32_t dtype, void* stream) {
  int st = check_sizes(cache, batch);
  if (st != NVFP4_OK) return st;
  const int64_t bytes = value_bytes(dtype);
  if (!bytes) return api_fail(NVFP4_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  const kv_cache& c = *cache;
  const kv_batch& b = *batch;
  if (b.entries == 0 || b.tokens == 0) return api_ok();
  st = check_pointers(c, b);
  if (st != NVFP4_OK) return st;
  if (!k_out_dev || !v_out_dev) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL output");
  if (!aligned(k_out_dev, 16) || !aligned(v_out_dev, 16))
    return api_fail(NVFP4_ERR_INVALID_ARG, "outputs must be 16-byte aligned");
  const KvParams p = params(c, b);
  st = check_blocks(kv_page_blocks(p));
  if (st != NVFP4_OK) return st;
  const int64_t n = product({b.tokens, c.kv_heads, c.head_dim, bytes});
  const Range k{k_out_dev, n}, v{v_out_dev, n};
  const CacheRanges r = ranges(c);
  for (const Range& own : {k, v})
    if (meets(own, {r.codes, r.scales, r.tails, r.tail_scales, table_range(b), lens_range(b), slots_range(b), cu_range(b)}))
      return api_fail(NVFP4_ERR_ALIAS, "an output overlaps an input");
  if (meets(k, {v})) return api_fail(NVFP4_ERR_ALIAS, "the outputs overlap");
  const hipError_t e = launch_kv_read(p, k_out_dev, v_out_dev, dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "kv_read launch");
  return api_ok();
}

int kv_fork(const kv_cache* cache, const kv_batch* batch, const int32_t* src_dev, const int32_t* dst_dev, int64_t pairs,
            void* stream) {
  if (!cache || !batch) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL cache or batch");
  kv_batch b = *batch;
  b.cu_dev = nullptr;
  b.tokens = b.entries;
  int st = check_sizes(cache, &b);
  if (st != NVFP4_OK) return st;
  const kv_cache& c = *cache;
  if (pairs < 0 || pairs > INT32_MAX)
    return api_fail(NVFP4_ERR_INVALID_ARG, "pairs must be in [0, 2^31) (got %lld)", (long long)pairs);
  if (b.entries == 0 || pairs == 0) return api_ok();
  st = check_pointers(c, b);
  if (st == NVFP4_OK) st = check_blocks(pairs * (1 + 2 * int64_t{c.kv_heads}));
  if (st != NVFP4_OK) return st;
  if (!src_dev || !dst_dev || !aligned(src_dev, 4) || !aligned(dst_dev, 4))
    return api_fail(NVFP4_ERR_INVALID_ARG, "src and dst must be given, aligned to their element");
  const Range s{src_dev, pairs * 4}, d{dst_dev, pairs * 4};
  const CacheRanges r = ranges(c);
  if (meets(table_range(b), {lens_range(b), slots_range(b), s, d}) || meets(lens_range(b), {slots_range(b), s, d}))
    return api_fail(NVFP4_ERR_ALIAS, "table and lens are written: they overlap each other or an input");
  for (const Range& own : {r.tails, r.tail_scales, r.codes, r.scales})
    if (meets(own, {table_range(b), lens_range(b), slots_range(b), s, d}))
      return api_fail(NVFP4_ERR_ALIAS, "the cache overlaps an input");
  const hipError_t e = launch_kv_fork(params(c, b), src_dev, dst_dev, static_cast<int>(pairs),
                                      static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "kv_fork launch");
  return api_ok();
}

}  // extern "C"
