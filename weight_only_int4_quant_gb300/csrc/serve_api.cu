// C ABI of the multi-request serving operators: argument validation and dispatch.
#include <algorithm>
#include <cmath>

#include "serve.cuh"

using namespace tlq;

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// [a, a + an) and [b, b + bn) share bytes
bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an && bn && x < y + bn && y < x + an;
}

// bytes of rows of `inner` elements of `size` bytes at stride ld
size_t span(long long rows, long long ld, long long inner, size_t size) {
  return rows < 1 ? 0 : (size_t)((rows - 1) * ld + inner) * size;
}

int check_geometry(int page, int head_dim, int group, const char* who) {
  if (page < 16 || page > 256 || (page & (page - 1)))
    return set_error(TLQ_EINVAL, "%s: page_size=%d (16, 32, 64, 128 or 256 tokens)", who, page);
  if (head_dim != 64 && head_dim != 128)
    return set_error(head_dim > 0 ? TLQ_EUNSUPPORTED : TLQ_EINVAL, "%s: head_dim=%d (64 or 128)", who, head_dim);
  if (group != 64 && group != 128)
    return set_error(group > 0 ? TLQ_EUNSUPPORTED : TLQ_EINVAL, "%s: group=%d (64 or 128)", who, group);
  if (head_dim % group) return set_error(TLQ_EINVAL, "%s: head_dim=%d is not a multiple of group=%d", who, head_dim, group);
  return TLQ_OK;
}

tlq_status check_cache(const tl_kv4_cache* c, KvCache* out, const char* who) {
  if (!c) return set_error(TLQ_EINVAL, "%s: null cache", who);
  const tlq_status st = (tlq_status)check_geometry(c->page_size, c->head_dim, c->group, who);
  if (st != TLQ_OK) return st;
  if (!c->blocks) return set_error(TLQ_EINVAL, "%s: null cache blocks", who);
  if (!aligned(c->blocks, 16)) return set_error(TLQ_EINVAL, "%s: cache blocks must be 16-byte aligned", who);
  if (c->heads < 1 || c->heads > 4096) return set_error(TLQ_EINVAL, "%s: heads=%d (1..4096)", who, c->heads);
  if (c->num_pages < 1 || c->num_pages > 0x7fffffffll)
    return set_error(TLQ_EINVAL, "%s: num_pages=%lld (1..2^31-1)", who, (long long)c->num_pages);
  if (c->num_pages * c->heads > 0x7fffffffll)
    return set_error(TLQ_EINVAL, "%s: num_pages=%lld x heads=%d (at most 2^31 - 1 blocks)", who, (long long)c->num_pages,
                     c->heads);
  out->blocks = static_cast<uint8_t*>(c->blocks);
  out->num_pages = c->num_pages;
  out->heads = c->heads;
  out->page = c->page_size;
  out->group = c->group;
  out->page_shift = 0;
  while ((1 << out->page_shift) < c->page_size) ++out->page_shift;
  out->block_bytes = kv_block_bytes(c->page_size, c->head_dim, c->group);
  return TLQ_OK;
}

// Up to this many (query, head) rows to a key head a request's attention runs
// on the kernel for few rows.  Its time grows with every 16 rows, the other
// kernel's tiles are 256 rows high.  Few / many, 8 key heads of 128: 16 requests on
// 8000 tokens, 32 rows 96 / 189 us, 64 rows 179 / 188, 96 rows 261 / 185; on 2000
// tokens, 64 rows 60 / 80, 96 rows 84 / 81.  That is the crossing of batches that
// fill the GPU; the rule knows rows alone, and a single short request above it
// would do better here (one on 1000 tokens, 128 rows: 16 / 36).
constexpr int kFewRows = 64;

size_t cache_bytes(const KvCache& c) { return (size_t)c.num_pages * c.heads * c.block_bytes; }

}  // namespace

extern "C" {

size_t tl_kv4_block_bytes(int page_size, int head_dim, int group) {
  clear_error();
  if (check_geometry(page_size, head_dim, group, "tl_kv4_block_bytes") != TLQ_OK) return 0;
  return (size_t)kv_block_bytes(page_size, head_dim, group);
}

tlq_status tl_kv_plan(const int32_t* cached, const int32_t* added, int requests, int32_t* table, int ld_table,
                      const int32_t* free_pages, int num_free, const int32_t* free_head, int page_size,
                      int64_t num_pages, int32_t* q_start, int32_t* seq_lens, int32_t* token_req, int32_t* token_pos,
                      int64_t* slots, int capacity, int32_t* counts, void* stream) {
  clear_error();
  const char* who = "tl_kv_plan";
  if (requests < 0) return set_error(TLQ_EINVAL, "%s: requests=%d", who, requests);
  if (capacity < 0) return set_error(TLQ_EINVAL, "%s: capacity=%d", who, capacity);
  if (num_free < 0) return set_error(TLQ_EINVAL, "%s: num_free=%d", who, num_free);
  if (page_size < 1 || page_size > 65536 || (page_size & (page_size - 1)))
    return set_error(TLQ_EINVAL, "%s: page_size=%d (a power of two)", who, page_size);
  if (num_pages < 1 || num_pages > 0x7fffffffll)
    return set_error(TLQ_EINVAL, "%s: num_pages=%lld (1..2^31-1)", who, (long long)num_pages);
  if (requests > 0 && ld_table < 1) return set_error(TLQ_EINVAL, "%s: ld_table=%d (must be >= 1)", who, ld_table);
  if (!q_start || !counts || (requests > 0 && (!cached || !added || !table || !seq_lens)) ||
      (num_free > 0 && !free_pages) || (capacity > 0 && (!token_req || !token_pos || !slots)))
    return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (!aligned(cached, 4) || !aligned(added, 4) || !aligned(table, 4) || !aligned(free_pages, 4) ||
      !aligned(free_head, 4) || !aligned(q_start, 4) || !aligned(seq_lens, 4) || !aligned(token_req, 4) ||
      !aligned(token_pos, 4) || !aligned(counts, 4) || !aligned(slots, 8))
    return set_error(TLQ_EINVAL, "%s: arrays must be aligned to their elements", who);
  const struct {
    const void* p;
    size_t n;
  } in[4] = {{cached, 4 * (size_t)requests}, {added, 4 * (size_t)requests}, {free_pages, 4 * (size_t)num_free},
             {free_head, free_head ? size_t(4) : 0}},
    res[7] = {{table, 4 * (size_t)requests * ld_table}, {q_start, 4 * ((size_t)requests + 1)},
              {seq_lens, 4 * (size_t)requests}, {token_req, 4 * (size_t)capacity}, {token_pos, 4 * (size_t)capacity},
              {slots, 8 * (size_t)capacity}, {counts, 16}};
  for (int i = 0; i < 7; ++i) {
    for (int j = 0; j < 4; ++j)
      if (overlap(res[i].p, res[i].n, in[j].p, in[j].n))
        return set_error(TLQ_EINVAL, "%s: an output overlaps an input", who);
    for (int j = 0; j < i; ++j)
      if (overlap(res[i].p, res[i].n, res[j].p, res[j].n))
        return set_error(TLQ_EINVAL, "%s: two outputs overlap", who);
  }
  KvPlanArgs a;
  a.cached = cached;
  a.added = added;
  a.requests = requests;
  a.table = table;
  a.ld_table = ld_table;
  a.free_pages = free_pages;
  a.num_free = num_free;
  a.free_head = free_head;
  a.page = page_size;
  a.num_pages = num_pages;
  a.q_start = q_start;
  a.seq_lens = seq_lens;
  a.token_req = token_req;
  a.token_pos = token_pos;
  a.slots = reinterpret_cast<long long*>(slots);
  a.capacity = capacity;
  a.counts = counts;
  return launch_kv_plan(a, static_cast<cudaStream_t>(stream));
}

tlq_status tl_kv4_append(const tl_kv4_cache* cache, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                         const int64_t* slots, int tokens, void* stream) {
  clear_error();
  const char* who = "tl_kv4_append";
  KvCache c;
  const tlq_status st = check_cache(cache, &c, who);
  if (st != TLQ_OK) return st;
  if (tokens < 0) return set_error(TLQ_EINVAL, "%s: tokens=%d", who, tokens);
  if (tokens == 0) return TLQ_OK;
  if (!k || !v || !slots) return set_error(TLQ_EINVAL, "%s: null pointer", who);
  const long long row = (long long)c.heads * cache->head_dim;
  if (tokens > 1 && (ldk < row || ldv < row || ldk % 8 || ldv % 8))
    return set_error(TLQ_EINVAL, "%s: ldk=%lld ldv=%lld (at least heads*head_dim = %lld, multiples of 8)", who,
                     (long long)ldk, (long long)ldv, row);
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return set_error(TLQ_EINVAL, "%s: k and v must be 16-byte aligned, slots 8-byte", who);
  if (overlap(c.blocks, cache_bytes(c), k, span(tokens, ldk, row, 2)) ||
      overlap(c.blocks, cache_bytes(c), v, span(tokens, ldv, row, 2)) ||
      overlap(c.blocks, cache_bytes(c), slots, 8 * (size_t)tokens))
    return set_error(TLQ_EINVAL, "%s: the cache overlaps an input", who);
  return launch_kv4_append(c, cache->head_dim, reinterpret_cast<const __half*>(k), ldk,
                           reinterpret_cast<const __half*>(v), ldv, reinterpret_cast<const long long*>(slots), tokens,
                           static_cast<cudaStream_t>(stream));
}

tlq_status tl_kv4_read(const tl_kv4_cache* cache, const int64_t* slots, int tokens, uint16_t* k, uint16_t* v,
                       void* stream) {
  clear_error();
  const char* who = "tl_kv4_read";
  KvCache c;
  const tlq_status st = check_cache(cache, &c, who);
  if (st != TLQ_OK) return st;
  if (tokens < 0) return set_error(TLQ_EINVAL, "%s: tokens=%d", who, tokens);
  if (tokens == 0) return TLQ_OK;
  if (!k || !v || !slots) return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8))
    return set_error(TLQ_EINVAL, "%s: k and v must be 16-byte aligned, slots 8-byte", who);
  const size_t bytes = 2 * (size_t)tokens * c.heads * cache->head_dim;
  if (overlap(k, bytes, v, bytes) || overlap(k, bytes, c.blocks, cache_bytes(c)) ||
      overlap(v, bytes, c.blocks, cache_bytes(c)) || overlap(k, bytes, slots, 8 * (size_t)tokens) ||
      overlap(v, bytes, slots, 8 * (size_t)tokens))
    return set_error(TLQ_EINVAL, "%s: an output overlaps an input or the other output", who);
  return launch_kv4_read(c, cache->head_dim, reinterpret_cast<const long long*>(slots), tokens,
                         reinterpret_cast<__half*>(k), reinterpret_cast<__half*>(v),
                         static_cast<cudaStream_t>(stream));
}

size_t tl_kv4_attention_workspace_size(int q_heads, int heads, int head_dim, int max_q) {
  clear_error();
  if (q_heads < 1 || heads < 1 || q_heads % heads || (head_dim != 64 && head_dim != 128) || max_q < 0) return 0;
  return kv4_decode_workspace(head_dim) + kv4_prefill_workspace(head_dim);
}

tlq_status tl_kv4_attention(const tl_kv4_cache* cache, const uint16_t* q, int64_t ldq, int q_heads, uint16_t* out,
                            int64_t ldo, const int32_t* q_start, const int32_t* seq_lens, const int32_t* table,
                            int ld_table, int requests, int tokens, int max_q, float scale, int window,
                            void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  const char* who = "tl_kv4_attention";
  KvAttention a{};
  const tlq_status st = check_cache(cache, &a.cache, who);
  if (st != TLQ_OK) return st;
  if (q_heads < 1 || q_heads % a.cache.heads)
    return set_error(TLQ_EINVAL, "%s: q_heads=%d is not a positive multiple of the cache's heads=%d", who, q_heads,
                     a.cache.heads);
  if (requests < 0 || tokens < 0 || max_q < 0)
    return set_error(TLQ_EINVAL, "%s: requests=%d tokens=%d max_q=%d", who, requests, tokens, max_q);
  if (window < 0) return set_error(TLQ_EINVAL, "%s: window=%d (0: none)", who, window);
  if (!std::isfinite(scale)) return set_error(TLQ_EINVAL, "%s: scale is not finite", who);
  if (requests == 0 || tokens == 0 || max_q == 0) return TLQ_OK;
  if (!q || !out || !q_start || !seq_lens || !table) return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (ld_table < 1) return set_error(TLQ_EINVAL, "%s: ld_table=%d (must be >= 1)", who, ld_table);
  const long long row = (long long)q_heads * cache->head_dim;
  if (tokens > 1 && (ldq < row || ldo < row || ldq % 8 || ldo % 8))
    return set_error(TLQ_EINVAL, "%s: ldq=%lld ldo=%lld (at least q_heads*head_dim = %lld, multiples of 8)", who,
                     (long long)ldq, (long long)ldo, row);
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(q_start, 4) ||
      !aligned(seq_lens, 4) || !aligned(table, 4))
    return set_error(TLQ_EINVAL, "%s: q, out and the workspace must be 16-byte aligned", who);
  max_q = std::min(max_q, tokens);
  if ((long long)max_q * (q_heads / a.cache.heads) > 0x3fffffff)
    return set_error(TLQ_EUNSUPPORTED, "%s: max_q=%d x %d query heads to a key head (at most 2^30 rows)", who, max_q,
                     q_heads / a.cache.heads);
  const size_t need = tl_kv4_attention_workspace_size(q_heads, a.cache.heads, cache->head_dim, max_q);
  if (!workspace || workspace_bytes < need)
    return set_error(TLQ_EINVAL, "%s: workspace of %zu bytes (%zu needed)", who, workspace ? workspace_bytes : size_t(0),
                     need);
  const size_t qb = span(tokens, ldq, row, 2), ob = span(tokens, ldo, row, 2), cb = cache_bytes(a.cache);
  if (overlap(out, ob, q, qb) || overlap(out, ob, a.cache.blocks, cb) || overlap(workspace, need, q, qb) ||
      overlap(workspace, need, out, ob) || overlap(workspace, need, a.cache.blocks, cb))
    return set_error(TLQ_EINVAL, "%s: out or the workspace overlaps another buffer", who);
  const struct {
    const void* p;
    size_t n;
  } lengths[3] = {{q_start, 4 * ((size_t)requests + 1)}, {seq_lens, 4 * (size_t)requests},
                  {table, 4 * (size_t)requests * ld_table}};
  for (const auto& l : lengths)
    if (overlap(out, ob, l.p, l.n) || overlap(workspace, need, l.p, l.n))
      return set_error(TLQ_EINVAL, "%s: out or the workspace overlaps the batch's arrays", who);
  a.batch = KvBatch{q_start, seq_lens, table, ld_table, requests, tokens, max_q};
  a.head_dim = cache->head_dim;
  a.q_heads = q_heads;
  a.q = reinterpret_cast<const __half*>(q);
  a.ldq = ldq;
  a.out = reinterpret_cast<__half*>(out);
  a.ldo = ldo;
  a.scale = scale;
  a.window = window >= kMaxContext ? 0 : window;  // a window that no context outgrows is none
  // The tensor-core kernel takes one scale a row, so rows in two groups stay
  // with the other one whatever their number (a prompt of 2048 tokens, 16 heads:
  // 246 us, where rows in one group take 68).
  const int few = cache->head_dim == cache->group ? kFewRows : 0x7fffffff;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KvJoin few_parts{}, many_parts{};
  tlq_status ls = launch_kv4_decode(a, few, workspace, &few_parts, s);
  if (ls == TLQ_OK && (long long)max_q * (q_heads / a.cache.heads) > few)
    ls = launch_kv4_prefill(a, few, static_cast<uint8_t*>(workspace) + kv4_decode_workspace(cache->head_dim),
                            &many_parts, s);
  return ls == TLQ_OK ? launch_kv4_join(a, few_parts, many_parts, s) : ls;
}

tlq_status tl_lora_add(const uint16_t* x, int64_t ldx, const uint16_t* A, const uint16_t* B, const float* scales,
                       const int32_t* q_start, const int32_t* adapters, int requests, int tokens, int max_q, int K,
                       int N, int rank, int num_adapters, const uint16_t* y, int64_t ldy, uint16_t* out, int64_t ldo,
                       void* stream) {
  clear_error();
  const char* who = "tl_lora_add";
  if (requests < 0 || tokens < 0 || max_q < 0)
    return set_error(TLQ_EINVAL, "%s: requests=%d tokens=%d max_q=%d", who, requests, tokens, max_q);
  if (K < 8 || K % 8) return set_error(TLQ_EINVAL, "%s: K=%d (a positive multiple of 8)", who, K);
  if (N < 8 || N % 8) return set_error(TLQ_EINVAL, "%s: N=%d (a positive multiple of 8)", who, N);
  if (rank < 8 || rank % 8) return set_error(TLQ_EINVAL, "%s: rank=%d (a positive multiple of 8)", who, rank);
  if (rank > 64) return set_error(TLQ_EUNSUPPORTED, "%s: rank=%d (at most 64)", who, rank);
  if (num_adapters < 0) return set_error(TLQ_EINVAL, "%s: num_adapters=%d", who, num_adapters);
  if (requests == 0 || tokens == 0 || max_q == 0) return TLQ_OK;
  if (!x || !q_start || !adapters || !y || !out || (num_adapters > 0 && (!A || !B || !scales)))
    return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (tokens > 1 && (ldx < K || ldx % 8)) return set_error(TLQ_EINVAL, "%s: ldx=%lld", who, (long long)ldx);
  if (tokens > 1 && (ldy < N || ldo < N || ldy % 8 || ldo % 8))
    return set_error(TLQ_EINVAL, "%s: ldy=%lld ldo=%lld (at least N = %d, multiples of 8)", who, (long long)ldy,
                     (long long)ldo, N);
  if (!aligned(x, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(y, 16) || !aligned(out, 16) ||
      !aligned(scales, 4) || !aligned(q_start, 4) || !aligned(adapters, 4))
    return set_error(TLQ_EINVAL, "%s: x, A, B, y and out must be 16-byte aligned", who);
  const size_t xb = span(tokens, ldx, K, 2), yb = span(tokens, ldy, N, 2), ob = span(tokens, ldo, N, 2);
  const size_t ab = 2 * (size_t)num_adapters * rank * K, bb = 2 * (size_t)num_adapters * rank * N;
  if (overlap(out, ob, x, xb) || overlap(out, ob, A, ab) || overlap(out, ob, B, bb) ||
      overlap(out, ob, scales, 4 * (size_t)num_adapters) || overlap(out, ob, q_start, 4 * ((size_t)requests + 1)) ||
      overlap(out, ob, adapters, 4 * (size_t)requests) ||
      (overlap(out, ob, y, yb) && !(out == y && (ldo == ldy || tokens == 1))))
    return set_error(TLQ_EINVAL, "%s: out overlaps an input (out may be exactly y)", who);
  LoraArgs a{};
  a.x = reinterpret_cast<const __half*>(x);
  a.ldx = ldx;
  a.A = reinterpret_cast<const __half*>(A);
  a.B = reinterpret_cast<const __half*>(B);
  a.scales = scales;
  a.q_start = q_start;
  a.adapters = adapters;
  a.requests = requests;
  a.tokens = tokens;
  a.max_q = std::min(max_q, tokens);
  a.K = K;
  a.N = N;
  a.rank = rank;
  a.num_adapters = num_adapters;
  a.y = reinterpret_cast<const __half*>(y);
  a.ldy = ldy;
  a.out = reinterpret_cast<__half*>(out);
  a.ldo = ldo;
  return launch_lora(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
