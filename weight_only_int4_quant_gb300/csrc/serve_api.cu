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

// The checks that both attention calls share; *a is filled in where there is
// something to do (requests, tokens and max_q above 0).
struct AttentionCall {
  const char* who;
  const tl_kv4_cache* cache;
  const uint16_t* q;
  int64_t ldq;
  int q_heads;
  uint16_t* out;
  int64_t ldo;
  const int32_t *q_start, *seq_lens, *table;
  int ld_table, requests, tokens, max_q;
  float scale;
  int window;
  bool shared;  // of a batch with a prefix:
  const int32_t *prefix_len, *prefix_table;
  int prefix_pages;
  void* workspace;
  size_t workspace_bytes;
};

// bytes of workspace: the kernels' parts, and behind them the sums of all rows of a batch with a prefix
size_t attention_workspace(int head_dim) { return kv4_decode_workspace(head_dim) + kv4_prefill_workspace(head_dim); }
size_t prefix_workspace(int q_heads, int head_dim, long long tokens) {
  const size_t sums = (kv_row_sums_bytes(tokens * q_heads, head_dim) + 255) & ~size_t(255);
  return ((attention_workspace(head_dim) + 255) & ~size_t(255)) + 2 * sums;
}

tlq_status check_attention(const AttentionCall& c, KvAttention* a, bool* empty) {
  const char* who = c.who;
  *empty = true;
  const tlq_status st = check_cache(c.cache, &a->cache, who);
  if (st != TLQ_OK) return st;
  if (c.q_heads < 1 || c.q_heads % a->cache.heads)
    return set_error(TLQ_EINVAL, "%s: q_heads=%d is not a positive multiple of the cache's heads=%d", who, c.q_heads,
                     a->cache.heads);
  if (c.requests < 0 || c.tokens < 0 || c.max_q < 0)
    return set_error(TLQ_EINVAL, "%s: requests=%d tokens=%d max_q=%d", who, c.requests, c.tokens, c.max_q);
  if (c.window < 0) return set_error(TLQ_EINVAL, "%s: window=%d (0: none)", who, c.window);
  if (c.shared && c.prefix_pages < 0) return set_error(TLQ_EINVAL, "%s: prefix_pages=%d", who, c.prefix_pages);
  if (!std::isfinite(c.scale)) return set_error(TLQ_EINVAL, "%s: scale is not finite", who);
  if (c.requests == 0 || c.tokens == 0 || c.max_q == 0) return TLQ_OK;
  if (!c.q || !c.out || !c.q_start || !c.seq_lens || !c.table ||
      (c.shared && (!c.prefix_len || (c.prefix_pages > 0 && !c.prefix_table))))
    return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (c.ld_table < 1) return set_error(TLQ_EINVAL, "%s: ld_table=%d (must be >= 1)", who, c.ld_table);
  const int head_dim = c.cache->head_dim;
  const long long row = (long long)c.q_heads * head_dim;
  if (c.tokens > 1 && (c.ldq < row || c.ldo < row || c.ldq % 8 || c.ldo % 8))
    return set_error(TLQ_EINVAL, "%s: ldq=%lld ldo=%lld (at least q_heads*head_dim = %lld, multiples of 8)", who,
                     (long long)c.ldq, (long long)c.ldo, row);
  if (!aligned(c.q, 16) || !aligned(c.out, 16) || !aligned(c.workspace, 16) || !aligned(c.q_start, 4) ||
      !aligned(c.seq_lens, 4) || !aligned(c.table, 4) || !aligned(c.prefix_len, 4) || !aligned(c.prefix_table, 4))
    return set_error(TLQ_EINVAL, "%s: q, out and the workspace must be 16-byte aligned", who);
  const int max_q = std::min(c.max_q, c.tokens), share = c.q_heads / a->cache.heads;
  if ((long long)max_q * share > 0x3fffffff)
    return set_error(TLQ_EUNSUPPORTED, "%s: max_q=%d x %d query heads to a key head (at most 2^30 rows)", who, max_q,
                     share);
  if (c.shared && ((long long)c.tokens * share > 0x3fffffff || c.requests == 0x7fffffff))
    return set_error(TLQ_EUNSUPPORTED, "%s: tokens=%d x %d query heads to a key head, requests=%d (at most 2^30 rows)",
                     who, c.tokens, share, c.requests);
  const size_t need = c.shared ? prefix_workspace(c.q_heads, head_dim, c.tokens) : attention_workspace(head_dim);
  if (!c.workspace || c.workspace_bytes < need)
    return set_error(TLQ_EINVAL, "%s: workspace of %zu bytes (%zu needed)", who,
                     c.workspace ? c.workspace_bytes : size_t(0), need);
  const size_t qb = span(c.tokens, c.ldq, row, 2), ob = span(c.tokens, c.ldo, row, 2), cb = cache_bytes(a->cache);
  if (overlap(c.out, ob, c.q, qb) || overlap(c.out, ob, a->cache.blocks, cb) || overlap(c.workspace, need, c.q, qb) ||
      overlap(c.workspace, need, c.out, ob) || overlap(c.workspace, need, a->cache.blocks, cb))
    return set_error(TLQ_EINVAL, "%s: out or the workspace overlaps another buffer", who);
  const struct {
    const void* p;
    size_t n;
  } lengths[5] = {{c.q_start, 4 * ((size_t)c.requests + 1)}, {c.seq_lens, 4 * (size_t)c.requests},
                  {c.table, 4 * (size_t)c.requests * c.ld_table}, {c.prefix_len, c.shared ? size_t(4) : 0},
                  {c.prefix_table, c.shared ? 4 * (size_t)c.prefix_pages : 0}};
  for (const auto& l : lengths)
    if (overlap(c.out, ob, l.p, l.n) || overlap(c.workspace, need, l.p, l.n))
      return set_error(TLQ_EINVAL, "%s: out or the workspace overlaps the batch's arrays", who);
  a->batch = KvBatch{c.q_start, c.seq_lens, c.table, c.ld_table, c.requests, c.tokens, max_q,
                     c.prefix_len, c.prefix_table, c.prefix_pages};
  a->head_dim = head_dim;
  a->q_heads = c.q_heads;
  a->q = reinterpret_cast<const __half*>(c.q);
  a->ldq = c.ldq;
  a->out = reinterpret_cast<__half*>(c.out);
  a->ldo = c.ldo;
  a->scale = c.scale;
  a->window = c.window >= kMaxContext ? 0 : c.window;  // a window that no context outgrows is none
  *empty = false;
  return TLQ_OK;
}

// The tensor-core kernel takes one scale a row, so rows in two groups stay
// with the other one whatever their number (a prompt of 2048 tokens, 16 heads:
// 246 us, where rows in one group take 68).
int few_rows_of(const tl_kv4_cache& c) { return c.head_dim == c.group ? kFewRows : 0x7fffffff; }

// Whether the few-rows kernel takes a batch with a prefix alone, whatever its rows.
// By the tables' capacity, since lengths are known on the GPU only.  What 300
// measured batches come to, in us: a stage of 128 tokens takes the few-rows kernel
// 0.0037 for 8 rows of a key head of 128 and 0.0026 of 64, half as much again and
// more in prompts (whose items are short, and count two stages more); the other
// kernel 0.022 and 0.016 for 256 rows, and 17 and 15 for its launch, its search and
// its first stage.  Key and query heads of 128, 64 tokens: 8 and 32 behind 256 19 us
// for 35, behind 2048 34 for 39, behind 8190 78 for 47; 1 and 4 behind 8190 20 for 36.
// A prompt of 100 tokens, 8 and 32 heads: behind 16 18 for 23, behind 2048 46 for 33.
bool few_rows_alone(const KvAttention& a) {
  if (a.head_dim != a.cache.group) return true;  // as in few_rows_of()
  auto stages_of = [&](int pages) { return ((long long)pages * a.cache.page + 127) / 128; };
  const long long share = a.q_heads / a.cache.heads, rows = a.batch.tokens * share;
  if (rows <= kFewRows) return true;
  const bool prompts = a.batch.max_q * share > kFewRows, small = a.head_dim == 64;
  const double prefix = (double)stages_of(a.batch.prefix_pages) * a.cache.heads;
  const double own = prompts ? (double)(stages_of(a.batch.ld_table) + 2) * a.cache.heads : 0.0;
  const double here = (prompts ? (small ? 0.0045 : 0.0065) : (small ? 0.0026 : 0.0037)) * (prefix + own) *
                      (double)((rows + 7) / 8);
  const double there = (small ? 15.0 : 17.0) + (small ? 0.016 : 0.022) * prefix * (double)((rows + 255) / 256);
  return here < there;
}

// Rows that may lie in others' gaps (columns of a fused projection's rows).
struct RowSet {
  const void* p;
  size_t step, bytes;  // from row to row, of a row
};

// Two sets of `rows` rows share bytes.
bool meet(const RowSet& a, const RowSet& b, long long rows) {
  if (!a.bytes || !b.bytes || rows < 1) return false;
  if (!overlap(a.p, (rows - 1) * a.step + a.bytes, b.p, (rows - 1) * b.step + b.bytes)) return false;
  if (rows == 1 || a.step != b.step) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  const size_t d = y >= x ? (y - x) % a.step : (a.step - (x - y) % a.step) % a.step;  // b's rows behind a's
  return d < a.bytes || a.step - d < b.bytes;
}

long long row_values(const RopeRows& r, const RopeArgs& a) { return (long long)r.heads * a.head_dim; }
RowSet rows_in(const RopeRows& r, const RopeArgs& a) {
  return RowSet{r.x, 2 * (size_t)r.ld, 2 * (size_t)row_values(r, a)};
}
RowSet rows_out(const RopeRows& r, const RopeArgs& a) {
  return RowSet{r.out, 2 * (size_t)r.ldo, 2 * (size_t)row_values(r, a)};
}
size_t table_bytes(const RopeTable& t) { return 4 * (size_t)t.positions * t.rot; }
size_t positions_bytes(const RopeArgs& a) { return a.rope.rot ? 4 * (size_t)a.rope.axes * a.tokens : 0; }

// r's output overlaps an input other than its own rows, or those but not exactly.
bool output_meets(const RopeRows& r, const RopeArgs& a) {
  if (!r.heads) return false;
  const RowSet out = rows_out(r, a);
  for (const RopeRows* x : {&a.q, &a.k, &a.v}) {
    if (x->heads && !(x == &r && r.out == r.x && (r.ld == r.ldo || a.tokens == 1)) && meet(out, rows_in(*x, a), a.tokens))
      return true;
    if (x->weight && overlap(r.out, span(a.tokens, r.ldo, row_values(r, a), 2), x->weight, 2 * (size_t)a.head_dim))
      return true;
  }
  const size_t n = span(a.tokens, r.ldo, row_values(r, a), 2);
  return overlap(r.out, n, a.positions, positions_bytes(a)) || overlap(r.out, n, a.rope.table, table_bytes(a.rope)) ||
         overlap(r.out, n, a.slots, a.slots ? 8 * (size_t)a.tokens : 0);
}

tlq_status check_rope(const char* who, const tl_rope* rope, const int32_t* positions, int head_dim, float eps, int tokens,
                      RopeArgs* a) {
  if (tokens < 0) return set_error(TLQ_EINVAL, "%s: tokens=%d", who, tokens);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return set_error(TLQ_EINVAL, "%s: eps=%g (finite, not negative)", who, eps);
  a->who = who;
  a->tokens = tokens;
  a->head_dim = head_dim;
  a->eps = eps;
  if (!rope) return TLQ_OK;
  const int rot = rope->rot_dim;
  if (rot < 16 || rot > head_dim || rot % 16)
    return set_error(TLQ_EINVAL, "%s: rot_dim=%d (a multiple of 16, up to head_dim=%d)", who, rot, head_dim);
  if (rope->num_positions < 1 || rope->num_positions > kMaxContext)
    return set_error(TLQ_EINVAL, "%s: num_positions=%lld (1..2^30)", who, (long long)rope->num_positions);
  if (rope->axes < 1 || rope->axes > 3) return set_error(TLQ_EINVAL, "%s: axes=%d (1..3)", who, rope->axes);
  long long pairs = 0;
  for (int i = 0; i < rope->axes; ++i) {
    if (rope->sections[i] < 0) return set_error(TLQ_EINVAL, "%s: sections[%d]=%d", who, i, rope->sections[i]);
    pairs += rope->sections[i];
  }
  if (pairs != rot / 2)
    return set_error(TLQ_EINVAL, "%s: the sections hold %lld pairs, rot_dim=%d has %d", who, pairs, rot, rot / 2);
  if (tokens > 0 && (!rope->table || !positions)) return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (!aligned(rope->table, 16) || !aligned(positions, 4))
    return set_error(TLQ_EINVAL, "%s: the table must be 16-byte aligned, positions 4-byte", who);
  a->rope = RopeTable{reinterpret_cast<const float2*>(rope->table), (int)rope->num_positions, rot,
                      rope->interleaved != 0, rope->axes, rope->sections[0],
                      rope->axes > 1 ? rope->sections[0] + rope->sections[1] : rot / 2};
  a->positions = positions;
  return TLQ_OK;
}

tlq_status check_heads(const char* who, const char* name, const uint16_t* x, int64_t ld, int heads,
                       const uint16_t* weight, uint16_t* out, int64_t ldo, bool has_out, const RopeArgs& a, RopeRows* r) {
  if (heads < 0 || heads > 4096) return set_error(TLQ_EINVAL, "%s: %s_heads=%d (0..4096)", who, name, heads);
  if (heads == 0 || a.tokens == 0) return TLQ_OK;
  const long long row = (long long)heads * a.head_dim;
  if (!x || (has_out && !out)) return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (a.tokens > 1 && (ld < row || ld % 8 || (has_out && (ldo < row || ldo % 8))))
    return set_error(TLQ_EINVAL, "%s: ld%s=%lld ld%s_out=%lld (at least heads*head_dim = %lld, multiples of 8)", who, name,
                     (long long)ld, name, (long long)ldo, row);
  if (!aligned(x, 16) || !aligned(out, 16) || !aligned(weight, 16))
    return set_error(TLQ_EINVAL, "%s: %s, its output and its weight must be 16-byte aligned", who, name);
  *r = RopeRows{reinterpret_cast<const __half*>(x), ld, reinterpret_cast<__half*>(out), ldo,
                reinterpret_cast<const __half*>(weight), heads};
  return TLQ_OK;
}

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
  return attention_workspace(head_dim);
}

tlq_status tl_kv4_attention(const tl_kv4_cache* cache, const uint16_t* q, int64_t ldq, int q_heads, uint16_t* out,
                            int64_t ldo, const int32_t* q_start, const int32_t* seq_lens, const int32_t* table,
                            int ld_table, int requests, int tokens, int max_q, float scale, int window,
                            void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  KvAttention a{};
  bool empty;
  const tlq_status st = check_attention(
      AttentionCall{"tl_kv4_attention", cache, q, ldq, q_heads, out, ldo, q_start, seq_lens, table, ld_table, requests,
                    tokens, max_q, scale, window, false, nullptr, nullptr, 0, workspace, workspace_bytes},
      &a, &empty);
  if (st != TLQ_OK || empty) return st;
  const int few = few_rows_of(*cache);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KvJoin few_parts{}, many_parts{};
  tlq_status ls = launch_kv4_decode(a, few, workspace, &few_parts, s);
  if (ls == TLQ_OK && (long long)a.batch.max_q * (q_heads / a.cache.heads) > few)
    ls = launch_kv4_prefill(a, few, static_cast<uint8_t*>(workspace) + kv4_decode_workspace(cache->head_dim),
                            &many_parts, s);
  return ls == TLQ_OK ? launch_kv4_join(a, few_parts, many_parts, s) : ls;
}

size_t tl_kv4_attention_prefix_workspace_size(int q_heads, int heads, int head_dim, int tokens, int max_q) {
  clear_error();
  if (q_heads < 1 || heads < 1 || q_heads % heads || (head_dim != 64 && head_dim != 128) || tokens < 0 || max_q < 0)
    return 0;
  return prefix_workspace(q_heads, head_dim, tokens);
}

tlq_status tl_kv4_attention_prefix(const tl_kv4_cache* cache, const uint16_t* q, int64_t ldq, int q_heads,
                                   uint16_t* out, int64_t ldo, const int32_t* q_start, const int32_t* seq_lens,
                                   const int32_t* table, int ld_table, const int32_t* prefix_len,
                                   const int32_t* prefix_table, int prefix_pages, int requests, int tokens, int max_q,
                                   float scale, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  KvAttention a{};
  bool empty;
  const tlq_status st = check_attention(
      AttentionCall{"tl_kv4_attention_prefix", cache, q, ldq, q_heads, out, ldo, q_start, seq_lens, table, ld_table,
                    requests, tokens, max_q, scale, 0, true, prefix_len, prefix_table, prefix_pages, workspace,
                    workspace_bytes},
      &a, &empty);
  if (st != TLQ_OK || empty) return st;
  const int d = cache->head_dim, few = few_rows_alone(a) ? 0x7fffffff : kFewRows;
  const long long rows = (long long)tokens * q_heads;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  uint8_t* sums = at + ((attention_workspace(d) + 255) & ~size_t(255));
  const size_t each = (kv_row_sums_bytes(rows, d) + 255) & ~size_t(255);
  for (KvRowSums* r : {&a.shared.own, &a.shared.prefix}) {
    r->o = reinterpret_cast<float*>(sums);
    r->ml = reinterpret_cast<float2*>(r->o + rows * d);
    sums += each;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  KvJoin few_parts{}, many_parts{};
  tlq_status ls = launch_kv4_decode_shared(a, few, at, &few_parts, s);
  if (ls == TLQ_OK && (long long)tokens * (q_heads / a.cache.heads) > few)
    ls = launch_kv4_prefill_shared(a, few, at + kv4_decode_workspace(d), &many_parts, s);
  return ls == TLQ_OK ? launch_kv4_finish_shared(a, few, few_parts, many_parts, s) : ls;
}

tlq_status tl_rope_table(const double* inv_freq, int64_t num_positions, int rot_dim, double scale, float* table,
                         void* stream) {
  clear_error();
  const char* who = "tl_rope_table";
  if (rot_dim < 16 || rot_dim > 256 || rot_dim % 16)
    return set_error(TLQ_EINVAL, "%s: rot_dim=%d (a multiple of 16, 16..256)", who, rot_dim);
  if (num_positions < 1 || num_positions > kMaxContext)
    return set_error(TLQ_EINVAL, "%s: num_positions=%lld (1..2^30)", who, (long long)num_positions);
  if (!std::isfinite(scale)) return set_error(TLQ_EINVAL, "%s: scale is not finite", who);
  if (!inv_freq || !table) return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (!aligned(table, 16) || !aligned(inv_freq, 8))
    return set_error(TLQ_EINVAL, "%s: table must be 16-byte aligned, inv_freq 8-byte", who);
  if (overlap(table, 4 * (size_t)num_positions * rot_dim, inv_freq, 4 * (size_t)rot_dim))
    return set_error(TLQ_EINVAL, "%s: table overlaps inv_freq", who);
  return launch_rope_table(inv_freq, table, num_positions, rot_dim / 2, scale, static_cast<cudaStream_t>(stream));
}

tlq_status tl_qk_norm_rope(const tl_rope* rope, const int32_t* positions, const uint16_t* q, int64_t ldq, int q_heads,
                           const uint16_t* q_weight, uint16_t* q_out, int64_t ldqo, const uint16_t* k, int64_t ldk,
                           int k_heads, const uint16_t* k_weight, uint16_t* k_out, int64_t ldko, int head_dim,
                           float eps, int tokens, void* stream) {
  clear_error();
  const char* who = "tl_qk_norm_rope";
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return set_error(head_dim > 0 ? TLQ_EUNSUPPORTED : TLQ_EINVAL, "%s: head_dim=%d (64, 128 or 256)", who, head_dim);
  RopeArgs a{};
  tlq_status st = check_rope(who, rope, positions, head_dim, eps, tokens, &a);
  if (st == TLQ_OK) st = check_heads(who, "q", q, ldq, q_heads, q_weight, q_out, ldqo, true, a, &a.q);
  if (st == TLQ_OK) st = check_heads(who, "k", k, ldk, k_heads, k_weight, k_out, ldko, true, a, &a.k);
  if (st != TLQ_OK || tokens == 0 || q_heads + k_heads == 0) return st;
  if (output_meets(a.q, a) || output_meets(a.k, a) || meet(rows_out(a.q, a), rows_out(a.k, a), tokens))
    return set_error(TLQ_EINVAL, "%s: an output overlaps an input or the other output (it may be exactly its input)", who);
  return launch_rope(a, static_cast<cudaStream_t>(stream));
}

tlq_status tl_kv4_append_rope(const tl_kv4_cache* cache, const tl_rope* rope, const int32_t* positions,
                              const uint16_t* k, int64_t ldk, const uint16_t* k_weight, const uint16_t* v, int64_t ldv,
                              const int64_t* slots, const uint16_t* q, int64_t ldq, int q_heads,
                              const uint16_t* q_weight, uint16_t* q_out, int64_t ldqo, float eps, int tokens,
                              void* stream) {
  clear_error();
  const char* who = "tl_kv4_append_rope";
  RopeArgs a{};
  tlq_status st = check_cache(cache, &a.cache, who);
  if (st == TLQ_OK) st = check_rope(who, rope, positions, cache->head_dim, eps, tokens, &a);
  if (st == TLQ_OK) st = check_heads(who, "q", q, ldq, q_heads, q_weight, q_out, ldqo, true, a, &a.q);
  if (st == TLQ_OK) st = check_heads(who, "k", k, ldk, a.cache.heads, k_weight, nullptr, 0, false, a, &a.k);
  if (st == TLQ_OK) st = check_heads(who, "v", v, ldv, a.cache.heads, nullptr, nullptr, 0, false, a, &a.v);
  if (st != TLQ_OK || tokens == 0) return st;
  if (!slots) return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (!aligned(slots, 8)) return set_error(TLQ_EINVAL, "%s: slots must be 8-byte aligned", who);
  a.slots = reinterpret_cast<const long long*>(slots);
  if (output_meets(a.q, a)) return set_error(TLQ_EINVAL, "%s: q_out overlaps an input (it may be exactly q)", who);
  const size_t cb = cache_bytes(a.cache);
  bool in_cache = overlap(a.cache.blocks, cb, slots, 8 * (size_t)tokens);
  for (const RopeRows* r : {&a.q, &a.k, &a.v}) {
    in_cache |= overlap(a.cache.blocks, cb, r->x, span(r->heads ? tokens : 0, r->ld, row_values(*r, a), 2));
    in_cache |= overlap(a.cache.blocks, cb, r->weight, r->weight ? 2 * (size_t)a.head_dim : 0);
  }
  in_cache |= overlap(a.cache.blocks, cb, a.q.out, span(a.q.heads ? tokens : 0, a.q.ldo, row_values(a.q, a), 2));
  in_cache |= overlap(a.cache.blocks, cb, a.positions, positions_bytes(a)) ||
              overlap(a.cache.blocks, cb, a.rope.table, table_bytes(a.rope));
  if (in_cache) return set_error(TLQ_EINVAL, "%s: the cache overlaps another buffer", who);
  return launch_rope(a, static_cast<cudaStream_t>(stream));
}

tlq_status tl_sample(const void* logits, int fp16, int64_t ld, int rows, int vocab, const float* uniform,
                     const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                     int32_t* tokens, float* logprobs, void* stream) {
  clear_error();
  const char* who = "tl_sample";
  if (rows < 0) return set_error(TLQ_EINVAL, "%s: rows=%d", who, rows);
  if (vocab < 1) return set_error(TLQ_EINVAL, "%s: vocab=%d (must be >= 1)", who, vocab);
  if (vocab > kMaxVocab) return set_error(TLQ_EUNSUPPORTED, "%s: vocab=%d (at most %d)", who, vocab, kMaxVocab);
  if (rows > 0x0fffffff) return set_error(TLQ_EUNSUPPORTED, "%s: rows=%d (at most 2^28 - 1)", who, rows);
  if (fp16 != 0 && fp16 != 1) return set_error(TLQ_EINVAL, "%s: fp16=%d (1: FP16, 0: FP32)", who, fp16);
  if (rows == 0) return TLQ_OK;
  if (!logits || !uniform || !tokens) return set_error(TLQ_EINVAL, "%s: null pointer", who);
  if (rows > 1 && ld < vocab) return set_error(TLQ_EINVAL, "%s: ld=%lld (at least vocab = %d)", who, (long long)ld, vocab);
  const size_t size = fp16 ? 2 : 4, n = 4 * (size_t)rows;
  if (!aligned(logits, size) || !aligned(uniform, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
      !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4))
    return set_error(TLQ_EINVAL, "%s: arrays must be aligned to their elements", who);
  const void* const in[5] = {uniform, temperature, top_k, top_p, min_p};
  const void* const res[2] = {tokens, logprobs};
  for (const void* o : res) {
    if (!o) continue;
    bool meets = overlap(o, n, logits, span(rows, ld, vocab, size));
    for (const void* i : in) meets |= i && overlap(o, n, i, n);
    if (meets) return set_error(TLQ_EINVAL, "%s: an output overlaps an input", who);
  }
  if (logprobs && overlap(tokens, n, logprobs, n)) return set_error(TLQ_EINVAL, "%s: the outputs overlap", who);
  SampleArgs a{};
  a.logits = logits;
  a.half = fp16 != 0;
  a.ld = ld;
  a.rows = rows;
  a.vocab = vocab;
  a.uniform = uniform;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.tokens = tokens;
  a.logprobs = logprobs;
  return launch_sample(a, static_cast<cudaStream_t>(stream));
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
