// Attention of few query rows over the paged 4-bit cache (decode, drafts).
//
//   k = s c + b, v = s' c' + b',  O = softmax(scale q . k) v
//
// Both products run on the codes.  With p_t the softmax weight of token t,
//   q . k_t      = s_t (q . c_t) + b_t sum(q)
//   sum_t p_t v_t = sum_t (p_t s'_t) c'_t + sum_t p_t b'_t
// so scales and minima are folded outside and a code enters the matrix
// instruction as the FP16 subnormal c * 2^-24: one AND per pair of codes, no
// conversion (16 c * 2^-24 for the odd nibbles, paid back by q / 16 and by the
// output rows).  Products and sums are exact in FP32 to its own rounding.
//
// Layout: mma.sync m16n8k16 with the cache on the M side, eight (query, head)
// rows of one key head on the N side (NT = 1 or 2 such tiles):
//   S^T [16 tokens x 8 rows] = K [16 x D] Q^T,  O^T [D x 8] += V^T [D x 16] P^T.
// K fragments are 8-byte reads of a token's row, V fragments pairs of tokens
// interleaved by PRMT, P^T comes from S^T by movmatrix: no tile is transposed
// or dequantized through shared memory.
//
// The running reference m of the softmax is kept per row and group in log2
// units of p * s' (not p), so that no FP16 weight p s' overflows and the
// largest keep all of their bits: they lie below 2^14 and the largest is at
// least 2^6.  m moves only when a weight would pass that.  (One reference for
// both groups of a row takes 76 us for 79 where the scales are alike, four
// contexts of up to 131072 tokens, and loses the weights of the group whose
// scales are the smaller.)  Value codes are centred:
// 8 sum(p s') is kept beside O, by the same kind of instruction so that both
// round alike, and taken off every other stage; minima are b' + 8 s'.  (On
// 131072 tokens uncentred sums are 400 times the result: an error of 4.9e-4
// against 2.9e-4, for 69 against 78 us.)  Sums of p and of p b' are FP32, of the
// weights before their rounding to FP16: where scales differ, the weights of
// the tokens with small ones end in FP16's last bits or below them, while their
// p may be most of the softmax (a zero or constant value row has scale 2^-24).
// Only the share of codes that s' makes small is rounded with them.  Value codes
// are entered as 4 c and 64 c: the instruction aligns a subnormal factor as if
// its leading bit were there, and what it cuts off a product of c alone adds up
// to 2e-6 of the values' spread in every even channel, the same for any length.
//
// Work: a unit is a stage of 128 tokens, 32 to each of a block's four warps.
// All units of the batch (requests x key heads x row blocks x stages) lie on
// one line that the blocks cut into equal spans, so ragged lengths balance
// whatever they are; a block that begins or ends inside an item leaves a
// partial (FP32) in the workspace and a second, small kernel joins an item's
// partials in order (no atomics: repeatable).  A fifth warp streams the stages
// through a ring of bulk copies, one per page (a page and head is one
// contiguous piece), and runs ahead over the ends of items.
//
// Long batches are bound by issue: 290 instructions per 16 tokens and key head,
// all warps' beside the tiles included, on 55 % of the clocks, the ALU pipe 54 %
// busy, DRAM 55 %.  64 requests on up to 8192 tokens, 32 / 8 heads of 128: 80 us,
// 4.0 TB/s; four on up to 131072 with two groups: 79 us, 3.7 TB/s.  Short ones by latency: 500 tokens, 16 heads: 9 us
// with the join, half of it the start of the two launches.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "serve.cuh"

#ifndef TLQ_KV_SHARED_UNIT
#define TLQ_KV_SHARED_UNIT 0  // 1: the forms for a batch with a shared prefix, built by themselves
#endif

namespace tlq {
namespace {

constexpr bool kShared = TLQ_KV_SHARED_UNIT;
// What beginning and ending an item costs, in stages, on the line of work.  With a
// prefix the items are short (a request's own tokens).
constexpr int kItemCost = kShared ? 1 : 0;

constexpr int kStage = 128;  // tokens of a stage
constexpr int kTile = 16;    // tokens of a matrix instruction
constexpr int kTiles = 2;    // tiles of a warp in a stage
constexpr float kHeadroom = 6.0f;   // a new reference puts the largest weight at 2^6
constexpr float kTrigger = 14.0f;   // weights stay at or below 2^14
constexpr uint32_t kEight = 0x00200020u, kEight16 = 0x02000200u;  // two codes of 8 * 4, of 8 * 64
constexpr float kNone = -1e30f;     // the reference of a row that has seen no key (finite: differences stay numbers)

template <int D, int NG, int NT>
struct DCfg {
  static constexpr int WARPS = 4;  // that compute; one more loads
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int CTAS = NT == 1 ? 3 : 2;  // resident per SM
  static constexpr int JOINT = NT * NG == 1 ? 2 : 1;  // tiles whose steps are interleaved (registers)
  static constexpr int DEPTH = 3;         // stages of the ring
  static constexpr int H = D / 64;        // 64-channel halves
  static constexpr int R = 8 * NT;        // rows of an item
  static constexpr int STAGE_BYTES = kStage * (D + 8 * NG);
  static constexpr int RING = DEPTH * STAGE_BYTES;
  static constexpr int OSTRIDE = D + 4;   // floats per row of the merge buffer
  static constexpr int MERGE = WARPS * 8 * OSTRIDE * 4;
  static constexpr int STATS = WARPS * R * (2 + NG) * 4;
  static constexpr int SMEM = RING + MERGE + STATS + DEPTH * 20 + 64;
};

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D = A B
__device__ __forceinline__ void mma_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

struct DecodeParams {
  KvCache cache;
  KvBatch batch;
  const __half* q;
  long long ldq;
  __half* out;
  long long ldo;
  float scale_log2;  // softmax scale * log2(e)
  int window, share;  // share: query heads per key head
  int few_rows;       // requests of more rows are not this kernel's
  FastDiv by_share;
  KvJoin join;
  KvShared shared;
  int q_heads;
};

// Units of one request, the same for each of its items (key head, row block).
struct ItemShape {
  int items, units;
};

template <int R>
__device__ __forceinline__ ItemShape item_shape(const DecodeParams& p, const KvRequest& r) {
  ItemShape s;
  if (r.q_len * p.share > p.few_rows) return ItemShape{0, 1};
  s.items = p.cache.heads * ((r.q_len * p.share + R - 1) / R);
  int span = r.len;
  if (p.window > 0) {
    const int queries = min(r.q_len, (R + p.share - 2) / p.share + 1);  // a row block's queries
    // window + queries - 1 keys, wherever they lie in their stages
    span = (int)min((long long)r.len, (long long)p.window + queries + kStage);
  }
  s.units = max(1, (span + kStage - 1) / kStage) + kItemCost;
  return s;
}

// A block's share of an item: stages [s0, s1) of one request, key head and row block.
struct Segment {
  KvRequest rq;
  int req, head, row0, rows;
  int lo, hi;             // keys that any row sees
  int all_lo, all_hi;     // keys that every row sees
  int s0, s1;             // stages (absolute: token / kStage)
  bool first, last;       // holds the item's first, last unit
  long long item_end;     // unit behind the item
  int units;              // units of the share
};

// Walks a block's span of units; every thread walks by itself.
template <int R>
struct Walk {
  long long u, u_end, req_u;
  int req;

  __device__ __forceinline__ bool next(const DecodeParams& p, Segment* s) {
    while (u < u_end && req < kv_requests<kShared>(p.batch)) {
      const KvRequest rq = kv_request_or_prefix<kShared>(p.batch, p.cache.page, req);
      const ItemShape shape = item_shape<R>(p, rq);
      const long long units = (long long)shape.items * shape.units;
      if (u >= req_u + units) {  // on to the next request (one without queries is passed over)
        req_u += units;
        ++req;
        continue;
      }
      const int item = (int)((u - req_u) / shape.units);
      const int c0 = (int)((u - req_u) - (long long)item * shape.units);
      const int c1 = (int)min((long long)shape.units, c0 + (u_end - u));
      if (kItemCost > 0 && c1 <= kItemCost) {  // the share ends before the item's first stage
        u += c1 - c0;
        continue;
      }
      const int row_blocks = shape.items / p.cache.heads;
      s->rq = rq;
      s->req = req;
      s->head = item / row_blocks;
      s->row0 = (item - s->head * row_blocks) * R;
      s->rows = min(R, rq.q_len * p.share - s->row0);
      const int first_q = divide(s->row0, p.by_share), last_q = divide(s->row0 + s->rows - 1, p.by_share);
      s->hi = max(0, min(rq.len, rq.base + last_q + 1));
      s->lo = p.window > 0 ? max(0, rq.base + first_q - p.window + 1) : 0;
      s->all_hi = min(s->hi, rq.base + first_q + 1);
      s->all_lo = p.window > 0 ? rq.base + last_q - p.window + 1 : 0;
      const int stage = s->lo / kStage;
      s->s0 = stage + max(0, c0 - kItemCost);
      s->s1 = min(stage + c1 - kItemCost, (s->hi + kStage - 1) / kStage);
      s->first = c0 <= kItemCost;
      s->last = c1 == shape.units;
      s->item_end = req_u + (long long)(item + 1) * shape.units;
      s->units = c1 - c0;
      u += c1 - c0;
      return true;
    }
    return false;
  }
};

template <int D, int NG, int NT>
__global__ void __launch_bounds__(DCfg<D, NG, NT>::THREADS, DCfg<D, NG, NT>::CTAS) decode_attention_kernel(
    const DecodeParams p) {
  using C = DCfg<D, NG, NT>;
  constexpr int H = C::H, R = C::R, W = C::WARPS, DEPTH = C::DEPTH;
  extern __shared__ __align__(128) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + C::RING);
  float* stats = reinterpret_cast<float*>(smem + C::RING + C::MERGE);  // [W][R][m, l, beta...]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::RING + C::MERGE + C::STATS);  // [DEPTH]
  uint64_t* empty = full + DEPTH;                                                    // [DEPTH]
  uint32_t* there = reinterpret_cast<uint32_t*>(empty + DEPTH);  // [DEPTH] 16-token tiles whose page exists
  __shared__ UnitSearch<C::THREADS> search;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, qd = lane & 3;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < DEPTH; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], W);
    }
    fence_mbar_init();
  }
  pdl_wait();
  KvJoinHeader* const header = &p.join.headers[blockIdx.x];
  if (!kShared && tid == 0) header->followers = 0;

  auto count = [&](int i) -> long long {
    const ItemShape s = item_shape<R>(p, kv_request_or_prefix<kShared>(p.batch, p.cache.page, i));
    return (long long)s.items * s.units;
  };
  long long own, mine;
  search.count_all(kv_requests<kShared>(p.batch), count, &own, &mine);  // its barriers publish the mbarriers too
  const long long U = search.total;
  const long long n = min((long long)gridDim.x, U);
  if ((long long)blockIdx.x >= n) return;
  Walk<R> walk;
  walk.u = U * blockIdx.x / n;
  walk.u_end = U * (blockIdx.x + 1) / n;
  search.find(kv_requests<kShared>(p.batch), count, walk.u, own, mine);
  walk.req = search.request;
  walk.req_u = search.first;
  if (walk.req < 0) return;  // not reached: u < U
  Segment sg;
  int stage_i = 0;  // stages of this block so far

  // chunk: the tokens of a stage that lie in one page
  const int chunk = min(p.cache.page, kStage), chunk_shift = min(p.cache.page_shift, 7);
  const int chunk_bytes = chunk * (D + 8 * NG);

  if (warp == W) {
    // ---------------- loader ----------------
    const int chunks = kStage >> chunk_shift;
    bool ok = true;
    while (ok && walk.next(p, &sg)) {
      const int* row = kv_table_row<kShared>(p.batch, sg.req);
      const int pages = (sg.hi + p.cache.page - 1) >> p.cache.page_shift;  // pages that hold a visible key
      auto page_of = [&](int s) {  // lane i: the page of chunk i of stage s
        const int at = (int)(((long long)s * kStage + lane * chunk) >> p.cache.page_shift);
        const bool seen = (long long)s * kStage + (lane + 1) * chunk > sg.lo;
        return s < sg.s1 && lane < chunks && at < pages && seen ? __ldg(row + at) : -1;
      };
      int page = page_of(sg.s0);
      for (int s = sg.s0; s < sg.s1; ++s, ++stage_i) {
        const int slot = stage_i % DEPTH;
        const int next = page_of(s + 1);
        if (!mbar_wait_long(&empty[slot], ((stage_i / DEPTH) & 1) ^ 1, 0x302)) {
          ok = false;
          break;
        }
        const bool in = page >= 0 && page < p.cache.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, in);
        uint8_t* dst = smem + slot * C::STAGE_BYTES + lane * chunk_bytes;
        if (lane == 0) {
          // chunk bit -> bits of its 16-token tiles
          uint32_t tiles = 0;
          for (int i = 0; i < chunks; ++i)
            if (mask >> i & 1u) tiles |= ((1u << (chunk / kTile)) - 1u) << (i * (chunk / kTile));
          there[slot] = tiles;
          mbar_arrive_expect_tx(&full[slot], (uint32_t)__popc(mask) * chunk_bytes);
        }
        __syncwarp();
        if (in) {
          const uint8_t* blk =
              p.cache.blocks + ((long long)page * p.cache.heads + sg.head) * (long long)p.cache.block_bytes;
          if (p.cache.page <= kStage) {
            bulk_load(smem_u32(dst), blk, chunk_bytes, &full[slot]);
          } else {
            const int off = (s * kStage) & (p.cache.page - 1), half = p.cache.page * (D / 2);
            const uint32_t d0 = smem_u32(dst);
            bulk_load(d0, blk + off * (D / 2), kStage * (D / 2), &full[slot]);
            bulk_load(d0 + kStage * (D / 2), blk + half + off * (D / 2), kStage * (D / 2), &full[slot]);
            bulk_load(d0 + kStage * D, blk + 2 * half + off * (NG * 4), kStage * NG * 4, &full[slot]);
            bulk_load(d0 + kStage * (D + 4 * NG), blk + 2 * half + (p.cache.page + off) * (NG * 4), kStage * NG * 4,
                      &full[slot]);
          }
        }
        page = next;
      }
    }
    // no copy is under way when the block ends
    for (int i = max(0, stage_i - DEPTH); i < stage_i; ++i)
      if (!mbar_wait_long(&full[i % DEPTH], (i / DEPTH) & 1, 0x303)) break;
    return;
  }

  const int sw = qd & 1, other = sw ? -(D / 2) : D / 2;
  const uint32_t sel_lo = sw ? 0x1054u : 0x5410u, sel_hi = sw ? 0x3276u : 0x7632u;
  // this warp's tiles inside a stage
  uint32_t kofs[kTiles], pofs[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const int tk = (warp * kTiles + i) * kTile;
    const uint32_t base = (tk >> chunk_shift) * chunk_bytes;
    kofs[i] = base + (tk & (chunk - 1)) * (D / 2);
    pofs[i] = base + chunk * D + (tk & (chunk - 1)) * (NG * 4);
  }
  bool ok = true;
  while (walk.next(p, &sg)) {
    const KvRequest rq = sg.rq;
    const int head = sg.head, row0 = sg.row0, rows = sg.rows, base_pos = rq.base;
    // Query fragments: row n = 8 nt + r, channels 64 h + 16 qd .. + 15, scaled
    // by a power of two so that the item's largest value lies in [2^14, 2^15)
    // (exact, and q / 16 for the odd nibbles stays normal, down to 2^-24 of it).
    uint32_t qf[NT][4 * H][2];
    float2 qs[NT][NG];  // scaled sums of this thread's columns (rows 2 qd, 2 qd + 1)
    float f;            // codes' products to logits
    {
      uint4 raw[NT][H][2];
      float sum[NT][H], big = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = 8 * nt + r;
        const bool on = row < rows;
        const int gr = row0 + (on ? row : 0);
        const int t = divide(gr, p.by_share), g = gr - t * p.share;
        const __half* src = p.q + (long long)(rq.q0 + t) * p.ldq + (long long)(head * p.share + g) * D;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            raw[nt][h][j] =
                on ? *reinterpret_cast<const uint4*>(src + 64 * h + 16 * qd + 8 * j) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          sum[nt][h] = 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w[4] = {raw[nt][h][j].x, raw[nt][h][j].y, raw[nt][h][j].z, raw[nt][h][j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
              sum[nt][h] += v.x + v.y;
              big = fmaxf(big, fmaxf(fabsf(v.x), fabsf(v.y)));
            }
          }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) sum[nt][h] += __shfl_xor_sync(0xffffffffu, sum[nt][h], o);
        }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      int e = 0;  // 2^e * big in [2^14, 2^15); 0 where all are zero or one is infinite
      if (big > 0.f && big < 65536.f) e = 14 + 127 - (int)(__float_as_uint(big) >> 23);
      const float up = __uint_as_float((uint32_t)(127 + e) << 23);
      const float up16 = __uint_as_float((uint32_t)(127 + e - 4) << 23);
      f = p.scale_log2 * __uint_as_float((uint32_t)(127 + 24 - e) << 23);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w[4] = {raw[nt][h][j].x, raw[nt][h][j].y, raw[nt][h][j].z, raw[nt][h][j].w};
            // pairs (ch 0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16 of the code word
            float2 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
            const __half2 a0 = __floats2half2_rn(v[0].x * up, v[2].x * up);
            const __half2 a1 = __floats2half2_rn(v[0].y * up16, v[2].y * up16);
            const __half2 a2 = __floats2half2_rn(v[1].x * up, v[3].x * up);
            const __half2 a3 = __floats2half2_rn(v[1].y * up16, v[3].y * up16);
            qf[nt][4 * h + 2 * j][0] = *reinterpret_cast<const uint32_t*>(&a0);
            qf[nt][4 * h + 2 * j][1] = *reinterpret_cast<const uint32_t*>(&a1);
            qf[nt][4 * h + 2 * j + 1][0] = *reinterpret_cast<const uint32_t*>(&a2);
            qf[nt][4 * h + 2 * j + 1][1] = *reinterpret_cast<const uint32_t*>(&a3);
          }
        }
        float s[2][2];  // [column][half]
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int h = 0; h < H; ++h)
            s[c][h] = __shfl_sync(0xffffffffu, sum[nt][h], (2 * qd + c) * 4) * p.scale_log2;
        if constexpr (H == 1) {
          qs[nt][0] = make_float2(s[0][0], s[1][0]);
        } else if constexpr (NG == 1) {
          qs[nt][0] = make_float2(s[0][0] + s[0][1], s[1][0] + s[1][1]);
        } else {
          qs[nt][0] = make_float2(s[0][0], s[1][0]);
          qs[nt][NG - 1] = make_float2(s[0][1], s[1][1]);
        }
      }
    }

    float o[NT][4 * H][4];
    float2 m[NT][NG];            // by column, as are the sums: l under the first group's reference
    float2 l[NT], beta[NT][NG];
    float eight[NT][NG][4];      // 8 sum(p s') since it was last taken off O, in the layout of O's registers
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt] = make_float2(0.f, 0.f);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        m[nt][g] = make_float2(kNone, kNone);
        beta[nt][g] = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) eight[nt][g][k] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4 * H; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nt][j][k] = 0.f;
    }

    auto centre = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 4 * H; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[nt][j][k] -= eight[nt][NG == 1 ? 0 : j / 4][k];
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int k = 0; k < 4; ++k) eight[nt][g][k] = 0.f;
      }
    };
    for (int s = sg.s0; s < sg.s1; ++s, ++stage_i) {
      if ((s & 1) == 0) centre();
      const int slot = stage_i % DEPTH;
      ok = ok && mbar_wait(&full[slot], (stage_i / DEPTH) & 1, 0x301);
      if (!ok) break;
      const int tok0 = s * kStage + warp * (kTiles * kTile);
      const uint32_t tiles = lds32(smem_u32(&there[slot])) >> (warp * kTiles);
      const uint32_t sb = smem_u32(smem) + slot * C::STAGE_BYTES;
      // EDGE: some row does not see some key of the tiles, or a page is missing
      auto work = [&](auto edge_form) __attribute__((always_inline)) {
        constexpr bool EDGE = decltype(edge_form)::value;
        constexpr int JT = C::JOINT;
#pragma unroll
        for (int i0 = 0; i0 < kTiles; i0 += JT) {
          float2 lw[JT][NT][2];  // [token half]: logits of the two columns, in log2 units
          float vlg[JT][2][NG], vrc[JT][2][NG], vmi[JT][2][NG];
#pragma unroll
          for (int i = 0; i < JT; ++i) {
            // S^T = K Q^T on the codes, per group of channels
            float sc[NT][NG][4];
            const uint32_t kb = sb + kofs[i0 + i];
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const uint2 ka = lds64(kb + r * (D / 2) + 32 * h + 8 * qd);
              const uint2 kc = lds64(kb + (r + 8) * (D / 2) + 32 * h + 8 * qd);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t wa = j ? ka.y : ka.x, wc = j ? kc.y : kc.x;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t xa = e ? wa >> 8 : wa, xc = e ? wc >> 8 : wc;
                  const uint32_t a0 = xa & 0x000F000Fu, a1 = xc & 0x000F000Fu;
                  const uint32_t a2 = xa & 0x00F000F0u, a3 = xc & 0x00F000F0u;
                  const int ks = 4 * h + 2 * j + e;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    float(&d)[4] = sc[nt][NG == 1 ? 0 : h];
                    if (NG == 1 ? ks == 0 : ks == 4 * h)
                      mma_16816_first(d, a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
                    else
                      mma_16816(d, a0, a1, a2, a3, qf[nt][ks][0], qf[nt][ks][1]);
                  }
                }
              }
            }
            // parameters of tokens r and r + 8
            const uint32_t kp = sb + pofs[i0 + i], vp = kp + chunk * (NG * 4);
            float ksc[2][NG], kmi[2][NG];
            bool in[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int tk = r + 8 * y, key = tok0 + (i0 + i) * kTile + tk;
              in[y] = !EDGE || (key >= sg.lo && key < sg.hi && (tiles >> (i0 + i) & 1u));  // else no token of ours lies there
#pragma unroll
              for (int g = 0; g < NG; ++g) {
                uint32_t a = lds32(kp + (tk * NG + g) * 4), b = lds32(vp + (tk * NG + g) * 4);
                if (!in[y]) a = b = 0x00003C00u;  // scale 1, minimum 0
                const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
                const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
                ksc[y][g] = fa.x * f;
                kmi[y][g] = fa.y;
                const float vs = fmaxf(fb.x, 5.9604644775390625e-8f);
                vlg[i][y][g] = lg2(vs);
                vrc[i][y][g] = reciprocal(vs);
                vmi[i][y][g] = fmaf(8.0f, fb.x, fb.y);  // of the centred codes
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int y = 0; y < 2; ++y)
              {
                float2 x = mul2(make_float2(kmi[y][0], kmi[y][0]), qs[nt][0]);
                x = fma2(make_float2(sc[nt][0][2 * y], sc[nt][0][2 * y + 1]), make_float2(ksc[y][0], ksc[y][0]), x);
                if constexpr (NG == 2) {
                  x = fma2(make_float2(kmi[y][1], kmi[y][1]), qs[nt][1], x);
                  x = fma2(make_float2(sc[nt][1][2 * y], sc[nt][1][2 * y + 1]), make_float2(ksc[y][1], ksc[y][1]), x);
                }
                if constexpr (EDGE) {
                  const int key = tok0 + (i0 + i) * kTile + r + 8 * y;
#pragma unroll
                  for (int c = 0; c < 2; ++c) {
                    const int at = base_pos + divide(row0 + min(8 * nt + 2 * qd + c, rows - 1), p.by_share);  // the row's position
                    const bool see = in[y] && key <= at && (p.window <= 0 || key > at - p.window);
                    if (!see) (c ? x.y : x.x) = -INFINITY;
                  }
                }
                lw[i][nt][y] = x;
              }
          }
          // exponents of the weights p s', under the rows' references
          float2 ew[JT][NT][2][NG];
          auto exponents = [&]() __attribute__((always_inline)) {
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < JT; ++i)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                  for (int g = 0; g < NG; ++g) {
                    const float2 less =
                        add2(make_float2(vlg[i][y][g], vlg[i][y][g]), make_float2(-m[nt][g].x, -m[nt][g].y));
                    ew[i][nt][y][g] = add2(lw[i][nt][y], less);
                    top = fmaxf(top, fmaxf(ew[i][nt][y][g].x, ew[i][nt][y][g].y));
                  }
            return top;
          };
          if (__any_sync(0xffffffffu, exponents() > kTrigger)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  float x = -INFINITY;
#pragma unroll
                  for (int i = 0; i < JT; ++i)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                      x = fmaxf(x, (c ? lw[i][nt][y].y : lw[i][nt][y].x) + vlg[i][y][g]);
                  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                  float& ref = c ? m[nt][g].y : m[nt][g].x;
                  const float next = fmaxf(ref, x - kHeadroom);
                  if (next > ref) {
                    const float w = ex2(ref - next);  // 0 for the first reference
                    ref = next;
                    if (g == 0) (c ? l[nt].y : l[nt].x) *= w;
                    (c ? beta[nt][g].y : beta[nt][g].x) *= w;
                    eight[nt][g][c] *= w;
                    eight[nt][g][2 + c] *= w;
#pragma unroll
                    for (int j = 4 * H / NG * g; j < 4 * H / NG * (g + 1); ++j) {
                      o[nt][j][c] *= w;
                      o[nt][j][2 + c] *= w;
                    }
                  }
                }
            exponents();
          }

#pragma unroll
          for (int i = 0; i < JT; ++i) {
            // weights p s' as FP16, their sums, and P^T fragments
            uint32_t pf[NT][NG][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                  const float2 e = make_float2(ex2(ew[i][nt][y][g].x), ex2(ew[i][nt][y][g].y));
                  const __half2 h2 = __floats2half2_rn(e.x, e.y);
                  const float2 w = mul2(e, make_float2(vrc[i][y][g], vrc[i][y][g]));  // p, before any rounding to FP16
                  if (g == 0) l[nt] = add2(l[nt], w);
                  if constexpr (EDGE) {  // a minimum that a row does not see is left out, whatever it holds
                    if (w.x != 0.f) beta[nt][g].x = fmaf(w.x, vmi[i][y][g], beta[nt][g].x);
                    if (w.y != 0.f) beta[nt][g].y = fmaf(w.y, vmi[i][y][g], beta[nt][g].y);
                  } else {
                    beta[nt][g] = fma2(w, make_float2(vmi[i][y][g], vmi[i][y][g]), beta[nt][g]);
                  }
                  pf[nt][g][y] = movmatrix(*reinterpret_cast<const uint32_t*>(&h2));
                }

#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int g = 0; g < NG; ++g)
                mma_16816(eight[nt][g], kEight, kEight16, kEight, kEight16, pf[nt][g][0], pf[nt][g][1]);

            // O^T += V^T P^T: word 8 h + r of tokens 2 qd, 2 qd + 1, + 8, + 9.
            // Odd lanes of a quad read their two tokens in the other order
            // (banks), the byte selectors put them back.
            const uint32_t vb = sb + kofs[i0 + i] + chunk * (D / 2) + 4 * r + (2 * qd + sw) * (D / 2);
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const uint32_t t0 = lds32(vb + 32 * h), t1 = lds32(vb + 32 * h + other);
              const uint32_t t8 = lds32(vb + 32 * h + 8 * (D / 2)), t9 = lds32(vb + 32 * h + 8 * (D / 2) + other);
              const uint32_t wl[2] = {prmt(t0, t1, sel_lo), prmt(t0, t1, sel_hi)};
              const uint32_t wh[2] = {prmt(t8, t9, sel_lo), prmt(t8, t9, sel_hi)};
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t xa = e ? wl[j] >> 6 : wl[j] << 2, xc = e ? wh[j] >> 6 : wh[j] << 2;
                  const uint32_t a0 = xa & 0x003C003Cu, a1 = xa & 0x03C003C0u;  // channels 4 j + 2 e, + 1 of the word
                  const uint32_t a2 = xc & 0x003C003Cu, a3 = xc & 0x03C003C0u;
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
                    mma_16816(o[nt][4 * h + 2 * j + e], a0, a1, a2, a3, pf[nt][NG == 1 ? 0 : h][0],
                              pf[nt][NG == 1 ? 0 : h][1]);
                }
            }
          }
        }
      };
      const uint32_t both = (1u << kTiles) - 1u;
      if (tok0 >= sg.all_lo && tok0 + kTiles * kTile <= sg.all_hi && (tiles & both) == both)
        work(std::false_type{});
      else if (tok0 < sg.hi && tok0 + kTiles * kTile > sg.lo && (tiles & both))
        work(std::true_type{});
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
    }

    // ---------------- join the warps ----------------
    centre();
    // The second group's sums go over to the first one's reference.  The two lie
    // within 60 of each other (scales 2^-24 .. 2^13 and the play of the references).
    if constexpr (NG == 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float w = ex2(c ? m[nt][1].y - m[nt][0].y : m[nt][1].x - m[nt][0].x);
          (c ? beta[nt][1].y : beta[nt][1].x) *= w;
#pragma unroll
          for (int j = 2 * H; j < 4 * H; ++j) {
            o[nt][j][c] *= w;
            o[nt][j][2 + c] *= w;
          }
        }
    }
    named_barrier(1, 32 * W);  // the merge buffer and statistics of the last item have been read
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float lc = c ? l[nt].y : l[nt].x, bc[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) bc[g] = c ? beta[nt][g].y : beta[nt][g].x;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          lc += __shfl_xor_sync(0xffffffffu, lc, x);
#pragma unroll
          for (int g = 0; g < NG; ++g) bc[g] += __shfl_xor_sync(0xffffffffu, bc[g], x);
        }
        if (r == 0) {
          float* st = stats + (warp * R + 8 * nt + 2 * qd + c) * (2 + NG);
          st[0] = c ? m[nt][0].y : m[nt][0].x;
          st[1] = lc;
#pragma unroll
          for (int g = 0; g < NG; ++g) st[2 + g] = bc[g];
        }
      }
    const bool whole = sg.first && sg.last;
    // the block that holds the item's last unit
    int end_block = 0;
    if (!whole && sg.first && (kShared || tid == 0)) {
      const long long last_u = sg.item_end - 1;
      long long b = ((last_u + 1) * n - 1) / U;
      while (U * b / n > last_u) --b;
      while (U * (b + 1) / n <= last_u) ++b;
      end_block = (int)b;
    }
    const KvRowSums& sums = sg.req < p.batch.requests ? p.shared.own : p.shared.prefix;
    auto sums_row = [&](int row) -> size_t {
      const int gr = row0 + row, t = divide(gr, p.by_share), g = gr - t * p.share;
      return (size_t)(rq.q0 + t) * p.q_heads + head * p.share + g;
    };
    float* part = nullptr;
    if (!whole)
      part = p.join.parts + ((size_t)blockIdx.x * 2 + (sg.first ? 1 : 0)) * (R * (D + 2));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt > 0) named_barrier(1, 32 * W);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* dst = merge + (warp * 8 + 2 * qd + c) * C::OSTRIDE + 8 * r;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float k22 = 4194304.0f, k18 = 262144.0f;
            *reinterpret_cast<float4*>(dst + 64 * h + 4 * j) =
                make_float4(o[nt][4 * h + 2 * j][c] * k22, o[nt][4 * h + 2 * j][2 + c] * k18,
                            o[nt][4 * h + 2 * j + 1][c] * k22, o[nt][4 * h + 2 * j + 1][2 + c] * k18);
          }
      }
      named_barrier(1, 32 * W);
      for (int e = tid; e < 8 * (D / 4); e += 32 * W) {
        const int row8 = e / (D / 4), ch = (e - row8 * (D / 4)) * 4;
        const int row = 8 * nt + row8;
        float mm = kNone;
#pragma unroll
        for (int w = 0; w < W; ++w) mm = fmaxf(mm, stats[(w * R + row) * (2 + NG)]);
        float ll = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float* st = stats + (w * R + row) * (2 + NG);
          const float wm = ex2(st[0] - mm);
          ll = fmaf(wm, st[1], ll);
          const float bt = st[2 + (NG == 2 ? ch / 64 : 0)];
          const float4 v = *reinterpret_cast<const float4*>(merge + (w * 8 + row8) * C::OSTRIDE + ch);
          acc[0] = fmaf(wm, v.x + bt, acc[0]);
          acc[1] = fmaf(wm, v.y + bt, acc[1]);
          acc[2] = fmaf(wm, v.z + bt, acc[2]);
          acc[3] = fmaf(wm, v.w + bt, acc[3]);
        }
        if (kShared && whole) {
          if (row < rows) {
            const size_t at = sums_row(row);
            *reinterpret_cast<float4*>(sums.o + at * D + ch) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (ch == 0) sums.ml[at] = make_float2(mm, ll);
          }
        } else if (whole) {
          if (row < rows) {
            const float inv = ll == 0.f ? 0.f : 1.0f / ll;  // no key seen: zeros
            const int gr = row0 + row, t = divide(gr, p.by_share), g = gr - t * p.share;
            const __half2 a = __floats2half2_rn(acc[0] * inv, acc[1] * inv);
            const __half2 b = __floats2half2_rn(acc[2] * inv, acc[3] * inv);
            *reinterpret_cast<uint2*>(p.out + (long long)(rq.q0 + t) * p.ldo +
                                      (long long)(head * p.share + g) * D + ch) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
          }
        } else {
          *reinterpret_cast<float4*>(part + row * D + ch) = make_float4(acc[0], acc[1], acc[2], acc[3]);
          if (ch == 0) {
            part[R * D + row] = mm;
            part[R * D + R + row] = ll;
            if (kShared && sg.first && row < rows) sums.ml[sums_row(row)] = kv_row_in_parts(blockIdx.x, end_block - blockIdx.x);
          }
        }
      }
    }
    if (!kShared && !whole && sg.first && tid == 0)
      *header = KvJoinHeader{(int)(end_block - blockIdx.x), rq.q0, row0, rows, head};
  }
}

template <int D, int NG, int NT>
tlq_status launch_one(const DecodeParams& base, void* ws, KvJoin* join, cudaStream_t stream) {
  using C = DCfg<D, NG, NT>;
  auto kernel = decode_attention_kernel<D, NG, NT>;
  const cudaError_t attr = opt_in_smem<decode_attention_kernel<D, NG, NT>>(C::SMEM);
  if (attr != cudaSuccess) return cuda_error(attr, "kv4 attention: shared memory");
  const int blocks = device_info().sms * C::CTAS;
  DecodeParams p = base;
  p.join = *join = kv_join_at(ws, blocks, C::R);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)blocks, 1, 1);
  lc.blockDim = dim3(C::THREADS, 1, 1);
  lc.dynamicSmemBytes = C::SMEM;
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  return cuda_error(cudaLaunchKernelEx(&lc, kernel, p), "kv4 attention: launch");
}

template <int D, int NG>
tlq_status launch_rows(const DecodeParams& p, int rows, void* ws, KvJoin* join, cudaStream_t stream) {
  return rows <= 8 ? launch_one<D, NG, 1>(p, ws, join, stream) : launch_one<D, NG, 2>(p, ws, join, stream);
}

}  // namespace

#if !TLQ_KV_SHARED_UNIT
// The most that any form of the kernel takes at this head size, so that one
// workspace serves steps of every shape.
size_t kv4_decode_workspace(int head_dim) {
  const int sms = device_info().sms;
  return std::max(kv_join_bytes(3 * sms, 8, head_dim), kv_join_bytes(2 * sms, 16, head_dim));
}
#endif

#if TLQ_KV_SHARED_UNIT
tlq_status launch_kv4_decode_shared(
#else
tlq_status launch_kv4_decode(
#endif
    const KvAttention& a, int few_rows, void* ws, KvJoin* join, cudaStream_t stream) {
  DecodeParams p{};
  p.cache = a.cache;
  p.batch = a.batch;
  p.q = a.q;
  p.ldq = a.ldq;
  p.out = a.out;
  p.ldo = a.ldo;
  p.scale_log2 = (float)((double)a.scale * M_LOG2E);
  p.window = a.window;
  p.share = a.q_heads / a.cache.heads;
  p.few_rows = few_rows;
  p.by_share = fast_div((uint32_t)p.share);
  p.shared = a.shared;
  p.q_heads = a.q_heads;
  // Items of 8 or 16 rows by a request's own rows; a prefix's many are cut into the
  // same (128 behind a prefix of 2048 beside own tokens of 150, 32 / 8 heads: 21 us in
  // eights, 25 in sixteens, of which single tokens fill a quarter).
  const int rows = (int)std::min<long long>((long long)a.batch.max_q * p.share, few_rows);
  if (a.head_dim == 64) return launch_rows<64, 1>(p, rows, ws, join, stream);
  return a.cache.group == 64 ? launch_rows<128, 2>(p, rows, ws, join, stream)
                             : launch_rows<128, 1>(p, rows, ws, join, stream);
}

}  // namespace tlq
