// Attention of many query rows over the paged 4-bit cache (prompts, chunks) on
// the 5th-generation tensor cores (tcgen05 + TMEM).
//
//   S = K Q, O = P V on the codes:  with k = s c + b, v = s' c' + b',
//   logit_ij = scale (s_j (q_i . c_j) + b_j sum(q_i)),  p' = p s'_j,
//   o_i = (sum_j p'_ij c'_j + sum_j p_ij b'_j) / sum_j p_ij
// The codes go to the matrix instructions exactly, as the FP16 subnormals
// c * 2^-24 (a mask, and a shift for most, per pair); scales and minima are
// applied in FP32 in the softmax.  The only roundings to FP16 are those of the
// weights p' and of the result.  Value codes enter as c - 8: a weight's rounding
// then meets a factor of about the spread of the values (an uncentred code's
// mean is three times that), with minima b + 8 s beside it in FP32.
//
// A block takes two tiles of 128 (query, head) rows of one key head against
// stages of 128 tokens:
//   warps 0-3, 4-7  softmax of the first, second tile: S from TMEM, weights
//                   back to TMEM over it (FP16, the A operand of P V)
//   warps 8-10      a thread to a row of codes (a token's key or value): from
//                   global memory to registers a stage ahead, then into the K
//                   and V tiles; scales and minima into the softmax's tables
//   warp 11         issues the MMAs
// The two tiles go their own ways through the stages, so that one tile's MMAs
// run while the other's softmax works; the weights of a stage are handed over in
// two halves, the first of which is multiplied during the softmax of the second.
// (An S for each half, to be formed ahead, reads Q twice as often: shared memory,
// 4600 of a stage's 5400 clocks busy, then bounds the stage.)  Twelve warps,
// three to a scheduler, leave the softmax 168 registers a thread.
// Both operands lie in shared memory as the cache has them, a token to a
// 128-byte swizzled row: K-major for S, N-major (transposed by descriptor)
// for P V, so no tile is transposed.  The order of channels inside a code
// word's eight, (0 4 1 5 2 6 3 7), is that of the masks; Q is stored in the
// same order and O's columns are put back at the end.
//
// TMEM is read in the 16x256b form: a thread holds pairs of columns of four
// rows, so the five constants of a token are read from shared memory once for
// four rows.  (With a row to a thread those reads alone, 20 bytes for every
// element, took longer than the MMAs: shared memory gives 128 bytes a clock.)
//
// Work is cut as in the kernel for few rows: all (request, row tile, key head,
// stage) units lie on one line, each of the persistent blocks takes an equal
// span, and partial items are joined by a second kernel in a fixed order.
//
// Long spans are bound by the softmax of a stage (5400 clocks, its MMAs 2000 of
// them): chunks on up to 16384 tokens, 32 / 8 heads of 128, take 870 us, 753
// TFLOP/s.  A prompt of 2048 tokens, 16 heads, takes 68 us, 254 TFLOP/s: about
// 9 us pass before a block's first stage (search, page, codes: dependent loads
// and cold instructions) and 6 us at a change of item.
#include <algorithm>
#include <cmath>

#include "serve.cuh"
#include "tc_common.cuh"

#ifndef TLQ_KV_SHARED_UNIT
#define TLQ_KV_SHARED_UNIT 0  // 1: the forms for a batch with a shared prefix, built by themselves
#endif

namespace tlq {
namespace {

constexpr bool kShared = TLQ_KV_SHARED_UNIT;

constexpr int kStage = 128;       // tokens of a stage
constexpr int kRows = 128;        // rows of a tile
constexpr int kItemRows = 256;    // rows of an item: two tiles
constexpr int kHalf = 64;         // tokens whose weights are handed over at once
constexpr int kItemCost = kShared ? 6 : 2;  // what beginning and ending an item costs, in stages; with a
                                            // prefix short items lie beside long ones (329 us with 6, 332 with 4,
                                            // 342 with 2: 992 queries behind 12001 tokens)
constexpr int kCodeWarps = 3;     // warps that write the K and V tiles
constexpr int kThreads = (8 + kCodeWarps + 1) * 32;
constexpr float kHeadroom = 6.0f;   // a new reference puts the largest weight at 2^6
constexpr float kTrigger = 14.0f;   // weights stay at or below 2^14
constexpr float kNone = -1e30f;

template <int D>
struct PCfg {
  static constexpr int KD = 2, VD = 2, TD = 3;  // stages of keys, values and tables
  static constexpr int BLOCK = kStage * 128;    // 128 rows of 64 channels
  static constexpr int TILE = BLOCK * (D / 64);
  // tables: per pair of tokens (A0 A1 B0 B1), (lg0 lg1 rc0 rc1), (rb0 rb1)
  static constexpr int TABLE = kStage * 20;
  static constexpr int BARS = 8 * 32;
  static constexpr int SMEM = 1024 + 2 * TILE + KD * TILE + VD * TILE + TD * TABLE + BARS;
  static_assert(SMEM <= 232448 - 6144, "shared memory");
};

struct PrefillAttnParams {
  KvCache cache;
  KvBatch batch;
  const __half* q;
  long long ldq;
  __half* out;
  long long ldo;
  float scale_log2;
  int window, share, few_rows;
  FastDiv by_share;
  KvJoin join;
  KvShared shared;
  int q_heads;
};

// Bounds of one row tile of a request.
struct TileShape {
  int lo, hi;  // keys that any row sees
  int s0, n;   // first stage, stages (at least one)
};
__device__ __forceinline__ TileShape tile_shape(const PrefillAttnParams& p, const KvRequest& r, int rows, int qt) {
  TileShape t;
  const int first_q = divide(qt * kItemRows, p.by_share);
  const int last_q = divide(min(rows, (qt + 1) * kItemRows) - 1, p.by_share);
  t.hi = max(0, min(r.len, r.base + last_q + 1));
  t.lo = p.window > 0 ? max(0, r.base + first_q - p.window + 1) : 0;
  t.s0 = t.lo / kStage;
  t.n = max(1, (t.hi + kStage - 1) / kStage - t.s0);
  return t;
}
// rows of a request that this kernel takes (0: the kernel for few rows does)
__device__ __forceinline__ int many_rows(const PrefillAttnParams& p, const KvRequest& r) {
  const int rows = r.q_len * p.share;
  return rows > p.few_rows ? rows : 0;
}

// A block's share of an item.  On the line of work an item is kItemCost units
// and then one for each stage.
struct PSegment {
  KvRequest rq;
  int req, head, row0, rows;
  int lo, hi;
  int s0, s1;         // stages of the share (absolute: token / kStage)
  int tile_end[2];    // by tile: behind the last of them that one of its rows sees (s0: none)
  bool first, last;   // holds the item's first, last stage
  long long item_end;
};

struct PWalk {
  long long u, u_end, item_u;  // item_u: first unit of the item at hand
  int req, qt, head;
  int rows, tiles;             // of the request at hand
  KvRequest rq;

  __device__ __forceinline__ void enter(const PrefillAttnParams& p) {
    rq = kv_request_or_prefix<kShared>(p.batch, p.cache.page, req);
    rows = many_rows(p, rq);
    tiles = (rows + kItemRows - 1) / kItemRows;
    qt = head = 0;
  }
  // To the row tile that u lies in; a warp together, 32 row tiles at a time.
  __device__ __forceinline__ void start(const PrefillAttnParams& p, int request, long long first) {
    const int lane = threadIdx.x & 31;
    req = request;
    item_u = first;
    enter(p);
    for (int q0 = 0; q0 < tiles; q0 += 32) {
      const long long n =
          q0 + lane < tiles ? (long long)(tile_shape(p, rq, rows, q0 + lane).n + kItemCost) * p.cache.heads : 0;
      long long upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, n > 0 && u < item_u + upto);
      if (hit) {
        const int f = __ffs(hit) - 1;
        qt = q0 + f;
        item_u += __shfl_sync(0xffffffffu, upto - n, f);
        return;
      }
      item_u += __shfl_sync(0xffffffffu, upto, 31);
    }
    qt = tiles;
  }
  __device__ __forceinline__ bool next(const PrefillAttnParams& p, PSegment* s) {
    while (u < u_end) {
      if (qt >= tiles) {
        if (++req >= kv_requests<kShared>(p.batch)) return false;
        enter(p);
        continue;
      }
      const TileShape t = tile_shape(p, rq, rows, qt);
      const int units = t.n + kItemCost;
      if (u >= item_u + units) {
        long long skip = 1;
        if (u >= item_u + 2 * units) skip = min((long long)(p.cache.heads - head), (u - item_u) / units);
        item_u += skip * units;
        head += (int)skip;
        if (head >= p.cache.heads) {
          head = 0;
          ++qt;
        }
        continue;
      }
      const int c0 = max(0, (int)(u - item_u) - kItemCost);
      const int c1 = (int)min((long long)units, u_end - item_u) - kItemCost;
      const bool begins = u <= item_u + kItemCost;
      u = min(u_end, item_u + units);
      if (c1 <= c0) continue;  // the share ends before the item's first stage
      s->rq = rq;
      s->req = req;
      s->head = head;
      s->row0 = qt * kItemRows;
      s->rows = min(kItemRows, rows - s->row0);
      s->lo = t.lo;
      s->hi = t.hi;
      s->s0 = t.s0 + c0;
      s->s1 = t.s0 + c1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int last = min(s->rows, kRows * (i + 1)) - 1;  // the tile's last row
        const int hi = last < kRows * i ? 0 : rq.base + divide(s->row0 + last, p.by_share) + 1;
        s->tile_end[i] = max(s->s0, min(s->s1, (max(min(hi, t.hi), 0) + kStage - 1) / kStage));
      }
      s->first = begins;
      s->last = c1 == t.n;
      s->item_end = item_u + units;
      return true;
    }
    return false;
  }
};

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

// ---- TMEM in the 16-lane forms.  x4 of 16x256b: 32 columns of 16 rows; thread
// (r, q) = (lane / 4, lane % 4) holds in v[4 k + 0, 1] columns 8 k + 2 q, + 1 of
// row r and in v[4 k + 2, 3] those of row r + 8. ----
__device__ __forceinline__ void tmem_ld_16x256(uint32_t addr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st_16x256(uint32_t addr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"f"(
          v[0]),
      "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
      "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "r"(addr)
      : "memory");
}
// x4 of 16x128b: 16 columns of 16 rows; v[2 k] is column 4 k + q of row r, v[2 k + 1] of row r + 8.
__device__ __forceinline__ void tmem_st_16x128(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(addr)
               : "memory");
}
// The waits name the registers that the loads fill, so that nothing reads them earlier.
__device__ __forceinline__ void tmem_wait_ld(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// N-major operand, SWIZZLE_128B: rows of 64 channels (128 bytes), 8 tokens to
// an atom of 1024 bytes (stride offset), 64-channel blocks BLOCK bytes apart
// (leading offset).
__device__ __forceinline__ uint64_t sw128_desc_n(uint32_t saddr, uint32_t block_bytes) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(block_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::f16, D = F32, A = B = F16, M = 128; bit 16: B is N-major.
constexpr uint32_t kIdescS =
    (1u << 4) | ((uint32_t)(kStage >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
template <int D>
constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);

// The MMAs and commits are executed by a converged warp, of which one elected
// thread issues (the same one every time): the operands stay in uniform
// registers.  Issued from a one-thread branch, each MMA's operands were moved
// there one by one, 2 us for the sixteen of a stage and tile.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

__device__ __forceinline__ void sts_f32(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Barriers of a block.
struct PBars {
  uint64_t q_full[2];              // by tile: Q written (4 warps)
  uint64_t s_full[2];              // by tile: S complete
  uint64_t p_full[2][2];           // by tile and half: the weights written (4 warps)
  uint64_t o_done[2][2];           // by tile and half: P V complete
  uint64_t k_full[2], k_empty[2];  // written (4 warps), read (2 tiles)
  uint64_t v_full[2], v_empty[2];
  uint64_t t_full[3], t_empty[3];  // table written (4 warps), read (8 warps)
  uint32_t tmem;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_attention_kernel(const PrefillAttnParams p) {
  using C = PCfg<D>;
  constexpr int KD = C::KD, VD = C::VD, TD = C::TD;
  // Declared with 16 bytes' alignment, since more is not kept behind the static
  // arrays (and the compiler would take it as given); rounded up to 1024 by hand.
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // still a shared address to the compiler
  uint8_t* const sq = smem;                       // [2][TILE]
  uint8_t* const sk = sq + 2 * C::TILE;           // [KD][TILE]
  uint8_t* const sv = sk + KD * C::TILE;          // [VD][TILE]
  uint8_t* const st = sv + VD * C::TILE;          // [TD][TABLE]
  PBars* const bar = reinterpret_cast<PBars*>(st + TD * C::TABLE);
  static_assert(sizeof(PBars) <= C::BARS, "barriers fit");
  __shared__ UnitSearch<kThreads> search;
  // each warp's place in the block's work: in shared memory, since it is needed
  // once an item and the softmax has no registers to spare
  __shared__ PWalk walks[kThreads / 32];
  __shared__ PSegment segments[kThreads / 32];
  __shared__ long long request_units[kThreads];
  __shared__ uint16_t long_requests[kThreads];  // those that a warp counts together
  __shared__ int long_count;

  const int tid = threadIdx.x, warp = (int)uniform(tid >> 5), lane = tid & 31;
  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->q_full[i], 4);
      mbar_init(&bar->s_full[i], 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(&bar->p_full[i][h], 4);
        mbar_init(&bar->o_done[i][h], 1);
      }
      mbar_init(&bar->k_full[i], 4);
      mbar_init(&bar->k_empty[i], 2);
      mbar_init(&bar->v_full[i], 4);
      mbar_init(&bar->v_empty[i], 2);
    }
    for (int i = 0; i < TD; ++i) {
      mbar_init(&bar->t_full[i], 4);
      mbar_init(&bar->t_empty[i], 8);
    }
    fence_mbar_init();
    long_count = 0;
  }
  if (warp == 0) tmem_alloc(&bar->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(bar->tmem);
  pdl_wait();
  KvJoinHeader* const header = &p.join.headers[blockIdx.x];
  if (!kShared && tid == 0) header->followers = 0;

  // units of a request; a warp to a request where all fit the block at once
  auto lane_units = [&](const KvRequest& r, int first, int step) {
    const int rows = many_rows(p, r);
    long long n = 0;
    for (int qt = first; qt * kItemRows < rows; qt += step) n += tile_shape(p, r, rows, qt).n + kItemCost;
    return n * p.cache.heads;
  };
  const int requests = kv_requests<kShared>(p.batch);
  const bool small = requests <= kThreads;
  if (small) {
    // short ones a thread to a request; those of many row tiles a warp each, dealt to
    // all warps wherever they stand among the requests
    if (tid < requests) {
      const KvRequest r = kv_request_or_prefix<kShared>(p.batch, p.cache.page, tid);
      if (many_rows(p, r) > 4 * kItemRows)
        long_requests[atomicAdd(&long_count, 1)] = (uint16_t)tid;  // in any order: each has its own sum
      else
        request_units[tid] = lane_units(r, 0, 1);
    }
    __syncthreads();
    for (int j = warp; j < long_count; j += kThreads / 32) {
      const int i = long_requests[j];
      long long v = lane_units(kv_request_or_prefix<kShared>(p.batch, p.cache.page, i), lane, 32);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) request_units[i] = v;
    }
    __syncthreads();
  }
  auto count = [&](int i) -> long long {
    return small ? request_units[i] : lane_units(kv_request_or_prefix<kShared>(p.batch, p.cache.page, i), 0, 1);
  };
  long long own, mine;
  search.count_all(requests, count, &own, &mine);
  const long long U = search.total;
  const long long n = min((long long)gridDim.x, U);
  const bool busy = (long long)blockIdx.x < n;
  if (busy) search.find(requests, count, U * blockIdx.x / n, own, mine);
  {
    PWalk w;
    w.u = w.u_end = 0;
    if (busy && search.request >= 0) {
      w.u = U * blockIdx.x / n;
      w.u_end = U * (blockIdx.x + 1) / n;
      w.start(p, search.request, search.first);
    }
    if (lane == 0) walks[warp] = w;
  }
  const PSegment& sg = segments[warp];
  auto next_segment = [&]() -> bool {  // all lanes of a warp
    __syncwarp();
    int there = 0;
    if (lane == 0) {
      PWalk w = walks[warp];
      PSegment s;
      there = w.next(p, &s);
      walks[warp] = w;
      if (there) segments[warp] = s;
    }
    __syncwarp();
    return __shfl_sync(0xffffffffu, there, 0) != 0;
  };
  uint32_t it = 0;  // stages so far

  if (warp >= 8 && warp < 8 + kCodeWarps) {
    // ---------------- codes into the tiles ----------------
    // A step writes the keys of one stage and the values of the stage before it
    // (S of a stage is formed during the softmax of the one before, its values
    // are needed a stage later).  Their 256 rows, keys then values, go round the
    // 96 threads: row 96 j + (thread) in round j; a warp's rows are all keys or
    // all values.
    constexpr int W = D / 32;  // 16-byte pieces of a row of codes
    constexpr int ROUNDS = 3, N = 32 * kCodeWarps;
    static_assert(ROUNDS * N >= 2 * kStage && (2 * kStage) % 32 == 0, "rounds");
    const int me = tid - 8 * 32;
    struct Place {
      int req, head, lo, hi, stage;
      bool have;
    };
    uint4 cw[ROUNDS][W];  // codes of the step at hand, then of the next
    uint32_t kpar[2], vpar[2];  // of this thread's tokens: the rows of keys are in the first two rounds
    bool live[ROUNDS];
    int page[ROUNDS];     // of the next step's rows
    auto pages = [&](const Place& kp, const Place& vp) {
#pragma unroll
      for (int j = 0; j < ROUNDS; ++j) {
        const int t = j * N + me;
        const Place& at = t < kStage ? kp : vp;
        const int key = at.stage * kStage + (t & (kStage - 1));
        page[j] = at.have && t < 2 * kStage && key >= at.lo && key < at.hi
                      ? __ldg(kv_table_row<kShared>(p.batch, at.req) + (key >> p.cache.page_shift))
                      : -1;
      }
    };
    auto load = [&](const Place& kp, const Place& vp) {
#pragma unroll
      for (int j = 0; j < ROUNDS; ++j) {
        live[j] = page[j] >= 0 && page[j] < p.cache.num_pages;
        if (j < 2) kpar[j] = vpar[j] = 0;
        if (live[j]) {
          const int t = j * N + me, part = t >> 7;
          const Place& at = t < kStage ? kp : vp;
          const int P = p.cache.page, off = (at.stage * kStage + (t & (kStage - 1))) & (P - 1);
          const uint8_t* blk = p.cache.blocks + ((uint32_t)page[j] * (uint32_t)p.cache.heads + at.head) *
                                                    (uint64_t)p.cache.block_bytes;
          const uint4* src = reinterpret_cast<const uint4*>(blk + (part * P + off) * (D / 2));
#pragma unroll
          for (int i = 0; i < W; ++i) cw[j][i] = __ldg(src + i);
          if (j < 2 && part == 0) {
            kpar[j] = __ldg(reinterpret_cast<const uint32_t*>(blk + P * D) + off);
            vpar[j] = __ldg(reinterpret_cast<const uint32_t*>(blk + P * D) + P + off);
          }
        } else {
#pragma unroll
          for (int i = 0; i < W; ++i) cw[j][i] = make_uint4(0, 0, 0, 0);
        }
      }
    };
    auto place = [&](bool have, int stage) { return Place{sg.req, sg.head, sg.lo, sg.hi, stage, have}; };
    bool ok = true;
    Place kp = place(next_segment(), 0), vp = kp;
    if (kp.have) kp.stage = sg.s0;
    vp.have = false;
    pages(kp, vp);
    load(kp, vp);
    uint32_t kit = 0, vit = 0;  // stages of keys, of values so far
    while (kp.have || vp.have) {
      Place nk = kp;  // the stage of keys after this one
      if (kp.have) {
        if (kp.stage + 1 < sg.s1) {
          ++nk.stage;
        } else {
          const bool more = next_segment();
          nk = place(more, more ? sg.s0 : 0);
        }
      }
      pages(nk, kp);
      const int ks = kit % KD, kt = kit % TD, vs = vit % VD;
      if (kp.have)
        ok = mbar_wait_long(&bar->t_empty[kt], ((kit / TD) & 1) ^ 1, 0x311, 100) &&
             mbar_wait_long(&bar->k_empty[ks], ((kit / KD) & 1) ^ 1, 0x312, 100);
      if (vp.have) ok = ok && mbar_wait_long(&bar->v_empty[vs], ((vit / VD) & 1) ^ 1, 0x313, 100);
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < ROUNDS; ++j) {
        const int t = j * N + me, tk = t & (kStage - 1);
        const bool val = t >= kStage;
        if ((t & ~31) >= 2 * kStage || !(val ? vp.have : kp.have)) continue;
        const uint32_t dst = smem_u32((val ? sv + vs * C::TILE : sk + ks * C::TILE)) + (uint32_t)tk * 128u;
        const uint32_t sw = (uint32_t)(tk & 7);
        if (!val) {
          // the softmax's constants of this token, its value's among them: the
          // softmax of a stage begins before the stage's values are here.  No
          // token: its logit is -infinity whatever the row.  A NaN among the
          // value's makes the logit NaN instead of the sums, which rows that
          // do not see the token share with those that do (0 times NaN)
          const float2 kb = __half22float2(*reinterpret_cast<const __half2*>(&kpar[j & 1]));
          const float2 vb = __half22float2(*reinterpret_cast<const __half2*>(&vpar[j & 1]));
          const float vsc = fmaxf(vb.x, 5.9604644775390625e-8f), rc = __fdividef(1.0f, vsc);
          const bool fine = live[j] && !isnan(vb.x + vb.y);
          const uint32_t tab = smem_u32(st + kt * C::TABLE) + (tk & 1) * 4;
          const uint32_t t1 = tab + (tk >> 1) * 16, t2 = t1 + kStage * 8, t3 = tab + kStage * 16 + (tk >> 1) * 8;
          sts_f32(t1, kb.x * (p.scale_log2 * 16777216.0f));
          sts_f32(t1 + 8, kb.y * p.scale_log2);
          sts_f32(t2, !live[j] ? -INFINITY : fine ? lg2(vsc) : NAN);
          sts_f32(t2 + 8, fine ? rc : 0.f);
          sts_f32(t3, fine ? fmaf(rc, vb.y, 8.0f) : 0.f);  // the value codes are centred: c - 8
        }
        // c 2^-24 of a key, (c - 8) 2^-24 of a value, exact; one form of the code
        // for both (the kernel's loops together outgrow the instruction cache)
        const uint32_t eight = val ? 0x00080008u : 0u;
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const uint32_t w4[4] = {cw[j][i].x, cw[j][i].y, cw[j][i].z, cw[j][i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t w = w4[k], c = 4 * i + k;  // 8-channel piece c
            sts128(dst + (c >> 3) * C::BLOCK + (((c & 7) ^ sw) << 4), hsub2u(w & 0x000F000Fu, eight),
                   hsub2u((w >> 4) & 0x000F000Fu, eight), hsub2u((w >> 8) & 0x000F000Fu, eight),
                   hsub2u((w >> 12) & 0x000F000Fu, eight));
          }
        }
      }
      load(nk, kp);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
#pragma unroll
        for (int j = 0; j < ROUNDS; ++j) {
          const int t = j * N + me;
          const bool val = t >= kStage;
          if (t >= 2 * kStage || !(val ? vp.have : kp.have)) continue;
          mbar_arrive(val ? &bar->v_full[vs] : &bar->k_full[ks]);
          if (!val) mbar_arrive(&bar->t_full[kt]);
        }
      }
      kit += kp.have;
      vit += vp.have;
      vp = kp;
      kp = nk;
    }
  } else if (warp >= 8) {
    // ---------------- MMA issue (one warp, converged) ----------------
    {
      bool ok = true;
      uint32_t q_seg[2] = {0, 0}, stages[2] = {0, 0};  // of each tile so far: the phases of q_full, p_full
      auto wait = [&](uint64_t* b, uint32_t parity, uint32_t where) -> bool {
        const bool there = mbar_wait_long(b, parity, where);
        return __all_sync(0xffffffffu, there);
      };
      // S of a tile and the stage in ring slot `slot` of the keys
      auto issue_s = [&](uint32_t tile, uint32_t slot) {
        const uint64_t a0 = sw128_desc(smem_u32(sq) + tile * C::TILE);
        const uint64_t b0 = sw128_desc(smem_u32(sk) + slot * C::TILE);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * C::BLOCK + (kk & 3) * 32) >> 4;
          mma_ss(tmem + kStage * tile, a0 + o, b0 + o, kIdescS, kk != 0);
        }
        commit(smem_u32(&bar->s_full[0]) + 8 * tile);
        commit(smem_u32(&bar->k_empty[0]) + 8 * slot);
      };
      // MMAs of one thread run in order, so the S issued next may overwrite the weights these read
      auto issue_o = [&](uint32_t tile, uint32_t slot, uint32_t half, uint32_t accum) {
        const uint64_t b0 = sw128_desc_n(smem_u32(sv) + slot * C::TILE + half * (kHalf * 128), C::BLOCK);
#pragma unroll
        for (int kk = 0; kk < kHalf / 16; ++kk)
          mma_ts(tmem + 2 * kStage + D * tile, tmem + kStage * tile + (kHalf / 2) * half + kk * 8, b0 + kk * (2048 >> 4),
                 kIdescO<D>, kk ? 1u : accum);
        commit(smem_u32(&bar->o_done[0][0]) + 16 * tile + 8 * half);
        if (half) commit(smem_u32(&bar->v_empty[0]) + 8 * slot);
      };
      while (ok && next_segment()) {
        it = uniform(it);
        uint32_t left[2], at[2] = {it, it}, half[2] = {0, 0};  // by tile: stages left, the stage and half whose weights come next
        ok = wait(&bar->k_full[it % KD], (it / KD) & 1, 0x321);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          left[i] = uniform((uint32_t)(sg.tile_end[i] - sg.s0));
          if (!ok || left[i] == 0) continue;
          ok = wait(&bar->q_full[i], q_seg[i] & 1, 0x322);
          ++q_seg[i];
          if (!ok) continue;
          tc_fence_after();
          issue_s(i, it % KD);
        }
        // whichever tile's weights are there first
        uint64_t since = 0;
        uint32_t tries = 0;  // without a result
        while (ok && (left[0] | left[1])) {
          bool idle = true;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (left[i] == 0 || !ok) continue;
            const bool there = mbar_try_wait(&bar->p_full[i][half[i]], stages[i] & 1);
            if (!__all_sync(0xffffffffu, there)) continue;
            idle = false;
            tc_fence_after();
            const uint32_t a = at[i], h = half[i];
            if (h == 0) ok = wait(&bar->v_full[a % VD], (a / VD) & 1, 0x324);
            if (!ok) continue;
            issue_o(i, a % VD, h, a != it || h ? 1u : 0u);
            half[i] = h ^ 1;
            if (h) {
              ++stages[i];
              ++at[i];
              if (--left[i]) {
                ok = wait(&bar->k_full[(a + 1) % KD], ((a + 1) / KD) & 1, 0x323);
                if (ok) issue_s(i, (a + 1) % KD);
              }
            }
          }
          if (!idle) {
            tries = 0;
          } else if ((++tries & 255u) == 0) {
            const uint64_t now = globaltimer_ns();
            if (tries == 256) since = now;
            if (now - since > kWaitLimitNs) {
              record_timeout(0x325);
              ok = false;
            }
            ok = __all_sync(0xffffffffu, ok);
          }
        }
        it += uniform((uint32_t)(sg.s1 - sg.s0));
      }
    }
  } else {
    // ---------------- softmax ----------------
    const int tile = warp >> 2, quarter = warp & 3;
    const int r = lane >> 2, qd = lane & 3;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t ts_tile = lanes + kStage * tile;              // S of the two halves, and the weights over them
    const uint32_t to_addr = lanes + 2 * kStage + D * tile;      // O
    uint32_t done = 0;  // stages of this tile so far: the phase of its barriers
    // A wait that gave up ends waiting for good, but nothing else.
    bool ok = true;
    while (next_segment()) {
      const KvRequest rq = sg.rq;
      const int rows = min(kRows, sg.rows - kRows * tile);  // of this tile; below 1: none
      const int base_pos = rq.base;
      const int end = sg.tile_end[tile], s_end = sg.s1;
      const bool none = end == sg.s0;  // no row of the tile sees a key of the share
      // Q: a thread to a row, in the codes' channel order
      float qsum = 0.f;
      if (!none) {
        const int my = 32 * quarter + lane;
        const int grow = sg.row0 + kRows * tile + my;
        const bool on = my < rows;
        const int t = divide(grow, p.by_share), g = grow - t * p.share;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(rq.q0 + (on ? t : 0)) * p.ldq +
                                                          (long long)(sg.head * p.share + (on ? g : 0)) * D);
        const uint32_t dst = smem_u32(sq + tile * C::TILE) + my * 128u;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = on ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
            qsum += f.x + f.y;
          }
          sts128(dst + (c >> 3) * C::BLOCK + (((c & 7) ^ (my & 7)) << 4), prmt(v.x, v.z, 0x5410), prmt(v.x, v.z, 0x7632),
                 prmt(v.y, v.w, 0x5410), prmt(v.y, v.w, 0x7632));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->q_full[tile]);
      }
      float qs[4], m[4];
      float l[4], beta[4];
      int pos[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // rows r + 8 k of this warp's 32
        qs[k] = __shfl_sync(0xffffffffu, qsum, r + 8 * k);
        pos[k] = base_pos + divide(sg.row0 + min(kRows * tile + 32 * quarter + r + 8 * k, sg.rows - 1), p.by_share);
        m[k] = kNone;
        l[k] = beta[k] = 0.f;
      }
      // keys below all_hi and from all_lo are seen by every row of the tile
      const int all_hi = base_pos + divide(sg.row0 + kRows * tile, p.by_share) + 1;
      const int all_lo =
          p.window > 0 ? base_pos + divide(sg.row0 + max(0, kRows * tile + rows - 1), p.by_share) - p.window + 1 : 0;

      int s = sg.s0;
      for (; s < end; ++s, ++it, ++done) {
        ok = ok && mbar_wait_long(&bar->t_full[it % TD], (it / TD) & 1, 0x332) &&
             mbar_wait(&bar->s_full[tile], done & 1, 0x333);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int key0 = s * kStage + half * kHalf;
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          const uint8_t* tab = st + (it % TD) * C::TABLE + half * (kHalf * 8) + qd * 16;
          const uint8_t* tab3 = st + (it % TD) * C::TABLE + kStage * 16 + half * (kHalf * 4) + qd * 8;
          const uint32_t ts_addr = ts_tile + kHalf * half, tp_addr = ts_tile + (kHalf / 2) * half;  // S, weights over the first half
          // v[c][0]: columns 32 c .. of rows r, r + 8; v[c][1]: of rows r + 16, r + 24
          float v[2][2][16];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_ld_16x256(ts_addr + 32 * c, v[c][0]);
            tmem_ld_16x256(ts_addr + 32 * c + (16u << 16), v[c][1]);
          }
          float2 rc[2][4];
          float top[4];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_wait_ld(v[c][0]);
            tmem_wait_ld(v[c][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {  // column pair 32 c + 8 k + 2 qd
              const float4 ab = *reinterpret_cast<const float4*>(tab + (16 * c + 4 * k) * 16);
              const float4 lr = *reinterpret_cast<const float4*>(tab + (16 * c + 4 * k) * 16 + kStage * 8);
              rc[c][k] = make_float2(lr.z, lr.w);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                float* x = &v[c][y >> 1][4 * k + 2 * (y & 1)];
                const float2 z =
                    fma2(make_float2(x[0], x[1]), make_float2(ab.x, ab.y),
                         fma2(make_float2(qs[y], qs[y]), make_float2(ab.z, ab.w), make_float2(lr.x, lr.y)));
                x[0] = z.x;
                x[1] = z.y;
              }
            }
          }
          if (key0 < all_lo || key0 + kHalf > all_hi) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int to = pos[y] - key0 - 2 * qd;  // the last column that row y sees, counted from this thread's first
              const int from = p.window > 0 ? to - p.window : -kStage;  // and the one before the first
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int col = 8 * (e >> 1) + (e & 1);
                float* x = &v[e >> 3][y >> 1][4 * ((e >> 1) & 3) + 2 * (y & 1) + (e & 1)];
                if (col > to || col <= from) *x = -INFINITY;
              }
            }
          }
          bool over = false;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float* x = &v[0][y >> 1][2 * (y & 1)];
            const float* z = &v[1][y >> 1][2 * (y & 1)];
            top[y] = max3(max3(max3(x[0], x[1], x[4]), max3(x[5], x[8], x[9]), max3(x[12], x[13], z[0])),
                          max3(z[1], z[4], z[5]), max3(max3(z[8], z[9], z[12]), z[13], kNone));
            over |= top[y] > m[y] + kTrigger;
          }
          if (__any_sync(0xffffffffu, over)) {
            // a new reference: the sums and O move with it (the weights of the
            // other half are in O by now, or will have been added before it moves)
            float w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              float x = top[y];
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
              const float next = fmaxf(m[y], x - kHeadroom);
              w[y] = ex2(m[y] - next);
              m[y] = next;
              l[y] *= w[y];
              beta[y] *= w[y];
            }
            if (s > sg.s0 || half) {
              ok = ok && mbar_wait_long(&bar->o_done[tile][half ^ 1], (half ? done : done - 1) & 1, 0x334);
              ok = __all_sync(0xffffffffu, ok);
              tc_fence_after();
#pragma unroll 1
              for (int b = 0; b < D / 32; ++b) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  float ov[16];
                  tmem_ld_16x256(to_addr + 32 * b + ((16u * h) << 16), ov);
                  tmem_wait_ld(ov);
#pragma unroll
                  for (int k = 0; k < 16; ++k) ov[k] *= w[2 * h + ((k >> 1) & 1)];
                  tmem_st_16x256(to_addr + 32 * b + ((16u * h) << 16), ov);
                }
              }
            }
          }
          // weights, and this half's sums by even and odd columns
          float2 lt[4], bt[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) lt[y] = bt[y] = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pw[2][8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 rb = *reinterpret_cast<const float2*>(tab3 + (16 * c + 4 * k) * 8);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float* x = &v[c][y >> 1][4 * k + 2 * (y & 1)];
                const float2 a = add2(make_float2(x[0], x[1]), make_float2(-m[y], -m[y]));
                const float2 e = make_float2(ex2(a.x), ex2(a.y));
                const __half2 h2 = __floats2half2_rn(e.x, e.y);
                pw[y >> 1][2 * k + (y & 1)] = *reinterpret_cast<const uint32_t*>(&h2);
                lt[y] = fma2(e, rc[c][k], lt[y]);
                bt[y] = fma2(e, rb, bt[y]);
              }
            }
            tmem_st_16x128(tp_addr + 16 * c, pw[0]);
            tmem_st_16x128(tp_addr + 16 * c + (16u << 16), pw[1]);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            l[y] += lt[y].x + lt[y].y;
            beta[y] += bt[y].x + bt[y].y;
          }
          if (lane == 0) mbar_arrive(&bar->p_full[tile][half]);
        }
        if (lane == 0) mbar_arrive(&bar->t_empty[it % TD]);
      }
      // stages that the tile does not see: let the rings go on
      for (; s < s_end; ++s, ++it) {
        ok = ok && mbar_wait_long(&bar->t_full[it % TD], (it / TD) & 1, 0x331) &&
             mbar_wait_long(&bar->v_full[it % VD], (it / VD) & 1, 0x336);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bar->t_empty[it % TD]);
          if (quarter == 0) {
            mbar_arrive(&bar->k_empty[it % KD]);
            mbar_arrive(&bar->v_empty[it % VD]);
          }
        }
      }
      if (rows <= 0) continue;

      // ---- the item's end: sums of the quads, then a thread to a row ----
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          l[k] += __shfl_xor_sync(0xffffffffu, l[k], o);
          beta[k] += __shfl_xor_sync(0xffffffffu, beta[k], o);
        }
      }
      if (!none) ok = ok && mbar_wait_long(&bar->o_done[tile][1], (done - 1) & 1, 0x335);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const bool whole = sg.first && sg.last;
      auto end_block = [&]() -> int {  // the block that holds the item's last unit
        const long long last_u = sg.item_end - 1;
        long long b = ((last_u + 1) * n - 1) / U;
        while (U * b / n > last_u) --b;
        while (U * (b + 1) / n <= last_u) ++b;
        return (int)b;
      };
      const int row0 = 32 * quarter + r;  // this thread's rows: row0 + 8 y
      const float up = 16777216.0f;       // codes were entered as c 2^-24
      if (!kShared && whole) {
        float inv[4];
        __half* orow[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          inv[y] = l[y] == 0.f ? 0.f : 1.0f / l[y];  // no key seen: zeros
          const int gr = sg.row0 + kRows * tile + min(row0 + 8 * y, rows - 1);
          const int t = divide(gr, p.by_share), g = gr - t * p.share;
          orow[y] = p.out + (long long)(rq.q0 + t) * p.ldo + (long long)(sg.head * p.share + g) * D + 8 * qd;
        }
#pragma unroll 1
        for (int b = 0; b < D / 32; ++b) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[16];
            tmem_ld_16x256(to_addr + 32 * b + ((16u * h) << 16), x);
            tmem_wait_ld(x);
            if (none) {  // O was not formed
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int y = 2 * h + e;
              // Of 8 channels k = 0 .. 3 this thread holds qd' and qd' + 4 (qd' = 0 1 2 3:
              // positions 0 1 | 2 3 | 4 5 | 6 7 are channels 0 4 | 1 5 | 2 6 | 3 7).  The
              // quad transposes: each thread takes one whole group of 8, k = qd.
              uint32_t mine[4];  // (channel qd, channel qd + 4) of group k
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const __half2 o2 = __floats2half2_rn(fmaf(x[4 * k + 2 * e], up, beta[y]) * inv[y],
                                                     fmaf(x[4 * k + 2 * e + 1], up, beta[y]) * inv[y]);
                mine[k] = *reinterpret_cast<const uint32_t*>(&o2);
              }
              // afterwards mine[i] is thread i's pair of group qd
              {
                const bool odd = qd & 1, high = qd & 2;
                const uint32_t a = __shfl_xor_sync(0xffffffffu, odd ? mine[0] : mine[1], 1);
                const uint32_t c = __shfl_xor_sync(0xffffffffu, odd ? mine[2] : mine[3], 1);
                mine[0] = odd ? a : mine[0];
                mine[1] = odd ? mine[1] : a;
                mine[2] = odd ? c : mine[2];
                mine[3] = odd ? mine[3] : c;
                const uint32_t d = __shfl_xor_sync(0xffffffffu, high ? mine[0] : mine[2], 2);
                const uint32_t f = __shfl_xor_sync(0xffffffffu, high ? mine[1] : mine[3], 2);
                mine[0] = high ? d : mine[0];
                mine[1] = high ? f : mine[1];
                mine[2] = high ? mine[2] : d;
                mine[3] = high ? mine[3] : f;
              }
              if (row0 + 8 * y < rows)
                *reinterpret_cast<uint4*>(orow[y] + 32 * b) =
                    make_uint4(prmt(mine[0], mine[1], 0x5410), prmt(mine[2], mine[3], 0x5410),
                               prmt(mine[0], mine[1], 0x7632), prmt(mine[2], mine[3], 0x7632));
            }
          }
        }
      } else {
        // a partial (or a whole row's sums), its columns in TMEM's order
        float *po[4], *pm[4];
        int lstep = kItemRows;  // from m to l
        float* const part = p.join.parts + ((size_t)blockIdx.x * 2 + (sg.first ? 1 : 0)) * (kItemRows * (D + 2));
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          po[y] = part + (size_t)(kRows * tile + row0 + 8 * y) * D + 2 * qd;
          pm[y] = part + kItemRows * D + kRows * tile + row0 + 8 * y;
        }
        if (kShared && sg.first) {
          const KvRowSums& sums = sg.req < p.batch.requests ? p.shared.own : p.shared.prefix;
          const int followers = whole ? 0 : end_block() - (int)blockIdx.x;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int gr = sg.row0 + kRows * tile + min(row0 + 8 * y, rows - 1);
            const int t = divide(gr, p.by_share), g = gr - t * p.share;
            const size_t at = (size_t)(rq.q0 + t) * p.q_heads + sg.head * p.share + g;
            if (whole) {
              lstep = 1;
              po[y] = sums.o + at * D + 2 * qd;
              pm[y] = reinterpret_cast<float*>(sums.ml + at);
            } else if (qd == 0 && row0 + 8 * y < rows) {
              sums.ml[at] = kv_row_in_parts(blockIdx.x | kPartsOfMany, followers);
            }
          }
        }
#pragma unroll 1
        for (int b = 0; b < D / 32; ++b) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[16];
            tmem_ld_16x256(to_addr + 32 * b + ((16u * h) << 16), x);
            tmem_wait_ld(x);
            if (none) {  // O was not formed
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int y = 2 * h + e;
              if (row0 + 8 * y < rows) {
                float* dst = po[y] + 32 * b;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  *reinterpret_cast<float2*>(dst + 8 * k) =
                      make_float2(fmaf(x[4 * k + 2 * e], up, beta[y]), fmaf(x[4 * k + 2 * e + 1], up, beta[y]));
              }
            }
          }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
          if (qd == 0 && row0 + 8 * y < rows) {
            pm[y][0] = m[y];
            pm[y][lstep] = l[y];
          }
      }
      tc_fence_before();
      if (!kShared && !whole && sg.first && tid == 0)
        *header = KvJoinHeader{end_block() - (int)blockIdx.x, rq.q0, sg.row0, sg.rows, sg.head};
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D>
tlq_status launch_one(const PrefillAttnParams& p, cudaStream_t stream) {
  using C = PCfg<D>;
  auto kernel = prefill_attention_kernel<D>;
  const cudaError_t attr = opt_in_smem<prefill_attention_kernel<D>>(C::SMEM);
  if (attr != cudaSuccess) return cuda_error(attr, "kv4 attention: shared memory");
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)p.join.blocks, 1, 1);
  lc.blockDim = dim3(kThreads, 1, 1);
  lc.dynamicSmemBytes = C::SMEM;
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  return cuda_error(cudaLaunchKernelEx(&lc, kernel, p), "kv4 prompt attention: launch");
}

}  // namespace

#if !TLQ_KV_SHARED_UNIT
size_t kv4_prefill_workspace(int head_dim) { return kv_join_bytes(device_info().sms, kItemRows, head_dim); }
#endif

#if TLQ_KV_SHARED_UNIT
tlq_status launch_kv4_prefill_shared(
#else
tlq_status launch_kv4_prefill(
#endif
    const KvAttention& a, int few_rows, void* ws, KvJoin* join, cudaStream_t stream) {
  PrefillAttnParams p{};
  p.cache = a.cache;
  p.batch = a.batch;
  p.q = a.q;
  p.ldq = a.ldq;
  p.out = a.out;
  p.ldo = a.ldo;
  p.scale_log2 = (float)((double)a.scale * M_LOG2E);
  p.window = a.window;
  p.share = a.q_heads / a.cache.heads;
  p.by_share = fast_div((uint32_t)p.share);
  p.few_rows = few_rows;
  p.shared = a.shared;
  p.q_heads = a.q_heads;
  p.join = *join = kv_join_at(ws, device_info().sms, kItemRows);
  return a.head_dim == 64 ? launch_one<64>(p, stream) : launch_one<128>(p, stream);
}

}  // namespace tlq
