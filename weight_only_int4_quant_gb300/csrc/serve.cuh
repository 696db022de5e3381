// Shared parts of the multi-request serving operators: the geometry of the
// paged 4-bit cache, the batch a kernel is given, and the search that turns a
// position in the batch's work into a request.
#pragma once

#include <atomic>

#include "common.cuh"

namespace tlq {

// n / d for n < 2^31 by one multiplication (d >= 1): m = ceil(2^(31 + s) / d)
// with 2^s >= d errs by less than 1 / d.
struct FastDiv {
  uint32_t d, m;
  int s;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1ull << f.s) < d) ++f.s;
  f.m = (uint32_t)(((1ull << (31 + f.s)) + d - 1) / d);
  return f;
}
__device__ __forceinline__ int divide(int n, const FastDiv& f) {
  return (int)(((uint64_t)(uint32_t)n * f.m) >> (31 + f.s));
}

// Two FP32 operations in one instruction, each rounded as by itself.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
      " fma.rn.f32x2 w, x, y, z;\n mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 w, x, y;\n"
      " mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 w, x, y;\n"
      " mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// The cache: blocks is [pages][heads][block_bytes]; a block holds the key
// codes [page][D/2], the value codes [page][D/2], the key parameters
// [page][D/group][2] and the value parameters (FP16 scale, minimum).  Keys and
// values of one page and head are one contiguous piece, so a 16-token page
// moves with a single bulk copy.
struct KvCache {
  uint8_t* blocks;
  long long num_pages;
  int heads, page, group;  // page: tokens, a power of two >= 16
  int page_shift;
  int block_bytes;
};

__host__ __device__ inline int kv_block_bytes(int page, int head_dim, int group) {
  return page * head_dim + 8 * page * (head_dim / group);
}

// The step's requests.  Request b has queries [q_start[b], q_start[b+1]) and
// seq_lens[b] tokens in the cache, the queries' own among them.
struct KvBatch {
  const int* q_start;
  const int* seq_lens;
  const int* table;
  int ld_table;
  int requests, tokens, max_q;
};

// The longest context (positions and windows stay far from 32-bit limits).
constexpr long long kMaxContext = 1ll << 30;

struct KvRequest {
  int q0, q_len;  // first query's row; queries that are worked on
  int base;       // the first query's position (negative: before the first token)
  int len;        // tokens that the table's row has room for
};

// Lengths as the kernels use them: queries outside [0, tokens) and tokens
// behind the table's row count as none.  Positions come from the request's own
// lengths, whatever is left out of its queries or tokens.
__device__ __forceinline__ KvRequest kv_request(const KvBatch& b, int page, int i) {
  KvRequest r;
  r.q0 = b.q_start[i];
  const int q1 = b.q_start[i + 1];
  const int queries = (r.q0 >= 0 && q1 >= r.q0 && q1 <= b.tokens) ? q1 - r.q0 : 0;
  const int tokens = min(max(b.seq_lens[i], 0), (int)kMaxContext);
  r.q_len = min(queries, b.max_q);
  r.base = max(tokens - queries, -(int)kMaxContext);
  r.len = (int)min((long long)tokens, (long long)b.ld_table * page);
  return r;
}

// Where unit `u` of the batch's work lies: requests have count(i) units each,
// in order.  All THREADS threads of a block call it together; the totals and
// the request found come back through shared memory.
template <int THREADS>
struct UnitSearch {
  long long warp_sum[THREADS / 32];
  long long total;
  long long first;  // first unit of the request found
  int request;      // -1: none

  __device__ long long scan(long long v, long long* sum) {  // inclusive scan over the block
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += n;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = v;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      all += warp_sum[w];
    }
    *sum = all;
    return v + before;
  }

  // total units of the batch; with one chunk of requests *own is this thread's
  // inclusive prefix and *mine its count, which find() takes again
  template <class F>
  __device__ void count_all(int requests, F count, long long* own, long long* mine) {
    long long v = 0;
    for (int i = threadIdx.x; i < requests; i += THREADS) v += count(i);
    long long sum;
    *own = scan(v, &sum);
    *mine = v;
    if (threadIdx.x == 0) {
      total = sum;
      request = -1;
    }
    __syncthreads();
  }

  template <class F>
  __device__ void find(int requests, F count, long long u, long long own, long long mine) {
    if (requests <= THREADS) {
      if (mine > 0 && own - mine <= u && u < own) {
        request = threadIdx.x;
        first = own - mine;
      }
    } else {
      long long base = 0;
      for (int c = 0; c < requests; c += THREADS) {
        const int i = c + threadIdx.x;
        const long long n = i < requests ? count(i) : 0;
        long long sum;
        const long long upto = scan(n, &sum) + base;
        if (n > 0 && upto - n <= u && u < upto) {
          request = i;
          first = upto - n;
        }
        base += sum;
        if (base > u) break;  // the same for every thread
      }
    }
    __syncthreads();
  }
};

// mbar_wait for waits that last a stage or more, with a pause between tries, so
// that a waiting warp leaves the scheduler to the others (waiting warps issued a
// third of the prompt kernel's instructions).  Bounded like mbar_wait.
__device__ __forceinline__ bool mbar_wait_long(uint64_t* bar, uint32_t parity, uint32_t where, uint32_t pause_ns = 20) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    __nanosleep(pause_ns);
    if ((i & 63u) == 63u && globaltimer_ns() - t0 > kWaitLimitNs) {
      record_timeout(where);
      return false;
    }
  }
}

// Opts a kernel in to `bytes` of dynamic shared memory on the current device:
// the attribute is the device's, so it is set once on each, and again after a
// failure.
template <auto kKernel>
cudaError_t opt_in_smem(int bytes) {
  static std::atomic<uint64_t> done{0};  // a bit for each of the first 64 devices
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t set = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (set == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return set;
}

// Launchers (arguments validated by the entry points).
struct KvPlanArgs {
  const int* cached;
  const int* added;
  int requests;
  int* table;
  int ld_table;
  const int* free_pages;
  int num_free;
  const int* free_head;
  int page;
  long long num_pages;
  int* q_start;
  int* seq_lens;
  int* token_req;
  int* token_pos;
  long long* slots;
  int capacity;
  int* counts;
};
tlq_status launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream);
tlq_status launch_kv4_append(const KvCache& c, int head_dim, const __half* k, long long ldk, const __half* v,
                             long long ldv, const long long* slots, int tokens, cudaStream_t stream);
tlq_status launch_kv4_read(const KvCache& c, int head_dim, const long long* slots, int tokens, __half* k, __half* v,
                           cudaStream_t stream);

struct KvAttention {
  KvCache cache;
  KvBatch batch;
  int head_dim, q_heads;
  const __half* q;
  long long ldq;
  __half* out;
  long long ldo;
  float scale;
  int window;
};
// What the joining kernel needs of an item that a block began but did not end.
struct KvJoinHeader {
  int followers;  // blocks after this one that hold a part of the item; 0: nothing to join
  int q0;         // first query of the request
  int row0;       // first (query, head) row of the item
  int rows;
  int head;       // key head
};
// The parts that one kernel leaves: two to a block, of the item it ends (0) and
// of the one it begins (1).
struct KvJoin {
  KvJoinHeader* headers;  // [blocks]
  float* parts;           // [blocks][2][O [rows][D], m [rows], l [rows]]
  int blocks, rows;
};
inline size_t kv_join_bytes(int blocks, int rows, int head_dim) {
  return ((blocks * sizeof(KvJoinHeader) + 255) & ~size_t(255)) +
         (size_t)blocks * 2 * rows * (head_dim + 2) * sizeof(float);
}
inline KvJoin kv_join_at(void* ws, int blocks, int rows) {
  KvJoin j;
  j.headers = static_cast<KvJoinHeader*>(ws);
  j.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + ((blocks * sizeof(KvJoinHeader) + 255) & ~size_t(255)));
  j.blocks = blocks;
  j.rows = rows;
  return j;
}

// Requests of up to few_rows (query, head) rows to a key head go through the
// first kernel, the others through the second; each passes over what is not its
// own.  *_workspace: bytes of the parts; the launches say where they lie.
size_t kv4_decode_workspace(int head_dim);
size_t kv4_prefill_workspace(int head_dim);
tlq_status launch_kv4_decode(const KvAttention& a, int few_rows, void* ws, KvJoin* join, cudaStream_t stream);
tlq_status launch_kv4_prefill(const KvAttention& a, int few_rows, void* ws, KvJoin* join, cudaStream_t stream);
tlq_status launch_kv4_join(const KvAttention& a, const KvJoin& few, const KvJoin& many, cudaStream_t stream);

struct LoraArgs {
  const __half* x;
  long long ldx;
  const __half* A;
  const __half* B;
  const float* scales;
  const int* q_start;
  const int* adapters;
  int requests, tokens, max_q;
  int K, N, rank, num_adapters;
  const __half* y;
  long long ldy;
  __half* out;
  long long ldo;
};
tlq_status launch_lora(const LoraArgs& a, cudaStream_t stream);

}  // namespace tlq
