// Block tables, slots and positions of a step's tokens, from request lengths.
//
//   held_b = ceil(cached_b / P), need_b = ceil((cached_b + added_b) / P) - held_b
//   table[b][held_b + i] = free[head + sum_{c<b} need_c + i],  i < need_b
//   q_start = exclusive sums of added;  token t of request b: position
//   cached_b + (t - q_start_b), slot = table[b][position / P] * P + position % P
//
// Whole-number work of a few hundred kilobytes at most: latency bounds it, so
// it is one launch in which no block waits for another.  Every block sums the
// lengths of the requests before its 256 by itself (8 bytes each, from L2)
// instead of passing sums between blocks (so its work grows with the square of
// the requests: right for thousands, seconds for tens of millions); the blocks
// of one set of 256 requests share that set's tokens and table rows.  1000 requests with 55000 new
// tokens: 5.6 us; 16 requests: 2.7 us, most of it the launch.
#include <algorithm>

#include "serve.cuh"

namespace tlq {
namespace {

constexpr int kPlanThreads = 256;

struct PlanShape {
  int cached, added, held, need, wanted;
};

__device__ __forceinline__ PlanShape plan_shape(const KvPlanArgs& a, int i) {
  PlanShape s{0, 0, 0, 0, 0};
  if (i >= a.requests) return s;
  s.cached = max(a.cached[i], 0);
  s.added = max(a.added[i], 0);
  const long long P = a.page, total = (long long)s.cached + s.added;
  const long long held = ((long long)s.cached + P - 1) / P, all = (total + P - 1) / P;
  s.held = (int)min(held, (long long)a.ld_table);
  s.need = (int)min(all, (long long)a.ld_table) - s.held;
  s.wanted = (int)(all - held);
  return s;
}

// inclusive scan over the block of two values packed by the caller
__device__ __forceinline__ longlong2 scan2(longlong2 v, longlong2* warp_sum, longlong2* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += x;
      v.y += y;
    }
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  longlong2 before{0, 0}, all{0, 0};
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const longlong2 s = warp_sum[w];
    if (w < warp) {
      before.x += s.x;
      before.y += s.y;
    }
    all.x += s.x;
    all.y += s.y;
  }
  *sum = all;
  return longlong2{v.x + before.x, v.y + before.y};
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const KvPlanArgs a, int page_shift) {
  __shared__ longlong2 warp_sum[kPlanThreads / 32];
  __shared__ long long tok[kPlanThreads + 1];   // first token of each request of the set
  __shared__ long long pages[kPlanThreads];     // first new page of each request (an index into free_pages)
  __shared__ int held_s[kPlanThreads], need_s[kPlanThreads], cached_s[kPlanThreads];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  const int c0 = (int)blockIdx.x * kPlanThreads;

  // tokens, new pages and wanted pages of the requests before this set
  longlong2 before{0, 0}, wanted{0, 0}, sum;
  for (int i = tid; i < c0; i += kPlanThreads) {
    const PlanShape s = plan_shape(a, i);
    before.x += s.added;
    before.y += s.need;
    wanted.x += s.wanted;
  }
  if (c0 > 0) {
    scan2(before, warp_sum, &sum);
    before = sum;
    scan2(wanted, warp_sum, &sum);
    wanted = sum;
  }

  const PlanShape s = plan_shape(a, c0 + tid);
  const longlong2 upto = scan2(longlong2{s.added, s.need}, warp_sum, &sum);
  const long long head = a.free_head ? (long long)max(*a.free_head, 0) : 0;
  const long long t0 = before.x + upto.x - s.added;
  tok[tid] = t0;
  pages[tid] = head + before.y + upto.y - s.need;
  held_s[tid] = s.held;
  need_s[tid] = s.need;
  cached_s[tid] = s.cached;
  if (tid == kPlanThreads - 1) tok[kPlanThreads] = before.x + sum.x;
  longlong2 wsum;
  scan2(longlong2{s.wanted, 0}, warp_sum, &wsum);  // its barriers also publish the arrays above

  const bool last = blockIdx.x + 1 == gridDim.x;
  const long long total = before.x + sum.x;
  if (blockIdx.y == 0) {
    if (c0 + tid < a.requests) {
      a.q_start[c0 + tid] = (int)min(t0, 0x7fffffffll);
      a.seq_lens[c0 + tid] = (int)min((long long)s.cached + s.added, 0x7fffffffll);
    }
    if (last && tid == 0) {
      a.q_start[a.requests] = (int)min(total, 0x7fffffffll);
      const long long avail = max(0ll, (long long)a.num_free - head);
      const long long taken = min(before.y + sum.y, avail);
      a.counts[0] = (int)min(total, 0x7fffffffll);
      a.counts[1] = (int)taken;
      a.counts[2] = (int)(head + taken);
      a.counts[3] = (int)(wanted.x + wsum.x - taken);
    }
  }

  auto free_page = [&](long long at) { return at < a.num_free ? a.free_pages[at] : -1; };

  // table rows: a warp to a request
  const int lane = tid & 31;
  for (int i = (int)blockIdx.y * (kPlanThreads / 32) + (tid >> 5); i < kPlanThreads && c0 + i < a.requests;
       i += (int)gridDim.y * (kPlanThreads / 32)) {
    int* row = a.table + (size_t)(c0 + i) * a.ld_table + held_s[i];
    const long long p0 = pages[i];
    for (int j = lane; j < need_s[i]; j += 32) row[j] = free_page(p0 + j);
  }

  // tokens: a thread to a token; new pages are read from the free list, not
  // from the table, whose rows other blocks are writing
  const long long end = min(tok[kPlanThreads], (long long)a.capacity);
  const int P = 1 << page_shift;
  for (long long t = tok[0] + (long long)blockIdx.y * kPlanThreads + tid; t < end;
       t += (long long)gridDim.y * kPlanThreads) {
    int lo = 0, hi = kPlanThreads;  // the last request with tok[i] <= t (requests without tokens are passed over)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tok[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const long long pos = cached_s[lo] + (t - tok[lo]);
    const long long pi = pos >> page_shift;
    int page = -1;
    if (pi < held_s[lo])
      page = a.table[(size_t)(c0 + lo) * a.ld_table + pi];
    else if (pi - held_s[lo] < need_s[lo])
      page = free_page(pages[lo] + pi - held_s[lo]);
    a.token_req[t] = c0 + lo;
    a.token_pos[t] = (int)min(pos, 0x7fffffffll);
    a.slots[t] = page >= 0 && page < a.num_pages ? (long long)page * P + (pos & (P - 1)) : -1;
  }
  if (last) {
    for (long long t = total + (long long)blockIdx.y * kPlanThreads + tid; t < a.capacity;
         t += (long long)gridDim.y * kPlanThreads) {
      a.token_req[t] = -1;
      a.token_pos[t] = -1;
      a.slots[t] = -1;
    }
  }
}

}  // namespace

tlq_status launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
  int shift = 0;
  while ((1 << shift) < a.page) ++shift;
  const int sets = a.requests > 0 ? (a.requests - 1) / kPlanThreads + 1 : 1;
  // enough blocks for one token or one table row per thread or warp, at most a wave;
  // sets go along x, which has no limit that requests could reach
  long long y = ((long long)a.capacity + kPlanThreads - 1) / kPlanThreads / sets + 1;
  y = std::min<long long>(y, std::max(1, 2 * device_info().sms / sets));
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)sets, (unsigned)y, 1);
  lc.blockDim = dim3(kPlanThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  return cuda_error(cudaLaunchKernelEx(&lc, plan_kernel, a, shift), "kv plan: launch");
}

}  // namespace tlq
