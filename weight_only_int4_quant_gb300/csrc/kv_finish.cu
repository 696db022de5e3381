// The last step of the attention of a batch with a shared prefix: a row's sums
// lie in parts, of the prefix and of its request's own tokens, each either one
// row (an item that one block did whole) or one in every block that did a piece
// of the item:  o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,  m = max m_i,
// in the order of the blocks, the own parts first.
//
// A thread to 8 channels of a row, so that all rows' parts are under way at
// once: a prefix of 8 heads lies in 19 parts each, and a set of blocks to an
// item took 29 us where this takes 6 (64 requests, 32 / 8 heads of 128).  Latency
// bounds it: row, parts, sums.
#include <algorithm>

#include "serve.cuh"

namespace tlq {
namespace {

constexpr int kThreads = 128;

// One row's parts on one side.
struct RowParts {
  const float *o, *m, *l;
  size_t f;  // floats of a part
  int n;
  bool permuted;  // of the tensor-core kernel, whose channels lie as 0 4 1 5 2 6 3 7
  __device__ __forceinline__ size_t at(int i) const { return i ? (size_t)(2 * i - 1) * f : 0; }
};

// gr: the row among its request's (query, head) rows; many: which kernel takes
// that request.  Where parts lie goes by what their kernel wrote, checked against
// its blocks, so that lengths that contradict each other (requests whose queries
// overlap) lead to no address outside the workspace.
template <int D>
__device__ __forceinline__ RowParts row_parts(const KvRowSums& sums, size_t row, int gr, bool many, const KvJoin& few_parts,
                                              const KvJoin& many_parts) {
  const float2 ml = sums.ml[row];
  RowParts r;
  if (ml.y < 0.f) {
    const int mark = __float_as_int(ml.x), block = mark & (kPartsOfMany - 1), followers = (int)fminf(-ml.y, 1e6f);
    r.permuted = mark & kPartsOfMany;
    const KvJoin& j = r.permuted ? many_parts : few_parts;
    const int R = j.rows, item_row = gr % max(R, 1);
    r.f = (size_t)R * (D + 2);  // a part: O [R][D], m [R], l [R]
    const float* first = j.parts + ((size_t)block * 2 + 1) * r.f;  // follower i at (block + i) * 2 parts
    r.o = first + (size_t)item_row * D;
    r.m = first + (size_t)R * D + item_row;
    r.l = r.m + R;
    r.n = block + followers < j.blocks ? 1 + followers : 0;
  } else {
    r.f = 0;
    r.o = sums.o + row * D;
    r.m = &sums.ml[row].x;
    r.l = &sums.ml[row].y;
    r.n = 1;
    r.permuted = many;
  }
  return r;
}

// The grid's x goes over requests, its y over their rows.  kBatch: parts whose
// loads are under way together.
template <int D, int kBatch>
__global__ void __launch_bounds__(kThreads) finish_kernel(const KvBatch batch, const KvShared shared, const KvJoin few,
                                                          const KvJoin many, __half* out, long long ldo, int q_heads,
                                                          FastDiv by_heads, int share, int page, int few_rows) {
  pdl_launch_dependents();
  pdl_wait();
  const KvRequest r = kv_request(batch, page, blockIdx.x);
  const long long n = (long long)r.q_len * q_heads * (D / 8);
  const bool own_many = r.q_len * share > few_rows, prefix_many = batch.tokens * share > few_rows;
  for (long long e = blockIdx.y * (long long)kThreads + threadIdx.x; e < n; e += (long long)gridDim.y * kThreads) {
    const int row = (int)(e / (D / 8)), ch = (int)(e % (D / 8)) * 8;
    const int t = divide(row, by_heads), head = row - t * q_heads, g = head % share;
    const size_t at = (size_t)(r.q0 + t) * q_heads + head;
    const RowParts parts[2] = {row_parts<D>(shared.own, at, t * share + g, own_many, few, many),
                               row_parts<D>(shared.prefix, at, (r.q0 + t) * share + g, prefix_many, few, many)};
    float m = -INFINITY, l = 0.f, sum[8] = {};
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      float acc[8] = {};
      // kBatch parts under way at a time, the sums moved to the greatest m so far
      for (int i0 = 0; i0 < parts[s].n; i0 += kBatch) {
        float pm[kBatch], pl[kBatch];
        float4 a[kBatch], b[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const bool on = i0 + i < parts[s].n;
          const size_t o = parts[s].at(on ? i0 + i : 0);
          pm[i] = on ? parts[s].m[o] : -INFINITY;
          pl[i] = on ? parts[s].l[o] : 0.f;
          const float4* src = reinterpret_cast<const float4*>(parts[s].o + o + ch);
          a[i] = on ? src[0] : make_float4(0.f, 0.f, 0.f, 0.f);
          b[i] = on ? src[1] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float next = m;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) next = fmaxf(next, pm[i]);
        const float moved = exp2f(m - next);  // 0 before the first
        m = next;
        l *= moved;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          acc[k] *= moved;
          sum[k] *= moved;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const float w = exp2f(pm[i] - m);
          l = fmaf(w, pl[i], l);
          const float x[8] = {a[i].x, a[i].y, a[i].z, a[i].w, b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, x[k], acc[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum[k] += parts[s].permuted ? acc[((k & 3) << 1) + (k >> 2)] : acc[k];
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;  // no key seen: zeros
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 y = __floats2half2_rn(sum[2 * k] * inv, sum[2 * k + 1] * inv);
      o[k] = *reinterpret_cast<const uint32_t*>(&y);
    }
    *reinterpret_cast<uint4*>(out + (long long)(r.q0 + t) * ldo + (long long)head * D + ch) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
}

}  // namespace

tlq_status launch_kv4_finish_shared(const KvAttention& a, int few_rows, const KvJoin& few, const KvJoin& many,
                                    cudaStream_t stream) {
  const long long most = (long long)a.batch.max_q * a.q_heads * (a.head_dim / 8);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)a.batch.requests, (unsigned)std::min<long long>((most + kThreads - 1) / kThreads, 1024), 1);
  lc.blockDim = dim3(kThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  // Rows of prompts lie in one or two parts, and there are many of them: fewer
  // registers (992 queries: 329 us with four, 341 with eight).  Single tokens' lie in
  // many: more under way (four requests: 11.2 us with eight, 11.8 with four).
  const bool prompts = (long long)a.batch.max_q * (a.q_heads / a.cache.heads) > few_rows;
  auto kernel = a.head_dim == 64 ? (prompts ? finish_kernel<64, 4> : finish_kernel<64, 8>)
                                 : (prompts ? finish_kernel<128, 4> : finish_kernel<128, 8>);
  return cuda_error(cudaLaunchKernelEx(&lc, kernel, a.batch, a.shared, few, many, a.out, a.ldo, a.q_heads,
                                       fast_div((uint32_t)a.q_heads), a.q_heads / a.cache.heads, a.cache.page, few_rows),
                    "kv4 attention finish: launch");
}

}  // namespace tlq
