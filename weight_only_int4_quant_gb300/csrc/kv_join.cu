// The attention kernels cut items (a request, a key head and a set of rows) at
// the ends of their blocks' equal spans of work.  Here the parts of an item are
// put together, in the order of the blocks, so that the result is the same
// every time:  o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,  m = max m_i.
//
// A set of blocks (one for the few rows of the one kernel, kManyBlocks for the
// 256 of the other) looks at what one main block began and did not end, a
// thread to 8 channels of a row.  Latency bounds it (a part is a few hundred
// kilobytes in L2): the parts of both kernels of a mixed batch are joined by
// one launch.  8 blocks to a main block take a prompt of 2048 tokens, 16 heads, in
// 70 us, 4 in 77; a grid of 608 x 32 blocks, most with nothing to join, took 75.
// 96 registers keep the loads of four parts under way: at 64 the 14 parts
// an item of four long contexts took 9 us longer.
#include <algorithm>

#include "serve.cuh"

namespace tlq {
namespace {

constexpr int kJoinThreads = 128;
constexpr int kManyBlocks = 8;

// SHARED: a batch with a prefix, whose sums go to the rows' (their channels in
// the order of the kernel that made them) to be merged.
template <int D, bool SHARED>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const KvJoin few, const KvJoin many, __half* out,
                                                           long long ldo, int share, const KvShared shared,
                                                           int q_heads) {
  pdl_launch_dependents();
  const bool first_kind = (int)blockIdx.x < few.blocks;
  const KvJoin& j = first_kind ? few : many;
  const int at = first_kind ? blockIdx.x : blockIdx.x - few.blocks;
  const int each = first_kind ? 1 : kManyBlocks, block = at / each;
  pdl_wait();
  const KvJoinHeader h = j.headers[block];
  if (h.followers <= 0) return;
  const int R = j.rows;
  const size_t F = (size_t)R * (D + 2);  // a part: O [R][D], m [R], l [R]
  const float* first = j.parts + ((size_t)block * 2 + 1) * F;
  const float* rest = j.parts + ((size_t)block + 1) * 2 * F;  // follower i at i * 2 F
  for (int e = (at - block * each) * kJoinThreads + threadIdx.x; e < h.rows * (D / 8); e += each * kJoinThreads) {
    const int row = e / (D / 8), ch = (e - row * (D / 8)) * 8;
    float m = first[R * D + row];
    for (int i = 0; i < h.followers; ++i) m = fmaxf(m, rest[(size_t)i * 2 * F + R * D + row]);
    float l = 0.f, acc[8] = {};
#pragma unroll 4
    for (int i = -1; i < h.followers; ++i) {
      const float* part = i < 0 ? first : rest + (size_t)i * 2 * F;
      const float w = exp2f(part[R * D + row] - m);
      const float4* src = reinterpret_cast<const float4*>(part + (size_t)row * D + ch);
      const float4 a = src[0], b = src[1];
      l = fmaf(w, part[R * D + R + row], l);
      const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, x[k], acc[k]);
    }
    const int gr = h.row0 + row, t = gr / share, g = gr - t * share;
    if constexpr (SHARED) {
      const KvRowSums& to = h.prefix ? shared.prefix : shared.own;
      const size_t to_row = (size_t)(h.q0 + t) * q_heads + h.head * share + g;
      float4* dst = reinterpret_cast<float4*>(to.o + to_row * D + ch);
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (ch == 0) to.ml[to_row] = make_float2(m, l);
      continue;
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;  // no key seen: zeros
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // channels 2 k, 2 k + 1; the tensor-core kernel's parts hold 0 4 1 5 2 6 3 7
      const int c0 = 2 * k, c1 = c0 + 1, p0 = ((c0 & 3) << 1) + (c0 >> 2), p1 = ((c1 & 3) << 1) + (c1 >> 2);
      const __half2 y = first_kind ? __floats2half2_rn(acc[c0] * inv, acc[c1] * inv)
                                   : __floats2half2_rn(acc[p0] * inv, acc[p1] * inv);
      o[k] = *reinterpret_cast<const uint32_t*>(&y);
    }
    *reinterpret_cast<uint4*>(out + (long long)(h.q0 + t) * ldo + (long long)(h.head * share + g) * D + ch) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// A row of a batch with a prefix: o = (2^(m1 - m) O1 + 2^(m2 - m) O2) / (2^(m1 - m) l1
// + 2^(m2 - m) l2) of the prefix's and the request's own sums.  A thread to 8
// channels; the grid's x goes over requests, its y over their rows.
constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const KvBatch batch, const KvShared shared, __half* out,
                                                              long long ldo, int q_heads, int share, int page,
                                                              int few_rows) {
  pdl_launch_dependents();
  pdl_wait();
  const KvRequest r = kv_request(batch, page, blockIdx.x);
  const long long n = (long long)r.q_len * q_heads * (D / 8);
  const bool own_many = r.q_len * share > few_rows, prefix_many = batch.tokens * share > few_rows;
  for (long long e = blockIdx.y * (long long)kMergeThreads + threadIdx.x; e < n; e += (long long)gridDim.y * kMergeThreads) {
    const long long row = e / (D / 8);
    const int ch = (int)(e - row * (D / 8)) * 8;
    const size_t at = (size_t)r.q0 * q_heads + row;
    const float2 a = shared.own.ml[at], b = shared.prefix.ml[at];
    float x[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4* src = reinterpret_cast<const float4*>((i ? shared.prefix.o : shared.own.o) + at * D + ch);
      const float4 u = src[0], v = src[1];
      const float raw[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
      // the tensor-core kernel's channels lie as 0 4 1 5 2 6 3 7
      const bool many = i ? prefix_many : own_many;
#pragma unroll
      for (int k = 0; k < 8; ++k) x[i][k] = many ? raw[((k & 3) << 1) + (k >> 2)] : raw[k];
    }
    const float m = fmaxf(a.x, b.x), wa = exp2f(a.x - m), wb = exp2f(b.x - m);
    const float l = wa * a.y + wb * b.y, inv = l == 0.f ? 0.f : 1.0f / l;  // no key seen: zeros
    uint32_t o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 y = __floats2half2_rn((wa * x[0][2 * k] + wb * x[1][2 * k]) * inv,
                                          (wa * x[0][2 * k + 1] + wb * x[1][2 * k + 1]) * inv);
      o[k] = *reinterpret_cast<const uint32_t*>(&y);
    }
    const long long t = row / q_heads;
    *reinterpret_cast<uint4*>(out + (r.q0 + t) * ldo + (row - t * q_heads) * D + ch) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <bool SHARED>
tlq_status launch_join(const KvAttention& a, const KvJoin& few, const KvJoin& many, cudaStream_t stream) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(few.blocks + many.blocks * kManyBlocks), 1, 1);
  lc.blockDim = dim3(kJoinThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  const int share = a.q_heads / a.cache.heads;
  auto kernel = a.head_dim == 64 ? join_kernel<64, SHARED> : join_kernel<128, SHARED>;
  return cuda_error(cudaLaunchKernelEx(&lc, kernel, few, many, a.out, a.ldo, share, a.shared, a.q_heads),
                    "kv4 attention join: launch");
}

}  // namespace

tlq_status launch_kv4_join(const KvAttention& a, const KvJoin& few, const KvJoin& many, cudaStream_t stream) {
  return launch_join<false>(a, few, many, stream);
}

tlq_status launch_kv4_join_shared(const KvAttention& a, const KvJoin& few, const KvJoin& many, cudaStream_t stream) {
  return launch_join<true>(a, few, many, stream);
}

tlq_status launch_kv4_merge(const KvAttention& a, int few_rows, cudaStream_t stream) {
  const long long most = (long long)a.batch.max_q * a.q_heads * (a.head_dim / 8);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)a.batch.requests, (unsigned)std::min<long long>((most + kMergeThreads - 1) / kMergeThreads, 1024), 1);
  lc.blockDim = dim3(kMergeThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  const int share = a.q_heads / a.cache.heads;
  auto kernel = a.head_dim == 64 ? merge_kernel<64> : merge_kernel<128>;
  return cuda_error(cudaLaunchKernelEx(&lc, kernel, a.batch, a.shared, a.out, a.ldo, a.q_heads, share, a.cache.page,
                                       few_rows),
                    "kv4 attention merge: launch");
}

}  // namespace tlq
