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
#include "serve.cuh"

namespace tlq {
namespace {

constexpr int kJoinThreads = 128;
constexpr int kManyBlocks = 8;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const KvJoin few, const KvJoin many, __half* out,
                                                           long long ldo, int share) {
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
    const float inv = l == 0.f ? 0.f : 1.0f / l;  // no key seen: zeros
    const int gr = h.row0 + row, t = gr / share, g = gr - t * share;
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

}  // namespace

tlq_status launch_kv4_join(const KvAttention& a, const KvJoin& few, const KvJoin& many, cudaStream_t stream) {
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
  return cuda_error(a.head_dim == 64 ? cudaLaunchKernelEx(&lc, join_kernel<64>, few, many, a.out, a.ldo, share)
                                     : cudaLaunchKernelEx(&lc, join_kernel<128>, few, many, a.out, a.ldo, share),
                    "kv4 attention join: launch");
}

}  // namespace tlq
