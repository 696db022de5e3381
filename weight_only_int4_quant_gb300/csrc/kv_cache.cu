// Writing and reading the paged 4-bit cache.
//
// A row of `group` channels x of one token and head becomes
//   b = fp16(min x), s = max(fp16((max x - min x) / 15), 2^-24)
//   c = clamp(rint((x - b) / s), 0, 15)
// (binary32, rounded to nearest even at every step) and stands for c * s + b.
// The smallest FP16 number as the least scale keeps constant rows exact
// (c = 0) and every scale's logarithm finite for the attention kernels.  Where
// an x is not finite, s is not either: s and b are stored as NaN and the whole
// group stands for NaN (no infinity reaches the attention kernels' sums).
//
// DRAM traffic is the floor of both kernels (2.5 bytes a value and a group's
// parameters, one pass): 16 channels a lane, a row's lanes side by side, the
// next row asked for before the current one's arithmetic, stores of whole
// sectors.  Writing is bound by issue (a rounding, a check of it and a shift per
// code), reading by outstanding loads.  16001 tokens x 16 heads of 128, keys and
// values, groups of 64 (168 MB each way): append 42.5 us (4.0 TB/s; 46 without
// the row ahead), read 32.8 us (5.1 TB/s; 35.8 with 4 and 35.3 with 8 blocks to
// an SM for 6).  Few tokens are bound by latency: 16 tokens take 2.1 us each way.
#include <algorithm>

#include "kv_codes.cuh"

namespace tlq {
namespace {

constexpr int kRowThreads = 256;
constexpr int kAppendBlocks = 4, kReadBlocks = 6;  // resident to an SM (registers)

// D / 16 lanes per row of D channels, 16 channels (32 bytes in, 8 out) to a
// lane, GL lanes to a group; a token's heads follow one another, keys and
// values are the grid's y.
template <int D, int GL>
__global__ void __launch_bounds__(kRowThreads, kAppendBlocks)
    append_kernel(const KvCache c, const __half* __restrict__ k, long long ldk, const __half* __restrict__ v,
                  long long ldv, const long long* __restrict__ slots, uint32_t rows, FastDiv heads) {
  constexpr int L = D / 16, RPB = kRowThreads / L;
  pdl_launch_dependents();
  pdl_wait();
  const int part = blockIdx.y;
  const __half* const base = part ? v : k;
  const long long ld = part ? ldv : ldk;
  const int sub = threadIdx.x % L;
  // Every lane of a warp takes the same number of turns (the shuffles need all);
  // lanes past the end do the last row again.  A row is asked for a turn ahead.
  uint4 raw[2];
  long long slot;
  auto fetch = [&](uint32_t r0) {
    const uint32_t row = min(r0 + threadIdx.x / L, rows - 1);
    const uint32_t t = (uint32_t)divide((int)row, heads);
    const uint4* src = reinterpret_cast<const uint4*>(base + t * ld + (int)(row - t * heads.d) * D + sub * 16);
    raw[0] = __ldg(src);
    raw[1] = __ldg(src + 1);
    slot = __ldg(slots + t);
  };
  uint32_t r0 = blockIdx.x * RPB;
  if (r0 < rows) fetch(r0);
  for (; r0 < rows; r0 += gridDim.x * RPB) {
    const uint32_t row = min(r0 + threadIdx.x / L, rows - 1);
    const int head = (int)(row - (uint32_t)divide((int)row, heads) * heads.d);
    const long long here = slot;
    append_row<D, GL>(c, raw, true, here, head, part, sub,
                      [&]() { if (rows - r0 > gridDim.x * RPB) fetch(r0 + gridDim.x * RPB); });
  }
}

template <int D, int GL>
__global__ void __launch_bounds__(kRowThreads, kReadBlocks)
    read_kernel(const KvCache c, const long long* __restrict__ slots, uint32_t rows, FastDiv heads,
                __half* __restrict__ k, __half* __restrict__ v) {
  constexpr int L = D / 16, U = 2, RPB = kRowThreads / L;  // U rows of a thread under way at a time
  pdl_launch_dependents();
  pdl_wait();
  const int part = blockIdx.y;
  __half* const base = part ? v : k;
  const int sub = threadIdx.x % L;
  for (uint32_t r0 = blockIdx.x * (RPB * U); r0 < rows; r0 += gridDim.x * (RPB * U)) {
    uint2 word[U];
    uint32_t par[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t row = min(r0 + u * RPB + threadIdx.x / L, rows - 1);
      const uint32_t t = (uint32_t)divide((int)row, heads);
      const long long slot = __ldg(slots + t);
      word[u] = make_uint2(0, 0);
      par[u] = 0;  // scale and minimum 0: zeros
      if (in_cache(c, slot)) {
        const CodeRow in = code_row<D>(c, slot, (int)(row - t * heads.d), part);
        word[u] = reinterpret_cast<const uint2*>(in.codes)[sub];
        par[u] = in.par[sub / GL];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t row = r0 + u * RPB + threadIdx.x / L;
      const float2 sb = __half22float2(*reinterpret_cast<const __half2*>(&par[u]));
      const float2 s2 = make_float2(sb.x, sb.x);
      // 2^23 + code, from the bits; the constant goes out again exactly: the
      // code itself, then one FMA
      uint32_t h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w = (i < 4 ? word[u].x : word[u].y) >> (8 * (i & 3));
        const float2 q = add2(make_float2(__uint_as_float(0x4B000000u | (w & 15u)),
                                          __uint_as_float(0x4B000000u | ((w >> 4) & 15u))),
                              make_float2(-8388608.0f, -8388608.0f));
        const float2 f = fma2(q, s2, make_float2(sb.y, sb.y));
        const __half2 p = __floats2half2_rn(f.x, f.y);
        h[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
      // Two neighbours' 64 bytes go out as two stores of whole 32-byte sectors:
      // first the even lane's, a half from each lane, then the odd one's.
      const bool odd = sub & 1;
      uint32_t got[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) got[i] = __shfl_xor_sync(0xffffffffu, odd ? h[i] : h[i + 4], 1);
      if (row < rows) {
        uint4* dst = reinterpret_cast<uint4*>(base + (long long)row * D + (sub & ~1) * 16 + (odd ? 8 : 0));
        dst[0] = odd ? make_uint4(got[0], got[1], got[2], got[3]) : make_uint4(h[0], h[1], h[2], h[3]);
        dst[2] = odd ? make_uint4(h[4], h[5], h[6], h[7]) : make_uint4(got[0], got[1], got[2], got[3]);
      }
    }
  }
}

template <class K, class... Args>
tlq_status launch_rows(K kernel, int resident, long long rows, int lanes, const char* what, cudaStream_t stream,
                       Args... args) {
  if (rows > 0x7fffffffll)
    return set_error(TLQ_EUNSUPPORTED, "%s: %lld rows (tokens x heads, at most 2^31 - 1)", what, rows);
  const long long per = kRowThreads / lanes;  // a block's first turn, one row a thread group, while blocks are few
  // at most one wave of `resident` blocks to an SM, keys and values together
  const long long blocks = std::min<long long>((rows + per - 1) / per, (long long)device_info().sms * resident / 2);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)std::max<long long>(blocks, 1), 2, 1);
  lc.blockDim = dim3(kRowThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  return cuda_error(cudaLaunchKernelEx(&lc, kernel, args...), what);
}

}  // namespace

tlq_status launch_kv4_append(const KvCache& c, int head_dim, const __half* k, long long ldk, const __half* v,
                             long long ldv, const long long* slots, int tokens, cudaStream_t stream) {
  const long long rows = (long long)tokens * c.heads;
  const FastDiv heads = fast_div((uint32_t)c.heads);
  if (head_dim == 128)
    return launch_rows(c.group == 64 ? append_kernel<128, 4> : append_kernel<128, 8>, kAppendBlocks, rows, 8,
                       "kv4 append: launch", stream, c, k, ldk, v, ldv, slots, (uint32_t)rows, heads);
  return launch_rows(append_kernel<64, 4>, kAppendBlocks, rows, 4, "kv4 append: launch", stream, c, k, ldk, v, ldv, slots,
                     (uint32_t)rows, heads);
}

tlq_status launch_kv4_read(const KvCache& c, int head_dim, const long long* slots, int tokens, __half* k, __half* v,
                           cudaStream_t stream) {
  const long long rows = (long long)tokens * c.heads;
  const FastDiv heads = fast_div((uint32_t)c.heads);
  if (head_dim == 128)
    return launch_rows(c.group == 64 ? read_kernel<128, 4> : read_kernel<128, 8>, kReadBlocks, rows, 8,
                       "kv4 read: launch", stream, c, slots, (uint32_t)rows, heads, k, v);
  return launch_rows(read_kernel<64, 4>, kReadBlocks, rows, 4, "kv4 read: launch", stream, c, slots, (uint32_t)rows,
                     heads, k, v);
}

}  // namespace tlq
