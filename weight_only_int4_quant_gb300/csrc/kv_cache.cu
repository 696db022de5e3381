// Writing and reading the paged 4-bit cache.
//
// A row of `group` channels x of one token and head becomes
//   b = fp16(min x), s = max(fp16((max x - min x) / 15), 2^-24)
//   c = clamp(rint((x - b) / s), 0, 15)
// (binary32, rounded to nearest even at every step) and stands for c * s + b.
// The smallest FP16 number as the least scale keeps constant rows exact
// (c = 0) and every scale's logarithm finite for the attention kernels.
//
// DRAM traffic bounds both kernels: 16 bytes of activations against 4 bytes of
// codes per thread, one pass, a row's lanes side by side so that loads and
// stores cover whole sectors.
#include <algorithm>

#include "serve.cuh"

namespace tlq {
namespace {

constexpr int kRowThreads = 256;

struct CodeRow {
  uint8_t* codes;
  uint32_t* par;  // (scale, minimum) pairs, one per group
};

__device__ __forceinline__ CodeRow code_row(const KvCache& c, int head_dim, long long slot, int head, int part) {
  const int P = c.page, off = (int)(slot & (P - 1));
  uint8_t* blk = c.blocks + ((slot >> c.page_shift) * c.heads + head) * (long long)c.block_bytes;
  const int half = P * head_dim / 2, pw = 4 * (head_dim / c.group);
  CodeRow r;
  r.codes = blk + part * half + off * (head_dim / 2);
  r.par = reinterpret_cast<uint32_t*>(blk + 2 * half + part * P * pw + off * pw);
  return r;
}

// D / 8 lanes per row of D channels; rows are (token, key or value, head) with
// the head fastest, so that neighbouring rows of one token read on.
template <int D>
__global__ void __launch_bounds__(kRowThreads)
    append_kernel(const KvCache c, const __half* __restrict__ k, long long ldk, const __half* __restrict__ v,
                  long long ldv, const long long* __restrict__ slots, int tokens) {
  constexpr int L = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const long long rows = (long long)tokens * c.heads * 2;
  const int sub = threadIdx.x % L;
  const int gl = c.group / 8;  // lanes of a group (8 or 16)
  const long long step = (long long)gridDim.x * (kRowThreads / L);
  // every lane of a warp takes the same number of turns (the shuffles need all)
  for (long long r0 = (long long)blockIdx.x * (kRowThreads / L); r0 < rows; r0 += step) {
    const long long row = r0 + threadIdx.x / L;
    const bool on = row < rows;
    const long long t = on ? row / (2 * c.heads) : 0;
    const int rest = on ? (int)(row - t * 2 * c.heads) : 0;
    const int part = rest >= c.heads ? 1 : 0, head = rest - part * c.heads;
    const __half* src = (part ? v + t * ldv : k + t * ldk) + head * D + sub * 8;
    const uint4 raw = on ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
    const long long slot = on ? slots[t] : -1;
    float x[8];
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
    }
    for (int o = 1; o < gl; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const __half tiny = __ushort_as_half((unsigned short)1);
    const __half sh = __hmax(__float2half_rn((hi - lo) / 15.0f), tiny);
    const __half bh = __float2half_rn(lo);
    const float s = __half2float(sh), b = __half2float(bh);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = fminf(fmaxf(rintf((x[i] - b) / s), 0.0f), 15.0f);
      word |= (uint32_t)q << (4 * i);
    }
    if (slot >= 0 && slot < c.num_pages << c.page_shift) {
      const CodeRow out = code_row(c, D, slot, head, part);
      reinterpret_cast<uint32_t*>(out.codes)[sub] = word;
      if (sub % gl == 0)
        out.par[sub / gl] = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(bh) << 16);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads)
    read_kernel(const KvCache c, const long long* __restrict__ slots, int tokens, __half* __restrict__ k,
                __half* __restrict__ v) {
  constexpr int L = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const long long rows = (long long)tokens * c.heads * 2;
  const int sub = threadIdx.x % L;
  const int gl = c.group / 8;
  for (long long row = (long long)blockIdx.x * (kRowThreads / L) + threadIdx.x / L; row < rows;
       row += (long long)gridDim.x * (kRowThreads / L)) {
    const long long t = row / (2 * c.heads);
    const int rest = (int)(row - t * 2 * c.heads);
    const int part = rest >= c.heads ? 1 : 0, head = rest - part * c.heads;
    const long long slot = slots[t];
    uint32_t h[4] = {0, 0, 0, 0};
    if (slot >= 0 && slot < c.num_pages << c.page_shift) {
      const CodeRow in = code_row(c, D, slot, head, part);
      const uint32_t word = reinterpret_cast<const uint32_t*>(in.codes)[sub];
      const uint32_t par = in.par[sub / gl];
      const float2 sb = __half22float2(*reinterpret_cast<const __half2*>(&par));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 p = __floats2half2_rn(fmaf((float)((word >> (8 * i)) & 15u), sb.x, sb.y),
                                            fmaf((float)((word >> (8 * i + 4)) & 15u), sb.x, sb.y));
        h[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
    __half* dst = (part ? v : k) + (t * c.heads + head) * D + sub * 8;
    *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
  }
}

template <class K, class... Args>
tlq_status launch_rows(K kernel, long long rows, int lanes, const char* what, cudaStream_t stream, Args... args) {
  const long long per = kRowThreads / lanes;
  const long long blocks = std::min<long long>((rows + per - 1) / per, (long long)device_info().sms * 8);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)std::max<long long>(blocks, 1), 1, 1);
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
  const long long rows = 2ll * tokens * c.heads;
  if (head_dim == 128)
    return launch_rows(append_kernel<128>, rows, 16, "kv4 append: launch", stream, c, k, ldk, v, ldv, slots, tokens);
  return launch_rows(append_kernel<64>, rows, 8, "kv4 append: launch", stream, c, k, ldk, v, ldv, slots, tokens);
}

tlq_status launch_kv4_read(const KvCache& c, int head_dim, const long long* slots, int tokens, __half* k, __half* v,
                           cudaStream_t stream) {
  const long long rows = 2ll * tokens * c.heads;
  if (head_dim == 128)
    return launch_rows(read_kernel<128>, rows, 16, "kv4 read: launch", stream, c, slots, tokens, k, v);
  return launch_rows(read_kernel<64>, rows, 8, "kv4 read: launch", stream, c, slots, tokens, k, v);
}

}  // namespace tlq
