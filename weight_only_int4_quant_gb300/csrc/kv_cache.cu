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
constexpr int kRowsAtOnce = 2;  // rows of a thread under way at a time (16 bytes each)

// n / d for n < 2^31 by one multiplication (d >= 1): m = ceil(2^(31 + s) / d)
// with 2^s >= d errs by less than 1 / d.
struct FastDiv {
  uint32_t d, m;
  int s;
};
FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1ull << f.s) < d) ++f.s;
  f.m = (uint32_t)(((1ull << (31 + f.s)) + d - 1) / d);
  return f;
}
__device__ __forceinline__ uint32_t divide(uint32_t n, const FastDiv& f) {
  return (uint32_t)(((uint64_t)n * f.m) >> (31 + f.s));
}

struct CodeRow {
  uint8_t* codes;
  uint32_t* par;  // (scale, minimum) pairs, one per group
};

template <int D>
__device__ __forceinline__ CodeRow code_row(const KvCache& c, long long slot, int head, int part) {
  const int P = c.page, off = (int)(slot & (P - 1));
  uint8_t* blk = c.blocks + ((slot >> c.page_shift) * c.heads + head) * (long long)c.block_bytes;
  const int half = P * D / 2, pw = c.group == D ? 4 : 8;
  CodeRow r;
  r.codes = blk + part * half + off * (D / 2);
  r.par = reinterpret_cast<uint32_t*>(blk + 2 * half + part * P * pw + off * pw);
  return r;
}

__device__ __forceinline__ bool in_cache(const KvCache& c, long long slot) {
  return slot >= 0 && slot < c.num_pages << c.page_shift;
}

// The word of eight codes rint((x - b) / s), and whether all of them are
// certain.  With inv = fp32(1 / s), t = (x - b) * inv is within 2^-22 of the
// quotient relative to it, so n = rint(t) can only differ from the rounding of
// the IEEE quotient where the remainder (x - b) - n s comes within 2^-18 s of
// half a step (t <= 15: 15 * 2^-22 < 2^-18), or past it; such words are redone
// with divisions.  x >= b always: b is one of the row's own values.
__device__ __forceinline__ bool code_word(const float (&x)[8], float s, float b, float inv, uint32_t* word) {
  const float magic = 8388608.0f;  // 2^23: adding it rounds to whole numbers, kept in the low bits
  const float limit = s * (0.5f - 3.8147e-6f);
  float far = 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = x[i] - b;
    const float r = fminf(d * inv, 15.0f) + magic;
    far = fmaxf(far, fabsf(fmaf(magic - r, s, d)));
    w |= (__float_as_uint(r) & 15u) << (4 * i);
  }
  *word = w;
  return far < limit;
}

__device__ __noinline__ uint32_t code_word_by_division(const float (&x)[8], float s, float b) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= (uint32_t)fminf(fmaxf(rintf((x[i] - b) / s), 0.0f), 15.0f) << (4 * i);
  return w;
}

// D / 8 lanes per row of D channels, 8 channels (16 bytes in, 4 out) to a
// lane; a token's heads follow one another, keys and values are the grid's y.
template <int D>
__global__ void __launch_bounds__(kRowThreads)
    append_kernel(const KvCache c, const __half* __restrict__ k, long long ldk, const __half* __restrict__ v,
                  long long ldv, const long long* __restrict__ slots, uint32_t rows, FastDiv heads) {
  constexpr int L = D / 8, U = kRowsAtOnce, RPB = kRowThreads / L;
  pdl_launch_dependents();
  pdl_wait();
  const int part = blockIdx.y;
  const __half* const base = part ? v : k;
  const long long ld = part ? ldv : ldk;
  const int sub = threadIdx.x % L;
  const int gl = c.group / 8;  // lanes of a group (8 or 16)
  // every lane of a warp takes the same number of turns (the shuffles need all)
  for (uint32_t r0 = blockIdx.x * (RPB * U); r0 < rows; r0 += gridDim.x * (RPB * U)) {
    uint4 raw[U];
    long long slot[U];
    int head[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t row = r0 + u * RPB + threadIdx.x / L;
      const bool on = row < rows;
      const uint32_t t = divide(on ? row : 0, heads);
      head[u] = on ? (int)(row - t * heads.d) : 0;
      raw[u] = on ? __ldg(reinterpret_cast<const uint4*>(base + t * ld + head[u] * D + sub * 8))
                  : make_uint4(0, 0, 0, 0);
      slot[u] = on ? __ldg(slots + t) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[8];
      const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
      __half2 lo2, hi2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
        const float2 f = __half22float2(h);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
        lo2 = i ? __hmin2(lo2, h) : h;
        hi2 = i ? __hmax2(hi2, h) : h;
      }
      for (int o = 1; o < gl; o <<= 1) {
        lo2 = __hmin2(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
        hi2 = __hmax2(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
      }
      const __half bh = __hmin(__low2half(lo2), __high2half(lo2)), th = __hmax(__low2half(hi2), __high2half(hi2));
      const __half tiny = __ushort_as_half((unsigned short)1);
      const float b = __half2float(bh);
      const __half sh = __hmax(__float2half_rn((__half2float(th) - b) / 15.0f), tiny);
      const float s = __half2float(sh);
      uint32_t word;
      if (!code_word(x, s, b, 1.0f / s, &word)) word = code_word_by_division(x, s, b);
      if (in_cache(c, slot[u])) {
        const CodeRow out = code_row<D>(c, slot[u], head[u], part);
        reinterpret_cast<uint32_t*>(out.codes)[sub] = word;
        if (sub % gl == 0)
          out.par[sub / gl] = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(bh) << 16);
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads)
    read_kernel(const KvCache c, const long long* __restrict__ slots, uint32_t rows, FastDiv heads,
                __half* __restrict__ k, __half* __restrict__ v) {
  constexpr int L = D / 8, U = kRowsAtOnce, RPB = kRowThreads / L;
  pdl_launch_dependents();
  pdl_wait();
  const int part = blockIdx.y;
  __half* const base = part ? v : k;
  const int sub = threadIdx.x % L;
  const int gl = c.group / 8;
  for (uint32_t r0 = blockIdx.x * (RPB * U); r0 < rows; r0 += gridDim.x * (RPB * U)) {
    uint32_t word[U], par[U];
    bool there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t row = r0 + u * RPB + threadIdx.x / L;
      word[u] = par[u] = 0;
      there[u] = false;
      if (row < rows) {
        const uint32_t t = divide(row, heads);
        const long long slot = __ldg(slots + t);
        there[u] = in_cache(c, slot);
        if (there[u]) {
          const CodeRow in = code_row<D>(c, slot, (int)(row - t * heads.d), part);
          word[u] = reinterpret_cast<const uint32_t*>(in.codes)[sub];
          par[u] = in.par[sub / gl];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t row = r0 + u * RPB + threadIdx.x / L;
      if (row >= rows) continue;
      const float2 sb = __half22float2(*reinterpret_cast<const __half2*>(&par[u]));
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 p = __floats2half2_rn(fmaf((float)((word[u] >> (8 * i)) & 15u), sb.x, sb.y),
                                            fmaf((float)((word[u] >> (8 * i + 4)) & 15u), sb.x, sb.y));
        h[i] = there[u] ? *reinterpret_cast<const uint32_t*>(&p) : 0u;
      }
      *reinterpret_cast<uint4*>(base + (long long)row * D + sub * 8) = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

template <class K, class... Args>
tlq_status launch_rows(K kernel, long long rows, int lanes, const char* what, cudaStream_t stream, Args... args) {
  if (rows > 0x7fffffffll) return set_error(TLQ_EUNSUPPORTED, "%s: %lld rows (tokens x heads, at most 2^31 - 1)", what, rows);
  const long long per = kRowThreads / lanes;  // a block's first turn, one row a thread group, while blocks are few
  const long long blocks = std::min<long long>((rows + per - 1) / per, (long long)device_info().sms * 4);
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
    return launch_rows(append_kernel<128>, rows, 16, "kv4 append: launch", stream, c, k, ldk, v, ldv, slots,
                       (uint32_t)rows, heads);
  return launch_rows(append_kernel<64>, rows, 8, "kv4 append: launch", stream, c, k, ldk, v, ldv, slots,
                     (uint32_t)rows, heads);
}

tlq_status launch_kv4_read(const KvCache& c, int head_dim, const long long* slots, int tokens, __half* k, __half* v,
                           cudaStream_t stream) {
  const long long rows = (long long)tokens * c.heads;
  const FastDiv heads = fast_div((uint32_t)c.heads);
  if (head_dim == 128)
    return launch_rows(read_kernel<128>, rows, 16, "kv4 read: launch", stream, c, slots, (uint32_t)rows, heads, k, v);
  return launch_rows(read_kernel<64>, rows, 8, "kv4 read: launch", stream, c, slots, (uint32_t)rows, heads, k, v);
}

}  // namespace tlq
