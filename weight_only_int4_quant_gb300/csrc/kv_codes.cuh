// Rows of the paged 4-bit cache and the rounding of values to their codes, the
// same for every kernel that writes the cache.
#pragma once

#include "serve.cuh"

namespace tlq {

struct CodeRow {
  uint8_t* codes;
  uint32_t* par;  // (scale, minimum) pairs, one per group
};

template <int D>
__device__ __forceinline__ CodeRow code_row(const KvCache& c, long long slot, int head, int part) {
  const int P = c.page, off = (int)(slot & (P - 1));
  uint8_t* blk = c.blocks + ((uint32_t)(slot >> c.page_shift) * (uint32_t)c.heads + (uint32_t)head) * (uint64_t)c.block_bytes;
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
// certain.  inv is 1 / s to one unit in the last place and the product is
// rounded once, to a whole number n, by adding 2^23; so n - 1/2 <= t <= n + 1/2
// for a t within 15 * 2^-23 < 2^-19 of the true quotient.  n is the rounding of
// the IEEE quotient unless the remainder (x - b) - n s comes within 2^-18 s of
// half a step; such words, and rows whose top passes the last level (scales
// near 2^-24), or with a NaN or an infinity, are redone with divisions.  x >= b
// always: b is one of the row's own values.  The whole numbers' bits are 0x4B000000 + n: shifted together
// they leave a known constant on top of the codes.
__device__ __forceinline__ bool code_word(const float2 (&x)[4], float s, float b, float inv, uint32_t* word) {
  const float2 magic = make_float2(8388608.0f, 8388608.0f);
  const float2 neg_b = make_float2(-b, -b), inv2 = make_float2(inv, inv), s2 = make_float2(s, s);
  float far = 0.f;
  uint32_t w = 0, constant = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const float2 d = add2(x[i], neg_b);
    const float2 r = fma2(d, inv2, magic);
    const float2 e = fma2(fma2(r, make_float2(-1.0f, -1.0f), magic), s2, d);
    far = fmaxf(far, fmaxf(fabsf(e.x), fabsf(e.y)));
    w = (((w << 4) + __float_as_uint(r.y)) << 4) + __float_as_uint(r.x);
    constant = (((constant << 4) + 0x4B000000u) << 4) + 0x4B000000u;
  }
  *word = w - constant;
  return far < s * (0.5f - 3.8147e-6f);
}

__device__ __forceinline__ uint32_t code_word_by_divisions(float4 lo, float4 hi, float s, float b) {
  const float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= (uint32_t)fminf(fmaxf(rintf((x[i] - b) / s), 0.0f), 15.0f) << (4 * i);
  return w;
}
// The same as a call, where it would crowd out the code around it.
static __device__ __noinline__ uint32_t code_word_by_division(float4 lo, float4 hi, float s, float b) {
  return code_word_by_divisions(lo, hi, s, b);
}

// x / 15 as IEEE division gives it: a correctly rounded reciprocal, the
// product's remainder by FMA and one correction (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990).
__device__ __forceinline__ float fifteenth(float x) {
  const float inv = 1.0f / 15.0f;
  const float q = x * inv;
  return fmaf(fmaf(-15.0f, q, x), inv, q);
}

__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// An FP16 group's (scale, minimum) as the cache holds them, from its least and
// its greatest value: NaN for both where one of its values is not finite.
struct GroupScale {
  float s, b, top, inv;
  uint32_t pair;
};
__device__ __forceinline__ GroupScale group_scale(__half low, __half high) {
  GroupScale g;
  g.b = __half2float(low);
  g.top = __half2float(high);
  const __half sh = __hmax_nan(__float2half_rn(fifteenth(g.top - g.b)), __ushort_as_half((unsigned short)1));
  g.s = __half2float(sh);
  g.inv = reciprocal(g.s);
  g.pair = g.s < INFINITY ? (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(low) << 16) : 0x7FFF7FFFu;
  return g;
}

// A row's piece of 16 channels, one of D / 16 lanes side by side (GL to a group):
// codes and parameters into the row's slot, unless `put` is false or the slot is
// outside the cache.  All lanes of a warp take part.  next() is called once the
// row is in registers.
template <int D, int GL, class F>
__device__ __forceinline__ void append_row(const KvCache& c, const uint4 (&raw)[2], bool put, long long slot, int head,
                                           int part, int sub, F next) {
  float2 x[8];
  __half2 lo2, hi2;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4& q = raw[i >> 2];
    const uint32_t w = (i & 2) ? ((i & 1) ? q.w : q.z) : ((i & 1) ? q.y : q.x);
    const __half2 h = *reinterpret_cast<const __half2*>(&w);
    x[i] = __half22float2(h);
    lo2 = i ? __hmin2_nan(lo2, h) : h;
    hi2 = i ? __hmax2_nan(hi2, h) : h;
  }
  next();
#pragma unroll
  for (int o = 1; o < GL; o <<= 1) {
    lo2 = __hmin2_nan(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
    hi2 = __hmax2_nan(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
  }
  const GroupScale g = group_scale(__hmin_nan(__low2half(lo2), __high2half(lo2)),
                                   __hmax_nan(__low2half(hi2), __high2half(hi2)));
  uint32_t word[2];
  const float2 x0[4] = {x[0], x[1], x[2], x[3]}, x1[4] = {x[4], x[5], x[6], x[7]};
  const bool sure0 = code_word(x0, g.s, g.b, g.inv, &word[0]), sure1 = code_word(x1, g.s, g.b, g.inv, &word[1]);
  if (!(sure0 && sure1 && (g.top - g.b) * g.inv < 15.25f)) {
    word[0] = code_word_by_division(make_float4(x[0].x, x[0].y, x[1].x, x[1].y),
                                    make_float4(x[2].x, x[2].y, x[3].x, x[3].y), g.s, g.b);
    word[1] = code_word_by_division(make_float4(x[4].x, x[4].y, x[5].x, x[5].y),
                                    make_float4(x[6].x, x[6].y, x[7].x, x[7].y), g.s, g.b);
  }
  if (put && in_cache(c, slot)) {
    const CodeRow out = code_row<D>(c, slot, head, part);
    reinterpret_cast<uint2*>(out.codes)[sub] = make_uint2(word[0], word[1]);
    if (sub % GL == 0) out.par[sub / GL] = g.pair;
  }
}

}  // namespace tlq
