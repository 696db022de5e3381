// Norms of query and key heads with their rotation by position, and the same on
// the way into the paged 4-bit cache.
//
//   r = 1 / sqrt(sum x^2 / D + eps),  y = (x r) w
//   pair i of (a, b), (c, s) = table[position on i's axis][i]:
//   a' = a c - b s,  b' = b c + a s
// FP32, every operation rounded by itself (no contraction), and the squares are
// summed as a tree that the lanes' layout does not change (chunks of 8 channels
// by halves, then the chunks by halves; squares of FP16 are exact), so results
// are defined to the bit and a key quantized on the way gives the codes that it
// gives when it is written out and appended.
//
// Memory traffic is the floor: 2 bytes in and 2 out of a value (half a byte out
// into the cache).  A row of D channels is D / 16 lanes with two chunks of 8
// each.  Of a pair's channels both lie in one lane: for halves (i, i + rot / 2)
// lane l holds chunks l and l + rot / 16, for neighbours 2 l and 2 l + 1; either
// way its pairs are 8 l .. 8 l + 7, one piece of the table's row.  A lane takes
// up to eight rows one after another, of one token where heads allow it, so that
// weights and the table's row are read once for all of them; a row is asked for
// a turn ahead.  A block's rows are all queries, all keys or all values; values go
// the way of the plain append.
//
// 8192 tokens x 40 heads of 128 take 34.2 us (5.0 TB/s, three quarters of a copy's
// rate): three blocks of 80 registers a thread to an SM keep 24 KB under way, and
// four blocks spill (43 us).  Up to 4 rows to a lane take the append of 16001 tokens,
// 32 / 8 heads, with its read from 113 us to 120, up to 16 from 111 to 115, up to 48 to
// 125.  A ring of rows in shared memory, three ahead, is 5 % faster on that prompt and
// 14 % slower on rows of 64 channels.
// Few tokens are bound by latency (position, table row, head): 16 take 2.4 us.
#include <algorithm>

#include "kv_codes.cuh"

namespace tlq {
namespace {

constexpr int kThreads = 256, kResident = 3;  // blocks of an SM (registers)

struct Part {
  const __half* x;
  long long ld;
  __half* out;  // NULL: into the cache
  long long ldo;
  const __half* weight;
  uint32_t rows;  // tokens * heads
  uint32_t blocks;
  FastDiv heads;
};

struct RopeParams {
  RopeTable rope;
  const int* positions;
  long long ld_positions;
  Part part[3];  // queries, keys, values
  float eps, inv_d;
  float one;  // 1: a sum as one * a + b is not joined with the products before it to one rounding
  KvCache cache;
  const long long* slots;
  int turns;  // rows of a lane
};

// Lane l's two chunks.
template <int D>
__device__ __forceinline__ int2 chunks_of(int l, int rot, bool neighbours) {
  const bool apart = !neighbours && l * 16 < rot;
  return apart ? make_int2(l, l + rot / 16) : make_int2(2 * l, 2 * l + 1);
}

__device__ __forceinline__ float2 half2_at(const uint4& v, int i) {
  const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The sum of a chunk's squares: channels j and j + 4, then j and j + 2, then the two.
__device__ __forceinline__ float chunk_squares(const float2 (&x)[4]) {
  const float2 a = fma2(x[2], x[2], mul2(x[0], x[0])), b = fma2(x[3], x[3], mul2(x[1], x[1]));
  const float2 c = add2(a, b);
  return __fadd_rn(c.x, c.y);
}

// cos and sin of a lane's pairs 8 l .. 8 l + 7: one piece of one row where they
// are all of one axis; NaN past the table's end.
__device__ __forceinline__ void turn_of(const RopeTable& r, int l, const int (&at)[3], float2 (&co)[4], float2 (&si)[4]) {
  const int half = r.rot / 2, first = 8 * l, last = first + 7;
  auto axis = [&](int pair) { return pair < r.end0 ? at[0] : pair < r.end1 ? at[1] : at[2]; };
  if ((last < r.end0) | (first >= r.end0 && last < r.end1) | (first >= r.end1)) {
    const int pos = axis(first);
    if (pos < r.positions) {
      const float4* src = reinterpret_cast<const float4*>(r.table + (long long)pos * half + first);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 v = __ldg(src + j);
        co[j] = make_float2(v.x, v.z);
        si[j] = make_float2(v.y, v.w);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) co[j] = si[j] = make_float2(NAN, NAN);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int pos = axis(first + j);
      const float2 v = pos < r.positions ? __ldg(r.table + (long long)pos * half + first + j) : make_float2(NAN, NAN);
      (j & 1 ? co[j / 2].y : co[j / 2].x) = v.x;
      (j & 1 ? si[j / 2].y : si[j / 2].x) = v.y;
    }
  }
}

// GL: lanes of a group of the cache that keys and values go into; 0: there is none.
template <int D, int GL>
__global__ void __launch_bounds__(kThreads, kResident) rope_kernel(const RopeParams p) {
  constexpr bool CACHE = GL > 0;
  constexpr int L = D / 16;  // lanes of a row
  pdl_launch_dependents();
  pdl_wait();
  uint32_t block = blockIdx.x;
  int kind = 0;
  while (kind < 2 && block >= p.part[kind].blocks) block -= p.part[kind++].blocks;
  const Part& part = p.part[kind];
  const int l = threadIdx.x % L;
  const uint32_t first = (block * (kThreads / L) + threadIdx.x / L) * p.turns;
  const int rot = kind == 2 ? 0 : p.rope.rot;
  const bool turns = l * 16 < rot;
  const int2 ch = chunks_of<D>(l, rot, p.rope.neighbours);

  // A row is asked for a turn ahead.  Every lane of a warp takes part in all
  // shuffles: rows past the end do the last one again.
  uint4 raw[2];
  uint32_t next_t;
  auto fetch = [&](uint32_t row) {
    row = min(row, part.rows - 1);
    next_t = (uint32_t)divide((int)row, part.heads);
    const uint4* src = reinterpret_cast<const uint4*>(part.x + next_t * part.ld + (row - next_t * part.heads.d) * D);
    raw[0] = __ldg(src + ch.x);
    raw[1] = __ldg(src + ch.y);
  };
  fetch(first);
  if constexpr (CACHE) {
    if (kind == 2) {  // values: as they are
#pragma unroll 1
      for (int u = 0; u < p.turns; ++u) {
        const uint32_t t = next_t;
        const int head = (int)(min(first + u, part.rows - 1) - t * part.heads.d);
        bool there = true;
        if (p.rope.rot) {
#pragma unroll
          for (int a = 0; a < 3; ++a)
            if (a < p.rope.axes) there &= __ldg(p.positions + a * p.ld_positions + t) >= 0;
        }
        append_row<D, GL>(p.cache, raw, first + u < part.rows && there, __ldg(p.slots + t), head, 1, l,
                          [&]() { if (u + 1 < p.turns) fetch(first + u + 1); });
      }
      return;
    }
  }
  uint4 wraw[2];
  const bool normed = part.weight != nullptr;
  if (normed) {
    wraw[0] = __ldg(reinterpret_cast<const uint4*>(part.weight) + ch.x);
    wraw[1] = __ldg(reinterpret_cast<const uint4*>(part.weight) + ch.y);
  }
  float2 co[4], si[4];  // of the token at hand: pairs 2 j, 2 j + 1
  const float2 one = make_float2(p.one, p.one), minus_one = make_float2(-p.one, -p.one);
  bool there = true;
  uint32_t held = 0xffffffffu;
#pragma unroll 1
  for (int u = 0; u < p.turns; ++u) {
    const uint32_t row = min(first + u, part.rows - 1), t = next_t;
    const int head = (int)(row - t * part.heads.d);
    if (p.rope.rot && t != held) {
      held = t;
      int at[3] = {0, 0, 0};
      there = true;
#pragma unroll
      for (int a = 0; a < 3; ++a)
        if (a < p.rope.axes) {
          at[a] = __ldg(p.positions + a * p.ld_positions + t);
          there &= at[a] >= 0;
        }
      if (turns && there) turn_of(p.rope, l, at, co, si);
    }
    long long slot = -1;
    if (CACHE && part.out == nullptr) slot = __ldg(p.slots + t);
    float2 x[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[0][i] = half2_at(raw[0], i);
      x[1][i] = half2_at(raw[1], i);
    }
    if (u + 1 < p.turns) fetch(first + u + 1);
    if (normed) {
      float s0 = chunk_squares(x[0]), s1 = chunk_squares(x[1]), sum;
      if (!p.rope.neighbours && rot == D) {
        sum = __fadd_rn(s0, s1);
      } else {  // chunks l and l + L, wherever they lie
        float two[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = l + i * L;
          const bool apart = !p.rope.neighbours && c * 8 < rot;
          const int from = apart ? c % max(rot / 16, 1) : c / 2;
          const bool second = apart ? c >= rot / 16 : c & 1;
          const float a = __shfl_sync(0xffffffffu, s0, from, L), b = __shfl_sync(0xffffffffu, s1, from, L);
          two[i] = second ? b : a;
        }
        sum = __fadd_rn(two[0], two[1]);
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, o));
      const float r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(sum, p.inv_d), p.eps)));
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[k][i] = mul2(mul2(x[k][i], make_float2(r, r)), half2_at(wraw[k], i));
    }
    if (turns) {
      if (p.rope.neighbours) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = x[k][i], cj = co[2 * k + i / 2], sj = si[2 * k + i / 2];
            const float c = i & 1 ? cj.y : cj.x, n = i & 1 ? sj.y : sj.x;
            x[k][i] = fma2(mul2(make_float2(v.y, v.x), make_float2(-n, n)), one, mul2(v, make_float2(c, c)));
          }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 a = x[0][i], b = x[1][i], c = co[i], s = si[i];
          x[0][i] = fma2(mul2(b, s), minus_one, mul2(a, c));
          x[1][i] = fma2(mul2(a, s), one, mul2(b, c));
        }
      }
    }
    __half2 h[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) h[k][i] = __floats2half2_rn(x[k][i].x, x[k][i].y);
    const bool mine = first + u < part.rows && there;
    if (!CACHE || part.out != nullptr) {
      if (mine) {
        uint4* dst = reinterpret_cast<uint4*>(part.out + t * part.ldo + head * D);
#pragma unroll
        for (int k = 0; k < 2; ++k) dst[k ? ch.y : ch.x] = *reinterpret_cast<const uint4*>(h[k]);
      }
    } else if constexpr (CACHE) {
      int2 at = ch;  // the chunks at hand
      uint32_t word[2];
      GroupScale g0, g1;
      constexpr bool two = GL < L;  // groups of a row
      const bool split = two && !p.rope.neighbours && rot > 64;  // a lane's chunks are of two groups (some lanes')
      if (!split || rot == 128) {
        if (split) {
          // lanes l and l ^ 4 exchange a chunk: then each has two of one group
          const bool high = l >= 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 give = high ? h[0][i] : h[1][i];
            const __half2 got = __shfl_xor_sync(0xffffffffu, give, 4);
            h[0][i] = high ? got : h[0][i];
            h[1][i] = high ? h[1][i] : got;
          }
          at = high ? make_int2(l + 4, l + 8) : make_int2(l, l + 4);
        }
        __half2 lo2 = h[0][0], hi2 = h[0][0];
#pragma unroll
        for (int i = 1; i < 8; ++i) {
          lo2 = __hmin2_nan(lo2, h[i >> 2][i & 3]);
          hi2 = __hmax2_nan(hi2, h[i >> 2][i & 3]);
        }
#pragma unroll
        for (int o = 1; o < L; o <<= 1)
          if (o < GL) {
            lo2 = __hmin2_nan(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
            hi2 = __hmax2_nan(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
          }
        g0 = g1 = group_scale(__hmin_nan(__low2half(lo2), __high2half(lo2)), __hmax_nan(__low2half(hi2), __high2half(hi2)));
      } else {
        // least and greatest value of the row's first and second group
        const __half inf = __ushort_as_half((unsigned short)0x7C00), ninf = __ushort_as_half((unsigned short)0xFC00);
        __half2 lo2 = __half2half2(inf), hi2 = __half2half2(ninf);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const __half2 a = __hmin2_nan(__hmin2_nan(h[k][0], h[k][1]), __hmin2_nan(h[k][2], h[k][3]));
          const __half2 b = __hmax2_nan(__hmax2_nan(h[k][0], h[k][1]), __hmax2_nan(h[k][2], h[k][3]));
          const __half low = __hmin_nan(__low2half(a), __high2half(a)), high = __hmax_nan(__low2half(b), __high2half(b));
          const bool g = (k ? at.y : at.x) >> 3;
          lo2 = __hmin2_nan(lo2, g ? __halves2half2(inf, low) : __halves2half2(low, inf));
          hi2 = __hmax2_nan(hi2, g ? __halves2half2(ninf, high) : __halves2half2(high, ninf));
        }
#pragma unroll
        for (int o = 1; o < L; o <<= 1) {
          lo2 = __hmin2_nan(lo2, __shfl_xor_sync(0xffffffffu, lo2, o));
          hi2 = __hmax2_nan(hi2, __shfl_xor_sync(0xffffffffu, hi2, o));
        }
        const GroupScale a = group_scale(__low2half(lo2), __low2half(hi2)), b = group_scale(__high2half(lo2), __high2half(hi2));
        g0 = at.x >> 3 ? b : a;
        g1 = at.y >> 3 ? b : a;
      }
      bool sure = true;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const GroupScale& g = k ? g1 : g0;
        float2 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __half22float2(h[k][i]);
        sure &= code_word(y, g.s, g.b, g.inv, &word[k]) && (g.top - g.b) * g.inv < 15.25f;
      }
      if (!sure) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const GroupScale& g = k ? g1 : g0;
          const float2 a = __half22float2(h[k][0]), b = __half22float2(h[k][1]), c = __half22float2(h[k][2]),
                       d = __half22float2(h[k][3]);
          word[k] = code_word_by_divisions(make_float4(a.x, a.y, b.x, b.y), make_float4(c.x, c.y, d.x, d.y), g.s, g.b);
        }
      }
      if (mine && in_cache(p.cache, slot)) {
        const CodeRow out = code_row<D>(p.cache, slot, head, 0);
        uint32_t* codes = reinterpret_cast<uint32_t*>(out.codes);
        codes[at.x] = word[0];
        codes[at.y] = word[1];
        // a group's parameters are its first chunk's lane's to write
        if (at.x == 0) out.par[0] = g0.pair;
        if (two && at.x == 8) out.par[1] = g0.pair;
        if (two && at.y == 8) out.par[1] = g1.pair;
      }
    }
  }
}

// cos and sin of position * frequency in 64 bits, rounded once.
__global__ void table_kernel(const double* __restrict__ freq, float2* __restrict__ table, long long positions, int half,
                             double scale) {
  pdl_launch_dependents();
  pdl_wait();
  const long long n = positions * half;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
    double s, c;
    sincos((double)(i / half) * freq[i % half], &s, &c);
    table[i] = make_float2((float)(c * scale), (float)(s * scale));
  }
}

template <int D, int GL>
tlq_status launch_rows(RopeParams& p, cudaStream_t stream) {
  constexpr uint32_t groups = kThreads / (D / 16);  // rows of a block at a time
  long long rows = 0;
  for (const Part& part : p.part) rows += part.rows;
  // one turn each while they all fit the GPU at once, and up to eight
  const long long wave = (long long)device_info().sms * kResident * groups;
  p.turns = (int)std::min<long long>(8, (rows + wave - 1) / wave);
  uint32_t blocks = 0;
  for (Part& part : p.part) {
    const uint32_t per = groups * p.turns;
    part.blocks = (uint32_t)(((long long)part.rows + per - 1) / per);
    blocks += part.blocks;
  }
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(blocks, 1, 1);
  lc.blockDim = dim3(kThreads, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  return cuda_error(cudaLaunchKernelEx(&lc, rope_kernel<D, GL>, p), "rope: launch");
}

}  // namespace

tlq_status launch_rope(const RopeArgs& a, cudaStream_t stream) {
  RopeParams p{};
  p.rope = a.rope;
  p.positions = a.positions;
  p.ld_positions = a.tokens;
  const RopeRows* rows[3] = {&a.q, &a.k, &a.v};
  for (int i = 0; i < 3; ++i) {
    const long long n = (long long)a.tokens * rows[i]->heads;
    if (n > 0x7fffffffll)
      return set_error(TLQ_EUNSUPPORTED, "%s: %lld rows (tokens x heads, at most 2^31 - 1)", a.who, n);
    p.part[i] = Part{rows[i]->x, rows[i]->ld, rows[i]->out, rows[i]->ldo, rows[i]->weight, (uint32_t)n, 0,
                     fast_div((uint32_t)std::max(rows[i]->heads, 1))};
  }
  p.eps = a.eps;
  p.inv_d = 1.0f / (float)a.head_dim;
  p.one = 1.0f;
  p.cache = a.cache;
  p.slots = a.slots;
  if (a.slots != nullptr)
    return a.head_dim == 64      ? launch_rows<64, 4>(p, stream)
           : a.cache.group == 64 ? launch_rows<128, 4>(p, stream)
                                 : launch_rows<128, 8>(p, stream);
  return a.head_dim == 64    ? launch_rows<64, 0>(p, stream)
         : a.head_dim == 128 ? launch_rows<128, 0>(p, stream)
                             : launch_rows<256, 0>(p, stream);
}

tlq_status launch_rope_table(const double* freq, float* table, long long positions, int half, double scale,
                             cudaStream_t stream) {
  const long long blocks = std::min<long long>((positions * half + 255) / 256, 8ll * device_info().sms);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)blocks, 1, 1);
  lc.blockDim = dim3(256, 1, 1);
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  return cuda_error(cudaLaunchKernelEx(&lc, table_kernel, freq, reinterpret_cast<float2*>(table), positions, half, scale),
                    "rope table: launch");
}

}  // namespace tlq
