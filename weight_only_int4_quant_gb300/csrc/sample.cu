// Tokens from logits: temperature, top-k, top-p, min-p and one given uniform
// number a row.
//
//   w_i = exp((x_i - max x) / T); in the order of x falling, ties by rising index:
//   the first k; of those the shortest run with sum w >= p * (their sum); of
//   those w_i >= min_p; then the first of them, by index, whose running sum
//   passes u * (the sum)
//
// Which token that is depends on the last bits of long sums, so the weights are
// whole numbers, 2^43 for the largest, and their sums exact: the same whatever
// the order, and two rows differ only where the weights do.  A weight comes
// within about 2^-39 of its value (the exponent in two FP32 numbers: x - max
// exactly, times log2(e) / T; 2^(-j/256) from a table and a cubic for the rest),
// and then to a whole number: one of 2^-20 is good to 2^-23, one of 2^-40 to an
// eighth, in sums that are 2^43 at least.
// FP64, the plain way, would take 30 times the arithmetic's time here (2
// operations a clock and SM).
//
// A cluster of blocks takes a row, a block a piece of it that lies in shared
// memory from its first reading on (the row is read from DRAM once).
//
// top-p: one pass counts the values in bins of 1/64 octave.  The counts say about
// where the cut lies (weights as those of the bins' middles, the heaviest exactly);
// one more pass adds up the exact weights above that place and collects the values
// around it.  With the exact sums the cut is among them or not, and if it is, their
// ranking gives it.  Where it is not (flat or equal logits), the general way: bins
// with exact sums (three limbs of 15 bits, so that 32-bit atomics do), then further
// histograms over the values inside the bin that holds the cut, down to a single
// value and the index of the last that is needed.  Histograms of exact sums alone,
// the first form, took 238 us for 194 on 256 rows of 100003: shared atomics, 7
// clocks each, bound them.
// top-k, and few kept values: one block gets all that may be kept as a list.
//
// 256 rows of 100003 FP32, temperature and top-p: 166 us, 6 waves of clusters of six
// blocks.  Of 27 us of a block with 12500 values (of eight to a row) the exact
// weights (50 instructions a value, two values at a time) take 6.6, counting 4.2,
// loading 3, the rest barriers of the cluster and short phases of the block.  64 rows
// of 131072 FP16, all filters: 41 to 46 us.  One row of 32000: 10 to 15 us by its
// values, a chain of ten short phases.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "serve.cuh"

namespace cg = cooperative_groups;

namespace tlq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxBlocks = 8;        // of a cluster
constexpr int kBins = 2048;
constexpr int kOne = 43;             // the largest weight is 2^43
constexpr float kOctaves = 40.0f;    // weights below 2^-40 of it count as none
constexpr int kMaxSmem = 232448 - 1024;
static_assert(kMaxVocab / kMaxBlocks <= 1 << 17, "limbs of 15 bits of a block's values add up in 32");

// 2^(-j / 256) * 2^43, rounded: exp of -j ln 2 / 256 by its series in double.
struct PowerTable {
  uint64_t v[256];
};
constexpr double series_exp(double x) {
  double sum = 1.0, term = 1.0;
  for (int i = 1; i < 30; ++i) {
    term = term * x / i;
    sum += term;
  }
  return sum;
}
constexpr PowerTable make_powers() {
  PowerTable t{};
  for (int j = 0; j < 256; ++j)
    t.v[j] = (uint64_t)(series_exp(-0.693147180559945309417232121458 * j / 256.0) * 8796093022208.0 + 0.5);
  return t;
}
__device__ const PowerTable kPowers = make_powers();

struct SampleParams {
  const void* logits;
  long long ld;
  int vocab, piece;  // piece: values of a block
  const float *uniform, *temperature, *top_p, *min_p;
  const int* top_k;
  int* tokens;
  float* logprobs;
};

constexpr float kLn2 = 0.693147182f, kLn2Lo = -1.90465421e-9f;  // ln 2 in two FP32 numbers

// log2(e) / T in two FP32 numbers.
struct Exponent {
  float hi, lo;
};
__device__ __forceinline__ Exponent exponent_of(float t) {
  const float c = 1.44269502f, c_lo = 1.92596303e-8f;  // log2(e)
  Exponent e;
  e.hi = fminf(__fdiv_rn(c, t), 3e38f);
  e.lo = __fdiv_rn(fmaf(-e.hi, t, c) + c_lo, t);
  if (!isfinite(e.lo)) e.lo = 0.f;  // a T at the ends of FP32's range
  return e;
}

struct Row {
  float top;
  Exponent e;
};

// -h = (top - x) / T * log2(e), rounded: which bin x falls in goes by it alone.
__device__ __forceinline__ float octaves_of(const Row& r, float x) { return __fmul_rn(__fsub_rn(x, r.top), -r.e.hi); }
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it leaves a whole number's bits
constexpr int kMagicBits = 0x4B400000;
// A value's k: 256ths of an octave below the greatest; kNoStep: no weight.  64 bins
// to an octave, the last one up to kOctaves; kBins: no weight.
constexpr int kNoStep = 1 << 20;
__device__ __forceinline__ int bin_of_k(int k) { return k == kNoStep ? kBins : min(k >> 2, kBins - 1); }
__device__ __forceinline__ int first_bin(const Row& r, float x) {
  const float o = octaves_of(r, x);
  return o <= kOctaves ? min((__float_as_int(fmaf(o, 256.0f, kMagic)) - kMagicBits) >> 2, kBins - 1) : kBins;
}

// The weight in the middle of a bin, the largest being 1.
__device__ __forceinline__ float middle_of(int bin) { return exp2f(((float)bin + 0.5f) * (-1.0f / 64.0f)); }

__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

// exp((x - top) / T) * 2^43 of two values, 0 below 2^-40, and their k.  Two at
// a time: the FP32 part is in packed operations (none of them a product that
// goes into a plain sum, which the compiler would join).  The lowest bit is set
// instead of rounding the last shift, where there is one: the largest is 2^43.
__device__ __forceinline__ void weights_of(float x0, float x1, const Row& r, const uint64_t* __restrict__ powers,
                                           uint64_t (&w)[2], int (&step)[2]) {
  // x - top = d + d_lo exactly (Knuth's two-sum)
  const float2 x = make_float2(x0, x1), neg_top = pair(-r.top), minus = pair(-1.0f);
  const float2 d = add2(x, neg_top), back = fma2(x, minus, d);  // d - x
  const float2 d_lo = add2(add2(x, fma2(d, minus, back)), fma2(back, minus, neg_top));
  // -h, and the rest l:  (x - top) log2(e) / T = h + l
  const float2 e = pair(r.e.hi), nh = mul2(d, pair(-r.e.hi));
  const float2 l = fma2(d_lo, e, fma2(d, pair(r.e.lo), fma2(d, e, nh)));
  // h = -k / 256 - q
  const float2 kb = fma2(nh, pair(256.0f), pair(kMagic));
  const float2 q = fma2(add2(kb, pair(-kMagic)), pair(-1.0f / 256.0f), nh);  // exact, |q| <= 2^-9
  // z = 2^(l - q) - 1: -c1 q in two numbers, and what is below 2^-17.  In units of
  // 2^-31 the first is rounded to a whole number, all that is left to 1 / 256 of one.
  const float2 nzh = mul2(q, pair(kLn2)), rr = fma2(q, minus, l);
  float2 zl = fma2(q, pair(-kLn2), nzh);
  zl = fma2(l, pair(kLn2), fma2(q, pair(-kLn2Lo), zl));
  zl = fma2(mul2(rr, rr), fma2(rr, fma2(rr, pair(0.00961812911f), pair(0.0555041087f)), pair(0.240226507f)), zl);
  const float2 up = pair(2147483648.0f);
  const float2 a = fma2(nzh, pair(-2147483648.0f), pair(kMagic));
  const float2 rest = fma2(nzh, pair(-2147483648.0f), fma2(a, minus, pair(kMagic)));
  const float2 b = fma2(fma2(zl, up, rest), pair(256.0f), pair(kMagic));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = __float_as_int(i ? kb.y : kb.x) - kMagicBits;
    const int z = __float_as_int(i ? a.y : a.x) * 256 + __float_as_int(i ? b.y : b.x) -
                  (int)((unsigned)kMagicBits * 257u);  // units of 2^-39
    const uint64_t power = powers[k & 255];
    const uint64_t v = power + (uint64_t)(((long long)(int)(power >> 13) * z) >> 26);
    const bool some = (i ? nh.y : nh.x) <= kOctaves;
    w[i] = some ? (v >> (k >> 8)) | (uint32_t)min(k >> 8, 1) : 0;
    step[i] = some ? k : kNoStep;
  }
}

__device__ __forceinline__ uint64_t weight_of(float x, const Row& r, const uint64_t* __restrict__ powers) {
  uint64_t w[2];
  int step[2];
  weights_of(x, x, r, powers, w, step);
  return w[0];
}

// x in [0, 1) as a fraction of 2^64 (bits below that are cut off).
__device__ __forceinline__ uint64_t fraction_of(float x) {
  const uint32_t b = __float_as_uint(x);
  const uint64_t m = (uint64_t)((b & 0x7fffffu) | 0x800000u) << 40;  // x = m * 2^(e - 126) * 2^-64
  const int down = 126 - (int)(b >> 23);
  return b < 0x800000u || down > 63 ? 0 : m >> down;
}

// Order-preserving whole numbers for FP32 values (-0 as +0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kGroups = 64, kGroupBins = kBins / kGroups;
constexpr int kList = 512;  // candidates for a cut that are ranked one by one
// Beyond this many a cut by mass is looked for around its estimate: each candidate is
// compared with all others, so 420 of them take 13 us, 170 take 3, and that way takes 4
// (60 batches of all kinds: 17.1 us in the mean with 128 or 192, 17.9 with 512).
constexpr int kRanked = 192;
static_assert(kGroupBins == 32, "a lane to a bin");
static_assert(kWarps >= kMaxBlocks && kList <= kThreads, "a warp to a block, a thread to a candidate");
constexpr int kHeavyGroups = 12;  // groups whose weights are added up exactly beside the counts: 2^-6 and more

// The state of a block; other blocks of its cluster write what is marked.
struct Shared {
  uint32_t hist[kBins];                  // counts (read by others)
  uint64_t powers[256];
  uint64_t list[2][kList];               // candidates, of the cut by count and by mass (written by others)
  uint64_t local[kList];                 // this block's candidates
  uint64_t sum[kMaxBlocks], above[kMaxBlocks], heavy[kMaxBlocks];  // by block (written by others)
  float group_about[kMaxBlocks][kGroups];                          // likewise
  uint32_t merged, base[kMaxBlocks];     // candidates of the cluster (counted by others), where this block's go
  uint64_t list_mass[kList];             // their weights
  uint64_t group_mass[kMaxBlocks][kGroups];   // by block (written by others)
  uint32_t group_count[kMaxBlocks][kGroups];  // likewise
  uint64_t fine_mass[kMaxBlocks][kGroupBins];
  uint32_t fine_count[kMaxBlocks][kGroupBins];
  uint64_t mass[kMaxBlocks];                      // likewise
  uint32_t count[8], low[8], high[kMaxBlocks];    // likewise
  float top[kMaxBlocks];                          // likewise
  int top_at[8], bad[kMaxBlocks];                 // likewise
  uint64_t warp_mass[kWarps], warp_other[kWarps];
  uint32_t warp_count[kWarps];
  float warp_top[kWarps];
  int warp_at[kWarps], warp_bad[kWarps];
  // what a search has found
  int bin;
  uint32_t before_count, bin_count, offset, pushed;
  uint64_t before_mass, bin_mass;
  uint64_t cut, cut_mass;
  int found_index;                       // written by others
};

__device__ __forceinline__ float value_of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <class T>
__device__ __forceinline__ float value_of(T v);
template <>
__device__ __forceinline__ float value_of<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float value_of<__half>(__half v) {
  return __half2float(v);
}

// Exclusive sums over the block's threads.
__device__ __forceinline__ uint64_t block_scan(Shared& s, uint64_t mass) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t own = mass;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t m = __shfl_up_sync(0xffffffffu, mass, o);
    if (lane >= o) mass += m;
  }
  __syncthreads();
  if (lane == 31) s.warp_mass[warp] = mass;
  __syncthreads();
  mass -= own;
  for (int w = 0; w < warp; ++w) mass += s.warp_mass[w];
  return mass;
}

// The weights' limbs of the bins lie behind that (read by others), over the values,
// which are read from global memory again once they are needed.
constexpr size_t kFixed = (sizeof(Shared) + 15) & ~size_t(15);
constexpr size_t kLimbBytes = 3 * kBins * sizeof(uint32_t);
__device__ __forceinline__ uint32_t* limbs_of(Shared& s, int limb) {
  return reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(&s) + kFixed) + limb * kBins;
}

// Inclusive sums over a warp.
__device__ __forceinline__ void warp_scan(uint64_t& m, uint32_t& c) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, m, o);
    const uint32_t y = __shfl_up_sync(0xffffffffu, c, o);
    if ((threadIdx.x & 31) >= o) {
      m += x;
      c += y;
    }
  }
}

// The bin in which the running count reaches want_count or, with `counting`
// false, the running mass reaches want_mass: from the blocks' sums of 32 bins
// each, then those bins themselves, which a warp for each block fetches.  Every
// warp goes through the sums by itself; one barrier.  The values before the
// histogram's are in s.before_*.  s.bin is -1 where all bins stay below.
__device__ __forceinline__ void find_bin(Shared& s, cg::cluster_group& cluster, int C, int rank, bool with_mass,
                                         bool counting, uint32_t want_count, uint64_t want_mass) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t m[2] = {0, 0};
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int o = 0; o < kMaxBlocks; ++o)
    if (o < C) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        c[j] += s.group_count[o][2 * lane + j];
        if (with_mass) m[j] += s.group_mass[o][2 * lane + j];
      }
    }
  uint64_t pm = m[0] + m[1], base_m = s.before_mass;
  uint32_t pc = c[0] + c[1], base_c = s.before_count;
  warp_scan(pm, pc);
  const uint32_t hit = __ballot_sync(0xffffffffu, counting ? base_c + pc >= want_count : base_m + pm >= want_mass);
  int first = -1;
  if (hit) {
    const int from = __ffs(hit) - 1;
    base_m += __shfl_sync(0xffffffffu, pm - m[0] - m[1], from);
    base_c += __shfl_sync(0xffffffffu, pc - c[0] - c[1], from);
    const uint64_t m0 = __shfl_sync(0xffffffffu, m[0], from);
    const uint32_t c0 = __shfl_sync(0xffffffffu, c[0], from);
    const bool second = counting ? base_c + c0 < want_count : base_m + m0 < want_mass;
    if (second) {
      base_m += m0;
      base_c += c0;
    }
    first = (2 * from + (second ? 1 : 0)) * kGroupBins;
    if (warp < C) {
      Shared& of = *cluster.map_shared_rank(&s, warp);
      const uint32_t n = of.hist[first + lane];
      uint64_t x = 0;
      if (with_mass)
        x = limbs_of(of, 0)[first + lane] + ((uint64_t)limbs_of(of, 1)[first + lane] << 15) +
            ((uint64_t)limbs_of(of, 2)[first + lane] << 30);
      s.fine_count[warp][lane] = n;
      s.fine_mass[warp][lane] = x;
    }
  }
  __syncthreads();
  if (warp == 0) {
    uint64_t bm = 0;
    uint32_t bc = 0, offset = 0;
#pragma unroll
    for (int o = 0; o < kMaxBlocks; ++o)
      if (o < C) {
        if (o < rank) offset += s.fine_count[o][lane];
        bc += s.fine_count[o][lane];
        bm += s.fine_mass[o][lane];
      }
    pm = bm;
    pc = bc;
    warp_scan(pm, pc);
    const uint32_t there = __ballot_sync(0xffffffffu, counting ? base_c + pc >= want_count : base_m + pm >= want_mass);
    if (first < 0) {
      if (lane == 0) s.bin = -1;
    } else if (lane == __ffs(there) - 1) {
      s.bin = first + lane;
      s.before_mass = base_m + pm - bm;
      s.before_count = base_c + pc - bc;
      s.bin_mass = bm;
      s.bin_count = bc;
      s.offset = offset;
      s.pushed = 0;
    }
  }
  __syncthreads();
}

// Sums over the block of up to two numbers; every thread gets them.
__device__ __forceinline__ void block_sums(Shared& s, uint64_t& a, uint64_t& b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    s.warp_mass[threadIdx.x >> 5] = a;
    s.warp_other[threadIdx.x >> 5] = b;
  }
  __syncthreads();
  a = b = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    a += s.warp_mass[w];
    b += s.warp_other[w];
  }
}

// ceil(p * mass), of at least one value.
__device__ __forceinline__ uint64_t share_of(float p, uint64_t mass) {
  const uint64_t frac = fraction_of(fmaxf(p, 0.f));
  return max(1ull, (unsigned long long)(__umul64hi(frac, mass) + (frac * mass != 0)));
}

// About where the mass reaches p of the whole, from the counts: weights count as
// those of their bins' middles, the heaviest groups' exactly.  The same in every
// block.  upto: values of that bin's group, those before it and the next that has any
// after it; end: the k there.
struct About {
  int low, high;  // the k to look at (low > high: too many values lie there)
  int end;
  uint32_t upto;
};
__device__ __forceinline__ About find_about(Shared& s, cg::cluster_group& cluster, int C, float p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float a[2] = {0.f, 0.f};
  uint32_t c[2] = {0, 0};
  uint64_t heavy = 0;
#pragma unroll
  for (int o = 0; o < kMaxBlocks; ++o)
    if (o < C) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        a[j] += s.group_about[o][2 * lane + j];
        c[j] += s.group_count[o][2 * lane + j];
      }
      heavy += s.heavy[o];
    }
  // the exact sum of the heavy groups in the place of the estimate
  float estimate = lane < kHeavyGroups / 2 ? a[0] + a[1] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) estimate += __shfl_xor_sync(0xffffffffu, estimate, o);
  if (lane < kHeavyGroups / 2) {
    const float f = (float)heavy * 1.13686838e-13f / estimate;  // 2^-43; the largest value is among them
    a[0] *= f;
    a[1] *= f;
  }
  float sum = a[0] + a[1];
  uint32_t count = c[0] + c[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, sum, o);
    const uint32_t y = __shfl_up_sync(0xffffffffu, count, o);
    if (lane >= o) {
      sum += x;
      count += y;
    }
  }
  const float want = p * __shfl_sync(0xffffffffu, sum, 31);
  const uint32_t hit = __ballot_sync(0xffffffffu, sum >= want) | 0x80000000u;
  const int from = __ffs(hit) - 1;
  const float before = __shfl_sync(0xffffffffu, sum - a[0] - a[1], from), first = __shfl_sync(0xffffffffu, a[0], from);
  const bool second = before + first < want;
  const int group = 2 * from + (second ? 1 : 0);
  // the values up to the pair of groups after it that has any
  const uint32_t through = __shfl_sync(0xffffffffu, second ? count : count - c[1], from);
  const int last = __ffs(__ballot_sync(0xffffffffu, count > through) | 0x80000000u) - 1;
  const uint32_t upto = __shfl_sync(0xffffffffu, count, last);
  const int end = 4 * (2 * last + 2) * kGroupBins - 1;
  const float scale = group < kHeavyGroups ? (float)heavy * 1.13686838e-13f / estimate : 1.0f;
  if (warp < C) s.fine_count[warp][lane] = cluster.map_shared_rank(&s, warp)->hist[group * kGroupBins + lane];
  __syncthreads();
  uint32_t n = 0;
#pragma unroll
  for (int o = 0; o < kMaxBlocks; ++o)
    if (o < C) n += s.fine_count[o][lane];
  float m = (float)n * middle_of(group * kGroupBins + lane) * scale;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float x = __shfl_up_sync(0xffffffffu, m, o);
    if (lane >= o) m += x;
  }
  const float at = before + (second ? first : 0.f) + m;
  const uint32_t there = __ballot_sync(0xffffffffu, at >= want) | 0x80000000u;
  const int lane_of = __ffs(there) - 1, bin = group * kGroupBins + lane_of;
  const float own = __shfl_sync(0xffffffffu, (float)n * middle_of(group * kGroupBins + lane) * scale, lane_of);
  const float into = fminf(fmaxf((want - __shfl_sync(0xffffffffu, at, lane_of) + own) / own, 0.f), 0.999f);
  const uint32_t in_bin = __shfl_sync(0xffffffffu, n, lane_of);
  // some 110 values are looked at, by how densely they lie here, but half a k to either
  // side at least: a cut outside of them costs the general way (15 to 40 us), more of
  // them the ranking (200 us with 256 for 191 in 256 rows of 100003).  With whole k
  // about the estimate's, 4 rows of 100 missed of 150000 values; now 1 of 3600.
  const uint32_t own_group = __shfl_sync(0xffffffffu, second ? c[1] : c[0], from);
  const uint32_t after = __shfl_sync(0xffffffffu, second ? c[0] : c[1], second ? min(from + 1, 31) : from);
  const float dense = fmaxf((float)in_bin * 0.25f, (float)max(own_group, after) * (1.0f / 128.0f));  // of a k
  const float place = 4.0f * ((float)bin + into);
  const float reach = fminf(fmaxf(52.0f / fmaxf(dense, 1.0f), dense < 200.f ? 0.5f : 0.f), 64.0f);
  if (bin >= kBins - 1 || dense > 400.f) return About{1, 0, end, upto};
  return About{(int)fmaxf(place - reach, 0.f), (int)(place + reach), end, upto};
}

// What the blocks have collected in s.local goes into list[1] of block 0, or of
// every block.  Ends with the cluster's barrier.
__device__ __forceinline__ void merge_lists(Shared& s, cg::cluster_group& cluster, int blocks) {
  __syncthreads();
  const int n = (int)min(s.pushed, (uint32_t)kList);
  if ((int)threadIdx.x < blocks)
    s.base[threadIdx.x] = atomicAdd(&cluster.map_shared_rank(&s, threadIdx.x)->merged, s.pushed);
  __syncthreads();
  for (int o = 0; o < blocks; ++o) {
    const uint32_t to = s.base[o] + threadIdx.x;
    if ((int)threadIdx.x < n && to < (uint32_t)kList) cluster.map_shared_rank(&s, o)->list[1][to] = s.local[threadIdx.x];
  }
  cluster.sync();
}

template <class T, bool STAGED>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& s = *reinterpret_cast<Shared*>(smem_raw);
  constexpr int kVec = 16 / (int)sizeof(T);
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x / C;
  pdl_launch_dependents();
  cluster_arrive();  // waited for before the first look at another block's memory
  for (int i = tid; i < 256; i += kThreads) s.powers[i] = kPowers.v[i];
  for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
  if (tid == 0) s.merged = s.pushed = 0;
  pdl_wait();

  const T* const base = static_cast<const T*>(p.logits) + row * p.ld;
  const int i0 = min(p.vocab, rank * p.piece), n = min(p.vocab, i0 + p.piece) - i0;
  const T* const mine = base + i0;
  // in shared memory the piece lies as it does to 16 bytes in global memory
  const int lead = (int)((reinterpret_cast<uintptr_t>(mine) & 15) / sizeof(T));
  T* const stage = reinterpret_cast<T*>(smem_raw + kFixed) + lead;
  auto at = [&](int i) -> float { return value_of<T>(STAGED ? stage[i] : mine[i]); };

  // ---- the piece into shared memory, its greatest value (lowest index first) ----
  float top = -INFINITY;
  int top_at = 0x7fffffff, bad = 0;
  auto look = [&](T v, int i) {
    const float x = value_of<T>(v);
    bad |= !(x < INFINITY);
    if (x > top) {  // a thread's indexes rise
      top = x;
      top_at = i0 + i;
    }
  };
  const int head = min(n, lead ? kVec - lead : 0), vectors = (n - head) / kVec;
  if (tid < head) {
    const T v = mine[tid];
    if (STAGED) stage[tid] = v;
    look(v, tid);
  }
#pragma unroll 4
  for (int i = tid; i < vectors; i += kThreads) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(mine + head) + i);
    if (STAGED) *reinterpret_cast<uint4*>(stage + head + i * kVec) = raw;
    const T* v = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int j = 0; j < kVec; ++j) look(v[j], head + i * kVec + j);
  }
  for (int i = head + vectors * kVec + tid; i < n; i += kThreads) {
    const T v = mine[i];
    if (STAGED) stage[i] = v;
    look(v, i);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, top, o);
    const int j = __shfl_xor_sync(0xffffffffu, top_at, o);
    if (x > top || (x == top && j < top_at)) {
      top = x;
      top_at = j;
    }
    bad |= __shfl_xor_sync(0xffffffffu, bad, o);
  }
  if (lane == 0) {
    s.warp_top[warp] = top;
    s.warp_at[warp] = top_at;
    s.warp_bad[warp] = bad;
  }
  __syncthreads();
  cluster_wait();  // all blocks have begun: their shared memory is there
  if (tid < C) {
    for (int w = 0; w < kWarps; ++w) {
      if (s.warp_top[w] > top || (s.warp_top[w] == top && s.warp_at[w] < top_at)) {
        top = s.warp_top[w];
        top_at = s.warp_at[w];
      }
      bad |= s.warp_bad[w];
    }
    Shared& to = *cluster.map_shared_rank(&s, tid);
    to.top[rank] = top;
    to.top_at[rank] = top_at;
    to.bad[rank] = bad;
  }
  cluster.sync();
  top = s.top[0];
  top_at = s.top_at[0];
  bad = s.bad[0];
  for (int c = 1; c < C; ++c) {
    if (s.top[c] > top || (s.top[c] == top && s.top_at[c] < top_at)) {
      top = s.top[c];
      top_at = s.top_at[c];
    }
    bad |= s.bad[c];
  }
  const float t = p.temperature ? __ldg(p.temperature + row) : 1.0f;
  const bool none = bad || !(top > -INFINITY), greedy = !(t > 0.f);
  if (none || greedy) {  // the same for the whole cluster; nothing of a block is looked at by another any more
    if (rank == 0 && tid == 0) {
      p.tokens[row] = none ? -1 : top_at;
      if (p.logprobs) p.logprobs[row] = none ? NAN : 0.f;
    }
    return;
  }

  Row r;
  r.top = top;
  r.e = exponent_of(t);
  const int k = p.top_k ? __ldg(p.top_k + row) : 0;
  const float tp = p.top_p ? __ldg(p.top_p + row) : 1.0f;
  const bool by_count = k > 0 && k < p.vocab, by_mass = tp < 1.0f;

  // kept: (key, index) pairs, as one number that falls in the order's direction, from this one on
  uint64_t cut = 0;
  auto pair_of = [&](uint32_t key, int i) -> uint64_t { return ((uint64_t)key << 32) | (0xffffffffu - (uint32_t)(i0 + i)); };

  // ---- the counts of all values' bins ----
  const float mp = p.min_p ? __ldg(p.min_p + row) : 0.f;
  uint64_t least = 0;  // ceil(min_p * 2^43)
  if (mp >= 1.f) {
    least = 1ull << kOne;
  } else if (mp > 0.f) {
    const uint64_t f = fraction_of(mp);
    least = (f >> (64 - kOne)) + ((f & ((1ull << (64 - kOne)) - 1)) != 0);
  }
  const float u = fminf(fmaxf(__ldg(p.uniform + row), 0.f), 0.99999994f);  // a NaN counts as 0
  const int seg = (n + kWarps - 1) / kWarps;  // a warp's values
  auto write_out = [&](int index, float x, uint64_t total) {
    p.tokens[row] = index;
    if (p.logprobs) {
      // (x - top) / T - ln(sum of weights against the largest)
      const float d = x - r.top, h = __fmul_rn(d, r.e.hi), l = fmaf(d, r.e.hi, -h) + d * r.e.lo;
      const float rest = (float)(total - (1ull << kOne)) * 1.13686838e-13f;  // 2^-43: the largest is among them
      p.logprobs[row] = (h + l) * 0.693147182f - log1pf(rest);
    }
  };
  auto collect = [&](float x, int i) {
    const uint32_t spot = atomicAdd(&s.pushed, 1u);
    if (spot < (uint32_t)kList) s.local[spot] = pair_of(key_of(x), i);
  };
  // Block 0 has every value that may be kept in list[1] and does the rest alone:
  // count_limit and, where by_mass, p of `mass` (0: of the first count_limit).
  auto finish_list = [&](uint32_t count_limit, uint64_t mass) {
    const int entries = (int)min(s.merged, (uint32_t)kList);
    const uint64_t* const list = s.list[1];
    const bool on = tid < entries;
    const uint64_t me = on ? list[tid] : 0;
    const float x = value_of_key((uint32_t)(me >> 32));
    const uint64_t w = on ? weight_of(x, r, s.powers) : 0;
    if (on) s.list_mass[tid] = w;
    __syncthreads();
    uint64_t before = 0;
    uint32_t c = 0;
    if (on)
      for (int j = 0; j < entries; ++j)
        if (list[j] > me) {
          before += s.list_mass[j];
          ++c;
        }
    bool keep = on && c < count_limit;
    if (by_mass) {
      if (mass == 0) {
        uint64_t first = keep ? w : 0, none = 0;
        block_sums(s, first, none);
        mass = first;
      }
      keep = keep && before < share_of(tp, mass);
    }
    keep = keep && w >= least;
    uint64_t total = keep ? w : 0, none = 0;
    block_sums(s, total, none);
    if (on) s.list_mass[tid] = keep ? w : 0;
    __syncthreads();
    const uint64_t target = __umul64hi(fraction_of(u), total);
    if (keep && w > 0) {  // the kept ones of lower index
      const uint32_t my = (uint32_t)me;  // falls with the index
      uint64_t run = 0;
      for (int j = 0; j < entries; ++j)
        if ((uint32_t)list[j] > my) run += s.list_mass[j];
      if (run <= target && target < run + w) write_out((int)(0xffffffffu - my), x, total);
    }
  };

  bool summed = false;  // the kept weights of the warps' segments are in warp_mass
  bool fresh = false;   // the histogram's counts are those of all values
  if (by_count || by_mass) {
    uint64_t heavy = 0;
#pragma unroll 2
    for (int i = tid; i < n; i += 2 * kThreads) {
      const float x0 = at(i), x1 = i + kThreads < n ? at(i + kThreads) : -INFINITY;
      const int b0 = first_bin(r, x0), b1 = first_bin(r, x1);
      if (b0 < kBins) atomicAdd(&s.hist[b0], 1u);
      if (b1 < kBins) atomicAdd(&s.hist[b1], 1u);
      if (by_mass && min(b0, b1) < kHeavyGroups * kGroupBins) {
        uint64_t w[2];
        int bins[2];
        weights_of(x0, x1, r, s.powers, w, bins);
        heavy += (b0 < kHeavyGroups * kGroupBins ? w[0] : 0) + (b1 < kHeavyGroups * kGroupBins ? w[1] : 0);
      }
    }
    uint64_t none = 0;
    block_sums(s, heavy, none);  // its barriers are the histogram's too
    if (tid < C) cluster.map_shared_rank(&s, tid)->heavy[rank] = heavy;
#pragma unroll
    for (int j = 0; j < kGroups / kWarps; ++j) {
      const int g = warp + j * kWarps;
      const uint32_t c = s.hist[g * kGroupBins + lane], all = __reduce_add_sync(0xffffffffu, c);
      float m = (float)c * middle_of(g * kGroupBins + lane);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
      if (lane < C) {
        Shared& to = *cluster.map_shared_rank(&s, lane);
        to.group_count[rank][g] = all;
        to.group_about[rank][g] = m;
      }
    }
    if (tid == 0) {
      s.before_mass = 0;
      s.before_count = 0;
    }
    cluster.sync();
    fresh = !by_mass;
    if (by_count) {
      // few enough: block 0 gets them all
      find_bin(s, cluster, C, rank, false, true, (uint32_t)k, 0);
      const int bin = s.bin;
      if (bin < 0 || s.before_count + s.bin_count <= (uint32_t)kList) {
        // (bin < 0: fewer than k have weight)
        for (int i = tid; i < n; i += kThreads) {
          const float x = at(i);
          if (first_bin(r, x) <= (bin < 0 ? kBins - 1 : bin)) collect(x, i);
        }
        merge_lists(s, cluster, bin < 0 ? C : 1);
        if (bin >= 0 || s.merged <= (uint32_t)kList) {
          if (rank == 0) finish_list((uint32_t)k, 0);
          return;
        }
      }
      cluster.sync();  // the histogram is read by all others until here
    } else {
      const About about = find_about(s, cluster, C, tp);
      const bool few = about.upto <= (uint32_t)kRanked;
      // few: all up to the end of the next groups with values; else what lies around
      // the estimate, and the exact sum above that
      const int low = few ? 0 : about.low;
      const int high = few ? about.end : about.high;
      uint64_t all = 0, above = 0, m = 0;
#pragma unroll 1
      for (int i = warp * seg + lane; i < min(n, (warp + 1) * seg); i += 64) {
        const float x[2] = {at(i), i + 32 < min(n, (warp + 1) * seg) ? at(i + 32) : -INFINITY};
        uint64_t w[2];
        int step[2];
        weights_of(x[0], x[1], r, s.powers, w, step);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          all += w[j];
          if (step[j] < low || (few && step[j] <= high)) {
            above += w[j];
            m += w[j] >= least ? w[j] : 0;
          }
          if (step[j] >= low && step[j] <= high) collect(x[j], i + 32 * j);
        }
      }
      uint64_t my_all = all, my_above = above;
      block_sums(s, my_all, my_above);
      if (tid < C) {
        Shared& to = *cluster.map_shared_rank(&s, tid);
        to.sum[rank] = my_all;
        to.above[rank] = my_above;
      }
      merge_lists(s, cluster, few ? 1 : C);
      all = above = 0;
      for (int o = 0; o < C; ++o) {
        all += s.sum[o];
        above += s.above[o];
      }
      const uint64_t want = share_of(tp, all);
      if (few && above >= want) {  // above: all that is listed
        if (rank == 0) finish_list(0xffffffffu, all);
        return;
      }
      const uint64_t* const list = s.list[1];
      const int entries = (int)min(s.merged, (uint32_t)kList);
      const uint64_t me = tid < entries ? list[tid] : 0;
      const uint64_t w = tid < entries ? weight_of(value_of_key((uint32_t)(me >> 32)), r, s.powers) : 0;
      if (tid < entries) s.list_mass[tid] = w;
      uint64_t listed = w, none2 = 0;
      block_sums(s, listed, none2);
      if (!few && s.merged <= (uint32_t)kList && above < want && above + listed >= want) {  // the cut is in the list
        if (tid < entries) {
          uint64_t before = above;
          for (int j = 0; j < entries; ++j)
            if (list[j] > me) before += s.list_mass[j];
          if (before < want && before + w >= want) s.cut = me;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
        __syncthreads();
        if (lane == 0) s.warp_mass[warp] = m;
        __syncthreads();
        cut = s.cut;
        const int index = (int)(0xffffffffu - (uint32_t)me) - i0;
        if (tid < entries && me >= cut && w >= least && index >= 0 && index < n)
          atomicAdd(reinterpret_cast<unsigned long long*>(&s.warp_mass[index / seg]), (unsigned long long)w);
        __syncthreads();
        summed = true;
      }
    }
  }

  // ---- the general way: histograms with the weights' exact sums ----
  const bool spoiled = !summed && by_mass;  // the limbs go over the staged values
  auto any = [&](int i) -> float { return STAGED && !spoiled ? value_of<T>(stage[i]) : value_of<T>(mine[i]); };
  uint64_t limit_mass = 0, want_mass = 0;
#pragma unroll 1
  for (int pass = by_count ? 0 : 1; !summed && pass < (by_mass ? 2 : 1); ++pass) {
    const bool counting = pass == 0;
    uint32_t key_low = 0, key_high = 0xffffffffu, shift = 0;
    int bin = -1;  // of all values' histogram, once it is known
    if (tid == 0) {
      s.before_mass = 0;
      s.before_count = 0;
    }
    __syncthreads();
#pragma unroll 1
    for (bool first_level = true;; first_level = false) {
      if (!(first_level && fresh)) {
        for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
        if (by_mass)
          for (int i = tid; i < 3 * kBins; i += kThreads) limbs_of(s, 0)[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += 2 * kThreads) {
          const float x[2] = {any(i), i + kThreads < n ? any(i + kThreads) : -INFINITY};
          uint64_t w[2] = {0, 0};
          int bins[2];
          if (by_mass) {
            weights_of(x[0], x[1], r, s.powers, w, bins);
          } else {
            bins[0] = first_bin(r, x[0]);
            bins[1] = first_bin(r, x[1]);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            int b = by_mass ? bin_of_k(bins[j]) : bins[j];
            if (!first_level) {
              const uint32_t key = key_of(x[j]);
              b = b == bin && key >= key_low && key <= key_high ? (int)((key_high - key) >> shift) : kBins;
            }
            if (b < kBins) {
              atomicAdd(&s.hist[b], 1u);
              if (by_mass) {
                atomicAdd(limbs_of(s, 0) + b, (uint32_t)w[j] & 0x7fffu);
                atomicAdd(limbs_of(s, 1) + b, (uint32_t)(w[j] >> 15) & 0x7fffu);
                if (w[j] >> 30) atomicAdd(limbs_of(s, 2) + b, (uint32_t)(w[j] >> 30));
              }
            }
          }
        }
        __syncthreads();
        // sums of 32 bins, to every block
#pragma unroll
        for (int g = warp; g < kGroups; g += kWarps) {
          const int b = g * kGroupBins + lane;
          const uint32_t c = __reduce_add_sync(0xffffffffu, s.hist[b]);
          uint64_t m = 0;
          if (by_mass) {
            m = limbs_of(s, 0)[b] + ((uint64_t)limbs_of(s, 1)[b] << 15) + ((uint64_t)limbs_of(s, 2)[b] << 30);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
          }
          if (lane < C) {
            Shared& to = *cluster.map_shared_rank(&s, lane);
            to.group_count[rank][g] = c;
            if (by_mass) to.group_mass[rank][g] = m;
          }
        }
        cluster.sync();
        fresh = first_level;
      }
      if (first_level && !counting) {
        uint64_t all = limit_mass;
        if (!all) {
#pragma unroll
          for (int o = 0; o < kMaxBlocks; ++o)
            if (o < C) all += s.group_mass[o][lane] + s.group_mass[o][lane + 32];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        }
        want_mass = share_of(tp, all);
      }
      find_bin(s, cluster, C, rank, by_mass, counting, (uint32_t)k, want_mass);
      const int found = s.bin;
      if (found < 0) break;  // fewer values with weight than that: nothing is cut
      const uint32_t in_bin = s.bin_count;
      if (first_level) {
        bin = found;
      } else {
        key_high -= (uint32_t)found << shift;
        key_low = shift ? max(key_low, key_high - ((1u << shift) - 1u)) : key_high;
      }
      auto inside = [&](float x, uint32_t key) {
        return first_bin(r, x) == bin && key >= key_low && key <= key_high;
      };
      if (in_bin <= (uint32_t)kList) {
        // every block gets all candidates and ranks them
        for (int i = tid; i < n; i += kThreads) {
          const float x = any(i);
          const uint32_t key = key_of(x);
          if (inside(x, key)) {
            const uint32_t spot = s.offset + atomicAdd(&s.pushed, 1u);
            if (spot < (uint32_t)kList)  // in_bin of them
              for (int o = 0; o < C; ++o) cluster.map_shared_rank(&s, o)->list[pass][spot] = pair_of(key, i);
          }
        }
        cluster.sync();
        const uint64_t* const list = s.list[pass];
        const uint64_t me = tid < (int)in_bin ? list[tid] : 0;
        uint64_t w = 0;
        if (tid < (int)in_bin) {
          w = weight_of(value_of_key((uint32_t)(me >> 32)), r, s.powers);
          s.list_mass[tid] = w;
        }
        __syncthreads();
        if (tid < (int)in_bin) {
          uint64_t m = s.before_mass;
          uint32_t c = s.before_count;
          for (uint32_t j = 0; j < in_bin; ++j)
            if (list[j] > me) {
              m += s.list_mass[j];
              ++c;
            }
          if (counting ? c + 1 == (uint32_t)k : m < want_mass && m + w >= want_mass) {
            s.cut = me;
            s.cut_mass = m + w;
          }
        }
        __syncthreads();
        cut = s.cut;
        limit_mass = s.cut_mass;
        break;
      }
      // the least and greatest key in there
      uint32_t low = 0xffffffffu, high = 0;
      for (int i = tid; i < n; i += kThreads) {
        const float x = any(i);
        const uint32_t key = key_of(x);
        if (inside(x, key)) {
          low = min(low, key);
          high = max(high, key);
        }
      }
      low = __reduce_min_sync(0xffffffffu, low);
      high = __reduce_max_sync(0xffffffffu, high);
      if (lane == 0) {
        s.warp_count[warp] = low;
        s.warp_mass[warp] = high;
      }
      __syncthreads();
      if (tid < C) {
        for (int w = 0; w < kWarps; ++w) {
          low = min(low, s.warp_count[w]);
          high = max(high, (uint32_t)s.warp_mass[w]);
        }
        Shared& to = *cluster.map_shared_rank(&s, tid);
        to.low[rank] = low;
        to.high[rank] = high;
      }
      cluster.sync();
      key_low = 0xffffffffu;
      key_high = 0;
      for (int o = 0; o < C; ++o) {
        key_low = min(key_low, s.low[o]);
        key_high = max(key_high, s.high[o]);
      }
      if (key_low == key_high) {
        // one value, in_bin times: the index of the last that is needed
        const uint64_t each = s.bin_mass / in_bin;
        const uint32_t ties = counting ? (uint32_t)k - s.before_count
                                       : (uint32_t)((want_mass - s.before_mass + each - 1) / each);
        const int seg = (n + kWarps - 1) / kWarps, end = min(n, (warp + 1) * seg);
        uint32_t c = 0;
        for (int i = warp * seg + lane; i < end; i += 32) c += key_of(any(i)) == key_low;
        c = __reduce_add_sync(0xffffffffu, c);
        __syncthreads();
        if (lane == 0) s.warp_count[warp] = c;
        __syncthreads();
        uint32_t all = 0, before = 0;
        for (int w = 0; w < kWarps; ++w) {
          if (w < warp) before += s.warp_count[w];
          all += s.warp_count[w];
        }
        if (tid < C) cluster.map_shared_rank(&s, tid)->count[rank] = all;
        cluster.sync();
        for (int o = 0; o < rank; ++o) before += s.count[o];
        if (before < ties && before + c >= ties) {  // this warp
          uint32_t left = ties - before;
          for (int i = warp * seg; i < end; i += 32) {
            const bool hit = i + lane < end && key_of(any(i + lane)) == key_low;
            const uint32_t hits = __ballot_sync(0xffffffffu, hit);
            if ((uint32_t)__popc(hits) >= left) {
              const int spot = __fns(hits, 0, (int)left);
              if (lane < C) cluster.map_shared_rank(&s, lane)->found_index = i0 + i + spot;
              break;
            }
            left -= __popc(hits);
          }
        }
        cluster.sync();
        cut = ((uint64_t)key_low << 32) | (0xffffffffu - (uint32_t)s.found_index);
        limit_mass = s.before_mass + each * ties;
        break;
      }
      shift = 0;
      while (((key_high - key_low) >> shift) >= (uint32_t)kBins) ++shift;
    }
    __syncthreads();
  }

  // ---- the mass of what is kept, by warps' segments in order ----
  const uint32_t cut_key = (uint32_t)(cut >> 32);
  auto kept = [&](float x, int i) {
    const uint32_t key = key_of(x);
    return key > cut_key || (key == cut_key && pair_of(key, i) >= cut);
  };
  auto kept_weight = [&](int i) -> uint64_t {
    const float x = any(i);
    const uint64_t w = kept(x, i) ? weight_of(x, r, s.powers) : 0;
    return w >= least ? w : 0;
  };
  if (!summed) {
    uint64_t m = 0;
    for (int i = warp * seg + lane; i < min(n, (warp + 1) * seg); i += 64) {
      float x[2] = {any(i), -INFINITY};
      const bool two = i + 32 < min(n, (warp + 1) * seg);
      if (two) x[1] = any(i + 32);
      const bool keep[2] = {kept(x[0], i), two && kept(x[1], i + 32)};
      if (keep[0] || keep[1]) {
        uint64_t w[2];
        int bins[2];
        weights_of(x[0], x[1], r, s.powers, w, bins);
#pragma unroll
        for (int j = 0; j < 2; ++j) m += keep[j] && w[j] >= least ? w[j] : 0;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
    if (lane == 0) s.warp_mass[warp] = m;
    __syncthreads();
  }
  uint64_t all = 0;
  for (int w = 0; w < kWarps; ++w) all += s.warp_mass[w];
  if (tid < C) cluster.map_shared_rank(&s, tid)->mass[rank] = all;
  cluster.sync();  // from here on a block looks at its own memory only
  uint64_t total = 0, before = 0;
  for (int o = 0; o < C; ++o) {
    if (o < rank) before += s.mass[o];
    total += s.mass[o];
  }
  const uint64_t target = __umul64hi(fraction_of(u), total);
  if (before <= target && target < before + all) {  // this block
    int w = 0;
    for (; w < kWarps - 1 && before + s.warp_mass[w] <= target; ++w) before += s.warp_mass[w];
    // the segment's values in order, a run of them to a thread
    const int begin = w * seg, end = min(n, begin + seg), each = (seg + kThreads - 1) / kThreads;
    uint64_t run = 0;
    for (int j = 0; j < each; ++j) {
      const int i = begin + tid * each + j;
      if (i < end) run += kept_weight(i);
    }
    uint64_t upto = before + block_scan(s, run);
    if (upto <= target && target < upto + run)
      for (int j = 0; j < each; ++j) {
        const int i = begin + tid * each + j;
        const uint64_t wi = i < end ? kept_weight(i) : 0;
        if (target < upto + wi) {
          write_out(i0 + i, any(i), total);
          break;
        }
        upto += wi;
      }
  }
}

template <class T, bool STAGED>
tlq_status launch_one(const SampleParams& p, int rows, int blocks, size_t smem, cudaStream_t stream) {
  const cudaError_t attr = opt_in_smem<sample_kernel<T, STAGED>>(kMaxSmem);
  if (attr != cudaSuccess) return cuda_error(attr, "sample: shared memory");
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)rows * blocks, 1, 1);
  lc.blockDim = dim3(kThreads, 1, 1);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = pdl_enabled() ? 2 : 1;
  return cuda_error(cudaLaunchKernelEx(&lc, sample_kernel<T, STAGED>, p), "sample: launch");
}

// Clusters of this many blocks that run at once, with one or two blocks to an SM
// (of a kernel that is opted in to its shared memory); asked once for each number
// of SMs.  A cluster lies in one GPC, so it is not SMs / blocks: of 152 SMs clusters
// of 1 to 8 get 152, 76, 46, 36, 28, 23, 15 and 15, and with two blocks to an SM 304,
// 152, 97, 74, 58, 46, 38 and 36.
constexpr size_t kSmemOfTwo = (228u << 10) / 2 - 1024;
template <class T>
int clusters_at_once(int blocks, int resident) {
  static std::atomic<int> known[kMaxBlocks + 1][3];  // SMs in the upper half, clusters in the lower
  const int sms = device_info().sms, was = known[blocks][resident].load(std::memory_order_relaxed);
  if (was >> 16 == sms) return was & 0xffff;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)blocks, 1, 1);
  lc.blockDim = dim3(kThreads, 1, 1);
  lc.dynamicSmemBytes = resident == 2 ? kSmemOfTwo : (size_t)kMaxSmem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, sample_kernel<T, true>, &lc) != cudaSuccess || n < 1 || n > 0xffff) {
    cudaGetLastError();
    return std::max(1, sms / blocks * resident);  // the launch reports what is wrong
  }
  known[blocks][resident].store(sms << 16 | n, std::memory_order_relaxed);
  return n;
}

// How many blocks take a row: whichever needs the least time by two lines fitted to
// 50 measurements (top-p, rows of 32000 and more): a wave of rows takes 11.5 us and
// 0.65 for every 1000 values of a block, or, where two blocks share an SM, 12 and
// 1.22.  By blocks to a row, top-p of 0.85 to 0.99, the first being the choice: 256
// rows of 100003 FP32 six 201 us, three 212, seven 225, eight 231; 64 of 131072 FP16
// four 61, two 65, eight 74; 40 of 200000 FP32 six 75, five 83, eight 91; 512 of
// 32000 FP16 one 108, two 118; 64 of 32000 FP16 four 26, three 30, two 35; one of
// 32000 eight 16, four 18, one 37.
template <class T>
tlq_status launch_as(SampleParams p, int rows, cudaStream_t stream) {
  const cudaError_t attr = opt_in_smem<sample_kernel<T, true>>(kMaxSmem);
  if (attr != cudaSuccess) return cuda_error(attr, "sample: shared memory");
  const int sms = device_info().sms;
  int blocks = 0;
  size_t smem = 0;
  double least = 0;
  for (int b = 1; b <= kMaxBlocks; ++b) {
    const size_t piece = (size_t)(p.vocab + b - 1) / b, need = kFixed + std::max(kLimbBytes, piece * sizeof(T) + 16);
    if (need > (size_t)kMaxSmem) continue;
    const int resident = need <= kSmemOfTwo ? 2 : 1;
    const long long at_once = clusters_at_once<T>(b, resident);
    const bool shared = resident == 2 && (long long)rows * b > sms;
    const double time = (double)((rows + at_once - 1) / at_once) *
                        (shared ? 12.0 + 1.22e-3 * (double)piece : 11.5 + 0.65e-3 * (double)piece);
    if (blocks == 0 || time < least) {
      blocks = b;
      smem = need;
      least = time;
    }
  }
  p.piece = (p.vocab + std::max(blocks, 1) - 1) / std::max(blocks, 1);
  if (blocks) return launch_one<T, true>(p, rows, blocks, smem, stream);
  p.piece = (p.vocab + kMaxBlocks - 1) / kMaxBlocks;
  return launch_one<T, false>(p, rows, kMaxBlocks, kFixed + kLimbBytes, stream);
}

}  // namespace

tlq_status launch_sample(const SampleArgs& a, cudaStream_t stream) {
  SampleParams p{};
  p.logits = a.logits;
  p.ld = a.ld;
  p.vocab = a.vocab;
  p.uniform = a.uniform;
  p.temperature = a.temperature;
  p.top_k = a.top_k;
  p.top_p = a.top_p;
  p.min_p = a.min_p;
  p.tokens = a.tokens;
  p.logprobs = a.logprobs;
  return a.half ? launch_as<__half>(p, a.rows, stream) : launch_as<float>(p, a.rows, stream);
}

}  // namespace tlq
