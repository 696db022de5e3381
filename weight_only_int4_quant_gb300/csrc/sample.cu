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
// within about 2^-40 of its value: the exponent in two FP32 numbers (x - max
// exactly, times log2(e) / T), 2^(-j/256) from a table and a cubic for the rest.
// FP64, the plain way, would take 30 times the arithmetic's time here (2
// operations a clock and SM).
//
// A cluster of blocks takes a row, a block a piece of it that lies in shared
// memory from its first reading on (the row is read from DRAM once).  Cuts are
// found by histograms: first over (max - x) / T in 2048 equal bins, then over
// the values inside the one bin that holds the cut, until it is a single value;
// counts and weights (three limbs of 15 bits each, so that 32-bit atomics do)
// are added up over the cluster through distributed shared memory.
#include <cooperative_groups.h>

#include <algorithm>

#include "serve.cuh"

namespace cg = cooperative_groups;

namespace tlq {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kOne = 43;             // the largest weight is 2^43
constexpr float kOctaves = 40.0f;    // weights below 2^-40 of it count as none
constexpr int kMaxSmem = 232448 - 1024;
static_assert(kMaxVocab / 8 <= 1 << 17, "limbs of 15 bits of a block's values add up in 32");

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

// exp((x - top) / T) * 2^43, or 0 below 2^-40.
__device__ __forceinline__ uint64_t weight_of(float x, float top, Exponent e, const uint64_t* __restrict__ powers) {
  const float d = __fsub_rn(x, top), back = __fsub_rn(d, x);
  const float d_lo = __fadd_rn(__fsub_rn(x, __fsub_rn(d, back)), __fsub_rn(-top, back));
  const float h = __fmul_rn(d, e.hi);
  if (!(h >= -kOctaves)) return 0;
  const float l = fmaf(d, e.hi, -h) + fmaf(d, e.lo, d_lo * e.hi);
  // h = -k / 256 + r
  const float kf = rintf(h * -256.0f);
  const int k = (int)kf;
  const float r = fmaf(kf, 1.0f / 256.0f, h);  // exact, |r| <= 2^-9
  // z = 2^(r + l) - 1 in units of 2^-40: c1 r in two numbers, and the rest
  const float c1 = 0.693147182f, c1_lo = -1.90465421e-9f, c2 = 0.240226507f, c3 = 0.0555041087f, c4 = 0.00961812911f;
  const float zh = __fmul_rn(c1, r), rr = r + l;
  const float zl = fmaf(c1, r, -zh) + fmaf(c1_lo, r, c1 * l) + rr * rr * fmaf(rr, fmaf(rr, c4, c3), c2);
  const float a = __fadd_rn(__fmul_rn(zh, 2147483648.0f), 12582912.0f);  // units of 2^-31, a whole number
  const float rest = __fsub_rn(__fmul_rn(zh, 2147483648.0f), __fsub_rn(a, 12582912.0f));
  const float b = __fadd_rn(__fmul_rn(fmaf(zl, 2147483648.0f, rest), 512.0f), 12582912.0f);
  const int z = (__float_as_int(a) - 0x4B400000) * 512 + (__float_as_int(b) - 0x4B400000);
  const uint64_t power = powers[k & 255];
  const int n = k >> 8;
  const uint64_t v = power + (uint64_t)(((long long)((power + 2048) >> 12) * z + (1 << 27)) >> 28);
  return (v + ((1ull << n) >> 1)) >> n;
}

// Order-preserving whole numbers for FP32 values (-0 as +0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

struct Bin {
  uint32_t count, limb[3];
};

// What the blocks of a cluster tell each other.
struct Shared {
  uint32_t hist[4][kBins];  // counts, limbs
  uint64_t powers[256];
  uint64_t warp_mass[kWarps];
  uint32_t warp_count[kWarps];
  // of each block, written by all blocks into all
  float top[16];
  int top_at[16];
  uint32_t low[16], high[16];
  uint64_t mass[16];
  uint32_t count[16];
  int bad[16];
  // the answer of a search, written by the block that has it into all
  int found_bin, found_index;
  uint64_t above_mass;
  uint32_t above_count;
  uint64_t bin_mass;
  uint32_t bin_count;
};

struct Row {
  float top;
  Exponent e;
  float scale;  // bins of an octave
};

__device__ __forceinline__ int first_bin(const Row& r, float x) {  // kBins: below every weight
  const float t = (r.top - x) * r.scale;
  return t < (float)kBins ? (int)t : kBins;
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

// Sums over the block; every thread gets them.  Two barriers.
__device__ __forceinline__ void block_sum(Shared& s, uint64_t& mass, uint32_t& count) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mass += __shfl_xor_sync(0xffffffffu, mass, o);
    count += __shfl_xor_sync(0xffffffffu, count, o);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    s.warp_mass[threadIdx.x >> 5] = mass;
    s.warp_count[threadIdx.x >> 5] = count;
  }
  __syncthreads();
  mass = 0;
  count = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    mass += s.warp_mass[w];
    count += s.warp_count[w];
  }
}

// Exclusive sums over the block's threads, and the total.
__device__ __forceinline__ void block_scan(Shared& s, uint64_t& mass, uint32_t& count) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t m0 = mass;
  const uint32_t c0 = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t m = __shfl_up_sync(0xffffffffu, mass, o);
    const uint32_t c = __shfl_up_sync(0xffffffffu, count, o);
    if (lane >= o) {
      mass += m;
      count += c;
    }
  }
  __syncthreads();
  if (lane == 31) {
    s.warp_mass[warp] = mass;
    s.warp_count[warp] = count;
  }
  __syncthreads();
  mass -= m0;
  count -= c0;
  for (int w = 0; w < warp; ++w) {
    mass += s.warp_mass[w];
    count += s.warp_count[w];
  }
}

template <class T, bool STAGED>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& s = *reinterpret_cast<Shared*>(smem_raw);
  T* const stage = reinterpret_cast<T*>(smem_raw + ((sizeof(Shared) + 15) & ~size_t(15)));
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x / C;
  pdl_launch_dependents();
  for (int i = tid; i < 256; i += kThreads) s.powers[i] = kPowers.v[i];
  pdl_wait();

  const T* const base = static_cast<const T*>(p.logits) + row * p.ld;
  const int i0 = min(p.vocab, rank * p.piece), n = min(p.vocab, i0 + p.piece) - i0;
  const T* const mine = base + i0;
  auto at = [&](int i) -> float { return value_of<T>(STAGED ? stage[i] : mine[i]); };

  // ---- the piece into shared memory, its greatest value (lowest index first) ----
  float top = -INFINITY;
  int top_at = 0x7fffffff, bad = 0;
  auto look = [&](float x, int i) {
    bad |= !(x < INFINITY);
    if (x > top) {
      top = x;
      top_at = i;
    }
  };
  if (STAGED) {
    for (int i = tid; i < n; i += kThreads) {
      const T v = mine[i];
      stage[i] = v;
      look(value_of<T>(v), i0 + i);
    }
  } else {
    for (int i = tid; i < n; i += kThreads) look(value_of<T>(mine[i]), i0 + i);
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
  __shared__ float warp_top[kWarps];
  __shared__ int warp_at[kWarps], warp_bad[kWarps];
  if (lane == 0) {
    warp_top[warp] = top;
    warp_at[warp] = top_at;
    warp_bad[warp] = bad;
  }
  __syncthreads();
  if (tid < C) {
    float x = warp_top[0];
    int j = warp_at[0], b = warp_bad[0];
    for (int w = 1; w < kWarps; ++w) {
      if (warp_top[w] > x || (warp_top[w] == x && warp_at[w] < j)) {
        x = warp_top[w];
        j = warp_at[w];
      }
      b |= warp_bad[w];
    }
    Shared& to = *cluster.map_shared_rank(&s, tid);
    to.top[rank] = x;
    to.top_at[rank] = j;
    to.bad[rank] = b;
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
  const bool first_thread = rank == 0 && tid == 0;
  const float t = p.temperature ? __ldg(p.temperature + row) : 1.0f;
  const bool none = bad || !(top > -INFINITY), greedy = !(t > 0.f);
  if (none || greedy) {  // the same for the whole cluster
    if (first_thread) {
      p.tokens[row] = none ? -1 : top_at;
      if (p.logprobs) p.logprobs[row] = none ? NAN : 0.f;
    }
    cluster.sync();  // no block ends while another may write to it
    return;
  }

  Row r;
  r.top = top;
  r.e = exponent_of(t);
  r.scale = fminf(r.e.hi, 1e30f) * ((float)kBins / kOctaves);
  const int k = p.top_k ? __ldg(p.top_k + row) : 0;
  const float tp = p.top_p ? __ldg(p.top_p + row) : 1.0f;
  const float mp = p.min_p ? __ldg(p.min_p + row) : 0.f;
  const bool by_count = k > 0 && k < p.vocab, by_mass = tp < 1.0f;

  uint32_t cut_key = 0;       // kept: keys above it, and
  int cut_at = 0x7fffffff;    // those equal to it up to this index
  if (by_count || by_mass) {
    // Finds, in the falling order, the first value at which the count reaches
    // want_count (mass 0) or the mass want_mass: its key, and how many of that
    // value are needed.
    uint64_t limit_mass = 0;  // of the values that the count leaves
    uint32_t ties = 0xffffffffu;  // all of them
    for (int pass = by_count ? 0 : 1; pass < (by_mass ? 2 : 1); ++pass) {
      const bool counting = pass == 0;
      uint64_t before_mass = 0, want_mass = 0;
      uint32_t before_count = 0, key_low = 0, key_high = 0xffffffffu, shift = 0;
      int bin = -1;  // of the first level; -1: not known yet
      for (int level = 0; level < 8; ++level) {
        for (int i = tid; i < 4 * kBins; i += kThreads) (&s.hist[0][0])[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
          const float x = at(i);
          const int b1 = first_bin(r, x);
          int b = b1;
          if (level > 0) {
            const uint32_t key = key_of(x);
            b = b1 == bin && key >= key_low && key <= key_high ? (int)((key_high - key) >> shift) : kBins;
          }
          if (b < kBins) {
            atomicAdd(&s.hist[0][b], 1u);
            if (by_mass) {
              const uint64_t w = weight_of(x, r.top, r.e, s.powers);
              atomicAdd(&s.hist[1][b], (uint32_t)w & 0x7fffu);
              atomicAdd(&s.hist[2][b], (uint32_t)(w >> 15) & 0x7fffu);
              atomicAdd(&s.hist[3][b], (uint32_t)(w >> 30));
            }
          }
        }
        cluster.sync();
        // a block's share of the bins, added up over the cluster: bins [rank * share, + share)
        const int share = (kBins + C - 1) / C, each = (share + kThreads - 1) / kThreads;
        uint64_t m = 0, my_mass[4];
        uint32_t c = 0, my_count[4];
        for (int j = 0; j < each; ++j) {
          const int i = tid * each + j, b = rank * share + i;
          my_mass[j] = 0;
          my_count[j] = 0;
          if (i < share && b < kBins)
            for (int o = 0; o < C; ++o) {
              const Shared& from = *cluster.map_shared_rank(&s, o);
              my_count[j] += from.hist[0][b];
              if (by_mass)
                my_mass[j] += from.hist[1][b] + ((uint64_t)from.hist[2][b] << 15) + ((uint64_t)from.hist[3][b] << 30);
            }
          m += my_mass[j];
          c += my_count[j];
        }
        uint64_t all_m = m, pre_m = m;
        uint32_t all_c = c, pre_c = c;
        block_sum(s, all_m, all_c);
        block_scan(s, pre_m, pre_c);
        if (tid < C) {
          Shared& to = *cluster.map_shared_rank(&s, tid);
          to.mass[rank] = all_m;
          to.count[rank] = all_c;
          to.found_bin = -1;
        }
        cluster.sync();
        uint64_t total_m = 0, base_m = before_mass;
        uint32_t base_c = before_count;
        for (int o = 0; o < C; ++o) {
          if (o < rank) {
            base_m += s.mass[o];
            base_c += s.count[o];
          }
          total_m += s.mass[o];
        }
        if (level == 0 && !counting) {
          // the shortest run that reaches p of the mass: ceil(p * mass), of at least one value
          const uint64_t whole_m = by_count && limit_mass ? limit_mass : total_m;
          const float q = fmaxf(tp, 0.f);
          const uint64_t frac = (uint64_t)((double)q * 18446744073709551616.0);
          want_mass = max(1ull, (unsigned long long)(__umul64hi(frac, whole_m) + (frac * whole_m != 0)));
        }
        base_m += pre_m;
        base_c += pre_c;
        for (int j = 0; j < each; ++j) {
          const bool here = counting ? base_c < (uint32_t)k && base_c + my_count[j] >= (uint32_t)k
                                     : base_m < want_mass && base_m + my_mass[j] >= want_mass;
          if (here)
            for (int o = 0; o < C; ++o) {
              Shared& to = *cluster.map_shared_rank(&s, o);
              to.found_bin = rank * share + tid * each + j;
              to.above_mass = base_m;
              to.above_count = base_c;
              to.bin_mass = my_mass[j];
              to.bin_count = my_count[j];
            }
          base_m += my_mass[j];
          base_c += my_count[j];
        }
        cluster.sync();
        const int found = s.found_bin;
        if (found < 0) break;  // fewer values with weight than that: nothing is cut
        before_mass = s.above_mass;
        before_count = s.above_count;
        const uint32_t in_bin = s.bin_count;
        const uint64_t mass_in_bin = s.bin_mass;
        if (level == 0) {
          bin = found;
        } else {
          key_high -= (uint32_t)found << shift;
          key_low = shift ? max(key_low, key_high - ((1u << shift) - 1u)) : key_high;
        }
        // the least and greatest key in there
        uint32_t low = 0xffffffffu, high = 0;
        for (int i = tid; i < n; i += kThreads) {
          const float x = at(i);
          const uint32_t key = key_of(x);
          if (first_bin(r, x) == bin && key >= key_low && key <= key_high) {
            low = min(low, key);
            high = max(high, key);
          }
        }
        low = __reduce_min_sync(0xffffffffu, low);
        high = __reduce_max_sync(0xffffffffu, high);
        __syncthreads();
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
        if (key_low == key_high) {  // one value, in_bin times
          ties = counting ? (uint32_t)k - before_count
                          : (uint32_t)((want_mass - before_mass + mass_in_bin / in_bin - 1) / (mass_in_bin / in_bin));
          if (counting) limit_mass = before_mass + (mass_in_bin / in_bin) * ties;
          if (ties >= in_bin) ties = 0xffffffffu;
          cut_key = key_low;
          break;
        }
        shift = 0;
        while (((key_high - key_low) >> shift) >= (uint32_t)kBins) ++shift;
      }
    }
    if (ties != 0xffffffffu) {
      // the index of the last of the ties: warps hold pieces of 32 * steps values in order
      const int seg = (n + kWarps - 1) / kWarps;
      uint32_t c = 0;
      for (int i = warp * seg + lane; i < min(n, (warp + 1) * seg); i += 32) c += key_of(at(i)) == cut_key;
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
        for (int i = warp * seg; i < min(n, (warp + 1) * seg); i += 32) {
          const bool hit = i + lane < min(n, (warp + 1) * seg) && key_of(at(i + lane)) == cut_key;
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
      cut_at = s.found_index;
    }
  }

  // ---- the mass of what is kept, by warps' segments in order ----
  const uint64_t least = (uint64_t)ceil(fmin((double)fmaxf(mp, 0.f), 1.0) * 8796093022208.0);
  const bool cut = by_count || by_mass;
  auto kept_weight = [&](int i) -> uint64_t {
    const float x = at(i);
    if (cut) {
      const uint32_t key = key_of(x);
      if (key < cut_key || (key == cut_key && i0 + i > cut_at)) return 0;
    }
    const uint64_t w = weight_of(x, r.top, r.e, s.powers);
    return w >= least ? w : 0;
  };
  const int seg = (n + kWarps - 1) / kWarps;
  uint64_t m = 0;
  for (int i = warp * seg + lane; i < min(n, (warp + 1) * seg); i += 32) m += kept_weight(i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
  __syncthreads();
  if (lane == 0) s.warp_mass[warp] = m;
  __syncthreads();
  uint64_t all = 0;
  for (int w = 0; w < kWarps; ++w) all += s.warp_mass[w];
  if (tid < C) cluster.map_shared_rank(&s, tid)->mass[rank] = all;
  cluster.sync();
  uint64_t total = 0, before = 0;
  for (int o = 0; o < C; ++o) {
    if (o < rank) before += s.mass[o];
    total += s.mass[o];
  }
  const float u = fminf(fmaxf(__ldg(p.uniform + row), 0.f), 0.99999994f);  // a NaN counts as 0
  const uint64_t target = __umul64hi((uint64_t)((double)u * 18446744073709551616.0), total);
  if (before <= target && target < before + all) {  // this block
    int w = 0;
    for (; w < kWarps - 1 && before + s.warp_mass[w] <= target; ++w) before += s.warp_mass[w];
    // the segment's values in order, a run of them to a thread
    const int begin = w * seg, end = min(n, begin + seg), each = (seg + kThreads - 1) / kThreads;
    uint64_t run = 0;
    uint32_t unused = 0;
    for (int j = 0; j < each; ++j) {
      const int i = begin + tid * each + j;
      if (i < end) run += kept_weight(i);
    }
    uint64_t upto = run;
    block_scan(s, upto, unused);
    upto += before;
    if (upto <= target && target < upto + run)
      for (int j = 0; j < each; ++j) {
        const int i = begin + tid * each + j;
        const uint64_t wi = i < end ? kept_weight(i) : 0;
        if (target < upto + wi) {
          p.tokens[row] = i0 + i;
          if (p.logprobs) {
            // (x - top) / T - ln(sum of weights against the largest)
            const float d = at(i) - r.top, h = __fmul_rn(d, r.e.hi), l = fmaf(d, r.e.hi, -h) + d * r.e.lo;
            const float rest = (float)(total - (1ull << kOne)) * 1.13686838e-13f;  // 2^-43
            p.logprobs[row] = (h + l) * 0.693147182f - log1pf(rest);
          }
          break;
        }
        upto += wi;
      }
  }
  cluster.sync();  // no block ends while another may write to it
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

template <class T>
tlq_status launch_as(SampleParams p, int rows, cudaStream_t stream) {
  int blocks = 1;
  while (blocks < 8 && p.vocab > 4096 * blocks) blocks *= 2;
  p.piece = (p.vocab + blocks - 1) / blocks;
  const size_t fixed = (sizeof(Shared) + 15) & ~size_t(15), staged = fixed + (size_t)p.piece * sizeof(T);
  return staged <= (size_t)kMaxSmem ? launch_one<T, true>(p, rows, blocks, staged, stream)
                                    : launch_one<T, false>(p, rows, blocks, fixed, stream);
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
