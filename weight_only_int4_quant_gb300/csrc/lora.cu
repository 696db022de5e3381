// Low-rank adapters of many requests beside a shared projection:
//
//   out[t] = fp16(y[t] + scale_a * B_a (A_a x[t])),  a = the adapter of token t's request
//
// One launch.  A cluster of eight blocks takes a tile of one request's tokens:
// each block contracts an eighth of K, the partial A x (FP32) are summed over
// the cluster through shared memory in rank order, and each block then makes
// an eighth of N.  So x, y and out cross DRAM once, A x never does, and no
// workspace or second launch is needed.  At rank 16 there are 2 * 16 flops to
// every 2 bytes: memory bounds long batches, latency short ones.  32 tokens, 8
// adapters of rank 16, 2048 -> 6144: 6.5 us; 3600 tokens, rank 32, 2048 -> 8192:
// 53 us, 2.6 TB/s, held by memory latency at two blocks of 128 registers a thread
// to an SM (80 registers, or 32-token tiles, were slower).
//
// Both products run on mma.sync m16n8k16 with operands straight from global
// memory: the order of k (and of the output columns) inside a fragment is
// free, so each thread takes 8 (4) neighbouring values in one load.  A x is
// normalised by a power of two per token and split into two FP16 parts
// (22 bits together), so nothing is lost of the FP32 sums and none overflows.
#include <algorithm>

#include "serve.cuh"

namespace tlq {
namespace {

constexpr int kRanks = 8;  // blocks of a cluster
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float peer_f32(const float* p, uint32_t rank) {
  uint32_t a = smem_u32(p), r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

// MT: 16-token tiles of a cluster (1 or 4).  A warp takes one tile and one of
// WK shares of the block's k.
// KR: the most ranks a form takes, in 16s (1, 2 or 4: registers).
template <int MT, int KR>
struct LCfg {
  static constexpr int kMaxRank = 16 * KR;
  static constexpr int TT = 16 * MT;
  static constexpr int WK = kWarps / MT;
  static constexpr int PART = WK * TT * (kMaxRank + 1) * 4;
  static constexpr int SUMS = TT * kMaxRank * 4;
  static constexpr int SPLIT = 2 * TT * (kMaxRank + 8) * 2;
  static constexpr int SMEM = PART + SUMS + SPLIT + TT * 4;
  static_assert(PART % 16 == 0 && SUMS % 16 == 0, "alignment");
};

template <int MT, int KR>
__global__ void __cluster_dims__(kRanks, 1, 1) __launch_bounds__(kThreads, 2) lora_kernel(const LoraArgs a) {
  using C = LCfg<MT, KR>;
  constexpr int kMaxRank = C::kMaxRank;
  constexpr int TT = C::TT, WK = C::WK;
  extern __shared__ __align__(16) uint8_t smem[];
  float(*part)[TT][kMaxRank + 1] = reinterpret_cast<float(*)[TT][kMaxRank + 1]>(smem);  // [WK] A x by share of k
  float(*sums)[kMaxRank] = reinterpret_cast<float(*)[kMaxRank]>(smem + C::PART);        // [TT] of this block's k
  __half(*th)[TT][kMaxRank + 8] = reinterpret_cast<__half(*)[TT][kMaxRank + 8]>(smem + C::PART + C::SUMS);  // [2]
  float* back = reinterpret_cast<float*>(smem + C::PART + C::SUMS + C::SPLIT);          // 2^e * scale of each token
  __shared__ UnitSearch<kThreads> search;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, qd = lane & 3;
  const uint32_t rank = cluster_ctarank();
  pdl_launch_dependents();
  pdl_wait();

  auto length = [&](int i) {
    const int s = a.q_start[i], e = a.q_start[i + 1];
    return s >= 0 && e >= s && e <= a.tokens ? min(e - s, a.max_q) : 0;
  };
  auto count = [&](int i) -> long long { return (length(i) + TT - 1) / TT; };
  long long own, mine;
  search.count_all(a.requests, count, &own, &mine);
  const long long u = blockIdx.x / kRanks;
  if (u >= search.total) return;  // the same for the whole cluster
  search.find(a.requests, count, u, own, mine);
  const int req = search.request;
  const int off = (int)(u - search.first) * TT;
  const int t0 = a.q_start[req] + off;
  const int rows = min(TT, length(req) - off);
  int w = a.adapters[req];
  if (w < 0 || w >= a.num_adapters) w = -1;  // no adapter: y goes through as it is
  const int NR = a.rank, KS = (NR + 15) / 16;

  // Columns of the second product: 32 at a time to a warp; thread qd of a quad
  // holds columns 8 qd .. 8 qd + 7 of its rows.  The first 32 of y and B are
  // asked for here, before A x is known.
  const int blocks32 = (a.N + 31) / 32;
  const int b_lo = (int)((long long)blocks32 * rank / kRanks), b_hi = (int)((long long)blocks32 * (rank + 1) / kRanks);
  const __half* const B = a.B + (size_t)max(w, 0) * a.N * NR;
  uint2 bf[4][kMaxRank / 16];
  uint4 yv[MT][2];
  auto load_columns = [&](int nb) {
    const int n0 = 32 * nb, col = n0 + 8 * qd;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int row = 16 * mt + r + 8 * y;
        if (row < rows && col < a.N)
          yv[mt][y] = *reinterpret_cast<const uint4*>(a.y + (long long)(t0 + row) * a.ldy + col);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + 8 * (r >> 1) + 2 * j + (r & 1);
#pragma unroll
      for (int s = 0; s < kMaxRank / 16; ++s) {
        const int k = 16 * s + 4 * qd;
        bf[j][s] = w >= 0 && n < a.N && k < NR ? __ldg(reinterpret_cast<const uint2*>(B + (size_t)n * NR + k))
                                               : make_uint2(0, 0);
      }
    }
  };
  int nb = b_lo + warp;
  if (nb < b_hi) load_columns(nb);

  if (w >= 0) {
    // ---- A x: this block's k, 32 at a time to a warp ----
    const int chunks = (a.K + 31) / 32;
    const int k_lo = (int)((long long)chunks * rank / kRanks), k_hi = (int)((long long)chunks * (rank + 1) / kRanks);
    const __half* A = a.A + (size_t)w * NR * a.K;
    const int mt = warp % MT, wk = warp / MT;
    float acc[kMaxRank / 8][4];
#pragma unroll
    for (int j = 0; j < kMaxRank / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    const int ra = 16 * mt + r, rb = ra + 8;
    const __half* xa = a.x + (long long)(t0 + min(ra, rows - 1)) * a.ldx;
    const __half* xb = a.x + (long long)(t0 + min(rb, rows - 1)) * a.ldx;
    if (16 * mt < rows) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
      uint4 na = zero, nc = zero;  // x of the next 32 k
      auto load_x = [&](int c) {
        const int k = 32 * c + 8 * qd;
        const bool in = c < k_hi && k < a.K;
        na = in ? *reinterpret_cast<const uint4*>(xa + k) : zero;
        nc = in ? *reinterpret_cast<const uint4*>(xb + k) : zero;
      };
      load_x(k_lo + wk);
      for (int c = k_lo + wk; c < k_hi; c += WK) {
        const uint4 va = na, vb = nc;
        const int k = 32 * c + 8 * qd;
        const bool in = k < a.K;
        uint4 b[kMaxRank / 8];
#pragma unroll
        for (int j = 0; j < kMaxRank / 8; ++j)
          b[j] = in && 8 * j < NR ? __ldg(reinterpret_cast<const uint4*>(A + (size_t)(8 * j + r) * a.K + k)) : zero;
        load_x(c + WK);
#pragma unroll
        for (int j = 0; j < kMaxRank / 8; ++j) {
          if (8 * j < NR) {
            mma_16816(acc[j], va.x, vb.x, va.y, vb.y, b[j].x, b[j].y);
            mma_16816(acc[j], va.z, vb.z, va.w, vb.w, b[j].z, b[j].w);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kMaxRank / 8; ++j) {
      if (8 * j < NR) {
        part[wk][ra][8 * j + 2 * qd] = acc[j][0];
        part[wk][ra][8 * j + 2 * qd + 1] = acc[j][1];
        part[wk][rb][8 * j + 2 * qd] = acc[j][2];
        part[wk][rb][8 * j + 2 * qd + 1] = acc[j][3];
      }
    }
    __syncthreads();
    for (int e = tid; e < TT * NR; e += kThreads) {
      const int row = e / NR, col = e - row * NR;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < WK; ++i) s += part[i][row][col];
      sums[row][col] = s;
    }
  }
  cluster_sync();
  if (w >= 0) {
    // ---- the cluster's sums, in rank order; a warp to a token ----
    const float scale = a.scales[w];
    for (int row = warp; row < TT; row += kWarps) {
      constexpr int VC = (kMaxRank + 31) / 32;  // ranks of a lane
      float v[VC] = {}, big = 0.f;
#pragma unroll
      for (int i = 0; i < VC; ++i) {
        const int col = lane + 32 * i;
        if (col < NR && row < rows) {
          float got[kRanks];
#pragma unroll
          for (uint32_t k = 0; k < kRanks; ++k) got[k] = peer_f32(&sums[row][col], k);
#pragma unroll
          for (uint32_t k = 0; k < kRanks; ++k) v[i] += got[k];
        }
        big = fmaxf(big, fabsf(v[i]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      int e = 0;  // big * 2^-e in [2^14, 2^15); exponents whose powers are normal numbers
      if (big > 0.f && big < INFINITY) e = max(-126, min(126, (int)(__float_as_uint(big) >> 23) - 127 - 14));
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < VC; ++i) {
        const int col = lane + 32 * i;
        if (col < 16 * KS) {
          const float x = v[i] * down;
          const __half hi = __float2half_rn(x);
          th[0][row][col] = hi;
          th[1][row][col] = __float2half_rn(x - __half2float(hi));
        }
      }
      if (lane == 0) back[row] = __uint_as_float((uint32_t)(127 + e) << 23) * scale;
    }
  }
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // this block has read its peers

  // ---- out = y + B (A x) ----
  for (; nb < b_hi; nb += kWarps) {
    const int col = 32 * nb + 8 * qd;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (16 * mt >= rows) break;
      float acc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
      const int ra = 16 * mt + r, rb = ra + 8;
      if (w >= 0) {
#pragma unroll
        for (int s = 0; s < kMaxRank / 16; ++s) {
          if (s < KS) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint2 fa = *reinterpret_cast<const uint2*>(&th[half][ra][16 * s + 4 * qd]);
              const uint2 fb = *reinterpret_cast<const uint2*>(&th[half][rb][16 * s + 4 * qd]);
#pragma unroll
              for (int j = 0; j < 4; ++j) mma_16816(acc[j], fa.x, fb.x, fa.y, fb.y, bf[j][s].x, bf[j][s].y);
            }
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int row = y ? rb : ra;
        if (row < rows && col < a.N) {
          uint4 res = yv[mt][y];
          if (w >= 0) {
            const float up = back[row];
            const uint32_t in[4] = {res.x, res.y, res.z, res.w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&in[j]));
              const __half2 h = __floats2half2_rn(fmaf(acc[j][2 * y], up, f.x), fmaf(acc[j][2 * y + 1], up, f.y));
              o[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
            res = make_uint4(o[0], o[1], o[2], o[3]);
          }
          *reinterpret_cast<uint4*>(a.out + (long long)(t0 + row) * a.ldo + col) = res;
        }
      }
    }
    if (nb + kWarps < b_hi) load_columns(nb + kWarps);
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // no block leaves while a peer reads it
}

// Tiles of 16 MT tokens that the batch can come to, whatever its lengths are.
long long tile_bound(const LoraArgs& a, int mt) {
  return std::min<long long>((long long)a.tokens / (16 * mt) + a.requests,
                             (long long)a.requests * ((a.max_q + 16 * mt - 1) / (16 * mt)));
}

template <int MT, int KR>
tlq_status launch_form(const LoraArgs& a, cudaStream_t stream) {
  const long long tiles = tile_bound(a, MT);
  if (tiles * kRanks > 0x7fffffffll) return set_error(TLQ_EUNSUPPORTED, "lora: %lld token tiles", tiles);
  const cudaError_t attr = opt_in_smem<lora_kernel<MT, KR>>(LCfg<MT, KR>::SMEM);
  if (attr != cudaSuccess) return cuda_error(attr, "lora: shared memory");
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3((unsigned)(tiles * kRanks), 1, 1);
  lc.blockDim = dim3(kThreads, 1, 1);
  lc.dynamicSmemBytes = LCfg<MT, KR>::SMEM;
  lc.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = &at;
  lc.numAttrs = pdl_enabled() ? 1 : 0;
  return cuda_error(cudaLaunchKernelEx(&lc, lora_kernel<MT, KR>, a), "lora: launch");
}

}  // namespace

tlq_status launch_lora(const LoraArgs& a, cudaStream_t stream) {
  // 64-token tiles read A and B a quarter as often; 16-token tiles make more
  // blocks, which matters until every SM has its share.  Measured (K = 2048,
  // N = 6144; 16- against 64-token tiles): rank 16, 660 tokens of 4 requests 12.2
  // against 15.1 us, 1377 of 8 26.4 against 19.7, 4460 of 4 54.4 against 37.4;
  // 653 of 48 15.1 against 19.3.  At ranks above 32 A x and the registers that
  // hold it leave 64-token tiles one block to an SM: 20.1 against 39.4 us for the
  // 660 tokens, 75.1 against 72.5 for the 4460, and 90 against 111 with K = 8192.
  const bool tall = a.rank <= 32 && a.tokens > 1024 && a.tokens / 16 > a.requests;
  if (tall) return a.rank <= 16 ? launch_form<4, 1>(a, stream) : launch_form<4, 2>(a, stream);
  if (a.rank <= 16) return launch_form<1, 1>(a, stream);
  if (a.rank <= 32) return launch_form<1, 2>(a, stream);
  return launch_form<1, 4>(a, stream);
}

}  // namespace tlq
