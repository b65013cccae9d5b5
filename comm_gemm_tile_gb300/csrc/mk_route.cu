// mk_route.cu -- the expert router: top-k experts and gates of every token, rows
// per expert, the balance and z losses, and the gradient with respect to the logits.
//
//   lse = log sum_e exp(l_e);  p_e = exp(l_e - lse)
//   experts: the topk largest l > -inf, ties to the lower number (the rule of mk_moe_dispatch_gemm)
//   gate_k = scale p_k, or scale p_k / sum over the chosen (a softmax over their logits)
//   balance = E sum_e f_e P_e,  f_e = counts_e / (topk N),  P_e = 1/N sum_t p_te;  z = 1/N sum_t lse^2
// over the N tokens that are not masked and have an expert.  Gradient, with the counts held constant:
//   normalised gates  dl_k += gate_k (dg_k - sum_j gate_j dg_j / scale)
//   plain gates       dl_e += p_e (scale dg_e [e chosen] - sum_j scale p_j dg_j)
//   balance           dl_e += db E / N p_e (f_e - sum_j p_j f_j)
//   z                 dl_e += dz 2 lse p_e / N
//
// A warp has a token (and the next one's logits on their way), a lane a run of PER neighbouring
// experts, so that the lowest lane of equal logits is the lowest expert.  Per-expert
// sums of p stay in the lanes' registers, are added over a block's warps in shared
// memory and over the blocks by a second launch, always in the same order.  (Counts
// are whole numbers: shared memory's atomics do for them.)
//
// Choosing: at most two experts, by as many rounds of the largest logit over the warp.
// More: K rounds over the lanes' largest alone give a bound that at least K logits
// reach, and few more; those are gathered one to a lane, in the order of the experts, and
// each counts the larger ones.  (32768 tokens, us, rounds and gathered: 64 experts K 1 11.6 and 13.3, 2 12.7 and 14.0,
// 3 13.3 and 14.0, 8 18.9 and 16.0; 256 experts 1 14.2 and 17.3, 2 16.4 and 17.5, 3 18.4 and 17.4, 8 30.1 and 19.6.)
//
// What bounds it: 131072 tokens of 256 fp32 logits, a tenth of them masked, 8 chosen: 58 us for 129 MB (2.2 TB/s), at 3.3
// instructions a cycle and SM of the 4 that it can start, some 420 a token; more warps do not fit the
// registers.  The gradient: 47 us for 268 MB, 84 % of a copy's rate.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>

#include "mk_seq.cuh"

namespace mk {

namespace {

constexpr int RT_WARPS = 32;           // 131072 tokens, 256 experts: 114 us with the gradient; blocks of 16 warps 121, of 8 130
constexpr int RT_THREADS = 32 * RT_WARPS;
constexpr int RT_BLOCKS = 152;         // blocks of a call at most
constexpr int RS_WARPS = 32;           // of a block that adds the blocks' sums
constexpr int RG_WARPS = 8;            // the gradient's
constexpr int RG_THREADS = 32 * RG_WARPS;

struct RouteParams {
  const char* logits;
  long long row;                       // bytes
  const unsigned char* mask;           // null: every token
  int* idx;                            // [T x K]
  float* gates;                        // [T x K]
  int* counts;                         // [E]
  int* tokens;                         // N
  float* balance;
  float* z;
  float* part;                         // [blocks x (2 E + 2)]: p sums, counts (int), lse^2, N (int)
  int T, E, K, normalize, vec;
  float scale;
  int blocks;
  // gradient
  const float* dgates;                 // null: none
  const float* dbalance;
  const float* dz;
  char* dl;
  long long dl_row;
};

constexpr uint32_t KEY_NONE = 0x007fffffu;     // the key of -inf

// Order-preserving bits: a larger key is a larger logit; -0 as +0, which it ties with.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Two and four sums over a warp: halves of it (quarters) take one each after the first exchange.
__device__ __forceinline__ void warp_sums(float& a, float& b) {
  const bool up = threadIdx.x & 16;
  float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  a = __shfl_sync(0xffffffffu, v, 0);
  b = __shfl_sync(0xffffffffu, v, 16);
}
__device__ __forceinline__ void warp_sums(float& a, float& b, float& c, float& d) {
  const bool up = threadIdx.x & 16, right = threadIdx.x & 8;
  const float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
  const float w = (up ? d : c) + __shfl_xor_sync(0xffffffffu, up ? c : d, 16);
  float u = (right ? w : v) + __shfl_xor_sync(0xffffffffu, right ? v : w, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
  a = __shfl_sync(0xffffffffu, u, 0);
  b = __shfl_sync(0xffffffffu, u, 16);
  c = __shfl_sync(0xffffffffu, u, 8);
  d = __shfl_sync(0xffffffffu, u, 24);
}

// Both losses and N from the sums over tokens: b of counts times p, z of lse^2.
__device__ __forceinline__ void write_losses(const RouteParams& p, float b, float z, int n) {
  const float in = n > 0 ? 1.f / n : 0.f;
  *p.balance = b * in * in * (static_cast<float>(p.E) / p.K);
  *p.z = z * in;
  *p.tokens = n;
}

// The largest of a warp's values; NaN if there is one.
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// exp(x), x <= 0: off by about |x| 2^-24 and 4 2^-24 of itself (ex2.approx's documented 2^-22), 0 below 2^-126.  log(x) and
// 1 / x, x >= 1: lg2.approx is off by 2^-22, past 2 by 2^-22 of itself, rcp.approx by a step.  With expf, logf and a division
// to nearest instead 131072 x 256, 8 experts, takes 70 us forward and 51 back (58 and 47), and gates are off by 6.1e-8 (root mean
// square, relative) for 6.6e-8, gradients by 8.3e-8 for 8.6e-8.
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float LOG2_E = 1.4426950408889634f, LN_2 = 0.6931471805599453f;
__device__ __forceinline__ float exp_of(float x) { return exp2_of(x * LOG2_E); }
__device__ __forceinline__ float log_of(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y * LN_2;
}
__device__ __forceinline__ float inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// v[j] = exp(v[j] - top) and their sum: pairs where there are any.
template <int PER>
__device__ __forceinline__ float exps(float (&v)[PER], float top) {
  if constexpr (PER == 1) {
    v[0] = exp_of(v[0] - top);
    return v[0];
  } else {
    const uint64_t less = two(-top, -top), log2_e = two(LOG2_E, LOG2_E);
    uint64_t sum = 0;
#pragma unroll
    for (int j = 0; j < PER; j += 2) {
      float a, b;
      split(mul2(add2(two(v[j], v[j + 1]), less), log2_e), a, b);
      v[j] = exp2_of(a);
      v[j + 1] = exp2_of(b);
      sum = add2(sum, two(v[j], v[j + 1]));
    }
    float a, b;
    split(sum, a, b);
    return a + b;
  }
}
// s[j] += by v[j]
template <int PER>
__device__ __forceinline__ void add_times(float (&s)[PER], const float (&v)[PER], float by) {
  if constexpr (PER == 1) {
    s[0] = fmaf(v[0], by, s[0]);
  } else {
#pragma unroll
    for (int j = 0; j < PER; j += 2) split(fma2(two(v[j], v[j + 1]), two(by, by), two(s[j], s[j + 1])), s[j], s[j + 1]);
  }
}

// A lane's logits of a token, as they lie; -inf past the last expert.
template <class T, int PER>
struct Logits {
  static constexpr int BYTES = PER * static_cast<int>(sizeof(T));
  T v[PER];
  __device__ __forceinline__ void load(const RouteParams& p, int t) {
    const T* row = reinterpret_cast<const T*>(p.logits + t * p.row) + (threadIdx.x & 31) * PER;
    const int left = p.E - (threadIdx.x & 31) * PER;
    if (p.vec && BYTES >= 4) {                               // all of a lane's, or none
      if (left >= PER) {
        if constexpr (BYTES == 4) copy(__ldg(reinterpret_cast<const uint32_t*>(row)));
        else if constexpr (BYTES == 8) copy(__ldg(reinterpret_cast<const uint2*>(row)));
        else
#pragma unroll
          for (int i = 0; i < BYTES / 16; ++i) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(row) + i);
            memcpy(reinterpret_cast<char*>(v) + 16 * i, &w, 16);
          }
      } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] = Piece<T>::of(-INFINITY);
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) v[j] = j < left ? row[j] : Piece<T>::of(-INFINITY);
    }
  }
  template <class W>
  __device__ __forceinline__ void copy(const W& w) { memcpy(v, &w, sizeof(W)); }
  __device__ __forceinline__ void get(float (&f)[PER]) const {
#pragma unroll
    for (int j = 0; j < PER; ++j) f[j] = Piece<T>::one(v[j]);
  }
};

// The largest K of a warp's values (numbers, or keys), the lowest expert of equal ones first: lane r gets the r-th's
// expert and value.  Those not above `none` are not chosen.
__device__ __forceinline__ uint32_t most_of(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ float most_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ uint32_t warp_most(uint32_t a) { return __reduce_max_sync(0xffffffffu, a); }
__device__ __forceinline__ float warp_most(float a) { return warp_max(a); }
template <int PER, class W>
__device__ __forceinline__ void choose(W (&k)[PER], int K, W none, int lane, int& id, W& value) {
  for (int r = 0; r < K; ++r) {
    W m = k[0];
#pragma unroll
    for (int j = 1; j < PER; ++j) m = most_of(m, k[j]);
    const W best = warp_most(m);
    if (!(best > none)) return;                      // no expert left
    const int owner = __ffs(__ballot_sync(0xffffffffu, m == best)) - 1;
    int at = 0;
    if (lane == owner) {
#pragma unroll
      for (int j = PER - 1; j >= 0; --j)
        if (k[j] == best) at = j;
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (j == at) k[j] = none;
    }
    at = __shfl_sync(0xffffffffu, lane * PER + at, owner);
    if (lane == r) {
      id = at;
      value = best;
    }
  }
}

template <class T, int PER>
__global__ void __launch_bounds__(RT_THREADS) mk_route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ float s_p[RT_WARPS][32 * PER];
  __shared__ int s_c[32 * PER];
  __shared__ __align__(16) float s_value[RT_WARPS][32];      // logits that may be among the chosen,
  __shared__ int s_expert[RT_WARPS][32];                     // in the order of their experts
  __shared__ float s_z[RT_WARPS];
  __shared__ int s_n[RT_WARPS];
  __shared__ float scratch[RT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * PER;
  const uint32_t before = (1u << lane) - 1u;
  griddep_launch_dependents();
  for (int e = threadIdx.x; e < 32 * PER; e += RT_THREADS) s_c[e] = 0;
  __syncthreads();
  float psum[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) psum[j] = 0.f;
  float z = 0.f;
  int n = 0;
  const int step = gridDim.x * RT_WARPS;
  int t = blockIdx.x * RT_WARPS + warp;
  Logits<T, PER> next;
  bool next_real = false;
  auto ahead = [&](int t) {
    next_real = t < p.T && (p.mask == nullptr || p.mask[t] != 0);
    if (next_real) next.load(p, t);
  };
  ahead(t);
  for (; t < p.T; t += step) {
    const Logits<T, PER> now = next;
    const bool real = next_real;
    ahead(t > p.T - step ? p.T : t + step);        // (t + step may pass 2^31)
    int id = -1, slot = lane;                        // this lane's chosen expert, and its place among them
    float w = 0.f;                                   // its gate
    if (real) {
      float v[PER];
      now.get(v);
      float most = v[0];
#pragma unroll
      for (int j = 1; j < PER; ++j) most = max_nan(most, v[j]);
      const float first = warp_max(most);
      float top = first, chosen = -INFINITY;
      bool rounds = p.K <= 2, any = first > -INFINITY;
      if (first != first) {                          // by the keys, in whose order NaN has a place
        uint32_t k[PER], key = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) k[j] = key_of(v[j]);
        choose<PER>(k, p.K, KEY_NONE, lane, id, key);
        top = value_of(__shfl_sync(0xffffffffu, key, 0));
        chosen = id >= 0 ? value_of(key) : -INFINITY;
        any = __shfl_sync(0xffffffffu, id, 0) >= 0;
        rounds = false;
      } else if (!rounds) {
        float m = most, bound = first;
#pragma unroll
        for (int r = 1; r < MOE_MAX_TOPK; ++r) {
          if (r >= p.K) break;
          if (m == bound) m = -INFINITY;
          bound = warp_max(m);
        }
        bound = fmaxf(bound, -FLT_MAX);
        int own = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) own += v[j] >= bound;
        int upto = own;                              // with the lanes' before
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int a = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += a;
        }
        const int count = __shfl_sync(0xffffffffu, upto, 31);
        rounds = count > 32;                         // (many equal logits)
        if (!rounds) {
          int at = upto - own;
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (v[j] >= bound) {
              s_value[warp][at] = v[j];
              s_expert[warp][at++] = e0 + j;
            }
          if (lane >= count) s_value[warp][lane] = -INFINITY;
          __syncwarp();
          const float mine = s_value[warp][lane] + 0.f;      // (-0 is +0's equal)
          int larger = __popc(__match_any_sync(0xffffffffu, __float_as_uint(mine)) & before);
          for (int i = 0; i < count; i += 4) {
            const float4 o = *reinterpret_cast<const float4*>(&s_value[warp][i]);      // the same for every lane
            larger += o.x > mine;
            larger += o.y > mine;
            larger += o.z > mine;
            larger += o.w > mine;
          }
          // the places left over when fewer than K experts have a logit are the lanes' past the list
          slot = lane < count ? larger : lane;
          if (lane < count && larger < p.K) {
            id = s_expert[warp][lane];
            chosen = mine;
          }
          __syncwarp();                              // the list has been read
        }
      }
      if (rounds) {
        float k[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) k[j] = v[j];
        choose<PER>(k, p.K, -INFINITY, lane, id, chosen);
      }
      if (any) {
        w = id >= 0 ? exp_of(chosen - top) : 0.f;
        float sum = exps<PER>(v, top), own = w;      // own: of the chosen ones together
        warp_sums(sum, own);
        const float inv = inverse(sum);
        add_times<PER>(psum, v, inv);
        const float lse = top + log_of(sum);         // (sum is 1 .. 256, its lg2 up to 8: off by 22 2^-24 at most)
        z = fmaf(lse, lse, z);
        ++n;
        w *= (p.normalize ? inverse(own) : inv) * p.scale;
        if (id >= 0) atomicAdd(&s_c[id], 1);
      }
    }
    if (slot < p.K) {
      p.idx[static_cast<long long>(t) * p.K + slot] = id;
      p.gates[static_cast<long long>(t) * p.K + slot] = w;
    }
    if (t > p.T - step) break;
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) s_p[warp][e0 + j] = psum[j];
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = n;
  }
  __syncthreads();
  float* part = p.part + static_cast<long long>(blockIdx.x) * (2 * p.E + 2);
  for (int e = threadIdx.x; e < p.E; e += RT_THREADS) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < RT_WARPS; ++w) a += s_p[w][e];
    if (gridDim.x == 1) {
      s_p[0][e] = a;
    } else {
      part[e] = a;
      reinterpret_cast<int*>(part)[p.E + e] = s_c[e];
    }
  }
  z = 0.f;
  n = 0;
#pragma unroll
  for (int w = 0; w < RT_WARPS; ++w) {
    z += s_z[w];
    n += s_n[w];
  }
  if (gridDim.x > 1) {
    if (threadIdx.x == 0) {
      part[2 * p.E] = z;
      reinterpret_cast<int*>(part)[2 * p.E + 1] = n;
    }
    return;
  }
  // one block: the losses at once
  __syncthreads();
  float b = 0.f;
  for (int e = threadIdx.x; e < p.E; e += RT_THREADS) {
    b += s_p[0][e] * s_c[e];
    p.counts[e] = s_c[e];
  }
  b = warp_sum(b);
  if (lane == 0) scratch[warp] = b;
  __syncthreads();
  if (threadIdx.x == 0) {
    b = 0.f;
#pragma unroll
    for (int w = 0; w < RT_WARPS; ++w) b += scratch[w];
    write_losses(p, b, z, n);
  }
}

// The blocks' sums, in order: a cluster of blocks with 32 experts each, whose shares of the balance loss meet in
// the first.
__global__ void __launch_bounds__(32 * RS_WARPS) mk_route_sums_kernel(const __grid_constant__ RouteParams p) {
  __shared__ float s_p[RS_WARPS][32];
  __shared__ int s_c[RS_WARPS][32];
  __shared__ float share[8];                         // in the first block: every block's
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane, width = 2 * p.E + 2;
  cluster_arrive();                                  // this block has started
  griddep_wait();
  float a = 0.f;
  int c = 0;
  if (e < p.E) {
#pragma unroll 5
    for (int b = warp; b < p.blocks; b += RS_WARPS) {
      a += p.part[static_cast<long long>(b) * width + e];
      c += reinterpret_cast<const int*>(p.part)[static_cast<long long>(b) * width + p.E + e];
    }
  }
  s_p[warp][lane] = a;
  s_c[warp][lane] = c;
  float z = 0.f;
  int n = 0;
  if (blockIdx.x == 0 && warp == 1) {
#pragma unroll 5
    for (int b = lane; b < p.blocks; b += 32) {
      z += p.part[static_cast<long long>(b) * width + 2 * p.E];
      n += reinterpret_cast<const int*>(p.part)[static_cast<long long>(b) * width + 2 * p.E + 1];
    }
    z = warp_sum(z);
    n = __reduce_add_sync(0xffffffffu, n);
  }
  __syncthreads();
  cluster_wait();                                    // so has the first, whose shared memory is stored to
  if (warp == 0) {
    a = 0.f;
    c = 0;
#pragma unroll
    for (int w = 0; w < RS_WARPS; ++w) {
      a += s_p[w][lane];
      c += s_c[w][lane];
    }
    if (e < p.E) p.counts[e] = c;
    const float b = warp_sum(a * c);
    if (lane == 0) st_shared_cluster_f32(mapa_shared(smem_u32(&share[blockIdx.x]), 0), b);
    __syncwarp();
  }
  cluster_sync_all();
  if (blockIdx.x == 0 && threadIdx.x == 32) {
    float b = 0.f;
    for (unsigned w = 0; w < gridDim.x; ++w) b += share[w];
    write_losses(p, b, z, n);
  }
}

template <class T, int PER>
__global__ void __launch_bounds__(RG_THREADS) mk_route_grad_kernel(const __grid_constant__ RouteParams p) {
  __shared__ __align__(16) float s_add[RG_WARPS][32 * PER];      // what the chosen experts get besides
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * PER;
  const int n = max(1, *p.tokens);
  const float db = p.dbalance ? *p.dbalance * (static_cast<float>(p.E) / n) : 0.f;
  const float dz = p.dz ? *p.dz * (2.f / n) : 0.f;
  float f[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    f[j] = p.dbalance && e0 + j < p.E ? p.counts[e0 + j] / (static_cast<float>(p.K) * n) : 0.f;
    s_add[warp][e0 + j] = 0.f;
  }
  __syncwarp();
  const int step = gridDim.x * RG_WARPS;
  int t = blockIdx.x * RG_WARPS + warp;
  Logits<T, PER> next;
  int next_id = -1;
  float next_dg = 0.f;
  auto ahead = [&](int t) {
    next_id = -1;
    if (t >= p.T) return;
    next.load(p, t);
    if (lane < p.K) {
      next_id = p.idx[static_cast<long long>(t) * p.K + lane];
      if (p.dgates != nullptr) next_dg = p.dgates[static_cast<long long>(t) * p.K + lane];
    }
  };
  ahead(t);
  for (; t < p.T; t += step) {
    const Logits<T, PER> now = next;
    int id = next_id;
    float dg = next_dg * p.scale;
    ahead(t > p.T - step ? p.T : t + step);        // (t + step may pass 2^31)
    const bool real = __shfl_sync(0xffffffffu, id, 0) >= 0;
    float d[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) d[j] = 0.f;
    if (real) {
      float v[PER];
      now.get(v);
      float top = v[0];
#pragma unroll
      for (int j = 1; j < PER; ++j) top = max_nan(top, v[j]);
      top = warp_max(top);
      float sum = exps<PER>(v, top), pf = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) pf = fmaf(v[j], f[j], pf);
      const bool chosen = p.dgates != nullptr && id >= 0 && id < p.E;
      float w = 0.f;                                 // exp(logit - top) of this lane's chosen expert
      if (chosen) w = exp_of(Piece<T>::one(reinterpret_cast<const T*>(p.logits + t * p.row)[id]) - top);
      else dg = 0.f;
      float own = w;                                 // of the chosen ones together
      float dot = w * dg;
      if (p.dgates != nullptr) warp_sums(sum, pf, own, dot);
      else warp_sums(sum, pf);
      const float inv = inverse(sum), lse = top + log_of(sum);
      const float part = p.normalize ? inverse(own) : inv;
      dot *= part;
      const float mine = w * part * (p.normalize ? dg - dot : dg);
      const float all = (p.normalize || p.dgates == nullptr ? 0.f : -dot) - db * pf * inv + dz * lse;
      if (p.dgates != nullptr) {
        if (chosen) s_add[warp][id] = mine;          // (a token's experts differ)
        __syncwarp();
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) d[j] = v[j] * inv * fmaf(db, f[j], all);
      if (p.dgates != nullptr) {
#pragma unroll
        for (int j = 0; j < PER; ++j) d[j] += s_add[warp][e0 + j];
        __syncwarp();
        if (chosen) s_add[warp][id] = 0.f;
        __syncwarp();
      }
    }
    T* out = reinterpret_cast<T*>(p.dl + t * p.dl_row) + e0;
    const int left = p.E - e0;
    constexpr int BYTES = Logits<T, PER>::BYTES;
    if (p.vec && BYTES >= 4) {
      if (left >= PER) {
        T o[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) o[j] = Piece<T>::of(d[j]);
        if constexpr (BYTES == 4) {
          uint32_t w;
          memcpy(&w, o, 4);
          *reinterpret_cast<uint32_t*>(out) = w;
        } else if constexpr (BYTES == 8) {
          uint2 w;
          memcpy(&w, o, 8);
          *reinterpret_cast<uint2*>(out) = w;
        } else {
#pragma unroll
          for (int i = 0; i < BYTES / 16; ++i) {
            uint4 w;
            memcpy(&w, reinterpret_cast<char*>(o) + 16 * i, 16);
            reinterpret_cast<uint4*>(out)[i] = w;
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (j < left) out[j] = Piece<T>::of(d[j]);
    }
    if (t > p.T - step) break;
  }
}

// ------------------------------------------------------------------ host

// Up to MK_ROUTE_SMALL tokens one block, which writes the losses itself: 64 tokens 5.2 us (96: 6.2, and 5.6 by many
// blocks and a second launch; 256: 12.0 and 5.3).
int route_blocks(long long T) {
  if (T <= MK_ROUTE_SMALL) return 1;
  return static_cast<int>(std::min<long long>(ceil_div_ll(T, RT_WARPS), RT_BLOCKS));
}

template <class T, int PER>
cudaError_t launch_route(RouteParams p, bool grad, cudaStream_t s) {
  // whole pieces of PER logits, where every row has them
  const uintptr_t piece = PER * sizeof(T) < 16 ? PER * sizeof(T) : 16;
  uintptr_t lie = reinterpret_cast<uintptr_t>(p.logits) | (p.T > 1 ? static_cast<uintptr_t>(p.row) : 0);
  if (grad) lie |= reinterpret_cast<uintptr_t>(p.dl) | (p.T > 1 ? static_cast<uintptr_t>(p.dl_row) : 0);
  p.vec = p.E % PER == 0 && !(lie & (piece - 1));
  if (grad) mk_route_grad_kernel<T, PER><<<p.blocks, RG_THREADS, 0, s>>>(p);
  else mk_route_kernel<T, PER><<<p.blocks, RT_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <class T>
cudaError_t launch_route(const RouteParams& p, bool grad, cudaStream_t s) {
  if (p.E <= 32) return launch_route<T, 1>(p, grad, s);
  if (p.E <= 64) return launch_route<T, 2>(p, grad, s);
  if (p.E <= 128) return launch_route<T, 4>(p, grad, s);
  return launch_route<T, 8>(p, grad, s);
}
cudaError_t launch_route(const RouteParams& p, mk_dtype dtype, bool grad, cudaStream_t s) {
  if (dtype == MK_F32) return launch_route<float>(p, grad, s);
  if (dtype == MK_BF16) return launch_route<__nv_bfloat16>(p, grad, s);
  return launch_route<__half>(p, grad, s);
}

bool route_ok(mk_dtype dtype, long long T, int E, int topk, float scale) {
  if (dtype != MK_F32 && dtype != MK_BF16 && dtype != MK_F16) return false;
  if (T < 0 || T >= (1LL << 31) || E < 1 || E > MOE_MAX_E || topk < 1 || topk > MOE_MAX_TOPK || topk > E) return false;
  return std::isfinite(scale);
}
bool aligned(const void* p, unsigned to) { return !(reinterpret_cast<uintptr_t>(p) & (to - 1)); }

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

size_t mk_moe_route_workspace_size(long long T, int E) {
  if (!route_ok(MK_F32, T, E, 1, 1.f)) return 0;
  return static_cast<size_t>(route_blocks(T)) * (2 * E + 2) * sizeof(float);
}

mk_status mk_moe_route(const void* logits, mk_dtype dtype, long long T, int E, long long row, int topk, int normalize,
                       float scale, const unsigned char* mask, int* topk_idx, float* gates, int* counts, int* tokens,
                       float* balance_loss, float* z_loss, void* workspace, size_t ws_bytes, mk_stream_t stream) {
  if (!route_ok(dtype, T, E, topk, scale)) return MK_ERR_INVALID;
  const unsigned esz = dtype == MK_F32 ? 4 : 2;
  if (T > 0 && (!logits || !topk_idx || !gates)) return MK_ERR_INVALID;
  if (!counts || !tokens || !balance_loss || !z_loss) return MK_ERR_INVALID;
  if (!aligned(logits, esz) || !aligned(topk_idx, 4) || !aligned(gates, 4) || !aligned(counts, 4) || !aligned(tokens, 4) ||
      !aligned(balance_loss, 4) || !aligned(z_loss, 4))
    return MK_ERR_INVALID;
  RouteParams p;
  std::memset(&p, 0, sizeof(p));
  p.blocks = route_blocks(T);
  if (p.blocks > 1 && (!workspace || !aligned(workspace, 16) || ws_bytes < mk_moe_route_workspace_size(T, E)))
    return MK_ERR_INVALID;
  p.logits = static_cast<const char*>(logits);
  p.row = row * esz;
  p.mask = mask;
  p.idx = topk_idx;
  p.gates = gates;
  p.counts = counts;
  p.tokens = tokens;
  p.balance = balance_loss;
  p.z = z_loss;
  p.part = static_cast<float*>(workspace);
  p.T = static_cast<int>(T);
  p.E = E;
  p.K = topk;
  p.normalize = normalize != 0;
  p.scale = scale;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_route(p, dtype, false, s);
  if (e == cudaSuccess && p.blocks > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : 8);
    cfg.blockDim = dim3(32 * RS_WARPS);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cfg.gridDim.x;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, mk_route_sums_kernel, p);
  }
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

mk_status mk_moe_route_backward(const void* logits, mk_dtype dtype, long long T, int E, long long row, int topk,
                                int normalize, float scale, const int* topk_idx, const int* counts, const int* tokens,
                                const float* dgates, const float* dbalance, const float* dz, void* dlogits,
                                long long dl_row, mk_stream_t stream) {
  if (!route_ok(dtype, T, E, topk, scale)) return MK_ERR_INVALID;
  if (T == 0) return MK_OK;
  const unsigned esz = dtype == MK_F32 ? 4 : 2;
  if (!logits || !topk_idx || !counts || !tokens || !dlogits || (dl_row == 0 && T > 1)) return MK_ERR_INVALID;
  if (!aligned(logits, esz) || !aligned(dlogits, esz) || !aligned(topk_idx, 4) || !aligned(counts, 4) ||
      !aligned(tokens, 4) || !aligned(dgates, 4) || !aligned(dbalance, 4) || !aligned(dz, 4))
    return MK_ERR_INVALID;
  RouteParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = static_cast<const char*>(logits);
  p.row = row * esz;
  p.idx = const_cast<int*>(topk_idx);
  p.counts = const_cast<int*>(counts);
  p.tokens = const_cast<int*>(tokens);
  p.dgates = dgates;
  p.dbalance = dbalance;
  p.dz = dz;
  p.dl = static_cast<char*>(dlogits);
  p.dl_row = dl_row * esz;
  p.T = static_cast<int>(T);
  p.E = E;
  p.K = topk;
  p.normalize = normalize != 0;
  p.scale = scale;
  p.blocks = static_cast<int>(std::min<long long>(ceil_div_ll(T, RG_WARPS), 4 * RT_BLOCKS));
  const cudaError_t e = launch_route(p, dtype, true, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // extern "C"
