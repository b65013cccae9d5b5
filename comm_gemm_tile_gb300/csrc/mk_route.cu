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
// A warp has a token, a lane a run of PER neighbouring experts, so that the
// lowest lane of equal logits is the lowest expert.  Per-expert sums stay in the
// lanes' registers, are added over a block's warps in shared memory and over the
// blocks by a second launch, always in the same order.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk_seq.cuh"

namespace mk {

namespace {

constexpr int RT_WARPS = 8;
constexpr int RT_THREADS = 32 * RT_WARPS;
constexpr int RT_BLOCKS = 304;         // blocks of a call at most

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

// A lane's logits of a token; -inf past the last expert.
template <class T, int PER>
__device__ __forceinline__ void load_logits(const RouteParams& p, int t, float (&v)[PER]) {
  const T* row = reinterpret_cast<const T*>(p.logits + t * p.row);
  const int e0 = (threadIdx.x & 31) * PER;
#pragma unroll
  for (int j = 0; j < PER; ++j) v[j] = e0 + j < p.E ? Piece<T>::one(row[e0 + j]) : -INFINITY;
}

__device__ void finish(const RouteParams& p, const float* sp, const int* sc, float z, int n, float* scratch) {
  // sp, sc: [E] sums of p and counts; by the whole block
  const float f = n > 0 ? 1.f / (static_cast<float>(p.K) * n) : 0.f, in = n > 0 ? 1.f / n : 0.f;
  float b = 0.f;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    b += sc[e] * f * (sp[e] * in);
    p.counts[e] = sc[e];
  }
  b = warp_sum(b);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = b;
  __syncthreads();
  if (threadIdx.x == 0) {
    b = 0.f;
    for (unsigned w = 0; w < blockDim.x / 32; ++w) b += scratch[w];
    *p.balance = b * p.E;
    *p.z = z * in;
    *p.tokens = n;
  }
}

template <class T, int PER>
__global__ void __launch_bounds__(RT_THREADS) mk_route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ float s_p[RT_WARPS][32 * PER];
  __shared__ int s_c[RT_WARPS][32 * PER];
  __shared__ float s_z[RT_WARPS];
  __shared__ int s_n[RT_WARPS];
  __shared__ float scratch[RT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * PER;
  griddep_launch_dependents();
  float psum[PER];
  int cnt[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    psum[j] = 0.f;
    cnt[j] = 0;
  }
  float z = 0.f;
  int n = 0;
  for (int t = blockIdx.x * RT_WARPS + warp; t < p.T; t += gridDim.x * RT_WARPS) {
    int my_idx = -1;
    float my_gate = 0.f;
    if (p.mask == nullptr || p.mask[t] != 0) {
      float v[PER];
      uint32_t k[PER];
      load_logits<T, PER>(p, t, v);
#pragma unroll
      for (int j = 0; j < PER; ++j) k[j] = key_of(v[j]);
      float top = 0.f, chosen = 0.f;
      for (int r = 0; r < p.K; ++r) {
        uint32_t m = k[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) m = max(m, k[j]);
        const uint32_t best = __reduce_max_sync(0xffffffffu, m);
        if (best <= KEY_NONE) break;                     // no expert left
        const int owner = __ffs(__ballot_sync(0xffffffffu, m == best)) - 1;
        int at = 0;
        if (lane == owner) {
#pragma unroll
          for (int j = PER - 1; j >= 0; --j)
            if (k[j] == best) at = j;
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (j == at) {
              k[j] = 0;
              ++cnt[j];
            }
        }
        at = __shfl_sync(0xffffffffu, e0 + at, owner);
        const float value = value_of(best);
        if (r == 0) top = value;
        const float w = expf(value - top);
        chosen += w;
        if (lane == r) {
          my_idx = at;
          my_gate = w;
        }
      }
      if (__shfl_sync(0xffffffffu, my_idx, 0) >= 0) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          v[j] = expf(v[j] - top);
          sum += v[j];
        }
        sum = warp_sum(sum);
        const float inv = 1.f / sum;
#pragma unroll
        for (int j = 0; j < PER; ++j) psum[j] += v[j] * inv;
        const float lse = top + logf(sum);
        z += lse * lse;
        ++n;
        my_gate = my_gate / (p.normalize ? chosen : sum) * p.scale;
      }
    }
    if (lane < p.K) {
      p.idx[static_cast<long long>(t) * p.K + lane] = my_idx;
      p.gates[static_cast<long long>(t) * p.K + lane] = my_gate;
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    s_p[warp][e0 + j] = psum[j];
    s_c[warp][e0 + j] = cnt[j];
  }
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = n;
  }
  __syncthreads();
  float* part = p.part + static_cast<long long>(blockIdx.x) * (2 * p.E + 2);
  for (int e = threadIdx.x; e < p.E; e += RT_THREADS) {
    float a = 0.f;
    int c = 0;
#pragma unroll
    for (int w = 0; w < RT_WARPS; ++w) {
      a += s_p[w][e];
      c += s_c[w][e];
    }
    if (gridDim.x == 1) {
      s_p[0][e] = a;
      s_c[0][e] = c;
    } else {
      part[e] = a;
      reinterpret_cast<int*>(part)[p.E + e] = c;
    }
  }
  z = 0.f;
  n = 0;
#pragma unroll
  for (int w = 0; w < RT_WARPS; ++w) {
    z += s_z[w];
    n += s_n[w];
  }
  if (gridDim.x == 1) {
    __syncthreads();
    finish(p, s_p[0], s_c[0], z, n, scratch);
  } else if (threadIdx.x == 0) {
    part[2 * p.E] = z;
    reinterpret_cast<int*>(part)[2 * p.E + 1] = n;
  }
}

// One block: the blocks' sums in order, then the losses.
__global__ void __launch_bounds__(1024) mk_route_sums_kernel(const __grid_constant__ RouteParams p) {
  __shared__ float s_p[4][256 + 2];
  __shared__ int s_c[4][256 + 2];
  __shared__ float scratch[32];
  const int e = threadIdx.x & 255, q = threadIdx.x >> 8, width = 2 * p.E + 2;
  griddep_wait();
  float a = 0.f;
  int c = 0;
  if (e < p.E) {
#pragma unroll 4
    for (int b = q; b < p.blocks; b += 4) {
      a += p.part[static_cast<long long>(b) * width + e];
      c += reinterpret_cast<const int*>(p.part)[static_cast<long long>(b) * width + p.E + e];
    }
    s_p[q][e] = a;
    s_c[q][e] = c;
  }
  float z = 0.f;
  int n = 0;
  if (threadIdx.x < 32) {
    for (int b = threadIdx.x; b < p.blocks; b += 32) {
      z += p.part[static_cast<long long>(b) * width + 2 * p.E];
      n += reinterpret_cast<const int*>(p.part)[static_cast<long long>(b) * width + 2 * p.E + 1];
    }
    z = warp_sum(z);
    n = __reduce_add_sync(0xffffffffu, n);
    if (threadIdx.x == 0) {
      s_p[0][256] = z;
      s_c[0][256] = n;
    }
  }
  __syncthreads();
  if (threadIdx.x < p.E) {
    s_p[0][e] = s_p[0][e] + s_p[1][e] + s_p[2][e] + s_p[3][e];
    s_c[0][e] = s_c[0][e] + s_c[1][e] + s_c[2][e] + s_c[3][e];
  }
  __syncthreads();
  finish(p, s_p[0], s_c[0], s_p[0][256], s_c[0][256], scratch);
}

template <class T, int PER>
__global__ void __launch_bounds__(RT_THREADS) mk_route_grad_kernel(const __grid_constant__ RouteParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * PER;
  const int n = max(1, *p.tokens);
  const float db = p.dbalance ? *p.dbalance * (static_cast<float>(p.E) / n) : 0.f;
  const float dz = p.dz ? *p.dz * (2.f / n) : 0.f;
  float f[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j)
    f[j] = p.dbalance && e0 + j < p.E ? p.counts[e0 + j] / (static_cast<float>(p.K) * n) : 0.f;
  for (int t = blockIdx.x * RT_WARPS + warp; t < p.T; t += gridDim.x * RT_WARPS) {
    T* out = reinterpret_cast<T*>(p.dl + t * p.dl_row);
    const int id = lane < p.K ? p.idx[static_cast<long long>(t) * p.K + lane] : -1;
    float d[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) d[j] = 0.f;
    if (__shfl_sync(0xffffffffu, id, 0) >= 0) {
      float v[PER];
      load_logits<T, PER>(p, t, v);
      float top = v[0];
#pragma unroll
      for (int j = 1; j < PER; ++j) top = fmaxf(top, v[j]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      float sum = 0.f, pf = 0.f;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        v[j] = expf(v[j] - top);
        sum += v[j];
        pf = fmaf(v[j], f[j], pf);
      }
      sum = warp_sum(sum);
      pf = warp_sum(pf);
      const float inv = 1.f / sum, lse = top + logf(sum);
      float dg = 0.f, w = 0.f;                       // of lane k's chosen expert
      if (p.dgates != nullptr && id >= 0 && id < p.E) {
        dg = p.dgates[static_cast<long long>(t) * p.K + lane] * p.scale;
        w = expf(Piece<T>::one(reinterpret_cast<const T*>(p.logits + t * p.row)[id]) - top);
      }
      const float share = w / (p.normalize ? warp_sum(w) : sum);
      const float dot = warp_sum(share * dg);
      const float mine = share * (p.normalize ? dg - dot : dg);
      const float all = (p.normalize || p.dgates == nullptr ? 0.f : -dot) - db * pf * inv + dz * lse;
#pragma unroll
      for (int j = 0; j < PER; ++j) d[j] = v[j] * inv * (fmaf(db, f[j], all));
      if (p.dgates != nullptr)
        for (int k = 0; k < p.K; ++k) {
          const int at = __shfl_sync(0xffffffffu, id, k) - e0;
          const float c = __shfl_sync(0xffffffffu, mine, k);
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (j == at) d[j] += c;
        }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (e0 + j < p.E) out[e0 + j] = Piece<T>::of(d[j]);
  }
}

// ------------------------------------------------------------------ host

int route_blocks(long long T) {
  if (T <= MK_ROUTE_SMALL) return 1;
  return static_cast<int>(std::min<long long>(ceil_div_ll(T, RT_WARPS), RT_BLOCKS));
}

template <class T, int PER>
cudaError_t launch_route(const RouteParams& p, bool grad, cudaStream_t s) {
  if (grad) mk_route_grad_kernel<T, PER><<<p.blocks, RT_THREADS, 0, s>>>(p);
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
  if (e == cudaSuccess && p.blocks > 1) e = launch_dependent(mk_route_sums_kernel, dim3(1), dim3(1024), s, p);
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
  p.blocks = static_cast<int>(std::min<long long>(ceil_div_ll(T, RT_WARPS), 4 * RT_BLOCKS));
  const cudaError_t e = launch_route(p, dtype, true, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // extern "C"
