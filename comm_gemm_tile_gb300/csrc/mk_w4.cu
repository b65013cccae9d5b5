// mk_w4.cu -- few rows times a matrix of 4-bit weights with group scales.
//
//   y[m][n] = sum_k x[m][k] s[n][k / G] (c[n][k] - z[n][k / G]),   z = 8 without zero points
//
// Codes become 16-bit numbers exactly (c - 8 is a whole number of 4 bits), are
// multiplied with x on the tensor cores in fp32, and a group's sum is multiplied
// by its scale in fp32: nothing is rounded before the output.  Zero points enter
// as (8 - z) sum_k x[m][k] of the group, from one more product with ones.
//
// Here: few tokens, 8, 16 or 32 at a time (more of them, and large matrices, go to mk_w4_tiles.cu).  The products are mma.sync
// m16n8k16 with weights as the 16 rows and 8 tokens as the columns, one for each 8 of them.  They sum over k in any
// order, so a thread's own codes are its operands as they come, and x is read in the same order.  A block
// has 16 rows of the matrix; its warps share out k in pieces of 128, a thread 16 bytes
// (32 codes) of two rows of each, loaded one piece ahead, and add their sums in shared memory, in order.
//
// What bounds it: instructions, some 170 of a warp for 16 x 128 weights (28672 x 8192, groups of 128, one token: 36 us,
// 3.4 TB/s), and at small matrices how many pieces a warp has one after the other: the warps of an SM are shared by as many blocks as
// leave the fewest (1024 x 8192, one token, weights out of L2: 9.0 us with 8 warps a block, 5.0 with 32; 2432 x 16384 16.5 and 7.9;
// 8192 x 8192, groups of 64 with zero points 24 and 18).  More pieces ahead or two tiles of rows a
// block cost registers and with them warps; a ring of shared memory took half as long again.
// Columns past the last token hold another token's x and are dropped.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk_w4.h"

namespace mk {

namespace {

// Warps of an SM, and of a block at most, for TILES times 8 tokens: 64, 80, 102 or 128 registers a thread.
template <int WPG, bool ZEROS, int TILES>
constexpr int W4_WARPS = TILES == 1 ? (ZEROS || WPG == 1 ? 24 : 32) : TILES == 2 ? (ZEROS ? 20 : 24) : 16;
constexpr int W4_SMS = 152;
constexpr int W4_TOKENS = 8;
constexpr int W4_ROWS = 16;

template <class T>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What a thread has of a piece: the words of its two rows by group, scales and zero points.
template <class T, int GPC, bool ZEROS>
struct Step {
  uint32_t w[2][4];
  T s[2][GPC], z[2][ZEROS ? GPC : 1];
};

// 1, 2 or 4 neighbouring scales.
template <class T, int N>
__device__ __forceinline__ void read_groups(const T* p, T (&v)[N]) {
  if constexpr (N == 1) v[0] = *p;
  else if constexpr (N == 2) {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p));
    memcpy(v, &w, 4);
  } else {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    memcpy(v, &w, 8);
  }
}

// WPG: words of a thread in a group (4, 2, 1 for groups of 128, 64, 32).  WHOLE: k is whole pieces, whose scales
// (and zero points) lie on 8, 4 or 2 bytes.
template <class T, int WPG, bool ZEROS, bool WHOLE, int TILES>
__global__ void __launch_bounds__(32 * W4_WARPS<WPG, ZEROS, TILES>) mk_w4_kernel(const __grid_constant__ W4Params p) {
  constexpr int GPC = 4 / WPG;                       // groups of a piece
  __shared__ float red[W4_WARPS<WPG, ZEROS, TILES>][TILES * W4_TOKENS][W4_ROWS + 1];
  const int warps = blockDim.x >> 5;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, j = lane & 3;
  const int n0 = blockIdx.x * W4_ROWS;
  const uint8_t* codes[2];
  const T *scales[2], *zeros[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int row = min(n0 + 8 * t + r, p.n - 1);    // rows past the last repeat it
    codes[t] = p.codes + static_cast<long long>(row) * (p.k / 2) + j * (WPG * 4);
    scales[t] = static_cast<const T*>(p.scales) + static_cast<long long>(row) * p.groups;
    zeros[t] = static_cast<const T*>(p.zeros) + static_cast<long long>(row) * p.groups;
  }
  const int t0 = TILES == 4 ? blockIdx.y * (TILES * W4_TOKENS) : 0;
  const char* x[TILES];
#pragma unroll
  for (int i = 0; i < TILES; ++i) x[i] = p.x + min(t0 + 8 * i + r, p.m - 1) * p.x_row + j * (WPG * 16);
  const int pieces = (p.k + W4_PIECE - 1) / W4_PIECE;
  auto load = [&](int c, Step<T, GPC, ZEROS>& o) {
    if (WHOLE && c >= pieces) return;
#pragma unroll
    for (int g = 0; g < GPC; ++g) {
      const int group = c * GPC + g;
      const bool real = WHOLE || group < p.groups;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const uint8_t* a = codes[t] + group * (WPG * 16);
        if constexpr (WPG == 4) {
          const uint4 u = real ? ld_nc_v4(a) : make_uint4(0, 0, 0, 0);
          o.w[t][0] = u.x; o.w[t][1] = u.y; o.w[t][2] = u.z; o.w[t][3] = u.w;
        } else if constexpr (WPG == 2) {
          const uint2 u = real ? __ldg(reinterpret_cast<const uint2*>(a)) : make_uint2(0, 0);
          o.w[t][2 * g] = u.x; o.w[t][2 * g + 1] = u.y;
        } else {
          o.w[t][g] = real ? __ldg(reinterpret_cast<const uint32_t*>(a)) : 0;
        }
        if constexpr (!WHOLE) {
          o.s[t][g] = real ? scales[t][group] : Piece<T>::of(0.f);
          if constexpr (ZEROS) o.z[t][g] = real ? zeros[t][group] : Piece<T>::of(0.f);
        }
      }
    }
    if constexpr (WHOLE) {                           // a piece's at once: one at a time 1024 x 8192, groups of 32, took 11.7 us
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        read_groups(scales[t] + c * GPC, o.s[t]);
        if constexpr (ZEROS) read_groups(zeros[t] + c * GPC, o.z[t]);
      }
    }
  };
  float acc[TILES][4];
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  auto multiply = [&](int c, const Step<T, GPC, ZEROS>& now) {
#pragma unroll
    for (int g = 0; g < GPC; ++g) {
      const int group = c * GPC + g;
      float part[TILES][4], ones[TILES][4];
#pragma unroll
      for (int i = 0; i < TILES; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[i][e] = ones[i][e] = 0.f;
#pragma unroll
      for (int w = 0; w < WPG; ++w) {
        uint32_t a[4], b[4];
        Codes<T>::pairs(now.w[0][g * WPG + w], a);
        Codes<T>::pairs(now.w[1][g * WPG + w], b);
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
          uint32_t xs[4];
          const uint4 v = WHOLE || group < p.groups ? __ldg(reinterpret_cast<const uint4*>(x[i] + group * (WPG * 64)) + w) : make_uint4(0, 0, 0, 0);
          x_pairs(v, xs);
          mma<T>(part[i], a[0], b[0], a[1], b[1], xs[0], xs[1]);
          mma<T>(part[i], a[2], b[2], a[3], b[3], xs[2], xs[3]);
          if constexpr (ZEROS) {
            constexpr uint32_t I = Codes<T>::ONES;
            mma<T>(ones[i], I, I, I, I, xs[0], xs[1]);
            mma<T>(ones[i], I, I, I, I, xs[2], xs[3]);
          }
        }
      }
      const float fa = Piece<T>::one(now.s[0][g]), fb = Piece<T>::one(now.s[1][g]);
#pragma unroll
      for (int i = 0; i < TILES; ++i) {
        if constexpr (ZEROS) {
          const float oa = 8.f - Piece<T>::one(now.z[0][g]), ob = 8.f - Piece<T>::one(now.z[1][g]);
          part[i][0] = fmaf(oa, ones[i][0], part[i][0]);
          part[i][1] = fmaf(oa, ones[i][1], part[i][1]);
          part[i][2] = fmaf(ob, ones[i][2], part[i][2]);
          part[i][3] = fmaf(ob, ones[i][3], part[i][3]);
        }
        acc[i][0] = fmaf(fa, part[i][0], acc[i][0]);
        acc[i][1] = fmaf(fa, part[i][1], acc[i][1]);
        acc[i][2] = fmaf(fb, part[i][2], acc[i][2]);
        acc[i][3] = fmaf(fb, part[i][3], acc[i][3]);
      }
    }
  };
  Step<T, GPC, ZEROS> next;
  if (warp < pieces) load(warp, next);
  for (int c = warp; c < pieces; c += warps) {
    const Step<T, GPC, ZEROS> now = next;
    load(c + warps, next);
    multiply(c, now);
  }
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp][8 * i + 2 * j + (e & 1)][r + 8 * (e >> 1)] = acc[i][e];
  __syncthreads();
  const int row = threadIdx.x % W4_ROWS;
  if (n0 + row >= p.n) return;
  for (int t = threadIdx.x / W4_ROWS; t < min(p.m - t0, TILES * W4_TOKENS); t += blockDim.x / W4_ROWS) {
    float s = 0.f;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) s += red[w][t][row];
    w4_store<T>(p, t0 + t, n0 + row, s);
  }
}

// ------------------------------------------------------------------ host

// Warps of a block: those of an SM shared by 4 to 1 blocks, whichever leaves the fewest turns (waves of blocks times pieces a
// warp), then no more than the turns need.
int warps_of(int blocks, int pieces, int most) {
  int warps = 0, least = 0;
  for (int b = 4; b >= 1; --b) {
    const int w = std::min(most / b, pieces), turns = (blocks + W4_SMS * b - 1) / (W4_SMS * b) * ((pieces + w - 1) / w);
    if (warps == 0 || turns < least) {
      warps = w;
      least = turns;
    }
  }
  const int turns = (pieces + warps - 1) / warps;
  return (pieces + turns - 1) / turns;
}

template <class T, int WPG, bool ZEROS, bool WHOLE, int TILES>
cudaError_t launch_w4(const W4Params& p, cudaStream_t s) {
  const int grid = static_cast<int>(ceil_div_ll(p.n, W4_ROWS)), passes = (p.m + TILES * W4_TOKENS - 1) / (TILES * W4_TOKENS);
  const int warps = warps_of(grid * passes, (p.k + W4_PIECE - 1) / W4_PIECE, W4_WARPS<WPG, ZEROS, TILES>);
  mk_w4_kernel<T, WPG, ZEROS, WHOLE, TILES><<<dim3(grid, passes), 32 * warps, 0, s>>>(p);
  return cudaGetLastError();
}
template <class T, int WPG, bool ZEROS, bool WHOLE>
cudaError_t launch_w4(const W4Params& p, cudaStream_t s) {
  if (p.m <= 8) return launch_w4<T, WPG, ZEROS, WHOLE, 1>(p, s);
  return p.m <= 16 ? launch_w4<T, WPG, ZEROS, WHOLE, 2>(p, s) : launch_w4<T, WPG, ZEROS, WHOLE, 4>(p, s);
}
template <class T, int WPG, bool ZEROS>
cudaError_t launch_w4(const W4Params& p, cudaStream_t s) {
  const uintptr_t lie = reinterpret_cast<uintptr_t>(p.scales) | reinterpret_cast<uintptr_t>(p.zeros);
  const bool whole = p.k % W4_PIECE == 0 && !(lie & (8 / WPG - 1));
  return whole ? launch_w4<T, WPG, ZEROS, true>(p, s) : launch_w4<T, WPG, ZEROS, false>(p, s);
}
template <class T, int WPG>
cudaError_t launch_w4(const W4Params& p, cudaStream_t s) {
  return p.zeros ? launch_w4<T, WPG, true>(p, s) : launch_w4<T, WPG, false>(p, s);
}
template <class T>
cudaError_t launch_w4(const W4Params& p, int group, cudaStream_t s) {
  if (group == 128) return launch_w4<T, 4>(p, s);
  return group == 64 ? launch_w4<T, 2>(p, s) : launch_w4<T, 1>(p, s);
}

bool weight_ok(const mk_w4_weight* w, long long m) {
  if (!w || (w->dtype != MK_BF16 && w->dtype != MK_F16)) return false;
  if (w->group != 32 && w->group != 64 && w->group != 128) return false;
  if (w->n < 0 || w->n >= (1LL << 31) || w->k < w->group || w->k % w->group || w->k >= (1LL << 30)) return false;
  // steps of 128 x 128 weights for 16 tokens are counted in 31 bits
  return m >= 0 && m < (1LL << 24) && (w->n / 128 + 1) * (w->k / 128 + 1) < (1LL << 31) / (m / 16 + 1);
}
W4Params sizes_of(const mk_w4_weight* w, long long m) {
  W4Params p;
  std::memset(&p, 0, sizeof(p));
  p.codes = static_cast<const uint8_t*>(w->codes);
  p.scales = w->scales;
  p.zeros = w->zeros;
  p.m = static_cast<int>(m);
  p.n = static_cast<int>(w->n);
  p.k = static_cast<int>(w->k);
  p.groups = p.k / w->group;
  return p;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

size_t mk_w4_gemm_scratch_size(const mk_w4_weight* w, long long m) {
  if (!weight_ok(w, m) || !w4_use_tiles(sizes_of(w, m), w->group) || w->n == 0) return 0;
  return w4_tiles_scratch(sizes_of(w, m), w->group);
}

mk_status mk_w4_gemm(const void* x, long long x_row, const mk_w4_weight* w, void* y, long long y_row, mk_dtype dtype,
                     mk_dtype out_dtype, long long m, void* scratch, size_t scratch_bytes, void* workspace, size_t ws_bytes,
                     const mk_config* cfg, mk_stream_t stream) {
  if (!weight_ok(w, m) || w->dtype != dtype) return MK_ERR_INVALID;
  if (out_dtype != dtype && out_dtype != MK_F32) return MK_ERR_INVALID;
  if (m == 0 || w->n == 0) return MK_OK;
  const int osz = out_dtype == MK_F32 ? 4 : 2;
  if (!x || !y || !w->codes || !w->scales) return MK_ERR_INVALID;
  // rows of x and of the codes are read in 16-byte pieces
  if ((reinterpret_cast<uintptr_t>(x) & 15u) || ((x_row * 2) & 15) || (reinterpret_cast<uintptr_t>(w->codes) & 15u))
    return MK_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(w->scales) & 1u) || (reinterpret_cast<uintptr_t>(w->zeros) & 1u)) return MK_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(y) & (osz - 1)) || (y_row < w->n && m > 1)) return MK_ERR_INVALID;
  if (cfg && (cfg->max_ctas < 0 || cfg->mode != 0 || cfg->operand != 0 || cfg->reduce != 0 || cfg->wire != 0 ||
              cfg->trace != 0 || cfg->split_k != 0))
    return MK_ERR_INVALID;
  W4Params p = sizes_of(w, m);
  p.x = static_cast<const char*>(x);
  p.x_row = 2 * x_row;
  p.y = static_cast<char*>(y);
  p.y_row = osz * y_row;
  p.out_f32 = out_dtype == MK_F32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (w4_use_tiles(p, w->group)) {
    if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u) || scratch_bytes < w4_tiles_scratch(p, w->group)) return MK_ERR_INVALID;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) || ws_bytes < WS_HDR_BYTES) return MK_ERR_INVALID;
    return launch_w4_tiles(p, dtype, w->group, scratch, static_cast<uint32_t*>(workspace), cfg, s);
  }
  const cudaError_t e = dtype == MK_BF16 ? launch_w4<__nv_bfloat16>(p, w->group, s) : launch_w4<__half>(p, w->group, s);
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // extern "C"
