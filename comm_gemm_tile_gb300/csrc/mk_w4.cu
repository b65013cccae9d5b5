// mk_w4.cu -- few rows times a matrix of 4-bit weights with group scales.
//
//   y[m][n] = sum_k x[m][k] s[n][k / G] (c[n][k] - z[n][k / G]),   z = 8 without zero points
//
// Codes become 16-bit numbers exactly (c - 8 is a whole number of 4 bits), are
// multiplied with x on the tensor cores in fp32, and a group's sum is multiplied
// by its scale in fp32: nothing is rounded before the output.  Zero points enter
// as (8 - z) sum_k x[m][k] of the group, from one more product with ones.
//
// A block has 16 rows of the matrix; its warps share out k in pieces of 128 and
// add their sums in shared memory, in order.  A thread reads 16 bytes (32 codes) of two rows at
// a time.  The products (mma.sync m16n8k16, weights as the 16 rows, tokens as the
// 8 columns) sum over k in any order, so a thread's own codes are its operands as
// they come; x is read in the same order.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk_seq.cuh"

namespace mk {

namespace {

constexpr int W4_WARPS = 8;
constexpr int W4_THREADS = 32 * W4_WARPS;
constexpr int W4_ROWS = 16;
constexpr int W4_TOKENS = 64;          // tokens of a block at most

struct W4Params {
  const char* x;
  long long x_row;                     // bytes
  const uint8_t* codes;                // [n x k / 2]
  const void* scales;                  // [n x k / G], x's type
  const void* zeros;                   // the same, or null
  char* y;
  long long y_row;                     // bytes
  int m, n, k, groups, out_f32;
};

template <class T> struct Mma;
template <> struct Mma<__half> {
  // 8 codes of a word as four pairs (codes i and i + 4), minus 8
  static __device__ __forceinline__ void codes(uint32_t w, uint32_t (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x64006400u;      // 1024 + c in fp16
      __half2 h;
      memcpy(&h, &v, 4);
      h = __hsub2(h, __floats2half2_rn(1032.f, 1032.f));
      memcpy(&o[i], &h, 4);
    }
  }
  static constexpr uint32_t ONES = 0x3c003c00u;
  static __device__ __forceinline__ void run(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};
template <> struct Mma<__nv_bfloat16> {
  static __device__ __forceinline__ void codes(uint32_t w, uint32_t (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;      // 128 + c in bf16
      __nv_bfloat162 h;
      memcpy(&h, &v, 4);
      h = __hsub2(h, __floats2bfloat162_rn(136.f, 136.f));
      memcpy(&o[i], &h, 4);
    }
  }
  static constexpr uint32_t ONES = 0x3f803f80u;
  static __device__ __forceinline__ void run(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

// 8 neighbouring values of x as the pairs that codes() makes: (0, 4), (1, 5), (2, 6), (3, 7)
__device__ __forceinline__ void pairs(const uint4& w, uint32_t (&o)[4]) {
  o[0] = __byte_perm(w.x, w.z, 0x5410);
  o[1] = __byte_perm(w.x, w.z, 0x7632);
  o[2] = __byte_perm(w.y, w.w, 0x5410);
  o[3] = __byte_perm(w.y, w.w, 0x7632);
}

// MT: tiles of 8 tokens.  WPG: words of a thread in a group (4, 2, 1 for groups of 128, 64, 32).
template <class T, int MT, int WPG, bool ZEROS>
__global__ void __launch_bounds__(W4_THREADS) mk_w4_kernel(const __grid_constant__ W4Params p) {
  __shared__ float red[W4_WARPS][W4_ROWS][8 * MT + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, j = lane & 3;
  const int n0 = blockIdx.x * W4_ROWS, m0 = blockIdx.y * W4_TOKENS;
  constexpr int GPC = 4 / WPG;                       // groups of a piece of 128
  float acc[MT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  const int ra = min(n0 + r, p.n - 1), rb = min(n0 + r + 8, p.n - 1);      // rows past the last repeat it
  const uint8_t* ca = p.codes + static_cast<long long>(ra) * (p.k / 2);
  const uint8_t* cb = p.codes + static_cast<long long>(rb) * (p.k / 2);
  const T* sa = static_cast<const T*>(p.scales) + static_cast<long long>(ra) * p.groups;
  const T* sb = static_cast<const T*>(p.scales) + static_cast<long long>(rb) * p.groups;
  const T* za = static_cast<const T*>(p.zeros) + static_cast<long long>(ra) * p.groups;
  const T* zb = static_cast<const T*>(p.zeros) + static_cast<long long>(rb) * p.groups;
  for (int c = warp; c * 128 < p.k; c += W4_WARPS) {
#pragma unroll
    for (int g = 0; g < GPC; ++g) {
      const int group = c * GPC + g;
      if (group >= p.groups) break;
      const int k0 = group * (WPG * 32) + j * (WPG * 8);       // this thread's codes of the group
      uint32_t wa[WPG], wb[WPG];
      if constexpr (WPG == 4) {
        const uint4 a = ld_nc_v4(ca + k0 / 2), b = ld_nc_v4(cb + k0 / 2);
        wa[0] = a.x; wa[1] = a.y; wa[2] = a.z; wa[3] = a.w;
        wb[0] = b.x; wb[1] = b.y; wb[2] = b.z; wb[3] = b.w;
      } else if constexpr (WPG == 2) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(ca + k0 / 2)), b = __ldg(reinterpret_cast<const uint2*>(cb + k0 / 2));
        wa[0] = a.x; wa[1] = a.y;
        wb[0] = b.x; wb[1] = b.y;
      } else {
        wa[0] = __ldg(reinterpret_cast<const uint32_t*>(ca + k0 / 2));
        wb[0] = __ldg(reinterpret_cast<const uint32_t*>(cb + k0 / 2));
      }
      const float fa = Piece<T>::one(sa[group]), fb = Piece<T>::one(sb[group]);
      float part[MT][4], ones[MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) part[i][e] = ones[i][e] = 0.f;
#pragma unroll
      for (int w = 0; w < WPG; ++w) {
        uint32_t a[4], b[4];
        Mma<T>::codes(wa[w], a);
        Mma<T>::codes(wb[w], b);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int t = m0 + 8 * i + r;
          uint32_t xs[4] = {0, 0, 0, 0};
          if (t < p.m) pairs(__ldg(reinterpret_cast<const uint4*>(p.x + t * p.x_row) + (k0 / 8 + w)), xs);
          Mma<T>::run(part[i], a[0], b[0], a[1], b[1], xs[0], xs[1]);
          Mma<T>::run(part[i], a[2], b[2], a[3], b[3], xs[2], xs[3]);
          if (ZEROS) {
            Mma<T>::run(ones[i], Mma<T>::ONES, Mma<T>::ONES, Mma<T>::ONES, Mma<T>::ONES, xs[0], xs[1]);
            Mma<T>::run(ones[i], Mma<T>::ONES, Mma<T>::ONES, Mma<T>::ONES, Mma<T>::ONES, xs[2], xs[3]);
          }
        }
      }
      float oa = 0.f, ob = 0.f;
      if (ZEROS) {
        oa = 8.f - Piece<T>::one(za[group]);
        ob = 8.f - Piece<T>::one(zb[group]);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (ZEROS) {
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
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    red[warp][r][8 * i + 2 * j] = acc[i][0];
    red[warp][r][8 * i + 2 * j + 1] = acc[i][1];
    red[warp][r + 8][8 * i + 2 * j] = acc[i][2];
    red[warp][r + 8][8 * i + 2 * j + 1] = acc[i][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < W4_ROWS * 8 * MT; i += W4_THREADS) {
    const int row = i % W4_ROWS, t = i / W4_ROWS;
    if (n0 + row >= p.n || m0 + t >= p.m) continue;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < W4_WARPS; ++w) s += red[w][row][t];
    char* y = p.y + (m0 + t) * p.y_row;
    if (p.out_f32) reinterpret_cast<float*>(y)[n0 + row] = s;
    else reinterpret_cast<T*>(y)[n0 + row] = Piece<T>::of(s);
  }
}

// ------------------------------------------------------------------ host

template <class T, int MT, int WPG>
cudaError_t launch_w4(const W4Params& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div_ll(p.n, W4_ROWS)), static_cast<unsigned>(ceil_div_ll(p.m, W4_TOKENS)));
  if (p.zeros) mk_w4_kernel<T, MT, WPG, true><<<grid, W4_THREADS, 0, s>>>(p);
  else mk_w4_kernel<T, MT, WPG, false><<<grid, W4_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}
template <class T, int WPG>
cudaError_t launch_w4(const W4Params& p, cudaStream_t s) {
  if (p.m <= 8) return launch_w4<T, 1, WPG>(p, s);
  if (p.m <= 16) return launch_w4<T, 2, WPG>(p, s);
  if (p.m <= 32) return launch_w4<T, 4, WPG>(p, s);
  return launch_w4<T, 8, WPG>(p, s);
}
template <class T>
cudaError_t launch_w4(const W4Params& p, int group, cudaStream_t s) {
  if (group == 128) return launch_w4<T, 4>(p, s);
  return group == 64 ? launch_w4<T, 2>(p, s) : launch_w4<T, 1>(p, s);
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

mk_status mk_w4_gemm(const void* x, long long x_row, const mk_w4_weight* w, void* y, long long y_row, mk_dtype dtype,
                     mk_dtype out_dtype, long long m, mk_stream_t stream) {
  if (!w || (dtype != MK_BF16 && dtype != MK_F16) || w->dtype != dtype) return MK_ERR_INVALID;
  if (out_dtype != dtype && out_dtype != MK_F32) return MK_ERR_INVALID;
  if (w->group != 32 && w->group != 64 && w->group != 128) return MK_ERR_INVALID;
  if (w->n < 0 || w->n >= (1LL << 31) || w->k < w->group || w->k % w->group || w->k >= (1LL << 30)) return MK_ERR_INVALID;
  if (m < 0 || m > 65535LL * W4_TOKENS) return MK_ERR_INVALID;
  if (m == 0 || w->n == 0) return MK_OK;
  const int osz = out_dtype == MK_F32 ? 4 : 2;
  if (!x || !y || !w->codes || !w->scales) return MK_ERR_INVALID;
  // rows of x and of the codes are read in 16-byte pieces
  if ((reinterpret_cast<uintptr_t>(x) & 15u) || ((x_row * 2) & 15) || (reinterpret_cast<uintptr_t>(w->codes) & 15u))
    return MK_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(w->scales) & 1u) || (reinterpret_cast<uintptr_t>(w->zeros) & 1u)) return MK_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(y) & (osz - 1)) || (y_row < w->n && m > 1)) return MK_ERR_INVALID;
  W4Params p;
  std::memset(&p, 0, sizeof(p));
  p.x = static_cast<const char*>(x);
  p.x_row = 2 * x_row;
  p.codes = static_cast<const uint8_t*>(w->codes);
  p.scales = w->scales;
  p.zeros = w->zeros;
  p.y = static_cast<char*>(y);
  p.y_row = osz * y_row;
  p.m = static_cast<int>(m);
  p.n = static_cast<int>(w->n);
  p.k = static_cast<int>(w->k);
  p.groups = p.k / w->group;
  p.out_f32 = out_dtype == MK_F32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == MK_BF16 ? launch_w4<__nv_bfloat16>(p, w->group, s) : launch_w4<__half>(p, w->group, s);
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // extern "C"
