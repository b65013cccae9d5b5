// mk_norm.cu -- root-mean-square norm of rows, with the residual's addition and
// an e4m3 output, and its gradient.
//
//   h = x, or x + residual rounded to its type;  r = 1 / sqrt(mean(h^2) + eps)
//   y = h r w;  8 bits: s = max(amax / 448, 2^-100), codes y / s
//   g = dy w;  dx = r g - h r^3 mean(g h) + dh = r (g - u mean(g u)) + dh with u = h r;  dw = sum over rows dy u
// The norm is of the rounded h: the residual stream keeps values of its type,
// and the gradient, which starts from that h, is the gradient of what forward
// computed.  Everything else is fp32, rounded once.
//
// A row is read once and held in registers (16-byte pieces, as they came) from
// the sums to the stores: memory binds large calls.  A group of L threads has a
// row, thread t its pieces t, t + L, ...: a part of a warp for short rows (many
// rows a block), a whole block for long ones.
//
// A sum of squares that leaves fp32's range is taken again from h 2^-80 (rows
// with values past 1e16 or so; with h 2^80 where eps leaves tiny ones room).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk_seq.cuh"

namespace mk {

namespace {

constexpr int NM_MAX = 16384;          // elements of a row at most
constexpr int NM_THREADS = 256;        // threads of a block that has several rows
constexpr int NM_PARTS = 456;          // blocks, and partial sums of a column, of the gradient at most
constexpr float NM_LEAST = 7.888609052210118e-31f;   // 2^-100, the least scale of 8-bit rows

struct RowsOf {
  char* p;
  long long token, head;               // bytes
};

struct NormParams {
  RowsOf x, r, y, h;                   // gradient: dy, dh, dx, h
  const char* w;                       // null: ones
  float* scale;
  float* part;                         // gradient: [blocks x n] sums over a block's rows; null: not wanted
  unsigned rows, heads;
  int n, pieces, lanes, w_f32;
  float eps;
};

__device__ __forceinline__ char* row_of(const RowsOf& a, unsigned row, unsigned heads) {
  if (heads == 1) return a.p + static_cast<long long>(row) * a.token;
  const unsigned t = row / heads;
  return a.p + static_cast<long long>(t) * a.token + static_cast<long long>(row - t * heads) * a.head;
}

// A thread's piece of a row: 16 bytes, or one element (as fp32 bits) where rows are not whole 16-byte pieces.
template <class T, bool VEC>
struct Bit {
  static constexpr int N = VEC ? Piece<T>::N : 1;
  uint4 w;
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const char* row, int i) {
    if constexpr (VEC) w = ld_stream_v4(row + 16 * i);
    else w.x = __float_as_uint(Piece<T>::one(reinterpret_cast<const T*>(row)[i]));
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    if constexpr (VEC) Piece<T>::get(w, f);
    else f[0] = __uint_as_float(w.x);
  }
  __device__ __forceinline__ void set(const float (&f)[N]) {       // rounded to T
    if constexpr (VEC) w = Piece<T>::put(f);
    else w.x = __float_as_uint(Piece<T>::one(Piece<T>::of(f[0])));
  }
  __device__ __forceinline__ void store(char* row, int i) const {
    if constexpr (VEC) *reinterpret_cast<uint4*>(row + 16 * i) = w;
    else reinterpret_cast<T*>(row)[i] = Piece<T>::of(__uint_as_float(w.x));
  }
};

template <class T, bool VEC>
__device__ __forceinline__ void weights(const NormParams& p, int i, float (&f)[Bit<T, VEC>::N]) {
  constexpr int N = Bit<T, VEC>::N;
  if (p.w == nullptr) {
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = 1.f;
  } else if (p.w_f32) {
    const float* w = reinterpret_cast<const float*>(p.w) + i * N;
    if constexpr (VEC) {
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(w + e));
        f[e] = v.x; f[e + 1] = v.y; f[e + 2] = v.z; f[e + 3] = v.w;
      }
    } else {
      f[0] = __ldg(w);
    }
  } else if constexpr (VEC) {
    Piece<T>::get(__ldg(reinterpret_cast<const uint4*>(p.w) + i), f);
  } else {
    f[0] = Piece<T>::one(reinterpret_cast<const T*>(p.w)[i]);
  }
}

// Sums (or maxima) over the threads of a row, the result in each.  WIDE: the row is the block's, and `turn` says which
// of two buffers serves (a thread is at most one barrier ahead of another).
template <bool WIDE, bool MAX>
__device__ __forceinline__ float over_row(float v, int lanes, float (*buf)[32], int& turn) {
  const int width = WIDE ? 32 : lanes;
  for (int o = width >> 1; o > 0; o >>= 1) {
    const float a = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, a) : v + a;
  }
  if (WIDE) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) buf[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? buf[turn][lane] : 0.f;
    turn ^= 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float a = __shfl_xor_sync(0xffffffffu, v, o);
      v = MAX ? fmaxf(v, a) : v + a;
    }
  }
  return v;
}

// Two sums over a row at once.
template <bool WIDE>
__device__ __forceinline__ float2 over_row2(float2 v, int lanes, float2 (*buf)[32], int& turn) {
  const int width = WIDE ? 32 : lanes;
  for (int o = width >> 1; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (WIDE) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) buf[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? buf[turn][lane] : make_float2(0.f, 0.f);
    turn ^= 1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
      v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
  }
  return v;
}

// Whether fp32 did not hold a row's sum of squares: high (or not a number), or low where eps does not cover it.
__device__ __forceinline__ bool sum_high(float ss) { return !(ss <= 1e36f); }
__device__ __forceinline__ bool sum_low(float ss, int n, float eps) { return eps < 1e-30f && ss < 1e-30f * n; }
// r of a row whose sum of squares is ss; of (h by)^2 where that is not 1.  (A product of the two factors near fp32's
// least numbers, for rows past 1e38, keeps 21 bits.)
__device__ __forceinline__ float inverse_root(float ss, int n, float eps, float by) {
  return by / sqrtf(ss / n + eps * by * by);
}
constexpr float NM_DOWN = 8.271806125530277e-25f, NM_UP = 1.2089258196146292e24f;       // 2^-80, 2^80

template <class T, bool VEC, int U, bool WIDE, bool OUT8>
__global__ void __launch_bounds__(WIDE ? 1024 : NM_THREADS) mk_norm_kernel(const __grid_constant__ NormParams p) {
  using B = Bit<T, VEC>;
  constexpr int N = B::N;
  __shared__ float buf[2][32];
  int turn = 0;
  const int t = WIDE ? threadIdx.x : threadIdx.x & (p.lanes - 1);
  const unsigned per = WIDE ? 1 : NM_THREADS / p.lanes, mine = WIDE ? 0 : threadIdx.x / p.lanes;
  for (unsigned base = blockIdx.x * per; base < p.rows; base += gridDim.x * per) {
    const unsigned row = base + mine;
    const bool real = row < p.rows;
    B b[U];
    if (real) {
      const char* x = row_of(p.x, row, p.heads);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = t + u * p.lanes;
        if (i < p.pieces) b[u].load(x, i);
        else b[u].zero();
      }
      if (p.r.p != nullptr) {
        const char* r = row_of(p.r, row, p.heads);
        B a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = t + u * p.lanes;
          if (i < p.pieces) a[u].load(r, i);
          else a[u].zero();
        }
        char* h = row_of(p.h, row, p.heads);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[N], g[N];
          b[u].get(f);
          a[u].get(g);
#pragma unroll
          for (int e = 0; e < N; ++e) f[e] += g[e];
          b[u].set(f);
          const int i = t + u * p.lanes;
          if (i < p.pieces) b[u].store(h, i);
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) b[u].zero();
    }
    auto squares = [&](float by) {
      float s = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[N];
        b[u].get(f);
#pragma unroll
        for (int e = 0; e < N; ++e) s = fmaf(f[e] * by, f[e] * by, s);
      }
      return over_row<WIDE, false>(s, p.lanes, buf, turn);
    };
    float ss = squares(1.f), by = 1.f;
    // rows of one warp go the second way together; a row's numbers do not depend on its neighbours'
    const bool high = sum_high(ss), low = sum_low(ss, p.n, p.eps);
    if (__any_sync(0xffffffffu, high || low)) {
      by = high ? NM_DOWN : low ? NM_UP : 1.f;
      const float scaled = squares(by);
      ss = high || low ? scaled : ss;
    }
    const float r = inverse_root(ss, p.n, p.eps, by);
    float inv = 1.f;
    if (OUT8) {
      float top = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = t + u * p.lanes;
        if (i >= p.pieces) continue;
        float f[N], w[N];
        b[u].get(f);
        weights<T, VEC>(p, i, w);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float a = fabsf(f[e] * r * w[e]);
          if (a < INFINITY) top = fmaxf(top, a);
        }
      }
      top = over_row<WIDE, true>(top, p.lanes, buf, turn);
      const float s = fmaxf(top / E4M3_MAX, NM_LEAST);
      inv = 1.f / s;
      if (real && t == 0) p.scale[row] = s;
    }
    if (!real) continue;
    char* y = row_of(p.y, row, p.heads);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = t + u * p.lanes;
      if (i >= p.pieces) continue;
      float f[N], w[N];
      b[u].get(f);
      weights<T, VEC>(p, i, w);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = OUT8 ? f[e] * r * w[e] * inv : f[e] * r * w[e];
      if constexpr (!OUT8) {
        b[u].set(f);
        b[u].store(y, i);
      } else if constexpr (N == 8) {
        *reinterpret_cast<uint2*>(y + 8 * i) = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
      } else if constexpr (N == 4) {
        *reinterpret_cast<uint32_t*>(y + 4 * i) = e4m3x4(f[0], f[1], f[2], f[3]);
      } else {
        y[i] = static_cast<char>(e4m3x2(f[0], 0.f));
      }
    }
  }
}

// The gradient.  A block has every gridDim.x-th set of rows; a thread's columns are the same in all of them, so that it
// adds their dy u in registers.  The blocks' sums are added in the order of their numbers by
// mk_norm_columns_kernel: the same bits every time.
//
// Whole pieces come through shared memory, S sets of rows ahead (cp.async: no registers while they are on their way);
// a thread copies what it reads itself, so that no barrier is needed.  Single elements are loaded as they are used.
// Both sums of a row go over its threads at once: one barrier a row.
template <class T, bool VEC, int U>
struct GradShape {
  static constexpr int THREADS = !VEC ? 1024 : U == 2 ? NM_THREADS : sizeof(T) == 4 ? 1024 : 512;   // of a wide row at most
  static constexpr int BLOCKS = VEC && U == 2 ? 3 : 1;      // of an SM at least
};

template <class T, bool VEC, int U, bool WIDE, int S>
__global__ void __launch_bounds__(WIDE ? GradShape<T, VEC, U>::THREADS : NM_THREADS, GradShape<T, VEC, U>::BLOCKS)
    mk_norm_grad_kernel(const __grid_constant__ NormParams p) {
  using B = Bit<T, VEC>;
  constexpr int N = B::N;
  extern __shared__ __align__(16) uint4 ring[];              // [S][h, dy, dh][U][threads]
  __shared__ float2 buf[2][32];
  int turn = 0;
  const int t = WIDE ? threadIdx.x : threadIdx.x & (p.lanes - 1);
  const unsigned per = WIDE ? 1 : NM_THREADS / p.lanes, mine = WIDE ? 0 : threadIdx.x / p.lanes;
  const unsigned step = gridDim.x * per;
  const int tensors = p.r.p != nullptr ? 3 : 2;
  griddep_launch_dependents();
  float acc[U * N], wr[U * N];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float w[N];
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = 0.f;
    if (t + u * p.lanes < p.pieces) weights<T, VEC>(p, t + u * p.lanes, w);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      acc[u * N + e] = 0.f;
      wr[u * N + e] = w[e];
    }
  }
  auto place = [&](int stage, int which, int u) -> uint4* {
    return ring + ((stage * tensors + which) * U + u) * blockDim.x + threadIdx.x;
  };
  auto fetch = [&](unsigned base, int into) {
    if constexpr (VEC) {
      const unsigned row = base + mine;
      if (base < p.rows && row < p.rows) {
        const char* h = row_of(p.h, row, p.heads);
        const char* d = row_of(p.x, row, p.heads);
        const char* g = tensors == 3 ? row_of(p.r, row, p.heads) : nullptr;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = t + u * p.lanes;
          if (i >= p.pieces) continue;
          cp_async_16(smem_u32(place(into, 0, u)), h + 16 * i);
          cp_async_16(smem_u32(place(into, 1, u)), d + 16 * i);
          if (tensors == 3) cp_async_16(smem_u32(place(into, 2, u)), g + 16 * i);
        }
      }
      cp_async_commit();
    }
  };
  unsigned ahead = blockIdx.x * per;
  int fill = 0, stage = 0;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    fetch(ahead, fill++);
    ahead += step;
  }
  for (unsigned base = blockIdx.x * per; base < p.rows; base += step) {
    fetch(ahead, fill);
    ahead = ahead < p.rows ? ahead + step : ahead;           // (stays below 2^32)
    fill = fill + 1 == S ? 0 : fill + 1;
    cp_async_wait<S - 1>();
    const unsigned row = base + mine;
    const bool real = row < p.rows;
    // whole pieces are read where they lie, twice; single elements are held
    B single[VEC ? 1 : 2 * U];
    if constexpr (!VEC) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = t + u * p.lanes;
        single[2 * u].zero();
        single[2 * u + 1].zero();
        if (real && i < p.pieces) {
          single[2 * u].load(row_of(p.h, row, p.heads), i);
          single[2 * u + 1].load(row_of(p.x, row, p.heads), i);
        }
      }
    }
    auto read = [&](int u, float (&f)[N], float (&g)[N]) {
      B h, d;
      if constexpr (VEC) {
        h.zero();
        d.zero();
        if (real && t + u * p.lanes < p.pieces) {
          h.w = *place(stage, 0, u);
          d.w = *place(stage, 1, u);
        }
      } else {
        h = single[2 * u];
        d = single[2 * u + 1];
      }
      h.get(f);
      d.get(g);
    };
    // the sums of h^2 and of g h; mean(g u) is the second times r / n
    auto sums = [&](float by, float gby) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[N], g[N];
        read(u, f, g);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          s.x = fmaf(f[e] * by, f[e] * by, s.x);
          s.y = fmaf(g[e] * wr[u * N + e], f[e] * gby, s.y);
        }
      }
      return over_row2<WIDE>(s, p.lanes, buf, turn);
    };
    float2 s = sums(1.f, 1.f);
    float by = 1.f;
    const bool high = sum_high(s.x), low = sum_low(s.x, p.n, p.eps), far = high || low || !(fabsf(s.y) <= 1e36f);
    const bool again = __any_sync(0xffffffffu, far);
    if (again) {
      by = high ? NM_DOWN : low ? NM_UP : 1.f;
      const float scaled = sums(by, 1.f).x;
      s.x = high || low ? scaled : s.x;
    }
    const float r = inverse_root(s.x, p.n, p.eps, by);
    float dot = s.y * r / p.n;
    if (again) {                                             // sums of g u: u is at most sqrt(n)
      const float of_u = sums(1.f, r).y / p.n;
      dot = far ? of_u : dot;
    }
    if (real) {
      char* dx = row_of(p.y, row, p.heads);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = t + u * p.lanes;
        if (i >= p.pieces) continue;
        float f[N], g[N];
        read(u, f, g);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          f[e] *= r;
          acc[u * N + e] = fmaf(g[e], f[e], acc[u * N + e]);
          f[e] = fmaf(-f[e], dot, g[e] * wr[u * N + e]) * r;
        }
        if (tensors == 3) {
          B a;
          if constexpr (VEC) a.w = *place(stage, 2, u);
          else a.load(row_of(p.r, row, p.heads), i);
          a.get(g);
#pragma unroll
          for (int e = 0; e < N; ++e) f[e] += g[e];
        }
        B out;
        out.set(f);
        out.store(dx, i);
      }
    }
    stage = stage + 1 == S ? 0 : stage + 1;
  }
  if (p.part == nullptr) return;
  float* out = p.part + static_cast<long long>(blockIdx.x) * p.n;
  if (WIDE) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = t + u * p.lanes;
      if (i >= p.pieces) continue;
#pragma unroll
      for (int e = 0; e < N; ++e) out[i * N + e] = acc[u * N + e];
    }
    return;
  }
  // the rows that were handled side by side, in order
  float* sums = reinterpret_cast<float*>(ring);              // [U N][threads]
  cp_async_wait<0>();
  __syncthreads();
#pragma unroll
  for (int i = 0; i < U * N; ++i) sums[i * NM_THREADS + threadIdx.x] = acc[i];
  __syncthreads();
  for (int c = threadIdx.x; c < p.n; c += NM_THREADS) {
    const int i = c / N, e = c % N, u = i / p.lanes, tt = i % p.lanes;
    float s = 0.f;
    for (unsigned g = 0; g < per; ++g) s += sums[(u * N + e) * NM_THREADS + g * p.lanes + tt];
    out[c] = s;
  }
}

struct ColumnParams {
  const float* part;
  void* out;
  int n, parts, dtype;
};

// Column sums of part [parts x n]: a block has 32 columns, its 32 warps every 32nd part, all in flight at once.
constexpr int NC_WARPS = 32;
__global__ void __launch_bounds__(32 * NC_WARPS) mk_norm_columns_kernel(const __grid_constant__ ColumnParams p) {
  __shared__ float sums[NC_WARPS][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x * 32;
  griddep_wait();
  float s = 0.f;
  if (c0 + lane < p.n) {
#pragma unroll 15
    for (int i = warp; i < p.parts; i += NC_WARPS) s += p.part[static_cast<long long>(i) * p.n + c0 + lane];
  }
  sums[warp][lane] = s;
  __syncthreads();
  // warp w adds column w's
  s = sums[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int c = c0 + warp;
  if (lane != 0 || c >= p.n) return;
  if (p.dtype == MK_F32) static_cast<float*>(p.out)[c] = s;
  else if (p.dtype == MK_BF16) static_cast<__nv_bfloat16*>(p.out)[c] = __float2bfloat16_rn(s);
  else static_cast<__half*>(p.out)[c] = __float2half_rn(s);
}

// ------------------------------------------------------------------ host

int size_of(int dtype) { return dtype == MK_F32 ? 4 : dtype == MK_E4M3 ? 1 : 2; }

// A row's threads: u pieces each; part of a warp (a power of two of them), or whole warps.
struct Split {
  int u, lanes, wide;
};
Split split_row(int pieces, long long rows, bool vec) {
  Split s;
  const int most = vec ? 4 : 16;
  s.u = most;
  // few rows: more threads for each, since nothing else fills the SMs
  if (rows <= 304) s.u = 1;
  if ((pieces + s.u - 1) / s.u > 1024) s.u = 4;
  if ((pieces + s.u - 1) / s.u > 1024) s.u = 16;
  const int need = (pieces + s.u - 1) / s.u;
  s.wide = need > 32;
  s.lanes = 1;
  if (s.wide) s.lanes = (need + 31) / 32 * 32;
  else
    while (s.lanes < need) s.lanes *= 2;
  return s;
}

// The gradient's: two pieces a thread, four in rows of more than 512.
Split split_grad(int pieces, bool vec) {
  Split s;
  s.u = vec ? (pieces > 2 * NM_THREADS ? 4 : 2) : pieces > 4096 ? 16 : 4;
  const int need = (pieces + s.u - 1) / s.u;
  s.wide = need > 32;
  s.lanes = 1;
  if (s.wide) s.lanes = (need + 31) / 32 * 32;
  else
    while (s.lanes < need) s.lanes *= 2;
  return s;
}

int grad_blocks(long long rows, const Split& s) {
  const long long per = s.wide ? 1 : NM_THREADS / s.lanes;
  return static_cast<int>(std::min<long long>(ceil_div_ll(rows, per), NM_PARTS));
}

template <class T, bool VEC, int U, bool OUT8>
cudaError_t launch_norm(const NormParams& p, const Split& s, cudaStream_t st) {
  const long long per = s.wide ? 1 : NM_THREADS / s.lanes;
  const unsigned grid = static_cast<unsigned>(ceil_div_ll(p.rows, per));
  if (s.wide) mk_norm_kernel<T, VEC, U, true, OUT8><<<grid, s.lanes, 0, st>>>(p);
  else mk_norm_kernel<T, VEC, U, false, OUT8><<<grid, NM_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

template <class T, bool VEC, int U, int S>
cudaError_t launch_grad(const NormParams& p, const Split& s, cudaStream_t st) {
  const int threads = s.wide ? s.lanes : NM_THREADS;
  size_t smem = VEC ? sizeof(uint4) * S * (p.r.p ? 3 : 2) * U * threads : 0;
  if (!s.wide) smem = std::max(smem, sizeof(float) * U * Bit<T, VEC>::N * threads);
  auto k = mk_norm_grad_kernel<T, VEC, U, true, S>;
  static std::atomic<unsigned> done[2];
  if constexpr (U == (VEC ? 2 : 4))                          // (more a thread: rows of more than a warp)
    if (!s.wide) k = mk_norm_grad_kernel<T, VEC, U, false, S>;
  if (VEC) {
    constexpr size_t most = sizeof(uint4) * S * 3 * U * (S == 2 ? 512 : GradShape<T, VEC, U>::THREADS);
    const cudaError_t e = allow_smem(k, most, done[s.wide]);
    if (e != cudaSuccess) return e;
  }
  k<<<grad_blocks(p.rows, s), threads, smem, st>>>(p);
  return cudaGetLastError();
}

template <class T, bool OUT8>
cudaError_t launch_norm(const NormParams& p, const Split& s, bool vec, cudaStream_t st) {
  if (vec) return s.u == 1 ? launch_norm<T, true, 1, OUT8>(p, s, st) : launch_norm<T, true, 4, OUT8>(p, s, st);
  if (s.u == 1) return launch_norm<T, false, 1, OUT8>(p, s, st);
  return s.u == 4 ? launch_norm<T, false, 4, OUT8>(p, s, st) : launch_norm<T, false, 16, OUT8>(p, s, st);
}

// Shared memory: 24 KB a set of rows and block with two pieces a thread (three sets, three blocks of an SM), 48 to
// 192 KB with four (two sets up to 512 threads, one beyond).
template <class T>
cudaError_t launch_grad(const NormParams& p, const Split& s, bool vec, cudaStream_t st) {
  if (!vec) return s.u == 4 ? launch_grad<T, false, 4, 1>(p, s, st) : launch_grad<T, false, 16, 1>(p, s, st);
  if (s.u == 2) return launch_grad<T, true, 2, 3>(p, s, st);
  return s.lanes <= 512 ? launch_grad<T, true, 4, 2>(p, s, st) : launch_grad<T, true, 4, 1>(p, s, st);
}

bool sizes_ok(mk_dtype dtype, mk_dtype weight_dtype, long long tokens, int heads, int n, float eps) {
  if (dtype != MK_BF16 && dtype != MK_F16 && dtype != MK_F32) return false;
  if (weight_dtype != dtype && weight_dtype != MK_F32) return false;
  if (tokens < 0 || heads < 0 || n < 1 || n > NM_MAX || heads > (1 << 20)) return false;
  if (tokens >= (1LL << 31) || tokens * std::max(heads, 1) >= (1LL << 31)) return false;
  return eps > 0.f && std::isfinite(eps);
}

// Reads a set of rows; false where they cannot be used.  vec: cleared unless every row is whole pieces of `align` bytes.
bool read_rows(const mk_rows* a, int esz, int align, bool written, long long tokens, int heads, RowsOf& o, bool& vec) {
  if (!a->p || (reinterpret_cast<uintptr_t>(a->p) & (esz - 1))) return false;
  // rows that are written have memory of their own (expanded tensors do not)
  if (written && ((a->token == 0 && tokens > 1) || (a->head == 0 && heads > 1))) return false;
  o.p = static_cast<char*>(a->p);
  o.token = a->token * esz;
  o.head = a->head * esz;
  if ((reinterpret_cast<uintptr_t>(a->p) | static_cast<uintptr_t>(o.token) | static_cast<uintptr_t>(o.head)) & (align - 1))
    vec = false;
  return true;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

mk_status mk_rms_norm(const mk_rows* x, const mk_rows* residual, const void* weight, const mk_rows* y, const mk_rows* h,
                      float* scale, mk_dtype dtype, mk_dtype weight_dtype, mk_dtype out_dtype, long long tokens, int heads,
                      int n, float eps, mk_stream_t stream) {
  if (!sizes_ok(dtype, weight_dtype, tokens, heads, n, eps)) return MK_ERR_INVALID;
  if (out_dtype != dtype && out_dtype != MK_E4M3) return MK_ERR_INVALID;
  if (!x || !y || (residual == nullptr) != (h == nullptr)) return MK_ERR_INVALID;
  if (tokens == 0 || heads == 0) return MK_OK;
  if (h && h->p == y->p) return MK_ERR_INVALID;             // one would be written over the other
  const int esz = size_of(dtype), N = 16 / esz;
  bool vec = n % N == 0;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  if (!read_rows(x, esz, 16, false, tokens, heads, p.x, vec)) return MK_ERR_INVALID;
  if (residual && (!read_rows(residual, esz, 16, false, tokens, heads, p.r, vec) ||
                   !read_rows(h, esz, 16, true, tokens, heads, p.h, vec)))
    return MK_ERR_INVALID;
  if (!read_rows(y, size_of(out_dtype), out_dtype == MK_E4M3 ? N : 16, true, tokens, heads, p.y, vec)) return MK_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(weight) & (size_of(weight_dtype) - 1)) return MK_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(weight) & 15u) vec = false;
  if (out_dtype == MK_E4M3 && (!scale || (reinterpret_cast<uintptr_t>(scale) & 3u))) return MK_ERR_INVALID;
  p.w = static_cast<const char*>(weight);
  p.w_f32 = weight_dtype == MK_F32;
  p.scale = scale;
  p.rows = static_cast<unsigned>(tokens * heads);
  p.heads = static_cast<unsigned>(heads);
  p.n = n;
  p.eps = eps;
  p.pieces = vec ? n / N : n;
  const Split s = split_row(p.pieces, p.rows, vec);
  p.lanes = s.lanes;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool o8 = out_dtype == MK_E4M3;
  if (dtype == MK_BF16) e = o8 ? launch_norm<__nv_bfloat16, true>(p, s, vec, st) : launch_norm<__nv_bfloat16, false>(p, s, vec, st);
  else if (dtype == MK_F16) e = o8 ? launch_norm<__half, true>(p, s, vec, st) : launch_norm<__half, false>(p, s, vec, st);
  else e = o8 ? launch_norm<float, true>(p, s, vec, st) : launch_norm<float, false>(p, s, vec, st);
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

size_t mk_rms_norm_backward_workspace_size(long long tokens, int heads, int n) {
  if (!sizes_ok(MK_F32, MK_F32, tokens, heads, n, 1.f)) return 0;
  const long long blocks = std::min<long long>(NM_PARTS, std::max<long long>(1, tokens * heads));
  return static_cast<size_t>(blocks) * n * sizeof(float);
}

mk_status mk_rms_norm_backward(const mk_rows* dy, const mk_rows* dh, const mk_rows* h, const void* weight, const mk_rows* dx,
                               void* dweight, mk_dtype dtype, mk_dtype weight_dtype, long long tokens, int heads, int n,
                               float eps, void* workspace, size_t ws_bytes, mk_stream_t stream) {
  if (!sizes_ok(dtype, weight_dtype, tokens, heads, n, eps)) return MK_ERR_INVALID;
  if (!dy || !h || !dx) return MK_ERR_INVALID;
  if (dweight && (!weight || (reinterpret_cast<uintptr_t>(dweight) & (size_of(weight_dtype) - 1)))) return MK_ERR_INVALID;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0 || heads == 0)     // a sum over no rows
    return !dweight || cudaMemsetAsync(dweight, 0, static_cast<size_t>(n) * size_of(weight_dtype), st) == cudaSuccess
               ? MK_OK : MK_ERR_CUDA;
  if (dweight && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15u) ||
                  ws_bytes < mk_rms_norm_backward_workspace_size(tokens, heads, n)))
    return MK_ERR_INVALID;
  const int esz = size_of(dtype), N = 16 / esz;
  bool vec = n % N == 0;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  if (!read_rows(dy, esz, 16, false, tokens, heads, p.x, vec) || !read_rows(h, esz, 16, false, tokens, heads, p.h, vec) ||
      !read_rows(dx, esz, 16, true, tokens, heads, p.y, vec) ||
      (dh && !read_rows(dh, esz, 16, false, tokens, heads, p.r, vec)))
    return MK_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(weight) & (size_of(weight_dtype) - 1)) return MK_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(weight) & 15u) vec = false;
  p.w = static_cast<const char*>(weight);
  p.w_f32 = weight_dtype == MK_F32;
  p.part = dweight ? static_cast<float*>(workspace) : nullptr;
  p.rows = static_cast<unsigned>(tokens * heads);
  p.heads = static_cast<unsigned>(heads);
  p.n = n;
  p.eps = eps;
  p.pieces = vec ? n / N : n;
  const Split s = split_grad(p.pieces, vec);
  p.lanes = s.lanes;
  cudaError_t e;
  if (dtype == MK_BF16) e = launch_grad<__nv_bfloat16>(p, s, vec, st);
  else if (dtype == MK_F16) e = launch_grad<__half>(p, s, vec, st);
  else e = launch_grad<float>(p, s, vec, st);
  if (e != cudaSuccess) return MK_ERR_CUDA;
  if (!dweight) return MK_OK;
  ColumnParams c = {p.part, dweight, n, grad_blocks(p.rows, s), weight_dtype};
  e = launch_dependent(mk_norm_columns_kernel, dim3((n + 31) / 32), dim3(32 * NC_WARPS), st, c);
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // extern "C"
