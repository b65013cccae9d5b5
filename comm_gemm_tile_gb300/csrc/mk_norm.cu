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
// Rows of odd lengths begin anywhere in a 16-byte piece of memory, but every 8th
// (fp32: every 4th) begins at the same place in one, and as a rule all tensors of
// a call agree in that.  A block then takes rows of one such class: a row's pieces
// are the pieces of memory that it touches, its columns shifted by where it
// begins, and what lies outside of it at both ends is left out.  Rows that do not
// agree are moved element by element.  16384 x 4095 in bf16: 125 us this way, 178
// by elements; the gradient 134 and 430; 65536 x 129: 24 and 45, 39 and 200.
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
  const char *lo, *hi;                 // the rows lie in [lo, hi)
};
// How rows are taken: whole pieces; pieces of memory that rows begin and end inside of; single elements.
enum Way { PIECES, SHIFTED, ELEMENTS };

struct NormParams {
  RowsOf x, r, y, h;                   // gradient: dy, dh, dx, h
  const char* w;                       // null: ones
  float* scale;
  float* part;                         // gradient: [blocks x n] sums over a block's rows; null: not wanted
  unsigned rows, heads;
  int n, pieces, lanes, w_f32;         // pieces: of a row at most
  unsigned classes;                    // SHIFTED: rows r and r + classes begin at the same place in a piece
  float eps;
};

__device__ __forceinline__ char* row_of(const RowsOf& a, unsigned row, unsigned heads) {
  if (heads == 1) return a.p + static_cast<long long>(row) * a.token;
  const unsigned t = row / heads;
  return a.p + static_cast<long long>(t) * a.token + static_cast<long long>(row - t * heads) * a.head;
}

// A thread's piece of a row: 16 bytes, or one element (as fp32 bits) where rows are not whole 16-byte pieces.
template <class T, Way WAY>
struct Bit {
  static constexpr bool VEC = WAY != ELEMENTS;
  static constexpr int N = VEC ? Piece<T>::N : 1;
  uint4 w;
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  // piece i of a row that begins `before` elements into its first piece of memory; SHIFTED: zeros outside the row
  __device__ __forceinline__ void load(const RowsOf& a, const char* row, int i, int before, int n) {
    if constexpr (WAY == PIECES) {
      w = ld_stream_v4(row + 16 * i);
    } else if constexpr (WAY == SHIFTED) {
      const char* q = row + (i * N - before) * static_cast<int>(sizeof(T));
      if (q >= a.lo && q + 16 <= a.hi) {
        w = ld_stream_v4(q);
        inside(i, before, n);
      } else {                                               // (the first or last row's)
        T v[N];
#pragma unroll
        for (int e = 0; e < N; ++e)
          v[e] = static_cast<unsigned>(i * N - before + e) < static_cast<unsigned>(n) ? reinterpret_cast<const T*>(q)[e] : Piece<T>::of(0.f);
        memcpy(&w, v, 16);
      }
    } else {
      w.x = __float_as_uint(Piece<T>::one(reinterpret_cast<const T*>(row)[i]));
    }
  }
  // zeros in the place of what is outside the row
  __device__ __forceinline__ void inside(int i, int before, int n) {
    const int c = i * N - before;
    if (c >= 0 && c + N <= n) return;
    T v[N];
    memcpy(v, &w, 16);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (static_cast<unsigned>(c + e) >= static_cast<unsigned>(n)) v[e] = Piece<T>::of(0.f);
    memcpy(&w, v, 16);
  }
  __device__ __forceinline__ void get(float (&f)[N]) const {
    if constexpr (VEC) Piece<T>::get(w, f);
    else f[0] = __uint_as_float(w.x);
  }
  __device__ __forceinline__ void set(const float (&f)[N]) {       // rounded to T
    if constexpr (VEC) w = Piece<T>::put(f);
    else w.x = __float_as_uint(Piece<T>::one(Piece<T>::of(f[0])));
  }
  __device__ __forceinline__ void store(char* row, int i, int before, int n) const {
    if constexpr (WAY == PIECES) {
      *reinterpret_cast<uint4*>(row + 16 * i) = w;
    } else if constexpr (WAY == SHIFTED) {
      const int c = i * N - before;
      T* q = reinterpret_cast<T*>(row) + c;
      if (c >= 0 && c + N <= n) {
        *reinterpret_cast<uint4*>(q) = w;
      } else {
        T v[N];
        memcpy(v, &w, 16);
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (static_cast<unsigned>(c + e) < static_cast<unsigned>(n)) q[e] = v[e];
      }
    } else {
      reinterpret_cast<T*>(row)[i] = Piece<T>::of(__uint_as_float(w.x));
    }
  }
};

// The weights of piece i, 0 outside the row.
template <class T, Way WAY>
__device__ __forceinline__ void weights(const NormParams& p, int i, int before, float (&f)[Bit<T, WAY>::N]) {
  constexpr int N = Bit<T, WAY>::N;
  if constexpr (WAY == PIECES) {
    if (p.w == nullptr) {
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = 1.f;
    } else if (p.w_f32) {
      const float* w = reinterpret_cast<const float*>(p.w) + i * N;
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(w + e));
        f[e] = v.x; f[e + 1] = v.y; f[e + 2] = v.z; f[e + 3] = v.w;
      }
    } else {
      Piece<T>::get(__ldg(reinterpret_cast<const uint4*>(p.w) + i), f);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int c = i * N - before + e;
      if (static_cast<unsigned>(c) >= static_cast<unsigned>(p.n)) f[e] = 0.f;
      else if (p.w == nullptr) f[e] = 1.f;
      else if (p.w_f32) f[e] = __ldg(reinterpret_cast<const float*>(p.w) + c);
      else f[e] = Piece<T>::one(reinterpret_cast<const T*>(p.w)[c]);
    }
  }
}

// A block's rows: first, first + step, ... (with each `per` of them side by side, `apart`), below p.rows; and where they
// begin in their first piece of memory.
struct Rows {
  unsigned first, step, apart;
  int before, pieces;
};
template <class T, Way WAY>
__device__ __forceinline__ Rows rows_of(const NormParams& p, const RowsOf& a, unsigned per) {
  Rows r;
  if constexpr (WAY != SHIFTED) {
    r = {blockIdx.x * per, gridDim.x * per, 1, 0, p.pieces};
  } else {
    const unsigned c = blockIdx.x % p.classes;
    r.first = c + blockIdx.x / p.classes * per * p.classes;
    r.step = gridDim.x * per;
    r.apart = p.classes;
    r.before = static_cast<int>((reinterpret_cast<uintptr_t>(a.p) + c * a.head) & 15) / static_cast<int>(sizeof(T));
    r.pieces = (r.before + p.n + Piece<T>::N - 1) / Piece<T>::N;
  }
  return r;
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
// Whether products of a row's elements with a gradient may be below fp32's range where those of u are not: small rows
// that eps lets grow.
__device__ __forceinline__ bool row_small(float ss, int n, float eps) { return eps < 1e-12f && ss < 1e-12f * n; }
// r of a row whose sum of squares is ss; of (h by)^2 where that is not 1.  (A product of the two factors near fp32's
// least numbers, for rows past 1e38, keeps 21 bits.)
__device__ __forceinline__ float inverse_root(float ss, int n, float eps, float by) {
  return by / sqrtf(ss / n + eps * by * by);
}
constexpr float NM_DOWN = 8.271806125530277e-25f, NM_UP = 1.2089258196146292e24f;       // 2^-80, 2^80

// v / s to nearest, for inv = 1 / s to nearest: the product with inv is a step off at most, and its remainder, which fma has
// exactly, puts it right (Markstein 1990).  Where there is none (v infinite, or a quotient that is exact, -0 among them) it
// stays.  8192 x 8192 in bf16 with a residual, us:
// the product alone 74, so 78, `/` 90.
__device__ __forceinline__ float quotient(float v, float s, float inv) {
  const float q = v * inv, left = fmaf(-q, s, v);
  return fabsf(left) > 0.f ? fmaf(left, inv, q) : q;
}

template <class T, Way WAY, int U, bool WIDE, bool OUT8>
__global__ void __launch_bounds__(WIDE ? 1024 : NM_THREADS) mk_norm_kernel(const __grid_constant__ NormParams p) {
  using B = Bit<T, WAY>;
  constexpr int N = B::N;
  __shared__ float buf[2][32];
  int turn = 0;
  const int t = WIDE ? threadIdx.x : threadIdx.x & (p.lanes - 1);
  const unsigned per = WIDE ? 1 : NM_THREADS / p.lanes, mine = WIDE ? 0 : threadIdx.x / p.lanes;
  const Rows rs = rows_of<T, WAY>(p, p.x, per);
  for (unsigned base = rs.first; base < p.rows; base += rs.step) {
    const unsigned row = base + mine * rs.apart;
    const bool real = row < p.rows;
    B b[U];
    if (real) {
      const char* x = row_of(p.x, row, p.heads);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = t + u * p.lanes;
        if (i < rs.pieces) b[u].load(p.x, x, i, rs.before, p.n);
        else b[u].zero();
      }
      if (p.r.p != nullptr) {
        const char* r = row_of(p.r, row, p.heads);
        B a[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = t + u * p.lanes;
          if (i < rs.pieces) a[u].load(p.r, r, i, rs.before, p.n);
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
          if (i < rs.pieces) b[u].store(h, i, rs.before, p.n);
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
    float s8 = 1.f, inv8 = 1.f;                              // the row's scale
    if (OUT8) {
      float top = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = t + u * p.lanes;
        if (i >= rs.pieces) continue;
        float f[N], w[N];
        b[u].get(f);
        weights<T, WAY>(p, i, rs.before, w);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float a = fabsf(f[e] * r * w[e]);
          if (a < INFINITY) top = fmaxf(top, a);
        }
      }
      top = over_row<WIDE, true>(top, p.lanes, buf, turn);
      s8 = fmaxf(top / E4M3_MAX, NM_LEAST);
      inv8 = 1.f / s8;
      if (real && t == 0) p.scale[row] = s8;
    }
    if (!real) continue;
    char* y = row_of(p.y, row, p.heads);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = t + u * p.lanes;
      if (i >= rs.pieces) continue;
      float f[N], w[N];
      b[u].get(f);
      weights<T, WAY>(p, i, rs.before, w);
#pragma unroll
      for (int e = 0; e < N; ++e) f[e] = OUT8 ? quotient(f[e] * r * w[e], s8, inv8) : f[e] * r * w[e];
      if constexpr (!OUT8) {
        b[u].set(f);
        b[u].store(y, i, rs.before, p.n);
      } else if constexpr (WAY != PIECES) {                  // (8-bit rows begin elsewhere)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int c = i * N - rs.before + e;
          if (static_cast<unsigned>(c) < static_cast<unsigned>(p.n)) y[c] = static_cast<char>(e4m3x2(f[e], 0.f));
        }
      } else if constexpr (N == 8) {
        *reinterpret_cast<uint2*>(y + 8 * i) = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
      } else {
        *reinterpret_cast<uint32_t*>(y + 4 * i) = e4m3x4(f[0], f[1], f[2], f[3]);
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
template <class T, Way WAY, int U>
struct GradShape {
  static constexpr bool VEC = WAY != ELEMENTS;
  static constexpr int THREADS = !VEC ? (U == 8 ? 512 : 1024) : U == 2 ? NM_THREADS : sizeof(T) == 4 ? 1024 : 512;   // of a wide row at most
  static constexpr int BLOCKS = VEC && U == 2 ? 3 : 1;      // of an SM at least
};

template <class T, Way WAY, int U, bool WIDE, int S>
__global__ void __launch_bounds__(WIDE ? GradShape<T, WAY, U>::THREADS : NM_THREADS, GradShape<T, WAY, U>::BLOCKS)
    mk_norm_grad_kernel(const __grid_constant__ NormParams p) {
  using B = Bit<T, WAY>;
  constexpr int N = B::N;
  constexpr bool VEC = B::VEC;
  extern __shared__ __align__(16) uint4 ring[];              // [S][h, dy, dh][U][threads]
  __shared__ float2 buf[2][32];
  int turn = 0;
  const int t = WIDE ? threadIdx.x : threadIdx.x & (p.lanes - 1);
  const unsigned per = WIDE ? 1 : NM_THREADS / p.lanes, mine = WIDE ? 0 : threadIdx.x / p.lanes;
  const Rows rs = rows_of<T, WAY>(p, p.h, per);
  const unsigned step = rs.step;
  const int tensors = p.r.p != nullptr ? 3 : 2;
  griddep_launch_dependents();
  float acc[U * N], wr[U * N];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float w[N];
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = 0.f;
    if (t + u * p.lanes < rs.pieces) weights<T, WAY>(p, t + u * p.lanes, rs.before, w);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      acc[u * N + e] = 0.f;
      wr[u * N + e] = w[e];
    }
  }
  auto place = [&](int stage, int which, int u) -> uint4* {
    return ring + ((stage * tensors + which) * U + u) * blockDim.x + threadIdx.x;
  };
  // a piece of memory that a row may begin or end in: as it is, or (where it is not all the tensor's) the row's part
  auto bring = [&](uint4* to, const RowsOf& a, const char* row, int i) {
    const char* q = row + (i * N - rs.before) * static_cast<int>(sizeof(T));
    if (q >= a.lo && q + 16 <= a.hi) {
      cp_async_16(smem_u32(to), q);
    } else {
      B b;
      b.load(a, row, i, rs.before, p.n);
      *to = b.w;
    }
  };
  auto fetch = [&](unsigned base, int into) {
    if constexpr (VEC) {
      const unsigned row = base + mine * rs.apart;
      if (base < p.rows && row < p.rows) {
        const char* h = row_of(p.h, row, p.heads);
        const char* d = row_of(p.x, row, p.heads);
        const char* g = tensors == 3 ? row_of(p.r, row, p.heads) : nullptr;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = t + u * p.lanes;
          if (i >= rs.pieces) continue;
          if constexpr (WAY == SHIFTED) {
            bring(place(into, 0, u), p.h, h, i);
            bring(place(into, 1, u), p.x, d, i);
            if (tensors == 3) bring(place(into, 2, u), p.r, g, i);
          } else {
            cp_async_16(smem_u32(place(into, 0, u)), h + 16 * i);
            cp_async_16(smem_u32(place(into, 1, u)), d + 16 * i);
            if (tensors == 3) cp_async_16(smem_u32(place(into, 2, u)), g + 16 * i);
          }
        }
      }
      cp_async_commit();
    }
  };
  unsigned ahead = rs.first;
  int fill = 0, stage = 0;
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    fetch(ahead, fill++);
    ahead += step;
  }
  for (unsigned base = rs.first; base < p.rows; base += step) {
    fetch(ahead, fill);
    ahead = ahead < p.rows ? ahead + step : ahead;           // (stays below 2^32)
    fill = fill + 1 == S ? 0 : fill + 1;
    cp_async_wait<S - 1>();
    const unsigned row = base + mine * rs.apart;
    const bool real = row < p.rows;
    // whole pieces are read where they lie, twice; single elements are held
    B single[VEC ? 1 : 2 * U];
    if constexpr (!VEC) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = t + u * p.lanes;
        single[2 * u].zero();
        single[2 * u + 1].zero();
        if (real && i < rs.pieces) {
          single[2 * u].load(p.h, row_of(p.h, row, p.heads), i, 0, p.n);
          single[2 * u + 1].load(p.x, row_of(p.x, row, p.heads), i, 0, p.n);
        }
      }
    }
    auto read = [&](int u, float (&f)[N], float (&g)[N]) {
      B h, d;
      if constexpr (VEC) {
        h.zero();
        d.zero();
        if (real && t + u * p.lanes < rs.pieces) {
          h.w = *place(stage, 0, u);
          d.w = *place(stage, 1, u);
          if constexpr (WAY == SHIFTED) {
            h.inside(t + u * p.lanes, rs.before, p.n);
            d.inside(t + u * p.lanes, rs.before, p.n);
          }
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
    const bool high = sum_high(s.x), low = sum_low(s.x, p.n, p.eps), far = high || row_small(s.x, p.n, p.eps) || !(fabsf(s.y) <= 1e36f);
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
        if (i >= rs.pieces) continue;
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
          else a.load(p.r, row_of(p.r, row, p.heads), i, 0, p.n);
          a.get(g);
#pragma unroll
          for (int e = 0; e < N; ++e) f[e] += g[e];
        }
        B out;
        out.set(f);
        out.store(dx, i, rs.before, p.n);
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
      if (i >= rs.pieces) continue;
      if constexpr (WAY == PIECES) {                         // (single stores, 32 bytes apart: 2048 x 4096 20 us for 16)
#pragma unroll
        for (int e = 0; e < N; e += 4)
          *reinterpret_cast<float4*>(out + i * N + e) =
              make_float4(acc[u * N + e], acc[u * N + e + 1], acc[u * N + e + 2], acc[u * N + e + 3]);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int c = i * N - rs.before + e;
          if (WAY != SHIFTED || static_cast<unsigned>(c) < static_cast<unsigned>(p.n)) out[c] = acc[u * N + e];
        }
      }
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
    const int at = c + rs.before, i = at / N, e = at % N, u = i / p.lanes, tt = i % p.lanes;
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

// Column sums of part [parts x n]: a block has 32 columns, each of its warps every 8th part, or, past 64 parts, every
// 32nd (us of both kernels with 8 and 32 warps: 8 parts of 8192 columns 7.2 and 7.4, 456 of 4096 16.4 and 11.7).
__global__ void __launch_bounds__(1024) mk_norm_columns_kernel(const __grid_constant__ ColumnParams p) {
  __shared__ float sums[32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, c = blockIdx.x * 32 + lane;
  griddep_wait();
  float s = 0.f;
  if (c < p.n) {
#pragma unroll 8
    for (int i = warp; i < p.parts; i += warps) s += p.part[static_cast<long long>(i) * p.n + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= p.n) return;
  s = 0.f;
#pragma unroll 8
  for (int i = 0; i < warps; ++i) s += sums[i][lane];
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
void lanes_of(int pieces, Split& s) {
  const int need = (pieces + s.u - 1) / s.u;
  s.wide = need > 32;
  s.lanes = 1;
  if (s.wide) s.lanes = (need + 31) / 32 * 32;
  else
    while (s.lanes < need) s.lanes *= 2;
}
// Four pieces a thread (16 elements); up to 304 rows one, since nothing else fills the SMs (bf16 with a residual, us, one
// and four: 16 x 8192 2.83 and 3.20, 304 x 4096 2.75 and 3.40, 608 x 8192 6.49 and 4.93, 16384 x 4096 83.5 and 78.9).
Split split_row(int pieces, long long rows, Way way) {
  Split s;
  s.u = rows <= 304 ? 1 : way == ELEMENTS ? 16 : 4;
  if ((pieces + s.u - 1) / s.u > 1024) s.u = 4;
  if ((pieces + s.u - 1) / s.u > 1024) s.u = 16;
  lanes_of(pieces, s);
  return s;
}
// The gradient's: two pieces a thread, four in rows of more than 512 (16384 x 4096, bf16: two 84 us, four 86).  Single
// elements: 4 or 16 in rows of a part of a warp, 8 in rows of a block, 16 past 4096.
Split split_grad(int pieces, Way way) {
  Split s;
  if (way != ELEMENTS) s.u = pieces > 2 * NM_THREADS ? 4 : 2;
  else s.u = pieces <= 128 ? 4 : pieces <= 512 ? 16 : pieces <= 4096 ? 8 : 16;
  lanes_of(pieces, s);
  return s;
}

// Blocks for rows (of a class, where there are several): no more than run at once (three of an SM, or what its shared
// memory holds of rows of four pieces a thread: 32768 x 8192, bf16, 304 blocks 242 us, 456 274; 16384 x 4095, whose rows are
// 160 threads', 167 and 134), of at least two sets of rows, since
// every block leaves sums of all columns (us, least one, two, four sets: 16 x 8192 6.1, 7.2, 10.0; 304 x 8192 11.8, 8.9,
// 11.0; 1000 x 128 5.4, 5.9, 7.2; 1216 x 4096 16.3, 16.4, 12.2, with 32 warps for the columns 11.7 for two).
int grad_blocks(long long rows, const Split& s, Way way, unsigned classes) {
  const long long per = s.wide ? 1 : NM_THREADS / s.lanes, mine = ceil_div_ll(rows, classes);
  const int room = way == ELEMENTS || s.u == 2 ? 3 : static_cast<int>(227 * 1024 / (sizeof(uint4) * 2 * 3 * 4 * s.lanes + 2048));
  const int most = NM_PARTS / 3 * std::max(1, std::min(3, room));
  // (a whole number of each class; with fewer rows than classes one block a row, since the workspace has room for no more)
  return static_cast<int>(std::min<long long>(rows, std::min<long long>(ceil_div_ll(mine, 2 * per), most / classes) * classes));
}

template <class T, Way WAY, int U, bool OUT8>
cudaError_t launch_norm(const NormParams& p, const Split& s, cudaStream_t st) {
  const long long per = s.wide ? 1 : NM_THREADS / s.lanes;
  const unsigned grid = static_cast<unsigned>(ceil_div_ll(ceil_div_ll(p.rows, p.classes), per) * p.classes);
  if (s.wide) mk_norm_kernel<T, WAY, U, true, OUT8><<<grid, s.lanes, 0, st>>>(p);
  else mk_norm_kernel<T, WAY, U, false, OUT8><<<grid, NM_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

template <class T, Way WAY, int U, int S>
cudaError_t launch_grad(const NormParams& p, const Split& s, cudaStream_t st) {
  constexpr bool VEC = WAY != ELEMENTS;
  const int threads = s.wide ? s.lanes : NM_THREADS;
  size_t smem = VEC ? sizeof(uint4) * S * (p.r.p ? 3 : 2) * U * threads : 0;
  if (!s.wide) smem = std::max(smem, sizeof(float) * U * Bit<T, WAY>::N * threads);
  // which of the two the split gives: four pieces or eight elements a thread are a block's row, four elements a warp's
  constexpr bool WIDE = VEC || U != 4, NARROW = VEC ? U == 2 : U != 8;
  auto k = mk_norm_grad_kernel<T, WAY, U, WIDE, S>;
  static std::atomic<unsigned> done[2];
  if constexpr (WIDE && NARROW)
    if (!s.wide) k = mk_norm_grad_kernel<T, WAY, U, false, S>;
  if (VEC) {
    constexpr size_t most = sizeof(uint4) * S * 3 * U * (S == 2 ? 512 : GradShape<T, WAY, U>::THREADS);
    const cudaError_t e = allow_smem(k, most, done[s.wide]);
    if (e != cudaSuccess) return e;
  }
  k<<<grad_blocks(p.rows, s, WAY, p.classes), threads, smem, st>>>(p);
  return cudaGetLastError();
}

template <class T, bool OUT8>
cudaError_t launch_norm(const NormParams& p, const Split& s, Way way, cudaStream_t st) {
  if (way == PIECES) return s.u == 1 ? launch_norm<T, PIECES, 1, OUT8>(p, s, st) : launch_norm<T, PIECES, 4, OUT8>(p, s, st);
  if (way == SHIFTED) return s.u == 1 ? launch_norm<T, SHIFTED, 1, OUT8>(p, s, st) : launch_norm<T, SHIFTED, 4, OUT8>(p, s, st);
  if (s.u == 1) return launch_norm<T, ELEMENTS, 1, OUT8>(p, s, st);
  return s.u == 4 ? launch_norm<T, ELEMENTS, 4, OUT8>(p, s, st) : launch_norm<T, ELEMENTS, 16, OUT8>(p, s, st);
}

// Shared memory: 24 KB a set of rows and block with two pieces a thread (three sets, three blocks of an SM), 48 to
// 192 KB with four (two sets up to 512 threads, which no 16-bit row passes, one beyond).
template <class T, Way WAY>
cudaError_t launch_pieces(const NormParams& p, const Split& s, cudaStream_t st) {
  if (s.u == 2) return launch_grad<T, WAY, 2, 3>(p, s, st);
  if constexpr (sizeof(T) == 4)
    if (s.lanes > 512) return launch_grad<T, WAY, 4, 1>(p, s, st);
  return launch_grad<T, WAY, 4, 2>(p, s, st);
}
template <class T>
cudaError_t launch_grad(const NormParams& p, const Split& s, Way way, cudaStream_t st) {
  if (way == PIECES) return launch_pieces<T, PIECES>(p, s, st);
  if (way == SHIFTED) return launch_pieces<T, SHIFTED>(p, s, st);
  return s.u == 4 ? launch_grad<T, ELEMENTS, 4, 1>(p, s, st) : s.u == 8 ? launch_grad<T, ELEMENTS, 8, 1>(p, s, st)
                                                                          : launch_grad<T, ELEMENTS, 16, 1>(p, s, st);
}

bool sizes_ok(mk_dtype dtype, mk_dtype weight_dtype, long long tokens, int heads, int n, float eps) {
  if (dtype != MK_BF16 && dtype != MK_F16 && dtype != MK_F32) return false;
  if (weight_dtype != dtype && weight_dtype != MK_F32) return false;
  if (tokens < 0 || heads < 0 || n < 1 || n > NM_MAX || heads > (1 << 20)) return false;
  if (tokens >= (1LL << 31) || tokens * std::max(heads, 1) >= (1LL << 31)) return false;
  return eps > 0.f && std::isfinite(eps);
}

// Reads a set of rows; false where they cannot be used.
bool read_rows(const mk_rows* a, int esz, bool written, long long tokens, int heads, int n, RowsOf& o) {
  if (!a->p || (reinterpret_cast<uintptr_t>(a->p) & (esz - 1))) return false;
  // rows that are written have memory of their own (expanded tensors do not)
  if (written && ((a->token == 0 && tokens > 1) || (a->head == 0 && heads > 1))) return false;
  o.p = static_cast<char*>(a->p);
  o.token = a->token * esz;
  o.head = a->head * esz;
  const long long token = (tokens - 1) * o.token, head = (heads - 1) * o.head;
  o.lo = o.p + std::min(0LL, token) + std::min(0LL, head);
  o.hi = o.p + std::max(0LL, token) + std::max(0LL, head) + static_cast<long long>(n) * esz;
  return true;
}

// The way for a call's rows, and its pieces and classes.  all: the rows of the call's own type; eight: 8-bit output.
Way way_of(NormParams& p, RowsOf* const* all, int count, const RowsOf* eight, long long tokens, int heads, int esz) {
  const int N = 16 / esz;
  uintptr_t lie = reinterpret_cast<uintptr_t>(p.w);
  bool line = true, agree = true;                            // rows one stride apart; that begin alike in all tensors
  for (int i = 0; i < count; ++i) {
    RowsOf& a = *all[i];
    lie |= reinterpret_cast<uintptr_t>(a.p) | static_cast<uintptr_t>(tokens > 1 ? a.token : 0) | static_cast<uintptr_t>(heads > 1 ? a.head : 0);
    line = line && (heads == 1 || tokens == 1 || a.token == heads * a.head);
  }
  if (eight)
    line = line && (heads == 1 || tokens == 1 || eight->token == heads * eight->head);
  const uintptr_t lie8 = !eight ? 0 : reinterpret_cast<uintptr_t>(eight->p) | static_cast<uintptr_t>(tokens > 1 ? eight->token : 0) |
                                          static_cast<uintptr_t>(heads > 1 ? eight->head : 0);
  p.classes = 1;
  p.pieces = p.n / N;
  if (p.n % N == 0 && !(lie & 15u) && !(lie8 & (N - 1))) return PIECES;
  auto stride = [&](const RowsOf& a) { return heads > 1 ? a.head : a.token; };
  for (int i = 1; i < count && line; ++i) {
    agree = agree && !((reinterpret_cast<uintptr_t>(all[i]->p) ^ reinterpret_cast<uintptr_t>(all[0]->p)) & 15u) &&
            !((static_cast<uintptr_t>(stride(*all[i])) ^ static_cast<uintptr_t>(stride(*all[0]))) & 15u);
  }
  // (no more pieces than the longest row of whole ones has)
  if (line && agree && p.n >= 2 * N && p.n + 2 * N - 2 < NM_MAX + N) {
    // one dimension of rows: a.head is their stride
    const uintptr_t s = p.rows > 1 ? static_cast<uintptr_t>(stride(*all[0])) & 15u : 0;
    for (int i = 0; i < count; ++i) all[i]->token = all[i]->head = stride(*all[i]);
    p.heads = 1;
    while ((s * p.classes) & 15u) p.classes *= 2;
    p.pieces = (p.n + 2 * N - 2) / N;
    return SHIFTED;
  }
  p.pieces = p.n;
  return ELEMENTS;
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
  const int esz = size_of(dtype);
  const bool o8 = out_dtype == MK_E4M3;
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  if (!read_rows(x, esz, false, tokens, heads, n, p.x) || !read_rows(y, o8 ? 1 : esz, true, tokens, heads, n, p.y)) return MK_ERR_INVALID;
  if (residual && (!read_rows(residual, esz, false, tokens, heads, n, p.r) || !read_rows(h, esz, true, tokens, heads, n, p.h)))
    return MK_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(weight) & (size_of(weight_dtype) - 1)) return MK_ERR_INVALID;
  if (o8 && (!scale || (reinterpret_cast<uintptr_t>(scale) & 3u))) return MK_ERR_INVALID;
  p.w = static_cast<const char*>(weight);
  p.w_f32 = weight_dtype == MK_F32;
  p.scale = scale;
  p.rows = static_cast<unsigned>(tokens * heads);
  p.heads = static_cast<unsigned>(heads);
  p.n = n;
  p.eps = eps;
  RowsOf* all[4] = {&p.x, &p.r, &p.h, &p.y};
  if (!residual) all[1] = &p.y;
  const Way way = way_of(p, all, residual ? (o8 ? 3 : 4) : (o8 ? 1 : 2), o8 ? &p.y : nullptr, tokens, heads, esz);
  if (way == SHIFTED && o8) p.y.token = p.y.head = heads > 1 ? p.y.head : p.y.token;
  const Split s = split_row(p.pieces, p.rows, way);
  p.lanes = s.lanes;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MK_BF16) e = o8 ? launch_norm<__nv_bfloat16, true>(p, s, way, st) : launch_norm<__nv_bfloat16, false>(p, s, way, st);
  else if (dtype == MK_F16) e = o8 ? launch_norm<__half, true>(p, s, way, st) : launch_norm<__half, false>(p, s, way, st);
  else e = o8 ? launch_norm<float, true>(p, s, way, st) : launch_norm<float, false>(p, s, way, st);
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
  const int esz = size_of(dtype);
  NormParams p;
  std::memset(&p, 0, sizeof(p));
  if (!read_rows(dy, esz, false, tokens, heads, n, p.x) || !read_rows(h, esz, false, tokens, heads, n, p.h) ||
      !read_rows(dx, esz, true, tokens, heads, n, p.y) || (dh && !read_rows(dh, esz, false, tokens, heads, n, p.r)))
    return MK_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(weight) & (size_of(weight_dtype) - 1)) return MK_ERR_INVALID;
  p.w = static_cast<const char*>(weight);
  p.w_f32 = weight_dtype == MK_F32;
  p.part = dweight ? static_cast<float*>(workspace) : nullptr;
  p.rows = static_cast<unsigned>(tokens * heads);
  p.heads = static_cast<unsigned>(heads);
  p.n = n;
  p.eps = eps;
  RowsOf* all[4] = {&p.h, &p.x, &p.y, &p.r};
  const Way way = way_of(p, all, dh ? 4 : 3, nullptr, tokens, heads, esz);
  const Split s = split_grad(p.pieces, way);
  p.lanes = s.lanes;
  cudaError_t e;
  if (dtype == MK_BF16) e = launch_grad<__nv_bfloat16>(p, s, way, st);
  else if (dtype == MK_F16) e = launch_grad<__half>(p, s, way, st);
  else e = launch_grad<float>(p, s, way, st);
  if (e != cudaSuccess) return MK_ERR_CUDA;
  if (!dweight) return MK_OK;
  ColumnParams c = {p.part, dweight, n, grad_blocks(p.rows, s, way, p.classes), weight_dtype};
  e = launch_dependent(mk_norm_columns_kernel, dim3((n + 31) / 32), dim3(c.parts > 64 ? 1024 : 256), st, c);
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // extern "C"
