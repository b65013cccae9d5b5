// mk_rope.cu -- rotary positions, and the append of a step's keys and values
// to a paged cache with the rotation applied on the way.
//
// A head's pair (a, b) at position p with frequency f becomes
//   (a cos t - b sin t, b cos t + a sin t) * magnitude,   t = p f;
// the gradient of that map is the same with -t.  The pair is (x_i, x_{i+rot/2})
// or (x_{2i}, x_{2i+1}); elements past rot are copied.
//
// Angles: p f in fp32 would be off by p f 2^-24 (0.06 rad at p = 10^6).  Here
// f / 2 pi is taken as a 64-bit fraction of a turn and multiplied by the
// integer p modulo 2^64, which drops whole turns exactly; the upper 32 bits,
// as a signed fraction of a half turn, go through sincospif: about 1e-7 rad, and
// p times the error of the fraction, which is that of two 64-bit products and of
// its 64 bits: 2^-52 p f + 2^-62 p.  A block computes the cosines and sines of its tokens once,
// in shared memory, for all their heads.
//
// Both kernels move each value once and are bound by memory (large calls) or
// by the chain of dependent loads batch -> page -> store (a decode step), so
// the row loads are issued before that chain is walked.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk_seq.cuh"

namespace mk {

bool view_of(const mk_seq_batch* s, long long tokens, SeqView& out) {
  if (!s || s->batch < 0 || s->max_pages < 0 || tokens < 0 || tokens >= (1LL << 31)) return false;
  if (s->batch >= (1 << 24) || s->pages_stride < 0) return false;
  if (s->batch > 0 && (!s->cu_q || !s->kv_len || (!s->pages && s->max_pages > 0))) return false;
  if ((reinterpret_cast<uintptr_t>(s->cu_q) | reinterpret_cast<uintptr_t>(s->kv_len) |
       reinterpret_cast<uintptr_t>(s->pages)) & 3u)
    return false;
  out.cu_q = s->cu_q;
  out.kv_len = s->kv_len;
  out.pages = s->pages;
  out.pages_stride = s->pages_stride;
  out.batch = s->batch;
  out.max_pages = s->max_pages;
  out.tokens = static_cast<int>(tokens);
  return true;
}

bool view_of(const mk_kv_cache* c, CacheView& out) {
  if (!c || c->heads < 1 || c->heads > 1024 || c->d < 2 || c->d > 512 || c->n_pages < 0) return false;
  if (c->n_pages >= (1LL << 31)) return false;
  if (c->dtype != MK_BF16 && c->dtype != MK_F16 && c->dtype != MK_E4M3) return false;
  int lg = 0;
  while ((1 << lg) < c->page_size && lg < 30) ++lg;
  if (c->page_size < 8 || c->page_size > 256 || (1 << lg) != c->page_size) return false;
  if (c->page_stride < 0 || c->head_stride < 0 || c->slot_stride <= 0) return false;
  // pages or heads that share their memory: appends would race, and a tensor map has no stride of 0
  if ((c->page_stride == 0 && c->n_pages > 1) || (c->head_stride == 0 && c->heads > 1)) return false;
  if (c->n_pages > 0 && (!c->k || !c->v)) return false;
  if (c->dtype == MK_E4M3 && c->n_pages > 0 && (!c->k_scale || !c->v_scale)) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v);
  const long long size = (c->dtype == MK_E4M3) ? 1 : 2;
  // rows of whole 16-byte pieces, as for every operand of the library
  if ((a & 15u) || ((c->page_stride | c->head_stride | c->slot_stride) * size & 15)) return false;
  if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3u) return false;
  out.k = c->k;
  out.v = c->v;
  out.k_scale = c->k_scale;
  out.v_scale = c->v_scale;
  out.page_stride = c->page_stride;
  out.head_stride = c->head_stride;
  out.slot_stride = c->slot_stride;
  out.n_pages = c->n_pages;
  out.heads = c->heads;
  out.d = c->d;
  out.page_size = c->page_size;
  out.page_log2 = lg;
  return true;
}

namespace {

constexpr int RP_THREADS = 256;
constexpr int RP_UNITS = 4;            // units (2 x 16 bytes) a thread loads before it uses any
constexpr int RP_TABLE = 4096;         // (token, frequency) entries of a block's table: 32 KB
constexpr int RP_TOKENS = 64;          // tokens of a block at most
constexpr int RP_FREQS = 256;          // frequencies at most
constexpr int AP_CHUNK = 32;           // tokens of a page whose angles are in the table at once
constexpr int AP_HEADS = 4;            // heads of a block of the 8-bit append: 8 warps, k and v each

// A thread's place in a block's work (token, row, unit of the row; or token, frequency): found by
// multiplication and counted up from there.
struct Divide {
  uint32_t by, m;                            // m = ceil(2^32 / by): exact for numbers below 2^32 / by
  __host__ void set(int d) {
    by = static_cast<uint32_t>(std::max(1, d));
    m = static_cast<uint32_t>((0x100000000ull + by - 1) / by);
  }
  __device__ __forceinline__ int of(int n) const { return by == 1 ? n : static_cast<int>(__umulhi(n, m)); }
};
struct Place {
  int tok, row, u;
  __device__ __forceinline__ Place() {}
  __device__ __forceinline__ Place(int i, const Divide& rows, const Divide& units) {
    const int r = units.of(i);
    u = i - r * units.by;
    tok = rows.of(r);
    row = r - tok * rows.by;
  }
  __device__ __forceinline__ void add(const Place& step, const Divide& rows, const Divide& units) {
    u += step.u;
    row += step.row;
    tok += step.tok;
    if (u >= static_cast<int>(units.by)) {
      u -= units.by;
      ++row;
    }
    if (row >= static_cast<int>(rows.by)) {
      row -= rows.by;
      ++tok;
    }
  }
};

struct Rotation {
  const double* freqs;
  const void* positions;
  long long start;
  int positions_64, rot, inverse;
  float magnitude;
};

struct RowsParams {
  const void* x;                       // rope's input / the queries
  void* y;
  long long xs_t, xs_h, ys_t, ys_h;    // element strides of tokens and heads
  const void* nk;                      // new keys and values [tokens x heads]
  const void* nv;
  long long ks_t, ks_h, vs_t, vs_h;
  Rotation r;
  SeqView s;
  CacheView c;
  uint32_t* hdr;
  int heads, d, units;                 // query rows of a token; units of a row
  Divide by_rows, by_units, by_half;   // a block's rows of a token, units, frequencies
  int tokens, block_tokens, block_rows;
  int row_blocks;                      // blocks of rows per block of tokens
  int piece_blocks, head_blocks;       // 8-bit append: blocks that quantise come first
  int table;                           // entries of a block's cosine table (in shared memory, the sines after it)
};

__device__ __forceinline__ long long rope_position(const Rotation& r, int t, long long own) {
  if (r.positions == nullptr) return own;
  return r.positions_64 ? static_cast<const long long*>(r.positions)[t]
                        : static_cast<long long>(static_cast<const int*>(r.positions)[t]);
}

// The frequencies as 64-bit fractions of a turn, once a block: 64-bit floating point is slow here
// (2 operations a clock and SM; done for every angle it took half of a large call's time).
__device__ __forceinline__ void rope_turns(const Rotation& r, unsigned long long* turns) {
  for (int i = threadIdx.x; i < (r.rot >> 1); i += RP_THREADS) {
    double turn = r.freqs[i] * 0.15915494309189533577;       // 1 / (2 pi)
    turn -= floor(turn);
    turns[i] = __double2ull_rn(turn * 18446744073709551616.0);
  }
}

// The cosine / sine table of nt tokens, times the magnitude: entry tok * rot/2 + i (see the head of the file).
__device__ __forceinline__ void rope_table(const Rotation& r, const Divide& by_half, int nt, const long long* pos,
                                           const unsigned long long* turns, float* tc, float* ts) {
  const int half = r.rot >> 1;
  const float ms = r.inverse ? -r.magnitude : r.magnitude;
  for (int e = threadIdx.x; e < nt * half; e += RP_THREADS) {
    const int tok = by_half.of(e);
    const unsigned long long a = static_cast<unsigned long long>(pos[tok]) * turns[e - tok * half];
    float c, s;
    sincospif(static_cast<float>(static_cast<int>(a >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31
    tc[e] = c * r.magnitude;
    ts[e] = s * ms;
  }
}

// Where the new token at position pos of sequence b goes: its page and slot,
// page -1 where there is none (recorded as an error).
__device__ __forceinline__ int cache_page(const RowsParams& p, int b, long long pos) {
  const long long lp = pos >> p.c.page_log2;
  if (pos < 0 || lp >= p.s.max_pages) {
    seq_error(p.hdr, MK_ERR_CAPACITY, WHERE_COPY, b);
    return -1;
  }
  const int page = p.s.pages[b * p.s.pages_stride + lp];
  if (page < 0 || page >= p.c.n_pages) {
    seq_error(p.hdr, MK_ERR_INVALID, WHERE_COPY, b);
    return -1;
  }
  return page;
}

// n strides, n >= 0: a 32- by 64-bit product (strides may be negative: modulo 2^64).
__device__ __forceinline__ long long offset(int n, long long stride) {
  return static_cast<long long>(static_cast<unsigned>(n) * static_cast<unsigned long long>(stride));
}

// One unit of a row, 2 N elements: N pairs, or 2 N elements that are copied.
template <class T, bool INTER, bool VEC>
struct Unit {
  static constexpr int N = VEC ? Piece<T>::N : 1;
  uint4 w0, w1;                        // VEC: 16 bytes each; else one element each, as fp32 bits
  // element offsets of the two halves
  static __device__ __forceinline__ void where(int u, int rot, bool rotated, int& o0, int& o1) {
    if (!INTER && rotated && 2 * N * u < rot) {
      o0 = N * u;
      o1 = o0 + (rot >> 1);
    } else {
      o0 = 2 * N * u;
      o1 = o0 + N;
    }
  }
  __device__ __forceinline__ void load(const T* row, int o0, int o1) {
    if (VEC) {
      w0 = ld_stream_v4(row + o0);
      w1 = ld_stream_v4(row + o1);
    } else {
      w0.x = __float_as_uint(Piece<T>::one(row[o0]));
      w1.x = __float_as_uint(Piece<T>::one(row[o1]));
    }
  }
  __device__ __forceinline__ void get(float (&a)[N], float (&b)[N]) const {
    if constexpr (VEC) {
      Piece<T>::get(w0, a);
      Piece<T>::get(w1, b);
    } else {
      a[0] = __uint_as_float(w0.x);
      b[0] = __uint_as_float(w1.x);
    }
  }
  // pairs i = N u .. N u + N - 1 turned by the table's angles, in fp32
  static __device__ __forceinline__ void turn(float (&a)[N], float (&b)[N], const float* tc, const float* ts) {
    float x[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = a[i];
      x[N + i] = b[i];
    }
    float cs[N], sn[N];
    if constexpr (VEC) {                     // the table's rows are whole 16-byte pieces here
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        *reinterpret_cast<float4*>(cs + i) = *reinterpret_cast<const float4*>(tc + i);
        *reinterpret_cast<float4*>(sn + i) = *reinterpret_cast<const float4*>(ts + i);
      }
    } else {
      cs[0] = tc[0];
      sn[0] = ts[0];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float c = cs[i], s = sn[i];
      float& lo = INTER ? x[2 * i] : x[i];
      float& hi = INTER ? x[2 * i + 1] : x[N + i];
      const float u = lo, v = hi;
      lo = fmaf(u, c, -__fmul_rn(v, s));      // written out: the same bits in every variant
      hi = fmaf(v, c, __fmul_rn(u, s));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      a[i] = x[i];
      b[i] = x[N + i];
    }
  }
  static __device__ __forceinline__ void store(T* row, int o0, int o1, const float (&a)[N], const float (&b)[N]) {
    if constexpr (VEC) {
      *reinterpret_cast<uint4*>(row + o0) = Piece<T>::put(a);
      *reinterpret_cast<uint4*>(row + o1) = Piece<T>::put(b);
    } else {
      row[o0] = Piece<T>::of(a[0]);
      row[o1] = Piece<T>::of(b[0]);
    }
  }
  __device__ __forceinline__ void copy(T* row, int o0, int o1) const {   // the values as they are
    if constexpr (VEC) {
      *reinterpret_cast<uint4*>(row + o0) = w0;
      *reinterpret_cast<uint4*>(row + o1) = w1;
    } else {
      row[o0] = Piece<T>::of(__uint_as_float(w0.x));
      row[o1] = Piece<T>::of(__uint_as_float(w1.x));
    }
  }
};

// Rows of a block of tokens: the p.heads rows of x go rotated to y; with a
// 16-bit cache also the token's new keys (rotated) and values (copied) to
// their slots.  One unit of 2 x 16 bytes a thread and step: 256 bytes of a row
// by 8 neighbouring threads.  32768 tokens x 8 heads x 128, bf16: 25 us, 5.4 TB/s (79 % of a plain
// copy's rate); as much arithmetic as memory binds it (the issue slots are 60 % full: indices,
// conversions, the angles of a block's tokens).
template <class T, bool INTER, bool VEC, bool SEQ, bool CACHE>
__device__ __forceinline__ void rows_block(const RowsParams& p, int block, float* tc, float* ts) {
  using U = Unit<T, INTER, VEC>;
  constexpr int N = U::N;
  __shared__ long long pos[RP_TOKENS];
  __shared__ long long slot[RP_TOKENS];      // element offset of the token's slot in the cache, -1: none
  __shared__ unsigned long long turns[RP_FREQS];
  const int tb = block / p.row_blocks, rb = block - tb * p.row_blocks;
  const int t0 = tb * p.block_tokens, nt = min(p.block_tokens, p.tokens - t0);
  const int rows_all = p.heads + (CACHE ? 2 * p.c.heads : 0);
  const int r0 = rb * p.block_rows, nr = min(p.block_rows, rows_all - r0);
  const int total = nt * nr * p.units;
  const int half = p.r.rot >> 1;
  U un[RP_UNITS];
  const Place step(RP_THREADS, p.by_rows, p.by_units);
  Place at[RP_UNITS];
  at[0] = Place(threadIdx.x, p.by_rows, p.by_units);
#pragma unroll
  for (int j = 1; j < RP_UNITS; ++j) {
    at[j] = at[j - 1];
    at[j].add(step, p.by_rows, p.by_units);
  }
  const T* x0 = static_cast<const T*>(p.x) + t0 * p.xs_t;
  const T* k0 = CACHE ? static_cast<const T*>(p.nk) + t0 * p.ks_t : nullptr;
  const T* v0 = CACHE ? static_cast<const T*>(p.nv) + t0 * p.vs_t : nullptr;
  T* y0 = static_cast<T*>(p.y) + t0 * p.ys_t;
  auto load = [&](const Place& at, U& w) {
    int o0, o1;
    const int row = r0 + at.row;
    const T* src;
    if (!CACHE || row < p.heads) src = x0 + offset(at.tok, p.xs_t) + offset(row, p.xs_h);
    else if (row < p.heads + p.c.heads) src = k0 + offset(at.tok, p.ks_t) + offset(row - p.heads, p.ks_h);
    else src = v0 + offset(at.tok, p.vs_t) + offset(row - p.heads - p.c.heads, p.vs_h);
    U::where(at.u, p.r.rot, !CACHE || row < p.heads + p.c.heads, o0, o1);
    w.load(src, o0, o1);
  };
#pragma unroll
  for (int j = 0; j < RP_UNITS; ++j) {
    const int i = threadIdx.x + j * RP_THREADS;
    if (i < total) load(at[j], un[j]);
  }
  rope_turns(p.r, turns);
  if (SEQ) {
    for (int tok = threadIdx.x >> 5; tok < nt; tok += RP_THREADS / 32) {
      const int t = t0 + tok;
      const int b = warp_last_le(p.s.batch + 1, t, [&](int i) { return p.s.cu_q[i]; });
      if ((threadIdx.x & 31) == 0) {
        long long own = 0, at = -1;
        if (b >= 0 && b < p.s.batch) {
          own = static_cast<long long>(p.s.kv_len[b]) - p.s.cu_q[b + 1] + t;
          if (CACHE) {
            const int page = cache_page(p, b, own);
            if (page >= 0) at = page * p.c.page_stride + (own & (p.c.page_size - 1)) * p.c.slot_stride;
          }
        }
        pos[tok] = rope_position(p.r, t, own);
        slot[tok] = at;
      }
    }
  } else {
    for (int tok = threadIdx.x; tok < nt; tok += RP_THREADS) pos[tok] = rope_position(p.r, t0 + tok, p.r.start + t0 + tok);
  }
  __syncthreads();
  if (p.r.rot > 0) {
    rope_table(p.r, p.by_half, nt, pos, turns, tc, ts);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < RP_UNITS; ++j) {
    const int i = threadIdx.x + j * RP_THREADS;
    if (i >= total) break;
    int o0, o1;
    const int tok = at[j].tok, row = r0 + at[j].row, u = at[j].u;
    const bool is_v = CACHE && row >= p.heads + p.c.heads;
    T* dst;
    if (!CACHE || row < p.heads) {
      dst = y0 + offset(tok, p.ys_t) + offset(row, p.ys_h);
    } else {
      if (slot[tok] < 0) continue;
      const int h = row - p.heads - (is_v ? p.c.heads : 0);
      dst = static_cast<T*>(is_v ? p.c.v : p.c.k) + slot[tok] + offset(h, p.c.head_stride);
    }
    U::where(u, p.r.rot, !is_v, o0, o1);
    if (is_v || 2 * N * u >= p.r.rot) {
      un[j].copy(dst, o0, o1);
    } else {
      float a[N], b[N];
      un[j].get(a, b);
      U::turn(a, b, tc + tok * half + N * u, ts + tok * half + N * u);
      U::store(dst, o0, o1, a, b);
    }
  }
}

template <class T, bool INTER, bool VEC, bool SEQ, bool CACHE>
__global__ void __launch_bounds__(RP_THREADS, VEC ? 4 : 1) mk_rows_kernel(const __grid_constant__ RowsParams p) {
  extern __shared__ __align__(16) float table[];
  rows_block<T, INTER, VEC, SEQ, CACHE>(p, blockIdx.x, table, table + p.table);
}

// ------------------------------------------------------------------ 8-bit cache

__device__ __forceinline__ float2 e4m3_pair(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  __half2 x;
  memcpy(&x, &h, 4);
  return __half22float2(x);
}

// The least power of two s >= 2^-100 with amax <= 448 s (amax finite).
__device__ __forceinline__ float e4m3_scale(float amax) {
  int e;
  const float m = frexpf(amax / E4M3_MAX, &e);
  return ldexpf(1.f, amax > 0.f ? max(m > 0.5f ? e : e - 1, -100) : -100);
}

// A piece: the new tokens of one sequence that share a page; a block has one
// piece and up to four heads, a warp the keys or the values of one of them.
// The warp reads its rows twice (the second time out of L1 / L2): once for the
// largest finite magnitude, once to store the codes; older codes of the page
// are read and rounded again only where the scale grows.  18000 tokens in 5
// prompts, 8 heads x 128, bf16, with 32 query heads rotated: 78 us in all,
// 4.8 TB/s (70 % of a plain copy's rate).
template <class T, bool INTER>
__device__ __forceinline__ void quant_block(const RowsParams& p, float* tc, float* ts) {
  using U = Unit<T, INTER, true>;
  constexpr int N = U::N;
  __shared__ long long pos[AP_CHUNK];
  __shared__ unsigned long long turns[RP_FREQS];
  __shared__ int sh[5];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = blockIdx.x / p.head_blocks, hb = blockIdx.x - piece * p.head_blocks;
  const int size = p.c.page_size;
  rope_turns(p.r, turns);
  if (warp == 0) {
    // sequence b's pieces start at number cu_q[b] / page + 2 b: room for all of them
    const int b = warp_last_le(p.s.batch, piece, [&](int i) { return (p.s.cu_q[i] >> p.c.page_log2) + 2 * i; });
    if (lane == 0) {
      int page = -1, lo = 0, hi = 0, tok = 0, fresh = 0;
      if (b >= 0) {
        const int c0 = p.s.cu_q[b], c1 = min(p.s.cu_q[b + 1], p.s.tokens);
        const long long len = p.s.kv_len[b], first = len - (c1 - c0);
        const int number = piece - ((c0 >> p.c.page_log2) + 2 * b);
        const long long lp = (max(first, 0LL) >> p.c.page_log2) + number;
        const long long from = max(first, lp << p.c.page_log2);
        const long long to = min(len, (lp + 1) << p.c.page_log2);
        if (first < 0 && number == 0 && c1 > c0) seq_error(p.hdr, MK_ERR_CAPACITY, WHERE_COPY, b);
        if (c0 >= 0 && c1 > c0 && from < to) {
          page = cache_page(p, b, from);
          lo = static_cast<int>(from & (size - 1));
          hi = lo + static_cast<int>(to - from);
          tok = c0 + static_cast<int>(from - first);
          fresh = (lo == 0);
          pos[0] = from;
        }
      }
      sh[0] = page; sh[1] = lo; sh[2] = hi; sh[3] = tok; sh[4] = fresh;
    }
  }
  __syncthreads();
  const int page = sh[0], lo = sh[1], n = sh[2] - sh[1], tok0 = sh[3], fresh = sh[4];
  const long long own0 = pos[0];
  if (page < 0) return;                       // the whole block
  const int h = hb * AP_HEADS + (warp >> 1);
  const bool is_v = warp & 1, act = h < p.c.heads;
  const int half = p.r.rot >> 1;
  const int upr = p.units;                    // units (16 elements) of a row
  const T* src = is_v ? static_cast<const T*>(p.nv) + h * p.vs_h : static_cast<const T*>(p.nk) + h * p.ks_h;
  const long long st = is_v ? p.vs_t : p.ks_t;
  uint8_t* dst = static_cast<uint8_t*>(is_v ? p.c.v : p.c.k) + page * p.c.page_stride + h * p.c.head_stride;
  float* scale_at = (is_v ? p.c.v_scale : p.c.k_scale) + static_cast<long long>(page) * p.c.heads + h;
  float amax = 0.f, scale = 0.f, inv = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int c0 = 0; c0 < n; c0 += AP_CHUNK) {
      const int nc = min(AP_CHUNK, n - c0);
      if (half > 0 && (pass == 0 || n > AP_CHUNK)) {   // one chunk: its table still stands in the second pass
        __syncthreads();
        if (threadIdx.x < nc) pos[threadIdx.x] = rope_position(p.r, tok0 + c0 + threadIdx.x, own0 + c0 + threadIdx.x);
        __syncthreads();
        rope_table(p.r, p.by_half, nc, pos, turns, tc, ts);
        __syncthreads();
      }
      if (!act) continue;
      // two units a lane in flight
      for (int i0 = lane; i0 < nc * upr; i0 += 64) {
        U w[2];
        int tk[2], uu[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = i0 + 32 * k;
          if (i < nc * upr) {
            int o0, o1;
            tk[k] = p.by_units.of(i);
            uu[k] = i - tk[k] * upr;
            U::where(uu[k], p.r.rot, !is_v, o0, o1);
            const T* row = src + (tok0 + c0 + tk[k]) * st;
            w[k].w0 = *reinterpret_cast<const uint4*>(row + o0);
            w[k].w1 = *reinterpret_cast<const uint4*>(row + o1);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (i0 + 32 * k >= nc * upr) break;
          float a[N], b[N];
          w[k].get(a, b);
          if (!is_v && 2 * N * uu[k] < p.r.rot)
            U::turn(a, b, tc + tk[k] * half + N * uu[k], ts + tk[k] * half + N * uu[k]);
          if (pass == 0) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const float fa = fabsf(a[e]), fb = fabsf(b[e]);
              if (fa <= 3.4028235e38f) amax = fmaxf(amax, fa);   // finite ones only
              if (fb <= 3.4028235e38f) amax = fmaxf(amax, fb);
            }
          } else {
            int o0, o1;
            U::where(uu[k], p.r.rot, !is_v, o0, o1);
            uint8_t* row = dst + (lo + c0 + tk[k]) * p.c.slot_stride;
            *reinterpret_cast<uint2*>(row + o0) =
                make_uint2(e4m3x4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv),
                           e4m3x4(a[4] * inv, a[5] * inv, a[6] * inv, a[7] * inv));
            *reinterpret_cast<uint2*>(row + o1) =
                make_uint2(e4m3x4(b[0] * inv, b[1] * inv, b[2] * inv, b[3] * inv),
                           e4m3x4(b[4] * inv, b[5] * inv, b[6] * inv, b[7] * inv));
          }
        }
      }
    }
    if (pass == 0 && act) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      scale = e4m3_scale(amax);
      if (!fresh) {
        const float had = *scale_at;
        if (had >= scale) {
          scale = had;
        } else {
          const float ratio = had / scale;
          for (int i = lane; i < lo * (p.d >> 2); i += 32) {
            const int row = i / (p.d >> 2), q = i - row * (p.d >> 2);
            uint32_t* at = reinterpret_cast<uint32_t*>(dst + row * p.c.slot_stride) + q;
            const uint32_t w = *at;
            const float2 x = e4m3_pair(w & 0xffffu), y = e4m3_pair(w >> 16);
            *at = e4m3x4(x.x * ratio, x.y * ratio, y.x * ratio, y.y * ratio);
          }
        }
      }
      inv = 1.f / scale;      // exact: a power of two
      __syncwarp();           // every lane has read the old scale
      if (lane == 0) *scale_at = scale;
    }
  }
}

// The blocks that quantise come first (they are the long ones); the rest rotate the queries.
template <class T, bool INTER>
__global__ void __launch_bounds__(RP_THREADS, 3) mk_append8_kernel(const __grid_constant__ RowsParams p) {
  extern __shared__ __align__(16) float table[];
  float* ts = table + p.table;
  if (static_cast<int>(blockIdx.x) < p.piece_blocks) quant_block<T, INTER>(p, table, ts);
  else rows_block<T, INTER, true, true, false>(p, blockIdx.x - p.piece_blocks, table, ts);
}

// ------------------------------------------------------------------ launches

// How a call's rows are split: about 1024 units a block (4 a thread, all in
// flight), so several tokens where they are small, and several blocks a token
// where it is large; calls with less than 304 such blocks, two for each of 152 SMs,
// (a decode step) get 256 units a block, to be spread over more SMs.  Rows of at most RP_TABLE angles a block.  With 256 / 1024
// units, calls in a graph: 16 tokens x 40 heads x 128 2.5 / 3.1 us, an append
// for 64 sequences 3.4 / 3.9 us; 32768 tokens x 8 heads, forward and gradient,
// 78 / 56 us, an append of 18000 tokens to an 8-bit cache 107 / 78 us.
void split_rows(RowsParams& p, int rows) {
  const long long per_token = static_cast<long long>(rows) * p.units;
  const long long target = per_token * p.tokens < 1024LL * 304 ? 256 : 256 * RP_UNITS;
  const int half = std::max(1, p.r.rot / 2);
  int tb = static_cast<int>(std::max(1LL, target / std::max(1LL, per_token)));
  tb = std::min({tb, RP_TOKENS, std::max(1, RP_TABLE / half)});
  p.block_tokens = tb;
  p.table = (tb * (p.r.rot / 2) + 3) & ~3;
  int br = rows;
  if (tb == 1) br = static_cast<int>(std::min<long long>(rows, std::max(1LL, target / p.units)));
  p.block_rows = std::max(1, br);
  p.row_blocks = (rows + p.block_rows - 1) / p.block_rows;
  p.by_rows.set(p.block_rows);               // (where the last block has fewer, its block is of one token)
}

template <class T, bool INTER, bool VEC, bool SEQ, bool CACHE>
cudaError_t launch_rows(RowsParams& p, cudaStream_t s) {
  p.units = p.d / (2 * Unit<T, INTER, VEC>::N);
  p.by_units.set(p.units);
  p.by_half.set(p.r.rot / 2);
  const int rows = p.heads + (CACHE ? 2 * p.c.heads : 0);
  split_rows(p, rows);
  const long long blocks = ceil_div_ll(p.tokens, p.block_tokens) * p.row_blocks;
  if (blocks >= (1LL << 31)) return cudaErrorInvalidValue;
  mk_rows_kernel<T, INTER, VEC, SEQ, CACHE><<<static_cast<unsigned>(blocks), RP_THREADS, 8 * p.table, s>>>(p);
  return cudaGetLastError();
}
template <class T, bool SEQ, bool CACHE>
cudaError_t launch_rows(RowsParams& p, bool inter, bool vec, cudaStream_t s) {
  if (inter) return vec ? launch_rows<T, true, true, SEQ, CACHE>(p, s) : launch_rows<T, true, false, SEQ, CACHE>(p, s);
  return vec ? launch_rows<T, false, true, SEQ, CACHE>(p, s) : launch_rows<T, false, false, SEQ, CACHE>(p, s);
}

template <class T, bool INTER>
cudaError_t launch_append8(RowsParams& p, cudaStream_t s) {
  p.units = p.d / 16;
  p.by_units.set(p.units);
  p.by_half.set(p.r.rot / 2);
  p.head_blocks = (p.c.heads + AP_HEADS - 1) / AP_HEADS;
  const long long pieces = (p.tokens >> p.c.page_log2) + 2LL * p.s.batch;
  long long blocks = 0;
  p.row_blocks = 1;
  p.block_tokens = 1;
  p.block_rows = 1;
  if (p.heads > 0) {
    split_rows(p, p.heads);
    blocks = ceil_div_ll(p.tokens, p.block_tokens) * p.row_blocks;
  }
  if (pieces * p.head_blocks + blocks >= (1LL << 31)) return cudaErrorInvalidValue;
  p.piece_blocks = static_cast<int>(pieces * p.head_blocks);
  p.table = std::max(p.table, p.r.rot / 2 * std::min(p.c.page_size, AP_CHUNK));
  mk_append8_kernel<T, INTER><<<static_cast<unsigned>(p.piece_blocks + blocks), RP_THREADS, 8 * p.table, s>>>(p);
  return cudaGetLastError();
}

bool rotation_ok(const mk_rotation* r, int d, Rotation& out) {
  std::memset(&out, 0, sizeof(out));
  if (!r) return true;
  if (r->rot < 0 || r->rot > d || (r->rot & 1)) return false;
  if (r->rot > 0 && !r->freqs) return false;
  if (!std::isfinite(r->magnitude)) return false;
  if (reinterpret_cast<uintptr_t>(r->freqs) & 7u) return false;
  if (reinterpret_cast<uintptr_t>(r->positions) & (r->positions_64 ? 7u : 3u)) return false;
  out.freqs = r->freqs;
  out.positions = r->positions;
  out.positions_64 = r->positions_64;
  out.start = r->start;
  out.rot = r->rot;
  out.inverse = r->inverse;
  out.magnitude = r->magnitude;
  return true;
}

// 16-byte pieces throughout: base, strides, and the rotated and copied parts.
bool pieces_ok(const void* x, long long st, long long sh, int esz) {
  return !(reinterpret_cast<uintptr_t>(x) & 15u) && !((st * esz) & 15) && !((sh * esz) & 15);
}
// Whether rows that are written have memory of their own (expanded tensors do not).
bool rows_apart(long long st, long long sh, long long tokens, int heads) {
  return (st != 0 || tokens <= 1) && (sh != 0 || heads <= 1);
}
bool rows_vec(int d, int rot, int n) { return rot % (2 * n) == 0 && d % (2 * n) == 0; }

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

mk_status mk_rope(const void* x, void* y, mk_dtype dtype, long long tokens, int heads, int d, long long x_token,
                  long long x_head, long long y_token, long long y_head, const mk_rotation* rotation,
                  mk_stream_t stream) {
  if (dtype != MK_BF16 && dtype != MK_F16 && dtype != MK_F32) return MK_ERR_INVALID;
  if (tokens < 0 || heads < 0 || d < 2 || (d & 1) || d > 512 || !rotation) return MK_ERR_INVALID;
  if (tokens >= (1LL << 31) || heads > (1 << 20)) return MK_ERR_INVALID;
  RowsParams p;
  std::memset(&p, 0, sizeof(p));
  if (!rotation_ok(rotation, d, p.r)) return MK_ERR_INVALID;
  if (tokens == 0 || heads == 0) return MK_OK;
  const int esz = dtype == MK_F32 ? 4 : 2;
  if (!x || !y || ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & (esz - 1))) return MK_ERR_INVALID;
  if (!rows_apart(y_token, y_head, tokens, heads)) return MK_ERR_INVALID;
  p.x = x;
  p.y = y;
  p.xs_t = x_token;
  p.xs_h = x_head;
  p.ys_t = y_token;
  p.ys_h = y_head;
  p.heads = heads;
  p.d = d;
  p.tokens = static_cast<int>(tokens);
  const bool inter = rotation->interleaved != 0;
  // 16-byte pieces where every row has them; else element by element
  const bool vec = rows_vec(d, p.r.rot, 16 / esz) && pieces_ok(x, x_token, x_head, esz) &&
                   pieces_ok(y, y_token, y_head, esz);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == MK_BF16) e = launch_rows<__nv_bfloat16, false, false>(p, inter, vec, s);
  else if (dtype == MK_F16) e = launch_rows<__half, false, false>(p, inter, vec, s);
  else e = launch_rows<float, false, false>(p, inter, vec, s);
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

mk_status mk_kv_append(const mk_kv_cache* cache, const void* k, const void* v, mk_dtype dtype, long long tokens,
                       long long k_token, long long k_head, long long v_token, long long v_head, const void* q,
                       void* q_out, int heads_q, long long q_token, long long q_head, long long qo_token,
                       long long qo_head, const mk_seq_batch* seqs, const mk_rotation* rotation, void* workspace,
                       size_t ws_bytes, mk_stream_t stream) {
  if (dtype != MK_BF16 && dtype != MK_F16) return MK_ERR_INVALID;
  RowsParams p;
  std::memset(&p, 0, sizeof(p));
  if (!view_of(cache, p.c) || !view_of(seqs, tokens, p.s)) return MK_ERR_INVALID;
  if (cache->dtype != MK_E4M3 && cache->dtype != dtype) return MK_ERR_INVALID;
  const int d = cache->d;
  if ((d & 1) || !rotation_ok(rotation, d, p.r)) return MK_ERR_INVALID;
  if (rotation && rotation->inverse) return MK_ERR_INVALID;
  if (heads_q < 0 || heads_q > (1 << 20) || ((q == nullptr) != (q_out == nullptr))) return MK_ERR_INVALID;
  if (!q) heads_q = 0;
  if (!workspace || ws_bytes < WS_HDR_BYTES || (reinterpret_cast<uintptr_t>(workspace) & 15u)) return MK_ERR_INVALID;
  if (tokens == 0 || seqs->batch == 0) return MK_OK;
  if (!k || !v) return MK_ERR_INVALID;
  if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(q) |
        reinterpret_cast<uintptr_t>(q_out)) & 1u))
    return MK_ERR_INVALID;
  if (q && !rows_apart(qo_token, qo_head, tokens, heads_q)) return MK_ERR_INVALID;
  p.x = q;
  p.y = q_out;
  p.xs_t = q_token;
  p.xs_h = q_head;
  p.ys_t = qo_token;
  p.ys_h = qo_head;
  p.nk = k;
  p.nv = v;
  p.ks_t = k_token;
  p.ks_h = k_head;
  p.vs_t = v_token;
  p.vs_h = v_head;
  p.hdr = static_cast<uint32_t*>(workspace);
  p.heads = heads_q;
  p.d = d;
  p.tokens = static_cast<int>(tokens);
  const bool inter = rotation && rotation->interleaved;
  const bool vec = rows_vec(d, p.r.rot, 8) && pieces_ok(k, k_token, k_head, 2) && pieces_ok(v, v_token, v_head, 2) &&
                   (!q || (pieces_ok(q, q_token, q_head, 2) && pieces_ok(q_out, qo_token, qo_head, 2)));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == MK_E4M3) {
    if (!vec || p.r.rot / 2 * AP_CHUNK > RP_TABLE) return MK_ERR_INVALID;   // whole 16-element units only
    if (dtype == MK_BF16)
      e = inter ? launch_append8<__nv_bfloat16, true>(p, s) : launch_append8<__nv_bfloat16, false>(p, s);
    else
      e = inter ? launch_append8<__half, true>(p, s) : launch_append8<__half, false>(p, s);
  } else if (dtype == MK_BF16) {
    e = launch_rows<__nv_bfloat16, true, true>(p, inter, vec, s);
  } else {
    e = launch_rows<__half, true, true>(p, inter, vec, s);
  }
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // extern "C"
