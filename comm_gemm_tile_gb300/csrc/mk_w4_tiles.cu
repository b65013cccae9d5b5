// mk_w4_tiles.cu -- products with 4-bit weights for more than a handful of tokens, on tcgen05.
//
// A step is 128 rows of the matrix times 256 k, in two halves of 128 k.  Thread r of a
// half's warpgroup turns row r's 64 bytes of codes into 128 16-bit whole numbers (c - 8, exact) and
// stores them to its lane of tensor memory; one thread multiplies that with the
// tokens' 128 k in shared memory (A from tensor memory, M = 128, N = NT tokens, one
// accumulator for each group of the half); then thread r of two more warpgroups adds the
// accumulators of its lane, times its scales, to its sums of half the tokens in registers.
// Nothing is rounded to 16 bits but the output.  Each half has two or three places for its numbers, one or two for
// its accumulators in tensor memory, and a warp that issues its products (a look at a barrier takes 150
// cycles, a half's eight products of 64 tokens 350); codes and x come through rings of their own.
//
// Three launches.  w4_order_kernel copies x with each 8 values in the order in
// which a word's codes come out ((0, 4), (1, 5), (2, 6), (3, 7)) and, for zero points, forms
// sum x of every token and group.  The list of steps (token tile, row tile, k) is cut into equal
// runs, one for each CTA; a CTA writes the outputs of a row tile it has whole and leaves its
// part of others as fp32 in scratch; w4_join_kernel adds those in the order of k.
// Codes are loaded before the first kernel has ended: only x waits for it.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "mk_w4.h"

namespace mk {

namespace {

constexpr int WT_ROWS = 128;
constexpr int WT_MAX_CTAS = 152;
constexpr int WT_STEP = 256;           // k of a step
constexpr uint64_t WT_DRAIN_NS = 1000000000ull;

struct TileParams {
  CUtensorMap codes, x;
  W4Params w;
  uint32_t* hdr;
  const uint8_t* ordered;              // x as w4_order_kernel leaves it [m x k]
  float* sums;                         // [groups x pitch] sum x, zero points only
  float* part;                         // [CTAs x 2 x NT x 128]
  int sums_pitch;
  unsigned each, over;
  int whole_scales;                    // rows of scales are whole 16-byte pieces
  int ctas, steps, row_tiles, tok_tiles, NT;   // steps: of a tile
  long long wait_ns;
  int inject;
};

// CTA b's steps are start(b) .. start(b + 1) - 1, of all = ctas * each + over (fewer than 2^31).
__device__ __forceinline__ unsigned start_of(const TileParams& p, unsigned b) {
  return p.each * b + p.over * b / static_cast<unsigned>(p.ctas);
}

// ------------------------------------------------------------------ x in the order of the codes

// A block has 2048 k of a token, a thread 8 values.
template <class T>
__global__ void __launch_bounds__(256) w4_order_kernel(const __grid_constant__ TileParams p, int group) {
  griddep_launch_dependents();
  const int i = blockIdx.x * 256 + threadIdx.x;              // the i-th 8 values of a token
  const bool real = 8 * i < p.w.k;
  for (int tok = blockIdx.y; tok < p.w.m; tok += gridDim.y) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (real) {
      v = __ldg(reinterpret_cast<const uint4*>(p.w.x + tok * p.w.x_row) + i);
      uint32_t o[4];
      x_pairs(v, o);
      reinterpret_cast<uint4*>(const_cast<uint8_t*>(p.ordered))[static_cast<long long>(tok) * (p.w.k / 8) + i] =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (p.sums == nullptr) continue;
    float f[8], s = 0.f;
    Piece<T>::get(v, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += f[e];
    const int lanes = group / 8;                              // 4, 8 or 16 neighbours
    for (int o = lanes >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (real && (i & (lanes - 1)) == 0) p.sums[static_cast<long long>(i / lanes) * p.sums_pitch + tok] = s;
  }
}

// ------------------------------------------------------------------ the products

template <int NT, int GPC, bool ZEROS>
struct Tile {
  static constexpr int C = WT_ROWS * 128, SUMS = ZEROS ? GPC * NT * 4 : 0, X_TX = NT * 256 + SUMS;
  static constexpr int X = (X_TX + 1023) / 1024 * 1024;      // x of a half, then its groups' sums
  static constexpr int SC = 6, SX = NT == 64 ? 6 : 8;        // stages: steps of codes, halves of x
  static constexpr int XS = SC * C, BARS = XS + SX * X;
  static constexpr int SMEM = 1024 + BARS + 512;
  static constexpr int DP = GPC * NT <= 64 ? 4 : 2;          // places of accumulators, and of a half's numbers
  static constexpr int AP = (512 - DP * GPC * NT) / 128 > 3 ? 3 : (512 - DP * GPC * NT) / 128;
  static constexpr uint32_t A = 0, D = AP * 128;             // columns of tensor memory
  static_assert(D + DP * GPC * NT <= 512 && AP >= 2, "tensor memory");
  static_assert(SMEM <= 232448, "shared memory");
};
constexpr int WT_THREADS = 640;        // warps 0-7 codes, 8-15 sums, 16 loads codes, 17 loads x, 18 and 19 products
// barriers (byte offsets)
constexpr uint32_t B_CFULL = 0, B_CEMPTY = 64, B_XFULL = 128, B_XEMPTY = 192, B_AFULL = 256, B_AEMPTY = 304, B_DFULL = 352,
                   B_DEMPTY = 384, B_TMEM = 416, B_DEAD = 420;

__device__ __noinline__ bool wt_wait_slow(volatile int* dead, const TileParams& p, uint32_t bar, uint32_t parity, int where) {
  if (*dead) return false;
  const uint64_t t0 = globaltimer_ns();
  uint32_t it = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++it & 15u) == 0) {
      if (*dead) return false;
      if (globaltimer_ns() - t0 > static_cast<uint64_t>(p.wait_ns)) {
        seq_error(p.hdr, MK_ERR_TIMEOUT, where, blockIdx.x);
        *dead = 1;
        return false;
      }
    }
  }
  return true;
}
// False once the CTA has given up; then every wait returns at once.
__device__ __forceinline__ bool wt_wait(volatile int* dead, const TileParams& p, uint32_t bar, uint32_t parity, int where) {
  return mbar_test_wait(bar, parity) || wt_wait_slow(dead, p, bar, parity, where);
}
// Two or three barriers: looked at together, waited for one by one.
__device__ __forceinline__ bool wt_wait_warp(volatile int* dead, const TileParams& p, uint32_t bar0, uint32_t parity0, uint32_t bar1,
                                             uint32_t parity1, int where) {
  const bool a = mbar_test_wait(bar0, parity0), b = mbar_test_wait(bar1, parity1);
  if (__all_sync(0xffffffffu, a && b)) return true;
  return __all_sync(0xffffffffu, wt_wait(dead, p, bar0, parity0, where) && wt_wait(dead, p, bar1, parity1, where));
}
__device__ __forceinline__ bool wt_wait_warp(volatile int* dead, const TileParams& p, uint32_t bar0, uint32_t parity0, uint32_t bar1,
                                             uint32_t parity1, uint32_t bar2, uint32_t parity2, int where) {
  const bool a = mbar_test_wait(bar0, parity0), b = mbar_test_wait(bar1, parity1), c = mbar_test_wait(bar2, parity2);
  if (__all_sync(0xffffffffu, a && b && c)) return true;
  const bool all = wt_wait(dead, p, bar0, parity0, where) && wt_wait(dead, p, bar1, parity1, where) && wt_wait(dead, p, bar2, parity2, where);
  return __all_sync(0xffffffffu, all);
}
__device__ __forceinline__ bool wt_wait_warp(volatile int* dead, const TileParams& p, uint32_t bar, uint32_t parity, int where) {
  return __all_sync(0xffffffffu, wt_wait(dead, p, bar, parity, where));
}
__device__ __forceinline__ void wt_drain(const TileParams& p, uint32_t bar, uint32_t parity, int where) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > WT_DRAIN_NS) {
      seq_error(p.hdr, MK_ERR_TIMEOUT, where, blockIdx.x);
      return;
    }
}

// GPC: groups of a half (1, 2, 4 for groups of 128, 64, 32).
template <class T, int NT, int GPC, bool ZEROS>
__global__ void __launch_bounds__(WT_THREADS, 1) mk_w4_tiles_kernel(const __grid_constant__ TileParams p) {
  using L = Tile<NT, GPC, ZEROS>;
  constexpr int SC = L::SC, SX = L::SX, DP = L::DP, AP = L::AP;
  constexpr bool HALF = std::is_same<T, __half>::value;
  constexpr uint32_t IDESC = idesc_bf16_f32(WT_ROWS, NT, false, false) & (HALF ? ~((1u << 7) | (1u << 10)) : ~0u);
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem), bars = base + L::BARS;
  volatile int* dead = reinterpret_cast<volatile int*>(smem + L::BARS + B_DEAD);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned u0 = start_of(p, blockIdx.x);
  const int count = static_cast<int>(start_of(p, blockIdx.x + 1) - u0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < SC; ++i) {
      mbar_init(bars + B_CFULL + 8 * i, 1);
      mbar_init(bars + B_CEMPTY + 8 * i, 8);                 // the warps that read its halves
    }
    for (int i = 0; i < SX; ++i) {
      mbar_init(bars + B_XFULL + 8 * i, 1);
      mbar_init(bars + B_XEMPTY + 8 * i, 8);                 // the warps that add what came of it
    }
    for (int i = 0; i < 2 * AP; ++i) {
      mbar_init(bars + B_AFULL + 8 * i, 4);
      mbar_init(bars + B_AEMPTY + 8 * i, 1);
    }
    for (int i = 0; i < L::DP; ++i) {
      mbar_init(bars + B_DFULL + 8 * i, 1);
      mbar_init(bars + B_DEMPTY + 8 * i, 8);
    }
    *dead = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(bars + B_TMEM, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::BARS + B_TMEM);
  griddep_launch_dependents();
  const unsigned steps = p.steps, row_tiles = p.row_tiles;   // a step: token tile, row tile, place in k
  if (warp < 8) {
    // ---------------------------------------------------------------- codes to tensor memory
    const int h = warp >> 2, r = threadIdx.x & 127;
    const uint32_t ta = tmem + L::A + h * 64 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    for (int i = 0; i < count; ++i) {
      const int s = i % SC;
      const int place = i % AP;
      const uint32_t to = bars + 8 * (h + 2 * place), at = ta + 128 * place;
      // (a place's first use waits for the phase before the first, which has ended)
      if (!wt_wait_warp(dead, p, bars + B_CFULL + 8 * s, (i / SC) & 1, to + B_AEMPTY, (i / AP + 1) & 1, WHERE_COPY)) break;
      tc_fence_after();
      // the 128-byte swizzle of the codes' tile: 16-byte piece q of row r lies at q ^ (r & 7)
      const uint8_t* w = smem + s * L::C + r * 128;
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint4*>(w + 16 * ((4 * h + q) ^ (r & 7)));
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t o[32];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint4 u = v[2 * half + q];
          const uint32_t words[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t four[4];
            Codes<T>::pairs(words[e], four);
#pragma unroll
            for (int f = 0; f < 4; ++f) o[16 * q + 4 * e + f] = four[f];
          }
        }
        tc_st_32x32b_x32(at + 32 * half, o);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      // The codes' place is free only now that they have been used: released behind the loads, which were still on their
      // way, it was filled again before they came.
      if (lane == 0) {
        mbar_arrive(bars + B_CEMPTY + 8 * s);
        mbar_arrive(to + B_AFULL);
      }
    }
  } else if (warp < 16) {
    // ---------------------------------------------------------------- sums, of half the tokens
    constexpr int TOK = NT / 2;
    const int r = threadIdx.x & 127, t0 = warp < 12 ? 0 : TOK;
    const uint32_t td = tmem + L::D + t0 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    uint64_t acc[TOK / 2];                                   // two tokens each
#pragma unroll
    for (int e = 0; e < TOK / 2; ++e) acc[e] = 0;
    unsigned tile = u0 / steps, c = u0 - tile * steps;
    int row = tile % row_tiles * WT_ROWS + r, first = 0;
    // Scales and zero points, of rows past the last those of the last: 8 groups (PER steps) at once, loaded as many ahead
    // (a load of each step's own takes the load unit as long: every row has a line of its own); or, where rows of scales
    // are not whole 16-byte pieces, each step's, a step ahead.
    constexpr int PER = 4 / GPC;
    uint4 sc, sc_next, ze, ze_next;
    const T *ps, *pz;
    auto of_row = [&] {
      const long long at = static_cast<long long>(min(row, p.w.n - 1)) * p.w.groups;
      ps = static_cast<const T*>(p.w.scales) + at;
      pz = static_cast<const T*>(p.w.zeros) + at;
    };
    auto ahead = [&](unsigned c) {                           // the step's or its block's
      if (p.whole_scales) {
        sc_next = __ldg(reinterpret_cast<const uint4*>(ps) + c / PER);
        if (ZEROS) ze_next = __ldg(reinterpret_cast<const uint4*>(pz) + c / PER);
      } else {
        T v[8], u[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int g = c * (2 * GPC) + q;
          const bool real = q < 2 * GPC && g < p.w.groups;
          v[q] = real ? ps[g] : Piece<T>::of(0.f);
          u[q] = ZEROS && real ? pz[g] : Piece<T>::of(0.f);
        }
        memcpy(&sc_next, v, 16);
        memcpy(&ze_next, u, 16);
      }
    };
    of_row();
    ahead(c);
    bool fresh = true;                                       // sc_next is this step's
    for (int i = 0; i < count; ++i) {
      const bool ends = c + 1 == steps;
      const int row_now = row;
      if (fresh) {
        sc = sc_next;
        ze = ze_next;
      }
      if (ends) {
        row = (tile + 1) % row_tiles * WT_ROWS + r;
        of_row();
      }
      const unsigned after = ends ? 0 : c + 1, place_in = p.whole_scales ? c % PER : 0;
      // the next step's, if they are not in hand; what is loaded last is not used
      const bool had = fresh;
      fresh = ends || !p.whole_scales || after % PER == 0;
      if (p.whole_scales) {
        if (had || ends) ahead(ends ? 0 : min(c / PER * PER + PER, steps - 1));
      } else {
        ahead(after);
      }
      float fs[2 * GPC], fz[2 * GPC];
      {
        uint32_t w[4] = {sc.x, sc.y, sc.z, sc.w}, y[4] = {ze.x, ze.y, ze.z, ze.w};
        if (GPC == 1) {
          w[0] = place_in == 0 ? w[0] : place_in == 1 ? w[1] : place_in == 2 ? w[2] : w[3];
          y[0] = place_in == 0 ? y[0] : place_in == 1 ? y[1] : place_in == 2 ? y[2] : y[3];
        } else if (GPC == 2 && place_in == 1) {
          w[0] = w[2];
          w[1] = w[3];
          y[0] = y[2];
          y[1] = y[3];
        }
        T v[2 * GPC], u[2 * GPC];
        memcpy(v, w, sizeof(v));
        memcpy(u, y, sizeof(u));
#pragma unroll
        for (int q = 0; q < 2 * GPC; ++q) {
          fs[q] = Piece<T>::one(v[q]);
          fz[q] = ZEROS ? 8.f - Piece<T>::one(u[q]) : 0.f;
        }
      }
      const int x0 = 2 * i % SX, place0 = 2 * i % DP;        // (of the first half; the second's come after them)
      const uint32_t full = bars + B_DFULL + 8 * place0, turn = 2 * i / DP & 1, xfull = bars + B_XFULL + 8 * x0;
      if (!wt_wait_warp(dead, p, full, turn, full + 8, turn, WHERE_EPILOGUE)) break;
      if (ZEROS && !wt_wait_warp(dead, p, xfull, 2 * i / SX & 1, xfull + 8, 2 * i / SX & 1, WHERE_EPILOGUE)) break;   // (there already)
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int q = 0; q < GPC; ++q) {
          const uint64_t s = two(fs[h * GPC + q], fs[h * GPC + q]), z = two(fz[h * GPC + q], fz[h * GPC + q]);
          uint32_t d[TOK];
          const uint32_t from = td + ((place0 + h) * GPC + q) * NT;
          if constexpr (TOK == 32) tc_ld_32x32b_x32(from, d);
          else if constexpr (TOK == 16) tc_ld_32x32b_x16(from, d);
          else tc_ld_32x32b_x8(from, d);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < TOK; ++e) asm volatile("" : "+r"(d[e]));     // no use of them before the wait
          const ulonglong2* sx = reinterpret_cast<const ulonglong2*>(smem + L::XS + (x0 + h) * L::X + NT * 256 + (q * NT + t0) * 4);
#pragma unroll
          for (int e = 0; e < TOK / 2; e += 2) {
            uint64_t lo = two(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1]));
            uint64_t hi = two(__uint_as_float(d[2 * e + 2]), __uint_as_float(d[2 * e + 3]));
            if (ZEROS) {
              const ulonglong2 t = sx[e / 2];
              lo = fma2(z, t.x, lo);
              hi = fma2(z, t.y, hi);
            }
            acc[e] = fma2(s, lo, acc[e]);
            acc[e + 1] = fma2(s, hi, acc[e + 1]);
          }
        }
        if (h == 1) tc_fence_before();
      }
      // The sums' place is free only once every lane has them, not merely asked for them: which lane says so is known from
      // what they were added to (one word of each 8 bytes, however they were loaded).
      int who = 0;
      if (ZEROS) {
        uint64_t all = 0;
#pragma unroll
        for (int e = 0; e < TOK / 2; ++e) all ^= acc[e];
        who = __any_sync(0xffffffffu, static_cast<uint32_t>(all) & 1u) ? 1 : 0;
      }
      __syncwarp();
      if (lane == who) {
        mbar_arrive(bars + B_DEMPTY + 8 * place0);
        mbar_arrive(bars + B_DEMPTY + 8 * place0 + 8);
        mbar_arrive(bars + B_XEMPTY + 8 * x0);
        mbar_arrive(bars + B_XEMPTY + 8 * x0 + 8);
      }
      if (ends || i + 1 == count) {
        // all of a tile, or the run's part of it: that at the run's beginning first, another second
        const int m0 = tile / row_tiles * NT + t0;
        const bool whole = ends && i - first + 1 == p.steps;
        float* out = p.part + ((static_cast<long long>(blockIdx.x) * 2 + (first == 0 ? 0 : 1)) * NT + t0) * WT_ROWS + r;
        char* y = p.w.y + m0 * p.w.y_row + static_cast<long long>(row_now) * (p.w.out_f32 ? 4 : 2);
        const int tokens = row_now < p.w.n ? p.w.m - m0 : 0;
#pragma unroll
        for (int e = 0; e < TOK; ++e) {
          float v[2];
          split(acc[e / 2], v[0], v[1]);
          if (!whole) {
            out[e * WT_ROWS] = v[e & 1];
          } else if (e < tokens) {
            if (p.w.out_f32) *reinterpret_cast<float*>(y) = v[e & 1];
            else *reinterpret_cast<T*>(y) = Piece<T>::of(v[e & 1]);
            y += p.w.y_row;
          }
        }
#pragma unroll
        for (int e = 0; e < TOK / 2; ++e) acc[e] = 0;
        first = i + 1;
      }
      c = ends ? 0 : c + 1;
      tile += ends ? 1 : 0;
    }
  } else if (warp == 16) {
    // ---------------------------------------------------------------- loads of codes (the kernel before leaves them alone)
    if (lane == 0) tma_prefetch_map(&p.codes);
    const int stop = p.inject == 1 && blockIdx.x == 0 ? count - 1 : count;   // (test: the last step never comes)
    int i = 0;
    for (unsigned tile = u0 / steps, c = u0 - tile * steps; i < stop; ++i) {
      const int s = i % SC;
      if (i >= SC && !wt_wait_warp(dead, p, bars + B_CEMPTY + 8 * s, (i / SC - 1) & 1, WHERE_PRODUCER)) break;
      if (elect_one_sync()) {
        mbar_arrive_expect_tx(bars + B_CFULL + 8 * s, L::C);
        tma_load_2d(base + s * L::C, &p.codes, bars + B_CFULL + 8 * s, c * 128, tile % row_tiles * WT_ROWS);
      }
      __syncwarp();
      if (++c == steps) {
        c = 0;
        ++tile;
      }
    }
    // whoever gave up: no copy may land after the CTA has ended
    for (int q = max(0, i - SC); q < i; ++q) wt_drain(p, bars + B_CFULL + 8 * (q % SC), (q / SC) & 1, WHERE_PRODUCER);
    __syncwarp();
  } else if (warp == 17) {
    // ---------------------------------------------------------------- loads of x
    if (lane == 0) tma_prefetch_map(&p.x);
    griddep_wait();
    fence_proxy_async_global();
    int i = 0;
    for (unsigned tile = u0 / steps, c = 2 * (u0 - tile * steps); i < 2 * count; ++i) {
      const int s = i % SX;
      if (i >= SX && !wt_wait_warp(dead, p, bars + B_XEMPTY + 8 * s, (i / SX - 1) & 1, WHERE_PRODUCER)) break;
      if (elect_one_sync()) {
        const uint32_t bar = bars + B_XFULL + 8 * s, at = base + L::XS + s * L::X;
        const int m0 = tile / row_tiles * NT;
        mbar_arrive_expect_tx(bar, L::X_TX);
        tma_load_2d(at, &p.x, bar, c * W4_PIECE, m0);
        tma_load_2d(at + NT * 128, &p.x, bar, c * W4_PIECE + 64, m0);
        if (ZEROS)
#pragma unroll
          for (int q = 0; q < GPC; ++q)
            bulk_g2s(at + NT * 256 + q * NT * 4,
                     p.sums + static_cast<long long>(min(static_cast<int>(c * GPC + q), p.w.groups - 1)) * p.sums_pitch + m0, NT * 4, bar);
      }
      __syncwarp();
      if (++c == 2 * steps) {
        c = 0;
        ++tile;
      }
    }
    for (int q = max(0, i - SX); q < i; ++q) wt_drain(p, bars + B_XFULL + 8 * (q % SX), (q / SX) & 1, WHERE_PRODUCER);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- products of a half
    const int h = warp - 18;
    int i = 0;
    for (; i < count; ++i) {
      const int j = 2 * i + h, s = j % SX, place = h + 2 * (i % AP), to = j % DP;
      const uint32_t xfull = bars + B_XFULL + 8 * s, afull = bars + B_AFULL + 8 * place;
      const uint32_t xp = (j / SX) & 1, ap = (i / AP) & 1;
      // (a place's first use waits for the phase before the first, which has ended)
      if (!wt_wait_warp(dead, p, xfull, xp, afull, ap, bars + B_DEMPTY + 8 * to, (j / DP + 1) & 1, WHERE_MMA)) break;
      tc_fence_after();
      if (elect_one_sync()) {                                // (the same lane every time)
        const uint64_t b = sdesc_sw128(base + L::XS + s * L::X, 16u, 1024u);
        const uint32_t a = tmem + L::A + place * 64, d = tmem + L::D + to * (GPC * NT);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          constexpr int PER = 8 / GPC;                       // products of a group
          tc_mma_bf16_ts(d + ks / PER * NT, a + 8 * ks, b + ((ks / 4 * (NT * 128) + ks % 4 * 32) >> 4), IDESC, ks % PER != 0);
        }
        tc_commit(bars + B_AEMPTY + 8 * place);
        tc_commit(bars + B_DFULL + 8 * to);
      }
      __syncwarp();
    }
    // nothing may run on when the tensor memory is freed
    for (int j = max(h, 2 * i + h - DP); j < 2 * i + h; j += 2) wt_drain(p, bars + B_DFULL + 8 * (j % DP), j / DP & 1, WHERE_MMA);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A block has 8 tokens of a row tile that several CTAs had parts of, a thread 4.
template <class T>
__global__ void __launch_bounds__(256) w4_join_kernel(const __grid_constant__ TileParams p) {
  __shared__ int sh[3];                                      // the first and last CTA; whether the first starts with the tile
  const int tile = blockIdx.x, r = threadIdx.x & 127, m0 = tile / p.row_tiles * p.NT;
  if (threadIdx.x == 0) {
    const unsigned lo = static_cast<unsigned>(tile) * p.steps, hi = lo + p.steps;
    // the CTA that has step lo: start(b) <= lo < start(b + 1)
    int b = static_cast<int>(min(lo / p.each, static_cast<unsigned>(p.ctas - 1)));
    while (start_of(p, b) > lo) --b;
    int last = b;
    while (last + 1 < p.ctas && start_of(p, last + 1) < hi) ++last;
    sh[0] = b;
    sh[1] = last;
    sh[2] = start_of(p, b) == lo;
  }
  __syncthreads();
  const int b = sh[0], last = sh[1], starts = sh[2];
  const int row = tile % p.row_tiles * WT_ROWS + r, e0 = blockIdx.y * 8 + (threadIdx.x >> 7) * 4;
  griddep_wait();
  if (b == last) return;                                     // one CTA had all of it, and wrote it
  // a CTA's place is the first part of its run, or the last
  auto part = [&](int c, int e) { return p.part[((static_cast<long long>(c) * 2 + (c > b || starts ? 0 : 1)) * p.NT + e) * WT_ROWS + r]; };
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int c = b; c <= last; c += 4) {
    float f[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 4; ++e) f[q][e] = c + q <= last ? part(c + q, e0 + e) : 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += f[0][e] + f[1][e] + f[2][e] + f[3][e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (m0 + e0 + e < p.w.m && row < p.w.n) w4_store<T>(p.w, m0 + e0 + e, row, v[e]);
}

// ------------------------------------------------------------------ host

struct Plan {
  int NT, ctas, steps, row_tiles, tok_tiles, sums_pitch;
  size_t ordered, sums, part, total;   // offsets in the scratch, and its bytes
};
Plan plan_tiles(const W4Params& p, int group) {
  Plan l;
  const int most = group == 32 ? 32 : 64;
  l.NT = p.m <= 16 ? 16 : p.m <= 32 || most == 32 ? 32 : 64;
  l.steps = (p.k + WT_STEP - 1) / WT_STEP;
  l.row_tiles = (p.n + WT_ROWS - 1) / WT_ROWS;
  l.tok_tiles = (p.m + l.NT - 1) / l.NT;
  l.ctas = static_cast<int>(std::min<long long>(WT_MAX_CTAS, static_cast<long long>(l.steps) * l.row_tiles * l.tok_tiles));
  l.sums_pitch = l.tok_tiles * l.NT;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  l.ordered = 0;
  l.sums = up(static_cast<size_t>(p.m) * p.k * 2);
  l.part = l.sums + up(p.zeros ? static_cast<size_t>(p.groups) * l.sums_pitch * 4 : 0);
  l.total = l.part + static_cast<size_t>(l.ctas) * 2 * l.NT * WT_ROWS * 4;
  return l;
}

template <class T, int NT, int GPC, bool ZEROS>
cudaError_t launch_products(const TileParams& p, cudaStream_t s) {
  using L = Tile<NT, GPC, ZEROS>;
  auto k = mk_w4_tiles_kernel<T, NT, GPC, ZEROS>;
  static std::atomic<unsigned> done{0};
  const cudaError_t e = allow_smem(k, L::SMEM, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.ctas));
  cfg.blockDim = dim3(WT_THREADS);
  cfg.dynamicSmemBytes = L::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}
template <class T, int NT, int GPC>
cudaError_t launch_products(const TileParams& p, cudaStream_t s) {
  return p.w.zeros ? launch_products<T, NT, GPC, true>(p, s) : launch_products<T, NT, GPC, false>(p, s);
}
template <class T>
cudaError_t launch_products(const TileParams& p, int group, cudaStream_t s) {
  if (group == 32) return p.NT == 16 ? launch_products<T, 16, 4>(p, s) : launch_products<T, 32, 4>(p, s);
  if (group == 64)
    return p.NT == 16 ? launch_products<T, 16, 2>(p, s) : p.NT == 32 ? launch_products<T, 32, 2>(p, s) : launch_products<T, 64, 2>(p, s);
  return p.NT == 16 ? launch_products<T, 16, 1>(p, s) : p.NT == 32 ? launch_products<T, 32, 1>(p, s) : launch_products<T, 64, 1>(p, s);
}

template <class T>
cudaError_t launch_all(const TileParams& p, int group, cudaStream_t s) {
  w4_order_kernel<T><<<dim3((p.w.k + 2047) / 2048, std::min(p.w.m, 65535)), 256, 0, s>>>(p, group);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_products<T>(p, group, s);
  // tiles that no CTA has whole: unless every run is a number of tiles
  const long long tiles = static_cast<long long>(p.row_tiles) * p.tok_tiles;
  if (e != cudaSuccess || tiles % p.ctas == 0) return e;
  return launch_dependent(w4_join_kernel<T>, dim3(static_cast<unsigned>(tiles), p.NT / 8), dim3(256), s, p);
}

}  // namespace

size_t w4_tiles_scratch(const W4Params& p, int group) { return plan_tiles(p, group).total; }

mk_status launch_w4_tiles(const W4Params& w, mk_dtype dtype, int group, void* scratch, uint32_t* hdr, const mk_config* cfg,
                          cudaStream_t s) {
  TileParams p;
  std::memset(&p, 0, sizeof(p));
  const Plan l = plan_tiles(w, group);
  p.w = w;
  p.hdr = hdr;
  uint8_t* at = static_cast<uint8_t*>(scratch);
  p.ordered = at;
  p.sums = w.zeros ? reinterpret_cast<float*>(at + l.sums) : nullptr;
  p.part = reinterpret_cast<float*>(at + l.part);
  p.sums_pitch = l.sums_pitch;
  p.ctas = l.ctas;
  if (cfg && cfg->max_ctas > 0) p.ctas = std::min(p.ctas, cfg->max_ctas);
  p.steps = l.steps;
  p.row_tiles = l.row_tiles;
  p.tok_tiles = l.tok_tiles;
  const unsigned all = static_cast<unsigned>(l.steps) * l.row_tiles * l.tok_tiles;
  p.each = all / p.ctas;
  p.over = all % p.ctas;
  p.NT = l.NT;
  p.whole_scales = w.groups % 8 == 0 && !((reinterpret_cast<uintptr_t>(w.scales) | reinterpret_cast<uintptr_t>(w.zeros)) & 15u);
  p.wait_ns = default_wait_ns(cfg);
  p.inject = cfg ? cfg->inject : 0;
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(w.k / 2), static_cast<cuuint64_t>(w.n)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(w.k / 2)};
    const cuuint32_t box[2] = {128, WT_ROWS}, steps[2] = {1, 1};
    if (!encode_map(&p.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(w.codes), dims, strides, box, steps,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return MK_ERR_CUDA;
  }
  {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(w.k), static_cast<cuuint64_t>(w.m)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(w.k) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(l.NT)}, steps[2] = {1, 1};
    if (!encode_map(&p.x, dtype == MK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                    const_cast<uint8_t*>(p.ordered), dims, strides, box, steps, CU_TENSOR_MAP_SWIZZLE_128B))
      return MK_ERR_CUDA;
  }
  const cudaError_t e = dtype == MK_BF16 ? launch_all<__nv_bfloat16>(p, group, s) : launch_all<__half>(p, group, s);
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

}  // namespace mk
