// mk_paged.cu -- attention over a paged cache for sequences with few new
// tokens (decode steps), the join of partial results, and the entry point.
//
// Per (sequence, key head) the query rows are the new tokens times the query
// heads that share the key head, in groups of 16.  A decode step reads each
// visible key and value once and does 4 x 16 multiply-adds a value at most, so
// it is bound by HBM; everything here serves an even, deep stream of loads:
//   * the (sequence, head, row group, key tile) list of the whole batch is
//     cut into equal runs, one for each CTA (one CTA per SM), whatever the
//     lengths: every CTA finds its run from the lengths, so the host needs none
//     of them and a call can be captured into a graph;
//   * one warp issues a TMA load per page and 128 bytes of row into a ring of
//     32- or 64-key stages (192 KB; 128 KB with two column groups), so a page's end inside a tile
//     costs nothing;
//   * twelve warps take the tiles in turn, each with its own running maximum, sum and accumulator.
//     They compute the transposes, S^T = K Q^T and O^T += V^T P^T (mma.sync m16n8k16): keys and
//     elements fill the 16 rows of the instruction and the 8 query rows its 8 columns, so with
//     groups of up to 8 heads nothing is wasted (query rows as the 16 rows take twice the MMAs and
//     registers; a 128-row tcgen05 tile would be 15/16 empty).  More than 8 packed rows: two
//     column groups share the operands of K and V, on eight warps;
//   * the warps' results are joined in shared memory at the end of a run's part of a unit;
//   * units cut by a run's end leave normalised fp32 partial rows with their
//     log2 sums; the last of their CTAs to be done joins them, in the order of
//     the runs, so the result does not depend on which one it is.  (A second,
//     programmatically dependent launch for that took 3 to 5 us more a call.)
// 128 sequences of 100 to 32000 tokens, 64 query heads on 8, d = 128, e4m3: 714 us, 5.9 TB/s (86 %
// of a plain copy's rate).  48 windows of 4096 tokens, 8 heads, d = 64, fp16: 85.5 us, 4.6 TB/s.  One sequence of
// 2000 tokens: 12.7 us in a graph, all of it latency: lengths, page ids, loads, and the join.
// 8-bit caches: codes become fp16, exactly (the fp8 form of mma.sync does the same conversions
// inside, with more instructions); the query row is scaled by a power of two to fit fp16 (bf16 has
// fewer bits), the key scale multiplies the scores, the value scale the weights, and those
// products have a running maximum of their own: a small weight of a page with a large scale keeps
// its bits.  With two column groups, d = 128, what a lane holds does not fit its 168 registers
// (276 bytes of spills): 16 packed rows take 182 us below, where the bytes alone are 77.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "mk_paged.h"

namespace mk {

__device__ __noinline__ bool pg_wait_loop(volatile int* dead, const PagedParams& p, uint32_t bar, uint32_t parity,
                                          int where) {
  return pg_wait_slow(dead, p, bar, parity, where);
}

namespace {

constexpr int DC_MAX_ROWS = 16;        // packed query rows of a unit, at most
constexpr int DC_BATCH = 1024;         // sequences of one launch (the entry point slices larger batches)
constexpr int DC_JOIN = 256;           // threads that join a segment
constexpr int DC_ROUND = 4;            // warps whose rows are in the join buffer at a time

// NQ: groups of 8 query rows of a unit.
template <class T, bool E8, int D, int NQ>
struct Shape {
  static constexpr int KT = !E8 && D == 128 ? 32 : 64;                // keys of a tile: 16 KB (8-bit, d = 64: 8 KB)
  static constexpr int ROWS = 8 * NQ;
  static constexpr int WARPS = NQ == 1 ? 12 : 8;                      // consumer warps; one more loads
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int TILE = KT * D * (E8 ? 1 : 2);
  static constexpr int STAGE = 2 * TILE;
  static constexpr int PITCH = D + 4;                                 // floats of a row in the join buffer
  static constexpr int MERGE = DC_ROUND * ROWS * PITCH * 4;
  static constexpr int ML = WARPS * ROWS * 3 * 4;                     // maximum, sum, value factor
  static constexpr int PREFIX = (DC_BATCH + 1) * 8;
  static constexpr int FIXED = 1024 + MERGE + ML + ((PREFIX + 15) & ~15) + 512;
  // 32 keys a tile for 16-bit d = 128, so that the ring has a stage for each warp.
  // A warp's tiles come WARPS apart.  With a multiple of that many stages the fill before the one
  // it waits for was its own, so the barrier's phase parity cannot be mistaken.
  static constexpr int STAGES = std::min((232448 - FIXED) / STAGE, 24) / WARPS * WARPS;
  static constexpr int SMEM = FIXED + STAGES * STAGE;
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool half) {
  if (half)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t two) {   // two codes -> two fp16, exactly
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
// An 8 x 8 matrix of 16-bit values turned: rows in lanes / 4, two neighbours of a row in a lane.
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// x, or 3e38 where that is less; NaN stays NaN.  (A scale over the reference of weight times scale is past fp32's range
// where weights below 2^-118 stand beside it: their product is ordinary, so the factor must not be infinite.)
__device__ __forceinline__ float at_most_large(float x) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(3e38f));
  return y;
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) { return Piece<__half>::pack(a, b); }
// Byte offset of 16-byte piece ch of key row `key` in a tile: rows of 128 bytes
// (16-bit types: d / 64 such atoms, one after the other) or of 64 bytes, with
// the swizzle the TMA load applied.
template <int KT, bool E8, int D>
__device__ __forceinline__ uint32_t piece_at(int key, int ch) {
  if (E8 && D == 64) return key * 64 + ((ch ^ ((key >> 1) & 3)) << 4);
  return (ch >> 3) * (KT * 128) + key * 128 + (((ch & 7) ^ (key & 7)) << 4);
}

// Sets what is not finite in 16 bytes of a row to 0; whether there was any.
template <class T, bool E8>
__device__ __forceinline__ bool clear_not_finite(uint32_t (&w)[4]) {
  bool any = false;
  constexpr uint32_t BITS = E8 ? 8 : 16;
  constexpr uint32_t MASK = E8 ? 0x7fu : (std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (uint32_t b = 0; b < 32; b += BITS)
      if (((w[i] >> b) & MASK) == MASK) {
        w[i] &= ~(((1u << BITS) - 1u) << b);
        any = true;
      }
  return any;
}
// Part of a run: tiles k0 .. k1-1 of one unit (sequence b, head h, rows 16 rg ..).
struct Segment {
  int b, h, rg, n, len, row0;          // new tokens, tokens in all, first token row
  int k0, k1, count;
  KeyTiles t;
  long long u0;                        // number of the unit's first tile
};
template <int KT, int ROWS>
__device__ __forceinline__ Segment segment_at(const PagedParams& p, const long long* pre, int b, long long x,
                                              long long end) {
  Segment g;
  g.b = b;
  sequence_of(p, b, g.n, g.len, g.row0);
  g.t = key_tiles<KT>(p, g.len - g.n, g.len - 1, g.len);
  g.count = g.t.count();
  const int groups = (g.n * p.group + ROWS - 1) / ROWS;
  const long long rem = x - pre[b] * p.c.heads;
  const int unit = static_cast<int>(rem / g.count);
  g.k0 = static_cast<int>(rem - static_cast<long long>(unit) * g.count);
  g.u0 = x - g.k0;
  g.k1 = static_cast<int>(min(static_cast<long long>(g.count), g.k0 + (end - x)));
  g.h = unit / groups;
  g.rg = unit - g.h * groups;
  return g;
}

// Tiles of sequence b for one head, all its row groups; 0 for sequences of the other launch.
template <int KT, int ROWS>
__device__ __forceinline__ long long sequence_tiles(const PagedParams& p, int b) {
  int n, len, row0;
  if (!sequence_of(p, b, n, len, row0)) return 0;
  if (!rows_are_ours(p, n)) return 0;
  const long long rows = static_cast<long long>(n) * p.group;
  return ((rows + ROWS - 1) / ROWS) * key_tiles<KT>(p, len - n, len - 1, len).count();
}

// Returns the number of tiles that it has begun to load.
template <int KT, bool E8, int D, int NQ>
__device__ uint32_t dc_producer(const PagedParams& p, const long long* pre, volatile int* dead, uint32_t full, uint32_t empty,
                            uint32_t ring, int stages, long long x, long long end) {
  constexpr int TILE = KT * D * (E8 ? 1 : 2), ROWS = 8 * NQ;
  const int lane = threadIdx.x & 31;
  const int box = min(p.c.page_size, KT), boxes = KT / box;
  int b = warp_last_le(p.s.batch, 0, [&](int i) { return pre[i] * p.c.heads <= x ? 0 : 1; });
  int st = 0;
  uint32_t ph = 0, loads = 0;
  const uint32_t stop = stop_at(p);
  while (x < end) {
    while (pre[b + 1] * p.c.heads <= x) ++b;
    const Segment g = segment_at<KT, ROWS>(p, pre, b, x, end);
    const int n_pages = min(p.s.max_pages, ((g.len - 1) >> p.c.page_log2) + 1);
    const int* table = p.s.pages + g.b * p.s.pages_stride;
    // The pages of 32 boxes at a time, a lane each, the next 32 on their way meanwhile (a look-up for
    // every tile held the loads up for 700 cycles a tile): lane i has box i % boxes of tile
    // k + i / boxes; the maps' first absent page where there is none.
    auto pages_of = [&](int k) {
      k += lane / boxes;
      if (k >= g.k1) return p.map_pages;
      const int key = g.t.tile(k) * KT + (lane % boxes) * box, lp = key >> p.c.page_log2;
      if (lp >= n_pages) return p.map_pages;
      const int id = table[lp];
      if (id >= 0 && id < p.c.n_pages) return id;
      if (keys_seen(p, g.len - g.n, g.len - 1, g.len, key, box)) seq_error(p.hdr, MK_ERR_INVALID, WHERE_PRODUCER, g.b);
      return p.map_pages;
    };
    const int batch = 32 / boxes;
    int pages = 0, next = pages_of(g.k0);
    for (int k = g.k0, at = batch; k < g.k1; ++k, ++at) {
      if (at == batch) {
        at = 0;
        pages = next;
        if (k + batch < g.k1) next = pages_of(k + batch);
      }
      const int page = __shfl_sync(0xffffffffu, pages, at * boxes + (lane % boxes));
      if (!__all_sync(0xffffffffu, pg_wait(dead, p, empty + 8u * st, ph ^ 1u, WHERE_PRODUCER))) return loads;
      if (loads == stop) return loads;
      const uint32_t bar = full + 8u * st;
      if (lane == 0) mbar_arrive_expect_tx(bar, 2u * TILE);
      __syncwarp();
      // lanes below 16 load K, the others V
      if ((lane & 15) < boxes) {
        const int slot = (g.t.tile(k) * KT + (lane & 15) * box) & (p.c.page_size - 1);
        constexpr int ATOMS = E8 ? 1 : D / 64;
        constexpr uint32_t ROW = E8 ? D : 128;
        const uint32_t dst = ring + static_cast<uint32_t>(st) * 2u * TILE + (lane >> 4) * TILE + (lane & 15) * box * ROW;
#pragma unroll
        for (int a = 0; a < ATOMS; ++a)
          tma_load_4d(dst + a * (KT * 128u), lane < 16 ? &p.tmK : &p.tmV, bar, 64 * a, slot, g.h, page);
      }
      ++loads;
      if (++st == stages) {
        st = 0;
        ph ^= 1u;
      }
    }
    x += g.k1 - g.k0;
  }
  return loads;
}

// The first tile of a segment that is a warp's: the run's tiles are dealt to the warps in turn.
template <int WARPS>
__device__ __forceinline__ int first_tile(int warp, uint32_t done) {
  const int skip = static_cast<int>(done % WARPS);
  return warp >= skip ? warp - skip : warp - skip + WARPS;
}

// A consumer warp's part of a segment: what it needs, and where its result goes.
struct Work {
  volatile int* dead;
  uint32_t ring, full, empty;
  uint32_t done;                       // tiles of the run before this segment
  int first;                           // this warp's first tile of it
  float* merge;                        // the join buffer, and maximum, sum and value factor of
  float* ml;                           // every warp's rows
  const Deal& deal;
  volatile int* share;                 // the CTAs whose partial rows are this one's to join
};

// In a tile that not every row sees whole: 0 * NaN is NaN, so values no row sees (past the end,
// before the window) may hold anything and are cleared, and of those only some rows see (several
// new tokens) what is not finite is cleared; returns whether there was any of the latter, with the
// keys as bits.
template <class T, bool E8, int D, int KT>
__device__ __forceinline__ bool clear_values(const PagedParams& p, const Segment& g, uint32_t vt, int key0,
                                             uint32_t (&odd)[2]) {
  constexpr int CH = D * (E8 ? 1 : 2) / 16;
  const int lane = threadIdx.x & 31, p0 = g.len - g.n, p1 = g.len - 1;
  odd[0] = odd[1] = 0u;
  for (int e = lane; e < KT * CH; e += 32) {
    const int key = e / CH;
    const uint32_t at = vt + piece_at<KT, E8, D>(key, e - key * CH);
    if (!key_seen_by_any(p, p0, p1, g.len, key0 + key)) {
      sts128(at, make_uint4(0u, 0u, 0u, 0u));
    } else if (!all_seen(p, p0, p1, g.len, key0 + key, 1)) {
      uint32_t w[4];
      lds128(at, w);
      if (clear_not_finite<T, E8>(w)) {
        sts128(at, make_uint4(w[0], w[1], w[2], w[3]));
        odd[key >> 5] |= 1u << (key & 31);
      }
    }
  }
  odd[0] = __reduce_or_sync(0xffffffffu, odd[0]);
  odd[1] = __reduce_or_sync(0xffffffffu, odd[1]);
  __syncwarp();
  return (odd[0] | odd[1]) != 0u;
}

// A consumer warp's share of a segment, and of its end.
template <class T, bool E8, int D, int NQ>
__device__ __forceinline__ void consume(const PagedParams& p, const Segment& g, const Work& wk) {
  using S = Shape<T, E8, D, NQ>;
  constexpr bool HALF = E8 || !std::is_same<T, __nv_bfloat16>::value;   // fp16 operands of the products
  constexpr float SHIFT = HALF ? 10.f : 0.f;   // fp16 weights are taken 2^10 high: small ones keep their bits
  constexpr int KT = S::KT, KS = D / 16, MT = KT / 16, OT = D / 16;
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int p0 = g.len - g.n, p1 = g.len - 1, tiles = g.k1 - g.k0;
  // per column of S^T and O^T that this lane holds: query rows 8 q + 2 c and + 1
  float m[NQ][2], l[NQ][2];            // maximum and sum of the weights
  float mv[NQ][2];                     // 8-bit: log2 of the largest weight times value scale, next to m: O's reference
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[q][e] = mv[q][e] = -INFINITY;
      l[q][e] = 0.f;
    }
  float o[NQ][OT][4];
#pragma unroll
  for (int q = 0; q < NQ; ++q)
#pragma unroll
    for (int j = 0; j < OT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[q][j][e] = 0.f;
  if (wk.first < tiles) {
    // query rows 8 q + r as operand registers
    uint32_t qf[NQ][KS][2];
    int pos[NQ][2];
    float row_scale[NQ][2];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int row = g.rg * S::ROWS + 8 * q + r;
      const int tok = row / p.group, head = g.h * p.group + row - tok * p.group;
      const bool ok = tok < g.n;
      const T* src = static_cast<const T*>(p.q) + static_cast<long long>(g.row0 + (ok ? tok : 0)) * p.qs_t +
                     (ok ? head : 0) * p.qs_h;
      const int my_pos = p0 + (ok ? tok : 0);
      float my_scale = p.scale_log2;
      if (!E8) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qf[q][ks][e] = ok ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * c + 8 * e) : 0u;
      } else {
        // 16 neighbouring elements of every 64: the order in which the codes are read
        float f[D / 4], top = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            float v[8];
            const uint4 raw = ok ? *reinterpret_cast<const uint4*>(src + 64 * j + 16 * c + 8 * w)
                                 : make_uint4(0u, 0u, 0u, 0u);
            Piece<T>::get(raw, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              f[16 * j + 8 * w + e] = v[e];
              top = fmaxf(top, fabsf(v[e]));
            }
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // a power of two that brings the row's largest magnitude to 2^10 .. 2^11
        const int ex = min(max(static_cast<int>((__float_as_uint(top) >> 23) & 255) - 127, -100), 126);
        const float up = __uint_as_float(static_cast<uint32_t>(10 - ex + 127) << 23);
        my_scale *= __uint_as_float(static_cast<uint32_t>(ex - 10 + 127) << 23);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qf[q][ks][e] = f16x2(f[4 * ks + 2 * e] * up, f[4 * ks + 2 * e + 1] * up);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        pos[q][e] = __shfl_sync(0xffffffffu, my_pos, 4 * (2 * c + e));
        row_scale[q][e] = __shfl_sync(0xffffffffu, my_scale, 4 * (2 * c + e));
      }
    }
    // 8-bit: lane j < KT / 8 holds the scales of keys 8 j .. 8 j + 7 of a tile
    const int* table = p.s.pages + g.b * p.s.pages_stride;
    const int n_pages = min(p.s.max_pages, (p1 >> p.c.page_log2) + 1);
    auto id_of = [&](int k) {          // -1 for keys no row sees: their scales may be anything
      const int key = g.t.tile(k) * KT + 8 * (lane & (KT / 8 - 1)), lp = key >> p.c.page_log2;
      if (lp >= n_pages || !keys_seen(p, p0, p1, g.len, key, 8)) return -1;
      const int id = table[lp];
      return id < p.c.n_pages ? id : -1;
    };
    float ks_next = 0.f, vs_next = 0.f;
    auto scales_of = [&](int id) {
      const long long at = static_cast<long long>(id) * p.c.heads + g.h;
      ks_next = id >= 0 ? p.c.k_scale[at] : 0.f;
      vs_next = id >= 0 ? p.c.v_scale[at] : 0.f;
    };
    if (E8) scales_of(id_of(g.k0 + wk.first));
    for (int k = wk.first; k < tiles; k += S::WARPS) {
      const uint32_t i = wk.done + k;
      const int st = i % S::STAGES;
      const uint32_t kt = wk.ring + st * S::STAGE, vt = kt + S::TILE;
      int next_id = -1;
      if (E8 && k + S::WARPS < tiles) next_id = id_of(g.k0 + k + S::WARPS);
      const float ks_tile = ks_next, vs_tile = vs_next;
      const int there = pg_wait(wk.dead, p, wk.full + 8u * st, (i / S::STAGES) & 1u, WHERE_MMA) ? 1 : 0;
      if (!__all_sync(0xffffffffu, there)) break;
      const int key0 = g.t.tile(g.k0 + k) * KT;
      const bool masked = !all_seen(p, p0, p1, g.len, key0, KT);
      // ---- S^T = K Q^T: rows of 16-key group t are its keys, in order (16-bit) or permuted so that
      // neighbouring lanes read different banks (8-bit: row x is key (x >> 1 & 3) | (x & 1) << 2 | x & 8)
      float s[NQ][MT][4];
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[q][t][e] = 0.f;
      const int perm = E8 ? (r >> 1) | ((r & 1) << 2) : r;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (!E8) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t f[4];
            ldsm4(kt + piece_at<KT, E8, D>(16 * t + (lane & 15), 2 * ks + (lane >> 4)), f);
#pragma unroll
            for (int q = 0; q < NQ; ++q) mma16816(s[q][t], f, qf[q][ks][0], qf[q][ks][1], HALF);
          }
        } else {
#pragma unroll
          for (int a = 0; a < D / 64; ++a) {
            uint32_t f[2][4];
            lds128(kt + piece_at<KT, E8, D>(16 * t + perm, 4 * a + c), f[0]);
            lds128(kt + piece_at<KT, E8, D>(16 * t + 8 + perm, 4 * a + c), f[1]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t x[4] = {e4m3_f16x2(f[0][w] & 0xffffu), e4m3_f16x2(f[1][w] & 0xffffu),
                                     e4m3_f16x2(f[0][w] >> 16), e4m3_f16x2(f[1][w] >> 16)};
#pragma unroll
              for (int q = 0; q < NQ; ++q) mma16816(s[q][t], x, qf[q][4 * a + w][0], qf[q][4 * a + w][1], HALF);
            }
          }
        }
      }
      if (E8) scales_of(next_id);
      // ---- softmax of columns 2 c + e over keys 16 t + perm + 8 h
      float ks[2 * MT], lv[2 * MT], vs[2 * MT];
      if (E8) {
        const float lv_tile = log2f(vs_tile);
#pragma unroll
        for (int x = 0; x < 2 * MT; ++x) {
          ks[x] = __shfl_sync(0xffffffffu, ks_tile, x);
          vs[x] = __shfl_sync(0xffffffffu, vs_tile, x);
          lv[x] = __shfl_sync(0xffffffffu, lv_tile, x);
        }
      }
      uint32_t pf[NQ][MT][2];
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        // Scores are rounded products before the maximum is taken off, so that the largest weight is 1 however
        // far from 0 they are (one fma would leave in the rounding of the maximum: 64 at 2^31).
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int e = x & 1, h = x >> 1;
            s[q][t][x] = __fmul_rn(s[q][t][x], E8 ? row_scale[q][e] * ks[2 * t + h] : p.scale_log2);
            if (masked && !key_seen(p, pos[q][e], g.len, key0 + 16 * t + perm + 8 * h)) s[q][t][x] = -INFINITY;
            top[e] = fmaxf(top[e], s[q][t][x]);
          }
        float mref[2], alpha[2], rel[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int y = 4; y < 32; y <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], y));
          const float mn = fmaxf(m[q][e], top[e]);
          mref[e] = mn == -INFINITY ? 0.f : mn;
          const float down = m[q][e] - mref[e];
          alpha[e] = pg_ex2(down);
          m[q][e] = mn;
          l[q][e] *= alpha[e];
          if (E8) mv[q][e] += down;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[q][t][x] = __fsub_rn(s[q][t][x], mref[x & 1]);
        if (E8) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top_v = -INFINITY;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
              for (int h = 0; h < 2; ++h) top_v = fmaxf(top_v, s[q][t][2 * h + e] + lv[2 * t + h]);
#pragma unroll
            for (int y = 4; y < 32; y <<= 1) top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, y));
            const float mvn = fmaxf(mv[q][e], top_v), vref = mvn == -INFINITY ? 0.f : mvn;
            alpha[e] = pg_ex2(mv[q][e] - vref);
            mv[q][e] = mvn;
            rel[e] = mvn == -INFINITY ? 0.f : at_most_large(pg_ex2(-vref));
          }
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int j = 0; j < OT; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[q][j][x] *= alpha[x & 1];
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          float w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int e = x & 1;
            w[x] = pg_ex2(HALF ? s[q][t][x] + SHIFT : s[q][t][x]);
            l[q][e] += w[x];
            if (E8) w[x] = w[x] == 0.f ? 0.f : w[x] * at_most_large(vs[2 * t + (x >> 1)] * rel[e]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
            pf[q][t][h] = turn8x8(HALF ? f16x2(w[2 * h], w[2 * h + 1]) : pack_bf16x2(w[2 * h], w[2 * h + 1]));
        }
      }
      if (masked) {
        uint32_t odd[2];
        if (clear_values<T, E8, D, KT>(p, g, vt, key0, odd))
          for (int key = 0; key < KT; ++key) {     // the rows that see what was cleared get it here
            if (!((odd[key >> 5] >> (key & 31)) & 1u)) continue;
            int page;
            const long long row = value_row(p, g.b, g.h, key0 + key, page);
            if (row < 0) continue;
#pragma unroll
            for (int j = 0; j < OT; ++j)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const int el = E8 ? (D / 8) * r + 2 * j + (x >> 1) : 16 * j + r + 8 * (x >> 1);
                const float v = not_finite<T, E8>(p.c.v, row + el);
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                  if (v != 0.f && key_seen(p, pos[q][x & 1], g.len, key0 + key)) o[q][j][x] += v;
              }
          }
      }
      // ---- O^T += V^T P^T: row x of 16-element group j is element 16 j + x (16-bit) or, 8-bit, element
      // (D / 8) (x % 8) + 2 j + x / 8: lane (r, c) reads keys c, c+4, c+8, c+12 of 16, D / 8 codes each
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        if (!E8) {
#pragma unroll
          for (int j = 0; j < OT; ++j) {
            uint32_t f[4];
            ldsm4_t(vt + piece_at<KT, E8, D>(16 * t + (lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1)), f);
#pragma unroll
            for (int q = 0; q < NQ; ++q) mma16816(o[q][j], f, pf[q][t][0], pf[q][t][1], HALF);
          }
        } else {
          uint32_t f[4][4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int key = 16 * t + c + 4 * w;
            if (D == 128) {
              lds128(vt + piece_at<KT, E8, D>(key, r), f[w]);
            } else {
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
                           : "=r"(f[w][0]), "=r"(f[w][1])
                           : "r"(vt + piece_at<KT, E8, D>(key, r >> 1) + 8u * (r & 1))
                           : "memory");
            }
          }
#pragma unroll
          for (int w = 0; w < D / 32; ++w) {    // 4 x 4 bytes turned into pairs of keys
            const uint32_t x0 = __byte_perm(f[0][w], f[1][w], 0x5140), x1 = __byte_perm(f[0][w], f[1][w], 0x7362);
            const uint32_t y0 = __byte_perm(f[2][w], f[3][w], 0x5140), y1 = __byte_perm(f[2][w], f[3][w], 0x7362);
            const uint32_t a0[4] = {e4m3_f16x2(x0 & 0xffffu), e4m3_f16x2(x0 >> 16), e4m3_f16x2(y0 & 0xffffu),
                                    e4m3_f16x2(y0 >> 16)};
            const uint32_t a1[4] = {e4m3_f16x2(x1 & 0xffffu), e4m3_f16x2(x1 >> 16), e4m3_f16x2(y1 & 0xffffu),
                                    e4m3_f16x2(y1 >> 16)};
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              mma16816(o[q][2 * w], a0, pf[q][t][0], pf[q][t][1], HALF);
              mma16816(o[q][2 * w + 1], a1, pf[q][t][0], pf[q][t][1], HALF);
            }
          }
        }
      }
      if (masked) fence_proxy_async_smem();   // the cleared rows before the next load of this stage
      // The stage is free only once every lane has its values, not merely asked for them (behind loads from memory that
      // miss, theirs from shared memory may take longer than the next tile does): which lane says so is known from the
      // products' sums.  Those need the keys' values too, for the weights.
      uint32_t all = 0;
#pragma unroll
      for (int j = 0; j < OT; ++j) all ^= __float_as_uint(o[0][j][0]);
      const int who = __any_sync(0xffffffffu, all & 1u) ? 1 : 0;
      __syncwarp();
      if (lane == who) mbar_arrive(wk.empty + 8u * st);
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], y);
  }
  const int warp = threadIdx.x >> 5;
  if (r == 0) {
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* at = wk.ml + (warp * S::ROWS + 8 * q + 2 * c + e) * 3;
        at[0] = m[q][e];
        at[1] = l[q][e];
        at[2] = !E8 ? 1.f : pg_ex2(mv[q][e]);
      }
  }
  auto barrier = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * S::WARPS) : "memory"); };
  barrier();
  // The join: DC_JOIN threads share out the rows, EL neighbouring elements each; a few warps' rows
  // are in the buffer at a time.
  constexpr int PER = DC_JOIN / S::ROWS, EL = D / PER, V = EL < 4 ? EL : 4;
  const bool joins = threadIdx.x < DC_JOIN;
  const int row = joins ? threadIdx.x / PER : 0, d0 = (threadIdx.x % PER) * EL;
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < S::WARPS; ++w) top = fmaxf(top, wk.ml[(w * S::ROWS + row) * 3]);
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) acc[e] = 0.f;
  for (int w0 = 0; w0 < S::WARPS; w0 += DC_ROUND) {
    bool any = false;                          // none of these warps had a tile: nothing to add
#pragma unroll
    for (int w = 0; w < DC_ROUND; ++w) any |= first_tile<S::WARPS>(w0 + w, wk.done) < tiles;
    if (!any) continue;
    if (warp >= w0 && warp < w0 + DC_ROUND) {
      float* mine = wk.merge + (warp - w0) * S::ROWS * S::PITCH;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int j = 0; j < OT; ++j)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mine[(8 * q + 2 * c + (x & 1)) * S::PITCH +
                 (E8 ? (D / 8) * r + 2 * j + (x >> 1) : 16 * j + r + 8 * (x >> 1))] = o[q][j][x];
    }
    barrier();
    if (joins) {
#pragma unroll
      for (int w = 0; w < DC_ROUND; ++w) {
        const float* at = wk.ml + ((w0 + w) * S::ROWS + row) * 3;
        if (at[1] == 0.f) continue;            // no tile, or nothing seen (NaN stays in)
        const float f = pg_ex2(at[0] - ref);
        sum += f * at[1];
        const float fv = f * at[2];
        const float* from = wk.merge + (w * S::ROWS + row) * S::PITCH + d0;
#pragma unroll
        for (int e = 0; e < EL; e += V) {
          float v[V];
          if constexpr (V == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(from + e);
          else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(from + e);
#pragma unroll
          for (int x = 0; x < V; ++x) acc[e + x] += fv * v[x];
        }
      }
    }
    barrier();
  }
  const int prow = g.rg * S::ROWS + row;
  const bool real = joins && prow < g.n * p.group;
  auto store = [&](float total, float from) {    // acc / total, and the sum of exponentials total * 2^from
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int e = 0; e < EL; ++e) acc[e] *= inv;
    const int tok = prow / p.group, head = g.h * p.group + prow - tok * p.group;
    const long long t = g.row0 + tok;
    T* dst = static_cast<T*>(p.out) + t * p.os_t + head * p.os_h + d0;
    if constexpr (EL == 8) {
      *reinterpret_cast<uint4*>(dst) = Piece<T>::put(*reinterpret_cast<const float (*)[8]>(acc));
    } else {
#pragma unroll
      for (int e = 0; e < EL; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) =
            std::is_same<T, __half>::value ? f16x2(acc[e], acc[e + 1]) : pack_bf16x2(acc[e], acc[e + 1]);
    }
    if (p.lse != nullptr && d0 == 0) p.lse[t * p.heads_q + head] = total == 0.f ? -INFINITY : (from + log2f(total)) * LN2;
  };
  if (tiles == g.count) {                      // the whole unit: final
    if (real) store(sum, ref - SHIFT);
    return;
  }
  if (real) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long at = static_cast<long long>(part_slot(blockIdx.x, g.k0 == 0)) * S::ROWS + row;
#pragma unroll
    for (int e = 0; e < EL; e += 2)
      *reinterpret_cast<float2*>(p.part + at * D + d0 + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
    if (d0 == 0) p.part_lse[at] = sum == 0.f ? -INFINITY : ref + log2f(sum) - SHIFT;
  }
  barrier();
  if (threadIdx.x == 0) {                      // every CTA of the unit comes here once, waits run out or not
    const int c0 = wk.deal.owner(g.u0), c1 = wk.deal.owner(g.u0 + g.count - 1);
    __threadfence();
    const bool last = atomicAdd(p.turn + c0, 1u) == static_cast<uint32_t>(c1 - c0);
    if (last) {
      p.turn[c0] = 0u;
      __threadfence();
    }
    wk.share[0] = last ? c0 : -1;
    wk.share[1] = c1;
  }
  barrier();
  const int c0 = wk.share[0], c1 = wk.share[1];
  if (c0 < 0 || !joins) return;
  // The partial rows of CTAs c0 .. c1 in order, weighted by 2^(log2 sum - largest); PER threads a row.
  top = -INFINITY;
  for (int i = c0 + threadIdx.x % PER; i <= c1; i += PER)
    top = fmaxf(top, __ldcg(p.part_lse + static_cast<long long>(part_slot(i, i == c0)) * S::ROWS + row));
#pragma unroll
  for (int y = PER / 2; y > 0; y >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, y));
  const float first = top == -INFINITY ? 0.f : top;
  sum = 0.f;
#pragma unroll
  for (int e = 0; e < EL; ++e) acc[e] = 0.f;
#pragma unroll 8
  for (int i = c0; i <= c1; ++i) {
    const long long at = static_cast<long long>(part_slot(i, i == c0)) * S::ROWS + row;
    const float f = pg_ex2(__ldcg(p.part_lse + at) - first);
    sum += f;
#pragma unroll
    for (int e = 0; e < EL; e += V) {
      float v[V];
      const float* from = p.part + at * D + d0 + e;
      if constexpr (V == 4) *reinterpret_cast<float4*>(v) = __ldcg(reinterpret_cast<const float4*>(from));
      else *reinterpret_cast<float2*>(v) = __ldcg(reinterpret_cast<const float2*>(from));
#pragma unroll
      for (int x = 0; x < V; ++x) acc[e + x] += f * v[x];
    }
  }
  if (real) store(sum, first);
}

template <class T, bool E8, int D, int NQ>
__global__ void __launch_bounds__(Shape<T, E8, D, NQ>::THREADS, 1)
    mk_paged_decode_kernel(const __grid_constant__ PagedParams p) {
  using S = Shape<T, E8, D, NQ>;
  constexpr int KT = S::KT, ROWS = S::ROWS;
  extern __shared__ uint8_t dyn[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  float* merge = reinterpret_cast<float*>(sm + S::STAGES * S::STAGE);
  float* ml = reinterpret_cast<float*>(sm + S::STAGES * S::STAGE + S::MERGE);
  long long* pre = reinterpret_cast<long long*>(sm + S::STAGES * S::STAGE + S::MERGE + S::ML);
  uint8_t* tail = reinterpret_cast<uint8_t*>(pre) + ((S::PREFIX + 15) & ~15);
  volatile int* dead = reinterpret_cast<int*>(tail + 448);
  const uint32_t ring = smem_u32(sm), full = smem_u32(tail), empty = full + 8u * 24u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int batch = p.s.batch;

  griddep_launch_dependents();           // the prompt kernel's plan
  if (threadIdx.x == 0) {
    *dead = 0;
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(full + 8u * i, 1);
      mbar_init(empty + 8u * i, 1);
    }
    fence_mbar_init();
    pre[0] = 0;
    tma_prefetch_map(&p.tmK);
    tma_prefetch_map(&p.tmV);
  }
  for (int b = threadIdx.x; b < batch; b += S::THREADS) pre[b + 1] = sequence_tiles<KT, ROWS>(p, b);
  __syncthreads();
  if (warp == 0) {                       // prefix sums, a run of sequences a lane
    const int per = (batch + 31) / 32, lo = min(batch, lane * per), hi = min(batch, lo + per);
    long long sum = 0;
    for (int b = lo; b < hi; ++b) sum += pre[b + 1];
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    long long acc = incl - sum;
    for (int b = lo; b < hi; ++b) {
      acc += pre[b + 1];
      pre[b + 1] = acc;
    }
  }
  __syncthreads();
  const Deal deal(pre[batch] * p.c.heads, p.grid);
  for (int b = blockIdx.x; b < batch; b += gridDim.x) {   // sequences without a key: nothing is seen
    int n, len, row0;
    if (pre[b + 1] == pre[b] && sequence_of(p, b, n, len, row0) && rows_are_ours(p, n))
      no_keys<T, D>(p, b, row0, n, S::THREADS);
  }
  if (static_cast<int>(blockIdx.x) >= deal.c) return;
  long long x = deal.start(blockIdx.x);
  const long long end = deal.start(blockIdx.x + 1);
  if (warp == S::WARPS) {
    const uint32_t loads = dc_producer<KT, E8, D, NQ>(p, pre, dead, full, empty, ring, S::STAGES, x, end);
    __syncwarp();
    pg_drain(p, full, S::STAGES, loads);
  } else {
    int b = warp_last_le(batch, 0, [&](int i) { return pre[i] * p.c.heads <= x ? 0 : 1; });
    uint32_t done = 0;                   // tiles of the run before this segment
    while (x < end) {
      while (pre[b + 1] * p.c.heads <= x) ++b;
      const Segment g = segment_at<KT, ROWS>(p, pre, b, x, end);
      const Work wk = {dead, ring, full, empty, done, first_tile<S::WARPS>(warp, done), merge, ml, deal, dead + 2};
      consume<T, E8, D, NQ>(p, g, wk);
      done += g.k1 - g.k0;
      x += g.k1 - g.k0;
    }
  }
}

// ------------------------------------------------------------------ host

template <class T, bool E8, int D, int NQ>
cudaError_t launch_decode(const PagedParams& p, cudaStream_t s) {
  using S = Shape<T, E8, D, NQ>;
  static_assert(S::STAGES >= S::WARPS && S::SMEM <= 232448, "a stage for each warp");
  static int configured_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_dev != dev) {
    e = cudaFuncSetAttribute(mk_paged_decode_kernel<T, E8, D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    configured_dev = dev;
  }
  mk_paged_decode_kernel<T, E8, D, NQ><<<p.grid, S::THREADS, S::SMEM, s>>>(p);
  return cudaGetLastError();
}
template <class T, bool E8>
cudaError_t launch_decode(const PagedParams& p, int nq, cudaStream_t s) {
  if (p.c.d == 128) return nq == 1 ? launch_decode<T, E8, 128, 1>(p, s) : launch_decode<T, E8, 128, 2>(p, s);
  return nq == 1 ? launch_decode<T, E8, 64, 1>(p, s) : launch_decode<T, E8, 64, 2>(p, s);
}

// K / V as [d, slots, heads, pages]; a box is the part of a page that falls into a tile of `tile` keys.
bool cache_map(CUtensorMap* m, const mk_kv_cache* c, const void* base, const void* spare, int tile, bool swizzle) {
  const int esz = c->dtype == MK_E4M3 ? 1 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->heads),
                              static_cast<cuuint64_t>(std::max(1LL, c->n_pages))};
  // the stride of a dimension of one element may be 0 (view_of), but the map wants it positive
  const cuuint64_t row = static_cast<cuuint64_t>(c->d) * esz;
  const cuuint64_t strides[3] = {c->slot_stride > 0 ? static_cast<cuuint64_t>(c->slot_stride) * esz : row,
                                 c->head_stride > 0 ? static_cast<cuuint64_t>(c->head_stride) * esz : row,
                                 c->page_stride > 0 ? static_cast<cuuint64_t>(c->page_stride) * esz : row};
  const cuuint32_t inner = esz == 1 ? c->d : 64;
  const cuuint32_t box[4] = {inner, static_cast<cuuint32_t>(std::min(c->page_size, tile)), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle sw = !swizzle              ? CU_TENSOR_MAP_SWIZZLE_NONE
                                : inner * esz == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                     : CU_TENSOR_MAP_SWIZZLE_64B;
  const CUtensorMapDataType type = esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
  return encode_map(m, type, 4, const_cast<void*>(c->n_pages > 0 ? base : spare), dims, strides, box, one, sw);
}

// Packed rows (new tokens times query heads of a key head) up to which a sequence is the decode
// kernel's: that kernel reads the keys once per 16 rows, the prompt kernel computes 256 at a time.
// 16 sequences of 16000 tokens, 8 key heads, d = 128, decode / prompt kernel: 16 rows bf16 196 / 188
// us, e4m3 182 / 196; 20 rows 356 / 192 and 327 / 196; 64 rows 669 / 194 and 620 / 194.  Of 1000 tokens,
// bf16: 16 rows 47 / 49, 20 rows 61 / 54.
constexpr int PG_DECODE_ROWS = 16;

struct PagedLayout {
  size_t turn_off, cut_off, prefix_off, part_off, lse_off, total;
};
// Whether a call with this many tokens in all may hold a sequence for the prompt kernel.
bool may_be_prompt(long long max_tokens, int group) { return group <= 128 && max_tokens * group > PG_DECODE_ROWS; }
bool paged_layout(long long tokens, int group, int d, int batch, int sms, PagedLayout& L) {
  if (d != 64 && d != 128) return false;
  const bool prompt = may_be_prompt(tokens, group);
  const size_t rows = static_cast<size_t>(2) * sms * (prompt ? prompt_part_rows() : DC_MAX_ROWS);
  const size_t items = prompt ? prompt_entries(static_cast<int>(tokens), group, batch) : 0;
  L.turn_off = WS_HDR_BYTES;
  L.cut_off = L.turn_off + ((static_cast<size_t>(sms) * 4 + 255) & ~size_t(255));
  L.prefix_off = L.cut_off + ((static_cast<size_t>(sms) * sizeof(CutUnit) + 255) & ~size_t(255));
  L.part_off = L.prefix_off + (((items + 1) * 8 + 255) & ~size_t(255));
  L.lse_off = L.part_off + rows * d * 4;
  L.total = (L.lse_off + rows * 4 + 255) & ~size_t(255);
  return true;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" {

size_t mk_paged_attention_workspace_size(long long tokens, int heads_q, int heads, int d, int batch) {
  if (tokens < 0 || tokens >= (1LL << 31) || heads < 1 || heads_q < 1 || heads_q % heads || batch < 0) return 0;
  PagedLayout L;
  const int sms = std::max(1, device_sm_count());
  return paged_layout(tokens, heads_q / heads, d, batch, sms, L) ? L.total : 0;
}

mk_status mk_paged_attention(const void* q, void* out, float* lse, mk_dtype dtype, long long tokens, int heads_q,
                             long long q_token, long long q_head, long long o_token, long long o_head,
                             const mk_kv_cache* cache, const mk_seq_batch* seqs, float scale, int causal, int window,
                             int sinks, int max_q, void* workspace, size_t ws_bytes, const mk_config* cfg,
                             mk_stream_t stream) {
  if (dtype != MK_BF16 && dtype != MK_F16) return MK_ERR_INVALID;
  PagedParams p;
  std::memset(&p, 0, sizeof(p));
  if (!view_of(cache, p.c) || !view_of(seqs, tokens, p.s)) return MK_ERR_INVALID;
  const bool e8 = cache->dtype == MK_E4M3;
  if (e8 ? dtype != MK_BF16 : cache->dtype != dtype) return MK_ERR_INVALID;
  const int d = cache->d;
  if (heads_q < 1 || heads_q % cache->heads || heads_q > (1 << 16)) return MK_ERR_INVALID;
  if (!(scale > 0.f) || !std::isfinite(scale) || window < 0 || sinks < 0 || max_q < 0) return MK_ERR_INVALID;
  if (cfg && (cfg->operand != 0 || cfg->mode != 0 || cfg->max_ctas < 0)) return MK_ERR_INVALID;
  PagedLayout L;
  const int dev_sms = device_sm_count();
  if (!paged_layout(tokens, heads_q / cache->heads, d, seqs->batch, std::max(1, dev_sms), L)) return MK_ERR_INVALID;
  if (!workspace || ws_bytes < L.total || (reinterpret_cast<uintptr_t>(workspace) & 15u)) return MK_ERR_INVALID;
  if (tokens == 0 || seqs->batch == 0) return MK_OK;
  if (!q || !out) return MK_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out)) & 15u) return MK_ERR_INVALID;
  if (((q_token | q_head | o_token | o_head) * 2) & 15) return MK_ERR_INVALID;
  if (q_token < 0 || q_head < 0 || o_token < 0 || o_head < 0 || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MK_ERR_INVALID;
  if ((o_token == 0 && tokens > 1) || (o_head == 0 && heads_q > 1)) return MK_ERR_INVALID;   // rows that share memory
  if (dev_sms <= 0) return MK_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.qs_t = q_token;
  p.qs_h = q_head;
  p.os_t = o_token;
  p.os_h = o_head;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.hdr = reinterpret_cast<uint32_t*>(ws);
  p.turn = reinterpret_cast<uint32_t*>(ws + L.turn_off);
  p.cut = reinterpret_cast<CutUnit*>(ws + L.cut_off);
  p.prefix = reinterpret_cast<long long*>(ws + L.prefix_off);
  p.part = reinterpret_cast<float*>(ws + L.part_off);
  p.part_lse = reinterpret_cast<float*>(ws + L.lse_off);
  p.wait_ns = default_wait_ns(cfg);
  p.inject = cfg ? cfg->inject : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.heads_q = heads_q;
  p.group = heads_q / cache->heads;
  p.causal = causal ? 1 : 0;
  p.window = window;
  p.sinks = sinks;
  p.map_pages = static_cast<int>(std::max(1LL, cache->n_pages));
  // (and so far below 2^31 that the ends of tiles and boxes after it are ints)
  p.len_max = static_cast<int>(std::min(static_cast<long long>(p.s.max_pages) << p.c.page_log2, 0x7fffffffLL - 8192));
  p.grid = grid_cap(cfg);
  if (p.grid <= 0) return MK_ERR_UNSUPPORTED;
  // Which kernels: by the most new tokens a sequence can have.  A kernel that is launched alone
  // takes every sequence, whatever the hint was; of two, each takes its side of PG_DECODE_ROWS.
  // Queries with a stride of 0 are the decode kernel's: the prompt kernel's tensor map has no such stride.
  const long long most = max_q > 0 ? std::min<long long>(max_q, tokens) : tokens;
  const bool q_map = (q_token > 0 || tokens == 1) && (q_head > 0 || heads_q == 1);
  const bool prompt = q_map && may_be_prompt(most, p.group);
  const bool decode = !prompt || (seqs->batch > 1 && most * seqs->batch != tokens);
  if (decode) {
    const int tile = d == 128 && !e8 ? Shape<__half, false, 128, 1>::KT : 64;
    // 8 packed rows to a unit where no sequence has more, else 16: the keys are read once for either,
    // but 8 rows as 16 take twice the MMAs, on eight warps (128 sequences of up to 32000 tokens, e4m3,
    // 8 rows: 724 us alone, as 16: 1184; 48 windows of 4096, fp16, 4 rows: 103 and 114)
    const int nq = most * p.group <= 8 ? 1 : 2;
    if (!cache_map(&p.tmK, cache, cache->k, ws, tile, true) || !cache_map(&p.tmV, cache, cache->v, ws, tile, true))
      return MK_ERR_CUDA;
    p.rows_lo = 1;
    p.rows_hi = prompt ? PG_DECODE_ROWS : 0x7fffffff;
    for (int b0 = 0; b0 < seqs->batch; b0 += DC_BATCH) {
      PagedParams part = p;
      part.s.batch = std::min(DC_BATCH, seqs->batch - b0);
      part.s.cu_q = seqs->cu_q + b0;
      part.s.kv_len = seqs->kv_len + b0;
      part.s.pages = seqs->pages + static_cast<long long>(b0) * seqs->pages_stride;
      cudaError_t e;
      if (e8) e = launch_decode<__nv_bfloat16, true>(part, nq, s);
      else if (dtype == MK_BF16) e = launch_decode<__nv_bfloat16, false>(part, nq, s);
      else e = launch_decode<__half, false>(part, nq, s);
      if (e != cudaSuccess) return MK_ERR_CUDA;
    }
  }
  if (prompt) {
    if (!cache_map(&p.tmK, cache, cache->k, ws, 128, !e8) || !cache_map(&p.tmV, cache, cache->v, ws, 128, !e8))
      return MK_ERR_CUDA;
    // Q as [d, query heads, tokens]: a box holds the heads of one key head for the tokens of a tile
    const cuuint64_t row = static_cast<cuuint64_t>(d) * 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads_q),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {q_head > 0 ? static_cast<cuuint64_t>(q_head) * 2 : row,
                                   q_token > 0 ? static_cast<cuuint64_t>(q_token) * 2 : row};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(128 / p.group)};
    const cuuint32_t one[3] = {1, 1, 1};
    if (!encode_map(&p.tmQ, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(q), dims, strides, box, one,
                    CU_TENSOR_MAP_SWIZZLE_128B))
      return MK_ERR_CUDA;
    p.rows_lo = decode ? PG_DECODE_ROWS + 1 : 1;
    p.rows_hi = 0x7fffffff;
    if (launch_prompt(p, d, dtype, e8, decode, s) != cudaSuccess) return MK_ERR_CUDA;
  }
  return MK_OK;
}

}  // extern "C"
