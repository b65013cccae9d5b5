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
//     32- or 64-key stages (128 KB), so a page's end inside a tile costs nothing;
//   * eight warps take the tiles in turn, each with its own running maximum,
//     sum and 16 x d accumulator (mma.sync m16n8k16: the 16 rows fill the
//     instruction; a 128-row tcgen05 tile would be 7/8 empty), joined in shared
//     memory at the end of a run's part of a unit;
//   * units cut by a run's end leave normalised fp32 partial rows with their
//     log2 sums, joined by a second, programmatically dependent launch.
// 8-bit caches: codes become fp16, exactly; the query row is scaled by a power
// of two to fit fp16 (bf16 has fewer bits), the key scale multiplies the
// scores, the value scale (relative to the largest so far) the weights.
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

constexpr int DC_WARPS = 8;            // consumer warps; one more loads
constexpr int DC_THREADS = 32 * (DC_WARPS + 1);
constexpr int DC_ROWS = 16;            // packed query rows of a unit
constexpr int DC_BATCH = 1024;         // sequences of one launch (the entry point slices larger batches)

template <class T, bool E8, int D>
struct Shape {
  static constexpr int KT = (!E8 && D == 128) ? 32 : 64;              // keys of a tile: stages of 8 or 16 KB
  static constexpr int TILE = KT * D * (E8 ? 1 : 2);
  static constexpr int STAGE = 2 * TILE;
  static constexpr int PITCH = D + 4;                                 // floats of a row in the join buffer
  static constexpr int MERGE = DC_WARPS * DC_ROWS * PITCH * 4;
  static constexpr int ML = DC_WARPS * DC_ROWS * 3 * 4;               // maximum, sum, value scale
  static constexpr int PREFIX = (DC_BATCH + 1) * 8;
  static constexpr int FIXED = 1024 + MERGE + ML + ((PREFIX + 15) & ~15) + 512;
  // A warp's tiles come DC_WARPS apart.  With a multiple of that many stages the fill before
  // the one it waits for was its own, so the barrier's phase parity cannot be mistaken.
  static constexpr int STAGES = std::min((232448 - FIXED) / STAGE, 16) / DC_WARPS * DC_WARPS;
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
template <int KT>
__device__ __forceinline__ Segment segment_at(const PagedParams& p, const long long* pre, int b, long long x,
                                              long long end) {
  Segment g;
  g.b = b;
  sequence_of(p, b, g.n, g.len, g.row0);
  g.t = key_tiles<KT>(p, g.len - g.n, g.len - 1, g.len);
  g.count = g.t.count();
  const int groups = (g.n * p.group + DC_ROWS - 1) / DC_ROWS;
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
template <int KT>
__device__ __forceinline__ long long sequence_tiles(const PagedParams& p, int b) {
  int n, len, row0;
  if (!sequence_of(p, b, n, len, row0)) return 0;
  if (!rows_are_ours(p, n)) return 0;
  const long long rows = static_cast<long long>(n) * p.group;
  return ((rows + DC_ROWS - 1) / DC_ROWS) * key_tiles<KT>(p, len - n, len - 1, len).count();
}

template <int KT, bool E8, int D>
__device__ void dc_producer(const PagedParams& p, const long long* pre, volatile int* dead, uint32_t full, uint32_t empty,
                            uint32_t ring, int stages, long long x, long long end) {
  constexpr int TILE = KT * D * (E8 ? 1 : 2);
  const int lane = threadIdx.x & 31;
  const int box = min(p.c.page_size, KT), boxes = KT / box;
  int b = warp_last_le(p.s.batch, 0, [&](int i) { return pre[i] * p.c.heads <= x ? 0 : 1; });
  int st = 0;
  uint32_t ph = 0;
  while (x < end) {
    while (pre[b + 1] * p.c.heads <= x) ++b;
    const Segment g = segment_at<KT>(p, pre, b, x, end);
    const int n_pages = min(p.s.max_pages, ((g.len - 1) >> p.c.page_log2) + 1);
    const int* table = p.s.pages + g.b * p.s.pages_stride;
    // the page of this lane's box of tile k; the maps' first absent page where there is none
    auto page_of = [&](int k) {
      const int lp = (g.t.tile(k) * KT + lane * box) >> p.c.page_log2;
      if (lane >= boxes || lp >= n_pages) return p.map_pages;
      const int id = table[lp];
      if (id >= 0 && id < p.c.n_pages) return id;
      if (keys_seen(p, g.len - g.n, g.len - 1, g.len, g.t.tile(k) * KT + lane * box, box))
        seq_error(p.hdr, MK_ERR_INVALID, WHERE_PRODUCER, g.b);
      return p.map_pages;
    };
    if (lane == 0 && ((g.len - 1) >> p.c.page_log2) >= p.s.max_pages)
      seq_error(p.hdr, MK_ERR_CAPACITY, WHERE_PRODUCER, g.b);
    int next = page_of(g.k0);
    for (int k = g.k0; k < g.k1; ++k) {
      const int page = next;
      if (k + 1 < g.k1) next = page_of(k + 1);
      if (!__all_sync(0xffffffffu, pg_wait(dead, p, empty + 8u * st, ph ^ 1u, WHERE_PRODUCER))) return;
      const uint32_t bar = full + 8u * st;
      if (lane == 0) mbar_arrive_expect_tx(bar, 2u * TILE);
      __syncwarp();
      if (lane < boxes) {
        const uint32_t kdst = ring + static_cast<uint32_t>(st) * 2u * TILE;
        const int slot = (g.t.tile(k) * KT + lane * box) & (p.c.page_size - 1);
        constexpr int ATOMS = E8 ? 1 : D / 64;
        constexpr uint32_t ROW = E8 ? D : 128;
#pragma unroll
        for (int a = 0; a < ATOMS; ++a) {
          const uint32_t off = a * (KT * 128u) + lane * box * ROW;
          tma_load_4d(kdst + off, &p.tmK, bar, 64 * a, slot, g.h, page);
          tma_load_4d(kdst + TILE + off, &p.tmV, bar, 64 * a, slot, g.h, page);
        }
      }
      if (++st == stages) {
        st = 0;
        ph ^= 1u;
      }
    }
    x += g.k1 - g.k0;
  }
}

template <class T, bool E8, int D>
__global__ void __launch_bounds__(DC_THREADS, 1) mk_paged_decode_kernel(const __grid_constant__ PagedParams p) {
  using S = Shape<T, E8, D>;
  constexpr bool HALF = E8 || !std::is_same<T, __nv_bfloat16>::value;   // fp16 operands of the products
  constexpr float SHIFT = HALF ? 10.f : 0.f;   // fp16 weights are taken 2^10 high: small ones keep their bits
  constexpr int KT = S::KT, KS = D / 16, NT = KT / 8, OT = D / 8;
  extern __shared__ uint8_t dyn[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  float* merge = reinterpret_cast<float*>(sm + S::STAGES * S::STAGE);
  float* ml = reinterpret_cast<float*>(sm + S::STAGES * S::STAGE + S::MERGE);
  long long* pre = reinterpret_cast<long long*>(sm + S::STAGES * S::STAGE + S::MERGE + S::ML);
  uint8_t* tail = reinterpret_cast<uint8_t*>(pre) + ((S::PREFIX + 15) & ~15);
  volatile int* dead = reinterpret_cast<int*>(tail + 256);
  const uint32_t ring = smem_u32(sm), full = smem_u32(tail), empty = full + 128u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int batch = p.s.batch;

  griddep_launch_dependents();
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
  for (int b = threadIdx.x; b < batch; b += DC_THREADS) pre[b + 1] = sequence_tiles<KT>(p, b);
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
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= batch; b += DC_THREADS) p.prefix[b] = pre[b];
  const Deal deal(pre[batch] * p.c.heads, p.grid);
  for (int b = blockIdx.x; b < batch; b += gridDim.x) {   // sequences without a key: nothing is seen
    int n, len, row0;
    if (pre[b + 1] == pre[b] && sequence_of(p, b, n, len, row0) && rows_are_ours(p, n))
      no_keys<T, D>(p, row0, n, DC_THREADS);
  }
  if (static_cast<int>(blockIdx.x) >= deal.c) return;
  long long x = deal.start(blockIdx.x);
  const long long end = deal.start(blockIdx.x + 1);
  if (warp == DC_WARPS) {
    dc_producer<KT, E8, D>(p, pre, dead, full, empty, ring, S::STAGES, x, end);
    __syncwarp();
  } else {
    const int r = lane >> 2, c = lane & 3;
    int b = warp_last_le(batch, 0, [&](int i) { return pre[i] * p.c.heads <= x ? 0 : 1; });
    uint32_t done = 0;                   // tiles of the run before this segment
    while (x < end) {
      while (pre[b + 1] * p.c.heads <= x) ++b;
      const Segment g = segment_at<KT>(p, pre, b, x, end);
      if (done == 0 && threadIdx.x == 0)
        p.cut[blockIdx.x] = CutUnit{g.u0 < x ? g.u0 : -1, g.count, g.row0, g.n, g.h, g.rg};
      const int p0 = g.len - g.n, p1 = g.len - 1;
      const int tiles = g.k1 - g.k0;
      const int first = (warp - static_cast<int>(done % DC_WARPS) + DC_WARPS) % DC_WARPS;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, vrun = 0.f;
      float o[OT][4];
#pragma unroll
      for (int j = 0; j < OT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
      if (first < tiles) {
        // the query rows r and r + 8 of the group, as operand registers
        uint32_t qf[KS][4];
        int pos[2];
        float row_scale[2] = {p.scale_log2, p.scale_log2};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = g.rg * DC_ROWS + r + 8 * i;
          const int tok = row / p.group, head = g.h * p.group + row - tok * p.group;
          const bool ok = tok < g.n;
          pos[i] = p0 + (ok ? tok : 0);
          const T* src = static_cast<const T*>(p.q) + static_cast<long long>(g.row0 + (ok ? tok : 0)) * p.qs_t +
                         (ok ? head : 0) * p.qs_h;
          if (!E8) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              qf[ks][i] = ok ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * c) : 0u;
              qf[ks][i + 2] = ok ? *reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * c + 8) : 0u;
            }
          } else {
            // 16 neighbouring elements for every 64: the order in which the codes are read
            float f[D / 4], top = 0.f;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
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
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // a power of two that brings the row's largest magnitude to 2^10 .. 2^11
            const int ex = min(max(static_cast<int>((__float_as_uint(top) >> 23) & 255) - 127, -100), 126);
            const float up = __uint_as_float(static_cast<uint32_t>(10 - ex + 127) << 23);
            row_scale[i] *= __uint_as_float(static_cast<uint32_t>(max(ex - 10, -126) + 127) << 23);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              const int e = 16 * (ks >> 2) + 4 * (ks & 3);
              qf[ks][i] = f16x2(f[e] * up, f[e + 1] * up);
              qf[ks][i + 2] = f16x2(f[e + 2] * up, f[e + 3] * up);
            }
          }
        }
        // 8-bit: lane j < 8 holds the scales of keys 8 j .. 8 j + 7 of a tile
        const int* table = p.s.pages + g.b * p.s.pages_stride;
        const int n_pages = min(p.s.max_pages, (p1 >> p.c.page_log2) + 1);
        auto id_of = [&](int k) {      // -1 for keys no row sees: their scales may be anything
          const int key = g.t.tile(k) * KT + 8 * (lane & 7), lp = key >> p.c.page_log2;
          if (lp >= n_pages || !keys_seen(p, p0, p1, g.len, key, 8)) return -1;
          const int id = table[lp];
          return id < p.c.n_pages ? id : -1;
        };
        float ks_now = 0.f, vs_now = 0.f;
        auto scales_of = [&](int id) {
          const long long at = static_cast<long long>(id) * p.c.heads + g.h;
          ks_now = id >= 0 ? p.c.k_scale[at] : 0.f;
          vs_now = id >= 0 ? p.c.v_scale[at] : 0.f;
        };
        if (E8) scales_of(id_of(g.k0 + first));
        for (int k = first; k < tiles; k += DC_WARPS) {
          const uint32_t i = done + k;
          const int st = i % S::STAGES;
          const uint32_t kt = ring + st * S::STAGE, vt = kt + S::TILE;
          int next_id = -1;
          if (E8 && k + DC_WARPS < tiles) next_id = id_of(g.k0 + k + DC_WARPS);
          const float ks_tile = ks_now, vs_tile = vs_now;
          const int ok = pg_wait(dead, p, full + 8u * st, (i / S::STAGES) & 1u, WHERE_MMA) ? 1 : 0;
          if (!__all_sync(0xffffffffu, ok)) break;
          const int key0 = g.t.tile(g.k0 + k) * KT;
          const bool masked = !all_seen(p, p0, p1, g.len, key0, KT);
          // ---- scores
          float s[NT][4];
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
          if (!E8) {
            const int krow = ((lane >> 4) << 3) + (lane & 7), kch = (lane >> 3) & 1;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
              for (int j = 0; j < NT; j += 2) {
                uint32_t f[4];
                ldsm4(kt + piece_at<KT, E8, D>(8 * j + krow, 2 * ks + kch), f);
                mma16816(s[j], qf[ks], f[0], f[1], HALF);
                mma16816(s[j + 1], qf[ks], f[2], f[3], HALF);
              }
          } else {
            // column n of a group of 8 is key (n >> 1) | (n & 1) << 2: the four lanes of
            // neighbouring columns then read different banks
            const int kperm = (r >> 1) | ((r & 1) << 2);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int a = 0; a < D / 64; ++a) {
                uint32_t f[4];
                lds128(kt + piece_at<KT, E8, D>(8 * j + kperm, 4 * a + c), f);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                  mma16816(s[j], qf[4 * a + w], e4m3_f16x2(f[w] & 0xffffu), e4m3_f16x2(f[w] >> 16), HALF);
              }
          }
          // ---- softmax of rows r (e = 0, 1) and r + 8 (e = 2, 3)
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float f = E8 ? __shfl_sync(0xffffffffu, ks_tile, j) : 1.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float z = s[j][e] * (E8 ? row_scale[e >> 1] * f : p.scale_log2);
              if (masked) {
                const int key = key0 + 8 * j + (E8 ? c + 4 * (e & 1) : 2 * c + (e & 1));
                if (!key_seen(p, pos[e >> 1], g.len, key)) z = -INFINITY;
              }
              s[j][e] = z;
              top[e >> 1] = fmaxf(top[e >> 1], z);
            }
          }
          float mref[2], alpha[2];
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            top[i2] = fmaxf(top[i2], __shfl_xor_sync(0xffffffffu, top[i2], 1));
            top[i2] = fmaxf(top[i2], __shfl_xor_sync(0xffffffffu, top[i2], 2));
            const float mn = fmaxf(m[i2], top[i2]);
            mref[i2] = mn == -INFINITY ? 0.f : mn;
            alpha[i2] = pg_ex2(m[i2] - mref[i2]);
            m[i2] = mn;
            l[i2] *= alpha[i2];
          }
          if (E8) {                      // O is kept in units of the largest value scale so far
            float top_v = vs_tile;
            top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, 1));
            top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, 2));
            top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, 4));
            if (top_v > vrun) {
              const float f = vrun / top_v;
              alpha[0] *= f;
              alpha[1] *= f;
              vrun = top_v;
            }
          }
          if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < OT; ++j) {
              o[j][0] *= alpha[0];
              o[j][1] *= alpha[0];
              o[j][2] *= alpha[1];
              o[j][3] *= alpha[1];
            }
          }
          uint32_t pf[NT][2];
          const float vinv = E8 && vrun > 0.f ? 1.f / vrun : 0.f;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float w[4];
            const float f = E8 ? __shfl_sync(0xffffffffu, vs_tile, j) * vinv : 1.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              w[e] = pg_ex2(s[j][e] - mref[e >> 1] + SHIFT);
              l[e >> 1] += w[e];
              if (E8) w[e] = w[e] == 0.f ? 0.f : w[e] * f;
            }
            pf[j][0] = HALF ? f16x2(w[0], w[1]) : pack_bf16x2(w[0], w[1]);
            pf[j][1] = HALF ? f16x2(w[2], w[3]) : pack_bf16x2(w[2], w[3]);
          }
          if (E8) scales_of(next_id);
          if (masked) {
            // 0 * NaN is NaN: values no row sees (past the end, before the window) may hold
            // anything and are cleared, and of those only some rows see (several new tokens)
            // what is not finite is cleared and added below to the rows that do see it
            constexpr int CH = D * (E8 ? 1 : 2) / 16;
            uint32_t odd[2] = {0u, 0u};
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
            for (int key = 0; (odd[0] | odd[1]) != 0u && key < KT; ++key) {
              if (!((odd[key >> 5] >> (key & 31)) & 1u)) continue;
              int page;
              const long long row = value_row(p, g.b, g.h, key0 + key, page);
              if (row < 0) continue;
#pragma unroll
              for (int j = 0; j < OT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int col = 2 * c + (e & 1);
                  const float v = not_finite<T, E8>(p.c.v, row + (E8 ? (D / 8) * col + j : 8 * j + col));
                  if (v != 0.f && key_seen(p, pos[e >> 1], g.len, key0 + key)) o[j][e] += v;
                }
            }
            __syncwarp();
          }
          // ---- O += P V
          if (!E8) {
            const int vrow = (((lane >> 3) & 1) << 3) + (lane & 7), vch = lane >> 4;
#pragma unroll
            for (int t = 0; t < KT / 16; ++t) {
              const uint32_t a[4] = {pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1]};
#pragma unroll
              for (int j = 0; j < OT; j += 2) {
                uint32_t f[4];
                ldsm4_t(vt + piece_at<KT, E8, D>(16 * t + vrow, j + vch), f);
                mma16816(o[j], a, f[0], f[1], HALF);
                mma16816(o[j + 1], a, f[2], f[3], HALF);
              }
            }
          } else {
            // lane (r, c) reads keys c, c+4, c+8, c+12 of 16, elements (D/8) r ..: output
            // tile j has element (D/8) n + j in column n
#pragma unroll
            for (int t = 0; t < KT / 16; ++t) {
              const uint32_t a[4] = {pf[2 * t][0], pf[2 * t][1], pf[2 * t + 1][0], pf[2 * t + 1][1]};
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
              for (int w = 0; w < D / 32; ++w) {    // 4 x 4 bytes turned: element j of the four keys
                const uint32_t x0 = __byte_perm(f[0][w], f[1][w], 0x5140), x1 = __byte_perm(f[0][w], f[1][w], 0x7362);
                const uint32_t y0 = __byte_perm(f[2][w], f[3][w], 0x5140), y1 = __byte_perm(f[2][w], f[3][w], 0x7362);
                mma16816(o[4 * w], a, e4m3_f16x2(x0 & 0xffffu), e4m3_f16x2(y0 & 0xffffu), HALF);
                mma16816(o[4 * w + 1], a, e4m3_f16x2(x0 >> 16), e4m3_f16x2(y0 >> 16), HALF);
                mma16816(o[4 * w + 2], a, e4m3_f16x2(x1 & 0xffffu), e4m3_f16x2(y1 & 0xffffu), HALF);
                mma16816(o[4 * w + 3], a, e4m3_f16x2(x1 >> 16), e4m3_f16x2(y1 >> 16), HALF);
              }
            }
          }
          if (masked) fence_proxy_async_smem();   // the cleared rows before the next load of this stage
          __syncwarp();
          if (lane == 0) mbar_arrive(empty + 8u * st);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
          l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        }
        float* mine = merge + warp * DC_ROWS * S::PITCH;
#pragma unroll
        for (int j = 0; j < OT; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float* at = mine + (r + 8 * i) * S::PITCH;
            if (!E8) {
              *reinterpret_cast<float2*>(at + 8 * j + 2 * c) = make_float2(o[j][2 * i], o[j][2 * i + 1]);
            } else {
              at[(D / 8) * (2 * c) + j] = o[j][2 * i];
              at[(D / 8) * (2 * c + 1) + j] = o[j][2 * i + 1];
            }
          }
      }
      if (c == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float* at = ml + (warp * DC_ROWS + r + 8 * i) * 3;
          at[0] = m[i];
          at[1] = l[i];
          at[2] = E8 ? vrun : 1.f;
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      {
        // join: 16 threads a row, D / 16 neighbouring elements each
        constexpr int EL = D / 16;
        const int row = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * EL;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < DC_WARPS; ++w) top = fmaxf(top, ml[(w * DC_ROWS + row) * 3]);
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f, acc[EL];
#pragma unroll
        for (int e = 0; e < EL; ++e) acc[e] = 0.f;
        for (int w = 0; w < DC_WARPS; ++w) {
          const float* at = ml + (w * DC_ROWS + row) * 3;
          if (at[1] == 0.f) continue;             // no tile, or nothing seen (NaN stays in)
          const float f = pg_ex2(at[0] - ref);
          sum += f * at[1];
          const float fv = f * at[2];
#pragma unroll
          for (int e = 0; e < EL; e += 4) {
            const float4 v = *reinterpret_cast<const float4*>(merge + (w * DC_ROWS + row) * S::PITCH + d0 + e);
            acc[e] += fv * v.x;
            acc[e + 1] += fv * v.y;
            acc[e + 2] += fv * v.z;
            acc[e + 3] += fv * v.w;
          }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const float lse2 = sum == 0.f ? -INFINITY : ref + log2f(sum) - SHIFT;
        const int prow = g.rg * DC_ROWS + row;
        if (prow < g.n * p.group) {
          if (tiles == g.count) {                 // the whole unit: final
            const int tok = prow / p.group, head = g.h * p.group + prow - tok * p.group;
            const long long t = g.row0 + tok;
            T* dst = static_cast<T*>(p.out) + t * p.os_t + head * p.os_h + d0;
            if constexpr (EL == 8) {
              float v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = acc[e] * inv;
              *reinterpret_cast<uint4*>(dst) = Piece<T>::put(v);
            } else {
              uint2 w;
              w.x = HALF && !E8 ? f16x2(acc[0] * inv, acc[1] * inv) : pack_bf16x2(acc[0] * inv, acc[1] * inv);
              w.y = HALF && !E8 ? f16x2(acc[2] * inv, acc[3] * inv) : pack_bf16x2(acc[2] * inv, acc[3] * inv);
              *reinterpret_cast<uint2*>(dst) = w;
            }
            if (p.lse != nullptr && d0 == 0) p.lse[t * p.heads_q + head] = lse2 * LN2;
          } else {
            const long long at = static_cast<long long>(part_slot(blockIdx.x, g.k0 == 0)) * DC_ROWS + row;
#pragma unroll
            for (int e = 0; e < EL; e += 4)
              *reinterpret_cast<float4*>(p.part + at * D + d0 + e) =
                  make_float4(acc[e] * inv, acc[e + 1] * inv, acc[e + 2] * inv, acc[e + 3] * inv);
            if (d0 == 0) p.part_lse[at] = lse2;
          }
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      done += tiles;
      x += tiles;
    }
  }
  if (*dead) {   // loads whose barrier nobody waited for may still be landing
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 50000ull) __nanosleep(1000);
  }
}

// ------------------------------------------------------------------ join

// Block i - 1: if CTA i's run begins inside a unit that CTA i - 1 began, that unit's rows.
template <class T, int D>
__global__ void __launch_bounds__(256) mk_paged_join_kernel(const __grid_constant__ PagedParams p) {
  griddep_wait();
  const int i = blockIdx.x + 1;
  const CutUnit g = p.cut[i];
  const Deal deal(p.prefix[p.s.batch] * p.c.heads, p.grid);
  if (i >= deal.c || g.u0 < 0 || deal.start(i - 1) > g.u0) return;
  const int row = threadIdx.x >> 4, prow = g.at * DC_ROWS + row;
  if (prow >= g.n * p.group) return;
  const int tok = prow / p.group;
  join_row<T, D, DC_ROWS>(p, i - 1, deal.owner(g.u0 + g.count - 1), row, g.row0 + tok, g.h * p.group + prow - tok * p.group);
}

// ------------------------------------------------------------------ host

template <class T, bool E8, int D>
cudaError_t launch_decode(const PagedParams& p, cudaStream_t s) {
  using S = Shape<T, E8, D>;
  static_assert(S::STAGES >= DC_WARPS, "a stage for each warp");
  static int configured_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_dev != dev) {
    e = cudaFuncSetAttribute(mk_paged_decode_kernel<T, E8, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    configured_dev = dev;
  }
  mk_paged_decode_kernel<T, E8, D><<<p.grid, DC_THREADS, S::SMEM, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (p.grid < 2) return e;
  return launch_dependent(mk_paged_join_kernel<T, D>, dim3(p.grid - 1), dim3(256), s, p);
}

// K / V as [d, slots, heads, pages]; a box is the part of a page that falls into a tile of `tile` keys.
bool cache_map(CUtensorMap* m, const mk_kv_cache* c, const void* base, const void* spare, int tile, bool swizzle) {
  const int esz = c->dtype == MK_E4M3 ? 1 : 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->heads),
                              static_cast<cuuint64_t>(std::max(1LL, c->n_pages))};
  // a stride of a dimension of one element says nothing, but the map wants it positive
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
constexpr int PG_DECODE_ROWS = 64;

struct PagedLayout {
  size_t cut_off, prefix_off, part_off, lse_off, total;
};
// Whether a call with this many tokens in all may hold a sequence for the prompt kernel.
bool may_be_prompt(long long max_tokens, int group) { return group <= 128 && max_tokens * group > PG_DECODE_ROWS; }
bool paged_layout(long long tokens, int group, int d, int batch, int sms, PagedLayout& L) {
  if (d != 64 && d != 128) return false;
  const bool prompt = may_be_prompt(tokens, group);
  const size_t rows = static_cast<size_t>(2) * sms * (prompt ? prompt_part_rows() : DC_ROWS);
  const size_t units = std::max<size_t>(std::min(batch, DC_BATCH),
                                        prompt ? prompt_entries(static_cast<int>(tokens), group, batch) : 0);
  L.cut_off = WS_HDR_BYTES;
  L.prefix_off = L.cut_off + ((static_cast<size_t>(sms) * sizeof(CutUnit) + 255) & ~size_t(255));
  L.part_off = L.prefix_off + (((units + 1) * 8 + 255) & ~size_t(255));
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
  p.cut = reinterpret_cast<CutUnit*>(ws + L.cut_off);
  p.prefix = reinterpret_cast<long long*>(ws + L.prefix_off);
  p.part = reinterpret_cast<float*>(ws + L.part_off);
  p.part_lse = reinterpret_cast<float*>(ws + L.lse_off);
  p.wait_ns = default_wait_ns(cfg);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.heads_q = heads_q;
  p.group = heads_q / cache->heads;
  p.causal = causal ? 1 : 0;
  p.window = window;
  p.sinks = sinks;
  p.map_pages = static_cast<int>(std::max(1LL, cache->n_pages));
  p.grid = grid_cap(cfg);
  if (p.grid <= 0) return MK_ERR_UNSUPPORTED;
  // Which kernels: by the most new tokens a sequence can have.  A kernel that is launched alone
  // takes every sequence, whatever the hint was; of two, each takes its side of PG_DECODE_ROWS.
  const long long most = max_q > 0 ? std::min<long long>(max_q, tokens) : tokens;
  const bool prompt = may_be_prompt(most, p.group);
  const bool decode = !prompt || (seqs->batch > 1 && most * seqs->batch != tokens);
  if (decode) {
    const int tile = !e8 && d == 128 ? Shape<__nv_bfloat16, false, 128>::KT : Shape<__nv_bfloat16, true, 128>::KT;
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
      if (e8)
        e = d == 128 ? launch_decode<__nv_bfloat16, true, 128>(part, s) : launch_decode<__nv_bfloat16, true, 64>(part, s);
      else if (dtype == MK_BF16)
        e = d == 128 ? launch_decode<__nv_bfloat16, false, 128>(part, s) : launch_decode<__nv_bfloat16, false, 64>(part, s);
      else
        e = d == 128 ? launch_decode<__half, false, 128>(part, s) : launch_decode<__half, false, 64>(part, s);
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
    if (launch_prompt(p, d, dtype, e8, s) != cudaSuccess) return MK_ERR_CUDA;
  }
  return MK_OK;
}

}  // extern "C"
