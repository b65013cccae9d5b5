// mk_prompt.cu -- attention over a paged cache for sequences with many new
// tokens (prompts and pieces of prompts): tcgen05 products, bound by the tensor
// cores and by the chain score -> exponentials -> value product of a tile.
//
// The query rows of a (sequence, key head) are its new tokens times the G query
// heads that share the key head.  An item is two 128-row query tiles of
// floor(128 / G) tokens each, so every 128-key tile brought into shared memory
// serves up to 256 rows.  The list of all (item, head, key tile) of the batch is
// cut into one equal run per CTA (one CTA per SM), wherever that falls: causal
// items of any length and few long ones alike keep every SM busy to the end.
// Items cut by a run's end leave fp32 partial rows for the join (mk_paged.cu).
//
// Roles of a CTA's warps:
//   0-3, 4-7  softmax of query tile 0 / 1, one row a thread: the 128 scores of a
//             key tile are held in registers, the weights 2^(c s - m) go back into
//             tensor memory in 16 bits, over the scores; m is the running maximum,
//             which moves only when it grows by more than 2^8 (then O is scaled)
//   8         loads Q and K, 10 loads V: one TMA box a page and 64 columns
//   9         issues the MMAs: S_i = Q_i K^T, O_i += P_i V, in the order PV_0(u-1),
//             S_0(u), PV_1(u-1), S_1(u): one tile's products run while the other's
//             softmax does
//   11        clears the values that no row sees (see prompt_clear)
//   12-15     8-bit caches only: turn codes into bf16 tiles, scale and all
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "mk_paged.h"

namespace mk {

namespace {

constexpr int PR_T = 128;                    // query rows / keys of a tile
constexpr int PR_ST = 2;                     // K stages, V stages
constexpr uint32_t PR_COLS = 512;            // tensor memory: S_0, S_1, O_0, O_1, 128 columns each
constexpr uint32_t PR_O = 256;
constexpr float RESCALE = 8.f;
enum { W_LOAD = 8, W_MMA = 9, W_LOADV = 10, W_CLEAR = 11, W_TURN = 12 };

template <bool E8, int D>
struct Plan {
  static constexpr int THREADS = E8 ? 512 : 384;
  static constexpr uint32_t TILE = PR_T * D * 2;
  static constexpr uint32_t RAW = E8 ? PR_T * D : 0;      // codes as they arrive
  static constexpr uint32_t Q = 0, K = 2 * TILE, V = K + PR_ST * TILE, RK = V + PR_ST * TILE, RV = RK + RAW;
  static constexpr uint32_t BARS = RV + RAW;
  static constexpr int SMEM = 1024 + BARS + 512;
  static_assert(SMEM <= 232448, "dynamic shared memory per block");
  // registers: the launch gives every thread 168 (384 threads) or 128 (512); the softmax warps
  // hold a row of scores each, the others need few
  static constexpr int MANY = E8 ? 184 : 200, FEW = E8 ? 72 : 104;
  static_assert(256 * MANY + (THREADS - 256) * FEW <= THREADS * (E8 ? 128 : 168), "no more than the launch has");
};
// barriers (byte offsets)
constexpr uint32_t B_QFULL = 0, B_QEMPTY = 8, B_KFULL = 16, B_KEMPTY = 32, B_VFULL = 48, B_VEMPTY = 64, B_VREADY = 80,
                   B_S = 96, B_GO = 112, B_O = 128, B_DRAIN = 144, B_RKFULL = 152, B_RKEMPTY = 160, B_RVFULL = 168,
                   B_RVEMPTY = 176, B_TMEM = 192, B_DEAD = 196, B_ODD = 200;

__device__ __forceinline__ uint32_t idesc(int n, bool b_mn, bool half) {
  return idesc_bf16_f32(PR_T, n, false, b_mn) & (half ? ~((1u << 7) | (1u << 10)) : ~0u);
}

// Waits of a whole warp, which agrees by vote.  Inline: a kernel that divides its registers
// between warps cannot make calls.
__device__ __forceinline__ bool pr_wait_loop(volatile int* dead, const PagedParams& p, uint32_t bar, uint32_t parity,
                                          int where) {
  const uint64_t t0 = globaltimer_ns();
  uint32_t it = 0;
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    if ((++it & 15u) == 0) {
      int stop = 0;
      if ((threadIdx.x & 31) == 0) {
        if (*dead) {
          stop = 1;
        } else if (globaltimer_ns() - t0 > static_cast<uint64_t>(p.wait_ns)) {
          seq_error(p.hdr, MK_ERR_TIMEOUT, where, blockIdx.x);
          *dead = 1;
          stop = 1;
        }
      }
      if (__shfl_sync(0xffffffffu, stop, 0) != 0) return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool pr_wait(volatile int* dead, const PagedParams& p, uint32_t bar, uint32_t parity,
                                        int where) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return pr_wait_loop(dead, p, bar, parity, where);
}

// ------------------------------------------------------------------ work list

// Entries: item j of sequence b is entry cu_q[b] / T + b + j with T tokens an item: every
// sequence has room for its items, whatever the lengths; entries without one have no tiles.
struct Item {
  int b, n, len, row0, tok0;                 // sequence; new tokens, tokens in all, first row; first token
  KeyTiles t;
};
__device__ __forceinline__ bool item_of(const PagedParams& p, int e, int b, Item& it) {
  const int per = 2 * (PR_T / p.group);
  it.b = b;
  it.row0 = p.s.cu_q[b];
  it.n = min(p.s.cu_q[b + 1], p.s.tokens) - it.row0;
  it.len = p.s.kv_len[b];
  const int j = e - (it.row0 / per + b);
  if (it.row0 < 0 || it.n <= 0 || j < 0 || static_cast<long long>(j) * per >= it.n) return false;
  const long long rows = static_cast<long long>(it.n) * p.group;
  if (rows < p.rows_lo || rows > p.rows_hi) return false;
  it.tok0 = j * per;
  const int p0 = it.len - it.n + it.tok0;
  it.t = key_tiles<PR_T>(p, p0, min(p0 + per, it.len) - 1, it.len);
  return true;
}

// prefix[e] = tiles of one head in the entries before e; rows of items without tiles see nothing.
template <class T>
__global__ void __launch_bounds__(1024) mk_prompt_plan_kernel(const __grid_constant__ PagedParams p, int entries) {
  __shared__ long long part[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = 2 * (PR_T / p.group);
  griddep_launch_dependents();
  long long base = 0;
  for (int e0 = 0; e0 < entries; e0 += 1024) {
    const int e = e0 + threadIdx.x;
    long long n = 0;
    if (e < entries) {
      int lo = 0, hi = p.s.batch;            // the last b with cu_q[b] / per + b <= e
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.s.cu_q[mid] / per + mid <= e) lo = mid;
        else hi = mid;
      }
      Item it;
      if (item_of(p, e, lo, it)) n = it.t.count();
    }
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      const long long v = part[lane];
      long long s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
      }
      part[lane] = s - v;
      if (lane == 31) part[32] = s;
    }
    __syncthreads();
    if (e < entries) p.prefix[e] = base + part[warp] + incl - n;
    base += part[32];
    __syncthreads();
  }
  if (threadIdx.x == 0) p.prefix[entries] = base;
}

// A run's walk over its segments: the part of one item and head that lies in the run.
struct Walk {
  long long x, end;
  int e, entries;                            // current entry
  Item it;
  int h, k0, k1, count;
  long long u0;
  __device__ __forceinline__ Walk(const PagedParams& p, int entries_, const Deal& d) : entries(entries_) {
    x = d.start(blockIdx.x);
    end = d.start(blockIdx.x + 1);
    e = -1;
  }
  // The segment at x (by a whole warp); false at the run's end.
  __device__ __forceinline__ bool next(const PagedParams& p) {
    if (x >= end) return false;
    const long long heads = p.c.heads;
    if (e < 0) e = warp_last_le(entries, 0, [&](int i) { return p.prefix[i] * heads <= x ? 0 : 1; });
    while (p.prefix[e + 1] * heads <= x) ++e;
    const int per = 2 * (PR_T / p.group);
    const int b = warp_last_le(p.s.batch, e, [&](int i) { return p.s.cu_q[i] / per + i; });
    item_of(p, e, b, it);
    count = it.t.count();
    const long long rem = x - p.prefix[e] * heads;
    h = static_cast<int>(rem / count);
    k0 = static_cast<int>(rem - static_cast<long long>(h) * count);
    u0 = x - k0;
    k1 = static_cast<int>(min(static_cast<long long>(count), k0 + (end - x)));
    x += k1 - k0;
    return true;
  }
};

// The pages of a tile: box i of the tile has `box` keys from slot `slot`.
struct Pages {
  int box, boxes, n;
  const int* table;
  __device__ __forceinline__ Pages(const PagedParams& p, const Item& it) {
    box = min(p.c.page_size, PR_T);
    boxes = PR_T / box;
    n = min(p.s.max_pages, ((it.len - 1) >> p.c.page_log2) + 1);
    table = p.s.pages + it.b * p.s.pages_stride;
  }
  // the page of this lane's box; the maps' first absent page (zeros) where there is none
  __device__ __forceinline__ int of(const PagedParams& p, const Item& it, int tile, int lane) const {
    const int lp = (tile * PR_T + lane * box) >> p.c.page_log2;
    if (lane >= boxes || lp >= n) return p.map_pages;
    const int id = table[lp];
    if (id >= 0 && id < p.c.n_pages) return id;
    seq_error(p.hdr, MK_ERR_INVALID, WHERE_PRODUCER, it.b);
    return p.map_pages;
  }
};

// ------------------------------------------------------------------ loads

template <bool E8, int D>
__device__ __forceinline__ void load_tile(const PagedParams& p, const CUtensorMap* m, uint32_t dst, uint32_t bar,
                                          const Pages& g, int tile, int page, int h, int lane) {
  if (lane == 0) mbar_arrive_expect_tx(bar, E8 ? PR_T * D : PR_T * D * 2);
  __syncwarp();
  if (lane < g.boxes) {
    const int slot = (tile * PR_T + lane * g.box) & (p.c.page_size - 1);
    if (E8) {
      tma_load_4d(dst + lane * g.box * D, m, bar, 0, slot, h, page);
    } else {
#pragma unroll
      for (int a = 0; a < D / 64; ++a)
        tma_load_4d(dst + a * 16384u + lane * g.box * 128, m, bar, 64 * a, slot, h, page);
    }
  }
  __syncwarp();
}

// Warp 8: K, and after an item's first K tile its queries; 8-bit caches: V too.
template <bool E8, int D>
__device__ void pr_load(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint32_t base) {
  using P = Plan<E8, D>;
  const int lane = threadIdx.x & 31;
  const int toks = PR_T / p.group;
  uint32_t u = 0, q_ph = 0;
  while (w.next(p)) {
    const Pages g(p, w.it);
    if (lane == 0 && ((w.it.len - 1) >> p.c.page_log2) >= p.s.max_pages)
      seq_error(p.hdr, MK_ERR_CAPACITY, WHERE_PRODUCER, w.it.b);
    int next = g.of(p, w.it, w.it.t.tile(w.k0), lane);
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const int tile = w.it.t.tile(k), page = next;
      if (k + 1 < w.k1) next = g.of(p, w.it, w.it.t.tile(k + 1), lane);
      if (E8) {
        if (!pr_wait(dead, p, bars + B_RKEMPTY, (u & 1u) ^ 1u, WHERE_PRODUCER)) return;
        load_tile<E8, D>(p, &p.tmK, base + P::RK, bars + B_RKFULL, g, tile, page, w.h, lane);
      } else {
        const uint32_t st = u % PR_ST, ph = (u / PR_ST) & 1u;
        if (!pr_wait(dead, p, bars + B_KEMPTY + 8u * st, ph ^ 1u, WHERE_PRODUCER)) return;
        load_tile<E8, D>(p, &p.tmK, base + P::K + st * P::TILE, bars + B_KFULL + 8u * st, g, tile, page, w.h, lane);
      }
      if (k == w.k0) {
        if (!pr_wait(dead, p, bars + B_QEMPTY, q_ph ^ 1u, WHERE_PRODUCER)) return;
        q_ph ^= 1u;
        if (lane == 0) {
          mbar_arrive_expect_tx(bars + B_QFULL, 2u * toks * p.group * D * 2u);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
              tma_load_3d(base + P::Q + q * P::TILE + a * 16384u, &p.tmQ, bars + B_QFULL, 64 * a, w.h * p.group,
                          w.it.row0 + w.it.tok0 + q * toks);
        }
        __syncwarp();
      }
      if (E8) {
        if (!pr_wait(dead, p, bars + B_RVEMPTY, (u & 1u) ^ 1u, WHERE_PRODUCER)) return;
        load_tile<E8, D>(p, &p.tmV, base + P::RV, bars + B_RVFULL, g, tile, page, w.h, lane);
      }
    }
  }
}

// Warp 10 (16-bit caches): V.
template <int D>
__device__ void pr_load_v(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint32_t base) {
  using P = Plan<false, D>;
  const int lane = threadIdx.x & 31;
  uint32_t u = 0;
  while (w.next(p)) {
    const Pages g(p, w.it);
    int next = g.of(p, w.it, w.it.t.tile(w.k0), lane);
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const int tile = w.it.t.tile(k), page = next;
      if (k + 1 < w.k1) next = g.of(p, w.it, w.it.t.tile(k + 1), lane);
      const uint32_t st = u % PR_ST, ph = (u / PR_ST) & 1u;
      if (!pr_wait(dead, p, bars + B_VEMPTY + 8u * st, ph ^ 1u, WHERE_PRODUCER)) return;
      load_tile<false, D>(p, &p.tmV, base + P::V + st * P::TILE, bars + B_VFULL + 8u * st, g, tile, page, w.h, lane);
    }
  }
}

// ------------------------------------------------------------------ values that must not count

// The positions of an item's rows.
__device__ __forceinline__ void item_span(const PagedParams& p, const Item& it, int& p0, int& p1) {
  p0 = it.len - it.n + it.tok0;
  p1 = min(p0 + 2 * (PR_T / p.group), it.len) - 1;
}
__device__ __forceinline__ uint32_t v_piece(int key, int ch) {   // 16-byte piece of a value row in its tile
  return (ch >> 3) * 16384u + key * 128u + (((ch & 7) ^ (key & 7)) << 4);
}
template <class T>
__device__ __forceinline__ bool clear_not_finite16(uint4& w) {
  constexpr uint32_t MASK = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  bool any = false;
  uint32_t* v = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & MASK) == MASK) { v[i] &= 0xffff0000u; any = true; }
    if (((v[i] >> 16) & MASK) == MASK) { v[i] &= 0xffffu; any = true; }
  }
  return any;
}

// Warp 11 (16-bit caches): a weight of 0 times a NaN is NaN, so in a tile that not every row
// sees whole, values no row sees (past the end, before the window: whatever the slot holds) are
// cleared, and of the others what is not finite; if there was any, the item's rows that do see
// it add it when they are stored (B_ODD, one word for each of four segments in turn).
template <class T, int D>
__device__ void pr_clear(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint32_t base, uint8_t* sm,
                         volatile int* odd) {
  using P = Plan<false, D>;
  const int lane = threadIdx.x & 31;
  uint32_t u = 0;
  for (int seg = 0; w.next(p); ++seg) {
    int p0, p1;
    item_span(p, w.it, p0, p1);
    if (lane == 0) odd[(seg + 1) & 7] = 0;
    __syncwarp();
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const uint32_t st = u % PR_ST, ph = (u / PR_ST) & 1u;
      if (!pr_wait(dead, p, bars + B_VFULL + 8u * st, ph, WHERE_COPY)) return;
      const int key0 = w.it.t.tile(k) * PR_T;
      if (!all_seen(p, p0, p1, w.it.len, key0, PR_T)) {
        uint8_t* tile = sm + P::V + st * P::TILE;
        bool any = false;
        for (int i = lane; i < PR_T * (D / 8); i += 32) {
          const int key = i / (D / 8);
          uint4* at = reinterpret_cast<uint4*>(tile + v_piece(key, i - key * (D / 8)));
          if (!key_seen_by_any(p, p0, p1, w.it.len, key0 + key)) {
            *at = make_uint4(0u, 0u, 0u, 0u);
          } else {
            uint4 v = *at;
            if (clear_not_finite16<T>(v)) {
              *at = v;
              any = true;
            }
          }
        }
        if (any) odd[seg & 7] = 1;
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_VREADY + 8u * st);
    }
  }
}

// Warps 12-15 (8-bit caches): codes -> bf16 with the page's scale (a power of two: exact), K
// then V of every tile, and the clearing of warp 11.  A lane takes 16 codes of a row at a time.
template <int D>
__device__ void pr_turn(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint32_t base, uint8_t* sm,
                        volatile int* odd) {
  using P = Plan<true, D>;
  const int lane = threadIdx.x & 31, tw = (threadIdx.x >> 5) - W_TURN;
  uint32_t u = 0;
  for (int seg = 0; w.next(p); ++seg) {
    int p0, p1;
    item_span(p, w.it, p0, p1);
    if (lane == 0 && tw == 0) odd[(seg + 1) & 7] = 0;
    const int n_pages = min(p.s.max_pages, ((w.it.len - 1) >> p.c.page_log2) + 1);
    const int* table = p.s.pages + w.it.b * p.s.pages_stride;
    // lane i: the scale of keys 8 (i % 16) .. + 7 of a tile, K's for i < 16, V's above
    auto id_of = [&](int k) {
      const int lp = (w.it.t.tile(k) * PR_T + 8 * (lane & 15)) >> p.c.page_log2;
      const int id = lp < n_pages ? table[lp] : -1;
      return id < p.c.n_pages ? id : -1;
    };
    auto scale_of = [&](int id) {
      if (id < 0) return 0.f;
      return (lane < 16 ? p.c.k_scale : p.c.v_scale)[static_cast<long long>(id) * p.c.heads + w.h];
    };
    float scale = scale_of(id_of(w.k0));
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const uint32_t st = u % PR_ST, ph = (u / PR_ST) & 1u;
      const int next_id = k + 1 < w.k1 ? id_of(k + 1) : -1;
      const int key0 = w.it.t.tile(k) * PR_T;
      const bool masked = !all_seen(p, p0, p1, w.it.len, key0, PR_T);
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        if (!pr_wait(dead, p, bars + (v ? B_RVFULL : B_RKFULL), u & 1u, WHERE_COPY)) return;
        if (!pr_wait(dead, p, bars + (v ? B_VEMPTY : B_KEMPTY) + 8u * st, ph ^ 1u, WHERE_COPY)) return;
        const uint8_t* raw = sm + (v ? P::RV : P::RK);
        uint8_t* out = sm + (v ? P::V : P::K) + st * P::TILE;
        bool any = false;
        constexpr int PER = D / 16;                    // pieces of 16 codes in a row
#pragma unroll 4
        for (int i = tw * 32 + lane; i < PR_T * PER; i += 128) {
          const int key = i / PER, c = i - key * PER;
          const float f = __shfl_sync(0xffffffffu, scale, (key >> 3) + 16 * v);
          const uint4 in = *reinterpret_cast<const uint4*>(raw + key * D + 16 * c);
          const uint32_t x[4] = {in.x, in.y, in.z, in.w};
          uint32_t y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t h2;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(x[j >> 1] >> (16 * (j & 1)))));
            __half2 hv;
            memcpy(&hv, &h2, 4);
            const float2 fv = __half22float2(hv);
            y[j] = pack_bf16x2(fv.x * f, fv.y * f);
          }
          uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
          if (v && masked) {
            if (!key_seen_by_any(p, p0, p1, w.it.len, key0 + key)) {
              lo = hi = make_uint4(0u, 0u, 0u, 0u);
            } else {
              any |= clear_not_finite16<__nv_bfloat16>(lo);
              any |= clear_not_finite16<__nv_bfloat16>(hi);
            }
          }
          *reinterpret_cast<uint4*>(out + v_piece(key, 2 * c)) = lo;
          *reinterpret_cast<uint4*>(out + v_piece(key, 2 * c + 1)) = hi;
        }
        if (any) odd[seg & 7] = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bars + (v ? B_VREADY : B_KFULL) + 8u * st);
          mbar_arrive(bars + (v ? B_RVEMPTY : B_RKEMPTY));
        }
      }
      scale = scale_of(next_id);
    }
  }
}

// ------------------------------------------------------------------ MMAs (warp 9)

template <class T, bool E8, int D>
__device__ __forceinline__ void issue_s(uint32_t base, uint32_t tmem, int i, uint32_t st) {
  using P = Plan<E8, D>;
  constexpr bool HALF = std::is_same<T, __half>::value;
  const uint64_t dq = sdesc_sw128(base + P::Q + static_cast<uint32_t>(i) * P::TILE, 16u, 1024u);
  const uint64_t dk = sdesc_sw128(base + P::K + st * P::TILE, 16u, 1024u);
  if (elect_one_sync()) {
#pragma unroll
    for (int a = 0; a < D / 64; ++a)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        tc_mma_bf16(tmem + static_cast<uint32_t>(i) * PR_T, dq + ((16384u * a + 32u * k) >> 4),
                    dk + ((16384u * a + 32u * k) >> 4), idesc(PR_T, false, HALF), (a | k) ? 1u : 0u);
  }
  __syncwarp();
}
template <class T, bool E8, int D>
__device__ __forceinline__ void issue_pv(uint32_t base, uint32_t tmem, int i, uint32_t st, bool first) {
  using P = Plan<E8, D>;
  constexpr bool HALF = std::is_same<T, __half>::value;
  const uint64_t dv = sdesc_sw128(base + P::V + st * P::TILE, 16384u, 1024u);
  if (elect_one_sync()) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      tc_mma_bf16_ts(tmem + PR_O + static_cast<uint32_t>(i) * PR_T, tmem + static_cast<uint32_t>(i) * PR_T + 8u * k,
                     dv + ((2048u * k) >> 4), idesc(D, true, HALF), (!first || k) ? 1u : 0u);
  }
  __syncwarp();
}
__device__ __forceinline__ void commit(uint32_t bar) {
  if (elect_one_sync()) tc_commit(bar);
  __syncwarp();
}

template <class T, bool E8, int D>
__device__ void pr_mma(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint32_t base, uint32_t tmem) {
  uint32_t u = 0, q_ph = 0;
  bool prev_first = false, prev_last = false;
  auto value_step = [&](int i, uint32_t v) {       // O_i += P_i V of tile v, once both are there
    const uint32_t st = v % PR_ST;
    if (i == 0 && !pr_wait(dead, p, bars + B_VREADY + 8u * st, (v / PR_ST) & 1u, WHERE_MMA)) return false;
    if (!pr_wait(dead, p, bars + B_GO + 8u * i, v & 1u, WHERE_MMA)) return false;
    tc_fence_after();
    issue_pv<T, E8, D>(base, tmem, i, st, prev_first);
    if (i == 1) commit(bars + B_VEMPTY + 8u * st);
    if (prev_last) commit(bars + B_O + 8u * i);
    return true;
  };
  while (w.next(p)) {
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const uint32_t st = u % PR_ST;
      if (k == w.k0) {
        // the last products of the item before need not wait for this one's queries
        if (u > 0 && !value_step(0, u - 1)) goto done;
        if (!pr_wait(dead, p, bars + B_QFULL, q_ph, WHERE_MMA)) goto done;
        q_ph ^= 1u;
        if (!pr_wait(dead, p, bars + B_KFULL + 8u * st, (u / PR_ST) & 1u, WHERE_MMA)) goto done;
      } else {
        if (!pr_wait(dead, p, bars + B_KFULL + 8u * st, (u / PR_ST) & 1u, WHERE_MMA)) goto done;
        if (!value_step(0, u - 1)) goto done;
      }
      tc_fence_after();
      issue_s<T, E8, D>(base, tmem, 0, st);
      commit(bars + B_S);
      if (u > 0 && !value_step(1, u - 1)) goto done;
      issue_s<T, E8, D>(base, tmem, 1, st);
      commit(bars + B_S + 8u);
      commit(bars + B_KEMPTY + 8u * st);
      if (k == w.k1 - 1) commit(bars + B_QEMPTY);
      prev_first = (k == w.k0);
      prev_last = (k == w.k1 - 1);
    }
  }
  if (u > 0 && value_step(0, u - 1)) value_step(1, u - 1);
done:
  commit(bars + B_DRAIN);
  // even after giving up: nothing may run on when the tensor memory is freed
  {
    const uint64_t t0 = globaltimer_ns();
    while (!__all_sync(0xffffffffu, mbar_try_wait(bars + B_DRAIN, 0)))
      if (globaltimer_ns() - t0 > static_cast<uint64_t>(p.wait_ns)) break;
  }
}

// ------------------------------------------------------------------ softmax (warps 0-3, 4-7)

// Weights of a row from its 128 scores: 2^(c s - ref), keys outside [lo, hi) that are not below
// snk get 0 (MASK); stored as 16-bit pairs over the scores' columns.  Returns their sum; the largest
// score goes to mx.
template <class T, bool MASK>
__device__ __forceinline__ float emit(const uint32_t (&sv)[4][32], uint32_t col, float c, float ref, int lo, int hi,
                                      int snk) {
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    uint32_t w[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int k = 32 * a + 2 * q;
      float x = pg_ex2(fmaf(__uint_as_float(sv[a][2 * q]), c, -ref));
      float y = pg_ex2(fmaf(__uint_as_float(sv[a][2 * q + 1]), c, -ref));
      if (MASK) {
        x = (k < hi && (k >= lo || k < snk)) ? x : 0.f;
        y = (k + 1 < hi && (k + 1 >= lo || k + 1 < snk)) ? y : 0.f;
      }
      sum[q & 1] += x;
      sum[2 + (q & 1)] += y;
      w[q] = std::is_same<T, __half>::value ? Piece<__half>::pack(x, y) : pack_bf16x2(x, y);
    }
    tc_st_32x32b_x16(col + 16u * a, w);
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}
template <bool MASK>
__device__ __forceinline__ float largest(const uint32_t (&sv)[4][32], int lo, int hi, int snk) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int q = 0; q < 32; ++q) {
      const int k = 32 * a + q;
      if (!MASK || (k < hi && (k >= lo || k < snk))) m[q & 3] = fmaxf(m[q & 3], __uint_as_float(sv[a][q]));
    }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

template <class T, bool E8, int D>
__device__ void pr_softmax(const PagedParams& p, Walk w, const Deal& deal, volatile int* dead, uint32_t bars,
                           uint32_t tmem, volatile int* odd) {
  constexpr float SHIFT = std::is_same<T, __half>::value ? 7.f : 0.f;   // fp16 weights: 2^7 high, 2^15 at most
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp >> 2, row = 32 * (warp & 3) + lane;
  const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const uint32_t scol = tmem + lanes + static_cast<uint32_t>(g) * PR_T, ocol = scol + PR_O;
  const int toks = PR_T / p.group;
  const int my_tok = row / p.group, my_head = row - my_tok * p.group;
  const float c = p.scale_log2;
  uint32_t u = 0, o_ph = 0;
  for (int seg = 0; w.next(p); ++seg) {
    const Item& it = w.it;
    const int tok = it.tok0 + g * toks + my_tok;           // new token of this row
    const bool real = my_tok < toks && tok < it.n;
    const int pos = it.len - it.n + tok;
    const int g0 = it.len - it.n + it.tok0 + g * toks;       // positions of the tile's real rows
    const int g1 = min(g0 + toks, it.len) - 1;
    float m = -INFINITY, l = 0.f;
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const int key0 = it.t.tile(k) * PR_T;
      const bool masked = g1 >= g0 && !all_seen(p, g0, g1, it.len, key0, PR_T);
      if (!pr_wait(dead, p, bars + B_S + 8u * g, u & 1u, WHERE_EPILOGUE)) return;
      tc_fence_after();
      uint32_t sv[4][32];
#pragma unroll
      for (int a = 0; a < 4; ++a) tc_ld_32x32b_x32(scol + 32u * a, sv[a]);
      tc_wait_ld();
#pragma unroll
      for (int a = 0; a < 4; ++a) reg_fence(sv[a]);
      float factor = 1.f, sum;
      auto grow = [&](float top) {                         // moves the maximum
        const float mn = fmaxf(m, top * c);
        if (m == -INFINITY) {
          m = mn;
        } else if (mn > m + RESCALE) {
          factor = pg_ex2(m - mn);
          m = mn;
          l *= factor;
        }
      };
      if (masked) {
        int hi = PR_T, lo = 0, snk = 0;
        if (real) {
          hi = (p.causal ? min(it.len, pos + 1) : it.len) - key0;
          if (p.window > 0) {
            lo = pos - p.window + 1 - key0;
            snk = p.sinks - key0;
          }
        }
        grow(largest<true>(sv, lo, hi, snk));
        const float ref = (m == -INFINITY ? 0.f : m) - SHIFT;
        sum = emit<T, true>(sv, scol, c, ref, lo, hi, snk);
      } else {
        const float top = largest<false>(sv, 0, 0, 0);
        grow(top);
        sum = emit<T, false>(sv, scol, c, (m == -INFINITY ? 0.f : m) - SHIFT, 0, 0, 0);
      }
      l += sum;
      // S_g(u) complete implies the product of tile u-1 complete: O_g is settled until P_g(u) is published
      if (k > w.k0 && __any_sync(0xffffffffu, factor != 1.f)) {
#pragma unroll 1
        for (int a = 0; a < D / 32; ++a) {
          uint32_t v[32];
          tc_ld_32x32b_x32(ocol + 32u * a, v);
          tc_wait_ld();
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = __float_as_uint(__uint_as_float(v[q]) * factor);
          tc_st_32x32b_x32(ocol + 32u * a, v);
        }
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_GO + 8u * g);
    }
    if (!pr_wait(dead, p, bars + B_O + 8u * g, o_ph, WHERE_EPILOGUE)) return;
    o_ph ^= 1u;
    tc_fence_after();
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float lse2 = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + log2f(l) - SHIFT;
    const int head = w.h * p.group + my_head;
    const long long t = it.row0 + tok;
    const bool whole = w.k1 - w.k0 == w.count;
    const long long at = static_cast<long long>(part_slot(deal, blockIdx.x, w.u0)) * (2 * PR_T) + g * PR_T + row;
    const bool add = odd[seg & 7] != 0;
    T* dst = static_cast<T*>(p.out) + t * p.os_t + head * p.os_h;
    float* part = p.part + at * D;
#pragma unroll 1
    for (int a = 0; a < D / 32; ++a) {
      uint32_t v[32];
      __syncwarp();
      tc_ld_32x32b_x32(ocol + 32u * a, v);
      tc_wait_ld();
      if (!real) continue;
      float f[32];
#pragma unroll
      for (int q = 0; q < 32; ++q) f[q] = __uint_as_float(v[q]) * inv;
      if (add) {
        // values that were cleared because they are not finite: this row's share of them
        for (int k = w.k0; k < w.k1; ++k) {
          const int key0 = it.t.tile(k) * PR_T;
          int p0, p1;
          item_span(p, it, p0, p1);
          if (all_seen(p, p0, p1, it.len, key0, PR_T)) continue;
          for (int key = key0; key < key0 + PR_T; ++key) {
            if (!key_seen(p, pos, it.len, key)) continue;
            int page;
            const long long vr = value_row(p, it.b, w.h, key, page);
            if (vr < 0) continue;
            if (E8 && !(fabsf(p.c.v_scale[static_cast<long long>(page) * p.c.heads + w.h]) <= 3.4028235e38f)) {
#pragma unroll
              for (int q = 0; q < 32; ++q) f[q] = __int_as_float(0x7fffffff);
              continue;
            }
#pragma unroll
            for (int q = 0; q < 32; ++q) f[q] += not_finite<T, E8>(p.c.v, vr + 32 * a + q);
          }
        }
      }
      if (whole) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float (&f8)[8] = *reinterpret_cast<const float (*)[8]>(f + 8 * q);
          *reinterpret_cast<uint4*>(dst + 32 * a + 8 * q) = Piece<T>::put(f8);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<float4*>(part + 32 * a + 4 * q) = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
      }
    }
    __syncwarp();
    if (real) {
      if (!whole) p.part_lse[at] = lse2;
      else if (p.lse != nullptr) p.lse[t * p.heads_q + head] = lse2 * LN2;
    }
    tc_fence_before();
  }
}

template <class T, bool E8, int D>
__global__ void __launch_bounds__(Plan<E8, D>::THREADS, 1)
    mk_prompt_kernel(const __grid_constant__ PagedParams p, int entries) {
  using P = Plan<E8, D>;
  extern __shared__ uint8_t dyn[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dyn) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const uint32_t base = smem_u32(sm), bars = base + P::BARS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + P::BARS + B_TMEM);
  volatile int* dead = reinterpret_cast<int*>(sm + P::BARS + B_DEAD);
  volatile int* odd = reinterpret_cast<int*>(sm + P::BARS + B_ODD);
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    *dead = 0;
    for (int i = 0; i < 8; ++i) odd[i] = 0;
    mbar_init(bars + B_QFULL, 1);
    mbar_init(bars + B_QEMPTY, 1);
    for (int s = 0; s < PR_ST; ++s) {
      mbar_init(bars + B_KFULL + 8u * s, E8 ? 4 : 1);
      mbar_init(bars + B_KEMPTY + 8u * s, 1);
      mbar_init(bars + B_VFULL + 8u * s, 1);
      mbar_init(bars + B_VEMPTY + 8u * s, 1);
      mbar_init(bars + B_VREADY + 8u * s, E8 ? 4 : 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bars + B_S + 8u * g, 1);
      mbar_init(bars + B_GO + 8u * g, 4);
      mbar_init(bars + B_O + 8u * g, 1);
    }
    mbar_init(bars + B_DRAIN, 1);
    mbar_init(bars + B_RKFULL, 1);
    mbar_init(bars + B_RKEMPTY, 4);
    mbar_init(bars + B_RVFULL, 1);
    mbar_init(bars + B_RVEMPTY, 4);
    fence_mbar_init();
    tma_prefetch_map(&p.tmK);
    tma_prefetch_map(&p.tmV);
    tma_prefetch_map(&p.tmQ);
  }
  // query rows past the last whole token of a tile: never loaded, so zeros once and for all
  {
    const int used = PR_T / p.group * p.group;
    for (int i = threadIdx.x; i < 2 * (PR_T - used) * (D / 8); i += P::THREADS) {
      const int per = (PR_T - used) * (D / 8), q = i / per, j = i - q * per;
      const int r = used + j / (D / 8), ch = j % (D / 8);
      *reinterpret_cast<uint4*>(sm + P::Q + q * P::TILE + v_piece(r, ch)) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  if (warp == W_MMA) {
    tmem_alloc(smem_u32(tmem_slot), PR_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();                                          // the plan
  const Deal deal(p.prefix[entries] * p.c.heads, p.grid);
  // rows of items without a key tile see nothing: out = 0, lse = -inf
  for (int e = blockIdx.x; e < entries; e += gridDim.x) {
    if (p.prefix[e + 1] != p.prefix[e]) continue;
    const int per = 2 * (PR_T / p.group);
    const int b = warp_last_le(p.s.batch, e, [&](int i) { return p.s.cu_q[i] / per + i; });
    Item it;
    if (b >= 0 && item_of(p, e, b, it))
      no_keys<T, D>(p, it.row0 + it.tok0, min(per, it.n - it.tok0), P::THREADS);
  }
  if (static_cast<int>(blockIdx.x) < deal.c) {
    const Walk w(p, entries, deal);
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(P::MANY));
      pr_softmax<T, E8, D>(p, w, deal, dead, bars, tmem, odd);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(P::FEW));
      if (warp == W_LOAD) pr_load<E8, D>(p, w, dead, bars, base);
      else if (warp == W_MMA) pr_mma<T, E8, D>(p, w, dead, bars, base, tmem);
      else if (!E8 && warp == W_LOADV) pr_load_v<D>(p, w, dead, bars, base);
      else if (!E8 && warp == W_CLEAR) pr_clear<T, D>(p, w, dead, bars, base, sm, odd);
      else if (E8 && warp >= W_TURN) pr_turn<D>(p, w, dead, bars, base, sm, odd);
    }
    __syncwarp();
  }
  tc_fence_before();
  if (threadIdx.x == 0 && *dead) {   // loads whose barrier nobody waited for may still be landing
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 50000ull) __nanosleep(1000);
  }
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, PR_COLS);
  }
}

// ------------------------------------------------------------------ join

// Block (i, y): if CTA i's run begins inside an item that CTA i-1 began, the item's rows 16 y ..
// from the partial rows of all CTAs that worked on it.
template <class T, int D>
__global__ void __launch_bounds__(256) mk_prompt_join_kernel(const __grid_constant__ PagedParams p, int entries) {
  griddep_wait();
  const Deal deal(p.prefix[entries] * p.c.heads, p.grid);
  const int i = blockIdx.x + 1;
  if (i >= deal.c) return;
  const long long x = deal.start(i), heads = p.c.heads;
  const int e = warp_last_le(entries, 0, [&](int j) { return p.prefix[j] * heads <= x ? 0 : 1; });
  const int per = 2 * (PR_T / p.group);
  const int b = warp_last_le(p.s.batch, e, [&](int j) { return p.s.cu_q[j] / per + j; });
  Item it;
  if (e < 0 || b < 0 || !item_of(p, e, b, it)) return;
  const int count = it.t.count();
  const long long rem = x - p.prefix[e] * heads;
  const int h = static_cast<int>(rem / count);
  const long long u0 = x - (rem - static_cast<long long>(h) * count);
  if (u0 == x || deal.start(i - 1) > u0) return;
  const int r = blockIdx.y * 16 + (threadIdx.x >> 4);
  const int q = r / PR_T, rr = r - q * PR_T, toks = PR_T / p.group;
  const int tok = it.tok0 + q * toks + rr / p.group;
  if (rr / p.group >= toks || tok >= it.n) return;
  join_row<T, D, 2 * PR_T>(p, deal, i - 1, u0, count, r, it.row0 + tok, h * p.group + rr % p.group);
}

template <class T, bool E8, int D>
cudaError_t launch(const PagedParams& p, cudaStream_t s) {
  using P = Plan<E8, D>;
  static int configured_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_dev != dev) {
    e = cudaFuncSetAttribute(mk_prompt_kernel<T, E8, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM);
    if (e != cudaSuccess) return e;
    // the warps' shares come out of what the block is launched with: never ask for more
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, mk_prompt_kernel<T, E8, D>);
    if (e != cudaSuccess) return e;
    if (attr.numRegs * P::THREADS < 256 * P::MANY + (P::THREADS - 256) * P::FEW) return cudaErrorLaunchOutOfResources;
    configured_dev = dev;
  }
  const int entries = prompt_entries(p.s.tokens, p.group, p.s.batch);
  mk_prompt_plan_kernel<T><<<1, 1024, 0, s>>>(p, entries);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(P::THREADS);
  cfg.dynamicSmemBytes = P::SMEM;
  e = cudaLaunchKernelEx(&cfg, mk_prompt_kernel<T, E8, D>, p, entries);
  if (e != cudaSuccess || p.grid < 2) return e;
  cfg.gridDim = dim3(p.grid - 1, 2 * PR_T / 16);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, mk_prompt_join_kernel<T, D>, p, entries);
}

}  // namespace

int prompt_entries(int tokens, int group, int batch) { return tokens / (2 * (PR_T / group)) + batch; }
int prompt_part_rows() { return 2 * PR_T; }

cudaError_t launch_prompt(const PagedParams& p, int d, mk_dtype dtype, bool e8, cudaStream_t s) {
  if (e8) return d == 128 ? launch<__nv_bfloat16, true, 128>(p, s) : launch<__nv_bfloat16, true, 64>(p, s);
  if (dtype == MK_BF16)
    return d == 128 ? launch<__nv_bfloat16, false, 128>(p, s) : launch<__nv_bfloat16, false, 64>(p, s);
  return d == 128 ? launch<__half, false, 128>(p, s) : launch<__half, false, 64>(p, s);
}

}  // namespace mk
