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
// Items cut by a run's end leave fp32 partial rows for the join (below).
//
// Roles of a CTA's warps:
//   4-7, 8-11 softmax of query tile 0 / 1, one row a thread: the 128 scores of a
//             key tile in two halves, the weights 2^(c s - m) go back into
//             tensor memory in 16 bits, over the scores; m is the largest score of the
//             first tile and moves only when weights grow too large (then O is scaled)
//   1         loads Q and K, 2 loads V (and clears what must not count, see pr_load_v): one
//             TMA box a page and 64 columns
//   0, 3      issue the MMAs of query tile 0 / 1: O_i += P_i V of the tile before, in two halves
//             as their weights appear, then S_i = Q_i K^T.  A warp each, because the issuing
//             warp's own instructions take as long as the products they start
//   12-15     8-bit caches only: turn codes into fp16 (one conversion for two, exact; the scales
//             multiply the scores and the weights), and an item's queries, each row times a
//             power of two; warp 2 brings the scales
//
// A prompt of 8192 tokens, 32 query heads on 8, d = 128, bf16, causal: 428 us, 1.28 PFLOP/s of what
// the mask leaves (67 % of the burst rate of a plain product, 75 % of its rate under the power cap).
// The tensor pipe is busy 61 % of the time; a key tile takes the softmax warps about as long as the
// products (the exponentials alone half of that), and changing items 5 %.  Over 8-bit caches that
// chain is longer (two scales a weight; 32 scores at a time, since all sixteen warps have 128 registers)
// and the turning warps' conversions and shared memory traffic run beside it: two pieces of 1000 tokens
// after 15000 to 30000, 614 to 620 us, 1.04 PFLOP/s; the same over a bf16 cache 500 us.
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
// Changing items (queries, the first maximum, the output) takes about as long as this many tiles:
// an item's first OVER places in a run stand for that, its tiles come after them.  (The prompt
// above with 0, 1, 2, 3 places: 579, 463, 430, 432 us; six ragged windowed prompts 70, 65, 63, 64.)
constexpr int OVER = 2;
enum { W_MMA = 0, W_LOAD = 1, W_LOADV = 2, W_MMA1 = 3, W_SOFT = 4, W_TURN = 12 };

template <bool E8, int D>
struct Plan {
  static constexpr int THREADS = E8 ? 512 : 384;
  static constexpr uint32_t TILE = PR_T * D * 2;
  static constexpr uint32_t RAW = E8 ? PR_T * D : 0;      // codes as they arrive
  static constexpr uint32_t Q = 0, K = 2 * TILE, V = K + PR_ST * TILE, RK = V + PR_ST * TILE, RV = RK + RAW;
  static constexpr uint32_t BARS = RV + RAW;
  static constexpr uint32_t QEXP = BARS + 384;             // 8-bit: exponents of the query rows' factors,
  static constexpr uint32_t SCALES = QEXP + (E8 ? 512 : 0);  // by segment parity; scales of four tiles: 16 of
  static constexpr int SMEM = 1024 + SCALES + (E8 ? 512 : 0);  // keys and 16 of values, one for 8 tokens
  static_assert(SMEM <= 232448, "dynamic shared memory per block");
};
// barriers (byte offsets)
constexpr uint32_t B_QFULL = 0, B_QEMPTY = 8, B_KFULL = 16, B_KEMPTY = 32, B_VFULL = 48, B_VEMPTY = 64, B_VREADY = 80,
                   B_S = 96, B_GO = 112, B_O = 144, B_DRAIN = 160, B_RKFULL = 176, B_RKEMPTY = 184, B_RVFULL = 192,
                   B_RVEMPTY = 200, B_TURN = 208, B_TMEM = 240, B_DEAD = 244, B_ODD = 248, B_HALF = 280, B_QREADY = 296,
                   B_OTHER = 304, B_TAKEN = 312;
static_assert(B_TAKEN + 8 <= 384, "barrier block");

__device__ __forceinline__ uint32_t idesc(int n, bool b_mn, bool half) {
  return idesc_bf16_f32(PR_T, n, false, b_mn) & (half ? ~((1u << 7) | (1u << 10)) : ~0u);
}

// Waits of a whole warp, which agrees by vote.
__device__ __noinline__ bool pr_wait_loop(volatile int* dead, const PagedParams& p, uint32_t bar, uint32_t parity,
                                          int where) {
  if (__any_sync(0xffffffffu, *dead)) return false;
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
// The first look is the non-blocking test: a satisfied try_wait costs several hundred cycles.
__device__ __forceinline__ bool pr_wait(volatile int* dead, const PagedParams& p, uint32_t bar, uint32_t parity,
                                        int where) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
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
  it.n = new_tokens(p, b, it.row0);
  it.len = length_of(p, b);
  const int j = e - (it.row0 / per + b);
  if (it.n <= 0 || j < 0 || static_cast<long long>(j) * per >= it.n) return false;
  const long long rows = static_cast<long long>(it.n) * p.group;
  if (rows < p.rows_lo || rows > p.rows_hi) return false;
  it.tok0 = j * per;
  const int p0 = it.len - it.n + it.tok0;
  it.t = key_tiles<PR_T>(p, p0, min(p0 + per, it.len) - 1, it.len);
  return true;
}

// prefix[e] = places of one head in the entries before e; rows of items without tiles see nothing.
// Runs beside a decode launch before it (which has no part in this), and ends after it.
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
      if (n > 0) n += OVER;
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
  griddep_wait();
}

// A run's walk over its segments: the part of one item and head that lies in the run.
struct Walk {
  long long x, end;
  int e, entries;                            // current entry
  long long e_start, e_end;                  // its first place, the place after its last
  Item it;
  int h, k0, k1, count;
  long long u0;
  __device__ __forceinline__ Walk(const PagedParams& p, int entries_, const Deal& d) : entries(entries_) {
    x = d.start(blockIdx.x);
    end = d.start(blockIdx.x + 1);
    e = -1;
    e_start = e_end = 0;
  }
  // The segment at x (by a whole warp); false at the run's end.
  __device__ __forceinline__ bool next(const PagedParams& p) {
    const long long heads = p.c.heads;
    while (x < end) {
      if (x >= e_end) {                        // another item; else only another head of this one
        if (e < 0) e = warp_last_le(entries, 0, [&](int i) { return p.prefix[i] * heads <= x ? 0 : 1; });
        while ((e_end = p.prefix[e + 1] * heads) <= x) ++e;
        e_start = p.prefix[e] * heads;
        const int per = 2 * (PR_T / p.group);
        const int b = warp_last_le(p.s.batch, e, [&](int i) { return p.s.cu_q[i] / per + i; });
        item_of(p, e, b, it);
        count = it.t.count();
      }
      const long long rem = x - e_start;       // heads * (count + OVER) places: 32 bits but for monstrous items
      const uint32_t places = static_cast<uint32_t>(count) + OVER;
      h = (rem >> 32) == 0 ? static_cast<int>(static_cast<uint32_t>(rem) / places) : static_cast<int>(rem / places);
      const int at = static_cast<int>(rem - static_cast<long long>(h) * places);
      const int to = static_cast<int>(min(static_cast<long long>(count + OVER), at + (end - x)));
      u0 = x - at + OVER;                      // the place of the item's first tile
      k0 = max(at - OVER, 0);
      k1 = to - OVER;
      x += to - at;
      if (k1 > k0) return true;                // a run may end among an item's first places
    }
    return false;
  }
};

// A narrow item has rows for one query tile only (short sequences, ends of prompts): both query tiles are
// that one, each takes every other key tile of a segment, and the softmax warps of the first merge the two
// results.  16 sequences of 16000 tokens, 8 key heads, d = 128, 32 rows: bf16 192 us (5.5 TB/s), e4m3 196;
// with the second query tile left idle 203 and 258.
__device__ __forceinline__ bool narrow_item(const PagedParams& p, const Item& it) {
  return it.tok0 + PR_T / p.group >= it.n;
}

// The positions of an item's rows.
__device__ __forceinline__ void item_span(const PagedParams& p, const Item& it, int& p0, int& p1) {
  p0 = it.len - it.n + it.tok0;
  p1 = min(p0 + 2 * (PR_T / p.group), it.len) - 1;
}

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
    int p0, p1;
    item_span(p, it, p0, p1);
    if (keys_seen(p, p0, p1, it.len, tile * PR_T + lane * box, box)) seq_error(p.hdr, MK_ERR_INVALID, WHERE_PRODUCER, it.b);
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

// Loads begun: tiles of keys, of values, queries.
struct Loads {
  uint32_t k, v, q;
};
// Warp 1: K, and after an item's first K tile its queries; 8-bit caches: V too.
template <bool E8, int D>
__device__ void pr_load(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint32_t base, Loads& begun) {
  using P = Plan<E8, D>;
  const int lane = threadIdx.x & 31;
  const int toks = PR_T / p.group;
  const uint32_t stop = stop_at(p);
  uint32_t u = 0;
  while (w.next(p)) {
    const Pages g(p, w.it);
    int next = g.of(p, w.it, w.it.t.tile(w.k0), lane);
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const int tile = w.it.t.tile(k), page = next;
      if (k + 1 < w.k1) next = g.of(p, w.it, w.it.t.tile(k + 1), lane);
      if (u == stop) return;
      if (E8) {
        if (!pr_wait(dead, p, bars + B_RKEMPTY, (u & 1u) ^ 1u, WHERE_PRODUCER)) return;
        load_tile<E8, D>(p, &p.tmK, base + P::RK, bars + B_RKFULL, g, tile, page, w.h, lane);
      } else {
        const uint32_t st = u % PR_ST, ph = (u / PR_ST) & 1u;
        if (!pr_wait(dead, p, bars + B_KEMPTY + 8u * st, ph ^ 1u, WHERE_PRODUCER)) return;
        load_tile<E8, D>(p, &p.tmK, base + P::K + st * P::TILE, bars + B_KFULL + 8u * st, g, tile, page, w.h, lane);
      }
      ++begun.k;
      if (k == w.k0) {
        if (!pr_wait(dead, p, bars + B_QEMPTY, (begun.q & 1u) ^ 1u, WHERE_PRODUCER)) return;
        ++begun.q;
        if (lane == 0) {
          const int second = narrow_item(p, w.it) ? 0 : toks;
          mbar_arrive_expect_tx(bars + B_QFULL, 2u * toks * p.group * D * 2u);
#pragma unroll
          for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int a = 0; a < D / 64; ++a)
              tma_load_3d(base + P::Q + q * P::TILE + a * 16384u, &p.tmQ, bars + B_QFULL, 64 * a, w.h * p.group,
                          w.it.row0 + w.it.tok0 + q * second);
        }
        __syncwarp();
      }
      if (E8) {
        if (!pr_wait(dead, p, bars + B_RVEMPTY, (u & 1u) ^ 1u, WHERE_PRODUCER)) return;
        load_tile<E8, D>(p, &p.tmV, base + P::RV, bars + B_RVFULL, g, tile, page, w.h, lane);
        ++begun.v;
      }
    }
  }
}

// ------------------------------------------------------------------ values that must not count

__device__ __forceinline__ uint32_t v_piece(int key, int ch) {   // 16-byte piece of a value row in its tile
  return (ch >> 3) * 16384u + key * 128u + (((ch & 7) ^ (key & 7)) << 4);
}
template <class T>
__device__ __forceinline__ void clear_not_finite16(uint4& w) {
  constexpr uint32_t MASK = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  uint32_t* v = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((v[i] & MASK) == MASK) v[i] &= 0xffff0000u;
    if (((v[i] >> 16) & MASK) == MASK) v[i] &= 0xffffu;
  }
}

// The same question for all 8 at once: a full exponent field carries into the bit above it.
template <class T>
__device__ __forceinline__ bool has_not_finite16(const uint4& w) {
  constexpr uint32_t MASK = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
  constexpr uint32_t ONE = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
  return ((((w.x & MASK) + ONE) | ((w.y & MASK) + ONE) | ((w.z & MASK) + ONE) | ((w.w & MASK) + ONE)) & 0x80008000u) != 0u;
}

// Whether a value tile holds anything that is not finite: 0 * x summed, which is 0 otherwise; two
// instructions for 16 bytes, since nearly always there is nothing and the products wait for it.
template <class T, int D>
__device__ __forceinline__ bool any_not_finite(const uint8_t* tile, int lane) {
  using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
  T2 acc[4], zero;
  const uint32_t none = 0u;
  memcpy(&zero, &none, 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = zero;
#pragma unroll 8
  for (int i = lane; i < PR_T * (D / 8); i += 32) {
    const uint4 v = *reinterpret_cast<const uint4*>(tile + 16 * i);   // in any order
    T2 x[4];
    memcpy(x, &v, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = __hfma2(x[j], zero, acc[j]);
  }
  uint32_t bits[4];
  memcpy(bits, acc, 16);
  return __any_sync(0xffffffffu, ((bits[0] | bits[1] | bits[2] | bits[3]) & 0x7fff7fffu) != 0u);
}

// Warp 2 (16-bit caches): V.  A weight of 0 times a NaN is NaN, so in a tile that not every row
// sees whole, slots past the sequence's end (whatever they hold) and values that are not finite
// are cleared before the products may read it; if some row does see one of those, the item's rows
// that see it add it when they are stored.  B_ODD: a word for each of eight segments in turn,
// cleared one segment ahead; this warp is at most four segments ahead of the rows' last read.
template <class T, int D>
__device__ void pr_load_v(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint32_t base, uint8_t* sm,
                          volatile int* odd, Loads& begun) {
  using P = Plan<false, D>;
  const int lane = threadIdx.x & 31;
  uint32_t u = 0;
  for (int seg = 0; w.next(p); ++seg) {
    const Pages g(p, w.it);
    int p0, p1;
    item_span(p, w.it, p0, p1);
    if (lane == 0) odd[(seg + 1) & 7] = 0;
    __syncwarp();
    int next = g.of(p, w.it, w.it.t.tile(w.k0), lane);
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const int number = w.it.t.tile(k), page = next, key0 = number * PR_T;
      if (k + 1 < w.k1) next = g.of(p, w.it, w.it.t.tile(k + 1), lane);
      const uint32_t st = u % PR_ST, ph = (u / PR_ST) & 1u;
      if (!pr_wait(dead, p, bars + B_VEMPTY + 8u * st, ph ^ 1u, WHERE_PRODUCER)) return;
      load_tile<false, D>(p, &p.tmV, base + P::V + st * P::TILE, bars + B_VFULL + 8u * st, g, number, page, w.h, lane);
      ++begun.v;
      if (!all_seen(p, p0, p1, w.it.len, key0, PR_T)) {
        if (!pr_wait(dead, p, bars + B_VFULL + 8u * st, ph, WHERE_COPY)) return;
        uint8_t* tile = sm + P::V + st * P::TILE;
        for (int i = max(w.it.len - key0, 0) * (D / 8) + lane; i < PR_T * (D / 8); i += 32)   // slots without a token
          *reinterpret_cast<uint4*>(tile + v_piece(i / (D / 8), i % (D / 8))) = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();
        if (any_not_finite<T, D>(tile, lane)) {
          bool any = false;
          for (int i = lane; i < PR_T * (D / 8); i += 32) {
            const int key = i / (D / 8);
            uint4* at = reinterpret_cast<uint4*>(tile + v_piece(key, i % (D / 8)));
            uint4 v = *at;
            if (!has_not_finite16<T>(v)) continue;
            any |= key_seen_by_any(p, p0, p1, w.it.len, key0 + key);
            clear_not_finite16<T>(v);
            *at = v;
          }
          if (any) odd[seg & 7] = 1;
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(bars + B_VREADY + 8u * st);   // waited for where not every row sees the tile
    }
  }
}

__device__ __forceinline__ uint32_t codes_f16(uint32_t two_codes) {   // two e4m3 codes -> two fp16, exactly
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two_codes)));
  return h;
}

// A tile of codes to fp16, in the order the products read.  A lane takes 8 codes of a row at a time:
// eight lanes then store to eight different 16-byte columns (with 16 codes a lane, two to each).
template <int D>
struct Turn {
  static constexpr int PER = D / 8, ROWS = 128 / PER, N = PR_T / ROWS;   // lanes of a row, rows of a step, steps
  uint2 x[N];
  __device__ __forceinline__ void get(const uint8_t* in, int tw, int lane) {
    const uint8_t* from = in + (tw * (32 / PER) + lane / PER) * D + 8 * (lane % PER);
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = *reinterpret_cast<const uint2*>(from + j * ROWS * D);
  }
  // A lane of the warp, known only when get's loads have come: one that says so before, while they wait behind others,
  // would have their place filled again.
  __device__ __forceinline__ int come() const {
    uint32_t all = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) all ^= x[j].y;
    return __any_sync(0xffffffffu, all & 1u) ? 1 : 0;
  }
  __device__ __forceinline__ void put(uint8_t* out, int tw, int lane) const {
    uint8_t* to = out + v_piece(tw * (32 / PER) + lane / PER, lane % PER);
#pragma unroll
    for (int j = 0; j < N; ++j)
      *reinterpret_cast<uint4*>(to + j * ROWS * 128) = make_uint4(
          codes_f16(x[j].x & 0xffffu), codes_f16(x[j].x >> 16), codes_f16(x[j].y & 0xffffu), codes_f16(x[j].y >> 16));
  }
  // Over what put stored: 0 for keys that no row sees and for what is not finite (true if there was any).
  __device__ __forceinline__ static bool clear(const PagedParams& p, int p0, int p1, int len, int key0, uint8_t* out,
                                               int tw, int lane) {
    const int row = tw * (32 / PER) + lane / PER;
    uint8_t* to = out + v_piece(row, lane % PER);
    bool any = false;
#pragma unroll 1
    for (int j = 0; j < N; ++j) {
      uint4* at = reinterpret_cast<uint4*>(to + j * ROWS * 128);
      uint4 v = *at;
      if (!key_seen_by_any(p, p0, p1, len, key0 + row + j * ROWS)) {
        *at = make_uint4(0u, 0u, 0u, 0u);
      } else if (has_not_finite16<__half>(v)) {
        clear_not_finite16<__half>(v);
        *at = v;
        any = true;
      }
    }
    return any;
  }
};

// Warps 12-15 (8-bit caches): an item's queries, then K and V of every tile, with the clearing of
// pr_load_v.  Codes go to registers first, so that the next ones can come while these wait for room.
template <int D>
__device__ void pr_turn(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint8_t* sm, volatile int* odd) {
  using P = Plan<true, D>;
  const int lane = threadIdx.x & 31, tw = (threadIdx.x >> 5) - W_TURN;
  const int used = PR_T / p.group * p.group;               // query rows of a tile that are loaded
  uint32_t u = 0;
  for (int seg = 0; w.next(p); ++seg) {
    int p0, p1;
    item_span(p, w.it, p0, p1);
    if (lane == 0 && tw == 0) odd[(seg + 2) & 7] = 0;      // (pr_scales may be two tiles ahead)
    // queries: bf16 -> fp16 in place, the row's largest magnitude brought to 2^10 .. 2^11 (below
    // 2^-100 it stays smaller)
    if (!pr_wait(dead, p, bars + B_QFULL, seg & 1u, WHERE_COPY)) return;
    {
      constexpr int PER = D / 8, ROWS = 32 / PER;          // lanes of a row, rows of a step
      const int ch = lane % PER;
#pragma unroll 4
      for (int r0 = tw * ROWS; r0 < 2 * PR_T; r0 += 4 * ROWS) {
        const int r = r0 + lane / PER, row = r & (PR_T - 1);
        uint4* at = reinterpret_cast<uint4*>(sm + P::Q + (r / PR_T) * P::TILE + v_piece(row, ch));
        float f[8], top = 0.f;
        Piece<__nv_bfloat16>::get(*at, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
#pragma unroll
        for (int o = PER / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int ex = min(max(static_cast<int>((__float_as_uint(top) >> 23) & 255) - 127, -100), 126);
        const float up = __uint_as_float(static_cast<uint32_t>(10 - ex + 127) << 23);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= up;
        if (row < used) *at = Piece<__half>::put(f);
        if (ch == 0) reinterpret_cast<signed char*>(sm + P::QEXP)[(seg & 1) * 2 * PR_T + r] = static_cast<signed char>(ex - 10);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_QREADY);
    }
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const uint32_t st = u % PR_ST, ph = (u / PR_ST) & 1u;
      Turn<D> turn;
      // ---- K
      if (!pr_wait(dead, p, bars + B_RKFULL, u & 1u, WHERE_COPY)) return;
      turn.get(sm + P::RK, tw, lane);
      if (lane == turn.come()) mbar_arrive(bars + B_RKEMPTY);
      if (!pr_wait(dead, p, bars + B_KEMPTY + 8u * st, ph ^ 1u, WHERE_COPY)) return;
      turn.put(sm + P::K + st * P::TILE, tw, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_KFULL + 8u * st);
      // ---- V
      if (!pr_wait(dead, p, bars + B_RVFULL, u & 1u, WHERE_COPY)) return;
      turn.get(sm + P::RV, tw, lane);
      if (lane == turn.come()) mbar_arrive(bars + B_RVEMPTY);
      if (!pr_wait(dead, p, bars + B_VEMPTY + 8u * st, ph ^ 1u, WHERE_COPY)) return;
      uint8_t* out = sm + P::V + st * P::TILE;
      turn.put(out, tw, lane);
      const int key0 = w.it.t.tile(k) * PR_T;
      if (!all_seen(p, p0, p1, w.it.len, key0, PR_T) && Turn<D>::clear(p, p0, p1, w.it.len, key0, out, tw, lane))
        odd[seg & 7] = 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_VREADY + 8u * st);
    }
  }
}

// Warp 2 (8-bit caches): the scales of every tile, with its K: 16 of keys, 16 of values, one for 8
// tokens.  Those of tokens that no row sees may be anything; 1 stands in for them.
template <int D>
__device__ void pr_scales(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint8_t* sm, volatile int* odd) {
  using P = Plan<true, D>;
  const int lane = threadIdx.x & 31;
  uint32_t u = 0;
  for (int seg = 0; w.next(p); ++seg) {
    int p0, p1;
    item_span(p, w.it, p0, p1);
    const int n_pages = min(p.s.max_pages, ((w.it.len - 1) >> p.c.page_log2) + 1);
    const int* table = p.s.pages + w.it.b * p.s.pages_stride;
    auto id_of = [&](int k) {
      const int key = w.it.t.tile(k) * PR_T + 8 * (lane & 15), lp = key >> p.c.page_log2;
      if (k >= w.k1 || lp >= n_pages || !keys_seen(p, p0, p1, w.it.len, key, 8)) return -1;
      const int id = table[lp];
      return id < p.c.n_pages ? id : -1;
    };
    auto scale_of = [&](int id) {
      return id < 0 ? 1.f : (lane < 16 ? p.c.k_scale : p.c.v_scale)[static_cast<long long>(id) * p.c.heads + w.h];
    };
    float scale = scale_of(id_of(w.k0));
    int id = id_of(w.k0 + 1);
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const uint32_t st = u % PR_ST, ph = (u / PR_ST) & 1u;
      const float next = scale_of(id);
      id = id_of(k + 2);
      if (!pr_wait(dead, p, bars + B_KEMPTY + 8u * st, ph ^ 1u, WHERE_COPY)) return;
      const bool bad = lane >= 16 && !(fabsf(scale) <= 3.4028235e38f);
      if (bad) odd[seg & 7] = 1;                           // rows that see these values: NaN, when stored
      reinterpret_cast<float*>(sm + P::SCALES)[(u & 3u) * 32 + lane] = bad ? 0.f : scale;
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_KFULL + 8u * st);
      scale = next;
    }
  }
}

// ------------------------------------------------------------------ MMAs (warps 0, 3)

__device__ __forceinline__ void commit(uint32_t bar) {
  if (elect_one_sync()) tc_commit(bar);
  __syncwarp();
}

// Query tile i: for every key tile u, [V(u-1) there; first, second half of P_i(u-1) written] O_i += P_i V,
// then [K(u) there] S_i = Q_i K^T over the weights just read (the tensor pipe runs a thread's MMAs in
// order).  Stages are free once both warps' products have read them.
template <class T, bool E8, int D>
__device__ void pr_mma(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, uint32_t base, uint32_t tmem,
                       int i) {
  using P = Plan<E8, D>;
  constexpr bool HALF = std::is_same<T, __half>::value;
  const uint32_t scol = tmem + static_cast<uint32_t>(i) * PR_T, ocol = scol + PR_O;
  const uint64_t dq = sdesc_sw128(base + P::Q + static_cast<uint32_t>(i) * P::TILE, 16u, 1024u);
  const uint64_t dk0 = sdesc_sw128(base + P::K, 16u, 1024u), dv0 = sdesc_sw128(base + P::V, 16384u, 1024u);
  const uint32_t go = bars + B_GO + 16u * i;
  uint32_t u = 0, q_ph = 0;
  bool first = false, masked = false, idle = false, narrow = false;   // of the tile before
  uint32_t n = 0, turn = 0, taken = 0;                       // own tiles; tiles that took turns; narrow segments
  // The tiles take turns: PV_0(u-1), S_0(u), PV_1(u-1), S_1(u), PV_0(u), ...  So they stay half a
  // period out of step, and one's products run while the other's softmax does (left to
  // themselves they fall into step: 3800 cycles a key tile).  Each S_i(n) is handed over to the
  // other warp on barrier n % 2 of its pair; neither gets two ahead of a wait, as S_i(n+2) needs
  // the K stage that the other's S(n) has read.  An item's last products do not wait: the next
  // item's S waits for its queries.  In narrow items each warp goes its own way.
  auto handed = [&](uint32_t n) {
    return pr_wait(dead, p, bars + B_TURN + 16u * i + 8u * (n % 2), (n / 2) & 1u, WHERE_MMA);
  };
  auto arrive = [](uint32_t bar) {
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    __syncwarp();
  };
  // O_i += P_i V of the tile before, number v (idle: the other query tile's; turns: it has to wait for its turn)
  auto values = [&](uint32_t v, bool idle, bool turns) {
    const uint32_t st = v % PR_ST;
    if (!pr_wait(dead, p, bars + (E8 || masked ? B_VREADY : B_VFULL) + 8u * st, (v / PR_ST) & 1u, WHERE_MMA)) return false;
    if (idle) return true;
    const uint64_t dv = dv0 + ((P::TILE * st) >> 4);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (!pr_wait(dead, p, go + 8u * half, (n - 1) & 1u, WHERE_MMA)) return false;
      if (half == 0 && turns && !handed(turn - 1 + i)) return false;
      tc_fence_after();
      if (elect_one_sync()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_bf16_ts(ocol, scol + 32u * half + 8u * k, dv + ((8192u * half + 2048u * k) >> 4), idesc(D, true, E8 || HALF),
                         (!first || half || k) ? 1u : 0u);
      }
      __syncwarp();
      if (half == 0) commit(bars + B_HALF + 8u * i);
    }
    return true;
  };
  auto values_done = [&](uint32_t v, bool idle) {
    if (!idle) commit(bars + B_VEMPTY + 8u * (v % PR_ST));
    else arrive(bars + B_VEMPTY + 8u * (v % PR_ST));
  };
  // the last ones of a segment
  auto close = [&] {
    if (u == 0) return true;
    if (!values(u - 1, idle, false)) return false;
    values_done(u - 1, idle);
    commit(bars + B_O + 8u * i);
    return true;
  };
  auto segment = [&](auto kind) {
    constexpr bool NARROW = decltype(kind)::value;
    int p0, p1;
    item_span(p, w.it, p0, p1);
    for (int k = w.k0; k < w.k1; ++k, ++u) {
      const uint32_t st = u % PR_ST;
      const bool opens = k == w.k0, mine = !NARROW || ((k - w.k0) & 1) == i;
      if (!pr_wait(dead, p, bars + B_KFULL + 8u * st, (u / PR_ST) & 1u, WHERE_MMA)) return false;
      if (!mine) arrive(bars + B_KEMPTY + 8u * st);
      if (!opens && !values(u - 1, NARROW && mine, !NARROW)) return false;
      if (mine) {
        tc_fence_after();
        const uint64_t dk = dk0 + ((P::TILE * st) >> 4);
        if (elect_one_sync()) {
#pragma unroll
          for (int a = 0; a < D / 64; ++a)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_bf16(scol, dq + ((16384u * a + 32u * kk) >> 4), dk + ((16384u * a + 32u * kk) >> 4),
                          idesc(PR_T, false, E8 || HALF), (a | kk) ? 1u : 0u);
        }
        __syncwarp();
        commit(bars + B_S + 8u * i);
        if (!NARROW) {
          if ((threadIdx.x & 31) == 0) mbar_arrive(bars + B_TURN + 16u * (1 - i) + 8u * (turn % 2));
          ++turn;
        }
        commit(bars + B_KEMPTY + 8u * st);
        ++n;
      }
      if (!opens) values_done(u - 1, NARROW && mine);
      first = k == w.k0 + (NARROW ? i : 0);
      masked = !all_seen(p, p0, p1, w.it.len, w.it.t.tile(k) * PR_T, PR_T);
      if (NARROW) idle = !mine;
    }
    if (!NARROW) idle = false;
    commit(bars + B_QEMPTY);
    return true;
  };
  while (w.next(p)) {
    // the products before need not wait for this item's queries
    if (!close()) goto done;
    // what the second query tile's softmax left in S_1, and O_1, have been read
    if (i == 1 && narrow && !pr_wait(dead, p, bars + B_TAKEN, taken++ & 1u, WHERE_MMA)) goto done;
    if (!pr_wait(dead, p, bars + (E8 ? B_QREADY : B_QFULL), q_ph, WHERE_MMA)) goto done;
    q_ph ^= 1u;
    narrow = narrow_item(p, w.it);
    if (!(narrow ? segment(std::true_type()) : segment(std::false_type()))) goto done;
  }
  close();
done:
  commit(bars + B_DRAIN + 8u * i);
  // even after giving up: nothing may run on when the tensor memory is freed
  {
    const uint64_t t0 = globaltimer_ns();
    while (!__all_sync(0xffffffffu, mbar_try_wait(bars + B_DRAIN + 8u * i, 0)))
      if (globaltimer_ns() - t0 > DRAIN_NS) break;
  }
}

// ------------------------------------------------------------------ softmax (warps 4-7, 8-11)

// (products and sums of two fp32 values at once: mk_ptx.cuh has two, split, add2, mul2, fma2)

// The weights 2^(c s + nref) of 32 scores as 16-bit pairs; returns their sum.  8-bit caches: scales
// has those of the four groups of 8 keys, which c is multiplied by, and from 16 on those of their
// values; the weight of a value is the weight times its scale and F, summed in sum_v.  ABOVE: the scores
// went through above(), so c is 1 and the keys' scales are in them.
template <class T, bool E8, bool ABOVE = false>
__device__ __forceinline__ float weights(const uint32_t (&s)[32], uint32_t* w, float c, float nref, const float* scales,
                                         float F, float& sum_v) {
  const uint64_t nref2 = two(nref, nref);
  float total = 0.f;
  uint64_t sum[2] = {two(0.f, 0.f), two(0.f, 0.f)};
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float cg = c, vg = 1.f;
    if (E8) {
      if (!ABOVE) cg *= scales[g];
      if (cg == 0.f) cg = 1e-37f;              // a score of -infinity (masked) stays one
      vg = fminf(fmaxf(F * scales[16 + g], -3e38f), 3e38f);
    }
    const uint64_t c2 = two(cg, cg), v2 = two(vg, vg);
#pragma unroll
    for (int q = 4 * g; q < 4 * g + 4; ++q) {
      float x, y;
      split(fma2(two(__uint_as_float(s[2 * q]), __uint_as_float(s[2 * q + 1])), c2, nref2), x, y);
      x = pg_ex2(x);
      y = pg_ex2(y);
      const uint64_t xy = two(x, y);
      sum[q & 1] = E8 && q < 4 * g + 2 ? xy : add2(sum[q & 1], xy);
      if (E8) split(mul2(xy, v2), x, y);
      w[q] = E8 || std::is_same<T, __half>::value ? Piece<__half>::pack(x, y) : pack_bf16x2(x, y);
    }
    if (E8) {
      float x, y;
      split(add2(sum[0], sum[1]), x, y);
      total += x + y;
      sum_v = fmaf(x + y, fabsf(vg), sum_v);
    }
  }
  if (E8) return total;
  float s0, s1;
  split(add2(sum[0], sum[1]), s0, s1);
  return s0 + s1;
}
// Raises m to the largest of 32 scores times c and, for 8-bit caches, mv to the largest of those plus
// the logarithm of the value's scale.
template <bool E8>
__device__ __forceinline__ void largest(const uint32_t (&s)[32], float c, const float* scales, float& m, float& mv) {
  float top[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) top[g] = -INFINITY;
  if (E8) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float cg = c * scales[g];
      if (cg == 0.f) cg = 1e-37f;
#pragma unroll
      for (int q = 8 * g; q < 8 * g + 8; ++q) top[g] = fmaxf(top[g], __uint_as_float(s[q]) * cg);
      mv = fmaxf(mv, top[g] + __log2f(fabsf(scales[16 + g])));
    }
    m = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
  } else {
#pragma unroll
    for (int q = 0; q < 32; ++q) top[q & 7] = fmaxf(top[q & 7], __uint_as_float(s[q]));
#pragma unroll
    for (int g = 0; g < 4; ++g) top[g] = fmaxf(top[g], top[g + 4]);
    m = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c);
  }
}
// Bits 0 .. 31: keys 32 a .. 32 a + 31 that are below n.
__device__ __forceinline__ uint32_t below(int n, int a) {
  const int k = n - 32 * a;
  return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
}

// The keys among 32 a .. 32 a + 31 of the tile at key0 that the row at position pos sees, as bits.
__device__ __forceinline__ uint32_t seen_bits(const PagedParams& p, int pos, int len, int key0, int a) {
  uint32_t see = below((p.causal ? min(len, pos + 1) : len) - key0, a);
  // (keys before pos - window + 1, in an order that no window overflows)
  if (p.window > 0) see &= ~below(max(pos - key0 + 1, p.window) - p.window, a) | below(p.sinks - key0, a);
  return see;
}
// O of a query tile, this thread's row, times f.
template <int D>
__device__ __forceinline__ void scale_output(uint32_t ocol, float f) {
#pragma unroll 1
  for (int a = 0; a < D / 16; ++a) {
    uint32_t v[16];
    tc_ld_32x32b_x16(ocol + 16u * a, v);
    tc_wait_ld();
#pragma unroll
    for (int q = 0; q < 16; ++q) v[q] = __float_as_uint(__uint_as_float(v[q]) * f);
    tc_st_32x32b_x16(ocol + 16u * a, v);
  }
}

// Scores far from 0.  fma(s, c, -m) has in it what the rounding of m took off: 1/16 where |m| is 2^20, 64 at
// 2^31, so that the weight of the largest score itself would be far from 1, or nothing, or past every limit
// however often m moves.  From FAR on, the rest of a segment goes a slower way: m is moved to the largest
// score of every half tile first, and the products are rounded before m is taken off, as m's own was: the
// largest weight is 1 and none is larger.
constexpr float FAR = 1048576.f;             // 2^20
template <bool E8>
__device__ __forceinline__ void above(uint32_t (&s)[32], float c, const float* scales, float m) {
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float cg = c;
    if (E8) {
      cg *= scales[g];
      if (cg == 0.f) cg = 1e-37f;
    }
#pragma unroll
    for (int q = 8 * g; q < 8 * g + 8; ++q)
      s[q] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(s[q]), cg), ref));
  }
}
// A row's state inside a segment: as the loop over its tiles left it, and as far_rest does.
struct FarRow {
  float m, l, s_a, f, F;
  float vr;                                  // 8-bit: the largest log2 of a weight times its value's scale, next to m
  float c;
  uint32_t scol, ocol, u, n;
  int k, side, k0, k1, first;                // next tile and half of it; the segment's tiles, this row's first one
  int g, len, pos, g0, g1;
  KeyTiles t;
  bool real, narrow;
};
// The rest of a segment, once a row of the warp is far from 0.  (A function of its own, called outside the loop
// over tiles, after a test where m moves: with the test for every half, or the call inside, the two pieces above
// take 651 to 669 us in place of 618; without either 613.)
template <class T, bool E8, int D>
__device__ __noinline__ bool far_rest(const PagedParams& p, volatile int* dead, uint32_t bars, const uint8_t* sm,
                                      FarRow* row) {
  constexpr float SHIFT = std::is_same<T, __half>::value ? 7.f : 0.f;
  FarRow r = *row;
  tc_wait_st();                              // before a wait that may run out
  const int lane = threadIdx.x & 31;
  bool there = true;                         // the scores of tile k
#pragma unroll 1
  for (; r.k < r.k1; ++r.k, ++r.u) {
    if (r.narrow && ((r.k - r.k0) & 1) != r.g) continue;
    if (!there) {
      if (!pr_wait(dead, p, bars + B_S + 8u * r.g, r.n & 1u, WHERE_EPILOGUE)) return false;
      tc_fence_after();
    }
    there = false;
    const int key0 = r.t.tile(r.k) * PR_T;
    const bool cover = r.real && r.g1 >= r.g0 && !all_seen(p, r.g0, r.g1, r.len, key0, PR_T);
#pragma unroll 1
    for (; r.side < 2; ++r.side) {
      const float* scales =
          E8 ? reinterpret_cast<const float*>(sm + Plan<E8, D>::SCALES) + (r.u & 3u) * 32 + 8 * r.side : nullptr;
      uint32_t s[32], wt[16];
      auto get = [&](int a) {
        tc_ld_32x32b_x32(r.scol + 64u * r.side + 32u * a, s);
        tc_wait_ld_regs(s);
        if (cover) {
          const uint32_t see = seen_bits(p, r.pos, r.len, key0, 2 * r.side + a);
#pragma unroll
          for (int q = 0; q < 32; ++q)
            if (!(see & (1u << q))) s[q] = 0xff800000u;        // -inf
        }
      };
      float mn = r.m, factor = 1.f, factor_o = 1.f, none = -INFINITY;
#pragma unroll 1
      for (int a = 0; a < 2; ++a) {
        get(a);
        largest<E8>(s, r.c, E8 ? scales + 4 * a : scales, mn, none);
      }
      const float f_was = r.f;
      if (E8) {
        r.vr = r.m == -INFINITY ? -INFINITY : r.vr + (r.m - mn);
#pragma unroll 1
        for (int a = 0; a < 2; ++a) {
          get(a);
          above<E8>(s, r.c, scales + 4 * a, mn);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float top = -INFINITY;
#pragma unroll
            for (int q = 8 * g; q < 8 * g + 8; ++q) top = fmaxf(top, __uint_as_float(s[q]));
            r.vr = fmaxf(r.vr, top + __log2f(fabsf(scales[16 + 4 * a + g])));
          }
        }
        r.f = fminf(fmaxf(2.f - r.vr, -126.f), 100.f);
        r.F = pg_ex2(r.f);
      }
      if (r.l != 0.f || r.s_a != 0.f) {      // else O is nothing, or zeros
        factor = pg_ex2(r.m - mn);
        factor_o = E8 ? pg_ex2(r.m - mn + (r.f - f_was)) : factor;
      }
      r.m = mn;
      r.l *= factor;
      r.s_a *= factor;
      if ((r.side != 0 || r.k > r.first) && __any_sync(0xffffffffu, factor_o != 1.f)) {
        if (r.side != 0) {
          if (!pr_wait(dead, p, bars + B_HALF + 8u * r.g, r.n & 1u, WHERE_EPILOGUE)) return false;
          tc_fence_after();
        }
        scale_output<D>(r.ocol, factor_o);
      }
      float sum = 0.f, sum_v = 0.f;
#pragma unroll 1
      for (int a = 0; a < 2; ++a) {          // (the weights' columns are those of scores already read)
        get(a);
        above<E8>(s, r.c, E8 ? scales + 4 * a : scales, mn);
        sum += weights<T, E8, true>(s, wt, 1.f, SHIFT, E8 ? scales + 4 * a : scales, r.F, sum_v);
        tc_st_32x32b_x16(r.scol + 32u * r.side + 16u * a, wt);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + B_GO + 16u * r.g + 8u * r.side);
      if (r.side == 0) r.s_a = sum;
      else r.l += r.s_a + sum;
    }
    r.side = 0;
    ++r.n;
  }
  *row = r;
  return true;
}

// Pieces of four rows by row -> by place: lane i of four gets piece i of each of their rows.
__device__ __forceinline__ void trade4(uint4 (&c)[4], int lane) {
  auto swap = [&](uint4& lo, uint4& hi, int bit) {
    const bool up = lane & bit;
    const uint4 give = up ? lo : hi;
    uint4 got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, bit);
    got.y = __shfl_xor_sync(0xffffffffu, give.y, bit);
    got.z = __shfl_xor_sync(0xffffffffu, give.z, bit);
    got.w = __shfl_xor_sync(0xffffffffu, give.w, bit);
    if (up) lo = got;
    else hi = got;
  };
  swap(c[0], c[1], 1);
  swap(c[2], c[3], 1);
  swap(c[0], c[2], 2);
  swap(c[1], c[3], 2);
}

// This row's share of values that were cleared because they are not finite (elements d0 ..).
template <class T, bool E8>
__device__ __forceinline__ void add_not_finite(const PagedParams& p, const Walk& w, int pos, int d0, float (&f)[32]) {
  int p0, p1;
  item_span(p, w.it, p0, p1);
  for (int k = w.k0; k < w.k1; ++k) {
    const int key0 = w.it.t.tile(k) * PR_T;
    if (!E8 && all_seen(p, p0, p1, w.it.len, key0, PR_T)) continue;   // (8-bit: scales, of any tile)
    for (int key = key0; key < key0 + PR_T; ++key) {
      if (!key_seen(p, pos, w.it.len, key)) continue;
      int page;
      const long long vr = value_row(p, w.it.b, w.h, key, page);
      if (vr < 0) continue;
      if (E8 && !(fabsf(p.c.v_scale[static_cast<long long>(page) * p.c.heads + w.h]) <= 3.4028235e38f)) {
#pragma unroll
        for (int q = 0; q < 32; ++q) f[q] = __int_as_float(0x7fffffff);
        continue;
      }
#pragma unroll
      for (int q = 0; q < 32; ++q) f[q] += not_finite<T, E8>(p.c.v, vr + d0 + q);
    }
  }
}

// For 8-bit caches (128 registers) not inlined, so that the walk's state stays out of the registers of the
// loop over tiles: the two pieces above 614 us instead of 639; with 16-bit ones the prompt takes 456
// us that way, not 430.
__device__ __noinline__ bool next_apart(const PagedParams& p, Walk* w) { return w->next(p); }
template <bool E8>
__device__ __forceinline__ bool next_segment(const PagedParams& p, Walk& w) {
  if constexpr (E8) return next_apart(p, &w);
  else return w.next(p);
}

template <class T, bool E8, int D>
__device__ void pr_softmax(const PagedParams& p, Walk w, volatile int* dead, uint32_t bars, const uint8_t* sm,
                           uint32_t tmem, volatile int* odd) {
  // fp16 weights are taken 2^7 high, so that small ones keep their bits, and stay below 2^15
  constexpr bool HALF = std::is_same<T, __half>::value;
  constexpr float SHIFT = HALF ? 7.f : 0.f, LIMIT = HALF ? 32768.f : 1.152921504606847e18f;   // 2^15, 2^60
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = (warp - W_SOFT) >> 2, row = 32 * (warp & 3) + lane;
  const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
  const uint32_t scol = tmem + lanes + static_cast<uint32_t>(g) * PR_T, ocol = scol + PR_O;
  const int toks = PR_T / p.group;
  const int my_tok = row / p.group, my_head = row - my_tok * p.group;
  float c = p.scale_log2;
  uint32_t u = 0, n = 0, o_ph = 0, others = 0;             // tiles, own tiles, segments, narrow ones
  const long long begin = w.x;
  if (threadIdx.x == 32 * W_SOFT) p.cut[blockIdx.x].u0 = -1;
  for (int seg = 0; next_segment<E8>(p, w); ++seg) {
    if (seg == 0 && threadIdx.x == 32 * W_SOFT && w.u0 < begin)
      p.cut[blockIdx.x] = CutUnit{w.u0, w.count, w.it.row0, w.it.n, w.h, w.it.tok0};
    const typename std::conditional<E8, Item, Item&>::type it = w.it;
    const int k0 = w.k0, k1 = w.k1;
    const bool narrow = narrow_item(p, it);
    const int tok = it.tok0 + (narrow ? 0 : g * toks) + my_tok;   // new token of this row
    const bool real = my_tok < toks && tok < it.n;
    const int pos = it.len - it.n + tok;
    const int g0 = it.len - it.n + it.tok0 + (narrow ? 0 : g * toks);   // positions of the tile's real rows
    const int g1 = min(g0 + toks, it.len) - 1;
    float m = -INFINITY, l = 0.f;
    // 8-bit caches: a weight meets its value's code as fp16(weight x scale x F), F = 2^f; f brings
    // the largest so far (mv, its logarithm) to 2^2, and moves like m, on its own.  (At most 100, so
    // that its product with a scale below 2^27 is finite, and scales from 2^-100 on keep their bits.)
    float mv = -INFINITY, f = 0.f, F = 1.f;
    bool ready = false;                                    // every row of the warp has a reference
    const int k_first = k0 + (narrow ? g : 0);
    int k = k0, from = 0;                                  // from: the half to go on with
    float s_a = 0.f;                                       // the first half's sum
    for (; k < k1; ++k, ++u) {
      const int key0 = it.t.tile(k) * PR_T;
      const bool masked = g1 >= g0 && !all_seen(p, g0, g1, it.len, key0, PR_T);
      if (narrow && ((k - k0) & 1) != g) continue;
      if (!pr_wait(dead, p, bars + B_S + 8u * g, n & 1u, WHERE_EPILOGUE)) return;
      tc_fence_after();
      if (E8 && k == k_first) {
        const int ex = reinterpret_cast<const signed char*>(sm + Plan<E8, D>::QEXP)[(seg & 1) * 2 * PR_T + g * PR_T + row];
        c = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
      }
      // Half the row at a time, its weights handed over once written: the products start on the
      // first while the second is being computed.  (One copy of this code for both halves, 64
      // scores in registers: with the whole row unrolled the instructions did not come fast enough.)
      s_a = 0.f;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const float* scales = E8 ? reinterpret_cast<const float*>(sm + Plan<E8, D>::SCALES) + (u & 3u) * 32 + 8 * half : nullptr;
        // 16-bit caches hold the half's 64 scores; with 8-bit ones there are four more warps and
        // fewer registers: 32 scores at a time, read again when the reference moves (64: spills; 16,
        // the next on their way: 767 us where 32 take 645)
        constexpr int HELD = E8 ? 1 : 2;
        uint32_t sv[HELD][32], wt[32];
        auto fetch = [&](int a) {
          uint32_t (&s)[32] = sv[a & (HELD - 1)];
          tc_ld_32x32b_x32(scol + 64u * half + 32u * a, s);
        };
        auto cover = [&](int a) {
          uint32_t (&s)[32] = sv[a & (HELD - 1)];
          if (masked && real) {
            const uint32_t see = seen_bits(p, pos, it.len, key0, 2 * half + a);
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (!(see & (1u << q))) s[q] = 0xff800000u;          // -inf
          }
        };
        if (!E8) {
          fetch(0);
          fetch(1);
          tc_wait_ld_regs(sv[0]);
          reg_fence(sv[HELD - 1]);
          cover(0);
          cover(1);
        }
        auto scores = [&](int a) -> const uint32_t (&)[32] {
          if (E8) {
            fetch(a);
            tc_wait_ld_regs(sv[0]);
            cover(a);
          }
          return sv[a & (HELD - 1)];
        };
        // No maximum is taken of a tile: the reference m, the largest of the first scores, stands as
        // long as no sum of weights passes LIMIT, which bounds each weight too.  Once m has moved (and is
        // not FAR from 0) no sum of this half can: two passes at most.
        bool move = !ready;
        float sum;
        while (true) {
          if (move) {
            // m to the largest score so far, and what has been summed along with it.  O_g is settled
            // before P_g(u) is handed over, since S_g(u) complete implies the product of tile u-1
            // is; after the first half has been, once that half's product is complete.
            float mn = m;
            largest<E8>(scores(0), c, scales, mn, mv);
            largest<E8>(scores(1), c, E8 ? scales + 4 : scales, mn, mv);
            float factor = 1.f, factor_o = 1.f;
            const float f_was = f;
            if (E8) f = fminf(fmaxf(mn - mv + 2.f, -126.f), 100.f);
            if (mn > m || (E8 && f != f_was)) {
              if (m != -INFINITY) {
                factor = pg_ex2(m - mn);
                factor_o = E8 ? pg_ex2(m - mn + f - f_was) : factor;
              }
              m = mn;
            }
            if (E8) F = pg_ex2(f);
            l *= factor;
            s_a *= factor;
            ready = __all_sync(0xffffffffu, fabsf(m) < FAR);
            if ((half != 0 || k > k_first) && __any_sync(0xffffffffu, factor_o != 1.f)) {
              if (half != 0) {
                if (!pr_wait(dead, p, bars + B_HALF + 8u * g, n & 1u, WHERE_EPILOGUE)) return;
                tc_fence_after();
              }
              scale_output<D>(ocol, factor_o);
            }
            if (!ready) {                                  // nothing seen yet, or far from 0
              ready = __all_sync(0xffffffffu, m != -INFINITY);
              if (__builtin_expect(__any_sync(0xffffffffu, fabsf(m) >= FAR && m != -INFINITY), 0)) {
                from = half;
                goto far;
              }
            }
          }
          const float nref = SHIFT - (m == -INFINITY ? 0.f : m);
          float sum_v = 0.f;
          sum = weights<T, E8>(scores(0), wt, c, nref, scales, F, sum_v);
          sum += weights<T, E8>(scores(1), wt + 16, c, nref, E8 ? scales + 4 : scales, F, sum_v);
          move = __any_sync(0xffffffffu, sum > LIMIT || (E8 && sum_v > 32768.f));
          if (!move) break;
        }
        tc_st_32x32b_x32(scol + 32u * half, wt);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + B_GO + 16u * g + 8u * half);
        if (half == 0) s_a = sum;
        else l += s_a + sum;
      }
      ++n;
    }
    if (false) {
    far:                                                   // the rest of the segment, from tile k on
      FarRow r = {m, l, s_a, f, F, l == 0.f && s_a == 0.f ? -INFINITY : 2.f - f, c, scol, ocol, u, n, k, from, k0, k1,
                  k_first, g, it.len, pos, g0, g1, it.t, real, narrow};
      if (!far_rest<T, E8, D>(p, dead, bars, sm, &r)) return;
      m = r.m;
      l = r.l;
      f = r.f;
      u += k1 - k;                                         // (counted here: the same for every thread)
      n += narrow ? (k1 - k + 1) >> 1 : k1 - k;
    }
    if (!pr_wait(dead, p, bars + B_O + 8u * g, o_ph, WHERE_EPILOGUE)) return;
    o_ph ^= 1u;
    tc_fence_after();
    float mul = E8 ? pg_ex2(-f) : 1.f, mul_other = 0.f;
    const bool other = narrow && w.k1 - w.k0 > 1;          // the second query tile had a key tile
    if (narrow) {
      // maximum, sum and factor of the second tile's rows go through S_1, which no product reads any more
      // and none writes before B_TAKEN
      uint32_t x[16];
      if (g == 1) {
        x[0] = __float_as_uint(m);
        x[1] = __float_as_uint(l);
        x[2] = __float_as_uint(f);
#pragma unroll
        for (int q = 3; q < 16; ++q) x[q] = 0u;
        tc_st_32x32b_x16(scol, x);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + B_OTHER);
        continue;
      }
      if (!pr_wait(dead, p, bars + B_OTHER, others++ & 1u, WHERE_EPILOGUE)) return;
      tc_fence_after();
      if (other) {
        tc_ld_32x32b_x16(scol + PR_T, x);
        tc_wait_ld();
        const float m1 = __uint_as_float(x[0]), top = fmaxf(m, m1), ref = top == -INFINITY ? 0.f : top;
        const float a0 = pg_ex2(m - ref), a1 = pg_ex2(m1 - ref);
        l = l * a0 + __uint_as_float(x[1]) * a1;
        mul *= a0;
        mul_other = E8 ? pg_ex2(-__uint_as_float(x[2])) * a1 : a1;
        m = top;
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float lse2 = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m) + log2f(l) - SHIFT;
    const int head = w.h * p.group + my_head;
    const long long t = it.row0 + tok;
    const bool whole = w.k1 - w.k0 == w.count;
    const long long at = static_cast<long long>(part_slot(blockIdx.x, w.k0 == 0)) * (2 * PR_T) + g * PR_T + row;
    const bool add = odd[seg & 7] != 0;
    // 32 columns at a time; four lanes trade 16-byte pieces so that a store instruction covers 64
    // neighbouring bytes of 8 rows, not 16 of 32
    uint8_t* mine = whole ? reinterpret_cast<uint8_t*>(static_cast<T*>(p.out) + t * p.os_t + head * p.os_h)
                          : reinterpret_cast<uint8_t*>(p.part + at * D);
    uint8_t* to[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned long long a = real ? reinterpret_cast<unsigned long long>(mine) : 0ull;
      to[j] = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, a, (lane & ~3) + j));
    }
    const uint32_t piece = 16u * (lane & 3);
#pragma unroll 1
    for (int a = 0; a < D / 32; ++a) {
      uint32_t v[32];
      __syncwarp();
      tc_ld_32x32b_x32(ocol + 32u * a, v);
      tc_wait_ld();
      float f[32];
#pragma unroll
      for (int q = 0; q < 32; ++q) f[q] = __uint_as_float(v[q]) * mul;
      if (other) {
        __syncwarp();
        tc_ld_32x32b_x32(ocol + PR_T + 32u * a, v);
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 32; ++q) f[q] = fmaf(__uint_as_float(v[q]), mul_other, f[q]);
      }
#pragma unroll
      for (int q = 0; q < 32; ++q) f[q] *= inv;
      if (add && real) add_not_finite<T, E8>(p, w, pos, 32 * a, f);
      __syncwarp();
      uint4 out[4];
      if (whole) {
#pragma unroll
        for (int j = 0; j < 4; ++j) out[j] = Piece<T>::put(*reinterpret_cast<const float (*)[8]>(f + 8 * j));
        trade4(out, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (to[j] != nullptr) *reinterpret_cast<uint4*>(to[j] + 64 * a + piece) = out[j];
      } else {
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
#pragma unroll
          for (int j = 0; j < 4; ++j) out[j] = Piece<float>::put(*reinterpret_cast<const float (*)[4]>(f + 16 * h2 + 4 * j));
          trade4(out, lane);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (to[j] != nullptr) *reinterpret_cast<uint4*>(to[j] + 128 * a + 64 * h2 + piece) = out[j];
        }
      }
    }
    __syncwarp();
    if (real) {
      if (!whole) p.part_lse[at] = lse2;
      else if (p.lse != nullptr) p.lse[t * p.heads_q + head] = lse2 * LN2;
    }
    tc_fence_before();
    __syncwarp();
    if (narrow && lane == 0) mbar_arrive(bars + B_TAKEN);
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
    mbar_init(bars + B_QREADY, 4);
    mbar_init(bars + B_QEMPTY, 2);                          // both query tiles' MMA warps
    for (int s = 0; s < PR_ST; ++s) {
      mbar_init(bars + B_KFULL + 8u * s, E8 ? 5 : 1);          // 8-bit: the turning warps, the scales
      mbar_init(bars + B_KEMPTY + 8u * s, 2);
      mbar_init(bars + B_VFULL + 8u * s, 1);
      mbar_init(bars + B_VEMPTY + 8u * s, 2);
      mbar_init(bars + B_VREADY + 8u * s, E8 ? 4 : 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(bars + B_S + 8u * g, 1);
      mbar_init(bars + B_GO + 16u * g, 4);
      mbar_init(bars + B_GO + 16u * g + 8u, 4);
      mbar_init(bars + B_O + 8u * g, 1);
      mbar_init(bars + B_HALF + 8u * g, 1);
      mbar_init(bars + B_DRAIN + 8u * g, 1);
    }
    for (int s = 0; s < 4; ++s) mbar_init(bars + B_TURN + 8u * s, 1);
    mbar_init(bars + B_OTHER, 4);
    mbar_init(bars + B_TAKEN, 4);
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
      no_keys<T, D>(p, b, it.row0 + it.tok0, min(per, it.n - it.tok0), P::THREADS);
  }
  if (static_cast<int>(blockIdx.x) < deal.c) {
    const Walk w(p, entries, deal);
    if (warp >= W_SOFT && warp < W_SOFT + 8) {
      pr_softmax<T, E8, D>(p, w, dead, bars, sm, tmem, odd);
    } else {
      if (warp == W_LOAD) {
        Loads begun = {0, 0, 0};
        pr_load<E8, D>(p, w, dead, bars, base, begun);
        __syncwarp();
        pg_drain(p, bars + (E8 ? B_RKFULL : B_KFULL), E8 ? 1 : PR_ST, begun.k);
        pg_drain(p, bars + B_QFULL, 1, begun.q);
        pg_drain(p, bars + B_RVFULL, 1, begun.v);
      }
      else if (warp == W_MMA || warp == W_MMA1)
        pr_mma<T, E8, D>(p, w, dead, bars, base, tmem, warp == W_MMA1);
      else if (!E8 && warp == W_LOADV) {
        Loads begun = {0, 0, 0};
        pr_load_v<T, D>(p, w, dead, bars, base, sm, odd, begun);
        __syncwarp();
        pg_drain(p, bars + B_VFULL, PR_ST, begun.v);
      }
      else if (E8 && warp == W_LOADV) pr_scales<D>(p, w, dead, bars, sm, odd);
      else if (E8 && warp >= W_TURN) pr_turn<D>(p, w, dead, bars, sm, odd);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, PR_COLS);
  }
}

// ------------------------------------------------------------------ join

// Block (i - 1, y): if CTA i's run begins inside an item that CTA i-1 began, an eighth of the item's
// rows from the partial rows of all CTAs that worked on it.  (Blocks of an item: 4, 8, 16: ragged
// windowed prompts 65.6, 62.9, 63.5 us.  The last CTA to be done could join an item alone, as in decode
// steps, but 256 rows of many CTAs take one SM longer than the launch.)
constexpr int JOIN_Y = 8;
template <class T, int D>
__global__ void __launch_bounds__(256) mk_prompt_join_kernel(const __grid_constant__ PagedParams p, int entries) {
  griddep_wait();
  const int i = blockIdx.x + 1;
  const CutUnit g = p.cut[i];
  const Deal deal(p.prefix[entries] * p.c.heads, p.grid);
  if (i >= deal.c || g.u0 < 0 || deal.start(i - 1) > g.u0) return;
  const int toks = PR_T / p.group, c1 = deal.owner(g.u0 + g.count - 1);
  for (int r = blockIdx.y * 16 + (threadIdx.x >> 4); r < 2 * PR_T; r += 16 * JOIN_Y) {
    const int q = r / PR_T, rr = r - q * PR_T, tok = g.at + q * toks + rr / p.group;
    if (rr / p.group >= toks || tok >= g.n) continue;
    join_row<T, D, 2 * PR_T>(p, i - 1, c1, r, g.row0 + tok, g.h * p.group + rr % p.group);
  }
}

template <class T, bool E8, int D>
cudaError_t launch(const PagedParams& p, bool after_decode, cudaStream_t s) {
  using P = Plan<E8, D>;
  static int configured_dev = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_dev != dev) {
    e = cudaFuncSetAttribute(mk_prompt_kernel<T, E8, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM);
    if (e != cudaSuccess) return e;
    configured_dev = dev;
  }
  const int entries = prompt_entries(p.s.tokens, p.group, p.s.batch);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after_decode ? 1 : 0;
  cfg.stream = s;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  e = cudaLaunchKernelEx(&cfg, mk_prompt_plan_kernel<T>, p, entries);
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(P::THREADS);
  cfg.dynamicSmemBytes = P::SMEM;
  e = cudaLaunchKernelEx(&cfg, mk_prompt_kernel<T, E8, D>, p, entries);
  if (e != cudaSuccess || p.grid < 2) return e;
  cfg.gridDim = dim3(p.grid - 1, JOIN_Y);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, mk_prompt_join_kernel<T, D>, p, entries);
}

}  // namespace

int prompt_entries(int tokens, int group, int batch) { return tokens / (2 * (PR_T / group)) + batch; }
int prompt_part_rows() { return 2 * PR_T; }

cudaError_t launch_prompt(const PagedParams& p, int d, mk_dtype dtype, bool e8, bool after_decode, cudaStream_t s) {
  const auto f = e8 ? (d == 128 ? launch<__nv_bfloat16, true, 128> : launch<__nv_bfloat16, true, 64>)
                 : dtype == MK_BF16 ? (d == 128 ? launch<__nv_bfloat16, false, 128> : launch<__nv_bfloat16, false, 64>)
                                    : (d == 128 ? launch<__half, false, 128> : launch<__half, false, 64>);
  return f(p, after_decode, s);
}

}  // namespace mk
