// mk_paged.h -- what the two attention kernels over a paged cache share: the
// call, which keys a sequence's rows see, how tiles are dealt to CTAs, the
// partial results and their join.
#pragma once

#include <type_traits>

#include "mk_seq.cuh"

namespace mk {

// What a CTA of the prompt kernel leaves for the join: the item that its run begins inside of, u0 = -1
// if there is none.
struct CutUnit {
  long long u0;                        // place of the item's first tile
  int count;                           // its tiles
  int row0, n, h;                      // its sequence's first token row and new tokens; key head
  int at;                              // its first token
};

struct PagedParams {
  CUtensorMap tmK, tmV, tmQ;
  const void* q;
  void* out;
  float* lse;                          // [tokens x heads_q] or null
  long long qs_t, qs_h, os_t, os_h;    // element strides
  SeqView s;
  CacheView c;
  uint32_t* hdr;
  float* part;                         // partial rows: o [slot][row][d], then their log2 sums
  float* part_lse;
  uint32_t* turn;                      // decode: CTAs that are done with the unit begun by each CTA; 0 between calls
  CutUnit* cut;                        // prompts: one for each CTA
  long long* prefix;                   // prompts: places of one head before each item
  long long wait_ns;
  float scale_log2;                    // softmax scale * log2(e)
  int heads_q, group;                  // query heads; of them per key head
  int causal, window, sinks;
  int len_max;                         // tokens that the page table has room for
  int map_pages;                       // pages in the tensor maps; a load from this page reads zeros
  int rows_lo, rows_hi;                // sequences with this many packed rows (tokens x group) are this launch's
  int grid;
  int inject;                          // test only: 1 = the first CTA's loader stops after two tiles
};

// The keys a sequence's rows see, in tiles of KT keys: tiles 0 .. sink-1 (the
// first tokens that stay visible) and tiles from .. end-1.
struct KeyTiles {
  int sink, from, end;
  __device__ __forceinline__ int count() const { return sink + end - from; }
  __device__ __forceinline__ int tile(int k) const { return k < sink ? k : k - sink + from; }
};
// Rows at positions p0 .. p1 of a sequence of len tokens.
template <int KT>
__device__ __forceinline__ KeyTiles key_tiles(const PagedParams& p, int p0, int p1, int len) {
  KeyTiles t;
  const int end = p.causal ? min(len, p1 + 1) : len;
  t.end = end > 0 ? (end + KT - 1) / KT : 0;
  t.sink = t.from = 0;
  if (p.window > 0 && p0 >= p.window) {
    t.from = min((p0 - p.window + 1) / KT, t.end);
    t.sink = min((min(p.sinks, len) + KT - 1) / KT, t.from);
    if (t.sink == t.from) t.sink = t.from = 0;
  }
  return t;
}
// Whether every row at positions p0 .. p1 sees every one of keys k0 .. k0+n-1.
__device__ __forceinline__ bool all_seen(const PagedParams& p, int p0, int p1, int len, int k0, int n) {
  if (k0 + n > (p.causal ? min(len, p0 + 1) : len)) return false;
  return p.window == 0 || p1 - k0 < p.window || k0 + n <= p.sinks;
}
__device__ __forceinline__ bool key_seen(const PagedParams& p, int pos, int len, int key) {
  return key < len && (!p.causal || key <= pos) && (p.window == 0 || pos - key < p.window || key < p.sinks);
}
// Whether any of the rows at positions p0 .. p1 sees the key.
__device__ __forceinline__ bool key_seen_by_any(const PagedParams& p, int p0, int p1, int len, int key) {
  return key < len && (!p.causal || key <= p1) && (p.window == 0 || p0 - key < p.window || key < p.sinks);
}

// Whether any of the rows at positions p0 .. p1 sees any of keys key .. key+n-1.
__device__ __forceinline__ bool keys_seen(const PagedParams& p, int p0, int p1, int len, int key, int n) {
  const int end = p.causal ? min(len, p1 + 1) : len;
  return key < end && (p.window == 0 || p0 - (key + n - 1) < p.window || key < p.sinks);
}

// N tiles dealt to C = min(grid, N) CTAs in runs that differ by at most one
// tile; a unit (the tiles of one set of rows) may be cut by several runs.
struct Deal {
  long long n;
  int c;
  __device__ __forceinline__ Deal(long long total, int grid) : n(total), c(total < grid ? static_cast<int>(total) : grid) {}
  __device__ __forceinline__ long long start(int i) const { return n * i / c; }
  __device__ __forceinline__ int owner(long long x) const { return static_cast<int>(((x + 1) * c + n - 1) / n) - 1; }
};
// Where CTA i leaves its partial result of a unit: one place for a unit begun by an earlier
// CTA, one for a unit that it begins and does not finish.
__device__ __forceinline__ int part_slot(int i, bool begins) { return 2 * i + (begins ? 1 : 0); }

// ------------------------------------------------------------------ bounded waits
// No CTA of these kernels waits for another, so giving up is a CTA's own
// affair: a word in shared memory, after which every wait returns at once.  What is
// in flight then (loads, products) is still waited for, by the warp that issued it.
constexpr uint64_t DRAIN_NS = 1000000000ull;
__device__ __forceinline__ bool pg_wait_slow(volatile int* dead, const PagedParams& p, uint32_t bar, uint32_t parity,
                                             int where) {
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
__device__ __noinline__ bool pg_wait_loop(volatile int* dead, const PagedParams& p, uint32_t bar, uint32_t parity,
                                          int where);
__device__ __forceinline__ bool pg_wait(volatile int* dead, const PagedParams& p, uint32_t bar, uint32_t parity,
                                        int where) {
  if (mbar_try_wait(bar, parity)) return true;
  return pg_wait_loop(dead, p, bar, parity, where);
}

// The tile before which a CTA's loader stops (compared for every tile: worked out there, decode steps took 1 % more).
__device__ __forceinline__ uint32_t stop_at(const PagedParams& p) {
  return p.inject == 1 && blockIdx.x == 0 ? 2u : 0xffffffffu;
}

// The last `stages` of `count` loads that a warp issued, load i on barrier bar + 8 (i % stages): each is its barrier's
// latest phase, so that its parity cannot be mistaken.
__device__ __forceinline__ void pg_drain(const PagedParams& p, uint32_t bar, uint32_t stages, uint32_t count) {
  for (uint32_t i = count > stages ? count - stages : 0u; i < count; ++i) {
    const uint32_t at = bar + 8u * (i % stages), parity = (i / stages) & 1u;
    if (mbar_try_wait(at, parity)) continue;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(at, parity))
      if (globaltimer_ns() - t0 > DRAIN_NS) {
        seq_error(p.hdr, MK_ERR_TIMEOUT, WHERE_PRODUCER, blockIdx.x);
        return;
      }
  }
}

__device__ __forceinline__ float pg_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float LN2 = 0.69314718055994530942f;

// ------------------------------------------------------------------ rows and values

// A sequence's tokens; a length that the page table has no room for counts as none, so that no work or index
// comes of it.
__device__ __forceinline__ int length_of(const PagedParams& p, int b) {
  const int len = p.s.kv_len[b];
  return len > 0 && len <= p.len_max ? len : 0;
}
// Its new tokens: rows of the call's arrays, whatever cu_q holds.
__device__ __forceinline__ int new_tokens(const PagedParams& p, int b, int& row0) {
  row0 = p.s.cu_q[b];
  return row0 < 0 ? 0 : max(min(p.s.cu_q[b + 1], p.s.tokens), 0) - row0;
}
__device__ __forceinline__ bool sequence_of(const PagedParams& p, int b, int& n, int& len, int& row0) {
  n = new_tokens(p, b, row0);
  len = length_of(p, b);
  return n > 0;
}
__device__ __forceinline__ bool rows_are_ours(const PagedParams& p, int n) {
  const long long rows = static_cast<long long>(n) * p.group;
  return rows >= p.rows_lo && rows <= p.rows_hi;
}
// The rows of n tokens from row0, of sequence b, see nothing: out = 0, lse = -inf (by a whole block).
template <class T, int D>
__device__ __forceinline__ void no_keys(const PagedParams& p, int b, int row0, int n, int threads) {
  if (threadIdx.x == 0 && p.s.kv_len[b] > p.len_max) seq_error(p.hdr, MK_ERR_CAPACITY, WHERE_PRODUCER, b);
  const long long pieces = static_cast<long long>(n) * p.heads_q * (D / 8);
  for (long long i = threadIdx.x; i < pieces; i += threads) {
    const long long r = i / (D / 8);
    const long long t = row0 + r / p.heads_q;
    const int head = static_cast<int>(r % p.heads_q), piece = static_cast<int>(i % (D / 8));
    *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + t * p.os_t + head * p.os_h + piece * 8) =
        make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr && piece == 0) p.lse[t * p.heads_q + head] = -INFINITY;
  }
}
// Element offset of the value row of a sequence's token `key`, -1 where its page is not in the cache.
__device__ __forceinline__ long long value_row(const PagedParams& p, int b, int h, int key, int& page) {
  const int lp = key >> p.c.page_log2;
  if (lp >= p.s.max_pages) return -1;
  const int id = page = p.s.pages[b * p.s.pages_stride + lp];
  if (id < 0 || id >= p.c.n_pages) return -1;
  return id * p.c.page_stride + h * p.c.head_stride + (key & (p.c.page_size - 1)) * p.c.slot_stride;
}
// The value at an offset if it is NaN or infinite, else 0.
template <class T, bool E8>
__device__ __forceinline__ float not_finite(const void* v, long long at) {
  if (E8) return (static_cast<const uint8_t*>(v)[at] & 0x7f) == 0x7f ? __int_as_float(0x7fffffff) : 0.f;
  const float x = Piece<T>::one(static_cast<const T*>(v)[at]);
  return fabsf(x) <= 3.4028235e38f ? 0.f : x;
}

// Row r of a unit of ROWS rows: the partial rows of CTAs c0 .. c1 in order, weighted by 2^(lse - max),
// into out[t][head].  16 threads a row, D / 16 elements each.
template <class T, int D, int ROWS>
__device__ __forceinline__ void join_row(const PagedParams& p, int c0, int c1, int r, long long t, int head) {
  constexpr int EL = D / 16;
  const int lane = threadIdx.x & 15, d0 = lane * EL;
  const unsigned mask = 0xffffu << (threadIdx.x & 16);
  float top = -INFINITY;
  for (int i = c0 + lane; i <= c1; i += 16)
    top = fmaxf(top, p.part_lse[static_cast<long long>(part_slot(i, i == c0)) * ROWS + r]);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, o));
  const float ref = top == -INFINITY ? 0.f : top;
  float sum = 0.f, acc[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int i = c0; i <= c1; ++i) {
    const long long at = static_cast<long long>(part_slot(i, i == c0)) * ROWS + r;
    const float f = pg_ex2(p.part_lse[at] - ref);
    sum += f;
#pragma unroll
    for (int e = 0; e < EL; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p.part + at * D + d0 + e);
      acc[e] += f * v.x;
      acc[e + 1] += f * v.y;
      acc[e + 2] += f * v.z;
      acc[e + 3] += f * v.w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* dst = static_cast<T*>(p.out) + t * p.os_t + head * p.os_h + d0;
#pragma unroll
  for (int e = 0; e < EL; ++e) dst[e] = Piece<T>::of(acc[e] * inv);
  if (p.lse != nullptr && d0 == 0)
    p.lse[t * p.heads_q + head] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * LN2;
}

// The prompt kernel (mk_prompt.cu): entries of its work list, partial rows of a CTA's place.
int prompt_entries(int tokens, int group, int batch);
int prompt_part_rows();
cudaError_t launch_prompt(const PagedParams& p, int d, mk_dtype dtype, bool e8, bool after_decode, cudaStream_t s);

}  // namespace mk
