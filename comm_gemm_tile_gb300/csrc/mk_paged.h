// mk_paged.h -- what the two attention kernels over a paged cache share: the
// call, which keys a sequence's rows see, how tiles are dealt to CTAs, the
// partial results and their join.
#pragma once

#include "mk_seq.cuh"

namespace mk {

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
  long long* prefix;                   // tiles of the units before each sequence / item (see the kernels)
  long long wait_ns;
  float scale_log2;                    // softmax scale * log2(e)
  int heads_q, group;                  // query heads; of them per key head
  int causal, window, sinks;
  int map_pages;                       // pages in the tensor maps; a load from this page reads zeros
  int rows_lo, rows_hi;                // sequences with this many packed rows (tokens x group) are this launch's
  int grid;
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

// N tiles dealt to C = min(grid, N) CTAs in runs that differ by at most one
// tile; a unit (the tiles of one set of rows) may be cut by several runs.
struct Deal {
  long long n;
  int c;
  __device__ __forceinline__ Deal(long long total, int grid) : n(total), c(total < grid ? static_cast<int>(total) : grid) {}
  __device__ __forceinline__ long long start(int i) const { return n * i / c; }
  __device__ __forceinline__ int owner(long long x) const { return static_cast<int>(((x + 1) * c + n - 1) / n) - 1; }
};
// Where CTA i leaves its partial result of the unit that begins at tile u0: one
// place for a unit begun by an earlier CTA, one for a unit it does not finish.
__device__ __forceinline__ int part_slot(const Deal& d, int i, long long u0) { return 2 * i + (d.start(i) > u0 ? 0 : 1); }

// ------------------------------------------------------------------ bounded waits
// No CTA of these kernels waits for another, so giving up is a CTA's own
// affair: a word in shared memory, after which every wait returns at once.
__device__ __forceinline__ bool pg_wait_slow(volatile int* dead, const PagedParams& p, uint32_t bar, uint32_t parity,
                                             int where) {
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

__device__ __forceinline__ float pg_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float LN2 = 0.69314718055994530942f;

// Joins the partial rows of the units that several CTAs shared (mk_paged.cu).
cudaError_t launch_prefill(PagedParams& p, const mk_kv_cache* c, mk_dtype dtype, int sms, cudaStream_t s);
size_t prefill_part_rows(int sms);

}  // namespace mk
