// mk_seq.cuh -- the batch and cache descriptors as the kernels see them: which
// sequence a token row belongs to, where its key and value live, 16-byte row
// pieces as fp32 values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "mk_internal.h"
#include "mk_ptx.cuh"

namespace mk {

// mk_seq_batch and mk_kv_cache as the kernels take them (strides in elements).
struct SeqView {
  const int* cu_q;      // [batch + 1]
  const int* kv_len;    // [batch]
  const int* pages;     // [batch x max_pages], rows pages_stride apart
  long long pages_stride;
  int batch, max_pages, tokens;
};
struct CacheView {
  void* k;
  void* v;
  float* k_scale;       // [n_pages x heads], 8-bit caches
  float* v_scale;
  long long page_stride, head_stride, slot_stride;
  long long n_pages;
  int heads, d, page_size, page_log2;
};

// Host checks shared by the entry points (mk_rope.cu).
bool view_of(const mk_seq_batch* s, long long tokens, SeqView& out);
bool view_of(const mk_kv_cache* c, CacheView& out);

// Records the first error of a call in the workspace's status word.
__device__ __forceinline__ void seq_error(uint32_t* hdr, int code, int where, int index) {
  if (hdr == nullptr) return;
  if (atomicCAS(reinterpret_cast<int*>(&hdr[HDR_STATUS]), 0, code) == 0)
    atomicExch(reinterpret_cast<int*>(&hdr[HDR_DETAIL]), where * 1000000 + (index % 1000000));
}

// The last b in [0, n) with key(b) <= t for a non-decreasing key, -1 if there
// is none; by the whole warp, 32 probes a round (two rounds for 1024), since
// each round is one dependent trip to L2.  Any contents of the array end it.
template <class Key>
__device__ __forceinline__ int warp_last_le(int n, int t, Key key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;
  bool first = true;
  while (first || hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const int c = __popc(__ballot_sync(0xffffffffu, at < hi && key(at) <= t));
    if (c == 0) return first ? -1 : lo;
    lo += (c - 1) * step;
    hi = min(hi, lo + step);
    first = false;
  }
  return lo;
}

constexpr float E4M3_MAX = 448.f;
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t two;      // to nearest even; past 448 saturates, NaN stays NaN
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(b), "f"(a));
  return two;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// 16 bytes of a row as fp32 values, and back (one rounding, to nearest even).
template <class T> struct Piece;
template <> struct Piece<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y); f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float one(float x) { return x; }
  static __device__ __forceinline__ float of(float x) { return x; }
};
template <> struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& w, float (&f)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(v[i] << 16);
      f[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ float one(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 of(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Piece<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& w, float (&f)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 h;
      memcpy(&h, &v[i], 4);
      const float2 x = __half22float2(h);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    return make_uint4(pack(f[0], f[1]), pack(f[2], f[3]), pack(f[4], f[5]), pack(f[6], f[7]));
  }
  static __device__ __forceinline__ float one(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half of(float x) { return __float2half_rn(x); }
};

}  // namespace mk
