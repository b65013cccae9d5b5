// mk_w4.h -- 4-bit weights as the kernels of mk_w4.cu (few tokens) and mk_w4_tiles.cu (more of them) take them.
#pragma once

#include "mk_seq.cuh"

namespace mk {

struct W4Params {
  const char* x;
  long long x_row;                     // bytes
  const uint8_t* codes;                // [n x k / 2]
  const void* scales;                  // [n x k / G], x's type
  const void* zeros;                   // the same, or null
  char* y;
  long long y_row;                     // bytes
  int m, n, k, groups, out_f32;
};

constexpr int W4_PIECE = 128;          // k of a step

// Whether mk_w4_tiles.cu serves a call: more than 8 tokens, and fewer where small groups make the other way's scales
// dear and the matrix is large enough for three launches (graphs, us, mma.sync / tcgen05, one token: groups of 32,
// 1024 x 2048 4.5 / 6.6, 3584 x 8192 16.8 / 12.8, 28672 x 8192 90 / 53; of 64 with zero points 8192 x 8192 18.2 / 17.3,
// 28672 x 8192 52 / 46; of 128 without, 34 / 42).
inline bool w4_use_tiles(const W4Params& p, int group) {
  const long long weights = static_cast<long long>(p.n) * p.k;
  return p.m > 8 || (group == 32 && weights >= (1LL << 24)) || (group == 64 && weights >= (1LL << 27));
}
size_t w4_tiles_scratch(const W4Params& p, int group);
mk_status launch_w4_tiles(const W4Params& p, mk_dtype dtype, int group, void* scratch, uint32_t* hdr, const mk_config* cfg,
                          cudaStream_t s);

template <class T> struct Codes;
template <> struct Codes<__half> {
  // the 8 codes of a word as four pairs (codes i and i + 4), minus 8: exactly
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t (&o)[4]) {
    const uint32_t v = w >> 8;
    // 1024 + c, and 1024 + 16 c, in fp16
    const uint32_t a[4] = {(w & 0x000f000fu) | 0x64006400u, (w & 0x00f000f0u) | 0x64006400u,
                           (v & 0x000f000fu) | 0x64006400u, (v & 0x00f000f0u) | 0x64006400u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 h;
      memcpy(&h, &a[i], 4);
      h = (i & 1) ? __hfma2(h, __floats2half2_rn(0.0625f, 0.0625f), __floats2half2_rn(-72.f, -72.f))
                  : __hsub2(h, __floats2half2_rn(1032.f, 1032.f));
      memcpy(&o[i], &h, 4);
    }
  }
  static constexpr uint32_t ONES = 0x3c003c00u;
};
template <> struct Codes<__nv_bfloat16> {
  static __device__ __forceinline__ void pairs(uint32_t w, uint32_t (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;      // 128 + c in bf16
      __nv_bfloat162 h;
      memcpy(&h, &v, 4);
      h = __hsub2(h, __floats2bfloat162_rn(136.f, 136.f));
      memcpy(&o[i], &h, 4);
    }
  }
  static constexpr uint32_t ONES = 0x3f803f80u;
};

// 8 neighbouring values of x in the order that Codes::pairs gives the codes: (0, 4), (1, 5), (2, 6), (3, 7)
__device__ __forceinline__ void x_pairs(const uint4& w, uint32_t (&o)[4]) {
  o[0] = __byte_perm(w.x, w.z, 0x5410);
  o[1] = __byte_perm(w.x, w.z, 0x7632);
  o[2] = __byte_perm(w.y, w.w, 0x5410);
  o[3] = __byte_perm(w.y, w.w, 0x7632);
}

template <class T>
__device__ __forceinline__ void w4_store(const W4Params& p, int tok, int row, float v) {
  char* y = p.y + tok * p.y_row;
  if (p.out_f32) reinterpret_cast<float*>(y)[row] = v;
  else reinterpret_cast<T*>(y)[row] = Piece<T>::of(v);
}

}  // namespace mk
