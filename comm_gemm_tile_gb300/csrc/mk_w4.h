// mk_w4.h -- 4-bit weights as the kernels of mk_w4.cu (few tokens) and mk_w4_tiles.cu (more of them, and large matrices) take them.
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

// Whether mk_w4_tiles.cu serves a call: its three launches and its steps' waits pay with many tokens or a large matrix
// (graphs, weights out of L2, bf16, us, mma.sync / tcgen05.  32 tokens: 2048 x 4096, groups of 64 5.9 / 12.4, with zero points
// 7.6 / 12.7; 4096 x 4096 10.0 / 12.0, 13.5 / 12.8, groups of 128 12.7 / 11.8.  16 tokens: 4096 x 4096 7.4 / 11.5, 9.3 / 11.9;
// 3584 x 8192 11.9 / 14.2, 15.3 / 14.5; 8192 x 8192 21.7 / 19.3, 25.8 / 20.0.  One token: 8192 x 8192 15.0 / 18.8, 18.5 / 19.5;
// 28672 x 8192 38 / 45, 50 / 49, groups of 32 49 / 45.  More tokens, 32 at a time: 64 of 2048 x 2048, groups of 128, 7.3 / 9.5,
// of 4096 x 1024 7.6 / 8.4, 128 of them 13.7 / 11.4).
inline bool w4_use_tiles(const W4Params& p, int group) {
  const long long weights = static_cast<long long>(p.n) * p.k;
  if (p.m > 16) return weights * ((p.m + 31) / 32) >= (1LL << 24) || p.m > (1 << 20);      // (more blocks of tokens than a grid has)
  if (p.m > 8) return weights > (p.zeros ? 1LL << 24 : 1LL << 25);
  return weights >= (1LL << 27) && (p.zeros || group == 32);
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
