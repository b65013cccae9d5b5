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
// (graphs, weights out of L2, bf16, us, mma.sync / tcgen05, by groups and (z) zero points).
//   One token: 8192 x 8192 128 14.0 / 18.0, 64 15.0 / 18.3, 128 z 18.0 / 18.8, 32 17.2 / 18.8, 32 z 19.9 / 22.8;
//   28672 x 8192 128 36.1 / 44.3, 64 37.8 / 44.8, 128 z 50.1 / 47.1, 64 z 52.2 / 49.1, 32 46.7 / 46.4, 32 z 59.2 / 59.0.
//   16 tokens: 4096 x 4096 64 7.7 / 11.7, 128 z 10.0 / 11.8, 32 z 11.4 / 13.2; 3584 x 8192 128 13.7 / 13.8, 64 z 15.3 / 14.6;
//   8192 x 4096 64 12.4 / 13.4, 128 z 16.4 / 13.7; 8192 x 8192 64 22.2 / 18.7, 32 z 31.8 / 23.2.
//   More, 32 at a time: 17 and 32 tokens of 4096 x 4096 64 9.7 / 11.9 and 10.4 / 12.0, 128 10.8 / 11.9 and 12.8 / 12.0, 128 z 12.7 / 12.2 and
//   14.2 / 12.3, 32 z 14.3 / 15.0 and 15.8 / 15.1; of 3584 x 8192 64 16.2 / 14.3 and 17.1 / 14.4; 64 of 2048 x 4096 64 9.8 / 13.8, 32 z 15.3 / 14.4;
//   128 of 2048 x 2048 64 9.6 / 12.3, 128 12.5 / 12.2, 32 z 15.1 / 13.0, and of 2048 x 4096 17.3 / 13.1, 22.2 / 12.3, 27.6 / 18.2.
inline bool w4_use_tiles(const W4Params& p, int group) {
  const long long weights = static_cast<long long>(p.n) * p.k;
  if (p.m > 16) return weights * ((p.m + 31) / 32) > (1LL << 24) || p.m > (1 << 20);       // (more blocks of tokens than a grid has)
  if (p.m > 8) return weights > (p.zeros ? 1LL << 24 : 1LL << 25);
  return weights >= (1LL << 27) && (p.zeros || group == 32);
}
size_t w4_tiles_scratch(const W4Params& p, int group);
mk_status launch_w4_tiles(const W4Params& p, mk_dtype dtype, int group, void* scratch, uint32_t* hdr, const mk_config* cfg,
                          cudaStream_t s);

template <class T> struct Codes;
template <> struct Codes<__half> {
  // the 8 codes of a word as four pairs (codes i and i + 4), minus 8: exactly.  (A code in the low bits of 1024, or in
  // those from 16 on, is a number at once: the way that is commonly published for small codes.)
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
