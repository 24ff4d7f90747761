// Operands of the bf16 matrix product, float32 values as bf16 pieces, buffers that
// end where their data does, sums over the lanes of a wave.
#pragma once

#include "ops.h"

namespace rssm {

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

union Frag {  // eight bf16 of one lane: an operand of the 16x16x32 product
  s16x8 v;
  s16x4 h[2];
  uint32_t w[4];
};

__device__ __forceinline__ floatx4 mfma32(const Frag &a, const Frag &b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a.v), __builtin_bit_cast(bf16x8, b.v), c, 0, 0, 0);
}

// The transposing LDS read: 16 lanes of 8 bytes each, lane l from row l / 4 and columns
// 4 (l % 4) .. + 3, get column l of the four rows.
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
__device__ __forceinline__ s16x4 read_tr(const char *p) { return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p); }

__device__ __forceinline__ float upper(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float lower(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ uint32_t bits(float v) { return __float_as_uint(v); }

// A buffer of n bytes: loads past its end give zeros, stores past it do nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, size_t n) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)n, 0x00020000);
}
__device__ __forceinline__ uint4 buffer_load16(__amdgpu_buffer_rsrc_t b, int at, int plus) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(b, at, plus, 0));
}

// Two values as MP words of bf16 pairs: two pieces round to nearest (together within
// 2^-16 of the value), three pieces cut (8 bits each: the 24 bits of the value).
template <int MP>
__device__ __forceinline__ void pieces(float a, float b, uint32_t (&w)[MP]) {
  static_assert(MP == 2 || MP == 3);
  if constexpr (MP == 2) {
    w[0] = pack_bf16(a, b);
    w[1] = pack_bf16(a - lower(w[0]), b - upper(w[0]));
  } else {
#pragma unroll
    for (int u = 0; u < MP; ++u) {
      w[u] = __builtin_amdgcn_perm(bits(b), bits(a), 0x07060302u);  // the upper halves, b's on top
      if (u + 1 < MP) a -= upper(bits(a)), b -= upper(bits(b));
    }
  }
}

// Moves of the low and high half of a double between lanes; lanes without a source get 0.
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v) {
  const int2 w = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_update_dpp(0, w.x, CTRL, ROWS, 0xF, false),
                                              __builtin_amdgcn_update_dpp(0, w.y, CTRL, ROWS, 0xF, false)));
}
__device__ __forceinline__ double lane_value(double v, int lane) {  // lane: the same for the whole wave
  const int2 w = __builtin_bit_cast(int2, v);
  return __builtin_bit_cast(double, make_int2(__builtin_amdgcn_readlane(w.x, lane), __builtin_amdgcn_readlane(w.y, lane)));
}
// Inclusive prefix sum of a wave: within rows of 16 by shifts, then the last lane of a
// row to the next row, and lane 31 to the upper half.
__device__ __forceinline__ double scan64(double v) {
  v += moved<0x111, 0xF>(v);
  v += moved<0x112, 0xF>(v);
  v += moved<0x114, 0xF>(v);
  v += moved<0x118, 0xF>(v);
  v += moved<0x142, 0xA>(v);
  v += moved<0x143, 0xC>(v);
  return v;
}

}  // namespace rssm
