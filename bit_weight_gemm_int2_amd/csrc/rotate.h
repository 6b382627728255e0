// Rows of heads as the kernels of the cache and of the rotation take them: 16
// values a lane in two pieces, their rotation by position, and the norm of a
// head, whose D / 16 lanes lie side by side in a wave.
#pragma once
#include "common.h"

namespace lowbit {

// 8 consecutive values, 16-byte aligned. ONCE: values that nothing reads again
// from the caches (non-temporal, as all dense stores: 11000 tokens with their
// queries and the read-back took 86 us through the caches, 74 past them).
template <int DT, bool ONCE = false>
__device__ __forceinline__ void load8(const void* p, int64_t i, float* r) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const f32x4 w = *(const f32x4*)((const float*)p + i + 4 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) r[4 * j + e] = w[e];
    }
  } else {
    const u32x4* from = (const u32x4*)((const uint16_t*)p + i);
    const u32x4 w = ONCE ? __builtin_nontemporal_load(from) : *from;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint16_t h = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
      r[e] = DT == DT_F16 ? half_bits_to_float(h) : bf16_bits_to_float(h);
    }
  }
}

template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, const float* r) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      __builtin_nontemporal_store(f32x4{r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]},
                                  (f32x4*)((float*)p + i + 4 * j));
  } else {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = DT == DT_F16 ? (uint32_t)float_to_half_bits(r[2 * e]) | (uint32_t)float_to_half_bits(r[2 * e + 1]) << 16
                          : (uint32_t)float_to_bf16_bits(r[2 * e]) | (uint32_t)float_to_bf16_bits(r[2 * e + 1]) << 16;
    __builtin_nontemporal_store(w, (u32x4*)((uint16_t*)p + i));
  }
}

// Unit u of a row is 16 values in two pieces of 8, placed so that a rotated
// pair never leaves a unit: with halves apart (d, d + rot / 2) the pieces are
// 8 u and rot / 2 + 8 u, with neighbours paired (and past the rotated part)
// they are 16 u and 16 u + 8. Every piece is one 16-byte load of 16-bit
// values, and neighbouring lanes take neighbouring pieces.
__device__ __forceinline__ void unit_places(int u, int rot, int inter, int* d0, int* d1) {
  if (!inter && 16 * u < rot) {
    *d0 = 8 * u;
    *d1 = rot / 2 + 8 * u;
  } else {
    *d0 = 16 * u;
    *d1 = 16 * u + 8;
  }
}

struct Turn {             // cos and sin of a unit's eight pairs; none past the rotated part
  float c[8], s[8];
  bool on;
};
// The tables [positions][rot / 2] at position pos.
__device__ __forceinline__ void load_turn(const float* cos, const float* sin, int rot, int u, int64_t pos, Turn* t) {
  t->on = 16 * u < rot;
  if (!t->on) return;
  load8<DT_F32>(cos, pos * (rot / 2) + 8 * u, t->c);
  load8<DT_F32>(sin, pos * (rot / 2) + 8 * u, t->s);
}

// Rotate one unit in place: r[0 .. 7] is its first piece, r[8 .. 15] its second.
__device__ __forceinline__ void rotate_unit(float* r, const Turn& t, int inter) {
  if (!t.on) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = i, b = i + 8;
    if (!inter) {
      const float x = r[a], y = r[b];
      r[a] = __builtin_fmaf(x, t.c[i], -(y * t.s[i]));
      r[b] = __builtin_fmaf(x, t.s[i], y * t.c[i]);
    } else {
      const float x = r[2 * i], y = r[2 * i + 1];
      r[2 * i] = __builtin_fmaf(x, t.c[i], -(y * t.s[i]));
      r[2 * i + 1] = __builtin_fmaf(x, t.s[i], y * t.c[i]);
    }
  }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

__device__ __forceinline__ void load4(const float* p, float* r) {
  const f32x4 w = *(const f32x4*)p;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = w[e];
}

// x of the lane that a DPP control names, all within groups of 16 lanes: no trip through the LDS.
template <int CTRL>
__device__ __forceinline__ double other_lane(double x) {
  const u32x2 b = __builtin_bit_cast(u32x2, x);
  const uint32_t lo = b[0], hi = b[1];
  return __builtin_bit_cast(double, u32x2{(uint32_t)__builtin_amdgcn_mov_dpp((int)lo, CTRL, 0xf, 0xf, true),
                                          (uint32_t)__builtin_amdgcn_mov_dpp((int)hi, CTRL, 0xf, 0xf, true)});
}

// The norm of a head, y = x / sqrt(mean x^2 + eps) * w: the factor of its 16
// values in each of the U = D / 16 lanes that hold it (a power of two,
// consecutive lanes, all active). The squares and their sum are FP64: no FP32
// value overflows or vanishes there (squares of BF16 values of 2^64 pass FP32's
// range), and it took no longer than FP32 (both 28.5 us for 4608 tokens of 48
// heads, in an earlier form of the dense kernel, which takes 24.5 now). With a sum of 0 and no eps the row stays 0. The factor of a row of
// subnormal values without eps passes FP32's range (2^149 of 2^-149), and that of a
// row beyond 2^126 is subnormal itself, with 22 bits or fewer: a row whose mean is
// below 2^-252 or above 2^252 is moved up or down by 2^64 first, so that the factor
// is a normal number (where `norm`: a row that takes none stays as it is).
__device__ __forceinline__ float norm_factor(float* r, bool norm, int U, double inv_d, double eps) {
  double sum = 0.0;
#pragma unroll
  for (int e = 0; e < 16; ++e) sum = __builtin_fma((double)r[e], (double)r[e], sum);
  sum += other_lane<0xB1>(sum);                              // quad_perm: lanes 1, 0, 3, 2 of each four
  sum += other_lane<0x4E>(sum);                              // and 2, 3, 0, 1
  if (U > 4) sum += other_lane<0x141>(sum);                  // the mirrored lane of eight, whose four hold the other sum
  if (U > 8) sum += other_lane<0x140>(sum);                  // and of sixteen
  const double mean = __builtin_fma(sum, inv_d, eps);
  double root = rsqrt(mean);
  if (norm && (mean < 0x1p-252 || mean > 0x1p252)) {
    const float by = mean < 1.0 ? 0x1p64f : 0x1p-64f;
#pragma unroll
    for (int e = 0; e < 16; ++e) r[e] *= by;
    root *= mean < 1.0 ? 0x1p-64 : 0x1p64;
  }
  return mean > 0.0 ? (float)root : mean == 0.0 ? 0.0f : __builtin_nanf("");
}
__device__ __forceinline__ void norm_unit(float* r, const float* w, int U, double inv_d, double eps) {
  const float by = norm_factor(r, true, U, inv_d, eps);
#pragma unroll
  for (int e = 0; e < 16; ++e) r[e] = r[e] * by * w[e];
}

// A unit's weights (w_dtype: any of the three types).
__device__ __forceinline__ void load_weights(const void* p, int w_dtype, int d0, int d1, float* w) {
  if (w_dtype == DT_F32) {
    load8<DT_F32>(p, d0, w);
    load8<DT_F32>(p, d1, w + 8);
  } else if (w_dtype == DT_F16) {
    load8<DT_F16>(p, d0, w);
    load8<DT_F16>(p, d1, w + 8);
  } else {
    load8<DT_BF16>(p, d0, w);
    load8<DT_BF16>(p, d1, w + 8);
  }
}

}  // namespace lowbit
