// The microscaled format, shared by the quantiser and the 4-bit expert FFN.
//
// 32 consecutive values of a row share one byte b, the scale 2^(b - 127); the
// values are e2m1 (4 bits, two a byte, the first in the low half), e2m3 (6 bits,
// little-endian) or e4m3.  b is the smallest for which the block's largest
// magnitude still rounds to the format's largest value (6, 7.5, 448) or less, so
// nothing is clipped by more than a rounding.  b = 255 stands for NaN and marks a block that holds a NaN or an
// infinity.
#pragma once
#include "common.h"
#include "rows.h"

namespace mx {

constexpr int kBlock = 32;

// Bits a code.
constexpr int kF4 = 4, kF6 = 6, kF8 = 8;
__host__ __device__ constexpr int64_t code_bytes(int bits, int64_t n) { return (n * bits + 7) / 8; }

// The scale byte of a block from the bits of its largest magnitude.  The carry
// added to the float's bits raises the exponent just where the mantissa would
// round past the format's largest: from 1.75 on for e2m1 and 1.9375 on for e2m3
// (the ties at 7 and 7.75 go to 8), above 1.8125 for e4m3 (the tie at 464 goes
// to 448).
template <int kBits>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  constexpr uint32_t kCarry = kBits == kF8 ? 0x17ffffu : kBits == kF6 ? 0x80000u : 0x200000u;
  constexpr uint32_t kEmax = kBits == kF8 ? 8 : 2;
  if (amax_bits >= 0x7f800000u) return 255;
  const uint32_t e = (amax_bits + kCarry) >> 23;
  return e > kEmax ? e - kEmax : 0;
}

// 2^(b - 127) as a float: subnormal for b = 0, NaN for b = 255.
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x400000u : b == 255 ? 0x7fc00000u : b << 23);
}

typedef short s16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t encode4_fp8(float a, float b, float c, float d, float scale) {
  s16x2 r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a, b, scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, c, d, scale, true);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t encode8_fp4(const float* v, float scale) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
}
// e2m3: steps of 1/8 below 2, 1/4 below 4, 1/2 below 8.  (The conversion
// instruction takes a whole block of one lane.)
__device__ __forceinline__ uint2 encode8_fp6(const float (&v)[8], int shift) {
  uint64_t r = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float m = fabsf(ldexpf(v[u], shift));
    const float t = m < 2.f ? rintf(m * 8.f) : m < 4.f ? rintf(m * 4.f) + 8.f : rintf(m * 2.f) + 16.f;
    const uint32_t c = static_cast<uint32_t>(t) | (__float_as_uint(v[u]) >> 31 << 5);
    r |= static_cast<uint64_t>(c) << (6 * u);
  }
  return make_uint2(static_cast<uint32_t>(r), static_cast<uint32_t>(r >> 32));
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight values of a block: its codes times the scale.  The products are exact
// where they are normal floats (at most 4 significant bits).
__device__ __forceinline__ void decode8_fp8(uint2 q, float scale, float (&v)[8]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], true);
    v[4 * h] = lo.x * scale;
    v[4 * h + 1] = lo.y * scale;
    v[4 * h + 2] = hi.x * scale;
    v[4 * h + 3] = hi.y * scale;
  }
}
__device__ __forceinline__ void decode8_fp6(uint2 q, float scale, float (&v)[8]) {
  const uint64_t r = q.x | static_cast<uint64_t>(q.y) << 32;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const uint32_t c = static_cast<uint32_t>(r >> (6 * u)) & 63, e = (c >> 3) & 3, m = c & 7;
    const float a = e == 0 ? m * 0.125f : __uint_as_float((126 + e) << 23 | m << 20);
    v[u] = (c & 32 ? -a : a) * scale;
  }
}
__device__ __forceinline__ void decode8_fp4(uint32_t q, float scale, float (&v)[8]) {
  const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 1),
                      __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 3)};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = p[j].x * scale;
    v[2 * j + 1] = p[j].y * scale;
  }
}

// Rows in blocks: a lane takes a unit of V values, 32 / V lanes a block, so that a wave's
// access to the values is one run of 1 KB (V = 8 bf16, 4 float) and the block's largest
// magnitude two or three DPP steps.  A thread block's units are 256 * kUnits in a row of
// the flat order (row, unit).
//
// Addresses are a uniform 64-bit row base and 32-bit offsets from it: a block's units lie in
// two rows where a row has as many units as a block, and in a few thousand values at most
// otherwise.  (64-bit products for every unit were as long as the rest of the work.)
template <int kUnits>
struct Units {
  int64_t row0;
  uint32_t rem, per_row;
  bool wide;   // rows row0 and row0 + 1 alone
  __device__ __forceinline__ Units(int64_t block, uint32_t units_per_row) : per_row(units_per_row) {
    const int64_t base = block * (256 * kUnits);
    row0 = base / per_row;
    rem = static_cast<uint32_t>(base - row0 * per_row);
    wide = per_row >= 256 * kUnits;
  }
  // unit j of this thread: in row row0 + r
  __device__ __forceinline__ void at(int j, uint32_t* r, uint32_t* unit) const {
    const uint32_t v = rem + j * 256 + threadIdx.x;
    if (wide) {
      *r = v >= per_row;
      *unit = *r ? v - per_row : v;
    } else {
      *r = v / per_row;
      *unit = v - *r * per_row;
    }
  }
};

// Two floats to bf16, rounded to nearest even by the conversion instruction.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

// V consecutive values from element i on (the last n of a row): 16 bytes, with only the
// elements' own alignment.
template <bool kBf16, int V>
__device__ __forceinline__ void load_values(const void* p, uint32_t i, int n, float (&v)[V]) {
  if constexpr (V == 8) {
    rows::unpack8<kBf16>(rows::load8_part<kBf16>(p, i, n), v);
  } else {
    const float* q = static_cast<const float*>(p) + i;
    if (n >= 4) __builtin_memcpy(v, q, 16);
    else
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = u < n ? q[u] : 0.f;
  }
}
template <bool kBf16, int V>
__device__ __forceinline__ void store_values(void* p, uint32_t i, int n, const float (&v)[V]) {
  if (n < V) {
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (u < n) rows::store1<kBf16>(p, i + u, v[u]);
    return;
  }
  uint32_t w[kBf16 ? V / 2 : V];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    if constexpr (!kBf16) w[u] = __float_as_uint(v[u]);
    else if (u % 2 == 0) w[u / 2] = pack_bf16(v[u], v[u + 1]);
  }
  __builtin_memcpy(static_cast<char*>(p) + static_cast<uint64_t>(i) * (kBf16 ? 2 : 4), w, sizeof(w));
}

// The scale byte of the block that this lane's V values are a part of (its lanes together).
template <int kBits, int V>
__device__ __forceinline__ uint32_t shared_scale(const float (&v)[V]) {
  float a = fabsf(v[0]);   // (a NaN stays: IEEE 754-2019 maximum)
#pragma unroll
  for (int u = 1; u < V; ++u) a = __builtin_elementwise_maximum(a, fabsf(v[u]));
  uint32_t m = __float_as_uint(a) & 0x7fffffffu;
  m = max(m, static_cast<uint32_t>(dpp_partner<1>(static_cast<int>(m))));
  m = max(m, static_cast<uint32_t>(dpp_partner<2>(static_cast<int>(m))));
  if constexpr (V == 4) m = max(m, static_cast<uint32_t>(dpp_partner<4>(static_cast<int>(m))));
  return scale_byte<kBits>(m);
}

// The codes of V values, V * kBits / 8 bytes of them.
template <int kBits, int V>
__device__ __forceinline__ uint2 encode(const float (&v)[V], uint32_t byte) {
  if (byte == 255) return make_uint2(0, 0);
  const float s = scale_value(byte);
  if constexpr (V == 4) {
    static_assert(kBits != kF6, "e2m3 codes of four values end inside a byte");
    if constexpr (kBits == kF8) return make_uint2(encode4_fp8(v[0], v[1], v[2], v[3], s), 0);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
    return make_uint2(__builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1), 0);
  } else if constexpr (kBits == kF8) {
    return make_uint2(encode4_fp8(v[0], v[1], v[2], v[3], s), encode4_fp8(v[4], v[5], v[6], v[7], s));
  } else if constexpr (kBits == kF6) {
    return encode8_fp6(v, 127 - static_cast<int>(byte));
  } else {
    return make_uint2(encode8_fp4(v, s), 0);
  }
}
template <int kBits, int V>
__device__ __forceinline__ void decode(uint2 q, uint32_t byte, float (&v)[V]) {
  const float s = scale_value(byte);
  float w[8];
  if constexpr (kBits == kF8) decode8_fp8(q, s, w);
  else if constexpr (kBits == kF6) decode8_fp6(q, s, w);
  else decode8_fp4(q.x, s, w);
#pragma unroll
  for (int u = 0; u < V; ++u) v[u] = w[u];
}

// A whole block in one lane, as an operand of the matrix instructions: 16 bytes of
// e2m1, or 24 of e2m3 in two parts.
typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
struct Operand {
  uint4 first;
  uint2 rest;   // e2m3 only
  uint32_t byte;
};
template <int kBits>
__device__ __forceinline__ Operand encode_block(const float (&v)[32]) {
  float m = fabsf(v[0]);   // (a NaN stays: IEEE 754-2019 maximum, two values an instruction)
#pragma unroll
  for (int u = 1; u < 32; ++u) m = __builtin_elementwise_maximum(m, fabsf(v[u]));
  Operand o;
  o.byte = scale_byte<kBits>(__float_as_uint(m) & 0x7fffffffu);
  const float s = scale_value(o.byte);
  if constexpr (kBits == kF6) {
    f32x16 even, odd;   // the instruction takes its codes from the two in turn
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      even[u] = v[2 * u];
      odd[u] = v[2 * u + 1];
    }
    // The instruction writes its first results before it has read the scale for the
    // last: a result that shares the scale's register (as the builtin's may) comes out
    // wrong.  The asm keeps the result apart from all inputs; none of them comes straight
    // from a matrix instruction.
    u32x6 r;
    asm("v_cvt_scalef32_2xpk16_fp6_f32 %0, %1, %2, %3" : "=&v"(r) : "v"(even), "v"(odd), "v"(s));
    o.first = make_uint4(r[0], r[1], r[2], r[3]);
    o.rest = make_uint2(r[4], r[5]);
  } else {
    o.first = make_uint4(encode8_fp4(v, s), encode8_fp4(v + 8, s), encode8_fp4(v + 16, s), encode8_fp4(v + 24, s));
    o.rest = make_uint2(0, 0);
  }
  if (o.byte == 255) {
    o.first = make_uint4(0, 0, 0, 0);
    o.rest = make_uint2(0, 0);
  }
  return o;
}

}  // namespace mx
