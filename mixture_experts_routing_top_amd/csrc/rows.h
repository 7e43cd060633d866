// Row access and reductions shared by the memory-bound row kernels.
#pragma once
#include "common.h"

namespace rows {

// Eight consecutive elements from element offset i.  The address needs only the
// element's own alignment (rows of an odd width start anywhere): global
// accesses of 16 bytes may be unaligned on this target.
template <bool kBf16>
struct Raw8 {
  uint4 q[kBf16 ? 1 : 2];
};

template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> load8(const void* p, int64_t i) {
  Raw8<kBf16> r;
  __builtin_memcpy(&r, static_cast<const char*>(p) + i * (kBf16 ? 2 : 4), sizeof(r));
  return r;
}

template <bool kBf16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (kBf16) return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

template <bool kBf16>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (kBf16) static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(f32_to_bf16_bits(v));
  else static_cast<float*>(p)[i] = v;
}

// The first n (of eight) elements, the rest zero.
template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> load8_part(const void* p, int64_t i, int n) {
  if (n >= 8) return load8<kBf16>(p, i);
  Raw8<kBf16> r;
  uint32_t w[kBf16 ? 4 : 8] = {};
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (u < n) {
      if constexpr (kBf16) w[u / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i + u]) << (16 * (u & 1));
      else w[u] = static_cast<const uint32_t*>(p)[i + u];
    }
  __builtin_memcpy(&r, w, sizeof(r));
  return r;
}

template <bool kBf16>
__device__ __forceinline__ void unpack8(const Raw8<kBf16>& r, float (&v)[8]) {
  uint32_t w[kBf16 ? 4 : 8];
  __builtin_memcpy(w, &r, sizeof(r));
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if constexpr (kBf16) v[u] = (u & 1) ? __uint_as_float(w[u / 2] & 0xffff0000u) : __uint_as_float(w[u / 2] << 16);
    else v[u] = __uint_as_float(w[u]);
  }
}

template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> pack8(const float (&v)[8]) {
  uint32_t w[kBf16 ? 4 : 8];
#pragma unroll
  for (int u = 0; u < (kBf16 ? 4 : 8); ++u) {
    if constexpr (kBf16) w[u] = f32_to_bf16_bits(v[2 * u]) | (f32_to_bf16_bits(v[2 * u + 1]) << 16);
    else w[u] = __float_as_uint(v[u]);
  }
  Raw8<kBf16> r;
  __builtin_memcpy(&r, w, sizeof(r));
  return r;
}

template <bool kBf16>
__device__ __forceinline__ void store8_part(void* p, int64_t i, int n, const float (&v)[8]) {
  if (n >= 8) {
    const Raw8<kBf16> r = pack8<kBf16>(v);
    __builtin_memcpy(static_cast<char*>(p) + i * (kBf16 ? 2 : 4), &r, sizeof(r));
    return;
  }
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (u < n) store1<kBf16>(p, i + u, v[u]);
}

// Sum over the wave, the same value in every lane, in a fixed order: DPP
// pairings inside the 16-lane rows, then the four rows' sums.
__device__ __forceinline__ float wave_sum(float v) {
  v += __int_as_float(dpp_partner<1>(__float_as_int(v)));
  v += __int_as_float(dpp_partner<2>(__float_as_int(v)));
  v += __int_as_float(dpp_partner<4>(__float_as_int(v)));
  v += __int_as_float(dpp_partner<8>(__float_as_int(v)));
  const int x = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(x, 0)) + __int_as_float(__builtin_amdgcn_readlane(x, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(x, 32)) + __int_as_float(__builtin_amdgcn_readlane(x, 48)));
}

// Doubles: over the 16 lanes of a row, and over the wave.
template <int OFF>
__device__ __forceinline__ double partner64(double v) {
  return __hiloint2double(dpp_partner<OFF>(__double2hiint(v)), dpp_partner<OFF>(__double2loint(v)));
}
__device__ __forceinline__ double lane64(double v, int lane) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                          __builtin_amdgcn_readlane(__double2loint(v), lane));
}
__device__ __forceinline__ double row_max(double v) {
  v = fmax(v, partner64<1>(v));
  v = fmax(v, partner64<2>(v));
  v = fmax(v, partner64<4>(v));
  return fmax(v, partner64<8>(v));
}
__device__ __forceinline__ double row_sum(double v) {
  v += partner64<1>(v);
  v += partner64<2>(v);
  v += partner64<4>(v);
  return v + partner64<8>(v);
}
__device__ __forceinline__ double wave_max(double v) {
  v = row_max(v);
  return fmax(fmax(lane64(v, 0), lane64(v, 16)), fmax(lane64(v, 32), lane64(v, 48)));
}
__device__ __forceinline__ double wave_sum(double v) {
  v = row_sum(v);
  return (lane64(v, 0) + lane64(v, 16)) + (lane64(v, 32) + lane64(v, 48));
}

}  // namespace rows
