// moe_mx_quantize, moe_mx_dequantize: rows to blocks of 32 values with one
// power-of-two scale, in 4, 6 or 8 bits, and the values that they stand for back
// again (by a row map, as a dispatch copies rows).  moe_combine_backward: the
// gradient of the weighted combine, from expert outputs in the dtype or kept in
// 8-bit blocks.
//
// All three are bound by memory: every value is read once and written once, 16 bytes
// of them a lane, in accesses that a wave makes to one run of addresses.  mx.h has the
// format and the split of a row over lanes.  Measured out of cache, a launch included:
// 28672 x 4096 bf16 to 8 bits 63 us (5.7 TB/s) and back 63, to 4 bits 51 (5.8) and back 60;
// float to 4 bits 98 (5.4) and back 91 (5.8); e2m3 has no conversion for single values
// and takes some 25 instructions a value: 68 (4.8) and back 62, float 99 and back 137 (4.1).
#include <type_traits>

#include "common.h"
#include "mx.h"
#include "rows.h"

namespace {

using moe::ceil_div;
using namespace rows;

// Values a lane: 16 bytes, but eight floats where four e2m3 codes would end inside a byte.
template <bool kBf16, int kBits>
constexpr int kLane = kBf16 || kBits == mx::kF6 ? 8 : 4;

// Whole rows (kFlat: K a multiple of 32, and no row map): values, codes and scales are three
// flat runs, and a unit's places its number times a constant (28672 x 4096 bf16 to 4 bits
// 52 us; 28671 x 4095 by rows 70).
template <bool kBf16, int kBits, int kUnits>
__global__ __launch_bounds__(256) void quantize_flat_kernel(const void* __restrict__ x, int64_t n_units,
                                                            uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                            int32_t* __restrict__ check) {
  constexpr int V = kLane<kBf16, kBits>, P = mx::kBlock / V, kBytes = V * kBits / 8;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (256 * kUnits);
  const uint32_t left = static_cast<uint32_t>(min<int64_t>(n_units - base, 256 * kUnits));
  const char* const xb = static_cast<const char*>(x) + base * (V * (kBf16 ? 2 : 4));
  uint8_t* const qb = q + base * kBytes;
  uint8_t* const sb = scale + base / P;
  float v[kUnits][V];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t unit = j * 256 + threadIdx.x;
#pragma unroll
    for (int u = 0; u < V; ++u) v[j][u] = 0.f;
    if (unit < left) mx::load_values<kBf16, V>(xb, unit * V, V, v[j]);
  }
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t unit = j * 256 + threadIdx.x, byte = mx::shared_scale<kBits, V>(v[j]);
    bad |= byte == 255;
    const uint2 c = mx::encode<kBits, V>(v[j], byte);
    if (unit >= left) continue;
    __builtin_memcpy(qb + unit * kBytes, &c, kBytes);
    if (unit % P == 0) sb[unit / P] = static_cast<uint8_t>(byte);
  }
  if (check) raise_check(check, bad, MOE_CHECK_BLOCKS);
}

template <bool kBf16, int kBits, int kUnits>
__global__ __launch_bounds__(256) void dequantize_flat_kernel(const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ scale, int64_t n_units,
                                                              void* __restrict__ out) {
  constexpr int V = kLane<kBf16, kBits>, P = mx::kBlock / V, kBytes = V * kBits / 8;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (256 * kUnits);
  const uint32_t left = static_cast<uint32_t>(min<int64_t>(n_units - base, 256 * kUnits));
  const uint8_t* const qb = q + base * kBytes;
  const uint8_t* const sb = scale + base / P;
  char* const ob = static_cast<char*>(out) + base * (V * (kBf16 ? 2 : 4));
  uint2 c[kUnits];
  uint32_t byte[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t unit = j * 256 + threadIdx.x;
    c[j] = make_uint2(0, 0);
    byte[j] = 0;
    if (unit >= left) continue;
    __builtin_memcpy(&c[j], qb + unit * kBytes, kBytes);
    byte[j] = sb[unit / P];
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t unit = j * 256 + threadIdx.x;
    if (unit >= left) continue;
    float v[V];
    mx::decode<kBits, V>(c[j], byte[j], v);
    mx::store_values<kBf16, V>(ob, unit * V, V, v);
  }
}

template <bool kBf16, int kBits, int kUnits>
__global__ __launch_bounds__(256) void quantize_kernel(const void* __restrict__ x, int64_t R, int K, uint32_t blocks,
                                                       uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                       int32_t* __restrict__ check) {
  constexpr int V = kLane<kBf16, kBits>, P = mx::kBlock / V, kBytes = V * kBits / 8;
  const mx::Units<kUnits> units(blockIdx.x, P * blocks);
  const uint32_t row_bytes = static_cast<uint32_t>(mx::code_bytes(kBits, K));
  const char* const xb = static_cast<const char*>(x) + units.row0 * K * (kBf16 ? 2 : 4);
  uint8_t* const qb = q + units.row0 * row_bytes;
  uint8_t* const sb = scale + units.row0 * blocks;
  const uint32_t rows = static_cast<uint32_t>(min<int64_t>(R - units.row0, 1 << 30));
  float v[kUnits][V];
  uint32_t r[kUnits], unit[kUnits];
  int n[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    units.at(j, &r[j], &unit[j]);
    n[j] = r[j] < rows ? max(0, min(V, K - static_cast<int>(unit[j] * V))) : 0;
#pragma unroll
    for (int u = 0; u < V; ++u) v[j][u] = 0.f;
    if (n[j] > 0) mx::load_values<kBf16, V>(xb, r[j] * K + unit[j] * V, n[j], v[j]);
  }
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t byte = mx::shared_scale<kBits, V>(v[j]);   // (a block's lanes are in one row, or past the last)
    bad |= byte == 255;
    const uint2 c = mx::encode<kBits, V>(v[j], byte);
    if (r[j] >= rows) continue;
    if (unit[j] % P == 0) sb[r[j] * blocks + unit[j] / P] = static_cast<uint8_t>(byte);
    uint8_t* const p = qb + (r[j] * row_bytes + unit[j] * kBytes);
    const int bytes = static_cast<int>(mx::code_bytes(kBits, n[j]));
    if (bytes == kBytes) {
      __builtin_memcpy(p, &c, kBytes);
    } else {
      for (int u = 0; u < bytes; ++u) p[u] = static_cast<uint8_t>((u < 4 ? c.x : c.y) >> (8 * (u & 3)));
    }
  }
  if (check) raise_check(check, bad, MOE_CHECK_BLOCKS);
}

template <bool kBf16, int kBits, int kUnits>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                         int64_t R, int K, uint32_t blocks,
                                                         const int32_t* __restrict__ map, int64_t n_rows,
                                                         void* __restrict__ out, int32_t* __restrict__ check) {
  constexpr int V = kLane<kBf16, kBits>, P = mx::kBlock / V, kBytes = V * kBits / 8;
  const mx::Units<kUnits> units(blockIdx.x, P * blocks);
  const int64_t row_bytes = mx::code_bytes(kBits, K);
  char* const ob = static_cast<char*>(out) + units.row0 * K * (kBf16 ? 2 : 4);
  const uint32_t rows = static_cast<uint32_t>(min<int64_t>(n_rows - units.row0, 1 << 30));
  // a wide row's block reads two rows at most, through uniform loads of the map
  auto source = [&](int64_t row) -> int64_t { return row < n_rows ? (map ? map[row] : row) : -1; };
  const int64_t src0 = units.wide ? source(units.row0) : 0, src1 = units.wide ? source(units.row0 + 1) : 0;
  uint2 c[kUnits];
  uint32_t byte[kUnits], r[kUnits], unit[kUnits];
  int64_t src[kUnits];
  int n[kUnits];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    units.at(j, &r[j], &unit[j]);
    n[j] = r[j] < rows ? max(0, min(V, K - static_cast<int>(unit[j] * V))) : 0;
    src[j] = units.wide ? (r[j] ? src1 : src0) : n[j] > 0 ? source(units.row0 + r[j]) : -1;
    if (n[j] == 0 || src[j] < 0 || src[j] >= R) src[j] = -1;
    bad |= n[j] > 0 && src[j] < 0;   // such a row is zero
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    c[j] = make_uint2(0, 0);
    byte[j] = 127;
    if (src[j] < 0) continue;
    const uint8_t* const p = q + src[j] * row_bytes + unit[j] * kBytes;
    const int bytes = static_cast<int>(mx::code_bytes(kBits, n[j]));
    if (bytes == kBytes) {
      __builtin_memcpy(&c[j], p, kBytes);
    } else {
      for (int u = 0; u < bytes; ++u) (u < 4 ? c[j].x : c[j].y) |= static_cast<uint32_t>(p[u]) << (8 * (u & 3));
    }
    byte[j] = scale[src[j] * blocks + unit[j] / P];
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    if (n[j] == 0) continue;
    float v[V];
    mx::decode<kBits, V>(c[j], byte[j], v);
    mx::store_values<kBf16, V>(ob, r[j] * K + unit[j] * V, n[j], v);
  }
  if (check) raise_check(check, bad, MOE_CHECK_ROWS);
}

// d_y[inv[t,i]] = w[t,i] d_out[t] and d_w[t,i] = <d_out[t], y[inv[t,i]]>.  kWaves
// waves a token (kWaves = 1: four tokens a block), eight values of the row and of each
// of its KK expert rows a lane and step, all loads of a step before its sums.  Bound by
// memory: 8192 tokens of two kept rows, H = 4096, 271 MB in 58 us (4.7 TB/s; 46 where the
// output takes the last call's place); 16001 of six, H = 5120, 1.66 GB in 332 (5.0; the rows
// are written in the experts' order, a token's far apart).  Rows in bf16 62 and 424 us.
template <bool kBf16, bool kKept, int kWaves, int KK>
__global__ __launch_bounds__(256) void combine_backward_kernel(const void* __restrict__ d_out, const void* __restrict__ y,
                                                               const uint8_t* __restrict__ y_scale, int64_t M,
                                                               const int32_t* __restrict__ inv_pos,
                                                               const float* __restrict__ topk_w, int64_t T, int H,
                                                               uint32_t blocks, void* __restrict__ d_y,
                                                               float* __restrict__ d_topk_w,
                                                               int32_t* __restrict__ check) {
  __shared__ float part[4][KK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = kWaves == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + wave : blockIdx.x;
  if (kWaves == 1 && t >= T) return;
  int64_t at[KK];   // (an entry outside [0, M) reads row 0 and writes nothing)
  bool there[KK];
  float w[KK], acc[KK];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < KK; ++i) {
    const int32_t r = __builtin_amdgcn_readfirstlane(inv_pos[t * KK + i]);
    there[i] = r >= 0 && r < M;
    at[i] = there[i] ? r : 0;
    bad |= !there[i];
    w[i] = topk_w[t * KK + i];
    acc[i] = 0.f;
  }
  const int chunks = M > 0 ? H / 8 : 0;
  for (int c = (kWaves == 1 ? 0 : wave * 64) + lane; c < chunks; c += kWaves * 64) {
    const Raw8<kBf16> raw = load8<kBf16>(d_out, t * H + c * 8);
    uint2 q[KK];
    uint32_t byte[KK];
    Raw8<kBf16> yr[KK];
#pragma unroll
    for (int i = 0; i < KK; ++i) {
      if constexpr (kKept) {
        __builtin_memcpy(&q[i], static_cast<const uint8_t*>(y) + at[i] * H + c * 8, 8);
        byte[i] = y_scale[at[i] * blocks + (c >> 2)];
      } else {
        yr[i] = load8<kBf16>(y, at[i] * H + c * 8);
      }
    }
    float o[8];
    unpack8<kBf16>(raw, o);
#pragma unroll
    for (int i = 0; i < KK; ++i) {
      float v[8], s = 0.f, p[8];
      // (the values, exact, and not the codes: a block's largest code is 224 to 448 whatever its scale is)
      if constexpr (kKept) mx::decode8_fp8(q[i], mx::scale_value(byte[i]), v);
      else unpack8<kBf16>(yr[i], v);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        s = fmaf(o[u], v[u], s);
        p[u] = w[i] * o[u];
      }
      acc[i] += s;
      if (there[i]) mx::store_values<kBf16, 8>(static_cast<char*>(d_y) + at[i] * H * (kBf16 ? 2 : 4), c * 8, 8, p);
    }
  }
#pragma unroll
  for (int i = 0; i < KK; ++i) {
    const float v = there[i] ? wave_sum(acc[i]) : 0.f;
    if constexpr (kWaves == 1) {
      if (lane == 0) d_topk_w[t * KK + i] = v;
    } else if (lane == 0) {
      part[wave][i] = v;
    }
  }
  if constexpr (kWaves > 1) {
    __syncthreads();
    if (threadIdx.x < KK) {
      float v = part[0][threadIdx.x];
#pragma unroll
      for (int u = 1; u < kWaves; ++u) v += part[u][threadIdx.x];
      d_topk_w[t * KK + threadIdx.x] = v;
    }
  }
  if (check) raise_check(check, bad, MOE_CHECK_ROWS);
}

int check_format(const char* who, moe_dtype dt, moe_mx_format fmt, int64_t R, int64_t K) {
  using namespace moe;
  if (dt != MOE_F32 && dt != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dt);
  if (fmt != MOE_MX_FP4 && fmt != MOE_MX_FP8 && fmt != MOE_MX_FP6) return fail(MOE_ERR_INVALID_ARG, "%s: unknown format %d", who, (int)fmt);
  if (R < 0) return fail(MOE_ERR_INVALID_ARG, "%s: negative number of rows", who);
  if (K < 1 || K > (1 << 28)) return fail(MOE_ERR_INVALID_ARG, "%s: K=%lld outside [1, 2^28]", who, (long long)K);
  if (R > (int64_t(1) << 30) / ceil_div(K, mx::kBlock))   // (a launch has fewer than 2^32 threads)
    return fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^30 blocks of 32 values", who);
  return MOE_OK;
}

// Units a thread: 16 values' once that still fills the card several times over, so that
// more loads are in flight; one for a short call.  (28672 x 4096 bf16 to 8 bits 62.6 us with
// two units, 68 with four; float to 4 bits 97.8 with four, back 91 against 98 with two.)
template <bool kBf16, int kBits>
constexpr int kManyUnits = 16 / kLane<kBf16, kBits>;
template <bool kBf16, int kBits>
bool many(int64_t units) { return units >= int64_t(256) * 256 * 4 * kManyUnits<kBf16, kBits>; }

template <bool kBf16, int kBits, int kUnits>
void launch_quantize_units(const void* x, int64_t R, int K, int64_t units, uint8_t* q, uint8_t* scale, int32_t* check,
                           hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(ceil_div(units, 256 * kUnits));
  if (K % mx::kBlock == 0)
    quantize_flat_kernel<kBf16, kBits, kUnits><<<grid, 256, 0, s>>>(x, units, q, scale, check);
  else
    quantize_kernel<kBf16, kBits, kUnits><<<grid, 256, 0, s>>>(x, R, K, static_cast<uint32_t>(ceil_div(K, mx::kBlock)), q,
                                                               scale, check);
}

template <bool kBf16, int kBits>
void launch_quantize(const void* x, int64_t R, int K, uint8_t* q, uint8_t* scale, int32_t* check, hipStream_t s) {
  const int64_t units = R * ceil_div(K, mx::kBlock) * (mx::kBlock / kLane<kBf16, kBits>);
  if (many<kBf16, kBits>(units)) launch_quantize_units<kBf16, kBits, kManyUnits<kBf16, kBits>>(x, R, K, units, q, scale, check, s);
  else launch_quantize_units<kBf16, kBits, 1>(x, R, K, units, q, scale, check, s);
}

template <bool kBf16, int kBits, int kUnits>
void launch_dequantize_units(const uint8_t* q, const uint8_t* scale, int64_t R, int K, const int32_t* rows,
                             int64_t n_rows, int64_t units, void* out, int32_t* check, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(ceil_div(units, 256 * kUnits));
  if (!rows && K % mx::kBlock == 0)
    dequantize_flat_kernel<kBf16, kBits, kUnits><<<grid, 256, 0, s>>>(q, scale, units, out);
  else
    dequantize_kernel<kBf16, kBits, kUnits><<<grid, 256, 0, s>>>(q, scale, R, K, static_cast<uint32_t>(ceil_div(K, mx::kBlock)),
                                                                 rows, n_rows, out, check);
}

template <bool kBf16, int kBits>
void launch_dequantize(const uint8_t* q, const uint8_t* scale, int64_t R, int K, const int32_t* rows, int64_t n_rows,
                       void* out, int32_t* check, hipStream_t s) {
  const int64_t units = n_rows * ceil_div(K, mx::kBlock) * (mx::kBlock / kLane<kBf16, kBits>);
  if (many<kBf16, kBits>(units)) launch_dequantize_units<kBf16, kBits, kManyUnits<kBf16, kBits>>(q, scale, R, K, rows, n_rows, units, out, check, s);
  else launch_dequantize_units<kBf16, kBits, 1>(q, scale, R, K, rows, n_rows, units, out, check, s);
}

template <bool kBf16, bool kKept, int KK>
void launch_combine_backward(const void* d_out, const void* y, const uint8_t* y_scale, int64_t M, const int32_t* inv_pos,
                             const float* topk_w, int64_t T, int k, int H, void* d_y, float* d_topk_w, int32_t* check,
                             hipStream_t s) {
  if constexpr (KK < moe::kMaxTopK)
    if (k != KK)
      return launch_combine_backward<kBf16, kKept, KK + 1>(d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, d_y, d_topk_w,
                                                           check, s);
  const uint32_t blocks = static_cast<uint32_t>(ceil_div(H, mx::kBlock));
  // a wave a token once there are waves for every SIMD; else a block a token
  if (T >= 4096)
    combine_backward_kernel<kBf16, kKept, 1, KK><<<static_cast<unsigned>(ceil_div(T, 4)), 256, 0, s>>>(
        d_out, y, y_scale, M, inv_pos, topk_w, T, H, blocks, d_y, d_topk_w, check);
  else
    combine_backward_kernel<kBf16, kKept, 4, KK><<<static_cast<unsigned>(T), 256, 0, s>>>(
        d_out, y, y_scale, M, inv_pos, topk_w, T, H, blocks, d_y, d_topk_w, check);
}

}  // namespace

extern "C" int moe_mx_quantize(const void* x, moe_dtype dt, int64_t R, int64_t K, moe_mx_format fmt, uint8_t* q,
                               uint8_t* scale, int32_t* check, void* stream) {
  using namespace moe;
  if (int rc = check_format("moe_mx_quantize", dt, fmt, R, K)) return rc;
  if (R == 0) return MOE_OK;
  if (!x || !q || !scale) return fail(MOE_ERR_INVALID_ARG, "moe_mx_quantize: null pointer");
  const hipStream_t s = as_stream(stream);
  const int k = static_cast<int>(K);
  auto launch = [&](auto bits) {
    if (dt == MOE_BF16) launch_quantize<true, decltype(bits)::value>(x, R, k, q, scale, check, s);
    else launch_quantize<false, decltype(bits)::value>(x, R, k, q, scale, check, s);
  };
  if (fmt == MOE_MX_FP8) launch(std::integral_constant<int, mx::kF8>{});
  else if (fmt == MOE_MX_FP6) launch(std::integral_constant<int, mx::kF6>{});
  else launch(std::integral_constant<int, mx::kF4>{});
  return hip_status(hipGetLastError(), "moe_mx_quantize launch");
}

extern "C" int moe_mx_dequantize(const uint8_t* q, const uint8_t* scale, moe_mx_format fmt, int64_t R, int64_t K,
                                 const int32_t* rows, int64_t n_rows, moe_dtype dt, void* out, int32_t* check,
                                 void* stream) {
  using namespace moe;
  if (int rc = check_format("moe_mx_dequantize", dt, fmt, R, K)) return rc;
  if (!rows) n_rows = R;
  if (int rc = check_format("moe_mx_dequantize", dt, fmt, n_rows, K)) return rc;
  if (n_rows == 0) return MOE_OK;
  if (!out || (R > 0 && (!q || !scale))) return fail(MOE_ERR_INVALID_ARG, "moe_mx_dequantize: null pointer");
  const hipStream_t s = as_stream(stream);
  const int k = static_cast<int>(K);
  auto launch = [&](auto bits) {
    if (dt == MOE_BF16) launch_dequantize<true, decltype(bits)::value>(q, scale, R, k, rows, n_rows, out, check, s);
    else launch_dequantize<false, decltype(bits)::value>(q, scale, R, k, rows, n_rows, out, check, s);
  };
  if (fmt == MOE_MX_FP8) launch(std::integral_constant<int, mx::kF8>{});
  else if (fmt == MOE_MX_FP6) launch(std::integral_constant<int, mx::kF6>{});
  else launch(std::integral_constant<int, mx::kF4>{});
  return hip_status(hipGetLastError(), "moe_mx_dequantize launch");
}

extern "C" int moe_combine_backward(const void* d_out, moe_dtype dt, const void* y, const uint8_t* y_scale, int64_t M,
                                    const int32_t* inv_pos, const float* topk_w, int64_t T, int k, int H, void* d_y,
                                    float* d_topk_w, int32_t* check, void* stream) {
  using namespace moe;
  if (dt != MOE_F32 && dt != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "moe_combine_backward: unknown dtype %d", (int)dt);
  if (k < 1 || k > kMaxTopK) return fail(MOE_ERR_INVALID_ARG, "moe_combine_backward: k=%d outside [1, 8]", k);
  if (T < 0 || M < 0 || T * k >= (int64_t(1) << 31)) return fail(MOE_ERR_INVALID_ARG, "moe_combine_backward: bad T or M");
  if (H < 8 || H % 8 || H > (1 << 28))
    return fail(MOE_ERR_INVALID_ARG, "moe_combine_backward: H must be a positive multiple of 8 (H=%d)", H);
  if (T > (int64_t(1) << 25)) return fail(MOE_ERR_UNSUPPORTED, "moe_combine_backward: more than 2^25 tokens");
  if (T == 0) return MOE_OK;
  if (!d_out || !inv_pos || !topk_w || !d_topk_w || (M > 0 && (!y || !d_y)))
    return fail(MOE_ERR_INVALID_ARG, "moe_combine_backward: null pointer");
  for (const void* p : {d_out, y, static_cast<const void*>(d_y)})
    if (p && !aligned16(p)) return fail(MOE_ERR_INVALID_ARG, "moe_combine_backward: rows must be 16-byte aligned");
  const hipStream_t s = as_stream(stream);
  if (dt == MOE_BF16) {
    if (y_scale) launch_combine_backward<true, true, 1>(d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, d_y, d_topk_w, check, s);
    else launch_combine_backward<true, false, 1>(d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, d_y, d_topk_w, check, s);
  } else {
    if (y_scale) launch_combine_backward<false, true, 1>(d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, d_y, d_topk_w, check, s);
    else launch_combine_backward<false, false, 1>(d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, d_y, d_topk_w, check, s);
  }
  return hip_status(hipGetLastError(), "moe_combine_backward launch");
}
