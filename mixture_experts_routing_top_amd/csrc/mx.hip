// moe_mx_quantize, moe_mx_dequantize: rows to blocks of 32 values with one
// power-of-two scale, in 4, 6 or 8 bits, and the values that they stand for back
// again (by a row map, as a dispatch copies rows).  moe_combine_backward: the
// gradient of the weighted combine, from expert outputs in the dtype or kept in
// 8-bit blocks.
//
// All three are bound by memory: every value is read once and written once, eight
// values a lane, in accesses that a wave makes to one run of addresses.  mx.h has the format and the split of a row over lanes.
#include <type_traits>

#include "common.h"
#include "mx.h"
#include "rows.h"

namespace {

using moe::ceil_div;
using namespace rows;

template <bool kBf16, int kBits, int kUnits>
__global__ __launch_bounds__(256) void quantize_kernel(const void* __restrict__ x, int64_t R, int K, uint32_t blocks,
                                                       uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                                       int32_t* __restrict__ check) {
  const mx::Units<kUnits> units(blockIdx.x, 4 * blocks);
  const int64_t row_bytes = mx::code_bytes(kBits, K);
  Raw8<kBf16> raw[kUnits];
  int64_t row[kUnits];
  uint32_t unit[kUnits];
  int n[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    units.at(j, &row[j], &unit[j]);
    n[j] = row[j] < R ? max(0, min(8, K - static_cast<int>(unit[j] * 8))) : 0;
    raw[j] = Raw8<kBf16>{};
    if (n[j] > 0) raw[j] = load8_part<kBf16>(x, row[j] * K + unit[j] * 8, n[j]);
  }
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    float v[8];
    unpack8<kBf16>(raw[j], v);
    const uint32_t byte = mx::quad_scale<kBits>(v);   // (a block's four lanes are in one row, or past the last)
    bad |= byte == 255;
    const uint2 c = mx::encode8<kBits>(v, byte);
    if (row[j] >= R) continue;
    if ((unit[j] & 3) == 0) scale[row[j] * blocks + (unit[j] >> 2)] = static_cast<uint8_t>(byte);
    uint8_t* p = q + row[j] * row_bytes + static_cast<int64_t>(unit[j]) * kBits;
    const int bytes = static_cast<int>(mx::code_bytes(kBits, n[j]));
    if (bytes == kBits) {
      __builtin_memcpy(p, &c, kBits);
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
  const mx::Units<kUnits> units(blockIdx.x, 4 * blocks);
  const int64_t row_bytes = mx::code_bytes(kBits, K);
  uint2 c[kUnits];
  uint32_t byte[kUnits], unit[kUnits];
  int64_t row[kUnits];
  int n[kUnits];
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    units.at(j, &row[j], &unit[j]);
    n[j] = row[j] < n_rows ? max(0, min(8, K - static_cast<int>(unit[j] * 8))) : 0;
    c[j] = make_uint2(0, 0);
    byte[j] = 127;
    if (n[j] == 0) continue;
    const int64_t src = map ? map[row[j]] : row[j];
    if (src < 0 || src >= R) {   // such a row is zero
      bad = true;
      continue;
    }
    const uint8_t* p = q + src * row_bytes + static_cast<int64_t>(unit[j]) * kBits;
    const int bytes = static_cast<int>(mx::code_bytes(kBits, n[j]));
    if (bytes == kBits) {
      __builtin_memcpy(&c[j], p, kBits);
    } else {
      for (int u = 0; u < bytes; ++u) (u < 4 ? c[j].x : c[j].y) |= static_cast<uint32_t>(p[u]) << (8 * (u & 3));
    }
    byte[j] = scale[src * blocks + (unit[j] >> 2)];
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    if (n[j] == 0) continue;
    float v[8];
    mx::decode8<kBits>(c[j], byte[j], v);
    store8_part<kBf16>(out, row[j] * K + unit[j] * 8, n[j], v);
  }
  if (check) raise_check(check, bad, MOE_CHECK_ROWS);
}

// d_y[inv[t,i]] = w[t,i] d_out[t] and d_w[t,i] = <d_out[t], y[inv[t,i]]>.  kWaves
// waves a token (kWaves = 1: four tokens a block), eight values of the row and of
// each of its k expert rows a lane and step.
template <bool kBf16, bool kKept, int kWaves>
__global__ __launch_bounds__(256) void combine_backward_kernel(const void* __restrict__ d_out, const void* __restrict__ y,
                                                               const uint8_t* __restrict__ y_scale, int64_t M,
                                                               const int32_t* __restrict__ inv_pos,
                                                               const float* __restrict__ topk_w, int64_t T, int k,
                                                               int H, uint32_t blocks, void* __restrict__ d_y,
                                                               float* __restrict__ d_topk_w,
                                                               int32_t* __restrict__ check) {
  __shared__ float part[4][moe::kMaxTopK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = kWaves == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + wave : blockIdx.x;
  if (kWaves == 1 && t >= T) return;
  int64_t at[moe::kMaxTopK];
  float w[moe::kMaxTopK], acc[moe::kMaxTopK];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < moe::kMaxTopK; ++i) {
    at[i] = -1;
    w[i] = acc[i] = 0.f;
    if (i < k) {
      const int32_t r = inv_pos[t * k + i];
      if (r >= 0 && r < M) at[i] = r;
      else bad = true;
      w[i] = topk_w[t * k + i];
    }
  }
  for (int c = (kWaves == 1 ? 0 : wave * 64) + lane; c * 8 < H; c += kWaves * 64) {
    float o[8];
    unpack8<kBf16>(load8<kBf16>(d_out, t * H + c * 8), o);
#pragma unroll
    for (int i = 0; i < moe::kMaxTopK; ++i) {
      if (i >= k || at[i] < 0) continue;
      float v[8], s = 0.f, p[8];
      float scale = 1.f;
      if constexpr (kKept) {
        uint2 q;
        __builtin_memcpy(&q, static_cast<const uint8_t*>(y) + at[i] * H + c * 8, 8);
        scale = mx::scale_value(y_scale[at[i] * blocks + (c >> 2)]);
        mx::decode8_fp8(q, 1.f, v);
      } else {
        unpack8<kBf16>(load8<kBf16>(y, at[i] * H + c * 8), v);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        s = fmaf(o[u], v[u], s);
        p[u] = w[i] * o[u];
      }
      acc[i] = fmaf(s, scale, acc[i]);
      store8_part<kBf16>(d_y, at[i] * H + c * 8, 8, p);
    }
  }
#pragma unroll
  for (int i = 0; i < moe::kMaxTopK; ++i) {
    if (i >= k) break;
    const float v = wave_sum(acc[i]);
    if constexpr (kWaves == 1) {
      if (lane == 0) d_topk_w[t * k + i] = v;
    } else if (lane == 0) {
      part[wave][i] = v;
    }
  }
  if constexpr (kWaves > 1) {
    __syncthreads();
    if (threadIdx.x < k) {
      float v = part[0][threadIdx.x];
#pragma unroll
      for (int u = 1; u < kWaves; ++u) v += part[u][threadIdx.x];
      d_topk_w[t * k + threadIdx.x] = v;
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
  if (R > (int64_t(1) << 31) / ceil_div(K, mx::kBlock))
    return fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^31 blocks of 32 values", who);
  return MOE_OK;
}

// Units a thread: four once that still fills the card several times over, so that
// more loads are in flight; one for a short call.
constexpr int kManyUnits = 4;
bool many(int64_t units) { return units >= int64_t(256) * 256 * kManyUnits * 4; }

template <bool kBf16, int kBits>
void launch_quantize(const void* x, int64_t R, int K, uint8_t* q, uint8_t* scale, int32_t* check, hipStream_t s) {
  const uint32_t blocks = static_cast<uint32_t>(ceil_div(K, mx::kBlock));
  const int64_t units = R * blocks * 4;
  if (many(units))
    quantize_kernel<kBf16, kBits, kManyUnits><<<static_cast<unsigned>(ceil_div(units, 256 * kManyUnits)), 256, 0, s>>>(
        x, R, K, blocks, q, scale, check);
  else
    quantize_kernel<kBf16, kBits, 1><<<static_cast<unsigned>(ceil_div(units, 256)), 256, 0, s>>>(x, R, K, blocks, q, scale,
                                                                                               check);
}

template <bool kBf16, int kBits>
void launch_dequantize(const uint8_t* q, const uint8_t* scale, int64_t R, int K, const int32_t* rows, int64_t n_rows,
                       void* out, int32_t* check, hipStream_t s) {
  const uint32_t blocks = static_cast<uint32_t>(ceil_div(K, mx::kBlock));
  const int64_t units = n_rows * blocks * 4;
  if (many(units))
    dequantize_kernel<kBf16, kBits, kManyUnits><<<static_cast<unsigned>(ceil_div(units, 256 * kManyUnits)), 256, 0, s>>>(
        q, scale, R, K, blocks, rows, n_rows, out, check);
  else
    dequantize_kernel<kBf16, kBits, 1><<<static_cast<unsigned>(ceil_div(units, 256)), 256, 0, s>>>(
        q, scale, R, K, blocks, rows, n_rows, out, check);
}

template <bool kBf16, bool kKept>
void launch_combine_backward(const void* d_out, const void* y, const uint8_t* y_scale, int64_t M, const int32_t* inv_pos,
                             const float* topk_w, int64_t T, int k, int H, void* d_y, float* d_topk_w, int32_t* check,
                             hipStream_t s) {
  const uint32_t blocks = static_cast<uint32_t>(ceil_div(H, mx::kBlock));
  // a wave a token once there are waves for every SIMD; else a block a token
  if (T >= 4096)
    combine_backward_kernel<kBf16, kKept, 1><<<static_cast<unsigned>(ceil_div(T, 4)), 256, 0, s>>>(
        d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, blocks, d_y, d_topk_w, check);
  else
    combine_backward_kernel<kBf16, kKept, 4><<<static_cast<unsigned>(T), 256, 0, s>>>(
        d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, blocks, d_y, d_topk_w, check);
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
  if (T == 0) return MOE_OK;
  if (!d_out || !inv_pos || !topk_w || !d_topk_w || (M > 0 && (!y || !d_y)))
    return fail(MOE_ERR_INVALID_ARG, "moe_combine_backward: null pointer");
  for (const void* p : {d_out, y, static_cast<const void*>(d_y)})
    if (p && !aligned16(p)) return fail(MOE_ERR_INVALID_ARG, "moe_combine_backward: rows must be 16-byte aligned");
  const hipStream_t s = as_stream(stream);
  if (dt == MOE_BF16) {
    if (y_scale) launch_combine_backward<true, true>(d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, d_y, d_topk_w, check, s);
    else launch_combine_backward<true, false>(d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, d_y, d_topk_w, check, s);
  } else {
    if (y_scale) launch_combine_backward<false, true>(d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, d_y, d_topk_w, check, s);
    else launch_combine_backward<false, false>(d_out, y, y_scale, M, inv_pos, topk_w, T, k, H, d_y, d_topk_w, check, s);
  }
  return hip_status(hipGetLastError(), "moe_combine_backward launch");
}
