// moe_layer_norm, moe_layer_norm_backward: layer norm of rows, with the
// residual sum before it.
//
//   s = x + residual (rounded to the dtype, written to x_sum), or s = x
//   y = (s - mean) rstd weight + bias, rstd = 1 / sqrt(var + eps)
// backward, with s^ = (s - mean) rstd and g = d_y weight:
//   d_x = rstd (g - mean(g) - s^ mean(g s^)) + d_skip
//   d_weight = sum over rows of d_y s^,  d_bias = sum over rows of d_y
//
// HBM-bound: each row is read once into registers and written once.  The mean
// is taken first and the variance from the deviations; the sum of the
// deviations corrects the mean's own rounding, so a row whose mean is large
// against its spread keeps full precision.  The backward pass forms the
// statistics again from s (the row is in registers anyway) instead of reading
// saved ones.  8192 x 4096 bf16 (profiler, inputs out of cache): with residual 44 us for
// 268 MB, of which the rows written last may still lie in the last-level cache when it
// ends (51 us a call in a run of them: 5.3 TB/s); backward with d_skip 57 us for the same
// and 7 for the columns' sums.
//
// TPR threads own a row, NV pieces of 8 consecutive elements each.  A block
// keeps its columns of weight and bias (and the backward's column sums) in
// registers over the rows it walks.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "rows.h"

namespace {

using namespace rows;

constexpr int kMaxH = 16384;

// Sums of N values over the TPR threads of a row; `part` is this reduction's
// own LDS, [row of the block][wave of the row][N].  One barrier (none for rows
// of one wave): two reductions of a row use two buffers, so a buffer is free
// again once the other one's barrier is passed.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* part) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* mine = part + (threadIdx.x / TPR) * (W * N);
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) mine[((threadIdx.x % TPR) / 64) * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[i] += mine[w * N + i];
    }
  }
}

struct NormArgs {
  const void* x;
  const void* residual;
  const void* weight;
  const void* bias;
  void* x_sum;
  void* y;
  int64_t T;
  int H;
  float eps;
};

// n of eight elements from p, the rest zero; `fill` throughout where there is no p
template <bool kBf16>
__device__ __forceinline__ void load_piece(const void* p, int64_t at, int n, float fill, float (&v)[8]) {
  if (p && n > 0) unpack8<kBf16>(load8_part<kBf16>(p, at, n), v);
  else
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = fill;
}

template <bool kWBf16, int TPR, int NV>
__device__ __forceinline__ void load_vector(const void* p, int tid, int H, float fill, float (&v)[NV][8]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) load_piece<kWBf16>(p, (j * TPR + tid) * 8, H - (j * TPR + tid) * 8, fill, v[j]);
}

// a row's pieces as they lie in memory
template <bool kBf16, int NV>
struct RawRow {
  Raw8<kBf16> piece[NV];
};

template <bool kBf16, int TPR, int NV>
__device__ __forceinline__ void load_row(const void* p, int64_t row, int64_t T, int H, int tid,
                                         RawRow<kBf16, NV>& r) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tid) * 8;
    r.piece[j] = {};
    if (p && row < T && c < H) r.piece[j] = load8_part<kBf16>(p, row * H + c, H - c);
  }
}

// Blocks a CU is given of the forward kernel, by the registers the float32 kernel needs
// with a row ahead: 6 waves a SIMD with one piece a thread, 4 with two (the bf16 kernel
// takes fewer and would leave room for more).  The launch has just as
// many, and the next row is loaded while one is reduced: 8192 x 4096 bf16 with
// residual takes 47 us (5.7 TB/s), without the row ahead 50 on 5 blocks a CU, 56 on
// 4, 57 on 8 and 62 on a block for each row; 4096 x 8192 takes 46 against 55.
constexpr int fwd_blocks_per_cu(int tpr, int nv) { return tpr == 1024 ? 1 : tpr == 512 ? 2 : nv == 1 ? 6 : 4; }

template <bool kBf16, bool kWBf16, int TPR, int NV, int R>
__global__ __launch_bounds__(TPR* R, fwd_blocks_per_cu(TPR, NV)) void norm_kernel(NormArgs p) {
  __shared__ float part[2][R * (TPR / 64) * 2];
  const int tid = threadIdx.x % TPR, r = threadIdx.x / TPR;
  float w[NV][8], b[NV][8];
  load_vector<kWBf16, TPR, NV>(p.weight, tid, p.H, 1.f, w);
  load_vector<kWBf16, TPR, NV>(p.bias, tid, p.H, 0.f, b);
  const float inv_h = 1.f / static_cast<float>(p.H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  RawRow<kBf16, NV> xr, rr;
  load_row<kBf16, TPR, NV>(p.x, static_cast<int64_t>(blockIdx.x) * R + r, p.T, p.H, tid, xr);
  load_row<kBf16, TPR, NV>(p.residual, static_cast<int64_t>(blockIdx.x) * R + r, p.T, p.H, tid, rr);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * R; base < p.T; base += step) {
    const int64_t row = base + r;
    const bool active = row < p.T;
    const int64_t at = (active ? row : 0) * p.H;
    float v[NV][8];
    float sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tid) * 8;
      const int n = active ? p.H - c : 0;
      unpack8<kBf16>(xr.piece[j], v[j]);
      if (n > 0) {
        if (p.residual) {
          float q[8];
          unpack8<kBf16>(rr.piece[j], q);
#pragma unroll
          for (int u = 0; u < 8; ++u) v[j][u] += q[u];
          const Raw8<kBf16> s = pack8<kBf16>(v[j]);  // the sum as it is kept
          unpack8<kBf16>(s, v[j]);
          store8_part<kBf16>(p.x_sum, at + c, n, v[j]);
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) sum[0] += v[j][u];
    }
    // the next row is on its way while this one is reduced
    load_row<kBf16, TPR, NV>(p.x, row + step, p.T, p.H, tid, xr);
    load_row<kBf16, TPR, NV>(p.residual, row + step, p.T, p.H, tid, rr);
    row_sum<TPR, 1>(sum, part[0]);
    const float mean = sum[0] * inv_h;
    float dev[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = p.H - (j * TPR + tid) * 8;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        v[j][u] = u < n ? v[j][u] - mean : 0.f;
        dev[0] += v[j][u];
        dev[1] = fmaf(v[j][u], v[j][u], dev[1]);
      }
    }
    row_sum<TPR, 2>(dev, part[1]);
    const float shift = dev[0] * inv_h;
    const float var = fmaxf(fmaf(-shift, shift, dev[1] * inv_h), 0.f);
    const float rstd = 1.f / sqrtf(var + p.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tid) * 8;
      const int n = active ? p.H - c : 0;
      if (n <= 0) continue;
#pragma unroll
      for (int u = 0; u < 8; ++u) v[j][u] = fmaf((v[j][u] - shift) * rstd, w[j][u], b[j][u]);
      store8_part<kBf16>(p.y, at + c, n, v[j]);
    }
  }
}

// ------------------------------------------------------------------ backward
struct NormBwdArgs {
  const void* d_y;
  const void* x;
  const void* weight;
  const void* d_skip;
  void* d_x;
  float* partial;  // [blocks][2][Hp]: column sums of d_y s^ and d_y over a block's rows
  int64_t T;
  int H, Hp;
  float eps;
};

// Blocks a CU is given of the backward kernel, by the registers the float32 kernel needs:
// 4 waves a SIMD with one piece a thread, else 2 (179 - 182 registers; the bf16 kernel takes
// 152 and would fit three).
constexpr int bwd_blocks_per_cu(int tpr, int nv) { return tpr > 256 ? 1 : nv == 1 ? 4 : 2; }

template <bool kBf16, bool kWBf16, int TPR, int NV, int R>
__global__ __launch_bounds__(TPR* R, bwd_blocks_per_cu(TPR, NV)) void norm_backward_kernel(NormBwdArgs p) {
  __shared__ float part[2][R * (TPR / 64) * 4];
  __shared__ float cols[R > 1 ? 2 * NV * 8 * TPR : 1];
  const int tid = threadIdx.x % TPR, r = threadIdx.x / TPR;
  // the widest rows leave no registers for a row ahead; their weight is read per row
  constexpr bool kAhead = NV <= 2;
  float w[NV][8], dw[NV][8], db[NV][8];
  if constexpr (kAhead) load_vector<kWBf16, TPR, NV>(p.weight, tid, p.H, 1.f, w);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int u = 0; u < 8; ++u) dw[j][u] = db[j][u] = 0.f;
  const float inv_h = 1.f / static_cast<float>(p.H);
  const int64_t step = static_cast<int64_t>(gridDim.x) * R;
  RawRow<kBf16, NV> xr, gr, sr, sr_now;
  if constexpr (kAhead) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * R + r;
    load_row<kBf16, TPR, NV>(p.x, row, p.T, p.H, tid, xr);
    load_row<kBf16, TPR, NV>(p.d_y, row, p.T, p.H, tid, gr);
    load_row<kBf16, TPR, NV>(p.d_skip, row, p.T, p.H, tid, sr);
  }
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * R; base < p.T; base += step) {
    const int64_t row = base + r;
    const bool active = row < p.T;
    if constexpr (!kAhead) {
      load_row<kBf16, TPR, NV>(p.x, row, p.T, p.H, tid, xr);
      load_row<kBf16, TPR, NV>(p.d_y, row, p.T, p.H, tid, gr);
    }
    float v[NV][8], g[NV][8];
    float sum[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      unpack8<kBf16>(xr.piece[j], v[j]);
      unpack8<kBf16>(gr.piece[j], g[j]);
#pragma unroll
      for (int u = 0; u < 8; ++u) sum[0] += v[j][u];
    }
    // the next row is on its way while this one is reduced
    if constexpr (kAhead) {
      sr_now = sr;
      load_row<kBf16, TPR, NV>(p.x, row + step, p.T, p.H, tid, xr);
      load_row<kBf16, TPR, NV>(p.d_y, row + step, p.T, p.H, tid, gr);
      load_row<kBf16, TPR, NV>(p.d_skip, row + step, p.T, p.H, tid, sr);
    }
    row_sum<TPR, 1>(sum, part[0]);
    const float mean = sum[0] * inv_h;
    // sums of the deviations, their squares, g and g times the deviation
    float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = p.H - (j * TPR + tid) * 8;
      if constexpr (!kAhead) load_piece<kWBf16>(p.weight, p.H - n, n, 1.f, w[j]);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        v[j][u] = u < n ? v[j][u] - mean : 0.f;
        const float gw = g[j][u] * w[j][u];
        q[0] += v[j][u];
        q[1] = fmaf(v[j][u], v[j][u], q[1]);
        q[2] += gw;
        q[3] = fmaf(gw, v[j][u], q[3]);
      }
    }
    row_sum<TPR, 4>(q, part[1]);
    const float shift = q[0] * inv_h;
    const float rstd = 1.f / sqrtf(fmaxf(fmaf(-shift, shift, q[1] * inv_h), 0.f) + p.eps);
    const float c1 = q[2] * inv_h;
    const float c2 = rstd * fmaf(-shift, q[2], q[3]) * inv_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + tid) * 8;
      const int n = active ? p.H - c : 0;
      if (n <= 0) continue;
      float d[8];
      if constexpr (kAhead) {
        unpack8<kBf16>(sr_now.piece[j], d);
      } else {
        load_piece<kBf16>(p.d_skip, row * p.H + c, n, 0.f, d);
        load_piece<kWBf16>(p.weight, c, n, 1.f, w[j]);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float hat = (v[j][u] - shift) * rstd;
        d[u] += rstd * (fmaf(g[j][u], w[j][u], -c1) - hat * c2);
        dw[j][u] = fmaf(g[j][u], hat, dw[j][u]);
        db[j][u] += g[j][u];
      }
      store8_part<kBf16>(p.d_x, row * p.H + c, n, d);
    }
  }
  if (!p.partial) return;
  // the block's rows together, in row order
  if constexpr (R > 1) {
    for (int k = 1; k < R; ++k) {
      __syncthreads();
      if (r == k)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            cols[((j * 8 + u) * 2) * TPR + tid] = dw[j][u];
            cols[((j * 8 + u) * 2 + 1) * TPR + tid] = db[j][u];
          }
      __syncthreads();
      if (r == 0)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            dw[j][u] += cols[((j * 8 + u) * 2) * TPR + tid];
            db[j][u] += cols[((j * 8 + u) * 2 + 1) * TPR + tid];
          }
    }
    if (r != 0) return;
  }
  float* out = p.partial + static_cast<int64_t>(blockIdx.x) * 2 * p.Hp;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TPR + tid) * 8;
    if (c >= p.Hp) continue;
    store8_part<false>(out, c, 8, dw[j]);
    store8_part<false>(out + p.Hp, c, 8, db[j]);
  }
}

// d_weight and d_bias from the blocks' column sums: 16 columns of one of the two
// per block, 4 threads of 4 columns by 64 groups of blocks, added in a fixed order.
template <bool kWBf16>
__global__ __launch_bounds__(256) void norm_columns_kernel(const float* __restrict__ partial, int blocks, int H,
                                                           int Hp, void* __restrict__ d_weight,
                                                           void* __restrict__ d_bias) {
  __shared__ float4 part[64][4];
  void* out = blockIdx.y ? d_bias : d_weight;
  if (!out) return;
  const int x = threadIdx.x & 3, y = threadIdx.x >> 2;
  const int c = blockIdx.x * 16 + x * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < Hp) {
    const float* col = partial + static_cast<int64_t>(blockIdx.y) * Hp + c;
#pragma unroll 4
    for (int b = y; b < blocks; b += 64) {
      const float4 v = *reinterpret_cast<const float4*>(col + static_cast<int64_t>(b) * 2 * Hp);
      a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
    }
  }
  part[y][x] = a;
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) {
    __syncthreads();
    if (y < s) {
      const float4 v = part[y + s][x];
      a.x += v.x; a.y += v.y; a.z += v.z; a.w += v.w;
      part[y][x] = a;
    }
  }
  if (y != 0) return;
  const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (c + u < H) store1<kWBf16>(out, c + u, v[u]);
}

// Threads per row and pieces a thread for a width.  In the widest rows the forward
// pass takes 16 waves with 2 pieces (bf16 2048 x 16384, before the row ahead: 69 us,
// 8 waves with 4: 90), the backward pass, whose sums then spill, 8 waves with 4 (99 us
// against 125).
struct Shape {
  int tpr, nv;
};
Shape shape_of(int H, bool backward) {
  if (H <= 512) return {64, 1};
  if (H <= 1024) return {64, 2};
  if (H <= 2048) return {256, 1};
  if (H <= 4096) return {256, 2};
  if (H <= 8192) return {512, 2};
  return backward ? Shape{512, 4} : Shape{1024, 2};
}

constexpr int kFwdThreads = 256, kBwdThreads = 256;
constexpr int kCUs = 256;

// As many blocks as the CUs are given at once, so that none waits for another.  Where
// the rows do not fill them, three rows a thread group from 128 blocks on: each block
// costs a row of column sums, written and read again (bf16 1024 x 2048: 20.7 us with
// one row each, 15.1 with three; 300 x 5120: 19.4, 15.5; 64 x 4096: 8.6, 10.9).
int bwd_blocks(int64_t T, int H) {
  const Shape sh = shape_of(H, true);
  const int64_t one = moe::ceil_div(T, std::max(1, kBwdThreads / sh.tpr));
  const int64_t blocks = std::max(std::min<int64_t>(one, 128), moe::ceil_div(one, 3));
  return static_cast<int>(std::min<int64_t>(kCUs * bwd_blocks_per_cu(sh.tpr, sh.nv), blocks));
}
int padded(int H) { return static_cast<int>(moe::ceil_div(H, 8) * 8); }

template <bool kBf16, bool kWBf16, int TPR, int NV>
void launch_norm(const NormArgs& p, hipStream_t s) {
  constexpr int R = TPR >= kFwdThreads ? 1 : kFwdThreads / TPR;
  constexpr int64_t kBlocks = kCUs * fwd_blocks_per_cu(TPR, NV);
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(kBlocks, moe::ceil_div(p.T, R)));
  norm_kernel<kBf16, kWBf16, TPR, NV, R><<<blocks, TPR * R, 0, s>>>(p);
}

template <bool kBf16, bool kWBf16, int TPR, int NV>
void launch_norm_backward(const NormBwdArgs& p, hipStream_t s) {
  constexpr int R = TPR >= kBwdThreads ? 1 : kBwdThreads / TPR;
  norm_backward_kernel<kBf16, kWBf16, TPR, NV, R><<<bwd_blocks(p.T, p.H), TPR * R, 0, s>>>(p);
}

#define MOE_NORM_BY_SHAPE(fn, backward, a, b)                                  \
  switch (const Shape sh = shape_of(p.H, backward); sh.tpr * 8 + sh.nv) {      \
    case 64 * 8 + 1: fn<a, b, 64, 1>(p, s); break;                             \
    case 64 * 8 + 2: fn<a, b, 64, 2>(p, s); break;                             \
    case 256 * 8 + 1: fn<a, b, 256, 1>(p, s); break;                           \
    case 256 * 8 + 2: fn<a, b, 256, 2>(p, s); break;                           \
    case 512 * 8 + 2: fn<a, b, 512, 2>(p, s); break;                           \
    default: fn<a, b, backward ? 512 : 1024, backward ? 4 : 2>(p, s); break;   \
  }

int check_norm(const char* who, moe_dtype dt, moe_dtype w_dt, int64_t T, int H, float eps) {
  using namespace moe;
  if (dt != MOE_F32 && dt != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dt);
  if (w_dt != MOE_F32 && w_dt != dt)
    return fail(MOE_ERR_INVALID_ARG, "%s: weight and bias must be float32 or of the rows' dtype", who);
  if (H < 1) return fail(MOE_ERR_INVALID_ARG, "%s: H=%d", who, H);
  if (H > kMaxH) return fail(MOE_ERR_UNSUPPORTED, "%s: H=%d beyond %d", who, H, kMaxH);
  if (T < 0 || T >= (int64_t(1) << 40)) return fail(MOE_ERR_INVALID_ARG, "%s: T=%lld out of range", who, (long long)T);
  if (!(eps > 0.f) || !std::isfinite(eps)) return fail(MOE_ERR_INVALID_ARG, "%s: eps must be positive and finite", who);
  return MOE_OK;
}

bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

extern "C" int moe_layer_norm(const void* x, const void* residual, moe_dtype dt, int64_t T, int H, const void* weight,
                              const void* bias, moe_dtype w_dt, float eps, void* x_sum, void* y, void* stream) {
  using namespace moe;
  if (int rc = check_norm("moe_layer_norm", dt, w_dt, T, H, eps)) return rc;
  if ((residual != nullptr) != (x_sum != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "moe_layer_norm: residual and x_sum come together");
  if (T == 0) return MOE_OK;
  if (!x || !y) return fail(MOE_ERR_INVALID_ARG, "moe_layer_norm: null pointer");
  if (x_sum == y) return fail(MOE_ERR_INVALID_ARG, "moe_layer_norm: x_sum and y are the same buffer");
  for (const void* q : {x, residual, static_cast<const void*>(x_sum), static_cast<const void*>(y)})
    if (!aligned_to(q, elem_bytes(dt))) return fail(MOE_ERR_INVALID_ARG, "moe_layer_norm: misaligned rows");
  if (!aligned_to(weight, elem_bytes(w_dt)) || !aligned_to(bias, elem_bytes(w_dt)))
    return fail(MOE_ERR_INVALID_ARG, "moe_layer_norm: misaligned weight or bias");
  const NormArgs p{x, residual, weight, bias, x_sum, y, T, H, eps};
  const hipStream_t s = as_stream(stream);
  if (dt == MOE_F32) { MOE_NORM_BY_SHAPE(launch_norm, false, false, false) }
  else if (w_dt == MOE_F32) { MOE_NORM_BY_SHAPE(launch_norm, false, true, false) }
  else { MOE_NORM_BY_SHAPE(launch_norm, false, true, true) }
  return hip_status(hipGetLastError(), "moe_layer_norm launch");
}

extern "C" size_t moe_layer_norm_backward_workspace_bytes(int64_t T, int H) {
  if (T < 0 || H < 1 || H > kMaxH) return 0;
  return static_cast<size_t>(bwd_blocks(T, H)) * 2 * padded(H) * sizeof(float);
}

extern "C" int moe_layer_norm_backward(const void* d_y, const void* x, moe_dtype dt, int64_t T, int H,
                                       const void* weight, moe_dtype w_dt, float eps, const void* d_skip, void* d_x,
                                       void* d_weight, void* d_bias, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  using namespace moe;
  if (int rc = check_norm("moe_layer_norm_backward", dt, w_dt, T, H, eps)) return rc;
  const size_t need = moe_layer_norm_backward_workspace_bytes(T, H);
  const bool columns = d_weight || d_bias;
  if (T > 0 && (!d_y || !x || !d_x)) return fail(MOE_ERR_INVALID_ARG, "moe_layer_norm_backward: null pointer");
  for (const void* q : {d_y, x, d_skip, static_cast<const void*>(d_x)})
    if (!aligned_to(q, elem_bytes(dt))) return fail(MOE_ERR_INVALID_ARG, "moe_layer_norm_backward: misaligned rows");
  for (const void* q : {weight, static_cast<const void*>(d_weight), static_cast<const void*>(d_bias)})
    if (!aligned_to(q, elem_bytes(w_dt)))
      return fail(MOE_ERR_INVALID_ARG, "moe_layer_norm_backward: misaligned weight, d_weight or d_bias");
  if (columns && T > 0) {
    if (!workspace || workspace_bytes < need)
      return fail(MOE_ERR_WORKSPACE, "moe_layer_norm_backward: workspace has %zu bytes, needs %zu",
                  workspace ? workspace_bytes : size_t(0), need);
    if (!aligned16(workspace))
      return fail(MOE_ERR_INVALID_ARG, "moe_layer_norm_backward: workspace must be 16-byte aligned");
  }
  const hipStream_t s = as_stream(stream);
  const int blocks = bwd_blocks(T, H);
  if (T > 0) {
    const NormBwdArgs p{d_y, x, weight, d_skip, d_x, columns ? static_cast<float*>(workspace) : nullptr,
                        T, H, padded(H), eps};
    if (dt == MOE_F32) { MOE_NORM_BY_SHAPE(launch_norm_backward, true, false, false) }
    else if (w_dt == MOE_F32) { MOE_NORM_BY_SHAPE(launch_norm_backward, true, true, false) }
    else { MOE_NORM_BY_SHAPE(launch_norm_backward, true, true, true) }
    if (int rc = hip_status(hipGetLastError(), "moe_layer_norm_backward launch")) return rc;
  }
  if (columns) {
    const dim3 grid(static_cast<unsigned>(ceil_div(H, 16)), 2);
    const float* part = static_cast<const float*>(workspace);
    if (w_dt == MOE_BF16) norm_columns_kernel<true><<<grid, 256, 0, s>>>(part, blocks, H, padded(H), d_weight, d_bias);
    else norm_columns_kernel<false><<<grid, 256, 0, s>>>(part, blocks, H, padded(H), d_weight, d_bias);
    if (int rc = hip_status(hipGetLastError(), "moe_layer_norm_backward columns")) return rc;
  }
  return MOE_OK;
}
