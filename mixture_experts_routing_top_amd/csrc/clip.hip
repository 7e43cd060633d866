// moe_grad_norm, moe_clip_grads: the global norm of many gradients, and the
// gradients scaled so that it is at most max_norm.
//
//   norm = sqrt(sum over all tensors of all squares)
//   out = g * min(1, max_norm / (norm + eps))
//
// HBM-bound: everything is read for the norm before anything can be scaled, so
// a clip moves 2 reads and 1 write.  The product of two floats is exact in
// double, and double adds run at the vector rate here: squares neither
// overflow nor vanish, and the sum is in double, in a fixed order (no atomics).
//
// The list travels in the kernel arguments, up to kList tensors a launch, so a
// call can be captured into a graph and needs no device copy of it.  Tensors
// are cut into chunks of kChunk elements dealt to the blocks in turn.  Block b
// of every launch adds to slot b of the workspace; the scaling launches sum the
// slots again in each block, which saves a launch between the two passes.
#include <algorithm>
#include <cmath>
#include <new>

#include "common.h"
#include "rows.h"

namespace {

using namespace rows;

constexpr int kList = 96;       // tensors per launch: 2.8 KB of kernel arguments
constexpr int kChunk = 8192;    // elements
constexpr int kSlots = 1024;    // blocks per launch, partial sums
constexpr int kThreads = 256;

struct GradList {
  const void* in[kList];
  void* out[kList];
  int64_t numel[kList];
  int32_t first[kList + 1];  // chunks before tensor i
  uint32_t bf16[kList / 32];
  int count;
};

// tensor and element range of a chunk; `at` is the tensor of the chunk before it
__device__ __forceinline__ int chunk_of(const GradList& l, int chunk, int at) {
  while (chunk >= l.first[at + 1]) ++at;
  return at;
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

__device__ __forceinline__ double block_sum64(double v) {
  __shared__ double part[kThreads / 64];
  v = wave_sum64(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += part[w];
  return s;
}

template <bool kBf16>
__device__ __forceinline__ double chunk_squares(const void* p, int64_t begin, int n) {
  double a[2] = {0.0, 0.0};
#pragma unroll
  for (int i = 0; i < kChunk / (8 * kThreads); ++i) {
    const int c = (i * kThreads + threadIdx.x) * 8;
    if (c >= n) break;
    float v[8];
    unpack8<kBf16>(load8_part<kBf16>(p, begin + c, n - c), v);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const double d = v[u];
      a[u & 1] = fma(d, d, a[u & 1]);
    }
  }
  return a[0] + a[1];
}

__global__ __launch_bounds__(kThreads) void squares_kernel(GradList l, double* __restrict__ slots, bool add) {
  const int total = l.first[l.count];
  double a = 0.0;
  int at = 0;
  for (int chunk = blockIdx.x; chunk < total; chunk += gridDim.x) {
    at = chunk_of(l, chunk, at);
    const int64_t begin = static_cast<int64_t>(chunk - l.first[at]) * kChunk;
    const int n = static_cast<int>(min<int64_t>(kChunk, l.numel[at] - begin));
    a += (l.bf16[at >> 5] >> (at & 31)) & 1u ? chunk_squares<true>(l.in[at], begin, n)
                                             : chunk_squares<false>(l.in[at], begin, n);
  }
  a = block_sum64(a);
  if (threadIdx.x == 0) slots[blockIdx.x] = add ? slots[blockIdx.x] + a : a;
}

__device__ __forceinline__ double norm_of(const double* slots, int n) {
  double a = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) a += slots[i];
  return sqrt(block_sum64(a));
}

__device__ __forceinline__ void write_norm(double norm, float* out, int32_t* check) {
  if (threadIdx.x != 0) return;
  *out = static_cast<float>(norm);
  if (check && !(norm < INFINITY)) atomicOr(check, MOE_CHECK_GRADS);
}

__global__ __launch_bounds__(kThreads) void norm_value_kernel(const double* __restrict__ slots, int n,
                                                              float* __restrict__ norm, int32_t* __restrict__ check) {
  write_norm(norm_of(slots, n), norm, check);
}

template <bool kBf16>
__device__ __forceinline__ void scale_chunk(const void* in, void* out, int64_t begin, int n, float factor, int exp2) {
#pragma unroll
  for (int i = 0; i < kChunk / (8 * kThreads); ++i) {
    const int c = (i * kThreads + threadIdx.x) * 8;
    if (c >= n) break;
    float v[8];
    unpack8<kBf16>(load8_part<kBf16>(in, begin + c, n - c), v);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = ldexpf(v[u] * factor, exp2);
    store8_part<kBf16>(out, begin + c, n - c, v);
  }
}

// norm_out != nullptr in one launch of a call only
__global__ __launch_bounds__(kThreads) void scale_kernel(GradList l, const double* __restrict__ slots, int n_slots,
                                                         double max_norm, double eps, float* norm_out,
                                                         int32_t* check) {
  const double norm = norm_of(slots, n_slots);
  if (norm_out && blockIdx.x == 0) write_norm(norm, norm_out, check);
  double f = max_norm / (norm + eps);
  if (f > 1.0) f = 1.0;  // NaN stays
  // mantissa and exponent apart: the factor itself may lie below a float's range
  int exp2 = 0;
  const float factor = static_cast<float>(f == f ? frexp(f, &exp2) : f);
  const int total = l.first[l.count];
  int at = 0;
  for (int chunk = blockIdx.x; chunk < total; chunk += gridDim.x) {
    at = chunk_of(l, chunk, at);
    if (f == 1.0 && l.in[at] == l.out[at]) continue;
    const int64_t begin = static_cast<int64_t>(chunk - l.first[at]) * kChunk;
    const int n = static_cast<int>(min<int64_t>(kChunk, l.numel[at] - begin));
    if ((l.bf16[at >> 5] >> (at & 31)) & 1u) scale_chunk<true>(l.in[at], l.out[at], begin, n, factor, exp2);
    else scale_chunk<false>(l.in[at], l.out[at], begin, n, factor, exp2);
  }
}

struct Extent {
  uintptr_t lo, hi;
  int i;
};

int check_list(const char* who, const void* const* grads, const int64_t* numel, const moe_dtype* dt, int n) {
  using namespace moe;
  if (n < 0) return fail(MOE_ERR_INVALID_ARG, "%s: n=%d", who, n);
  if (n > 0 && (!grads || !numel || !dt)) return fail(MOE_ERR_INVALID_ARG, "%s: null list", who);
  for (int i = 0; i < n; ++i) {
    if (dt[i] != MOE_F32 && dt[i] != MOE_BF16)
      return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype %d of tensor %d", who, (int)dt[i], i);
    if (numel[i] < 0 || numel[i] >= (int64_t(1) << 37))
      return fail(MOE_ERR_INVALID_ARG, "%s: size %lld of tensor %d out of range", who, (long long)numel[i], i);
    if (numel[i] > 0 && !grads[i]) return fail(MOE_ERR_INVALID_ARG, "%s: null tensor %d", who, i);
    if (reinterpret_cast<uintptr_t>(grads[i]) % elem_bytes(dt[i]))
      return fail(MOE_ERR_INVALID_ARG, "%s: tensor %d is misaligned", who, i);
  }
  return MOE_OK;
}

// The tensors written must not overlap each other, nor a gradient other than their own.
int check_outputs(const char* who, const void* const* grads, void* const* out, const int64_t* numel,
                  const moe_dtype* dt, int n) {
  using namespace moe;
  for (int i = 0; i < n; ++i) {
    if (numel[i] > 0 && !out[i]) return fail(MOE_ERR_INVALID_ARG, "%s: null output %d", who, i);
    if (reinterpret_cast<uintptr_t>(out[i]) % elem_bytes(dt[i]))
      return fail(MOE_ERR_INVALID_ARG, "%s: output %d is misaligned", who, i);
  }
  Extent* e = new (std::nothrow) Extent[n > 0 ? n : 1];
  if (!e) return fail(MOE_ERR_HIP, "%s: out of host memory", who);
  int m = 0;
  for (int i = 0; i < n; ++i)
    if (numel[i] > 0) {
      const uintptr_t lo = reinterpret_cast<uintptr_t>(out[i]);
      e[m++] = {lo, lo + static_cast<uintptr_t>(numel[i]) * elem_bytes(dt[i]), i};
    }
  std::sort(e, e + m, [](const Extent& a, const Extent& b) { return a.lo < b.lo; });
  int bad = -1;
  for (int j = 0; j + 1 < m && bad < 0; ++j)
    if (e[j].hi > e[j + 1].lo) bad = e[j + 1].i;
  for (int i = 0; i < n && bad < 0; ++i) {
    if (numel[i] == 0) continue;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(grads[i]);
    const uintptr_t hi = lo + static_cast<uintptr_t>(numel[i]) * elem_bytes(dt[i]);
    // outputs are disjoint here: those that overlap [lo, hi) follow one another
    const Extent* q = std::upper_bound(e, e + m, lo, [](uintptr_t v, const Extent& a) { return v < a.hi; });
    for (; q != e + m && q->lo < hi && bad < 0; ++q)
      if (!(q->i == i && q->lo == lo)) bad = q->i;
  }
  delete[] e;
  if (bad >= 0)
    return fail(MOE_ERR_INVALID_ARG, "%s: output %d overlaps another tensor of the call", who, bad);
  return MOE_OK;
}

// Tensors i .. of the list that fit one launch; returns the index after them.
int fill(GradList& l, const void* const* grads, void* const* out, const int64_t* numel, const moe_dtype* dt, int n,
         int i) {
  l.count = 0;
  l.first[0] = 0;
  for (uint32_t& w : l.bf16) w = 0;
  for (; i < n && l.count < kList; ++i) {
    if (numel[i] == 0) continue;
    const int64_t chunks = moe::ceil_div(numel[i], kChunk);
    if (l.first[l.count] + chunks > INT32_MAX - kSlots) break;  // one tensor has at most 2^24
    l.in[l.count] = grads[i];
    l.out[l.count] = out ? out[i] : nullptr;
    l.numel[l.count] = numel[i];
    if (dt[i] == MOE_BF16) l.bf16[l.count >> 5] |= 1u << (l.count & 31);
    l.first[l.count + 1] = l.first[l.count] + static_cast<int32_t>(chunks);
    ++l.count;
  }
  return i;
}

unsigned grid_of(const GradList& l) {
  return static_cast<unsigned>(std::min<int32_t>(kSlots, std::max<int32_t>(1, l.first[l.count])));
}

// Squares of the whole list into the slots; the first launch writes every slot used.
int squares(const char* who, const void* const* grads, const int64_t* numel, const moe_dtype* dt, int n,
            double* slots, int* n_slots, hipStream_t s) {
  GradList l;
  int i = 0;
  bool more = false;
  *n_slots = 0;
  do {
    i = fill(l, grads, nullptr, numel, dt, n, i);
    // a list of several launches fills all slots in the first one
    const unsigned grid = !more && i < n ? static_cast<unsigned>(kSlots) : grid_of(l);
    squares_kernel<<<grid, kThreads, 0, s>>>(l, slots, more);
    if (int rc = moe::hip_status(hipGetLastError(), who)) return rc;
    *n_slots = std::max(*n_slots, static_cast<int>(grid));
    more = true;
  } while (i < n);
  return MOE_OK;
}

int check_workspace(const char* who, const void* workspace, size_t bytes) {
  using namespace moe;
  if (!workspace || bytes < kSlots * sizeof(double))
    return fail(MOE_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", who, workspace ? bytes : size_t(0),
                kSlots * sizeof(double));
  if (!aligned16(workspace)) return fail(MOE_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", who);
  return MOE_OK;
}

}  // namespace

extern "C" size_t moe_grad_norm_workspace_bytes(void) { return kSlots * sizeof(double); }

extern "C" int moe_grad_norm(const void* const* grads, const int64_t* numel, const moe_dtype* dt, int n, float* norm,
                             void* workspace, size_t workspace_bytes, int32_t* check, void* stream) {
  using namespace moe;
  if (int rc = check_list("moe_grad_norm", grads, numel, dt, n)) return rc;
  if (!norm) return fail(MOE_ERR_INVALID_ARG, "moe_grad_norm: null norm");
  if (int rc = check_workspace("moe_grad_norm", workspace, workspace_bytes)) return rc;
  const hipStream_t s = as_stream(stream);
  double* slots = static_cast<double*>(workspace);
  int n_slots = 0;
  if (int rc = squares("moe_grad_norm launch", grads, numel, dt, n, slots, &n_slots, s)) return rc;
  norm_value_kernel<<<1, kThreads, 0, s>>>(slots, n_slots, norm, check);
  return hip_status(hipGetLastError(), "moe_grad_norm value");
}

extern "C" int moe_clip_grads(const void* const* grads, void* const* out, const int64_t* numel, const moe_dtype* dt,
                              int n, float max_norm, float eps, float* norm, void* workspace, size_t workspace_bytes,
                              int32_t* check, void* stream) {
  using namespace moe;
  if (int rc = check_list("moe_clip_grads", grads, numel, dt, n)) return rc;
  if (n > 0 && !out) return fail(MOE_ERR_INVALID_ARG, "moe_clip_grads: null list");
  if (!(max_norm >= 0.f) || !std::isfinite(max_norm))
    return fail(MOE_ERR_INVALID_ARG, "moe_clip_grads: max_norm must be finite and not negative");
  if (!(eps > 0.f) || !std::isfinite(eps))
    return fail(MOE_ERR_INVALID_ARG, "moe_clip_grads: eps must be positive and finite");
  if (!norm) return fail(MOE_ERR_INVALID_ARG, "moe_clip_grads: null norm");
  if (int rc = check_workspace("moe_clip_grads", workspace, workspace_bytes)) return rc;
  if (int rc = check_outputs("moe_clip_grads", grads, out, numel, dt, n)) return rc;
  const hipStream_t s = as_stream(stream);
  double* slots = static_cast<double*>(workspace);
  int n_slots = 0;
  if (int rc = squares("moe_clip_grads squares", grads, numel, dt, n, slots, &n_slots, s)) return rc;
  GradList l;
  int i = 0;
  bool more = false;
  do {
    i = fill(l, grads, out, numel, dt, n, i);
    scale_kernel<<<grid_of(l), kThreads, 0, s>>>(l, slots, n_slots, max_norm, eps, more ? nullptr : norm, check);
    if (int rc = hip_status(hipGetLastError(), "moe_clip_grads scale")) return rc;
    more = true;
  } while (i < n);
  return MOE_OK;
}
