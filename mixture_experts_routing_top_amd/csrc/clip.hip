// moe_grad_norm, moe_clip_grads: the global norm of many gradients, and the
// gradients scaled so that it is at most max_norm.
//
//   norm = sqrt(sum over all tensors of all squares)
//   out = g * min(1, max_norm / (norm + eps))
//
// HBM-bound: everything is read for the norm before anything can be scaled, so
// a clip moves 2 reads and 1 write (1.07 GB of float32: 159 us for the norm, 6.7
// TB/s, and 376 us for the scaling, 5.7 TB/s).  The product of two floats is exact in
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

// The tensor a chunk belongs to: the lanes of a wave compare all tensors at once
// (a walk over the list is a chain of scalar loads, a microsecond for 50 tensors).
__device__ __forceinline__ int tensor_of(const GradList& l, int chunk) {
  const int lane = threadIdx.x & 63;
  int before = 0;   // tensors that end at or before the chunk
#pragma unroll
  for (int i = 0; i < kList; i += 64)
    before += __popcll(__ballot(i + lane < l.count && l.first[min(i + lane + 1, kList)] <= chunk));
  return __builtin_amdgcn_readfirstlane(before);
}

// Whether `chunk` (ascending or descending) is still the tensor's, else the right one.
__device__ __forceinline__ int tensor_near(const GradList& l, int chunk, int at) {
  return chunk >= l.first[at] && chunk < l.first[at + 1] ? at : tensor_of(l, chunk);
}

__device__ __forceinline__ double block_sum64(double v) {
  __shared__ double part[kThreads / 64];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += part[w];
  return s;
}

// A chunk is walked 16 bytes a thread at a time, so that each access of a wave
// covers whole lines; a whole chunk's loads are all issued before the first is used.
template <bool kBf16>
struct Piece {
  static constexpr int kWide = kBf16 ? 8 : 4;                      // elements of 16 bytes
  static constexpr int kCount = kChunk / (kWide * kThreads);       // pieces per thread of a whole chunk
  using Words = uint32_t __attribute__((ext_vector_type(4), aligned(kBf16 ? 2 : 4)));

  __device__ __forceinline__ static int first() { return threadIdx.x * kWide; }
  template <bool kOnce>
  __device__ __forceinline__ static Words load(const void* p, int64_t i) {
    const Words* q = reinterpret_cast<const Words*>(static_cast<const char*>(p) + i * (kBf16 ? 2 : 4));
    if constexpr (kOnce) return __builtin_nontemporal_load(q);
    else return *q;
  }
  __device__ __forceinline__ static float get(const Words& w, int u) {
    if constexpr (kBf16) return __uint_as_float((u & 1) ? w[u / 2] & 0xffff0000u : w[u / 2] << 16);
    else return __uint_as_float(w[u]);
  }
};

template <bool kBf16, bool kOnce>
__device__ __forceinline__ double chunk_squares(const void* p, int64_t begin, int n) {
  using P = Piece<kBf16>;
  double a[2] = {0.0, 0.0};
  auto add = [&](const typename P::Words& w) {
#pragma unroll
    for (int u = 0; u < P::kWide; ++u) {
      const double d = P::get(w, u);
      a[u & 1] = fma(d, d, a[u & 1]);
    }
  };
  if (n == kChunk) {
    typename P::Words w[P::kCount];
#pragma unroll
    for (int i = 0; i < P::kCount; ++i) w[i] = P::template load<kOnce>(p, begin + P::first() + i * kThreads * P::kWide);
#pragma unroll
    for (int i = 0; i < P::kCount; ++i) add(w[i]);
  } else {
    for (int c = P::first(); c + P::kWide <= n; c += kThreads * P::kWide) add(P::template load<kOnce>(p, begin + c));
    const int rest = n % P::kWide;
    if (threadIdx.x < rest) {
      const double d = load1<kBf16>(p, begin + n - rest + threadIdx.x);
      a[0] = fma(d, d, a[0]);
    }
  }
  return a[0] + a[1];
}

template <bool kOnce>
__global__ __launch_bounds__(kThreads) void squares_kernel(GradList l, double* __restrict__ slots, bool add) {
  const int total = l.first[l.count];
  double a = 0.0;
  int at = tensor_of(l, blockIdx.x);
  for (int chunk = blockIdx.x; chunk < total; chunk += gridDim.x) {
    at = tensor_near(l, chunk, at);
    const int64_t begin = static_cast<int64_t>(chunk - l.first[at]) * kChunk;
    const int n = static_cast<int>(min<int64_t>(kChunk, l.numel[at] - begin));
    a += (l.bf16[at >> 5] >> (at & 31)) & 1u ? chunk_squares<true, kOnce>(l.in[at], begin, n)
                                             : chunk_squares<false, kOnce>(l.in[at], begin, n);
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

template <bool kBf16, bool kOnce>
__device__ __forceinline__ void scale_chunk(const void* in, void* out, int64_t begin, int n, float factor, int exp2) {
  using P = Piece<kBf16>;
  auto scaled = [&](float v) { return ldexpf(v * factor, exp2); };
  auto put = [&](const typename P::Words& w, int64_t i) {
    float v[P::kWide];
#pragma unroll
    for (int u = 0; u < P::kWide; ++u) v[u] = scaled(P::get(w, u));
    typename P::Words o;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if constexpr (kBf16) o[u] = f32_to_bf16_bits(v[2 * u]) | (f32_to_bf16_bits(v[2 * u + 1]) << 16);
      else o[u] = __float_as_uint(v[u]);
    }
    // past the caches, which still hold some of what the norm has read (f32 400 MB: 233 -> 201 us)
    __builtin_nontemporal_store(o, reinterpret_cast<typename P::Words*>(static_cast<char*>(out) + i * (kBf16 ? 2 : 4)));
  };
  if (n == kChunk) {
    typename P::Words w[P::kCount];
#pragma unroll
    for (int i = 0; i < P::kCount; ++i) w[i] = P::template load<kOnce>(in, begin + P::first() + i * kThreads * P::kWide);
#pragma unroll
    for (int i = 0; i < P::kCount; ++i) put(w[i], begin + P::first() + i * kThreads * P::kWide);
  } else {
    for (int c = P::first(); c + P::kWide <= n; c += kThreads * P::kWide)
      put(P::template load<kOnce>(in, begin + c), begin + c);
    const int rest = n % P::kWide;
    const int64_t i = begin + n - rest + threadIdx.x;
    if (threadIdx.x < rest) store1<kBf16>(out, i, scaled(load1<kBf16>(in, i)));
  }
}

// norm_out != nullptr in one launch of a call only
template <bool kOnce>
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
  // from the end: what the norm read last may still lie in the last-level cache
  int at = 0;
  for (int left = blockIdx.x; left < total; left += gridDim.x) {
    const int chunk = total - 1 - left;
    at = tensor_near(l, chunk, at);
    if (f == 1.0 && l.in[at] == l.out[at]) continue;
    const int64_t begin = static_cast<int64_t>(chunk - l.first[at]) * kChunk;
    const int n = static_cast<int>(min<int64_t>(kChunk, l.numel[at] - begin));
    if ((l.bf16[at >> 5] >> (at & 31)) & 1u) scale_chunk<true, kOnce>(l.in[at], l.out[at], begin, n, factor, exp2);
    else scale_chunk<false, kOnce>(l.in[at], l.out[at], begin, n, factor, exp2);
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

// Whether the list is so far beyond the 256 MB of the last-level cache that its
// loads are better marked as read once (f32 1.6 GB: 871 -> 816 us, 800 MB: 421 ->
// 401, 400 MB: no difference, 100 MB: 52 -> 54).
bool beyond_cache(const int64_t* numel, const moe_dtype* dt, int n) {
  int64_t bytes = 0;
  for (int i = 0; i < n; ++i) bytes += numel[i] * moe::elem_bytes(dt[i]);
  return bytes > (int64_t(512) << 20);
}

// Squares of the whole list into the slots; the first launch writes every slot used.
int squares(const char* who, const void* const* grads, const int64_t* numel, const moe_dtype* dt, int n,
            double* slots, int* n_slots, bool once, hipStream_t s) {
  GradList l;
  int i = 0;
  bool more = false;
  *n_slots = 0;
  do {
    i = fill(l, grads, nullptr, numel, dt, n, i);
    // a list of several launches fills all slots in the first one
    const unsigned grid = !more && i < n ? static_cast<unsigned>(kSlots) : grid_of(l);
    if (once) squares_kernel<true><<<grid, kThreads, 0, s>>>(l, slots, more);
    else squares_kernel<false><<<grid, kThreads, 0, s>>>(l, slots, more);
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
  const bool once = beyond_cache(numel, dt, n);
  if (int rc = squares("moe_grad_norm launch", grads, numel, dt, n, slots, &n_slots, once, s)) return rc;
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
  const bool once = beyond_cache(numel, dt, n);
  if (int rc = squares("moe_clip_grads squares", grads, numel, dt, n, slots, &n_slots, once, s)) return rc;
  GradList l;
  int i = 0;
  bool more = false;
  do {
    i = fill(l, grads, out, numel, dt, n, i);
    float* norm_out = more ? nullptr : norm;
    if (once) scale_kernel<true><<<grid_of(l), kThreads, 0, s>>>(l, slots, n_slots, max_norm, eps, norm_out, check);
    else scale_kernel<false><<<grid_of(l), kThreads, 0, s>>>(l, slots, n_slots, max_norm, eps, norm_out, check);
    if (int rc = hip_status(hipGetLastError(), "moe_clip_grads scale")) return rc;
    more = true;
  } while (i < n);
  return MOE_OK;
}
