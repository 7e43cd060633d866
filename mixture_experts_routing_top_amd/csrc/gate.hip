// moe_gate, moe_gate_backward: the gates beyond a renormalised softmax.
//
// Scores s_e of the router logits (softmax over the row, or a sigmoid each), a
// per-expert bias that moves the selection and not the weights, a first
// choice among groups of experts, then the k best experts of the kept groups;
// the weights are the chosen scores, renormalised or not, times a scale.
//
// The experts taken are those of the real numbers s_e + b_e: two scores can
// lie closer than a float's rounding (some row in a few thousand has such a
// pair among its candidates), so keys are compared in double.  Without a bias
// a score's order is its logit's, and no score is formed for the selection.
//
// A masked expert (logit NaN or <= kMaskBelow) has score 0 and comes after
// every other expert of the kept groups, in index order.
#include <cfloat>
#include <cmath>

#include "common.h"

namespace {

constexpr float kMaskBelow = -1e38f;
constexpr double kMaskedKey = -1e300;    // below every key of a live expert (biases are clamped above it)
constexpr double kBiasLimit = 1e299;
constexpr int kMaxGroups = 64;

struct GateArgs {
  const void* logits;
  const float* bias;  // may be null
  int64_t T;
  int E, k, n_groups, keep, group_size;
  bool top2, softmax, renorm;
  float scale;
  int32_t* idx;
  float* w;
  int32_t* check;
};

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (kBf16) return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}

// false for NaN too
__device__ __forceinline__ bool is_live(float l) { return l > kMaskBelow; }

__device__ __forceinline__ bool ahead(double v1, int i1, double v2, int i2) {
  return v1 > v2 || (v1 == v2 && i1 < i2);
}

template <typename V>
__device__ __forceinline__ V wave_max(V v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const V o = __shfl_xor(v, off);
    v = o > v ? o : v;
  }
  return v;
}

template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// LDS written by some lanes of a wave and read by others of the same wave
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One token by one wave: lane holds experts lane, lane + 64, ...  `value` is E
// doubles of LDS of this wave.  Every lane of the wave calls it with the same t.
template <bool kBf16>
__device__ void gate_token(const GateArgs& p, int64_t t, int lane, double* value, bool write) {
  const int64_t row = t * p.E;
  float l[4];
  double key[4];
  bool live[4];
  bool bad = false;
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = lane + 64 * j;
    l[j] = e < p.E ? load_logit<kBf16>(p.logits, row + e) : -INFINITY;
    live[j] = is_live(l[j]);
    bad |= e < p.E && (l[j] != l[j] || l[j] == INFINITY);
    l[j] = live[j] ? fminf(l[j], FLT_MAX) : -INFINITY;
    m = fmaxf(m, l[j]);
  }
  if (p.check) raise_check(p.check, bad && write, MOE_CHECK_LOGITS);

  // scores, where the selection or the weights need all of them
  const bool two = p.top2 && p.keep < p.n_groups;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  double total = 1.0;
  if (p.softmax && (!p.renorm || p.bias || two)) {
    m = wave_max(m);
    total = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[j] = live[j] ? exp(static_cast<double>(l[j]) - m) : 0.0;
      total += s[j];
    }
    total = wave_sum(total);
  }
  if (p.bias || two) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p.softmax) s[j] = total > 0.0 ? s[j] / total : 0.0;
      else s[j] = live[j] ? 1.0 / (1.0 + exp(-static_cast<double>(l[j]))) : 0.0;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = lane + 64 * j;
    double b = 0.0;
    if (p.bias && e < p.E) b = fmin(fmax(static_cast<double>(p.bias[e]), -kBiasLimit), kBiasLimit);  // NaN: lowest
    key[j] = e >= p.E ? -INFINITY : !live[j] ? kMaskedKey : p.bias ? s[j] + b : static_cast<double>(l[j]);
    if (p.keep < p.n_groups && e < p.E) value[e] = !two ? key[j] : live[j] ? s[j] + b : -INFINITY;
  }

  if (p.keep < p.n_groups) {
    // lane g scores group g; a group stays if fewer than `keep` are ahead of it
    wave_lds_fence();
    double best = -INFINITY, second = -INFINITY;
    if (lane < p.n_groups)
      for (int i = 0; i < p.group_size; ++i) {
        const double v = value[lane * p.group_size + i];
        if (v > best) { second = best; best = v; }
        else if (v > second) second = v;
      }
    const double score = two && second > -INFINITY ? best + second : best;
    int rank = 0;
    for (int g = 0; g < p.n_groups; ++g) {
      const double o = __shfl(score, g);
      rank += g != lane && ahead(o, g, score, lane);
    }
    const uint64_t kept = __ballot(lane < p.n_groups && rank < p.keep);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = lane + 64 * j;
      if (e < p.E && !((kept >> (e / p.group_size)) & 1u)) key[j] = -INFINITY;
    }
    wave_lds_fence();
  }

  // k rounds of an arg-max over the wave; lane i keeps the i-th expert
  int mine = 0;
  for (int i = 0; i < p.k; ++i) {
    double bv = -INFINITY;
    int bi = INT32_MAX;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (key[j] > bv) { bv = key[j]; bi = lane + 64 * j; }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const double ov = __shfl_xor(bv, off);
      const int oi = __shfl_xor(bi, off);
      if (ahead(ov, oi, bv, bi)) { bv = ov; bi = oi; }
    }
    if (lane == i) mine = bi;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (bi == lane + 64 * j) key[j] = -INFINITY;
  }

  // weights of the k experts, in double, rounded once; lanes 0 .. k - 1
  float lk = -INFINITY;
  if (lane < p.k) lk = load_logit<kBf16>(p.logits, row + mine);
  const bool on = lane < p.k && is_live(lk);
  lk = on ? fminf(lk, FLT_MAX) : -INFINITY;
  double v;
  if (p.softmax) {
    const double top = p.renorm ? wave_max(static_cast<double>(lk)) : static_cast<double>(m);
    v = on ? exp(lk - top) : 0.0;
  } else {
    // with renormalisation, times exp(-top), top = min(0, the largest logit):
    // the ratios survive where every sigmoid underflows
    const double top = p.renorm ? fmin(wave_max(static_cast<double>(lk)), 0.0) : 0.0;
    const double x = lk;
    v = !on ? 0.0 : x > 0.0 ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / (1.0 + exp(x));
  }
  const double sum = p.renorm ? wave_sum(v) : total;
  if (write && lane < p.k) {
    p.idx[t * p.k + lane] = mine;
    p.w[t * p.k + lane] = static_cast<float>(sum > 0.0 ? p.scale * (v / sum) : 0.0);
  }
}

template <bool kBf16>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs p) {
  __shared__ double value[4][moe::kMaxExperts];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (t >= p.T) return;
  gate_token<kBf16>(p, t, lane, value[wave], true);
}

// ------------------------------------------------------------------ backward
// With g_i = scale * d_w[i] on the kept experts e_i and s their scores:
//   softmax, renormalised    d_l[e_i] = r_i (g_i - sum_j g_j r_j), r = s / sum over the kept
//   sigmoid, renormalised    the same times (1 - s_i)
//   sigmoid                  d_l[e_i] = g_i s_i (1 - s_i)
//   softmax                  d_l[e] = [e = e_i] g_i s_i - s_e sum_j g_j s_j, dense
// and zero elsewhere.  The bias only selects: it has no gradient.
struct GateBwdArgs {
  const void* logits;
  const int32_t* idx;
  const float* d_w;
  void* d_logits;
  int64_t T;
  int E, k;
  bool softmax, renorm;
  float scale;
  int32_t* check;
};

template <bool kBf16>
__global__ __launch_bounds__(256) void gate_grad_kernel(GateBwdArgs p) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (t >= p.T) return;
  const int64_t row = t * p.E;
  const bool dense = p.softmax && !p.renorm;

  // lanes 0 .. k - 1: the slot's expert, gradient and logit
  int e = -1;
  float g = 0.f, lk = -INFINITY;
  bool bad = false;
  if (lane < p.k) {
    e = p.idx[t * p.k + lane];
    bad = e < 0 || e >= p.E;
    if (!bad) {
      g = p.scale * p.d_w[t * p.k + lane];
      lk = load_logit<kBf16>(p.logits, row + e);
    } else {
      e = -1;
    }
  }
  if (p.check) raise_check(p.check, bad, MOE_CHECK_INDEX);
  const bool on = is_live(lk);
  lk = on ? fminf(lk, FLT_MAX) : -INFINITY;
  if (!on) g = 0.f;

  float l[4];
  float m = -INFINITY, total = 0.f;
  if (dense) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = lane + 64 * j;
      l[j] = c < p.E ? load_logit<kBf16>(p.logits, row + c) : -INFINITY;
      l[j] = is_live(l[j]) ? fminf(l[j], FLT_MAX) : -INFINITY;
      m = fmaxf(m, l[j]);
    }
    m = wave_max(m);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      l[j] = l[j] > -INFINITY ? expf(l[j] - m) : 0.f;
      total += l[j];
    }
    total = wave_sum(total);
  }

  float slot;   // the slot's part of d_l[e]
  float common = 0.f;
  if (p.softmax) {
    if (p.renorm) m = wave_max(lk);
    float s = on ? expf(lk - m) : 0.f;
    if (p.renorm) total = wave_sum(s);
    s = total > 0.f ? s / total : 0.f;
    common = wave_sum(g * s);
    slot = p.renorm ? s * (g - common) : g * s;
  } else {
    const float z = expf(-fabsf(lk));          // s = 1 / (1 + z) or z / (1 + z)
    const float other = on ? (lk > 0.f ? z : 1.f) / (1.f + z) : 0.f;   // 1 - s
    if (p.renorm) {
      const float top = fminf(wave_max(lk), 0.f);
      const float s = !on ? 0.f : (lk > 0.f ? 1.f : expf(lk - top)) / (1.f + z);
      const float sum = wave_sum(s);
      const float r = sum > 0.f ? s / sum : 0.f;
      slot = r * (g - wave_sum(g * r)) * other;
    } else {
      slot = on ? g * ((lk > 0.f ? 1.f : z) / (1.f + z)) * other : 0.f;
    }
  }

  float d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) d[j] = dense && l[j] > 0.f ? -(l[j] / total) * common : 0.f;
  for (int i = 0; i < p.k; ++i) {
    const int ei = __shfl(e, i);
    const float v = __shfl(slot, i);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (ei == lane + 64 * j) d[j] += v;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = lane + 64 * j;
    if (c >= p.E) continue;
    if constexpr (kBf16) static_cast<uint16_t*>(p.d_logits)[row + c] = static_cast<uint16_t>(f32_to_bf16_bits(d[j]));
    else static_cast<float*>(p.d_logits)[row + c] = d[j];
  }
}

int check_common(const char* who, moe_dtype dt, int64_t T, int E, int k, moe_score score, float scale) {
  using namespace moe;
  if (dt != MOE_F32 && dt != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dt);
  if (score != MOE_SOFTMAX && score != MOE_SIGMOID)
    return fail(MOE_ERR_INVALID_ARG, "%s: unknown score %d", who, (int)score);
  if (E < 1 || E > kMaxExperts)
    return fail(E < 1 ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED, "%s: E=%d outside [1, %d]", who, E, kMaxExperts);
  if (k < 1 || k > E || k > kMaxTopK) return fail(MOE_ERR_INVALID_ARG, "%s: k=%d outside [1, min(E, 8)]", who, k);
  if (T < 0 || T >= (int64_t(1) << 31) || T * k >= (int64_t(1) << 31))
    return fail(MOE_ERR_INVALID_ARG, "%s: T=%lld out of range", who, (long long)T);
  if (!std::isfinite(scale)) return fail(MOE_ERR_INVALID_ARG, "%s: scale must be finite", who);
  return MOE_OK;
}

}  // namespace

extern "C" int moe_gate(const void* logits, moe_dtype dt, int64_t T, int E, int k, moe_score score, const float* bias,
                        int n_groups, int keep_groups, moe_group_score group_score, int renorm, float scale,
                        int32_t* topk_idx, float* topk_w, int32_t* check, void* stream) {
  using namespace moe;
  if (int rc = check_common("moe_gate", dt, T, E, k, score, scale)) return rc;
  if (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2)
    return fail(MOE_ERR_INVALID_ARG, "moe_gate: unknown group score %d", (int)group_score);
  if (n_groups < 1 || E % n_groups)
    return fail(MOE_ERR_INVALID_ARG, "moe_gate: n_groups=%d does not divide E=%d", n_groups, E);
  if (n_groups > kMaxGroups)
    return fail(MOE_ERR_UNSUPPORTED, "moe_gate: n_groups=%d beyond %d", n_groups, kMaxGroups);
  const int size = E / n_groups;
  if (keep_groups < 1 || keep_groups > n_groups || static_cast<int64_t>(keep_groups) * size < k)
    return fail(MOE_ERR_INVALID_ARG, "moe_gate: keep_groups=%d of %d groups of %d experts cannot give k=%d",
                keep_groups, n_groups, size, k);
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !topk_w) return fail(MOE_ERR_INVALID_ARG, "moe_gate: null pointer");
  GateArgs p{logits, bias, T, E, k, n_groups, keep_groups, size, group_score == MOE_GROUP_TOP2,
             score == MOE_SOFTMAX, renorm != 0, scale, topk_idx, topk_w, check};
  const unsigned blocks = static_cast<unsigned>(ceil_div(T, 4));
  if (dt == MOE_BF16) gate_kernel<true><<<blocks, 256, 0, as_stream(stream)>>>(p);
  else gate_kernel<false><<<blocks, 256, 0, as_stream(stream)>>>(p);
  return hip_status(hipGetLastError(), "moe_gate launch");
}

extern "C" int moe_gate_backward(const void* logits, moe_dtype dt, int64_t T, int E, int k, moe_score score,
                                 int renorm, float scale, const int32_t* topk_idx, const float* d_topk_w,
                                 void* d_logits, int32_t* check, void* stream) {
  using namespace moe;
  if (int rc = check_common("moe_gate_backward", dt, T, E, k, score, scale)) return rc;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !d_topk_w || !d_logits)
    return fail(MOE_ERR_INVALID_ARG, "moe_gate_backward: null pointer");
  GateBwdArgs p{logits, topk_idx, d_topk_w, d_logits, T, E, k, score == MOE_SOFTMAX, renorm != 0, scale, check};
  const unsigned blocks = static_cast<unsigned>(ceil_div(T, 4));
  if (dt == MOE_BF16) gate_grad_kernel<true><<<blocks, 256, 0, as_stream(stream)>>>(p);
  else gate_grad_kernel<false><<<blocks, 256, 0, as_stream(stream)>>>(p);
  return hip_status(hipGetLastError(), "moe_gate_backward launch");
}
