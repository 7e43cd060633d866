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
//
// Two steps.  gate_kernel gives a token to 16 lanes and selects in float32 on
// 32-bit keys, 24 bits of the value in fixed point and 8 of the index, knowing
// a bound on its own error: a token whose order two candidates closer than the
// bound could turn (not if they are equal in logit and bias: then the index
// decides, in double as well) is done again by the whole wave in double
// (gate_token).  Doing every token in double costs ten times the time.
#include <algorithm>
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

// ------------------------------------------------------------ 16 lanes a token
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __int_as_float(dpp_partner<1>(__float_as_int(v))));
  v = fmaxf(v, __int_as_float(dpp_partner<2>(__float_as_int(v))));
  v = fmaxf(v, __int_as_float(dpp_partner<4>(__float_as_int(v))));
  return fmaxf(v, __int_as_float(dpp_partner<8>(__float_as_int(v))));
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(dpp_partner<1>(v)));
  v = max(v, static_cast<uint32_t>(dpp_partner<2>(v)));
  v = max(v, static_cast<uint32_t>(dpp_partner<4>(v)));
  return max(v, static_cast<uint32_t>(dpp_partner<8>(v)));
}
template <int OFF>
__device__ __forceinline__ double partner64(double v) {
  return __hiloint2double(dpp_partner<OFF>(__double2hiint(v)), dpp_partner<OFF>(__double2loint(v)));
}
__device__ __forceinline__ double row_sum(double v) {
  v += partner64<1>(v);
  v += partner64<2>(v);
  v += partner64<4>(v);
  return v + partner64<8>(v);
}
__device__ __forceinline__ float row_sum(float v) {
  v += __int_as_float(dpp_partner<1>(__float_as_int(v)));
  v += __int_as_float(dpp_partner<2>(__float_as_int(v)));
  v += __int_as_float(dpp_partner<4>(__float_as_int(v)));
  return v + __int_as_float(dpp_partner<8>(__float_as_int(v)));
}
// the value of the lane one up in the 16 (lane 15: its own)
__device__ __forceinline__ int next_lane(int v) { return __builtin_amdgcn_update_dpp(v, v, 0x101, 0xf, 0xf, false); }
// the value of the lane N down, around the 16
template <int N>
__device__ __forceinline__ float rotated(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + N, 0xf, 0xf, false));
}

// Groups ahead of this lane's: `rep` is the group's score in the first lane of
// each group and NaN, ahead of nothing, in the others; bit N of `ties` is set
// where the lane N down belongs to a group before this lane's.
template <int N>
__device__ __forceinline__ void count_ahead(float rep, float score, uint32_t ties, int& rank) {
  if constexpr (N < 16) {
    const float o = rotated<N>(rep);
    rank += o > score || (o == score && ((ties >> N) & 1u));
    count_ahead<N + 1>(rep, score, ties, rank);
  }
}

// the k-th largest key and those after it: with unsigned wrap-around the keys
// below `best` lie above those at or over it, so one subtraction and a maximum
// give the next one and nothing has to be struck out
template <int V>
__device__ __forceinline__ uint32_t next_key(const uint32_t (&key)[V], uint32_t best) {
  uint32_t d = key[0] - best;
#pragma unroll
  for (int j = 1; j < V; ++j) d = max(d, key[j] - best);
  return best + row_max(d);
}

enum { kByLogit, kSigmoid, kSoftmax };  // what the selection compares

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTop = 16777200.f;     // the largest fixed-point value, below 2^24

// Lane i of a token's 16 holds `per` consecutive experts (at most V) of one group:
// groups begin at multiples of `lanes` lanes.
template <bool kBf16, int V, int kBy>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs p, int lanes, int per) {
  __shared__ double value[4][moe::kMaxExperts];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l16 = lane & 15;
  const bool grouped = p.keep < p.n_groups;
  const int group = l16 / lanes;                      // == p.n_groups or more: an idle lane
  const int inside = (l16 % lanes) * per;
  const int e0 = group * p.group_size + inside;
  const int n = group < p.n_groups ? min(per, p.group_size - inside) : 0;   // this lane's experts
  const int64_t total = p.T * p.E;

  // the fixed-point scale, and the bound on the error of two values' difference
  float b[V];
  float scale = 0.f, offset = 0.f, near = 0.f, group_near = 0.f;
  if constexpr (kBy != kByLogit) {
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      b[j] = j < n && p.bias ? p.bias[e0 + j] : 0.f;
      if (!(fabsf(b[j]) <= 1e30f)) hi = INFINITY;     // left to the doubles
      if (j < n) { lo = fminf(lo, b[j]); hi = fmaxf(hi, b[j]); }
    }
    lo = -row_max(-lo);
    hi = row_max(hi);
    const float range = 1.f + (hi - lo), big = fmaxf(fabsf(lo), fabsf(hi));
    // s: exp2's argument, exp2, the sum and the reciprocal, 6 u in all (u = 2^-24);
    // a softmax's sum of up to 32 values in sequence and 4 steps: 36 u more.
    // s + b rounds once more.  In the key: half a unit of fma, one of the cut.
    const float err = (kBy == kSigmoid ? 7.f : 43.f) + big;
    scale = kTop / range;
    offset = 2.f - lo * scale;
    near = 2.f * (err / range + 2.f);
    group_near = (4.f * err + 4.f * (1.f + big)) * 0x1p-24f;
    if (!(hi < INFINITY)) near = group_near = INFINITY;
  } else {
    scale = kTop / 32.f;        // logits down to 32 below the largest: monotone, so only
    offset = 2.f + kTop;        // equal keys of unequal logits are in doubt
  }

  for (int64_t base = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * 4; base < p.T;
       base += static_cast<int64_t>(gridDim.x) * 16) {
    const int64_t t = base + (lane >> 4);
    const bool active = t < p.T;
    const int64_t row = (active ? t : 0) * p.E;
    float l[V];
    bool bad = false;
    float m = -INFINITY;
    {
      const int64_t at = row + e0;
      if (n > 0 && at + V <= total) {
        if constexpr (kBf16) {
          uint16_t raw[V];
          __builtin_memcpy(raw, static_cast<const uint16_t*>(p.logits) + at, sizeof(raw));
#pragma unroll
          for (int j = 0; j < V; ++j) l[j] = bf16_bits_to_f32(raw[j]);
        } else {
          __builtin_memcpy(l, static_cast<const float*>(p.logits) + at, sizeof(l));
        }
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = j < n ? load_logit<kBf16>(p.logits, at + j) : -INFINITY;
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (j >= n) l[j] = -INFINITY;
      bad |= l[j] != l[j] || l[j] == INFINITY;
      l[j] = is_live(l[j]) ? fminf(l[j], FLT_MAX) : -INFINITY;
      m = fmaxf(m, l[j]);
    }
    if (p.check) raise_check(p.check, bad && active, MOE_CHECK_LOGITS);
    m = row_max(m);
    if (m == -INFINITY) m = 0.f;   // nothing unmasked

    float v[V];
    double sum64 = 1.0;
    if constexpr (kBy == kByLogit) {
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = l[j];
    } else if constexpr (kBy == kSigmoid) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        v[j] = l[j] > -INFINITY ? __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l[j] * -kLog2e)) + b[j] : -INFINITY;
    } else {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[j] = __builtin_amdgcn_exp2f((l[j] - m) * kLog2e);
        sum += v[j];
      }
      sum = row_sum(sum);
      const float inv = sum > 0.f ? __builtin_amdgcn_rcpf(sum) : 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = l[j] > -INFINITY ? fmaf(v[j], inv, b[j]) : -INFINITY;
    }
    if (p.softmax && !p.renorm) {   // the weights' denominator
      sum64 = 0.0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j < n && l[j] > -INFINITY) sum64 += exp(static_cast<double>(l[j]) - static_cast<double>(m));
        __builtin_amdgcn_sched_barrier(0);   // one exponential's registers at a time
      }
      sum64 = row_sum(sum64);
    }

    uint32_t key[V];   // (value + 2) << 8 | 255 - index; 1 in the value's place: masked; 0: not to be taken
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float x = kBy == kByLogit ? v[j] - m : v[j];
      const uint32_t q = l[j] > -INFINITY ? static_cast<uint32_t>(fminf(fmaxf(fmaf(x, scale, offset), 2.f), 16777215.f)) : 1u;
      key[j] = j < n ? (q << 8) + static_cast<uint32_t>(255 - e0 - j) : 0u;
    }

    bool doubt = false;
    if (grouped) {
      float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        m2 = fmaxf(m2, fminf(m1, v[j]));
        m1 = fmaxf(m1, v[j]);
      }
      auto join = [&](float o1, float o2) {
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
      };
#define MOE_JOIN(OFF)                                                            \
  if (lanes > OFF)                                                               \
    join(__int_as_float(dpp_partner<OFF>(__float_as_int(m1))), __int_as_float(dpp_partner<OFF>(__float_as_int(m2))));
      MOE_JOIN(1) MOE_JOIN(2) MOE_JOIN(4)
#undef MOE_JOIN
      const float score = p.top2 && m2 > -INFINITY ? m1 + m2 : m1;
      const bool rep = l16 % lanes == 0 && group < p.n_groups;
      int rank = 0;
      count_ahead<1>(rep ? score : NAN, score, (2u << l16) - (2u << (l16 % lanes)), rank);
      const bool kept = rank < p.keep;
      if constexpr (kBy != kByLogit) {
        // the last group kept against the first one left out
        const float low = -row_max(rep && kept ? -score : -INFINITY);
        const float high = row_max(rep && !kept ? score : -INFINITY);
        doubt = high > -INFINITY && !(low - high > group_near);
      }
      if (!kept)
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = 0u;
    }

    // lane i takes the i-th key, lane k the best one left
    uint32_t best = 0, mine = 0;
#pragma unroll
    for (int i = 0; i <= moe::kMaxTopK; ++i)
      if (i <= p.k) {
        best = next_key<V>(key, best);
        if (l16 == i) mine = best;
      }
    const int e = min(255 - static_cast<int>(mine & 255u), p.E - 1);
    const bool some = l16 <= p.k && mine >= 512u;      // an unmasked expert
    float lk = some ? load_logit<kBf16>(p.logits, row + e) : -INFINITY;
    lk = fminf(lk, FLT_MAX);
    const uint32_t q = mine >> 8, q_next = static_cast<uint32_t>(next_lane(static_cast<int>(mine))) >> 8;
    const float l_next = __int_as_float(next_lane(__float_as_int(lk)));
    bool same = lk == l_next;
    float bk = 0.f;
    if constexpr (kBy != kByLogit) {
      if (p.bias && some) bk = p.bias[e];
      same = same && bk == __int_as_float(next_lane(__float_as_int(bk)));
    }
    doubt |= some && l16 < p.k && q_next >= 2u && static_cast<float>(q - q_next) <= near && !same;
    const uint64_t doubts = __ballot(doubt && active);
    const bool redo = (doubts >> (lane & 48)) & 0xffffu;

    // weights in double, rounded once
    const bool on = some && l16 < p.k;
    double w;
    if (p.softmax) {
      const double top = p.renorm ? static_cast<double>(row_max(on ? lk : -INFINITY)) : static_cast<double>(m);
      w = on ? exp(static_cast<double>(lk) - top) : 0.0;
    } else {
      // see gate_token
      const double top = p.renorm ? fmin(static_cast<double>(row_max(on ? lk : -INFINITY)), 0.0) : 0.0;
      const double x = lk;
      w = !on ? 0.0 : x > 0.0 ? 1.0 / (1.0 + exp(-x)) : exp(x - top) / (1.0 + exp(x));
    }
    const double sum = p.renorm ? row_sum(w) : sum64;
    if (active && !redo && l16 < p.k) {
      p.idx[t * p.k + l16] = e;
      p.w[t * p.k + l16] = static_cast<float>(sum > 0.0 ? p.scale * (w / sum) : 0.0);
    }
    if (doubts)
#pragma unroll 1
      for (int i = 0; i < 4; ++i)
        if ((doubts >> (16 * i)) & 0xffffu) gate_token<kBf16>(p, base + i, lane, value[wave], true);
  }
}

// One wave a token, in double throughout: more groups than 16 lanes hold.
template <bool kBf16>
__global__ __launch_bounds__(256) void gate_wave_kernel(GateArgs p) {
  __shared__ double value[4][moe::kMaxExperts];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (t >= p.T) return;
  gate_token<kBf16>(p, t, lane, value[wave], true);
}

template <bool kBf16, int kBy>
void launch_slots(const GateArgs& p, hipStream_t s) {
  int lanes = 16;
  if (p.keep < p.n_groups)
    while (16 / lanes < p.n_groups) lanes /= 2;
  GateArgs q = p;
  if (p.keep == p.n_groups) { q.n_groups = q.keep = 1; q.group_size = p.E; }
  const int per = static_cast<int>(moe::ceil_div(q.group_size, lanes));
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(2048, moe::ceil_div(p.T, 16)));
  if (per <= 2) gate_kernel<kBf16, 2, kBy><<<blocks, 256, 0, s>>>(q, lanes, per);
  else if (per <= 4) gate_kernel<kBf16, 4, kBy><<<blocks, 256, 0, s>>>(q, lanes, per);
  else if (per <= 8) gate_kernel<kBf16, 8, kBy><<<blocks, 256, 0, s>>>(q, lanes, per);
  else if (per <= 12) gate_kernel<kBf16, 12, kBy><<<blocks, 256, 0, s>>>(q, lanes, per);
  else if (per <= 16) gate_kernel<kBf16, 16, kBy><<<blocks, 256, 0, s>>>(q, lanes, per);
  else gate_kernel<kBf16, 32, kBy><<<blocks, 256, 0, s>>>(q, lanes, per);
}

template <bool kBf16>
void launch_gate(const GateArgs& p, hipStream_t s) {
  if (p.keep < p.n_groups && p.n_groups > 16)
    gate_wave_kernel<kBf16><<<static_cast<unsigned>(moe::ceil_div(p.T, 4)), 256, 0, s>>>(p);
  else if (!p.bias && !(p.top2 && p.keep < p.n_groups)) launch_slots<kBf16, kByLogit>(p, s);
  else if (p.softmax) launch_slots<kBf16, kSoftmax>(p, s);
  else launch_slots<kBf16, kSigmoid>(p, s);
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
  if (dt == MOE_BF16) launch_gate<true>(p, as_stream(stream));
  else launch_gate<false>(p, as_stream(stream));
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
