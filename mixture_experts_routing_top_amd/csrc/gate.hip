// moe_gate, moe_gate_backward: the gates beyond a renormalised softmax.
//
// Scores s_e of the router logits (softmax over the row, or a sigmoid each), a
// per-expert bias that moves the selection and not the weights, a first
// choice among groups of experts, then the k best experts of the kept groups;
// the weights are the chosen scores, renormalised or not, times a scale.
//
// The experts taken are those of the real numbers s_e + b_e: two scores can
// lie closer than a float's rounding (of 600000 random rows of 256 biased sigmoids
// float32 put 7 in another order), so what a float cannot tell is compared in double.  Without a bias
// a score's order is its logit's, and no score is formed for the selection.
//
// A masked expert (logit NaN or <= kMaskBelow) has score 0 and comes after
// every other expert of the kept groups, in index order.
//
// gate_kernel gives a token to 16 lanes and selects in float32 on 32-bit keys, 23
// bits of the value in fixed point and 8 of the index, knowing a bound on its own
// error.  Where two candidates lie closer than the bound (and are not equal in
// logit and bias: then the index decides, in double as well), the token's 16 best
// are put in the order of their values in double, which is the answer if the 16th
// lies clearly below the k-th.  A token for which that does not do, or whose last
// kept group is as close to the first one left out, is done again by the whole wave
// in double (gate_token).  In those rows a gap among the first nine below 2^-20 of the
// largest, about what the bound asks, was there 280 times.  A batch whose tokens all
// come to the doubles takes six times as long (65536 x 256, biased sigmoids in 8 groups:
// 258 us with one bias -inf or -1e9, 252 with 2^20 in every bias; without a bias, in one
// group, 22 us, 131 with one logit 30 above the rest, 548 with all logits equal).
//
// 827 vector instructions (counted) for four tokens of 256 experts and k = 8, about a third
// in the k + 1 rounds of selection; they take 74 % of the issue slots.  65536 tokens,
// biased sigmoids in 8 groups, bf16: 33 - 40 us by how many tokens are in doubt (168 us
// with a wave a token, in double); 16384 x 160, softmax, float32: 8.3 - 9 us (34).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "common.h"
#include "rows.h"

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

using rows::lane64;
using rows::row_max;
using rows::row_sum;
using rows::wave_max;
using rows::wave_sum;

// the smallest of some lanes' values
__device__ __forceinline__ int least_of(uint64_t lanes, int v) {
  int least = INT32_MAX;
  while (lanes) {
    const int lane = __ffsll(static_cast<unsigned long long>(lanes)) - 1;
    least = min(least, __builtin_amdgcn_readlane(v, lane));
    lanes &= lanes - 1;
  }
  return least;
}

// LDS written by some lanes of a wave and read by others of the same wave
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// (no NaN reaches it: the middle of two values and infinity is the larger one,
// without fmaxf's instruction more that quiets a signalling NaN)
__device__ __forceinline__ float larger(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }
__device__ __forceinline__ float row_max(float v) {
  v = larger(v, __int_as_float(dpp_partner<1>(__float_as_int(v))));
  v = larger(v, __int_as_float(dpp_partner<2>(__float_as_int(v))));
  v = larger(v, __int_as_float(dpp_partner<4>(__float_as_int(v))));
  return larger(v, __int_as_float(dpp_partner<8>(__float_as_int(v))));
}
// exp(x) for x <= 0 (0 below -745) to about 1e-11: far closer than the float a
// weight is rounded to, in half the instructions of the full function.  With
// x = (n + f) ln 2, |f| <= 1/2, it is 2^n times the exponential series in f ln 2,
// whose terms end at (ln 2 / 2)^9 / 9!.
__device__ __forceinline__ double exp_of(double x) {
  const double t = fmax(x, -800.0) * 1.4426950408889634;
  const double n = rint(t);
  const double r = (t - n) * 0.6931471805599453;
  double e = 1.0 / 362880.0;
  e = fma(e, r, 1.0 / 40320.0);
  e = fma(e, r, 1.0 / 5040.0);
  e = fma(e, r, 1.0 / 720.0);
  e = fma(e, r, 1.0 / 120.0);
  e = fma(e, r, 1.0 / 24.0);
  e = fma(e, r, 1.0 / 6.0);
  e = fma(e, r, 0.5);
  e = fma(e, r, 1.0);
  e = fma(e, r, 1.0);
  return ldexp(e, static_cast<int>(n));
}

// In double: a sigmoid, and a bias held within the keys of unmasked experts (NaN: lowest).
__device__ __forceinline__ double sigmoid_of(double x) {
  const double z = exp(-fabs(x));
  return (x > 0.0 ? 1.0 : z) / (1.0 + z);
}
__device__ __forceinline__ double bias_of(float b) {
  return fmin(fmax(static_cast<double>(b), -kBiasLimit), kBiasLimit);
}

// a / b in double for b in the normal range, to about an ulp: Newton's iteration for
// 1 / b, then the quotient corrected by its own remainder
__device__ __forceinline__ double quotient(double a, double b) {
  double r = __builtin_amdgcn_rcp(b);
  r = fma(fma(-b, r, 1.0), r, r);
  r = fma(fma(-b, r, 1.0), r, r);
  const double q = a * r;
  return fma(fma(-b, q, a), r, q);
}

// The weight of this lane's chosen expert (lanes 0 .. k - 1 of 16; `on` in those
// whose expert is unmasked), from its logit lk; m and total: the largest logit of
// the row and the sum of exp(l - m), for a softmax over all.
__device__ __forceinline__ double chosen_weight(bool softmax, bool renorm, float scale, float lk, bool on, float m,
                                                double total) {
  const float top = row_max(on ? lk : -INFINITY);
  double w;
  if (softmax) {
    w = on ? exp_of(static_cast<double>(lk) - static_cast<double>(renorm ? top : m)) : 0.0;
  } else {
    const double x = lk, z = exp_of(-fabs(x));          // s = 1 / (1 + z) or z / (1 + z)
    double up = x > 0.0 ? 1.0 : z;
    // ratios survive where every sigmoid underflows: times exp(-top).  (By the token's own
    // logits alone: the two forms differ by some 1e-11, which can turn a rounding.)
    if (renorm && top < -600.f) up = exp_of(x - static_cast<double>(top));
    w = on ? quotient(up, 1.0 + z) : 0.0;
  }
  const double sum = renorm ? row_sum(w) : softmax ? total : 1.0;
  return sum > 0.0 ? scale * quotient(w, sum) : 0.0;
}

using LdsDoubles = __attribute__((address_space(3))) double;

// One token by one wave: lane holds experts lane, lane + 64, ...  `value` is E
// doubles of LDS of this wave.  Every lane of the wave calls it with the same t.
template <bool kBf16, typename Args>
__device__ __forceinline__ void gate_token(const Args& p, int64_t t, int lane, LdsDoubles* value) {
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
  if (p.check) raise_check(p.check, bad, MOE_CHECK_LOGITS);

  // scores, where the selection or the weights need all of them
  const bool two = p.top2 && p.keep < p.n_groups;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  double total = 1.0;
  if (p.bias || two || (p.softmax && !p.renorm)) {
    if (p.softmax) {
      m = static_cast<float>(wave_max(static_cast<double>(m)));
      if (m == -INFINITY) m = 0.f;   // nothing unmasked
      total = 0.0;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double x = l[j];
      if (p.softmax) total += s[j] = exp(x - m);   // 0 where masked
      else s[j] = sigmoid_of(x);
    }
    if (p.softmax) {
      total = wave_sum(total);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = total > 0.0 ? s[j] / total : 0.0;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = lane + 64 * j;
    double b = 0.0;
    if (p.bias && e < p.E) b = bias_of(p.bias[e]);
    key[j] = e >= p.E ? -INFINITY : !live[j] ? kMaskedKey : p.bias ? s[j] + b : static_cast<double>(l[j]);
    if (p.keep < p.n_groups && e < p.E) value[e] = !two ? key[j] : live[j] ? s[j] + b : -INFINITY;
  }

  if (p.keep < p.n_groups) {
    // lane g scores group g; a group stays if fewer than `keep` are ahead of it
    wave_lds_fence();
    double best = -INFINITY, second = -INFINITY;
    for (int i = 0; i < p.group_size; i += 8) {
      double v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)   // (8 reads in flight; lanes without a group read the last value)
        v[u] = value[min(lane * p.group_size + min(i + u, p.group_size - 1), p.E - 1)];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i + u < p.group_size) {
          second = fmax(second, fmin(best, v[u]));
          best = fmax(best, v[u]);
        }
    }
    const double score = two && second > -INFINITY ? best + second : best;
    int rank = 0;
    for (int g = 0; g < p.n_groups; ++g) {
      const double o = lane64(score, g);
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
    double bv = key[0];
    int bi = lane;
#pragma unroll
    for (int j = 1; j < 4; ++j)
      if (key[j] > bv) { bv = key[j]; bi = lane + 64 * j; }
    bi = least_of(__ballot(bv == wave_max(bv)), bi);
    if (lane == i) mine = bi;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (bi == lane + 64 * j) key[j] = -INFINITY;
  }

  // weights of the k experts, in double, rounded once; lanes 0 .. k - 1
  float lk = -INFINITY;
  if (lane < p.k) lk = load_logit<kBf16>(p.logits, row + mine);
  const bool on = lane < p.k && is_live(lk);
  const double w = chosen_weight(p.softmax, p.renorm, p.scale, on ? fminf(lk, FLT_MAX) : -INFINITY, on, m, total);
  if (lane < p.k) {
    p.idx[t * p.k + lane] = mine;
    p.w[t * p.k + lane] = static_cast<float>(w);
  }
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  return static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32)))) << 32 | lo;
}

// gate_token called, not inlined, from a loop that few tokens leave: its double
// constants would otherwise be kept in that loop's registers.  The arguments are
// read from the kernel's own (its first parameter), so nothing is copied for it.
using KernelArgs = const __attribute__((address_space(4))) GateArgs;
template <bool kBf16>
__device__ __noinline__ void gate_token_call(KernelArgs* p, int64_t t, LdsDoubles* value) {
  // a function's arguments come in vector registers: they are the wave's all the same
  const uint64_t at = reinterpret_cast<uint64_t>(p);
  p = reinterpret_cast<KernelArgs*>(uniform64(at));
  gate_token<kBf16>(*p, static_cast<int64_t>(uniform64(static_cast<uint64_t>(t))), threadIdx.x & 63, value);
}

// ------------------------------------------------------------ 16 lanes a token
// (bound control on, which no lane of these pairings needs, lets the move be part of
// the maximum's own instruction)
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, true)));
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, true)));
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
__device__ __forceinline__ int rotated_bits(int v) {
  return __builtin_amdgcn_mov_dpp(v, 0x120 + N, 0xf, 0xf, false);
}
template <int N>
__device__ __forceinline__ float rotated(float v) {
  return __int_as_float(rotated_bits<N>(__float_as_int(v)));
}

// Groups ahead of this lane's, the groups being kLanes lanes each: `rep` is the
// group's score in its lanes and NaN, ahead of nothing, in lanes without a group.
template <int kLanes, int N = kLanes>
__device__ __forceinline__ int count_ahead(float rep, float score, int l16) {
  if constexpr (N >= 16) return 0;
  else {
    const float o = rotated<N>(rep);   // of the group N / kLanes before, around the 16
    return (o > score || (o == score && l16 >= N)) + count_ahead<kLanes, N + kLanes>(rep, score, l16);
  }
}

// How many of the token's other 15 lanes come before this one, by value and then index.
template <int N>
__device__ __forceinline__ int rank16(double v, int e) {
  if constexpr (N >= 16) return 0;
  else {
    const double o = __hiloint2double(rotated_bits<N>(__double2hiint(v)), rotated_bits<N>(__double2loint(v)));
    return ahead(o, rotated_bits<N>(e), v, e) + rank16<N + 1>(v, e);
  }
}

// The largest key below `best`: with unsigned wrap-around the differences of the
// keys below it exceed those of the keys at or over it, so nothing has to be
// struck out between two rounds.
template <int V>
__device__ __forceinline__ uint32_t next_key(const uint32_t (&key)[V], uint32_t best) {
  uint32_t d = key[0] - best;
#pragma unroll
  for (int j = 1; j < V; ++j) d = max(d, key[j] - best);
  return best + row_max(d);
}

enum By { kByLogit, kBySigmoid, kBySoftmax };          // what the selection compares
enum Weights { kSoftmaxKept, kSoftmaxAll, kSigmoids };  // softmax over the kept logits, over all; sigmoids

constexpr float kLog2e = 1.4426950408889634f;
// Keys are cut from floats between 2^23 and 2^24, whose low 23 bits count units:
// 8 bits further up they leave room for the index.
constexpr float kZero = 8388608.f;     // 2^23: a key's value of 0

// Lane i of a token's 16 holds `per` consecutive experts (at most V) of one group:
// groups begin at multiples of `lanes` lanes.  A wave takes 4 tokens at a time.
// Blocks a CU is given: what the variant with the most registers (biased sigmoids: 131
// at 12 slots, 139 at 16, 174 - 195 at 32) leaves room for.  Those by the logit or a softmax
// (105 - 118 at 12 and 16) would fit four; they were not tried with them.
constexpr int gate_blocks_per_cu(int V) { return V > 16 ? 2 : V > 8 ? 3 : 4; }

template <bool kBf16, int V, By kBy, Weights kW>
__global__ __launch_bounds__(256, gate_blocks_per_cu(V)) void gate_kernel(GateArgs p, int lanes_log2, int per) {
  __shared__ double value[4][moe::kMaxExperts];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, l16 = lane & 15;
  const int lanes = 1 << lanes_log2;
  const int group = l16 >> lanes_log2;                // == p.n_groups or more: an idle lane
  const int inside = (l16 & (lanes - 1)) * per;
  const int e0 = group * p.group_size + inside;
  const int n = group < p.n_groups ? max(0, min(per, p.group_size - inside)) : 0;   // this lane's experts
  const int64_t total = p.T * p.E;

  // A key is (value << 8) + c: the value at least 3, 2 for a masked expert (-inf is
  // cut to it), 1 where the group is not kept; c = 255 - index, or what takes a slot
  // without an expert below the masked ones.
  uint32_t c[V];
#pragma unroll
  for (int j = 0; j < V; ++j) c[j] = j < n ? static_cast<uint32_t>(255 - e0 - j) : static_cast<uint32_t>(-256);

  // b: 0, or the bias in units, and -inf in a slot without an expert; the units of a
  // score and the bound on the error of two values' difference
  float b[V];
  float scale = 0x1p19f;         // units of a logit, down to 16 below the largest.  The cut is
  float offset = 0.f;            // monotone: only equal keys of unequal logits are in doubt
  float near = 0.f, group_near = 0.f;
  bool wild = false;             // biases that no units measure: every token goes to the doubles
#pragma unroll
  for (int j = 0; j < V; ++j) b[j] = 0.f;
  if constexpr (kBy != kByLogit) {
    if (p.bias)
#pragma unroll
      for (int j = 0; j < V; ++j) b[j] = p.bias[min(e0 + j, p.E - 1)];
    float lo = INFINITY, hi = -INFINITY;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      odd |= (j < n) & !(fabsf(b[j]) <= 1e30f);
      lo = fminf(lo, j < n ? b[j] : INFINITY);
      hi = fmaxf(hi, j < n ? b[j] : -INFINITY);
    }
    if (odd) lo = hi = INFINITY;
    lo = -row_max(-lo);
    hi = row_max(hi);
    wild = !(hi < INFINITY);
    scale = (kZero - 1024.f) / (1.f + (hi - lo));
    // from the lowest bias on, so that every key lies in 16 .. 2^23 whatever the biases have in common
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = fmaf(b[j] - lo, scale, kZero + 16.f);
    // what a score of 0 without a bias has in these units; whole, as all values are
    offset = rintf(fmaf(-lo, scale, kZero + 16.f));
    // the largest |s + b|, in units.  In double, where the order is defined, it is rounded too
    const float most = (1.f + fmaxf(fabsf(lo), fabsf(hi))) * scale, defined = most * 0x1p-50f;
    // s: exp2's argument 0.4 u (u = 2^-24), exp2 0.5, the sum 1 and the reciprocal 2; a softmax's
    // sum of up to 32 values in sequence and 4 steps 36 u more, the terms' own errors in it
    // at most 10 u, and the scaled reciprocal.  b and the sum are below 2^24 units: half a unit
    // each, and b - lo u of itself.
    const float err = (kBy == kBySigmoid ? 5.f : 53.f) * 0x1p-24f * scale + 1.f + (hi - lo) * scale * 0x1p-24f;
    near = 2.f * err + 0.5f + defined;
    // a sum of two: twice that; below 2^24 units the offset half a unit (of a group with one
    // expert it is not taken off) and the sum 1 + most u, each once on both sides; beyond,
    // steps of at most u of the offset once and of `most` twice
    const float big = fmaxf(most, fabsf(offset));
    group_near = !p.top2 ? near
                         : 4.f * err + 3.f + most * 0x1p-23f + (big > 2.f * kZero ? big * 0x1p-21f : 0.f) + defined;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) b[j] = j < n ? b[j] : -INFINITY;

  for (int64_t base = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * 4; base < p.T;
       base += static_cast<int64_t>(gridDim.x) * 16) {
    const int64_t t = base + (lane >> 4);
    const bool active = t < p.T;
    const int64_t row = (active ? t : 0) * p.E;
    float l[V];
    const int64_t at = row + e0;
    if (at + V <= total) {         // (what follows a lane's own experts is not looked at)
      if constexpr (kBf16) {
        uint32_t raw[V / 2];
        __builtin_memcpy(raw, static_cast<const uint16_t*>(p.logits) + at, sizeof(raw));
#pragma unroll
        for (int j = 0; j < V; ++j) l[j] = __uint_as_float((j & 1) ? raw[j / 2] & 0xffff0000u : raw[j / 2] << 16);
      } else {
        __builtin_memcpy(l, static_cast<const float*>(p.logits) + at, sizeof(l));
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) l[j] = load_logit<kBf16>(p.logits, min(at + j, total - 1));
    }
    if (p.check) {
      bool bad = false;
#pragma unroll
      for (int j = 0; j < V; ++j) bad |= (j < n) & ((l[j] != l[j]) | (l[j] == INFINITY));
      raise_check(p.check, bad && active, MOE_CHECK_LOGITS);
    }

    // v: what is compared, in units (a logit as it is), -inf where masked or without an expert
    float v[V];
    float m = 0.f;
    double sum64 = 1.0;
    if constexpr (kBy == kBySigmoid) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l[j] * -kLog2e));
        v[j] = is_live(l[j]) ? fmaf(s, scale, b[j]) : -INFINITY;
      }
    } else {
      m = -INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (kBy == kByLogit) l[j] += b[j];
        else if (j >= n) l[j] = -INFINITY;
        l[j] = is_live(l[j]) ? fminf(l[j], FLT_MAX) : -INFINITY;
        m = larger(m, l[j]);
      }
      m = row_max(m);
      if (m == -INFINITY) m = 0.f;   // nothing unmasked
      if constexpr (kW == kSoftmaxAll) {   // the weights' denominator
        sum64 = 0.0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sum64 += exp_of(static_cast<double>(l[j]) - static_cast<double>(m));
          __builtin_amdgcn_sched_barrier(0);   // one exponential's registers at a time
        }
        sum64 = row_sum(sum64);
      }
      if constexpr (kBy == kBySoftmax) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[j] = __builtin_amdgcn_exp2f((l[j] - m) * kLog2e);
          sum += v[j];
        }
        sum = row_sum(sum);
        const float inv = sum > 0.f ? scale * __builtin_amdgcn_rcpf(sum) : 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = l[j] > -INFINITY ? fmaf(v[j], inv, b[j]) : -INFINITY;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = l[j];
      }
    }

    bool doubt = wild, kept = true;
    if (p.keep < p.n_groups) {
      float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (kBy != kByLogit) m2 = __builtin_amdgcn_fmed3f(m1, m2, v[j]);
        m1 = larger(m1, v[j]);
      }
      auto join = [&](int o1, int o2) {
        if (kBy != kByLogit) m2 = larger(__builtin_amdgcn_fmed3f(m1, m2, __int_as_float(o1)), __int_as_float(o2));
        m1 = larger(m1, __int_as_float(o1));
      };
      if (lanes > 1) join(dpp_partner<1>(__float_as_int(m1)), dpp_partner<1>(__float_as_int(m2)));
      if (lanes > 2) join(dpp_partner<2>(__float_as_int(m1)), dpp_partner<2>(__float_as_int(m2)));
      if (lanes > 4) join(dpp_partner<4>(__float_as_int(m1)), dpp_partner<4>(__float_as_int(m2)));
      // (a score of 0 has `offset` units: counted once in a sum of two)
      const float score = kBy != kByLogit && p.top2 && m2 > -INFINITY ? m1 + (m2 - offset) : m1;
      const bool real = group < p.n_groups;
      const float rep = real ? score : NAN;
      const int rank = lanes == 1 ? count_ahead<1>(rep, score, l16) : lanes == 2 ? count_ahead<2>(rep, score, l16)
                       : lanes == 4 ? count_ahead<4>(rep, score, l16) : count_ahead<8>(rep, score, l16);
      kept = real && rank < p.keep;
      if constexpr (kBy != kByLogit) {
        // the last group kept against the first one left out
        const float low = -row_max(kept ? -score : -INFINITY);
        const float high = row_max(real && !kept ? score : -INFINITY);
        doubt |= high > -INFINITY && !(low - high > group_near);
      }
    }

    uint32_t key[V];
    const float low = kZero + (kept ? 2.f : 1.f), high = kept ? 2.f * kZero - 1.f : low;
    const float down = 2.f * kZero - 64.f - m * scale;   // (by logit: the largest near the top)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float f = __builtin_amdgcn_fmed3f(kBy == kByLogit ? fmaf(v[j], scale, down) : v[j], low, high);
      key[j] = (__float_as_uint(f) << 8) + c[j];
    }

    // lane i takes the i-th key, lane k the best one left
    uint32_t best = 0, mine = 0;
#pragma unroll 1   // (a small call is bound by fetching its code)
    for (int i = 0; i <= p.k; ++i) {
      best = next_key<V>(key, best);
      if (l16 == i) mine = best;
    }
    int e = min(255 - static_cast<int>(mine & 255u), p.E - 1);
    bool some = l16 <= p.k && mine >= 768u;      // an unmasked expert
    const bool group_doubt = doubt;
    // a logit too far below the largest is cut to a masked one's value as well
    doubt |= l16 < p.k && !some;
    float lk = some ? load_logit<kBf16>(p.logits, row + e) : -INFINITY;
    lk = fminf(lk, FLT_MAX);
    const uint32_t q = mine >> 8, q_next = static_cast<uint32_t>(next_lane(static_cast<int>(mine))) >> 8;
    bool same = lk == __int_as_float(next_lane(__float_as_int(lk)));
    if constexpr (kBy != kByLogit) {
      const float bk = p.bias && some ? p.bias[e] : 0.f;
      // (moved in all lanes, before the comparison: from a lane that a branch has switched
      // off its reader would get its own value back)
      const float next_bk = __int_as_float(next_lane(__float_as_int(bk)));
      same &= bk == next_bk;
    }
    const bool close = some && l16 < p.k && q_next >= 3u && static_cast<float>(q - q_next) <= near;
    doubt |= close && !same;
    // the last one taken and the first one left are equal: the one after them may belong before both
    const bool tie = close && same && l16 == p.k - 1;
    if (__any(tie)) {
      const uint32_t next = next_key<V>(key, best);
      doubt |= tie && next < best && (next >> 8) >= 3u && static_cast<float>(q - (next >> 8)) <= near;
    }
    uint64_t doubts = __ballot(doubt && active);
    bool redo = (doubts >> (lane & 48)) & 0xffffu;
    if (kBy != kBySoftmax && doubts) {
      // The 16 best by key in the order of their exact values.  That is the answer where
      // the 16th lies clearly below the k-th, so that none of the others can pass it.
      const uint32_t last = static_cast<uint32_t>(__shfl(static_cast<int>(mine), (lane & 48) | (p.k - 1)));
      best = last;
#pragma unroll 1
      for (int i = p.k; i < 16; ++i) {
        const uint32_t next = next_key<V>(key, best);
        best = best != 0u && next < best ? next : 0u;   // (past the last key the largest comes again)
        if (l16 == i) mine = best;
      }
      e = min(255 - static_cast<int>(mine & 255u), p.E - 1);
      const bool there = mine >= 512u;
      const float raw = there ? load_logit<kBf16>(p.logits, row + e) : -INFINITY;
      const double x = fminf(raw, FLT_MAX);
      double exact = x;
      // (without a bias by the logit: large ones' sigmoids are 1 in double too)
      if constexpr (kBy == kBySigmoid)
        if (p.bias) exact = sigmoid_of(x) + bias_of(p.bias[e]);
      exact = !there ? -INFINITY : is_live(raw) ? exact : kMaskedKey;
      const uint32_t last_q = static_cast<uint32_t>(__shfl(static_cast<int>(mine), (lane & 48) | 15)) >> 8;
      redo = redo && (group_doubt || !(last_q < 2u || static_cast<float>((last >> 8) - last_q) > near));
      const int to = ((lane & 48) + rank16<1>(exact, e)) * 4;
      e = __builtin_amdgcn_ds_permute(to, e);
      lk = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(raw)));
      some = l16 < p.k && is_live(lk);
      lk = some ? fminf(lk, FLT_MAX) : -INFINITY;
      doubts = __ballot(redo && active);
    }

    // weights in double, rounded once
    const double w = chosen_weight(kW != kSigmoids, kW == kSigmoids ? p.renorm : kW == kSoftmaxKept, p.scale, lk,
                                   some && l16 < p.k, m, sum64);
    if (active && !redo && l16 < p.k) {
      p.idx[t * p.k + l16] = e;
      p.w[t * p.k + l16] = static_cast<float>(w);
    }
    if (doubts)
#pragma unroll 1
      for (int i = 0; i < 4; ++i)
        if ((doubts >> (16 * i)) & 0xffffu)
          gate_token_call<kBf16>((KernelArgs*)__builtin_amdgcn_kernarg_segment_ptr(), base + i, (LdsDoubles*)value[wave]);
  }
}

// One wave a token, in double throughout: more groups than 16 lanes hold.
template <bool kBf16>
__global__ __launch_bounds__(256) void gate_wave_kernel(GateArgs p) {
  __shared__ double value[4][moe::kMaxExperts];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (t >= p.T) return;
  gate_token<kBf16>(p, t, lane, (LdsDoubles*)value[wave]);
}

template <int V, bool kBf16, By kBy, Weights kW>
void launch_by(const GateArgs& p, int lanes_log2, int per, hipStream_t s) {
  constexpr int64_t kBlocks = 256 * gate_blocks_per_cu(V);
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(kBlocks, moe::ceil_div(p.T, 16)));
  gate_kernel<kBf16, V, kBy, kW><<<blocks, 256, 0, s>>>(p, lanes_log2, per);
}

template <bool kBf16, By kBy, Weights kW>
void launch_slots(GateArgs p, hipStream_t s) {
  int lanes_log2 = 4;
  if (p.keep == p.n_groups) {
    p.n_groups = p.keep = 1;
    p.group_size = p.E;
  }
  while ((16 >> lanes_log2) < p.n_groups) --lanes_log2;
  const int per = static_cast<int>(moe::ceil_div(p.group_size, 1 << lanes_log2));
  if (per <= 2) launch_by<2, kBf16, kBy, kW>(p, lanes_log2, per, s);
  else if (per <= 4) launch_by<4, kBf16, kBy, kW>(p, lanes_log2, per, s);
  else if (per <= 8) launch_by<8, kBf16, kBy, kW>(p, lanes_log2, per, s);
  else if (per <= 12) launch_by<12, kBf16, kBy, kW>(p, lanes_log2, per, s);
  else if (per <= 16) launch_by<16, kBf16, kBy, kW>(p, lanes_log2, per, s);
  else launch_by<32, kBf16, kBy, kW>(p, lanes_log2, per, s);
}

template <bool kBf16>
void launch_gate(const GateArgs& p, hipStream_t s) {
  const bool by_logit = !p.bias && !(p.top2 && p.keep < p.n_groups);
  if (p.keep < p.n_groups && p.n_groups > 16)
    gate_wave_kernel<kBf16><<<static_cast<unsigned>(moe::ceil_div(p.T, 4)), 256, 0, s>>>(p);
  else if (!p.softmax && by_logit) launch_slots<kBf16, kByLogit, kSigmoids>(p, s);
  else if (!p.softmax) launch_slots<kBf16, kBySigmoid, kSigmoids>(p, s);
  else if (p.renorm && by_logit) launch_slots<kBf16, kByLogit, kSoftmaxKept>(p, s);
  else if (p.renorm) launch_slots<kBf16, kBySoftmax, kSoftmaxKept>(p, s);
  else if (by_logit) launch_slots<kBf16, kByLogit, kSoftmaxAll>(p, s);
  else launch_slots<kBf16, kBySoftmax, kSoftmaxAll>(p, s);
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

// With the slot I after this lane's: its part, if it is for the same expert; and
// whether the slot I before is for that expert already.
template <int I>
__device__ __forceinline__ void join_repeats(int e, float slot, int l16, int k, bool& first, float& v) {
  if constexpr (I < moe::kMaxTopK) {
    const int after = __float_as_int(rotated<16 - I>(__int_as_float(e)));
    const float part = rotated<16 - I>(slot);
    if (after == e && l16 + I < k) v += part;
    if (__float_as_int(rotated<I>(__int_as_float(e))) == e && l16 >= I) first = false;
    join_repeats<I + 1>(e, slot, l16, k, first, v);
  }
}

// 16 lanes a token; a lane holds pieces of 8 consecutive experts, 128 apart.  The
// k parts meet the zeros (or the dense term) in LDS, so the row is written once,
// in whole pieces; float32 throughout.  60013 x 256 bf16, sparse: 12.7 us, bound by
// memory (the k scattered logits touch a whole row, 60 MB in all; a wave a token: 32
// us).  16384 x 160 float32, dense: 7.7 us for 21 MB, bound by the chain index ->
// logit -> row of one round of waves.
template <bool kBf16, bool kDense>
__global__ __launch_bounds__(256) void gate_grad_kernel(GateBwdArgs p) {
  constexpr int kPieces = moe::kMaxExperts / 128;
  __shared__ float4 parts[16][moe::kMaxExperts / 4];
  const int l16 = threadIdx.x & 15;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const bool active = t < p.T;
  const int64_t row = (active ? t : 0) * p.E;
  float4* mine = parts[threadIdx.x >> 4];

  rows::Raw8<kBf16> raw[kPieces];
  if constexpr (kDense)
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const int at = c * 128 + l16 * 8;
      raw[c] = {};
      if (active && at < p.E) raw[c] = rows::load8_part<kBf16>(p.logits, row + at, p.E - at);
    }

  // lanes 0 .. k - 1: the slot's expert, gradient and logit
  int e = -1;
  float g = 0.f, lk = -INFINITY;
  bool bad = false;
  if (active && l16 < p.k) {
    e = p.idx[t * p.k + l16];
    bad = e < 0 || e >= p.E;
    if (bad) {
      e = -1;
    } else {
      g = p.scale * p.d_w[t * p.k + l16];
      lk = load_logit<kBf16>(p.logits, row + e);
    }
  }
  if (p.check) raise_check(p.check, bad, MOE_CHECK_INDEX);
  const bool on = is_live(lk);
  lk = on ? fminf(lk, FLT_MAX) : -INFINITY;
  if (!on) g = 0.f;

  float l[kPieces][8];
  float m = -INFINITY, total = 0.f;
  if constexpr (kDense) {
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const int n = active ? p.E - (c * 128 + l16 * 8) : 0;
      rows::unpack8<kBf16>(raw[c], l[c]);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        l[c][u] = u < n && is_live(l[c][u]) ? fminf(l[c][u], FLT_MAX) : -INFINITY;
        m = larger(m, l[c][u]);
      }
    }
    m = row_max(m);
    const float top = m > -INFINITY ? m : 0.f;
#pragma unroll
    for (int c = 0; c < kPieces; ++c)
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        l[c][u] = __builtin_amdgcn_exp2f((l[c][u] - top) * kLog2e);   // (0 where masked)
        total += l[c][u];
      }
    total = row_sum(total);
  }

  float slot;   // the slot's part of d_l[e]
  float common = 0.f;
  if (p.softmax) {
    if (!kDense) m = row_max(lk);
    float s = on ? expf(lk - m) : 0.f;
    if (!kDense) total = row_sum(s);
    s = total > 0.f ? s / total : 0.f;
    common = row_sum(g * s);
    slot = kDense ? g * s : s * (g - common);
  } else {
    const float z = expf(-fabsf(lk));          // s = 1 / (1 + z) or z / (1 + z)
    const float other = on ? (lk > 0.f ? z : 1.f) / (1.f + z) : 0.f;   // 1 - s
    if (p.renorm) {
      const float top = fminf(row_max(lk), 0.f);
      const float s = !on ? 0.f : (lk > 0.f ? 1.f : expf(lk - top)) / (1.f + z);
      const float sum = row_sum(s);
      const float r = sum > 0.f ? s / sum : 0.f;
      slot = r * (g - row_sum(g * r)) * other;
    } else {
      slot = on ? g * ((lk > 0.f ? 1.f : z) / (1.f + z)) * other : 0.f;
    }
  }

  // an expert named twice: its first slot takes the others' parts, in slot order
  bool first = e >= 0;
  float v = slot;
  join_repeats<1>(e, slot, l16, p.k, first, v);
#pragma unroll
  for (int c = 0; c < kPieces; ++c)
    if (c * 128 + l16 * 8 < p.E) mine[c * 32 + l16 * 2] = mine[c * 32 + l16 * 2 + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
  wave_lds_fence();
  if (first) reinterpret_cast<float*>(mine)[e] = v;
  wave_lds_fence();
  if (!active) return;
  const float share = kDense && total > 0.f ? common / total : 0.f;
#pragma unroll
  for (int c = 0; c < kPieces; ++c) {
    const int at = c * 128 + l16 * 8, n = p.E - at;
    if (n <= 0) continue;
    const float4 a = mine[c * 32 + l16 * 2], b = mine[c * 32 + l16 * 2 + 1];
    float d[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if constexpr (kDense)
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (l[c][u] > 0.f) d[u] = fmaf(-l[c][u], share, d[u]);
    rows::store8_part<kBf16>(p.d_logits, row + at, n, d);
  }
}

template <bool kBf16>
void launch_gate_grad(const GateBwdArgs& p, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>(moe::ceil_div(p.T, 16));
  if (p.softmax && !p.renorm) gate_grad_kernel<kBf16, true><<<blocks, 256, 0, s>>>(p);
  else gate_grad_kernel<kBf16, false><<<blocks, 256, 0, s>>>(p);
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
  if (dt == MOE_BF16) launch_gate_grad<true>(p, as_stream(stream));
  else launch_gate_grad<false>(p, as_stream(stream));
  return hip_status(hipGetLastError(), "moe_gate_backward launch");
}
