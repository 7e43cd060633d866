// moe_mx_expert_ffn: the experts' FFNs on weights in microscaled 4-bit blocks,
// activations quantised by row blocks to 6 or 4 bits, on gfx950's scaled matrix
// instructions (v_mfma_scale_f32_*_f8f6f4: the operands' codes go in as they are
// kept, each block of 32 along K with its scale byte, fp32 accumulation).
//
// Q(x) the rows' quantised values:  h = act(Q(x) Wg^T, Q(x) Wu^T), y = Q(h) Wd^T.
// Three launches:
//   prepare:  the rows of x quantised, one block a lane, and in block 0 the list of
//             row tiles from the slot table;
//   gate/up:  per row tile and its columns of h, gate and up side by side; the
//             epilogue trades accumulators between lanes until each holds 32
//             adjacent columns of a row, quantises them in registers and writes
//             their codes;
//   down:     y = Q(h) Wd^T.
// A tile's weight rows, half of them the gate's and half the up weights' for SwiGLU:
// 256 beside 256 rows of A, 128 beside 64 or 128, 64 (or 32) beside the stream's 16.
// Two kernels multiply.  tile_kernel: BM rows x 128 or 256 weight rows a block, operands
// straight into LDS, 32x32x64 instructions.  stream_kernel: at most 16 rows by 64
// weight rows a block, K split over the block's waves: for few rows the time is the
// weights' bytes.
//
// Measured, and what bounds it: 8192 tokens, two of 8 experts of 4096 x 14336, in 6 bits
// 1.72 ms, 3.35 PFLOP/s (in 4 bits 1.57, 3.7): gate/up 1.15 and down 0.55.  The K loop runs at
// some 83 % of what the instructions reach alone under the power limit (5.1 to 5.3 PFLOP/s,
// 4 by 4 bits 5.6 to 6.1, from card to card), and beside a tile's epilogue, 6 to 7 us of a
// gate/up tile's 41 (32 K steps; a down tile has 112), nothing runs.  4001 tokens, two of 32
// GELU experts of 1024 x 4096, 115 us: gate/up 67, 8 K steps a tile beside the GELU's vector
// issue, and down 52, two rounds of tiles for 1.25.  Few rows an expert are the weights'
// bytes: 61 tokens, six of 160 experts of 5120 x 1536, 150 to 160 us (5 TB/s), 1021 tokens in
// 4 bits 463 to 477, one token 29.  Float rows for bf16 ones add the bytes of x and y (8192
// tokens 1.78 ms, 4001 of the GELU experts 125 us).
//
// Why 6 bits and not 8.  Lane group g (lane / rows) of an operand holds K = 32 g ..
// 32 g + 31 and their scale.  The instruction sums eight products at a time, each
// cut at 2^-13 of the largest's leading bit (found by probing): of e2m1 by e2m1 or
// e2m3, whose products are multiples of 2^-4 up to 45, that cuts nothing, and the
// sums of eight are added in fp32; of e2m1 by e4m3 it cuts products at some 2^-13
// of the largest beside them.  e2m3 has e4m3's four significant bits and runs at
// the 4-bit rate.
//
// Activations in the workspace, one row for each of the M.  K-major: for every step
// of 128 K values the rows' pieces follow one another, 64 bytes of codes (all of
// e2m1, the first two thirds of each block of e2m3), in a second plane e2m3's last 32
// bytes, and one dword of four scales.  A tile's step is then a run of whole lines
// whatever K is.  (Row-major codes were gathered through the row map before: 64- and
// 32-byte pieces, and the L2's request rate bounded the large products.)
#include <algorithm>

#include "common.h"
#include "gemm.h"
#include "mx.h"
#include "rows.h"

namespace {

using moe::ceil_div;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStepK = 128;   // K values of a step: four blocks
constexpr int kStreamRows = 16;

// One product: rows of A (K-major planes of M rows) times the experts' weights (codes
// [E, N, K / 2], scales [E, N, K / 32]); B1/S1 the up weights beside the gate's.
struct MxGemm {
  const uint8_t *A, *A2, *As;
  const uint8_t *B0, *B1, *S0, *S1;
  int K, N;
  int64_t M;
  const int4* tiles;   // expert, first row, end row
  const int32_t* n_tiles;
  int n_col_tiles;
  void* C;             // y [M, N], or h's codes
  uint8_t *C2, *Cs;    // h's second plane and scales
  int big;             // the experts' weights are far more than the last-level cache holds
};

// A block's codes and scale to their places in planes of M rows.
template <int kBits>
__device__ __forceinline__ void store_block(const mx::Operand& o, int64_t row, int64_t M, int block, uint8_t* q,
                                            uint8_t* q2, uint8_t* scale) {
  const int64_t at = (block / 4 * M + row) * 4 + block % 4;
  *reinterpret_cast<uint4*>(q + at * 16) = o.first;
  if constexpr (kBits == mx::kF6) *reinterpret_cast<uint2*>(q2 + at * 8) = o.rest;
  scale[at] = static_cast<uint8_t>(o.byte);
}

// ------------------------------------------------------------------- preparation
// Block (0, 0) lists the row tiles; blocks (1 and up, k) quantise step k of the M rows of
// x (through the row map; rows mapped outside x are zero), one block of 32 a lane.
template <bool kBf16, int kBits>
__global__ __launch_bounds__(256) void prepare_kernel(const void* __restrict__ x, const int32_t* __restrict__ row_src,
                                                      int64_t n_src, int K, uint8_t* __restrict__ q,
                                                      uint8_t* __restrict__ q2, uint8_t* __restrict__ scale,
                                                      const int32_t* __restrict__ slot_off,
                                                      const int32_t* __restrict__ slot_expert,
                                                      const int32_t* __restrict__ n_slots, int max_slots, int64_t M,
                                                      int E, int rows_per_tile, int cap, int4* __restrict__ tiles,
                                                      int32_t* __restrict__ n_tiles, int32_t* __restrict__ check) {
  if (blockIdx.x == 0) {
    if (blockIdx.y > 0) return;
    __shared__ int wave_sum[4];
    __shared__ int before;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int named = *n_slots;
    const int n = min(max(named, 0), max_slots);
    bool bad = named != n;
    if (tid == 0) before = 0;
    __syncthreads();
    for (int s0 = 0; s0 < n; s0 += 256) {
      const int s = s0 + tid;
      int64_t lo = 0, hi = 0;
      int e = -1;
      if (s < n) {
        lo = slot_off[s];
        hi = slot_off[s + 1];
        e = slot_expert[s];
        bad |= lo < 0 || hi < lo || hi > M || e < 0 || e >= E;
        lo = min<int64_t>(max<int64_t>(lo, 0), M);
        hi = min<int64_t>(max<int64_t>(hi, lo), M);
      }
      const int mine = e >= 0 && e < E ? static_cast<int>((hi - lo + rows_per_tile - 1) / rows_per_tile) : 0;
      int sum = mine;   // inclusive prefix sum over the block
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(sum, off);
        if (lane >= off) sum += v;
      }
      if (lane == 63) wave_sum[wave] = sum;
      __syncthreads();
      int at = before + sum - mine, total = 0;
      for (int w = 0; w < 4; ++w) {
        if (w < wave) at += wave_sum[w];
        total += wave_sum[w];
      }
      for (int i = 0; i < mine; ++i)
        if (at + i < cap) {
          const int64_t r = lo + static_cast<int64_t>(i) * rows_per_tile;
          tiles[at + i] = make_int4(e, static_cast<int>(r), static_cast<int>(min<int64_t>(r + rows_per_tile, hi)), 0);
        }
      __syncthreads();
      if (tid == 0) before += total;
      __syncthreads();
    }
    if (tid == 0) *n_tiles = min(before, cap);
    if (check) raise_check(check, bad, MOE_CHECK_SLOTS);
    return;
  }
  const int64_t i = static_cast<int64_t>(blockIdx.x - 1) * 256 + threadIdx.x, row = i >> 2;
  const int block = static_cast<int>(blockIdx.y) * 4 + static_cast<int>(i & 3);
  bool bad = false;
  if (row < M) {
    const int64_t src = row_src ? row_src[row] : row;
    float v[32] = {};
    if (src >= 0 && src < n_src)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float part[8];
        rows::unpack8<kBf16>(rows::load8<kBf16>(x, src * K + block * mx::kBlock + 8 * u), part);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * u + j] = part[j];
      }
    const mx::Operand o = mx::encode_block<kBits>(v);
    bad = o.byte == 255;
    store_block<kBits>(o, row, M, block, q, q2, scale);
  }
  if (check) raise_check(check, bad, MOE_CHECK_BLOCKS);
}

// --------------------------------------------------------------------- products
// Weights first: the accumulators come out transposed, a lane holding adjacent
// output columns of one row.  kOp picks the scale dwords' byte.
template <int kBits>
constexpr int kFormat = kBits == mx::kF6 ? 2 : 4;   // the instruction's names of e2m3 and e2m1
struct Frag {
  i32x4 first;
  i32x2 rest;
};
// The instruction reads as many of the eight registers as the format has.
__device__ __forceinline__ i32x8 wide(const i32x4& v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }
template <int kBits>
__device__ __forceinline__ i32x8 wide(const Frag& f) {
  if constexpr (kBits == mx::kF6)
    return __builtin_shufflevector(f.first, __builtin_shufflevector(f.rest, f.rest, 0, 1, -1, -1), 0, 1, 2, 3, 4, 5, -1, -1);
  else return wide(f.first);
}
template <int kBits, int kOp>
__device__ __forceinline__ f32x16 mma32(const i32x4& w, const Frag& a, const f32x16& c, uint32_t sw, uint32_t sa) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide(w), wide<kBits>(a), c, 4,
                                                         kFormat<kBits>, kOp, sw, kOp, sa);
}
template <int kBits>
__device__ __forceinline__ f32x4 mma16(const i32x4& w, const Frag& a, const f32x4& c, uint32_t sw, uint32_t sa) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(w), wide<kBits>(a), c, 4,
                                                          kFormat<kBits>, 0, sw, 0, sa);
}

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t r, int off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// Tile l of total_m x n_col_tiles: eight row tiles by the columns (gemm.h).
__device__ __forceinline__ void tile_at(int l, int total_m, int n_col_tiles, int* mt, int* nt) {
  const int grp = l / (kGroupM * n_col_tiles);
  const int gsz = min(kGroupM, total_m - grp * kGroupM);
  const int li = l - grp * kGroupM * n_col_tiles;
  *mt = grp * kGroupM + li % gsz;
  *nt = li / gsz;
}
// Block b's of `total` tiles, each XCD's in a run.
__device__ __forceinline__ int xcd_run(int b, int total) {
  const int xcd = b & 7, q = total >> 3, rem = total & 7;
  return xcd * q + min(xcd, rem) + (b >> 3);
}

// z Phi(z), the exact GELU: Phi(-|z|) = R(t) 2^(-z^2 log2(e) / 2), t = 1 / (1 + 0.3 |z|), R a
// polynomial fitted here (least largest relative error over |z| <= 13.2: 1.5e-7).  h is off
// by at most (16 + z^2) 2^-24 of itself, the exponent's rounding being the z^2: a negative
// z's h is a tail of its own and not 1 + erf, which has cancelled by then.  Fifteen
// instructions and two of the quarter rate, where erff takes some 36.
__device__ __forceinline__ float fast_gelu(float z) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.3f, 1.f));
  float p = fmaf(t, 0.0361417732f, -0.159168098f);
  p = fmaf(p, t, 0.209781963f);
  p = fmaf(p, t, -0.0568914098f);
  p = fmaf(p, t, 0.130297077f);
  p = fmaf(p, t, 0.099370426f);
  p = fmaf(p, t, 0.120845415f);
  p = fmaf(p, t, 0.119622796f) * t;
  const float tail = p * __builtin_amdgcn_exp2f(z * z * -0.72134752f);
  return fmaxf(z, 0.f) - fabsf(z * tail);
}

// What the epilogue makes of the accumulators.
enum MxEpi { kMxSwiGLU = 0, kMxGELU = 1, kMxBf16 = 2, kMxF32 = 3 };
constexpr int mats(int epi) { return epi == kMxSwiGLU ? 2 : 1; }

// ---- large batches ---------------------------------------------------------------
// A block: BM rows by BN weight rows.  LDS: stages of A (a K step of 128: two planes and
// the scales), stages of the weights' codes, 256 K values each, and two buffers of the
// weights' scales for 512.
// 256 K values are whole 128-byte lines of a weight row: 64-byte pieces a step apart
// fetched a third of the lines twice (61 tokens of 160 experts, 64-row tiles: 5.8
// million requests to memory against 4.5 million, 191 us against 177).
// 64- and 128-row tiles fit twice on a CU, so that one's fill and epilogue run beside the
// other's products; 64-row tiles have room for one stage more of both (173 us).
template <int kBits, int BM>
struct TileShape {
  static constexpr int BN = BM == 256 ? 256 : 128;
  static constexpr int kABytes = BM * 64, kA2Bytes = kBits == mx::kF6 ? BM * 32 : 0;
  static constexpr int kA2 = kABytes, kAScales = kA2 + kA2Bytes, kAStage = kAScales + BM * 4, kAStages = BM == 64 ? 4 : 3;
  static constexpr int kBStage = BN * 128, kBStages = BM == 64 ? 3 : 2;
  static constexpr int kB = kAStages * kAStage, kBScales = kB + kBStages * kBStage;
  static constexpr int kLds = kBScales + 2 * BN * 16;
};

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 4 bytes per lane straight into LDS (load_lds of gemm.h in dwords).
__device__ __forceinline__ void load_lds4(const u32x4& r, int off, unsigned lds_block) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds_block), "v"(off), "s"(r)
               : "m0");
}
#pragma clang diagnostic pop

// The product of rows row0 and n - 1 on with output columns n0 on.  kOnce: no other tile
// reads these weights, and their lines are the first that the caches give up.
template <int kBits, int EPI, int BM, bool kOnce>
__device__ __forceinline__ void tile_body(const MxGemm& g, char* lds, int e, int64_t row0, int n, int n0) {
  using S = TileShape<kBits, BM>;
  constexpr int BN = S::BN;
  constexpr int TM = BM / 2 / 32, TN = BN / 2 / 32;               // 32 x 32 tiles a wave, of 2 x 2 waves
  constexpr int NMAT = mats(EPI);
  constexpr int PA = S::kABytes / 4096, PB = S::kBStage / 4096;   // 16-byte loads a lane: a step of A, a stage of weights
  constexpr int PA2 = (S::kA2Bytes + 4095) / 4096;
  constexpr int LA = PA + PA2 + 1;                                // loads of a step of A, its scales with them
  constexpr int NSUB = BN / NMAT;                               // output columns a block
  const int K = g.K, KT = K / kStepK;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / 2, wn = wave % 2;
  const int b_bytes = K / 2, s_bytes = K / mx::kBlock;   // a weight row's codes and scales
  const int64_t wofs = static_cast<int64_t>(e) * g.N;
  const int64_t b_all = static_cast<int64_t>(g.N) * b_bytes, s_all = static_cast<int64_t>(g.N) * s_bytes;
  const u32x4 rb0 = dma_rsrc(g.B0 + wofs * b_bytes, b_all), rs0 = dma_rsrc(g.S0 + wofs * s_bytes, s_all);
  const u32x4 rb1 = NMAT == 2 ? dma_rsrc(g.B1 + wofs * b_bytes, b_all) : rb0;
  const u32x4 rs1 = NMAT == 2 ? dma_rsrc(g.S1 + wofs * s_bytes, s_all) : rs0;

  // Lane offsets of this wave's loads.  LDS rows hold a step in 16-byte chunks, chunk c at
  // c ^ swizzle(row): the loads write LDS in lane order, so the lane picks the chunk that
  // belongs there.  Rows past the tile's lie past A's descriptors, columns past N past the
  // weights'; they read as zero.
  const int ra_ = wave * 16 + lane / 4, offa = ra_ * 64 + ((lane % 4) ^ ((ra_ >> 2) & 3)) * 16;           // + 64 rows a load
  const int ra2_ = wave * 32 + lane / 2, offa2 = ra2_ * 32 + ((lane % 2) ^ ((ra2_ >> 3) & 1)) * 16;       // + 128 rows
  const int rsa_ = wave % (BM / 64) * 64 + lane;                                                          // (waves share rows)
  const int rb_ = wave * 8 + lane / 8, offb = (n0 + rb_) * b_bytes + ((lane % 8) ^ swz(rb_)) * 16;        // + 32 rows
  const int wsb = wave % (BN / 64);                                                                       // (and the scales')
  const int offsb = (n0 + (wsb * 64 + lane) % NSUB) * s_bytes;
  const int b_pass = 32 * b_bytes;
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) char*)lds));
  // Load q of step kt of A.  Past the last step the descriptors are empty: nothing is
  // read, and the count of loads in flight stays the same.
  auto issue_a = [&](int q, int kt, int stage) {
    const int64_t at = static_cast<int64_t>(kt) * g.M + row0;
    const int64_t rows = kt < KT ? n : 0;
    const unsigned base = lds0 + stage;
    if (q < PA) {
      load_lds(dma_rsrc(g.A + at * 64, rows * 64), offa + q * 4096, base + (q * 4 + wave) * 1024);
    } else if (q < PA + PA2 && (BM > 64 || wave < 2)) {
      const int p = q - PA;
      load_lds(dma_rsrc(g.A2 + at * 32, rows * 32), offa2 + p * 4096, base + S::kA2 + (p * 4 + wave) * 1024);
    } else {   // (also waves 2 and 3 of a 64-row tile in the second plane's place)
      load_lds4(dma_rsrc(g.As + at * 4, rows * 4), rsa_ * 4, base + S::kAScales + wave % (BM / 64) * 256);
    }
  };
  // Load p of stage ks of the weights; the scales of group kg (512 K values).
  auto issue_b = [&](int p, int ks, int stage) {
    const unsigned past = ks * 256 < K ? 0u : static_cast<unsigned>(kGatherOut);
    load_lds_hint<kOnce>(NMAT == 2 && p >= PB / 2 ? rb1 : rb0, offb + p % (PB / NMAT) * b_pass + ks * 128 + past,
             lds0 + stage + (p * 4 + wave) * 1024);
  };
  auto issue_scales = [&](int kg) {
    const unsigned past = kg * 512 < K ? 0u : static_cast<unsigned>(kGatherOut);
    load_lds(NMAT == 2 && wsb >= BN / 128 ? rs1 : rs0, offsb + kg * 16 + past, lds0 + S::kBScales + (kg & 1) * (BN * 16) + wsb * 1024);
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int u = 0; u < 16; ++u) acc[i][j][u] = 0.f;

  // the weight tiles of this wave: NMAT == 2: gate rows, then up rows 128 on
  const int half = lane >> 5, lr = lane & 31;
  auto b_row = [&](int j) { return NMAT == 2 ? (j < TN / 2 ? 0 : BN / 2) + wn * (TN / 2) * 32 + (j % (TN / 2)) * 32 : wn * TN * 32 + j * 32; };
  // Fragment read r of half step s: weight tile 0, the A tiles, the other weight tiles; a
  // step's scales come with its first half.  oa, ob: the stages' places in LDS; `odd`
  // says which half of the weights' stage.
  i32x4 fb[2][TN];
  Frag fa[2][TM];
  uint32_t sa[TM], sb[TN], next_sa[TM], next_sb[TN];
  const int a_row = wm * TM * 32 + lr;
  const int at_a = a_row * 64 + (half ^ ((lr >> 2) & 3)) * 16;                            // second half step: two chunks on
  const int at_a2 = S::kA2 + a_row * 32 + ((lr >> 3) & 1) * 16 + half * 8;                // (one on)
  const int at_b = lr * 128 + (half ^ swz(lr)) * 16;
  const int at_sa = S::kAScales + a_row * 4, at_sb = S::kBScales + lr * 16;
  constexpr int NR = TM + TN, NM = TM * TN;
  constexpr int kReads = (2 * NR + NM - 1) / NM;   // reads an instruction: all of them in the half's first half
  auto frag = [&](int r, int oa, int ob, int odd, int s, int os) {
    if (r >= 1 && r <= TM) {
      const int i = r - 1;
      fa[s][i].first = *reinterpret_cast<const i32x4*>(lds + ((at_a ^ (32 * s)) + oa) + i * 32 * 64);
      if constexpr (kBits == mx::kF6)
        fa[s][i].rest = *reinterpret_cast<const i32x2*>(lds + ((at_a2 ^ (16 * s)) + oa) + i * 32 * 32);
      if (s == 0) next_sa[i] = *reinterpret_cast<const uint32_t*>(lds + (at_sa + oa) + i * 128);
    } else {
      const int j = r == 0 ? 0 : r - TM;
      fb[s][j] = *reinterpret_cast<const i32x4*>(lds + ((at_b ^ (64 * odd + 32 * s)) + ob) + b_row(j) * 128);
      if (s == 0) next_sb[j] = *reinterpret_cast<const uint32_t*>(lds + (at_sb + os) + b_row(j) * 16);
    }
  };
  auto mma = [&](int m, int s) {
    const int i = m % TM, j = m / TM;
    acc[i][j] = s == 0 ? mma32<kBits, 0>(fb[s][j], fa[s][i], acc[i][j], sb[j], sa[i])
                       : mma32<kBits, 2>(fb[s][j], fa[s][i], acc[i][j], sb[j], sa[i]);
  };

  // A step's two halves run on registers that were read during the half before.  In the
  // middle of step kt the loads of step kt + 1 are awaited, those issued after them stay
  // in flight, and the waves meet: what step kt held in LDS has been read then and takes
  // the loads of step kt + kAStages, which are issued over this half and the next step's
  // first (in one half they filled the load queue and held the wave up).  The weights'
  // stage that an odd step ends is filled again over three halves.
  // The wait counts what follows the last load of A for kt + 1: A of the steps behind it,
  // and of the weights a whole stage where they have three, else those of two halves.
  // An odd count of steps is made even by one on zeros: no A is loaded for it and its
  // weights' scales are 2^-127.
  const int steps = (KT + 1) & ~1;
  int a_here = 0, a_free = (S::kAStages - 1) * S::kAStage, b_here = 0, b_free = (S::kBStages - 1) * S::kBStage;   // (free: the last step's)
  constexpr int kA1 = LA / 2, kA2 = LA - LA / 2, kB1 = (3 * PB + 7) / 8, kB2 = 3 * PB / 4;
  auto half_step = [&](int kt, auto odd_, auto second_) {
    constexpr int odd = decltype(odd_)::value, second = decltype(second_)::value;
    constexpr int kA = odd ? kA1 : kA2, kA_ = odd ? kA2 : kA1;     // of A issued in this step's second half, the last one's
    constexpr int from_a = second ? 0 : kA_, to_a = second ? kA : LA;
    constexpr int from_b = odd ? 0 : second ? kB2 : kB1, to_b = odd ? (second ? kB1 : 0) : second ? PB : kB2;
    constexpr int LS = second && !odd, LB = to_b - from_b, LT = LS + LB + to_a - from_a;
    const int a_next = a_here + S::kAStage == S::kB ? 0 : a_here + S::kAStage;
    const int b_next = !odd ? b_here : b_here + S::kBStage == S::kBStages * S::kBStage ? 0 : b_here + S::kBStage;
    const int os = (kt + 1) % 4 * 4 + (kt + 1) / 4 % 2 * (BN * 16);
    const int a_stage = second ? a_here : a_free, a_kt = second ? kt + S::kAStages : kt + S::kAStages - 1;
    const int b_stage = odd ? b_here : b_free, b_ks = (kt + odd) / 2 + S::kBStages - 1;
    int rd = 0, ld = 0;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      mma(m, second);
#pragma unroll
      for (; rd < NR && rd <= m * kReads; ++rd) {
        if constexpr (second) frag(rd, a_next, S::kB + b_next, odd ^ 1, 0, os);
        else frag(rd, a_here, S::kB + b_here, odd, 1, 0);
      }
#pragma unroll
      for (; ld < LT && ld * NM < (m + 1) * LT; ++ld) {
        if (ld < LB) {
          issue_b(from_b + ld, b_ks, S::kB + b_stage);
        } else if (LS && ld == LB) {
          if (kt % 4 == 0) issue_scales(kt / 4 + 1);
        } else {
          issue_a(from_a + ld - LB - LS, a_kt, a_stage);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (second) {
      a_free = a_here;
      a_here = a_next;
      if (odd) {
        b_free = b_here;
        b_here = b_next;
      }
    }
  };
  auto step = [&](int kt, auto odd_) {
    constexpr int odd = decltype(odd_)::value;
    const uint32_t live = kt < KT ? ~0u : 0u;
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = next_sa[i] >> (8 * half);   // this lane's two bytes lowest
#pragma unroll
    for (int j = 0; j < TN; ++j) sb[j] = (next_sb[j] & live) >> (8 * half);
    half_step(kt, odd_, std::integral_constant<int, 0>{});
    wait_vm<BM == 64 ? 2 * LA + PB : odd ? LA : LA + kB2>();
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    half_step(kt, odd_, std::integral_constant<int, 1>{});
  };
  issue_scales(0);
#pragma unroll
  for (int k = 0; k < S::kAStages - 1; ++k) {
#pragma unroll
    for (int q = 0; q < LA; ++q) issue_a(q, k, k * S::kAStage);
    if (k < S::kBStages - 1)
#pragma unroll
      for (int p = 0; p < PB; ++p) issue_b(p, k, S::kB + k * S::kBStage);
  }
#pragma unroll
  for (int p = 0; p < kB1; ++p) issue_b(p, S::kBStages - 1, S::kB + b_free);
#pragma unroll
  for (int q = 0; q < kA1; ++q) issue_a(q, S::kAStages - 1, a_free);
  wait_vm<(S::kAStages - 2) * LA + (S::kBStages - 2) * PB + kA1 + kB1>();
  __syncthreads();
#pragma unroll
  for (int r = 0; r < NR; ++r) frag(r, 0, S::kB, 0, 0, 0);
  for (int kt = 0; kt < steps; kt += 2) {
    step(kt, std::integral_constant<int, 0>{});
    step(kt + 1, std::integral_constant<int, 1>{});
  }
  wait_vm<0>();

  // ---- epilogue: lane (half, lr) holds row lr's columns 8 q + 4 half + i of each 32
  if constexpr (EPI == kMxSwiGLU || EPI == kMxGELU) {
    // Two blocks at a time: the halves trade, and lanes 0..31 hold the first block's 32
    // columns, lanes 32..63 the second's.
    constexpr int TC = TN / NMAT;
    auto value = [&](int b, int u) {
      const int i = b / TC, j = b % TC;
      if constexpr (NMAT == 2) return swiglu_h(acc[i][j][u], acc[i][j + TC][u]);
      else return fast_gelu(acc[i][j][u]);
    };
#pragma unroll
    for (int b = 0; b < TM * TC; b += 2) {   // (a wave's only block: both halves make it, one writes it)
      float v[32];
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(value(b, u)), __float_as_uint(value(min(b + 1, TM * TC - 1), u)), false, false);
        v[8 * (u / 4) + u % 4] = __uint_as_float(t[0]);
        v[8 * (u / 4) + 4 + u % 4] = __uint_as_float(t[1]);
      }
      const mx::Operand o = mx::encode_block<kBits>(v);
      const int mine = TM * TC == 1 ? 0 : b + half, i = mine / TC, j = mine % TC;
      const int r = (wm * TM + i) * 32 + lr, col = n0 + (wn * TC + j) * 32;
      if (r < n && col < g.N && (TM * TC > 1 || half == 0)) store_block<kBits>(o, row0 + r, g.M, col / mx::kBlock, static_cast<uint8_t*>(g.C), g.C2, g.Cs);
    }
  } else {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int r = (wm * TM + i) * 32 + lr, col = n0 + (wn * TN + j) * 32;
        if (col >= g.N) continue;   // (the same for the wave)
        constexpr int D = EPI == kMxBf16 ? 2 : 4;   // dwords of four columns
        uint32_t d[4][D];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int u = 0; u < D; ++u)
            d[q][u] = D == 2 ? mx::pack_bf16(acc[i][j][4 * q + 2 * u], acc[i][j][4 * q + 2 * u + 1])
                             : __float_as_uint(acc[i][j][4 * q + u]);
        uint32_t o[4 * D];   // the halves trade: sixteen adjacent columns each
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int u = 0; u < D; ++u) {
            const auto p = __builtin_amdgcn_permlane32_swap(d[q][u], d[q + 2][u], false, false);
            o[q * 2 * D + u] = p[0];
            o[q * 2 * D + D + u] = p[1];
          }
        if (r >= n) continue;
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint32_t*>(g.C) + (((row0 + r) * g.N + col + 16 * half) * D) / 4);
#pragma unroll
        for (int u = 0; u < D; ++u) out[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
      }
  }
}

// A 256-row tile fills a CU: where the last round of them would leave half the CUs or more
// idle, it is cut into quarters (of 128 rows by half the columns).  4 rounds and a quarter
// of down tiles (16384 rows of 8 experts, K = 14336, 6 bits) 625 us whole, 572 so.
constexpr int kCus = 256;

template <int kBits, int EPI, int BM, bool kBig>
__global__ __launch_bounds__(256, BM == 256 ? 1 : 2) void tile_kernel(const MxGemm g) {
  __shared__ __align__(1024) char lds[TileShape<kBits, BM>::kLds];
  constexpr int kCols = TileShape<kBits, BM>::BN / mats(EPI);
  const int total_m = *g.n_tiles, total = total_m * g.n_col_tiles, b = blockIdx.x;
  int rest = 0;
  if constexpr (BM == 256) rest = total % kCus <= kCus / 2 ? total % kCus : 0;
  const int whole = total - rest;
  if (b >= whole + 4 * rest) return;
  const int quarter = b < whole ? 0 : (b - whole) / rest;   // (a tile's on one XCD where rest is a multiple of 8)
  int mt, nt;
  tile_at(b < whole ? xcd_run(b, whole) : b - quarter * rest, total_m, g.n_col_tiles, &mt, &nt);
  const int4 tile = g.tiles[mt];
  const int e = __builtin_amdgcn_readfirstlane(tile.x);
  const int64_t row0 = __builtin_amdgcn_readfirstlane(tile.y);
  const int n = __builtin_amdgcn_readfirstlane(tile.z) - static_cast<int>(row0);
  if constexpr (BM == 256)
    if (b >= whole) {
      const int down = quarter / 2 * 128, right = quarter % 2 * (kCols / 2);
      if (down < n && nt * kCols + right < g.N)
        tile_body<kBits, EPI, 128, false>(g, lds, e, row0 + down, min(n - down, 128), nt * kCols + right);
      return;
    }
  // An expert with one row tile (its tiles follow one another in the list): 61 tokens of 160
  // experts 173 us without the hint, 160 with it; where other tiles read the same lines again
  // it costs (1021 tokens 473, with it for every tile 487, so 461), and also where all the
  // weights may wait in the last-level cache for the next call (2000 GELU tokens of 32 experts
  // of 1024 x 4096, 142 MB, over and over: 65 us without it, 75 with it).
  if constexpr (kBig) {
    const bool alone = (mt == 0 || g.tiles[mt - 1].x != e) && (mt + 1 == total_m || g.tiles[mt + 1].x != e);
    if (__builtin_amdgcn_readfirstlane(alone)) return tile_body<kBits, EPI, BM, true>(g, lds, e, row0, n, nt * kCols);
  }
  tile_body<kBits, EPI, BM, false>(g, lds, e, row0, n, nt * kCols);
}

// ---- few rows an expert ------------------------------------------------------------
// At most 16 rows by four 16-row weight tiles (two of the gate and two of the up
// weights, or 64 columns of y).  Wave w takes the w-th part of K, through a ring of its
// own in LDS, and the parts are added in wave order.  Why LDS, where nothing is shared:
// a load instruction takes the address path one cycle for every line that a quarter
// wave touches, and an operand's quarter is 16 weight rows; loaded in runs of 64 bytes
// a row it is four (measured: 64 against 16 cycles for 1 KB), and the operands' own
// loads came to 4.2 TB/s.
template <int kBits, int NT>
struct StreamShape {   // a wave's LDS: stages of one K step, two buffers of four steps' weight scales
  static constexpr int kRing = NT == 2 ? 4 : 3;
  static constexpr int kA = NT * 1024, kA2 = kA + 1024, kAScales = kA2 + (kBits == mx::kF6 ? 512 : 0);
  static constexpr int kStage = kAScales + 64;
  static constexpr int kBScales = kRing * kStage, kWave = kBScales + 2 * NT * 256;
};

template <int kBits, int EPI, int NT, int kStreamWaves>
__global__ __launch_bounds__(64 * kStreamWaves, 2) void stream_kernel(const MxGemm g) {
  using S = StreamShape<kBits, NT>;
  constexpr int NMAT = mats(EPI), NC = NT / NMAT, kCols = 16 * NC, R = S::kRing;
  constexpr int L = NT + 2 + (kBits == mx::kF6 ? 1 : 0);   // a step's loads (without the weights' scales)
  __shared__ __align__(1024) char lds[kStreamWaves * S::kWave];
  const int mt = blockIdx.x / g.n_col_tiles, nt = blockIdx.x - mt * g.n_col_tiles;
  const int4 tile = g.tiles[mt];   // (the list has room for every block of the grid)
  if (mt >= *g.n_tiles) return;
  const int e = __builtin_amdgcn_readfirstlane(tile.x);
  const int64_t row0 = __builtin_amdgcn_readfirstlane(tile.y);
  const int n = __builtin_amdgcn_readfirstlane(tile.z) - static_cast<int>(row0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, grp = lane >> 4;
  const int K = g.K, KT = K / kStepK, n0 = nt * kCols;
  const int b_bytes = K / 2, s_bytes = K / mx::kBlock;
  const int64_t wofs = static_cast<int64_t>(e) * g.N;
  const int64_t b_all = static_cast<int64_t>(g.N) * b_bytes, s_all = static_cast<int64_t>(g.N) * s_bytes;
  const u32x4 rb0 = dma_rsrc(g.B0 + wofs * b_bytes, b_all), rs0 = dma_rsrc(g.S0 + wofs * s_bytes, s_all);
  const u32x4 rb1 = NMAT == 2 ? dma_rsrc(g.B1 + wofs * b_bytes, b_all) : rb0;
  const u32x4 rs1 = NMAT == 2 ? dma_rsrc(g.S1 + wofs * s_bytes, s_all) : rs0;
  char* const mine = lds + wave * S::kWave;
  const unsigned at0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) char*)lds)) + wave * S::kWave;
  // a load's 16 rows of 64 bytes; chunk c of a row at c ^ swizzle(row)
  const int r4 = lane / 4, run = r4 * 64 + ((lane % 4) ^ ((r4 >> 2) & 3)) * 16;
  const int offb = (n0 + r4) * b_bytes + (run - r4 * 64), b_tile = 16 * b_bytes;
  const int offsb = (n0 + lane % kCols) * s_bytes;
  const int begin = KT * wave / kStreamWaves, end = KT * (wave + 1) / kStreamWaves;
  auto issue = [&](int kt) {   // past the end every offset lies past its descriptor's end
    const unsigned base = at0 + (kt - begin) % R * S::kStage;
    const unsigned past = kt < end ? 0u : static_cast<unsigned>(kGatherOut);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      load_lds(NMAT == 2 && j >= NC ? rb1 : rb0, offb + j % NC * b_tile + kt * 64 + past, base + j * 1024);
    const int64_t at = static_cast<int64_t>(kt) * g.M + row0;
    const int64_t rows = kt < end ? n : 0;
    load_lds(dma_rsrc(g.A + at * 64, rows * 64), run, base + S::kA);
    if (kBits == mx::kF6 && lane < 32) load_lds(dma_rsrc(g.A2 + at * 32, rows * 32), lane * 16, base + S::kA2);
    if (lane < 16) load_lds4(dma_rsrc(g.As + at * 4, rows * 4), lane * 4, base + S::kAScales);
  };
  auto issue_scales = [&](int kg) {   // steps begin + 4 kg and three on
    const int off = offsb + (begin + 4 * kg) * 4;
    const unsigned to = at0 + S::kBScales + (kg & 1) * (NT * 256);
    if (lane < kCols) load_lds(rs0, off, to);
    if (NMAT == 2 && lane >= kCols) load_lds(rs1, off, to);
  };
  f32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  issue_scales(0);
#pragma unroll
  for (int u = 0; u < R; ++u) issue(begin + u);
  for (int kt = begin; kt < end; ++kt) {
    const int k = kt - begin;
    wait_vm<(R - 1) * L>();
    asm volatile("" ::: "memory");
    const char* const at = mine + k % R * S::kStage;
    const int chunk = (grp ^ ((lr >> 2) & 3)) * 16;
    i32x4 w[NT];
    uint32_t sw[NT];
    Frag a{};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      w[j] = *reinterpret_cast<const i32x4*>(at + (16 * j + lr) * 64 + chunk);
      sw[j] = *reinterpret_cast<const uint32_t*>(mine + S::kBScales + (k / 4 & 1) * (NT * 256) + (16 * j + lr) * 16 + k % 4 * 4);
    }
    a.first = *reinterpret_cast<const i32x4*>(at + S::kA + lr * 64 + chunk);
    if constexpr (kBits == mx::kF6) a.rest = *reinterpret_cast<const i32x2*>(at + S::kA2 + lr * 32 + grp * 8);
    const uint32_t sa = *reinterpret_cast<const uint32_t*>(at + S::kAScales + lr * 4);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the stage is read: its next loads may land
    if (k % 4 == 0 && kt + 4 < end) issue_scales(k / 4 + 1);
    issue(kt + R);
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = mma16<kBits>(w[j], a, acc[j], sw[j] >> (8 * grp), sa >> (8 * grp));
  }
  wait_vm<0>();
  asm volatile("" ::: "memory");
  f32x4(*const part)[64] = reinterpret_cast<f32x4(*)[64]>(mine);
  if (wave > 0)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[j][lane] = acc[j];
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int u = 1; u < kStreamWaves; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] += reinterpret_cast<const f32x4(*)[64]>(lds + u * S::kWave)[j][lane];
  }
  // wave 0's lane (grp, lr) holds row lr's columns 16 j + 4 grp + i
  if constexpr (EPI == kMxSwiGLU || EPI == kMxGELU) {
    float(*const h)[kCols + 1] = reinterpret_cast<float(*)[kCols + 1]>(lds);   // a row's block goes to one lane
    if (wave == 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float v;
          if constexpr (NMAT == 2) v = swiglu_h(acc[c][u], acc[NC + c][u]);
          else v = fast_gelu(acc[c][u]);
          h[lr][16 * c + 4 * grp + u] = v;
        }
    }
    __syncthreads();
    const int r = threadIdx.x % kStreamRows, c = threadIdx.x / kStreamRows;
    if (r >= n || c >= kCols / mx::kBlock) return;
    float v[32];
#pragma unroll
    for (int u = 0; u < 32; ++u) v[u] = h[r][32 * c + u];
    store_block<kBits>(mx::encode_block<kBits>(v), row0 + r, g.M, n0 / mx::kBlock + c, static_cast<uint8_t*>(g.C), g.C2, g.Cs);
  } else {
    if (wave > 0 || lr >= n) return;
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      const float v[4] = {acc[c][0], acc[c][1], acc[c][2], acc[c][3]};
      const int64_t at = (row0 + lr) * g.N + n0 + 16 * c + 4 * grp;
      if constexpr (EPI == kMxBf16) store4(static_cast<uint16_t*>(g.C) + at, v);
      else store4(static_cast<float*>(g.C) + at, v);
    }
  }
}

// ------------------------------------------------------------------------ the call
struct MxLayout {
  size_t xq, xq2, xs, hq, hq2, hs, tiles, n_tiles, bytes;
  int cap;
};

// Rows of a tile, from the rows and the rows an expert has on average, fitted to
// sweeps over 160 experts of 5120 x 1536, 64 of 2048 x 1408, 16 of 6144 x 10752, 8 of
// 4096 x 14336 and 32 of 1024 x 4096 (GELU), us a call in 6 bits:
//   up to 24 rows the stream, which splits K: one token of two experts at H = 4096 39
//     against 62 in 64-row tiles, 18 rows at H = 5120 41 against 46; but 36 rows 55
//     against 52, 64 rows at H = 4096 176 against 145.
//   64-row tiles up to 64 rows an expert: 38 at H = 5120 496 against 511 in 128-row tiles;
//     76 there 691 against 654, 64 at H = 6144 470 against 454, at H = 4096 220 against 234.
//   256-row tiles where rows and K make up for one block a CU, from 2^19 rows * H an expert
//     on: 131 rows at H = 5120 794 against 827 in 128-row tiles, 256 at H = 4096 349 against
//     407; 76 at H = 5120 677 against 654, 250 at H = 1024 122 against 117.
int rows_per_tile(int64_t M, int E, int H) {
  const int64_t avg = M / E;
  if (M <= 24) return kStreamRows;
  if (avg <= 64) return 64;
  return avg * H < (int64_t(1) << 19) ? 128 : 256;
}

// Whatever E a call gives, the list has room for the smallest tiles.
MxLayout mx_layout(int64_t M, int H, int I, int max_slots, moe_mx_format fmt) {
  MxLayout w{};
  size_t at = 0;
  auto take = [&](size_t n) { size_t p = at; at = moe::align_up(at + n, 256); return p; };
  const size_t x_values = static_cast<size_t>(M) * H, h_values = static_cast<size_t>(M) * I;
  w.xq = take(x_values / 2);
  w.xq2 = take(fmt == MOE_MX_FP6 ? x_values / 4 : 0);
  w.xs = take(x_values / mx::kBlock);
  w.hq = take(h_values / 2);
  w.hq2 = take(fmt == MOE_MX_FP6 ? h_values / 4 : 0);
  w.hs = take(h_values / mx::kBlock);
  w.cap = static_cast<int>(std::min<int64_t>(M / kStreamRows + std::min<int64_t>(M, max_slots), 0x3fffffff));
  w.tiles = take(sizeof(int4) * w.cap);
  w.n_tiles = take(sizeof(int32_t));
  w.bytes = at;
  return w;
}

// Few rows.  Narrow blocks (32 columns instead of 64) where the wide ones come to fewer
// than 7 for every 4 CUs.  Whole calls, narrow against wide, by wide blocks of the down
// product: K = 1536 128 blocks 15.8 us against 16.4, 256 equal, 400 23.0 against 22.1, 512 25.2
// against 24.2; K = 14336 64 blocks 32.6 against 41.4, 128 48.8 against 57.1, 256 equal, 384
// 113.1 against 122.2, 448 134.4 against 135.4.  (A long K wins where the blocks are few or
// just past one a CU, a short one loses up to 1 us there.)  Eight waves a block where each CU
// has one block at most.
template <int kBits, int EPI>
int launch_stream(MxGemm p, int64_t row_tiles, hipStream_t s, const char* what) {
  constexpr int kWide = 64 / mats(EPI);
  constexpr bool kCanNarrow = EPI == kMxBf16 || EPI == kMxF32 || EPI == kMxGELU;
  const bool narrow = kCanNarrow && row_tiles * ceil_div(p.N, kWide) < 448;
  const int cols = narrow ? kWide / 2 : kWide;
  p.n_col_tiles = p.N / cols;
  const int64_t blocks = row_tiles * p.n_col_tiles;
  const unsigned grid = static_cast<unsigned>(blocks);
  const bool deep = blocks <= 256 && p.K / kStepK >= 16;
  if constexpr (kCanNarrow) {
    if (narrow) {
      if (deep) stream_kernel<kBits, EPI, 2, 8><<<grid, 512, 0, s>>>(p);
      else stream_kernel<kBits, EPI, 2, 4><<<grid, 256, 0, s>>>(p);
      return moe::hip_status(hipGetLastError(), what);
    }
  }
  if (deep) stream_kernel<kBits, EPI, 4, 8><<<grid, 512, 0, s>>>(p);
  else stream_kernel<kBits, EPI, 4, 4><<<grid, 256, 0, s>>>(p);
  return moe::hip_status(hipGetLastError(), what);
}

// Blocks of a tile_kernel launch (64 rows and up), the last round's quarters among them.
int tile_cols(int bm, int N, int n_mat) { return static_cast<int>(ceil_div(N, (bm == 256 ? 256 : 128) / n_mat)); }
int64_t tile_blocks(int bm, int64_t row_tiles, int n_col_tiles) {
  return row_tiles * n_col_tiles + (bm == 256 ? 3 * (kCus / 2) : 0);
}

template <int kBits, int EPI>
int launch_product(MxGemm p, int bm, int64_t row_tiles, hipStream_t s, const char* what) {
  if (bm == kStreamRows) return launch_stream<kBits, EPI>(p, row_tiles, s, what);
  p.n_col_tiles = tile_cols(bm, p.N, mats(EPI));
  const unsigned grid = static_cast<unsigned>(tile_blocks(bm, row_tiles, p.n_col_tiles));
  if (bm == 64 && p.big) tile_kernel<kBits, EPI, 64, true><<<grid, 256, 0, s>>>(p);
  else if (bm == 64) tile_kernel<kBits, EPI, 64, false><<<grid, 256, 0, s>>>(p);
  else if (bm == 128 && p.big) tile_kernel<kBits, EPI, 128, true><<<grid, 256, 0, s>>>(p);
  else if (bm == 128) tile_kernel<kBits, EPI, 128, false><<<grid, 256, 0, s>>>(p);
  else tile_kernel<kBits, EPI, 256, false><<<grid, 256, 0, s>>>(p);
  return moe::hip_status(hipGetLastError(), what);
}

template <int kBits>
int run(MxGemm up, MxGemm down, bool swiglu, bool bf16, int bm, int64_t row_tiles, hipStream_t s) {
  if (int rc = swiglu ? launch_product<kBits, kMxSwiGLU>(up, bm, row_tiles, s, "moe_mx_expert_ffn gate/up launch")
                      : launch_product<kBits, kMxGELU>(up, bm, row_tiles, s, "moe_mx_expert_ffn up launch"))
    return rc;
  return bf16 ? launch_product<kBits, kMxBf16>(down, bm, row_tiles, s, "moe_mx_expert_ffn down launch")
              : launch_product<kBits, kMxF32>(down, bm, row_tiles, s, "moe_mx_expert_ffn down launch");
}

}  // namespace

extern "C" size_t moe_mx_expert_ffn_workspace_bytes(int64_t M, int H, int I, int max_slots, moe_mx_format x_format) {
  if (M < 0 || H < 1 || I < 1 || max_slots < 1 || (x_format != MOE_MX_FP4 && x_format != MOE_MX_FP6)) return 0;
  return mx_layout(M, H, I, max_slots, x_format).bytes;
}

extern "C" int moe_mx_expert_ffn(const void* x, const int32_t* row_src, int64_t n_src, moe_dtype dt, int64_t M, int H,
                                 int I, int E, const int32_t* slot_off, const int32_t* slot_expert,
                                 const int32_t* n_slots, int max_slots, const uint8_t* w_gate, const uint8_t* s_gate,
                                 const uint8_t* w_up, const uint8_t* s_up, const uint8_t* w_down, const uint8_t* s_down,
                                 moe_act act, moe_mx_format x_format, void* y_perm, void* workspace,
                                 size_t workspace_bytes, int32_t* check, void* stream) {
  using namespace moe;
  const char* who = "moe_mx_expert_ffn";
  if (dt != MOE_F32 && dt != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dt);
  if (act != MOE_SWIGLU && act != MOE_GELU) return fail(MOE_ERR_INVALID_ARG, "%s: unknown activation", who);
  if (x_format != MOE_MX_FP4 && x_format != MOE_MX_FP6)
    return fail(MOE_ERR_INVALID_ARG, "%s: x_format must be MOE_MX_FP6 or MOE_MX_FP4, not %d", who, (int)x_format);
  if (M < 0 || M >= (int64_t(1) << 31)) return fail(MOE_ERR_INVALID_ARG, "%s: M out of range", who);
  if (!row_src) n_src = M;
  if (n_src < 0) return fail(MOE_ERR_INVALID_ARG, "%s: negative n_src", who);
  if (H < 128 || I < 128 || H % 128 || I % 128)
    return fail(MOE_ERR_UNSUPPORTED, "%s: H and I must be positive multiples of 128 (H=%d I=%d)", who, H, I);
  // 31-bit offsets into an expert's codes; a launch's K steps and lanes
  if (static_cast<int64_t>(H) * I / 2 >= kGatherLimit || H > (1 << 22) || I > (1 << 22))
    return fail(MOE_ERR_UNSUPPORTED, "%s: H or I too large for 32-bit offsets", who);
  if (M >= (int64_t(1) << 36) / std::max(H, I)) return fail(MOE_ERR_UNSUPPORTED, "%s: more than 2^36 values of x or h", who);
  if (E < 1 || max_slots < E) return fail(MOE_ERR_INVALID_ARG, "%s: need 1 <= E <= max_slots", who);
  if (act == MOE_SWIGLU && (!w_up || !s_up)) return fail(MOE_ERR_INVALID_ARG, "%s: SwiGLU needs w_up", who);
  if (act == MOE_GELU && (w_up || s_up)) return fail(MOE_ERR_INVALID_ARG, "%s: GELU takes no w_up (pass NULL)", who);
  if (!slot_off || !slot_expert || !n_slots || !w_gate || !s_gate || !w_down || !s_down || !workspace)
    return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  if (M > 0 && (!y_perm || (n_src > 0 && !x))) return fail(MOE_ERR_INVALID_ARG, "%s: null pointer", who);
  for (const void* p : {x, static_cast<const void*>(w_gate), static_cast<const void*>(w_up), static_cast<const void*>(w_down),
                        static_cast<const void*>(s_gate), static_cast<const void*>(s_up), static_cast<const void*>(s_down),
                        static_cast<const void*>(y_perm), static_cast<const void*>(workspace)})
    if (p && !aligned16(p)) return fail(MOE_ERR_INVALID_ARG, "%s: operands must be 16-byte aligned", who);
  const MxLayout w = mx_layout(M, H, I, max_slots, x_format);
  if (workspace_bytes < w.bytes)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", who, workspace_bytes, w.bytes);
  if (M == 0) return MOE_OK;
  const hipStream_t s = as_stream(stream);
  char* ws = static_cast<char*>(workspace);
  auto at = [&](size_t offset) { return reinterpret_cast<uint8_t*>(ws + offset); };
  int4* const tiles = reinterpret_cast<int4*>(ws + w.tiles);
  int32_t* const n_tiles = reinterpret_cast<int32_t*>(ws + w.n_tiles);
  const int bm = rows_per_tile(M, E, H);
  const int64_t row_tiles = M / bm + std::min<int64_t>(M, max_slots);
  if (bm != kStreamRows) {
    const int64_t most = std::max(tile_blocks(bm, row_tiles, tile_cols(bm, I, act == MOE_SWIGLU ? 2 : 1)),
                                  tile_blocks(bm, row_tiles, tile_cols(bm, H, 1)));
    if (most >= (int64_t(1) << 24)) return fail(MOE_ERR_UNSUPPORTED, "%s: %lld tiles in one launch", who, (long long)most);
  }
  const dim3 grid(static_cast<unsigned>(ceil_div(M * 4, 256) + 1), H / kStepK);
  auto prepare = [&](auto kernel) {
    kernel<<<grid, 256, 0, s>>>(x, row_src, n_src, H, at(w.xq), at(w.xq2), at(w.xs), slot_off, slot_expert, n_slots,
                                max_slots, M, E, bm, w.cap, tiles, n_tiles, check);
  };
  const bool bf16 = dt == MOE_BF16, fp6 = x_format == MOE_MX_FP6;
  if (bf16) prepare(fp6 ? prepare_kernel<true, mx::kF6> : prepare_kernel<true, mx::kF4>);
  else prepare(fp6 ? prepare_kernel<false, mx::kF6> : prepare_kernel<false, mx::kF4>);
  if (int rc = hip_status(hipGetLastError(), "moe_mx_expert_ffn prepare launch")) return rc;
  MxGemm up{};
  up.big = static_cast<int64_t>(E) * H * I * (act == MOE_SWIGLU ? 3 : 2) * 17 / 32 > (int64_t(1) << 29);   // (twice its 256 MB)
  up.A = at(w.xq);
  up.A2 = at(w.xq2);
  up.As = at(w.xs);
  up.B0 = w_gate;
  up.B1 = w_up;
  up.S0 = s_gate;
  up.S1 = s_up;
  up.K = H;
  up.N = I;
  up.M = M;
  up.tiles = tiles;
  up.n_tiles = n_tiles;
  up.C = at(w.hq);
  up.C2 = at(w.hq2);
  up.Cs = at(w.hs);
  MxGemm down = up;
  down.A = at(w.hq);
  down.A2 = at(w.hq2);
  down.As = at(w.hs);
  down.B0 = w_down;
  down.S0 = s_down;
  down.B1 = down.S1 = nullptr;
  down.K = I;
  down.N = H;
  down.C = y_perm;
  down.C2 = down.Cs = nullptr;
  return fp6 ? run<mx::kF6>(up, down, act == MOE_SWIGLU, bf16, bm, row_tiles, s)
             : run<mx::kF4>(up, down, act == MOE_SWIGLU, bf16, bm, row_tiles, s);
}
