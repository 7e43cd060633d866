// moe_mx_expert_ffn: the experts' FFNs on weights in microscaled 4-bit blocks,
// activations quantised by row blocks to 6 or 4 bits, on gfx950's scaled matrix
// instructions (v_mfma_scale_f32_*_f8f6f4: the operands' codes go in as they are
// kept, each block of 32 along K with its scale byte, fp32 accumulation).
//
// Q(x) the rows' quantised values:  h = act(Q(x) Wg^T, Q(x) Wu^T), y = Q(h) Wd^T.
// Three launches:
//   prepare:  the rows of x quantised, one block a lane, and in block 0 the list of
//             row tiles from the slot table;
//   gate/up:  per tile and 128 (or 32) columns of h, gate and up side by side; the
//             epilogue trades accumulators between lanes until each holds 32
//             adjacent columns of a row, quantises them in registers and writes
//             their codes;
//   down:     y = Q(h) Wd^T.
// Two kernels multiply.  tile_kernel: BM rows x 256 weight rows a block, operands
// straight into LDS, 32x32x64 instructions.  stream_kernel: at most 16 rows by 32
// columns a block, the weights from memory to registers, K split over the block's
// waves: for few rows an expert the time is the weights' bytes.
//
// Why 6 bits and not 8.  Lane group g (lane / rows) of an operand holds K = 32 g ..
// 32 g + 31 and their scale.  The instruction sums eight products at a time, each
// cut at 2^-13 of the largest's leading bit (found by probing): of e2m1 by e2m1 or
// e2m3, whose products are multiples of 2^-4 up to 45, that cuts nothing, and the
// sums of eight are added in fp32; of e2m1 by e4m3 it cuts products at some 2^-13
// of the largest beside them.  e2m3 has e4m3's four significant bits and runs at
// the 4-bit rate.
//
// Activations in the workspace.  A row's codes lie in two planes: 16 bytes a block
// (all of e2m1, the first two thirds of e2m3), then e2m3's last 8 bytes a block, so
// that either is loaded in 16-byte pieces.  Their scales are K-major: one dword of
// four bytes, a K step of 128, for every row in a run.
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
constexpr int kStreamRows = 16, kStreamCols = 32;

// One product: rows of A (codes [a_n, K / 2] and for e2m3 [a_n, K / 4], scales
// K-major [K / 128][a_n] dwords), through a_rows or in place, times the experts'
// weights (codes [E, N, K / 2], scales [E, N, K / 32]); B1/S1 the up weights beside
// the gate's.
struct MxGemm {
  const uint8_t *A, *A2, *As;
  const int32_t* a_rows;
  int64_t a_n;
  const uint8_t *B0, *B1, *S0, *S1;
  int K, N;
  int64_t M;
  const int4* tiles;   // expert, first row, end row
  const int32_t* n_tiles;
  int n_col_tiles;
  void* C;             // y [M, N], or h's codes
  uint8_t *C2, *Cs;    // h's second plane and scales
};

// A block's codes and scale to their places: row `row` of n, columns from `col`.
template <int kBits>
__device__ __forceinline__ void store_block(const mx::Operand& o, int64_t row, int64_t n, int K, int col, uint8_t* q,
                                            uint8_t* q2, uint8_t* scale) {
  *reinterpret_cast<uint4*>(q + (row * K + col) / 2) = o.first;
  if constexpr (kBits == mx::kF6) *reinterpret_cast<uint2*>(q2 + (row * K + col) / 4) = o.rest;
  scale[(col / kStepK * n + row) * 4 + (col / mx::kBlock) % 4] = static_cast<uint8_t>(o.byte);
}

// ------------------------------------------------------------------- preparation
// Block 0 lists the row tiles; the others quantise x.
template <bool kBf16, int kBits>
__global__ __launch_bounds__(256) void prepare_kernel(const void* __restrict__ x, int64_t R, int K,
                                                      uint8_t* __restrict__ q, uint8_t* __restrict__ q2,
                                                      uint8_t* __restrict__ scale,
                                                      const int32_t* __restrict__ slot_off,
                                                      const int32_t* __restrict__ slot_expert,
                                                      const int32_t* __restrict__ n_slots, int max_slots, int64_t M,
                                                      int E, int rows_per_tile, int cap, int4* __restrict__ tiles,
                                                      int32_t* __restrict__ n_tiles, int32_t* __restrict__ check) {
  if (blockIdx.x == 0) {
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
  const int64_t b = static_cast<int64_t>(blockIdx.x - 1) * 256 + threadIdx.x, per_row = K / mx::kBlock;
  bool bad = false;
  if (b < R * per_row) {
    const int64_t row = b / per_row;
    const int col = static_cast<int>(b - row * per_row) * mx::kBlock;
    float v[32];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float part[8];
      rows::unpack8<kBf16>(rows::load8<kBf16>(x, row * K + col + 8 * u), part);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * u + i] = part[i];
    }
    const mx::Operand o = mx::encode_block<kBits>(v);
    bad = o.byte == 255;
    store_block<kBits>(o, row, R, K, col, q, q2, scale);
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

// The block's place: XCD-contiguous runs of tiles, eight row tiles by the columns
// (gemm.h).  False past the last tile.
__device__ __forceinline__ bool place(int total_m, int n_col_tiles, int b, int* mt, int* nt) {
  const int total = total_m * n_col_tiles;
  if (b >= total) return false;
  const int xcd = b & 7, q = total >> 3, rem = total & 7;
  const int l = xcd * q + min(xcd, rem) + (b >> 3);
  const int grp = l / (kGroupM * n_col_tiles);
  const int gsz = min(kGroupM, total_m - grp * kGroupM);
  const int li = l - grp * kGroupM * n_col_tiles;
  *mt = grp * kGroupM + li % gsz;
  *nt = li / gsz;
  return true;
}

// What the epilogue makes of the accumulators.
enum MxEpi { kMxSwiGLU = 0, kMxGELU = 1, kMxBf16 = 2, kMxF32 = 3 };
constexpr int mats(int epi) { return epi == kMxSwiGLU ? 2 : 1; }

// ---- large batches ---------------------------------------------------------------
template <int kBits, int BM>
struct TileShape {
  static constexpr int kABytes = BM * 64;                  // a step's rows of A, first plane
  static constexpr int kA2Bytes = kBits == mx::kF6 ? (BM < 128 ? 128 : BM) * 32 : 0;
  static constexpr int kBBytes = 256 * 64;
  static constexpr int kA2 = kABytes, kB = kA2 + kA2Bytes, kScales = kB + kBBytes;
  static constexpr int kStage = kScales + 512 * 4;         // 256 weight rows' and up to 256 rows' dwords
  static constexpr int kStages = BM == 64 || (kBits == mx::kF6 && BM == 256) ? 3 : 4;
  static constexpr int kLds = kStages * kStage;
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

template <int kBits, int EPI, int BM>
__global__ __launch_bounds__(256, BM == 64 ? 2 : 1) void tile_kernel(const MxGemm g) {
  using S = TileShape<kBits, BM>;
  constexpr int WM = BM == 256 ? 2 : 1, WN = 4 / WM;      // the waves' grid
  constexpr int TM = BM / WM / 32, TN = 256 / WN / 32;    // 32 x 32 tiles a wave
  constexpr int NMAT = mats(EPI);
  constexpr int PA = S::kABytes / 4096, PA2 = S::kA2Bytes / 4096, PB = S::kBBytes / 4096;   // 16-byte loads a lane and step
  constexpr int L = PA + PA2 + PB + 2;                                                      // and all loads
  constexpr int NSUB = 256 / NMAT;                                // output columns a block
  constexpr int ST = S::kStages;
  __shared__ __align__(1024) char lds[S::kLds];
  int mt, nt;
  if (!place(*g.n_tiles, g.n_col_tiles, blockIdx.x, &mt, &nt)) return;
  const int4 tile = g.tiles[mt];
  const int e = __builtin_amdgcn_readfirstlane(tile.x);
  const int64_t row0 = __builtin_amdgcn_readfirstlane(tile.y);
  const int n = __builtin_amdgcn_readfirstlane(tile.z) - static_cast<int>(row0);
  const int n0 = nt * NSUB;
  const int K = g.K, KT = K / kStepK;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int b_bytes = K / 2, a2_bytes = K / 4, s_bytes = K / mx::kBlock;   // a row's codes (A's as the weights') and scales

  // sources: A by the row map, or the tile's own rows; one expert's weights
  const int64_t first = g.a_rows ? 0 : row0, span = g.a_rows ? g.a_n : n;
  const u32x4 ra = dma_rsrc(g.A + first * b_bytes, span * b_bytes);
  const u32x4 ra2 = kBits == mx::kF6 ? dma_rsrc(g.A2 + first * a2_bytes, span * a2_bytes) : ra;
  const u32x4 rsa = dma_rsrc(g.As, g.a_n * 4 * KT);
  const int64_t wofs = static_cast<int64_t>(e) * g.N;
  const int64_t b_all = static_cast<int64_t>(g.N) * b_bytes, s_all = static_cast<int64_t>(g.N) * s_bytes;
  const u32x4 rb0 = dma_rsrc(g.B0 + wofs * b_bytes, b_all), rs0 = dma_rsrc(g.S0 + wofs * s_bytes, s_all);
  const u32x4 rb1 = NMAT == 2 ? dma_rsrc(g.B1 + wofs * b_bytes, b_all) : rb0;
  const u32x4 rs1 = NMAT == 2 ? dma_rsrc(g.S1 + wofs * s_bytes, s_all) : rs0;

  // Lane offsets of this wave's loads.  LDS rows hold a step (64 bytes of the first
  // plane and of the weights, 32 of the second) in 16-byte chunks, chunk c at c ^
  // swizzle(row): the loads write LDS in lane order, so the lane picks the chunk
  // that belongs there.  Rows past the tile's and rows mapped outside x get an
  // offset past the descriptor's end and read as zero.
  auto source = [&](int r) -> int {
    if (r >= n) return -1;
    if (!g.a_rows) return r;
    const int src = g.a_rows[row0 + r];
    return src < g.a_n ? src : -1;
  };
  int offa[PA], offa2[PA2 ? PA2 : 1], offb[PB], offsa, offsb;
#pragma unroll
  for (int p = 0; p < PA; ++p) {
    const int idx = (p * 4 + wave) * 64 + lane, r = idx / 4, src = source(r);
    offa[p] = src >= 0 ? src * b_bytes + ((idx % 4) ^ ((r >> 2) & 3)) * 16 : kGatherOut;
  }
#pragma unroll
  for (int p = 0; p < PA2; ++p) {
    const int idx = (p * 4 + wave) * 64 + lane, r = idx / 2, src = source(r);
    offa2[p] = src >= 0 ? src * a2_bytes + ((idx % 2) ^ ((r >> 3) & 1)) * 16 : kGatherOut;
  }
  {
    const int r = wave * 64 + lane, src = r < BM ? source(r) : -1;
    offsa = src >= 0 ? static_cast<int>(first + src) * 4 : kGatherOut;
  }
#pragma unroll
  for (int p = 0; p < PB; ++p) {
    const int idx = (p * 4 + wave) * 64 + lane, r = idx / 4;
    const int c = (idx % 4) ^ ((r >> 2) & 3);
    offb[p] = (n0 + (NMAT == 2 ? r % 128 : r)) * b_bytes + c * 16;
  }
  {
    const int r = wave * 64 + lane;
    offsb = (n0 + (NMAT == 2 ? r % 128 : r)) * s_bytes;
  }
  const unsigned lds0 = static_cast<unsigned>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) char*)lds));
  const int a_step = static_cast<int>(g.a_n) * 4;
  auto issue = [&](int kt, int stage) {
    const unsigned base = lds0 + stage * S::kStage;
#pragma unroll
    for (int p = 0; p < PA; ++p) load_lds(ra, offa[p] + kt * 64, base + (p * 4 + wave) * 1024);
#pragma unroll
    for (int p = 0; p < PA2; ++p) load_lds(ra2, offa2[p] + kt * 32, base + S::kA2 + (p * 4 + wave) * 1024);
#pragma unroll
    for (int p = 0; p < PB; ++p)
      load_lds(NMAT == 2 && p >= PB / 2 ? rb1 : rb0, offb[p] + kt * 64, base + S::kB + (p * 4 + wave) * 1024);
    load_lds4(NMAT == 2 && wave >= 2 ? rs1 : rs0, offsb + kt * 4, base + S::kScales + wave * 256);
    load_lds4(rsa, offsa == kGatherOut ? kGatherOut : offsa + kt * a_step, base + S::kScales + 1024 + wave * 256);
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
  auto b_row = [&](int j) { return NMAT == 2 ? (j < TN / 2 ? 0 : 128) + wn * (TN / 2) * 32 + (j % (TN / 2)) * 32 : wn * TN * 32 + j * 32; };
  auto compute = [&](int stage) {
    const char* base = lds + stage * S::kStage;
    const char* a = base + (wm * TM * 32 + lr) * 64;
    const char* a2 = base + S::kA2 + (wm * TM * 32 + lr) * 32 + half * 8;
    const char* b = base + S::kB + lr * 64;
    const uint32_t* sc = reinterpret_cast<const uint32_t*>(base + S::kScales);
    uint32_t sa[TM], sb[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) sa[i] = sc[256 + wm * TM * 32 + i * 32 + lr] >> (8 * half);
#pragma unroll
    for (int j = 0; j < TN; ++j) sb[j] = sc[b_row(j) + lr] >> (8 * half);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      i32x4 fb[TN];
      Frag fa[TM];
      const int chunk = ((2 * s + half) ^ ((lr >> 2) & 3)) * 16;
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = *reinterpret_cast<const i32x4*>(b + b_row(j) * 64 + chunk);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        fa[i].first = *reinterpret_cast<const i32x4*>(a + i * 32 * 64 + chunk);
        if constexpr (kBits == mx::kF6)
          fa[i].rest = *reinterpret_cast<const i32x2*>(a2 + i * 32 * 32 + (s ^ ((lr >> 3) & 1)) * 16);
      }
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = s == 0 ? mma32<kBits, 0>(fb[j], fa[i], acc[i][j], sb[j], sa[i])
                             : mma32<kBits, 2>(fb[j], fa[i], acc[i][j], sb[j], sa[i]);
    }
  };

  // Stage kt % ST holds step kt.  A step waits for its own loads (those of the ST
  // - 2 steps after it stay in flight), meets the other waves, and loads into the
  // stage that all of them left in the step before.
#pragma unroll
  for (int kt = 0; kt < ST - 1; ++kt)
    if (kt < KT) issue(kt, kt);
  int kt = 0;
  for (; kt + ST - 1 < KT;) {
#pragma unroll
    for (int u = 0; u < ST; ++u) {
      if (kt + ST - 1 >= KT) break;
      wait_vm<(ST - 2) * L>();
      __syncthreads();
      issue(kt + ST - 1, (u + ST - 1) % ST);
      compute(u);
      ++kt;
    }
  }
  wait_vm<0>();
  __syncthreads();
  for (; kt < KT; ++kt) compute(kt % ST);

  // ---- epilogue: lane (half, lr) holds row lr's columns 8 q + 4 half + i of each 32
  if constexpr (EPI == kMxSwiGLU || EPI == kMxGELU) {
    // Two blocks at a time: the halves trade, and lanes 0..31 hold the first block's 32
    // columns, lanes 32..63 the second's.
    constexpr int TC = TN / NMAT;
    auto value = [&](int b, int u) {
      const int i = b / TC, j = b % TC;
      if constexpr (NMAT == 2) return swiglu_h(acc[i][j][u], acc[i][j + TC][u]);
      else return gelu_h(acc[i][j][u]);
    };
#pragma unroll
    for (int b = 0; b < TM * TC; b += 2) {
      float v[32];
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(value(b, u)), __float_as_uint(value(b + 1, u)), false, false);
        v[8 * (u / 4) + u % 4] = __uint_as_float(t[0]);
        v[8 * (u / 4) + 4 + u % 4] = __uint_as_float(t[1]);
      }
      const mx::Operand o = mx::encode_block<kBits>(v);
      const int mine = b + half, i = mine / TC, j = mine % TC;
      const int r = (wm * TM + i) * 32 + lr, col = n0 + (wn * TC + j) * 32;
      if (r < n && col < g.N) store_block<kBits>(o, row0 + r, g.M, g.N, col, static_cast<uint8_t*>(g.C), g.C2, g.Cs);
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
            d[q][u] = D == 2 ? f32_to_bf16_bits(acc[i][j][4 * q + 2 * u]) | (f32_to_bf16_bits(acc[i][j][4 * q + 2 * u + 1]) << 16)
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

// ---- few rows an expert ------------------------------------------------------------
constexpr int kStreamWaves = 4, kStreamUnroll = 4;

template <int kBits, int EPI>
__global__ __launch_bounds__(64 * kStreamWaves) void stream_kernel(const MxGemm g) {
  constexpr int NMAT = mats(EPI), NT = 2 * NMAT;   // 16-column weight tiles: two of each matrix
  __shared__ f32x4 part[kStreamWaves - 1][NT][64];
  const int mt = blockIdx.x / g.n_col_tiles, nt = blockIdx.x - mt * g.n_col_tiles;
  if (mt >= *g.n_tiles) return;
  const int4 tile = g.tiles[mt];
  const int e = __builtin_amdgcn_readfirstlane(tile.x);
  const int64_t row0 = __builtin_amdgcn_readfirstlane(tile.y);
  const int n = __builtin_amdgcn_readfirstlane(tile.z) - static_cast<int>(row0);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lr = lane & 15, grp = lane >> 4;
  const int K = g.K, KT = K / kStepK;
  const int b_bytes = K / 2, a2_bytes = K / 4, s_bytes = K / mx::kBlock;
  const int64_t wofs = static_cast<int64_t>(e) * g.N;
  const int64_t b_all = static_cast<int64_t>(g.N) * b_bytes, s_all = static_cast<int64_t>(g.N) * s_bytes;
  const __amdgpu_buffer_rsrc_t rb0 = rsrc(g.B0 + wofs * b_bytes, b_all), rs0 = rsrc(g.S0 + wofs * s_bytes, s_all);
  const __amdgpu_buffer_rsrc_t rb1 = NMAT == 2 ? rsrc(g.B1 + wofs * b_bytes, b_all) : rb0;
  const __amdgpu_buffer_rsrc_t rs1 = NMAT == 2 ? rsrc(g.S1 + wofs * s_bytes, s_all) : rs0;
  // rows past the tile's and rows mapped outside x read as zero: their offsets lie
  // past the descriptors' ends
  int src = lr < n ? lr : -1;
  if (g.a_rows && lr < n) {
    src = g.a_rows[row0 + lr];
    if (src >= g.a_n) src = -1;
  }
  const int64_t first = g.a_rows ? 0 : row0, span = g.a_rows ? g.a_n : n;
  const __amdgpu_buffer_rsrc_t ra = rsrc(g.A + first * b_bytes, span * b_bytes);
  const __amdgpu_buffer_rsrc_t ra2 = kBits == mx::kF6 ? rsrc(g.A2 + first * a2_bytes, span * a2_bytes) : ra;
  const __amdgpu_buffer_rsrc_t rsa = rsrc(g.As, g.a_n * 4 * KT);
  const int offa = src < 0 ? kGatherOut : src * b_bytes + grp * 16;
  const int offa2 = src < 0 ? kGatherOut : src * a2_bytes + grp * 8;
  const int offsa = src < 0 ? kGatherOut : static_cast<int>(first + src) * 4;
  const int a_step = static_cast<int>(g.a_n) * 4;
  const int col0 = nt * kStreamCols + lr;
  int offb[2], offs[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    offb[c] = (col0 + 16 * c) * b_bytes + grp * 16;
    offs[c] = (col0 + 16 * c) * s_bytes;
  }
  f32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int end = KT * (wave + 1) / kStreamWaves;
  for (int k0 = KT * wave / kStreamWaves; k0 < end; k0 += kStreamUnroll) {
    i32x4 w[kStreamUnroll][NT], sw[NT];
    Frag a[kStreamUnroll];
    uint32_t sa[kStreamUnroll];
#pragma unroll
    for (int j = 0; j < NT; ++j) sw[j] = load16(j >= 2 ? rs1 : rs0, offs[j % 2] + k0 * 4);   // four steps' scales
#pragma unroll
    for (int u = 0; u < kStreamUnroll; ++u) {
      if (k0 + u >= end) break;
#pragma unroll
      for (int j = 0; j < NT; ++j) w[u][j] = load16(j >= 2 ? rb1 : rb0, offb[j % 2] + (k0 + u) * 64);
      a[u].first = load16(ra, offa + (k0 + u) * 64);
      if constexpr (kBits == mx::kF6)
        a[u].rest = __builtin_bit_cast(i32x2, __builtin_amdgcn_raw_buffer_load_b64(ra2, offa2 + (k0 + u) * 32, 0, 0));
      sa[u] = __builtin_amdgcn_raw_buffer_load_b32(rsa, src < 0 ? kGatherOut : offsa + (k0 + u) * a_step, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kStreamUnroll; ++u) {
      if (k0 + u >= end) break;
#pragma unroll
      for (int j = 0; j < NT; ++j)
        acc[j] = mma16<kBits>(w[u][j], a[u], acc[j], static_cast<uint32_t>(sw[j][u]) >> (8 * grp), sa[u] >> (8 * grp));
    }
  }
  if (wave > 0)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave - 1][j][lane] = acc[j];
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int u = 0; u < kStreamWaves - 1; ++u)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] += part[u][j][lane];
  }
  // wave 0's lane (grp, lr) holds row lr's columns 16 c + 4 grp + i
  const int64_t row = row0 + lr;
  const int col = nt * kStreamCols;
  if constexpr (EPI == kMxSwiGLU || EPI == kMxGELU) {
    __shared__ float h[kStreamRows][kStreamCols + 1];   // a row's block goes to one lane
    if (wave == 0) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float v;
          if constexpr (NMAT == 2) v = swiglu_h(acc[c][u], acc[2 + c][u]);
          else v = gelu_h(acc[c][u]);
          h[lr][16 * c + 4 * grp + u] = v;
        }
    }
    __syncthreads();
    if (threadIdx.x >= n) return;
    float v[32];
#pragma unroll
    for (int u = 0; u < 32; ++u) v[u] = h[threadIdx.x][u];
    store_block<kBits>(mx::encode_block<kBits>(v), row0 + threadIdx.x, g.M, g.N, col, static_cast<uint8_t*>(g.C), g.C2, g.Cs);
  } else {
    if (wave > 0 || lr >= n) return;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float v[4] = {acc[c][0], acc[c][1], acc[c][2], acc[c][3]};
      const int64_t at = row * g.N + col + 16 * c + 4 * grp;
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

// Rows of a tile.  By the average rows an expert: few rows are bound by the
// weights' bytes, many by the matrix cores.
int rows_per_tile(int64_t M, int E) {
  const int64_t avg = M / E;
  return avg <= 16 ? kStreamRows : avg <= 96 ? 64 : avg <= 192 ? 128 : 256;
}

// Whatever E a call gives, the list has room for the smallest tiles.
MxLayout mx_layout(int64_t n_src, int64_t M, int H, int I, int max_slots, moe_mx_format fmt) {
  MxLayout w{};
  size_t at = 0;
  auto take = [&](size_t n) { size_t p = at; at = moe::align_up(at + n, 256); return p; };
  const size_t x_values = static_cast<size_t>(n_src) * H, h_values = static_cast<size_t>(M) * I;
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

template <int kBits, int EPI>
int launch_product(MxGemm p, int bm, int64_t row_tiles, hipStream_t s, const char* what) {
  const int64_t cols = bm == kStreamRows ? kStreamCols : 256 / mats(EPI);
  p.n_col_tiles = static_cast<int>(ceil_div(p.N, cols));
  const int64_t blocks = row_tiles * p.n_col_tiles;
  if (blocks >= (int64_t(1) << 24)) return moe::fail(MOE_ERR_UNSUPPORTED, "moe_mx_expert_ffn: %lld blocks in one launch", (long long)blocks);
  const unsigned grid = static_cast<unsigned>(blocks);
  if (bm == kStreamRows) stream_kernel<kBits, EPI><<<grid, 64 * kStreamWaves, 0, s>>>(p);
  else if (bm == 64) tile_kernel<kBits, EPI, 64><<<grid, 256, 0, s>>>(p);
  else if (bm == 128) tile_kernel<kBits, EPI, 128><<<grid, 256, 0, s>>>(p);
  else tile_kernel<kBits, EPI, 256><<<grid, 256, 0, s>>>(p);
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

extern "C" size_t moe_mx_expert_ffn_workspace_bytes(int64_t n_src, int64_t M, int H, int I, int max_slots,
                                                    moe_mx_format x_format) {
  if (n_src < 0 || M < 0 || H < 1 || I < 1 || max_slots < 1 || (x_format != MOE_MX_FP4 && x_format != MOE_MX_FP6)) return 0;
  return mx_layout(n_src, M, H, I, max_slots, x_format).bytes;
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
  // 31-bit offsets: an expert matrix's codes, a tile's rows and the gathered x's, the
  // scales of all rows
  const int64_t kLimit = kGatherLimit;
  if (static_cast<int64_t>(H) * I / 2 >= kLimit || static_cast<int64_t>(std::max(H, I)) * 128 >= kLimit)
    return fail(MOE_ERR_UNSUPPORTED, "%s: H or I too large for 32-bit tile offsets", who);
  if ((row_src && n_src * (H / 2) >= kLimit) || n_src * (H / mx::kBlock) >= kLimit || M * (I / mx::kBlock) >= kLimit)
    return fail(MOE_ERR_UNSUPPORTED, "%s: too many rows for 32-bit offsets (M=%lld, n_src=%lld)", who, (long long)M,
                (long long)n_src);
  if (n_src >= (int64_t(1) << 34) / H) return fail(MOE_ERR_UNSUPPORTED, "%s: x holds 2^34 values or more", who);
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
  const MxLayout w = mx_layout(n_src, M, H, I, max_slots, x_format);
  if (workspace_bytes < w.bytes)
    return fail(MOE_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", who, workspace_bytes, w.bytes);
  if (M == 0) return MOE_OK;
  const hipStream_t s = as_stream(stream);
  char* ws = static_cast<char*>(workspace);
  auto at = [&](size_t offset) { return reinterpret_cast<uint8_t*>(ws + offset); };
  int4* const tiles = reinterpret_cast<int4*>(ws + w.tiles);
  int32_t* const n_tiles = reinterpret_cast<int32_t*>(ws + w.n_tiles);
  const int bm = rows_per_tile(M, E);
  const int64_t row_tiles = M / bm + std::min<int64_t>(M, max_slots);
  const unsigned grid = static_cast<unsigned>(ceil_div(n_src * (H / mx::kBlock), 256) + 1);
  auto prepare = [&](auto kernel) {
    kernel<<<grid, 256, 0, s>>>(x, n_src, H, at(w.xq), at(w.xq2), at(w.xs), slot_off, slot_expert, n_slots, max_slots, M, E, bm, w.cap, tiles,
                                n_tiles, check);
  };
  const bool bf16 = dt == MOE_BF16, fp6 = x_format == MOE_MX_FP6;
  if (bf16) prepare(fp6 ? prepare_kernel<true, mx::kF6> : prepare_kernel<true, mx::kF4>);
  else prepare(fp6 ? prepare_kernel<false, mx::kF6> : prepare_kernel<false, mx::kF4>);
  if (int rc = hip_status(hipGetLastError(), "moe_mx_expert_ffn prepare launch")) return rc;
  MxGemm up{};
  up.A = at(w.xq);
  up.A2 = at(w.xq2);
  up.As = at(w.xs);
  up.a_rows = row_src;
  up.a_n = n_src;
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
  down.a_rows = nullptr;
  down.a_n = M;
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
