// Microscaled 4-bit operands (OCP MX: 32 E2M1 codes and one E8M0 scale to a
// block) for gfx950: quantisation along rows and columns, and the product of
// two operands by v_mfma_scale_f32_32x32x64_f8f6f4, which takes both blocks'
// scales with their codes.
//
// An operand of R rows and padded length Kp holds codes [Kp / 128][R][64] and
// scales [Kp / 128][R][4]: what one stage of the product takes of neighbouring
// rows is contiguous. With rows of Kp / 2 bytes instead, a stage's 64 bytes of
// each row were half lines at one distance, for a power of two all on one
// channel of the L2 (MLP-down's product at K 32768: 986 us against 845).
#pragma once

#include <type_traits>

#include "wgrad_kernels.hpp"

namespace forge {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// --------------------------------------------------------------------------
// quantisation
// --------------------------------------------------------------------------

struct QuantArgs {
  const void* x;
  uint8_t *row_codes, *row_scales, *col_codes, *col_scales;
  int64_t R, C;
  int64_t padded_c;                // padded length of the operand along rows
  uint32_t tiles_c;                // tiles across
  uint32_t tiles;
};

constexpr int kQuantRows = 128;    // a tile: 128 rows of kQuantWords words (2 bf16 or 1 float32)
constexpr int kQuantWords = 128;
constexpr int kQuantThreads = 4 * kQuantWords;
constexpr uint32_t kQuantGrid = 2048;        // most workgroups of a launch
template <bool BF16>
constexpr int kQuantCols = BF16 ? 2 * kQuantWords : kQuantWords;

typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// The scale byte of a block from its largest magnitude's biased exponent: 2
// less (so that the largest lands in [4, 8), the top two codes' range), at least
// 0; 255 for a NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t e) {
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// 4 values to 4 codes (the first in the low half of the first byte), rounded
// to nearest even and saturated by the conversion instruction. It takes the
// scale as a float32 power of two; blocks whose scale (or values) come near
// float32's denormals are multiplied by 2^64 first, exactly.
__device__ __forceinline__ uint32_t codes4(const f32x4_t& x, uint32_t s) {
  f32x4_t a = x;
  uint32_t e = s;
  if (s < 32u) {
    a = a * 0x1p64f;
    e = s + 64u;
  }
  const float scale = __builtin_bit_cast(float, e << 23);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, a[0], a[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, a[2], a[3], scale, 1);
  return s == 255u ? 0u : r;
}

// 8 codes from 8 bf16 values in four words, the earlier one in the low half.
__device__ __forceinline__ uint32_t codes8(const uint32_t (&w)[4], uint32_t s) {
  if (s < 32u)
    return codes4(unpack_bf16x4(u32x2_t{w[0], w[1]}), s) |
           codes4(unpack_bf16x4(u32x2_t{w[2], w[3]}), s) << 16;
  const float scale = __builtin_bit_cast(float, s << 23);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[0]), scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[1]), scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[2]), scale, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[3]), scale, 3);
  return s == 255u ? 0u : r;
}

__device__ __forceinline__ uint32_t abs_bits(uint32_t x) { return x & 0x7fffffffu; }
// The larger magnitude's bits in each half.
__device__ __forceinline__ uint32_t max_abs2(uint32_t top, uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(
      __builtin_bit_cast(u16x2_t, top), __builtin_bit_cast(u16x2_t, w & 0x7fff7fffu)));
}

// A workgroup goes from tile to tile. Loads are row-major, 16 bytes (8 bf16 or
// 4 float32 columns) to a thread, which is what the codes along rows need (4 or
// 8 lanes share a block); the codes along columns are formed from a copy of the
// tile in LDS, one 32-row block of a word's column (a pair of columns for bf16)
// to a thread. Word w of row r is kept at w ^ 16 (r / 32 mod 4), which puts the
// four blocks of 16 neighbouring words, read by one wave at a time, on 64
// different banks. The next tile's loads are in flight while a tile's codes
// along columns are formed and stored.
//
// Bound by HBM. bf16 8192 x 14336: 55 us by columns (297 MB, 5.4 TB/s), 52 by
// rows, 70 for both (360 MB); float32 4096 x 14336 48 us by columns (60 when a
// thread's two loads were neighbours instead of a wave's). Rows of 64 words and
// 32 KB of LDS: 61 and 52 us.
template <bool BF16, bool ROWS, bool COLS>
__global__ __launch_bounds__(kQuantThreads) void quantize_mxfp4_kernel(QuantArgs a) {
  constexpr int WPR = kQuantWords;
  constexpr int TC = kQuantCols<BF16>;
  constexpr int CPT = BF16 ? 8 : 4;          // columns of a load
  constexpr int TPR = WPR / 4;               // threads of a row
  constexpr int RPI = kQuantThreads / TPR, NIT = kQuantRows / RPI;
  __shared__ __attribute__((aligned(16))) uint32_t lds[COLS ? kQuantRows * WPR : 4];
  const int tid = threadIdx.x;
  const int j = tid % TPR, rt = tid / TPR;
  u32x4_t raw[NIT];
  auto load = [&](uint32_t b) {
    const uint32_t tr = b / a.tiles_c;
    const int64_t col = int64_t(b - tr * a.tiles_c) * TC + CPT * j;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const int64_t row = int64_t(tr) * kQuantRows + it * RPI + rt;
      const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(a.x) +
                                                          (row * a.C + col) * (BF16 ? 2 : 4));
      raw[it] = row < a.R && col < a.C ? __builtin_nontemporal_load(p) : u32x4_t{0u, 0u, 0u, 0u};
    }
  };
  load(blockIdx.x);
  for (uint32_t b = blockIdx.x; b < a.tiles; b += gridDim.x) {
    const uint32_t tr = b / a.tiles_c;
    const int64_t r0 = int64_t(tr) * kQuantRows, c0 = int64_t(b - tr * a.tiles_c) * TC;
    const int64_t col = c0 + CPT * j;
#pragma unroll
    for (int it = 0; it < NIT; ++it) {
      const int r = it * RPI + rt;
      if constexpr (COLS)
        *reinterpret_cast<u32x4_t*>(&lds[r * WPR + ((4 * j) ^ (((r >> 5) & 3) << 4))]) = raw[it];
      if constexpr (ROWS) {
        const int64_t row = r0 + r;
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          top = BF16 ? max_abs2(top, raw[it][k]) : max(top, abs_bits(raw[it][k]));
        if constexpr (BF16) top = max(top & 0xffffu, top >> 16) << 16;
        top = max(top, uint32_t(__shfl_xor(int(top), 1)));
        top = max(top, uint32_t(__shfl_xor(int(top), 2)));
        if constexpr (!BF16) top = max(top, uint32_t(__shfl_xor(int(top), 4)));
        const uint32_t s = scale_byte(top >> 23);
        if (row < a.R && col < a.padded_c) {
          const int64_t at = (col >> 7) * a.R + row;
          uint8_t* const out = a.row_codes + at * 64 + (col & 127) / 2;
          if constexpr (BF16) {
            const uint32_t w[4] = {raw[it][0], raw[it][1], raw[it][2], raw[it][3]};
            *reinterpret_cast<uint32_t*>(out) = codes8(w, s);
          } else {
            *reinterpret_cast<uint16_t*>(out) = uint16_t(codes4(__builtin_bit_cast(f32x4_t, raw[it]), s));
          }
          if (j % (32 / CPT) == 0)
            a.row_scales[at * 4 + ((col >> 5) & 3)] = uint8_t(s);
        }
      }
    }
    if (a.tiles - b > gridDim.x) load(b + gridDim.x);
    if constexpr (!COLS) continue;
    __syncthreads();
    // Thread: block `blk` of word column `w`.
    const int blk = tid & 3, w = tid >> 2;
    uint32_t v[32], top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      v[i] = lds[(blk * 32 + i) * WPR + (w ^ (blk << 4))];
      top = BF16 ? max_abs2(top, v[i]) : max(top, abs_bits(v[i]));
    }
    constexpr int NC = BF16 ? 2 : 1;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t column = c0 + w * NC + c;
      if (column < a.C) {
        const uint32_t s = scale_byte(BF16 ? (top >> (16 * c + 7)) & 255u : top >> 23);
        u32x4_t out;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (BF16) {
            uint32_t pair[4];                // the column's values of two rows in a word
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t e = v[8 * k + 2 * q], o = v[8 * k + 2 * q + 1];
              pair[q] = c == 0 ? (e & 0xffffu) | (o << 16) : (e >> 16) | (o & 0xffff0000u);
            }
            out[k] = codes8(pair, s);
          } else {
            f32x4_t lo, hi;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              lo[q] = __builtin_bit_cast(float, v[8 * k + q]);
              hi[q] = __builtin_bit_cast(float, v[8 * k + 4 + q]);
            }
            out[k] = codes4(lo, s) | codes4(hi, s) << 16;
          }
        }
        const int64_t at = int64_t(tr) * a.C + column;
        *reinterpret_cast<u32x4_t*>(a.col_codes + at * 64 + 16 * blk) = out;
        a.col_scales[at * 4 + blk] = uint8_t(s);
      }
    }
    __syncthreads();                         // the next tile reuses the LDS
  }
}

// --------------------------------------------------------------------------
// product
// --------------------------------------------------------------------------
//
// acc[i, o] = sum_k I[i, k] O[o, k]: in the weight gradient's terms (see
// wgrad_kernels.hpp) I is X and O is dY, both already K-major, so an MFMA
// operand (32 columns of one row: one block) is 16 consecutive bytes.
//
// Mainloop: stages of 128 columns, rows of 64 bytes and then their scale words,
// straight from memory into a ring of 4 LDS slots, as the bf16 kernel (the same
// bytes of operands per stage and tile). 16-byte chunk c of row r is kept at
// chunk c ^ (r / 4 mod 4), which puts 16 neighbouring rows' reads on different
// banks. Per slot of one stage, two k-steps of 64:
//   step 0: request the second half of slot s + 3 into the previous one; MFMAs;
//   read step 1's operands from this slot.
//   wait for this wave's LDS reads and for its loads of the next slot; barrier.
//   step 1: request the first half of slot s + 4 into this one; MFMAs; read the
//   scales and step 0's operands from the next slot.
// Slots of two stages have four such steps, and the wait before the last.
// Loads that queue up hold back the wave that issues them: with all of a stage's
// in step 1, MLP-down's product took 222 us against 217, K 32768 805 against 785.
// Columns enter each element in ascending steps of 64, whatever the tile.
//
// Held back by the board's power limit: MLP-down (4096 x 14336 x 8192) takes
// 204-228 us on different boards, 4.2-4.7 PFLOP/s, at 1400 W and a clock of 1.68-1.73
// GHz instead of 2.4, with the matrix cores busy in 64% of the cycles; K 32768
// 769-826 us, 4.7-5.0 PFLOP/s. The limit is not the only thing: fewer cycles per
// stage bought half of their share in time. Small outputs are bound by what a wave
// issues in a stage: 0.1 us of it for 64x64 tiles.
struct MxArgs {
  const uint8_t *i_scales, *o_scales;
  int64_t kp;
};

// Tiles smaller than the other kernels have, for outputs that do not fill the
// chip: fields as TileCfg.
template <int BM_, int BN_, int WAVES_M_, int WAVES_N_, int OCC_, int KS_>
struct SmallTileCfg {
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WAVES_M_, WAVES_N = WAVES_N_, BK = 32, OCC = OCC_;
  static constexpr int KS = KS_;                        // stages of a slot
  static constexpr int WAVES = WAVES_M * WAVES_N, THREADS = 64 * WAVES;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N, TM = WM / 32, TN = WN / 32;
  static constexpr int STAGE = BK * (BM + BN);
  static_assert(WAVES == 4 && TM >= 1 && TN >= 1, "4 waves of whole MFMA blocks");
};
using Mx128x64 = SmallTileCfg<128, 64, 2, 2, 3, 1>;
using Mx64x64 = SmallTileCfg<64, 64, 2, 2, 4, 1>;
using Mx64x64x2 = SmallTileCfg<64, 64, 2, 2, 2, 2>;

// Stages of a slot.
template <class C, class = void>
constexpr int mx_stages = 1;
template <class C>
constexpr int mx_stages<C, std::void_t<decltype(C::KS)>> = C::KS;

// 16-bit elements of a stage's codes and scale words, and of a slot.
template <class C>
__host__ __device__ constexpr int mx_stage() {
  return C::STAGE + 2 * (C::BM + C::BN);
}
template <class C>
__host__ __device__ constexpr int mx_slot() {
  return mx_stages<C> * mx_stage<C>();
}

// 4 bytes per lane from a buffer window straight into LDS: lane t writes at
// dst + 4 t (see load16_to_lds).
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, uint16_t* dst, uint32_t voff,
                                             int soff) {
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 4, voff, soff, 0, 0);
}

template <class C, int EPI>
__device__ __forceinline__ void mxfp4_tile(const WgradArgs& a, const MxArgs& x, int tile_m,
                                           int tile_n, const Slots& sl) {
  constexpr int BM = C::BM, BN = C::BN, TM = C::TM, TN = C::TN;
  constexpr int RB = 64;                                // bytes of a row in a stage
  constexpr int QX = BM * RB / 1024, QY = BN * RB / 1024;
  constexpr int NQW = (QX + QY) / C::WAVES;             // 1 KB loads per wave and stage
  constexpr int SI = BM / 64, SO = BN / 64;             // 256-byte loads of scale words
  constexpr int NSW = (SI + SO + C::WAVES - 1) / C::WAVES;
  constexpr int KS = mx_stages<C>;
  static_assert(KS <= 2, "a slot's halves are its stages");
  constexpr int NL = KS * (NQW + NSW);                  // loads per wave and slot
  // The first half of a slot's loads: its first stage, or the scales and H of the
  // codes of its only one.
  constexpr int H = KS > 1 ? NQW : NL / 2 > NSW ? NL / 2 - NSW : 1;
  constexpr int NL0 = NSW + H, NL1 = NL - NL0;
  constexpr int kScales = RB * (BM + BN);               // their place in a slot
  static_assert((QX + QY) % C::WAVES == 0, "stage loads split evenly over the waves");
  static_assert(RB * (BM + BN) <= C::STAGE * 2, "stage exceeds a slot");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % C::WAVES_M, wn = wave / C::WAVES_M;
  const int d_in = a.d_in, d_out = a.d_out;
  const int i0 = tile_m * BM, o0 = tile_n * BN;
  const int nk = int(x.kp / 128);

  // Loads: instruction q covers 16 rows of I (q < QX) or O, 1 KB on end; lane t
  // fills row t / 4, physical chunk t % 4. Tiles with as many rows of I as of O
  // have waves for each, others give every wave its share of both. Rows past the
  // edge repeat the last one (their products are not stored). A window reaches
  // from the tile's first row to the operand's end, so that stages past the last
  // lie past its end and read zeros; a stage is an offset to it, and it moves on
  // every round of slots. This keeps the scalar instructions few, of which a wave
  // issues one every 8 cycles or so: with windows built for each stage, 1 x 4096 x
  // 14336 took 18.8 us against 14.4, MLP-down's product with K 32768 785 against 769.
  constexpr bool SIDES = QX == QY;
  constexpr int NF = SIDES ? 1 : 2, QXW = SIDES ? NQW : QX / C::WAVES;
  static_assert(SIDES ? QX % NQW == 0 : QX % C::WAVES == 0 && QY % C::WAVES == 0, "whole loads");
  static_assert(SI % NSW == 0 && SO % NSW == 0, "a wave's scale loads are of one side");
  const int left_i = d_in - i0, left_o = d_out > o0 ? d_out - o0 : 1;
  const int row_o = d_out > o0 ? o0 : d_out - 1;        // a half tile may lie past the edge
  struct Feed {
    const uint8_t* p;
    int64_t left, stage;                                // bytes to the end, and of a stage
    __amdgpu_buffer_rsrc_t window;
    __device__ __forceinline__ void open() {
      window = window32(p, left < 0 ? 0u : uint32_t(left < 0x7fffffff ? left : 0x7fffffff));
    }
    __device__ __forceinline__ void advance(int stages) {
      p += stage * stages;
      left -= stage * stages;
      open();
    }
  };
  auto feed = [&](bool o_side, const void* i_base, const void* o_base, int row_bytes) {
    const int rows = o_side ? d_out : d_in, row0 = o_side ? row_o : i0;
    Feed f;
    f.p = static_cast<const uint8_t*>(o_side ? o_base : i_base) + int64_t(row0) * row_bytes;
    f.stage = int64_t(rows) * row_bytes;
    f.left = f.stage * nk - int64_t(row0) * row_bytes;
    f.open();
    return f;
  };
  const int sq0 = wave * NSW % (SI + SO);               // with 6 loads for 4 waves, two are made twice
  Feed codes[NF], scales = feed(sq0 >= SI, x.i_scales, x.o_scales, 4);
  codes[0] = feed(SIDES && wave >= C::WAVES / 2, a.X, a.dY, RB);
  if constexpr (!SIDES) codes[1] = feed(true, a.X, a.dY, RB);
  uint32_t voff[NQW], soff[NSW];
  auto load_of = [&](int i) { return i < QXW ? wave * QXW + i : QX + wave * (NQW - QXW) + i - QXW; };
#pragma unroll
  for (int i = 0; i < NQW; ++i) {
    const int q = load_of(i);
    const int row = (q < QX ? q : q - QX) * 16 + (lane >> 2);
    voff[i] = uint32_t(min(row, (q < QX ? left_i : left_o) - 1) * RB + ((lane & 3) ^ ((lane >> 4) & 3)) * 16);
  }
#pragma unroll
  for (int i = 0; i < NSW; ++i) {
    const int q = sq0 + i;
    soff[i] = uint32_t(min((q < SI ? q : q - SI) * 64 + lane, (q < SI ? left_i : left_o) - 1) * 4);
  }
  // The first or second half of slot j of a round.
  auto load_half = [&](uint16_t* slot, int j, auto second) {
    constexpr bool SECOND = decltype(second)::value;
    const int u = KS * j + (SECOND && KS > 1);
    if constexpr (SECOND && KS > 1) slot += mx_stage<C>();
    if constexpr (!SECOND || KS > 1)
#pragma unroll
      for (int i = 0; i < NSW; ++i)
        load4_to_lds(scales.window, slot + kScales / 2 + (sq0 + i) * 128, soff[i], int(scales.stage) * u);
#pragma unroll
    for (int i = SECOND && KS == 1 ? H : 0; i < (SECOND ? NQW : H); ++i) {
      const Feed& f = codes[i < QXW ? 0 : NF - 1];
      load16_to_lds(f.window, slot + load_of(i) * 512, voff[i], int(f.stage) * u);
    }
  };
  auto advance = [&]() {
#pragma unroll
    for (int k = 0; k < NF; ++k) codes[k].advance(4 * KS);
    scales.advance(4 * KS);
  };
  const std::false_type first_half{};
  const std::true_type second_half{};

  // Operand addresses in a slot for step 0; step 1 is 32 bytes away (chunk
  // 2 + h, and the swizzle is an exclusive or). A scale word holds the four
  // blocks of a row in a stage; this lane's half h of the wave takes blocks
  // 2 kk + h, so the word is shifted by h bytes once and step kk picks byte 2 kk.
  const int l32 = lane & 31, h = lane >> 5;
  uint32_t fa[TM], fb[TN];
  const uint32_t ch0 = uint32_t((h ^ ((l32 >> 2) & 3)) * 16);
#pragma unroll
  for (int m = 0; m < TM; ++m) fa[m] = uint32_t((wm * C::WM + m * 32 + l32) * RB) + ch0;
#pragma unroll
  for (int n = 0; n < TN; ++n) fb[n] = uint32_t((BM + wn * C::WN + n * 32 + l32) * RB) + ch0;
  const uint32_t sa = uint32_t(kScales + (wm * C::WM + l32) * 4);
  const uint32_t sb = uint32_t(kScales + (BM + wn * C::WN + l32) * 4);
  i32x4_t frag[2][TM + TN];
  auto read_frags = [&](int f, const uint16_t* slot, int kk) {
    const char* base = reinterpret_cast<const char*>(slot);
#pragma unroll
    for (int m = 0; m < TM; ++m)
      frag[f][m] = *reinterpret_cast<const i32x4_t*>(base + (fa[m] ^ (32u * kk)));
#pragma unroll
    for (int n = 0; n < TN; ++n)
      frag[f][TM + n] = *reinterpret_cast<const i32x4_t*>(base + (fb[n] ^ (32u * kk)));
  };
  uint32_t sc[TM + TN], now[TM + TN];
  auto read_scales = [&](const uint16_t* slot) {
    const char* base = reinterpret_cast<const char*>(slot);
#pragma unroll
    for (int m = 0; m < TM; ++m) sc[m] = *reinterpret_cast<const uint32_t*>(base + sa + m * 128);
#pragma unroll
    for (int n = 0; n < TN; ++n)
      sc[TM + n] = *reinterpret_cast<const uint32_t*>(base + sb + n * 128);
  };
  auto shift_scales = [&]() {
#pragma unroll
    for (int t = 0; t < TM + TN; ++t) now[t] = sc[t] >> (8 * h);
  };
  f32x16_t acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][n][r] = 0.0f;
  auto wide = [](const i32x4_t& v) { return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; };
  constexpr int kFp4 = 4;                               // operand format code of the instruction
  auto mfmas0 = [&]() {
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int n = 0; n < TN; ++n)
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            wide(frag[0][m]), wide(frag[0][TM + n]), acc[m][n], kFp4, kFp4, 0, int(now[m]), 0,
            int(now[TM + n]));
  };
  auto mfmas1 = [&]() {
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int n = 0; n < TN; ++n)
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            wide(frag[1][m]), wide(frag[1][TM + n]), acc[m][n], kFp4, kFp4, 2, int(now[m]), 2,
            int(now[TM + n]));
  };
  auto interleave = [&](int reads, int loads) {
#pragma unroll
    for (int i = 0; i < TM * TN; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // MFMA
      if (i < reads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);        // DS read
      if (i % 2 == 0 && i / 2 < loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
    }
  };
  constexpr int kWaitMid = waitcnt_imm(2 * NL, 0);
  constexpr int kWaitFirst = waitcnt_imm(2 * NL + NL0, 15);
#define FORGE_MX_BARRIER(IMM)                 \
  do {                                        \
    __builtin_amdgcn_sched_barrier(0);        \
    __builtin_amdgcn_s_waitcnt(IMM);          \
    asm volatile("" ::: "memory");            \
    __builtin_amdgcn_s_barrier();             \
    asm volatile("" ::: "memory");            \
    __builtin_amdgcn_sched_barrier(0);        \
  } while (0)
  // Slot j of a round of four.
  auto run_slot = [&](uint16_t* prv, uint16_t* cur, uint16_t* nxt, int j) {
    shift_scales();
    load_half(prv, (j + 3) % 4, second_half);    // of slot s + 3
    if (j == 0) advance();
    read_frags(1, cur, 1);
    mfmas0();
    interleave(TM + TN, NL1);
    if constexpr (KS > 1) {                      // its second stage
      __builtin_amdgcn_sched_barrier(0);
      const uint16_t* const two = cur + mx_stage<C>();
      read_scales(two);
      read_frags(0, two, 0);
      mfmas1();
      interleave(2 * (TM + TN), 0);
      __builtin_amdgcn_sched_barrier(0);
      shift_scales();
      read_frags(1, two, 1);
      mfmas0();
      interleave(TM + TN, 0);
    }
    FORGE_MX_BARRIER(kWaitMid);
    load_half(cur, j, first_half);               // of slot s + 4, into the freed one
    read_scales(nxt);
    read_frags(0, nxt, 0);
    mfmas1();
    interleave(2 * (TM + TN), NL0);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (nk > 0) {
    for (int j = 0; j < 3; ++j) {
      uint16_t* const slot = j == 0 ? sl.s0 : j == 1 ? sl.s1 : sl.s2;
      load_half(slot, j, first_half);
      load_half(slot, j, second_half);
    }
    load_half(sl.s3, 3, first_half);
    FORGE_MX_BARRIER(kWaitFirst);
    read_scales(sl.s0);
    read_frags(0, sl.s0, 0);
    // Whole rounds of 4 slots: the accumulators keep their registers. Stages
    // past the last add products of zero codes and zero scale bytes: exactly +0.
    const int rounds = (nk + 4 * KS - 1) / (4 * KS);
    for (int r = 0; r < rounds; ++r) {
      run_slot(sl.s3, sl.s0, sl.s1, 0);
      run_slot(sl.s0, sl.s1, sl.s2, 1);
      run_slot(sl.s1, sl.s2, sl.s3, 2);
      run_slot(sl.s2, sl.s3, sl.s0, 3);
    }
  }
#undef FORGE_MX_BARRIER
  uint16_t* ep = wave == 0 ? sl.s0 : wave == 1 ? sl.s1 : wave == 2 ? sl.s2 : sl.s3;
  epilogue<C, EPI>(a, acc, a.W, a.S1, a.S2, i0, o0, wm, wn, lane, reinterpret_cast<float*>(ep));
}

template <class C, int EPI>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(C::OCC, C::OCC)))
void mxfp4_kernel(WgradArgs a, MxArgs x) {
  FORGE_DECLARE_SLOTS(mx_slot<C>());
  int e, tm, tn;
  map_tile(blockIdx.x, a.num_tiles, a.tiles_m, a.tiles_n, a.group_m, e, tm, tn);
  mxfp4_tile<C, EPI>(a, x, tm, tn, ring);
}

// The persistent schedule of the bf16 kernel.
template <class CF, class CH, int EPI>
__global__ __launch_bounds__(CF::THREADS) __attribute__((amdgpu_waves_per_eu(1, 1)))
void mxfp4_persistent_kernel(WgradArgs a, MxArgs x) {
  static_assert(CF::THREADS == CH::THREADS && CF::BM == CH::BM && CF::BN == 2 * CH::BN,
                "half tiles must split the full tile's columns");
  FORGE_DECLARE_SLOTS(mx_slot<CF>());
  const int b = blockIdx.x, xcd = b & 7, j = b >> 3, nw = gridDim.x >> 3;
  const int per = a.num_tiles >> 3, rem = a.num_tiles & 7;
  const int start = xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per;
  const int R = per + (xcd < rem ? 1 : 0);
  const int phase = schedule_phase(xcd, R, nw);
  for (int k = 0;; ++k) {
    int tile, half;
    if (!schedule_item(k, j, nw, R, phase, tile, half)) break;
    int tm, tn;
    grouped_walk(start + tile, a.tiles_m, a.tiles_n, a.group_m, tm, tn);
    if (half < 0)
      mxfp4_tile<CF, EPI>(a, x, tm, tn, ring);
    else
      mxfp4_tile<CH, EPI>(a, x, tm, 2 * tn + half, ring);
    __syncthreads();
  }
}

}  // namespace forge
