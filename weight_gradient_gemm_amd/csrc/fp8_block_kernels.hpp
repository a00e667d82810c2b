// 8-bit floating point operands with a power-of-two scale for each block of 128
// for gfx950: quantisation along rows and columns, and the product of two
// operands by v_mfma_scale_f32_32x32x64_f8f6f4, which takes the scales with the
// codes (its blocks are of 32 values, so four of them have one byte).
//
// An operand of R rows and padded length Kp holds codes [Kp / 64][R][64], what one
// stage of the product takes of neighbouring rows on end, and scales
// [Kp / 128][R to a multiple of 128], in each 128 of which the four rows at a
// distance of 32 share a word: a lane's rows of a wave's tile.
#pragma once

#include "mxfp4_kernels.hpp"
#include "row_io.hpp"

namespace forge {

// --------------------------------------------------------------------------
// quantisation
// --------------------------------------------------------------------------

struct Fp8QuantArgs {
  const void* x;
  uint8_t *row_codes, *row_scales, *col_codes, *col_scales;
  int64_t R, C;
  int64_t row_pitch, col_pitch;      // bytes of a group of scales
  uint32_t tiles, tiles_c;           // tiles, and tiles across
  int32_t square;
};

constexpr int kFp8Tile = 128;        // rows and columns of a tile: a block each way
constexpr int kFp8QuantThreads = 256;

// The scale byte of a block from its largest magnitude's bits: the least
// exponent that brings it to at most 1.75 * 2^REACH (448 or 57344), which is one
// more where its fraction is beyond 1.75; 255 for a NaN or an infinity.
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t top) {
  constexpr uint32_t reach = E5M2 ? 15 : 8;
  const uint32_t e = (top + 0x1fffffu) >> 23;
  return (top >> 23) == 255u ? 255u : e > reach ? e - reach : 0u;
}

// What values are multiplied by to be encoded: 2^(127 - s), a normal float32 for
// every s of finite values. Products that are not exact lie below the least code.
__device__ __forceinline__ float fp8_factor(uint32_t s) {
  return s == 255u ? 0.0f : __builtin_bit_cast(float, (254u - s) << 23);
}

// Four values times their factors to four codes, rounded to nearest even.
template <bool E5M2>
__device__ __forceinline__ uint32_t fp8_codes4(const float (&v)[4]) {
  int r = 0;
  if constexpr (E5M2) {
    r = __builtin_amdgcn_cvt_pk_bf8_f32(v[0], v[1], r, false);
    r = __builtin_amdgcn_cvt_pk_bf8_f32(v[2], v[3], r, true);
  } else {
    r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], r, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], r, true);
  }
  return uint32_t(r);
}

struct Larger {
  __device__ __forceinline__ uint32_t operator()(uint32_t x, uint32_t y) const { return max(x, y); }
};

// Byte of row r's scale among its 128.
__device__ __forceinline__ int fp8_scale_place(int r) { return (r & 31) * 4 + (r >> 5); }

// A tile of 128 x 128 values to a workgroup: thread (j, t) holds rows 8 t .. 8 t + 7
// of eight columns, bf16 8 j .. 8 j + 7, float32 4 j .. 4 j + 3 of each half (so that a
// load instruction's 16 lanes are on end: 8192 x 14336 by columns 97 us, 112 with
// 8 columns on end). So it has eight codes on end of the operand along columns, and
// eight or twice four of that along rows. They pass through LDS on the way out, 64
// bytes of a row (or column) in each half of the tile, and leave as whole lines. Row q
// of a half is kept at q ^ (q / 8 mod 4) and its 16-byte chunk c at c ^ (q / 32),
// which spreads one write instruction's rows over all banks.
//
// Rows alone come here in squares only. Bound by HBM: 8192 x 14336 takes, from bf16, 61 us
// by columns (5.8 TB/s) and 97 for both, 4.8 TB/s, what a copy reaches; from float32 97 and 138.
template <bool BF16, bool E5M2, bool ROWS, bool COLS>
__global__ __launch_bounds__(kFp8QuantThreads) void quantize_fp8_block_kernel(Fp8QuantArgs a) {
  constexpr int NW = BF16 ? 4 : 8;               // words of 8 values
  __shared__ __attribute__((aligned(16))) uint8_t out[(ROWS ? 16384 : 0) + (COLS ? 16384 : 0)];
  __shared__ uint32_t col_top[4][kFp8Tile];
  __shared__ uint32_t all_top[4];
  __shared__ __attribute__((aligned(4))) uint8_t scales[2][kFp8Tile];
  uint8_t* const out_r = out;
  uint8_t* const out_c = out + (ROWS ? 16384 : 0);
  const int tid = threadIdx.x, j = tid & 15, t = tid >> 4, wave = tid >> 6;
  const uint32_t tr = blockIdx.x / a.tiles_c, tc = blockIdx.x - tr * a.tiles_c;
  const int64_t r0 = int64_t(tr) * kFp8Tile, c0 = int64_t(tc) * kFp8Tile;
  auto column = [&](int k) { return BF16 ? 8 * j + k : (k >> 2) * 64 + 4 * j + (k & 3); };
  float v[8][8];
  uint32_t top[8] = {};                          // of columns
  uint32_t row_top[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + 8 * t + i;
    u32x4_t raw[NW / 4];
#pragma unroll
    for (int k = 0; k < NW / 4; ++k) raw[k] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < NW / 4; ++k) {
      const int64_t c = c0 + column(4 * k);
      if (row < a.R && c < a.C)
        raw[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(
            static_cast<const char*>(a.x) + (row * a.C + c) * (BF16 ? 2 : 4)));
    }
    row_top[i] = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t w = BF16 ? raw[0][k / 2] : raw[(k / 4) % (NW / 4)][k % 4];
      const uint32_t bits = BF16 ? (k & 1 ? w & 0xffff0000u : w << 16) : w;
      v[i][k] = __builtin_bit_cast(float, bits);
      const uint32_t m = abs_bits(bits);
      top[k] = max(top[k], m);
      row_top[i] = max(row_top[i], m);
    }
  }
  if (!COLS || a.square) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, top[k]);
    m = rows_all(row16_all(m, Larger()), Larger());
    if ((tid & 63) == 0) all_top[wave] = m;
    __syncthreads();
    m = max(max(all_top[0], all_top[1]), max(all_top[2], all_top[3]));
#pragma unroll
    for (int k = 0; k < 8; ++k) top[k] = row_top[k] = m;
  } else {
    if constexpr (ROWS)
#pragma unroll
      for (int i = 0; i < 8; ++i) row_top[i] = row16_all(row_top[i], Larger());
#pragma unroll
    for (int k = 0; k < 8; ++k) top[k] = rows_all(top[k], Larger());
    if ((tid & 63) < 16)
#pragma unroll
      for (int k = 0; k < 8; ++k) col_top[wave][column(k)] = top[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      top[k] = max(max(col_top[0][column(k)], col_top[1][column(k)]),
                   max(col_top[2][column(k)], col_top[3][column(k)]));
  }
  auto place = [](int half, int q, int byte) {
    return half * 8192 + (q ^ ((q >> 3) & 3)) * 64 + (byte ^ (((q >> 5) & 3) << 4));
  };
  if constexpr (ROWS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 8 * t + i;
      const uint32_t s = fp8_scale_byte<E5M2>(row_top[i]);
      const float f = fp8_factor(s);
      const float lo[4] = {v[i][0] * f, v[i][1] * f, v[i][2] * f, v[i][3] * f};
      const float hi[4] = {v[i][4] * f, v[i][5] * f, v[i][6] * f, v[i][7] * f};
      const uint32_t w0 = s == 255u ? 0u : fp8_codes4<E5M2>(lo), w1 = s == 255u ? 0u : fp8_codes4<E5M2>(hi);
      if constexpr (BF16) {
        *reinterpret_cast<u32x2_t*>(out_r + place(j >> 3, r, (j & 7) * 8)) = u32x2_t{w0, w1};
      } else {
        *reinterpret_cast<uint32_t*>(out_r + place(0, r, 4 * j)) = w0;
        *reinterpret_cast<uint32_t*>(out_r + place(1, r, 4 * j)) = w1;
      }
      if (j == 0) scales[0][fp8_scale_place(r)] = r0 + r < a.R ? uint8_t(s) : 0;
    }
  }
  if constexpr (COLS) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = column(k);
      const uint32_t s = fp8_scale_byte<E5M2>(top[k]);
      const float f = fp8_factor(s);
      const float lo[4] = {v[0][k] * f, v[1][k] * f, v[2][k] * f, v[3][k] * f};
      const float hi[4] = {v[4][k] * f, v[5][k] * f, v[6][k] * f, v[7][k] * f};
      const uint32_t w0 = s == 255u ? 0u : fp8_codes4<E5M2>(lo), w1 = s == 255u ? 0u : fp8_codes4<E5M2>(hi);
      *reinterpret_cast<u32x2_t*>(out_c + place(t >> 3, c, (t & 7) * 8)) = u32x2_t{w0, w1};
      if (t == 0) scales[1][fp8_scale_place(c)] = c0 + c < a.C ? uint8_t(s) : 0;
    }
  }
  __syncthreads();
  if (tid < kFp8Tile / 4) {
    if constexpr (ROWS)
      *reinterpret_cast<uint32_t*>(a.row_scales + tc * a.row_pitch + r0 + 4 * tid) =
          *reinterpret_cast<const uint32_t*>(&scales[0][4 * tid]);
    if constexpr (COLS)
      *reinterpret_cast<uint32_t*>(a.col_scales + tr * a.col_pitch + c0 + 4 * tid) =
          *reinterpret_cast<const uint32_t*>(&scales[1][4 * tid]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = i * 256 + tid, half = n >> 9, q = (n >> 2) & 127, byte = (n & 3) * 16;
    if constexpr (ROWS)
      if (r0 + q < a.R)
        *reinterpret_cast<u32x4_t*>(a.row_codes + ((int64_t(tc) * 2 + half) * a.R + r0 + q) * 64 + byte) =
            *reinterpret_cast<const u32x4_t*>(out_r + place(half, q, byte));
    if constexpr (COLS)
      if (c0 + q < a.C)
        *reinterpret_cast<u32x4_t*>(a.col_codes + ((int64_t(tr) * 2 + half) * a.C + c0 + q) * 64 + byte) =
            *reinterpret_cast<const u32x4_t*>(out_c + place(half, q, byte));
  }
}

// Along rows alone, 128 at a time: 16 lanes to a block, 16 rows of one block to a
// workgroup, so that a store instruction's codes are two runs of 1 KB at most, and nothing goes
// through LDS. The last rows' workgroup clears the scales behind them. 1 x 14336 bf16 takes
// 2.5 us (4.0 by the kernel of tiles), 333 x 1024 2.6 (4.2), 4096 x 4096 10.5 (12.6), 8192 x
// 14336 65 (69), from float32 107 (110). Loads past the caches: 4096 x 4096 11.4 us,
// from float32 17 instead of 13.5.
constexpr int kFp8RowsOf = 16;
template <bool BF16, bool E5M2>
__global__ __launch_bounds__(kFp8QuantThreads) void quantize_fp8_block_rows_kernel(Fp8QuantArgs a) {
  const int tid = threadIdx.x, j = tid & 15;
  for (uint32_t item = blockIdx.x; item < a.tiles; item += gridDim.x) {
    const uint32_t tr = item / a.tiles_c, tc = item - tr * a.tiles_c;
    const int64_t row = int64_t(tr) * kFp8RowsOf + (tid >> 4), c = int64_t(tc) * 128 + 8 * j;
    u32x4_t raw[BF16 ? 1 : 2] = {};
    if (row < a.R && c < a.C) {
      const u32x4_t* const p =
          reinterpret_cast<const u32x4_t*>(static_cast<const char*>(a.x) + (row * a.C + c) * (BF16 ? 2 : 4));
      raw[0] = p[0];
      if constexpr (!BF16) raw[1] = p[1];
    }
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t w = BF16 ? raw[0][k / 2] : raw[BF16 ? 0 : k / 4][k % 4];
      v[k] = __builtin_bit_cast(float, BF16 ? (k & 1 ? w & 0xffff0000u : w << 16) : w);
    }
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, abs_bits(__builtin_bit_cast(uint32_t, v[k])));
    const uint32_t s = fp8_scale_byte<E5M2>(row16_all(top, Larger()));
    const float f = fp8_factor(s);
    const float lo[4] = {v[0] * f, v[1] * f, v[2] * f, v[3] * f}, hi[4] = {v[4] * f, v[5] * f, v[6] * f, v[7] * f};
    const uint32_t w0 = s == 255u ? 0u : fp8_codes4<E5M2>(lo), w1 = s == 255u ? 0u : fp8_codes4<E5M2>(hi);
    uint8_t* const scales = a.row_scales + tc * a.row_pitch;
    if (row < a.R) {
      *reinterpret_cast<u32x2_t*>(a.row_codes + ((int64_t(tc) * 2 + (j >> 3)) * a.R + row) * 64 + (j & 7) * 8) =
          u32x2_t{w0, w1};
      if (j == 0) scales[(row & ~127) + fp8_scale_place(int(row & 127))] = uint8_t(s);
    }
    if ((int64_t(tr) + 1) * kFp8RowsOf >= a.R && tid < 128) {
      const int64_t pad = (a.R & ~127) + tid;
      if (pad >= a.R && pad < a.row_pitch) scales[(pad & ~127) + fp8_scale_place(int(pad & 127))] = 0;
    }
  }
}

// --------------------------------------------------------------------------
// product
// --------------------------------------------------------------------------
//
// acc[i, o] = sum_k I[i, k] O[o, k], in the weight gradient's terms (see
// wgrad_kernels.hpp): I is B of the entry point, O is A.
//
// Stages of 64 columns (one MFMA k-step), rows of 64 bytes and then their scale
// words, straight from memory into a ring of 4 LDS slots. 16-byte chunk c of row r is
// kept at chunk c ^ (r / 4 mod 4), which puts 16 neighbouring rows' reads on
// different banks. A slot of one stage: request stage s + 4 into the slot that the last
// barrier freed, MFMAs on stage s, whose operands are in registers, while those of
// stage s + 1 are read from its slot; then wait for these reads and for this
// wave's loads of stage s + 2, and one barrier. Small tiles, whose waves have few
// MFMAs to a stage, have slots of two: the barrier comes between their stages.
// Columns enter each element in ascending steps of 64, whatever the tile.
//
// Bound by the board's power: MLP-down's output (8192 x 4096 x 14336) takes 308 to 318 us,
// 3.0-3.1 PFLOP/s, at 1400 W and 1.72 GHz with the matrix cores busy 84% of the cycles; the
// instruction alone, without operand traffic, reaches 4.06 PFLOP/s there on codes of
// normal values. The 16 x 16 x 128 form alone reaches 4.42, but its stages of 128
// columns leave room for two slots of 256x256 tiles where a load needs three. Fewer
// LDS reads or loads between two MFMAs, or the loads last, take the same time; without
// the interleaving, or with s_setprio around the MFMAs, it is 13% slower. Slots of two
// stages pay off at 128x64 and 64x64 only (128x128: 0.21 us a stage and 0.18).
struct Fp8BlockArgs {
  const uint8_t *i_scales, *o_scales;
  int64_t kp;
};

// 16-bit elements of a slot: the codes of its stages, and 256 bytes of scales of
// each side.
template <class C>
__host__ __device__ constexpr int fp8_block_slot() {
  return mx_stages<C> * C::STAGE + 256;
}

template <class C, int FI, int FO>
__device__ __forceinline__ void fp8_block_tile(const WgradArgs& a, const Fp8BlockArgs& x, int tile_m,
                                               int tile_n, const Slots& sl) {
  constexpr int BM = C::BM, BN = C::BN, TM = C::TM, TN = C::TN;
  constexpr int RB = 64;                                // bytes of a row in a stage
  constexpr int QX = BM * RB / 1024, QY = BN * RB / 1024;
  constexpr int NQW = (QX + QY) / C::WAVES;             // 1 KB loads per wave and stage
  constexpr int KS = mx_stages<C>;                      // stages of a slot
  static_assert(KS <= 2, "a slot is within a group of scales");
  constexpr int NL = KS * NQW + 1;                      // with 256 bytes of scales
  constexpr int kStage = RB * (BM + BN), kScales = KS * kStage;   // places in a slot
  static_assert((QX + QY) % C::WAVES == 0, "stage loads split evenly over the waves");
  static_assert(RB * (BM + BN) <= C::STAGE * 2 && BM <= 256 && BN <= 256, "stage exceeds a slot");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % C::WAVES_M, wn = wave / C::WAVES_M;
  const int d_in = a.d_in, d_out = a.d_out;
  const int i0 = tile_m * BM, o0 = tile_n * BN;
  const int nk = int(x.kp / 64);

  // Loads: instruction q covers 16 rows of I (q < QX) or O, 1 KB on end; lane t
  // fills row t / 4, physical chunk t % 4. Rows past the edge repeat the last one
  // (their products are not stored). A window reaches from the tile's first row
  // to the operand's end, so that stages past the last read zeros; a stage is an
  // offset to it, and it moves on every round of slots.
  constexpr bool SIDES = QX == QY;                      // waves for each side, else each its share of both
  constexpr int NF = SIDES ? 1 : 2, QXW = SIDES ? NQW : QX / C::WAVES;
  static_assert(SIDES ? QX % NQW == 0 : QX % C::WAVES == 0 && QY % C::WAVES == 0, "whole loads");
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
  auto feed = [&](const void* base, int64_t stage, int64_t first, int stages) {
    Feed f;
    f.p = static_cast<const uint8_t*>(base) + first;
    f.stage = stage;
    f.left = stage * stages - first;
    f.open();
    return f;
  };
  auto code_feed = [&](bool o_side) {
    return feed(o_side ? a.dY : a.X, int64_t(o_side ? d_out : d_in) * RB, int64_t(o_side ? row_o : i0) * RB, nk);
  };
  const bool scales_o = wave >= C::WAVES / 2;           // two waves load the same words
  const int rows_s = scales_o ? d_out : d_in, first_s = (scales_o ? row_o : i0) & ~127;
  Feed codes[NF], scales = feed(scales_o ? x.o_scales : x.i_scales, (rows_s + 127) & ~127, first_s, nk / 2);
  codes[0] = code_feed(SIDES && wave >= C::WAVES / 2);
  if constexpr (!SIDES) codes[1] = code_feed(true);
  uint32_t voff[NQW];
  auto load_of = [&](int i) { return i < QXW ? wave * QXW + i : QX + wave * (NQW - QXW) + i - QXW; };
#pragma unroll
  for (int i = 0; i < NQW; ++i) {
    const int q = load_of(i);
    const int row = (q < QX ? q : q - QX) * 16 + (lane >> 2);
    voff[i] = uint32_t(min(row, (q < QX ? left_i : left_o) - 1) * RB + ((lane & 3) ^ ((lane >> 4) & 3)) * 16);
  }
  const uint32_t soff = uint32_t(lane * 4);
  // Slot j of the round that the windows are at.
  auto load_slot = [&](uint16_t* slot, int j) {
    load4_to_lds(scales.window, slot + kScales / 2 + (scales_o ? 128 : 0), soff,
                 int(scales.stage) * (KS == 1 ? j >> 1 : j));
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int i = 0; i < NQW; ++i) {
        const Feed& f = codes[i < QXW ? 0 : NF - 1];
        load16_to_lds(f.window, slot + k * kStage / 2 + load_of(i) * 512, voff[i], int(f.stage) * (KS * j + k));
      }
  };
  auto advance = [&]() {
#pragma unroll
    for (int k = 0; k < NF; ++k) codes[k].advance(4 * KS);
    scales.advance(2 * KS);
  };

  // Operand addresses in a slot: lane l takes columns 32 (l / 32) .. + 31 of row
  // l % 32 of a block, two chunks. Its scale is a byte of the word of row l % 32:
  // block t of the wave's rows has byte t, counted from the wave's first row.
  const int l32 = lane & 31, h = lane >> 5;
  uint32_t fa[TM], fb[TN];
  const uint32_t ch0 = uint32_t(((2 * h) ^ ((l32 >> 2) & 3)) * 16);
#pragma unroll
  for (int m = 0; m < TM; ++m) fa[m] = uint32_t((wm * C::WM + m * 32 + l32) * RB) + ch0;
#pragma unroll
  for (int n = 0; n < TN; ++n) fb[n] = uint32_t((BM + wn * C::WN + n * 32 + l32) * RB) + ch0;
  const int ri = (i0 & 127) + wm * C::WM, ro = (row_o & 127) + wn * C::WN;
  const uint32_t sa = uint32_t(kScales + (ri >> 7) * 128 + l32 * 4);
  const uint32_t sb = uint32_t(kScales + 256 + (ro >> 7) * 128 + l32 * 4);
  const int shift_i = ((ri >> 5) & 3) * 8, shift_o = ((ro >> 5) & 3) * 8;
  i32x8_t frag[2][TM + TN];
  uint32_t sc[2][2];
  auto read_frags = [&](int f, const uint16_t* slot, int k) {
    const char* base = reinterpret_cast<const char*>(slot);
    sc[f][0] = *reinterpret_cast<const uint32_t*>(base + sa);
    sc[f][1] = *reinterpret_cast<const uint32_t*>(base + sb);
    base += k * kStage;
    auto operand = [&](uint32_t at) {
      const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(base + at);
      const i32x4_t hi = *reinterpret_cast<const i32x4_t*>(base + (at ^ 16u));
      return i32x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
#pragma unroll
    for (int m = 0; m < TM; ++m) frag[f][m] = operand(fa[m]);
#pragma unroll
    for (int n = 0; n < TN; ++n) frag[f][TM + n] = operand(fb[n]);
  };
  f32x16_t acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][n][r] = 0.0f;
  auto mfmas = [&](int f) {
    uint32_t now[TM + TN];
#pragma unroll
    for (int m = 0; m < TM; ++m) now[m] = sc[f][0] >> (shift_i + 8 * m);
#pragma unroll
    for (int n = 0; n < TN; ++n) now[TM + n] = sc[f][1] >> (shift_o + 8 * n);
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int n = 0; n < TN; ++n)
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(frag[f][m], frag[f][TM + n], acc[m][n],
                                                                    FI, FO, 0, int(now[m]), 0, int(now[TM + n]));
  };
  constexpr int NREAD = 2 * (TM + TN) + 2, NM = TM * TN;
  auto interleave = [&]() {
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // MFMA
      if (i * 3 < NREAD) __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);    // DS read
      if (i < NL) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);           // VMEM read
    }
  };
  constexpr int kWaitSlot = waitcnt_imm(2 * NL, 0);
#define FORGE_FP8_BARRIER(IMM)                \
  do {                                        \
    __builtin_amdgcn_sched_barrier(0);        \
    __builtin_amdgcn_s_waitcnt(IMM);          \
    asm volatile("" ::: "memory");            \
    __builtin_amdgcn_s_barrier();             \
    asm volatile("" ::: "memory");            \
    __builtin_amdgcn_sched_barrier(0);        \
  } while (0)
  // Slot j of a round of four.
  auto run_slot = [&](uint16_t* cur, const uint16_t* nxt, int j) {
    if constexpr (KS == 1) {
      if (j == 0) advance();
      load_slot(cur, j);                         // stage s + 4
      read_frags((j & 1) ^ 1, nxt, 0);
      mfmas(j & 1);
      interleave();
      FORGE_FP8_BARRIER(kWaitSlot);
    } else {
      read_frags(1, cur, 1);
      mfmas(0);
      FORGE_FP8_BARRIER(kWaitSlot);
      if (j == 0) advance();
      load_slot(cur, j);                         // of the next round
      read_frags(0, nxt, 0);
      mfmas(1);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (nk > 0) {
    load_slot(sl.s0, 0);
    load_slot(sl.s1, 1);
    load_slot(sl.s2, 2);
    load_slot(sl.s3, 3);
    FORGE_FP8_BARRIER(waitcnt_imm(KS == 1 ? 2 * NL : 3 * NL, 15));
    read_frags(0, sl.s0, 0);
    if constexpr (KS == 1) {
      // Slot 0 is refilled at once: every wave has read it by then.
      FORGE_FP8_BARRIER(waitcnt_imm(63, 0));
    }
    // Whole rounds of 4 slots: the accumulators keep their registers. Stages past
    // the last add products of zero codes and zero scale bytes: exactly +0.
    const int rounds = (nk + 4 * KS - 1) / (4 * KS);
    for (int r = 0; r < rounds; ++r) {
      run_slot(sl.s0, sl.s1, 0);
      run_slot(sl.s1, sl.s2, 1);
      run_slot(sl.s2, sl.s3, 2);
      run_slot(sl.s3, sl.s0, 3);
    }
  }
#undef FORGE_FP8_BARRIER
  uint16_t* ep = wave == 0 ? sl.s0 : wave == 1 ? sl.s1 : wave == 2 ? sl.s2 : sl.s3;
  epilogue<C, EPI_GRAD | EPI_BF16_OUT>(a, acc, a.W, a.S1, a.S2, i0, o0, wm, wn, lane,
                                       reinterpret_cast<float*>(ep));
}

template <class C, int FI, int FO>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(C::OCC, C::OCC)))
void fp8_block_kernel(WgradArgs a, Fp8BlockArgs x) {
  FORGE_DECLARE_SLOTS(fp8_block_slot<C>());
  int e, tm, tn;
  map_tile(blockIdx.x, a.num_tiles, a.tiles_m, a.tiles_n, a.group_m, e, tm, tn);
  fp8_block_tile<C, FI, FO>(a, x, tm, tn, ring);
}

// The persistent schedule of the bf16 kernel.
template <class CF, class CH, int FI, int FO>
__global__ __launch_bounds__(CF::THREADS) __attribute__((amdgpu_waves_per_eu(1, 1)))
void fp8_block_persistent_kernel(WgradArgs a, Fp8BlockArgs x) {
  static_assert(CF::THREADS == CH::THREADS && CF::BM == CH::BM && CF::BN == 2 * CH::BN,
                "half tiles must split the full tile's columns");
  FORGE_DECLARE_SLOTS(fp8_block_slot<CF>());
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
      fp8_block_tile<CF, FI, FO>(a, x, tm, tn, ring);
    else
      fp8_block_tile<CH, FI, FO>(a, x, tm, 2 * tn + half, ring);
    __syncthreads();
  }
}

// --------------------------------------------------------------------------
// product of few rows
// --------------------------------------------------------------------------
//
// Up to 16 MB rows of O (A of the entry point): 16 rows of I to a workgroup, whose W
// waves cut the contraction by its groups of 128 columns, one MFMA of 16 x 16 x 128
// for each 16 rows of O, and join their sums through LDS in the order of the
// waves. Bound by the bytes of I, which go straight into registers, U groups at a
// time: a lane holds 16 bytes of either half of a group, so that each load is
// 1 KB on end (a run of 8 columns stays one, and the order of runs does not
// matter to a sum that is joined in any case). Groups past the end read zeros.
// Launched for N of up to 12288, so that offsets within a batch (16 groups of 128 N bytes) are
// small. 1 x 4096 x 14336 takes 11.8 us, 5.0 TB/s of its 59 MB, of which the chip's caches may
// hold all; 4 x 12288 x 14336 31 us, 5.6 TB/s; 16 waves and U = 4 take 1.7 times as long where N is large.
template <int MB, int W, int U, int FI, int FO>
__global__ __launch_bounds__(64 * W) void fp8_block_rows_kernel(WgradArgs a, Fp8BlockArgs x) {
  __shared__ float join[W][MB * 4][64];
  const int lane = threadIdx.x & 63, r16 = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int N = a.d_in, M = a.d_out, n0 = blockIdx.x * 16;
  const int64_t groups = x.kp / 128, pitch_i = (N + 127) & ~127, pitch_o = (M + 127) & ~127;
  const int ni = min(n0 + r16, N - 1);
  const uint32_t vi = uint32_t((ni - n0) * 64 + q * 16), si = uint32_t((ni & ~127) + fp8_scale_place(ni & 127));
  uint32_t vo[MB], so[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) {
    const int m = min(16 * b + r16, M - 1);              // M <= 16 MB <= 128
    vo[b] = uint32_t(m * 64 + q * 16);
    so[b] = uint32_t(fp8_scale_place(m));
  }
  f32x4_t acc[MB];
#pragma unroll
  for (int b = 0; b < MB; ++b) acc[b] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const uint8_t* const ic = reinterpret_cast<const uint8_t*>(a.X);
  const uint8_t* const oc = reinterpret_cast<const uint8_t*>(a.dY);
  for (int64_t g = wave; g < groups; g += U * W) {
    const int64_t left = groups - g;
    const __amdgpu_buffer_rsrc_t wi = window(ic + (2 * g * N + n0) * 64, 2 * left * N * 64 - int64_t(n0) * 64);
    const __amdgpu_buffer_rsrc_t wo = window(oc + 2 * g * M * 64, 2 * left * M * 64);
    const __amdgpu_buffer_rsrc_t wsi = window(x.i_scales + g * pitch_i, left * pitch_i);
    const __amdgpu_buffer_rsrc_t wso = window(x.o_scales + g * pitch_o, left * pitch_o);
    u32x4_t fi[U][2], fo[U][MB][2];
    uint32_t ci[U], co[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        fi[u][h] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wi, int(vi), (2 * u * W + h) * N * 64, 0));
      ci[u] = __builtin_amdgcn_raw_buffer_load_b8(wsi, int(si), u * W * int(pitch_i), 0);
#pragma unroll
      for (int b = 0; b < MB; ++b) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          fo[u][b][h] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(wo, int(vo[b]), (2 * u * W + h) * M * 64, 0));
        co[u][b] = __builtin_amdgcn_raw_buffer_load_b8(wso, int(so[b]), u * W * int(pitch_o), 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);                   // all loads in flight
#pragma unroll
    for (int u = 0; u < U; ++u) {
      auto wide = [](const u32x4_t (&v)[2]) {
        return i32x8_t{int(v[0][0]), int(v[0][1]), int(v[0][2]), int(v[0][3]),
                       int(v[1][0]), int(v[1][1]), int(v[1][2]), int(v[1][3])};
      };
#pragma unroll
      for (int b = 0; b < MB; ++b)
        acc[b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(fo[u][b]), wide(fi[u]), acc[b], FO, FI,
                                                                  0, int(co[u][b]), 0, int(ci[u]));
    }
  }
  // Lane (q, r16) holds rows 4 q .. 4 q + 3 of O and row r16 of I.
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int k = 0; k < 4; ++k) join[wave][b * 4 + k][lane] = acc[b][k];
  __syncthreads();
  __bf16* const out = reinterpret_cast<__bf16*>(a.W);
  for (int e = threadIdx.x; e < MB * 256; e += 64 * W) {
    float s = join[0][e >> 6][e & 63];
#pragma unroll
    for (int w = 1; w < W; ++w) s += join[w][e >> 6][e & 63];
    const int m = (e >> 8) * 16 + ((e & 63) >> 4) * 4 + ((e >> 6) & 3), n = n0 + (e & 15);
    if (m < M && n < N) out[int64_t(m) * N + n] = __bf16(s);
  }
}

}  // namespace forge
