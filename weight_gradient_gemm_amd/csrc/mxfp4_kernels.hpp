// Microscaled 4-bit operands (OCP MX: 32 E2M1 codes and one E8M0 scale to a
// block) for gfx950: quantisation along rows and columns, and the product of
// two operands by v_mfma_scale_f32_32x32x64_f8f6f4, which takes both blocks'
// scales with their codes.
//
// An operand of R rows and padded length Kp holds codes [R][Kp / 2] and scales
// [Kp / 128][R][4]: the scales of 128 columns of one row are one 32-bit word,
// and the words of neighbouring rows are neighbours, so the matrix kernel's
// lanes (a row each) load them from whole lines and pick a byte in registers.
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
  int64_t row_pitch, col_pitch;    // bytes of a row of codes
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
        if (row < a.R && col < 2 * a.row_pitch) {
          uint8_t* const out = a.row_codes + row * a.row_pitch + col / 2;
          if constexpr (BF16) {
            const uint32_t w[4] = {raw[it][0], raw[it][1], raw[it][2], raw[it][3]};
            *reinterpret_cast<uint32_t*>(out) = codes8(w, s);
          } else {
            *reinterpret_cast<uint16_t*>(out) = uint16_t(codes4(__builtin_bit_cast(f32x4_t, raw[it]), s));
          }
          if (j % (32 / CPT) == 0)
            a.row_scales[((col >> 7) * a.R + row) * 4 + ((col >> 5) & 3)] = uint8_t(s);
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
        *reinterpret_cast<u32x4_t*>(a.col_codes + column * a.col_pitch + r0 / 2 + 16 * blk) = out;
        a.col_scales[(int64_t(tr) * a.C + column) * 4 + blk] = uint8_t(s);
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
// Mainloop: stages of 128 columns, rows of 64 bytes, straight from memory into
// a ring of 4 LDS slots, as the bf16 kernel (same bytes per stage and tile).
// 16-byte chunk c of row r is kept at chunk c ^ (r / 2 mod 4): the 8 rows that
// LDS serves at a time then fall on different banks. The scale words go from
// memory to registers, three stages ahead. Per stage, two k-steps of 64:
//   step 0: MFMAs; read step 1's operands from this slot.
//   wait for this wave's LDS reads and for its loads of the next stage; barrier.
//   step 1: request the scales of stage s + 3 and the codes of stage s + 4;
//   MFMAs; read step 0's operands from the next slot.
// Columns enter each element in ascending steps of 64, whatever the tile.
struct MxArgs {
  const uint8_t *i_scales, *o_scales;
  int64_t kp;
};

template <class C, int EPI>
__device__ __forceinline__ void mxfp4_tile(const WgradArgs& a, const MxArgs& x, int tile_m,
                                           int tile_n, const Slots& sl) {
  constexpr int BM = C::BM, BN = C::BN, TM = C::TM, TN = C::TN;
  constexpr int RB = 64;                                // bytes of a row in a stage
  constexpr int QX = BM * RB / 1024, QY = BN * RB / 1024;
  constexpr int NQW = (QX + QY) / C::WAVES;             // 1 KB loads per wave and stage
  constexpr int NSC = TM + TN;                          // scale words per lane and stage
  static_assert((QX + QY) % C::WAVES == 0, "stage loads split evenly over the waves");
  static_assert(RB * (BM + BN) <= C::STAGE * 2, "stage exceeds a slot");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % C::WAVES_M, wn = wave / C::WAVES_M;
  const int d_in = a.d_in, d_out = a.d_out;
  const int i0 = tile_m * BM, o0 = tile_n * BN;
  const int pitch = int(x.kp / 2);
  const int nk = int(x.kp / 128);

  // Loads: instruction q covers 16 rows of I (q < QX) or O; lane t fills row
  // t / 4, physical chunk t % 4.
  uint32_t voff[NQW];
  int soff[NQW];
#pragma unroll
  for (int i = 0; i < NQW; ++i) {
    const int q = wave * NQW + i;
    const bool isx = q < QX;
    const int row0 = (isx ? q : q - QX) * 16, lrow = lane >> 2;
    const int ch = (lane & 3) ^ ((lrow >> 1) & 3);
    voff[i] = (isx ? i0 : o0) + row0 + lrow < (isx ? d_in : d_out) ? uint32_t(lrow * pitch + 16 * ch) : kOOB;
    soff[i] = row0 * pitch;
  }
  int g_stage = 0;
  const uint8_t* gi = reinterpret_cast<const uint8_t*>(a.X) + int64_t(i0) * pitch;
  const uint8_t* go = reinterpret_cast<const uint8_t*>(a.dY) + int64_t(o0) * pitch;
  auto load_stage = [&](uint16_t* slot) {
    // Rows past the edge have an out-of-window offset, so the window only has
    // to reach the tile's last row (256 pitch < 2^31), and nothing past the
    // last stage, which loads zeros. No branches: the compiler would sink
    // MFMAs below them, out of their stage.
    const uint32_t bytes = g_stage < nk ? kOOB - 1u : 0u;
    const __amdgpu_buffer_rsrc_t ri = window32(gi, bytes), ro = window32(go, bytes);
    gi += RB;
    go += RB;
    ++g_stage;
#pragma unroll
    for (int i = 0; i < NQW; ++i) {
      const int q = wave * NQW + i;
      load16_to_lds(q < QX ? ri : ro, slot + q * 512, voff[i], soff[i]);
    }
  };

  // Scale words: the four blocks of this lane's row in a stage; the lane's half
  // h of the wave takes blocks 2 kk + h, so the word is shifted by h bytes once
  // and step kk picks byte 2 kk.
  const int l32 = lane & 31, h = lane >> 5;
  uint32_t sv[NSC];
#pragma unroll
  for (int m = 0; m < TM; ++m) sv[m] = uint32_t(i0 + wm * C::WM + m * 32 + l32) * 4u;
#pragma unroll
  for (int n = 0; n < TN; ++n) sv[TM + n] = uint32_t(o0 + wn * C::WN + n * 32 + l32) * 4u;
  int s_stage = 0;
  const uint8_t *si = x.i_scales, *so = x.o_scales;
  uint32_t sc[4][NSC];
  auto load_scales = [&](int k) {
    const __amdgpu_buffer_rsrc_t ri = window32(si, s_stage < nk ? uint32_t(d_in) * 4u : 0u);
    const __amdgpu_buffer_rsrc_t ro = window32(so, s_stage < nk ? uint32_t(d_out) * 4u : 0u);
    si += int64_t(d_in) * 4;
    so += int64_t(d_out) * 4;
    ++s_stage;
#pragma unroll
    for (int t = 0; t < NSC; ++t)
      sc[k][t] = __builtin_amdgcn_raw_buffer_load_b32(t < TM ? ri : ro, int(sv[t]), 0, 0);
  };

  // Operand addresses in a slot for step 0; step 1 is 32 bytes away (chunk
  // 2 + h, and the swizzle is an exclusive or).
  uint32_t fa[TM], fb[TN];
  const uint32_t ch0 = uint32_t((h ^ ((l32 >> 1) & 3)) * 16);
#pragma unroll
  for (int m = 0; m < TM; ++m) fa[m] = uint32_t((wm * C::WM + m * 32 + l32) * RB) + ch0;
#pragma unroll
  for (int n = 0; n < TN; ++n) fb[n] = uint32_t((BM + wn * C::WN + n * 32 + l32) * RB) + ch0;
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
  f32x16_t acc[TM][TN];
#pragma unroll
  for (int m = 0; m < TM; ++m)
#pragma unroll
    for (int n = 0; n < TN; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[m][n][r] = 0.0f;
  auto wide = [](const i32x4_t& v) { return i32x8_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; };
  uint32_t now[NSC];
  auto shift_scales = [&](int k) {
#pragma unroll
    for (int t = 0; t < NSC; ++t) now[t] = sc[k][t] >> (8 * h);
  };
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
  auto interleave = [&](int loads) {
#pragma unroll
    for (int i = 0; i < TM * TN; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                       // MFMA
      if (i < TM + TN) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);      // DS read
      if (i < loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);        // VMEM read
    }
  };
  // Requests in order: codes 0, codes 1, scales 0, codes 2, scales 1, codes 3,
  // scales 2, then per stage s: scales s + 3, codes s + 4. At stage s the codes
  // of stage s + 1 have landed once at most two stages' requests are left.
  constexpr int kWaitMid = waitcnt_imm(2 * (NQW + NSC), 0);
  constexpr int kWaitFirst = waitcnt_imm(3 * (NQW + NSC), 15);
#define FORGE_MX_BARRIER(IMM)                 \
  do {                                        \
    __builtin_amdgcn_sched_barrier(0);        \
    __builtin_amdgcn_s_waitcnt(IMM);          \
    asm volatile("" ::: "memory");            \
    __builtin_amdgcn_s_barrier();             \
    asm volatile("" ::: "memory");            \
    __builtin_amdgcn_sched_barrier(0);        \
  } while (0)
  auto stage = [&](uint16_t* cur, uint16_t* nxt, int k) {
    shift_scales(k);
    read_frags(1, cur, 1);
    mfmas0();
    interleave(0);
    FORGE_MX_BARRIER(kWaitMid);
    load_scales((k + 3) & 3);
    load_stage(cur);                             // stage s + 4 into the freed slot
    read_frags(0, nxt, 0);
    mfmas1();
    interleave(NQW + NSC);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (nk > 0) {
    load_stage(sl.s0);
    load_stage(sl.s1);
    load_scales(0);
    load_stage(sl.s2);
    load_scales(1);
    load_stage(sl.s3);
    load_scales(2);
    FORGE_MX_BARRIER(kWaitFirst);
    read_frags(0, sl.s0, 0);
    // Whole rounds of 4 stages: the accumulators keep their registers. Stages
    // past the last add products of zero codes and zero scale bytes: exactly +0.
    const int rounds = (nk + 3) / 4;
    for (int r = 0; r < rounds; ++r) {
      stage(sl.s0, sl.s1, 0);
      stage(sl.s1, sl.s2, 1);
      stage(sl.s2, sl.s3, 2);
      stage(sl.s3, sl.s0, 3);
    }
  }
#undef FORGE_MX_BARRIER
  uint16_t* ep = wave == 0 ? sl.s0 : wave == 1 ? sl.s1 : wave == 2 ? sl.s2 : sl.s3;
  epilogue<C, EPI>(a, acc, a.W, a.S1, a.S2, i0, o0, wm, wn, lane, reinterpret_cast<float*>(ep));
}

template <class C, int EPI>
__global__ __launch_bounds__(C::THREADS) __attribute__((amdgpu_waves_per_eu(C::OCC, C::OCC)))
void mxfp4_kernel(WgradArgs a, MxArgs x) {
  FORGE_DECLARE_SLOTS(C::STAGE);
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
  FORGE_DECLARE_SLOTS(CF::STAGE);
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
