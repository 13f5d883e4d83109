// fp8adam_layer_product.h -- the forward products of the layer operators, instantiated
// for each pair of formats in fp8adam_layer_product_*.hip.
//
// Both operands are codes with one power-of-two scale per row and 128 columns, and
// gfx950's scaled matrix instruction multiplies 16 x 128 by 128 x 16 codes with a scale for
// every row and 32 columns: one instruction takes exactly one block of 16 rows of each, with
// its scales.  (As 32 x 64 by 64 x 32 it reached 8% less on the whole card.)
//
// The instruction sums eight consecutive products at a time, each cut (towards zero) at 2^-13 of the
// power of two of the largest product's exponents, and adds these sums to 32 bits (measured with
// one large and one small product in every place; the unscaled FP8 instructions do the
// same).  Sums of normal numbers are off by 1.5e-5 of the sums' rms, and where a hundredth of the columns is eight times as
// large by 2.6e-5: a thirtieth or a twentieth of half a step of fp16, less than a hundredth of one of bf16, so it
// serves outputs of 8 and 16 bits.  (Where large products cancel, what is left may be off by more than that of itself.)
// For outputs of 32 bits (WIDE), for few tokens, where the weights' bytes are what
// counts, whether or not something is kept, and where the caller asks for it, both operands are widened to
// bf16 times their scales, which is exact (but for what lies below 2^-133, under scales below 2^-124
// of E4M3 and 2^-117 of E5M2), and multiplied by the bf16 instruction, which adds every product in 32
// bits (4096 tokens x 4096 x 2 * 11008, both kept: 630 us in place of 329; 2048 x 768 x 2 * 2048: 21 and 17).
//
// The order of the products in one instruction is free, so a lane may take any 32 columns of
// its row as long as both operands take the same: here two of a row's 16-byte pieces.
#pragma once

#include "fp8adam_layer.h"

namespace fp8adam_layer {

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kProdThreads = 512;
constexpr int kWRows = 256;       // rows of weights in a tile; gated: 128 of each projection
constexpr int kScaleChunk = 56;   // blocks whose scales are in shared memory at a time
constexpr int kScaleLd = 60;      // bytes between rows of them: 15 dwords, which spreads 16 rows over the banks

__device__ __forceinline__ v8i frag(const uint8_t* row, int p0, int p1) {
  const vu4 a = *reinterpret_cast<const vu4*>(row + p0), b = *reinterpret_cast<const vu4*>(row + p1);
  return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// 32 codes times 2^(scale - 127) in bf16, as operands of four bf16 instructions.
template <int FMT>
__device__ __forceinline__ void widen(const v8i& c, uint32_t scale, v8bf (&out)[4]) {
  const float s = __uint_as_float(scale << 23);
#pragma unroll
  for (int q = 0; q < 4; q++) {
    vu4 w;
#pragma unroll
    for (int e = 0; e < 2; e++) {
      const uint32_t d = (uint32_t)c[2 * q + e];
      if constexpr (FMT == 0) {
        w[2 * e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, s, false));
        w[2 * e + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d, s, true));
      } else {
        w[2 * e] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(d, s, false));
        w[2 * e + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(d, s, true));
      }
    }
    out[q] = __builtin_bit_cast(v8bf, w);
  }
}

__device__ __forceinline__ vf4_t mfma_wide(const v8bf (&w)[4], const v8bf (&x)[4], vf4_t c) {
#pragma unroll
  for (int q = 0; q < 4; q++) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[q], x[q], c, 0, 0, 0);
  return c;
}

// The E8M0 bytes of up to kScaleChunk blocks of a row, from entry i of the scales on, into shared memory.  All
// loads go out together: one after the other they took a sixth of a product of 4096 columns.
__device__ __forceinline__ void put_scales(const void* scales, bool f32, int64_t i, int n, uint8_t* to) {
  constexpr int kGroups = kScaleChunk / 4;
  uint32_t w[kGroups];
  if (f32) {
    const float* p = static_cast<const float*>(scales) + i;
    vu4 v[kGroups];
#pragma unroll
    for (int u = 0; u < kGroups; u++) {
      if (4 * u + 4 <= n) {
        v[u] = ld_global<vu4_any>(p + 4 * u);
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++) v[u][j] = 4 * u + j < n ? ld_global<uint32_t>(p + 4 * u + j) : 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < kGroups; u++)
      w[u] = (v[u].x >> 23 & 0xFFu) | (v[u].y >> 23 & 0xFFu) << 8 | (v[u].z >> 23 & 0xFFu) << 16 | v[u].w >> 23 << 24;
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(scales) + i;  // whole dwords
#pragma unroll
    for (int u = 0; u < kGroups; u++) w[u] = 4 * u < n ? ld_global<uint32_t>(p + 4 * u) : 0u;
  }
#pragma unroll
  for (int u = 0; u < kGroups; u++)
    if (4 * u < n) *reinterpret_cast<uint32_t*>(to + 4 * u) = w[u];
}

// A tile of 256 weight rows by TT tokens: eight waves, WN along the rows, each 256/WN rows by
// TT/WT tokens in products of 16 x 128 by 128 x 16.
//
// A block of 128 columns takes two phases: the first multiplies the first half of each wave's
// rows (gated: the gate's) by its tokens, the second the second half (the up projection's) by the
// same, which stay in registers.  Rows of 128 bytes (whole cache lines: half lines load 25% slower) go straight
// into shared memory, where each of the three parts, tokens and both halves of the weights, has
// two places: a phase after all waves have read a part, the block after the next is loaded into
// its place.
//
// The two waves of a SIMD take turns: while waves 0 .. 3 multiply, waves 4 .. 7 read their
// operands from shared memory and the other way round, with a barrier at each turn, so
// that the matrix cores need not wait for shared memory.  (Phase p is read by the first waves in
// turn 2p and by the others in 2p + 1; loads into what it read go out in turns 2p + 2 and 2p + 3, and
// have arrived, each wave's own before a barrier, when phase p + 4 is read from turn 2p + 8 on.)
//
// A row's eight 16-byte pieces are stored in the order piece ^ (row / 2 & 7), by giving each lane
// of the load another source, so that 16 rows of a fragment lie on all banks.
//
// The sums then go through shared memory, 32 tokens of each wave at a time, into rows of
// 128 columns for 16 lanes each: bias, activation, product, residual and the blocks' amax
// are made there, and whole lines are stored.
//
// Measured (E4M3, SiLU, both projections kept): 4096 tokens x 4096 x 2 * 11008 in 330 us, 2240 TFLOP/s;
// 8192 x 4096 x 4096 with a residual in 135 us, 2040; 8192^3 without in 2.8 PFLOP/s, where the
// card's power is what bounds it (a loop of the instruction alone reaches 3.9 to 4.5).  What is lost
// against that is each tile's start, 9K cycles until its first operands and scales are there, and its end,
// 7K to 12K cycles of activation and rounding, in which its CU does not multiply.
template <int XF, int WF, bool GATED, int TT, bool WIDE>
__global__ __launch_bounds__(kProdThreads, 2) void k_product(const ProductArgs a) {
  constexpr int WN = TT == 64 ? 4 : 2, WT = 8 / WN;
  constexpr int kRowsW = kWRows / WN, kTokW = TT / WT;  // of a wave
  constexpr int kI = kRowsW / 16, kJ = kTokW / 16;      // products of a wave
  constexpr int kXBytes = TT * 128, kWBytes = kWRows / 2 * 128;
  constexpr int kAtW = 2 * kXBytes;                     // the weights' places: first half, second half, twice
  constexpr int kRoom = kAtW + 4 * kWBytes > WT * 32768 ? kAtW + 4 * kWBytes : WT * 32768;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRoom + (kWRows + TT) * kScaleLd];
  uint8_t* const sc = lds + kRoom;

  // tiles in bands of four along the rows, an eighth of them on each XCD, so that what one XCD works
  // on shares weights and tokens in its L2
  const int total = a.tiles_n * a.tiles_t;
  const int per = (total + 7) >> 3;
  const int pos = (int)(blockIdx.x & 7u) * per + (int)(blockIdx.x >> 3);
  if (pos >= total || (int)(blockIdx.x >> 3) >= per) return;
  const int band = pos / (4 * a.tiles_t), in = pos - band * 4 * a.tiles_t, width = min(4, a.tiles_n - 4 * band);
  const int tile_n = 4 * band + in % width;
  const int64_t t0 = (int64_t)(in / width) * TT;
  const int n0 = tile_n * (GATED ? 128 : 256);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / WT, wt = wave % WT;
  const int nk = (a.cols + 127) >> 7;

  // The weight row, in the tile, of row q (of 128) of half `part`.
  auto row_of = [](int part, int q) { return GATED ? q : kRowsW * (q / (kRowsW / 2)) + kRowsW / 2 * part + q % (kRowsW / 2); };

  // loads: 8 rows of 128 bytes per wave and instruction
  const int lrow = lane >> 3, piece = (lane & 7) ^ (4 * (wave & 1) + (lane >> 4));
  const int64_t vt = min((int64_t)TT, a.tokens - t0);
  const int64_t vn = min((int64_t)(GATED ? 128 : 256), (int64_t)a.rows - n0);
  const int64_t ldw = a.w[0].ld, ldu = GATED ? a.w[1].ld : ldw;
  uint32_t ow[2][2], ox[TT / 64];
#pragma unroll
  for (int part = 0; part < 2; part++)
#pragma unroll
    for (int i = 0; i < 2; i++)
      ow[part][i] = (uint32_t)(row_of(part, 8 * (wave + 8 * i)) + lrow) * (uint32_t)(part ? ldu : ldw) + 16u * piece;
#pragma unroll
  for (int i = 0; i < TT / 64; i++) ox[i] = (uint32_t)(8 * (wave + 8 * i) + lrow) * (uint32_t)a.x.ld + 16u * piece;
  const uint8_t* const xbase = a.x.codes + t0 * a.x.ld;
  const uint8_t* const wbase = a.w[0].codes + (int64_t)n0 * ldw;
  const uint8_t* const ubase = GATED ? a.w[1].codes + (int64_t)n0 * ldu : wbase;
  // What phase p needs that the one before it does not; behind the last zeros (a resource of no bytes), so
  // that every phase has the same number of loads to wait for.
  auto load = [&](int place, int part, int k) {
    const bool there = k < nk;
    if (part == 0) {
      const vu4 rx = rsrc4(xbase, there ? vt * a.x.ld : 0);
#pragma unroll
      for (int i = 0; i < TT / 64; i++) load_lds(rx, lds + place * kXBytes + 1024 * (wave + 8 * i), ox[i], 128u * k);
    }
    const vu4 rw = rsrc4(part ? ubase : wbase, there ? vn * (part ? ldu : ldw) : 0);
#pragma unroll
    for (int i = 0; i < 2; i++) load_lds(rw, lds + kAtW + (2 * place + part) * kWBytes + 1024 * (wave + 8 * i), ow[part][i], 128u * k);
  };
  constexpr int kLoads = TT / 64 + 4;  // of two phases

  vf4_t acc[kI][kJ];
#pragma unroll
  for (int i = 0; i < kI; i++)
#pragma unroll
    for (int j = 0; j < kJ; j++) acc[i][j] = vf4_t{0, 0, 0, 0};
  const int g = lane >> 4, fr = lane & 15, turned = fr >> 1;
  const int p0 = 16 * (g ^ turned), p1 = 16 * ((g + 4) ^ turned);
  const int wrow = kRowsW / 2 * wn + fr, xrow = kTokW * wt + fr;
  int wsc[2][kI / 2], xsc[kJ];

  load(0, 0, 0);
  load(0, 1, 0);
  load(1, 0, 1);
  for (int kc = 0; kc < nk; kc += kScaleChunk) {
    if (kc > 0) __syncthreads();  // the scales before have been read
    const int here = min(kScaleChunk, nk - kc);
    for (int q = threadIdx.x; q < kWRows + TT; q += kProdThreads) {
      const bool is_x = q >= kWRows;
      const int part = is_x ? 0 : q >> 7;
      const int64_t row = is_x ? t0 + (q - kWRows) : n0 + row_of(part, q & 127);
      const bool there = is_x ? row < a.tokens : row < a.rows, up = GATED && part;
      const void* s = is_x ? a.x.scales : up ? a.w[1].scales : a.w[0].scales;
      const int64_t ld = is_x ? a.x.ld_scale : up ? a.w[1].ld_scale : a.w[0].ld_scale;
      put_scales(s, is_x ? a.x.f32 : a.w[0].f32, (there ? row : is_x ? t0 : n0) * ld + kc, here, sc + q * kScaleLd);
    }
    stage_barrier<kLoads>();  // the first phase's operands are there, and the scales
    if (wave >= 4) bare_barrier();
    const int end = min(nk, kc + kScaleChunk);
    for (int k = kc; k < end; k += 4) {
      v8i x[kJ];
      auto one = [&](auto which) {
        constexpr int S = decltype(which)::value, B = S >> 1, part = S & 1;  // block and half
        if (k + B >= end) return;
        load(part ? B & 1 : (B + 1) & 1, part ^ 1, k + B + 1 + part);
        if constexpr (S == 0) {
#pragma unroll
          for (int i = 0; i < kI; i++)
            wsc[i / (kI / 2)][i % (kI / 2)] = *reinterpret_cast<const int*>(sc + (128 * (i / (kI / 2)) + wrow + 16 * (i % (kI / 2))) * kScaleLd + (k - kc));
#pragma unroll
          for (int j = 0; j < kJ; j++) xsc[j] = *reinterpret_cast<const int*>(sc + (kWRows + xrow + 16 * j) * kScaleLd + (k - kc));
        }
        if constexpr (part == 0) {
#pragma unroll
          for (int j = 0; j < kJ; j++) x[j] = frag(lds + (B & 1) * kXBytes + (xrow + 16 * j) * 128, p0, p1);
        }
        v8i w[kI / 2];
#pragma unroll
        for (int i = 0; i < kI / 2; i++) w[i] = frag(lds + kAtW + (2 * (B & 1) + part) * kWBytes + (wrow + 16 * i) * 128, p0, p1);
        stage_barrier<kLoads>();  // the next phase's operands are there
        __builtin_amdgcn_s_setprio(1);
        if constexpr (WIDE) {
          v8bf xw[kJ][4];
#pragma unroll
          for (int j = 0; j < kJ; j++) widen<XF>(x[j], (uint32_t)xsc[j] >> (8 * B) & 0xFFu, xw[j]);
#pragma unroll
          for (int i = 0; i < kI / 2; i++) {
            v8bf ww[4];
            widen<WF>(w[i], (uint32_t)wsc[part][i] >> (8 * B) & 0xFFu, ww);
#pragma unroll
            for (int j = 0; j < kJ; j++) acc[part * kI / 2 + i][j] = mfma_wide(ww, xw[j], acc[part * kI / 2 + i][j]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < kI / 2; i++)
#pragma unroll
            for (int j = 0; j < kJ; j++)  // rows of D are A's rows (weights), columns B's (tokens)
              acc[part * kI / 2 + i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                  w[i], x[j], acc[part * kI / 2 + i][j], WF, XF, B, wsc[part][i], B, xsc[j]);
        }
        // (keeps the products on this side of the barrier: they would be moved to where the sums are used next)
#pragma unroll
        for (int i = 0; i < kI / 2; i++)
#pragma unroll
          for (int j = 0; j < kJ; j++) asm volatile("" : "+v"(acc[part * kI / 2 + i][j]));
        __builtin_amdgcn_s_setprio(0);
        bare_barrier();
      };
      one(std::integral_constant<int, 0>{});
      one(std::integral_constant<int, 1>{});
      one(std::integral_constant<int, 2>{});
      one(std::integral_constant<int, 3>{});
      one(std::integral_constant<int, 4>{});
      one(std::integral_constant<int, 5>{});
      one(std::integral_constant<int, 6>{});
      one(std::integral_constant<int, 7>{});
    }
    if (wave < 4) bare_barrier();
  }
  wait_loads();

  // (the arguments are read again from where the launch left them: kept in scalar registers through the loop
  // they would not leave it enough)
  const auto* e = (const __attribute__((address_space(4))) ProductArgs*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(e));
  auto out_of = [](const __attribute__((address_space(4))) Out8& o) { return Out8{o.codes, o.scales, o.ld, o.ld_scale, o.format}; };
  const Out8 keep0 = out_of(e->keep[0]), keep1 = out_of(e->keep[1]), y8 = out_of(e->y8);
  const void *bias = e->bias, *res = e->res;
  void* const y = e->y;
  const int64_t tokens = e->tokens, res_ld = e->res_ld, y_ld = e->y_ld;
  const int rows = e->rows, act = e->act, bias_dt = e->bias_dt, res_dt = e->res_dt, y_dt = e->y_dt;

  // the sums: 32 tokens of every wave along the tokens, 32 KB for each of them, 256 columns a token whose
  // 16-byte units lie in the order unit ^ (token & 15)
  const int hw = threadIdx.x >> 4, hl = threadIdx.x & 15;
  // Each 16 lanes take kBatch rows of 128 at a time, step by step: one after the other they took twice as long,
  // waiting for every branch and every read.  FULL: the whole tile is there.
  constexpr int kRowsOut = 32 * WT * (GATED ? 1 : 2), kBatch = kRowsOut / 32 < 4 ? kRowsOut / 32 : 4;
  auto finish = [&](int j, auto which) __attribute__((always_inline)) {
    constexpr bool FULL = decltype(which)::value;
#pragma unroll 1
    for (int q = hw; q < kRowsOut; q += 32 * kBatch) {
      float z[kBatch][8];
      int64_t t[kBatch], block[kBatch];
      int n[kBatch], left[kBatch];
      bool there[kBatch];
      auto sums = [&](int b, int tok, int col, float (&v)[8]) __attribute__((always_inline)) {  // zeros behind the last row of weights
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const vf4_t s = *reinterpret_cast<const vf4_t*>(lds + tok * 1024 + 16 * ((col / 4 + 2 * hl + h) ^ (tok & 15)));
#pragma unroll
          for (int c = 0; c < 4; c++) v[4 * h + c] = FULL || 4 * h + c < left[b] ? s[c] : 0.0f;
        }
      };
      auto tok_of = [&](int b) { return GATED ? q + 32 * b : (q + 32 * b) >> 1; };
#pragma unroll
      for (int b = 0; b < kBatch; b++) {
        const int tok = tok_of(b), blk = GATED ? 0 : q & 1;
        t[b] = t0 + kTokW * (tok >> 5) + 32 * j + (tok & 31);
        n[b] = n0 + 128 * blk + 8 * hl;
        left[b] = FULL ? 8 : rows - n[b];
        block[b] = (n0 >> 7) + blk;
        there[b] = FULL || (t[b] < tokens && n0 + 128 * blk < rows);  // the same in the 16 lanes
        if (!FULL && !there[b]) left[b] = 0;
        sums(b, tok, 128 * blk, z[b]);
      }
      if (!GATED && bias) {
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
          float v[8];
          ld8(bias_dt, bias, n[b], left[b], v);
#pragma unroll
          for (int c = 0; c < 8; c++) z[b][c] += v[c];
        }
      }
      if (keep0.codes) put_blocks(keep0, t, block, there, hl, z);
      act_all(act, z);
      if constexpr (GATED) {
        float u[kBatch][8];
#pragma unroll
        for (int b = 0; b < kBatch; b++) sums(b, tok_of(b), 128, u[b]);
        if (keep1.codes) put_blocks(keep1, t, block, there, hl, u);
#pragma unroll
        for (int b = 0; b < kBatch; b++)
#pragma unroll
          for (int c = 0; c < 8; c++) z[b][c] *= u[b][c];
      } else if (res) {
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
          float v[8];
          ld8(res_dt, res, t[b] * res_ld + n[b], left[b], v);
#pragma unroll
          for (int c = 0; c < 8; c++) z[b][c] += v[c];
        }
      }
      if (y) {
#pragma unroll
        for (int b = 0; b < kBatch; b++) st8(y_dt, y, t[b] * y_ld + n[b], left[b], z[b]);
      }
      if (y8.codes) put_blocks(y8, t, block, there, hl, z);
    }
  };
  auto tokens32 = [&](auto which) __attribute__((always_inline)) {
    constexpr int J = decltype(which)::value;
    if constexpr (J < kTokW / 32) {
      stage_barrier<63>();
#pragma unroll
      for (int i = 0; i < kI; i++)
#pragma unroll
        for (int c = 0; c < 2; c++) {
          const int part = i / (kI / 2), q = kRowsW / 2 * wn + 16 * (i % (kI / 2));
          const int unit = ((GATED ? 128 * part : 0) + row_of(part, q)) / 4 + g;
          *reinterpret_cast<vf4_t*>(lds + (32 * wt + 16 * c + fr) * 1024 + 16 * (unit ^ fr)) = acc[i][2 * J + c];
        }
      stage_barrier<63>();
      if (n0 + (GATED ? 128 : 256) <= rows && t0 + TT <= tokens) finish(J, std::true_type{});
      else finish(J, std::false_type{});
    }
  };
  tokens32(std::integral_constant<int, 0>{});
  tokens32(std::integral_constant<int, 1>{});
}

// Few tokens, nothing kept: bound by the weights' bytes.  A work-group takes 16 rows of
// weights (gated: 16 of each projection); in every chunk of the blocks of 128 columns each of its
// waves takes four (with more than 16 tokens two), weights straight into registers, and the
// waves' sums meet in shared memory at the end.  Four waves, of which three work-groups share a CU
// and load while others multiply, or eight where there are too few work-groups for that.
// PACK: up to 4 tokens in 16 or 32 bits on whole dwords.  The work-group turns a chunk of them into codes
// in shared memory, 16 lanes a block, while its weights are on their way (the first work-group stores
// them too).  (One launch less, 5 us; packed by each wave into its own fragments, 15 of whose 16
// lanes have nothing to do for one token, one token x 4096 x 2 * 11008 took 36 us.  Every work-group
// packs every token, so with more of them a launch of its own is faster.)
// XDT: the type of x that the kernel packs, or kCodes where x is packed already.
using fp8adam_list::kCodes;
template <int XF, int WF, bool GATED, int NT, int XDT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, WAVES == 4 ? 3 : 2) void k_product_few(const ProductArgs a) {
  constexpr int G = GATED ? 2 : 1;
  constexpr bool PACK = XDT != kCodes;
  constexpr int kAhead = NT > 1 ? 2 : 4;        // blocks of a wave in a chunk
  constexpr int kBlocks = WAVES * kAhead;       // of a chunk
  constexpr int kLd = kBlocks * 128 + 16;       // bytes between tokens in shared memory: spread over the banks
  __shared__ vf4_t red[WAVES][G][NT][64];
  __shared__ __attribute__((aligned(16))) uint8_t packed[PACK ? 16 * kLd : 16];
  __shared__ uint8_t bytes[PACK ? 16 : 1][kBlocks];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, fr = lane & 15;
  const int n0 = blockIdx.x * 16;
  const int nk = (a.cols + 127) >> 7;
  const int64_t vn = min((int64_t)16, (int64_t)a.rows - n0);
  Rsrc rw[G];
#pragma unroll
  for (int p = 0; p < G; p++) rw[p] = rsrc(a.w[p].codes + (int64_t)n0 * a.w[p].ld, vn * a.w[p].ld);
  const Rsrc rx = PACK ? rsrc(a.xin, dtype_bytes(PACK ? XDT : 0) * ((a.tokens - 1) * a.xin_ld + a.cols))
                       : rsrc(a.x.codes, a.tokens * a.x.ld);
  const int64_t wrow = n0 + min(fr, (int)vn - 1);

  vf4_t acc[G][NT];
#pragma unroll
  for (int p = 0; p < G; p++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[p][j] = vf4_t{0, 0, 0, 0};

  auto two = [](Rsrc r, uint32_t o) {
    const vu4 a = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0), b = __builtin_amdgcn_raw_buffer_load_b128(r, o + 64, 0, 0);
    return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
  };
  // x to 8 bits: item i is block i % kBlocks of token i / kBlocks, for 16 lanes
  constexpr int kEl = PACK ? (int)dtype_bytes(XDT) : 2;
  const int items = (int)a.tokens * kBlocks, hl = threadIdx.x & 15;
  struct Raw8 {
    vu4 x[kEl / 2];
  };
  auto load_x = [&](int kc, int i) __attribute__((always_inline)) {
    const int k = kc + i % kBlocks;
    Raw8 r;
    const uint32_t o = i < items && k < nk ? (uint32_t)(kEl * (i / kBlocks * a.xin_ld + 128 * k + 8 * hl)) : 0x7FFFFF00u;
#pragma unroll
    for (int q = 0; q < kEl / 2; q++) r.x[q] = __builtin_amdgcn_raw_buffer_load_b128(rx, o + 16 * q, 0, 0);
    return r;
  };
  auto pack_x = [&](int kc, int i, const Raw8& r) __attribute__((always_inline)) {
    const int tok = i / kBlocks, blk = i % kBlocks, k = kc + blk;
    float lo[4], hi[4];
    constexpr int DT = PACK ? XDT : FP8ADAM_BF16;
    if constexpr (DT == FP8ADAM_F32) {
      unpack4<DT>(Raw4<DT>{r.x[0]}, lo);
      unpack4<DT>(Raw4<DT>{r.x[kEl / 2 - 1]}, hi);
    } else {
      unpack4<DT>(Raw4<DT>{vu2{r.x[0].x, r.x[0].y}}, lo);
      unpack4<DT>(Raw4<DT>{vu2{r.x[0].z, r.x[0].w}}, hi);
    }
    uint32_t am = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {  // (a load behind the row's end gives the next row's values)
      lo[j] = 128 * k + 8 * hl + j < a.cols ? lo[j] : 0.0f;
      hi[j] = 128 * k + 8 * hl + 4 + j < a.cols ? hi[j] : 0.0f;
      am = max(am, max(abs_bits(lo[j]), abs_bits(hi[j])));
    }
    am = row_max(am);
    const uint32_t byte = scale_byte<XF>(am);
    const float s = __uint_as_float(byte << 23);
    const bool odd = nonfinite_amax(am);
    vu2 c{codes4_pow2<XF>(lo, s, false), codes4_pow2<XF>(hi, s, false)};
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(odd) != 0, 0)) {
      if (odd) c = vu2{codes4_pow2<XF>(lo, 1.0f, true), codes4_pow2<XF>(hi, 1.0f, true)};
    }
    if (i >= items) return;
    *reinterpret_cast<vu2*>(packed + tok * kLd + 128 * blk + 8 * hl) = c;
    if (hl == 0) bytes[tok][blk] = (uint8_t)byte;
    if (blockIdx.x == 0 && k < nk) {
      st_global<vu2>(a.x8.codes + tok * a.x8.ld + 128 * (int64_t)k + 8 * hl, c);
      if (hl == 0) st_global<uint8_t>(a.x8.scales + tok * a.x8.ld_scale + k, (uint8_t)byte);
    }
  };

  constexpr int kGroups = WAVES * 4, kItems = PACK ? kFewPackTokens * kBlocks / kGroups : 1;  // of 16 lanes, at most
  const int first = threadIdx.x >> 4;
  struct Chunk {
    Raw8 raw[kItems];
    v8i x[kAhead][NT], w[kAhead][G];
    uint32_t xs[kAhead][NT], ws[kAhead][G];
  };
  // x first: loads come back in their order, and x is packed while the weights are on their way
  auto load = [&](Chunk& c, int kc) __attribute__((always_inline)) {
    if constexpr (PACK) {
#pragma unroll
      for (int i = 0; i < kItems; i++) c.raw[i] = load_x(kc, first + kGroups * i);
    } else {
#pragma unroll
      for (int u = 0; u < kAhead; u++) {
        const int k = kc + wave + WAVES * u;
#pragma unroll
        for (int j = 0; j < NT; j++) {
          const int64_t t = 16 * j + fr;  // behind the last token or block: outside the resource, zeros
          c.x[u][j] = two(rx, t < a.tokens && k < nk ? (uint32_t)t * (uint32_t)a.x.ld + 128u * k + 16u * g : 0x7FFFFF00u);
          c.xs[u][j] = __float_as_uint(scale_at(a.x.scales, min(t, a.tokens - 1) * a.x.ld_scale + min(k, nk - 1), a.x.f32)) >> 23;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
      const int k = kc + wave + WAVES * u;
#pragma unroll
      for (int p = 0; p < G; p++) {
        c.w[u][p] = two(rw[p], k < nk ? (uint32_t)fr * (uint32_t)a.w[p].ld + 128u * k + 16u * g : 0x7FFFFF00u);
        c.ws[u][p] = __float_as_uint(scale_at(a.w[p].scales, wrow * a.w[p].ld_scale + min(k, nk - 1), a.w[p].f32)) >> 23;
      }
    }
  };
  auto multiply = [&](Chunk& c, int kc) __attribute__((always_inline)) {
    if constexpr (PACK) {
#pragma unroll
      for (int i = 0; i < kItems; i++)
        if (kGroups * i < items) pack_x(kc, first + kGroups * i, c.raw[i]);
      stage_barrier<63>();
#pragma unroll
      for (int u = 0; u < kAhead; u++) {
        const uint8_t* p = packed + fr * kLd + 128 * (wave + WAVES * u) + 16 * g;
        c.x[u][0] = frag(p, 0, 64);  // (behind the last token whatever lies there: it reaches no other)
        c.xs[u][0] = bytes[fr][wave + WAVES * u];
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; u++) {
      v8bf wide[G][4];
#pragma unroll
      for (int p = 0; p < G; p++) widen<WF>(c.w[u][p], c.ws[u][p], wide[p]);
#pragma unroll
      for (int j = 0; j < NT; j++) {
        v8bf xw[4];
        widen<XF>(c.x[u][j], c.xs[u][j], xw);
#pragma unroll
        for (int p = 0; p < G; p++) acc[p][j] = mfma_wide(wide[p], xw, acc[p][j]);
      }
    }
    if constexpr (PACK) stage_barrier<63>();  // the codes have been read
  };
  for (int kc = 0; kc < nk; kc += kBlocks) {
    Chunk c;
    load(c, kc);
    multiply(c, kc);
  }
#pragma unroll
  for (int p = 0; p < G; p++)
#pragma unroll
    for (int j = 0; j < NT; j++) red[wave][p][j][lane] = acc[p][j];
  __syncthreads();
  if (wave >= NT) return;
  const int64_t t = 16 * wave + fr;
  const int64_t n = n0 + 4 * g, left = a.rows - n;
  if (t >= a.tokens || left <= 0) return;
  float z[G][4];
#pragma unroll
  for (int p = 0; p < G; p++) {
    vf4_t s = red[0][p][wave][lane];
#pragma unroll
    for (int k = 1; k < WAVES; k++) s += red[k][p][wave][lane];
    z[p][0] = s.x, z[p][1] = s.y, z[p][2] = s.z, z[p][3] = s.w;
  }
  if (!GATED && a.bias) {
    float b[4];
    ld4(a.bias_dt, a.bias, n, left, b);
#pragma unroll
    for (int e = 0; e < 4; e++) z[0][e] += b[e];
  }
  float (&one)[1][4] = reinterpret_cast<float (&)[1][4]>(z[0]);
  act_all(a.act, one);
  if constexpr (GATED) {
#pragma unroll
    for (int e = 0; e < 4; e++) z[0][e] *= z[G - 1][e];
  } else if (a.res) {
    float r[4];
    ld4(a.res_dt, a.res, t * a.res_ld + n, left, r);
#pragma unroll
    for (int e = 0; e < 4; e++) z[0][e] += r[e];
  }
  st4(a.y_dt, a.y, t * a.y_ld + n, left, z[0]);
}

template <int XF, int WF, bool GATED, int TT, bool WIDE = false>
int launch_tiles(ProductArgs a, hipStream_t s) {
  a.tiles_n = (int)((a.rows + (GATED ? 127 : 255)) / (GATED ? 128 : 256));
  const int64_t tt = (a.tokens + TT - 1) / TT, total = tt * a.tiles_n;
  if (total > (int64_t)(UINT32_MAX / kProdThreads) - 8) return fail(FP8ADAM_EINVAL, "too many tokens for one call");
  a.tiles_t = (int)tt;
  return launch(k_product<XF, WF, GATED, TT, WIDE>, dim3((unsigned)((total + 7) / 8 * 8)), dim3(kProdThreads), 0, s, a);
}

template <int XF, int WF, bool GATED, int WAVES>
int launch_few(const ProductArgs& a, hipStream_t s) {
  auto go = [&](auto kernel) { return launch(kernel, dim3((unsigned)((a.rows + 15) / 16)), dim3(64 * WAVES), 0, s, a); };
  if (a.xin) {
    if (a.xin_dt == FP8ADAM_F32) return go(k_product_few<XF, WF, GATED, 1, FP8ADAM_F32, WAVES>);
    if (a.xin_dt == FP8ADAM_BF16) return go(k_product_few<XF, WF, GATED, 1, FP8ADAM_BF16, WAVES>);
    return go(k_product_few<XF, WF, GATED, 1, FP8ADAM_F16, WAVES>);
  }
  if (a.tokens <= 16) return go(k_product_few<XF, WF, GATED, 1, kCodes, WAVES>);
  if (a.tokens <= 32) return go(k_product_few<XF, WF, GATED, 2, kCodes, WAVES>);
  return go(k_product_few<XF, WF, GATED, 4, kCodes, WAVES>);
}

// 17 to 64 tokens: whether tiles of 64 tokens, with codes widened, take less time than k_product_few, in us.  That
// reads the weights at 4 TB/s and has every work-group of 16 rows read every token, at 7 TB/s from the caches; a tile takes
// 0.88 for each block of 128 columns.  (4096 to 2 * 11008 with 17, 32 and 64 tokens: few 29, 35 and 54,
// estimated 29, 35 and 48; tiles 33, estimated 33.  11008 to 4096 with 64: few 32, tiles, of which there are 16, 80 estimated.
// Where there are tiles enough to fill the card, what bounds them is the weights' bytes, which are not in their estimate: k_product_few
// reads the same bytes and the tokens besides.)
inline bool tile_is_faster(const ProductArgs& a, bool gated) {
  const double nk = (a.cols + 127) >> 7, weights = (gated ? 256.0 : 128.0) * nk * a.rows;
  const double few = weights / 4e6 + 128.0 * nk * (double)a.tokens * (double)((a.rows + 15) / 16) / 7e6;
  const int64_t tiles = (a.rows + (gated ? 127 : 255)) / (gated ? 128 : 256);
  return 5.0 + 0.88 * nk * (double)((tiles + 255) / 256) < few;
}

template <int XF, int WF, bool GATED>
int launch_product_of(const ProductArgs& a, hipStream_t s) {
  if (few_tokens(a)) {
    if (a.tokens > 16 && tile_is_faster(a, GATED)) return launch_tiles<XF, WF, GATED, 64, true>(a, s);
    return a.rows >= 16 * 512 ? launch_few<XF, WF, GATED, 4>(a, s) : launch_few<XF, WF, GATED, 8>(a, s);
  }
  if (a.tokens <= kFewTokens) return launch_tiles<XF, WF, GATED, 64, true>(a, s);  // kept or packed: the same precision as without
  if (a.exact || (a.y && a.y_dt == FP8ADAM_F32)) return launch_tiles<XF, WF, GATED, 128, true>(a, s);
  // the tile whose rounds over 256 CUs cost least: a tile of 128 and of 64 tokens takes about 0.68 and
  // 0.45 of the time of one of 256 (2048 x 8192 x 2048, in one, two and four rounds: 34, 44, 59 us)
  const int64_t tn = (a.rows + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
  auto cost = [&](int tt, double c) { return c * (double)(((a.tokens + tt - 1) / tt * tn + 255) / 256); };
  const double c256 = cost(256, 1.0), c128 = cost(128, 0.68), c64 = cost(64, 0.45);
  if (c256 <= c128 && c256 <= c64) return launch_tiles<XF, WF, GATED, 256>(a, s);
  if (c128 <= c64) return launch_tiles<XF, WF, GATED, 128>(a, s);
  return launch_tiles<XF, WF, GATED, 64>(a, s);
}

template <int XF, int WF>
int launch_product(const ProductArgs& a, bool gated, hipStream_t s) {
  return gated ? launch_product_of<XF, WF, true>(a, s) : launch_product_of<XF, WF, false>(a, s);
}

}  // namespace fp8adam_layer
