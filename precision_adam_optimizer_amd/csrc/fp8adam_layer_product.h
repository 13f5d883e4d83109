// fp8adam_layer_product.h -- the forward products of the layer operators, instantiated
// for each pair of formats in fp8adam_layer_product_*.hip.
//
// Both operands are codes with one power-of-two scale per row and 128 columns, and
// gfx950's scaled matrix instruction multiplies 16 x 128 by 128 x 16 codes with a
// scale for every row and 32 columns: one instruction takes exactly one block of 16
// rows of each, with its scales.
//
// The instruction sums eight consecutive products at a time, each cut (towards zero) at 2^-13 of the
// power of two of the largest product's exponents, and adds these sums to 32 bits (measured with
// one large and one small product in every place; the unscaled FP8 instructions do the
// same).  On normally distributed codes a sum of 128 is off by 1.4e-5 of the sums' rms: a fortieth of
// half a step of fp16, a three-hundredth of one of bf16, so it serves outputs of 8 and 16 bits.
// For outputs of 32 bits (WIDE), and for few tokens, where the weights' bytes are what
// counts, both operands are widened to bf16 times their scales, which is exact, and
// multiplied by the bf16 instruction, which adds every product in 32 bits.
//
// The order of the 128 products in one instruction is free, so a lane may take any 32
// columns of its row as long as both operands take the same: here the 16-byte pieces
// g and g + 4 of the row's eight, g = lane / 16.
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

// Byte S of each lane's scale dwords; rows of D are A's rows (weights), columns B's (tokens).
template <int XF, int WF, int S>
__device__ __forceinline__ vf4_t mfma_scaled(v8i w, v8i x, vf4_t c, int ws, int xs) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, WF, XF, S, ws, S, xs);
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

// The E8M0 bytes of four blocks of a row from block k on, of which n exist.
__device__ __forceinline__ uint32_t scale_bytes(const In8& m, int64_t row, int k, int n) {
  if (!m.f32) return ld_global<uint32_t>(static_cast<const uint8_t*>(m.scales) + row * m.ld_scale + k);
  const float* p = static_cast<const float*>(m.scales) + row * m.ld_scale + k;
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; j++)
    if (j < n) w |= (__float_as_uint(ld_global<float>(p + j)) >> 23 & 0xFFu) << (8 * j);
  return w;
}

// A tile of 256 weight rows by TT tokens: eight waves, two along the rows and four along the
// tokens, each 128 x TT/4.  Blocks of 128 columns of both operands go straight into shared
// memory, double-buffered: the next block is on its way while this one is multiplied.  A
// row's eight 16-byte pieces are stored in the order piece ^ (row & 7), by giving each
// lane of the load another source, so that the 16 rows of a fragment lie on all banks.
//
// The sums then go through shared memory, 64 tokens at a time, into rows of 128 columns
// for half a wave each: bias, activation, product, residual and the blocks' amax are made
// there, and whole lines are stored.
template <int XF, int WF, bool GATED, int TT, bool WIDE>
__global__ __launch_bounds__(kProdThreads, 2) void k_product(const ProductArgs a) {
  constexpr int kJ = TT / 64;                     // tiles of 16 tokens per wave
  constexpr int kBuf = (kWRows + TT) * 128;
  constexpr int kLdZ = 256 * 4 + 16;              // bytes between tokens of the sums: spread over the banks
  __shared__ __attribute__((aligned(16))) uint8_t buf0[kBuf];
  __shared__ __attribute__((aligned(16))) uint8_t buf1[kBuf < 64 * kLdZ ? 64 * kLdZ : kBuf];
  __shared__ __attribute__((aligned(16))) uint8_t sc[(kWRows + TT) * kScaleLd];

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
  const int half = wave >> 2, quarter = wave & 3;
  const int nk = (a.cols + 127) >> 7;

  // loads: 8 rows of 128 bytes per wave and instruction
  const int lrow = lane >> 3;
  const int64_t vt = min((int64_t)TT, a.tokens - t0);
  const int64_t vn = min((int64_t)(GATED ? 128 : 256), (int64_t)a.rows - n0);
  const Rsrc rx = rsrc(a.x.codes + t0 * a.x.ld, vt * a.x.ld);
  const Rsrc rw = rsrc(a.w[0].codes + (int64_t)n0 * a.w[0].ld, vn * a.w[0].ld);
  const Rsrc ru = GATED ? rsrc(a.w[1].codes + (int64_t)n0 * a.w[1].ld, vn * a.w[1].ld) : rw;
  uint32_t ow[4], ox[TT / 64];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int q = 8 * (wave + 8 * i);  // the first of the 8 rows in shared memory
    const int row = GATED ? 64 * (q >> 7) + (q & 63) + lrow : q + lrow;
    ow[i] = (uint32_t)row * (uint32_t)a.w[GATED && (q & 64) ? 1 : 0].ld + 16u * ((lane & 7) ^ lrow);
  }
#pragma unroll
  for (int i = 0; i < TT / 64; i++) ox[i] = (uint32_t)(8 * (wave + 8 * i) + lrow) * (uint32_t)a.x.ld + 16u * ((lane & 7) ^ lrow);
  auto load = [&](uint8_t* buf, int k) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int q = 8 * (wave + 8 * i);
      if (GATED && (q & 64)) load_lds(ru, buf + q * 128, ow[i], 128u * k);
      else load_lds(rw, buf + q * 128, ow[i], 128u * k);
    }
#pragma unroll
    for (int i = 0; i < TT / 64; i++) load_lds(rx, buf + (kWRows + 8 * (wave + 8 * i)) * 128, ox[i], 128u * k);
  };

  vf4_t acc[8][kJ];
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int j = 0; j < kJ; j++) acc[i][j] = vf4_t{0, 0, 0, 0};
  const int g = lane >> 4, fr = lane & 15;
  const int p0 = 16 * (g ^ (fr & 7)), p1 = 16 * ((g + 4) ^ (fr & 7));
  const int wrow = 128 * half + fr, xrow = kWRows + (TT / 4) * quarter + fr;
  int wsc[8], xsc[kJ];

  auto step = [&](const uint8_t* buf, auto which) {
    constexpr int S = decltype(which)::value;
    if constexpr (WIDE) {
      v8bf x[kJ][4];
#pragma unroll
      for (int j = 0; j < kJ; j++) widen<XF>(frag(buf + (xrow + 16 * j) * 128, p0, p1), (uint32_t)xsc[j] >> (8 * S) & 0xFFu, x[j]);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        v8bf w[4];
        widen<WF>(frag(buf + (wrow + 16 * i) * 128, p0, p1), (uint32_t)wsc[i] >> (8 * S) & 0xFFu, w);
#pragma unroll
        for (int j = 0; j < kJ; j++) acc[i][j] = mfma_wide(w, x[j], acc[i][j]);
      }
    } else {
      v8i x[kJ];
#pragma unroll
      for (int j = 0; j < kJ; j++) x[j] = frag(buf + (xrow + 16 * j) * 128, p0, p1);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const v8i w = frag(buf + (wrow + 16 * i) * 128, p0, p1);
#pragma unroll
        for (int j = 0; j < kJ; j++) acc[i][j] = mfma_scaled<XF, WF, S>(w, x[j], acc[i][j], wsc[i], xsc[j]);
      }
    }
  };

  load(buf0, 0);
  for (int kc = 0; kc < nk; kc += kScaleChunk) {
    if (kc > 0) __syncthreads();  // the scales before have been read
    for (int q = threadIdx.x; q < kWRows + TT; q += kProdThreads) {
      const bool is_x = q >= kWRows;
      const bool up = GATED && !is_x && (q & 64);
      const int64_t row = is_x ? t0 + (q - kWRows) : n0 + (GATED ? 64 * (q >> 7) + (q & 63) : q);
      const bool there = is_x ? row < a.tokens : row < a.rows;
      const In8& m = is_x ? a.x : up ? a.w[1] : a.w[0];
      for (int k = 0; k < kScaleChunk && kc + k < nk; k += 4)
        *reinterpret_cast<uint32_t*>(sc + q * kScaleLd + k) = there ? scale_bytes(m, row, kc + k, nk - kc - k) : 0x7F7F7F7Fu;
    }
    const int end = min(nk, kc + kScaleChunk);
    for (int k = kc; k < end; k += 4) {
      auto one = [&](auto which) {
        constexpr int S = decltype(which)::value;
        if (k + S >= end) return;
        wait_loads();
        __syncthreads();  // this block is there, and the other buffer has been read
        if (k + S + 1 < nk) load(S & 1 ? buf0 : buf1, k + S + 1);
        if constexpr (S == 0) {
#pragma unroll
          for (int i = 0; i < 8; i++) wsc[i] = *reinterpret_cast<const int*>(sc + (wrow + 16 * i) * kScaleLd + (k - kc));
#pragma unroll
          for (int j = 0; j < kJ; j++) xsc[j] = *reinterpret_cast<const int*>(sc + (xrow + 16 * j) * kScaleLd + (k - kc));
        }
        step(S & 1 ? buf1 : buf0, which);
      };
      one(std::integral_constant<int, 0>{});
      one(std::integral_constant<int, 1>{});
      one(std::integral_constant<int, 2>{});
      one(std::integral_constant<int, 3>{});
    }
  }

  // the sums, through shared memory (64 tokens: tile j of every wave)
  const int hw = threadIdx.x >> 5, hl = threadIdx.x & 31;
  uint8_t* z8 = buf1;
#pragma unroll 1
  for (int j = 0; j < kJ; j++) {
    __syncthreads();
    auto put = [&](auto which) {
      constexpr int J = decltype(which)::value;
      if constexpr (J < kJ) {
        if (j == J) {
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const int col = GATED ? 128 * (i >> 2) + 64 * half + 16 * (i & 3) : 128 * half + 16 * i;
            *reinterpret_cast<vf4_t*>(z8 + (16 * quarter + fr) * kLdZ + 4 * (col + 4 * g)) = acc[i][J];
          }
        }
      }
    };
    put(std::integral_constant<int, 0>{});
    put(std::integral_constant<int, 1>{});
    put(std::integral_constant<int, 2>{});
    put(std::integral_constant<int, 3>{});
    __syncthreads();
#pragma unroll 1
    for (int q = hw; q < (GATED ? 64 : 128); q += kProdThreads / 32) {
      const int tok = GATED ? q : q >> 1, blk = GATED ? 0 : q & 1;
      const int64_t t = t0 + (TT / 4) * (tok >> 4) + 16 * j + (tok & 15);
      const int64_t n = n0 + 128 * blk + 4 * hl, left = a.rows - n;
      if (t >= a.tokens || n0 + 128 * blk >= a.rows) continue;  // the same in the half-wave
      const vf4_t v = *reinterpret_cast<const vf4_t*>(z8 + tok * kLdZ + 4 * (128 * blk + 4 * hl));
      float z[4] = {v.x, v.y, v.z, v.w};
      if (!GATED && a.bias) {
        float b[4];
        ld4(a.bias_dt, a.bias, n, left, b);
#pragma unroll
        for (int e = 0; e < 4; e++) z[e] += b[e];
      }
#pragma unroll
      for (int e = 0; e < 4; e++) z[e] = e < left ? z[e] : 0.0f;
      const int64_t block = (n0 >> 7) + blk;
      if (a.keep[0].codes) put_block(a.keep[0], t, block, hl, z);
      act4(a.act, z);
      if constexpr (GATED) {
        const vf4_t w = *reinterpret_cast<const vf4_t*>(z8 + tok * kLdZ + 4 * (128 + 4 * hl));
        const float u[4] = {left > 0 ? w.x : 0.0f, left > 1 ? w.y : 0.0f, left > 2 ? w.z : 0.0f, left > 3 ? w.w : 0.0f};
        if (a.keep[1].codes) put_block(a.keep[1], t, block, hl, u);
#pragma unroll
        for (int e = 0; e < 4; e++) z[e] *= u[e];
      } else if (a.res) {
        float r[4];
        ld4(a.res_dt, a.res, t * a.res_ld + n, left, r);
#pragma unroll
        for (int e = 0; e < 4; e++) z[e] += r[e];
      }
      if (a.y) st4(a.y_dt, a.y, t * a.y_ld + n, left, z);
      if (a.y8.codes) put_block(a.y8, t, block, hl, z);
    }
  }
}

// Few tokens, nothing kept: bound by the weights' bytes.  A work-group takes 16 rows of
// weights (gated: 16 of each projection) and its eight waves an eighth of the blocks of 128
// each, weights straight into registers; their sums meet in shared memory.
// PACK: up to 16 tokens in 16 or 32 bits, which each wave turns into codes itself as the
// fragments it needs (the first work-group stores them).
constexpr int kFewWaves = 8;
constexpr int kFewAhead = 4;  // blocks in flight per wave

template <int FMT>
__device__ __forceinline__ v8i pack_frag(const ProductArgs& a, int64_t t, int k, int g, bool store, int& xs) {
  float x[8][4];
  uint32_t am = 0;
#pragma unroll
  for (int q = 0; q < 8; q++) {
    const int64_t c = 128 * (int64_t)k + 32 * g + 4 * q;
    ld4(a.xin_dt, a.xin, t * a.xin_ld + c, t < a.tokens ? a.cols - c : 0, x[q]);
#pragma unroll
    for (int j = 0; j < 4; j++) am = max(am, abs_bits(x[q][j]));
  }
  am = max(am, (uint32_t)__shfl_xor((int)am, 16));
  am = max(am, (uint32_t)__shfl_xor((int)am, 32));
  float s, inv;
  choose_scale<FMT, 0>(am, s, inv);
  v8i f;
#pragma unroll
  for (int q = 0; q < 8; q++) f[q] = (int)codes4_pow2<FMT>(x[q], s, nonfinite_amax(am));
  xs = (int)(__float_as_uint(s) >> 23);
  if (store && t < a.tokens) {
    uint8_t* p = a.x8.codes + t * a.x8.ld + 128 * (int64_t)k + 32 * g;
    st_global<vu4>(p, vu4{(uint32_t)f[0], (uint32_t)f[1], (uint32_t)f[2], (uint32_t)f[3]});
    st_global<vu4>(p + 16, vu4{(uint32_t)f[4], (uint32_t)f[5], (uint32_t)f[6], (uint32_t)f[7]});
    if (g == 0) st_global<uint8_t>(a.x8.scales + t * a.x8.ld_scale + k, (uint8_t)xs);
  }
  return f;
}

template <int XF, int WF, bool GATED, int NT, bool PACK>
__global__ __launch_bounds__(64 * kFewWaves) void k_product_few(const ProductArgs a) {
  constexpr int G = GATED ? 2 : 1;
  __shared__ vf4_t red[kFewWaves][G][NT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, fr = lane & 15;
  const int n0 = blockIdx.x * 16;
  const int nk = (a.cols + 127) >> 7;
  const int64_t vn = min((int64_t)16, (int64_t)a.rows - n0);
  Rsrc rw[G];
#pragma unroll
  for (int p = 0; p < G; p++) rw[p] = rsrc(a.w[p].codes + (int64_t)n0 * a.w[p].ld, vn * a.w[p].ld);
  const Rsrc rx = rsrc(PACK ? nullptr : a.x.codes, PACK ? 0 : a.tokens * a.x.ld);
  const int64_t wrow = n0 + min(fr, (int)vn - 1);

  vf4_t acc[G][NT];
#pragma unroll
  for (int p = 0; p < G; p++)
#pragma unroll
    for (int j = 0; j < NT; j++) acc[p][j] = vf4_t{0, 0, 0, 0};

  auto two = [](Rsrc r, uint32_t o) {
    const vu4 a = __builtin_amdgcn_raw_buffer_load_b128(r, o, 0, 0), b = __builtin_amdgcn_raw_buffer_load_b128(r, o + 16, 0, 0);
    return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
  };
  for (int k0 = wave; k0 < nk; k0 += kFewWaves * kFewAhead) {
    v8i w[kFewAhead][G];
    int ws[kFewAhead][G];
#pragma unroll
    for (int u = 0; u < kFewAhead; u++) {
      const int k = k0 + kFewWaves * u;
#pragma unroll
      for (int p = 0; p < G; p++) {
        // behind the last block: outside the resource, zeros
        w[u][p] = two(rw[p], k < nk ? (uint32_t)fr * (uint32_t)a.w[p].ld + 128u * k + 32u * g : 0x7FFFFF00u);
        ws[u][p] = (int)(__float_as_uint(scale_at(a.w[p].scales, wrow * a.w[p].ld_scale + min(k, nk - 1), a.w[p].f32)) >> 23);
      }
    }
#pragma unroll
    for (int u = 0; u < kFewAhead; u++) {
      const int k = k0 + kFewWaves * u;
      if (k >= nk) break;  // the same in the wave
      v8bf wide[G][4];
#pragma unroll
      for (int p = 0; p < G; p++) widen<WF>(w[u][p], ws[u][p], wide[p]);
#pragma unroll
      for (int j = 0; j < NT; j++) {
        const int64_t t = 16 * j + fr;
        int xs;
        v8i x;
        if constexpr (PACK) {
          x = pack_frag<XF>(a, t, k, g, blockIdx.x == 0, xs);
        } else {
          x = two(rx, (uint32_t)t * (uint32_t)a.x.ld + 128u * k + 32u * g);
          xs = t < a.tokens ? (int)(__float_as_uint(scale_at(a.x.scales, t * a.x.ld_scale + k, a.x.f32)) >> 23) : 127;
        }
        v8bf xw[4];
        widen<XF>(x, xs, xw);
#pragma unroll
        for (int p = 0; p < G; p++) acc[p][j] = mfma_wide(wide[p], xw, acc[p][j]);
      }
    }
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
    for (int k = 1; k < kFewWaves; k++) s += red[k][p][wave][lane];
    z[p][0] = s.x, z[p][1] = s.y, z[p][2] = s.z, z[p][3] = s.w;
  }
  if (!GATED && a.bias) {
    float b[4];
    ld4(a.bias_dt, a.bias, n, left, b);
#pragma unroll
    for (int e = 0; e < 4; e++) z[0][e] += b[e];
  }
  act4(a.act, z[0]);
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

template <int XF, int WF, bool GATED>
int launch_few(const ProductArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.rows + 15) / 16)), block(64 * kFewWaves);
  if (a.xin) return launch(k_product_few<XF, WF, GATED, 1, true>, grid, block, 0, s, a);
  if (a.tokens <= 16) return launch(k_product_few<XF, WF, GATED, 1, false>, grid, block, 0, s, a);
  if (a.tokens <= 32) return launch(k_product_few<XF, WF, GATED, 2, false>, grid, block, 0, s, a);
  return launch(k_product_few<XF, WF, GATED, 4, false>, grid, block, 0, s, a);
}

template <int XF, int WF, bool GATED>
int launch_product_of(const ProductArgs& a, hipStream_t s) {
  if (few_tokens(a)) return launch_few<XF, WF, GATED>(a, s);
  if (a.y && a.y_dt == FP8ADAM_F32) return launch_tiles<XF, WF, GATED, 128, true>(a, s);
  // the tile whose rounds over 256 CUs cost least: a tile of 128 and of 64 tokens takes about 0.6 and
  // 0.4 of the time of one of 256
  const int64_t tn = (a.rows + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
  auto cost = [&](int tt, double c) { return c * (double)(((a.tokens + tt - 1) / tt * tn + 255) / 256); };
  const double c256 = cost(256, 1.0), c128 = cost(128, 0.6), c64 = cost(64, 0.4);
  if (c256 <= c128 && c256 <= c64) return launch_tiles<XF, WF, GATED, 256>(a, s);
  if (c128 <= c64) return launch_tiles<XF, WF, GATED, 128>(a, s);
  return launch_tiles<XF, WF, GATED, 64>(a, s);
}

template <int XF, int WF>
int launch_product(const ProductArgs& a, bool gated, hipStream_t s) {
  return gated ? launch_product_of<XF, WF, true>(a, s) : launch_product_of<XF, WF, false>(a, s);
}

}  // namespace fp8adam_layer
