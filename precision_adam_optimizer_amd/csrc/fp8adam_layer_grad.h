// fp8adam_layer_grad.h -- the products of the backward pass, out[m][k] = sum over r of
// A(m, r) B[r][k], instantiated for each format of B in fp8adam_layer_grad_*.hip.
//
// A is a gradient in bf16 and B a matrix in 8 bits whose rows run along the sum: the
// input's checkpoint for a weight gradient (r = tokens, A stored [r][m]), the weights for
// an input gradient (r = their rows, A stored [m][r]).  B's scale changes from row to row
// of the sum, so its codes are widened to bf16 times their scale, which is exact, as
// they are staged: once per tile, sixteen codes of one block per lane.  The product is
// then one of bf16 on the matrix cores.
//
// Where a stored row runs along m or k and the instruction wants eight consecutive r
// of one column, shared memory is read through its transposing loads (16 lanes take 4 rows of
// 16 columns and get a column of 4 each).
#pragma once

#include "fp8adam_layer.h"

namespace fp8adam_layer {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s* TrPtr;

constexpr int kStep = 64;  // of the sum, at a time

// Rows of a tile along the sum lie in shared memory with their 32-byte units (16
// columns) in the order unit ^ turn(row): the rows that two neighbouring groups of 16
// lanes read together, 8g + q and 8g + 8 + q (q < 4), lie on different banks.
__device__ __forceinline__ int turn(int row) { return (row >> 1 & 4) | (row & 3); }

// Eight r (8g .. 8g + 7 of the 32 from `row` on) of column 16 * unit + lane % 16.
template <int LD>
__device__ __forceinline__ v8s tr_frag(const uint8_t* tile, int row, uint32_t off) {
  const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TrPtr)(tile + row * LD + off));
  const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TrPtr)(tile + (row + 4) * LD + off));
  return v8s{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Sixteen codes times their scale, in bf16 (exact: a code has at most four significant bits).
template <int BF>
__device__ __forceinline__ void widen(const vu4& c, float s, vu4 (&out)[2]) {
#pragma unroll
  for (int q = 0; q < 4; q++) {
    uint32_t lo, hi;
    if constexpr (BF == 0) {
      lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[q], s, false));
      hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[q], s, true));
    } else {
      lo = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[q], s, false));
      hi = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(c[q], s, true));
    }
    out[q >> 1][2 * (q & 1)] = lo;
    out[q >> 1][2 * (q & 1) + 1] = hi;
  }
}

// A tile of MT x KT of out; waves WM along m and WK along k.
template <bool TRANS, int BF, int MT, int KT, int WM, int WK>
__global__ __launch_bounds__(64 * WM * WK, 2) void k_grad(const GradArgs a, int splits, int tiles_m, int tiles_k) {
  constexpr int kT = 64 * WM * WK, kWaves = WM * WK;
  constexpr int kI = MT / WM / 16, kJ = KT / WK / 16;       // tiles of 16 per wave
  constexpr int kLdA = TRANS ? MT * 2 : kStep * 2, kLdB = KT * 2;
  constexpr int kA = MT * kStep * 2, kB = KT * kStep * 2;
  constexpr int kLoadsA = kA / 1024 / kWaves;               // wave loads of 1024 bytes
  constexpr int kPassB = kStep * (KT / 16) / kT;            // 16 codes per lane
  __shared__ __attribute__((aligned(16))) uint8_t buf0[kA + kB];
  __shared__ __attribute__((aligned(16))) uint8_t buf1[kA + kB];

  // tiles in bands of four along m, an eighth of each part of the sum on each XCD
  const int tiles = tiles_m * tiles_k;
  const int64_t total = (int64_t)tiles * splits, per = (total + 7) >> 3;
  const int64_t pos = (int64_t)(blockIdx.x & 7u) * per + (blockIdx.x >> 3);
  if (pos >= total || (int64_t)(blockIdx.x >> 3) >= per) return;
  const int split = (int)(pos / tiles), tile = (int)(pos - (int64_t)split * tiles);
  const int band = tile / (4 * tiles_k), in = tile - band * 4 * tiles_k, width = min(4, tiles_m - 4 * band);
  const int64_t m0 = (int64_t)(4 * band + in % width) * MT;
  const int k0 = in / width * KT;

  const int64_t spp = (a.r + kStep - 1) / kStep, steps = spp * a.npairs;
  const int64_t part = (steps + splits - 1) / splits;
  const int64_t s0 = min(steps, split * part), s1 = min(steps, s0 + part);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wk = wave / WM;
  const int g = lane >> 4, fr = lane & 15;

  // A's loads, in 16-byte pieces (its rows are whole pieces: a.lda is at least m or r rounded up to 8, with
  // zeros behind them): kRows rows of the stored tile per wave and instruction
  constexpr int kChunks = kLdA / 16, kRows = 64 / kChunks;
  uint32_t oa[kLoadsA];
  int ca[kLoadsA];  // not transposed: the lane's first r in the step
#pragma unroll
  for (int i = 0; i < kLoadsA; i++) {
    const int row = (wave + kWaves * i) * kRows + lane / kChunks, p = lane % kChunks;
    const int c = TRANS ? ((((p >> 1) ^ turn(row)) << 1) | (p & 1)) : p ^ (row & 7);
    oa[i] = (uint32_t)row * (uint32_t)(2 * a.lda) + 16u * c;
    ca[i] = 8 * c;
  }
  // B's loads
  const int brow = threadIdx.x / (KT / 16), bcol = threadIdx.x % (KT / 16);
  constexpr int kRowsB = kT / (KT / 16);
  const int64_t nb = ((int64_t)a.k + 127) >> 7, block = min(nb - 1, (int64_t)((k0 >> 7) + (bcol >> 3)));
  vu4 bc[kPassB];
  float bs[kPassB];

  auto load = [&](uint8_t* buf, int64_t s) {
    int pair = 0;
    int64_t r0 = s * kStep;
    if (a.npairs > 1) {
      pair = (int)(s / spp);
      r0 = (s - pair * spp) * kStep;
    }
    const uint16_t* A = pair == 0 ? a.a[0] : pair == 1 ? a.a[1] : pair == 2 ? a.a[2] : a.a[3];
    const uint8_t* codes = pair == 0 ? a.b[0].codes : pair == 1 ? a.b[1].codes : pair == 2 ? a.b[2].codes : a.b[3].codes;
    const void* scales = pair == 0 ? a.b[0].scales : pair == 1 ? a.b[1].scales : pair == 2 ? a.b[2].scales : a.b[3].scales;
    const int64_t ldb = pair == 0 ? a.b[0].ld : pair == 1 ? a.b[1].ld : pair == 2 ? a.b[2].ld : a.b[3].ld;
    const int64_t ldbs = pair == 0 ? a.b[0].ld_scale : pair == 1 ? a.b[1].ld_scale : pair == 2 ? a.b[2].ld_scale : a.b[3].ld_scale;
    const int64_t rows = min((int64_t)kStep, a.r - r0);
    if constexpr (TRANS) {
      const Rsrc r = rsrc(A + r0 * a.lda + m0, 2 * ((rows - 1) * a.lda + ((min((int64_t)MT, a.m - m0) + 7) & ~(int64_t)7)));
#pragma unroll
      for (int i = 0; i < kLoadsA; i++) load_lds(r, buf + (wave + kWaves * i) * 1024, oa[i], 0);
    } else {
      const int64_t mr = min((int64_t)MT, a.m - m0);
      const Rsrc r = rsrc(A + m0 * a.lda + r0, 2 * ((mr - 1) * a.lda + ((a.r - r0 + 7) & ~(int64_t)7)));
#pragma unroll
      for (int i = 0; i < kLoadsA; i++)  // columns behind the sum's end: outside the resource, zeros
        load_lds(r, buf + (wave + kWaves * i) * 1024, r0 + ca[i] < a.r ? oa[i] : 0x7FFFFF00u, 0);
    }
    const Rsrc rb = rsrc(codes + r0 * ldb, (rows - 1) * ldb + 128 * nb);
#pragma unroll
    for (int p = 0; p < kPassB; p++) {
      const int row = brow + kRowsB * p;
      bc[p] = __builtin_amdgcn_raw_buffer_load_b128(rb, (uint32_t)row * (uint32_t)ldb + k0 + 16 * bcol, 0, 0);
      bs[p] = scale_at(scales, min(r0 + row, a.r - 1) * ldbs + block, a.b[0].f32);
    }
  };
  auto store_b = [&](uint8_t* buf) {
#pragma unroll
    for (int p = 0; p < kPassB; p++) {
      const int row = brow + kRowsB * p;
      vu4 w[2];
      widen<BF>(bc[p], bs[p], w);
      uint8_t* d = buf + kA + row * kLdB + 32 * (bcol ^ turn(row));
      // lanes eight apart have the same banks: each half of them begins with another half of the unit
      const int h = bcol >> 3 & 1;
      *reinterpret_cast<vu4*>(d + 16 * h) = h ? w[1] : w[0];
      *reinterpret_cast<vu4*>(d + 16 * (h ^ 1)) = h ? w[0] : w[1];
    }
  };

  // fragments: the byte offsets in a row of the lane's units
  const int trow = 8 * g + (fr >> 2);
  uint32_t fa[kI], fb[kJ];
#pragma unroll
  for (int i = 0; i < kI; i++)
    fa[i] = TRANS ? 32 * (((MT / WM / 16) * wm + i) ^ turn(trow)) + 8 * (fr & 3) : ((MT / WM) * wm + 16 * i + fr) * kLdA;
#pragma unroll
  for (int j = 0; j < kJ; j++) fb[j] = 32 * (((KT / WK / 16) * wk + j) ^ turn(trow)) + 8 * (fr & 3);

  vf4_t acc[kI][kJ];
#pragma unroll
  for (int i = 0; i < kI; i++)
#pragma unroll
    for (int j = 0; j < kJ; j++) acc[i][j] = vf4_t{0, 0, 0, 0};

  auto compute = [&](const uint8_t* buf) {
#pragma unroll
    for (int h = 0; h < kStep / 32; h++) {
      v8s b[kJ];
#pragma unroll
      for (int j = 0; j < kJ; j++) b[j] = tr_frag<kLdB>(buf + kA, 32 * h + trow, fb[j]);
#pragma unroll
      for (int i = 0; i < kI; i++) {
        v8s x;
        if constexpr (TRANS) x = tr_frag<kLdA>(buf, 32 * h + trow, fa[i]);
        else x = *reinterpret_cast<const v8s*>(buf + fa[i] + 16 * ((4 * h + g) ^ (fr & 7)));
#pragma unroll
        for (int j = 0; j < kJ; j++)  // rows of D: four consecutive k per lane
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, b[j]), __builtin_bit_cast(v8bf, x),
                                                              acc[i][j], 0, 0, 0);
      }
    }
  };

  if (s0 < s1) {
    load(buf0, s0);
    store_b(buf0);
    auto one = [&](uint8_t* cur, uint8_t* next, int64_t s) {
      wait_loads();
      __syncthreads();  // this step's tiles are there, and the other buffer has been read
      if (s + 1 < s1) load(next, s + 1);
      compute(cur);
      if (s + 1 < s1) store_b(next);
    };
    for (int64_t s = s0; s < s1; s += 2) {
      one(buf0, buf1, s);
      if (s + 1 < s1) one(buf1, buf0, s + 1);
    }
  }

  const int64_t ldp = ((int64_t)a.k + 3) & ~(int64_t)3;
#pragma unroll
  for (int i = 0; i < kI; i++) {
    const int64_t m = m0 + (MT / WM) * wm + 16 * i + fr;
    if (m >= a.m) continue;
#pragma unroll
    for (int j = 0; j < kJ; j++) {
      const int k = k0 + (KT / WK) * wk + 16 * j + 4 * g, left = a.k - k;
      if (left <= 0) continue;
      float x[4] = {acc[i][j].x, acc[i][j].y, acc[i][j].z, acc[i][j].w};
      if (a.partial) {
        st_global<vu4>(a.partial + ((int64_t)split * a.m + m) * ldp + k, pack4<FP8ADAM_F32>(x).x);
      } else {
        if (a.accumulate) {
          float o[4];
          ld4(a.out_dt, a.out, m * a.ld_out + k, left, o);
#pragma unroll
          for (int e = 0; e < 4; e++) x[e] += o[e];
        }
        st4(a.out_dt, a.out, m * a.ld_out + k, left, x);
      }
    }
  }
}

// out (+)= the sum of the parts, in their order.
template <int DUMMY>
__global__ __launch_bounds__(kThreads) void k_grad_join(const GradArgs a, int splits) {
  const int64_t ldp = ((int64_t)a.k + 3) & ~(int64_t)3, groups = ldp >> 2;
  const int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (q >= a.m * groups) return;
  const int64_t m = q / groups;
  const int k = (int)(q - m * groups) * 4;
  const float* p = a.partial + m * ldp + k;
  vf4_t s = {0, 0, 0, 0};
#pragma unroll 4
  for (int i = 0; i < splits; i++) s += __builtin_bit_cast(vf4_t, ld_global<vu4>(p + (int64_t)i * a.m * ldp));
  float x[4] = {s.x, s.y, s.z, s.w};
  if (a.accumulate) {
    float o[4];
    ld4(a.out_dt, a.out, m * a.ld_out + k, a.k - k, o);
#pragma unroll
    for (int e = 0; e < 4; e++) x[e] += o[e];
  }
  st4(a.out_dt, a.out, m * a.ld_out + k, a.k - k, x);
}

template <int BF, int MT, int KT, int WM, int WK>
int launch_grad_tile(const GradArgs& a, const GradPlan& p, hipStream_t s) {
  const int64_t tm = (a.m + MT - 1) / MT, tk = (a.k + KT - 1) / KT, total = tm * tk * p.splits;
  if (total > (int64_t)(UINT32_MAX / (64 * WM * WK)) - 8) return fail(FP8ADAM_EINVAL, "too many tokens for one call");
  const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * WM * WK);
  int r = a.trans ? launch(k_grad<true, BF, MT, KT, WM, WK>, grid, block, 0, s, a, p.splits, (int)tm, (int)tk)
                  : launch(k_grad<false, BF, MT, KT, WM, WK>, grid, block, 0, s, a, p.splits, (int)tm, (int)tk);
  if (r || p.splits == 1) return r;
  const int64_t threads = a.m * (((int64_t)a.k + 3) >> 2);
  return launch(k_grad_join<0>, dim3((unsigned)((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a, p.splits);
}

template <int BF>
int launch_grad(const GradArgs& a, const GradPlan& p, hipStream_t s) {
  return p.tile == 0 ? launch_grad_tile<BF, 256, 256, 2, 4>(a, p, s) : launch_grad_tile<BF, 128, 128, 2, 2>(a, p, s);
}

}  // namespace fp8adam_layer
