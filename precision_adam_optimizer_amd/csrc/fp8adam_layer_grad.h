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

constexpr int kStep = 32;  // of the sum, at a time

// Rows of a tile along the sum lie in shared memory with their 32-byte units (16
// columns) in the order unit ^ turn(row): the four rows whose pairs of units half a wave
// reads together lie on different banks.
__device__ __forceinline__ int turn(int row) { return (row & 3) << 1; }

// Eight r of a column: rows `row` .. row + 3 and row + 4 .. row + 7 through a lane's offset `off`.
template <int LD>
__device__ __forceinline__ v8bf tr_frag(const uint8_t* tile, uint32_t off) {
  const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TrPtr)(tile + off));
  const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TrPtr)(tile + off + 4 * LD));
  return __builtin_bit_cast(v8bf, v8s{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
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

// A tile of MT x KT of out, waves WM along m and WK along k.  The sum goes in stages of 32:
// A's rows and B's codes and scales go straight into shared memory, three stages ahead
// (four of codes); each stage's codes are widened into one of two buffers while the stage
// before is multiplied.
//
// The sums then go through shared memory into whole rows of the tile, so that whole lines are
// read (accumulate) and written.
template <bool TRANS, int BF, int MT, int KT, int WM, int WK>
__global__ __launch_bounds__(64 * WM * WK, 2) void k_grad(const GradArgs a, int splits, int tiles_m, int tiles_k) {
  constexpr int kT = 64 * WM * WK, kWaves = WM * WK;
  constexpr int kI = MT / WM / 32, kJ = KT / WK / 32;       // products of a wave
  constexpr int kLdA = TRANS ? MT * 2 : kStep * 2, kLdB = KT * 2;
  constexpr int kA = MT * kStep * 2, kRaw = KT * kStep, kB = KT * kStep * 2;
  constexpr int kLoadsA = kA / 1024 / kWaves;               // wave loads of 1024 bytes
  static_assert(kRaw == 16 * kT && kLoadsA * kWaves * 1024 == kA, "a lane's share");
  static_assert(64 * KT * 4 <= 4 * kA && WM == 2, "the sums of 64 rows fit in A's buffers");
  constexpr int kAtRaw = 4 * kA, kAtB = kAtRaw + 4 * kRaw, kAtSc = kAtB + 2 * kB;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kAtSc + 4 * 256];

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
  const int64_t s0 = min(steps, split * part), n = min(steps, s0 + part) - s0;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % WM, wk = wave / WM;

  // A's loads, in 16-byte pieces (its rows are whole pieces: a.lda is at least m or r rounded up to 8, with
  // zeros behind them): kRows rows of the stored tile per wave and instruction
  constexpr int kChunks = kLdA / 16, kRows = 64 / kChunks;
  uint32_t oa[kLoadsA];
  int ca[kLoadsA];  // not transposed: the lane's first r in the stage
#pragma unroll
  for (int i = 0; i < kLoadsA; i++) {
    const int row = (wave + kWaves * i) * kRows + lane / kChunks, p = lane % kChunks;
    const int c = TRANS ? ((((p >> 1) ^ turn(row)) << 1) | (p & 1)) : p ^ (row >> 2 & 3);
    oa[i] = (uint32_t)row * (uint32_t)(2 * a.lda) + 16u * c;
    ca[i] = 8 * c;
  }
  // B's loads: 16 codes per lane, which the same lane widens; its scales, one wave's load
  const int brow = threadIdx.x / (KT / 16), bcol = threadIdx.x % (KT / 16);
  const int nb = (int)(((int64_t)a.k + 127) >> 7);
  const bool f32 = a.b[0].f32;
  const int srow = lane & 31, sblock = min(nb - 1, (k0 >> 7) + min(lane >> 5, KT / 128 - 1));
  const uint32_t sc_at = 4u * (brow + 32 * (bcol >> 3));

  // The next stage to load, of A and of B: where it lies, and where it stands in the sum.
  struct CursorA {
    const uint16_t* p;  // transposed: the stage's first row; otherwise its first column
    int64_t r;
    int pair;
  };
  struct CursorB {
    const uint8_t* codes;
    const uint8_t* scales;
    int64_t ld, ld_scale, r;
    int pair;
  };
  const int esize = f32 ? 4 : 1;
  const int64_t a_step = TRANS ? kStep * a.lda : kStep, a_first = TRANS ? m0 : m0 * a.lda;
  auto a_of = [&](int pair, int64_t r) {
    return CursorA{(pair == 0 ? a.a[0] : pair == 1 ? a.a[1] : pair == 2 ? a.a[2] : a.a[3]) + a_first + r / kStep * a_step, r, pair};
  };
  auto b_of = [&](int pair, int64_t r) {
    const In8& m = pair == 0 ? a.b[0] : pair == 1 ? a.b[1] : pair == 2 ? a.b[2] : a.b[3];
    return CursorB{m.codes + r * m.ld, static_cast<const uint8_t*>(m.scales) + r * m.ld_scale * esize, m.ld, m.ld_scale, r, pair};
  };
  auto next_a = [&](CursorA& c) {
    c.r += kStep;
    c.p += a_step;
    if (c.r >= a.r) c = a_of(c.pair + 1, 0);
  };
  auto next_b = [&](CursorB& c) {
    c.r += kStep;
    c.codes += kStep * c.ld;
    c.scales += kStep * c.ld_scale * esize;
    if (c.r >= a.r) c = b_of(c.pair + 1, 0);
  };
  // Behind the last pair nothing is there: resources of no bytes, zeros.
  const int64_t a_width = TRANS ? (min((int64_t)MT, a.m - m0) + 7) & ~(int64_t)7 : 0;
  const int64_t a_rows = TRANS ? 0 : (min((int64_t)MT, a.m - m0) - 1) * a.lda;
  auto load_a = [&](uint8_t* buf, const CursorA& c) {
    const int64_t bytes = 2 * (TRANS ? (min((int64_t)kStep, a.r - c.r) - 1) * a.lda + a_width : a_rows + ((a.r - c.r + 7) & ~(int64_t)7));
    const vu4 r = rsrc4(c.p, c.pair < a.npairs ? bytes : 0);
#pragma unroll
    for (int i = 0; i < kLoadsA; i++)  // not transposed: columns behind the sum's end lie outside the resource too
      load_lds(r, buf + (wave + kWaves * i) * 1024, TRANS || c.r + ca[i] < a.r ? oa[i] : 0x7FFFFF00u, 0);
  };
  auto load_b = [&](int slot, const CursorB& c) {
    const int64_t rows = c.pair < a.npairs ? min((int64_t)kStep, a.r - c.r) : 0;
    load_lds(rsrc4(c.codes, rows > 0 ? (rows - 1) * c.ld + 128 * (int64_t)nb : 0), lds + kAtRaw + slot * kRaw + wave * 1024,
             (uint32_t)brow * (uint32_t)c.ld + k0 + 16 * bcol, 0);
    if (wave == slot)  // the waves in turn; the one whose turn it is waits for one load more than it has to
      load_lds_scalars(rsrc4(c.scales, rows > 0 ? ((rows - 1) * c.ld_scale + nb) * esize : 0), lds + kAtSc + slot * 256,
                       (uint32_t)(srow * (uint32_t)c.ld_scale + sblock) * esize, f32);
  };
  auto widen_b = [&](int slot, int to) {
    const uint32_t sb = *reinterpret_cast<const uint32_t*>(lds + kAtSc + slot * 256 + sc_at);
    vu4 w[2];
    widen<BF>(*reinterpret_cast<const vu4*>(lds + kAtRaw + slot * kRaw + 16 * threadIdx.x), __uint_as_float(f32 ? sb : sb << 23), w);
    uint8_t* d = lds + kAtB + to * kB + brow * kLdB + 32 * (bcol ^ turn(brow));
    // lanes eight apart have the same banks: each half of them begins with another half of the unit
    const int h = bcol >> 3 & 1;
    *reinterpret_cast<vu4*>(d + 16 * h) = h ? w[1] : w[0];
    *reinterpret_cast<vu4*>(d + 16 * (h ^ 1)) = h ? w[0] : w[1];
  };

  // fragments: groups of 16 lanes take 16 columns and four of the rows; lanes 32 .. 63 the second eight r
  const int g = lane >> 5, fr = lane & 31;
  const int trow = 8 * g + (lane >> 2 & 3), unit0 = lane >> 4 & 1;
  uint32_t fa[kI], fb[kJ];
#pragma unroll
  for (int i = 0; i < kI; i++)
    fa[i] = TRANS ? trow * kLdA + 32 * ((2 * (kI * wm + i) + unit0) ^ turn(trow)) + 8 * (lane & 3)
                  : ((MT / WM) * wm + 32 * i + fr) * kLdA;
#pragma unroll
  for (int j = 0; j < kJ; j++) fb[j] = trow * kLdB + 32 * ((2 * (kJ * wk + j) + unit0) ^ turn(trow)) + 8 * (lane & 3);

  vf16_t acc[kI][kJ];
#pragma unroll
  for (int i = 0; i < kI; i++)
#pragma unroll
    for (int j = 0; j < kJ; j++) acc[i][j] = vf16_t{};

  auto compute = [&](const uint8_t* A, const uint8_t* B) {
#pragma unroll
    for (int h = 0; h < kStep / 16; h++) {
      v8bf b[kJ];
#pragma unroll
      for (int j = 0; j < kJ; j++) b[j] = tr_frag<kLdB>(B + 16 * h * kLdB, fb[j]);
#pragma unroll
      for (int i = 0; i < kI; i++) {
        v8bf x;
        if constexpr (TRANS) x = tr_frag<kLdA>(A + 16 * h * kLdA, fa[i]);
        else x = *reinterpret_cast<const v8bf*>(A + fa[i] + 16 * ((2 * h + g) ^ (fr >> 2 & 3)));
#pragma unroll
        for (int j = 0; j < kJ; j++)  // rows of D: four consecutive k per lane
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], x, acc[i][j], 0, 0, 0);
      }
    }
  };

  if (n > 0) {
    const int pair = a.npairs > 1 ? (int)(s0 / spp) : 0;
    CursorA at_a = a_of(pair, (s0 - pair * spp) * kStep);
    CursorB at_b = b_of(pair, (s0 - pair * spp) * kStep);
    load_b(0, at_b), next_b(at_b);
#pragma unroll
    for (int s = 0; s < 3; s++) {
      load_a(lds + s * kA, at_a), next_a(at_a);
      load_b(s + 1, at_b), next_b(at_b);
    }
    constexpr int kLoads = kLoadsA + 1;  // of a stage, at least
    stage_barrier<3 * kLoads>();
    widen_b(0, 0);
    auto one = [&](int64_t s, auto which) {
      constexpr int S = decltype(which)::value;
      if (s + S >= n) return;
      // A's rows of this stage and B's codes of the next are there, two stages may be on their way; this one's
      // widened codes are written, and what the stage before read is free
      stage_barrier<2 * kLoads>();
      load_a(lds + (S + 3) % 4 * kA, at_a), next_a(at_a);
      load_b(S, at_b), next_b(at_b);
      widen_b((S + 1) % 4, (S + 1) % 2);
      compute(lds + S * kA, lds + kAtB + S % 2 * kB);
    };
    for (int64_t s = 0; s < n; s += 4) {
      one(s, std::integral_constant<int, 0>{});
      one(s, std::integral_constant<int, 1>{});
      one(s, std::integral_constant<int, 2>{});
      one(s, std::integral_constant<int, 3>{});
    }
    wait_loads();
  }

  // 32 rows of each of the two waves along m at a time, KT sums a row whose 16-byte units lie in the order
  // unit ^ (row & 15)
  const int64_t ldp = ((int64_t)a.k + 3) & ~(int64_t)3;
  constexpr int kUnits = KT / 4, kRowsOut = kT / kUnits;  // rows that the work-group takes at a time
#pragma unroll 1
  for (int i = 0; i < kI; i++) {
    __syncthreads();
    auto put = [&](auto which) {
      constexpr int I = decltype(which)::value;
      if constexpr (I < kI) {
        if (i == I) {
#pragma unroll
          for (int j = 0; j < kJ; j++)
#pragma unroll
            for (int r = 0; r < 4; r++) {
              const int unit = (KT / WK * wk + 32 * j + 8 * r) / 4 + g;
              const vf16_t& v = acc[I][j];
              *reinterpret_cast<vf4_t*>(lds + (32 * wm + fr) * (KT * 4) + 16 * (unit ^ (fr & 15))) =
                  vf4_t{v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
            }
        }
      }
    };
    put(std::integral_constant<int, 0>{});
    put(std::integral_constant<int, 1>{});
    put(std::integral_constant<int, 2>{});
    put(std::integral_constant<int, 3>{});
    const int unit = threadIdx.x % kUnits, k = k0 + 4 * unit, left = a.k - k;
    auto row_of = [&](int q) { return m0 + (MT / WM) * (q >> 5) + 32 * i + (q & 31); };
    float old[64 / kRowsOut][4];
    if (a.accumulate && !a.partial) {
#pragma unroll
      for (int e = 0; e < 64 / kRowsOut; e++) {
        const int64_t m = row_of((int)threadIdx.x / kUnits + e * kRowsOut);
        ld4(a.out_dt, a.out, m * a.ld_out + k, m < a.m ? left : 0, old[e]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 64 / kRowsOut; e++) {
      const int q = (int)threadIdx.x / kUnits + e * kRowsOut;
      const int64_t m = row_of(q);
      if (m >= a.m || left <= 0) continue;
      const vf4_t v = *reinterpret_cast<const vf4_t*>(lds + q * (KT * 4) + 16 * (unit ^ (q & 15)));
      float x[4] = {v.x, v.y, v.z, v.w};
      if (a.partial) {
        st_global<vu4>(a.partial + ((int64_t)split * a.m + m) * ldp + k, pack4<FP8ADAM_F32>(x).x);
      } else {
        if (a.accumulate) {
#pragma unroll
          for (int c = 0; c < 4; c++) x[c] += old[e][c];
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
