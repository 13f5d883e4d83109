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

// Rows of a tile along the sum, LD bytes long, lie in shared memory with their 32-byte units (16
// columns) in the order unit ^ turn(row): the rows that half a wave reads together, 0 .. 3 and
// 8 .. 11 of 16, lie on different banks.
template <int LD>
__device__ __forceinline__ int turn(int row) {
  return LD == 128 ? (row >> 1 & 1) | (row >> 2 & 2) : (row & 3) | (row >> 1 & 4);
}

// Eight r of a column: rows `row` .. row + 3 and row + 4 .. row + 7 through a lane's offset `off`.
template <int LD>
__device__ __forceinline__ v8bf tr_frag(const uint8_t* tile, uint32_t off) {
  const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TrPtr)(tile + off));
  const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TrPtr)(tile + off + 4 * LD));
  return __builtin_bit_cast(v8bf, v8s{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w});
}

// Sixteen codes times their scale, in bf16 (exact, a code has at most four significant bits, but for what lies below 2^-133).
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

// A tile of MT x KT of out, waves two along m and WK along k, in products of 16 x 32 by 32 x 16.
//
// The sum goes in blocks of 64, each in two phases: the first multiplies the first half of
// each wave's rows of m by its columns, the second the second half by the same, which stay in
// registers.  A's halves and B's codes and scales go straight into shared memory, whole cache lines
// at a time, where each has two places; what a phase has read is loaded again three phases before it
// is read.  In a block's second phase the next block's codes are widened into the place that
// the first phase has read.
//
// With eight waves the two of a SIMD take turns: while waves 0 .. 3 multiply, waves 4 .. 7 read
// their operands from shared memory and the other way round, with a barrier at each turn.  (Phase p
// is read by the first waves in turn 2p and by the others in 2p + 1; what either does in its part of
// phase p + 1 comes after that.)  With four, two work-groups share a CU.
//
// The sums then go through shared memory into whole rows of the tile, so that whole lines are
// read (accumulate) and written.
//
// Measured: 4096 tokens x 11008 x 4096 added to fp32 in 434 us (850 TFLOP/s; the gradient's 360 MB alone
// take 61), the input's gradient of two such layers in 673 (1100; the library's product of bf16 by bf16
// reaches 1224 of 8192^3); of fp32 gradients, three terms each, in 1148 and 1978.  There the matrix cores are busy 45% of the time and shared memory's reads 31%
// (a fifth of that conflicts of the transposing ones): a turn takes about 1040 cycles, of which its
// products need 512 and the other waves' 64 KB of reads as many, behind the issue of the loads and
// before the barrier.  Blocks of 32 in two buffers took 669 us, and in four with half lines 740.
template <bool TRANS, int BF, int MT, int KT, int WK>
__global__ __launch_bounds__(128 * WK, 2) void k_grad(const GradArgs a, int splits, int tiles_m, int tiles_k) {
  constexpr int kT = 128 * WK, kWaves = 2 * WK;
  constexpr bool TURNS = kWaves == 8;
  constexpr int kI = MT / 2 / 16, kJ = KT / WK / 16;        // products of a wave; kI / 2 of a phase
  constexpr int kHalf = MT / 2;                             // rows of m of a phase
  constexpr int kLdA = TRANS ? kHalf * 2 : kStep * 2, kLdB = KT * 2;
  constexpr int kA = kHalf * kStep * 2, kRaw = KT * kStep, kB = KT * kStep * 2;
  static_assert(kA == 2 * 1024 * kWaves && kRaw == 2 * 1024 * kWaves, "two loads of a wave each");
  constexpr int kAtRaw = 4 * kA, kAtB = kAtRaw + 2 * kRaw, kAtSc = kAtB + kB;
  static_assert(kHalf * KT * 4 <= kAtSc, "the sums of a phase's rows fit");
  __shared__ __attribute__((aligned(16))) uint8_t lds[kAtSc + 2 * 512];

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
  const int64_t part_len = (steps + splits - 1) / splits;
  const int64_t s0 = min(steps, split * part_len), n = min(steps, s0 + part_len) - s0;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WK, wk = wave % WK;  // (the first four of eight waves are those of the first rows)

  // A's loads, in 16-byte pieces (its rows are whole pieces: a.lda is at least m or r rounded up to 8, with
  // zeros behind them): kRows rows of the stored half per wave and instruction.  Row q of half `part` is row
  // kHalf / 2 * part + q of the tile for q < kHalf / 2, and as far into the second waves' rows behind that.
  constexpr int kChunks = kLdA / 16, kRows = 64 / kChunks;
  auto row_of = [](int part, int q) { return kHalf * (q / (kHalf / 2)) + kHalf / 2 * part + q % (kHalf / 2); };
  uint32_t oa[2][2];
  int ca[2];  // not transposed: the lane's first r in the block
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int row = (wave + kWaves * i) * kRows + lane / kChunks, p = lane % kChunks;
    const int c = TRANS ? ((((p >> 1) ^ turn<kLdA>(row)) << 1) | (p & 1)) : p ^ (row >> 1 & 7);
    ca[i] = 8 * c;
#pragma unroll
    for (int part = 0; part < 2; part++)
      oa[part][i] = TRANS ? (uint32_t)row * (uint32_t)(2 * a.lda) + 2u * row_of(part, 8 * c)
                          : (uint32_t)row_of(part, row) * (uint32_t)(2 * a.lda) + 16u * c;
  }
  // B's loads: twice 16 codes per lane, which the same lane widens; its scales, one wave's load
  constexpr int kColsB = KT / 16, kRowsB = kT / kColsB;
  const int brow = threadIdx.x / kColsB, bcol = threadIdx.x % kColsB;
  const int nb = (int)(((int64_t)a.k + 127) >> 7);
  const bool f32 = a.b[0].f32;

  // The next block to load, of either half of A and of B: where it lies, and where it stands in the sum.  (The step from
  // one pair to the next is kept out of the loop: between its loads the large products take 1 to 2% longer.)
  struct CursorA {
    const uint16_t* p;  // transposed: the block's first row; otherwise its first column
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
    return CursorA{(pair == 0 ? a.a[0] : pair == 1 ? a.a[1] : pair == 2 ? a.a[2] : pair == 3 ? a.a[3] : pair == 4 ? a.a[4] : a.a[5]) + a_first + r / kStep * a_step, r, pair};
  };
  auto b_of = [&](int pair, int64_t r) {
    const In8& m = pair == 0 ? a.b[0] : pair == 1 ? a.b[1] : pair == 2 ? a.b[2] : pair == 3 ? a.b[3] : pair == 4 ? a.b[4] : a.b[5];
    return CursorB{m.codes + r * m.ld, static_cast<const uint8_t*>(m.scales) + r * m.ld_scale * esize, m.ld, m.ld_scale, r, pair};
  };
  // Behind the last pair nothing is there: resources of no bytes, zeros.
  const int64_t a_width = TRANS ? (min((int64_t)MT, a.m - m0) + 7) & ~(int64_t)7 : 0;
  const int64_t a_rows = TRANS ? 0 : (min((int64_t)MT, a.m - m0) - 1) * a.lda;
  auto load_a = [&](int place, int part, CursorA& c) __attribute__((always_inline)) {
    const int64_t bytes = 2 * (TRANS ? (min((int64_t)kStep, a.r - c.r) - 1) * a.lda + a_width : a_rows + ((a.r - c.r + 7) & ~(int64_t)7));
    const vu4 r = rsrc4(c.p, c.pair < a.npairs ? bytes : 0);
#pragma unroll
    for (int i = 0; i < 2; i++)  // not transposed: columns behind the sum's end lie outside the resource too
      load_lds(r, lds + (2 * place + part) * kA + (wave + kWaves * i) * 1024, TRANS || c.r + ca[i] < a.r ? oa[part][i] : 0x7FFFFF00u, 0);
    c.r += kStep;
    c.p += a_step;
    if (__builtin_expect(c.r >= a.r, 0)) c = a_of(c.pair + 1, 0);
  };
  auto load_b = [&](int place, CursorB& c) __attribute__((always_inline)) {
    const int64_t rows = c.pair < a.npairs ? min((int64_t)kStep, a.r - c.r) : 0;
    const vu4 r = rsrc4(c.codes, rows > 0 ? (rows - 1) * c.ld + 128 * (int64_t)nb : 0);
#pragma unroll
    for (int i = 0; i < 2; i++)
      load_lds(r, lds + kAtRaw + place * kRaw + (wave + kWaves * i) * 1024, (uint32_t)(brow + kRowsB * i) * (uint32_t)c.ld + k0 + 16 * bcol, 0);
    if (wave < KT / 128)  // one block of 128 columns each; these waves wait for one load more than they have to
      load_lds_scalars(rsrc4(c.scales, rows > 0 ? ((rows - 1) * c.ld_scale + nb) * esize : 0), lds + kAtSc + place * 512 + 256 * wave,
                       (uint32_t)(lane * (uint32_t)c.ld_scale + min(nb - 1, (k0 >> 7) + wave)) * esize, f32);
    c.r += kStep;
    c.codes += kStep * c.ld;
    c.scales += kStep * c.ld_scale * esize;
    if (__builtin_expect(c.r >= a.r, 0)) c = b_of(c.pair + 1, 0);
  };
  auto widen_b = [&](int place) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int row = brow + kRowsB * i;
      const uint32_t sb = *reinterpret_cast<const uint32_t*>(lds + kAtSc + place * 512 + 256 * (bcol >> 3) + 4 * row);
      vu4 w[2];
      widen<BF>(*reinterpret_cast<const vu4*>(lds + kAtRaw + place * kRaw + 16 * (threadIdx.x + kT * i)), __uint_as_float(f32 ? sb : sb << 23), w);
      uint8_t* d = lds + kAtB + row * kLdB + 32 * (bcol ^ turn<kLdB>(row));
      // lanes eight apart have the same banks: each half of them begins with another half of the unit
      const int h = bcol >> 3 & 1;
      *reinterpret_cast<vu4*>(d + 16 * h) = h ? w[1] : w[0];
      *reinterpret_cast<vu4*>(d + 16 * (h ^ 1)) = h ? w[0] : w[1];
    }
  };

  // fragments: lane group g of 16 takes r = 8g .. 8g + 7 of 32 of one column or row each
  const int g = lane >> 4, fr = lane & 15;
  const int trow = 8 * g + (fr >> 2);
  uint32_t fb[kJ];
#pragma unroll
  for (int j = 0; j < kJ; j++) fb[j] = kAtB + trow * kLdB + 32 * ((kJ * wk + j) ^ turn<kLdB>(trow)) + 8 * (fr & 3);
  auto frag_a = [&](int place, int part, int i, int h) __attribute__((always_inline)) {
    const uint8_t* t = lds + (2 * place + part) * kA;
    if constexpr (TRANS)
      return tr_frag<kLdA>(t + 32 * h * kLdA, trow * kLdA + 32 * (((kI / 2) * wm + i) ^ turn<kLdA>(trow)) + 8 * (fr & 3));
    else
      return *reinterpret_cast<const v8bf*>(t + (kHalf / 2 * wm + 16 * i + fr) * kLdA + 16 * ((4 * h + g) ^ (fr >> 1)));
  };

  vf4_t acc[kI][kJ];
#pragma unroll
  for (int i = 0; i < kI; i++)
#pragma unroll
    for (int j = 0; j < kJ; j++) acc[i][j] = vf4_t{0, 0, 0, 0};

  if (n > 0) {
    const int pair = a.npairs > 1 ? (int)(s0 / spp) : 0;
    CursorA at0 = a_of(pair, (s0 - pair * spp) * kStep), at1 = at0;
    CursorB at_b = b_of(pair, (s0 - pair * spp) * kStep);
    load_b(0, at_b);
    load_a(0, 0, at0);
    load_a(0, 1, at1);
    load_b(1, at_b);
    load_a(1, 0, at0);
    stage_barrier<6>();
    widen_b(0);
    stage_barrier<6>();
    if (TURNS && wave >= 4) bare_barrier();
    v8bf b[kJ][2];
    auto one = [&](auto which) __attribute__((always_inline)) {
      constexpr int place = decltype(which)::value >> 1, part = decltype(which)::value & 1;
      if constexpr (part == 0) {
        load_a(place ^ 1, 1, at1);
        load_b(place, at_b);
#pragma unroll
        for (int j = 0; j < kJ; j++)
#pragma unroll
          for (int h = 0; h < 2; h++) b[j][h] = tr_frag<kLdB>(lds + 32 * h * kLdB, fb[j]);
      } else {
        load_a(place, 0, at0);
        widen_b(place ^ 1);
      }
      v8bf x[kI / 2][2];
#pragma unroll
      for (int i = 0; i < kI / 2; i++)
#pragma unroll
        for (int h = 0; h < 2; h++) x[i][h] = frag_a(place, part, i, h);
      stage_barrier<6>();  // the next phase's operands are there, this one's have been read
      if constexpr (TURNS) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int i = 0; i < kI / 2; i++)
#pragma unroll
          for (int j = 0; j < kJ; j++)  // rows of D: four consecutive k per lane
            acc[part * kI / 2 + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j][h], x[i][h], acc[part * kI / 2 + i][j], 0, 0, 0);
      if constexpr (TURNS) {
        // (keeps the products on this side of the barrier: they would be moved to where the sums are used next)
#pragma unroll
        for (int i = 0; i < kI / 2; i++)
#pragma unroll
          for (int j = 0; j < kJ; j++) asm volatile("" : "+v"(acc[part * kI / 2 + i][j]));
        __builtin_amdgcn_s_setprio(0);
        bare_barrier();
      }
    };
    for (int64_t s = 0; s < n; s += 2) {
      one(std::integral_constant<int, 0>{});
      one(std::integral_constant<int, 1>{});
      if (s + 1 >= n) break;
      one(std::integral_constant<int, 2>{});
      one(std::integral_constant<int, 3>{});
    }
    if (TURNS && wave < 4) bare_barrier();
    wait_loads();
  }

  // the sums of a phase's rows at a time, KT a row whose 16-byte units lie in the order unit ^ (row & 15)
  const int64_t ldp = ((int64_t)a.k + 3) & ~(int64_t)3;
  constexpr int kUnits = KT / 4, kRowsOut = kT / kUnits, kN = kHalf / kRowsOut;  // rows that the work-group takes at a time
  const int unit = threadIdx.x % kUnits, k = k0 + 4 * unit, left = a.k - k;
  auto rows_out = [&](auto which) __attribute__((always_inline)) {
    constexpr int part = decltype(which)::value;
    stage_barrier<63>();
#pragma unroll
    for (int i = 0; i < kI / 2; i++)
#pragma unroll
      for (int j = 0; j < kJ; j++)
        *reinterpret_cast<vf4_t*>(lds + (kHalf / 2 * wm + 16 * i + fr) * (KT * 4) + 16 * ((KT / WK / 4 * wk + 4 * j + g) ^ fr)) =
            acc[part * kI / 2 + i][j];
    stage_barrier<63>();
    if (left <= 0) return;
    constexpr int kBatch = kN < 8 ? kN : 8;
#pragma unroll 1
    for (int e0 = 0; e0 < kN; e0 += kBatch) {
      float old[kBatch][4];
      const bool adds = a.accumulate && !a.partial;
      if (adds) {
#pragma unroll
        for (int e = 0; e < kBatch; e++) {
          const int64_t m = m0 + row_of(part, (int)threadIdx.x / kUnits + (e0 + e) * kRowsOut);
          ld4(a.out_dt, a.out, m * a.ld_out + k, m < a.m ? left : 0, old[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < kBatch; e++) {
        const int q = (int)threadIdx.x / kUnits + (e0 + e) * kRowsOut;
        const int64_t m = m0 + row_of(part, q);
        if (m >= a.m) continue;
        const vf4_t v = *reinterpret_cast<const vf4_t*>(lds + q * (KT * 4) + 16 * (unit ^ (q & 15)));
        float x[4] = {v.x, v.y, v.z, v.w};
        if (a.partial) {
          st_global<vu4>(a.partial + ((int64_t)split * a.m + m) * ldp + k, pack4<FP8ADAM_F32>(x).x);
        } else {
          if (adds) {
#pragma unroll
            for (int c = 0; c < 4; c++) x[c] += old[e][c];
          }
          st4(a.out_dt, a.out, m * a.ld_out + k, left, x);
        }
      }
    }
  };
  rows_out(std::integral_constant<int, 0>{});
  rows_out(std::integral_constant<int, 1>{});
}

// out (+)= the sum of the parts, in their order.
static __global__ __launch_bounds__(kThreads) void k_grad_join(const GradArgs a, int splits) {
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

template <int BF, int MT, int KT, int WK>
int launch_grad_tile(const GradArgs& a, const GradPlan& p, hipStream_t s) {
  const int64_t tm = (a.m + MT - 1) / MT, tk = (a.k + KT - 1) / KT, total = tm * tk * p.splits;
  if (total > (int64_t)(UINT32_MAX / (128 * WK)) - 8) return fail(FP8ADAM_EINVAL, "too many tokens for one call");
  const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(128 * WK);
  int r = a.trans ? launch(k_grad<true, BF, MT, KT, WK>, grid, block, 0, s, a, p.splits, (int)tm, (int)tk)
                  : launch(k_grad<false, BF, MT, KT, WK>, grid, block, 0, s, a, p.splits, (int)tm, (int)tk);
  if (r || p.splits == 1) return r;
  const int64_t threads = a.m * (((int64_t)a.k + 3) >> 2);
  return launch(k_grad_join, dim3((unsigned)((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a, p.splits);
}

template <int BF>
int launch_grad(const GradArgs& a, const GradPlan& p, hipStream_t s) {
  return p.tile == 0 ? launch_grad_tile<BF, 256, 256, 4>(a, p, s) : launch_grad_tile<BF, 128, 128, 2>(a, p, s);
}

}  // namespace fp8adam_layer
