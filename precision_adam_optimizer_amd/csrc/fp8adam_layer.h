// fp8adam_layer.h -- what the kernels of the layer operators (include/fp8adam_layer.h)
// share: typed rows, activations, blocks of 128 columns in 8 bits, direct loads into
// shared memory, and the launch functions between their translation units.
#pragma once

#include "../../include/fp8adam_layer.h"
#include "fp8adam_list.h"

namespace fp8adam_layer {

using namespace fp8adam;
using namespace fp8adam_engine;
using fp8adam_list::codes4_pow2;
using fp8adam_list::dtype_bytes;
using fp8adam_list::ld_elem;
using fp8adam_list::nonfinite_amax;
using fp8adam_list::pack4;
using fp8adam_list::Raw4;
using fp8adam_list::st_elem;
using fp8adam_list::unpack4;
using fp8adam_list::vu2_any;
using fp8adam_list::vu4_any;

typedef float vf4_t __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------- typed rows

// Up to four consecutive elements from `base` on, of which `n` exist (none if n <= 0; zeros
// for the others), at any address of the element's alignment.
template <int DT>
__device__ __forceinline__ void ld4(const void* base, int64_t i, int64_t n, float (&x)[4]) {
  if (n >= 4) {
    const char* p = static_cast<const char*>(base) + dtype_bytes(DT) * i;
    if constexpr (DT == FP8ADAM_F32) unpack4<DT>(Raw4<DT>{ld_global<vu4_any>(p)}, x);
    else unpack4<DT>(Raw4<DT>{ld_global<vu2_any>(p)}, x);
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = j < n ? ld_elem<DT>(base, i + j) : 0.0f;
  }
}

template <int DT>
__device__ __forceinline__ void st4(void* base, int64_t i, int64_t n, const float (&x)[4]) {
  if (n >= 4) {
    char* p = static_cast<char*>(base) + dtype_bytes(DT) * i;
    if constexpr (DT == FP8ADAM_F32) st_global<vu4_any>(p, pack4<DT>(x).x);
    else st_global<vu2_any>(p, pack4<DT>(x).x);
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (j < n) st_elem<DT>(base, i + j, x[j]);
  }
}

typedef vu4 __attribute__((aligned(2))) vu4_any2;

template <int DT>
__device__ __forceinline__ void ld8(const void* base, int64_t i, int64_t n, float (&x)[8]) {
  float a[4], b[4];
  if (DT != FP8ADAM_F32 && n >= 8) {
    constexpr int D = DT == FP8ADAM_F32 ? FP8ADAM_BF16 : DT;
    const vu4 w = ld_global<vu4_any2>(static_cast<const char*>(base) + 2 * i);
    unpack4<D>(Raw4<D>{vu2{w.x, w.y}}, a);
    unpack4<D>(Raw4<D>{vu2{w.z, w.w}}, b);
  } else {
    ld4<DT>(base, i, n, a);
    ld4<DT>(base, i + 4, n - 4, b);
  }
#pragma unroll
  for (int j = 0; j < 4; j++) x[j] = a[j], x[4 + j] = b[j];
}

template <int DT>
__device__ __forceinline__ void st8(void* base, int64_t i, int64_t n, const float (&x)[8]) {
  const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
  if (DT != FP8ADAM_F32 && n >= 8) {
    constexpr int D = DT == FP8ADAM_F32 ? FP8ADAM_BF16 : DT;
    const vu2 p = pack4<D>(a).x, q = pack4<D>(b).x;
    st_global<vu4_any2>(static_cast<char*>(base) + 2 * i, vu4{p.x, p.y, q.x, q.y});
  } else {
    st4<DT>(base, i, n, a);
    st4<DT>(base, i + 4, n - 4, b);
  }
}

// The same with the type known at run time (the same in every lane).
__device__ __forceinline__ void ld4(int dt, const void* base, int64_t i, int64_t n, float (&x)[4]) {
  if (dt == FP8ADAM_F32) ld4<FP8ADAM_F32>(base, i, n, x);
  else if (dt == FP8ADAM_BF16) ld4<FP8ADAM_BF16>(base, i, n, x);
  else ld4<FP8ADAM_F16>(base, i, n, x);
}
__device__ __forceinline__ void st4(int dt, void* base, int64_t i, int64_t n, const float (&x)[4]) {
  if (dt == FP8ADAM_F32) st4<FP8ADAM_F32>(base, i, n, x);
  else if (dt == FP8ADAM_BF16) st4<FP8ADAM_BF16>(base, i, n, x);
  else st4<FP8ADAM_F16>(base, i, n, x);
}

__device__ __forceinline__ void ld8(int dt, const void* base, int64_t i, int64_t n, float (&x)[8]) {
  if (dt == FP8ADAM_F32) ld8<FP8ADAM_F32>(base, i, n, x);
  else if (dt == FP8ADAM_BF16) ld8<FP8ADAM_BF16>(base, i, n, x);
  else ld8<FP8ADAM_F16>(base, i, n, x);
}
__device__ __forceinline__ void st8(int dt, void* base, int64_t i, int64_t n, const float (&x)[8]) {
  if (dt == FP8ADAM_F32) st8<FP8ADAM_F32>(base, i, n, x);
  else if (dt == FP8ADAM_BF16) st8<FP8ADAM_BF16>(base, i, n, x);
  else st8<FP8ADAM_F16>(base, i, n, x);
}

// ------------------------------------------------------------------ activations

// e^x from the hardware's 2^x, with the rounding of x * log2 e put right to first order: within
// 2 ulp for |x| < 87.3 (2^126).  Beyond that it is 0, Inf or, without the correction, which would be Inf * 0, within
// 2^-17: sigmoid(z) and e^(-z^2/2) are below the normal numbers there, or 1 is added.
__device__ __forceinline__ float exp_of(float x) {
  constexpr float kL = 1.44269502f, kLlo = 1.92596303e-8f, kLn2 = 0.693147182f;  // log2 e in two parts
  const float t = x * kL;
  const float e = __builtin_amdgcn_exp2f(t);
  const float r = __builtin_fmaf(x, kLlo, __builtin_fmaf(x, kL, -t));
  return __builtin_fabsf(t) < 126.0f ? __builtin_fmaf(e, r * kLn2, e) : e;
}

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_of(-z)); }

// The normal distribution's Phi(z), and e^(-z^2/2): erfc by Abramowitz and Stegun's formula
// 7.1.26 (|error| <= 1.5e-7) on e^(-x^2), x = |z| / sqrt 2.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float x = __builtin_fabsf(z) * 0.707106781f;
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.0f));
  float p = __builtin_fmaf(t, 1.061405429f, -1.453152027f);
  p = __builtin_fmaf(t, p, 1.421413741f);
  p = __builtin_fmaf(t, p, -0.284496736f);
  p = __builtin_fmaf(t, p, 0.254829592f);
  e = exp_of(-0.5f * z * z);
  const float tail = 0.5f * t * p * e;  // Phi(-|z|)
  return z < 0.0f ? tail : 1.0f - tail;
}

// act(z) and act'(z).  A NaN stays one; act of an infinite z is what the formula gives (NaN for
// silu and gelu of -Inf).
template <int ACT>
__device__ __forceinline__ float act(float z) {
  if constexpr (ACT == FP8ADAM_ACT_RELU) return z > 0.0f ? z : z != z ? z : 0.0f;
  if constexpr (ACT == FP8ADAM_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == FP8ADAM_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  return z;
}

template <int ACT>
__device__ __forceinline__ void act_slope(float z, float& a, float& da) {
  if constexpr (ACT == FP8ADAM_ACT_SILU) {
    const float p = sigmoid(z);
    a = z * p;
    da = __builtin_fmaf(a, 1.0f - p, p);
  } else if constexpr (ACT == FP8ADAM_ACT_GELU) {
    float e;
    const float p = normal_cdf(z, e);
    a = z * p;
    da = __builtin_fmaf(z * 0.398942280f, e, p);
  } else {
    a = act<ACT>(z);
    da = ACT == FP8ADAM_ACT_NONE || z > 0.0f ? 1.0f : z != z ? z : 0.0f;
  }
}

// With the activation known at run time (the same in every lane).
template <int N, int M>
__device__ __forceinline__ void act_all(int which, float (&z)[N][M]) {
  auto all = [&](auto f) {
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
      for (int j = 0; j < M; j++) z[i][j] = f(z[i][j]);
  };
  if (which == FP8ADAM_ACT_RELU) all(act<FP8ADAM_ACT_RELU>);
  else if (which == FP8ADAM_ACT_SILU) all(act<FP8ADAM_ACT_SILU>);
  else if (which == FP8ADAM_ACT_GELU) all(act<FP8ADAM_ACT_GELU>);
}

// -------------------------------------------------------- blocks of 128 in 8 bits

// Where a matrix in 8 bits with E8M0 scales is written.  codes null: nowhere.
struct Out8 {
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld, ld_scale;
  int32_t format;
};

// The largest of 16 lanes in each of them: maxima with fused DPP operands.
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));   // quad_perm [1,0,3,2]
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));   // quad_perm [2,3,0,1]
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, true));  // row_half_mirror
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, true));  // row_mirror
}

// choose_scale's POW2 scale as its exponent's byte, without branches: a subnormal amax comes out at the
// lower limit by itself.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int k = (int)(amax >> 23) + (1 - Format<FMT>::kMaxExp) + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  const int byte = min(max(k, 1), 253);
  return amax - 1u < 0x7F7FFFFFu ? (uint32_t)byte : 127u;  // zero, Inf and NaN: 1
}

// N blocks that 16 lanes hold, eight consecutive values each (zeros behind the row's end, whose
// codes are zeros): their codes and scales to column 128 * block[i] of row[i] where `there`.  `lane` is the
// lane among the 16, all of which come here and agree on the rest.
template <int FMT, int N>
__device__ __forceinline__ void put_blocks_as(const Out8& o, const int64_t (&row)[N], const int64_t (&block)[N], const bool (&there)[N],
                                              int lane, const float (&x)[N][8]) {
  uint32_t am[N], byte[N];
  vu2 codes[N];
  bool any = false;
#pragma unroll
  for (int i = 0; i < N; i++) {
    am[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) am[i] = max(am[i], abs_bits(x[i][j]));
  }
#pragma unroll
  for (int i = 0; i < N; i++) {
    am[i] = row_max(am[i]);
    byte[i] = scale_byte<FMT>(am[i]);
    const float s = __uint_as_float(byte[i] << 23);
    const float lo[4] = {x[i][0], x[i][1], x[i][2], x[i][3]}, hi[4] = {x[i][4], x[i][5], x[i][6], x[i][7]};
    codes[i] = vu2{codes4_pow2<FMT>(lo, s, false), codes4_pow2<FMT>(hi, s, false)};
    any = any || nonfinite_amax(am[i]);
  }
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(any) != 0, 0)) {  // uniform: one test for the wave
#pragma unroll
    for (int i = 0; i < N; i++) {
      const float lo[4] = {x[i][0], x[i][1], x[i][2], x[i][3]}, hi[4] = {x[i][4], x[i][5], x[i][6], x[i][7]};
      if (nonfinite_amax(am[i])) codes[i] = vu2{codes4_pow2<FMT>(lo, 1.0f, true), codes4_pow2<FMT>(hi, 1.0f, true)};
    }
  }
#pragma unroll
  for (int i = 0; i < N; i++)
    if (there[i]) st_global<vu2>(o.codes + row[i] * o.ld + 128 * block[i] + 8 * lane, codes[i]);
#pragma unroll
  for (int i = 0; i < N; i++)
    if (there[i] && lane == 0) st_global<uint8_t>(o.scales + row[i] * o.ld_scale + block[i], (uint8_t)byte[i]);
}
template <int N>
__device__ __forceinline__ void put_blocks(const Out8& o, const int64_t (&row)[N], const int64_t (&block)[N], const bool (&there)[N],
                                           int lane, const float (&x)[N][8]) {
  if (o.format == FP8ADAM_E4M3) put_blocks_as<0, N>(o, row, block, there, lane, x);
  else put_blocks_as<1, N>(o, row, block, there, lane, x);
}

// The scale of block `block` of row `row`.
__device__ __forceinline__ float scale_at(const void* scales, int64_t i, bool f32) {
  return f32 ? ld_global<float>(static_cast<const float*>(scales) + i)
             : __uint_as_float((uint32_t)ld_global<uint8_t>(static_cast<const uint8_t*>(scales) + i) << 23);
}

// ------------------------------------------------- direct loads into shared memory

// A buffer resource as four scalars, for the loads below.
__device__ __forceinline__ vu4 rsrc4(const void* base, int64_t bytes) {
  const uint64_t p = (uint64_t)(uintptr_t)base;
  return vu4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p), (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32)),
             (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), (uint32_t)kRawBufferWord3};
}

// 16 bytes per lane, to dst + 16 * lane (dst the same in every lane of the wave); lanes whose
// offset lies outside the resource write zeros.  In assembly (it has no register output), because the
// compiler waits for every such load it knows of before it reads shared memory; the kernels
// count them themselves (stage_barrier).  A write of m0 needs one wait state before the load.
__device__ __forceinline__ void load_lds(const vu4& r, const uint8_t* dst, uint32_t voffset, uint32_t soffset) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)dst;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)at)), "v"(voffset), "s"(r), "s"(soffset)
               : "memory", "m0");
}

// The same of one scale per lane, to dst + 4 * lane: a 32-bit number, or a byte widened to 32 bits.
__device__ __forceinline__ void load_lds_scalars(const vu4& r, const uint8_t* dst, uint32_t voffset, bool dwords) {
  const uint32_t at = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)dst);
  if (dwords)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" : : "s"(at), "v"(voffset), "s"(r) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, 0 offen lds" : : "s"(at), "v"(voffset), "s"(r) : "memory", "m0");
}

// The loads above are counted as vector memory loads: a barrier alone does not wait for them.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0)

// Between the stages of a pipeline in shared memory: at most N of this wave's loads are still on their way,
// its reads and writes of shared memory are done, and so are those of the other waves.  (A
// __syncthreads() would wait for every load.)
template <int N>
__device__ __forceinline__ void stage_barrier() {
  static_assert(N < 64, "the counter's six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);  // vmcnt(N), lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A barrier that waits for nothing else, and that nothing is moved across.
__device__ __forceinline__ void bare_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// ----------------------------------------------------------------- forward product

// A matrix in 8 bits that is read.
struct In8 {
  const uint8_t* codes;
  const void* scales;
  int64_t ld, ld_scale;
  int32_t f32;  // scales in fp32
  int32_t pad;
};

struct ProductArgs {
  In8 x, w[2];               // w[1]: the up projection
  int64_t tokens;
  int32_t rows, cols;
  const void* xin;           // the kernel for few tokens packs x itself (as x8), or null
  int64_t xin_ld;
  Out8 x8;
  const void* bias;
  const void* res;
  void* y;
  int64_t res_ld, y_ld;
  Out8 y8, keep[2];
  int32_t act, xin_dt, bias_dt, res_dt, y_dt;
  int32_t tiles_n, tiles_t;
  int32_t exact;             // host: every product is added in 32 bits, whatever is written
};

// The kernel for few tokens, which keeps nothing in 8 bits (a block of 128 outputs spans its
// work-groups); with the fewest it packs x itself.
constexpr int kFewTokens = 64, kFewPackTokens = 4;
inline bool few_tokens(const ProductArgs& a) {
  return a.tokens <= kFewTokens && !a.keep[0].codes && !a.keep[1].codes && !a.y8.codes;
}
inline bool packs_itself(const ProductArgs& a, const fp8adam_matrix& x) {  // rows of whole dwords
  const int64_t e = dtype_bytes(x.dtype);
  return few_tokens(a) && a.tokens <= kFewPackTokens && (uintptr_t)x.data % 4 == 0 && a.cols * e % 4 == 0 &&
         (a.tokens == 1 || x.ld * e % 4 == 0);
}

template <int XF, int WF>
int launch_product(const ProductArgs& a, bool gated, hipStream_t s);

// ------------------------------------------------------------------------ gradients

// out[m][k] (+)= sum over pairs and r of A(m, r) B[r][k]: A in bf16, stored [r][m] (trans) or
// [m][r], rows 16-byte aligned and whole multiples of 8 elements (zeros behind the last); B in 8 bits.
constexpr int kMaxParts = 3, kMaxPairs = 2 * kMaxParts;  // of a gradient, and of two layers
struct GradArgs {
  const uint16_t* a[kMaxPairs];
  int64_t lda;               // the same for all pairs
  In8 b[kMaxPairs];
  int32_t npairs;
  int32_t trans;
  int64_t m, r;              // rows of out, length of the sum
  int32_t k;                 // columns of out
  int32_t out_dt, accumulate;
  void* out;
  int64_t ld_out;
  float* partial;            // [splits][m][k rounded up to 4], or null
};

// The kernel's tile, and into how many parts the sum is split (1: no partials).
struct GradPlan {
  int tile;                  // 0: 256 x 256, 1: 128 x 128
  int splits;
  int64_t partial_bytes;
};
GradPlan plan_grad(int64_t m, int64_t k, int64_t r, int npairs);
template <int BF>
int launch_grad(const GradArgs& a, const GradPlan& p, hipStream_t s);

}  // namespace fp8adam_layer
