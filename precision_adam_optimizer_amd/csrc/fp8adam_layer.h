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
using fp8adam_list::half_wave_max;
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

// ------------------------------------------------------------------ activations

// e^x from the hardware's 2^x, with the rounding of x * log2 e put right to first order: within
// 2 ulp.  Out of its range it is 0 or Inf (and without the correction, which would be Inf * 0).
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
__device__ __forceinline__ void act4(int which, float (&z)[4]) {
#pragma unroll
  for (int j = 0; j < 4; j++) {
    if (which == FP8ADAM_ACT_RELU) z[j] = act<FP8ADAM_ACT_RELU>(z[j]);
    else if (which == FP8ADAM_ACT_SILU) z[j] = act<FP8ADAM_ACT_SILU>(z[j]);
    else if (which == FP8ADAM_ACT_GELU) z[j] = act<FP8ADAM_ACT_GELU>(z[j]);
  }
}

// -------------------------------------------------------- blocks of 128 in 8 bits

// Where a matrix in 8 bits with E8M0 scales is written.  codes null: nowhere.
struct Out8 {
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld, ld_scale;
  int32_t format;
};

// The block that 32 lanes hold, four consecutive values each (zeros behind the row's end, whose
// codes are zeros): its codes and its scale to column 128 * block of a row.  `lane` is the lane
// in the half-wave; all 32 come here.
template <int FMT>
__device__ __forceinline__ void put_block(const Out8& o, int64_t row, int64_t block, int lane, const float (&x)[4]) {
  uint32_t am = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) am = max(am, abs_bits(x[j]));
  am = half_wave_max(am);
  float s, inv;
  choose_scale<FMT, 0>(am, s, inv);
  st_global<uint32_t>(o.codes + row * o.ld + 128 * block + 4 * lane, codes4_pow2<FMT>(x, s, nonfinite_amax(am)));
  if (lane == 0) st_global<uint8_t>(o.scales + row * o.ld_scale + block, (uint8_t)(__float_as_uint(s) >> 23));
}
__device__ __forceinline__ void put_block(const Out8& o, int64_t row, int64_t block, int lane, const float (&x)[4]) {
  if (o.format == FP8ADAM_E4M3) put_block<0>(o, row, block, lane, x);
  else put_block<1>(o, row, block, lane, x);
}

// The scale of block `block` of row `row`.
__device__ __forceinline__ float scale_at(const void* scales, int64_t i, bool f32) {
  return f32 ? ld_global<float>(static_cast<const float*>(scales) + i)
             : __uint_as_float((uint32_t)ld_global<uint8_t>(static_cast<const uint8_t*>(scales) + i) << 23);
}

// ------------------------------------------------- direct loads into shared memory

typedef __attribute__((address_space(3))) void* LdsPtr;

// 16 bytes per lane, to dst + 16 * lane (dst the same in every lane of the wave); lanes whose
// offset lies outside the resource write zeros.
__device__ __forceinline__ void load_lds(Rsrc r, uint8_t* dst, uint32_t voffset, uint32_t soffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (LdsPtr)dst, 16, voffset, soffset, 0, 0);
}

// The loads above are counted as vector memory loads: a barrier alone does not wait for them.
__device__ __forceinline__ void wait_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }  // vmcnt(0)

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
};

// The kernel for few tokens, which keeps nothing in 8 bits (a block of 128 outputs spans its
// work-groups); with the fewest it packs x itself.
constexpr int kFewTokens = 64, kFewPackTokens = 16;
inline bool few_tokens(const ProductArgs& a) {
  return a.tokens <= kFewTokens && !a.keep[0].codes && !a.keep[1].codes && !a.y8.codes;
}
inline bool packs_itself(const ProductArgs& a) { return few_tokens(a) && a.tokens <= kFewPackTokens; }

template <int XF, int WF>
int launch_product(const ProductArgs& a, bool gated, hipStream_t s);

// ------------------------------------------------------------------------ gradients

// out[m][k] (+)= sum over pairs and r of A(m, r) B[r][k]: A in bf16, stored [r][m] (trans) or
// [m][r], rows 16-byte aligned and whole multiples of 8 elements (zeros behind the last); B in 8 bits.
constexpr int kMaxPairs = 4;
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
