// fp8adam_list.h -- kernels of the list operators (include/fp8adam_list.h) and
// the plan they run from, shared by the translation units that instantiate the
// AdamW kernels (one for 32-bit moments, one per format pair for 8-bit ones)
// and by fp8adam_list.hip, which holds the C ABI.
//
// A plan cuts every tensor into parts of a fixed number of elements and keeps
// one table (part -> tensor) for each kind of tensor in the list: a kind is a
// combination of types, and has a kernel instantiation and a launch of its own.
// A work-group owns one part and finds its tensor's descriptor through the
// table.
#pragma once

#include <utility>
#include <vector>

#include "../../include/fp8adam_list.h"
#include "fp8adam_engine.h"

namespace fp8adam_list {

using namespace fp8adam;
using namespace fp8adam_engine;

// --------------------------------------------------------------- typed elements

template <int DT> struct Elem { using T = float; };
template <> struct Elem<FP8ADAM_BF16> { using T = uint16_t; };
template <> struct Elem<FP8ADAM_F16> { using T = uint16_t; };

constexpr int64_t dtype_bytes(int dt) { return dt == FP8ADAM_F32 ? 4 : 2; }

typedef float vf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int DT>
__device__ __forceinline__ float ld_elem(const void* base, int64_t i) {
  if constexpr (DT == FP8ADAM_F32) return ld_global<float>(static_cast<const float*>(base) + i);
  const uint16_t x = ld_global<uint16_t>(static_cast<const uint16_t*>(base) + i);
  if constexpr (DT == FP8ADAM_BF16) return __uint_as_float((uint32_t)x << 16);
  return (float)__builtin_bit_cast(_Float16, x);
}

// To fp16 from a value that has been rounded to fp32: without the empty asm
// statement the compiler folds the product or sum before it into one instruction
// that rounds only to fp16 (v_fma_mixlo_f16), and a copy would not be that of the
// fp32 weight.
__device__ __forceinline__ _Float16 to_f16(float x) {
  asm("" : "+v"(x));
  return (_Float16)x;
}

// To nearest even (v_cvt_pk_bf16_f32, v_cvt_f16_f32).
template <int DT>
__device__ __forceinline__ void st_elem(void* base, int64_t i, float x) {
  if constexpr (DT == FP8ADAM_F32) st_global<float>(static_cast<float*>(base) + i, x);
  else if constexpr (DT == FP8ADAM_BF16)
    st_global<uint16_t>(static_cast<uint16_t*>(base) + i, __builtin_bit_cast(uint16_t, (__bf16)x));
  else st_global<uint16_t>(static_cast<uint16_t*>(base) + i, __builtin_bit_cast(uint16_t, to_f16(x)));
}

// The codes of four values, to nearest even, saturating, where a NaN stays one
// (the clamp of encode4 alone would make it -FMAX).  `odd`: the values' block or
// tensor holds a NaN or Inf, which its amax tells; without one the test is not
// made.
template <int FMT>
__device__ __forceinline__ uint32_t encode4_nan(const float (&x)[4], bool odd) {
  uint32_t w = encode4<FMT>(x[0], x[1], x[2], x[3]);
  if (odd) {
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (x[j] != x[j]) w |= 0x7Fu << (8 * j);  // a NaN code in both formats
  }
  return w;
}

__device__ __forceinline__ bool nonfinite_amax(uint32_t amax_bits) { return amax_bits >= 0x7F800000u; }

// ------------------------------------------------------------------------ AdamW

struct AdamwDesc {
  void* p;
  const void* g;
  void* copy;
  void* m;
  void* v;
  float* sm;
  float* sv;
  int64_t numel;
  int64_t part0;   // the tensor's first part in its kind's table
  int32_t group;
  int32_t pad;
};

// One parameter group's constants, computed on the host from its hyperparameters.
struct GroupConsts {
  float b1, omb1, b2, omb2;
  float lr_wd;      // lr * weight_decay
  float step_size;  // lr / (1 - beta1^t)
  float inv_bc2;    // 1 / (1 - beta2^t)
  float eps;
};
struct AdamwConsts {
  GroupConsts g[FP8ADAM_MAX_GROUPS];
};

// With loss scaling: the decision of the step in flight, written on the device.
struct AdamwCtl {
  int32_t skip;
  float gfac;
  float step_size[FP8ADAM_MAX_GROUPS];
  float inv_bc2[FP8ADAM_MAX_GROUPS];
};

// The fresh moments and the weight of one element.  The moments are the step's
// (moment_update: fp32, one rounding in the product and one in the fma, so that
// 8-bit codes are exact functions of the inputs).  The weight changes by one
// sum, rounded once: decay and update are added first, which keeps a decay of
// less than half an ulp of 1 that a factor 1 - lr * wd would round away.
__device__ __forceinline__ float adamw_element(const GroupConsts& c, float g, float p, float m, float v, float& m1,
                                               float& v1) {
#pragma clang fp contract(off)
  const float gm = c.omb1 * g;
  const float gg = g * g;
  const float gv = c.omb2 * gg;
  m1 = __builtin_fmaf(c.b1, m, gm);
  v1 = __builtin_fmaf(c.b2, v, gv);
  const float den = __builtin_amdgcn_sqrtf(v1 * c.inv_bc2) + c.eps;
  const float upd = (c.step_size * m1) * __builtin_amdgcn_rcpf(den);
  return p - __builtin_fmaf(c.lr_wd, p, upd);
}

// Elements of an AdamW part: 256 lanes of 4.
constexpr int kAdamwPartLog2 = 10;

// One work-group per part.  32 lanes own one run of 128 elements (a block of
// 8-bit moments): lane h holds its elements h, h + 32, h + 64 and h + 96, so
// every access of a wave is contiguous at any alignment.
template <int PD, int CD, int GD, bool S8, int MF, int VF>
__global__ __launch_bounds__(kThreads) void k_adamw(const AdamwDesc* __restrict__ descs,
                                                    const int32_t* __restrict__ part_tid, AdamwConsts C, int64_t nparts,
                                                    const AdamwCtl* __restrict__ ctl) {
  const int64_t w = work_index<kXcdStreams>(nparts);
  if (w < 0) return;
  const AdamwDesc d = descs[part_tid[w]];
  GroupConsts c = C.g[d.group];
  float gfac = 1.0f;
  if (ctl != nullptr) {
    if (ctl->skip) return;
    gfac = ctl->gfac;
    c.step_size = ctl->step_size[d.group];
    c.inv_bc2 = ctl->inv_bc2[d.group];
  }
  const int64_t block = ((w - d.part0) << (kAdamwPartLog2 - 7)) + (threadIdx.x >> 5);
  const int64_t i0 = block * kBlock + (threadIdx.x & 31);
  const bool any = block * kBlock < d.numel;  // uniform for the 32 lanes
  float sm = 1.0f, sv = 1.0f;
  if constexpr (S8) {
    if (any) {
      sm = ld_global<float>(d.sm + block);
      sv = ld_global<float>(d.sv + block);
    }
  }
  float p[4], m1[4], v1[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int64_t i = i0 + 32 * j;
    p[j] = m1[j] = v1[j] = 0.0f;
    if (i < d.numel) {
      const float g = ld_elem<GD>(d.g, i) * gfac;
      float m, v;
      if constexpr (S8) {
        m = decode1<MF>(ld_global<uint8_t>(static_cast<const uint8_t*>(d.m) + i)) * sm;
        v = decode1<VF>(ld_global<uint8_t>(static_cast<const uint8_t*>(d.v) + i)) * sv;
      } else {
        m = ld_global<float>(static_cast<const float*>(d.m) + i);
        v = ld_global<float>(static_cast<const float*>(d.v) + i);
      }
      p[j] = adamw_element(c, g, ld_elem<PD>(d.p, i), m, v, m1[j], v1[j]);
    }
  }
  uint32_t wm = 0, wv = 0;
  if constexpr (S8) {
    float ism, isv;
    uint32_t am = 0, av = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      am = max(am, abs_bits(m1[j]));
      av = max(av, abs_bits(v1[j]));
    }
    am = group32_max(am);
    av = group32_max(av);
    choose_scale<MF, 0>(am, sm, ism);
    choose_scale<VF, 0>(av, sv, isv);
    if (any && (threadIdx.x & 31) == 0) {
      st_global<float>(d.sm + block, sm);
      st_global<float>(d.sv + block, sv);
    }
    const float qm[4] = {m1[0] * ism, m1[1] * ism, m1[2] * ism, m1[3] * ism};
    const float qv[4] = {v1[0] * isv, v1[1] * isv, v1[2] * isv, v1[3] * isv};
    wm = encode4_nan<MF>(qm, nonfinite_amax(am));
    wv = encode4_nan<VF>(qv, nonfinite_amax(av));
  }
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int64_t i = i0 + 32 * j;
    if (i < d.numel) {
      st_elem<PD>(d.p, i, p[j]);
      if constexpr (CD != 0) st_elem<CD>(d.copy, i, p[j]);
      if constexpr (S8) {
        st_global<uint8_t>(static_cast<uint8_t*>(d.m) + i, (uint8_t)(wm >> (8 * j)));
        st_global<uint8_t>(static_cast<uint8_t*>(d.v) + i, (uint8_t)(wv >> (8 * j)));
      } else {
        st_global<float>(static_cast<float*>(d.m) + i, m1[j]);
        st_global<float>(static_cast<float*>(d.v) + i, v1[j]);
      }
    }
  }
}

// A kind of AdamW tensor: its types (copy: 0 for none).
struct AdamwKind {
  int p, copy, g;
  bool moments8;
  bool operator==(const AdamwKind& o) const {
    return p == o.p && copy == o.copy && g == o.g && moments8 == o.moments8;
  }
};

template <int PD, int CD, int GD, bool S8, int MF, int VF>
inline void launch_adamw_kind(const AdamwDesc* descs, const int32_t* part_tid, const AdamwConsts& C, int64_t nparts,
                              const AdamwCtl* ctl, hipStream_t s) {
  hipLaunchKernelGGL((k_adamw<PD, CD, GD, S8, MF, VF>), dim3(grid_for<kXcdStreams>(nparts)), dim3(kThreads), 0, s, descs,
                     part_tid, C, nparts, ctl);
}

// The launch of one kind's parts (the caller checks the launch).
template <bool S8, int MF, int VF>
void launch_adamw(const AdamwKind& k, const AdamwDesc* descs, const int32_t* part_tid, const AdamwConsts& C,
                  int64_t nparts, const AdamwCtl* ctl, hipStream_t s) {
  auto by_grad = [&](auto pd, auto cd) {
    constexpr int P = decltype(pd)::value, Y = decltype(cd)::value;
    if (k.g == FP8ADAM_F32) launch_adamw_kind<P, Y, FP8ADAM_F32, S8, MF, VF>(descs, part_tid, C, nparts, ctl, s);
    else if (k.g == FP8ADAM_BF16) launch_adamw_kind<P, Y, FP8ADAM_BF16, S8, MF, VF>(descs, part_tid, C, nparts, ctl, s);
    else launch_adamw_kind<P, Y, FP8ADAM_F16, S8, MF, VF>(descs, part_tid, C, nparts, ctl, s);
  };
  using std::integral_constant;
  if (k.p == FP8ADAM_BF16) by_grad(integral_constant<int, FP8ADAM_BF16>{}, integral_constant<int, 0>{});
  else if (k.p == FP8ADAM_F16) by_grad(integral_constant<int, FP8ADAM_F16>{}, integral_constant<int, 0>{});
  else if (k.copy == FP8ADAM_BF16) by_grad(integral_constant<int, FP8ADAM_F32>{}, integral_constant<int, FP8ADAM_BF16>{});
  else if (k.copy == FP8ADAM_F16) by_grad(integral_constant<int, FP8ADAM_F32>{}, integral_constant<int, FP8ADAM_F16>{});
  else by_grad(integral_constant<int, FP8ADAM_F32>{}, integral_constant<int, 0>{});
}

}  // namespace fp8adam_list
