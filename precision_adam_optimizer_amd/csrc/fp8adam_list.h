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

// The part of this work-group.  Work-groups go round-robin over the 8 XCDs; in this
// order each XCD takes runs of kXcdRun consecutive parts, and the XCDs take
// neighbouring runs, so that the whole chip works on one stretch of the list.
// Measured with 32-part runs (of 1024 elements) against parts round-robin and
// against one contiguous eighth of the list per XCD, with eight work-groups on a CU:
// 842M weights with 32-bit moments 4.08, 4.24 and 4.17 ms; 842M bf16 weights with 8-bit moments 1.36, 1.42
// and 1.40 ms; 7M weights in ragged tensors 36, 37 and 40 us.  Runs of 16 and of
// 64 are 2 to 6% slower on the largest.  A surplus work-group gets -1.
constexpr int64_t kXcdRun = 32;

template <int64_t RUN = kXcdRun>
__device__ __forceinline__ int64_t run_index(int64_t nparts) {
  const int64_t xcd = blockIdx.x & 7u, k = blockIdx.x >> 3;
  const int64_t w = (k / RUN) * (8 * RUN) + xcd * RUN + k % RUN;
  return w < nparts ? w : -1;
}

template <int64_t RUN = kXcdRun>
inline unsigned run_grid(int64_t nparts) {
  return (unsigned)((nparts + 8 * RUN - 1) / (8 * RUN) * (8 * RUN));
}

// Shared memory that a launch reserves, and does not use, so that at most `groups`
// of its work-groups share a CU (8 do without).  Where most of the traffic is
// writes, fewer of them in flight reach HBM faster; each launch that does this says
// what it gains.
constexpr unsigned kCuLds = 160 * 1024;
constexpr unsigned lds_for(int groups) { return groups >= 8 ? 0u : kCuLds / (groups + 1) + 1024u; }

// --------------------------------------------------------------- typed elements

constexpr int64_t dtype_bytes(int dt) { return dt == FP8ADAM_F32 ? 4 : 2; }

typedef float vf2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

template <int DT>
__device__ __forceinline__ float ld_elem(const void* base, int64_t i) {
  if constexpr (DT == FP8ADAM_F32) {
    return ld_global<float>(static_cast<const float*>(base) + i);
  } else {
    const uint16_t x = ld_global<uint16_t>(static_cast<const uint16_t*>(base) + i);
    if constexpr (DT == FP8ADAM_BF16) return __uint_as_float((uint32_t)x << 16);
    else return (float)__builtin_bit_cast(_Float16, x);
  }
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

// Four consecutive elements of a type, or four codes, as they lie in memory.
constexpr int kCodes = -1;
template <int DT> struct Raw4 { vu2 x; };
template <> struct Raw4<FP8ADAM_F32> { vu4 x; };
template <> struct Raw4<kCodes> { uint32_t x; };

constexpr int64_t elem_bytes(int dt) { return dt == kCodes ? 1 : dt == FP8ADAM_F32 ? 4 : 2; }

// A whole part of one stream, accessed four elements per lane, non-temporally.
// DWORD: it starts on a dword, and goes through a buffer resource, which streams
// faster (the updates' byte mixes 6.4 against 6.0 TB/s).  Otherwise it starts on
// any element, and goes through global instructions, which take any address.
template <int DT, bool DWORD>
struct Stream {
  Rsrc r;
  __device__ __forceinline__ Stream(const void* base, int64_t first, int64_t n)
      : r(rsrc(static_cast<const char*>(base) + elem_bytes(DT) * first, elem_bytes(DT) * n)) {}
  __device__ __forceinline__ Raw4<DT> load(uint32_t o) const {
    if constexpr (DT == kCodes) return Raw4<DT>{__builtin_amdgcn_raw_buffer_load_b32(r, o, 0, kLdPol)};
    else if constexpr (DT == FP8ADAM_F32) return Raw4<DT>{__builtin_amdgcn_raw_buffer_load_b128(r, 4 * o, 0, kLdPol)};
    else return Raw4<DT>{__builtin_amdgcn_raw_buffer_load_b64(r, 2 * o, 0, kLdPol)};
  }
  __device__ __forceinline__ void store(uint32_t o, const Raw4<DT>& w) const {
    if constexpr (DT == kCodes) __builtin_amdgcn_raw_buffer_store_b32(w.x, r, o, 0, kStPol);
    else if constexpr (DT == FP8ADAM_F32) __builtin_amdgcn_raw_buffer_store_b128(w.x, r, 4 * o, 0, kStPol);
    else __builtin_amdgcn_raw_buffer_store_b64(w.x, r, 2 * o, 0, kStPol);
  }
};

typedef vu4 __attribute__((aligned(4))) vu4_any;
typedef vu2 __attribute__((aligned(2))) vu2_any;
typedef uint32_t __attribute__((aligned(1))) u32_any;

template <int DT>
struct Stream<DT, false> {
  const char* p;
  __device__ __forceinline__ Stream(const void* base, int64_t first, int64_t)
      : p(static_cast<const char*>(base) + elem_bytes(DT) * first) {}
  __device__ __forceinline__ Raw4<DT> load(uint32_t o) const {
    if constexpr (DT == kCodes) return Raw4<DT>{ld_stream<u32_any, true>(p + o)};
    else if constexpr (DT == FP8ADAM_F32) return Raw4<DT>{ld_stream<vu4_any, true>(p + 4 * o)};
    else return Raw4<DT>{ld_stream<vu2_any, true>(p + 2 * o)};
  }
  __device__ __forceinline__ void store(uint32_t o, const Raw4<DT>& w) const {
    char* q = const_cast<char*>(p);
    if constexpr (DT == kCodes) st_stream<u32_any, true>(q + o, w.x);
    else if constexpr (DT == FP8ADAM_F32) st_stream<vu4_any, true>(q + 4 * o, w.x);
    else st_stream<vu2_any, true>(q + 2 * o, w.x);
  }
};

template <int DT>
__device__ __forceinline__ void unpack4(const Raw4<DT>& w, float (&x)[4]) {
  if constexpr (DT == FP8ADAM_F32) {
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = __uint_as_float(w.x[j]);
  } else if constexpr (DT == FP8ADAM_BF16) {
    x[0] = bf16_lo(w.x.x); x[1] = bf16_hi(w.x.x); x[2] = bf16_lo(w.x.y); x[3] = bf16_hi(w.x.y);
  } else {
    const uint32_t lo = w.x.x, hi = w.x.y;  // (a bit cast of a vector's component takes the vector's first)
    const f16x2 a = __builtin_bit_cast(f16x2, lo), b = __builtin_bit_cast(f16x2, hi);
    x[0] = (float)a[0]; x[1] = (float)a[1]; x[2] = (float)b[0]; x[3] = (float)b[1];
  }
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == FP8ADAM_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(vf2{a, b}, bf16x2));
  else return __builtin_bit_cast(uint32_t, f16x2{to_f16(a), to_f16(b)});
}

template <int DT>
__device__ __forceinline__ Raw4<DT> pack4(const float (&x)[4]) {
  if constexpr (DT == FP8ADAM_F32)
    return Raw4<DT>{vu4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])}};
  else return Raw4<DT>{vu2{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3])}};
}

// The codes of four values at the inverse scale of their own amax, to nearest even,
// saturating, where a NaN stays one (the clamp of encode4 alone would make it
// -FMAX).  `odd`: the amax is not finite; without that the test is not made.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float inv, bool odd) {
  const float q[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
  uint32_t w = encode4<FMT>(q[0], q[1], q[2], q[3]);
  if (odd) {
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (q[j] != q[j]) w |= 0x7Fu << (8 * j);  // a NaN code in both formats
  }
  return w;
}

// codes4 where the scale s is a power of two and the POW2 scale of the amax, so that
// no value passes FMAX: the scaled converts divide by it as they round, without
// clamps and products.  The codes are those of encode4 of x / s (tested at every
// scale exponent: subnormal x, results down to zero, every tie of both formats and
// the fp32 numbers beside it).
template <int FMT>
__device__ __forceinline__ uint32_t codes4_pow2(const float (&x)[4], float s, bool odd) {
  if (odd) return codes4<FMT>(x, 1.0f, true);  // such a block's scale is 1
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  s16x2 w{0, 0};
  if constexpr (FMT == 0) {
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[0], x[1], s, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, x[2], x[3], s, true);
  } else {
    w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, x[0], x[1], s, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, x[2], x[3], s, true);
  }
  return __builtin_bit_cast(uint32_t, w);
}

// The largest of the 32 lanes of a half-wave, in each of them: four maxima with
// fused DPP operands (every lane has a source), and lane ^ 16.
__device__ __forceinline__ uint32_t half_wave_max(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));   // quad_perm [1,0,3,2]
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));   // quad_perm [2,3,0,1]
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, true));  // row_half_mirror
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, true));  // row_mirror
  return max(x, (uint32_t)__builtin_amdgcn_ds_swizzle((int)x, 0x401F));
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
  int32_t head;    // elements in front of the first part (0 or 1), which the first part's work-group does alone
  int32_t vec;     // every stream starts on a dword at element `head` (otherwise head is 0)
  int32_t pad;
};

// One parameter group's constants, computed on the host from its hyperparameters.
// The hardware's square root takes a subnormal v' as 0: next to an eps of 2^-38 or
// more that is less than half an ulp of their sum.  For a smaller eps the host
// scales the denominator by denom_scale = 2^12 (eps and step_size by as much,
// inv_bc2 by its square, which lifts every subnormal): the same bits otherwise, at
// no cost here.  The hardware's reciprocal takes a subnormal denominator as 0 too:
// the 2^24 for an eps below 2^-114 lift every eps that fp32 holds to 2^-125 or more.
struct GroupConsts {
  float b1, omb1, b2, omb2;
  float lr_wd;      // lr * weight_decay
  float step_size;  // lr / (1 - beta1^t), times denom_scale
  float inv_bc2;    // 1 / (1 - beta2^t), times its square
  float eps;        // times denom_scale
};
inline double denom_scale(float eps) {
  return eps >= 0x1p-38f ? 1.0 : eps >= 0x1p-114f || eps == 0.0f ? 0x1p12 : 0x1p24;
}
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

// log2 of a part's elements: 256 lanes of 4, twice where an element moves few bytes
// (8-bit moments of 16-bit weights).  With eight work-groups on a CU, 842M fp32
// weights with 32-bit moments: 1024 elements 4.15 ms, 2048 4.24, 4096 4.35; 109.5M with 8-bit moments, scaled and
// clipped: 1024 320 us, 2048 330; 842M bf16 weights with 8-bit moments: 1024 1.37
// ms, 2048 1.36, 4096 1.44.
constexpr int adamw_part_log2(int pd, bool s8) { return s8 && pd != FP8ADAM_F32 ? 11 : 10; }

// The moments of a run of 128 elements that 32 lanes own, four each: new scales
// and codes.
template <int MF, int VF>
__device__ __forceinline__ void moments_to_codes(const float (&m1)[4], const float (&v1)[4], float& sm, float& sv,
                                                 uint32_t& wm, uint32_t& wv) {
  uint32_t am = 0, av = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    am = max(am, abs_bits(m1[j]));
    av = max(av, abs_bits(v1[j]));
  }
  am = half_wave_max(am);
  av = half_wave_max(av);
  float inv;
  choose_scale<MF, 0>(am, sm, inv);
  choose_scale<VF, 0>(av, sv, inv);
  wm = codes4_pow2<MF>(m1, sm, nonfinite_amax(am));
  wv = codes4_pow2<VF>(v1, sv, nonfinite_amax(av));
}

// A whole part, [lo, lo + 2^PL), in groups of four consecutive elements per lane.
template <bool DWORD, int PL, int PD, int CD, int GD, bool S8, int MF, int VF>
__device__ __forceinline__ void adamw_whole(const AdamwDesc& d, const GroupConsts& c, float gfac, int64_t lo) {
  constexpr int64_t kLen = (int64_t)1 << PL;
  constexpr int kU = (int)(kLen / kSubTile);
  constexpr int MD = S8 ? kCodes : FP8ADAM_F32;
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  const Stream<PD, DWORD> sp(d.p, lo, kLen);
  const Stream<GD, DWORD> sg(d.g, lo, kLen);
  const Stream<MD, DWORD> smom(d.m, lo, kLen), svar(d.v, lo, kLen);
  Raw4<PD> rp[kU];
  Raw4<GD> rg[kU];
  Raw4<MD> rm[kU], rv[kU];
  float sm[kU], sv[kU];
  const int64_t block0 = (lo >> 7) + run;
#pragma unroll
  for (int u = 0; u < kU; u++) {
    const uint32_t o = 4 * threadIdx.x + u * kSubTile;
    rg[u] = sg.load(o);
    rm[u] = smom.load(o);
    rv[u] = svar.load(o);
    if constexpr (S8) {
      sm[u] = ld_global<float>(d.sm + block0 + 8 * u);
      sv[u] = ld_global<float>(d.sv + block0 + 8 * u);
    }
    rp[u] = sp.load(o);
  }
#pragma unroll
  for (int u = 0; u < kU; u++) {
    const uint32_t o = 4 * threadIdx.x + u * kSubTile;
    float p[4], g[4], m[4], v[4], m1[4], v1[4];
    unpack4<GD>(rg[u], g);
    if constexpr (S8) {
      decode4<MF>(rm[u].x, m);
      decode4<VF>(rv[u].x, v);
#pragma unroll
      for (int j = 0; j < 4; j++) {
        m[j] *= sm[u];
        v[j] *= sv[u];
      }
    } else {
      unpack4<FP8ADAM_F32>(rm[u], m);
      unpack4<FP8ADAM_F32>(rv[u], v);
    }
    unpack4<PD>(rp[u], p);
#pragma unroll
    for (int j = 0; j < 4; j++) p[j] = adamw_element(c, g[j] * gfac, p[j], m[j], v[j], m1[j], v1[j]);
    sp.store(o, pack4<PD>(p));
    if constexpr (CD != 0) Stream<CD, DWORD>(d.copy, lo, kLen).store(o, pack4<CD>(p));
    if constexpr (S8) {
      uint32_t wm, wv;
      float ns, nv;
      moments_to_codes<MF, VF>(m1, v1, ns, nv, wm, wv);
      smom.store(o, Raw4<MD>{wm});
      svar.store(o, Raw4<MD>{wv});
      if (lane == 0) {
        st_global<float>(d.sm + block0 + 8 * u, ns);
        st_global<float>(d.sv + block0 + 8 * u, nv);
      }
    } else {
      smom.store(o, pack4<FP8ADAM_F32>(m1));
      svar.store(o, pack4<FP8ADAM_F32>(v1));
    }
  }
}

// One work-group per part.  32 lanes own one run of 128 elements (a block of
// 8-bit moments).  A whole part goes in groups of four consecutive elements per
// lane, the last part of a tensor element by element, where lane h of the 32 holds
// elements h, h + 32, h + 64 and h + 96 of its run.
//
// Bound by HBM, each stream read and written once (counters: 14.0 bytes fetched and
// 14.0 written per fp32 weight with a bf16 gradient, a bf16 copy and 32-bit
// moments).  842M of those take 4.0 ms, 5.95 TB/s: a little over what a 1:1 copy
// reaches on the card (5.86), and 92% of reads and writes one after the other at
// their own rates.
// 842M bf16 weights with bf16 gradients and 8-bit moments (10.1 bytes): 1.35 ms,
// 6.3 TB/s, 95% of that bound.  The smallest lists are bound by the launch: 65
// tensors of 4096 take 3 us on the device, 5.5 us with the call.  Packed fp32
// tensors of odd sizes cost no more (every fp32 stream starts on a dword): 7M
// weights in 48 of them 35 us, 5.7 TB/s.
template <int PD, int CD, int GD, bool S8, int MF, int VF>
__global__ __launch_bounds__(kThreads) void k_adamw(const AdamwDesc* __restrict__ descs,
                                                    const int32_t* __restrict__ part_tid, AdamwConsts C, int64_t nparts,
                                                    const AdamwCtl* __restrict__ ctl) {
  constexpr int PL = adamw_part_log2(PD, S8);
  constexpr int64_t kLen = (int64_t)1 << PL;
  constexpr int kU = (int)(kLen / kSubTile);
  const int64_t w = run_index(nparts);
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
  const int64_t lo = d.head + ((w - d.part0) << PL);
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;  // of 8 runs per tile of 1024
  if (d.vec && lo + kLen <= d.numel) {
    adamw_whole<true, PL, PD, CD, GD, S8, MF, VF>(d, c, gfac, lo);
  } else if (lo + kLen <= d.numel) {
    adamw_whole<false, PL, PD, CD, GD, S8, MF, VF>(d, c, gfac, lo);
  } else {
    for (int u = 0; u < kU; u++) {
      const int64_t first = lo + u * kSubTile + run * kBlock, block = first >> 7;
      const bool any = first < d.numel;  // uniform for the 32 lanes
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
        const int64_t i = first + lane + 32 * j;
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
        moments_to_codes<MF, VF>(m1, v1, sm, sv, wm, wv);
        if (any && lane == 0) {
          st_global<float>(d.sm + block, sm);
          st_global<float>(d.sv + block, sv);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int64_t i = first + lane + 32 * j;
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
  }
  if constexpr (!S8) {
    if (d.head && w == d.part0 && threadIdx.x == 0) {
      float m1, v1;
      const float p = adamw_element(c, ld_elem<GD>(d.g, 0) * gfac, ld_elem<PD>(d.p, 0),
                                    ld_global<float>(d.m), ld_global<float>(d.v), m1, v1);
      st_elem<PD>(d.p, 0, p);
      if constexpr (CD != 0) st_elem<CD>(d.copy, 0, p);
      st_global<float>(d.m, m1);
      st_global<float>(d.v, v1);
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
inline int launch_adamw_kind(const AdamwDesc* descs, const int32_t* part_tid, const AdamwConsts& C, int64_t nparts,
                             const AdamwCtl* ctl, hipStream_t s) {
  // 32-bit moments: five work-groups on a CU.  842M fp32 weights with a copy 3.96 ms against 4.09 with
  // eight (four: 3.98, three: 4.03), without one 3.59 against 3.73; 109.5M with a copy 507 us against 519
  // (four: 525); 842M bf16 weights 3.04 ms against 3.06.  8-bit moments read more than they write: they lose.
  return launch(k_adamw<PD, CD, GD, S8, MF, VF>, dim3(run_grid(nparts)), dim3(kThreads), lds_for(S8 ? 8 : 5), s, descs,
                part_tid, C, nparts, ctl);
}

// The launch of one kind's parts.
template <bool S8, int MF, int VF>
int launch_adamw(const AdamwKind& k, const AdamwDesc* descs, const int32_t* part_tid, const AdamwConsts& C,
                 int64_t nparts, const AdamwCtl* ctl, hipStream_t s) {
  auto by_grad = [&](auto pd, auto cd) -> int {
    constexpr int P = decltype(pd)::value, Y = decltype(cd)::value;
    if (k.g == FP8ADAM_F32) return launch_adamw_kind<P, Y, FP8ADAM_F32, S8, MF, VF>(descs, part_tid, C, nparts, ctl, s);
    if (k.g == FP8ADAM_BF16) return launch_adamw_kind<P, Y, FP8ADAM_BF16, S8, MF, VF>(descs, part_tid, C, nparts, ctl, s);
    return launch_adamw_kind<P, Y, FP8ADAM_F16, S8, MF, VF>(descs, part_tid, C, nparts, ctl, s);
  };
  using std::integral_constant;
  if (k.p == FP8ADAM_BF16) return by_grad(integral_constant<int, FP8ADAM_BF16>{}, integral_constant<int, 0>{});
  if (k.p == FP8ADAM_F16) return by_grad(integral_constant<int, FP8ADAM_F16>{}, integral_constant<int, 0>{});
  if (k.copy == FP8ADAM_BF16) return by_grad(integral_constant<int, FP8ADAM_F32>{}, integral_constant<int, FP8ADAM_BF16>{});
  if (k.copy == FP8ADAM_F16) return by_grad(integral_constant<int, FP8ADAM_F32>{}, integral_constant<int, FP8ADAM_F16>{});
  return by_grad(integral_constant<int, FP8ADAM_F32>{}, integral_constant<int, 0>{});
}

}  // namespace fp8adam_list
