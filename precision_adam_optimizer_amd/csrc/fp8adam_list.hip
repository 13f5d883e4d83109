// fp8adam_list.hip -- the list operators of include/fp8adam_list.h: plans and
// their checks, the gradient norm and clipping, the conversion to 8 bits and
// back, and the C ABI.  The AdamW kernels are in fp8adam_list.h, instantiated
// in fp8adam_list_adamw*.hip.
#include <string.h>

#include <algorithm>

#include "fp8adam_list.h"

using namespace fp8adam;
using namespace fp8adam_engine;
using namespace fp8adam_list;

namespace fp8adam_list {

extern template int launch_adamw<false, 0, 0>(const AdamwKind&, const AdamwDesc*, const int32_t*, const AdamwConsts&,
                                              int64_t, const AdamwCtl*, hipStream_t);
extern template int launch_adamw<true, 0, 1>(const AdamwKind&, const AdamwDesc*, const int32_t*, const AdamwConsts&,
                                             int64_t, const AdamwCtl*, hipStream_t);
extern template int launch_adamw<true, 0, 0>(const AdamwKind&, const AdamwDesc*, const int32_t*, const AdamwConsts&,
                                             int64_t, const AdamwCtl*, hipStream_t);
extern template int launch_adamw<true, 1, 0>(const AdamwKind&, const AdamwDesc*, const int32_t*, const AdamwConsts&,
                                             int64_t, const AdamwCtl*, hipStream_t);
extern template int launch_adamw<true, 1, 1>(const AdamwKind&, const AdamwDesc*, const int32_t*, const AdamwConsts&,
                                             int64_t, const AdamwCtl*, hipStream_t);

namespace {

// ---------------------------------------------------------- norm and clipping
//
// The norm pass runs a fixed grid over the chunks of the list; each work-group
// sums its chunks' squares in fp64 (a sum over 1e9 fp32 squares spans more than
// fp32 holds; the square of a bf16, fp16 or fp32 number is exact in it) and
// writes one partial.  The partials are summed in one fixed order by whoever
// needs the norm, so the result is the same in every run.  A NaN or Inf needs no
// count of its own: no sum of finite squares overflows fp64, so the sum is not
// finite exactly if an element is not.  Bound by HBM: 438 MB of fp32 in 64 us, 6.9
// TB/s (the read-only rate is 7.2).

struct GradDesc {
  const void* src;
  void* dst;       // clipping only; may be null, or src
  int64_t numel;
  int64_t chunk0;
  int32_t sdt, ddt;
};

// Two work-groups per CU with 8 16-byte loads per lane keep the norm pass at the
// read-only rate (7.0 TB/s), and the clipping pass, whose every work-group sums
// the partials, reads few of them: clipping 842M fp32 gradients to bf16 took 1264
// us with 512 and 1284 with 2048 (both passes, parts in plain order; 1229 us with
// the order of k_list_clip).
constexpr int kListNormGroups = 512;

__device__ __forceinline__ void sumsq_word(uint32_t x, double& acc, std::integral_constant<int, FP8ADAM_F32>) {
  const double a = __uint_as_float(x);
  acc = __builtin_fma(a, a, acc);
}
__device__ __forceinline__ void sumsq_word(uint32_t x, double& acc, std::integral_constant<int, FP8ADAM_BF16>) {
  const double a = bf16_lo(x), b = bf16_hi(x);
  acc = __builtin_fma(a, a, acc);
  acc = __builtin_fma(b, b, acc);
}
__device__ __forceinline__ void sumsq_word(uint32_t x, double& acc, std::integral_constant<int, FP8ADAM_F16>) {
  const f16x2 h = __builtin_bit_cast(f16x2, x);
  const double a = (float)h[0], b = (float)h[1];
  acc = __builtin_fma(a, a, acc);
  acc = __builtin_fma(b, b, acc);
}

// The squares of elements [lo, hi): single ones up to a 16-byte boundary, then
// 16-byte loads, kSumUnroll in flight per lane (the buffer resource ends with the
// last whole vector: a load behind it gives zeros, which add nothing), then the
// rest.
constexpr int kSumUnroll = 8;
template <int DT>
__device__ __forceinline__ void sumsq_range(const void* src, int64_t lo, int64_t hi, double& acc) {
  constexpr int kBytes = DT == FP8ADAM_F32 ? 4 : 2, kVec = 16 / kBytes;
  const char* base = static_cast<const char*>(src) + kBytes * lo;
  const int n = (int)(hi - lo);
  const int head = min(n, (int)((16u - ((uintptr_t)base & 15u)) & 15u) / kBytes);
  const int nvec = (n - head) / kVec, tail = head + nvec * kVec;
  const Rsrc r = rsrc(base + kBytes * head, 16 * (int64_t)nvec);
  for (int v = threadIdx.x; v < nvec; v += kThreads * kSumUnroll) {
    vu4 x[kSumUnroll];
#pragma unroll
    for (int u = 0; u < kSumUnroll; u++) x[u] = __builtin_amdgcn_raw_buffer_load_b128(r, 16 * (v + u * kThreads), 0, kLdPol);
#pragma unroll
    for (int u = 0; u < kSumUnroll; u++)
#pragma unroll
      for (int j = 0; j < 4; j++) sumsq_word(x[u][j], acc, std::integral_constant<int, DT>{});
  }
  const int single = (int)threadIdx.x < head ? (int)threadIdx.x : tail + (int)threadIdx.x - head;
  if (single < n) {  // at most 7 in front and 7 behind
    const double x = ld_elem<DT>(base, single);
    acc = __builtin_fma(x, x, acc);
  }
}

// Sum over the work-group's threads in a fixed order, returned to every thread.
__device__ __forceinline__ double block_sum(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  __shared__ double part[kThreads / 64];
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = part[0];
#pragma unroll
  for (int k = 1; k < kThreads / 64; k++) s += part[k];
  return s;
}

// This work-group's share of the sum, in every thread.
__device__ __forceinline__ double sumsq_share(const GradDesc* __restrict__ descs, const int32_t* __restrict__ chunk_tid,
                                              int64_t nchunks, int chunk_log2) {
  double acc = 0.0;
  for (int64_t w = blockIdx.x; w < nchunks; w += gridDim.x) {
    const GradDesc d = descs[chunk_tid[w]];
    const int64_t lo = (w - d.chunk0) << chunk_log2;
    const int64_t hi = min(lo + ((int64_t)1 << chunk_log2), d.numel);
    if (d.sdt == FP8ADAM_F32) sumsq_range<FP8ADAM_F32>(d.src, lo, hi, acc);
    else if (d.sdt == FP8ADAM_BF16) sumsq_range<FP8ADAM_BF16>(d.src, lo, hi, acc);
    else sumsq_range<FP8ADAM_F16>(d.src, lo, hi, acc);
  }
  return block_sum(acc);
}

__global__ __launch_bounds__(kThreads) void k_list_sumsq(const GradDesc* __restrict__ descs,
                                                         const int32_t* __restrict__ chunk_tid, int64_t nchunks,
                                                         int chunk_log2, double* __restrict__ partial) {
  const double acc = sumsq_share(descs, chunk_tid, nchunks, chunk_log2);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// The whole sum from the partials, in every thread: the same order in every
// work-group that asks.
__device__ __forceinline__ double total_of(const double* __restrict__ partial, int n) {
  double acc = 0.0;
#pragma unroll 4
  for (int k = threadIdx.x; k < n; k += kThreads) acc += partial[k];
  return block_sum(acc);
}

// What the loss scaler's decision reads of its state: loaded before the sum that
// the decision waits for.
struct ScalerState {
  float scale;
  int32_t growth_tracker;
  int64_t step;
};

__device__ __forceinline__ ScalerState load_scaler(const fp8adam_amp_state* st) {
  return ScalerState{ld_global<float>(&st->scale), ld_global<int32_t>(&st->growth_tracker), ld_global<int64_t>(&st->step)};
}

// The loss scaler's decision (one thread), the rules and roundings of
// fp8adam_step_amp's: from the sum of squares of every (scaled) gradient and whether
// one was not finite, update the state `st` (which held `was`) and return true with
// the gradient factor and the step's t, or false if the step is skipped.
__device__ inline bool scaler_decide(fp8adam_amp_state* st, const ScalerState& was, const fp8adam_amp_config& cfg,
                                     double sumsq, bool bad, float& gfac, int64_t& t) {
  const float scale = was.scale;
  const float inv = __double2float_rn(__ddiv_rn(1.0, (double)scale));
  if (bad) {
    st_global(&st->found_inf, 1);
    st_global(&st->grad_norm, __builtin_nanf(""));
    st_global(&st->clip_coef, 1.0f);
    st_global(&st->grad_factor, 0.0f);
    st_global(&st->scale, __fmul_rn(scale, cfg.backoff_factor));
    st_global(&st->growth_tracker, 0);
    return false;
  }
  const double norm = __dmul_rn(__dsqrt_rn(sumsq), (double)inv);
  double cc = 1.0;
  if (cfg.max_norm > 0.0f) {
    cc = __ddiv_rn((double)cfg.max_norm, __dadd_rn(norm, 1e-6));
    if (cc > 1.0) cc = 1.0;
  }
  const float c32 = __double2float_rn(cc);
  gfac = __fmul_rn(c32, inv);
  t = was.step + 1;
  st_global(&st->found_inf, 0);
  st_global(&st->grad_norm, __double2float_rn(norm));
  st_global(&st->clip_coef, c32);
  st_global(&st->grad_factor, gfac);
  st_global(&st->step, t);
  const int32_t next = was.growth_tracker + 1;
  if (next == cfg.growth_interval) {
    const float grown = __fmul_rn(scale, cfg.growth_factor);
    if (isfinite(grown)) st_global(&st->scale, grown);
    st_global(&st->growth_tracker, 0);
  } else {
    st_global(&st->growth_tracker, next);
  }
  return true;
}

// Loss scaling: the scaler's decision, and each group's bias corrections at the
// device-side t (of the step about to be taken; of no use to a skipped one).  What
// does not need the sum is done before it.
struct GroupRates {
  double lr[FP8ADAM_MAX_GROUPS], beta1[FP8ADAM_MAX_GROUPS], beta2[FP8ADAM_MAX_GROUPS];
  double v_scale[FP8ADAM_MAX_GROUPS];  // denom_scale squared (lr carries denom_scale)
};

struct AmpArgs {
  fp8adam_amp_state* st;
  AdamwCtl* ctl;
  fp8adam_amp_config cfg;
  int32_t n_groups;
  GroupRates R;
};

__device__ __forceinline__ void bias_corrections(const AmpArgs& a, const ScalerState& was) {
  const int q = threadIdx.x;
  if (q < a.n_groups) {
    const double t = (double)(was.step + 1);
    a.ctl->step_size[q] = (float)(a.R.lr[q] / (1.0 - pow(a.R.beta1[q], t)));
    a.ctl->inv_bc2[q] = (float)(a.R.v_scale[q] / (1.0 - pow(a.R.beta2[q], t)));
  }
}

__device__ __forceinline__ void decide(const AmpArgs& a, const ScalerState& was, double sumsq) {
  float gfac = 0.0f;
  int64_t t = 0;
  const bool run = scaler_decide(a.st, was, a.cfg, sumsq, !isfinite(sumsq), gfac, t);
  a.ctl->skip = run ? 0 : 1;
  a.ctl->gfac = gfac;
}

__global__ __launch_bounds__(kThreads) void k_list_ctl(const double* __restrict__ partial, int npartial, AmpArgs a) {
  const ScalerState was = load_scaler(a.st);
  bias_corrections(a, was);
  const double sumsq = total_of(partial, npartial);
  if (threadIdx.x == 0) decide(a, was, sumsq);
}

// Norm and decision in one launch, for a list of few chunks: the work-group that
// arrives last (by a ticket of the plan's workspace, zero before and after) sums the
// partials, in their order, and decides.  Its ticket's acquire sees the partials,
// each stored before its work-group's release.  A release costs more the more
// work-groups make one (100 us of 2048).  Among other calls, where the host's
// launches count, a scaled step over 1 to 64 tensors of 4000 takes 9.7 to 11.4 us
// with the ticket and 12.1 to 12.4 without; replayed from a graph the two are within
// 0.4 us of each other (8.1 to 10.5), the ticket ahead on one chunk and behind on 64.
constexpr int kTicketGroups = 64;

__global__ __launch_bounds__(kThreads) void k_list_sumsq_ctl(const GradDesc* __restrict__ descs,
                                                             const int32_t* __restrict__ chunk_tid, int64_t nchunks,
                                                             int chunk_log2, double* partial, uint32_t* ticket, AmpArgs a) {
  const ScalerState was = load_scaler(a.st);
  const double acc = sumsq_share(descs, chunk_tid, nchunks, chunk_log2);
  __shared__ bool last;
  if (threadIdx.x == 0) {
    __hip_atomic_store(&partial[blockIdx.x], acc, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  bias_corrections(a, was);
  if (threadIdx.x >= 64) return;
  double sum = threadIdx.x < gridDim.x
                   ? __hip_atomic_load(&partial[threadIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                   : 0.0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (threadIdx.x != 0) return;
  __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  decide(a, was, sum);
}
static_assert(kTicketGroups <= 64, "one wave sums the partials");

constexpr int kClipUnroll = 4;

template <int SD, int DD, bool DWORD>
__device__ __forceinline__ void scale_groups(const char* src, char* dst, int first, int ngroups, float coef) {
  const Stream<SD, DWORD> ss(src, first, 4 * ngroups);
  const Stream<DD, DWORD> sd(dst, first, 4 * ngroups);
  for (int v = threadIdx.x; v < ngroups; v += kThreads * kClipUnroll) {
    Raw4<SD> w[kClipUnroll];
#pragma unroll
    for (int u = 0; u < kClipUnroll; u++)
      if (DWORD || v + u * kThreads < ngroups) w[u] = ss.load(4 * (v + u * kThreads));
#pragma unroll
    for (int u = 0; u < kClipUnroll; u++) {
      float x[4];
      unpack4<SD>(w[u], x);
#pragma unroll
      for (int j = 0; j < 4; j++) x[j] *= coef;
      // (a buffer resource drops what lies behind the last group)
      if (DWORD || v + u * kThreads < ngroups) sd.store(4 * (v + u * kThreads), pack4<DD>(x));
    }
  }
}

// dst = src * coef over [lo, hi), in groups of four elements per lane: on dwords in
// both, after one single element where the 16-bit pointers are all off by one;
// from any element where one of two 16-bit pointers is.
template <int SD, int DD>
__device__ __forceinline__ void scale_range(const GradDesc& d, int64_t lo, int64_t hi, float coef) {
  const char* src = static_cast<const char*>(d.src) + elem_bytes(SD) * lo;
  char* dst = static_cast<char*>(d.dst) + elem_bytes(DD) * lo;
  const int n = (int)(hi - lo);
  const int soff = SD != FP8ADAM_F32 ? (int)((uintptr_t)src >> 1 & 1u) : -1;
  const int doff = DD != FP8ADAM_F32 ? (int)((uintptr_t)dst >> 1 & 1u) : -1;
  const bool dword = soff < 0 || doff < 0 || soff == doff;  // uniform
  const int head = dword ? max(max(soff, doff), 0) : 0;
  const int ngroups = max(n - head, 0) >> 2, tail = head + 4 * ngroups;
  if (dword) scale_groups<SD, DD, true>(src, dst, head, ngroups, coef);
  else scale_groups<SD, DD, false>(src, dst, head, ngroups, coef);
  const int single = (int)threadIdx.x < head ? (int)threadIdx.x : tail + (int)threadIdx.x - head;
  if (single < n) st_elem<DD>(dst, single, ld_elem<SD>(src, single) * coef);
}

template <int SD>
__device__ __forceinline__ void scale_range_to(const GradDesc& d, int64_t lo, int64_t hi, float coef) {
  if (d.ddt == FP8ADAM_F32) scale_range<SD, FP8ADAM_F32>(d, lo, hi, coef);
  else if (d.ddt == FP8ADAM_BF16) scale_range<SD, FP8ADAM_BF16>(d, lo, hi, coef);
  else scale_range<SD, FP8ADAM_F16>(d, lo, hi, coef);
}

// Every work-group makes the coefficient from the partials (4 KB of the L2, the same
// order everywhere) and scales its 2^kClipPartLog2 elements, from the list's end to
// its start: what the norm pass read last may still be in the last-level cache (1%
// of 109.5M fp32).  842M fp32 gradients into bf16 take 770 us (6.6 TB/s); a fixed
// grid striding over the list took 918.  Letting the norm pass's last work-group
// finish the sum instead costs each of them a release to the other XCDs: 137 us
// against 34 for 219 MB in 2048 work-groups.
constexpr int kClipPartLog2 = 12;
// Parts in an XCD's run: 842M take 1233 us (both passes), 1247 with 32, 1264 in plain order.
constexpr int64_t kClipXcdRun = 16;
constexpr int kGradChunkMinLog2 = 12, kGradChunkMaxLog2 = 15;
static_assert(kClipPartLog2 <= kGradChunkMinLog2, "a chunk holds whole parts");

__global__ __launch_bounds__(kThreads) void k_list_clip(const GradDesc* __restrict__ descs,
                                                        const int32_t* __restrict__ chunk_tid, int64_t nparts,
                                                        int chunk_log2, const double* __restrict__ partial, int npartial,
                                                        float max_norm, float* __restrict__ result) {
  const int64_t w = nparts - 1 - run_index<kClipXcdRun>(nparts);
  if (w >= nparts && blockIdx.x != 0) return;  // a surplus work-group; the first one still gives the result
  const double norm = __dsqrt_rn(total_of(partial, npartial));
  double cc = 1.0;
  if (max_norm > 0.0f && isfinite(norm)) {
    cc = __ddiv_rn((double)max_norm, __dadd_rn(norm, 1e-6));
    if (cc > 1.0) cc = 1.0;
  }
  const float coef = __double2float_rn(cc);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    st_global<float>(result, __double2float_rn(norm));
    st_global<float>(result + 1, coef);
  }
  if (w >= nparts) return;  // nothing is written
  const GradDesc d = descs[chunk_tid[w >> (chunk_log2 - kClipPartLog2)]];
  if (d.dst == nullptr || (coef == 1.0f && d.dst == d.src)) return;  // uniform: nothing to write, or nothing changes
  const int64_t lo = (w - (d.chunk0 << (chunk_log2 - kClipPartLog2))) << kClipPartLog2;
  const int64_t hi = min(lo + ((int64_t)1 << kClipPartLog2), d.numel);
  if (lo >= hi) return;  // behind the tensor's end, in its last chunk
  if (d.sdt == FP8ADAM_F32) scale_range_to<FP8ADAM_F32>(d, lo, hi, coef);
  else if (d.sdt == FP8ADAM_BF16) scale_range_to<FP8ADAM_BF16>(d, lo, hi, coef);
  else scale_range_to<FP8ADAM_F16>(d, lo, hi, coef);
}

// -------------------------------------------------------- conversion to 8 bits

struct QuantDesc {
  void* x;
  uint8_t* codes;
  float* scale;
  int64_t numel;
  int64_t part0;
  int64_t chunk0;    // per-tensor scales: its first amax chunk, the chunks' length
  int64_t chunk_len;
  int64_t slot0;     // the first slot of their maxima, a multiple of 4; unused slots up to the next tensor hold 0
  int32_t slots;     // their number, a multiple of 4
  int32_t head;      // per-tensor scales: elements in front of the first part (0 .. 3)
  int32_t vec;       // values and codes both start on a dword at element `head`
};

// log2 of the elements of a one-shot work-group.  Blocks, both ways: 2048 (109.5M
// fp32 to E4M3 blocks 83 us, back 93 us with eight work-groups on a CU; 1024: 93 and
// 99, 4096: 85 and 98, 8192: 91 and 103; dequant_lds takes the 93 to 83).  With a tensor's scale: 4096 (202M bf16 in 150 us; 2048: 161, 8192: 153),
// since each wave reads the tensor's maxima first.
constexpr int kQuantPartLog2 = 11;
constexpr int kQuantTensorPartLog2 = 12;
// Amax chunks per tensor at most: each quantizing wave reads them all, with one 16-byte load per lane.
constexpr int64_t kAmaxMaxChunks = 256;
constexpr int64_t kAmaxMinChunk = 8192;

template <int FMT>
__device__ __forceinline__ void choose_scale_mode(uint32_t amax, int smode, float& s, float& inv) {
  if (smode == FP8ADAM_SCALE_POW2) choose_scale<FMT, 0>(amax, s, inv);
  else choose_scale<FMT, 1>(amax, s, inv);
}

// The new scale and the codes of a run of 128 values that 32 lanes hold, four each.
template <int FMT>
__device__ __forceinline__ uint32_t block_to_codes(const float (&x)[4], int smode, float& s) {
  uint32_t am = 0;
#pragma unroll
  for (int j = 0; j < 4; j++) am = max(am, abs_bits(x[j]));
  am = half_wave_max(am);
  float inv;
  choose_scale_mode<FMT>(am, smode, s, inv);
  return codes4<FMT>(x, inv, nonfinite_amax(am));
}

template <bool DWORD, int DT, int FMT>
__device__ __forceinline__ void quant_block_whole(const QuantDesc& d, int64_t lo, int smode) {
  constexpr int64_t kLen = (int64_t)1 << kQuantPartLog2;
  constexpr int kU = (int)(kLen / kSubTile);
  const Stream<DT, DWORD> sx(d.x, lo, kLen);
  const Stream<kCodes, DWORD> sc(d.codes, lo, kLen);
  Raw4<DT> r[kU];
#pragma unroll
  for (int u = 0; u < kU; u++) r[u] = sx.load(4 * threadIdx.x + u * kSubTile);
#pragma unroll
  for (int u = 0; u < kU; u++) {
    float x[4], s;
    unpack4<DT>(r[u], x);
    sc.store(4 * threadIdx.x + u * kSubTile, Raw4<kCodes>{block_to_codes<FMT>(x, smode, s)});
    if ((threadIdx.x & 31) == 0) st_global<float>(d.scale + (lo >> 7) + 8 * u + (threadIdx.x >> 5), s);
  }
}

// One work-group per part, 32 lanes per block of 128, four consecutive elements
// per lane; in the last part of a tensor lane h takes the block's elements h,
// h + 32, h + 64, h + 96.  Bound by HBM: 109.5M fp32 (5.03 bytes each) in 83 us, 6.6
// TB/s, 97% of its reads and writes at their own rates.
template <int DT, int FMT>
__global__ __launch_bounds__(kThreads) void k_quant_block(const QuantDesc* __restrict__ descs,
                                                          const int32_t* __restrict__ part_tid, int64_t nparts,
                                                          int smode) {
  constexpr int64_t kLen = (int64_t)1 << kQuantPartLog2;
  constexpr int kU = (int)(kLen / kSubTile);
  const int64_t w = run_index(nparts);
  if (w < 0) return;
  const QuantDesc d = descs[part_tid[w]];
  const int64_t lo = (w - d.part0) << kQuantPartLog2;
  const int lane = threadIdx.x & 31, run = threadIdx.x >> 5;
  // loaded with the rest of the descriptor: left to itself the compiler loads the field behind the
  // first branch, one more wait (84.6 us against 83.8)
  int vec = d.vec;
  asm volatile("" : "+s"(vec));
  if (lo + kLen <= d.numel) {
    if (vec) quant_block_whole<true, DT, FMT>(d, lo, smode);
    else quant_block_whole<false, DT, FMT>(d, lo, smode);
    return;
  }
  for (int u = 0; u < kU; u++) {
    const int64_t first = lo + u * kSubTile + run * kBlock;
    float x[4], s;
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] = first + lane + 32 * j < d.numel ? ld_elem<DT>(d.x, first + lane + 32 * j) : 0.0f;
    const uint32_t codes = block_to_codes<FMT>(x, smode, s);
    if (first < d.numel && lane == 0) st_global<float>(d.scale + (first >> 7), s);
#pragma unroll
    for (int j = 0; j < 4; j++)
      if (first + lane + 32 * j < d.numel)
        st_global<uint8_t>(d.codes + first + lane + 32 * j, (uint8_t)(codes >> (8 * j)));
  }
}

// The largest |value| bits of two 16-bit values or of one in a dword, as fp32 bits.
template <int DT>
__device__ __forceinline__ uint32_t amax_word(uint32_t am, uint32_t x) {
  if constexpr (DT == FP8ADAM_F32) return max(am, x & 0x7FFFFFFFu);
  if constexpr (DT == FP8ADAM_BF16) return max(max(am, (x << 16) & 0x7FFF0000u), x & 0x7FFF0000u);
  const f16x2 h = __builtin_bit_cast(f16x2, x);
  return max(max(am, abs_bits((float)h[0])), abs_bits((float)h[1]));
}

// Per-tensor scales, first pass: the amax of one chunk, as sumsq_range reads it.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_quant_amax(const QuantDesc* __restrict__ descs,
                                                         const int32_t* __restrict__ chunk_tid,
                                                         uint32_t* __restrict__ amax) {
  constexpr int kBytes = DT == FP8ADAM_F32 ? 4 : 2, kVec = 16 / kBytes;
  const int64_t w = blockIdx.x;
  const QuantDesc d = descs[chunk_tid[w]];
  const int64_t lo = (w - d.chunk0) * d.chunk_len, n = min(d.chunk_len, d.numel - lo);
  const char* base = static_cast<const char*>(d.x) + kBytes * lo;
  const int64_t head = min(n, (int64_t)((16u - ((uintptr_t)base & 15u)) & 15u) / kBytes);
  const int64_t nvec = (n - head) / kVec, tail = head + nvec * kVec;
  uint32_t am = 0, none = 0;
  // a piece at a time, so that offsets into the buffer resource stay small
  constexpr int64_t kPiece = (int64_t)1 << 20;
  for (int64_t v0 = 0; v0 < nvec; v0 += kPiece) {
    const int nv = (int)min(kPiece, nvec - v0);
    const Rsrc r = rsrc(base + kBytes * head + 16 * v0, 16 * (int64_t)nv);
    for (int v = threadIdx.x; v < nv; v += kThreads * kSumUnroll) {
      vu4 x[kSumUnroll];
#pragma unroll
      for (int u = 0; u < kSumUnroll; u++)
        x[u] = __builtin_amdgcn_raw_buffer_load_b128(r, 16 * (v + u * kThreads), 0, kLdPol);
#pragma unroll
      for (int u = 0; u < kSumUnroll; u++)
#pragma unroll
        for (int j = 0; j < 4; j++) am = amax_word<DT>(am, x[u][j]);
    }
  }
  const int64_t single = (int64_t)threadIdx.x < head ? (int64_t)threadIdx.x : tail + (int64_t)threadIdx.x - head;
  if (single < n) am = max(am, abs_bits(ld_elem<DT>(base, single)));
  block_max2(am, none);
  if (threadIdx.x == 0) amax[d.slot0 + (w - d.chunk0)] = am;
}

// The tensor's scale from its chunk maxima: at most kAmaxMaxChunks of them, one
// 16-byte load per lane, from the L2.
struct TensorScale {
  vu4 maxima;
  __device__ __forceinline__ TensorScale(const uint32_t* amax, const QuantDesc& d)
      : maxima(__builtin_amdgcn_raw_buffer_load_b128(rsrc(amax + d.slot0, 4 * d.slots), 16 * (threadIdx.x & 63), 0, 0)) {}
  // called by whole waves
  template <int FMT>
  __device__ __forceinline__ void get(int smode, float& s, float& inv, bool& odd) const {
    const uint32_t am = wave_max(max(max(maxima.x, maxima.y), max(maxima.z, maxima.w)));
    choose_scale_mode<FMT>(am, smode, s, inv);
    odd = nonfinite_amax(am);
  }
};

// The maxima are loaded first, then the values: the scale is ready when they arrive.
template <bool DWORD, int DT, int FMT>
__device__ __forceinline__ void quant_tensor_whole(const QuantDesc& d, int64_t lo, const TensorScale& t, int smode,
                                                   float& s, float& inv, bool& odd) {
  constexpr int64_t kLen = (int64_t)1 << kQuantTensorPartLog2;
  constexpr int kU = (int)(kLen / kSubTile);
  const Stream<DT, DWORD> sx(d.x, lo, kLen);
  const Stream<kCodes, DWORD> sc(d.codes, lo, kLen);
  Raw4<DT> r[kU];
#pragma unroll
  for (int u = 0; u < kU; u++) r[u] = sx.load(4 * threadIdx.x + u * kSubTile);
  t.get<FMT>(smode, s, inv, odd);
#pragma unroll
  for (int u = 0; u < kU; u++) {
    float x[4];
    unpack4<DT>(r[u], x);
    sc.store(4 * threadIdx.x + u * kSubTile, Raw4<kCodes>{codes4<FMT>(x, inv, odd)});
  }
}

// Second pass: every wave makes its tensor's scale and quantizes its share of the
// part.  Bound by HBM: 202M bf16 values in 61 us (first pass) and 89 us (6.8 TB/s); a
// list past the caches is read twice, since the scale needs all of a tensor.
template <int DT, int FMT>
__global__ __launch_bounds__(kThreads) void k_quant_tensor(const QuantDesc* __restrict__ descs,
                                                           const int32_t* __restrict__ part_tid, int64_t nparts,
                                                           const uint32_t* __restrict__ amax, int smode) {
  constexpr int64_t kLen = (int64_t)1 << kQuantTensorPartLog2;
  const int64_t w = run_index(nparts);
  if (w < 0) return;
  const QuantDesc d = descs[part_tid[w]];
  const int64_t lo = d.head + ((w - d.part0) << kQuantTensorPartLog2);
  const bool whole = lo + kLen <= d.numel;
  const TensorScale t(amax, d);
  float s, inv;
  bool odd;
  if (d.vec && whole) quant_tensor_whole<true, DT, FMT>(d, lo, t, smode, s, inv, odd);
  else if (!whole) t.get<FMT>(smode, s, inv, odd);
  else quant_tensor_whole<false, DT, FMT>(d, lo, t, smode, s, inv, odd);
  const bool first = w == d.part0;
  if (first && threadIdx.x == 0) st_global<float>(d.scale, s);
  // what is not in groups: all of another part, and the elements in front of the first
  const int64_t from = first ? 0 : lo, to = whole ? first ? (int64_t)d.head : lo : min(lo + kLen, d.numel);
  for (int64_t i = from + threadIdx.x; i < to; i += kThreads) {
    const float x[4] = {ld_elem<DT>(d.x, i), 0.0f, 0.0f, 0.0f};
    st_global<uint8_t>(d.codes + i, (uint8_t)codes4<FMT>(x, inv, odd));
  }
}

template <bool DWORD, int PL, int DT, int FMT, bool BLK>
__device__ __forceinline__ void dequant_whole(const QuantDesc& d, int64_t lo) {
  constexpr int64_t kLen = (int64_t)1 << PL;
  constexpr int kU = (int)(kLen / kSubTile);
  const Stream<DT, DWORD> sx(d.x, lo, kLen);
  const Stream<kCodes, DWORD> sc(d.codes, lo, kLen);
  Raw4<kCodes> c[kU];
  float s[kU];
#pragma unroll
  for (int u = 0; u < kU; u++) {
    c[u] = sc.load(4 * threadIdx.x + u * kSubTile);
    s[u] = ld_global<float>(d.scale + (BLK ? (lo >> 7) + 8 * u + (threadIdx.x >> 5) : 0));
  }
#pragma unroll
  for (int u = 0; u < kU; u++) {
    float x[4];
    decode4<FMT>(c[u].x, x);
#pragma unroll
    for (int j = 0; j < 4; j++) x[j] *= s[u];
    sx.store(4 * threadIdx.x + u * kSubTile, pack4<DT>(x));
  }
}

// Back to values: 109.5M E5M2 codes to fp32 in 83 us, 6.6 TB/s, bound by the writes
// (four bytes of five).
template <int DT, int FMT, bool BLK>
__global__ __launch_bounds__(kThreads) void k_dequant(const QuantDesc* __restrict__ descs,
                                                      const int32_t* __restrict__ part_tid, int64_t nparts) {
  constexpr int PL = BLK ? kQuantPartLog2 : kQuantTensorPartLog2;
  constexpr int64_t kLen = (int64_t)1 << PL;
  const int64_t w = run_index(nparts);
  if (w < 0) return;
  const QuantDesc d = descs[part_tid[w]];
  const int64_t lo = d.head + ((w - d.part0) << PL);
  const bool whole = lo + kLen <= d.numel, first = w == d.part0;
  if (d.vec && whole) dequant_whole<true, PL, DT, FMT, BLK>(d, lo);
  else if (whole) dequant_whole<false, PL, DT, FMT, BLK>(d, lo);
  const int64_t from = first ? 0 : lo, to = whole ? first ? (int64_t)d.head : lo : min(lo + kLen, d.numel);
  for (int64_t i = from + threadIdx.x; i < to; i += kThreads)
    st_elem<DT>(d.x, i, decode1<FMT>(ld_global<uint8_t>(d.codes + i)) * ld_global<float>(d.scale + (BLK ? i >> 7 : 0)));
}

// ------------------------------------------------------------------- host side

enum PlanKind { kPlanAdamw = 0, kPlanClip = 1, kPlanQuant = 2 };

// The parts of one kind of tensor.
struct Span {
  AdamwKind kind{};          // AdamW
  int dtype = 0, format = 0; // conversion
  std::vector<int32_t> tid;  // part -> tensor (host copy, until it is uploaded)
  const int32_t* d_tid = nullptr;
  int64_t nparts = 0;
  std::vector<int32_t> ctid; // amax chunk -> tensor
  const int32_t* d_ctid = nullptr;
  int64_t nchunks = 0;
};

bool valid_dtype(int32_t d) { return d >= FP8ADAM_F32 && d <= FP8ADAM_F16; }
bool valid_format(int32_t f) { return f == FP8ADAM_E4M3 || f == FP8ADAM_E5M2; }

// Elements of one plan: every launch has to fit one grid dimension (2^32 - 1
// work-items of work-groups of 1024 elements).
constexpr int64_t kMaxGroupsPerLaunch = ((int64_t)UINT32_MAX / kThreads) / (8 * kXcdRun) * (8 * kXcdRun);

std::string of_tensor(const char* what, int32_t t) { return std::string(what) + " of tensor " + std::to_string(t); }

// The memory ranges of a list: what a call writes may not overlap anything else.
struct Range {
  uintptr_t lo, hi;
  bool written;
  int32_t tensor;
};

struct Ranges {
  std::vector<Range> all;
  // One tensor of n elements of `bytes` each: null and alignment are checked too.
  int add(const void* p, int64_t n, int64_t bytes, bool written, const char* what, int32_t t) {
    if (!p) return fail(FP8ADAM_EINVAL, of_tensor(what, t) + " is null");
    const uintptr_t a = (uintptr_t)p;
    if (a % (uintptr_t)bytes)
      return fail(FP8ADAM_EALIGN, of_tensor(what, t) + " is not aligned to its element size (" + std::to_string(bytes) + ")");
    all.push_back(Range{a, a + (uintptr_t)(n * bytes), written, t});
    return 0;
  }
  int check() {
    std::sort(all.begin(), all.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    const Range *any = nullptr, *written = nullptr;  // the earlier ranges that reach furthest
    for (const Range& r : all) {
      const Range* hit = written && r.lo < written->hi ? written : r.written && any && r.lo < any->hi ? any : nullptr;
      if (hit)
        return fail(FP8ADAM_EINVAL, "memory that the call writes overlaps other memory of the list (tensors " +
                                        std::to_string(hit->tensor) + " and " + std::to_string(r.tensor) + ")");
      if (!any || r.hi > any->hi) any = &r;
      if (r.written && (!written || r.hi > written->hi)) written = &r;
    }
    return 0;
  }
};

int check_numel(int64_t numel, int64_t& total, int32_t t) {
  if (numel < 0) return fail(FP8ADAM_EINVAL, of_tensor("numel", t) + " is negative");
  constexpr int64_t most = kMaxGroupsPerLaunch << 10;
  if (numel > most || (total += numel) > most)
    return fail(FP8ADAM_EINVAL, "too many elements for one plan (at most " + std::to_string(most) +
                                    "); split the list over several plans");
  return 0;
}

int check_parts(int64_t parts) {
  if (parts > kMaxGroupsPerLaunch)
    return fail(FP8ADAM_EINVAL, "too many elements for one plan once each tensor is rounded up to whole parts");
  return 0;
}

}  // namespace
}  // namespace fp8adam_list

struct fp8adam_plan {
  PlanKind kind = kPlanAdamw;
  int device = 0;
  int mf = 0, vf = 0, n_groups = 1;       // AdamW
  int granularity = 0, smode = 0;         // conversion
  std::vector<Span> spans;
  unsigned char* mem = nullptr;           // one allocation: descriptors, tables, workspace
  const void* d_desc = nullptr;
  // the gradient list (AdamW and clipping)
  const GradDesc* d_grad = nullptr;
  const int32_t* d_grad_tid = nullptr;
  int64_t grad_chunks = 0;
  int grad_chunk_log2 = 0;
  int64_t clip_parts = 0;                 // clipping: work-groups of the second pass (0: nothing is written)
  double* d_partial = nullptr;
  uint32_t* d_ticket = nullptr;           // AdamW with loss scaling, few chunks: zero between calls
  AdamwCtl* d_ctl = nullptr;
  uint32_t* d_amax = nullptr;             // conversion with per-tensor scales: one per chunk
  int norm_groups() const { return (int)std::min<int64_t>(grad_chunks, kListNormGroups); }
  ~fp8adam_plan() {
    if (mem) (void)hipFree(mem);
  }
};

namespace fp8adam_list {
namespace {

// The device image of a plan: pieces at 256-byte offsets of one allocation.
struct Image {
  std::vector<unsigned char> bytes;  // what is uploaded
  size_t size = 0;                   // and the workspace behind it
  size_t put(const void* p, size_t n) {
    const size_t at = bytes.size();
    bytes.resize((at + n + 255) & ~(size_t)255);
    if (n) memcpy(bytes.data() + at, p, n);
    size = bytes.size();
    return at;
  }
  size_t room(size_t n) {  // after every put
    const size_t at = size;
    size = (size + n + 255) & ~(size_t)255;
    return at;
  }
  int upload(fp8adam_plan* p, hipStream_t stream) {
    hipError_t e = hipMalloc((void**)&p->mem, std::max<size_t>(size, 256));
    if (e == hipErrorOutOfMemory) {
      (void)hip_fail(e, "hipMalloc");  // (takes the error from the runtime)
      return fail(FP8ADAM_ENOMEM, "device allocation failed");
    }
    if (e == hipSuccess && !bytes.empty())
      e = hipMemcpyAsync(p->mem, bytes.data(), bytes.size(), hipMemcpyHostToDevice, stream);
    if (e == hipSuccess) e = hipStreamSynchronize(stream);
    return e == hipSuccess ? 0 : hip_fail(e, "uploading the plan");
  }
};

// The current device, which the stream has to belong to.  Building allocates, copies and waits,
// which a capture neither records nor survives: a stream that is being captured is refused first.
int plan_device(fp8adam_plan* p, hipStream_t stream) {
  hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
  HIP_TRY(hipStreamIsCapturing(stream, &capture));
  if (capture != hipStreamCaptureStatusNone)
    return fail(FP8ADAM_EINVAL, "the stream is being captured: build the plan before the capture");
  HIP_TRY(hipGetDevice(&p->device));
  hipDevice_t dev = -1;
  HIP_TRY(hipStreamGetDevice(stream, &dev));
  if (dev != p->device)
    return fail(FP8ADAM_EINVAL, "the stream belongs to device " + std::to_string(dev) + ", not the current device " +
                                    std::to_string(p->device));
  return 0;
}

int check_call(const fp8adam_plan* p, PlanKind kind, const char* what, hipStream_t stream) {
  if (!p) return fail(FP8ADAM_EINVAL, "plan is null");
  if (p->kind != kind) return fail(FP8ADAM_EINVAL, std::string("the plan is not one of ") + what);
  hipDevice_t dev = -1;
  HIP_TRY(hipStreamGetDevice(stream, &dev));
  if (dev != p->device)
    return fail(FP8ADAM_EINVAL, "the stream belongs to device " + std::to_string(dev) + ", the plan to device " +
                                    std::to_string(p->device));
  return 0;
}

// Chunks of the gradient list: the largest power of two of 4096 .. 32768
// elements that still gives the norm pass a work-group for each of its places.
void chunk_grads(std::vector<GradDesc>& g, int64_t total, int& chunk_log2, std::vector<int32_t>& tid) {
  chunk_log2 = kGradChunkMaxLog2;
  while (chunk_log2 > kGradChunkMinLog2 && (total >> chunk_log2) < kListNormGroups) chunk_log2--;
  for (size_t t = 0; t < g.size(); t++) {
    g[t].chunk0 = (int64_t)tid.size();
    const int64_t nc = (g[t].numel + ((int64_t)1 << chunk_log2) - 1) >> chunk_log2;
    tid.insert(tid.end(), (size_t)nc, (int32_t)t);
  }
}

int launch_sumsq(const fp8adam_plan* p, hipStream_t s) {
  if (!p->grad_chunks) return 0;
  return launch(k_list_sumsq, dim3((unsigned)p->norm_groups()), dim3(kThreads), 0, s, p->d_grad, p->d_grad_tid,
                p->grad_chunks, p->grad_chunk_log2, p->d_partial);
}

int run_adamw(fp8adam_plan* p, const AdamwConsts& C, const AdamwCtl* ctl, hipStream_t s) {
  const AdamwDesc* d = static_cast<const AdamwDesc*>(p->d_desc);
  for (const Span& k : p->spans) {
    int r;
    if (!k.kind.moments8) r = launch_adamw<false, 0, 0>(k.kind, d, k.d_tid, C, k.nparts, ctl, s);
    else if (p->mf == 0 && p->vf == 1) r = launch_adamw<true, 0, 1>(k.kind, d, k.d_tid, C, k.nparts, ctl, s);
    else if (p->mf == 0) r = launch_adamw<true, 0, 0>(k.kind, d, k.d_tid, C, k.nparts, ctl, s);
    else if (p->vf == 0) r = launch_adamw<true, 1, 0>(k.kind, d, k.d_tid, C, k.nparts, ctl, s);
    else r = launch_adamw<true, 1, 1>(k.kind, d, k.d_tid, C, k.nparts, ctl, s);
    if (r) return r;
  }
  return 0;
}

int check_groups(const fp8adam_plan* p, const fp8adam_adamw_hparams* h, int32_t n_groups) {
  if (!h) return fail(FP8ADAM_EINVAL, "groups is null");
  if (n_groups != p->n_groups)
    return fail(FP8ADAM_EINVAL, "n_groups is " + std::to_string(n_groups) + ", the plan has " + std::to_string(p->n_groups));
  for (int q = 0; q < n_groups; q++) {
    if (!(h[q].beta1 >= 0.0 && h[q].beta1 < 1.0) || !(h[q].beta2 >= 0.0 && h[q].beta2 < 1.0))
      return fail(FP8ADAM_EINVAL, "beta1 and beta2 must lie in [0, 1)");
    if (!(h[q].eps >= 0.0) || !isfinite(h[q].eps)) return fail(FP8ADAM_EINVAL, "eps must be finite and >= 0");
    if (!isfinite(h[q].lr) || !isfinite(h[q].weight_decay))
      return fail(FP8ADAM_EINVAL, "lr and weight_decay must be finite");
    // what the kernels take of them in fp32 (1 / (1 - beta) bounds the bias corrections)
    const double sc = denom_scale((float)h[q].eps);
    if (!isfinite((float)(h[q].lr * sc / (1.0 - h[q].beta1))) || !isfinite((float)(h[q].lr * h[q].weight_decay)) ||
        !isfinite((float)h[q].eps) || !isfinite((float)(sc * sc / (1.0 - h[q].beta2))))
      return fail(FP8ADAM_EINVAL, "lr, lr * weight_decay, lr / (1 - beta1), 1 / (1 - beta2) and eps must be finite in fp32");
  }
  return 0;
}

// t < 1: the bias corrections come from the device.
void group_consts(const fp8adam_adamw_hparams* h, int n_groups, int64_t t, AdamwConsts& C) {
  for (int q = 0; q < n_groups; q++) {
    GroupConsts& c = C.g[q];
    c.b1 = (float)h[q].beta1;
    c.omb1 = (float)(1.0 - h[q].beta1);
    c.b2 = (float)h[q].beta2;
    c.omb2 = (float)(1.0 - h[q].beta2);
    c.lr_wd = (float)(h[q].lr * h[q].weight_decay);
    const double sc = denom_scale((float)h[q].eps);
    c.eps = (float)((float)h[q].eps * sc);
    c.step_size = t < 1 ? 0.0f : (float)(h[q].lr * sc / (1.0 - pow(h[q].beta1, (double)t)));
    c.inv_bc2 = t < 1 ? 0.0f : (float)(sc * sc / (1.0 - pow(h[q].beta2, (double)t)));
  }
}

template <int DT, int FMT>
int run_quantize(fp8adam_plan* p, const Span& k, hipStream_t s) {
  const QuantDesc* d = static_cast<const QuantDesc*>(p->d_desc);
  const dim3 grid(run_grid(k.nparts));
  if (p->granularity == FP8ADAM_SCALE_BLOCK128)
    return launch(k_quant_block<DT, FMT>, grid, dim3(kThreads), 0, s, d, k.d_tid, k.nparts, p->smode);
  if (int r = launch(k_quant_amax<DT>, dim3((unsigned)k.nchunks), dim3(kThreads), 0, s, d, k.d_ctid, p->d_amax)) return r;
  return launch(k_quant_tensor<DT, FMT>, grid, dim3(kThreads), 0, s, d, k.d_tid, k.nparts, p->d_amax, p->smode);
}

// Dequantizing writes four bytes of five (two of three): as many work-groups on a CU
// as write 48 KB between them.  109.5M codes to fp32: by blocks (8 KB each) 83 us
// with six against 93 with eight (five: 86), by tensors (16 KB) 85 with three
// against 99; to bf16 by tensors (8 KB) 53 against 54; by blocks (4 KB) eight are
// fastest.
constexpr unsigned dequant_lds(int part_log2, int dt) {
  return lds_for((int)std::min<int64_t>(8, (48 << 10) / (dtype_bytes(dt) << part_log2)));
}

template <int DT, int FMT>
int run_dequantize(fp8adam_plan* p, const Span& k, hipStream_t s) {
  const QuantDesc* d = static_cast<const QuantDesc*>(p->d_desc);
  const dim3 grid(run_grid(k.nparts));
  if (p->granularity == FP8ADAM_SCALE_BLOCK128)
    return launch(k_dequant<DT, FMT, true>, grid, dim3(kThreads), dequant_lds(kQuantPartLog2, DT), s, d, k.d_tid, k.nparts);
  return launch(k_dequant<DT, FMT, false>, grid, dim3(kThreads), dequant_lds(kQuantTensorPartLog2, DT), s, d, k.d_tid,
                k.nparts);
}

template <int FMT>
int run_convert(fp8adam_plan* p, const Span& k, bool back, hipStream_t s) {
  if (k.dtype == FP8ADAM_F32)
    return back ? run_dequantize<FP8ADAM_F32, FMT>(p, k, s) : run_quantize<FP8ADAM_F32, FMT>(p, k, s);
  if (k.dtype == FP8ADAM_BF16)
    return back ? run_dequantize<FP8ADAM_BF16, FMT>(p, k, s) : run_quantize<FP8ADAM_BF16, FMT>(p, k, s);
  return back ? run_dequantize<FP8ADAM_F16, FMT>(p, k, s) : run_quantize<FP8ADAM_F16, FMT>(p, k, s);
}

int convert(fp8adam_plan* p, bool back, hipStream_t stream) {
  if (int r = check_call(p, kPlanQuant, "fp8adam_quant_plan", stream)) return r;
  for (const Span& k : p->spans)
    if (int r = k.format == FP8ADAM_E4M3 ? run_convert<0>(p, k, back, stream) : run_convert<1>(p, k, back, stream))
      return r;
  return 0;
}

// A new plan, freed unless it is handed out.
struct NewPlan {
  fp8adam_plan* p = new fp8adam_plan();
  ~NewPlan() { delete p; }
  fp8adam_plan* release() {
    fp8adam_plan* q = p;
    p = nullptr;
    return q;
  }
};

int adamw_plan(fp8adam_plan** out, const fp8adam_adamw_tensor* T, int32_t n, const fp8adam_adamw_config* cfg,
               hipStream_t stream) {
  if (!T || !cfg) return fail(FP8ADAM_EINVAL, "tensors or cfg is null");
  if (n <= 0) return fail(FP8ADAM_EINVAL, "n must be positive");
  if (!valid_format(cfg->m_format) || !valid_format(cfg->v_format))
    return fail(FP8ADAM_EINVAL, "m_format / v_format must be FP8ADAM_E4M3 or FP8ADAM_E5M2");
  if (cfg->n_groups < 1 || cfg->n_groups > FP8ADAM_MAX_GROUPS)
    return fail(FP8ADAM_EINVAL, "n_groups must lie in [1, " + std::to_string(FP8ADAM_MAX_GROUPS) + "]");
  int64_t total = 0;
  Ranges ranges;
  for (int32_t t = 0; t < n; t++) {
    const fp8adam_adamw_tensor& x = T[t];
    if (int r = check_numel(x.numel, total, t)) return r;
    if (!valid_dtype(x.param_dtype) || !valid_dtype(x.grad_dtype)) return fail(FP8ADAM_EINVAL, of_tensor("bad dtype", t));
    if (x.copy && (x.param_dtype != FP8ADAM_F32 || (x.copy_dtype != FP8ADAM_BF16 && x.copy_dtype != FP8ADAM_F16)))
      return fail(FP8ADAM_EINVAL, of_tensor("copy", t) + " must be bf16 or fp16, and its weights fp32");
    if (x.moments != FP8ADAM_MOMENTS_32 && x.moments != FP8ADAM_MOMENTS_8)
      return fail(FP8ADAM_EINVAL, of_tensor("bad moments", t));
    if (x.group < 0 || x.group >= cfg->n_groups) return fail(FP8ADAM_EINVAL, of_tensor("group", t) + " is out of range");
    if (x.numel == 0) continue;
    const bool s8 = x.moments == FP8ADAM_MOMENTS_8;
    if (int r = ranges.add(x.param, x.numel, dtype_bytes(x.param_dtype), true, "param", t)) return r;
    if (int r = ranges.add(x.grad, x.numel, dtype_bytes(x.grad_dtype), false, "grad", t)) return r;
    if (int r = ranges.add(x.m, x.numel, s8 ? 1 : 4, true, "m", t)) return r;
    if (int r = ranges.add(x.v, x.numel, s8 ? 1 : 4, true, "v", t)) return r;
    if (x.copy)
      if (int r = ranges.add(x.copy, x.numel, 2, true, "copy", t)) return r;
    if (s8) {
      const int64_t ns = (x.numel + kBlock - 1) / kBlock;
      if (int r = ranges.add(x.m_scale, ns, 4, true, "m_scale", t)) return r;
      if (int r = ranges.add(x.v_scale, ns, 4, true, "v_scale", t)) return r;
    }
  }
  if (int r = ranges.check()) return r;

  NewPlan np;
  fp8adam_plan* p = np.p;
  p->kind = kPlanAdamw;
  p->mf = cfg->m_format;
  p->vf = cfg->v_format;
  p->n_groups = cfg->n_groups;
  std::vector<AdamwDesc> desc((size_t)n);
  std::vector<GradDesc> grads((size_t)n);
  for (int32_t t = 0; t < n; t++) {
    const fp8adam_adamw_tensor& x = T[t];
    grads[t] = GradDesc{x.grad, nullptr, x.numel, 0, x.grad_dtype, 0};
    const bool s8 = x.moments == FP8ADAM_MOMENTS_8;
    desc[t] = AdamwDesc{x.param, x.grad, x.copy, x.m, x.v, x.m_scale, x.v_scale, x.numel, 0, x.group, 0, 0, 0};
    if (x.numel == 0) continue;
    const AdamwKind kind{x.param_dtype, x.copy ? x.copy_dtype : 0, x.grad_dtype, s8};
    // Streams that start on dwords: fp32 ones always do; 16-bit ones with 32-bit moments either at
    // element 0 or, if all are off by one, at element 1; blocks of codes start at element 0.
    auto odd = [](const void* q, int dt) { return dt == FP8ADAM_F32 ? -1 : (int)((uintptr_t)q >> 1 & 1); };
    int off = -1;
    bool vec = !s8 || (((uintptr_t)x.m | (uintptr_t)x.v) & 3u) == 0;
    for (int o : {odd(x.param, x.param_dtype), odd(x.grad, x.grad_dtype), x.copy ? odd(x.copy, x.copy_dtype) : -1}) {
      vec = vec && (o < 0 || off < 0 || o == off);
      off = std::max(off, o);
    }
    vec = vec && !(s8 && off == 1);
    desc[t].vec = vec ? 1 : 0;
    desc[t].head = vec && off == 1 ? 1 : 0;
    auto it = std::find_if(p->spans.begin(), p->spans.end(), [&](const Span& k) { return k.kind == kind; });
    if (it == p->spans.end()) {
      p->spans.emplace_back();
      it = p->spans.end() - 1;
      it->kind = kind;
    }
    desc[t].part0 = (int64_t)it->tid.size();
    const int pl = adamw_part_log2(x.param_dtype, s8);
    const int64_t parts = std::max<int64_t>(1, (x.numel - desc[t].head + ((int64_t)1 << pl) - 1) >> pl);
    if (int r = check_parts(desc[t].part0 + parts)) return r;
    it->tid.insert(it->tid.end(), (size_t)parts, t);
  }
  std::vector<int32_t> gtid;
  chunk_grads(grads, total, p->grad_chunk_log2, gtid);
  p->grad_chunks = (int64_t)gtid.size();
  if (int r = plan_device(p, stream)) return r;
  Image im;
  const size_t at_desc = im.put(desc.data(), sizeof(AdamwDesc) * desc.size());
  const size_t at_grad = im.put(grads.data(), sizeof(GradDesc) * grads.size());
  const size_t at_gtid = im.put(gtid.data(), sizeof(int32_t) * gtid.size());
  std::vector<size_t> at;
  for (Span& k : p->spans) at.push_back(im.put(k.tid.data(), sizeof(int32_t) * k.tid.size()));
  const uint32_t zero = 0;
  const size_t at_ticket = im.put(&zero, sizeof(zero));
  const size_t at_partial = im.room(sizeof(double) * kListNormGroups), at_ctl = im.room(sizeof(AdamwCtl));
  if (int r = im.upload(p, stream)) return r;
  p->d_desc = p->mem + at_desc;
  p->d_grad = reinterpret_cast<const GradDesc*>(p->mem + at_grad);
  p->d_grad_tid = reinterpret_cast<const int32_t*>(p->mem + at_gtid);
  p->d_partial = reinterpret_cast<double*>(p->mem + at_partial);
  p->d_ticket = reinterpret_cast<uint32_t*>(p->mem + at_ticket);
  p->d_ctl = reinterpret_cast<AdamwCtl*>(p->mem + at_ctl);
  for (size_t k = 0; k < at.size(); k++) {
    p->spans[k].d_tid = reinterpret_cast<const int32_t*>(p->mem + at[k]);
    p->spans[k].nparts = (int64_t)p->spans[k].tid.size();
    std::vector<int32_t>().swap(p->spans[k].tid);
  }
  *out = np.release();
  return 0;
}

int clip_plan(fp8adam_plan** out, const fp8adam_clip_tensor* T, int32_t n, hipStream_t stream) {
  if (!T) return fail(FP8ADAM_EINVAL, "tensors is null");
  if (n <= 0) return fail(FP8ADAM_EINVAL, "n must be positive");
  int64_t total = 0;
  Ranges ranges;
  for (int32_t t = 0; t < n; t++) {
    const fp8adam_clip_tensor& x = T[t];
    if (int r = check_numel(x.numel, total, t)) return r;
    if (!valid_dtype(x.src_dtype) || (x.dst && !valid_dtype(x.dst_dtype)))
      return fail(FP8ADAM_EINVAL, of_tensor("bad dtype", t));
    if (x.numel == 0) continue;
    const bool in_place = x.dst == x.src;
    if (in_place && x.dst && x.dst_dtype != x.src_dtype)
      return fail(FP8ADAM_EINVAL, of_tensor("dst", t) + " is src itself, so it must have its type");
    if (int r = ranges.add(x.src, x.numel, dtype_bytes(x.src_dtype), in_place, "src", t)) return r;
    if (x.dst && !in_place)
      if (int r = ranges.add(x.dst, x.numel, dtype_bytes(x.dst_dtype), true, "dst", t)) return r;
  }
  if (int r = ranges.check()) return r;
  NewPlan np;
  fp8adam_plan* p = np.p;
  p->kind = kPlanClip;
  std::vector<GradDesc> grads((size_t)n);
  for (int32_t t = 0; t < n; t++)
    grads[t] = GradDesc{T[t].src, T[t].dst, T[t].numel, 0, T[t].src_dtype, T[t].dst_dtype};
  std::vector<int32_t> gtid;
  chunk_grads(grads, total, p->grad_chunk_log2, gtid);
  p->grad_chunks = (int64_t)gtid.size();
  if (std::any_of(grads.begin(), grads.end(), [](const GradDesc& g) { return g.numel > 0 && g.dst; }))
    p->clip_parts = p->grad_chunks << (p->grad_chunk_log2 - kClipPartLog2);
  if (int r = check_parts(p->clip_parts)) return r;
  if (int r = plan_device(p, stream)) return r;
  Image im;
  const size_t at_grad = im.put(grads.data(), sizeof(GradDesc) * grads.size());
  const size_t at_gtid = im.put(gtid.data(), sizeof(int32_t) * gtid.size());
  const size_t at_partial = im.room(sizeof(double) * kListNormGroups);
  if (int r = im.upload(p, stream)) return r;
  p->d_grad = reinterpret_cast<const GradDesc*>(p->mem + at_grad);
  p->d_grad_tid = reinterpret_cast<const int32_t*>(p->mem + at_gtid);
  p->d_partial = reinterpret_cast<double*>(p->mem + at_partial);
  *out = np.release();
  return 0;
}

int quant_plan(fp8adam_plan** out, const fp8adam_quant_tensor* T, int32_t n, const fp8adam_quant_config* cfg,
               hipStream_t stream) {
  if (!T || !cfg) return fail(FP8ADAM_EINVAL, "tensors or cfg is null");
  if (n <= 0) return fail(FP8ADAM_EINVAL, "n must be positive");
  if (cfg->granularity != FP8ADAM_SCALE_TENSOR && cfg->granularity != FP8ADAM_SCALE_BLOCK128)
    return fail(FP8ADAM_EINVAL, "bad granularity");
  if (cfg->scale_mode != FP8ADAM_SCALE_POW2 && cfg->scale_mode != FP8ADAM_SCALE_AMAX)
    return fail(FP8ADAM_EINVAL, "bad scale_mode");
  const bool block = cfg->granularity == FP8ADAM_SCALE_BLOCK128;
  int64_t total = 0;
  Ranges ranges;
  for (int32_t t = 0; t < n; t++) {
    const fp8adam_quant_tensor& x = T[t];
    if (int r = check_numel(x.numel, total, t)) return r;
    if (!valid_dtype(x.dtype)) return fail(FP8ADAM_EINVAL, of_tensor("bad dtype", t));
    if (!valid_format(x.format)) return fail(FP8ADAM_EINVAL, of_tensor("bad format", t));
    if (x.numel == 0) continue;
    if (int r = ranges.add(x.values, x.numel, dtype_bytes(x.dtype), true, "values", t)) return r;
    if (int r = ranges.add(x.codes, x.numel, 1, true, "codes", t)) return r;
    if (int r = ranges.add(x.scale, block ? (x.numel + kBlock - 1) / kBlock : 1, 4, true, "scale", t)) return r;
  }
  if (int r = ranges.check()) return r;
  NewPlan np;
  fp8adam_plan* p = np.p;
  p->kind = kPlanQuant;
  p->granularity = cfg->granularity;
  p->smode = cfg->scale_mode;
  const int pl = block ? kQuantPartLog2 : kQuantTensorPartLog2;
  std::vector<QuantDesc> desc((size_t)n);
  int64_t slots = 0;
  for (int32_t t = 0; t < n; t++) {
    const fp8adam_quant_tensor& x = T[t];
    QuantDesc& d = desc[t];
    d = QuantDesc{x.values, x.codes, x.scale, x.numel, 0, 0, 0, 0, 0, 0, 0};
    if (x.numel == 0) continue;
    // the first element from which values and codes both lie on dwords (blocks start at element 0)
    const bool wide = x.dtype == FP8ADAM_F32;
    for (int h = 0; h < (block ? 1 : 4) && !d.vec; h++)
      if ((((uintptr_t)x.codes + h) & 3u) == 0 && (wide || (((uintptr_t)x.values + 2 * h) & 3u) == 0)) {
        d.head = h;
        d.vec = 1;
      }
    auto it = std::find_if(p->spans.begin(), p->spans.end(),
                           [&](const Span& k) { return k.dtype == x.dtype && k.format == x.format; });
    if (it == p->spans.end()) {
      p->spans.emplace_back();
      it = p->spans.end() - 1;
      it->dtype = x.dtype;
      it->format = x.format;
    }
    d.part0 = (int64_t)it->tid.size();
    const int64_t parts = std::max<int64_t>(1, (x.numel - d.head + ((int64_t)1 << pl) - 1) >> pl);
    if (int r = check_parts(d.part0 + parts)) return r;
    it->tid.insert(it->tid.end(), (size_t)parts, t);
    if (!block) {
      d.chunk0 = (int64_t)it->ctid.size();
      const int64_t len = (x.numel + kAmaxMaxChunks - 1) / kAmaxMaxChunks;
      d.chunk_len = (len + kAmaxMinChunk - 1) / kAmaxMinChunk * kAmaxMinChunk;
      const int64_t nc = (x.numel + d.chunk_len - 1) / d.chunk_len;
      it->ctid.insert(it->ctid.end(), (size_t)nc, t);
      d.slot0 = slots;
      d.slots = (int32_t)((nc + 3) & ~(int64_t)3);
      slots += d.slots;
    }
  }
  if (int r = plan_device(p, stream)) return r;
  Image im;
  const size_t at_desc = im.put(desc.data(), sizeof(QuantDesc) * desc.size());
  std::vector<size_t> at, atc;
  for (Span& k : p->spans) {
    at.push_back(im.put(k.tid.data(), sizeof(int32_t) * k.tid.size()));
    atc.push_back(im.put(k.ctid.data(), sizeof(int32_t) * k.ctid.size()));
  }
  const std::vector<uint32_t> zeros((size_t)slots, 0u);
  const size_t at_amax = im.put(zeros.data(), sizeof(uint32_t) * zeros.size());
  if (int r = im.upload(p, stream)) return r;
  p->d_desc = p->mem + at_desc;
  p->d_amax = reinterpret_cast<uint32_t*>(p->mem + at_amax);
  for (size_t k = 0; k < at.size(); k++) {
    Span& s = p->spans[k];
    s.d_tid = reinterpret_cast<const int32_t*>(p->mem + at[k]);
    s.d_ctid = reinterpret_cast<const int32_t*>(p->mem + atc[k]);
    s.nparts = (int64_t)s.tid.size();
    s.nchunks = (int64_t)s.ctid.size();
    std::vector<int32_t>().swap(s.tid);
    std::vector<int32_t>().swap(s.ctid);
  }
  *out = np.release();
  return 0;
}

// Nothing is thrown across the ABI: every entry point runs its body in here.
template <typename F>
int guarded(const char* what, F&& body) {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return fail(FP8ADAM_ENOMEM, "host allocation failed");
  } catch (...) {
    return fail(FP8ADAM_EINVAL, std::string("unexpected error in ") + what);
  }
}

template <typename F>
int guarded_plan(fp8adam_plan** out, const char* what, F&& body) {
  return guarded(what, [&]() -> int {
    if (!out) return fail(FP8ADAM_EINVAL, "out is null");
    *out = nullptr;
    return body();
  });
}

}  // namespace
}  // namespace fp8adam_list

// ================================================================== C ABI

extern "C" {

void fp8adam_plan_destroy(fp8adam_plan* plan) { delete plan; }

int fp8adam_adamw_plan(fp8adam_plan** out, const fp8adam_adamw_tensor* tensors, int32_t n,
                       const fp8adam_adamw_config* cfg, hipStream_t stream) {
  return guarded_plan(out, "fp8adam_adamw_plan", [&] { return adamw_plan(out, tensors, n, cfg, stream); });
}

int fp8adam_clip_plan(fp8adam_plan** out, const fp8adam_clip_tensor* tensors, int32_t n, hipStream_t stream) {
  return guarded_plan(out, "fp8adam_clip_plan", [&] { return clip_plan(out, tensors, n, stream); });
}

int fp8adam_quant_plan(fp8adam_plan** out, const fp8adam_quant_tensor* tensors, int32_t n,
                       const fp8adam_quant_config* cfg, hipStream_t stream) {
  return guarded_plan(out, "fp8adam_quant_plan", [&] { return quant_plan(out, tensors, n, cfg, stream); });
}

int fp8adam_adamw_step(fp8adam_plan* plan, const fp8adam_adamw_hparams* groups, int32_t n_groups, int64_t step,
                       hipStream_t stream) {
  return guarded("fp8adam_adamw_step", [&]() -> int {
    if (int r = check_call(plan, kPlanAdamw, "fp8adam_adamw_plan", stream)) return r;
    if (int r = check_groups(plan, groups, n_groups)) return r;
    if (step < 1) return fail(FP8ADAM_EINVAL, "step must be >= 1");
    AdamwConsts C{};
    group_consts(groups, n_groups, step, C);
    return run_adamw(plan, C, nullptr, stream);
  });
}

int fp8adam_adamw_step_amp(fp8adam_plan* plan, const fp8adam_adamw_hparams* groups, int32_t n_groups,
                           const fp8adam_amp_config* amp, fp8adam_amp_state* state, hipStream_t stream) {
  return guarded("fp8adam_adamw_step_amp", [&]() -> int {
    if (int r = check_call(plan, kPlanAdamw, "fp8adam_adamw_plan", stream)) return r;
    if (int r = check_groups(plan, groups, n_groups)) return r;
    if (!amp || !state) return fail(FP8ADAM_EINVAL, "amp or state is null");
    if ((uintptr_t)state & 7u) return fail(FP8ADAM_EINVAL, "state must be 8-byte aligned");
    if (!(amp->growth_factor > 1.0f) || !isfinite(amp->growth_factor) || !(amp->backoff_factor > 0.0f) ||
        !(amp->backoff_factor < 1.0f) || amp->growth_interval < 1 || !isfinite(amp->max_norm))
      return fail(FP8ADAM_EINVAL, "growth_factor must exceed 1, backoff_factor lie in (0, 1), "
                                  "growth_interval be >= 1 and max_norm be finite");
    AdamwConsts C{};
    group_consts(groups, n_groups, 0, C);
    AmpArgs a{state, plan->d_ctl, *amp, n_groups, {}};
    for (int q = 0; q < n_groups; q++) {
      const double sc = denom_scale((float)groups[q].eps);
      a.R.lr[q] = groups[q].lr * sc;
      a.R.beta1[q] = groups[q].beta1;
      a.R.beta2[q] = groups[q].beta2;
      a.R.v_scale[q] = sc * sc;
    }
    if (plan->grad_chunks > 0 && plan->grad_chunks <= kTicketGroups) {
      if (int r = launch(k_list_sumsq_ctl, dim3((unsigned)plan->grad_chunks), dim3(kThreads), 0, stream, plan->d_grad,
                         plan->d_grad_tid, plan->grad_chunks, plan->grad_chunk_log2, plan->d_partial, plan->d_ticket, a))
        return r;
    } else {
      if (int r = launch_sumsq(plan, stream)) return r;
      if (int r = launch(k_list_ctl, dim3(1), dim3(kThreads), 0, stream, plan->d_partial, plan->norm_groups(), a))
        return r;
    }
    return run_adamw(plan, C, plan->d_ctl, stream);
  });
}

int fp8adam_clip_grads(fp8adam_plan* plan, float max_norm, float* result, hipStream_t stream) {
  return guarded("fp8adam_clip_grads", [&]() -> int {
    if (int r = check_call(plan, kPlanClip, "fp8adam_clip_plan", stream)) return r;
    if (!isfinite(max_norm)) return fail(FP8ADAM_EINVAL, "max_norm must be finite");
    if (!result) return fail(FP8ADAM_EINVAL, "result is null");
    if ((uintptr_t)result & 3u) return fail(FP8ADAM_EALIGN, "result is not 4-byte aligned");
    if (int r = launch_sumsq(plan, stream)) return r;
    return launch(k_list_clip, dim3(run_grid<kClipXcdRun>(std::max<int64_t>(1, plan->clip_parts))), dim3(kThreads), 0,
                  stream, plan->d_grad, plan->d_grad_tid, plan->clip_parts, plan->grad_chunk_log2, plan->d_partial,
                  plan->norm_groups(), max_norm, result);
  });
}

int fp8adam_quantize(fp8adam_plan* plan, hipStream_t stream) {
  return guarded("fp8adam_quantize", [&] { return convert(plan, false, stream); });
}

int fp8adam_dequantize(fp8adam_plan* plan, hipStream_t stream) {
  return guarded("fp8adam_dequantize", [&] { return convert(plan, true, stream); });
}

}  // extern "C"
