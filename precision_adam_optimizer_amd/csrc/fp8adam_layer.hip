// fp8adam_layer.hip -- the layer operators of include/fp8adam_layer.h: conversion of
// matrices to 8 bits and back, the backward pass of the activations, the gradients'
// preparation and plans, and the C ABI.  The products are in fp8adam_layer_product.h and
// fp8adam_layer_grad.h.
#include "fp8adam_layer.h"

using namespace fp8adam;
using namespace fp8adam_engine;
using namespace fp8adam_layer;

namespace fp8adam_layer {

extern template int launch_product<0, 0>(const ProductArgs&, bool, hipStream_t);
extern template int launch_product<0, 1>(const ProductArgs&, bool, hipStream_t);
extern template int launch_product<1, 0>(const ProductArgs&, bool, hipStream_t);
extern template int launch_product<1, 1>(const ProductArgs&, bool, hipStream_t);
extern template int launch_grad<0>(const GradArgs&, const GradPlan&, hipStream_t);
extern template int launch_grad<1>(const GradArgs&, const GradPlan&, hipStream_t);

namespace {

// ------------------------------------------------------------ to 8 bits and back

// Blocks per 16 lanes, whose loads go out together.
constexpr int kPackUnroll = 4;
constexpr int kPackBlocks = kThreads / 16 * kPackUnroll;  // of a work-group

template <int DT>
__global__ __launch_bounds__(kThreads) void k_pack(const void* x, int64_t ld, Out8 o, int64_t rows, int cols, int64_t nb) {
  const int lane = threadIdx.x & 15;
  const int64_t first = (int64_t)blockIdx.x * kPackBlocks + (threadIdx.x >> 4), total = rows * nb;
  float v[kPackUnroll][8];
  int64_t row[kPackUnroll], blk[kPackUnroll];
  bool there[kPackUnroll], inside = true;
#pragma unroll
  for (int u = 0; u < kPackUnroll; u++) {
    const int64_t i = first + u * (kThreads / 16);
    there[u] = i < total;
    const int64_t in = min(i, total - 1);
    row[u] = total >> 32 ? in / nb : (uint32_t)in / (uint32_t)nb;
    blk[u] = in - row[u] * nb;
    inside = inside && 128 * blk[u] + 8 * lane + 8 <= cols;
  }
  if (inside) {  // no branch between the loads: all are on their way at once
#pragma unroll
    for (int u = 0; u < kPackUnroll; u++) ld8<DT>(x, row[u] * ld + 128 * blk[u] + 8 * lane, 8, v[u]);
  } else {
#pragma unroll
    for (int u = 0; u < kPackUnroll; u++) ld8<DT>(x, row[u] * ld + 128 * blk[u] + 8 * lane, cols - 128 * blk[u] - 8 * lane, v[u]);
  }
  put_blocks(o, row, blk, there, lane, v);
}

// Eight codes times their scale.
__device__ __forceinline__ void decode8(int format, const vu2& c, float s, float (&x)[8]) {
#pragma unroll
  for (int q = 0; q < 4; q++) {
    const uint32_t w = q < 2 ? c.x : c.y;
    float v[2];
    if (format == FP8ADAM_E4M3) {
      const auto p = (q & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, true) : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(w, s, false);
      v[0] = p[0], v[1] = p[1];
    } else {
      const auto p = (q & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, s, true) : __builtin_amdgcn_cvt_scalef32_pk_f32_bf8(w, s, false);
      v[0] = p[0], v[1] = p[1];
    }
    x[2 * q] = v[0];
    x[2 * q + 1] = v[1];
  }
}

// A work-group of 16 rows of 16 lanes, eight columns each: a block of 128 columns of
// `chunk` rows.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_unpack(const In8 in, int format, void* x, int64_t ld, int64_t rows, int cols,
                                                     int nb) {
  constexpr int kRows = 64;
  const int64_t r0 = (int64_t)(blockIdx.x / nb) * kRows;
  const int blk = (int)(blockIdx.x % nb);
  const int64_t c = 128 * (int64_t)blk + 8 * (threadIdx.x & 15);
#pragma unroll
  for (int u = 0; u < kRows / 16; u++) {
    const int64_t row = r0 + 16 * u + (threadIdx.x >> 4);
    if (row >= rows || c >= cols) continue;
    float v[8];
    decode8(format, ld_global<vu2>(in.codes + row * in.ld + c), scale_at(in.scales, row * in.ld_scale + blk, in.f32), v);
    st8<DT>(x, row * ld + c, cols - c, v);
  }
}

// --------------------------------------------------- back through the activations

struct ActArgs {
  const void* dy;
  void* dz;
  void* dup;
  int64_t ld_dy, ld_dz, ld_dup;
  In8 z[2];
  int64_t tokens;
  int32_t rows, nb;
  int32_t format[2];
  float* partial;   // [chunks][128 nb], or null
};

constexpr int kActRows = 64;  // of a work-group

// One block of 128 columns of kActRows rows, eight columns per lane: reads and writes at once, bound
// by HBM (4096 x 11008 gated in bf16: 71 us, 5.0 TB/s).  Each row is loaded when the one before has
// been written; all four loaded first took 77 us (twice the registers, half the waves).  The sums over
// the rows, for the bias, are added up in fp32 by each lane and then over the work-group's 16 rows of
// lanes, always in the same order; k_bias_join adds the chunks.
template <bool GATED, int ACT, int DT>
__global__ __launch_bounds__(kThreads) void k_act_backward(const ActArgs a) {
  const int64_t chunk = blockIdx.x / a.nb;
  const int blk = (int)(blockIdx.x % a.nb);
  const int64_t c = 128 * (int64_t)blk + 8 * (threadIdx.x & 15), left = a.rows - c;
  float sum[8] = {};
#pragma unroll
  for (int u = 0; u < kActRows / 16; u++) {
    const int64_t t = chunk * kActRows + 16 * u + (threadIdx.x >> 4);
    if (t >= a.tokens || left <= 0) continue;
    float dy[8], z[8], up[8], da[8], act[8];
    ld8<DT>(a.dy, t * a.ld_dy + c, left, dy);
    if constexpr (GATED || ACT != FP8ADAM_ACT_NONE)
      decode8(a.format[0], ld_global<vu2>(a.z[0].codes + t * a.z[0].ld + c), scale_at(a.z[0].scales, t * a.z[0].ld_scale + blk, a.z[0].f32), z);
    if constexpr (GATED)
      decode8(a.format[1], ld_global<vu2>(a.z[1].codes + t * a.z[1].ld + c), scale_at(a.z[1].scales, t * a.z[1].ld_scale + blk, a.z[1].f32), up);
#pragma unroll
    for (int e = 0; e < 8; e++) {
      if constexpr (GATED || ACT != FP8ADAM_ACT_NONE) act_slope<ACT>(z[e], act[e], da[e]);
      else da[e] = 1.0f;
      if constexpr (GATED) {
        da[e] *= dy[e] * up[e];
        act[e] *= dy[e];
      } else {
        da[e] *= dy[e];
        sum[e] += da[e];
      }
    }
    if constexpr (GATED || ACT != FP8ADAM_ACT_NONE) st8<DT>(a.dz, t * a.ld_dz + c, left, da);
    if constexpr (GATED) st8<DT>(a.dup, t * a.ld_dup + c, left, act);
  }
  if constexpr (!GATED) {
    if (!a.partial) return;
    __shared__ float s[16][128 + 4];
#pragma unroll
    for (int e = 0; e < 8; e++) s[threadIdx.x >> 4][8 * (threadIdx.x & 15) + e] = sum[e];
    __syncthreads();
    if (threadIdx.x >= 128) return;
    float x = 0.0f;
#pragma unroll
    for (int r = 0; r < 16; r++) x += s[r][threadIdx.x];
    st_global<float>(a.partial + (chunk * a.nb + blk) * 128 + threadIdx.x, x);
  }
}

// The bias's gradient from the chunks' sums: 32 columns, eight threads each.
__global__ __launch_bounds__(kThreads) void k_bias_join(const float* partial, int64_t chunks, int64_t ld, int rows, void* out,
                                                        int dt, int accumulate) {
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float x = 0.0f;
  if (c < rows) {
#pragma unroll 4
    for (int64_t k = part; k < chunks; k += 8) x += ld_global<float>(partial + k * ld + c);
  }
  __shared__ float s[8][32];
  s[part][lane] = x;
  __syncthreads();
  if (part || c >= rows) return;
#pragma unroll
  for (int k = 1; k < 8; k++) x += s[k][lane];
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (accumulate) ld4(dt, out, c, 1, o);
  o[0] += x;
  st4(dt, out, c, 1, o);
}

// ----------------------------------------------------------- the gradients' left side

// A gradient as the products take it: bf16 with rows padded to a multiple of 8 (zeros), and where
// it has more bits than bf16 what that part leaves, as a second (the 11 bits of fp16 in 8 + 3), and what these
// leave, as a third (the 24 of fp32 in 8 + 8 + 8).  All but the last are cut, not rounded, so that they never pass the
// largest number and what is left has the bits that follow; a NaN or Inf is in the first part alone.
template <int DT, int PARTS>
__global__ __launch_bounds__(kThreads) void k_split(const void* x, int64_t ld, int64_t rows, int cols, int64_t ldo,
                                                    uint16_t* out, int64_t part) {
  const int64_t groups = ldo >> 3, i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= rows * groups) return;
  const int64_t row = i / groups, c = (i - row * groups) * 8;
  float v[8];
  ld8<DT>(x, row * ld + c, cols - c, v);
#pragma unroll
  for (int p = 0; p < PARTS; p++) {
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; q++) {
      if (p > 0 && p == PARTS - 1) {
        w[q] = fp8adam_list::pack2<FP8ADAM_BF16>(v[2 * q], v[2 * q + 1]);
        continue;
      }
      uint32_t h[2];
#pragma unroll
      for (int e = 0; e < 2; e++) {
        float& x = v[2 * q + e];
        const uint32_t b = __float_as_uint(x);
        const bool odd = (b & 0x7F800000u) == 0x7F800000u;
        h[e] = odd ? f32_to_bf16_rne(x) : b >> 16;
        x = odd ? 0.0f : x - __uint_as_float(b & 0xFFFF0000u);
      }
      w[q] = h[0] | h[1] << 16;
    }
    st_global<vu4>(out + p * part + row * ldo + c, vu4{w[0], w[1], w[2], w[3]});
  }
}

// ------------------------------------------------------------------------ host side

int stream_device(hipStream_t stream) {
  int dev = -1;
  HIP_TRY(hipGetDevice(&dev));
  hipDevice_t of = -1;
  HIP_TRY(hipStreamGetDevice(stream, &of));
  if (of != dev)
    return fail(FP8ADAM_EINVAL, "the stream belongs to device " + std::to_string(of) + ", not the current device " + std::to_string(dev));
  return 0;
}

// What a call reads and writes, as rows of memory.
struct Memory {
  struct Piece {
    uintptr_t lo;
    int64_t row, ld, rows;  // bytes
    bool written;
    const char* name;
    uintptr_t hi() const { return lo + (uintptr_t)((rows - 1) * ld + row); }
  };
  std::vector<Piece> all;

  static bool apart(const Piece& a, const Piece& b) {
    if (a.hi() <= b.lo || b.hi() <= a.lo) return true;
    if (a.rows == 1 || b.rows == 1 || a.ld != b.ld) return false;
    const int64_t d = (int64_t)(b.lo - a.lo) % a.ld, off = d < 0 ? d + a.ld : d;  // columns of one wider matrix
    return off >= a.row && off + b.row <= a.ld;
  }
  void add(const void* p, int64_t row, int64_t ld, int64_t rows, bool written, const char* name) {
    if (rows > 0 && row > 0) all.push_back(Piece{(uintptr_t)p, row, ld, rows, written, name});
  }
  // `same`: two names whose matrices may be one and the same
  int check(std::initializer_list<std::pair<const char*, const char*>> same = {}) const {
    for (size_t i = 0; i < all.size(); i++)
      for (size_t j = i + 1; j < all.size(); j++) {
        const Piece &a = all[i], &b = all[j];
        if ((!a.written && !b.written) || apart(a, b)) continue;
        bool ok = false;
        for (const auto& s : same)
          ok = ok || (((!strcmp(a.name, s.first) && !strcmp(b.name, s.second)) || (!strcmp(b.name, s.first) && !strcmp(a.name, s.second))) &&
                      a.lo == b.lo && a.row == b.row && (a.rows == 1 || a.ld == b.ld));
        if (!ok)
          return fail(FP8ADAM_EINVAL, std::string("memory that the call writes overlaps other memory of it (") + a.name + " and " + b.name + ")");
      }
    return 0;
  }
};

int check_sizes(int64_t tokens, int64_t rows, int64_t cols) {
  if (tokens < 0 || tokens > INT32_MAX) return fail(FP8ADAM_EINVAL, "the number of tokens must lie in [0, 2^31)");
  if (rows < 1 || rows > FP8ADAM_LAYER_MAX_COLS || cols < 1 || cols > FP8ADAM_LAYER_MAX_COLS)
    return fail(FP8ADAM_EINVAL, "rows and cols must lie in [1, " + std::to_string(FP8ADAM_LAYER_MAX_COLS) + "]");
  return 0;
}

int check_matrix(Memory& mem, const fp8adam_matrix& x, int64_t rows, int64_t cols, bool written, const char* name) {
  if (x.dtype < FP8ADAM_F32 || x.dtype > FP8ADAM_F16) return fail(FP8ADAM_EINVAL, std::string("bad dtype of ") + name);
  if (rows > 1 && (x.ld < cols || x.ld > FP8ADAM_LAYER_MAX_LD))
    return fail(FP8ADAM_EINVAL, std::string("ld of ") + name + " must lie in [" + std::to_string(cols) + ", " + std::to_string(FP8ADAM_LAYER_MAX_LD) + "]");
  if (rows == 0) return 0;
  if (!x.data) return fail(FP8ADAM_EINVAL, std::string(name) + " is null");
  const int64_t e = dtype_bytes(x.dtype);
  if ((uintptr_t)x.data % (uintptr_t)e) return fail(FP8ADAM_EALIGN, std::string(name) + " is not aligned to its element size (" + std::to_string(e) + ")");
  mem.add(x.data, e * cols, e * x.ld, rows, written, name);
  return 0;
}

int check_matrix8(Memory& mem, const fp8adam_matrix8& x, int64_t rows, int64_t cols, bool written, const char* name) {
  if (x.format != FP8ADAM_E4M3 && x.format != FP8ADAM_E5M2) return fail(FP8ADAM_EINVAL, std::string("bad format of ") + name);
  if (x.scale_type != FP8ADAM_SCALES_E8M0 && x.scale_type != FP8ADAM_SCALES_F32)
    return fail(FP8ADAM_EINVAL, std::string("bad scale_type of ") + name);
  const bool f32 = x.scale_type == FP8ADAM_SCALES_F32;
  if (written && f32) return fail(FP8ADAM_EINVAL, std::string("the scales of ") + name + ", which the call writes, must be E8M0");
  const int64_t nb = (cols + 127) >> 7, width = 128 * nb, nbs = f32 ? nb : (nb + 3) & ~(int64_t)3;
  if (x.ld < width || x.ld > FP8ADAM_LAYER_MAX_LD || x.ld % 16)
    return fail(FP8ADAM_EINVAL, std::string("ld of ") + name + " must be a multiple of 16 in [" + std::to_string(width) + ", " + std::to_string(FP8ADAM_LAYER_MAX_LD) + "]");
  if (x.ld_scale < nbs || x.ld_scale > FP8ADAM_LAYER_MAX_LD || (!f32 && x.ld_scale % 4))
    return fail(FP8ADAM_EINVAL, std::string("ld_scale of ") + name + " must be at least " + std::to_string(nbs) + (f32 ? "" : " and a multiple of 4"));
  if (rows == 0) return 0;
  if (!x.codes || !x.scales) return fail(FP8ADAM_EINVAL, std::string(name) + " is null");
  if ((uintptr_t)x.codes & 15u) return fail(FP8ADAM_EALIGN, std::string("codes of ") + name + " are not 16-byte aligned");
  if ((uintptr_t)x.scales & 3u) return fail(FP8ADAM_EALIGN, std::string("scales of ") + name + " are not 4-byte aligned");
  mem.add(x.codes, width, x.ld, rows, written, name);
  mem.add(x.scales, f32 ? 4 * nb : nbs, (f32 ? 4 : 1) * x.ld_scale, rows, written, name);
  return 0;
}

int check_groups(int64_t n) {
  return n > (int64_t)(UINT32_MAX / kThreads) ? fail(FP8ADAM_EINVAL, "too many elements for one call") : 0;
}

In8 in8(const fp8adam_matrix8& x) {
  return In8{static_cast<const uint8_t*>(x.codes), x.scales, x.ld, x.ld_scale, x.scale_type == FP8ADAM_SCALES_F32, 0};
}
Out8 out8(const fp8adam_matrix8& x) {
  return Out8{static_cast<uint8_t*>(x.codes), static_cast<uint8_t*>(x.scales), x.ld, x.ld_scale, x.format};
}

int run_pack(const fp8adam_matrix& x, const fp8adam_matrix8& o, int64_t rows, int64_t cols, hipStream_t s) {
  const int64_t nb = (cols + 127) >> 7, groups = (rows * nb + kPackBlocks - 1) / kPackBlocks;
  if (int r = check_groups(groups)) return r;
  auto go = [&](auto kernel) { return launch(kernel, dim3((unsigned)groups), dim3(kThreads), 0, s, x.data, x.ld, out8(o), rows, (int)cols, nb); };
  if (x.dtype == FP8ADAM_F32) return go(k_pack<FP8ADAM_F32>);
  return x.dtype == FP8ADAM_BF16 ? go(k_pack<FP8ADAM_BF16>) : go(k_pack<FP8ADAM_F16>);
}

int pack8(const fp8adam_matrix* x, const fp8adam_matrix8* o, int64_t rows, int64_t cols, bool back, hipStream_t s) {
  if (!x || !o) return fail(FP8ADAM_EINVAL, "x or the matrix in 8 bits is null");
  if (int r = check_sizes(rows, 1, cols)) return r;
  Memory mem;
  if (int r = check_matrix(mem, *x, rows, cols, back, "x")) return r;
  if (int r = check_matrix8(mem, *o, rows, cols, !back, back ? "in" : "out")) return r;
  if (int r = mem.check()) return r;
  if (int r = stream_device(s)) return r;
  if (rows == 0) return 0;
  if (!back) return run_pack(*x, *o, rows, cols, s);
  const int64_t nb = (cols + 127) >> 7, groups = (rows + 63) / 64 * nb;
  if (int r = check_groups(groups)) return r;
  auto go = [&](auto kernel) {
    return launch(kernel, dim3((unsigned)groups), dim3(kThreads), 0, s, in8(*o), o->format, x->data, x->ld, rows, (int)cols, (int)nb);
  };
  if (x->dtype == FP8ADAM_F32) return go(k_unpack<FP8ADAM_F32>);
  return x->dtype == FP8ADAM_BF16 ? go(k_unpack<FP8ADAM_BF16>) : go(k_unpack<FP8ADAM_F16>);
}

bool valid_act(int32_t a) { return a >= FP8ADAM_ACT_NONE && a <= FP8ADAM_ACT_GELU; }

int product8(const fp8adam_product8* p, bool gated, hipStream_t s) {
  if (!p) return fail(FP8ADAM_EINVAL, "args is null");
  const int64_t T = p->tokens, N = p->rows, K = p->cols;
  if (int r = check_sizes(T, N, K)) return r;
  if (!valid_act(p->activation)) return fail(FP8ADAM_EINVAL, "bad activation");
  if (p->exact != 0 && p->exact != 1) return fail(FP8ADAM_EINVAL, "exact must be 0 or 1");
  Memory mem;
  const bool packs = p->x_in.data != nullptr;
  if (packs)
    if (int r = check_matrix(mem, p->x_in, T, K, false, "x_in")) return r;
  if (int r = check_matrix8(mem, p->x, T, K, packs, "x")) return r;
  if (int r = check_matrix8(mem, p->w, N, K, false, "w")) return r;
  if (gated) {
    if (int r = check_matrix8(mem, p->w_up, N, K, false, "w_up")) return r;
    if (p->w_up.format != p->w.format || p->w_up.scale_type != p->w.scale_type)
      return fail(FP8ADAM_EINVAL, "w and w_up must have one format and one type of scales");
    if (p->bias.data || p->residual.data) return fail(FP8ADAM_EINVAL, "gated8 takes no bias and no residual");
    if (!p->keep.codes != !p->keep_up.codes) return fail(FP8ADAM_EINVAL, "keep and keep_up are given together");
    if (p->keep.codes && p->keep.format != p->keep_up.format) return fail(FP8ADAM_EINVAL, "keep and keep_up must have one format");
  } else if (p->w_up.codes || p->keep_up.codes) {
    return fail(FP8ADAM_EINVAL, "linear8 takes no w_up and no keep_up");
  }
  if (p->bias.data)
    if (int r = check_matrix(mem, p->bias, 1, N, false, "bias")) return r;
  if (p->residual.data)
    if (int r = check_matrix(mem, p->residual, T, N, false, "residual")) return r;
  if (!p->y.data && !p->y8.codes && T > 0) return fail(FP8ADAM_EINVAL, "y and y8 are null");
  if (p->y.data)
    if (int r = check_matrix(mem, p->y, T, N, true, "y")) return r;
  if (p->y8.codes)
    if (int r = check_matrix8(mem, p->y8, T, N, true, "y8")) return r;
  if (p->keep.codes)
    if (int r = check_matrix8(mem, p->keep, T, N, true, "keep")) return r;
  if (p->keep_up.codes)
    if (int r = check_matrix8(mem, p->keep_up, T, N, true, "keep_up")) return r;
  const bool in_place = p->residual.data && p->residual.data == p->y.data && p->residual.dtype == p->y.dtype;
  if (int r = in_place ? mem.check({{"residual", "y"}}) : mem.check()) return r;
  if (int r = stream_device(s)) return r;
  if (T == 0) return 0;

  ProductArgs a{};
  a.x = in8(p->x);
  a.w[0] = in8(p->w);
  if (gated) a.w[1] = in8(p->w_up);
  a.tokens = T;
  a.rows = (int32_t)N;
  a.cols = (int32_t)K;
  a.bias = p->bias.data;
  a.bias_dt = p->bias.dtype;
  a.res = p->residual.data;
  a.res_dt = p->residual.dtype;
  a.res_ld = p->residual.ld;
  a.y = p->y.data;
  a.y_dt = p->y.dtype;
  a.y_ld = p->y.ld;
  if (p->y8.codes) a.y8 = out8(p->y8);
  if (p->keep.codes) a.keep[0] = out8(p->keep);
  if (p->keep_up.codes) a.keep[1] = out8(p->keep_up);
  a.act = p->activation;
  a.exact = p->exact;
  if (packs) {
    if (packs_itself(a, p->x_in)) {
      a.xin = p->x_in.data;
      a.xin_dt = p->x_in.dtype;
      a.xin_ld = p->x_in.ld;
      a.x8 = out8(p->x);
    } else if (int r = run_pack(p->x_in, p->x, T, K, s)) {
      return r;
    }
  }
  const int xf = p->x.format, wf = p->w.format;
  if (xf == 0) return wf == 0 ? launch_product<0, 0>(a, gated, s) : launch_product<0, 1>(a, gated, s);
  return wf == 0 ? launch_product<1, 0>(a, gated, s) : launch_product<1, 1>(a, gated, s);
}

// ---- back through the activations

int64_t act_chunks(int64_t tokens) { return (tokens + kActRows - 1) / kActRows; }

int64_t act_workspace(const fp8adam_act_backward8* p) {
  if (!p) return fail(FP8ADAM_EINVAL, "args is null");
  if (int r = check_sizes(p->tokens, p->rows, 1)) return r;
  return p->bias_grad.data ? act_chunks(p->tokens) * ((p->rows + 127) >> 7) * 128 * (int64_t)sizeof(float) : 0;
}

template <bool GATED, int DT>
int launch_act(int act, dim3 grid, hipStream_t s, const ActArgs& a) {
  auto go = [&](auto kernel) { return launch(kernel, grid, dim3(kThreads), 0, s, a); };
  if (act == FP8ADAM_ACT_NONE) return go(k_act_backward<GATED, FP8ADAM_ACT_NONE, DT>);
  if (act == FP8ADAM_ACT_RELU) return go(k_act_backward<GATED, FP8ADAM_ACT_RELU, DT>);
  if (act == FP8ADAM_ACT_SILU) return go(k_act_backward<GATED, FP8ADAM_ACT_SILU, DT>);
  return go(k_act_backward<GATED, FP8ADAM_ACT_GELU, DT>);
}

int act_backward(const fp8adam_act_backward8* p, bool gated, hipStream_t s) {
  const int64_t need = act_workspace(p);
  if (need < 0) return (int)need;
  const int64_t T = p->tokens, N = p->rows;
  if (!valid_act(p->activation)) return fail(FP8ADAM_EINVAL, "bad activation");
  Memory mem;
  if (int r = check_matrix(mem, p->dy, T, N, false, "dy")) return r;
  const bool none = !gated && p->activation == FP8ADAM_ACT_NONE;
  if (none) {
    if (p->keep.codes || p->dz.data) return fail(FP8ADAM_EINVAL, "without an activation dz is dy: keep and dz must be null");
    if (!p->bias_grad.data) return fail(FP8ADAM_EINVAL, "without an activation and bias_grad there is nothing to do");
  } else {
    if (int r = check_matrix8(mem, p->keep, T, N, false, "keep")) return r;
    if (int r = check_matrix(mem, p->dz, T, N, true, "dz")) return r;
  }
  if (gated) {
    if (int r = check_matrix8(mem, p->keep_up, T, N, false, "keep_up")) return r;
    if (int r = check_matrix(mem, p->dup, T, N, true, "dup")) return r;
    if (p->bias_grad.data) return fail(FP8ADAM_EINVAL, "gated8_backward takes no bias_grad");
  } else if (p->keep_up.codes || p->dup.data) {
    return fail(FP8ADAM_EINVAL, "linear8_backward takes no keep_up and no dup");
  }
  if ((!none && p->dz.dtype != p->dy.dtype) || (gated && p->dup.dtype != p->dy.dtype))
    return fail(FP8ADAM_EINVAL, "dz and dup must have dy's dtype");
  if (p->bias_grad.data) {
    if (int r = check_matrix(mem, p->bias_grad, 1, N, true, "bias_grad")) return r;
    if (need > 0 && !p->workspace) return fail(FP8ADAM_EINVAL, "workspace is null");
    if (p->workspace_bytes < need) return fail(FP8ADAM_EINVAL, "workspace has fewer than " + std::to_string(need) + " bytes");
    if ((uintptr_t)p->workspace & 15u) return fail(FP8ADAM_EALIGN, "workspace is not 16-byte aligned");
    mem.add(p->workspace, need, need, 1, true, "workspace");
  }
  if (int r = mem.check({{"dy", "dz"}, {"dy", "dup"}})) return r;
  const int64_t nb = (N + 127) >> 7, chunks = act_chunks(T), groups = chunks * nb;
  if (int r = check_groups(groups)) return r;
  if (int r = stream_device(s)) return r;
  if (T > 0) {
    ActArgs a{};
    a.dy = p->dy.data, a.ld_dy = p->dy.ld;
    a.dz = p->dz.data, a.ld_dz = p->dz.ld;
    a.dup = p->dup.data, a.ld_dup = p->dup.ld;
    if (!none) a.z[0] = in8(p->keep), a.format[0] = p->keep.format;
    if (gated) a.z[1] = in8(p->keep_up), a.format[1] = p->keep_up.format;
    a.tokens = T, a.rows = (int32_t)N, a.nb = (int32_t)nb;
    a.partial = p->bias_grad.data ? static_cast<float*>(p->workspace) : nullptr;
    const dim3 grid((unsigned)groups);
    auto go = [&](auto g) {
      constexpr bool G = decltype(g)::value;
      if (p->dy.dtype == FP8ADAM_F32) return launch_act<G, FP8ADAM_F32>(p->activation, grid, s, a);
      if (p->dy.dtype == FP8ADAM_BF16) return launch_act<G, FP8ADAM_BF16>(p->activation, grid, s, a);
      return launch_act<G, FP8ADAM_F16>(p->activation, grid, s, a);
    };
    if (int r = gated ? go(std::true_type{}) : go(std::false_type{})) return r;
  }
  if (!p->bias_grad.data) return 0;
  return launch(k_bias_join, dim3((unsigned)((N + 31) / 32)), dim3(kThreads), 0, s, static_cast<const float*>(p->workspace), chunks,
                nb * 128, (int)N, p->bias_grad.data, p->bias_grad.dtype, p->accumulate);
}

// ---- gradients of weights and inputs

// dy goes into the product as it is where it is bf16 with rows of whole 16-byte pieces; otherwise through
// k_split, in one part (bf16), two (fp16, and fp32 in 16 bits) or three (fp32 in all of its bits).
struct Left {
  bool direct;
  int parts;
  int64_t ld, bytes;  // of one part
};

Left left_of(const fp8adam_matrix& dy, int64_t tokens, int64_t rows, bool exact) {
  Left l{};
  const int64_t ld = tokens > 1 ? dy.ld : rows;  // one row's is not used
  l.direct = dy.dtype == FP8ADAM_BF16 && rows % 8 == 0 && ld % 8 == 0 && ((uintptr_t)dy.data & 15u) == 0;
  l.parts = dy.dtype == FP8ADAM_BF16 ? 1 : dy.dtype == FP8ADAM_F32 && exact ? kMaxParts : 2;
  l.ld = l.direct ? ld : (rows + 7) & ~(int64_t)7;
  l.bytes = l.direct ? 0 : (tokens * l.ld * 2 + 255) & ~(int64_t)255;
  return l;
}

struct GradCall {
  GradPlan plan;
  Left left[2];
  bool direct;  // every dy as it is, all with one ld
  int64_t bytes;
};

int grad_call(const fp8adam_grad8* p, bool weights, GradCall& c) {
  if (!p) return fail(FP8ADAM_EINVAL, "args is null");
  if (int r = check_sizes(p->tokens, p->rows, p->cols)) return r;
  if (p->exact != 0 && p->exact != 1) return fail(FP8ADAM_EINVAL, "exact must be 0 or 1");
  if (p->n < 1 || p->n > (weights ? 1 : 2)) return fail(FP8ADAM_EINVAL, weights ? "n must be 1" : "n must be 1 or 2");
  for (int i = 0; i < p->n; i++)
    if (p->dy[i].dtype < FP8ADAM_F32 || p->dy[i].dtype > FP8ADAM_F16 || p->dy[i].dtype != p->dy[0].dtype)
      return fail(FP8ADAM_EINVAL, "bad dtype of dy, or more than one");
  c.direct = true;
  for (int i = 0; i < p->n; i++) {
    c.left[i] = left_of(p->dy[i], p->tokens, p->rows, p->exact);
    c.direct = c.direct && c.left[i].direct && c.left[i].ld == c.left[0].ld;
  }
  c.bytes = 0;
  if (!c.direct)
    for (int i = 0; i < p->n; i++) {
      fp8adam_matrix other = p->dy[i];
      other.data = reinterpret_cast<void*>(2);  // not 16-byte aligned: through k_split
      c.left[i] = left_of(other, p->tokens, p->rows, p->exact);
      c.bytes += c.left[i].parts * c.left[i].bytes;
    }
  const int pairs = p->n * c.left[0].parts;
  c.plan = weights ? plan_grad(p->rows, p->cols, p->tokens, pairs) : plan_grad(p->tokens, p->cols, p->rows, pairs);
  c.bytes += c.plan.partial_bytes;
  return 0;
}

int64_t grad_workspace(const fp8adam_grad8* p, bool weights) {
  GradCall c;
  if (int r = grad_call(p, weights, c)) return r;
  return p->tokens > 0 ? c.bytes : 0;
}

int run_split(const fp8adam_matrix& dy, int64_t tokens, int64_t rows, const Left& l, uint16_t* out, hipStream_t s) {
  const int64_t groups = (tokens * (l.ld >> 3) + kThreads - 1) / kThreads;
  if (int r = check_groups(groups)) return r;
  auto go = [&](auto kernel) {
    return launch(kernel, dim3((unsigned)groups), dim3(kThreads), 0, s, dy.data, dy.ld, tokens, (int)rows, l.ld, out, l.bytes / 2);
  };
  if (dy.dtype == FP8ADAM_F32) return l.parts == 3 ? go(k_split<FP8ADAM_F32, 3>) : go(k_split<FP8ADAM_F32, 2>);
  return dy.dtype == FP8ADAM_BF16 ? go(k_split<FP8ADAM_BF16, 1>) : go(k_split<FP8ADAM_F16, 2>);
}

int grad8(const fp8adam_grad8* p, bool weights, hipStream_t s) {
  GradCall c;
  if (int r = grad_call(p, weights, c)) return r;
  const int64_t T = p->tokens, N = p->rows, K = p->cols;
  Memory mem;
  for (int i = 0; i < p->n; i++) {
    if (int r = check_matrix(mem, p->dy[i], T, N, false, "dy")) return r;
    if (int r = check_matrix8(mem, p->b[i], weights ? T : N, K, false, weights ? "x" : "w")) return r;
    if (p->b[i].format != p->b[0].format || p->b[i].scale_type != p->b[0].scale_type)
      return fail(FP8ADAM_EINVAL, "the layers' weights must have one format and one type of scales");
  }
  if (int r = check_matrix(mem, p->out, weights ? N : T, K, true, "out")) return r;
  const int64_t need = T > 0 ? c.bytes : 0;
  if (need > 0) {
    if (!p->workspace) return fail(FP8ADAM_EINVAL, "workspace is null");
    if (p->workspace_bytes < need) return fail(FP8ADAM_EINVAL, "workspace has fewer than " + std::to_string(need) + " bytes");
    if ((uintptr_t)p->workspace & 15u) return fail(FP8ADAM_EALIGN, "workspace is not 16-byte aligned");
    mem.add(p->workspace, need, need, 1, true, "workspace");
  }
  if (int r = mem.check()) return r;
  if (int r = stream_device(s)) return r;
  if (T == 0 && (!weights || p->accumulate)) return 0;

  GradArgs a{};
  unsigned char* ws = static_cast<unsigned char*>(p->workspace);
  for (int i = 0; i < p->n; i++) {
    const Left& l = c.left[i];
    for (int q = 0; q < l.parts; q++) {
      a.a[a.npairs] = static_cast<const uint16_t*>(c.direct ? p->dy[i].data : ws + q * l.bytes);
      a.b[a.npairs++] = in8(p->b[i]);
    }
    if (!c.direct && T > 0) {
      if (int r = run_split(p->dy[i], T, N, l, reinterpret_cast<uint16_t*>(ws), s)) return r;
      ws += l.parts * l.bytes;
    }
  }
  a.lda = c.left[0].ld;
  a.trans = weights;
  a.m = weights ? N : T;
  a.r = weights ? T : N;
  a.k = (int32_t)K;
  a.out = p->out.data;
  a.out_dt = p->out.dtype;
  a.ld_out = p->out.ld;
  a.accumulate = p->accumulate != 0;
  a.partial = c.plan.splits > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  return p->b[0].format == FP8ADAM_E4M3 ? launch_grad<0>(a, c.plan, s) : launch_grad<1>(a, c.plan, s);
}

// Nothing is thrown across the ABI: every entry point runs its body in here.
template <typename F>
auto guarded(const char* what, F&& body) -> decltype(body()) {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return fail(FP8ADAM_ENOMEM, "host allocation failed");
  } catch (...) {
    return fail(FP8ADAM_EINVAL, std::string("unexpected error in ") + what);
  }
}

}  // namespace

// The tiles and the number of parts of the sum whose estimated time is least, in us: 64 of the sum
// take a work-group of 256 x 256 (one on a CU) 2, one of 128 x 128 1, or 1.35 where there are two on
// a CU; the parts are written and read again at about 5 TB/s, by one launch more.  (The estimates are
// within a sixth of what was measured, and their order right: 2048 x 2048 x 2048 as 128 x 128 in one
// part 45 estimated 38, as 256 x 256 in four parts 51 estimated 53; 2048 tokens x 2 pairs of 2048 x 768
// as 128 x 128 in five parts 35 estimated 40, as 256 x 256 in eight 40 estimated 46; 16384 tokens
// x 2048 x 768 as 256 x 256 in ten parts 80 estimated 87, as 128 x 128 in five 88 estimated 93.)  From 16 on the numbers
// of parts that are looked at grow by an eighth: all 768 of a single tile would take the host longer than the kernel's launch.
GradPlan plan_grad(int64_t m, int64_t k, int64_t r, int npairs) {
  const int64_t steps = (r + 63) / 64 * npairs, ldp = (k + 3) & ~(int64_t)3;
  GradPlan best{0, 1, 0};
  double least = 0.0;
  for (int tile = 0; tile < 2; tile++) {
    const int64_t size = tile ? 128 : 256, slots = tile ? 512 : 256;
    const int64_t tiles = std::max<int64_t>(1, (m + size - 1) / size * ((k + size - 1) / size));
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(slots / tiles, steps / 2));
    for (int64_t splits = 1;; splits = std::min(most, splits + std::max<int64_t>(1, splits / 8))) {
      const int64_t groups = tiles * splits;
      const double step = tile ? (groups > 256 ? 1.35 : 1.0) : 2.0;
      double t = (double)((groups + slots - 1) / slots) * (double)((steps + splits - 1) / splits) * step;
      if (splits > 1) t += 4.0 + 8.0 * (double)(splits * m * ldp) / 5e6;
      if (tile + splits == 1 || t < least) {
        least = t;
        best = GradPlan{tile, (int)splits, splits > 1 ? splits * m * ldp * (int64_t)sizeof(float) : 0};
      }
      if (splits == most) break;
    }
  }
  return best;
}

}  // namespace fp8adam_layer

// ================================================================== C ABI

extern "C" {

int fp8adam_pack8(const fp8adam_matrix* x, const fp8adam_matrix8* out, int64_t rows, int64_t cols, hipStream_t stream) {
  return guarded("fp8adam_pack8", [&] { return pack8(x, out, rows, cols, false, stream); });
}

int fp8adam_unpack8(const fp8adam_matrix8* in, const fp8adam_matrix* x, int64_t rows, int64_t cols, hipStream_t stream) {
  return guarded("fp8adam_unpack8", [&] { return pack8(x, in, rows, cols, true, stream); });
}

int fp8adam_linear8(const fp8adam_product8* args, hipStream_t stream) {
  return guarded("fp8adam_linear8", [&] { return product8(args, false, stream); });
}

int fp8adam_gated8(const fp8adam_product8* args, hipStream_t stream) {
  return guarded("fp8adam_gated8", [&] { return product8(args, true, stream); });
}

int64_t fp8adam_linear8_backward_workspace(const fp8adam_act_backward8* args) {
  return guarded("fp8adam_linear8_backward_workspace", [&] { return act_workspace(args); });
}

int fp8adam_linear8_backward(const fp8adam_act_backward8* args, hipStream_t stream) {
  return guarded("fp8adam_linear8_backward", [&] { return act_backward(args, false, stream); });
}

int fp8adam_gated8_backward(const fp8adam_act_backward8* args, hipStream_t stream) {
  return guarded("fp8adam_gated8_backward", [&] { return act_backward(args, true, stream); });
}

int64_t fp8adam_weight_grad8_workspace(const fp8adam_grad8* args) {
  return guarded("fp8adam_weight_grad8_workspace", [&] { return grad_workspace(args, true); });
}

int64_t fp8adam_input_grad8_workspace(const fp8adam_grad8* args) {
  return guarded("fp8adam_input_grad8_workspace", [&] { return grad_workspace(args, false); });
}

int fp8adam_weight_grad8(const fp8adam_grad8* args, hipStream_t stream) {
  return guarded("fp8adam_weight_grad8", [&] { return grad8(args, true, stream); });
}

int fp8adam_input_grad8(const fp8adam_grad8* args, hipStream_t stream) {
  return guarded("fp8adam_input_grad8", [&] { return grad8(args, false, stream); });
}

}  // extern "C"
