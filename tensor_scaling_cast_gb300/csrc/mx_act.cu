// Decoding MX matrices, and the activation of an MLP whose inputs are kept as
// 8-bit MX blocks for the backward pass.
//
//   forward   h = f(z) * u (or f(z)), from the plain z and u; MX(z), MX(u) are
//             written for the backward pass, h plain or as MX blocks or both
//   backward  dz = dh * u * f'(z), du = dh * f(z) and, where asked for, h
//             again, with z and u as the 8-bit blocks hold them
//
//   SILU       f = z s, f' = s (1 + z (1 - s)), s = 1 / (1 + e^-z)
//   GELU       f = z P, f' = P + z e^(-z z / 2) / sqrt(2 pi), P = (1 + erf(z / sqrt 2)) / 2
//   GELU_TANH  f = z s, f' = s + z s (1 - s) y', s = 1 / (1 + e^-y),
//              y = 2 sqrt(2 / pi) (z + 0.044715 z^3): (1 + tanh(y / 2)) / 2 is s
//
// All three are streaming passes bound by HBM.  A unit is eight elements of a
// row; four neighbouring lanes hold one block.  16384 x 8192 bf16: decoding 4
// bits 51.0 us (6.66 TB/s); forward, gated, with both inputs kept, 170 us (SILU,
// 6.3 TB/s), 178 (GELU_TANH), 206 (GELU); backward 158, 182, 200.  GELU's are
// bound by issue slots, 76% of which forward SILU already uses; two units a
// thread in flight (with four the registers cost more than the loads gain: 1.25
// times as long).
#include <cuda_runtime.h>

#include "mx_linear.cuh"

namespace fp8q {

// ---- decode ---------------------------------------------------------------------

constexpr int kDecodeAhead = 4;

template <int FMT, int DT>
__global__ void __launch_bounds__(kUnitThreads) mx_decode_kernel(const __grid_constant__ MxView m, void* out,
                                                                 int64_t out_stride, const __grid_constant__ Units u) {
  constexpr int U = kDecodeAhead;
  grid_begin();
  const int64_t i0 = (int64_t)blockIdx.x * (U * kUnitThreads) + threadIdx.x;
  uint2 v[U];
  uint32_t e[U];
  int64_t row[U], col[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t i = i0 + j * kUnitThreads;
    if (i >= u.count) continue;
    u.place(i, &row[j], &col[j]);
    const uint8_t* src = m.q + row[j] * m.q_stride + (FMT == FP8Q_E2M1 ? col[j] / 2 : col[j]);
    if (FMT == FP8Q_E2M1) v[j].x = __ldcs(reinterpret_cast<const uint32_t*>(src));
    else v[j] = __ldcs(reinterpret_cast<const uint2*>(src));
    e[j] = m.e8m0[row[j] * m.e_stride + (col[j] >> 5)];
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (i0 + j * kUnitThreads >= u.count) continue;
    float f[8];
    decode8<FMT>(v[j], e8m0_value(e[j]), f);
    store8<DT>(out, row[j] * out_stride + col[j], f);
  }
}

template <int DT>
static const void* decode_kernel(int format) {
  return format == FP8Q_E2M1   ? reinterpret_cast<const void*>(mx_decode_kernel<FP8Q_E2M1, DT>)
         : format == FP8Q_E4M3 ? reinterpret_cast<const void*>(mx_decode_kernel<FP8Q_E4M3, DT>)
                               : reinterpret_cast<const void*>(mx_decode_kernel<FP8Q_E5M2, DT>);
}

cudaError_t launch_mx_decode(const MxView& m, void* out, int dtype, int64_t out_stride, cudaStream_t s, int* launches) {
  Units u(m.rows, m.cols);
  const int64_t grid = unit_grid(u, kDecodeAhead);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  MxView view = m;
  void* args[] = {&view, &out, &out_stride, &u};
  return launch_dependent(dtype == FP8Q_BF16 ? decode_kernel<FP8Q_BF16>(m.format) : decode_kernel<FP8Q_F32>(m.format),
                          dim3((unsigned)grid), kUnitThreads, 0, args, s, launches);
}

// ---- activations ------------------------------------------------------------------

// f(z) and f'(z).  Where the tensors are bf16 (FAST) exponentials and
// reciprocals are the approximate instructions, good to 2^-22 and 2^-23 of the
// value (below 2^-126 it is 0); in 32 bits the C functions.
//
// Errors, in units of 2^-24, w the magnitude of the exponential's argument: the
// exponential has 4 of its own and, for each rounding on the way to its argument,
// w more: 1.3 for the base's constant and the product with it, then none for
// SILU, 1 for z z / 2, 6 for y.  s = 1 / (1 + E) has E's times 1 - s, and 3; f one
// more: (4 + 7.3 w) (1 - s) + 4 of f at most.  GELU's tail has e's, 8 of the
// polynomial, 8 for t and 3 for the products: 23 + 2.3 w.  t = f (1 - s) has f's,
// s's times s and 2 of t, and 3 |z| s s of its own where 1 - s cancels; times y'
// (6 more, and |z| y' <= 3 w) and added to s: at most 20 + 16.3 w of s + |t y'|.
// With u, dh and the gate come up to 2 products: 24 + 8 w and 24 + 17 w.  With
// both instructions rounding to nearest every bf16 z gives less than 24 + 1.6 w.
template <bool FAST>
__device__ __forceinline__ float exp_of(float x) {
  if (!FAST) return expf(x);
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
template <bool FAST>
__device__ __forceinline__ float reciprocal(float x) {
  if (!FAST) return 1.0f / x;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <bool FAST>
__device__ __forceinline__ float sigmoid(float x) {
  return reciprocal<FAST>(1.0f + exp_of<FAST>(-x));
}

// (1 + erf(z / sqrt 2)) / 2 and e = e^(-z z / 2).  Approximate: with x =
// |z| / sqrt 2 and t = 1 / (1 + 0.425 x), erfc(x) = e t P(t), P the polynomial of
// degree 7 that is nearest in relative error for x up to 10 (a least-squares fit
// at Chebyshev points, weights moved towards the largest error: 1.5e-7, and
// 4.5e-7 as evaluated here); further out e is below 2^-126.
template <bool FAST>
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  e = exp_of<FAST>(-0.5f * z * z);
  if (!FAST) return 0.5f * erfcf(-0.70710678118654752f * z);
  const float t = reciprocal<FAST>(fmaf(0.425f * 0.70710678118654752f, fabsf(z), 1.0f));
  float p = 0.07147661596536636f;
  p = fmaf(p, t, -0.3131510317325592f);
  p = fmaf(p, t, 0.40760907530784607f);
  p = fmaf(p, t, -0.1032443568110466f);
  p = fmaf(p, t, 0.2550836503505707f);
  p = fmaf(p, t, 0.20070675015449524f);
  p = fmaf(p, t, 0.24184052646160126f);
  p = fmaf(p, t, 0.23967863619327545f);
  const float half = 0.5f * t * p * e;
  return z < 0.0f ? half : 1.0f - half;
}

template <int ACT, bool FAST, bool WITH_D>
__device__ __forceinline__ void activation(float z, float& f, float& d) {
  if (ACT == MX_ACT_GELU) {
    float e;
    const float p = normal_cdf<FAST>(z, e);
    f = z * p;
    if (WITH_D) d = fmaf(z * 0.39894228040143268f, e, p);
  } else {
    constexpr float C = 1.5957691216057308f;             // 2 sqrt(2 / pi)
    const float z2 = z * z;
    const float y = ACT == MX_ACT_SILU ? z : C * z * fmaf(0.044715f, z2, 1.0f);
    const float s = sigmoid<FAST>(y);
    f = z * s;
    if (WITH_D) {
      const float t = f * (1.0f - s);
      // far out s is 0 or 1 and so is f', while y' may have overflowed
      d = ACT == MX_ACT_SILU ? t + s
                             : t == 0.0f ? s : fmaf(t, C * fmaf(3.0f * 0.044715f, z2, 1.0f), s);
    }
  }
}

// Eight elements as a block's codes; every lane of the warp calls it.
template <int FMT>
__device__ __forceinline__ void write_block(const MxView& m, int64_t row, int64_t col, bool on, const float (&f)[8],
                                            uint32_t amax, int rule) {
  amax = block_max4(amax);
  uint2 o;
  uint32_t ebyte;
  if (amax >= 0x7F800000u) {
    uint32_t signs = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) signs |= (__float_as_uint(f[k]) >> 31) << k;
    o = nonfinite8<FMT>(signs);
    ebyte = 255u;
  } else {
    const int E = block_exp<FMT>(amax, rule, 0);
    const float s = block_inv_scale<FMT>(E);
    float g[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = f[k] * s;
    o = encode8<FMT>(g);
    ebyte = (uint32_t)(E + 127);
  }
  if (!on) return;
  uint8_t* dst = m.q + row * m.q_stride + (FMT == FP8Q_E2M1 ? col / 2 : col);
  if (FMT == FP8Q_E2M1) __stcs(reinterpret_cast<uint32_t*>(dst), o.x);
  else __stcs(reinterpret_cast<uint2*>(dst), o);
  if ((threadIdx.x & 3) == 0) m.e8m0[row * m.e_stride + (col >> 5)] = (uint8_t)ebyte;
}
// The same in the format that the matrix has, decided per call.
__device__ __forceinline__ void write_block_any(const MxView& m, int64_t row, int64_t col, bool on, const float (&f)[8],
                                                uint32_t amax, int rule) {
  if (m.format == FP8Q_E4M3) write_block<FP8Q_E4M3>(m, row, col, on, f, amax, rule);
  else if (m.format == FP8Q_E5M2) write_block<FP8Q_E5M2>(m, row, col, on, f, amax, rule);
  else write_block<FP8Q_E2M1>(m, row, col, on, f, amax, rule);
}
__device__ __forceinline__ uint32_t absmax_of(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(f[k]) & 0x7FFFFFFFu);
  return m;
}

constexpr int kActAhead = 2;

template <int ACT, int DT, bool GATED, int FMT>
__global__ void __launch_bounds__(kUnitThreads) mx_act_forward_kernel(const __grid_constant__ MxActForward a,
                                                                      const __grid_constant__ Units u) {
  constexpr int U = kActAhead;
  constexpr bool FAST = DT == FP8Q_BF16;
  grid_begin();
  const int64_t i0 = (int64_t)blockIdx.x * (U * kUnitThreads) + threadIdx.x;
  Plain8<DT> z[U], g[GATED ? U : 1];
  int64_t row[U], col[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t i = i0 + j * kUnitThreads;
    z[j] = zero8<DT>();
    if (GATED) g[j] = zero8<DT>();
    row[j] = col[j] = 0;
    if (i >= u.count) continue;
    u.place(i, &row[j], &col[j]);
    z[j] = load8<DT>(a.z, row[j] * a.z_stride + col[j]);
    if (GATED) g[j] = load8<DT>(a.u, row[j] * a.u_stride + col[j]);
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const bool on = i0 + j * kUnitThreads < u.count;
    float x[8], y[8], h[8], unused;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[k] = __uint_as_float(bits8<DT>(z[j], k));
      if (GATED) y[k] = __uint_as_float(bits8<DT>(g[j], k));
    }
    if (a.z_saved.q) {
      write_block<FMT>(a.z_saved, row[j], col[j], on, x, absmax8<DT>(z[j]), a.rule);
      if (GATED) write_block<FMT>(a.u_saved, row[j], col[j], on, y, absmax8<DT>(g[j]), a.rule);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      activation<ACT, FAST, false>(x[k], h[k], unused);
      if (GATED) h[k] *= y[k];
    }
    if (a.h && on) store8<DT>(a.h, row[j] * a.h_stride + col[j], h);
    if (a.h_mx.q) write_block_any(a.h_mx, row[j], col[j], on, h, absmax_of(h), a.rule);
  }
}

template <int ACT, int DT, bool GATED, int FMT>
__global__ void __launch_bounds__(kUnitThreads) mx_act_backward_kernel(const __grid_constant__ MxActBackward a,
                                                                       const __grid_constant__ Units u) {
  constexpr int U = kActAhead;
  constexpr bool FAST = DT == FP8Q_BF16;
  grid_begin();
  const int64_t i0 = (int64_t)blockIdx.x * (U * kUnitThreads) + threadIdx.x;
  Plain8<DT> dh[U];
  uint2 zq[U], uq[GATED ? U : 1];
  uint32_t ze[U], ue[GATED ? U : 1];
  int64_t row[U], col[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t i = i0 + j * kUnitThreads;
    if (i >= u.count) continue;
    u.place(i, &row[j], &col[j]);
    dh[j] = load8<DT>(a.dh, row[j] * a.dh_stride + col[j]);
    zq[j] = __ldcs(reinterpret_cast<const uint2*>(a.z.q + row[j] * a.z.q_stride + col[j]));
    ze[j] = a.z.e8m0[row[j] * a.z.e_stride + (col[j] >> 5)];
    if (GATED) {
      uq[j] = __ldcs(reinterpret_cast<const uint2*>(a.u.q + row[j] * a.u.q_stride + col[j]));
      ue[j] = a.u.e8m0[row[j] * a.u.e_stride + (col[j] >> 5)];
    }
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (i0 + j * kUnitThreads >= u.count) continue;
    float x[8], y[8], dz[8], du[8], h[8];
    decode8<FMT>(zq[j], e8m0_value(ze[j]), x);
    if (GATED) decode8<FMT>(uq[j], e8m0_value(ue[j]), y);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float g = __uint_as_float(bits8<DT>(dh[j], k));
      float f, d;
      activation<ACT, FAST, true>(x[k], f, d);
      dz[k] = GATED ? g * y[k] * d : g * d;
      if (GATED) du[k] = g * f;
      h[k] = GATED ? f * y[k] : f;
    }
    store8<DT>(a.dz, row[j] * a.dz_stride + col[j], dz);
    if (GATED) store8<DT>(a.du, row[j] * a.du_stride + col[j], du);
    if (a.h) store8<DT>(a.h, row[j] * a.h_stride + col[j], h);
  }
}

template <int ACT, int DT, bool GATED>
static const void* forward_of(int format) {
  return format == FP8Q_E5M2 ? reinterpret_cast<const void*>(mx_act_forward_kernel<ACT, DT, GATED, FP8Q_E5M2>)
                             : reinterpret_cast<const void*>(mx_act_forward_kernel<ACT, DT, GATED, FP8Q_E4M3>);
}
template <int ACT>
static const void* forward_kernel(int dtype, bool gated, int format) {
  if (dtype == FP8Q_BF16)
    return gated ? forward_of<ACT, FP8Q_BF16, true>(format) : forward_of<ACT, FP8Q_BF16, false>(format);
  return gated ? forward_of<ACT, FP8Q_F32, true>(format) : forward_of<ACT, FP8Q_F32, false>(format);
}
template <int ACT, int DT, bool GATED>
static const void* backward_of(int format) {
  return format == FP8Q_E4M3 ? reinterpret_cast<const void*>(mx_act_backward_kernel<ACT, DT, GATED, FP8Q_E4M3>)
                             : reinterpret_cast<const void*>(mx_act_backward_kernel<ACT, DT, GATED, FP8Q_E5M2>);
}
template <int ACT>
static const void* backward_kernel(int dtype, bool gated, int format) {
  if (dtype == FP8Q_BF16)
    return gated ? backward_of<ACT, FP8Q_BF16, true>(format) : backward_of<ACT, FP8Q_BF16, false>(format);
  return gated ? backward_of<ACT, FP8Q_F32, true>(format) : backward_of<ACT, FP8Q_F32, false>(format);
}

cudaError_t launch_mx_act_forward(const MxActForward& a, int act, int dtype, int64_t rows, int64_t cols, cudaStream_t s,
                                  int* launches) {
  Units u(rows, cols);
  const int64_t grid = unit_grid(u, kActAhead);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  MxActForward args_a = a;
  void* args[] = {&args_a, &u};
  const bool gated = a.u != nullptr;
  const void* k = act == MX_ACT_SILU   ? forward_kernel<MX_ACT_SILU>(dtype, gated, a.z_saved.format)
                  : act == MX_ACT_GELU ? forward_kernel<MX_ACT_GELU>(dtype, gated, a.z_saved.format)
                                       : forward_kernel<MX_ACT_GELU_TANH>(dtype, gated, a.z_saved.format);
  return launch_dependent(k, dim3((unsigned)grid), kUnitThreads, 0, args, s, launches);
}

cudaError_t launch_mx_act_backward(const MxActBackward& a, int act, int dtype, cudaStream_t s, int* launches) {
  Units u(a.z.rows, a.z.cols);
  const int64_t grid = unit_grid(u, kActAhead);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  MxActBackward args_a = a;
  void* args[] = {&args_a, &u};
  const bool gated = a.u.q != nullptr;
  const void* k = act == MX_ACT_SILU   ? backward_kernel<MX_ACT_SILU>(dtype, gated, a.z.format)
                  : act == MX_ACT_GELU ? backward_kernel<MX_ACT_GELU>(dtype, gated, a.z.format)
                                       : backward_kernel<MX_ACT_GELU_TANH>(dtype, gated, a.z.format);
  return launch_dependent(k, dim3((unsigned)grid), kUnitThreads, 0, args, s, launches);
}

}  // namespace fp8q
