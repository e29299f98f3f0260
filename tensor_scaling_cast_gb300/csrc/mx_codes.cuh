// Codes of MX blocks in 4 and 8 bits, as every kernel that writes or reads them
// converts them, and the launch helpers those kernels share.
#pragma once

#include <stdint.h>

#include "fp8q_device.cuh"
#include "mx_device.cuh"

namespace fp8q {

// Exact division of n < 2^31 by a fixed d >= 1: q = (hi(n * mul) + n) >> shift
// (round-up reciprocal of the invariant divisor).
struct FastDiv {
  uint32_t mul, shift, d;
  FastDiv() = default;
  explicit FastDiv(uint32_t v) : d(v) {
    shift = 0;
    while ((1ull << shift) < v) ++shift;
    mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - v)) / v + 1);
  }
  __device__ __forceinline__ int div(int n) const { return (int)div((uint32_t)n); }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

// Programmatic dependent launch: every CTA waits until the grid before it in
// the stream has completed, before any access to memory, and then lets the
// next one be set up, so that back-to-back calls (a step's write, then its
// attention) do not pay for launches one after the other.
__device__ __forceinline__ void grid_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
inline cudaError_t launch_dependent(const void* kernel, dim3 grid, int threads, int smem, void** args, cudaStream_t st,
                                    int* launches) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kernel, args);
  if (e == cudaSuccess) ++*launches;
  return e;
}

// 2^(byte - 127) of an E8M0 byte as fp32; 0xFF is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FFFFFFFu : b == 0u ? 0x00400000u : b << 23);
}

// Eight fp32 values -> eight E2M1 codes in a word (element i in bits 4i..),
// round to nearest even, saturating to +-6.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The eight codes of a word -> four f16 pairs (exact).
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Four 8-bit codes of a word -> two f16 pairs (exact for both formats).
template <int FMT>
__device__ __forceinline__ void fp8x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (FMT == FP8Q_E4M3)
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}" : "=r"(lo), "=r"(hi) : "r"(w));
  else
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
        " cvt.rn.f16x2.e5m2x2 %0, a;\n cvt.rn.f16x2.e5m2x2 %1, b;\n}" : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ float2 f16x2_f32(uint32_t h) {
  float2 f;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
      : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// Two fp32 -> a bf16 pair, round to nearest even (`lo` in the low half).
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace fp8q
