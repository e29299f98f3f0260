// Matrices in MX blocks as the kernels of linear layers see them: the 4-bit
// casts (mx4.cu), decoding and the activations kept in 8 bits (mx_act.cu) and
// products (mx_matmul.cuh).
#pragma once

#include <stdint.h>

#include "fp8q_device.cuh"
#include "mx_codes.cuh"

namespace fp8q {

// A checked mx_matrix: rows of `cols` codes q_stride bytes apart and of
// cols / 32 E8M0 bytes e_stride bytes apart.
struct MxView {
  uint8_t* q;
  uint8_t* e8m0;
  int64_t rows, cols, q_stride, e_stride;
  int32_t format;
  int64_t row_bytes() const { return format == FP8Q_E2M1 ? cols / 2 : cols; }
};

// Eight values in a word (E2M1) or two (8 bits, .x first).
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float (&f)[8]) {
  uint2 o;
  if constexpr (FMT == FP8Q_E2M1) {
    o.x = cvt_e2m1x8(f);
    o.y = 0;
  } else {
    o.x = cvt_pair<FMT>(f[0], f[1]) | (cvt_pair<FMT>(f[2], f[3]) << 16);
    o.y = cvt_pair<FMT>(f[4], f[5]) | (cvt_pair<FMT>(f[6], f[7]) << 16);
  }
  return o;
}
// sign|largest for eight elements of a block that is not finite; bit k of
// `signs` is element k's.
template <int FMT>
__device__ __forceinline__ uint2 nonfinite8(uint32_t signs) {
  uint2 o = FMT == FP8Q_E2M1 ? make_uint2(0x77777777u, 0u) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t b = (signs >> k) & 1u;
    if (FMT == FP8Q_E2M1) o.x |= b << (4 * k + 3);
    else if (k < 4) o.x |= b << (8 * k + 7);
    else o.y |= b << (8 * (k - 4) + 7);
  }
  return o;
}
// The values of eight codes times s.
template <int FMT>
__device__ __forceinline__ void decode8(uint2 v, float s, float (&f)[8]) {
  uint32_t h[4];
  if constexpr (FMT == FP8Q_E2M1) {
    e2m1x8_f16(v.x, h);
  } else {
    fp8x4_f16<FMT>(v.x, h[0], h[1]);
    fp8x4_f16<FMT>(v.y, h[2], h[3]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = f16x2_f32(h[k]);
    f[2 * k] = a.x * s;
    f[2 * k + 1] = a.y * s;
  }
}

// Eight elements of a plain row: one 16-byte load of bf16, two of fp32.
template <int DT>
struct Plain8 {
  static constexpr int W = DT == FP8Q_BF16 ? 1 : 2;
  uint4 v[W];
};
template <int DT>
__device__ __forceinline__ Plain8<DT> zero8() {
  Plain8<DT> r;
#pragma unroll
  for (int w = 0; w < Plain8<DT>::W; ++w) r.v[w] = make_uint4(0, 0, 0, 0);
  return r;
}
template <int DT>
__device__ __forceinline__ Plain8<DT> load8(const void* base, int64_t at) {
  Plain8<DT> r;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (DT == FP8Q_BF16 ? 2 : 4));
#pragma unroll
  for (int w = 0; w < Plain8<DT>::W; ++w) r.v[w] = __ldcs(src + w);
  return r;
}
template <int DT>
__device__ __forceinline__ uint32_t bits8(const Plain8<DT>& r, int k) {
  return elem_bits<DT>(r.v[Plain8<DT>::W == 1 ? 0 : k >> 2], Plain8<DT>::W == 1 ? k : k & 3);
}
// Max of |x| as fp32 bits.
template <int DT>
__device__ __forceinline__ uint32_t absmax8(const Plain8<DT>& r) {
  uint32_t m = absmax_load<DT>(r.v[0]);
  if (Plain8<DT>::W == 2) m = absmax_merge<DT>(m, absmax_load<DT>(r.v[Plain8<DT>::W - 1]));
  return unpack_max<DT>(m);
}
template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&f)[8]) {
  uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(base) + at * (DT == FP8Q_BF16 ? 2 : 4));
  if (DT == FP8Q_BF16) {
    __stcs(dst, make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                           cvt_bf16x2(f[6], f[7])));
  } else {
    __stcs(dst, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])));
    __stcs(dst + 1,
           make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
  }
}
// A block's maximum from its four lanes' (every lane of the warp calls it).
__device__ __forceinline__ uint32_t block_max4(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
}

// Units of eight elements over a [rows, cols] matrix, dealt to threads: CTA b's
// thread t has units b * U * T + t, + T, ...  Four neighbouring lanes hold one
// block, since rows are whole blocks.
struct Units {
  int64_t count;       // rows * per_row
  uint32_t per_row;
  FastDiv div;
  Units() = default;
  Units(int64_t rows, int64_t cols) : count(rows * (cols / 8)), per_row((uint32_t)(cols / 8)), div(per_row) {}
  // Row and first column of unit i; past 2^31 units by a 64-bit division.
  __device__ __forceinline__ void place(int64_t i, int64_t* row, int64_t* col) const {
    if (count < (1ll << 31)) {
      const uint32_t r = div.div((uint32_t)i);
      *row = r;
      *col = (int64_t)((uint32_t)i - r * per_row) * 8;
    } else {
      *row = i / per_row;
      *col = (i - *row * per_row) * 8;
    }
  }
};
constexpr int kUnitThreads = 256;
inline int64_t unit_grid(const Units& u, int ahead) {
  return (u.count + (int64_t)kUnitThreads * ahead - 1) / ((int64_t)kUnitThreads * ahead);
}

// ---- launches ---------------------------------------------------------------
// mx4.cu
cudaError_t launch_mx4_rows(const void* x, int dtype, int64_t nelem, int headroom, int rule, uint8_t* q, uint8_t* e8m0,
                            unsigned long long* clipped, cudaStream_t s, int* launches);
cudaError_t launch_mx4_dual(const void* x, int dtype, int64_t rows, int64_t cols, int rule, int headroom,
                            uint8_t* q_row, uint8_t* e8_row, uint8_t* q_colt, uint8_t* e8_colt,
                            unsigned long long* cr, unsigned long long* cc, cudaStream_t s, int* launches);
cudaError_t read_mx4_wait_timeouts(unsigned int* count);      // and reset to 0
// mx_act.cu
cudaError_t launch_mx_decode(const MxView& m, void* out, int dtype, int64_t out_stride, cudaStream_t s, int* launches);
struct MxActForward {
  const void* z;
  const void* u;               // or null
  int64_t z_stride, u_stride;
  MxView z_saved, u_saved;     // q null: not kept
  void* h;                     // or null
  int64_t h_stride;
  MxView h_mx;                 // q null: not written
  int32_t rule;
};
cudaError_t launch_mx_act_forward(const MxActForward& a, int act, int dtype, int64_t rows, int64_t cols, cudaStream_t s,
                                  int* launches);
struct MxActBackward {
  MxView z, u;                 // u.q null: no gate
  const void* dh;
  int64_t dh_stride;
  void *dz, *du, *h;           // h or null
  int64_t dz_stride, du_stride, h_stride;
};
cudaError_t launch_mx_act_backward(const MxActBackward& a, int act, int dtype, cudaStream_t s, int* launches);
// mx_matmul_4.cu, mx_matmul_8.cu
struct MxProduct {
  MxView a, b;                 // [m, k] and [n, k]
  void* out;                   // [m, n]
  const void* add;             // or null
  int64_t out_stride, add_stride;
  int32_t fp32;                // type of out and add
};
cudaError_t launch_mx_matmul_4(const MxProduct& p, cudaStream_t s, int* launches);
cudaError_t launch_mx_matmul_8(const MxProduct& p, cudaStream_t s, int* launches);
cudaError_t read_mm4_wait_timeouts(unsigned int* count);      // and reset to 0
cudaError_t read_mm8_wait_timeouts(unsigned int* count);

}  // namespace fp8q
