// Quantising keys and values into cache slots, and reading slots back.
//
// Both are streaming codecs bound by HBM: a write moves 2 or 4 bytes in and
// 0.53 (E2M1) or 1.03 bytes out per element, a read the reverse.  The unit of
// work is eight elements of a row: 16 bytes of bf16, 4 of E2M1, so that a
// warp's accesses cover whole 128-byte lines of the plain tensor and 64-byte
// runs of a cached row; four neighbouring lanes hold one block and share its
// maximum by two shuffles.  A thread keeps its place in the rows (head and
// columns) and goes over tokens, several of them in flight: per unit only the
// slot's address is left to find.  (With a division per unit the 16384-token
// write was bound by its instructions, 23 us a launch against 18.)  Four tokens
// in flight: with eight, a read of 131072 tokens takes 138 us against 115.
// Measured, 8 heads x 128 columns, E2M1, bf16: 131072 tokens read in 116 us,
// 5.9 TB/s, 0.88 of the measured copy rate; 16384 written and read back in 37
// us (4.6 TB/s, 0.69: the two launches' ramps are a third of it); one token
// 2.8 us for both calls in a graph, all launch.
#include "kv_device.cuh"

namespace fp8q {

constexpr int kKvThreads = 256;
constexpr int kKvWriteAhead = 4;          // tokens a thread has in flight
constexpr int kKvReadAhead = 4;

struct KvCopy {
  KvShape s;
  KvPool pool[2];           // keys, values
  char* x[2];               // plain rows
  int64_t tok[2], head[2];  // strides in elements
  const int64_t* slots;
  int64_t tokens;
  FastDiv row_units, dim_units;   // units per token (heads * dim / 8) and per row (dim / 8)
  int32_t abreast, rule;          // tokens side by side in a CTA
};

// A thread's place: its units lie at x + token * tok in the plain tensor and
// at q + page * page_elems + (token of the page) * dim in the cache.
struct KvPlace {
  int64_t token, x, q;
  bool on;
};
__device__ __forceinline__ KvPlace kv_place(const KvCopy& p, int which, int ahead) {
  KvPlace u;
  const uint32_t i = blockIdx.z * kKvThreads + threadIdx.x;
  const uint32_t t = p.row_units.div(i), r = i - t * p.row_units.d;
  const uint32_t h = p.dim_units.div(r), c = r - h * p.dim_units.d;
  u.on = t < (uint32_t)p.abreast;
  u.token = (int64_t)blockIdx.x * (p.abreast * ahead) + t;
  u.x = h * p.head[which] + c * 8;
  u.q = ((int64_t)h << p.s.page_shift) * p.s.dim + c * 8;
  return u;
}
// Slot of the j-th token of a thread; below 0: none.
__device__ __forceinline__ int64_t kv_slot(const KvCopy& p, const KvPlace& u, int j) {
  const int64_t t = u.token + j * p.abreast;
  if (!u.on || t >= p.tokens) return -1;
  // a plain load: the grid before this one may still be writing slots when this
  // CTA comes to the SM, so they are not read-only for the whole kernel
  const int64_t s = p.slots[t];
  return s < p.s.slots ? s : -1;
}
__device__ __forceinline__ int64_t kv_at(const KvCopy& p, const KvPlace& u, int64_t slot) {
  const int64_t page = slot >> p.s.page_shift, off = slot & ((1ll << p.s.page_shift) - 1);
  return u.q + ((page * p.s.heads << p.s.page_shift) + off) * p.s.dim;
}

template <int FMT, int DT>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const __grid_constant__ KvCopy p) {
  constexpr int W = DT == FP8Q_BF16 ? 1 : 2, U = kKvWriteAhead;        // W: 16-byte loads per unit
  grid_begin();
  const int which = blockIdx.y;
  const KvPlace u = kv_place(p, which, U);
  const KvPool pool = p.pool[which];
  int64_t slot[U];
  uint4 v[U][W];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    slot[j] = kv_slot(p, u, j);
#pragma unroll
    for (int w = 0; w < W; ++w) v[j][w] = make_uint4(0, 0, 0, 0);
    if (slot[j] < 0) continue;
    const uint4* src = reinterpret_cast<const uint4*>(
        p.x[which] + (u.x + (u.token + j * p.abreast) * p.tok[which]) * (DT == FP8Q_BF16 ? 2 : 4));
#pragma unroll
    for (int w = 0; w < W; ++w) v[j][w] = __ldcs(src + w);
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    // rows are whole blocks: the four lanes of one have the same token or none
    uint32_t m = absmax_load<DT>(v[j][0]);
    if (W == 2) m = absmax_merge<DT>(m, absmax_load<DT>(v[j][W - 1]));
    m = unpack_max<DT>(m);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (slot[j] < 0) continue;
    const int64_t at = kv_at(p, u, slot[j]);
    const bool finite = m < 0x7F800000u;
    constexpr int F8 = FMT == FP8Q_E2M1 ? FP8Q_E4M3 : FMT;
    const int E = !finite ? 0 : block_exp<FMT>(m, p.rule, 0);
    const float s = pow2f(-E);
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      f[k] = __uint_as_float(elem_bits<DT>(v[j][W == 1 ? 0 : k >> 2], W == 1 ? k : k & 3)) * s;
    uint2 o;
    if (FMT == FP8Q_E2M1) {
      o.x = cvt_e2m1x8(f);
    } else {
      o.x = cvt_pair<F8>(f[0], f[1]) | (cvt_pair<F8>(f[2], f[3]) << 16);
      o.y = cvt_pair<F8>(f[4], f[5]) | (cvt_pair<F8>(f[6], f[7]) << 16);
    }
    if (!finite) {                         // sign|largest for every element
      uint32_t sign = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        sign |= (elem_bits<DT>(v[j][W == 1 ? 0 : k >> 2], W == 1 ? k : k & 3) >> 31) << k;
      o.x = FMT == FP8Q_E2M1 ? 0x77777777u : 0x7F7F7F7Fu;
      o.y = 0x7F7F7F7Fu;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t b = (sign >> k) & 1u;
        if (FMT == FP8Q_E2M1) o.x |= b << (4 * k + 3);
        else if (k < 4) o.x |= b << (8 * k + 7);
        else o.y |= b << (8 * (k - 4) + 7);
      }
    }
    if (FMT == FP8Q_E2M1) *reinterpret_cast<uint32_t*>(pool.q + (at >> 1)) = o.x;
    else *reinterpret_cast<uint2*>(pool.q + at) = o;
    if ((threadIdx.x & 3) == 0) pool.e8m0[at >> 5] = (uint8_t)(finite ? E + 127 : 255);
  }
}

template <int FMT, int DT>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const __grid_constant__ KvCopy p) {
  constexpr int U = kKvReadAhead;
  grid_begin();
  const int which = blockIdx.y;
  const KvPlace u = kv_place(p, which, U);
  const KvPool pool = p.pool[which];
  uint2 v[U];
  uint32_t e[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t slot = kv_slot(p, u, j);
    v[j] = make_uint2(0, 0);
    e[j] = 127;
    if (slot < 0) continue;
    const int64_t at = kv_at(p, u, slot);
    if (FMT == FP8Q_E2M1) v[j].x = __ldcs(reinterpret_cast<const uint32_t*>(pool.q + (at >> 1)));
    else v[j] = __ldcs(reinterpret_cast<const uint2*>(pool.q + at));
    e[j] = pool.e8m0[at >> 5];
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t t = u.token + j * p.abreast;
    if (!u.on || t >= p.tokens) continue;
    uint32_t h[4];
    if (FMT == FP8Q_E2M1) {
      e2m1x8_f16(v[j].x, h);
    } else {
      constexpr int F8 = FMT == FP8Q_E2M1 ? FP8Q_E4M3 : FMT;
      fp8x4_f16<F8>(v[j].x, h[0], h[1]);
      fp8x4_f16<F8>(v[j].y, h[2], h[3]);
    }
    const float s = e8m0_value(e[j]);
    float f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 a = f16x2_f32(h[k]);
      f[2 * k] = a.x * s;
      f[2 * k + 1] = a.y * s;
    }
    uint4* dst = reinterpret_cast<uint4*>(p.x[which] + (u.x + t * p.tok[which]) * (DT == FP8Q_BF16 ? 2 : 4));
    if (DT == FP8Q_BF16) {
      __stcs(dst, make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                             cvt_bf16x2(f[6], f[7])));
    } else {
      const uint32_t* b = reinterpret_cast<const uint32_t*>(f);
      __stcs(dst, make_uint4(b[0], b[1], b[2], b[3]));
      __stcs(dst + 1, make_uint4(b[4], b[5], b[6], b[7]));
    }
  }
}

template <int FMT, int DT>
static const void* copy_kernel(bool write) {
  return write ? reinterpret_cast<const void*>(kv_write_kernel<FMT, DT>)
               : reinterpret_cast<const void*>(kv_read_kernel<FMT, DT>);
}

static cudaError_t launch_any(bool write, const KvShape& s, int format, KvPool k, KvPool v, void* kx, void* vx,
                              int dtype, int64_t tokens, const int64_t* strides, const int64_t* slots, int rule,
                              cudaStream_t st, int* launches) {
  KvCopy p;
  p.s = s;
  p.pool[0] = k;
  p.pool[1] = v;
  p.x[0] = static_cast<char*>(kx);
  p.x[1] = static_cast<char*>(vx);
  p.tok[0] = strides[0];
  p.head[0] = strides[1];
  p.tok[1] = strides[2];
  p.head[1] = strides[3];
  p.slots = slots;
  p.tokens = tokens;
  p.rule = rule;
  const uint32_t row = (uint32_t)s.heads * (s.dim / 8);
  p.row_units = FastDiv(row);
  p.dim_units = FastDiv((uint32_t)s.dim / 8);
  // a CTA has several tokens abreast, or one token's row takes several CTAs (grid z)
  p.abreast = row >= kKvThreads ? 1 : kKvThreads / row;
  const int64_t per = (int64_t)p.abreast * (write ? kKvWriteAhead : kKvReadAhead);
  const dim3 grid((unsigned)((tokens + per - 1) / per), 2, (row + kKvThreads - 1) / kKvThreads);
  const bool b = dtype == FP8Q_BF16;
  const void* kernel;
  if (format == FP8Q_E2M1) kernel = b ? copy_kernel<FP8Q_E2M1, FP8Q_BF16>(write) : copy_kernel<FP8Q_E2M1, FP8Q_F32>(write);
  else if (format == FP8Q_E4M3) kernel = b ? copy_kernel<FP8Q_E4M3, FP8Q_BF16>(write) : copy_kernel<FP8Q_E4M3, FP8Q_F32>(write);
  else kernel = b ? copy_kernel<FP8Q_E5M2, FP8Q_BF16>(write) : copy_kernel<FP8Q_E5M2, FP8Q_F32>(write);
  void* args[1] = {&p};
  return launch_dependent(kernel, grid, kKvThreads, 0, args, st, launches);
}

cudaError_t launch_kv_write(const KvShape& s, int format, KvPool k, KvPool v, const void* kx, const void* vx,
                            int dtype, int64_t tokens, const int64_t* strides, const int64_t* slots, int rule,
                            cudaStream_t st, int* launches) {
  return launch_any(true, s, format, k, v, const_cast<void*>(kx), const_cast<void*>(vx), dtype, tokens, strides,
                    slots, rule, st, launches);
}

cudaError_t launch_kv_read(const KvShape& s, int format, KvPool k, KvPool v, void* kx, void* vx, int dtype,
                           int64_t tokens, const int64_t* strides, const int64_t* slots, cudaStream_t st,
                           int* launches) {
  return launch_any(false, s, format, k, v, kx, vx, dtype, tokens, strides, slots, 0, st, launches);
}

}  // namespace fp8q
