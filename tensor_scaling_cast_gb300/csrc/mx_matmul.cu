// Products of two matrices in MX blocks: out = a b^T (+ add), 4 bits by 4 bits
// or 8 by 8, on the block-scaled tensor core instructions.
//
// A K block is 128 bytes of a row, 256 elements of 4 bits or 128 of 8: one
// 128-byte swizzle row of shared memory, four products.  Its codes come by TMA
// (zeros outside the matrices); its scales, rows of E8M0 bytes in memory, are
// read by four warps that write them in the order that the tensor core takes
// them in (tcgen05.cuh), one thread a row.
#include <cuda.h>
#include <cuda_runtime.h>

#include "mx_linear.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace fp8q {

static __device__ unsigned int g_mm_wait_timeouts;   // see fp8q_pipeline_status

cudaError_t read_mm_wait_timeouts(unsigned int* count) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(count, g_mm_wait_timeouts, sizeof(unsigned int));
  if (e == cudaSuccess && *count) e = cudaMemcpyToSymbol(g_mm_wait_timeouts, &zero, sizeof(unsigned int));
  return e;
}

// Scales of one operand: rows of `bytes` E8M0 bytes.
struct MmScales {
  const uint8_t* e8m0;
  int64_t stride;
  int32_t rows, bytes;
  int32_t whole;             // rows start at multiples of a K block's bytes
};
struct MmArgs {
  CUtensorMap w, t;          // codes of the operand with 128-row tiles, of the other
  MmScales ws, ts;
  int32_t kblocks, w_tiles, splits;
  uint32_t idesc;
  void* out;
  const void* add;
  int64_t out_stride, add_stride;
  int32_t fp32, w_is_a;      // out row: index in w (else in t)
};

// E8M0 bytes of a row's K block (8 in 4 bits, 4 in 8 bits); 1 where there are
// none: the codes there are zeros.
template <bool F4>
__device__ __forceinline__ uint2 load_scales(const MmScales& s, int64_t row, int kb) {
  constexpr int SB = F4 ? 8 : 4;
  uint2 v = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  if (row >= s.rows) return v;
  const int at = kb * SB;
  const uint8_t* src = s.e8m0 + row * s.stride + at;
  if (s.whole && at + SB <= s.bytes) {
    if (F4) v = *reinterpret_cast<const uint2*>(src);
    else v.x = *reinterpret_cast<const uint32_t*>(src);
    return v;
  }
#pragma unroll
  for (int k = 0; k < SB; ++k) {
    if (at + k >= s.bytes) break;
    uint32_t& word = k < 4 ? v.x : v.y;
    word = (word & ~(0xFFu << (8 * (k & 3)))) | ((uint32_t)src[k] << (8 * (k & 3)));
  }
  return v;
}
// Into the place of row r of 128: 512 bytes for each 128 elements.
template <bool F4>
__device__ __forceinline__ void store_scales(uint32_t smem, int r, uint2 v) {
  const uint32_t at = smem + (r & 31) * 16 + (r >> 5) * 4;
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v.x) : "memory");
  if (F4) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 512), "r"(v.y) : "memory");
}

__device__ __forceinline__ float add_of(const MmArgs& p, int64_t m, int64_t n) {
  if (!p.add) return 0.0f;
  const int64_t at = m * p.add_stride + n;
  return p.fp32 ? static_cast<const float*>(p.add)[at]
                : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.add)[at] << 16);
}
__device__ __forceinline__ void put(const MmArgs& p, int64_t m, int64_t n, float v) {
  if (p.add) v += add_of(p, m, n);
  const int64_t at = m * p.out_stride + n;
  if (p.fp32) static_cast<float*>(p.out)[at] = v;
  else static_cast<uint16_t*>(p.out)[at] = (uint16_t)cvt_bf16x2(v, v);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float cluster_load(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.f32 %0, [a];\n}"
               : "=f"(v) : "r"(addr), "r"(rank) : "memory");
  return v;
}

// ---- tiles of 128 x NT, the sum split over a cluster -----------------------------

template <bool F4, int NT>
struct SplitCfg {
  static constexpr int kScales = F4 ? 1024 : 512;                  // of 128 rows
  static constexpr int kT = 128 * 128, kWs = kT + NT * 128, kTs = kWs + kScales;
  static constexpr int kStage = kTs + kScales;                     // a multiple of 1024
  // two CTAs per SM, so that one's loads run while the other starts or ends
  static constexpr int kStages = 112 * 1024 / kStage;
  static constexpr int kSmem = kStages * kStage + 1024;
  static constexpr int kColumns = NT + 16 <= 32 ? 32 : NT + 16 <= 64 ? 64 : NT + 16 <= 128 ? 128 : 256;
  static_assert(kStage % 1024 == 0 && 128 * NT * 4 <= kStages * kStage, "swizzled tiles; the parts of the sum");
};
constexpr int kSplitThreads = 192;         // TMA, products, and four warps of scales that end as the epilogue
constexpr int kScalesAhead = 4;            // K blocks whose scales a thread has in flight

template <bool F4, int NT>
__global__ void __launch_bounds__(kSplitThreads, 2) mm_split_kernel(const __grid_constant__ MmArgs p) {
  using C = SplitCfg<F4, NT>;
  constexpr int ST = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[ST], empty[ST], done;
  __shared__ uint32_t s_tmem;
  const uint32_t smem = smem_addr(smem_raw) + (-smem_addr(smem_raw) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1 + 4);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    fence_barrier_init();
    prefetch_tensormap(&p.w);
    prefetch_tensormap(&p.t);
  }
  if (warp == 1) tmem_alloc(&s_tmem, C::kColumns);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  // not before: the next grid's CTAs may take tensor memory once they come to the SM
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = s_tmem;
  const uint32_t rank = p.splits > 1 ? cluster_rank() : 0u;
  const int tile = blockIdx.x / p.splits;
  const int tt = tile / p.w_tiles, tw = tile - tt * p.w_tiles;
  const int kb0 = (int)((int64_t)p.kblocks * rank / p.splits);
  const int n = (int)((int64_t)p.kblocks * (rank + 1) / p.splits) - kb0;
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (; i < n; ++i) {
        const int st = i % ST;
        if (i >= ST && !mbar_wait(&empty[st], (i / ST - 1) & 1)) {
          ok = false;
          break;
        }
        const uint32_t at = smem + st * C::kStage;
        mbar_arrive_expect_tx(&full[st], C::kWs);
        tma_load_2d_at(at, &p.w, &full[st], (kb0 + i) * 128, tw * 128);
        tma_load_2d_at(at + C::kT, &p.t, &full[st], (kb0 + i) * 128, tt * NT);
      }
      if (!ok)                                       // loads in flight land before the CTA leaves
        for (int k = max(0, i - ST); k < i; ++k) mbar_wait(&full[k % ST], (k / ST) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t sf_w = tmem + NT, sf_t = tmem + NT + 8;
      const uint32_t hi = desc_hi(1024);
      for (int i = 0; i < n; ++i) {
        const int st = i % ST;
        if (!mbar_wait(&full[st], (i / ST) & 1)) {
          ok = false;
          break;
        }
        tmem_fence_after();
        const uint32_t at = smem + st * C::kStage;
        // copies and products are carried out in the order of their issue
#pragma unroll
        for (int c = 0; c < (F4 ? 2 : 1); ++c) {
          sf_copy<1>(sf_w + 4 * c, sf_desc(at + C::kWs + 512 * c));
          sf_copy<1>(sf_t + 4 * c, sf_desc(at + C::kTs + 512 * c));
        }
        const uint32_t w_lo = desc_lo(at, 16), t_lo = desc_lo(at + C::kT, 16);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t col = F4 ? 4 * (s >> 1) : 0;
          mma_mx<F4, 1>(tmem, w_lo + 2 * s, t_lo + 2 * s, hi, mx_idesc_step<F4>(p.idesc, F4 ? s & 1 : s), sf_w + col,
                        sf_t + col, i > 0 || s > 0);
        }
        mma_commit(&empty[st]);
      }
      mma_commit(&done);
    }
  } else {
    const int r = threadIdx.x - 64;
    const int64_t wr = (int64_t)tw * 128 + r, tr = r < NT ? (int64_t)tt * NT + r : p.ts.rows;
    uint2 w[kScalesAhead], t[kScalesAhead], w2[kScalesAhead], t2[kScalesAhead];
#pragma unroll
    for (int j = 0; j < kScalesAhead; ++j) {
      if (j >= n) break;
      w[j] = load_scales<F4>(p.ws, wr, kb0 + j);
      t[j] = load_scales<F4>(p.ts, tr, kb0 + j);
    }
    for (int b = 0; b < n && ok; b += kScalesAhead) {
#pragma unroll
      for (int j = 0; j < kScalesAhead; ++j) {
        if (b + kScalesAhead + j >= n) break;
        w2[j] = load_scales<F4>(p.ws, wr, kb0 + b + kScalesAhead + j);
        t2[j] = load_scales<F4>(p.ts, tr, kb0 + b + kScalesAhead + j);
      }
#pragma unroll
      for (int j = 0; j < kScalesAhead; ++j) {
        const int i = b + j, st = i % ST;
        if (i >= n) break;
        if (i >= ST) {
          const bool got = mbar_wait(&empty[st], (i / ST - 1) & 1);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            break;
          }
        }
        const uint32_t at = smem + st * C::kStage;
        store_scales<F4>(at + C::kWs, r, w[j]);
        if (r < NT) store_scales<F4>(at + C::kTs, r, t[j]);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        w[j] = w2[j];
        t[j] = t2[j];
      }
    }
    if (!mbar_wait(&done, 0)) ok = false;
    __syncwarp();
    tmem_fence_after();
    const int q = warp & 3, row = 32 * q + lane;     // this warp's lanes of tensor memory
    const int64_t wi = (int64_t)tw * 128 + row, t0 = (int64_t)tt * NT;
#pragma unroll 1
    for (int c = 0; c < NT; c += 16) {
      uint32_t v[16];
      tmem_ld16(v, tmem + ((uint32_t)(32 * q) << 16) + c);
      tmem_wait_ld(v);
      if (p.splits > 1) {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(smem + ((c + k) * 128 + row) * 4), "r"(v[k]) : "memory");
      } else if (wi < p.ws.rows) {
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int64_t ti = t0 + c + k;
          if (ti < p.ts.rows) put(p, p.w_is_a ? wi : ti, p.w_is_a ? ti : wi, __uint_as_float(v[k]));
        }
      }
    }
    tmem_fence_before();
  }
  if (!ok && lane == 0) atomicAdd(&g_mm_wait_timeouts, 1u);
  __syncwarp();
  if (p.splits > 1) {
    // each CTA of the cluster adds up its share of the columns, parts in order
    cluster_barrier();
    if (warp >= 2) {
      const int row = threadIdx.x - 64;
      const int64_t wi = (int64_t)tw * 128 + row;
      const int c1 = NT * ((int)rank + 1) / p.splits;
      for (int c = NT * (int)rank / p.splits; c < c1; ++c) {
        const int64_t ti = (int64_t)tt * NT + c;
        if (ti >= p.ts.rows) break;
        float sum = 0.0f;
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) sum += cluster_load(smem + (c * 128 + row) * 4, s);
        if (wi < p.ws.rows) put(p, p.w_is_a ? wi : ti, p.w_is_a ? ti : wi, sum);
      }
    }
    cluster_barrier();                               // nobody leaves while its part is read
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tmem_fence_after();
    tmem_free(tmem, C::kColumns);
  }
}

// Tensor map of a matrix's codes as bytes: boxes of 128 bytes x `box` rows,
// 128-byte swizzle, zeros outside.
static cudaError_t encode_codes(CUtensorMap* map, const MxView& m, int box) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)m.row_bytes(), (cuuint64_t)m.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)m.q_stride};
  const cuuint32_t shape[2] = {128u, (cuuint32_t)box}, step[2] = {1u, 1u};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.q, dims, strides, shape, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}
static MmScales scales_of(const MxView& m) {
  const int64_t block = m.format == FP8Q_E2M1 ? 8 : 4;
  MmScales s;
  s.e8m0 = m.e8m0;
  s.stride = m.e_stride;
  s.rows = (int32_t)m.rows;
  s.bytes = (int32_t)(m.cols / 32);
  s.whole = reinterpret_cast<uintptr_t>(m.e8m0) % block == 0 && (m.rows == 1 || m.e_stride % block == 0);
  return s;
}

template <bool F4, int NT>
static cudaError_t launch_split(const MxProduct& p, const MxView& w, const MxView& t, bool w_is_a, cudaStream_t s,
                                int* launches) {
  using C = SplitCfg<F4, NT>;
  const void* kern = reinterpret_cast<const void*>(mm_split_kernel<F4, NT>);
  int occ = 1;
  cudaError_t e = kernel_occupancy(kern, kSplitThreads, C::kSmem, &occ);
  if (e != cudaSuccess) return e;
  MmArgs a;
  if ((e = encode_codes(&a.w, w, 128)) != cudaSuccess) return e;
  if ((e = encode_codes(&a.t, t, NT)) != cudaSuccess) return e;
  a.ws = scales_of(w);
  a.ts = scales_of(t);
  a.kblocks = (int32_t)((w.row_bytes() + 127) / 128);
  a.w_tiles = (int32_t)((w.rows + 127) / 128);
  const int64_t tiles = (int64_t)a.w_tiles * ((t.rows + NT - 1) / NT);
  const int sms = sm_count(device_of_current());
  int splits = 1;
  while (splits < 8 && tiles * splits * 2 <= 2 * sms && a.kblocks / (splits * 2) >= 2) splits *= 2;
  a.splits = splits;
  a.idesc = mx_idesc(F4, w.format, t.format, 128, NT);
  a.out = p.out;
  a.add = p.add;
  a.out_stride = p.out_stride;
  a.add_stride = p.add_stride;
  a.fp32 = p.fp32;
  a.w_is_a = w_is_a;
  if (tiles * splits > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * splits));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  void* args[] = {&a};
  e = cudaLaunchKernelExC(&cfg, kern, args);
  if (e == cudaSuccess) ++*launches;
  return e;
}

template <bool F4>
static cudaError_t launch_format(const MxProduct& p, cudaStream_t s, int* launches) {
  const bool w_is_a = p.a.rows > p.b.rows;           // the operand with more rows has the 128-row tiles
  const MxView &w = w_is_a ? p.a : p.b, &t = w_is_a ? p.b : p.a;
  if (t.rows <= 16) return launch_split<F4, 16>(p, w, t, w_is_a, s, launches);
  if (t.rows <= 32) return launch_split<F4, 32>(p, w, t, w_is_a, s, launches);
  if (t.rows <= 64) return launch_split<F4, 64>(p, w, t, w_is_a, s, launches);
  return launch_split<F4, 128>(p, w, t, w_is_a, s, launches);
}

cudaError_t launch_mx_matmul(const MxProduct& p, cudaStream_t s, int* launches) {
  return p.a.format == FP8Q_E2M1 ? launch_format<true>(p, s, launches) : launch_format<false>(p, s, launches);
}

}  // namespace fp8q
