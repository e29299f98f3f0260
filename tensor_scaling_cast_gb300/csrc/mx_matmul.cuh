// Products of two matrices in MX blocks: out = a b^T (+ add), 4 bits by 4 bits
// or 8 by 8, on the block-scaled tensor core instructions.
//
// A K block is 128 bytes of a row, 256 elements of 4 bits or 128 of 8: one
// 128-byte swizzle row of shared memory, four products.  Its codes come by TMA
// (zeros outside the matrices); its scales, rows of E8M0 bytes in memory, are
// read by four warps that write them in the order that the tensor core takes
// them in (tcgen05.cuh), one thread a row.
//
// Few rows are bound by the latency of a launch, a first load and a join, then
// by HBM: 1 x 8192 x 2048 in 4 bits 4.7 us, 1 x 8192 x 8192 8.7 us (36 MB, 4.1
// TB/s), 64 x 2048 x 8192 7.4 us.  Large ones are bound by the tensor cores,
// 75% of whose cycles in 4 bits and 85% in 8 have a product (8192 x 8192 x 8192:
// 165 us = 6.7 PFLOP/s and 340 us = 3.2, there with the clock at 1.56 GHz for
// the power); short sums by storing them (16384 x 8192 x 2048 in 4 bits 91 us
// for 268 MB of bf16).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "mx_linear.cuh"
#include "mx_matmul_plan.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace fp8q {

static __device__ unsigned int g_mm_wait_timeouts;   // of this translation unit; see fp8q_pipeline_status

static cudaError_t read_timeouts(unsigned int* count) {
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
  int32_t sectors;           // every row is a number of whole 32-byte sectors
};
struct MmArgs {
  CUtensorMap w, t;          // codes of the operand with 128-row tiles, of the other
  CUtensorMap o;             // out, where it leaves by TMA
  MmScales ws, ts;
  int32_t kblocks, w_tiles, t_tiles, splits;
  uint32_t idesc;
  void* out;
  const void* add;
  int64_t out_stride, add_stride;
  int32_t fp32, w_is_a;      // out row: index in w (else in t)
  int32_t out_quads, add_quads;     // rows start at multiples of four elements
  int32_t out_vector, add_vector;   // of 16 bytes
};

__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 32 bytes at a multiple of 32, past L1; all 1 (0x7F) from nowhere.
__device__ __forceinline__ void load_sector(const uint8_t* src, uint32_t (&v)[8]) {
  if (src) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(src));
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0x7F7F7F7Fu;
  }
}

// One warp brings the scales of 128 rows (`row0` on, up to `limit`) for K blocks
// kb0 .. kb0 + n - 1; lane l has rows l, l + 32, l + 64 and l + 96, whose words
// for the same 128 elements lie together in the order of the copies, so that a
// K block's go out as one or two 16-byte stores without conflicts.  Rows are
// read in whole sectors, 32 bytes at multiples of 32, past L1 (whose bandwidth
// the operands need): a row that starts in the middle of one takes its bytes
// from two neighbours, of which it reads one at a time.  A sector is read only
// if some byte of it is the row's.  Bytes past the row's end are 1 (0x7F): the
// codes there are zeros.
// put(i, words): K block i's words of the four rows, [word][row]; false: stop.
template <bool F4, int R, bool SHIFTED, class Put>
__device__ __forceinline__ bool feed_groups(const uint8_t* const (&base)[R], const uint32_t (&off)[R], const int (&end)[R],
                                            int bytes, int n, Put put) {
  constexpr int W = F4 ? 2 : 1, G = 8 / W;           // words of a block, blocks of 32 bytes
  const auto load = [&](int i, uint32_t (&v)[R][8]) {
#pragma unroll
    for (int j = 0; j < R; ++j) load_sector(32 * i < end[j] ? base[j] + 32 * (int64_t)i : nullptr, v[j]);
  };
  const int groups = (n + G - 1) / G;
  uint32_t held[R][8], next[R][8], then[SHIFTED ? R : 1][8];
  load(0, held);
  if constexpr (SHIFTED) load(1, next);
#pragma unroll 1
  for (int i = 0; i < groups; ++i) {
    uint32_t g[R][8];
    if constexpr (SHIFTED) {
      load(i + 2, then);                             // on its way meanwhile
#pragma unroll
      for (int j = 0; j < R; ++j) {
        uint32_t x[16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          x[k] = held[j][k];
          x[k + 8] = next[j][k];
        }
#pragma unroll
        for (int k = 0; k < 12; ++k) x[k] = off[j] & 16 ? x[k + 4] : x[k];
#pragma unroll
        for (int k = 0; k < 10; ++k) x[k] = off[j] & 8 ? x[k + 2] : x[k];
#pragma unroll
        for (int k = 0; k < 9; ++k) x[k] = off[j] & 4 ? x[k + 1] : x[k];
#pragma unroll
        for (int k = 0; k < 8; ++k) g[j][k] = __funnelshift_r(x[k], x[k + 1], 8 * (off[j] & 3));
      }
    } else {
      load(i + 1, next);
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) g[j][k] = held[j][k];
    }
    if (32 * i + 32 > bytes) {                       // the rows end in this group
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int in = bytes - 32 * i - 4 * k;
        const uint32_t mask = in >= 4 ? 0xFFFFFFFFu : in <= 0 ? 0u : (1u << (8 * in)) - 1u;
#pragma unroll
        for (int j = 0; j < R; ++j) g[j][k] = (g[j][k] & mask) | (0x7F7F7F7Fu & ~mask);
      }
    }
#pragma unroll
    for (int b = 0; b < G; ++b) {
      if (i * G + b >= n) break;
      uint32_t words[W][4];
#pragma unroll
      for (int w = 0; w < W; ++w)
#pragma unroll
        for (int j = 0; j < 4; ++j) words[w][j] = j < R ? g[j < R ? j : 0][W * b + w] : 0x7F7F7F7Fu;
      if (!put(i * G + b, words)) return false;
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        held[j][k] = next[j][k];
        if constexpr (SHIFTED) next[j][k] = then[j][k];
      }
  }
  return true;
}
template <bool F4, int ROWS, class Put>
__device__ __forceinline__ bool feed_scales(const MmScales& sc, int64_t row0, int64_t limit, int kb0, int n, Put put) {
  constexpr int R = (ROWS + 31) / 32;                // rows of a lane
  const int lane = threadIdx.x & 31, at = kb0 * (F4 ? 8 : 4), bytes = sc.bytes - at;
  const uint8_t* base[R];
  uint32_t off[R], any = 0;
  int end[R];                                        // bytes from base to the row's end; 0 for no row
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int64_t row = row0 + lane + 32 * j;
    const uint8_t* src = sc.e8m0 + row * sc.stride + at;
    off[j] = (uint32_t)(reinterpret_cast<uintptr_t>(src) & 31u);
    base[j] = src - off[j];
    end[j] = row < limit ? (int)off[j] + bytes : 0;
    any |= off[j];
  }
  return __any_sync(0xFFFFFFFFu, any != 0) ? feed_groups<F4, R, true>(base, off, end, bytes, n, put)
                                           : feed_groups<F4, R, false>(base, off, end, bytes, n, put);
}

__device__ __forceinline__ float add_of(const MmArgs& p, int64_t m, int64_t n) {
  const int64_t at = m * p.add_stride + n;
  return p.fp32 ? static_cast<const float*>(p.add)[at]
                : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p.add)[at] << 16);
}
// add's four values of row m from column n on, the first of them inside.
__device__ __forceinline__ float4 add4(const MmArgs& p, int64_t m, int64_t n, int64_t cols) {
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (p.add_quads && n + 4 <= cols) {
    const char* src = static_cast<const char*>(p.add) + (m * p.add_stride + n) * (p.fp32 ? 4 : 2);
    if (p.fp32) return *reinterpret_cast<const float4*>(src);
    const uint2 x = *reinterpret_cast<const uint2*>(src);
    return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xFFFF0000u), __uint_as_float(x.y << 16),
                       __uint_as_float(x.y & 0xFFFF0000u));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (n + k < cols) v[k] = add_of(p, m, n + k);
  return make_float4(v[0], v[1], v[2], v[3]);
}
// Four values of row m of out from column n on, the first of them inside.
__device__ __forceinline__ void put4(const MmArgs& p, int64_t m, int64_t n, int64_t cols, const float4& sum) {
  const float v[4] = {sum.x, sum.y, sum.z, sum.w};
  char* dst = static_cast<char*>(p.out) + (m * p.out_stride + n) * (p.fp32 ? 4 : 2);
  if (p.out_quads && n + 4 <= cols) {
    if (p.fp32) *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    else *reinterpret_cast<uint2*>(dst) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
    return;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (n + k >= cols) break;
    if (p.fp32) reinterpret_cast<float*>(dst)[k] = v[k];
    else reinterpret_cast<uint16_t*>(dst)[k] = (uint16_t)cvt_bf16x2(v[k], v[k]);
  }
}

// The warp's index as a value that the compiler knows to be the warp's: the
// issuing warps' addresses and descriptors then stay in uniform registers,
// where the tensor core instructions take them from.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float4 load_shared4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// ---- tiles of 128 x NT, the sum split over a cluster -----------------------------
//
// The matrix of more rows has the 128 lanes of tensor memory, the other NT
// columns.  A CTA sums a range of K; parts meet in the cluster's shared memory
// and are added in the order of K.

template <bool F4, int NT>
struct SplitCfg {
  static constexpr int kScales = F4 ? 1024 : 512;                  // of 128 rows
  static constexpr int kT = 128 * 128, kWs = kT + NT * 128, kTs = kWs + kScales;
  static constexpr int kStage = kTs + kScales;                     // a multiple of 1024
  // two CTAs per SM, so that one's loads run while the other starts or ends
  static constexpr int kStages = 112 * 1024 / kStage;
  static constexpr int kSmem = kStages * kStage + 1024;
  static constexpr int kColumns = NT + 16 * kStages <= 128 ? 128 : 256;   // sums, scales of each stage
  static_assert(NT + 16 * kStages <= kColumns, "two CTAs per SM have 256 columns each");
  static_assert(kStage % 1024 == 0 && 132 * NT * 4 <= kStages * kStage && 128 * (NT + 4) * 4 <= kStages * kStage, "swizzled tiles; the parts of the sum");
};
constexpr int kSplitThreads = 192;         // TMA, products, and four warps of the epilogue, the first two of which bring scales

template <bool F4, int NT>
__global__ void __launch_bounds__(kSplitThreads, 2) mm_split_kernel(const __grid_constant__ MmArgs p) {
  using C = SplitCfg<F4, NT>;
  constexpr int ST = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[ST], empty[ST], done;
  __shared__ uint32_t s_tmem;
  const uint32_t smem = uniform(smem_addr(smem_raw) + (-smem_addr(smem_raw) & 1023u));
  const int warp = warp_index(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1 + 2);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    fence_barrier_init();
    prefetch_tensormap(&p.w);
    prefetch_tensormap(&p.t);
  }
  const uint32_t rank = p.splits > 1 ? cluster_rank() : 0u;
  const int tile = blockIdx.x / p.splits;
  const int tt = tile / p.w_tiles, tw = tile - tt * p.w_tiles;
  const int kb0 = (int)((int64_t)p.kblocks * rank / p.splits);
  const int n = (int)((int64_t)p.kblocks * (rank + 1) / p.splits) - kb0;
  bool ok = true;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const auto load = [&](int i) {
    const int st = i % ST;
    const uint32_t at = smem + st * C::kStage;
    mbar_arrive_expect_tx(&full[st], C::kWs);
    tma_load_2d_at(at, &p.w, &full[st], (kb0 + i) * 128, tw * 128);
    tma_load_2d_at(at + C::kT, &p.t, &full[st], (kb0 + i) * 128, tt * NT);
  };
  // the first codes are on their way before there is tensor memory
  if (warp == 0 && lane == 0)
    for (int i = 0; i < min(n, ST); ++i) load(i);
  if (warp == 1) tmem_alloc(&s_tmem, C::kColumns);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  // not before: the next grid's CTAs may take tensor memory once they come to the SM
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = uniform(s_tmem);

  if (warp == 0) {
    if (lane == 0) {
      int i = ST;
      for (; i < n; ++i) {
        if (!mbar_wait(&empty[i % ST], (i / ST - 1) & 1)) {
          ok = false;
          break;
        }
        load(i);
      }
      if (!ok)                                       // loads in flight land before the CTA leaves
        for (int k = max(0, i - ST); k < i; ++k) mbar_wait(&full[k % ST], (k / ST) & 1);
    }
  } else if (warp == 1) {
    const uint32_t hi = desc_hi(1024);
    // scales are copied ahead of the block before, to their stage's place (see mm_pair_kernel)
    const auto copy = [&](int i) {
      const int st = i % ST;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[st], (i / ST) & 1))) return false;
      tmem_fence_after();
      const uint32_t at = smem + st * C::kStage, to = tmem + NT + st * 16;
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < (F4 ? 2 : 1); ++c) {
          sf_copy<1>(to + 4 * c, sf_desc(at + C::kWs + 512 * c));
          sf_copy<1>(to + 8 + 4 * c, sf_desc(at + C::kTs + 512 * c));
        }
      }
      __syncwarp();
      return true;
    };
    ok = copy(0);
    for (int i = 0; i < n && ok; ++i) {
      if (i + 1 < n) ok = copy(i + 1);
      if (!ok) break;
      const int st = i % ST;
      const uint32_t at = smem + st * C::kStage, sf = tmem + NT + st * 16;
      const uint32_t w_lo = desc_lo(at, 16), t_lo = desc_lo(at + C::kT, 16);
      if (elect_one()) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t col = F4 ? 4 * (s >> 1) : 0;
          mma_mx<F4, 1>(tmem, w_lo + 2 * s, t_lo + 2 * s, hi, mx_idesc_step<F4>(p.idesc, F4 ? s & 1 : s), sf + col,
                        sf + 8 + col, i > 0 || s > 0);
        }
        mma_commit(&empty[st]);
        if (i + 1 == n) mma_commit(&done);
      }
      __syncwarp();
    }
    if (!ok) {                             // for the epilogue, which waits
      if (elect_one()) mma_commit(&done);
      __syncwarp();
    }
  } else {
    if (warp < 4) {
      const auto put = [&](uint32_t at, int i, const auto& w) {
        const int st = i % ST;
        if (i >= ST && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], (i / ST - 1) & 1))) return false;
        const uint32_t to = smem + st * C::kStage + at + lane * 16;
#pragma unroll
        for (int c = 0; c < (F4 ? 2 : 1); ++c) st_shared16(to + 512 * c, w[c][0], w[c][1], w[c][2], w[c][3]);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        return true;
      };
      if (warp == 2)
        ok = feed_scales<F4, 128>(p.ws, (int64_t)tw * 128, p.ws.rows, kb0, n,
                                  [&](int i, const auto& w) { return put(C::kWs, i, w); });
      else
        ok = feed_scales<F4, NT>(p.ts, (int64_t)tt * NT, min((int64_t)p.ts.rows, (int64_t)(tt + 1) * NT), kb0, n,
                                 [&](int i, const auto& w) { return put(C::kTs, i, w); });
    }
    if (!mbar_wait(&done, 0)) ok = false;
    __syncwarp();
    tmem_fence_after();
    const int q = warp & 3, row = 32 * q + lane;     // this warp's lanes of tensor memory
    // this CTA's sums into shared memory, in rows of out with four words between
    // them: [row of a][row of b], whichever of the two the 128 rows are
#pragma unroll 1
    for (int c = 0; c < NT; c += 16) {
      uint32_t v[16];
      tmem_ld16(v, tmem + ((uint32_t)(32 * q) << 16) + c);
      tmem_wait_ld(v);
      if (p.w_is_a) {
#pragma unroll
        for (int k = 0; k < 16; k += 4) st_shared16(smem + (row * (NT + 4) + c + k) * 4, v[k], v[k + 1], v[k + 2], v[k + 3]);
      } else {
#pragma unroll
        for (int k = 0; k < 16; ++k)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(smem + ((c + k) * 132 + row) * 4), "r"(v[k]) : "memory");
      }
    }
    tmem_fence_before();
  }
  if (!ok && lane == 0) atomicAdd(&g_mm_wait_timeouts, 1u);
  __syncwarp();
  // Each CTA of the cluster adds up its share of the rows, parts in order, four
  // neighbours of a row at a time and all parts' loads in flight together.
  if (p.splits > 1) cluster_barrier();
  else __syncthreads();
  const int inner = p.w_is_a ? NT : 128, outer = p.w_is_a ? 128 : NT;
  const int shift = p.w_is_a ? (NT == 16 ? 2 : NT == 32 ? 3 : NT == 64 ? 4 : 5) : 5, quads = 1 << shift;   // inner / 4
  const int o0 = outer * (int)rank / p.splits, o1 = outer * ((int)rank + 1) / p.splits;
  const int64_t m0 = p.w_is_a ? (int64_t)tw * 128 : (int64_t)tt * NT, n0 = p.w_is_a ? (int64_t)tt * NT : (int64_t)tw * 128;
  const int rows = (int)min((int64_t)outer, (p.w_is_a ? p.ws.rows : p.ts.rows) - m0);
  const int64_t cols = p.w_is_a ? p.ts.rows : p.ws.rows;
  const auto join = [&](auto parts) {
    constexpr int S = decltype(parts)::value, U = 8 / S;
    const int units = (min(o1, rows) - o0) * quads;
    for (int u0 = threadIdx.x; u0 < units; u0 += U * kSplitThreads) {
      float4 part[U][S];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int u = min(u0 + x * kSplitThreads, units - 1);
        const uint32_t at = smem + ((o0 + (u >> shift)) * (inner + 4) + (u & (quads - 1)) * 4) * 4;
#pragma unroll
        for (int s = 0; s < S; ++s)
          part[x][s] = S == 1                       ? load_shared4(at)
                       : S < 8 || s < p.splits ? cluster_load4(at, s)
                                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      float4 extra[U];                               // add may be out: before the first store
      if (p.add) {
#pragma unroll
        for (int x = 0; x < U; ++x) {
          const int u = u0 + x * kSplitThreads;
          const int64_t n = n0 + (u & (quads - 1)) * 4;
          if (u < units && n < cols) extra[x] = add4(p, m0 + o0 + (u >> shift), n, cols);
        }
      }
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int u = u0 + x * kSplitThreads;
        const int64_t n = n0 + (u & (quads - 1)) * 4;
        if (u >= units || n >= cols) continue;
#pragma unroll
        for (int s = 1; s < S; ++s) {
          part[x][0].x += part[x][s].x;
          part[x][0].y += part[x][s].y;
          part[x][0].z += part[x][s].z;
          part[x][0].w += part[x][s].w;
        }
        if (p.add) {
          part[x][0].x += extra[x].x;
          part[x][0].y += extra[x].y;
          part[x][0].z += extra[x].z;
          part[x][0].w += extra[x].w;
        }
        put4(p, m0 + o0 + (u >> shift), n, cols, part[x][0]);
      }
    }
  };
  // (forms for one, two, four and up to eight: a form for each costs small calls
  // 2 to 5%, for the code that they fetch)
  if (p.splits == 1) join(std::integral_constant<int, 1>());
  else if (p.splits == 2) join(std::integral_constant<int, 2>());
  else if (p.splits == 4) join(std::integral_constant<int, 4>());
  else join(std::integral_constant<int, 8>());
  if (p.splits > 1) cluster_barrier();               // nobody leaves while its part is read
  else __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    tmem_free(tmem, C::kColumns);
  }
}

// ---- large products: tiles of 256 x NT on pairs of SMs ----------------------------
//
// A cluster of two CTAs, one per SM and as many as there are SMs, goes over
// tiles of 256 rows of a and NT of b.  Each CTA loads half the rows of both, so
// that an SM reads 32 bytes of K of (128 + NT / 2) rows for 128 x NT sums: for
// NT = 256 64 bytes a cycle at the 4-bit rate, and one CTA by itself would read
// 96.  Sums stay in tensor memory, in two buffers (the scales have the last
// columns); where the two do not fit, they share some columns, which the
// epilogue reads first, so that the next tile's products start while the others
// are still being stored.
constexpr int kPairThreads = 288;          // TMA, products, four warps of epilogue, three of scales
constexpr int kPairBand = 8;               // tiles of a in a band: pairs in flight cover a compact block (4 and 16 no faster)

template <bool F4, int NT>
struct PairCfg {
  static constexpr int kB = 128 * 128;                             // codes of b within a stage
  static constexpr int kCodes = kB + NT / 2 * 128;
  static constexpr int kScaleA = F4 ? 1024 : 512, kScales = 3 * kScaleA;   // 128 rows of a, 256 of b
  static constexpr int kOut = 4096;                                // 32 rows x 128 bytes of out
  static constexpr int kBars = 256;
  static constexpr int kStages = (227 * 1024 - kBars - 4 * kOut) / (kCodes + kScales);
  static constexpr int kSmem = kStages * (kCodes + kScales) + 4 * kOut + kBars;
  // Tensor-memory columns of the scales of a K block, a buffer of them for each
  // stage or (where there is no room) two, and two buffers of sums.
  static constexpr int kSfB = F4 ? 8 : 4, kSf = 3 * kSfB, kSfBufs = NT <= 128 ? kStages : 2;
  static constexpr int kSums = NT <= 128 ? 256 : (512 - kSfBufs * kSf) / 32 * 32;
  static constexpr int kOver = 2 * NT > kSums ? 2 * NT - kSums : 0;
  static_assert(kSums + kSfBufs * kSf <= 512 && kCodes % 1024 == 0 && kOver % 32 == 0 && NT % 32 == 0 && NT <= 256 && kOver < NT && kSmem <= 227 * 1024, "");
};

// `chunks` times 32 columns of sums of 32 rows (row `lane` of the warp's lanes
// of tensor memory, at `from` on) into out, in fp32 or with ADD added; bar, where
// not 0, is told once they have left tensor memory.  LINES: all of it lies inside
// and its rows start at multiples of 16 bytes; the sums then pass through shared
// memory so that they leave in whole lines, four of a row at a time.  Otherwise
// a row's columns leave side by side.  add may be out: a chunk's values are read
// before any of it is stored, while its sums go to shared memory.
template <class T, bool ADD, bool LINES>
__device__ __forceinline__ void store_sums(uint32_t from, int chunks, uint32_t bar, uint32_t stage, T* out, int64_t stride,
                                           const T* add, int64_t add_stride, int rows, int width) {
  const int lane = threadIdx.x & 31;
  uint32_t mine[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) mine[k] = stage + lane * 128 + ((k ^ (lane & 7)) << 4);
  out += LINES ? (lane >> 3) * stride + 4 * (lane & 7) : lane;
  if (ADD) add += LINES ? (lane >> 3) * add_stride + 4 * (lane & 7) : lane;
  uint32_t x[32];
  const auto fetch = [&](int i, uint32_t (&to)[32]) {
    if (LINES) {
      const T* at = add + 32 * i;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (sizeof(T) == 4) {
          const uint4 t = *reinterpret_cast<const uint4*>(at);
          to[4 * k] = t.x, to[4 * k + 1] = t.y, to[4 * k + 2] = t.z, to[4 * k + 3] = t.w;
        } else {
          const uint2 t = *reinterpret_cast<const uint2*>(at);
          to[4 * k] = t.x << 16, to[4 * k + 1] = t.x & 0xFFFF0000u;
          to[4 * k + 2] = t.y << 16, to[4 * k + 3] = t.y & 0xFFFF0000u;
        }
        at += 4 * add_stride;
      }
    } else if (32 * i + lane < width && rows > 0) {
      const T* at = add + 32 * i;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        to[r] = sizeof(T) == 4 ? (uint32_t)*at : (uint32_t)*at << 16;
        at += r + 1 < rows ? add_stride : 0;         // past the last row: that one again
      }
    }
  };
#pragma unroll 1
  for (int i = 0; i < chunks; ++i) {
    if (ADD) fetch(i, x);
    {
      uint32_t v[32];
      tmem_ld32(v, from + 32 * i);
      tmem_wait_ld(v);
      if (i + 1 == chunks && bar) {
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(bar);
      }
      __syncwarp();                        // the chunk before has left shared memory
#pragma unroll
      for (int k = 0; k < 8; ++k) st_shared16(mine[k], v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
    __syncwarp();
    T* dst = out + 32 * i;
    if (LINES) {
      float4 t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = 4 * k + (lane >> 3);
        t[k] = load_shared4(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (ADD) {
          t[k].x += __uint_as_float(x[4 * k]);
          t[k].y += __uint_as_float(x[4 * k + 1]);
          t[k].z += __uint_as_float(x[4 * k + 2]);
          t[k].w += __uint_as_float(x[4 * k + 3]);
        }
        if constexpr (sizeof(T) == 4) *reinterpret_cast<float4*>(dst) = t[k];
        else *reinterpret_cast<uint2*>(dst) = make_uint2(cvt_bf16x2(t[k].x, t[k].y), cvt_bf16x2(t[k].z, t[k].w));
        dst += 4 * stride;
      }
    } else if (32 * i + lane < width) {
#pragma unroll
      for (int h = 0; h < 32; h += 16) {
        float v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r)
          asm volatile("ld.shared.f32 %0, [%1];"
                       : "=f"(v[r]) : "r"(stage + (h + r) * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4) : "memory");
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          if (ADD) v[r] += __uint_as_float(x[h + r]);
          if (h + r < rows) {
            if constexpr (sizeof(T) == 4) *dst = __float_as_uint(v[r]);
            else *dst = (uint16_t)cvt_bf16x2(v[r], v[r]);
          }
          dst += stride;
        }
      }
    }
  }
  __syncwarp();
}

// The form for anywhere as a function of its own, with registers of its own.
template <class T, bool ADD>
static __device__ __noinline__ void store_sums_anywhere(uint32_t from, int chunks, uint32_t bar, uint32_t stage, T* out,
                                                        int64_t stride, const T* add, int64_t add_stride, int rows,
                                                        int width) {
  store_sums<T, ADD, false>(from, chunks, bar, stage, out, stride, add, add_stride, rows, width);
}

// `chunks` times 32 columns of bf16 whose rows start anywhere, or at the edges
// of out, from tensor memory at `from` on; bar, where not 0, is told once they
// have left it.  Row `lane` passes through shared memory as far past a multiple
// of 16 bytes as it lies in out, so that its 16-byte pieces leave whole, what is
// left of a chunk with the next one; the elements before the first piece and
// behind the last leave in two or three stores: 8192 x 8190 x 512 in 4 bits 56 us
// (66 with the ends element by element and each chunk waited for), 8192 columns,
// whole lines, 31.  (One warp per scheduler: its
// instructions count.  Moving rows in registers instead, without conflicts in
// shared memory, takes twice the selects that this takes stores; multiples of 32
// bytes, for whole sectors, three times.  fp32 is done sooner column by column,
// in store_sums: 3830 x 11557 x 128 in 8 bits 55 us, by pieces 60 to 74.)
static __device__ __noinline__ void store_anywhere(uint32_t from, int chunks, uint32_t bar, uint32_t stage, uint16_t* out,
                                                   int64_t stride, int rows, int width) {
  const int lane = threadIdx.x & 31;
  // in elements, and only the low bits count
  const uint32_t start = (uint32_t)(reinterpret_cast<uintptr_t>(out) >> 1), step = (uint32_t)stride;
  const uint32_t phase = (start + lane * step) & 7u, odd = 16 * (phase & 1);
  const uint32_t row = stage + lane * 80, to = row + (phase >> 1) * 4;
  uint16_t* const mine = out + lane * stride - (int)phase;           // piece 0 of the first chunk
  uint32_t before = 0;
  uint32_t v[32];
  tmem_ld32(v, from);
  tmem_wait_ld(v);
#pragma unroll 1
  for (int i = 0; i < chunks; ++i) {
    uint32_t h[17];
#pragma unroll
    for (int k = 0; k < 16; ++k) h[k] = cvt_bf16x2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
    h[16] = 0;
    if (i + 1 < chunks) {
      tmem_ld32(v, from + 32 * (i + 1));                             // on its way meanwhile
    } else if (bar) {
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(bar);
    }
    if (rows > 0 && 32 * i < width) {
      __syncwarp();
      if (i) {                             // what the chunk before left
        const float4 left = load_shared4(row + 64);
        st_shared16(row, __float_as_uint(left.x), __float_as_uint(left.y), __float_as_uint(left.z), __float_as_uint(left.w));
      }
#pragma unroll
      for (int k = 0; k < 17; ++k)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + 4 * k), "r"(__funnelshift_l(k ? h[k ? k - 1 : 0] : before, h[k], odd))
                     : "memory");
      before = h[15];
      __syncwarp();
      const int held = min(32, width - 32 * i);      // columns of this chunk
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = 8 * x + (lane >> 2), j = lane & 3;
        const float4 t = load_shared4(stage + r * 80 + j * 16);
        const int moved = (int)((start + r * step) & 7u);
        if (r < rows && (i > 0 || j > 0 || moved == 0) && 8 * j + 8 <= moved + held)
          *reinterpret_cast<float4*>(out + r * stride + 32 * i + 8 * j - moved) = t;
      }
      const int end = (int)phase + held;             // of what the row holds
      const bool within = i == 0 && phase && end < 8;
      if (i == 0 && phase && lane < rows) {          // before the first whole piece
        const float4 t = load_shared4(row);
        const uint32_t w[4] = {__float_as_uint(t.x), __float_as_uint(t.y), __float_as_uint(t.z), __float_as_uint(t.w)};
        if (within) {
#pragma unroll
          for (int e = 1; e < 7; ++e)
            if (e >= (int)phase && e < end) mine[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        } else {
          const int two = (phase + 1) & ~1, four = (two + 2) & ~3;   // where 4 bytes start, and 8
          if (phase & 1) mine[phase] = (uint16_t)((phase < 4 ? phase < 2 ? w[0] : w[1] : phase < 6 ? w[2] : w[3]) >> 16);
          if (two & 2) *reinterpret_cast<uint32_t*>(mine + two) = two == 2 ? w[1] : w[3];
          if (four == 4) *reinterpret_cast<uint2*>(mine + 4) = make_uint2(w[2], w[3]);
        }
      }
      if ((i + 1 == chunks || held < 32 || 32 * i + 32 == width) && lane < rows && !within) {     // behind the last one
        const int k = end >> 3, n = end & 7;
        const float4 t = load_shared4(row + 16 * k);
        const uint32_t w[4] = {__float_as_uint(t.x), __float_as_uint(t.y), __float_as_uint(t.z), __float_as_uint(t.w)};
        uint16_t* const at = mine + 32 * i + 8 * k;
        if (n & 4) *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
        if (n & 2) *reinterpret_cast<uint32_t*>(at + (n & 4)) = n & 4 ? w[2] : w[0];
        if (n & 1) at[n - 1] = (uint16_t)(n & 4 ? n & 2 ? w[3] : w[2] : n & 2 ? w[1] : w[0]);
      }
    }
    if (i + 1 < chunks) tmem_wait_ld(v);
  }
  __syncwarp();
}

template <bool F4, int NT, MmOut OUT>
__global__ void __launch_bounds__(kPairThreads, 1) mm_pair_kernel(const __grid_constant__ MmArgs p) {
  using C = PairCfg<F4, NT>;
  constexpr int ST = C::kStages;
  // all of the SM's shared memory: no room to align within it, and nothing static
  extern __shared__ __align__(1024) uint8_t pair_smem[];
  const uint32_t smem = uniform(smem_addr(pair_smem));
  const uint32_t staging = smem + ST * C::kCodes, scales = staging + 4 * C::kOut;
  uint64_t* const full = reinterpret_cast<uint64_t*>(pair_smem + C::kSmem - C::kBars);
  uint64_t *const empty = full + ST, *const sums_full = empty + ST, *const sums_empty = sums_full + 2,
           *const shared_empty = sums_empty + 2;
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(shared_empty + 1);
  static_assert(8 * (2 * ST + 5) + 4 <= C::kBars, "barriers");
  if (smem & 1023u) {                      // the swizzle's tiles start at multiples of 1024; nothing has begun yet
    if (threadIdx.x == 0) atomicAdd(&g_mm_wait_timeouts, 1u);
    return;
  }
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1 + 6);          // the even CTA's: bytes of both, and both CTAs' scales
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sums_full[i], 1);
      mbar_init(&sums_empty[i], 8);        // the even CTA's: both epilogues
    }
    mbar_init(shared_empty, 8);
    fence_barrier_init();
    prefetch_tensormap(&p.w);
    prefetch_tensormap(&p.t);
    if (OUT == MmOut::kTma) prefetch_tensormap(&p.o);
  }
  __syncwarp();
  cluster_barrier();                       // the other CTA's barriers are there
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 1) tmem_alloc_pair(s_tmem, 512);
  // The next grid may be set up from here on, whether or not there is tensor memory
  // yet: no CTA finds room in shared memory beside one of this kernel, and the
  // kernels here that take tensor memory wait for the grid before them first.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tmem_fence_before();
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  // both CTAs have their tensor memory; the loads of codes do not wait for it
  const auto wait_for_tmem = [&] {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    tmem_fence_after();
    return uniform(*s_tmem);
  };
  uint32_t tmem = 0;
  if (warp != 0) tmem = wait_for_tmem();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = p.w_tiles * p.t_tiles;
  const auto place = [&](int tile, int* tw, int* tt) {
    const int band = tile / (kPairBand * p.t_tiles), in = tile - band * (kPairBand * p.t_tiles);
    const int height = min(kPairBand, p.w_tiles - band * kPairBand);
    *tt = in / height;
    *tw = band * kPairBand + in - *tt * height;
  };
  bool ok = true;

  if (warp == 0) {
    int st = 0, phase = 1;                 // a stage's first fill waits for nothing
    for (int tile = pair; tile < tiles && ok; tile += pairs) {
      int tw, tt;
      place(tile, &tw, &tt);
      for (int i = 0; i < p.kblocks; ++i) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], phase))) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * C::kCodes);
          const uint32_t bar = lead_bar(&full[st]), at = smem + st * C::kCodes;
          tma_load_2d_pair(at, &p.w, bar, i * 128, tw * 256 + (int)rank * 128);
          tma_load_2d_pair(at + C::kB, &p.t, bar, i * 128, tt * NT + (int)rank * (NT / 2));
        }
        __syncwarp();
        if (++st == ST) {
          st = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t hi = desc_hi(1024);
      const int own = tiles > pair ? (tiles - pair - 1) / pairs + 1 : 0, total = own * p.kblocks;
      // A block's scales are copied into the buffer of an earlier block, whose
      // products have to be done: products wait for the copies issued before
      // them, but a copy need not wait for products that still read its buffer.
      // With a buffer for each stage the stage's new contents tell that, and they
      // are copied ahead of the block before.  With two the products are waited
      // for, and the copies follow the block before (ahead of it the tensor cores
      // run dry: 8192 x 8192 x 8192 in 4 bits 167 -> 239 us); for the short
      // blocks of 128 columns the wait alone cost 512 x 2048 x 8192 12.0 -> 13.7.
      constexpr int NB = C::kSfBufs;
      int cst = 0, cphase = 0, dst = 0, dphase = 0;
      const auto copy = [&](int it) {
        if (NB < ST && it >= NB) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[dst], dphase))) return false;
          if (++dst == ST) {
            dst = 0;
            dphase ^= 1;
          }
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[cst], cphase))) return false;
        tmem_fence_after();
        const uint32_t from = scales + cst * C::kScales, to = tmem + C::kSums + (NB == ST ? cst : it & 1) * C::kSf;
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < (F4 ? 2 : 1); ++c) {
            sf_copy<2>(to + 4 * c, sf_desc(from + 512 * c));
            sf_copy<2>(to + C::kSfB + 8 * c, sf_desc(from + C::kScaleA + 1024 * c));
            sf_copy<2>(to + C::kSfB + 8 * c + 4, sf_desc(from + C::kScaleA + 1024 * c + 512));
          }
        }
        __syncwarp();
        if (++cst == ST) {
          cst = 0;
          cphase ^= 1;
        }
        return true;
      };
      if (total) ok = copy(0);
      int it = 0, st = 0;
      for (int lt = 0; lt < own && ok; ++lt) {
        const int b = lt & 1;
        const uint32_t d = tmem + (b ? C::kSums - NT : 0);
        if (lt >= 2 && !mbar_wait(&sums_empty[b], (lt / 2 - 1) & 1)) ok = false;
        if (C::kOver && lt >= 1 && !mbar_wait(shared_empty, (lt - 1) & 1)) ok = false;
        ok = __all_sync(0xFFFFFFFFu, ok);
        tmem_fence_after();
        for (int i = 0; i < p.kblocks && ok; ++i, ++it) {
          if (NB == ST && it + 1 < total) ok = copy(it + 1);
          if (!ok) break;
          const uint32_t at = smem + st * C::kCodes, sf = tmem + C::kSums + (NB == ST ? st : it & 1) * C::kSf;
          const uint32_t a_lo = desc_lo(at, 16), b_lo = desc_lo(at + C::kB, 16);
          if (elect_one()) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_mx<F4, 2>(d, a_lo + 2 * s, b_lo + 2 * s, hi, mx_idesc_step<F4>(p.idesc, F4 ? s & 1 : s),
                            sf + (F4 ? 4 * (s >> 1) : 0), sf + C::kSfB + (F4 ? 8 * (s >> 1) : 0), i > 0 || s > 0);
            mma_commit_pair(&empty[st]);
            if (i + 1 == p.kblocks) mma_commit_pair(&sums_full[b]);
          }
          __syncwarp();
          if (++st == ST) st = 0;
          if (NB < ST && it + 1 < total) ok = copy(it + 1);
        }
        if (!ok) {                         // for the epilogue, which waits
          if (elect_one()) mma_commit_pair(&sums_full[b]);
          __syncwarp();
        }
      }
    }
  } else if (warp < 6) {
    const int q = warp & 3;                          // this warp's lanes of tensor memory: 32 q on
    const uint32_t lane_at = tmem + ((uint32_t)(32 * q) << 16);
    const uint32_t stage = staging + (warp - 2) * C::kOut;
    const int64_t cols = p.ts.rows;
    int lt = 0;
    for (int tile = pair; tile < tiles; tile += pairs, ++lt) {
      int tw, tt;
      place(tile, &tw, &tt);
      const int b = lt & 1;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sums_full[b], (lt / 2) & 1))) {
        ok = false;
        break;
      }
      tmem_fence_after();
      const int64_t m0 = (int64_t)tw * 256 + rank * 128 + 32 * q, n0 = (int64_t)tt * NT;
      const int rows = (int)min((int64_t)32, p.ws.rows - m0);      // may be none
      const uint32_t from = lane_at + (b ? C::kSums - NT : 0);
      if constexpr (OUT == MmOut::kTma) {
        // 64 columns of bf16, or 32 of fp32, at a time: two boxes of 64 bytes a
        // row; the columns after them leave tensor memory meanwhile.  One fence
        // and one wait for both boxes: each costs the warp hundreds of cycles.
        const bool down = C::kOver && !b;      // shared columns first: the last ones of the first buffer
        const int sw = (lane >> 1) & 3;
        const auto box = [&](uint32_t to, const uint32_t (&w)[16]) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            st_shared16(to + lane * 64 + ((k ^ sw) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        };
        const auto pack = [](const uint32_t (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = cvt_bf16x2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
        };
        const int most = p.fp32 ? 32 : 64;
        uint32_t v[32], u[32], w[16];
        int c = down ? NT - 32 : 0;
        tmem_ld32(v, from + c);
        tmem_wait_ld(v);
#pragma unroll 1
        for (int x = 0; x < NT;) {
          // v: columns c .. c + 31; u: the next 32, up or down
          const int width = min(most, NT - x), c2 = down ? c - 32 : c + 32;
          if (width == 64) tmem_ld32(u, from + c2);
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          if (p.fp32) {
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = v[k];
            box(stage, w);
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = v[16 + k];
            box(stage + C::kOut / 2, w);
          } else {
            pack(v, w);
            box(stage, w);
          }
          if (width == 64) tmem_wait_ld(u);
          const bool shared_done = C::kOver && x < C::kOver && x + width >= C::kOver;
          x += width;
          if (shared_done || x == NT) {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(lead_bar(x == NT ? &sums_empty[b] : shared_empty));
          }
          const int c_next = down ? c - width : c + width;
          if (x < NT) tmem_ld32(v, from + c_next);
          if (width == 64) {
            pack(u, w);
            box(stage + C::kOut / 2, w);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            const int64_t n = n0 + c, n2 = p.fp32 ? n + 16 : n0 + c2;
            if (rows > 0 && n < cols) tma_store_2d_from(&p.o, stage, (int)n, (int)m0);
            if (rows > 0 && n2 < cols && (p.fp32 || width == 64))
              tma_store_2d_from(&p.o, stage + C::kOut / 2, (int)n2, (int)m0);
            bulk_commit();
          }
          if (x < NT) tmem_wait_ld(v);
          c = c_next;
        }
        continue;
      }
      // inside, and rows of whole 16-byte pieces
      const bool lines = rows == 32 && n0 + NT <= cols && p.out_vector && (!p.add || p.add_vector);
      if (OUT != MmOut::kBf16 || !lines) {
        // two parts: the columns that the other buffer shares first
#pragma unroll 1
        for (int part = C::kOver ? 0 : 1; part < 2; ++part) {
          const int c = (part == 0) == (b != 0) ? 0 : b ? C::kOver : part ? 0 : NT - C::kOver;
          const int n = part ? NT - C::kOver : C::kOver;
          const uint32_t bar = lead_bar(part ? &sums_empty[b] : shared_empty);
          const int64_t at = m0 * p.out_stride + n0 + c, add_at = m0 * p.add_stride + n0 + c;
          const int width = (int)max((int64_t)0, min((int64_t)n, cols - n0 - c));
          if constexpr (OUT == MmOut::kBf16)
            store_anywhere(from + c, n / 32, bar, stage, static_cast<uint16_t*>(p.out) + at, p.out_stride, rows, width);
          else if constexpr (OUT != MmOut::kTma) {
            using T = std::conditional_t<OUT == MmOut::kAddBf16, uint16_t, uint32_t>;
            constexpr bool ADD = OUT != MmOut::kF32;
            T* const out = static_cast<T*>(p.out) + at;
            const T* const add = ADD ? static_cast<const T*>(p.add) + add_at : nullptr;
            if (lines) store_sums<T, ADD, true>(from + c, n / 32, bar, stage, out, p.out_stride, add, p.add_stride, rows, width);
            else store_sums_anywhere<T, ADD>(from + c, n / 32, bar, stage, out, p.out_stride, add, p.add_stride, rows, width);
          }
        }
        continue;
      }
      if constexpr (OUT == MmOut::kBf16) {
        // 128 bytes of 32 rows pass through shared memory, swizzled: chunk k of row
        // `lane`; chunk lane % 8 of rows 4 i + lane / 8, i even or odd
        uint32_t mine[8], theirs[2];
#pragma unroll
        for (int k = 0; k < 8; ++k) mine[k] = stage + lane * 128 + ((k ^ (lane & 7)) << 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) theirs[k] = stage + (lane >> 3) * 128 + (((lane & 7) ^ (4 * k + (lane >> 3))) << 4);
#pragma unroll 1
        for (int x = 0; x < NT;) {
          const int w = min(64, NT - x);
          // the columns that the other buffer shares first: the last ones of the first, the first of the second
          const int c = C::kOver && !b ? NT - w - x : x;
          uint32_t v[32], u[32];
          tmem_ld32(v, from + c);
          if (w == 64) tmem_ld32(u, from + c + 32);
          tmem_wait_ld(v);
          tmem_wait_ld(u);
          const bool shared_done = C::kOver && x < C::kOver && x + w >= C::kOver;
          x += w;
          if (shared_done || x == NT) {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(lead_bar(x == NT ? &sums_empty[b] : shared_empty));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[4], g[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              h[z] = cvt_bf16x2(__uint_as_float(v[8 * k + 2 * z]), __uint_as_float(v[8 * k + 2 * z + 1]));
              g[z] = cvt_bf16x2(__uint_as_float(u[8 * k + 2 * z]), __uint_as_float(u[8 * k + 2 * z + 1]));
            }
            st_shared16(mine[k], h[0], h[1], h[2], h[3]);
            st_shared16(mine[k + 4], g[0], g[1], g[2], g[3]);        // not read where there are 32 columns
          }
          __syncwarp();
          uint16_t* const dst = static_cast<uint16_t*>(p.out) + m0 * p.out_stride + n0 + c;
          if (w == 64) {
            // whole lines: 16 bytes of row 4 i + lane / 8 at a time
            uint16_t* at = dst + (lane >> 3) * p.out_stride + (lane & 7) * 8;
            float4 t[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = load_shared4(theirs[i & 1] + 512 * i);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              *reinterpret_cast<float4*>(at) = t[i];
              at += 4 * p.out_stride;
            }
          } else {
            // half lines: of row 8 i + lane / 4
            uint16_t* at = dst + (lane >> 2) * p.out_stride + (lane & 3) * 8;
            float4 t[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              t[i] = load_shared4(stage + (8 * i + (lane >> 2)) * 128 + (((lane & 3) ^ (lane >> 2)) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              *reinterpret_cast<float4*>(at) = t[i];
              at += 8 * p.out_stride;
            }
          }
          __syncwarp();
        }
      }
    }
    if (OUT == MmOut::kTma && lane == 0) bulk_wait_all();
    __syncwarp();
  } else {
    // warp 6 brings the scales of 128 rows of a, warps 7 and 8 of 128 rows of b each
    const int part = warp - 6;
    const uint32_t to = scales + (part == 0 ? 0 : C::kScaleA + (part - 1) * 512) + lane * 16;
    const uint32_t pitch = part == 0 ? 512 : 1024;
    int st = 0, phase = 1;
    const auto put = [&](int, const auto& w) {
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[st], phase))) return false;
      const uint32_t at = to + st * C::kScales;
#pragma unroll
      for (int c = 0; c < (F4 ? 2 : 1); ++c) st_shared16(at + c * pitch, w[c][0], w[c][1], w[c][2], w[c][3]);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead_bar(&full[st]));
      if (++st == ST) {
        st = 0;
        phase ^= 1;
      }
      return true;
    };
    const MmScales& sc = part == 0 ? p.ws : p.ts;
    const auto first_row = [&](int tile) {
      int tw, tt;
      place(tile, &tw, &tt);
      return part == 0 ? (int64_t)tw * 256 + rank * 128 : (int64_t)tt * NT + (part - 1) * 128;
    };
    if (sc.sectors) {
      // rows of whole sectors: the next group's are on their way meanwhile, the next tile's too
      constexpr int W = F4 ? 2 : 1, G = 8 / W;
      const uint8_t* base[4];
      uint32_t g[4][8], next[4][8];
      const auto open = [&](int tile) {
        const int64_t row = first_row(min(tile, tiles - 1)) + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          base[j] = tile < tiles && row + 32 * j < sc.rows ? sc.e8m0 + (row + 32 * j) * sc.stride : nullptr;
      };
      const auto load = [&](int at, uint32_t (&v)[4][8]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) load_sector(base[j] && at < sc.bytes ? base[j] + at : nullptr, v[j]);
      };
      open(pair);
      load(0, g);
      for (int tile = pair; tile < tiles && ok; tile += pairs) {
#pragma unroll 1
        for (int i = 0; i < p.kblocks && ok; i += G) {
          if (i + G >= p.kblocks) open(tile + pairs);
          load(i + G >= p.kblocks ? 0 : (i + G) * 4 * W, next);
#pragma unroll
          for (int b = 0; b < G; ++b) {
            if (i + b >= p.kblocks) break;
            uint32_t words[W][4];
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
              for (int j = 0; j < 4; ++j) words[w][j] = g[j][W * b + w];
            ok = put(i + b, words);
            if (!ok) break;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) g[j][k] = next[j][k];
        }
      }
    } else {
      for (int tile = pair; tile < tiles && ok; tile += pairs)
        ok = feed_scales<F4, 128>(sc, first_row(tile), sc.rows, 0, p.kblocks, put);
    }
  }
  if (!ok) {
    // loads in flight land (within microseconds) before the CTAs leave
    if (lane == 0) atomicAdd(&g_mm_wait_timeouts, 1u);
    const long long until = clock64() + (1ll << 24);
    while (clock64() < until) __nanosleep(1000);
  }
  __syncwarp();
  if (warp == 0) tmem = wait_for_tmem();
  tmem_fence_before();
  cluster_barrier();                       // barriers and shared memory are no longer used by the other CTA
  if (warp == 1) {
    tmem_fence_after();
    tmem_free_pair(tmem, 512);
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
// Tensor map of out: boxes of 32 rows x 64 bytes, 64-byte swizzle.
static cudaError_t encode_out(CUtensorMap* map, const MxProduct& p) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  const int size = p.fp32 ? 4 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)p.b.rows, (cuuint64_t)p.a.rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(p.out_stride * size)};
  const cuuint32_t shape[2] = {64u / size, 32u}, step[2] = {1u, 1u};
  return encode(map, p.fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.out, dims, strides,
                shape, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}
static MmScales scales_of(const MxView& m) {
  MmScales s;
  s.e8m0 = m.e8m0;
  s.stride = m.e_stride;
  s.rows = (int32_t)m.rows;
  s.bytes = (int32_t)(m.cols / 32);
  s.sectors = (reinterpret_cast<uintptr_t>(m.e8m0) | (uintptr_t)m.e_stride | (uintptr_t)s.bytes) % 32 == 0;
  return s;
}

static cudaError_t set_args(MmArgs* a, const MxProduct& p, const MxView& w, const MxView& t, int w_box, int t_box) {
  cudaError_t e = encode_codes(&a->w, w, w_box);
  if (e == cudaSuccess) e = encode_codes(&a->t, t, t_box);
  a->ws = scales_of(w);
  a->ts = scales_of(t);
  a->kblocks = (int32_t)((w.row_bytes() + 127) / 128);
  a->out = p.out;
  a->add = p.add;
  a->out_stride = p.out_stride;
  a->add_stride = p.add_stride;
  a->fp32 = p.fp32;
  const int size = p.fp32 ? 4 : 2;
  const uintptr_t out = reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_stride * size);
  const uintptr_t add = reinterpret_cast<uintptr_t>(p.add) | (uintptr_t)(p.add_stride * size);
  a->out_quads = out % (4 * size) == 0;
  a->add_quads = add % (4 * size) == 0;
  a->out_vector = out % 16 == 0;
  a->add_vector = add % 16 == 0;
  return e;
}
static cudaError_t launch_clusters(const void* kern, MmArgs& a, int64_t ctas, int cluster, int threads, int smem,
                                   cudaStream_t s, int* launches) {
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  void* args[] = {&a};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, kern, args);
  if (e == cudaSuccess) ++*launches;
  return e;
}

// SMs of the current device; without a GPU, where the launch will say so, a pair.
static int64_t sms_or_a_pair() { return std::max(2, sm_count(device_of_current())); }

template <bool F4, int NT>
static cudaError_t launch_split(const MxProduct& p, const MmPlan& plan, cudaStream_t s, int* launches) {
  using C = SplitCfg<F4, NT>;
  const MxView &w = plan.w_is_a ? p.a : p.b, &t = plan.w_is_a ? p.b : p.a;
  const void* kern = reinterpret_cast<const void*>(mm_split_kernel<F4, NT>);
  int occ = 1;
  cudaError_t e = kernel_occupancy(kern, kSplitThreads, C::kSmem, &occ);
  if (e != cudaSuccess) return e;
  MmArgs a;
  if ((e = set_args(&a, p, w, t, 128, NT)) != cudaSuccess) return e;
  a.w_tiles = (int32_t)((w.rows + 127) / 128);
  a.t_tiles = (int32_t)((t.rows + NT - 1) / NT);
  a.splits = plan.splits;
  a.idesc = mx_idesc(F4, w.format, t.format, 128, NT);
  a.w_is_a = plan.w_is_a;
  return launch_clusters(kern, a, plan.tiles * plan.splits, plan.splits, kSplitThreads, C::kSmem, s, launches);
}

template <bool F4, int NT, MmOut OUT>
static cudaError_t launch_pair(const MxProduct& p, const MmPlan& plan, cudaStream_t s, int* launches) {
  using C = PairCfg<F4, NT>;
  const void* kern = reinterpret_cast<const void*>(mm_pair_kernel<F4, NT, OUT>);
  int occ = 1;
  cudaError_t e = kernel_occupancy(kern, kPairThreads, C::kSmem, &occ);
  if (e != cudaSuccess) return e;
  MmArgs a;
  if ((e = set_args(&a, p, p.a, p.b, 128, NT / 2)) != cudaSuccess) return e;
  a.w_tiles = (int32_t)((p.a.rows + 255) / 256);
  a.t_tiles = (int32_t)((p.b.rows + NT - 1) / NT);
  const int64_t tiles = plan.tiles;
  if (tiles > (1 << 27)) return cudaErrorInvalidValue;          // 32-bit tile counts
  a.splits = 1;
  a.idesc = mx_idesc(F4, p.a.format, p.b.format, 256, NT);
  a.w_is_a = 1;
  const int64_t pairs = sms_or_a_pair() / 2;
  if (OUT == MmOut::kTma && (e = encode_out(&a.o, p)) != cudaSuccess) return e;
  return launch_clusters(kern, a, 2 * (tiles < pairs ? tiles : pairs), 2, kPairThreads, C::kSmem, s, launches);
}

template <bool F4, int NT>
static cudaError_t launch_pair_out(const MxProduct& p, const MmPlan& plan, cudaStream_t s, int* launches) {
  switch (plan.out) {
    case MmOut::kTma: return launch_pair<F4, NT, MmOut::kTma>(p, plan, s, launches);
    case MmOut::kBf16: return launch_pair<F4, NT, MmOut::kBf16>(p, plan, s, launches);
    case MmOut::kF32: return launch_pair<F4, NT, MmOut::kF32>(p, plan, s, launches);
    case MmOut::kAddBf16: return launch_pair<F4, NT, MmOut::kAddBf16>(p, plan, s, launches);
    default: return launch_pair<F4, NT, MmOut::kAddF32>(p, plan, s, launches);
  }
}

template <bool F4>
static cudaError_t launch_format(const MxProduct& p, cudaStream_t s, int* launches) {
  const MmPlan plan = plan_product(p, sms_or_a_pair());
  if (!plan.pair)
    return plan.columns == 16   ? launch_split<F4, 16>(p, plan, s, launches)
           : plan.columns == 32 ? launch_split<F4, 32>(p, plan, s, launches)
                                : launch_split<F4, 64>(p, plan, s, launches);
  if (plan.columns == 128) return launch_pair_out<F4, 128>(p, plan, s, launches);
  // 224 columns leave in two ways (see plan_pair)
  if (plan.columns == 224)
    return plan.out == MmOut::kTma ? launch_pair<F4, 224, MmOut::kTma>(p, plan, s, launches)
                                   : launch_pair<F4, 224, MmOut::kAddF32>(p, plan, s, launches);
  return launch_pair_out<F4, 256>(p, plan, s, launches);
}

}  // namespace fp8q
