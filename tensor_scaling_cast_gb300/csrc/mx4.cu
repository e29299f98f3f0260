// MX casts to 4 bits (E2M1, two codes per byte, the even element in the low
// half): row by row, and the dual cast that writes the transpose's blocks from
// the same read.
//
// Rows: a unit is eight elements (16 bytes of bf16 in, 4 bytes of codes out),
// four neighbouring lanes hold one block and share its maximum by two shuffles.
// Bound by HBM: 2.53 bytes per bf16 element, 16384 x 8192 in 53.4 us (6.4 TB/s).
#include <cuda.h>
#include <cuda_runtime.h>

#include "mx_linear.cuh"
#include "tma.cuh"
#include "warp_tiles.cuh"

namespace fp8q {

constexpr int kMx4Ahead = 4;       // units a thread has in flight

template <int DT>
__global__ void __launch_bounds__(kUnitThreads) mx4_rows_kernel(const void* __restrict__ x, int64_t units,
                                                                uint8_t* __restrict__ q, uint8_t* __restrict__ e8m0,
                                                                unsigned long long* clipped, int headroom, int rule) {
  constexpr int U = kMx4Ahead;
  __shared__ uint32_t red[kUnitThreads / 32];
  grid_begin();
  const int64_t i0 = (int64_t)blockIdx.x * (U * kUnitThreads) + threadIdx.x;
  Plain8<DT> v[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t i = i0 + j * kUnitThreads;
    v[j] = i < units ? load8<DT>(x, i * 8) : zero8<DT>();
  }
  uint32_t clip = 0;
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int64_t i = i0 + j * kUnitThreads;
    const uint32_t m = block_max4(absmax8<DT>(v[j]));
    uint32_t ebyte, o;
    if (m >= 0x7F800000u) {
      uint32_t signs = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) signs |= (bits8<DT>(v[j], k) >> 31) << k;
      o = nonfinite8<FP8Q_E2M1>(signs).x;
      ebyte = 255u;
    } else {
      const int E = block_exp<FP8Q_E2M1>(m, rule, headroom);
      const float s = block_inv_scale<FP8Q_E2M1>(E);
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(bits8<DT>(v[j], k)) * s;
      o = cvt_e2m1x8(f);
      ebyte = (uint32_t)(E + 127);
      if (clipped && mx_block_may_clip<FP8Q_E2M1>(m, E)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) clip += clips<FP8Q_E2M1>(f[k]) ? 1u : 0u;
      }
    }
    if (i < units) {
      __stcs(reinterpret_cast<uint32_t*>(q + i * 4), o);
      if ((threadIdx.x & 3) == 0) e8m0[i >> 2] = (uint8_t)ebyte;
    }
  }
  if (clipped) {
    clip = __reduce_add_sync(0xFFFFFFFFu, clip);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = clip;
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long total = 0;
      for (int w = 0; w < kUnitThreads / 32; ++w) total += red[w];
      if (total) atomicAdd(clipped, total);
    }
  }
}

cudaError_t launch_mx4_rows(const void* x, int dtype, int64_t nelem, int headroom, int rule, uint8_t* q, uint8_t* e8m0,
                            unsigned long long* clipped, cudaStream_t s, int* launches) {
  int64_t units = nelem / 8;
  const int64_t grid = (units + kUnitThreads * kMx4Ahead - 1) / (kUnitThreads * kMx4Ahead);
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  void* args[] = {&x, &units, &q, &e8m0, &clipped, &headroom, &rule};
  return launch_dependent(dtype == FP8Q_BF16 ? reinterpret_cast<const void*>(mx4_rows_kernel<FP8Q_BF16>)
                                             : reinterpret_cast<const void*>(mx4_rows_kernel<FP8Q_F32>),
                          dim3((unsigned)grid), kUnitThreads, 0, args, s, launches);
}

// ---- dual ---------------------------------------------------------------------
//
// The per-warp TMA pipeline of warp_tiles.cuh over 32-row x 128-byte sub-tiles,
// as the 8-bit dual cast runs it: lane l casts row l (its blocks of the
// row-wise form) and then columns 2l, 2l + 1 (bf16) or l (fp32), whose 32 rows
// are one block of the transpose.  A block's codes are 16 bytes, half a memory
// sector, so two row tiles' transposed blocks are gathered in shared memory
// into 32-byte rows before they go out.  16384 x 8192 bf16 in 67.7 us (6.1 TB/s
// of 3.06 bytes an element): HBM, and issue slots, half of which are in use; the
// sixteen warps of one CTA per SM keep its tiles side by side (12 and 14 warps
// were slower).

// A warp's output: two row tiles of up to 64 columns' transposed codes, and one
// row tile's row-wise ones.
constexpr int kMx4OutBytes = 64 * 32 + 32 * 32;
template <bool COUNT>
using Mx4DualCfg = TpCfg<2, 1, 4, true, kMx4OutBytes, 1, COUNT, 16, COUNT>;
constexpr int kMx4SmallMore = 27;          // percent a sub-tile, see tp_small
// Few sub-tiles: chunks of two row tiles and CTAs of two warps, so that every SM
// has some (see tp_small).
template <bool COUNT>
using Mx4DualSmallCfg = TpCfg<2, 1, 2, true, kMx4OutBytes, 0, COUNT, 2, COUNT>;

static __device__ unsigned int g_mx4_wait_timeouts;   // see fp8q_pipeline_status

cudaError_t read_mx4_wait_timeouts(unsigned int* count) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(count, g_mx4_wait_timeouts, sizeof(unsigned int));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_mx4_wait_timeouts, &zero, sizeof(unsigned int));
  return e;
}

// One block from the fp32 bits of its 32 elements: its codes into o, returns
// its E8M0 byte and adds its clipped elements to clip.
template <bool COUNT, class Bits>
__device__ __forceinline__ uint32_t mx4_block(Bits bits, uint32_t m, int rule, int headroom, uint32_t& clip,
                                              uint32_t (&o)[4]) {
  if (m >= 0x7F800000u) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      uint32_t signs = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) signs |= (bits(8 * g + k) >> 31) << k;
      o[g] = nonfinite8<FP8Q_E2M1>(signs).x;
    }
    return 255u;
  }
  const int E = block_exp<FP8Q_E2M1>(m, rule, headroom);
  const float s = block_inv_scale<FP8Q_E2M1>(E);
  const bool count = COUNT && mx_block_may_clip<FP8Q_E2M1>(m, E);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(bits(8 * g + k)) * s;
    o[g] = cvt_e2m1x8(f);
    if (count) {
#pragma unroll
      for (int k = 0; k < 8; ++k) clip += clips<FP8Q_E2M1>(f[k]) ? 1u : 0u;
    }
  }
  return (uint32_t)(E + 127);
}

template <int DT, class C>
__global__ void __launch_bounds__(C::kThreads, C::kMinBlocks) mx4_dual_kernel(
    const __grid_constant__ CUtensorMap tmap, const __grid_constant__ CUtensorMap qmap,
    const __grid_constant__ CUtensorMap qtmap, int64_t rows, int64_t cols, int rule, int headroom,
    uint8_t* __restrict__ q_colt, uint8_t* __restrict__ e8_row, uint8_t* __restrict__ e8_colt,
    unsigned long long* clipped_row, unsigned long long* clipped_col) {
  using G = TileGeom<DT>;
  constexpr int EPL = G::EPL, TILE_C = G::TILE_C, NG = G::NG;
  static_assert(C::kOutBufs == 1, "the transposed part outlives a sub-tile");
  static_assert(C::kChunk % 2 == 0, "pairs of row tiles start on even ones");
  extern __shared__ __align__(1024) uint4 dyn_smem[];
  __shared__ __align__(8) uint64_t full[C::kWarps][C::kStages];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t ctiles = (uint32_t)((cols + TILE_C - 1) / TILE_C);
  uint8_t* region = warp_region<C>(dyn_smem, warp);
  WarpPipe<C> pipe;
  pipe.setup(&tmap, reinterpret_cast<uint4*>(region), full[warp], (uint32_t)(rows / 32), ctiles, TILE_C,
             &g_mx4_wait_timeouts);
  const OutStage<C> out{region + C::kStages * kWTileBytes};
  pipe.start();
  const int64_t cb = cols / 32, rb = rows / 32;      // E8M0 row lengths
  uint32_t clip_r = 0, clip_c = 0;
  E8Acc<C::kChunk> e8c0 = 0, e8c1 = 0;               // this chunk's column E8M0 bytes so far
  for (uint32_t j = 0; pipe.valid(pipe.cur); ++j) {
    if (!pipe.wait(j)) {
      out.drain();
      return;
    }
    const uint4* tile = pipe.tile(j);
    const int64_t r0 = pipe.r0(), c0 = pipe.c0();
    out.acquire();
    uint8_t* ob = out.buf(j);

    // A. row-wise blocks of tile row `lane`: 16 bytes each
    uint32_t ebytes = 0;
#pragma unroll
    for (int b = 0; b < G::BPR; ++b) {
      uint4 v[NG];
      load_row_block<NG>(tile, lane, b, v);
      uint32_t pm = mag_load<DT>(v[0]);
#pragma unroll
      for (int k = 1; k < NG; ++k) pm = mag_max<DT>(pm, mag_load<DT>(v[k]));
      uint32_t o[4];
      ebytes |= mx4_block<C::kClipCount>([&](int k) { return elem_bits<DT>(v[k / EPL], k % EPL); }, mag_bits<DT>(pm), rule, headroom,
                          clip_r, o)
                << (8 * b);
      if (G::BPR == 2) stage16<32>(ob + 2048, lane, b, o[0], o[1], o[2], o[3]);
      else *reinterpret_cast<uint4*>(ob + 2048 + lane * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    {
      uint8_t* e8 = e8_row + (r0 + lane) * cb + (c0 >> 5);
      if (G::BPR == 2 && c0 + 64 <= cols) {
        if ((reinterpret_cast<uintptr_t>(e8) & 1u) == 0) {
          *reinterpret_cast<uint16_t*>(e8) = (uint16_t)ebytes;
        } else {
          e8[0] = (uint8_t)ebytes;
          e8[1] = (uint8_t)(ebytes >> 8);
        }
      } else {
        e8[0] = (uint8_t)ebytes;
      }
    }

    // B. column-wise blocks: half `ci & 1` of a 32-byte row of the transpose
    const uint32_t ci = pipe.cur.i;
    const bool flush = pipe.chunk_end(pipe.cur);
    const bool single = flush && (ci & 1) == 0;       // an odd row tile at the end: no pair
    const int64_t rt0 = (r0 >> 5) - ci;               // the chunk's first row tile
    uint32_t w[32], o[4];
    const auto put = [&](int c, const uint32_t (&p)[4]) {
      if (single) *reinterpret_cast<uint4*>(q_colt + (c0 + c) * (rows / 2) + r0 / 2) = make_uint4(p[0], p[1], p[2], p[3]);
      else stage16<32>(ob, c, ci & 1, p[0], p[1], p[2], p[3]);
    };
    if (DT == FP8Q_BF16) {
      const int64_t c = c0 + 2 * lane;
      if (c < cols) {
        load_column_words(tile, lane, w);
        const uint32_t pm = tree_absmax32<true>(w);
        e8c0 |= (E8Acc<C::kChunk>)mx4_block<C::kClipCount>([&](int k) { return half_bits<0>(w[k]); }, pm << 16, rule, headroom, clip_c, o)
                << (8 * ci);
        put(2 * lane, o);
        e8c1 |= (E8Acc<C::kChunk>)mx4_block<C::kClipCount>([&](int k) { return half_bits<1>(w[k]); }, pm & 0xFFFF0000u, rule, headroom,
                                            clip_c, o)
                << (8 * ci);
        put(2 * lane + 1, o);
        if (flush) {
          store_e8_run<C::kChunk>(e8_colt + c * rb + rt0, e8c0, ci + 1);
          store_e8_run<C::kChunk>(e8_colt + (c + 1) * rb + rt0, e8c1, ci + 1);
        }
      }
    } else {
      const int64_t c = c0 + lane;
      if (c < cols) {
        load_column_words(tile, lane, w);
        e8c0 |= (E8Acc<C::kChunk>)mx4_block<C::kClipCount>([&](int k) { return w[k]; }, tree_absmax32<false>(w), rule, headroom, clip_c, o)
                << (8 * ci);
        put(lane, o);
        if (flush) store_e8_run<C::kChunk>(e8_colt + c * rb + rt0, e8c0, ci + 1);
      }
    }
    if (flush) e8c0 = e8c1 = 0;
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(&qmap, ob + 2048, (int)(c0 / 2), (int)r0);
      if (ci & 1) tma_store_2d(&qtmap, ob, (int)((r0 - 32) / 2), (int)c0);
      bulk_commit();
    }
    pipe.release();
  }
  out.drain();
  clip_r = __reduce_add_sync(0xFFFFFFFFu, clip_r);
  clip_c = __reduce_add_sync(0xFFFFFFFFu, clip_c);
  if (lane == 0) {
    if (clipped_row && clip_r) atomicAdd(clipped_row, (unsigned long long)clip_r);
    if (clipped_col && clip_c) atomicAdd(clipped_col, (unsigned long long)clip_c);
  }
}

template <int DT, class C>
static cudaError_t launch_dual(const void* x, int64_t rows, int64_t cols, int rule, int headroom, uint8_t* q_row,
                               uint8_t* e8_row, uint8_t* q_colt, uint8_t* e8_colt, unsigned long long* cr,
                               unsigned long long* cc, cudaStream_t s, int* launches) {
  constexpr int TILE_C = TileGeom<DT>::TILE_C;
  auto kern = mx4_dual_kernel<DT, C>;
  const int64_t ctiles = (cols + TILE_C - 1) / TILE_C;
  if ((rows / 32) * ctiles >= (int64_t(1) << 31)) return cudaErrorInvalidValue;   // 32-bit tile counts
  int occ = 1;
  cudaError_t e = kernel_occupancy(reinterpret_cast<const void*>(kern), C::kThreads, C::kSmemBytes, &occ);
  if (e != cudaSuccess) return e;
  if (C::kMaxCtasPerSm > 0 && occ > C::kMaxCtasPerSm) occ = C::kMaxCtasPerSm;
  const int64_t chunks = ((rows / 32 + C::kChunk - 1) / C::kChunk) * ctiles;
  int64_t grid = (int64_t)sm_count(device_of_current()) * occ;
  if (grid > (chunks + C::kWarps - 1) / C::kWarps) grid = (chunks + C::kWarps - 1) / C::kWarps;
  CUtensorMap in, qm, qtm;
  e = encode_tile_map(&in, x, DT == FP8Q_BF16, rows, cols, TILE_C, true, 128);
  // an odd last row tile has no pair: its box would start inside and end past the row, and is stored by hand
  if (e == cudaSuccess) e = encode_byte_map(&qm, q_row, rows, cols / 2, TILE_C / 2, 32, TILE_C / 2);
  if (e == cudaSuccess) e = encode_byte_map(&qtm, q_colt, cols, rows / 2, rows >= 64 ? 32 : 16, TILE_C, rows >= 64 ? 32 : 0);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)grid, C::kThreads, C::kSmemBytes, s>>>(in, qm, qtm, rows, cols, rule, headroom, q_colt, e8_row,
                                                        e8_colt, cr, cc);
  ++*launches;
  return cudaGetLastError();
}

template <bool COUNT>
static cudaError_t launch_dual_counting(const void* x, int dtype, int64_t rows, int64_t cols, int rule, int headroom,
                                        uint8_t* q_row, uint8_t* e8_row, uint8_t* q_colt, uint8_t* e8_colt,
                                        unsigned long long* cr, unsigned long long* cc, cudaStream_t s, int* launches) {
  const bool b = dtype == FP8Q_BF16;
  const auto launch = tp_small(rows, cols, dtype, Mx4DualCfg<COUNT>::kWarps, kMx4SmallMore)
                          ? (b ? launch_dual<FP8Q_BF16, Mx4DualSmallCfg<COUNT>> : launch_dual<FP8Q_F32, Mx4DualSmallCfg<COUNT>>)
                          : (b ? launch_dual<FP8Q_BF16, Mx4DualCfg<COUNT>> : launch_dual<FP8Q_F32, Mx4DualCfg<COUNT>>);
  return launch(x, rows, cols, rule, headroom, q_row, e8_row, q_colt, e8_colt, cr, cc, s, launches);
}

cudaError_t launch_mx4_dual(const void* x, int dtype, int64_t rows, int64_t cols, int rule, int headroom,
                            uint8_t* q_row, uint8_t* e8_row, uint8_t* q_colt, uint8_t* e8_colt,
                            unsigned long long* cr, unsigned long long* cc, cudaStream_t s, int* launches) {
  // nothing to count where nobody asks or nothing can clip
  return (cr || cc) && !mx_clip_free(rule, headroom)
             ? launch_dual_counting<true>(x, dtype, rows, cols, rule, headroom, q_row, e8_row, q_colt, e8_colt, cr, cc, s, launches)
             : launch_dual_counting<false>(x, dtype, rows, cols, rule, headroom, q_row, e8_row, q_colt, e8_colt, cr, cc, s, launches);
}

}  // namespace fp8q
