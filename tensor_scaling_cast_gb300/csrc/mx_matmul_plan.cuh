// Which kernel takes a product of two matrices in MX blocks, with which tiles,
// how often a tile's sum is split and how out leaves: on the host, from sizes,
// alignment and the number of SMs alone.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "mx_linear.cuh"

namespace fp8q {

// How out leaves: by TMA, or from registers as bf16 or fp32, or as one of them
// after something is added.  Kernels of their own: one with all of them needs
// more registers than there are.
enum class MmOut { kTma, kBf16, kF32, kAddBf16, kAddF32 };

struct MmPlan {
  bool pair;                 // mm_pair_kernel, else mm_split_kernel
  int32_t columns;           // of a tile
  MmOut out;                 // of the pair kernel
  bool w_is_a;               // the rows that tiles have 128 (a pair 256) of are a's
  int32_t splits;            // CTAs that share a tile's sum
  int64_t tiles;
};

constexpr int kSplitLeast = 4;             // K blocks of a CTA that are worth a join

// CTAs that share a tile's sum, up to a portable cluster.  One per SM, with at
// least kSplitLeast K blocks each (1 x 8192 x 2048 in 4 bits: two of four blocks
// 4.5 us, four of two 5.1, one of eight 5.1); two per SM where each still has
// `twice` blocks (0: never): their loads overlap more (1 x 8192 x 8192 9.9 -> 8.7
// us, in 8 bits 128 x 4096 x 8192 16.9 -> 13.2), but with shorter sums their
// starts and ends cost more than that gains (64 x 8192 x 2048 in 8 bits, eight
// blocks each, 7.4 -> 9.3).
inline int splits_of(int64_t tiles, int64_t kblocks, int64_t sms, int64_t twice) {
  const int64_t one = std::min(sms / tiles, kblocks / kSplitLeast);
  const int64_t two = twice ? std::min(2 * sms / tiles, kblocks / twice) : 0;
  return (int)std::max<int64_t>(1, std::min<int64_t>(8, std::max(one, two)));
}

// How the pair kernel would take a product with NT columns a tile, and the
// cycles of its products: whole rounds of tiles, 2 NT a K block (4 products of
// NT / 2) and, fitted to measurements, 512 a tile where the buffers of sums share
// columns, 3% for 224 columns and 30% and 300 a tile for 128, which read more for
// each product and have more tiles to start.
struct PairPlan {
  int64_t cycles;
  bool by_tma;
};
inline PairPlan plan_pair(const MxProduct& p, int nt, int64_t kblocks, int64_t pairs) {
  const int64_t tiles = ((p.a.rows + 255) / 256) * ((p.b.rows + nt - 1) / nt);
  const int64_t size = p.fp32 ? 4 : 2;
  const bool lines = (reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)(p.out_stride * size)) % 16 == 0;
  // Out leaves by TMA, a few boxes at a time, where the products of the next
  // tile take about as long: stores from registers hold up the warps that bring
  // scales (4 bits, 16384 x 8192 x 2048 96 us against 102).  Under shorter
  // products stores from registers are done sooner (4096 x 4096 x 1024 12.5 us
  // against 16.5; one round of tiles, 512 x 8192 x 2048, 7.7 against 8.7), and
  // under long ones they hardly matter (8192 x 8192 x 8192 158 against 162).
  const int64_t products = kblocks * 2 * nt;
  const bool by_tma = lines && !p.add && (nt == 224 || (tiles > pairs && products >= 3000 && products < 12000));
  const int64_t block = nt == 256 ? 512 : nt == 224 ? 461 : 333;
  int64_t cycles = (tiles + pairs - 1) / pairs * (kblocks * block + (nt == 256 ? 512 : nt == 224 ? 100 : 300));
  // 448 bytes of bf16 a row are no whole lines: by TMA, or for fp32 sums that are added to
  if (nt == 224 && !by_tma && !(p.fp32 && p.add)) cycles *= 2;
  return {cycles, by_tma};
}

inline MmPlan split_plan(const MxProduct& p, int columns, bool w_is_a, int64_t kblocks, int64_t sms) {
  const int64_t w = w_is_a ? p.a.rows : p.b.rows, t = w_is_a ? p.b.rows : p.a.rows;
  MmPlan plan = {false, columns, MmOut::kBf16, w_is_a, 1, ((w + 127) / 128) * ((t + columns - 1) / columns)};
  plan.splits = splits_of(plan.tiles, kblocks, sms, columns <= 32 ? 8 : w <= 256 ? 16 : 0);
  return plan;
}

inline MmPlan plan_product(const MxProduct& p, int64_t sms) {
  const bool a_few = p.a.rows <= p.b.rows;
  const MxView &few = a_few ? p.a : p.b, &many = a_few ? p.b : p.a;
  const int64_t kblocks = (p.a.row_bytes() + 127) / 128;
  // Few rows on one side, as when decoding: they are the columns of tiles of 128
  // of the others.
  if (few.rows <= 16) return split_plan(p, 16, !a_few, kblocks, sms);
  if (few.rows <= 32) return split_plan(p, 32, !a_few, kblocks, sms);
  const PairPlan c256 = plan_pair(p, 256, kblocks, sms / 2), c224 = plan_pair(p, 224, kblocks, sms / 2),
                 c128 = plan_pair(p, 128, kblocks, sms / 2);
  // Where all tiles of 128 x 64 run at once, the few rows being those of 128, the
  // sum can be split: up to 256 rows always (4 bits, 64 x 2048 x 8192 7.4 us
  // against 11.9 in pairs; 256 x 8192 x 2048, where they do not all run at once,
  // 8.1 against 6.8), for more by the K blocks that a CTA then has, 330 cycles
  // each and 2500 for the join.  A short sum needs no split and takes narrower
  // tiles (128 x 4096 x 1024 4.7 us against 5.4).
  const int64_t bands = (few.rows + 127) / 128, tiles = bands * ((many.rows + 63) / 64);
  if (tiles <= sms) {
    if (bands <= 2 && kblocks <= 2 * kSplitLeast && bands * ((many.rows + 31) / 32) <= sms)
      return split_plan(p, 32, a_few, kblocks, sms);
    const int64_t blocks = kblocks / splits_of(tiles, kblocks, sms, 0);
    if (bands <= 2 || blocks * 330 + 2500 < std::min(c128.cycles, std::min(c224.cycles, c256.cycles)))
      return split_plan(p, 64, a_few, kblocks, sms);
  }
  const int nt = c128.cycles < c224.cycles && c128.cycles < c256.cycles ? 128 : c224.cycles < c256.cycles ? 224 : 256;
  const PairPlan& c = nt == 128 ? c128 : nt == 224 ? c224 : c256;
  const MmOut out = c.by_tma  ? MmOut::kTma
                    : p.add   ? (p.fp32 ? MmOut::kAddF32 : MmOut::kAddBf16)
                    : p.fp32  ? MmOut::kF32
                              : MmOut::kBf16;
  return {true, nt, out, true, 1, ((p.a.rows + 255) / 256) * ((p.b.rows + nt - 1) / nt)};
}

}  // namespace fp8q
