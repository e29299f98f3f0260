// Attention of a few query rows per key/value head over the 4-bit cache
// (decoding one token, or checking a few).
//
// Mathematics.  With a row's codes c (E2M1) and block exponents E, a score is
//   x = scale * log2(e) * sum_blocks 2^E * (q . c)
// and the output sum_j 2^(x_j - M) v_j over the same factors' sum.  The codes
// are exact in 16-bit floats.  The key scales multiply the fp32 sums of each
// block.  Values are held relative to the largest block scale 2^R of their 32
// tokens, code times 2^(E - R) in f16, exact down to 2^-22; the running
// reference M is of x + R, so that the weights p = 2^(x + R - M) stay at or
// below 2^8 in f16 whatever the scales are, and the softmax sum takes p * 2^-R.
// (The scales on the weights instead, 2 products for 8, take 219 us where this
// takes 223, but p * 2^(E - R) leaves f16's range where a small weight meets a
// small block.)  M moves only when a tile passes it by 2^8 (one vote per tile),
// which is when the sums are rescaled.
//
// What bounds it: HBM and the unpacking together.  A token and head at D = 128
// is 136 bytes of cache, and a tile of 32 of them 606 warp instructions for up
// to eight query rows, a quarter of them the conversions of the 8192 codes.  8
// sequences of 131072 tokens, 32 heads over 8: 223 us, 5.1 TB/s, 0.77 of the
// measured copy rate (the same copies without the arithmetic: 180 us; ALU pipe
// 55%, issue slots 59%, DRAM reads 1.00 of the cache's bytes); half as wide
// rows (D = 64, the same softmax for half the bytes) 153 us.  mma.sync and not
// tcgen05: with 16 tokens x 8 query rows a product it takes 1 of the 19
// instructions of a token, its operands come straight from the unpacked
// registers, and nothing waits on a tensor-memory round trip.
//
// Layout.  A warp owns tiles of 32 tokens, copied by cp.async into a ring of
// its own (no CTA barrier while it streams; four stages at three CTAs per SM
// took 229 us when three stages at four CTAs took 233, both before later steps).  Keys are the A operand (16 tokens x
// 16 columns, the columns of a block permuted alike in q so that a lane's
// 32-bit word of codes is one lane's share of two products); values are the A
// operand of the transposed product (16 columns x 16 tokens), read by
// ldmatrix.trans from rows stored in an order that puts the codes of two
// tokens where one mask makes a byte of them.  The scores come out with tokens
// down and query rows across, so that a weight tile needs one movmatrix per
// 8 x 8 to become the B operand.
//
// Work is split over the tiles of all sequences and heads: CTA i takes
// positions [i * per, (i + 1) * per) in (sequence, head) order, each of them
// kDecSetup positions and its tiles, so that uneven lengths fill the GPU
// evenly and the host needs to know none of them.  (Set-up of 12 against 6
// and 20 tiles: 64 sequences of 512 tokens and 8 heads 20.4 us against 21.3 and
// 21.3, 64 of up to 8192 and 4 heads 43.5 against 45.9 and 44.3.)  A (sequence, head) that spans several CTAs is
// joined by the last of them to arrive, in the order of the tiles (the result
// does not depend on which that is).
#include "kv_device.cuh"

namespace fp8q {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecStages = 4;
constexpr int kTile = 32;                 // tokens of a warp tile
constexpr int kDecSetup = 12;             // what a (sequence, head) costs beyond its tiles, in tiles
// Positions of a CTA, at least.  With fewer, short calls have more parts to join:
// of two sequences of 4000 and 900 tokens (window 4096, 20 rows) 16.7 us at 8,
// 19.9 at 4, 16.8 at 16; one of 4096 tokens and 8 heads 11.7, 13.3, 11.7; one of
// 1000 tokens and 4 heads 8.8, 8.6, 9.6.
constexpr int kMinTiles = 8;

template <int D>
struct DecSmem {
  static constexpr int kRow = D / 2;      // bytes of a row of codes
  static constexpr int kBlocks = D / 32;
  struct Stage {
    uint8_t k[kTile * kRow];
    uint8_t v[kTile * kRow];
    uint8_t ke[kTile * kBlocks];
    uint8_t ve[kTile * kBlocks];
  };
  struct Warp {
    Stage stage[kDecStages];
    // value scales of the tile being used, f16; token u * 16 + h * 8 + 2 c + i of
    // a block at c * 8 + u * 4 + h * 2 + i: what a lane needs lies together
    __half factor[kBlocks][kTile];
    uint32_t valid[kDecStages];           // tokens of the stage that exist
    uint32_t pad[4 - kDecStages % 4];
  };
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// d += a (16 x 16, row) * b (16 x 8, column), f16 in, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = a * b.
__device__ __forceinline__ void mma_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%10, %10, %10, %10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// Two E8M0 bytes (the low half of w) -> 2^(byte - 127), NaN for 0xFF.
__device__ __forceinline__ float2 e8m0x2_f32(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %1;\n cvt.rn.bf16x2.ue8m0x2 %0, a;\n}" : "=r"(r) : "r"(w));
  return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xFFFF0000u));
}

// A sequence's tiles: the ones that hold a key some query sees.
struct DecSeq : KvSeq {
  int tile0, tiles;
  int cost;              // of one head, in tiles: kDecSetup and the tiles
};
__device__ __forceinline__ DecSeq dec_seq(const KvAttn& a, int b) {
  DecSeq s;
  static_cast<KvSeq&>(s) = kv_seq(a, b);
  s.tile0 = (a.window > 0 ? max(0, s.pos0 - a.window + 1) : 0) / kTile;
  // a sequence with queries and no keys still has its zeros to write
  s.tiles = s.nq == 0 ? 0 : max(1, (s.len + kTile - 1) / kTile - s.tile0);
  s.cost = s.nq == 0 ? 0 : s.tiles + kDecSetup;
  return s;
}

struct DecPlan {
  uint32_t* ticket;      // [kMaxGrid], zero between calls
  float* part;           // [2 * grid][rows * (D + 2)]
};

// Three CTAs per SM for one group of eight rows; with more, two, as three leave
// 168 registers a thread and the sums spill (16 rows over 8 x 131072 tokens 306
// us at two, 345 at three; three queries of four heads over a 4096 window 20.7
// and 26.8; 24 rows 28 and 35).
template <int D, int NT>
__global__ void __launch_bounds__(kDecThreads, NT == 1 ? 3 : 2)
kv_decode_kernel(const __grid_constant__ KvAttn a, const __grid_constant__ DecPlan plan) {
  constexpr int NB = D / 32, RB = D / 2, ROWS = 8 * NT;
  constexpr bool QS = NT > 1;                    // queries in shared memory
  using Smem = DecSmem<D>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane >> 2, lc = lane & 3;
  typename Smem::Warp& sm = reinterpret_cast<typename Smem::Warp*>(smem_raw)[warp];
  __shared__ long long s_scan[kDecThreads / 32 + 1];
  __shared__ int s_start[2];
  __shared__ long long s_before;
  __shared__ uint32_t s_last;
  __shared__ Joined s_rows[8 * NT];
  __shared__ uint4 s_q[QS ? NT * NB * 32 : 1];
  __shared__ float s_f[8 * NT];
  // the lane's row of 8 x 8 code matrices (the swizzle repeats every 8 rows),
  // and the place of its token's value scales
  const uint32_t lane_at = D == 128 ? code_offset<D>(lane & 7, lane >> 3)
                                    : code_offset<D>((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1);
  const int factor_at = ((lane >> 1) & 3) * 8 + (lane >> 4) * 4 + ((lane >> 3) & 1) * 2 + (lane & 1);

  grid_begin();
  // ---- this CTA's range of tiles: a scan of the sequences' tile counts
  const int per_thread = (a.batch + kDecThreads - 1) / kDecThreads;
  const int b_lo = min(a.batch, (int)threadIdx.x * per_thread), b_hi = min(a.batch, b_lo + per_thread);
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += (long long)dec_seq(a, b).cost * a.shape.heads;
  long long incl = mine;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, incl, x);
    if (lane >= x) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kDecWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const long long per = max((long long)kMinTiles, (total + gridDim.x - 1) / gridDim.x);
  const long long begin = (long long)blockIdx.x * per, end = min(total, begin + per);
  if (begin >= end) return;
  if (before <= begin && begin < before + mine) {
    int b = b_lo;
    for (; b < b_hi; ++b) {
      const long long n = (long long)dec_seq(a, b).cost * a.shape.heads;
      if (begin < before + n) break;
      before += n;
    }
    s_start[0] = b;
    s_before = before;
  }
  __syncthreads();
  int b = s_start[0];
  DecSeq sq = dec_seq(a, b);
  int head = (int)((begin - s_before) / sq.cost);
  // position of the first tile of (b, head): its cost lies from kDecSetup before
  long long seg0 = s_before + (long long)head * sq.cost + kDecSetup;

  if (seg0 >= end) return;                       // only the set-up of one: its tiles are the next CTA's

  // ---- what is fetched: tiles [t0, t1) of the (sequence, head) at seg0
  int t0, t1, n_mine, tile0_at;
  const int32_t* table;
  // The warp's k-th tile begins at token tile0_at + k * (kDecWarps * kTile).
  // Pages of 32 tokens or more hold all of a tile's rows in one run; smaller ones
  // are looked up by each lane for its own token (8 x 131072 tokens in pages of
  // 64: 223 us, of 16 or 8: 236).
  const bool runs = a.shape.page_shift >= 5;
  auto page_of = [&](int k) {
    const int tok = tile0_at + k * (kDecWarps * kTile) + (runs ? 0 : lane);
    return k < n_mine && tok < sq.len ? table[tok >> a.shape.page_shift] : -1;
  };
  const int page_mask = (1 << a.shape.page_shift) - 1;
  auto issue = [&](int k, int st, int page) {
    if (k < n_mine) {
      const int at = tile0_at + k * (kDecWarps * kTile), tok = at + (runs ? 0 : lane);
      const bool ok = (uint32_t)page < (uint32_t)a.shape.pages;
      const int64_t row = ok ? kv_row(a.shape, page, tok & page_mask, head) : 0;
      const uint32_t kd = smem_u32(sm.stage[st].k), vd = smem_u32(sm.stage[st].v);
      const uint32_t ke = smem_u32(sm.stage[st].ke), ve = smem_u32(sm.stage[st].ve);
      uint32_t valid;
      if (runs) {
        const int n = ok ? min(sq.len - at, 32) : 0;
        valid = low_bits(n);
        copy_run<D, false>(kd, ke, a.k, row, n);
        copy_run<D, true>(vd, ve, a.v, row, n);
      } else {
        valid = __ballot_sync(0xFFFFFFFFu, ok);
        copy_rows<D, false>(kd, ke, a.k, row, valid, a.shape.page_shift);
        copy_rows<D, true>(vd, ve, a.v, row, valid, a.shape.page_shift);
      }
      sm.valid[st] = valid;                    // the same from every lane
    }
    cp_commit();
  };
  int pages[kDecStages];
  auto open = [&]() {
    t0 = (int)max(0ll, begin - seg0);
    t1 = (int)min((long long)sq.tiles, end - seg0);
    n_mine = t1 - t0 > warp ? (t1 - t0 - warp + kDecWarps - 1) / kDecWarps : 0;
    tile0_at = (sq.tile0 + t0 + warp) * kTile;
    table = a.table + b * a.table_stride;
#pragma unroll
    for (int k = 0; k < kDecStages; ++k) pages[k] = page_of(k);
  };
  // With one group of eight rows the queries stay in registers; with more
  // each warp prepares some of the groups and all read them from shared
  // memory, which leaves the registers to the sums (four groups over 8 x 131072
  // tokens: 539 us against 681 from registers, 515 by now).
  constexpr int QN = QS ? 1 : NT;              // groups of a warp at a time
  uint4 qw[QN][NB];
  auto load_q = [&]() {
    if (QS && warp >= NT) return;
    const int r = (QS ? warp : 0) * 8 + li;
    const bool on = r < sq.nq * a.group;
    const int qi = on ? a.by_group.div(r) : 0, g = on ? r - qi * a.group : 0;
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t)(sq.q0 + qi) * a.q_tok +
                             (int64_t)(head * a.group + g) * a.q_head + lc * 8;
#pragma unroll
    for (int x = 0; x < NB; ++x) qw[0][x] = on ? *reinterpret_cast<const uint4*>(q + x * 32) : make_uint4(0, 0, 0, 0);
  };
  // The join takes a warp's last NT stages, so that with one group of rows the
  // queries and the first EARLY tiles of the next (sequence, head) are on their
  // way meanwhile: 8 x 131072 tokens 223 us against 227 (in pages of 16: 236
  // against 256), at D = 64 153 against 151, 64 sequences of up to 8192 the same.  With more groups the registers for it are missing
  // (five queries of four heads over a 4096 window 26.5 us with it, 25.8 without).
  constexpr int EARLY = kDecStages - NT;
  static_assert(ROWS * (D + 2) * 4 <= NT * (int)sizeof(typename Smem::Stage) && EARLY >= 0, "the join's place");
  constexpr bool AHEAD = NT == 1;
  auto fetch = [&]() {
    load_q();
#pragma unroll
    for (int k = 0; k < EARLY; ++k) issue(k, k, pages[k]);
  };
  open();
  fetch();

  while (true) {
    // ---- one (sequence, head)
    const DecSeq cur = sq;
    const int cur_head = head;
    const long long cur_seg0 = seg0;
    const int rows = cur.nq * a.group, pos0 = cur.pos0;
    const bool whole = t0 == 0 && t1 == cur.tiles;
    const int first_tile = cur.tile0 + t0 + warp;
#pragma unroll
    for (int k = EARLY; k < kDecStages - 1; ++k) issue(k, k, pages[k]);
    int page_next = pages[kDecStages - 1];

    // ---- queries: f16, each row scaled by a power of two to a largest
    // magnitude in [2^14, 2^15), which keeps bf16 exact down to 2^-29 of it
    uint32_t qf[QN][NB][4];
    float fx[NT][2];                             // score factor of query rows 2 lc, 2 lc + 1
    float f = 0.0f;                              // of row li of the warp's group
    if (!QS || warp < NT) {
      uint32_t m = 0;
#pragma unroll
      for (int x = 0; x < NB; ++x) m = vmax_u16x2(m, absmax_load<FP8Q_BF16>(qw[0][x]));
      m = unpack_max<FP8Q_BF16>(m);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const int e = m == 0 ? 0 : max(-112, (int)(m >> 23) - 127) - 14;   // q = q' * 2^e, e in [-126, 113]
      // NaN or Inf: every score of the row is NaN, but those the masks replace
      // (a NaN factor would spoil them too: -inf times NaN)
      const float s = m >= 0x7F800000u ? __uint_as_float(0x7FFFFFFFu) : pow2f(-e);
      f = fmaxf(a.scale * 1.4426950408889634f * pow2f(e), kMinFactor);
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        const uint32_t ws[4] = {qw[0][x].x, qw[0][x].y, qw[0][x].z, qw[0][x].w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
          qf[0][x][y] = cvt_f16x2(__uint_as_float(ws[y] << 16) * s, __uint_as_float(ws[y] & 0xFFFF0000u) * s);
        if (QS) s_q[(warp * NB + x) * 32 + lane] = make_uint4(qf[0][x][0], qf[0][x][1], qf[0][x][2], qf[0][x][3]);
      }
      if (QS && lc == 0) s_f[warp * 8 + li] = f;
    }
    if (QS) {
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        fx[nt][0] = s_f[nt * 8 + lc * 2];
        fx[nt][1] = s_f[nt * 8 + lc * 2 + 1];
      }
    } else {
      fx[0][0] = __shfl_sync(0xFFFFFFFFu, f, lc * 8);
      fx[0][1] = __shfl_sync(0xFFFFFFFFu, f, lc * 8 + 4);
    }

    float o[NT][NB][2][4];
    float mref[NT][2], l[NT][2];
    uint32_t nan_blocks = 0;                     // bit x * 8 + nt * 2 + y: block x of query row 8 nt + 2 lc + y is NaN
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 2; ++x) { mref[nt][x] = kNoMax; l[nt][x] = 0.0f; }
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int y = 0; y < 8; ++y) o[nt][x][y >> 2][y & 3] = 0.0f;
    }

    for (int k = 0, st = 0; k < n_mine; ++k, st = st == kDecStages - 1 ? 0 : st + 1) {
      cp_wait<kDecStages - 2>();
      __syncwarp();
      const typename Smem::Stage& tile = sm.stage[st];
      const uint32_t valid = sm.valid[st];
      const int tok = (first_tile + k * kDecWarps) * kTile;

      // ---- value scales: one token per lane, relative to the tile's largest
      float rv, unscale;
      bool v_nan;
      uint32_t nan_tokens[NB];
      {
        const uint32_t w = NB == 4 ? reinterpret_cast<const uint32_t*>(tile.ve)[lane]
                                   : reinterpret_cast<const uint16_t*>(tile.ve)[lane];
        const bool ok = (valid >> lane) & 1;
        float e[NB], top = 0.0f, all = 0.0f;
#pragma unroll
        for (int x = 0; x < NB; x += 2) {
          const float2 f = e8m0x2_f32(x ? w >> 16 : w);
          e[x] = f.x;
          e[x + 1] = f.y;
          top = fmaxf(top, fmaxf(f.x, f.y));     // leaves NaN out
          all += f.x + f.y;                      // and takes it in
        }
        v_nan = __any_sync(0xFFFFFFFFu, ok && all != all);
        if (v_nan) {                             // NaN blocks count as zeros here; which rows see them is noted below
#pragma unroll
          for (int x = 0; x < NB; ++x) {
            nan_tokens[x] = __ballot_sync(0xFFFFFFFFu, ok && e[x] != e[x]);
            if (e[x] != e[x]) e[x] = 0.0f;
          }
        }
        // positive floats order like their bits
        const uint32_t most = min(max(__reduce_max_sync(0xFFFFFFFFu, ok ? __float_as_uint(top) : 0u), kMinScale << 23),
                                  kMaxScale << 23) & 0x7F800000u;
        rv = (float)((int)(most >> 23) - 127);
        unscale = __uint_as_float((254u << 23) - most);
#pragma unroll
        for (int x = 0; x < NB; x += 2) {
          const uint32_t f = ok ? cvt_f16x2(e[x] * unscale, e[x + 1] * unscale) : 0u;
          reinterpret_cast<uint16_t*>(sm.factor[x])[factor_at] = (uint16_t)f;
          reinterpret_cast<uint16_t*>(sm.factor[x + 1])[factor_at] = (uint16_t)(f >> 16);
        }
        __syncwarp();
      }

      // ---- scores: tokens down, query rows across
      float s[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 4; ++y) s[u][nt][y] = 0.0f;
        uint32_t kw[2][NB];                      // [token half][block]
        const uint32_t base = smem_u32(tile.k);
        if (D == 128) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[4];
            ldmatrix4<false>(r, base + (u * 16 + h * 8) * RB + lane_at);
#pragma unroll
            for (int x = 0; x < NB; ++x) kw[h][x] = r[x & 3];
          }
        } else {
          uint32_t r[4];
          ldmatrix4<false>(r, base + u * 16 * RB + lane_at);
          kw[0][0] = r[0]; kw[0][1] = r[1]; kw[1][0] = r[2]; kw[1][1] = r[3];
        }
        float ks[2][NB];                         // scales of tokens li, li + 8
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = u * 16 + h * 8 + li;
          const uint32_t w = NB == 4 ? reinterpret_cast<const uint32_t*>(tile.ke)[t]
                                     : reinterpret_cast<const uint16_t*>(tile.ke)[t];
#pragma unroll
          for (int x = 0; x < NB; x += 2) {
            const float2 f = e8m0x2_f32(x ? w >> 16 : w);
            ks[h][x] = f.x;
            ks[h][x + 1] = f.y;
          }
        }
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          uint32_t ka[4], kb[4];
          e2m1x8_f16(kw[0][x], ka);
          e2m1x8_f16(kw[1][x], kb);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float c[4];
            const uint4 q = QS ? s_q[(nt * NB + x) * 32 + lane]
                               : make_uint4(qf[0][x][0], qf[0][x][1], qf[0][x][2], qf[0][x][3]);
            mma_zero(c, ka[0], kb[0], ka[1], kb[1], q.x, q.y);
            mma(c, ka[2], kb[2], ka[3], kb[3], q.z, q.w);
            s[u][nt][0] += c[0] * ks[0][x];
            s[u][nt][1] += c[1] * ks[0][x];
            s[u][nt][2] += c[2] * ks[1][x];
            s[u][nt][3] += c[3] * ks[1][x];
          }
        }
      }

      // ---- masks, only where the tile has any
      const bool edge = valid != 0xFFFFFFFFu || tok + kTile - 1 > pos0 ||
                        (a.window > 0 && tok <= pos0 + cur.nq - 1 - a.window);
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int pos = pos0 + a.by_group.div(nt * 8 + lc * 2 + y);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const int t = z * 8 + li, j = tok + t;
              const bool seen = ((valid >> t) & 1) && j <= pos && (a.window == 0 || j > pos - a.window);
              float& x = s[z >> 1][nt][(z & 1) * 2 + y];
              x = seen ? x : -INFINITY;
            }
          }
      }

      if (v_nan) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int pos = pos0 + a.by_group.div(nt * 8 + lc * 2 + y);
            uint32_t seen = valid & low_bits(pos - tok + 1);
            if (a.window > 0) seen &= ~low_bits(pos - a.window + 1 - tok);
#pragma unroll
            for (int x = 0; x < NB; ++x) nan_blocks |= (nan_tokens[x] & seen) ? 1u << (x * 8 + nt * 2 + y) : 0u;
          }
      }

      // ---- the reference moves when some score passes it by 2^kSlack
      bool move = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          top[nt][y] = fmaxf(fmaxf(s[0][nt][y], s[0][nt][y + 2]), fmaxf(s[1][nt][y], s[1][nt][y + 2])) * fx[nt][y] + rv;
          move |= top[nt][y] > mref[nt][y] + kSlack;
        }
      if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float t = top[nt][y];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, x));
            t = fmaxf(t, mref[nt][y]);
            const float fix = ex2(mref[nt][y] - t);
            mref[nt][y] = t;
            l[nt][y] *= fix;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                o[nt][x][z][y] *= fix;
                o[nt][x][z][y + 2] *= fix;
              }
          }
      }

      // ---- weights, their sum, and the second product
      uint32_t p[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float c0 = rv - mref[nt][0], c1 = rv - mref[nt][1];
          const float a0 = ex2(fmaf(s[u][nt][0], fx[nt][0], c0)), a1 = ex2(fmaf(s[u][nt][1], fx[nt][1], c1));
          const float a2 = ex2(fmaf(s[u][nt][2], fx[nt][0], c0)), a3 = ex2(fmaf(s[u][nt][3], fx[nt][1], c1));
          l[nt][0] += (a0 + a2) * unscale;
          l[nt][1] += (a1 + a3) * unscale;
          p[u][nt][0] = movmatrix(cvt_f16x2(a0, a1));
          p[u][nt][1] = movmatrix(cvt_f16x2(a2, a3));
        }
      uint4 fac[NB];
#pragma unroll
      for (int x = 0; x < NB; ++x) fac[x] = *reinterpret_cast<const uint4*>(&sm.factor[x][lc * 8]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t vw[2][NB];                      // [matrix][block]: codes 4 li .. 4 li + 3 of two tokens
        const uint32_t base = smem_u32(tile.v);
        if (D == 128) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[4];
            ldmatrix4<true>(r, base + (u * 16 + h * 8) * RB + lane_at);
#pragma unroll
            for (int x = 0; x < NB; ++x) vw[h][x] = r[x & 3];
          }
        } else {
          uint32_t r[4];
          ldmatrix4<true>(r, base + u * 16 * RB + lane_at);
          vw[0][0] = r[0]; vw[0][1] = r[1]; vw[1][0] = r[2]; vw[1][1] = r[3];
        }
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          // Bytes that pair a token's code with its neighbour's: the rows lie
          // swapped, so that the first matrix holds tokens 2 lc and 2 lc + 8,
          // the second the ones after them.
          const uint32_t m = 0x0F0F0F0Fu;
          uint32_t c02[4], c13[4];               // columns 0, 2 then 1, 3; tokens 2 lc, + 1, then 2 lc + 8, + 9
          e2m1x8_f16((vw[0][x] & m) | ((vw[1][x] << 4) & ~m), c02);
          e2m1x8_f16(((vw[0][x] >> 4) & m) | (vw[1][x] & ~m), c13);
          const uint32_t f0 = u ? fac[x].z : fac[x].x, f1 = u ? fac[x].w : fac[x].y;
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            c02[y] = mul_f16x2(c02[y], y < 2 ? f0 : f1);
            c13[y] = mul_f16x2(c13[y], y < 2 ? f0 : f1);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma(o[nt][x][0], c02[0], c13[0], c02[2], c13[2], p[u][nt][0], p[u][nt][1]);
            mma(o[nt][x][1], c02[1], c13[1], c02[3], c13[3], p[u][nt][0], p[u][nt][1]);
          }
        }
      }
      __syncwarp();
      issue(k + kDecStages - 1, st == 0 ? kDecStages - 1 : st - 1, page_next);
      page_next = page_of(k + kDecStages);
    }

    // ---- the next (sequence, head): its pages
    seg0 += sq.cost;
    const bool more = seg0 < end;
    if (++head == a.shape.heads) {
      head = 0;
      if (more) {                                // then there is one
        do sq = dec_seq(a, ++b);
        while (sq.tiles == 0);
      }
    }
    if (AHEAD && more) open();

    // ---- join the warps: sums of a row over its lanes, then over the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[nt][y] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][y], x);
    if (nan_blocks) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if ((nan_blocks >> (x * 8 + nt * 2 + (y & 1))) & 1)
              o[nt][x][0][y] = o[nt][x][1][y] = __uint_as_float(0x7FFFFFFFu);
    }
    auto warp_part = [&](int i) {                // [rows][D], then M, then l
      return reinterpret_cast<const float*>(&reinterpret_cast<typename Smem::Warp*>(smem_raw)[i].stage[EARLY]);
    };
    float* so = const_cast<float*>(warp_part(warp));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = nt * 8 + lc * 2 + y;
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          float* d = so + r * D + x * 32 + li * 4;
          d[0] = o[nt][x][0][y];
          d[1] = o[nt][x][0][y + 2];
          d[2] = o[nt][x][1][y];
          d[3] = o[nt][x][1][y + 2];
        }
        if (li == 0) {
          so[ROWS * D + r] = mref[nt][y];
          so[ROWS * D + ROWS + r] = l[nt][y];
        }
      }
    if (AHEAD && more) fetch();
    __syncthreads();

    // Each thread has the same four columns of U rows, of the warps' sums
    // first and of the CTAs' parts where there are several.
    constexpr int PART = ROWS * (D + 2), U = ROWS * (D / 4) / kDecThreads, STEP = kDecThreads / (D / 4);
    constexpr int PER_ROW = NT == 1 ? 16 : NT == 2 ? 8 : 4;     // threads that find a row's reference
    const int r0 = threadIdx.x / (D / 4), c = threadIdx.x % (D / 4);
    auto join = [&](auto part_at, int n, float* dst) {          // dst: where the joined part goes; NULL: the output
      const int r = threadIdx.x / PER_ROW;
      Joined j = {kNoMax, 0.0f};
      if (r < rows) j = row_of_parts<ROWS, D>(part_at, threadIdx.x % PER_ROW, PER_ROW, n, r);
#pragma unroll
      for (int x = 1; x < PER_ROW; x <<= 1)
        j = join2(j, {__shfl_xor_sync(0xFFFFFFFFu, j.m, x), __shfl_xor_sync(0xFFFFFFFFu, j.l, x)});
      if (r < rows && threadIdx.x % PER_ROW == 0) {
        s_rows[r] = j;
        if (dst) {
          dst[ROWS * D + r] = j.m;
          dst[ROWS * D + ROWS + r] = j.l;
        } else {
          const int qi = a.by_group.div(r);
          store_lse(a, cur.q0 + qi, cur_head * a.group + r - qi * a.group, j.m, j.l);
        }
      }
      __syncthreads();
      int rs[U];
      float m[U];
      float4 v[U];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        rs[x] = min(r0 + x * STEP, rows - 1);
        m[x] = s_rows[rs[x]].m;
      }
      columns_of_parts<ROWS, D, U, (U >= 4 ? 2 : 8 / U)>(part_at, n, rs, c, m, v);
#pragma unroll
      for (int x = 0; x < U; ++x) {
        if (r0 + x * STEP >= rows) continue;
        if (dst) {
          *reinterpret_cast<float4*>(dst + rs[x] * D + c * 4) = v[x];
        } else {
          const int qi = a.by_group.div(rs[x]);
          store_columns(a, cur.q0 + qi, cur_head * a.group + rs[x] - qi * a.group, c, v[x], s_rows[rs[x]].l);
        }
      }
    };
    if (whole) {
      join(warp_part, kDecWarps, nullptr);
    } else {
      // parts of this (sequence, head): CTAs first .. last; a CTA's slot is 0
      // where the (sequence, head) covers the start of its range, else 1
      const long long first = cur_seg0 / per, last = (cur_seg0 + cur.tiles - 1) / per;
      join(warp_part, kDecWarps, plan.part + (2 * (long long)blockIdx.x + (cur_seg0 <= begin ? 0 : 1)) * PART);
      __syncthreads();
      if (threadIdx.x == 0) {
        // a CTA starts at most one that others go on with
        s_last = take_ticket(plan.ticket + first, (uint32_t)(last - first), 0);
      }
      __syncthreads();
      if (s_last) {
        join([&](int i) {
          const long long x = first + i;
          return static_cast<const float*>(plan.part) + (2 * x + (cur_seg0 <= x * per ? 0 : 1)) * PART;
        }, (int)(last - first) + 1, nullptr);
      }
    }
    if (!more) break;
    __syncthreads();
    if (!AHEAD) {
      open();
      fetch();
    }
  }
}

// ---- host side ---------------------------------------------------------------

static int dec_nt(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4; }

template <int D, int NT>
static int dec_smem() {
  const int ring = kDecWarps * (int)sizeof(typename DecSmem<D>::Warp), join = kDecWarps * 8 * NT * (D + 2) * 4;
  return ring > join ? ring : join;
}

struct DecLaunch {
  const void* kernel;
  int smem, nt;
};
template <int D>
static DecLaunch dec_pick(int nt) {
  switch (nt) {
    case 1: return {reinterpret_cast<const void*>(kv_decode_kernel<D, 1>), dec_smem<D, 1>(), 1};
    case 2: return {reinterpret_cast<const void*>(kv_decode_kernel<D, 2>), dec_smem<D, 2>(), 2};
    case 3: return {reinterpret_cast<const void*>(kv_decode_kernel<D, 3>), dec_smem<D, 3>(), 3};
    default: return {reinterpret_cast<const void*>(kv_decode_kernel<D, 4>), dec_smem<D, 4>(), 4};
  }
}

// CTAs of a call: as many as are resident at once, or one per kMinTiles of the
// cost that the longest sequences would have, if that is fewer.
static cudaError_t dec_grid(const DecLaunch& k, const KvShape& s, int batch, int table_width, int sms, int* grid) {
  int occ = 1;
  const cudaError_t e = kernel_occupancy(k.kernel, kDecThreads, k.smem, &occ);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (((int64_t)table_width << s.page_shift) + kTile - 1) / kTile;
  const int64_t most = ((tiles + kDecSetup) * batch * s.heads + kMinTiles - 1) / kMinTiles;
  int64_t n = most < (int64_t)sms * occ ? most : (int64_t)sms * occ;
  *grid = (int)(n < kMaxGrid ? n : kMaxGrid);
  return cudaSuccess;
}

// Up to 32 rows a key/value head: 8, 16, 24, 32 rows over a 4096 window take 18,
// 21, 26, 32 us here and 45 to 47 in kv_prompt.cu, over 8 x 131072 tokens 223,
// 306, 401, 515 and 708 to 712; beyond, every further 32 rows would read and
// unpack the cache again, while that kernel does it once for 256 (64 rows:
// 48 and 714 us).
bool kv_decode_takes(int max_q, int group) { return (int64_t)max_q * group <= 32; }

static int64_t dec_bytes(int grid, int nt, int dim) {
  return grid < 2 ? 0 : kMaxGrid * 4 + (int64_t)grid * 2 * 8 * nt * (dim + 2) * 4;
}

cudaError_t kv_decode_workspace(const KvShape& s, int group, int batch, int max_q, int table_width, int sms,
                                int64_t* bytes) {
  const int nt = dec_nt(max_q * group);
  const DecLaunch k = s.dim == 128 ? dec_pick<128>(nt) : dec_pick<64>(nt);
  int grid = 0;
  const cudaError_t e = dec_grid(k, s, batch, table_width, sms, &grid);
  *bytes = dec_bytes(grid, nt, s.dim);
  return e;
}

cudaError_t launch_kv_decode(const KvAttn& a, const KvWork& w, int sms, cudaStream_t st, int* status, int* launches) {
  const int nt = dec_nt(a.max_q * a.group);
  const DecLaunch k = a.shape.dim == 128 ? dec_pick<128>(nt) : dec_pick<64>(nt);
  int grid = 0;
  cudaError_t e = dec_grid(k, a.shape, a.batch, a.table_width, sms, &grid);
  if (e != cudaSuccess) return e;
  *status = w.check(dec_bytes(grid, nt, a.shape.dim));
  if (*status != FP8Q_OK) return cudaSuccess;
  DecPlan plan = {w.tickets(), w.parts()};
  void* args[2] = {const_cast<KvAttn*>(&a), &plan};
  return launch_dependent(k.kernel, dim3(grid), kDecThreads, k.smem, args, st, launches);
}

}  // namespace fp8q
