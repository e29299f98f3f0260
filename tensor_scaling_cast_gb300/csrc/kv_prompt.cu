// Attention of many query rows per key/value head over the 4-bit cache
// (prompt chunks), on tcgen05 with tensor-memory accumulators.
//
// Mathematics: that of kv_decode.cu, with both operands of each product
// brought to f16 once per 128 tokens and used by up to 256 query rows.  A
// group of 32 tokens is held relative to its largest block scale, for keys
// 2^Rk and for values 2^Rv, so that its codes times 2^(E - R) are exact in
// f16 down to 2^-22 of the largest; a score is then 2^Rk * (q . k'), the
// weights are 2^(x + Rv - M) and the softmax sum takes them times 2^-Rv.
//
// What bounds it: the issue slots.  A unit (128 keys x 256 rows, D = 128)
// takes 2560 clocks of the tensor cores (4096 f16 multiply-adds a clock, the
// score products at two thirds of that: 64 keys wide, they are fed at the
// shared memory's 128 bytes a clock), 1024 of the exponentials, and 11.2 K
// warp instructions, 2800 clocks of the SM's four schedulers; measured are
// 4100.  2048 queries after 14336 tokens, 32 heads over 8: 435 us, 1184
// TFLOP/s, 0.62 of the measured bf16 rate; at D = 64, where the exponentials
// and the instructions are the same and the products half, about a tenth less.
//
// Layout: one CTA per SM.  Two warpgroups hold the softmax of 128 rows each
// (rows are query tokens times the heads that share a key/value head, one row
// per thread), two unpack keys and values (a warp's 32 rows come by cp.async
// and go, as f16, into two-stage rings of 128-byte-swizzled tiles), and two
// warps issue the products, one for each softmax warpgroup.  A unit's scores
// are made and used in two halves of 64 keys, so that a warpgroup works on one
// half while the other half's products run; weights return to tensor memory
// over the scores they came from (f16, the A operand of the second product);
// values are the B operand with D consecutive, so neither is transposed.
// Sizes: scores 2 x 128 and sums 2 x D columns fill the 512 of tensor memory
// at D = 128; queries 64 KB, keys and values 128 KB, raw rows 17 KB of shared
// memory.  Registers: 640 threads launch with 96, which setmaxnreg turns into
// 144 for the softmax and 64 for the others.
//
// Work is split as in kv_decode.cu: CTA i takes positions [i * per, (i + 1) *
// per) over all units in (sequence, head, rows) order, each item of 256 rows
// with kPrSetup positions more for its queries and output, and what spans CTAs
// is joined by the last of them to arrive.  (Set-up of 4 against 3, 6 and 8
// positions: four ragged prompts 282 us against 298, 294 and 303 when it was
// chosen; 262 now, some 14 more with 3 and 10 more with 6.)
#include "kv_device.cuh"
#include "tcgen05.cuh"

namespace fp8q {

constexpr int kPrThreads = 640;
constexpr int kPrIssuer = 16;             // this warp and the next issue the products; it owns tensor memory
constexpr int kPrRows = 256;              // query rows of an item: two warpgroups of 128
constexpr int kPrKeys = 128;              // keys of a unit
constexpr int kPrHalf = 64;               // and of a half of it: scores are made and used by halves
constexpr int kPrStages = 2;              // units of unpacked keys, and of values, in shared memory
// Units of a CTA, at least.  128 queries after 896 tokens, 32 heads over 8: 33 us
// at 8, 35 at 5, 54 at 16; 64 queries after 1984, 8 heads over one: 40, 36, 56;
// four ragged prompts up to 256 tokens: 28, 27, 41.
constexpr int kPrMinUnits = 8;
constexpr int kPrSetup = 4;               // what an item costs beyond its units, in units

// Registers a thread: what a launch gives (__launch_bounds__ of 640 threads),
// and the roles' shares of it.  setmaxnreg waits for registers, so shares
// beyond the launch's would wait forever.
constexpr int kPrRegs = 96, kSoftmaxRegs = 144, kUnpackRegs = 64, kIssueRegs = 64;
static_assert(256 * kSoftmaxRegs + 256 * kUnpackRegs + 128 * kIssueRegs <= kPrThreads * kPrRegs, "register shares");

__device__ unsigned int g_kv_wait_timeouts = 0;

constexpr int kPrInfos = 4;               // more units than the unpacking warps can be ahead
struct __align__(16) PrInfo {             // of a unit, by its groups of 32 tokens; written by the unpacking warps
  float rk[4], rv[4], unscale[4];         // 2^Rk, Rv, 2^-Rv
  uint32_t valid[4], any_nan[4];          // tokens that exist, tokens with a NaN block of values
  uint32_t vnan[4][4];                    // tokens with block b of the values NaN (set where any_nan is not 0)
};

// One item: 256 rows of one (sequence, head) and the units of 128 keys that
// some of the rows see.
struct PrItem {
  KvSeq sq;
  int b, head, rt;          // sequence, head, row tile
  int rows, tiles_r;        // rows of the (sequence, head), row tiles
  int tile0, n;             // first 128 keys, units
};
template <int D>
struct PrSmem {
  static constexpr int kQHalf = 128 * 128, kHalf = kPrKeys * 128;      // 64 columns of f16 rows
  static constexpr int kQBytes = kQHalf * (D / 64), kTileBytes = kHalf * (D / 64);
  uint8_t q[2][kQBytes];
  uint8_t k[kPrStages][kTileBytes];
  uint8_t v[kPrStages][kTileBytes];
  struct Raw {                                        // a warp's 32 rows as they lie in the cache
    uint8_t codes[32 * D / 2];
    uint8_t scales[32 * D / 32];
  } raw[8];
  PrInfo info[kPrInfos];
  PrItem item[kPrThreads / 32];                       // each warp's place in the CTA's items
  uint64_t q_full[2];                                 // per warpgroup of rows
  uint64_t s_full[2][2], p_full[2][2], o_full[2][2];  // and half of a unit (o: the product of its weights)
  uint64_t k_full[kPrStages], k_empty[kPrStages], v_full[kPrStages], v_empty[kPrStages];
  uint64_t info_full[kPrInfos];
  uint64_t join_all, join_last, drain;
  uint32_t tmem, last;
  uint32_t taken, gave_up;                            // tickets taken; some wait ran out
};

__device__ __forceinline__ void pr_units(const KvAttn& a, const KvSeq& s, int rt, int* tile0, int* n) {
  const int rows = s.nq * a.group;
  const int first = a.by_group.div(rt * kPrRows), last = a.by_group.div(min(rows, (rt + 1) * kPrRows) - 1);
  const int begin = a.window > 0 ? max(0, s.pos0 + first - a.window + 1) : 0;
  const int end = min(s.len, s.pos0 + last + 1);
  *tile0 = begin / kPrKeys;
  *n = max(1, (max(end, 0) + kPrKeys - 1) / kPrKeys - *tile0);     // rows that see nothing have zeros to write
}
__device__ __forceinline__ void pr_set(const KvAttn& a, PrItem& it) {
  it.rows = it.sq.nq * a.group;
  it.tiles_r = (it.rows + kPrRows - 1) / kPrRows;
}
// The item after this one; only called while one exists.
__device__ __forceinline__ void pr_next(const KvAttn& a, PrItem& it) {
  if (++it.rt == it.tiles_r) {
    it.rt = 0;
    if (++it.head == a.shape.heads) {
      it.head = 0;
      do it.sq = kv_seq(a, ++it.b);
      while (it.sq.nq == 0);
      pr_set(a, it);
    }
  }
  pr_units(a, it.sq, it.rt, &it.tile0, &it.n);
}

// Sums of a half's weights above this move the reference: no weight reaches
// f16's largest value below it.
constexpr float kMostSum = 16384.0f;

struct PrPlan {
  uint32_t* ticket;
  float* part;             // [2 * grid][kPrRows * (D + 2)]
};

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1)
kv_prompt_kernel(const __grid_constant__ KvAttn a, const __grid_constant__ PrPlan plan) {
  using Smem = PrSmem<D>;
  constexpr int NB = D / 32;
  constexpr uint32_t kS = 0, kO = 256;               // tensor-memory columns of warpgroup 0 (+ 128 for 1)
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + (-smem_addr(smem_raw) & 1023u));      // 1024-byte aligned
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;

  grid_begin();
  // ---- this CTA's range of units
  __shared__ long long s_scan[kPrThreads / 32];
  __shared__ long long s_first[2];                   // begin's (sequence, its first unit)
  __shared__ long long s_range[2];                   // begin, units of a CTA
  constexpr int W = kPrThreads / 32;
  const int per_warp = (a.batch + W - 1) / W;
  const int b_lo = min(a.batch, warp * per_warp), b_hi = min(a.batch, b_lo + per_warp);
  auto seq_units = [&](const KvSeq& s) {             // of one head; the whole warp calls it
    const int tiles_r = (int)(((long long)s.nq * a.group + kPrRows - 1) / kPrRows);
    long long u = 0;
    for (int rt = lane; rt < tiles_r; rt += 32) {
      int t0, n;
      pr_units(a, s, rt, &t0, &n);
      u += n + kPrSetup;
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, x);
    return u;
  };
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += seq_units(kv_seq(a, b)) * a.shape.heads;
  if (lane == 0) s_scan[warp] = mine;
  __syncthreads();
  long long before = 0, total = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const long long per = max((long long)kPrMinUnits, (total + gridDim.x - 1) / gridDim.x);
  const long long begin = (long long)blockIdx.x * per, end = min(total, begin + per);
  if (begin >= end) return;
  if (threadIdx.x == 0) {
    s_range[0] = begin;
    s_range[1] = per;
  }
  if (before <= begin && begin < before + mine) {
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = seq_units(kv_seq(a, b)) * a.shape.heads;
      if (begin < before + n) {
        if (lane == 0) { s_first[0] = b; s_first[1] = before; }
        break;
      }
      before += n;
    }
  }

  // ---- barriers and tensor memory
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sm.q_full[x], 4);
      for (int y = 0; y < 2; ++y) {
        mbar_init(&sm.s_full[x][y], 1);
        mbar_init(&sm.p_full[x][y], 4);
        mbar_init(&sm.o_full[x][y], 1);
      }
    }
    for (int x = 0; x < kPrStages; ++x) {
      mbar_init(&sm.k_full[x], 4);
      mbar_init(&sm.k_empty[x], 2);
      mbar_init(&sm.v_full[x], 4);
      mbar_init(&sm.v_empty[x], 2);
    }
    for (int x = 0; x < kPrInfos; ++x) mbar_init(&sm.info_full[x], 8);
    mbar_init(&sm.join_all, 8);
    mbar_init(&sm.join_last, 1);
    mbar_init(&sm.drain, 2);
    sm.taken = sm.gave_up = 0;
    fence_barrier_init();
  }
  if (warp == kPrIssuer) tmem_alloc(&sm.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sm.tmem;

  // each warp's item is warp-uniform and used now and then: it lives in shared memory
  PrItem& it = sm.item[warp];
  long long seg0 = s_first[1];                       // global unit of the item's first one
  {
    PrItem x;
    x.b = (int)s_first[0];
    x.sq = kv_seq(a, x.b);
    pr_set(a, x);
    const long long u = seq_units(x.sq);
    x.head = (int)((begin - seg0) / u);
    seg0 += x.head * u;
    // the row tile that holds `begin`: 32 at a time
    for (x.rt = 0;; x.rt += 32) {
      int t0 = 0, n = 0;
      if (x.rt + lane < x.tiles_r) pr_units(a, x.sq, x.rt + lane, &t0, &n);
      long long upto = x.rt + lane < x.tiles_r ? n + kPrSetup : 0;
#pragma unroll
      for (int y = 1; y < 32; y <<= 1) {
        const long long z = __shfl_up_sync(0xFFFFFFFFu, upto, y);
        if (lane >= y) upto += z;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, seg0 + upto > begin);
      if (past) {
        const int l = __ffs(past) - 1;
        x.tile0 = __shfl_sync(0xFFFFFFFFu, t0, l);
        x.n = __shfl_sync(0xFFFFFFFFu, n, l);
        seg0 += __shfl_sync(0xFFFFFFFFu, upto, l) - (x.n + kPrSetup);
        x.rt += l;
        break;
      }
      seg0 += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    if (lane == 0) it = x;
    __syncwarp();
  }
  auto next_item = [&]() {
    __syncwarp();
    if (lane == 0) pr_next(a, it);
    __syncwarp();
  };

  // From here on positions count from `begin`: an item lies at rel .. (not above
  // 0 for the first item), kPrSetup positions and then its units.
  const int units = (int)(end - begin);
  int rel = (int)(seg0 - begin);
  // the item's units that are this CTA's, and the step to the next item that has any
  auto unit0 = [&]() { return max(0, -rel - kPrSetup); };
  auto unit1 = [&]() { return min(it.n, units - rel - kPrSetup); };
  auto advance = [&]() {
    rel += kPrSetup + it.n;
    if (rel + kPrSetup >= units) return false;
    next_item();
    return true;
  };

  // Every wait is bounded; a role whose wait runs out counts it and returns,
  // and so do the others in turn, to the common end.  A warp's lanes each try
  // for themselves and might see a barrier complete at different tries; the
  // vote brings them together again, and to one outcome, before the aligned
  // instructions that follow.  (The 2048-query chunk takes 435 us with it and 437
  // without at D = 128, 409 and 400 at D = 64.)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xFFFFFFFFu, mbar_wait_lean(bar, parity & 1))) return true;
    atomicAdd(&g_kv_wait_timeouts, 1u);
    sm.gave_up = 1;
    return false;
  };
  auto arrive = [&](uint64_t* bar) {                             // of a whole warp, as one
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (wg < 2) {
    // ================= softmax of 128 rows, one per thread =================
    regs_inc<kSoftmaxRegs>();
    [&]() {
      const int rl = threadIdx.x & 127;              // row within the warpgroup, tensor-memory lane
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      constexpr int CPR = D / 8, RPI = 32 / CPR;     // 16-byte chunks of a bf16 row; rows in 32 lanes' worth
      const uint32_t t_s0 = tmem + lanes + kS + wg * 128, t_o = tmem + lanes + kO + wg * 128;
      uint32_t kt = 0, mine_t = 0, items = 0;   // tiles of the CTA, tiles and items of this warpgroup
      uint32_t joins = 0, all_n = 0;                 // phases of join_last, join_all
      for (bool more = unit0() < unit1(); more; more = advance()) {
        const int u0 = unit0(), u1 = unit1();
        const int row0 = it.rt * kPrRows + wg * 128, r = row0 + rl;
        const bool active = row0 < it.rows, on = r < it.rows;
        const int qi = on ? a.by_group.div(r) : 0, g = on ? r - qi * a.group : 0;
        const int pos = on ? it.sq.pos0 + qi : -1;
        const int first_pos = it.sq.pos0 + a.by_group.div(row0);
        const int last_pos = it.sq.pos0 + a.by_group.div(min(it.rows, row0 + 128) - 1);
        float f_row = 0.0f, m_ref = kNoMax, l = 0.0f;
        uint32_t nan_blocks = 0;
        if (active) {
          // q: f16, each row scaled by a power of two to a largest magnitude in
          // [2^14, 2^15).  A warp takes its 32 rows RPI at a time, 16 bytes a lane.
          f_row = 0.0f;
          constexpr int QN = 32 / RPI < 8 ? 32 / RPI : 8;          // loads in flight
#pragma unroll 1
          for (int x0 = 0; x0 < 32 / RPI; x0 += QN) {
            const int c = lane % CPR, rw0 = (warp & 3) * 32 + x0 * RPI + lane / CPR;
            uint4 w[QN];
#pragma unroll
            for (int x = 0; x < QN; ++x) {
              const int rr = row0 + rw0 + x * RPI, i = a.by_group.div(rr);
              w[x] = make_uint4(0, 0, 0, 0);
              if (rr < it.rows)
                w[x] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                       (int64_t)(it.sq.q0 + i) * a.q_tok +
                                                       (int64_t)(it.head * a.group + rr - i * a.group) * a.q_head + c * 8);
            }
#pragma unroll
            for (int x = 0; x < QN; ++x) {
              uint32_t m = unpack_max<FP8Q_BF16>(absmax_load<FP8Q_BF16>(w[x]));
#pragma unroll
              for (int y = 1; y < CPR; y <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, y));
              const int e = m == 0 ? 0 : max(-112, (int)(m >> 23) - 127) - 14;
              // 2^-e; NaN or Inf: every score of the row is NaN, but those the masks
              // replace.  (Picked as bits: between floats, four ragged prompts take
              // 269 us and not 260.)
              const float s = __uint_as_float(m >= 0x7F800000u ? 0x7FFFFFFFu : (uint32_t)(127 - e) << 23);
              float f = a.scale * 1.4426950408889634f * pow2f(e);
              f = __shfl_sync(0xFFFFFFFFu, f, (lane % RPI) * CPR);
              if (lane / RPI == x0 + x) f_row = f;
              uint4 h;
              h.x = cvt_f16x2(__uint_as_float(w[x].x << 16) * s, __uint_as_float(w[x].x & 0xFFFF0000u) * s);
              h.y = cvt_f16x2(__uint_as_float(w[x].y << 16) * s, __uint_as_float(w[x].y & 0xFFFF0000u) * s);
              h.z = cvt_f16x2(__uint_as_float(w[x].z << 16) * s, __uint_as_float(w[x].z & 0xFFFF0000u) * s);
              h.w = cvt_f16x2(__uint_as_float(w[x].w << 16) * s, __uint_as_float(w[x].w & 0xFFFF0000u) * s);
              const int row = rw0 + x * RPI;
              *reinterpret_cast<uint4*>(sm.q[wg] + (c >> 3) * Smem::kQHalf + row * 128 + (((c & 7) ^ (row & 7)) * 16)) = h;
            }
          }
          fence_proxy_async();
          arrive(&sm.q_full[wg]);
          ++items;
          // The item's first scores, before its first unit's scales and masks.  A
          // warpgroup that skipped units may be any number of phases ahead of
          // info_full, where the parity says nothing; once its scores are made, the
          // unpacking warps are past unit kt - 4, the slot's one before (kt - 1 for
          // the values, whose stage the issuing warp has waited for), and cannot be
          // at kt + 4.  From unit to unit that stays so.  (It cost the 2048-query
          // chunk 1.5 us of 436; with this order in every unit, so that the masks'
          // test follows the scores, 18.)
          if (!wait(&sm.s_full[wg][0], mine_t)) return;
        }
        for (int u = u0; u < u1; ++u, ++kt) {
          if (!active) continue;
          const int tok = (it.tile0 + u) * kPrKeys;
          if (!wait(&sm.info_full[kt % kPrInfos], kt / kPrInfos)) return;
          const PrInfo& info = sm.info[kt % kPrInfos];
          bool edge = tok + kPrKeys - 1 > first_pos || (a.window > 0 && tok <= last_pos - a.window);
          {
            const uint4 all = *reinterpret_cast<const uint4*>(info.valid), nan = *reinterpret_cast<const uint4*>(info.any_nan);
            edge |= (all.x & all.y & all.z & all.w) != 0xFFFFFFFFu || (nan.x | nan.y | nan.z | nan.w) != 0;
          }
          // 16 scores from column c on: what this row does not see becomes -inf
          auto mask = [&](int c, uint32_t (&v)[16]) {
            const int x = c >> 5, base = tok + x * 32;
            uint32_t m = info.valid[x] & low_bits(pos - base + 1);
            if (a.window > 0) m &= ~low_bits(pos - a.window + 1 - base);
            m = (m >> (c & 16)) & 0xFFFFu;
#pragma unroll
            for (int y = 0; y < 16; ++y) v[y] = (m >> y) & 1 ? v[y] : 0xFF800000u;
            if (info.any_nan[x])
              for (int y = 0; y < NB; ++y) nan_blocks |= ((info.vnan[x][y] >> (c & 16)) & m) ? 1u << y : 0u;
          };
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (!wait(&sm.s_full[wg][h], mine_t)) return;
            tmem_fence_after();
            const uint32_t t_s = t_s0 + h * kPrHalf;
            // Weights are made against the reference of the tiles before, in one
            // pass over the scores.  Where their sum passes kMostSum (then some
            // weight might not fit f16), and on an item's first scores, the
            // reference moves to the largest score first and the scores, still
            // in place, are read once more.
            uint32_t p[kPrHalf / 2];
            bool again = u == u0 && h == 0;
            while (true) {
              if (again) {
                float top = m_ref;
#pragma unroll 1
                for (int x = 0; x < kPrHalf / 16; ++x) {
                  const int c = h * kPrHalf + x * 16;
                  uint32_t v[16];
                  tmem_ld16(v, t_s + x * 16);
                  tmem_wait_ld(v);
                  if (edge) mask(c, v);
                  float t = __uint_as_float(v[0]);
#pragma unroll
                  for (int y = 1; y < 15; y += 2) t = max3(t, __uint_as_float(v[y]), __uint_as_float(v[y + 1]));
                  t = fmaxf(t, __uint_as_float(v[15]));
                  top = fmaxf(top, t * fmaxf(f_row * info.rk[c >> 5], kMinFactor) + info.rv[c >> 5]);
                }
                const float fix = ex2(m_ref - top);
                m_ref = top;
                l *= fix;
                if (u > u0 || h > 0) {                 // the sums so far, once the product that made them is done
                  if (!wait(&sm.o_full[wg][h ^ 1], h ? mine_t : mine_t - 1)) return;
                  tmem_fence_after();
#pragma unroll 1
                  for (int x = 0; x < D / 16; ++x) {
                    uint32_t o[16];
                    tmem_ld16(o, t_o + x * 16);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * fix);
                    tmem_st16(t_o + x * 16, o);
                  }
                }
              }
              uint32_t s[2][16];
              float sum_p = 0.0f, sum_l = 0.0f;
              tmem_ld16(s[0], t_s);
              const float2 rk = reinterpret_cast<const float2*>(info.rk)[h], rv = reinterpret_cast<const float2*>(info.rv)[h];
              const float2 un = reinterpret_cast<const float2*>(info.unscale)[h];
#pragma unroll
              for (int x = 0; x < kPrHalf / 16; ++x) {
                uint32_t(&v)[16] = s[x & 1];
                tmem_wait_ld(v);
                if (x + 1 < kPrHalf / 16) tmem_ld16(s[(x + 1) & 1], t_s + (x + 1) * 16);
                if (edge) mask(h * kPrHalf + x * 16, v);
                const float f1 = f_row * (x < 2 ? rk.x : rk.y), f = f1 < kMinFactor ? kMinFactor : f1, c = (x < 2 ? rv.x : rv.y) - m_ref;
                const uint64_t f2 = pack2(f, f), c2 = pack2(c, c);
                uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                for (int y = 0; y < 16; y += 4) {
                  float e0, e1, e2, e3;
                  unpack2(fma2(pack2(__uint_as_float(v[y]), __uint_as_float(v[y + 1])), f2, c2), e0, e1);
                  unpack2(fma2(pack2(__uint_as_float(v[y + 2]), __uint_as_float(v[y + 3])), f2, c2), e2, e3);
                  e0 = ex2(e0);
                  e1 = ex2(e1);
                  e2 = ex2(e2);
                  e3 = ex2(e3);
                  sum0 = add2(sum0, pack2(e0, e1));
                  sum1 = add2(sum1, pack2(e2, e3));
                  p[x * 8 + y / 2] = cvt_f16x2(e0, e1);
                  p[x * 8 + y / 2 + 1] = cvt_f16x2(e2, e3);
                }
                float a0, a1;
                unpack2(add2(sum0, sum1), a0, a1);
                sum_p += a0 + a1;
                sum_l += (a0 + a1) * (x < 2 ? un.x : un.y);
              }
              if (again || !__any_sync(0xFFFFFFFFu, sum_p > kMostSum)) {
                l += sum_l;
                break;
              }
              again = true;
            }
            tmem_st32(t_s, p);                         // over the scores
            tmem_wait_st();
            tmem_fence_before();
            arrive(&sm.p_full[wg][h]);
          }
          ++mine_t;
        }

        // ---- the item's end: output, or a part to be joined
        const bool whole = u0 == 0 && u1 == it.n;
        constexpr int PART = kPrRows * (D + 2);
        float* part = plan.part + (2 * (long long)blockIdx.x + (rel + kPrSetup <= 0 ? 0 : 1)) * PART;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t out_row = it.sq.q0 + qi;
        const int out_head = it.head * a.group + g;
        if (active) {
          if (!wait(&sm.o_full[wg][1], mine_t - 1)) return;
          tmem_fence_after();
          // Through shared memory (the queries' place: the products are done with
          // them), so that rows leave RPI at a time: 16-byte chunk c of row r at
          // chunk c ^ (r & 7).  Outputs are bf16, parts fp32 in two halves.
          uint4* stage = reinterpret_cast<uint4*>(sm.q[wg]) + (warp & 3) * 32 * CPR;
          const int c = lane % CPR;
#pragma unroll 1
          for (int z = 0; z < (whole ? 1 : 2); ++z) {
#pragma unroll 1
            for (int x = 0; x < (whole ? D / 32 : D / 64); ++x) {
              const int col = z * (D / 2) + x * 32;
              uint32_t o[32];
              tmem_ld32(o, t_o + col);
              tmem_wait_ld(o);
              if ((nan_blocks >> (col >> 5)) & 1)
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = 0x7FFFFFFFu;
              if (whole) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  uint32_t w[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    w[k] = l == 0.0f ? 0u : cvt_bf16x2(__uint_as_float(o[y * 8 + k * 2]) * inv,
                                                       __uint_as_float(o[y * 8 + k * 2 + 1]) * inv);
                  stage[lane * CPR + ((x * 4 + y) ^ (lane & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
                }
              } else {
#pragma unroll
                for (int y = 0; y < 8; ++y)
                  stage[lane * CPR + ((x * 8 + y) ^ (lane & 7))] = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
              }
            }
            __syncwarp();
#pragma unroll 4
            for (int x = 0; x < 32 / RPI; ++x) {
              const int rw = x * RPI + lane / CPR, rr = row0 + (warp & 3) * 32 + rw;
              if (rr >= it.rows) continue;
              const uint4 v = stage[rw * CPR + (c ^ (rw & 7))];
              if (whole) {
                const int i = a.by_group.div(rr);
                *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)(it.sq.q0 + i) * a.out_tok +
                                          (int64_t)(it.head * a.group + rr - i * a.group) * a.out_head + c * 8) = v;
              } else {
                *reinterpret_cast<uint4*>(part + (rr - it.rt * kPrRows) * D + z * (D / 2) + c * 4) = v;
              }
            }
            __syncwarp();
          }
          if (on && whole) store_lse(a, out_row, out_head, m_ref, l);
          if (on && !whole) {
            part[kPrRows * D + wg * 128 + rl] = m_ref;
            part[kPrRows * D + kPrRows + wg * 128 + rl] = l;
          }
          tmem_fence_before();
        }
        if (!whole) {
          const long long per = s_range[1], seg0 = s_range[0] + rel + kPrSetup, first = seg0 / per, last = (seg0 + it.n - 1) / per;
          arrive(&sm.join_all);
          if (warp == 0 && !wait(&sm.join_all, all_n)) return;
          if (threadIdx.x == 0) {
            // a CTA starts at most one that others go on with
            sm.last = take_ticket(plan.ticket + first, (uint32_t)(last - first), 0);
            ++sm.taken;
            mbar_arrive(&sm.join_last);
          }
          __syncwarp();
          if (!wait(&sm.join_last, joins++)) return;
          ++all_n;
          if (*reinterpret_cast<volatile uint32_t*>(&sm.last)) {
            const int n = (int)(last - first) + 1;
            const int here = min(kPrRows, it.rows - it.rt * kPrRows);
            auto part_at = [&](int i) {
              const long long c = first + i;
              return static_cast<const float*>(plan.part) + (2 * c + (seg0 <= c * per ? 0 : 1)) * PART;
            };
            // the products are done with this item's queries: their place takes
            // the rows' references and sums
            Joined* rows = reinterpret_cast<Joined*>(sm.q[0]);
            if (static_cast<int>(threadIdx.x) < here) {
              const int row = it.rt * kPrRows + threadIdx.x, i = a.by_group.div(row);
              const Joined x = row_of_parts<kPrRows, D>(part_at, 0, 1, n, threadIdx.x);
              rows[threadIdx.x] = x;
              store_lse(a, it.sq.q0 + i, it.head * a.group + row - i * a.group, x.m, x.l);
            }
            arrive(&sm.join_all);
            if (!wait(&sm.join_all, all_n++)) return;
            constexpr int U = 8, STEP = 256 / (D / 4);
            const int c = threadIdx.x % (D / 4);
            for (int r0 = threadIdx.x / (D / 4); r0 < here; r0 += U * STEP) {
              int r[U];
              float m[U];
              float4 o[U];
#pragma unroll
              for (int x = 0; x < U; ++x) {
                r[x] = min(r0 + x * STEP, here - 1);
                m[x] = rows[r[x]].m;
              }
              columns_of_parts<kPrRows, D, U, 1>(part_at, n, r, c, m, o);
#pragma unroll
              for (int x = 0; x < U; ++x) {
                if (r0 + x * STEP >= here) continue;
                const int row = it.rt * kPrRows + r[x], i = a.by_group.div(row);
                store_columns(a, it.sq.q0 + i, it.head * a.group + row - i * a.group, c, o[x], rows[r[x]].l);
              }
            }
            arrive(&sm.join_all);                      // the queries' place is free again
            if (!wait(&sm.join_all, all_n++)) return;
          }
        }
      }
    }();
  } else if (wg < 4) {
    // ================= unpacking keys and values =================
    regs_dec<kUnpackRegs>();
    [&]() {
      const bool values = wg == 3;                   // a warpgroup for keys, one for values
      const int grp = warp & 3;                      // tokens 32 grp .. + 31 of a unit
      const int sub = lane & 7;                      // token of 8 within a step
      // a lane's units are the 16-byte blocks blk of U tokens: eight lanes write
      // the same chunk of eight rows, which the swizzle spreads over all banks
      constexpr int U = D == 128 ? 4 : 2;
      const int blk = D == 128 ? lane >> 3 : (lane >> 3) & 1;
      auto token_of = [&](int j) { return D == 128 ? j * 8 + sub : j * 16 + (lane >> 4) * 8 + sub; };
      const int page_mask = (1 << a.shape.page_shift) - 1;
      const KvPool pool = values ? a.v : a.k;
      int u = unit0(), u_end = unit1();              // unit of the item, the last that is this CTA's
      if (u >= u_end) return;
      typename Smem::Raw& raw = sm.raw[warp - 8];
      // pages of 32 tokens or more hold a group's rows in one run; smaller ones
      // are looked up by each lane for its own token
      const bool runs = a.shape.page_shift >= 5;
      auto page_of = [&]() {
        const int tok = (it.tile0 + u) * kPrKeys + grp * 32 + (runs ? 0 : lane);
        return tok < it.sq.len ? a.table[it.b * a.table_stride + (tok >> a.shape.page_shift)] : -1;
      };
      // starts the copy of this warp's rows of the unit; gives the mask of those that exist
      auto fetch = [&](int page) {
        const int at = (it.tile0 + u) * kPrKeys + grp * 32, tok = at + (runs ? 0 : lane);
        const bool ok = (uint32_t)page < (uint32_t)a.shape.pages;
        const int64_t row = ok ? kv_row(a.shape, page, tok & page_mask, it.head) : 0;
        uint32_t there;
        if (runs) {
          const int n = ok ? min(it.sq.len - at, 32) : 0;
          there = low_bits(n);
          copy_run<D, false>(smem_addr(raw.codes), smem_addr(raw.scales), pool, row, n);
        } else {
          there = __ballot_sync(0xFFFFFFFFu, ok);
          copy_rows<D, false>(smem_addr(raw.codes), smem_addr(raw.scales), pool, row, there, a.shape.page_shift);
        }
        cp_commit();
        return there;
      };

      // The items' units in turn.  A unit's codes go to registers as soon as
      // they have arrived, and the copy of the next one starts at once.
      auto step = [&]() {                            // one unit on; false past the last
        if (++u < u_end) return true;
        if (!advance()) return false;
        u = 0;
        u_end = unit1();
        return true;
      };
      uint32_t next = fetch(page_of());
      bool more = step();
      int page = more ? page_of() : -1;
      uint64_t* full = values ? sm.v_full : sm.k_full;
      uint64_t* empty = values ? sm.v_empty : sm.k_empty;
      for (int kt = 0;; ++kt) {
        PrInfo& info = sm.info[kt % kPrInfos];
        const int stg = kt % kPrStages;
        cp_wait<0>();
        __syncwarp();
        const uint32_t valid = next;
        uint4 codes[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
          codes[j] = *reinterpret_cast<const uint4*>(raw.codes + code_offset<D>(token_of(j), blk));
        // scales of the lane's token; the pair copy may have brought those of a token that does not exist
        uint32_t sc = NB == 4 ? reinterpret_cast<const uint32_t*>(raw.scales)[lane]
                              : reinterpret_cast<const uint16_t*>(raw.scales)[lane];
        sc = (valid >> lane) & 1 ? sc : 0u;
        __syncwarp();
        const bool last = !more;
        if (more) {
          next = fetch(page);
          more = step();
          if (more) page = page_of();
        }
        if (kt >= kPrStages && !wait(&empty[stg], kt / kPrStages - 1)) return;

        // the group's largest block scale 2^R
        uint32_t top = 0;
        bool bad = false;
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          const uint32_t e = (sc >> (8 * x)) & 0xFFu;
          bad |= e == 255u;
          top = max(top, e == 255u ? 0u : e);
        }
        top = __reduce_max_sync(0xFFFFFFFFu, top);   // tokens that do not exist have scale bytes 0
        top = min(max(top, values ? kMinScale : 1u), kMaxScale);      // keys: 2^Rk is a normal number
        if (values) {
          const uint32_t any = __ballot_sync(0xFFFFFFFFu, bad);
          if (any) {
#pragma unroll
            for (int x = 0; x < NB; ++x) {
              const uint32_t m = __ballot_sync(0xFFFFFFFFu, ((sc >> (8 * x)) & 0xFFu) == 255u);
              if (lane == 0) info.vnan[grp][x] = m;
            }
          }
          if (lane == 0) {
            info.any_nan[grp] = any;
            info.rv[grp] = (float)((int)top - 127);
            info.unscale[grp] = pow2f(127 - (int)top);
          }
        } else if (lane == 0) {
          info.rk[grp] = pow2f((int)top - 127);
          info.valid[grp] = valid;
        }
        if (lane == 0) mbar_arrive(&sm.info_full[kt % kPrInfos]);

        // codes * 2^(E - R) into the swizzled tile
        uint8_t* tile = (values ? sm.v[stg] : sm.k[stg]) + (blk >> 1) * Smem::kHalf + grp * 32 * 128;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int t = token_of(j);
          const uint32_t e = (__shfl_sync(0xFFFFFFFFu, sc, t) >> (8 * blk)) & 0xFFu;
          const int d = min(126, (int)(top - e));
          float f = __uint_as_float((uint32_t)(127 - d) << 23);
          // a NaN block of keys is NaN to every row that sees the token; one of
          // values would reach rows that do not, so it goes by the flags
          if (e == 255u) f = values ? 0.0f : __uint_as_float(0x7FFFFFFFu);
          const uint32_t f2 = cvt_f16x2(f, f);
          const uint32_t ws[4] = {codes[j].x, codes[j].y, codes[j].z, codes[j].w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t h[4];
            e2m1x8_f16(ws[x], h);
            *reinterpret_cast<uint4*>(tile + t * 128 + ((((blk & 1) * 4 + x) ^ sub) * 16)) =
                make_uint4(mul_f16x2(h[0], f2), mul_f16x2(h[1], f2), mul_f16x2(h[2], f2), mul_f16x2(h[3], f2));
          }
        }
        fence_proxy_async();
        arrive(&full[stg]);
        if (last) return;
      }
    }();
    cp_wait<0>();                                    // no copy outlives its warp
  } else {
    // ================= two warps issue the products, one for each 128 rows =================
    // Issuing blocks while the tensor cores are busy, and a wait costs about 80
    // clocks even where nothing is waited for; with a warp each, one side's waits
    // pass while the other's products run.  The whole warp goes through the
    // loop, so that addresses and descriptors stay in uniform registers; one
    // elected lane issues.
    regs_dec<kIssueRegs>();
    if (warp < kPrIssuer + 2) {
      [&]() {
        constexpr uint32_t kQK = f16_idesc(128, kPrHalf, false), kPV = f16_idesc(128, D, true);
        constexpr uint32_t kHi = desc_hi(1024), kHalfBytes = kPrHalf * 128;
        const int w = __shfl_sync(0xFFFFFFFFu, warp - kPrIssuer, 0);
        const uint32_t qa = desc_lo(smem_addr(sm.q[w]), 16), ka = desc_lo(smem_addr(sm.k[0]), 16);
        const uint32_t va = desc_lo(smem_addr(sm.v[0]), Smem::kHalf);
        const bool lead = elect_one();
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0) + w * 128;
        uint32_t kt = 0, items = 0, mine_t = 0;       // units of the CTA; this side's items and units
        auto scores = [&](uint32_t stg, int h) {
          const uint32_t k = ka + ((stg * Smem::kTileBytes + h * kHalfBytes) >> 4), d = tm + kS + h * kPrHalf;
          if (lead) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
              mma_ss(d, qa + (((x >> 2) * Smem::kQHalf + (x & 3) * 32) >> 4),
                     k + (((x >> 2) * Smem::kHalf + (x & 3) * 32) >> 4), kHi, kQK, x > 0);
            mma_commit(&sm.s_full[w][h]);
            if (h) mma_commit(&sm.k_empty[stg]);
          }
          __syncwarp();
        };
        auto values = [&](uint32_t stg, int h, bool first) {
          const uint32_t v = va + ((stg * Smem::kTileBytes + h * kHalfBytes) >> 4), p = tm + kS + h * kPrHalf;
          if (lead) {
#pragma unroll
            for (int x = 0; x < kPrHalf / 16; ++x)
              mma_ts(tm + kO, p + x * 8, v + x * (2048 >> 4), kHi, kPV, !first || x > 0);
            mma_commit(&sm.o_full[w][h]);
            if (h) mma_commit(&sm.v_empty[stg]);
          }
          __syncwarp();
        };
        // Each half's scores of the next unit are made as soon as the weights
        // that lie over them have been used, while the other half is in work.
        for (bool go = unit0() < unit1(); go; go = advance()) {
          const int n = unit1() - unit0();
          const bool active = it.rt * kPrRows + w * 128 < it.rows;
          if (active) {
            if (!wait(&sm.q_full[w], items++)) return;
            if (!wait(&sm.k_full[kt % kPrStages], kt / kPrStages)) return;
            tmem_fence_after();
            scores(kt % kPrStages, 0);
            scores(kt % kPrStages, 1);
            for (int u = 0; u < n; ++u, ++kt, ++mine_t) {
              const uint32_t stg = kt % kPrStages, nk = kt + 1, ns = nk % kPrStages;
              if (!wait(&sm.v_full[stg], kt / kPrStages)) return;
              if (!wait(&sm.p_full[w][0], mine_t)) return;
              tmem_fence_after();
              values(stg, 0, u == 0);
              if (u + 1 < n) {
                if (!wait(&sm.k_full[ns], nk / kPrStages)) return;
                scores(ns, 0);
              }
              if (!wait(&sm.p_full[w][1], mine_t)) return;
              tmem_fence_after();
              values(stg, 1, false);
              if (u + 1 < n) scores(ns, 1);
            }
          } else {                                   // no such rows: the stages still need this side's word
            for (int u = 0; u < n; ++u, ++kt) {
              const uint32_t stg = kt % kPrStages;
              if (!wait(&sm.k_full[stg], kt / kPrStages)) return;
              if (lane == 0) mbar_arrive(&sm.k_empty[stg]);
              if (!wait(&sm.v_full[stg], kt / kPrStages)) return;
              if (lane == 0) mbar_arrive(&sm.v_empty[stg]);
              __syncwarp();
            }
          }
        }
      }();
      // nothing may still be running when the tensor memory goes back
      if (elect_one()) mma_commit(&sm.drain);
      __syncwarp();
      wait(&sm.drain, 0);
    }
    __syncwarp();
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == kPrIssuer) {
    tmem_fence_after();
    tmem_free(tmem, 512);
  }
  // A CTA that gave up still takes the tickets of the parts it owes, so that
  // none outlives the call: by a warp that had no role and is at the first item.
  if (warp == kPrIssuer + 2 && sm.gave_up) {
    uint32_t parts = 0;
    for (bool go = unit0() < unit1(); go; go = advance()) {
      if (unit0() == 0 && unit1() == it.n) continue;
      if (lane == 0 && parts >= sm.taken) {
        const long long per = s_range[1], seg0 = s_range[0] + rel + kPrSetup, first = seg0 / per;
        take_ticket(plan.ticket + first, (uint32_t)((seg0 + it.n - 1) / per - first), kGaveUp);
      }
      ++parts;
    }
  }
}

// ---- host side ---------------------------------------------------------------

template <int D>
static int pr_smem() {
  return (int)sizeof(PrSmem<D>) + 1024;
}

static int pr_grid(const KvShape& s, int group, int batch, int64_t total_q, int max_q, int table_width, int sms) {
  const int64_t by_max = (int64_t)batch * (((int64_t)max_q * group + kPrRows - 1) / kPrRows);
  const int64_t by_total = total_q * group / kPrRows + batch;
  const int64_t units = (((int64_t)table_width << s.page_shift) + kPrKeys - 1) / kPrKeys;
  const int64_t all = (by_max < by_total ? by_max : by_total) * s.heads * (units + kPrSetup);
  const int64_t most = (all + kPrMinUnits - 1) / kPrMinUnits;
  const int64_t n = most < sms ? most : sms;
  return (int)(n < kMaxGrid ? n : kMaxGrid);
}

static bool pr_regs_ok(const void* kernel) {
  cudaFuncAttributes f;
  return cudaFuncGetAttributes(&f, kernel) == cudaSuccess && f.numRegs >= kPrRegs;
}

static int64_t pr_bytes(int grid, int dim) {
  return grid < 2 ? 0 : kMaxGrid * 4 + (int64_t)grid * 2 * kPrRows * (dim + 2) * 4;
}

cudaError_t kv_prompt_workspace(const KvShape& s, int group, int batch, int64_t total_q, int max_q, int table_width,
                                int sms, int64_t* bytes) {
  const int grid = pr_grid(s, group, batch, total_q, max_q, table_width, sms);
  *bytes = pr_bytes(grid, s.dim);
  return cudaSuccess;
}

cudaError_t launch_kv_prompt(const KvAttn& a, const KvWork& w, int sms, cudaStream_t st, int* status, int* launches) {
  const int grid = pr_grid(a.shape, a.group, a.batch, a.total_q, a.max_q, a.table_width, sms);
  const void* k = a.shape.dim == 128 ? reinterpret_cast<const void*>(kv_prompt_kernel<128>)
                                     : reinterpret_cast<const void*>(kv_prompt_kernel<64>);
  const int smem = a.shape.dim == 128 ? pr_smem<128>() : pr_smem<64>();
  int occ = 1;
  cudaError_t e = kernel_occupancy(k, kPrThreads, smem, &occ);
  if (e != cudaSuccess) return e;
  *status = w.check(pr_bytes(grid, a.shape.dim));
  if (*status != FP8Q_OK) return cudaSuccess;
  // built with fewer registers than the shares count on, it is not launched
  static const bool regs64 = pr_regs_ok(reinterpret_cast<const void*>(kv_prompt_kernel<64>));
  static const bool regs128 = pr_regs_ok(reinterpret_cast<const void*>(kv_prompt_kernel<128>));
  if (!(a.shape.dim == 128 ? regs128 : regs64)) return cudaErrorInvalidKernelImage;
  PrPlan plan = {w.tickets(), w.parts()};
  void* args[2] = {const_cast<KvAttn*>(&a), &plan};
  return launch_dependent(k, dim3(grid), kPrThreads, smem, args, st, launches);
}

cudaError_t read_kv_wait_timeouts(unsigned int* count) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_kv_wait_timeouts, sizeof *count);
  const unsigned int zero = 0;
  if (e == cudaSuccess && *count) e = cudaMemcpyToSymbol(g_kv_wait_timeouts, &zero, sizeof zero);
  return e;
}

}  // namespace fp8q
