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
// What bounds it: 4 D flops per visible pair on the tensor cores (4096 f16
// multiply-adds a clock and SM), against one exponential (32 a clock) and
// about six other instructions per pair, and 2 x 16 K elements to unpack per
// tile of 128 tokens.
//
// Layout: one CTA per SM.  Two warpgroups hold the softmax of 128 rows each
// (rows are query tokens times the heads that share a key/value head; one row
// per thread, scores read from tensor memory at once), a third unpacks keys
// and values into two-stage rings of 128-byte-swizzled tiles, and one thread
// issues the products in turn, scores of one warpgroup's rows while the other
// one's weights are made.  Weights return to tensor memory over the scores
// (f16, the A operand of the second product); values are the B operand with D
// consecutive, so neither is transposed.
//
// Work is split as in kv_decode.cu: CTA i takes units [i * per, (i + 1) * per)
// of 128 keys x 256 rows in (sequence, head, rows) order, and what spans CTAs
// is joined by the last of them to arrive.
#include "kv_device.cuh"
#include "tcgen05.cuh"

namespace fp8q {

constexpr int kPrThreads = 512;
constexpr int kPrRows = 256;              // query rows of an item: two warpgroups of 128
constexpr int kPrKeys = 128;              // keys of a unit
constexpr int kPrMinUnits = 4;            // units of a CTA, at least

__device__ unsigned int g_kv_wait_timeouts = 0;

struct PrInfo {                           // per tile, written by the unpacking warps
  float rk[4];                            // 2^Rk of each 32 tokens
  float rv[4];                            // Rv
  uint32_t valid[4];                      // tokens that exist
  uint32_t any_nan[4];                    // tokens with a NaN block of values,
  uint32_t vnan[4][4];                    // and with block b NaN (set where any_nan is not 0)
};

template <int D>
struct PrSmem {
  static constexpr int kHalf = 128 * 128;             // 128 rows of 64 f16
  static constexpr int kTileBytes = kHalf * (D / 64);
  uint8_t q[2][kTileBytes];
  uint8_t k[2][kTileBytes];
  uint8_t v[2][kTileBytes];
  PrInfo info[4];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2];     // per warpgroup of rows
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];   // per stage
  uint64_t join_all, join_last, drain;
  uint32_t tmem, last;
};

// One item: 256 rows of one (sequence, head) and the units of 128 keys that
// some of the rows see.
struct PrItem {
  KvSeq sq;
  int b, head, rt;          // sequence, head, row tile
  int rows, tiles_r;        // rows of the (sequence, head), row tiles
  int tile0, n;             // first 128 keys, units
};
__device__ __forceinline__ void pr_units(const KvAttn& a, const KvSeq& s, int rt, int* tile0, int* n) {
  const int rows = s.nq * a.group;
  const int first = rt * kPrRows / a.group, last = (min(rows, (rt + 1) * kPrRows) - 1) / a.group;
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

// Low n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }

template <int D>
__global__ void __launch_bounds__(kPrThreads, 1)
kv_prompt_kernel(const __grid_constant__ KvAttn a, const __grid_constant__ PrPlan plan) {
  using Smem = PrSmem<D>;
  constexpr int NB = D / 32;
  constexpr uint32_t kS = 0, kO = 256;               // tensor-memory columns of warpgroup 0 (+ 128 for 1)
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wg = warp >> 2;

  // ---- this CTA's range of units
  __shared__ long long s_scan[kPrThreads / 32];
  __shared__ long long s_first[2];                   // begin's (sequence, its first unit)
  constexpr int W = kPrThreads / 32;
  const int per_warp = (a.batch + W - 1) / W;
  const int b_lo = min(a.batch, warp * per_warp), b_hi = min(a.batch, b_lo + per_warp);
  auto seq_units = [&](const KvSeq& s) {             // of one head; the whole warp calls it
    const int tiles_r = (int)(((long long)s.nq * a.group + kPrRows - 1) / kPrRows);
    long long u = 0;
    for (int rt = lane; rt < tiles_r; rt += 32) {
      int t0, n;
      pr_units(a, s, rt, &t0, &n);
      u += n;
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
      mbar_init(&sm.q_full[x], 128);
      mbar_init(&sm.s_full[x], 1);
      mbar_init(&sm.p_full[x], 128);
      mbar_init(&sm.o_full[x], 1);
      mbar_init(&sm.k_full[x], 128);
      mbar_init(&sm.k_empty[x], 1);
      mbar_init(&sm.v_full[x], 128);
      mbar_init(&sm.v_empty[x], 1);
    }
    mbar_init(&sm.join_all, 256);
    mbar_init(&sm.join_last, 1);
    mbar_init(&sm.drain, 1);
    fence_barrier_init();
  }
  if (warp == 12) tmem_alloc(&sm.tmem, 512);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = sm.tmem;

  PrItem it;
  it.b = (int)s_first[0];
  long long seg0 = s_first[1];                       // global unit of the item's first one
  it.sq = kv_seq(a, it.b);
  pr_set(a, it);
  {
    const long long u = seq_units(it.sq);
    it.head = (int)((begin - seg0) / u);
    seg0 += it.head * u;
    it.rt = 0;
    pr_units(a, it.sq, 0, &it.tile0, &it.n);
    while (begin >= seg0 + it.n) {
      seg0 += it.n;
      ++it.rt;
      pr_units(a, it.sq, it.rt, &it.tile0, &it.n);
    }
  }

  // Every wait is bounded; a role whose wait runs out counts it and returns,
  // and so do the others in turn, to the common end.
  auto wait1 = [&](uint64_t* bar, uint32_t parity) {             // one thread
    if (mbar_wait(bar, parity & 1)) return true;
    atomicAdd(&g_kv_wait_timeouts, 1u);
    return false;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {              // a whole warp: one answer for all its lanes
    return __all_sync(0xFFFFFFFFu, wait1(bar, parity)) != 0;
  };

  if (wg < 2) {
    // ================= softmax of 128 rows, one per thread =================
    regs_inc<144>();
    [&]() {
      const int rl = threadIdx.x & 127;              // row within the warpgroup, tensor-memory lane
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t t_s = tmem + lanes + kS + wg * 128, t_o = tmem + lanes + kO + wg * 128;
      uint32_t kt = 0, mine_t = 0, items = 0, joins = 0;   // tiles of the CTA, tiles and items of this warpgroup
      for (long long at = begin; at < end;) {
        const int u0 = (int)(at - seg0), u1 = (int)min((long long)it.n, end - seg0);
        const int row0 = it.rt * kPrRows + wg * 128, r = row0 + rl;
        const bool active = row0 < it.rows, on = r < it.rows;
        const int qi = on ? r / a.group : 0, g = on ? r - qi * a.group : 0;
        const int pos = on ? it.sq.pos0 + qi : -1;
        const int first_pos = it.sq.pos0 + row0 / a.group;
        const int last_pos = it.sq.pos0 + (min(it.rows, row0 + 128) - 1) / a.group;
        float f_row = 0.0f, m_ref = kNoMax, l = 0.0f;
        uint32_t nan_blocks = 0;
        if (active) {
          // q: f16, scaled by a power of two to a largest magnitude in [2^14, 2^15)
          const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.q) +
                                                          (int64_t)(it.sq.q0 + qi) * a.q_tok +
                                                          (int64_t)(it.head * a.group + g) * a.q_head);
          uint32_t m = 0;
          if (on)
#pragma unroll 4
            for (int x = 0; x < D / 8; ++x) m = vmax_u16x2(m, absmax_load<FP8Q_BF16>(q[x]));
          m = unpack_max<FP8Q_BF16>(m);
          const int e = m == 0 ? 0 : max(-112, (int)(m >> 23) - 127) - 14;
          const float s = pow2f(-e);
          f_row = a.scale * 1.4426950408889634f * pow2f(e);
          if (m >= 0x7F800000u) f_row = __uint_as_float(0x7FFFFFFFu);
#pragma unroll 4
          for (int x = 0; x < D / 8; ++x) {
            const uint4 w = on ? q[x] : make_uint4(0, 0, 0, 0);
            uint4 h;
            h.x = cvt_f16x2(__uint_as_float(w.x << 16) * s, __uint_as_float(w.x & 0xFFFF0000u) * s);
            h.y = cvt_f16x2(__uint_as_float(w.y << 16) * s, __uint_as_float(w.y & 0xFFFF0000u) * s);
            h.z = cvt_f16x2(__uint_as_float(w.z << 16) * s, __uint_as_float(w.z & 0xFFFF0000u) * s);
            h.w = cvt_f16x2(__uint_as_float(w.w << 16) * s, __uint_as_float(w.w & 0xFFFF0000u) * s);
            *reinterpret_cast<uint4*>(sm.q[wg] + (x >> 3) * Smem::kHalf + rl * 128 + (((x & 7) ^ (rl & 7)) * 16)) = h;
          }
          fence_proxy_async();
          mbar_arrive(&sm.q_full[wg]);
          ++items;
        }
        for (int u = u0; u < u1; ++u, ++kt) {
          if (!active) continue;
          const int tok = (it.tile0 + u) * kPrKeys;
          if (!wait(&sm.v_full[kt & 1], kt >> 1)) return;
          if (!wait(&sm.s_full[wg], mine_t)) return;
          tmem_fence_after();
          const PrInfo& info = sm.info[kt & 3];
          const bool any_nan = (info.any_nan[0] | info.any_nan[1] | info.any_nan[2] | info.any_nan[3]) != 0;
          const bool edge = tok + kPrKeys - 1 > first_pos || (a.window > 0 && tok <= last_pos - a.window) || any_nan ||
                            (info.valid[0] & info.valid[1] & info.valid[2] & info.valid[3]) != 0xFFFFFFFFu;
          // bit y: this row sees token y of the x-th 32
          auto seen = [&](int x) {
            const int base = tok + x * 32;
            uint32_t m = info.valid[x] & low_bits(pos - base + 1);
            if (a.window > 0) m &= ~low_bits(pos - a.window + 1 - base);
            return m;
          };
          // The scores are read twice, 32 at a time, for the largest one and for
          // the weights: 128 of them in registers would not leave room for the rest.
          uint32_t s[2][32];
          float top = kNoMax;
          tmem_ld32(s[0], t_s);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t(&v)[32] = s[x & 1];
            tmem_wait_ld(v);
            tmem_ld32(s[(x + 1) & 1], t_s + ((x + 1) & 3) * 32);    // the last one is the second pass's first
            if (edge) {
              const uint32_t m = seen(x);
#pragma unroll
              for (int y = 0; y < 32; ++y) v[y] = (m >> y) & 1 ? v[y] : 0xFF800000u;
              if (info.any_nan[x])
                for (int y = 0; y < NB; ++y) nan_blocks |= (info.vnan[x][y] & m) ? 1u << y : 0u;
            }
            float t0 = __uint_as_float(v[0]), t1 = __uint_as_float(v[1]);
#pragma unroll
            for (int y = 2; y < 30; y += 4) {
              t0 = max3(t0, __uint_as_float(v[y]), __uint_as_float(v[y + 1]));
              t1 = max3(t1, __uint_as_float(v[y + 2]), __uint_as_float(v[y + 3]));
            }
            t0 = max3(t0, __uint_as_float(v[30]), __uint_as_float(v[31]));
            top = fmaxf(top, fmaxf(t0, t1) * (f_row * info.rk[x]) + info.rv[x]);
          }
          if (__any_sync(0xFFFFFFFFu, top > m_ref + kSlack)) {
            const float m2 = fmaxf(m_ref, top), fix = ex2(m_ref - m2);
            m_ref = m2;
            l *= fix;
            if (u > u0) {                              // the sums so far, once the product that made them is done
              if (!wait(&sm.o_full[wg], mine_t - 1)) return;
              tmem_fence_after();
#pragma unroll 1
              for (int x = 0; x < D / 32; ++x) {
                tmem_wait_ld(s[0]);                    // the first scores stay as they are
                uint32_t o[32];
                tmem_ld32(o, t_o + x * 32);
                tmem_wait_ld(o);
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * fix);
                tmem_st32(t_o + x * 32, o);
              }
            }
          }
          uint32_t p[32];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t(&v)[32] = s[x & 1];
            tmem_wait_ld(v);
            if (x < 3) tmem_ld32(s[(x + 1) & 1], t_s + (x + 1) * 32);
            if (edge) {
              const uint32_t m = seen(x);
#pragma unroll
              for (int y = 0; y < 32; ++y) v[y] = (m >> y) & 1 ? v[y] : 0xFF800000u;
            }
            const float rv = info.rv[x], f = f_row * info.rk[x], c = rv - m_ref;
            const uint64_t f2 = pack2(f, f), c2 = pack2(c, c);
            uint64_t sum = 0;
#pragma unroll
            for (int y = 0; y < 32; y += 2) {
              float e0, e1;
              unpack2(fma2(pack2(__uint_as_float(v[y]), __uint_as_float(v[y + 1])), f2, c2), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum = add2(sum, pack2(e0, e1));
              p[(x & 1) * 16 + y / 2] = cvt_f16x2(e0, e1);
            }
            float a0, a1;
            unpack2(sum, a0, a1);
            l += (a0 + a1) * pow2f(-(int)rv);
            // the weights of 64 tokens go over scores that both passes are done with
            if (x == 1) tmem_st32(t_s, p);
            if (x == 3) tmem_st32(t_s + 32, p);
          }
          tmem_wait_st();
          tmem_fence_before();
          mbar_arrive(&sm.p_full[wg]);
          ++mine_t;
        }

        // ---- the item's end: output, or a part to be joined
        const bool whole = u0 == 0 && u1 == it.n;
        constexpr int PART = kPrRows * (D + 2);
        float* part = plan.part + (2 * (long long)blockIdx.x + (seg0 <= begin ? 0 : 1)) * PART;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t out_row = it.sq.q0 + qi;
        const int out_head = it.head * a.group + g;
        if (active) {
          if (!wait(&sm.o_full[wg], mine_t - 1)) return;
          tmem_fence_after();
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            uint32_t o[32];
            tmem_ld32(o, t_o + x * 32);
            tmem_wait_ld(o);
            if ((nan_blocks >> x) & 1)
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = 0x7FFFFFFFu;
            if (!on) continue;
            if (whole) {
              uint4* out = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + out_row * a.out_tok +
                                                    (int64_t)out_head * a.out_head + x * 32);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                uint32_t w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  w[z] = l == 0.0f ? 0u : cvt_bf16x2(__uint_as_float(o[y * 8 + z * 2]) * inv,
                                                     __uint_as_float(o[y * 8 + z * 2 + 1]) * inv);
                out[y] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
              uint4* d = reinterpret_cast<uint4*>(part + (wg * 128 + rl) * D + x * 32);
#pragma unroll
              for (int y = 0; y < 8; ++y) d[y] = make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
            }
          }
          if (on && whole && a.lse)
            a.lse[out_row * a.q_heads + out_head] = l == 0.0f ? -INFINITY : (m_ref + log2f(l)) * 0.6931471805599453f;
          if (on && !whole) {
            part[kPrRows * D + wg * 128 + rl] = m_ref;
            part[kPrRows * D + kPrRows + wg * 128 + rl] = l;
          }
          tmem_fence_before();
        }
        if (!whole) {
          const long long first = seg0 / per, last = (seg0 + it.n - 1) / per;
          __threadfence();
          mbar_arrive(&sm.join_all);
          if (warp == 0 && !wait(&sm.join_all, joins)) return;
          if (threadIdx.x == 0) {
            uint32_t* t = plan.ticket + first;       // a CTA starts at most one that others go on with
            const uint32_t got = atomicAdd(t, 1u);
            sm.last = got == (uint32_t)(last - first);
            if (sm.last) *t = 0;
            __threadfence();
            mbar_arrive(&sm.join_last);
          }
          __syncwarp();
          if (!wait(&sm.join_last, joins)) return;
          ++joins;
          if (*reinterpret_cast<volatile uint32_t*>(&sm.last)) {
            __threadfence();
            const int n = (int)(last - first) + 1;
            const int here = min(kPrRows, it.rows - it.rt * kPrRows);
            auto part_at = [&](int i) {
              const long long c = first + i;
              return static_cast<const float*>(plan.part) + (2 * c + (seg0 <= c * per ? 0 : 1)) * PART;
            };
            for (int w = threadIdx.x; w < here * (D / 4); w += 256) {
              const int rr = w / (D / 4), c = w % (D / 4);
              float m = kNoMax;
              for (int i = 0; i < n; ++i) m = fmaxf(m, part_at(i)[kPrRows * D + rr]);
              float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              float sum = 0.0f;
              for (int i = 0; i < n; ++i) {
                const float* q = part_at(i);
                const float f = ex2(q[kPrRows * D + rr] - m);
                const float4 v = *reinterpret_cast<const float4*>(q + rr * D + c * 4);
                o.x += v.x * f;
                o.y += v.y * f;
                o.z += v.z * f;
                o.w += v.w * f;
                sum += q[kPrRows * D + kPrRows + rr] * f;
              }
              const int row = it.rt * kPrRows + rr, i = row / a.group, h = it.head * a.group + row - i * a.group;
              const float k = sum == 0.0f ? 0.0f : 1.0f / sum;
              uint2 v;
              v.x = sum == 0.0f ? 0u : cvt_bf16x2(o.x * k, o.y * k);
              v.y = sum == 0.0f ? 0u : cvt_bf16x2(o.z * k, o.w * k);
              *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t)(it.sq.q0 + i) * a.out_tok +
                                        (int64_t)h * a.out_head + c * 4) = v;
              if (a.lse && c == 0)
                a.lse[(int64_t)(it.sq.q0 + i) * a.q_heads + h] =
                    sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
            }
          }
        }
        at = seg0 + u1;
        seg0 += it.n;
        if (at < end) pr_next(a, it);
      }
    }();
  } else if (wg == 2) {
    // ================= unpacking keys and values =================
    regs_inc<152>();
    [&]() {
      const int grp = warp & 3;                      // tokens 32 grp .. + 31 of a tile
      const int sub = lane & 7;                      // token of 8 within a step
      // a lane's units are the 16-byte blocks blk of U tokens: eight lanes write
      // the same chunk of eight rows, which the swizzle spreads over all banks
      constexpr int U = D == 128 ? 4 : 2;
      const int blk = D == 128 ? lane >> 3 : (lane >> 3) & 1;
      auto token_of = [&](int j) { return D == 128 ? j * 8 + sub : j * 16 + (lane >> 4) * 8 + sub; };
      const int page_mask = (1 << a.shape.page_shift) - 1;
      uint4 kc[U], vc[U];
      uint32_t kw = 0, vw = 0, valid = 0;            // scales of this lane's token; tokens that exist
      int64_t row = 0;                               // this lane's token in the cache
      auto page_of = [&](const PrItem& x, int u) {
        const int tok = (x.tile0 + u) * kPrKeys + grp * 32 + lane;
        return tok < x.sq.len ? a.table[x.b * a.table_stride + (tok >> a.shape.page_shift)] : -1;
      };
      // the unit's rows (row, the mask) and one kind of their codes and scales
      auto locate = [&](const PrItem& x, int u, int page) {
        const int tok = (x.tile0 + u) * kPrKeys + grp * 32 + lane;
        const int64_t slot = ((int64_t)page << a.shape.page_shift) + (tok & page_mask);
        const bool ok = page >= 0 && slot < a.shape.slots;
        row = ok ? kv_row(a.shape, slot, x.head) : 0;
        return __ballot_sync(0xFFFFFFFFu, ok);
      };
      auto load = [&](const KvPool& pool, uint32_t there, uint4 (&codes)[U], uint32_t& w) {
        if (D == 128) w = (there >> lane) & 1 ? reinterpret_cast<const uint32_t*>(pool.e8m0)[row] : 0;
        else w = (there >> lane) & 1 ? reinterpret_cast<const uint16_t*>(pool.e8m0)[row] : 0;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int t = token_of(j);
          const int64_t rr = __shfl_sync(0xFFFFFFFFu, row, t);
          codes[j] = (there >> t) & 1 ? *reinterpret_cast<const uint4*>(pool.q + rr * (D / 2) + blk * 16)
                                      : make_uint4(0, 0, 0, 0);
        }
      };
      // codes * 2^(E - R) of this warp's 32 tokens into a swizzled tile; gives R
      auto unpack = [&](uint8_t* tile, const uint4 (&codes)[U], uint32_t w, bool values, PrInfo& info) {
        uint32_t top = 0;
        bool bad = false;
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          const uint32_t e = (w >> (8 * x)) & 0xFFu;
          bad |= e == 255u;
          top = max(top, e == 255u ? 0u : e);
        }
        const bool there = (valid >> lane) & 1;
        top = __reduce_max_sync(0xFFFFFFFFu, there ? top : 0u);
        top = min(max(top, (uint32_t)kMinScale), (uint32_t)kMaxScale);
        if (values) {
          const uint32_t any = __ballot_sync(0xFFFFFFFFu, there && bad);
          if (any) {
#pragma unroll
            for (int x = 0; x < NB; ++x) {
              const uint32_t m = __ballot_sync(0xFFFFFFFFu, there && ((w >> (8 * x)) & 0xFFu) == 255u);
              if (lane == 0) info.vnan[grp][x] = m;
            }
          }
          if (lane == 0) info.any_nan[grp] = any;
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int t = token_of(j);
          const uint32_t e = (__shfl_sync(0xFFFFFFFFu, w, t) >> (8 * blk)) & 0xFFu;
          const int d = min(126, (int)(top - e));
          float f = __uint_as_float((uint32_t)(127 - d) << 23);
          // a NaN block of keys is NaN to every row that sees the token; one of
          // values would reach rows that do not, so it goes by the flags
          if (e == 255u) f = values ? 0.0f : __uint_as_float(0x7FFFFFFFu);
          const uint32_t f2 = cvt_f16x2(f, f);
          const uint32_t ws[4] = {codes[j].x, codes[j].y, codes[j].z, codes[j].w};
          const int row = grp * 32 + t;
          uint8_t* dst = tile + (blk >> 1) * Smem::kHalf + row * 128;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t h[4];
            e2m1x8_f16(ws[x], h);
            *reinterpret_cast<uint4*>(dst + ((((blk & 1) * 4 + x) ^ (row & 7)) * 16)) =
                make_uint4(mul_f16x2(h[0], f2), mul_f16x2(h[1], f2), mul_f16x2(h[2], f2), mul_f16x2(h[3], f2));
          }
        }
        return top;
      };

      // The items' units in turn.  While one kind of a unit is unpacked, the
      // other kind's codes are in flight, and the page of the unit after.
      PrItem nx = it;
      long long nseg = seg0, at = begin;
      auto step = [&]() {                            // nx, nseg, at: one unit on; false at the end
        ++at;
        if (at >= end) return false;
        if (at == nseg + nx.n) {
          nseg += nx.n;
          pr_next(a, nx);
        }
        return true;
      };
      int page = page_of(nx, (int)(at - nseg));
      valid = locate(nx, (int)(at - nseg), page);
      load(a.k, valid, kc, kw);
      load(a.v, valid, vc, vw);
      bool more = step();
      if (more) page = page_of(nx, (int)(at - nseg));
      const uint32_t units = (uint32_t)(end - begin);
      for (uint32_t kt = 0; kt < units; ++kt) {
        PrInfo& info = sm.info[kt & 3];
        const int stg = kt & 1;
        if (kt >= 2 && !wait(&sm.k_empty[stg], (kt >> 1) - 1)) return;
        const uint32_t rk = unpack(sm.k[stg], kc, kw, false, info);
        if (lane == 0) {
          info.rk[grp] = pow2f((int)rk - 127);
          info.valid[grp] = valid;
        }
        fence_proxy_async();
        mbar_arrive(&sm.k_full[stg]);
        uint32_t next = 0;
        if (more) {
          next = locate(nx, (int)(at - nseg), page);
          load(a.k, next, kc, kw);
        }
        if (kt >= 2 && !wait(&sm.v_empty[stg], (kt >> 1) - 1)) return;
        const uint32_t rv = unpack(sm.v[stg], vc, vw, true, info);
        if (lane == 0) info.rv[grp] = (float)((int)rv - 127);
        fence_proxy_async();
        mbar_arrive(&sm.v_full[stg]);
        if (more) {
          load(a.v, next, vc, vw);
          more = step();
          if (more) page = page_of(nx, (int)(at - nseg));
        }
        valid = next;
      }
    }();
  } else {
    // ================= one warp issues the products =================
    // The whole warp goes through the loop, so that addresses and descriptors
    // stay in uniform registers; one elected lane issues.
    regs_dec<72>();
    if (warp == 12) {
      [&]() {
        constexpr uint32_t kQK = f16_idesc(128, kPrKeys, false), kPV = f16_idesc(128, D, true);
        constexpr uint32_t kHi = desc_hi(1024);
        const uint32_t qa = desc_lo(smem_addr(sm.q[0]), 16), ka = desc_lo(smem_addr(sm.k[0]), 16);
        const uint32_t va = desc_lo(smem_addr(sm.v[0]), Smem::kHalf);
        const bool lead = elect_one();
        const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
        uint32_t kt = 0, items0 = 0, items1 = 0, done0 = 0, done1 = 0;
        auto scores = [&](int w, int stg) {
          const uint32_t q = qa + w * (Smem::kTileBytes >> 4), k = ka + stg * (Smem::kTileBytes >> 4);
          if (lead) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              const uint32_t off = ((x >> 2) * Smem::kHalf + (x & 3) * 32) >> 4;
              mma_ss(tm + kS + w * 128, q + off, k + off, kHi, kQK, x > 0);
            }
            mma_commit(&sm.s_full[w]);
          }
          __syncwarp();
        };
        auto values = [&](int w, int stg, bool first) {
          const uint32_t v = va + stg * (Smem::kTileBytes >> 4);
          if (lead) {
#pragma unroll
            for (int x = 0; x < kPrKeys / 16; ++x)
              mma_ts(tm + kO + w * 128, tm + kS + w * 128 + x * 8, v + x * (2048 >> 4), kHi, kPV, !first || x > 0);
            mma_commit(&sm.o_full[w]);
          }
          __syncwarp();
        };
        for (long long at = begin; at < end;) {
          const int u0 = (int)(at - seg0), u1 = (int)min((long long)it.n, end - seg0);
          const bool two = it.rt * kPrRows + 128 < it.rows;
          if (!wait(&sm.k_full[kt & 1], kt >> 1)) return;
          if (!wait(&sm.q_full[0], items0++)) return;
          tmem_fence_after();
          scores(0, kt & 1);
          if (two) {
            if (!wait(&sm.q_full[1], items1++)) return;
            tmem_fence_after();
            scores(1, kt & 1);
          }
          if (lead) mma_commit(&sm.k_empty[kt & 1]);
          for (int u = u0; u < u1; ++u, ++kt) {
            const uint32_t nk = kt + 1;
            const bool more = u + 1 < u1;
            if (!wait(&sm.v_full[kt & 1], kt >> 1)) return;
            if (!wait(&sm.p_full[0], done0++)) return;
            tmem_fence_after();
            values(0, kt & 1, u == u0);
            if (more) {
              if (!wait(&sm.k_full[nk & 1], nk >> 1)) return;
              scores(0, nk & 1);
            }
            if (two) {
              if (!wait(&sm.p_full[1], done1++)) return;
              tmem_fence_after();
              values(1, kt & 1, u == u0);
              if (more) scores(1, nk & 1);
            }
            if (lead) {
              mma_commit(&sm.v_empty[kt & 1]);
              if (more) mma_commit(&sm.k_empty[nk & 1]);
            }
            __syncwarp();
          }
          at = seg0 + u1;
          seg0 += it.n;
          if (at < end) pr_next(a, it);
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
  if (warp == 12) {
    tmem_fence_after();
    tmem_free(tmem, 512);
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
  const int64_t all = (by_max < by_total ? by_max : by_total) * s.heads * units;
  const int64_t most = (all + kPrMinUnits - 1) / kPrMinUnits;
  const int64_t n = most < sms ? most : sms;
  return (int)(n < kMaxGrid ? n : kMaxGrid);
}

cudaError_t kv_prompt_workspace(const KvShape& s, int group, int batch, int64_t total_q, int max_q, int table_width,
                                int sms, int64_t* bytes) {
  const int grid = pr_grid(s, group, batch, total_q, max_q, table_width, sms);
  *bytes = grid < 2 ? 0 : kMaxGrid * 4 + (int64_t)grid * 2 * kPrRows * (s.dim + 2) * 4;
  return cudaSuccess;
}

cudaError_t launch_kv_prompt(const KvAttn& a, void* workspace, int sms, cudaStream_t st, int* launches) {
  const int grid = pr_grid(a.shape, a.group, a.batch, a.total_q, a.max_q, a.table_width, sms);
  const void* k = a.shape.dim == 128 ? reinterpret_cast<const void*>(kv_prompt_kernel<128>)
                                     : reinterpret_cast<const void*>(kv_prompt_kernel<64>);
  const int smem = a.shape.dim == 128 ? pr_smem<128>() : pr_smem<64>();
  int occ = 1;
  cudaError_t e = kernel_occupancy(k, kPrThreads, smem, &occ);
  if (e != cudaSuccess) return e;
  PrPlan plan;
  plan.ticket = static_cast<uint32_t*>(workspace);
  plan.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kMaxGrid * 4);
  void* args[2] = {const_cast<KvAttn*>(&a), &plan};
  e = cudaLaunchKernel(k, dim3(grid), dim3(kPrThreads), args, (size_t)smem, st);
  if (e == cudaSuccess) *launches += 1;
  return e;
}

cudaError_t read_kv_wait_timeouts(unsigned int* count) {
  cudaError_t e = cudaMemcpyFromSymbol(count, g_kv_wait_timeouts, sizeof *count);
  const unsigned int zero = 0;
  if (e == cudaSuccess && *count) e = cudaMemcpyToSymbol(g_kv_wait_timeouts, &zero, sizeof zero);
  return e;
}

}  // namespace fp8q
