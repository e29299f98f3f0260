// The quantised key/value cache: its layout, the 4-bit format and the small
// device helpers that the write, read and attention kernels share.
//
// A cached row (one token of one head, D elements) is D / 32 MX blocks: codes
// in E2M1 (two per byte, the even element in the low half), E4M3 or E5M2, and
// one E8M0 byte (E + 127) per block.  Rows of one head and page are
// consecutive, so a page of a head is one contiguous run of codes and one of
// E8M0 bytes.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "mx_codes.cuh"

namespace fp8q {

// One kind (keys or values) of the cache as the kernels see it.
struct KvPool {
  uint8_t* q;
  uint8_t* e8m0;
};

struct KvShape {
  int64_t slots;        // num_pages * page_size
  int32_t pages;
  uint32_t page_rows;   // rows of a page, all heads: heads * page_size < 2^31
  int32_t page_shift;   // log2(page_size)
  int32_t heads, dim;
};

// Row index of a page's off-th token for a head: the codes of a row start at
// row * row bytes, its E8M0 bytes at row * (dim / 32).
__device__ __forceinline__ int64_t kv_row(const KvShape& s, int page, int off, int head) {
  return (int64_t)((uint64_t)(uint32_t)page * s.page_rows) + (((int64_t)head << s.page_shift) + off);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 16 (4) bytes into shared memory, asynchronously; zeros past the first
// `bytes` of them, which alone are read.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Chunk c (16 bytes) of row r of a code tile: swizzled so that the eight rows
// of an 8 x 8 load fall on different banks.
template <int D>
__device__ __forceinline__ uint32_t code_offset(int r, int c) {
  return D == 128 ? r * 64 + ((c ^ (r >> 1)) & 3) * 16 : r * 32 + ((c ^ (r >> 2)) & 1) * 16;
}

// Low n bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }

// This warp's copy of the codes and scales of 32 cached rows into shared
// memory, asynchronously; zeros are written for tokens that do not exist.  SWAP: token t's codes go to row t with bits 0 and 3
// exchanged (see the decode kernel's values).  One run of rows from `row` on
// (pages of 32 tokens or more: tiles start at multiples of 32), the first n of
// which exist:
template <bool SWAP>
__device__ __forceinline__ int tile_row(int t) {
  return SWAP ? (t & ~9) | ((t >> 3) & 1) | ((t & 1) << 3) : t;
}
template <int D, bool SWAP>
__device__ __forceinline__ void copy_run(uint32_t codes, uint32_t scales, const KvPool& pool, int64_t row, int n) {
  constexpr int RB = D / 2, NB = D / 32, CH = RB / 16;
  const int lane = threadIdx.x & 31;
  const uint8_t* src = pool.q + row * RB + lane * 16;       // chunk `lane` and every 32nd from there
  const uint8_t* es = pool.e8m0 + row * NB + lane * 4;
  if (n == 32) {
#pragma unroll
    for (int x = 0; x < CH; ++x)
      cp_async16(codes + code_offset<D>(tile_row<SWAP>(x * (32 / CH) + lane / CH), lane % CH), src + x * 512, 16);
    if (D == 128 || lane < 16) cp_async4(scales + lane * 4, es, 4);
  } else {
    // rolled up: a branch, and not both sides' instructions under predicates
#pragma unroll 1
    for (int x = 0; x < CH; ++x) {
      const int r = x * (32 / CH) + lane / CH;
      cp_async16(codes + code_offset<D>(tile_row<SWAP>(r), lane % CH), src + x * 512, r < n ? 16 : 0);
    }
    if (D == 128 || lane < 16) cp_async4(scales + lane * 4, es, lane * (D == 128 ? 1 : 2) < n ? 4 : 0);
  }
}
// Or any rows, `row` being that of the lane's token (smaller pages), bit t of
// valid saying whether token t exists.
template <int D, bool SWAP>
__device__ __forceinline__ void copy_rows(uint32_t codes, uint32_t scales, const KvPool& pool, int64_t row,
                                          uint32_t valid, int page_shift) {
  constexpr int RB = D / 2, CH = RB / 16;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 0; x < CH; ++x) {
    const int r = x * (32 / CH) + lane / CH, c = lane % CH;
    const int64_t rr = __shfl_sync(0xFFFFFFFFu, row, r);
    cp_async16(codes + code_offset<D>(tile_row<SWAP>(r), c), pool.q + rr * RB + c * 16, (valid >> r) & 1 ? 16 : 0);
  }
  const bool ok = (valid >> lane) & 1;
  if (D == 128) {
    cp_async4(scales + lane * 4, pool.e8m0 + row * 4, ok ? 4 : 0);
  } else if (page_shift > 0) {           // two tokens' scales are one word, the even one's row even
    if (!(lane & 1)) cp_async4(scales + lane * 2, pool.e8m0 + row * 2, ok ? 4 : 0);
  } else {
    const uint16_t e = ok ? *reinterpret_cast<const uint16_t*>(pool.e8m0 + row * 2) : 0;
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(scales + lane * 2), "h"(e) : "memory");
  }
}

// The online softmax of both attention kernels keeps a reference M per row:
// weights are 2^(x - M), and M moves only when a score passes it by
// 2^kSlack.  Value scales are taken relative to a group's largest R, which
// stays within [-80, 126] (as E8M0 bytes), so that the sum's terms, weights
// times 2^-R, are finite and 2^-R is a normal number.
constexpr float kNoMax = -3.0e38f;        // M before the first score
constexpr float kSlack = 8.0f;
constexpr uint32_t kMinScale = 127 - 80;
constexpr uint32_t kMaxScale = 127 + 126;
// Score factors stay above zero: a hidden key's -inf times one stays -inf.
constexpr float kMinFactor = 1.17549435e-38f;

// A workspace: tickets (zero between calls), then the parts of rows whose
// keys several CTAs share.
constexpr int kMaxGrid = 4096;            // tickets, and CTAs of a call at most
static_assert(kMaxGrid * 4 == MX_KV_WORKSPACE_ZEROED, "the tickets are what a caller zeroes");
struct KvWork {
  void* at;
  int64_t bytes;
  // FP8Q_OK, or why it cannot serve a call that needs `need` bytes
  int check(int64_t need) const {
    if (need > bytes) return FP8Q_ESIZE;
    if (need > 0 && !at) return FP8Q_EINVAL;
    return need > 0 && (reinterpret_cast<uintptr_t>(at) & 15u) ? FP8Q_EALIGN : FP8Q_OK;
  }
  uint32_t* tickets() const { return static_cast<uint32_t*>(at); }
  float* parts() const { return at ? reinterpret_cast<float*>(static_cast<char*>(at) + kMaxGrid * 4) : nullptr; }
};
// A ticket: the CTAs of a row's parts that have arrived, and above them those
// that gave up (one whose wait ran out takes its tickets all the same, so that
// the count is complete and the last one can set it back).
constexpr uint32_t kGaveUp = 1u << 16;
static_assert(kMaxGrid < (int)kGaveUp, "the count's place");
// Called by one thread between two barriers of its CTA, whose part is written
// before the first: true for the last of `others` + 1 CTAs, where no part is
// missing.  The ticket is zero again then.  The fences are this thread's, next
// to the atomic: what the CTA's other threads wrote, the first barrier orders
// before them; what they read, the second after them.
__device__ __forceinline__ bool take_ticket(uint32_t* t, uint32_t others, uint32_t mark) {
  __threadfence();
  const uint32_t got = atomicAdd(t, 1u + mark);
  if ((got & (kGaveUp - 1)) != others) return false;
  __threadfence();
  *t = 0;
  return got + mark < kGaveUp;
}

// ---- launches (kv_cache.cu, kv_attention.cu) --------------------------------
cudaError_t launch_kv_write(const KvShape& s, int format, KvPool k, KvPool v, const void* kx, const void* vx,
                            int dtype, int64_t tokens, const int64_t* strides, const int64_t* slots, int rule,
                            cudaStream_t st, int* launches);
cudaError_t launch_kv_read(const KvShape& s, int format, KvPool k, KvPool v, void* kx, void* vx, int dtype,
                           int64_t tokens, const int64_t* strides, const int64_t* slots, cudaStream_t st,
                           int* launches);

// Arguments of one attention call, checked on the host.
struct KvAttn {
  KvShape shape;
  KvPool k, v;
  const void* q;
  void* out;
  float* lse;
  const int32_t* cu_q;
  const int32_t* kv_lens;
  const int32_t* table;
  int64_t q_tok, q_head, out_tok, out_head;   // strides in elements
  int64_t table_stride;
  int32_t table_width, batch, total_q, max_q, q_heads, group, window;
  FastDiv by_group;                            // division by group
  float scale;
};
// What a call has to do for sequence b.  Query i of the sequence sits at
// position pos0 + i; lengths and offsets that point outside are clamped.
struct KvSeq {
  int q0, nq, len, pos0;      // first query row, queries, keys, position of query 0
};
__device__ __forceinline__ KvSeq kv_seq(const KvAttn& a, int b) {
  KvSeq s;
  s.q0 = a.cu_q ? a.cu_q[b] : b;
  const int n = a.cu_q ? max(0, a.cu_q[b + 1] - s.q0) : 1;
  s.q0 = max(s.q0, 0);
  s.nq = max(0, min(min(n, a.max_q), a.total_q - s.q0));
  const int64_t most = (int64_t)a.table_width << a.shape.page_shift;
  s.len = (int)min((int64_t)max(a.kv_lens[b], 0), most);
  s.pos0 = s.len - n;
  return s;
}

// ---- joining the parts of rows --------------------------------------------------
//
// A part holds, for R rows, the sums o [R][D] under the row's own reference
// m [R] and softmax sum l [R].  Joined: M = max m, o = sum 2^(m - M) o and l
// alike, in the order of the parts.  Two steps, both with several parts'
// loads in flight: row_of_parts finds M and l per row (one thread per row),
// then every four columns of a row are one thread's.

struct Joined {
  float m, l;
};
__device__ __forceinline__ Joined join2(const Joined& a, const Joined& b) {
  const float m = fmaxf(a.m, b.m);
  return {m, a.l * ex2(a.m - m) + b.l * ex2(b.m - m)};
}
// Row r of parts first, first + step, ..
template <int R, int D, class PartAt>
__device__ __forceinline__ Joined row_of_parts(PartAt part_at, int first, int step, int n, int r) {
  Joined j = {kNoMax, 0.0f};
#pragma unroll 4
  for (int i = first; i < n; i += step) {
    const float* q = part_at(i) + R * D + r;
    j = join2(j, {q[0], q[R]});
  }
  return j;
}
// Columns 4 c .. 4 c + 3 of U rows r[] under their joined references m[];
// AHEAD parts at a time.
template <int R, int D, int U, int AHEAD, class PartAt>
__device__ __forceinline__ void columns_of_parts(PartAt part_at, int n, const int (&r)[U], int c, const float (&m)[U],
                                                 float4 (&o)[U]) {
#pragma unroll
  for (int x = 0; x < U; ++x) o[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll AHEAD
  for (int i = 0; i < n; ++i) {
    const float* q = part_at(i);
    float4 v[U];
    float f[U];
#pragma unroll
    for (int x = 0; x < U; ++x) {
      v[x] = *reinterpret_cast<const float4*>(q + r[x] * D + c * 4);
      f[x] = q[R * D + r[x]];
    }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const float k = ex2(f[x] - m[x]);
      o[x].x += v[x].x * k;
      o[x].y += v[x].y * k;
      o[x].z += v[x].z * k;
      o[x].w += v[x].w * k;
    }
  }
}
// Four columns of one row's output, from its sums.
__device__ __forceinline__ void store_columns(const KvAttn& a, int64_t row, int head, int c, const float4& o, float l) {
  const float k = l == 0.0f ? 0.0f : 1.0f / l;       // a row that sees no key gets zeros
  uint2 v;
  v.x = l == 0.0f ? 0u : cvt_bf16x2(o.x * k, o.y * k);
  v.y = l == 0.0f ? 0u : cvt_bf16x2(o.z * k, o.w * k);
  *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.out_tok + head * a.out_head + c * 4) = v;
}
__device__ __forceinline__ void store_lse(const KvAttn& a, int64_t row, int head, float m, float l) {
  if (a.lse) a.lse[row * a.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Few query rows per key/value head (kv_decode.cu).
bool kv_decode_takes(int max_q, int group);
cudaError_t kv_decode_workspace(const KvShape& s, int group, int batch, int max_q, int table_width, int sms,
                                int64_t* bytes);
cudaError_t launch_kv_decode(const KvAttn& a, const KvWork& w, int sms, cudaStream_t st, int* status, int* launches);
// Any number of them (kv_prompt.cu).
cudaError_t kv_prompt_workspace(const KvShape& s, int group, int batch, int64_t total_q, int max_q, int table_width,
                                int sms, int64_t* bytes);
cudaError_t launch_kv_prompt(const KvAttn& a, const KvWork& w, int sms, cudaStream_t st, int* status, int* launches);
cudaError_t read_kv_wait_timeouts(unsigned int* count);   // and reset to 0
// Any call: the kernel that fits it (kv_attention.cu).
cudaError_t kv_attention_workspace(const KvShape& s, int q_heads, int batch, int64_t total_q, int max_q,
                                   int table_width, int sms, int64_t* bytes);
cudaError_t launch_kv_attention(const KvAttn& a, const KvWork& w, int sms, cudaStream_t st, int* status, int* launches);

}  // namespace fp8q
