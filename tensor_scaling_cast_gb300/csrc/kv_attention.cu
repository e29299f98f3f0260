// Attention of query tokens over the 4-bit cache of their sequences:
// o = sum_j softmax_j(scale * q . k_j) v_j over the keys j that the causal
// mask and the window leave a query at position kv_len - n_q + i.
#include "kv_device.cuh"

namespace fp8q {

constexpr int kAttnWarps = 4;

// One warp per (query token, query head): scores of 32 keys at a time, one
// key per lane, then the values with each lane holding D / 32 columns.  One
// pass over the keys with a running maximum and sum.
template <int D>
__global__ void __launch_bounds__(32 * kAttnWarps) kv_attention_kernel(const __grid_constant__ KvAttn a) {
  constexpr int C = D / 32;
  __shared__ float sq[kAttnWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, i = blockIdx.y, head = blockIdx.x * kAttnWarps + warp;
  if (head >= a.q_heads) return;
  const int q0 = a.cu_q ? a.cu_q[b] : b, nq = a.cu_q ? a.cu_q[b + 1] - q0 : 1;
  if (i >= nq || q0 < 0 || q0 + i >= a.total_q) return;
  const int64_t row = q0 + i;
  const int kvh = head / a.group;
  const int64_t most = (int64_t)a.table_width << a.shape.page_shift;
  const int len = (int)min((int64_t)max(a.kv_lens[b], 0), most);
  const int pos = len - nq + i;
  const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + row * a.q_tok + head * a.q_head;
  for (int d = lane; d < D; d += 32) sq[warp][d] = __bfloat162float(q[d]) * (a.scale * 1.4426950408889634f);
  __syncwarp();
  float m = -INFINITY, l = 0.0f, o[C] = {};
  for (int j0 = begin; j0 <= pos; j0 += 32) {
    const int j = j0 + lane;
    int64_t r = -1;
    if (j <= pos) {
      const int page = a.table[b * a.table_stride + (j >> a.shape.page_shift)];
      const int64_t slot = ((int64_t)page << a.shape.page_shift) + (j & ((1 << a.shape.page_shift) - 1));
      if (page >= 0 && slot < a.shape.slots) r = kv_row(a.shape, slot, kvh);
    }
    float s = -INFINITY;
    if (r >= 0) {
      s = 0.0f;
      for (int blk = 0; blk < C; ++blk) {
        const uint4 w = *reinterpret_cast<const uint4*>(a.k.q + r * (D / 2) + blk * 16);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
        float t = 0.0f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t h[4];
          e2m1x8_f16(ws[x], h);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float2 f = f16x2_f32(h[y]);
            t += f.x * sq[warp][blk * 32 + x * 8 + 2 * y] + f.y * sq[warp][blk * 32 + x * 8 + 2 * y + 1];
          }
        }
        s += t * e8m0_value(a.k.e8m0[r * C + blk]);
      }
    }
    float top = s;
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    const float m2 = fmaxf(m, top), base = m2 == -INFINITY ? 0.0f : m2;
    const float fix = exp2f(m - base), p = exp2f(s - base);
    m = m2;
    l = l * fix + p;
#pragma unroll
    for (int x = 0; x < C; ++x) o[x] *= fix;
    for (int y = 0; y < 32; ++y) {
      const float py = __shfl_sync(0xFFFFFFFFu, p, y);
      const int64_t ry = __shfl_sync(0xFFFFFFFFu, r, y);
      if (ry < 0) continue;
#pragma unroll
      for (int x = 0; x < C; ++x) {
        const uint32_t byte = a.v.q[ry * (D / 2) + (x * 32 + lane) / 2];
        uint32_t h[4];
        e2m1x8_f16(byte, h);
        const float2 f = f16x2_f32(h[0]);
        o[x] += py * ((lane & 1) ? f.y : f.x) * e8m0_value(a.v.e8m0[ry * C + x]);
      }
    }
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, x);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.out_tok + head * a.out_head;
#pragma unroll
  for (int x = 0; x < C; ++x) out[x * 32 + lane] = __float2bfloat16_rn(l == 0.0f ? 0.0f : o[x] * inv);
  if (a.lse && lane == 0) a.lse[row * a.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

cudaError_t kv_attention_workspace(const KvShape& s, int q_heads, int batch, int max_q, int table_width, int sms,
                                   int64_t* bytes) {
  *bytes = 0;
  if (kv_decode_takes(max_q, q_heads / s.heads))
    return kv_decode_workspace(s, q_heads / s.heads, batch, max_q, table_width, sms, bytes);
  return cudaSuccess;
}

cudaError_t launch_kv_attention(const KvAttn& a, void* workspace, int sms, cudaStream_t st, int* launches) {
  if (kv_decode_takes(a.max_q, a.group)) return launch_kv_decode(a, workspace, sms, st, launches);
  const dim3 grid((a.q_heads + kAttnWarps - 1) / kAttnWarps, a.max_q, a.batch);
  if (a.shape.dim == 64) kv_attention_kernel<64><<<grid, 32 * kAttnWarps, 0, st>>>(a);
  else kv_attention_kernel<128><<<grid, 32 * kAttnWarps, 0, st>>>(a);
  *launches += 1;
  return cudaGetLastError();
}

}  // namespace fp8q
