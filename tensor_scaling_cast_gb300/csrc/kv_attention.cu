// Which attention kernel a call takes.
#include "kv_device.cuh"

namespace fp8q {

cudaError_t kv_attention_workspace(const KvShape& s, int q_heads, int batch, int64_t total_q, int max_q,
                                   int table_width, int sms, int64_t* bytes) {
  const int group = q_heads / s.heads;
  if (kv_decode_takes(max_q, group)) return kv_decode_workspace(s, group, batch, max_q, table_width, sms, bytes);
  return kv_prompt_workspace(s, group, batch, total_q, max_q, table_width, sms, bytes);
}

cudaError_t launch_kv_attention(const KvAttn& a, const KvWork& w, int sms, cudaStream_t st, int* status, int* launches) {
  if (kv_decode_takes(a.max_q, a.group)) return launch_kv_decode(a, w, sms, st, status, launches);
  return launch_kv_prompt(a, w, sms, st, status, launches);
}

}  // namespace fp8q
