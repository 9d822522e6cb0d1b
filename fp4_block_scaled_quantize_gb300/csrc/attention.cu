// attention.cu -- attention of one new token per sequence over a paged cache in
// 16 bits without first positions (attention16.cuh), and the choice between that
// and attention_sinks.cu.
#include "attention16.cuh"

namespace fp4 {

int64_t decode_attention_workspace(int64_t seqs, int64_t room, int heads, int kv_heads, int head_dim) {
  const int dp = dp_of(head_dim), nt = nt_of(heads / kv_heads, dp), cols = 8 * nt;
  if (cluster_of(seqs * kv_heads * ceil_div(heads / kv_heads, cols), room, dp, nt)) return 0;
  return (int64_t)sm_count() * kPerSM * 2 * slot_floats(cols, dp) * sizeof(float);
}

fp4_status launch_decode_attention(const fp4_attention_params &p, cudaStream_t s) {
  return p.window && p.sinks ? launch_decode_attention_sinks(p, s) : launch_attention<false>(p, s);
}

}  // namespace fp4
