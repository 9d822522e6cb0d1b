// attention_sinks.cu -- attention of one new token per sequence over a paged cache
// in 16 bits, windows with first positions that stay visible (attention16.cuh).
#include "attention16.cuh"

namespace fp4 {

fp4_status launch_decode_attention_sinks(const fp4_attention_params &p, cudaStream_t s) {
  return launch_attention<true>(p, s);
}

}  // namespace fp4
