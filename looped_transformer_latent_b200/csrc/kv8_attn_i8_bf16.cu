// Attention over a cache of int8 codes, bfloat16 queries and outputs.
#include "kv8_attn.cuh"

namespace lla {
cudaError_t launch_kv8_attn_i8_bf16(const Kv8AttnArgs& a, cudaStream_t st) { return kv8::launch_d<LLA_KV8_I8, 1>(a, st); }
}  // namespace lla
