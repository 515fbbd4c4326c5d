// decode_int8b.cu -- decode kernels for int8 codes with a scale per block of tokens and kv head.
#include "decode_inst.cuh"

namespace pa {
cudaError_t launch_decode_int8b(int dqk, int dvo, int hp, const DecodeLaunch& L, const char** variant) {
  return dispatch_decode<KV_INT8B>(dqk, dvo, hp, L, variant);
}
}  // namespace pa
