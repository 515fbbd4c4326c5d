// prefill_block.cu -- instantiates the tcgen05 prefill kernel for 8-bit codes with a scale per
// block of tokens and kv head: read from their 16-bit copy, or converted in the kernel.
#include "launch.h"
#include "prefill_impl.cuh"

namespace pa {

namespace {

template <int KVT, int DQK, int DVO, bool GEN>
cudaError_t run(const PrefillLaunch& L) {
  using C = PrefillCfg<DQK, DVO, KVT, false, true>;
  auto kern = prefill_kernel<KVT, DQK, DVO, false, GEN, true>;
  static std::atomic<uint64_t> smem_set;
  const cudaError_t e = set_smem_limit_once(kern, C::ALLOC, smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(L.grid), dim3(C::THREADS), C::ALLOC, L.stream, 1, L.tq, L.tk, L.tv, L.tsfk, L.tsfv,
                    L.tp, L.p);
}

// the 16-bit copy without a custom mask or padded pages: the instantiation without that code
template <int KVT, int DQK, int DVO>
cudaError_t run_any(const PrefillLaunch& L) {
  if constexpr (KVT == KV_BF16) {
    if (L.p.mask == nullptr && L.p.box_rows == L.p.page_size) return run<KVT, DQK, DVO, false>(L);
  }
  return run<KVT, DQK, DVO, true>(L);
}

template <int KVT>
cudaError_t dispatch(int dqk, int dvo, const PrefillLaunch& L, const char** variant) {
  if (dqk == 512 && dvo == 512) {
    *variant = "prefill_512x512";
    return run_any<KVT, 512, 512>(L);
  }
  if (dqk == 512 && dvo == 256) {
    *variant = "prefill_512x256";
    return run_any<KVT, 512, 256>(L);
  }
  if (dqk == 256 && dvo == 256) {
    *variant = "prefill_256x256";
    return run_any<KVT, 256, 256>(L);
  }
  return cudaErrorInvalidValue;
}

template <int KVT>
int smem_bytes(int dqk, int dvo) {
  if (dqk == 512 && dvo == 512) return PrefillCfg<512, 512, KVT, false, true>::ALLOC;
  if (dqk == 512 && dvo == 256) return PrefillCfg<512, 256, KVT, false, true>::ALLOC;
  return PrefillCfg<256, 256, KVT, false, true>::ALLOC;
}

}  // namespace

cudaError_t launch_prefill_block(int kvt, int dqk, int dvo, const PrefillLaunch& L, const char** variant) {
  if (kvt == KV_BF16) return dispatch<KV_BF16>(dqk, dvo, L, variant);
  if (kvt == KV_INT8B) return dispatch<KV_INT8B>(dqk, dvo, L, variant);
  if (kvt == KV_FP8B) return dispatch<KV_FP8B>(dqk, dvo, L, variant);
  return cudaErrorInvalidValue;
}

int prefill_block_smem_bytes(int kvt, int dqk, int dvo) {
  if (kvt == KV_INT8B) return smem_bytes<KV_INT8B>(dqk, dvo);
  if (kvt == KV_FP8B) return smem_bytes<KV_FP8B>(dqk, dvo);
  return smem_bytes<KV_BF16>(dqk, dvo);
}

}  // namespace pa
