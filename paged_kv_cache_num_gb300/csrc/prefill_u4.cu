// prefill_u4.cu -- prefill kernel instances for 4-bit caches.
#include "prefill_instance.cuh"

namespace pkv {
cudaError_t launch_prefill_u4(const PrefillLaunch &a)
{
    return a.p->d.q_is_bf16 ? launch_dim<kBF16, kU4, kFeedCodes, true>(a) : launch_dim<kF16, kU4, kFeedCodes, true>(a);
}
}  // namespace pkv
