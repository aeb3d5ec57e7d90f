// prefill_u3.cu -- prefill kernel instances for 3-bit caches.
#include "prefill_instance.cuh"

namespace pkv {
cudaError_t launch_prefill_u3(const PrefillLaunch &a)
{
    return a.p->d.q_is_bf16 ? launch_dim<kBF16, kU3, kFeedCodes, true>(a) : launch_dim<kF16, kU3, kFeedCodes, true>(a);
}
}  // namespace pkv
