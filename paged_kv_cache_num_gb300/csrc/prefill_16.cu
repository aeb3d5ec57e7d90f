// prefill_16.cu -- prefill kernel instances for 16-bit caches.
#include "prefill_instance.cuh"

namespace pkv {
cudaError_t launch_prefill_16(const PrefillLaunch &a)
{
    if (a.p->d.q_is_bf16)
        return a.tma ? launch_dim<kBF16, kBF16, kFeedTma, false>(a) : launch_dim<kBF16, kBF16, kFeedCopy, false>(a);
    return a.tma ? launch_dim<kF16, kF16, kFeedTma, false>(a) : launch_dim<kF16, kF16, kFeedCopy, false>(a);
}
}  // namespace pkv
