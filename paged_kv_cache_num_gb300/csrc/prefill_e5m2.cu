// prefill_e5m2.cu -- prefill kernel instances for e5m2 caches.
#include "prefill_instance.cuh"

namespace pkv {
cudaError_t launch_prefill_e5m2(const PrefillLaunch &a) { return launch_q8<kE5M2>(a); }
}  // namespace pkv
