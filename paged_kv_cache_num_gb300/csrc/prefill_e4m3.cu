// prefill_e4m3.cu -- prefill kernel instances for e4m3 caches.
#include "prefill_instance.cuh"

namespace pkv {
cudaError_t launch_prefill_e4m3(const PrefillLaunch &a) { return launch_q8<kE4M3>(a); }
}  // namespace pkv
