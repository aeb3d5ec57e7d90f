// prefill_i8.cu -- prefill kernel instances for i8 caches.
#include "prefill_instance.cuh"

namespace pkv {
cudaError_t launch_prefill_i8(const PrefillLaunch &a) { return launch_q8<kI8>(a); }
}  // namespace pkv
