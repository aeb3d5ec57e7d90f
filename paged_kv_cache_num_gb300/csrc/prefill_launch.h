// prefill_launch.h -- what prefill.cu hands to the instances of the kernel.
#pragma once

#include <cuda.h>

#include "pkv_internal.h"

namespace pkv {

// A CTA's share of the work, as find_start finds it.
struct PrefillStart {
    int64_t u0, u1, total;      // this CTA's cost units, all of them
    int ctas;                   // CTAs that have work
    int b, h, tile, at;
};

struct PrefillLaunch {
    const PrefillParams *p;
    int grid;
    bool join;                  // launch the join kernel too
    bool tma;                   // K/V, or their raw codes, by TMA (tmk, tmv)
    int raw_unit;               // else raw codes by copies; 3-bit rows in pieces of 8 bytes, 4 or 1
    int out32;                  // output rows at multiples of 32 bytes
    void *desc, *starts, *redo, *part_ml, *part_acc;
    bool q_tma;                 // Q by TMA (tmq)
    bool flip_q;                // the kernel gives a negative scale's sign to Q where it converts it
    CUtensorMap tmk, tmv, tmq;
    cudaStream_t stream;
};

cudaError_t launch_prefill_16(const PrefillLaunch &a);
cudaError_t launch_prefill_e4m3(const PrefillLaunch &a);
cudaError_t launch_prefill_e5m2(const PrefillLaunch &a);
cudaError_t launch_prefill_i8(const PrefillLaunch &a);
cudaError_t launch_prefill_u3(const PrefillLaunch &a);

}  // namespace pkv
