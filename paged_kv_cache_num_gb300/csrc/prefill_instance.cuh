// prefill_instance.cuh -- launches of one cache kind's kernel instances.
#pragma once

#include "prefill_kernel.cuh"
#include "prefill_launch.h"

namespace pkv {
namespace {

template <int QK, int CK, int D, int FEED, bool GS>
cudaError_t launch_instance(const PrefillLaunch &a)
{
    auto kernel = prefill_kernel<QK, CK, D, FEED, GS>;
    // the attribute is per device and cheap to set
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<CK, D>::alloc);
    if (e != cudaSuccess) return e;
    PrefillFast f{};
    f.desc = static_cast<int4 *>(a.desc);
    f.starts = static_cast<Start *>(a.starts);
    f.redo = static_cast<int *>(a.redo);
    f.later = a.join;
    f.part_ml = static_cast<float *>(a.part_ml);
    f.part_acc = static_cast<float *>(a.part_acc);
    f.out32 = a.out32;
    f.q_tma = a.q_tma;
    f.flip_q = a.flip_q;
    f.raw_tma = a.tma;
    f.raw_unit = a.raw_unit;
    e = launch_pdl(kernel, a.grid, prefill_threads<CK, FEED>(), Smem<CK, D>::alloc, a.stream, *a.p, f, a.tmk, a.tmv, a.tmq);
    if (e != cudaSuccess || !a.join) return e;
    return launch_pdl(prefill_join_kernel<QK, CK, D>, dim3(a.grid, D / 16), kRowTile, 0, a.stream, *a.p, f);
}

template <int QK, int CK, int FEED, bool GS>
cudaError_t launch_dim(const PrefillLaunch &a)
{
    return a.p->d.head_dim == 128 ? launch_instance<QK, CK, 128, FEED, GS>(a) : launch_instance<QK, CK, 64, FEED, GS>(a);
}

// one-byte codes: per-head scales, or scales per row
template <int CK>
cudaError_t launch_q8(const PrefillLaunch &a)
{
    const bool gs = a.p->d.scale_mode != 0;
    if (a.p->d.q_is_bf16) return gs ? launch_dim<kBF16, CK, kFeedCodes, true>(a) : launch_dim<kBF16, CK, kFeedCodes, false>(a);
    return gs ? launch_dim<kF16, CK, kFeedCodes, true>(a) : launch_dim<kF16, CK, kFeedCodes, false>(a);
}

}  // namespace
}  // namespace pkv
