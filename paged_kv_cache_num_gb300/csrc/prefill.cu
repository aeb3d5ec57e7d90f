// prefill.cu -- causal attention of packed new tokens over the paged cache.
//
// Sequence b owns rows q_starts[b] .. q_starts[b+1]-1 of q, the last n_b of
// its ctx_b cached tokens; row i sees tokens 0 .. ctx_b - n_b + i:
//   out_i = sum_t exp(s_it - m_i) v_t / sum_t exp(s_it - m_i), s_it = sm_scale q_i . k_t,
// with q head h reading kv head h / group.
//
// One warp per (token, q head) row: the plainest form.
#include <type_traits>

#include "prefill_row.cuh"

namespace pkv {
namespace {

template <int QK, int CK, int D>
__global__ void __launch_bounds__(128) prefill_rows_kernel(PrefillParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const DecodeParams &d = p.d;
    const int lane = threadIdx.x & 31;
    const int64_t rows = int64_t(p.num_tokens) * d.num_heads;
    const int64_t step = (int64_t(gridDim.x) * blockDim.x) >> 5;
    for (int b = blockIdx.x * blockDim.x + threadIdx.x; b < d.batch; b += gridDim.x * blockDim.x) {
        const int a = p.q_starts[b * p.qs_stride], e = p.q_starts[(b + 1) * p.qs_stride];
        if (a < 0 || e < a || e > p.num_tokens) raise_err(d.err_flag, PKV_DEVERR_QSTART_RANGE);
    }
    for (int64_t r = (blockIdx.x * int64_t(blockDim.x) + threadIdx.x) >> 5; r < rows; r += step) {
        const int tok = int(r / d.num_heads), head = int(r - int64_t(tok) * d.num_heads);
        int lo = 0, hi = d.batch;                   // the last sequence that starts at or before tok
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.q_starts[mid * p.qs_stride] <= tok) lo = mid; else hi = mid;
        }
        const int s0 = p.q_starts[lo * p.qs_stride], s1 = p.q_starts[(lo + 1) * p.qs_stride];
        if (tok < s0 || tok >= s1) continue;
        if (s0 < 0 || s1 > p.num_tokens) continue;
        int ctx = d.context_lens[lo * d.cl_stride];
        const int cap = d.max_blocks << d.block_shift;
        if (ctx < 0 || ctx > cap) {
            if (lane == 0) raise_err(d.err_flag, PKV_DEVERR_CONTEXT_RANGE);
            ctx = ctx < 0 ? 0 : cap;
        }
        prefill_row<QK, CK, D>(d, d.block_tables + lo * d.bt_b, tok, head, max(0, ctx - (s1 - s0) + (tok - s0) + 1));
    }
}

}  // namespace

PrefillPlan plan_prefill(const PrefillParams &, int, int)
{
    PrefillPlan pl{};
    pl.launches = 1;
    return pl;
}

cudaError_t launch_prefill(const PrefillParams &p, const PrefillPlan &, int cache_kind, void *, cudaStream_t s)
{
    const int64_t rows = int64_t(p.num_tokens) * p.d.num_heads;
    const int g = int(rows / 4 + 1 < 152 * 64 ? rows / 4 + 1 : 152 * 64);
    auto go = [&](auto qk_c, auto ck_c) -> cudaError_t {
        constexpr int QK = decltype(qk_c)::value;
        constexpr int CK = decltype(ck_c)::value;
        return p.d.head_dim == 128 ? launch_pdl(prefill_rows_kernel<QK, CK, 128>, g, 128, 0, s, p)
                                   : launch_pdl(prefill_rows_kernel<QK, CK, 64>, g, 128, 0, s, p);
    };
    auto q8 = [&](auto qk_c) -> cudaError_t {
        if (cache_kind == kE4M3) return go(qk_c, std::integral_constant<int, kE4M3>{});
        if (cache_kind == kE5M2) return go(qk_c, std::integral_constant<int, kE5M2>{});
        if (cache_kind == kI8) return go(qk_c, std::integral_constant<int, kI8>{});
        return go(qk_c, std::integral_constant<int, kU3>{});
    };
    using HF = std::integral_constant<int, kF16>;
    using BF = std::integral_constant<int, kBF16>;
    if (cache_kind == kF16) return go(HF{}, HF{});
    if (cache_kind == kBF16) return go(BF{}, BF{});
    return p.d.q_is_bf16 ? q8(BF{}) : q8(HF{});
}

}  // namespace pkv
