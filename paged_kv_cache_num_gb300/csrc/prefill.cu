// prefill.cu -- host side of the prefill attention: plan, tensor maps, and
// the choice of the kernel instance (built in prefill_*.cu).
//
// Sequence b owns rows q_starts[b] .. q_starts[b+1]-1 of q, the last n_b of
// its ctx_b cached tokens; row i sees tokens 0 .. ctx_b - n_b + i:
//   out_i = sum_t exp(s_it - m_i) v_t / sum_t exp(s_it - m_i), s_it = sm_scale q_i . k_t,
// with q head h reading kv head h / group.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "prefill_launch.h"

namespace pkv {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// A box is one block's slots (at most 128) of one kv head.  K of 16-bit
// caches: (element, slot, kv head, block), 64 elements (one 128-byte swizzled
// row) wide; V: (element of a chunk of 64, slot, chunk, kv head, block), the
// row's chunks together.  Codes: the whole rows as bytes, (byte, slot,
// kv head, block), or x-vectorised (byte of a piece, slot, piece, kv head,
// block).
bool cache_map(CUtensorMap *m, const char *base, const DecodeParams &d, int kind, bool v)
{
    auto enc = encoder();
    if (!enc || d.num_blocks == 0) return false;
    const bool coded = kind != kF16 && kind != kBF16;
    const int row = kind == kU3 ? 3 * d.head_dim / 8 : d.head_dim;
    const cuuint32_t slots = cuuint32_t(std::min(d.block_size, 128));
    const cuuint64_t n_slots = cuuint64_t(d.block_size), heads = cuuint64_t(d.num_kv_heads), blocks = cuuint64_t(d.num_blocks);
    const cuuint64_t slot = cuuint64_t(d.c_slot), head = cuuint64_t(d.c_head), block = cuuint64_t(d.c_blk);
    const CUtensorMapDataType type = coded ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : kind == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    auto encode = [&](int rank, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
        return enc(m, type, rank, const_cast<char *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   coded ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (coded && d.c_chunk != 16) {
        const cuuint64_t dims[5] = {16, n_slots, cuuint64_t(row / 16), heads, blocks};
        const cuuint64_t strides[4] = {slot, cuuint64_t(d.c_chunk), head, block};
        const cuuint32_t box[5] = {16, slots, cuuint32_t(row / 16), 1, 1};
        return encode(5, dims, strides, box);
    }
    if (!coded && v) {
        const cuuint64_t dims[5] = {64, n_slots, cuuint64_t(row / 64), heads, blocks};
        const cuuint64_t strides[4] = {slot, 128, head, block};
        const cuuint32_t box[5] = {64, slots, cuuint32_t(row / 64), 1, 1};
        return encode(5, dims, strides, box);
    }
    const cuuint64_t dims[4] = {cuuint64_t(row), n_slots, heads, blocks};
    const cuuint64_t strides[3] = {slot, head, block};
    const cuuint32_t box[4] = {cuuint32_t(coded ? row : 64), slots, 1, 1};
    return encode(4, dims, strides, box);
}

// (element, q head, token) of q: boxes of 64 elements, a group's heads, a subtile's tokens
bool q_map(CUtensorMap *m, const PrefillParams &p)
{
    auto enc = encoder();
    const DecodeParams &d = p.d;
    if (!enc || d.group > 128) return false;
    const cuuint64_t dims[3] = {cuuint64_t(d.head_dim), cuuint64_t(d.num_heads), cuuint64_t(p.num_tokens)};
    const cuuint64_t strides[2] = {cuuint64_t(d.q_h), cuuint64_t(d.q_b)};
    const cuuint32_t box[3] = {64, cuuint32_t(d.group), cuuint32_t(p.sub_rows / d.group)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, d.q_is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
               const_cast<char *>(d.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

PrefillPlan plan_prefill(const PrefillParams &p, int sm_count)
{
    PrefillPlan pl{};
    const DecodeParams &d = p.d;
    // an upper bound of the units, from the shapes alone: every sequence's
    // rows end in a row tile of their own, every tile sees the whole table
    const int64_t tiles = int64_t(p.num_tokens) * d.group / (2 * p.sub_rows) + d.batch;
    const int64_t keys = (int64_t(d.max_blocks) * d.block_size + 127) / 128;
    const int64_t units = tiles * d.num_kv_heads * std::max<int64_t>(keys, 1);
    pl.grid = int(std::max<int64_t>(1, std::min<int64_t>(units, sm_count)));
    pl.join = keys > 1 && pl.grid > 1;
    pl.launches = pl.join ? 2 : 1;
    pl.workspace_bytes = round256(size_t(pl.grid) * sizeof(int4));
    if (pl.join)
        pl.workspace_bytes += round256(size_t(pl.grid) * sizeof(PrefillStart)) + round256(size_t(pl.grid) * sizeof(int)) +
                              size_t(pl.grid) * 2 * 256 * (2 + size_t(d.head_dim)) * sizeof(float);
    return pl;
}

cudaError_t launch_prefill(const PrefillParams &p, const PrefillPlan &pl, int cache_kind, void *ws, cudaStream_t s)
{
    PrefillLaunch a{};
    a.p = &p;
    a.grid = pl.grid;
    a.join = pl.join;
    a.stream = s;
    char *w = static_cast<char *>(ws);
    a.desc = w;
    w += round256(size_t(pl.grid) * sizeof(int4));
    a.starts = w;
    w += round256(size_t(pl.grid) * sizeof(PrefillStart));
    a.redo = w;
    w += round256(size_t(pl.grid) * sizeof(int));
    a.part_ml = w;
    a.part_acc = w + size_t(pl.grid) * 2 * 256 * 2 * sizeof(float);
    const DecodeParams &d = p.d;
    a.out32 = (reinterpret_cast<uintptr_t>(d.out) | uintptr_t(d.o_b) | uintptr_t(d.o_h)) % 32 == 0;
    // by TMA where a map of the cache can be made (and, for 16-bit caches, the
    // rows are contiguous: x-vectorised ones take 16-byte copies)
    const bool coded = cache_kind != kF16 && cache_kind != kBF16;
    a.tma = (coded || d.c_chunk == 16) && cache_map(&a.tmk, d.k_cache, d, cache_kind, false) &&
            cache_map(&a.tmv, d.v_cache, d, cache_kind, true);
    // a negative scale's sign goes into Q: where bf16 Q becomes f16 in any case,
    // or by a warp that copies it
    a.flip_q = d.scale_log2 < 0.0f && coded && d.q_is_bf16;
    a.q_tma = (d.scale_log2 >= 0.0f || a.flip_q) && q_map(&a.tmq, p);
    const uintptr_t at = uintptr_t(d.c_slot) | uintptr_t(d.c_head);        // blocks lie on multiples of 16 bytes
    a.raw_unit = at % 8 == 0 ? 8 : at % 4 == 0 ? 4 : 1;
    switch (cache_kind) {
    case kF16:
    case kBF16: return launch_prefill_16(a);
    case kE4M3: return launch_prefill_e4m3(a);
    case kE5M2: return launch_prefill_e5m2(a);
    case kI8: return launch_prefill_i8(a);
    default: return launch_prefill_u3(a);
    }
}

}  // namespace pkv
