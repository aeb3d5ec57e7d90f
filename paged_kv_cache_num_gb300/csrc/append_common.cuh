// append_common.cuh -- what the append kernels share: the slot of a token,
// the walk over work items, and the one-byte casts.
#pragma once

#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kAppendThreads = 256;

// slot of token t from its (request, position) through the block table:
// blk = block_tables[req][pos >> log2(BS)], slot = blk * BS + (pos & (BS-1));
// -1 for pos < 0 (padding), and for positions outside the table (raising
// PKV_DEVERR_POS_RANGE)
__device__ __forceinline__ int64_t slot_from_position(const SlotMapParams &p, int64_t t)
{
    const int32_t pos = p.pos[t * p.pos_stride];
    const int32_t req = p.req[t * p.req_stride];
    int64_t slot = -1;
    if (pos >= 0) {
        const int32_t logical = pos >> p.block_shift;
        if (logical >= p.max_blocks || req < 0 || req >= p.batch) {
            raise_err(p.err_flag, PKV_DEVERR_POS_RANGE);
        } else {
            const int64_t blk = p.bt[req * p.bt_b + logical * p.bt_j];
            slot = (blk << p.block_shift) + (pos & ((1 << p.block_shift) - 1));
        }
    }
    return slot;
}

// the slot of token t; `first`: this caller writes a computed slot out
// (from_pos)
__device__ __forceinline__ int64_t fetch_slot(const AppendParams &p, int64_t t, bool first)
{
    if (p.from_pos) {
        const int64_t slot = slot_from_position(p.pos_map, t);
        if (first) p.pos_map.slot_mapping[t] = slot;
        return slot;
    }
    return p.slot_mapping[t * p.slot_stride];
}

// (block, offset) of a slot; false for a padding token (slot < 0) and for a
// slot outside the pool (raising PKV_DEVERR_SLOT_RANGE)
__device__ __forceinline__ bool place_slot(const AppendParams &p, int64_t slot, int64_t &blk, int64_t &off)
{
    if (slot < 0) return false;                 // padding token: nothing to read or write
    if (slot >= p.num_slots) {
        raise_err(p.err_flag, PKV_DEVERR_SLOT_RANGE);
        return false;
    }
    if (p.block_shift >= 0) {
        blk = slot >> p.block_shift;
        off = slot & ((int64_t(1) << p.block_shift) - 1);
    } else {                                    // e.g. one block per request of max_seq_len
        blk = slot / p.block_size;
        off = slot - blk * p.block_size;
    }
    return true;
}

// `first`: this caller writes the token's computed slot out (from_pos)
__device__ __forceinline__ bool resolve_slot(const AppendParams &p, int64_t t, int64_t &blk,
                                             int64_t &off, bool first = false)
{
    return place_slot(p, fetch_slot(p, t, first), blk, off);
}

// A grid-stride walk over items i = major * n + minor (0 <= minor < n)
// that keeps (major, minor) current by additions: two 32-bit divisions per
// warp at the start, none per item (a 64-bit division by a runtime value
// costs about a hundred instructions).  The first item and the stride are
// warp counts of grids capped at a few thousand blocks, far below 2^32.
struct Walk2 {
    int64_t major, step_major;
    int minor, step_minor, n;
    __device__ __forceinline__ Walk2(int64_t first, int64_t step, int n_) : n(n_)
    {
        const uint32_t f = uint32_t(first), s = uint32_t(step), un = uint32_t(n_);
        const uint32_t fq = f / un, sq = s / un;
        major = fq;
        minor = int(f - fq * un);
        step_major = sq;
        step_minor = int(s - sq * un);
    }
    __device__ __forceinline__ void next()
    {
        major += step_major;
        minor += step_minor;
        if (minor >= n) {
            minor -= n;
            ++major;
        }
    }
};

// Two values already divided by the scale -> two one-byte codes (low byte
// first): fp8 satfinite casts, or int8 nearest-even saturated to +-127
// (NaN -> 0).
template <int Q8>
__device__ __forceinline__ uint32_t q8x2_encode(float2 x)
{
    if constexpr (Q8 == kI8) {
        auto one = [](float v) -> uint32_t {
            int c = isnan(v) ? 0 : __float2int_rn(fminf(fmaxf(v, -127.0f), 127.0f));
            return uint32_t(c) & 0xffu;
        };
        return one(x.x) | (one(x.y) << 8);
    } else {
        return __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, Q8 == kE4M3 ? __NV_E4M3 : __NV_E5M2);
    }
}

inline int grid_for(int64_t work, int threads)
{
    const int64_t blocks = (work + threads - 1) / threads;
    const int64_t cap = int64_t(sm_count_current_device()) * 16;
    return int(blocks < cap ? (blocks > 0 ? blocks : 1) : cap);
}

}  // namespace
}  // namespace pkv
