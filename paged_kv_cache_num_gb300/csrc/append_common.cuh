// append_common.cuh -- what the append kernels share: the slot of a token,
// the walk over work items, the one-byte casts and the quotient of the 3- and
// 4-bit rows.
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

// RN(x / s) for 16-bit float x and fp16 s > 0, through the correctly
// rounded reciprocal rs = RN(1 / s): with y1 = RN(x rs) and the exact
// residual e = x - y1 s (one FMA), RN(y1 + e rs) is within far less than
// half an ulp of x / s (Markstein's refinement), so it equals x / s
// wherever x / s is an fp32 value -- at every half-integer in particular.
// Off the half-integers rint of it is rint(fl(x / s)) in the codes' range:
// x and s have at most 11 significant bits, so an x / s with |x / s| < 2^10
// that is not a half-integer lies at least 2^-13 away from one.
__device__ __forceinline__ float row_quotient(float x, float s, float rs)
{
    const float y1 = __fmul_rn(x, rs);
    return __fmaf_rn(__fmaf_rn(-y1, s, x), rs, y1);
}

// min / max of two pairs of 16-bit floats (non-NaN operand wins, as fminf /
// fmaxf); exact, the values being 16-bit floats
template <int SRC>
__device__ __forceinline__ uint32_t min2_16(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (SRC == kBF16) asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int SRC>
__device__ __forceinline__ uint32_t max2_16(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (SRC == kBF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A 4-bit row by LPR neighbouring lanes, each with 8 W of its elements (e, pairs
// in order): this lane's W words of codes, and the row's scale and zero.  Every
// lane of the warp calls it.
//   lo = min(0, min), hi = max(0, max), s = fp16((hi - lo) / 15), z = clamp(rint(-lo / s), 0, 15),
//   code = clamp(rint(x / s) + z, 0, 15)
// The quotient by 15 is the division's, by Markstein's refinement (row_quotient;
// below 2^-100, where its residual underflows, s is 0 in any case).  A quotient is
// cut to -z .. 15 - z before it is rounded, by adding 1.5 2^23: the sum's bits are a
// constant plus the integer, and a word is the sum of 16^i times them.
template <int W>
struct RowU4 {
    uint32_t codes[W];
    uint16_t scale;
    uint32_t zero;
};
template <int SRC, int LPR, int W>
__device__ __forceinline__ RowU4<W> row_u4(const uint32_t (&e)[4 * W])
{
    uint32_t mn = e[0], mx = e[0];
#pragma unroll
    for (int j = 1; j < 4 * W; ++j) {
        mn = min2_16<SRC>(mn, e[j]);
        mx = max2_16<SRC>(mx, e[j]);
    }
    mn = min2_16<SRC>(mn, __byte_perm(mn, 0u, 0x1032));         // both halves
    mx = max2_16<SRC>(mx, __byte_perm(mx, 0u, 0x1032));
    uint32_t both = min2_16<SRC>(__byte_perm(mn, mx ^ 0x80008000u, 0x5410), 0u);    // (min, -max), zero among them
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) both = min2_16<SRC>(both, __shfl_xor_sync(0xffffffffu, both, o));
    const float lo = h2f<SRC>(uint16_t(both)), hi = -h2f<SRC>(uint16_t(both >> 16));
    const float range = fminf(__fsub_rn(hi, lo), 3.0e38f);      // (bf16 rows may overflow: s is 65504 then)
    uint16_t sbits = __half_as_ushort(__float2half_rn(row_quotient(range, 15.0f, 1.0f / 15.0f)));
    if ((sbits & 0x7fff) == 0x7c00) sbits = 0x7bff;             // the largest finite fp16
    const float s = __half2float(__ushort_as_half(sbits));
    // s = 0: all quotients, z and the codes become 0
    const float rs = s != 0.0f ? __frcp_rn(s) : 0.0f;
    constexpr float kMagic = 12582912.0f;
    const float z = __fsub_rn(__fadd_rn(fminf(fmaxf(row_quotient(-lo, s, rs), 0.0f), 15.0f), kMagic), kMagic);
    const uint32_t zi = uint32_t(z);
    const float least = -z, most = 15.0f - z;
    RowU4<W> r;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        uint32_t sum = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const float2 x = h2f2<SRC>(e[4 * w + i]);
            const float q1 = fminf(fmaxf(row_quotient(x.y, s, rs), least), most);
            const float q0 = fminf(fmaxf(row_quotient(x.x, s, rs), least), most);
            sum = sum * 16u + __float_as_uint(__fadd_rn(q1, kMagic));
            sum = sum * 16u + __float_as_uint(__fadd_rn(q0, kMagic));
        }
        r.codes[w] = sum + (zi - 0x4b400000u) * 0x11111111u;
    }
    r.scale = sbits;
    r.zero = zi;
    return r;
}

inline int grid_for(int64_t work, int threads)
{
    const int64_t blocks = (work + threads - 1) / threads;
    const int64_t cap = int64_t(sm_count_current_device()) * 16;
    return int(blocks < cap ? (blocks > 0 ? blocks : 1) : cap);
}

}  // namespace
}  // namespace pkv
