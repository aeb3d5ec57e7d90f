// decode_u4.cu -- paged decode over 4-bit caches: the persistent kernel, its
// plan and its launches.  (The merge of sequences split between CTAs is
// merge_kernel of decode_tma_kernel.cuh, which walks the same units.)
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(c q . k_t - max),
//   k_t = sk_t (u_t - zk_t), v_t = sv_t (w_t - zv_t), codes u, w in 0 .. 15.
// With that, per query head
//   c q . k_t = c sk_t (q . u_t - zk_t sum q),
//   sum_t p_t v_t = sum_t P_t w_t - sum_t P_t zv_t,  P_t = p_t sv_t,
// so both products are of 16-bit numbers and bare codes.  K's zero points cost one
// operation per score, V's one more row of the product, taken off every 256 tokens.
//
// Codes as operands.  A 4-bit code at bit 2 of an otherwise zero 16-bit half is
// the f16 subnormal u 2^-22, at bit 6 u 2^-18, exact: two shifts and four ANDs make
// four pairs of a word's eight codes.  The 2^4 between the two goes into q (times
// 1/16 for the codes at bit 6) and into the output.  The tensor core aligns
// products by their exponents as stored, 2^-14 for a subnormal, and cuts off what is
// 2^23 below: of a score at most 2^-14 of |q|'s largest element times sk per k-step,
// of the sums over the keys 2^-15 of a step of the code per 16 keys whose largest
// weight is one.  (Codes at bits 0 and 4, a shift less: 2^-12 and 2^-13.  Codes made
// normal numbers, (1024 + w) - (1024 + zv): exact, but a third more instructions,
// which bound this kernel.)  Pairs of V are two tokens' codes: a transposed 8 x 8 load
// of 16-bit pieces brings four codes of each.
//
// Work.  A unit is 32 tokens of a group of nh kv heads (two blocks of 16
// slots, one of 32, or a part of a larger one).  All (head group, sequence,
// unit) lie in one flat index space and CTA i takes [i N / S, (i + 1) N / S):
// equal shares whatever the lengths.  A sequence that lies in one CTA is written
// out, others leave (max, sum, accumulator) for the merge.
//
// A CTA is nh consumer warps, one per kv head, and a producer warp that keeps
// a ring of stages full: K and V tiles [block][nh][slots][row] by tensor copies
// and the rows' scales and zeros by bulk copies.  Rows are 64 or 32 bytes, swizzled
// by as much, so that neither the loads of K rows (4 lanes a row) nor the transposed
// ones of V meet a bank twice.
// Every wait is bounded (about 2 s) and raises PKV_DEVERR_TIMEOUT.
//
// What bounds it.  16 sequences of 16K to 32K tokens, 64 q over 8 kv heads of 128
// (421 MB): 81 us for this kernel, 85 us a call (0.73 of the copy bandwidth); the
// copies alone, without any arithmetic, take 68 to 70 us (6.1 TB/s with start and
// end).  32 sequences of 1K to 8K, 32 heads (677 MB): 130 us a call (0.77), copies
// alone 104 to 108.  The rest is the instructions: about 490 a warp for 32 tokens of
// a kv head (QK and softmax 186, PV 148, scales and zeros 54, ring, walk and the zeros'
// sums 100 with the producer's), of which an SM sub-partition issues 0.55 a cycle; the
// logic pipe is 55 % busy, in bursts.  Tried, against a kernel of 81 us: four CTAs an SM
// (96 registers, spills: 98 us), units of 64 tokens (83), eight heads a CTA (88), shifts
// to the right as products' upper halves (no gain), two or three stages (84, 83); scores'
// operations two heads at a time (fma.rn.f32x2: 6 us more).
#include "decode_tma_kernel.cuh"

namespace pkv {
namespace {

constexpr int kUnit = 32;                           // tokens of a unit
constexpr int kUnitShift = 5;

// kv heads of a CTA at most, and CTAs that an SM is to hold.  Three CTAs of five warps
// leave each SM sub-partition at most four warps of 128 registers; with 16 head
// columns (twice the accumulators) it is three of 168, two CTAs (128 q over 8 kv heads
// on the long contexts: 132 us; before that, against 135, four CTAs of two heads 140, three of four heads 207).
template <int NG> constexpr int kHeadsU4 = 4;
template <int NG> constexpr int kCtasU4 = NG == 1 ? 3 : 2;

constexpr uint32_t kAt2 = 0x003c003cu, kAt6 = 0x03c003c0u;       // codes at bits 2 and 6 of both halves
constexpr int kConvBytes = kUnit * (16 + 4 + 2) + 64;        // per consumer warp: see unit(), and a number a head
// The maximum is raised when a score passes it by more than this (log2 units): P
// then is at most 2^6, far within f16's range, and few units rescale.
constexpr float kRaise = 6.0f;

// The zero points' sums are taken off the codes' every so many units.  Both grow with the number
// of keys, and the tensor core cuts off up to 2^-23 of a sum per 16 keys; their difference grows
// with the root of the number where weights are flat.  Taken off at a sequence's end, 32K keys of
// equal weight in one CTA left an error of 1.1 % of the row, 128K 4.7 %; so it is 0.02 %, f16's own
// rounding, at both.  Costs 1 % (every 16 units 0.8 %; the zeros as a second product in each tile
// 6 %).
constexpr int kZeroUnits = 8;

struct U4Smem {
    int tile, meta, stage, conv, bars, mask, prefix, ctx, total;
};
__host__ __device__ inline U4Smem u4_smem(int nh, int meta_heads, int row, int stages, int batch)
{
    U4Smem L;
    L.tile = nh * kUnit * row;                      // of K or V
    L.meta = 6 * kUnit * meta_heads;                // K scales, V scales, K zeros, V zeros
    L.stage = (2 * L.tile + L.meta + 1023) / 1024 * 1024;
    L.conv = stages * L.stage;
    L.bars = L.conv + nh * kConvBytes;
    L.mask = L.bars + 2 * stages * 8;
    L.prefix = L.mask + stages * 4;
    L.ctx = L.prefix + (batch + 1) * 4;
    L.total = L.ctx + batch * 4 + 1024;             // the base is rounded up to 1024
    return L;
}

// D head_dim; NB blocks of a unit (2: 16-slot blocks; 1: larger ones); NG groups of
// 8 head columns (2 for 9 to 16 q heads per kv head)
template <int D, int NB, int NG>
__global__ void __launch_bounds__(32 * (kHeadsU4<NG> + 1), (kCtasU4<NG>))
    decode_u4_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, DecodeParams p, FastParams f)
{
    constexpr int ROW = D / 2;
    constexpr int KT = kUnit / 16;                  // 16-token tiles
    constexpr int QK = D / 16;                      // k-steps of q . u
    constexpr int OT = D / 16;                      // 16-element tiles of the output
    constexpr int WK = D / 32;                      // words of a K row that a lane takes
    constexpr int WV = D / 64;                      // words of a V row that a lane takes
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nh = f.nh, B = p.batch, G = p.group, stages = f.stages, MH = f.meta_heads;
    const U4Smem L = u4_smem(nh, MH, ROW, stages, B);
    const uint32_t sbase = ptx::smem_u32(smem);
    const uint32_t bar_full = sbase + L.bars, bar_empty = bar_full + 8 * stages;
    volatile uint32_t *stage_mask = reinterpret_cast<volatile uint32_t *>(smem + L.mask);     // bit i: block i of the unit is there
    int *prefix = reinterpret_cast<int *>(smem + L.prefix);     // units before each sequence
    int *ctxs = reinterpret_cast<int *>(smem + L.ctx);
    const int slots = NB == 2 ? 16 : kUnit;         // slots of a block's part in a unit
    // the stream's previous kernel is done (with early_inputs: only before the
    // producer's first copy)
    if (!p.early_inputs) griddep_wait();

    const int cap = p.max_blocks << p.block_shift;
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
        int ctx = p.context_lens[b * p.cl_stride];
        if (ctx < 0 || ctx > cap) {
            if (blockIdx.x == 0) raise_err(p.err_flag, PKV_DEVERR_CONTEXT_RANGE);
            ctx = ctx < 0 ? 0 : cap;
        }
        ctxs[b] = ctx;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            ptx::mbar_init(bar_full + 8 * s, 1);
            ptx::mbar_init(bar_empty + 8 * s, nh);
        }
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (warp == 0) {                                // exclusive scan of the units, 32 sequences a step
        int carry = 0;
        for (int b0 = 0; b0 < B; b0 += 32) {
            const int v = b0 + lane < B ? (ctxs[b0 + lane] + kUnit - 1) >> kUnitShift : 0;
            int incl = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += t;
            }
            if (b0 + lane < B) prefix[b0 + lane] = carry + incl - v;
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) prefix[B] = carry;
    }
    __syncthreads();

    griddep_launch_dependents();                    // the merge waits for this grid's end by itself
    const int64_t NU = prefix[B];                   // units per head group
    const int64_t N = NU * f.n_hg;
    const int64_t lo = int64_t(blockIdx.x) * N / gridDim.x;
    const int64_t hi = int64_t(blockIdx.x + 1) * N / gridDim.x;
    if (lo >= hi) return;

    // ======================================================== producer warp
    if (warp == nh) {
        if (lane == 0) {
            ptx::prefetch_tmap(&tmk);
            ptx::prefetch_tmap(&tmv);
        }
        if (p.early_inputs) griddep_wait();
        const uint64_t once = ptx::policy_evict_first();
        const int sub = p.block_shift - kUnitShift;             // units of a block, log2 (NB == 1)
        const uint32_t part = uint32_t(slots) * ROW * nh;       // bytes of a block's part of the K tile
        const uint32_t block_tx = 2 * part + 6u * uint32_t(slots) * MH;
        // the copies of scales and zeros, one by a lane: by array and block, or by array and head
        // where a unit is part of a block and the arrays are head-major
        const bool by_head = f.meta_hmaj && p.block_size > kUnit;
        const int arr = lane & 3, nth = lane >> 2;              // K scales, V scales, K zeros, V zeros; block or head
        const bool copies = nth < (by_head ? nh : NB);
        const int es = arr < 2 ? 2 : 1, my_blk = by_head ? 0 : nth & (NB - 1);
        const uint32_t bytes = uint32_t((by_head ? slots : slots * MH) * es);
        const uint32_t meta_to = 2 * L.tile + (arr < 2 ? 2 * arr : 2 + arr) * kUnit * MH + nth * bytes;
        const char *meta_src = (arr == 0   ? reinterpret_cast<const char *>(p.k_qs)
                                : arr == 1 ? reinterpret_cast<const char *>(p.v_qs)
                                : arr == 2 ? reinterpret_cast<const char *>(p.k_qz)
                                           : reinterpret_cast<const char *>(p.v_qz)) +
                               (by_head ? nth * p.block_size * es : 0);
        const int64_t meta_blk = arr < 2 ? 2 * p.m_blk : p.z_blk;
        const int meta_hg = f.meta_hmaj ? nh * p.block_size * es : 0, meta_slot = (f.meta_hmaj ? 1 : MH) * es;
        int64_t issued = 0;
        int s = 0;
        uint32_t phase = 0;
        bool aborted = false;
        for (int64_t base = lo; base < hi && !aborted; base += 32 / NB) {
            // lane -> (unit, block of it)
            const int64_t x = base + lane / NB;
            int pb = -1, at = 0;                                // block; head group and first slot
            if (x < hi) {
                const int hg = int(x / NU), r = int(x - int64_t(hg) * NU);
                const int b = find_seq(prefix, B, r), j = r - prefix[b];
                int64_t lb;                                     // logical block
                if constexpr (NB == 2) {
                    lb = 2 * int64_t(j) + lane % NB;
                    at = hg;
                } else {
                    lb = j >> sub;
                    at = hg | ((j & ((1 << sub) - 1)) << 16);   // (hg < 2^15, see plan_decode_u4)
                }
                if ((lb << p.block_shift) < ctxs[b]) {          // entries behind the context are not read
                    pb = p.block_tables[b * p.bt_b + lb * p.bt_j];
                    if (pb < 0 || pb >= p.num_blocks) {
                        raise_err(p.err_flag, PKV_DEVERR_BLOCK_RANGE);
                        pb = -1;
                    }
                }
            }
            const uint32_t in = __ballot_sync(0xffffffffu, pb >= 0);
            const int n = int(hi - base < 32 / NB ? hi - base : 32 / NB);
            for (int k = 0; k < n; ++k) {
                const int atk = __shfl_sync(0xffffffffu, at, k * NB);
                const int tile_blk = __shfl_sync(0xffffffffu, pb, k * NB + (lane & (NB - 1)));
                const int meta_b = NB == 1 ? tile_blk : __shfl_sync(0xffffffffu, pb, k * NB + my_blk);
                const int hgk = NB == 2 ? atk : atk & 0xffff, s0k = NB == 2 ? 0 : (atk >> 16) << kUnitShift;
                const uint32_t there = (in >> (k * NB)) & ((1u << NB) - 1);
                const uint32_t fb = bar_full + 8 * s;
                if (lane == 0) {
                    if (issued >= stages && !ptx::mbar_wait_bounded(bar_empty + 8 * s, phase ^ 1u, kTimeoutNs)) {
                        raise_err(p.err_flag, PKV_DEVERR_TIMEOUT);
                        aborted = true;
                    } else {
                        stage_mask[s] = there;
                        ptx::mbar_arrive_expect_tx(fb, uint32_t(__popc(there)) * block_tx);
                    }
                }
                aborted = __any_sync(0xffffffffu, aborted);
                if (aborted) break;
                const uint32_t dst = sbase + s * L.stage;
                if (lane < NB && tile_blk >= 0) {
                    ptx::tma_load_4d_hint(dst + lane * part, &tmk, fb, 0, s0k, hgk * nh, tile_blk, once);
                    ptx::tma_load_4d_hint(dst + L.tile + lane * part, &tmv, fb, 0, s0k, hgk * nh, tile_blk, once);
                }
                if (copies && meta_b >= 0)
                    ptx::bulk_load(dst + meta_to, meta_src + meta_b * meta_blk + (hgk * meta_hg + s0k * meta_slot), bytes, fb);
                __syncwarp();
                ++issued;
                if (++s == stages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
        // the copies in flight land before this warp retires
        if (lane == 0) {
            for (int64_t it = issued > stages ? issued - stages : 0; it < issued; ++it)
                ptx::mbar_wait_bounded(bar_full + 8 * int(it % stages), uint32_t((it / stages) & 1), kTimeoutNs);
        }
        return;
    }

    // ======================================================== consumer warps
    // Tokens on the products' M, this warp's q heads on N:
    //   S^T[tok][head] = K[tok][:] . Q[head][:],  O^T[d][head] += V^T[d][tok] P^T[tok][head].
    // A lane (gid, tig) of the results holds heads 2 tig, 2 tig + 1 of rows gid, gid + 8.
    const int kvl = warp, gid = lane >> 2, tig = lane & 3;
    const int GW = min(8 * NG, G);
    int hg = int(lo / NU), b, j;
    {
        const int r = int(lo - int64_t(hg) * NU);
        b = find_seq(prefix, B, r);
        j = r - prefix[b];
    }
    int64_t seg_start = lo;
    // shifts to the left by 2 are products with a number that the compiler does not know: they go
    // to the multiplier's pipe, the ANDs have the logic one (1 to 2 %)
    const uint32_t four = f.four;
    // byte offsets within a tile's 16 rows: this lane's words of K row gid, and the 16-byte piece
    // of a V row whose address it gives to a transposed load (matrices: tokens 0 - 7 and 8 - 15
    // of one piece, then of the next)
    const int vrow = lane & 15;
    const uint32_t koff = D == 128 ? gid * ROW + (((tig ^ (gid >> 1)) & 3) << 4) : gid * ROW + ((((tig >> 1) ^ (gid >> 2)) & 1) << 4) + 8 * (tig & 1);
    const uint32_t voff = D == 128 ? vrow * ROW + ((((lane >> 4) ^ (vrow >> 1)) & 3) << 4) : vrow * ROW + ((((lane >> 4) ^ (vrow >> 2)) & 1) << 4);
    // what the products take of the unit's tokens: (sk in log2 units, zk, e, sv
    // 2^-e) with e about log2 sv, 2^-e, and zv as f16
    const uint32_t conv = sbase + L.conv + warp * kConvBytes, conv_e = conv + kUnit * 16, conv_z = conv_e + kUnit * 4, conv_up = conv_z + kUnit * 2;
    // places of this lane's token's scales and zeros among the unit's
    const int meta_k = (NB == 2 ? lane >> 4 : 0) * slots * MH +
                       (f.meta_hmaj ? kvl * slots + (lane & (slots - 1)) : (lane & (slots - 1)) * MH + kvl);

    uint32_t qb[NG][QK][2];                         // q as the B operand
    float o[NG][OT][4];
    float m[NG][2], l[NG][2];                       // maximum and sum of p, of heads 2 tig, 2 tig + 1
    float zs[NG][4];                                // sum of P zv, of lanes 0 - 3 (row 0)
    float q1[NG][2];                                // sum of q 2^-22 as in qb, times the head's own factor
    uint32_t keep = 0;                              // all ones: the heads' factors differ (theirs are at
                                                    // conv_up); else all ones less one
    float mult = 0.0f;                              // what makes q . u (times theirs) log2 units
    int ctx_b = 0;

    auto start_segment = [&]() {
        ctx_b = ctxs[b];
        // column gid of group g: q head 8 g + gid; this lane's elements are those of its words
        // of K, 8 w .. 8 w + 7 from d0 on, in pairs (n, n + 4)
        float v[NG][8 * WK], top[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int head = 8 * g + gid;
            top[g] = 0.0f;
            const uint16_t *qr = reinterpret_cast<const uint16_t *>(p.q + b * p.q_b + ((hg * nh + kvl) * G + head) * p.q_h) + 8 * WK * tig;
#pragma unroll
            for (int c = 0; c < WK; ++c) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (head < GW) u = *reinterpret_cast<const uint4 *>(qr + 8 * c);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 t;
                    if (p.q_is_bf16) t = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
                    else t = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                    v[g][8 * c + 2 * e] = t.x;
                    v[g][8 * c + 2 * e + 1] = t.y;
                    top[g] = fmaxf(top[g], fmaxf(fabsf(t.x), fabsf(t.y)));
                }
            }
        }
        // Times the power of two that brings the largest element to 2^13 .. 2^14: that of all heads,
        // which are then off by at most 2^-24 of their own largest; where one is smaller than another
        // by 2^10 or more, each head's own, and a product more per score.  (That product in every
        // unit: 84 -> 86 us on the long contexts.)  What is not finite counts for no factor: it
        // is no matter of the other heads.
        float all = 0.0f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            top[g] = fmaxf(top[g], __shfl_xor_sync(0xffffffffu, top[g], 1));
            top[g] = fmaxf(top[g], __shfl_xor_sync(0xffffffffu, top[g], 2));
            all = fmaxf(all, top[g] <= 3.4e38f ? top[g] : 0.0f);
        }
#pragma unroll
        for (int s = 4; s < 32; s <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, s));
        auto exponent = [](float x) { return min(max(int(__float_as_uint(x) >> 23), 13), 253); };
        bool far = all > 0x1p73f;                   // (up to there mult is finite)
#pragma unroll
        for (int g = 0; g < NG; ++g) far = far || (top[g] > 0.0f && top[g] < all * 0x1p-10f);
        const bool apart = __any_sync(0xffffffffu, far);
        keep = apart ? 0xffffffffu : 0xfffffffeu;
        // c 2^22 / qs is mult times 2^(e - 135), at most 2^118: nothing overflows that is not a score
        // beyond fp32
        const int most = exponent(all);
        mult = p.scale_log2 * 0x1p17f * (apart ? 1.0f : __uint_as_float(uint32_t(most - 8) << 23));
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int e = apart && top[g] > 0.0f && top[g] <= 3.4e38f ? exponent(top[g]) : most;
            const float qs = __uint_as_float(uint32_t(267 - e) << 23);         // 2^(140 - e)
            const float back = apart ? __uint_as_float(uint32_t(e - 8) << 23) : 1.0f;
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < QK; ++k) {
                const int n = 8 * (k >> 1) + 2 * (k & 1);
                float a0, a1, b0, b1;
                qb[g][k][0] = pack_f16(v[g][n] * qs, v[g][n + 4] * qs, a0, a1);
                qb[g][k][1] = pack_f16(v[g][n + 1] * (0.0625f * qs), v[g][n + 5] * (0.0625f * qs), b0, b1);
                sum += (a0 + a1) + 16.0f * (b0 + b1);
            }
            __syncwarp();                           // (the segment before is done with the place)
            if (tig == 0)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(conv_up + 4 * (8 * g + gid)), "f"(back) : "memory");
            __syncwarp();
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                q1[g][c] = __shfl_sync(0xffffffffu, 0x1p-22f * sum * back, 4 * (2 * tig + c));
                m[g][c] = NEG_INF;
                l[g][c] = 0.0f;
            }
#pragma unroll
            for (int t = 0; t < OT; ++t) o[g][t][0] = o[g][t][1] = o[g][t][2] = o[g][t][3] = 0.0f;
            zs[g][0] = zs[g][1] = zs[g][2] = zs[g][3] = 0.0f;
        }
    };

    // what the zero points have summed up to, off the sums of codes (kZeroUnits)
    auto take_zeros = [&]() {
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float zt = __shfl_sync(0xffffffffu, zs[g][c], tig);
                zs[g][c] = 0.0f;
#pragma unroll
                for (int t = 0; t < OT; ++t) {
                    o[g][t][c] = fmaf(-0x1p-22f, zt, o[g][t][c]);
                    o[g][t][2 + c] = fmaf(-0x1p-18f, zt, o[g][t][2 + c]);
                }
            }
    };

    // tile 2 i + h, row half r of lane gid: element 32 i + 4 gid + 2 h + r of the output
    auto finish_segment = [&](int64_t seg_end) {
        const int64_t first = int64_t(hg) * NU + prefix[b];
        const bool whole = seg_start == first && seg_end == int64_t(hg) * NU + prefix[b + 1] - 1;
        const int64_t key = int64_t(blockIdx.x) + int64_t(hg) * B + b;
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float lt = l[g][c];
#pragma unroll
                for (int s = 4; s < 32; s <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, s);
                const float zt = __shfl_sync(0xffffffffu, zs[g][c], tig);
                const int head = 8 * g + 2 * tig + c;
                if (head >= GW) continue;
                const int local = kvl * G + head;
                const float inv = whole ? (lt > 0.0f ? 1.0f / lt : 0.0f) : 1.0f;
                uint16_t *to = reinterpret_cast<uint16_t *>(p.out + b * p.o_b + int64_t(hg * nh * G + local) * p.o_h) + 4 * gid;
                const int64_t row = key * (int64_t(nh) * G) + local;
                if (!whole && gid == 0) {
                    f.part_ml[2 * row] = m[g][c];
                    f.part_ml[2 * row + 1] = lt;
                }
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const float v[4] = {(o[g][2 * i][c] * 0x1p22f - zt) * inv, (o[g][2 * i][2 + c] * 0x1p18f - zt) * inv,
                                        (o[g][2 * i + 1][c] * 0x1p22f - zt) * inv, (o[g][2 * i + 1][2 + c] * 0x1p18f - zt) * inv};
                    if (!whole) {
                        *reinterpret_cast<float4 *>(f.part_acc + row * D + 32 * i + 4 * gid) = make_float4(v[0], v[1], v[2], v[3]);
                        continue;
                    }
                    float r0, r1;
                    const uint32_t w0 = p.q_is_bf16 ? pack_bf16(v[0], v[1], r0, r1) : pack_f16(v[0], v[1], r0, r1);
                    const uint32_t w1 = p.q_is_bf16 ? pack_bf16(v[2], v[3], r0, r1) : pack_f16(v[2], v[3], r0, r1);
                    if (p.out_vec_ok) {
                        *reinterpret_cast<uint2 *>(to + 32 * i) = make_uint2(w0, w1);
                    } else {
                        to[32 * i] = uint16_t(w0);
                        to[32 * i + 1] = uint16_t(w0 >> 16);
                        to[32 * i + 2] = uint16_t(w1);
                        to[32 * i + 3] = uint16_t(w1 >> 16);
                    }
                }
            }
    };

    // one unit in stage s; bit i of `live`: token i counts (all of them do where ALL, and the heads
    // have one factor)
    auto unit = [&](auto all_c, int s, uint32_t live) {
        constexpr bool ALL = decltype(all_c)::value;
        // ---- scales and zeros of a token by its lane, for all lanes
        {
            const uint32_t raw = sbase + s * L.stage + 2 * L.tile + meta_k + (f.meta_hmaj ? 0 : hg * nh), sc = raw + meta_k + (f.meta_hmaj ? 0 : hg * nh);
            uint32_t ks, vs, kz, vz;
            asm volatile("ld.shared.u16 %0, [%1];" : "=r"(ks) : "r"(sc));
            asm volatile("ld.shared.u16 %0, [%1];" : "=r"(vs) : "r"(sc + 2 * kUnit * MH));
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(kz) : "r"(raw + 4 * kUnit * MH));
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(vz) : "r"(raw + 5 * kUnit * MH));
            const float sv = __half2float(__ushort_as_half(uint16_t(vs)));
            // e: the exponent of an fp16 number as fp32, within +-40 (zero: -40)
            const int e = min(max(int((__float_as_uint(sv) >> 23) & 0xffu) - 126, -40), 40);
            const float down = __uint_as_float(uint32_t(127 - e) << 23);
            const bool on = ALL || ((live >> lane) & 1u);       // a scale behind the context may be anything
            __syncwarp();                           // the unit before is done with the place
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(conv + 16 * lane),
                         "f"(mult * __half2float(__ushort_as_half(uint16_t(ks)))), "f"(float(kz)), "f"(float(e)), "f"(on ? sv * down : 0.0f)
                         : "memory");
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(conv_e + 4 * lane), "f"(down) : "memory");
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(conv_z + 2 * lane), "h"(__half_as_ushort(__float2half_rn(float(vz)))) : "memory");
            __syncwarp();
        }
        // first row of tile t's rows 8 r .. 8 r + 7
        auto rows_at = [&](int t) -> uint32_t {
            return sbase + s * L.stage + (NB == 2 ? (t * nh + kvl) * 16 * ROW : (kvl * 32 + 16 * t) * ROW);
        };
        // ---- S^T = K Q^T
        float sc[NG][KT][4];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[g][t][e] = 0.0f;
            const uint32_t at = rows_at(t) + koff;
            uint32_t xw[WK], yw[WK];
            if constexpr (D == 128) {
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(xw[0]), "=r"(xw[1]), "=r"(xw[2]), "=r"(xw[3]) : "r"(at));
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(yw[0]), "=r"(yw[1]), "=r"(yw[2]), "=r"(yw[3]) : "r"(at + 8 * ROW));
            } else {
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(xw[0]), "=r"(xw[1]) : "r"(at));
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(yw[0]), "=r"(yw[1]) : "r"(at + 8 * ROW));
            }
#pragma unroll
            for (int k = 0; k < QK; ++k) {
                const uint32_t xa = k & 1 ? xw[k >> 1] >> 6 : xw[k >> 1] * four, ya = k & 1 ? yw[k >> 1] >> 6 : yw[k >> 1] * four;
                const uint32_t a[4] = {xa & kAt2, ya & kAt2, xa & kAt6, ya & kAt6};
#pragma unroll
                for (int g = 0; g < NG; ++g) ptx::mma16816<false>(sc[g][t], a, qb[g][k][0], qb[g][k][1]);
            }
        }
        if (!ALL && keep == 0xffffffffu) {          // the heads' own factors
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float up[2];
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(up[0]), "=f"(up[1]) : "r"(conv_up + 4 * (8 * g + 2 * tig)));
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[g][t][e] *= up[e & 1];       // (exact)
            }
        }
        // ---- online softmax per head column, log2 units.  P = p sv is packed to f16,
        // so the maximum is that of score + e, e about log2(sv): the largest P is about
        // one and keeps its bits, whatever the scales.  With x = 2^(score + e - max), P = x
        // (sv 2^-e) and p = x 2^-e.
        uint32_t pb[NG][KT][2];
        float4 mt[KT][2];
        float dn[KT][2];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 16 * t + 8 * r + gid;
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(mt[t][r].x), "=f"(mt[t][r].y), "=f"(mt[t][r].z), "=f"(mt[t][r].w) : "r"(conv + 16 * row));
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(dn[t][r]) : "r"(conv_e + 4 * row));
            }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float mx[2] = {NEG_INF, NEG_INF};
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const bool ok = ALL || ((live >> (16 * t + 8 * r + gid)) & 1u);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float v = fmaf(fmaf(-mt[t][r].y, q1[g][c], sc[g][t][2 * r + c]), mt[t][r].x, mt[t][r].z);
                        sc[g][t][2 * r + c] = ok ? v : NEG_INF;
                        mx[c] = fmaxf(mx[c], sc[g][t][2 * r + c]);
                    }
                }
            // a unit that passes no maximum by much skips the reductions and the rescale
            if (__any_sync(0xffffffffu, mx[0] > m[g][0] + kRaise || mx[1] > m[g][1] + kRaise)) {
                float alpha[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 4));
                    mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 8));
                    mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], 16));
                    const float mn = fmaxf(m[g][c], mx[c]);
                    alpha[c] = mn == NEG_INF ? 1.0f : exp2_approx(m[g][c] - mn);
                    m[g][c] = mn;
                    l[g][c] *= alpha[c];
                }
#pragma unroll
                for (int t = 0; t < OT; ++t) {
                    o[g][t][0] *= alpha[0];
                    o[g][t][1] *= alpha[1];
                    o[g][t][2] *= alpha[0];
                    o[g][t][3] *= alpha[1];
                }
                zs[g][0] *= alpha[0];
                zs[g][1] *= alpha[1];
            }
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float x0 = exp2_approx(sc[g][t][2 * r] - m[g][0]), x1 = exp2_approx(sc[g][t][2 * r + 1] - m[g][1]);
                    l[g][0] = fmaf(x0, dn[t][r], l[g][0]);
                    l[g][1] = fmaf(x1, dn[t][r], l[g][1]);
                    float r0, r1;
                    pb[g][t][r] = ptx::movmatrix_trans(pack_f16(x0 * mt[t][r].w, x1 * mt[t][r].w, r0, r1));
                }
        }
        // ---- O^T += V^T P^T: piece i of the rows holds elements 32 i ..; a lane gets those
        // from 32 i + 4 gid on, of tokens 2 tig and 2 tig + 1 (and + 8), tile 2 i + h taking
        // two of the four
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const uint32_t at = rows_at(t) + L.tile + voff;
            {                                       // zv as row 0 of another tile
                uint32_t z[4] = {0, 0, 0, 0};
                if (gid == 0) {
                    z[0] = ld_shared_u32(conv_z + 2 * (16 * t + 2 * tig));
                    z[2] = ld_shared_u32(conv_z + 2 * (16 * t + 8 + 2 * tig));
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) ptx::mma16816<false>(zs[g], z, pb[g][t][0], pb[g][t][1]);
            }
#pragma unroll
            for (int i2 = 0; i2 < D / 64; ++i2) {
                uint32_t v[4];
                ptx::ldmatrix_x4_trans(at ^ (32 * i2), v[0], v[1], v[2], v[3]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t xa = h ? v[2 * i] >> 6 : v[2 * i] * four, ya = h ? v[2 * i + 1] >> 6 : v[2 * i + 1] * four;
                        const uint32_t a[4] = {xa & kAt2, xa & kAt6, ya & kAt2, ya & kAt6};
#pragma unroll
                        for (int g = 0; g < NG; ++g) ptx::mma16816<false>(o[g][4 * i2 + 2 * i + h], a, pb[g][t][0], pb[g][t][1]);
                    }
            }
        }
    };

    start_segment();
    int cs = 0;
    uint32_t cphase = 0;
    int valid = ctx_b - j * kUnit;                  // tokens from this unit on, at least 1
    for (int left = int(hi - lo); left > 0; --left, valid -= kUnit) {
        const int s = cs;
        if (!ptx::mbar_wait_bounded(bar_full + 8 * s, cphase, kTimeoutNs)) {
            raise_err(p.err_flag, PKV_DEVERR_TIMEOUT);
            return;
        }
        if (++cs == stages) {
            cs = 0;
            cphase ^= 1u;
        }
        uint32_t live = valid >= kUnit ? 0xffffffffu : (1u << valid) - 1u;
        const uint32_t there = stage_mask[s];
        if (NB == 2) live &= ((there & 1u) ? 0xffffu : 0u) | ((there & 2u) ? 0xffff0000u : 0u);
        else if (there == 0) live = 0;
        if (live > keep) unit(std::true_type{}, s, live);
        else if (live != 0) unit(std::false_type{}, s, live);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_empty + 8 * s);
        if (valid > kUnit && left > 1) {            // the sequence goes on here
            if ((left & (kZeroUnits - 1)) == 0) take_zeros();
            continue;
        }
        const int64_t x = hi - left;
        finish_segment(x);
        if (left == 1) break;
        do {
            if (++b == B) {
                b = 0;
                ++hg;
            }
        } while (prefix[b] == prefix[b + 1]);
        seg_start = x + 1;
        start_segment();
        valid = ctx_b + kUnit;                      // (less a unit by the loop)
    }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// (byte of a row, slot, kv head, block): a box is a unit's slots of a block and nh heads
bool u4_map(CUtensorMap *m, const char *base, const DecodeParams &p, int nh)
{
    auto enc = encoder();
    if (!enc || p.num_blocks == 0) return false;
    const cuuint32_t row = cuuint32_t(p.head_dim / 2);
    const cuuint64_t dims[4] = {row, cuuint64_t(p.block_size), cuuint64_t(p.num_kv_heads), cuuint64_t(p.num_blocks)};
    const cuuint64_t strides[3] = {cuuint64_t(p.c_slot), cuuint64_t(p.c_head), cuuint64_t(p.c_blk)};
    const cuuint32_t box[4] = {row, cuuint32_t(p.block_size < kUnit ? p.block_size : kUnit), cuuint32_t(nh), 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<char *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t partial_rows(const DecodeParams &p, const FastParams &f)
{
    return (int64_t(f.grid) + int64_t(f.n_hg) * p.batch) * f.nh * p.group;
}

size_t ml_bytes(int64_t rows) { return (size_t(rows) * 2 * 4 + 255) / 256 * 256; }

template <int D, int NB, int NG>
cudaError_t launch_u4(const DecodeParams &p, const FastParams &f, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t s)
{
    auto kern = decode_u4_kernel<D, NB, NG>;
    static std::atomic<int> configured[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (configured[dev].load(std::memory_order_relaxed) < f.smem_bytes) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem_bytes);
        if (e != cudaSuccess) return e;
        configured[dev].store(f.smem_bytes, std::memory_order_relaxed);
    }
    e = launch_pdl(kern, dim3(f.grid), dim3((f.nh + 1) * 32), f.smem_bytes, s, mk, mv, p, f);
    if (e != cudaSuccess) return e;
    const int rows = p.batch * p.num_heads;
    return launch_pdl(merge_kernel<D>, dim3((rows + kMergeWarps - 1) / kMergeWarps), dim3(32 * kMergeWarps), size_t(p.batch + 1) * 4, s, p, f);
}

}  // namespace

// Heads per CTA, CTAs per SM, ring and grid; false where the general kernel is to run.
bool plan_decode_u4(const DecodeParams &p, bool meta_head_major, int sm_count, FastParams &f, size_t &workspace)
{
    if (p.block_size < 16 || p.batch < 1 || p.batch > 4096 || p.group < 1) return false;
    // token numbers, and units of all sequences, in 32 bits
    const int64_t tokens = int64_t(p.max_blocks) * p.block_size;
    if (tokens > (int64_t(1) << 31) - 64 || p.batch * ((tokens + kUnit - 1) / kUnit) >= (int64_t(1) << 31)) return false;
    if (p.num_kv_heads >= 1 << 15) return false;                                            // head groups in 15
    const int row = p.head_dim / 2, ng = p.group > 8 ? 2 : 1;
    const int most = ng == 1 ? kHeadsU4<1> : kHeadsU4<2>, per_sm = ng == 1 ? kCtasU4<1> : kCtasU4<2>;
    int nh = most;
    while (p.num_kv_heads % nh != 0) --nh;
    const int ctas = per_sm * (most + 1) / (nh + 1);            // as many warps as the registers are shared out for
    const int meta_heads = meta_head_major ? nh : p.num_kv_heads;
    const int budget = 228 * 1024 / ctas - 1024;
    int stages = 8;
    while (stages > 2 && u4_smem(nh, meta_heads, row, stages, p.batch).total > budget) --stages;
    const U4Smem L = u4_smem(nh, meta_heads, row, stages, p.batch);
    if (L.total > 227 * 1024) return false;
    CUtensorMap m;
    if (!u4_map(&m, p.k_cache, p, nh) || !u4_map(&m, p.v_cache, p, nh)) return false;
    f.nh = nh;
    f.ng = ng;
    f.hpw = 1;
    f.ncons = nh;
    f.n_hg = p.num_kv_heads / nh;
    f.stages = stages;
    f.unit_shift = kUnitShift;
    f.four = 4;
    f.meta_heads = meta_heads;
    f.meta_hmaj = meta_head_major ? 1 : 0;
    f.smem_bytes = L.total;
    const int64_t units = int64_t(f.n_hg) * p.batch * ((tokens + kUnit - 1) / kUnit);
    const int64_t room = int64_t(sm_count) * ctas;
    f.grid = int(units < room ? (units > 0 ? units : 1) : room);
    const int64_t rows = partial_rows(p, f);
    workspace = ml_bytes(rows) + size_t(rows) * p.head_dim * 4;
    return true;
}

cudaError_t launch_decode_u4(const DecodeParams &p, FastParams f, void *ws, cudaStream_t s)
{
    char *c = static_cast<char *>(ws);
    f.part_ml = reinterpret_cast<float *>(c);
    f.part_acc = reinterpret_cast<float *>(c + ml_bytes(partial_rows(p, f)));
    CUtensorMap mk, mv;
    if (!u4_map(&mk, p.k_cache, p, f.nh) || !u4_map(&mv, p.v_cache, p, f.nh)) return cudaErrorInvalidValue;
    auto go = [&](auto d_c) -> cudaError_t {
        constexpr int D = decltype(d_c)::value;
        if (p.block_size == 16) return f.ng == 2 ? launch_u4<D, 2, 2>(p, f, mk, mv, s) : launch_u4<D, 2, 1>(p, f, mk, mv, s);
        return f.ng == 2 ? launch_u4<D, 1, 2>(p, f, mk, mv, s) : launch_u4<D, 1, 1>(p, f, mk, mv, s);
    };
    return p.head_dim == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
}

}  // namespace pkv
