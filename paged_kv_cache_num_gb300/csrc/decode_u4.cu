// decode_u4.cu -- paged decode over 4-bit caches: the persistent kernel, its
// plan and its launches.  (The merge of sequences split between CTAs is
// merge_kernel of decode_tma_kernel.cuh, which walks the same units.)
//
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(c q . k_t - max),
//   k_t = sk_t (u_t - zk_t), v_t = sv_t (w_t - zv_t), codes u, w in 0 .. 15.
// With that, per query head
//   c q . k_t = c sk_t (q . u_t - zk_t sum q),
//   sum_t p_t v_t = sum_t P_t (w_t - zv_t),  P_t = p_t sv_t,
// so K's zero points cost one operation per score, and V's leave the operand as
// it is made.
//
// Codes as operands.  K: a 4-bit code at bit 4 of an otherwise zero 16-bit half
// is the f16 subnormal u 2^-20, exact; an AND makes a pair, 7 operations for 8
// codes.  The tensor core aligns products by their exponents as stored, 2^-14 for
// a subnormal, so up to 2^-16 of |q|'s largest element times sk is cut off in a
// k-step (codes at bit 0 would make that 2^-12).  V: under 0x6400 a code at bit 0
// is 1024 + w, at bit 4 1024 + 16 w, of which one f16 addition or FMA (in another
// pipe than the ANDs) makes w - zv, exactly.  The sums over the keys then hold what
// they are to hold, without a part that is taken off at the end.  Pairs of V are two
// tokens' codes, brought together by byte permutes of two rows.
//
// Work.  A unit is 32 tokens of a group of nh kv heads (two blocks of 16
// slots, one of 32, or a part of a larger one).  All (head group, sequence,
// unit) lie in one flat index space and CTA i takes [i N / S, (i + 1) N / S):
// equal shares whatever the lengths.  A sequence that lies in one CTA is written
// out, others leave (max, sum, accumulator) for the merge.
//
// A CTA is nh consumer warps, one per kv head, and a producer warp that keeps
// a ring of stages full: K and V tiles [block][nh][slots][row] by tensor copies
// and the rows' scales and zeros by bulk copies.  Rows are 64 bytes (swizzled by
// 64) or 32; the token that is row r of a 16-token product is chosen (row_token)
// so that the loads of K rows (4 lanes a row) and of V rows (8 lanes a row) meet no
// bank twice.
// Every wait is bounded (about 2 s) and raises PKV_DEVERR_TIMEOUT.
#include "decode_tma_kernel.cuh"

namespace pkv {
namespace {

constexpr int kUnit = 32;                           // tokens of a unit
constexpr int kUnitShift = 5;

// kv heads of a CTA at most, and CTAs that an SM is to hold: see plan_decode_u4
template <int NG> constexpr int kHeadsU4 = 4;
template <int NG> constexpr int kCtasU4 = NG == 1 ? 3 : 2;

// Token (of 8) that is row r of a product's tile.  head_dim 128, rows of 64
// bytes swizzled by 64 (16-byte piece c of row i at piece c ^ (i >> 1 & 3)): lanes
// of K take rows in pairs, which have to differ in parity; lanes of V rows 0 2 4
// 6 or 1 3 5 7, of which those of one parity have to differ in bit 2.  head_dim 64,
// rows of 32 bytes: K takes rows 0 - 3 and 4 - 7, V the even and the odd ones, each
// different modulo 4.
template <int D> __host__ __device__ constexpr int row_token(int r)
{
    return D == 128 ? r ^ ((r >> 1) & 1) : int((0x57463120u >> (4 * r)) & 7u);
}
// its inverse
template <int D> __host__ __device__ constexpr int token_row(int t)
{
    return D == 128 ? t ^ ((t >> 1) & 1) : int((0x64753120u >> (4 * t)) & 7u);
}
constexpr bool rows_match(int (*f)(int), int (*g)(int))
{
    for (int r = 0; r < 8; ++r)
        if (g(f(r)) != r) return false;
    return true;
}
static_assert(rows_match(row_token<128>, token_row<128>) && rows_match(row_token<64>, token_row<64>), "inverse");

constexpr int kConvBytes = kUnit * (16 + 2);        // per consumer warp: see unit()

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
        // the copies of scales and zeros: by array and block, or by array and head where a
        // unit is part of a block and the arrays are head-major
        const bool by_head = f.meta_hmaj && p.block_size > kUnit;
        const int n_meta = 4 * (by_head ? nh : NB);
        bool aborted = false;
        int64_t issued = 0;
        int ps = 0;
        uint32_t pphase = 0;
        for (int64_t base = lo; base < hi && !aborted; base += 32 / NB) {
            // lane -> (unit, block of it)
            const int64_t x = base + lane / NB;
            int pb = -1, hg = 0, slot0 = 0;
            if (x < hi) {
                hg = int(x / NU);
                const int r = int(x - int64_t(hg) * NU);
                const int b = find_seq(prefix, B, r);
                const int j = r - prefix[b];
                int64_t lb;                                     // logical block
                if constexpr (NB == 2) {
                    lb = 2 * int64_t(j) + lane % NB;
                } else {
                    lb = j >> sub;
                    slot0 = (j & ((1 << sub) - 1)) << kUnitShift;
                }
                if ((lb << p.block_shift) < ctxs[b]) {          // entries behind the context are not read
                    pb = p.block_tables[b * p.bt_b + lb * p.bt_j];
                    if (pb < 0 || pb >= p.num_blocks) {
                        raise_err(p.err_flag, PKV_DEVERR_BLOCK_RANGE);
                        pb = -1;
                    }
                }
            }
            const int n = int(hi - base < 32 / NB ? hi - base : 32 / NB);
            for (int k = 0; k < n; ++k) {
                const int hgk = __shfl_sync(0xffffffffu, hg, k * NB);
                const int s0k = __shfl_sync(0xffffffffu, slot0, k * NB);
                int pbk[NB];
                uint32_t there = 0;
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    pbk[i] = __shfl_sync(0xffffffffu, pb, k * NB + i);
                    there |= (pbk[i] >= 0 ? 1u : 0u) << i;
                }
                const int s = ps;
                const uint32_t fb = bar_full + 8 * s;
                if (lane == 0) {
                    if (issued >= stages && !ptx::mbar_wait_bounded(bar_empty + 8 * s, pphase ^ 1u, kTimeoutNs)) {
                        raise_err(p.err_flag, PKV_DEVERR_TIMEOUT);
                        aborted = true;
                    } else {
                        stage_mask[s] = there;
                        ptx::mbar_arrive_expect_tx(fb, uint32_t(__popc(there)) * block_tx);
                    }
                }
                aborted = __shfl_sync(0xffffffffu, aborted, 0);
                if (aborted) break;
                if (++ps == stages) {
                    ps = 0;
                    pphase ^= 1u;
                }
                ++issued;
                const uint32_t kdst = sbase + s * L.stage, md = kdst + 2 * L.tile;
                if (lane < NB) {
                    const int blk = NB == 2 && lane == 1 ? pbk[NB - 1] : pbk[0];
                    if (blk >= 0) {
                        ptx::tma_load_4d_hint(kdst + lane * part, &tmk, fb, 0, s0k, hgk * nh, blk, once);
                        ptx::tma_load_4d_hint(kdst + L.tile + lane * part, &tmv, fb, 0, s0k, hgk * nh, blk, once);
                    }
                }
                if (lane < n_meta) {
                    const int a = lane & 3, i = lane >> 2;      // array; block or head
                    const int blk = NB == 2 && i == 1 ? pbk[NB - 1] : pbk[0];
                    if (blk >= 0) {
                        const int h0 = f.meta_hmaj ? hgk * nh : 0;
                        const int es = a < 2 ? 2 : 1;
                        // entries of one copy, the first one's place in the block and in the stage
                        const int cnt = by_head ? slots : slots * MH;
                        const int64_t at = f.meta_hmaj ? int64_t(h0 + (by_head ? i : 0)) * p.block_size + s0k : int64_t(s0k) * MH;
                        const char *src = a == 0   ? reinterpret_cast<const char *>(p.k_qs + int64_t(blk) * p.m_blk + at)
                                          : a == 1 ? reinterpret_cast<const char *>(p.v_qs + int64_t(blk) * p.m_blk + at)
                                          : a == 2 ? reinterpret_cast<const char *>(p.k_qz + int64_t(blk) * p.z_blk + at)
                                                   : reinterpret_cast<const char *>(p.v_qz + int64_t(blk) * p.z_blk + at);
                        const uint32_t to = md + (a < 2 ? 2 * a : 2 + a) * kUnit * MH + i * cnt * es;
                        ptx::bulk_load(to, src, uint32_t(cnt * es), fb);
                    }
                }
                __syncwarp();
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
    int64_t x = lo;
    int hg = int(x / NU), b, j;
    {
        const int r = int(x - int64_t(hg) * NU);
        b = find_seq(prefix, B, r);
        j = r - prefix[b];
    }
    int64_t seg_start = lo;
    const int ktok = row_token<D>(gid);             // token of this lane's score rows (and + 8, of each tile)
    const int vtok[2] = {row_token<D>((2 * tig) & 7), row_token<D>((2 * tig + 1) & 7)};
    // byte offsets of this lane's words within a tile's rows
    const uint32_t koff = D == 128 ? ktok * ROW + (((tig ^ (ktok >> 1)) & 3) << 4) : ktok * ROW + 8 * tig;
    uint32_t voff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        voff[i] = D == 128 ? vtok[i] * ROW + ((((gid >> 1) ^ (vtok[i] >> 1)) & 3) << 4) + 8 * (gid & 1) : vtok[i] * ROW + 4 * gid;
    // of the unit's tokens (sk, zk, sv, log2 sv), and zv as f16 by their rows in the products
    float4 *conv = reinterpret_cast<float4 *>(smem + L.conv + warp * kConvBytes);
    __half *conv_z = reinterpret_cast<__half *>(conv + kUnit);

    uint32_t qb[NG][QK][2];                         // q as the B operand
    float o[NG][OT][4];
    float m[NG][2], l[NG][2];                       // maximum and sum of p, of heads 2 tig, 2 tig + 1
    float q1[NG][2], mult[NG][2];                   // sum of q 2^-20 as in qb; what makes q . u log2 units
    int ctx_b = 0;

    auto start_segment = [&]() {
        ctx_b = ctxs[b];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            // column gid: q head 8 g + gid; this lane's elements are those of its words of K:
            // words w of codes d0 + 8 w .. + 7, pairs (n, n + 4)
            const int head = 8 * g + gid;
            const uint16_t *qr = reinterpret_cast<const uint16_t *>(p.q + b * p.q_b + ((hg * nh + kvl) * G + head) * p.q_h) + 8 * WK * tig;
            float v[8 * WK], top = 0.0f;
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
                    v[8 * c + 2 * e] = t.x;
                    v[8 * c + 2 * e + 1] = t.y;
                    top = fmaxf(top, fmaxf(fabsf(t.x), fabsf(t.y)));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // times the power of two that brings the row's largest element to 2^13 .. 2^14: what
            // falls below f16's normal range then is off by at most 2^-38 of the largest
            const int e = min(max(int(__float_as_uint(top) >> 23), 13), 253);
            const float qs = __uint_as_float(uint32_t(267 - e) << 23);         // 2^(140 - e)
            float sum = 0.0f;
#pragma unroll
            for (int k = 0; k < QK; ++k) {
                const int n = 8 * (k >> 1) + 2 * (k & 1);
                float a0, a1, b0, b1;
                qb[g][k][0] = pack_f16(v[n] * qs, v[n + 4] * qs, a0, a1);
                qb[g][k][1] = pack_f16(v[n + 1] * qs, v[n + 5] * qs, b0, b1);
                sum += (a0 + a1) + (b0 + b1);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            // c 2^20 / qs
            const float mu = p.scale_log2 * __uint_as_float(uint32_t(min(max(e - 120 + 127, 1), 254)) << 23);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                q1[g][c] = 0x1p-20f * __shfl_sync(0xffffffffu, sum, 4 * (2 * tig + c));
                mult[g][c] = __shfl_sync(0xffffffffu, mu, 4 * (2 * tig + c));
                m[g][c] = NEG_INF;
                l[g][c] = 0.0f;
            }
#pragma unroll
            for (int t = 0; t < OT; ++t) o[g][t][0] = o[g][t][1] = o[g][t][2] = o[g][t][3] = 0.0f;
        }
    };

    // lane gid holds elements d = (D / 8) gid + 2 t + r of the output (tile t, row half r)
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
                const int head = 8 * g + 2 * tig + c;
                if (head >= GW) continue;
                const int local = kvl * G + head;
                const float inv = whole ? (lt > 0.0f ? 1.0f / lt : 0.0f) : 1.0f;
                float v[D / 8];
#pragma unroll
                for (int t = 0; t < OT; ++t) {
                    v[2 * t] = o[g][t][c] * inv;
                    v[2 * t + 1] = o[g][t][2 + c] * inv;
                }
                if (whole) {
                    uint16_t *to = reinterpret_cast<uint16_t *>(p.out + b * p.o_b + int64_t(hg * nh * G + local) * p.o_h) + D / 8 * gid;
                    uint32_t w[D / 16];
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        float r0, r1;
                        w[i] = p.q_is_bf16 ? pack_bf16(v[2 * i], v[2 * i + 1], r0, r1) : pack_f16(v[2 * i], v[2 * i + 1], r0, r1);
                    }
                    if (p.out_vec_ok) {
#pragma unroll
                        for (int i = 0; i < D / 16; i += 4) *reinterpret_cast<uint4 *>(to + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) to[i] = uint16_t(w[i >> 1] >> (16 * (i & 1)));
                    }
                } else {
                    const int64_t row = key * (int64_t(nh) * G) + local;
                    float *acc = f.part_acc + row * D + D / 8 * gid;
                    if (gid == 0) {
                        f.part_ml[2 * row] = m[g][c];
                        f.part_ml[2 * row + 1] = lt;
                    }
#pragma unroll
                    for (int i = 0; i < D / 8; i += 4) *reinterpret_cast<float4 *>(acc + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
            }
    };

    // one unit in stage s; bit i of `live`: token i counts
    auto unit = [&](int s, uint32_t live) {
        const bool all = live == 0xffffffffu;
        // ---- scales and zeros of a token by its lane, for all lanes
        {
            const unsigned char *raw = smem + (s * L.stage + 2 * L.tile);
            const int i = NB == 2 ? lane >> 4 : 0, slot = NB == 2 ? lane & 15 : lane;
            const int k = i * slots * MH + (f.meta_hmaj ? kvl * slots + slot : slot * MH + hg * nh + kvl);
            const __half *qs = reinterpret_cast<const __half *>(raw);
            const unsigned char *qz = raw + 4 * kUnit * MH;
            const float sv = __half2float(qs[kUnit * MH + k]);
            __syncwarp();                           // the unit before is done with the place
            conv[lane] = make_float4(__half2float(qs[k]), float(qz[k]), sv, scale_exp<40>((__float_as_uint(sv) >> 23) & 0xffu));
            conv_z[(lane & 24) | token_row<D>(lane & 7)] = __float2half_rn(float(qz[kUnit * MH + k]));
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
            float odd[NG][4];                       // a second chain
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[g][t][e] = odd[g][e] = 0.0f;
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
                const uint32_t xa = xw[k >> 1], ya = yw[k >> 1];
                constexpr uint32_t kAt4 = 0x00f000f0u;
                const uint32_t a[4] = {(k & 1 ? xa >> 4 : xa << 4) & kAt4, (k & 1 ? ya >> 4 : ya << 4) & kAt4,
                                       (k & 1 ? xa >> 8 : xa) & kAt4, (k & 1 ? ya >> 8 : ya) & kAt4};
#pragma unroll
                for (int g = 0; g < NG; ++g) ptx::mma16816<false>((k & 1) ? odd[g] : sc[g][t], a, qb[g][k][0], qb[g][k][1]);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[g][t][e] += odd[g][e];
        }
        // ---- online softmax per head column, log2 units.  P = p sv is packed to f16,
        // so the maximum is that of score + log2(sv), by sv's exponent: the largest P is
        // about one and keeps its bits, whatever the scales (an fp16 scale's exponent
        // lies within the bounds of scale_exp)
        uint32_t pb[NG][KT][2];
        float4 mt[KT][2];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) mt[t][r] = conv[16 * t + 8 * r + ktok];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            float mx[2] = {NEG_INF, NEG_INF};
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const bool ok = all || ((live >> (16 * t + 8 * r + ktok)) & 1u);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float v = fmaf(-mt[t][r].y, q1[g][c], sc[g][t][2 * r + c]) * (mt[t][r].x * mult[g][c]);
                        if (!ok) v = NEG_INF;
                        sc[g][t][2 * r + c] = v;
                        mx[c] = fmaxf(mx[c], v + mt[t][r].w);
                    }
                }
            // a unit that raises no maximum skips the reductions and the rescale
            float alpha[2] = {1.0f, 1.0f};
            const bool raise = __any_sync(0xffffffffu, mx[0] > m[g][0] || mx[1] > m[g][1]);
            if (raise) {
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
            }
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float p0 = exp2_approx(sc[g][t][2 * r] - m[g][0]), p1 = exp2_approx(sc[g][t][2 * r + 1] - m[g][1]);
                    l[g][0] += p0;
                    l[g][1] += p1;
                    // (a scale behind the context may be anything)
                    const float sv = all || ((live >> (16 * t + 8 * r + ktok)) & 1u) ? mt[t][r].z : 0.0f;
                    float q0, qq;
                    const uint32_t w = pack_f16(p0 * sv, p1 * sv, q0, qq);
                    pb[g][t][r] = ptx::movmatrix_trans(w);
                }
            if (raise && __any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
                for (int t = 0; t < OT; ++t) {
                    o[g][t][0] *= alpha[0];
                    o[g][t][1] *= alpha[1];
                    o[g][t][2] *= alpha[0];
                    o[g][t][3] *= alpha[1];
                }
            }
        }
        // ---- O^T += V^T P^T: a lane takes codes (D / 8) gid .. of four tokens, tile
        // 4 w + i holding codes 8 w + 2 i (row gid, at bit 0) and + 1 (row gid + 8, at bit 4)
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            const uint32_t at = rows_at(t) + L.tile;
            uint32_t v[4][WV];
            // -1024 - zv and -64 - zv of rows 2 tig, 2 tig + 1 and of those + 8
            __half2 nz0[2], nz4[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const __half2 z = *reinterpret_cast<const __half2 *>(conv_z + 16 * t + 8 * i + 2 * tig);
                nz0[i] = __hsub2(__float2half2_rn(-1024.0f), z);
                nz4[i] = __hsub2(__float2half2_rn(-64.0f), z);
            }
            auto at0 = [](uint32_t x, __half2 nz) -> uint32_t {
                const uint32_t u = (x & 0x000f000fu) | 0x64006400u;
                const __half2 y = __hadd2(*reinterpret_cast<const __half2 *>(&u), nz);
                return *reinterpret_cast<const uint32_t *>(&y);
            };
            auto at4 = [](uint32_t x, __half2 nz) -> uint32_t {
                const uint32_t u = (x & 0x00f000f0u) | 0x64006400u;
                const __half2 y = __hfma2(*reinterpret_cast<const __half2 *>(&u), __float2half2_rn(0.0625f), nz);
                return *reinterpret_cast<const uint32_t *>(&y);
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a = at + voff[i & 1] + (i >> 1) * 8 * ROW;
                if constexpr (D == 128) asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[i][0]), "=r"(v[i][1]) : "r"(a));
                else v[i][0] = ld_shared_u32(a);
            }
#pragma unroll
            for (int w = 0; w < WV; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t x01 = ptx::prmt(v[0][w], v[1][w], h ? 0x7632u : 0x5410u);
                    const uint32_t x23 = ptx::prmt(v[2][w], v[3][w], h ? 0x7632u : 0x5410u);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t xa = x01 >> (8 * i), ya = x23 >> (8 * i);
                        const uint32_t a[4] = {at0(xa, nz0[0]), at4(xa, nz4[0]), at0(ya, nz0[1]), at4(ya, nz4[1])};
#pragma unroll
                        for (int g = 0; g < NG; ++g) ptx::mma16816<false>(o[g][4 * w + 2 * h + i], a, pb[g][t][0], pb[g][t][1]);
                    }
                }
        }
    };

    start_segment();
    int cs = 0;
    uint32_t cphase = 0;
    for (; x < hi; ++x) {
        const int s = cs;
        if (!ptx::mbar_wait_bounded(bar_full + 8 * s, cphase, kTimeoutNs)) {
            raise_err(p.err_flag, PKV_DEVERR_TIMEOUT);
            return;
        }
        if (++cs == stages) {
            cs = 0;
            cphase ^= 1u;
        }
        const int valid = ctx_b - j * kUnit;        // at least 1
        uint32_t live = valid >= kUnit ? 0xffffffffu : (1u << valid) - 1u;
        const uint32_t there = stage_mask[s];
        if (NB == 2) live &= ((there & 1u) ? 0xffffu : 0u) | ((there & 2u) ? 0xffff0000u : 0u);
        else if (there == 0) live = 0;
        if (live != 0) unit(s, live);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar_empty + 8 * s);
        if (x + 1 < hi) {
            ++j;
            if (prefix[b] + j == prefix[b + 1]) {   // the sequence's last unit
                finish_segment(x);
                j = 0;
                do {
                    if (++b == B) {
                        b = 0;
                        ++hg;
                    }
                } while (prefix[b] == prefix[b + 1]);
                seg_start = x + 1;
                start_segment();
            }
        } else {
            finish_segment(x);
        }
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
               row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
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
    if (int64_t(p.max_blocks) * p.block_size > (int64_t(1) << 31) - 64) return false;      // token numbers in 32 bits
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
    f.meta_heads = meta_heads;
    f.meta_hmaj = meta_head_major ? 1 : 0;
    f.smem_bytes = L.total;
    const int64_t units = int64_t(f.n_hg) * p.batch * ((int64_t(p.max_blocks) * p.block_size + kUnit - 1) / kUnit);
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
