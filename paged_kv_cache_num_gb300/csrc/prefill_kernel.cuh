// prefill_kernel.cuh -- the prefill attention on the tensor cores, and the
// kernel that joins the parts of row tiles that several CTAs worked on.
//
// Mathematics.  One pass over the keys with a running maximum and sum per
// row: for each tile of 128 keys S = Q K^T, m' = max(m, max S),
// P = 2^(c (S - m')), l = l 2^(c (m - m')) + sum P, O = O 2^(c (m - m')) + P V,
// out = O / l, c = |sm_scale| log2(e) (the sign goes into Q).  m is kept as
// a reference that moves only when a row's maximum passes it by more than
// 2^8 in P: until then the old reference stays, P is at most 2^8, and O is
// not touched; the quotient is the same.  P is rounded to the 16-bit operand
// type of the second product (S, m, l and O stay in fp32).
//
// Decomposition.  The rows of one (sequence, kv head) are its tokens times
// the group's q heads, token major: a K/V tile read once serves all heads of
// the group, and the causal border is as sharp as the rows allow.  256 of
// them (two subtiles of 128) make a row tile; a unit of work is one row tile
// times one tile of 128 keys that some of its rows see.  All units lie in one
// flat order (sequence, kv head, row tile, key tile), and CTA i takes
// [i N / S, (i + 1) N / S): equal work for any mix of lengths, decided on the
// device (no host read of lengths; graph safe).  A CTA that has the whole key
// range of a row tile writes its rows; otherwise it writes an fp32 partial
// (m, l, O), and prefill_join_kernel combines them.
//
// CTA.  Two softmax warpgroups (one per subtile, a thread per row), one warp
// that issues the products (tcgen05.mma, accumulators and P in tensor
// memory), two warps that load Q, and the K/V producer: TMA copies of whole
// block pieces for 16-bit caches in the flash layout (one warp), or four
// warps that load, convert and store codes (one-byte and 3-bit caches) or
// copy 16-byte pieces (other layouts).  While one subtile's softmax runs the
// tensor core works on the other's products.
//
// Codes are converted exactly (every code of every kind is a number of both
// 16-bit types); their scales are applied in fp32: per-head scales to c and
// to the result, per-row scales to the columns of S and of P.
#pragma once

#include <type_traits>

#include "prefill_row.cuh"
#include "tc_ptx.cuh"

namespace pkv {

struct PrefillFast {
    int4 *desc;                 // [grid] (sequence, kv head, row tile, last CTA) of the row tile split at a CTA's end
    float *part_ml;             // [2 grid][2][256]
    float *part_acc;            // [2 grid][D / 4][256][4]
    int rows_aligned;           // 3-bit rows at multiples of 4 bytes
};

namespace {

constexpr int kRowTile = 256;
constexpr int kKeyTile = 128;
constexpr int kBins = 1024;
constexpr uint64_t kPrefillTimeoutNs = 4000000000ull;

// One (sequence)'s lengths, cleaned: n = 0 for a sequence that is left out.
struct Seq {
    int s0, n, ctx, rows, nt;
};

__device__ __forceinline__ Seq seq_load(const PrefillParams &p, int b, bool flag)
{
    Seq s;
    const int a = p.q_starts[b * p.qs_stride], e = p.q_starts[(b + 1) * p.qs_stride];
    int ctx = p.d.context_lens[b * p.d.cl_stride];
    const int cap = p.d.max_blocks << p.d.block_shift;
    const bool bad_q = a < 0 || e < a || e > p.num_tokens, bad_c = ctx < 0 || ctx > cap;
    if (flag && (bad_q || bad_c))
        raise_err(p.d.err_flag, (bad_q ? PKV_DEVERR_QSTART_RANGE : 0) | (bad_c ? PKV_DEVERR_CONTEXT_RANGE : 0));
    s.s0 = a;
    s.n = bad_q ? 0 : e - a;
    s.ctx = ctx < 0 ? 0 : ctx > cap ? cap : ctx;
    s.rows = s.n * p.d.group;
    s.nt = (s.rows + kRowTile - 1) / kRowTile;
    return s;
}

// keys that row r (token r / group) of the sequence sees
__device__ __forceinline__ int row_limit(const PrefillParams &p, const Seq &s, int r)
{
    return max(0, s.ctx - s.n + r / p.d.group + 1);
}
// keys that some row of the tile sees
__device__ __forceinline__ int tile_limit(const PrefillParams &p, const Seq &s, int tile)
{
    return row_limit(p, s, min((tile + 1) * kRowTile, s.rows) - 1);
}
// units of a row tile: at least one, so that rows that see nothing are written
__device__ __forceinline__ int tile_units(int limit) { return max(1, (limit + kKeyTile - 1) / kKeyTile); }

// A CTA's walk over its segments: maximal runs of key tiles of one row tile.
struct Walk {
    int64_t left;               // units from this segment on
    Seq s;
    int b, h, tile, k0, k1, units, limit;
    __device__ __forceinline__ void shape(const PrefillParams &p)
    {
        limit = tile_limit(p, s, tile);
        units = tile_units(limit);
        k1 = int(min(int64_t(units), k0 + left));
    }
    __device__ __forceinline__ bool next(const PrefillParams &p)
    {
        left -= k1 - k0;
        if (left <= 0) return false;
        k0 = 0;
        if (++tile == s.nt) {
            tile = 0;
            if (++h == p.d.num_kv_heads) {
                h = 0;
                do s = seq_load(p, ++b, false); while (s.n == 0);
            }
        }
        shape(p);
        return true;
    }
    __device__ __forceinline__ int subtiles() const { return s.rows - tile * kRowTile > 128 ? 2 : 1; }
};

struct Start {
    int64_t u0, u1, total;      // this CTA's units, all units
    int ctas;                   // CTAs that have work
    int b, h, tile, k0;
};

__device__ __forceinline__ Walk walk_from(const PrefillParams &p, const Start &st)
{
    Walk w;
    w.left = st.u1 - st.u0;
    w.b = st.b;
    w.h = st.h;
    w.tile = st.tile;
    w.k0 = st.k0;
    w.s = seq_load(p, st.b, false);
    w.shape(p);
    return w;
}

// units of sequence s and one kv head, summed over `lanes` (a power of two)
// threads of a warp; every thread of the warp calls it
__device__ __forceinline__ int64_t seq_units(const PrefillParams &p, const Seq &s, int lane, int lanes)
{
    int64_t u = 0;
    for (int i = lane; i < s.nt; i += lanes) u += tile_units(tile_limit(p, s, i));
    for (int o = lanes >> 1; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    return u;
}

// This CTA's share.  Sequences are counted in at most kBins bins (`bins`,
// kBins + 1 entries of shared memory, dead afterwards).
__device__ __forceinline__ void find_start(const PrefillParams &p, int64_t *bins, Start *out)
{
    const int B = p.d.batch, Hkv = p.d.num_kv_heads;
    const int per = (B + kBins - 1) / kBins, nb = (B + per - 1) / per;
    const int lane = threadIdx.x & 31;
    int lanes = 32;
    while (lanes > 1 && nb * lanes > int(blockDim.x)) lanes >>= 1;
    const int groups = blockDim.x / lanes, group = threadIdx.x / lanes, sub = threadIdx.x % lanes;
    for (int b0 = 0; b0 < nb; b0 += groups) {
        const int bin = b0 + group;
        int64_t u = 0;
        for (int j = 0; j < per; ++j) {
            const int b = bin * per + j;
            Seq s{};
            if (bin < nb && b < B) s = seq_load(p, b, blockIdx.x == 0 && sub == 0);
            u += seq_units(p, s, sub, lanes);
        }
        if (bin < nb && sub == 0) bins[bin] = u * Hkv;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int64_t total = 0;
        for (int b0 = 0; b0 < nb; b0 += 32) {           // exclusive sums
            const int64_t v = b0 + lane < nb ? bins[b0 + lane] : 0;
            int64_t x = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (b0 + lane < nb) bins[b0 + lane] = total + x - v;
            total += __shfl_sync(0xffffffffu, x, 31);
        }
        __syncwarp();
        Start st{};
        st.total = total;
        st.ctas = int(min(int64_t(gridDim.x), total));
        if (int(blockIdx.x) < st.ctas) {
            st.u0 = blockIdx.x * total / st.ctas;
            st.u1 = (blockIdx.x + 1) * total / st.ctas;
            int bin = -1;                               // the last bin that starts at or before u0
            for (int b0 = 0; b0 < nb; b0 += 32)
                bin += __popc(__ballot_sync(0xffffffffu, b0 + lane < nb && bins[b0 + lane] <= st.u0));
            int64_t u = st.u0 - bins[bin], su = 0;
            Seq s{};
            for (st.b = bin * per;; ++st.b) {
                s = seq_load(p, st.b, false);
                su = seq_units(p, s, lane, 32);
                if (u < su * Hkv) break;
                u -= su * Hkv;
            }
            st.h = int(u / su);
            u -= st.h * su;
            const int c = (s.nt + 31) / 32;             // row tiles per lane
            int64_t mine = 0;
            for (int i = lane * c; i < min((lane + 1) * c, s.nt); ++i) mine += tile_units(tile_limit(p, s, i));
            int64_t x = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const unsigned below = __ballot_sync(0xffffffffu, x <= u);      // lanes wholly before u
            const int at = __popc(below);
            u -= at ? __shfl_sync(0xffffffffu, x, at - 1) : 0;
            for (st.tile = at * c;; ++st.tile) {
                const int t = tile_units(tile_limit(p, s, st.tile));
                if (u < t) break;
                u -= t;
            }
            st.k0 = int(u);
        }
        if (lane == 0) *out = st;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- shared memory
template <int D>
struct Smem {
    static constexpr int kTile = 128 * D * 2;                   // bytes of 128 rows
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kColSlots = kStages;                    // see ColSlot
    static constexpr int q = 0;
    static constexpr int ring = 2 * kTile;
    static constexpr int cols = ring + kStages * kTile;         // kColSlots x ColSlot
    static constexpr int kColBytes = 2 * kKeyTile * 4 + 32;
    static constexpr int bars = cols + kColSlots * kColBytes;
    static constexpr int n_bars = 2 * kStages + 2 + 4 * 2 + 1;
    static constexpr int misc = bars + 8 * n_bars;
    static constexpr int total = misc + 128;
    static constexpr int alloc = total + 1024;                  // the base is rounded up to 1024
    static_assert(kStages * kTile >= (kBins + 1) * 8, "bins lie in the ring");
    static_assert(alloc <= 232448, "shared memory of a CTA");
    static_assert(sizeof(Start) <= 96, "misc");
};

// Column data of a key tile: scales of its 128 K and V rows, the largest V
// scale of each 32 rows, and which groups of 8 rows are there.  Tile T's is
// written once K's stage of tile T - kStages / 2 is free: its products are
// done then, and both subtiles' softmax of the tiles before it, so a ring of
// kStages / 2 + 1 slots or more is never written while it is read.
struct ColSlot {
    float k[kKeyTile];
    float v[kKeyTile];
    float vmax[4];
    uint32_t mask[4];           // 4 bits per 32 rows (one word per loader warp; word 0 holds all 16 for the TMA producer)
};

struct Bars {
    uint32_t base;
    int stages;
    __device__ __forceinline__ uint32_t full(int s) const { return base + 8 * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return base + 8 * (stages + s); }
    __device__ __forceinline__ uint32_t q_full() const { return base + 8 * (2 * stages); }
    __device__ __forceinline__ uint32_t q_empty() const { return base + 8 * (2 * stages + 1); }
    __device__ __forceinline__ uint32_t s_full(int i) const { return base + 8 * (2 * stages + 2 + i); }
    __device__ __forceinline__ uint32_t p_full(int i) const { return base + 8 * (2 * stages + 4 + i); }
    __device__ __forceinline__ uint32_t o_full(int i) const { return base + 8 * (2 * stages + 6 + i); }
    __device__ __forceinline__ uint32_t p_half(int i) const { return base + 8 * (2 * stages + 8 + i); }
    __device__ __forceinline__ uint32_t tail() const { return base + 8 * (2 * stages + 10); }
};

// Wait for a phase, giving up when it takes too long or another warp gave up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *gone)
{
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    uint32_t n = 0;
    while (!ptx::mbar_try_wait(bar, parity)) {
        if ((++n & 15u) == 0 && (*gone || ptx::globaltimer() - t0 > kPrefillTimeoutNs)) {
            *gone = 1;
            return false;
        }
    }
    return true;
}

// the same for a whole warp: every lane gives up or none
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *gone)
{
    return __all_sync(0xffffffffu, bar_wait(bar, parity, gone));
}

// byte offset of 16-byte piece `c` of row `r` in a tile of 128-byte swizzled
// rows, [64-element chunk][128 rows][128 bytes]
__device__ __forceinline__ uint32_t piece_at(int r, int c)
{
    return uint32_t((c >> 3) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <int N> __device__ __forceinline__ float2 f2(const uint32_t (&x)[N], int j)
{
    return make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1]));
}

// ---------------------------------------------------------------- codes -> 16 bits
__device__ __forceinline__ uint32_t sub16x2(uint32_t a, uint32_t b, bool bf16)
{
    uint32_t r;
    if (bf16)
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// four one-byte codes -> four 16-bit numbers, exactly
template <int QK, int CK>
__device__ __forceinline__ uint2 q8x4_to_16(uint32_t w)
{
    if constexpr (CK == kI8) {
        const uint32_t u = w ^ 0x80808080u;                     // c + 128
        if constexpr (QK == kF16) {                             // 1024 + (c + 128), minus 1152
            return make_uint2(sub16x2(ptx::prmt(u, 0x64646464u, 0x4140), 0x64806480u, false),
                              sub16x2(ptx::prmt(u, 0x64646464u, 0x4342), 0x64806480u, false));
        } else {                                                // 2^23 + (c + 128) in fp32, minus 2^23 + 128
            float f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                f[j] = __uint_as_float(ptx::prmt(u, 0x4b000000u, 0x7540 | j)) - 8388736.0f;
            return make_uint2(tc::pack16<kBF16>(f[0], f[1]), tc::pack16<kBF16>(f[2], f[3]));
        }
    } else {
        uint32_t lo, hi;
        if constexpr (CK == kE4M3)
            asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
                : "=r"(lo), "=r"(hi) : "r"(w));
        else
            asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e5m2x2 %0, l;\ncvt.rn.f16x2.e5m2x2 %1, h;\n}"
                : "=r"(lo), "=r"(hi) : "r"(w));
        if constexpr (QK == kF16) {
            return make_uint2(lo, hi);
        } else {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            return make_uint2(tc::pack16<kBF16>(a.x, a.y), tc::pack16<kBF16>(b.x, b.y));
        }
    }
}

// eight 3-bit codes (the low 24 bits of w) minus their zero point, as 16-bit
// numbers: the code under a power of two whose unit step is 1.  zero2: the
// zero point twice (bf16), or 1024 more (f16)
template <int QK>
__device__ __forceinline__ uint4 u3x8_to_16(uint32_t w, uint32_t zero2)
{
    // bf16 takes the zero point off in a second step: 128 + z need not be a bf16 number
    constexpr uint32_t magic = QK == kBF16 ? 0x43004300u : 0x64006400u;     // 128, 1024
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t x = w >> (6 * j);
        const uint32_t u = (x & 7u) | ((x << 13) & 0x70000u) | magic;
        o[j] = QK == kBF16 ? sub16x2(sub16x2(u, magic, true), zero2, true) : sub16x2(u, zero2, false);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// ---------------------------------------------------------------- K/V by loads
// Rows 32 lw .. 32 lw + 31 of every key tile, by one warp (lane = row for
// the lookups): codes are loaded, converted to the 16-bit operand type and
// stored swizzled; 16-bit pieces are copied.  A stage's loads are issued
// before the stage before it is converted.
template <int QK, int CK, int D, bool GS>
__device__ __forceinline__ void load_rows(const PrefillParams &p, const PrefillFast &f, const Start &st, bool work,
                                          uint32_t ring, ColSlot *cols, const Bars &bars, volatile int *gone, int lw,
                                          int lane)
{
    using L = Smem<D>;
    constexpr int ST = L::kStages;
    constexpr bool kCopy = CK == kF16 || CK == kBF16;
    constexpr int kLoads = CK == kU3 ? D / 32 : D / 16;         // per lane and stage (codes)
    constexpr int kWords = CK == kU3 ? 3 : 4;
    if (!work) return;
    const DecodeParams &d = p.d;
    const int row = 32 * lw + lane;
    Walk w = walk_from(p, st);
    uint32_t pos = 0, tile_n = 0;
    int k = w.k0;
    // this lane's row of the current tile
    int64_t at = 0;
    bool in = false;
    float ks = 0.0f, vs = 0.0f, kz = 0.0f, vz = 0.0f;
    auto lookup = [&]() {
        const int t = k * kKeyTile + row;
        in = t < w.limit;
        int64_t blk = 0;
        if (in) {
            blk = d.block_tables[w.b * d.bt_b + int64_t(t >> d.block_shift) * d.bt_j];
            if (blk < 0 || blk >= d.num_blocks) {
                raise_err(d.err_flag, PKV_DEVERR_BLOCK_RANGE);
                in = false;
            }
        }
        const int64_t slot = t & (d.block_size - 1);
        at = in ? blk * d.c_blk + slot * d.c_slot + w.h * d.c_head : 0;
        if constexpr (GS) {
            ks = vs = kz = vz = 0.0f;
            if (in) {
                if constexpr (CK == kU3) {
                    const int64_t m = blk * d.m_blk + slot * d.m_slot + w.h * d.m_head;
                    const int64_t z = blk * d.z_blk + slot * d.z_slot + w.h * d.z_head;
                    ks = __half2float(__ushort_as_half(__ldg(d.k_qs + m)));
                    vs = __half2float(__ushort_as_half(__ldg(d.v_qs + m)));
                    kz = float(__ldg(d.k_qz + z));
                    vz = float(__ldg(d.v_qz + z));
                } else {
                    const int64_t m = blk * d.gs_blk + slot * d.gs_slot + w.h * d.gs_head;
                    ks = __ldg(d.k_gs + m);
                    vs = __ldg(d.v_gs + m);
                }
            }
        }
    };
    auto columns = [&]() {                                      // before K's arrival
        ColSlot &cs = cols[tile_n % L::kColSlots];
        const unsigned got = __ballot_sync(0xffffffffu, in);
        if constexpr (GS) {
            cs.k[row] = ks;
            cs.v[row] = vs;
            float mx = vs;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane == 0) cs.vmax[lw] = mx;
        }
        if (lane == 0) {
            uint32_t there = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) there |= ((got >> (8 * i)) & 0xffu ? 1u : 0u) << (4 * lw + i);
            cs.mask[lw] = there;
        }
    };
    auto step = [&]() -> bool {                                 // to the next tile
        ++tile_n;
        if (++k < w.k1) return true;
        if (!w.next(p)) return false;
        k = w.k0;
        return true;
    };
    auto room = [&]() -> bool {
        return pos < ST || warp_wait(bars.empty(pos % ST), (pos / ST - 1) & 1, gone);
    };
    auto arrive = [&](uint32_t stage) {
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars.full(stage));
    };
    if constexpr (kCopy) {
        // a lane copies its row's 16-byte pieces (neighbouring slots are
        // neighbours in the x-vectorised layout); a stage is handed over
        // once the next one's copies are under way
        int pending = -1;
        auto flush = [&](bool all) {
            if (pending < 0) return;
            if (all) tc::cp_async_wait<0>(); else tc::cp_async_wait<1>();
            arrive(pending);
            pending = -1;
        };
        bool more = true;
        while (more) {
            lookup();
            for (int kv = 0; kv < 2; ++kv, ++pos) {
                // never wait for room with a stage in hand
                if (!__all_sync(0xffffffffu, pos < ST || ptx::mbar_try_wait(bars.empty(pos % ST), (pos / ST - 1) & 1)))
                    flush(true);
                if (!room()) return;
                if (kv == 0) columns();
                const char *src = (kv ? d.v_cache : d.k_cache) + at;
                const uint32_t dst = ring + (pos % ST) * L::kTile;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) tc::cp_async16(dst + piece_at(row, c), src + (in ? c * d.c_chunk : 0), in);
                tc::cp_async_commit();
                flush(false);
                pending = int(pos % ST);
            }
            more = step();
        }
        flush(true);
    } else {
        uint32_t kr[kLoads][kWords], vr[kLoads][kWords];
        // lane -> (row of 32, piece): 16 codes of a one-byte row, 32 codes
        // (12 bytes) of a 3-bit row; the 8 lanes of a store phase hit
        // 8 different 16-byte columns of the banks
        auto place = [&](int i, int &r, int &c) {
            if constexpr (CK == kU3) {
                r = (lane >> 1) + 16 * (i & 1);
                c = (lane & 1) + 2 * (i >> 1);
            } else {
                r = i * (32 / kLoads) + lane / kLoads;
                c = lane % kLoads;
            }
        };
        auto load = [&](const char *cache, uint32_t (&x)[kLoads][kWords]) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                int r, c;
                place(i, r, c);
                const int64_t o = __shfl_sync(0xffffffffu, at, r);
                const bool ok = __shfl_sync(0xffffffffu, int(in), r);
#pragma unroll
                for (int j = 0; j < kWords; ++j) x[i][j] = 0u;
                if constexpr (CK == kU3) {
                    const char *src = cache + o + 12 * c;
                    if (!ok) {
                    } else if (f.rows_aligned) {
#pragma unroll
                        for (int j = 0; j < 3; ++j) x[i][j] = __ldg(reinterpret_cast<const uint32_t *>(src) + j);
                    } else {
#pragma unroll
                        for (int j = 0; j < 12; ++j)
                            x[i][j >> 2] |= uint32_t(__ldg(reinterpret_cast<const uint8_t *>(src) + j)) << (8 * (j & 3));
                    }
                } else {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (ok) v = __ldg(reinterpret_cast<const uint4 *>(cache + o + c * d.c_chunk));
                    x[i][0] = v.x;
                    x[i][1] = v.y;
                    x[i][2] = v.z;
                    x[i][kWords - 1] = v.w;
                }
            }
        };
        auto store = [&](uint32_t dst, const uint32_t (&x)[kLoads][kWords], float zero) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                int r, c;
                place(i, r, c);
                const int rr = 32 * lw + r;
                if constexpr (CK == kU3) {
                    const float z = __shfl_sync(0xffffffffu, zero, r);
                    const uint32_t z2 = QK == kBF16 ? tc::pack16<QK>(z, z) : tc::pack16<QK>(1024.0f + z, 1024.0f + z);
                    const uint32_t w0 = x[i][0], w1 = x[i][1], w2 = x[i][2];
                    const uint32_t fl[4] = {w0, __funnelshift_r(w0, w1, 24), __funnelshift_r(w1, w2, 16), w2 >> 8};
#pragma unroll
                    for (int j = 0; j < 4; ++j) tc::st_shared16(dst + piece_at(rr, 4 * c + j), u3x8_to_16<QK>(fl[j], z2));
                } else {
                    uint4 o[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint2 a = q8x4_to_16<QK, CK>(x[i][2 * j]), b = q8x4_to_16<QK, CK>(x[i][2 * j + 1]);
                        o[j] = make_uint4(a.x, a.y, b.x, b.y);
                    }
                    const int a = D == 128 ? c >> 2 : 0;
                    tc::st_shared16(dst + piece_at(rr, 2 * c + a), a ? o[1] : o[0]);
                    tc::st_shared16(dst + piece_at(rr, 2 * c + 1 - a), a ? o[0] : o[1]);
                }
            }
        };
        lookup();
        load(d.k_cache, kr);
        bool more = true;
        while (more) {
            load(d.v_cache, vr);
            const float kz_now = kz, vz_now = vz;
            if (!room()) return;
            columns();
            more = step();
            if (more) lookup();
            store(ring + (pos % ST) * L::kTile, kr, kz_now);
            arrive(pos % ST);
            ++pos;
            if (more) load(d.k_cache, kr);
            if (!room()) return;
            store(ring + (pos % ST) * L::kTile, vr, vz_now);
            arrive(pos % ST);
            ++pos;
        }
    }
}

// ---------------------------------------------------------------- the kernel
template <bool TMA> constexpr int prefill_threads() { return TMA ? 384 : 448; }

template <int QK, int CK, int D, bool TMA, bool GS>
__global__ void __launch_bounds__(prefill_threads<TMA>(), 1)
    prefill_kernel(PrefillParams p, PrefillFast f, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv)
{
    using L = Smem<D>;
    constexpr int ST = L::kStages;
    constexpr bool BF = QK == kBF16;
    constexpr int kMmaWarp = TMA ? 8 : 12;
    constexpr int kQWarp = TMA ? 10 : 13;
    constexpr int kQWarps = TMA ? 2 : 1;
    constexpr bool kVRef = GS && QK == kF16;                    // V scales are taken relative to a power of two
    const DecodeParams &d = p.d;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm32 = ptx::smem_u32(sm);
    Start *start = reinterpret_cast<Start *>(sm + L::misc);
    volatile int *gone = reinterpret_cast<volatile int *>(sm + L::misc + 96);
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(sm + L::misc + 104);
    ColSlot *cols = reinterpret_cast<ColSlot *>(sm + L::cols);
    static_assert(sizeof(ColSlot) == L::kColBytes, "column slots");
    const Bars bars{sm32 + L::bars, ST};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            ptx::mbar_init(bars.full(i), TMA ? 1 : 4);
            ptx::mbar_init(bars.empty(i), 1);
        }
        ptx::mbar_init(bars.q_full(), kQWarps);
        ptx::mbar_init(bars.q_empty(), 1);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bars.s_full(i), 1);
            ptx::mbar_init(bars.p_full(i), 4);
            ptx::mbar_init(bars.p_half(i), 4);
            ptx::mbar_init(bars.o_full(i), 1);
        }
        ptx::mbar_init(bars.tail(), 1);
        ptx::fence_mbar_init();
        *gone = 0;
    }
    if (warp == kMmaWarp) tc::tmem_alloc(ptx::smem_u32(tmem_at), 512);
    griddep_wait();
    griddep_launch_dependents();
    find_start(p, reinterpret_cast<int64_t *>(sm + L::ring), start);     // ends with __syncthreads
    tc::fence_after();
    const uint32_t tmem = *tmem_at;
    const Start st = *start;
    const bool work = st.u1 > st.u0;

    if (warp < 8) {
        // ------------------------------------------------ softmax, a thread per row
        const int sub = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + sub * 128, to = tmem + lanes + 256 + sub * 128;
        uint32_t tile_n = 0, mine_n = 0, item_n = 0;            // key tiles of the CTA, of this subtile, segments
        if (work) {
            Walk w = walk_from(p, st);
            do {
                if (sub >= w.subtiles()) {
                    tile_n += w.k1 - w.k0;
                    continue;
                }
                const int r = w.tile * kRowTile + sub * 128 + row;
                const bool live = r < w.s.rows;
                const int lim = live ? row_limit(p, w.s, r) : 0;
                float c = fabsf(d.scale_log2);
                if constexpr (is_q8(CK) && !GS) c *= fabsf(d.k_scale[w.h]);
                c = fmaxf(c, 1e-30f);                           // keeps 0 * -inf out: masked weights stay zero
                const float ninf = -__int_as_float(0x7f800000);
                float m = ninf, l = 0.0f, vref = 0.0f;
                bool ok = true;
                for (int k = w.k0; k < w.k1; ++k, ++tile_n, ++mine_n) {
                    ok = warp_wait(bars.s_full(sub), mine_n & 1, gone);
                    if (!ok) break;
                    tc::fence_after();
                    const ColSlot &cs = cols[tile_n % L::kColSlots];
                    // the tile's columns in four chunks of 32.  Three stay in registers from
                    // the maximum on; chunk 2 is read twice, which costs less than the
                    // registers would.
                    uint32_t a[32], b[32], t[32];
                    tc::tmem_ld32(ts, a, 0);
                    tc::tmem_ld32(ts + 64, t, 0);
                    tc::tmem_ld32(ts + 32, b, 0);
                    // keys behind the row's limit, and blocks that are not there
                    uint32_t there = cs.mask[0];
                    if constexpr (!TMA) there |= cs.mask[1] | cs.mask[2] | cs.mask[3];
                    const int rel = lim - k * kKeyTile;
                    const bool masked = __any_sync(0xffffffffu, rel < kKeyTile || there != 0xffffu);
                    // scales and mask of a chunk
                    auto prepare = [&](uint32_t (&x)[32], int ch) {
                        if constexpr (GS) {
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                const float4 ks = *reinterpret_cast<const float4 *>(cs.k + 32 * ch + j);
                                const float2 u = tc::mul2(f2(x, j), make_float2(ks.x, ks.y));
                                const float2 v = tc::mul2(f2(x, j + 2), make_float2(ks.z, ks.w));
                                x[j] = __float_as_uint(u.x);
                                x[j + 1] = __float_as_uint(u.y);
                                x[j + 2] = __float_as_uint(v.x);
                                x[j + 3] = __float_as_uint(v.y);
                            }
                        }
                        if (masked) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (32 * ch + j >= rel || !((there >> (4 * ch + (j >> 3))) & 1u)) x[j] = 0xff800000u;
                        }
                    };
                    float mx[4] = {ninf, ninf, ninf, ninf};
                    auto largest = [&](const uint32_t (&x)[32]) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mx[i] = fmaxf(fmaxf(mx[i], __uint_as_float(x[j + i])), __uint_as_float(x[j + 4 + i]));
                    };
                    tc::tmem_ld_wait32(a, 0);
                    tc::tmem_ld_wait32(t, 0);
                    tc::tmem_ld_wait32(b, 0);
                    prepare(t, 2);
                    largest(t);
                    tc::tmem_ld32(ts + 96, t, 0);
                    prepare(a, 0);
                    largest(a);
                    prepare(b, 1);
                    largest(b);
                    tc::tmem_ld_wait32(t, 0);
                    prepare(t, 3);
                    largest(t);
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    float grow = 1.0f;                          // what O and l shrink by
                    if (top > m && (m == ninf || (top - m) * c > 8.0f)) {
                        grow = m == ninf ? 0.0f : exp2_approx((m - top) * c);
                        l *= grow;
                        m = top;
                    }
                    float vinv = 1.0f;
                    if constexpr (kVRef) {
                        // a power of two at or above the tile's V scales
                        const float vm = fmaxf(fmaxf(cs.vmax[0], cs.vmax[1]), fmaxf(cs.vmax[2], cs.vmax[3]));
                        const float v2 = __uint_as_float(min((__float_as_uint(fmaxf(vm, 1e-30f)) >> 23) + 1, 254u) << 23);
                        if (v2 > vref) {
                            grow *= vref / v2;
                            vref = v2;
                        }
                        vinv = 1.0f / vref;
                    }
                    if (k > w.k0 && __any_sync(0xffffffffu, grow != 1.0f)) {
                        // seldom: a rolled loop keeps its registers out of the way
#pragma unroll 1
                        for (int o = 0; o < D; o += 16) {
                            uint32_t x[16];
                            tc::tmem_ld16_wait(to + o, x);
#pragma unroll
                            for (int j = 0; j < 16; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * grow);
                            tc::tmem_st16(to + o, x);
                        }
                    }
                    const float off = m == ninf ? 0.0f : m * c;
                    const float2 c2 = make_float2(c, c), off2 = make_float2(-off, -off);
                    float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                    auto weights = [&](const uint32_t (&x)[32], int ch) {
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            const float2 y = tc::fma2(f2(x, j), c2, off2);
                            float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                            sum[(j >> 1) & 1] = tc::add2(sum[(j >> 1) & 1], e);
                            if constexpr (GS) {
                                float2 vs = *reinterpret_cast<const float2 *>(cs.v + 32 * ch + j);
                                if constexpr (kVRef) vs = tc::mul2(vs, make_float2(vinv, vinv));
                                const float2 z = tc::mul2(e, vs);
                                e.x = masked && e.x == 0.0f ? 0.0f : z.x;
                                e.y = masked && e.y == 0.0f ? 0.0f : z.y;
                            }
                            pk[j >> 1] = tc::pack16<QK>(e.x, e.y);
                        }
                        tc::tmem_st16(ts + 16 * ch, pk);
                    };
                    auto hand = [&](uint32_t bar) {
                        tc::tmem_st_wait();
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bar);
                    };
                    // P overwrites chunks 0 and 1, which are in registers by now
                    weights(a, 0);
                    tc::tmem_ld32(ts + 64, a, 0);
                    weights(b, 1);
                    tc::tmem_ld_wait32(a, 0);
                    hand(bars.p_half(sub));
                    prepare(a, 2);
                    weights(a, 2);
                    weights(t, 3);
                    hand(bars.p_full(sub));
                    sum[0] = tc::add2(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                }
                if (!ok || !warp_wait(bars.o_full(sub), item_n & 1, gone)) break;
                ++item_n;
                tc::fence_after();
                const bool whole = w.k0 == 0 && w.k1 == w.units;
                float fac = kVRef ? vref : 1.0f;
                if constexpr (is_q8(CK) && !GS) fac = d.v_scale[w.h];
                if (whole) {
                    fac = l == 0.0f ? 0.0f : fac / l;
                    const int tok = r / d.group;
                    const int head = w.h * d.group + (r - tok * d.group);
                    char *o_row = d.out + int64_t(w.s.s0 + tok) * d.o_b + int64_t(head) * d.o_h;
                    float bad = 0.0f;
#pragma unroll
                    for (int o = 0; o < D; o += 32) {
                        uint32_t a[32];
                        tc::tmem_ld32(to + o, a, 0);
                        tc::tmem_ld_wait32(a, 0);
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            // a row without keys is zero whatever O holds
                            const float x = l == 0.0f ? 0.0f : __uint_as_float(a[j]) * fac;
                            const float y = l == 0.0f ? 0.0f : __uint_as_float(a[j + 1]) * fac;
                            bad = fmaf(x, 0.0f, fmaf(y, 0.0f, bad));
                            pk[j / 2] = tc::pack16<QK>(x, y);
                        }
                        if (live) {
                            if (d.out_vec_ok) {
#pragma unroll
                                for (int j = 0; j < 16; j += 4)
                                    *reinterpret_cast<uint4 *>(o_row + 2 * (o + 2 * j)) =
                                        make_uint4(pk[j], pk[j + 1], pk[j + 2], pk[j + 3]);
                            } else {
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    reinterpret_cast<uint16_t *>(o_row)[o + 2 * j] = uint16_t(pk[j]);
                                    reinterpret_cast<uint16_t *>(o_row)[o + 2 * j + 1] = uint16_t(pk[j] >> 16);
                                }
                            }
                        }
                    }
                    // not finite: weights of zero met values that are not; such a row is done again by itself
                    unsigned redo = __ballot_sync(0xffffffffu, live && bad != 0.0f);
                    if (redo) tc::fence_before();
                    while (redo) {
                        const int who = __ffs(redo) - 1;
                        redo &= redo - 1;
                        const int rr = __shfl_sync(0xffffffffu, r, who), ll = __shfl_sync(0xffffffffu, lim, who);
                        const int tt = rr / d.group;
                        redo_row<QK, CK, D>(d, d.block_tables + w.b * d.bt_b, int64_t(w.s.s0) + tt,
                                            w.h * d.group + (rr - tt * d.group), ll, w.limit, 0, D);
                    }
                } else {
                    const int slot = 2 * blockIdx.x + (w.k0 == 0 ? 1 : 0);
                    float *ml = f.part_ml + int64_t(slot) * 2 * kRowTile + sub * 128 + row;
                    ml[0] = m == ninf ? m : m * c;
                    ml[kRowTile] = l;
                    float4 *acc = reinterpret_cast<float4 *>(f.part_acc) +
                                  int64_t(slot) * (D / 4) * kRowTile + sub * 128 + row;
#pragma unroll
                    for (int o = 0; o < D; o += 32) {
                        uint32_t a[32];
                        tc::tmem_ld32(to + o, a, 0);
                        tc::tmem_ld_wait32(a, 0);
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            acc[(o + j) / 4 * kRowTile] =
                                make_float4(__uint_as_float(a[j]) * fac, __uint_as_float(a[j + 1]) * fac,
                                            __uint_as_float(a[j + 2]) * fac, __uint_as_float(a[j + 3]) * fac);
                    }
                }
                tc::fence_before();
            } while (w.next(p));
        }
    } else {
        if (warp == kMmaWarp) {
            // -------------------------------------------- the products
            if (work && lane == 0) {
                constexpr uint32_t id_qk = tc::instr_desc<BF, false, 128, 128>();
                constexpr uint32_t id_pv = tc::instr_desc<BF, true, 128, D>();
                uint32_t pos = 0, item = 0, n_p[2] = {0, 0};
                Walk w = walk_from(p, st);
                auto qk = [&](int i, uint32_t stage) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t o = (ks >> 2) * 16384 + (ks & 3) * 32;
                        tc::mma_ss(tmem + i * 128, tc::smem_desc(sm32 + L::q + i * L::kTile + o, 16, 1024),
                                   tc::smem_desc(sm32 + L::ring + stage * L::kTile + o, 16, 1024), id_qk, ks > 0);
                    }
                    tc::commit(bars.s_full(i));
                };
                bool ok = true;
                do {
                    const int ns = w.subtiles(), nk = w.k1 - w.k0;
                    ok = bar_wait(bars.q_full(), item & 1, gone) &&
                         bar_wait(bars.full(pos % ST), (pos / ST) & 1, gone);
                    if (!ok) break;
                    tc::fence_after();
                    for (int i = 0; i < ns; ++i) qk(i, pos % ST);
                    tc::commit(bars.empty(pos % ST));
                    if (nk == 1) tc::commit(bars.q_empty());
                    for (int j = 0; j < nk && ok; ++j) {
                        const uint32_t vpos = pos + 1, kpos = pos + 2;
                        for (int i = 0; i < ns; ++i) {
                            ok = bar_wait(bars.p_half(i), n_p[i] & 1, gone);
                            if (ok && i == 0) ok = bar_wait(bars.full(vpos % ST), (vpos / ST) & 1, gone);
                            if (!ok) break;
                            tc::fence_after();
                            // P in two halves: the first keys' products run while the others' weights are made
                            auto pv = [&](int ks) {
                                tc::mma_ts(tmem + 256 + i * 128, tmem + i * 128 + ks * 8,
                                           tc::smem_desc(sm32 + L::ring + (vpos % ST) * L::kTile + ks * 2048, 16384, 1024),
                                           id_pv, j > 0 || ks > 0);
                            };
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks) pv(ks);
                            ok = bar_wait(bars.p_full(i), n_p[i] & 1, gone);
                            if (!ok) break;
                            ++n_p[i];
                            tc::fence_after();
#pragma unroll
                            for (int ks = 4; ks < 8; ++ks) pv(ks);
                            if (j + 1 < nk) {
                                if (i == 0) {
                                    ok = bar_wait(bars.full(kpos % ST), (kpos / ST) & 1, gone);
                                    if (!ok) break;
                                    tc::fence_after();
                                }
                                qk(i, kpos % ST);
                            } else {
                                tc::commit(bars.o_full(i));
                            }
                        }
                        if (!ok) break;
                        tc::commit(bars.empty(vpos % ST));
                        if (j + 1 < nk) {
                            tc::commit(bars.empty(kpos % ST));
                            if (j + 2 == nk) tc::commit(bars.q_empty());
                        }
                        pos += 2;
                    }
                    ++item;
                } while (ok && w.next(p));
            }
            __syncwarp();
        } else if (warp >= kQWarp && warp < kQWarp + kQWarps) {
            // -------------------------------------------- Q, a warp per subtile or one for both
            const int first = warp - kQWarp;
            const bool negate = d.scale_log2 < 0.0f;
            constexpr int PPR = D / 8;                          // pieces per row
            constexpr int RPI = 32 / PPR;                       // rows per instruction
            Walk w;
            uint32_t item = 0;
            bool have = work;
            if (work) w = walk_from(p, st);
            while (have) {
                if (item > 0 && !warp_wait(bars.q_empty(), (item - 1) & 1, gone)) break;
                for (int sub = first; sub < w.subtiles(); sub += kQWarps) {
                    const int c = lane % PPR;
                    int r = w.tile * kRowTile + sub * 128 + lane / PPR;
                    int tok = r / d.group, g = r - tok * d.group;
                    const uint32_t dst = sm32 + L::q + sub * L::kTile;
#pragma unroll 4
                    for (int i = lane / PPR; i < 128; i += RPI, r += RPI) {
                        const bool in = r < w.s.rows;
                        const char *src = d.q + int64_t(w.s.s0 + tok) * d.q_b + int64_t(w.h * d.group + g) * d.q_h + 16 * c;
                        tc::cp_async16(dst + piece_at(i, c), in ? src : d.q, in);
                        g += RPI;
                        while (g >= d.group) {
                            g -= d.group;
                            ++tok;
                        }
                    }
                }
                tc::cp_async_wait_all();
                for (int sub = first; negate && sub < w.subtiles(); sub += kQWarps) {
                    const uint32_t dst = sm32 + L::q + sub * L::kTile;
                    const int c = lane % PPR;
                    for (int i = lane / PPR; i < 128; i += RPI) {
                        uint4 v = tc::ld_shared16(dst + piece_at(i, c));
                        v.x ^= 0x80008000u;
                        v.y ^= 0x80008000u;
                        v.z ^= 0x80008000u;
                        v.w ^= 0x80008000u;
                        tc::st_shared16(dst + piece_at(i, c), v);
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bars.q_full());
                ++item;
                have = w.next(p);
            }
            if (first == 0 && lane == 0) {
                // the row tile that this CTA begins and does not end
                int4 ds = make_int4(0, 0, 0, -1);
                if (work && !have && w.k0 == 0 && w.k1 < w.units) {
                    const int64_t end = st.u1 - w.k1 + w.units;
                    ds = make_int4(w.b, w.h, w.tile, int((end * st.ctas + st.total - 1) / st.total) - 1);
                }
                f.desc[blockIdx.x] = ds;
            }
        } else if (TMA && warp == 9) {
            // -------------------------------------------- K/V by TMA: whole blocks' pieces of 64 elements
            const int shift = min(d.block_shift, 7);            // rows per box
            const int rows = 1 << shift, nblk = kKeyTile >> shift;
            const uint32_t box = uint32_t(rows) * 128u;
            uint32_t pos = 0, tile_n = 0, fixes = 0;
            if (lane == 0) {
                ptx::prefetch_tmap(&tmk);
                ptx::prefetch_tmap(&tmv);
            }
            if (work) {
                Walk w = walk_from(p, st);
                bool ok = true;
                do {
                    const int32_t *table = d.block_tables + w.b * d.bt_b;
                    auto lookup = [&](int k) -> int {           // this lane's block of key tile k
                        const int t = k * kKeyTile + lane * rows;
                        return lane < nblk && t < w.limit ? table[int64_t(t >> d.block_shift) * d.bt_j] : -1;
                    };
                    int blk = lookup(w.k0);
                    for (int k = w.k0; k < w.k1 && ok; ++k, ++tile_n) {
                        const int t = k * kKeyTile + lane * rows;
                        const bool want = lane < nblk && t < w.limit;
                        const bool in = want && blk >= 0 && blk < d.num_blocks;
                        if (want && !in) raise_err(d.err_flag, PKV_DEVERR_BLOCK_RANGE);
                        const unsigned got = __ballot_sync(0xffffffffu, in);
                        const int next = k + 1 < w.k1 ? lookup(k + 1) : -1;
                        const uint32_t bytes = __popc(got) * box * (D / 64);
                        const int slot0 = t & (d.block_size - 1);
#pragma unroll
                        for (int kv = 0; kv < 2; ++kv, ++pos) {
                            const uint32_t stage = pos % ST;
                            if (pos >= ST) ok = warp_wait(bars.empty(stage), (pos / ST - 1) & 1, gone);
                            if (!ok) break;
                            // V rows that nothing loads, or that no row sees, are zeroed: a weight of zero
                            // must not meet what lies there
                            const bool fix = kv == 1 && (__popc(got) < nblk || w.limit < (k + 1) * kKeyTile);
                            const uint32_t bar = fix ? bars.tail() : bars.full(stage);
                            const uint32_t dst = sm32 + L::ring + stage * L::kTile;
                            if (lane == 0) {
                                if (kv == 0) {
                                    uint32_t there = 0;         // by groups of 8 rows
                                    for (int i = 0; i < 16; ++i) there |= ((got >> ((i * 8) >> shift)) & 1u) << i;
                                    cols[tile_n % L::kColSlots].mask[0] = there;
                                }
                                ptx::mbar_arrive_expect_tx(bar, bytes);
                            }
                            __syncwarp();
                            if (in) {
#pragma unroll
                                for (int c = 0; c < D / 64; ++c)
                                    ptx::tma_load_4d(dst + c * 16384 + lane * box, kv ? &tmv : &tmk, bar, c * 64, slot0,
                                                     w.h, blk);
                            }
                            if (fix) {
                                ok = warp_wait(bar, fixes & 1, gone);
                                ++fixes;
                                if (!ok) break;
                                for (int i = lane; i < kKeyTile * (D / 8); i += 32) {
                                    const int rr = i / (D / 8);
                                    if (k * kKeyTile + rr >= w.limit || !((got >> (rr >> shift)) & 1u))
                                        tc::st_shared16(dst + piece_at(rr, i % (D / 8)), make_uint4(0, 0, 0, 0));
                                }
                                ptx::fence_proxy_async_smem();
                                __syncwarp();
                                if (lane == 0) ptx::mbar_arrive(bars.full(stage));
                            }
                        }
                        blk = next;
                    }
                } while (ok && w.next(p));
            }
        } else if (!TMA && warp < 12) {
            // -------------------------------------------- K/V by loads, 32 rows of a tile per warp
            load_rows<QK, CK, D, GS>(p, f, st, work, sm32 + L::ring, cols, bars, gone, warp - 8, lane);
        }
    }
    __syncthreads();
    if (*gone) {
        // copies and products under way end by themselves
        const uint64_t t0 = ptx::globaltimer();
        while (ptx::globaltimer() - t0 < 1000000ull) {
        }
        if (threadIdx.x == 0) raise_err(d.err_flag, PKV_DEVERR_TIMEOUT);
        __syncthreads();
    }
    tc::fence_after();
    if (warp == kMmaWarp) tc::tmem_free(tmem, 512);
}

// Joins the row tile that CTA blockIdx.x begins and a later one ends: with
// M = max m_i, out = sum O_i 2^(m_i - M) / sum l_i 2^(m_i - M).  A thread per
// row, 16 columns per block row of the grid; the parts lie column major, so
// the reads of a warp are whole lines.
template <int QK, int CK, int D>
__global__ void __launch_bounds__(kRowTile) prefill_join_kernel(PrefillParams p, PrefillFast f)
{
    griddep_wait();
    griddep_launch_dependents();
    const int4 ds = f.desc[blockIdx.x];
    if (ds.w < 0) return;
    const DecodeParams &d = p.d;
    const Seq s = seq_load(p, ds.x, false);
    const int row = threadIdx.x, r = ds.z * kRowTile + row;
    const bool live = r < s.rows;
    const int lim = live ? row_limit(p, s, r) : 0;
    const int tok = r / d.group, head = ds.y * d.group + (r - tok * d.group);
    const int c0 = blockIdx.y * 16;
    const int first = blockIdx.x, last = ds.w;
    auto slot = [&](int i) -> int64_t { return 2 * i + (i == first ? 1 : 0); };
    const float ninf = -__int_as_float(0x7f800000);
    bool redo = false;
    if (live) {
        float m = ninf;
        for (int i = first; i <= last; ++i) m = fmaxf(m, f.part_ml[slot(i) * 2 * kRowTile + row]);
        float l = 0.0f, acc[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
        for (int i = first; i <= last; ++i) {
            const float *ml = f.part_ml + slot(i) * 2 * kRowTile + row;
            const float wgt = ml[0] == ninf ? 0.0f : exp2_approx(ml[0] - m);
            const float li = ml[kRowTile];
            // a part without keys (l = 0) has no O, whatever lies there
            if (li == 0.0f) continue;
            l = fmaf(li, wgt, l);
            const float4 *a = reinterpret_cast<const float4 *>(f.part_acc) + (slot(i) * (D / 4) + c0 / 4) * kRowTile + row;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 v = a[j * kRowTile];
                acc[4 * j] = fmaf(v.x, wgt, acc[4 * j]);
                acc[4 * j + 1] = fmaf(v.y, wgt, acc[4 * j + 1]);
                acc[4 * j + 2] = fmaf(v.z, wgt, acc[4 * j + 2]);
                acc[4 * j + 3] = fmaf(v.w, wgt, acc[4 * j + 3]);
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        float bad = 0.0f;
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            bad = fmaf(acc[j] * inv, 0.0f, fmaf(acc[j + 1] * inv, 0.0f, bad));
            pk[j / 2] = tc::pack16<QK>(acc[j] * inv, acc[j + 1] * inv);
        }
        redo = bad != 0.0f;
        char *o = d.out + int64_t(s.s0 + tok) * d.o_b + int64_t(head) * d.o_h + 2 * c0;
        if (d.out_vec_ok) {
            reinterpret_cast<uint4 *>(o)[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            reinterpret_cast<uint4 *>(o)[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                reinterpret_cast<uint16_t *>(o)[j] = uint16_t(pk[j >> 1] >> (16 * (j & 1)));
        }
    }
    unsigned todo = __ballot_sync(0xffffffffu, redo);
    while (todo) {
        const int who = __ffs(todo) - 1;
        todo &= todo - 1;
        redo_row<QK, CK, D>(d, d.block_tables + ds.x * d.bt_b, int64_t(s.s0) + __shfl_sync(0xffffffffu, tok, who),
                            __shfl_sync(0xffffffffu, head, who), __shfl_sync(0xffffffffu, lim, who),
                            tile_limit(p, s, ds.z), c0, c0 + 16);
    }
}

}  // namespace
}  // namespace pkv
