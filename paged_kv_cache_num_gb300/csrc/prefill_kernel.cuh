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
// the group, and the causal border is as sharp as the rows allow.  Two
// subtiles of 128 rows (the whole tokens that fit) make a row tile; a unit of
// work is one row tile times one tile of 128 keys that some of its rows see.
// All units lie in one flat order (sequence, kv head, row tile, key tile),
// each row tile's preceded by kTileCost more for what it costs to begin and
// end one, and CTA i takes [i N / S, (i + 1) N / S): equal work for any mix
// of lengths, decided on the device (no host read of lengths; graph safe).
// A CTA that has the whole key range of a row tile writes its rows; otherwise
// it writes an fp32 partial (m, l, O), and prefill_join_kernel combines them.
//
// CTA.  Two softmax warpgroups (one per subtile, a thread per row), a warp per
// subtile that issues its products (tcgen05.mma, accumulators and P in tensor
// memory), a warpgroup that writes finished accumulators out while the next
// row tile is under way, a warp that loads Q, and the K/V producers.  While
// one subtile's softmax runs the tensor core works on the other's products: a
// subtile's scores wait for its last P V (they share tensor memory), which
// waits for its softmax, so that chain bounds the tile rate (about 3400 clocks
// per pair of subtiles, whose products alone take 2048; 12001-token prompt, 32
// q over 8 kv heads: 0.86 to 0.91 ms, 1290 to 1370 TFLOP/s, 0.68 to 0.72 of the
// measured cuBLAS rate).  A row tile of at most 128 rows has one subtile: then
// the warpgroups take its key tiles in turn, with states of their own that are
// joined at the end; few rows over long contexts run at HBM's rate that way.
//
// K/V.  16-bit caches in the flash layout: one warp issues TMA copies of
// whole block pieces into the operand ring; x-vectorised 16-bit caches: four
// warps copy 16-byte pieces.  One-byte and 3-bit caches: one warp issues TMA
// copies of the raw codes, four (3-bit: eight) warps convert them into the
// operand ring.  (3-bit rows at head_dim 64 are 24 bytes, which no tensor map
// takes: that warp loads them.)
// Codes become f16 exactly (every code of every kind is an f16 number); their
// scales are applied in fp32: per-head scales to c and to the result, per-row
// scales to the columns of S and of P, whose product is what P's operand holds:
// there the reference m is of the largest c S + log2(V scale) that the row sees
// (see kScaleSpread).  bf16 queries of such caches are
// brought to f16 by a power of two per row, exactly but for elements below
// 2^-31 of the row's largest, which are rounded to multiples of 2^-38 of it.
#pragma once

#include <type_traits>

#include "prefill_launch.h"
#include "prefill_row.cuh"
#include "tc_ptx.cuh"

namespace pkv {

using Start = PrefillStart;

struct PrefillFast {
    int4 *desc;                 // [grid] (sequence, kv head, row tile, last CTA) of the row tile split at a CTA's end
    int *redo;                  // [grid] whether the CTA has written rows that are not finite
    Start *starts;              // [grid] ... and then its share
    int later;                  // the join kernel looks through them (else the CTA itself, at its end: there is no
                                // join kernel where the table holds one key tile to a sequence)
    float *part_ml;             // [2 grid][2][256]
    float *part_acc;            // [2 grid][D / 4][256][4]
    int out32;                  // output rows at multiples of 32 bytes
    int q_tma;                  // Q by TMA
    int flip_q;                 // a negative scale's sign is still to be given to Q
    int raw_tma;                // raw codes by TMA (else by loads of the producer warp)
    int raw_unit;               // ... 3-bit rows in pieces of 8 bytes, 4 or 1
};

namespace {

enum Feed : int { kFeedTma, kFeedCopy, kFeedCodes };
// warps that convert codes: 3-bit ones take the most work and have room
template <int CK> constexpr int conv_warps() { return CK == kU3 ? 8 : 4; }

template <int CK, int FEED> constexpr int prefill_threads()
{
    return FEED == kFeedTma ? 512 : FEED == kFeedCodes ? 512 + 32 * conv_warps<CK>() : 640;
}

constexpr int kRowTile = 256;   // rows of a row tile, those between a subtile's whole tokens and 128 included
// Beginning and ending a row tile costs as much as this many units.  (16 prompts
// of 60 to 1500 tokens, times relative to that with 2: 0.99, 1, 1.04, 1.07 with 1, 2, 3,
// 4; few tokens over long contexts: 1.04, 1, 0.99, 0.97.)
constexpr int kTileCost = 2;
constexpr int kKeyTile = 128;
// P is handed to its product after this many keys and after all.  The early
// hand-over gets the issuing warp past its waits for V and for the
// accumulators while the other weights are made; the fewer keys go with it, the
// less the two subtiles' products are cut up in the tensor core's queue (a
// 12001-token prompt, times relative to that with 16: 1.03 with 32, 1.11 with 64, 1.14
// with 96, 1.09 without; a third hand-over in between 1.10 to 1.14).
constexpr int kFirst = 16;
// In long segments the two subtiles' softmax take turns: run at the same time
// they share the exponential unit and then leave it idle together while both
// wait for products (12001-token prompt: without 0.99 to 1.14 of the time with,
// depending on how the two happen to fall; e4m3 chunks 1.06).  In short segments
// the order costs more than it brings (packed prompts 1.13 of the time without),
// and so it does with scales per row, whose softmax is long enough by itself
// (3-bit chunks 1.2).
constexpr int kTurnTiles = 16;
// Scales per row: weights times V scales become the second product's operand, so
// they are held relative to their own largest value, L = max of weight times
// scale over the keys that the row sees; what is far below it loses bits in f16's
// subnormals (2^-25 of the reference at most), as any sum of 16-bit terms does.  Where
// the V scales of a key tile lie within 2^kScaleSpread of each other, and every row
// of the warp sees all of it, the tile's maxima of score and scale bound L from above by at
// most 2^(kScaleSpread + 1); else each row takes its maximum column by column
// over the keys that it sees, with the scales' exponents, in a pass of its own
// (e4m3 chunks over 8K to 16K, scales per token: 0.92 ms, and 1.30 with scales drawn
// over 2^9, where every tile takes that pass).
// Exponents are clamped to +-kScaleExp: the sum of weights l, relative to the same
// reference, then stays below 2^(80 + 8 + 31).  It can be as small as 2^-80, so where
// the reference moves l is scaled in two steps: a factor of 2^-130 is nothing to
// O, but may leave l the larger part.
constexpr int kScaleSpread = 4;
constexpr int kScaleExp = 80;
constexpr int kBins = 1024;
// A wait gives up after the first time and the second for each key tile of the
// table's rows: some waits last a whole segment (2^24 key tiles at the longest,
// about 1 us each; 5 us in the slowest form).
constexpr uint64_t kPrefillTimeoutNs = 4000000000ull, kPrefillTimeoutTileNs = 50000ull;

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
    s.nt = (s.rows + 2 * p.sub_rows - 1) / (2 * p.sub_rows);
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
    return row_limit(p, s, min((tile + 1) * 2 * p.sub_rows, s.rows) - 1);
}
// units of a row tile: at least one, so that rows that see nothing are written
__device__ __forceinline__ int tile_units(int limit) { return max(1, (limit + kKeyTile - 1) / kKeyTile); }

// A CTA's walk over its segments: maximal runs of key tiles of one row tile.
// `at` counts a row tile's cost units, its kTileCost first.
struct Walk {
    int64_t left;               // cost units from this segment on
    Seq s;
    int b, h, tile, at, k0, k1, units, limit;
    __device__ __forceinline__ bool shape(const PrefillParams &p)
    {
        limit = tile_limit(p, s, tile);
        units = tile_units(limit);
        const int end = int(min(int64_t(units + kTileCost), at + left));
        k0 = max(0, at - kTileCost);
        k1 = max(0, end - kTileCost);
        return k1 > k0;
    }
    __device__ __forceinline__ bool next(const PrefillParams &p)
    {
        left -= k1 + kTileCost - at;
        if (left <= kTileCost) return false;            // ends before the next row tile's first unit
        at = 0;
        if (++tile == s.nt) {
            tile = 0;
            if (++h == p.d.num_kv_heads) {
                h = 0;
                do s = seq_load(p, ++b, false); while (s.n == 0);
            }
        }
        return shape(p);
    }
    // which warpgroups take key tile k: one of them, or (2) both
    __device__ __forceinline__ int set(const PrefillParams &p, int k) const { return subtiles(p) == 2 ? 2 : (k - k0) & 1; }
    // tokens of the sequence that the key tiles reach
    __device__ __forceinline__ int reach() const { return min(s.ctx, units * kKeyTile); }
    __device__ __forceinline__ int subtiles(const PrefillParams &p) const
    {
        return s.rows - tile * 2 * p.sub_rows > p.sub_rows ? 2 : 1;
    }
};

__device__ __forceinline__ Walk walk_from(const PrefillParams &p, const Start &st)
{
    Walk w;
    w.left = st.u1 - st.u0;
    w.b = st.b;
    w.h = st.h;
    w.tile = st.tile;
    w.at = st.at;
    w.s = seq_load(p, st.b, false);
    w.shape(p);
    return w;
}

// cost units of sequence s and one kv head, summed over `lanes` (a power of two)
// threads of a warp; every thread of the warp calls it
__device__ __forceinline__ int64_t seq_units(const PrefillParams &p, const Seq &s, int lane, int lanes)
{
    int64_t u = 0;
    for (int i = lane; i < s.nt; i += lanes) u += tile_units(tile_limit(p, s, i)) + kTileCost;
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
        // a share is more than kTileCost: every CTA with work has a unit
        st.ctas = int(min(int64_t(gridDim.x), total / (kTileCost + 1)));
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
            for (int i = lane * c; i < min((lane + 1) * c, s.nt); ++i) mine += tile_units(tile_limit(p, s, i)) + kTileCost;
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
                const int t = tile_units(tile_limit(p, s, st.tile)) + kTileCost;
                if (u < t) break;
                u -= t;
            }
            st.at = int(u);
        }
        if (lane == 0) *out = st;
    }
    ptx::fence_proxy_async_smem();          // the bins' place is written by asynchronous copies next
    __syncthreads();
}

// ---------------------------------------------------------------- shared memory
template <int CK> constexpr bool is_coded() { return CK != kF16 && CK != kBF16; }
template <int CK, int D> constexpr int raw_row() { return CK == kU3 ? 3 * D / 8 : D; }

template <int CK, int D>
struct Smem {
    static constexpr bool kCoded = is_coded<CK>();
    static constexpr int kTile = 128 * D * 2;                   // bytes of 128 operand rows
    // stages of operands and of raw codes: what fits.  One-byte codes have three
    // operand stages, the others four
    static constexpr int kStages = (kCoded && CK != kU3 ? 3 : 4) * (D == 128 ? 1 : 2);
    static constexpr int kRaw = kCoded ? 3 * (D == 128 ? 1 : 2) : 0;
    static constexpr int kRawTile = kCoded ? 128 * raw_row<CK, D>() : 0;
    static constexpr int kColSlots = (kCoded ? 4 : 8) * (D == 128 ? 1 : 2);      // see ColSlot
    static constexpr int q = 0;
    static constexpr int ring = 2 * kTile;
    static constexpr int raw = ring + kStages * kTile;
    static constexpr int cols = raw + kRaw * kRawTile;
    static constexpr int kColBytes = 3 * kKeyTile * 4 + 64;
    static constexpr int state = cols + kColSlots * kColBytes;  // (m, l) of a row tile's rows: [subtile][2][128]
    static constexpr int q_scale = state + 2048;                // per row of subtile 0, of even and of odd segments
    static constexpr int bars = q_scale + 1024;
    static constexpr int n_bars = 4 * kStages + 2 * kRaw + 2 + 4 * 2 + 1 + 4 + 1 + 2;
    static constexpr int info = bars + 8 * n_bars;              // per raw stage: which blocks are there
    static constexpr int misc = (info + 4 * 8 + 15) / 16 * 16;
    static constexpr int total = misc + 128;
    static constexpr int alloc = total + 1024;                  // the base is rounded up to 1024
    static_assert(kStages * kTile >= (kBins + 1) * 8, "bins lie in the ring");
    static_assert(kRaw <= 8, "info");
    static_assert(alloc <= 232448, "shared memory of a CTA");
    static_assert(kColSlots >= kStages / 2 + 2, "see ColSlot");
    static_assert(sizeof(Start) <= 96, "misc");
};

// Column data of a key tile: scales of its 128 K and V rows and the V scales'
// exponents, their range by producer warp, and which groups of 8 rows are there.
// Tile T's is written once the ring has room for K of tile T.
//   K and V in rings of their own, R = stages / 2 tiles each: the scores of tile
//   T - R are done, and (row tiles of one subtile) those of T - R - 1 by the other
//   warpgroup; whoever issued them had finished the softmax of its tile before.
//   So the softmax of T - R - 1 is the earliest that may be under way.
//   One ring in the order K, V, K, V ...: V of tile T - 1 has had room (with three
//   stages K of tile T itself), in the place of V of tile T - R - 1, so that tile's
//   product with it is done, and its softmax before that.
// In either case the column data of at most R + 2 tiles, T's included, is in use.
struct ColSlot {
    float k[kKeyTile];
    float v[kKeyTile];
    float v_log2[kKeyTile];     // of the V scale, at most 1 above it, clamped
    uint32_t vexp[8];           // by producer warp, unused ones 0: biased exponent of its rows' largest V scale, and
                                // in the low half 255 minus the smallest one's
    uint32_t mask[8];           // likewise: the bits of its groups of 8 rows
};

struct Bars {
    uint32_t base;
    int stages, raws;
    // A stage that is filled: for subtile 0 or 1 alone, or (set 2) for both, so
    // that whoever waits on one of these barriers waits for each of its phases
    __device__ __forceinline__ uint32_t full(int set, int s) const { return base + 8 * (set * stages + s); }
    __device__ __forceinline__ uint32_t empty(int s) const { return base + 8 * (3 * stages + s); }
    __device__ __forceinline__ uint32_t q_full() const { return base + 8 * (4 * stages); }
    __device__ __forceinline__ uint32_t q_empty() const { return base + 8 * (4 * stages + 1); }
    __device__ __forceinline__ uint32_t s_full(int i) const { return base + 8 * (4 * stages + 2 + i); }
    __device__ __forceinline__ uint32_t p_full(int i) const { return base + 8 * (4 * stages + 4 + i); }
    __device__ __forceinline__ uint32_t o_full(int i) const { return base + 8 * (4 * stages + 6 + i); }
    __device__ __forceinline__ uint32_t p_first(int i) const { return base + 8 * (4 * stages + 8 + i); }
    __device__ __forceinline__ uint32_t tail() const { return base + 8 * (4 * stages + 10); }
    // a subtile's rows are finished (their m and l are there), and have been read
    __device__ __forceinline__ uint32_t e_full(int i) const { return base + 8 * (4 * stages + 11 + i); }
    __device__ __forceinline__ uint32_t e_empty(int i) const { return base + 8 * (4 * stages + 13 + i); }
    // bf16 Q that is to become f16
    __device__ __forceinline__ uint32_t q_raw() const { return base + 8 * (4 * stages + 15); }
    // subtile i is through a tile's softmax (long segments of two subtiles)
    __device__ __forceinline__ uint32_t turn(int i) const { return base + 8 * (4 * stages + 16 + i); }
    __device__ __forceinline__ uint32_t raw_full(int s) const { return base + 8 * (4 * stages + 18 + s); }
    __device__ __forceinline__ uint32_t raw_empty(int s) const { return base + 8 * (4 * stages + 18 + raws + s); }
};

// Wait for a phase, giving up when it takes too long (the limit lies behind
// `gone`) or another warp gave up.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *gone)
{
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::globaltimer();
    uint32_t n = 0;
    while (!ptx::mbar_try_wait(bar, parity)) {
        if ((++n & 15u) == 0 && (*gone || ptx::globaltimer() - t0 > *reinterpret_cast<volatile uint64_t *>(gone + 4))) {
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

// whether a phase is complete
__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, ptx::mbar_test(bar, parity));
}

// Where tile T's K and V lie in the operand ring: TMA fills a ring of each
// with a warp of its own, the others fill one in the order K, V, K, V ...
template <int FEED, int ST>
struct Ring {
    static __device__ __forceinline__ uint32_t stage(uint32_t t, int kv)
    {
        return FEED == kFeedTma ? t % (ST / 2) + kv * (ST / 2) : (2 * t + kv) % ST;
    }
    static __device__ __forceinline__ uint32_t turn(uint32_t t, int kv)
    {
        return FEED == kFeedTma ? t / (ST / 2) : (2 * t + kv) / ST;
    }
};

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
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// four one-byte codes -> four f16 numbers, exactly
template <int CK>
__device__ __forceinline__ uint2 q8x4_to_f16(uint32_t w)
{
    uint32_t lo, hi;
    if constexpr (CK == kI8) {                                  // 1024 + (c + 128), minus 1152
        const uint32_t u = w ^ 0x80808080u;
        lo = sub_f16x2(ptx::prmt(u, 0x64646464u, 0x4140), 0x64806480u);
        hi = sub_f16x2(ptx::prmt(u, 0x64646464u, 0x4342), 0x64806480u);
    } else if constexpr (CK == kE4M3) {
        asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
            : "=r"(lo), "=r"(hi) : "r"(w));
    } else {                                                    // e5m2 is the upper byte of an f16 number
        lo = ptx::prmt(w, 0u, 0x1404);
        hi = ptx::prmt(w, 0u, 0x3424);
    }
    return make_uint2(lo, hi);
}

// eight 3-bit codes (the low 24 bits of w) minus their zero point z, as f16
// numbers.  Of 12 bits x with codes a b c d, x + (x << 13) has a at bit 0, b
// at 16, c at 6 and d at 22: under 0x6400 they are 1024 + a and 1024 + 64 c;
// z0 = -1024 - z, z6 = -16 - z (twice each).
__device__ __forceinline__ uint4 u3x8_to_f16(uint32_t w, uint32_t z0, uint32_t z6)
{
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t y = ((w >> (12 * j)) & 0xfffu) * 0x2001u;
        const uint32_t lo = (y & 0x00070007u) | 0x64006400u, hi = (y & 0x01c001c0u) | 0x64006400u;
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(o[2 * j]) : "r"(lo), "r"(z0));
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[2 * j + 1]) : "r"(hi), "r"(0x24002400u), "r"(z6));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// bf16 pair -> f16 pair times s, a power of two
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float s)
{
    return tc::pack16<kF16>(__uint_as_float(w << 16) * s, __uint_as_float(w & 0xffff0000u) * s);
}

// ---------------------------------------------------------------- K/V producers
// Where a producer stands: the key tiles of the CTA's segments in order.
struct TileWalk {
    Walk w;
    int k;
    __device__ __forceinline__ bool next(const PrefillParams &p)
    {
        if (++k < w.k1) return true;
        if (!w.next(p)) return false;
        k = w.k0;
        return true;
    }
};

// Q of a segment's row tile, once the products of the segment before have
// read theirs: boxes of (64 elements, heads of the group, tokens) -- rows
// behind the sequence's last are other rows of q, and nothing comes of them
// -- or 16-byte copies; then `full` completes a phase.
template <int D>
__device__ __forceinline__ bool load_q(const PrefillParams &p, const PrefillFast &f, const Walk &w, uint32_t item,
                                       uint32_t q, const Bars &bars, uint32_t full, const CUtensorMap *tmq,
                                       volatile int *gone, int lane)
{
    const DecodeParams &d = p.d;
    constexpr int kTile = 128 * D * 2;
    constexpr int PPR = D / 8;                                  // pieces per row
    constexpr int RPI = 32 / PPR;                               // rows per instruction
    if (item > 0 && !warp_wait(bars.q_empty(), (item - 1) & 1, gone)) return false;
    const int ns = w.subtiles(p);
    if (f.q_tma) {
        if (lane == 0) {
            const int toks = p.sub_rows / d.group;
            ptx::mbar_arrive_expect_tx(full, uint32_t(ns * p.sub_rows * D * 2));
            for (int sub = 0; sub < ns; ++sub)
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    ptx::tma_load_3d(q + sub * kTile + c * 16384, tmq, full, c * 64, w.h * d.group,
                                     w.s.s0 + (2 * w.tile + sub) * toks);
        }
        __syncwarp();
        return true;
    }
    for (int sub = 0; sub < ns; ++sub) {
        const int c = lane % PPR;
        int r = (2 * w.tile + sub) * p.sub_rows + lane / PPR;
        int tok = r / d.group, g = r - tok * d.group;
#pragma unroll 4
        for (int i = lane / PPR; i < 128; i += RPI, r += RPI) {
            const bool in = i < p.sub_rows && r < w.s.rows;
            const char *src = d.q + int64_t(w.s.s0 + tok) * d.q_b + int64_t(w.h * d.group + g) * d.q_h + 16 * c;
            tc::cp_async16(q + sub * kTile + piece_at(i, c), in ? src : d.q, in);
            g += RPI;
            while (g >= d.group) {
                g -= d.group;
                ++tok;
            }
        }
    }
    tc::cp_async_wait_all();
    // a negative scale's sign, on the pieces that this lane copied
    for (int i = d.scale_log2 < 0.0f && !f.flip_q ? lane : ns * 128 * PPR; i < ns * 128 * PPR; i += 32) {
        const uint32_t at = q + i / (128 * PPR) * kTile + piece_at((i / PPR) & 127, i % PPR);
        uint4 v = tc::ld_shared16(at);
        v.x ^= 0x80008000u;
        v.y ^= 0x80008000u;
        v.z ^= 0x80008000u;
        v.w ^= 0x80008000u;
        tc::st_shared16(at, v);
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(full);
    return true;
}

// The row tile that a CTA begins and does not end, and the CTA that ends it;
// w: its walk after the last segment.
__device__ __forceinline__ int4 split_end(const Walk &w, const Start &st, bool done)
{
    if (!done || w.k0 != 0 || w.k1 >= w.units) return make_int4(0, 0, 0, -1);
    const int64_t end = st.u1 - w.left - w.k1 + w.units;       // next() has taken the segment's cost off `left`
    return make_int4(w.b, w.h, w.tile, int((end * st.ctas + st.total - 1) / st.total) - 1);
}

// 16-bit rows by 16-byte copies, rows 32 lw .. 32 lw + 31 of every tile by
// one warp: a lane copies its row's pieces (neighbouring slots are neighbours
// in the x-vectorised layout).  A stage is handed over once the second behind it
// is under way, or as soon as there is no room to go on.
template <int CK, int D>
__device__ __forceinline__ void copy_rows(const PrefillParams &p, const Start &st, uint32_t ring, ColSlot *cols,
                                          const Bars &bars, volatile int *gone, int lw, int lane)
{
    using L = Smem<CK, D>;
    constexpr int ST = L::kStages;
    const DecodeParams &d = p.d;
    const int row = 32 * lw + lane;
    TileWalk tw{walk_from(p, st), 0};
    tw.k = tw.w.k0;
    uint32_t pos = 0, tile_n = 0;
    uint32_t p0 = 0, p1 = 0, p2 = 0;                            // barriers of the stages in hand, the oldest first
    auto hand_over = [&]() {                                    // the oldest, once it is there
        if (p2 != 0) tc::cp_async_wait<2>(); else if (p1 != 0) tc::cp_async_wait<1>(); else tc::cp_async_wait<0>();
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p0);
        p0 = p1;
        p1 = p2;
        p2 = 0;
    };
    auto lookup = [&]() -> int {                                // this row's block of the tile, -1 where it wants none
        const int t = tw.k * kKeyTile + row;
        return t < tw.w.reach() ? d.block_tables[tw.w.b * d.bt_b + int64_t(t >> d.block_shift) * d.bt_j] : -1;
    };
    int next_blk = lookup();
    bool more = true;
    while (more) {
        const int t = tw.k * kKeyTile + row, h = tw.w.h;
        const bool want = t < tw.w.reach();
        const int64_t blk = next_blk;
        const bool in = want && blk >= 0 && blk < d.num_blocks;
        if (want && !in) raise_err(d.err_flag, PKV_DEVERR_BLOCK_RANGE);
        const int64_t at = in ? blk * d.c_blk + int64_t(t & (d.block_size - 1)) * d.c_slot + h * d.c_head : 0;
        const unsigned got = __ballot_sync(0xffffffffu, in);
        const int set = tw.w.set(p, tw.k);
        more = tw.next(p);
        if (more) next_blk = lookup();                          // a tile ahead
        for (int kv = 0; kv < 2; ++kv, ++pos) {
            // never wait for room with a stage in hand
            while (pos >= ST && p0 != 0 && !warp_test(bars.empty(pos % ST), (pos / ST - 1) & 1)) hand_over();
            if (pos >= ST && !warp_wait(bars.empty(pos % ST), (pos / ST - 1) & 1, gone)) {
                tc::cp_async_wait<0>();
                return;
            }
            if (kv == 0 && lane == 0) {
                uint32_t there = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) there |= ((got >> (8 * i)) & 0xffu ? 1u : 0u) << (4 * lw + i);
                cols[tile_n % L::kColSlots].mask[lw] = there;
            }
            const char *src = (kv ? d.v_cache : d.k_cache) + at;
            const uint32_t dst = ring + (pos % ST) * L::kTile;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) tc::cp_async16(dst + piece_at(row, c), src + (in ? c * d.c_chunk : 0), in);
            tc::cp_async_commit();
            const uint32_t bar = bars.full(set, pos % ST);
            (p0 == 0 ? p0 : p1 == 0 ? p1 : p2) = bar;
            if (p2 != 0) hand_over();
        }
        ++tile_n;
    }
    while (p0 != 0) hand_over();
}

// Raw codes of every tile into the raw ring, by one warp: one TMA copy per
// block, [rows][row bytes], or [16-byte piece][rows][16] of an x-vectorised
// cache; or by copies of 16 bytes or less where no tensor map can be made.
template <int CK, int D, bool TMA>
__device__ __forceinline__ void raw_codes(const PrefillParams &p, const PrefillFast &f, const Start &st, unsigned char *sm,
                                          uint32_t sm32, const Bars &bars, const CUtensorMap *tmk, const CUtensorMap *tmv,
                                          volatile int *gone, int lane)
{
    using L = Smem<CK, D>;
    constexpr int RB = raw_row<CK, D>();
    const DecodeParams &d = p.d;
    const int shift = min(d.block_shift, 7), rows = 1 << shift, nblk = kKeyTile >> shift;
    uint32_t *info = reinterpret_cast<uint32_t *>(sm + L::info);
    TileWalk tw{walk_from(p, st), 0};
    tw.k = tw.w.k0;
    if (TMA && lane == 0) {
        ptx::prefetch_tmap(tmk);
        ptx::prefetch_tmap(tmv);
    }
    // this lane's block of the tile, -1 where it wants none
    auto lookup = [&]() -> int {
        const int t = tw.k * kKeyTile + lane * rows;
        return lane < nblk && t < tw.w.reach()
                   ? d.block_tables[tw.w.b * d.bt_b + int64_t(t >> d.block_shift) * d.bt_j] : -1;
    };
    uint32_t pos = 0, pending = 0;                              // barrier of a stage that loads are still filling
    auto flush = [&]() {
        tc::cp_async_wait<0>();
        __syncwarp();
        if (lane == 0 && pending != 0) ptx::mbar_arrive(pending);
        pending = 0;
    };
    int blk = lookup();
    bool more = true;
    while (more) {
        const int t = tw.k * kKeyTile + lane * rows, h = tw.w.h;
        const bool want = lane < nblk && t < tw.w.reach();
        const bool in = want && blk >= 0 && blk < d.num_blocks;
        if (want && !in) raise_err(d.err_flag, PKV_DEVERR_BLOCK_RANGE);
        const unsigned got = __ballot_sync(0xffffffffu, in);
        const int now = blk, slot0 = t & (d.block_size - 1);
        more = tw.next(p);
        if (more) blk = lookup();
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++pos) {
            const uint32_t s = pos % L::kRaw;
            if (pos >= L::kRaw) {                               // never wait for room with a stage in hand
                if (!TMA && pending != 0 && !warp_test(bars.raw_empty(s), (pos / L::kRaw - 1) & 1)) flush();
                if (!warp_wait(bars.raw_empty(s), (pos / L::kRaw - 1) & 1, gone)) {
                    tc::cp_async_wait<0>();
                    return;
                }
            }
            if (lane == 0) info[s] = got;
            const uint32_t dst = sm32 + L::raw + s * L::kRawTile;
            if constexpr (TMA) {
                if (lane == 0) ptx::mbar_arrive_expect_tx(bars.raw_full(s), uint32_t(__popc(got) * rows * RB));
                __syncwarp();
                if (in) {
                    const CUtensorMap *m = kv ? tmv : tmk;
                    if (d.c_chunk == 16 || CK == kU3)
                        ptx::tma_load_4d(dst + lane * rows * RB, m, bars.raw_full(s), 0, slot0, h, now);
                    else
                        ptx::tma_load_5d(dst + lane * rows * RB, m, bars.raw_full(s), 0, slot0, 0, h, now);
                }
            } else {
                // a lane takes rows; one stage is filled while the one before
                // arrives.  Short loops: this code shares the instruction cache
                // with the softmax (unrolled: e4m3 chunks that never come here
                // 615 -> 702 us).
                const char *cache = kv ? d.v_cache : d.k_cache;
                const bool xv = d.c_chunk != 16 && CK != kU3;
#pragma unroll 1
                for (int i = lane; i < kKeyTile; i += 32) {
                    const int in_blk = i & (rows - 1);
                    const int b = __shfl_sync(0xffffffffu, now, i >> shift);
                    const int o = __shfl_sync(0xffffffffu, slot0, i >> shift) + in_blk;
                    if ((got >> (i >> shift)) & 1u) {
                        const char *src = cache + b * d.c_blk + o * d.c_slot + h * d.c_head;
                        const uint32_t at = dst + (i >> shift) * rows * RB + in_blk * (xv ? 16 : RB);
                        if constexpr (CK != kU3) {
#pragma unroll 1
                            for (int j = 0; j < RB / 16; ++j)
                                tc::cp_async16(at + j * (xv ? rows * 16 : 16), src + j * d.c_chunk, true);
                        } else if (f.raw_unit == 8) {
#pragma unroll 1
                            for (int j = 0; j < RB; j += 8) tc::cp_async_small<8>(at + j, src + j);
                        } else if (f.raw_unit == 4) {
#pragma unroll 1
                            for (int j = 0; j < RB; j += 4) tc::cp_async_small<4>(at + j, src + j);
                        } else {
                            unsigned char *to = sm + (at - sm32);
#pragma unroll 1
                            for (int j = 0; j < RB; ++j)
                                to[j] = __ldg(reinterpret_cast<const unsigned char *>(src) + j);
                        }
                    }
                    __syncwarp();
                }
                tc::cp_async_commit();
                if (pending != 0) {
                    tc::cp_async_wait<1>();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(pending);
                }
                pending = bars.raw_full(s);
            }
        }
    }
    if constexpr (!TMA) flush();
}

// Raw codes -> operand ring, 128 / conv_warps rows of every tile by one warp
// (lane = row for the scales).
template <int CK, int D, bool GS>
__device__ __forceinline__ void convert_rows(const PrefillParams &p, const Start &st, unsigned char *sm, uint32_t sm32,
                                             const Bars &bars, volatile int *gone, int lw, int lane)
{
    using L = Smem<CK, D>;
    constexpr int ST = L::kStages, RB = raw_row<CK, D>();
    constexpr int kPieces = CK == kU3 ? D / 32 : D / 16;        // per row and per lane: 16 one-byte codes, or 32
                                                                // 3-bit ones (12 bytes)
    const DecodeParams &d = p.d;
    const uint32_t *info = reinterpret_cast<const uint32_t *>(sm + L::info);
    ColSlot *cols = reinterpret_cast<ColSlot *>(sm + L::cols);
    constexpr int NR = kKeyTile / conv_warps<CK>();             // rows of this warp: 32 or 16
    const int row0 = NR * lw, row = row0 + lane % NR;
    const int shift = min(d.block_shift, 7), rows = 1 << shift;
    const bool xv = d.c_chunk != 16 && CK != kU3;
    TileWalk tw{walk_from(p, st), 0};
    tw.k = tw.w.k0;
    uint32_t pos = 0, tile_n = 0;
    // scales of this lane's row: a tile ahead, its table entry two ahead
    int64_t entry = -1;
    uint32_t ks = 0, vs = 0, kz = 0, vz = 0;                    // as stored: nothing waits for them before their use
    TileWalk ahead = tw;
    bool ahead_more = GS;
    auto fetch = [&]() {
        const int t = ahead.k * kKeyTile + row;
        entry = t < ahead.w.reach()
                    ? d.block_tables[ahead.w.b * d.bt_b + int64_t(t >> d.block_shift) * d.bt_j] : -1;
    };
    auto scales = [&](const TileWalk &x) {
        ks = vs = kz = vz = 0;
        if (entry < 0 || entry >= d.num_blocks) return;
        const int64_t slot = (x.k * kKeyTile + row) & (d.block_size - 1);
        if constexpr (CK == kU3) {
            const int64_t m = entry * d.m_blk + slot * d.m_slot + x.w.h * d.m_head;
            const int64_t z = entry * d.z_blk + slot * d.z_slot + x.w.h * d.z_head;
            ks = __ldg(d.k_qs + m);
            vs = __ldg(d.v_qs + m);
            kz = __ldg(d.k_qz + z);
            vz = __ldg(d.v_qz + z);
        } else {
            const int64_t m = entry * d.gs_blk + slot * d.gs_slot + x.w.h * d.gs_head;
            ks = __float_as_uint(__ldg(d.k_gs + m));
            vs = __float_as_uint(__ldg(d.v_gs + m));
        }
    };
    if constexpr (GS) {
        fetch();
        scales(tw);
        ahead_more = ahead.next(p);
        if (ahead_more) fetch();
    }
    bool more = true;
    while (more) {
        const int limit = tw.w.reach() - tw.k * kKeyTile;       // rows of the tile that are wanted
        const int set = tw.w.set(p, tw.k);
        const uint32_t kz_now = kz, vz_now = vz;
        unsigned ok = 0;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++pos) {
            const uint32_t rs = pos % L::kRaw, s = pos % ST;
            if (!warp_wait(bars.raw_full(rs), (pos / L::kRaw) & 1, gone)) return;
            if (pos >= ST && !warp_wait(bars.empty(s), (pos / ST - 1) & 1, gone)) return;
            if (kv == 0) {
                const unsigned got = info[rs];
                ok = __ballot_sync(0xffffffffu, row < limit && ((got >> (row >> shift)) & 1u));     // twice 16 rows, or 32
                ColSlot &cs = cols[tile_n % L::kColSlots];
                if constexpr (GS) {
                    auto value = [](uint32_t x) {
                        return CK == kU3 ? __half2float(__ushort_as_half(uint16_t(x))) : __uint_as_float(x);
                    };
                    cs.k[row] = value(ks);
                    cs.v[row] = value(vs);
                    const uint32_t e = (__float_as_uint(value(vs)) >> 23) & 0xffu;
                    cs.v_log2[row] = scale_exp<kScaleExp>(e);
                    const uint32_t hi = __reduce_max_sync(0xffffffffu, e), lo = __reduce_min_sync(0xffffffffu, e);
                    if (lane == 0) cs.vexp[lw] = (hi << 16) | (255u - lo);
                }
                if (lane == 0) {
                    uint32_t there = 0;
#pragma unroll
                    for (int i = 0; i < NR / 8; ++i) there |= ((ok >> (8 * i)) & 0xffu ? 1u : 0u) << (NR / 8 * lw + i);
                    cs.mask[lw] = there;
                }
                if constexpr (GS) {                             // the next tile's scales, the one after's entry
                    if (ahead_more) {
                        scales(ahead);
                        ahead_more = ahead.next(p);
                        if (ahead_more) fetch();
                    }
                }
            }
            const unsigned char *from = sm + L::raw + rs * L::kRawTile;
            const uint32_t dst = sm32 + L::ring + s * L::kTile;
            const bool all = ok == 0xffffffffu;
            // lane -> (row, piece) so that the 8 lanes of a load or store phase hit
            // different banks; four pieces' loads before their conversion
            if constexpr (CK == kU3) {
                const int r = lane >> 1, rr = row0 + r, h = lane & 1;
                const float z = float(__shfl_sync(0xffffffffu, kv ? vz_now : kz_now, r));
                const bool there = (ok >> r) & 1u;
                const uint32_t z0 = tc::pack16<kF16>(-1024.0f - z, -1024.0f - z);
                const uint32_t z6 = tc::pack16<kF16>(-16.0f - z, -16.0f - z);
                uint32_t w[kPieces / 2][3];
                const uint32_t *src = reinterpret_cast<const uint32_t *>(from + rr * RB + 12 * h);
#pragma unroll
                for (int i = 0; i < kPieces / 2; ++i)
#pragma unroll
                    for (int j = 0; j < 3; ++j) w[i][j] = there ? src[6 * i + j] : 0u;
#pragma unroll
                for (int i = 0; i < kPieces / 2; ++i) {
                    const uint32_t fl[4] = {w[i][0], __funnelshift_r(w[i][0], w[i][1], 24),
                                            __funnelshift_r(w[i][1], w[i][2], 16), w[i][2] >> 8};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        tc::st_shared16(dst + i * 16384 + piece_at(rr, 4 * h + j), u3x8_to_f16(fl[j], z0, z6));
                }
            } else if (xv) {
                const int rr = row;
                const unsigned char *src = from + (rr >> shift) * rows * RB + (rr & (rows - 1)) * 16;
                const bool there = (ok >> lane) & 1u;
#pragma unroll 2
                for (int c = 0; c < kPieces; ++c) {
                    uint4 v = *reinterpret_cast<const uint4 *>(src + c * rows * 16);
                    if (!there) v = make_uint4(0, 0, 0, 0);
                    const uint2 a = q8x4_to_f16<CK>(v.x), e = q8x4_to_f16<CK>(v.y);
                    const uint2 g = q8x4_to_f16<CK>(v.z), k = q8x4_to_f16<CK>(v.w);
                    tc::st_shared16(dst + piece_at(rr, 2 * c), make_uint4(a.x, a.y, e.x, e.y));
                    tc::st_shared16(dst + piece_at(rr, 2 * c + 1), make_uint4(g.x, g.y, k.x, k.y));
                }
            } else {
                // 8 rows and four of a row's pieces at a time; at head_dim 128 odd rows take
                // the other four
                const int r = lane >> 2, rr = row0 + r;
#pragma unroll
                for (int b = 0; b < kPieces / 4; ++b) {
                    const int c = (lane & 3) | (kPieces == 8 ? ((b ^ r) & 1) << 2 : 0);
                    const unsigned char *src = from + rr * RB + 16 * c;
                    const uint32_t at0 = dst + piece_at(rr, 2 * c), at1 = dst + piece_at(rr, 2 * c + 1);
                    uint4 v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = *reinterpret_cast<const uint4 *>(src + i * 8 * RB);
                        if (!all && !((ok >> (r + 8 * i)) & 1u)) v[i] = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint2 a = q8x4_to_f16<CK>(v[i].x), e = q8x4_to_f16<CK>(v[i].y);
                        const uint2 g = q8x4_to_f16<CK>(v[i].z), k = q8x4_to_f16<CK>(v[i].w);
                        tc::st_shared16(at0 + i * 1024, make_uint4(a.x, a.y, e.x, e.y));
                        tc::st_shared16(at1 + i * 1024, make_uint4(g.x, g.y, k.x, k.y));
                    }
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(bars.full(set, s));
                ptx::mbar_arrive(bars.raw_empty(rs));
            }
        }
        ++tile_n;
        more = tw.next(p);
    }
}

// ---------------------------------------------------------------- rows that are not finite
// The whole row tiles of a CTA's share, warp `me` of `warps` in turn, `n` rows
// (modulo `warps`) having been dealt before; returns that for the next share.  Out of
// line: called where the output warps had written the row, it cost them
// registers (packed prompts 165 -> 171 us).
template <int QK, int CK, int D, int U>
__device__ __noinline__ int redo_share(const PrefillParams &p, const Start &st, int n, int me, int warps)
{
    const DecodeParams &d = p.d;
    Walk w = walk_from(p, st);
    do {
        if (w.k0 != 0 || w.k1 != w.units) continue;             // joined from several CTAs: see redo_rows
        const int r0 = w.tile * 2 * p.sub_rows, rows = min(2 * p.sub_rows, w.s.rows - r0);
        for (int i = (me - n + warps) % warps; i < rows; i += warps) {
            const int r = r0 + i, tok = r / d.group;
            redo_row<QK, CK, D, U>(d, d.block_tables + w.b * d.bt_b, int64_t(w.s.s0) + tok,
                                   w.h * d.group + (r - tok * d.group), row_limit(p, w.s, r), w.reach());
        }
        n = (n + rows) % warps;
    } while (w.next(p));
    return n;
}

// ---------------------------------------------------------------- the kernel
// Warps 0-7 softmax; 16-bit caches by TMA: 8 and 9 products, 10 K and Q, 11 V,
// 12-15 output; the others: 8-11 producers, 12 and 13 products, 14 raw codes,
// 15 Q, 16-19 output, and for 3-bit codes 20-23 producers.
template <int QK, int CK, int D, int FEED, bool GS>
__global__ void __launch_bounds__(prefill_threads<CK, FEED>(), 1)
    prefill_kernel(PrefillParams p, PrefillFast f, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv, const __grid_constant__ CUtensorMap tmq)
{
    using L = Smem<CK, D>;
    constexpr int ST = L::kStages;
    constexpr bool TMA = FEED == kFeedTma;
    constexpr int OK = is_coded<CK>() ? int(kF16) : QK;         // operands of the products
    constexpr bool kRawQ = OK != QK;                            // bf16 Q becomes f16
    constexpr int kMmaWarp = TMA ? 8 : 12;                     // two of them
    constexpr int kQWarp = TMA ? 11 : 15;                       // by TMA that of V too
    constexpr int kOutWarp = TMA ? 12 : 16;                     // four of them
    constexpr int kProducers = FEED == kFeedCodes ? conv_warps<CK>() : 4;
    constexpr int CH = 16;                                      // columns that a softmax thread reads at a time
    using R = Ring<FEED, ST>;
    const DecodeParams &d = p.d;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sm32 = ptx::smem_u32(sm);
    Start *start = reinterpret_cast<Start *>(sm + L::misc);
    volatile int *gone = reinterpret_cast<volatile int *>(sm + L::misc + 96);
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(sm + L::misc + 104);
    volatile int *not_finite = reinterpret_cast<volatile int *>(sm + L::misc + 108);
    ColSlot *cols = reinterpret_cast<ColSlot *>(sm + L::cols);
    static_assert(sizeof(ColSlot) == L::kColBytes, "column slots");
    const Bars bars{sm32 + L::bars, ST, L::kRaw};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            for (int set = 0; set < 3; ++set) ptx::mbar_init(bars.full(set, i), TMA ? 1 : kProducers);
            ptx::mbar_init(bars.empty(i), 2);
        }
        for (int i = 0; i < L::kRaw; ++i) {
            ptx::mbar_init(bars.raw_full(i), 1);
            ptx::mbar_init(bars.raw_empty(i), kProducers);
        }
        ptx::mbar_init(bars.q_full(), kRawQ ? 8 : 1);
        ptx::mbar_init(bars.q_raw(), 1);
        ptx::mbar_init(bars.q_empty(), 2);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bars.s_full(i), 1);
            ptx::mbar_init(bars.p_full(i), 4);
            ptx::mbar_init(bars.p_first(i), 4);
            ptx::mbar_init(bars.turn(i), 4);
            ptx::mbar_init(bars.e_full(i), 4);
            ptx::mbar_init(bars.e_empty(i), 4);
            ptx::mbar_init(bars.o_full(i), 1);
        }
        ptx::mbar_init(bars.tail(), 1);
        ptx::fence_mbar_init();
        *gone = 0;
        *reinterpret_cast<volatile uint64_t *>(gone + 4) =
            kPrefillTimeoutNs + kPrefillTimeoutTileNs * uint64_t((int64_t(d.max_blocks) << d.block_shift) / kKeyTile);
        *not_finite = 0;
    }
    if (threadIdx.x < 16 * L::kColSlots) (cols[threadIdx.x / 16].vexp)[threadIdx.x % 16] = 0u;
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
        float *state = reinterpret_cast<float *>(sm + L::state) + sub * 256 + row;
        float *q_scale = reinterpret_cast<float *>(sm + L::q_scale) + row;
        uint32_t turns = 0;                                     // tiles taken in turn
        uint32_t tile_n = 0, mine_n = 0, item = 0, outs = 0;    // key tiles of the CTA, of this warpgroup; segments, and
                                                                // those that use this warpgroup's accumulators
        if (work) {
            Walk w = walk_from(p, st);
            do {
                const int nk = w.k1 - w.k0;
                const bool split = w.subtiles(p) == 1;          // both warpgroups on one subtile
                const bool two = !split || nk > 1;              // both accumulators are in use
                const int r = w.tile * 2 * p.sub_rows + (split ? 0 : sub * p.sub_rows) + row;
                const bool live = row < p.sub_rows && r < w.s.rows;
                const bool idle = !__any_sync(0xffffffffu, live);
                const int lim = live ? row_limit(p, w.s, r) : 1 << 30;      // rows that are not there need no mask
                float c = fabsf(d.scale_log2);
                if constexpr (is_q8(CK) && !GS) c *= fabsf(d.k_scale[w.h]);
                bool ok = true;
                if constexpr (kRawQ) {
                    // this row of Q to f16, in place: its largest element to [2^14, 2^15)
                    float back = 1.0f;
                    ok = warp_wait(bars.q_raw(), item & 1, gone);
                    if (!ok) break;
                    // two places in turn: nothing orders this segment's write after warpgroup 1's read
                    // of the one before, but q_full of the one between does (every warp arrives there
                    // after its read)
                    float *scale_at = q_scale + 128 * (item & 1);
                    if (!split || sub == 0) {
                        const uint32_t q = sm32 + L::q + sub * L::kTile;
                        uint32_t top = 0;
#pragma unroll 4
                        for (int i = 0; i < D / 8; ++i) {
                            const uint4 v = tc::ld_shared16(q + piece_at(row, i));
                            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) top = max(top, max((x[j] << 16) & 0x7fff0000u, x[j] & 0x7fff0000u));
                        }
                        // exponents that keep both powers of two normal; the sign of the scale goes along
                        const int e = min(max(int(top >> 23), 16), 254);
                        const float s = __uint_as_float(uint32_t(268 - e) << 23);
                        back = __uint_as_float(uint32_t(254 - (__float_as_uint(s) >> 23)) << 23);
                        const float sg = f.flip_q ? -s : s;
#pragma unroll 4
                        for (int i = 0; i < D / 8; ++i) {
                            uint4 v = tc::ld_shared16(q + piece_at(row, i));
                            v.x = bf16x2_to_f16x2(v.x, sg);
                            v.y = bf16x2_to_f16x2(v.y, sg);
                            v.z = bf16x2_to_f16x2(v.z, sg);
                            v.w = bf16x2_to_f16x2(v.w, sg);
                            tc::st_shared16(q + piece_at(row, i), v);
                        }
                        if (split) *scale_at = back;
                        ptx::fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bars.q_full());
                    if (split && sub == 1) {
                        ok = warp_wait(bars.q_full(), item & 1, gone);
                        if (!ok) break;
                        back = *scale_at;
                    }
                    c *= back;
                }
                ++item;
                // keeps 0 * -inf out, so that masked weights stay zero: the smallest number, which makes
                // nothing of any score
                c = fmaxf(c, __uint_as_float(1u));
                const float ninf = -__int_as_float(0x7f800000);
                float m = ninf, l = 0.0f;                       // m: of S, or (GS) of c S + log2(V scale)
                const int step = split ? 2 : 1, j0 = split ? sub : 0;
                const bool in_turn = !GS && !split && nk >= kTurnTiles;
                for (int j = j0; j < nk; j += step, ++mine_n) {
                    ok = warp_wait(bars.s_full(sub), mine_n & 1, gone);
                    if (!ok) break;
                    tc::fence_after();
                    // the accumulators are overwritten from here on: their last contents are out
                    if (j == j0 && outs > 0) {
                        ok = warp_wait(bars.e_empty(sub), (outs - 1) & 1, gone);
                        if (!ok) break;
                        tc::fence_after();
                    }
                    if (in_turn) {
                        if (sub == 1 || turns > 0) ok = warp_wait(bars.turn(1 - sub), (turns + sub - 1) & 1, gone);
                        ++turns;
                        if (!ok) break;
                    }
                    if (idle) {                                 // no row of the warp is there
                        tc::fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            ptx::mbar_arrive(bars.p_first(sub));
                            ptx::mbar_arrive(bars.p_full(sub));
                            if (in_turn) ptx::mbar_arrive(bars.turn(sub));
                        }
                        continue;
                    }
                    const ColSlot &cs = cols[(tile_n + j) % L::kColSlots];
                    // keys behind the row's limit, and blocks that are not there
                    uint32_t there = cs.mask[0];
                    if constexpr (!TMA) there |= cs.mask[1] | cs.mask[2] | cs.mask[3];
                    if constexpr (kProducers == 8) there |= cs.mask[4] | cs.mask[5] | cs.mask[6] | cs.mask[7];
                    const int rel = lim - (w.k0 + j) * kKeyTile;
                    const int seen = there == 0xffffu ? __reduce_min_sync(0xffffffffu, max(rel, 0)) : 0;    // by all rows
                    if (!GS && seen < kKeyTile) {
                        // few tiles: masked in place, in a rolled loop, before the others' path
#pragma unroll 1
                        for (int o = seen & ~15; o < kKeyTile; o += 16) {
                            uint32_t x[16];
                            tc::tmem_ld16_wait(ts + o, x);
                            const uint32_t g = there >> (o >> 3);
                            const int n = rel - o;
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (i >= n || !((g >> (i >> 3)) & 1u)) x[i] = 0xff800000u;
                            tc::tmem_st16(ts + o, x);
                        }
                        tc::tmem_st_wait();
                    }
                    // the tile's columns in chunks, read twice, for the maximum and for the
                    // weights: that costs less than the registers would
                    constexpr int NC = kKeyTile / CH;
                    uint32_t x[2][CH];
                    // per-row K scales: the scores are scaled on the way to the maximum and put
                    // back.  They are masked after that: the scales of hidden keys are then no matter,
                    // and one that is NaN stays so where it is seen
                    auto scaled = [&](uint32_t (&v)[CH], int o) {
#pragma unroll
                        for (int i = 0; i < CH; i += 4) {
                            const float4 k4 = *reinterpret_cast<const float4 *>(cs.k + o + i);
                            const float2 u = tc::mul2(f2(v, i), make_float2(k4.x, k4.y));
                            const float2 y = tc::mul2(f2(v, i + 2), make_float2(k4.z, k4.w));
                            v[i] = __float_as_uint(u.x);
                            v[i + 1] = __float_as_uint(u.y);
                            v[i + 2] = __float_as_uint(y.x);
                            v[i + 3] = __float_as_uint(y.y);
                        }
                        tc::tmem_st(ts + o, v);
                    };
                    float mx[4] = {ninf, ninf, ninf, ninf};
                    tc::tmem_ld(ts, x[0]);
#pragma unroll
                    for (int q = 0; q < NC; ++q) {
                        tc::tmem_ld_wait(x[q & 1]);
                        // after the last chunk the first again
                        if (!GS || q < NC - 1) tc::tmem_ld(ts + CH * ((q + 1) % NC), x[(q + 1) & 1]);
                        if constexpr (GS) scaled(x[q & 1], CH * q);
#pragma unroll
                        for (int u = 0; u < CH; u += 8)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mx[i] = fmaxf(fmaxf(mx[i], __uint_as_float(x[q & 1][u + i])), __uint_as_float(x[q & 1][u + 4 + i]));
                    }
                    float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if constexpr (GS) {
                        tc::tmem_st_wait();
                        uint32_t ve = __vmaxu2(__vmaxu2(cs.vexp[0], cs.vexp[1]), __vmaxu2(cs.vexp[2], cs.vexp[3]));
                        if constexpr (kProducers == 8)
                            ve = __vmaxu2(ve, __vmaxu2(__vmaxu2(cs.vexp[4], cs.vexp[5]), __vmaxu2(cs.vexp[6], cs.vexp[7])));
                        if (seen < kKeyTile || (ve >> 16) + (ve & 0xffffu) > 255u + kScaleSpread) {
                            // the scaled scores are masked here, and the maximum taken column by
                            // column: what a row does not see has no part in it
                            top = ninf;
#pragma unroll 1
                            for (int o = 0; o < kKeyTile; o += 16) {
                                uint32_t y[16];
                                tc::tmem_ld16_wait(ts + o, y);
                                const uint32_t g = there >> (o >> 3);
                                const int n = rel - o;
#pragma unroll
                                for (int i = 0; i < 16; i += 4) {
                                    const float4 e4 = *reinterpret_cast<const float4 *>(cs.v_log2 + o + i);
                                    const float e[4] = {e4.x, e4.y, e4.z, e4.w};
#pragma unroll
                                    for (int u = 0; u < 4; ++u) {
                                        if (i + u >= n || !((g >> (i >> 3)) & 1u)) y[i + u] = 0xff800000u;
                                        top = fmaxf(top, fmaf(__uint_as_float(y[i + u]), c, e[u]));
                                    }
                                }
                                tc::tmem_st16(ts + o, y);
                            }
                            tc::tmem_st_wait();
                        } else {
                            top = fmaf(top, c, scale_exp<kScaleExp>(ve >> 16));
                        }
                        tc::tmem_ld(ts, x[0]);
                    }
                    float grow = 1.0f;                          // what O and l shrink by
                    const float unit = GS ? 1.0f : c;
                    if (top > m && (m == ninf || (top - m) * unit > 8.0f)) {
                        if constexpr (GS) {                     // l in two steps: see kScaleSpread
                            const float h = m == ninf ? 0.0f : exp2_approx(0.5f * (m - top));
                            grow = h * h;
                            l = l * h * h;
                        } else {
                            grow = m == ninf ? 0.0f : exp2_approx((m - top) * c);
                            l *= grow;
                        }
                        m = top;
                    }
                    if (j > j0 && __any_sync(0xffffffffu, grow != 1.0f)) {
                        // seldom: a rolled loop keeps its registers out of the way
#pragma unroll 1
                        for (int o = 0; o < D; o += 16) {
                            uint32_t y[16];
                            tc::tmem_ld16_wait(to + o, y);
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * grow);
                            tc::tmem_st16(to + o, y);
                        }
                    }
                    const float off = m == ninf ? 0.0f : m * unit;
                    const float2 c2 = make_float2(c, c), off2 = make_float2(-off, -off);
                    float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
                    for (int q = 0; q < NC; ++q) {
                        uint32_t (&v)[CH] = x[q & 1];
                        tc::tmem_ld_wait(v);
                        if (q < NC - 1) tc::tmem_ld(ts + CH * (q + 1), x[(q + 1) & 1]);
                        uint32_t pk[CH / 2];
#pragma unroll
                        for (int i = 0; i < CH; i += 4) {
                            const float2 y0 = tc::fma2(f2(v, i), c2, off2), y1 = tc::fma2(f2(v, i + 2), c2, off2);
                            float2 e0 = make_float2(exp2_approx(y0.x), exp2_approx(y0.y));
                            float2 e1 = make_float2(exp2_approx(y1.x), exp2_approx(y1.y));
                            sum[0] = tc::add2(sum[0], e0);
                            sum[1] = tc::add2(sum[1], e1);
                            if constexpr (GS) {
                                const float4 v4 = *reinterpret_cast<const float4 *>(cs.v + CH * q + i);
                                e0 = tc::mul2(e0, make_float2(v4.x, v4.y));
                                e1 = tc::mul2(e1, make_float2(v4.z, v4.w));
                            }
                            pk[i >> 1] = tc::pack16<OK>(e0.x, e0.y);
                            pk[(i >> 1) + 1] = tc::pack16<OK>(e1.x, e1.y);
                        }
                        if (in_turn && q == NC - 2 && lane == 0) ptx::mbar_arrive(bars.turn(sub));
                        // over columns that have been read for the last time
                        tc::tmem_st(ts + CH / 2 * q, pk);
                        if (CH * (q + 1) == kFirst || q == NC - 1) {    // the first keys, then all
                            tc::tmem_st_wait();
                            tc::fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(q < NC - 1 ? bars.p_first(sub) : bars.p_full(sub));
                        }
                    }
                    sum[0] = tc::add2(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                }
                tile_n += nk;
                if (!ok) break;
                if (sub == 1 && !two) continue;
                state[0] = GS || m == ninf ? m : m * c;
                state[128] = l;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bars.e_full(sub));
                ++outs;
            } while (w.next(p));
        }
    } else if (warp >= kOutWarp && warp < kOutWarp + 4) {
        // ------------------------------------------------ finished rows, a thread per row
        const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
        const int row = (warp & 3) * 32 + lane;
        const float ninf = -__int_as_float(0x7f800000);
        const float *states = reinterpret_cast<const float *>(sm + L::state) + row;
        uint32_t outs[2] = {0, 0};                              // segments that use each accumulator
        if (work) {
            Walk w = walk_from(p, st);
            bool ok = true;
            do {
                const bool split = w.subtiles(p) == 1, join = split && w.k1 - w.k0 > 1;
                const bool whole = w.k0 == 0 && w.k1 == w.units;
                for (int sub = 0; sub < (split ? 1 : 2); ++sub) {
                    const int r = w.tile * 2 * p.sub_rows + sub * p.sub_rows + row;
                    const bool live = row < p.sub_rows && r < w.s.rows;
                    const bool idle = !__any_sync(0xffffffffu, live);
                    const uint32_t to = tmem + lanes + 256 + sub * 128;
                    for (int i = sub; i < (join ? 2 : sub + 1); ++i) {
                        ok = ok && warp_wait(bars.e_full(i), outs[i] & 1, gone) && warp_wait(bars.o_full(i), outs[i] & 1, gone);
                        ++outs[i];
                    }
                    if (!ok) break;
                    tc::fence_after();
                    float off = states[sub * 256], l = states[sub * 256 + 128];
                    // weights of this O and of warpgroup 1's.  An O without keys (l = 0) holds anything
                    // and has no part; every other one has, so that what is not finite stays: a weight
                    // that underflows makes infinities NaN, and scores that are all NaN (a maximum of
                    // -inf, l NaN) make the row NaN
                    float w0 = 1.0f, w1 = 0.0f;
                    const bool use0 = l != 0.0f;
                    bool use1 = false;
                    if (join) {
                        const float m1 = states[256], l1 = states[384];
                        use1 = l1 != 0.0f;
                        const float top = fmaxf(off, m1);
                        w0 = !use0 ? 0.0f : off == ninf ? l : exp2_approx(off - top);
                        w1 = !use1 ? 0.0f : m1 == ninf ? l1 : exp2_approx(m1 - top);
                        if constexpr (GS) {                     // in two steps, as everywhere
                            const float h0 = !use0 || off == ninf ? w0 : exp2_approx(0.5f * (off - top));
                            const float h1 = !use1 || m1 == ninf ? w1 : exp2_approx(0.5f * (m1 - top));
                            l = fmaf(l * h0, h0, l1 * h1 * h1);
                        } else {
                            l = fmaf(l, w0, l1 * w1);
                        }
                        off = top;
                    }
                    float fac = 1.0f;
                    if constexpr (is_q8(CK) && !GS) {
                        fac = d.v_scale[w.h];
                        // a K scale that is NaN is seen by every row with a key; kept out of c, where
                        // it would meet masked scores
                        if (isnan(d.k_scale[w.h])) fac = d.k_scale[w.h];
                    }
                    if (whole) fac = l == 0.0f ? 0.0f : fac / l;
                    w0 *= fac;
                    w1 *= fac;
                    const int tok = r / d.group;
                    const int head = w.h * d.group + (r - tok * d.group);
                    char *o_row = d.out + int64_t(w.s.s0 + tok) * d.o_b + int64_t(head) * d.o_h;
                    const int slot = 2 * blockIdx.x + (w.k0 == 0 ? 1 : 0);
                    const int prow = sub * 128 + row;
                    float4 *acc = reinterpret_cast<float4 *>(f.part_acc) + int64_t(slot) * (D / 4) * kRowTile + prow;
                    if (!whole) {
                        float *ml = f.part_ml + int64_t(slot) * 2 * kRowTile + prow;
                        ml[0] = off;
                        ml[kRowTile] = l;
                    }
                    float bad = 0.0f;
                    // 16 columns at o, in `a`, while the next are on their way
                    auto columns = [&](int o, uint32_t (&a)[16]) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) a[i] = use0 ? __float_as_uint(__uint_as_float(a[i]) * w0) : 0u;
                        if (join) {
                            uint32_t b[16];
                            tc::tmem_ld16_wait(to + 128 + o, b);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (use1)
                                    a[i] = __float_as_uint(fmaf(__uint_as_float(b[i]), w1, __uint_as_float(a[i])));
                        }
                        if (!whole) {
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                acc[(o + i) / 4 * kRowTile] = make_float4(__uint_as_float(a[i]), __uint_as_float(a[i + 1]),
                                                                          __uint_as_float(a[i + 2]), __uint_as_float(a[i + 3]));
                            return;
                        }
                        uint32_t pk[8];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            bad = fmaf(__uint_as_float(a[i]), 0.0f, fmaf(__uint_as_float(a[i + 1]), 0.0f, bad));
                            pk[i / 2] = tc::pack16<QK>(__uint_as_float(a[i]), __uint_as_float(a[i + 1]));
                        }
                        if (!live) return;
                        if (f.out32) {
                            tc::st_global32(o_row + 2 * o, pk);
                        } else if (d.out_vec_ok) {
#pragma unroll
                            for (int i = 0; i < 8; i += 4)
                                *reinterpret_cast<uint4 *>(o_row + 2 * (o + 2 * i)) = make_uint4(pk[i], pk[i + 1], pk[i + 2], pk[i + 3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                reinterpret_cast<uint16_t *>(o_row)[o + 2 * i] = uint16_t(pk[i]);
                                reinterpret_cast<uint16_t *>(o_row)[o + 2 * i + 1] = uint16_t(pk[i] >> 16);
                            }
                        }
                    };
                    if (!idle) {
                        uint32_t a[16], b[16];
                        tc::tmem_ld16(to, a);
#pragma unroll 1
                        for (int o = 0; o < D; o += 32) {
                            tc::tmem_ld_wait16(a);
                            tc::tmem_ld16(to + o + 16, b);
                            columns(o, a);
                            tc::tmem_ld_wait16(b);
                            if (o + 32 < D) tc::tmem_ld16(to + o + 32, a);
                            columns(o + 16, b);
                        }
                    }
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(bars.e_empty(sub));
                        if (join) ptx::mbar_arrive(bars.e_empty(1));
                    }
                    // not finite: weights of zero may have met values that are not.  Such rows are done
                    // again later (see redo_row)
                    if (__any_sync(0xffffffffu, whole && live && bad != 0.0f) && lane == 0) *not_finite = 1;
                }
            } while (ok && w.next(p));
        }
    } else {
        if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // -------------------------------------------- the products
            if (work) {
                constexpr uint32_t id_qk = tc::instr_desc<OK == kBF16, false, 128, 128>();
                constexpr uint32_t id_pv = tc::instr_desc<OK == kBF16, true, 128, D>();
                const bool leader = tc::elect_one();
                // V tiles: [64-element chunk][128 rows]; by TMA [block][chunk][rows of a block]
                const int rows = min(d.block_size, 128);
                const uint32_t v_lbo = TMA ? rows * 128 : 16384, v_sbo = TMA && rows == 8 ? 128 * D / 8 : 1024;
                const uint32_t q_lo = tc::desc_lo(sm32 + L::q, 16), k_lo = tc::desc_lo(sm32 + L::ring, 16);
                const uint32_t v_lo = tc::desc_lo(sm32 + L::ring, v_lbo), v_hi = tc::desc_hi(v_sbo);
                uint32_t v_at[8];                               // 16 keys each, in units of 16 bytes
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v_at[i] = TMA ? ((16 * i / rows) * (rows * D * 2) + ((16 * i) & (rows - 1)) * 128) >> 4 : 16 * i * 128 >> 4;
                const int i = warp - kMmaWarp;                  // the subtile
                const uint32_t ti = tmem + i * 128;
                // S = Q K^T of a ring stage
                auto qk = [&](int q, uint32_t stage) {
                    const uint32_t a = q_lo + q * (L::kTile >> 4), b = k_lo + stage * (L::kTile >> 4);
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t o = (ks >> 2) * (16384 >> 4) + (ks & 3) * (32 >> 4);
                            tc::mma_ss(ti, a + o, b + o, id_qk, ks > 0);
                        }
                        tc::commit(bars.s_full(i));
                    }
                };
                // O (+)= P V, the first keys and then the others
                auto pv = [&](int from, int to, uint32_t stage, bool acc) {
                    const uint32_t b = v_lo + stage * (L::kTile >> 4);
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            if (ks >= from && ks < to)
                                tc::mma_ts(ti + 256, ti + 8 * ks, b + v_at[ks], v_hi, id_pv, ks > 0 || acc);
                    }
                };
                auto release = [&](uint32_t bar) {
                    if (leader) tc::commit(bar);
                };
                // a stage is free when both subtiles have used it; on a row tile of one
                // subtile each key tile has one user, who counts twice
                auto done = [&](uint32_t stage, bool twice) {
                    release(bars.empty(stage));
                    if (twice) release(bars.empty(stage));
                };
                uint32_t phases[2] = {0, 0};                    // by stage: this subtile's own set, the common one
                auto there = [&](uint32_t t, int kv, bool split) -> bool {
                    const uint32_t s = R::stage(t, kv);
                    const bool ok = warp_wait(bars.full(split ? i : 2, s), (phases[split ? 0 : 1] >> s) & 1, gone);
                    phases[0] ^= uint32_t(split) << s;
                    phases[1] ^= uint32_t(!split) << s;
                    tc::fence_after();
                    return ok;
                };
                uint32_t tile_n = 0, item = 0, n_p = 0;
                Walk w = walk_from(p, st);
                bool ok = true;
                do {
                    const int nk = w.k1 - w.k0;
                    const bool split = w.subtiles(p) == 1;
                    const int step = split ? 2 : 1, j0 = split ? i : 0;
                    ok = warp_wait(bars.q_full(), item & 1, gone);
                    if (!ok) break;
                    tc::fence_after();
                    ok = j0 >= nk || there(tile_n + j0, 0, split);
                    // K of tile j is there
                    for (int j = j0; ok && j < nk; j += step, ++n_p) {
                        const bool last = j + step >= nk;
                        const uint32_t t = tile_n + j, ks = R::stage(t, 0), vs = R::stage(t, 1);
                        qk(split ? 0 : i, ks);
                        done(ks, split);
                        if (last) release(bars.q_empty());
                        ok = there(t, 1, split) && warp_wait(bars.p_first(i), n_p & 1, gone);
                        if (!ok) break;
                        tc::fence_after();
                        pv(0, kFirst / 16, vs, j > j0);
                        // the next tile's K, before the wait that the next scores depend on -- but in a
                        // ring of three, K two tiles on takes this V's place
                        const bool early = !split || FEED == kFeedTma || ST > 3;
                        if (!last && early) ok = there(t + step, 0, split);
                        ok = ok && warp_wait(bars.p_full(i), n_p & 1, gone);
                        if (!ok) break;
                        tc::fence_after();
                        pv(kFirst / 16, 8, vs, true);
                        done(vs, split);
                        if (last) release(bars.o_full(i));
                        if (!last && !early) ok = there(t + step, 0, split);
                    }
                    if (!ok) break;
                    if (j0 >= nk && lane == 0) ptx::mbar_arrive(bars.q_empty());    // had nothing to do
                    tile_n += nk;
                    ++item;
                } while (w.next(p));
            }
            __syncwarp();
        } else if (!TMA && warp == kQWarp) {
            // -------------------------------------------- Q
            Walk w;
            uint32_t item = 0;
            bool have = work;
            if (work) w = walk_from(p, st);
            while (have) {
                if (!load_q<D>(p, f, w, item++, sm32 + L::q, bars, kRawQ ? bars.q_raw() : bars.q_full(), &tmq, gone, lane)) break;
                have = w.next(p);
            }
            if (lane == 0) f.desc[blockIdx.x] = split_end(w, st, work && !have);
        } else if (TMA) {
            // -------------------------------------------- K (warp 10) and V (11) by TMA: whole blocks.  K boxes are
            // 64 elements wide, V's take the row's 64-element chunks together.  K's warp
            // loads Q too: both are needed at once
            const int kv = warp - 10;
            const CUtensorMap *map = kv ? &tmv : &tmk;
            const int shift = min(d.block_shift, 7);            // rows per box
            const int rows = 1 << shift, nblk = kKeyTile >> shift;
            uint32_t tile_n = 0, fixes = 0;
            if (lane == 0) ptx::prefetch_tmap(map);
            if (work) {
                TileWalk tw{walk_from(p, st), 0};
                tw.k = tw.w.k0;
                // this lane's block of the tile, -1 where it wants none
                auto lookup = [&]() -> int {
                    const int t = tw.k * kKeyTile + lane * rows;
                    return lane < nblk && t < tw.w.reach()
                               ? d.block_tables[tw.w.b * d.bt_b + int64_t(t >> d.block_shift) * d.bt_j] : -1;
                };
                int blk = lookup();
                bool ok = true, more = true;
                uint32_t item = 0;
                for (; more && ok; ++tile_n) {
                    if (kv == 0 && tw.k == tw.w.k0) {
                        ok = load_q<D>(p, f, tw.w, item++, sm32 + L::q, bars, bars.q_full(), &tmq, gone, lane);
                        if (!ok) break;
                    }
                    const int t = tw.k * kKeyTile + lane * rows, h = tw.w.h;
                    const int limit = tw.w.reach() - tw.k * kKeyTile;
                    const int set = tw.w.set(p, tw.k);
                    const bool want = lane < nblk && t < tw.w.reach();
                    const bool in = want && blk >= 0 && blk < d.num_blocks;
                    if (want && !in) raise_err(d.err_flag, PKV_DEVERR_BLOCK_RANGE);
                    const unsigned got = __ballot_sync(0xffffffffu, in);
                    const int now = blk, slot0 = t & (d.block_size - 1);
                    more = tw.next(p);
                    if (more) blk = lookup();
                    const uint32_t stage = R::stage(tile_n, kv), turn = R::turn(tile_n, kv);
                    if (turn > 0) ok = warp_wait(bars.empty(stage), (turn - 1) & 1, gone);
                    if (!ok) break;
                    // V rows that nothing loads, or behind the context, are zeroed: a weight of
                    // zero must not meet what lies there
                    const bool fix = kv == 1 && (__popc(got) < nblk || limit < kKeyTile);
                    const uint32_t bar = fix ? bars.tail() : bars.full(set, stage);
                    const uint32_t dst = sm32 + L::ring + stage * L::kTile;
                    if (lane == 0) {
                        if (kv == 0) {
                            uint32_t there = 0;                 // by groups of 8 rows
                            for (int i = 0; i < 16; ++i) there |= ((got >> ((i * 8) >> shift)) & 1u) << i;
                            cols[tile_n % L::kColSlots].mask[0] = there;
                        }
                        ptx::mbar_arrive_expect_tx(bar, uint32_t(__popc(got) * rows * D * 2));
                    }
                    __syncwarp();
                    if (in) {
                        if (kv) {
                            ptx::tma_load_5d(dst + lane * rows * D * 2, map, bar, 0, slot0, 0, h, now);
                        } else {
#pragma unroll
                            for (int c = 0; c < D / 64; ++c)
                                ptx::tma_load_4d(dst + c * 16384 + lane * rows * 128, map, bar, c * 64, slot0, h, now);
                        }
                    }
                    if (fix) {
                        ok = warp_wait(bar, fixes & 1, gone);
                        ++fixes;
                        if (!ok) break;
                        for (int i = lane; i < kKeyTile * (D / 8); i += 32) {
                            const int rr = i / (D / 8), c = i % (D / 8), in_blk = rr & (rows - 1);
                            if (rr >= limit || !((got >> (rr >> shift)) & 1u))
                                tc::st_shared16(dst + (rr >> shift) * rows * D * 2 + (c >> 3) * rows * 128 + in_blk * 128 +
                                                    (((c & 7) ^ (in_blk & 7)) << 4),
                                                make_uint4(0, 0, 0, 0));
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(bars.full(set, stage));
                    }
                }
                if (kv == 0 && lane == 0) f.desc[blockIdx.x] = split_end(tw.w, st, ok);
            } else if (kv == 0 && lane == 0) {
                f.desc[blockIdx.x] = make_int4(0, 0, 0, -1);
            }
        } else if (warp < 12 || warp >= 20) {
            if (work) {
                if constexpr (FEED == kFeedCodes)
                    convert_rows<CK, D, GS>(p, st, sm, sm32, bars, gone, warp < 12 ? warp - 8 : warp - 16, lane);
                else if constexpr (FEED == kFeedCopy)
                    copy_rows<CK, D>(p, st, sm32 + L::ring, cols, bars, gone, warp - 8, lane);
            }
        } else if (FEED == kFeedCodes && warp == 14) {
            if constexpr (FEED == kFeedCodes) {
                constexpr bool kCanMap = raw_row<CK, D>() % 16 == 0;
                if (work && kCanMap && f.raw_tma)
                    raw_codes<CK, D, kCanMap>(p, f, st, sm, sm32, bars, &tmk, &tmv, gone, lane);
                else if (work)
                    raw_codes<CK, D, false>(p, f, st, sm, sm32, bars, &tmk, &tmv, gone, lane);
            }
        }
    }
    __syncthreads();
    if (f.later) {
        if (threadIdx.x == 0) {
            f.redo[blockIdx.x] = *not_finite;
            if (*not_finite) f.starts[blockIdx.x] = *start;
        }
    } else if (*not_finite) {
        redo_share<QK, CK, D, 1>(p, *start, 0, warp, prefill_threads<CK, FEED>() / 32);
    }
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

constexpr int kJoinWarps = kRowTile / 32;

// row of the sequence at place i of a row tile's parts
__device__ __forceinline__ int tile_row(const PrefillParams &p, int tile, int i)
{
    return (2 * tile + (i >> 7)) * p.sub_rows + (i & 127);
}

// The join kernel's rows that are not finite (see redo_row).  todo: by warp of
// the block, those of the 32 rows that it has joined 16 columns of.  Kept out
// of the kernel's body, whose registers it would take.
template <int QK, int CK, int D>
__device__ __noinline__ void redo_rows(const PrefillParams &p, const PrefillFast &f, const unsigned *todo)
{
    const DecodeParams &d = p.d;
    const int warp = threadIdx.x >> 5;
    const int4 ds = f.desc[blockIdx.x];
    if (ds.w >= 0) {
        const Seq s = seq_load(p, ds.x, false);
        const int hi = min(s.ctx, tile_units(tile_limit(p, s, ds.z)) * kKeyTile);
        constexpr int kSlices = D / 16;
        int n = 0;
        for (int g = 0; g < kJoinWarps; g += kSlices) {         // warps of the same rows
            unsigned rows = 0;
            for (int i = 0; i < kSlices; ++i) rows |= todo[g + i];
            for (; rows; rows &= rows - 1) {
                if (n++ % kJoinWarps != warp) continue;
                const int at = (blockIdx.y * kJoinWarps + g) / kSlices * 32 + __ffs(rows) - 1;
                const int r = tile_row(p, ds.z, at), tok = r / d.group;
                redo_row<QK, CK, D, 4>(d, d.block_tables + ds.x * d.bt_b, int64_t(s.s0) + tok,
                                    ds.y * d.group + (r - tok * d.group), row_limit(p, s, r), hi);
            }
        }
    }
    const int warps = gridDim.x * gridDim.y * kJoinWarps, me = (blockIdx.y * gridDim.x + blockIdx.x) * kJoinWarps + warp;
    int n = 0;
    for (int c = 0; c < int(gridDim.x); ++c)
        if (f.redo[c]) n = redo_share<QK, CK, D, 4>(p, f.starts[c], n, me, warps);
}

// Joins the row tile that CTA blockIdx.x begins and a later one ends: with
// M = max m_i, out = sum O_i 2^(m_i - M) / sum l_i 2^(m_i - M).  A thread per
// row and 16 columns, all columns of a row by one block; the parts lie column
// major, so the reads of a warp are whole lines.
//
// Rows that are not finite (see redo_row) are done again here, with the whole
// grid: those of a joined tile by the warps of their block in turn, those of
// whole tiles, in CTAs that have marked themselves, by all warps of the grid in
// turn.  Nothing waits for them.
template <int QK, int CK, int D>
__global__ void __launch_bounds__(kRowTile, 2) prefill_join_kernel(const __grid_constant__ PrefillParams p,
                                                                const __grid_constant__ PrefillFast f)
{
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kSlices = D / 16;                 // of a row's columns
    __shared__ unsigned todo[kJoinWarps];
    const DecodeParams &d = p.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 ds = f.desc[blockIdx.x];
    int again = 0;
    for (int i = threadIdx.x; i < int(gridDim.x); i += kRowTile) again |= f.redo[i];
    unsigned mine = 0;
    if (ds.w >= 0) {
        const Seq s = seq_load(p, ds.x, false);
        const int part = blockIdx.y * kJoinWarps + warp, row = part / kSlices * 32 + lane, c0 = part % kSlices * 16;
        const int r = tile_row(p, ds.z, row);
        const bool live = (row & 127) < p.sub_rows && r < s.rows;
        const int first = blockIdx.x, last = ds.w;
        auto slot = [&](int i) -> int64_t { return 2 * i + (i == first ? 1 : 0); };
        const float ninf = -__int_as_float(0x7f800000);
        bool redo = false;
        if (live) {
            const int tok = r / d.group, head = ds.y * d.group + (r - tok * d.group);
            float m = ninf;
            for (int i = first; i <= last; ++i) m = fmaxf(m, f.part_ml[slot(i) * 2 * kRowTile + row]);
            float l = 0.0f, acc[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[j] = 0.0f;
            for (int i = first; i <= last; ++i) {
                const float *ml = f.part_ml + slot(i) * 2 * kRowTile + row;
                const float half = ml[0] == ninf ? 0.0f : exp2_approx(0.5f * (ml[0] - m)), wgt = half * half;
                const float li = ml[kRowTile];
                // a part without keys (l = 0) has no O, whatever lies there
                if (li == 0.0f) continue;
                l = fmaf(li * half, half, l);       // in two steps: see kScaleSpread
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
        mine = __ballot_sync(0xffffffffu, redo);
        if (lane == 0) todo[warp] = mine;
    }
    if (__syncthreads_or(again | int(mine != 0u))) redo_rows<QK, CK, D>(p, f, todo);
}

}  // namespace
}  // namespace pkv
