// tables.cu -- block tables, context lengths and slots of a step, from the
// requests' lengths, on the device; and the blocks of tokens that are dropped,
// back to the pool.
//
// Request b has cached_b tokens and gets new_b more: it needs
//   need_b = ceil((cached_b + new_b) / BS) - ceil(cached_b / BS)
// blocks, and with S_b = need_0 + .. + need_{b-1} its j-th one is the S_b + j -th
// from the top of the stack of free blocks.  Its rows of the step follow those of
// the requests before it; row i is position cached_b + i.
//
// One launch of one cluster: every CTA makes the prefix sums over the requests by
// itself (reads of a few bytes per request), then takes its share of the blocks and
// rows, finding their request by bisection in shared memory.  The cluster's
// barrier parts the reads of lengths and counts from the writes, which may be to
// the same memory.  Bound by latency, a launch and three trips to memory: 64 requests
// of 1 to 8 new tokens 5 us on the device, 601 prompts' 150000 rows 14 us with sixteen
// CTAs (eight: 20; a row at a time: 32).
#include <cooperative_groups.h>

#include <atomic>

#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kTableThreads = 1024;                 // at most
constexpr int kTableMaxDevices = 64;

// Inclusive sums of two numbers over the threads of the CTA.
__device__ __forceinline__ void cta_scan(int64_t &a, int64_t &b, int64_t (*sums)[2])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    if (lane == 31) {
        sums[warp][0] = a;
        sums[warp][1] = b;
    }
    __syncthreads();
    int64_t x = lane < (blockDim.x >> 5) ? sums[lane][0] : 0, y = lane < (blockDim.x >> 5) ? sums[lane][1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    const int64_t u = __shfl_sync(0xffffffffu, x, (warp + 31) & 31), v = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
    if (warp > 0) {
        a += u;
        b += v;
    }
    __syncthreads();
}

// largest b in [0, n) with start[b] <= i
__device__ __forceinline__ int find(const int *start, int n, int i)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

// TRIM: `second` holds the lengths to keep; else the numbers of new tokens
template <bool TRIM>
__global__ void __launch_bounds__(kTableThreads) tables_kernel(TableParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    extern __shared__ int sm[];
    __shared__ int64_t sums[kTableThreads / 32][2];
    __shared__ int totals[2];                       // rows and blocks of the requests that are served
    const int B = p.batch, tid = threadIdx.x;
    int *row0 = sm, *blk0 = sm + B, *len = sm + 2 * B;          // first row, first block, cached tokens (TRIM: kept blocks in row0)
    const int64_t cap = int64_t(p.max_blocks) << p.block_shift;
    const int64_t low = (int64_t(1) << p.block_shift) - 1;      // the slot within a block of a position
    int64_t count = p.free_count[0];
    bool bad_pool = count < 0 || count > p.pool;
    count = count < 0 ? 0 : count > p.pool ? p.pool : count;
    // what a stack can give, or take
    const int64_t room = TRIM ? p.pool - count : count;
    if (tid < 2) totals[tid] = 0;
    const int threads = blockDim.x;
    const int per = (B + threads - 1) / threads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    // rows and blocks of request b
    bool bad_len = false;
    auto request = [&](int b, int64_t &cached, int64_t &rows, int64_t &blocks) {
        cached = p.first[b * p.first_stride];
        int64_t n = p.second[b * p.second_stride];
        if (cached < 0 || cached > cap) {
            bad_len = true;
            cached = cached < 0 ? 0 : cap;
        }
        if (TRIM) {
            n = n < 0 ? 0 : n > cached ? cached : n;            // tokens kept
            rows = n;
            blocks = ((cached + low) >> p.block_shift) - ((n + low) >> p.block_shift);
        } else {
            if (n < 0 || cached + n > cap) {
                bad_len = true;
                n = 0;
            }
            rows = n;
            blocks = ((cached + n + low) >> p.block_shift) - ((cached + low) >> p.block_shift);
        }
    };
    int64_t ra = 0, bl = 0;
    for (int b = b0; b < b1; ++b) {
        int64_t cached, rows, blocks;
        request(b, cached, rows, blocks);
        ra += rows;
        bl += blocks;
    }
    int64_t r_end = ra, b_end = bl;
    cta_scan(r_end, b_end, sums);
    int64_t r = r_end - ra, k = b_end - bl;
    // Served is who fits together with all before him; the others, as the sums only
    // grow, are those from some request on, and count as without new rows.  Their
    // starts are corrected below: every start is at most the total.
    int most_rows = 0, most_blocks = 0;
    for (int b = b0; b < b1; ++b) {
        int64_t cached, rows, blocks;
        request(b, cached, rows, blocks);
        const bool fits = (TRIM || r + rows <= p.num_rows) && k + blocks <= room;
        if (fits) {
            if (!TRIM) most_rows = int(r + rows);
            most_blocks = int(k + blocks);
        } else if (rows > 0 || blocks > 0) {
            bad_pool = true;
        }
        row0[b] = TRIM ? int(fits ? rows : cached) : int(r < p.num_rows ? r : p.num_rows);
        blk0[b] = int(k < room ? k : room);
        len[b] = int(cached);
        r += rows;
        k += blocks;
    }
    most_rows = __reduce_max_sync(0xffffffffu, most_rows);
    most_blocks = __reduce_max_sync(0xffffffffu, most_blocks);
    if ((tid & 31) == 0 && (most_rows | most_blocks) != 0) {
        atomicMax(&totals[0], most_rows);
        atomicMax(&totals[1], most_blocks);
    }
    if (blockIdx.x == 0) {
        if (bad_len) raise_err(p.err_flag, PKV_DEVERR_CONTEXT_RANGE);
        if (bad_pool) raise_err(p.err_flag, PKV_DEVERR_POOL_RANGE);
    }
    __syncthreads();
    const int total_rows = totals[0], total_blocks = totals[1];
    for (int b = tid; b < B; b += threads) {
        if (!TRIM) row0[b] = min(row0[b], total_rows);
        blk0[b] = min(blk0[b], total_blocks);
    }
    // all CTAs have read the lengths and counts that are written below
    cooperative_groups::this_cluster().sync();

    const int at = blockIdx.x * threads + tid, step = gridDim.x * threads;
    for (int b = at; b < B; b += step) {
        if (TRIM) {
            p.lens_out[b * p.lens_stride] = row0[b];
        } else {
            const int end = b + 1 < B ? row0[b + 1] : total_rows;
            p.lens_out[b * p.lens_stride] = len[b] + end - row0[b];
            p.q_starts[b + 1] = end;
        }
    }
    if (at == 0) {
        if (!TRIM) p.q_starts[0] = 0;
        p.free_left[0] = int(TRIM ? count + total_blocks : count - total_blocks);
    }
    for (int i = at; i < total_blocks; i += step) {
        const int b = find(blk0, B, i);
        if (TRIM) {
            const int64_t j = ((int64_t(row0[b]) + low) >> p.block_shift) + (i - blk0[b]);
            p.free_blocks[count + i] = p.bt[b * p.bt_b + j * p.bt_j];
        } else {
            const int64_t j = ((int64_t(len[b]) + low) >> p.block_shift) + (i - blk0[b]);
            p.bt[b * p.bt_b + j * p.bt_j] = p.free_blocks[count - 1 - i];
        }
    }
    if (TRIM) return;
    // four neighbouring rows a thread: one bisection for those of a request, and their loads together
    const bool quads = ((reinterpret_cast<uintptr_t>(p.req) | reinterpret_cast<uintptr_t>(p.pos) |
                         reinterpret_cast<uintptr_t>(p.slot_mapping)) & 15) == 0;
    const int num_rows = int(p.num_rows);
    for (int64_t i0 = 4 * int64_t(at); i0 < num_rows; i0 += 4 * int64_t(step)) {
        int b[4], pos[4];
        int64_t slot[4];
        int cur = i0 < total_rows ? find(row0, B, int(i0)) : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = int(i0) + u;
            b[u] = pos[u] = -1;
            slot[u] = -1;
            if (i < total_rows) {
                if (cur + 1 < B && row0[cur + 1] <= i) cur = find(row0, B, i);
                b[u] = cur;
                pos[u] = len[cur] + (i - row0[cur]);
                const int64_t j = pos[u] >> p.block_shift, have = (int64_t(len[cur]) + low) >> p.block_shift;
                // the request's own last block, or one of those handed out now (which are not read back)
                const int32_t *entry = j < have ? p.bt + cur * p.bt_b + j * p.bt_j : p.free_blocks + (count - 1 - (blk0[cur] + (j - have)));
                slot[u] = *entry;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (pos[u] >= 0) slot[u] = (slot[u] << p.block_shift) + (pos[u] & low);
        if (quads && i0 + 4 <= num_rows) {
            *reinterpret_cast<int4 *>(p.req + i0) = make_int4(b[0], b[1], b[2], b[3]);
            *reinterpret_cast<int4 *>(p.pos + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<longlong2 *>(p.slot_mapping + i0) = make_longlong2(slot[0], slot[1]);
            *reinterpret_cast<longlong2 *>(p.slot_mapping + i0 + 2) = make_longlong2(slot[2], slot[3]);
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + u < num_rows) {
                    p.req[i0 + u] = b[u];
                    p.pos[i0 + u] = pos[u];
                    p.slot_mapping[i0 + u] = slot[u];
                }
        }
    }
}

template <bool TRIM>
cudaError_t launch_tables_t(const TableParams &p, int ctas, int threads, cudaStream_t s)
{
    const size_t smem = size_t(p.batch) * 12;
    static std::atomic<int> configured[kTableMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kTableMaxDevices) return cudaErrorInvalidDevice;
    if (int(smem) > 40 * 1024 && configured[dev].load(std::memory_order_relaxed) < int(smem)) {
        e = cudaFuncSetAttribute(tables_kernel<TRIM>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTableMaxBatch * 12);
        if (e != cudaSuccess) return e;
        configured[dev].store(kTableMaxBatch * 12, std::memory_order_relaxed);
    }
    if (ctas > 8) {                                 // beyond the portable size, if this GPU has room for it
        static std::atomic<int> wide[kTableMaxDevices];         // 0: not asked yet, else 8 or 16
        int w = wide[dev].load(std::memory_order_relaxed);
        if (w == 0) {
            w = cudaFuncSetAttribute(tables_kernel<TRIM>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess ? 16 : 8;
            if (w == 8) cudaGetLastError();
            wide[dev].store(w, std::memory_order_relaxed);
        }
        ctas = w;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (ctas > 8) {
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, tables_kernel<TRIM>, &cfg) != cudaSuccess || clusters < 1) {
            cudaGetLastError();
            cfg.gridDim = dim3(8);
            attr[1].val.clusterDim.x = 8;
        }
    }
    return cudaLaunchKernelEx(&cfg, tables_kernel<TRIM>, p);
}

}  // namespace

cudaError_t launch_tables(const TableParams &p, bool trim, cudaStream_t s)
{
    // one CTA, or the eight of a portable cluster, or sixteen, where there are many rows,
    // or many requests that may drop blocks
    const int64_t work = trim ? int64_t(p.batch) * p.max_blocks / 8 : p.num_rows;
    const int ctas = work > 16 * kTableThreads ? 16 : work > 4 * kTableThreads ? 8 : 1;
    // a decode step's few requests and rows: fewer warps to bring together
    const int threads = p.batch <= 256 && work <= 1024 ? 256 : kTableThreads;
    return trim ? launch_tables_t<true>(p, ctas, threads, s) : launch_tables_t<false>(p, ctas, threads, s);
}

}  // namespace pkv
