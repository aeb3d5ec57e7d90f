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
// the same memory.  Bound by latency: a launch and three trips to memory.
#include <cooperative_groups.h>

#include <atomic>

#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kTableThreads = 512;
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
    for (int w = 0; w < warp; ++w) {
        a += sums[w][0];
        b += sums[w][1];
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
    const int64_t round = (int64_t(1) << p.block_shift) - 1;
    int64_t count = p.free_count[0];
    bool bad_pool = count < 0 || count > p.pool;
    count = count < 0 ? 0 : count > p.pool ? p.pool : count;
    // what a stack can give, or take
    const int64_t room = TRIM ? p.pool - count : count;
    if (tid < 2) totals[tid] = 0;
    const int per = (B + kTableThreads - 1) / kTableThreads;
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
            blocks = ((cached + round) >> p.block_shift) - ((n + round) >> p.block_shift);
        } else {
            if (n < 0 || cached + n > cap) {
                bad_len = true;
                n = 0;
            }
            rows = n;
            blocks = ((cached + n + round) >> p.block_shift) - ((cached + round) >> p.block_shift);
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
    for (int b = b0; b < b1; ++b) {
        int64_t cached, rows, blocks;
        request(b, cached, rows, blocks);
        const bool fits = (TRIM || r + rows <= p.num_rows) && k + blocks <= room;
        if (fits) {
            if (!TRIM) atomicMax(&totals[0], int(r + rows));
            atomicMax(&totals[1], int(k + blocks));
        } else if (rows > 0 || blocks > 0) {
            bad_pool = true;
        }
        row0[b] = TRIM ? int(fits ? rows : cached) : int(r < p.num_rows ? r : p.num_rows);
        blk0[b] = int(k < room ? k : room);
        len[b] = int(cached);
        r += rows;
        k += blocks;
    }
    if (blockIdx.x == 0) {
        if (bad_len) raise_err(p.err_flag, PKV_DEVERR_CONTEXT_RANGE);
        if (bad_pool) raise_err(p.err_flag, PKV_DEVERR_POOL_RANGE);
    }
    __syncthreads();
    const int total_rows = totals[0], total_blocks = totals[1];
    for (int b = tid; b < B; b += kTableThreads) {
        if (!TRIM) row0[b] = min(row0[b], total_rows);
        blk0[b] = min(blk0[b], total_blocks);
    }
    // all CTAs have read the lengths and counts that are written below
    cooperative_groups::this_cluster().sync();

    const int at = blockIdx.x * kTableThreads + tid, step = gridDim.x * kTableThreads;
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
            const int64_t j = ((int64_t(row0[b]) + round) >> p.block_shift) + (i - blk0[b]);
            p.free_blocks[count + i] = p.bt[b * p.bt_b + j * p.bt_j];
        } else {
            const int64_t j = ((int64_t(len[b]) + round) >> p.block_shift) + (i - blk0[b]);
            p.bt[b * p.bt_b + j * p.bt_j] = p.free_blocks[count - 1 - i];
        }
    }
    if (TRIM) return;
    for (int i = at; i < p.num_rows; i += step) {
        int b = -1, pos = -1;
        int64_t slot = -1;
        if (i < total_rows) {
            b = find(row0, B, i);
            pos = len[b] + (i - row0[b]);
            const int64_t j = pos >> p.block_shift, have = (int64_t(len[b]) + round) >> p.block_shift;
            // the request's own last block, or one of those handed out now (which are not read back)
            const int64_t blk = j < have ? p.bt[b * p.bt_b + j * p.bt_j] : p.free_blocks[count - 1 - (blk0[b] + (j - have))];
            slot = (blk << p.block_shift) + (pos & round);
        }
        p.req[i] = b;
        p.pos[i] = pos;
        p.slot_mapping[i] = slot;
    }
}

template <bool TRIM>
cudaError_t launch_tables_t(const TableParams &p, int ctas, cudaStream_t s)
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kTableThreads);
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
    return cudaLaunchKernelEx(&cfg, tables_kernel<TRIM>, p);
}

}  // namespace

cudaError_t launch_tables(const TableParams &p, bool trim, cudaStream_t s)
{
    // one CTA, or the eight of a portable cluster where there are many rows, or many
    // requests that may drop blocks
    const int64_t work = trim ? int64_t(p.batch) * p.max_blocks / 8 : p.num_rows;
    const int ctas = work > 4 * kTableThreads ? 8 : 1;
    return trim ? launch_tables_t<true>(p, ctas, s) : launch_tables_t<false>(p, ctas, s);
}

}  // namespace pkv
