// Pages, rows and cache slots of a chunk from the request lengths, in one launch.
//
// Sums over the requests decide everything: rows asked for (does the row buffer hold them), pages needed by those
// (does the free list), rows of the placed ones (the row offsets).  Each CTA runs the scans itself over all
// requests -- a few hundred integers, a run of consecutive ones per thread -- and then writes its own slice of the
// rows: no CTA waits for another.  When everything fits, which the first scan tells, it is the only one.  A row
// whose page is new takes it from the free list, not from the table another CTA is writing, and the row that
// starts a new page writes its table entry (a new page always starts inside the chunk).
//
// Bound: the latency of the launch, two dependent loads and the scans, and for large batches the searches and the 12
// bytes written per row.  Measured inside a graph: 32 single tokens 2.4 us (an empty kernel takes as long), 256
// ragged prompts that do not all fit, 131072 rows, 6.6 us (with 256, 1024 or 2048 rows a CTA 7.9, 7.3 and 10.2).
#include "chunk.h"

namespace focus {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = 512;

// Inclusive scan of x and y over the block; the totals in tx, ty.  `red` holds 2 x 8 long longs; two barriers.
__device__ __forceinline__ void block_scan2(long long& x, long long& y, long long& tx, long long& ty, long long (*red)[8]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    __syncthreads();  // red has been read by the scan before
    if (lane == 31) {
        red[0][warp] = x;
        red[1][warp] = y;
    }
    __syncthreads();
    tx = ty = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) {
            x += tx;
            y += ty;
        }
        tx += red[0][w];
        ty += red[1][w];
    }
}

__global__ void __launch_bounds__(kThreads) chunk_plan_kernel(ChunkPlanDev a) {
    pdl_wait();  // (and no early trigger: the next kernel's waiting CTAs cost this one's scans more than they gain)
    const focus_chunk_plan& p = a.p;
    extern __shared__ int32_t sm[];
    const int N = p.n_requests, S = p.page_size;
    int32_t* off = sm;                // [N + 1] row offsets
    int32_t* pre = off + N + 1;       // [N] prefix lengths
    int32_t* first = pre + N;         // [N] free-list index of a request's first new page
    __shared__ long long red[2][8];
    const int tid = threadIdx.x;
    const bool lead = blockIdx.x == 0;
    const long long cap = (long long)a.max_pages * S;

    const int head = *p.free_head;
    const bool head_ok = head >= 0 && head <= p.n_free;
    const int avail = head_ok ? p.n_free - head : 0;
    if (!head_ok && lead && tid == 0) raise_err(a.err, FOCUS_DEVERR_PAGE_ID);

    const int per = (N + kThreads - 1) / kThreads, b0 = min(N, tid * per), b1 = min(N, b0 + per);
    // request b's lengths (n = -1: out of range, no rows) and the pages n new tokens need
    auto lens = [&](int b, int& pl, int& n) {
        pl = p.prefix_len[b];
        n = p.new_len[b];
        if (pl < 0 || n < 0 || (long long)pl + n > cap) n = -1;
    };
    auto need = [&](int pl, int n) { return (pl + n + S - 1) / S - (pl + S - 1) / S; };
    auto write = [&](int b, int pl, int rows, long long row, long long page) {
        off[b] = (int)row;
        pre[b] = pl;
        first[b] = head + (int)page;
        if (lead) {
            p.row_offsets[b] = (int)row;
            p.kv_len[b] = pl + rows;
        }
    };
    long long ask = 0, want = 0, all_ask, all_want;
    int pl1 = 0, n1 = 0;  // the thread's lengths when it has one request
    for (int b = b0; b < b1; ++b) {
        lens(b, pl1, n1);
        if (n1 < 0 && lead) raise_err(a.err, FOCUS_DEVERR_PREFIX);
        if (n1 > 0) {
            ask += n1;
            want += need(pl1, n1);
        }
    }
    long long ask_end = ask, want_end = want;
    block_scan2(ask_end, want_end, all_ask, all_want, red);
    long long total = all_ask, taken = all_want;
    if (all_ask <= p.max_rows && all_want <= avail) {
        // everything fits: what was asked for is what is placed
        long long row = ask_end - ask, page = want_end - want;
        for (int b = b0; b < b1; ++b) {
            if (per > 1) lens(b, pl1, n1);
            const int rows = max(n1, 0);
            write(b, pl1, rows, row, page);
            row += rows;
            if (rows > 0) page += need(pl1, rows);
        }
    } else {
        // the row test over all requests, then the page test over those that passed it, then the placed ones' rows
        auto rows_fit = [&](int n, long long& run) {
            if (n <= 0) return n == 0;
            run += n;
            return run <= p.max_rows;
        };
        long long run = ask_end - ask, w = 0, dummy = 0, tw, td;
        for (int b = b0; b < b1; ++b) {
            int pl, n;
            lens(b, pl, n);
            if (rows_fit(n, run)) w += need(pl, n);
        }
        long long w_end = w;
        block_scan2(w_end, dummy, tw, td, red);
        auto placed = [&](int pl, int n, long long& r, long long& pg, int& pages) {
            if (!rows_fit(n, r)) return false;
            pages = need(pl, n);
            pg += pages;
            return pages == 0 || pg <= avail;
        };
        long long mine = 0, got = 0;
        run = ask_end - ask;
        long long pg = w_end - w;
        for (int b = b0; b < b1; ++b) {
            int pl, n, pages = 0;
            lens(b, pl, n);
            if (placed(pl, n, run, pg, pages)) {
                mine += n;
                got += pages;
            }
        }
        long long mine_end = mine, got_end = got;
        block_scan2(mine_end, got_end, total, taken, red);
        run = ask_end - ask;
        pg = w_end - w;
        long long row = mine_end - mine, page = got_end - got;
        for (int b = b0; b < b1; ++b) {
            int pl, n, pages = 0;
            lens(b, pl, n);
            if (!placed(pl, n, run, pg, pages)) n = pages = 0;
            write(b, pl, n, row, page);
            row += n;
            page += pages;
        }
    }
    const int rows_all = (int)total;
    if (tid == 0) {
        off[N] = rows_all;
        if (lead) p.row_offsets[N] = rows_all;
    }
    __syncthreads();

    auto checked = [&](int page) {
        if (page >= 0 && page < p.n_pages) return page;
        raise_err(a.err, FOCUS_DEVERR_PAGE_ID);
        return -1;
    };
    const unsigned r1 = min((unsigned)p.max_rows, (blockIdx.x + 1) * kRowsPerCta);  // (up to 2^31 and a step beyond)
    for (unsigned r0 = blockIdx.x * kRowsPerCta + tid; r0 < r1; r0 += kThreads) {
        const int r = (int)r0;
        int req = -1, pos = -1, slot = -1;
        if (r < rows_all) {
            int lo = 0, hi = N;  // largest b with off[b] <= r: it has rows, since off[b + 1] > r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (off[mid] <= r) lo = mid;
                else hi = mid;
            }
            req = lo;
            pos = pre[lo] + r - off[lo];
            const int i = pos / S, have = (pre[lo] + S - 1) / S;
            int32_t* entry = p.page_table + (size_t)lo * a.max_pages + i;
            const int page = checked(i < have ? *entry : p.free_pages[first[lo] + i - have]);
            if (i >= have && pos == i * S) *entry = page;
            slot = page < 0 ? -1 : page * S + pos - i * S;
        }
        p.row_req[r] = req;
        p.row_pos[r] = pos;
        p.row_slot[r] = slot;
    }
    // free_next may be free_head: it is written once every CTA has read the head
    if (gridDim.x == 1) {
        if (tid == 0) *p.free_next = head + (int)taken;
    } else {
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            if (atomicInc(reinterpret_cast<unsigned*>(a.arrivals), gridDim.x - 1) == gridDim.x - 1)
                *p.free_next = head + (int)taken;
        }
    }
}

__global__ void __launch_bounds__(kThreads) chunk_tokens_kernel(focus_chunk_plan p, const int32_t* __restrict__ tokens,
                                                                int max_new, int32_t* __restrict__ out,
                                                                int32_t* __restrict__ row_at, int* err) {
    pdl_entry();
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i < p.max_rows) {
        const int b = p.row_req[i];
        int tok = 0;
        if (b >= 0) {
            const int at = i - p.row_offsets[b];
            if (at < max_new) tok = tokens[(size_t)b * max_new + at];
            else raise_err(err, FOCUS_DEVERR_ROWS);
        }
        out[i] = tok;
        row_at[i] = max(p.row_pos[i], 0);
    }
    if (i < p.n_requests) const_cast<int32_t*>(p.prefix_len)[i] = p.kv_len[i];
}

}  // namespace

int launch_chunk_tokens(const focus_chunk_plan& p, const int32_t* tokens, int max_new, int32_t* out, int32_t* at, int* err,
                        cudaStream_t s) {
    const int n = p.max_rows > p.n_requests ? p.max_rows : p.n_requests;
    return launched(launch_pdl(chunk_tokens_kernel, dim3((n + kThreads - 1) / kThreads), dim3(kThreads), 0, s, 0, p, tokens,
                               max_new, out, at, err));
}

bool configure_chunk_plan_kernel() {
    return cudaFuncSetAttribute(chunk_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (3 * kChunkMaxRequests + 1) * 4) == cudaSuccess &&
           max_shared_carveout((const void*)chunk_plan_kernel) &&
           max_shared_carveout((const void*)chunk_tokens_kernel);
}

int launch_chunk_plan(const ChunkPlanDev& a, cudaStream_t s) {
    const int ctas = a.p.max_rows > kRowsPerCta ? (int)(((long long)a.p.max_rows + kRowsPerCta - 1) / kRowsPerCta) : 1;
    return launched(launch_pdl(chunk_plan_kernel, dim3(ctas), dim3(kThreads), (3 * a.p.n_requests + 1) * 4, s, 0, a));
}

}  // namespace focus
