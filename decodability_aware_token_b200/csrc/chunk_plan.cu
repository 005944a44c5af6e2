// Pages, rows and cache slots of a chunk from the request lengths, in one launch.
//
// Three sums over the requests decide everything: rows asked for (does the row buffer hold them), pages
// needed by those (does the free list), rows of the placed ones (the row offsets).  Each CTA runs the three
// scans itself over all requests (they are a few hundred integers) and then writes its own slice of the
// rows and every gridDim-th request's new pages: no CTA waits for another, and a row whose page is new
// takes it from the free list, not from the table another CTA is writing.  Bound: latency of two dependent
// loads and the scan for small batches, the 12 bytes written per row for large ones.
#include "chunk.h"

namespace focus {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerCta = 1024;

__global__ void __launch_bounds__(kThreads) chunk_plan_kernel(ChunkPlanDev a) {
    pdl_entry();
    const focus_chunk_plan& p = a.p;
    extern __shared__ int32_t sm[];
    const int N = p.n_requests, S = p.page_size;
    int32_t* off = sm;                // [N + 1] row offsets
    int32_t* pre = off + N + 1;       // [N] prefix lengths
    int32_t* first = pre + N;         // [N] free-list index of a request's first new page
    __shared__ long long red[3][kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool lead = blockIdx.x == 0;
    const long long cap = (long long)a.max_pages * S;

    const int head = *p.free_head;
    const bool head_ok = head >= 0 && head <= p.n_free;
    const int avail = head_ok ? p.n_free - head : 0;
    if (!head_ok && lead && tid == 0) raise_err(a.err, FOCUS_DEVERR_PAGE_ID);

    // running totals over the earlier requests: rows asked, pages needed, rows placed, pages taken
    long long c_ask = 0, c_need = 0, c_rows = 0, c_taken = 0;
    for (int b0 = 0; b0 < N; b0 += kThreads) {
        const int b = b0 + tid;
        int pl = 0, n = 0;
        bool valid = false;
        if (b < N) {
            pl = p.prefix_len[b];
            n = p.new_len[b];
            valid = pl >= 0 && n >= 0 && (long long)pl + n <= cap;
            if (!valid && lead) raise_err(a.err, FOCUS_DEVERR_PREFIX);
        }
        auto scan = [&](long long v, int which, long long& total) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (lane == 31) red[which][warp] = v;
            __syncthreads();
            total = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) v += red[which][w];
                total += red[which][w];
            }
            return v;
        };
        long long t_ask, t_need, t_rows;
        const long long ask = c_ask + scan(valid ? n : 0, 0, t_ask);
        const bool rows_ok = valid && (n == 0 || ask <= p.max_rows);
        const int have = rows_ok ? (pl + S - 1) / S : 0;
        const int need = rows_ok ? (pl + n + S - 1) / S - have : 0;
        const long long upto = c_need + scan(need, 1, t_need);
        const bool placed = rows_ok && (need == 0 || upto <= avail);
        const int rows = placed ? n : 0;
        const long long end = c_rows + scan(rows, 2, t_rows);
        if (b < N) {
            off[b] = (int)(end - rows);
            pre[b] = pl;
            first[b] = placed && need > 0 ? head + (int)(upto - need) : head;
            if (lead) {
                p.row_offsets[b] = (int)(end - rows);
                p.kv_len[b] = pl + rows;
            }
        }
        // pages taken: the needs of the placed requests are a prefix of all needs
        long long mine = placed && need > 0 ? upto : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const long long u = __shfl_xor_sync(0xffffffffu, mine, o);
            mine = u > mine ? u : mine;
        }
        __syncthreads();  // red has been read
        if (lane == 0) red[0][warp] = mine;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) c_taken = red[0][w] > c_taken ? red[0][w] : c_taken;
        c_ask += t_ask;
        c_need += t_need;
        c_rows += t_rows;
        __syncthreads();  // red is reused by the next round
    }
    const int total = (int)c_rows;
    if (tid == 0) {
        off[N] = total;
        if (lead) p.row_offsets[N] = total;
    }
    __syncthreads();

    auto checked = [&](int page) {
        if (page >= 0 && page < p.n_pages) return page;
        raise_err(a.err, FOCUS_DEVERR_PAGE_ID);
        return -1;
    };
    // new pages of every gridDim-th request
    for (int b = blockIdx.x; b < N; b += gridDim.x) {
        const int n = off[b + 1] - off[b];
        if (n <= 0) continue;
        const int have = (pre[b] + S - 1) / S, all = (pre[b] + n + S - 1) / S;
        for (int i = have + tid; i < all; i += kThreads)
            p.page_table[(size_t)b * a.max_pages + i] = checked(p.free_pages[first[b] + i - have]);
    }
    // this CTA's rows
    const int r1 = min(p.max_rows, (int)(blockIdx.x + 1) * kRowsPerCta);
    for (int r = blockIdx.x * kRowsPerCta + tid; r < r1; r += kThreads) {
        int req = -1, pos = -1, slot = -1;
        if (r < total) {
            int lo = 0, hi = N;  // largest b with off[b] <= r: it has rows, since off[b + 1] > r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (off[mid] <= r) lo = mid;
                else hi = mid;
            }
            req = lo;
            pos = pre[lo] + r - off[lo];
            const int i = pos / S, have = (pre[lo] + S - 1) / S;
            const int page = checked(i < have ? p.page_table[(size_t)lo * a.max_pages + i]
                                              : p.free_pages[first[lo] + i - have]);
            slot = page < 0 ? -1 : page * S + pos - i * S;
        }
        p.row_req[r] = req;
        p.row_pos[r] = pos;
        p.row_slot[r] = slot;
    }
    // free_next may be free_head: it is written once every CTA has read the head
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        if (atomicInc(reinterpret_cast<unsigned*>(a.arrivals), gridDim.x - 1) == gridDim.x - 1)
            *p.free_next = head + (int)c_taken;
    }
}

}  // namespace

bool configure_chunk_plan_kernel() {
    return cudaFuncSetAttribute(chunk_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (3 * kChunkMaxRequests + 1) * 4) == cudaSuccess &&
           max_shared_carveout((const void*)chunk_plan_kernel);
}

int launch_chunk_plan(const ChunkPlanDev& a, cudaStream_t s) {
    const int ctas = a.p.max_rows > kRowsPerCta ? (a.p.max_rows + kRowsPerCta - 1) / kRowsPerCta : 1;
    return launched(launch_pdl(chunk_plan_kernel, dim3(ctas), dim3(kThreads), (3 * a.p.n_requests + 1) * 4, s, 0, a));
}

}  // namespace focus
