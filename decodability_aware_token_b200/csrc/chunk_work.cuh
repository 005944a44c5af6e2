// Work split of the chunk attention kernels.
//
// A unit is (request b, KV head g, tile k of `tok` tokens); it walks ceil(visible keys / KEYS) key blocks
// (at least one, so that rows that see nothing are still written).  The units of a launch, in the order
// b, g, k, form one line of W blocks, and CTA c of C takes an equal share of it (W / C blocks, the first W % C
// CTAs one more): every CTA walks the same number of key blocks whatever the lengths are, and at most its
// first and its last unit are shared with neighbours.  Shared units write unnormalised partial results; the CTA that
// arrives last adds them in block order, so the result does not depend on the order of arrival.
//
// Each CTA finds its own range from the lengths alone, by a scan over the requests (in registers when every thread
// has at most one): no scheduling kernel, no host copy of the lengths.
#pragma once
#include "chunk.h"

namespace focus {
namespace {

struct ChunkReq {
    int row0, n, kv;  // first row, rows, cached keys (n = 0: nothing to do)
};

// Request b's rows and keys; a request whose numbers are out of range is flagged and skipped.  (Read from L2: a kernel
// that does not wait for the one before it must not meet an old line.)  *back becomes 1 where the row offsets decrease.
__device__ __forceinline__ ChunkReq chunk_req(const ChunkAttnDev& a, int b, bool flag, int* back = nullptr) {
    ChunkReq r;
    r.row0 = __ldcg(a.row_offsets + b);
    const int end = __ldcg(a.row_offsets + b + 1);
    r.kv = __ldcg(a.kv_len + b);
    r.n = 0;
    if (back != nullptr && end < r.row0) *back = 1;
    if (r.row0 < 0 || end < r.row0 || end > a.rows || end - r.row0 > a.max_new) {
        if (flag) raise_err(a.err, FOCUS_DEVERR_ROWS);
    } else if (r.kv < 0 || r.kv > a.max_pages * a.S) {
        if (flag) raise_err(a.err, FOCUS_DEVERR_PREFIX);
    } else {
        r.n = end - r.row0;
    }
    return r;
}

// Keys visible at position pos (the API clamps mask_block so that nothing overflows).
__device__ __forceinline__ int chunk_visible(int pos, int kv, int mask_block) {
    if (pos < 0) return 0;
    return min(kv, mask_block == 1 ? pos + 1 : (pos / mask_block + 1) * mask_block);
}

// Key blocks of tile k
template <int KEYS>
__device__ __forceinline__ int chunk_tile_blocks(const ChunkReq& r, int mask_block, int tok, int k) {
    const int last = min(r.n, (k + 1) * tok) - 1;
    const int v = chunk_visible(r.kv - r.n + last, r.kv, mask_block);
    return max(1, (v + KEYS - 1) / KEYS);
}

// Which requests a kernel serves: lo < n G <= hi.
struct ChunkShape {
    int tok, lo, hi;
};
__device__ __forceinline__ int chunk_tiles(const ChunkAttnDev& a, const ChunkShape& sh, const ChunkReq& r) {
    const long long v = (long long)r.n * a.G;
    return v > sh.lo && v <= sh.hi ? (r.n + sh.tok - 1) / sh.tok : 0;
}

// 64-bit quotient, in 32 bits where both fit (five times as fast)
__device__ __forceinline__ long long chunk_div(long long x, long long y) {
    return ((unsigned long long)(x | y) >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)y) : x / y;
}

struct ChunkRange {
    long long w0, w1;     // this CTA's blocks of the line (w0 == w1: none)
    long long share;      // W / C
    int extra;            // W % C: CTAs 0 .. extra - 1 have share + 1 blocks
    int b, g, k, blk;     // where w0 lies
    int tiles;            // tiles of request b
    ChunkReq req;         // request b

    __device__ __forceinline__ long long start(int c) const { return share * c + min(c, extra); }
    // CTA whose range holds block w
    __device__ __forceinline__ int owner(long long w) const {
        const long long big = (share + 1) * extra;
        return w < big ? (int)chunk_div(w, share + 1) : extra + (int)chunk_div(w - big, share);
    }
};

// The share of CTA blockIdx.x in a line of W blocks over at most gridDim.x CTAs of at least MINB blocks each.
template <int MINB> __device__ __forceinline__ ChunkRange chunk_share(long long W) {
    ChunkRange rg{};
    if (W > 0) {
        const long long want = chunk_div(W + MINB - 1, MINB);
        const int C = (int)(want < gridDim.x ? want : (long long)gridDim.x), c = blockIdx.x;
        rg.share = chunk_div(W, C);
        rg.extra = (int)(W - rg.share * C);
        if (c < C) {
            rg.w0 = rg.start(c);
            rg.w1 = rg.start(c + 1);
        }
    }
    return rg;
}

// Fill *out (shared memory) for this CTA.  `scr` holds N long longs of shared memory, `red` 32.  Every thread of
// the block calls it; it ends with a barrier.  MINB: smallest useful share of a CTA.
template <int KEYS, int MINB>
__device__ void chunk_schedule(const ChunkAttnDev& a, const ChunkShape& sh, long long* scr, long long* red,
                               ChunkRange* out) {
    const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
    // Tiles one thread counts by itself; a request of more takes the general way below, with its 64-bit scans.  (A
    // prompt of 8192 tokens has 64: its attention took 279 us this way, 287 the other, in short runs.  At the limit both take
    // as long, over seconds: a prompt of 128 tiles 1090 us this way, 1095 the other; one of 129 tiles 1107 and 1109; one of
    // 128 beside 200 short chunks 1433 and 1439.)
    constexpr int kSerial = 128;
    int any_long = 0;
    if (a.N <= nt && a.small_walk) {
        // a request per thread, sums in registers and 32 bits, three barriers; falls through if some request has
        // many tiles, or if the row offsets decrease somewhere: the ranges behind and before that place may overlap, and
        // the sums be many times what a.small_walk allows for
        ChunkReq r{};
        int tiles = 0;
        uint32_t s = 0;
        if (tid < a.N) {
            r = chunk_req(a, tid, blockIdx.x == 0, &any_long);
            tiles = chunk_tiles(a, sh, r);
            if (tiles > kSerial) any_long = 1;
            else
                for (int k = 0; k < tiles; ++k) s += (uint32_t)chunk_tile_blocks<KEYS>(r, a.mask_block, sh.tok, k);
        }
        uint32_t hi = s * a.Hkv;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, hi, o);
            if (lane >= o) hi += u;
        }
        uint32_t* red32 = reinterpret_cast<uint32_t*>(red);
        if (lane == 31) red32[warp] = hi;
        if (!__syncthreads_or(any_long)) {
            uint32_t before = 0, all = 0;
#pragma unroll
            for (int w = 0; w < 16; ++w) {
                const uint32_t x = w < nw ? red32[w] : 0u;
                if (w < warp) before += x;
                all += x;
            }
            hi += before;
            const uint32_t lo = hi - s * a.Hkv;
            ChunkRange rg = chunk_share<MINB>(all);
            const uint32_t w0 = (uint32_t)rg.w0;
            if (rg.w0 < rg.w1 && hi > w0 && lo <= w0) {
                rg.b = tid;
                rg.g = (int)((w0 - lo) / s);
                rg.req = r;
                rg.tiles = tiles;
                int rem = (int)(w0 - lo - (uint32_t)rg.g * s);
                for (;; ++rg.k) {
                    const int nb = chunk_tile_blocks<KEYS>(r, a.mask_block, sh.tok, rg.k);
                    if (rem < nb) break;
                    rem -= nb;
                }
                rg.blk = rem;
                *out = rg;
            } else if (rg.w0 >= rg.w1 && tid == 0) {
                *out = rg;
            }
            __syncthreads();
            return;
        }
    }
    // blocks of one KV head per request; requests of many tiles are left to whole warps
    for (int b = tid; b < a.N; b += nt) {
        const ChunkReq r = chunk_req(a, b, blockIdx.x == 0);
        const int tiles = chunk_tiles(a, sh, r);
        long long s = 0;
        if (tiles <= kSerial) {
            for (int k = 0; k < tiles; ++k) s += chunk_tile_blocks<KEYS>(r, a.mask_block, sh.tok, k);
        } else {
            s = -1;
            any_long = 1;
        }
        scr[b] = s;
    }
    if (__syncthreads_or(any_long)) {
        for (int b = warp; b < a.N; b += nw) {
            if (scr[b] >= 0) continue;
            const ChunkReq r = chunk_req(a, b, false);
            const int tiles = chunk_tiles(a, sh, r);
            long long s = 0;
            for (int k = lane; k < tiles; k += 32) s += chunk_tile_blocks<KEYS>(r, a.mask_block, sh.tok, k);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) scr[b] = s;
            __syncwarp();
        }
        __syncthreads();
    }
    // inclusive scan over the requests (all KV heads)
    long long carry = 0;
    for (int b0 = 0; b0 < a.N; b0 += nt) {
        const int b = b0 + tid;
        long long v = b < a.N ? scr[b] * a.Hkv : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) red[warp] = v;
        __syncthreads();
        long long before = carry, all = 0;
        for (int w = 0; w < nw; ++w) {
            const long long x = red[w];
            if (w < warp) before += x;
            all += x;
        }
        if (b < a.N) scr[b] = before + v;
        carry += all;
        __syncthreads();
    }
    const long long W = carry;
    const ChunkRange rg = chunk_share<MINB>(W);
    if (tid == 0) *out = rg;
    __syncthreads();
    if (rg.w0 < rg.w1) {  // (the same in every thread)
        int many = 0;
        for (int b = tid; b < a.N; b += nt) {
            const long long hi = scr[b], lo = b ? scr[b - 1] : 0;
            if (hi <= rg.w0 || lo > rg.w0) continue;
            const long long per = chunk_div(hi - lo, a.Hkv), off = rg.w0 - lo;  // blocks of one KV head
            const int g = (int)chunk_div(off, per);
            out->b = b;
            out->g = g;
            out->k = 0;
            out->blk = (int)(off - g * per);  // (more than an int holds only with many tiles, found below)
            out->req = chunk_req(a, b, false);
            out->tiles = chunk_tiles(a, sh, out->req);
            if (out->tiles > 1) many = 1;
        }
        if (__syncthreads_or(many) && warp == 0) {
            const int b = out->b, g = out->g, tiles = out->tiles;
            const ChunkReq r = out->req;
            const long long lo = b ? scr[b - 1] : 0;
            long long rem = rg.w0 - lo - g * chunk_div(scr[b] - lo, a.Hkv);
            for (int k0 = 0; k0 < tiles; k0 += 32) {
                const int k = k0 + lane;
                const long long mine = k < tiles ? chunk_tile_blocks<KEYS>(r, a.mask_block, sh.tok, k) : 0;
                long long v = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long u = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += u;
                }
                const bool here = v > rem && v - mine <= rem;
                if (here) {
                    out->k = k;
                    out->blk = (int)(rem - (v - mine));
                }
                if (__any_sync(0xffffffffu, here)) break;
                rem -= __shfl_sync(0xffffffffu, v, 31);
            }
        }
    }
    __syncthreads();
}

// One thread's walk along its CTA's range, unit piece by unit piece.
template <int KEYS>
struct ChunkWalk {
    long long w, w1;   // next block, end
    int b, g, k;       // the unit at w
    int blk0, blk1;    // the piece's blocks within the unit
    int nblk;          // blocks of the whole unit
    int tiles;
    ChunkReq r;

    __device__ __forceinline__ void start(const ChunkAttnDev& a, const ChunkShape& sh, const ChunkRange& rg) {
        w = rg.w0;
        w1 = rg.w1;
        b = rg.b;
        g = rg.g;
        k = rg.k;
        blk0 = rg.blk;
        if (w < w1) {
            r = rg.req;
            tiles = rg.tiles;
            fit(a, sh);
        }
    }
    __device__ __forceinline__ bool live() const { return w < w1; }
    __device__ __forceinline__ void fit(const ChunkAttnDev& a, const ChunkShape& sh) {
        nblk = chunk_tile_blocks<KEYS>(r, a.mask_block, sh.tok, k);
        const long long left = w1 - w;
        blk1 = nblk - blk0 <= left ? nblk : blk0 + (int)left;
    }
    __device__ __forceinline__ void next(const ChunkAttnDev& a, const ChunkShape& sh) {
        w += blk1 - blk0;
        if (w >= w1) return;
        blk0 = 0;
        if (++k == tiles) {
            k = 0;
            if (++g == a.Hkv) {
                g = 0;
                do {  // the range ends inside the line, so a request with work follows
                    if (++b >= a.N) {
                        w = w1;  // (only if the lengths changed under the launch)
                        return;
                    }
                    r = chunk_req(a, b, false);
                    tiles = chunk_tiles(a, sh, r);
                } while (tiles == 0);
            }
        }
        fit(a, sh);
    }
    __device__ __forceinline__ bool whole() const { return blk0 == 0 && blk1 == nblk; }
    // the CTAs that hold the unit's pieces, and the scratch slot of c0's: its first (2 c0) unless the unit
    // starts inside its range; a later CTA's piece of the unit is its first
    __device__ __forceinline__ void pieces(const ChunkRange& rg, int& c0, int& c1, int& slot0) const {
        const long long u0 = w - blk0;
        c0 = rg.owner(u0);
        c1 = rg.owner(u0 + nblk - 1);
        slot0 = 2 * c0 + (rg.start(c0) < u0 ? 1 : 0);
    }
};

}  // namespace
}  // namespace focus
