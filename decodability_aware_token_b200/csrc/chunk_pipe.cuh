// What the two bf16 chunk attention kernels share beside the work split: bounded waits, and the queue of unit
// descriptors through which the copy warp, which walks the CTA's range, tells the other warps what comes.
#pragma once
#include "chunk_work.cuh"
#include "tc_gemm_kernel.cuh"

namespace focus {
namespace {

using tc::mbar_arrive;
using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::smem_u32;

// As tc::mbar_wait, but the clock is read only every 64 failed tries: the waiting warps share their SM
// quarter's issue slots with the ones that work.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, int* err) {
    const uint32_t addr = smem_u32(bar);
    if (tc::mbar_try(addr, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (tc::mbar_try(addr, parity)) return true;
        if (clock64() - t0 > tc::kWaitCycles) {
            raise_err(err, FOCUS_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// The same for a whole warp.  Its lanes leave together: one that ran on alone could pass the barrier's next two
// phases while the others still look for this one, and they would then wait for a parity that has come and gone.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, err)) != 0;
}

// N threads meet at named barrier `id`; all_agree also tells whether `ok` held in every one of them.
template <int N> __device__ __forceinline__ void named_sync(int id) { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory"); }
template <int N> __device__ __forceinline__ bool all_agree(int id, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "bar.red.and.pred p, %1, %3, q;\n\tselp.b32 %0, 1, 0, p;\n\t}\n"
        : "=r"(all)
        : "r"(id), "r"((uint32_t)ok), "n"(N)
        : "memory");
    return all != 0;
}

// One piece of a unit, written by the copy thread as it reaches it and read by the other roles.
struct UnitDesc {
    int row0, n, kv;          // the request
    int b, g, tok0;           // request number, KV head, first token
    int blk0, nb;             // key blocks of the piece (nb = 0: no more units)
    int c0, c1, slot0;        // CTAs that hold pieces (c0 = -1: the whole unit is here), scratch slot of c0's
};

template <int KEYS>
__device__ __forceinline__ void describe(UnitDesc& ud, const ChunkWalk<KEYS>& wk, const ChunkRange& rg, const ChunkShape& sh,
                                         bool live) {
    ud.nb = 0;
    if (!live) return;
    ud.row0 = wk.r.row0;
    ud.n = wk.r.n;
    ud.kv = wk.r.kv;
    ud.b = wk.b;
    ud.g = wk.g;
    ud.tok0 = wk.k * sh.tok;
    ud.blk0 = wk.blk0;
    ud.nb = wk.blk1 - wk.blk0;
    ud.c0 = -1;
    if (!wk.whole()) wk.pieces(rg, ud.c0, ud.c1, ud.slot0);
}

// The pool's rows of 128 columns for TMA, as (64 columns, S tokens, column half, K / V, x) with
// x = (page L + layer) 2 Hkv + head: one copy takes a page's K or V of a head, or both, as `halves` x `kvs`
// tiles of [S][64 columns] with 128-byte rows, swizzled.  A copy instruction takes its issuing warp
// 65 to 100 cycles whatever it moves (measured; lanes of one warp take turns, warps do not), so the fewest
// and largest are used.
inline bool make_pool_map(CUtensorMap* m, const ChunkAttnDev& a, int halves, int kvs) {
    auto fn = tc::encode_fn();
    if (!fn) return false;
    const cuuint64_t row = 256, head = (cuuint64_t)a.S * row;
    const cuuint64_t dims[5] = {64, (cuuint64_t)a.S, 2, 2, (cuuint64_t)a.n_pages * a.L * 2 * a.Hkv};
    const cuuint64_t strides[4] = {row, 128, head * a.Hkv, head};
    const cuuint32_t box[5] = {64, (cuuint32_t)a.S, (cuuint32_t)halves, (cuuint32_t)kvs, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(a.kv_pool), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
__device__ __forceinline__ void tma_load_pool(const CUtensorMap* map, uint64_t* bar, void* dst, int half, int kv, int x) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %4, %5, %6}], [%2];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(0), "r"(half), "r"(kv), "r"(x)
        : "memory");
}

// The pages of one key block at a time, for a whole warp: the next 32 entries of the request's table row sit in
// the lanes, so a block's ids cost a shuffle, not a load, and each lane issues the copies of its own page.
struct PageWalk {
    const int32_t* pt;
    int pages, max_pages, at, ahead0, ahead;  // pages that hold keys, row length, next entry, entries ahead0 + lane
    __device__ __forceinline__ void start(const ChunkAttnDev& a, int b, int kv, int first) {
        pt = a.page_table + (size_t)b * a.max_pages;
        pages = (kv + a.S - 1) / a.S;
        max_pages = a.max_pages;
        at = first;
        load();
    }
    __device__ __forceinline__ void load() {
        const int i = at + (int)(threadIdx.x & 31);
        ahead0 = at;
        ahead = i < max_pages ? __ldcg(pt + i) : -1;
    }
    // Lane p < ppb gets the id of the block's page p, -1 if there is none (`got` false) or it is not in the pool;
    // `bad` (every lane): the block's 16-key groups that a bad id covers; returns the number of good pages.
    __device__ __forceinline__ int block(const ChunkAttnDev& a, int ppb, int& page, uint32_t& bad) {
        if (at + ppb > ahead0 + 32) load();
        const int lane = threadIdx.x & 31;
        page = __shfl_sync(0xffffffffu, ahead, (at + lane - ahead0) & 31);
        const bool in = lane < ppb && at + lane < pages;
        const bool good = in && page >= 0 && page < a.n_pages;
        if (!good) page = -1;
        const uint32_t good_m = __ballot_sync(0xffffffffu, good), bad_m = __ballot_sync(0xffffffffu, in && !good);
        bad = 0;
        if (bad_m) {
            const int groups = a.S / 16;
            for (int p = 0; p < ppb; ++p)
                if ((bad_m >> p) & 1u) bad |= ((1u << groups) - 1u) << (p * groups);
        }
        return __popc(good_m);
    }
};

// One lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}\n" : "=r"(e));
    return e;
}

}  // namespace
}  // namespace focus
