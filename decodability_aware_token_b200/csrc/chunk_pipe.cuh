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
using tc::tma_load_2d;

constexpr int kUnits = 4;  // unit descriptors in flight

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
    int g, tok0;              // KV head, first token
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
    ud.g = wk.g;
    ud.tok0 = wk.k * sh.tok;
    ud.blk0 = wk.blk0;
    ud.nb = wk.blk1 - wk.blk0;
    ud.c0 = -1;
    if (!wk.whole()) {
        wk.pieces(rg, ud.c0, ud.c1);
        ud.slot0 = wk.slot(rg, ud.c0);  // (a later CTA's piece of the unit is its first: slot 2c)
    }
}

}  // namespace
}  // namespace focus
