// bf16 attention of a chunk over the paged cache on the 5th-generation tensor cores: requests with more
// than kChunkFewRows query vectors per KV head (prompt chunks).  See chunk_work.cuh for how the key walks
// are split over the CTAs.
//
// Unit: request b, KV head g and up to 256 query vectors (token r / G, head r % G) in two tiles of up to
// 128.  Keys come in blocks of 128 through a ring of five 32 KB slots, K_0 V_0 K_1 V_1 ..., each filled from
// whole pages by TMA (two 64-column halves, 128-byte swizzle).  Per tile t and block i:
//   S_t = Q_t K_i^T     tcgen05.mma 128 x 128 x 128, both operands in shared memory, into TMEM
//   softmax             one warpgroup per tile, one thread per query vector: the 128 scores from TMEM,
//                       running maximum and denominator in registers, P = 2^(s - m) as bf16 back into TMEM
//                       over S_t (64 of its 128 columns)
//   O_t += P_t V_i      tcgen05.mma 128 x 128 x 128, P from TMEM, V MN-major straight from the page tile
// The MMA thread issues PV_0(i), S_0(i+1), PV_1(i), S_1(i+1): while one tile is in its softmax the tensor core
// works for the other.  TMEM: S_0, S_1, O_0, O_1, 128 fp32 columns each, all 512.
//
// The running maximum is raised only when a block exceeds it by more than 2^8; O and the denominator are then
// rescaled in TMEM (S_t(i) was issued behind PV_t(i-1), so O is complete when the scores are).  Weights are
// at most 2^8, sums are float32, and the softmax is the same.  P is rounded to bf16 (relative 2^-9 per
// weight, as the storage type of the values it multiplies); the denominator sums the unrounded weights.
//
// Every mbarrier wait is bounded; on expiry the role flags FOCUS_DEVERR_TIMEOUT and stops issuing, copies and
// MMAs in flight are waited for (bounded), and TMEM is released.
#include <math_constants.h>

#include "chunk_work.cuh"
#include "tc_gemm_kernel.cuh"

namespace focus {
namespace {

using tc::idesc_bf16;
using tc::mbar_arrive;
using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;
using tc::mma_bf16;
using tc::mma_commit;
using tc::smem_desc_sw128;
using tc::smem_u32;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tma_load_2d;
using tc::tmem_ld32;

constexpr int kD = 128;
constexpr int kKeys = 128;                    // keys per block
constexpr int kHalf = 128 * 128;              // [128 rows][64 columns] bf16: 16 KB
constexpr int kSlot = 2 * kHalf;              // K or V of one block: 32 KB
constexpr int kSlots = 5;
constexpr int kQTile = 2 * kHalf;             // one query tile: 32 KB
constexpr int kSmem = 2 * kQTile + kSlots * kSlot + 1024;
constexpr int kTileThreads = 384;             // warps 0-3, 4-7: softmax of tile 0, 1; 8: copies; 9: MMAs
constexpr int kFlags = 8;                     // bad-page flags, one per block in flight
constexpr float kRaise = 8.f;
static_assert(kSmem <= 227 * 1024, "shared memory");
static_assert((kChunkMaxRequests + 1) * 8 <= kSlots * kSlot, "the schedule's sums fit in the ring");

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// A (the weights) in TMEM, B in shared memory
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc));
}

// V tile as MN-major operand: 64 columns per 128-byte row, keys on consecutive rows, the next 64 columns
// kHalf on, the next 8 keys 1024 bytes on
__device__ __forceinline__ uint64_t v_desc(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)(kHalf >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

#define TM_LIST32(r)                                                                                          \
    r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], r[10], r[11], r[12], r[13], r[14], r[15], r[16], \
        r[17], r[18], r[19], r[20], r[21], r[22], r[23], r[24], r[25], r[26], r[27], r[28], r[29], r[30], r[31]

// Start reading 32 columns; the registers are valid behind tm_wait on them.
__device__ __forceinline__ void tm_ld(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tm_wait(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                   "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tm_st(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ void sync_group(int t) {
    if (t == 0) asm volatile("bar.sync 1, 128;" ::: "memory");
    else asm volatile("bar.sync 2, 128;" ::: "memory");
}

// Registers by role: 384 threads start with 168 each (64512); the two softmax warpgroups hold a row's 128
// scores, the third (copies, MMAs) needs few: 2 x 128 x 208 + 128 x 88 = 64512.
constexpr int kSoftRegs = 208, kIssueRegs = 88;
static_assert(2 * 128 * kSoftRegs + 128 * kIssueRegs <= 384 * 168, "register split");

__global__ void __launch_bounds__(kTileThreads, 1)
chunk_attn_tile_kernel(const __grid_constant__ CUtensorMap pool_map, const __grid_constant__ CUtensorMap q_map,
                       ChunkAttnDev a, int min_blocks) {
    pdl_trigger();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* q_s = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* ring = q_s + 2 * kQTile;
    __shared__ __align__(8) uint64_t q_full, q_empty, kv_full[kSlots], kv_empty[kSlots], s_full[2], p_full[2], o_full[2],
        done_bar;
    __shared__ uint32_t bad_s[kFlags];  // per block: 16-key groups whose page id is invalid
    __shared__ uint32_t tmem_slot;
    __shared__ ChunkRange rg;
    __shared__ long long red[32];
    __shared__ int last_s[2];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 1);
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&kv_full[s], 1);
            mbar_init(&kv_empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);  // one arrival per softmax warp
            mbar_init(&o_full[t], 1);
        }
        mbar_init(&done_bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 8 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&pool_map) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&q_map) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_wait();

    const int tpt = 128 / a.G;  // tokens per tile
    const ChunkShape sh{2 * tpt, kChunkFewRows, 0x7fffffff};
    chunk_schedule<kKeys>(a, sh, min_blocks, reinterpret_cast<long long*>(ring), red, &rg);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring held the schedule's sums
    __syncthreads();

    ChunkWalk<kKeys> wk;
    wk.start(a, sh, rg);
    auto tiles_of = [&]() { return wk.r.n - wk.k * sh.tok > tpt ? 2 : 1; };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 8 && lane == 0) {
            // ---- copies
            const uint32_t half_q = (uint32_t)(a.G * tpt) * 128u;
            uint32_t n = 0, u = 0;  // ring slots filled, units
            bool ok = true;
            uint32_t blocks = 0;
            for (; ok && wk.live(); wk.next(a, sh), ++u) {
                if (!mbar_wait(&q_empty, (u & 1u) ^ 1u, a.err)) break;
                const int two = tiles_of();
                mbar_expect_tx(&q_full, 2u * half_q * two);
                for (int t = 0; t < two; ++t)
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(&q_map, &q_full, q_s + t * kQTile + h * kHalf, h * 64, wk.g * a.G,
                                    wk.r.row0 + wk.k * sh.tok + t * tpt);
                const int32_t* pt = a.page_table + (size_t)wk.b * a.max_pages;
                for (int blk = wk.blk0; ok && blk < wk.blk1; ++blk, ++blocks) {
                    const int key0 = blk * kKeys;
                    const int np = (min(kKeys, wk.r.kv - key0) + a.S - 1) / a.S;  // pages (<= 0: none)
                    int page[kKeys / 16];
                    uint32_t bad = 0;
                    int good = 0;
#pragma unroll
                    for (int p = 0; p < kKeys / 16; ++p) {
                        if (p < np) {
                            page[p] = pt[key0 / a.S + p];
                            if (page[p] < 0 || page[p] >= a.n_pages) {
                                raise_err(a.err, FOCUS_DEVERR_PAGE_ID);
                                bad |= ((1u << (a.S / 16)) - 1u) << (p * (a.S / 16));
                                page[p] = -1;
                            } else {
                                ++good;
                            }
                        }
                    }
                    bad_s[blocks % kFlags] = bad;
                    for (int kv = 0; kv < 2; ++kv, ++n) {
                        const uint32_t st = n % kSlots;
                        if (!mbar_wait(&kv_empty[st], ((n / kSlots) & 1u) ^ 1u, a.err)) {
                            ok = false;
                            break;
                        }
                        mbar_expect_tx(&kv_full[st], (uint32_t)(good * a.S) * 256u);
                        uint8_t* dst = ring + st * kSlot;
#pragma unroll
                        for (int p = 0; p < kKeys / 16; ++p) {
                            if (p < np && page[p] >= 0) {
                                const int row = (int)(((((long long)page[p] * a.L + a.layer) * 2 + kv) * a.Hkv + wk.g) * a.S);
                                tma_load_2d(&pool_map, &kv_full[st], dst + p * a.S * 128, 0, row);
                                tma_load_2d(&pool_map, &kv_full[st], dst + kHalf + p * a.S * 128, 64, row);
                            }
                        }
                    }
                }
            }
            // never leave with copies in flight
            if (u > 0) mbar_wait(&q_full, (u - 1) & 1u, a.err);
            for (uint32_t i = n > kSlots ? n - kSlots : 0; i < n; ++i) mbar_wait(&kv_full[i % kSlots], (i / kSlots) & 1u, a.err);
        } else if (warp == 9 && lane == 0) {
            // ---- MMAs
            constexpr uint32_t idesc_s = idesc_bf16(128, 128);
            constexpr uint32_t idesc_o = idesc_bf16(128, 128) | (1u << 16);  // V MN-major
            const uint32_t q_addr = smem_u32(q_s), ring_addr = smem_u32(ring);
            uint32_t n = 0, u = 0, pc[2] = {0, 0};  // ring slot of the unit's next K, units, P phases
            bool ok = true;
            auto scores = [&](int t, uint32_t slot) {
                const uint32_t qa = q_addr + (uint32_t)t * kQTile, ka = ring_addr + slot * kSlot;
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk) {
                    const uint32_t off = (uint32_t)((kk >> 2) * kHalf + (kk & 3) * 32);
                    mma_bf16(tmem + (uint32_t)t * 128u, smem_desc_sw128(qa + off), smem_desc_sw128(ka + off), idesc_s,
                             kk > 0 ? 1u : 0u);
                }
                mma_commit(&s_full[t]);
            };
            auto full = [&](uint32_t i) { return mbar_wait(&kv_full[i % kSlots], (i / kSlots) & 1u, a.err); };
            for (; ok && wk.live(); wk.next(a, sh), ++u) {
                const int two = tiles_of(), nb = wk.blk1 - wk.blk0;
                if (!mbar_wait(&q_full, u & 1u, a.err) || !full(n)) break;
                tc_fence_after();
                for (int t = 0; t < two; ++t) scores(t, n % kSlots);
                mma_commit(&kv_empty[n % kSlots]);
                if (nb == 1) mma_commit(&q_empty);
                for (int i = 0; ok && i < nb; ++i) {
                    const uint32_t vs = n + 2 * i + 1, kn = n + 2 * i + 2;
                    if (!full(vs)) {
                        ok = false;
                        break;
                    }
                    for (int t = 0; t < two; ++t) {
                        if (!mbar_wait(&p_full[t], pc[t] & 1u, a.err)) {
                            ok = false;
                            break;
                        }
                        ++pc[t];
                        tc_fence_after();
                        const uint32_t va = ring_addr + (vs % kSlots) * kSlot;
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            mma_bf16_ts(tmem + 256u + (uint32_t)t * 128u, tmem + (uint32_t)t * 128u + kk * 8,
                                        v_desc(va + kk * 2048), idesc_o, (i > 0 || kk > 0) ? 1u : 0u);
                        if (i + 1 < nb) {
                            if (t == 0 && !full(kn)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            scores(t, kn % kSlots);
                        } else {
                            mma_commit(&o_full[t]);
                        }
                    }
                    if (!ok) break;
                    if (i + 1 < nb) mma_commit(&kv_empty[kn % kSlots]);
                    mma_commit(&kv_empty[vs % kSlots]);
                    if (i + 2 == nb) mma_commit(&q_empty);  // the unit's last scores have been issued
                }
                n += 2 * nb;
            }
            mma_commit(&done_bar);
            mbar_wait(&done_bar, 0u, a.err);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ---- softmax and output of tile t
        const int t = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_addr = lane_base + (uint32_t)t * 128u, o_addr = lane_base + 256u + (uint32_t)t * 128u;
        const float sl2 = a.scale * 1.4426950408889634f;
        uint32_t n = 0, blocks = 0, sc = 0, units = 0;  // ring slots, blocks, S phases, units of this tile
        bool alive = true;
        for (; wk.live(); wk.next(a, sh)) {
            const int nb = wk.blk1 - wk.blk0;
            const int tok0 = wk.k * sh.tok + t * tpt;             // the tile's first token
            const int nrow = min(tpt, wk.r.n - tok0) * a.G;
            if (nrow <= 0) {  // only tile 1, the same decision as tiles_of()
                n += 2 * nb;
                blocks += nb;
                continue;
            }
            const int pos0 = wk.r.kv - wk.r.n + tok0, rt = r / a.G;
            const int lim0 = chunk_visible(pos0, wk.r.kv, a.mask_block);  // the fewest keys a row of the tile sees
            const int lim = chunk_visible(pos0 + rt, wk.r.kv, a.mask_block);
            float m = -CUDART_INF_F, l = 0.f;
            for (int i = 0; i < nb; ++i, n += 2, ++blocks) {
                const int key0 = (wk.blk0 + i) * kKeys;
                alive = alive && mbar_wait(&s_full[t], sc & 1u, a.err);
                ++sc;
                alive = __all_sync(0xffffffffu, alive);
                if (!alive) continue;
                tc_fence_after();
                uint32_t s[128];
                float mx0 = -CUDART_INF_F, mx1 = -CUDART_INF_F, mx2 = -CUDART_INF_F, mx3 = -CUDART_INF_F;
                const uint32_t bad = bad_s[blocks % kFlags];
                const bool masked = key0 + kKeys > lim0 || bad != 0;  // the same for the whole tile
                tm_ld(s_addr, s);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tm_wait(s + 32 * c);
                    if (c < 3) tm_ld(s_addr + 32 * (c + 1), s + 32 * (c + 1));
                    if (masked) {
                        const int left = lim - key0 - 32 * c;
                        const uint32_t b2 = bad >> (2 * c);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= left || ((b2 >> (j >> 4)) & 1u)) s[32 * c + j] = __float_as_uint(-CUDART_INF_F);
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        mx0 = fmaxf(fmaxf(mx0, __uint_as_float(s[32 * c + j])), __uint_as_float(s[32 * c + j + 1]));
                        mx1 = fmaxf(fmaxf(mx1, __uint_as_float(s[32 * c + j + 2])), __uint_as_float(s[32 * c + j + 3]));
                        mx2 = fmaxf(fmaxf(mx2, __uint_as_float(s[32 * c + j + 4])), __uint_as_float(s[32 * c + j + 5]));
                        mx3 = fmaxf(fmaxf(mx3, __uint_as_float(s[32 * c + j + 6])), __uint_as_float(s[32 * c + j + 7]));
                    }
                }
                const float cm = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sl2;
                float f = 1.f;
                if (m == -CUDART_INF_F) {
                    m = cm;  // no weight has been summed yet: O is zero or not yet written
                } else if (cm > m + kRaise) {
                    f = ex2(m - cm);
                    l *= f;
                    m = cm;
                }
                if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < kD; c += 32) {
                        float v[32];
                        tmem_ld32(o_addr + c, v);
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(v[j] * f);
                        tm_st(o_addr + c, w);
                    }
                    tm_wait_st();
                }
                const float mu = m == -CUDART_INF_F ? 0.f : m;
                float l0 = 0.f, l1 = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t pk[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float p0 = ex2(fmaf(__uint_as_float(s[64 * h + 2 * j]), sl2, -mu));
                        const float p1 = ex2(fmaf(__uint_as_float(s[64 * h + 2 * j + 1]), sl2, -mu));
                        l0 += p0;
                        l1 += p1;
                        pk[j] = pack2(p0, p1);
                    }
                    tm_st(s_addr + 32 * h, pk);
                }
                l += l0 + l1;
                // V rows of keys that do not exist may hold anything (a page's tail, an old copy): their weight
                // is 0, so make them 0 as well
                if (key0 + kKeys > wk.r.kv || bad != 0) {
                    alive = __all_sync(0xffffffffu, mbar_wait(&kv_full[(n + 1) % kSlots], ((n + 1) / kSlots) & 1u, a.err));
                    if (key0 + r >= wk.r.kv || ((bad >> (r >> 4)) & 1u)) {
                        uint8_t* vr = ring + ((n + 1) % kSlots) * kSlot + r * 128;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            *reinterpret_cast<uint4*>(vr + 16 * c) = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4*>(vr + kHalf + 16 * c) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                tm_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t]);
            }
            alive = alive && mbar_wait(&o_full[t], units & 1u, a.err);
            ++units;
            alive = __all_sync(0xffffffffu, alive);
            tc_fence_after();
            bf16* dst = reinterpret_cast<bf16*>(a.out) + (long long)(wk.r.row0 + tok0 + rt) * a.out_stride +
                        (wk.g * a.G + r - rt * a.G) * kD;
            const bool live = r < nrow;
            auto store = [&](int c, const float (&v)[32], float inv) {  // 32 columns of the row
#pragma unroll
                for (int j = 0; j < 32; j += 8)
                    *reinterpret_cast<uint4*>(dst + c + j) =
                        make_uint4(pack2(v[j] * inv, v[j + 1] * inv), pack2(v[j + 2] * inv, v[j + 3] * inv),
                                   pack2(v[j + 4] * inv, v[j + 5] * inv), pack2(v[j + 6] * inv, v[j + 7] * inv));
            };
            if (wk.whole()) {
                const float inv = l > 0.f ? 1.f / l : 0.f;
                if (alive) {
#pragma unroll 1
                    for (int c = 0; c < kD; c += 32) {
                        float v[32];
                        tmem_ld32(o_addr + c, v);
                        if (live) store(c, v, inv);
                    }
                    tc_fence_before();
                }
                continue;
            }
            // ---- a shared unit: leave the piece in scratch; the group that arrives last adds them in order
            int c0, c1;
            wk.pieces(rg, c0, c1);
            float4* po = reinterpret_cast<float4*>(a.part_o);
            float2* pm = reinterpret_cast<float2*>(a.part_ml);
            auto piece = [&](int c) { return (size_t)wk.slot(rg, c) * 2 + t; };
            const size_t mine = piece(blockIdx.x);
            if (alive) {
#pragma unroll 1
                for (int c = 0; c < kD; c += 32) {
                    float v[32];
                    tmem_ld32(o_addr + c, v);
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        __stcg(po + (mine * 32 + (c + j) / 4) * 128 + r, make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
                }
                tc_fence_before();
            }
            __stcg(pm + mine * 128 + r, make_float2(m, l));
            __threadfence();
            sync_group(t);
            if (r == 0)
                last_s[t] = atomicInc(reinterpret_cast<unsigned*>(a.counters) + 2 * c0 + t, (unsigned)(c1 - c0)) ==
                            (unsigned)(c1 - c0);
            sync_group(t);
            if (!last_s[t]) continue;
            __threadfence();
            float mm = -CUDART_INF_F, ll = 0.f;
            for (int c = c0; c <= c1; ++c) mm = fmaxf(mm, __ldcg(pm + piece(c) * 128 + r).x);
            const float mu = mm == -CUDART_INF_F ? 0.f : mm;
            for (int c = c0; c <= c1; ++c) {
                const float2 v = __ldcg(pm + piece(c) * 128 + r);
                ll = fmaf(v.y, ex2(v.x - mu), ll);
            }
            const float inv = ll > 0.f ? 1.f / ll : 0.f;
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.f;
                for (int p = c0; p <= c1; ++p) {
                    const size_t at = piece(p);
                    const float f = ex2(__ldcg(pm + at * 128 + r).x - mu);
                    if (f == 0.f) continue;  // nothing summed there (the piece's O may be unwritten)
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 o = __ldcg(po + (at * 32 + (c + j) / 4) * 128 + r);
                        v[j] = fmaf(o.x, f, v[j]);
                        v[j + 1] = fmaf(o.y, f, v[j + 1]);
                        v[j + 2] = fmaf(o.z, f, v[j + 2]);
                        v[j + 3] = fmaf(o.w, f, v[j + 3]);
                    }
                }
                if (live) store(c, v, inv);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Query rows as (64-column half, head, row): one box is G heads of 128 / G tokens, 128-byte rows, swizzled.
bool make_q_map(CUtensorMap* m, const ChunkAttnDev& a) {
    auto fn = tc::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)a.Hq, (cuuint64_t)a.rows};
    const cuuint64_t strides[2] = {(cuuint64_t)kD * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)a.G, (cuuint32_t)(128 / a.G)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool configure_chunk_attention_tile() {
    return cudaFuncSetAttribute(chunk_attn_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) ==
               cudaSuccess &&
           max_shared_carveout((const void*)chunk_attn_tile_kernel);
}

int launch_chunk_attention_tile(const ChunkAttnDev& a, int sms, cudaStream_t s) {
    CUtensorMap q_map, pool_map;
    if (!make_q_map(&q_map, a)) return -1;
    const uint64_t rows = (uint64_t)a.n_pages * a.L * 2 * a.Hkv * a.S;
    if (a.n_pages > 0) {
        if (!tc::make_map(&pool_map, a.kv_pool, rows, kD, (uint32_t)a.S)) return -1;
    } else {
        pool_map = q_map;  // never used: without pages every key is invalid
    }
    const dim3 grid(sms < kChunkCtas ? sms : kChunkCtas), block(kTileThreads);
    return launched(launch_pdl(chunk_attn_tile_kernel, grid, block, kSmem, s, 0, pool_map, q_map, a, 2));
}

}  // namespace focus
