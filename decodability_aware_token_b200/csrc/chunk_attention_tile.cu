// bf16 attention of a chunk over the paged cache on the 5th-generation tensor cores: requests with more
// than kChunkFewRows query vectors per KV head (prompt chunks).  See chunk_work.cuh for how the key walks
// are split over the CTAs.
//
// Unit: request b, KV head g and up to 256 query vectors (token r / G, head r % G) in two tiles of up to
// 128.  Keys come in blocks of 64 through rings of four K and five V slots of 16 KB, each filled from
// whole pages by TMA (two 64-column halves, 128-byte swizzle).  Per tile t and block i:
//   S_t = Q_t K_i^T     tcgen05.mma 128 x 64 x 128, both operands in shared memory, into one of the tile's two
//                       S buffers in TMEM
//   softmax             one warpgroup per tile, one thread per query vector: the 64 scores from TMEM, reference m
//                       and denominator in registers, P = 2^(s - m) as bf16 back into TMEM over S_t
//   O_t += P_t V_i      tcgen05.mma 128 x 128 x 64, P from TMEM, V MN-major straight from the page tile
// One warp per tile issues its MMAs, S_t(i + 2) behind P V_t(i): the next block's scores are there when the
// softmax has finished with this one, and while one tile is in its softmax the tensor core works for the other.
// TMEM: two S buffers of 64 columns per tile, O_0, O_1 of 128, all 512 columns.
//
// softmax(s) does not change with the reference that is subtracted, so m only has to keep 2^(s - m) in range: it
// is the first visible block's maximum, and it is raised to the running one (O and the denominator rescaled in TMEM and
// registers, the block's weights computed again) when a block's weights sum to more than 2^40.  That takes the
// 64-step maximum out of most blocks.  2^24 blocks of at most 2^40 sum to 2^64, which leaves O in range for |V| < 2^64.
// P is rounded to bf16, the type of the values it multiplies (off by at most 2^-8 of a weight); the denominator
// sums the unrounded weights in float32.
//
// Bound by the tensor core and the softmax side by side: a pair of blocks keeps the tensor core for 1360 cycles (S at
// 52 a K step of 16, its operands read from shared memory as fast as that goes, P V at 66) and the exponential unit
// for 1062 of the 1800 that it takes.  Measured over seconds, at the clock where the card's power management
// holds it: the 8192-token prompt (16/8 heads) 308 us at 1.79 GHz, 892 TFLOP/s (287 in short runs; 316 and 323 on other
// cards); two chunks of 1024 tokens over 65000 cached, 32/8 heads, 2519 us at 1.43 GHz, 878 TFLOP/s.  In short runs,
// when the prompt took 290, leaving out the MMAs left 265, leaving out the softmax's arithmetic 283, and leaving out both,
// which is the copies out of L2, 205.
// Why this shape (short runs): with 128 keys a block only one S buffer per tile fits in TMEM, and the prompt took 368 us; with
// one MMA warp for both tiles and one S buffer 347 us; with two threads per query vector (16 softmax warps) 325 against
// 290; with the two tiles' exponentials kept half a block apart 302.
//
// Every mbarrier wait is bounded; on expiry the role flags FOCUS_DEVERR_TIMEOUT and stops issuing, copies and
// MMAs in flight are waited for (bounded), and TMEM is released.
#include <math_constants.h>

#include "chunk_pipe.cuh"

namespace focus {
namespace {

using tc::idesc_bf16;
using tc::smem_desc_sw128;
using tc::tc_fence_after;
using tc::tc_fence_before;
using tc::tmem_ld32;

constexpr int kD = 128;
constexpr int kKeys = 64;                     // keys per block
constexpr int kHalf = kKeys * 128;            // [64 keys][64 columns] bf16: 8 KB
constexpr int kSlot = 2 * kHalf;              // K or V of one block: 16 KB
constexpr int kKSlots = 4, kVSlots = 5;       // K is used two blocks ahead of V, V a block longer
constexpr int kUnits = 4;                     // unit descriptors in flight
constexpr int kQHalf = 128 * 128;             // [128 query vectors][64 columns]
constexpr int kQTile = 2 * kQHalf;            // one query tile: 32 KB
constexpr int kTurn = 32 * 64;                // bytes a warp turns its output in: 32 rows of 32 columns
constexpr int kSmem = 2 * kQTile + (kKSlots + kVSlots) * kSlot + 8 * kTurn + 1024;
constexpr int kSoftWarps = 8;                 // 4 per tile: one thread per query vector
constexpr int kTileThreads = 32 * kSoftWarps + 128;  // then two warps for the copies and one per tile for the MMAs
constexpr int kCopyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1, kCopyVWarp = kSoftWarps + 3;  // MMAs of tile t: kMmaWarp + t
constexpr int kFlags = 16;                    // bad-page flags, one per block in flight
constexpr float kRaise = 1099511627776.f;     // 2^40
static_assert(kSmem <= 226 * 1024 - 512, "shared memory");
static_assert(kChunkMaxRequests * 8 <= (kKSlots + kVSlots) * kSlot, "the schedule's sums fit in the ring");

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// The MMA warp runs its loop with all lanes and one elected lane issues: loop counters and descriptors stay
// uniform, which the issue needs (a loop inside `if (lane == 0)` issued one MMA per 85 cycles, slower than
// the 64 that one takes).
__device__ __forceinline__ void mma_ss(uint32_t elected, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(elected));
}
// A (the weights) in TMEM, B in shared memory
__device__ __forceinline__ void mma_ts(uint32_t elected, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc), "r"(elected));
}
__device__ __forceinline__ void commit_one(uint32_t elected, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n"
        ::"r"(smem_u32(bar)), "r"(elected)
        : "memory");
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
// two float32 in one 64-bit register: the FMA pipe takes both in one instruction
__device__ __forceinline__ uint64_t f2(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ uint64_t f2(float lo, float hi) { return f2(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    return d;
}
__device__ __forceinline__ uint64_t exp2_2(uint64_t x) {
    return f2(ex2(__uint_as_float((uint32_t)x)), ex2(__uint_as_float((uint32_t)(x >> 32))));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// The four warps of tile t meet at named barrier 1 + t.
__device__ __forceinline__ void sync_tile(int t) { named_sync<128>(1 + t); }

// Registers by role: 384 threads start with 168 each (64512); the softmax warps hold a row's 64 scores and weights, the
// last warpgroup (copies, MMAs) needs few: 256 x 208 + 128 x 88 = 64512.
constexpr int kSoftRegs = 208, kIssueRegs = 88;
static_assert(32 * kSoftWarps * kSoftRegs + 128 * kIssueRegs <= kTileThreads * 168, "register split");

__global__ void __launch_bounds__(kTileThreads, 1)
chunk_attn_tile_kernel(const __grid_constant__ CUtensorMap pool_map, const __grid_constant__ CUtensorMap q_map,
                       ChunkAttnDev a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* q_s = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* k_ring = q_s + 2 * kQTile;
    uint8_t* v_ring = k_ring + kKSlots * kSlot;
    uint8_t* turn_s = v_ring + kVSlots * kSlot;  // [softmax warp][kTurn]
    __shared__ __align__(8) uint64_t q_full, q_empty, k_full[kKSlots], k_empty[kKSlots], v_full[kVSlots],
        v_empty[kVSlots], s_full[2][2],
        p_full[2][2], o_full[2][2], done_bar[2], u_full[kUnits], u_empty[kUnits];
    __shared__ UnitDesc unit_s[kUnits];
    __shared__ uint32_t bad_s[kFlags];  // per block: 16-key groups whose page id is invalid
    __shared__ uint32_t tmem_slot;
    __shared__ ChunkRange rg;
    __shared__ long long red[32];
    __shared__ int last_s[2];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 2);  // both tiles' MMA warps
        for (int s = 0; s < kKSlots; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 2);
        }
        for (int s = 0; s < kVSlots; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 2);
        }
        for (int t = 0; t < 2; ++t) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(&s_full[t][b], 1);
                mbar_init(&p_full[t][b], 4);  // one arrival per softmax warp
                mbar_init(&o_full[t][b], 1);  // P V of even / odd blocks complete
            }
            mbar_init(&done_bar[t], 1);
        }
        for (int s = 0; s < kUnits; ++s) {
            mbar_init(&u_full[s], 1);
            mbar_init(&u_empty[s], 3 + kSoftWarps);  // the V copies, the MMA and the softmax warps
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == kCopyWarp && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&pool_map) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&q_map) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (!a.pair) pdl_wait();  // (and no early trigger: norm and rotation, then the 8192-token prompt, repeated: 373 us -> 360)

    const int tpt = 128 / a.G;  // tokens per tile
    // The copies leave the query rows past G tokens' heads alone; whatever is there would send its warp through the
    // recomputation below in every block, so make them zero.
    const int dead = 128 - a.G * tpt;
    for (int i = threadIdx.x; i < 4 * dead * 8; i += kTileThreads)
        *reinterpret_cast<uint4*>(q_s + i / (dead * 8) * kQHalf + a.G * tpt * 128 + i % (dead * 8) * 16) = make_uint4(0, 0, 0, 0);
    const ChunkShape sh{2 * tpt, a.G <= kChunkFewRows ? kChunkFewRows : 0, 0x7fffffff};
    chunk_schedule<kKeys, 4>(a, sh, reinterpret_cast<long long*>(k_ring), red, &rg);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the rings held the schedule's sums (and the zeros)
    __syncthreads();

    // the copy thread walks the range; the others read what it has found
    auto unit_wait = [&](uint32_t u) { return warp_wait(&u_full[u % kUnits], (u / kUnits) & 1u, a.err); };

    if (warp >= kSoftWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == kCopyWarp || warp == kCopyVWarp) {
            // ---- copies: one warp walks the range and fetches Q and K, the other follows it and fetches V
            const bool is_k = warp == kCopyWarp;
            const int kv = is_k ? 0 : 1, slots = is_k ? kKSlots : kVSlots, ppb = kKeys / a.S;
            uint8_t* ring = is_k ? k_ring : v_ring;
            uint64_t *full = is_k ? k_full : v_full, *empty = is_k ? k_empty : v_empty;
            const uint32_t el = elect_one(), half_q = (uint32_t)(a.G * tpt) * 128u;
            uint32_t n = 0, u = 0;  // blocks copied, units
            int st = 0;             // n % slots
            uint32_t turn = 0;      // n / slots
            bool ok = true;
            PageWalk pw;
            auto blocks_of = [&](int g, int blk0, int nb) {
                for (int i = 0; ok && i < nb; ++i, ++n, pw.at += ppb) {
                    int page;
                    uint32_t bad;
                    const int good = pw.block(a, ppb, page, bad);
                    ok = warp_wait(&empty[st], (turn & 1u) ^ 1u, a.err);
                    if (!ok) break;
                    if (el) {
                        if (is_k) {
                            if (bad) raise_err(a.err, FOCUS_DEVERR_PAGE_ID);
                            bad_s[n % kFlags] = bad;
                        }
                        mbar_expect_tx(&full[st], (uint32_t)(good * a.S) * 256u);
                    }
                    __syncwarp();
                    if (page >= 0) {
                        uint8_t* dst = ring + st * kSlot + lane * a.S * 128;
                        const int x = (int)(((long long)page * a.L + a.layer) * 2 * a.Hkv) + g;
                        // (the map's box holds both column halves when a page is a whole block)
                        tma_load_pool(&pool_map, &full[st], dst, 0, kv, x);
                        if (a.S < kKeys) tma_load_pool(&pool_map, &full[st], dst + kHalf, 1, kv, x);
                    }
                    __syncwarp();
                    if (++st == slots) st = 0, ++turn;
                }
            };
            if (is_k) {
                ChunkWalk<kKeys> wk;
                uint32_t d = 0;
                auto publish = [&](bool live) {
                    if (!warp_wait(&u_empty[d % kUnits], ((d / kUnits) & 1u) ^ 1u, a.err)) return false;
                    if (lane == 0) {
                        describe(unit_s[d % kUnits], wk, rg, sh, live);
                        mbar_arrive(&u_full[d % kUnits]);
                    }
                    __syncwarp();
                    ++d;
                    return true;
                };
                for (wk.start(a, sh, rg); ok && wk.live(); wk.next(a, sh)) {
                    pw.start(a, wk.b, wk.r.kv, wk.blk0 * ppb);
                    ok = publish(true) && warp_wait(&q_empty, (u & 1u) ^ 1u, a.err);
                    if (!ok) break;
                    const int two = wk.r.n - wk.k * sh.tok > tpt ? 2 : 1;
                    if (el) {
                        mbar_expect_tx(&q_full, 2u * half_q * two);
                        for (int t = 0; t < two; ++t)
                            for (int h = 0; h < 2; ++h)
                                tma_load_3d(&q_map, &q_full, q_s + t * kQTile + h * kQHalf, h * 64, wk.g * a.G,
                                            wk.r.row0 + wk.k * sh.tok + t * tpt);
                    }
                    __syncwarp();
                    ++u;
                    blocks_of(wk.g, wk.blk0, wk.blk1 - wk.blk0);
                }
                if (ok) publish(false);
                if (u > 0) warp_wait(&q_full, (u - 1) & 1u, a.err);
            } else {
                for (; ok; ++u) {
                    ok = unit_wait(u);
                    if (!ok) break;
                    const UnitDesc& ud = unit_s[u % kUnits];
                    const int b = ud.b, g = ud.g, len = ud.kv, blk0 = ud.blk0, nb = ud.nb;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&u_empty[u % kUnits]);
                    if (nb == 0) break;
                    pw.start(a, b, len, blk0 * ppb);
                    blocks_of(g, blk0, nb);
                }
            }
            // never leave with copies in flight
            for (uint32_t i = n > (uint32_t)slots ? n - slots : 0; i < n; ++i) warp_wait(&full[i % slots], (i / slots) & 1u, a.err);
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ---- MMAs of tile t: S(j + 2) goes out behind P V(j), so the scores of the next block are ready when the
            // softmax has finished this one.  (One warp for both tiles left the tensor core idle while it waited
            // and committed for the other tile.)
            const int t = warp - kMmaWarp;
            constexpr uint32_t idesc_s = idesc_bf16(128, kKeys);
            constexpr uint32_t idesc_o = idesc_bf16(128, kD) | (1u << 16);  // V MN-major
            const uint32_t el = elect_one();
            const uint64_t q_desc = smem_desc_sw128(smem_u32(q_s + t * kQTile)), k_desc = smem_desc_sw128(smem_u32(k_ring)),
                           val_desc = v_desc(smem_u32(v_ring));
            const uint32_t s_col = tmem + (uint32_t)t * 128u, o_col = tmem + 256u + (uint32_t)t * 128u;
            // K blocks used and V blocks used (slot and turn of the ring), blocks of S and of P
            uint32_t ks = 0, kt = 0, vs = 0, vt = 0, sc = 0, pc = 0;
            auto next_k = [&]() {
                if (++ks == kKSlots) ks = 0, ++kt;
            };
            auto next_v = [&]() {
                if (++vs == kVSlots) vs = 0, ++vt;
            };
            // descriptors count 16-byte units
            auto scores = [&]() {
                const uint64_t kd = k_desc + (uint64_t)(ks * (kSlot >> 4));
                const uint32_t d = s_col + (sc & 1u) * 64u;
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk)
                    mma_ss(el, d, q_desc + (uint64_t)(((kk >> 2) * kQHalf + (kk & 3) * 32) >> 4),
                           kd + (uint64_t)(((kk >> 2) * kHalf + (kk & 3) * 32) >> 4), idesc_s, kk > 0 ? 1u : 0u);
                commit_one(el, &s_full[t][sc & 1u]);
                commit_one(el, &k_empty[ks]);
                ++sc;
                next_k();
            };
            auto k_here = [&]() { return warp_wait(&k_full[ks], kt & 1u, a.err); };
            auto v_here = [&]() { return warp_wait(&v_full[vs], vt & 1u, a.err); };
            bool ok = true;
            for (uint32_t u = 0; ok; ++u) {
                if (!unit_wait(u)) break;
                const int nb = unit_s[u % kUnits].nb;
                const bool mine = t == 0 || unit_s[u % kUnits].n - unit_s[u % kUnits].tok0 > tpt;
                __syncwarp();
                if (el) mbar_arrive(&u_empty[u % kUnits]);
                if (nb == 0) break;
                if (!mine) {
                    // a short unit's second tile: give the queries and the ring slots back as they come (waiting for
                    // each, since a parity wait must not be two phases ahead)
                    if (!warp_wait(&q_full, u & 1u, a.err)) break;
                    __syncwarp();
                    if (el) mbar_arrive(&q_empty);
                    for (int j = 0; ok && j < nb; ++j) {
                        ok = k_here() && v_here();
                        __syncwarp();
                        if (ok && el) {
                            mbar_arrive(&k_empty[ks]);
                            mbar_arrive(&v_empty[vs]);
                        }
                        next_k();
                        next_v();
                    }
                    continue;
                }
                if (!warp_wait(&q_full, u & 1u, a.err)) break;
                for (int j = 0; ok && j < 2 && j < nb; ++j) {
                    ok = k_here();
                    if (!ok) break;
                    tc_fence_after();
                    scores();
                }
                if (nb <= 2) commit_one(el, &q_empty);
                for (int j = 0; ok && j < nb; ++j) {
                    const uint32_t b = pc & 1u;
                    ok = v_here() && warp_wait(&p_full[t][b], (pc >> 1) & 1u, a.err);
                    if (!ok) break;
                    ++pc;
                    tc_fence_after();
                    const uint64_t vd = val_desc + (uint64_t)(vs * (kSlot >> 4));
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        mma_ts(el, o_col, s_col + b * 64u + kk * 8, vd + (uint64_t)(kk * (2048 >> 4)), idesc_o,
                               (j > 0 || kk > 0) ? 1u : 0u);
                    commit_one(el, &o_full[t][b]);
                    commit_one(el, &v_empty[vs]);
                    next_v();
                    if (j + 2 < nb) {
                        // (only when P V is done: MMAs issued into a full queue hold up the softmax warp of this SM
                        // quarter; 8192-token prompt 297 -> 290 us)
                        ok = k_here() && warp_wait(&o_full[t][b], ((pc - 1) >> 1) & 1u, a.err);
                        if (!ok) break;
                        tc_fence_after();
                        scores();
                    }
                    if (j + 3 == nb) commit_one(el, &q_empty);  // the unit's last scores have been issued
                }
            }
            commit_one(el, &done_bar[t]);
            warp_wait(&done_bar[t], 0u, a.err);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // ---- softmax and output of tile t, one thread per query vector
        const int t = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_addr = lane_base + (uint32_t)(t * 128), o_addr = lane_base + 256u + (uint32_t)(t * 128);
        const float sl2 = a.scale * 1.4426950408889634f;
        uint32_t blocks = 0, sc = 0;  // blocks (V of block j is in V slot j), blocks of this tile
        bool alive = true;
        // P V of this tile's block j is complete.  Asked for the last block whose P has been handed over, or the one
        // before it: each of the two barriers is then at this phase or has just left it (the P V two blocks back is
        // complete, since the scores issued behind it have arrived), so the parity is unambiguous.
        auto o_wait = [&](uint32_t j) { return warp_wait(&o_full[t][j & 1u], (j >> 1) & 1u, a.err); };
        for (uint32_t u = 0;; ++u) {
            // the tile's warps go on or stop together: a wait that gave up in one of them alone would leave the
            // others at a named barrier
            if (!all_agree<128>(1 + t, unit_wait(u))) break;
            const UnitDesc& ud = unit_s[u % kUnits];
            const int nb = ud.nb;
            if (nb == 0) break;
            const int tok0 = ud.tok0 + t * tpt;                   // the tile's first token
            const int nrow = min(tpt, ud.n - tok0) * a.G;
            auto unit_done = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(&u_empty[u % kUnits]);
            };
            if (nrow <= 0) {  // only tile 1 of a short unit
                blocks += nb;
                unit_done();
                continue;
            }
            const int kv = ud.kv, rt = r / a.G;
            const int lim0 = chunk_visible(kv - ud.n + tok0, kv, a.mask_block);  // the fewest keys a row of the tile sees
            const int lim = chunk_visible(kv - ud.n + tok0 + rt, kv, a.mask_block);
            int key0 = ud.blk0 * kKeys;
            float m = -CUDART_INF_F, l = 0.f;
            for (int i = 0; i < nb; ++i, ++blocks, key0 += kKeys) {
                const uint32_t b = sc & 1u;
                alive = alive && warp_wait(&s_full[t][b], (sc >> 1) & 1u, a.err);
                ++sc;
                if (!alive) continue;
                tc_fence_after();
                uint32_t s[64];
                const uint32_t sb = s_addr + 64 * b;
                const uint32_t bad = bad_s[blocks % kFlags];
                tm_ld(sb, s);
                tm_ld(sb + 32, s + 32);
                tm_wait(s);       // waits for both,
                tm_wait(s + 32);  // this one ties the registers
                if (key0 + kKeys > lim0 || bad != 0) {  // the same for the whole tile
                    const int left = lim - key0;
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (j >= left || ((bad >> (j >> 4)) & 1u)) s[j] = __float_as_uint(-CUDART_INF_F);
                }
                // V rows of keys that do not exist may hold anything (a page's tail, an old copy): their weight
                // is 0, so make them 0 as well
                if (key0 + kKeys > kv || bad != 0) {
                    const uint32_t vs = blocks % kVSlots;
                    alive = warp_wait(&v_full[vs], (blocks / kVSlots) & 1u, a.err);
                    const int key = r & 63;
                    if (key0 + key >= kv || ((bad >> (key >> 4)) & 1u)) {
                        uint8_t* vr = v_ring + vs * kSlot + (r >> 6) * kHalf + key * 128;
#pragma unroll
                        for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vr + 16 * c) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                const uint64_t sl2x2 = f2(sl2, sl2);
                uint32_t pk[32];
                float bsum;
                auto weights = [&]() {
                    const float mu = m == -CUDART_INF_F ? 0.f : m;
                    const uint64_t mux2 = f2(-mu, -mu);
                    uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const uint64_t x = exp2_2(fma2(f2(s[2 * j], s[2 * j + 1]), sl2x2, mux2));
                        if (j & 1) sum1 = add2(sum1, x);
                        else sum0 = add2(sum0, x);
                        pk[j] = pack2(__uint_as_float((uint32_t)x), __uint_as_float((uint32_t)(x >> 32)));
                    }
                    const uint64_t sum = add2(sum0, sum1);
                    bsum = __uint_as_float((uint32_t)sum) + __uint_as_float((uint32_t)(sum >> 32));
                };
                if (i > 0) weights();
                // The reference m only has to keep the weights in range: it is set by the first keys a row sees and
                // raised when a block's weights sum to more than 2^40 (they are then computed again), by the rows
                // that need it alone: what a row gets does not depend on its neighbours.
                if (i == 0 || __any_sync(0xffffffffu, m == -CUDART_INF_F || !(bsum <= kRaise))) {
                    const bool need = i == 0 || m == -CUDART_INF_F || !(bsum <= kRaise);
                    float cm = -CUDART_INF_F;
#pragma unroll
                    for (int j = 0; j < 64; ++j) cm = fmaxf(cm, __uint_as_float(s[j]));
                    cm *= sl2;
                    float f = 1.f;
                    if (!need) {
                        // (its weights come out as they were)
                    } else if (m == -CUDART_INF_F) {
                        m = cm;  // no weight has been summed yet: O is zero or not yet written
                    } else if (cm > m) {
                        f = ex2(m - cm);
                        l *= f;
                        m = cm;
                    }
                    if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
                        // O has to hold the previous block's P V
                        alive = o_wait(sc - 2);
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < kD; c += 32) {
                            uint32_t w[32];
                            tm_ld(o_addr + c, w);
                            tm_wait(w);
#pragma unroll
                            for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * f);
                            tm_st(o_addr + c, w);
                        }
                        tm_wait_st();
                    }
                    weights();
                }
                l += bsum;
                tm_st(sb, pk);
                tm_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[t][b]);
            }
            alive = alive && o_wait(sc - 1);
            tc_fence_after();
            // A lane's row of 32 columns goes through shared memory, so that four lanes write 64 bytes of a row and a
            // store touches 8 rows, not 32 (16-byte pieces of 32 rows cost the store path four times as long)
            const int rq = quarter * 32 + (lane >> 2);  // first of the four rows, 8 apart, this lane writes
            bf16* dst[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int rr = rq + 8 * i, tok = rr / a.G;
                dst[i] = reinterpret_cast<bf16*>(a.out) + (long long)(ud.row0 + tok0 + tok) * a.out_stride +
                         (ud.g * a.G + rr - tok * a.G) * kD + (lane & 3) * 8;
            }
            uint8_t* turn = turn_s + warp * kTurn;
            auto store = [&](int c, const float (&v)[32], float inv) {  // columns c .. c + 31 of the warp's rows
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4*>(turn + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                        make_uint4(pack2(v[8 * j] * inv, v[8 * j + 1] * inv), pack2(v[8 * j + 2] * inv, v[8 * j + 3] * inv),
                                   pack2(v[8 * j + 4] * inv, v[8 * j + 5] * inv), pack2(v[8 * j + 6] * inv, v[8 * j + 7] * inv));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 8 * i + (lane >> 2);
                    const uint4 x = *reinterpret_cast<const uint4*>(turn + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
                    if (rq + 8 * i < nrow) *reinterpret_cast<uint4*>(dst[i] + c) = x;
                }
                __syncwarp();
            };
            const int c0 = ud.c0, c1 = ud.c1, slot0 = ud.slot0;
            unit_done();
            if (c0 < 0) {
                const float inv = l > 0.f ? 1.f / l : 0.f;
                if (alive) {
#pragma unroll 1
                    for (int c = 0; c < kD; c += 32) {
                        float v[32];
                        tmem_ld32(o_addr + c, v);
                        store(c, v, inv);
                    }
                    tc_fence_before();
                }
                continue;
            }
            // ---- a shared unit: leave the piece in scratch; the group that arrives last adds them in order
            float4* po = reinterpret_cast<float4*>(a.part_o);
            float2* pm = reinterpret_cast<float2*>(a.part_ml);
            auto piece = [&](int c) { return (size_t)(c == c0 ? slot0 : 2 * c) * 2 + t; };
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
            // (a row whose scores are all NaN has no maximum; a NaN there keeps its piece from being skipped as empty)
            __stcg(pm + mine * 128 + r, make_float2(l == l ? m : l, l));
            __threadfence();
            sync_tile(t);
            if (r == 0)
                last_s[t] = atomicInc(reinterpret_cast<unsigned*>(a.counters) + 2 * c0 + t, (unsigned)(c1 - c0)) ==
                            (unsigned)(c1 - c0);
            sync_tile(t);
            if (!last_s[t]) continue;
            __threadfence();
            // (loads of several pieces in flight: a piece is a trip to L2, and this is the end of the CTA's work)
            float mm = -CUDART_INF_F, ll = 0.f;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
                const float2 x = __ldcg(pm + piece(c) * 128 + r);
                const float m1 = fmaxf(mm, x.x), mu = m1 == -CUDART_INF_F ? 0.f : m1;
                ll = fmaf(x.y, ex2(x.x - mu), ll * ex2(mm - mu));
                mm = m1;
            }
            const float mu = mm == -CUDART_INF_F ? 0.f : mm;
            const float inv = ll > 0.f ? 1.f / ll : 0.f;
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.f;
#pragma unroll 2
                for (int p = c0; p <= c1; ++p) {
                    const size_t at = piece(p);
                    const float f = ex2(__ldcg(pm + at * 128 + r).x - mu);
                    float4 o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = __ldcg(po + (at * 32 + c / 4 + j) * 128 + r);
                    const bool none = f == 0.f;  // nothing summed there: the piece's O may be unwritten
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        v[4 * j] = none ? v[4 * j] : fmaf(o[j].x, f, v[4 * j]);
                        v[4 * j + 1] = none ? v[4 * j + 1] : fmaf(o[j].y, f, v[4 * j + 1]);
                        v[4 * j + 2] = none ? v[4 * j + 2] : fmaf(o[j].z, f, v[4 * j + 2]);
                        v[4 * j + 3] = none ? v[4 * j + 3] : fmaf(o[j].w, f, v[4 * j + 3]);
                    }
                }
                store(c, v, inv);
            }
        }
    }
    if (a.pair) pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
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
    if (a.n_pages > 0) {
        if (!make_pool_map(&pool_map, a, a.S == kKeys ? 2 : 1, 1)) return -1;
    } else {
        pool_map = q_map;  // never used: without pages every key is invalid
    }
    const dim3 grid(sms < kChunkCtas ? sms : kChunkCtas), block(kTileThreads);
    return launched(launch_pdl(chunk_attn_tile_kernel, grid, block, kSmem, s, 0, pool_map, q_map, a));
}

}  // namespace focus
