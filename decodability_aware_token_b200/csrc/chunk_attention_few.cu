// bf16 attention of requests with at most kChunkFewRows query vectors per KV head (single tokens, a few
// speculative ones) over the paged cache, on mma.sync m16n8k16: with 16 rows the tensor work is a fraction of the
// copy time whatever the instruction, and fragments in registers need no TMEM round trip per block.
//
// Bound by memory: each cached key and value is read once, so the design is a copy that never stops.  One CTA
// per SM walks its equal share of the batch's key blocks (chunk_work.cuh); one warp issues the pages of 64-key
// blocks by TMA into a ring of six 32 KB stages and runs on across unit ends.  Two groups of four warps consume
// alternate units, 16 keys of a block per warp: a group keeps up with the copies, and while it joins its warps'
// results and writes them, the other one is already at the next unit.  A warp keeps its own running maximum, denominator
// and 16 x 128 output, so nothing is exchanged while a unit lasts.  Pieces of a unit that spans CTAs are joined by the
// CTA that finishes last, in block order.  Measured over seconds: 256 requests of 512 to 2048 tokens, 32/8 heads, 216 us at
// 1.81 GHz (power cap) = 5.9 TB/s, 90 % of the copy rate, 205 in short runs; 32 requests of 256 to 1024 tokens, 16/8 heads,
// 25 us at 1.97 GHz against 11.7 at that rate (start-up, unit ends and the joins of split units).
//
// Weights are rounded to bf16 for the product with V, the values' own type (off by at most 2^-8 of a weight); maxima,
// denominators and outputs are float32.  (As the sum of two bf16 each, with twice the MMAs, they bring the error against
// 64 bits from 0.0022 to 0.0017 of the outputs' scale, which is the outputs' own rounding, and 256 requests from 217 to
// 242 us, 32 from 24.6 to 26.0.)  The running maximum is raised only by more than 8 (weights up to 2^8),
// which spares most blocks the rescaling of O.
#include <math_constants.h>

#include "chunk_pipe.cuh"

namespace focus {
namespace {

constexpr int kD = 128;
constexpr int kKeys = 64;
constexpr int kUnits = 4;                    // unit descriptors in flight
constexpr int kHalf = kKeys * 128;           // [64 keys][64 columns] bf16
constexpr int kStage = 4 * kHalf;            // per page: K lo, K hi, V lo, V hi of S rows; 32 KB in all
constexpr int kStages = 6;
constexpr int kRows = kChunkFewRows;
static_assert(kRows == 16, "one m16 tile");
constexpr int kConsumers = 8;
constexpr int kGroup = 4;                    // warps that consume a unit
static_assert(kUnits % 2 == 0, "a descriptor slot belongs to one group: its waits see every phase");
constexpr int kFewThreads = 32 * (kConsumers + 1);
constexpr int kJoinF = 2 * kD;               // floats of a warp's join buffer: 2 rows
constexpr int kQRow = kD * 2 + 16;           // bytes of a query row in shared memory: rows 4 banks apart
constexpr int kQBytes = kRows * kQRow;
constexpr int kFewSmem = kStages * kStage + kConsumers * kJoinF * 4 + kUnits * kQBytes + 1024;
static_assert(kFewSmem <= 224 * 1024, "shared memory");
static_assert(kChunkMaxRequests * 8 <= kStages * kStage, "the schedule's sums fit in the ring");
constexpr float kRaise = 8.f;                // in units of log2

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

__global__ void __launch_bounds__(kFewThreads, 1)
chunk_attn_few_kernel(const __grid_constant__ CUtensorMap pool_map, ChunkAttnDev a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* join = reinterpret_cast<float*>(ring + kStages * kStage);  // [warp][2 rows][128]
    uint8_t* q_s = reinterpret_cast<uint8_t*>(join + kConsumers * kJoinF);  // [unit][16 rows][kQRow bytes]
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], u_full[kUnits], u_empty[kUnits];
    __shared__ UnitDesc unit_s[kUnits];
    __shared__ uint32_t bad_s[kStages];       // 16-key groups of the stage whose page id is invalid
    __shared__ volatile uint32_t tag_s[kStages];  // block the stage is being filled with
    __shared__ uint32_t first_s[kUnits];      // number of the unit's first block in the CTA's walk
    __shared__ ChunkRange rg;
    __shared__ long long red[32];
    __shared__ float jm[kConsumers][kRows], jl[kConsumers][kRows];
    __shared__ int last_s[2];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kGroup);
            tag_s[s] = ~0u;
        }
        for (int s = 0; s < kUnits; ++s) {
            mbar_init(&u_full[s], 1);
            mbar_init(&u_empty[s], kGroup);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&pool_map) : "memory");
    }
    pdl_wait();
    if (a.pair) pdl_trigger();  // (behind the wait: the tile kernel may rely on it)
    const ChunkShape sh{kRows / a.G, 0, kRows};
    chunk_schedule<kKeys, 2>(a, sh, reinterpret_cast<long long*>(ring), red, &rg);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring held the schedule's sums
    __syncthreads();

    if (warp == kConsumers) {
        // ---- copies: the whole warp walks, lane p issues the block's page p
        const uint32_t el = elect_one();
        const int ppb = kKeys / a.S;  // pages per block
        uint32_t n = 0, d = 0;        // stages filled, units described
        bool ok = true;
        ChunkWalk<kKeys> wk;
        // describe the unit and start its query rows on their way
        auto publish = [&](bool live) {
            const uint32_t s = d % kUnits;
            if (!warp_wait(&u_empty[s], ((d / kUnits) & 1u) ^ 1u, a.err)) return false;
            const int nrow = live ? min(sh.tok, wk.r.n - wk.k * sh.tok) * a.G : 0;
            if (lane == 0) {
                describe(unit_s[s], wk, rg, sh, live);
                first_s[s] = n;
                mbar_expect_tx(&u_full[s], (uint32_t)nrow * 256u);
            }
            __syncwarp();
            if (lane < nrow) {
                const bf16* src = reinterpret_cast<const bf16*>(a.q) +
                                  (long long)(wk.r.row0 + wk.k * sh.tok + lane / a.G) * a.q_stride + (wk.g * a.G + lane % a.G) * kD;
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                             ::"r"(smem_u32(q_s + s * kQBytes + lane * kQRow)), "l"(src), "n"(kD * 2), "r"(smem_u32(&u_full[s]))
                             : "memory");
            }
            __syncwarp();
            ++d;
            return true;
        };
        PageWalk pw;
        for (wk.start(a, sh, rg); ok && wk.live(); wk.next(a, sh)) {
            pw.start(a, wk.b, wk.r.kv, wk.blk0 * ppb);
            ok = publish(true);
            for (int blk = wk.blk0; ok && blk < wk.blk1; ++blk, ++n, pw.at += ppb) {
                const uint32_t st = n % kStages;
                int page;
                uint32_t bad;
                const int good = pw.block(a, ppb, page, bad);
                ok = warp_wait(&empty[st], ((n / kStages) & 1u) ^ 1u, a.err);
                if (!ok) break;
                if (el) {
                    if (bad) raise_err(a.err, FOCUS_DEVERR_PAGE_ID);
                    bad_s[st] = bad;
                    tag_s[st] = n;
                    mbar_expect_tx(&full[st], (uint32_t)(good * a.S) * 512u);
                }
                __syncwarp();
                if (page >= 0)
                    tma_load_pool(&pool_map, &full[st], ring + st * kStage + lane * a.S * 512, 0, 0,
                                  (int)(((long long)page * a.L + a.layer) * 2 * a.Hkv) + wk.g);
                __syncwarp();
            }
        }
        // (Not earlier, unless the tile kernel follows: the next operator's CTAs, waiting on the SMs, cost more than their
        // early launch gives.  Norm and rotation, then attention of 32 single tokens, repeated: 26.0 us -> 23.8.)
        pdl_trigger();
        if (ok && publish(false)) publish(false);  // an end for each group
        // never leave with copies in flight
        for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i) warp_wait(&full[i % kStages], (i / kStages) & 1u, a.err);
        for (uint32_t i = d > kUnits ? d - kUnits : 0; i < d; ++i) warp_wait(&u_full[i % kUnits], (i / kUnits) & 1u, a.err);
        return;
    }

    // ---- consumers: warps 0-3 take the even units of the CTA's walk, 4-7 the odd ones
    const int grp = warp / kGroup, wq = warp % kGroup, ks = wq * 16;  // this warp's 16 keys of a block
    const int g4 = lane >> 2, t4 = lane & 3;          // fragment row, column pair
    const float sl2 = a.scale * 1.4426950408889634f;
    // row / G for rows below 16
    const uint32_t g_inv = (65536u + a.G - 1) / a.G;
    auto token = [&](int r) { return (int)(((uint32_t)r * g_inv) >> 16); };
    const int tk0 = token(g4), tk1 = token(g4 + 8);
    // ldmatrix row addresses within a stage: K (keys x 32 columns a step), V transposed (16 keys x 16 columns)
    // (the warp's 16 keys lie in one page: S is a multiple of 16)
    const uint32_t key_off = (uint32_t)(ks / a.S * a.S * 512 + ks % a.S * 128), half_off = (uint32_t)a.S * 128u;
    const int krow = lane & 7, kc = lane >> 3;                      // + 8 keys per n tile, 16-byte column kc
    const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8, vc = lane >> 4;
    bool alive = true;
    // Block n has landed in its stage.  The stage's earlier blocks may have been the other group's, so first wait
    // until it is being filled with block n: the earlier phases are over then, and the parity is unambiguous.
    auto block_here = [&](uint32_t n) {
        const uint32_t st = n % kStages;
        bool seen = tag_s[st] == n;
        if (!seen) {
            const long long t0 = clock64();
            while (!(seen = tag_s[st] == n)) {
                if (clock64() - t0 > tc::kWaitCycles) {
                    raise_err(a.err, FOCUS_DEVERR_TIMEOUT);
                    break;
                }
                __nanosleep(20);  // (a group waits here while the other one is at its unit)
            }
        }
        return __all_sync(0xffffffffu, seen) && warp_wait(&full[st], (n / kStages) & 1u, a.err);
    };
    for (uint32_t u = grp;; u += 2) {
        // the group's warps go on or stop together: a wait that gave up in one of them alone would leave the others
        // at a named barrier
        if (!all_agree<32 * kGroup>(1 + grp, warp_wait(&u_full[u % kUnits], (u / kUnits) & 1u, a.err))) break;
        const UnitDesc& ud = unit_s[u % kUnits];
        const int nb = ud.nb;
        if (nb == 0) break;
        const int nrow = min(sh.tok, ud.n - ud.tok0) * a.G, kv = ud.kv;
        const int pos0 = kv - ud.n + ud.tok0;
        // query fragments: rows g4 and g4 + 8, columns 16 s + 2 t4 (+ 1) and + 8
        uint32_t q[8][4];
        const bool in0 = g4 < nrow, in1 = g4 + 8 < nrow;
        const uint8_t* qr = q_s + (u % kUnits) * kQBytes + g4 * kQRow + 4 * t4;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            q[s][0] = in0 ? *reinterpret_cast<const uint32_t*>(qr + 32 * s) : 0u;
            q[s][1] = in1 ? *reinterpret_cast<const uint32_t*>(qr + 8 * kQRow + 32 * s) : 0u;
            q[s][2] = in0 ? *reinterpret_cast<const uint32_t*>(qr + 32 * s + 16) : 0u;
            q[s][3] = in1 ? *reinterpret_cast<const uint32_t*>(qr + 8 * kQRow + 32 * s + 16) : 0u;
        }
        const int lim0 = in0 ? chunk_visible(pos0 + tk0, kv, a.mask_block) : 0;
        const int lim1 = in1 ? chunk_visible(pos0 + tk1, kv, a.mask_block) : 0;
        const int lim_all = chunk_visible(pos0, kv, a.mask_block);  // the fewest keys a row sees
        float m0 = -CUDART_INF_F, m1 = -CUDART_INF_F, l0 = 0.f, l1 = 0.f;
        float o[16][4];
#pragma unroll
        for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

        uint32_t n = first_s[u % kUnits];
        for (int i = 0; i < nb; ++i, ++n) {
            const uint32_t st = n % kStages;
            alive = alive && block_here(n);
            if (!alive) continue;
            const int key0 = (ud.blk0 + i) * kKeys + ks;
            const uint32_t bad = (bad_s[st] >> (ks >> 4)) & 1u;
            uint8_t* stage = ring + st * kStage;
            const uint32_t kb = smem_u32(stage) + key_off, vb = kb + 2 * half_off;
            // S: 16 rows x 16 keys, 128 columns; even and odd steps of 16 columns in chains of their own
            float s[2][4], s_odd[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[j][e] = s_odd[j][e] = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // 32 columns: 16-byte chunks 4 c .. 4 c + 3 of 16
                const int ch = 4 * (c & 1) + kc;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int row = krow + 8 * j;
                    uint32_t b[4];
                    ldsm4(b, kb + (c >> 1) * half_off + row * 128 + ((ch ^ (row & 7)) << 4));
                    mma16816(s[j], q[2 * c], b[0], b[1]);
                    mma16816(s_odd[j], q[2 * c + 1], b[2], b[3]);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[j][e] += s_odd[j][e];
            if (key0 + 16 > lim_all || bad) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + 8 * j + 2 * t4 + (e & 1);
                        if (key >= (e < 2 ? lim0 : lim1) || bad) s[j][e] = -CUDART_INF_F;
                    }
            }
            // V rows of keys that do not exist may hold anything: their weight is 0, so make them 0 as well
            if (key0 + 16 > kv || bad) {
                if (key0 + (lane & 15) >= kv || bad) {
                    uint8_t* vr = stage + key_off + (2 + (lane >> 4)) * half_off + (lane & 15) * 128;
#pragma unroll
                    for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vr + 16 * c) = make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the copy that reuses the stage
                __syncwarp();
            }
            float c0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
            float c1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
            for (int w = 1; w < 4; w <<= 1) {
                c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, w));
                c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, w));
            }
            c0 *= sl2;
            c1 *= sl2;
            float f0 = 1.f, f1 = 1.f;
            if (m0 == -CUDART_INF_F) m0 = c0;
            else if (c0 > m0 + kRaise) f0 = ex2f(m0 - c0), m0 = c0;
            if (m1 == -CUDART_INF_F) m1 = c1;
            else if (c1 > m1 + kRaise) f1 = ex2f(m1 - c1), m1 = c1;
            if (__any_sync(0xffffffffu, f0 != 1.f || f1 != 1.f)) {
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    o[k][0] *= f0;
                    o[k][1] *= f0;
                    o[k][2] *= f1;
                    o[k][3] *= f1;
                }
            }
            const float mu0 = m0 == -CUDART_INF_F ? 0.f : m0, mu1 = m1 == -CUDART_INF_F ? 0.f : m1;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s[j][0] = ex2f(fmaf(s[j][0], sl2, -mu0));
                s[j][1] = ex2f(fmaf(s[j][1], sl2, -mu0));
                s[j][2] = ex2f(fmaf(s[j][2], sl2, -mu1));
                s[j][3] = ex2f(fmaf(s[j][3], sl2, -mu1));
                l0 += s[j][0] + s[j][1];
                l1 += s[j][2] + s[j][3];
            }
            uint32_t p[4] = {pack_bf16(s[0][0], s[0][1]), pack_bf16(s[0][2], s[0][3]), pack_bf16(s[1][0], s[1][1]),
                             pack_bf16(s[1][2], s[1][3])};
            // O += P V: 16 keys, 16 columns a step
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int ch = 2 * (c & 3) + vc;
                uint32_t b[4];
                ldsm4t(b, vb + (c >> 2) * half_off + vrow * 128 + ((ch ^ (vrow & 7)) << 4));
                mma16816(o[2 * c], p, b[0], b[1]);
                mma16816(o[2 * c + 1], p, b[2], b[3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
        // ---- join the group's warps: maxima and denominators, then the outputs, two rows at a time, in warp order
#pragma unroll
        for (int w = 1; w < 4; w <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, w);
            l1 += __shfl_xor_sync(0xffffffffu, l1, w);
        }
        if (t4 == 0) {
            jm[warp][g4] = m0;
            jm[warp][g4 + 8] = m1;
            jl[warp][g4] = l0;
            jl[warp][g4 + 8] = l1;
        }
        const int row0 = ud.row0, tok0 = ud.tok0, g = ud.g, p0 = ud.c0, p1 = ud.c1, slot0 = ud.slot0;
        bf16* out = reinterpret_cast<bf16*>(a.out);
        auto out_ptr = [&](int r) {
            return out + (long long)(row0 + tok0 + token(r)) * a.out_stride + (g * a.G + r - token(r) * a.G) * kD;
        };
        const size_t mine = (size_t)((int)blockIdx.x == p0 ? slot0 : 2 * blockIdx.x) * kRows;
        auto sync = [&]() { named_sync<32 * kGroup>(1 + grp); };
#pragma unroll 1
        for (int pass = 0; 2 * pass < nrow; ++pass) {
            if (pass) sync();  // the rows before have been read (pass 0: by the barrier at the unit's start)
            if ((g4 >> 1) == (pass & 3) && (pass < 4 ? in0 : in1)) {
                // groups of eight columns change places by row, so that both rows' stores use all banks
                float* buf = join + warp * kJoinF + (g4 & 1) * kD + 2 * t4;
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    *reinterpret_cast<float2*>(buf + 8 * (k ^ (g4 & 1))) =
                        pass < 4 ? make_float2(o[k][0], o[k][1]) : make_float2(o[k][2], o[k][3]);
            }
            sync();
            if (pass == 0 && lane == 0) mbar_arrive(&u_empty[u % kUnits]);
            const int rr = wq & 1, r = 2 * pass + rr;  // two warps per row, two columns per lane
            if (r < nrow) {
                const int c = (wq >> 1) * 64 + lane * 2;
                const float* src = join + grp * kGroup * kJoinF + rr * kD + 8 * ((c >> 3) ^ rr) + (c & 7);
                float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
                for (int w = 0; w < kGroup; ++w) M = fmaxf(M, jm[grp * kGroup + w][r]);
                const float mu = M == -CUDART_INF_F ? 0.f : M;
                float2 v = make_float2(0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kGroup; ++w) {
                    const float f = ex2f(jm[grp * kGroup + w][r] - mu);
                    const float2 x = *reinterpret_cast<const float2*>(src + w * kJoinF);
                    L = fmaf(jl[grp * kGroup + w][r], f, L);
                    v.x = fmaf(x.x, f, v.x);
                    v.y = fmaf(x.y, f, v.y);
                }
                if (p0 < 0) {
                    const float inv = L > 0.f ? 1.f / L : 0.f;
                    if (alive) *reinterpret_cast<uint32_t*>(out_ptr(r) + c) = pack_bf16(v.x * inv, v.y * inv);
                } else {
                    __stcg(reinterpret_cast<float2*>(a.part_o + (mine + r) * kD + c), v);
                    if (wq < 2 && lane == 0) __stcg(reinterpret_cast<float2*>(a.part_ml) + mine + r, make_float2(M, L));
                }
            }
        }
        if (p0 >= 0) {
            // a unit shared with other CTAs: whoever arrives last adds the pieces in order, a warp per row
            __threadfence();
            sync();
            if (wq == 0 && lane == 0)
                last_s[grp] = atomicInc(reinterpret_cast<unsigned*>(a.counters) + p0, (unsigned)(p1 - p0)) ==
                              (unsigned)(p1 - p0);
            sync();
            if (last_s[grp]) {
                __threadfence();
                const int cnt = p1 - p0 + 1;
                for (int r = wq; r < nrow; r += kGroup) {
                    auto at = [&](int k) { return (size_t)(k == 0 ? slot0 : 2 * (p0 + k)) * kRows + r; };
                    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
                    float M = -CUDART_INF_F;
                    for (int k = lane; k < cnt; k += 32) M = fmaxf(M, __ldcg(ml + at(k)).x);
                    M = warp_max(M);
                    const float mu = M == -CUDART_INF_F ? 0.f : M;
                    float L = 0.f;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int k0 = 0; k0 < cnt; k0 += 32) {
                        float f = 0.f;
                        if (k0 + lane < cnt) {
                            const float2 x = __ldcg(ml + at(k0 + lane));
                            f = ex2f(x.x - mu);
                            L = fmaf(x.y, f, L);
                        }
                        const int n_here = min(32, cnt - k0);
#pragma unroll 4
                        for (int k = 0; k < n_here; ++k) {
                            const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part_o + at(k0 + k) * kD + lane * 4));
                            const float w = __shfl_sync(0xffffffffu, f, k);
                            v.x = fmaf(x.x, w, v.x);
                            v.y = fmaf(x.y, w, v.y);
                            v.z = fmaf(x.z, w, v.z);
                            v.w = fmaf(x.w, w, v.w);
                        }
                    }
                    L = warp_sum(L);
                    const float inv = L > 0.f ? 1.f / L : 0.f;
                    if (alive) store4<bf16>(out_ptr(r) + lane * 4, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                }
            }
        }
    }
}

}  // namespace

bool configure_chunk_attention_few() {
    return cudaFuncSetAttribute(chunk_attn_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem) ==
               cudaSuccess &&
           max_shared_carveout((const void*)chunk_attn_few_kernel);
}

int launch_chunk_attention_few(const ChunkAttnDev& a, int sms, cudaStream_t s) {
    CUtensorMap pool_map{};  // (without pages every key is invalid and the map is never used)
    if (a.n_pages > 0 && !make_pool_map(&pool_map, a, 2, 2)) return -1;
    const dim3 grid(sms < kChunkCtas ? sms : kChunkCtas), block(kFewThreads);
    return launched(launch_pdl(chunk_attn_few_kernel, grid, block, kFewSmem, s, 0, pool_map, a));
}

}  // namespace focus
