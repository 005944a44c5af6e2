// Attention of a chunk of new tokens over the paged cache on the CUDA cores (float32 models).
//
//   out[row] = sum_j 2^(s_j - m) V_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q . K_j,  m = max_j s_j
//
// in one pass over the keys: per block of KEYS keys the running maximum m, the denominator and the output
// are rescaled by 2^(m_old - m_new) and the block is added.  A unit is (request, KV head, TR query vectors
// of the G = Hq / Hkv heads that share it; query vector r is token r / G, head r % G), so K and V are read
// once per group.  Two shapes: TR = 64 (chunks; 4 x (KEYS / 16) scores per thread, bound by the FMA pipe),
// TR = 8 (8 query vectors or fewer: single tokens, short chunks).  Measured, 4/4 heads of 64, TR = 8 / TR = 64 for
// single tokens over 512 to 2048 keys: 8 requests 21.7 / 34.8 us, 64 requests 63.9 / 165.7; 5 single tokens and 6
// prompts of up to 401 tokens 35 us.  K and V of the next block are
// on their way while one is used (cp.async, two buffers).  The walk over the keys is split over the CTAs by
// chunk_work.cuh.
#include <math_constants.h>

#include "chunk_work.cuh"

namespace focus {
namespace {

constexpr int kThreads = 256;
constexpr int kFew = kChunkSimtFew;

template <int D, int TR> struct SimtShape {
    static constexpr int KEYS = D == 128 ? 32 : 64;
    static constexpr int KSTR = D + 4;      // padded rows: 16 keys' float4 fall on distinct banks
    static constexpr int PSTR = KEYS + 4;
    static constexpr int Q_F = TR * KSTR, K_F = KEYS * KSTR, V_F = KEYS * D, P_F = TR * PSTR;
    static constexpr int SMEM = (Q_F + 2 * (K_F + V_F) + P_F + 4 * TR) * 4 + 3 * KEYS * 8;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool there) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst), n = there ? 16u : 0u;  // 0: the 16 bytes become zero
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}

template <typename T, int D, int TR> __device__ __forceinline__ void simt_walk(const ChunkAttnDev& a) {
    static_assert(sizeof(T) == 4, "copies move float32 rows as they are");
    using S = SimtShape<D, TR>;
    constexpr int KEYS = S::KEYS, KSTR = S::KSTR, PSTR = S::PSTR;
    constexpr bool kTile = TR == 64;
    extern __shared__ __align__(16) float smem[];
    float* qs = smem;                 // [TR][KSTR]
    float* ks = qs + S::Q_F;          // [2][KEYS][KSTR]
    float* vs = ks + 2 * S::K_F;      // [2][KEYS][D]
    float* ps = vs + 2 * S::V_F;      // [TR][PSTR]
    float* ms = ps + S::P_F;          // [TR] running maxima
    float* ls = ms + TR;              // [TR] denominators
    float* al = ls + TR;              // [TR] rescale factors of the block; a piece's weight at the end
    int* vis = reinterpret_cast<int*>(al + TR);                  // [TR] visible keys of each row
    // [3][KEYS] element offset of the key's row, -1: none.  Three blocks' worth: a warp that is done with block b - 1
    // writes block b + 1's while others still read block b - 1's, and block b's are for its copies.
    long long* row_at = reinterpret_cast<long long*>(vis + TR);
    __shared__ ChunkRange rg;
    __shared__ long long red[32];
    __shared__ int last_s;
    extern __shared__ __align__(16) long long scr_raw[];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ChunkShape sh{TR / a.G > 0 ? TR / a.G : 1, kTile ? kFew : 0, kTile ? 0x7fffffff : kFew};
    chunk_schedule<KEYS, kTile ? 1 : 4>(a, sh, scr_raw, red, &rg);
    const float sl2 = a.scale * 1.4426950408889634f;
    const T* pool = reinterpret_cast<const T*>(a.kv_pool);
    const long long v_off = (long long)a.Hkv * a.S * D;

    ChunkWalk<KEYS> wk;
    for (wk.start(a, sh, rg); wk.live(); wk.next(a, sh)) {
        const int t0 = wk.k * sh.tok, nrow = min(sh.tok, wk.r.n - t0) * a.G;
        const int nb = wk.blk1 - wk.blk0;
        // key `tid` of block blk (threads below KEYS): its page number, then its row's offset
        auto page_of = [&](int blk) {
            const int key = blk * KEYS + tid;
            return tid < KEYS && blk < wk.blk1 && key < wk.r.kv ? a.page_table[(size_t)wk.b * a.max_pages + key / a.S] : -1;
        };
        auto place = [&](int blk, int page) {
            if (tid >= KEYS) return;
            const int key = blk * KEYS + tid;
            long long at = -1;
            if (key < wk.r.kv) {
                if (page >= 0 && page < a.n_pages)
                    at = (long long)(((((size_t)page * a.L + a.layer) * 2) * a.Hkv + wk.g) * a.S + key % a.S) * D;
                else
                    raise_err(a.err, FOCUS_DEVERR_PAGE_ID);
            }
            row_at[blk % 3 * KEYS + tid] = at;
        };
        auto copy = [&](int blk) {
            float *kd = ks + (blk & 1) * S::K_F, *vd = vs + (blk & 1) * S::V_F;
#pragma unroll
            for (int i = tid; i < KEYS * (D / 4); i += kThreads) {
                const int j = i / (D / 4), c = (i - j * (D / 4)) * 4;
                const long long at = row_at[blk % 3 * KEYS + j];
                const T* src = pool + (at < 0 ? 0 : at) + c;
                cp_async16(kd + j * KSTR + c, src, at >= 0);
                cp_async16(vd + j * D + c, at < 0 ? src : src + v_off, at >= 0);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int page = page_of(wk.blk0);
        __syncthreads();  // the previous unit's shared memory has been read
        for (int i = tid; i < TR * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4, tok = r / a.G;
            const bool in = r < nrow;
            const T* src = reinterpret_cast<const T*>(a.q) +
                           (in ? (long long)(wk.r.row0 + t0 + tok) * a.q_stride + (wk.g * a.G + r - tok * a.G) * D + c : 0);
            cp_async16(qs + r * KSTR + c, src, in);
        }
        if (tid < TR) {
            const int pos = wk.r.kv - wk.r.n + t0 + tid / a.G;
            vis[tid] = tid < nrow ? chunk_visible(pos, wk.r.kv, a.mask_block) : 0;
            ms[tid] = -CUDART_INF_F;
            ls[tid] = 0.f;
        }
        place(wk.blk0, page);
        page = page_of(wk.blk0 + 1);
        __syncthreads();
        copy(wk.blk0);
        // accumulators: TR = 64: rows 4 ty .. + 3, columns 4 tx + 64 j .. + 3; TR = 8: rows 4 (warp & 1) .. + 3,
        // D / 32 columns from lane * D / 32, over the keys of quarter warp / 2
        constexpr int AC = kTile ? D / 16 : D / 32;
        float acc[4][AC];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < AC; ++j) acc[i][j] = 0.f;

        for (int b = 0; b < nb; ++b) {
            const int blk = wk.blk0 + b;
            if (b + 1 < nb) {
                place(blk + 1, page);
                page = page_of(blk + 2);
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();  // this block has landed, the one before has been read
            if (b + 1 < nb) copy(blk + 1);
            const float *kb = ks + (blk & 1) * S::K_F, *vb = vs + (blk & 1) * S::V_F;
            const long long* there = row_at + blk % 3 * KEYS;
            if constexpr (kTile) {
                constexpr int KPT = KEYS / 16;
                const int ty = tid >> 4, tx = tid & 15;
                float s[4][KPT];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < KPT; ++j) s[i][j] = 0.f;
#pragma unroll 4
                for (int c = 0; c < D; c += 4) {
                    float4 kv[KPT];
#pragma unroll
                    for (int j = 0; j < KPT; ++j) kv[j] = *reinterpret_cast<const float4*>(kb + (tx + 16 * j) * KSTR + c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 q = *reinterpret_cast<const float4*>(qs + (4 * ty + i) * KSTR + c);
#pragma unroll
                        for (int j = 0; j < KPT; ++j) {
                            s[i][j] = fmaf(q.x, kv[j].x, s[i][j]);
                            s[i][j] = fmaf(q.y, kv[j].y, s[i][j]);
                            s[i][j] = fmaf(q.z, kv[j].z, s[i][j]);
                            s[i][j] = fmaf(q.w, kv[j].w, s[i][j]);
                        }
                    }
                }
                bool ok[KPT];
#pragma unroll
                for (int j = 0; j < KPT; ++j) ok[j] = there[tx + 16 * j] >= 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * ty + i;
                    const int lim = vis[r] - blk * KEYS;
                    float mx = -CUDART_INF_F;
#pragma unroll
                    for (int j = 0; j < KPT; ++j) {
                        s[i][j] = tx + 16 * j < lim && ok[j] ? s[i][j] * sl2 : -CUDART_INF_F;
                        mx = fmaxf(mx, s[i][j]);
                    }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    const float m0 = ms[r], m1 = fmaxf(m0, mx);
                    const float mu = m1 == -CUDART_INF_F ? 0.f : m1;
                    const float f = exp2f(m0 - mu);  // 0 while nothing has been summed
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < KPT; ++j) {
                        const float p = exp2f(s[i][j] - mu);
                        sum += p;
                        ps[r * PSTR + tx + 16 * j] = p;
                    }
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    __syncwarp();
                    if (tx == 0) {
                        ms[r] = m1;
                        ls[r] = ls[r] * f + sum;
                    }
#pragma unroll
                    for (int j = 0; j < AC; ++j) acc[i][j] *= f;
                }
                __syncwarp();  // a row's weights are written and read by one warp
#pragma unroll 2
                for (int k4 = 0; k4 < KEYS; k4 += 4) {
                    float4 p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(ps + (4 * ty + i) * PSTR + k4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                        for (int j = 0; j < AC; j += 4) {
                            const float4 v = *reinterpret_cast<const float4*>(vb + (k4 + kk) * D + 4 * tx + 16 * j);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                                acc[i][j] = fmaf(w, v.x, acc[i][j]);
                                acc[i][j + 1] = fmaf(w, v.y, acc[i][j + 1]);
                                acc[i][j + 2] = fmaf(w, v.z, acc[i][j + 2]);
                                acc[i][j + 3] = fmaf(w, v.w, acc[i][j + 3]);
                            }
                        }
                    }
                }
            } else {
                // scores: one key and TR KEYS / 256 rows per thread
                constexpr int RPT = TR * KEYS / kThreads;
                const int key = tid % KEYS, r0 = tid / KEYS * RPT;
                float s[RPT];
#pragma unroll
                for (int i = 0; i < RPT; ++i) s[i] = 0.f;
#pragma unroll 8
                for (int c = 0; c < D; c += 4) {
                    const float4 k4 = *reinterpret_cast<const float4*>(kb + key * KSTR + c);
#pragma unroll
                    for (int i = 0; i < RPT; ++i) {
                        const float4 q = *reinterpret_cast<const float4*>(qs + (r0 + i) * KSTR + c);
                        s[i] = fmaf(q.x, k4.x, s[i]);
                        s[i] = fmaf(q.y, k4.y, s[i]);
                        s[i] = fmaf(q.z, k4.z, s[i]);
                        s[i] = fmaf(q.w, k4.w, s[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < RPT; ++i)
                    ps[(r0 + i) * PSTR + key] =
                        blk * KEYS + key < vis[r0 + i] && there[key] >= 0 ? s[i] * sl2 : -CUDART_INF_F;
                __syncthreads();
                {
                    const int r = warp;  // eight warps, eight rows
                    float mx = -CUDART_INF_F, sum = 0.f;
#pragma unroll
                    for (int j = lane; j < KEYS; j += 32) mx = fmaxf(mx, ps[r * PSTR + j]);
                    mx = warp_max(mx);
                    const float m0 = ms[r], m1 = fmaxf(m0, mx);
                    const float mu = m1 == -CUDART_INF_F ? 0.f : m1;
#pragma unroll
                    for (int j = lane; j < KEYS; j += 32) {
                        const float p = exp2f(ps[r * PSTR + j] - mu);
                        ps[r * PSTR + j] = p;
                        sum += p;
                    }
                    sum = warp_sum(sum);
                    __syncwarp();
                    if (lane == 0) {
                        const float f = exp2f(m0 - mu);
                        al[r] = f;
                        ms[r] = m1;
                        ls[r] = ls[r] * f + sum;
                    }
                }
                __syncthreads();
                const int rb = (warp & 1) * 4, kq = (warp >> 1) * (KEYS / 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = al[rb + i];
#pragma unroll
                    for (int j = 0; j < AC; ++j) acc[i][j] *= f;
                }
#pragma unroll 4
                for (int k1 = kq; k1 < kq + KEYS / 4; ++k1) {
                    float v[AC];
#pragma unroll
                    for (int j = 0; j < AC; ++j) v[j] = vb[k1 * D + lane * AC + j];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = ps[(rb + i) * PSTR + k1];
#pragma unroll
                        for (int j = 0; j < AC; ++j) acc[i][j] = fmaf(p, v[j], acc[i][j]);
                    }
                }
            }
        }
        __syncthreads();  // maxima and denominators are final; K, V and the queries have been read
        T* out = reinterpret_cast<T*>(a.out);
        auto out_ptr = [&](int r) {
            const int tok = r / a.G;
            return out + (long long)(wk.r.row0 + t0 + tok) * a.out_stride + (wk.g * a.G + r - tok * a.G) * D;
        };
        const bool whole = wk.whole();
        int c0 = 0, c1 = 0, slot0 = 0;
        if (!whole) wk.pieces(rg, c0, c1, slot0);
        auto piece = [&](int c) { return (size_t)(c == c0 ? slot0 : 2 * c); };
        const size_t mine = piece(blockIdx.x);
        // four columns of a row: the result, or this piece's unnormalised share
        auto put = [&](int r, int c, float4 v) {
            if (whole) {
                const float inv = ls[r] > 0.f ? 1.f / ls[r] : 0.f;
                store4<T>(out_ptr(r) + c, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            } else {
                __stcg(reinterpret_cast<float4*>(a.part_o + (mine * TR + r) * D + c), v);
            }
        };
        if constexpr (kTile) {
            const int ty = tid >> 4, tx = tid & 15;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * ty + i < nrow)
#pragma unroll
                    for (int j = 0; j < AC; j += 4)
                        put(4 * ty + i, 4 * tx + 16 * j, make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]));
        } else {
            float* part = ks;  // [4 key quarters][TR][D]
            static_assert(4 * TR * D <= 2 * S::K_F || kTile, "the quarters' sums fit in the K buffers");
            const int rb = (warp & 1) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < AC; ++j) part[((warp >> 1) * TR + rb + i) * D + lane * AC + j] = acc[i][j];
            __syncthreads();
            for (int i = tid; i < nrow * (D / 4); i += kThreads) {
                const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 x = *reinterpret_cast<const float4*>(part + (q * TR + r) * D + c);
                    v.x += x.x;
                    v.y += x.y;
                    v.z += x.z;
                    v.w += x.w;
                }
                put(r, c, v);
            }
        }
        if (whole) continue;
        // ---- a shared unit: the last CTA to arrive adds the pieces in order
        float2* pml = reinterpret_cast<float2*>(a.part_ml);
        if (tid < nrow) __stcg(pml + mine * TR + tid, make_float2(ms[tid], ls[tid]));
        __threadfence();
        __syncthreads();
        if (tid == 0) last_s = atomicInc(reinterpret_cast<unsigned*>(a.counters) + c0, (unsigned)(c1 - c0)) == (unsigned)(c1 - c0);
        __syncthreads();
        if (!last_s) continue;
        __threadfence();
        const int cnt = c1 - c0 + 1;
        for (int r = tid; r < nrow; r += kThreads) {  // each row's maximum and denominator over the pieces
            float m = -CUDART_INF_F;
#pragma unroll 4
            for (int p = 0; p < cnt; ++p) m = fmaxf(m, __ldcg(pml + piece(c0 + p) * TR + r).x);
            const float mu = m == -CUDART_INF_F ? 0.f : m;
            float l = 0.f;
#pragma unroll 4
            for (int p = 0; p < cnt; ++p) {
                const float2 x = __ldcg(pml + piece(c0 + p) * TR + r);
                l = fmaf(x.y, exp2f(x.x - mu), l);
            }
            ms[r] = mu;
            ls[r] = l > 0.f ? 1.f / l : 0.f;
        }
        __syncthreads();
        for (int i = tid; i < nrow * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
            const float mu = ms[r], inv = ls[r];
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int p = 0; p < cnt; ++p) {
                const size_t at = piece(c0 + p) * TR + r;
                const float f = exp2f(__ldcg(pml + at).x - mu);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + c));
                o.x = fmaf(v.x, f, o.x);
                o.y = fmaf(v.y, f, o.y);
                o.z = fmaf(v.z, f, o.z);
                o.w = fmaf(v.w, f, o.w);
            }
            store4<T>(out_ptr(r) + c, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        }
    }
}

template <typename T, int D, int TR> __global__ void __launch_bounds__(kThreads, 2) chunk_attn_simt_kernel(ChunkAttnDev a) {
    pdl_entry();
    simt_walk<T, D, TR>(a);
}

// Both shapes in one launch: row 0 of the grid takes the requests of many query vectors, row 1 the others as its CTAs make
// room, each with scratch of its own (5 single tokens and 6 chunks: 52 us as two launches, 35 us; 40 and 5 larger ones,
// 8/8 heads of 128: 381 and 368).
template <typename T, int D> __global__ void __launch_bounds__(kThreads, 2) chunk_attn_simt_both_kernel(ChunkAttnDev a) {
    pdl_entry();
    if (blockIdx.y == 0) {
        simt_walk<T, D, 64>(a);
    } else {
        a.part_o += (size_t)2 * kChunkSimtCtas * kChunkSimtRows * D;
        a.part_ml += (size_t)2 * kChunkSimtCtas * kChunkSimtRows * 2;
        a.counters += kChunkSimtCtas;
        simt_walk<T, D, kFew>(a);
    }
}

// dynamic shared memory: the tiles, or the schedule's sums if there are very many requests
template <int D, int TR> int simt_smem(int N) {
    const int sched = (N + 1) * 8;
    return SimtShape<D, TR>::SMEM > sched ? SimtShape<D, TR>::SMEM : sched;
}

template <int D> int simt_smem_both(int N) {
    return simt_smem<D, 64>(N) > simt_smem<D, kFew>(N) ? simt_smem<D, 64>(N) : simt_smem<D, kFew>(N);
}

bool configure_one(const void* kernel, int smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess &&
           max_shared_carveout(kernel);
}
template <int D> bool configure_all() {
    return configure_one((const void*)chunk_attn_simt_kernel<float, D, kFew>, simt_smem<D, kFew>(kChunkMaxRequests)) &&
           configure_one((const void*)chunk_attn_simt_kernel<float, D, 64>, simt_smem<D, 64>(kChunkMaxRequests)) &&
           configure_one((const void*)chunk_attn_simt_both_kernel<float, D>, simt_smem_both<D>(kChunkMaxRequests));
}

}  // namespace

bool configure_chunk_attention_simt() { return configure_all<64>() && configure_all<128>(); }

template <typename T, int D> int launch_chunk_attention_simt(const ChunkAttnDev& a, int sms, cudaStream_t s) {
    const dim3 block(kThreads);
    const unsigned ctas = 2 * sms < kChunkSimtCtas ? 2 * sms : kChunkSimtCtas;
    const bool many = (long long)a.max_new * a.G > kFew, few = a.G <= kFew;   // shapes that requests may need
    if (many && few)
        return launched(launch_pdl(chunk_attn_simt_both_kernel<T, D>, dim3(ctas, 2), block, simt_smem_both<D>(a.N), s, 0, a));
    if (many) return launched(launch_pdl(chunk_attn_simt_kernel<T, D, 64>, dim3(ctas), block, simt_smem<D, 64>(a.N), s, 0, a));
    return launched(launch_pdl(chunk_attn_simt_kernel<T, D, kFew>, dim3(ctas), block, simt_smem<D, kFew>(a.N), s, 0, a));
}

template int launch_chunk_attention_simt<float, 64>(const ChunkAttnDev&, int, cudaStream_t);
template int launch_chunk_attention_simt<float, 128>(const ChunkAttnDev&, int, cudaStream_t);

}  // namespace focus
