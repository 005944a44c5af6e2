// Attention of a chunk of new tokens over the paged cache on the CUDA cores (float32 models).
//
//   out[row] = sum_j 2^(s_j - m) V_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q . K_j,  m = max_j s_j
//
// in one pass over the keys: per block of KEYS keys the running maximum m, the denominator and the output
// are rescaled by 2^(m_old - m_new) and the block is added.  A unit is (request, KV head, TR query vectors
// of the G = Hq / Hkv heads that share it; query vector r is token r / G, head r % G), so K and V are read
// once per group.  Two shapes: TR = 64 (chunks; 4 x (KEYS / 16) scores per thread, bound by the FMA pipe),
// TR = 8 (single tokens: 8 query vectors or fewer, bound by memory).  The walk over the keys is split
// over the CTAs by chunk_work.cuh.
#include <math_constants.h>

#include "chunk_work.cuh"

namespace focus {
namespace {

constexpr int kThreads = 256;
constexpr int kFew = 8;  // query vectors of the few-row shape

template <int D, int TR> struct SimtShape {
    static constexpr int KEYS = D == 128 ? 32 : 64;
    static constexpr int KSTR = D + 4;      // padded rows: 16 keys' float4 fall on distinct banks
    static constexpr int PSTR = KEYS + 4;
    static constexpr int Q_F = TR * KSTR, K_F = KEYS * KSTR, V_F = KEYS * D, P_F = TR * PSTR;
    static constexpr int SMEM = (Q_F + K_F + V_F + P_F + 4 * TR) * 4 + KEYS * 4;
};

template <typename T, int D, int TR>
__global__ void __launch_bounds__(kThreads, 2) chunk_attn_simt_kernel(ChunkAttnDev a) {
    using S = SimtShape<D, TR>;
    constexpr int KEYS = S::KEYS, KSTR = S::KSTR, PSTR = S::PSTR;
    constexpr bool kTile = TR == 64;
    pdl_entry();
    extern __shared__ __align__(16) float smem[];
    float* qs = smem;                 // [TR][KSTR]; the output rows at the end of a unit
    float* ks = qs + S::Q_F;          // [KEYS][KSTR]
    float* vs = ks + S::K_F;          // [KEYS][D]
    float* ps = vs + S::V_F;          // [TR][PSTR]
    float* ms = ps + S::P_F;          // [TR] running maxima
    float* ls = ms + TR;              // [TR] denominators
    float* al = ls + TR;              // [TR] rescale factors of the block
    int* vis = reinterpret_cast<int*>(al + TR);  // [TR] visible keys of each row
    int* ok = vis + TR;               // [KEYS] key present
    __shared__ ChunkRange rg;
    __shared__ long long red[32];
    __shared__ int last_s;
    extern __shared__ __align__(16) long long scr_raw[];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const ChunkShape sh{TR / a.G > 0 ? TR / a.G : 1, kTile ? kFew : 0, kTile ? 0x7fffffff : kFew};
    chunk_schedule<KEYS, kTile ? 2 : 4>(a, sh, scr_raw, red, &rg);
    const float sl2 = a.scale * 1.4426950408889634f;
    const T* pool = reinterpret_cast<const T*>(a.kv_pool);

    ChunkWalk<KEYS> wk;
    for (wk.start(a, sh, rg); wk.live(); wk.next(a, sh)) {
        const int t0 = wk.k * sh.tok, nrow = min(sh.tok, wk.r.n - t0) * a.G;
        __syncthreads();  // the previous unit's shared memory has been read
        for (int i = tid; i < TR * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < nrow) {
                const int tok = t0 + r / a.G, h = wk.g * a.G + r % a.G;
                v = load4<T>(reinterpret_cast<const T*>(a.q) + (long long)(wk.r.row0 + tok) * a.q_stride + h * D + c);
            }
            *reinterpret_cast<float4*>(qs + r * KSTR + c) = v;
        }
        if (tid < TR) {
            const int pos = wk.r.kv - wk.r.n + t0 + tid / a.G;
            vis[tid] = tid < nrow ? chunk_visible(pos, wk.r.kv, a.mask_block) : 0;
            ms[tid] = -CUDART_INF_F;
            ls[tid] = 0.f;
        }
        // accumulators: TR = 64: rows 4 ty .. + 3, columns 4 tx + 64 j .. + 3; TR = 8: rows 4 (warp & 1) .. + 3,
        // D / 32 columns from lane * D / 32, over the keys of quarter warp / 2
        constexpr int AC = kTile ? D / 16 : D / 32;
        float acc[4][AC];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < AC; ++j) acc[i][j] = 0.f;

        for (int blk = wk.blk0; blk < wk.blk1; ++blk) {
            __syncthreads();  // the previous block's K, V, P have been read
            for (int j = warp; j < KEYS; j += kThreads / 32) {
                const int key = blk * KEYS + j;
                int page = -1;
                if (key < wk.r.kv) {
                    page = a.page_table[(size_t)wk.b * a.max_pages + key / a.S];
                    if (page < 0 || page >= a.n_pages) {
                        if (lane == 0) raise_err(a.err, FOCUS_DEVERR_PAGE_ID);
                        page = -1;
                    }
                }
                const size_t kr = ((((size_t)max(page, 0) * a.L + a.layer) * 2) * a.Hkv + wk.g) * a.S + key % a.S;
                const T* kp = pool + kr * D;
                const T* vp = kp + (size_t)a.Hkv * a.S * D;
                for (int c = lane * 4; c < D; c += 128) {
                    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                    *reinterpret_cast<float4*>(ks + j * KSTR + c) = page >= 0 ? load4<T>(kp + c) : z;
                    *reinterpret_cast<float4*>(vs + j * D + c) = page >= 0 ? load4<T>(vp + c) : z;
                }
                if (lane == 0) ok[j] = page >= 0;
            }
            __syncthreads();
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
                    for (int j = 0; j < KPT; ++j) kv[j] = *reinterpret_cast<const float4*>(ks + (tx + 16 * j) * KSTR + c);
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
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * ty + i;
                    const int lim = vis[r] - blk * KEYS;
                    float mx = -CUDART_INF_F;
#pragma unroll
                    for (int j = 0; j < KPT; ++j) {
                        const int key = tx + 16 * j;
                        s[i][j] = key < lim && ok[key] ? s[i][j] * sl2 : -CUDART_INF_F;
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
                            const float4 v = *reinterpret_cast<const float4*>(vs + (k4 + kk) * D + 4 * tx + 16 * j);
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
                    const float4 k4 = *reinterpret_cast<const float4*>(ks + key * KSTR + c);
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
                        blk * KEYS + key < vis[r0 + i] && ok[key] ? s[i] * sl2 : -CUDART_INF_F;
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
                    for (int j = 0; j < AC; ++j) v[j] = vs[k1 * D + lane * AC + j];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = ps[(rb + i) * PSTR + k1];
#pragma unroll
                        for (int j = 0; j < AC; ++j) acc[i][j] = fmaf(p, v[j], acc[i][j]);
                    }
                }
            }
        }
        // ---- the piece's unnormalised rows to shared memory
        __syncthreads();
        if constexpr (kTile) {
            const int ty = tid >> 4, tx = tid & 15;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < AC; j += 4)
                    *reinterpret_cast<float4*>(qs + (4 * ty + i) * KSTR + 4 * tx + 16 * j) =
                        make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
        } else {
            float* part = ks;  // [4 key quarters][TR][D]
            const int rb = (warp & 1) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < AC; ++j) part[((warp >> 1) * TR + rb + i) * D + lane * AC + j] = acc[i][j];
            __syncthreads();
            for (int i = tid; i < TR * D; i += kThreads)
                qs[i / D * KSTR + i % D] = (part[i] + part[TR * D + i]) + (part[2 * TR * D + i] + part[3 * TR * D + i]);
        }
        __syncthreads();
        T* out = reinterpret_cast<T*>(a.out);
        auto out_ptr = [&](int r) {
            return out + (long long)(wk.r.row0 + t0 + r / a.G) * a.out_stride + (wk.g * a.G + r % a.G) * D;
        };
        if (wk.whole()) {
            for (int i = tid; i < nrow * (D / 4); i += kThreads) {
                const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
                const float inv = ls[r] > 0.f ? 1.f / ls[r] : 0.f;
                const float4 v = *reinterpret_cast<const float4*>(qs + r * KSTR + c);
                store4<T>(out_ptr(r) + c, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            }
            continue;
        }
        // ---- a shared unit: leave the piece in scratch; the last CTA to arrive adds the pieces in order
        int c0, c1, slot0;
        wk.pieces(rg, c0, c1, slot0);
        auto piece = [&](int c) { return (size_t)(c == c0 ? slot0 : 2 * c); };
        const size_t mine = piece(blockIdx.x);
        for (int i = tid; i < nrow * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
            __stcg(reinterpret_cast<float4*>(a.part_o + (mine * TR + r) * D + c),
                   *reinterpret_cast<const float4*>(qs + r * KSTR + c));
        }
        if (tid < nrow) __stcg(reinterpret_cast<float2*>(a.part_ml) + mine * TR + tid, make_float2(ms[tid], ls[tid]));
        __threadfence();
        __syncthreads();
        if (tid == 0) last_s = atomicInc(reinterpret_cast<unsigned*>(a.counters) + c0, (unsigned)(c1 - c0)) == (unsigned)(c1 - c0);
        __syncthreads();
        if (!last_s) continue;
        __threadfence();
        for (int i = tid; i < nrow * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
            float m = -CUDART_INF_F;
            for (int p = c0; p <= c1; ++p)
                m = fmaxf(m, __ldcg(reinterpret_cast<const float2*>(a.part_ml) + piece(p) * TR + r).x);
            const float mu = m == -CUDART_INF_F ? 0.f : m;
            float l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int p = c0; p <= c1; ++p) {
                const size_t at = piece(p) * TR + r;
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(a.part_ml) + at);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + at * D + c));
                const float f = exp2f(ml.x - mu);
                l = fmaf(ml.y, f, l);
                o.x = fmaf(v.x, f, o.x);
                o.y = fmaf(v.y, f, o.y);
                o.z = fmaf(v.z, f, o.z);
                o.w = fmaf(v.w, f, o.w);
            }
            const float inv = l > 0.f ? 1.f / l : 0.f;
            store4<T>(out_ptr(r) + c, o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        }
    }
}

// dynamic shared memory: the tiles, or the schedule's sums if there are very many requests
template <int D, int TR> int simt_smem(int N) {
    const int sched = (N + 1) * 8;
    return SimtShape<D, TR>::SMEM > sched ? SimtShape<D, TR>::SMEM : sched;
}

template <typename T, int D, int TR> bool configure_one() {
    return cudaFuncSetAttribute(chunk_attn_simt_kernel<T, D, TR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                simt_smem<D, TR>(kChunkMaxRequests)) == cudaSuccess &&
           max_shared_carveout((const void*)chunk_attn_simt_kernel<T, D, TR>);
}

}  // namespace

bool configure_chunk_attention_simt() {
    return configure_one<float, 64, 8>() && configure_one<float, 64, 64>() && configure_one<float, 128, 8>() &&
           configure_one<float, 128, 64>();
}

template <typename T, int D> int launch_chunk_attention_simt(const ChunkAttnDev& a, int sms, cudaStream_t s) {
    const dim3 grid(2 * sms < kChunkSimtCtas ? 2 * sms : kChunkSimtCtas), block(kThreads);
    int n = 0;
    const long long most = (long long)a.max_new * a.G;
    if (most > kFew) {  // units of 64 query vectors
        if (launched(launch_pdl(chunk_attn_simt_kernel<T, D, 64>, grid, block, simt_smem<D, 64>(a.N), s, 0, a)) < 0)
            return -1;
        ++n;
    }
    if (a.G <= kFew) {
        if (launched(launch_pdl(chunk_attn_simt_kernel<T, D, 8>, grid, block, simt_smem<D, 8>(a.N), s, 0, a)) < 0)
            return -1;
        ++n;
    }
    return n;
}

template int launch_chunk_attention_simt<float, 64>(const ChunkAttnDev&, int, cudaStream_t);
template int launch_chunk_attention_simt<float, 128>(const ChunkAttnDev&, int, cudaStream_t);

}  // namespace focus
