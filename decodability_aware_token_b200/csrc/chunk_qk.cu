// Per-head RMSNorm of queries and keys, rotate-half RoPE and the write into the paged cache, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * gain
//   (y_i, y_{i + d/2}) -> (y_i c - y_{i + d/2} s, y_{i + d/2} c + y_i s),  c + i s = exp(i pos theta^(-2i/d))
//
// Bound by memory: each of the (Hq + 2 Hkv) d values of a row is read once and written once.  A lane holds
// 16 bytes of a head's lower half and the 16 bytes of the same pairs in its upper half, so the rotation needs
// no exchange and every access is a full 16 bytes; D / 2 / (16 bytes) lanes form a head and a warp works
// on several heads of one row at once.  A row's angles are computed once per warp and used for all its heads:
// pos / pi theta^(-2i/d) in double, reduced to [-1, 1] exactly, then sincospif.  (Float angles lose
// pos 2^-24 radians: 4e-3 at position 65536.)  The result is rounded once, to T.
#include "chunk.h"

namespace focus {
namespace {

constexpr int kThreads = 256;

template <typename T, int V> struct Pack;  // 16 bytes
template <> struct Pack<bf16, 8> {
    uint4 u;
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        u = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Pack<float, 4> {
    uint4 u;
    __device__ __forceinline__ void get(float (&f)[4]) const {
        f[0] = __uint_as_float(u.x);
        f[1] = __uint_as_float(u.y);
        f[2] = __uint_as_float(u.z);
        f[3] = __uint_as_float(u.w);
    }
    __device__ __forceinline__ void set(const float (&f)[4]) {
        u = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) chunk_qk_kernel(ChunkQkDev a, int warps_per_row) {
    constexpr int V = 16 / (int)sizeof(T);      // values per access
    constexpr int LPH = D / 2 / V;              // lanes per head
    constexpr int HPW = 32 / LPH;               // heads a warp works on at once
    using P = Pack<T, V>;
    pdl_entry();
    const focus_chunk_qk& p = a.p;
    const int gw = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int row = gw / warps_per_row, part = gw - row * warps_per_row;
    if (row >= p.rows) return;
    const int pos = p.row_pos[row];
    if (pos < 0) return;
    int slot = p.row_slot[row];
    if (slot >= 0 && slot / p.page_size >= p.n_pages) {
        if (lane == 0 && part == 0) raise_err(a.err, FOCUS_DEVERR_PAGE_ID);
        slot = -1;
    }
    const int page = slot < 0 ? 0 : slot / p.page_size, at = slot < 0 ? 0 : slot - page * p.page_size;
    const int hl = lane % LPH, hw = lane / LPH, c0 = hl * V;
    float cn[V], sn[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const double t = (double)pos * a.freq_over_pi[c0 + i];
        sincospif((float)(t - 2.0 * rint(0.5 * t)), &sn[i], &cn[i]);
    }
    const int heads = a.Hq + 2 * a.Hkv;
    const T* q = reinterpret_cast<const T*>(p.q) + (long long)row * p.q_stride;
    const T* k = reinterpret_cast<const T*>(p.k) + (long long)row * p.k_stride;
    const T* v = reinterpret_cast<const T*>(p.v) + (long long)row * p.v_stride;
    T* out = reinterpret_cast<T*>(p.q_out) + (long long)row * p.out_stride;
    T* pool = reinterpret_cast<T*>(p.kv_pool);
    const int step = warps_per_row * HPW;
#pragma unroll 4
    for (int h0 = part * HPW; h0 < heads; h0 += step) {
        const int h = h0 + hw;
        const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv, live = h < heads;
        const T* src = is_q ? q + h * D : is_k ? k + (h - a.Hq) * D : v + (h - a.Hq - a.Hkv) * D;
        P lo, hi;
        lo.u = hi.u = make_uint4(0, 0, 0, 0);
        if (live) {
            lo.u = *reinterpret_cast<const uint4*>(src + c0);
            hi.u = *reinterpret_cast<const uint4*>(src + D / 2 + c0);
        }
        const T* gain = reinterpret_cast<const T*>(is_q ? p.q_norm : p.k_norm);
        const bool norm = (is_q || is_k) && gain != nullptr;
        float x[V], y[V];
        lo.get(x);
        hi.get(y);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (is_q || is_k) {
            if (norm) {
                const float inv = rsqrtf(ss / D + p.eps);
                P gl, gh;
                gl.u = __ldg(reinterpret_cast<const uint4*>(gain + c0));
                gh.u = __ldg(reinterpret_cast<const uint4*>(gain + D / 2 + c0));
                float g0[V], g1[V];
                gl.get(g0);
                gh.get(g1);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    x[i] *= inv * g0[i];
                    y[i] *= inv * g1[i];
                }
            }
            float r0[V], r1[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                r0[i] = x[i] * cn[i] - y[i] * sn[i];
                r1[i] = y[i] * cn[i] + x[i] * sn[i];
            }
            lo.set(r0);
            hi.set(r1);
        }
        if (!live) continue;
        T* dst = out + h * D;
        if (!is_q) {
            if (slot < 0) continue;
            const int kv = is_k ? 0 : 1, g = h - a.Hq - kv * a.Hkv;
            dst = pool + (((((size_t)page * a.L + p.layer) * 2 + kv) * a.Hkv + g) * p.page_size + at) * D;
        }
        *reinterpret_cast<uint4*>(dst + c0) = lo.u;
        *reinterpret_cast<uint4*>(dst + D / 2 + c0) = hi.u;
    }
}

}  // namespace

template <typename T, int D> int launch_chunk_qk(const ChunkQkDev& a, cudaStream_t s) {
    constexpr int HPW = 32 / (D / 2 / (16 / (int)sizeof(T)));
    const int groups = (a.Hq + 2 * a.Hkv + HPW - 1) / HPW;
    // one warp per row once the rows fill the SMs (32 warps each); fewer rows are shared by several warps
    const int fill = kChunkCtas * 32;
    int wpr = a.p.rows >= fill ? 1 : (fill + a.p.rows - 1) / a.p.rows;
    wpr = wpr < groups ? wpr : groups;
    const long long warps = (long long)a.p.rows * wpr;
    const int per = kThreads / 32;
    return launched(launch_pdl(chunk_qk_kernel<T, D>, dim3((unsigned)((warps + per - 1) / per)), dim3(kThreads), 0, s, 0,
                               a, wpr));
}

template int launch_chunk_qk<float, 64>(const ChunkQkDev&, cudaStream_t);
template int launch_chunk_qk<float, 128>(const ChunkQkDev&, cudaStream_t);
template int launch_chunk_qk<bf16, 128>(const ChunkQkDev&, cudaStream_t);

}  // namespace focus
