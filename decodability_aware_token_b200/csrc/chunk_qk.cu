// Per-head RMSNorm of queries and keys, rotate-half RoPE and the write into the paged cache, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * gain
//   (y_i, y_{i + d/2}) -> (y_i c - y_{i + d/2} s, y_{i + d/2} c + y_i s),  c + i s = exp(i pos theta^(-2i/d))
//
// Bound by memory: each of the (Hq + 2 Hkv) d values of a row is read once and written once (16384 rows of 32/8
// heads, bf16, over seconds: 73.6 us at 1.78 GHz = 5.5 TB/s, 84 % of the copy rate; with two groups of heads in flight per
// warp 90 us, since registers spill).  A lane holds 16 bytes of a head's lower half and the 16 bytes of the same pairs in its upper half, so the rotation needs
// no exchange and every access is a full 16 bytes; D / 2 / (16 bytes) lanes form a head and a warp works
// on several heads of one row at once.  A row's angles are computed once per warp and used for all its heads:
// pos / pi theta^(-2i/d) in double, less the nearest quarter turn, which leaves [-1/4, 1/4] exactly, then rounded to
// float32 (off by at most 2^-27 half turns, 2.4e-8 radians; four times that if whole turns alone were taken off) for
// sincospif.  (Float angles lose pos 2^-24 radians: 4e-3 at position 65536.)  The result is rounded once, to T.
#include "chunk.h"

namespace focus {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 1;  // groups of heads whose loads are in flight while one is turned

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
__global__ void __launch_bounds__(kThreads, 12) chunk_qk_kernel(ChunkQkDev a, int warps_per_row) {
    constexpr int V = 16 / (int)sizeof(T);      // values per access
    constexpr int LPH = D / 2 / V;              // lanes per head
    constexpr int HPW = 32 / LPH;               // heads a warp works on at once
    using P = Pack<T, V>;
    __shared__ __align__(16) float cos_s[kThreads / 32][D / 2], sin_s[kThreads / 32][D / 2];
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
    // groups of HPW heads: the query heads', the key heads', the value heads' (none straddles)
    const int gq = (a.Hq + HPW - 1) / HPW, gk = (a.Hkv + HPW - 1) / HPW, groups = gq + 2 * gk;
    const T* q = reinterpret_cast<const T*>(p.q) + (long long)row * p.q_stride + c0;
    const T* k = reinterpret_cast<const T*>(p.k) + (long long)row * p.k_stride + c0;
    const T* v = reinterpret_cast<const T*>(p.v) + (long long)row * p.v_stride + c0;
    P lo[kAhead], hi[kAhead];
    auto fetch = [&](int g, P& l, P& u) {
        const int kind = g < gq ? 0 : g < gq + gk ? 1 : 2;
        const int h = (kind == 0 ? g : kind == 1 ? g - gq : g - gq - gk) * HPW + hw;
        const T* src = (kind == 0 ? q : kind == 1 ? k : v) + h * D;
        l.u = u.u = make_uint4(0, 0, 0, 0);
        if (g < groups && h < (kind == 0 ? a.Hq : a.Hkv)) {
            l.u = *reinterpret_cast<const uint4*>(src);
            u.u = *reinterpret_cast<const uint4*>(src + D / 2);
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(part + i * warps_per_row, lo[i], hi[i]);

    // the row's angles, D / 64 pairs per lane, to shared memory
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = lane; i < D / 2; i += 32) {
        const double t = (double)pos * a.freq_over_pi[i];
        const long long turn = __double2ll_rn(2.0 * t);  // quarter turns
        float s, c;
        sincospif((float)(t - 0.5 * (double)turn), &s, &c);
        const float x = turn & 1 ? s : c, y = turn & 1 ? c : s;  // a quarter turn: (c, s) -> (-s, c)
        cos_s[warp][i] = (turn + 1) & 2 ? -x : x;
        sin_s[warp][i] = turn & 2 ? -y : y;
    }
    __syncwarp();
    T* out = reinterpret_cast<T*>(p.q_out) + (long long)row * p.out_stride + c0;
    T* pool = reinterpret_cast<T*>(p.kv_pool) +
              (((size_t)page * a.L + p.layer) * 2 * a.Hkv * p.page_size + at) * D + c0;  // K of head 0 at this slot
    const size_t head_step = (size_t)p.page_size * D;
    auto turn = [&](int g, P& l, P& u) {
        const int kind = g < gq ? 0 : g < gq + gk ? 1 : 2;
        const int h = (kind == 0 ? g : kind == 1 ? g - gq : g - gq - gk) * HPW + hw;
        if (kind < 2) {
            float x[V], y[V];
            l.get(x);
            u.get(y);
            const T* gain = reinterpret_cast<const T*>(kind == 0 ? p.q_norm : p.k_norm);
            if (gain != nullptr) {
                P gl, gh;
                gl.u = __ldg(reinterpret_cast<const uint4*>(gain + c0));
                gh.u = __ldg(reinterpret_cast<const uint4*>(gain + D / 2 + c0));
                float ss = 0.f, st = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    ss = fmaf(x[j], x[j], ss);
                    st = fmaf(y[j], y[j], st);
                }
                ss += st;
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float inv = rsqrtf(ss * (1.f / D) + p.eps);
                float g0[V], g1[V];
                gl.get(g0);
                gh.get(g1);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    x[j] *= inv * g0[j];
                    y[j] *= inv * g1[j];
                }
            }
            float r0[V], r1[V];
#pragma unroll
            for (int j = 0; j < V; j += 4) {
                const float4 c4 = *reinterpret_cast<const float4*>(&cos_s[warp][c0 + j]);
                const float4 s4 = *reinterpret_cast<const float4*>(&sin_s[warp][c0 + j]);
                const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    r0[j + e] = x[j + e] * c[e] - y[j + e] * s[e];
                    r1[j + e] = y[j + e] * c[e] + x[j + e] * s[e];
                }
            }
            l.set(r0);
            u.set(r1);
        }
        if (h >= (kind == 0 ? a.Hq : a.Hkv) || (kind > 0 && slot < 0)) return;
        T* dst = kind == 0 ? out + h * D : pool + (h + (kind == 2 ? a.Hkv : 0)) * head_step;
        *reinterpret_cast<uint4*>(dst) = l.u;
        *reinterpret_cast<uint4*>(dst + D / 2) = u.u;
    };
    for (int g = part; g < groups; g += kAhead * warps_per_row) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int gi = g + i * warps_per_row;
            if (gi >= groups) break;  // (the whole warp)
            turn(gi, lo[i], hi[i]);
            fetch(gi + kAhead * warps_per_row, lo[i], hi[i]);
        }
    }
}

}  // namespace

template <typename T, int D> int launch_chunk_qk(const ChunkQkDev& a, cudaStream_t s) {
    constexpr int HPW = 32 / (D / 2 / (16 / (int)sizeof(T)));
    const int groups = (a.Hq + HPW - 1) / HPW + 2 * ((a.Hkv + HPW - 1) / HPW);
    // One warp per row once the rows fill the SMs (32 warps each); fewer rows are shared by several warps.  Measured, 32/8
    // heads, one warp per row / this rule / a warp per group of heads: 1024 rows 10.6 / 8.0 / 8.4 us, 4096 rows 28.7 / 20.6 /
    // 28.7, 6000 rows 29.7 / 29.7 / 41.2; 32 rows of 16/8 heads 6.2 / 2.5 / 2.5.
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
