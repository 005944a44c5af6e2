// C ABI of the prompt-chunk operators: validation, workspace, and the choice of kernels.
#include <math.h>

#include <new>
#include <vector>

#include <nvtx3/nvToolsExt.h>  // header-only; ranges are no-ops unless a profiler is attached

#include "chunk.h"

using namespace focus;

struct focus_chunk_ctx {
    focus_chunk_cfg cfg;
    focus_chunk_limits lim;
    int device, sms;
    void* ws;
    double* freq_over_pi;
    int* err;
    int* arrivals;
    float *part_o, *part_ml;
    int* counters;
};

const focus_chunk_cfg* focus::chunk_cfg(const focus_chunk_ctx* c) { return &c->cfg; }
int64_t focus::chunk_positions(const focus_chunk_ctx* c, int page_size) { return (int64_t)c->lim.max_pages_per_req * page_size; }

namespace {

bool cfg_ok(const focus_chunk_cfg* c) {
    return c && c->n_layers >= 1 && c->n_q_heads >= 1 && c->n_kv_heads >= 1 && c->n_q_heads % c->n_kv_heads == 0 &&
           (c->dtype == FOCUS_DTYPE_F32 || c->dtype == FOCUS_DTYPE_BF16) && c->rope_theta > 0.f && isfinite(c->rope_theta);
}
int cfg_supported(const focus_chunk_cfg* c) {
    if (c->head_dim != 128 && !(c->head_dim == 64 && c->dtype == FOCUS_DTYPE_F32)) return FOCUS_ERR_UNSUPPORTED;
    if (c->n_q_heads / c->n_kv_heads > 64) return FOCUS_ERR_UNSUPPORTED;
    return FOCUS_OK;
}
bool lim_ok(const focus_chunk_limits* l) { return l && l->max_requests >= 1 && l->max_pages_per_req >= 1; }

struct Layout {
    size_t freq, words, part_o, part_ml, total;
};
size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// words: error word, plan arrivals, attention counters (all zero between calls)
Layout plan_layout(const focus_chunk_cfg* c) {
    const size_t vecs = c->dtype == FOCUS_DTYPE_BF16 ? (size_t)2 * kChunkCtas * (kChunkTileRows + kChunkFewRows)
                                                     : (size_t)2 * kChunkSimtCtas * (kChunkSimtRows + kChunkSimtFew);
    Layout l{};
    l.freq = 0;
    l.words = align_up(l.freq + (size_t)c->head_dim / 2 * 8, 256);
    l.part_ml = align_up(l.words + (2 + (size_t)2 * kChunkSimtCtas) * 4, 256);
    l.part_o = align_up(l.part_ml + vecs * 2 * 4, 256);
    l.total = align_up(l.part_o + vecs * c->head_dim * 4, 256);
    return l;
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t elt_of(const focus_chunk_ctx* c) { return c->cfg.dtype == FOCUS_DTYPE_BF16 ? 2 : 4; }

bool device_ok(const focus_chunk_ctx* c) {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess && dev == c->device;
}

// rows of `heads` dense heads, `stride` elements apart, 16-byte aligned
bool rows_ok(const focus_chunk_ctx* c, const void* p, int64_t stride, int heads) {
    return p && aligned(p, 16) && stride >= (int64_t)heads * c->cfg.head_dim && stride * (int64_t)elt_of(c) % 16 == 0 &&
           stride < ((int64_t)1 << 40);
}

// The bytes of `rows` rows of `heads` heads, `stride` elements apart.
struct Span {
    uintptr_t at, end, step, len;
};
Span span_of(const focus_chunk_ctx* c, const void* p, int64_t stride, int heads, int rows) {
    const uintptr_t e = elt_of(c), at = reinterpret_cast<uintptr_t>(p), len = (uintptr_t)heads * c->cfg.head_dim * e,
                    step = (uintptr_t)stride * e;
    return {at, at + (uintptr_t)(rows - 1) * step + len, step, len};
}
// Do two sets of rows share a byte?  Views of one buffer have the same step, and their rows lie side by side or do not;
// rows that interleave at different steps count as sharing.
bool share(const Span& x, const Span& y) {
    if (x.end <= y.at || y.end <= x.at) return false;
    if (x.step != y.step) return true;
    const uintptr_t d = y.at >= x.at ? (y.at - x.at) % x.step : (x.step - (x.at - y.at) % x.step) % x.step;
    return d < x.len || d + y.len > x.step;
}
bool in_pool(const focus_chunk_ctx* c, const Span& x, const void* pool, int64_t n_pages, int64_t page_size) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(pool), bytes = (uintptr_t)n_pages * (uintptr_t)c->cfg.n_layers * 2 *
                                                                   c->cfg.n_kv_heads * (uintptr_t)page_size * c->cfg.head_dim * elt_of(c);
    return x.at < at + bytes && at < x.end;
}

struct Range {
    explicit Range(const char* n) { nvtxRangePushA(n); }
    ~Range() { nvtxRangePop(); }
};

}  // namespace

extern "C" {

size_t focus_chunk_workspace_bytes(const focus_chunk_cfg* cfg, const focus_chunk_limits* lim) {
    if (!cfg_ok(cfg) || cfg_supported(cfg) != FOCUS_OK || !lim_ok(lim)) return 0;
    return plan_layout(cfg).total;
}

int focus_chunk_init(const focus_chunk_cfg* cfg, const focus_chunk_limits* lim, focus_chunk_ctx** out) {
    if (!out) return FOCUS_ERR_INVALID_ARG;
    *out = nullptr;
    if (!cfg_ok(cfg) || !lim_ok(lim)) return FOCUS_ERR_INVALID_ARG;
    const int sup = cfg_supported(cfg);
    if (sup != FOCUS_OK) return sup;
    if (lim->max_requests > kChunkMaxRequests) return FOCUS_ERR_LIMITS;
    focus_chunk_ctx* c = new (std::nothrow) focus_chunk_ctx();
    if (!c) return FOCUS_ERR_NO_MEMORY;
    c->cfg = *cfg;
    c->lim = *lim;
    if (cudaGetDevice(&c->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&c->sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess) {
        (void)cudaGetLastError();
        delete c;
        return FOCUS_ERR_CUDA;
    }
    const Layout l = plan_layout(cfg);
    if (cudaMalloc(&c->ws, l.total) != cudaSuccess) {
        (void)cudaGetLastError();
        delete c;
        return FOCUS_ERR_NO_MEMORY;
    }
    char* base = static_cast<char*>(c->ws);
    c->freq_over_pi = reinterpret_cast<double*>(base + l.freq);
    c->err = reinterpret_cast<int*>(base + l.words);
    c->arrivals = c->err + 1;
    c->counters = c->err + 2;
    c->part_ml = reinterpret_cast<float*>(base + l.part_ml);
    c->part_o = reinterpret_cast<float*>(base + l.part_o);
    double freq[64];
    for (int i = 0; i < cfg->head_dim / 2; ++i)
        freq[i] = pow((double)cfg->rope_theta, -2.0 * i / cfg->head_dim) / 3.14159265358979323846;
    if (cudaMemcpy(c->freq_over_pi, freq, (size_t)cfg->head_dim / 2 * 8, cudaMemcpyHostToDevice) != cudaSuccess ||
        cudaMemset(c->err, 0, l.part_ml - l.words) != cudaSuccess || !configure_chunk_plan_kernel() ||
        !configure_chunk_attention_simt() || !configure_chunk_attention_few() ||
        !configure_chunk_attention_tile() || cudaDeviceSynchronize() != cudaSuccess) {
        (void)cudaGetLastError();
        cudaFree(c->ws);
        delete c;
        return FOCUS_ERR_CUDA;
    }
    *out = c;
    return FOCUS_OK;
}

int focus_chunk_destroy(focus_chunk_ctx* c) {
    if (!c) return FOCUS_OK;
    int prev = -1;
    cudaGetDevice(&prev);
    int rc = FOCUS_OK;
    if (cudaSetDevice(c->device) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) rc = FOCUS_ERR_CUDA;
    if (cudaFree(c->ws) != cudaSuccess) rc = FOCUS_ERR_CUDA;
    if (prev >= 0) cudaSetDevice(prev);
    delete c;
    return rc;
}

int focus_chunk_get_device_error(focus_chunk_ctx* c, int32_t* bits) {
    if (bits) *bits = 0;
    if (!c) return FOCUS_ERR_INVALID_ARG;
    int prev = -1, v = 0;
    cudaGetDevice(&prev);
    bool ok = cudaSetDevice(c->device) == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess &&
              cudaMemcpy(&v, c->err, 4, cudaMemcpyDeviceToHost) == cudaSuccess;
    // a launch that gave up may have left arrivals behind: the counters are zero again as well
    const Layout l = plan_layout(&c->cfg);
    const size_t words = (v & FOCUS_DEVERR_TIMEOUT) ? l.part_ml - l.words : sizeof(int);
    ok = ok && cudaMemset(c->err, 0, words) == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess;
    if (prev >= 0) cudaSetDevice(prev);
    if (!ok) return FOCUS_ERR_CUDA;
    if (bits) *bits = v;
    if (v == 0) return FOCUS_OK;
    return (v & FOCUS_DEVERR_TIMEOUT) ? FOCUS_ERR_TIMEOUT : FOCUS_ERR_DEVICE_BOUNDS;
}

int focus_chunk_plan_rows(focus_chunk_ctx* c, const focus_chunk_plan* p, void* stream) {
    if (!c || !p) return FOCUS_ERR_INVALID_ARG;
    if (p->n_requests < 0 || p->max_rows < 0 || p->page_size < 1 || p->n_pages < 0 || p->n_free < 0)
        return FOCUS_ERR_INVALID_ARG;
    if (p->n_requests > c->lim.max_requests || (int64_t)p->n_pages * p->page_size >= ((int64_t)1 << 31) ||
        (int64_t)c->lim.max_pages_per_req * p->page_size > ((int64_t)1 << 30))
        return FOCUS_ERR_LIMITS;
    if (!p->free_head || !p->row_offsets || !p->free_next || (p->n_free > 0 && !p->free_pages) ||
        (p->max_rows > 0 && (!p->row_req || !p->row_pos || !p->row_slot)))
        return FOCUS_ERR_INVALID_ARG;
    if (p->n_requests > 0 && (!p->prefix_len || !p->new_len || !p->page_table || !p->kv_len || p->kv_len == p->prefix_len ||
                              p->kv_len == p->new_len || p->row_offsets == p->prefix_len || p->row_offsets == p->new_len))
        return FOCUS_ERR_INVALID_ARG;
    const void* words[] = {p->prefix_len, p->new_len, p->page_table, p->free_pages, p->free_head, p->row_offsets,
                           p->kv_len, p->row_req, p->row_pos, p->row_slot, p->free_next};
    for (const void* w : words)
        if (!aligned(w, 4)) return FOCUS_ERR_INVALID_ARG;
    if (!device_ok(c)) return FOCUS_ERR_INVALID_ARG;
    Range range("chunk_plan");
    const ChunkPlanDev a{*p, c->lim.max_pages_per_req, c->arrivals, c->err};
    return launch_chunk_plan(a, static_cast<cudaStream_t>(stream)) < 0 ? FOCUS_ERR_CUDA : FOCUS_OK;
}

int focus_chunk_qk_norm_rope(focus_chunk_ctx* c, const focus_chunk_qk* p, void* stream) {
    if (!c || !p) return FOCUS_ERR_INVALID_ARG;
    if (p->rows < 0 || p->layer < 0 || p->layer >= c->cfg.n_layers || p->page_size < 1 || p->n_pages < 0 ||
        !(p->eps >= 0.f))
        return FOCUS_ERR_INVALID_ARG;
    if ((int64_t)p->n_pages * p->page_size >= ((int64_t)1 << 31)) return FOCUS_ERR_LIMITS;
    if (p->rows == 0) return FOCUS_OK;
    const int hq = c->cfg.n_q_heads, hkv = c->cfg.n_kv_heads;
    if (!rows_ok(c, p->q, p->q_stride, hq) || !rows_ok(c, p->k, p->k_stride, hkv) || !rows_ok(c, p->v, p->v_stride, hkv) ||
        !rows_ok(c, p->q_out, p->out_stride, hq))
        return FOCUS_ERR_INVALID_ARG;
    const Span out = span_of(c, p->q_out, p->out_stride, hq, p->rows);
    const bool in_place = p->q_out == p->q && p->out_stride == p->q_stride;
    if ((!in_place && share(out, span_of(c, p->q, p->q_stride, hq, p->rows))) ||
        share(out, span_of(c, p->k, p->k_stride, hkv, p->rows)) || share(out, span_of(c, p->v, p->v_stride, hkv, p->rows)) ||
        in_pool(c, out, p->kv_pool, p->n_pages, p->page_size))
        return FOCUS_ERR_INVALID_ARG;
    if (!p->row_pos || !p->row_slot || !aligned(p->row_pos, 4) || !aligned(p->row_slot, 4) ||
        (p->n_pages > 0 && !p->kv_pool) || !aligned(p->kv_pool, 16) || !aligned(p->q_norm, 16) || !aligned(p->k_norm, 16))
        return FOCUS_ERR_INVALID_ARG;
    if (!device_ok(c)) return FOCUS_ERR_INVALID_ARG;
    Range range("chunk_qk_norm_rope");
    const ChunkQkDev a{*p, c->cfg.n_layers, hq, hkv, c->freq_over_pi, c->err};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int n = c->cfg.dtype == FOCUS_DTYPE_BF16 ? launch_chunk_qk<bf16, 128>(a, s)
                  : c->cfg.head_dim == 64          ? launch_chunk_qk<float, 64>(a, s)
                                                   : launch_chunk_qk<float, 128>(a, s);
    return n < 0 ? FOCUS_ERR_CUDA : FOCUS_OK;
}

int focus_chunk_attention(focus_chunk_ctx* c, const focus_chunk_attn* p, void* stream) {
    if (!c || !p) return FOCUS_ERR_INVALID_ARG;
    if (p->n_requests < 0 || p->rows < 0 || p->max_new < 1 || p->page_size < 1 || p->n_pages < 0 || p->layer < 0 ||
        p->layer >= c->cfg.n_layers || p->mask_block < 1 || !(p->scale >= 0.f) || !isfinite(p->scale))
        return FOCUS_ERR_INVALID_ARG;
    const int64_t max_kv = (int64_t)c->lim.max_pages_per_req * p->page_size;
    // rows of the pool are addressed by 32-bit TMA coordinates
    const int64_t pool_rows = (int64_t)p->n_pages * c->cfg.n_layers * 2 * c->cfg.n_kv_heads;
    if (p->n_requests > c->lim.max_requests || max_kv > ((int64_t)1 << 30) ||
        pool_rows >= ((int64_t)1 << 31) / p->page_size)
        return FOCUS_ERR_LIMITS;
    const bool bf = c->cfg.dtype == FOCUS_DTYPE_BF16;
    if (bf && p->page_size != 16 && p->page_size != 32 && p->page_size != 64) return FOCUS_ERR_UNSUPPORTED;
    if (p->n_requests == 0 || p->rows == 0) return FOCUS_OK;
    const int hq = c->cfg.n_q_heads, hkv = c->cfg.n_kv_heads;
    if (!rows_ok(c, p->q, p->q_stride, hq) || !rows_ok(c, p->out, p->out_stride, hq) ||
        !p->row_offsets || !p->kv_len || !p->page_table || !aligned(p->row_offsets, 4) || !aligned(p->kv_len, 4) ||
        !aligned(p->page_table, 4) || (p->n_pages > 0 && !p->kv_pool) || !aligned(p->kv_pool, 16))
        return FOCUS_ERR_INVALID_ARG;
    const Span out = span_of(c, p->out, p->out_stride, hq, p->rows);
    if (share(out, span_of(c, p->q, p->q_stride, hq, p->rows)) || in_pool(c, out, p->kv_pool, p->n_pages, p->page_size))
        return FOCUS_ERR_INVALID_ARG;
    if (!device_ok(c)) return FOCUS_ERR_INVALID_ARG;
    ChunkAttnDev a{};
    a.q = p->q;
    a.out = p->out;
    a.kv_pool = p->kv_pool;
    a.row_offsets = p->row_offsets;
    a.kv_len = p->kv_len;
    a.page_table = p->page_table;
    a.q_stride = p->q_stride;
    a.out_stride = p->out_stride;
    a.N = p->n_requests;
    a.rows = p->rows;
    a.max_new = p->max_new < p->rows ? p->max_new : p->rows;
    a.Hq = hq;
    a.Hkv = hkv;
    a.G = hq / hkv;
    a.L = c->cfg.n_layers;
    a.layer = p->layer;
    a.S = p->page_size;
    a.n_pages = p->n_pages;
    a.max_pages = c->lim.max_pages_per_req;
    // a block that holds every position a request can reach: the mask is the same, the products fit
    a.mask_block = p->mask_block < max_kv ? p->mask_block : (int)max_kv;
    a.scale = p->scale > 0.f ? p->scale : 1.f / sqrtf((float)c->cfg.head_dim);
    // (a unit is at least one row of one request and a key block at least 32 keys)
    a.small_walk = (double)hkv * ((double)p->rows + p->n_requests) * ((double)max_kv / 32 + 1) < 2147483648.0;
    a.part_o = c->part_o;
    a.part_ml = c->part_ml;
    a.counters = c->counters;
    a.err = c->err;
    Range range("chunk_attention");
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    int n;
    if (bf) {
        // each kernel serves the requests on its side of kChunkFewRows query vectors and skips the others
        const bool tile = (int64_t)a.max_new * a.G > kChunkFewRows;
        const bool few = a.G <= kChunkFewRows;
        a.pair = few && tile;
        ChunkAttnDev f = a;
        f.part_o += (size_t)2 * kChunkCtas * kChunkTileRows * c->cfg.head_dim;
        f.part_ml += (size_t)2 * kChunkCtas * kChunkTileRows * 2;
        f.counters += 2 * kChunkCtas;
        n = few ? launch_chunk_attention_few(f, c->sms, s) : 0;
        if (n >= 0 && tile) n = launch_chunk_attention_tile(a, c->sms, s);
    } else {
        n = c->cfg.head_dim == 64 ? launch_chunk_attention_simt<float, 64>(a, c->sms, s)
                                  : launch_chunk_attention_simt<float, 128>(a, c->sms, s);
    }
    return n < 0 ? FOCUS_ERR_CUDA : FOCUS_OK;
}

}  // extern "C"
