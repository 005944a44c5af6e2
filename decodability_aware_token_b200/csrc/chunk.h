// Internal interface of the prompt-chunk operators: the API file (chunk_api.cu) checks the arguments and
// picks the kernels; each operator's kernels are in their own translation unit.
#pragma once
#include "launch.h"

namespace focus {

constexpr int kChunkCtas = 148;          // CTAs (one per SM of a B200) that share a split attention launch
constexpr int kChunkMaxRequests = 16384; // the plan and the attention schedule keep per-request sums in shared memory

struct ChunkPlanDev {
    focus_chunk_plan p;
    int max_pages;
    int* arrivals;   // [1] zero between launches
    int* err;
};
int launch_chunk_plan(const ChunkPlanDev& a, cudaStream_t s);
bool configure_chunk_plan_kernel();
// out[r] = the token of row r, at[r] its position (0 for rows of nobody); then prefix_len[b] = kv_len[b]
int launch_chunk_tokens(const focus_chunk_plan& p, const int32_t* tokens, int max_new, int32_t* out, int32_t* at, int* err,
                        cudaStream_t s);
const focus_chunk_cfg* chunk_cfg(const focus_chunk_ctx* c);
int64_t chunk_positions(const focus_chunk_ctx* c, int page_size);  // positions a page table row reaches

struct ChunkQkDev {
    focus_chunk_qk p;
    int L, Hq, Hkv;
    const double* freq_over_pi;  // [d / 2] theta^(-2i/d) / pi
    int* err;
};
template <typename T, int D> int launch_chunk_qk(const ChunkQkDev& a, cudaStream_t s);

struct ChunkAttnDev {
    const void* q;
    void* out;
    const void* kv_pool;
    const int32_t* row_offsets;
    const int32_t* kv_len;
    const int32_t* page_table;
    long long q_stride, out_stride;  // elements
    int N, rows, max_new, Hq, Hkv, G, L, layer, S, n_pages, max_pages, mask_block;
    float scale;
    // bf16: the few-row and the tile kernel both run in this call.  They share nothing, so the tile kernel does not wait for
    // the other one: its CTAs start as the SMs come free, and it only waits at its end, so that who waits for it
    // has waited for both (40 single tokens and 8 chunks, short runs: 308 -> 292 us).
    bool pair;
    bool small_walk;  // the launch's key blocks fit 31 bits, as long as the requests' row ranges do not overlap
    // scratch of units whose key walk is split over CTAs: slot 2c / 2c + 1 is CTA c's first / last piece
    float* part_o;
    float* part_ml;
    int* counters;   // arrivals at the unit (tile kernel: at each of its two tiles) whose first piece is CTA c's; zero
                     // between launches
    int* err;
};
// bf16 models: requests of at most kChunkFewRows query vectors per KV head (single tokens) go to one kernel, the others
// to the tile kernel.  16 is what one mma.sync tile holds.  Measured over seconds, few / tile kernel, 32/8 heads: 256 single
// tokens 216 / 319 us (1.80 / 1.69 GHz), 256 requests of 4 tokens (16 vectors) 242 / 327, 32 of them 48 / 55.
constexpr int kChunkFewRows = 16;
constexpr int kChunkTileRows = 256;  // query vectors per unit of the tile kernel
int launch_chunk_attention_few(const ChunkAttnDev& a, int sms, cudaStream_t s);
bool configure_chunk_attention_few();
int launch_chunk_attention_tile(const ChunkAttnDev& a, int sms, cudaStream_t s);
bool configure_chunk_attention_tile();

// CUDA-core kernels: float32 models
constexpr int kChunkSimtCtas = 2 * kChunkCtas;
constexpr int kChunkSimtRows = 64, kChunkSimtFew = 8;  // query vectors per unit of the two shapes
template <typename T, int D> int launch_chunk_attention_simt(const ChunkAttnDev& a, int sms, cudaStream_t s);
bool configure_chunk_attention_simt();

}  // namespace focus
