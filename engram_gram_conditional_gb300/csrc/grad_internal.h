// Internal declarations of the training operators: their kernels' launchers
// (kernels_grad.cu, kernels_few.cu, kernels_embed.cu, kernels_gate.cu) as
// grad_api.cpp calls them.
#pragma once

#include "engram_internal.h"

namespace engram {

enum GradEpilogue : int {
    kGradLse = 0,  // softmax statistics of the logits
    kGradDz = 1,   // dz of a piece of the vocabulary, BF16, in 128 x 64 tiles
    kGradOut = 2,  // a product's output
};

// The loss's dz is kept as (exp(z - lse) - [v = label]) dloss[t] / unit, and the
// products are multiplied by the unit: with equal weights, the usual case, the
// large term of every row is then close to -1 and rounds almost exactly, where
// -1 / T (every row with the same error of up to 2^-8) would scale the whole
// gradient.
#ifdef __CUDACC__
__device__ __forceinline__ float loss_unit(const float* dloss) {
    const float u = dloss[0], size = fabsf(u);
    return size >= 0x1p-30f && size <= 0x1p30f ? u : 1.0f;
}
#endif

struct FastDiv {
    uint32_t d, m, s;  // divisor, multiplier, shift
};

// One matrix product out [M][N] (BF16) of a launch, reduced over kb blocks of 64.
struct GradProblem {
    int m_units, n_tiles;  // 256-row units, 256-column tiles
    int kb, splits;        // k-blocks; the reduction is cut into `splits` items
    int items;             // m_units * n_tiles * splits (set by the launcher)
    int a_mn;              // A is stored with M contiguous
    int a_tiled;           // A in 128 x 64 tiles: tiles per row of tiles (0: row-major)
    int group_m;           // item order: groups of group_m units, M inner
    FastDiv per_split, per_group, in_group, in_last;  // (set by the launcher)
    int64_t M, N;          // bounds of the output; N a multiple of 8
    uint16_t* out;         // bf16 [M][N]
    float* acc;            // fp32 [splits][M][N]; acc_read: added to, acc_write: the
    int acc_read, acc_write;  // result stays there instead of going to out
};

struct GradArgs {
    GradProblem pr[2];
    int pairs_more, rounds_fewer;  // how the items are dealt (set by the launcher)
    uint32_t* err;
    long long wait_limit_ns;
    int starve;            // test hook: no operand is loaded
    const float* unit;     // kGradOut: outputs are multiplied by loss_unit(unit); null: by 1
    // softmax epilogues
    int64_t T, v0;         // rows; first vocabulary column of the piece
    int vocab, dz_chunks;  // 64-column chunks of the piece
    const int32_t* labels;
    const float* lse;
    const float* dloss;
    float* zlabel;
    float2* part;          // [2 n_tiles][T] (maximum, sum)
    uint16_t* dz;          // 128 x 64 tiles [row block][64-column chunk of the piece]
};

int grad_pairs();  // CTA pairs of a launch that fills the device
// tm: A and B of problem 0, A and B of problem 1
cudaError_t launch_grad_lse(GradArgs& a, const CUtensorMap* tm, cudaStream_t s);
cudaError_t launch_grad_dz(GradArgs& a, const CUtensorMap* tm, cudaStream_t s);
cudaError_t launch_grad_products(GradArgs& a, const CUtensorMap* tm, cudaStream_t s);
// ---- the loss's logits of at most kFewTokens tokens (kernels_few.cu) ----
constexpr int kFewTokens = 16;
struct FewArgs {
    int T, kb;             // tokens, blocks of 64 columns
    int rows, vocab;       // vocabulary rows of the piece, of the head
    int64_t v0;            // first of the piece
    const int32_t* labels;
    const float *lse, *dloss;
    float* zlabel;
    float2* part;          // [few_groups(rows)][T]
    uint16_t* dz;          // 128 x 64 tiles, one row of them; tokens 0..63 are written
    uint32_t* err;
    long long wait_limit_ns;
    int starve;
};
int few_groups(int64_t rows);
cudaError_t launch_few_lse(const FewArgs& a, const uint16_t* x, const uint16_t* head, int dim, cudaStream_t s);
// (head: its row v0)
cudaError_t launch_few_dz(const FewArgs& a, const uint16_t* x, const uint16_t* head, int dim, cudaStream_t s);

cudaError_t launch_loss_combine(const float2* part, int groups, int64_t T, const float* zlabel,
                                const int32_t* labels, int vocab, float* loss, float* lse,
                                uint32_t* err, cudaStream_t s);
cudaError_t launch_sum_splits(const float* acc, int splits, int64_t n, const float* unit,
                              uint16_t* out, cudaStream_t s);


// ---- embedding (kernels_embed.cu) ----
cudaError_t launch_embed(const void* table, bool f32, uint64_t rows, int dim, const uint32_t* ids,
                         int64_t n, float scale, int copies, uint16_t* out, uint32_t* err,
                         cudaStream_t s);
// The sort of n ids and its segments.
struct EmbedSort {
    const uint32_t* ids;
    int64_t n;
    uint64_t rows;           // ids at or above are not rows
    int passes, digit_bits;  // embed_sort_digits
    uint2 *pairs0, *pairs1;  // (id, position) [n]; the sorted one is number passes & 1
    uint32_t* hist;          // [2^digit_bits][blocks]
    uint32_t* digit_total;   // [2^digit_bits]
    uint32_t* block_heads;   // [blocks]
    uint32_t* barrier;       // arrivals; right behind it:
    uint32_t* failed;        // set where a wait ran out: the results are not whole
    uint32_t* n_valid;       // ids that are rows
    uint32_t* segpos;        // [n] segment of each sorted place
    uint32_t* seg_start;     // [n + 1] first place of each segment
    uint32_t* unique;        // [n] id of each segment
    uint32_t* count;         // segments
    uint32_t* err;
    long long wait_limit_ns;
    int starve;              // test hook: one block keeps its arrivals at the barriers back
};
int embed_sort_blocks(int64_t n);
void embed_sort_digits(uint64_t rows, int* passes, int* bits);
cudaError_t launch_embed_sort(const EmbedSort& a, cudaStream_t s);
// The rows' sums: grad[segment or, dense, its id] = scale x the sum of its rows of dout.
struct EmbedSum {
    const uint2* sorted;     // (id, position)
    const uint32_t *segpos, *seg_start, *unique, *n_valid, *failed;
    const uint16_t* dout;    // bf16 [n][copies][dim]
    int dim, copies;
    float scale;
    int dense, accumulate;
    float* grad;
    int rows_per_chunk;      // embed_rows_per_chunk
    float* partial;          // [chunks][2][dim]
    int lanes, slices;       // set by the launcher
};
int embed_rows_per_chunk(int64_t n, int dim, int copies);
// Chunks of any number of copies and at most n ids.
int64_t embed_most_chunks(int64_t n, int dim);
cudaError_t launch_embed_sum(EmbedSum a, int64_t n, cudaStream_t s);

// ---- gate (kernels_gate.cu) ----
enum SavedKind : int { kSavedF32 = 0, kSavedBf16 = 1, kSavedMx = 2 };  // as ENGRAM_KV_*
struct GateTrain {
    int64_t T;
    int hc, d;
    float eps;
    const uint4* windows;
    const uint16_t* hidden;  // bf16 [T][hc][d]
    const void* kv;          // [T][(hc + 1) d]
    const float *wqk, *wq, *wk;
    // forward with checkpoint
    uint16_t* hidden_out;
    float* gates;
    uint8_t *codes_out, *scales_out;
    // backward
    const uint8_t *codes, *scales;
    const uint16_t* dout;
    uint16_t *dhidden, *dkv;
    float *dwq, *dwk;
    float4* factors;         // [T][hc]
    float* dw_part;          // [gate_backward_shares][hc][d]
    uint32_t* err;
    long long wait_limit_ns;
};
cudaError_t launch_gate_checkpoint(const GateTrain& a, bool kv_f32, cudaStream_t s);
int gate_backward_shares(int64_t T, int d);
cudaError_t launch_gate_backward(const GateTrain& a, int saved, cudaStream_t s);

}  // namespace engram
