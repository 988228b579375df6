// Host side of the training operators of libengram.so: the embedding and its
// gradient, the gate with an 8-bit checkpoint and its backward pass, the
// projection's backward pass, and the large-vocabulary loss (include/engram.h).
#include <algorithm>

#include "api_internal.h"
#include "grad_internal.h"

using namespace engram;

namespace {

// Carves a workspace into 256-byte aligned parts (the caller's pointer need only
// be 16-byte aligned); with a null base it only counts bytes.
struct Carver {
    uint8_t* base;
    size_t at = 0;
    explicit Carver(void* p)
        : base(reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 255) & ~(uintptr_t)255)) {}
    template <class T>
    T* take(size_t n) {
        T* p = base ? reinterpret_cast<T*>(base + at) : nullptr;
        at = (at + n * sizeof(T) + 255) & ~(size_t)255;
        return p;
    }
    size_t bytes() const { return at ? at + 240 : 0; }  // with what aligning the base may skip
};

// The current device, and the context's device word on it (a context that has
// no bound layer gets it here).
engram_status train_device(engram_ctx* ctx) {
    if (!ctx) return fail(ENGRAM_EINVAL, "null context");
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (ctx->device >= 0 && ctx->device != dev)
        return fail(ENGRAM_ESTATE, "context already bound on another device");
    return ensure_device_word(ctx, dev);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- embedding -------------------------------------------------------------------------

engram_status check_embed(uint64_t rows, uint32_t dim, int64_t n, uint32_t copies) {
    if (rows < 1 || rows >= 0xFFFFFFFFull) return fail(ENGRAM_EINVAL, "rows must be in [1, 2^32 - 2]");
    if (dim < 8 || dim % 8 || dim > 65536) return fail(ENGRAM_EINVAL, "dim must be a multiple of 8 in [8, 65536]");
    if (n < 0 || n > (int64_t)1 << 30) return fail(ENGRAM_EINVAL, "n must be in [0, 2^30]");
    if (copies < 1 || copies > 8) return fail(ENGRAM_EINVAL, "copies must be in [1, 8]");
    if ((uint64_t)n * copies >= 1ull << 32) return fail(ENGRAM_EINVAL, "n x copies must be below 2^32");
    return ENGRAM_OK;
}

struct EmbedWs {
    uint2 *pairs0, *pairs1;
    uint32_t *hist, *digit_total, *block_heads, *barrier, *n_valid,
        *segpos, *seg_start, *unique, *count;
    float* partial;
    size_t bytes;
};

EmbedWs embed_ws(void* p, int64_t n, uint64_t rows, uint32_t dim) {
    int passes, bits;
    embed_sort_digits(rows, &passes, &bits);
    const size_t blocks = embed_sort_blocks(n), bins = (size_t)1 << bits;
    Carver c(p);
    EmbedWs w{};
    w.pairs0 = c.take<uint2>(n);
    w.pairs1 = c.take<uint2>(n);
    w.hist = c.take<uint32_t>(blocks * bins);
    w.digit_total = c.take<uint32_t>(bins);
    w.block_heads = c.take<uint32_t>(blocks);
    w.barrier = c.take<uint32_t>(2);
    w.n_valid = c.take<uint32_t>(1);
    w.count = c.take<uint32_t>(1);
    w.segpos = c.take<uint32_t>(n);
    w.seg_start = c.take<uint32_t>(n + 1);
    w.unique = c.take<uint32_t>(n);
    w.partial = c.take<float>((size_t)embed_most_chunks(n, (int)dim) * 2 * dim);
    w.bytes = c.bytes();
    return w;
}

// ---- gate ------------------------------------------------------------------------------

GateTrain gate_args(const engram_ctx* ctx, int layer, const uint32_t* windows, int64_t T) {
    GateTrain a{};
    const LayerState& L = ctx->layers[layer];
    a.T = T;
    a.hc = (int)ctx->desc.hc;
    a.d = (int)ctx->desc.d;
    a.eps = (float)ctx->desc.eps;
    a.windows = reinterpret_cast<const uint4*>(windows);
    a.wqk = L.wqk;
    a.wq = L.w.wq;
    a.wk = L.w.wk;
    a.err = ctx->d_err;
    a.wait_limit_ns = ctx->wait_limit_ns;
    return a;
}

size_t gate_backward_ws(GateTrain* a, void* p, int64_t T, int hc, int d) {
    Carver c(p);
    float4* f = c.take<float4>((size_t)T * hc);
    float* part = c.take<float>((size_t)gate_backward_shares(std::max<int64_t>(T, 1), d) * hc * d);
    if (a) {
        a->factors = f;
        a->dw_part = part;
    }
    return c.bytes();
}

engram_status gate_backward_call(const engram_ctx* ctx, GateTrain& a, int saved, void* ws,
                                 cudaStream_t s) {
    const size_t nw = (size_t)a.hc * a.d * sizeof(float);
    if (a.T == 0) {
        cudaError_t e = cudaSuccess;
        if (a.dwq) e = cudaMemsetAsync(a.dwq, 0, nw, s);
        if (e == cudaSuccess && a.dwk) e = cudaMemsetAsync(a.dwk, 0, nw, s);
        return e == cudaSuccess ? ok() : cuda_fail(e, "gate backward of no tokens");
    }
    gate_backward_ws(&a, ws, a.T, a.hc, a.d);
    cudaError_t e = launch_gate_backward(a, saved, s);
    if (e != cudaSuccess) return cuda_fail(e, "gate backward launch");
    return ok();
}

// ---- products ----------------------------------------------------------------------------

GradArgs grad_args(const engram_ctx* ctx) {
    GradArgs a{};
    a.err = ctx->d_err;
    a.wait_limit_ns = ctx->wait_limit_ns;
    a.starve = ctx->starve_b;
    return a;
}

// One of the two gradient products of a launch.
GradProblem product(int64_t M, int64_t N, int64_t reduce, bool a_mn) {
    GradProblem q{};
    q.m_units = (int)ceil_div(M, 2 * kBM);
    q.n_tiles = (int)ceil_div(N, kBN);
    q.kb = (int)ceil_div(reduce, kBK);
    q.splits = 1;
    q.a_mn = a_mn;
    q.group_m = 8;
    q.M = M;
    q.N = N;
    return q;
}

// How often the long product's reduction is cut, so that its few tiles keep
// every pair busy: not at all while one item costs no more than a pair's mean
// share of the launch.
int long_splits(const GradProblem& lng, const GradProblem* shrt) {
    const double P = grad_pairs();
    const double tiles = (double)lng.m_units * lng.n_tiles;
    const double light = shrt ? (double)shrt->m_units * shrt->n_tiles * shrt->kb : 0.0;
    int best = 1;
    double best_t = 1e300;
    for (int s = 1; s <= 8 && s <= lng.kb; ++s) {
        const double item = (double)lng.kb / s;
        const double rounds = (double)ceil_div((int64_t)(tiles * s), (int64_t)P);
        const double mean = (tiles * lng.kb + light) / P;
        // parking and adding a split's partial sums costs about a k-block per item
        const double t = std::max(rounds * item, mean) + (s > 1 ? rounds * 2.0 + s : 0.0);
        if (t < best_t * 0.98) {
            best_t = t;
            best = s;
        }
    }
    return best;
}

// fp32 values that the cut products of any batch of at most T tokens park.  The cut
// follows the tokens in steps of a k-block, and there is none once demb's tiles go
// 50 times round the pairs: uncut, the last round then costs at most 2% of the mean
// share, and a cut never makes less than the mean share.
size_t project_parked(const engram_ctx* ctx, int64_t T) {
    int64_t most = 0;
    for (int64_t t = 0; t < T;) {
        t = std::min<int64_t>(T, t + kBK);
        const GradProblem demb = product(t, ctx->K, ctx->N, false);
        const GradProblem dw = product(ctx->N, ctx->K, t, true);
        if (demb.m_units * (int64_t)demb.n_tiles >= 50 * (int64_t)grad_pairs()) break;
        // with or without the other product the cut may differ: room for either
        const int splits = std::max(long_splits(demb, &dw), long_splits(demb, nullptr));
        if (splits > 1) most = std::max(most, splits * t);
    }
    return (size_t)most * ctx->K;
}

// ---- loss -------------------------------------------------------------------------------

engram_status check_loss(uint32_t vocab, uint32_t dim, int64_t T) {
    if (vocab < 1 || vocab > (1u << 30)) return fail(ENGRAM_EINVAL, "vocab must be in [1, 2^30]");
    if (dim < 8 || dim % 8 || dim > 65536) return fail(ENGRAM_EINVAL, "dim must be a multiple of 8 in [8, 65536]");
    return check_T(T);
}

// Column groups whose (maximum, sum) pairs a row's loss is joined from.
int loss_groups(int64_t T, uint32_t vocab) {
    return T <= kFewTokens ? few_groups(vocab) : (int)ceil_div(vocab, kBN) * 2;
}

// Room for any batch of at most T tokens (few of them may make more pairs than
// many: their vocabulary is cut finer).
struct LossWs {
    float2* part;
    float* zlabel;
    size_t bytes;
};
LossWs loss_ws(void* p, int64_t T, uint32_t vocab) {
    const int64_t few = std::min<int64_t>(T, kFewTokens);
    Carver c(p);
    LossWs w{};
    w.part = c.take<float2>((size_t)std::max(loss_groups(T, vocab) * T, loss_groups(few, vocab) * few));
    w.zlabel = c.take<float>(T);
    w.bytes = c.bytes();
    return w;
}

int loss_group_m(uint32_t dim) {  // M units whose x rows (40 MB) stay in L2 beside the head
    return (int)std::max<int64_t>(1, std::min<int64_t>(64, ((int64_t)40 << 20) / (512 * (int64_t)dim)));
}

// Vocabulary columns per piece of the backward pass: whole waves of z tiles
// while dz [T][piece] stays within half of L2, and at least one wave; at least 16
// tiles for a very long batch.
constexpr int64_t kPieceBytes = (int64_t)64 << 20, kPieceTiles = 16;
constexpr int64_t kDzTileBytes = 2 * kBM * kBN * 2;
int64_t loss_piece(int64_t T, uint32_t vocab) {
    const int64_t units = std::max<int64_t>(1, ceil_div(T, 2 * kBM)), P = grad_pairs();
    const int64_t all = ceil_div(vocab, kBN);
    const int64_t fit = kPieceBytes / (units * kDzTileBytes);  // tiles within 64 MB
    int64_t waves = fit * units / P;
    int64_t tiles = std::max<int64_t>(kPieceTiles, waves >= 1 ? waves * P / units : P / units);
    tiles = std::min(std::max<int64_t>(1, tiles), all);
    return tiles * kBN;
}

FewArgs few_args(const engram_ctx* ctx, int64_t T, uint32_t vocab, uint32_t dim) {
    FewArgs f{};
    f.T = (int)T;
    f.kb = (int)ceil_div(dim, kBK);
    f.vocab = (int)vocab;
    f.err = ctx->d_err;
    f.wait_limit_ns = ctx->wait_limit_ns;
    f.starve = ctx->starve_b;
    return f;
}

struct LossBackWs {
    uint16_t* dz;
    float* acc;
    int splits;
    size_t bytes;
};
GradProblem loss_dx(int64_t T, uint32_t dim, int64_t piece) {
    GradProblem q = product(T, dim, piece, false);
    q.a_tiled = (int)(piece / 64);
    return q;
}
GradProblem loss_dhead(int64_t T, uint32_t dim, int64_t cols, int64_t piece) {
    GradProblem q = product(cols, dim, T, true);
    q.a_tiled = (int)(piece / 64);
    return q;
}
// The cut of dx, before the splits' fp32 dx are held to 64 MB, as dz is.
int loss_splits(int64_t T, uint32_t vocab, uint32_t dim, bool want_dhead) {
    const int64_t piece = loss_piece(T, vocab);
    const GradProblem dx = loss_dx(T, dim, piece), dh = loss_dhead(T, dim, piece, piece);
    return long_splits(dx, want_dhead ? &dh : nullptr);
}
// fp32 values of dx that any batch of at most T tokens keeps between pieces (one dx)
// or parks (as project_parked; with and without the other product the cut may differ).
size_t loss_parked(int64_t T, uint32_t vocab, uint32_t dim) {
    const int64_t fit = kPieceBytes / (int64_t)sizeof(float);
    int64_t most = T * dim;
    for (int64_t t = 0; t < T && t * dim < fit;) {
        t = std::min<int64_t>(T, t + kBK);
        if (ceil_div(t, 2 * kBM) * ceil_div(dim, kBN) >= 50 * (int64_t)grad_pairs()) break;
        const int splits = std::max(loss_splits(t, vocab, dim, true), loss_splits(t, vocab, dim, false));
        most = std::max(most, std::min(fit, splits * t * dim));
    }
    return (size_t)most;
}
// Room for any batch of at most T tokens; acc, the last part, has loss_parked values.
LossBackWs loss_backward_ws(void* p, int64_t T, uint32_t vocab, uint32_t dim, bool want_dhead) {
    const int64_t units = ceil_div(T, 2 * kBM), P = grad_pairs();
    LossBackWs w{};
    const int fit = (int)std::max<int64_t>(1, kPieceBytes / (T * (int64_t)dim * 4));
    w.splits = std::min(fit, loss_splits(T, vocab, dim, want_dhead));
    Carver c(p);
    // units x tiles of dz (loss_piece): whole waves within 64 MB, one at least, or 16
    // tiles a unit, and no more than the vocabulary has
    const int64_t waves = std::max<int64_t>(1, kPieceBytes / kDzTileBytes / P) * P;
    w.dz = reinterpret_cast<uint16_t*>(c.take<uint8_t>(
        std::min(units * ceil_div(vocab, kBN), std::max(waves, units * kPieceTiles)) * kDzTileBytes));
    w.acc = c.take<float>(p ? 0 : loss_parked(T, vocab, dim));
    w.bytes = c.bytes();
    return w;
}

}  // namespace

extern "C" {

engram_status engram_embed(engram_ctx* ctx, const void* d_table, int table_format, uint64_t rows,
                           uint32_t dim, const uint32_t* d_ids, int64_t n, float scale,
                           uint32_t copies, uint16_t* d_out, void* stream) {
    engram_status st = check_embed(rows, dim, n, copies);
    if (st) return st;
    if (!ctx) return fail(ENGRAM_EINVAL, "null context");
    if (table_format != ENGRAM_EMBED_F32 && table_format != ENGRAM_EMBED_BF16)
        return fail(ENGRAM_EINVAL, "unknown table format");
    if (n == 0) return ok();
    if (!d_table || !d_ids || !d_out || !aligned16(d_table) || !aligned4(d_ids) || !aligned16(d_out))
        return fail(ENGRAM_EINVAL, "table, out (16-byte aligned) / ids");
    if ((st = train_device(ctx))) return st;
    cudaError_t e = launch_embed(d_table, table_format == ENGRAM_EMBED_F32, rows, (int)dim, d_ids, n,
                                 scale, (int)copies, d_out, ctx->d_err, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "embed launch");
    return ok();
}

size_t engram_embed_grad_workspace_bytes(int64_t n, uint64_t rows, uint32_t dim) {
    if (check_embed(rows, dim, n, 1)) return 0;
    return embed_ws(nullptr, n, rows, dim).bytes;
}

engram_status engram_embed_grad(engram_ctx* ctx, uint64_t rows, uint32_t dim, const uint32_t* d_ids,
                                int64_t n, float scale, uint32_t copies, const uint16_t* d_dout,
                                uint32_t* d_unique, uint32_t* d_count, float* d_grad,
                                int accumulate, void* d_workspace, void* stream) {
    engram_status st = check_embed(rows, dim, n, copies);
    if (st) return st;
    if (!ctx) return fail(ENGRAM_EINVAL, "null context");
    const bool dense = d_unique == nullptr;
    if (accumulate != 0 && accumulate != 1) return fail(ENGRAM_EINVAL, "accumulate must be 0 or 1");
    if (accumulate && !dense) return fail(ENGRAM_EINVAL, "only a dense gradient accumulates");
    if (!d_grad || !aligned16(d_grad) || (!dense && (!d_count || !aligned4(d_unique))) ||
        !aligned4(d_count))
        return fail(ENGRAM_EINVAL, "grad (16-byte aligned) / unique / count");
    if (n > 0 && (!d_ids || !d_dout || !d_workspace || !aligned4(d_ids) || !aligned16(d_dout) ||
                  !aligned16(d_workspace)))
        return fail(ENGRAM_EINVAL, "ids / dout, workspace (16-byte aligned)");
    if ((st = train_device(ctx))) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    if (dense && !accumulate) e = cudaMemsetAsync(d_grad, 0, rows * dim * sizeof(float), s);
    if (e == cudaSuccess && n == 0 && d_count) e = cudaMemsetAsync(d_count, 0, sizeof(uint32_t), s);
    if (e != cudaSuccess) return cuda_fail(e, "embed gradient clear");
    if (n == 0) return ok();
    const EmbedWs w = embed_ws(d_workspace, n, rows, dim);
    EmbedSort a{};
    a.ids = d_ids;
    a.n = n;
    a.rows = rows;
    embed_sort_digits(rows, &a.passes, &a.digit_bits);
    a.pairs0 = w.pairs0;
    a.pairs1 = w.pairs1;
    a.hist = w.hist;
    a.digit_total = w.digit_total;
    a.block_heads = w.block_heads;
    a.barrier = w.barrier;
    a.failed = w.barrier + 1;
    a.n_valid = w.n_valid;
    a.segpos = w.segpos;
    a.seg_start = w.seg_start;
    a.unique = dense ? w.unique : d_unique;
    a.count = d_count ? d_count : w.count;
    a.err = ctx->d_err;
    a.wait_limit_ns = ctx->wait_limit_ns;
    a.starve = ctx->starve_b;
    e = launch_embed_sort(a, s);
    if (e != cudaSuccess) return cuda_fail(e, "embed sort launch");
    EmbedSum u{};
    u.sorted = a.passes & 1 ? w.pairs1 : w.pairs0;
    u.segpos = w.segpos;
    u.seg_start = w.seg_start;
    u.unique = a.unique;
    u.n_valid = w.n_valid;
    u.failed = a.failed;
    u.dout = d_dout;
    u.dim = (int)dim;
    u.copies = (int)copies;
    u.scale = scale;
    u.dense = dense;
    u.accumulate = accumulate;
    u.grad = d_grad;
    u.rows_per_chunk = embed_rows_per_chunk(n, (int)dim, (int)copies);
    u.partial = w.partial;
    e = launch_embed_sum(u, n, s);
    if (e != cudaSuccess) return cuda_fail(e, "embed gradient launch");
    return ok();
}

engram_status engram_gate_checkpoint(const engram_ctx* ctx, int layer, const void* d_kv,
                                     int kv_format, const uint32_t* d_windows, int64_t T,
                                     const uint16_t* d_hidden, uint16_t* d_hidden_out,
                                     float* d_gates, uint8_t* d_codes, uint8_t* d_scales,
                                     void* stream) {
    engram_status st = check_layer(ctx, layer, true);
    if (st || (st = check_T(T))) return st;
    if (kv_format != ENGRAM_KV_F32 && kv_format != ENGRAM_KV_BF16)
        return fail(ENGRAM_EINVAL, "kv_format");
    if (T == 0) return ok();
    if (!d_kv || !d_windows || !d_hidden || !d_hidden_out || !d_codes || !d_scales ||
        !aligned16(d_kv) || !aligned16(d_windows) || !aligned16(d_hidden) ||
        !aligned16(d_hidden_out) || !aligned4(d_gates) || !aligned16(d_codes) || !aligned16(d_scales))
        return fail(ENGRAM_EINVAL, "kv / windows / hidden / codes / scales (16-byte aligned) / gates");
    GateTrain a = gate_args(ctx, layer, d_windows, T);
    a.kv = d_kv;
    a.hidden = d_hidden;
    a.hidden_out = d_hidden_out;
    a.gates = d_gates;
    a.codes_out = d_codes;
    a.scales_out = d_scales;
    cudaError_t e = launch_gate_checkpoint(a, kv_format == ENGRAM_KV_F32, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "gate checkpoint launch");
    return ok();
}

size_t engram_gate_backward_workspace_bytes(const engram_ctx* ctx, int64_t T) {
    if (!ctx || check_T(T)) return 0;
    return gate_backward_ws(nullptr, nullptr, T, (int)ctx->desc.hc, (int)ctx->desc.d);
}

engram_status engram_gate_backward(const engram_ctx* ctx, int layer, const void* d_kv,
                                   int kv_format, const uint16_t* d_hidden,
                                   const uint32_t* d_windows, int64_t T, const uint16_t* d_dout,
                                   uint16_t* d_dhidden, uint16_t* d_dkv, float* d_dwq, float* d_dwk,
                                   void* d_workspace, void* stream) {
    engram_status st = check_layer(ctx, layer, true);
    if (st || (st = check_T(T))) return st;
    if (kv_format != ENGRAM_KV_F32 && kv_format != ENGRAM_KV_BF16)
        return fail(ENGRAM_EINVAL, "kv_format");
    if (T > 0 && (!d_kv || !d_hidden || !d_windows || !d_dout || !d_dhidden || !d_dkv ||
                  !d_workspace || !aligned16(d_kv) || !aligned16(d_hidden) ||
                  !aligned16(d_windows) || !aligned16(d_dout) || !aligned16(d_dhidden) ||
                  !aligned16(d_dkv) || !aligned16(d_workspace)))
        return fail(ENGRAM_EINVAL, "kv / hidden / windows / gradients / workspace (16-byte aligned)");
    if (!aligned16(d_dwq) || !aligned16(d_dwk))
        return fail(ENGRAM_EINVAL, "dwq / dwk (16-byte aligned)");
    GateTrain a = gate_args(ctx, layer, d_windows, T);
    a.kv = d_kv;
    a.hidden = d_hidden;
    a.dout = d_dout;
    a.dhidden = d_dhidden;
    a.dkv = d_dkv;
    a.dwq = d_dwq;
    a.dwk = d_dwk;
    return gate_backward_call(ctx, a, kv_format == ENGRAM_KV_F32 ? kSavedF32 : kSavedBf16,
                              d_workspace, (cudaStream_t)stream);
}

engram_status engram_gate_backward_checkpoint(const engram_ctx* ctx, int layer,
                                              const uint8_t* d_codes, const uint8_t* d_scales,
                                              const uint32_t* d_windows, int64_t T,
                                              const uint16_t* d_dout, uint16_t* d_dhidden,
                                              uint16_t* d_dkv, float* d_dwq, float* d_dwk,
                                              void* d_workspace, void* stream) {
    engram_status st = check_layer(ctx, layer, true);
    if (st || (st = check_T(T))) return st;
    if (T > 0 && (!d_codes || !d_scales || !d_windows || !d_dout || !d_dhidden || !d_dkv ||
                  !d_workspace || !aligned16(d_codes) || !aligned16(d_scales) ||
                  !aligned16(d_windows) || !aligned16(d_dout) || !aligned16(d_dhidden) ||
                  !aligned16(d_dkv) || !aligned16(d_workspace)))
        return fail(ENGRAM_EINVAL, "codes / scales / windows / gradients / workspace (16-byte aligned)");
    if (!aligned16(d_dwq) || !aligned16(d_dwk))
        return fail(ENGRAM_EINVAL, "dwq / dwk (16-byte aligned)");
    GateTrain a = gate_args(ctx, layer, d_windows, T);
    a.codes = d_codes;
    a.scales = d_scales;
    a.dout = d_dout;
    a.dhidden = d_dhidden;
    a.dkv = d_dkv;
    a.dwq = d_dwq;
    a.dwk = d_dwk;
    return gate_backward_call(ctx, a, kSavedMx, d_workspace, (cudaStream_t)stream);
}

size_t engram_project_backward_workspace_bytes(const engram_ctx* ctx, int64_t T) {
    if (!ctx || check_T(T) || T == 0) return 0;
    Carver c(nullptr);
    c.take<float>(project_parked(ctx, T));
    return c.bytes();
}

engram_status engram_project_backward(const engram_ctx* ctx, int layer, const uint16_t* d_emb,
                                      const uint16_t* d_dkv, int64_t T, uint16_t* d_demb,
                                      uint16_t* d_dwkv, void* d_workspace, void* stream) {
    engram_status st = check_layer(ctx, layer, true);
    if (st || (st = check_T(T))) return st;
    if (!aligned16(d_demb) || !aligned16(d_dwkv) || !aligned16(d_workspace))
        return fail(ENGRAM_EINVAL, "demb / dwkv / workspace (16-byte aligned)");
    const cudaStream_t s = (cudaStream_t)stream;
    const int64_t N = ctx->N, K = ctx->K;
    if (T == 0) {
        cudaError_t e = d_dwkv ? cudaMemsetAsync(d_dwkv, 0, (size_t)N * K * 2, s) : cudaSuccess;
        return e == cudaSuccess ? ok() : cuda_fail(e, "project backward of no tokens");
    }
    if (!d_dkv || !aligned16(d_dkv) || (d_dwkv && (!d_emb || !aligned16(d_emb))))
        return fail(ENGRAM_EINVAL, "emb / dkv (16-byte aligned)");
    if (!d_demb && !d_dwkv) return ok();
    const LayerState& L = ctx->layers[layer];
    GradArgs a = grad_args(ctx);
    CUtensorMap tm[4];
    cudaError_t e = cudaSuccess;
    if (d_dwkv) {
        a.pr[1] = product(N, K, T, true);
        a.pr[1].out = d_dwkv;
        e = make_tma_16bit(&tm[2], d_dkv, T, N, 64, false);
        if (e == cudaSuccess) e = make_tma_16bit(&tm[3], d_emb, T, K, 64, false);
    }
    if (d_demb && e == cudaSuccess) {
        a.pr[0] = product(T, ctx->K, ctx->N, false);
        a.pr[0].out = d_demb;
        a.pr[0].splits = long_splits(a.pr[0], d_dwkv ? &a.pr[1] : nullptr);
        if (a.pr[0].splits > 1) {
            if (!d_workspace) return fail(ENGRAM_EINVAL, "null workspace");
            a.pr[0].acc = Carver(d_workspace).take<float>(1);
            a.pr[0].acc_write = 1;
        }
        e = make_tma_16bit(&tm[0], d_dkv, T, N, kBM, false);
        if (e == cudaSuccess) e = make_tma_16bit(&tm[1], L.w.wkv, N, K, 64, false);
    }
    if (e != cudaSuccess) return cuda_fail(e, "project backward tensor maps");
    if (!d_demb) tm[0] = tm[2], tm[1] = tm[3];
    if (!d_dwkv) tm[2] = tm[0], tm[3] = tm[1];
    e = launch_grad_products(a, tm, s);
    if (e == cudaSuccess && a.pr[0].acc_write)
        e = launch_sum_splits(a.pr[0].acc, a.pr[0].splits, T * K, nullptr, d_demb, s);
    if (e != cudaSuccess) return cuda_fail(e, "project backward launch");
    return ok();
}

size_t engram_loss_workspace_bytes(int64_t T, uint32_t vocab, uint32_t dim) {
    if (check_loss(vocab, dim, T)) return 0;
    return loss_ws(nullptr, T, vocab).bytes;
}

engram_status engram_loss(engram_ctx* ctx, const uint16_t* d_x, const uint16_t* d_head,
                          uint32_t vocab, uint32_t dim, const int32_t* d_labels, int64_t T,
                          float* d_loss, float* d_lse, void* d_workspace, void* stream) {
    engram_status st = check_loss(vocab, dim, T);
    if (st) return st;
    if (!ctx) return fail(ENGRAM_EINVAL, "null context");
    if (T == 0) return ok();
    if (!d_x || !d_head || !d_labels || !d_workspace || !aligned16(d_x) || !aligned16(d_head) ||
        !aligned4(d_labels) || !aligned16(d_workspace) || !aligned4(d_loss) || !aligned4(d_lse))
        return fail(ENGRAM_EINVAL, "x / head / workspace (16-byte aligned) / labels / loss / lse");
    if ((st = train_device(ctx))) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    const LossWs w = loss_ws(d_workspace, T, vocab);
    const int groups = loss_groups(T, vocab);
    cudaError_t e;
    if (T <= kFewTokens) {
        FewArgs f = few_args(ctx, T, vocab, dim);
        f.rows = (int)vocab;
        f.labels = d_labels;
        f.zlabel = w.zlabel;
        f.part = w.part;
        e = launch_few_lse(f, d_x, d_head, (int)dim, s);
    } else {
        GradArgs a = grad_args(ctx);
        a.pr[0] = product(T, vocab, dim, false);
        a.pr[0].group_m = loss_group_m(dim);
        a.T = T;
        a.vocab = (int)vocab;
        a.labels = d_labels;
        a.zlabel = w.zlabel;
        a.part = w.part;
        CUtensorMap tm[4];
        e = make_tma_16bit(&tm[0], d_x, T, dim, kBM, false);
        if (e == cudaSuccess) e = make_tma_16bit(&tm[1], d_head, vocab, dim, kBM, false);
        if (e != cudaSuccess) return cuda_fail(e, "loss tensor maps");
        tm[2] = tm[0], tm[3] = tm[1];
        e = launch_grad_lse(a, tm, s);
    }
    if (e == cudaSuccess)
        e = launch_loss_combine(w.part, groups, T, w.zlabel, d_labels, (int)vocab, d_loss, d_lse, ctx->d_err, s);
    if (e != cudaSuccess) return cuda_fail(e, "loss launch");
    return ok();
}

size_t engram_loss_backward_workspace_bytes(int64_t T, uint32_t vocab, uint32_t dim) {
    if (check_loss(vocab, dim, T) || T == 0) return 0;
    return loss_backward_ws(nullptr, T, vocab, dim, true).bytes;
}

engram_status engram_loss_backward(engram_ctx* ctx, const uint16_t* d_x, const uint16_t* d_head,
                                   uint32_t vocab, uint32_t dim, const int32_t* d_labels, int64_t T,
                                   const float* d_lse, const float* d_dloss, uint16_t* d_dx,
                                   uint16_t* d_dhead, void* d_workspace, void* stream) {
    engram_status st = check_loss(vocab, dim, T);
    if (st) return st;
    if (!ctx) return fail(ENGRAM_EINVAL, "null context");
    if (!aligned16(d_dx) || !aligned16(d_dhead)) return fail(ENGRAM_EINVAL, "dx / dhead (16-byte aligned)");
    const cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {
        cudaError_t e = d_dhead ? cudaMemsetAsync(d_dhead, 0, (size_t)vocab * dim * 2, s) : cudaSuccess;
        return e == cudaSuccess ? ok() : cuda_fail(e, "loss backward of no tokens");
    }
    if (!d_x || !d_head || !d_labels || !d_lse || !d_dloss || !d_workspace || !aligned16(d_x) ||
        !aligned16(d_head) || !aligned4(d_labels) || !aligned4(d_lse) || !aligned4(d_dloss) ||
        !aligned16(d_workspace))
        return fail(ENGRAM_EINVAL, "x / head / workspace (16-byte aligned) / labels / lse / dloss");
    if (!d_dx && !d_dhead) return ok();
    if ((st = train_device(ctx))) return st;
    const LossBackWs w = loss_backward_ws(d_workspace, T, vocab, dim, d_dhead != nullptr);
    const int64_t step = loss_piece(T, vocab), rows = ceil_div(T, 2 * kBM) * 2 * kBM;
    CUtensorMap x_k, x_mn;
    cudaError_t e = make_tma_16bit(&x_k, d_x, T, dim, kBM, false);
    if (e == cudaSuccess) e = make_tma_16bit(&x_mn, d_x, T, dim, 64, false);
    for (int64_t v0 = 0; v0 < vocab && e == cudaSuccess; v0 += step) {
        const int64_t cols = std::min<int64_t>(step, vocab - v0);
        const int64_t piece = ceil_div(cols, kBN) * kBN;
        const bool first = v0 == 0, last = v0 + step >= vocab;
        const uint16_t* head = d_head + v0 * dim;
        // z of the piece, and dz from it
        CUtensorMap tm[4];
        if (T <= kFewTokens) {
            FewArgs f = few_args(ctx, T, vocab, dim);
            f.rows = (int)piece;
            f.v0 = v0;
            f.labels = d_labels;
            f.lse = d_lse;
            f.dloss = d_dloss;
            f.dz = w.dz;
            e = launch_few_dz(f, d_x, head, (int)dim, s);
        } else {
            GradArgs a = grad_args(ctx);
            a.pr[0] = product(T, piece, dim, false);
            a.pr[0].group_m = loss_group_m(dim);
            a.T = T;
            a.v0 = v0;
            a.vocab = (int)vocab;
            a.dz_chunks = (int)(piece / 64);
            a.labels = d_labels;
            a.lse = d_lse;
            a.dloss = d_dloss;
            a.dz = w.dz;
            tm[0] = tm[2] = x_k;
            e = make_tma_16bit(&tm[1], head, vocab - v0, dim, kBM, false);
            if (e != cudaSuccess) break;
            tm[3] = tm[1];
            e = launch_grad_dz(a, tm, s);
        }
        if (e != cudaSuccess) break;
        // dx += dz head, dhead = dz^T x
        GradArgs g = grad_args(ctx);
        g.unit = d_dloss;
        const uint64_t dz_rows = (uint64_t)rows * piece / 64;
        e = make_tma_16bit(&tm[0], w.dz, dz_rows, 64, kBM, false);
        if (e == cudaSuccess) e = make_tma_16bit(&tm[1], head, vocab - v0, dim, 64, false);
        if (e == cudaSuccess) e = make_tma_16bit(&tm[2], w.dz, dz_rows, 64, 64, false);
        if (e != cudaSuccess) break;
        tm[3] = x_mn;
        if (d_dx) {
            g.pr[0] = loss_dx(T, dim, piece);
            g.pr[0].out = d_dx;
            g.pr[0].splits = std::min(w.splits, g.pr[0].kb);
            g.pr[0].acc = w.acc;
            g.pr[0].acc_read = !first;
            g.pr[0].acc_write = !last || w.splits > 1;
        }
        if (d_dhead) {
            g.pr[1] = loss_dhead(T, dim, cols, piece);
            g.pr[1].out = d_dhead + v0 * dim;
        }
        e = launch_grad_products(g, tm, s);
    }
    if (e == cudaSuccess && d_dx && w.splits > 1)
        e = launch_sum_splits(w.acc, w.splits, T * (int64_t)dim, d_dloss, d_dx, s);
    if (e != cudaSuccess) return cuda_fail(e, "loss backward launch");
    return ok();
}

}  // extern "C"
