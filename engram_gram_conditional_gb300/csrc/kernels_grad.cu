// Matrix products of the training step on CTA pairs (tcgen05 cta_group::2,
// TMEM accumulators, TMA operands, sm_103a):
//
//   loss             z = x head^T                softmax statistics as epilogue
//   loss backward    z again, a piece of the vocabulary at a time; the epilogue
//                    stores dz = (exp(z - lse) - [v = label]) dloss / unit as BF16
//                    dx += dz head (piece),  dhead (piece) = dz^T x
//   project backward demb = dkv wkv,  dwkv = dkv^T emb
//
// One persistent pair per two SMs walks 256 x 256 output tiles; each CTA
// stages its 128 rows of A and its 128 columns' half of B, 64 of the reduction
// per stage (2 x 16 KB).  The gradient products read their operands as they lie
// in memory: a transposed operand is loaded in boxes of 64 contiguous elements
// x 64 reduction rows and described to the tensor core as MN-major, so nothing
// is transposed in memory.  Two products (problems) share one launch: the long
// one (dx, demb: few tiles, long reduction) goes first, round robin, and the
// short one (dhead, dwkv) fills the pairs up, so that they end together.
//
// Bound by the tensor cores, and these by the power limit: over seconds cuBLAS
// BF16 runs at 1,722 TFLOP/s on such a GPU (1,920 in bursts).  2,048 tokens,
// 129,280 x 5,120, back to back: loss 1.49 ms (1,810 TFLOP/s), its backward pass
// 4.68 ms (1,740); project backward at 25,600 x 6,144 0.72 ms (1,790).  In one
// launch alone the tensor pipe is active 97% of the cycles.  256 x 256 tiles on
// pairs: a pair takes in 64 KB per 512 cycles of MMA, two thirds of what two
// single CTAs with 128 x 256 tiles would.  Six stages: five or seven differ by 1-2%.
//
// Warp roles (320 threads): warps 0..7 epilogue, two per TMEM quadrant, each on
// 128 of the tile's 256 columns; warp 8 TMA; warp 9 MMA issue (even CTA of the
// pair).  Every wait is bounded as in kernels_mma.cu.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "device_common.cuh"
#include "grad_internal.h"
#include "per_device.h"
#include "tcgen05_common.cuh"

namespace engram {

namespace {

constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kWarpTma = 8, kWarpMma = 9;
constexpr int kCols = kBN / (kEpiWarps / 4);  // of a tile, per epilogue warp
constexpr int kOperand = kBM * kBK * 2;   // 16 KB: one CTA's A or B of a stage
constexpr int kStage = 2 * kOperand;
constexpr int kTmemCols = 2 * kBN;
// k-blocks that the loss's logits sum in one accumulator.  The tensor core's
// additions to an accumulator truncate: over 5,120 products that took 1.5e-6 off
// a loss (relative; 1e-7 with sums rounded to nearest).  So the epilogue takes
// the accumulator every 1,024 products and adds it in registers.  The gradient
// products keep one accumulator: over 25,600 products that takes 2.9e-5 off demb,
// whose rounding to BF16 is off by 1.66e-3.
constexpr int kLseSegment = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kChunk = 64 * kBK * 2;      // 8 KB: 64 MN elements x 64 k of an MN-major tile
// An epilogue warp turns 32 rows x 64 BF16 of a tile from a row per lane into
// whole 128-byte lines through a box of shared memory.  (16-byte stores of a row
// per lane, straight to memory, took 4.5 us per tile where the MMAs of a
// 384-long reduction take 1.6; bulk copies of the boxes make 16 tokens' project
// backward 6% faster, 333 tokens' no different and the loss's backward 0.5% slower.)
constexpr int kBox = 32 * 64 * 2;

// Shared memory of each variant.
template <int kEpi>
struct Layout {
    static constexpr int kStages = 6;
    static constexpr int kOffOut = kStages * kStage;
    static constexpr int kOffBar = kOffOut + (kEpi == kGradLse ? 0 : kEpiWarps * kBox);
    static constexpr int kNumBars = 2 * kStages + 4;
    static constexpr int kOffTmem = kOffBar + kNumBars * 8;
    static constexpr int kOffFlag = kOffTmem + 4;
    static constexpr int kSmem = kOffFlag + 4 + 1024;
    static_assert(kSmem <= 232448, "shared memory above the per-block limit");
};

// Instruction descriptor, kind::f16, BF16 operands, fp32 accumulate, M = 256
// (a pair), N = 256; bit 15 / 16: A / B is MN-major.
__host__ __device__ constexpr uint32_t grad_idesc(bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           ((uint32_t)(kBN >> 3) << 17) | ((uint32_t)(2 * kBM >> 4) << 24);
}

// Shared-memory descriptor of an MN-major operand in 128-byte swizzled rows of
// 64 elements: 64-element chunks kChunk bytes apart (LBO), groups of eight k
// 1,024 bytes apart (SBO).
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kChunk >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Row r of a warp's box, 16-byte piece j (of 8), swizzled against bank conflicts.
__device__ __forceinline__ uint32_t out_piece(uint32_t box, int r, int j) {
    return box + (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4));
}
// The box to memory, four rows per instruction: rows `ld` elements apart from
// `dst`, of which the first `rows` and the first `cols` columns (a multiple of 8)
// are written.
__device__ __forceinline__ void put_box(uint32_t box, int lane, uint16_t* dst, int64_t ld, int64_t rows,
                                        int64_t cols) {
    const int j = lane & 7, r0 = lane >> 3;
    const int n = 8 * j < cols ? (int)min(rows, (int64_t)32) : 0;
    dst += r0 * ld + 8 * j;
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w)
                     : "r"(out_piece(box, 4 * k + r0, j)));
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (4 * k + r0 < n) *reinterpret_cast<uint4*>(dst + 4 * k * ld) = v[k];
}
// Arrival on a barrier of the pair's even CTA that hands an accumulator back.
// Relaxed: what has to come before it are this warp's reads of tensor memory, which
// tcgen05.wait::ld has completed and the tcgen05 fence orders.  A release at cluster
// scope would wait for the warp's stores of the tile before (850 to 2,200 cycles per
// tile).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// 32 bytes at a time: a whole sector per thread.
__device__ __forceinline__ void ld_global_v8(const float* p, float (&f)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void st_global_v8(float* p, const float (&f)[8]) {
    asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(f[0]), "f"(f[1]), "f"(f[2]),
                 "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]), "l"(p)
                 : "memory");
}

// Work item i of pair p: problem, M unit, N tile and k-block range.
struct Item {
    int pr, mu, nt, kb_lo, nkb, split;
};

// The long problem's items go round robin: pair p has items p, p + pairs, ...; so
// the first `a.pairs_more` pairs may have one more than the others.  The short
// problem's items follow in order of the rounds in which the pairs get to them:
// in the first a.rounds_fewer rounds only the pairs with fewer long items take
// one each, then all pairs do, so that the pairs end together and those that run
// at the same time work on neighbouring tiles.
__device__ __forceinline__ int short_index(const GradArgs& a, int p, int pairs, int i) {
    const int fewer = pairs - a.pairs_more;
    if (p < a.pairs_more) return a.rounds_fewer * fewer + i * pairs + p;
    if (i < a.rounds_fewer) return i * fewer + (p - a.pairs_more);
    return a.rounds_fewer * fewer + (i - a.rounds_fewer) * pairs + p;
}

__device__ __forceinline__ int item_count(const GradArgs& a, int p, int pairs) {
    const int nh = a.pr[0].items > p ? (a.pr[0].items - p + pairs - 1) / pairs : 0;
    const int L = a.pr[1].items, fewer = pairs - a.pairs_more;
    if (L == 0) return nh;
    // items of this pair with short_index < L
    const int first = a.rounds_fewer * fewer;
    const int all = L > first + p ? (L - first - p + pairs - 1) / pairs : 0;
    if (p < a.pairs_more) return nh + all;
    const int b = p - a.pairs_more, upto = min(L, first);
    return nh + (upto > b ? (upto - b + fewer - 1) / fewer : 0) + all;
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
}

// n / d for n < 2^31 (see fast_div on the host).
__device__ __forceinline__ int divide(int n, const FastDiv& d) {
    return d.d == 1 ? n : (int)(__umulhi((uint32_t)n, d.m) >> d.s);
}

__device__ __forceinline__ Item get_item(const GradArgs& a, int p, int pairs, int n_long, int i) {
    Item it;
    int idx;
    if (i < n_long) {
        it.pr = 0;
        idx = p + i * pairs;
    } else {
        it.pr = 1;
        idx = short_index(a, p, pairs, i - n_long);
    }
    const GradProblem& q = a.pr[it.pr];
    it.split = 0;
    it.kb_lo = 0;
    it.nkb = q.kb;
    if (q.splits > 1) {
        it.split = divide(idx, q.per_split);
        idx -= it.split * (int)q.per_split.d;
        it.kb_lo = it.split * q.kb / q.splits;
        it.nkb = (it.split + 1) * q.kb / q.splits - it.kb_lo;
    }
    // groups of group_m units, M inner: the pairs in flight share tiles of both
    // operands in L2
    const int g = divide(idx, q.per_group), first = g * q.group_m;
    const int r = idx - g * (int)q.per_group.d;
    const FastDiv& gm = first + q.group_m <= q.m_units ? q.in_group : q.in_last;
    it.nt = divide(r, gm);
    it.mu = first + (r - it.nt * (int)gm.d);
    return it;
}

// kEpi: what becomes of a tile.
template <int kEpi>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
k_grad(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmB0,
       const __grid_constant__ CUtensorMap tmA1, const __grid_constant__ CUtensorMap tmB1,
       const __grid_constant__ GradArgs a) {
    using L = Layout<kEpi>;
    constexpr int kSegment = kEpi == kGradLse ? kLseSegment : 1 << 30;
    constexpr int kStages = L::kStages, kOffBar = L::kOffBar;
    const uint32_t rank = cluster_ctarank();
    const bool issuer = rank == 0u;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto full = [&](int s) { return sbase + kOffBar + 8u * (uint32_t)s; };
    auto empty = [&](int s) { return sbase + kOffBar + 8u * (uint32_t)(kStages + s); };
    auto tfull = [&](int acc) { return sbase + kOffBar + 8u * (uint32_t)(2 * kStages + acc); };
    auto tempty = [&](int acc) { return sbase + kOffBar + 8u * (uint32_t)(2 * kStages + 2 + acc); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffFlag);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffTmem);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1u);
            mbar_init(empty(s), 1u);
        }
        for (int acc = 0; acc < 2; ++acc) {
            mbar_init(tfull(acc), 1u);
            mbar_init(tempty(acc), 2u * kEpiWarps);  // the epilogue warps of both CTAs
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWarpMma) tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers exist before either signals the other
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();

    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    const int n_items = item_count(a, pair, pairs);
    const int n_long = a.pr[0].items > pair ? (a.pr[0].items - pair + pairs - 1) / pairs : 0;
    const long long lim = a.wait_limit_ns;
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(a.err, kErrTimeout);
    };

    if (warp == kWarpTma) {
        // The whole warp walks the items, one elected lane loads: coordinates and
        // addresses stay in uniform registers, and what does not change within an
        // item is out of the loop.  (The tensor cores feel every few instructions
        // in the load and issue loops, 1-5% of a launch; the issuing warp is best
        // walked by one lane alone.)
        const bool leader = elect_one();
        auto wait = [&](uint32_t b, uint32_t parity) {
            bool ok = true;
            if (kEpi == kGradOut) {
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_suspended(b, parity, abort_flag, lim));
            } else {  // (one lane waits: 2% less for the softmax epilogues, 1% more for the products)
                if (lane == 0) ok = mbar_wait_suspended(b, parity, abort_flag, lim);
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            }
            if (!ok && leader) fail();
            return ok;
        };
        int s = 0;
        uint32_t phase = 1;  // of the stage's empty barrier
        const uint32_t full0 = map_rank(full(0), 0);  // the even CTA's barriers
        bool ok = !a.starve;
        for (int i = 0; i < n_items && ok; ++i) {
            const Item w = get_item(a, pair, pairs, n_long, i);
            const GradProblem& q = a.pr[w.pr];
            const CUtensorMap* tmA = w.pr ? &tmA1 : &tmA0;
            const CUtensorMap* tmB = w.pr ? &tmB1 : &tmB0;
            const int mb = 2 * w.mu + (int)rank;               // this CTA's 128 rows of A
            const int n0 = w.nt * kBN + (int)rank * (kBN / 2);      // and its half of B
            // the A box of the first k-block, its steps to the next (from an even and
            // from an odd block), and an MN-major operand's second box
            constexpr bool b_mn = kEpi == kGradOut;  // (the products read B as it lies)
            const bool a_mn = kEpi == kGradOut && q.a_mn;
            const int tiled = kEpi == kGradOut ? q.a_tiled : 0;
            int ax, ay, asx = 0, as0, as1, aox = 0, aoy = 0;
            if (a_mn && tiled) {  // 128 x 64 tiles [reduction block][M chunk]
                ax = 0;
                ay = ((w.kb_lo >> 1) * tiled + 2 * mb) * 128 + (w.kb_lo & 1) * 64;
                as0 = 64;
                as1 = tiled * 128 - 64;
                aoy = 128;
            } else if (a_mn) {
                ax = mb * kBM;
                ay = w.kb_lo * kBK;
                as0 = as1 = kBK;
                aox = 64;
            } else if (tiled) {  // 128 x 64 tiles [M block][reduction chunk]
                ax = 0;
                ay = (mb * tiled + w.kb_lo) * 128;
                as0 = as1 = 128;
            } else {
                ax = w.kb_lo * kBK;
                ay = mb * kBM;
                asx = kBK;
                as0 = as1 = 0;
            }
            int bx = b_mn ? n0 : w.kb_lo * kBK, by = b_mn ? w.kb_lo * kBK : n0;
            const int bsx = b_mn ? 0 : kBK, bsy = b_mn ? kBK : 0;
            bool odd = (w.kb_lo & 1) != 0;
            for (int j = 0; j < w.nkb; ++j) {
                ok = wait(empty(s), phase);
                if (!ok) break;
                if (leader) {
                    const uint32_t sa = sbase + (uint32_t)(s * kStage), sb = sa + kOperand;
                    const uint32_t bar = full0 + 8u * (uint32_t)s;
                    if (issuer) mbar_expect_tx(full(s), 2 * kStage);
                    tma_load_2d_pair(sa, tmA, bar, ax, ay);
                    if (a_mn) tma_load_2d_pair(sa + kChunk, tmA, bar, ax + aox, ay + aoy);
                    tma_load_2d_pair(sb, tmB, bar, bx, by);
                    if (b_mn) tma_load_2d_pair(sb + kChunk, tmB, bar, bx + 64, by);
                }
                ax += asx;
                ay += odd ? as1 : as0;
                odd = !odd;
                bx += bsx;
                by += bsy;
                if (++s == kStages) {
                    s = 0;
                    phase ^= 1u;
                }
            }
        }
    } else if (warp == kWarpMma) {
        if (issuer && lane == 0) {
            auto wait = [&](uint32_t b, uint32_t parity) {
                const bool ok = mbar_wait_suspended(b, parity, abort_flag, lim);
                if (!ok) fail();
                return ok;
            };
            int s = 0, use = 0;  // stage, accumulators used so far
            uint32_t phase = 0;  // of the stage's full barrier
            // nkb k-blocks of operands stored as kAMn and kBMn say, kSegment to an
            // accumulator; false on a time-out
            auto issue = [&](auto kAMn, auto kBMn, int nkb) {
                constexpr bool a_mn = decltype(kAMn)::value, b_mn = decltype(kBMn)::value;
                constexpr uint32_t id = grad_idesc(a_mn, b_mn);
                // 16 of the reduction: 32 bytes of a K-major row, or 16 rows of 128 bytes
                constexpr uint64_t a_step = a_mn ? 128ull : 2ull, b_step = b_mn ? 128ull : 2ull;
                const uint64_t a_desc = a_mn ? sdesc_mn(sbase) : sdesc_sw128(sbase);
                const uint64_t b_desc = b_mn ? sdesc_mn(sbase + kOperand) : sdesc_sw128(sbase + kOperand);
                for (int kb0 = 0; kb0 < nkb; kb0 += kSegment, ++use) {
                    const int acc = use & 1, n = min(kSegment, nkb - kb0);
                    if (!wait(tempty(acc), ((uint32_t)(use >> 1) & 1u) ^ 1u)) return false;
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kBN);
                    for (int j = 0; j < n; ++j) {
                        if (!wait(full(s), phase)) return false;
                        tc_fence_after();
                        // (a stage is kStage / 16 descriptor units further)
                        const uint64_t ad = a_desc + (uint64_t)(s * (kStage >> 4));
                        const uint64_t bd = b_desc + (uint64_t)(s * (kStage >> 4));
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k)
                            umma_f16kind_pair(d_tmem, ad + a_step * k, bd + b_step * k, id, (j != 0) || (k != 0));
                        umma_commit_pair(empty(s));
                        if (++s == kStages) {
                            s = 0;
                            phase ^= 1u;
                        }
                    }
                    umma_commit_pair(tfull(acc));
                }
                return true;
            };
            using Mn = std::true_type;
            using K = std::false_type;
            bool ok = true;
            for (int i = 0; i < n_items && ok; ++i) {
                const GradProblem& q = a.pr[i < n_long ? 0 : 1];
                int nkb = q.kb;
                if (q.splits > 1) nkb = get_item(a, pair, pairs, n_long, i).nkb;
                if constexpr (kEpi != kGradOut)
                    ok = issue(K{}, K{}, nkb);
                else if (q.a_mn)
                    ok = issue(Mn{}, Mn{}, nkb);
                else
                    ok = issue(K{}, Mn{}, nkb);
            }
        }
    } else {
        // ---- epilogue ----
        const int q4 = warp & 3, grp = warp >> 2;  // TMEM quadrant; columns [kCols grp, kCols grp + kCols)
        const int m = q4 * 32 + lane;
        const uint32_t box = sbase + L::kOffOut + (uint32_t)(warp * kBox);
        const float unit = kEpi == kGradDz ? loss_unit(a.dloss)
                           : kEpi == kGradOut && a.unit ? loss_unit(a.unit) : 1.0f;
        int use = 0;  // accumulators used so far
        auto acc_ready = [&]() {
            const int acc = use & 1;
            int ready = 1;
            if (lane == 0) ready = mbar_wait_suspended(tfull(acc), (uint32_t)(use >> 1) & 1u, abort_flag, lim);
            ready = __shfl_sync(0xFFFFFFFFu, ready, 0);
            if (!ready && lane == 0) fail();
            tc_fence_after();
            return ready != 0;
        };
        auto acc_done = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(map_rank(tempty(use & 1), 0));
            ++use;
        };
        for (int i = 0; i < n_items; ++i) {
            const Item w = get_item(a, pair, pairs, n_long, i);
            const GradProblem& q = a.pr[w.pr];
            const int64_t row = ((int64_t)2 * w.mu + rank) * kBM + m;
            const int col0 = w.nt * kBN + grp * kCols;
            auto acc_addr = [&]() {
                return tmem_base + (uint32_t)((use & 1) * kBN + grp * kCols) + ((uint32_t)(q4 * 32) << 16);
            };
            float lse = 0.f, dl = 0.f;
            int label = -1;
            if (kEpi == kGradLse || kEpi == kGradDz) {
                if (row < a.T) {
                    label = a.labels[row];
                    if (label >= a.vocab) label = -1;
                    if (kEpi == kGradDz) {
                        lse = a.lse[row];
                        dl = label >= 0 ? a.dloss[row] / unit : 0.f;
                    }
                }
            }
            if constexpr (kEpi == kGradLse) {
                float v[4][32];
                bool ok = true;
                for (int seg = 0; seg < w.nkb && ok; seg += kSegment) {
                    ok = acc_ready();
                    const uint32_t taddr = acc_addr();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tmem_ld32(taddr + (uint32_t)(c * 32), r);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            v[c][j] = seg ? v[c][j] + __uint_as_float(r[j]) : __uint_as_float(r[j]);
                    }
                    acc_done();
                }
                if (!ok) break;
                // running maximum and sum over this warp's 128 columns
                float mx = -INFINITY, sum = 0.f;
                const int64_t zrel = (int64_t)label - col0;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (label >= 0 && zrel >= c * 32 && zrel < c * 32 + 32) {
                        float z = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (zrel == c * 32 + j) z = v[c][j];
                        a.zlabel[row] = z;
                    }
                    const int lastc = a.vocab - (col0 + c * 32);
                    if (lastc < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= lastc) v[c][j] = -INFINITY;
                    }
                    float cm = v[c][0];
                    bool nan = v[c][0] != v[c][0];
#pragma unroll
                    for (int j = 1; j < 32; ++j) {
                        nan |= v[c][j] != v[c][j];
                        cm = fmaxf(cm, v[c][j]);
                    }
                    const float nm = fmaxf(mx, cm);
                    const float base = nm == -INFINITY ? 0.f : nm;
                    float cs = 0.f;
#pragma unroll
                    for (int j = 0; j < 32; ++j) cs += exp2f((v[c][j] - base) * kLog2e);
                    sum = sum * exp2f((mx - base) * kLog2e) + cs;
                    if (nan) sum = NAN;
                    mx = nm;
                }
                if (row < a.T)
                    a.part[((int64_t)w.nt * 2 + grp) * a.T + row] = make_float2(mx, sum);
                continue;
            }
            if (!acc_ready()) break;
            const uint32_t taddr = acc_addr();
            if constexpr (kEpi == kGradDz) {
                // this warp's columns are two 64-wide chunks of the tiled dz
                const int64_t tb = 2 * w.mu + rank;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const int chunk = (col0 >> 6) + half;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t r[32];
                        tmem_ld32(taddr + (uint32_t)(half * 64 + c * 32), r);
                        tmem_wait_ld();
                        const int64_t v0 = a.v0 + chunk * 64 + c * 32;  // column within the vocabulary
                        const int64_t rel = (int64_t)label - v0;
                        uint32_t o[16];
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            float d[2];
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                // (z - lse first: exact where p is near 1)
                                float p = exp2f((__uint_as_float(r[j + u]) - lse) * kLog2e);
                                if (rel == j + u) p -= 1.f;
                                d[u] = label >= 0 && v0 + j + u < a.vocab ? p * dl : 0.f;
                            }
                            o[j / 2] = bf16x2_pack_rn(d[0], d[1]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            st_shared_v4(out_piece(box, lane, c * 4 + j),
                                         make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]));
                    }
                    __syncwarp();
                    put_box(box, lane, a.dz + ((tb * a.dz_chunks + chunk) * 128 + q4 * 32) * 64, 64, 32, 64);
                    __syncwarp();
                }
            } else if constexpr (kEpi == kGradOut) {
                if (!q.acc) {
                    // the accumulator is handed back before the first store
                    uint32_t o[4][16];
#pragma unroll
                    for (int c = 0; c < 4; c += 2) {
                        uint32_t r[2][32];
                        tmem_ld32(taddr + (uint32_t)(c * 32), r[0]);
                        tmem_ld32(taddr + (uint32_t)(c * 32 + 32), r[1]);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[c + j / 16][j % 16] =
                                bf16x2_pack_rn(__uint_as_float(r[j / 16][2 * (j % 16)]) * unit,
                                               __uint_as_float(r[j / 16][2 * (j % 16) + 1]) * unit);
                    }
                    acc_done();
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint32_t* p = o[2 * half + j / 4] + 4 * (j % 4);
                            st_shared_v4(out_piece(box, lane, j), make_uint4(p[0], p[1], p[2], p[3]));
                        }
                        __syncwarp();
                        const int64_t x = col0 + half * 64, y = row - lane;
                        put_box(box, lane, q.out + y * q.N + x, q.N, q.M - y, q.N - x);
                        __syncwarp();
                    }
                    continue;
                }
                // added to what earlier pieces left in fp32; out as BF16 from the
                // last piece, else (and from a split) as fp32
                const bool in = row < q.M;
                float* accp = q.acc + ((int64_t)w.split * q.M + row) * q.N;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t r[32];
                        tmem_ld32(taddr + (uint32_t)(half * 64 + c * 32), r);
                        tmem_wait_ld();
                        const int64_t n = col0 + half * 64 + c * 32;
                        // N is a multiple of 8: groups of eight columns are in or out whole
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            float v[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) v[u] = __uint_as_float(r[j + u]);
                            if (in && n + j < q.N) {
                                if (q.acc_read) {
                                    float x[8];
                                    ld_global_v8(accp + n + j, x);
#pragma unroll
                                    for (int u = 0; u < 8; ++u) v[u] += x[u];
                                }
                                if (q.acc_write) st_global_v8(accp + n + j, v);
                            }
                            if (!q.acc_write)
                                st_shared_v4(out_piece(box, lane, c * 4 + j / 8),
                                             make_uint4(bf16x2_pack_rn(v[0] * unit, v[1] * unit),
                                                        bf16x2_pack_rn(v[2] * unit, v[3] * unit),
                                                        bf16x2_pack_rn(v[4] * unit, v[5] * unit),
                                                        bf16x2_pack_rn(v[6] * unit, v[7] * unit)));
                        }
                    }
                    __syncwarp();
                    if (!q.acc_write) {
                        const int64_t x = col0 + half * 64, y = row - lane;
                        put_box(box, lane, q.out + y * q.N + x, q.N, q.M - y, q.N - x);
                        __syncwarp();
                    }
                }
            }
            acc_done();
        }
    }

    __syncthreads();
    if (*abort_flag) {
        // let copies and MMAs still in flight land before TMEM is freed
        if (threadIdx.x == 0) {
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
        }
        __syncthreads();
    }
    cluster_sync();  // no arrival or multicast may target a CTA that exited
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, kTmemCols);
    }
}

// loss and lse of each row from the column groups' (maximum, sum) pairs: 32 rows a
// block, each of its slices a contiguous share of the groups in column order, in
// batches whose loads leave together, then the slices in order.  2,048 rows of 1,010
// groups, 16 MB from L2: the loss takes 1.49 ms; with the groups taken one by one,
// each behind the exponentials of the one before, 1.52.
constexpr int kCombineSlices = 16, kCombineBatch = 16;

__device__ __forceinline__ void add_pair(float& mx, float& sum, float2 p) {
    const float nm = fmaxf(mx, p.x);
    const float b = nm == -INFINITY ? 0.f : nm;
    sum = sum * expf(mx - b) + p.y * expf(p.x - b);
    mx = nm;
}
__global__ void __launch_bounds__(32 * kCombineSlices)
k_loss_combine(const float2* part, int groups, int64_t T, const float* zlabel, const int32_t* labels,
               int vocab, float* loss, float* lse, uint32_t* err) {
    pdl_wait();
    __shared__ float2 sm[kCombineSlices][32];
    const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * 32 + lane;
    float mx = -INFINITY, sum = 0.f;
    if (t < T) {
        const int lo = sl * groups / kCombineSlices, hi = (sl + 1) * groups / kCombineSlices;
        for (int g = lo; g < hi; g += kCombineBatch) {
            float2 p[kCombineBatch];
            float nm = mx;
#pragma unroll
            for (int u = 0; u < kCombineBatch; ++u)
                p[u] = g + u < hi ? part[(int64_t)(g + u) * T + t] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int u = 0; u < kCombineBatch; ++u) nm = fmaxf(nm, p[u].x);
            const float b = nm == -INFINITY ? 0.f : nm;
            sum *= expf(mx - b);
#pragma unroll
            for (int u = 0; u < kCombineBatch; ++u) sum += p[u].y * expf(p[u].x - b);
            mx = nm;
        }
    }
    sm[sl][lane] = make_float2(mx, sum);
    __syncthreads();
    if (sl || t >= T) return;
    for (int k = 1; k < kCombineSlices; ++k) add_pair(mx, sum, sm[k][lane]);
    const float l = mx + logf(sum);
    const int y = labels[t];
    if (y >= vocab) atomicOr(err, kErrBounds);
    if (lse) lse[t] = l;
    if (loss) loss[t] = y >= 0 && y < vocab ? l - zlabel[t] : 0.f;
}

// out = the sum of the splits' fp32 buffers, in order, times the unit, rounded to
// BF16 (n a multiple of 8).
__global__ void k_sum_splits(const float* acc, int splits, int64_t n, const float* unit, uint16_t* out) {
    pdl_wait();
    const float by = unit ? loss_unit(unit) : 1.0f;
    const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8;
    if (i >= n) return;
    float v[8] = {};
    for (int s = 0; s < splits; ++s) {
        const float4 x = *reinterpret_cast<const float4*>(acc + s * n + i);
        const float4 y = *reinterpret_cast<const float4*>(acc + s * n + i + 4);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= by;
    *reinterpret_cast<uint4*>(out + i) =
        make_uint4(bf16x2_pack_rn(v[0], v[1]), bf16x2_pack_rn(v[2], v[3]),
                   bf16x2_pack_rn(v[4], v[5]), bf16x2_pack_rn(v[6], v[7]));
}

// q = floor(n / d) = floor(n m / 2^(31 + l)) for n < 2^31, with l = ceil(log2 d)
// and m = ceil(2^(31 + l) / d): the excess m d - 2^(31 + l) < d <= 2^l, times n,
// stays below 2^(31 + l).  (Granlund and Montgomery, PLDI 1994.)
FastDiv fast_div(int d) {
    int l = 0;
    while (((int64_t)1 << l) < d) ++l;
    FastDiv f{};
    f.d = (uint32_t)d;
    if (d > 1) {
        f.m = (uint32_t)((((uint64_t)1 << (31 + l)) + (uint32_t)d - 1) / (uint32_t)d);
        f.s = (uint32_t)(l - 1);
    }
    return f;
}

// How many rounds of short items fit into the time of one long item.
void share_items(GradArgs& a, int pairs) {
    a.pairs_more = a.pr[0].items % pairs;
    a.rounds_fewer = 0;
    if (!a.pr[0].items || !a.pr[1].items || !a.pairs_more) return;
    // an item takes its k-blocks and a little; a short one what writing out its
    // tile takes (measured: 7 k-blocks' time at one k-block, 11 at six, 34 at 32)
    auto cost = [](const GradProblem& q) {
        const double kb = (double)q.kb / q.splits;
        return std::max(kb + 2.0, 7.0 + 0.7 * kb);
    };
    const int fewer = pairs - a.pairs_more;
    a.rounds_fewer = std::min((int)(cost(a.pr[0]) / cost(a.pr[1]) + 0.5), (a.pr[1].items + fewer - 1) / fewer);
}

cudaError_t pdl_launch(void* f, dim3 grid, dim3 block, void** args, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, f, args);
}

// CTA pairs that are resident at once: a launch has no more, since its items are
// dealt out for pairs that all run from the start.
template <int kEpi>
cudaError_t resident_pairs(int* pairs) {
    static PerDevice known, allowed;
    return known.get(pairs, [](int* found) {
        auto kern = k_grad<kEpi>;
        cudaError_t e = allow_shared(allowed, kern, Layout<kEpi>::kSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2 * (device_sm_count() / 2));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Layout<kEpi>::kSmem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        *found = std::min(n, device_sm_count() / 2);
        return cudaSuccess;
    });
}

template <int kEpi>
cudaError_t launch(GradArgs& a, const CUtensorMap* tm, cudaStream_t s) {
    auto kern = k_grad<kEpi>;
    for (GradProblem& q : a.pr) {
        q.items = q.m_units * q.n_tiles * q.splits;
        if (!q.items) continue;
        q.per_split = fast_div(q.m_units * q.n_tiles);
        q.per_group = fast_div(q.group_m * q.n_tiles);
        q.in_group = fast_div(q.group_m);
        q.in_last = fast_div(q.m_units % q.group_m ? q.m_units % q.group_m : q.group_m);
    }
    const int total = a.pr[0].items + a.pr[1].items;
    if (!total) return cudaSuccess;
    int pairs = 0;
    cudaError_t e = resident_pairs<kEpi>(&pairs);
    if (e != cudaSuccess) return e;
    pairs = std::min(pairs, total);
    share_items(a, pairs);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<kEpi>::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tm[0], tm[1], tm[2], tm[3], a);
}

}  // namespace

int grad_pairs() { return device_sm_count() / 2; }

cudaError_t launch_grad_lse(GradArgs& a, const CUtensorMap* tm, cudaStream_t s) {
    return launch<kGradLse>(a, tm, s);
}
cudaError_t launch_grad_dz(GradArgs& a, const CUtensorMap* tm, cudaStream_t s) {
    return launch<kGradDz>(a, tm, s);
}
cudaError_t launch_grad_products(GradArgs& a, const CUtensorMap* tm, cudaStream_t s) {
    return launch<kGradOut>(a, tm, s);
}

cudaError_t launch_loss_combine(const float2* part, int groups, int64_t T, const float* zlabel,
                                const int32_t* labels, int vocab, float* loss, float* lse,
                                uint32_t* err, cudaStream_t s) {
    void* args[] = {&part, &groups, &T, &zlabel, &labels, &vocab, &loss, &lse, &err};
    return pdl_launch((void*)k_loss_combine, dim3((unsigned)((T + 31) / 32)), dim3(32 * kCombineSlices), args, s);
}

cudaError_t launch_sum_splits(const float* acc, int splits, int64_t n, const float* unit, uint16_t* out,
                              cudaStream_t s) {
    void* args[] = {&acc, &splits, &n, &unit, &out};
    return pdl_launch((void*)k_sum_splits, dim3((unsigned)((n / 8 + 255) / 256)), dim3(256), args, s);
}

}  // namespace engram
