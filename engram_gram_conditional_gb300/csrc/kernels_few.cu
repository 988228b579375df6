// The loss's logits of at most 16 tokens (sm_103a): softmax statistics, or dz of a
// piece of the vocabulary.
//
// With so few tokens the head's bytes are the whole cost, so the product is
// turned round: 128 rows of the head are the M of a tcgen05.mma (one CTA), 16
// tokens its N - an MMA that takes a fraction of its operand's way through
// memory.  (The 256 x 256 tiles of kernels_grad.cu compute 256 rows of tokens
// whatever their number: over 129,280 x 5,120 one token's loss takes 323 us with
// them, 8 tokens' 287 and 16 tokens' 222, and 206 here, 95% of the copy bandwidth;
// 32 and 64 tokens as N take 214 and 243 against 223 and 228 with the tiles, and
// over 32,000 x 2,048 39 and 68 against 33 and 34: N is 16 at most.  The gradient
// of 1, 8 and 16 tokens: 793, 751 and 696 us with the tiles, 677, 683 and 687
// here.)  Every CTA owns a contiguous range of the
// vocabulary, in units of 32 rows, and streams it once through a ring of TMA
// stages of 64 columns; a thread of the epilogue owns a vocabulary row of the
// tile and keeps each token's running maximum and sum over all its rows, so
// lanes and warps are joined once per CTA.
//
// Warp roles (192 threads): warps 0..3 epilogue, warp 4 TMA, warp 5 MMA issue.
#include <algorithm>

#include "device_common.cuh"
#include "grad_internal.h"
#include "per_device.h"
#include "tcgen05_common.cuh"

namespace engram {

namespace {

constexpr int kThreads = 192;
constexpr int kWarpTma = 4, kWarpMma = 5;
constexpr int kUnit = 32;               // vocabulary rows that a CTA's range is a multiple of
constexpr int kRowsBytes = kBM * kBK * 2;  // 16 KB: 128 rows x 64
constexpr int kN = kFewTokens;          // tokens of an MMA
constexpr int kSegment = 16;            // k-blocks per accumulator (as in kernels_grad.cu)
constexpr float kLog2e = 1.4426950408889634f;

struct Layout {
    static constexpr int kStage = kRowsBytes + kN * kBK * 2;
    static constexpr int kStages = 216 * 1024 / kStage;
    static constexpr int kOffBar = kStages * kStage;
    static constexpr int kNumBars = 2 * kStages + 4;
    static constexpr int kOffTmem = kOffBar + kNumBars * 8;
    static constexpr int kOffFlag = kOffTmem + 4;
    static constexpr int kOffJoin = (kOffFlag + 4 + 15) / 16 * 16;  // float2 [4][kN]
    static constexpr int kSmem = kOffJoin + 4 * kN * 8 + 1024;
    static_assert(kStage % 1024 == 0 && kSmem <= 232448, "");
    static constexpr uint32_t kTmemCols = 2 * kN;  // two accumulators (a power of two, at least 32)
};

__host__ __device__ constexpr uint32_t few_idesc() {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kN >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
}

// 32 lanes x 16 consecutive 32-bit columns of tensor memory.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// (maximum, sum of exponentials below it) of two sets joined.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
    const float top = fmaxf(m, m2);
    const float base = top == -INFINITY ? 0.f : top;
    s = s * exp2f((m - base) * kLog2e) + s2 * exp2f((m2 - base) * kLog2e);
    m = top;
}

// kDz: dz of vocabulary rows [v0, v0 + rows); else the statistics of all rows.
// tmV: head rows in boxes of 128 x 64, tmU: of 32 x 64 (a range's last tile),
// tmX: x in boxes of kN x 64.
template <bool kDz>
__global__ void __launch_bounds__(kThreads, 1)
k_few(const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmU,
      const __grid_constant__ CUtensorMap tmX, const FewArgs a) {
    using L = Layout;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~(uintptr_t)1023);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto full = [&](int s) { return sbase + L::kOffBar + 8u * (uint32_t)s; };
    auto empty = [&](int s) { return sbase + L::kOffBar + 8u * (uint32_t)(kStages + s); };
    auto tfull = [&](int acc) { return sbase + L::kOffBar + 8u * (uint32_t)(2 * kStages + acc); };
    auto tempty = [&](int acc) { return sbase + L::kOffBar + 8u * (uint32_t)(2 * kStages + 2 + acc); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffFlag);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kOffTmem);
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full(s), 1u);
            mbar_init(empty(s), 1u);
        }
        for (int acc = 0; acc < 2; ++acc) {
            mbar_init(tfull(acc), 1u);
            mbar_init(tempty(acc), 4u);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWarpMma) tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();

    // this CTA's vocabulary rows [r0, r1) of the piece
    const int units = (a.rows + kUnit - 1) / kUnit;
    const int r0 = (int)((int64_t)units * blockIdx.x / gridDim.x) * kUnit;
    const int r1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x) * kUnit;
    const int tiles = (r1 - r0 + kBM - 1) / kBM;
    const int kb_all = a.kb;
    const long long lim = a.wait_limit_ns;
    auto fail = [&]() {
        *abort_flag = 1;
        atomicOr(a.err, kErrTimeout);
    };
    float2* joined = reinterpret_cast<float2*>(smem + L::kOffJoin);

    if (warp == kWarpTma) {
        if (lane == 0) {
            int it = 0;
            bool ok = !a.starve;
            for (int i = 0; i < tiles && ok; ++i) {
                const int row = r0 + i * kBM, n = min(kBM, r1 - row);  // n: a multiple of 32
                for (int kb = 0; kb < kb_all; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(empty(s), ((uint32_t)(it / kStages) & 1u) ^ 1u, abort_flag, lim)) {
                        fail();
                        ok = false;
                        break;
                    }
                    const uint32_t sv = sbase + (uint32_t)(s * L::kStage), sx = sv + kRowsBytes;
                    mbar_expect_tx(full(s), (uint32_t)((n + kN) * kBK * 2));
                    if (n == kBM)
                        tma_load_2d(sv, &tmV, full(s), kb * kBK, row);
                    else  // (the rest of the tile keeps what it held: those rows are not used)
                        for (int u = 0; u < n; u += kUnit)
                            tma_load_2d(sv + (uint32_t)(u * kBK * 2), &tmU, full(s), kb * kBK, row + u);
                    tma_load_2d(sx, &tmX, full(s), kb * kBK, 0);
                }
            }
        }
    } else if (warp == kWarpMma) {
        if (lane == 0) {
            int it = 0, use = 0;
            bool ok = true;
            for (int i = 0; i < tiles && ok; ++i) {
                uint32_t d_tmem = 0;
                int seg = 0;
                for (int kb = 0; kb < kb_all; ++kb, ++it) {
                    const int s = it % kStages;
                    if (seg == 0) {
                        if (!mbar_wait(tempty(use & 1), ((uint32_t)(use >> 1) & 1u) ^ 1u, abort_flag, lim)) {
                            fail();
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        d_tmem = tmem_base + (uint32_t)((use & 1) * kN);
                    }
                    if (!mbar_wait(full(s), (uint32_t)(it / kStages) & 1u, abort_flag, lim)) {
                        fail();
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sv = sbase + (uint32_t)(s * L::kStage);
                    const uint64_t ad = sdesc_sw128(sv), bd = sdesc_sw128(sv + kRowsBytes);
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        umma_f16kind(d_tmem, ad + 2ull * k, bd + 2ull * k, few_idesc(), (seg != 0) || (k != 0));
                    umma_commit(empty(s));
                    if (++seg == kSegment || kb + 1 == kb_all) {
                        umma_commit(tfull(use & 1));
                        ++use;
                        seg = 0;
                    }
                }
            }
        }
    } else {
        float m[kN], s[kN];
        if (!kDz)
#pragma unroll
            for (int t = 0; t < kN; ++t) {
                m[t] = -INFINITY;
                s[t] = 0.f;
            }
        int use = 0;
        bool ok = true;
        for (int i = 0; i < tiles && ok; ++i) {
            float z[kN];
            for (int seg = 0; seg < kb_all && ok; seg += kSegment, ++use) {
                int ready = 1;
                if (lane == 0) ready = mbar_wait(tfull(use & 1), (uint32_t)(use >> 1) & 1u, abort_flag, lim);
                ok = __shfl_sync(0xFFFFFFFFu, ready, 0) != 0;
                if (!ok && lane == 0) fail();
                tc_fence_after();
                const uint32_t taddr = tmem_base + (uint32_t)((use & 1) * kN) + ((uint32_t)(warp * 32) << 16);
                uint32_t r[kN];
                tmem_ld16(taddr, r);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < kN; ++j) z[j] = seg ? z[j] + __uint_as_float(r[j]) : __uint_as_float(r[j]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(tempty(use & 1));
            }
            if (!ok) break;
            const int row = r0 + i * kBM + warp * 32 + lane;  // within the piece
            const int64_t v = a.v0 + row;                      // within the vocabulary
            const bool in = row < r1 && v < a.vocab;
            if constexpr (kDz) {
                if (row >= r1) continue;  // (uniform in the warp: ranges are multiples of 32)
                const float unit = loss_unit(a.dloss);
                uint16_t* out = a.dz + (int64_t)(row >> 6) * (128 * 64) + (row & 63);
#pragma unroll
                for (int t = 0; t < kN; ++t) {
                    // (rows of tokens past T are zero: dhead's product reads 64 of them)
                    float d = 0.f;
                    if (t < a.T) {
                        const int label = a.labels[t];
                        // (z - lse first: exact where p is near 1)
                        float p = exp2f((z[t] - a.lse[t]) * kLog2e);
                        if (label == v) p -= 1.f;
                        if (in && label >= 0 && label < a.vocab) d = p * (a.dloss[t] / unit);
                    }
                    out[t * 64] = (uint16_t)(bf16x2_pack_rn(d, d) & 0xFFFFu);
                }
                for (int t = kN; t < 64; ++t) out[t * 64] = 0;
            } else if (in) {
#pragma unroll
                for (int t = 0; t < kN; ++t) {
                    if (t < a.T && a.labels[t] == v) a.zlabel[t] = z[t];
                    const float e = z[t] == m[t] ? 1.f : exp2f(-fabsf(z[t] - m[t]) * kLog2e);
                    s[t] = z[t] > m[t] ? fmaf(s[t], e, 1.f) : s[t] + e;
                    m[t] = fmaxf(m[t], z[t]);
                }
            }
        }
        if constexpr (!kDz) {
#pragma unroll
            for (int t = 0; t < kN; ++t) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    join(m[t], s[t], __shfl_xor_sync(0xFFFFFFFFu, m[t], o), __shfl_xor_sync(0xFFFFFFFFu, s[t], o));
                if (lane == 0) joined[warp * kN + t] = make_float2(m[t], s[t]);
            }
        }
    }

    __syncthreads();
    if (!kDz && (int)threadIdx.x < a.T) {
        float2 x = joined[threadIdx.x];
        for (int w = 1; w < 4; ++w) join(x.x, x.y, joined[w * kN + threadIdx.x].x, joined[w * kN + threadIdx.x].y);
        a.part[(int64_t)blockIdx.x * a.T + threadIdx.x] = x;
    }
    if (*abort_flag) {
        // let copies and MMAs still in flight land before TMEM is freed
        if (threadIdx.x == 0) {
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
        }
        __syncthreads();
    }
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem_base, L::kTmemCols);
    }
}

template <bool kDz>
cudaError_t launch(const FewArgs& a, const uint16_t* x, const uint16_t* head, int64_t head_rows, int dim,
                   int groups, cudaStream_t s) {
    CUtensorMap tmV, tmU, tmX;
    cudaError_t e = make_tma_16bit(&tmV, head, head_rows, dim, kBM, false);
    if (e == cudaSuccess) e = make_tma_16bit(&tmU, head, head_rows, dim, kUnit, false);
    if (e == cudaSuccess) e = make_tma_16bit(&tmX, x, a.T, dim, kN, false);
    auto kern = k_few<kDz>;
    static PerDevice allowed;
    if (e == cudaSuccess) e = allow_shared(allowed, kern, Layout::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(groups);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tmV, tmU, tmX, a);
}

}  // namespace

int few_groups(int64_t rows) {
    return (int)std::min<int64_t>(device_sm_count(), (rows + kUnit - 1) / kUnit);
}

cudaError_t launch_few_lse(const FewArgs& a, const uint16_t* x, const uint16_t* head, int dim, cudaStream_t s) {
    return launch<false>(a, x, head, a.vocab, dim, few_groups(a.rows), s);
}

cudaError_t launch_few_dz(const FewArgs& a, const uint16_t* x, const uint16_t* head, int dim, cudaStream_t s) {
    return launch<true>(a, x, head, a.vocab - a.v0, dim, few_groups(a.rows), s);
}

}  // namespace engram
