// The gate with an 8-bit checkpoint of its activations, and the gate's backward
// pass (sm_103a).
//
// Both read a token's rows (hidden and keys of every branch, the value, and
// backward the gradient) twice, once for sums over the columns and once for the
// outputs, and both are bound by memory if the second reading is not from HBM.
// So a cluster of CTAs keeps a token in shared memory between the two.  At hc 4,
// d 5,120 and 2,048 tokens (GB300, copy bandwidth 6.77 TB/s): forward with fp32
// kv 86 us (475 MB, 81%; a block per token that reads hidden again 97), with BF16
// kv 76; backward from the checkpoint 81 us (370 MB, 67%: the kernel 75, neither HBM
// nor its issue slots full, and the weights' sums 6; two kernels over the tokens
// 214), from BF16 kv 89, from fp32 kv 111.  With 5 to 8 branches the backward kernel
// spills 150 to 320 bytes a thread: from the checkpoint 115 us at hc 8, d 2,560 and
// 172 at hc 5, d 4,096, where the bytes take 52 and 54.
#include <algorithm>

#include "grad_internal.h"
#include "per_device.h"
#include "tcgen05_common.cuh"
#include "train_common.cuh"

namespace engram {

namespace {

// ---- 8-bit blocks ---------------------------------------------------------------------------
// MXFP8 of 32 values held by four neighbouring lanes, 8 each: the block's
// exponent is the smallest for which its largest magnitude, scaled, stays at or
// below E4M3's 448 (so no value saturates: above 1.75 x 2^e the exponent is one
// higher), the codes are rounded to nearest even.  A block that holds an
// infinity or NaN decodes to NaN.  Zeros, and blocks below 2^-118, take exponent 0.
__device__ __forceinline__ uint2 encode_mx8(const float (&f)[8], uint32_t& exponent) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(f[j]) & 0x7FFFFFFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (m >= 0x7F800000u) {
        exponent = 255u;
        return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    }
    const int e = (int)(m >> 23) - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    exponent = (uint32_t)max(e, 0);
    const float inv = __uint_as_float((254u - exponent) << 23);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint16_t c;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
            : "=h"(c)
            : "f"(f[2 * j + 1] * inv), "f"(f[2 * j] * inv));
        w[j] = c;
    }
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}
__device__ __forceinline__ void decode_mx8(uint2 w, uint32_t exponent, float (&f)[8]) {
    const float s = e8m0_to_f32(exponent);
    const uint32_t h[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t x;
        asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
            : "=r"(x)
            : "r"(h[j]));
        const float2 v = __half22float2(*reinterpret_cast<__half2*>(&x));
        f[2 * j] = v.x * s;
        f[2 * j + 1] = v.y * s;
    }
}

// Sums of the block's threads for kN values, in every thread.
template <int kN>
__device__ __forceinline__ void block_sum(float (&v)[kN], float (*sm)[kN]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int k = 0; k < kN; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    __syncthreads();
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < kN; ++k) sm[warp][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += sm[w][k];
        v[k] = s;
    }
}

// ---- gate backward --------------------------------------------------------------------------
// Saved activations of token t, 8 columns at a time: element index `at` within
// the token's hidden [hc][d] or kv [(hc + 1) d].
template <int kSaved>
struct Saved {
    const uint16_t* h;
    const void* kv;
    const uint8_t* codes;
    const uint8_t* scales;
    int hd;  // hc * d
    __device__ __forceinline__ Saved(const GateTrain& a, int64_t t) {
        hd = a.hc * a.d;
        if (kSaved == kSavedMx) {
            codes = a.codes + t * (int64_t)(2 * hd + a.d);
            scales = a.scales + t * (int64_t)((2 * hd + a.d) / 32);
        } else {
            h = a.hidden + t * (int64_t)hd;
            kv = static_cast<const char*>(a.kv) + t * (int64_t)(hd + a.d) * (kSaved == kSavedF32 ? 4 : 2);
        }
    }
    __device__ __forceinline__ void mx(int64_t at, float (&f)[8]) const {
        decode_mx8(*reinterpret_cast<const uint2*>(codes + at), scales[at / 32], f);
    }
    __device__ __forceinline__ void hidden(int64_t at, float (&f)[8]) const {
        if (kSaved == kSavedMx)
            mx(at, f);
        else
            unpack8(*reinterpret_cast<const uint4*>(h + at), f);
    }
    __device__ __forceinline__ void keyvalue(int64_t at, float (&f)[8]) const {
        if (kSaved == kSavedMx)
            mx(hd + at, f);
        else if (kSaved == kSavedF32)
            load8_f32(static_cast<const float*>(kv) + at, f);
        else
            unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(kv) + at), f);
    }
};

// The factors of token-branch gradients, from the sums over its columns
// S_kk = sum k^2, S_hh = sum h^2, S = sum h w k, D = sum dy v:
//   x = rh rk S / sqrt(d), s = copysign(sqrt(max(|x|, 1e-6)), x), g = sigmoid(s)
//   dx = D g (1 - g) / (2 |s|) where |x| > 1e-6, else 0
//   dh = dy + (dx rh rk / sqrt(d)) w k - (dx x rh^2 / d) h, dk likewise
__device__ __forceinline__ float4 gate_factors(float skk, float shh, float s, float dyv, int d,
                                               float eps) {
    const float inv_d = 1.0f / (float)d;
    const float rh = 1.0f / sqrtf(shh * inv_d + eps);
    const float rk = 1.0f / sqrtf(skk * inv_d + eps);
    const float rs = rh * rk / sqrtf((float)d);
    const float x = rs * s;
    const float root = sqrtf(fmaxf(fabsf(x), 1e-6f));
    // g (1 - g) = e / (1 + e)^2 with e = exp(-|s|): 1 - g itself would lose a
    // saturated gate's slope to cancellation
    const float e = expf(-root);
    const float g = (signbit(x) ? e : 1.0f) / (1.0f + e);
    const float dx = fabsf(x) > 1e-6f ? dyv * e / ((1.0f + e) * (1.0f + e) * 2.0f * root) : 0.f;
    return make_float4(dx * rs, dx * x * rh * rh * inv_d, dx * x * rk * rk * inv_d, g);
}

// ---- fused: one pass over a token's activations --------------------------------------------
// A cluster of CTAs takes one token at a time, each CTA a range of its columns:
// bulk copies bring the range of every row (hidden, keys, value, dout) into a
// ring of stages; phase 1 sums over the columns, the CTAs exchange 4 sums per
// branch through distributed shared memory, and phase 2 reads the stage again
// for the outputs, so each byte comes from HBM once.  Phase 2 of token i - 1
// runs after phase 1 of token i, which hides the exchange.  A thread of the
// compute warps owns 8 columns of every branch: its norm weights and its share
// of their gradient stay in registers over all tokens of the cluster.  Two more
// warps: one loads, one adds the warps' sums, exchanges them and turns them into
// the factors, so that the compute warps wait for data and factors only.
// What bounds it beside HBM is the issue rate, so the arithmetic runs on pairs of
// values (f32x2), and an 8-bit block's scale multiplies the sums and factors
// instead of its values.
constexpr int kFusedMaxWarps = 10;  // compute warps
constexpr int kFusedSlots = 4;      // exchanges: those of the tokens in flight and one more
constexpr int kFusedMaxStages = 8;
constexpr int kFusedFixed =
    kFusedSlots * (kFusedMaxWarps * 32 + 8 * 32 + 32) * 4 + (2 * kFusedMaxStages + 3 * kFusedSlots) * 8 + 128;
static_assert(kFusedFixed % 16 == 0, "");

template <int kSaved>
__host__ __device__ constexpr int fused_row_bytes(int hc) {  // of all rows, per column
    return kSaved == kSavedMx ? (2 * hc + 1) + 2 * hc
                              : 2 * hc + (hc + 1) * (kSaved == kSavedF32 ? 4 : 2) + 2 * hc;
}
template <int kSaved>
__host__ __device__ constexpr int fused_stage_bytes(int hc, int cols) {
    return (fused_row_bytes<kSaved>(hc) * cols + (kSaved == kSavedMx ? (2 * hc + 1) * cols / 32 : 0) +
            127) / 128 * 128;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Eight E4M3 codes without their block's scale.
__device__ __forceinline__ void decode8(uint2 w, f32x2 (&f)[4]) {
    const uint32_t h[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t x;
        asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
            : "=r"(x)
            : "r"(h[j]));
        const float2 v = __half22float2(*reinterpret_cast<__half2*>(&x));
        f[j] = pair(v.x, v.y);
    }
}

// Sums over the warp of kN values (a power of two, at most 32), each exchange
// halving what a lane still holds; lane l ends with value l / (32 / kN).
template <int kN>
__device__ __forceinline__ float warp_sums(float (&v)[kN], int lane) {
#pragma unroll
    for (int k = 0; (kN >> k) > 1; ++k) {
        const int o = 16 >> k, half = kN >> (k + 1);
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int j = 0; j < half; ++j) {
            const float send = up ? v[j] : v[j + half];
            const float keep = up ? v[j + half] : v[j];
            v[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
        }
    }
#pragma unroll
    for (int o = 16 / kN; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
    return v[0];
}

// kExact: hc == kHc (no branch is left out).
template <int kSaved, int kHc, bool kExact>
__global__ void __launch_bounds__((kFusedMaxWarps + 2) * 32, kHc == 1 ? 2 : 1)
k_gate_backward_fused(const GateTrain a, int stages, int cs, int lag) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kSums = 4 * kHc;
    const int hc = kExact ? kHc : a.hc;
    const int d = a.d;
    const int rank = cs > 1 ? (int)cluster_ctarank() : 0;
    const int groups = d / 256;  // 256 columns: a warp's
    const int g0 = groups * rank / cs, warps = groups * (rank + 1) / cs - g0;
    const int max_cols = ((groups + cs - 1) / cs) * 256;
    const int cols = warps * 256, col0 = g0 * 256;
    const int stage_bytes = fused_stage_bytes<kSaved>(hc, max_cols);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int loader = (int)(blockDim.x >> 5) - 2, joiner = loader + 1;

    float* wred = reinterpret_cast<float*>(smem);            // [slots][warps][32]
    float* red = wred + kFusedSlots * kFusedMaxWarps * 32;   // [slots][8 ranks][32]
    float4* fac = reinterpret_cast<float4*>(red + kFusedSlots * 8 * 32);  // [slots][8]
    uint64_t* bars = reinterpret_cast<uint64_t*>(fac + kFusedSlots * 8);
    volatile int* aborted = reinterpret_cast<volatile int*>(bars + 2 * kFusedMaxStages + 3 * kFusedSlots);
    uint8_t* ring = smem + (kFusedFixed + 127) / 128 * 128;
    auto bar = [&](int s) { return smem_u32(bars + s); };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(kFusedMaxStages + s); };
    auto parts = [&](int i) { return bar(2 * kFusedMaxStages + i % kFusedSlots); };
    auto sums_in = [&](int i) { return bar(2 * kFusedMaxStages + kFusedSlots + i % kFusedSlots); };
    auto factors = [&](int i) { return bar(2 * kFusedMaxStages + 2 * kFusedSlots + i % kFusedSlots); };
    auto slot_phase = [&](int i) { return (uint32_t)(i / kFusedSlots) & 1u; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full(s), kSaved == kSavedMx ? 33u : 1u);
            mbar_init(empty(s), (uint32_t)warps);
        }
        for (int s = 0; s < kFusedSlots; ++s) {
            mbar_init(parts(s), (uint32_t)warps);
            mbar_init(sums_in(s), (uint32_t)cs);
            mbar_init(factors(s), 1u);
        }
        *aborted = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (cs > 1) cluster_sync();
    pdl_launch_dependents();
    pdl_wait();

    const int64_t cluster = blockIdx.x / cs, clusters = gridDim.x / cs;
    const int n = (int)((a.T - cluster + clusters - 1) / clusters);
    auto token = [&](int i) { return cluster + (int64_t)i * clusters; };
    // Bounded waits of all 32 lanes; after one ran out every other ends too.
    auto ready = [&](bool ok) {
        if (ok) return true;
        *aborted = 1;
        atomicOr(a.err, kErrTimeout);
        return false;
    };
    auto wait = [&](uint32_t b, uint32_t phase) {
        return __all_sync(0xFFFFFFFFu, ready(mbar_wait(b, phase, aborted, a.wait_limit_ns)));
    };

    if (warp == loader) {
        // rows of a stage: hidden [hc], keys and value [hc + 1], dout [hc]
        const int rows = 3 * hc + 1;
        for (int i = 0; i < n; ++i) {
            const int s = i % stages;
            if (!wait(empty(s), ((uint32_t)(i / stages) & 1u) ^ 1u)) break;
            const int64_t t = token(i);
            const uint32_t base = smem_u32(ring + s * stage_bytes);
            if (lane == 0) mbar_expect_tx(full(s), (uint32_t)(fused_row_bytes<kSaved>(hc) * cols));
            __syncwarp();
            for (int r = lane; r < rows; r += 32) {
                const char* src;
                int size, off;  // bytes per value; of the row within the stage
                if (r >= 2 * hc + 1) {
                    const int b = r - (2 * hc + 1);
                    size = 2;
                    src = reinterpret_cast<const char*>(a.dout + (t * hc + b) * d);
                    off = (fused_row_bytes<kSaved>(hc) - 2 * hc + 2 * b) * max_cols;
                } else if (kSaved == kSavedMx) {
                    size = 1;
                    src = reinterpret_cast<const char*>(a.codes + (t * (2 * hc + 1) + r) * d);
                    off = r * max_cols;
                } else if (r < hc) {
                    size = 2;
                    src = reinterpret_cast<const char*>(a.hidden + (t * hc + r) * d);
                    off = 2 * r * max_cols;
                } else {
                    size = kSaved == kSavedF32 ? 4 : 2;
                    src = static_cast<const char*>(a.kv) + (t * (hc + 1) + (r - hc)) * d * size;
                    off = (2 * hc + size * (r - hc)) * max_cols;
                }
                bulk_load(base + (uint32_t)off, src + (int64_t)col0 * size, (uint32_t)(cols * size), full(s));
            }
            if (kSaved == kSavedMx) {  // the exponents, 4 at a time
                const uint32_t dst = base + (uint32_t)(fused_row_bytes<kSaved>(hc) * max_cols);
                const int per = cols / 128, all = (2 * hc + 1) * per;
                for (int x = lane; x < all; x += 32) {
                    const int r = x / per, c = x - r * per;
                    const uint8_t* src = a.scales + (t * (2 * hc + 1) + r) * (d / 32) + col0 / 32 + 4 * c;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                                     dst + (uint32_t)(r * (max_cols / 32) + 4 * c)),
                                 "l"(src)
                                 : "memory");
                }
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full(s))
                             : "memory");
            }
        }
        if (kSaved == kSavedMx) asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == joiner) {
        for (int i = 0; i < n; ++i) {
            const int slot = i % kFusedSlots;
            if (!wait(parts(i), slot_phase(i))) break;
            float s = 0.f;
            if (lane < kSums)
                for (int x = 0; x < warps; ++x) s += wred[(slot * kFusedMaxWarps + x) * 32 + lane];
            float* out = red + (slot * 8 + rank) * 32 + lane;
            if (cs == 1) {
                *out = s;
                __syncwarp();
            } else {
                const uint32_t at = smem_u32(out);
                for (int r = 0; r < cs; ++r)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_rank(at, (uint32_t)r)), "f"(s)
                                 : "memory");
                __syncwarp();
                if (lane < cs) mbar_arrive_cluster(map_rank(sums_in(i), (uint32_t)lane));
                if (!__all_sync(0xFFFFFFFFu, ready(mbar_wait_cluster(sums_in(i), slot_phase(i), aborted,
                                                                     a.wait_limit_ns))))
                    break;
            }
            if (lane < hc) {
                float x[4] = {};
                for (int r = 0; r < cs; ++r) {
                    const float4 y = *reinterpret_cast<const float4*>(red + (slot * 8 + r) * 32 + 4 * lane);
                    x[0] += y.x; x[1] += y.y; x[2] += y.z; x[3] += y.w;
                }
                fac[slot * 8 + lane] = gate_factors(x[0], x[1], x[2], x[3], d, a.eps);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(factors(i));
        }
    } else if (warp < warps) {
        const int lc = warp * 256 + lane * 8;  // column within the CTA's range
        f32x2 w[kHc][4], acc[kHc][4];
#pragma unroll
        for (int b = 0; b < kHc; ++b) {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[b][j] = 0ull;
            if (kExact || b < hc) {
                float f[8];
                load8_f32(a.wqk + (int64_t)b * d + col0 + lc, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[b][j] = pair(f[2 * j], f[2 * j + 1]);
            }
        }
        // row r (hidden [hc], keys and value [hc + 1]) of a stage, this thread's
        // columns, without the scale that is returned
        auto saved = [&](const uint8_t* st, int r, f32x2 (&f)[4]) {
            if (kSaved == kSavedMx) {
                decode8(*reinterpret_cast<const uint2*>(st + r * max_cols + lc), f);
                return e8m0_to_f32(st[fused_row_bytes<kSaved>(hc) * max_cols + r * (max_cols / 32) + lc / 32]);
            }
            if (r < hc || kSaved == kSavedBf16) {
                unpack8(*reinterpret_cast<const uint4*>(st + 2 * (r * max_cols + lc)), f);
            } else {
                const ulonglong2* p = reinterpret_cast<const ulonglong2*>(st + 2 * hc * max_cols +
                                                                          4 * ((r - hc) * max_cols + lc));
                f[0] = p[0].x; f[1] = p[0].y; f[2] = p[1].x; f[3] = p[1].y;
            }
            return 1.0f;
        };
        auto dout = [&](const uint8_t* st, int b) {
            return *reinterpret_cast<const uint4*>(
                st + (fused_row_bytes<kSaved>(hc) - 2 * hc + 2 * b) * max_cols + 2 * lc);
        };
        for (int i = 0; i < n + lag; ++i) {
            const int p = i - lag;  // phase 2's token
            const bool image = p >= 0 && a.windows[token(p)].x == kDead;
            if (i < n) {
                const int s = i % stages;
                const uint8_t* st = ring + s * stage_bytes;
                if (!wait(full(s), (uint32_t)(i / stages) & 1u)) break;
                float sum[kSums];
                f32x2 v[4];
                const float cv = saved(st, 2 * hc, v);
#pragma unroll
                for (int b = 0; b < kHc; ++b) {
                    float* sb = sum + 4 * b;
                    sb[0] = sb[1] = sb[2] = sb[3] = 0.f;
                    if (!kExact && b >= hc) continue;
                    f32x2 h[4], k[4], dy[4];
                    const float ch = saved(st, b, h), ck = saved(st, hc + b, k);
                    unpack8(dout(st, b), dy);
                    f32x2 q[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        q[0] = fma2(k[j], k[j], q[0]);
                        q[1] = fma2(h[j], h[j], q[1]);
                        q[2] = fma2(mul2(h[j], w[b][j]), k[j], q[2]);
                        q[3] = fma2(dy[j], v[j], q[3]);
                    }
                    sb[0] = both(q[0]);
                    sb[1] = both(q[1]);
                    sb[2] = both(q[2]);
                    sb[3] = both(q[3]);
                    if (kSaved == kSavedMx) {
                        sb[0] *= ck * ck;
                        sb[1] *= ch * ch;
                        sb[2] *= ch * ck;
                        sb[3] *= cv;
                    }
                }
                const float mine = warp_sums<kSums>(sum, lane);
                constexpr int kPer = 32 / kSums;
                if (lane % kPer == 0)
                    wred[((i % kFusedSlots) * kFusedMaxWarps + warp) * 32 + lane / kPer] = mine;
                __syncwarp();
                if (lane == 0) mbar_arrive(parts(i));
            }
            if (p < 0) continue;
            const int s = p % stages;
            const uint8_t* st = ring + s * stage_bytes;
            const int64_t t = token(p);
            if (!wait(factors(p), slot_phase(p))) break;
            const float4* fp = fac + (p % kFusedSlots) * 8;
            uint16_t* dh_t = a.dhidden + t * (int64_t)hc * d + col0 + lc;
            uint16_t* dkv_t = a.dkv + t * (int64_t)(hc + 1) * d + col0 + lc;
            f32x2 dv[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int b = 0; b < kHc; ++b) {
                if (!kExact && b >= hc) continue;
                const uint4 raw = dout(st, b);
                uint4 odh = raw, odk = make_uint4(0u, 0u, 0u, 0u);
                if (!image) {
                    const float4 f = fp[b];
                    f32x2 dy[4], h[4], k[4], dh[4], dk[4];
                    unpack8(raw, dy);
                    const float ch = saved(st, b, h), ck = saved(st, hc + b, k);
                    const float xk = f.x * ck, xh = f.x * ch, yh = -f.y * ch, zk = -f.z * ck, xhk = xk * ch;
                    const f32x2 xk2 = pair(xk, xk), xh2 = pair(xh, xh), yh2 = pair(yh, yh), zk2 = pair(zk, zk),
                                xhk2 = pair(xhk, xhk), g2 = pair(f.w, f.w);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        dh[j] = fma2(xk2, mul2(w[b][j], k[j]), fma2(yh2, h[j], dy[j]));
                        dk[j] = fma2(xh2, mul2(w[b][j], h[j]), mul2(zk2, k[j]));
                        dv[j] = fma2(g2, dy[j], dv[j]);
                        acc[b][j] = fma2(xhk2, mul2(h[j], k[j]), acc[b][j]);
                    }
                    odh = pack8(dh);
                    odk = pack8(dk);
                }
                __stcs(reinterpret_cast<uint4*>(dh_t + (int64_t)b * d), odh);
                __stcs(reinterpret_cast<uint4*>(dkv_t + (int64_t)b * d), odk);
            }
            __stcs(reinterpret_cast<uint4*>(dkv_t + (int64_t)hc * d), pack8(dv));
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(s));
        }
        float* part = a.dw_part + cluster * hc * d + col0 + lc;
#pragma unroll
        for (int b = 0; b < kHc; ++b)
            if (kExact || b < hc) {
                float f[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = unpair(acc[b][j]);
                    f[2 * j] = x.x;
                    f[2 * j + 1] = x.y;
                }
                store8_f32(part + (int64_t)b * d, f);
            }
    }
    __syncthreads();
    if (*aborted) {  // let copies in flight land
        if (threadIdx.x == 0) {
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
        }
        __syncthreads();
    }
    if (cs > 1) cluster_sync();  // no arrival may target a CTA that exited
}

// ---- gate with checkpoint, one pass -------------------------------------------------------
// The same shape for the forward step: phase 1 packs the rows and sums, phase 2
// turns the gates into hidden + g v from the stage.  Bound by HBM.
template <bool kF32Kv>
__host__ __device__ constexpr int ckpt_stage_bytes(int hc, int cols) {
    return (2 * hc + (hc + 1) * (kF32Kv ? 4 : 2)) * cols;
}

__device__ __forceinline__ uint2 encode_mx8(const f32x2 (&v)[4], uint32_t& exponent) {
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 x = unpair(v[j]);
        f[2 * j] = x.x;
        f[2 * j + 1] = x.y;
    }
    return encode_mx8(f, exponent);
}

template <bool kF32Kv, int kHc, bool kExact>
__global__ void __launch_bounds__((kFusedMaxWarps + 2) * 32, kHc <= 2 ? 2 : 1)
k_gate_checkpoint_fused(const GateTrain a, int stages, int cs, int lag) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kSums = 4 * kHc;  // (three used per branch)
    const int hc = kExact ? kHc : a.hc;
    const int d = a.d;
    const int rank = cs > 1 ? (int)cluster_ctarank() : 0;
    const int groups = d / 256;
    const int g0 = groups * rank / cs, warps = groups * (rank + 1) / cs - g0;
    const int max_cols = ((groups + cs - 1) / cs) * 256;
    const int cols = warps * 256, col0 = g0 * 256;
    const int stage_bytes = ckpt_stage_bytes<kF32Kv>(hc, max_cols);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int loader = (int)(blockDim.x >> 5) - 2, joiner = loader + 1;

    float* wred = reinterpret_cast<float*>(smem);            // [slots][warps][32]
    float* red = wred + kFusedSlots * kFusedMaxWarps * 32;   // [slots][8 ranks][32]
    float* gate = red + kFusedSlots * 8 * 32;                // [slots][8]
    uint64_t* bars = reinterpret_cast<uint64_t*>(gate + kFusedSlots * 32);
    volatile int* aborted = reinterpret_cast<volatile int*>(bars + 2 * kFusedMaxStages + 3 * kFusedSlots);
    uint8_t* ring = smem + (kFusedFixed + 127) / 128 * 128;
    auto bar = [&](int s) { return smem_u32(bars + s); };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(kFusedMaxStages + s); };
    auto parts = [&](int i) { return bar(2 * kFusedMaxStages + i % kFusedSlots); };
    auto sums_in = [&](int i) { return bar(2 * kFusedMaxStages + kFusedSlots + i % kFusedSlots); };
    auto gates_in = [&](int i) { return bar(2 * kFusedMaxStages + 2 * kFusedSlots + i % kFusedSlots); };
    auto slot_phase = [&](int i) { return (uint32_t)(i / kFusedSlots) & 1u; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full(s), 1u);
            mbar_init(empty(s), (uint32_t)warps);
        }
        for (int s = 0; s < kFusedSlots; ++s) {
            mbar_init(parts(s), (uint32_t)warps);
            mbar_init(sums_in(s), (uint32_t)cs);
            mbar_init(gates_in(s), 1u);
        }
        *aborted = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (cs > 1) cluster_sync();
    pdl_launch_dependents();
    pdl_wait();

    const int64_t cluster = blockIdx.x / cs, clusters = gridDim.x / cs;
    const int n = (int)((a.T - cluster + clusters - 1) / clusters);
    auto token = [&](int i) { return cluster + (int64_t)i * clusters; };
    auto ready = [&](bool ok) {
        if (ok) return true;
        *aborted = 1;
        atomicOr(a.err, kErrTimeout);
        return false;
    };
    auto wait = [&](uint32_t b, uint32_t phase) {
        return __all_sync(0xFFFFFFFFu, ready(mbar_wait(b, phase, aborted, a.wait_limit_ns)));
    };

    if (warp == loader) {
        for (int i = 0; i < n; ++i) {
            const int s = i % stages;
            if (!wait(empty(s), ((uint32_t)(i / stages) & 1u) ^ 1u)) break;
            const int64_t t = token(i);
            const uint32_t base = smem_u32(ring + s * stage_bytes);
            if (lane == 0) mbar_expect_tx(full(s), (uint32_t)ckpt_stage_bytes<kF32Kv>(hc, cols));
            __syncwarp();
            for (int r = lane; r < 2 * hc + 1; r += 32) {
                const int size = r < hc || !kF32Kv ? 2 : 4;
                const char* src = r < hc ? reinterpret_cast<const char*>(a.hidden + (t * hc + r) * d)
                                         : static_cast<const char*>(a.kv) + (t * (hc + 1) + (r - hc)) * d * size;
                const int off = (r < hc ? 2 * r : 2 * hc + size * (r - hc)) * max_cols;
                bulk_load(base + (uint32_t)off, src + (int64_t)col0 * size, (uint32_t)(cols * size), full(s));
            }
        }
    } else if (warp == joiner) {
        for (int i = 0; i < n; ++i) {
            const int slot = i % kFusedSlots;
            const int64_t t = token(i);
            const bool image = a.windows[t].x == kDead;  // (on its way during the wait)
            if (!wait(parts(i), slot_phase(i))) break;
            float s = 0.f;
            if (lane < kSums)
                for (int x = 0; x < warps; ++x) s += wred[(slot * kFusedMaxWarps + x) * 32 + lane];
            float* out = red + (slot * 8 + rank) * 32 + lane;
            if (cs == 1) {
                *out = s;
                __syncwarp();
            } else {
                const uint32_t at = smem_u32(out);
                for (int r = 0; r < cs; ++r)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_rank(at, (uint32_t)r)), "f"(s)
                                 : "memory");
                __syncwarp();
                if (lane < cs) mbar_arrive_cluster(map_rank(sums_in(i), (uint32_t)lane));
                if (!__all_sync(0xFFFFFFFFu, ready(mbar_wait_cluster(sums_in(i), slot_phase(i), aborted,
                                                                     a.wait_limit_ns))))
                    break;
            }
            if (lane < hc) {
                float x[3] = {};
                for (int r = 0; r < cs; ++r) {
                    const float4 y = *reinterpret_cast<const float4*>(red + (slot * 8 + r) * 32 + 4 * lane);
                    x[0] += y.x; x[1] += y.y; x[2] += y.z;
                }
                const float g = image ? 0.f : gate_from_sums(x[0], x[1], x[2], d, a.eps);
                gate[slot * 8 + lane] = g;
                if (a.gates && rank == 0) a.gates[t * hc + lane] = g;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(gates_in(i));
        }
    } else if (warp < warps) {
        const int lc = warp * 256 + lane * 8;
        f32x2 w[kHc][4];
#pragma unroll
        for (int b = 0; b < kHc; ++b)
            if (kExact || b < hc) {
                float f[8];
                load8_f32(a.wqk + (int64_t)b * d + col0 + lc, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[b][j] = pair(f[2 * j], f[2 * j + 1]);
            }
        auto hidden_raw = [&](const uint8_t* st, int b) {
            return *reinterpret_cast<const uint4*>(st + 2 * (b * max_cols + lc));
        };
        auto keyvalue = [&](const uint8_t* st, int r, f32x2 (&f)[4]) {
            if (kF32Kv) {
                const ulonglong2* p = reinterpret_cast<const ulonglong2*>(st + 2 * hc * max_cols +
                                                                          4 * (r * max_cols + lc));
                const ulonglong2 x = p[0], y = p[1];
                f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
            } else {
                unpack8(*reinterpret_cast<const uint4*>(st + 2 * ((hc + r) * max_cols + lc)), f);
            }
        };
        uint32_t id = n > 0 ? a.windows[token(0)].x : 0u;
        for (int i = 0; i < n + lag; ++i) {
            const int p = i - lag;  // phase 2's token
            // (slot 0 of the windows of the tokens in both phases, on their way early)
            const bool img = id == kDead;
            if (i + 1 < n) id = a.windows[token(i + 1)].x;
            const bool image = p >= 0 && a.windows[token(p)].x == kDead;
            if (i < n) {
                const int64_t t = token(i);
                const int s = i % stages;
                const uint8_t* st = ring + s * stage_bytes;
                uint8_t* codes = a.codes_out + t * (int64_t)(2 * hc + 1) * d + col0 + lc;
                uint8_t* scales = a.scales_out + t * (int64_t)((2 * hc + 1) * (d / 32)) + (col0 + lc) / 32;
                auto keep = [&](int r, const f32x2 (&f)[4]) {
                    uint32_t e;
                    uint2 c = encode_mx8(f, e);
                    if (img) c = make_uint2(0u, 0u), e = 0u;  // an image row's checkpoint is zero
                    __stcs(reinterpret_cast<uint2*>(codes + (int64_t)r * d), c);
                    if ((lane & 3) == 0) scales[r * (d / 32)] = (uint8_t)e;
                };
                if (!wait(full(s), (uint32_t)(i / stages) & 1u)) break;
                float sum[kSums];
#pragma unroll
                for (int b = 0; b < kHc; ++b) {
                    float* sb = sum + 4 * b;
                    sb[0] = sb[1] = sb[2] = sb[3] = 0.f;
                    if (!kExact && b >= hc) continue;
                    f32x2 h[4], k[4];
                    unpack8(hidden_raw(st, b), h);
                    keyvalue(st, b, k);
                    f32x2 q[3] = {0ull, 0ull, 0ull};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        q[0] = fma2(k[j], k[j], q[0]);
                        q[1] = fma2(h[j], h[j], q[1]);
                        q[2] = fma2(mul2(h[j], w[b][j]), k[j], q[2]);
                    }
                    sb[0] = both(q[0]);
                    sb[1] = both(q[1]);
                    sb[2] = both(q[2]);
                    keep(b, h);
                    keep(hc + b, k);
                }
                const float mine = warp_sums<kSums>(sum, lane);
                constexpr int kPer = 32 / kSums;
                if (lane % kPer == 0)
                    wred[((i % kFusedSlots) * kFusedMaxWarps + warp) * 32 + lane / kPer] = mine;
                __syncwarp();
                if (lane == 0) mbar_arrive(parts(i));
                f32x2 v[4];
                keyvalue(st, hc, v);
                keep(2 * hc, v);
            }
            if (p < 0) continue;
            const int s = p % stages;
            const uint8_t* st = ring + s * stage_bytes;
            uint16_t* ho = a.hidden_out + token(p) * (int64_t)hc * d + col0 + lc;
            if (!wait(gates_in(p), slot_phase(p))) break;
            const float* gp = gate + (p % kFusedSlots) * 8;
            f32x2 v[4];
            keyvalue(st, hc, v);
#pragma unroll
            for (int b = 0; b < kHc; ++b) {
                if (!kExact && b >= hc) continue;
                uint4 o = hidden_raw(st, b);
                if (!image) {
                    f32x2 h[4];
                    unpack8(o, h);
                    const f32x2 g = pair(gp[b], gp[b]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = fma2(g, v[j], h[j]);
                    o = pack8(h);
                }
                __stcs(reinterpret_cast<uint4*>(ho + (int64_t)b * d), o);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(s));
        }
    }
    __syncthreads();
    if (*aborted) {  // let copies in flight land
        if (threadIdx.x == 0) {
            const uint64_t t0 = globaltimer();
            while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
        }
        __syncthreads();
    }
    if (cs > 1) cluster_sync();  // no arrival may target a CTA that exited
}

// ---- geometries whose tokens do not fit the one-pass kernels ----------------------------------
// One block per token: per branch, the sums of h^2, k^2 and h w k while h and k
// are packed into the checkpoint; then hidden_out = h + g v for every branch
// from one read of v (h comes from L2 the second time).
template <bool kF32Kv>
__global__ void __launch_bounds__(320)
k_gate_checkpoint(const GateTrain a) {
    __shared__ float sm[10][3];
    __shared__ float gates[8];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    const int hc = a.hc, d = a.d, chunks = d / 8;
    const int kept = (2 * hc + 1) * d;
    const uint16_t* h = a.hidden + t * hc * (int64_t)d;
    uint16_t* ho = a.hidden_out + t * hc * (int64_t)d;
    uint8_t* codes = a.codes_out + t * (int64_t)kept;
    uint8_t* scales = a.scales_out + t * (int64_t)(kept / 32);
    if (a.windows[t].x == kDead) {  // an image row passes through; its checkpoint is zero
        for (int c = threadIdx.x; c < hc * chunks; c += blockDim.x)
            reinterpret_cast<uint4*>(ho)[c] = reinterpret_cast<const uint4*>(h)[c];
        for (int c = threadIdx.x; c < kept / 8; c += blockDim.x)
            reinterpret_cast<uint2*>(codes)[c] = make_uint2(0u, 0u);
        for (int c = threadIdx.x; c < kept / 32; c += blockDim.x) scales[c] = 0;
        if (a.gates && threadIdx.x < hc) a.gates[t * hc + threadIdx.x] = 0.f;
        return;
    }
    const char* kv = static_cast<const char*>(a.kv) + t * (int64_t)(hc + 1) * d * (kF32Kv ? 4 : 2);
    auto load_kv = [&](int64_t at, float (&f)[8]) {
        if (kF32Kv)
            load8_f32(reinterpret_cast<const float*>(kv) + at, f);
        else
            unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(kv) + at), f);
    };
    auto keep = [&](int64_t at, const float (&f)[8]) {
        uint32_t e;
        const uint2 w = encode_mx8(f, e);
        *reinterpret_cast<uint2*>(codes + at) = w;
        if ((threadIdx.x & 3) == 0) scales[at / 32] = (uint8_t)e;
    };
    for (int b = 0; b < hc; ++b) {
        float s[3] = {};
        for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
            const int64_t at = (int64_t)b * d + c * 8;
            float hf[8], kf[8], w[8];
            unpack8(*reinterpret_cast<const uint4*>(h + at), hf);
            load_kv(at, kf);
            load8_f32(a.wqk + at, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[0] += kf[j] * kf[j];
                s[1] += hf[j] * hf[j];
                s[2] += hf[j] * w[j] * kf[j];
            }
            keep(at, hf);
            keep((int64_t)hc * d + at, kf);
        }
        block_sum<3>(s, sm);
        const float g = gate_from_sums(s[0], s[1], s[2], d, a.eps);
        if (threadIdx.x == 0) {
            gates[b] = g;
            if (a.gates) a.gates[t * hc + b] = g;
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
        float v[8];
        load_kv((int64_t)hc * d + c * 8, v);
        keep((int64_t)2 * hc * d + c * 8, v);
        for (int b = 0; b < hc; ++b) {
            const int64_t at = (int64_t)b * d + c * 8;
            float hf[8];
            unpack8(*reinterpret_cast<const uint4*>(h + at), hf);
#pragma unroll
            for (int j = 0; j < 8; ++j) hf[j] = fmaf(gates[b], v[j], hf[j]);
            *reinterpret_cast<uint4*>(ho + at) = pack8(hf);
        }
    }
}

// The factors of every token and branch: one block per token.
template <int kSaved>
__global__ void __launch_bounds__(320)
k_gate_backward_sums(const GateTrain a) {
    __shared__ float sm[10][4];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    const int hc = a.hc, d = a.d, chunks = d / 8;
    float4* out = a.factors + t * hc;
    if (a.windows[t].x == kDead) {
        if (threadIdx.x < hc) out[threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
        return;
    }
    const Saved<kSaved> sv(a, t);
    for (int b = 0; b < hc; ++b) {
        float s[4] = {};
        for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
            const int64_t at = (int64_t)b * d + c * 8;
            float h[8], k[8], v[8], dy[8], w[8];
            sv.hidden(at, h);
            sv.keyvalue(at, k);
            sv.keyvalue((int64_t)hc * d + c * 8, v);
            unpack8(*reinterpret_cast<const uint4*>(a.dout + t * (int64_t)hc * d + at), dy);
            load8_f32(a.wqk + at, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[0] += k[j] * k[j];
                s[1] += h[j] * h[j];
                s[2] += h[j] * w[j] * k[j];
                s[3] += dy[j] * v[j];
            }
        }
        block_sum<4>(s, sm);
        if (threadIdx.x == 0) out[b] = gate_factors(s[0], s[1], s[2], s[3], d, a.eps);
    }
}

// dh, dk, dv, and this block's share of sum_t dS h k: a thread owns 8 columns
// of every branch and walks its block's tokens, the weights' gradient in
// registers.
template <int kSaved, int kHc>
__global__ void __launch_bounds__(128)
k_gate_backward_columns(const GateTrain a) {
    pdl_wait();
    pdl_launch_dependents();
    const int hc = a.hc, d = a.d;
    const int col = ((int)blockIdx.x * blockDim.x + threadIdx.x) * 8;
    if (col >= d) return;
    float w[kHc][8], acc[kHc][8];
#pragma unroll
    for (int b = 0; b < kHc; ++b) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[b][j] = 0.f;
        if (b < hc) load8_f32(a.wqk + (int64_t)b * d + col, w[b]);
    }
    const int64_t t0 = a.T * blockIdx.y / gridDim.y, t1 = a.T * (blockIdx.y + 1) / gridDim.y;
    for (int64_t t = t0; t < t1; ++t) {
        const uint16_t* dy_t = a.dout + t * (int64_t)hc * d + col;
        uint16_t* dh_t = a.dhidden + t * (int64_t)hc * d + col;
        uint16_t* dkv_t = a.dkv + t * (int64_t)(hc + 1) * d + col;
        const bool image = a.windows[t].x == kDead;
        const Saved<kSaved> sv(a, t);
        float dv[8] = {};
#pragma unroll
        for (int b = 0; b < kHc; ++b) {
            if (b >= hc) continue;
            const int64_t at = (int64_t)b * d;
            const uint4 raw = *reinterpret_cast<const uint4*>(dy_t + at);
            if (image) {
                *reinterpret_cast<uint4*>(dh_t + at) = raw;
                *reinterpret_cast<uint4*>(dkv_t + at) = make_uint4(0u, 0u, 0u, 0u);
                continue;
            }
            float dy[8], h[8], k[8], dh[8], dk[8];
            unpack8(raw, dy);
            sv.hidden(at + col, h);
            sv.keyvalue(at + col, k);
            const float4 f = a.factors[t * hc + b];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float sk = f.x * k[j];
                dh[j] = dy[j] + (sk * w[b][j] - f.y * h[j]);
                dk[j] = f.x * h[j] * w[b][j] - f.z * k[j];
                dv[j] = fmaf(f.w, dy[j], dv[j]);
                acc[b][j] = fmaf(sk, h[j], acc[b][j]);
            }
            *reinterpret_cast<uint4*>(dh_t + at) = pack8(dh);
            *reinterpret_cast<uint4*>(dkv_t + at) = pack8(dk);
        }
        *reinterpret_cast<uint4*>(dkv_t + (int64_t)hc * d) = pack8(dv);
    }
    float* part = a.dw_part + (int64_t)blockIdx.y * hc * d + col;
#pragma unroll
    for (int b = 0; b < kHc; ++b)
        if (b < hc) store8_f32(part + (int64_t)b * d, acc[b]);
}

// dwq = wk sum, dwk = wq sum over the shares: a block takes 128 columns, each of
// its eight warps every eighth share in order, then the warps' sums in order.
__global__ void __launch_bounds__(256)
k_gate_backward_weights(const GateTrain a, int shares) {
    pdl_wait();
    __shared__ float4 sm[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t n = (int64_t)a.hc * a.d, i = (int64_t)blockIdx.x * 128 + lane * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int p = warp; p < shares; p += 8) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(a.dw_part + p * n + i));
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    sm[warp][lane] = s;
    __syncthreads();
    if (warp) return;
    for (int w = 1; w < 8; ++w) {
        const float4 x = sm[w][lane];
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    auto put = [&](float* out, const float* w) {
        if (!out) return;
        const float4 x = *reinterpret_cast<const float4*>(w + i);
        *reinterpret_cast<float4*>(out + i) = make_float4(s.x * x.x, s.y * x.y, s.z * x.z, s.w * x.w);
    };
    put(a.dwq, a.wk);
    put(a.dwk, a.wq);
}

// Cluster size and stages of a one-pass kernel for d columns and a stage of
// bytes(cols) bytes; 0 if no cluster holds two.  The smallest cluster that does:
// at hc 4, d 5,120 two CTAs with two stages of fp32 kv and gradient (and no lag)
// 111 us, four with four stages 144, since half as many warps share an SM's
// work.  Where three stages fit half of an SM's shared memory, they take no more than
// that, so that two CTAs share the SM if the registers allow (hc 1, d 5,120: forward
// with fp32 kv 57 -> 40 us, backward from the checkpoint 54 -> 38; hc 2, d 5,120:
// forward with BF16 kv 61 -> 44; hc 4, d 1,024: with fp32 kv 26 -> 17, from the
// checkpoint 30 -> 24; hc 3, d 3,840 from the checkpoint 71 -> 73): a token of few
// bytes is bound by the latency of its cluster's exchange.  The lag
// is what the stages allow beside one that fills: none of two, one of three, two of
// four or more.
template <class Bytes>
int one_pass_cluster(int d, Bytes bytes, int* stages) {
    const int groups = d / 256;
    for (int cs = 1; cs <= 8 && cs <= groups; cs *= 2) {
        const int per = (groups + cs - 1) / cs;
        const int n = (227 * 1024 - kFusedFixed - 128) / bytes(per * 256);
        if (per <= kFusedMaxWarps && n >= 2) {
            const int half = (113 * 1024 - kFusedFixed - 128) / bytes(per * 256);
            *stages = std::min(half >= 3 ? half : n, 6);
            return cs;
        }
    }
    return 0;
}

template <auto kKernel>
cudaError_t one_pass_launch(const GateTrain& a, int cs, int stages, int stage_bytes, int most, int* clusters,
                            cudaStream_t s) {
    const int per = (a.d / 256 + cs - 1) / cs;
    const int smem = (kFusedFixed + 127) / 128 * 128 + stages * stage_bytes;
    static PerDevice allowed;
    int dev = 0;
    cudaError_t e = allow_shared(allowed, kKernel, 227 * 1024);
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    // as many clusters as are resident at once (larger ones leave SMs of a GPC over),
    // asked for when the shape or the device changes, and no more than `most`
    static thread_local struct { int dev, cs, per, smem, clusters; } known = {};
    cfg.gridDim = dim3(device_sm_count() / cs * cs);
    cfg.blockDim = dim3((per + 2) * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    if (known.dev != dev || known.cs != cs || known.per != per || known.smem != smem) {
        int resident = 1;
        e = cs > 1 ? cudaOccupancyMaxActiveClusters(&resident, kKernel, &cfg)
                   : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&resident, kKernel, (per + 2) * 32, smem);
        if (e != cudaSuccess) return e;
        if (cs == 1) resident *= device_sm_count();
        known = {dev, cs, per, smem, std::max(1, resident)};
    }
    *clusters = (int)std::min<int64_t>(a.T, std::min(known.clusters, most));
    cfg.gridDim = dim3(*clusters * cs);
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kKernel, a, stages, cs, std::min(2, stages - 2));
}

template <int kSaved, int kHc>
cudaError_t fused_launch(const GateTrain& a, int cs, int stages, int* shares, cudaStream_t s) {
    const int bytes = fused_stage_bytes<kSaved>(a.hc, (a.d / 256 + cs - 1) / cs * 256);
    const int most = gate_backward_shares(a.T, a.d);
    return a.hc == kHc
               ? one_pass_launch<k_gate_backward_fused<kSaved, kHc, true>>(a, cs, stages, bytes, most, shares, s)
               : one_pass_launch<k_gate_backward_fused<kSaved, kHc, false>>(a, cs, stages, bytes, most, shares, s);
}

template <bool kF32Kv, int kHc>
cudaError_t ckpt_launch(const GateTrain& a, int cs, int stages, cudaStream_t s) {
    const int bytes = ckpt_stage_bytes<kF32Kv>(a.hc, (a.d / 256 + cs - 1) / cs * 256);
    int clusters;
    return a.hc == kHc
               ? one_pass_launch<k_gate_checkpoint_fused<kF32Kv, kHc, true>>(a, cs, stages, bytes, 1 << 30, &clusters, s)
               : one_pass_launch<k_gate_checkpoint_fused<kF32Kv, kHc, false>>(a, cs, stages, bytes, 1 << 30, &clusters, s);
}

template <bool kF32Kv>
cudaError_t gate_checkpoint(const GateTrain& a, cudaStream_t s) {
    int stages = 0;
    if (const int cs = one_pass_cluster(a.d, [&](int c) { return ckpt_stage_bytes<kF32Kv>(a.hc, c); }, &stages))
        return a.hc == 1   ? ckpt_launch<kF32Kv, 1>(a, cs, stages, s)
               : a.hc == 2 ? ckpt_launch<kF32Kv, 2>(a, cs, stages, s)
               : a.hc <= 4 ? ckpt_launch<kF32Kv, 4>(a, cs, stages, s)
                           : ckpt_launch<kF32Kv, 8>(a, cs, stages, s);
    return pdl_launch(k_gate_checkpoint<kF32Kv>, dim3((unsigned)a.T), dim3(std::min(320, a.d / 8)), 0, s, a);
}

template <int kSaved>
cudaError_t gate_backward(GateTrain a, cudaStream_t s) {
    const dim3 wgrid((unsigned)((int64_t)a.hc * a.d / 128));
    int stages = 0, shares = 0;
    if (const int cs = one_pass_cluster(a.d, [&](int c) { return fused_stage_bytes<kSaved>(a.hc, c); }, &stages)) {
        cudaError_t e = a.hc == 1   ? fused_launch<kSaved, 1>(a, cs, stages, &shares, s)
                        : a.hc == 2 ? fused_launch<kSaved, 2>(a, cs, stages, &shares, s)
                        : a.hc <= 4 ? fused_launch<kSaved, 4>(a, cs, stages, &shares, s)
                                    : fused_launch<kSaved, 8>(a, cs, stages, &shares, s);
        if (e != cudaSuccess || (!a.dwq && !a.dwk)) return e;
        return pdl_launch(k_gate_backward_weights, wgrid, dim3(256), 0, s, a, shares);
    }
    shares = gate_backward_shares(a.T, a.d);
    const int chunks = a.d / 8;
    cudaError_t e = pdl_launch(k_gate_backward_sums<kSaved>, dim3((unsigned)a.T),
                               dim3(std::min(320, chunks)), 0, s, a);
    if (e != cudaSuccess) return e;
    const int threads = std::min(128, chunks);
    const dim3 grid((chunks + threads - 1) / threads, shares);
    auto f = a.hc == 1   ? k_gate_backward_columns<kSaved, 1>
             : a.hc == 2 ? k_gate_backward_columns<kSaved, 2>
             : a.hc <= 4 ? k_gate_backward_columns<kSaved, 4>
                         : k_gate_backward_columns<kSaved, 8>;
    e = pdl_launch(f, grid, dim3(threads), 0, s, a);
    if (e != cudaSuccess || (!a.dwq && !a.dwk)) return e;
    return pdl_launch(k_gate_backward_weights, wgrid, dim3(256), 0, s, a, shares);
}

}  // namespace

cudaError_t launch_gate_checkpoint(const GateTrain& a, bool kv_f32, cudaStream_t s) {
    return kv_f32 ? gate_checkpoint<true>(a, s) : gate_checkpoint<false>(a, s);
}

int gate_backward_shares(int64_t T, int d) {
    const int blocks = (d / 8 + 127) / 128;
    // (the fused kernel launches no more clusters than these)
    return (int)std::max<int64_t>(1, std::min<int64_t>(T, device_sm_count() * std::max(1, 4 / blocks)));
}

cudaError_t launch_gate_backward(const GateTrain& a, int saved, cudaStream_t s) {
    if (saved == kSavedMx) return gate_backward<kSavedMx>(a, s);
    if (saved == kSavedF32) return gate_backward<kSavedF32>(a, s);
    return gate_backward<kSavedBf16>(a, s);
}

}  // namespace engram
