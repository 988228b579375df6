// What uses a step's gradients (sm_103a): their norms, and the AdamW step of many
// tensors at once or of the rows of a table.
//
//   m = b1 m + (1 - b1) f g;  v = b2 v + (1 - b2) (f g)^2
//   p = p (1 - lr wd) - lr / (1 - b1^t)  m / (sqrt(v / (1 - b2^t)) + eps)
//
// All are bound by memory: every value is read once and written once, in 16-byte pieces.
// What is read at a time has to lie together for HBM to reach a copy's rate: blocks take
// short stretches and follow one another in order, instead of staying and drifting apart.
// Measured, against the bytes at a copy's 6.79 TB/s: wkv (157M values) with masters and
// fp32 states 648 us (1.00); wkv and head (820M, BF16) with 8-bit states 1,281 us (0.95);
// 4,915 rows of 5,120 with masters and fp32 states 117 us (0.95); 1.08M rows of 256, MXFP8
// with masters, 8-bit states 726 us (0.96); norms of 1.74 GB of gradients 246 us (1.04).
//
// 8-bit states are MXFP8 blocks of m and of r = sqrt(v).  A step moves r by a part of
// (1 - b2) / 2, 0.05 % at b2 = 0.999, while E4M3's neighbours are 6 to 12 % apart: to
// nearest, r would never move again after the first dozen steps.  Codes are rounded
// stochastically, by 16 random bits a value below the 3 mantissa bits that a code
// keeps; what is expected of a code is then the value, around which it stays by a step or two (a
// root under gradients of one size: a standard deviation of 15 %).  (Below 2^-6 of a code's scale,
// 1 / 28,672 of a block's largest, the cut value is rounded once more, to nearest.)
// A positive r never takes code 0: m / r stays as small as it was.
#include <algorithm>

#include "mx8.cuh"
#include "per_device.h"
#include "philox.cuh"
#include "train_common.cuh"
#include "update_internal.h"

namespace engram {

namespace {

constexpr int kThreads = 256;

// The steps' kernels do not call pdl_launch_dependents: the layer's kernels read wkv and the table
// before they wait for the kernel before them, as nothing but these (and a bind) writes them.

// ---- the element's step -------------------------------------------------------------------

// A step's numbers as an element needs them.
struct Rates {
    float factor, lr, lr_c1, rc2;
    uint32_t step;
};
__device__ __forceinline__ Rates rates_of(const AdamwStep& h) {
    Rates r{1.0f, h.lr, h.lr_c1, h.rc2, h.step};
    if (h.d_factor) r.factor = *h.d_factor;
    if (h.d_lr || h.d_step) {
        if (h.d_step) r.step = *h.d_step;
        const float t = (float)max(r.step, 1u);
        if (h.d_lr) r.lr = *h.d_lr;
        r.lr_c1 = r.lr / -expm1f(t * h.ln_b1);
        r.rc2 = 1.0f / sqrtf(-expm1f(t * h.ln_b2));
    }
    return r;
}

// A step on fp32 states, in place; the root and the quotient are rounded.
__device__ __forceinline__ void step1(const AdamwStep& h, const Rates& q, float keep, float lr, float& p, float g,
                                      float& m, float& v) {
    const float f = g * q.factor;
    m = fmaf(f, h.nb1, m * h.b1);
    v = fmaf(f * f, h.nb2, v * h.b2);
    p = p * keep - lr * (m / fmaf(sqrtf(v), q.rc2, h.eps));
}

// ---- 8-bit states ---------------------------------------------------------------------------

// A thread holds 16 values, half a block of 32, in pairs: 10 bytes a value leave 54 of an
// SM's issue slots for it, of which a thread's 8 values one by one took 87; two values an
// instruction, and 16 to share what a block costs, take 42, and the slots are two thirds busy.

// 1 / sqrt(v) and 1 / v, off by up to 2^-22 and 2^-23 of themselves.
__device__ __forceinline__ float inverse_root(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float inverse(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// Roots of values that are not negative (of those below 2^-126 less than the root), by a step of
// Newton's from s = v y, y about 1 / sqrt(v): s + (v - s^2) y / 2, whose remainder an fma gives
// exactly (Markstein, IBM J. Res. Dev. 34, 1990).  What is then rounded is off by 2^-43 of the root:
// it is the nearest fp32 number but for one value in some 10^5.  Codes and scales are made of it: of
// 276M values one code differs from those of rounded roots; with an approximate root 122 and
// two blocks' scales did.  820M BF16 values take 1,283 us (the approximate root 1,237, sqrtf 1,403),
// 61M 106 (102, 117); rows and tensors with masters what they took.
__device__ __forceinline__ f32x2 root2(f32x2 v) {
    const float2 a = unpair(v);
    const f32x2 y = pair(inverse_root(fmaxf(a.x, 0x1p-126f)), inverse_root(fmaxf(a.y, 0x1p-126f)));
    const float2 s = unpair(mul2(v, y));
    return fma2(pair(fmaf(-s.x, s.x, a.x), fmaf(-s.y, s.y, a.y)), mul2(y, twice(0.5f)), pair(s.x, s.y));
}
__device__ __forceinline__ float low3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float top16(const f32x2 (&f)[8]) {
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t = top3(t, unpair(f[j]).x, unpair(f[j]).y);
    return t;
}

// The four pairs of 8 codes, unscaled.
__device__ __forceinline__ void codes8(uint32_t lo, uint32_t hi, f32x2* f) {
    const uint32_t w[2] = {lo, hi};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t x, y;
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(x), "=r"(y)
            : "r"(w[j]));
        const float2 u = __half22float2(*reinterpret_cast<__half2*>(&x));
        const float2 v = __half22float2(*reinterpret_cast<__half2*>(&y));
        f[2 * j] = pair(u.x, u.y);
        f[2 * j + 1] = pair(v.x, v.y);
    }
}

// To nearest, as encode_mx8.
__device__ __forceinline__ uint4 encode16(const f32x2 (&f)[8], uint32_t& exponent) {
    exponent = mx8_exponent<2>(top16(f));
    const f32x2 inv = twice(mx8_inverse(exponent));
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 a = unpair(mul2(f[2 * j], inv)), b = unpair(mul2(f[2 * j + 1], inv));
        w[j] = code4(a.x, a.y, b.x, b.y);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Stochastically: 16 random bits a value (noise[j]: the values 2 j and 2 j + 1) are added
// below the 3 mantissa bits that a code keeps, and what is below is cut.
template <bool kPositive>
__device__ __forceinline__ uint4 encode_random(const f32x2 (&f)[8], const uint32_t (&noise)[8], uint32_t& exponent) {
    exponent = mx8_exponent<2>(top16(f));
    const float inv = mx8_inverse(exponent);
    float y[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float2 x = unpair(mul2(f[j], twice(inv)));
        y[2 * j] = __uint_as_float((__float_as_uint(x.x) + ((noise[j] & 0xFFFFu) << 4)) & 0xFFF00000u);
        y[2 * j + 1] = __uint_as_float((__float_as_uint(x.y) + (noise[j] >> 16 << 4)) & 0xFFF00000u);
    }
    if (kPositive) {
        float least = INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) least = low3(least, y[2 * j], y[2 * j + 1]);
        if (least < 0x1p-9f) {  // (a value far below its block's largest)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 x = unpair(f[j]);
                y[2 * j] = x.x > 0.f ? fmaxf(y[2 * j], 0x1p-9f) : y[2 * j];
                y[2 * j + 1] = x.y > 0.f ? fmaxf(y[2 * j + 1], 0x1p-9f) : y[2 * j + 1];
            }
        }
    }
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = code4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Philox4x32-10 with the round keys that the host has made; its words go to noise[0..3].
__device__ __forceinline__ void noise8(const AdamwStep& h, uint64_t place8, uint32_t tensor, uint32_t step,
                                       uint32_t* noise) {
    uint32_t x = (uint32_t)place8, y = (uint32_t)(place8 >> 32), z = tensor, w = step;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p = (uint64_t)kPhiloxM0 * x, q = (uint64_t)kPhiloxM1 * z;
        x = (uint32_t)(q >> 32) ^ y ^ h.key[2 * r];
        z = (uint32_t)(p >> 32) ^ w ^ h.key[2 * r + 1];
        y = (uint32_t)q;
        w = (uint32_t)p;
    }
    noise[0] = x, noise[1] = y, noise[2] = z, noise[3] = w;
}

// A step of 16 values; the states' codes and exponents in place.  take(half, p, g) gives the
// parameters and gradients of 8 of them, give(half, p) gets the new parameters: no more
// than 8 are held at a time.  Gradients and roots take their factor and scale before they are
// squared: the squares of a small factor or scale alone leave fp32's range long before v does.
template <class Take, class Give>
__device__ __forceinline__ void step16(const AdamwStep& h, const Rates& q, float kept, float rate, uint64_t place,
                                       uint32_t tensor, uint4& mc, uint4& vc, uint32_t& me, uint32_t& ve, Take take,
                                       Give give) {
    f32x2 m[8], r[8];
    {
        const f32x2 sm = twice(e8m0_to_f32(me) * h.b1), sv = twice(e8m0_to_f32(ve));
        const f32x2 factor = twice(q.factor), nb1 = twice(h.nb1), b2 = twice(h.b2), nb2 = twice(h.nb2);
        const f32x2 rc2 = twice(q.rc2), eps = twice(h.eps);
        const f32x2 keep = twice(kept), lr = twice(-rate);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            f32x2 p[4], g[4];
            take(half, p, g);
            codes8(half ? mc.z : mc.x, half ? mc.w : mc.y, m + 4 * half);
            codes8(half ? vc.z : vc.x, half ? vc.w : vc.y, r + 4 * half);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 4 * half + i;
                const f32x2 f = mul2(g[i], factor);
                r[j] = mul2(r[j], sv);
                m[j] = fma2(f, nb1, mul2(m[j], sm));
                r[j] = root2(fma2(mul2(f, f), nb2, mul2(mul2(r[j], r[j]), b2)));
                // (a quotient off by 2^-22 of a step that is a small part of p: one more mended by
                // Newton's step changes 25 of 820M BF16 parameters and takes 4 %)
                const float2 den = unpair(fma2(r[j], rc2, eps));
                p[i] = fma2(p[i], keep, mul2(mul2(m[j], pair(inverse(den.x), inverse(den.y))), lr));
            }
            give(half, p);
        }
    }
    uint32_t noise[8];
    noise8(h, place / 8, tensor, q.step, noise);
    noise8(h, place / 8 + 1, tensor, q.step, noise + 4);
    mc = encode_random<false>(m, noise, me);
    vc = encode_random<true>(r, noise, ve);
}

// ---- loads and stores of up to 8 values of a tensor's end ------------------------------------

__device__ __forceinline__ void load8(const void* p, bool f32, size_t at, int count, float (&f)[8]) {
    if (count >= 8) {  // (0 or less: zeros)
        if (f32)
            load8_f32(static_cast<const float*>(p) + at, f);
        else
            unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at), f);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = j >= count ? 0.f
               : f32      ? static_cast<const float*>(p)[at + j]
                          : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[at + j] << 16);
}
__device__ __forceinline__ void store8(void* p, bool f32, size_t at, int count, const float (&f)[8]) {
    if (count >= 8) {
        if (f32)
            store8_f32(static_cast<float*>(p) + at, f);
        else
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = pack8(f);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < count) {
            if (f32)
                static_cast<float*>(p)[at + j] = f[j];
            else
                static_cast<uint16_t*>(p)[at + j] = (uint16_t)bf16x2_pack_rn(f[j], 0.f);
        }
}
__device__ __forceinline__ void load8(const void* p, bool f32, size_t at, int count, f32x2 (&f)[4]) {
    float e[8];
    load8(p, f32, at, count, e);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = pair(e[2 * j], e[2 * j + 1]);
}
__device__ __forceinline__ void store8(void* p, bool f32, size_t at, int count, const f32x2 (&f)[4]) {
    float e[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[2 * j] = unpair(f[j]).x, e[2 * j + 1] = unpair(f[j]).y;
    store8(p, f32, at, count, e);
}
__device__ __forceinline__ uint4 load_codes(const void* p, size_t at, int count) {
    const uint8_t* c = static_cast<const uint8_t*>(p) + at;
    if (count == 16) return *reinterpret_cast<const uint4*>(c);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 15; ++j)
        if (j < count) w[j >> 2] |= (uint32_t)c[j] << (8 * (j & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_codes(void* p, size_t at, int count, uint4 codes) {
    uint8_t* c = static_cast<uint8_t*>(p) + at;
    if (count == 16) {
        *reinterpret_cast<uint4*>(c) = codes;
        return;
    }
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int j = 0; j < 15; ++j)
        if (j < count) c[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
}

// ---- AdamW over a list of tensors -------------------------------------------------------------

// The last of `count` ascending beginnings that is at or before `at`.  (They lie together in
// the parameters: a search among the tensors' own data misses the constant cache at every
// step.)
__device__ __forceinline__ int last_before(const uint32_t* first, int count, uint64_t at) {
    int lo = 0, hi = count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first[mid] <= at)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// One block per chunk of kThreads x 8 x iters values of one tensor, fp32 states.
template <int kN>
__global__ void __launch_bounds__(kThreads)
    k_adamw(const __grid_constant__ AdamwStep h, const __grid_constant__ AdamwTensors<kN> list, int count,
            int iters) {
    const int k = last_before(list.first, count, blockIdx.x);
    const AdamwTensor& t = list.t[k];
    const uint64_t n = t.n;
    const bool pf32 = t.kind & kParamF32, gf32 = t.kind & kGradF32, master = t.kind & kMaster;
    pdl_wait();
    const Rates q = rates_of(h);
    const float keep = 1.0f - q.lr * t.lr_scale * t.decay, lr = q.lr_c1 * t.lr_scale;
    size_t base = (size_t)(blockIdx.x - list.first[k]) * iters * (kThreads * 8);
    for (int it = 0; it < iters && base < n; ++it, base += kThreads * 8) {
        const size_t at = base + threadIdx.x * 8;
        const int have = at < n ? (int)min((uint64_t)8, n - at) : 0;
        float p[8], g[8], m[8], v[8];
        load8(t.grad, gf32, at, have, g);
        load8(master ? t.master : t.param, pf32 || master, at, have, p);
        load8(t.m, true, at, have, m);
        load8(t.v, true, at, have, v);
        if (q.factor != q.factor) return;  // the gradients are not finite: no step
#pragma unroll
        for (int j = 0; j < 8; ++j) step1(h, q, keep, lr, p[j], g[j], m[j], v[j]);
        if (!have) continue;
        if (master) store8(t.master, true, at, have, p);
        store8(t.param, pf32, at, have, p);
        store8(t.m, true, at, have, m);
        store8(t.v, true, at, have, v);
    }
}

// 8-bit states.  A block takes some neighbouring cells of kMxThreads x 16 values, tensor by
// tensor: within one nothing is asked again and addresses only grow, and while a block works
// on a cell the next one's values are on their way to shared memory.
// 61M values, with an approximate root: 256 threads, two blocks of an SM and two stages 100 us; 128
// threads and four blocks 105; three blocks (fewer registers, spills) 112; three stages 102.
constexpr int kMxThreads = 256;
constexpr int kStages = 2;
constexpr int kCell = kMxThreads * 16;

// The 512 values of a warp, fp32 or BF16, in 16-byte pieces: a lane owns 4 or 2 neighbouring
// ones, but copies every 32nd, so that an instruction covers whole sectors (pieces at a
// lane's own places would take half of each, twice).  Pieces are swapped within 128 bytes so
// that neither the copies nor the lanes' reads meet in a bank.
template <bool kF32>
struct WarpValues {
    static constexpr int kPieces = kF32 ? 4 : 2, kBytes = kF32 ? 4 : 2;
    __device__ static __forceinline__ int at(int piece) { return piece ^ (piece >> 3 & (kF32 ? 3 : 1)); }
    // p: the warp's first value plus 16 bytes a lane
    __device__ static __forceinline__ void send(uint4* s, const char* p, int lane) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) async16(s + at(32 * j + lane), p + 512 * j);
    }
    __device__ static __forceinline__ void store(const uint4* s, char* p, int lane) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) __stcs(reinterpret_cast<uint4*>(p + 512 * j), s[at(32 * j + lane)]);
    }
    // 8 of a lane's 16 values
    __device__ static __forceinline__ void take(const uint4* s, int lane, int half, f32x2 (&f)[4]) {
        if (kF32) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(s + at(4 * lane + 2 * half + j));
                f[2 * j] = v.x;
                f[2 * j + 1] = v.y;
            }
        } else {
            unpack8(s[at(2 * lane + half)], f);
        }
    }
    __device__ static __forceinline__ void give(uint4* s, int lane, int half, const f32x2 (&f)[4]) {
        if (kF32) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<ulonglong2*>(s + at(4 * lane + 2 * half + j)) = make_ulonglong2(f[2 * j], f[2 * j + 1]);
        } else {
            s[at(2 * lane + half)] = pack8(f);
        }
    }
};

// 16-byte pieces that a thread has in a stage.
__host__ __device__ constexpr int pieces_of(bool p32, bool g32) { return (p32 ? 4 : 2) + (g32 ? 4 : 2) + 2; }

// Whole cells [first, first + cells) of a tensor, by all of the block.
template <bool kParam32, bool kGrad32, bool kMasters>
__device__ __forceinline__ void whole_cells(const AdamwStep& h, const Rates& q, const AdamwTensor& t, uint64_t first,
                                            uint32_t cells, uint4* stages) {
    constexpr bool kP = kParam32 || kMasters;
    using P = WarpValues<kP>;
    using G = WarpValues<kGrad32>;
    constexpr int kPieces = pieces_of(kP, kGrad32), kG = P::kPieces * 32, kM = kG + G::kPieces * 32, kV = kM + 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t from = first * kCell + warp * 512;  // the warp's first value
    uint64_t at = from + lane * 16;
    char* p = static_cast<char*>(kMasters ? (void*)t.master : t.param) + from * P::kBytes + lane * 16;
    char* copy = static_cast<char*>(t.param) + from * 2 + lane * 16;  // kMasters
    const char* g = static_cast<const char*>(t.grad) + from * G::kBytes + lane * 16;
    char *m = static_cast<char*>(t.m) + at, *v = static_cast<char*>(t.v) + at;
    uint8_t *ms = t.m_scales + at / 32, *vs = t.v_scales + at / 32;
    stages += warp * kPieces * 32;
    constexpr int kStage = kPieces * kMxThreads;
    uint32_t scales[kStages - 1][2];  // of the cells on their way, the next one first
    auto fetch = [&](int ahead, uint4* s, uint32_t(&e)[2]) {  // the cell `ahead` cells on
        e[0] = ms[ahead * (kCell / 32)];
        e[1] = vs[ahead * (kCell / 32)];
        P::send(s, p + ahead * kCell * P::kBytes, lane);
        G::send(s + kG, g + ahead * kCell * G::kBytes, lane);
        async16(s + kM + lane, m + ahead * kCell);
        async16(s + kV + lane, v + ahead * kCell);
    };
    __syncthreads();  // the tensor before may be of another kind, whose warps have other places
#pragma unroll
    for (int ahead = 0; ahead < kStages - 1; ++ahead) {
        if (ahead < cells) fetch(ahead, stages + ahead * kStage, scales[ahead]);
        async_commit();
    }
    const float keep = 1.0f - q.lr * t.lr_scale * t.decay, lr = q.lr_c1 * t.lr_scale;
    const uint32_t ordinal = t.ordinal;
    int stage = 0, free = kStages - 1;
    for (uint32_t left = cells; left > 0; --left) {
        uint32_t me = scales[0][0], ve = scales[0][1];
#pragma unroll
        for (int j = 1; j < kStages - 1; ++j) scales[j - 1][0] = scales[j][0], scales[j - 1][1] = scales[j][1];
        uint4* s = stages + stage * kStage;
        if (left > kStages - 1) fetch(kStages - 1, stages + free * kStage, scales[kStages - 2]);
        stage = stage + 1 == kStages ? 0 : stage + 1;
        free = free + 1 == kStages ? 0 : free + 1;
        async_commit();
        async_wait<kStages - 1>();
        __syncwarp();
        uint4 mc = s[kM + lane], vc = s[kV + lane];
        if (kMasters) __syncwarp();  // the codes' places get the parameters' copy
        step16(
            h, q, keep, lr, at, ordinal, mc, vc, me, ve,
            [&](int half, f32x2(&pp)[4], f32x2(&gg)[4]) {
                P::take(s, lane, half, pp);
                G::take(s + kG, lane, half, gg);
            },
            [&](int half, const f32x2(&pp)[4]) {  // over what it has just taken
                P::give(s, lane, half, pp);
                if (kMasters) WarpValues<false>::give(s + kM, lane, half, pp);
            });
        __syncwarp();
        P::store(s, p, lane);
        if (kMasters) WarpValues<false>::store(s + kM, copy, lane);
        __stcs(reinterpret_cast<uint4*>(m), mc);
        __stcs(reinterpret_cast<uint4*>(v), vc);
        if (!(lane & 1)) {
            *ms = (uint8_t)me;
            *vs = (uint8_t)ve;
        }
        __syncwarp();  // read back before the stage is sent for again
        at += kCell;
        p += kCell * P::kBytes;
        if (kMasters) copy += kCell * 2;
        g += kCell * G::kBytes;
        m += kCell;
        v += kCell;
        ms += kCell / 32;
        vs += kCell / 32;
    }
}

// A tensor's last values, less than a cell.
__device__ __noinline__ void last_cell(const AdamwStep& h, const Rates& q, const AdamwTensor& t) {
    const uint64_t at = t.n / kCell * kCell + threadIdx.x * 16;
    const bool pf32 = t.kind & kParamF32, gf32 = t.kind & kGradF32, master = t.kind & kMaster;
    const int have = at < t.n ? (int)min((uint64_t)16, t.n - at) : 0;
    uint4 mc = load_codes(t.m, at, have), vc = load_codes(t.v, at, have);
    uint32_t me = have ? t.m_scales[at / 32] : 0u, ve = have ? t.v_scales[at / 32] : 0u;
    step16(
        h, q, 1.0f - q.lr * t.lr_scale * t.decay, q.lr_c1 * t.lr_scale, at, t.ordinal, mc, vc, me, ve,
        [&](int half, f32x2(&p)[4], f32x2(&g)[4]) {
            load8(master ? t.master : t.param, pf32 || master, at + 8 * half, have - 8 * half, p);
            load8(t.grad, gf32, at + 8 * half, have - 8 * half, g);
        },
        [&](int half, const f32x2(&p)[4]) {
            if (master) store8(t.master, true, at + 8 * half, have - 8 * half, p);
            store8(t.param, pf32, at + 8 * half, have - 8 * half, p);
        });
    store_codes(t.m, at, have, mc);
    store_codes(t.v, at, have, vc);
    if (have && !(threadIdx.x & 1)) {
        t.m_scales[at / 32] = (uint8_t)me;
        t.v_scales[at / 32] = (uint8_t)ve;
    }
}

// 820M values, with an approximate root: 8 cells a block 1,219 us, 4 (their beginnings show) 1,303;
// 61M: 100, 4 104, 16 (an uneven last wave) 107, blocks that stay 104.
constexpr unsigned kCellsPerBlock = 8;
constexpr int kMxBlocks = 2;  // of an SM, at 128 registers a thread

template <int kN>
__global__ void __launch_bounds__(kMxThreads, kMxBlocks)
    k_adamw_mx(const __grid_constant__ AdamwStep h, const __grid_constant__ AdamwTensors<kN> list, int count,
               uint32_t cells, uint32_t per_block) {
    extern __shared__ uint4 stages[];
    pdl_wait();
    const Rates q = rates_of(h);
    if (q.factor != q.factor) return;  // the gradients are not finite: no step
    const uint64_t end = min((uint64_t)cells, (uint64_t)(blockIdx.x + 1) * per_block);
    for (uint64_t c = (uint64_t)blockIdx.x * per_block; c < end;) {
        const int k = last_before(list.first, count, c);
        const AdamwTensor& t = list.t[k];
        const uint64_t first = c - list.first[k], whole = t.n / kCell;
        if (first < whole) {
            const uint32_t mine = (uint32_t)min(end - c, whole - first);
            switch (t.kind) {
                case 0: whole_cells<false, false, false>(h, q, t, first, mine, stages); break;
                case kGradF32: whole_cells<false, true, false>(h, q, t, first, mine, stages); break;
                case kParamF32: whole_cells<true, false, false>(h, q, t, first, mine, stages); break;
                case kParamF32 | kGradF32: whole_cells<true, true, false>(h, q, t, first, mine, stages); break;
                case kMaster: whole_cells<false, false, true>(h, q, t, first, mine, stages); break;
                case kMaster | kGradF32: whole_cells<false, true, true>(h, q, t, first, mine, stages); break;
            }
            c += mine;
        } else {
            last_cell(h, q, t);
            ++c;
        }
    }
}

// ---- AdamW on rows ----------------------------------------------------------------------------

// Whether row i of the list names a row of the table: ids ascend.
__device__ __forceinline__ bool goes(const AdamwRows& a, uint64_t i, uint32_t id, uint32_t before) {
    return id < a.rows && (i == 0 || before < id);
}

// fp32 states.  A thread takes 4 columns of a row: 16 bytes of everything but a 16- or 8-bit
// table; the id of its next row is on its way while it works on one.
template <bool kTableMx>
__global__ void __launch_bounds__(kThreads)
    k_adamw_rows(const __grid_constant__ AdamwStep h, const __grid_constant__ AdamwRows a) {
    const uint32_t V = a.dim / 4;
    const bool pf32 = a.kind & kParamF32, master = a.kind & kMaster;
    float* const param = master ? a.master : static_cast<float*>(a.table);
    pdl_wait();
    const Rates q = rates_of(h);
    if (q.factor != q.factor) return;
    const float keep = 1.0f - q.lr * a.lr_scale * a.decay, lr = q.lr_c1 * a.lr_scale;
    const uint64_t rows = min((uint64_t)*a.count, (uint64_t)a.n), total = rows * V;
    const uint64_t threads = (uint64_t)gridDim.x * kThreads, step_i = threads / V;
    const uint32_t step_c = (uint32_t)(threads - step_i * V);
    uint64_t base = (uint64_t)blockIdx.x * kThreads, item = base + threadIdx.x, i = item / V;
    uint32_t c = (uint32_t)(item - i * V), id = 0, before = 0;
    auto look = [&] {
        if (i < rows) {
            id = a.ids[i];
            before = i ? a.ids[i - 1] : 0;
        }
    };
    look();
    for (; base < total; base += threads) {
        bool ok = i < rows;
        const size_t from = (size_t)i * a.dim + c * 4, at = (size_t)id * a.dim + c * 4;
        if (ok && !goes(a, i, id, before)) {
            ok = false;
            if (c == 0) atomicOr(a.err, kErrBounds);
        }
        const uint32_t col = c;
        i += step_i;
        c += step_c;
        if (c >= V) c -= V, ++i;
        look();
        float4 p{}, g{}, m{}, v{};
        if (ok) {
            g = *reinterpret_cast<const float4*>(a.grad + from);
            m = *reinterpret_cast<const float4*>(static_cast<const float*>(a.m) + at);
            v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.v) + at);
            if (master || pf32) {
                p = *reinterpret_cast<const float4*>(param + at);
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.table) + at);
                p = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
            }
        }
        step1(h, q, keep, lr, p.x, g.x, m.x, v.x);
        step1(h, q, keep, lr, p.y, g.y, m.y, v.y);
        step1(h, q, keep, lr, p.z, g.z, m.z, v.z);
        step1(h, q, keep, lr, p.w, g.w, m.w, v.w);
        uint32_t e = 0, codes = 0;
        if (kTableMx) {  // a block is in 8 lanes
            e = mx8_exponent<8>(top3(top3(p.x, p.y, p.z), p.w, p.w));
            const float inv = mx8_inverse(e);
            codes = code4(p.x * inv, p.y * inv, p.z * inv, p.w * inv);
        }
        if (!ok) continue;
        if (master || pf32) *reinterpret_cast<float4*>(param + at) = p;
        if (kTableMx) {
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.table) + at) = codes;
            if (!(col & 7)) a.scales[at / 32] = (uint8_t)e;
        } else if (!pf32) {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.table) + at) =
                make_uint2(bf16x2_pack_rn(p.x, p.y), bf16x2_pack_rn(p.z, p.w));
        }
        *reinterpret_cast<float4*>(static_cast<float*>(a.m) + at) = m;
        *reinterpret_cast<float4*>(static_cast<float*>(a.v) + at) = v;
    }
}

// 8-bit states.  A warp takes 512 values at a time, of one row or of several; its next ones
// are on their way to shared memory while it works (as in whole_cells: a lane owns 16
// neighbouring values and copies every 32nd piece), and the ids of those after are on theirs.
template <bool kParam32, bool kMasters, bool kTableMx>
__global__ void __launch_bounds__(kMxThreads, kMxBlocks)
    k_adamw_rows_mx(const __grid_constant__ AdamwStep h, const __grid_constant__ AdamwRows a) {
    extern __shared__ uint4 stages[];
    constexpr bool kP = kParam32 || kMasters;
    using P = WarpValues<kP>;
    using G = WarpValues<true>;
    constexpr int kPieces = pieces_of(kP, true), kG = P::kPieces * 32, kM = kG + G::kPieces * 32, kV = kM + 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t V = a.dim / 16;
    char* const param = static_cast<char*>(kMasters ? (void*)a.master : a.table);
    pdl_wait();
    const Rates q = rates_of(h);
    if (q.factor != q.factor) return;
    const uint64_t rows = min((uint64_t)*a.count, (uint64_t)a.n), total = rows * V;
    // this lane's 16 columns: piece c of row i of the list; step: from one of its rows to the next
    const uint64_t threads = (uint64_t)gridDim.x * kMxThreads, step_i = threads / V;
    const uint32_t step_c = (uint32_t)(threads - step_i * V);
    uint64_t item = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x, i = item / V;
    uint32_t c = (uint32_t)(item - i * V);
    uint64_t base = item - lane;  // the warp's first
    if (base >= total) return;
    uint4* ring = stages + warp * kPieces * 32;
    constexpr int kStage = kPieces * kMxThreads;
    constexpr uint64_t kNone = ~0ull;

    uint32_t id = 0, before = 0;  // of the values after the next ones
    auto look = [&] {
        if (i < rows) {
            id = a.ids[i];
            before = i ? a.ids[i - 1] : 0;
        }
    };
    auto hop = [&] {
        i += step_i;
        c += step_c;
        if (c >= V) c -= V, ++i;
    };
    uint64_t at_next = kNone;
    uint32_t me_next = 0, ve_next = 0;
    // sends for the values whose ids are there; from: the warp's first value in the list
    auto fetch = [&](uint64_t from, uint4* s) {
        at_next = kNone;
        if (i < rows) {
            if (goes(a, i, id, before))
                at_next = (uint64_t)id * a.dim + c * 16;
            else if (c == 0)
                atomicOr(a.err, kErrBounds);
        }
        if (at_next != kNone) {
            me_next = a.m_scales[at_next / 32];
            ve_next = a.v_scales[at_next / 32];
            async16(s + kM + lane, static_cast<const uint8_t*>(a.m) + at_next);
            async16(s + kV + lane, static_cast<const uint8_t*>(a.v) + at_next);
        }
#pragma unroll
        for (int j = 0; j < P::kPieces; ++j) {
            const int piece = 32 * j + lane;
            const uint64_t o = __shfl_sync(0xFFFFFFFFu, at_next, piece / P::kPieces);
            if (o != kNone) async16(s + P::at(piece), param + o * P::kBytes + piece % P::kPieces * 16);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int piece = 32 * j + lane;
            if (from + piece / 4 < total)
                async16(s + kG + G::at(piece), reinterpret_cast<const char*>(a.grad) + from * 64 + piece * 16);
        }
    };
    look();
    fetch(base, ring);
    async_commit();
    hop();
    look();
    for (int stage = 0; base < total; base += threads, stage ^= 1) {
        const uint64_t at = at_next;
        uint32_t me = me_next, ve = ve_next;
        uint4* s = ring + stage * kStage;
        if (base + threads < total) {
            fetch(base + threads, ring + (stage ^ 1) * kStage);
            hop();
            look();
        }
        async_commit();
        async_wait<1>();
        __syncwarp();
        uint4 mc = s[kM + lane], vc = s[kV + lane];
        if (kMasters && !kTableMx) __syncwarp();  // the codes' places get the parameters' copy
        f32x2 all[8];
        step16(
            h, q, 1.0f - q.lr * a.lr_scale * a.decay, q.lr_c1 * a.lr_scale, at, 0, mc, vc, me, ve,
            [&](int half, f32x2(&p)[4], f32x2(&g)[4]) {
                P::take(s, lane, half, p);
                G::take(s + kG, lane, half, g);
            },
            [&](int half, const f32x2(&p)[4]) {
                P::give(s, lane, half, p);
                if (kMasters && !kTableMx) WarpValues<false>::give(s + kM, lane, half, p);
                if (kTableMx)
#pragma unroll
                    for (int j = 0; j < 4; ++j) all[4 * half + j] = p[j];
            });
        uint4 pc;
        uint32_t pe = 0;
        if (kTableMx) pc = encode16(all, pe);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < P::kPieces; ++j) {
            const int piece = 32 * j + lane;
            const uint64_t o = __shfl_sync(0xFFFFFFFFu, at, piece / P::kPieces);
            if (o != kNone)
                __stcs(reinterpret_cast<uint4*>(param + o * P::kBytes + piece % P::kPieces * 16), s[P::at(piece)]);
        }
        if (kMasters && !kTableMx) {
            using C = WarpValues<false>;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int piece = 32 * j + lane;
                const uint64_t o = __shfl_sync(0xFFFFFFFFu, at, piece / 2);
                if (o != kNone)
                    *reinterpret_cast<uint4*>(static_cast<char*>(a.table) + o * 2 + piece % 2 * 16) = s[kM + C::at(piece)];
            }
        }
        if (at != kNone) {
            if (kTableMx) __stcs(reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.table) + at), pc);
            __stcs(reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.m) + at), mc);
            __stcs(reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.v) + at), vc);
            if (!(at & 31)) {
                if (kTableMx) a.scales[at / 32] = (uint8_t)pe;
                a.m_scales[at / 32] = (uint8_t)me;
                a.v_scales[at / 32] = (uint8_t)ve;
            }
        }
        __syncwarp();  // read back before the stage is sent for again
    }
}

// ---- gradient norm ------------------------------------------------------------------------------

constexpr int kNormLoads = 8;                      // 16-byte loads that a thread has on their way
constexpr int kNormUnit = kThreads * 8 * kNormLoads;  // values that a block takes at a time

// The squares of this thread's part of a unit that begins at value `base` of n; 64 values in
// 8 running sums.
template <bool kF32>
__device__ __forceinline__ float unit_squares(const void* p, uint64_t base, uint64_t n) {
    constexpr int kPer = kF32 ? 4 : 8;  // values of a load
    f32x2 s[4] = {0, 0, 0, 0};
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + base * (kF32 ? 4 : 2)) + threadIdx.x;
    const bool whole = base + kNormUnit <= n;
    const int64_t vectors = (int64_t)((n - base) / kPer) - threadIdx.x;  // of the tensor, from this thread's first on
#pragma unroll
    for (int half = 0; half < kNormUnit / (kThreads * kPer * kNormLoads); ++half) {
        uint4 v[kNormLoads];
        if (whole) {
#pragma unroll
            for (int k = 0; k < kNormLoads; ++k) v[k] = __ldcs(q + (half * kNormLoads + k) * kThreads);
        } else {
#pragma unroll
            for (int k = 0; k < kNormLoads; ++k) {
                const int at = (half * kNormLoads + k) * kThreads;
                v[k] = at < vectors ? __ldcs(q + at) : make_uint4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int k = 0; k < kNormLoads; ++k) {
            if (kF32) {
                const f32x2 a = pair(__uint_as_float(v[k].x), __uint_as_float(v[k].y));
                const f32x2 b = pair(__uint_as_float(v[k].z), __uint_as_float(v[k].w));
                s[2 * (k & 1)] = fma2(a, a, s[2 * (k & 1)]);
                s[2 * (k & 1) + 1] = fma2(b, b, s[2 * (k & 1) + 1]);
            } else {
                f32x2 f[4];
                unpack8(v[k], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] = fma2(f[j], f[j], s[j]);
            }
        }
    }
    float sum = both(add2(add2(s[0], s[1]), add2(s[2], s[3])));
    if (!whole && threadIdx.x < n % kPer) {  // what fills no vector
        const uint64_t at = n / kPer * kPer + threadIdx.x;
        const float g = kF32 ? static_cast<const float*>(p)[at]
                             : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[at] << 16);
        sum = fmaf(g, g, sum);
    }
    return sum;
}

// A block takes every gridDim.x-th unit of all parts, in order, so that the units that are
// read at a time are neighbours (614 MB 98 us; a stretch for each block 109).  Units are
// counted as if every part had all its rows; those past a part's count are left out, which
// costs every block the same.  Its sum of a part goes to part[slot of the part + index of its
// first unit there]; range[part]: where its sums begin and end, and its place in the
// caller's list.
template <int kN>
__global__ void __launch_bounds__(kThreads)
    k_grad_squares(const __grid_constant__ GradParts<kN> list, int count, uint32_t units, double* part, uint4* range) {
    __shared__ double warp_sum[kThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    for (uint64_t u = blockIdx.x; u < units;) {
        const int lo = last_before(list.first, count, u);
        const GradPart& p = list.p[lo];
        const uint64_t n = (p.count ? min((uint64_t)*p.count, p.n) : p.n) * p.dim;
        const uint64_t have = (n + kNormUnit - 1) / kNormUnit, first = u - list.first[lo];
        if (first == 0 && threadIdx.x == 0)
            range[lo] = make_uint4(p.slot, p.slot + (uint32_t)min(have, (uint64_t)gridDim.x), p.index, 0);
        if (first < have) {
            double sum = 0.0;
            for (uint64_t i = first; i < have; i += gridDim.x)
                sum += p.f32 ? unit_squares<true>(p.grad, i * kNormUnit, n) : unit_squares<false>(p.grad, i * kNormUnit, n);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = sum;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int w = 1; w < kThreads / 32; ++w) sum += warp_sum[w];
                part[p.slot + first] = sum;
            }
        }
        const uint32_t next = lo + 1 < count ? list.first[lo + 1] : units;
        u += (next - u + gridDim.x - 1) / gridDim.x * gridDim.x;
    }
}

// The root of a sum of squares: in fp32 (64-bit roots are slow), scaled into its range; an
// fp32 square is not below 2^-149 nor are 2^60 of them above 2^188.
__device__ __forceinline__ float root_of(double s) {
    return s > 1.0 ? sqrtf((float)(s * 0x1p-64)) * 0x1p32f : sqrtf((float)(s * 0x1p64)) * 0x1p-32f;
}

__global__ void __launch_bounds__(1024) k_grad_norm(const GradNormArgs a) {
    __shared__ double sm[64];
    pdl_launch_dependents();
    const int group = threadIdx.x >> 4, lane = threadIdx.x & 15;  // half a warp sums a part
    pdl_wait();
    double all = 0.0;
    for (int base = 0; base < a.count; base += 64) {
        const int k = base + group;
        double s = 0.0;
        uint4 b = make_uint4(0, 0, 0, 0);
        if (k < a.count) {
            b = a.range[k];
#pragma unroll 4
            for (uint32_t i = b.x + lane; i < b.y; i += 16) s += a.part[i];
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0 && k < a.count && a.each) a.each[b.z] = root_of(s);
        all += s;
    }
    if (lane == 0) sm[group] = all;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    all = sm[threadIdx.x] + sm[threadIdx.x + 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    if (threadIdx.x == 0) {
        const float norm = root_of(all);
        if (a.norm) *a.norm = norm;
        if (a.factor)
            *a.factor = !(norm <= 3.402823466e+38f) ? __uint_as_float(0x7FC00000u)
                        : norm > a.max_norm         ? a.max_norm / norm
                                                    : 1.0f;
    }
}

template <int kN>
cudaError_t adamw_of(const AdamwStep& h, const AdamwTensor* t, const uint32_t* first, int count, uint32_t chunks,
                     int iters, cudaStream_t s) {
    AdamwTensors<kN> list;
    std::copy(t, t + count, list.t);
    std::copy(first, first + count, list.first);
    return pdl_launch(k_adamw<kN>, dim3(chunks), dim3(kThreads), 0, s, h, list, count, iters);
}

template <int kN>
cudaError_t adamw_mx_of(const AdamwStep& h, const AdamwTensor* t, const uint32_t* first, int count, uint32_t cells,
                        cudaStream_t s) {
    constexpr int kPiece = kStages * kMxThreads * 16;
    static PerDevice allowed;
    cudaError_t e = allow_shared(allowed, k_adamw_mx<kN>, kPiece * pieces_of(true, true));
    if (e != cudaSuccess) return e;
    AdamwTensors<kN> list;
    std::copy(t, t + count, list.t);
    std::copy(first, first + count, list.first);
    bool p32 = false, g32 = false;
    for (int i = 0; i < count; ++i) {
        p32 |= (t[i].kind & (kParamF32 | kMaster)) != 0;
        g32 |= (t[i].kind & kGradF32) != 0;
    }
    const int smem = kPiece * pieces_of(p32, g32), per_sm = std::min(kMxBlocks, 220 * 1024 / (smem + 1024));
    const unsigned full = device_sm_count() * per_sm;
    const unsigned per_block = std::max(1u, std::min(kCellsPerBlock, (cells + full - 1) / full));
    return pdl_launch(k_adamw_mx<kN>, dim3((cells + per_block - 1) / per_block), dim3(kMxThreads), smem, s, h, list,
                      count, cells, per_block);
}

}  // namespace

cudaError_t launch_adamw(const AdamwStep& h, const AdamwTensor* tensors, int count, bool mx, cudaStream_t s) {
    uint64_t all = 0;
    for (int i = 0; i < count; ++i) all += tensors[i].n;
    // fp32 states: four rounds a block, or, where that leaves SMs idle, one
    const int iters = all >= (uint64_t)device_sm_count() * 8 * kThreads * 8 * 4 ? 4 : 1;
    const uint64_t chunk = mx ? kCell : (uint64_t)kThreads * 8 * iters;
    for (int first = 0; first < count;) {
        uint64_t chunks = 0;
        int n = 0;
        uint32_t begins[kMostTensors];
        for (; first + n < count && n < kMostTensors; ++n) {
            const uint64_t mine = (tensors[first + n].n + chunk - 1) / chunk;
            if (n && chunks + mine > 0x7FFFFFFFu) break;
            begins[n] = (uint32_t)chunks;
            chunks += mine;
        }
        cudaError_t e;
        const AdamwTensor* t = tensors + first;
        if (n <= kFewTensors)
            e = mx ? adamw_mx_of<kFewTensors>(h, t, begins, n, (uint32_t)chunks, s)
                   : adamw_of<kFewTensors>(h, t, begins, n, (uint32_t)chunks, iters, s);
        else
            e = mx ? adamw_mx_of<kMostTensors>(h, t, begins, n, (uint32_t)chunks, s)
                   : adamw_of<kMostTensors>(h, t, begins, n, (uint32_t)chunks, iters, s);
        if (e != cudaSuccess) return e;
        first += n;
    }
    return cudaSuccess;
}

namespace {
template <bool kParam32, bool kMasters, bool kTableMx>
cudaError_t rows_mx_of(const AdamwStep& h, const AdamwRows& a, cudaStream_t s) {
    constexpr int kSmem = 2 * kMxThreads * 16 * pieces_of(kParam32 || kMasters, true);
    static PerDevice allowed;
    auto f = k_adamw_rows_mx<kParam32, kMasters, kTableMx>;
    cudaError_t e = allow_shared(allowed, f, kSmem);
    if (e != cudaSuccess) return e;
    // four rounds a block, so that blocks follow one another in the table's order (1.08M rows of
    // 256: 735 us, 811 with blocks that stay), or fewer where SMs would be idle
    const uint64_t rounds = ((uint64_t)a.n * (a.dim / 16) + kMxThreads - 1) / kMxThreads;
    const uint64_t full = (uint64_t)device_sm_count() * kMxBlocks;
    const unsigned grid = (unsigned)std::min<uint64_t>(std::max((rounds + 3) / 4, std::min(rounds, full)), 0x7FFFFFFF);
    return pdl_launch(f, dim3(grid), dim3(kMxThreads), kSmem, s, h, a);
}
}  // namespace

cudaError_t launch_adamw_rows(const AdamwStep& h, const AdamwRows& a, bool mx, cudaStream_t s) {
    const bool table_mx = a.kind & kParamMx;
    const uint64_t full_rows = (uint64_t)device_sm_count() * 6;
    if (mx)
        return table_mx             ? rows_mx_of<false, true, true>(h, a, s)
               : a.kind & kMaster   ? rows_mx_of<false, true, false>(h, a, s)
               : a.kind & kParamF32 ? rows_mx_of<true, false, false>(h, a, s)
                                    : rows_mx_of<false, false, false>(h, a, s);
    // as above, of two rounds (4,915 rows of 5,120: 118 us, 131 with blocks that stay)
    const uint64_t rounds = ((uint64_t)a.n * (a.dim / 4) + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)std::min<uint64_t>(std::max((rounds + 1) / 2, std::min(rounds, full_rows)), 0x7FFFFFFF);
    return pdl_launch(table_mx ? k_adamw_rows<true> : k_adamw_rows<false>, dim3(grid), dim3(kThreads), 0, s, h, a);
}

static int grad_norm_blocks() { return device_sm_count() * 4; }

size_t grad_norm_slots(uint64_t values) {
    return (size_t)std::min<uint64_t>((values + kNormUnit - 1) / kNormUnit, grad_norm_blocks());
}

namespace {
template <int kN>
cudaError_t squares_of(const GradPart* parts, const uint32_t* first, int n, uint32_t units, double* part,
                       uint4* range, cudaStream_t s) {
    GradParts<kN> list;
    std::copy(parts, parts + n, list.p);
    std::copy(first, first + n, list.first);
    const unsigned blocks = std::min<unsigned>(units, grad_norm_blocks());
    return pdl_launch(k_grad_squares<kN>, dim3(blocks), dim3(kThreads), 0, s, list, n, units, part, range);
}
}  // namespace

cudaError_t launch_grad_norm(const GradNormArgs& a, GradPart* parts, cudaStream_t s) {
    uint32_t slot = 0;
    cudaError_t e = cudaSuccess;
    for (int first = 0; first < a.count && e == cudaSuccess;) {
        uint64_t units = 0;
        int n = 0;
        uint32_t begins[kMostParts];
        for (; first + n < a.count && n < kMostParts; ++n) {
            const uint64_t values = parts[first + n].n * parts[first + n].dim;
            const uint64_t mine = (values + kNormUnit - 1) / kNormUnit;
            if (n && units + mine > 0x7FFFFFFFu) break;
            begins[n] = (uint32_t)units;
            units += mine;
            parts[first + n].slot = slot;
            slot += (uint32_t)grad_norm_slots(values);
        }
        e = n <= kFewParts
                ? squares_of<kFewParts>(parts + first, begins, n, (uint32_t)units, a.part, a.range + first, s)
                : squares_of<kMostParts>(parts + first, begins, n, (uint32_t)units, a.part, a.range + first, s);
        first += n;
    }
    if (e != cudaSuccess) return e;
    return pdl_launch(k_grad_norm, dim3(1), dim3(1024), 0, s, a);
}

}  // namespace engram
