// Memory-bound kernels of the training step (sm_103a): the scaled embedding
// lookup, its gradient by sorted ids, the gate with an 8-bit checkpoint of its
// activations, and the gate's backward pass.
#include <algorithm>

#include "device_common.cuh"
#include "grad_internal.h"
#include "tcgen05_common.cuh"

namespace engram {

namespace {

template <class... Exp, class... Act>
cudaError_t pdl_launch(void (*f)(Exp...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Act... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, f, static_cast<Exp>(args)...);
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(bf16x2_pack_rn(f[0], f[1]), bf16x2_pack_rn(f[2], f[3]),
                      bf16x2_pack_rn(f[4], f[5]), bf16x2_pack_rn(f[6], f[7]));
}
__device__ __forceinline__ void load8_f32(const float* p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void store8_f32(float* p, const float (&f)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

// ---- embedding ----------------------------------------------------------------------
// out[t][c] = scale table[ids[t]], c < copies, rounded once to BF16.  A group of
// `lanes` threads takes one id, 8 columns per thread and step, and writes every
// copy of what it read, so the table row is read once.
template <bool kF32>
__global__ void __launch_bounds__(256)
k_embed(const void* __restrict__ table, uint64_t rows, int dim, const uint32_t* __restrict__ ids,
        int64_t n, float scale, int copies, int lanes, uint16_t* __restrict__ out, uint32_t* err) {
    pdl_wait();
    pdl_launch_dependents();
    const int per = 256 / lanes, chunks = dim / 8;
    const int l = threadIdx.x % lanes;
    const int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / lanes;
    if (t >= n) return;
    const uint32_t id = ids[t];
    const bool in = id < rows;
    if (!in && id != kMasked && l == 0) atomicOr(err, kErrBounds);
    for (int c = l; c < chunks; c += lanes) {
        float f[8] = {};
        if (in) {
            const int64_t at = (int64_t)id * dim + c * 8;
            if (kF32)
                load8_f32(static_cast<const float*>(table) + at, f);
            else
                unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(table) + at)), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= scale;
        }
        const uint4 o = pack8(f);
        for (int k = 0; k < copies; ++k)
            *reinterpret_cast<uint4*>(out + (t * copies + k) * (int64_t)dim + c * 8) = o;
    }
}

// ---- sort of the ids -------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWarps = 32;

// A barrier of the cooperative launch's blocks, bounded: false on a time-out.
__device__ __forceinline__ bool grid_barrier(const EmbedSort& a, uint32_t& phase, int* flag) {
    __syncthreads();
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) {
            ++phase;
            const uint32_t want = phase * gridDim.x;
            __threadfence();
            atomicAdd(a.barrier, 1u);
            const uint64_t t0 = globaltimer();
            uint32_t spin = 0;
            while (ld_acquire_u32(a.barrier) < want) {
                if ((++spin & 63u) == 0u && (long long)(globaltimer() - t0) > a.wait_limit_ns) {
                    atomicOr(a.err, kErrTimeout);
                    *flag = 1;
                    break;
                }
            }
            __threadfence();
        }
        __syncthreads();
    }
    return *flag == 0;
}

// Stable radix sort of (id, position), least significant digit first, then the
// segments of equal ids.  A block owns a contiguous range of the keys and a
// warp a contiguous part of it, so the order of equal digits is kept: per pass,
// every warp counts its digits (lanes with equal digits found by match_any, one
// of them adds their number), the counts are turned into first places over
// (digit, block, warp), and each warp hands them out in key order.  Ids that
// are masked or outside the table become `rows`, the largest key: they sort
// behind every row and take no part.
__global__ void __launch_bounds__(kSortThreads)
k_embed_sort(const EmbedSort a) {
    extern __shared__ uint32_t cnt[];  // [kSortWarps][bins]
    __shared__ uint32_t warp_sum[kSortWarps];
    __shared__ uint32_t shared_base;
    __shared__ int flag;
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lt = (1u << lane) - 1u;
    const int B = (int)gridDim.x, b = (int)blockIdx.x;
    const int bins = 1 << a.digit_bits;
    const uint32_t dmask = (uint32_t)bins - 1u;
    // ranges in whole rounds of 32 keys
    const int64_t rounds = (a.n + 31) / 32;
    const int64_t r0 = rounds * b / B, r1 = rounds * (b + 1) / B;
    const int64_t w0 = r0 + (r1 - r0) * warp / kSortWarps;
    const int64_t w1 = r0 + (r1 - r0) * (warp + 1) / kSortWarps;
    uint32_t phase = 0;
    if (threadIdx.x == 0) flag = 0;
    __syncthreads();
    const uint32_t rows = (uint32_t)a.rows;

    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.digit_bits;
        const uint32_t* kin = pass & 1 ? a.keys1 : a.keys0;
        const uint32_t* vin = pass & 1 ? a.vals1 : a.vals0;
        uint32_t* kout = pass & 1 ? a.keys0 : a.keys1;
        uint32_t* vout = pass & 1 ? a.vals0 : a.vals1;
        auto key = [&](int64_t i) {
            if (pass) return __ldcg(kin + i);
            const uint32_t id = a.ids[i];
            return id < rows ? id : rows;
        };
        for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) cnt[i] = 0;
        __syncthreads();
        uint32_t* mine = cnt + warp * bins;
        for (int64_t r = w0; r < w1; ++r) {
            const int64_t i = r * 32 + lane;
            const bool on = i < a.n;
            if (pass == 0 && on) {
                const uint32_t id = a.ids[i];
                if (id >= rows && id != kMasked) atomicOr(a.err, kErrBounds);
            }
            const uint32_t d = on ? (key(i) >> shift) & dmask : 0xFFFFFFFFu;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, d);
            if (on && (same & lt) == 0u) mine[d] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        for (int d = threadIdx.x; d < bins; d += kSortThreads) {
            uint32_t s = 0;
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = cnt[w * bins + d];
                cnt[w * bins + d] = s;
                s += c;
            }
            __stcg(a.hist + (int64_t)d * B + b, s);
        }
        if (!grid_barrier(a, phase, &flag)) return;
        // first place of each (digit, block) within its digit
        for (int d = b * kSortWarps + warp; d < bins; d += B * kSortWarps) {
            uint32_t run = 0;
            for (int x0 = 0; x0 < B; x0 += 32) {
                const int x = x0 + lane;
                const uint32_t c = x < B ? __ldcg(a.hist + (int64_t)d * B + x) : 0u;
                uint32_t inc = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                    if (lane >= o) inc += y;
                }
                if (x < B) __stcg(a.hist + (int64_t)d * B + x, run + inc - c);
                run += __shfl_sync(0xFFFFFFFFu, inc, 31);
            }
            if (lane == 0) __stcg(a.digit_total + d, run);
        }
        if (!grid_barrier(a, phase, &flag)) return;
        // places over the digits (bins <= 1,024: one digit per thread)
        {
            const int d = threadIdx.x;
            const uint32_t c = d < bins ? __ldcg(a.digit_total + d) : 0u;
            uint32_t inc = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) warp_sum[warp] = inc;
            __syncthreads();
            if (warp == 0) {
                const uint32_t s = warp_sum[lane];
                uint32_t si = s;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, si, o);
                    if (lane >= o) si += y;
                }
                warp_sum[lane] = si - s;
            }
            __syncthreads();
            if (d < bins) {
                const uint32_t base = warp_sum[warp] + inc - c + __ldcg(a.hist + (int64_t)d * B + b);
                for (int w = 0; w < kSortWarps; ++w) cnt[w * bins + d] += base;
            }
            __syncthreads();
        }
        for (int64_t r = w0; r < w1; ++r) {
            const int64_t i = r * 32 + lane;
            const bool on = i < a.n;
            const uint32_t k = on ? key(i) : 0u;
            const uint32_t v = on ? (pass ? __ldcg(vin + i) : (uint32_t)i) : 0u;
            const uint32_t d = on ? (k >> shift) & dmask : 0xFFFFFFFFu;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, d);
            uint32_t at = 0;
            if (on) at = mine[d] + __popc(same & lt);
            __syncwarp();
            if (on && (same & lt) == 0u) mine[d] += __popc(same);
            __syncwarp();
            if (on) {
                __stcg(kout + at, k);
                __stcg(vout + at, v);
            }
        }
        if (!grid_barrier(a, phase, &flag)) return;
    }

    // segments of equal ids among the n_valid ids of table rows
    const uint32_t* keys = a.passes & 1 ? a.keys1 : a.keys0;
    auto head = [&](int64_t i, uint32_t k) {
        return k < rows && (i == 0 || __ldcg(keys + i - 1) != k);
    };
    const int64_t i0 = r0 * 32, i1 = min(r1 * 32, a.n);
    uint32_t heads = 0;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) {
        const uint32_t k = __ldcg(keys + i);
        heads += head(i, k) ? 1u : 0u;
        if (i == 0 && k >= rows) __stcg(a.n_valid, 0u);
        if (k < rows && (i == a.n - 1 || __ldcg(keys + i + 1) >= rows)) __stcg(a.n_valid, (uint32_t)(i + 1));
    }
    heads = __reduce_add_sync(0xFFFFFFFFu, heads);
    if (lane == 0) warp_sum[warp] = heads;
    __syncthreads();
    if (warp == 0) {
        const uint32_t s = __reduce_add_sync(0xFFFFFFFFu, warp_sum[lane]);
        if (lane == 0) __stcg(a.block_heads + b, s);
    }
    if (!grid_barrier(a, phase, &flag)) return;
    if (warp == 0) {
        uint32_t before = 0, all = 0;
        for (int x = lane; x < B; x += 32) {
            const uint32_t c = __ldcg(a.block_heads + x);
            all += c;
            if (x < b) before += c;
        }
        before = __reduce_add_sync(0xFFFFFFFFu, before);
        all = __reduce_add_sync(0xFFFFFFFFu, all);
        if (lane == 0) {
            shared_base = before;
            if (b == B - 1) {
                *a.count = all;
                a.seg_start[all] = __ldcg(a.n_valid);
            }
        }
    }
    __syncthreads();
    uint32_t base = shared_base;
    for (int64_t t0 = i0; t0 < i1; t0 += kSortThreads) {
        const int64_t i = t0 + threadIdx.x;
        const uint32_t k = i < i1 ? __ldcg(keys + i) : rows;
        const bool h = i < i1 && head(i, k);
        const uint32_t bal = __ballot_sync(0xFFFFFFFFu, h);
        __syncthreads();  // warp_sum of the round before is read
        if (lane == 0) warp_sum[warp] = __popc(bal);
        __syncthreads();
        const uint32_t s = warp_sum[lane];
        const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s : 0u);
        const uint32_t round_all = __reduce_add_sync(0xFFFFFFFFu, s);
        const uint32_t upto = base + before + __popc(bal & (lt | (1u << lane)));
        if (i < i1 && k < rows) {
            a.segpos[i] = upto - 1u;
            if (h) {
                a.unique[upto - 1u] = k;
                a.seg_start[upto - 1u] = (uint32_t)i;
            }
        }
        base += round_all;
    }
}

// ---- sums over the segments ---------------------------------------------------------------
// A chunk is kSumRows consecutive places of the sorted order; a group of `lanes`
// threads sums one chunk's rows over 8 columns per thread, in order, and writes
// each segment that begins and ends in the chunk.  A segment that crosses
// chunks leaves one partial sum per chunk - the chunk's head (it began earlier)
// or tail (it begins here) - for k_embed_join, which adds them in order.  So no
// sum depends on the order in which blocks run, and a hot id's rows are spread
// over as many threads as a cold one's.
constexpr int kSumBatch = 8;

__device__ __forceinline__ void put_row(const EmbedSum& a, uint32_t seg, int col,
                                        const float (&acc)[8]) {
    const int64_t dest = a.dense ? a.unique[seg] : seg;
    float* p = a.grad + dest * a.dim + col;
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = acc[j] * a.scale;
    if (a.accumulate) {
        float x[8];
        load8_f32(p, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += x[j];
    }
    store8_f32(p, o);
}

__global__ void __launch_bounds__(256)
k_embed_sum(const EmbedSum a) {
    pdl_wait();
    pdl_launch_dependents();
    const int l = threadIdx.x % a.lanes;
    const int64_t work = ((int64_t)blockIdx.x * 256 + threadIdx.x) / a.lanes;
    const int64_t chunk = work / a.slices;
    const int col = ((int)(work - chunk * a.slices) * a.lanes + l) * 8;
    const int64_t nv = *a.n_valid;
    const int64_t lo = chunk * a.rows_per_chunk, hi = min(lo + a.rows_per_chunk, nv);
    if (lo >= hi || col >= a.dim) return;
    float acc[8] = {};
    uint32_t cur = a.segpos[lo];
    auto flush = [&](uint32_t seg) {
        const int64_t s0 = a.seg_start[seg], s1 = a.seg_start[seg + 1];
        if (s0 >= lo && s1 <= hi)
            put_row(a, seg, col, acc);
        else
            store8_f32(a.partial + (2 * chunk + (s0 >= lo ? 1 : 0)) * a.dim + col, acc);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    };
    // rows are (place, copy) pairs, a batch of them loaded before they are added
    const int64_t total = (hi - lo) * a.copies;
    int64_t pos = lo;
    int copy = 0;
    for (int64_t q0 = 0; q0 < total; q0 += kSumBatch) {
        uint4 v[kSumBatch];
        uint32_t seg[kSumBatch];
#pragma unroll
        for (int u = 0; u < kSumBatch; ++u) {
            if (q0 + u < total) {
                seg[u] = a.segpos[pos];
                v[u] = __ldcs(reinterpret_cast<const uint4*>(
                    a.dout + ((int64_t)a.perm[pos] * a.copies + copy) * a.dim + col));
                if (++copy == a.copies) {
                    copy = 0;
                    ++pos;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kSumBatch; ++u) {
            if (q0 + u < total) {
                if (seg[u] != cur) {
                    flush(cur);
                    cur = seg[u];
                }
                float f[8];
                unpack8(v[u], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += f[j];
            }
        }
    }
    flush(cur);
}

// One block per (chunk, 256 columns): if a segment begins in the chunk and
// leaves it, its row is the chunk's tail and the following chunks' heads, each
// of the block's eight warps adding a contiguous share in order, the shares
// then in order.
__global__ void __launch_bounds__(256)
k_embed_join(const EmbedSum a) {
    pdl_wait();
    __shared__ float sm[8][32][9];
    const int64_t chunk = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = ((int)blockIdx.y * 32 + lane) * 8;
    const int64_t nv = *a.n_valid;
    const int64_t lo = chunk * a.rows_per_chunk, hi = lo + a.rows_per_chunk;
    if (hi >= nv) return;  // (a last chunk's segment ends in it)
    const uint32_t seg = a.segpos[hi - 1];
    const int64_t s0 = a.seg_start[seg], s1 = a.seg_start[seg + 1];
    if (s0 < lo || s1 <= hi) return;
    const int64_t parts = (s1 - 1) / a.rows_per_chunk - chunk + 1;  // tail, then heads
    const int64_t p0 = parts * warp / 8, p1 = parts * (warp + 1) / 8;
    float acc[8] = {};
    if (col < a.dim) {
#pragma unroll 4
        for (int64_t p = p0; p < p1; ++p) {
            float x[8];
            load8_f32(a.partial + (2 * (chunk + p) + (p == 0 ? 1 : 0)) * a.dim + col, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += x[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sm[warp][lane][j] = acc[j];
    __syncthreads();
    if (warp || col >= a.dim) return;
    for (int w = 1; w < 8; ++w)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += sm[w][lane][j];
    put_row(a, seg, col, acc);
}

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

// ---- gate with checkpoint ------------------------------------------------------------------
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
    const float g = 1.0f / (1.0f + expf(-copysignf(root, x)));
    const float dx = fabsf(x) > 1e-6f ? dyv * g * (1.0f - g) / (2.0f * root) : 0.f;
    return make_float4(dx * rs, dx * x * rh * rh * inv_d, dx * x * rk * rk * inv_d, g);
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

// dwq = wk sum, dwk = wq sum, the shares added in order.
__global__ void __launch_bounds__(256)
k_gate_backward_weights(const GateTrain a, int shares) {
    pdl_wait();
    const int64_t n = (int64_t)a.hc * a.d;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
#pragma unroll 8
    for (int p = 0; p < shares; ++p) s += __ldcg(a.dw_part + p * n + i);
    if (a.dwq) a.dwq[i] = s * a.wk[i];
    if (a.dwk) a.dwk[i] = s * a.wq[i];
}

template <int kSaved>
cudaError_t gate_backward(const GateTrain& a, int shares, cudaStream_t s) {
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
    if (e != cudaSuccess) return e;
    return pdl_launch(k_gate_backward_weights, dim3((unsigned)(((int64_t)a.hc * a.d + 255) / 256)),
                      dim3(256), 0, s, a, shares);
}

int log2_ceil(int64_t x) {
    int b = 0;
    while (((int64_t)1 << b) < x) ++b;
    return b;
}

}  // namespace

cudaError_t launch_embed(const void* table, bool f32, uint64_t rows, int dim, const uint32_t* ids,
                         int64_t n, float scale, int copies, uint16_t* out, uint32_t* err,
                         cudaStream_t s) {
    const int lanes = 1 << std::min(8, log2_ceil(dim / 8));
    const int per = 256 / lanes;
    return pdl_launch(f32 ? k_embed<true> : k_embed<false>, dim3((unsigned)((n + per - 1) / per)),
                      dim3(256), 0, s, table, rows, dim, ids, n, scale, copies, lanes, out, err);
}

int embed_sort_blocks(int64_t n) {
    return (int)std::min<int64_t>(device_sm_count(), std::max<int64_t>(1, (n + 8191) / 8192));
}

void embed_sort_digits(uint64_t rows, int* passes, int* bits) {
    int need = 1;
    while (need < 32 && (rows >> need)) ++need;  // the largest key is `rows`
    *passes = (need + 8) / 9;
    *bits = (need + *passes - 1) / *passes;
}

cudaError_t launch_embed_sort(const EmbedSort& a, cudaStream_t s) {
    const int blocks = embed_sort_blocks(a.n);
    const int smem = kSortWarps * (1 << a.digit_bits) * 4;
    cudaError_t e = cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (blocks > 1) {
        e = cudaMemsetAsync(a.barrier, 0, 4, s);
        if (e != cudaSuccess) return e;
        EmbedSort copy = a;
        void* args[] = {&copy};
        return cudaLaunchCooperativeKernel((void*)k_embed_sort, dim3(blocks), dim3(kSortThreads),
                                           args, smem, s);
    }
    return pdl_launch(k_embed_sort, dim3(1), dim3(kSortThreads), smem, s, a);
}

int embed_rows_per_chunk(int64_t n, int dim, int copies) {
    (void)copies;
    // long enough that partial sums are few beside the rows read, short enough
    // that the chunks fill the GPU
    return n * (int64_t)dim >= (int64_t)1 << 26 ? 64 : n * (int64_t)dim >= (int64_t)1 << 22 ? 32 : 8;
}

cudaError_t launch_embed_sum(EmbedSum a, int64_t n, cudaStream_t s) {
    a.lanes = 1 << std::min(5, log2_ceil(a.dim / 8));
    a.slices = (a.dim / 8 + a.lanes - 1) / a.lanes;
    const int64_t chunks = (n + a.rows_per_chunk - 1) / a.rows_per_chunk;
    const int64_t threads = chunks * a.slices * a.lanes;
    cudaError_t e = pdl_launch(k_embed_sum, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a);
    if (e != cudaSuccess || chunks < 2) return e;
    return pdl_launch(k_embed_join, dim3((unsigned)(chunks - 1), (unsigned)((a.dim + 255) / 256)),
                      dim3(256), 0, s, a);
}

cudaError_t launch_gate_checkpoint(const GateTrain& a, bool kv_f32, cudaStream_t s) {
    return pdl_launch(kv_f32 ? k_gate_checkpoint<true> : k_gate_checkpoint<false>,
                      dim3((unsigned)a.T), dim3(std::min(320, a.d / 8)), 0, s, a);
}

int gate_backward_shares(int64_t T, int d) {
    const int blocks = (d / 8 + 127) / 128;
    return (int)std::max<int64_t>(1, std::min<int64_t>(T, device_sm_count() * 4 / blocks));
}

cudaError_t launch_gate_backward(const GateTrain& a, int saved, cudaStream_t s) {
    const int shares = gate_backward_shares(a.T, a.d);
    if (saved == kSavedMx) return gate_backward<kSavedMx>(a, shares, s);
    if (saved == kSavedF32) return gate_backward<kSavedF32>(a, shares, s);
    return gate_backward<kSavedBf16>(a, shares, s);
}

}  // namespace engram
