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
constexpr int kSortBatch = 8;  // rounds of 32 keys that a warp loads at once
constexpr int kSmallSort = kSortThreads * 8 * 4;  // keys of the one-cluster sort

// A barrier of the cooperative launch's blocks in two halves, so that a block can
// work between them; the wait is bounded: false on a time-out.
__device__ __forceinline__ void grid_arrive(const EmbedSort& a) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atomicAdd(a.barrier, 1u);
    }
}
__device__ __forceinline__ bool grid_wait(const EmbedSort& a, uint32_t& phase, int* flag) {
    if (threadIdx.x == 0) {
        const uint32_t want = ++phase * gridDim.x;
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
    return *flag == 0;
}

// The lanes whose digit equals this lane's (of `bits` bits), among the `on`
// lanes: one vote per bit (faster than match.any: 27 us against 33 for the sort
// of 8,192 ids in one block).
__device__ __forceinline__ uint32_t same_digit(uint32_t d, int bits, uint32_t on) {
    uint32_t same = on;
#pragma unroll
    for (int b = 0; b < 9; ++b) {
        if (b < bits) {
            const bool set = (d >> b) & 1u;
            const uint32_t v = __ballot_sync(0xFFFFFFFFu, set);
            same &= set ? v : ~v;
        }
    }
    return same;
}

// Exclusive sums over the block of one value per thread; *all gets the total.
__device__ __forceinline__ uint32_t block_scan(uint32_t c, uint32_t* warp_sum, uint32_t* all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
    }
    __syncthreads();  // what an earlier call left in warp_sum is read
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    const uint32_t s = warp_sum[lane];
    const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s : 0u);
    *all = __reduce_add_sync(0xFFFFFFFFu, s);
    return before + inc - c;
}

// Exclusive sums of each digit's counts over the warps, in place; the digit's
// total for the thread that holds it (bins <= 512 of the 1,024 threads).
__device__ __forceinline__ uint32_t scan_warps(uint32_t* cnt, int bins) {
    uint32_t total = 0;
    if ((int)threadIdx.x < bins) {
#pragma unroll
        for (int w0 = 0; w0 < kSortWarps; w0 += 16) {
            uint32_t c[16];
#pragma unroll
            for (int w = 0; w < 16; ++w) c[w] = cnt[(w0 + w) * bins + threadIdx.x];
#pragma unroll
            for (int w = 0; w < 16; ++w) {
                cnt[(w0 + w) * bins + threadIdx.x] = total;
                total += c[w];
            }
        }
    }
    return total;
}
__device__ __forceinline__ void add_warps(uint32_t* cnt, int bins, uint32_t base) {
    if ((int)threadIdx.x < bins) {
#pragma unroll 16
        for (int w = 0; w < kSortWarps; ++w) cnt[w * bins + threadIdx.x] += base;
    }
}

// Eight neighbouring sorted keys (from place i0) and the ones beside them: which
// of them begin a segment, and where the ids of table rows end.
struct Heads {
    uint32_t key[kSortBatch];
    uint32_t begins;  // bit u: place i0 + u begins a segment
    uint32_t last;    // bit u: place i0 + u holds the last id of a table row
};
__device__ __forceinline__ Heads find_heads(const uint32_t (&key)[kSortBatch], uint32_t before,
                                            uint32_t after, int64_t i0, int64_t end, uint32_t rows) {
    Heads h;
    h.begins = h.last = 0;
    uint32_t prev = before;
#pragma unroll
    for (int u = 0; u < kSortBatch; ++u) {
        h.key[u] = key[u];
        const bool valid = i0 + u < end && key[u] < rows;
        const uint32_t next = u + 1 < kSortBatch ? key[u + 1 < kSortBatch ? u + 1 : u] : after;
        if (valid && (i0 + u == 0 || key[u] != prev)) h.begins |= 1u << u;
        if (valid && (i0 + u + 1 >= end || next >= rows)) h.last |= 1u << u;
        prev = key[u];
    }
    return h;
}
// Stable radix sort of (id, position), least significant digit first, then the
// segments of equal ids.  A block owns a contiguous range of the keys, in tiles
// of up to 8,192, a warp a contiguous part of a tile, so the order of equal
// digits is kept.  Per pass: every warp counts its digits (one of the lanes with
// equal digits adds their number); the counts become first places over (digit,
// block); the tile is put in digit order in shared memory and leaves in runs of
// equal digits.  (Written from where they lay, each key to a sector of its own,
// 1.2 million keys took 30 us a pass, bound by L2's sectors.)  Ids that are
// masked or outside the table become `rows`, the largest key: they sort behind
// every row and take no part.
__global__ void __launch_bounds__(kSortThreads)
k_embed_sort(const EmbedSort a) {
    extern __shared__ uint32_t cnt[];  // [kSortWarps][bins], then the tile in digit order
    __shared__ uint32_t place[512];    // of the block's next key of each digit, less its place in the tile
    __shared__ uint32_t warp_sum[kSortWarps];
    __shared__ uint32_t shared_base;
    __shared__ int flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lt = (1u << lane) - 1u;
    const int B = (int)gridDim.x, b = (int)blockIdx.x;
    const int bins = 1 << a.digit_bits;
    const uint32_t dmask = (uint32_t)bins - 1u;
    uint2* const tile = reinterpret_cast<uint2*>(cnt + kSortWarps * bins);
    // ranges in whole multiples of 32 keys; a tile is `per` keys of every warp
    const int64_t rounds = (a.n + 31) / 32;
    const int64_t lo = rounds * b / B * 32, hi = min(rounds * (b + 1) / B * 32, a.n);
    const int per = (int)min((int64_t)kSortBatch, (hi - lo + kSortThreads - 1) / kSortThreads);  // rounds
    const int64_t tile_keys = (int64_t)per * kSortThreads;
    const bool one = hi - lo <= tile_keys;
    uint32_t phase = 0;
    if (threadIdx.x == 0) flag = 0;
    __syncthreads();
    const uint32_t rows = (uint32_t)a.rows;
    uint32_t* const mine = cnt + warp * bins;
    const bool has_digit = (int)threadIdx.x < bins;  // (bins <= 512)

    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.digit_bits;
        const uint2* in = pass & 1 ? a.pairs1 : a.pairs0;
        uint2* out = pass & 1 ? a.pairs0 : a.pairs1;
        uint2 kv[kSortBatch];
        uint32_t at[kSortBatch];
        auto key_index = [&](int64_t t0, int u) { return t0 + (warp * per + u) * 32 + lane; };
        auto load = [&](int64_t t0) {
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                if (u >= per) break;
                const int64_t i = key_index(t0, u);
                kv[u] = make_uint2(0u, 0u);
                if (i < hi) kv[u] = pass ? __ldcg(in + i) : make_uint2(min(a.ids[i], rows), (uint32_t)i);
            }
        };
        // a key's place among its warp's keys of the same digit
        auto rank = [&](int64_t t0) {
            for (int i = lane; i < bins; i += 32) mine[i] = 0;
            __syncwarp();
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                if (u >= per) break;
                const bool on = key_index(t0, u) < hi;
                const uint32_t all_on = __ballot_sync(0xFFFFFFFFu, on);
                const uint32_t d = (kv[u].x >> shift) & dmask;
                const uint32_t same = same_digit(d, a.digit_bits, all_on);
                at[u] = on ? mine[d] + __popc(same & lt) : 0u;
                __syncwarp();
                if (on && (same & lt) == 0u) mine[d] += __popc(same);
                __syncwarp();
            }
            __syncthreads();
        };
        // the tile in digit order; `total`: the tile's keys of this thread's digit
        auto reorder = [&](int64_t t0, uint32_t total) {
            uint32_t all;
            const uint32_t start = block_scan(total, warp_sum, &all);
            add_warps(cnt, bins, start);
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u) {
                if (u >= per) break;
                if (key_index(t0, u) < hi) tile[at[u] + mine[(kv[u].x >> shift) & dmask]] = kv[u];
            }
            __syncthreads();
            return start;
        };
        uint32_t total = 0, start = 0;
        if (one) {
            load(lo);
            rank(lo);
            total = scan_warps(cnt, bins);
        } else {  // only the counts of the whole range
            for (int i = threadIdx.x; i < bins; i += kSortThreads) cnt[i] = 0;
            __syncthreads();
            for (int64_t t0 = lo; t0 < hi; t0 += tile_keys) {
                load(t0);
#pragma unroll
                for (int u = 0; u < kSortBatch; ++u)
                    if (key_index(t0, u) < hi) atomicAdd(cnt + ((kv[u].x >> shift) & dmask), 1u);
            }
            __syncthreads();
            total = has_digit ? cnt[threadIdx.x] : 0u;
        }
        if (pass == 0)  // ids outside the table
            for (int64_t i = lo + threadIdx.x; i < hi; i += kSortThreads)
                if (a.ids[i] >= rows && a.ids[i] != kMasked) atomicOr(a.err, kErrBounds);
        if (has_digit) __stcg(a.hist + (int64_t)threadIdx.x * B + b, total);
        grid_arrive(a);
        if (one) start = reorder(lo, total);
        if (!grid_wait(a, phase, &flag)) return;
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
        grid_arrive(a);
        if (!grid_wait(a, phase, &flag)) return;
        uint32_t all;
        const uint32_t base = block_scan(has_digit ? __ldcg(a.digit_total + threadIdx.x) : 0u, warp_sum, &all);
        uint32_t next = has_digit ? base + __ldcg(a.hist + (int64_t)threadIdx.x * B + b) : 0u;
        for (int64_t t0 = lo; t0 < hi; t0 += tile_keys) {
            if (!one) {
                load(t0);
                rank(t0);
                total = scan_warps(cnt, bins);
                start = reorder(t0, total);
            }
            if (has_digit) place[threadIdx.x] = next - start;
            next += total;
            __syncthreads();
            const int count = (int)min(tile_keys, hi - t0);
            for (int i = threadIdx.x; i < count; i += kSortThreads) {
                const uint2 x = tile[i];
                __stcg(out + (place[(x.x >> shift) & dmask] + (uint32_t)i), x);
            }
            __syncthreads();
        }
        grid_arrive(a);
        if (!grid_wait(a, phase, &flag)) return;
    }

    // segments of equal ids among the ids of table rows
    const uint2* pairs = a.passes & 1 ? a.pairs1 : a.pairs0;
    auto heads_at = [&](int64_t i0) {
        uint32_t key[kSortBatch];
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u) key[u] = i0 + u < hi ? __ldcg(pairs + i0 + u).x : rows;
        const uint32_t before = i0 > 0 && i0 < hi ? __ldcg(pairs + i0 - 1).x : rows;
        const uint32_t after = i0 + kSortBatch < a.n ? __ldcg(pairs + i0 + kSortBatch).x : rows;
        // (hi is a multiple of eight unless it is n: `after` is the next place's key)
        return find_heads(key, before, after, i0, hi < a.n && i0 + kSortBatch >= hi ? hi + 1 : hi, rows);
    };
    Heads h;
    h.begins = h.last = 0;
    uint32_t heads = 0;
    for (int64_t i0 = lo + threadIdx.x * kSortBatch; i0 < hi; i0 += kSortThreads * kSortBatch) {
        h = heads_at(i0);
        heads += __popc(h.begins);
        if (h.last) __stcg(a.n_valid, (uint32_t)(i0 + __ffs(h.last)));
    }
    if (b == 0 && threadIdx.x == 0 && __ldcg(pairs).x >= rows) __stcg(a.n_valid, 0u);
    uint32_t block_heads;
    block_scan(heads, warp_sum, &block_heads);
    if (threadIdx.x == 0) __stcg(a.block_heads + b, block_heads);
    grid_arrive(a);
    if (!grid_wait(a, phase, &flag)) return;
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
    for (int64_t t0 = lo; t0 < hi; t0 += kSortThreads * kSortBatch) {
        const int64_t i0 = t0 + threadIdx.x * kSortBatch;
        if (hi - lo > kSortThreads * kSortBatch) {  // (else as found above)
            h.begins = 0;
            if (i0 < hi) h = heads_at(i0);
        }
        uint32_t all;
        uint32_t seg = block_scan(__popc(h.begins), warp_sum, &all);
        // the segments that begin here go out through shared memory, in order
        uint32_t pos[kSortBatch];
        bool valid = i0 + kSortBatch <= hi;
#pragma unroll
        for (int u = 0; u < kSortBatch; ++u) {
            if ((h.begins >> u) & 1u) tile[seg++] = make_uint2(h.key[u], (uint32_t)(i0 + u));
            pos[u] = base + seg - 1u;
            valid &= i0 < hi && h.key[u] < rows;
        }
        if (valid) {
            uint4* p = reinterpret_cast<uint4*>(a.segpos + i0);
            p[0] = make_uint4(pos[0], pos[1], pos[2], pos[3]);
            p[1] = make_uint4(pos[4], pos[5], pos[6], pos[7]);
        } else if (i0 < hi) {
#pragma unroll
            for (int u = 0; u < kSortBatch; ++u)
                if (i0 + u < hi && h.key[u] < rows) a.segpos[i0 + u] = pos[u];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < (int)all; i += kSortThreads) {
            const uint2 x = tile[i];
            a.unique[base + i] = x.x;
            a.seg_start[base + i] = x.y;
        }
        __syncthreads();
        base += all;
    }
}

// The same sort for at most kSmallSort ids by one cluster of up to eight CTAs,
// kPer keys a thread: the keys move between the CTAs' shared memories, no pass
// touches global memory, and the cluster's barrier takes the grid's place.  (One
// block with eight keys a thread took 27 us for 8,192 ids, bound by its issue
// rate, a cluster with one 15.)
template <int kPer>
__global__ void __launch_bounds__(kSortThreads)
k_embed_sort_small(const EmbedSort a) {
    constexpr int kKeys = kSortThreads * kPer;  // of a CTA
    extern __shared__ uint32_t cnt[];           // [kSortWarps][bins], then pairs [2][kKeys]
    __shared__ uint32_t totals[512];
    __shared__ uint32_t warp_sum[kSortWarps];
    __shared__ uint32_t edge[3];  // first and last key, segments that begin here
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lt = (1u << lane) - 1u;
    const uint32_t rank = cluster_ctarank(), cs = gridDim.x;
    const int n = (int)a.n, bins = 1 << a.digit_bits;
    const uint32_t dmask = (uint32_t)bins - 1u, rows = (uint32_t)a.rows;
    uint2* const pairs = reinterpret_cast<uint2*>(cnt + kSortWarps * bins);
    pdl_wait();
    pdl_launch_dependents();
    const int own = warp * 32 * kPer + lane;  // this thread's first key within the CTA, then every 32nd
    uint2 kv[kPer];
    uint32_t same[kPer], at[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int i = (int)rank * kKeys + own + 32 * u;
        kv[u] = make_uint2(0xFFFFFFFFu, (uint32_t)i);  // keys beyond n are larger than any: they stay behind
        if (i < n) {
            const uint32_t id = a.ids[i];
            kv[u].x = min(id, rows);
            if (id >= rows && id != kMasked) atomicOr(a.err, kErrBounds);
        }
    }
    uint32_t* const mine = cnt + warp * bins;
    auto remote = [&](const uint32_t* p, uint32_t r) {
        uint32_t x;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(map_rank(smem_u32(p), r)) : "memory");
        return x;
    };
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.digit_bits, to = pass & 1;
        for (int x = lane; x < bins; x += 32) mine[x] = 0;
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const uint32_t d = (kv[u].x >> shift) & dmask;
            same[u] = same_digit(d, a.digit_bits, 0xFFFFFFFFu);
            at[u] = mine[d] + __popc(same[u] & lt);
            __syncwarp();
            if ((same[u] & lt) == 0u) mine[d] += __popc(same[u]);
            __syncwarp();
        }
        __syncthreads();
        const uint32_t total = scan_warps(cnt, bins);
        if ((int)threadIdx.x < bins) totals[threadIdx.x] = total;
        cluster_sync();
        uint32_t before = 0, sum = 0;
        if ((int)threadIdx.x < bins)
            for (uint32_t r = 0; r < cs; ++r) {
                const uint32_t c = remote(totals + threadIdx.x, r);
                sum += c;
                if (r < rank) before += c;
            }
        uint32_t all;
        const uint32_t base = block_scan(sum, warp_sum, &all);
        add_warps(cnt, bins, base + before);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const uint32_t p = at[u] + mine[(kv[u].x >> shift) & dmask];
            const uint32_t dst = map_rank(smem_u32(pairs + to * kKeys + (p & (kKeys - 1))), p / kKeys);
            asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(kv[u].x), "r"(kv[u].y)
                         : "memory");
        }
        cluster_sync();
#pragma unroll
        for (int u = 0; u < kPer; ++u) kv[u] = pairs[to * kKeys + own + 32 * u];
    }
    // the sorted pairs and the segments; here a thread takes kPer neighbours
    const uint2* const in = pairs + ((a.passes - 1) & 1) * kKeys;
    uint2* const out = a.passes & 1 ? a.pairs1 : a.pairs0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int i = (int)rank * kKeys + own + 32 * u;
        if (i < n) out[i] = kv[u];
    }
    if (threadIdx.x == 0) {
        edge[0] = in[0].x;
        edge[1] = in[kKeys - 1].x;
    }
    cluster_sync();
    const int j0 = (int)threadIdx.x * kPer, i0 = (int)rank * kKeys + j0;
    uint32_t key[kPer + 2];  // with the neighbours
    key[0] = j0 ? in[j0 - 1].x : rank ? remote(edge + 1, rank - 1) : rows;
    key[kPer + 1] = j0 + kPer < kKeys ? in[j0 + kPer].x : rank + 1 < cs ? remote(edge, rank + 1) : rows;
    uint32_t begins = 0;
#pragma unroll
    for (int u = 0; u < kPer; ++u) key[u + 1] = in[j0 + u].x;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
        if (i0 + u < n && key[u + 1] < rows && (i0 + u == 0 || key[u + 1] != key[u])) begins |= 1u << u;
    uint32_t here;
    uint32_t seg = block_scan(__popc(begins), warp_sum, &here);
    if (threadIdx.x == 0) edge[2] = here;
    cluster_sync();
    uint32_t all = 0;
    for (uint32_t r = 0; r < cs; ++r) {
        const uint32_t c = remote(edge + 2, r);
        all += c;
        if (r < rank) seg += c;
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int i = i0 + u;
        if (i >= n || key[u + 1] >= rows) continue;
        if ((begins >> u) & 1u) {
            a.unique[seg] = key[u + 1];
            a.seg_start[seg] = (uint32_t)i;
            ++seg;
        }
        a.segpos[i] = seg - 1u;
        if (i + 1 == n || key[u + 2] >= rows) {
            *a.n_valid = (uint32_t)(i + 1);
            a.seg_start[all] = (uint32_t)(i + 1);
        }
    }
    if (i0 == 0) {
        *a.count = all;
        if (all == 0) *a.n_valid = a.seg_start[0] = 0u;
    }
    cluster_sync();  // no CTA exits while another reads its shared memory
}

// ---- sums over the segments ---------------------------------------------------------------
// A chunk is rows_per_chunk consecutive places of the sorted order; a group of
// `lanes` threads sums one chunk's rows over 8 columns per thread, in order.  The
// chunk in which a segment begins finishes it where at most half a chunk of it
// lies beyond, and the next chunk starts after it.  A longer segment leaves one
// partial sum per chunk - the chunk's head (it began earlier) or tail (it begins
// here) - for k_embed_join, which adds them in order.  So no sum depends on the
// order in which blocks run, and a hot id's rows are spread over as many threads
// as a cold one's.
constexpr int kSumBatch = 8;  // rows loaded before they are added

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

// kC: copies, rounded up to 1, 2, 4 or 8.  Whether a segment crosses the chunk's
// ends is known from the places beside it, so finishing a segment loads nothing.
template <int kC>
__global__ void __launch_bounds__(256)
k_embed_sum(const EmbedSum a) {
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kPlaces = kSumBatch / kC;  // of a batch
    const int l = threadIdx.x % a.lanes;
    const int64_t work = ((int64_t)blockIdx.x * 256 + threadIdx.x) / a.lanes;
    const int64_t chunk = work / a.slices;
    const int col = ((int)(work - chunk * a.slices) * a.lanes + l) * 8;
    const int64_t nv = *a.n_valid;
    int64_t lo = chunk * a.rows_per_chunk, hi = min(lo + a.rows_per_chunk, nv);
    const int beyond = a.rows_per_chunk / 2;
    bool began_before = false, goes_on = false;
    uint32_t cur = 0u;
    if (lo < hi) {
        // (loads of neighbouring places and, where a segment crosses, its ends)
        cur = a.segpos[lo];
        const uint32_t tail = a.segpos[hi - 1];
        began_before = lo > 0 && a.segpos[lo - 1] == cur;
        goes_on = hi < nv && a.segpos[hi] == tail;
        if (goes_on) {
            const int64_t s0 = a.seg_start[tail], s1 = a.seg_start[tail + 1];
            if (s0 >= lo && s1 - hi <= beyond) {
                hi = s1;
                goes_on = false;
            }
        }
        if (began_before) {
            const int64_t s0 = a.seg_start[cur], s1 = a.seg_start[cur + 1];
            if (s0 >= lo - a.rows_per_chunk && s1 - lo <= beyond) {  // the chunk before finishes it
                lo = s1;
                ++cur;
                began_before = false;
            }
        }
    }
    // (a group beyond the last place, or a lane beyond dim, takes part in the
    // shuffles with nothing to add)
    const int count = (int)max((int64_t)0, hi - lo);
    const int most = __reduce_max_sync(0xFFFFFFFFu, count);  // of the warp's groups
    const bool in = count > 0 && col < a.dim;
    float acc[8] = {};
    auto flush = [&](bool ends) {
        if (in) {
            if (ends && !began_before)
                put_row(a, cur, col, acc);
            else
                store8_f32(a.partial + (2 * chunk + (began_before ? 0 : 1)) * a.dim + col, acc);
        }
        began_before = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    };
    // the group loads `lanes` places at a time, one per lane, the next ones while
    // these are added
    auto place = [&](int i, uint32_t& seg, uint32_t& row) {
        seg = row = 0u;
        if (i + l < count) {
            seg = a.segpos[lo + i + l];
            row = a.sorted[lo + i + l].y;
        }
    };
    uint32_t seg, row;
    place(0, seg, row);
    for (int i0 = 0; i0 < most; i0 += a.lanes) {
        uint32_t next_seg, next_row;
        place(i0 + a.lanes, next_seg, next_row);
        for (int j0 = 0; j0 < a.lanes; j0 += kPlaces) {
            uint4 v[kPlaces][kC];
#pragma unroll
            for (int u = 0; u < kPlaces; ++u) {
                const uint32_t r = __shfl_sync(0xFFFFFFFFu, row, j0 + u, a.lanes);
                if (in && i0 + j0 + u < count && j0 + u < a.lanes) {
                    const uint16_t* p = a.dout + (int64_t)r * a.copies * a.dim + col;
#pragma unroll
                    for (int c = 0; c < kC; ++c)
                        if (c < a.copies) v[u][c] = __ldcs(reinterpret_cast<const uint4*>(p + (int64_t)c * a.dim));
                }
            }
#pragma unroll
            for (int u = 0; u < kPlaces; ++u) {
                const uint32_t sg = __shfl_sync(0xFFFFFFFFu, seg, j0 + u, a.lanes);
                if (i0 + j0 + u < count && j0 + u < a.lanes) {
                    if (sg != cur) {
                        flush(true);
                        cur = sg;
                    }
#pragma unroll
                    for (int c = 0; c < kC; ++c)
                        if (c < a.copies) {
                            float f[8];
                            unpack8(v[u][c], f);
#pragma unroll
                            for (int j = 0; j < 8; ++j) acc[j] += f[j];
                        }
                }
            }
        }
        seg = next_seg;
        row = next_row;
    }
    if (count > 0) flush(!goes_on);
}

// The rows of the segments that left partial sums: the tail of the chunk in which
// one begins and the heads of the chunks after it, added in order.  A block looks
// for them in `look` chunks (at most kJoinMost), then each warp takes one after the other; one
// of more than kJoinAlone parts (a hot id) is added by the whole block, each warp
// a contiguous share, then the shares in order.
constexpr int kJoinMost = 64, kJoinAlone = 32;

__device__ __forceinline__ void add_parts(const EmbedSum& a, int64_t chunk, int64_t p0, int64_t p1, int col,
                                          float (&acc)[8]) {
    if (col >= a.dim) return;
#pragma unroll 8
    for (int64_t p = p0; p < p1; ++p) {
        float x[8];
        load8_f32(a.partial + (2 * (chunk + p) + (p == 0 ? 1 : 0)) * a.dim + col, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += x[j];
    }
}

__global__ void __launch_bounds__(256, 3)
k_embed_join(const EmbedSum a, int64_t chunks, int look) {
    pdl_wait();
    __shared__ float sm[8][32][9];
    __shared__ int parts_of[kJoinMost];
    __shared__ uint32_t seg_of[kJoinMost];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = ((int)blockIdx.y * 32 + lane) * 8;
    const int64_t first = (int64_t)blockIdx.x * look;
    if ((int)threadIdx.x < look) {
        const int64_t nv = *a.n_valid;
        const int64_t chunk = first + threadIdx.x;
        const int64_t lo = chunk * a.rows_per_chunk, hi = lo + a.rows_per_chunk;
        int parts = 0;
        uint32_t seg = 0;
        if (chunk < chunks - 1) {
            // (three independent loads; places past nv hold nothing)
            seg = a.segpos[hi - 1];
            const uint32_t next = a.segpos[hi];
            const uint32_t prev = lo ? a.segpos[lo - 1] : 0xFFFFFFFFu;
            if (hi < nv && next == seg && prev != seg) {
                const int64_t s1 = a.seg_start[seg + 1];
                if (s1 - hi > a.rows_per_chunk / 2)
                    parts = (int)((s1 - 1) / a.rows_per_chunk - chunk + 1);  // tail, heads
            }
        }
        parts_of[threadIdx.x] = parts;
        seg_of[threadIdx.x] = seg;
    }
    __syncthreads();
    for (int c = warp; c < look; c += 8) {
        const int parts = parts_of[c];
        if (parts == 0 || parts > kJoinAlone || col >= a.dim) continue;
        float acc[8] = {};
        add_parts(a, first + c, 0, parts, col, acc);
        put_row(a, seg_of[c], col, acc);
    }
    for (int c = 0; c < look; ++c) {
        const int64_t parts = parts_of[c];
        if (parts <= kJoinAlone) continue;
        float acc[8] = {};
        add_parts(a, first + c, parts * warp / 8, parts * (warp + 1) / 8, col, acc);
#pragma unroll
        for (int j = 0; j < 8; ++j) sm[warp][lane][j] = acc[j];
        __syncthreads();
        if (warp == 0 && col < a.dim) {
            for (int x = 1; x < 8; ++x)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += sm[x][lane][j];
            put_row(a, seg_of[c], col, acc);
        }
        __syncthreads();
    }
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

// ---- gate with checkpoint: geometries whose tokens do not fit the one-pass kernel ---------------
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
constexpr int kFusedSlots = 4;      // tokens between phase 1 and phase 2 at most 2
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

// Pairs of fp32 values.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpair(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float both(f32x2 v) {
    const float2 f = unpair(v);
    return f.x + f.y;
}
__device__ __forceinline__ void unpack8(uint4 v, f32x2 (&f)[4]) {
    f[0] = pair(bf16_lo(v.x), bf16_hi(v.x));
    f[1] = pair(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = pair(bf16_lo(v.z), bf16_hi(v.z));
    f[3] = pair(bf16_lo(v.w), bf16_hi(v.w));
}
__device__ __forceinline__ uint32_t pack2(f32x2 v) {
    const float2 f = unpair(v);
    return bf16x2_pack_rn(f.x, f.y);
}
__device__ __forceinline__ uint4 pack8(const f32x2 (&f)[4]) {
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
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
__global__ void __launch_bounds__((kFusedMaxWarps + 2) * 32, 1)
k_gate_backward_fused(const GateTrain a, int stages, int cs) {
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
        for (int i = 0; i <= n; ++i) {
            const bool image = i > 0 && a.windows[token(i - 1)].x == kDead;  // of phase 2's token
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
            if (i == 0) continue;
            const int p = i - 1, s = p % stages;
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
// turns the gates into hidden + g v from the stage.
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
__global__ void __launch_bounds__((kFusedMaxWarps + 2) * 32, 1)
k_gate_checkpoint_fused(const GateTrain a, int stages, int cs) {
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
        uint32_t id = n > 0 ? a.windows[token(0)].x : 0u, id_before = 0u;
        for (int i = 0; i <= n; ++i) {
            // slot 0 of the windows of the tokens in phases 1 and 2, the next one's on its way
            const bool img = id == kDead, image = id_before == kDead;
            id_before = id;
            if (i + 1 < n) id = a.windows[token(i + 1)].x;
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
            if (i == 0) continue;
            const int p = i - 1, s = p % stages;
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

// ---- two passes: geometries whose tokens do not fit ------------------------------------------
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
// bytes(cols) bytes; 0 if no cluster holds three stages of a token (one in each
// phase and one on its way).
template <class Bytes>
int one_pass_cluster(int d, Bytes bytes, int* stages) {
    const int groups = d / 256;
    for (int cs = 1; cs <= 8 && cs <= groups; cs *= 2) {
        const int per = (groups + cs - 1) / cs;
        const int n = (227 * 1024 - kFusedFixed - 128) / bytes(per * 256);
        if (per <= kFusedMaxWarps && n >= 3) {
            *stages = std::min(n, 6);
            return cs;
        }
    }
    return 0;
}

template <class F>
cudaError_t one_pass_launch(F kern, const GateTrain& a, int cs, int stages, int stage_bytes, int* clusters,
                            cudaStream_t s) {
    const int per = (a.d / 256 + cs - 1) / cs;
    const int smem = (kFusedFixed + 127) / 128 * 128 + stages * stage_bytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    *clusters = (int)std::min<int64_t>(a.T, device_sm_count() / cs);
    cfg.gridDim = dim3(*clusters * cs);
    cfg.blockDim = dim3((per + 2) * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, stages, cs);
}

template <int kSaved, int kHc>
cudaError_t fused_launch(const GateTrain& a, int cs, int stages, int* shares, cudaStream_t s) {
    const int bytes = fused_stage_bytes<kSaved>(a.hc, (a.d / 256 + cs - 1) / cs * 256);
    return a.hc == kHc ? one_pass_launch(k_gate_backward_fused<kSaved, kHc, true>, a, cs, stages, bytes, shares, s)
                       : one_pass_launch(k_gate_backward_fused<kSaved, kHc, false>, a, cs, stages, bytes, shares, s);
}

template <bool kF32Kv, int kHc>
cudaError_t ckpt_launch(const GateTrain& a, int cs, int stages, cudaStream_t s) {
    const int bytes = ckpt_stage_bytes<kF32Kv>(a.hc, (a.d / 256 + cs - 1) / cs * 256);
    int clusters;
    return a.hc == kHc
               ? one_pass_launch(k_gate_checkpoint_fused<kF32Kv, kHc, true>, a, cs, stages, bytes, &clusters, s)
               : one_pass_launch(k_gate_checkpoint_fused<kF32Kv, kHc, false>, a, cs, stages, bytes, &clusters, s);
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

// A block per 1,024 keys, a key per thread, until every SM has one.
int embed_sort_blocks(int64_t n) {
    return (int)std::min<int64_t>(device_sm_count(), std::max<int64_t>(1, (n + kSortThreads - 1) / kSortThreads));
}

void embed_sort_digits(uint64_t rows, int* passes, int* bits) {
    int need = 1;
    while (need < 32 && (rows >> need)) ++need;  // the largest key is `rows`
    *passes = (need + 8) / 9;
    *bits = (need + *passes - 1) / *passes;
}

cudaError_t launch_embed_sort(const EmbedSort& a, cudaStream_t s) {
    if (a.n <= kSmallSort) {
        const int per = a.n <= kSortThreads * 8 ? 1 : a.n <= kSortThreads * 16 ? 2 : 4;
        auto f = per == 1 ? k_embed_sort_small<1> : per == 2 ? k_embed_sort_small<2> : k_embed_sort_small<4>;
        const int smem = kSortWarps * (1 << a.digit_bits) * 4 + 2 * kSortThreads * per * 8;
        cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        unsigned cs = 1;
        while (cs * kSortThreads * per < a.n) cs *= 2;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cs;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.gridDim = dim3(cs);
        cfg.blockDim = dim3(kSortThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        return cudaLaunchKernelEx(&cfg, f, a);
    }
    const int blocks = embed_sort_blocks(a.n);
    const int smem = kSortWarps * (1 << a.digit_bits) * 4 + kSortThreads * kSortBatch * 8;
    cudaError_t e = cudaFuncSetAttribute(k_embed_sort, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaMemsetAsync(a.barrier, 0, 4, s);
    if (e != cudaSuccess) return e;
    EmbedSort copy = a;
    void* args[] = {&copy};
    return cudaLaunchCooperativeKernel((void*)k_embed_sort, dim3(blocks), dim3(kSortThreads), args, smem, s);
}

// Sorted places per chunk: 64 rows of dout (a chunk's two partial rows are then
// a few percent of what it reads), fewer while the chunks do not fill the GPU
// four times over.
int embed_rows_per_chunk(int64_t n, int dim, int copies) {
    const int64_t lanes = 1 << std::min(5, log2_ceil(dim / 8));
    const int64_t slices = (dim / 8 + lanes - 1) / lanes;
    int r = 64 / copies;
    while (r > 4 && n / r * slices * lanes < (int64_t)device_sm_count() * 4 * 768) r /= 2;
    return r;
}

cudaError_t launch_embed_sum(EmbedSum a, int64_t n, cudaStream_t s) {
    a.lanes = 1 << std::min(5, log2_ceil(a.dim / 8));
    a.slices = (a.dim / 8 + a.lanes - 1) / a.lanes;
    const int64_t chunks = (n + a.rows_per_chunk - 1) / a.rows_per_chunk;
    const int64_t threads = chunks * a.slices * a.lanes;
    auto f = a.copies == 1   ? k_embed_sum<1>
             : a.copies == 2 ? k_embed_sum<2>
             : a.copies <= 4 ? k_embed_sum<4>
                             : k_embed_sum<8>;
    cudaError_t e = pdl_launch(f, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a);
    if (e != cudaSuccess || chunks < 2) return e;
    // about four blocks per SM
    const int64_t slices = (a.dim + 255) / 256, want = chunks * slices / (device_sm_count() * 4) + 1;
    const int look = (int)std::min<int64_t>(kJoinMost, std::max<int64_t>(8, want));
    return pdl_launch(k_embed_join, dim3((unsigned)((chunks + look - 1) / look), (unsigned)slices), dim3(256), 0, s,
                      a, chunks, look);
}

cudaError_t launch_gate_checkpoint(const GateTrain& a, bool kv_f32, cudaStream_t s) {
    return kv_f32 ? gate_checkpoint<true>(a, s) : gate_checkpoint<false>(a, s);
}

int gate_backward_shares(int64_t T, int d) {
    const int blocks = (d / 8 + 127) / 128;
    // (the fused kernel's clusters are no more than the SMs)
    return (int)std::max<int64_t>(1, std::min<int64_t>(T, device_sm_count() * std::max(1, 4 / blocks)));
}

cudaError_t launch_gate_backward(const GateTrain& a, int saved, cudaStream_t s) {
    if (saved == kSavedMx) return gate_backward<kSavedMx>(a, s);
    if (saved == kSavedF32) return gate_backward<kSavedF32>(a, s);
    return gate_backward<kSavedBf16>(a, s);
}

}  // namespace engram
