// The scaled embedding lookup and its gradient by sorted ids (sm_103a).
//
//   out[t][c] = s W[id_t]                     c < copies
//   dW[v] = s sum_{t: id_t = v} sum_c dout[t][c]
//
// Both are bound by memory: the lookup by writing out, the gradient by reading
// dout once, in the order of the sorted ids, and writing a row per distinct id.
// The gradient is a sort of (id, position) with its segments of equal ids, the
// sums over chunks of the sorted order, and the joins of the segments that are
// longer than a chunk: no atomics on values, so the same sums on every run.
// Measured (GB300, copy bandwidth 6.77 TB/s): 8,192 tokens x 4 branches x 5,120:
// 100 us - sort 15, sums 74 (5.6 TB/s), joins 14 (cold caches); 50,032 x 24 rows
// of 256 from 64 million: 271 us - sort 66, sums 181 (5.8 TB/s), joins 21.  Past
// 8,192 keys a block (1,245,184 ids on 152 SMs) the sort reads every key twice a
// pass: 1,244,000 ids 279 us, 1,246,000 340.
#include <algorithm>

#include "grad_internal.h"
#include "per_device.h"
#include "tcgen05_common.cuh"
#include "train_common.cuh"

namespace engram {

namespace {

// ---- embedding ----------------------------------------------------------------------
// out[t][c] = scale table[ids[t]], c < copies, rounded once to BF16.  A group of
// `lanes` threads takes one id, 8 columns per thread and step, and writes every
// copy of what it read, so the table row is read once.  50,032 ids x 4 copies x
// 5,120 BF16: 345 us, 95% of the copy bandwidth.
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
// work between them; the wait is bounded: false on a time-out.  The block's barrier
// orders its writes before the release, and the acquire before what it reads next.
// A block whose wait ran out leaves the sort unfinished: it says so in *a.failed, and
// the kernels behind the sort, whose loops and addresses come from its results, then
// take it that there are no ids.
__device__ __forceinline__ void grid_arrive(const EmbedSort& a) {
    __syncthreads();
    const bool starved = a.starve && blockIdx.x + 1 == gridDim.x;
    if (threadIdx.x == 0 && !starved)
        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.barrier) : "memory");
}
__device__ __forceinline__ bool grid_wait(const EmbedSort& a, uint32_t& phase, int* flag) {
    if (threadIdx.x == 0) {
        const uint32_t want = ++phase * gridDim.x;
        const uint64_t t0 = globaltimer();
        uint32_t spin = 0;
        while (ld_acquire_u32(a.barrier) < want) {
            if ((++spin & 63u) == 0u && (long long)(globaltimer() - t0) > a.wait_limit_ns) {
                atomicOr(a.err, kErrTimeout);
                *a.failed = 1u;
                *flag = 1;
                break;
            }
        }
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
        *a.failed = 0u;  // (no wait of this kernel is bounded)
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

// Ids that are rows; none if the sort did not finish.
__device__ __forceinline__ int64_t valid_ids(const EmbedSum& a) {
    const uint32_t n = *a.n_valid, failed = *a.failed;
    return failed ? 0 : n;
}

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
    const int64_t nv = valid_ids(a);
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
// for them in `look` chunks (at most kJoinMost), then each group of kLanes threads
// (as many as a row has columns by eight, 32 at most) takes one after the other;
// one of more than kJoinAlone parts (a hot id) is added by the whole block, each
// group a contiguous share, then the shares in order.  (3 million rows of 8
// columns, 200,000 ids: 484 us with whole warps as groups, 391 so; at 50,032 x 24
// rows of 256 a group's size known only at run time costs 4 us of 271.)
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

template <int kLanes>
__global__ void __launch_bounds__(256, 3)
k_embed_join(const EmbedSum a, int64_t chunks, int look) {
    constexpr int kGroups = 256 / kLanes;
    __shared__ float sm[kGroups][kLanes][9];
    __shared__ int parts_of[kJoinMost];
    __shared__ uint32_t seg_of[kJoinMost];
    const int lane = threadIdx.x % kLanes, g = threadIdx.x / kLanes;
    const int col = ((int)blockIdx.y * kLanes + lane) * 8;
    const int64_t first = (int64_t)blockIdx.x * look;
    if ((int)threadIdx.x < look) {
        const int64_t nv = valid_ids(a);
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
    pdl_wait();  // for the sums; the places were there before their kernel's blocks began
    for (int c = g; c < look; c += kGroups) {
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
        add_parts(a, first + c, parts * g / kGroups, parts * (g + 1) / kGroups, col, acc);
#pragma unroll
        for (int j = 0; j < 8; ++j) sm[g][lane][j] = acc[j];
        __syncthreads();
        if (g == 0 && col < a.dim) {
#pragma unroll 8
            for (int x = 1; x < kGroups; ++x)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += sm[x][lane][j];
            put_row(a, seg_of[c], col, acc);
        }
        __syncthreads();
    }
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

// Shared memory for digits of `bits` bits and `keys` pairs.
static int embed_sort_smem(int bits, int keys) { return kSortWarps * (1 << bits) * 4 + keys * 8; }

cudaError_t launch_embed_sort(const EmbedSort& a, cudaStream_t s) {
    if (a.n <= kSmallSort) {
        static PerDevice allowed[3];
        const int size = a.n <= kSortThreads * 8 ? 0 : a.n <= kSortThreads * 16 ? 1 : 2, per = 1 << size;
        auto f = per == 1 ? k_embed_sort_small<1> : per == 2 ? k_embed_sort_small<2> : k_embed_sort_small<4>;
        const int keys = 2 * kSortThreads * per, smem = embed_sort_smem(a.digit_bits, keys);
        const cudaError_t e = allow_shared(allowed[size], f, embed_sort_smem(9, keys));
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
    static PerDevice allowed;
    const int keys = kSortThreads * kSortBatch, smem = embed_sort_smem(a.digit_bits, keys);
    cudaError_t e = allow_shared(allowed, k_embed_sort, embed_sort_smem(9, keys));
    if (e == cudaSuccess) e = cudaMemsetAsync(a.barrier, 0, 8, s);  // with *a.failed
    if (e != cudaSuccess) return e;
    EmbedSort copy = a;
    void* args[] = {&copy};
    return cudaLaunchCooperativeKernel((void*)k_embed_sort, dim3(blocks), dim3(kSortThreads), args, smem, s);
}

// Chunks that fill the GPU four times over.
static int64_t embed_chunks_wanted(int dim) {
    const int64_t lanes = 1 << std::min(5, log2_ceil(dim / 8));
    const int64_t slices = (dim / 8 + lanes - 1) / lanes;
    return ((int64_t)device_sm_count() * 4 * 768 + slices * lanes - 1) / (slices * lanes);
}

// Sorted places per chunk: 64 rows of dout (a chunk's two partial rows are then
// a few percent of what it reads), fewer while the chunks do not fill the GPU
// four times over.
int embed_rows_per_chunk(int64_t n, int dim, int copies) {
    const int64_t want = embed_chunks_wanted(dim);
    int r = 64 / copies;
    while (r > 4 && n / r < want) r /= 2;
    return r;
}

// Where chunks of r places are too few, r is halved: so 2 r places make a chunk of
// the most ids at which half as many chunks were still too few.
int64_t embed_most_chunks(int64_t n, int dim) {
    const int64_t want = embed_chunks_wanted(dim);
    int64_t most = 0;
    for (int copies = 1; copies <= 8; ++copies) {
        int64_t upto = n;  // ids that chunks of r places take at most
        for (int r = 64 / copies;; r /= 2) {
            most = std::max(most, (upto + r - 1) / r);
            if (r <= 4) break;
            upto = std::min(upto, want * r - 1);
        }
    }
    return most;
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
    const int64_t slices = a.slices, want = chunks * slices / (device_sm_count() * 4) + 1;
    const int look = (int)std::min<int64_t>(kJoinMost, std::max<int64_t>(8, want));
    auto join = a.lanes == 32   ? k_embed_join<32>
                : a.lanes == 16 ? k_embed_join<16>
                : a.lanes == 8  ? k_embed_join<8>
                : a.lanes == 4  ? k_embed_join<4>
                : a.lanes == 2  ? k_embed_join<2>
                                : k_embed_join<1>;
    return pdl_launch(join, dim3((unsigned)((chunks + look - 1) / look), (unsigned)slices), dim3(256), 0, s,
                      a, chunks, look);
}

}  // namespace engram
