// Root-mean-square norm of a residual stream and its backward pass (sm_103a).
//
//   s = scale sum_c x[t][c] + residual[t],  r = 1 / sqrt(mean s^2 + eps),  y = s r w
//   u = w dy,  ds = r u - s r^3 mean(u s) + dsum,  dx[c] = scale ds,  dw = sum_t dy s r
//
// Both are bound by memory: every value is read once, stays in registers or shared memory
// between the sum over its row and its use, and is written once.  A short row belongs to a
// power-of-two group of lanes of one warp (sums by shuffles alone), a longer one to a block
// (forward from 257 values on: 100,000 rows of 1,024 take 121 us, in lanes 175; backward
// from 1,025 on, whose shares of dw cost a block more).  Where a block has several long
// rows, the next ones are on their way to shared memory while it works on one: the sum
// over a row is a wait for all of its values, which otherwise leaves HBM idle (8,192 rows
// of 4 x 5,120: 78 us, 124 without).  Sums are fp32.
//
// Measured, against the bytes at a copy's 6.79 TB/s: 50,032 x 5,120 BF16 with residual
// 298 us (1.01), 20,000 rows to 8 bits 113 (0.94), 2,048 rows of 4 branches 19 (0.97),
// backward 8,192 rows into 4 branches 95 (0.92), 16,000 rows into one 109 (0.89), 256 rows
// to 8 bits 3.4 (0.4: latency).  The backward pass is held back by its rows' chain of sum,
// barrier and second use: a block has one row, or a pair, in work at a time.
#include <algorithm>

#include "mx8.cuh"
#include "per_device.h"
#include "train_common.cuh"
#include "update_internal.h"

namespace engram {

namespace {

constexpr int kGroupThreads = 256;  // block of the kernels whose rows belong to lanes
// most threads of a block that a row belongs to
constexpr int row_threads(int vec, bool lean) { return vec == 1 || (vec == 2 && lean) ? 1024 : 512; }

// Eight values of a stream of either type.
template <bool kF32>
struct Eight {
    uint4 q[kF32 ? 2 : 1];
    __device__ __forceinline__ void load(const void* p, size_t at) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * (kF32 ? 4 : 2));
#pragma unroll
        for (int j = 0; j < (kF32 ? 2 : 1); ++j) q[j] = src[j];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < (kF32 ? 2 : 1); ++j) q[j] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(f32x2 (&f)[4]) const {
        if (kF32) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint4 v = q[kF32 ? j : 0];
                f[2 * j] = pair(__uint_as_float(v.x), __uint_as_float(v.y));
                f[2 * j + 1] = pair(__uint_as_float(v.z), __uint_as_float(v.w));
            }
        } else {
            unpack8(q[0], f);
        }
    }
};
template <bool kF32>
__device__ __forceinline__ void store8(void* p, size_t at, const f32x2 (&f)[4]) {
    if (kF32)
        store8_f32(static_cast<float*>(p) + at, f);
    else
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at), pack8(f));
}

// A block's row of a stream in shared memory, 8 values at a time: a thread sends for 16-byte
// pieces and reads its own 8 values back.  BF16: one piece, its own.  fp32: two, and 32
// neighbouring threads share their copies so that an instruction covers whole sectors; the
// pieces are swapped within 128 bytes so that the reads do not meet in a bank.
template <bool kF32>
struct Row {
    __device__ static __forceinline__ int at(int piece) { return piece ^ (piece >> 3 & 1); }
    __host__ __device__ static int pieces(int V) { return kF32 ? (V + 31) / 32 * 64 : V; }
    // v: this thread's vector of 8
    __device__ static __forceinline__ void send(uint4* s, const void* row, int v, int V) {
        if (kF32) {
            const int first = v & ~31, lane = v & 31;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int piece = 32 * j + lane;
                if (first + piece / 2 < V)
                    async16(s + 2 * first + at(piece), static_cast<const float*>(row) + (2 * first + piece) * 4);
            }
        } else if (v < V) {
            async16(s + v, static_cast<const uint16_t*>(row) + v * 8);
        }
    }
    __device__ static __forceinline__ Eight<kF32> get(const uint4* s, int v) {
        Eight<kF32> e;
        if (kF32) {
            const int first = v & ~31, lane = v & 31;
#pragma unroll
            for (int j = 0; j < 2; ++j) e.q[kF32 ? j : 0] = s[2 * first + at(2 * lane + j)];
        } else {
            e.q[0] = s[v];
        }
        return e;
    }
};

// Sums over the threads of a row.  kWarp: over groups of `lanes` lanes.  Otherwise over
// the block; `parity` changes from row to row, so that one barrier does.
template <bool kWarp, int kN>
__device__ __forceinline__ void row_sum(float (&v)[kN], int lanes, float (*sm)[32][kN], int parity) {
    if (kWarp) {
        for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < kN; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
        if (lane == 0) sm[parity][warp][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        float s = lane < warps ? sm[parity][lane][k] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        v[k] = s;
    }
}

// 1 / sqrt(x), the approximation (2 units in the last place) mended by a step of Newton's: a
// whole row is multiplied by it.
__device__ __forceinline__ float inverse_root(float x) {
    const float r = rsqrtf(x);
    return x < 3e38f ? fmaf(0.5f * r, fmaf(-x * r, r, 1.0f), r) : r;  // (0 where x is infinite)
}

// Where a thread stands: its group's first row, the rows between two of its rows, its
// place in the row.
struct Place {
    int64_t row, step;
    int lane, lanes;
};
template <bool kWarp>
__device__ __forceinline__ Place place(int lanes) {
    if (!kWarp) return {(int64_t)blockIdx.x, (int64_t)gridDim.x, (int)threadIdx.x, (int)blockDim.x};
    const int groups = kGroupThreads / lanes;
    return {(int64_t)blockIdx.x * groups + threadIdx.x / lanes, (int64_t)gridDim.x * groups,
            (int)threadIdx.x & (lanes - 1), lanes};
}
// Whether any lane of this warp has a row (in a warp of several rows the first one's row
// is the lowest).
template <bool kWarp>
__device__ __forceinline__ bool any_row(int64_t row, const Place& p, int64_t n) {
    return (kWarp ? row - (int)(threadIdx.x & 31) / p.lanes : row) < n;
}

// kStages: stages of shared memory, or 0: rows are loaded when they are worked on.
template <int kVec, bool kWarp, bool kF32, bool kMx, int kStages>
__global__ void __launch_bounds__(kWarp ? kGroupThreads : row_threads(kVec, !kF32)) k_norm(NormArgs a) {
    __shared__ float sm[2][32][1];
    extern __shared__ uint4 stages[];  // [kStages][copies and residual][Row pieces]
    pdl_launch_dependents();
    const Place p = place<kWarp>(a.lanes);
    const int V = a.dim / 8;
    const int pieces = Row<kF32>::pieces(V), stage_size = pieces * (a.copies + (a.residual != nullptr));
    const size_t row_bytes = (size_t)a.dim * (kF32 ? 4 : 2);
    pdl_wait();
    f32x2 w[kVec > 2 ? 1 : kVec][4];
    if (kVec <= 2) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (p.lane + i * p.lanes < V) load8_f32(a.weight + (p.lane + i * p.lanes) * 8, w[kVec > 2 ? 0 : i]);
    }
    const float inv_dim = 1.0f / (float)a.dim;
    auto send = [&](int64_t row, int stage) {
        if (row < a.n) {
            uint4* s = stages + stage * stage_size;
            const char* x = static_cast<const char*>(a.x) + (size_t)row * a.copies * row_bytes;
            for (int c = 0; c < a.copies; ++c)
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    Row<kF32>::send(s + c * pieces, x + c * row_bytes, p.lane + i * p.lanes, V);
            if (a.residual)
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    Row<kF32>::send(s + a.copies * pieces, static_cast<const char*>(a.residual) + row * row_bytes,
                                    p.lane + i * p.lanes, V);
        }
        async_commit();
    };
    int parity = 0, stage = 0, free = kStages - 1;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) send(p.row + k * p.step, k);
    for (int64_t row = p.row; any_row<kWarp>(row, p, a.n); row += p.step, parity ^= 1) {
        const bool mine = !kWarp || row < a.n;
        const uint4* s_row = stages + stage * stage_size;
        if (kStages) {
            if (kF32) __syncwarp();  // what the stage held has been read
            send(row + (kStages - 1) * p.step, free);
            async_wait<kStages ? kStages - 1 : 0>();
            if (kF32) __syncwarp();
            stage = stage + 1 == kStages ? 0 : stage + 1;
            free = free + 1 == kStages ? 0 : free + 1;
        }
        f32x2 s[kVec][4];
#pragma unroll
        for (int i = 0; i < kVec; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = 0;
        Eight<kF32> res[kVec];
        if (!kStages && a.residual) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = p.lane + i * p.lanes;
                if (mine && v < V) res[i].load(a.residual, (size_t)row * a.dim + v * 8);
            }
        }
#pragma unroll 4
        for (int c = 0; c < a.copies; ++c) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = p.lane + i * p.lanes;
                if (mine && v < V) {
                    Eight<kF32> x;
                    f32x2 f[4];
                    if (kStages)
                        x = Row<kF32>::get(s_row + c * pieces, v);
                    else
                        x.load(a.x, ((size_t)row * a.copies + c) * a.dim + v * 8);
                    x.get(f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] = add2(s[i][j], f[j]);
                }
            }
        }
        const f32x2 scale = twice(a.scale);
        f32x2 squares[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = p.lane + i * p.lanes;
            if (mine && v < V) {
                f32x2 f[4] = {0, 0, 0, 0};
                if (a.residual) {
                    if (kStages) res[i] = Row<kF32>::get(s_row + a.copies * pieces, v);
                    res[i].get(f);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = fma2(s[i][j], scale, f[j]);
                    squares[j & 1] = fma2(s[i][j], s[i][j], squares[j & 1]);
                }
            }
        }
        float total[1] = {both(add2(squares[0], squares[1]))};
        row_sum<kWarp>(total, p.lanes, sm, parity);
        const float r = inverse_root(fmaf(total[0], inv_dim, a.eps));
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = p.lane + i * p.lanes;
            const bool valid = mine && v < V;
            const size_t at = (size_t)row * a.dim + v * 8;
            f32x2 y[4] = {0, 0, 0, 0};
            if (kVec > 2 && valid) load8_f32(a.weight + v * 8, w[0]);
            if (valid)
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = mul2(mul2(s[i][j], twice(r)), w[kVec > 2 ? 0 : i][j]);
            if (valid && a.sum) store8<kF32>(a.sum, at, s[i]);
            if (kMx) {
                uint32_t e;
                const uint2 codes = encode_mx8_pairs(y, e);
                if (valid) {
                    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + at), codes);
                    if (!(v & 3)) a.y_scales[at / 32] = (uint8_t)e;
                }
            } else if (valid) {
                store8<false>(a.y, at, y);
            }
        }
    }
}

// A row's backward pass, of one vector of 8: its part of the two sums, and, with them, ds and
// the vector's share of dw.
__device__ __forceinline__ void back_sums(const f32x2 (&f)[4], const f32x2 (&g)[4], const f32x2 (&w)[4],
                                          f32x2& squares, f32x2& dots) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        squares = fma2(f[j], f[j], squares);
        dots = fma2(mul2(f[j], g[j]), w[j], dots);
    }
}
__device__ __forceinline__ void back_step(const f32x2 (&f)[4], const f32x2 (&g)[4], const f32x2 (&w)[4], float r,
                                          float c, f32x2 (&ds)[4], f32x2 (&dw)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x2 gr = mul2(g[j], twice(r));
        ds[j] = fma2(gr, w[j], fma2(twice(-c), f[j], ds[j]));
        dw[j] = fma2(gr, f[j], dw[j]);
    }
}
// ds to dresidual and, scaled, to every copy of dx: 8 values at `res` and `dx`.
template <bool kF32>
__device__ __forceinline__ void back_store(const NormBackArgs& a, char* res, char* dx, f32x2 (&ds)[4]) {
    if (a.dresidual) store8<kF32>(res, 0, ds);
    if (a.dx) {
#pragma unroll
        for (int j = 0; j < 4; ++j) ds[j] = mul2(ds[j], twice(a.scale));
        const uint32_t copy_bytes = a.dim * (kF32 ? 4 : 2);
        for (int k = 0; k < a.copies; ++k, dx += copy_bytes) store8<kF32>(dx, 0, ds);
    }
}

// A block's rows, loaded when they are worked on; its share of the weights' gradient goes to
// part[block].
template <int kVec, bool kWarp, bool kF32>
__global__ void __launch_bounds__(kWarp ? kGroupThreads : row_threads(kVec, false)) k_norm_backward(NormBackArgs a) {
    __shared__ float sm[2][32][2];
    extern __shared__ __align__(16) float dw_groups[];  // kWarp: [groups][lanes kVec 8], the groups' shares of dw
    constexpr int kBytes = kF32 ? 4 : 2;
    pdl_launch_dependents();
    const Place p = place<kWarp>(a.lanes);
    const int V = a.dim / 8;
    pdl_wait();
    f32x2 w[kVec > 2 ? 1 : kVec][4], dw[kVec][4];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (kVec <= 2 && p.lane + i * p.lanes < V) load8_f32(a.weight + (p.lane + i * p.lanes) * 8, w[kVec > 2 ? 0 : i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[i][j] = 0;
    }
    const float inv_dim = 1.0f / (float)a.dim;
    int parity = 0;
    for (int64_t row = p.row; any_row<kWarp>(row, p, a.n); row += p.step, parity ^= 1) {
        const bool mine = !kWarp || row < a.n;
        Eight<kF32> s[kVec], more[kVec];
        Eight<false> dy[kVec];
        f32x2 squares = 0, dots = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = p.lane + i * p.lanes;
            more[i].zero();
            if (!mine || v >= V) continue;
            const size_t at = (size_t)row * a.dim + v * 8;
            s[i].load(a.sum, at);
            dy[i].load(a.dy, at);
            if (a.dsum) more[i].load(a.dsum, at);
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = p.lane + i * p.lanes;
            if (!mine || v >= V) continue;
            f32x2 f[4], g[4];
            s[i].get(f);
            dy[i].get(g);
            if (kVec > 2) load8_f32(a.weight + v * 8, w[0]);
            back_sums(f, g, w[kVec > 2 ? 0 : i], squares, dots);
        }
        float total[2] = {both(squares), both(dots)};
        row_sum<kWarp>(total, p.lanes, sm, parity);
        const float r = inverse_root(fmaf(total[0], inv_dim, a.eps));
        const float c = total[1] * inv_dim * r * r * r;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            const int v = p.lane + i * p.lanes;
            if (!mine || v >= V) continue;
            f32x2 f[4], g[4], ds[4];
            s[i].get(f);
            dy[i].get(g);
            more[i].get(ds);
            if (kVec > 2) load8_f32(a.weight + v * 8, w[0]);
            back_step(f, g, w[kVec > 2 ? 0 : i], r, c, ds, dw[i]);
            const size_t at = (size_t)row * a.dim + v * 8, at_dx = (size_t)row * a.copies * a.dim + v * 8;
            back_store<kF32>(a, static_cast<char*>(a.dresidual) + at * kBytes,
                             static_cast<char*>(a.dx) + at_dx * kBytes, ds);
        }
    }
    if (!a.dweight) return;
    float* part = a.part + (size_t)blockIdx.x * a.dim;
    if (!kWarp) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (p.lane + i * p.lanes < V) store8_f32(part + (p.lane + i * p.lanes) * 8, dw[i]);
        return;
    }
    const int wide = p.lanes * kVec * 8, group = threadIdx.x / p.lanes;
#pragma unroll
    for (int i = 0; i < kVec; ++i) store8_f32(dw_groups + group * wide + (p.lane + i * p.lanes) * 8, dw[i]);
    __syncthreads();
    for (int col = threadIdx.x; col < a.dim; col += kGroupThreads) {
        float t = 0.f;
        for (int g = 0; g < kGroupThreads / p.lanes; ++g) t += dw_groups[g * wide + col];
        part[col] = t;
    }
}

// Of many rows: kRows neighbouring ones at a time, one barrier for their sums, the next ones
// on their way to shared memory.  A row's values are read there again where they are used.
template <int kVec, bool kF32, int kRows, int kStages>
__global__ void __launch_bounds__(row_threads(kVec, false)) k_norm_backward_staged(NormBackArgs a) {
    __shared__ float sm[2][32][2 * kRows];
    extern __shared__ uint4 stages[];  // [kStages][kRows][sum, dsum, dy pieces]
    constexpr int kBytes = kF32 ? 4 : 2;
    pdl_launch_dependents();
    const int V = a.dim / 8, threads = blockDim.x, me = threadIdx.x;
    const int pieces = Row<kF32>::pieces(V), row_size = pieces * (1 + (a.dsum != nullptr)) + V;
    pdl_wait();
    f32x2 w[kVec > 2 ? 1 : kVec][4], dw[kVec][4];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        if (kVec <= 2 && me + i * threads < V) load8_f32(a.weight + (me + i * threads) * 8, w[kVec > 2 ? 0 : i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[i][j] = 0;
    }
    const float inv_dim = 1.0f / (float)a.dim;
    // addresses only grow: `hop` values from one of this block's groups of rows to the next
    const int64_t step = (int64_t)gridDim.x * kRows;
    const size_t hop = (size_t)step * a.dim, begin = (size_t)blockIdx.x * kRows * a.dim;
    const char* in_sum = static_cast<const char*>(a.sum) + begin * kBytes;
    const char* in_dsum = static_cast<const char*>(a.dsum) + begin * kBytes;
    const char* in_dy = reinterpret_cast<const char*>(a.dy) + begin * 2;
    int64_t in_row = (int64_t)blockIdx.x * kRows;
    auto send = [&](int stage) {
        uint4* s = stages + stage * kRows * row_size;
#pragma unroll
        for (int q = 0; q < kRows; ++q, s += row_size) {
            if (in_row + q >= a.n) continue;
            const size_t off = (size_t)q * a.dim;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = me + i * threads;
                Row<kF32>::send(s, in_sum + off * kBytes, v, V);
                if (a.dsum) Row<kF32>::send(s + pieces, in_dsum + off * kBytes, v, V);
                Row<false>::send(s + row_size - V, in_dy + off * 2, v, V);
            }
        }
        async_commit();
        in_row += step;
        in_sum += hop * kBytes;
        in_dsum += hop * kBytes;
        in_dy += hop * 2;
    };
    char* out_dx = static_cast<char*>(a.dx) + begin * a.copies * kBytes + me * (8 * kBytes);
    char* out_dres = static_cast<char*>(a.dresidual) + begin * kBytes + me * (8 * kBytes);
    int parity = 0, stage = 0, free = kStages - 1;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) send(k);
    for (int64_t row = (int64_t)blockIdx.x * kRows; row < a.n; row += step, parity ^= 1) {
        const uint4* s_rows = stages + stage * kRows * row_size;
        if (kF32) __syncwarp();  // what the stage held has been read
        send(free);
        async_wait<kStages - 1>();
        if (kF32) __syncwarp();
        stage = stage + 1 == kStages ? 0 : stage + 1;
        free = free + 1 == kStages ? 0 : free + 1;
        float total[2 * kRows];
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            const uint4* s = s_rows + q * row_size;
            f32x2 squares = 0, dots = 0;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = me + i * threads;
                if (v >= V || row + q >= a.n) continue;
                f32x2 f[4], g[4];
                Row<kF32>::get(s, v).get(f);
                Row<false>::get(s + row_size - V, v).get(g);
                if (kVec > 2) load8_f32(a.weight + v * 8, w[0]);
                back_sums(f, g, w[kVec > 2 ? 0 : i], squares, dots);
            }
            total[2 * q] = both(squares);
            total[2 * q + 1] = both(dots);
        }
        row_sum<false>(total, threads, sm, parity);
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            if (row + q >= a.n) continue;
            const uint4* s = s_rows + q * row_size;
            const float r = inverse_root(fmaf(total[2 * q], inv_dim, a.eps));
            const float c = total[2 * q + 1] * inv_dim * r * r * r;
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const int v = me + i * threads;
                if (v >= V) continue;
                f32x2 f[4], g[4], ds[4] = {0, 0, 0, 0};
                Row<kF32>::get(s, v).get(f);
                Row<false>::get(s + row_size - V, v).get(g);
                if (a.dsum) Row<kF32>::get(s + pieces, v).get(ds);
                if (kVec > 2) load8_f32(a.weight + v * 8, w[0]);
                back_step(f, g, w[kVec > 2 ? 0 : i], r, c, ds, dw[i]);
                const size_t off = (size_t)q * a.dim * kBytes + i * threads * (8 * kBytes);
                const size_t off_dx = (size_t)q * a.copies * a.dim * kBytes + i * threads * (8 * kBytes);
                back_store<kF32>(a, out_dres + off, out_dx + off_dx, ds);
            }
        }
        out_dx += hop * a.copies * kBytes;
        out_dres += hop * kBytes;
    }
    if (!a.dweight) return;
    float* part = a.part + (size_t)blockIdx.x * a.dim;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
        if (me + i * threads < V) store8_f32(part + (me + i * threads) * 8, dw[i]);
}

// dweight = the blocks' shares, 32 columns a block, each summed by 8 threads.
__global__ void __launch_bounds__(256) k_norm_weights(const float* part, int blocks, int dim, float* dweight) {
    __shared__ float sm[8][32];
    pdl_launch_dependents();
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
    pdl_wait();
    float t = 0.f;
    if (col < dim)
#pragma unroll 8
        for (int b = slice; b < blocks; b += 8) t += part[(size_t)b * dim + col];
    sm[slice][threadIdx.x & 31] = t;
    __syncthreads();
    if (slice == 0 && col < dim) {
#pragma unroll
        for (int k = 1; k < 8; ++k) t += sm[k][threadIdx.x];
        dweight[col] = t;
    }
}

// How a row is laid over threads.
struct Shape {
    bool warp;
    int vec, lanes, threads, rows;  // vectors of 8 a thread, threads a row, of a block; rows a block
};
// wide: two vectors a thread.  It pays for an 8-bit output, whose blocks of 32 take shuffles
// and scales (20,000 rows of 5,120: 115 us, with one vector 123; with an output in BF16 one
// vector 127, two 144: more threads send for a row and sum it sooner).
// lane_rows: the widest row, in vectors, that belongs to lanes of a warp.  lean: a kernel whose
// two vectors a thread leave room for 1,024 threads; it takes them from 641 vectors on (16,000
// rows of 6,144: 124 us, with one 147; 12,000 of 8,192 125 and 133; 8,000 of 12,288 127, with
// four 136; 6,000 of 16,384 to 8 bits 114 and 146, but to BF16 140 and 129).
Shape shape_of(int dim, bool wide, int lane_rows, bool lean) {
    const int V = dim / 8;
    if (V <= lane_rows) {
        const int vec = V <= 32 ? 1 : V <= 64 ? 2 : 4;
        int lanes = 1;
        while (lanes * vec < V) lanes *= 2;
        return {true, vec, lanes, kGroupThreads, kGroupThreads / lanes};
    }
    const int vec = V > 1024 ? (lean && (wide || V <= 1536) ? 2 : 4) : (wide && V > 320) || (lean && V > 640) ? 2 : 1;
    const int threads = ((V + vec - 1) / vec + 31) / 32 * 32;
    return {false, vec, threads, threads, 1};
}

constexpr int kPairRows = 4;  // rows a block from which the backward pass takes them two at a time

// Shared memory of an SM that the blocks' stages may take.
constexpr int kStageBytes = 216 * 1024, kSharedBytes = 228 * 1024;

// How many blocks walk over n rows, and with how many stages in how much shared memory; rows
// that are worked on together.
struct Walk {
    int blocks, stages, bytes, rows = 1;
};
// per_sm blocks of an SM with `stages` stages of `bytes` a row, or what of them fits; without
// stages where a block has a row or two, and where not even two stages fit.
Walk walk_of(const Shape& sh, int64_t n, int per_sm, int stages, int64_t bytes, int rows_a_block) {
    const int64_t groups = (n + sh.rows - 1) / sh.rows, sms = device_sm_count();
    const int64_t direct = sms * std::max(1, 1024 / sh.threads);
    if (!sh.warp && groups > direct) {
        while (per_sm > 1 && per_sm * (stages * bytes + 1024) > kStageBytes) --per_sm;
        while (stages > 1 && stages * bytes + 1024 > kStageBytes) --stages;
        // Blocks of a few rows each follow one another in order, so that the rows that are
        // worked on at a time are neighbours (40,000 rows of 2,560: 122 us with 4 rows a block,
        // 140 with blocks that stay; 50,032 of 5,120 301 and 311).  One that has an SM to itself
        // would show its beginning, and stays (rows_a_block 0).
        if (stages > 1) {
            const int64_t turns = rows_a_block ? (groups + rows_a_block - 1) / rows_a_block : 0;
            int64_t smem = stages * bytes;
            // Blocks that stay are spread evenly only where no SM has room for one more: the first
            // of a dependent launch come while the kernel before still holds most SMs (13,000 rows
            // of 4,608, blocks of 576 threads: 158 us with two of them on some SMs, 104 without).
            if (!turns) smem = std::max<int64_t>(smem, kSharedBytes / (per_sm + 1));
            return {(int)std::min(groups, std::max(sms * per_sm, turns)), stages, (int)smem};
        }
    }
    return {(int)std::max<int64_t>(1, std::min(groups, direct)), 0, 0};
}

// 8,192 rows of 4 x 5,120 (40 KB): one block and three stages 78 us, two and two 8 more; 20,000
// rows of 2 x 5,120: two blocks and two stages 127 us, three stages 137, one block and four
// 131; an 8-bit output: two blocks and three stages 115, two stages 123.
Walk norm_walk(const Shape& sh, int64_t n, bool mx, int64_t bytes) {
    if (mx) return walk_of(sh, n, std::max(1, (sh.vec == 2 ? 640 : 1344) / sh.threads), 3, bytes, 4);
    const int blocks = std::max(1, 1344 / sh.threads);
    return blocks * 2 * bytes > 120 * 1024 ? walk_of(sh, n, std::max(1, blocks / 2), 3, bytes, 0)
                                           : walk_of(sh, n, blocks, 2, bytes, blocks > 2 ? 4 : 8);
}
template <int kVec, bool kF32, bool kMx, int kStages>
cudaError_t norm_staged(const NormArgs& a, const Shape& sh, const Walk& walk, cudaStream_t s) {
    static PerDevice allowed;
    auto f = k_norm<kVec, false, kF32, kMx, kStages>;
    cudaError_t e = allow_shared(allowed, f, kStageBytes);
    if (e != cudaSuccess) return e;
    return pdl_launch(f, dim3(walk.blocks), dim3(sh.threads), walk.bytes, s, a);
}
template <int kVec, bool kWarp, bool kF32, bool kMx>
cudaError_t norm_of(const NormArgs& a, const Shape& sh, cudaStream_t s) {
    const int64_t bytes = (int64_t)Row<kF32>::pieces(a.dim / 8) * 16 * (a.copies + (a.residual != nullptr));
    const Walk walk = norm_walk(sh, a.n, kMx, bytes);
    if constexpr (!kWarp) {
        if (walk.stages == 3) return norm_staged<kVec, kF32, kMx, 3>(a, sh, walk, s);
        if (walk.stages == 2) return norm_staged<kVec, kF32, kMx, 2>(a, sh, walk, s);
    }
    return pdl_launch(k_norm<kVec, kWarp, kF32, kMx, 0>, dim3(walk.blocks), dim3(sh.threads), 0, s, a);
}
template <bool kF32, bool kMx>
cudaError_t norm_type(NormArgs a, cudaStream_t s) {
    const Shape sh = shape_of(a.dim, kMx, 32, !kF32);
    a.lanes = sh.lanes;
    if (sh.warp) return norm_of<1, true, kF32, kMx>(a, sh, s);
    if constexpr (kMx || !kF32)
        if (sh.vec == 2) return norm_of<2, false, kF32, kMx>(a, sh, s);
    return sh.vec == 1 ? norm_of<1, false, kF32, kMx>(a, sh, s) : norm_of<4, false, kF32, kMx>(a, sh, s);
}

// Two vectors a thread where dx has one copy (16,000 rows of 5,120: 112 us, with one vector
// 129), one where several are written (8,192 rows, four copies: 97 us, with two 107).
Shape back_shape(const NormBackArgs& a) { return shape_of(a.dim, a.copies == 1, 128, false); }
// About 1,024 threads and three stages (40,000 rows of 2,560: three blocks of 320 148 us, two
// 203), more of the smallest blocks (100,000 rows of 1,032: 189 us, 212).  BF16 rows of one
// copy in pairs with two stages (12,000 rows of 8,192: 123 us, 136 one by one; 40,000 of
// 2,560: 136, 142); not where more is written (8,192 rows, four copies: 106, 97) nor fp32
// (10,000 rows of 5,120: 114, 109).  As if there were dsum, so that the same blocks make the
// same sums with and without it.
Walk back_walk(const Shape& sh, int64_t n, int dim, bool f32, bool pairs) {
    const int V = dim / 8, blocks = std::max(1, (sh.threads <= 160 ? 1344 : 1024) / sh.threads);
    const int64_t bytes = (2 * (f32 ? Row<true>::pieces(V) : Row<false>::pieces(V)) + V) * 16;
    if (pairs && n >= kPairRows * (int64_t)device_sm_count() * blocks) {
        Walk two = walk_of(sh, n, blocks, 2, 2 * bytes, 0);
        two.rows = 2;
        if (two.stages == 2) return two;
    }
    return walk_of(sh, n, blocks, 3, bytes, 0);
}
template <int kVec, bool kF32, int kRows, int kStages>
cudaError_t back_staged(const NormBackArgs& a, const Shape& sh, const Walk& walk, cudaStream_t s) {
    static PerDevice allowed;
    auto f = k_norm_backward_staged<kVec, kF32, kRows, kStages>;
    cudaError_t e = allow_shared(allowed, f, kStageBytes);
    if (e != cudaSuccess) return e;
    return pdl_launch(f, dim3(walk.blocks), dim3(sh.threads), walk.bytes, s, a);
}
template <int kVec, bool kWarp, bool kF32>
cudaError_t back_of(const NormBackArgs& a, const Shape& sh, const Walk& walk, cudaStream_t s) {
    if constexpr (!kWarp) {
        if constexpr (!kF32)
            if (walk.rows == 2) return back_staged<kVec, kF32, 2, 2>(a, sh, walk, s);
        if (walk.stages == 3) return back_staged<kVec, kF32, 1, 3>(a, sh, walk, s);
        if (walk.stages == 2) return back_staged<kVec, kF32, 1, 2>(a, sh, walk, s);
    }
    return pdl_launch(k_norm_backward<kVec, kWarp, kF32>, dim3(walk.blocks), dim3(sh.threads),
                      kWarp ? kGroupThreads * kVec * 32 : 0, s, a);
}
template <bool kF32>
cudaError_t back_type(NormBackArgs a, const Shape& sh, const Walk& walk, cudaStream_t s) {
    a.lanes = sh.lanes;
    if (sh.warp)
        return sh.vec == 1   ? back_of<1, true, kF32>(a, sh, walk, s)
               : sh.vec == 2 ? back_of<2, true, kF32>(a, sh, walk, s) : back_of<4, true, kF32>(a, sh, walk, s);
    if (sh.vec == 2) return back_of<2, false, kF32>(a, sh, walk, s);
    return sh.vec == 1 ? back_of<1, false, kF32>(a, sh, walk, s) : back_of<4, false, kF32>(a, sh, walk, s);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, bool f32, bool mx, cudaStream_t s) {
    return f32 ? (mx ? norm_type<true, true>(a, s) : norm_type<true, false>(a, s))
               : (mx ? norm_type<false, true>(a, s) : norm_type<false, false>(a, s));
}

int norm_backward_most_blocks(int64_t n, int dim) {
    const Shape sh = shape_of(dim, true, 128, false);  // (smaller blocks than the other shape's)
    const int per_sm = std::max(1, 1344 / sh.threads);
    return (int)std::min<int64_t>((n + sh.rows - 1) / sh.rows, (int64_t)device_sm_count() * per_sm);
}

cudaError_t launch_norm_backward(const NormBackArgs& a, bool f32, cudaStream_t s) {
    const Shape sh = back_shape(a);
    Walk walk = back_walk(sh, a.n, a.dim, f32, !f32 && a.copies == 1);
    walk.blocks = std::min(walk.blocks, norm_backward_most_blocks(a.n, a.dim));  // what the workspace holds
    cudaError_t e = f32 ? back_type<true>(a, sh, walk, s) : back_type<false>(a, sh, walk, s);
    if (e != cudaSuccess || !a.dweight) return e;
    return pdl_launch(k_norm_weights, dim3((a.dim + 31) / 32), dim3(256), 0, s, a.part, walk.blocks, a.dim,
                      a.dweight);
}

}  // namespace engram
