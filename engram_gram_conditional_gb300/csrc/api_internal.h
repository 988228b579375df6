// What the host translation units of libengram.so share: the context, and the
// argument checks and error reporting of the C ABI.
#pragma once

#include <stdint.h>

#include <string>
#include <vector>

#include "../../include/engram.h"
#include "engram_internal.h"

struct LayerState {
    std::vector<uint64_t> mult;    // [nb][4]
    std::vector<uint64_t> prime;   // [nb]
    std::vector<uint64_t> offset;  // [nb]
    uint64_t rows = 0;
    bool bound = false;
    engram_layer_weights w{};
    CUtensorMap tm_wkv{};          // the caller's BF16 wkv
    CUtensorMap tm_wkv_half{};     // the same with 128-row boxes (CTA-pair kernels)
    // FP16 operand path of the fused kernels (see engram_layer_info)
    bool f16 = false;
    uint16_t* wkv_f16 = nullptr;   // library-owned copy, wkv x 2^wkv_exp
    float* wqk = nullptr;          // library-owned w_q * w_k [hc][d], made at bind
    CUtensorMap tm_wkv_f16{};
    CUtensorMap tm_wkv_f16_2k{};   // the tiled FP16 copy with 256-row boxes (2 k-blocks)
    int wkv_exp = 0;
    int a_exp_shift = 0;
    uint32_t scale_min = 0, scale_max = 0;
    bool bucket_gather = false;    // whole 256-wide rows gathered once per tile and bucket
    bool table_bf16 = false;       // BF16 rows without scales (ENGRAM_BIND_TABLE_BF16)
    // bound to a shard of the table (engram_layer_bind_shard): rows
    // [row_lo, row_lo + shard_rows) of the layer's table
    bool shard = false;
    uint64_t row_lo = 0, shard_rows = 0;
};

struct engram_ctx {
    engram_ctx_desc desc{};
    std::vector<uint64_t> seeds, bases;
    std::vector<uint32_t> map;
    int nb = 0, K = 0, N = 0;
    std::vector<LayerState> layers;
    uint32_t* d_err = nullptr;  // [0] error word, [1..3] bind-time scan results
    int device = -1;
    long long wait_limit_ns = 4000000000LL;
    int starve_b = 0;
};

namespace engram {

engram_status fail(engram_status st, const std::string& msg);
engram_status ok();
engram_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

engram_status check_layer(const engram_ctx* ctx, int layer, bool need_bound);
engram_status check_T(int64_t T);
// The context's device word (error word and scan results), allocated at the
// first bind, scan or training call on device dev.
engram_status ensure_device_word(engram_ctx* ctx, int dev);

}  // namespace engram
