// Helpers shared by the training operators' memory-bound kernels: launches as
// programmatic dependents, eight values at a time.
#pragma once

#include "device_common.cuh"

namespace engram {

template <class... Exp, class... Act>
inline cudaError_t pdl_launch(void (*f)(Exp...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
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

}  // namespace engram
