// Rounding of fp32 values to the library's two 8-bit activation formats.
//   FP8: groups of 128 values, s = max|y| / 448 (fp32), code = E4M3(y / s), nearest even
//   q8_1: groups of 32 values, d = max|y| / 127, code = round-half-away(y / d) in [-127, 127],
//         stored with fp16(d) and fp16(d * sum of the codes)
// A group whose values are all zero has scale 0 and codes 0.  A NaN, or an
// infinity (whose quotient by an infinite scale is NaN), makes the E4M3 codes of
// its group NaN where the quotient is.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace qmm {

// Launches of these kernels overlap (programmatic dependent launch): a kernel says at
// its start that the next one may be started, and before its first access to global
// memory waits until the one before has finished and its writes are visible.  One
// after the other, a kernel's start (barriers, TMEM, descriptors) and its launch then
// run beside the end of the one before: 0.5 to 1 us a call.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_prerequisites() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
inline cudaLaunchAttribute overlap_attribute() {
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    return a;
}

// max that hands a NaN on (fmaxf drops it): a group with a NaN has a NaN scale
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// the same over the magnitudes of three
__device__ __forceinline__ float max_nan_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Four consecutive elements of an fp32 or bf16 array, i a multiple of 4; and one.
__device__ __forceinline__ float4 load4(const void* a, int bf16, long i) {
    if (!bf16) return *reinterpret_cast<const float4*>(static_cast<const float*>(a) + i);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a) + i);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const void* a, int bf16, long i) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a)[i]) : static_cast<const float*>(a)[i];
}
__device__ __forceinline__ void store4(void* a, int bf16, long i, float4 v) {
    if (bf16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a) + i) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
        *reinterpret_cast<float4*>(static_cast<float*>(a) + i) = v;
    }
}

// Two fp32 values in one 64-bit register, and packed arithmetic on them.
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) { return pack2u(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
    return make_float2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Four values to E4M3 codes, the first in the low byte; finite values past +-448
// saturate, NaN stays NaN (0x7F).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// The scale of a group, top / LEVELS, and the factor 1 / scale that turns its values
// into code units.  Both divisions are products with a reciprocal (1 / LEVELS rounded;
// the reciprocal instruction, within an ulp), so the scale is within 1 ulp and a quotient
// within 3 ulp of the formula's: a code moves only where y / s lies that close to a
// rounding boundary.  A scale below 2^-120, whose reciprocal could leave the fp32 range,
// has up = 2^120: such a group's values are multiplied by it first.
struct GroupScale {
    float s, inv, up;
    __device__ __forceinline__ bool tiny() const { return up != 1.0f; }
    __device__ __forceinline__ float operator()(float y) const { return y * up * inv; }
    __device__ __forceinline__ uint64_t two(uint64_t y) const {   // (the same quotients)
        return tiny() ? mul2(mul2(y, pack2(up, up)), pack2(inv, inv)) : mul2(y, pack2(inv, inv));
    }
};
template <int LEVELS>
__device__ __forceinline__ GroupScale group_scale(float top) {
    GroupScale g;
    g.s = top * (1.0f / LEVELS);
    g.up = g.s < 7.52316384526264e-37f ? 1.329227995784916e36f : 1.0f;   // 2^-120, 2^120
    float x = g.s * g.up;
    asm("rcp.approx.f32 %0, %1;" : "=f"(g.inv) : "f"(x));
    if (g.s == 0.0f) g.inv = 0.0f;
    return g;
}

}  // namespace qmm
