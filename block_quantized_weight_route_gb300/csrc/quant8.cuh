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

// Four values to E4M3 codes, the first in the low byte; finite values past +-448
// saturate, NaN stays NaN (0x7F).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// The factor that turns a group's values into code units.  y / s is formed as
// y * (1 / s), within 1.5 ulp of the quotient: a code moves only where y / s lies
// that close to a rounding boundary.  Below 2^-120 the reciprocal could leave the
// fp32 range, so such a (denormal or nearly) group is scaled up by 2^120 first.
struct GroupScale {
    float pre, inv;
    __device__ __forceinline__ float operator()(float y) const { return y * pre * inv; }
};
__device__ __forceinline__ GroupScale group_scale(float s) {
    constexpr float kUp = 1.329227995784916e36f;   // 2^120
    GroupScale g;
    const bool tiny = s < 7.52316384526264e-37f;   // 2^-120
    g.pre = tiny ? kUp : 1.0f;
    g.inv = (s == 0.0f) ? 0.0f : 1.0f / (s * g.pre);
    return g;
}

}  // namespace qmm
