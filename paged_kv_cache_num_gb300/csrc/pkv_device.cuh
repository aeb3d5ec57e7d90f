// pkv_device.cuh -- small device helpers shared by the kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "pkv_internal.h"

namespace pkv {

// Programmatic dependent launch.  A kernel launched with
// launch_pdl may start while the previous kernel of its stream still runs:
// it must call griddep_wait() before touching any global memory that kernel
// may write, and calls griddep_launch_dependents() once the next kernel may
// be scheduled.  Both are no-ops for a normally launched kernel.
__device__ __forceinline__ void griddep_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void griddep_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;");
}

__device__ __forceinline__ void raise_err(int32_t *flag, int bits)
{
    if (flag) atomicOr(flag, bits);
}

// 2^x on the SFU (ex2.approx, flush-to-zero); exp(x) = 2^(x*log2 e).
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 of a scale, at most 1 above it, from its biased exponent, within +-K: what
// a softmax's reference takes of V scales whose products with the weights are
// packed to 16 bits
template <int K> __device__ __forceinline__ float scale_exp(uint32_t e) { return float(min(max(int(e) - 126, -K), K)); }

// 16-bit element <-> float
template <int KIND> __device__ __forceinline__ float h2f(uint16_t v);
template <> __device__ __forceinline__ float h2f<kF16>(uint16_t v)
{
    return __half2float(__ushort_as_half(v));
}
template <> __device__ __forceinline__ float h2f<kBF16>(uint16_t v)
{
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

template <int KIND> __device__ __forceinline__ uint16_t f2h(float v);
template <> __device__ __forceinline__ uint16_t f2h<kF16>(float v)
{
    return __half_as_ushort(__float2half_rn(v));
}
template <> __device__ __forceinline__ uint16_t f2h<kBF16>(float v)
{
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// two 16-bit elements -> two floats, without a shift for the upper one
template <int KIND> __device__ __forceinline__ float2 h2f2(uint32_t w)
{
    if constexpr (KIND == kF16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// two floats -> two 16-bit elements, rounded to nearest even
template <int KIND> __device__ __forceinline__ uint32_t f2h2(float x, float y)
{
    if constexpr (KIND == kF16) {
        const __half2 v = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// Eight 4-bit codes (element j at bits 4j .. 4j+3) minus their zero point z, as
// pairs of f16 numbers in order, exactly: under 0x6400 a byte with code u is
// 1024 + u; nz holds -1024 - z twice.
__device__ __forceinline__ void u4x8_to_f16(uint32_t w, uint32_t nz, uint32_t (&o)[4])
{
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    const uint32_t lo = __byte_perm(even, odd, 0x5140), hi = __byte_perm(even, odd, 0x7362);
    o[0] = __byte_perm(lo, 0x64646464u, 0x4140);
    o[1] = __byte_perm(lo, 0x64646464u, 0x4342);
    o[2] = __byte_perm(hi, 0x64646464u, 0x4140);
    o[3] = __byte_perm(hi, 0x64646464u, 0x4342);
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("add.rn.f16x2 %0, %0, %1;" : "+r"(o[i]) : "r"(nz));
}

// Two fp8 codes of cache kind FP8 (kE4M3 / kE5M2), bytes 2HI and 2HI+1 of w
// (low byte first) -> two floats, exactly: cvt.rn.f16x2 on the 16-bit half
// of the register, then the f16 -> f32 widening.
template <int FP8, int HI>
__device__ __forceinline__ float2 fp8x2_to_float2(uint32_t w)
{
    uint32_t h;
    if constexpr (FP8 == kE4M3) {
        if constexpr (HI)
            asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(h) : "r"(w));
        else
            asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(h) : "r"(w));
    } else {
        if constexpr (HI)
            asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e5m2x2 %0, h;\n}" : "=r"(h) : "r"(w));
        else
            asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e5m2x2 %0, l;\n}" : "=r"(h) : "r"(w));
    }
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace pkv
