// pairs.cuh -- two fp32 values in a register pair: the add, multiply and fused multiply-add that take both at once,
// and two bf16 values as such a pair.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace bsa {
namespace {

// Two channels per instruction: fp32 add, multiply and fused multiply-add on register pairs.
using f2 = unsigned long long;

__device__ __forceinline__ f2 pair(float a, float b)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 twice(float a) { return pair(a, a); }
__device__ __forceinline__ void split(f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ float two(f2 v)
{
    float a, b;
    split(v, a, b);
    return a + b;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ f2 widen(uint32_t w) { return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t narrow(f2 v)
{
    float a, b;
    split(v, a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace
}  // namespace bsa
