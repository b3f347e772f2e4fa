// Two fp32 values that one instruction works on (sm_100 and later): kernels that
// have little time per byte run out of issue slots before they run out of
// arithmetic, and these take one slot for two operations.
#pragma once

namespace spco {

struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 pair(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 both(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
// a - b: the product with -1 is exact, so it rounds as a subtraction does
__device__ __forceinline__ F2 operator-(F2 a, F2 b) { return fma2(b, pair(-1.f, -1.f), a); }
__device__ __forceinline__ float sum2(F2 a) {
    const float2 f = both(a);
    return f.x + f.y;
}

}  // namespace spco
