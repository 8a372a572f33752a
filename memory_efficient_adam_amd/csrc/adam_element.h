// Device code that the kernels of a step share: streaming accesses, bf16, and
// the exact square root and quotient of the update.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace adam_mi355x {
namespace {

// ---------------------------------------------------------------- streaming access
// Every byte of params, grads and state is touched exactly once per step, so
// all data accesses are non-temporal (the "nt" cache policy): measured on
// MI355X this raises the mixed read/write stream rate by 5-10% over the
// default policy, and only when loads and stores both use it.
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 ld_f32x4(const float *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
}
__device__ __forceinline__ u32x2 ld_u32x2(const void *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
}
__device__ __forceinline__ uint32_t ld_u32(const void *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(p));
}
template <class T>
__device__ __forceinline__ T ld_one(const T *p) {
    return __builtin_nontemporal_load(p);
}
__device__ __forceinline__ void st_f32x4(float *p, f32x4 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(p));
}
__device__ __forceinline__ void st_u32x2(void *p, u32x2 v) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x2 *>(p));
}
__device__ __forceinline__ void st_u32(void *p, uint32_t v) {
    __builtin_nontemporal_store(v, reinterpret_cast<uint32_t *>(p));
}
__device__ __forceinline__ void st_one(float *p, float v) { __builtin_nontemporal_store(v, p); }

// ---------------------------------------------------------------- bf16
__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __uint_as_float(h << 16); }

// Round to nearest, ties to even, on the upper 16 bits; NaN -> 0x7FC0.
__device__ __forceinline__ uint32_t f32_to_bf16(float x) {
    if (x != x) return 0x7FC0u;
    const uint32_t u = __float_as_uint(x);
    return (u + 0x7FFFu + ((u >> 16) & 1u)) >> 16;
}

// ---------------------------------------------------------------- exact sqrt / divide
// Correctly rounded square root and quotient for operands in a normal range,
// without the range handling of the general sequences (which scale tiny or
// huge operands and patch zeros, infinities and NaNs).  Where they apply
// they perform the same operations as the general correctly rounded
// sequences, so the results are the same bits.
//
// sqrt_rn: x in [2^-96, 2^128).  The hardware square root is within one ulp
// of sqrt(x), so the rounded root is it or a neighbour; the sign of the
// exact residual x - s' * s (one fma) tells which: x <= s_- * s means sqrt(x)
// lies below the midpoint of s_- and s, x > s_+ * s that it lies above the
// midpoint of s and s_+ (x, s_- * s and s * s_+ sit on a grid too coarse for
// x to fall strictly between a product and its midpoint square).
__device__ __forceinline__ float sqrt_rn(float x) {
    const float s = __builtin_amdgcn_sqrtf(x);
    const float sm = __uint_as_float(__float_as_uint(s) - 1u);
    const float sp = __uint_as_float(__float_as_uint(s) + 1u);
    float r = fmaf(-sm, s, x) <= 0.0f ? sm : s;
    return fmaf(-sp, s, x) > 0.0f ? sp : r;
}

// div_rn: d in [2^-40, 2^77], |n| in [2^-40, 2^40] (quotient and reciprocal
// normal, no intermediate over- or underflow): the hardware reciprocal, one
// Newton step, and two quotient corrections whose remainders n - d*q are
// exact (fma).
__device__ __forceinline__ float div_rn(float n, float d) {
    float r = __builtin_amdgcn_rcpf(d);
    r = fmaf(fmaf(-d, r, 1.0f), r, r);
    float q = n * r;
    q = fmaf(fmaf(-d, q, n), r, q);
    return fmaf(fmaf(-d, q, n), r, q);
}

}  // namespace
}  // namespace adam_mi355x
