#ifndef ZS_CODES_H
#define ZS_CODES_H

// Device-side arithmetic of the lists of tensors that takes fewer operations
// than the compiler's forms, or other ones, and gives the same bits:
// conversion to bf16, roots, a block's quotient and the 8-bit codes.  What is
// said of every input of a range was compared for each of them, by
// tests/test_tensors_forms_gpu.py.

#include <hip/hip_runtime.h>

#include <cstdint>

namespace {

// Two fp32 values -> bf16 bits, nearest even; NaN -> quiet NaN keeping sign
// and the top payload bits (the instruction gives what the step kernels of
// zs_step.hip compute, for every one of the 2^32 inputs).
__device__ __forceinline__ uint32_t to_bf16(float lo, float hi)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(
        uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// The root of x, correctly rounded, for x in [2^-96, infinity): from the
// reciprocal root y, g = x y and a step of Newton's method for x - g^2,
// g + (x - g g) y / 2.  The compiler's root takes 17 operations.
__device__ __forceinline__ float root_of(float x)
{
    const float y = __builtin_amdgcn_rsqf(x);
    const float g = x * y;
    return __builtin_fmaf(__builtin_fmaf(-g, g, x), 0.5f * y, g);
}

// The whole number q with (q - 1/2)^2 <= y < (q + 1/2)^2, y >= 0, as a float.
// The hardware's root is within an ulp; less 2^-10 the guess is q or one
// below it, and (q + 1/2)^2 = q (q + 1) + 1/4 is exact in fp32 up to 255.
__device__ __forceinline__ float root_code(float y)
{
    const float q = floorf(__builtin_amdgcn_sqrtf(y) + (0.5f - 0x1p-10f));
    return __builtin_fmaf(q, q + 1.0f, 0.25f) <= y ? q + 1.0f : q;
}

constexpr float kTopM = 127.0f * 127.0f, kTopR = 255.0f * 255.0f;

// top / A for top of kTopM and kTopR, correctly rounded for A in
// [2^-100, 2^126): the product with the reciprocal, and what that leaves over
// by the same reciprocal (a step of Newton's method).
__device__ __forceinline__ float quotient_of(float top, float A)
{
    const float rcp = __builtin_amdgcn_rcpf(A);
    const float q = top * rcp;
    return __builtin_fmaf(__builtin_fmaf(-A, q, top), rcp, q);
}

// Low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b,
                                              uint32_t c, uint32_t d)
{
    return __builtin_amdgcn_perm(b, a, 0x0c0c0400u) |
           __builtin_amdgcn_perm(d, c, 0x04000c0cu);
}

// Codes of four m whose scaled sizes are |m| im, and of four roots.
//
// The hardware's root s of y is within 2^-16 of the true one below 256, so
// the whole number nearest to s is the code unless s is within 2^-15 of
// halfway between two: about one unit in 30 has such a value (2^-14 for each
// of 512 codes) and takes root_code().  Adding 2^23 (for m with its sign
// 1.5 2^23) rounds s to a whole number, which is then the sum's low byte, in
// two's complement.
constexpr float kNear = 0.5f - 0x1p-15f;

__device__ __forceinline__ void codes(const float (&m)[4],
                                      const float (&r)[4], float im, float ir,
                                      uint32_t& cm, uint32_t& cr)
{
    float tm[4], tr[4], ym[4], yr[4], far = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        ym[j] = fabsf(m[j]) * im;
        const float s = copysignf(__builtin_amdgcn_sqrtf(ym[j]), m[j]);
        tm[j] = s + 0x1.8p+23f;
        const float dm = s - (tm[j] - 0x1.8p+23f);
        // a root that is not 0 keeps a code of 1: y is at least 2^-123 there
        // and is lifted to 0.36
        yr[j] = r[j] * ir;
        yr[j] = __builtin_amdgcn_fmed3f(yr[j], 0.36f, yr[j] * 0x1p+125f);
        const float u = __builtin_amdgcn_sqrtf(yr[j]);
        tr[j] = u + 0x1p+23f;
        const float dr = u - (tr[j] - 0x1p+23f);
        far = fmaxf(far, fmaxf(fabsf(dm), fabsf(dr)));
    }
    if (__builtin_expect(__any(!(far < kNear)), 0)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            tm[j] = copysignf(root_code(ym[j]), m[j]) + 0x1.8p+23f;
            tr[j] = root_code(yr[j]) + 0x1p+23f;
        }
    }
    cm = low_bytes(__float_as_uint(tm[0]), __float_as_uint(tm[1]),
                   __float_as_uint(tm[2]), __float_as_uint(tm[3]));
    cr = low_bytes(__float_as_uint(tr[0]), __float_as_uint(tr[1]),
                   __float_as_uint(tr[2]), __float_as_uint(tr[3]));
}

}  // namespace

#endif  // ZS_CODES_H
