// Shared by the 4-bit (OCP MXFP4) kernels: the block scale rule, the cast of
// eight elements to a word of E2M1 codes, the stochastic rounding's random
// bits.  gfx950 only.
//
// A row is cut into blocks of 32 elements that share one E8M0 scale byte b,
// standing for s = 2^(b-127); an element is an E2M1 code (sign, 2 exponent
// and 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6).  Two codes share a byte,
// the even column in the low half.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fp8mi.h"

namespace fp8mi {
namespace mx4 {

constexpr int kBlock = 32;         // elements that share a scale
constexpr int kRowAlign = 256;     // a row of codes is padded to this many elements (128 bytes)
constexpr int kPanel = 512;        // columns whose 16 scale bytes lie side by side

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// Scale byte of a block from the bits of its finite fp32 amax = m 2^e, m in
// [1, 2): the smallest power of two s with amax / s <= 6 = 1.5 * 2^2 is
// 2^(e-2), or 2^(e-1) when m > 1.5; adding 0x3FFFFF carries into the
// exponent field exactly when m > 1.5.  Not under 2^-126; 1 for amax 0.
__device__ inline uint32_t scale_byte(uint32_t amax_bits)
{
    const int b = (int)((amax_bits + 0x3FFFFFu) >> 23) - 2;
    return amax_bits == 0 ? 127u : (uint32_t)max(b, 1);
}
// 2^(b-127) as the conversions and matrix instructions take it: they read the
// exponent field alone (0 stands for 2^-127, 255 for NaN; measured over every
// byte and code, subnormal results included).
__device__ inline float scale_float(uint32_t b) { return __builtin_bit_cast(float, b << 23); }

__device__ inline uint32_t mix(uint32_t v)
{
    v ^= v >> 16;
    v *= 0x6A09E667u;
    v ^= v >> 15;
    v *= 0xBB67AE85u;
    return v ^ (v >> 16);
}
// The 32 random bits of a row's column pair: even columns take the low half,
// odd ones the high half.
__device__ inline uint32_t row_key(uint32_t row, uint32_t seed_lo) { return mix(row * 0x9E3779B1u + seed_lo); }
__device__ inline uint32_t pair_key(uint32_t pair, uint32_t seed_hi) { return pair * 0x3C6EF373u + seed_hi; }

// Eight elements to a word of codes.
__device__ inline uint32_t cast8_rne(const float x[8], float s)
{
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
}
// The same of eight bf16 elements, two to a word.
__device__ inline uint32_t cast8_rne(const uint32_t x[4], float s)
{
    uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, __builtin_bit_cast(v2bf, x[0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, x[1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, x[2]), s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(v2bf, x[3]), s, 3);
}

// Stochastic rounding: |x| / s between two grid values goes up when its
// fraction of the way plus r / 65536 reaches 1, r the element's 16 random
// bits.  The conversion adds its 32-bit seed to the fraction, for element 0
// as it is and for element 1 from bit 30 down, so one conversion cannot give
// both elements bits of their own: each pair is converted twice, and the
// even halves of the one and the odd halves of the other are joined.
// se[p] = r(even) << 16, so[p] = r(odd) << 15.
__device__ inline uint32_t cast8_sr(const float x[8], const uint32_t se[4], const uint32_t so[4], float s)
{
    uint32_t a[4], b[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const v2f v = v2f{x[2 * p], x[2 * p + 1]};
        a[p] = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, v, se[p], s, 0);
        b[p] = __builtin_amdgcn_cvt_scalef32_sr_pk_fp4_f32(0u, v, so[p], s, 0);
    }
    // bytes 0 of four words to one word
    const auto join = [](const uint32_t w[4]) {
        const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(w[3], w[2], 0x04000C0Cu);
        return lo | hi;
    };
    return (join(a) & 0x0F0F0F0Fu) | (join(b) & 0xF0F0F0F0u);
}

// A kernel's LDS limit, raised once a device.
struct LdsLimit {
    std::atomic<uint64_t> done{0};
    hipError_t raise(const void* kernel, int bytes)
    {
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        if (e != hipSuccess) return e;
        const uint64_t bit = 1ull << (dev & 63);
        if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
        e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

}  // namespace mx4
}  // namespace fp8mi
