// kvr_q4.cuh -- the paged 4-bit K/V cache: layout of a page and the quantiser
// of one group, shared by the kernels that write, read and attend over it.
#pragma once

#include <cuda_fp16.h>

#include "kvr_device.cuh"

namespace kvr {

// A page of one head, ps tokens: K codes [ps][D/2], V codes [ps][D/2], then per
// token the fp16 parameters K s[NG], K z[NG], V s[NG], V z[NG].
template <int D> struct Q4 {
    static constexpr int NG = D / 32;         // groups of a row
    static constexpr int CB = D / 2;          // code bytes of a row
    static constexpr int PB = D / 4;          // parameter bytes of a token (K and V)
    static constexpr int TB = 2 * CB + PB;    // bytes of a token, 5 D / 4
};

// Device view of a cache (kvr_q4_cache with the page size as a shift).
struct Q4Pages {
    uint8_t *base;
    int64_t n_pages;
    int ps_log2, Hkv;
};

// First byte of head h's block of page p (64-bit: pools pass 4 GB).
template <int D>
__device__ __forceinline__ uint8_t *q4_block(const Q4Pages &c, int64_t p, int h)
{
    return c.base + (p * c.Hkv + h) * ((int64_t)Q4<D>::TB << c.ps_log2);
}

// Minimum and maximum that keep a NaN operand.
__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The least and the greatest of 8 values in memory order, of 16 or 32 bytes.
__device__ __forceinline__ void range8(const float (&x)[8], float &mn, float &mx)
{
    mn = mx = x[0];
#pragma unroll
    for (int i = 1; i < 8; i++) {
        mn = min_nan(mn, x[i]);
        mx = max_nan(mx, x[i]);
    }
}

// Scale and zero of a group from its minimum and maximum: z = the fp16 toward
// -inf of the minimum (a zero is +0), s = the smallest fp16 >= 0 with
// fmaf(15, s, z) >= max. A group without such fp16 values (a NaN or an
// infinity in it, too wide a range) gets s = z = NaN and false.
// NARROW: the range may be under 2^-13 of z, as of fp32 rows. Of bf16 ones it is 0 or at least 2^-11 of z where z
// is more than 16 (and below that the smallest scale, 2^-24, is more than 15 s + z rounds by); with the search the
// append of 131072 bf16 rows would take 1% longer.
template <bool NARROW>
__device__ __forceinline__ bool q4_params(float mn, float mx, __half &sh, __half &zh)
{
    zh = __float2half_rd(mn);
    const float z = __half2float(zh) + 0.0f;
    zh = __float2half_rn(z);
    // (+ 0 again, for a maximum of -0) the quotient is within three fp32 roundings of exact: one step up
    // always covers. Down, one step is enough unless the range is under about 2^-13 of z (15 s + z rounds
    // at the size of z): the smallest covering fp16 is then as little as half of the quotient, and searched.
    // fmaf is monotone in s.
    uint32_t sb = __half_as_ushort(__float2half_ru((__fsub_rn(mx, z) + 0.0f) * (1.0f / 15.0f)));
    auto covers = [&](uint32_t bits) { return fmaf(15.0f, __half2float(__ushort_as_half((unsigned short)bits)), z) >= mx; };
    const uint32_t below = sb - (sb > 0);
    if (covers(below)) {
        sb = below;
        if (NARROW && sb > 0 && covers(sb - 1)) {
            uint32_t lo = 0;
            sb--;
            while (lo < sb) {  // sb covers; what is under lo does not
                const uint32_t mid = (lo + sb) >> 1;
                if (covers(mid)) sb = mid;
                else lo = mid + 1;
            }
        }
    } else if (!covers(sb)) {
        sb++;
    }
    // sb < 0x7c00: a finite, non-negative scale (a NaN maximum or minimum makes the quotient NaN)
    const bool ok = sb < 0x7c00u && fabsf(z) <= 65504.0f;
    sh = __ushort_as_half((unsigned short)(ok ? sb : 0x7e00u));
    if (!ok) zh = __ushort_as_half((unsigned short)0x7e00u);
    return ok;
}

// rint((x - z) * inv), the product unrounded, plus the bits of 1.5 * 2^23: the sum's
// low mantissa bits are the integer (one FADD, one FFMA, no conversion). x >= z,
// so it is never negative; inv = 0 gives 0.
constexpr uint32_t kMagic = 0x4b400000u;
__device__ __forceinline__ uint32_t q4_step(float x, float z, float inv)
{
    return __float_as_uint(fmaf(__fsub_rn(x, z), inv, 12582912.0f));
}

// Codes of 8 values as nibbles: Horner's sum of the raw bits, minus what the
// magic numbers add up to. For groups whose largest code is 15 at most.
__device__ __forceinline__ uint32_t q4_codes8(const float (&x)[8], float z, float inv)
{
    uint32_t w = 0;
#pragma unroll
    for (int i = 7; i >= 0; i--) w = w * 16u + q4_step(x[i], z, inv);
    return w - kMagic * 0x11111111u;
}

// For any group: codes past 15 (z so large beside s that 15 s + z rounds up to the maximum)
// are clamped, and a group without scale and zero (inv < 0) gets 0.
__device__ __forceinline__ uint32_t q4_codes8_any(const float (&x)[8], float z, float inv)
{
    if (inv < 0.0f) return 0u;
    uint32_t w = 0;
#pragma unroll
    for (int i = 7; i >= 0; i--) {
        const uint32_t c = q4_step(x[i], z, inv) - kMagic;
        w = w * 16u + (c < 15u ? c : 15u);
    }
    return w;
}

}  // namespace kvr
