// kvr_q4_rows.cuh -- a warp's share of an attention over the paged 4-bit cache:
// scores, running softmax and weighted values of 16-token tiles for blocks of 8
// query rows, and the merge of the warps of a CTA.
//
// Both products run on the tensor cores (mma.sync m16n8k16, fp16 in, fp32
// accumulate) with the tokens or channels as the 16-row operand and the query
// rows of a KV head as the 8 columns:
//   S^T [16 tokens x 8 rows]   = Kc [tokens x channels] . q^T
//   O^T [16 channels x 8 rows] = Vc^T [channels x tokens] . P'^T
// A decode step has few query rows, so the 16-row side must be the cache: the
// 128-row tiles of tcgen05 would be 94% padding, and its operands would have
// to be written to shared memory as fp16, four times the bytes the codes have.
// Codes are masked out of their words two at a time: 8 codes become 4 operand
// registers with one shift and four LOP3. Every other pair is 16 times the code, and the factor goes
// into the query (exactly: a power of two) or into the output channel.
//   S: a logit's error counts as it is, however large the logit, so codes enter as normal
//   numbers, (0x6400 | c) - 1024, one more HADD2 per pair. (A masked nibble as it lies is the
//   denormal c * 2^-24. The tensor core aligns a denormal by its nominal exponent, which costs about 8 of the
//   product's 24 bits beside the row's largest query channel: logits off by up to 3500 * 2^-24 of their magnitude,
//   the sum of |q_c k_c|, where one channel outweighs the others, by 70 as it is. 128K tokens, bf16: 43.3 us, 40.9
//   with denormals.)
//   O: for bf16 outputs the codes are those denormals, in units of 2^-24: 2^-16 of the sum beside the
//   output's 2^-8. For fp32 outputs (EXACT) they are normal numbers.
// Scales and zeros stay outside the products with the codes:
//   q . k   = sum over groups g of s_g (q . c)_g + z_g (sum of q over g)
//   p . v_g = sum over tokens of (p s_g) c + p z_g
// z parts are one more m16n8k16 product each (sums of q as three fp16 terms; z
// itself as the 16-row operand). With bf16 outputs p and p s_g are rounded to
// fp16 (2^-11 each, beside the output's 2^-8, and averaged over the tokens), and the rounded p
// are what the softmax divides by. With
// fp32 outputs both are sums of two fp16 terms: p = hi + lo, u = fl(hi s), and
// fl(lo s + (hi s - u)) beside it, the bracket exact as a fused multiply-add.
#pragma once

#include <cfloat>

#include "kvr_paged.h"
#include "kvr_q4.cuh"

namespace kvr {

Q4Pages q4_pages(const kvr_q4_cache &c);

namespace q4a {

constexpr int kTile = 16;                // tokens of a tile
constexpr int kSpan = 2 * kTile;         // tokens that a warp takes at once
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kEmpty = -FLT_MAX;       // largest score before the first token
constexpr float kSlack = 3.0f;           // logits (log2) may pass the running maximum by this much
constexpr float kExp = 11.0f;            // log2 of the largest token's probability as it is kept
static_assert(kExp + kSlack + 1.0f <= 15.0f, "fp16's range, times a scale under 2");

// What both attention kernels get.
struct Args {
    Q4Pages c;
    int B, Lq, Hq, G, R, RB;  // R = G Lq query rows per KV head in RB blocks
    int64_t q_stride, max_pages, cap;
    const void *q;
    const int32_t *table, *seq_len;
    float scale;
    void *out;
    int out_bf16;
    int32_t *err;
};

// The order of a tile's 16 tokens: row r of the score tile is token T(r). Rows
// 2j and 2j + 1 have opposite parity and rows 0, 2, 4, 6 are tokens 0 .. 3:
// reads of K rows (64 or 32 bytes apart) are free of bank conflicts, those
// of V rows two-way at worst.
__device__ __forceinline__ int token_of_row(int r)
{
    return (r & 8) + ((r & 1) ? 7 - ((r & 7) >> 1) : ((r & 7) >> 1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 floats_of(uint32_t h)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
__device__ __forceinline__ __half2 as_half2(uint32_t h) { return *reinterpret_cast<const __half2 *>(&h); }

// Codes of a word as fp16 pairs: nibbles (0, 4), 16 x (1, 5), (2, 6), 16 x (3, 7), as denormals
// in units of 2^-24 or as the numbers themselves.
template <bool NORMAL> __device__ __forceinline__ void unpack(uint32_t w, uint32_t (&r)[4])
{
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        if constexpr (NORMAL) {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                // (w & mask) | 0x6400 in one LOP3: two of its operands are constants, so they go
                // through registers
                uint32_t u;
                asm("lop3.b32 %0, %1, %2, %3, 0xEA;\n" : "=r"(u) : "r"(w), "r"(k ? 0x00f000f0u : 0x000f000fu), "r"(0x64006400u));
                const __half2 h = __hsub2(as_half2(u), as_half2(0x64006400u));
                r[i + k] = *reinterpret_cast<const uint32_t *>(&h);
            }
        } else {
            r[i] = w & 0x000f000fu;
            r[i + 1] = w & 0x00f000f0u;
        }
        w >>= 8;
    }
}

__device__ __forceinline__ void store4(const Args &a, int64_t at, float4 o, float inv)
{
    if (a.out_bf16) {
        const __nv_bfloat162 u = __floats2bfloat162_rn(o.x * inv, o.y * inv);
        const __nv_bfloat162 v = __floats2bfloat162_rn(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
}

// First output element of query row r of (b, h).
__device__ __forceinline__ int64_t out_at(const Args &a, int b, int h, int r, int D)
{
    return (((int64_t)b * a.Lq + r / a.G) * a.Hq + h * a.G + r % a.G) * D;
}

__device__ __forceinline__ void fma4(float4 &o, float f, const float4 &v)
{
    o.x = fmaf(f, v.x, o.x);
    o.y = fmaf(f, v.y, o.y);
    o.z = fmaf(f, v.z, o.z);
    o.w = fmaf(f, v.w, o.w);
}

// The state of one of WARPS warps for a unit, NT blocks of 8 query rows. Q2: queries as two
// fp16 terms (fp32 queries). EXACT: fp32 outputs (the values' codes as normal numbers,
// probabilities times scales as two fp16 terms).
template <int D, bool Q2, bool EXACT, int WARPS, int NT> struct Rows {
    static constexpr int NG = D / 32, RT = 8 * NT;
    static constexpr int ROW = D + 4;                    // merge row, floats
    static constexpr int MERGE = WARPS * RT * ROW * 4;  // bytes of the merge rows, then
    static constexpr int STAT = WARPS * RT * 8;         // of (reference, sum) of each
    // Spans between additions of the tensor cores' sums to the merge rows. An
    // accumulation step truncates, always downward in magnitude: 430 steps were
    // measured to lose 5e-4 of the sum. EXACT adds every tile's sum in fp32
    // instead (32 FADD) and folds once, at the end.
    static constexpr int FOLD = EXACT ? INT32_MAX : 32;

    // Scores are kept as x with logit (log2) = x * kq, kq > 0. Probabilities are
    // 2^((x - top) kq + kExp), top the largest x so far or a little less: up to 2^14. The difference comes
    // first: x kq - (top kq - kExp) would round the reference at the logits' size, and from 2^27 on
    // the largest token itself to 0 or past fp16.
    // [NT]: blocks of 8 rows.
    uint32_t qf[NT][NG][4], ql[NT][Q2 ? NG : 1][4], qz[NT][2];
    float kq[NT][2], top[NT][2], kept[NT][2], O[NT][NG][2][4];
    // [0], [1]: row gr, sum of p z of group gr; [2], [3]: sum of p, which the other rows of the same
    // product give (a million tokens, bf16: 249 -> 241 us); EXACT, where a product's sums are added
    // in fp32 (342 us so, 333), this lane's tokens
    float zo[NT][4];
    int lim[NT][2], lim_min, folds;
    float *rows;       // this warp's merge rows
    float2 *stat;      // all warps'

    __device__ __forceinline__ void attach(uint8_t *smem, int warp)
    {
        rows = reinterpret_cast<float *>(smem) + warp * RT * ROW;
        stat = reinterpret_cast<float2 *>(smem + MERGE);
    }

    // Channels of a block of query rows as open() takes them: of rows r0 + lane / 4, channels
    // 32 gr + 8 (lane % 4) .. + 7; 0 for rows behind the last.
    using Query = float[NG][8];
    template <typename TQ>
    static __device__ __forceinline__ void load_query(const Args &a, int b, int h, int r0, Query &x)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
        const int r = r0 + g, t = r / a.G;
        const TQ *q = static_cast<const TQ *>(a.q) + ((int64_t)b * a.Lq + t) * a.q_stride +
                      (int64_t)(h * a.G + r - t * a.G) * D + j * 8;
#pragma unroll
        for (int gr = 0; gr < NG; gr++) {
#pragma unroll
            for (int i = 0; i < 8; i++) x[gr][i] = 0.0f;
            if (r < a.R) widen<8>(q + gr * 32, x[gr]);
        }
    }
    // The same from a block of 8 rows in shared memory.
    template <typename TQ>
    static __device__ __forceinline__ void load_query(const Args &a, const TQ *q, int r0, Query &x)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
#pragma unroll
        for (int gr = 0; gr < NG; gr++) {
#pragma unroll
            for (int i = 0; i < 8; i++) x[gr][i] = 0.0f;
            if (r0 + g < a.R) widen<8>(q + g * D + gr * 32 + j * 8, x[gr]);
        }
    }

    static __device__ __forceinline__ float pow2(int e)  // 2^e, -126 <= e <= 127
    {
        return __int_as_float((e + 127) << 23);
    }

    // Starts block t, query rows r0 .., of a request of N tokens. Row r sees tokens before
    // N - Lq + 1 + r / G (all when !causal).
    __device__ __forceinline__ void open(const Args &a, Query &q, int t, int r0, int N, bool causal)
    {
        const int lane = threadIdx.x & 31, j = lane & 3;
        // the sign of the scale goes into the query; scale 0 makes the query 0
        const float kscale = fabsf(a.scale), sign = a.scale < 0.0f ? -1.0f : a.scale > 0.0f ? 1.0f : 0.0f;
        if (t == 0) lim_min = causal ? N - a.Lq + 1 + r0 / a.G : INT32_MAX;
        float (&x)[NG][8] = q;
        float amax = 0.0f, odd = 0.0f;
#pragma unroll
        for (int gr = 0; gr < NG; gr++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                amax = fmaxf(amax, fabsf(x[gr][i]));
                odd = fmaf(x[gr][i], 0.0f, odd);  // NaN for a query that is not finite
            }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
            odd += __shfl_xor_sync(kFull, odd, o);
        }
        // scaled by a power of two so that the largest channel lies in [2^13, 2^14): fp16
        // then holds a bf16 query exactly down to 2^-30 of it. 2^up as a product of two
        // factors (up is -114 .. 139; a denormal row is scaled as 2^-126 would be)
        const int up = amax > 0.0f && odd == 0.0f ? 13 + 127 - max((int)(__float_as_uint(amax) >> 23), 1) : 0;
        const float f0 = pow2(up >> 1) * sign, f1 = pow2(up - (up >> 1));
        float qs[NG];
#pragma unroll
        for (int gr = 0; gr < NG; gr++) {
            qs[gr] = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                x[gr][i] = odd == 0.0f ? x[gr][i] * f0 * f1 : odd;
                qs[gr] += x[gr][i];
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) qs[gr] += __shfl_xor_sync(kFull, qs[gr], o);
            qs[gr] *= 1.0f / 64.0f;  // 32 channels of 2^14 pass fp16; given back in span_of()
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float f = (i & 1) ? 0.0625f : 1.0f;
                const float u = x[gr][i] * f, v = x[gr][i + 4] * f;
                qf[t][gr][i] = half2_of(u, v);
                if constexpr (Q2) {
                    const float2 w = floats_of(qf[t][gr][i]);
                    ql[t][gr][i] = half2_of(u - w.x, v - w.y);
                }
            }
        }
        // sums of q as three fp16 terms along the product's channels: with 4 groups, k = 0-3,
        // 4-7 and 8-11; with 2, k = 0-1, 2-3 and 4-5
        uint32_t part[3][NG / 2];
#pragma unroll
        for (int gr = 0; gr < NG; gr += 2) {
            float u = qs[gr], v = qs[gr + 1];
#pragma unroll
            for (int k = 0; k < 3; k++) {
                part[k][gr / 2] = half2_of(u, v);
                const float2 w = floats_of(part[k][gr / 2]);
                u -= w.x;
                v -= w.y;
            }
        }
        if constexpr (NG == 4) {
            qz[t][0] = j == 0 ? part[0][0] : j == 1 ? part[0][1] : j == 2 ? part[1][0] : part[1][1];
            qz[t][1] = j == 0 ? part[2][0] : j == 1 ? part[2][1] : 0u;
        } else {
            qz[t][0] = j == 0 ? part[0][0] : j == 1 ? part[1][0] : j == 2 ? part[2][0] : 0u;
            qz[t][1] = 0u;
        }
        // (log2 e comes last: with a scale of 3e38 it would pass fp32, whatever the query)
        const int ke = -up;  // -139 .. 114, in two factors
        // (below 2^-110 all logits vanish: x is under 2^50, and a factor of 0 would make a masked
        // score's -inf a NaN, as an infinite one a difference of 0)
        const float k = kscale == 0.0f ? 1.0f : fminf(fmaxf(kscale * pow2(ke >> 1) * pow2(ke - (ke >> 1)) * kLog2e, 0x1p-110f), FLT_MAX);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            kq[t][i] = __shfl_sync(kFull, k, (2 * j + i) * 4);
            lim[t][i] = causal ? N - a.Lq + 1 + min(r0 + 2 * j + i, a.R - 1) / a.G : INT32_MAX;
            top[t][i] = kept[t][i] = kEmpty;
#pragma unroll
            for (int gr = 0; gr < NG; gr++)
#pragma unroll
                for (int u = 0; u < 2; u++) O[t][gr][u][i] = O[t][gr][u][i + 2] = 0.0f;
        }
        zo[t][0] = zo[t][1] = zo[t][2] = zo[t][3] = 0.0f;
        folds = 0;
    }

    // The sums of the last tiles added to the merge rows (which hold the
    // earlier ones against `kept`).
    __device__ __forceinline__ void fold()
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
        const float up0 = EXACT ? 1.0f : 0x1p24f, up1 = up0 * 0.0625f;
#pragma unroll
        for (int t = 0; t < NT; t++) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const float f = ex2((kept[t][i] - top[t][i]) * kq[t][i]);
                kept[t][i] = top[t][i];
#pragma unroll
                for (int gr = 0; gr < NG; gr++) {
                    float(&o)[2][4] = O[t][gr];
                    float4 *p = reinterpret_cast<float4 *>(rows + (8 * t + 2 * j + i) * ROW + gr * 32 + g * 4);
                    float4 v = make_float4(o[0][i] * up0, o[0][i + 2] * up1, o[1][i] * up0, o[1][i + 2] * up1);
                    // row gr of the z product, columns 2j and 2j + 1
                    const float z = __shfl_sync(kFull, zo[t][i], gr * 4 + j);
                    v = make_float4(v.x + z, v.y + z, v.z + z, v.w + z);
                    if (folds > 0) fma4(v, f, *p);
                    *p = v;
                    o[0][i] = o[0][i + 2] = o[1][i] = o[1][i + 2] = 0.0f;
                }
                float l = zo[t][i + 2];
                if constexpr (EXACT) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(kFull, l, o);
                }
                if (g == 0) {
                    float2 *p = stat + (threadIdx.x >> 5) * RT + 8 * t + 2 * j + i;
                    *p = make_float2(fmaf(top[t][i], kq[t][i], -kExp), folds > 0 ? fmaf(p->y, f, l) : l);
                }
            }
            zo[t][0] = zo[t][1] = zo[t][2] = zo[t][3] = 0.0f;
        }
        folds++;
    }

    // 32 tokens: rows of codes and parameters in shared memory; bit t of
    // `live`: token t counts; base: position of the first.
    __device__ __forceinline__ void span(const uint8_t *kc, const uint8_t *vc, const uint8_t *par,
                                         uint32_t live, int base)
    {
        if (live != 0xffffffffu || base + kSpan > lim_min) span_of<true>(kc, vc, par, live, base);
        else span_of<false>(kc, vc, par, live, base);
    }

    // The two tiles go through every step side by side: with one tile at a time a
    // warp waits for its own products (128K tokens, 9 warps an SM: 60.1 us, side by
    // side 55.0 us).
    template <bool MASKED>
    __device__ __forceinline__ void span_of(const uint8_t *kc, const uint8_t *vc, const uint8_t *par,
                                            uint32_t live, int base)
    {
        constexpr int H = kSpan / kTile;
        const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
        const int t0 = token_of_row(g);  // and t0 + 8, of each tile
        // ---- scores
        float x[NT][H][4];
#pragma unroll
        for (int h = 0; h < H; h++) {
            uint32_t ks[2][NG / 2], kz[2][NG / 2], wa[NG], wb[NG];
            const uint8_t *k = kc + (h * kTile + t0) * Q4<D>::CB, *pr = par + (h * kTile + t0) * Q4<D>::PB;
            if constexpr (NG == 4) {
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(pr + 8 * i * Q4<D>::PB);
                    ks[i][0] = u.x; ks[i][1] = u.y; kz[i][0] = u.z; kz[i][1] = u.w;
                }
                const uint4 u = *reinterpret_cast<const uint4 *>(k + j * 16);
                const uint4 v = *reinterpret_cast<const uint4 *>(k + 8 * Q4<D>::CB + j * 16);
                wa[0] = u.x; wa[1] = u.y; wa[2] = u.z; wa[3] = u.w;
                wb[0] = v.x; wb[1] = v.y; wb[2] = v.z; wb[3] = v.w;
            } else {
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(pr + 8 * i * Q4<D>::PB);
                    ks[i][0] = u.x; kz[i][0] = u.y;
                }
                const uint2 u = *reinterpret_cast<const uint2 *>(k + j * 8);
                const uint2 v = *reinterpret_cast<const uint2 *>(k + 8 * Q4<D>::CB + j * 8);
                wa[0] = u.x; wa[1] = u.y;
                wb[0] = v.x; wb[1] = v.y;
            }
            const uint32_t za = NG == 4 && (j & 1) ? kz[0][NG / 2 - 1] : kz[0][0];
            const uint32_t zb = NG == 4 && (j & 1) ? kz[1][NG / 2 - 1] : kz[1][0];
#pragma unroll
            for (int t = 0; t < NT; t++) {
                float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_f16(z, za, zb, za, zb, qz[t][0], qz[t][1]);
#pragma unroll
                for (int i = 0; i < 4; i++) x[t][h][i] = z[i] * 64.0f;
            }
#pragma unroll
            for (int gr = 0; gr < NG; gr++) {
                uint32_t ra[4], rb[4];
                unpack<true>(wa[gr], ra);
                unpack<true>(wb[gr], rb);
                const float2 sa2 = floats_of(ks[0][gr / 2]), sb2 = floats_of(ks[1][gr / 2]);
                const float sa = (gr & 1) ? sa2.y : sa2.x, sb = (gr & 1) ? sb2.y : sb2.x;
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    if constexpr (Q2) {
                        mma_f16(d, ra[0], rb[0], ra[1], rb[1], ql[t][gr][0], ql[t][gr][1]);
                        mma_f16(d, ra[2], rb[2], ra[3], rb[3], ql[t][gr][2], ql[t][gr][3]);
                    }
                    mma_f16(d, ra[0], rb[0], ra[1], rb[1], qf[t][gr][0], qf[t][gr][1]);
                    mma_f16(d, ra[2], rb[2], ra[3], rb[3], qf[t][gr][2], qf[t][gr][3]);
                    x[t][h][0] = fmaf(sa, d[0], x[t][h][0]);
                    x[t][h][1] = fmaf(sa, d[1], x[t][h][1]);
                    x[t][h][2] = fmaf(sb, d[2], x[t][h][2]);
                    x[t][h][3] = fmaf(sb, d[3], x[t][h][3]);
                }
            }
        }
        // ---- the values' scales, of T(2j), T(2j + 1) and those + 8, where the transposed
        // probabilities lie
        const int ta = token_of_row(2 * j), tb = token_of_row(2 * j + 1);
        uint32_t vs[H][4][NG / 2];
#pragma unroll
        for (int h = 0; h < H; h++)
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int t = h * kTile + ((i & 1) ? tb : ta) + 8 * (i >> 1);
                const uint8_t *pr = par + t * Q4<D>::PB + Q4<D>::PB / 2;
                if constexpr (NG == 4) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(pr);
                    vs[h][i][0] = v.x; vs[h][i][1] = v.y;
                } else {
                    vs[h][i][0] = *reinterpret_cast<const uint32_t *>(pr);
                }
                // what lies in shared memory behind the list has no scales
                if (MASKED && !((live >> t) & 1u)) {
#pragma unroll
                    for (int k = 0; k < NG / 2; k++) vs[h][i][k] = 0u;
                }
            }
        // ---- probabilities against the running maximum
        if (MASKED) {
#pragma unroll
            for (int h = 0; h < H; h++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int at = h * kTile + t0 + 8 * (i >> 1);
#pragma unroll
                    for (int t = 0; t < NT; t++)
                        if (!((live >> at) & 1u) || base + at >= lim[t][i & 1]) x[t][h][i] = -INFINITY;
                }
        }
        float y[NT][H][4];
        auto against = [&]() {
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int h = 0; h < H; h++)
#pragma unroll
                    for (int i = 0; i < 4; i++) y[t][h][i] = fmaf(x[t][h][i] - top[t][i & 1], kq[t][i & 1], kExp);
        };
        against();
        float over = y[0][0][0];
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int h = 0; h < H; h++)
#pragma unroll
                for (int i = 0; i < 4; i++) over = fmaxf(over, y[t][h][i]);
        const bool raise = over > kExp + kSlack;
        // scales of 2 and more (or negative ones, or NaN), and a group whose scales are all under 2^-11
        // (EXACT: 2^-7), want units of their own: the top bits of the scales' OR. A group of zeros alone, or of
        // tokens that are masked, passes the first test and not the second.
        constexpr uint32_t kLow = EXACT ? 0x2000u : 0x1000u;  // 2^-7, 2^-11 as fp16 bits
        uint32_t bits[NG / 2], odd_bits = 0;
#pragma unroll
        for (int k = 0; k < NG / 2; k++) {
            bits[k] = 0;
#pragma unroll
            for (int h = 0; h < H; h++)
#pragma unroll
                for (int i = 0; i < 4; i++) bits[k] |= vs[h][i][k];
            const uint32_t top = bits[k] & (0x10001u * (0x10000u - kLow));
            odd_bits |= ((bits[k] << 1) & 0x80008000u) | bits[k] | ((top - 0x10001u * kLow) & ~top);
        }
        bool odd = (odd_bits & 0x80008000u) != 0u;
        if (__any_sync(kFull, raise || odd)) {
            if (__any_sync(kFull, raise)) {
                raise_top(x);
                against();
            }
            odd = false;
#pragma unroll
            for (int k = 0; k < NG / 2; k++)
                odd = odd || (bits[k] & 0xc000c000u) || (bits[k] & 0xffffu) - 1u < kLow - 1u || (bits[k] >> 16) - 1u < kLow - 1u;
            odd = __any_sync(kFull, odd);
        } else {
            odd = false;
        }
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int h = 0; h < H; h++) {
#pragma unroll
                for (int i = 0; i < 4; i++) x[t][h][i] = ex2(y[t][h][i]);
                if constexpr (EXACT) {
                    zo[t][2] += x[t][h][0] + x[t][h][2];
                    zo[t][3] += x[t][h][1] + x[t][h][3];
                }
            }
        // ---- values: tokens T(2j), T(2j + 1) and those + 8, channels 4g .. 4g + 3 of each group
        uint32_t va[H][NG], vb[H][NG];
#pragma unroll
        for (int h = 0; h < H; h++) {
            const uint8_t *vr = vc + h * kTile * Q4<D>::CB;
            if constexpr (NG == 4) {
                auto at = [&](int t) { return *reinterpret_cast<const uint2 *>(vr + t * Q4<D>::CB + g * 8); };
                const uint2 p0 = at(ta), p1 = at(tb), p2 = at(ta + 8), p3 = at(tb + 8);
                va[h][0] = __byte_perm(p0.x, p1.x, 0x5410); va[h][1] = __byte_perm(p0.x, p1.x, 0x7632);
                va[h][2] = __byte_perm(p0.y, p1.y, 0x5410); va[h][3] = __byte_perm(p0.y, p1.y, 0x7632);
                vb[h][0] = __byte_perm(p2.x, p3.x, 0x5410); vb[h][1] = __byte_perm(p2.x, p3.x, 0x7632);
                vb[h][2] = __byte_perm(p2.y, p3.y, 0x5410); vb[h][3] = __byte_perm(p2.y, p3.y, 0x7632);
            } else {
                auto at = [&](int t) { return *reinterpret_cast<const uint32_t *>(vr + t * Q4<D>::CB + g * 4); };
                const uint32_t p0 = at(ta), p1 = at(tb), p2 = at(ta + 8), p3 = at(tb + 8);
                va[h][0] = __byte_perm(p0, p1, 0x5410); va[h][1] = __byte_perm(p0, p1, 0x7632);
                vb[h][0] = __byte_perm(p2, p3, 0x5410); vb[h][1] = __byte_perm(p2, p3, 0x7632);
            }
        }
        // probabilities as the 8-column operand (and, EXACT, what fp16 leaves of them)
        uint32_t b[NT][H][2], bl[NT][EXACT ? H : 1][2];
#pragma unroll
        for (int h = 0; h < H; h++) {
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float u = x[t][h][2 * i], v = x[t][h][2 * i + 1];
                    const uint32_t p = half2_of(u, v);
                    b[t][h][i] = transpose8(p);
                    if constexpr (EXACT) {
                        const float2 w = floats_of(p);
                        bl[t][h][i] = transpose8(half2_of(u - w.x, v - w.y));
                    }
                }
            // zeros: row g of the 16-row operand is group g mod NG
            const uint8_t *pz = par + h * kTile * Q4<D>::PB + Q4<D>::PB / 2 + 2 * NG + (g & (NG - 1)) * 2;
            auto at = [&](int t) {
                uint32_t z = *reinterpret_cast<const uint16_t *>(pz + t * Q4<D>::PB);
                // behind the list, or NaN (a row that sees the token has it from the scale)
                if (MASKED && (!((live >> (h * kTile + t)) & 1u) || (z & 0x7fffu) > 0x7c00u)) z = 0;
                return z;
            };
            const uint32_t za = __byte_perm(at(ta), at(tb), 0x5410), zb = __byte_perm(at(ta + 8), at(tb + 8), 0x5410);
            constexpr uint32_t one = EXACT ? 0u : 0x3c003c00u;
#pragma unroll
            for (int t = 0; t < NT; t++) {
                if constexpr (EXACT) {
                    float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma_f16(z, za, one, zb, one, bl[t][h][0], bl[t][h][1]);
                    mma_f16(z, za, one, zb, one, b[t][h][0], b[t][h][1]);
                    zo[t][0] += z[0];
                    zo[t][1] += z[1];
                } else {
                    mma_f16(zo[t], za, one, zb, one, b[t][h][0], b[t][h][1]);
                }
            }
        }
        if (odd) values<MASKED, true>(va, vb, vs, b, bl, live, base);
        else values<MASKED, false>(va, vb, vs, b, bl, live, base);
    }

    // The weighted codes of a span. ODD: the products of a group are computed in fp32 and rounded to fp16
    // in units of a power of two per row and group, in which the row's largest product in the span lies in
    // [2^13, 2^14). Probabilities are up to 2^14, so a product with a scale of 2 and more could
    // pass fp16, and with small scales the products would sink under its smallest numbers. The product and not the
    // scale decides: a large value that a row gives no weight leaves its other tokens as they are.
    template <bool MASKED, bool ODD>
    __device__ __forceinline__ void values(const uint32_t (&va)[kSpan / kTile][NG], const uint32_t (&vb)[kSpan / kTile][NG],
                                           const uint32_t (&vs)[kSpan / kTile][4][NG / 2],
                                           const uint32_t (&b)[NT][kSpan / kTile][2],
                                           const uint32_t (&bl)[NT][EXACT ? kSpan / kTile : 1][2],
                                           uint32_t live, int base)
    {
        constexpr int H = kSpan / kTile;
        const int g = (threadIdx.x & 31) >> 2, ta = token_of_row(2 * (threadIdx.x & 3)), tb = token_of_row(2 * (threadIdx.x & 3) + 1);
        uint32_t seen[NT];  // the tokens that row g of a block sees
#pragma unroll
        for (int t = 0; t < NT; t++) {
            seen[t] = live;
            if (MASKED && ODD) {
                const int even = __shfl_sync(kFull, lim[t][0], g >> 1), other = __shfl_sync(kFull, lim[t][1], g >> 1);
                const int n = ((g & 1) ? other : even) - base;
                seen[t] = live & (n <= 0 ? 0u : n >= kSpan ? 0xffffffffu : (1u << n) - 1u);
            }
        }
        constexpr bool FRESH = EXACT || ODD;  // a tile's products are summed from 0, and added in fp32
#pragma unroll
        for (int gr = 0; gr < NG; gr++) {
            const uint32_t sel = (gr & 1) ? 0x7632 : 0x5410;
            auto scales = [&](int h, int i) { return __byte_perm(vs[h][2 * i][gr / 2], vs[h][2 * i + 1][gr / 2], sel); };
            auto product = [&](int t, int h, int i) {  // in fp32, of the lane's row and two tokens
                float2 p = floats_of(b[t][h][i]);
                const float2 sc = floats_of(scales(h, i));
                if constexpr (EXACT) {
                    const float2 r = floats_of(bl[t][h][i]);
                    p = make_float2(p.x + r.x, p.y + r.y);
                }
                return make_float2(p.x * sc.x, p.y * sc.y);
            };
            float unit[NT], back[NT][2];  // factor of the lane's row's products; of the sums of columns 2j, 2j + 1
            if constexpr (ODD) {
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    float m = 0.0f;  // (fmaxf passes over NaN)
#pragma unroll
                    for (int h = 0; h < H; h++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            const float2 v = product(t, h, i);
                            m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
                        }
                    m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
                    // 2^-48 .. 2^31
                    const int e = m > 0.0f ? min(max((int)(__float_as_uint(m) >> 23) - 127 - 13, -62), 18) : 0;
                    unit[t] = pow2(-e);
#pragma unroll
                    for (int i = 0; i < 2; i++) back[t][i] = pow2(__shfl_sync(kFull, e, (2 * (int)(threadIdx.x & 3) + i) * 4));
                }
            }
#pragma unroll
            for (int h = 0; h < H; h++) {
                uint32_t ra[4], rb[4];
                unpack<EXACT>(va[h][gr], ra);
                unpack<EXACT>(vb[h][gr], rb);
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    uint32_t u[2], l[2];
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        l[i] = 0u;
                        if constexpr (ODD) {
                            float2 v = product(t, h, i);
                            v = make_float2(v.x * unit[t], v.y * unit[t]);
                            u[i] = half2_of(v.x, v.y);
                            if constexpr (EXACT) {
                                const float2 w = floats_of(u[i]);
                                l[i] = half2_of(v.x - w.x, v.y - w.y);
                            }
                        } else {
                            const __half2 p = as_half2(b[t][h][i]), sc = as_half2(scales(h, i)), ps = __hmul2(p, sc);
                            u[i] = *reinterpret_cast<const uint32_t *>(&ps);
                            if constexpr (EXACT) {
                                const __half2 rest = __hfma2(as_half2(bl[t][h][i]), sc, __hfma2(p, sc, __hneg2(ps)));
                                l[i] = *reinterpret_cast<const uint32_t *>(&rest);
                            }
                        }
                        if (MASKED && ODD) {  // (NaN scales are odd)
                            // a token that the row does not see does not enter it, whatever its values are; one that
                            // it sees does, a NaN of a probability of 0 too
                            const uint32_t two = seen[t] >> (h * kTile + 8 * i);
                            const uint32_t enter = ((two >> ta) & 1u ? 0xffffu : 0u) | ((two >> tb) & 1u ? 0xffff0000u : 0u);
                            u[i] &= enter;
                            l[i] &= enter;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        float(&o)[4] = FRESH ? w : O[t][gr][k];
                        if constexpr (EXACT) mma_f16(o, ra[2 * k], ra[2 * k + 1], rb[2 * k], rb[2 * k + 1], l[0], l[1]);
                        mma_f16(o, ra[2 * k], ra[2 * k + 1], rb[2 * k], rb[2 * k + 1], u[0], u[1]);
                        if constexpr (FRESH) {
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                if constexpr (ODD) O[t][gr][k][i] = fmaf(w[i], back[t][i & 1], O[t][gr][k][i]);
                                else O[t][gr][k][i] += w[i];
                            }
                        }
                    }
                }
            }
        }
    }

    // A logit passed the running maximum by the slack (rare): a new one.
    __device__ __forceinline__ void raise_top(const float (&x)[NT][kSpan / kTile][4])
    {
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                float m = fmaxf(fmaxf(x[t][0][i], x[t][0][i + 2]), fmaxf(x[t][1][i], x[t][1][i + 2]));
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                const float r = fmaxf(m, top[t][i]);
                // nothing summed yet: the old one may be any
                const float f = top[t][i] == kEmpty ? 0.0f : ex2((top[t][i] - r) * kq[t][i]);
                top[t][i] = r;
                zo[t][i] *= f;
                zo[t][i + 2] *= f;
#pragma unroll
                for (int gr = 0; gr < NG; gr++)
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        O[t][gr][u][i] *= f;
                        O[t][gr][u][i + 2] *= f;
                    }
            }
    }

    // This warp's totals into its merge rows.
    __device__ __forceinline__ void finish() { fold(); }

    // Channels ch .. ch + 3 of a row over the CTA's warps (after finish() and a barrier).
    static __device__ __forceinline__ float4 merged(const uint8_t *smem, int row, int ch, float &m, float &l)
    {
        const float *mr = reinterpret_cast<const float *>(smem);
        const float2 *st = reinterpret_cast<const float2 *>(smem + MERGE);
        m = kEmpty;
        l = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; w++)
            if (st[w * RT + row].y != 0.0f) m = fmaxf(m, st[w * RT + row].x);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < WARPS; w++) {
            const float2 s = st[w * RT + row];
            const float f = s.y == 0.0f ? 0.0f : ex2(s.x - m);
            l = fmaf(f, s.y, l);
            fma4(o, f, *reinterpret_cast<const float4 *>(mr + (w * RT + row) * ROW + ch));
        }
        return o;
    }
};

inline Args make_args(const kvr_q4_cache &c, const Q4AttendArgs &s, int RT)
{
    Args a;
    a.c = q4_pages(c);
    a.B = s.B;
    a.Lq = s.Lq;
    a.Hq = s.Hq;
    a.G = s.Hq / c.Hkv;
    a.R = a.G * s.Lq;
    a.RB = (a.R + RT - 1) / RT;
    a.q_stride = s.q_stride;
    a.max_pages = s.max_pages;
    a.cap = s.max_pages * c.page_size;
    a.q = s.q;
    a.table = s.table;
    a.seq_len = s.seq_len;
    a.scale = s.scale;
    a.out = s.out;
    a.out_bf16 = s.out_dtype == KVR_BF16;
    a.err = s.err;
    return a;
}

}  // namespace q4a

}  // namespace kvr
