// kvr_q4.cu -- rows into and out of the paged 4-bit K/V cache.
//
//   append_q4_kernel  quantises new K and V rows and writes codes and
//                     parameters at their slots
//   read_q4_kernel    the values that the slots' codes stand for
//
// Both are bound by memory: a token and head moves 4 D bytes of bf16 rows
// (8 D of fp32) on one side and 5 D / 4 bytes on the other.
#include "kvr_paged.h"
#include "kvr_q4.cuh"

namespace kvr {

namespace {

constexpr int kQ4Threads = 256;

// (page, offset) of a slot; false for a negative slot (a padding row) and,
// with the error bit, for one past the pool.
__device__ __forceinline__ bool q4_locate(const Q4Pages &c, int64_t slot, int64_t &page, int &off,
                                          int32_t *err)
{
    if (slot < 0) return false;
    page = slot >> c.ps_log2;
    off = (int)(slot & ((1 << c.ps_log2) - 1));
    if (page >= c.n_pages) {
        set_err(err, KVR_DEVERR_POSITION);
        return false;
    }
    return true;
}

// The least and greatest channel of a lane's 8 (as raw 16 or 32 bytes).
struct Range {
    float mn, mx;
};
__device__ __forceinline__ Range lane_range(const float (&x)[8])
{
    Range r;
    range8(x, r.mn, r.mx);
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        r.mn = min_nan(r.mn, __shfl_xor_sync(kFull, r.mn, o));
        r.mx = max_nan(r.mx, __shfl_xor_sync(kFull, r.mx, o));
    }
    return r;
}

// bf16: pairs side by side; across lanes the maximum and the negated minimum as one pair.
__device__ __forceinline__ Range pair_range(const uint4 &v)
{
    auto b2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
    __nv_bfloat162 mn = __hmin2_nan(__hmin2_nan(b2(v.x), b2(v.y)), __hmin2_nan(b2(v.z), b2(v.w)));
    __nv_bfloat162 mx = __hmax2_nan(__hmax2_nan(b2(v.x), b2(v.y)), __hmax2_nan(b2(v.z), b2(v.w)));
    const uint32_t n = *reinterpret_cast<const uint32_t *>(&mn), m = *reinterpret_cast<const uint32_t *>(&mx);
    // (max of the low halves, -min of the low halves) and the same of the high ones
    const uint32_t neg = n ^ 0x80008000u;
    uint32_t p = __byte_perm(m, neg, 0x5410), q = __byte_perm(m, neg, 0x7632);
    __nv_bfloat162 r = __hmax2_nan(b2(p), b2(q));
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        const uint32_t w = __shfl_xor_sync(kFull, *reinterpret_cast<const uint32_t *>(&r), o);
        r = __hmax2_nan(r, b2(w));
    }
    const uint32_t w = *reinterpret_cast<const uint32_t *>(&r);
    return Range{-bf16_hi(w), bf16_lo(w)};
}

// 8 channels of a row as loaded: bf16 in one register quad, fp32 in two.
template <typename T> struct Raw {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++) v[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; i++) v[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const
    {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[sizeof(T) / 2 - 1].x, v[sizeof(T) / 2 - 1].y,
                               v[sizeof(T) / 2 - 1].z, v[sizeof(T) / 2 - 1].w};
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
            else x[i] = (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        }
    }
    __device__ __forceinline__ Range range() const
    {
        if constexpr (sizeof(T) == 2) {
            return pair_range(v[0]);
        } else {
            float x[8];
            widen(x);
            return lane_range(x);
        }
    }
};

// What a run of D / 8 lanes takes: heads h and h + 1 of a token.
struct Pair {
    uint32_t t;
    int h, off;
    int64_t page;
    bool live, both;   // the token has a slot; head h + 1 exists
};
template <int D>
__device__ __forceinline__ Pair pair_of(const Q4Pages &c, const int64_t *slots, uint32_t pairs, int32_t *err)
{
    const uint32_t hp = (uint32_t)(c.Hkv + 1) / 2;
    const uint32_t p = (uint32_t)(((uint64_t)blockIdx.x * kQ4Threads + threadIdx.x) / (D / 8));
    Pair r;
    r.live = p < pairs;
    r.t = r.live ? p / hp : 0u;
    r.h = 2 * (int)(r.live ? p - r.t * hp : 0u);
    r.both = r.h + 1 < c.Hkv;
    r.page = r.off = 0;
    if (r.live) r.live = q4_locate(c, slots[r.t], r.page, r.off, threadIdx.x % (D / 8) == 0 ? err : nullptr);
    return r;
}

// 8 channels of K and of V of two heads per lane. A group is 4 lanes, which have four
// groups at hand; each lane finds scale and zero of one (40 of some 70
// instructions a group), the others get them by shuffles. 131072 tokens of 8 heads of
// bf16: 204 us with one head per lane and every lane finding both of its groups'
// parameters, 123 us so (5.7 TB/s; reading back 117 us); of fp32 427 us with their read back (5.9 TB/s).
template <int D, typename T>
__global__ void __launch_bounds__(kQ4Threads)
append_q4_kernel(Q4Pages c, const T *__restrict__ K, int64_t k_stride, const T *__restrict__ V,
                 int64_t v_stride, const int64_t *__restrict__ slots, uint32_t pairs, int32_t *err)
{
    constexpr int L = D / 8, NG = Q4<D>::NG;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lr = threadIdx.x % L, g = lr / 4, j = lr % 4;
    const Pair p = pair_of<D>(c, slots, pairs, err);
    Raw<T> x[4];         // K, V of the first head, K, V of the second
#pragma unroll
    for (int i = 0; i < 4; i++) x[i].zero();
    if (p.live) {
        const T *k = K + p.t * k_stride + p.h * D + lr * 8, *v = V + p.t * v_stride + p.h * D + lr * 8;
        x[0].load(k);
        x[1].load(v);
        if (p.both) {
            x[2].load(k + D);
            x[3].load(v + D);
        }
    }
    float mn = 0.0f, mx = 0.0f;  // of the group this lane answers for: x[j]
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const Range a = x[i].range();
        if (i == j) {
            mn = a.mn;
            mx = a.mx;
        }
    }
    __half sh, zh;
    const bool ok = q4_params<sizeof(T) == 4>(mn, mx, sh, zh);
    const float s = __half2float(sh), zero = __half2float(zh);
    const float inv = !ok ? -1.0f : s > 0.0f ? __frcp_rn(s) : 0.0f;
    if (!ok && p.live) set_err(err, KVR_DEVERR_RANGE);
    const bool plain = __all_sync(kFull, ok && q4_step(mx, zero, inv) <= kMagic + 15u);
    uint32_t code[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int from = (threadIdx.x & 28) + i;
        const float zi = __shfl_sync(kFull, zero, from), vi = __shfl_sync(kFull, inv, from);
        float y[8];
        x[i].widen(y);
        code[i] = plain ? q4_codes8(y, zi, vi) : q4_codes8_any(y, zi, vi);
    }
    // neighbouring groups' scales and zeros: even ones store the pair of scales, odd ones of zeros
    const uint32_t mine = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(zh) << 16);
    const uint32_t next = __shfl_xor_sync(kFull, mine, 4);
    const uint32_t both = (g & 1) ? __byte_perm(next, mine, 0x7632) : __byte_perm(mine, next, 0x5410);
    // a V word holds the 4 codes of two neighbouring groups: even groups take the pair's first
    // runs, odd ones the second
#pragma unroll
    for (int i = 1; i < 4; i += 2) {
        const uint32_t other = __shfl_xor_sync(kFull, (g & 1) ? code[i] & 0xffffu : code[i] >> 16, 4);
        code[i] = (g & 1) ? __byte_perm(other, code[i], 0x7610) : __byte_perm(code[i], other, 0x5410);
    }
    if (!p.live) return;
    const int ps = 1 << c.ps_log2;
    uint8_t *blk = q4_block<D>(c, p.page, p.h) + (size_t)p.off * Q4<D>::CB;
    const int64_t block = (int64_t)Q4<D>::TB << c.ps_log2;
    const int kw = (j * NG + g) * 4, vw = ps * Q4<D>::CB + ((2 * j + (g & 1)) * NG + (g & ~1)) * 2;
    *reinterpret_cast<uint32_t *>(blk + kw) = code[0];
    *reinterpret_cast<uint32_t *>(blk + vw) = code[1];
    if (p.both) {
        *reinterpret_cast<uint32_t *>(blk + block + kw) = code[2];
        *reinterpret_cast<uint32_t *>(blk + block + vw) = code[3];
    }
    if (j < 2 || p.both)
        *reinterpret_cast<uint32_t *>(blk + (j < 2 ? 0 : block) + ps * 2 * Q4<D>::CB -
                                      p.off * (Q4<D>::CB - Q4<D>::PB) +
                                      (((j & 1) * 2 + (g & 1)) * (NG / 2) + g / 2) * 4) = both;
}

__device__ __forceinline__ void store8(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Values of 8 codes. A nibble under 2^23's exponent is 2^23 + c 16^k where it
// lies (k < 4: no shift, and a conversion instruction would run at an eighth of the rate);
// 16^k goes into the scale.
__device__ __forceinline__ void values8(uint32_t w, float s, float z, float (&x)[8])
{
    float sk = s;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const uint32_t m = 15u << (4 * k);
        x[k] = fmaf(__uint_as_float((w & m) | 0x4b000000u) - 8388608.0f, sk, z);
        x[k + 4] = fmaf(__uint_as_float(((w >> 16) & m) | 0x4b000000u) - 8388608.0f, sk, z);
        sk *= 0.0625f;
    }
}

// 8 channels of K and of V of two heads per lane: ten loads in flight.
template <int D, typename T>
__global__ void __launch_bounds__(kQ4Threads)
read_q4_kernel(Q4Pages c, const int64_t *__restrict__ slots, uint32_t pairs, T *__restrict__ K,
               int64_t k_stride, T *__restrict__ V, int64_t v_stride, int32_t *err)
{
    constexpr int L = D / 8, NG = Q4<D>::NG;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lr = threadIdx.x % L, g = lr / 4, j = lr % 4;
    const Pair p = pair_of<D>(c, slots, pairs, err);
    uint32_t kw[2] = {0, 0}, vw[2] = {0, 0};
    uint16_t par[2][4] = {};  // K s, K z, V s, V z
    if (p.live) {
        const int ps = 1 << c.ps_log2;
        const uint8_t *blk = q4_block<D>(c, p.page, p.h) + (size_t)p.off * Q4<D>::CB;
        const int64_t block = (int64_t)Q4<D>::TB << c.ps_log2;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (i == 0 || p.both) {
                kw[i] = *reinterpret_cast<const uint32_t *>(blk + (j * NG + g) * 4);
                vw[i] = *reinterpret_cast<const uint32_t *>(blk + ps * Q4<D>::CB + ((2 * j + (g & 1)) * NG + (g & ~1)) * 2);
                const uint16_t *q = reinterpret_cast<const uint16_t *>(blk + ps * 2 * Q4<D>::CB - p.off * (Q4<D>::CB - Q4<D>::PB)) + g;
#pragma unroll
                for (int k = 0; k < 4; k++) par[i][k] = q[k * NG];
            }
            blk += block;
        }
    }
    T *k = K + p.t * k_stride + p.h * D + lr * 8, *v = V + p.t * v_stride + p.h * D + lr * 8;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        // a V word holds 4 codes of two neighbouring groups (see the append kernel)
        const uint32_t other = __shfl_xor_sync(kFull, (g & 1) ? vw[i] & 0xffffu : vw[i] >> 16, 4);
        const uint32_t w = (g & 1) ? __byte_perm(other, vw[i], 0x7610) : __byte_perm(vw[i], other, 0x5410);
        if (!p.live || (i == 1 && !p.both)) continue;
        float x[8];
        values8(kw[i], __half2float(__ushort_as_half(par[i][0])), __half2float(__ushort_as_half(par[i][1])), x);
        store8(k + i * D, x);
        values8(w, __half2float(__ushort_as_half(par[i][2])), __half2float(__ushort_as_half(par[i][3])), x);
        store8(v + i * D, x);
    }
}

template <int D> dim3 pairs_grid(uint32_t pairs)
{
    return dim3((unsigned)(((uint64_t)pairs * (D / 8) + kQ4Threads - 1) / kQ4Threads));
}

template <int D, typename T>
kvr_status append_t(const Q4Pages &c, const void *K, int64_t ks, const void *V, int64_t vs,
                    const int64_t *slot, int64_t n, int32_t *err, cudaStream_t stream)
{
    const uint32_t pairs = (uint32_t)(n * ((c.Hkv + 1) / 2));
    return launch_pdl(append_q4_kernel<D, T>, pairs_grid<D>(pairs), kQ4Threads, 0, stream, c,
                      static_cast<const T *>(K), ks, static_cast<const T *>(V), vs, slot, pairs, err);
}

template <int D, typename T>
kvr_status read_t(const Q4Pages &c, const int64_t *slot, int64_t n, void *K, int64_t ks, void *V,
                  int64_t vs, int32_t *err, cudaStream_t stream)
{
    const uint32_t pairs = (uint32_t)(n * ((c.Hkv + 1) / 2));
    return launch_pdl(read_q4_kernel<D, T>, pairs_grid<D>(pairs), kQ4Threads, 0, stream, c, slot, pairs,
                      static_cast<T *>(K), ks, static_cast<T *>(V), vs, err);
}

}  // namespace

Q4Pages q4_pages(const kvr_q4_cache &c)
{
    int l = 0;
    while ((1 << l) < c.page_size) l++;
    return Q4Pages{c.pages, c.n_pages, l, c.Hkv};
}

kvr_status append_q4_dispatch(const kvr_q4_cache &c, kvr_dtype dt, const void *K, int64_t ks,
                              const void *V, int64_t vs, const int64_t *slot, int64_t n, int32_t *err,
                              cudaStream_t stream)
{
    const Q4Pages p = q4_pages(c);
    if (c.d == 128)
        return dt == KVR_BF16 ? append_t<128, __nv_bfloat16>(p, K, ks, V, vs, slot, n, err, stream)
                              : append_t<128, float>(p, K, ks, V, vs, slot, n, err, stream);
    return dt == KVR_BF16 ? append_t<64, __nv_bfloat16>(p, K, ks, V, vs, slot, n, err, stream)
                          : append_t<64, float>(p, K, ks, V, vs, slot, n, err, stream);
}

kvr_status read_q4_dispatch(const kvr_q4_cache &c, kvr_dtype dt, const int64_t *slot, int64_t n,
                            void *K, int64_t ks, void *V, int64_t vs, int32_t *err,
                            cudaStream_t stream)
{
    const Q4Pages p = q4_pages(c);
    if (c.d == 128)
        return dt == KVR_BF16 ? read_t<128, __nv_bfloat16>(p, slot, n, K, ks, V, vs, err, stream)
                              : read_t<128, float>(p, slot, n, K, ks, V, vs, err, stream);
    return dt == KVR_BF16 ? read_t<64, __nv_bfloat16>(p, slot, n, K, ks, V, vs, err, stream)
                          : read_t<64, float>(p, slot, n, K, ks, V, vs, err, stream);
}

}  // namespace kvr
