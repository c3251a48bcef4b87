// kvr_q4_dense.cuh -- attention of every request's newest tokens over all of
// its tokens in the paged 4-bit cache.
//
// Work: the token lists of all units (request, KV head, block of query rows)
// are cut into chunks of 352 (or 224) tokens, and the CTAs of one resident wave take
// equal runs of them, whatever the lengths (each CTA sums the lengths itself).
// One warp of a CTA looks pages up and fills a ring of chunks with bulk copies (a
// page holds a head's codes and parameters in three contiguous pieces); eleven (or
// seven) warps take 32 tokens of a chunk each, keep their own softmax state and are
// merged at the end of a unit. A unit that a run's end cuts leaves partial results in
// the workspace, which combine_q4_kernel merges in the order of the CTAs: the
// same bits every time.
//
// A million tokens of 8 KV heads, d = 128, bf16: 238 us, 5.6 TB/s (0.83 of the
// measured copy); copies without the computation take 195 us, the computation without
// the copies took 229 us. So the computation bounds it, but by latency and not by a unit that is full:
// three warps a scheduler use half of the issue slots and 46% of the integer pipe, and wait for operands,
// shared memory and the tensor pipe (20%) in between. With fp32 outputs it is 321 us, with fp32 queries 358.
// 128K tokens: 43 us, of which 4.6 us go by until the first chunk has landed
// and 3.7 us after the last, in the two merges and the second launch. A unit that is opened and closed
// costs some 3 us of a CTA: 60000 requests of 16 tokens, one KV head, take 2.4 ms.
#pragma once

#include <algorithm>

#include "kvr_q4_rows.cuh"

namespace kvr {
namespace q4a {

// One warp issues a bulk copy in about 50 ns, three a page. Pages of 64 tokens and more leave it
// idle part of a chunk's time (1.2 us at the bandwidth of memory). Of smaller ones every
// warp copies its own 32 tokens, 16 bytes a lane: a million tokens (bf16) in pages of 32 take 288 us
// so, in pages of 64 272 us, and 287 if the warps copied those too. (With bulk copies of the
// warps' own, pages of 32 took 15% longer.)
constexpr int kOwnCopies = 32;              // pages of up to so many tokens

// An arrival at an mbarrier of this CTA.
__device__ __forceinline__ void mbar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

struct DenseArgs : Args {
    int32_t *meta;   // [grid][4]: request, block, CTAs (0: no cut unit starts here), slot of the first
    float *part;     // [grid][2][RT][D + 2]: rows of o, then reference and sum
};

// Computing warps: with the copying one three a scheduler at 168 registers or, for two blocks of
// query rows a warp (NT), two a scheduler at 255.
template <int D, bool Q2, bool EXACT, int NT, typename TQ> struct Dense {
    static constexpr int kWarps = NT == 1 ? 11 : 7;
    static constexpr int kChunk = kSpan * kWarps;      // tokens of a chunk
    static constexpr int kThreads = 32 * (kWarps + 1); // and the warp that copies
    static constexpr int kPieces = kChunk / kTile;     // a page holds whole 16-token pieces
    static_assert(kPieces <= 32, "a lane per piece");
    using R = Rows<D, Q2, EXACT, kWarps, NT>;
    static constexpr int STAGE = kChunk * Q4<D>::TB;     // K codes, V codes, parameters of a chunk
    static constexpr int S = 3 * (128 / D);  // chunks in the ring
    static constexpr int P = 2 * S;          // places: pages are looked up that far ahead
    // a block of query rows per place; fp32 ones, which would not fit, are read where they are
    static constexpr int QUERY = Q2 ? 0 : R::RT * D * (int)sizeof(TQ);
    static constexpr int SMEM = S * STAGE + P * QUERY + R::MERGE + R::STAT;
};

// A chunk's place, from the copying warp to the others.
struct Chunk {
    int b, h, rb, N;
    int base;     // position of the chunk's first token
    int flags;    // kOpen: first chunk of its unit in this run; kClose: last
    int slot;     // at kClose: -1 the unit is whole, else the partial to fill
    uint32_t bad; // bit l: the page of the chunk's 16-token piece l is outside the pool
};
constexpr int kOpen = 1, kClose = 2, kLast = 4, kNone = 8;  // kLast: the run's last chunk; kNone: an empty run

__device__ __forceinline__ int request_len(const Args &a, int b)
{
    const int N = a.seq_len[b];
    if (N >= 0 && N <= a.cap) return N;
    set_err(a.err, KVR_DEVERR_SEQ_LEN);
    return 0;
}

template <int CHUNK> __device__ __forceinline__ int chunks_in(int n) { return n > 0 ? (n - 1) / CHUNK + 1 : 1; }

// A unit is as long as its chunks and kUnitCost more: opening and closing one
// takes a CTA about as long as that many chunks, and a run of short requests
// would otherwise end long after the others.
constexpr int kUnitCost = 2;

// Start of run i among n over `total`, and the run that holds position x.
__device__ __forceinline__ int64_t run_start(int64_t total, int i, int n)
{
    // 64-bit divisions take hundreds of instructions
    return total < (1 << 20) ? (int64_t)((uint32_t)total * (uint32_t)i / (uint32_t)n) : total * i / n;
}
__device__ __forceinline__ int run_of(int64_t total, int64_t x, int n) { return (int)(((x + 1) * n - 1) / total); }

__device__ __forceinline__ int64_t warp_sum64(int64_t x)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

// A 16-token tile's codes and parameters into tokens t .. of a chunk's stage, 16 bytes a lane and step.
template <int D, int kChunk>
__device__ __forceinline__ void copy_tile(uint8_t *stage, int t, const uint8_t *k, const uint8_t *v,
                                          const uint8_t *par, int lane)
{
#pragma unroll
    for (int i = lane * 16; i < kTile * Q4<D>::CB; i += 32 * 16) {
        cp_async16(stage + t * Q4<D>::CB + i, k + i);
        cp_async16(stage + (kChunk + t) * Q4<D>::CB + i, v + i);
    }
    if (lane * 16 < kTile * Q4<D>::PB)
        cp_async16(stage + 2 * kChunk * Q4<D>::CB + t * Q4<D>::PB + lane * 16, par + lane * 16);
}

template <int D, bool Q2, bool EXACT, bool OWN, int NT, typename TQ>
__global__ void __launch_bounds__(Dense<D, Q2, EXACT, NT, TQ>::kThreads, 1) dense_q4_kernel(DenseArgs a)
{
    using C = Dense<D, Q2, EXACT, NT, TQ>;
    using Rw = typename C::R;
    constexpr int S = C::S, P = C::P, RT = Rw::RT;
    constexpr int kWarps = C::kWarps, kChunk = C::kChunk, kPieces = C::kPieces;
    extern __shared__ __align__(128) uint8_t sm[];
    uint8_t *queries = sm + S * C::STAGE, *merge = queries + P * C::QUERY;
    // whole: a chunk has landed (the copying warp's copies); ready: a place is filled (the warps copy);
    // empty: all warps are through with a place's chunk
    __shared__ __align__(8) uint64_t whole[S], ready[P], empty[P], meet;
    __shared__ __align__(16) Chunk place[P];
    __shared__ const uint8_t *piece[P][kPieces];  // first byte of a piece in its page, or null

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr bool own = OWN;  // pages of up to kOwnCopies tokens
    if (tid == 0) {
        for (int s = 0; s < S; s++) mbar_init(&whole[s], 1);
        for (int k = 0; k < P; k++) {
            mbar_init(&ready[k], 1);
            mbar_init(&empty[k], kWarps);
            place[k] = Chunk{};
        }
        mbar_init(&meet, kWarps);
        mbar_fence_init();
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();

    if (warp == kWarps) {
        // ================= the copying warp: this CTA's run of chunks
        const int units = a.c.Hkv * a.RB;  // of a request
        const int ps_log2 = a.c.ps_log2, ps = 1 << ps_log2;
        const int64_t block = (int64_t)Q4<D>::TB << ps_log2;
        int32_t *meta = a.meta + 4 * blockIdx.x;
        auto length = [&](int e) { return e < a.B ? request_len(a, e) : -1; };
        auto weight = [&](int n) { return n < 0 ? (int64_t)0 : (int64_t)(chunks_in<kChunk>(n) + kUnitCost) * units; };
        int N = length(lane);
        int64_t total = weight(N);
        for (int e = lane + 32; e < a.B; e += 32) total += weight(request_len(a, e));
        total = warp_sum64(total);
        const int runs = (int)min((int64_t)gridDim.x, total), run = blockIdx.x;
        const int64_t w0 = run < runs ? run_start(total, run, runs) : total;
        const int64_t w1 = run < runs ? run_start(total, run + 1, runs) : total;
        // the request that holds w0
        int b = a.B;
        int64_t unit_at = 0;   // position of the unit at hand
        for (int e0 = 0; e0 < a.B && run < runs; e0 += 32) {
            if (e0 > 0) N = length(e0 + lane);
            const int64_t w = weight(N);
            int64_t incl = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(kFull, incl, o);
                incl += lane >= o ? y : 0;
            }
            const uint32_t here = __ballot_sync(kFull, w0 < unit_at + incl);
            if (here) {
                const int src = __ffs(here) - 1;
                b = e0 + src;
                unit_at += __shfl_sync(kFull, incl - w, src);
                N = __shfl_sync(kFull, N, src);
                break;
            }
            unit_at += __shfl_sync(kFull, incl, 31);
        }
        int chunks = 1, u = 0, c = 0;
        bool any = b < a.B;
        auto next_unit = [&]() {
            unit_at += chunks + kUnitCost;
            c = 0;
            if (++u == units) {
                u = 0;
                if (++b < a.B) {
                    N = request_len(a, b);
                    chunks = chunks_in<kChunk>(N);
                }
            }
        };
        if (any) {
            chunks = chunks_in<kChunk>(N);
            const int64_t into = w0 - unit_at;
            const int one = chunks + kUnitCost;
            u = into < INT32_MAX ? (int)into / one : (int)(into / one);
            c = (int)(into - (int64_t)u * one);
            unit_at += (int64_t)u * one;
            if (c >= chunks) next_unit();
            any = b < a.B && unit_at + c < w1;
        }
        if (!any) {
            if (lane == 0) {
                meta[2] = 0;
                place[0].flags = kLast | kNone;
                mbar_arrive(own ? &ready[0] : &whole[0]);
            }
            return;
        }
        // A lane looks up the page of one piece, a chunk ahead: -1 behind the request
        auto look = [&]() {
            const int64_t at = (int64_t)c * kChunk + lane * kTile;
            if (lane >= kPieces || at >= N) return -1;
            const int page = a.table[(int64_t)b * a.max_pages + (at >> ps_log2)];
            return page < 0 ? INT32_MAX : page;
        };
        int next = look();
        int from = c;          // chunk at which the run enters the unit at hand
        bool first = true;     // it is the run's first unit
        bool ok = true;
        int s = 0, k = 0;                // stage and place of the chunk
        uint32_t lap = 0, round = 0;     // times the stages and the places were gone round
        for (;;) {
            // the chunk whose stage (or, where the warps copy, whose place) this one takes is done
            if (own ? round > 0 : lap > 0) {
                const int e = own ? k : k >= S ? k - S : k + P - S;
                const uint32_t turn = own || k < S ? round - 1 : round;
                ok = __all_sync(kFull, mbar_wait(&empty[e], turn & 1, a.err));
            }
            if (!ok) break;
            int page = next;
            int bytes_of = 0;
            const uint32_t bad = __ballot_sync(kFull, page >= a.c.n_pages);  // entries outside the pool
            if (page >= a.c.n_pages) {
                set_err(a.err, KVR_DEVERR_PAGE);
                page = -1;
            }
            const bool unit_ends = c + 1 == chunks;
            const bool run_ends = (unit_ends ? unit_at + chunks + kUnitCost : unit_at + c + 1) >= w1;
            const int h = u / a.RB, rb = u - h * a.RB;
            const int base = c * kChunk, stop = min(base + kChunk, N);
            const int pos = base + lane * kTile, off = pos & (ps - 1);  // of the lane's piece
            const uint8_t *src = nullptr;
            if (page >= 0)
                src = a.c.base + ((int64_t)page * a.c.Hkv + h) * block + (int64_t)off * Q4<D>::CB;
            // the query rows of a unit come with its first chunk; those of one token are contiguous,
            // a lane copies its token's
            int q_first = 0, q_rows = 0, q_token = 0;
            const int r0 = rb * RT, q_all = !Q2 && c == from ? min(RT, a.R - r0) * C::QUERY / RT : 0;
            if (!Q2 && c == from) {
                q_token = r0 / a.G + lane;
                q_first = max(r0, q_token * a.G);
                q_rows = min(min(r0 + RT, a.R), (q_token + 1) * a.G) - q_first;
            }
            uint64_t *bar = own ? &ready[k] : &whole[s];
            if (own && lane < kPieces) piece[k][lane] = src;
            // a lane copies from its piece on what the chunk has of the page
            int n = 0;
            if (!own) {
                if (page >= 0 && (lane == 0 || off == 0)) n = min(ps - off, stop - pos);
                bytes_of = __reduce_add_sync(kFull, n) * Q4<D>::TB;
            }
            __syncwarp();
            if (lane == 0) {
                Chunk p;
                p.b = b;
                p.h = h;
                p.rb = rb;
                p.N = N;
                p.base = base;
                p.flags = (c == from ? kOpen : 0) | (unit_ends || run_ends ? kClose : 0) | (run_ends ? kLast : 0);
                p.slot = from == 0 && unit_ends ? -1 : first ? 0 : 1;
                p.bad = bad;
                place[k] = p;
                mbar_arrive_expect_tx(bar, (uint32_t)(bytes_of + q_all));
            }
            __syncwarp();
            if (q_rows > 0)
                bulk_g2s(queries + k * C::QUERY + (q_first - r0) * (C::QUERY / RT),
                         static_cast<const TQ *>(a.q) + ((int64_t)b * a.Lq + q_token) * a.q_stride +
                             (int64_t)(h * a.G + q_first - q_token * a.G) * D,
                         q_rows * (C::QUERY / RT), bar);
            if (n > 0) {
                uint8_t *dst = sm + s * C::STAGE;
                const int at = pos - base;
                bulk_g2s(dst + at * Q4<D>::CB, src, n * Q4<D>::CB, bar);
                bulk_g2s(dst + (kChunk + at) * Q4<D>::CB, src + ps * Q4<D>::CB, n * Q4<D>::CB, bar);
                bulk_g2s(dst + 2 * kChunk * Q4<D>::CB + at * Q4<D>::PB,
                         src + ps * 2 * Q4<D>::CB - off * (Q4<D>::CB - Q4<D>::PB), n * Q4<D>::PB, bar);
            }
            if (run_ends) {
                // a unit that starts here and goes on in later CTAs is merged from here
                if (lane == 0) {
                    meta[0] = b;
                    meta[1] = u;
                    meta[2] = from == 0 && !unit_ends ? run_of(total, unit_at + chunks - 1, runs) - run + 1 : 0;
                    meta[3] = first ? 0 : 1;
                }
                break;
            }
            if (unit_ends) {
                next_unit();
                from = 0;
                first = false;
            } else {
                c++;
            }
            next = look();
            if (++s == S) {
                s = 0;
                lap++;
            }
            if (++k == P) {
                k = 0;
                round++;
            }
        }
        // The CTA's shared memory is held until the last copies have landed
        if (ok) {
            const int last = own ? k : s;
            const uint32_t turns = own ? round : lap;
            for (int i = 0; i < (own ? P : S); i++)
                if (i <= last || turns > 0)
                    mbar_wait(own ? &ready[i] : &whole[i], (i <= last ? turns : turns - 1) & 1, a.err);
        } else {  // after a wait that ran out: nothing to merge
            if (lane == 0) meta[2] = 0;
            for (int i = 0; i < (own ? P : S); i++)
                for (uint32_t par = 0; par < 2; par++) mbar_wait(own ? &ready[i] : &whole[i], par, a.err);
        }
        return;
    }

    // ================= the computing warps
    Rw rows;
    rows.attach(merge, warp);
    int spans = 0;
    uint32_t met = 0;
    // After a wait that ran out a warp ends with the chunk at hand (outputs are invalid; its place
    // names a unit, zeros at first), and the others' waits for it run out in turn.
    bool ok = true;
    auto meet_warps = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&meet);
        if (ok) ok = __all_sync(kFull, mbar_wait(&meet, met & 1, a.err));
        met++;
    };
    // A warp's own copies of its 32 tokens of the chunk at place `slot`, into stage `s`.
    bool more = own;       // the run's last chunk is not yet copied
    int issue_slot = 0;
    uint32_t issue_round = 0;
    auto copy_span = [&](int s) {
        ok = __all_sync(kFull, mbar_wait(&ready[issue_slot], issue_round & 1, a.err));
        if (!ok) return;
        const Chunk k = place[issue_slot];
        if (k.flags & kNone) {
            more = false;
            return;
        }
        // whole 16-token tiles: what a page holds behind the request is copied too, and masked
        const int pos = k.base + warp * kSpan, ps = 1 << a.c.ps_log2;
#pragma unroll
        for (int h = 0; h < kSpan / kTile; h++) {
            const uint8_t *src = piece[issue_slot][2 * warp + h];
            if (src) {
                const int off = (pos + h * kTile) & (ps - 1);
                copy_tile<D, kChunk>(sm + s * C::STAGE, warp * kSpan + h * kTile, src, src + ps * Q4<D>::CB,
                             src + ps * 2 * Q4<D>::CB - off * (Q4<D>::CB - Q4<D>::PB), lane);
            }
        }
        more = !(k.flags & kLast);
        if (++issue_slot == P) {
            issue_slot = 0;
            issue_round++;
        }
    };
    auto copy_own = [&](int s) {  // a group per call, so that a wait counts them
        if constexpr (own) {
            if (more && ok) copy_span(s);
            cp_async_commit();
        }
    };
    for (int i = 0; i < S; i++) copy_own(i);
    int s = 0, slot = 0;
    uint32_t lap = 0;
    for (bool last = false; ok && !last;) {
        if (own && !more && issue_slot == 0 && issue_round == 0) return;  // an empty run
        if constexpr (own) {
            cp_async_wait<S - 1>();
            __syncwarp();
        } else {
            ok = __all_sync(kFull, mbar_wait(&whole[s], lap & 1, a.err));
        }
        const Chunk k = place[slot];
        if (k.flags & kNone) return;
        last = k.flags & kLast;
        const int pos = k.base + warp * kSpan, count = min(k.N - pos, kSpan);
        uint32_t bits = count <= 0 ? 0u : 0xffffffffu >> (kSpan - count);  // the warp's tokens that count
        if (k.bad) bits &= ~__ballot_sync(kFull, (k.bad >> ((warp * kSpan + lane) / kTile)) & 1u);
        if (k.flags & kOpen) {
#pragma unroll
            for (int t = 0; t < NT; t++) {
                const int r0 = k.rb * RT + 8 * t;
                typename Rw::Query q;
                if constexpr (Q2) Rw::template load_query<TQ>(a, k.b, k.h, r0, q);
                else Rw::template load_query<TQ>(a, reinterpret_cast<const TQ *>(queries + slot * C::QUERY) + 8 * t * D, r0, q);
                rows.open(a, q, t, r0, k.N, true);
            }
            spans = 0;
        }
        const uint8_t *p = sm + s * C::STAGE + warp * kSpan * Q4<D>::CB;
        if (bits) rows.span(p, p + kChunk * Q4<D>::CB,
                            sm + s * C::STAGE + 2 * kChunk * Q4<D>::CB + warp * kSpan * Q4<D>::PB, bits, pos);
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
        copy_own(s);
        if constexpr (!EXACT) spans++;
        if (k.flags & kClose) {
            rows.finish();
            meet_warps();
            constexpr int LR = D / 4;  // 4 channels per thread
            for (int e = tid; e < RT * LR; e += 32 * kWarps) {
                const int row = e / LR, ch = e % LR * 4, r = k.rb * RT + row;
                float m, l;
                const float4 o = Rw::merged(merge, row, ch, m, l);
                if (k.slot >= 0) {
                    float *q = a.part + ((int64_t)(2 * blockIdx.x + k.slot) * RT + row) * (D + 2);
                    *reinterpret_cast<float2 *>(q + ch) = make_float2(o.x, o.y);
                    *reinterpret_cast<float2 *>(q + ch + 2) = make_float2(o.z, o.w);
                    if (ch == 0) *reinterpret_cast<float2 *>(q + D) = make_float2(m, l);
                } else if (r < a.R) {
                    store4(a, out_at(a, k.b, k.h, r, D) + ch, o, l == 0.0f ? 0.0f : 1.0f / l);
                }
            }
            meet_warps();
        } else if (spans >= Rw::FOLD) {
            rows.fold();
            spans = 0;
        }
        if (++s == S) {
            s = 0;
            lap++;
        }
        if (++slot == P) slot = 0;
    }
    if (own) cp_async_wait<0>();
}

// Merges the partial results of a unit that several CTAs share, in their
// order. Grid: (CTAs of the attention, rows of a block). Each of P thread groups
// takes every P-th partial, kAhead of them in flight.
constexpr int kCombineThreads = 256;

template <int D, int RT>
__global__ void __launch_bounds__(kCombineThreads) combine_q4_kernel(DenseArgs a)
{
    constexpr int LR = D / 4, P = kCombineThreads / LR, kAhead = 4;
    __shared__ float4 so[P][LR];
    __shared__ float2 sl[P];
    grid_dependency_wait();
    grid_launch_dependents();
    const int4 meta = reinterpret_cast<const int4 *>(a.meta)[blockIdx.x];
    const int n = meta.z;
    if (n == 0) return;
    const int b = meta.x, u = meta.y, row = blockIdx.y;
    const int h = u / a.RB, r = u % a.RB * RT + row;
    if (r >= a.R) return;
    const int k0 = threadIdx.x / LR, ch = threadIdx.x % LR * 4;
    float m = kEmpty, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int k = k0; k < n; k += P * kAhead) {
        float2 st[kAhead], v0[kAhead], v1[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            const int part = k + i * P, slot = 2 * ((int)blockIdx.x + part) + (part == 0 ? meta.w : 0);
            const float *p = a.part + ((int64_t)slot * RT + row) * (D + 2);
            st[i] = make_float2(kEmpty, 0.0f);
            v0[i] = v1[i] = make_float2(0.0f, 0.0f);
            if (part < n) {
                st[i] = *reinterpret_cast<const float2 *>(p + D);
                v0[i] = *reinterpret_cast<const float2 *>(p + ch);
                v1[i] = *reinterpret_cast<const float2 *>(p + ch + 2);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
            if (st[i].y == 0.0f) continue;
            const float mn = fmaxf(m, st[i].x), f = l == 0.0f ? 0.0f : ex2(m - mn), w = ex2(st[i].x - mn);
            l = fmaf(w, st[i].y, l * f);
            o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
            fma4(o, w, make_float4(v0[i].x, v0[i].y, v1[i].x, v1[i].y));
            m = mn;
        }
    }
    so[k0][ch / 4] = o;
    if (ch == 0) sl[k0] = make_float2(m, l);
    __syncthreads();
    if (k0 != 0) return;
    m = kEmpty;
#pragma unroll
    for (int k = 0; k < P; k++) m = fmaxf(m, sl[k].x);
    o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < P; k++) {
        const float2 st = sl[k];
        const float f = st.y == 0.0f ? 0.0f : ex2(st.x - m);
        l = fmaf(f, st.y, l);
        fma4(o, f, so[k][ch / 4]);
    }
    store4(a, out_at(a, b, h, r, D) + ch, o, l == 0.0f ? 0.0f : 1.0f / l);
}

template <int D, bool Q2, bool EXACT, int NT, typename TQ>
kvr_status launch_dense(const kvr_q4_cache &c, const Q4AttendArgs &s, cudaStream_t stream)
{
    using C = Dense<D, Q2, EXACT, NT, TQ>;
    DenseArgs a;
    static_cast<Args &>(a) = make_args(c, s, C::R::RT);
    // one resident wave, fewer CTAs when the requests cannot hold that many chunks
    const int64_t per = (a.cap + C::kChunk - 1) / C::kChunk;
    const int grid = (int)std::min((int64_t)sm_count(), (int64_t)s.B * c.Hkv * a.RB * per);
    a.meta = reinterpret_cast<int32_t *>(s.ws);
    a.part = reinterpret_cast<float *>(s.ws + align_up((size_t)grid * 16, 256));
    const auto kern = c.page_size <= kOwnCopies ? dense_q4_kernel<D, Q2, EXACT, true, NT, TQ>
                                                : dense_q4_kernel<D, Q2, EXACT, false, NT, TQ>;
    kvr_status st = raise_smem_limit((const void *)kern, C::SMEM);
    if (st != KVR_OK) return st;
    st = launch_pdl(kern, dim3(grid), C::kThreads, C::SMEM, stream, a);
    if (st != KVR_OK || per == 1) return st;  // a unit of one chunk is never cut
    return launch_pdl(combine_q4_kernel<D, C::R::RT>, dim3(grid, std::min(a.R, C::R::RT)), kCombineThreads, 0,
                      stream, a);
}

// Workspace of any dense launch.
inline size_t dense_ws_bytes(int d)
{
    const size_t grid = (size_t)sm_count();
    return align_up(grid * 16, 256) + grid * 2 * 16 * (d + 2) * 4;
}

// Query rows go 8 at a time, or as two blocks of 8 that share the unpacked codes, in a warp of 255
// registers, seven of them an SM (fp32 queries at d = 128 would need more). A pair takes so much
// longer than a block, in tenths: 12 requests of 16K tokens, 4 KV heads, pages of 64, 16 rows in pairs and by
// blocks: d = 64 39 and 55 us (fp32 outputs 45 and 60, fp32 queries 48 and 58), d = 128 51 and 63 (69
// and 74); 24 rows: 67 and 77 (78 and 85, 83 and 81), 87 and 88 (125 and 104); 56 rows, d = 128: 162 and
// 187 (237 and 224). (At 12 warps an SM the pair spills: 133 us for what took 102 by blocks then.)
constexpr int pair_cost(int d, bool q2, bool exact) { return d == 64 ? (q2 ? 17 : 14) : exact ? 18 : 16; }

template <int D>
kvr_status dense_d(const kvr_q4_cache &c, const Q4AttendArgs &s, cudaStream_t stream)
{
    const int blocks = (s.Hq / c.Hkv * s.Lq + 7) / 8;
    const bool two = (blocks + 1) / 2 * pair_cost(D, s.q_dtype == KVR_F32, s.out_dtype == KVR_F32) < 10 * blocks;
    if constexpr (D == 64) {
        if (two && s.q_dtype == KVR_F32) return launch_dense<D, true, true, 2, float>(c, s, stream);
    }
    if (s.q_dtype == KVR_F32) return launch_dense<D, true, true, 1, float>(c, s, stream);
    if (s.out_dtype == KVR_F32)
        return two ? launch_dense<D, false, true, 2, __nv_bfloat16>(c, s, stream)
                   : launch_dense<D, false, true, 1, __nv_bfloat16>(c, s, stream);
    return two ? launch_dense<D, false, false, 2, __nv_bfloat16>(c, s, stream)
               : launch_dense<D, false, false, 1, __nv_bfloat16>(c, s, stream);
}

}  // namespace q4a
}  // namespace kvr
