// kvr_q4_list.cuh -- attention over the paged 4-bit cache where a cluster takes a
// unit's whole list at once: selected tokens (a list, the first `sink` tokens and
// those from the window or region end on), and all tokens of short requests.
//
// A unit (request, KV head, block of query rows) belongs to a cluster of CTAs, as
// many as let all units run at once and still give every warp a span (with more units
// than SMs to a CTA of fewer warps); its
// list is dealt to the cluster's warps in 32-token spans. A warp looks the
// list and the pages up ahead of its two stages and gathers the rows with
// cp.async (a token's K codes, V codes and parameters lie in whole 32-byte
// sectors at d = 128: 160 bytes move for 160 read). The warps of a CTA merge in
// its shared memory; each CTA then sends its part of every output to the CTA that
// writes it (distributed shared memory), and one barrier later that one adds
// the parts up in the order of the CTAs. One launch, no workspace.
//
// What bounds it is the chain of dependent reads (length, list, page, rows: 0.6, 1.0 and
// 0.9 us), then the products (0.5 us), the two merges and the barrier (2 us). 2048 selected
// tokens and a window of 128 of a 128K request (8 KV heads): 8.2 us, for 0.4 us of bytes. With 16 CTAs a
// unit, of which seven clusters and not eight are resident, it took 14.3 us for 7.5 at that time.
#pragma once

#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "kvr_q4_rows.cuh"

namespace kvr {
namespace q4a {

constexpr int kListWarps = 12;  // of a CTA, one CTA an SM
constexpr int kFewWarps = 4;    // of a CTA of which three share an SM
constexpr int kMaxCluster = 16;
// Spans of a warp up to which all tokens of a request go this way rather than through
// the dense kernel, which needs a second one to merge. bf16, d = 128, this way and that:
// 8 units of 4096 tokens (one span) 8.4 and 10.0 us, 64 of 2048 (three) 12.4 and 14.6,
// 128 of 1024 (three) 10.6 and 15.5; of four spans, 8 units of 16000 14.6 and 13.3.
// (The lengths are on the device, so what counts is what the page table has room for: short requests under a
// wide table go the other way.)
constexpr int kListSteps = 3;

// With more units than SMs a unit is a CTA of four warps, three to an SM, while its list gives a warp
// no more spans than this. bf16, d = 128, 192 units: 120 tokens 6.7 us so and 11.4 through the dense
// kernel, 380 9.0 to 10.9 and 15.8, 1000 17.4 and 19.7, 1400 (12 spans) both 22.6; 3200 units of 380 tokens 81
// and 128. Selected tokens, and with CTAs of 12 warps: 192 lists of 428 11.7 and 15.5, of 1128 23.4 and 26.0.
constexpr int kFewSteps = 10;

struct ListArgs : Args {
    int sparse;  // else all tokens
    const int32_t *idx, *count, *region_end;
    int kmax, W, sink;
};

template <int D, bool Q2, bool EXACT, int W> struct List {
    static constexpr int THREADS = 32 * W, CTAS = kListWarps / W;  // CTAs of an SM
    using R = Rows<D, Q2, EXACT, W, 1>;
    static constexpr int STAGE = kSpan * Q4<D>::TB;
    static constexpr int S = 2;
    static constexpr int RING = W * S * STAGE;
    static constexpr int ITEMS = R::RT * D / 4;  // 4 channels of a row: what a thread merges
    // parts sent to this CTA: [CTA][slot], slots = ceil(ITEMS / CTAs); then [CTA][row] references, sums
    static constexpr int RECV = (ITEMS + kMaxCluster) * 16;
    static constexpr int SMEM = RING + R::MERGE + R::STAT + RECV + kMaxCluster * R::RT * 8;
};

template <int D, bool Q2, bool EXACT, int W, typename TQ>
__global__ void __launch_bounds__(32 * W, kListWarps / W) list_q4_kernel(ListArgs a)
{
    namespace cg = cooperative_groups;
    using C = List<D, Q2, EXACT, W>;
    using Rw = typename C::R;
    constexpr int S = C::S, RT = Rw::RT, LR = D / 4;
    extern __shared__ __align__(128) uint8_t sm[];
    uint8_t *merge = sm + C::RING;
    float4 *recv = reinterpret_cast<float4 *>(merge + Rw::MERGE + Rw::STAT);
    float2 *recv_stat = reinterpret_cast<float2 *>(merge + Rw::MERGE + Rw::STAT + C::RECV);
    __shared__ uint32_t masks[W][S];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int CL = gridDim.x, rank = blockIdx.x;  // the cluster spans the grid's x
    const int e = blockIdx.y, b = e / a.c.Hkv, h = e % a.c.Hkv, rb = blockIdx.z;
    const int stride = CL * W, mine = rank * W + warp;
    if (CL > 1) cluster_arrive_release();  // waited for before the first write to another CTA
    grid_dependency_wait();
    grid_launch_dependents();

    typename Rw::Query query;
    Rw::template load_query<TQ>(a, b, h, rb * RT, query);

    // ---- the unit's list. The first span's listed tokens are read beside the length, as if the
    // sink were full
    const int first = mine * kSpan + lane - a.sink;
    const int guess = a.sparse && first >= 0 && first < a.kmax ? a.idx[(int64_t)e * a.kmax + first] : -1;
    int N = a.seq_len[b], count = a.sparse ? a.count[e] : 0;
    int64_t end = 0;
    if (a.sparse) end = a.region_end ? (int64_t)a.region_end[b] : (int64_t)N - a.W;
    if (N < 0 || N > a.cap) {
        set_err(a.err, KVR_DEVERR_SEQ_LEN);
        N = 0;
    }
    const int sink = a.sparse ? min(a.sink, N) : 0, rest = (int)min(max(end, (int64_t)sink), (int64_t)N);
    count = N > 0 ? min(max(count, 0), a.kmax) : 0;
    const int64_t n = (int64_t)sink + count + (N - rest);
    const int64_t spans = (n + kSpan - 1) / kSpan;
    const int steps = spans > mine ? (int)((spans - mine - 1) / stride) + 1 : 0;

    // ---- copies, two look-ups ahead of the stages: list entry, page, rows
    int pos = -1, lo = 0, hi = 0, page = -1, off = 0, looked = 0;
    uint8_t *ring = sm + warp * S * C::STAGE;
    const int ps_log2 = a.c.ps_log2, ps = 1 << ps_log2;
    const int64_t block = (int64_t)Q4<D>::TB << ps_log2;
    auto read_list = [&]() {  // the entry of this lane's token, and the bounds of a listed one
        pos = -1;
        lo = 0;
        hi = INT32_MAX;
        if (looked < steps) {
            int64_t i = (mine + (int64_t)looked * stride) * kSpan + lane;
            if (i < n) {
                if (i < sink) {
                    pos = (int)i;
                } else if ((i -= sink) < count) {
                    pos = looked == 0 && sink == a.sink ? guess : a.idx[(int64_t)e * a.kmax + i];
                    lo = sink;
                    hi = rest;
                } else {
                    pos = (int)(rest + i - count);
                }
            }
        }
        looked++;
    };
    auto read_page = [&]() {
        const bool in = pos >= lo && pos < hi;
        if (!in && hi != INT32_MAX) set_err(a.err, KVR_DEVERR_INDEX);
        page = -1;
        if (in) {
            page = a.table[(int64_t)b * a.max_pages + (pos >> ps_log2)];
            off = pos & (ps - 1);
            if (page < 0) page = INT32_MAX;
        }
    };
    auto copy_rows = [&](int stage) {
        if (page >= a.c.n_pages) {
            set_err(a.err, KVR_DEVERR_PAGE);
            page = -1;
        }
        const uint32_t live = __ballot_sync(kFull, page >= 0);
        if (lane == 0) masks[warp][stage] = live;
        if (live) {
            uint8_t *dst = ring + stage * C::STAGE;
            constexpr int KC = Q4<D>::CB / 16;  // 16-byte pieces of a code row: 4 or 2
            constexpr int PC = Q4<D>::PB / 16;  // of a token's parameters: 2 or 1
#pragma unroll
            for (int i = 0; i < KC; i++) {
                const int t = (i * 32 + lane) / KC, p = lane % KC;
                const int pg = __shfl_sync(kFull, page, t), of = __shfl_sync(kFull, off, t);
                if (pg >= 0) {
                    const uint8_t *src = a.c.base + ((int64_t)pg * a.c.Hkv + h) * block + of * Q4<D>::CB + p * 16;
                    uint8_t *to = dst + t * Q4<D>::CB + p * 16;
                    cp_async16(to, src);
                    cp_async16(to + kSpan * Q4<D>::CB, src + ps * Q4<D>::CB);
                }
            }
#pragma unroll
            for (int i = 0; i < PC; i++) {
                const int t = (i * 32 + lane) / PC, p = lane % PC;
                const int pg = __shfl_sync(kFull, page, t), of = __shfl_sync(kFull, off, t);
                if (pg >= 0)
                    cp_async16(dst + kSpan * 2 * Q4<D>::CB + t * Q4<D>::PB + p * 16,
                               a.c.base + ((int64_t)pg * a.c.Hkv + h) * block + (int64_t)ps * 2 * Q4<D>::CB +
                                   of * Q4<D>::PB + p * 16);
            }
        }
        cp_async_commit();
    };
    read_list();
    read_page();
    read_list();
#pragma unroll
    for (int s = 0; s < S; s++) {
        copy_rows(s);
        read_page();
        read_list();
    }

    Rw rows;
    rows.attach(merge, warp);
    rows.open(a, query, 0, rb * RT, N, !a.sparse);
    int stage = 0, since = 0;
    for (int i = 0; i < steps; i++) {
        cp_async_wait<S - 1>();
        __syncwarp();
        const uint32_t live = masks[warp][stage];
        const uint8_t *p = ring + stage * C::STAGE;
        if (live)
            rows.span(p, p + kSpan * Q4<D>::CB, p + 2 * kSpan * Q4<D>::CB, live,
                      a.sparse ? 0 : (mine + i * stride) * kSpan);
        __syncwarp();
        copy_rows(stage);
        read_page();
        read_list();
        stage = stage == S - 1 ? 0 : stage + 1;
        if (++since == Rw::FOLD) {
            rows.fold();
            since = 0;
        }
    }
    cp_async_wait<0>();

    // ---- the CTA's rows, then the cluster's
    rows.finish();
    __syncthreads();
    cg::cluster_group cluster = cg::this_cluster();
    const int slots = (C::ITEMS + CL - 1) / CL;
    if (CL > 1) cluster_wait_acquire();  // every CTA of the cluster runs
    for (int x = tid; x < C::ITEMS; x += C::THREADS) {
        const int row = x / LR, ch = x % LR * 4, r = rb * RT + row;
        float m, l;
        const float4 o = Rw::merged(merge, row, ch, m, l);
        if (CL == 1) {
            if (r < a.R) store4(a, out_at(a, b, h, r, D) + ch, o, l == 0.0f ? 0.0f : 1.0f / l);
        } else {
            // CTA x mod CL writes this item
            cluster.map_shared_rank(recv, x % CL)[rank * slots + x / CL] = o;
            if (ch == 0)
                for (int k = 0; k < CL; k++) cluster.map_shared_rank(recv_stat, k)[rank * RT + row] = make_float2(m, l);
        }
    }
    if (CL == 1) return;
    __syncthreads();
    cluster_arrive_release();
    cluster_wait_acquire();
    for (int s = tid; s < slots; s += C::THREADS) {
        const int x = s * CL + rank, row = x / LR, ch = x % LR * 4, r = rb * RT + row;
        if (x >= C::ITEMS || r >= a.R) continue;
        float m = kEmpty, l = 0.0f;
        for (int k = 0; k < CL; k++)
            if (recv_stat[k * RT + row].y != 0.0f) m = fmaxf(m, recv_stat[k * RT + row].x);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k = 0; k < CL; k++) {
            const float2 st = recv_stat[k * RT + row];
            const float f = st.y == 0.0f ? 0.0f : ex2(st.x - m);
            l = fmaf(f, st.y, l);
            fma4(o, f, recv[k * slots + s]);
        }
        store4(a, out_at(a, b, h, r, D) + ch, o, l == 0.0f ? 0.0f : 1.0f / l);
    }
}

// Clusters of `cl` CTAs of a kernel that are resident at once (asked once per device).
template <int D, bool Q2, bool EXACT, typename TQ> int resident(int cl)
{
    static std::atomic<int> known[64][kMaxCluster + 1];  // 0: not asked
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev][cl].load(std::memory_order_relaxed);
    if (n == 0) {
        n = 1 + max_active_clusters((const void *)list_q4_kernel<D, Q2, EXACT, kListWarps, TQ>, cl, 32 * kListWarps,
                                    List<D, Q2, EXACT, kListWarps>::SMEM);
        known[dev][cl].store(n, std::memory_order_relaxed);
    }
    return n - 1;
}

template <int D, bool Q2, bool EXACT, int W, typename TQ>
kvr_status enqueue_list(const ListArgs &a, int cl, cudaStream_t stream)
{
    using C = List<D, Q2, EXACT, W>;
    const auto kern = list_q4_kernel<D, Q2, EXACT, W, TQ>;
    const kvr_status st = prepare_cluster_kernel((const void *)kern, C::SMEM);
    if (st != KVR_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cl, a.B * a.c.Hkv, a.RB);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cl;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
        (void)cudaGetLastError();
        return KVR_ERR_CUDA;
    }
    return check_launch();
}

// The call runs here if it is sparse, or if its lists, as long as the page table allows, give a warp few
// spans; else nothing is done and *taken is false.
template <int D, bool Q2, bool EXACT, typename TQ>
kvr_status launch_list(const kvr_q4_cache &c, const Q4AttendArgs &s, cudaStream_t stream, bool *taken)
{
    ListArgs a;
    static_cast<Args &>(a) = make_args(c, s, Rows<D, Q2, EXACT, kListWarps, 1>::RT);
    a.sparse = s.sparse;
    a.idx = s.idx;
    a.count = s.count;
    a.region_end = s.region_end;
    a.kmax = s.kmax;
    a.W = s.W;
    a.sink = s.sink;
    *taken = s.sparse;
    // the longest list a unit can have (with a region end, as long as the cache)
    const int64_t list = s.sparse && !s.region_end ? std::min(a.cap, (int64_t)s.kmax + s.W + s.sink) : a.cap;
    const int64_t units = (int64_t)s.B * c.Hkv * a.RB, spans = std::max<int64_t>(1, (list + kSpan - 1) / kSpan);
    if (units > sm_count() && spans <= kFewSteps * kFewWarps) {
        *taken = true;
        return enqueue_list<D, Q2, EXACT, kFewWarps, TQ>(a, 1, stream);
    }
    if (!s.sparse && (units > sm_count() || spans > kListSteps * kListWarps * kMaxCluster)) return KVR_OK;
    const kvr_status st = prepare_cluster_kernel((const void *)list_q4_kernel<D, Q2, EXACT, kListWarps, TQ>,
                                                 List<D, Q2, EXACT, kListWarps>::SMEM);
    if (st != KVR_OK) return st;
    // the largest cluster with which all units are resident at once and every warp gets a span
    int cl = (int)std::min<int64_t>(kMaxCluster, (spans + kListWarps - 1) / kListWarps);
    while (cl > 1 && resident<D, Q2, EXACT, TQ>(cl) < units) cl--;
    if (!s.sparse) {
        if (spans > kListSteps * kListWarps * cl) return KVR_OK;
        *taken = true;
    }
    return enqueue_list<D, Q2, EXACT, kListWarps, TQ>(a, cl, stream);
}

template <int D>
kvr_status list_d(const kvr_q4_cache &c, const Q4AttendArgs &s, cudaStream_t stream, bool *taken)
{
    if (s.q_dtype == KVR_F32) return launch_list<D, true, true, float>(c, s, stream, taken);
    return s.out_dtype == KVR_F32 ? launch_list<D, false, true, __nv_bfloat16>(c, s, stream, taken)
                                  : launch_list<D, false, false, __nv_bfloat16>(c, s, stream, taken);
}

}  // namespace q4a
}  // namespace kvr
