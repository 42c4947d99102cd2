// tokens.cu — token rows sorted by expert and back, with the routing weights applied, and the
// gradients of both: the differentiable form of an expert-parallel dispatch and return ("MAX 中
// Step-3.5-Flash 架构解析", section "并行模式TP_TP / TP_EP / DP_EP": experts split over ranks
// with an EP combine after the MoE; NeMo AutoModel Step-5-Preview page: the layer is trained
// with expert parallelism).
//
// With T tokens, k entries each, E experts; entry n = t * k + j has the expert id idx[t, j] and
// is kept when 0 <= id < E:
//   sort             slot_of[t, j] = place of (id, n) among the kept entries in that order, -1
//                    for a dropped entry; offsets[e] = kept entries with id < e;
//                    x_sorted[slot_of[t, j]] = x[t]
//   sort backward    dx[t] = sum_j dx_sorted[slot_of[t, j]]
//   unsort           y[t] = add[t] + sum_j w[t, j] y_sorted[slot_of[t, j]]
//   unsort backward  dy_sorted[slot_of[t, j]] = w[t, j] dy[t],
//                    dw[t, j] = <dy[t], y_sorted[slot_of[t, j]]>
// Every kernel reads and writes each row once and does a handful of operations per element: HBM
// bandwidth bounds the large calls, launch and dependent-load latency the small ones. Sums
// run in fp32, over j in rank order, and round once to the rows' type.
#include <atomic>
#include <type_traits>

#include <cuda_fp16.h>

#include "../../include/moe_b200.h"
#include "context.h"

namespace moe {
namespace {

constexpr int kMaxK = 32;
constexpr int kMaxExperts = 1024;

// ---------------------------------------------------------------------------------- sort
// Small calls, one launch: an entry's place is the number of entries with a smaller key
// id * N + n (N = T * k entries in all), so every block counts for its own token, with no
// dependence between blocks: N compares per entry in place of another launch and the hand-over. Measured
// against the two launches below: 512 entries 2.6 us, where the two launches alone take longer; 3108
// entries of 2 KB rows 6.2 against 5.4 us; 4096 entries of 8 KB rows 9.8 against 10.3 us.
constexpr int kSmallEntries = 2048;
constexpr int kRowThreads = 128;
constexpr int kDroppedKey = 0x7fffffff;

__device__ __forceinline__ int entry_key(int id, int n, int E, int N)
{
    return static_cast<unsigned>(id) < static_cast<unsigned>(E) ? id * N + n : kDroppedKey;
}

// A row (units of U) to the rows slots[0..k) of x_sorted, up to column c1, by LANES threads. Every load of a piece
// (V units per thread) is issued before its k copies are stored; load() may run before the
// slots are known.
template <typename U, int LANES>
struct RowCopy {
    static constexpr int V = sizeof(U) >= 8 ? 4 : 8;
    U v[V];
    __device__ __forceinline__ void load(const U *__restrict__ src, int64_t c, int64_t c1)
    {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i * LANES < c1)
                v[i] = src[c + i * LANES];
    }
    __device__ __forceinline__ void store(U *__restrict__ out, int64_t units, int64_t c, int64_t c1, const int *slots,
                                          int k) const
    {
        for (int j = 0; j < k; ++j) {
            const int64_t s = slots[j];
            if (s < 0)
                continue;
            U *dst = out + s * units;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i * LANES < c1)
                    dst[c + i * LANES] = v[i];
        }
    }
};

// Block 0 of the small sort: offsets[0..E] from a histogram in shared memory.
__device__ __forceinline__ void small_offsets(const int32_t *__restrict__ idx, int N, int E, int32_t *hist,
                                              int32_t *__restrict__ offsets)
{
    __shared__ int warp_sum[kRowThreads / 32];
    for (int e = threadIdx.x; e < kMaxExperts; e += kRowThreads)
        hist[e] = 0;
    __syncthreads();
    for (int n = threadIdx.x; n < N; n += kRowThreads) {
        const int id = idx[n];
        if (static_cast<unsigned>(id) < static_cast<unsigned>(E))
            atomicAdd(&hist[id], 1);  // integer counts: any order gives the same
    }
    __syncthreads();
    constexpr int per = kMaxExperts / kRowThreads;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int c[per], sum = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
        c[i] = hist[threadIdx.x * per + i];
        sum += c[i];
    }
    int incl = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        warp_sum[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w)
        run += warp_sum[w];
#pragma unroll
    for (int i = 0; i < per; ++i) {
        const int e = threadIdx.x * per + i;
        if (e <= E)
            offsets[e] = run;
        run += c[i];
    }
    if (threadIdx.x == kRowThreads - 1 && E == kMaxExperts)
        offsets[E] = run;
}

// Grid (1 + T, chunks): block (0, 0) writes the offsets, block (1 + t, c) the places of token t
// and columns [c, c + 1) * chunk of its rows.
template <typename U>
__global__ void __launch_bounds__(kRowThreads)
    sort_small_kernel(const U *__restrict__ x, const int32_t *__restrict__ idx, int T, int k, int E, int64_t units,
                      int64_t chunk, U *__restrict__ x_sorted, int32_t *__restrict__ offsets,
                      int32_t *__restrict__ slot_of)
{
    __shared__ int32_t tab[kSmallEntries];
    __shared__ int part[kRowThreads / 32][8];
    __shared__ int slots[kMaxK];
    static_assert(kSmallEntries >= kMaxExperts, "the histogram shares the key table");
    const int N = T * k;
    if (blockIdx.x == 0) {
        if (blockIdx.y == 0)
            small_offsets(idx, N, E, tab, offsets);
        return;
    }
    const int t = blockIdx.x - 1;
    const U *src = x + static_cast<int64_t>(t) * units;
    const int64_t c1 = (blockIdx.y + 1) * chunk < units ? (blockIdx.y + 1) * chunk : units;
    int64_t c = blockIdx.y * chunk + threadIdx.x;
    RowCopy<U, kRowThreads> row;
    row.load(src, c, c1);  // on its way while the places are counted
    for (int n = threadIdx.x; n < N; n += kRowThreads)
        tab[n] = entry_key(idx[n], n, E, N);
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j0 = 0; j0 < k; j0 += 8) {
        int mine[8], cnt[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            mine[j] = j0 + j < k ? tab[t * k + j0 + j] : 0;
            cnt[j] = 0;
        }
        for (int n = threadIdx.x; n < N; n += kRowThreads) {
            const int key = tab[n];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                cnt[j] += key < mine[j] ? 1 : 0;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cnt[j] = __reduce_add_sync(0xFFFFFFFFu, cnt[j]);
            if (lane == 0)
                part[warp][j] = cnt[j];
        }
        __syncthreads();
        if (threadIdx.x < 8 && j0 + static_cast<int>(threadIdx.x) < k) {
            int s = 0;
            for (int w = 0; w < kRowThreads / 32; ++w)
                s += part[w][threadIdx.x];
            s = tab[t * k + j0 + threadIdx.x] == kDroppedKey ? -1 : s;
            slots[j0 + threadIdx.x] = s;
            if (blockIdx.y == 0)
                slot_of[t * k + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
    for (;;) {
        row.store(x_sorted, units, c, c1, slots, k);
        c += RowCopy<U, kRowThreads>::V * kRowThreads;
        if (c >= c1)
            break;
        row.load(src, c, c1);
    }
}

// Larger calls, one launch for the places and one for the rows. The places: one cluster of
// kPlaceCtas CTAs, CTA c owning consecutive entries, its warps consecutive parts of them in R rounds
// of 32, all in registers. An entry's rank among its warp's earlier entries of the same expert
// comes from a warp-wide comparison on per-warp counters; counters are summed over warps, over the CTAs
// through distributed shared memory, and scanned over experts.
constexpr int kPlaceCtas = 8;
constexpr int kPlaceThreads = 1024;
constexpr int kPlaceWarps = kPlaceThreads / 32;
// Up to kPlaceCtas * kPlaceThreads * kMaxRounds = 65536 entries: there 11.7 us for 352 experts (14.2 for 1024), the count
// and scan below 13.2 (13.9); for 96000 entries 14.7 against 14.1 us. A round costs 0.8 us: 16384 entries in two 6.4, in four 8.0.
constexpr int kMaxRounds = 8;

// Lanes of the warp that hold the same value of `bits` bits. A ballot per bit: __match_any_sync, which
// answers the same, takes about 70 cycles of a unit that the SM's warps share (65536 entries of 352
// experts, 8-element rows: 15.1 us a sort with it, 11.6 us with ballots; 16384 entries 7.3 and 6.5).
__device__ __forceinline__ unsigned same_value(int v, int bits)
{
    unsigned m = 0xFFFFFFFFu;
    for (int b = 0; b < bits; ++b) {
        const bool on = v >> b & 1;
        const unsigned vote = __ballot_sync(0xFFFFFFFFu, on);
        m &= on ? vote : ~vote;
    }
    return m;
}

// Exclusive prefix over the block's 1024 threads.
__device__ __forceinline__ int block_exclusive(int v, int *warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o)
            incl += u;
    }
    if (lane == 31)
        warp_sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int s = warp_sums[lane];
        int si = s;
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, si, o);
            if (lane >= o)
                si += u;
        }
        warp_sums[lane] = si - s;
    }
    __syncthreads();
    return warp_sums[warp] + incl - v;
}

template <int R>
__global__ void __launch_bounds__(kPlaceThreads)
    sort_places_kernel(const int32_t *__restrict__ idx, int N, int E, int32_t *__restrict__ offsets,
                       int32_t *__restrict__ slot_of)
{
    allow_dependents();
    extern __shared__ int32_t cnt[];    // [kPlaceWarps][E]
    int32_t *total = cnt + kPlaceWarps * E;  // [E] this CTA's counts, read by its peers
    __shared__ int warp_sums[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cta = static_cast<int>(cluster_ctarank());
    const int base = (cta * kPlaceWarps + warp) * R * 32 + lane;
    const int bits = 32 - __clz(E);  // of the values 0 .. E
    int id[R], rank[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = base + r * 32;
        id[r] = n < N ? idx[n] : -1;
    }
    for (int i = threadIdx.x; i < kPlaceWarps * E; i += kPlaceThreads)
        cnt[i] = 0;
    __syncthreads();
    int32_t *mine = cnt + warp * E;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const bool kept = static_cast<unsigned>(id[r]) < static_cast<unsigned>(E);
        const unsigned m = same_value(kept ? id[r] : E, bits);
        const int before = kept ? mine[id[r]] : 0;
        __syncwarp();
        if (kept && lane == 31 - __clz(m))
            mine[id[r]] = before + __popc(m);
        __syncwarp();
        rank[r] = kept ? before + __popc(m & ((1u << lane) - 1u)) : -1;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kPlaceThreads) {  // E <= kPlaceThreads: one pass
        int run = 0;
#pragma unroll
        for (int w = 0; w < kPlaceWarps; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += c;
        }
        total[e] = run;
    }
    cluster_sync_all();
    int below = 0, all = 0;
    const int e = threadIdx.x;
    if (e < E) {
        const uint32_t local = smem_u32(total + e);
#pragma unroll
        for (int c = 0; c < kPlaceCtas; ++c) {
            const int v = dsmem_ld_s32(dsmem_addr(local, c));
            below += c < cta ? v : 0;
            all += v;
        }
    }
    const int start = block_exclusive(all, warp_sums);
    cluster_sync_all();  // the peers have read this CTA's counts: they become the expert's base here
    if (e < E) {
        total[e] = start + below;
        if (cta == 0) {
            offsets[e] = start;
            if (e == E - 1)
                offsets[E] = start + all;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = base + r * 32;
        if (n < N)
            slot_of[n] = rank[r] < 0 ? -1 : total[id[r]] + mine[id[r]] + rank[r];
    }
}

// Still larger ones, two launches for the places. count: block b owns `per` consecutive entries,
// ranked within the block as above; scan: hist[b][e] becomes the first place of block b's entries of
// expert e. The rows' launch adds the two.
constexpr int kCountThreads = 256;
constexpr int kCountWarps = kCountThreads / 32;
constexpr int kCountBlocks = 128;  // most blocks of the count
constexpr int kScanCtas = 8;
constexpr int kScanGroups = 32;  // most parts of the blocks that are summed side by side

__global__ void __launch_bounds__(kCountThreads)
    sort_count_kernel(const int32_t *__restrict__ idx, int64_t N, int E, int per, int32_t *__restrict__ hist,
                      int32_t *__restrict__ rank)
{
    allow_dependents();
    extern __shared__ int32_t cnt[];  // [kCountWarps][E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kCountWarps * E; i += kCountThreads)
        cnt[i] = 0;
    __syncthreads();
    const int bits = 32 - __clz(E);
    const int per_warp = per / kCountWarps;  // a multiple of 32
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * per + warp * per_warp;
    int32_t *mine = cnt + warp * E;
    for (int i = 0; i < per_warp; i += 32) {
        const int64_t n = begin + i + lane;
        const int id = n < N ? idx[n] : -1;
        const bool kept = static_cast<unsigned>(id) < static_cast<unsigned>(E);
        const unsigned m = same_value(kept ? id : E, bits);
        const int before = kept ? mine[id] + __popc(m & ((1u << lane) - 1u)) : -1;
        __syncwarp();
        if (kept && lane == 31 - __clz(m))
            mine[id] += __popc(m);
        __syncwarp();
        if (n < N)
            rank[n] = before;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kCountThreads) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < kCountWarps; ++w) {
            const int c = cnt[w * E + e];
            cnt[w * E + e] = run;
            run += c;
        }
        hist[static_cast<int64_t>(blockIdx.x) * E + e] = run;
    }
    __syncthreads();
    for (int i = lane; i < per_warp; i += 32) {
        const int64_t n = begin + i;
        if (n < N && rank[n] >= 0)
            rank[n] += mine[idx[n]];
    }
}

// One cluster of kScanCtas CTAs; CTA c owns the experts [c, c + 1) * ep. Thread (g, e) sums the
// counts of the g-th part of the blocks, the parts meet in shared memory, the CTA totals
// through distributed shared memory.
__global__ void __launch_bounds__(1024)
    sort_scan_kernel(int32_t *__restrict__ hist, int nb, int E, int ep, int ep_pad, int32_t *__restrict__ offsets)
{
    __shared__ int part[1024];
    __shared__ int start[kMaxExperts / kScanCtas];
    __shared__ int cta_total;
    allow_dependents();
    dependency_wait();
    const int groups = 1024 / ep_pad < kScanGroups ? 1024 / ep_pad : kScanGroups;  // threads beyond idle
    const int le = threadIdx.x % ep_pad, g = threadIdx.x / ep_pad;
    const int e = static_cast<int>(cluster_ctarank()) * ep + le;
    const bool on = le < ep && e < E && g < groups;
    const int span = (nb + groups - 1) / groups;
    const int b0 = g * span < nb ? g * span : nb, b1 = b0 + span < nb ? b0 + span : nb;
    int sum = 0;
    if (on)
        for (int b = b0; b < b1; ++b)
            sum += hist[static_cast<int64_t>(b) * E + e];
    part[threadIdx.x] = sum;
    __syncthreads();
    int before = 0, total = 0;
    for (int i = 0; i < groups; ++i) {
        const int v = part[i * ep_pad + le];
        before += i < g ? v : 0;
        total += v;
    }
    if (threadIdx.x < 32) {  // exclusive scan of the CTA's expert totals, ep_pad <= 128
        int run = 0;
        for (int base = 0; base < ep_pad; base += 32) {
            int v = 0;
            if (base + static_cast<int>(threadIdx.x) < ep_pad)
                for (int i = 0; i < groups; ++i)
                    v += part[i * ep_pad + base + threadIdx.x];
            int incl = v;
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (static_cast<int>(threadIdx.x) >= o)
                    incl += u;
            }
            if (base + static_cast<int>(threadIdx.x) < ep_pad)
                start[base + threadIdx.x] = run + incl - v;
            run += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (threadIdx.x == 0)
            cta_total = run;
    }
    cluster_sync_all();
    int below = 0;
    for (uint32_t c = 0; c < cluster_ctarank(); ++c)
        below += dsmem_ld_s32(dsmem_addr(smem_u32(&cta_total), c));
    if (on) {
        int run = below + start[le];
        if (g == 0) {
            offsets[e] = run;
            if (e == E - 1)
                offsets[E] = run + total;
        }
        run += before;
        for (int b = b0; b < b1; ++b) {
            int32_t *h = hist + static_cast<int64_t>(b) * E + e;
            const int c = *h;
            *h = run;
            run += c;
        }
    }
    cluster_sync_all();  // no CTA leaves while a peer may still read its total
}

// Blocks copy the rows of kRowThreads / LANES tokens each; their loads are on their way before the places
// are. kFinal: slot_of holds the places already (sort_places_kernel). What the launch before wrote is read
// through pointers without __restrict__: such loads could move above the wait.
template <typename U, bool kFinal, int LANES>
__global__ void __launch_bounds__(kRowThreads)
    sort_rows_kernel(const U *__restrict__ x, const int32_t *__restrict__ idx, int T, int k, int E, int per,
                     const int32_t *hist, const int32_t *rank, int64_t units, U *__restrict__ x_sorted,
                     int32_t *slot_of)
{
    constexpr int kTokens = kRowThreads / LANES;
    __shared__ int slots[kMaxK * kTokens];
    const int mine = threadIdx.x / LANES;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens, t = t0 + mine;
    const U *src = x + t * units;
    int64_t c = threadIdx.x % LANES;
    const int64_t end = t < T ? units : 0;
    RowCopy<U, LANES> row;
    row.load(src, c, end);
    dependency_wait();
    const int64_t n0 = t0 * k;
    const int count = static_cast<int>(T - t0 < kTokens ? T - t0 : kTokens) * k;
    for (int i = threadIdx.x; i < count; i += kRowThreads) {
        const int64_t n = n0 + i;
        int s;
        if (kFinal) {
            s = slot_of[n];
        } else {
            const int r = rank[n];
            s = r < 0 ? -1 : hist[n / per * E + idx[n]] + r;
            slot_of[n] = s;
        }
        slots[i] = s;
    }
    __syncthreads();
    while (c < end) {
        row.store(x_sorted, units, c, end, slots + mine * k, k);
        c += RowCopy<U, LANES>::V * LANES;
        if (c < end)
            row.load(src, c, end);
    }
}

// Rows of up to 8 units share a block of 16 tokens, rows that a warp holds at once one of 4: 8000 rows of 128
// bytes copied to 8 places each 13 us, 26 us with a block per row; 20000 of 180 bytes to 4 places 20 for 33 us; 16000 of 528
// bytes to 2 places 9.7 for 15 us; 4000 of 1040 bytes 6.1 for 6.7 us.
template <typename U, bool kFinal>
cudaError_t launch_rows(const U *x, const int32_t *idx, int T, int k, int E, int per, const int32_t *hist,
                        const int32_t *rank, int64_t units, U *x_sorted, int32_t *slot_of, cudaStream_t stream)
{
    const int lanes = units <= 8 ? 8 : (units <= 32 * RowCopy<U, 32>::V ? 32 : kRowThreads);
    auto kernel = lanes == 8    ? sort_rows_kernel<U, kFinal, 8>
                  : lanes == 32 ? sort_rows_kernel<U, kFinal, 32>
                                : sort_rows_kernel<U, kFinal, kRowThreads>;
    const int tokens = kRowThreads / lanes;
    return launch_dependent(kernel, dim3((T + tokens - 1) / tokens), kRowThreads, 0, stream, 1, x, idx, T, k, E, per,
                            hist, rank, units, x_sorted, slot_of);
}

struct SortPlan {
    int nb, per;  // blocks of the count and entries of each
    size_t hist, rank, total;
};

SortPlan sort_plan(int64_t N, int E)
{
    SortPlan p{};
    const int64_t unit = 32 * kCountWarps;
    int64_t per = (N + kCountBlocks - 1) / kCountBlocks;
    per = (per + unit - 1) / unit * unit;
    p.per = static_cast<int>(per);
    p.nb = static_cast<int>((N + per - 1) / per);
    p.hist = 0;
    p.rank = (static_cast<size_t>(kCountBlocks) * E * 4 + 255) / 256 * 256;
    p.total = p.rank + (static_cast<size_t>(N) * 4 + 255) / 256 * 256;
    return p;
}

template <int R>
cudaError_t launch_places_r(const int32_t *idx, int N, int E, int32_t *offsets, int32_t *slot_of, cudaStream_t stream)
{
    const int smem = (kPlaceWarps + 1) * E * 4;
    const cudaError_t err =
        cudaFuncSetAttribute(sort_places_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPlaceCtas);
    cfg.blockDim = dim3(kPlaceThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kPlaceCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sort_places_kernel<R>, idx, N, E, offsets, slot_of);
}

cudaError_t launch_places(const int32_t *idx, int N, int E, int32_t *offsets, int32_t *slot_of, cudaStream_t stream)
{
    switch ((N + kPlaceCtas * kPlaceThreads - 1) / (kPlaceCtas * kPlaceThreads)) {
    case 1: return launch_places_r<1>(idx, N, E, offsets, slot_of, stream);
    case 2: return launch_places_r<2>(idx, N, E, offsets, slot_of, stream);
    case 3:
    case 4: return launch_places_r<4>(idx, N, E, offsets, slot_of, stream);
    case 5:
    case 6: return launch_places_r<6>(idx, N, E, offsets, slot_of, stream);
    default: return launch_places_r<kMaxRounds>(idx, N, E, offsets, slot_of, stream);
    }
}

template <typename U>
cudaError_t launch_sort(const void *x, const int32_t *idx, int T, int k, int E, int64_t row_bytes, void *x_sorted,
                        int32_t *offsets, int32_t *slot_of, void *ws, int num_sms, cudaStream_t stream)
{
    const int64_t units = row_bytes / static_cast<int64_t>(sizeof(U));
    const U *xs = static_cast<const U *>(x);
    U *out = static_cast<U *>(x_sorted);
    const int64_t N = static_cast<int64_t>(T) * k;
    if (N <= kSmallEntries) {
        // few tokens: the columns of a row are split until every SM has two blocks
        int64_t chunks = (2 * num_sms + T - 1) / T;
        const int64_t most = (units + kRowThreads - 1) / kRowThreads;
        chunks = chunks < most ? chunks : most;
        const int64_t chunk = ((units + chunks - 1) / chunks + kRowThreads - 1) / kRowThreads * kRowThreads;
        const dim3 grid(T + 1, static_cast<unsigned>((units + chunk - 1) / chunk));
        sort_small_kernel<U><<<grid, kRowThreads, 0, stream>>>(xs, idx, T, k, E, units, chunk, out, offsets, slot_of);
        return cudaGetLastError();
    }
    if (N <= static_cast<int64_t>(kPlaceCtas) * kPlaceThreads * kMaxRounds) {
        cudaError_t err = launch_places(idx, static_cast<int>(N), E, offsets, slot_of, stream);
        if (err != cudaSuccess)
            return err;
        return launch_rows<U, true>(xs, idx, T, k, E, 1, nullptr, nullptr, units, out, slot_of, stream);
    }
    const SortPlan p = sort_plan(N, E);
    int32_t *hist = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + p.hist);
    int32_t *rank = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(ws) + p.rank);
    sort_count_kernel<<<p.nb, kCountThreads, kCountWarps * E * 4, stream>>>(idx, N, E, p.per, hist, rank);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess)
        return err;
    const int ep = (E + kScanCtas - 1) / kScanCtas;
    int ep_pad = 1;
    while (ep_pad < ep)
        ep_pad *= 2;
    err = launch_dependent(sort_scan_kernel, dim3(kScanCtas), 1024, 0, stream, kScanCtas, hist, p.nb, E, ep, ep_pad,
                           offsets);
    if (err != cudaSuccess)
        return err;
    return launch_rows<U, false>(xs, idx, T, k, E, p.per, hist, rank, units, out, slot_of, stream);
}

// --------------------------------------------------------------------- rows in fp32 and back
template <typename S, int VEC>
struct alignas(sizeof(S) * VEC) Pack {
    S v[VEC];
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename S>
__device__ __forceinline__ S from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// p = *src where `on`; p is undefined elsewhere. One predicated load: as a branch around it, the loads of a batch
// wait for one another.
template <typename P>
__device__ __forceinline__ void load_if(P &p, const P *src, bool on)
{
    static_assert(sizeof(P) == 2 || sizeof(P) == 4 || sizeof(P) == 8 || sizeof(P) == 16, "pack");
    const int q = on;
    if constexpr (sizeof(P) == 16) {
        uint4 u;
        asm("{\n.reg .pred q;\nsetp.ne.b32 q, %5, 0;\n@q ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
            : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
            : "l"(src), "r"(q));
        memcpy(&p, &u, sizeof(P));
    } else if constexpr (sizeof(P) == 8) {
        uint2 u;
        asm("{\n.reg .pred q;\nsetp.ne.b32 q, %3, 0;\n@q ld.global.nc.v2.u32 {%0, %1}, [%2];\n}"
            : "=r"(u.x), "=r"(u.y)
            : "l"(src), "r"(q));
        memcpy(&p, &u, sizeof(P));
    } else if constexpr (sizeof(P) == 4) {
        uint32_t u;
        asm("{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n@q ld.global.nc.u32 %0, [%1];\n}" : "=r"(u) : "l"(src), "r"(q));
        memcpy(&p, &u, sizeof(P));
    } else {
        uint16_t u;
        asm("{\n.reg .pred q;\nsetp.ne.b32 q, %2, 0;\n@q ld.global.nc.u16 %0, [%1];\n}" : "=h"(u) : "l"(src), "r"(q));
        memcpy(&p, &u, sizeof(P));
    }
}

// Packs of a row that a thread has in flight per entry.
template <typename P>
__host__ __device__ constexpr int unsort_batch()
{
    return sizeof(P) <= 4 ? 4 : 1;
}

// y[t] = add[t] + sum_j w[t, j] rows[slot_of[t, j]] (w NULL: 1, add NULL: 0) by LANES threads per token
// for packs [c0, c0 + chunk) of the row; a slot outside [0, N) contributes nothing. The chunks of a
// token are neighbours in the grid, so that a row's 8 KB are read at one time: with the tokens
// innermost DRAM saw 2 KB pieces, 4.8 against 6.6 TB/s over 1.2 GB. K: the most slots (4 or 8), which stay in registers
// with their weights; 0: any number, eight at a time. Narrow packs (rows that are not 16-byte aligned) go four at a time, for as many bytes in flight.
template <typename S, int VEC, int K, int LANES, int THREADS>
__global__ void __launch_bounds__(THREADS)
    unsort_kernel(const S *__restrict__ rows, const int32_t *__restrict__ slot_of, const float *__restrict__ w,
                  const S *__restrict__ add, int T, int k, int64_t N, int H, int chunk, int chunks, S *__restrict__ y)
{
    using P = Pack<S, VEC>;
    constexpr int KB = K ? K : 8;
    constexpr int NV = unsort_batch<P>();
    const int group = blockIdx.x / chunks;  // of THREADS / LANES tokens
    const int64_t t = static_cast<int64_t>(group) * (THREADS / LANES) + threadIdx.x / LANES;
    if (t >= T)
        return;
    const int c0 = (blockIdx.x - group * chunks) * chunk;
    const int c1 = c0 + chunk < H / VEC ? c0 + chunk : H / VEC;
    int s[KB];
    float wj[KB];
    auto fetch = [&](int j0) {
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            s[j] = -1;
            wj[j] = 1.0f;
            if (j0 + j < k) {
                s[j] = slot_of[t * k + j0 + j];
                if (w)
                    wj[j] = w[t * k + j0 + j];
                if (s[j] >= N)
                    s[j] = -1;
            }
        }
    };
    if (K)
        fetch(0);
    for (int c = c0 + threadIdx.x % LANES; c < c1; c += NV * LANES) {
        P a[NV];
        float acc[NV][VEC];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (add && (NV == 1 || c + v * LANES < c1))
                a[v] = *reinterpret_cast<const P *>(add + t * H + static_cast<int64_t>(c + v * LANES) * VEC);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                acc[v][i] = 0.0f;
        }
        for (int j0 = 0; j0 < k; j0 += KB) {
            if (!K)
                fetch(j0);
            P r[KB][NV];
#pragma unroll
            for (int j = 0; j < KB; ++j)
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    load_if(r[j][v],
                            reinterpret_cast<const P *>(rows + static_cast<int64_t>(s[j]) * H +
                                                        static_cast<int64_t>(c + v * LANES) * VEC),
                            s[j] >= 0 && (NV == 1 || c + v * LANES < c1));
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (s[j] >= 0)
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        if (NV == 1 || c + v * LANES < c1)
#pragma unroll
                            for (int i = 0; i < VEC; ++i)
                                acc[v][i] = fmaf(wj[j], to_f32(r[j][v].v[i]), acc[v][i]);
            if (K)
                break;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (NV > 1 && c + v * LANES >= c1)
                break;
            P o;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                o.v[i] = from_f32<S>(add ? acc[v][i] + to_f32(a[v].v[i]) : acc[v][i]);
            *reinterpret_cast<P *>(y + t * H + static_cast<int64_t>(c + v * LANES) * VEC) = o;
        }
    }
}

// The gradient of the unsort: per entry its row of dy_sorted and, through a sum in a fixed order,
// its dw. LANES threads per entry, the entries of a token in one block or neighbouring ones, so that dy
// comes from L1 for all but the first; no barrier, U packs of both rows in flight per lane (of 16-byte packs four:
// 53175 entries of 2128 bytes take 49 us, with two 46, with eight 74; 8000 of 16 KB 48, 54 and 51). A warp
// for 32768 entries of 8 KB: 89 us, 6.4 TB/s. Eight lanes for rows of up to 8 packs: 64000 entries of 128 bytes 6 us,
// a warp for each 18 us.
constexpr int kBackThreads = 256;

template <typename S, int VEC, int LANES>
__global__ void __launch_bounds__(kBackThreads)
    unsort_backward_kernel(const S *__restrict__ dy, const S *__restrict__ rows, const int32_t *__restrict__ slot_of,
                           const float *__restrict__ w, int k, int64_t N, int H, S *__restrict__ drows,
                           float *__restrict__ dw)
{
    using P = Pack<S, VEC>;
    constexpr int U = sizeof(P) >= 16 ? 4 : 8;
    const int lane = threadIdx.x % LANES;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * (kBackThreads / LANES) + threadIdx.x / LANES;
    const bool on = n < N;  // lanes without an entry stay for the others' sums
    const int64_t s = on ? slot_of[n] : -1;
    float acc = 0.0f;
    if (s >= 0 && s < N) {
        const float wn = w ? w[n] : 1.0f;
        const int64_t t = static_cast<uint32_t>(n) / static_cast<uint32_t>(k);
        const P *g_row = reinterpret_cast<const P *>(dy + t * H);
        const P *r_row = reinterpret_cast<const P *>(rows + s * H);
        P *d_row = reinterpret_cast<P *>(drows + s * H);
        const int packs = H / VEC;
        for (int c = lane; c < packs; c += U * LANES) {
            P g[U], r[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                load_if(g[u], g_row + c + u * LANES, c + u * LANES < packs);
                load_if(r[u], r_row + c + u * LANES, dw && c + u * LANES < packs);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u * LANES < packs) {
                    if (dw)
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
                            acc = fmaf(to_f32(g[u].v[i]), to_f32(r[u].v[i]), acc);
                    if (drows) {
                        P o;
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
                            o.v[i] = from_f32<S>(wn * to_f32(g[u].v[i]));
                        d_row[c + u * LANES] = o;
                    }
                }
        }
    }
    if (!dw)
        return;
    for (int o = LANES / 2; o > 0; o >>= 1)
        acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
    if (on && lane == 0)
        dw[n] = acc;
}

// JB entries of one token per block. Four or eight for rows of 9 to 64 packs and many tokens: 32000 entries of
// 528 bytes 13 us, a warp for each 18 us; for 32768 of 8 KB 99 against 89 us. One for few entries, so that they fill
// the SMs (dy is then read k times): 512 entries 3.2 us, a warp per entry or eight entries per block 4.5 us and more.
template <typename S, int VEC, int JB, int THREADS>
__global__ void __launch_bounds__(THREADS)
    unsort_backward_token_kernel(const S *__restrict__ dy, const S *__restrict__ rows,
                                 const int32_t *__restrict__ slot_of, const float *__restrict__ w, int k, int64_t N,
                                 int H, S *__restrict__ drows, float *__restrict__ dw)
{
    using P = Pack<S, VEC>;
    __shared__ float part[THREADS / 32][JB];
    const int64_t t = blockIdx.x;
    const int j0 = blockIdx.y * JB;
    int s[JB];
    float wj[JB], acc[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
        s[j] = -1;
        wj[j] = 1.0f;
        acc[j] = 0.0f;
        if (j0 + j < k) {
            s[j] = slot_of[t * k + j0 + j];
            if (w)
                wj[j] = w[t * k + j0 + j];
            if (s[j] >= N)
                s[j] = -1;
        }
    }
    for (int col = threadIdx.x * VEC; col < H; col += THREADS * VEC) {
        const P g = *reinterpret_cast<const P *>(dy + t * H + col);
        P r[JB];
        if (dw) {
#pragma unroll
            for (int j = 0; j < JB; ++j)
                load_if(r[j], reinterpret_cast<const P *>(rows + static_cast<int64_t>(s[j]) * H + col), s[j] >= 0);
#pragma unroll
            for (int j = 0; j < JB; ++j)
                if (s[j] >= 0)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        acc[j] = fmaf(to_f32(g.v[i]), to_f32(r[j].v[i]), acc[j]);
        }
        if (drows) {
#pragma unroll
            for (int j = 0; j < JB; ++j)
                if (s[j] >= 0) {
                    P o;
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        o.v[i] = from_f32<S>(wj[j] * to_f32(g.v[i]));
                    *reinterpret_cast<P *>(drows + static_cast<int64_t>(s[j]) * H + col) = o;
                }
        }
    }
    if (!dw)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < JB; ++j) {
        for (int o = 16; o > 0; o >>= 1)
            acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
        if (lane == 0)
            part[warp][j] = acc[j];
    }
    __syncthreads();
    if (threadIdx.x < JB && j0 + static_cast<int>(threadIdx.x) < k) {
        float sum = 0.0f;
        for (int i = 0; i < THREADS / 32; ++i)
            sum += part[i][threadIdx.x];
        dw[t * k + j0 + threadIdx.x] = sum;
    }
}

// The widest pack that divides the row and to which every array is aligned.
int pack_bytes(int64_t row_bytes, int elem, std::initializer_list<const void *> ptrs)
{
    uintptr_t bits = static_cast<uintptr_t>(row_bytes);
    for (const void *p : ptrs)
        bits |= reinterpret_cast<uintptr_t>(p);  // NULL adds no bit
    for (int b = 16; b > elem; b >>= 1)
        if (bits % b == 0)
            return b;
    return elem;
}

// Packs of a row per block and blocks per row: whole rows, but for few tokens as many pieces of at
// least `least` packs as give every SM four blocks (sixteen: 777 x 514 fp32, k = 4, 3.2 against 2.5 us, 600 x 2048 bf16,
// k = 8, 4.3 against 3.8 us, 200 x 4096 3.5 against 3.7 us).
void split_row(int64_t packs, int T, int num_sms, int least, int &chunk, int &chunks)
{
    int64_t pieces = (4 * static_cast<int64_t>(num_sms) + T - 1) / T;
    const int64_t most = (packs + least - 1) / least;
    pieces = pieces < most ? pieces : most;
    chunk = static_cast<int>(((packs + pieces - 1) / pieces + 31) / 32 * 32);
    chunks = static_cast<int>((packs + chunk - 1) / chunk);
}

// Rows of up to 8 packs share a block of 16 tokens, up to 64 one of 4, and up to 160 too where there are
// tokens for every SM: 8000 tokens x 8 rows of 128 bytes 3.1 us, 128 threads a row 12.7; 4000 x 8 of 528 bytes 5.4 for
// 7.7 us; 10635 x 5 of 2128 bytes 31 for 35 us, but 500 x 4 of them 3.8 for 2.6 us.
template <typename S, int VEC>
cudaError_t unsort_vec(const void *rows, const int32_t *slot_of, const float *w, const void *add, int T, int k, int H,
                       void *y, int num_sms, cudaStream_t stream)
{
    const int packs = H / VEC;
    const auto launch = [&](auto lanes_c, auto threads_c) {
        constexpr int LANES = decltype(lanes_c)::value, THREADS = decltype(threads_c)::value;
        int chunk = packs, chunks = 1;
        if (LANES == THREADS)
            split_row(packs, T, num_sms, THREADS * unsort_batch<Pack<S, VEC>>(), chunk, chunks);
        const int tokens = THREADS / LANES;
        auto kernel = k <= 4   ? unsort_kernel<S, VEC, 4, LANES, THREADS>
                      : k <= 8 ? unsort_kernel<S, VEC, 8, LANES, THREADS>
                               : unsort_kernel<S, VEC, 0, LANES, THREADS>;
        kernel<<<static_cast<unsigned>(static_cast<int64_t>((T + tokens - 1) / tokens) * chunks), THREADS, 0, stream>>>(
            static_cast<const S *>(rows), slot_of, w, static_cast<const S *>(add), T, k, static_cast<int64_t>(T) * k, H,
            chunk, chunks, static_cast<S *>(y));
        return cudaGetLastError();
    };
    using std::integral_constant;
    if (packs <= 8)
        return launch(integral_constant<int, 8>{}, integral_constant<int, 128>{});
    if (packs <= 64 || (packs <= 160 && T >= 16 * num_sms))
        return launch(integral_constant<int, 32>{}, integral_constant<int, 128>{});
    return launch(integral_constant<int, 128>{}, integral_constant<int, 128>{});
}

template <typename S, int VEC>
cudaError_t unsort_backward_vec(const void *dy, const void *rows, const int32_t *slot_of, const float *w, int T, int k,
                                int H, void *drows, float *dw, int num_sms, cudaStream_t stream)
{
    const S *g = static_cast<const S *>(dy), *r = static_cast<const S *>(rows);
    S *d = static_cast<S *>(drows);
    const int64_t N = static_cast<int64_t>(T) * k;
    const int packs = H / VEC;
    const auto entries = [&](auto lanes_c) {
        constexpr int LANES = decltype(lanes_c)::value;
        const int64_t blocks = (N * LANES + kBackThreads - 1) / kBackThreads;
        unsort_backward_kernel<S, VEC, LANES><<<static_cast<unsigned>(blocks), kBackThreads, 0, stream>>>(
            g, r, slot_of, w, k, N, H, d, dw);
        return cudaGetLastError();
    };
    const auto tokens = [&](auto jb) {
        constexpr int JB = decltype(jb)::value, THREADS = JB == 1 ? kBackThreads : 64;
        unsort_backward_token_kernel<S, VEC, JB, THREADS>
            <<<dim3(T, (k + JB - 1) / JB), THREADS, 0, stream>>>(g, r, slot_of, w, k, N, H, d, dw);
        return cudaGetLastError();
    };
    if (N < 8 * static_cast<int64_t>(num_sms))
        return tokens(std::integral_constant<int, 1>{});
    if (packs <= 8)
        return entries(std::integral_constant<int, 8>{});
    if (packs <= 64 && k > 1 && T >= 2 * num_sms) {
        if (k <= 4)
            return tokens(std::integral_constant<int, 4>{});
        return tokens(std::integral_constant<int, 8>{});
    }
    return entries(std::integral_constant<int, 32>{});
}

template <typename S, int VEC>
struct VecTag {
    using type = S;
    static constexpr int vec = VEC;
};

// f(VecTag<S, VEC>) for the row type and the pack width.
template <typename F>
cudaError_t by_type(int dtype, int bytes, F f)
{
    if (dtype == MOE_DTYPE_F32) {
        switch (bytes) {
        case 16: return f(VecTag<float, 4>{});
        case 8: return f(VecTag<float, 2>{});
        default: return f(VecTag<float, 1>{});
        }
    }
    if (dtype == MOE_DTYPE_BF16) {
        switch (bytes) {
        case 16: return f(VecTag<__nv_bfloat16, 8>{});
        case 8: return f(VecTag<__nv_bfloat16, 4>{});
        case 4: return f(VecTag<__nv_bfloat16, 2>{});
        default: return f(VecTag<__nv_bfloat16, 1>{});
        }
    }
    switch (bytes) {
    case 16: return f(VecTag<__half, 8>{});
    case 8: return f(VecTag<__half, 4>{});
    case 4: return f(VecTag<__half, 2>{});
    default: return f(VecTag<__half, 1>{});
    }
}

int elem_size(int dtype)
{
    return dtype == MOE_DTYPE_F32 ? 4 : 2;
}

moe_status_t check_tokens(const moe_token_desc *d)
{
    if (!d || d->T < 0 || d->H <= 0 || d->E <= 0 || d->k <= 0 || d->k > kMaxK)
        return MOE_ERR_INVALID_ARG;
    if (d->dtype != MOE_DTYPE_F32 && d->dtype != MOE_DTYPE_BF16 && d->dtype != MOE_DTYPE_F16)
        return MOE_ERR_INVALID_ARG;
    // entry counts stay below 2^31 with room for the count's rounding; 65535 column chunks
    if (d->E > kMaxExperts || d->H > (1 << 22) ||
        static_cast<int64_t>(d->T) * d->k >= (int64_t(1) << 31) - (int64_t(1) << 20))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool aligned_to(const void *p, int bytes)
{
    return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

// SMs of the current device: an attribute that does not change, asked for once per device.
moe_status_t sm_count(int &sms)
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return MOE_ERR_CUDA;
    sms = known[dev].load(std::memory_order_relaxed);
    if (sms == 0) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return MOE_ERR_CUDA;
        known[dev].store(sms, std::memory_order_relaxed);
    }
    return MOE_OK;
}

moe_status_t launched(cudaError_t e)
{
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_sort_workspace_size(const moe_token_desc *desc, size_t *bytes)
{
    const moe_status_t st = check_tokens(desc);
    if (st != MOE_OK)
        return st;
    if (!bytes)
        return MOE_ERR_INVALID_ARG;
    const int64_t N = static_cast<int64_t>(desc->T) * desc->k;
    *bytes = sort_plan(N > kSmallEntries ? N : kSmallEntries + 1, desc->E).total;
    return MOE_OK;
}

moe_status_t moe_sort_tokens(const moe_token_desc *desc, const void *x, const int32_t *topk_idx, void *x_sorted,
                             int32_t *offsets, int32_t *slot_of, void *ws, size_t ws_bytes, void *stream)
{
    moe_status_t st = check_tokens(desc);
    if (st != MOE_OK)
        return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (desc->T == 0) {
        if (!offsets)
            return MOE_OK;
        if (!aligned_to(offsets, 4))
            return MOE_ERR_UNSUPPORTED;
        return launched(cudaMemsetAsync(offsets, 0, (static_cast<size_t>(desc->E) + 1) * 4, s));
    }
    if (!x || !topk_idx || !x_sorted || !offsets || !slot_of || !ws)
        return MOE_ERR_INVALID_ARG;
    const int elem = elem_size(desc->dtype);
    if (!aligned_to(x, elem) || !aligned_to(x_sorted, elem) || !aligned_to(topk_idx, 4) || !aligned_to(offsets, 4) ||
        !aligned_to(slot_of, 4) || !aligned_to(ws, 16))
        return MOE_ERR_UNSUPPORTED;
    size_t need = 0;
    if ((st = moe_sort_workspace_size(desc, &need)) != MOE_OK)
        return st;
    if (ws_bytes < need)
        return MOE_ERR_WORKSPACE;
    int sms = 0;
    if ((st = sm_count(sms)) != MOE_OK)
        return st;
    const int64_t row = static_cast<int64_t>(desc->H) * elem;
    auto go = [&](auto u) {
        return launch_sort<decltype(u)>(x, topk_idx, desc->T, desc->k, desc->E, row, x_sorted, offsets, slot_of, ws,
                                        sms, s);
    };
    switch (pack_bytes(row, elem, {x, x_sorted})) {
    case 16: return launched(go(uint4{}));
    case 8: return launched(go(uint2{}));
    case 4: return launched(go(uint32_t{}));
    default: return launched(go(uint16_t{}));
    }
}

moe_status_t moe_unsort_tokens(const moe_token_desc *desc, const void *y_sorted, const int32_t *slot_of,
                               const float *topk_w, const void *add, void *y, void *stream)
{
    moe_status_t st = check_tokens(desc);
    if (st != MOE_OK)
        return st;
    if (desc->T == 0)
        return MOE_OK;
    if (!y_sorted || !slot_of || !y)
        return MOE_ERR_INVALID_ARG;
    const int elem = elem_size(desc->dtype);
    if (!aligned_to(y_sorted, elem) || !aligned_to(y, elem) || !aligned_to(add, elem) || !aligned_to(slot_of, 4) ||
        !aligned_to(topk_w, 4))
        return MOE_ERR_UNSUPPORTED;
    int sms = 0;
    if ((st = sm_count(sms)) != MOE_OK)
        return st;
    const int bytes = pack_bytes(static_cast<int64_t>(desc->H) * elem, elem, {y_sorted, add, y});
    return launched(by_type(desc->dtype, bytes, [&](auto tag) {
        using V = decltype(tag);
        return unsort_vec<typename V::type, V::vec>(y_sorted, slot_of, topk_w, add, desc->T, desc->k, desc->H, y,
                                                    sms, static_cast<cudaStream_t>(stream));
    }));
}

moe_status_t moe_sort_tokens_backward(const moe_token_desc *desc, const void *dx_sorted, const int32_t *slot_of,
                                      void *dx, void *stream)
{
    // the gradient of copying a row to k places is the sum of the k gradients
    return moe_unsort_tokens(desc, dx_sorted, slot_of, nullptr, nullptr, dx, stream);
}

moe_status_t moe_unsort_tokens_backward(const moe_token_desc *desc, const void *dy, const void *y_sorted,
                                        const int32_t *slot_of, const float *topk_w, void *dy_sorted, float *dtopk_w,
                                        void *stream)
{
    moe_status_t st = check_tokens(desc);
    if (st != MOE_OK)
        return st;
    if (desc->T == 0)
        return MOE_OK;
    if (!dy || !slot_of || (!dy_sorted && !dtopk_w) || (dtopk_w && !y_sorted))
        return MOE_ERR_INVALID_ARG;
    const int elem = elem_size(desc->dtype);
    if (!aligned_to(dy, elem) || !aligned_to(y_sorted, elem) || !aligned_to(dy_sorted, elem) ||
        !aligned_to(slot_of, 4) || !aligned_to(topk_w, 4) || !aligned_to(dtopk_w, 4))
        return MOE_ERR_UNSUPPORTED;
    int sms = 0;
    if ((st = sm_count(sms)) != MOE_OK)
        return st;
    const int bytes = pack_bytes(static_cast<int64_t>(desc->H) * elem, elem, {dy, y_sorted, dy_sorted});
    return launched(by_type(desc->dtype, bytes, [&](auto tag) {
        using V = decltype(tag);
        return unsort_backward_vec<typename V::type, V::vec>(dy, y_sorted, slot_of, topk_w, desc->T, desc->k, desc->H,
                                                             dy_sorted, dtopk_w, sms,
                                                             static_cast<cudaStream_t>(stream));
    }));
}

}  // extern "C"
