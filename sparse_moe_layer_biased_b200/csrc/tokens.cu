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
// dependence between blocks: N compares per entry in place of two more launches and their hand-over.
constexpr int kSmallEntries = 4096;
constexpr int kRowThreads = 128;
constexpr int kDroppedKey = 0x7fffffff;

__device__ __forceinline__ int entry_key(int id, int n, int E, int N)
{
    return static_cast<unsigned>(id) < static_cast<unsigned>(E) ? id * N + n : kDroppedKey;
}

// Row t of x (units of U) to the rows slots[0..k) of out; columns [c0, c1) of the row. Every
// load of a piece is issued before its k copies are stored.
template <typename U>
__device__ __forceinline__ void scatter_row(const U *__restrict__ src, U *__restrict__ out, int64_t units, int64_t c0,
                                            int64_t c1, const int *slots, int k)
{
    constexpr int V = 4;
    for (int64_t c = c0 + threadIdx.x; c < c1; c += V * kRowThreads) {
        U v[V];
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i * kRowThreads < c1)
                v[i] = src[c + i * kRowThreads];
        for (int j = 0; j < k; ++j) {
            const int64_t s = slots[j];
            if (s < 0)
                continue;
            U *dst = out + s * units;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i * kRowThreads < c1)
                    dst[c + i * kRowThreads] = v[i];
        }
    }
}

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
    const int64_t c0 = blockIdx.y * chunk;
    const int64_t c1 = c0 + chunk < units ? c0 + chunk : units;
    scatter_row(x + static_cast<int64_t>(t) * units, x_sorted, units, c0, c1, slots, k);
}

// Larger calls, three launches. count: block b owns `per` consecutive entries, its warps
// consecutive parts of them; an entry's rank among the block's entries of its expert comes from
// __match_any_sync (32 entries at a time) on per-warp counters. scan: hist[b][e] becomes the
// first place of block b's entries of expert e. place: slot = hist[b][e] + rank, and the rows.
constexpr int kCountThreads = 256;
constexpr int kCountWarps = kCountThreads / 32;
constexpr int kCountBlocks = 128;  // most blocks of the count
constexpr int kScanCtas = 8;

__global__ void __launch_bounds__(kCountThreads)
    sort_count_kernel(const int32_t *__restrict__ idx, int64_t N, int E, int per, int32_t *__restrict__ hist,
                      int32_t *__restrict__ rank)
{
    extern __shared__ int32_t cnt[];  // [kCountWarps][E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < kCountWarps * E; i += kCountThreads)
        cnt[i] = 0;
    __syncthreads();
    const int per_warp = per / kCountWarps;  // a multiple of 32
    const int64_t begin = static_cast<int64_t>(blockIdx.x) * per + warp * per_warp;
    int32_t *mine = cnt + warp * E;
    for (int i = 0; i < per_warp; i += 32) {
        const int64_t n = begin + i + lane;
        const int id = n < N ? idx[n] : -1;
        const bool kept = static_cast<unsigned>(id) < static_cast<unsigned>(E);
        const unsigned m = __match_any_sync(0xFFFFFFFFu, kept ? id : E + lane);
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
    const int groups = 1024 / ep_pad;
    const int le = threadIdx.x % ep_pad, g = threadIdx.x / ep_pad;
    const int e = static_cast<int>(cluster_ctarank()) * ep + le;
    const bool on = le < ep && e < E;
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

template <typename U>
__global__ void __launch_bounds__(kRowThreads)
    sort_place_kernel(const U *__restrict__ x, const int32_t *__restrict__ idx, int k, int E, int per,
                      const int32_t *__restrict__ hist, const int32_t *__restrict__ rank, int64_t units,
                      U *__restrict__ x_sorted, int32_t *__restrict__ slot_of)
{
    __shared__ int slots[kMaxK];
    const int64_t t = blockIdx.x;
    if (threadIdx.x < k) {
        const int64_t n = t * k + threadIdx.x;
        const int r = rank[n];
        const int s = r < 0 ? -1 : hist[n / per * E + idx[n]] + r;
        slots[threadIdx.x] = s;
        slot_of[n] = s;
    }
    __syncthreads();
    scatter_row(x + t * units, x_sorted, units, 0, units, slots, k);
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kScanCtas);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kScanCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, sort_scan_kernel, hist, p.nb, E, ep, ep_pad, offsets);
    if (err != cudaSuccess)
        return err;
    sort_place_kernel<U><<<T, kRowThreads, 0, stream>>>(xs, idx, k, E, p.per, hist, rank, units, out, slot_of);
    return cudaGetLastError();
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

// y[t] = add[t] + sum_j w[t, j] rows[slot_of[t, j]] (w NULL: 1, add NULL: 0) for columns of one
// kRowThreads * VEC wide chunk. A slot outside [0, rows) contributes nothing.
template <typename S, int VEC>
__global__ void __launch_bounds__(kRowThreads)
    unsort_kernel(const S *__restrict__ rows, const int32_t *__restrict__ slot_of, const float *__restrict__ w,
                  const S *__restrict__ add, int k, int64_t N, int H, S *__restrict__ y)
{
    using P = Pack<S, VEC>;
    const int64_t t = blockIdx.x;
    const int col = (blockIdx.y * kRowThreads + threadIdx.x) * VEC;
    if (col >= H)
        return;
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += 8) {
        P r[8];
        int64_t s[8];
        float wj[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] = -1;
            wj[j] = 1.0f;
            if (j0 + j < k) {
                s[j] = slot_of[t * k + j0 + j];
                if (w)
                    wj[j] = w[t * k + j0 + j];
            }
            if (s[j] >= N)
                s[j] = -1;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (s[j] >= 0)
                r[j] = *reinterpret_cast<const P *>(rows + s[j] * H + col);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (s[j] >= 0)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    acc[i] = fmaf(wj[j], to_f32(r[j].v[i]), acc[i]);
    }
    if (add) {
        const P a = *reinterpret_cast<const P *>(add + t * H + col);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            acc[i] += to_f32(a.v[i]);
    }
    P o;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        o.v[i] = from_f32<S>(acc[i]);
    *reinterpret_cast<P *>(y + t * H + col) = o;
}

// Entries j0 .. j0 + JB of token t (block (t, j0 / JB)): their rows of dy_sorted and, through a
// block-wide sum in a fixed order, their dw.
constexpr int kBackThreads = 256;

template <typename S, int VEC, int JB>
__global__ void __launch_bounds__(kBackThreads)
    unsort_backward_kernel(const S *__restrict__ dy, const S *__restrict__ rows, const int32_t *__restrict__ slot_of,
                           const float *__restrict__ w, int k, int64_t N, int H, S *__restrict__ drows,
                           float *__restrict__ dw)
{
    using P = Pack<S, VEC>;
    __shared__ float part[kBackThreads / 32][JB];
    const int64_t t = blockIdx.x;
    const int j0 = blockIdx.y * JB;
    int64_t s[JB];
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
        }
        if (s[j] >= N)
            s[j] = -1;
    }
    for (int64_t col = static_cast<int64_t>(threadIdx.x) * VEC; col < H; col += kBackThreads * VEC) {
        const P g = *reinterpret_cast<const P *>(dy + t * H + col);
        P r[JB];
        if (dw) {
#pragma unroll
            for (int j = 0; j < JB; ++j)
                if (s[j] >= 0)
                    r[j] = *reinterpret_cast<const P *>(rows + s[j] * H + col);
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
                    *reinterpret_cast<P *>(drows + s[j] * H + col) = o;
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
        for (int i = 0; i < kBackThreads / 32; ++i)
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

template <typename S, int VEC>
cudaError_t unsort_vec(const void *rows, const int32_t *slot_of, const float *w, const void *add, int T, int k, int H,
                       void *y, cudaStream_t stream)
{
    const dim3 grid(T, (H + kRowThreads * VEC - 1) / (kRowThreads * VEC));
    unsort_kernel<S, VEC><<<grid, kRowThreads, 0, stream>>>(
        static_cast<const S *>(rows), slot_of, w, static_cast<const S *>(add), k, static_cast<int64_t>(T) * k, H,
        static_cast<S *>(y));
    return cudaGetLastError();
}

template <typename S, int VEC>
cudaError_t unsort_backward_vec(const void *dy, const void *rows, const int32_t *slot_of, const float *w, int T, int k,
                                int H, void *drows, float *dw, int num_sms, cudaStream_t stream)
{
    const S *g = static_cast<const S *>(dy), *r = static_cast<const S *>(rows);
    S *d = static_cast<S *>(drows);
    const int64_t N = static_cast<int64_t>(T) * k;
    // few tokens: a block per entry, so that the entries fill the SMs (dy is then read k times)
    if (T < 4 * num_sms)
        unsort_backward_kernel<S, VEC, 1><<<dim3(T, k), kBackThreads, 0, stream>>>(g, r, slot_of, w, k, N, H, d, dw);
    else
        unsort_backward_kernel<S, VEC, 8>
            <<<dim3(T, (k + 7) / 8), kBackThreads, 0, stream>>>(g, r, slot_of, w, k, N, H, d, dw);
    return cudaGetLastError();
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
    DeviceContext dc;
    if ((st = static_cast<moe_status_t>(device_context(dc))) != MOE_OK)
        return st;
    const int64_t row = static_cast<int64_t>(desc->H) * elem;
    auto go = [&](auto u) {
        return launch_sort<decltype(u)>(x, topk_idx, desc->T, desc->k, desc->E, row, x_sorted, offsets, slot_of, ws,
                                        dc.num_sms, s);
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
    const moe_status_t st = check_tokens(desc);
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
    const int bytes = pack_bytes(static_cast<int64_t>(desc->H) * elem, elem, {y_sorted, add, y});
    return launched(by_type(desc->dtype, bytes, [&](auto tag) {
        using V = decltype(tag);
        return unsort_vec<typename V::type, V::vec>(y_sorted, slot_of, topk_w, add, desc->T, desc->k, desc->H, y,
                                                    static_cast<cudaStream_t>(stream));
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
    DeviceContext dc;
    if ((st = static_cast<moe_status_t>(device_context(dc))) != MOE_OK)
        return st;
    const int bytes = pack_bytes(static_cast<int64_t>(desc->H) * elem, elem, {dy, y_sorted, dy_sorted});
    return launched(by_type(desc->dtype, bytes, [&](auto tag) {
        using V = decltype(tag);
        return unsort_backward_vec<typename V::type, V::vec>(dy, y_sorted, slot_of, topk_w, desc->T, desc->k, desc->H,
                                                             dy_sorted, dtopk_w, dc.num_sms,
                                                             static_cast<cudaStream_t>(stream));
    }));
}

}  // extern "C"
