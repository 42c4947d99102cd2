// orthogonalize.cu — orthogonalised updates of a stack of weight matrices (the update rule of
// the Muon optimiser) for the expert weights that the backward pass yields gradients of (NeMo
// AutoModel Step-5-Preview page: the layer is trained with optimizer steps).
//
// Per matrix [rows, cols], p = the shorter side, q = the longer one:
//   m <- beta m + g;  u = g + beta m (Nesterov), m, or g without momentum
//   X_0 = u / (|u|_F + eps)
//   X <- a X + B X,  B = b A + c A A,  A = X X^T           (rows <= cols)
//   X <- a X + X B,  A = X^T X                              (rows > cols)   `steps` times
//   out = bf16(scale X)
// 3 p p q + p p p flops a step, the two symmetric products counted on and above the diagonal:
// the tensor cores bound it, so each of the three products is a tcgen05 GEMM with the rest of the
// step in its epilogue.
//
// Number format. The products' operands are fp16, not bf16: every iterate is bounded (singular
// values at most max p(s), checked on the host), so fp16's range suffices with fixed
// powers of two (kSx, kSa, kSb), and its 11 bits make the rounding of an operand eight times
// smaller. The iteration multiplies a small singular value by up to a^steps (485 for the
// customary coefficients), and a rounding error outside the matrix's range with it, so
// what is not an operand stays exact to about 22 bits: X and A are held as hi + lo
// pairs of fp16 (hi the operand, lo the remainder times 2^11) and enter a X and b A in full.
// Diagonals carry most of A and B once the iterate is nearly orthogonal: the remainder of a
// rounded diagonal is kept in fp32 (ra, rb) and multiplied in by the epilogues. B X with X
// rounded is harmless, since B vanishes outside the range of X. Simulated against 64 bits, the
// result is off by 1.2e-3 (n = 320 x 1024) before its bf16 rounding (1.7e-3), against 3e-3
// without the diagonals and up to 0.15 (rank one) with X itself rounded between steps.
//
// Sums are fp32 (the tensor cores' accumulators); |u|_F is summed in 64 bits in a fixed order, so
// neither range nor order matters. No atomics: the same input gives the same bits.
#include <atomic>
#include <cmath>

#include <cuda_fp16.h>

#include "../../include/moe_b200.h"
#include "context.h"
#include "gemm_common.cuh"

namespace moe {
namespace {

constexpr float kSx = 8192.0f, kSa = 2048.0f, kSb = 2048.0f;  // scales of X, A and B in fp16
constexpr float kLo = 2048.0f;                                // scale of a lo part

enum OrthKind { kGram = 0, kSquare = 1, kUpdate = 2 };

struct OrthArgs {
    int n, p, rows, cols;
    int64_t r_mat;           // floats per matrix of ra and rb
    float *ra, *rb;          // diagonal remainders of A and B
    __nv_bfloat16 *out;      // [n, rows, cols], the last update's destination (else NULL)
    int out_wide;            // rows of out are 16-byte aligned: they leave by TMA
    float a, b, c, out_scale;
};

// ------------------------------------------------------------------------ norm and first X
struct PrepArgs {
    const void *grad;
    float *momentum;
    double *part;  // [n][parts] sums of squares
    __half *xh, *xl;
    int rows, cols, parts;
    int64_t x_pitch, x_mat;
    float beta;
    int nesterov;
    double eps;
};

__device__ __forceinline__ float load_g(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_g(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }

template <int V>
__device__ __forceinline__ void load_gv(const float *p, int64_t i, float (&v)[V])
{
    if (V % 4 == 0) {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + i + k);
            v[k] = f.x;
            v[k + 1] = f.y;
            v[k + 2] = f.z;
            v[k + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            v[k] = p[i + k];
    }
}

template <int V>
__device__ __forceinline__ void load_gv(const __nv_bfloat16 *p, int64_t i, float (&v)[V])
{
    if (V % 8 == 0) {
#pragma unroll
        for (int k = 0; k < V; k += 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(p + i + k);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                v[k + 2 * h] = __uint_as_float(w[h] << 16);
                v[k + 2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
            }
        }
    } else if (V == 4) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p + i);
        v[0] = __uint_as_float(u.x << 16);
        v[1 % V] = __uint_as_float(u.x & 0xffff0000u);
        v[2 % V] = __uint_as_float(u.y << 16);
        v[3 % V] = __uint_as_float(u.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            v[k] = __bfloat162float(p[i + k]);
    }
}

// Sum of squares in fp32 whatever the elements' size: large, small and ordinary ones have sums of their
// own, scaled so that no square leaves the range (Blue's three accumulators, 1978); 64-bit conversions
// run at a quarter of a warp a cycle and would bound the kernels.
struct Squares {
    float big = 0.0f, mid = 0.0f, small = 0.0f;
    __device__ __forceinline__ void add(float u)
    {
        const float m = fabsf(u);
        if (m > 0x1p50f) {
            const float v = u * 0x1p-70f;
            big = fmaf(v, v, big);
        } else if (m < 0x1p-50f) {
            const float v = u * 0x1p90f;
            small = fmaf(v, v, small);
        } else {
            mid = fmaf(u, u, mid);  // a NaN too
        }
    }
    // Several at once: their plain sum of squares, if it is an ordinary number, else one by one. (What
    // underflows beside an ordinary sum is below its last bit.)
    template <int V>
    __device__ __forceinline__ void add(const float (&u)[V])
    {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k)
            s = fmaf(u[k], u[k], s);
        if (s > 0x1p-90f && s < 0x1p100f)
            mid += s;
        else
#pragma unroll
            for (int k = 0; k < V; ++k)
                add(u[k]);
    }
    __device__ __forceinline__ double total() const
    {
        return static_cast<double>(big) * 0x1p140 + mid + static_cast<double>(small) * 0x1p-180;
    }
};

// u * factor in fp32 for a factor that fp32 may not hold: a power of two near its root first, which is
// exact, so that neither factor nor product leaves the range where the result does not.
struct Scale {
    float first, second;
    __device__ __forceinline__ explicit Scale(double factor)
    {
        int e;
        frexp(factor, &e);  // 0 for 0, infinities and NaN: they then pass through `second`
        e = isfinite(factor) ? e / 2 : 0;
        first = static_cast<float>(ldexp(1.0, e));
        second = static_cast<float>(ldexp(factor, -e));
    }
    __device__ __forceinline__ Scale(float f, float s) : first(f), second(s) {}
    __device__ __forceinline__ float operator()(float u) const { return u * first * second; }
};

// Updates the momentum and sums u^2 over part blockIdx.x of matrix blockIdx.y. V elements at a
// time: 8 when every matrix starts on a 32-byte boundary, else 1.
template <typename G, int V>
__global__ void __launch_bounds__(256)
    orth_norm_kernel(const PrepArgs a)
{
    __shared__ double warp_sum[8];
    allow_dependents();
    const int64_t elems = static_cast<int64_t>(a.rows) * a.cols;
    const int64_t base = blockIdx.y * elems;
    const G *g = static_cast<const G *>(a.grad) + base;
    float *m = a.momentum ? a.momentum + base : nullptr;
    const int64_t step = static_cast<int64_t>(a.parts) * 256 * V;
    Squares squares;
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V; i < elems; i += step) {
        float u[V];
        load_gv<V>(g, i, u);
        if (m) {
            float mv[V];
            load_gv<V>(m, i, mv);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                mv[k] = fmaf(a.beta, mv[k], u[k]);
                u[k] = a.nesterov ? fmaf(a.beta, mv[k], u[k]) : mv[k];
            }
            if (V % 4 == 0) {
#pragma unroll
                for (int k = 0; k < V; k += 4)
                    *reinterpret_cast<float4 *>(m + i + k) = make_float4(mv[k], mv[k + 1], mv[k + 2], mv[k + 3]);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    m[i + k] = mv[k];
            }
        }
        squares.add(u);
    }
    double sum = squares.total();
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((threadIdx.x & 31) == 0)
        warp_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < 8; ++w)
            s += warp_sum[w];
        a.part[static_cast<int64_t>(blockIdx.y) * a.parts + blockIdx.x] = s;
    }
}

__device__ __forceinline__ void split_f16(float v, __half &hi, __half &lo)
{
    hi = __float2half_rn(v);
    lo = __float2half_rn((v - __half2float(hi)) * kLo);
}

// X_0 = u / (|u|_F + eps) as hi + lo, eight columns of a row per thread (one vector load of the
// input when rows keep its alignment: kVec).
template <typename G, bool kVec>
__global__ void __launch_bounds__(256)
    orth_cast_kernel(const PrepArgs a)
{
    __shared__ double warp_sum[8];
    allow_dependents();
    dependency_wait();
    double sum = 0.0;
    for (int i = threadIdx.x; i < a.parts; i += 256)
        sum += a.part[static_cast<int64_t>(blockIdx.y) * a.parts + i];
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if ((threadIdx.x & 31) == 0)
        warp_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < 8; ++w)
        sum += warp_sum[w];
    const Scale scale(static_cast<double>(kSx) / (sqrt(sum) + a.eps));
    const int64_t base = static_cast<int64_t>(blockIdx.y) * a.rows * a.cols;
    const G *g = static_cast<const G *>(a.grad) + base;
    const float *m = a.momentum ? a.momentum + base : nullptr;
    const int groups = (a.cols + 7) / 8;
    const int64_t total = static_cast<int64_t>(groups) * a.rows;
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; w < total;
         w += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = w / groups;
        const int col = static_cast<int>(w - row * groups) * 8;
        const int64_t i = row * a.cols + col;
        float u[8];
        if (kVec) {
            load_gv<8>(g, i, u);
            if (m) {
                float mv[8];
                load_gv<8>(m, i, mv);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    u[k] = a.nesterov ? fmaf(a.beta, mv[k], u[k]) : mv[k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                u[k] = 0.0f;
                if (col + k < a.cols) {
                    u[k] = load_g(g, i + k);
                    if (m)
                        u[k] = a.nesterov ? fmaf(a.beta, m[i + k], u[k]) : m[i + k];
                }
            }
        }
        alignas(16) __half hi[8], lo[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            split_f16(scale(u[k]), hi[k], lo[k]);
        const int64_t at = blockIdx.y * a.x_mat + row * a.x_pitch + col;
        *reinterpret_cast<uint4 *>(a.xh + at) = *reinterpret_cast<const uint4 *>(hi);
        *reinterpret_cast<uint4 *>(a.xl + at) = *reinterpret_cast<const uint4 *>(lo);
    }
}

// -------------------------------------------------------------------------------- products
// One persistent kernel per product: warp 0 TMA producer, warp 1 MMA issuer and TMEM owner, warp 2
// the epilogue's mover, warps 3.. the epilogue; two accumulators in TMEM let a tile's epilogue overlap the next tile's K loop. An
// operand is K-major (X rows in A = X X^T) or MN-major (X columns in X^T X and B X), as the layout
// gives it: X is never transposed. Symmetric products compute the tiles on and above the diagonal
// and store each tile also mirrored.
//
// Two shapes. CTA pairs (cta_group::2): tiles of 256 x 256, each CTA holding 128 rows of A and of B
// and its 128 rows of the result, so an MMA reads half as much shared memory per flop. Single CTAs:
// tiles of 128 x 128, for matrices that 256-wide tiles would fill badly.
//
// The epilogue works on blocks of 128 rows x 32 columns in a ring of kBlocks buffers: a mover thread
// brings a block's old hi and lo in by TMA, one of four groups of four warps replaces them in place,
// each thread its part of one row, and the mover stores them and refills the buffer, up to kBlocks
// blocks ahead and across tiles. The update's K loop is short (p), and its epilogue bounds it: the 36 x
// 4096 x 1280 update took 554 us with one row per thread straight from and to global memory (32 lines
// an access), 475 us with a buffer per group that it refilled itself, 456 us so; 297 us without
// any epilogue, 365 us without its stores, 382 us without its arithmetic.
template <bool PAIR>
struct OrthGeo {
    static constexpr int kTile = PAIR ? 256 : 128;     // rows and columns of a tile
    static constexpr int kStages = 4;                  // 64-wide K slices in flight
    static constexpr int kGroups = 4;                  // epilogue groups of four warps
    static constexpr int kBlocks = 6;                  // epilogue buffers
    static constexpr int kThreads = 96 + 128 * kGroups;
    static constexpr uint32_t kOperand = 16384;        // 128 x 64 fp16: an operand's K slice
    static constexpr uint32_t kBlock = 8192;           // 128 x 32 fp16: a block's hi or lo
    static constexpr uint32_t kStageBytes = 2 * kOperand;
    static constexpr uint32_t kEpiOff = kStages * kStageBytes;
    static constexpr uint32_t kBarOff = kEpiOff + kBlocks * 2 * kBlock;
    static constexpr uint32_t kMiscOff = kBarOff + 8 * (2 * kStages + 5 + 2 * kBlocks);
    static constexpr uint32_t kSmem = kMiscOff + 16 + 1024;  // misc: TMEM holder, abort flag, the peer's flag and stage count
    static constexpr uint32_t kTmemCols = 2 * kTile;
    static_assert(kSmem <= static_cast<uint32_t>(kMaxDynSmem), "ring exceeds shared memory");
    static_assert(kBlocks >= kGroups && (kGroups & (kGroups - 1)) == 0, "a group's blocks are kGroups apart");
};

__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N)
{
    return (1u << 4)  // D format fp32; A and B format 0 = fp16
           | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// MN-major operand in 128-byte swizzle: 64-element MN chunks 8 KB apart, 8-row K groups 1 KB apart.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr)
{
    uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
    d |= static_cast<uint64_t>(8192 >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}

// One box into this CTA's shared memory; the bytes count on `bar`, a shared::cluster address (on CTA
// pairs the leader's barrier).
template <bool PAIR>
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *m, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2)
{
    if (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
            "{%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
            "[%2];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
            : "memory");
}

// Counts `bytes` of `bar`'s current phase as landed that no copy will bring.
__device__ __forceinline__ void mbar_complete_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void dsmem_st_s32(uint32_t addr, int v)
{
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// A pair's loads still in flight after an expired wait, which count on the leader's full barriers: the leader
// issued stages [0, mine), the peer [0, theirs), and of either at most the last S may not have landed. Neither can be
// more than S ahead, since a stage is issued when the one S before it has been multiplied, which takes both
// CTAs' bytes. A stage of one CTA alone would never complete its phase: the bytes that the other did not ask
// for are counted as landed, or the stage is armed for the peer's bytes, and then its barrier waits
// for exactly what was issued. Run by one thread of the leader once both CTAs' roles have ended.
template <int S>
__device__ __forceinline__ void drain_pair(uint64_t *full, int mine, int theirs, uint32_t stage_bytes, const WaitCfg &wc)
{
    const int most = mine > theirs ? mine : theirs;
    for (int i = most > S ? most - S : 0; i < most; ++i) {
        if (i >= theirs)
            mbar_complete_tx(&full[i % S], stage_bytes);
        else if (i >= mine)
            mbar_arrive_expect_tx(&full[i % S], stage_bytes);
        mbar_wait_drain(&full[i % S], (i / S) & 1, wc);
    }
}

struct OrthTile {
    int mat, ti, tj;  // matrix, block row and block column of the result
};

// Tiles of one matrix: the triangle ti <= tj of nm x nm, or nm x nn.
template <int KIND>
__device__ __forceinline__ int tiles_of(int nm, int nn)
{
    return KIND == kUpdate ? nm * nn : nm * (nm + 1) / 2;
}

template <int KIND>
__device__ __forceinline__ OrthTile tile_at(int tile, int per, int nm, int nn)
{
    OrthTile t;
    t.mat = tile / per;
    const int u = tile - t.mat * per;
    if (KIND == kUpdate) {
        t.ti = u / nn;
        t.tj = u - t.ti * nn;
    } else {
        int first = 0;  // first tile of block row ti
        t.ti = 0;
        while (first + nm - t.ti <= u) {
            first += nm - t.ti;
            ++t.ti;
        }
        t.tj = t.ti + (u - first);
    }
    return t;
}

// The maps of the epilogue's blocks (32 columns x 128 rows, 64-byte swizzle): old hi and lo in, new hi and lo out.
struct EpiMaps {
    CUtensorMap in_hi, in_lo, out_hi, out_lo;
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *m, const void *src, int32_t c0, int32_t c1, int32_t c2)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}

__device__ __forceinline__ float2 join_f16(uint32_t hi, uint32_t lo)
{
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    const float2 l = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    return make_float2(fmaf(l.x, 1.0f / kLo, h.x), fmaf(l.y, 1.0f / kLo, h.y));
}

// hi and lo parts of two values: hi = fp16(v), lo = fp16((v - hi) kLo), both exact but for their last rounding.
__device__ __forceinline__ float2 split_pair(float v0, float v1, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(v0, v1);
    const float2 f = __half22float2(h);
    const float2 rest = make_float2(v0 - f.x, v1 - f.y);
    const __half2 l = __floats2half2_rn(rest.x * kLo, rest.y * kLo);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
    return rest;
}

// 16 columns [col0, col0 + 16) of row `row`, which is row r and 16-byte chunks 2 * part .. of the staged
// block (64-byte swizzle). Columns from N on and rows from M on are cut off by the stores.
template <int KIND, bool TALL>
__device__ __forceinline__ void epi_part(const OrthArgs &a, int mat, int row, int col0, int M, int N,
                                         const float (&acc)[16], uint8_t *hi, uint8_t *lo, int r, int part)
{
    const float *rd = (KIND == kUpdate ? a.rb : a.ra) + mat * a.r_mat;  // padded to a multiple of 64
    constexpr bool per_row = KIND == kSquare || (KIND == kUpdate && !TALL);
    constexpr bool per_col = KIND == kSquare || (KIND == kUpdate && TALL);
    const float r_row = per_row && row < M ? rd[row] : 0.0f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t at = r * 64 + (((part * 2 + c) ^ ((r >> 1) & 3)) << 4);
        uint4 h4 = make_uint4(0, 0, 0, 0), l4 = make_uint4(0, 0, 0, 0);
        if (KIND != kGram) {
            h4 = *reinterpret_cast<const uint4 *>(hi + at);
            l4 = *reinterpret_cast<const uint4 *>(lo + at);
        }
        uint32_t h[4] = {h4.x, h4.y, h4.z, h4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = col0 + 8 * c + 2 * i;
            const float m0 = acc[8 * c + 2 * i], m1 = acc[8 * c + 2 * i + 1];
            float v0, v1;
            if (KIND == kGram) {
                v0 = m0 * (kSa / (kSx * kSx));
                v1 = m1 * (kSa / (kSx * kSx));
            } else {
                const float2 old = join_f16(h[i], l[i]);
                float2 rr = make_float2(r_row, r_row);
                if (per_col) {
                    const float2 rc = *reinterpret_cast<const float2 *>(rd + col);
                    rr.x += rc.x;
                    rr.y += rc.y;
                }
                if (KIND == kSquare) {
                    const float f = a.c * (kSb / kSa) * (1.0f / kSa);
                    v0 = fmaf(a.b, old.x, f * fmaf(rr.x, old.x, m0));
                    v1 = fmaf(a.b, old.y, f * fmaf(rr.y, old.y, m1));
                } else {
                    v0 = fmaf(fmaf(rr.x, 1.0f / kSb, a.a), old.x, m0 * (1.0f / kSb));
                    v1 = fmaf(fmaf(rr.y, 1.0f / kSb, a.a), old.y, m1 * (1.0f / kSb));
                }
            }
            if (KIND == kUpdate && a.out) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v0 * a.out_scale, v1 * a.out_scale);
                h[i] = *reinterpret_cast<const uint32_t *>(&b);
            } else {
                const float2 rest = split_pair(v0, v1, h[i], l[i]);
                if (KIND != kUpdate && row - col >= 0 && row - col < 2 && row < M)  // the diagonal
                    ((KIND == kGram) ? a.ra : a.rb)[mat * a.r_mat + row] = row == col ? rest.x : rest.y;
            }
        }
        if (KIND == kUpdate && a.out && !a.out_wide) {
            __nv_bfloat16 *o = a.out + (static_cast<int64_t>(mat) * a.rows + row) * a.cols + col0 + 8 * c;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (row < M && col0 + 8 * c + i < N)
                    o[i] = __ushort_as_bfloat16(static_cast<uint16_t>(h[i / 2] >> (i % 2 * 16)));
            continue;
        }
        *reinterpret_cast<uint4 *>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
        if (KIND == kGram || (KIND == kUpdate && !a.out))
            *reinterpret_cast<uint4 *>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// An operand from a symmetric matrix of which only the blocks on and above the diagonal are
// stored: rows of block row `blk`, K slice k0. Block (blk, k0 / TILE) is stored if it is not below
// the diagonal (K-major boxes); else its mirror image is, and is read as an MN-major operand.
template <int TILE>
__device__ __forceinline__ bool stored_mirrored(int blk, int k0)
{
    return k0 / TILE < blk;
}

// 128 rows (from mn0) x 64 (from k0) of an operand into shared memory.
template <bool PAIR>
__device__ __forceinline__ void load_operand(uint8_t *dst, const CUtensorMap *km, const CUtensorMap *mn, uint32_t bar,
                                             int mn0, int k0, int mat, bool mn_major)
{
    if (mn_major) {
        tma_load_3d<PAIR>(dst, mn, bar, mn0, k0, mat);
        tma_load_3d<PAIR>(dst + 8192, mn, bar, mn0 + 64, k0, mat);
    } else {
        tma_load_3d<PAIR>(dst, km, bar, k0, mn0, mat);
    }
}

// The epilogue's blocks of one CTA in order: the 32-column blocks of its tiles. A pair's second half of
// a tile that lies outside the matrix has none.
template <int KIND, int TILE>
struct BlockWalk {
    int tile, b, nb, row0, n0;
    OrthTile t;
    __device__ __forceinline__ void start(int first, int tiles, int stride, int per, int nm, int nn, int rank, int M, int N)
    {
        tile = first - stride;
        b = nb = 0;
        next(tiles, stride, per, nm, nn, rank, M, N);
    }
    // to the next block (b = nb = 0 on entry: to the first block of the tile after `tile`)
    __device__ __forceinline__ void next(int tiles, int stride, int per, int nm, int nn, int rank, int M, int N)
    {
        if (++b < nb)
            return;
        do {
            tile += stride;
            if (tile >= tiles)
                return;
            t = tile_at<KIND>(tile, per, nm, nn);
            row0 = t.ti * TILE + rank * 128;
            n0 = t.tj * TILE;
            nb = row0 < M ? ((N - n0 < TILE ? N - n0 : TILE) + 31) / 32 : 0;
        } while (nb == 0);
        b = 0;
    }
};

// MN-major operands: X in A = X^T X (tall) and the right factor X of B X (wide).
//
// On CTA pairs the leader (cluster rank 0) issues the MMAs; both CTAs' loads count on the leader's
// full barriers, the leader's commits arrive in both CTAs, and both epilogues arrive on the leader's
// accumulator-empty barriers. Without an expired wait every load was multiplied and has landed with that;
// with one in either CTA, both hear of it in the final cluster barrier, and neither leaves before drain_pair.
template <int KIND, bool TALL, bool PAIR>
__global__ void __launch_bounds__(OrthGeo<PAIR>::kThreads, 1)
    orth_gemm_kernel(const __grid_constant__ CUtensorMap a_km, const __grid_constant__ CUtensorMap a_mn,
                     const __grid_constant__ CUtensorMap b_km, const __grid_constant__ CUtensorMap b_mn,
                     const __grid_constant__ EpiMaps em, const OrthArgs a, const WaitCfg wc)
{
    using G = OrthGeo<PAIR>;
    constexpr int S = G::kStages, TILE = G::kTile;
    // operand sources: a symmetric matrix (A, B), or X as its layout gives it
    constexpr bool kAsym = KIND == kSquare || (KIND == kUpdate && !TALL);
    constexpr bool kBsym = KIND == kSquare || (KIND == kUpdate && TALL);
    constexpr bool kAmn = KIND == kGram && TALL;
    constexpr bool kBmn = (KIND == kGram && TALL) || (KIND == kUpdate && !TALL);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + G::kBarOff);
    uint64_t *empty = full + S;
    uint64_t *accf = empty + S;
    uint64_t *acce = accf + 2;
    uint64_t *drain = acce + 2;
    uint64_t *bfull = drain + 1;           // [kBlocks] a block's old values have landed
    uint64_t *bdone = bfull + G::kBlocks;  // [kBlocks] its new ones are written
    uint32_t *holder = reinterpret_cast<uint32_t *>(smem + G::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + G::kMiscOff + 4);
    volatile int *peer_abort = abort_flag + 1, *peer_issued = abort_flag + 2;  // written by the pair's other CTA
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
    const uint32_t full0 = PAIR ? dsmem_addr(smem_u32(full), 0) : smem_u32(full);
    const uint32_t acce0 = PAIR ? dsmem_addr(smem_u32(acce), 0) : smem_u32(acce);
    allow_dependents();
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], (PAIR ? 2 : 1) * 4 * G::kGroups);
        }
        for (int b = 0; b < G::kBlocks; ++b) {
            mbar_init(&bfull[b], 1);
            mbar_init(&bdone[b], 4);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        *peer_abort = 0;
        *peer_issued = 0;
        fence_barrier_init();
        tma_prefetch_map(&a_km);
        tma_prefetch_map(&a_mn);
        tma_prefetch_map(&b_km);
        tma_prefetch_map(&b_mn);
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(holder, G::kTmemCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(holder, G::kTmemCols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    if (PAIR)
        cluster_sync_all();  // both CTAs' barriers are initialised before any remote arrival
    else
        __syncthreads();
    tc_fence_after();
    dependency_wait();  // the launch before has written this one's operands
    const uint32_t tmem = *holder;
    const int M = KIND == kUpdate ? a.rows : a.p, N = KIND == kUpdate ? a.cols : a.p;
    const int K = KIND == kGram ? (TALL ? a.rows : a.cols) : a.p;
    const int nm = (M + TILE - 1) / TILE, nn = (N + TILE - 1) / TILE;
    const int nk = (K + 63) / 64;  // K slices of a tile
    const int per = tiles_of<KIND>(nm, nn);
    const int tiles = per * a.n;
    const int first = PAIR ? blockIdx.x >> 1 : blockIdx.x, stride = PAIR ? gridDim.x >> 1 : gridDim.x;

    int it = 0;  // stages that the producer has issued
    if (warp == 0) {
        if (lane == 0) {
            bool stop = false;
            for (int tile = first; tile < tiles && !stop; tile += stride) {
                const OrthTile t = tile_at<KIND>(tile, per, nm, nn);
                const int m0 = t.ti * TILE + rank * 128, n0 = t.tj * TILE + rank * 128;
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = it % S;
                    if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1, wc, abort_flag)) {
                        stop = true;
                        break;
                    }
                    if (rank == 0)
                        mbar_arrive_expect_tx(&full[s], (PAIR ? 2 : 1) * G::kStageBytes);
                    uint8_t *A = smem + s * G::kStageBytes, *B = A + G::kOperand;
                    const uint32_t bar = full0 + 8 * s;
                    const int k0 = kb * 64;
                    load_operand<PAIR>(A, &a_km, &a_mn, bar, m0, k0, t.mat,
                                       kAsym ? stored_mirrored<TILE>(t.ti, k0) : kAmn);
                    load_operand<PAIR>(B, &b_km, &b_mn, bar, n0, k0, t.mat,
                                       kBsym ? stored_mirrored<TILE>(t.tj, k0) : kBmn);
                }
            }
            // the loads this CTA issued have landed before it leaves (a pair's: behind the roles)
            if (PAIR) {
                if (rank == 1)
                    dsmem_st_s32(dsmem_addr(smem_u32(const_cast<const int *>(peer_issued)), 0), it);
            } else {
                for (int i = it > S ? it - S : 0; i < it; ++i)
                    mbar_wait_drain(&full[i % S], (i / S) & 1, wc);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int tc = 0, s = 0;
            uint32_t par = 0;
            bool ok = true;
            for (int tile = first; tile < tiles && ok; tile += stride, ++tc) {
                const OrthTile t = tile_at<KIND>(tile, per, nm, nn);
                const int buf = tc & 1;
                if (!mbar_wait(&acce[buf], ((tc >> 1) & 1) ^ 1, wc, abort_flag))
                    break;
                tc_fence_after();
                const int left = N - t.tj * TILE;
                const int cols = !PAIR && left < TILE ? (left + 15) & ~15 : TILE;
                const uint32_t d = tmem + buf * TILE;
                bool ready = mbar_test(&full[s], par);
                for (int kb = 0; kb < nk; ++kb) {
                    if (!ready && !mbar_wait(&full[s], par, wc, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int cur = s;
                    if (++s == S) {
                        s = 0;
                        par ^= 1;
                    }
                    // the next slice's barrier is asked for ahead of this slice's MMAs: its answer comes
                    // while they are issued, and the pipe does not run dry for the length of a test
                    ready = mbar_test(&full[s], par);
                    const uint32_t sa = smem_u32(smem + cur * G::kStageBytes), sb = sa + G::kOperand;
                    const bool amn = kAsym ? stored_mirrored<TILE>(t.ti, kb * 64) : kAmn;
                    const bool bmn = kBsym ? stored_mirrored<TILE>(t.tj, kb * 64) : kBmn;
                    // one K step of 16: 32 bytes of a K-major row, 16 rows of an MN-major operand
                    const uint64_t ad = amn ? sdesc_mn(sa) : sdesc_kmajor_sw128(sa);
                    const uint64_t bd = bmn ? sdesc_mn(sb) : sdesc_kmajor_sw128(sb);
                    const int as = amn ? 2048 >> 4 : 2, bs = bmn ? 2048 >> 4 : 2;
                    const uint32_t idesc =
                        idesc_f16_f32(TILE, cols) | (amn ? 1u << 15 : 0u) | (bmn ? 1u << 16 : 0u);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        // kind::f16: the operands' type, fp16, is in idesc
                        if (PAIR)
                            umma_bf16_pair(d, ad + as * ks, bd + bs * ks, idesc, (kb | ks) != 0);
                        else
                            umma_bf16(d, ad + as * ks, bd + bs * ks, idesc, (kb | ks) != 0);
                    }
                    if (PAIR)
                        umma_commit_pair_mc(&empty[cur], 0x3);
                    else
                        umma_commit(&empty[cur]);
                }
                if (ok) {
                    if (PAIR)
                        umma_commit_pair_mc(&accf[buf], 0x3);
                    else
                        umma_commit(&accf[buf]);
                }
            }
            if (PAIR)
                umma_commit_pair_mc(drain, 0x3);
            else
                umma_commit(drain);
        }
        if (lane == 0)
            mbar_wait_drain(drain, 0, wc);
    } else if (warp == 2) {
        if (lane == 0) {
            const bool last = KIND == kUpdate && a.out != nullptr;
            BlockWalk<KIND, TILE> in, out;
            in.start(first, tiles, stride, per, nm, nn, rank, M, N);
            out = in;
            int loaded = 0;
            const auto fetch = [&]() {
                const int u = loaded % G::kBlocks;
                uint8_t *hi = smem + G::kEpiOff + u * 2 * G::kBlock;
                if (KIND == kGram) {
                    mbar_arrive(&bfull[u]);
                } else {
                    mbar_arrive_expect_tx(&bfull[u], 2 * G::kBlock);
                    tma_load_3d<false>(hi, &em.in_hi, smem_u32(&bfull[u]), in.n0 + in.b * 32, in.row0, in.t.mat);
                    tma_load_3d<false>(hi + G::kBlock, &em.in_lo, smem_u32(&bfull[u]), in.n0 + in.b * 32, in.row0,
                                       in.t.mat);
                }
                ++loaded;
                in.next(tiles, stride, per, nm, nn, rank, M, N);
            };
            while (loaded < G::kBlocks && in.tile < tiles)
                fetch();
            for (int i = 0; out.tile < tiles; ++i) {
                const int u = i % G::kBlocks;
                if (!mbar_wait(&bdone[u], (i / G::kBlocks) & 1, wc, abort_flag))
                    break;
                const uint8_t *hi = smem + G::kEpiOff + u * 2 * G::kBlock;
                if (!last || a.out_wide)
                    tma_store_3d(&em.out_hi, hi, out.n0 + out.b * 32, out.row0, out.t.mat);
                if (KIND == kGram || (KIND == kUpdate && !last))
                    tma_store_3d(&em.out_lo, hi + G::kBlock, out.n0 + out.b * 32, out.row0, out.t.mat);
                bulk_commit();
                out.next(tiles, stride, per, nm, nn, rank, M, N);
                if (in.tile < tiles) {
                    bulk_wait_read<0>();
                    fetch();
                }
            }
            // every load has landed and every store arrived before the CTA (and its shared memory) goes
            for (int i = loaded > G::kBlocks ? loaded - G::kBlocks : 0; i < loaded; ++i)
                mbar_wait_drain(&bfull[i % G::kBlocks], (i / G::kBlocks) & 1, wc);
            bulk_wait<0>();
        }
    } else {
        const int q = warp & 3, grp = (warp - 3) / 4, r = q * 32 + lane;
        int tc = 0, i0 = 0;  // i0: blocks of the CTA before the tile's
        bool ok = true;
        for (int tile = first; tile < tiles && ok; tile += stride, ++tc) {
            const OrthTile t = tile_at<KIND>(tile, per, nm, nn);
            const int buf = tc & 1;
            const int row0 = t.ti * TILE + rank * 128, n0 = t.tj * TILE;
            const int nb = row0 < M ? ((N - n0 < TILE ? N - n0 : TILE) + 31) / 32 : 0;
            ok = warp_wait(&accf[buf], (tc >> 1) & 1, wc, abort_flag);
            tc_fence_after();
            // Groups go by the CTA's block number, so that a group's next block is never more than
            // kBlocks behind its last one: a barrier's parity could not tell phases two apart.
            for (int b = (grp - i0) & (G::kGroups - 1); b < nb && ok; b += G::kGroups) {
                const int i = i0 + b, u = i % G::kBlocks;
                ok = warp_wait(&bfull[u], (i / G::kBlocks) & 1, wc, abort_flag);
                if (!ok)
                    break;
                uint8_t *hi = smem + G::kEpiOff + u * 2 * G::kBlock;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const int off = b * 32 + part * 16;
                    float v[16];
                    tmem_load16(tmem + buf * TILE + (static_cast<uint32_t>(q * 32) << 16) + off, v);
                    epi_part<KIND, TALL>(a, t.mat, row0 + r, n0 + off, M, N, v, hi, hi + G::kBlock, r, part);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bdone[u]);
            }
            i0 += nb;
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && ok) {
                if (PAIR)
                    mbar_arrive_cluster(acce0 + 8 * buf);
                else
                    mbar_arrive(&acce[buf]);
            }
        }
    }
    tc_fence_before();
    if (PAIR) {
        if (*abort_flag)  // seen by the thread that set it, if by no other
            dsmem_st_s32(dsmem_addr(smem_u32(const_cast<const int *>(peer_abort)), rank ^ 1), 1);
        cluster_sync_all();  // both CTAs are done with TMEM, shared memory and each other's barriers
        if (*abort_flag || *peer_abort) {
            if (threadIdx.x == 0 && rank == 0)
                drain_pair<S>(full, it, *peer_issued, G::kStageBytes, wc);
            cluster_sync_all();
        }
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        if (PAIR)
            tmem_dealloc_pair(tmem, G::kTmemCols);
        else
            tmem_dealloc(tmem, G::kTmemCols);
    }
}

template <int KIND, bool TALL, bool PAIR>
cudaError_t launch_gemm(const CUtensorMap &a_km, const CUtensorMap &a_mn, const CUtensorMap &b_km,
                        const CUtensorMap &b_mn, const EpiMaps &em, const OrthArgs &a, const DeviceContext &dc,
                        cudaStream_t stream)
{
    using G = OrthGeo<PAIR>;
    auto kernel = orth_gemm_kernel<KIND, TALL, PAIR>;
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(G::kSmem));
    if (err != cudaSuccess)
        return err;
    const int M = KIND == kUpdate ? a.rows : a.p, N = KIND == kUpdate ? a.cols : a.p;
    const int nm = (M + G::kTile - 1) / G::kTile, nn = (N + G::kTile - 1) / G::kTile;
    const int64_t tiles = static_cast<int64_t>(KIND == kUpdate ? nm * nn : nm * (nm + 1) / 2) * a.n;
    const int64_t slots = PAIR ? dc.num_sms / 2 : dc.num_sms;
    const int grid = static_cast<int>(tiles < slots ? tiles : slots) * (PAIR ? 2 : 1);
    return launch_dependent(kernel, dim3(grid), G::kThreads, G::kSmem, stream, PAIR ? 2 : 1, a_km, a_mn,
                            b_km, b_mn, em, a, dc.wait);
}

__device__ __forceinline__ uint32_t cluster_nctarank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ float4 dsmem_ld_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// ---------------------------------------------------------------------- products split over K
// Products of few tiles: a cluster of C CTAs per 128 x 128 tile, each with its share of the K slices; the
// parts are summed through distributed shared memory in rank order, each CTA a share of the tile's rows, with the same
// arithmetic behind as in epi_part. A tile on the diagonal of A or B loads its slices once. What bounds such products
// is the way through one tile, so both the K loop and the epilogue get shorter: 1 x 256 x 4096 (A: 3 tiles of
// 64 slices) 199 -> 108 us a call, 1 x 1000 x 1000 178 -> 136, 4 x 200 x 600 119 -> 100.
constexpr int kSplitThreads = 512;
constexpr int kSplitMaxC = 8;
constexpr uint32_t kSplitRed = OrthGeo<false>::kStages * OrthGeo<false>::kStageBytes;  // this CTA's part, fp32
constexpr uint32_t kSplitBar = kSplitRed + 128 * 128 * 4;
constexpr uint32_t kSplitSmem = kSplitBar + 8 * (2 * OrthGeo<false>::kStages + 1) + 16 + 1024;
static_assert(kSplitSmem <= static_cast<uint32_t>(kMaxDynSmem), "shared memory");

struct SplitArgs {
    const __half *old_hi, *old_lo;  // what the epilogue multiplies in (A; X), NULL for A's product
    __half *hi, *lo;                // the result; lo NULL for B
    int64_t pitch, mat;             // of all of them, elements
};

template <int KIND, bool TALL>
__global__ void __launch_bounds__(kSplitThreads, 1)
    orth_split_kernel(const __grid_constant__ CUtensorMap a_km, const __grid_constant__ CUtensorMap a_mn,
                      const __grid_constant__ CUtensorMap b_km, const __grid_constant__ CUtensorMap b_mn,
                      const OrthArgs a, const SplitArgs sp, const WaitCfg wc)
{
    using G = OrthGeo<false>;
    constexpr int S = G::kStages;
    // operand sources as in orth_gemm_kernel
    constexpr bool kAsym = KIND == kSquare || (KIND == kUpdate && !TALL);
    constexpr bool kBsym = KIND == kSquare || (KIND == kUpdate && TALL);
    constexpr bool kAmn = KIND == kGram && TALL;
    constexpr bool kBmn = (KIND == kGram && TALL) || (KIND == kUpdate && !TALL);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *red = reinterpret_cast<float *>(smem + kSplitRed);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kSplitBar);
    uint64_t *empty = full + S, *done = empty + S;
    uint32_t *holder = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(holder + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
    allow_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_barrier_init();
        tma_prefetch_map(&a_km);
        tma_prefetch_map(&a_mn);
        tma_prefetch_map(&b_km);
        tma_prefetch_map(&b_mn);
    }
    if (warp == 1) {
        tmem_alloc(holder, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    dependency_wait();
    const uint32_t tmem = *holder;
    const int M = KIND == kUpdate ? a.rows : a.p, N = KIND == kUpdate ? a.cols : a.p;
    const int K = KIND == kGram ? (TALL ? a.rows : a.cols) : a.p;
    const int nm = (M + 127) / 128, nn = (N + 127) / 128, nk = (K + 63) / 64, share = (nk + C - 1) / C;
    const int parts = (nk + share - 1) / share;  // CTAs that have slices
    const int kb0 = rank * share, kb1 = kb0 + share < nk ? kb0 + share : nk;
    const OrthTile t = tile_at<KIND>(blockIdx.x / C, tiles_of<KIND>(nm, nn), nm, nn);
    const int m0 = t.ti * 128, n0 = t.tj * 128;
    const bool one = KIND != kUpdate && t.ti == t.tj;  // both operands are the same rows

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % S;
                if (!mbar_wait(&empty[s], ((it / S) & 1) ^ 1, wc, abort_flag))
                    break;
                mbar_arrive_expect_tx(&full[s], one ? G::kOperand : G::kStageBytes);
                uint8_t *A = smem + s * G::kStageBytes;
                const int k0 = kb * 64;
                load_operand<false>(A, &a_km, &a_mn, smem_u32(&full[s]), m0, k0, t.mat,
                                    kAsym ? stored_mirrored<128>(t.ti, k0) : kAmn);
                if (!one)
                    load_operand<false>(A + G::kOperand, &b_km, &b_mn, smem_u32(&full[s]), n0, k0, t.mat,
                                        kBsym ? stored_mirrored<128>(t.tj, k0) : kBmn);
            }
            for (int i = it > S ? it - S : 0; i < it; ++i)
                mbar_wait_drain(&full[i % S], (i / S) & 1, wc);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % S;
                if (!mbar_wait(&full[s], (it / S) & 1, wc, abort_flag))
                    break;
                tc_fence_after();
                const uint32_t sa = smem_u32(smem + s * G::kStageBytes), sb = one ? sa : sa + G::kOperand;
                const bool amn = kAsym ? stored_mirrored<128>(t.ti, kb * 64) : kAmn;
                const bool bmn = kBsym ? stored_mirrored<128>(t.tj, kb * 64) : kBmn;
                const uint64_t ad = amn ? sdesc_mn(sa) : sdesc_kmajor_sw128(sa);
                const uint64_t bd = bmn ? sdesc_mn(sb) : sdesc_kmajor_sw128(sb);
                const int as = amn ? 2048 >> 4 : 2, bs = bmn ? 2048 >> 4 : 2;
                const uint32_t idesc = idesc_f16_f32(128, 128) | (amn ? 1u << 15 : 0u) | (bmn ? 1u << 16 : 0u);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    umma_bf16(tmem, ad + as * ks, bd + bs * ks, idesc, (it | ks) != 0);
                umma_commit(&empty[s]);
            }
            umma_commit(done);
            mbar_wait_drain(done, 0, wc);
        }
        __syncwarp();
    }
    warp_wait(done, 0, wc, abort_flag);
    tc_fence_after();
    // 16-byte columns rotated by the row, which keeps a column's stores off one bank
    if (kb0 < kb1) {
        const int r = (warp & 3) * 32 + lane, cg = warp >> 2;
        float v[32];
        tmem_load32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + cg * 32, v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            *reinterpret_cast<float4 *>(red + r * 128 + ((cg * 8 + k + r) & 31) * 4) =
                make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
    tc_fence_before();
    cluster_sync_all();
    constexpr bool per_row = KIND == kSquare || (KIND == kUpdate && !TALL);
    constexpr bool per_col = KIND == kSquare || (KIND == kUpdate && TALL);
    const float *rd = (KIND == kUpdate ? a.rb : a.ra) + t.mat * a.r_mat;  // padded to a multiple of 64
    const bool last = KIND == kUpdate && a.out != nullptr;
    for (int e = rank * kSplitThreads + threadIdx.x; e < 128 * 32; e += C * kSplitThreads) {
        const int i = e >> 5, row = m0 + i, col = n0 + (e & 31) * 4;
        if (row >= M || col >= N)  // (the columns of the last four that are not the matrix's are in its padding)
            continue;
        const int64_t at = t.mat * sp.mat + row * sp.pitch + col;
        uint2 oh = make_uint2(0, 0), ol = make_uint2(0, 0);
        float4 rest = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (KIND != kGram) {
            oh = *reinterpret_cast<const uint2 *>(sp.old_hi + at);
            ol = *reinterpret_cast<const uint2 *>(sp.old_lo + at);
        }
        if (per_col)
            rest = *reinterpret_cast<const float4 *>(rd + col);
        if (per_row) {
            const float x = rd[row];
            rest = make_float4(rest.x + x, rest.y + x, rest.z + x, rest.w + x);
        }
        const uint32_t from = smem_u32(red + i * 128 + (((e & 31) + i) & 31) * 4);
        float4 v[kSplitMaxC];
#pragma unroll
        for (int c = 0; c < kSplitMaxC; ++c)
            if (c < parts)
                v[c] = dsmem_ld_f4(dsmem_addr(from, c));
        float4 m = v[0];
#pragma unroll
        for (int c = 1; c < kSplitMaxC; ++c)
            if (c < parts) {
                m.x += v[c].x;
                m.y += v[c].y;
                m.z += v[c].z;
                m.w += v[c].w;
            }
        const float2 o0 = join_f16(oh.x, ol.x), o1 = join_f16(oh.y, ol.y);
        if (KIND == kGram) {
            const float f = kSa / (kSx * kSx);
            m = make_float4(m.x * f, m.y * f, m.z * f, m.w * f);
        } else if (KIND == kSquare) {
            const float f = a.c * (kSb / kSa) * (1.0f / kSa);
            m.x = fmaf(a.b, o0.x, f * fmaf(rest.x, o0.x, m.x));
            m.y = fmaf(a.b, o0.y, f * fmaf(rest.y, o0.y, m.y));
            m.z = fmaf(a.b, o1.x, f * fmaf(rest.z, o1.x, m.z));
            m.w = fmaf(a.b, o1.y, f * fmaf(rest.w, o1.y, m.w));
        } else {
            const float f = 1.0f / kSb;
            m.x = fmaf(fmaf(rest.x, f, a.a), o0.x, m.x * f);
            m.y = fmaf(fmaf(rest.y, f, a.a), o0.y, m.y * f);
            m.z = fmaf(fmaf(rest.z, f, a.a), o1.x, m.z * f);
            m.w = fmaf(fmaf(rest.w, f, a.a), o1.y, m.w * f);
        }
        uint2 h, l;
        if (last) {
            const __nv_bfloat162 b0 = __floats2bfloat162_rn(m.x * a.out_scale, m.y * a.out_scale);
            const __nv_bfloat162 b1 = __floats2bfloat162_rn(m.z * a.out_scale, m.w * a.out_scale);
            __nv_bfloat16 *o = a.out + (static_cast<int64_t>(t.mat) * M + row) * N + col;
            if (a.out_wide) {  // N is a multiple of 8
                *reinterpret_cast<uint2 *>(o) = make_uint2(*reinterpret_cast<const uint32_t *>(&b0),
                                                           *reinterpret_cast<const uint32_t *>(&b1));
            } else {
                const __nv_bfloat16 b[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (col + k < N)
                        o[k] = b[k];
            }
            continue;
        }
        const float2 r0 = split_pair(m.x, m.y, h.x, l.x), r1 = split_pair(m.z, m.w, h.y, l.y);
        *reinterpret_cast<uint2 *>(sp.hi + at) = h;
        if (KIND != kSquare)
            *reinterpret_cast<uint2 *>(sp.lo + at) = l;
        if (KIND != kUpdate && row >= col && row < col + 4)  // the diagonal
            (KIND == kGram ? a.ra : a.rb)[t.mat * a.r_mat + row] =
                row == col ? r0.x : (row == col + 1 ? r0.y : (row == col + 2 ? r1.x : r1.y));
    }
    cluster_sync_all();  // no CTA leaves while a peer may still read its part
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 128);
    }
}

// Clusters of each size (2, 4, 8) that the current device runs at a time, which its groups of SMs decide. The same for
// every product's kernel: one CTA per SM.
struct SplitRoom {
    int clusters[3];
};

cudaError_t split_room(SplitRoom &room)
{
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][3];  // clusters + 1
    int device = 0;
    cudaError_t err = cudaGetDevice(&device);
    for (int i = 0; i < 3 && err == cudaSuccess; ++i) {
        const int have = device < kDevices ? known[device][i].load(std::memory_order_relaxed) : 0;
        if (have) {
            room.clusters[i] = have - 1;
            continue;
        }
        auto kernel = orth_split_kernel<kGram, false>;
        err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSplitSmem));
        if (err != cudaSuccess)
            break;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 << i);
        cfg.blockDim = dim3(kSplitThreads);
        cfg.dynamicSmemBytes = kSplitSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2 << i;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        err = cudaOccupancyMaxActiveClusters(&room.clusters[i], kernel, &cfg);
        if (err == cudaSuccess && device < kDevices)
            known[device][i].store(room.clusters[i] + 1, std::memory_order_relaxed);
    }
    return err;
}

// CTAs per tile, 0: not split. The most for which all clusters run at once and each CTA has a K slice:
// 5 x 256 x 1000 (15 tiles by 8) 132 -> 108 us, 22 x 256 x 2000 (66 by 2) 249 -> 217 us; the 36 tiles of 12 x 256 x 256 by 4
// are too many for one wave, 153 us, by 2 105, not split 112 us.
int split_of(int64_t tiles, int K, const SplitRoom &room)
{
    for (int i = 2; i >= 0; --i)
        if (tiles <= room.clusters[i] && (K + 63) / 64 >= 2 << i)
            return 2 << i;
    return 0;
}

template <int KIND, bool TALL>
cudaError_t launch_split(int C, int64_t tiles, const CUtensorMap &a_km, const CUtensorMap &a_mn,
                         const CUtensorMap &b_km, const CUtensorMap &b_mn, const OrthArgs &a, const SplitArgs &sp,
                         const DeviceContext &dc, cudaStream_t stream)
{
    auto kernel = orth_split_kernel<KIND, TALL>;
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSplitSmem));
    if (err != cudaSuccess)
        return err;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(tiles * C)), kSplitThreads, kSplitSmem, stream, C, a_km,
                            a_mn, b_km, b_mn, a, sp, dc.wait);
}

// --------------------------------------------------------------------------- short matrices
// p <= 128: a whole call in one launch, a cluster of C CTAs per matrix. CTA c holds columns [c W, (c + 1) W)
// of X (rows of the input, for a tall matrix) for all steps: X in fp32 in tensor memory, one row per
// lane, and its fp16 rounding in shared memory, a buffer that serves the Gram product K-major and the
// update MN-major. Per step: A's partial products (M = N = 128, K = W), summed over the cluster through distributed
// shared memory (each CTA a share of the elements, in rank order) and handed to every CTA as hi and lo; A A, B and
// the update in each CTA for its own columns. What is exact and what is rounded is as in the products
// below, but that X is fp32 itself. In place of 17 launches, whose latency bounds such matrices: 32 x
// 128 x 256 99 -> 37 us, 1 x 128 x 1024 112 -> 56 us.
constexpr int kShortThreads = 512;
constexpr int kShortMaxP = 128;
constexpr int kShortMaxW = 256;    // columns of a CTA: X and the update's accumulator share tensor memory
constexpr int kShortMaxC = 8;      // CTAs of a cluster
constexpr uint32_t kChunk = 16384; // 128 rows x 64 columns fp16
constexpr uint32_t kShortXh = 0;                      // 4 chunks
constexpr uint32_t kShortAh = 4 * kChunk;             // 2 chunks
constexpr uint32_t kShortAl = kShortAh + 2 * kChunk;  // 2 chunks
constexpr uint32_t kShortRed = kShortAl + 2 * kChunk; // this CTA's part of A, fp32; then B, fp16
constexpr uint32_t kShortStage = kShortAh;            // the first X before it is scaled, then A, B's place
constexpr uint32_t kShortVec = kShortStage + kShortMaxP * (kShortMaxW + 4) * 4;  // ra, rb [128] floats
static_assert(kShortVec >= kShortRed + 4 * kChunk, "the stage covers the buffers behind Xh");
constexpr uint32_t kShortMisc = kShortVec + 1024;
constexpr uint32_t kShortSmem = kShortMisc + 512 + 1024;
static_assert(kShortSmem <= static_cast<uint32_t>(kMaxDynSmem), "shared memory");
static_assert(kShortAh + kShortMaxP * (kShortMaxW + 8) * 2 <= kShortVec, "the result is staged behind X");

struct ShortArgs {
    const void *grad;
    float *momentum;
    __nv_bfloat16 *out;
    int rows, cols, p, W, steps, nesterov;
    float a, b, c, out_scale, beta;
    double eps;
};

__device__ __forceinline__ void fence_proxy_async_all()
{
    asm volatile("fence.proxy.async;" ::: "memory");
}

__device__ __forceinline__ double dsmem_ld_f64(uint32_t addr)
{
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void dsmem_st_u2(uint32_t addr, uint32_t x, uint32_t y)
{
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ void dsmem_st_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// MN-major operand like sdesc_mn, its 64-element MN chunks a whole chunk (128 K rows) apart.
__device__ __forceinline__ uint64_t sdesc_mn_chunk(uint32_t saddr)
{
    uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
    d |= static_cast<uint64_t>(kChunk >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}

// Byte offset of columns [col, col + 8) of row r in a buffer of 64-column chunks (128-byte swizzle).
__device__ __forceinline__ uint32_t chunk_at8(int r, int col)
{
    return static_cast<uint32_t>(col >> 6) * kChunk + r * 128 + ((((col >> 3) & 7) ^ (r & 7)) << 4);
}

template <typename G, bool TALL, int V>
__global__ void __launch_bounds__(kShortThreads, 1)
    orth_short_kernel(const ShortArgs a, const WaitCfg wc)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *ra = reinterpret_cast<float *>(smem + kShortVec), *rb = ra + 128;
    uint64_t *mma = reinterpret_cast<uint64_t *>(smem + kShortMisc);
    uint32_t *holder = reinterpret_cast<uint32_t *>(smem + kShortMisc + 8);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kShortMisc + 12);
    double *part = reinterpret_cast<double *>(smem + kShortMisc + 16);   // [1] this CTA's sum of squares
    float *factors = reinterpret_cast<float *>(smem + kShortMisc + 24);  // [2] of the first X's scale
    double *warp_sum = reinterpret_cast<double *>(smem + kShortMisc + 64);  // [16]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
    const int mat = blockIdx.x / C;
    const int p = a.p, W = a.W, q = TALL ? a.rows : a.cols;
    const int q0 = rank * W, w = q - q0 < W ? (q - q0 > 0 ? q - q0 : 0) : W;  // this CTA's columns of X
    if (threadIdx.x == 0) {
        mbar_init(mma, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc(holder, 512);
        tmem_relinquish();
    }
    if (threadIdx.x < 256)
        ra[threadIdx.x] = 0.0f;  // ra and rb: rows that A and B do not have stay zero

    // u (and the momentum) in the order of memory, summed and staged as floats [p][pitch]; V elements
    // an access, kLoads accesses in flight
    float *stage = reinterpret_cast<float *>(smem + kShortStage);
    const int pitch = TALL ? W + 1 : W + 4;  // few bank conflicts of the transposing stores; of vector ones none
    const int64_t base = static_cast<int64_t>(mat) * a.rows * a.cols;
    const int mr = TALL ? w : p, mc = TALL ? p : w;  // memory rows and columns of this CTA's part
    const int64_t off = base + (TALL ? static_cast<int64_t>(q0) * a.cols : q0);
    {
        constexpr int kLoads = 4;
        const G *g = static_cast<const G *>(a.grad) + off;
        float *m = a.momentum ? a.momentum + off : nullptr;
        const int per_row = mc / V > 0 ? mc / V : 1, items = mc > 0 ? mr * per_row : 0;
        // a thread's items are kShortThreads apart: their rows and columns by addition
        const int dr = kShortThreads / per_row, dc = kShortThreads - dr * per_row;
        int row = threadIdx.x / per_row, col = threadIdx.x - row * per_row;
        Squares squares;
        for (int i0 = threadIdx.x; i0 < items; i0 += kLoads * kShortThreads) {
            float u[kLoads][V], mv[kLoads][V];
            int at[kLoads], place[kLoads];  // offsets in memory (below 2^31: at most 128 rows or columns) and in the stage
#pragma unroll
            for (int l = 0; l < kLoads; ++l) {
                at[l] = row * a.cols + col * V;
                place[l] = TALL ? col * V * pitch + row : row * pitch + col * V;
                if (i0 + l * kShortThreads < items) {
                    load_gv<V>(g, at[l], u[l]);
                    if (m)
                        load_gv<V>(m, at[l], mv[l]);
                }
                row += dr;
                col += dc;
                if (col >= per_row) {
                    col -= per_row;
                    ++row;
                }
            }
#pragma unroll
            for (int l = 0; l < kLoads; ++l) {
                if (i0 + l * kShortThreads >= items)
                    break;
                if (m) {
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        mv[l][k] = fmaf(a.beta, mv[l][k], u[l][k]);
                        u[l][k] = a.nesterov ? fmaf(a.beta, mv[l][k], u[l][k]) : mv[l][k];
                    }
                    if (V == 4)
                        *reinterpret_cast<float4 *>(m + at[l]) =
                            make_float4(mv[l][0], mv[l][1 % V], mv[l][2 % V], mv[l][3 % V]);
                    else
                        m[at[l]] = mv[l][0];
                }
                squares.add(u[l]);
                if (TALL) {
#pragma unroll
                    for (int k = 0; k < V; ++k)
                        stage[place[l] + k * pitch] = u[l][k];
                } else if (V == 4) {
                    *reinterpret_cast<float4 *>(stage + place[l]) =
                        make_float4(u[l][0], u[l][1 % V], u[l][2 % V], u[l][3 % V]);
                } else {
                    stage[place[l]] = u[l][0];
                }
            }
        }
        double sum = squares.total();
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == 0)
            warp_sum[warp] = sum;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int i = 0; i < kShortThreads / 32; ++i)
            s += warp_sum[i];
        *part = s;
    }
    cluster_sync_all();
    const uint32_t tmem = *holder;
    if (threadIdx.x == 0) {
        double total = 0.0;
        for (int c = 0; c < C; ++c)
            total += dsmem_ld_f64(dsmem_addr(smem_u32(part), c));
        // X lives in tensor memory columns [0, W) as X kSb kSx, the scale of the update's accumulator
        const Scale s(static_cast<double>(kSb) * kSx / (sqrt(total) + a.eps));
        factors[0] = s.first;
        factors[1] = s.second;
    }
    __syncthreads();
    const Scale scale(factors[0], factors[1]);
    const int r = (warp & 3) * 32 + lane;      // this thread's row of X, A and B
    const int cg = warp >> 2;                  // its quarter of a row's columns
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int wq = W / 4;                      // a multiple of 16
    // (loops over a row's columns are not unrolled: each runs once or twice, and instructions that
    // are fetched to run once cost more than the loop)
#pragma unroll 1
    for (int i = 0; i < wq; i += 16) {
        const int col = cg * wq + i;
        const float *from = stage + r * pitch + col;
        uint32_t bits[16], h[8];
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (r < p) {
                if (TALL)  // a row of the stage is W + 1 floats: no alignment
                    v = make_float4(from[k], from[k + 1], from[k + 2], from[k + 3]);
                else
                    v = *reinterpret_cast<const float4 *>(from + k);
            }
            // what lies behind column w was never staged
            const float x[4] = {col + k < w ? scale(v.x) : 0.0f, col + k + 1 < w ? scale(v.y) : 0.0f,
                                col + k + 2 < w ? scale(v.z) : 0.0f, col + k + 3 < w ? scale(v.w) : 0.0f};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                bits[k + e] = __float_as_uint(x[e]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const __half2 t = __floats2half2_rn(x[2 * e] * (1.0f / kSb), x[2 * e + 1] * (1.0f / kSb));
                h[k / 2 + e] = *reinterpret_cast<const uint32_t *>(&t);
            }
        }
        tmem_store16(tmem + lanes + col, bits);
        *reinterpret_cast<uint4 *>(smem + kShortXh + chunk_at8(r, col)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(smem + kShortXh + chunk_at8(r, col + 8)) = make_uint4(h[4], h[5], h[6], h[7]);
    }
    __syncthreads();  // the stage gives way to the buffers
    tmem_store_wait();

    const int np = (p + 15) & ~15;  // A and B: rows and columns in use
    const uint32_t t_acc = tmem + kShortMaxW, t_a = t_acc, t_a2 = t_acc + 128;
    uint32_t phase = 0, issued = 1;  // parity of the latest product that thread 0 issued
    // Every thread's writes made visible to the tensor core, one thread's MMAs, every thread behind them.
    // After an expired wait the rest runs through without waiting (the results are void).
    const auto product = [&](auto issue) {
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (threadIdx.x == 0 && !*abort_flag) {
            tc_fence_after();
            issue();
            umma_commit(mma);
            issued = phase;
        }
        warp_wait(mma, phase, wc, abort_flag);
        phase ^= 1;
        tc_fence_after();
    };
    const uint32_t xh = smem_u32(smem + kShortXh), ah = smem_u32(smem + kShortAh), bh = smem_u32(smem + kShortRed);

    for (int step = 0; step < a.steps; ++step) {
        product([&]() {
            for (int ks = 0; ks < W / 16; ++ks) {
                const uint64_t d = sdesc_kmajor_sw128(xh + (ks >> 2) * kChunk) + 2 * (ks & 3);
                umma_bf16(t_a, d, d, idesc_f16_f32(128, np), ks != 0);
            }
        });
        if (C > 1) {
            // this CTA's part of A, then its share of the sum, to every CTA
            float *red = reinterpret_cast<float *>(smem + kShortRed);
            if (cg * 32 < np) {
                float v[32];
                tmem_load32(t_a + lanes + cg * 32, v);
                // 16-byte columns rotated by the row, which keeps a column's stores off one bank
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<float4 *>(red + r * 128 + ((cg * 8 + k + r) & 31) * 4) =
                        make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
            cluster_sync_all();
            const int per_row = np / 4;
            for (int e = rank * kShortThreads + threadIdx.x; e < p * per_row; e += C * kShortThreads) {
                const int i = e / per_row, j = (e - i * per_row) * 4;
                const uint32_t at = smem_u32(red + i * 128 + ((j / 4 + i) & 31) * 4);
                float4 v[kShortMaxC];
#pragma unroll
                for (int c = 0; c < kShortMaxC; ++c)
                    if (c < C)
                        v[c] = dsmem_ld_f4(dsmem_addr(at, c));
                float4 s4 = v[0];
#pragma unroll
                for (int c = 1; c < kShortMaxC; ++c)
                    if (c < C) {
                        s4.x += v[c].x;
                        s4.y += v[c].y;
                        s4.z += v[c].z;
                        s4.w += v[c].w;
                    }
                const float f = kSa / (kSx * kSx);
                uint32_t h0, l0, h1, l1;
                const float2 r0 = split_pair(s4.x * f, s4.y * f, h0, l0), r1 = split_pair(s4.z * f, s4.w * f, h1, l1);
                const uint32_t o = chunk_at8(i, j) + (j & 7) * 2;
                const uint32_t la = smem_u32(smem + kShortAh + o), ll = smem_u32(smem + kShortAl + o);
                const bool diag = i >= j && i < j + 4;
                const float rest = i - j == 0 ? r0.x : (i - j == 1 ? r0.y : (i - j == 2 ? r1.x : r1.y));
#pragma unroll 1
                for (int c = 0; c < C; ++c) {
                    dsmem_st_u2(dsmem_addr(la, c), h0, h1);
                    dsmem_st_u2(dsmem_addr(ll, c), l0, l1);
                    if (diag)
                        dsmem_st_f32(dsmem_addr(smem_u32(ra + i), c), rest);
                }
            }
            if (step == 0)  // rows from p on of the operand stay zero
                for (int e = threadIdx.x; e < (128 - p) * 16; e += kShortThreads) {
                    const int i = p + e / 16;
                    *reinterpret_cast<uint4 *>(smem + kShortAh + chunk_at8(i, e % 16 * 8)) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4 *>(smem + kShortAl + chunk_at8(i, e % 16 * 8)) = make_uint4(0, 0, 0, 0);
                }
            fence_proxy_async_all();
            cluster_sync_all();
        } else {
            if (cg * 32 < np) {
                float v[32];
                tmem_load32(t_a + lanes + cg * 32, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float f = kSa / (kSx * kSx);
                        const int col = cg * 32 + 8 * k + 2 * i;
                        const float2 rest = split_pair(v[8 * k + 2 * i] * f, v[8 * k + 2 * i + 1] * f, h[i], l[i]);
                        if (col == r && r < p)
                            ra[r] = rest.x;
                        if (col + 1 == r && r < p)
                            ra[r] = rest.y;
                    }
                    const uint32_t o = chunk_at8(r, cg * 32 + 8 * k);
                    *reinterpret_cast<uint4 *>(smem + kShortAh + o) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4 *>(smem + kShortAl + o) = make_uint4(l[0], l[1], l[2], l[3]);
                }
            }
        }
        product([&]() {
            for (int ks = 0; ks < np / 16; ++ks) {
                const uint64_t d = sdesc_kmajor_sw128(ah + (ks >> 2) * kChunk) + 2 * (ks & 3);
                umma_bf16(t_a2, d, d, idesc_f16_f32(128, np), ks != 0);
            }
        });
        const float ra_row = ra[r];
        if (cg * 32 < np) {
            float v[32];
            tmem_load32(t_a2 + lanes + cg * 32, v);
            const float f = a.c * (kSb / kSa) * (1.0f / kSa);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t o = chunk_at8(r, cg * 32 + 8 * k);
                const uint4 h4 = *reinterpret_cast<const uint4 *>(smem + kShortAh + o);
                const uint4 l4 = *reinterpret_cast<const uint4 *>(smem + kShortAl + o);
                uint32_t h[4] = {h4.x, h4.y, h4.z, h4.w}, l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = cg * 32 + 8 * k + 2 * i;
                    const float2 old = join_f16(h[i], l[i]);
                    const float2 rc = *reinterpret_cast<const float2 *>(ra + col);
                    const float2 rest =
                        split_pair(fmaf(a.b, old.x, f * fmaf(ra_row + rc.x, old.x, v[8 * k + 2 * i])),
                                   fmaf(a.b, old.y, f * fmaf(ra_row + rc.y, old.y, v[8 * k + 2 * i + 1])), h[i], l[i]);
                    if (col == r && r < p)
                        rb[r] = rest.x;
                    if (col + 1 == r && r < p)
                        rb[r] = rest.y;
                }
                *reinterpret_cast<uint4 *>(smem + kShortRed + o) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
        product([&]() {
            for (int ks = 0; ks < np / 16; ++ks)
                umma_bf16(t_acc, sdesc_kmajor_sw128(bh + (ks >> 2) * kChunk) + 2 * (ks & 3),
                          sdesc_mn_chunk(xh + ks * 2048), idesc_f16_f32(128, W) | 1u << 16, ks != 0);
        });
        const float f = fmaf(rb[r], 1.0f / kSb, a.a);
        const bool last = step + 1 == a.steps;
        __nv_bfloat16 *result = reinterpret_cast<__nv_bfloat16 *>(smem + kShortAh);
#pragma unroll 1
        for (int i = 0; i < wq; i += 16) {
            const int col = cg * wq + i;
            float old[16], acc[16];
            tmem_load16(tmem + lanes + col, old);
            tmem_load16(t_acc + lanes + col, acc);
            uint32_t bits[16], h[8];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                old[k] = fmaf(f, old[k], acc[k]);
                bits[k] = __float_as_uint(old[k]);
            }
            if (last) {  // staged where A was: tall as memory has it, [w][p], wide in rows of W + 8
                if (TALL) {
                    if (r < p)
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (col + k < w)
                                result[(col + k) * p + r] = __float2bfloat16_rn(old[k] * a.out_scale);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const __nv_bfloat162 v =
                            __floats2bfloat162_rn(old[2 * k] * a.out_scale, old[2 * k + 1] * a.out_scale);
                        h[k] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    uint4 *to = reinterpret_cast<uint4 *>(result + r * (W + 8) + col);
                    to[0] = make_uint4(h[0], h[1], h[2], h[3]);
                    to[1] = make_uint4(h[4], h[5], h[6], h[7]);
                }
                continue;
            }
            tmem_store16(tmem + lanes + col, bits);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const __half2 v = __floats2half2_rn(old[2 * k] * (1.0f / kSb), old[2 * k + 1] * (1.0f / kSb));
                h[k] = *reinterpret_cast<const uint32_t *>(&v);
            }
            *reinterpret_cast<uint4 *>(smem + kShortXh + chunk_at8(r, col)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4 *>(smem + kShortXh + chunk_at8(r, col + 8)) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        if (!last)
            tmem_store_wait();
    }
    __syncthreads();
    {
        const __nv_bfloat16 *result = reinterpret_cast<const __nv_bfloat16 *>(smem + kShortAh);
        __nv_bfloat16 *o = a.out + off;
        const int count = mr * mc;
        const bool wide = reinterpret_cast<uintptr_t>(o) % 16 == 0 && (TALL || (a.cols % 8 == 0 && mc % 8 == 0));
        if (wide) {
            const int per_row = TALL ? 1 : mc / 8;
            const int items = TALL ? count / 8 : mr * per_row;
            for (int i = threadIdx.x; i < items; i += kShortThreads) {
                const int row = TALL ? 0 : i / per_row;
                const int col = TALL ? i * 8 : (i - row * per_row) * 8;
                *reinterpret_cast<uint4 *>(o + static_cast<int64_t>(row) * a.cols + col) =
                    *reinterpret_cast<const uint4 *>(result + row * (W + 8) + col);
            }
            if (TALL)
                for (int i = count / 8 * 8 + threadIdx.x; i < count; i += kShortThreads)
                    o[i] = result[i];
        } else {
            for (int i = threadIdx.x; i < count; i += kShortThreads) {
                const int row = i / mc, col = i - row * mc;
                o[static_cast<int64_t>(row) * a.cols + col] = result[TALL ? i : row * (W + 8) + col];
            }
        }
    }
    if (threadIdx.x == 0 && *abort_flag)
        mbar_wait_drain(mma, issued, wc);  // a product that was given up on may still be running
    tc_fence_before();
    cluster_sync_all();  // no CTA leaves while a peer may still reach its shared memory
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// -------------------------------------------------------------------------------- host, short
// Columns per CTA and CTAs per matrix; false if the matrix takes the products' path.
bool short_split(int p, int q, int &W, int &C)
{
    if (p > kShortMaxP || q > kShortMaxC * kShortMaxW)
        return false;
    C = (q + kShortMaxW - 1) / kShortMaxW;
    W = ((q + C - 1) / C + 63) / 64 * 64;
    return true;
}

template <typename G, bool TALL>
cudaError_t launch_short(const ShortArgs &a, int n, int C, const WaitCfg &wc, cudaStream_t stream)
{
    // four elements an access where every memory row keeps that alignment
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.grad) * (16 / (4 * sizeof(G))) |
                           reinterpret_cast<uintptr_t>(a.momentum);
    auto kernel = a.cols % 4 == 0 && bits % 16 == 0 ? orth_short_kernel<G, TALL, 4> : orth_short_kernel<G, TALL, 1>;
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kShortSmem));
    if (err != cudaSuccess)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n) * C);
    cfg.blockDim = dim3(kShortThreads);
    cfg.dynamicSmemBytes = kShortSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, wc);
}

// ------------------------------------------------------------------------------------ host
constexpr int kMaxSide = 16384;
constexpr int kMaxSteps = 32;
constexpr size_t kChunkBytes = size_t(2) << 30;  // matrices worked on together fill at most this

// Whether a step is faster on CTA pairs: the waves of tiles of the three products, weighted by their
// K, a 256 x 256 pair tile taking 1.4 times a 128 x 128 one. Measured, single / pairs (us): 16 x
// 384 x 1536 228 / 284, 64 x 300 x 900 620 / 766, 64 x 256 x 1024 320 / 322, 16 x 768 x 2048 696 / 600, 12 x 1280 x
// 4096 2139 / 1619.
bool use_pairs(int64_t n, int64_t p, int64_t q, int num_sms)
{
    const auto cost = [&](int64_t tile, int64_t slots) {
        const int64_t nm = (p + tile - 1) / tile, nq = (q + tile - 1) / tile;
        const auto waves = [&](int64_t tiles) { return (tiles * n + slots - 1) / slots; };
        return waves(nm * (nm + 1) / 2) * (q + p) + waves(nm * nq) * p;
    };
    return cost(128, num_sms) * 10 > cost(256, num_sms / 2) * 14;
}

size_t up(size_t v, size_t to)
{
    return (v + to - 1) / to * to;
}

struct OrthLayout {
    int chunk;  // matrices worked on together
    int p, parts;
    size_t x_pitch, x_mat, a_pitch, a_mat, r_mat;
    size_t xh0, xh1, xl, ah, al, bh, ra, rb, part, total;
};

OrthLayout orth_layout(const moe_orthogonalize_desc &d)
{
    OrthLayout L{};
    const size_t rows = d.rows, cols = d.cols;
    L.p = d.rows < d.cols ? d.rows : d.cols;
    int W, C;
    if (short_split(L.p, d.rows < d.cols ? d.cols : d.rows, W, C)) {
        L.total = 256;  // one launch, all of it on chip: the least that a caller can hand over
        return L;
    }
    L.x_pitch = up(cols, 64);
    L.x_mat = rows * L.x_pitch;
    L.a_pitch = up(L.p, 64);
    L.a_mat = L.p * L.a_pitch;
    L.r_mat = up(L.p, 64);
    const size_t elems = rows * cols;
    const size_t parts = (elems + 8191) / 8192;  // 32 elements a thread, or more
    L.parts = static_cast<int>(parts > 512 ? 512 : parts);
    const size_t each = 6 * L.x_mat + 6 * L.a_mat + 8 * L.r_mat + 8 * L.parts;
    size_t most = kChunkBytes / each;
    most = most < 1 ? 1 : most;
    const size_t n = d.n > 0 ? d.n : 1;
    const size_t chunks = (n + most - 1) / most;
    const size_t nc = (n + chunks - 1) / chunks;
    L.chunk = static_cast<int>(nc);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off += up(bytes, 256);
        return o;
    };
    L.xh0 = take(nc * L.x_mat * 2);
    L.xh1 = take(nc * L.x_mat * 2);
    L.xl = take(nc * L.x_mat * 2);
    L.ah = take(nc * L.a_mat * 2);
    L.al = take(nc * L.a_mat * 2);
    L.bh = take(nc * L.a_mat * 2);
    L.ra = take(nc * L.r_mat * 4);
    L.rb = take(nc * L.r_mat * 4);
    L.part = take(nc * L.parts * 8);
    L.total = off;
    return L;
}

// Whether every iterate of singular values in [0, 1] stays inside the scaled fp16 operands: X
// below 65504 / kSx, A below 65504 / kSa, B below 65504 / kSb (with 1% to spare for rounding).
bool iterates_fit(const moe_orthogonalize_desc &d)
{
    const double a = d.a, b = d.b, c = d.c;
    double top = 1.01;
    for (int s = 0; s < d.steps; ++s) {
        if (!(top <= 7.9) || !(top * top <= 31.0))
            return false;
        const double l = top * top;  // eigenvalues of A lie in [0, l]
        // |b t + c t^2| is largest at l or at its vertex
        const auto bt = [&](double t) { return std::fabs(t * (b + c * t)); };
        double bmax = bt(l);
        if (c != 0.0 && -b / (2.0 * c) > 0.0 && -b / (2.0 * c) < l)
            bmax = std::fmax(bmax, bt(-b / (2.0 * c)));
        if (!(bmax <= 31.0))
            return false;
        // |x (a + b x^2 + c x^4)| at top or where 5 c t^2 + 3 b t + a = 0, t = x^2
        const auto px = [&](double t) { return std::fabs(std::sqrt(t) * (a + t * (b + c * t))); };
        double next = px(l);
        double roots[2] = {-1.0, -1.0};
        if (c != 0.0) {
            const double disc = 9.0 * b * b - 20.0 * a * c;
            if (disc >= 0.0) {
                roots[0] = (-3.0 * b + std::sqrt(disc)) / (10.0 * c);
                roots[1] = (-3.0 * b - std::sqrt(disc)) / (10.0 * c);
            }
        } else if (b != 0.0) {
            roots[0] = -a / (3.0 * b);
        }
        for (double t : roots)
            if (t > 0.0 && t < l)
                next = std::fmax(next, px(t));
        top = 1.01 * next;
    }
    return std::isfinite(top);
}

moe_status_t check_orth(const moe_orthogonalize_desc *d)
{
    if (!d || d->n < 0 || d->rows <= 0 || d->cols <= 0 || d->steps < 1 || d->steps > kMaxSteps)
        return MOE_ERR_INVALID_ARG;
    if (d->dtype != MOE_DTYPE_F32 && d->dtype != MOE_DTYPE_BF16 && d->dtype != MOE_DTYPE_F16)
        return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(d->a) || !std::isfinite(d->b) || !std::isfinite(d->c) || !std::isfinite(d->eps) ||
        d->eps < 0.0f || !std::isfinite(d->scale) || !std::isfinite(d->beta) || (d->nesterov != 0 && d->nesterov != 1))
        return MOE_ERR_INVALID_ARG;
    if (d->dtype == MOE_DTYPE_F16 || d->rows > kMaxSide || d->cols > kMaxSide || d->n > 65535 || !iterates_fit(*d))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

template <typename G>
cudaError_t launch_prep(const PrepArgs &a, int n, cudaStream_t stream)
{
    const int64_t elems = static_cast<int64_t>(a.rows) * a.cols;
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.grad) | reinterpret_cast<uintptr_t>(a.momentum);
    const dim3 grid(a.parts, n);
    if (elems % 8 == 0 && at % 16 == 0)
        orth_norm_kernel<G, 8><<<grid, 256, 0, stream>>>(a);
    else
        orth_norm_kernel<G, 1><<<grid, 256, 0, stream>>>(a);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess)
        return err;
    const int64_t work = ((a.cols + 7) / 8 * static_cast<int64_t>(a.rows) + 255) / 256;
    const dim3 cgrid(static_cast<unsigned>(work < 512 ? work : 512), n);
    return launch_dependent(a.cols % 8 == 0 && at % 16 == 0 ? orth_cast_kernel<G, true> : orth_cast_kernel<G, false>,
                            cgrid, 256, 0, stream, 1, a);
}

template <bool TALL, bool PAIR>
moe_status_t run_steps(const moe_orthogonalize_desc &d, const OrthLayout &L, const DeviceContext &dc, int n, uint8_t *w,
                       __nv_bfloat16 *out, cudaStream_t s)
{
    OrthArgs a{};
    a.n = n;
    a.p = L.p;
    a.rows = d.rows;
    a.cols = d.cols;
    a.r_mat = L.r_mat;
    a.ra = reinterpret_cast<float *>(w + L.ra);
    a.rb = reinterpret_cast<float *>(w + L.rb);
    a.a = d.a;
    a.b = d.b;
    a.c = d.c;
    a.out_scale = d.scale / kSx;
    a.out_wide = d.cols % 8 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0;
    // each matrix with K-major boxes, with MN-major ones and with the epilogue's
    const auto sym = [&](CUtensorMap *m, size_t off, uint32_t cols, uint32_t rows) {
        return map_stack_f16(m, w + off, L.p, L.p, n, L.a_pitch, L.a_mat, cols, rows);
    };
    const auto xs = [&](CUtensorMap *m, size_t off, uint32_t cols, uint32_t rows) {
        return map_stack_f16(m, w + off, d.cols, d.rows, n, L.x_pitch, L.x_mat, cols, rows);
    };
    const size_t xh[2] = {L.xh0, L.xh1};
    CUtensorMap xk[2], xm[2], xe[2], xl, ak, am, ae, al, bk, bm, be, oe;
    bool ok = sym(&ak, L.ah, 64, 128) && sym(&am, L.ah, 64, 64) && sym(&ae, L.ah, 32, 128) &&
              sym(&al, L.al, 32, 128) && sym(&bk, L.bh, 64, 128) && sym(&bm, L.bh, 64, 64) &&
              sym(&be, L.bh, 32, 128) && xs(&xl, L.xl, 32, 128);
    for (int i = 0; i < 2; ++i)
        ok = ok && xs(&xk[i], xh[i], 64, 128) && xs(&xm[i], xh[i], 64, 64) && xs(&xe[i], xh[i], 32, 128);
    oe = xl;  // unused unless out_wide (to a copy bf16 and fp16 are the same 16 bits)
    if (a.out_wide)
        ok = ok && map_stack_f16(&oe, out, d.cols, d.rows, n, d.cols, static_cast<int64_t>(d.rows) * d.cols, 32, 128);
    if (!ok)
        return MOE_ERR_CUDA;
    const auto half = [&](size_t off) { return reinterpret_cast<__half *>(w + off); };
    const int64_t nm = (L.p + 127) / 128, a_tiles = nm * (nm + 1) / 2 * n;
    const int64_t x_tiles = static_cast<int64_t>((d.rows + 127) / 128) * ((d.cols + 127) / 128) * n;
    SplitRoom room{};
    if (!PAIR && split_room(room) != cudaSuccess)
        return MOE_ERR_CUDA;
    const int gram = PAIR ? 0 : split_of(a_tiles, TALL ? d.rows : d.cols, room);
    const int square = PAIR ? 0 : split_of(a_tiles, L.p, room);
    const int update = PAIR ? 0 : split_of(x_tiles, L.p, room);
    const int64_t a_pitch = L.a_pitch, a_mat = L.a_mat, x_pitch = L.x_pitch, x_mat = L.x_mat;
    cudaError_t e = cudaSuccess;
    for (int step = 0; step < d.steps && e == cudaSuccess; ++step) {
        const int cur = step & 1;
        a.out = step + 1 == d.steps ? out : nullptr;
        if (gram) {
            const SplitArgs sp{nullptr, nullptr, half(L.ah), half(L.al), a_pitch, a_mat};
            e = launch_split<kGram, TALL>(gram, a_tiles, xk[cur], xm[cur], xk[cur], xm[cur], a, sp, dc, s);
        } else {
            const EpiMaps em{ae, al, ae, al};
            e = launch_gemm<kGram, TALL, PAIR>(xk[cur], xm[cur], xk[cur], xm[cur], em, a, dc, s);
        }
        if (e != cudaSuccess)
            break;
        if (square) {
            const SplitArgs sp{half(L.ah), half(L.al), half(L.bh), nullptr, a_pitch, a_mat};
            e = launch_split<kSquare, TALL>(square, a_tiles, ak, am, ak, am, a, sp, dc, s);
        } else {
            const EpiMaps em{ae, al, be, be};
            e = launch_gemm<kSquare, TALL, PAIR>(ak, am, ak, am, em, a, dc, s);
        }
        if (e != cudaSuccess)
            break;
        const CUtensorMap &lk = TALL ? xk[cur] : bk, &lm = TALL ? xm[cur] : bm;
        const CUtensorMap &rk = TALL ? bk : xk[cur], &rm = TALL ? bm : xm[cur];
        if (update) {
            const SplitArgs sp{half(xh[cur]), half(L.xl), half(xh[cur ^ 1]), half(L.xl), x_pitch, x_mat};
            e = launch_split<kUpdate, TALL>(update, x_tiles, lk, lm, rk, rm, a, sp, dc, s);
        } else {
            const EpiMaps em{xe[cur], xl, a.out ? oe : xe[cur ^ 1], xl};
            e = launch_gemm<kUpdate, TALL, PAIR>(lk, lm, rk, rm, em, a, dc, s);
        }
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_orthogonalize_workspace_size(const moe_orthogonalize_desc *desc, size_t *bytes)
{
    const moe_status_t st = check_orth(desc);
    if (st != MOE_OK)
        return st;
    if (!bytes)
        return MOE_ERR_INVALID_ARG;
    *bytes = orth_layout(*desc).total;
    return MOE_OK;
}

moe_status_t moe_orthogonalize(const moe_orthogonalize_desc *desc, const void *grad, float *momentum, uint16_t *out,
                               void *ws, size_t ws_bytes, void *stream)
{
    moe_status_t st = check_orth(desc);
    if (st != MOE_OK)
        return st;
    if (desc->n == 0)
        return MOE_OK;
    if (!grad || !out || !ws)
        return MOE_ERR_INVALID_ARG;
    const moe_orthogonalize_desc &d = *desc;
    const int elem = d.dtype == MOE_DTYPE_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(grad) % elem || reinterpret_cast<uintptr_t>(momentum) % 4 ||
        reinterpret_cast<uintptr_t>(out) % 2 || reinterpret_cast<uintptr_t>(ws) % 256)
        return MOE_ERR_UNSUPPORTED;
    const OrthLayout L = orth_layout(d);
    if (ws_bytes < L.total)
        return MOE_ERR_WORKSPACE;
    DeviceContext dc;
    if ((st = static_cast<moe_status_t>(device_context(dc))) != MOE_OK)
        return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *w = static_cast<uint8_t *>(ws);
    const int64_t elems = static_cast<int64_t>(d.rows) * d.cols;
    int W, C;
    if (short_split(L.p, d.rows < d.cols ? d.cols : d.rows, W, C)) {
        const ShortArgs sa{grad, momentum, reinterpret_cast<__nv_bfloat16 *>(out), d.rows, d.cols, L.p, W, d.steps,
                           d.nesterov, d.a, d.b, d.c, d.scale / (kSx * kSb), d.beta, d.eps};
        const bool f32 = d.dtype == MOE_DTYPE_F32;
        const cudaError_t e =
            d.rows > d.cols ? (f32 ? launch_short<float, true>(sa, d.n, C, dc.wait, s)
                                   : launch_short<__nv_bfloat16, true>(sa, d.n, C, dc.wait, s))
                            : (f32 ? launch_short<float, false>(sa, d.n, C, dc.wait, s)
                                   : launch_short<__nv_bfloat16, false>(sa, d.n, C, dc.wait, s));
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    for (int first = 0; first < d.n; first += L.chunk) {
        const int n = d.n - first < L.chunk ? d.n - first : L.chunk;
        PrepArgs pa{};
        pa.grad = static_cast<const uint8_t *>(grad) + first * elems * elem;
        pa.momentum = momentum ? momentum + first * elems : nullptr;
        pa.part = reinterpret_cast<double *>(w + L.part);
        pa.xh = reinterpret_cast<__half *>(w + L.xh0);
        pa.xl = reinterpret_cast<__half *>(w + L.xl);
        pa.rows = d.rows;
        pa.cols = d.cols;
        pa.parts = L.parts;
        pa.x_pitch = L.x_pitch;
        pa.x_mat = L.x_mat;
        pa.beta = d.beta;
        pa.nesterov = d.nesterov;
        pa.eps = d.eps;
        const cudaError_t e = d.dtype == MOE_DTYPE_F32 ? launch_prep<float>(pa, n, s)
                                                       : launch_prep<__nv_bfloat16>(pa, n, s);
        if (e != cudaSuccess)
            return MOE_ERR_CUDA;
        __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(out) + first * elems;
        const bool pair = use_pairs(n, L.p, d.rows < d.cols ? d.cols : d.rows, dc.num_sms);
        st = d.rows > d.cols ? (pair ? run_steps<true, true>(d, L, dc, n, w, o, s)
                                     : run_steps<true, false>(d, L, dc, n, w, o, s))
                             : (pair ? run_steps<false, true>(d, L, dc, n, w, o, s)
                                     : run_steps<false, false>(d, L, dc, n, w, o, s));
        if (st != MOE_OK)
            return st;
    }
    return MOE_OK;
}

}  // extern "C"
