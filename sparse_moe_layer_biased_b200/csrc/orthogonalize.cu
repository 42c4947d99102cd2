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
// 2 p p q + p p p multiply-adds a step for the two symmetric products' triangles and the update:
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
    int64_t x_pitch, x_mat;  // X buffers: row and matrix pitch in elements
    int64_t a_pitch, a_mat;  // A and B
    int64_t r_mat;           // diagonal remainders: floats per matrix
    const __half *xh;        // X, hi (the GEMM operand)
    __half *xh_out;          // next X, hi
    __half *xl;              // X, lo: updated in place
    __half *ah, *al, *bh;
    float *ra, *rb;
    __nv_bfloat16 *out;      // [n, rows, cols], the last update's destination (else NULL)
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
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            v[k] = __bfloat162float(p[i + k]);
    }
}

// Updates the momentum and sums u^2 over part blockIdx.x of matrix blockIdx.y. V elements at a
// time: 8 when every matrix starts on a 32-byte boundary, else 1.
template <typename G, int V>
__global__ void __launch_bounds__(256)
    orth_norm_kernel(const PrepArgs a)
{
    __shared__ double warp_sum[8];
    const int64_t elems = static_cast<int64_t>(a.rows) * a.cols;
    const int64_t base = blockIdx.y * elems;
    const G *g = static_cast<const G *>(a.grad) + base;
    float *m = a.momentum ? a.momentum + base : nullptr;
    const int64_t step = static_cast<int64_t>(a.parts) * 256 * V;
    double sum = 0.0;
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
#pragma unroll
        for (int k = 0; k < V; ++k)
            sum += static_cast<double>(u[k]) * u[k];
    }
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
    __shared__ double inv_s;
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int i = 0; i < a.parts; ++i)
            s += a.part[static_cast<int64_t>(blockIdx.y) * a.parts + i];
        inv_s = static_cast<double>(kSx) / (sqrt(s) + a.eps);
    }
    __syncthreads();
    const double inv = inv_s;
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
            split_f16(static_cast<float>(u[k] * inv), hi[k], lo[k]);
        const int64_t at = blockIdx.y * a.x_mat + row * a.x_pitch + col;
        *reinterpret_cast<uint4 *>(a.xh + at) = *reinterpret_cast<const uint4 *>(hi);
        *reinterpret_cast<uint4 *>(a.xl + at) = *reinterpret_cast<const uint4 *>(lo);
    }
}

// -------------------------------------------------------------------------------- products
// One persistent kernel per product, one CTA per SM: warp 0 TMA producer, warp 1 MMA issuer and
// TMEM owner, warps 2.. epilogue. A tile is 128 rows x 128 columns of one matrix; two
// accumulators in TMEM let a tile's epilogue overlap the next tile's K loop. An operand is K-major
// (X rows in A = X X^T) or MN-major (X columns in X^T X and B X), as the layout gives it: X is never
// transposed. Symmetric products compute the tiles on and above the diagonal and store each
// tile also mirrored.
constexpr int kBM = 128, kBN = 128;
constexpr int kStages = 6;
constexpr uint32_t kOperand = 16384;  // 128 x 64 fp16
constexpr uint32_t kStageBytes = 2 * kOperand;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kBarOff = kStages * kStageBytes;
constexpr uint32_t kMiscOff = kBarOff + 8 * (2 * kStages + 5);
constexpr uint32_t kSmem = kMiscOff + 16 + 1024;
static_assert(kSmem <= static_cast<uint32_t>(kMaxDynSmem), "ring exceeds shared memory");

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

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *m, uint64_t *bar, int32_t c0, int32_t c1,
                                            int32_t c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

struct OrthTile {
    int mat, m0, n0;
    bool mirror;  // a symmetric product's tile above the diagonal
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
    int ti, tj;
    if (KIND == kUpdate) {
        ti = u / nn;
        tj = u - ti * nn;
    } else {
        // row ti of the triangle starts at ti * nm - ti (ti - 1) / 2
        ti = 0;
        int first = 0;
        while (first + nm - ti <= u) {
            first += nm - ti;
            ++ti;
        }
        tj = ti + (u - first);
    }
    t.m0 = ti * kBM;
    t.n0 = tj * kBN;
    t.mirror = KIND != kUpdate && tj > ti;
    return t;
}

// Eight columns [col, col + 8) of a row as floats (hi + lo).
__device__ __forceinline__ void load_pair8(const __half *hi, const __half *lo, int64_t at, float (&v)[8])
{
    const uint4 h = *reinterpret_cast<const uint4 *>(hi + at), l = *reinterpret_cast<const uint4 *>(lo + at);
    const __half2 *hp = reinterpret_cast<const __half2 *>(&h), *lp = reinterpret_cast<const __half2 *>(&l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = __half22float2(hp[i]), b = __half22float2(lp[i]);
        v[2 * i] = fmaf(b.x, 1.0f / kLo, a.x);
        v[2 * i + 1] = fmaf(b.y, 1.0f / kLo, a.y);
    }
}

// Epilogue of 32 columns [col0, col0 + 32) of this thread's row of a tile.
template <int KIND, bool TALL>
__device__ __forceinline__ void orth_epilogue(const OrthArgs &a, const OrthTile &t, int row, int col0,
                                              const float (&acc)[32])
{
    const int M = KIND == kUpdate ? a.rows : a.p, N = KIND == kUpdate ? a.cols : a.p;
    if (row >= M)
        return;
    if (KIND == kUpdate) {
        const int64_t base = t.mat * a.x_mat + row * a.x_pitch;
        const float *rb = a.rb + t.mat * a.r_mat;
        const float row_r = TALL ? 0.0f : a.a + rb[row] * (1.0f / kSb);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int col = col0 + 8 * g;
            if (col >= N)
                break;
            float x[8];
            load_pair8(a.xh, a.xl, base + col, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = TALL ? a.a + (col + i < N ? rb[col + i] : 0.0f) * (1.0f / kSb) : row_r;
                x[i] = fmaf(f, x[i], acc[8 * g + i] * (1.0f / kSb));
            }
            if (a.out) {
                const int64_t o = (static_cast<int64_t>(t.mat) * a.rows + row) * a.cols + col;
                alignas(16) __nv_bfloat16 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = __float2bfloat16_rn(x[i] * a.out_scale);
                if (a.cols % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0) {
                    *reinterpret_cast<uint4 *>(a.out + o) = *reinterpret_cast<const uint4 *>(v);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (col + i < N)
                            a.out[o + i] = v[i];
                }
            } else {
                alignas(16) __half hi[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    split_f16(x[i], hi[i], lo[i]);
                *reinterpret_cast<uint4 *>(a.xh_out + base + col) = *reinterpret_cast<const uint4 *>(hi);
                *reinterpret_cast<uint4 *>(a.xl + base + col) = *reinterpret_cast<const uint4 *>(lo);
            }
        }
        return;
    }
    const int64_t mat = t.mat * a.a_mat;
    const int64_t base = mat + row * a.a_pitch;
    const float *ra = a.ra + t.mat * a.r_mat;
    const float ra_row = KIND == kSquare ? ra[row] : 0.0f;
    __half *dst = KIND == kGram ? a.ah : a.bh;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int col = col0 + 8 * g;
        if (col >= N)
            break;
        float v[8];
        if (KIND == kGram) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = acc[8 * g + i] * (kSa / (kSx * kSx));
        } else {
            float x[8];
            load_pair8(a.ah, a.al, base + col, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float r = ra_row + (col + i < N ? ra[col + i] : 0.0f);
                v[i] = fmaf(a.b, x[i], a.c * (kSb / kSa) * (fmaf(r, x[i], acc[8 * g + i]) * (1.0f / kSa)));
            }
        }
        alignas(16) __half hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            split_f16(v[i], hi[i], lo[i]);
            if (col + i == row)
                (KIND == kGram ? a.ra : a.rb)[t.mat * a.r_mat + row] = v[i] - __half2float(hi[i]);
        }
        *reinterpret_cast<uint4 *>(dst + base + col) = *reinterpret_cast<const uint4 *>(hi);
        if (KIND == kGram)
            *reinterpret_cast<uint4 *>(a.al + base + col) = *reinterpret_cast<const uint4 *>(lo);
        if (t.mirror)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (col + i < N)
                    dst[mat + (col + i) * a.a_pitch + row] = hi[i];
    }
}

// MN-major operands: X in A = X^T X (tall) and the right factor X of B X (wide).
template <int KIND, bool TALL>
__global__ void __launch_bounds__(kThreads, 1)
    orth_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const OrthArgs a, const WaitCfg wc)
{
    constexpr bool kAmn = KIND == kGram && TALL;
    constexpr bool kBmn = (KIND == kGram && TALL) || (KIND == kUpdate && !TALL);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kBarOff);
    uint64_t *empty = full + kStages;
    uint64_t *accf = empty + kStages;
    uint64_t *acce = accf + 2;
    uint64_t *drain = acce + 2;
    uint32_t *holder = reinterpret_cast<uint32_t *>(smem + kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kMiscOff + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(holder, 2 * kBN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *holder;
    const int M = KIND == kUpdate ? a.rows : a.p, N = KIND == kUpdate ? a.cols : a.p;
    const int K = KIND == kGram ? (TALL ? a.rows : a.cols) : a.p;
    const int nm = (M + kBM - 1) / kBM, nn = (N + kBN - 1) / kBN;
    const int nk = (K + 63) / 64;
    const int per = tiles_of<KIND>(nm, nn);
    const int tiles = per * a.n;

    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_map(&tm_a);
            tma_prefetch_map(&tm_b);
            int it = 0;
            bool stop = false;
            for (int tile = blockIdx.x; tile < tiles && !stop; tile += gridDim.x) {
                const OrthTile t = tile_at<KIND>(tile, per, nm, nn);
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(&empty[s], ((it / kStages) & 1) ^ 1, wc, abort_flag)) {
                        stop = true;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[s], kStageBytes);
                    uint8_t *A = smem + s * kStageBytes, *B = A + kOperand;
                    if (kAmn) {
                        tma_load_3d(A, &tm_a, &full[s], t.m0, kb * 64, t.mat);
                        tma_load_3d(A + 8192, &tm_a, &full[s], t.m0 + 64, kb * 64, t.mat);
                    } else {
                        tma_load_3d(A, &tm_a, &full[s], kb * 64, t.m0, t.mat);
                    }
                    if (kBmn) {
                        tma_load_3d(B, &tm_b, &full[s], t.n0, kb * 64, t.mat);
                        tma_load_3d(B + 8192, &tm_b, &full[s], t.n0 + 64, kb * 64, t.mat);
                    } else {
                        tma_load_3d(B, &tm_b, &full[s], kb * 64, t.n0, t.mat);
                    }
                }
            }
            for (int i = it > kStages ? it - kStages : 0; i < it; ++i)
                mbar_wait_drain(&full[i % kStages], (i / kStages) & 1, wc);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int it = 0, tc = 0;
            bool ok = true;
            for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, ++tc) {
                const OrthTile t = tile_at<KIND>(tile, per, nm, nn);
                const int buf = tc & 1;
                if (!mbar_wait(&acce[buf], ((tc >> 1) & 1) ^ 1, wc, abort_flag))
                    break;
                tc_fence_after();
                const int left = N - t.n0;
                const int cols = left < kBN ? (left + 15) & ~15 : kBN;
                const uint32_t idesc = idesc_f16_f32(kBM, cols) | (kAmn ? 1u << 15 : 0u) | (kBmn ? 1u << 16 : 0u);
                for (int kb = 0; kb < nk; ++kb, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(&full[s], (it / kStages) & 1, wc, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + s * kStageBytes), sb = sa + kOperand;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t ad = kAmn ? sdesc_mn(sa + ks * 2048) : sdesc_kmajor_sw128(sa) + 2 * ks;
                        const uint64_t bd = kBmn ? sdesc_mn(sb + ks * 2048) : sdesc_kmajor_sw128(sb) + 2 * ks;
                        umma_bf16(tmem + buf * kBN, ad, bd, idesc, (kb | ks) != 0);  // kind::f16: fp16 by idesc
                    }
                    umma_commit(&empty[s]);
                }
                if (ok)
                    umma_commit(&accf[buf]);
            }
            umma_commit(drain);
            mbar_wait_drain(drain, 0, wc);
        }
    } else {
        const int q = warp & 3;
        int tc = 0;
        for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, ++tc) {
            const OrthTile t = tile_at<KIND>(tile, per, nm, nn);
            const int buf = tc & 1;
            if (!warp_wait(&accf[buf], (tc >> 1) & 1, wc, abort_flag))
                break;
            tc_fence_after();
            const int row = t.m0 + q * 32 + lane;
            for (int cb = 0; cb < kBN && t.n0 + cb < N; cb += 32) {
                float v[32];
                tmem_load32(tmem + buf * kBN + (static_cast<uint32_t>(q * 32) << 16) + cb, v);
                orth_epilogue<KIND, TALL>(a, t, row, t.n0 + cb, v);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&acce[buf]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kBN);
    }
}

template <int KIND, bool TALL>
cudaError_t launch_gemm(const CUtensorMap &ma, const CUtensorMap &mb, const OrthArgs &a, const DeviceContext &dc,
                        cudaStream_t stream)
{
    const cudaError_t err = cudaFuncSetAttribute(orth_gemm_kernel<KIND, TALL>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (err != cudaSuccess)
        return err;
    const int M = KIND == kUpdate ? a.rows : a.p, N = KIND == kUpdate ? a.cols : a.p;
    const int nm = (M + kBM - 1) / kBM, nn = (N + kBN - 1) / kBN;
    const int64_t tiles = static_cast<int64_t>(KIND == kUpdate ? nm * nn : nm * (nm + 1) / 2) * a.n;
    const int grid = static_cast<int>(tiles < dc.num_sms ? tiles : dc.num_sms);
    orth_gemm_kernel<KIND, TALL><<<grid, kThreads, kSmem, stream>>>(ma, mb, a, dc.wait);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------------ host
constexpr int kMaxSide = 16384;
constexpr int kMaxSteps = 32;
constexpr size_t kChunkBytes = size_t(2) << 30;  // matrices worked on together fill at most this

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
    L.x_pitch = up(cols, 64);
    L.x_mat = rows * L.x_pitch;
    L.a_pitch = up(L.p, 64);
    L.a_mat = L.p * L.a_pitch;
    L.r_mat = up(L.p, 64);
    const size_t elems = rows * cols;
    const size_t parts = (elems + 16383) / 16384;  // 64 elements a thread
    L.parts = static_cast<int>(parts < 1 ? 1 : (parts > 64 ? 64 : parts));
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
        double next = 0.0, bmax = 0.0;
        constexpr int kPoints = 4096;
        for (int i = 0; i <= kPoints; ++i) {
            const double x = top * i / kPoints, l = x * x;
            const double bb = std::fabs(b * l + c * l * l), px = std::fabs(x * (a + b * l + c * l * l));
            next = px > next ? px : next;
            bmax = bb > bmax ? bb : bmax;
        }
        if (!(bmax <= 31.0))
            return false;
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
    if (a.cols % 8 == 0 && at % 16 == 0)
        orth_cast_kernel<G, true><<<cgrid, 256, 0, stream>>>(a);
    else
        orth_cast_kernel<G, false><<<cgrid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

template <bool TALL>
moe_status_t run_steps(const moe_orthogonalize_desc &d, const OrthLayout &L, const DeviceContext &dc, int n, uint8_t *w,
                       __nv_bfloat16 *out, cudaStream_t s)
{
    __half *xh[2] = {reinterpret_cast<__half *>(w + L.xh0), reinterpret_cast<__half *>(w + L.xh1)};
    OrthArgs a{};
    a.n = n;
    a.p = L.p;
    a.rows = d.rows;
    a.cols = d.cols;
    a.x_pitch = L.x_pitch;
    a.x_mat = L.x_mat;
    a.a_pitch = L.a_pitch;
    a.a_mat = L.a_mat;
    a.r_mat = L.r_mat;
    a.xl = reinterpret_cast<__half *>(w + L.xl);
    a.ah = reinterpret_cast<__half *>(w + L.ah);
    a.al = reinterpret_cast<__half *>(w + L.al);
    a.bh = reinterpret_cast<__half *>(w + L.bh);
    a.ra = reinterpret_cast<float *>(w + L.ra);
    a.rb = reinterpret_cast<float *>(w + L.rb);
    a.a = d.a;
    a.b = d.b;
    a.c = d.c;
    a.out_scale = d.scale / kSx;
    CUtensorMap mk[2], mm[2], am, bm;  // X with K-major boxes (tall update, wide gram) and MN-major ones
    bool ok = map_stack_f16(&am, a.ah, L.p, L.p, n, L.a_pitch, L.a_mat, 128) &&
              map_stack_f16(&bm, a.bh, L.p, L.p, n, L.a_pitch, L.a_mat, 128);
    for (int i = 0; i < 2 && ok; ++i)
        ok = map_stack_f16(&mk[i], xh[i], d.cols, d.rows, n, L.x_pitch, L.x_mat, 128) &&
             map_stack_f16(&mm[i], xh[i], d.cols, d.rows, n, L.x_pitch, L.x_mat, 64);
    if (!ok)
        return MOE_ERR_CUDA;
    cudaError_t e = cudaSuccess;
    for (int step = 0; step < d.steps && e == cudaSuccess; ++step) {
        const int cur = step & 1;
        a.xh = xh[cur];
        a.xh_out = xh[cur ^ 1];
        a.out = step + 1 == d.steps ? out : nullptr;
        const CUtensorMap &gx = TALL ? mm[cur] : mk[cur];
        e = launch_gemm<kGram, TALL>(gx, gx, a, dc, s);
        if (e == cudaSuccess)
            e = launch_gemm<kSquare, TALL>(am, am, a, dc, s);
        if (e == cudaSuccess)
            e = TALL ? launch_gemm<kUpdate, TALL>(mk[cur], bm, a, dc, s)
                     : launch_gemm<kUpdate, TALL>(bm, mm[cur], a, dc, s);
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
        st = d.rows > d.cols ? run_steps<true>(d, L, dc, n, w, o, s) : run_steps<false>(d, L, dc, n, w, o, s);
        if (st != MOE_OK)
            return st;
    }
    return MOE_OK;
}

}  // extern "C"
