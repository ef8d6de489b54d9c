/*
 * layernorm.cu -- layer norm over rows of activations, forward and backward.
 *
 * Per row of d elements: mean = sum x / d, rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
 * y = (x - mean) * rstd * weight + bias.  The variance is that of the differences (a second
 * pass over registers), so a row whose mean is large against its spread keeps its digits.
 * Backward, with xh = (x - mean) * rstd and g = dy * weight:
 *   dx = rstd * (g - sum(g)/d - xh * sum(g * xh)/d)
 *   dweight = sum over rows of dy * xh,  dbias = sum over rows of dy
 */
#include "rows.cuh"

namespace zero {
namespace {

constexpr uint32_t kMaxDim = 16384;
constexpr uint32_t kMaxParts = 912;  // blocks of the backward pass: 6 on each of 152 SMs
constexpr uint32_t kRing = 4;        // stages of a ring, at most
constexpr uint32_t kRingWarps = 8;   // forward: warps per block, each with a ring of its own

struct ForwardArgs {
    const void* x;
    const void* weight;
    const void* bias;
    void* y;
    float* mean;
    float* rstd;
    uint64_t x_stride, y_stride;
    uint32_t rows, d;
    float eps;
};

/* Sums of U values over n lanes of a warp (a power of two), the same in each of them; step by
 * step for all U, whose exchanges then wait together. */
template <int U>
__device__ __forceinline__ void lanes_sums(float (&x)[U], uint32_t n)
{
#pragma unroll
    for (uint32_t o = 16; o; o >>= 1)
        if (o < n) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                x[u] = __fadd_rn(x[u], __shfl_xor_sync(0xffffffffu, x[u], o));
        }
}

/* The same over the n threads of U rows: lanes of a warp, or (one row) the whole block. */
template <int U>
__device__ __forceinline__ void row_sums(float (&x)[U], float* slots, uint32_t n)
{
    lanes_sums(x, n);
    if (U > 1 || n <= 32)
        return;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        slots[warp] = x[0];
    __syncthreads();
    x[0] = warp_sum(lane < n / 32 ? slots[lane] : 0.0f);
}

/* U rows, `apart` from each other, of n threads each from their chunks: the statistics, and y
 * (nothing is written of rows behind the last).  params(i, w, b) gives chunk i's weights and
 * biases. */
template <zero_dtype_t DT, int U, int NV, bool VEC, typename Params>
__device__ __forceinline__ void norm_rows(const ForwardArgs& a, uint32_t row, uint32_t apart,
                                          const typename Elem<DT>::Raw (&raw)[U][NV], float (&slots)[2][32], uint32_t k,
                                          uint32_t n, Params params)
{
    using T = typename Elem<DT>::T;
    const uint32_t d = a.d;
    float mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint64_t s = 0;  // a pair of zeros
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint64_t v[4];
            widen2<DT>(raw[u][i], v);
            s = f2_add(s, f2_add(f2_add(v[0], v[1]), f2_add(v[2], v[3])));
        }
        mean[u] = f2_sum(s);
    }
    row_sums(mean, slots[0], n);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        mean[u] = __fdiv_rn(mean[u], (float)d);
        const uint64_t mean2 = f2(mean[u], mean[u]);
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint64_t v[4];
            widen2<DT>(raw[u][i], v);
            if (VEC && elem_of<VEC>(i, 0, k, n) >= d)
                continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint64_t c = f2_sub(v[q], mean2);
                if constexpr (!VEC) {
                    float c0, c1;
                    f2_split(c, c0, c1);
                    c = f2(elem_of<VEC>(i, 2 * q, k, n) < d ? c0 : 0.0f, elem_of<VEC>(i, 2 * q + 1, k, n) < d ? c1 : 0.0f);
                }
                s = f2_fma(c, c, s);
            }
        }
        rstd[u] = f2_sum(s);
    }
    row_sums(rstd, slots[1], n);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float var = __fdiv_rn(rstd[u], (float)d);
        rstd[u] = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t at = row + u * apart;
        if (at >= a.rows)
            break;
        if (k == 0 && a.mean)
            a.mean[at] = mean[u];
        if (k == 0 && a.rstd)
            a.rstd[at] = rstd[u];
        const uint64_t mean2 = f2(mean[u], mean[u]), rstd2 = f2(rstd[u], rstd[u]);
        T* y = static_cast<T*>(a.y) + (uint64_t)at * a.y_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            uint64_t v[4], w[4] = {0, 0, 0, 0}, b[4] = {0, 0, 0, 0};
            widen2<DT>(raw[u][i], v);
            params(i, w, b);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] = f2_fma(f2_mul(f2_sub(v[q], mean2), rstd2), w[q], b[q]);
            float out[8];
            split4(v, out);
            store_chunk<DT, VEC>(y, d, i, k, n, out);
        }
    }
}

/* One row per n threads: a warp (blockDim.y rows per block) or the whole block.  Calls of few rows,
 * where the launch counts, long rows, and rows off the 16-byte grid; of the last a warp would have
 * its 2-byte loads one after another (403 rows of 1,400: 19 us, 9 with 256 threads to a row). */
template <zero_dtype_t DT, zero_dtype_t PT, int NV, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT) k_layernorm(const ForwardArgs a)
{
    using T = typename Elem<DT>::T;
    using P = typename Elem<PT>::T;
    __shared__ float slots[2][32];
    grid_dependency_wait();
    const uint32_t n = blockDim.x, k = threadIdx.x, row = blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= a.rows)
        return;
    const T* x = static_cast<const T*>(a.x) + (uint64_t)row * a.x_stride;
    typename Elem<DT>::Raw raw[1][NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        raw[0][i] = load_chunk<DT, VEC>(x, a.d, i, k, n);
    norm_rows<DT, 1, NV, VEC>(a, row, 0, raw, slots, k, n, [&](int i, uint64_t(&w)[4], uint64_t(&b)[4]) {
        widen2<PT>(load_chunk<PT, VEC>(static_cast<const P*>(a.weight), a.d, i, k, n), w);
        if (a.bias)
            widen2<PT>(load_chunk<PT, VEC>(static_cast<const P*>(a.bias), a.d, i, k, n), b);
    });
}

/* Rows of at most 256 elements (heads' norms): n = 4 to 32 lanes to a row, U rows of each such
 * group in flight, and the weights of a lane's columns in registers.  What bounds it is how many
 * loads are in flight: 204,800 rows of 64 bf16 take 18.5 us (7.7 for their bytes), a warp to a row
 * took 68.  16-bit rows off the 16-byte grid, whose every access is 2 bytes wide, by as many blocks as
 * fit, over the rows in turns: their weights' 16 narrow loads come once, not with every 4 rows (20,909
 * rows of 135 bf16 25.0 us with a block to every 4 rows of its groups, so 23.2; 100,000 of 65 41.3, so 34.5;
 * 200,000 of 33 fp16 28.9, so 26.3; 50,000 of 255 the same).  All others with a block to its rows (in turns: 204,800 of 64 bf16 18.5, 20.3;
 * of 64 fp32 23.0, 24.3; 20,909 of 135 fp32, whose accesses are twice as wide, 18.8, 20.2). */
constexpr uint32_t kShortWarps = 8;

template <zero_dtype_t DT, int U, bool VEC>
constexpr bool kShortTurns = !VEC && DT != ZERO_F32 && U > 1;

template <zero_dtype_t DT, zero_dtype_t PT, int U, bool VEC>
__global__ void __launch_bounds__(32 * kShortWarps) k_layernorm_short(const ForwardArgs a, const uint32_t n)
{
    using T = typename Elem<DT>::T;
    using P = typename Elem<PT>::T;
    __shared__ float slots[2][32];  // not used by single warps
    grid_dependency_wait();
    const uint32_t lane = threadIdx.x & 31, k = lane & (n - 1), rows = 32 / n;
    uint32_t first = (blockIdx.x * kShortWarps + (threadIdx.x >> 5)) * U * rows + lane / n;
    typename Elem<DT>::Raw raw[U][1];
    auto load = [&] {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t row = first + u * rows;
            raw[u][0] =
                load_chunk<DT, VEC>(static_cast<const T*>(a.x) + (uint64_t)row * a.x_stride, row < a.rows ? a.d : 0, 0, k, n);
        }
    };
    uint64_t wk[4], bk[4] = {0, 0, 0, 0};
    auto weights = [&] {
        widen2<PT>(load_chunk<PT, VEC>(static_cast<const P*>(a.weight), a.d, 0, k, n), wk);
        if (a.bias)
            widen2<PT>(load_chunk<PT, VEC>(static_cast<const P*>(a.bias), a.d, 0, k, n), bk);
    };
    auto norm = [&] {
        norm_rows<DT, U, 1, VEC>(a, first, rows, raw, slots, k, n, [&](int, uint64_t(&w)[4], uint64_t(&b)[4]) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                w[q] = wk[q], b[q] = bk[q];
        });
    };
    if constexpr (kShortTurns<DT, U, VEC>) {
        weights();
        const uint32_t step = gridDim.x * kShortWarps * U * rows;
        for (; first - lane / n < a.rows; first += step) {  // the same for the whole warp
            load();
            norm();
        }
    } else {
        load();
        weights();
        norm();
    }
}

#ifdef ZERO_TEST_HOOKS
/* Test builds only (never the product library): the turn of the first block's first ring whose
 * copies are withheld, so that the waits on it run out without any fault. */
__device__ unsigned long long zero_test_withheld_norm_turn = ~0ull;
#define ZERO_WITHHELD(turn) (blockIdx.x == 0 && (turn) == zero_test_withheld_norm_turn)
#else
#define ZERO_WITHHELD(turn) false
#endif

/* A chunk from shared memory. */
template <zero_dtype_t DT>
__device__ __forceinline__ typename Elem<DT>::Raw shared_chunk(const uint4* row, uint32_t c)
{
    typename Elem<DT>::Raw r;
    if constexpr (DT == ZERO_F32)
        r.a = as_f4(row[2 * c]), r.b = as_f4(row[2 * c + 1]);
    else
        r.v = row[c];
    return r;
}

__device__ __forceinline__ void ring_init(uint64_t& full, uint64_t& empty, uint32_t readers)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&full)));
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&empty)), "r"(readers));
}

__device__ __forceinline__ void ring_expect(uint64_t& full, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(&full)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void ring_release(uint64_t& empty)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty)) : "memory");
}

/* At most ~2 s (wait_parity_bounded), the first look without reading the clock. */
__device__ __forceinline__ bool ring_wait(uint64_t& bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(smem_addr(&bar)), "r"(parity)
                 : "memory");
    return ok || wait_parity_bounded(smem_addr(&bar), parity);
}

/* A warp per row, many rows to a warp: lane 0 bulk-copies the warp's next rows into a ring of
 * its own, so that they are on their way while one is worked on.  The weights and biases lie in
 * shared memory (read from global memory row after row they were what a warp waited for).
 * 8,192 rows of 1,600 bf16: 12.8 us a call, its 52 MB 7.7 at the copy's rate; the first, one row to
 * a warp straight from global memory, took 17.7.  What is left is the launch (about 3 us) and
 * issue slots: 32 lanes' conversions and paired arithmetic took 58% of them.  Rows kept ahead in
 * registers (21.5 us) and one copying warp for all rings (15.8) were slower. */
template <zero_dtype_t DT, zero_dtype_t PT, int NV>
__global__ void __launch_bounds__(32 * kRingWarps, 3) k_layernorm_staged(const ForwardArgs a, const uint32_t stages)
{
    using T = typename Elem<DT>::T;
    using P = typename Elem<PT>::T;
    extern __shared__ uint4 rings[];
    __shared__ uint64_t full[kRingWarps][kRing];
    __shared__ float slots[2][32];  // not used by single warps
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = a.d, row_bytes = d * sizeof(T);
    if (lane == 0) {
        for (uint32_t q = 0; q < stages; ++q)
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&full[warp][q])));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    grid_dependency_wait();
    const uint32_t param_words = d * sizeof(P) / 16;
    uint4 *const weight = rings, *const bias = rings + param_words;
    const uint4* ring = rings + 2 * param_words + (uint64_t)warp * stages * row_bytes / 16;
    const uint64_t first = blockIdx.x * kRingWarps + warp, step = gridDim.x * kRingWarps;
    auto fetch = [&](uint32_t turn) {
        const uint64_t row = first + turn * step;
        if (row >= a.rows)
            return;
        const uint32_t q = turn % stages, bar = smem_addr(&full[warp][q]);
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(row_bytes) : "memory");
        if (!(warp == 0 && ZERO_WITHHELD(turn)))
            bulk_load<false>(smem_addr(ring) + q * row_bytes, static_cast<const T*>(a.x) + row * a.x_stride, row_bytes, bar);
    };
    if (lane == 0)
        for (uint32_t q = 0; q < stages; ++q)
            fetch(q);
    for (uint32_t i = threadIdx.x; i < param_words; i += blockDim.x) {
        weight[i] = ld_v4(static_cast<const P*>(a.weight) + i * (16 / sizeof(P)));
        bias[i] = a.bias ? ld_v4(static_cast<const P*>(a.bias) + i * (16 / sizeof(P))) : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    uint32_t turn = 0;
    for (uint64_t row = first; row < a.rows; row += step, ++turn) {
        const uint32_t q = turn % stages;
        const bool ok = __all_sync(0xffffffffu, wait_parity_bounded(smem_addr(&full[warp][q]), turn / stages & 1));
        const uint4* at = ring + q * row_bytes / 16;
        typename Elem<DT>::Raw raw[1][NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t c = i * 32 + lane;
            raw[0][i] = {};
            if (c * 8 < d)
                raw[0][i] = shared_chunk<DT>(at, c);
        }
        __syncwarp();  // the stage has been read
        if (!ok) {     // a copy did not arrive within 2 s: this row and the warp's later ones tell, as NaN
            if (lane == 0)
                for (uint32_t t = turn; t < turn + stages && first + t * step < a.rows; ++t)
                    wait_parity_bounded(smem_addr(&full[warp][t % stages]), t / stages & 1);
            const float nan = __int_as_float(0x7fc00000);
            for (; row < a.rows; row += step) {
                for (uint32_t c = lane; c < d; c += 32)
                    static_cast<T*>(a.y)[row * a.y_stride + c] = from_f32<DT>(nan);
                if (lane == 0 && a.mean)
                    a.mean[row] = nan;
                if (lane == 0 && a.rstd)
                    a.rstd[row] = nan;
            }
            return;
        }
        if (lane == 0)
            fetch(turn + stages);
        norm_rows<DT, 1, NV, true>(a, (uint32_t)row, 0, raw, slots, lane, 32, [&](int i, uint64_t(&w)[4], uint64_t(&b)[4]) {
            const uint32_t c = i * 32 + lane;
            if (c * 8 < d) {
                widen2<PT>(shared_chunk<PT>(weight, c), w);
                widen2<PT>(shared_chunk<PT>(bias, c), b);
            }
        });
    }
}

struct BackwardArgs {
    const void* x;
    const void* weight;
    const float* mean;
    const float* rstd;
    const void* dy;
    void* dx;
    float* parts;  // [blocks][2][d]: each block's sums of dy * xh and of dy
    uint64_t x_stride, dy_stride, dx_stride;
    uint32_t rows, d;
};

/* What a thread keeps over all its block's rows: the weights of its columns, and their sums; in
 * pairs of neighbours. */
template <int NV>
struct Columns {
    uint64_t w[NV][4], dw[NV][4], db[NV][4];

    template <zero_dtype_t PT, bool VEC>
    __device__ __forceinline__ void begin(const BackwardArgs& a, uint32_t k, uint32_t n)
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            widen2<PT>(load_chunk<PT, VEC>(static_cast<const typename Elem<PT>::T*>(a.weight), a.d, i, k, n), w[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                dw[i][q] = db[i][q] = 0;
        }
    }

    /* A chunk of a row into the columns' sums and the row's two, of g and of g * xh, which stay.
     * Past the row's end dy and xh are 0 (the latter too: mean * rstd may be more than fp32 holds
     * where the row's own differences are 0). */
    template <zero_dtype_t DT, bool VEC>
    __device__ __forceinline__ void add(int i, const typename Elem<DT>::Raw& x, const typename Elem<DT>::Raw& dy,
                                        float mean, float rstd, uint64_t (&xh)[4], uint64_t (&g)[4], uint64_t& sg,
                                        uint64_t& sx, uint32_t d, uint32_t k, uint32_t n)
    {
        if (VEC && elem_of<VEC>(i, 0, k, n) >= d)
            mean = 0.0f;
        const uint64_t mean2 = f2(mean, mean), rstd2 = f2(rstd, rstd);
        widen2<DT>(x, xh);
        widen2<DT>(dy, g);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            xh[q] = f2_sub(xh[q], mean2);
            if constexpr (!VEC) {
                float c0, c1;
                f2_split(xh[q], c0, c1);
                xh[q] = f2(elem_of<VEC>(i, 2 * q, k, n) < d ? c0 : 0.0f, elem_of<VEC>(i, 2 * q + 1, k, n) < d ? c1 : 0.0f);
            }
            xh[q] = f2_mul(xh[q], rstd2);
            dw[i][q] = f2_fma(g[q], xh[q], dw[i][q]);
            db[i][q] = f2_add(db[i][q], g[q]);
            g[q] = f2_mul(g[q], w[i][q]);
            sg = f2_add(sg, g[q]);
            sx = f2_fma(g[q], xh[q], sx);
        }
    }

    template <bool VEC>
    __device__ __forceinline__ void end(const BackwardArgs& a, uint32_t k, uint32_t n) const
    {
        float* mine = a.parts + (uint64_t)blockIdx.x * 2 * a.d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float v[8];
            split4(dw[i], v);
            store_chunk<ZERO_F32, VEC>(mine, a.d, i, k, n, v);
            split4(db[i], v);
            store_chunk<ZERO_F32, VEC>(mine + a.d, a.d, i, k, n, v);
        }
    }
};

/* A chunk's dx = rstd * (g - c1 - xh * c2), from the row's two sums over d. */
template <zero_dtype_t DT, bool VEC>
__device__ __forceinline__ void put_dx(int i, typename Elem<DT>::T* dx, uint32_t d, uint32_t k, uint32_t n,
                                       const uint64_t (&xh)[4], const uint64_t (&g)[4], float rstd, float c1, float c2)
{
    const uint64_t rstd2 = f2(rstd, rstd), less1 = f2(c1, c1), less2 = f2(-c2, -c2);
    uint64_t v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
        v[q] = f2_mul(rstd2, f2_fma(xh[q], less2, f2_sub(g[q], less1)));
    float out[8];
    split4(v, out);
    store_chunk<DT, VEC>(dx, d, i, k, n, out);
}

/* Sums of N values over the first n threads; slots are of this turn, so one barrier is enough. */
template <int N>
__device__ __forceinline__ void block_sums(float (&s)[N], float (&slots)[N][32], uint32_t n)
{
#pragma unroll
    for (int q = 0; q < N; ++q)
        s[q] = warp_sum(s[q]);
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
#pragma unroll
        for (int q = 0; q < N; ++q)
            slots[q][warp] = s[q];
    }
    asm volatile("bar.sync 1, %0;" ::"r"(n) : "memory");
#pragma unroll
    for (int q = 0; q < N; ++q)
        s[q] = warp_sum(lane < n / 32 ? slots[q][lane] : 0.0f);
}

/* The same for 4 values over at most 8 warps: halves of the warp, then quarters, take over one
 * value's sum each, which leaves 13 exchanges instead of 40. */
__device__ __forceinline__ void block_sums4(float (&s)[4], float (&slots)[8][4], uint32_t n)
{
    const uint32_t all = 0xffffffffu, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool upper = lane & 16, odd = lane & 8;
    const float a = __fadd_rn(upper ? s[2] : s[0], __shfl_xor_sync(all, upper ? s[0] : s[2], 16));
    const float b = __fadd_rn(upper ? s[3] : s[1], __shfl_xor_sync(all, upper ? s[1] : s[3], 16));
    float v = __fadd_rn(odd ? b : a, __shfl_xor_sync(all, odd ? a : b, 8));
    v = __fadd_rn(v, __shfl_xor_sync(all, v, 4));
    v = __fadd_rn(v, __shfl_xor_sync(all, v, 2));
    v = __fadd_rn(v, __shfl_xor_sync(all, v, 1));
    if ((lane & 7) == 0)
        slots[warp][lane >> 3] = v;
    asm volatile("bar.sync 1, %0;" ::"r"(n) : "memory");
    v = (lane & 7) < n / 32 ? slots[lane & 7][lane >> 3] : 0.0f;
    v = __fadd_rn(v, __shfl_xor_sync(all, v, 4));
    v = __fadd_rn(v, __shfl_xor_sync(all, v, 2));
    v = __fadd_rn(v, __shfl_xor_sync(all, v, 1));
#pragma unroll
    for (int q = 0; q < 4; ++q)
        s[q] = __shfl_sync(all, v, 8 * q);
}

/* R rows at a time per block, straight from global memory: rows that the bulk copies do not
 * take, and the longest.  Bound by the latency of a turn's loads and of its exchanges: 4,099 rows
 * of 641 fp16 take 13.4 us with the join (2.3 for the bytes), 15.4 by at most 4 blocks to an SM
 * instead of 6, 17 with 40 exchanges a turn instead of 13. */
template <zero_dtype_t DT, zero_dtype_t PT, int NV, int R, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT) k_layernorm_backward(const BackwardArgs a)
{
    using T = typename Elem<DT>::T;
    __shared__ float slots[2][R == 2 ? 8 : 2 * R][R == 2 ? 4 : 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t n = blockDim.x, k = threadIdx.x, d = a.d;
    Columns<NV> c;
    c.template begin<PT, VEC>(a, k, n);
    const float inv_d = __fdiv_rn(1.0f, (float)d);
    uint32_t turn = 0;
    for (uint32_t row0 = blockIdx.x * R; row0 < a.rows; row0 += gridDim.x * R, turn ^= 1) {
        typename Elem<DT>::Raw x[R][NV], dy[R][NV];
        uint64_t xh[R][NV][4], g[R][NV][4];
        float mean[R], rstd[R], s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t row = row0 + r, len = row < a.rows ? d : 0;
            mean[r] = len ? a.mean[row] : 0.0f;
            rstd[r] = len ? a.rstd[row] : 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[r][i] = load_chunk<DT, VEC>(static_cast<const T*>(a.x) + (uint64_t)row * a.x_stride, len, i, k, n);
                dy[r][i] = load_chunk<DT, VEC>(static_cast<const T*>(a.dy) + (uint64_t)row * a.dy_stride, len, i, k, n);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint64_t sg = 0, sx = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                c.template add<DT, VEC>(i, x[r][i], dy[r][i], mean[r], rstd[r], xh[r][i], g[r][i], sg, sx, d, k, n);
            s[2 * r] = f2_sum(sg);
            s[2 * r + 1] = f2_sum(sx);
        }
        if constexpr (R == 2)
            block_sums4(s, slots[turn], n);
        else
            block_sums(s, slots[turn], n);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= a.rows)
                break;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                put_dx<DT, VEC>(i, static_cast<T*>(a.dx) + (uint64_t)(row0 + r) * a.dx_stride, d, k, n, xh[r][i], g[r][i],
                                rstd[r], __fmul_rn(s[2 * r], inv_d), __fmul_rn(s[2 * r + 1], inv_d));
        }
    }
    c.template end<VEC>(a, k, n);
}

/* The same through a ring of stages of R rows of x and dy, bulk-copied ahead by one warp more:
 * the rows of the next turns are on their way while one is worked on, without registers.
 * 8,192 rows of 1,600 bf16: 21.7 us a call with the join, 11.6 for its 79 MB at the copy's rate;
 * 38.8 straight from global memory with two barriers a turn.  Left are two launches and, in a
 * turn, the sums' 13 exchanges and barrier.  Blocks of two groups that take turns (27.8 us) and three
 * blocks to an SM, whose registers spill (27.7), were slower. */
template <zero_dtype_t DT, zero_dtype_t PT, int R, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) k_layernorm_backward_staged(const BackwardArgs a, const uint32_t stages)
{
    using T = typename Elem<DT>::T;
    extern __shared__ uint4 ring[];
    __shared__ float slots[2][R == 2 ? 8 : 2 * R][R == 2 ? 4 : 32];
    __shared__ uint64_t full[kRing], empty[kRing];
    __shared__ volatile uint32_t gave_up[2];  // in even turns, in odd ones
    const uint32_t n = blockDim.x - 32, k = threadIdx.x, d = a.d, row_bytes = d * sizeof(T);
    if (k == 0) {
        for (uint32_t q = 0; q < stages; ++q)
            ring_init(full[q], empty[q], n / 32);
        gave_up[0] = gave_up[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    grid_dependency_wait();
    grid_launch_dependents();
    const uint64_t step = (uint64_t)gridDim.x * R;
    if (k >= n) {
        if (k == n) {
            uint32_t q = 0, phase = 1, sent = 0;
            bool ok = true;
            for (uint64_t row0 = (uint64_t)blockIdx.x * R; row0 < a.rows; row0 += step, ++sent) {
                if (sent >= stages && !ring_wait(empty[q], phase)) {
                    ok = false;
                    break;
                }
                const uint32_t rows = a.rows - row0 < R ? (uint32_t)(a.rows - row0) : R;
                const uint32_t bar = smem_addr(&full[q]), to = smem_addr(ring) + q * 2 * R * row_bytes;
                ring_expect(full[q], 2 * rows * row_bytes);
                for (uint32_t r = 0; r < rows && !ZERO_WITHHELD(sent); ++r) {
                    bulk_load<false>(to + 2 * r * row_bytes, static_cast<const T*>(a.x) + (row0 + r) * a.x_stride,
                                     row_bytes, bar);
                    bulk_load<false>(to + (2 * r + 1) * row_bytes, static_cast<const T*>(a.dy) + (row0 + r) * a.dy_stride,
                                     row_bytes, bar);
                }
                q = q + 1 == stages ? 0 : q + 1;
                phase ^= q == 0;
            }
            if (!ok)  // what is on its way lands before the block ends
                for (uint32_t t = sent > stages ? sent - stages : 0; t < sent; ++t)
                    wait_parity_bounded(smem_addr(&full[t % stages]), t / stages & 1);
        }
        __syncthreads();
        return;
    }
    Columns<1> c;
    c.template begin<PT, true>(a, k, n);
    const float inv_d = __fdiv_rn(1.0f, (float)d);
    const bool in = k * 8 < d;
    float mean[R], rstd[R];
    auto statistics = [&](uint64_t row0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            mean[r] = row0 + r < a.rows ? a.mean[row0 + r] : 0.0f;
            rstd[r] = row0 + r < a.rows ? a.rstd[row0 + r] : 0.0f;
        }
    };
    statistics((uint64_t)blockIdx.x * R);
    uint32_t q = 0, phase = 0, turn = 0;
    uint64_t row0 = (uint64_t)blockIdx.x * R;
    for (; row0 < a.rows; row0 += step, turn ^= 1) {
        if (!ring_wait(full[q], phase))
            gave_up[turn] = 1;
        const uint4* stage = ring + (uint64_t)q * 2 * R * row_bytes / 16;
        uint64_t xh[R][4], g[R][4];
        typename Elem<DT>::Raw x[R], dy[R];
        float s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r] = dy[r] = {};
            if (in && row0 + r < a.rows) {
                const uint4 *px = stage + 2 * r * row_bytes / 16, *py = px + row_bytes / 16;
                x[r] = shared_chunk<DT>(px, k);
                dy[r] = shared_chunk<DT>(py, k);
            }
        }
        __syncwarp();
        if ((k & 31) == 0)
            ring_release(empty[q]);
        q = q + 1 == stages ? 0 : q + 1;
        phase ^= q == 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint64_t sg = 0, sx = 0;
            c.template add<DT, true>(0, x[r], dy[r], mean[r], rstd[r], xh[r], g[r], sg, sx, d, k, n);
            s[2 * r] = f2_sum(sg);
            s[2 * r + 1] = f2_sum(sx);
        }
        float rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            rs[r] = rstd[r];
        statistics(row0 + step);  // of the next turn
        if constexpr (R == 2)
            block_sums4(s, slots[turn], n);
        else
            block_sums(s, slots[turn], n);
        if (gave_up[turn])  // set before the sums' barrier: the same answer in every thread
            break;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= a.rows)
                break;
            put_dx<DT, true>(0, static_cast<T*>(a.dx) + (row0 + r) * a.dx_stride, d, k, n, xh[r], g[r], rs[r],
                             __fmul_rn(s[2 * r], inv_d), __fmul_rn(s[2 * r + 1], inv_d));
        }
    }
    if (gave_up[0] | gave_up[1]) {  // a copy did not arrive within 2 s: the rows left and the weights' gradients tell, as NaN
        const float nan = __int_as_float(0x7fc00000);
        c.dw[0][0] = c.db[0][0] = f2(nan, 0.0f);
        for (; row0 < a.rows; row0 += step)
            for (uint32_t i = k; i < R * d && row0 + i / d < a.rows; i += n)
                static_cast<T*>(a.dx)[(row0 + i / d) * a.dx_stride + i % d] = from_f32<DT>(nan);
    }
    c.template end<true>(a, k, n);
    __syncthreads();
}

/* Rows of at most 256 elements: n = 4 to 32 lanes to a row as in the forward pass, R rows of each
 * group in flight; at the end the groups' sums of a column are joined, those of a warp over its
 * lanes, then the warps' in order.  204,800 rows of 64 bf16: 26 us with the join (11.6 for the
 * bytes), 142 with a block to two rows; 20,909 rows of 135: 25 us instead of 64. */
template <zero_dtype_t DT, zero_dtype_t PT, int R, bool VEC>
__global__ void __launch_bounds__(32 * kShortWarps) k_layernorm_backward_short(const BackwardArgs a, const uint32_t n)
{
    using T = typename Elem<DT>::T;
    __shared__ float sums[kShortWarps][2][8][33];  // [warp][of dweight, dbias][element of the chunk][lane]
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, k = lane & (n - 1), groups = 32 / n, d = a.d;
    Columns<1> c;
    c.template begin<PT, VEC>(a, k, n);
    const float inv_d = __fdiv_rn(1.0f, (float)d);
    const uint32_t step = gridDim.x * kShortWarps * R * groups;
    for (uint32_t row0 = (blockIdx.x * kShortWarps + warp) * R * groups; row0 < a.rows; row0 += step) {
        typename Elem<DT>::Raw x[R], dy[R];
        float mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t row = row0 + r * groups + lane / n, len = row < a.rows ? d : 0;
            x[r] = load_chunk<DT, VEC>(static_cast<const T*>(a.x) + (uint64_t)row * a.x_stride, len, 0, k, n);
            dy[r] = load_chunk<DT, VEC>(static_cast<const T*>(a.dy) + (uint64_t)row * a.dy_stride, len, 0, k, n);
            mean[r] = len ? a.mean[row] : 0.0f;
            rstd[r] = len ? a.rstd[row] : 0.0f;
        }
        uint64_t xh[R][4], g[R][4];
        float s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            uint64_t sg = 0, sx = 0;
            c.template add<DT, VEC>(0, x[r], dy[r], mean[r], rstd[r], xh[r], g[r], sg, sx, d, k, n);
            s[2 * r] = f2_sum(sg);
            s[2 * r + 1] = f2_sum(sx);
        }
        lanes_sums(s, n);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t row = row0 + r * groups + lane / n;
            if (row < a.rows)
                put_dx<DT, VEC>(0, static_cast<T*>(a.dx) + (uint64_t)row * a.dx_stride, d, k, n, xh[r], g[r], rstd[r],
                                __fmul_rn(s[2 * r], inv_d), __fmul_rn(s[2 * r + 1], inv_d));
        }
    }
    float v[2][8];
    split4(c.dw[0], v[0]);
    split4(c.db[0], v[1]);
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            for (uint32_t o = 16; o >= n; o >>= 1)
                v[q][j] = __fadd_rn(v[q][j], __shfl_xor_sync(0xffffffffu, v[q][j], o));
            sums[warp][q][j][lane] = v[q][j];
        }
    __syncthreads();
    if (warp >= 2 || lane >= n)
        return;
    float s[8];  // the first warp joins dweight's, the second dbias's
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        s[j] = sums[0][warp][j][lane];
#pragma unroll
        for (uint32_t w = 1; w < kShortWarps; ++w)
            s[j] = __fadd_rn(s[j], sums[w][warp][j][lane]);
    }
    store_chunk<ZERO_F32, VEC>(a.parts + ((uint64_t)blockIdx.x * 2 + warp) * d, d, 0, k, n, s);
}

struct JoinArgs {
    const float* parts;
    void* dweight;
    void* dbias;
    uint32_t n_parts, d;
    uint32_t dtype, accumulate;
};

/* The blocks' sums of one column: 32 columns by 32 runs of parts per block, in a fixed order. */
__global__ void __launch_bounds__(1024) k_layernorm_join(const JoinArgs a)
{
    __shared__ float part[32][33];
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    uint32_t col = blockIdx.x * 32 + lane;
    const uint32_t n = 2 * a.d;
    float s = 0.0f;
    if (col < n) {
#pragma unroll 10
        for (uint32_t p = run; p < a.n_parts; p += 32)
            s = __fadd_rn(s, a.parts[(uint64_t)p * n + col]);
    }
    part[run][lane] = s;
    __syncthreads();
    // a warp per column now: its 32 runs
    s = warp_sum(part[lane][run]);
    col = blockIdx.x * 32 + run;
    if (lane || col >= n)
        return;
    void* out = col < a.d ? a.dweight : a.dbias;
    if (!out)
        return;
    const uint32_t c = col < a.d ? col : col - a.d;
    if (a.dtype == ZERO_F32) {
        float* p = static_cast<float*>(out) + c;
        *p = a.accumulate ? __fadd_rn(*p, s) : s;
    } else {
        uint16_t* p = static_cast<uint16_t*>(out) + c;
        const bool h = a.dtype == ZERO_F16;
        if (a.accumulate)
            s = __fadd_rn(s, h ? one16<ZERO_F16>(*p) : one16<ZERO_BF16>(*p));
        *p = h ? pack1<true>(s) : pack1<false>(s);
    }
}

/* Rows by warps with rings, if there are several rows to a warp. */
template <auto KERNEL>
cudaError_t forward_staged(const ForwardArgs& a, size_t params, size_t row_bytes, bool& taken, cudaStream_t s)
{
    // three blocks to an SM; two stages of the longest fp32 rows leave room for two of them (from 1,280
    // elements up) or one (from 1,600), still not slower than a row to a warp straight from global memory:
    // 8,192 rows of fp32, L2 flushed, 1,024 elements 20.1 us (20.9 without rings), 1,280 22.9 (25.0),
    // 1,600 27.1 (28.9), 2,048 32.4 (32.6); of 640 16.8 (15.9), where the rings cost 6%
    size_t stages = (72 * 1024 - params) / (kRingWarps * row_bytes);
    stages = stages < 2 ? 2 : stages > kRing ? kRing : stages;
    const size_t smem = params + kRingWarps * stages * row_bytes;
    uint32_t fit = 0;
    cudaError_t e = allow_smem<KERNEL>();
    if (e == cudaSuccess)
        e = resident<KERNEL>(32 * kRingWarps, smem, fit);
    taken = e == cudaSuccess && a.rows > fit * kRingWarps;
    return taken ? launch_pdl(KERNEL, dim3(fit), dim3(32 * kRingWarps), smem, s, a, (uint32_t)stages) : e;
}

/* Lanes to a row of at most 256 elements. */
uint32_t short_lanes(uint32_t chunks) { return chunks <= 4 ? 4 : chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32; }

template <zero_dtype_t DT, zero_dtype_t PT, bool VEC>
cudaError_t forward(const ForwardArgs& a, cudaStream_t s)
{
    const uint32_t chunks = (a.d + 7) / 8;
    if (chunks <= 32) {
        const uint32_t lanes = short_lanes(chunks), rows = kShortWarps * (32 / lanes);
        const bool many = a.rows > 4 * rows * (uint32_t)sm_count();  // a block on each SM, with 4 rows to a group
        uint32_t blocks = many ? (a.rows + 4 * rows - 1) / (4 * rows) : (a.rows + rows - 1) / rows;
        if (kShortTurns<DT, 4, VEC> && many) {
            uint32_t fit = 0;
            const cudaError_t e = resident<k_layernorm_short<DT, PT, 4, VEC>>(32 * kShortWarps, 0, fit);
            if (e != cudaSuccess)
                return e;
            blocks = blocks < fit ? blocks : fit;
        }
        const dim3 grid(blocks);
        return many ? launch_pdl(k_layernorm_short<DT, PT, 4, VEC>, grid, dim3(32 * kShortWarps), 0, s, a, lanes)
                    : launch_pdl(k_layernorm_short<DT, PT, 1, VEC>, grid, dim3(32 * kShortWarps), 0, s, a, lanes);
    }
    // in 128-bit accesses a warp per row up to 2,048 elements (no barrier), then 128 and 512 threads;
    // element by element a chunk or two to a thread (4,096 rows of 1,601: 37 us with 128 threads, 29
    // with 256, 53 with 512; 1,957 of 3,235: 42, 35, 31; 403 of 1,400: 13, 9, 13)
    const uint32_t n = VEC ? (chunks <= 256 ? 32 : chunks <= 1024 ? 128 : 512) : chunks <= 128 ? 128 : chunks <= 1024 ? 256 : 512;
    const uint32_t per = (chunks + n - 1) / n, rows = n == 32 ? 4 : 1;
    if constexpr (VEC) {
        if (n == 32) {
            const size_t params = 2 * a.d * sizeof(typename Elem<PT>::T), row = a.d * sizeof(typename Elem<DT>::T);
            bool taken = false;
            cudaError_t e = cudaSuccess;
            // exactly the chunks that a lane holds: an eighth for 1,600 elements (7) cost 10%
            switch (per) {
            case 2: e = forward_staged<k_layernorm_staged<DT, PT, 2>>(a, params, row, taken, s); break;
            case 3: e = forward_staged<k_layernorm_staged<DT, PT, 3>>(a, params, row, taken, s); break;
            case 4: e = forward_staged<k_layernorm_staged<DT, PT, 4>>(a, params, row, taken, s); break;
            case 5: e = forward_staged<k_layernorm_staged<DT, PT, 5>>(a, params, row, taken, s); break;
            case 6: e = forward_staged<k_layernorm_staged<DT, PT, 6>>(a, params, row, taken, s); break;
            case 7: e = forward_staged<k_layernorm_staged<DT, PT, 7>>(a, params, row, taken, s); break;
            default: e = forward_staged<k_layernorm_staged<DT, PT, 8>>(a, params, row, taken, s); break;
            }
            if (taken || e != cudaSuccess)
                return e;
        }
    }
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3((a.rows + rows - 1) / rows), dim3(n, rows), 0, s, a);
    };
    if (n == 512)
        return per <= 2 ? go(k_layernorm<DT, PT, 2, VEC, 512>) : go(k_layernorm<DT, PT, 4, VEC, 512>);
    if constexpr (VEC)
        return per <= 2   ? go(k_layernorm<DT, PT, 2, VEC, 128>)
               : per <= 4 ? go(k_layernorm<DT, PT, 4, VEC, 128>)
                          : go(k_layernorm<DT, PT, 8, VEC, 128>);
    else
        return per <= 1   ? go(k_layernorm<DT, PT, 1, VEC, 256>)
               : per <= 2 ? go(k_layernorm<DT, PT, 2, VEC, 256>)
                          : go(k_layernorm<DT, PT, 4, VEC, 256>);
}

/* As many blocks as fit at once, each with its share of the rows and its part of the sums. */
template <auto KERNEL, typename... More>
cudaError_t backward_blocks(const BackwardArgs& a, uint32_t threads, uint32_t rows, size_t smem, uint32_t& parts,
                            cudaStream_t s, More... more)
{
    uint32_t fit = 0;
    cudaError_t e = smem ? allow_smem<KERNEL>() : cudaSuccess;
    if (e == cudaSuccess)
        e = resident<KERNEL>(threads, smem, fit);
    if (e != cudaSuccess)
        return e;
    const uint32_t want = (a.rows + rows - 1) / rows;
    parts = fit < kMaxParts ? fit : kMaxParts;
    parts = parts < want ? parts : want;
    return launch_pdl(KERNEL, dim3(parts), dim3(threads), smem, s, a, more...);
}

template <zero_dtype_t DT, zero_dtype_t PT, bool VEC>
cudaError_t backward(const BackwardArgs& a, uint32_t& parts, cudaStream_t s)
{
    // one warp more than the chunks need copies rows in
    const uint32_t chunks = (a.d + 7) / 8, n = chunks <= 992 ? (chunks + 31) / 32 * 32 : 1024;
    if (chunks <= 32) {
        const uint32_t lanes = short_lanes(chunks), rows = kShortWarps * (32 / lanes);
        constexpr uint32_t R = VEC ? 4 : 2;  // element by element 4 take 147 registers: 48 us instead of 34
        return a.rows > R * rows * (uint32_t)sm_count()
                   ? backward_blocks<k_layernorm_backward_short<DT, PT, R, VEC>>(a, 32 * kShortWarps, R * rows, 0, parts, s, lanes)
                   : backward_blocks<k_layernorm_backward_short<DT, PT, 1, VEC>>(a, 32 * kShortWarps, rows, 0, parts, s, lanes);
    }
    if (chunks > 992)
        return backward_blocks<k_layernorm_backward<DT, PT, 2, 1, VEC, 1024>>(a, n, 1, 0, parts, s);
    if constexpr (VEC) {
        // a ring of up to 48 KB: two blocks and more to an SM
        const uint32_t rows = chunks <= 256 ? 2 : 1, stage = 2 * rows * a.d * (uint32_t)sizeof(typename Elem<DT>::T);
        uint32_t stages = 49152 / stage;
        stages = stages < 2 ? 2 : stages > kRing ? kRing : stages;
        const size_t smem = (size_t)stages * stage;
        return chunks <= 256
                   ? backward_blocks<k_layernorm_backward_staged<DT, PT, 2, 288>>(a, n + 32, 2, smem, parts, s, stages)
                   : backward_blocks<k_layernorm_backward_staged<DT, PT, 1, 1024>>(a, n + 32, 1, smem, parts, s, stages);
    } else {
        return chunks <= 256 ? backward_blocks<k_layernorm_backward<DT, PT, 1, 2, VEC, 256>>(a, n, 2, 0, parts, s)
                             : backward_blocks<k_layernorm_backward<DT, PT, 1, 1, VEC, 1024>>(a, n, 1, 0, parts, s);
    }
}

/* Calls f with the types and the layout as template arguments. */
template <typename F>
cudaError_t with_types(zero_dtype_t dtype, zero_dtype_t param, bool vec, F&& f)
{
#define ZERO_LN_CASE(D, P)                                                                    \
    if (dtype == D && param == P)                                                             \
        return vec ? f.template operator()<D, P, true>() : f.template operator()<D, P, false>();
    ZERO_LN_CASE(ZERO_BF16, ZERO_BF16)
    ZERO_LN_CASE(ZERO_F16, ZERO_F16)
    ZERO_LN_CASE(ZERO_F32, ZERO_F32)
    ZERO_LN_CASE(ZERO_BF16, ZERO_F32)
    ZERO_LN_CASE(ZERO_F16, ZERO_F32)
#undef ZERO_LN_CASE
    return cudaErrorInvalidValue;
}

struct RunForward {
    const ForwardArgs& a;
    cudaStream_t s;
    template <zero_dtype_t D, zero_dtype_t P, bool VEC>
    cudaError_t operator()() const { return forward<D, P, VEC>(a, s); }
};

struct RunBackward {
    const BackwardArgs& a;
    uint32_t& parts;
    cudaStream_t s;
    template <zero_dtype_t D, zero_dtype_t P, bool VEC>
    cudaError_t operator()() const { return backward<D, P, VEC>(a, parts, s); }
};

bool types_ok(zero_dtype_t dtype, zero_dtype_t param)
{
    return float_dtype(dtype) && (param == dtype || param == ZERO_F32);
}

bool sizes_ok(uint64_t rows, uint32_t dim)
{
    return rows <= (1ull << 30) && dim >= 1 && dim <= kMaxDim;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

#ifdef ZERO_TEST_HOOKS
int zero_test_withhold_norm_turn(unsigned long long turn)
{
    return cudaMemcpyToSymbol(zero_test_withheld_norm_turn, &turn, sizeof turn) == cudaSuccess ? 0 : -4;
}
#endif

int zero_layernorm(zero_dtype_t dtype, uint64_t rows, uint32_t dim, const void* x, uint64_t x_stride,
                   const void* weight, const void* bias, zero_dtype_t param_dtype, float eps, void* y,
                   uint64_t y_stride, float* mean, float* rstd, zero_stream_t stream)
{
    NvtxRange range("zero_layernorm");
    if (!types_ok(dtype, param_dtype) || !sizes_ok(rows, dim) || !(eps >= 0.0f) || !(eps <= 3.0e38f))
        return ZERO_EINVAL;
    if (rows == 0)
        return ZERO_OK;
    if (!x || !weight || !y || (rows > 1 && (x_stride < dim || y_stride < dim)) ||
        x_stride > (1ull << 32) || y_stride > (1ull << 32))
        return ZERO_EINVAL;
    const size_t e = dtype_size(dtype), p = dtype_size(param_dtype);
    if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(weight, p) || !aligned_to(bias, p) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return ZERO_EALIGN;
    if (!apart({{y, rows, y_stride, dim, dtype}, {mean, rows * 4}, {rstd, rows * 4}},
               {{x, rows, x_stride, dim, dtype}, {weight, dim * p}, {bias, dim * p}}))
        return ZERO_EINVAL;
    const ForwardArgs a{x, weight, bias, y, mean, rstd, x_stride, y_stride, (uint32_t)rows, dim, eps};
    const bool vec = rows_vec(x, x_stride, dim, dtype) && rows_vec(y, y_stride, dim, dtype) &&
                     aligned_to(weight, 16) && aligned_to(bias, 16);
    return rows_status(with_types(dtype, param_dtype, vec, RunForward{a, stream}));
}

size_t zero_layernorm_workspace_bytes(uint64_t rows, uint32_t dim)
{
    if (!sizes_ok(rows, dim))
        return 0;
    const uint64_t parts = rows < kMaxParts ? rows : kMaxParts;
    return (size_t)((parts ? parts : 1) * 2 * dim * sizeof(float));
}

int zero_layernorm_backward(zero_dtype_t dtype, uint64_t rows, uint32_t dim, const void* x, uint64_t x_stride,
                            const void* weight, zero_dtype_t param_dtype, const float* mean, const float* rstd,
                            const void* dy, uint64_t dy_stride, void* dx, uint64_t dx_stride, void* dweight,
                            void* dbias, zero_dtype_t grad_dtype, uint32_t accumulate, void* workspace,
                            zero_stream_t stream)
{
    NvtxRange range("zero_layernorm_backward");
    if (!types_ok(dtype, param_dtype) || !sizes_ok(rows, dim) || accumulate > 1 ||
        (grad_dtype != dtype && grad_dtype != ZERO_F32) || !workspace)
        return ZERO_EINVAL;
    if (rows && (!x || !weight || !mean || !rstd || !dy || !dx ||
                 (rows > 1 && (x_stride < dim || dy_stride < dim || dx_stride < dim)) || x_stride > (1ull << 32) ||
                 dy_stride > (1ull << 32) || dx_stride > (1ull << 32)))
        return ZERO_EINVAL;
    const size_t e = dtype_size(dtype), g = dtype_size(grad_dtype);
    if (!aligned_to(x, e) || !aligned_to(dy, e) || !aligned_to(dx, e) || !aligned_to(weight, dtype_size(param_dtype)) ||
        !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dweight, g) || !aligned_to(dbias, g) ||
        !aligned_to(workspace, 16))
        return ZERO_EALIGN;
    if (!apart({{dx, rows, dx_stride, dim, dtype},
                {dweight, dim * g},
                {dbias, dim * g},
                {workspace, zero_layernorm_workspace_bytes(rows, dim)}},
               {{x, rows, x_stride, dim, dtype},
                {dy, rows, dy_stride, dim, dtype},
                {weight, dim * dtype_size(param_dtype)},
                {mean, rows * 4},
                {rstd, rows * 4}}))
        return ZERO_EINVAL;
    uint32_t parts = 0;
    if (rows) {
        const BackwardArgs a{x,        weight,    mean,      rstd,           dy, dx, static_cast<float*>(workspace),
                             x_stride, dy_stride, dx_stride, (uint32_t)rows, dim};
        const bool vec = rows_vec(x, x_stride, dim, dtype) && rows_vec(dy, dy_stride, dim, dtype) &&
                         rows_vec(dx, dx_stride, dim, dtype) && aligned_to(weight, 16);
        const int rc = rows_status(with_types(dtype, param_dtype, vec, RunBackward{a, parts, stream}));
        if (rc != ZERO_OK)
            return rc;
    }
    if (!dweight && !dbias)
        return ZERO_OK;
    const JoinArgs j{static_cast<const float*>(workspace), dweight, dbias, parts, dim, (uint32_t)grad_dtype, accumulate};
    return rows_status(launch_pdl(k_layernorm_join, dim3((2 * dim + 31) / 32), dim3(1024), 0, stream, j));
}

}  // extern "C"
