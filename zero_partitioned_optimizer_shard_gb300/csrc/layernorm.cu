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

#include <atomic>

namespace zero {
namespace {

constexpr uint32_t kMaxDim = 16384;
constexpr uint32_t kMaxParts = 608;  // blocks of the backward pass: 4 on each of 152 SMs

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

/* A sum over the block (of one warp: over the warp), the same in every thread. */
__device__ __forceinline__ float row_sum(float x, float* slots, uint32_t n)
{
    x = warp_sum(x);
    if (n == 32)
        return x;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
        slots[warp] = x;
    __syncthreads();
    return warp_sum(lane < n / 32 ? slots[lane] : 0.0f);
}

/* One row per n threads: a warp (blockDim.y rows per block) or the whole block. */
template <zero_dtype_t DT, zero_dtype_t PT, int NV, bool VEC>
__global__ void __launch_bounds__(512) k_layernorm(const ForwardArgs a)
{
    using T = typename Elem<DT>::T;
    using P = typename Elem<PT>::T;
    __shared__ float slots[2][32];
    grid_dependency_wait();
    const uint32_t n = blockDim.x, k = threadIdx.x, d = a.d;
    const uint32_t row = blockIdx.x * blockDim.y + threadIdx.y;
    if (row >= a.rows)
        return;
    const T* x = static_cast<const T*>(a.x) + (uint64_t)row * a.x_stride;
    typename Elem<DT>::Raw raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        raw[i] = load_chunk<DT, VEC>(x, d, i, k, n);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float v[8];
        widen<DT>(raw[i], v);
        s = __fadd_rn(s, __fadd_rn(__fadd_rn(__fadd_rn(v[0], v[1]), __fadd_rn(v[2], v[3])),
                                   __fadd_rn(__fadd_rn(v[4], v[5]), __fadd_rn(v[6], v[7]))));
    }
    const float mean = __fdiv_rn(row_sum(s, slots[0], n), (float)d);
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float v[8];
        widen<DT>(raw[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float c = elem_of<VEC>(i, j, k, n) < d ? __fsub_rn(v[j], mean) : 0.0f;
            s = __fmaf_rn(c, c, s);
        }
    }
    const float var = __fdiv_rn(row_sum(s, slots[1], n), (float)d);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
    if (k == 0 && a.mean)
        a.mean[row] = mean;
    if (k == 0 && a.rstd)
        a.rstd[row] = rstd;
    T* y = static_cast<T*>(a.y) + (uint64_t)row * a.y_stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float v[8], w[8], b[8];
        widen<DT>(raw[i], v);
        widen<PT>(load_chunk<PT, VEC>(static_cast<const P*>(a.weight), d, i, k, n), w);
        if (a.bias) {
            widen<PT>(load_chunk<PT, VEC>(static_cast<const P*>(a.bias), d, i, k, n), b);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                b[j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = __fmaf_rn(__fmul_rn(__fsub_rn(v[j], mean), rstd), w[j], b[j]);
        store_chunk<DT, VEC>(y, d, i, k, n, v);
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

/* R rows at a time per block; a thread keeps its columns' sums over the block's rows. */
template <zero_dtype_t DT, zero_dtype_t PT, int NV, int R, bool VEC>
__global__ void __launch_bounds__(1024) k_layernorm_backward(const BackwardArgs a)
{
    using T = typename Elem<DT>::T;
    using P = typename Elem<PT>::T;
    __shared__ float slots[2][2 * R][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t n = blockDim.x, k = threadIdx.x, d = a.d, warp = k >> 5, lane = k & 31;
    float w[NV][8], dw[NV][8], db[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        widen<PT>(load_chunk<PT, VEC>(static_cast<const P*>(a.weight), d, i, k, n), w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            dw[i][j] = db[i][j] = 0.0f;
    }
    const float inv_d = __fdiv_rn(1.0f, (float)d);
    uint32_t turn = 0;
    for (uint32_t row0 = blockIdx.x * R; row0 < a.rows; row0 += gridDim.x * R, turn ^= 1) {
        typename Elem<DT>::Raw x[R][NV], dy[R][NV];
        float mean[R], rstd[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t row = row0 + r;
            const uint32_t len = row < a.rows ? d : 0;
            mean[r] = len ? a.mean[row] : 0.0f;
            rstd[r] = len ? a.rstd[row] : 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[r][i] = load_chunk<DT, VEC>(static_cast<const T*>(a.x) + (uint64_t)row * a.x_stride, len, i, k, n);
                dy[r][i] = load_chunk<DT, VEC>(static_cast<const T*>(a.dy) + (uint64_t)row * a.dy_stride, len, i, k, n);
            }
        }
        float s[2 * R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[2 * r] = s[2 * r + 1] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float xv[8], dv[8];
                widen<DT>(x[r][i], xv);
                widen<DT>(dy[r][i], dv);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    // places past the row's end hold dy = 0, and xh must not make a NaN of it
                    const bool in = VEC ? (i * n + k) * 8 < d : elem_of<VEC>(i, j, k, n) < d;
                    const float xh = in ? __fmul_rn(__fsub_rn(xv[j], mean[r]), rstd[r]) : 0.0f;
                    const float g = __fmul_rn(dv[j], w[i][j]);
                    s[2 * r] = __fadd_rn(s[2 * r], g);
                    s[2 * r + 1] = __fmaf_rn(g, xh, s[2 * r + 1]);
                    dw[i][j] = __fmaf_rn(dv[j], xh, dw[i][j]);
                    db[i][j] = __fadd_rn(db[i][j], dv[j]);
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 2 * R; ++q)
            s[q] = warp_sum(s[q]);
        if (n > 32) {
            if (lane == 0) {
#pragma unroll
                for (int q = 0; q < 2 * R; ++q)
                    slots[turn][q][warp] = s[q];
            }
            __syncthreads();  // the other set of slots is written next: one barrier a turn
#pragma unroll
            for (int q = 0; q < 2 * R; ++q)
                s[q] = warp_sum(lane < n / 32 ? slots[turn][q][lane] : 0.0f);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t row = row0 + r;
            if (row >= a.rows)
                break;
            const float c1 = __fmul_rn(s[2 * r], inv_d), c2 = __fmul_rn(s[2 * r + 1], inv_d);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float xv[8], dv[8];
                widen<DT>(x[r][i], xv);
                widen<DT>(dy[r][i], dv);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float xh = __fmul_rn(__fsub_rn(xv[j], mean[r]), rstd[r]);
                    xv[j] = __fmul_rn(rstd[r], __fmaf_rn(-xh, c2, __fsub_rn(__fmul_rn(dv[j], w[i][j]), c1)));
                }
                store_chunk<DT, VEC>(static_cast<T*>(a.dx) + (uint64_t)row * a.dx_stride, d, i, k, n, xv);
            }
        }
    }
    float* mine = a.parts + (uint64_t)blockIdx.x * 2 * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        store_chunk<ZERO_F32, VEC>(mine, d, i, k, n, dw[i]);
        store_chunk<ZERO_F32, VEC>(mine + d, d, i, k, n, db[i]);
    }
}

struct JoinArgs {
    const float* parts;
    void* dweight;
    void* dbias;
    uint32_t n_parts, d;
    uint32_t dtype, accumulate;
};

/* The blocks' sums of one column, in the order of the blocks: 32 columns by 8 runs of parts
 * per block. */
__global__ void __launch_bounds__(256) k_layernorm_join(const JoinArgs a)
{
    __shared__ float part[8][33];
    grid_dependency_wait();
    const uint32_t lane = threadIdx.x & 31, run = threadIdx.x >> 5;
    const uint32_t col = blockIdx.x * 32 + lane, n = 2 * a.d;
    float s = 0.0f;
    if (col < n) {
        const uint32_t each = (a.n_parts + 7) / 8, lo = run * each;
        const uint32_t hi = lo + each < a.n_parts ? lo + each : a.n_parts;
#pragma unroll 8
        for (uint32_t p = lo; p < hi; ++p)
            s = __fadd_rn(s, a.parts[(uint64_t)p * n + col]);
    }
    part[run][lane] = s;
    __syncthreads();
    if (run || col >= n)
        return;
#pragma unroll
    for (int r = 1; r < 8; ++r)
        s = __fadd_rn(s, part[r][lane]);
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

template <zero_dtype_t DT, zero_dtype_t PT, bool VEC>
cudaError_t forward(const ForwardArgs& a, cudaStream_t s)
{
    // a warp per row up to 2,048 elements (no barrier), then 128 and 512 threads
    const uint32_t chunks = (a.d + 7) / 8, n = chunks <= 256 ? 32 : chunks <= 1024 ? 128 : 512;
    const uint32_t per = (chunks + n - 1) / n, rows = n == 32 ? 4 : 1;
    const dim3 grid((a.rows + rows - 1) / rows), block(n, rows);
    if (per <= 1)
        return launch_pdl(k_layernorm<DT, PT, 1, VEC>, grid, block, 0, s, a);
    if (per <= 2)
        return launch_pdl(k_layernorm<DT, PT, 2, VEC>, grid, block, 0, s, a);
    if (per <= 4)
        return launch_pdl(k_layernorm<DT, PT, 4, VEC>, grid, block, 0, s, a);
    return launch_pdl(k_layernorm<DT, PT, 8, VEC>, grid, block, 0, s, a);
}

template <zero_dtype_t DT, zero_dtype_t PT, bool VEC>
cudaError_t backward(const BackwardArgs& a, uint32_t& parts, cudaStream_t s)
{
    constexpr int R = DT == ZERO_F32 ? 2 : 4;
    const uint32_t chunks = (a.d + 7) / 8;
    const uint32_t n = chunks <= 1024 ? (chunks + 31) / 32 * 32 : 1024;
    auto go = [&](auto kernel, int rows) {
        int per_sm = 0;
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, (int)n, 0);
        if (e != cudaSuccess)
            return e;
        uint32_t grid = (uint32_t)(sm_count() * (per_sm > 0 ? per_sm : 1));
        grid = grid < kMaxParts ? grid : kMaxParts;
        const uint32_t want = (a.rows + rows - 1) / rows;
        parts = grid < want ? grid : want;
        return launch_pdl(kernel, dim3(parts), dim3(n), 0, s, a);
    };
    if (chunks > 1024)
        return go(k_layernorm_backward<DT, PT, 2, 1, VEC>, 1);
    return go(k_layernorm_backward<DT, PT, 1, R, VEC>, R);
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

bool weight_vec(const void* p, zero_dtype_t t) { return !p || (aligned_to(p, 16) && float_dtype(t)); }

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

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
    const uint64_t ny = span(rows, y_stride, dim, dtype), nx = span(rows, x_stride, dim, dtype), np = dim * p;
    if (overlap(y, ny, x, nx) || overlap(y, ny, weight, np) || overlap(y, ny, bias, np) ||
        overlap(y, ny, mean, rows * 4) || overlap(y, ny, rstd, rows * 4) || overlap(mean, rows * 4, rstd, rows * 4))
        return ZERO_EINVAL;
    const ForwardArgs a{x, weight, bias, y, mean, rstd, x_stride, y_stride, (uint32_t)rows, dim, eps};
    const bool vec = rows_vec(x, x_stride, dim, dtype) && rows_vec(y, y_stride, dim, dtype) &&
                     weight_vec(weight, param_dtype) && weight_vec(bias, param_dtype);
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
    const uint64_t nx = span(rows, x_stride, dim, dtype), ny = span(rows, dy_stride, dim, dtype),
                   nd = span(rows, dx_stride, dim, dtype), np = dim * dtype_size(param_dtype), ng = dim * g,
                   nw = zero_layernorm_workspace_bytes(rows, dim);
    const struct {
        const void* p;
        uint64_t n;
    } in[] = {{x, nx}, {dy, ny}, {weight, np}, {mean, rows * 4}, {rstd, rows * 4}},
      out[] = {{dx, nd}, {dweight, ng}, {dbias, ng}, {workspace, nw}};
    for (int i = 0; i < 4; ++i) {
        for (const auto& b : in)
            if (overlap(out[i].p, out[i].n, b.p, b.n))
                return ZERO_EINVAL;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
                return ZERO_EINVAL;
    }
    uint32_t parts = 0;
    if (rows) {
        const BackwardArgs a{x,        weight,    mean,      rstd,           dy, dx, static_cast<float*>(workspace),
                             x_stride, dy_stride, dx_stride, (uint32_t)rows, dim};
        const bool vec = rows_vec(x, x_stride, dim, dtype) && rows_vec(dy, dy_stride, dim, dtype) &&
                         rows_vec(dx, dx_stride, dim, dtype) && weight_vec(weight, param_dtype);
        const int rc = rows_status(with_types(dtype, param_dtype, vec, RunBackward{a, parts, stream}));
        if (rc != ZERO_OK)
            return rc;
    }
    if (!dweight && !dbias)
        return ZERO_OK;
    const JoinArgs j{static_cast<const float*>(workspace), dweight, dbias, parts, dim, (uint32_t)grad_dtype, accumulate};
    return rows_status(launch_pdl(k_layernorm_join, dim3((2 * dim + 31) / 32), dim3(256), 0, stream, j));
}

}  // extern "C"
