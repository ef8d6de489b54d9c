/*
 * rows.cuh -- what the operators beside the matrix products share (layernorm.cu,
 * embedding.cu, head_loss.cu): a row of activations in chunks of 8 elements, its loads and
 * stores in 16 or 32 bits, and the host's checks.
 *
 * Two layouts of a row over the n threads that hold it.  VEC: chunk c is elements
 * [8c, 8c + 8), one or two 128-bit accesses; every row starts on a 16-byte boundary and is a
 * whole number of chunks.  Otherwise chunk c of thread k is the elements
 * (8 * (c / n) + j) * n + k, j < 8, so that each access of a warp is 32 neighbours, whatever
 * the row's alignment and length.
 */
#pragma once

#include "adamw_elem.cuh"
#include "reduce_elem.cuh"

#include <atomic>
#include <initializer_list>
#include <string.h>

namespace zero {
namespace {

template <zero_dtype_t DT>
struct Elem {
    using T = uint16_t;
    struct Raw {
        uint4 v;
    };
};
template <>
struct Elem<ZERO_F32> {
    using T = float;
    struct Raw {
        float4 a, b;
    };
};

template <zero_dtype_t DT>
__device__ __forceinline__ float to_f32(typename Elem<DT>::T x)
{
    if constexpr (DT == ZERO_F32)
        return x;
    else
        return one16<DT>(x);
}

/* A chunk as 4 pairs of neighbours, for the paired fp32 arithmetic. */
template <zero_dtype_t DT>
__device__ __forceinline__ void widen2(const typename Elem<DT>::Raw& r, uint64_t (&x)[4])
{
    if constexpr (DT == ZERO_F32) {
        x[0] = f2(r.a.x, r.a.y), x[1] = f2(r.a.z, r.a.w), x[2] = f2(r.b.x, r.b.y), x[3] = f2(r.b.z, r.b.w);
    } else {
        const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
            x[q] = f2(lo16<DT>(w[q]), hi16<DT>(w[q]));
    }
}

__device__ __forceinline__ void split4(const uint64_t (&p)[4], float (&x)[8])
{
#pragma unroll
    for (int q = 0; q < 4; ++q)
        f2_split(p[q], x[2 * q], x[2 * q + 1]);
}

__device__ __forceinline__ float f2_sum(uint64_t p)
{
    float a, b;
    f2_split(p, a, b);
    return __fadd_rn(a, b);
}

/* Rounded to nearest even: the one rounding of an operator's 16-bit output. */
template <zero_dtype_t DT>
__device__ __forceinline__ typename Elem<DT>::T from_f32(float x)
{
    if constexpr (DT == ZERO_F32)
        return x;
    else
        return pack1<DT == ZERO_F16>(x);
}

template <zero_dtype_t DT>
__device__ __forceinline__ void widen(const typename Elem<DT>::Raw& r, float (&x)[8])
{
    if constexpr (DT == ZERO_F32) {
        x[0] = r.a.x, x[1] = r.a.y, x[2] = r.a.z, x[3] = r.a.w;
        x[4] = r.b.x, x[5] = r.b.y, x[6] = r.b.z, x[7] = r.b.w;
    } else {
        x[0] = lo16<DT>(r.v.x), x[1] = hi16<DT>(r.v.x), x[2] = lo16<DT>(r.v.y), x[3] = hi16<DT>(r.v.y);
        x[4] = lo16<DT>(r.v.z), x[5] = hi16<DT>(r.v.z), x[6] = lo16<DT>(r.v.w), x[7] = hi16<DT>(r.v.w);
    }
}

template <zero_dtype_t DT>
__device__ __forceinline__ typename Elem<DT>::Raw narrow(const float (&x)[8])
{
    typename Elem<DT>::Raw r;
    if constexpr (DT == ZERO_F32) {
        r.a = make_float4(x[0], x[1], x[2], x[3]);
        r.b = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        constexpr bool h = DT == ZERO_F16;
        r.v = make_uint4(pack2<h>(x[0], x[1]), pack2<h>(x[2], x[3]), pack2<h>(x[4], x[5]), pack2<h>(x[6], x[7]));
    }
    return r;
}

/* Loads of what an earlier launch may have written: volatile keeps them behind
 * grid_dependency_wait(). */
__device__ __forceinline__ uint4 ld_v4(const void* p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

/* (A load through a volatile pointer would pass L1 by.) */
__device__ __forceinline__ uint16_t ld_one(const uint16_t* p)
{
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ float ld_one(const float* p)
{
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ float4 as_f4(const uint4& v)
{
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

/* The chunk of 8 elements that thread k of n holds in its place i; elements past d are 0. */
template <zero_dtype_t DT, bool VEC>
__device__ __forceinline__ typename Elem<DT>::Raw load_chunk(const typename Elem<DT>::T* row, uint32_t d, uint32_t i,
                                                             uint32_t k, uint32_t n)
{
    typename Elem<DT>::Raw r;
    if constexpr (VEC) {
        const uint32_t c = i * n + k;
        if (c * 8 < d) {
            if constexpr (DT == ZERO_F32) {
                r.a = as_f4(ld_v4(row + c * 8));
                r.b = as_f4(ld_v4(row + c * 8 + 4));
            } else {
                r.v = ld_v4(row + c * 8);
            }
        } else {
            r = {};
        }
    } else {
        typename Elem<DT>::T x[8];
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
            const uint32_t e = (i * 8 + j) * n + k;
            x[j] = e < d ? ld_one(row + e) : typename Elem<DT>::T(0);
        }
        if constexpr (DT == ZERO_F32) {
            r.a = make_float4(x[0], x[1], x[2], x[3]);
            r.b = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            r.v = make_uint4(x[0] | (uint32_t)x[1] << 16, x[2] | (uint32_t)x[3] << 16, x[4] | (uint32_t)x[5] << 16,
                             x[6] | (uint32_t)x[7] << 16);
        }
    }
    return r;
}

template <zero_dtype_t DT, bool VEC>
__device__ __forceinline__ void store_chunk(typename Elem<DT>::T* row, uint32_t d, uint32_t i, uint32_t k, uint32_t n,
                                            const float (&x)[8])
{
    if constexpr (VEC) {
        const uint32_t c = i * n + k;
        if (c * 8 >= d)
            return;
        const typename Elem<DT>::Raw r = narrow<DT>(x);
        if constexpr (DT == ZERO_F32) {
            *reinterpret_cast<float4*>(row + c * 8) = r.a;
            *reinterpret_cast<float4*>(row + c * 8 + 4) = r.b;
        } else {
            *reinterpret_cast<uint4*>(row + c * 8) = r.v;
        }
    } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) {
            const uint32_t e = (i * 8 + j) * n + k;
            if (e < d)
                row[e] = from_f32<DT>(x[j]);
        }
    }
}

/* Element j of the chunk in place i, as an index into the row. */
template <bool VEC>
__device__ __forceinline__ uint32_t elem_of(uint32_t i, uint32_t j, uint32_t k, uint32_t n)
{
    return VEC ? (i * n + k) * 8 + j : (i * 8 + j) * n + k;
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

/* ------------------------------------------------------------------------------------ */
/* host side                                                                              */
/* ------------------------------------------------------------------------------------ */

inline size_t dtype_size(zero_dtype_t t) { return t == ZERO_F32 ? 4 : 2; }
inline bool float_dtype(zero_dtype_t t) { return t == ZERO_F16 || t == ZERO_BF16 || t == ZERO_F32; }
inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

/* Whether rows of `dim` elements allow 128-bit accesses. */
inline bool rows_vec(const void* p, uint64_t stride, uint32_t dim, zero_dtype_t t)
{
    return aligned_to(p, 16) && stride * dtype_size(t) % 16 == 0 && dim % 8 == 0;
}

/* Bytes of an argument: rows of `width` bytes, each `stride` after the one before. */
struct Area {
    const void* p;
    uint64_t width, rows, stride;

    Area(const void* p_, uint64_t bytes) : p(p_), width(bytes), rows(1), stride(0) {}
    Area(const void* p_, uint64_t rows_, uint64_t stride_, uint64_t dim, zero_dtype_t t)
        : p(p_), width(rows_ ? dim * dtype_size(t) : 0), rows(rows_), stride(stride_ * dtype_size(t))
    {
    }
    uint64_t span() const { return rows ? (rows - 1) * stride + width : 0; }
};

inline bool clash(const Area& a, const Area& b)
{
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    if (!a.p || !b.p || !a.width || !b.width || x >= y + b.span() || y >= x + a.span())
        return false;
    if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {  // columns of one buffer, side by side
        const uint64_t at = y >= x ? (y - x) % a.stride : (a.stride - (x - y) % a.stride) % a.stride;  // of b in a's rows
        return at < a.width || at + b.width > a.stride;
    }
    return true;
}

/* No output overlaps an input or another output. */
inline bool apart(std::initializer_list<Area> out, std::initializer_list<Area> in)
{
    for (const Area* o = out.begin(); o != out.end(); ++o) {
        for (const Area& i : in)
            if (clash(*o, i))
                return false;
        for (const Area* q = out.begin(); q != o; ++q)
            if (clash(*o, *q))
                return false;
    }
    return true;
}

/* Lets a kernel take all of an SM's shared memory, once per kernel and device. */
template <auto KERNEL>
cudaError_t allow_smem()
{
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (e != cudaSuccess || (done.load(std::memory_order_relaxed) & bit))
        return e;
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, KERNEL);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448 - (int)at.sharedSizeBytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

/* Blocks of a kernel that fit on the current device at once; the last answer is kept. */
template <auto KERNEL>
cudaError_t resident(uint32_t threads, size_t smem, uint32_t& blocks)
{
    static std::atomic<uint64_t> last{0};  // device + 1, threads, 16-byte units of shared memory, blocks per SM
    int dev = 0, per_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t key = (uint64_t)(dev + 1) << 40 | (uint64_t)threads << 24 | (smem / 16) << 8;
    const uint64_t have = last.load(std::memory_order_relaxed);
    if (e == cudaSuccess && (have & ~255ull) == key) {
        per_sm = (int)(have & 255);
    } else if (e == cudaSuccess) {
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, KERNEL, (int)threads, smem);
        if (e == cudaSuccess)
            last.store(key | (uint64_t)per_sm, std::memory_order_relaxed);
    }
    blocks = (uint32_t)(sm_count() * (per_sm > 0 ? per_sm : 1));
    return e;
}

inline int rows_status(cudaError_t e)
{
    if (e == cudaSuccess)
        return ZERO_OK;
    record_cuda_error((int)e);
    return ZERO_ECUDA;
}

}  // namespace
}  // namespace zero
