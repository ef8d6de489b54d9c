/*
 * tensors.cu -- the step over lists of tensors: global gradient norm, AdamW with 32-bit
 * states, AdamW with 8-bit states, and the 8-bit states' values read and written.
 *
 * The tensors lie where the caller's model has them.  Each launch carries its part of the
 * list by value in the kernel's parameters (up to 32 KB of constant memory), so a call
 * needs no device table, nothing is kept from one call for the next, and a captured graph
 * holds the list it was captured with.  The list is cut into chunks; `begin[k]` counts the
 * chunks before tensor k, and a block finds the tensor of its chunk by binary search.
 *
 * A chunk is 2048 elements, 8 per thread: warp w holds the chunk's w-th block of 256, which
 * is the 8-bit states' block too.  Tensors whose arrays are all 16-byte aligned move in
 * 128-bit accesses of 8 consecutive elements per thread; others element by element, a
 * warp's lanes side by side.
 */
#include "adamw_elem.cuh"
#include "reduce_elem.cuh"
#include "state8.cuh"
#include "step_scalars.cuh"

#include <atomic>
#include <string.h>

namespace zero {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                              // elements per thread and chunk
constexpr uint32_t kTensorChunk = kThreads * kPer;   // 2048
constexpr uint32_t kBlk = ZERO_STATE8_BLOCK;
static_assert(kBlk == 32 * kPer, "a warp holds one block of the 8-bit states");

constexpr uint32_t kGradMask = 3;    // the gradient's zero_dtype_t
constexpr uint32_t kOutF16 = 4;      // 16-bit parameters are fp16
constexpr uint32_t kAligned = 8;     // every array allows 128-bit accesses
constexpr uint32_t kValueBF16 = 16;  // values read out as bf16

/* One tensor of a launch.  The codec keeps the 32-bit arrays in x and y. */
struct Ref {
    union {
        const void* grad;
        void* x;
    };
    union {
        float* master;
        void* y;
    };
    void* m;
    void* v;
    uint8_t* exps;
    uint16_t* params;
    uint64_t elems;
    float lr_scale, decay;
    uint32_t flags;
    uint32_t group0;  // groups of 8 elements of the list before this tensor (mod 2^32)
};

/* Tensors per launch: the parameters may be 32,764 bytes. */
constexpr int kCap = 384;

struct List {
    uint32_t n, n_chunks;
    uint32_t begin[kCap + 1];
    Ref t[kCap];
};

struct NormArgs {
    zero_step_state_t* st;
    double* slots;              // one partial sum per block
    zero_adamw_hparams_t hp;
    uint32_t slot0, last;       // this launch's first slot; 1 in the list's last launch
    List l;
};

struct TensorsArgs {
    const zero_step_state_t* st;
    uint64_t seed;
    float beta1, beta2, eps;
    List l;
};
static_assert(sizeof(NormArgs) <= 32764 && sizeof(TensorsArgs) <= 32764, "kernel parameters");

/* The tensor of chunk c: the last k with begin[k] <= c (empty tensors have no chunk). */
__device__ __forceinline__ uint32_t tensor_of(const List& l, uint32_t c)
{
    uint32_t lo = 0, hi = l.n;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (l.begin[mid] <= c)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ float one_grad(const void* g, uint64_t i, uint32_t dtype)
{
    if (dtype == ZERO_F32)
        return __ldcs(static_cast<const float*>(g) + i);
    const uint16_t b = ld_stream_u16(static_cast<const uint16_t*>(g) + i);
    return dtype == ZERO_F16 ? one16<ZERO_F16>(b) : one16<ZERO_BF16>(b);
}

__device__ __forceinline__ void load8(const float* p, float (&x)[8])
{
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ void store8(float* p, const float (&x)[8])
{
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

template <zero_dtype_t DT>
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8])
{
    x[0] = lo16<DT>(w.x), x[1] = hi16<DT>(w.x), x[2] = lo16<DT>(w.y), x[3] = hi16<DT>(w.y);
    x[4] = lo16<DT>(w.z), x[5] = hi16<DT>(w.z), x[6] = lo16<DT>(w.w), x[7] = hi16<DT>(w.w);
}

__device__ __forceinline__ void load_grad8(const void* g, uint64_t i, uint32_t dtype, float (&x)[8])
{
    if (dtype == ZERO_F32) {
        load8(static_cast<const float*>(g) + i, x);
        return;
    }
    const uint4 w = ld_stream_v4(static_cast<const uint16_t*>(g) + i);
    if (dtype == ZERO_F16)
        widen8<ZERO_F16>(w, x);
    else
        widen8<ZERO_BF16>(w, x);
}

__device__ __forceinline__ void store_params8(uint16_t* p, uint32_t f16, const float (&x)[8])
{
    uint4 o;
    if (f16)
        o = make_uint4(pack2<true>(x[0], x[1]), pack2<true>(x[2], x[3]), pack2<true>(x[4], x[5]),
                       pack2<true>(x[6], x[7]));
    else
        o = make_uint4(pack2<false>(x[0], x[1]), pack2<false>(x[2], x[3]), pack2<false>(x[4], x[5]),
                       pack2<false>(x[6], x[7]));
    __stcs(reinterpret_cast<uint4*>(p), o);
}

__device__ __forceinline__ Scalars step_scalars(const TensorsArgs& a)
{
    Scalars s;
    s.c = a.st->clip_coef;
    s.step = a.st->step_size;
    s.rbc2 = a.st->rbc2;
    s.decay = 1.0f;
    s.b1 = a.beta1;
    s.b2 = a.beta2;
    s.omb1 = __fsub_rn(1.0f, a.beta1);
    s.omb2 = __fsub_rn(1.0f, a.beta2);
    s.eps = a.eps;
    return s;
}

/* ------------------------------------------------------------------------------------ */
/* gradient norm                                                                          */
/* ------------------------------------------------------------------------------------ */

constexpr int kNormGroups = 4;                               // groups of 8 per thread in flight
constexpr uint32_t kNormChunk = kTensorChunk * kNormGroups;  // 8192 elements
constexpr uint32_t kNormMaxBlocks = 2048;                    // slots per launch

/* A thread's sum of squares: fp32 sums of 8 squares, joined by error-free additions
 * (hi + lo), so that only a group's own 8 roundings remain; groups whose sum leaves fp32's
 * safe range (below 2^-80 or above 2^120: an infinity, a NaN, or a square that would
 * overflow or vanish) are summed in fp64 instead. */
struct Squares {
    float hi = 0.0f, lo = 0.0f;
    double wide = 0.0;
    bool bad = false;

    __device__ __forceinline__ void add(const float (&x)[8], float inv)
    {
        float s0 = __fmul_rn(x[0], x[0]), s1 = __fmul_rn(x[1], x[1]);
#pragma unroll
        for (int e = 2; e < 8; e += 2) {
            s0 = __fmaf_rn(x[e], x[e], s0);
            s1 = __fmaf_rn(x[e + 1], x[e + 1], s1);
        }
        const float s = __fadd_rn(s0, s1);
        if (s < 0x1p120f && s > 0x1p-80f && inv < 0x1p60f) {
            const float t = __fadd_rn(hi, s);
            const float bb = __fsub_rn(t, hi);
            lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, bb)), __fsub_rn(s, bb)));
            hi = t;
        } else {
            wide += sumsq_wide(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], 0xffu);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                bad |= not_finite(__fmul_rn(x[e], inv));
        }
    }
};

/* Adds v over the block: a fixed shuffle tree per warp, the warps in order.  Valid in
 * thread 0. */
__device__ __forceinline__ double block_sum(double v, double* warp_sum)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0)
        warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kThreads / 32; ++w)
            t += warp_sum[w];
    return t;
}

/* Sum of squares over the list's gradients; in the last launch the block that finishes
 * last adds the blocks' partial sums in order and finalises the step as zero_grad_norm. */
__global__ void __launch_bounds__(kThreads) k_tensors_norm(const __grid_constant__ NormArgs a)
{
    __shared__ double warp_sum[kThreads / 32];
    __shared__ int is_last;
    grid_dependency_wait();
    zero_step_state_t* st = a.st;
    const float inv = st->inv_scale;
    Squares acc;
    for (uint32_t c = blockIdx.x; c < a.l.n_chunks; c += gridDim.x) {
        const uint32_t k = tensor_of(a.l, c);
        const Ref& t = a.l.t[k];
        const uint32_t dtype = t.flags & kGradMask;
        const uint64_t off = (uint64_t)(c - a.l.begin[k]) * kNormChunk;
        if ((t.flags & kAligned) && off + kNormChunk <= t.elems) {
            float x[kNormGroups][8];
#pragma unroll
            for (int q = 0; q < kNormGroups; ++q)
                load_grad8(t.grad, off + q * kTensorChunk + threadIdx.x * kPer, dtype, x[q]);
#pragma unroll
            for (int q = 0; q < kNormGroups; ++q)
                acc.add(x[q], inv);
        } else {
#pragma unroll 1
            for (int q = 0; q < kNormGroups; ++q) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint64_t i = off + (q * 8 + e) * kThreads + threadIdx.x;
                    x[e] = i < t.elems ? one_grad(t.grad, i, dtype) : 0.0f;
                }
                acc.add(x, inv);
            }
        }
    }
    if (__any_sync(0xffffffffu, acc.bad) && (threadIdx.x & 31) == 0)
        atomicOr(&st->overflow, 1u);
    const double part = block_sum((double)acc.hi + (double)acc.lo + acc.wide, warp_sum);
    if (threadIdx.x == 0)
        a.slots[a.slot0 + blockIdx.x] = part;
    if (!a.last)
        return;
    // arrival, as in the norm over the flat buffer: the block's writes are ordered before
    // the count by the barrier and one fence of thread 0
    __syncthreads();
    if (threadIdx.x == 0) {
        asm volatile("fence.acq_rel.gpu;" ::: "memory");
        is_last = atomicAdd(&st->arrivals, 1u) == gridDim.x - 1;
        if (is_last)
            asm volatile("fence.acq_rel.gpu;" ::: "memory");
    }
    __syncthreads();
    if (!is_last)
        return;
    const uint32_t n_slots = a.slot0 + gridDim.x;
    double v = 0.0;
    for (uint32_t i = threadIdx.x; i < n_slots; i += kThreads)
        v += __ldcg(a.slots + i);
    const double total = block_sum(v, warp_sum) * ((double)inv * (double)inv);
    const uint32_t overflow = __ldcg(&st->overflow) != 0, next = st->t + 1;
    __syncthreads();  // every thread has read t and the overflow flag
    if (threadIdx.x == 32 && !overflow)
        st->step_size = bias_step_size(a.hp, next);
    if (threadIdx.x == 64 && !overflow)
        st->rbc2 = bias_rbc2(a.hp, next);
    if (threadIdx.x == 96)
        scaler_update(st, a.hp, st->n_ranks, overflow, next);
    if (threadIdx.x == 0) {
        const double norm = sqrt(total);
        const float clip = clip_coefficient(norm, overflow, a.hp.max_grad_norm);
        st->arrivals = 0;
        st->sumsq = total;
        st->norm = norm;
        st->clip_coef = clip;
        st->applied_c = overflow ? -1.0f : clip;
        st->overflow = 0;
        st->n_steps += 1;
    }
}

/* ------------------------------------------------------------------------------------ */
/* AdamW                                                                                  */
/* ------------------------------------------------------------------------------------ */

__global__ void __launch_bounds__(kThreads) k_tensors_adamw(const __grid_constant__ TensorsArgs a)
{
    grid_dependency_wait();
    if (a.st->skip)
        return;
    Scalars s = step_scalars(a);
    const float inv = a.st->inv_scale_used, step = s.step;
    for (uint32_t c = blockIdx.x; c < a.l.n_chunks; c += gridDim.x) {
        const uint32_t k = tensor_of(a.l, c);
        const Ref& t = a.l.t[k];
        const uint32_t dtype = t.flags & kGradMask;
        float* m = static_cast<float*>(t.m);
        float* v = static_cast<float*>(t.v);
        s.step = __fmul_rn(step, t.lr_scale);
        s.decay = t.decay;
        const uint64_t off = (uint64_t)(c - a.l.begin[k]) * kTensorChunk;
        if ((t.flags & kAligned) && off + kTensorChunk <= t.elems) {
            const uint64_t i = off + threadIdx.x * kPer;
            float x8[8], p8[8], m8[8], v8[8];
            load_grad8(t.grad, i, dtype, x8);
            load8(t.master + i, p8);
            load8(m + i, m8);
            load8(v + i, v8);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                adamw_one(__fmul_rn(x8[e], inv), p8[e], m8[e], v8[e], s);
            store8(t.master + i, p8);
            store8(m + i, m8);
            store8(v + i, v8);
            if (t.params)
                store_params8(t.params + i, t.flags & kOutF16, p8);
        } else {
#pragma unroll 4
            for (int e = 0; e < kPer; ++e) {
                const uint64_t i = off + e * kThreads + threadIdx.x;
                if (i < t.elems) {
                    float p = t.master[i], mi = m[i], vi = v[i];
                    adamw_one(__fmul_rn(one_grad(t.grad, i, dtype), inv), p, mi, vi, s);
                    t.master[i] = p;
                    m[i] = mi;
                    v[i] = vi;
                    if (t.params)
                        t.params[i] = (t.flags & kOutF16) ? pack1<true>(p) : pack1<false>(p);
                }
            }
        }
    }
}

/* A lane's 8 codes of a block. */
struct Codes {
    uint32_t c[8];

    __device__ __forceinline__ void unpack(uint2 w)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            c[e] = w.x >> (8 * e) & 0xffu;
            c[4 + e] = w.y >> (8 * e) & 0xffu;
        }
    }
    __device__ __forceinline__ uint2 pack() const
    {
        return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                          c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
    }
};

/* The AdamW element update with this form's denominator: one multiplication by 1/rbc2,
 * rounded once per step, in place of a division per element. */
__device__ __forceinline__ void moments(float gc, float& m, float& v, const Scalars& s)
{
    m = __fadd_rn(__fmul_rn(s.b1, m), __fmul_rn(s.omb1, gc));
    v = __fadd_rn(__fmul_rn(s.b2, v), __fmul_rn(s.omb2, __fmul_rn(gc, gc)));
}

__device__ __forceinline__ float updated(float p, float m, float v, float inv_rbc2, const Scalars& s)
{
    const float denom = __fadd_rn(__fmul_rn(__fsqrt_rn(v), inv_rbc2), s.eps);
    return __fsub_rn(__fmul_rn(p, s.decay), __fmul_rn(s.step, __fdiv_rn(m, denom)));
}

__global__ void __launch_bounds__(kThreads) k_tensors_adamw8(const __grid_constant__ TensorsArgs a)
{
    grid_dependency_wait();
    if (a.st->skip)
        return;
    Scalars s = step_scalars(a);
    const float inv = a.st->inv_scale_used, step = s.step, inv_rbc2 = __fdiv_rn(1.0f, s.rbc2);
    const uint32_t key = step_key(a.seed, a.st->t);
    const uint32_t lane = threadIdx.x & 31;
    // the generator's outputs for this lane's elements where lanes lie side by side
    Jump jm = jump(1), jv = jump(9);
    for (uint32_t q = 0; q < (lane & 7); ++q) {
        jm.add = jm.add * kLcgMul + kLcgAdd, jm.mul *= kLcgMul;
        jv.add = jv.add * kLcgMul + kLcgAdd, jv.mul *= kLcgMul;
    }
    for (uint32_t c = blockIdx.x; c < a.l.n_chunks; c += gridDim.x) {
        const uint32_t k = tensor_of(a.l, c);
        const Ref& t = a.l.t[k];
        const uint32_t dtype = t.flags & kGradMask;
        uint8_t* m = static_cast<uint8_t*>(t.m);
        uint8_t* v = static_cast<uint8_t*>(t.v);
        s.step = __fmul_rn(step, t.lr_scale);
        s.decay = t.decay;
        const uint64_t blk = (uint64_t)(c - a.l.begin[k]) * (kTensorChunk / kBlk) + (threadIdx.x >> 5);
        const uint64_t off = blk * kBlk;
        if (off >= t.elems)
            continue;  // a whole warp past the tensor's last block
        const bool vec = (t.flags & kAligned) && off + kBlk <= t.elems;
        // element e of this lane: consecutive in 128-bit accesses, else lanes side by side
        const uint64_t i0 = vec ? off + lane * kPer : off + lane;
        const uint64_t left = i0 < t.elems ? t.elems - i0 : 0;
        float x8[8], p8[8], m8[8], v8[8];
        Codes cm, cv;
        if (vec) {
            load_grad8(t.grad, i0, dtype, x8);
            load8(t.master + i0, p8);
            cm.unpack(__ldcs(reinterpret_cast<const uint2*>(m + i0)));
            cv.unpack(__ldcs(reinterpret_cast<const uint2*>(v + i0)));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = e * 32u < left;
                x8[e] = in ? one_grad(t.grad, i0 + e * 32, dtype) : 0.0f;
                p8[e] = in ? t.master[i0 + e * 32] : 0.0f;
                cm.c[e] = in ? m[i0 + e * 32] : 0u;
                cv.c[e] = in ? v[i0 + e * 32] : 0u;
            }
        }
        const float scale_m = exp_scale(t.exps[2 * blk]), scale_v = exp_scale(t.exps[2 * blk + 1]);
        uint32_t top_m = 0, top_v = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            m8[e] = decode_m(cm.c[e], scale_m);
            v8[e] = decode_v(cv.c[e], scale_v);
            moments(__fmul_rn(s.c, __fmul_rn(x8[e], inv)), m8[e], v8[e], s);
            p8[e] = updated(p8[e], m8[e], v8[e], inv_rbc2, s);
            top_m = max(top_m, __float_as_uint(m8[e]) & 0x7fffffffu);
            top_v = max(top_v, __float_as_uint(v8[e]) & 0x7fffffffu);
        }
        const uint32_t bm = block_exponent(__reduce_max_sync(0xffffffffu, top_m));
        const uint32_t bv = block_exponent(__reduce_max_sync(0xffffffffu, top_v));
        const float unscale_m = exp_unscale(bm), unscale_v = exp_unscale(bv);
        const uint32_t group = t.group0 + (uint32_t)blk * 32;
        if (vec) {
            const uint32_t s0 = mix32(key + (group + lane) * kGolden);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const Jump a1 = jump(e + 1), a9 = jump(e + 9);
                cm.c[e] = encode_m(m8[e], unscale_m, (s0 * a1.mul + a1.add) >> 12);
                cv.c[e] = encode_v(v8[e], unscale_v, (s0 * a9.mul + a9.add) >> 12);
            }
            store8(t.master + i0, p8);
            if (t.params)
                store_params8(t.params + i0, t.flags & kOutF16, p8);
            __stcs(reinterpret_cast<uint2*>(m + i0), cm.pack());
            __stcs(reinterpret_cast<uint2*>(v + i0), cv.pack());
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t s0 = mix32(key + (group + e * 4 + (lane >> 3)) * kGolden);
                if (e * 32u < left) {
                    const uint64_t i = i0 + e * 32;
                    m[i] = (uint8_t)encode_m(m8[e], unscale_m, (s0 * jm.mul + jm.add) >> 12);
                    v[i] = (uint8_t)encode_v(v8[e], unscale_v, (s0 * jv.mul + jv.add) >> 12);
                    t.master[i] = p8[e];
                    if (t.params)
                        t.params[i] = (t.flags & kOutF16) ? pack1<true>(p8[e]) : pack1<false>(p8[e]);
                }
            }
        }
        if (lane == 0) {
            t.exps[2 * blk] = (uint8_t)bm;
            t.exps[2 * blk + 1] = (uint8_t)bv;
        }
    }
}

/* ------------------------------------------------------------------------------------ */
/* 8-bit states to values and back                                                        */
/* ------------------------------------------------------------------------------------ */

template <bool WRITE>
__global__ void __launch_bounds__(kThreads) k_tensors_state8(const __grid_constant__ List l)
{
    grid_dependency_wait();
    const uint32_t lane = threadIdx.x & 31;
    for (uint32_t c = blockIdx.x; c < l.n_chunks; c += gridDim.x) {
        const uint32_t k = tensor_of(l, c);
        const Ref& t = l.t[k];
        uint8_t* m = static_cast<uint8_t*>(t.m);
        uint8_t* v = static_cast<uint8_t*>(t.v);
        const uint64_t blk = (uint64_t)(c - l.begin[k]) * (kTensorChunk / kBlk) + (threadIdx.x >> 5);
        const uint64_t off = blk * kBlk;
        if (off >= t.elems)
            continue;
        const bool vec = (t.flags & kAligned) && off + kBlk <= t.elems;
        const uint64_t i0 = vec ? off + lane * kPer : off + lane;
        const uint64_t left = i0 < t.elems ? t.elems - i0 : 0;
        float m8[8], v8[8];
        Codes cm, cv;
        if (WRITE) {
            const float* xm = static_cast<const float*>(t.x);
            const float* xv = static_cast<const float*>(t.y);
            if (vec) {
                load8(xm + i0, m8);
                load8(xv + i0, v8);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    m8[e] = e * 32u < left ? xm[i0 + e * 32] : 0.0f;
                    v8[e] = e * 32u < left ? xv[i0 + e * 32] : 0.0f;
                }
            }
            uint32_t top_m = 0, top_v = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                top_m = max(top_m, __float_as_uint(m8[e]) & 0x7fffffffu);
                top_v = max(top_v, __float_as_uint(v8[e]) & 0x7fffffffu);
            }
            const uint32_t bm = block_exponent(__reduce_max_sync(0xffffffffu, top_m));
            const uint32_t bv = block_exponent(__reduce_max_sync(0xffffffffu, top_v));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                cm.c[e] = encode_m(m8[e], exp_unscale(bm), kNearest);
                cv.c[e] = encode_v(v8[e], exp_unscale(bv), kNearest);
            }
            if (vec) {
                __stcs(reinterpret_cast<uint2*>(m + i0), cm.pack());
                __stcs(reinterpret_cast<uint2*>(v + i0), cv.pack());
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e * 32u < left) {
                        m[i0 + e * 32] = (uint8_t)cm.c[e];
                        v[i0 + e * 32] = (uint8_t)cv.c[e];
                    }
            }
            if (lane == 0) {
                t.exps[2 * blk] = (uint8_t)bm;
                t.exps[2 * blk + 1] = (uint8_t)bv;
            }
        } else {
            if (vec) {
                cm.unpack(__ldcs(reinterpret_cast<const uint2*>(m + i0)));
                cv.unpack(__ldcs(reinterpret_cast<const uint2*>(v + i0)));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    cm.c[e] = e * 32u < left ? m[i0 + e * 32] : 0u;
                    cv.c[e] = e * 32u < left ? v[i0 + e * 32] : 0u;
                }
            }
            const float scale_m = exp_scale(t.exps[2 * blk]), scale_v = exp_scale(t.exps[2 * blk + 1]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                m8[e] = decode_m(cm.c[e], scale_m);
                v8[e] = decode_v(cv.c[e], scale_v);
            }
            const bool bf16 = t.flags & kValueBF16;
            if (vec && bf16) {
                store_params8(static_cast<uint16_t*>(t.x) + i0, 0, m8);
                store_params8(static_cast<uint16_t*>(t.y) + i0, 0, v8);
            } else if (vec) {
                store8(static_cast<float*>(t.x) + i0, m8);
                store8(static_cast<float*>(t.y) + i0, v8);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e * 32u < left) {
                        const uint64_t i = i0 + e * 32;
                        if (bf16) {
                            static_cast<uint16_t*>(t.x)[i] = pack1<false>(m8[e]);
                            static_cast<uint16_t*>(t.y)[i] = pack1<false>(v8[e]);
                        } else {
                            static_cast<float*>(t.x)[i] = m8[e];
                            static_cast<float*>(t.y)[i] = v8[e];
                        }
                    }
            }
        }
    }
}

/* ------------------------------------------------------------------------------------ */
/* host side                                                                              */
/* ------------------------------------------------------------------------------------ */

enum class Op { kNorm, kAdamw, kAdamw8, kRead, kWrite };

bool finite_f(float x) { return x == x && x <= 3.4e38f && x >= -3.4e38f; }

bool at(const void* p, uintptr_t align) { return ((uintptr_t)p & (align - 1)) == 0; }

/* What an operator needs of tensor t (and, for the codec, of its 32-bit partner). */
int check_tensor(const zero_tensor_t& t, const zero_tensor_t* other, Op op)
{
    if (t.elems == 0)
        return other && other->elems != 0 ? ZERO_EINVAL : ZERO_OK;
    if (t.elems > (1ull << 42))
        return ZERO_EINVAL;
    const bool codec = op == Op::kRead || op == Op::kWrite;
    const bool adamw = op == Op::kAdamw || op == Op::kAdamw8;
    if (!codec) {
        if (!t.grad || (t.grad_dtype != ZERO_F16 && t.grad_dtype != ZERO_BF16 && t.grad_dtype != ZERO_F32))
            return ZERO_EINVAL;
        if (!at(t.grad, t.grad_dtype == ZERO_F32 ? 4 : 2))
            return ZERO_EALIGN;
    }
    if (adamw) {
        if (!t.master || !t.m || !t.v)
            return ZERO_EINVAL;
        if (t.params_dtype != 0 && t.params_dtype != ZERO_BF16 && t.params_dtype != ZERO_F16)
            return ZERO_EINVAL;
        if (!finite_f(t.lr_scale) || t.lr_scale < 0.0f || !finite_f(t.weight_decay))
            return ZERO_EINVAL;
        if (!at(t.master, 4) || !at(t.params, 2))
            return ZERO_EALIGN;
    }
    if (op == Op::kAdamw) {
        if (t.state_dtype != ZERO_F32)
            return ZERO_EINVAL;
        if (!at(t.m, 4) || !at(t.v, 4))
            return ZERO_EALIGN;
    }
    if (op == Op::kAdamw8 || codec)
        if (t.state_dtype != ZERO_U8 || !t.m || !t.v || !t.exps)
            return ZERO_EINVAL;
    if (codec) {
        const bool bf16 = op == Op::kRead && other->state_dtype == ZERO_BF16;
        if (other->elems != t.elems || !other->m || !other->v || (other->state_dtype != ZERO_F32 && !bf16))
            return ZERO_EINVAL;
        if (!at(other->m, bf16 ? 2 : 4) || !at(other->v, bf16 ? 2 : 4))
            return ZERO_EALIGN;
    }
    return ZERO_OK;
}

/* Every array of the operator allows 128-bit accesses of 8 elements. */
bool vector_ok(const zero_tensor_t& t, const zero_tensor_t* other, Op op)
{
    switch (op) {
    case Op::kNorm: return at(t.grad, 16);
    case Op::kAdamw:
        return at(t.grad, 16) && at(t.master, 16) && at(t.m, 16) && at(t.v, 16) && at(t.params, 16);
    case Op::kAdamw8:
        return at(t.grad, 16) && at(t.master, 16) && at(t.m, 8) && at(t.v, 8) && at(t.params, 16);
    default: return at(t.m, 8) && at(t.v, 8) && at(other->m, 16) && at(other->v, 16);
    }
}

/* Fills `l` with tensors from index `next` on, as many as fit; returns the next index. */
uint64_t fill(List& l, const zero_tensor_t* tensors, const zero_tensor_t* others, uint64_t n,
              uint64_t next, Op op, const zero_adamw_hparams_t* hp, uint32_t& group0)
{
    const uint64_t chunk = op == Op::kNorm ? kNormChunk : kTensorChunk;
    uint64_t chunks = 0;
    l.n = 0;
    l.begin[0] = 0;
    for (; next < n && l.n < (uint32_t)kCap; ++next) {
        const zero_tensor_t& t = tensors[next];
        const zero_tensor_t* other = others ? others + next : nullptr;
        if (t.elems == 0)
            continue;
        const uint64_t c = (t.elems + chunk - 1) / chunk;
        if (chunks + c > 0xffffffffull - (1u << 20))
            break;  // chunk counters are 32-bit; check_tensor bounds one tensor's chunks
        Ref& r = l.t[l.n];
        memset(&r, 0, sizeof r);
        r.elems = t.elems;
        r.m = t.m;
        r.v = t.v;
        r.exps = t.exps;
        if (other) {
            r.x = other->m;
            r.y = other->v;
            if (other->state_dtype == ZERO_BF16)
                r.flags |= kValueBF16;
        } else {
            r.grad = t.grad;
            r.master = t.master;
            r.params = t.params;
            r.flags |= t.grad_dtype;
        }
        if (hp) {
            r.lr_scale = t.lr_scale;
            r.decay = (float)(1.0 - (double)hp->lr * (double)t.lr_scale * (double)t.weight_decay);
            if ((t.params_dtype ? t.params_dtype : hp->params_dtype) == ZERO_F16)
                r.flags |= kOutF16;
        }
        if (vector_ok(t, other, op))
            r.flags |= kAligned;
        r.group0 = group0;
        group0 += (uint32_t)((t.elems + kBlk - 1) / kBlk) * 32u;
        chunks += c;
        l.begin[++l.n] = (uint32_t)chunks;
    }
    l.n_chunks = (uint32_t)chunks;
    return next;
}

int check_list(const zero_tensor_t* tensors, const zero_tensor_t* others, uint64_t n, Op op)
{
    const bool codec = op == Op::kRead || op == Op::kWrite;
    if (n > (1ull << 31) || (n && (!tensors || (codec && !others))))
        return ZERO_EINVAL;
    int align = ZERO_OK;
    for (uint64_t k = 0; k < n; ++k) {
        const int rc = check_tensor(tensors[k], codec ? others + k : nullptr, op);
        if (rc == ZERO_EINVAL)
            return rc;
        if (rc != ZERO_OK)
            align = rc;
    }
    return align;
}

template <typename K>
unsigned blocks_for(K kernel, uint64_t chunks, std::atomic<int> (&per_sm)[64])
{
    int dev = 0;
    cudaGetDevice(&dev);
    int occ = per_sm[dev & 63].load(std::memory_order_relaxed);
    if (occ == 0) {
        int o = 0;
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, kernel, kThreads, 0);
        occ = o > 0 ? o : 1;
        per_sm[dev & 63].store(occ, std::memory_order_relaxed);
    }
    const uint64_t cap = (uint64_t)sm_count() * (uint64_t)occ;
    return (unsigned)(chunks < cap ? chunks : cap);
}

int status_of(cudaError_t e)
{
    if (e == cudaSuccess)
        return ZERO_OK;
    record_cuda_error((int)e);
    return ZERO_ECUDA;
}

int run_adamw(const zero_tensor_t* tensors, uint64_t n, const zero_adamw_hparams_t* hp, uint64_t seed,
              const zero_step_state_t* st, cudaStream_t s, Op op)
{
    static std::atomic<int> occ[64], occ8[64];
    TensorsArgs a;
    a.st = st;
    a.seed = seed;
    a.beta1 = hp->beta1;
    a.beta2 = hp->beta2;
    a.eps = hp->eps;
    uint32_t group0 = 0;
    for (uint64_t next = 0; next < n;) {
        next = fill(a.l, tensors, nullptr, n, next, op, hp, group0);
        if (a.l.n_chunks == 0)
            continue;
        const auto kernel = op == Op::kAdamw ? k_tensors_adamw : k_tensors_adamw8;
        const unsigned grid = blocks_for(kernel, a.l.n_chunks, op == Op::kAdamw ? occ : occ8);
        const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, s, a);
        if (e != cudaSuccess)
            return status_of(e);
    }
    return ZERO_OK;
}

int run_codec(const zero_tensor_t* t8, const zero_tensor_t* t32, uint64_t n, cudaStream_t s, Op op)
{
    static std::atomic<int> occ_r[64], occ_w[64];
    List l;
    uint32_t group0 = 0;
    for (uint64_t next = 0; next < n;) {
        next = fill(l, t8, t32, n, next, op, nullptr, group0);
        if (l.n_chunks == 0)
            continue;
        const auto kernel = op == Op::kRead ? k_tensors_state8<false> : k_tensors_state8<true>;
        const unsigned grid = blocks_for(kernel, l.n_chunks, op == Op::kRead ? occ_r : occ_w);
        const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kThreads), 0, s, l);
        if (e != cudaSuccess)
            return status_of(e);
    }
    return ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" size_t zero_tensors_workspace_bytes(uint64_t n_tensors)
{
    const uint64_t launches = n_tensors / kCap + 1;
    return (size_t)(launches * kNormMaxBlocks * sizeof(double));
}

extern "C" int zero_tensors_state_init(uint32_t n_ranks, float loss_scale, uint32_t dynamic,
                                       uint32_t growth_interval, zero_step_state_t* st,
                                       zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_state_init");
    if (n_ranks == 0 || !st || !(loss_scale > 0.0f) || loss_scale > 3.0e38f)
        return ZERO_EINVAL;
    if (!at(st, 16))
        return ZERO_EALIGN;
    InitArgs a;
    a.st = st;
    a.partials = nullptr;
    a.n_tiles = 0;
    a.loss_scale = loss_scale;
    a.dynamic = dynamic ? 1u : 0u;
    a.growth_interval = growth_interval;
    a.n_ranks = n_ranks;
    return status_of(launch_state_init(a, (cudaStream_t)stream));
}

extern "C" int zero_tensors_grad_norm(const zero_tensor_t* tensors, uint64_t n_tensors,
                                      const zero_adamw_hparams_t* hp, double* workspace,
                                      zero_step_state_t* st, zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_grad_norm");
    const int rc = check_list(tensors, nullptr, n_tensors, Op::kNorm);
    if (rc == ZERO_EINVAL || !hparams_ok(hp) || !workspace || !st)
        return ZERO_EINVAL;
    if (rc != ZERO_OK || !at(workspace, 16) || !at(st, 16))
        return ZERO_EALIGN;
    static std::atomic<int> occ[64];
    NormArgs a;
    a.st = st;
    a.slots = workspace;
    a.hp = *hp;
    a.slot0 = 0;
    uint32_t group0 = 0;
    uint64_t next = 0;
    do {
        next = fill(a.l, tensors, nullptr, n_tensors, next, Op::kNorm, nullptr, group0);
        a.last = next == n_tensors;
        unsigned grid = blocks_for(k_tensors_norm, a.l.n_chunks, occ);
        grid = grid < 1 ? 1 : grid > kNormMaxBlocks ? kNormMaxBlocks : grid;
        const cudaError_t e = launch_pdl(k_tensors_norm, dim3(grid), dim3(kThreads), 0,
                                         (cudaStream_t)stream, a);
        if (e != cudaSuccess)
            return status_of(e);
        a.slot0 += grid;
    } while (next < n_tensors);
    return ZERO_OK;
}

extern "C" int zero_tensors_adamw(const zero_tensor_t* tensors, uint64_t n_tensors,
                                  const zero_adamw_hparams_t* hp, const zero_step_state_t* st,
                                  zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_adamw");
    const int rc = check_list(tensors, nullptr, n_tensors, Op::kAdamw);
    if (rc == ZERO_EINVAL || !hparams_ok(hp) || !st)
        return ZERO_EINVAL;
    if (rc != ZERO_OK || !at(st, 16))
        return ZERO_EALIGN;
    return run_adamw(tensors, n_tensors, hp, 0, st, (cudaStream_t)stream, Op::kAdamw);
}

extern "C" int zero_tensors_adamw8(const zero_tensor_t* tensors, uint64_t n_tensors,
                                   const zero_adamw_hparams_t* hp, uint64_t seed,
                                   const zero_step_state_t* st, zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_adamw8");
    const int rc = check_list(tensors, nullptr, n_tensors, Op::kAdamw8);
    if (rc == ZERO_EINVAL || !hparams_ok(hp) || !st)
        return ZERO_EINVAL;
    if (rc != ZERO_OK || !at(st, 16))
        return ZERO_EALIGN;
    return run_adamw(tensors, n_tensors, hp, seed, st, (cudaStream_t)stream, Op::kAdamw8);
}

extern "C" int zero_tensors_state8_read(const zero_tensor_t* from, const zero_tensor_t* to,
                                        uint64_t n_tensors, zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_state8_read");
    const int rc = check_list(from, to, n_tensors, Op::kRead);
    return rc != ZERO_OK ? rc : run_codec(from, to, n_tensors, (cudaStream_t)stream, Op::kRead);
}

extern "C" int zero_tensors_state8_write(const zero_tensor_t* to, const zero_tensor_t* from,
                                         uint64_t n_tensors, zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_state8_write");
    const int rc = check_list(to, from, n_tensors, Op::kWrite);
    return rc != ZERO_OK ? rc : run_codec(to, from, n_tensors, (cudaStream_t)stream, Op::kWrite);
}
