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

enum class Op { kNorm, kAdamw, kAdamw8, kRead, kWrite };

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 8;                              // elements per lane and unit
constexpr uint32_t kUnit = ZERO_STATE8_BLOCK;        // elements a warp takes at a time
static_assert(kUnit == 32 * kPer, "a warp holds one block of the 8-bit states");

constexpr uint32_t kGradMask = 3;    // the gradient's zero_dtype_t
constexpr uint32_t kOutF16 = 4;      // 16-bit parameters are fp16
constexpr uint32_t kVector = 8;      // every array allows 128-bit accesses (past `head` elements)
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
    union {
        uint32_t group0;  // 8-bit states: groups of 8 elements of the list before this tensor
        uint32_t head;    // 32-bit states: elements before the arrays' first 16-byte boundary
    };
};

/* A launch's part of the list.  Kernel parameters may be 32,764 bytes; short lists take the
 * small form, whose launch costs the host less (measured: 16 tensors, 8.4 us a call with
 * the large form, see kSmall's callers). */
constexpr int kSmall = 32, kLarge = 424;

template <int CAP>
struct List {
    uint32_t n, n_units;
    alignas(16) uint32_t end[CAP];  // units up to and including each tensor's, then ~0
    Ref t[CAP];
};

template <int CAP>
struct ListArgs {
    const zero_step_state_t* st;
    uint64_t seed;
    float beta1, beta2, eps;
    List<CAP> l;
};
static_assert(sizeof(ListArgs<kLarge>) <= 32764, "kernel parameters");

/* The tensor of unit u, by the whole warp: one count of the ends at or below u, its loads
 * all in flight at once.  They go through global addressing of the parameters: a binary
 * search in constant memory misses its cache once per step on a launch's first unit. */
template <int CAP>
__device__ __forceinline__ uint32_t find_unit(const List<CAP>& l, uint32_t u)
{
    const uint4* end = reinterpret_cast<const uint4*>(l.end);
    asm volatile("" : "+l"(end));
    const uint32_t lane = threadIdx.x & 31, n = l.n;
    uint32_t below = 0;
#pragma unroll
    for (uint32_t j = 0; j < (uint32_t)CAP; j += 128) {
        if (j + lane * 4 < n) {
            const uint4 e = end[j / 4 + lane];
            below += (e.x <= u) + (e.y <= u) + (e.z <= u) + (e.w <= u);
        }
    }
    return __reduce_add_sync(0xffffffffu, below);
}

/* Where a warp's unit lies: its tensor and the unit's number in it. */
struct Place {
    uint32_t k, begin, end;  // the tensor, and the units [begin, end) it holds
    uint32_t unit;           // the unit's number in the tensor
};

template <int CAP>
__device__ __forceinline__ void locate(const List<CAP>& l, uint32_t u, Place& p)
{
    if (u < p.begin || u >= p.end) {
        p.k = find_unit(l, u);
        p.begin = p.k ? l.end[p.k - 1] : 0;
        p.end = l.end[p.k];
    }
    p.unit = u - p.begin;
}

__device__ __forceinline__ float one_grad(const void* g, uint64_t i, uint32_t dtype)
{
    if (dtype == ZERO_F32)
        return __ldcs(static_cast<const float*>(g) + i);
    const uint16_t b = ld_stream_u16(static_cast<const uint16_t*>(g) + i);
    return dtype == ZERO_F16 ? one16<ZERO_F16>(b) : one16<ZERO_BF16>(b);
}

/* 8 consecutive floats in one 256-bit access (32-byte aligned): with two of 128 bits each
 * would touch every 32-byte sector of the warp's kilobyte and write it half. */
__device__ __forceinline__ void load8(const float* p, float (&x)[8])
{
    asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7])
                 : "l"(p));
}

__device__ __forceinline__ void store8(float* p, const float (&x)[8])
{
    asm volatile("st.global.L1::no_allocate.L2::evict_first.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}

template <zero_dtype_t DT>
__device__ __forceinline__ void widen8(const uint4& w, float (&x)[8])
{
    x[0] = lo16<DT>(w.x), x[1] = hi16<DT>(w.x), x[2] = lo16<DT>(w.y), x[3] = hi16<DT>(w.y);
    x[4] = lo16<DT>(w.z), x[5] = hi16<DT>(w.z), x[6] = lo16<DT>(w.w), x[7] = hi16<DT>(w.w);
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

template <int CAP>
__device__ __forceinline__ Scalars step_scalars(const ListArgs<CAP>& a)
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

constexpr int kNormLoads = 8;                // 128-bit loads in flight per thread
constexpr uint32_t kNormPass = kThreads * kNormLoads;
constexpr uint32_t kNormMaxBlocks = 2048;    // slots per launch
constexpr int kNormBlocksPerSm = 4;

/* A gradient as 16-byte granules, cut at the addresses' multiples of 16 whatever the
 * tensor's own alignment: the first and the last may be partial. */
struct NormRef {
    const char* base;      // the first granule's address
    uint64_t end;          // granules of the launch up to and including this tensor's
    uint64_t elems;
    uint32_t dtype;
    uint32_t skip;         // elements of the first granule before the tensor
};

constexpr int kNormCap = 1000;

/* What the step's scalars are once the norm is known, formed ahead of it; in the workspace
 * after the last launch's sums. */
struct NormReady {
    ScalerCand cand;
    float step_size, rbc2;
};

template <int CAP>
struct NormArgs {
    zero_step_state_t* st;
    double* slots;              // one partial sum per block, then the step's scalar candidates
    zero_adamw_hparams_t hp;
    uint32_t slot0, last;       // this launch's first slot; 1 in the list's last launch
    uint32_t n;
    uint64_t quota;             // granules per block
    NormRef t[CAP];
};
static_assert(sizeof(NormReady) <= 64, "the workspace's tail");
static_assert(sizeof(NormArgs<kNormCap>) <= 32764, "kernel parameters");

/* A thread's sum of squares: fp32 sums of a granule's 8 (or 4) squares, joined by
 * error-free additions (hi + lo), so that only a granule's own roundings remain (at most
 * 6); granules whose sum leaves fp32's safe range (below 2^-80 or above 2^120: an
 * infinity, a NaN, or a square that would overflow or vanish) are summed in fp64. */
struct Squares {
    float hi = 0.0f, lo = 0.0f;
    double wide = 0.0;
    bool bad = false;

    __device__ __forceinline__ void add(float s)
    {
        const float t = __fadd_rn(hi, s);
        const float bb = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, bb)), __fsub_rn(s, bb)));
        hi = t;
    }

    /* floor: 2^-80, or infinity where 1/(N*L) is so large that a finite gradient could
     * unscale to infinity (then every granule is looked at element by element) */
    template <uint32_t DT>
    __device__ __forceinline__ void granule(const uint4& w, float inv, float floor)
    {
        if (DT == ZERO_F32) {
            const float x0 = __uint_as_float(w.x), x1 = __uint_as_float(w.y);
            const float x2 = __uint_as_float(w.z), x3 = __uint_as_float(w.w);
            const float s = __fadd_rn(__fmaf_rn(x0, x0, __fmul_rn(x1, x1)),
                                      __fmaf_rn(x2, x2, __fmul_rn(x3, x3)));
            if (s < 0x1p120f && s > floor) {
                add(s);
            } else if (((w.x | w.y | w.z | w.w) & 0x7fffffffu) != 0) {
                wide += sumsq_wide(x0, x1, x2, x3, 0.f, 0.f, 0.f, 0.f, 0xfu);
                bad |= not_finite(__fmul_rn(x0, inv)) || not_finite(__fmul_rn(x1, inv)) ||
                       not_finite(__fmul_rn(x2, inv)) || not_finite(__fmul_rn(x3, inv));
            }
        } else {
            constexpr zero_dtype_t D = DT == ZERO_F16 ? ZERO_F16 : ZERO_BF16;
            float x[8];
            widen8<D>(w, x);
            const uint64_t a = f2(x[0], x[1]), b = f2(x[2], x[3]), c = f2(x[4], x[5]), d = f2(x[6], x[7]);
            const uint64_t s2 = f2_add(f2_fma(a, a, f2_mul(b, b)), f2_fma(c, c, f2_mul(d, d)));
            float s0, s1;
            f2_split(s2, s0, s1);
            const float s = __fadd_rn(s0, s1);
            if (s < 0x1p120f && s > floor) {
                add(s);
            } else if (((w.x | w.y | w.z | w.w) & 0x7fff7fffu) != 0) {
                wide += sumsq_wide(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], 0xffu);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    bad |= not_finite(__fmul_rn(x[e], inv));
            }
        }
    }
};

/* A partial granule, element by element; what lies outside the tensor reads as 0. */
__device__ __forceinline__ uint4 partial_granule(const NormRef& t, uint64_t j)
{
    uint32_t w[4] = {0, 0, 0, 0};
    const uint64_t past = t.skip + t.elems;  // elements from the first granule's start to the end
    if (t.dtype == ZERO_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t i = j * 4 + e;
            if (i >= t.skip && i < past)
                w[e] = *reinterpret_cast<const uint32_t*>(t.base + i * 4);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint64_t i = j * 8 + e;
            if (i >= t.skip && i < past)
                w[e >> 1] |= (uint32_t)ld_stream_u16(t.base + i * 2) << (16 * (e & 1));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

/* Granule j of tensor t, whole or partial. */
__device__ __forceinline__ uint4 any_granule(const NormRef& t, uint64_t j)
{
    const uint64_t n = t.dtype == ZERO_F32 ? 4 : 8;
    if (j * n >= t.skip && (j + 1) * n <= t.skip + t.elems)
        return ld_stream_v4(t.base + j * 16);
    return partial_granule(t, j);
}

/* Whole passes, none of their granules partial, of one tensor. */
template <uint32_t DT>
__device__ __forceinline__ void norm_passes(const char* p, uint64_t passes, float inv, float floor, Squares& acc)
{
    p += threadIdx.x * 16;
    for (; passes; --passes, p += kNormPass * 16) {
        uint4 w[kNormLoads];
#pragma unroll
        for (int q = 0; q < kNormLoads; ++q)
            w[q] = ld_stream_v4(p + q * kThreads * 16);
#pragma unroll
        for (int q = 0; q < kNormLoads; ++q)
            acc.granule<DT>(w[q], inv, floor);
    }
}

/* The first tensor of t[k .. upper] whose end lies past granule g. */
template <int CAP>
__device__ __forceinline__ uint32_t norm_find(const NormArgs<CAP>& a, uint64_t g, uint32_t k, uint32_t upper)
{
    while (k < upper) {
        const uint32_t mid = (k + upper) / 2;
        if (a.t[mid].end > g)
            upper = mid;
        else
            k = mid + 1;
    }
    return k;
}

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

/* Sum of squares over the list's gradients: block b takes granules [b*quota, (b+1)*quota)
 * of the launch, whatever tensors they lie in.  In the last launch the block that finishes
 * last adds the blocks' partial sums in order and finalises the step as zero_grad_norm. */
template <int CAP>
__global__ void __launch_bounds__(kThreads, kNormBlocksPerSm) k_tensors_norm(const __grid_constant__ NormArgs<CAP> a)
{
    __shared__ double warp_sum[kThreads / 32];
    __shared__ int is_last;
    // this block's share, from the parameters alone, before the wait for what came before
    const uint32_t n_sum = a.last ? gridDim.x - 1 : gridDim.x;  // the last launch has one block more
    uint64_t lo = blockIdx.x * a.quota;
    const uint64_t total = a.n ? a.t[a.n - 1].end : 0, hi = lo + a.quota < total ? lo + a.quota : total;
    uint32_t k = lo < hi ? norm_find(a, lo, 0, a.n - 1) : 0;
    grid_dependency_wait();
    grid_launch_dependents();
    zero_step_state_t* st = a.st;
    const float inv = st->inv_scale;
    const float floor = inv < 0x1p60f ? 0x1p-80f : __int_as_float(0x7f800000);
    Squares acc;
    NormReady* ready = reinterpret_cast<NormReady*>(a.slots + a.slot0 + n_sum);
    while (lo < hi) {
        const NormRef& t = a.t[k];
        const uint64_t first = k ? a.t[k - 1].end : 0;
        // whole passes inside this tensor, past its first granule and short of its last
        const uint64_t inner = (t.end - 1 < hi ? t.end - 1 : hi), from = lo - first;
        if ((from || !t.skip) && lo + kNormPass <= inner) {
            const uint64_t passes = (inner - lo) / kNormPass;
            const char* p = t.base + from * 16;
            if (t.dtype == ZERO_BF16)
                norm_passes<ZERO_BF16>(p, passes, inv, floor, acc);
            else if (t.dtype == ZERO_F16)
                norm_passes<ZERO_F16>(p, passes, inv, floor, acc);
            else
                norm_passes<ZERO_F32>(p, passes, inv, floor, acc);
            lo += passes * kNormPass;
            continue;
        }
        // one pass over what follows, whichever tensors it meets: all its loads are in
        // flight at once, however short the tensors are
        const uint64_t stop = lo + kNormPass < hi ? lo + kNormPass : hi;
        const uint32_t last = norm_find(a, stop - 1, k, k + kNormPass < a.n ? k + kNormPass : a.n - 1);
        uint4 w[kNormLoads];
        uint32_t type[kNormLoads];
#pragma unroll
        for (int q = 0; q < kNormLoads; ++q) {
            const uint64_t g = lo + q * kThreads + threadIdx.x;
            w[q] = make_uint4(0, 0, 0, 0);
            type[q] = 0;
            if (g < stop) {
                const uint32_t i = norm_find(a, g, k, last);
                w[q] = any_granule(a.t[i], g - (i ? a.t[i - 1].end : 0));
                type[q] = a.t[i].dtype;
            }
        }
#pragma unroll
        for (int q = 0; q < kNormLoads; ++q) {
            if (type[q] == ZERO_BF16)
                acc.granule<ZERO_BF16>(w[q], inv, floor);
            else if (type[q] == ZERO_F16)
                acc.granule<ZERO_F16>(w[q], inv, floor);
            else if (type[q] == ZERO_F32)
                acc.granule<ZERO_F32>(w[q], inv, floor);
        }
        lo = stop;
        k = lo < hi ? norm_find(a, lo, last, last + 1 < a.n ? last + 1 : last) : last;
    }
    if (__any_sync(0xffffffffu, acc.bad) && (threadIdx.x & 31) == 0)
        atomicOr(&st->overflow, 1u);
    if (a.last && blockIdx.x == n_sum) {
        // what does not need the norm, beside the sums (the fp64 powers of beta are a long
        // chain): for either outcome of the overflow check, chosen once it is known
        if (threadIdx.x == 0)
            ready->cand = scaler_candidates(*st, a.hp, st->n_ranks);
        if (threadIdx.x == 32)
            ready->step_size = bias_step_size(a.hp, st->t + 1);
        if (threadIdx.x == 64)
            ready->rbc2 = bias_rbc2(a.hp, st->t + 1);
    } else {
        const double part = block_sum((double)acc.hi + (double)acc.lo + acc.wide, warp_sum);
        if (threadIdx.x == 0)
            a.slots[a.slot0 + blockIdx.x] = part;
    }
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
    double v = 0.0;
    for (uint32_t i = threadIdx.x; i < a.slot0 + n_sum; i += kThreads)
        v += __ldcg(a.slots + i);
    const uint32_t overflow = __ldcg(&st->overflow) != 0;
    const double sumsq = block_sum(v, warp_sum) * ((double)inv * (double)inv);
    // block_sum's barrier: every thread has read the overflow flag
    if (threadIdx.x == 32) {
        const ScalerCand cand{__ldcg(&ready->cand.L_skip), __ldcg(&ready->cand.inv_skip),
                              __ldcg(&ready->cand.L_ok), __ldcg(&ready->cand.inv_ok),
                              __ldcg(&ready->cand.good_ok), __ldcg(&ready->cand.decay)};
        scaler_apply(st, cand, overflow, st->t + 1);
        if (!overflow) {
            st->step_size = __ldcg(&ready->step_size);
            st->rbc2 = __ldcg(&ready->rbc2);
        }
    }
    if (threadIdx.x == 0) {
        const double norm = sqrt(sumsq);
        const float clip = clip_coefficient(norm, overflow, a.hp.max_grad_norm);
        st->arrivals = 0;
        st->sumsq = sumsq;
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

/* A lane's 8 gradients as they lie in memory. */
struct RawGrad {
    float w[8];  // 16-bit gradients: the first four words

    __device__ __forceinline__ void load(const void* g, uint64_t i, uint32_t dtype)
    {
        if (dtype == ZERO_F32) {
            load8(static_cast<const float*>(g) + i, w);
        } else {
            const uint4 a = ld_stream_v4(static_cast<const uint16_t*>(g) + i);
            w[0] = __uint_as_float(a.x), w[1] = __uint_as_float(a.y);
            w[2] = __uint_as_float(a.z), w[3] = __uint_as_float(a.w);
        }
    }
    __device__ __forceinline__ void values(uint32_t dtype, float (&x)[8]) const
    {
        const uint4 a = make_uint4(__float_as_uint(w[0]), __float_as_uint(w[1]), __float_as_uint(w[2]),
                                   __float_as_uint(w[3]));
        if (dtype == ZERO_F16) {
            widen8<ZERO_F16>(a, x);
        } else if (dtype == ZERO_BF16) {
            widen8<ZERO_BF16>(a, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = w[e];
        }
    }
};

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) k_tensors_adamw(const __grid_constant__ ListArgs<CAP> a)
{
    const uint32_t lane = threadIdx.x & 31;
    uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5);
    Place at{0, 1, 0, 0};
    if (u < a.l.n_units)
        locate(a.l, u, at);  // the parameters are this launch's own: no need to wait
    grid_dependency_wait();
    grid_launch_dependents();
    const bool skip = a.st->skip;
    Scalars s = step_scalars(a);
    const float inv = a.st->inv_scale_used, step = s.step;
    for (; u < a.l.n_units; u += gridDim.x * kWarps) {
        locate(a.l, u, at);
        const Ref& t = a.l.t[at.k];
        const uint32_t dtype = t.flags & kGradMask;
        float* m = static_cast<float*>(t.m);
        float* v = static_cast<float*>(t.v);
        s.step = __fmul_rn(step, t.lr_scale);
        s.decay = t.decay;
        const bool vec = t.flags & kVector;
        const uint64_t off = t.head + (uint64_t)at.unit * kUnit;
        // consecutive elements per lane in 128-bit accesses, else lanes side by side
        const uint64_t i = vec ? off + lane * kPer : off + lane;
        const uint32_t stride = vec ? 1 : 32;
        float x8[8], p8[8], m8[8], v8[8];
        const bool whole = vec && i + kPer <= t.elems;
        if (whole) {
            RawGrad raw;
            raw.load(t.grad, i, dtype);
            load8(t.master + i, p8);
            load8(m + i, m8);
            load8(v + i, v8);
            raw.values(dtype, x8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t q = i + e * stride;
                const bool in = q < t.elems;
                x8[e] = in ? one_grad(t.grad, q, dtype) : 0.0f;
                p8[e] = in ? __ldcs(t.master + q) : 0.0f;
                m8[e] = in ? __ldcs(m + q) : 0.0f;
                v8[e] = in ? __ldcs(v + q) : 0.0f;
            }
        }
        if (skip)  // only now: the loads need not wait for the state's
            return;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            adamw_one(__fmul_rn(x8[e], inv), p8[e], m8[e], v8[e], s);
        if (whole) {
            store8(t.master + i, p8);
            store8(m + i, m8);
            store8(v + i, v8);
            if (t.params)
                store_params8(t.params + i, t.flags & kOutF16, p8);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t q = i + e * stride;
                if (q < t.elems) {
                    __stcs(t.master + q, p8[e]);
                    __stcs(m + q, m8[e]);
                    __stcs(v + q, v8[e]);
                    if (t.params)
                        t.params[q] = (t.flags & kOutF16) ? pack1<true>(p8[e]) : pack1<false>(p8[e]);
                }
            }
        }
        if (at.unit == 0 && lane < t.head && lane < t.elems) {  // before the 16-byte boundary
            float p = t.master[lane], mi = m[lane], vi = v[lane];
            adamw_one(__fmul_rn(one_grad(t.grad, lane, dtype), inv), p, mi, vi, s);
            t.master[lane] = p;
            m[lane] = mi;
            v[lane] = vi;
            if (t.params)
                t.params[lane] = (t.flags & kOutF16) ? pack1<true>(p) : pack1<false>(p);
        }
    }
}

/* The largest magnitude, NaN above all. */
__device__ __forceinline__ float max_abs(float top, float x)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(top), "f"(fabsf(x)));
    return r;
}

__device__ __forceinline__ float sqrt_fast(float x)
{
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp_fast(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

/* Four codes of a word as floats with the code's exponent in fp32's field. */
__device__ __forceinline__ float raw_m(uint32_t w, int byte)
{
    const int top = (int)__byte_perm(w, 0, byte << 12 | 0x444);  // the code in bits 31..24
    return __uint_as_float((uint32_t)(top >> 4) & 0x87f00000u);
}

__device__ __forceinline__ float raw_v(uint32_t w, int byte)
{
    return __uint_as_float(__byte_perm(w, 0, byte << 12 | 0x444) >> 4);
}

/* The code of a float from raw_m's or raw_v's scale, rounded with r, in the top byte. */
__device__ __forceinline__ uint32_t top_code(float y, uint32_t r)
{
    return __float_as_uint(y) * 16u + (r >> 8);
}

/* Four codes, each in its word's top byte, as one word. */
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

/* The block exponents up to which one multiplication by a power of two stands for the two
 * of the definition (their product is a normal float both ways). */
constexpr uint32_t kPlainM = 141, kPlainV = 157;

struct Step8 {
    float inv, c, step, decay, b1, b2, omb1, omb2, eps, inv_rbc2;
    uint32_t key;
    bool exact;  // eps too small for the fast reciprocal
};

/* The random words of a lane's element e, their top 20 bits to round with: consecutive
 * elements of the lane's own group ... */
struct RandomInGroup {
    uint32_t seed;

    __device__ __forceinline__ uint32_t m(int e) const { return seed * jump(e + 1).mul + jump(e + 1).add; }
    __device__ __forceinline__ uint32_t v(int e) const { return seed * jump(e + 9).mul + jump(e + 9).add; }
};

/* ... or, lanes side by side, element e in group 4e + lane/8 (whose seed lane 4e + lane/8
 * holds) at place lane%8. */
struct RandomAcross {
    uint32_t seed[8];
    Jump jm, jv;

    __device__ __forceinline__ RandomAcross(uint32_t own, uint32_t lane) : jm(jump(1)), jv(jump(9))
    {
        for (uint32_t q = 0; q < (lane & 7); ++q) {
            jm.add = jm.add * kLcgMul + kLcgAdd, jm.mul *= kLcgMul;
            jv.add = jv.add * kLcgMul + kLcgAdd, jv.mul *= kLcgMul;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            seed[e] = __shfl_sync(0xffffffffu, own, e * 4 + (lane >> 3));
    }
    __device__ __forceinline__ uint32_t m(int e) const { return seed[e] * jm.mul + jm.add; }
    __device__ __forceinline__ uint32_t v(int e) const { return seed[e] * jv.mul + jv.add; }
};

/* One block of 256 elements, 8 per lane: moments, parameters, new codes and exponents.
 *   x p        gradients; parameters, updated
 *   ym yv      the codes as floats (raw_m, raw_v)
 *   bm bv      the exponents, replaced
 *   cm cv      the new codes, element e in byte e
 * The moments are fp32 operations each rounded as written (the codes follow from them bit
 * for bit): decoding needs no instruction of its own, since b1 * (y * 2^k) = y * (b1 * 2^k)
 * exactly.  The parameter's square root, division and sums use the fast forms (within 2
 * ulp): the rounding of p itself is larger than what they add to the update. */
template <typename Random>
__device__ __forceinline__ void block8(const float (&x)[8], float (&p)[8], float (&ym)[8], float (&yv)[8],
                                       uint32_t& bm, uint32_t& bv, const Random& random, uint2& cm,
                                       uint2& cv, const Step8& s)
{
    float fm = bm ? __uint_as_float((bm + 112u) << 23) : 0.0f;
    float fv = bv ? __uint_as_float((bv + 96u) << 23) : 0.0f;
    if (bm > kPlainM || bv > kPlainV) {  // the whole warp: far above any gradient met in earnest
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ym[e] = __fmul_rn(ym[e], 0x1p112f);
            yv[e] = __fmul_rn(yv[e], 0x1p96f);
        }
        fm = exp_scale(bm);
        fv = exp_scale(bv);
    }
    fm = __fmul_rn(s.b1, fm);
    fv = __fmul_rn(s.b2, fv);
    const uint64_t inv2 = f2(s.inv, s.inv), c2 = f2(s.c, s.c), fm2 = f2(fm, fm), fv2 = f2(fv, fv);
    const uint64_t o1 = f2(s.omb1, s.omb1), o2 = f2(s.omb2, s.omb2);
    float m[8], v[8], top_m = 0.0f, top_v = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint64_t gc = f2_mul(c2, f2_mul(f2(x[e], x[e + 1]), inv2));
        // the sums are scalar: a paired sum of paired products came out contracted (one
        // product unrounded), 1 ulp off the definition where a code's boundary showed it
        float a0, a1, b0, b1;
        f2_split(f2_mul(f2(ym[e], ym[e + 1]), fm2), a0, a1);
        f2_split(f2_mul(o1, gc), b0, b1);
        m[e] = __fadd_rn(a0, b0);
        m[e + 1] = __fadd_rn(a1, b1);
        f2_split(f2_mul(f2(yv[e], yv[e + 1]), fv2), a0, a1);
        f2_split(f2_mul(o2, f2_mul(gc, gc)), b0, b1);
        v[e] = __fadd_rn(a0, b0);
        v[e + 1] = __fadd_rn(a1, b1);
        top_m = max_abs(max_abs(top_m, m[e]), m[e + 1]);
        top_v = max_abs(max_abs(top_v, v[e]), v[e + 1]);
    }
    bm = block_exponent(__reduce_max_sync(0xffffffffu, __float_as_uint(top_m) & 0x7fffffffu));
    bv = block_exponent(__reduce_max_sync(0xffffffffu, __float_as_uint(top_v) & 0x7fffffffu));
    uint32_t word_m[2], word_v[2];
    if (bm <= kPlainM && bv <= kPlainV && !s.exact) {
        const uint64_t um = f2(__uint_as_float((142u - bm) << 23), __uint_as_float((142u - bm) << 23));
        const uint64_t uv = f2(__uint_as_float((158u - bv) << 23), __uint_as_float((158u - bv) << 23));
        // sqrt(v) = sqrt(v * 2^24) * 2^-12: no subnormal v reaches the fast square root
        const float r = __fmul_rn(s.inv_rbc2, 0x1p-12f);
        const uint64_t up = f2(0x1p24f, 0x1p24f), r2 = f2(r, r), eps2 = f2(s.eps, s.eps);
        const uint64_t decay2 = f2(s.decay, s.decay), step2 = f2(-s.step, -s.step);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t code_m[4], code_v[4];  // in the words' top bytes
#pragma unroll
            for (int o = 0; o < 4; o += 2) {
                const int e = 4 * h + o;
                const uint64_t m2 = f2(m[e], m[e + 1]), v2 = f2(v[e], v[e + 1]);
                float v0, v1, d0, d1, y0, y1;
                f2_split(f2_mul(v2, up), v0, v1);
                f2_split(f2_fma(f2(sqrt_fast(v0), sqrt_fast(v1)), r2, eps2), d0, d1);
                const uint64_t q = f2_mul(f2_mul(m2, step2), f2(rcp_fast(d0), rcp_fast(d1)));
                f2_split(f2_fma(f2(p[e], p[e + 1]), decay2, q), p[e], p[e + 1]);
                f2_split(f2_mul(m2, um), y0, y1);
                // the bits times 16 put the code into the top byte (m's sign falls out); four
                // more random bits below the 20 change no carry, since all else there is 0
                code_m[o] = top_code(y0, random.m(e)) & 0x7fffffffu | __float_as_uint(y0) & 0x80000000u;
                code_m[o + 1] = top_code(y1, random.m(e + 1)) & 0x7fffffffu | __float_as_uint(y1) & 0x80000000u;
                f2_split(f2_mul(v2, uv), y0, y1);
                code_v[o] = top_code(y0, random.v(e));
                code_v[o + 1] = top_code(y1, random.v(e + 1));
                if (v[e] != 0.0f)
                    code_v[o] = max(code_v[o], 1u << 24);
                if (v[e + 1] != 0.0f)
                    code_v[o + 1] = max(code_v[o + 1], 1u << 24);
            }
            word_m[h] = top_bytes(code_m[0], code_m[1], code_m[2], code_m[3]);
            word_v[h] = top_bytes(code_v[0], code_v[1], code_v[2], code_v[3]);
        }
    } else {
        const float um = exp_unscale(bm), uv = exp_unscale(bv);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            word_m[h] = word_v[h] = 0;
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                const int e = 4 * h + o;
                const float denom = __fadd_rn(__fmul_rn(__fsqrt_rn(v[e]), s.inv_rbc2), s.eps);
                p[e] = __fsub_rn(__fmul_rn(p[e], s.decay), __fmul_rn(s.step, __fdiv_rn(m[e], denom)));
                word_m[h] |= encode_m(m[e], um, random.m(e) >> 12) << (8 * o);
                word_v[h] |= encode_v(v[e], uv, random.v(e) >> 12) << (8 * o);
            }
        }
    }
    cm = make_uint2(word_m[0], word_m[1]);
    cv = make_uint2(word_v[0], word_v[1]);
}

__device__ __forceinline__ bool whole_unit(const Ref& t, uint32_t unit)
{
    return (t.flags & kVector) && ((uint64_t)unit + 1) * kUnit <= t.elems;
}

template <int CAP>
__device__ __forceinline__ Step8 step8(const ListArgs<CAP>& a)
{
    const zero_step_state_t* st = a.st;
    Step8 s;
    s.inv = st->inv_scale_used;
    s.c = st->clip_coef;
    s.step = st->step_size;
    s.decay = 1.0f;
    s.b1 = a.beta1;
    s.b2 = a.beta2;
    s.omb1 = __fsub_rn(1.0f, a.beta1);
    s.omb2 = __fsub_rn(1.0f, a.beta2);
    s.eps = a.eps;
    s.inv_rbc2 = __fdiv_rn(1.0f, st->rbc2);
    s.key = step_key(a.seed, st->t);
    s.exact = a.eps < 0x1p-100f;
    return s;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) k_tensors_adamw8(const __grid_constant__ ListArgs<CAP> a)
{
    const uint32_t lane = threadIdx.x & 31, stride = gridDim.x * kWarps;
    uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5);
    Place at{0, 1, 0, 0};
    if (u < a.l.n_units)
        locate(a.l, u, at);  // the parameters are this launch's own: no need to wait
    grid_dependency_wait();
    grid_launch_dependents();
    const bool skip = a.st->skip;
    Step8 s = step8(a);
    const float step = s.step;
    for (; u < a.l.n_units; u += stride) {
        locate(a.l, u, at);
        const Ref& t = a.l.t[at.k];
        const uint32_t dtype = t.flags & kGradMask, unit = at.unit;
        s.step = __fmul_rn(step, t.lr_scale);
        s.decay = t.decay;
        const bool whole = whole_unit(t, unit);
        // consecutive elements per lane, else lanes side by side
        const uint64_t i = (uint64_t)unit * kUnit + (whole ? lane * kPer : lane);
        uint8_t* m = static_cast<uint8_t*>(t.m) + i;
        uint8_t* v = static_cast<uint8_t*>(t.v) + i;
        uint8_t* exps = t.exps + 2 * (uint64_t)unit;
        uint32_t bm = exps[0], bv = exps[1];
        // lane L's seed is that of the block's group L
        const uint32_t seed = mix32(s.key + (t.group0 + unit * 32 + lane) * kGolden);
        uint2 cm, cv;
        float x[8], p[8], ym[8], yv[8];
        if (whole) {
            RawGrad raw;
            raw.load(t.grad, i, dtype);
            load8(t.master + i, p);
            cm = __ldcs(reinterpret_cast<const uint2*>(m));
            cv = __ldcs(reinterpret_cast<const uint2*>(v));
            raw.values(dtype, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ym[e] = raw_m(e < 4 ? cm.x : cm.y, e & 3);
                yv[e] = raw_v(e < 4 ? cv.x : cv.y, e & 3);
            }
            if (skip)
                return;
            block8(x, p, ym, yv, bm, bv, RandomInGroup{seed}, cm, cv, s);
            store8(t.master + i, p);
            if (t.params)
                store_params8(t.params + i, t.flags & kOutF16, p);
            __stcs(reinterpret_cast<uint2*>(m), cm);
            __stcs(reinterpret_cast<uint2*>(v), cv);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = i + e * 32 < t.elems;
                x[e] = in ? one_grad(t.grad, i + e * 32, dtype) : 0.0f;
                p[e] = in ? __ldcs(t.master + i + e * 32) : 0.0f;
                ym[e] = in ? raw_m(m[e * 32], 0) : 0.0f;
                yv[e] = in ? raw_v(v[e * 32], 0) : 0.0f;
            }
            if (skip)
                return;
            block8(x, p, ym, yv, bm, bv, RandomAcross(seed, lane), cm, cv, s);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (i + e * 32 < t.elems) {
                    m[e * 32] = (uint8_t)((e < 4 ? cm.x : cm.y) >> (8 * (e & 3)));
                    v[e * 32] = (uint8_t)((e < 4 ? cv.x : cv.y) >> (8 * (e & 3)));
                    __stcs(t.master + i + e * 32, p[e]);
                    if (t.params)
                        t.params[i + e * 32] = (t.flags & kOutF16) ? pack1<true>(p[e]) : pack1<false>(p[e]);
                }
            }
        }
        if (lane == 0) {
            exps[0] = (uint8_t)bm;
            exps[1] = (uint8_t)bv;
        }
    }
}

/* ------------------------------------------------------------------------------------ */
/* 8-bit states to values and back                                                        */
/* ------------------------------------------------------------------------------------ */

/* A block's values, 8 per lane, to their nearest codes; the exponents (m's, v's). */
__device__ __forceinline__ uint2 nearest_codes(const float (&m)[8], const float (&v)[8], uint2& cm, uint2& cv)
{
    uint32_t top_m = 0, top_v = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        top_m = max(top_m, __float_as_uint(m[e]) & 0x7fffffffu);
        top_v = max(top_v, __float_as_uint(v[e]) & 0x7fffffffu);
    }
    const uint32_t bm = block_exponent(__reduce_max_sync(0xffffffffu, top_m));
    const uint32_t bv = block_exponent(__reduce_max_sync(0xffffffffu, top_v));
    const float um = exp_unscale(bm), uv = exp_unscale(bv);
    uint32_t wm[2] = {0, 0}, wv[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        wm[e / 4] |= encode_m(m[e], um, kNearest) << (8 * (e & 3));
        wv[e / 4] |= encode_v(v[e], uv, kNearest) << (8 * (e & 3));
    }
    cm = make_uint2(wm[0], wm[1]);
    cv = make_uint2(wv[0], wv[1]);
    return make_uint2(bm, bv);
}

/* A warp per unit, straight from global memory, as many warps as fit: there is little
 * arithmetic to hide and twice to four times as much to write as to read. */
template <int CAP>
__global__ void __launch_bounds__(kThreads, 8) k_state8_read(const __grid_constant__ ListArgs<CAP> a)
{
    const uint32_t lane = threadIdx.x & 31, stride = gridDim.x * kWarps;
    uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5);
    Place place{0, 1, 0, 0};
    if (u < a.l.n_units)
        locate(a.l, u, place);  // the parameters are this launch's own: no need to wait
    grid_dependency_wait();
    grid_launch_dependents();
    for (; u < a.l.n_units; u += stride) {
        locate(a.l, u, place);
        const Ref& t = a.l.t[place.k];
        const bool whole = whole_unit(t, place.unit), bf16 = t.flags & kValueBF16;
        const uint64_t at = (uint64_t)place.unit * kUnit + (whole ? lane * kPer : lane);
        const uint8_t* exps = t.exps + 2 * (uint64_t)place.unit;
        const uint8_t* cm = static_cast<const uint8_t*>(t.m) + at;
        const uint8_t* cv = static_cast<const uint8_t*>(t.v) + at;
        const float scale_m = exp_scale(exps[0]), scale_v = exp_scale(exps[1]);
        auto value_m = [&](float y) { return __fmul_rn(__fmul_rn(y, 0x1p112f), scale_m); };
        auto value_v = [&](float y) { return __fmul_rn(__fmul_rn(y, 0x1p96f), scale_v); };
        if (whole) {
            const uint2 wm = __ldcs(reinterpret_cast<const uint2*>(cm)), wv = __ldcs(reinterpret_cast<const uint2*>(cv));
            float m[8], v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                m[e] = value_m(raw_m(e < 4 ? wm.x : wm.y, e & 3));
                v[e] = value_v(raw_v(e < 4 ? wv.x : wv.y, e & 3));
            }
            if (bf16) {
                store_params8(static_cast<uint16_t*>(t.x) + at, 0, m);
                store_params8(static_cast<uint16_t*>(t.y) + at, 0, v);
            } else {
                store8(static_cast<float*>(t.x) + at, m);
                store8(static_cast<float*>(t.y) + at, v);
            }
        } else {
            uint32_t c[8];  // m's code, v's above it
#pragma unroll
            for (int e = 0; e < 8; ++e)
                c[e] = at + e * 32 < t.elems ? cm[e * 32] | cv[e * 32] << 8 : 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t q = at + e * 32;
                if (q >= t.elems)
                    continue;
                const float m = value_m(raw_m(c[e], 0)), v = value_v(raw_v(c[e], 1));
                if (bf16) {
                    static_cast<uint16_t*>(t.x)[q] = pack1<false>(m);
                    static_cast<uint16_t*>(t.y)[q] = pack1<false>(v);
                } else {
                    static_cast<float*>(t.x)[q] = m;
                    static_cast<float*>(t.y)[q] = v;
                }
            }
        }
    }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 6) k_state8_write(const __grid_constant__ ListArgs<CAP> a)
{
    const uint32_t lane = threadIdx.x & 31, stride = gridDim.x * kWarps;
    uint32_t u = blockIdx.x * kWarps + (threadIdx.x >> 5);
    Place place{0, 1, 0, 0};
    if (u < a.l.n_units)
        locate(a.l, u, place);
    grid_dependency_wait();
    grid_launch_dependents();
    for (; u < a.l.n_units; u += stride) {
        locate(a.l, u, place);
        const Ref& t = a.l.t[place.k];
        const bool whole = whole_unit(t, place.unit);
        const uint64_t at = (uint64_t)place.unit * kUnit + (whole ? lane * kPer : lane);
        const float* xm = static_cast<const float*>(t.x) + at;
        const float* xv = static_cast<const float*>(t.y) + at;
        uint8_t* cm = static_cast<uint8_t*>(t.m) + at;
        uint8_t* cv = static_cast<uint8_t*>(t.v) + at;
        float m[8], v[8];
        if (whole) {
            load8(xm, m);
            load8(xv, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                m[e] = at + e * 32 < t.elems ? __ldcs(xm + e * 32) : 0.0f;
                v[e] = at + e * 32 < t.elems ? __ldcs(xv + e * 32) : 0.0f;
            }
        }
        uint2 wm, wv;
        const uint2 b = nearest_codes(m, v, wm, wv);
        if (whole) {
            __stcs(reinterpret_cast<uint2*>(cm), wm);
            __stcs(reinterpret_cast<uint2*>(cv), wv);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (at + e * 32 < t.elems) {
                    cm[e * 32] = (uint8_t)((e < 4 ? wm.x : wm.y) >> (8 * (e & 3)));
                    cv[e * 32] = (uint8_t)((e < 4 ? wv.x : wv.y) >> (8 * (e & 3)));
                }
        }
        if (lane == 0) {
            t.exps[2 * (uint64_t)place.unit] = (uint8_t)b.x;
            t.exps[2 * (uint64_t)place.unit + 1] = (uint8_t)b.y;
        }
    }
}

/* ------------------------------------------------------------------------------------ */
/* AdamW on long lists: staged through shared memory                                      */
/* ------------------------------------------------------------------------------------ */

/* One block per SM: a producer warp fills a ring of stages with the bulk-copy engine, the
 * consumer warps take a 256-element unit each from every stage, release it as soon as its
 * values are in registers, and store their results straight to global memory.  A stage is
 * a chunk of one tensor, a unit for each consumer warp; its slots are 128 bytes longer than
 * a chunk's data: an array that does not start on 16 bytes keeps its offset from the
 * boundary below. */
template <bool S8>
struct Ring {
    static constexpr int kWarps = S8 ? 23 : 16, kThreads = (kWarps + 1) * 32;
    static constexpr uint32_t kChunk = kWarps * kUnit;
    static constexpr uint32_t kWide = kChunk * 4 + 128, kState = kChunk * (S8 ? 1 : 4) + 128;
    static constexpr uint32_t kGrad = 0, kMaster = kWide, kM = 2 * kWide, kV = kM + kState, kExps = kV + kState;
    static constexpr uint32_t kBytes = kExps + (S8 ? 256 : 0);
    static constexpr uint32_t kStages = 3, kSmem = kBytes * kStages;
};
static_assert(Ring<false>::kSmem <= 220 * 1024 && Ring<true>::kSmem <= 220 * 1024, "shared memory");

/* What the producer tells the consumers of a stage, so that each warp need not work it out:
 * arrays at the chunk's first element. */
struct alignas(16) StageInfo {
    uint32_t n;      // elements; 0: the queue is empty
    uint32_t flags;  // the tensor's
    float lr_scale, decay;
    uint32_t group;  // 8-bit states: the chunk's first group of 8 elements
    uint32_t grad, master, m, v, exps;  // in the stage
    float* out_master;
    char* out_m;
    char* out_v;
    uint8_t* out_exps;
    uint16_t* out_params;  // or null
};

/* Phase `parity` of a stage's barrier; the clock is read only where the first try fails. */
__device__ __forceinline__ bool stage_wait(const uint64_t& bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(smem_addr(&bar)), "r"(parity)
                 : "memory");
    return ok || wait_parity_bounded(smem_addr(&bar), parity);
}

/* The producer warp's copy of bytes [at, at + len) of an array of `bytes` bytes into a
 * slot, at the same offset from a 16-byte boundary.  Whole 16-byte granules go by bulk
 * copy, over the chunk's ends where the array goes on there; the granules that the array's
 * own ends cut are filled byte by byte, so nothing outside the array is read.  Returns the
 * bulk copy's span in lo, hi (for expect_tx, before bulk()). */
struct SlotCopy {
    const char* from;
    uint32_t dst, len;
    uint32_t offset;  // the first byte's place in the slot

    __device__ __forceinline__ SlotCopy(const void* base, uint64_t bytes, uint64_t at, uint32_t n, char* slot,
                                        uint32_t lane)
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(base), first = a + at, end = first + n;
        const uintptr_t origin = first & ~(uintptr_t)15;
        uintptr_t lo = origin, hi = (end + 15) & ~(uintptr_t)15;
        if (lo < a || hi > a + bytes) {
            const uintptr_t stop = a + bytes < end ? a + bytes : end;
            if (lo < a)
                lo += 16;
            if (hi > a + bytes)
                hi -= 16;
            if (hi < lo)
                hi = lo;  // one granule cut at both ends: all of it byte by byte
            // at most 15 bytes before lo and 15 from hi on (16 to `stop` when lo == hi)
            const uintptr_t x = lane < 16 ? first + lane : hi + (lane - 16);
            if (lane < 16 ? x < lo && x < stop : x < stop)
                slot[x - origin] = *reinterpret_cast<const char*>(x);
        }
        from = reinterpret_cast<const char*>(lo);
        offset = (uint32_t)(first - origin);
        dst = smem_addr(slot) + (uint32_t)(lo - origin);
        len = (uint32_t)(hi - lo);
    }
    __device__ __forceinline__ void bulk(uint32_t bar) const
    {
        if (len)
            bulk_load<true>(dst, from, len, bar);
    }
};

/* Fills the stages until the list's chunks are used up: one at a time from a queue in the
 * step state, so that the chunks in flight stay together at the front of the list however
 * the blocks' speeds differ. */
template <bool S8, int CAP>
__device__ __forceinline__ void produce(const ListArgs<CAP>& a, char* stages, uint64_t* full, uint64_t* empty,
                                        StageInfo* info)
{
    using R = Ring<S8>;
    const uint32_t lane = threadIdx.x & 31;
    zero_step_state_t* st = const_cast<zero_step_state_t*>(a.st);
    unsigned long long* queue = reinterpret_cast<unsigned long long*>(&st->adamw_next_chunk);
    unsigned long long next = 0;
    if (lane == 0)
        next = atomicAdd(queue, 1ull);
    Place at{0, 1, 0, 0};
    uint32_t issued = 0, live = R::kStages - 1;  // stages before `issued` that may be unread
    for (;; ++issued) {
        const uint32_t k = issued % R::kStages;
        if (issued >= R::kStages && !stage_wait(empty[k], (issued / R::kStages - 1) & 1)) {
            if (lane == 0)
                atomicOr(&st->error, 1u);
            live = R::kStages;
            break;
        }
        const unsigned long long c = __shfl_sync(0xffffffffu, next, 0);
        const uint32_t bar = smem_addr(&full[k]);
        if (c >= a.l.n_units) {
            if (lane == 0) {
                info[k].n = 0;
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
            }
            break;
        }
        if (lane == 0)  // one ahead: its latency stays off the ring's path
            next = atomicAdd(queue, 1ull);
        locate(a.l, (uint32_t)c, at);
        const Ref& t = a.l.t[at.k];
        char* s = stages + k * R::kBytes;
        const uint64_t first = (uint64_t)at.unit * R::kChunk;
        const uint32_t n = t.elems - first < R::kChunk ? (uint32_t)(t.elems - first) : R::kChunk;
        auto copy = [&](const void* base, uint32_t size, uint32_t slot) {
            return SlotCopy(base, t.elems * size, first * size, n * size, s + slot, lane);
        };
        const SlotCopy g = copy(t.grad, (t.flags & kGradMask) == ZERO_F32 ? 4 : 2, R::kGrad);
        const SlotCopy p = copy(t.master, 4, R::kMaster);
        const SlotCopy m = copy(t.m, S8 ? 1 : 4, R::kM);
        const SlotCopy v = copy(t.v, S8 ? 1 : 4, R::kV);
        SlotCopy b = m;
        uint32_t bytes = g.len + p.len + m.len + v.len;
        if (S8) {
            b = SlotCopy(t.exps, (t.elems + kUnit - 1) / kUnit * 2, first / kUnit * 2, (n + kUnit - 1) / kUnit * 2,
                         s + R::kExps, lane);
            bytes += b.len;
        }
        // the bytes the lanes wrote come before the arrival, and before any later bulk copy
        // into the same slot
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            StageInfo& w = info[k];
            w.n = n;
            w.flags = t.flags;
            w.lr_scale = t.lr_scale;
            w.decay = t.decay;
            w.group = t.group0 + (uint32_t)(first / kPer);
            w.grad = R::kGrad + g.offset;
            w.master = R::kMaster + p.offset;
            w.m = R::kM + m.offset;
            w.v = R::kV + v.offset;
            w.exps = S8 ? R::kExps + b.offset : 0;
            w.out_master = t.master + first;
            w.out_m = static_cast<char*>(t.m) + first * (S8 ? 1 : 4);
            w.out_v = static_cast<char*>(t.v) + first * (S8 ? 1 : 4);
            w.out_exps = S8 ? t.exps + first / kUnit * 2 : nullptr;
            w.out_params = t.params ? t.params + first : nullptr;
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
            g.bulk(bar);
            p.bulk(bar);
            m.bulk(bar);
            v.bulk(bar);
            if (S8)
                b.bulk(bar);
        }
    }
    // every copy has landed before the block may end (a consumer that gave up leaves stages
    // unread)
    for (uint32_t i = issued > live ? issued - live : 0; i < issued; ++i)
        wait_parity_bounded(smem_addr(&full[i % R::kStages]), (i / R::kStages) & 1);
    if (lane == 0) {  // the queue back to 0 for the next launch, by the last block
        __threadfence();
        if (atomicAdd(&st->adamw_done, 1u) == gridDim.x - 1) {
            __threadfence();
            atomicExch(queue, 0ull);
            atomicExch(&st->adamw_done, 0u);
        }
    }
}

/* A lane's elements of a stage: 8 consecutive ones where every array allows it and the
 * warp's unit is whole, else one of every 32. */
struct InStage {
    const char* slot;
    uint32_t e0, n;  // the first of them; the stage's elements
    bool whole;

    __device__ __forceinline__ bool in(int e) const { return e0 + e * 32 < n; }

    __device__ __forceinline__ void floats(uint32_t array, float (&to)[8]) const
    {
        const float* from = reinterpret_cast<const float*>(slot + array) + e0;
        if (whole) {
            const float4 lo = reinterpret_cast<const float4*>(from)[0], hi = reinterpret_cast<const float4*>(from)[1];
            to[0] = lo.x, to[1] = lo.y, to[2] = lo.z, to[3] = lo.w;
            to[4] = hi.x, to[5] = hi.y, to[6] = hi.z, to[7] = hi.w;
        } else {  // past n: what the slot holds there, never stored
#pragma unroll
            for (int e = 0; e < 8; ++e)
                to[e] = from[e * 32];
        }
    }
    __device__ __forceinline__ void grads(uint32_t array, uint32_t dtype, float (&to)[8]) const
    {
        if (dtype == ZERO_F32) {
            floats(array, to);
            return;
        }
        const uint16_t* from = reinterpret_cast<const uint16_t*>(slot + array) + e0;
        if (whole) {
            const uint4 w = *reinterpret_cast<const uint4*>(from);
            if (dtype == ZERO_F16)
                widen8<ZERO_F16>(w, to);
            else
                widen8<ZERO_BF16>(w, to);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                to[e] = dtype == ZERO_F16 ? one16<ZERO_F16>(from[e * 32]) : one16<ZERO_BF16>(from[e * 32]);
        }
    }
    /* The codes of m and v as floats; 0 past n, so that what lies there does not count in
     * the block's exponents. */
    __device__ __forceinline__ void codes(uint32_t m, uint32_t v, float (&ym)[8], float (&yv)[8]) const
    {
        const uint8_t* cm = reinterpret_cast<const uint8_t*>(slot + m) + e0;
        const uint8_t* cv = reinterpret_cast<const uint8_t*>(slot + v) + e0;
        if (whole) {
            const uint2 wm = *reinterpret_cast<const uint2*>(cm), wv = *reinterpret_cast<const uint2*>(cv);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ym[e] = raw_m(e < 4 ? wm.x : wm.y, e & 3);
                yv[e] = raw_v(e < 4 ? wv.x : wv.y, e & 3);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ym[e] = in(e) ? raw_m(cm[e * 32], 0) : 0.0f;
                yv[e] = in(e) ? raw_v(cv[e * 32], 0) : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void put(void* to, const float (&x)[8]) const
    {
        float* p = static_cast<float*>(to) + e0;
        if (whole) {
            store8(p, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (in(e))
                    __stcs(p + e * 32, x[e]);
        }
    }
    __device__ __forceinline__ void put_params(uint16_t* to, bool f16, const float (&x)[8]) const
    {
        if (whole) {
            store_params8(to + e0, f16, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (in(e))
                    to[e0 + e * 32] = f16 ? pack1<true>(x[e]) : pack1<false>(x[e]);
        }
    }
    __device__ __forceinline__ void put_codes(char* to, uint2 c) const
    {
        if (whole) {
            __stcs(reinterpret_cast<uint2*>(to + e0), c);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (in(e))
                    to[e0 + e * 32] = (char)((e < 4 ? c.x : c.y) >> (8 * (e & 3)));
        }
    }
};

template <bool S8, int CAP>
__global__ void __launch_bounds__(Ring<S8>::kThreads, 1) k_tensors_ring(const __grid_constant__ ListArgs<CAP> a)
{
    using R = Ring<S8>;
    extern __shared__ __align__(128) char stages[];
    __shared__ __align__(8) uint64_t full[R::kStages], empty[R::kStages];
    __shared__ StageInfo info[R::kStages];
    grid_dependency_wait();
    if (a.st->skip)
        return;
    if (threadIdx.x == 0) {
        for (uint32_t k = 0; k < R::kStages; ++k) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&full[k])));
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&empty[k])), "n"(R::kWarps));
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == R::kWarps) {
        produce<S8>(a, stages, full, empty, info);
        return;
    }
    Scalars s;
    Step8 s8;
    float inv = 1.0f, step = 0.0f;
    if (S8) {
        s8 = step8(a);
        step = s8.step;
    } else {
        s = step_scalars(a);
        inv = a.st->inv_scale_used;
        step = s.step;
    }
    for (uint32_t i = 0;; ++i) {
        const uint32_t q = i % R::kStages;
        if (!stage_wait(full[q], (i / R::kStages) & 1)) {
            if (lane == 0)
                atomicOr(&const_cast<zero_step_state_t*>(a.st)->error, 1u);
            return;
        }
        const StageInfo t = info[q];
        if (t.n == 0)
            return;
        auto release = [&] {  // this warp has what it needs of the stage
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty[q])) : "memory");
        };
        if (warp * kUnit >= t.n) {
            release();
            continue;
        }
        InStage u;
        u.slot = stages + q * R::kBytes;
        u.n = t.n;
        u.whole = (t.flags & kVector) && (warp + 1) * kUnit <= t.n;
        u.e0 = warp * kUnit + (u.whole ? lane * kPer : lane);
        float x[8], p[8];
        u.grads(t.grad, t.flags & kGradMask, x);
        u.floats(t.master, p);
        if (S8) {
            const uint8_t* b = reinterpret_cast<const uint8_t*>(u.slot + t.exps) + 2 * warp;
            float ym[8], yv[8];
            u.codes(t.m, t.v, ym, yv);
            uint32_t bm = b[0], bv = b[1];
            release();
            s8.step = __fmul_rn(step, t.lr_scale);
            s8.decay = t.decay;
            const uint32_t seed = mix32(s8.key + (t.group + warp * 32 + lane) * kGolden);
            uint2 cm, cv;
            if (u.whole) {
                block8(x, p, ym, yv, bm, bv, RandomInGroup{seed}, cm, cv, s8);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = u.in(e) ? x[e] : 0.0f;
                block8(x, p, ym, yv, bm, bv, RandomAcross(seed, lane), cm, cv, s8);
            }
            u.put_codes(t.out_m, cm);
            u.put_codes(t.out_v, cv);
            if (lane == 0) {
                t.out_exps[2 * warp] = (uint8_t)bm;
                t.out_exps[2 * warp + 1] = (uint8_t)bv;
            }
        } else {
            float m[8], v[8];
            u.floats(t.m, m);
            u.floats(t.v, v);
            release();
            s.step = __fmul_rn(step, t.lr_scale);
            s.decay = t.decay;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                adamw_one(__fmul_rn(x[e], inv), p[e], m[e], v[e], s);
            u.put(t.out_m, m);
            u.put(t.out_v, v);
        }
        u.put(t.out_master, p);
        if (t.out_params)
            u.put_params(t.out_params, t.flags & kOutF16, p);
    }
}

/* ------------------------------------------------------------------------------------ */
/* host side                                                                              */
/* ------------------------------------------------------------------------------------ */

bool finite_f(float x) { return x == x && x <= 3.4e38f && x >= -3.4e38f; }

bool at(const void* p, uintptr_t align) { return ((uintptr_t)p & (align - 1)) == 0; }

constexpr bool is_adamw(Op op) { return op == Op::kAdamw || op == Op::kAdamw8; }
constexpr bool is_codec(Op op) { return op == Op::kRead || op == Op::kWrite; }

/* What an operator needs of tensor t (and, for the codec, of its 32-bit partner). */
template <Op OP>
int check_tensor(const zero_tensor_t& t, const zero_tensor_t* other)
{
    if (t.elems == 0)
        return other && other->elems != 0 ? ZERO_EINVAL : ZERO_OK;
    if (t.elems > (1ull << 39))
        return ZERO_EINVAL;
    bool aligned = true;
    if (!is_codec(OP)) {
        if (!t.grad || (t.grad_dtype != ZERO_F16 && t.grad_dtype != ZERO_BF16 && t.grad_dtype != ZERO_F32))
            return ZERO_EINVAL;
        aligned &= at(t.grad, t.grad_dtype == ZERO_F32 ? 4 : 2);
    }
    if (is_adamw(OP)) {
        if (!t.master || (t.params_dtype != 0 && t.params_dtype != ZERO_BF16 && t.params_dtype != ZERO_F16))
            return ZERO_EINVAL;
        if (!finite_f(t.lr_scale) || t.lr_scale < 0.0f || !finite_f(t.weight_decay))
            return ZERO_EINVAL;
        aligned &= at(t.master, 4) && at(t.params, 2);
    }
    if (OP != Op::kNorm && (!t.m || !t.v))
        return ZERO_EINVAL;
    if (OP == Op::kAdamw) {
        if (t.state_dtype != ZERO_F32)
            return ZERO_EINVAL;
        aligned &= at(t.m, 4) && at(t.v, 4);
    }
    if ((OP == Op::kAdamw8 || is_codec(OP)) && (t.state_dtype != ZERO_U8 || !t.exps))
        return ZERO_EINVAL;
    if (is_codec(OP)) {
        const bool bf16 = OP == Op::kRead && other->state_dtype == ZERO_BF16;
        if (other->elems != t.elems || !other->m || !other->v || (other->state_dtype != ZERO_F32 && !bf16))
            return ZERO_EINVAL;
        aligned &= at(other->m, bf16 ? 2 : 4) && at(other->v, bf16 ? 2 : 4);
    }
    return aligned ? ZERO_OK : ZERO_EALIGN;
}

/* The whole list, and its number of elements. */
template <Op OP>
int check_list(const zero_tensor_t* tensors, const zero_tensor_t* others, uint64_t n, uint64_t& total)
{
    total = 0;
    if (n > (1ull << 31) || (n && (!tensors || (is_codec(OP) && !others))))
        return ZERO_EINVAL;
    int align = ZERO_OK;
    for (uint64_t k = 0; k < n; ++k) {
        const int rc = check_tensor<OP>(tensors[k], is_codec(OP) ? others + k : nullptr);
        if (rc == ZERO_EINVAL)
            return rc;
        if (rc != ZERO_OK)
            align = rc;
        total += tensors[k].elems;
    }
    return align;
}

/* Every array of the operator allows one access per 8 elements from element h on: fp32 at
 * 32 bytes, 16-bit arrays at 16, codes at 8. */
template <Op OP>
bool vector_from(const zero_tensor_t& t, const zero_tensor_t* other, uint32_t h)
{
    // the bits of the addresses below their alignment, as multiples of 8 elements
    auto off = [h](const void* p, uintptr_t size) { return ((uintptr_t)p + h * size) & (8 * size - 1); };
    if (is_codec(OP)) {
        const uintptr_t size = other->state_dtype == ZERO_BF16 ? 2 : 4;
        return (off(t.m, 1) | off(t.v, 1) | off(other->m, size) | off(other->v, size)) == 0;
    }
    const uintptr_t size = OP == Op::kAdamw8 ? 1 : 4;
    return (off(t.grad, t.grad_dtype == ZERO_F32 ? 4 : 2) | off(t.master, 4) | off(t.m, size) | off(t.v, size) |
            (t.params ? off(t.params, 2) : 0)) == 0;
}

/* Fills `l` with tensors from index `next` on, as many as fit, in units of UNIT elements;
 * returns the next index. */
template <Op OP, uint32_t UNIT>
uint64_t fill(List<kLarge>& l, const zero_tensor_t* tensors, const zero_tensor_t* others, uint64_t n,
              uint64_t next, const zero_adamw_hparams_t* hp, uint32_t& group0)
{
    uint64_t units = 0;
    uint32_t filled = 0;
    for (; next < n && filled < (uint32_t)kLarge; ++next) {
        const zero_tensor_t& t = tensors[next];
        const zero_tensor_t* other = is_codec(OP) ? others + next : nullptr;
        if (t.elems == 0)
            continue;
        // 32-bit states, straight from global memory: an offset that all arrays share
        // (pieces of flat buffers) is stepped over; 8-bit blocks start at element 0
        bool vec = vector_from<OP>(t, other, 0);
        uint32_t head = 0;
        if (OP == Op::kAdamw && UNIT == kUnit && !vec) {
            for (uint32_t h = 1; h < 8 && !vec; ++h)
                if (vector_from<OP>(t, other, h)) {
                    vec = true;
                    head = h;
                }
        }
        const uint64_t body = t.elems > head ? t.elems - head : 1;
        const uint64_t c = (body + UNIT - 1) / UNIT;
        if (units + c > 0xf0000000ull)
            break;  // unit counters are 32-bit; check_tensor bounds one tensor's units
        Ref& r = l.t[filled];
        r.m = t.m;
        r.v = t.v;
        r.exps = t.exps;
        r.elems = t.elems;
        uint32_t flags = vec ? kVector : 0;
        if (is_codec(OP)) {
            r.x = other->m;
            r.y = other->v;
            flags |= other->state_dtype == ZERO_BF16 ? kValueBF16 : 0;
        } else {
            r.grad = t.grad;
            r.master = t.master;
            r.params = t.params;
            r.lr_scale = t.lr_scale;
            r.decay = (float)(1.0 - (double)hp->lr * (double)t.lr_scale * (double)t.weight_decay);
            flags |= t.grad_dtype;
            flags |= (t.params_dtype ? t.params_dtype : hp->params_dtype) == ZERO_F16 ? kOutF16 : 0;
        }
        r.flags = flags;
        if (OP == Op::kAdamw)
            r.head = head;
        else
            r.group0 = group0;
        group0 += (uint32_t)((t.elems + kUnit - 1) / kUnit) * 32u;
        units += c;
        l.end[filled++] = (uint32_t)units;
    }
    for (uint32_t k = filled; k < (uint32_t)kLarge && k % 4; ++k)
        l.end[k] = ~0u;  // read with the last tensors', never at or below a unit's number
    l.n = filled;
    l.n_units = (uint32_t)units;
    return next;
}

/* The same list in the small form. */
void shrink(const List<kLarge>& from, List<kSmall>& to)
{
    to.n = from.n;
    to.n_units = from.n_units;
    memcpy(to.end, from.end, sizeof to.end);
    memcpy(to.t, from.t, from.n * sizeof(Ref));
}

int status_of(cudaError_t e)
{
    if (e == cudaSuccess)
        return ZERO_OK;
    record_cuda_error((int)e);
    return ZERO_ECUDA;
}

/* A launch over `units` units, a warp each, on at most as many blocks as fit at once. */
template <typename Args>
int launch_units(void (*kernel)(Args), std::atomic<int> (&per_sm)[64], uint32_t units, cudaStream_t s,
                 const Args& a)
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
    const uint64_t want = ((uint64_t)units + kWarps - 1) / kWarps, cap = (uint64_t)sm_count() * (uint64_t)occ;
    return status_of(launch_pdl(kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(kThreads), 0, s, a));
}

/* The staged form: one block per SM. */
template <bool S8, int CAP>
int launch_ring(const ListArgs<CAP>& a, cudaStream_t s)
{
    static std::atomic<bool> configured[64];  // per device; a race only repeats the set-up
    int dev = 0;
    cudaGetDevice(&dev);
    if (!configured[dev & 63].load(std::memory_order_relaxed)) {
        const cudaError_t e = cudaFuncSetAttribute(k_tensors_ring<S8, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)Ring<S8>::kSmem);
        if (e != cudaSuccess)
            return status_of(e);
        configured[dev & 63].store(true, std::memory_order_relaxed);
    }
    const uint32_t cap = (uint32_t)sm_count(), want = a.l.n_units;
    return status_of(launch_pdl(k_tensors_ring<S8, CAP>, dim3(want < cap ? want : cap), dim3(Ring<S8>::kThreads),
                                Ring<S8>::kSmem, s, a));
}

/* One launch of an operator over its part of the list. */
template <Op OP, bool RING, int CAP>
int launch_op(const ListArgs<CAP>& a, cudaStream_t s)
{
    static std::atomic<int> occ[64];  // per device; a race only repeats the set-up
    if constexpr (RING)
        return launch_ring<OP == Op::kAdamw8>(a, s);
    else if constexpr (OP == Op::kAdamw)
        return launch_units(k_tensors_adamw<CAP>, occ, a.l.n_units, s, a);
    else if constexpr (OP == Op::kAdamw8)
        return launch_units(k_tensors_adamw8<CAP>, occ, a.l.n_units, s, a);
    else if constexpr (OP == Op::kRead)
        return launch_units(k_state8_read<CAP>, occ, a.l.n_units, s, a);
    else
        return launch_units(k_state8_write<CAP>, occ, a.l.n_units, s, a);
}

template <Op OP, bool RING>
int run_list(const zero_tensor_t* tensors, const zero_tensor_t* others, uint64_t n,
             const zero_adamw_hparams_t* hp, uint64_t seed, const zero_step_state_t* st, cudaStream_t s)
{
    constexpr uint32_t kElems = !RING ? kUnit : Ring<OP == Op::kAdamw8>::kChunk;
    ListArgs<kLarge> a;
    a.st = st;
    a.seed = seed;
    a.beta1 = hp ? hp->beta1 : 0.0f;
    a.beta2 = hp ? hp->beta2 : 0.0f;
    a.eps = hp ? hp->eps : 0.0f;
    uint32_t group0 = 0;
    for (uint64_t next = 0; next < n;) {
        next = fill<OP, kElems>(a.l, tensors, others, n, next, hp, group0);
        if (a.l.n == 0)
            continue;
        int rc;
        if (a.l.n <= (uint32_t)kSmall) {
            ListArgs<kSmall> b;
            b.st = a.st;
            b.seed = a.seed;
            b.beta1 = a.beta1;
            b.beta2 = a.beta2;
            b.eps = a.eps;
            shrink(a.l, b.l);
            rc = launch_op<OP, RING>(b, s);
        } else {
            rc = launch_op<OP, RING>(a, s);
        }
        if (rc != ZERO_OK)
            return rc;
    }
    return ZERO_OK;
}

/* Lists of this many elements take the staged kernel.  Measured, direct against staged, us a
 * launch (32-bit states; 8-bit): 2^20 elements 5.3 / 8.9 (4.2 / 7.1), 2^22 21.8 / 22.7
 * (14.8 / 15.1), 2^23 41.0 / 39.7 (25.9 / 24.7), 2^24 78.7 / 73.0 (51.0 / 43.8). */
constexpr uint64_t kRingElems = 3ull << 21;

template <Op OP>
int adamw_list(const zero_tensor_t* tensors, uint64_t n, const zero_adamw_hparams_t* hp, uint64_t seed,
               const zero_step_state_t* st, cudaStream_t s)
{
    uint64_t total;
    const int rc = check_list<OP>(tensors, nullptr, n, total);
    if (rc == ZERO_EINVAL || !hparams_ok(hp) || !st)
        return ZERO_EINVAL;
    if (rc != ZERO_OK || !at(st, 16))
        return ZERO_EALIGN;
    return total >= kRingElems ? run_list<OP, true>(tensors, nullptr, n, hp, seed, st, s)
                               : run_list<OP, false>(tensors, nullptr, n, hp, seed, st, s);
}

template <Op OP>
int codec_list(const zero_tensor_t* t8, const zero_tensor_t* t32, uint64_t n, cudaStream_t s)
{
    uint64_t total;
    const int rc = check_list<OP>(t8, t32, n, total);
    return rc != ZERO_OK ? rc : run_list<OP, false>(t8, t32, n, nullptr, 0, nullptr, s);
}

/* The norm's launches: a list in its parameters' form, then equal shares for the blocks. */
template <int CAP>
uint64_t fill_norm(NormArgs<CAP>& a, const zero_tensor_t* tensors, uint64_t n, uint64_t next)
{
    uint64_t end = 0;
    uint32_t filled = 0;
    for (; next < n && filled < (uint32_t)CAP; ++next) {
        const zero_tensor_t& t = tensors[next];
        if (t.elems == 0)
            continue;
        const uint32_t shift = t.grad_dtype == ZERO_F32 ? 2 : 1;  // log2 of the element's size
        NormRef& r = a.t[filled++];
        const uintptr_t off = (uintptr_t)t.grad & 15u;
        r.base = static_cast<const char*>(t.grad) - off;
        r.skip = (uint32_t)(off >> shift);
        r.elems = t.elems;
        r.dtype = t.grad_dtype;
        end += (((r.skip + t.elems) << shift) + 15) >> 4;
        r.end = end;
    }
    a.n = filled;
    return next;
}

template <int CAP>
int run_norm(const zero_tensor_t* tensors, uint64_t n, const zero_adamw_hparams_t* hp, double* workspace,
             zero_step_state_t* st, cudaStream_t s)
{
    NormArgs<CAP> a;
    a.st = st;
    a.slots = workspace;
    a.hp = *hp;
    a.slot0 = 0;
    const uint64_t cap = (uint64_t)sm_count() * kNormBlocksPerSm, blocks = cap < kNormMaxBlocks ? cap : kNormMaxBlocks;
    uint64_t next = 0;
    do {
        next = fill_norm(a, tensors, n, next);
        a.last = next == n;
        // equal shares, in whole passes of a block's loads; short lists one load per thread
        const uint64_t total = a.n ? a.t[a.n - 1].end : 0;
        const uint64_t pass = total <= blocks * kNormPass ? kThreads : kNormPass;
        a.quota = ((total + blocks - 1) / blocks + pass - 1) / pass * pass;
        const unsigned grid = total ? (unsigned)((total + a.quota - 1) / a.quota) : 0u;
        const cudaError_t e = launch_pdl(k_tensors_norm<CAP>, dim3(grid + a.last), dim3(kThreads), 0, s, a);
        if (e != cudaSuccess)
            return status_of(e);
        a.slot0 += grid;
    } while (next < n);
    return ZERO_OK;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" size_t zero_tensors_workspace_bytes(uint64_t n_tensors)
{
    const uint64_t launches = n_tensors / kNormCap + 1;
    return (size_t)(launches * kNormMaxBlocks * sizeof(double) + 64);
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
    uint64_t total;
    const int rc = check_list<Op::kNorm>(tensors, nullptr, n_tensors, total);
    if (rc == ZERO_EINVAL || !hparams_ok(hp) || !workspace || !st)
        return ZERO_EINVAL;
    if (rc != ZERO_OK || !at(workspace, 16) || !at(st, 16))
        return ZERO_EALIGN;
    return n_tensors <= (uint64_t)kSmall
               ? run_norm<kSmall>(tensors, n_tensors, hp, workspace, st, (cudaStream_t)stream)
               : run_norm<kNormCap>(tensors, n_tensors, hp, workspace, st, (cudaStream_t)stream);
}

extern "C" int zero_tensors_adamw(const zero_tensor_t* tensors, uint64_t n_tensors,
                                  const zero_adamw_hparams_t* hp, const zero_step_state_t* st,
                                  zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_adamw");
    return adamw_list<Op::kAdamw>(tensors, n_tensors, hp, 0, st, (cudaStream_t)stream);
}

extern "C" int zero_tensors_adamw8(const zero_tensor_t* tensors, uint64_t n_tensors,
                                   const zero_adamw_hparams_t* hp, uint64_t seed,
                                   const zero_step_state_t* st, zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_adamw8");
    return adamw_list<Op::kAdamw8>(tensors, n_tensors, hp, seed, st, (cudaStream_t)stream);
}

extern "C" int zero_tensors_state8_read(const zero_tensor_t* from, const zero_tensor_t* to,
                                        uint64_t n_tensors, zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_state8_read");
    return codec_list<Op::kRead>(from, to, n_tensors, (cudaStream_t)stream);
}

extern "C" int zero_tensors_state8_write(const zero_tensor_t* to, const zero_tensor_t* from,
                                         uint64_t n_tensors, zero_stream_t stream)
{
    const NvtxRange range("zero_tensors_state8_write");
    return codec_list<Op::kWrite>(to, from, n_tensors, (cudaStream_t)stream);
}
