/*
 * tensors.cuh -- lists of tensors: a launch's part of the list, how a warp finds its unit in
 * it, and the checks and launches shared by the operators over lists (tensors_norm.cu,
 * tensors_adamw.cu, tensors_codec.cu).
 *
 * The tensors lie where the caller's model has them.  Each launch carries its part of the
 * list by value in the kernel's parameters (up to 32 KB of constant memory), so a call
 * needs no device table, nothing is kept from one call for the next, and a captured graph
 * holds the list it was captured with.  The list is cut into units of a fixed number of
 * elements; `end[k]` counts the units up to and including tensor k's.
 */
#pragma once

#include "adamw_elem.cuh"
#include "reduce_elem.cuh"
#include "state8.cuh"

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
constexpr uint32_t kVector = 8;      // every array allows one access per 8 elements (past `head`)
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
        uint32_t head;    // 32-bit states: elements before the arrays' common boundary
    };
};

/* A launch's part of the list.  Kernel parameters may be 32,764 bytes, which bounds the
 * large form; lists of up to 32 tensors take the small one, 2.5 KB to hand over instead of
 * 32 (measured: a norm call on 16 tensors costs the host 3.9 us with it, 5.5 without). */
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
 * all in flight at once.  They go through global addressing of the parameters (the asm hides
 * where the address comes from): a binary search in constant memory would miss its cache
 * once per step on a launch's first unit. */
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

/* Loads of what an earlier launch may have written.  A kernel over a list works out its
 * first addresses before grid_dependency_wait(): volatile keeps these loads behind the wait
 * (and the norm's behind its arrival), in the order written.  They do not take the read-only
 * path (.nc): its promise, that nothing writes while the kernel runs, does not hold for a
 * kernel that starts before its predecessor ends. */
__device__ __forceinline__ uint4 ld_list_v4(const void* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ uint2 ld_list_v2(const void* p)
{
    uint2 v;
    asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ uint16_t ld_list_u16(const void* p)
{
    unsigned short v;
    asm volatile("ld.global.L1::no_allocate.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ float ld_list_f32(const float* p)
{
    float v;
    asm volatile("ld.global.cs.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ float one_grad(const void* g, uint64_t i, uint32_t dtype)
{
    if (dtype == ZERO_F32)
        return ld_list_f32(static_cast<const float*>(g) + i);
    const uint16_t b = ld_list_u16(static_cast<const uint16_t*>(g) + i);
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

__device__ __forceinline__ bool whole_unit(const Ref& t, uint32_t unit)
{
    return (t.flags & kVector) && ((uint64_t)unit + 1) * kUnit <= t.elems;
}

/* ------------------------------------------------------------------------------------ */
/* host side                                                                              */
/* ------------------------------------------------------------------------------------ */

inline bool finite_f(float x) { return x == x && x <= 3.4e38f && x >= -3.4e38f; }

inline bool at(const void* p, uintptr_t align) { return ((uintptr_t)p & (align - 1)) == 0; }

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
inline void shrink(const List<kLarge>& from, List<kSmall>& to)
{
    to.n = from.n;
    to.n_units = from.n_units;
    memcpy(to.end, from.end, sizeof to.end);
    memcpy(to.t, from.t, from.n * sizeof(Ref));
}

inline int status_of(cudaError_t e)
{
    if (e == cudaSuccess)
        return ZERO_OK;
    record_cuda_error((int)e);
    return ZERO_ECUDA;
}

/* launch_pdl for a kernel whose one argument is large: handed over where it lies (a call by
 * value would copy the 32 KB once more). */
template <typename Args>
cudaError_t launch_args(void (*kernel)(Args), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                        const Args& a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    void* args[1] = {const_cast<Args*>(&a)};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), args);
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
    return status_of(launch_args(kernel, (unsigned)(want < cap ? want : cap), kThreads, 0, s, a));
}

/* Runs an operator over the list, in units of UNIT elements and in as many launches as it
 * takes: launch(args) makes one, with its part of the list in the small or the large form. */
template <Op OP, uint32_t UNIT, typename Launch>
int run_list(const zero_tensor_t* tensors, const zero_tensor_t* others, uint64_t n,
             const zero_adamw_hparams_t* hp, uint64_t seed, const zero_step_state_t* st, Launch launch)
{
    ListArgs<kLarge> a;
    a.st = st;
    a.seed = seed;
    a.beta1 = hp ? hp->beta1 : 0.0f;
    a.beta2 = hp ? hp->beta2 : 0.0f;
    a.eps = hp ? hp->eps : 0.0f;
    uint32_t group0 = 0;
    for (uint64_t next = 0; next < n;) {
        next = fill<OP, UNIT>(a.l, tensors, others, n, next, hp, group0);
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
            rc = launch(b);
        } else {
            rc = launch(a);
        }
        if (rc != ZERO_OK)
            return rc;
    }
    return ZERO_OK;
}

}  // namespace
}  // namespace zero
