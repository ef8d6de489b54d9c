/*
 * tensors_norm.cu -- global gradient norm over a list of tensors: loss-scale removal,
 * overflow check, norm, clip coefficient and the step's scalars (the Megatron
 * distributed-optimizer page, sec. 1: one norm before clipping).
 *
 * norm = sqrt(sum of (x * inv)^2) over every gradient element x.  Nothing but a read of the
 * gradients, 2 or 4 bytes an element, so it is bound by HBM: GPT-2 1.5B's 580 bf16
 * gradients (3.1 GB) take 440 to 450 us, by the card, 104-106% of the measured copy peak
 * (6,669 GB/s); a short list takes 7 us, most of it the blocks' arrival and the fp64 chain
 * behind it.  What that took:
 *   - each gradient is a run of 16-byte granules at the addresses' own multiples of 16, so
 *     every tensor moves in 128-bit loads whatever its alignment and only a first and a
 *     last granule can be partial (a sum does not care which lane holds what);
 *   - every block takes an equal share of the launch's granules, across tensor boundaries
 *     (chunks of 8192 elements handed out in turn, each looked up anew: 1,068 us);
 *   - 8 loads in flight per thread in 3 blocks per SM (4 blocks 464 us, with spills; 16
 *     loads in 2 blocks 456);
 *   - a pass that crosses tensors looks each granule's tensor up on its own, so a run of
 *     short tensors costs one memory latency and not one each;
 *   - squares in fp32, two at a time, in sums of 8; the sums joined by error-free additions;
 *     fp64 only per block and for values whose squares fp32 cannot hold.
 */
#include "tensors.cuh"
#include "step_scalars.cuh"

namespace zero {
namespace {

constexpr int kNormLoads = 8;                // 128-bit loads in flight per thread
constexpr uint32_t kNormPass = kThreads * kNormLoads;
constexpr uint32_t kNormMaxBlocks = 2048;    // slots per launch
constexpr int kNormBlocksPerSm = 3;

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
 * 6).  Granules whose sum leaves fp32's safe range are summed in fp64: below 2^-120, where
 * what underflows could reach 2^-27 of it, or from 2^100 up, which an infinity, a NaN and a
 * square that overflows exceed too.  Below that hi stays finite over 2^27 granules and more;
 * a thread's share of gradients that fill the GPU's memory is 2^18. */
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

    /* floor: 2^-120, or infinity where 1/(N*L) is so large that a finite gradient could
     * unscale to infinity (then every granule is looked at element by element) */
    template <uint32_t DT>
    __device__ __forceinline__ void granule(const uint4& w, float inv, float floor)
    {
        if (DT == ZERO_F32) {
            const float x0 = __uint_as_float(w.x), x1 = __uint_as_float(w.y);
            const float x2 = __uint_as_float(w.z), x3 = __uint_as_float(w.w);
            const float s = __fadd_rn(__fmaf_rn(x0, x0, __fmul_rn(x1, x1)),
                                      __fmaf_rn(x2, x2, __fmul_rn(x3, x3)));
            if (s < 0x1p100f && s > floor) {
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
            if (s < 0x1p100f && s > floor) {
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
                w[e >> 1] |= (uint32_t)ld_list_u16(t.base + i * 2) << (16 * (e & 1));
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

/* Granule j of tensor t, whole or partial. */
__device__ __forceinline__ uint4 any_granule(const NormRef& t, uint64_t j)
{
    const uint64_t n = t.dtype == ZERO_F32 ? 4 : 8;
    if (j * n >= t.skip && (j + 1) * n <= t.skip + t.elems)
        return ld_list_v4(t.base + j * 16);
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
            w[q] = ld_list_v4(p + q * kThreads * 16);
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

/* What other blocks of this launch have written, read past L1 after their arrival. */
__device__ __forceinline__ uint32_t ld_other(const uint32_t* p)
{
    uint32_t x;
    asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
    return x;
}

__device__ __forceinline__ float ld_other(const float* p)
{
    return __uint_as_float(ld_other(reinterpret_cast<const uint32_t*>(p)));
}

__device__ __forceinline__ double ld_other(const double* p)
{
    double x;
    asm volatile("ld.global.cg.f64 %0, [%1];" : "=d"(x) : "l"(p) : "memory");
    return x;
}

/* Adds v over the block in a fixed order: a shuffle tree per warp, then one over the warps'
 * sums.  Valid in warp 0. */
__device__ __forceinline__ double block_sum(double v, double* warp_sum)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0)
        warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = threadIdx.x < kWarps ? warp_sum[threadIdx.x] : 0.0;
#pragma unroll
        for (int o = kWarps / 2; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
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
    const float floor = inv < 0x1p60f ? 0x1p-120f : __int_as_float(0x7f800000);
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
    // arrival: thread 0 has written the block's sum itself, and block_sum's barrier came
    // after every thread's overflow flag (the scalar block has a barrier of its own)
    if (blockIdx.x == n_sum)
        __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t before;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(&st->arrivals) : "memory");
        is_last = before == gridDim.x - 1;
    }
    __syncthreads();
    if (!is_last)
        return;
    double v = 0.0;
    for (uint32_t i = threadIdx.x; i < a.slot0 + n_sum; i += kThreads)
        v += ld_other(a.slots + i);
    const uint32_t overflow = ld_other(&st->overflow) != 0;
    const double sumsq = block_sum(v, warp_sum) * ((double)inv * (double)inv);
    // block_sum's barrier: every thread has read the overflow flag
    if (threadIdx.x == 32) {
        const ScalerCand cand{ld_other(&ready->cand.L_skip), ld_other(&ready->cand.inv_skip),
                              ld_other(&ready->cand.L_ok), ld_other(&ready->cand.inv_ok),
                              ld_other(&ready->cand.good_ok), ld_other(&ready->cand.decay)};
        scaler_apply(st, cand, overflow, st->t + 1);
        if (!overflow) {
            st->step_size = ld_other(&ready->step_size);
            st->rbc2 = ld_other(&ready->rbc2);
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
        const cudaError_t e = launch_args(k_tensors_norm<CAP>, grid + a.last, kThreads, 0, s, a);
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
