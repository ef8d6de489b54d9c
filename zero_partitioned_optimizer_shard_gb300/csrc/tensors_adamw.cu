/*
 * tensors_adamw.cu -- AdamW over a list of tensors, with 32-bit and with 8-bit states, and
 * the cast into the 16-bit parameters (the operatorworld ZeRO article: AdamW, bf16 weights).
 *
 * Per element, in fp32 (include/zero.h has the definitions): g = x * inv, gc = c * g, both
 * moments, and the parameter; 32-bit states through the flat step's own element function,
 * so that the same tensors give the same bits either way.
 *
 * Both are bound by HBM: 28 bytes an element with 32-bit states and bf16 gradients, 16 with
 * 8-bit states.  Two forms of each:
 *   direct   a warp per 256-element unit, straight from and to global memory.  For short
 *            lists, where a memory latency or two is all there is: 16,384 elements take 2.8
 *            us (8-bit states 2.4), a million 5.1 (4.2).
 *   staged   one block per SM; a producer warp bulk-copies chunks into a ring in shared
 *            memory, consumer warps compute (k_tensors_ring).  For long lists: GPT-2
 *            1.5B's 580 tensors take 6,146 us with 32-bit states (106% of the measured copy
 *            peak; the direct form 6,929) and 3,552 us with 8-bit states (105%; 4,122).
 */
#include "tensors.cuh"

namespace zero {
namespace {

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

/* A parameter's update from its new moments, as adamw_one (adamw_elem.cuh) has it, bit for
 * bit.  ANY: without the slow ways of fp32 division and square root, which are taken for
 * zeros and for operands near fp32's lower end.  That is what the rows of an embedding that
 * saw no token hold: m = v = 0, or an m that has decayed into the subnormals; with half of
 * 400 million elements so, the plain form took 2,665 us; this one takes 1,582, as long as
 * other values do.
 *   sqrt(v)        below 2^-100: sqrt(v * 2^64) * 2^-32, both factors exact and no result
 *                  subnormal; for v = 0 any operand, and 0 put in its place after the division;
 *                  a v < 0 gives NaN either way
 *   step * (m / d) r = m where m = 0 (the same signed zero); and where |m| < tiny and
 *                  |p| >= 2^-40: tiny is 2^-110 where step <= 2^40 eps, so that the true
 *                  value lies below 2^-70, under a quarter of p's last place, as does m: p - r
 *                  is p either way.  The division gets 1 for m there. */
template <bool ANY>
__device__ __forceinline__ float new_param(float p, float m, float v, const Scalars& s, float tiny)
{
    p = __fmul_rn(p, s.decay);
    if (!ANY) {
        const float denom = __fadd_rn(__fdiv_rn(__fsqrt_rn(v), s.rbc2), s.eps);
        return __fsub_rn(p, __fmul_rn(s.step, __fdiv_rn(m, denom)));
    }
    const bool small = fabsf(v) < 0x1p-100f;
    const float up = small ? __fmul_rn(v, 0x1p64f) : v;
    const float root = __fmul_rn(__fsqrt_rn(v == 0.0f ? 1.0f : up), small ? 0x1p-32f : 1.0f);
    const float quotient = __fdiv_rn(root, s.rbc2);
    const float denom = __fadd_rn(v == 0.0f ? 0.0f : quotient, s.eps);
    const bool same = (m == 0.0f || (fabsf(m) < tiny && fabsf(p) >= 0x1p-40f)) && v >= 0.0f;
    const float r = __fmul_rn(s.step, __fdiv_rn(same ? 1.0f : m, denom));
    return __fsub_rn(p, same ? m : r);
}

/* The AdamW update of a lane's N elements with gradients x * inv: the moments, and the
 * parameters in the form that the whole warp's values allow (ANY costs 13 instructions an
 * element more: 4% on misaligned pieces). */
template <int N>
__device__ __forceinline__ void adamw_list_elems(const float (&x)[N], float inv, float (&p)[N], float (&m)[N],
                                                 float (&v)[N], const Scalars& s, float tiny)
{
    float low = 1.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float gc = __fmul_rn(s.c, __fmul_rn(x[e], inv));
        m[e] = __fadd_rn(__fmul_rn(s.b1, m[e]), __fmul_rn(s.omb1, gc));
        v[e] = __fadd_rn(__fmul_rn(s.b2, v[e]), __fmul_rn(s.omb2, __fmul_rn(gc, gc)));
        low = fminf(low, fminf(fabsf(m[e]), v[e]));
    }
    if (__any_sync(0xffffffffu, low < 0x1p-100f)) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            p[e] = new_param<true>(p[e], m[e], v[e], s, tiny);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            p[e] = new_param<false>(p[e], m[e], v[e], s, tiny);
    }
}

/* Below this |m| the update leaves a parameter of 2^-40 or more as it is (new_param). */
__device__ __forceinline__ float tiny_moment(float step, float eps)
{
    return step <= __fmul_rn(eps, 0x1p40f) ? 0x1p-110f : 0.0f;
}

/* ------------------------------------------------------------------------------------ */
/* short lists: straight from global memory                                               */
/* ------------------------------------------------------------------------------------ */

/* A lane's 8 gradients as they lie in memory. */
struct RawGrad {
    float w[8];  // 16-bit gradients: the first four words

    __device__ __forceinline__ void load(const void* g, uint64_t i, uint32_t dtype)
    {
        if (dtype == ZERO_F32) {
            load8(static_cast<const float*>(g) + i, w);
        } else {
            const uint4 a = ld_list_v4(static_cast<const uint16_t*>(g) + i);
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
        const float tiny = tiny_moment(s.step, s.eps);
        const bool vec = t.flags & kVector;
        const uint64_t off = t.head + (uint64_t)at.unit * kUnit;
        // 8 consecutive elements per lane, one access an array; else lanes side by side
        const uint64_t i = vec ? off + lane * kPer : off + lane;
        const uint32_t stride = vec ? 1 : 32;
        float x8[8], p8[8], m8[8], v8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)  // what lanes past the end compute with: ordinary values
            x8[e] = p8[e] = m8[e] = v8[e] = 1.0f;
        RawGrad raw;
        const bool whole = vec && i + kPer <= t.elems;
        if (whole) {
            raw.load(t.grad, i, dtype);
            load8(t.master + i, p8);
            load8(m + i, m8);
            load8(v + i, v8);
        } else if (i < t.elems) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint64_t q = i + e * stride;
                const bool in = q < t.elems;
                x8[e] = in ? one_grad(t.grad, q, dtype) : 1.0f;
                p8[e] = in ? ld_list_f32(t.master + q) : 1.0f;
                m8[e] = in ? ld_list_f32(m + q) : 1.0f;
                v8[e] = in ? ld_list_f32(v + q) : 1.0f;
            }
        }
        if (whole)  // only here: inside the branch above they would wait for its loads
            raw.values(dtype, x8);
        if (skip)  // only now: the loads need not wait for the state's
            return;
        adamw_list_elems(x8, inv, p8, m8, v8, s, tiny);
        if (whole) {
            store8(t.master + i, p8);
            store8(m + i, m8);
            store8(v + i, v8);
            if (t.params)
                store_params8(t.params + i, t.flags & kOutF16, p8);
        } else if (i < t.elems) {
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
        if (at.unit == 0 && t.head) {  // before the common boundary: an element each
            const bool in = lane < t.head && lane < t.elems;
            float x1[1] = {in ? one_grad(t.grad, lane, dtype) : 1.0f}, p1[1] = {in ? t.master[lane] : 1.0f};
            float m1[1] = {in ? m[lane] : 1.0f}, v1[1] = {in ? v[lane] : 1.0f};
            adamw_list_elems(x1, inv, p1, m1, v1, s, tiny);
            if (in) {
                t.master[lane] = p1[0];
                m[lane] = m1[0];
                v[lane] = v1[0];
                if (t.params)
                    t.params[lane] = (t.flags & kOutF16) ? pack1<true>(p1[0]) : pack1<false>(p1[0]);
            }
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
                // the quotient first: step * m would lose bits among the subnormals
                const uint64_t q = f2_mul(f2_mul(m2, f2(rcp_fast(d0), rcp_fast(d1))), step2);
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
        const bool vec = t.flags & kVector;
        // 8 consecutive elements per lane, one access an array; else lanes side by side
        const uint64_t i = (uint64_t)unit * kUnit + (vec ? lane * kPer : lane);
        const uint32_t apart = vec ? 1 : 32;
        const bool full = vec && i + kPer <= t.elems;
        uint8_t* m = static_cast<uint8_t*>(t.m) + i;
        uint8_t* v = static_cast<uint8_t*>(t.v) + i;
        uint8_t* exps = t.exps + 2 * (uint64_t)unit;
        uint32_t bm = exps[0], bv = exps[1];
        uint2 cm = make_uint2(0, 0), cv = cm;
        float x[8], p[8], ym[8], yv[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)  // past the end: zeros do not count in the exponents
            x[e] = p[e] = 0.0f;
        RawGrad raw;
        if (full) {
            raw.load(t.grad, i, dtype);
            load8(t.master + i, p);
            cm = ld_list_v2(m);
            cv = ld_list_v2(v);
        } else if (i < t.elems) {
            uint32_t am[8], av[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = i + e * apart < t.elems;
                x[e] = in ? one_grad(t.grad, i + e * apart, dtype) : 0.0f;
                p[e] = in ? ld_list_f32(t.master + i + e * apart) : 0.0f;
                am[e] = in ? m[e * apart] : 0u;
                av[e] = in ? v[e * apart] : 0u;
            }
            cm = make_uint2(am[0] | am[1] << 8 | am[2] << 16 | am[3] << 24, am[4] | am[5] << 8 | am[6] << 16 | am[7] << 24);
            cv = make_uint2(av[0] | av[1] << 8 | av[2] << 16 | av[3] << 24, av[4] | av[5] << 8 | av[6] << 16 | av[7] << 24);
        }
        if (full)  // only here: inside the branch above they would wait for its loads
            raw.values(dtype, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ym[e] = raw_m(e < 4 ? cm.x : cm.y, e & 3);
            yv[e] = raw_v(e < 4 ? cv.x : cv.y, e & 3);
        }
        if (skip)
            return;
        // lane L's seed is that of the block's group L
        const uint32_t seed = mix32(s.key + (t.group0 + unit * 32 + lane) * kGolden);
        if (vec)
            block8(x, p, ym, yv, bm, bv, RandomInGroup{seed}, cm, cv, s);
        else
            block8(x, p, ym, yv, bm, bv, RandomAcross(seed, lane), cm, cv, s);
        if (full) {
            store8(t.master + i, p);
            if (t.params)
                store_params8(t.params + i, t.flags & kOutF16, p);
            __stcs(reinterpret_cast<uint2*>(m), cm);
            __stcs(reinterpret_cast<uint2*>(v), cv);
        } else if (i < t.elems) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (i + e * apart < t.elems) {
                    m[e * apart] = (uint8_t)((e < 4 ? cm.x : cm.y) >> (8 * (e & 3)));
                    v[e * apart] = (uint8_t)((e < 4 ? cv.x : cv.y) >> (8 * (e & 3)));
                    __stcs(t.master + i + e * apart, p[e]);
                    if (t.params)
                        t.params[i + e * apart] = (t.flags & kOutF16) ? pack1<true>(p[e]) : pack1<false>(p[e]);
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
/* long lists: staged through shared memory                                               */
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
    /* Without an L2 policy: an evict-first one, which the flat kernel gains from, cost 2% on
     * misaligned pieces (176 against 180 us; neighbouring chunks share their end granules)
     * and gained nothing on large lists. */
    __device__ __forceinline__ void bulk(uint32_t bar) const
    {
        if (len)
            bulk_load<false>(dst, from, len, bar);
    }
};

#ifdef ZERO_TEST_HOOKS
/* Test builds only (never the product library): the chunk whose copies are withheld, so that
 * the waits on its stage run out without any fault. */
__device__ unsigned long long zero_test_withheld_tensors_chunk = ~0ull;
#endif

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
#ifdef ZERO_TEST_HOOKS
            if (c == zero_test_withheld_tensors_chunk)
                continue;
#endif
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
            const float tiny = tiny_moment(s.step, s.eps);
            adamw_list_elems(x, inv, p, m, v, s, tiny);
            u.put(t.out_m, m);
            u.put(t.out_v, v);
        }
        u.put(t.out_master, p);
        if (t.out_params)
            u.put_params(t.out_params, t.flags & kOutF16, p);
    }
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
    return status_of(launch_args(k_tensors_ring<S8, CAP>, want < cap ? want : cap, Ring<S8>::kThreads,
                                 Ring<S8>::kSmem, s, a));
}

/* Lists of this many elements, and this many per tensor on average, take the staged kernel.
 * Measured, us a call, direct / staged, 32-bit states (8-bit states):
 *   4 tensors     2^20 elements 5.1 / 9.1 (4.2 / 7.1), 2^22 21.8 / 23.1 (14.8 / 15.0),
 *                 2^23 41.2 / 40.4 (25.7 / 25.1), 2^24 79.6 / 73.5 (50.1 / 44.4)
 *   2^25 elements in tensors of 8,192: 172 / 193 (124 / 152), of 16,384: 169 / 168
 *                 (110 / 109), of 65,536: 158 / 149 (106 / 92)
 *   2^23 elements in tensors of 1,024: 89 / 165 (65 / 183): a short tensor leaves most of a
 *                 stage empty */
constexpr uint64_t kRingElems = 3ull << 21, kRingTensor = 1ull << 15;

/* One launch of the direct form. */
template <Op OP, int CAP>
int launch_direct(const ListArgs<CAP>& a, cudaStream_t s)
{
    static std::atomic<int> occ[64];  // per device; a race only repeats the set-up
    return launch_units(OP == Op::kAdamw ? k_tensors_adamw<CAP> : k_tensors_adamw8<CAP>, occ, a.l.n_units, s, a);
}

template <Op OP>
int adamw_list(const zero_tensor_t* tensors, uint64_t n, const zero_adamw_hparams_t* hp, uint64_t seed,
               const zero_step_state_t* st, cudaStream_t s)
{
    constexpr bool kS8 = OP == Op::kAdamw8;
    uint64_t total;
    const int rc = check_list<OP>(tensors, nullptr, n, total);
    if (rc == ZERO_EINVAL || !hparams_ok(hp) || !st)
        return ZERO_EINVAL;
    if (rc != ZERO_OK || !at(st, 16))
        return ZERO_EALIGN;
    if (total >= kRingElems && total >= n * kRingTensor)
        return run_list<OP, Ring<kS8>::kChunk>(tensors, nullptr, n, hp, seed, st,
                                               [s](const auto& a) { return launch_ring<kS8>(a, s); });
    return run_list<OP, kUnit>(tensors, nullptr, n, hp, seed, st,
                               [s](const auto& a) { return launch_direct<OP>(a, s); });
}

}  // namespace
}  // namespace zero

using namespace zero;

#ifdef ZERO_TEST_HOOKS
extern "C" int zero_test_withhold_tensors_chunk(unsigned long long chunk)
{
    return cudaMemcpyToSymbol(zero_test_withheld_tensors_chunk, &chunk, sizeof chunk) == cudaSuccess ? 0 : -4;
}
#endif

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
