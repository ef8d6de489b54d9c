/*
 * tensors_codec.cu -- the 8-bit states' values read out (for a checkpoint, for monitoring),
 * and 32-bit states written into the 8-bit form (a run that changes over).
 *
 * A warp per 256-element unit, which is a block of the 8-bit form: 8 elements per lane, the
 * block's largest magnitude by one warp reduction.  Bound by HBM: reading moves 1 + 1 bytes
 * in and 2 + 2 (bf16) or 4 + 4 out per element, writing 4 + 4 in and 1 + 1 out.  GPT-2
 * 1.5B's states read as bf16 in 1,460 us (96% of the measured copy peak), as fp32 in 2,633
 * (89%); 80 million elements written in 121 us (99%).  The staged form of the AdamW kernels gained nothing
 * here (read 1,760 us, written 120): what reading needs is many warps with stores in
 * flight (32 registers, 64 warps per SM; with 40 and 48 warps 1,572 us).
 */
#include "tensors.cuh"

namespace zero {
namespace {

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
            const uint2 wm = ld_list_v2(cm), wv = ld_list_v2(cv);
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
                m[e] = at + e * 32 < t.elems ? ld_list_f32(xm + e * 32) : 0.0f;
                v[e] = at + e * 32 < t.elems ? ld_list_f32(xv + e * 32) : 0.0f;
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

template <Op OP, int CAP>
int launch_codec(const ListArgs<CAP>& a, cudaStream_t s)
{
    static std::atomic<int> occ[64];  // per device; a race only repeats the set-up
    return launch_units(OP == Op::kRead ? k_state8_read<CAP> : k_state8_write<CAP>, occ, a.l.n_units, s, a);
}

template <Op OP>
int codec_list(const zero_tensor_t* t8, const zero_tensor_t* t32, uint64_t n, cudaStream_t s)
{
    uint64_t total;
    const int rc = check_list<OP>(t8, t32, n, total);
    if (rc != ZERO_OK)
        return rc;
    return run_list<OP, kUnit>(t8, t32, n, nullptr, 0, nullptr, [s](const auto& a) { return launch_codec<OP>(a, s); });
}

}  // namespace
}  // namespace zero

using namespace zero;

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
