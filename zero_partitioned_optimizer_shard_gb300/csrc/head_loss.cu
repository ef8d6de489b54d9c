/*
 * head_loss.cu -- softmax cross entropy of logits = hidden . weight^T over a large vocabulary,
 * with its gradients; the logits are never kept.
 *
 * With l = hidden . weight^T (n tokens by V), f_t = scale * row_scale[t] * loss scale:
 *   lse_t  = log(sum over v of exp(l_tv)),  loss_t = lse_t - l_t,target
 *   D_tv   = f_t * (exp(l_tv - lse_t) - [v = target_t])
 *   dhidden = D . weight,  dweight (+)= D^T . hidden
 * Forward: one product whose epilogue leaves, per token and tile of 128 logits, their maximum
 * and the sum of exponentials below it; a second kernel joins them.  Backward: pieces of the
 * vocabulary.  A piece's logits are formed again, D goes to 16 bits into the workspace, and two
 * products take it from there: dhidden summed in fp32 over the pieces, dweight's rows of the
 * piece whole.  One product more than keeping the logits would need, against n * V * 4 bytes.
 *
 * Tokens without a target are dropped first: the tokens that have one are listed, and unless
 * that is all of them their hidden rows are gathered, so such a token costs nothing and
 * whatever its row holds reaches no sum.
 *
 * D's 16 bits: the products take operands of hidden's type.  f_t goes into D in units of the
 * largest |f_t|, the unit into the products' results: where all f_t are equal D is the softmax
 * less 1 at the target, and nothing of f is rounded (with f inside, f's own rounding would shift
 * every target's share the same way: 2.9e-3 of dweight in one case, 1.7e-3 without).  bf16 has
 * fp32's range; for fp16 the unit is 2^14, so that softmax values down to 2^-28 stay normal
 * numbers.  Each D is rounded once, by at most 2^-8 of its value (bf16) or 2^-11 (fp16): the size
 * of the one rounding of the 16-bit gradients themselves.  Before that it is good to fp32's digits of
 * the softmax, but for the target's: a difference from 1, it is off by what lse is (half a unit, and
 * the roundings of a sum of 1 and a little) and by 2^-22 as well: one or two per cent of it where the
 * target has all but 1e-4 of the softmax.
 */
#include "pad.h"
#include "tcgen05.cuh"

namespace zero {
namespace {

constexpr uint32_t kTileM = 256, kTileN = 256;
constexpr uint32_t kRows = kTileM / 2;  // of a block of the pair
constexpr uint32_t kRingBytes = 192 * 1024;
constexpr uint32_t kMaxRing = 6;
constexpr uint32_t kSumBlocks = 16;     // logits: blocks of 64 that the matrix unit sums by itself
constexpr uint32_t kEpilogueWarps = 8, kThreads = 128 + 32 * kEpilogueWarps;
constexpr uint32_t kOutBytes = 4096;    // of an epilogue warp: 32 rows of 128 bytes
constexpr uint32_t kSmem = kRingBytes + kEpilogueWarps * kOutBytes + 1024;  // and to a 1,024-byte boundary
static_assert(kSmem <= 226 * 1024, "beside the barriers, of 227 KB");
constexpr uint32_t kSms = 152;  // of a GB300: sizes the workspace and the splits
constexpr float kLog2e = 1.4426950408889634f, kMaxFloat = 3.402823466e38f;

/* Head of the workspace. */
struct Header {
    uint32_t valid;  // tokens that have a target
    uint32_t error;  // 1: a bounded wait gave up
    float post;      // the gradients' factor beside D
    uint32_t pad[61];
};
static_assert(sizeof(Header) == 256, "the workspace's head");

/* What a launch forms: the losses' statistics, a piece of D, or both gradients from it. */
enum Mode { kStats, kD, kGrads };
/* The products behind them. */
enum Product { kLogits, kDhidden, kDweight };
/* Along the sum a stage of the ring holds 64 of the logits' and 128 of the gradients' (whose
 * MN-major boxes are 128 of it high): 6 stages of 32 KB, or 3 of 64. */
constexpr uint32_t kLogitsK = 64, kGradsK = 128;

struct ProductArgs {
    CUtensorMap hidden;    // the caller's rows, or (where they cannot be used as they lie) the gathered ones
    CUtensorMap gathered;  // the rows of the tokens that have a target
    CUtensorMap weight;
    CUtensorMap d;         // D's piece
    CUtensorMap out;       // what the launch writes: D's piece, or dhidden's sums
    CUtensorMap out_w;     // and dweight, or its sums
    Header* head;
    uint32_t* state_error;  // the step state's error word, or null
    const int* target;      // [valid]
    const float* factor;    // [valid]
    const float* lse;       // [valid]
    float* target_logit;    // [valid]
    float2* stats;          // [valid][2 * column tiles]
    void* dweight;
    uint32_t rows;          // of the call, with or without a target
    uint32_t rows_pad, dim, dim8, vocab;
    uint32_t v0, cols;      // the piece: columns [v0, v0 + cols) of the vocabulary
    uint32_t piece;
    uint32_t splits;        // dweight: of the sum over the tokens
    uint32_t group;         // row tiles that share a run through the columns
    uint32_t first_piece;   // sums start here
    uint32_t want_h, want_w;
    uint32_t grad_dtype, accumulate;
    uint32_t bulk;          // dweight leaves by bulk copies
};

struct Tile {
    uint32_t m, n, width;  // first row and column, columns
    uint32_t k0, k1;       // blocks of kLogitsK or kGradsK along the sum
    uint32_t split, nt;
    Product product;
};

/* Into how many parts a gradient's sum over k blocks of 128 is cut: few tiles leave SMs without
 * work, and 4 blocks at least are worth a part. */
__host__ __device__ inline uint32_t splits_of(uint32_t tiles, uint32_t k)
{
    const uint32_t want = tiles && tiles < kSms / 2 ? kSms / 2 / tiles : 1, most = k / 4;
    return want < most ? want : most > 0 ? most : 1;
}

/* A product's tiles, known once the number of tokens with a target is. */
template <Product P>
struct Tiles {
    uint32_t mt, nt, units, blocks, splits, group, total;

    __device__ __forceinline__ Tiles(const ProductArgs& a, uint32_t valid)
    {
        const uint32_t m = P == kDweight ? a.cols : valid;
        const uint32_t k = P == kDweight ? valid : P == kDhidden ? a.cols : a.dim;
        const uint32_t n = P == kLogits ? a.cols : a.dim;
        mt = (m + kTileM - 1) / kTileM;
        units = (n + 31) / 32;
        nt = (n + kTileN - 1) / kTileN;
        blocks = P == kLogits ? (k + kLogitsK - 1) / kLogitsK : (k + kGradsK - 1) / kGradsK;
        splits = P == kDhidden ? splits_of(mt * nt, blocks) : P == kDweight ? a.splits : 1;
        group = a.group;
        total = mt * nt * splits;
    }

    __device__ __forceinline__ Tile at(uint32_t t) const
    {
        Tile r;
        uint32_t m, n;
        r.product = P;
        r.split = t / (mt * nt);
        t -= r.split * mt * nt;
        if (P == kLogits) {
            // a group's rows of hidden stay in L2 while the columns pass once
            const uint32_t g = t / (group * nt), first = g * group, in = mt - first < group ? mt - first : group;
            t -= g * group * nt;
            n = t / in;
            m = first + t - n * in;
        } else {
            m = t / nt;  // D's tile is read once for all its columns
            n = t - m * nt;
        }
        r.m = m * kTileM;
        if (P == kLogits) {
            r.n = n * kTileN;
            r.width = kTileN;
        } else {  // dim in equal tiles, to a multiple of 32
            r.n = units * n / nt * 32;
            r.width = units * (n + 1) / nt * 32 - r.n;
        }
        r.nt = n;
        r.k0 = (uint32_t)((uint64_t)blocks * r.split / splits);
        r.k1 = (uint32_t)((uint64_t)blocks * (r.split + 1) / splits);
        return r;
    }
};

/* A launch's tiles. */
template <Mode MODE>
struct Work {
    Tiles<kLogits> logits;
    uint32_t total;
    __device__ __forceinline__ Work(const ProductArgs& a, uint32_t valid) : logits(a, valid), total(logits.total) {}
    __device__ __forceinline__ Tile at(uint32_t i) const { return logits.at(i); }
};
template <>
struct Work<kGrads> {
    Tiles<kDhidden> h;
    Tiles<kDweight> w;
    uint32_t first_w, total;
    __device__ __forceinline__ Work(const ProductArgs& a, uint32_t valid)
        : h(a, valid), w(a, valid), first_w(a.want_h ? h.total : 0), total(first_w + (a.want_w ? w.total : 0))
    {
    }
    __device__ __forceinline__ Tile at(uint32_t i) const { return i < first_w ? h.at(i) : w.at(i - first_w); }
};

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // within 2 ulp, far below the 16 bits it ends in
    return y;
}

/* What a row's exponentials are taken relative to, its maximum; of a row of -inf anything will do,
 * exp gives 0.  It is subtracted before log2(e) goes in: near the maximum that is exact, whatever the
 * logits' size, and the maximum's own exponential is 1, so that a sum is 1 at least and its logarithm
 * not negative.  (x * log2(e) - round(maximum * log2(e)) in one instruction has the rounding of a number
 * of the logits' size in every exponent: lse off by 5.7e-5 at logits of 110, and losses below 0.) */
__device__ __forceinline__ float reference(float top) { return top == __int_as_float(0xff800000) ? 0.0f : top; }

struct Shared {
    uint64_t full[kMaxRing], empty[kMaxRing], acc_full[2], acc_empty[2], drain;
    uint32_t tmem, gave_up;
};

/* The part of a tile that one warp of the epilogue has: 32 rows, 128 of the columns (half). */
struct Part {
    uint32_t acc;   // tensor memory address
    uint32_t row;   // this thread's row
    uint32_t half;
    uint32_t stage, lane;
    bool empty;     // no block along the sum: zeros
};

__device__ __forceinline__ void load_part(const Part& p, uint32_t c, float (&x)[32])
{
    if (p.empty) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            x[j] = 0.0f;
    } else {
        tmem_load32(p.acc + c, x);
    }
}

/* x: the row's 128 logits of the tile. */
__device__ __forceinline__ void stats_epilogue(const ProductArgs& a, const Tile& t, const Part& p, uint32_t valid,
                                               float (&x)[4][32])
{
    const float none = __int_as_float(0xff800000);
    const int target = p.row < valid ? a.target[p.row] : -1;
    const uint32_t col = t.n + p.half * (kTileN / 2);
    if (col + kTileN / 2 > a.vocab) {
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q)
#pragma unroll
            for (uint32_t j = 0; j < 32; ++j)
                x[q][j] = col + 32 * q + j < a.vocab ? x[q][j] : none;
    }
    const uint32_t off = (uint32_t)target - col;
    if (off < kTileN / 2) {
        float v = 0.0f;
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q)
#pragma unroll
            for (uint32_t j = 0; j < 32; ++j)
                v = off == 32 * q + j ? x[q][j] : v;
        a.target_logit[p.row] = v;
    }
    float top[4] = {none, none, none, none}, s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q)
#pragma unroll
        for (uint32_t j = 0; j < 32; ++j)
            top[j & 3] = fmaxf(top[j & 3], x[q][j]);
    const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    const uint64_t ref = f2(reference(m), reference(m));
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q)
#pragma unroll
        for (uint32_t j = 0; j < 32; j += 2) {
            float e0, e1;
            f2_split(f2_mul(f2_sub(f2(x[q][j], x[q][j + 1]), ref), f2(kLog2e, kLog2e)), e0, e1);
            s[j & 3] = __fadd_rn(s[j & 3], exp2_approx(e0));
            s[(j + 1) & 3] = __fadd_rn(s[(j + 1) & 3], exp2_approx(e1));
        }
    if (p.row < valid) {
        const uint32_t tiles = 2 * ((a.cols + kTileN - 1) / kTileN);
        a.stats[(uint64_t)p.row * tiles + 2 * t.nt + p.half] =
            make_float2(m, __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3])));
    }
}

/* x: the row's 128 logits of the tile, summed as the forward pass sums them, less lse before log2(e)
 * goes in: at the target of a confident token D is a small difference from 1, of which a logit that
 * differs from the one in lse by 1e-5, or an exponent rounded at lse's size, would leave little. */
template <bool F16>
__device__ __forceinline__ void d_epilogue(const ProductArgs& a, const Tile& t, const Part& p, uint32_t valid,
                                           const float (&x)[4][32])
{
    const bool in = p.row < valid;
    const int target = in ? a.target[p.row] - (int)a.v0 : -1;
    const float f = in ? a.factor[p.row] : 0.0f;
    const float lse = in ? a.lse[p.row] : 0.0f;
    const uint32_t col = t.n + p.half * (kTileN / 2), off = (uint32_t)target - col;
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q) {  // 32 columns at a time: registers
        uint32_t v[16];
#pragma unroll
        for (uint32_t j = 0; j < 32; j += 2) {
            float e[2];
            f2_split(f2_mul(f2_sub(f2(x[q][j], x[q][j + 1]), f2(lse, lse)), f2(kLog2e, kLog2e)), e[0], e[1]);
#pragma unroll
            for (uint32_t i = 0; i < 2; ++i) {
                e[i] = exp2_approx(e[i]);
                e[i] = off == 32 * q + j + i ? __fsub_rn(e[i], 1.0f) : e[i];
                e[i] = in && col + 32 * q + j + i < a.cols ? __fmul_rn(f, e[i]) : 0.0f;  // 0 behind the vocabulary
            }
            v[j / 2] = pack2<F16>(e[0], e[1]);
        }
        if (q % 2 == 0)
            stage_wait(p.lane);
        stage_row<128>(p.stage, p.lane,
                       {make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7]),
                        make_uint4(v[8], v[9], v[10], v[11]), make_uint4(v[12], v[13], v[14], v[15])},
                       q % 2 * 4);
        if (q % 2)
            stage_send(p.stage, p.lane, &a.out, col + 32 * (q - 1), p.row - p.lane, false);
    }
}

/* 32 columns of a warp's 32 rows of the weight's gradient where the TMA does not take its rows:
 * through shared memory, so that a store is 32 neighbours of a row (a lane writing its own row
 * took 8 times as long on rows of 2,223). */
template <zero_dtype_t GT>
__device__ __forceinline__ void put_rows(uint32_t stage, uint32_t lane, typename Elem<GT>::T* to, uint32_t rows, uint32_t col,
                                         uint32_t dim, float post, bool accumulate, const float (&x)[32])
{
    using G = typename Elem<GT>::T;
    to += col + lane;
    const bool in = col + lane < dim;
    uint4 v[8];
#pragma unroll
    for (uint32_t q = 0; q < 8; ++q)
        v[q] = make_uint4(__float_as_uint(x[4 * q]), __float_as_uint(x[4 * q + 1]), __float_as_uint(x[4 * q + 2]),
                          __float_as_uint(x[4 * q + 3]));
    stage_wait(lane);  // a bulk copy of an earlier tile may still read it
    stage_row<128>(stage, lane, v);
    __syncwarp();
    if (!in)
        return;
    auto batch = [&](uint32_t r0, const G* old) {  // 8 rows; what they held, or null
        float y[8];
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r)
            asm volatile("ld.shared.f32 %0, [%1];"
                         : "=f"(y[r])
                         : "r"(stage + (r0 + r) * 128 + ((lane / 4 ^ r) << 4) + lane % 4 * 4));
#pragma unroll
        for (uint32_t r = 0; r < 8; ++r)
            if (r0 + r < rows)
                to[(uint64_t)(r0 + r) * dim] = from_f32<GT>(old ? __fmaf_rn(y[r], post, to_f32<GT>(old[r])) : __fmul_rn(y[r], post));
    };
    if (accumulate) {  // all 32 asked for at once (8 at a time: 439 us for 100 x 2970 x 16881, not 306)
        G old[32];
#pragma unroll
        for (uint32_t r = 0; r < 32; ++r)
            old[r] = r < rows ? *const_cast<const volatile G*>(to + (uint64_t)r * dim) : G(0);
#pragma unroll
        for (uint32_t r0 = 0; r0 < 32; r0 += 8)
            batch(r0, old + r0);
    } else {
#pragma unroll
        for (uint32_t r0 = 0; r0 < 32; r0 += 8)
            batch(r0, nullptr);
    }
}

/* 16-bit rows of dweight that are added to: what a lane's row holds now in the tile's 128 columns,
 * asked for before the tile's sums are waited for (asked for afterwards, 32 columns at a time, it
 * took 358 us instead of 75 to add 10 tokens' gradient to 74 MB). */
struct OldRow {
    uint4 v[16];

    __device__ __forceinline__ void load(const ProductArgs& a, const Tile& t, const Part& p)
    {
        const uint32_t col = t.n + p.half * (kTileN / 2);
        const uint16_t* row = static_cast<const uint16_t*>(a.dweight) + (uint64_t)(a.v0 + p.row) * a.dim + col;
#pragma unroll
        for (uint32_t q = 0; q < 16; ++q) {
            const bool in = p.row < a.cols && p.half * (kTileN / 2) + 8 * q < t.width && col + 8 * q < a.dim;
            v[q] = in ? ld_v4(row + 8 * q) : make_uint4(0, 0, 0, 0);
        }
    }
};

template <bool F16>
__device__ __forceinline__ void put_nan(const ProductArgs& a, uint64_t at)
{
    const float nan = __int_as_float(0x7fc00000);
    if (a.grad_dtype == ZERO_F32)
        static_cast<float*>(a.dweight)[at] = nan;
    else
        static_cast<uint16_t*>(a.dweight)[at] = from_f32<F16 ? ZERO_F16 : ZERO_BF16>(nan);
}

/* The weight gradient's factor beside D: NaN once a wait has given up, in an earlier launch of the
 * call or in this one. */
__device__ __forceinline__ float weight_factor(const ProductArgs& a)
{
    return *const_cast<const volatile uint32_t*>(&a.head->error) ? __int_as_float(0x7fc00000) : a.head->post;
}

template <bool F16>
__device__ __forceinline__ void add_epilogue(const ProductArgs& a, const Tile& t, const Part& p, const OldRow& old)
{
    constexpr zero_dtype_t GT = F16 ? ZERO_F16 : ZERO_BF16;
    const float post = weight_factor(a);
    const uint32_t row0 = p.row - p.lane;
#pragma unroll
    for (uint32_t c = 0; c < kTileN / 2; c += 32) {
        const uint32_t at = p.half * (kTileN / 2) + c, col = t.n + at;
        if (at >= t.width || col >= a.dim || row0 >= a.cols)
            break;  // the same for the whole warp
        float x[32];
        load_part(p, c, x);
        uint4 v[4];
#pragma unroll
        for (uint32_t q = 0; q < 4; ++q) {
            typename Elem<GT>::Raw raw;
            float o[8];
            raw.v = old.v[c / 8 + q];
            widen<GT>(raw, o);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                o[j] = __fmaf_rn(x[8 * q + j], post, o[j]);
            v[q] = narrow<GT>(o).v;
        }
        stage_wait(p.lane);
        stage_row<64>(p.stage, p.lane, v);
        stage_send(p.stage, p.lane, &a.out_w, col, a.v0 + row0, false);
    }
}

/* Sums in fp32 (of a piece after the first: added in L2, one launch after another), or dweight's
 * rows of the piece (fp32 ones that are added to: in L2 too). */
template <Product P, bool F16>
__device__ __forceinline__ void sum_epilogue(const ProductArgs& a, const Tile& t, const Part& p, uint32_t rows)
{
    const float post = P == kDweight && a.splits == 1 ? weight_factor(a) : 1.0f;
    const uint32_t row0 = p.row - p.lane;
#pragma unroll 1
    for (uint32_t c = 0; c < kTileN / 2; c += 32) {
        const uint32_t at = p.half * (kTileN / 2) + c, col = t.n + at;
        if (at >= t.width || col >= a.dim)
            break;  // the same for the whole warp
        float x[32];
        load_part(p, c, x);
        if (row0 >= rows)
            break;
        if (P == kDweight && a.splits == 1 && !a.bulk) {
            const uint64_t at_row = (uint64_t)(a.v0 + row0) * a.dim;
            if (a.grad_dtype == ZERO_F32)
                put_rows<ZERO_F32>(p.stage, p.lane, static_cast<float*>(a.dweight) + at_row, rows - row0, col, a.dim, post,
                                   a.accumulate, x);
            else
                put_rows<F16 ? ZERO_F16 : ZERO_BF16>(p.stage, p.lane, static_cast<uint16_t*>(a.dweight) + at_row, rows - row0,
                                                     col, a.dim, post, a.accumulate, x);
            continue;
        }
#pragma unroll
        for (uint32_t j = 0; j < 32; ++j)
            x[j] = __fmul_rn(x[j], post);
        stage_wait(p.lane);
        if (P == kDweight && a.splits == 1 && a.grad_dtype != ZERO_F32) {
            uint4 v[4];
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q)
                v[q] = make_uint4(pack2<F16>(x[8 * q], x[8 * q + 1]), pack2<F16>(x[8 * q + 2], x[8 * q + 3]),
                                  pack2<F16>(x[8 * q + 4], x[8 * q + 5]), pack2<F16>(x[8 * q + 6], x[8 * q + 7]));
            stage_row<64>(p.stage, p.lane, v);
        } else {
            uint4 v[8];
#pragma unroll
            for (uint32_t q = 0; q < 8; ++q)
                v[q] = make_uint4(__float_as_uint(x[4 * q]), __float_as_uint(x[4 * q + 1]), __float_as_uint(x[4 * q + 2]),
                                  __float_as_uint(x[4 * q + 3]));
            stage_row<128>(p.stage, p.lane, v);
        }
        const uint32_t first = P == kDhidden ? t.split * rows : a.splits == 1 ? a.v0 : t.split * a.piece;
        stage_send(p.stage, p.lane, P == kDhidden ? &a.out : &a.out_w, col, first + row0,
                   P == kDhidden ? !a.first_piece : a.splits == 1 && a.accumulate);
    }
}

#ifdef ZERO_TEST_HOOKS
/* Test builds only (never the product library): the first block's stage whose copies of A are
 * withheld, so that the waits on it run out without any fault. */
__device__ unsigned long long zero_test_withheld_head_stage = ~0ull;
#endif

/* A launch's products over all their tiles: a pair of blocks on every two SMs takes tiles of
 * 256 x 256 in turn.  Warp 0 copies operands in, warp 1 of the pair's first block issues the
 * matrix instructions (one elected lane each), warps 4 to 11 take finished accumulators out while
 * the next tile's are formed in the other half of tensor memory.
 *
 * What bounds it: a tile's matrix instructions take 512 cycles per 64 of the sum (128 for each 16,
 * measured alone), and in them shared memory gives 32 KB of operands and takes 32 KB of the next,
 * 128 bytes a cycle, its limit; the TMA unit needs 486 for the copies.  A long launch of logits
 * runs at 7% above the 512 (GPT-2 1.5B's 8,192 tokens: 612-640 us for 1.32 TFLOP, 2.1 PFLOP/s).
 * A launch has about 8 us of its own: start, first copies, last epilogue.
 *
 * The matrix unit cuts its fp32 sums off instead of rounding them, always toward 0: 256 steps
 * for a logit of 4,096 terms left the losses 1.5e-5 too small on the average.  The logits are
 * therefore taken in parts of 1,024 terms, added up in registers (4e-6 there, at no cost in time), by
 * the losses and by D alike: D's logit and the one in lse have the same bits.  (D from logits in one
 * part: of a target with all but 1e-4 of the softmax, over 4,096 terms of one sign, it was off by 80%.)
 * The gradients' sums take operands of 16 bits, whose roundings pass what is cut off (2^-23 of the
 * sum so far in each of its steps of 16 terms), and go without. */
template <Mode MODE, bool F16>
__global__ void __launch_bounds__(kThreads, 1) k_head_product(const __grid_constant__ ProductArgs a)
{
    constexpr uint32_t kPart = MODE == kGrads ? ~0u : kSumBlocks;
    constexpr uint32_t kK = MODE == kGrads ? kGradsK : kLogitsK, kHalf = kK / 64 * kBoxBytes, kStageBytes = 2 * kHalf;
    constexpr uint32_t kRing = kRingBytes / kStageBytes;
    static_assert(kRing <= kMaxRing, "barriers");
    extern __shared__ uint8_t raw[];
    __shared__ Shared sh;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rank = block_of_pair();
    const uint32_t stages = (smem_addr(raw) + 1023) / 1024 * 1024;
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < kRing; ++s) {
            bar_init(smem_addr(&sh.full[s]), 1);
            bar_init(smem_addr(&sh.empty[s]), 1);
        }
        for (uint32_t b = 0; b < 2; ++b) {
            bar_init(smem_addr(&sh.acc_full[b]), 1);
            bar_init(smem_addr(&sh.acc_empty[b]), 2 * kEpilogueWarps);
        }
        bar_init(smem_addr(&sh.drain), 1);
        sh.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2)
        tmem_alloc(smem_addr(&sh.tmem), 512);
    if (threadIdx.x == 32) {
        map_prefetch(&a.hidden);
        map_prefetch(&a.weight);
        if (MODE != kStats)
            map_prefetch(&a.out);
        if (MODE == kGrads)
            map_prefetch(&a.d);
    }
    tmem_fence_before();
    __syncthreads();
    pair_sync();
    tmem_fence_after();
    const uint32_t tmem = sh.tmem;
    volatile uint32_t* gave_up = &sh.gave_up;
    grid_dependency_wait();
    grid_launch_dependents();  // the next kernel's blocks get ready as this one's leave
    const uint32_t valid = *const_cast<const volatile uint32_t*>(&a.head->valid);
    const Work<MODE> tiles(a, valid);
    const uint32_t first = blockIdx.x / 2, step = gridDim.x / 2;

    if (warp == 0) {
        // what earlier kernels wrote through the generic proxy, for the TMA's reads
        asm volatile("fence.proxy.async.global;" ::: "memory");
        const CUtensorMap* hidden = valid == a.rows ? &a.hidden : &a.gathered;
        uint32_t issued = 0;
        bool ok = true;
        for (uint32_t i = first; ok && i < tiles.total; i += step) {
            const Tile t = tiles.at(i);
            const bool a_mn = t.product == kDweight, b_mn = t.product != kLogits;
            const CUtensorMap *ma = b_mn ? &a.d : hidden, *mb = a_mn ? hidden : &a.weight;
            const uint32_t b0 = a_mn ? 0 : a.v0;  // weight's rows of the piece
            const uint32_t m = t.m + rank * kRows, n = t.n + rank * (t.width / 2);
            const uint32_t boxes = b_mn ? (t.width / 2 + 63) / 64 : 1;
            for (uint32_t k = t.k0; k < t.k1; ++k, ++issued) {
                const uint32_t s = issued % kRing, turn = issued / kRing;
                if (turn && !warp_wait(smem_addr(&sh.empty[s]), (turn - 1) & 1, gave_up)) {
                    ok = false;
                    break;
                }
                // both blocks' copies count on the first one's barrier
                const uint32_t bar = of_first(smem_addr(&sh.full[s])), to = stages + s * kStageBytes, kk = k * kK;
                if (elect_one()) {
                    if (rank == 0)
                        bar_expect(smem_addr(&sh.full[s]), 2 * (kK / 64 + boxes) * kBoxBytes);
#ifdef ZERO_TEST_HOOKS
                    if (blockIdx.x != 0 || issued != zero_test_withheld_head_stage)
#endif
#pragma unroll
                    for (uint32_t j = 0; j < kK / 64; ++j)
                        tma_box(to + j * kBoxBytes, ma, (int)(a_mn ? m + 64 * j : kk + 64 * j), (int)(a_mn ? kk : m), bar);
                    for (uint32_t j = 0; j < boxes; ++j)
                        tma_box(to + kHalf + j * kBoxBytes, mb, (int)(b_mn ? n + 64 * j : kk), (int)(b_mn ? b0 + kk : b0 + n),
                                bar);
                }
                __syncwarp();
            }
        }
        if (!ok) {  // copies still in flight land before the block's shared memory goes
            uint32_t none = 0;
            if (rank == 0) {
                for (uint32_t q = issued > kRing ? issued - kRing : 0; q < issued; ++q)
                    bar_wait(smem_addr(&sh.full[q % kRing]), (q / kRing) & 1, &none);
            } else {
                for (const long long t0 = clock64(); clock64() - t0 < 100000000LL;) {
                }
            }
        }
    } else if (warp == 1 && rank == 0) {
        uint32_t s = 0, phase = 0, buf = 0;
        bool ok = true, ready = false;
        for (uint32_t i = first; ok && i < tiles.total; i += step) {
            const Tile t = tiles.at(i);
            const bool a_mn = t.product == kDweight, b_mn = t.product != kLogits;
            const uint32_t idesc = instr_desc(F16, a_mn, b_mn, kTileM, t.width);
            const uint64_t desc_a = operand_desc(stages, a_mn), desc_b = operand_desc(stages + kHalf, b_mn);
            for (uint32_t k = t.k0; ok && k < t.k1; ++buf) {
                const uint32_t b = buf & 1, turn = buf >> 1, begin = k, end = t.k1 - k > kPart ? k + kPart : t.k1;
                if (turn && !warp_wait(smem_addr(&sh.acc_empty[b]), (turn - 1) & 1, gave_up)) {
                    ok = false;
                    break;
                }
                tmem_fence_after();
                for (; k < end; ++k) {
                    if (!ready && !warp_wait(smem_addr(&sh.full[s]), phase, gave_up)) {
                        ok = false;
                        break;
                    }
                    tmem_fence_after();
                    const uint32_t at = s;
                    s = s + 1 == kRing ? 0 : s + 1;
                    phase ^= s == 0;
                    const bool next = bar_test(smem_addr(&sh.full[s]), phase);
                    if (elect_one()) {
                        const uint64_t da = desc_a + at * (kStageBytes / 16), db = desc_b + at * (kStageBytes / 16);
#pragma unroll
                        for (uint32_t q = 0; q < kK / 16; ++q)
                            mma_pair(tmem + b * kTileN, da + k_step(a_mn, q), db + k_step(b_mn, q), idesc,
                                     k > begin || q > 0);
                        mma_commit(smem_addr(&sh.empty[at]));
                    }
                    ready = __all_sync(0xffffffffu, next);
                }
                if (ok && elect_one())
                    mma_commit(smem_addr(&sh.acc_full[b]));
                __syncwarp();
            }
        }
        if (!ok) {  // matrix instructions in flight finish before tensor memory goes
            uint32_t none = 0;
            if (elect_one())
                mma_commit(smem_addr(&sh.drain));
            __syncwarp();
            bar_wait(smem_addr(&sh.drain), 0, &none);
        }
    } else if (warp >= 4) {
        const uint32_t quarter = warp & 3;
        uint32_t buf = 0;
        bool ok = true;
        Part p;
        p.half = (warp - 4) / 4;
        p.lane = lane;
        p.stage = stages + kRingBytes + (warp - 4) * kOutBytes;
        auto acquire = [&] {
            const uint32_t b = buf & 1;
            p.acc = tmem + (quarter * 32 << 16) + b * kTileN + p.half * (kTileN / 2);
            ok = warp_wait(smem_addr(&sh.acc_full[b]), (buf >> 1) & 1, gave_up);
            tmem_fence_after();
        };
        auto release = [&] {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0)
                bar_arrive(of_first(smem_addr(&sh.acc_empty[buf & 1])));
            ++buf;
        };
        uint32_t i = first;
        for (; i < tiles.total; i += step) {
            const Tile t = tiles.at(i);
            p.row = t.m + rank * kRows + quarter * 32 + lane;
            p.empty = t.k0 >= t.k1;
            if constexpr (MODE != kGrads) {
                // the first part's sums, then the others' added 16 columns at a time (both in one loop, 32 at
                // a time, D's epilogue spilled 110 registers)
                float x[4][32];
                acquire();
                if (!ok)
                    break;
#pragma unroll
                for (uint32_t q = 0; q < 4; ++q)
                    tmem_load32(p.acc + 32 * q, x[q]);
                release();
#pragma unroll 1
                for (uint32_t k = t.k0 + kPart; k < t.k1; k += kPart) {
                    acquire();
                    if (!ok)
                        break;
#pragma unroll
                    for (uint32_t q = 0; q < 8; ++q) {
                        float y[16];
                        tmem_load16(p.acc + 16 * q, y);
#pragma unroll
                        for (uint32_t j = 0; j < 16; ++j)
                            x[q / 2][q % 2 * 16 + j] = __fadd_rn(x[q / 2][q % 2 * 16 + j], y[j]);
                    }
                    release();
                }
                if (!ok)
                    break;
                if constexpr (MODE == kStats)
                    stats_epilogue(a, t, p, valid, x);
                else
                    d_epilogue<F16>(a, t, p, valid, x);
            } else {
                OldRow old;
                const bool add16 = t.product == kDweight && a.bulk && a.accumulate && a.grad_dtype != ZERO_F32;
                if (add16)
                    old.load(a, t, p);
                if (!p.empty) {
                    acquire();
                    if (!ok)
                        break;
                }
                if (t.product == kDhidden)
                    sum_epilogue<kDhidden, F16>(a, t, p, tiles.h.mt * kTileM);
                else if (add16)
                    add_epilogue<F16>(a, t, p, old);
                else
                    sum_epilogue<kDweight, F16>(a, t, p, a.cols);
                if (!p.empty)
                    release();
            }
        }
        if (lane == 0)  // what is on its way out has left shared memory, and is written
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if constexpr (MODE == kGrads) {  // a wait gave up: the tiles of dweight left undone tell, as NaN
            __syncwarp();
            for (; i < tiles.total && a.splits == 1; i += step) {
                const Tile t = tiles.at(i);
                if (t.product != kDweight)
                    continue;
                const uint32_t row = t.m + rank * kRows + quarter * 32 + lane, at = p.half * (kTileN / 2);
                const uint32_t end = t.width < at + kTileN / 2 ? t.width : at + kTileN / 2;
                if (row < a.cols)
                    for (uint32_t c = at; c < end && t.n + c < a.dim; ++c)
                        put_nan<F16>(a, (uint64_t)(a.v0 + row) * a.dim + t.n + c);
            }
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    pair_sync();  // neither block's memory goes while the other may still reach it
    tmem_fence_after();
    if (warp == 2)
        tmem_free(tmem, 512);
    if (threadIdx.x == 0 && sh.gave_up) {
        a.head->error = 1;
        if (a.state_error)
            *a.state_error = 1;
    }
}

/* ------------------------------------------------------------------------------------ */
/* before and after the products                                                          */
/* ------------------------------------------------------------------------------------ */
struct TokenArgs {
    const void* targets;
    uint32_t wide, rows, vocab, dim, pitch;
    uint32_t direct;       // hidden can be used as it lies
    uint32_t blocks, per;  // blocks with tokens, tokens of each (a multiple of 32)
    Header* head;
    uint32_t* token;       // [valid]: the token in its place
    int* target;           // [valid]
    float* loss;           // forward: of tokens without a target, 0
    float* lse;
    const float* lse_in;   // backward
    float* lse_out;        // [valid]
    float* factor;         // [valid]
    const float* row_scale;
    const zero_step_state_t* st;
    float scale;
    uint32_t backward, f16;
    const uint16_t* hidden;
    uint64_t hidden_stride;
    uint16_t* gathered;    // [rows_pad][pitch]
    uint16_t* dhidden;     // backward: rows of tokens without a target are written 0
    uint64_t dhidden_stride;
    const uint16_t* weight;
    uint16_t* padded;      // [vocab][pitch], or null: weight is used as it lies
};

__device__ __forceinline__ int head_target(const void* p, uint32_t wide, uint32_t vocab, uint32_t t)
{
    if (wide) {
        const long long v = *(static_cast<const volatile long long*>(p) + t);
        return v >= 0 && v < (long long)vocab ? (int)v : -1;
    }
    const int v = *(static_cast<const volatile int*>(p) + t);
    return v >= 0 && v < (int)vocab ? v : -1;
}

/* 8 outputs of a padded row at once, from 8 neighbours of the dense one: one 128-bit load, or the
 * 32-bit words that hold at least one of them (pad.h). */
struct PadChunk {
    uint32_t w[5], c, dim, odd;
    uint4* to;

    template <bool VEC>
    __device__ __forceinline__ void load(const uint16_t* from, uint16_t* to_, uint32_t c_, uint32_t dim_)
    {
        c = c_;
        dim = dim_;
        to = reinterpret_cast<uint4*>(to_) + c;
        if constexpr (VEC) {
            const uint4 v = 8 * c < dim ? ld_v4(from + 8 * c) : make_uint4(0, 0, 0, 0);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            return;
        }
        odd = (uintptr_t)from >> 1 & 1;
        pad_load(w, c, dim, odd, [&](int64_t e) { return *reinterpret_cast<const volatile uint32_t*>(from + e); },
                 [&](int64_t e) { return ld_one(from + e); });
    }

    template <bool VEC>
    __device__ __forceinline__ void store()
    {
        if constexpr (!VEC)
            pad_shift(w, c, dim, odd);
        *to = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

/* The tokens that have a target, in order: their places, targets, factors and lse; and unless
 * that is all of them (or hidden cannot be used as it lies) their rows next to each other, with
 * zeros behind them up to a multiple of 256 rows.  Every block counts the targets before its own
 * tokens itself: with 8,192 of them that is 8 loads to a thread, less than a second launch.
 * 7 to 8 us, a launch and four round trips one after another (counts, masks, targets, rows). */
__device__ __forceinline__ void list_tokens(const TokenArgs& a, uint32_t* groups)
{
    // groups: of 32 own tokens: which have a target; then the count before them
    __shared__ uint32_t before[32], total[32];
    __shared__ float most[32];
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n_groups = a.per / 32;
    const uint32_t lo = blockIdx.x * a.per, hi = lo + a.per < a.rows ? lo + a.per : a.rows;
    const float common = a.backward ? __fmul_rn(a.scale, a.st ? *const_cast<const volatile float*>(&a.st->loss_scale) : 1.0f) : 0.0f;
    auto target_of = [&](uint32_t t) { return t < a.rows ? head_target(a.targets, a.wide, a.vocab, t) : -1; };
    auto factor_of = [&](uint32_t t) {
        return a.row_scale ? __fmul_rn(common, *const_cast<const volatile float*>(a.row_scale + t)) : common;
    };
    // all targets: how many there are, how many before this block's, and the largest |f|
    uint32_t earlier = 0, n = 0;
    float top = 0.0f;
    for (uint32_t from = threadIdx.x; from < a.rows; from += 8 * 1024) {
        int target[8];
        float f[8];
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            const uint32_t t = from + i * 1024;
            target[i] = target_of(t);
            f[i] = a.backward && t < a.rows ? factor_of(t) : 0.0f;
        }
#pragma unroll
        for (uint32_t i = 0; i < 8; ++i) {
            const uint32_t there = target[i] >= 0;
            n += there;
            earlier += from + i * 1024 < lo ? there : 0;
            if (there && fabsf(f[i]) <= kMaxFloat)  // one that is not finite says nothing of the others' size
                top = fmaxf(top, fabsf(f[i]));
        }
    }
    auto warp_max = [](float x) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
        return x;
    };
    earlier = __reduce_add_sync(0xffffffffu, earlier);
    n = __reduce_add_sync(0xffffffffu, n);
    top = warp_max(top);
    if (lane == 0) {
        before[warp] = earlier;
        total[warp] = n;
        most[warp] = top;
    }
    for (uint32_t g = warp; g < n_groups; g += 32) {
        const uint32_t mask = __ballot_sync(0xffffffffu, target_of(lo + 32 * g + lane) >= 0 && lo + 32 * g + lane < hi);
        if (lane == 0)
            groups[g] = mask;
    }
    __syncthreads();
    const uint32_t valid = __reduce_add_sync(0xffffffffu, total[lane]);
    top = warp_max(most[lane]);
    uint32_t* const counts = groups + n_groups;
    if (warp == 0) {  // the groups' counts before each
        uint32_t at = __reduce_add_sync(0xffffffffu, before[lane]);
        for (uint32_t g = 0; g < n_groups; g += 32) {
            const uint32_t c = g + lane < n_groups ? __popc(groups[g + lane]) : 0;
            uint32_t sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
                sum += lane >= (uint32_t)o ? up : 0;
            }
            if (g + lane < n_groups)
                counts[g + lane] = at + sum - c;
            at += __shfl_sync(0xffffffffu, sum, 31);
        }
    }
    __syncthreads();
    // f in units of the largest finite |f| (fp16: of 2^-14 of it); without one it stays as it is
    const bool scaled = top > 0.0f;
    const float most_units = a.f16 ? 16384.0f : 1.0f, post = scaled ? __fdiv_rn(top, most_units) : 1.0f;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.head->valid = valid;
        a.head->error = 0;
        a.head->post = post;
    }
    for (uint32_t g = warp; g < n_groups; g += 32) {
        const uint32_t t = lo + 32 * g + lane, mask = groups[g], r = counts[g] + __popc(mask & ((1u << lane) - 1));
        if (t >= hi)
            continue;
        if (mask >> lane & 1) {
            a.token[r] = t;
            a.target[r] = target_of(t);
            if (a.backward) {
                a.lse_out[r] = *const_cast<const volatile float*>(a.lse_in + t);
                a.factor[r] = scaled ? __fmul_rn(__fdiv_rn(factor_of(t), top), most_units) : factor_of(t);
            }
        } else if (!a.backward) {
            a.loss[t] = 0.0f;
            a.lse[t] = 0.0f;
        }
    }
    const bool gather = valid != a.rows || !a.direct;
    if (!gather && !(a.dhidden && valid != a.rows))
        return;
    const bool vec = a.dim % 8 == 0 && a.hidden_stride % 8 == 0 && ((uintptr_t)a.hidden & 15) == 0;
    const uint32_t chunks = a.pitch / 8;
    for (uint32_t t = lo + warp; t < hi; t += 32) {  // a row to a warp
        const uint32_t g = (t - lo) / 32, bit = (t - lo) % 32, mask = groups[g];
        if (!(mask >> bit & 1)) {
            if (a.dhidden)
                for (uint32_t c = lane; c < a.dim; c += 32)
                    a.dhidden[t * a.dhidden_stride + c] = 0;
            continue;
        }
        if (!gather)
            continue;
        const uint32_t r = counts[g] + __popc(mask & ((1u << bit) - 1));
        const uint16_t* from = a.hidden + t * a.hidden_stride;
        uint16_t* to = a.gathered + (uint64_t)r * a.pitch;
        if (vec) {
#pragma unroll 4
            for (uint32_t c = lane; c < chunks; c += 32)
                reinterpret_cast<uint4*>(to)[c] = c * 8 < a.dim ? ld_v4(from + c * 8) : make_uint4(0, 0, 0, 0);
        } else {
            for (uint32_t c = lane; c < chunks; c += 32) {
                PadChunk pad;
                pad.load<false>(from, to, c, a.dim);
                pad.store<false>();
            }
        }
    }
    const uint32_t end = (valid + kTileM - 1) / kTileM * kTileM;
    for (uint32_t r = valid + blockIdx.x * 32 + warp; gather && r < end; r += a.blocks * 32)
        for (uint32_t c = lane; c < chunks; c += 32)
            reinterpret_cast<uint4*>(a.gathered + (uint64_t)r * a.pitch)[c] = make_uint4(0, 0, 0, 0);
}

/* Weight's rows at another pitch, by all blocks: a thread's chunks lie a whole grid apart; row and
 * place in it step along, without a division. */
template <bool VEC>
__device__ __forceinline__ void pad_rows(const TokenArgs& a)
{
    const uint32_t chunks = a.pitch / 8, threads = gridDim.x * blockDim.x, first = blockIdx.x * blockDim.x + threadIdx.x;
    const uint32_t rows_on = threads / chunks, on = threads % chunks;
    uint32_t r = first / chunks, c = first % chunks;
    while (r < a.vocab) {  // four in flight
        PadChunk pad[4];
        uint32_t n = 0;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            if (r >= a.vocab)
                break;
            pad[i].load<VEC>(a.weight + (uint64_t)r * a.dim, a.padded + (uint64_t)r * a.pitch, c, a.dim);
            c += on;
            const bool next = c >= chunks;
            c -= next ? chunks : 0;
            r += rows_on + next;
            ++n;
        }
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            if (i < n)
                pad[i].store<VEC>();
    }
}

__global__ void __launch_bounds__(1024, 1) k_head_tokens(const TokenArgs a)
{
    extern __shared__ uint32_t groups[];
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x < a.blocks)
        list_tokens(a, groups);
    if (a.padded && a.dim % 8)
        pad_rows<false>(a);
    else if (a.padded)
        pad_rows<true>(a);
}

struct LossArgs {
    const Header* head;
    const uint32_t* token;
    const float2* stats;
    const float* target_logit;
    float* loss;
    float* lse;
    uint32_t tiles;
};

/* A sum of exponentials relative to top, relative to m instead. */
__device__ __forceinline__ float below(float sum, float top, float m)
{
    return __fmul_rn(sum, exp2f(__fmul_rn(__fsub_rn(top, reference(m)), kLog2e)));
}

/* The tiles' statistics of a token, a warp per token: 7 us for 8,192 tokens of 50,257 logits, whose 26
 * MB come out of L2. */
__global__ void __launch_bounds__(256) k_head_loss(const LossArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t valid = a.head->valid, lane = threadIdx.x & 31, warps = gridDim.x * (blockDim.x / 32);
    for (uint32_t r = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); r < valid; r += warps) {
        const float2* s = a.stats + (uint64_t)r * a.tiles;
        float top = __int_as_float(0xff800000), sum = 0.0f;
        for (uint32_t i = lane; i < a.tiles; i += 32) {
            const float2 x = s[i];
            const float m = fmaxf(top, x.x);
            sum = __fadd_rn(below(sum, top, m), below(x.y, x.x, m));
            top = m;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float ot = __shfl_xor_sync(0xffffffffu, top, o), os = __shfl_xor_sync(0xffffffffu, sum, o);
            const float m = fmaxf(top, ot);
            sum = __fadd_rn(below(sum, top, m), below(os, ot, m));
            top = m;
        }
        if (lane == 0) {
            // the maximum is taken off the target's logit before the logarithm comes in: a confident
            // token's loss keeps its own digits, and is not negative
            const float more = a.head->error ? __int_as_float(0x7fc00000) : logf(sum);
            a.lse[a.token[r]] = __fadd_rn(top, more);
            a.loss[a.token[r]] = __fadd_rn(__fsub_rn(top, a.target_logit[r]), more);
        }
    }
}

struct JoinArgs {
    const Header* head;
    const float* sums;
    const uint32_t* token;  // dhidden: row r goes to token[r]; dweight: null, row r to v0 + r
    void* out;
    uint64_t out_stride, split_stride;
    uint32_t rows, v0, dim, dim8, splits, accumulate;
    uint32_t k_blocks;      // dhidden: of the first piece's sum
};

/* The splits' sums in order, times the common factor, rounded once.  Bound by memory: dhidden of
 * 8,192 x 1,600 reads 52 MB and writes 26 in 16 us; where the sums were cut into many splits (few
 * tokens) 4 of them are in flight. */
template <zero_dtype_t GT, bool VEC>
__global__ void __launch_bounds__(256) k_head_join(const JoinArgs a)
{
    using G = typename Elem<GT>::T;
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t rows = a.token ? a.head->valid : a.rows, lane = threadIdx.x & 31;
    const float post = a.head->error ? __int_as_float(0x7fc00000) : a.head->post;  // a wait gave up: NaN
    const uint32_t pieces = (a.dim + 255) / 256, mt = (rows + kTileM - 1) / kTileM;
    // of dhidden: the splits and their distance that the products' blocks came to; a last, narrower
    // piece of the vocabulary may have been cut into fewer, added to the first of these
    const uint32_t splits = a.token ? splits_of(mt * ((a.dim + kTileN - 1) / kTileN), a.k_blocks) : a.splits;
    const uint64_t split_stride = a.token ? (uint64_t)mt * kTileM * a.dim8 : a.split_stride;
    const uint64_t warps = (uint64_t)gridDim.x * (blockDim.x / 32), total = (uint64_t)rows * pieces;
    for (uint64_t u = (uint64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); u < total; u += warps) {
        const uint32_t r = (uint32_t)(u / pieces), piece = (uint32_t)(u - (uint64_t)r * pieces);
        G* row = static_cast<G*>(a.out) + (a.token ? a.token[r] : a.v0 + r) * a.out_stride;
        const float* from = a.sums + (uint64_t)r * a.dim8;
        float s[8], v[8];
        widen<ZERO_F32>(load_chunk<ZERO_F32, VEC>(from, a.dim, piece, lane, 32), s);
        for (uint32_t k = 1; k < splits; k += 4) {  // four splits' loads in flight
            typename Elem<ZERO_F32>::Raw raw[4];
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q)
                raw[q] = load_chunk<ZERO_F32, VEC>(from + (k + q) * split_stride, k + q < splits ? a.dim : 0, piece, lane, 32);
#pragma unroll
            for (uint32_t q = 0; q < 4; ++q) {
                if (k + q >= splits)
                    break;
                widen<ZERO_F32>(raw[q], v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    s[j] = __fadd_rn(s[j], v[j]);
            }
        }
        if (a.accumulate)
            widen<GT>(load_chunk<GT, VEC>(row, a.dim, piece, lane, 32), v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            s[j] = a.accumulate ? __fmaf_rn(s[j], post, v[j]) : __fmul_rn(s[j], post);
        store_chunk<GT, VEC>(row, a.dim, piece, lane, 32, s);
    }
}

/* ------------------------------------------------------------------------------------ */
/* host side                                                                              */
/* ------------------------------------------------------------------------------------ */
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

/* The driver's encoder, through the runtime (the library does not link libcuda). */
EncodeTiled encoder()
{
    static EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

bool tensor_map(CUtensorMap* map, const void* p, zero_dtype_t t, uint64_t cols, uint64_t rows, uint64_t stride,
                uint32_t box_cols, uint32_t box_rows)
{
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {stride * dtype_size(t)};
    const cuuint32_t box[2] = {box_cols, box_rows}, step[2] = {1, 1};
    const CUtensorMapDataType type = t == ZERO_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : t == ZERO_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encoder() &&
           encoder()(map, type, 2, const_cast<void*>(p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     box_cols * dtype_size(t) == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int map_refused()
{
    record_cuda_error((int)cudaErrorInvalidValue);
    return ZERO_ECUDA;
}

uint64_t up(uint64_t x, uint64_t to) { return (x + to - 1) / to * to; }

/* A 128-byte row of a TMA box that does not start on 128 bytes touches two lines: rows of 840
 * instead of 832 or 896 slow the products by a fifth.  Calls of so many rows copy hidden and weight
 * to 128-byte boundaries first (840 by 33,140, forward and backward: 8,192 rows 325 + 1,077 us, so 281 + 979;
 * 2,048 rows 102 + 308, 100 + 299; 1,024 rows the same either way). */
constexpr uint32_t kAlignRows = 2048;

/* How a call is cut, and where its parts lie in the workspace. */
struct Plan {
    uint32_t rows_pad, dim8, pitch, piece, rows_h, splits_w;
    bool pad;  // weight's rows are copied to another pitch
    uint64_t token, target, factor, lse, logit, gathered, weight, stats, d, sums_h, sums_w, bytes;
};

Plan make_plan(uint64_t rows, uint32_t dim, uint32_t vocab)
{
    Plan p;
    p.rows_pad = (uint32_t)up(rows ? rows : 1, kTileM);
    p.dim8 = (uint32_t)up(dim, 8);
    p.pitch = (uint32_t)up(dim, 64);
    p.pad = dim % 8 || (dim % 64 && rows >= kAlignRows);
    const uint64_t vp = up(vocab, kTileN), tiles = vp / kTileN, nt = (dim + kTileN - 1) / kTileN;
    // D of a piece: 64 million elements (128 MB, about the L2) or 8,192 columns, whichever is more.
    // Within a factor of two above that, the width whose dweight tiles leave the fewest SMs idle
    // over all pieces (GPT-2 1.5B's head at 8,192 tokens: 32 tiles of 256 take 19 turns of the
    // 76 pairs of SMs, 7 equal pieces of 29 took 21)
    uint64_t least = up((64ull << 20) / p.rows_pad, kTileN) / kTileN;
    least = least < 32 ? 32 : least;
    uint64_t best = ~0ull, width = tiles;
    for (uint64_t w = least; w <= 2 * least && w < tiles; ++w) {
        auto turns = [&](uint64_t n) { return (n * nt + kSms / 2 - 1) / (kSms / 2); };
        const uint64_t all = tiles / w * turns(w) + turns(tiles % w);
        if (all < best) {
            best = all;
            width = w;
        }
    }
    p.piece = (uint32_t)(width * kTileN);
    p.splits_w = splits_of((uint32_t)(width * nt), p.rows_pad / kGradsK);
    // dhidden's sums: one of all rows, or as many parts of fewer rows as the SMs take
    p.rows_h = kSms / 2 / (uint32_t)nt * kTileM;
    p.rows_h = p.rows_h < p.rows_pad ? p.rows_pad : p.rows_h;
    uint64_t at = sizeof(Header);
    auto take = [&](uint64_t bytes) {
        const uint64_t q = at;
        at += up(bytes, 256);
        return q;
    };
    p.token = take(4ull * p.rows_pad);
    p.target = take(4ull * p.rows_pad);
    p.factor = take(4ull * p.rows_pad);
    p.lse = take(4ull * p.rows_pad);
    p.logit = take(4ull * p.rows_pad);
    p.gathered = take(2ull * p.rows_pad * p.pitch);
    p.weight = take(p.pad ? 2ull * vocab * p.pitch : 0);
    const uint64_t shared = at;
    p.stats = take(8ull * p.rows_pad * (vp / 128));
    const uint64_t forward = at;
    at = shared;
    p.d = take(2ull * p.rows_pad * p.piece);
    p.sums_h = take(4ull * p.rows_h * p.dim8);
    p.sums_w = take(p.splits_w > 1 ? 4ull * p.splits_w * p.piece * p.dim8 : 0);
    p.bytes = at > forward ? at : forward;
    return p;
}

bool sizes_ok(uint64_t rows, uint32_t dim, uint32_t vocab)
{
    return rows <= (1ull << 24) && dim >= 1 && dim <= 65536 && vocab >= 1 && vocab <= (1u << 24) &&
           (rows / kTileM + 1) * (vocab / kTileN + 1) <= 1ull << 30;  // tiles are counted in 32 bits
}

struct Call {
    zero_dtype_t dtype;
    uint64_t rows;
    uint32_t dim, vocab;
    const void* hidden;
    uint64_t hidden_stride;
    const void* weight;
    const void* targets;
    uint32_t target_bytes;
    char* work;
    cudaStream_t stream;
};

int check_call(const Call& c)
{
    if ((c.dtype != ZERO_BF16 && c.dtype != ZERO_F16) || !sizes_ok(c.rows, c.dim, c.vocab) ||
        (c.target_bytes != 4 && c.target_bytes != 8) || !c.weight || !c.work)
        return ZERO_EINVAL;
    if (c.rows && (!c.hidden || !c.targets || (c.rows > 1 && c.hidden_stride < c.dim) || c.hidden_stride > (1ull << 32)))
        return ZERO_EINVAL;
    if (!aligned_to(c.hidden, 2) || !aligned_to(c.weight, c.dim % 8 ? 2 : 16) ||
        !aligned_to(c.targets, c.target_bytes) || !aligned_to(c.work, 256))
        return ZERO_EALIGN;
    return ZERO_OK;
}

unsigned warps_grid(uint64_t warps)
{
    const uint64_t want = (warps + 7) / 8, cap = (uint64_t)sm_count() * 8;
    return (unsigned)(want < cap ? (want ? want : 1) : cap);
}

/* Lists and gathers the tokens, pads weight's rows where they need it, and fills what the
 * products of the call share. */
int prologue(const Call& c, const Plan& p, TokenArgs l, ProductArgs& a)
{
    Header* head = reinterpret_cast<Header*>(c.work);
    l.targets = c.targets;
    l.wide = c.target_bytes == 8;
    l.rows = (uint32_t)c.rows;
    l.vocab = c.vocab;
    l.dim = c.dim;
    l.pitch = p.pitch;
    l.head = head;
    l.token = reinterpret_cast<uint32_t*>(c.work + p.token);
    l.target = reinterpret_cast<int*>(c.work + p.target);
    l.lse_out = reinterpret_cast<float*>(c.work + p.lse);
    l.factor = reinterpret_cast<float*>(c.work + p.factor);
    l.f16 = c.dtype == ZERO_F16;
    const bool direct = c.rows < kAlignRows ? c.dim % 8 == 0 && c.hidden_stride % 8 == 0 && aligned_to(c.hidden, 16)
                                            : c.dim % 8 == 0 && c.hidden_stride % 64 == 0 && aligned_to(c.hidden, 128);
    l.direct = direct;
    l.hidden = static_cast<const uint16_t*>(c.hidden);
    l.hidden_stride = c.hidden_stride;
    uint16_t* gathered = reinterpret_cast<uint16_t*>(c.work + p.gathered);
    l.gathered = gathered;
    l.weight = static_cast<const uint16_t*>(c.weight);
    l.padded = p.pad ? reinterpret_cast<uint16_t*>(c.work + p.weight) : nullptr;
    const void* weight = p.pad ? l.padded : c.weight;
    memset(&a, 0, sizeof a);
    const uint64_t stride = c.rows > 1 ? c.hidden_stride : p.dim8, pitch_w = p.pad ? p.pitch : c.dim;
    if (!tensor_map(&a.gathered, gathered, c.dtype, c.dim, p.rows_pad, p.pitch, 64, kBoxRows) ||
        !tensor_map(&a.weight, weight, c.dtype, c.dim, c.vocab, pitch_w, 64, kBoxRows) ||
        (l.backward && !tensor_map(&a.d, c.work + p.d, c.dtype, p.piece, p.rows_pad, p.piece, 64, kBoxRows)) ||
        (direct && c.rows && !tensor_map(&a.hidden, c.hidden, c.dtype, c.dim, c.rows, stride, 64, kBoxRows)))
        return map_refused();
    if (!direct || !c.rows)
        a.hidden = a.gathered;
    a.head = head;
    a.target = l.target;
    a.factor = l.factor;
    a.lse = l.lse_out;
    a.target_logit = reinterpret_cast<float*>(c.work + p.logit);
    a.stats = reinterpret_cast<float2*>(c.work + p.stats);
    a.rows = (uint32_t)c.rows;
    a.rows_pad = p.rows_pad;
    a.dim = c.dim;
    a.dim8 = p.dim8;
    a.vocab = c.vocab;
    a.piece = p.piece;
    a.splits = 1;
    // row tiles whose hidden rows (32 MB) stay in L2 while weight passes by
    const uint64_t group = (32ull << 20) / (kTileM * 2ull * p.pitch);
    a.group = (uint32_t)(group ? group : 1);
    // tokens to at most a block per SM, 32 at least to each; rows to pad to all of them
    const uint64_t sms = (uint64_t)sm_count(), want = (c.rows + 31) / 32;
    l.blocks = (uint32_t)(want < sms ? (want ? want : 1) : sms);
    l.per = (uint32_t)up((c.rows + l.blocks - 1) / l.blocks, 32);
    cudaError_t e = allow_smem<k_head_tokens>();
    if (e == cudaSuccess)
        e = launch_pdl(k_head_tokens, dim3(p.pad ? (unsigned)sms : l.blocks), dim3(1024),
                       (size_t)l.per / 32 * 8, c.stream, l);
    return rows_status(e);
}

template <Mode MODE>
cudaError_t product(const ProductArgs& a, bool f16, uint64_t tiles, cudaStream_t s)
{
    auto* kernel = f16 ? k_head_product<MODE, true> : k_head_product<MODE, false>;
    const cudaError_t e = f16 ? allow_smem<k_head_product<MODE, true>>() : allow_smem<k_head_product<MODE, false>>();
    if (e != cudaSuccess)
        return e;
    const uint64_t pairs = (uint64_t)sm_count() / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * (tiles < pairs ? tiles : pairs)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = 2;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <zero_dtype_t GT>
cudaError_t join(const JoinArgs& j, uint64_t rows, bool vec, cudaStream_t s)
{
    const unsigned grid = warps_grid(rows * ((j.dim + 255) / 256));
    return vec ? launch_pdl(k_head_join<GT, true>, dim3(grid), dim3(256), 0, s, j)
               : launch_pdl(k_head_join<GT, false>, dim3(grid), dim3(256), 0, s, j);
}

cudaError_t join(const JoinArgs& j, uint64_t rows, zero_dtype_t t, bool vec, cudaStream_t s)
{
    return t == ZERO_F32   ? join<ZERO_F32>(j, rows, vec, s)
           : t == ZERO_F16 ? join<ZERO_F16>(j, rows, vec, s)
                           : join<ZERO_BF16>(j, rows, vec, s);
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

#ifdef ZERO_TEST_HOOKS
int zero_test_withhold_head_stage(unsigned long long stage)
{
    return cudaMemcpyToSymbol(zero_test_withheld_head_stage, &stage, sizeof stage) == cudaSuccess ? 0 : -4;
}
#endif

size_t zero_head_workspace_bytes(uint64_t rows, uint32_t dim, uint32_t vocab)
{
    return sizes_ok(rows, dim, vocab) ? (size_t)make_plan(rows, dim, vocab).bytes : 0;
}

int zero_head_loss(zero_dtype_t dtype, uint64_t rows, uint32_t dim, uint32_t vocab, const void* hidden,
                   uint64_t hidden_stride, const void* weight, const void* targets, uint32_t target_bytes, float* loss,
                   float* lse, void* workspace, zero_stream_t stream)
{
    NvtxRange range("zero_head_loss");
    const Call c{dtype,  rows,    dim,          vocab,  hidden, hidden_stride,
                 weight, targets, target_bytes, static_cast<char*>(workspace), stream};
    const uint64_t bytes = zero_head_workspace_bytes(rows, dim, vocab);
    int rc = check_call(c);
    if (rc == ZERO_EINVAL || (rows && (!loss || !lse)))
        return ZERO_EINVAL;
    if (rc != ZERO_OK || !aligned_to(loss, 4) || !aligned_to(lse, 4))
        return ZERO_EALIGN;
    if (!apart({{loss, rows * 4}, {lse, rows * 4}, {workspace, bytes}},
               {{hidden, rows, hidden_stride, dim, dtype}, {weight, 2ull * vocab * dim}, {targets, rows * target_bytes}}))
        return ZERO_EINVAL;
    if (rows == 0)
        return ZERO_OK;
    const Plan p = make_plan(rows, dim, vocab);
    TokenArgs l = {};
    l.loss = loss;
    l.lse = lse;
    ProductArgs a;
    rc = prologue(c, p, l, a);
    if (rc != ZERO_OK)
        return rc;
    a.cols = vocab;
    const uint32_t tiles = (vocab + kTileN - 1) / kTileN;
    cudaError_t e = product<kStats>(a, dtype == ZERO_F16, (uint64_t)p.rows_pad / kTileM * tiles, stream);
    if (e != cudaSuccess)
        return rows_status(e);
    const LossArgs j{a.head, reinterpret_cast<const uint32_t*>(c.work + p.token), a.stats, a.target_logit, loss, lse, 2 * tiles};
    return rows_status(launch_pdl(k_head_loss, dim3(warps_grid(rows)), dim3(256), 0, stream, j));
}

int zero_head_loss_backward(zero_dtype_t dtype, uint64_t rows, uint32_t dim, uint32_t vocab, const void* hidden,
                            uint64_t hidden_stride, const void* weight, const void* targets, uint32_t target_bytes,
                            const float* lse, float scale, const float* row_scale, zero_step_state_t* st,
                            void* dhidden, uint64_t dhidden_stride, void* dweight, zero_dtype_t grad_dtype,
                            uint32_t accumulate, void* workspace, zero_stream_t stream)
{
    NvtxRange range("zero_head_loss_backward");
    const Call c{dtype,  rows,    dim,          vocab,  hidden, hidden_stride,
                 weight, targets, target_bytes, static_cast<char*>(workspace), stream};
    const uint64_t bytes = zero_head_workspace_bytes(rows, dim, vocab);
    int rc = check_call(c);
    if (rc == ZERO_EINVAL || (rows && !lse) || (!dhidden && !dweight) || accumulate > 1 ||
        (dweight && grad_dtype != dtype && grad_dtype != ZERO_F32) || !(scale >= -3.0e38f && scale <= 3.0e38f) ||
        (dhidden && ((rows > 1 && dhidden_stride < dim) || dhidden_stride > (1ull << 32))))
        return ZERO_EINVAL;
    const size_t g = dtype_size(grad_dtype);
    if (rc != ZERO_OK || !aligned_to(lse, 4) || !aligned_to(row_scale, 4) || !aligned_to(st, 16) ||
        !aligned_to(dhidden, 2) || !aligned_to(dweight, g))
        return ZERO_EALIGN;
    if (!apart({{dhidden, rows, dhidden_stride, dim, dtype},
                {dweight, (uint64_t)vocab * dim * g},
                {workspace, bytes}},
               {{hidden, rows, hidden_stride, dim, dtype},
                {weight, 2ull * vocab * dim},
                {targets, rows * target_bytes},
                {lse, rows * 4},
                {row_scale, rows * 4},
                {st, sizeof *st}}))
        return ZERO_EINVAL;
    if (rows == 0 && (!dweight || accumulate))
        return ZERO_OK;
    const bool f16 = dtype == ZERO_F16;
    const Plan p = make_plan(rows, dim, vocab);
    TokenArgs l = {};
    l.dhidden = static_cast<uint16_t*>(dhidden);
    l.dhidden_stride = dhidden_stride;
    l.lse_in = lse;
    l.row_scale = row_scale;
    l.st = st;
    l.scale = scale;
    l.backward = 1;
    ProductArgs a;
    rc = prologue(c, p, l, a);
    if (rc != ZERO_OK)
        return rc;
    a.state_error = st ? &st->error : nullptr;
    a.grad_dtype = (uint32_t)grad_dtype;
    a.accumulate = accumulate;
    const bool whole = p.splits_w == 1 && dweight, vec = dweight && rows_vec(dweight, dim, dim, grad_dtype);
    a.dweight = dweight;
    a.bulk = whole && vec;
    a.splits = p.splits_w;
    a.want_h = dhidden != nullptr;
    a.want_w = dweight != nullptr;
    CUtensorMap out_d, out_h;
    float *sums_h = reinterpret_cast<float*>(c.work + p.sums_h), *sums_w = reinterpret_cast<float*>(c.work + p.sums_w);
    if (!tensor_map(&out_d, c.work + p.d, dtype, p.piece, p.rows_pad, p.piece, 64, 32) ||
        !tensor_map(&out_h, sums_h, ZERO_F32, p.dim8, p.rows_h, p.dim8, 32, 32) ||
        (a.bulk && !tensor_map(&a.out_w, dweight, grad_dtype, dim, vocab, dim, 32, 32)) ||
        (dweight && !whole &&
         !tensor_map(&a.out_w, sums_w, ZERO_F32, p.dim8, (uint64_t)p.splits_w * p.piece, p.dim8, 32, 32)))
        return map_refused();
    const uint64_t mt = p.rows_pad / kTileM;
    cudaError_t e = cudaSuccess;
    for (uint32_t v0 = 0; v0 < vocab && e == cudaSuccess; v0 += p.piece) {
        a.v0 = v0;
        a.cols = vocab - v0 < p.piece ? vocab - v0 : p.piece;
        a.first_piece = v0 == 0;
        a.out = out_d;
        e = product<kD>(a, f16, mt * ((a.cols + kTileN - 1) / kTileN), stream);
        if (e != cudaSuccess)
            break;
        a.out = out_h;
        e = product<kGrads>(a, f16, kSms / 2, stream);  // with the tokens' number it finds its tiles
        if (e == cudaSuccess && dweight && p.splits_w > 1) {
            const JoinArgs j{a.head, sums_w, nullptr, dweight, dim, (uint64_t)p.piece * p.dim8, a.cols, v0, dim,
                             p.dim8, p.splits_w, accumulate, 0};
            e = join(j, a.cols, grad_dtype, vec, stream);
        }
    }
    if (e == cudaSuccess && dhidden && rows) {
        const JoinArgs j{a.head,
                         sums_h,
                         reinterpret_cast<const uint32_t*>(c.work + p.token),
                         dhidden,
                         dhidden_stride,
                         0,
                         (uint32_t)rows,
                         0,
                         dim,
                         p.dim8,
                         0,
                         0,
                         ((vocab < p.piece ? vocab : p.piece) + kGradsK - 1) / kGradsK};
        e = join(j, rows, dtype, rows_vec(dhidden, dhidden_stride, dim, dtype), stream);
    }
    return rows_status(e);
}

}  // extern "C"
