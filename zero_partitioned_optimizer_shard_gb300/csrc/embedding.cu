/*
 * embedding.cu -- rows of a table by token id, with a scale, and the table's gradient summed
 * over the tokens in a fixed order.
 *
 * Forward: out[t] = scale * table[token[t]].
 * Backward: dtable[v] (+)= scale * (sum over the places t with token[t] = v of dout[t]).  The
 * places are sorted by token (stable), cut into chunks of a fixed number of sorted places, and each
 * chunk's tokens are summed in fp32 by one block, in the order of the places; a token whose places
 * lie in several chunks leaves one partial sum per chunk, which a second kernel adds in an order
 * that the chunks alone give.  No atomics on values: the same call gives the same bits.
 * Ids outside [0, vocab) sort behind all others and are dropped.
 */
#include "rows.cuh"

namespace zero {
namespace {

constexpr uint32_t kMaxDim = 65536;
constexpr uint32_t kPlaces = 16;      // sorted places per chunk, at most
constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kItems = 8;        // per thread and tile of the sort
constexpr uint32_t kTile = kSortThreads * kItems;
constexpr uint32_t kBins = 256;       // 8 bits of the key per pass
constexpr uint32_t kSortWarps = kSortThreads / 32;

struct Tokens {
    const void* p;
    uint32_t wide;  // 64-bit ids
    uint32_t vocab;

    /* The id at place t, or vocab where there is none. */
    __device__ __forceinline__ uint32_t at(uint32_t t) const
    {
        if (wide) {
            const uint64_t v = (uint64_t) * (static_cast<const volatile long long*>(p) + t);
            return v < vocab ? (uint32_t)v : vocab;
        }
        const uint32_t v = (uint32_t) * (static_cast<const volatile int*>(p) + t);
        return v < vocab ? v : vocab;
    }
};

/* ------------------------------------------------------------------------------------ */
/* forward                                                                                */
/* ------------------------------------------------------------------------------------ */
struct LookupArgs {
    Tokens tokens;
    const void* table;
    void* out;
    uint64_t out_stride;
    uint32_t n, d, pieces;  // pieces of a row: 32 chunks of 8 elements, a warp's
    float scale;
};

/* A warp takes W neighbouring pieces of rows, all in flight at a time.  A scale of 1 leaves the
 * values as they are, without a detour over fp32.  Bound by memory: 16,384 tokens of 4,096 bf16 from
 * a table of 32,000 take 29.8 us a call, 39.6 for reading each row that occurs once and writing
 * the output at the copy's rate (its writes stay in L2 in part).  With a warp to a piece, W = 1,
 * it was issue-bound (70% of the slots, 34.5 us). */
template <zero_dtype_t DT, bool VEC>
__global__ void __launch_bounds__(256) k_embedding(const LookupArgs a)
{
    using T = typename Elem<DT>::T;
    constexpr uint32_t W = 4;
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t lane = threadIdx.x & 31;
    const uint64_t first = ((uint64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)) * W;
    uint32_t row[W], at[W], id[W];
    row[0] = first >> 32 ? (uint32_t)(first / a.pieces) : (uint32_t)first / a.pieces;
    at[0] = (uint32_t)(first - (uint64_t)row[0] * a.pieces);
#pragma unroll
    for (uint32_t i = 1; i < W; ++i) {
        const bool next = at[i - 1] + 1 == a.pieces;
        row[i] = row[i - 1] + next;
        at[i] = next ? 0 : at[i - 1] + 1;
    }
#pragma unroll
    for (uint32_t i = 0; i < W; ++i)
        id[i] = row[i] < a.n ? a.tokens.at(row[i]) : 0xffffffffu;
    typename Elem<DT>::Raw x[W];
#pragma unroll
    for (uint32_t i = 0; i < W; ++i)
        x[i] = load_chunk<DT, VEC>(static_cast<const T*>(a.table) + (uint64_t)id[i] * a.d,
                                   id[i] < a.tokens.vocab ? a.d : 0, at[i], lane, 32);
#pragma unroll
    for (uint32_t i = 0; i < W; ++i) {
        if (id[i] == 0xffffffffu)
            return;
        T* out = static_cast<T*>(a.out) + row[i] * a.out_stride;
        if (VEC && a.scale == 1.0f) {
            const uint32_t c = at[i] * 32 + lane;
            if (c * 8 < a.d)
                *reinterpret_cast<typename Elem<DT>::Raw*>(out + c * 8) = x[i];
            continue;
        }
        float v[8];
        widen<DT>(x[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j)  // rows without a token: 0, whatever the scale
            v[j] = id[i] < a.tokens.vocab ? __fmul_rn(v[j], a.scale) : 0.0f;
        store_chunk<DT, VEC>(out, a.d, at[i], lane, 32, v);
    }
}

/* ------------------------------------------------------------------------------------ */
/* the sort: least significant digit first, 8 bits a pass, stable                         */
/* ------------------------------------------------------------------------------------ */
struct RankSmem {
    uint32_t of_warp[kSortWarps][kBins];  // counts, then offsets, of each warp's keys
    uint32_t base[kBins];                 // where a digit's keys begin
    uint32_t warp_total[8];
};

/* base[digit threadIdx.x] = first + the sum of `count` over the digits below. */
__device__ __forceinline__ void digit_base(RankSmem& sm, uint32_t count, uint32_t first)
{
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t sum = count;
    if (threadIdx.x < kBins) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
            sum += lane >= (uint32_t)o ? up : 0;
        }
        if (lane == 31)
            sm.warp_total[warp] = sum;
    }
    __syncthreads();
    if (threadIdx.x < kBins) {
        for (uint32_t w = 0; w < warp; ++w)
            first += sm.warp_total[w];
        sm.base[threadIdx.x] = first + sum - count;
    }
    __syncthreads();
}

/* Each thread's ITEMS keys (a warp's are 32 * ITEMS neighbours, taken 32 at a time) get
 * their rank among the tile's keys of the same digit, in the keys' order.  The answer is the
 * number of the tile's keys of digit threadIdx.x. */
template <uint32_t ITEMS>
__device__ __forceinline__ uint32_t rank_tile(RankSmem& sm, const uint32_t (&key)[ITEMS], uint32_t shift,
                                              uint32_t (&rank)[ITEMS])
{
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (uint32_t b = lane; b < kBins; b += 32)
        sm.of_warp[warp][b] = 0;
    __syncwarp();
#pragma unroll
    for (uint32_t i = 0; i < ITEMS; ++i) {
        const uint32_t digit = key[i] >> shift & (kBins - 1);
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        const uint32_t below = __popc(peers & ((1u << lane) - 1));
        const uint32_t before = sm.of_warp[warp][digit];
        __syncwarp();
        if (below == 0)
            sm.of_warp[warp][digit] = before + __popc(peers);
        __syncwarp();
        rank[i] = before + below;
    }
    __syncthreads();
    uint32_t count = 0;
    if (threadIdx.x < kBins) {
#pragma unroll 8
        for (uint32_t w = 0; w < kSortWarps; ++w) {
            const uint32_t c = sm.of_warp[w][threadIdx.x];
            sm.of_warp[w][threadIdx.x] = count;
            count += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < ITEMS; ++i)
        rank[i] += sm.of_warp[warp][key[i] >> shift & (kBins - 1)];
    return count;
}

/* A barrier over the cluster; what its blocks wrote before is seen behind it. */
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n"
                 "barrier.cluster.wait.acquire;" ::: "memory");
}

/* This address in shared memory as block b of the cluster has it. */
__device__ __forceinline__ uint32_t of_block(const uint32_t* p, uint32_t b)
{
    uint32_t at, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(b));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

/* The place in its tile of item i of the calling thread. */
template <uint32_t ITEMS>
__device__ __forceinline__ uint32_t item_at(uint32_t i)
{
    return (threadIdx.x >> 5) * 32 * ITEMS + i * 32 + (threadIdx.x & 31);
}

struct SortArgs {
    Tokens tokens;
    uint2* from;       // (token, place), or null: the caller's ids, place = index
    uint2* to;
    uint32_t* hist;    // [kBins][tiles]
    uint32_t n, tiles, shift;
};

__device__ __forceinline__ uint2 sort_item(const SortArgs& a, uint32_t i)
{
    if (i >= a.n)
        return make_uint2(0xffffffffu, 0);
    return a.from ? a.from[i] : make_uint2(a.tokens.at(i), i);
}

__global__ void __launch_bounds__(kSortThreads) k_sort_count(const SortArgs a)
{
    __shared__ uint32_t count[kBins];
    grid_dependency_wait();
    if (threadIdx.x < kBins)
        count[threadIdx.x] = 0;
    __syncthreads();
    for (uint32_t i = 0; i < kItems; ++i) {
        const uint32_t at = blockIdx.x * kTile + item_at<kItems>(i);
        if (at < a.n)
            atomicAdd(&count[sort_item(a, at).x >> a.shift & (kBins - 1)], 1u);
    }
    __syncthreads();
    if (threadIdx.x < kBins)
        a.hist[threadIdx.x * a.tiles + blockIdx.x] = count[threadIdx.x];
}

/* Exclusive sums of the histogram (digit major), in place, by one block. */
__global__ void __launch_bounds__(kSortThreads) k_sort_scan(uint32_t* hist, uint32_t n)
{
    __shared__ uint32_t total[kSortWarps];
    grid_dependency_wait();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t carry = 0;
    for (uint32_t at = 0; at < n; at += kSortThreads) {
        const uint32_t i = at + threadIdx.x;
        const uint32_t x = i < n ? hist[i] : 0;
        uint32_t sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
            sum += lane >= (uint32_t)o ? up : 0;
        }
        if (lane == 31)
            total[warp] = sum;
        __syncthreads();
        uint32_t more = carry, all = carry;
        for (uint32_t w = 0; w < kSortWarps; ++w) {
            more += w < warp ? total[w] : 0;
            all += total[w];
        }
        if (i < n)
            hist[i] = more + sum - x;
        carry = all;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads) k_sort_scatter(const SortArgs a)
{
    extern __shared__ uint4 smem[];
    RankSmem& sm = *reinterpret_cast<RankSmem*>(smem);
    grid_dependency_wait();
    uint32_t key[kItems], place[kItems], rank[kItems];
#pragma unroll
    for (uint32_t i = 0; i < kItems; ++i) {
        const uint2 x = sort_item(a, blockIdx.x * kTile + item_at<kItems>(i));
        key[i] = x.x;
        place[i] = x.y;
    }
    rank_tile(sm, key, a.shift, rank);
#pragma unroll
    for (uint32_t i = 0; i < kItems; ++i)
        if (blockIdx.x * kTile + item_at<kItems>(i) < a.n)
            a.to[a.hist[(key[i] >> a.shift & (kBins - 1)) * a.tiles + blockIdx.x] + rank[i]] =
                make_uint2(key[i], place[i]);
}

struct Fill {
    uint4* p;
    uint64_t n16;
    uint8_t* tail;
    uint32_t tail_bytes;
};

__device__ __forceinline__ void zero_fill(const Fill& f, uint32_t block, uint32_t blocks)
{
    for (uint64_t i = (uint64_t)block * blockDim.x + threadIdx.x; i < f.n16; i += (uint64_t)blocks * blockDim.x)
        f.p[i] = make_uint4(0, 0, 0, 0);
    if (block == 0 && threadIdx.x < f.tail_bytes)
        f.tail[threadIdx.x] = 0;
}

__global__ void __launch_bounds__(512) k_zero_fill(const Fill f)
{
    grid_dependency_wait();
    zero_fill(f, blockIdx.x, gridDim.x);
}

struct SmallSmem {
    RankSmem rank;
    uint2 item[2 * kSortThreads];
};

/* All passes over at most 1,024 * ITEMS tokens, by block 0, while the other blocks write the
 * table's zeros. */
template <uint32_t ITEMS>
__global__ void __launch_bounds__(kSortThreads) k_sort_small(const SortArgs a, const uint32_t bits, const Fill f)
{
    extern __shared__ uint4 smem[];
    SmallSmem& sm = *reinterpret_cast<SmallSmem*>(smem);
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x) {
        zero_fill(f, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    uint32_t key[ITEMS], place[ITEMS], rank[ITEMS];
#pragma unroll
    for (uint32_t i = 0; i < ITEMS; ++i) {
        const uint2 x = sort_item(a, item_at<ITEMS>(i));
        key[i] = x.x;
        place[i] = x.y;
    }
    for (uint32_t shift = 0; shift < bits; shift += 8) {
        digit_base(sm.rank, rank_tile(sm.rank, key, shift, rank), 0);
#pragma unroll
        for (uint32_t i = 0; i < ITEMS; ++i)
            sm.item[sm.rank.base[key[i] >> shift & (kBins - 1)] + rank[i]] = make_uint2(key[i], place[i]);
        __syncthreads();
#pragma unroll
        for (uint32_t i = 0; i < ITEMS; ++i) {
            const uint2 x = sm.item[item_at<ITEMS>(i)];
            key[i] = x.x;
            place[i] = x.y;
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < ITEMS; ++i)
        if (item_at<ITEMS>(i) < a.n)
            a.to[item_at<ITEMS>(i)] = make_uint2(key[i], place[i]);
}

/* All passes over at most 8 * 1,024 * ITEMS tokens, by the first cluster: each of its 8 blocks
 * ranks a tile, the blocks read each other's counts of a digit, and the items change places
 * through memory, to[] and other[] in turn.  The other clusters write the table's zeros meanwhile
 * (161 MB of them take 26 us, the sort of 8,192 tokens less).  A pass is bound by its steps one
 * after another: three barriers of the block, two of the cluster.  By one block 8,192 tokens took 11 us
 * more; 16,384 in launches of their own, with the zeros before them, 40 more (97 -> 57 us for the whole gradient
 * of a 50,257 x 1,600 table). */
constexpr uint32_t kCluster = 8;

template <uint32_t ITEMS>
__global__ void __launch_bounds__(kSortThreads) k_sort_cluster(const SortArgs a, uint2* const other, const uint32_t bits,
                                                               const Fill f)
{
    extern __shared__ uint4 smem[];
    RankSmem& sm = *reinterpret_cast<RankSmem*>(smem);
    __shared__ uint32_t count[kBins];  // of the tile, for the cluster
    grid_dependency_wait();
    grid_launch_dependents();
    if (blockIdx.x >= kCluster) {
        zero_fill(f, blockIdx.x - kCluster, gridDim.x - kCluster);
        return;
    }
    const uint32_t first = blockIdx.x * kSortThreads * ITEMS;
    uint2* to = a.to;
    for (uint32_t shift = 0; shift < bits; shift += 8) {
        uint32_t key[ITEMS], place[ITEMS], rank[ITEMS];
#pragma unroll
        for (uint32_t i = 0; i < ITEMS; ++i) {
            const uint32_t at = first + item_at<ITEMS>(i);
            uint2 x = make_uint2(0xffffffffu, 0);
            if (at < a.n)
                x = shift ? __ldcg((to == a.to ? other : a.to) + at) : make_uint2(a.tokens.at(at), at);
            key[i] = x.x;
            place[i] = x.y;
        }
        const uint32_t mine = rank_tile(sm, key, shift, rank);
        if (threadIdx.x < kBins)
            count[threadIdx.x] = mine;
        cluster_sync();
        uint32_t before = 0, all = 0;
        if (threadIdx.x < kBins) {
#pragma unroll
            for (uint32_t b = 0; b < kCluster; ++b) {
                const uint32_t c = of_block(&count[threadIdx.x], b);
                before += b < blockIdx.x ? c : 0;
                all += c;
            }
        }
        digit_base(sm, all, before);
#pragma unroll
        for (uint32_t i = 0; i < ITEMS; ++i)
            if (first + item_at<ITEMS>(i) < a.n)
                to[sm.base[key[i] >> shift & (kBins - 1)] + rank[i]] = make_uint2(key[i], place[i]);
        cluster_sync();
        to = to == a.to ? other : a.to;
    }
}

/* ------------------------------------------------------------------------------------ */
/* backward: the sums                                                                     */
/* ------------------------------------------------------------------------------------ */
struct GradArgs {
    const uint2* sorted;  // (token, place)
    uint32_t* last;       // [vocab]: the last sorted place of each token that occurs
    const void* dout;
    float* head;          // [chunks][d]: sums of the token that continues from an earlier chunk
    float* tail;          // [chunks][d]: sums of the token that starts here and goes on
    void* dtable;
    uint64_t dout_stride;
    uint32_t n, d, vocab;
    uint32_t places;      // sorted places per chunk: 16, or 8 of few tokens
    uint32_t accumulate;
    float scale;
};

template <zero_dtype_t GT>
__device__ __forceinline__ typename Elem<GT>::T* grad_row(const GradArgs& a, uint32_t token)
{
    return static_cast<typename Elem<GT>::T*>(a.dtable) + (uint64_t)token * a.d;
}

/* One row's piece of the gradient, with the scale, added to what was there (add). */
template <zero_dtype_t GT, bool VEC>
__device__ __forceinline__ void put_grad(const GradArgs& a, uint32_t token, uint32_t i, uint32_t k, uint32_t n,
                                         const float (&s)[8], bool add, const typename Elem<GT>::Raw& old)
{
    float v[8];
    widen<GT>(old, v);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = add ? __fmaf_rn(s[j], a.scale, v[j]) : __fmul_rn(s[j], a.scale);
    store_chunk<GT, VEC>(grad_row<GT>(a, token), a.d, i, k, n, v);
}

/* A block per chunk of sorted places and (rows beyond 2,048 elements) piece of the row, Q rows in
 * flight to a thread.  Bound by memory and by the chunk's latency: 8,192 rows of 1,600 bf16 take 10
 * us, 26 MB at 2.6 TB/s.  A chunk is 16 places, so that few tokens reach over two of them and
 * a block still has two turns of loads; of few tokens 8, for twice the blocks.  What rows are added
 * to (ADD) is loaded with the places that end them: row after row it was a round trip each (the whole call on 8,192
 * rows of 1,600 33.6 us, so 31.5). */
template <zero_dtype_t DT, zero_dtype_t GT, bool VEC, bool ADD>
__global__ void __launch_bounds__(256) k_embedding_sum(const GradArgs a)
{
    using T = typename Elem<DT>::T;
    __shared__ uint2 item[kPlaces + 2];  // the chunk's, between its neighbours
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t chunk = blockIdx.x, lo = chunk * a.places;
    const uint32_t len = a.n - lo < a.places ? a.n - lo : a.places;
    if (threadIdx.x < a.places + 2) {
        const uint32_t i = lo + threadIdx.x;  // of sorted place i - 1
        item[threadIdx.x] = i >= 1 && i <= a.n ? a.sorted[i - 1] : make_uint2(0xffffffffu, 0);
    }
    __syncthreads();
    if (blockIdx.y == 0 && threadIdx.x >= 1 && threadIdx.x <= len) {
        const uint32_t k = threadIdx.x, token = item[k].x;
        if (token < a.vocab && item[k + 1].x != token)
            a.last[token] = lo + k - 1;
    }
    const uint32_t n = blockDim.x, piece = blockIdx.y, k = threadIdx.x;
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    bool from_before = item[0].x == item[1].x;
    // places in flight; element by element 8 take 168 registers (8,192 rows of 1,001: 66 us a call, 53 with 4)
    constexpr uint32_t Q = VEC ? 8 : 4;
    for (uint32_t at = 0; at < len; at += Q) {
        typename Elem<DT>::Raw x[Q];
        typename Elem<GT>::Raw old[Q];
#pragma unroll
        for (uint32_t q = 0; q < Q; ++q) {
            const uint2 it = item[1 + (at + q < len ? at + q : 0)];
            x[q] = load_chunk<DT, VEC>(static_cast<const T*>(a.dout) + it.y * a.dout_stride,
                                       at + q < len && it.x < a.vocab ? a.d : 0, piece, k, n);
            old[q] = {};
            if constexpr (ADD) {
                const bool here = at + q < len && it.x < a.vocab && it.x != item[0].x && it.x != item[2 + at + q].x;
                old[q] = load_chunk<GT, VEC>(grad_row<GT>(a, here ? it.x : 0), here ? a.d : 0, piece, k, n);
            }
        }
#pragma unroll
        for (uint32_t q = 0; q < Q; ++q) {
            if (at + q >= len)
                break;
            const uint32_t token = item[1 + at + q].x;
            if (token >= a.vocab)
                return;  // no token from here on
            float v[8];
            widen<DT>(x[q], v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[j] = __fadd_rn(s[j], v[j]);
            const bool ends = item[2 + at + q].x != token;
            if (!ends && at + q + 1 < len)
                continue;
            if (from_before)
                store_chunk<ZERO_F32, VEC>(a.head + (uint64_t)chunk * a.d, a.d, piece, k, n, s);
            else if (ends)
                put_grad<GT, VEC>(a, token, piece, k, n, s, ADD, old[q]);
            else
                store_chunk<ZERO_F32, VEC>(a.tail + (uint64_t)chunk * a.d, a.d, piece, k, n, s);
            from_before = false;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[j] = 0.0f;
        }
    }
}

/* Tokens over several chunks: their partial sums.  A block looks at the last tokens of `per` chunks
 * (at most 8); for each that starts in its chunk and goes on, 8 warps sum every eighth of the partials
 * each, over 32 places of the row's piece, then the 8 results are added: always in that order.  7 us,
 * nearly all of it launch and one round trip; a token in half of a million places takes a block
 * thousands of turns (524,288 places of 256 elements, L2 flushed: 2.1 ms where all hold one token, 1.1 where
 * half do; a padding id belongs outside the table, where it costs nothing). */
template <zero_dtype_t GT, bool VEC>
__global__ void __launch_bounds__(256) k_embedding_join(const GradArgs a, const uint32_t per)
{
    __shared__ float part[8][8][33];
    __shared__ uint32_t owner[8];  // the token, or none
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t lane = threadIdx.x & 31, run = threadIdx.x >> 5, piece = blockIdx.y;
    if (lane == 0) {
        const uint32_t end = (blockIdx.x * per + run + 1) * a.places;
        uint32_t token = 0xffffffffu;
        if (run < per && end < a.n) {
            const uint32_t before = end > a.places ? a.sorted[end - a.places - 1].x : 0xffffffffu;
            const uint32_t last = a.sorted[end - 1].x, next = a.sorted[end].x;
            token = last < a.vocab && next == last && before != last ? last : token;
        }
        owner[run] = token;
    }
    __syncthreads();
    for (uint32_t o = 0; o < per; ++o) {
        const uint32_t token = owner[o], chunk = blockIdx.x * per + o;
        if (token == 0xffffffffu)
            continue;
        const uint32_t chunks = a.last[token] / a.places - chunk;  // with a partial in head[]
        float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (run == 0)
            widen<ZERO_F32>(load_chunk<ZERO_F32, VEC>(a.tail + (uint64_t)chunk * a.d, a.d, piece, lane, 32), s);
#pragma unroll 4
        for (uint32_t c = run; c < chunks; c += 8) {
            float v[8];
            widen<ZERO_F32>(load_chunk<ZERO_F32, VEC>(a.head + (uint64_t)(chunk + 1 + c) * a.d, a.d, piece, lane, 32), v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s[j] = __fadd_rn(s[j], v[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            part[run][j][lane] = s[j];
        __syncthreads();
        if (run == 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    s[j] = __fadd_rn(s[j], part[r][j][lane]);
            put_grad<GT, VEC>(a, token, piece, lane, 32, s, a.accumulate,
                              load_chunk<GT, VEC>(grad_row<GT>(a, token), a.accumulate ? a.d : 0, piece, lane, 32));
        }
        __syncthreads();
    }
}

/* ------------------------------------------------------------------------------------ */
/* host side                                                                              */
/* ------------------------------------------------------------------------------------ */
struct Workspace {
    uint64_t sorted[2], hist, last, head, tail, bytes;
};

/* Few tokens: twice as many blocks, of half the length. */
uint32_t places_of(uint64_t n) { return n <= 4096 ? kPlaces / 2 : kPlaces; }

uint64_t up16(uint64_t x) { return (x + 15) / 16 * 16; }

Workspace layout(uint64_t n, uint32_t d, uint32_t vocab)
{
    Workspace w;
    const uint64_t tiles = (n + kTile - 1) / kTile, places = places_of(n), chunks = (n + places - 1) / places;
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t p = at;
        at += up16(bytes);
        return p;
    };
    w.sorted[0] = take(n * 8);
    w.sorted[1] = take(n * 8);
    w.hist = take((uint64_t)kBins * tiles * 4);
    w.last = take((uint64_t)vocab * 4);
    w.head = take(chunks * d * 4);
    w.tail = take(chunks * d * 4);
    w.bytes = at ? at : 16;
    return w;
}

bool sizes_ok(uint64_t n, uint32_t d, uint32_t vocab)
{
    return n <= (1ull << 28) && d >= 1 && d <= kMaxDim && vocab >= 1 && vocab <= (1u << 30);
}

template <zero_dtype_t DT>
cudaError_t lookup(const LookupArgs& a, bool vec, cudaStream_t s)
{
    const uint64_t warps = ((uint64_t)a.n * a.pieces + 3) / 4;
    const dim3 grid((unsigned)((warps + 7) / 8));
    return vec ? launch_pdl(k_embedding<DT, true>, grid, dim3(256), 0, s, a)
               : launch_pdl(k_embedding<DT, false>, grid, dim3(256), 0, s, a);
}

template <zero_dtype_t DT, zero_dtype_t GT, bool VEC>
cudaError_t sums(const GradArgs& a, cudaStream_t s)
{
    auto* kernel = a.accumulate ? k_embedding_sum<DT, GT, VEC, true> : k_embedding_sum<DT, GT, VEC, false>;
    const uint32_t chunks = (a.n + a.places - 1) / a.places, eights = (a.d + 7) / 8;
    const uint32_t threads = eights < 256 ? (eights + 31) / 32 * 32 : 256;
    cudaError_t e = launch_pdl(kernel, dim3(chunks, (eights + threads - 1) / threads),
                               dim3(threads), 0, s, a);
    if (e != cudaSuccess)
        return e;
    // a wave of blocks or two, as few chunks to a block as that allows
    const uint32_t pieces = (eights + 31) / 32, per = chunks * pieces <= 1216 ? 1 : chunks * pieces <= 4864 ? 4 : 8;
    return launch_pdl(k_embedding_join<GT, VEC>, dim3((chunks + per - 1) / per, pieces), dim3(256), 0, s, a, per);
}

template <zero_dtype_t DT, zero_dtype_t GT>
cudaError_t sums(const GradArgs& a, bool vec, cudaStream_t s)
{
    return vec ? sums<DT, GT, true>(a, s) : sums<DT, GT, false>(a, s);
}

Fill fill_of(void* p, uint64_t bytes)
{
    const uint64_t n16 = aligned_to(p, 16) ? bytes / 16 : 0;
    return {static_cast<uint4*>(p), n16, static_cast<uint8_t*>(p) + n16 * 16, (uint32_t)(bytes - n16 * 16)};
}

template <uint32_t ITEMS>
cudaError_t sort_small(const SortArgs& a, uint32_t bits, const Fill& f, unsigned fillers, cudaStream_t s)
{
    const cudaError_t e = allow_smem<k_sort_small<ITEMS>>();
    return e != cudaSuccess ? e
                            : launch_pdl(k_sort_small<ITEMS>, dim3(1 + fillers), dim3(kSortThreads), sizeof(SmallSmem), s,
                                         a, bits, f);
}

/* The first cluster sorts, the others fill: as many as fit at once (35 with it; a second wave of
 * three more cost 2 us of 40). */
template <uint32_t ITEMS>
cudaError_t sort_cluster(const SortArgs& a, uint2* other, uint32_t bits, const Fill& f, cudaStream_t s)
{
    static std::atomic<uint64_t> last{0};  // device + 1, clusters
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sizeof(RankSmem);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    if (f.n16 || f.tail_bytes) {
        int dev = 0, fit = 0;
        cudaError_t e = cudaGetDevice(&dev);
        const uint64_t have = last.load(std::memory_order_relaxed);
        if (e == cudaSuccess && have >> 32 == (uint64_t)dev + 1) {
            fit = (int)(uint32_t)have;
        } else if (e == cudaSuccess) {
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&fit, k_sort_cluster<ITEMS>, &cfg);
            cfg.numAttrs = 2;
            if (e == cudaSuccess)
                last.store((uint64_t)(dev + 1) << 32 | (uint32_t)fit, std::memory_order_relaxed);
        }
        if (e != cudaSuccess)
            return e;
        const uint64_t want = (f.n16 + 4096 * kCluster - 1) / (4096 * kCluster), most = fit > 2 ? fit - 1 : 1;
        cfg.gridDim = dim3((unsigned)(kCluster * (1 + (want < most ? (want ? want : 1) : most))));
    }
    return cudaLaunchKernelEx(&cfg, k_sort_cluster<ITEMS>, a, other, bits, f);
}

/* Zeros over the table's gradient (bytes of it, 0: none) and the tokens' places in order. */
cudaError_t fill_and_sort(const Tokens& tokens, uint32_t n, void* table, uint64_t bytes, uint2* buf[2], uint32_t* hist,
                          const uint2*& sorted, cudaStream_t s)
{
    uint32_t bits = 1;
    while (bits < 32 && tokens.vocab >> bits)
        ++bits;  // of the largest key, vocab itself
    const uint32_t tiles = (n + kTile - 1) / kTile;
    cudaError_t e = cudaSuccess;
    if (bytes && !aligned_to(table, 16)) {
        e = cudaMemsetAsync(table, 0, bytes, s);
        if (e != cudaSuccess)
            return e;
        bytes = 0;
    }
    const Fill f = fill_of(table, bytes);
    const uint64_t want = (f.n16 + 4095) / 4096, cap = (uint64_t)sm_count() * 2 - 1;
    const unsigned fillers = bytes ? (unsigned)(want < cap ? (want ? want : 1) : cap) : 0;
    SortArgs a{tokens, nullptr, buf[0], hist, n, tiles, 0};
    // one block up to 2,048 tokens (14.9 us for a whole call there, a cluster 17.0), a cluster up to
    // 65,536 (of 8,192 tokens: 32.4 us, one block 43.6; of 65,536: 67, launches of a step each 80)
    if (n && n <= 2 * kSortThreads) {
        sorted = buf[0];
        return n <= kSortThreads ? sort_small<1>(a, bits, f, fillers, s) : sort_small<2>(a, bits, f, fillers, s);
    }
    if (n && n <= kCluster * kTile) {
        const uint32_t each = (n + kCluster * kSortThreads - 1) / (kCluster * kSortThreads);
        sorted = buf[(bits + 7) / 8 & 1 ? 0 : 1];
        return each <= 1   ? sort_cluster<1>(a, buf[1], bits, f, s)
               : each <= 2 ? sort_cluster<2>(a, buf[1], bits, f, s)
               : each <= 4 ? sort_cluster<4>(a, buf[1], bits, f, s)
                           : sort_cluster<8>(a, buf[1], bits, f, s);
    }
    if (fillers)
        e = launch_pdl(k_zero_fill, dim3(fillers * 2), dim3(512), 0, s, f);
    for (uint32_t turn = 0; tiles && a.shift < bits && e == cudaSuccess; a.shift += 8, ++turn) {
        a.to = buf[turn & 1];
        e = launch_pdl(k_sort_count, dim3(tiles), dim3(kSortThreads), 0, s, a);
        if (e == cudaSuccess)
            e = launch_pdl(k_sort_scan, dim3(1), dim3(kSortThreads), 0, s, hist, tiles * kBins);
        if (e == cudaSuccess)
            e = launch_pdl(k_sort_scatter, dim3(tiles), dim3(kSortThreads), sizeof(RankSmem), s, a);
        a.from = a.to;
    }
    sorted = a.from;
    return e;
}

}  // namespace
}  // namespace zero

using namespace zero;

extern "C" {

int zero_embedding(zero_dtype_t dtype, uint64_t n_tokens, uint32_t dim, uint32_t vocab, const void* tokens,
                   uint32_t token_bytes, const void* table, float scale, void* out, uint64_t out_stride,
                   zero_stream_t stream)
{
    NvtxRange range("zero_embedding");
    if (!float_dtype(dtype) || !sizes_ok(n_tokens, dim, vocab) || (token_bytes != 4 && token_bytes != 8) ||
        !(scale >= -3.0e38f && scale <= 3.0e38f))
        return ZERO_EINVAL;
    if (n_tokens == 0)
        return ZERO_OK;
    if (!tokens || !table || !out || (n_tokens > 1 && out_stride < dim) || out_stride > (1ull << 32))
        return ZERO_EINVAL;
    const size_t e = dtype_size(dtype);
    if (!aligned_to(tokens, token_bytes) || !aligned_to(table, e) || !aligned_to(out, e))
        return ZERO_EALIGN;
    if (!apart({{out, n_tokens, out_stride, dim, dtype}}, {{table, (uint64_t)vocab * dim * e}, {tokens, n_tokens * token_bytes}}))
        return ZERO_EINVAL;
    const LookupArgs a{{tokens, token_bytes == 8, vocab}, table, out, out_stride, (uint32_t)n_tokens, dim,
                       (dim + 255) / 256, scale};
    const bool vec = rows_vec(table, dim, dim, dtype) && rows_vec(out, out_stride, dim, dtype);
    return rows_status(dtype == ZERO_BF16  ? lookup<ZERO_BF16>(a, vec, stream)
                       : dtype == ZERO_F16 ? lookup<ZERO_F16>(a, vec, stream)
                                           : lookup<ZERO_F32>(a, vec, stream));
}

size_t zero_embedding_workspace_bytes(uint64_t n_tokens, uint32_t dim, uint32_t vocab)
{
    return sizes_ok(n_tokens, dim, vocab) ? (size_t)layout(n_tokens, dim, vocab).bytes : 0;
}

int zero_embedding_backward(zero_dtype_t dtype, uint64_t n_tokens, uint32_t dim, uint32_t vocab, const void* tokens,
                            uint32_t token_bytes, const void* dout, uint64_t dout_stride, float scale, void* dtable,
                            zero_dtype_t grad_dtype, uint32_t accumulate, void* workspace, zero_stream_t stream)
{
    NvtxRange range("zero_embedding_backward");
    if (!float_dtype(dtype) || (grad_dtype != dtype && grad_dtype != ZERO_F32) || accumulate > 1 ||
        !sizes_ok(n_tokens, dim, vocab) || (token_bytes != 4 && token_bytes != 8) ||
        !(scale >= -3.0e38f && scale <= 3.0e38f) || !dtable || !workspace)
        return ZERO_EINVAL;
    if (n_tokens && (!tokens || !dout || (n_tokens > 1 && dout_stride < dim) || dout_stride > (1ull << 32)))
        return ZERO_EINVAL;
    if (!aligned_to(tokens, token_bytes) || !aligned_to(dout, dtype_size(dtype)) ||
        !aligned_to(dtable, dtype_size(grad_dtype)) || !aligned_to(workspace, 16))
        return ZERO_EALIGN;
    const Workspace w = layout(n_tokens, dim, vocab);
    const uint64_t nt = (uint64_t)vocab * dim * dtype_size(grad_dtype);
    if (!apart({{dtable, nt}, {workspace, w.bytes}},
               {{dout, n_tokens, dout_stride, dim, dtype}, {tokens, n_tokens * token_bytes}}))
        return ZERO_EINVAL;
    char* base = static_cast<char*>(workspace);
    uint2* buf[2] = {reinterpret_cast<uint2*>(base + w.sorted[0]), reinterpret_cast<uint2*>(base + w.sorted[1])};
    const uint2* sorted = nullptr;
    const int rc = rows_status(fill_and_sort({tokens, token_bytes == 8, vocab}, (uint32_t)n_tokens, dtable,
                                             accumulate ? 0 : nt, buf, reinterpret_cast<uint32_t*>(base + w.hist), sorted,
                                             stream));
    if (rc != ZERO_OK || n_tokens == 0)
        return rc;
    const GradArgs a{sorted,
                     reinterpret_cast<uint32_t*>(base + w.last),
                     dout,
                     reinterpret_cast<float*>(base + w.head),
                     reinterpret_cast<float*>(base + w.tail),
                     dtable,
                     dout_stride,
                     (uint32_t)n_tokens,
                     dim,
                     vocab,
                     places_of(n_tokens),
                     accumulate,
                     scale};
    const bool vec = rows_vec(dout, dout_stride, dim, dtype) && rows_vec(dtable, dim, dim, grad_dtype);
    if (grad_dtype == ZERO_F32)
        return rows_status(dtype == ZERO_BF16  ? sums<ZERO_BF16, ZERO_F32>(a, vec, stream)
                           : dtype == ZERO_F16 ? sums<ZERO_F16, ZERO_F32>(a, vec, stream)
                                               : sums<ZERO_F32, ZERO_F32>(a, vec, stream));
    return rows_status(dtype == ZERO_BF16 ? sums<ZERO_BF16, ZERO_BF16>(a, vec, stream)
                                          : sums<ZERO_F16, ZERO_F16>(a, vec, stream));
}

}  // extern "C"
