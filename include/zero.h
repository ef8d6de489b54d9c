/*
 * zero.h -- C ABI of the GB300 (sm_103a) ZeRO-DP partitioned mixed-precision AdamW step.
 *
 * One optimizer step of ZeRO-DP data parallelism with all N data-parallel ranks held as
 * buffers on one GPU (or, through the rank-local entry points, spread over processes):
 *   1. partition      Psi flat parameters into N equal, padded shards (rank r owns
 *                     flat [r*S, (r+1)*S)), with the per-rank model-state ledger
 *   2. reduce-scatter average the N ranks' fp16/bf16 gradient copies into fp32, remove
 *                     the loss scale, flag inf/NaN, and sum g^2 per tile of a shard
 *   3. grad norm      global L2 norm of the averaged gradient, clip coefficient,
 *                     loss-scale update and the skip decision, all on the device
 *   4. AdamW + cast   update the fp32 master / momentum / variance of every shard and
 *                     write each shard's bf16 parameters at its own offset r*S of one
 *                     gathered buffer (the layout the parameter all-gather produces);
 *                     the state may also live in host memory
 * plus the per-tensor segment map (which rank owns which piece of each model tensor).
 * zero_step runs steps 2-4 as one kernel per part (a reduce per gradient bucket, the
 * norm, AdamW) on large layouts and as ONE cooperative kernel, with the same bits, on
 * small ones (zero_step_launches).
 *
 * Sources (web pages on ZeRO):
 *   [ZW] "【论文解读】ZeRO", wkq9411.github.io: sec. 4(1)-(3) the three partitioning stages,
 *        sec. 6(1)-(2) reduce-scatter / all-gather and the 8-parameter, 4-GPU example
 *   [ZM] "ZeRO 显存优化：ZeRO-1、ZeRO-2 与 ZeRO-3", xiangdong0520.pages.dev: sec. 2-3 ledger,
 *        sec. 6 optimizer state offloaded to the CPU
 *   [ZS] operatorworld.com ZeRO optimizer-sharding article: AdamW 16-byte ledger (bf16
 *        weights and gradients), stage flows, communication accounting
 *   [ZO] "3、ZeRO技术概述：ZeRO三个阶段原理与对比", 5688vip.com: stage-2 iteration flow,
 *        DeepSpeed config with "fp16": enabled
 *   [MD] gitcode.csdn.net article on Megatron's distributed optimizer: sec. 1 global
 *        grad-norm all-reduce before clip_coeff
 *
 * Conventions for every function below:
 *   - Ownership: the caller allocates and frees every buffer.  No function allocates or
 *     frees device memory; zero_step_host creates and destroys four CUDA events.
 *   - Device pointers must be 16-byte aligned (ZERO_EALIGN otherwise) where an entry point
 *     does not say otherwise.
 *   - Asynchrony: device work is enqueued on the caller's stream and the call returns
 *     without waiting, except zero_step_state_read / zero_step_state_write, which wait.
 *   - Errors: arguments are validated on the host before anything is enqueued; a
 *     rejected call changes nothing.  A launch failure returns ZERO_ECUDA and
 *     zero_last_cuda_error() gives the CUDA error code.  Faults inside kernels surface at
 *     the caller's next synchronisation.  Overflow of the gradients is not an error: it
 *     is reported in the step state and the step is skipped.
 *   - Thread safety: calls on different streams may run concurrently if they share no
 *     buffers.
 *   - Profiling: every device entry point opens an NVTX range named after itself.
 */
#ifndef ZERO_H
#define ZERO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The CUDA runtime's cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st* zero_stream_t;

#define ZERO_OK 0
#define ZERO_EINVAL (-1)   /* invalid argument */
#define ZERO_EALIGN (-2)   /* pointer or window not aligned as required */
#define ZERO_ENOMEM (-3)   /* caller-provided buffer too small */
#define ZERO_ECUDA (-4)    /* CUDA launch or copy failed; see zero_last_cuda_error() */
#define ZERO_ETIMEOUT (-5) /* reserved; a device wait that gives up records 1 in the step
                              state's error word instead */

/* The flat entry points take ZERO_F16 and ZERO_BF16; the entry points over lists of tensors
 * also ZERO_F32 (gradients, states) and ZERO_U8 (block-scaled 8-bit states). */
typedef enum zero_dtype { ZERO_F16 = 1, ZERO_BF16 = 2, ZERO_F32 = 3, ZERO_U8 = 4 } zero_dtype_t;

#define ZERO_MAX_RANKS (1u << 20)   /* zero_partition (ledger and layout) */
#define ZERO_MAX_KERNEL_RANKS 64u   /* device entry points: replicas summed per element */
#define ZERO_TILE_ELEMS 8192u       /* grid of the sum-of-squares partials' tiles */

/* Partition of Psi flat parameters over N ranks.  Filled by zero_partition; pass it back
 * unchanged to the device entry points (they re-check its invariants). */
typedef struct zero_layout {
    uint64_t psi;                    /* Psi: parameters */
    uint64_t shard;                  /* S = ceil(Psi/N) rounded up to align: elements per rank */
    uint64_t psi_padded;             /* N*S: length of every flat buffer */
    uint64_t pad;                    /* N*S - Psi: trailing padding, gradient 0, output 0 */
    uint64_t bucket_elems;           /* W: window of one reduce launch in zero_step */
    uint64_t n_buckets;              /* ceil(N*S / W) */
    uint64_t tiles_per_rank;         /* ceil(S / tile_elems) + 1: a shard meets at most this
                                        many cells of the flat tile grid */
    uint64_t n_tiles;                /* N * tiles_per_rank: fp64 partial slots */
    uint64_t bytes_per_rank[4];      /* model-state bytes per rank: [0] plain DP 16*Psi,
                                        [1] 4*N*S + 12*S, [2] 2*N*S + 14*S, [3] 16*S */
    uint64_t comm_elems_per_rank[4]; /* elements each rank sends per step on a ring:
                                        2(N-1)S for [0..2], 3(N-1)S for stage 3 */
    uint32_t n_ranks;                /* N */
    uint32_t stage;                  /* 0 plain DP, 1 P_os, 2 P_os+g, 3 P_os+g+p */
    uint32_t align;                  /* S is a multiple of align */
    uint32_t tile_elems;             /* ZERO_TILE_ELEMS */
} zero_layout_t;

typedef struct zero_adamw_hparams {
    float lr;
    float beta1;            /* in [0, 1) */
    float beta2;            /* in [0, 1) */
    float eps;              /* > 0 */
    float weight_decay;     /* decoupled: p *= 1 - lr*weight_decay */
    float max_grad_norm;    /* global-norm clip threshold; <= 0 disables clipping */
    uint32_t params_dtype;  /* gathered parameters: 0 or ZERO_BF16 = bf16 (the default);
                               ZERO_F16 = fp16, the FP16 replicated parameters of
                               "【论文解读】ZeRO" sec. 4(1) */
} zero_adamw_hparams_t;

/* Scalar step state.  Lives in DEVICE memory (caller allocates sizeof(zero_step_state_t)
 * bytes, 16-byte aligned); read it with zero_step_state_read. */
typedef struct zero_step_state {
    double sumsq;           /* sum of g^2 of the last finalised step (fp64) */
    double norm;            /* its square root: the global L2 gradient norm */
    float clip_coef;        /* c applied by the last finalised step (1 when skipped) */
    float loss_scale;       /* L of the NEXT step's gradients */
    float inv_scale;        /* f32(1 / (N*L)): the reduce's unscale factor */
    float step_size;        /* lr / (1 - beta1^t) for the step being applied */
    float rbc2;             /* sqrt(1 - beta2^t) */
    float decay;            /* 1 - lr*weight_decay */
    uint32_t overflow;      /* non-finite seen by this step's reduce windows so far */
    uint32_t skip;          /* 1 if the last finalised step was skipped (overflow) */
    uint32_t t;             /* applied optimizer steps */
    uint32_t good_steps;    /* consecutive applied steps since the last scale change */
    uint32_t growth_interval;
    uint32_t dynamic;       /* 1: dynamic loss scale (halve on overflow, double every
                               growth_interval good steps, floor 1, cap 2^24) */
    uint32_t n_ranks;
    uint32_t n_steps;       /* finalised steps, applied or skipped */
    uint32_t n_skipped;
    uint32_t error;         /* device error word: 0 = none; 1 = a bounded wait gave up;
                               2 = (checked test builds only) a store outside its range */
    uint32_t arrivals;      /* internal to zero_grad_norm: its blocks that have finished
                               (0 between steps; keep it 0 when writing a state) */
    float inv_scale_used;   /* the inv_scale the last finalised step's reduce used */
    uint32_t launch_arrivals; /* internal to zero_step's single launch: its blocks that
                               have finished their reduce (0 between steps; keep it 0
                               when writing a state) */
    float applied_c;        /* the clip coefficient the last finalised step applied, -1
                               when it was skipped, 0 before the first step; the single
                               launch hands it to its blocks together with
                               launch_arrivals in one 64-bit store */
    uint64_t adamw_next_chunk; /* internal to the AdamW pass: the next chunk its blocks
                               take (0 between steps; keep it 0 when writing a state) */
    uint32_t adamw_done;    /* internal to the AdamW pass: its blocks that have finished;
                               the last one puts both words back to 0 */
    uint32_t reserved[5];
} zero_step_state_t;        /* 128 bytes */

/* -------------------------------------------------------------------------------------
 * zero_partition -- host only, no CUDA call.
 * [ZW] sec. 4(1)-(3): N equal partitions, rank r owns partition r; the ledger per stage
 * ([ZW] sec. 2(1) and 8, [ZM] sec. 3): 16*Psi, (4 + 12/N)Psi, (2 + 14/N)Psi, 16*Psi/N,
 * counted on the padded buffers; the ring traffic of [ZW] sec. 6 eq. dp-comm.
 *   psi           >= 1, <= 2^56
 *   n_ranks       1 .. ZERO_MAX_RANKS
 *   stage         0 .. 3 (0 = plain data parallelism, for the ledger only)
 *   align         S is rounded up to a multiple of align (1 .. 2^20)
 *   bucket_elems  window of one reduce launch in zero_step; 0, or any value of at least
 *                 N*S, = one window over the whole flat buffer; otherwise a multiple of 8
 *   out           written on success
 * Returns ZERO_OK or ZERO_EINVAL.
 * ------------------------------------------------------------------------------------- */
int zero_partition(uint64_t psi, uint32_t n_ranks, uint32_t stage, uint32_t align,
                   uint64_t bucket_elems, zero_layout_t* out);

/* One piece of a model tensor inside one rank's shard. */
typedef struct zero_segment {
    uint64_t tensor;         /* index in the caller's tensor list */
    uint64_t rank;           /* owner of the piece */
    uint64_t tensor_offset;  /* first element of the piece within the tensor */
    uint64_t shard_offset;   /* the same element's position in the owner's shard
                                (flat index - rank*S) */
    uint64_t count;          /* elements in the piece (>= 1) */
} zero_segment_t;            /* 40 bytes */

/* -------------------------------------------------------------------------------------
 * zero_segment_map -- host only, no CUDA call.
 * [ZW] sec. 4(2): gradients are bucketed by partition and reduced at the partition
 * boundary, so a tensor that crosses a shard boundary belongs to two or more ranks.
 * The model's tensors are laid end to end over the flat buffer [0, psi) in list order;
 * this lists each tensor's piece on each rank, in flat order (so by rank, then tensor).
 * Empty tensors have no piece; padding [psi, psi_padded) belongs to no tensor.
 *   tensor_elems   HOST array of n_tensors element counts; they must sum to layout->psi
 *   out            HOST array of `capacity` pieces, or NULL to only count them
 *   n_segments     HOST, receives the number of pieces (always, on ZERO_OK or ZERO_ENOMEM)
 * Returns ZERO_OK; ZERO_EINVAL (bad layout or pointers, sizes not summing to psi);
 * ZERO_ENOMEM when capacity is too small (out untouched).  There are
 * (non-empty tensors) + (shard boundaries strictly inside a tensor) pieces.
 * ------------------------------------------------------------------------------------- */
int zero_segment_map(const zero_layout_t* layout, const uint64_t* tensor_elems,
                     uint64_t n_tensors, zero_segment_t* out, uint64_t capacity,
                     uint64_t* n_segments);

/* Bytes of the fp64 partials workspace the device entry points need:
 * layout->n_tiles * 8.  0 for an invalid layout. */
size_t zero_workspace_bytes(const zero_layout_t* layout);

/* -------------------------------------------------------------------------------------
 * zero_step_state_init -- start a fresh optimizer (t = 0) on the device.
 *   loss_scale       initial L (> 0, finite); 1 for bf16 training
 *   dynamic          1: dynamic loss scaling (fp16 training, [ZO] "fp16": enabled);
 *                    0: static scale, overflow still skips the step
 *   growth_interval  good steps between doublings of a dynamic scale (0 = never)
 *   st               device, sizeof(zero_step_state_t)
 *   partials         device, zero_workspace_bytes(layout); zeroed here
 * Enqueues one kernel on `stream`.
 * ------------------------------------------------------------------------------------- */
int zero_step_state_init(const zero_layout_t* layout, float loss_scale, uint32_t dynamic,
                         uint32_t growth_interval, zero_step_state_t* st, double* partials,
                         zero_stream_t stream);

/* Copy the device state to host memory and wait for it (checkpoints, monitoring). */
int zero_step_state_read(const zero_step_state_t* st, zero_step_state_t* host_out,
                         zero_stream_t stream);

/* Copy a host state (e.g. from a checkpoint) to the device and wait for it.  The
 * kernels' internal counters (arrivals, launch_arrivals, adamw_next_chunk, adamw_done)
 * are written as 0 whatever host_in holds. */
int zero_step_state_write(zero_step_state_t* st, const zero_step_state_t* host_in,
                          zero_stream_t stream);

/* -------------------------------------------------------------------------------------
 * zero_reduce_shard_unscale -- the reduce-scatter arithmetic on one flat window.
 * [ZW] sec. 6(1)-(2): the ranks' gradients are averaged; with gradient partitioning the
 * average is reduce-scattered so rank r receives only flat [r*S, (r+1)*S).  [ZW] sec. 4(2):
 * gradients are bucketed and each bucket reduced as it becomes ready.
 * For every flat i in [begin, begin+count):
 *   g[i] = (sum over k = 0..N-1, ascending, in fp32, of x_k[i]) * st->inv_scale
 *   with g[i] = 0 for padding (i >= psi; replica values there are ignored);
 *   st->overflow |= any non-finite g[i];
 *   partials[tile of i] += sum of g^2 over the window's part of each tile.  Tiles cut
 *   each shard at the flat multiples of T = tile_elems (so interior tiles start on
 *   128-byte lines of every array): tile j of rank r is the intersection of
 *   [r*S, (r+1)*S) with [(c+j)*T, (c+j+1)*T), c = floor(r*S/T); slot r*tiles_per_rank + j.
 *   A rank's trailing slots may be empty (always 0).
 *   dtype      ZERO_F16 or ZERO_BF16 (the replicas' element type)
 *   replicas   HOST array of N DEVICE pointers; replicas[k] points at flat element
 *              `begin` of rank k's gradient copy and holds at least `count` elements
 *   begin      multiple of 8 (ZERO_EALIGN otherwise); begin + count <= psi_padded
 *   g          DEVICE fp32 array of psi_padded elements (indexed by the flat index)
 *   partials   DEVICE, zero_workspace_bytes(layout); zeroed by zero_step_state_init and
 *              by every zero_grad_norm, accumulated here
 *   st         DEVICE step state
 * N must be <= ZERO_MAX_KERNEL_RANKS.  Windows of one step may come in any order but
 * must not overlap; together they must cover [0, psi_padded) before zero_grad_norm.
 * ------------------------------------------------------------------------------------- */
int zero_reduce_shard_unscale(const zero_layout_t* layout, zero_dtype_t dtype,
                              const void* const* replicas, uint64_t begin, uint64_t count,
                              float* g, double* partials, zero_step_state_t* st,
                              zero_stream_t stream);

/* -------------------------------------------------------------------------------------
 * zero_grad_norm -- global norm, clip coefficient, loss scaler and skip decision.
 * [MD] sec. 1: inside optimizer.step(), before clipping, one all-reduce forms the global
 * L2 gradient norm that sets clip_coeff.  Here the all-reduce is the fixed-order sum of
 * the per-rank partial sums (each rank's tiles, then ranks in order):
 *   norm = sqrt(sumsq);  c = min(1, max_norm / (norm + 1e-6)) (fp64, rounded to fp32)
 *   overflow: skip = 1, c = 1, t unchanged, dynamic L = max(L/2, 1)
 *   else:     skip = 0, t += 1, step_size = f32(lr/(1-beta1^t)), rbc2 = f32(sqrt(1-beta2^t)),
 *             decay = f32(1 - lr*wd); dynamic L doubles after growth_interval good steps
 *   inv_scale = f32(1/(N*L)) for the next step; overflow flag and partials reset to 0.
 * One kernel (the partial sums spread over up to 128 blocks, the last block to finish
 * forms the norm); no host synchronisation.
 * ------------------------------------------------------------------------------------- */
int zero_grad_norm(const zero_layout_t* layout, const zero_adamw_hparams_t* hp,
                   double* partials, zero_step_state_t* st, zero_stream_t stream);

/* -------------------------------------------------------------------------------------
 * zero_adamw_cast_gather -- fused AdamW on every shard plus the gathered write (bf16, or
 * fp16 when hp->params_dtype == ZERO_F16).
 * [ZW] sec. 6(2): each rank updates its own parameters from its own reduced gradient and
 * the all-gather rebuilds [p0' ... p7'] in order; [ZS]: AdamW, bf16 weights.
 * Does nothing (on the device) when st->skip.  Otherwise, per flat i < psi, in fp32:
 *   gc = c*g;  m = b1*m + (1-b1)*gc;  v = b2*v + (1-b2)*(gc*gc)
 *   p  = p*decay - step_size * (m / (sqrt(v)/rbc2 + eps));  params[i] = bf16_rne(p)
 * and params[i] = 0 for padding (master/m/v there untouched).
 *   g, master, m, v   DEVICE fp32, psi_padded elements each (master/m/v updated in place)
 *   params            DEVICE bf16 (or fp16) bit patterns (uint16), psi_padded elements
 *   hp                must equal the hp given to zero_grad_norm for this step
 * ------------------------------------------------------------------------------------- */
int zero_adamw_cast_gather(const zero_layout_t* layout, const zero_adamw_hparams_t* hp,
                           const float* g, float* master, float* m, float* v, uint16_t* params,
                           const zero_step_state_t* st, zero_stream_t stream);

/* -------------------------------------------------------------------------------------
 * zero_adamw_cast_gather_host_state -- zero_adamw_cast_gather with the optimizer state
 * (master, m, v) resident in HOST memory.
 * [ZM] sec. 6: when device memory is short the optimizer state can be offloaded to the
 * CPU, at a transfer cost that has to be measured on the machine.  Here the state stays
 * in the host memory of the Grace CPU and the kernel reads and writes it in place over
 * the CPU-GPU link (NVLink-C2C on GB300) while g is read from, and the gathered
 * parameters written to, device memory; 12 B per element cross the link each way.
 * Same update, same bits as zero_adamw_cast_gather.
 *   master, m, v   HOST fp32, psi_padded elements each, PAGE-LOCKED (cudaHostAlloc /
 *                  cudaMallocHost / cudaHostRegister, e.g. torch pin_memory); updated in
 *                  place.  Pageable or device memory is refused with ZERO_EINVAL.  The
 *                  host must not touch them until the stream has passed this call.
 *   g, params, st  DEVICE, as in zero_adamw_cast_gather
 * ------------------------------------------------------------------------------------- */
int zero_adamw_cast_gather_host_state(const zero_layout_t* layout,
                                      const zero_adamw_hparams_t* hp, const float* g,
                                      float* master, float* m, float* v, uint16_t* params,
                                      const zero_step_state_t* st, zero_stream_t stream);

/* -------------------------------------------------------------------------------------
 * Rank-local entry points: the step with the ranks spread over processes (one process per
 * GPU), each process holding only its own ranks' part of g and of the optimizer state.
 * [ZW] sec. 6(2) and [ZO] stage-2 flow: each rank receives every rank's gradient for its
 * own partition (reduce-scatter), updates only its partition, and the updated parameters
 * are all-gathered; [MD] sec. 1: the global norm needs one all-reduce before clipping.
 *
 * A process holds the contiguous ranks [rank_begin, rank_begin + rank_count) (one rank per
 * process, or several); their flat range starts at origin = rank_begin*S and is
 * local_len = rank_count*S long.  Local buffers are indexed by flat index - origin.
 * origin must be a multiple of 8 (partition with align = 8; ZERO_EALIGN otherwise).
 * One step, per process, with the exchanges done by the caller (e.g. NCCL):
 *   1. exchange: every rank's gradient copy of the local range arrives (rank k's copy of
 *      flat [origin, origin + local_len)), whole or window by window (an all-to-all, or
 *      point-to-point sends of each window);
 *   2. zero_reduce_shard_unscale_local over the local range (one or more windows; the
 *      result does not depend on the windows when their boundaries lie on the flat
 *      multiples of ZERO_TILE_ELEMS);
 *   3. exchange: all-gather every process's partial slots [rank_begin*tiles_per_rank,
 *      (rank_begin + rank_count)*tiles_per_rank) into the full partials array, and
 *      combine the step state's `overflow` word over processes (maximum);
 *   4. zero_grad_norm on the full partials (every process forms the same norm, clip
 *      coefficient, scaler update and skip decision, bit for bit);
 *   5. zero_adamw_cast_gather_local on the local range;
 *   6. exchange: all-gather the local parameters into the full gathered buffer.
 * With the ranks' sums taken in ascending rank order in step 2 and the fixed-order sum of
 * step 4, every output equals the one-GPU step's (zero_step) bit for bit.
 * ------------------------------------------------------------------------------------- */

/* zero_reduce_shard_unscale on a window inside the local range, g stored locally.
 *   replicas   HOST array of N DEVICE pointers; replicas[k] points at flat element `begin`
 *              of rank k's gradient copy (e.g. inside the chunk received from rank k)
 *   begin      multiple of 8; [begin, begin + count) inside [origin, origin + local_len)
 *   g_local    DEVICE fp32, local_len elements: g of flat i is stored at g_local[i - origin]
 *   partials   DEVICE, zero_workspace_bytes(layout) (all ranks' slots); the local ranks'
 *              slots are accumulated as in zero_reduce_shard_unscale
 *   st         DEVICE step state of this process (its overflow word is set as there)
 * ZERO_EINVAL for a bad rank range or a window outside it. */
int zero_reduce_shard_unscale_local(const zero_layout_t* layout, zero_dtype_t dtype,
                                    uint32_t rank_begin, uint32_t rank_count,
                                    const void* const* replicas, uint64_t begin, uint64_t count,
                                    float* g_local, double* partials, zero_step_state_t* st,
                                    zero_stream_t stream);

/* zero_adamw_cast_gather on the local range only: element j of every local array is flat
 * origin + j; elements at flat >= psi are padding (parameters written 0, state untouched).
 *   g_local, master_local, m_local, v_local   DEVICE fp32, local_len elements each
 *   params_local   DEVICE 16-bit, local_len elements: this process's part of the gathered
 *                  buffer (it may point at flat `origin` of the full buffer, so that an
 *                  in-place all-gather completes it)
 *   st             DEVICE step state after zero_grad_norm of this step */
int zero_adamw_cast_gather_local(const zero_layout_t* layout, const zero_adamw_hparams_t* hp,
                                 uint32_t rank_begin, uint32_t rank_count, const float* g_local,
                                 float* master_local, float* m_local, float* v_local,
                                 uint16_t* params_local, const zero_step_state_t* st,
                                 zero_stream_t stream);

/* -------------------------------------------------------------------------------------
 * zero_step -- one whole step: every bucket's reduce, the norm, AdamW + cast.
 *   replicas   HOST array of n_buckets * N DEVICE pointers, bucket-major:
 *              replicas[b*N + k] holds rank k's gradient for flat
 *              [b*W, min((b+1)*W, psi_padded)).  With n_buckets = 1 these are simply
 *              the N full gradient copies.
 *   g          as in zero_reduce_shard_unscale, or NULL when N = 2 and n_buckets = 1:
 *              the re-reading schedule.  Clipping needs the global norm before any
 *              update, so an exact step either writes the fp32 g and reads it back
 *              (34 + 2N bytes per parameter) or reads the N copies twice (26 + 4N); at
 *              N = 2 the second moves 34 instead of 38 B.  The reduce then stores no g
 *              and AdamW forms each g[i] again from the two copies with the same
 *              arithmetic (same bits).  ZERO_EINVAL for NULL g with any other layout.
 *   other arguments as in the three calls above.
 * Launches: n_buckets + 2 kernels (the reduce per bucket, the norm, AdamW).  A small
 * layout (one bucket, at most 128 tile slots per rank, and every one of its n_tiles tiles
 * able to hold a resident block at once: up to a few million parameters) runs instead
 * as ONE cooperative kernel with the same bits: each block reduces one tile and keeps
 * its g in shared memory (with at most one tile per SM, also the tile's master, m and v,
 * bulk-copied in as the block starts), the block that finishes last forms the global norm
 * and the step's scalars, and every block then updates its tile.  g is still written when given
 * (never read back), so such a step moves 2N + 30 bytes per parameter, 2N + 26 with
 * g = NULL (+2 with at most one tile per SM: the gathered parameters are read too, so
 * that an update made ahead of the norm can be undone).  zero_step_launches tells which way a layout goes.  If the cooperative launch
 * is refused because fewer blocks fit on the GPU than its occupancy promised (another
 * context holds part of it), the same call makes the three launches instead.
 * ------------------------------------------------------------------------------------- */
int zero_step(const zero_layout_t* layout, const zero_adamw_hparams_t* hp, zero_dtype_t dtype,
              const void* const* replicas, float* g, double* partials, float* master, float* m,
              float* v, uint16_t* params, zero_step_state_t* st, zero_stream_t stream);

/* Kernel launches one zero_step call makes for this layout and gradient type on the
 * current device: 1 (the single-launch step) or n_buckets + 2.  ZERO_EINVAL (negative) for
 * an invalid layout or dtype.  Enqueues nothing; the first call on a device queries the
 * kernel's occupancy there. */
int zero_step_launches(const zero_layout_t* layout, zero_dtype_t dtype);

/* -------------------------------------------------------------------------------------
 * zero_step_host -- zero_step with the gradients in HOST memory.
 * The N gradient copies arrive from pinned host memory, one bucket of W elements at a
 * time, through a two-slot device staging ring: the copy of bucket b+1 (on copy_stream,
 * one cudaMemcpyAsync per rank) overlaps the reduce of bucket b (on stream).
 *   host_replicas   HOST array of N HOST pointers (pinned for overlap), each psi_padded
 *                   elements of dtype; read asynchronously, so they must stay unchanged
 *                   until the step has completed on `stream`
 *   staging         DEVICE buffer of staging_bytes >= 2 * N * W8 * sizeof(dtype), W8 = W
 *                   rounded up to a multiple of 8 (so every staged copy is 16-byte
 *                   aligned; W itself is a multiple of 8 whenever there are several
 *                   buckets); not touched when the copies are read in place
 *   host_state_out  optional HOST pointer (pinned): the step state is copied there at
 *                   the end of the step on `stream` (the caller synchronises)
 *   copy_stream     must differ from stream
 * A small layout in one bucket (one that zero_step runs as a single launch) runs as that
 * single launch here too.  When every copy lies in page-locked host memory (through its
 * whole psi_padded range, 16-byte aligned), the launch reads the copies there directly
 * over the CPU-GPU link, and staging is not touched; otherwise the copies are staged
 * first.
 * Returns ZERO_ENOMEM if staging is too small.
 * ------------------------------------------------------------------------------------- */
int zero_step_host(const zero_layout_t* layout, const zero_adamw_hparams_t* hp,
                   zero_dtype_t dtype, const void* const* host_replicas, void* staging,
                   uint64_t staging_bytes, float* g, double* partials, float* master, float* m,
                   float* v, uint16_t* params, zero_step_state_t* st,
                   zero_step_state_t* host_state_out, zero_stream_t stream,
                   zero_stream_t copy_stream);

/* -------------------------------------------------------------------------------------
 * zero_step_static_workspace -- zero_step for callers that cannot allocate device memory.
 * The ZeRO pages have no counterpart of this call; it exists for how the library is used.
 * Some callers cannot give the library a scratch buffer: their memory manager already
 * holds all of the GPU's memory, or they must not take the device-wide synchronisation
 * that a cudaMalloc or cudaFree can cause in the middle of a training step.  This call
 * runs the same step as zero_step, but keeps the step's only scratch, the per-tile
 * sum-of-squares partials, in a static device array of ZERO_STATIC_WORKSPACE_SLOTS
 * 8-byte slots (8 MiB) inside the library.  It calls no cudaMalloc, no cudaFree and no
 * other allocating routine.
 *   - The array is held on every GPU where the library's device code is loaded, from
 *     load until the process exits.
 *   - Layouts with n_tiles > ZERO_STATIC_WORKSPACE_SLOTS (more than about 8.6e9 padded
 *     parameters) are rejected with ZERO_ENOMEM before anything is enqueued.
 *   - The first call on each device looks up the array's device address (a one-time
 *     set-up, with that device current); make that first call before any stream capture
 *     begins.
 *   - Every call shares the one array and clears the slots it uses at its start, so two
 *     calls whose work overlaps on the GPU (different streams or threads) race: issue them
 *     one after another on one stream.
 *   - Arguments as in zero_step, without `partials`, except that g must not be NULL:
 *     this call has no re-reading schedule (ZERO_EINVAL for NULL g).  To initialise st
 *     with zero_step_state_init without allocating, pass any 16-byte-aligned device buffer
 *     of at least zero_workspace_bytes(layout) bytes as its `partials` argument, e.g. `g`
 *     whenever 4*psi_padded >= zero_workspace_bytes(layout), which holds for every shard
 *     size S >= 4 (every step overwrites g before reading it).
 *   - The address lookup is cached per device for the life of the process; after a
 *     cudaDeviceReset the library's device code may be loaded at another address, so do
 *     not call this entry point again in that process.
 * ------------------------------------------------------------------------------------- */
#define ZERO_STATIC_WORKSPACE_SLOTS (1u << 20)
int zero_step_static_workspace(const zero_layout_t* layout, const zero_adamw_hparams_t* hp,
                               zero_dtype_t dtype, const void* const* replicas, float* g,
                               float* master, float* m, float* v, uint16_t* params,
                               zero_step_state_t* st, zero_stream_t stream);

/* -------------------------------------------------------------------------------------
 * Lists of tensors: the norm and the AdamW step on a model's tensors where they lie, with
 * no flat copy, each with its own learning-rate scale and weight decay, and with optimizer
 * states of 32 or of 8 bits.  [ZS]: the AdamW ledger and update; [MD] sec. 1: the global
 * norm before clipping; [ZW] sec. 4(2): a rank's shard as pieces of tensors (the pieces
 * zero_segment_map lists are such a list).
 *
 * One step, on one stream:
 *   1. zero_tensors_grad_norm  over the list (scalars into the step state)
 *   2. zero_tensors_adamw or zero_tensors_adamw8 over the same list
 * A step state serves one stream at a time: AdamW hands out a long list's work through the
 * state's internal counters (adamw_next_chunk, adamw_done), although it takes it as const.
 * Two lists under one state on two streams would each skip part of their elements; give
 * each a copy of the state (its 128 bytes, taken after the norm).
 * The norm and the overflow check are those of the list given.  A rank whose list is its own
 * shard gets its shard's norm: clipping by the norm over all ranks takes the step state of
 * zero_grad_norm over the partials that the ranks have exchanged.
 * The list is a HOST array that each call reads before it returns; its pointers are DEVICE
 * pointers.  Every array is contiguous and holds `elems` elements at the natural alignment
 * of its element type (ZERO_EALIGN otherwise); tensors whose fp32 arrays are 32-byte, 16-bit
 * arrays 16-byte and code arrays 8-byte aligned move in one access per 8 elements, others
 * element by element.  A tensor may be empty (its pointers are then not
 * looked at), and so may the list.  No two arrays may overlap.  One launch covers several
 * hundred tensors; a longer list takes more than one.
 *
 * 8-bit states.  A tensor's elements are cut into blocks of 256 (the last may be shorter);
 * m and v hold one code byte per element, exps two bytes per block (m's, then v's exponent
 * b).  b = 0 stands for a block of zeros; else the block's largest magnitude lies at or
 * below 1.875 * 2^(b-127), b in [27, 253].  A code is a small float scaled by 2^(b-127):
 *   m   sign, 4 exponent bits E, 3 mantissa bits M:  (1 + M/8) * 2^(E-15), or M/8 * 2^-14
 *       for E = 0
 *   v   5 exponent bits E, 3 mantissa bits M:        (1 + M/8) * 2^(E-31), or M/8 * 2^-30
 *       for E = 0
 * Arrays of zeros are the states of a fresh optimizer.  zero_tensors_adamw8 rounds each
 * new value up or down at random so that its mean is the value itself: with beta2 = 0.999
 * a step moves v by about 0.1%, far less than the codes' spacing of 6-12%, and rounding to
 * nearest would leave v where it was.  A v > 0 is never stored as 0 (the update would
 * divide by eps alone).  Magnitudes above 1.875 * 2^126, and NaN, are stored as the
 * largest code.  The random bits are a function of `seed`, of the step state's t and of the
 * element's place in the list, so a step repeats bit for bit:
 *   mix(x):  x ^= x>>16; x *= 0x6A09E667; x ^= x>>15; x *= 0xBB67AE85; x ^= x>>16   (mod 2^32)
 *   K = mix(mix(lo32(seed) + t * 0x9E3779B9) ^ hi32(seed))
 *   G = 32 * (blocks of the list before the element's) + (element's index in its block) / 8
 *   s_0 = mix(K + G * 0x9E3779B9);  s_j = 1664525 * s_(j-1) + 1013904223;  q = index mod 8
 *   m's 20 random bits: s_(q+1) >> 12;  v's: s_(q+9) >> 12
 * ------------------------------------------------------------------------------------- */
#define ZERO_STATE8_BLOCK 256u /* elements that share an exponent byte */

typedef struct zero_tensor {
    uint64_t elems;          /* at most 2^39 */
    const void* grad;        /* of grad_dtype */
    float* master;           /* fp32 parameters, updated in place */
    void* m;                 /* optimizer state of state_dtype, updated in place */
    void* v;
    uint8_t* exps;           /* ZERO_U8 states: 2 * ceil(elems/256) exponent bytes */
    uint16_t* params;        /* 16-bit parameters out, or NULL (fp32 training: master is it) */
    uint32_t grad_dtype;     /* ZERO_F16, ZERO_BF16 or ZERO_F32 */
    uint32_t state_dtype;    /* ZERO_F32 or ZERO_U8 (a target of zero_tensors_state8_read may
                                also be ZERO_BF16) */
    uint32_t params_dtype;   /* ZERO_BF16, ZERO_F16, or 0: the hyperparameters' */
    float lr_scale;          /* this tensor's learning rate is lr * lr_scale (>= 0) */
    float weight_decay;      /* this tensor's decoupled decay, in place of the hyperparameters' */
    uint32_t reserved;       /* 0 */
} zero_tensor_t;             /* 80 bytes */

/* Bytes of the workspace zero_tensors_grad_norm needs for a list of n_tensors. */
size_t zero_tensors_workspace_bytes(uint64_t n_tensors);

/* zero_step_state_init for a list of tensors (no layout, no partials).
 *   n_ranks   the gradients are sums of this many copies (1: already averaged):
 *             inv_scale = f32(1 / (n_ranks * L)) */
int zero_tensors_state_init(uint32_t n_ranks, float loss_scale, uint32_t dynamic,
                            uint32_t growth_interval, zero_step_state_t* st, zero_stream_t stream);

/* zero_grad_norm over a list: with g = x * st->inv_scale for every gradient element x,
 *   norm = sqrt(sum of g^2);  overflow when any g is not finite
 * and everything zero_grad_norm writes: clip coefficient, skip decision, t, the scaler and
 * the bias corrections.  Reads elems, grad and grad_dtype of each tensor.
 *   workspace   DEVICE, zero_tensors_workspace_bytes(n_tensors), 16-byte aligned; needs no
 *               initialisation
 * The sums are formed in a fixed order: the same list gives the same bits. */
int zero_tensors_grad_norm(const zero_tensor_t* tensors, uint64_t n_tensors,
                           const zero_adamw_hparams_t* hp, double* workspace,
                           zero_step_state_t* st, zero_stream_t stream);

/* AdamW over a list with fp32 states, and the cast into the 16-bit parameters.  Does
 * nothing (on the device) when st->skip.  For every element, in fp32:
 *   gc = c * (x * st->inv_scale_used);  m = b1*m + (1-b1)*gc;  v = b2*v + (1-b2)*(gc*gc)
 *   p  = p*decay - step*(m / (sqrt(v)/rbc2 + eps));  params = rounded to nearest even
 * with step = st->step_size * lr_scale and decay = f32(1 - lr * lr_scale * weight_decay).
 * With lr_scale 1 and the hyperparameters' weight decay, zero_adamw_cast_gather's bits for
 * the same gradient and step state.
 *   hp   must equal the hp given to zero_tensors_grad_norm for this step */
int zero_tensors_adamw(const zero_tensor_t* tensors, uint64_t n_tensors,
                       const zero_adamw_hparams_t* hp, const zero_step_state_t* st,
                       zero_stream_t stream);

/* The same with 8-bit states: m and v are decoded, updated in fp32, used in fp32 for the
 * parameters (with sqrt(v) * (1/rbc2) in the denominator; the square root and the quotient
 * are within 2 ulp), and stored in 8 bits again.
 * master and params stay as in zero_tensors_adamw.
 *   seed   of the rounding; any value, the same for a whole run */
int zero_tensors_adamw8(const zero_tensor_t* tensors, uint64_t n_tensors,
                        const zero_adamw_hparams_t* hp, uint64_t seed,
                        const zero_step_state_t* st, zero_stream_t stream);

/* The 8-bit states' values: for every tensor k, `to[k].m` and `to[k].v` (fp32 or bf16; both
 * hold the values exactly) from the codes of `from[k]`.  Reads elems, m, v, exps and
 * state_dtype; to[k].elems must equal from[k].elems. */
int zero_tensors_state8_read(const zero_tensor_t* from, const zero_tensor_t* to,
                             uint64_t n_tensors, zero_stream_t stream);

/* fp32 states into 8 bits, each to the nearest code (half away from zero): `to[k]`'s codes
 * and exponents from `from[k].m` and `from[k].v`; v must not be negative.  Writing what
 * zero_tensors_state8_read gave keeps every value. */
int zero_tensors_state8_write(const zero_tensor_t* to, const zero_tensor_t* from,
                              uint64_t n_tensors, zero_stream_t stream);

/* -------------------------------------------------------------------------------------
 * Beside a model's matrix products: layer norm, token embedding and the softmax cross entropy
 * of a large vocabulary, forward and backward.  These are where the gradients of a model's
 * vectors and of its embedding and head come from; zero_tensors_grad_norm and
 * zero_tensors_adamw read them where they are written, and the loss's gradient takes the
 * step state's loss scale on the device.  [ZW] sec. 2(1): the gradients and the activations
 * of a training step; [ZO] stage-2 flow: forward, backward, then the step.
 *
 * Rows of activations (x, y, dy, dx, out, dout, hidden, dhidden) are `dim` elements each, the
 * next row `*_stride` elements further (at least dim, at most 2^32; any value for a single
 * row).  Weights, tables and their gradients are contiguous.  Every pointer has the natural
 * alignment of its element type (ZERO_EALIGN otherwise) unless said otherwise; rows on 16-byte
 * boundaries with dim % 8 == 0 move in 128-bit accesses, others element by element.
 * dtype: ZERO_F16, ZERO_BF16 or (not the head) ZERO_F32.  Sums, statistics and all
 * arithmetic are fp32; 16-bit outputs are rounded once, to nearest even.
 * grad_dtype, of weights' gradients: dtype or ZERO_F32.  accumulate = 1 adds to what they hold
 * (an earlier micro-batch; the other end of a tied embedding), 0 overwrites all of them.
 * Outputs must not overlap inputs or each other (ZERO_EINVAL).  A workspace needs no
 * initialisation, keeps nothing from one call for the next, and serves one call at a time:
 * calls (or captured graphs) that share one run one after another.
 * No call adds in an order that varies: the same call gives the same bits.
 * ------------------------------------------------------------------------------------- */

/* Layer norm.  Per row: mean = sum(x)/dim, rstd = 1/sqrt(sum((x - mean)^2)/dim + eps),
 * y = (x - mean) * rstd * weight + bias.
 *   rows          at most 2^30
 *   dim           1 .. 16384
 *   weight, bias  param_dtype (dtype or ZERO_F32); bias may be NULL (0)
 *   eps           >= 0
 *   mean, rstd    fp32 per row, for the backward pass; each may be NULL */
int zero_layernorm(zero_dtype_t dtype, uint64_t rows, uint32_t dim, const void* x, uint64_t x_stride,
                   const void* weight, const void* bias, zero_dtype_t param_dtype, float eps, void* y,
                   uint64_t y_stride, float* mean, float* rstd, zero_stream_t stream);

/* Bytes of zero_layernorm_backward's workspace; 0 for sizes that it refuses. */
size_t zero_layernorm_workspace_bytes(uint64_t rows, uint32_t dim);

/* Its gradients.  With xh = (x - mean) * rstd and g = dy * weight:
 *   dx = rstd * (g - sum(g)/dim - xh * sum(g * xh)/dim)
 *   dweight (+)= sum over rows of dy * xh;  dbias (+)= sum over rows of dy
 *   mean, rstd      as zero_layernorm wrote them
 *   dweight, dbias  grad_dtype, dim elements; each may be NULL (not wanted)
 *   workspace       DEVICE, zero_layernorm_workspace_bytes(rows, dim), 16-byte aligned
 * Without rows dweight and dbias are 0 (or left as they are, accumulate).  Should a bounded wait
 * inside give up, dweight, dbias and the rows of dx left undone are NaN; of zero_layernorm, the rows of
 * y left undone with their mean and rstd. */
int zero_layernorm_backward(zero_dtype_t dtype, uint64_t rows, uint32_t dim, const void* x, uint64_t x_stride,
                            const void* weight, zero_dtype_t param_dtype, const float* mean, const float* rstd,
                            const void* dy, uint64_t dy_stride, void* dx, uint64_t dx_stride, void* dweight,
                            void* dbias, zero_dtype_t grad_dtype, uint32_t accumulate, void* workspace,
                            zero_stream_t stream);

/* Embedding: out[t] = scale * table[tokens[t]]; a row of zeros where the id lies outside
 * [0, vocab) (padding).
 *   n_tokens     at most 2^28
 *   dim          1 .. 65536;  vocab  1 .. 2^30
 *   tokens       int32 or int64 ids (token_bytes 4 or 8), contiguous
 *   table        dtype, [vocab][dim] */
int zero_embedding(zero_dtype_t dtype, uint64_t n_tokens, uint32_t dim, uint32_t vocab, const void* tokens,
                   uint32_t token_bytes, const void* table, float scale, void* out, uint64_t out_stride,
                   zero_stream_t stream);

/* Bytes of zero_embedding_backward's workspace; 0 for sizes that it refuses. */
size_t zero_embedding_workspace_bytes(uint64_t n_tokens, uint32_t dim, uint32_t vocab);

/* Its gradient: dtable[v] (+)= scale * (sum over the places t with tokens[t] = v of dout[t]),
 * in an order that the tokens alone give.  Ids outside [0, vocab) have none.  With accumulate the rows of
 * tokens that do not occur are not touched; without, they are written 0.
 *   dtable      grad_dtype, [vocab][dim]
 *   workspace   DEVICE, zero_embedding_workspace_bytes(...), 16-byte aligned */
int zero_embedding_backward(zero_dtype_t dtype, uint64_t n_tokens, uint32_t dim, uint32_t vocab, const void* tokens,
                            uint32_t token_bytes, const void* dout, uint64_t dout_stride, float scale, void* dtable,
                            zero_dtype_t grad_dtype, uint32_t accumulate, void* workspace, zero_stream_t stream);

/* Bytes of the head's workspace, forward or backward; 0 for sizes that they refuse. */
size_t zero_head_workspace_bytes(uint64_t rows, uint32_t dim, uint32_t vocab);

/* Softmax cross entropy of the logits l[t][v] = sum over k of hidden[t][k] * weight[v][k], which
 * are never kept:
 *   lse[t] = log(sum over v of exp(l[t][v]));  loss[t] = lse[t] - l[t][targets[t]]
 * A token whose target lies outside [0, vocab) (e.g. -100) has none: loss = lse = 0, whatever its
 * hidden row holds.
 *   dtype      ZERO_BF16 or ZERO_F16
 *   rows       at most 2^24;  dim  1 .. 65536;  vocab  1 .. 2^24
 *   weight     dtype, [vocab][dim]; 16-byte aligned when dim % 8 == 0
 *   targets    int32 or int64 (target_bytes 4 or 8), contiguous
 *   loss, lse  fp32 per token
 *   workspace  DEVICE, zero_head_workspace_bytes(...), 256-byte aligned
 * Should a bounded wait inside give up, the workspace's second 32-bit word is 1 and the losses
 * are NaN. */
int zero_head_loss(zero_dtype_t dtype, uint64_t rows, uint32_t dim, uint32_t vocab, const void* hidden,
                   uint64_t hidden_stride, const void* weight, const void* targets, uint32_t target_bytes, float* loss,
                   float* lse, void* workspace, zero_stream_t stream);

/* Its gradients.  With f[t] = scale * row_scale[t] * st->loss_scale:
 *   D[t][v]   = f[t] * (exp(l[t][v] - lse[t]) - (v == targets[t]))
 *   dhidden   = D . weight  (0 for tokens without a target);  dweight (+)= D^T . hidden
 * D is formed a piece of the vocabulary at a time, in units of the largest finite |f| (fp16: of 2^-14
 * of it), and rounded to dtype before the two products; also for an fp32 dweight, whose rows are
 * thus good to dtype's digits.  fp16: tokens whose |f| is less than 2^-14 of the largest lose
 * digits.
 *   lse         as zero_head_loss wrote it
 *   scale       e.g. 1 / tokens, for the gradient of a mean
 *   row_scale   fp32 per token (what arrives at loss[t]), or NULL: 1
 *   st          the step state whose loss_scale the gradients get, or NULL: 1.  A bounded wait
 *               that gives up puts 1 into its error word (and the workspace's second word);
 *               dhidden is NaN then, and so is what was not formed of dweight
 *   dhidden     dtype, or NULL (not wanted);  dweight  grad_dtype, or NULL (not wanted) */
int zero_head_loss_backward(zero_dtype_t dtype, uint64_t rows, uint32_t dim, uint32_t vocab, const void* hidden,
                            uint64_t hidden_stride, const void* weight, const void* targets, uint32_t target_bytes,
                            const float* lse, float scale, const float* row_scale, zero_step_state_t* st,
                            void* dhidden, uint64_t dhidden_stride, void* dweight, zero_dtype_t grad_dtype,
                            uint32_t accumulate, void* workspace, zero_stream_t stream);

/* Text for a status code. */
const char* zero_strerror(int status);

/* cudaError_t of the last ZERO_ECUDA returned on this thread (0 if none). */
int zero_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_H */
