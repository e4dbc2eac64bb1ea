/*
 * ag.h -- C ABI of libag: a symmetric heap of logical ranks on one MI355X
 * (gfx950), a persistent tiled multi-destination all-gather, a tiled GEMM
 * whose epilogue performs the same multi-destination store, and what a rank
 * works with between collectives: a linear layer with its epilogue, its
 * gradients, the root-mean-square norm, rows in 8 bits with the products and
 * gradients that read them, and an AdamW step over many tensors.
 *
 * Sources (the three pages on the iris all-gather):
 *  - ROCm/iris #626, "Summary": the device-side all-gather loads the local
 *    and every peer heap base once, before the first store, keeps each peer
 *    as a pointer delta (peer_base - local_base), stores the local copy
 *    first and then the peers in rotated order (rank+1, rank+2, ...).
 *  - ROCm/iris #626, "Triton CCL all-gather": the persistent kernel walks
 *    tiles with a grid stride and translates the output base once per peer
 *    before the tile loop.
 *  - ROCm/iris #626, "Assembly" table: the fused matmul + all-gather kernel
 *    stores its 256x256 fp16 C tile to every rank, with the heap-base loads
 *    hoisted above the K loop.
 *  - ROCm/iris #594, "Multi-GPU CI" / "Local validation": the result is that
 *    of torch.distributed.all_gather_into_tensor; logical ranks may be
 *    independent regions of memory on one GPU.
 *  - ROCm/iris #591, "Hoist the peer heap bases": groups are described by
 *    (rank_start, rank_stride, world_size); heap_bases is a device array of
 *    every rank's heap base.
 *
 * Conventions shared by every entry point
 *  - All pointers named dev_* or passed as input/A/B are device addresses in
 *    the current HIP device's memory; host pointers are named out/plan/etc.
 *  - Every entry point returns ag_status_t.  On any status other than AG_OK
 *    nothing was launched and no output argument was written, and
 *    ag_last_error_message() gives a one-line reason (thread-local).
 *  - Launching entry points are asynchronous and ordered on the given
 *    hipStream_t (NULL = the null stream).  They never synchronise.  A launch
 *    failure reported by the runtime returns AG_ERR_HIP.  They launch on the
 *    current HIP device, which must be the device the heap was created or
 *    wrapped on (AG_ERR_INVALID_ARG otherwise).
 *  - Argument validation is done on the host before any HIP call; values are
 *    never remapped: 0 means "documented default", anything else is used as
 *    given or rejected.
 */
#ifndef AG_H
#define AG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ag_status {
    AG_OK = 0,
    AG_ERR_INVALID_ARG = 1,   /* an argument is out of range, misaligned, null or overlapping */
    AG_ERR_UNSUPPORTED = 2,   /* valid request this library does not implement (e.g. W > 8) */
    AG_ERR_OUT_OF_MEMORY = 3, /* device allocation failed or the symmetric heap is exhausted */
    AG_ERR_HIP = 4            /* a HIP runtime call failed (no device, launch error, ...) */
} ag_status_t;

typedef enum ag_dtype {
    AG_F16 = 0,   /* IEEE binary16, 2 bytes */
    AG_BF16 = 1,  /* bfloat16, 2 bytes */
    AG_F32 = 2    /* IEEE binary32, 4 bytes (the copies only, not the GEMM) */
} ag_dtype_t;

/* Largest group the kernels are instantiated for (destination loop is a static unroll). */
#define AG_MAX_WORLD 8
/* Alignment (and unit) of every region stride created by ag_heap_create. */
#define AG_REGION_ALIGN ((size_t)2 << 20)

typedef struct ag_heap ag_heap_t;  /* opaque */

/* Where a heap lives; filled by ag_heap_geometry, or by hand for planning only. */
typedef struct ag_heap_geometry {
    uint64_t slab_addr;       /* device address of region 0 (region r = slab_addr + r*bytes_per_rank) */
    uint64_t bytes_per_rank;  /* region stride in bytes, a multiple of 256 */
    int32_t n_ranks;          /* number of regions, >= 1 */
    int32_t rank;             /* calling rank of a view, or -1 for the root handle */
    int32_t num_cus;          /* compute units of the heap's device (default n_programs) */
    int32_t reserved;         /* must be 0 */
} ag_heap_geometry_t;

/* What a call will launch: filled by the ag_plan_* functions (pure host logic). */
typedef struct ag_plan {
    int32_t group_rank;          /* g = (rank - rank_start) / rank_stride */
    int32_t vec_bytes;           /* bytes per vector access of the copy kernel (16/8/4/2) */
    int32_t tile_m, tile_n, tile_k; /* effective tile (tile_k = 0 for the all-gather) */
    int32_t n_programs;          /* persistent workgroups launched */
    int32_t threads;             /* threads per workgroup */
    int32_t lds_bytes;           /* LDS per workgroup */
    int32_t vectors_per_thread;  /* copy kernel: vector accesses per thread per tile */
    int32_t variant;             /* library-internal kernel variant (informational) */
    int64_t tiles_m, tiles_n, total_tiles;
    uint64_t rank_block_offset;  /* byte offset of this rank's rows inside every region (out_offset + g*M_local*N*e) */
    uint64_t bytes_read;         /* algorithmic bytes read per call */
    uint64_t bytes_written;      /* algorithmic bytes written per call (W destinations) */
    double flops;                /* 2*M_local*N*K for the GEMM, 0 for the all-gather */
    int32_t dest_group;          /* copy kernels: destinations stored per wait (0 = all of them, no wait) */
    int32_t schedule;            /* copy kernels: ag_schedule_t of the launch */
    int32_t tile_order;          /* copy kernels: ag_tile_order_t applied (AG_ORDER_STRIDE or AG_ORDER_TICKETS) */
    int32_t tiles_per_ticket;    /* copy kernels with AG_ORDER_TICKETS: consecutive tiles per ticket (else 0) */
    int32_t ticket_wait;         /* AG_ORDER_TICKETS on wide launches: 1 when each program takes its next
                                    ticket after the stores of the batch in hand (its first wave waits for
                                    its own stores to complete, and the barrier that hands the ticket out
                                    holds the other waves until then), 0 when it takes it before them */
    int32_t reserved_plan;       /* 0 */
} ag_plan_t;

/* Tile schedules of the all-gather (ag_all_gather_ex) and the all-to-all (ag_all_to_all_ex). */
typedef enum ag_schedule {
    AG_SCHEDULE_TILES = 0,       /* each program walks tiles and stores every tile to all W destinations
                                    (the all-to-all: each chunk tile to its one destination) */
    AG_SCHEDULE_PARTITIONED = 1  /* each program owns one destination and walks the tiles for it alone */
} ag_schedule_t;

/* Order in which the persistent programs of AG_SCHEDULE_TILES take their tiles (the all-to-all's
 * tiles: the W chunk copies as one sequence, destination by destination).  The result does not
 * depend on it. */
typedef enum ag_tile_order {
    AG_ORDER_AUTO = 0,     /* the library's choice: AG_ORDER_TICKETS where a ticket kernel exists and,
                              for the all-gather, the call has at least 64 tiles per program; for the
                              all-to-all, at least 64 tiles per program and vector per thread with
                              programs x vectors per thread below twice the CU count.
                              AG_ORDER_STRIDE otherwise */
    AG_ORDER_STRIDE = 1,   /* fixed grid stride: program p takes tiles p, p + P, p + 2P, ... */
    AG_ORDER_TICKETS = 2   /* programs take G consecutive tiles at a time from a device counter of the
                              calling rank, in increasing tile order; 16-byte vectors, one or two per
                              thread and tile, no destination groups, every tile row of the block below
                              2 GiB.  G is one of 3, 4, 8, 16 (one vector per thread) or 2, 4, 8 (two):
                              the smallest whose tiles move at least 96 KiB of HBM traffic (the
                              all-gather's read once and written W times, the all-to-all's read and
                              written once; the largest where none does), and on launches with fewer
                              programs than CUs at least the largest of 16, 8 and 4 (within those
                              sizes) with G x programs <= 1024.  When programs x vectors per thread
                              reach three quarters of the CU count, each program takes its next ticket
                              after the stores of the batch in hand (plan.ticket_wait) */
} ag_tile_order_t;

/* Options of ag_all_gather_ex and ag_all_to_all_ex; all-zero (or a NULL pointer) is the plain call. */
typedef struct ag_copy_options {
    int32_t dest_group;   /* 0: one straight run of W destination stores per tile (default).
                             1, 2 or 4 (< W): store that many destinations, then wait until the
                             stores before them have completed, then the next group */
    int32_t schedule;     /* ag_schedule_t */
    int32_t tile_order;   /* ag_tile_order_t (AG_SCHEDULE_TILES only; else 0) */
    int32_t reserved[5];  /* must be 0 */
} ag_copy_options_t;

/* ------------------------------------------------------------------------
 * Symmetric heap (ROCm/iris #626 "Summary" and #591: one heap per rank,
 * tensors at the same offset in every heap, kernels read the device array
 * heap_bases).  Here the n_ranks heaps are disjoint regions of one device
 * allocation (ROCm/iris #594 "Local validation": logical ranks as separate
 * memory on one GPU), and heap_bases[r] = slab + r*bytes_per_rank lives in
 * a separate device array of n_ranks uint64_t.
 * ------------------------------------------------------------------------ */

/* The region stride ag_heap_create uses for bytes_per_rank (ROCm/iris #594
 * "Local validation": logical ranks as separate memory of one GPU; how the
 * regions sit in HBM is this library's choice).  bytes_per_rank rounded up
 * to AG_REGION_ALIGN, plus one AG_REGION_ALIGN when the result is a power of
 * two of 512 MiB or more: the W copies of a tile are stored at the same
 * offset of W regions at once, and strides of a large power of two alias
 * them in the HBM channel interleave (W=8, 16384x8192 fp16 per rank: 349-354
 * against 354-360 us per call).  Callers of ag_heap_wrap can lay out their
 * slab the same way.  Host-only.  AG_ERR_INVALID_ARG when region_bytes is
 * NULL or bytes_per_rank is 0 or above 1 TiB. */
ag_status_t ag_heap_region_bytes(size_t bytes_per_rank, size_t* region_bytes);

/* Allocate a slab of n_ranks regions of bytes_per_rank bytes (the region
 * stride is ag_heap_region_bytes(bytes_per_rank)) plus the device base
 * table, on the current device.  The
 * heap owns both.  n_ranks in [1, 1024], bytes_per_rank >= 1.  Contents of
 * the slab are undefined.  AG_ERR_OUT_OF_MEMORY if hipMalloc fails,
 * AG_ERR_HIP if no device is usable. */
ag_status_t ag_heap_create(int n_ranks, size_t bytes_per_rank, ag_heap_t** out);

/* Build a heap over caller-owned device memory of n_ranks*bytes_per_rank
 * bytes (e.g. a torch uint8 tensor).  dev_slab must be 256-byte aligned and
 * bytes_per_rank a non-zero multiple of 256.  dev_slab must be device (or
 * managed) memory of the current device, and its allocation must hold the
 * n_ranks*bytes_per_rank bytes from dev_slab on (AG_ERR_INVALID_ARG
 * otherwise: checked with hipPointerGetAttributes and, where the runtime
 * reports the allocation's extent, hipMemGetAddressRange).
 * The library allocates and owns only the base table; the caller keeps the
 * slab alive until every handle on it is destroyed. */
ag_status_t ag_heap_wrap(void* dev_slab, int n_ranks, size_t bytes_per_rank, ag_heap_t** out);

/* A handle for one calling rank ("the caller's rank", as the context object
 * of iris knows its rank).  Views share the slab, the table and the
 * allocator of the heap; the shared state lives until the last handle is
 * destroyed. */
ag_status_t ag_heap_view(const ag_heap_t* heap, int rank, ag_heap_t** view);

/* Release a handle.  The caller must have synchronised every stream that
 * uses the heap.  NULL is accepted and ignored. */
ag_status_t ag_heap_destroy(ag_heap_t* heap);

/* Symmetric bump allocation: returns a byte offset valid in every region.
 * align must be a power of two >= 256 (0 = 256).  AG_ERR_OUT_OF_MEMORY when
 * the region is exhausted.  Host-only; thread-safe per heap. */
ag_status_t ag_heap_alloc(ag_heap_t* heap, size_t bytes, size_t align, size_t* offset);

/* Forget every allocation (offsets restart at 0). */
ag_status_t ag_heap_reset(ag_heap_t* heap);

/* Zero every rank's tile counters (the ticket order's; see ag_all_gather) with a small kernel on stream
 * (hipStream_t; no memset, so the call can be captured in a graph).  The counters are zero between calls
 * and need no clearing in correct use; this restores them after calls of one rank overlapped in time,
 * which the all-gather and the all-to-all do not allow and which can leave a counter non-zero for the
 * rank's later calls.
 * Stream-ordered; no call of this heap may run concurrently with it. */
ag_status_t ag_heap_clear_tickets(const ag_heap_t* heap, void* stream);

/* Device address of offset in region rank.  offset <= bytes_per_rank. */
ag_status_t ag_heap_rank_ptr(const ag_heap_t* heap, int rank, size_t offset, void** dev_ptr);

/* Device address of the uint64_t[n_ranks] base table the kernels read. */
ag_status_t ag_heap_base_table(const ag_heap_t* heap, const uint64_t** dev_table);

/* Geometry of a handle (host copy, no device access). */
ag_status_t ag_heap_geometry(const ag_heap_t* heap, ag_heap_geometry_t* geom);

/* What a device kernel needs to reach every rank's heap (ROCm/iris #591,
 * "Hoist the peer heap bases": the context knows its rank and keeps the
 * heap bases of all ranks in one device array, heap_bases, which the kernels
 * read).  Host-only, no device access:
 *   *n_ranks         number of regions (ranks) of the heap;
 *   *rank            the calling rank of a view (ag_heap_view), -1 for the
 *                    root handle;
 *   *bytes_per_rank  region stride in bytes (region r starts at
 *                    heap_bases[r] = region 0 + r*bytes_per_rank);
 *   *dev_base_table  device address of heap_bases, uint64_t[n_ranks], owned
 *                    by the heap (valid until its last handle is destroyed;
 *                    the caller must not write or free it).
 * Each output pointer may be NULL, and that item is then not reported.
 * AG_ERR_INVALID_ARG when heap is NULL.  The same values as
 * ag_heap_geometry (n_ranks, rank, bytes_per_rank) and ag_heap_base_table. */
ag_status_t ag_heap_info(const ag_heap_t* heap, int* n_ranks, int* rank, size_t* bytes_per_rank,
                         const uint64_t** dev_base_table);

/* ------------------------------------------------------------------------
 * All-gather (ROCm/iris #626 "Summary" and "Triton CCL all-gather"; result
 * defined by ROCm/iris #594 "Multi-GPU CI").
 *
 * heap          a view (ag_heap_view) of the calling rank
 * W             group size, 1..AG_MAX_WORLD
 * rank_start,
 * rank_stride   group members are regions rank_start + j*rank_stride, j < W;
 *               the view's rank must be one of them; g is its group index
 * input         device pointer to M_local x N elements, row-major, ld = N
 * out_offset    byte offset (multiple of the element size) of the gathered
 *               W*M_local x N output inside every member region
 * tile_m,tile_n tile of the persistent loop; 0,0 = 8x256.  Powers of two with
 *               tile_n in [8, 4096], tile_m in [1, 256]; one tile must hold
 *               between 1 and 8 vector accesses per thread of a 256-thread
 *               workgroup at the vector width chosen (AG_ERR_UNSUPPORTED
 *               otherwise)
 * n_programs    persistent workgroups; 0 = number of CUs
 * stream        hipStream_t
 *
 * After the call completes on stream, rows [g*M_local, (g+1)*M_local) of the
 * output in every member region hold input; no other byte of the slab
 * changes.  The input tile is read once and stored to the local region
 * first, then to the peers in rotated group order (g+1, g+2, ... mod W).
 * Calls for different ranks of a group write disjoint rows and may run
 * concurrently on different streams.  Calls for the same rank must not
 * overlap in time (order them on one stream): a call in ticket order
 * (AG_ORDER_TICKETS, the library's choice for long calls) takes its tiles
 * from a counter the heap keeps for each rank, zero between calls; calls of
 * one rank that overlap give undefined output and may leave the counter
 * non-zero for that rank's later calls (ag_heap_clear_tickets restores it).
 * M_local = 0 is a no-op.  input must not overlap any member's output
 * block, except that it may be exactly this rank's own rows in its own
 * region (in-place).
 * ------------------------------------------------------------------------ */
ag_status_t ag_all_gather(const ag_heap_t* heap, int W, int rank_start, int rank_stride,
                          const void* input, size_t out_offset, int64_t M_local, int64_t N,
                          ag_dtype_t dtype, int tile_m, int tile_n, int n_programs, void* stream);

/* The validation and launch decisions of ag_all_gather for a heap
 * geometry, without touching any device (input_addr is the device address
 * as an integer).  Returns the status ag_all_gather would return before
 * launching; fills *plan on AG_OK. */
ag_status_t ag_plan_all_gather(const ag_heap_geometry_t* geom, int W, int rank_start, int rank_stride,
                               uint64_t input_addr, size_t out_offset, int64_t M_local, int64_t N,
                               ag_dtype_t dtype, int tile_m, int tile_n, int n_programs, ag_plan_t* plan);

/* ------------------------------------------------------------------------
 * All-gather variants (ROCm/iris #594, "Reviewer performance evaluation"
 * and "Compiler inspection and grouping"; ROCm/iris #591, "INLINE
 * grouping"; ROCm/iris #626, "Triton CCL all-gather").  Same arguments,
 * result and errors as ag_all_gather, plus:
 *
 * options->dest_group  peers stored per wait.  The pages leave open whether
 *               keeping every destination's stores in flight at once costs
 *               link efficiency; grouping stores G destinations, then waits
 *               for the memory counter to retire everything before them.
 *               Supported: 0 (no grouping), and 1, 2 or 4 when it is below
 *               W and the vector width is 16 or 8 bytes (AG_ERR_UNSUPPORTED
 *               otherwise).  G >= W is the same as 0.
 * options->schedule    AG_SCHEDULE_PARTITIONED: the persistent programs are
 *               split into W equal sets, set i storing only to destination
 *               i of the rotated order (i = 0 is the local region); each
 *               program walks its set's share of the tiles, so every input
 *               tile is read W times (once per destination).  n_programs is
 *               rounded down to a multiple of W (at least W); dest_group
 *               must be 0.
 * options->tile_order  ag_tile_order_t, for AG_SCHEDULE_TILES without
 *               destination groups: AG_ORDER_STRIDE or AG_ORDER_TICKETS force
 *               the order (AG_ERR_UNSUPPORTED where no ticket kernel fits the
 *               call: vectors other than 16 bytes or more than two per thread,
 *               destination groups).  Ticket order at 256 programs, W=8,
 *               16384x8192 fp16: 6.77 TB/s against 5.28 for the grid stride;
 *               below about 64 tiles per program the counter's round trips
 *               cost more than they save.
 * Plan: ag_plan_all_gather_ex reports dest_group, schedule and tile_order as
 * applied, and bytes_read of the schedule (W times the input when
 * partitioned).
 * ------------------------------------------------------------------------ */
ag_status_t ag_all_gather_ex(const ag_heap_t* heap, int W, int rank_start, int rank_stride,
                             const void* input, size_t out_offset, int64_t M_local, int64_t N,
                             ag_dtype_t dtype, int tile_m, int tile_n, int n_programs,
                             const ag_copy_options_t* options, void* stream);

ag_status_t ag_plan_all_gather_ex(const ag_heap_geometry_t* geom, int W, int rank_start, int rank_stride,
                                  uint64_t input_addr, size_t out_offset, int64_t M_local, int64_t N,
                                  ag_dtype_t dtype, int tile_m, int tile_n, int n_programs,
                                  const ag_copy_options_t* options, ag_plan_t* plan);

/* ------------------------------------------------------------------------
 * ag_all_gather_ex for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, result, errors and kernels as
 * ag_all_gather_ex; it calls no allocating routine.  The only device memory
 * it uses beyond the input and the heap is the ticket order's tile counter,
 * which here lives in a fixed device array of the library (one counter per
 * rank index, AG_NOALLOC_MAX_RANKS of them, 4 KiB per GPU, held until the
 * process ends) instead of in the heap; each call first zeroes the calling
 * rank's counter with a small kernel on stream.  Heaps of more than
 * AG_NOALLOC_MAX_RANKS ranks give AG_ERR_UNSUPPORTED.  Every call on a GPU
 * shares that GPU's array: calls that overlap in time and use the same
 * rank index race, whichever heaps they use.
 * ------------------------------------------------------------------------ */
#define AG_NOALLOC_MAX_RANKS 64
ag_status_t ag_all_gather_noalloc(const ag_heap_t* heap, int W, int rank_start, int rank_stride,
                                  const void* input, size_t out_offset, int64_t M_local, int64_t N,
                                  ag_dtype_t dtype, int tile_m, int tile_n, int n_programs,
                                  const ag_copy_options_t* options, void* stream);

/* ------------------------------------------------------------------------
 * All-to-all on the same heap and destination machinery (ROCm/iris #594,
 * "Compiler inspection and grouping", and ROCm/iris #591, "Hoist the peer
 * heap bases": the all_to_all collective has the same per-destination
 * heap-base pattern).  The result is that of
 * torch.distributed.all_to_all_single with equal splits:
 *
 * input         device, W chunks of M_chunk x N elements, row-major (ld = N),
 *               chunk c at input + c*M_chunk*N*e; chunk c is destined for
 *               group member c
 * out_offset    byte offset (multiple of the element size) of the W*M_chunk x N
 *               output inside every member region
 * After the call completes, rows [g*M_chunk, (g+1)*M_chunk) of member j's
 * output hold chunk j of this rank's input; no other byte of the slab
 * changes.  Every destination base is translated once before the tile loop.
 * The W chunk copies are walked as one sequence of W x (tiles per chunk)
 * tiles, destination by destination: the local region first, then the peers
 * in rotated order; each tile is loaded once and stored once.  Tiles as for
 * ag_all_gather (0,0 = 8x256): 1 to 8 vectors per thread of a 256-thread
 * workgroup (AG_ERR_UNSUPPORTED otherwise; 8x256 always fits); W x tiles per
 * chunk below 2^31.  Calls for different ranks may run concurrently on
 * different streams; calls for the same rank must not overlap in time (a
 * call in ticket order uses the rank's counter, as ag_all_gather does).
 * M_chunk = 0 is a no-op.  input must not overlap any member's output
 * block.
 * ------------------------------------------------------------------------ */
ag_status_t ag_all_to_all(const ag_heap_t* heap, int W, int rank_start, int rank_stride,
                          const void* input, size_t out_offset, int64_t M_chunk, int64_t N,
                          ag_dtype_t dtype, int tile_m, int tile_n, int n_programs, void* stream);

ag_status_t ag_plan_all_to_all(const ag_heap_geometry_t* geom, int W, int rank_start, int rank_stride,
                               uint64_t input_addr, size_t out_offset, int64_t M_chunk, int64_t N,
                               ag_dtype_t dtype, int tile_m, int tile_n, int n_programs, ag_plan_t* plan);

/* ag_all_to_all with options (NULL or all-zero = ag_all_to_all).  Same
 * result.  dest_group must be 0 (AG_ERR_INVALID_ARG otherwise).  tile_order
 * as for ag_all_gather_ex (AG_SCHEDULE_TILES only).  schedule
 * AG_SCHEDULE_PARTITIONED (the partitioned schedule of ag_all_gather_ex
 * applied to the exchange): program p owns destination i = p mod W of the
 * rotated order and copies chunk (g + i) mod W there, the programs of one
 * destination walking all tiles among themselves; every chunk is read once.
 * n_programs is rounded down to a multiple of W (at least W). */
ag_status_t ag_all_to_all_ex(const ag_heap_t* heap, int W, int rank_start, int rank_stride,
                             const void* input, size_t out_offset, int64_t M_chunk, int64_t N,
                             ag_dtype_t dtype, int tile_m, int tile_n, int n_programs,
                             const ag_copy_options_t* options, void* stream);

ag_status_t ag_plan_all_to_all_ex(const ag_heap_geometry_t* geom, int W, int rank_start, int rank_stride,
                                  uint64_t input_addr, size_t out_offset, int64_t M_chunk, int64_t N,
                                  ag_dtype_t dtype, int tile_m, int tile_n, int n_programs,
                                  const ag_copy_options_t* options, ag_plan_t* plan);

/* ------------------------------------------------------------------------
 * Fused GEMM + all-gather (ROCm/iris #626 "Assembly" table and "Benchmark").
 *
 * C = A . B with fp32 accumulation, rounded once (nearest-even) to dtype,
 * then stored exactly as ag_all_gather stores its input: rows
 * [g*M_local, (g+1)*M_local) of the W*M_local x N output at out_offset in
 * every member region, local region first, peers in rotated order.
 *
 * A             device, M_local x K, row-major, element (m,k) at A[m*lda + k], lda >= K
 * B             device, K-contiguous: element (k,n) at B[n*ldb + k], ldb >= K
 *               (the N x K row-major weight of a linear layer)
 * dtype         AG_F16 or AG_BF16 (A, B and C share it); AG_F32 -> AG_ERR_UNSUPPORTED
 * tile_m,tile_n,tile_k   0,0,0 = chosen by the library: the configuration
 *               with the fewest rounds-of-tiles x tile-area on the busiest
 *               program (ties to the larger tile); explicit values must be
 *               one of 256x256x64, 256x224x64, 128x128x64
 * n_programs    persistent workgroups; 0 = number of CUs (capped at the tile count)
 * Requirements: K a positive multiple of 64, lda/ldb multiples of 8, A, B
 * 16-byte aligned, N*2 and out_offset multiples of 16 bytes.  M_local and N
 * need not be tile multiples.  M_local = 0 is a no-op.  A and B must not
 * overlap any member's output block.
 * ------------------------------------------------------------------------ */
ag_status_t ag_gemm_all_gather(const ag_heap_t* heap, int W, int rank_start, int rank_stride,
                               const void* A, int64_t lda, const void* B, int64_t ldb,
                               size_t out_offset, int64_t M_local, int64_t N, int64_t K,
                               ag_dtype_t dtype, int tile_m, int tile_n, int tile_k,
                               int n_programs, void* stream);

/* Host-only validation and launch decisions of ag_gemm_all_gather. */
ag_status_t ag_plan_gemm_all_gather(const ag_heap_geometry_t* geom, int W, int rank_start, int rank_stride,
                                    uint64_t a_addr, int64_t lda, uint64_t b_addr, int64_t ldb,
                                    size_t out_offset, int64_t M_local, int64_t N, int64_t K,
                                    ag_dtype_t dtype, int tile_m, int tile_n, int tile_k,
                                    int n_programs, ag_plan_t* plan);

/* Storage of B for ag_gemm_all_gather_ex. */
typedef enum ag_b_layout {
    AG_B_K_CONTIGUOUS = 0,  /* element (k,n) at B[n*ldb + k], ldb >= K (as ag_gemm_all_gather) */
    AG_B_N_CONTIGUOUS = 1   /* element (k,n) at B[k*ldb + n], ldb >= N (a row-major K x N matrix) */
} ag_b_layout_t;

/* Options of ag_gemm_all_gather_ex; all-zero (or a NULL pointer) is ag_gemm_all_gather. */
typedef struct ag_gemm_options {
    int32_t b_layout;     /* ag_b_layout_t */
    int32_t reserved[7];  /* must be 0 */
} ag_gemm_options_t;

/* ag_gemm_all_gather with options: the same product and stores, with B in
 * either layout.  With AG_B_N_CONTIGUOUS, ldb >= N (multiple of 8), B
 * 16-byte aligned, and 64 rows of B plus a tile's columns
 * ((64*ldb + tile_n)*2 bytes) under 2 GiB (AG_ERR_UNSUPPORTED otherwise);
 * B itself may be larger.  The tiles are 256x224x64 or
 * 128x128x64 (0,0,0 chooses between them; 256x256x64 gives
 * AG_ERR_UNSUPPORTED).  The kernel reads the N-contiguous stage with LDS
 * transposing reads instead of a transpose pass. */
ag_status_t ag_gemm_all_gather_ex(const ag_heap_t* heap, int W, int rank_start, int rank_stride,
                                  const void* A, int64_t lda, const void* B, int64_t ldb,
                                  size_t out_offset, int64_t M_local, int64_t N, int64_t K,
                                  ag_dtype_t dtype, int tile_m, int tile_n, int tile_k,
                                  int n_programs, const ag_gemm_options_t* options, void* stream);

ag_status_t ag_plan_gemm_all_gather_ex(const ag_heap_geometry_t* geom, int W, int rank_start, int rank_stride,
                                       uint64_t a_addr, int64_t lda, uint64_t b_addr, int64_t ldb,
                                       size_t out_offset, int64_t M_local, int64_t N, int64_t K,
                                       ag_dtype_t dtype, int tile_m, int tile_n, int tile_k,
                                       int n_programs, const ag_gemm_options_t* options, ag_plan_t* plan);

/* ------------------------------------------------------------------------
 * Linear layer: the matrix product with bias, activation and residual in its
 * epilogue, and its gradients.  One rank's product on dense matrices anywhere
 * in device memory (a region of the heap, a tensor): what a sequence-parallel
 * rank does between an all-gather of its input and its own loss.
 *
 *   z = x . w^T + bias                       (fp32)
 *   y = act(z) + residual                    (fp32, rounded once to dtype)
 *
 * x         device, M x K, element (m,k) at x[m*ldx + k]
 * w         device, N x K, element (n,k) at w[n*ldw + k]
 * bias      device, N elements, or NULL
 * residual  device, M x N (row stride ldr), or NULL; may be y itself (same
 *           address and stride)
 * y         device, M x N (row stride ldy)
 * z         device, M x N (row stride ldz), or NULL: the pre-activation
 *           rounded to dtype, which the backward pass reads
 * dtype     AG_F16 or AG_BF16, shared by all of them (AG_F32 -> AG_ERR_UNSUPPORTED)
 * M, N, K   any size from 0 (K = 0: y = act(bias) + residual)
 * ld*       row strides in elements; 0 = dense (K or N); any value >= the row
 * Pointers need only their element's alignment.  Operands of a tiled product
 * whose rows are not 4-byte aligned are copied to the workspace first (the
 * plan's `packed`; few rows of x need no tiles and no copy).  Row strides are
 * at most 2^20 elements (AG_ERR_UNSUPPORTED otherwise).
 * Outputs must not overlap inputs or each other (but y and residual, above).
 * What lies between a matrix's rows (ld > row) is never written and never has
 * an effect; nothing is read before a matrix's first element or after the
 * aligned 4 bytes that hold its last one.
 *
 * workspace  device memory of at least the plan's workspace_bytes, 256-byte
 *            aligned, not shared by calls that may run at once; its contents
 *            need no initialisation and are not kept.  May be NULL if 0 bytes.
 * The result does not depend on the stream, on the workspace or on timing
 * (partial sums are joined in a fixed order, without atomics).
 * ------------------------------------------------------------------------ */
typedef enum ag_act {
    AG_ACT_NONE = 0,
    AG_ACT_RELU = 1,       /* z < 0 ? 0 : z, slope 0 at z <= 0 */
    AG_ACT_GELU = 2,       /* z/2 (1 + erf(z/sqrt 2)) */
    AG_ACT_GELU_TANH = 3,  /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
    AG_ACT_SILU = 4        /* z / (1 + exp(-z)) */
} ag_act_t;

typedef struct ag_linear_args {
    const void* x;
    const void* w;
    const void* bias;
    const void* residual;
    void* y;
    void* z;
    int64_t ldx, ldw, ldr, ldy, ldz;
    int64_t M, N, K;
    int32_t dtype;        /* ag_dtype_t */
    int32_t act;          /* ag_act_t */
    int32_t reserved[6];  /* must be 0 */
} ag_linear_args_t;

/* One matrix product as it will be launched. */
typedef struct ag_product_plan {
    int32_t variant;      /* 0 = not computed, 1 = row streaming (few rows of x), 2 = tiles */
    int32_t tile_m, tile_n, tile_k;
    int32_t full_tiles;   /* tiles that one workgroup computes whole */
    int32_t splits;       /* parts that the others' reductions are cut into; a second kernel joins them */
    int32_t n_programs;   /* persistent workgroups */
    int32_t packed;       /* bit 0 / 1: first / second operand copied to aligned rows first */
} ag_product_plan_t;

typedef struct ag_linear_plan {
    ag_product_plan_t product;     /* y (linear); dx (linear_backward) */
    ag_product_plan_t product_dw;  /* dw (linear_backward) */
    uint64_t workspace_bytes;
    uint64_t bytes_read;           /* algorithmic: each input once */
    uint64_t bytes_written;
    double flops;
    int32_t launches;
    int32_t reserved;
} ag_linear_plan_t;

ag_status_t ag_linear(const ag_linear_args_t* args, void* workspace, size_t workspace_bytes, void* stream);

/* Host-only validation and launch decisions of ag_linear on a device of
 * num_cus compute units (0 = the current HIP device's). */
ag_status_t ag_plan_linear(const ag_linear_args_t* args, int num_cus, ag_linear_plan_t* plan);

/* Gradients of the linear layer, from the gradient dy of y:
 *
 *   dz = dy * act'(z)
 *   dx = dz . w            (M x K)
 *   dw = dz^T . x          (N x K)       + dw if accumulate
 *   db = sum over rows dz  (N)           + db if accumulate
 *
 * (the residual's gradient is dy itself).  Sums are fp32; dx has the
 * operands' dtype, dw and db have dw_dtype: the operands' dtype or AG_F32.
 * With an activation, dz is rounded once to dtype, the type its products'
 * matrix instructions take, for dx and for a dw of that type; a dw in AG_F32
 * takes dz in two terms of dtype (the rounded one and what it leaves, rounded)
 * and so two products.  db sums the unrounded dz.  z is the pre-activation
 * that ag_linear stored; it may be NULL when act is AG_ACT_NONE.  dx, dw and
 * db may each be NULL (not computed); accumulate adds to dw and db in fp32
 * before the one rounding.  x is read only for dw, w only for dx; either may
 * be NULL when its gradient's partner is not asked for.  Sizes, strides,
 * alignment, overlap and the workspace are as for ag_linear.  M = 0 gives
 * zero gradients dw and db (or leaves them, with accumulate). */
typedef struct ag_linear_backward_args {
    const void* dy;
    const void* z;
    const void* x;
    const void* w;
    void* dx;
    void* dw;
    void* db;
    int64_t lddy, ldz, ldx, ldw, lddx, lddw;
    int64_t M, N, K;
    int32_t dtype;        /* ag_dtype_t of dy, z, x, w and dx */
    int32_t act;          /* ag_act_t */
    int32_t dw_dtype;     /* ag_dtype_t of dw and db */
    int32_t accumulate;   /* 0 or 1 */
    int32_t reserved[4];  /* must be 0 */
} ag_linear_backward_args_t;

ag_status_t ag_linear_backward(const ag_linear_backward_args_t* args, void* workspace, size_t workspace_bytes,
                               void* stream);
ag_status_t ag_plan_linear_backward(const ag_linear_backward_args_t* args, int num_cus, ag_linear_plan_t* plan);

/* ------------------------------------------------------------------------
 * Rows in 8 bits.  One format serves activations, weights and checkpoints: a
 * row of K numbers v becomes K codes and one fp32 scale,
 *
 *   a = max |v_k|,  q_k = the whole number nearest to 127 v_k / a (ties to
 *   even),  scale = a / 127,                v_k stands as q_k * scale
 *
 * so that |q| <= 127.  The codes are those of exact arithmetic, whatever the
 * row's size or the kernel that made them.  A row of zeros has zero codes and
 * scale 0; a NaN or an infinity makes its row's scale NaN and its codes 0.
 *
 * x       device, M x K of dtype (AG_F16, AG_BF16 or AG_F32), row stride ldx
 * q       device, M x K int8, row stride ldq
 * scale   device, M floats
 * y       device, M x K of dtype, row stride ldy: q * scale, rounded once
 * M below 2^31, K up to 2^20; strides as for ag_linear (0 = dense).  Outputs
 * must not overlap inputs or each other.  One launch each; nothing to do for
 * M = 0 (K = 0: the scales are 0).
 * ------------------------------------------------------------------------ */
ag_status_t ag_quantize_rows(const void* x, int64_t ldx, int8_t* q, int64_t ldq, float* scale, int64_t M, int64_t K,
                             ag_dtype_t dtype, void* stream);
ag_status_t ag_dequantize_rows(const int8_t* q, int64_t ldq, const float* scale, void* y, int64_t ldy, int64_t M,
                               int64_t K, ag_dtype_t dtype, void* stream);

/* ------------------------------------------------------------------------
 * Root-mean-square norm, with the residual's addition before it and an output
 * in 16 or in 8 bits: what stands between two linear layers.
 *
 *   h = x + residual                  (rounded to dtype: the norm is of what is stored)
 *   rstd = 1 / sqrt(mean of h^2 over the row + eps)
 *   y = h rstd weight                 (rounded once)
 *   q, scale: the row h weight in 8 bits as above, its scale times rstd
 *
 * x, residual, h, y   device, M x K of dtype (AG_F16 or AG_BF16); residual,
 *            h and y may be NULL; h may be x or residual itself (same address
 *            and stride)
 * weight     device, K of dtype, or NULL (ones)
 * q, scale   device, M x K int8 and M floats, or both NULL
 * rstd       device, M floats, or NULL (ag_rms_norm_backward reads it)
 * eps        finite, 1e-60 or more
 * Squares are summed in fp64: no size of h leaves their range.  Products h
 * weight are exact in fp32 wherever they lie within its normal numbers, and
 * the codes are those of exact arithmetic there.  A product past fp32's
 * largest is an infinity: in y, and its row's scale is NaN with codes 0, as
 * one with a NaN or an infinity.
 * Sizes, strides and overlaps as above.  One launch.
 * ------------------------------------------------------------------------ */
typedef struct ag_rms_norm_args {
    const void* x;
    const void* residual;
    const void* weight;
    void* h;
    void* y;
    int8_t* q;
    float* scale;
    float* rstd;
    int64_t ldx, ldr, ldh, ldy, ldq;
    int64_t M, K;
    double eps;
    int32_t dtype;        /* ag_dtype_t */
    int32_t reserved[7];  /* must be 0 */
} ag_rms_norm_args_t;

typedef struct ag_rows_plan {
    int32_t threads_per_row;       /* of a workgroup */
    int32_t vectors_per_thread;    /* of 8 elements, kept in registers; 0: the row is read twice */
    int32_t n_programs;            /* workgroups */
    int32_t launches;
    uint64_t workspace_bytes;
    uint64_t bytes_read;           /* algorithmic: each input once */
    uint64_t bytes_written;
} ag_rows_plan_t;

ag_status_t ag_rms_norm(const ag_rms_norm_args_t* args, void* stream);
ag_status_t ag_plan_rms_norm(const ag_rms_norm_args_t* args, int num_cus, ag_rows_plan_t* plan);

/* Gradients of the norm, from the gradient dy of y and, where h goes on past
 * the norm (the residual's way), the gradient dh that reaches h there:
 *
 *   g = dy weight
 *   dx = rstd (g - h rstd^2 mean(g h)) + dh     (x's gradient and the residual's alike)
 *   dw = sum over rows dy h rstd                + dw if accumulate
 *
 * dy, h, dh, dx  device, M x K of dtype; dh may be NULL, dx may be dh itself
 *                (same address and stride); h is what ag_rms_norm normalised
 * rstd           device, M floats
 * weight         device, K of dtype, or NULL (ones)
 * dx, dw         either may be NULL (not computed); dw has dw_dtype: dtype or
 *                AG_F32
 * Sums are fp32 (mean(g h): one row's; dw: rows dealt to the workgroups, then
 * their sums in a fixed order, without atomics).  The workspace is as for
 * ag_linear.  M = 0 gives a zero dw (or leaves it, with accumulate). */
typedef struct ag_rms_norm_backward_args {
    const void* dy;
    const void* h;
    const void* dh;
    const void* weight;
    const float* rstd;
    void* dx;
    void* dw;
    int64_t lddy, ldh, lddh, lddx;
    int64_t M, K;
    int32_t dtype;        /* ag_dtype_t */
    int32_t dw_dtype;     /* ag_dtype_t */
    int32_t accumulate;   /* 0 or 1 */
    int32_t reserved[5];  /* must be 0 */
} ag_rms_norm_backward_args_t;

ag_status_t ag_rms_norm_backward(const ag_rms_norm_backward_args_t* args, void* workspace, size_t workspace_bytes,
                                 void* stream);
ag_status_t ag_plan_rms_norm_backward(const ag_rms_norm_backward_args_t* args, int num_cus, ag_rows_plan_t* plan);

/* ------------------------------------------------------------------------
 * Linear layer on 8-bit integers with a scale for each row of x (token) and
 * of w (output channel), as ag_quantize_rows or ag_rms_norm make them:
 *
 *   z = x_scale[m] w_scale[n] sum_k x(m,k) w(n,k) + bias
 *   y = act(z) + residual                    (fp32, rounded once to dtype)
 *
 * The sums are exact (int32), and with finite scales z leaves fp32's range only
 * where x_scale w_scale times the sum does, whatever x_scale times the sum is.
 * x is M x K, w N x K, both int8; K up to 131071 (131072 products of -128 and
 * -128 would leave int32).  bias, residual, y and z have dtype (AG_F16 or
 * AG_BF16).  Everything else is as for ag_linear;
 * operands of a tiled product whose rows do not start on 4 bytes are copied.
 * ------------------------------------------------------------------------ */
typedef struct ag_linear_i8_args {
    const int8_t* x;
    const int8_t* w;
    const float* x_scale;  /* M */
    const float* w_scale;  /* N */
    const void* bias;
    const void* residual;
    void* y;
    void* z;
    int64_t ldx, ldw, ldr, ldy, ldz;
    int64_t M, N, K;
    int32_t dtype;        /* ag_dtype_t */
    int32_t act;          /* ag_act_t */
    int32_t reserved[6];  /* must be 0 */
} ag_linear_i8_args_t;

ag_status_t ag_linear_i8(const ag_linear_i8_args_t* args, void* workspace, size_t workspace_bytes, void* stream);
ag_status_t ag_plan_linear_i8(const ag_linear_i8_args_t* args, int num_cus, ag_linear_plan_t* plan);

/* ag_linear_backward from activations that were kept in 8 bits: where x_scale
 * (M floats) is not NULL, args->x holds int8 codes (ldx in codes), and where
 * z_scale is not NULL, args->z does.  The gradients are those of the values
 * that the codes stand for.  For dw, x_scale times dz is rounded to dtype, but for
 * a power of two, which goes to the codes and leaves them exact: one rounding,
 * and no rounded copy of x.  (Without codes dz is rounded behind gelu,
 * gelu_tanh and silu, and exact behind none and relu.)  A dw in AG_F32 takes
 * dz in two terms of AG_F16 or three of AG_BF16, and their products.
 * In AG_BF16 the other factor lies in [1/2, 1) for scales of 2^-126 to 2^119.  In
 * AG_F16 the power is taken from the scale and the row's largest finite |dy|,
 * D: an element of dz is off by at most half a step of itself in one term and
 * 2^-22 of itself in two, or by 2^-24 D where that is more (by 2^-49 / x_scale
 * where x_scale D is below 2^-23); dz x_scale of 2^24 and more leaves AG_F16.
 * The workspace holds dz, its terms and x's codes as values of dtype: for a dw in
 * AG_F32 one copy of these per term unless M / 32 (rounded down) is above N or
 * the copies past the first would take more than 128 MiB.  Either scale may be
 * NULL. */
ag_status_t ag_linear_backward_q8(const ag_linear_backward_args_t* args, const float* x_scale, const float* z_scale,
                                  void* workspace, size_t workspace_bytes, void* stream);
ag_status_t ag_plan_linear_backward_q8(const ag_linear_backward_args_t* args, const float* x_scale, const float* z_scale,
                                       int num_cus, ag_linear_plan_t* plan);

/* ------------------------------------------------------------------------
 * AdamW over many tensors in one launch, with states in 32 or in 8 bits.
 * A handle keeps a device table of the tensors' addresses, made once (as a
 * heap keeps its base table); the tensors must stay where they are while the
 * handle is used.  For every element, with g = grad * grad_scale:
 *
 *   m = beta1 m + (1 - beta1) g
 *   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
 *
 * in fp32 (m and v of 8-bit states in fp64).  p is the master copy where
 * there is one (fp32; param then receives it rounded), else param itself.
 *
 * 8-bit states: blocks of AG_ADAMW_BLOCK consecutive elements of a tensor
 * share one fp32 maximum S per state.  A code c stands for
 *   m = sign(c) (|c|/127)^2 S   (int8)       v = (c/255)^4 S   (uint8),
 * so that an m reaches down to 6.2e-5 of its block's largest (to nearest,
 * below 1.6e-5 it is 0) and a sqrt(v) to 1.5e-5.  A value's code is floor(t + u), t its place on that scale and
 * u = 1/2 (nearest), or with stochastic rounding a number in (0,1) that a
 * counter hash makes from the seed and the element's place: updates far
 * smaller than a code's step then count on average instead of never.  v > 0
 * never rounds to the code 0, so no live first moment meets a zero
 * denominator.  All-zero codes and scales are the zero state.  A NaN or an
 * infinity (also a v past fp32's largest, from gradients of about 1e20 on)
 * makes its whole block's state NaN (the parameters: its element).
 * ------------------------------------------------------------------------ */
#define AG_ADAMW_BLOCK 256

typedef struct ag_adamw ag_adamw_t;  /* opaque */

typedef struct ag_adamw_tensor {
    void* param;
    const void* grad;
    void* exp_avg;            /* float[n], or int8_t[n] */
    void* exp_avg_sq;         /* float[n], or uint8_t[n] */
    float* exp_avg_scale;     /* 8-bit states: float[ceil(n / AG_ADAMW_BLOCK)], else NULL */
    float* exp_avg_sq_scale;
    float* master;            /* float[n], or NULL (all tensors of a handle alike) */
    int64_t n;                /* elements, >= 0 */
} ag_adamw_tensor_t;

/* Pointers need their element's alignment.  param_dtype and grad_dtype: any
 * ag_dtype_t; master weights only with a 16-bit param_dtype.  state_bits: 32
 * or 8.  Tensors must not overlap.  Allocates and fills the table (a
 * synchronising call); 1 <= count <= 2^20, below 2^40 elements in all. */
ag_status_t ag_adamw_create(const ag_adamw_tensor_t* tensors, int64_t count, ag_dtype_t param_dtype,
                            ag_dtype_t grad_dtype, int state_bits, ag_adamw_t** out);
/* The steps that use the table must have completed, and no captured graph that holds one may run any more. */
ag_status_t ag_adamw_destroy(ag_adamw_t* optimizer);

typedef struct ag_adamw_hyper {
    double lr, beta1, beta2, eps, weight_decay, grad_scale;
    int64_t step;                 /* >= 1: the number of this step */
    const int64_t* dev_step;      /* optional device scalars, read by the kernel instead of the host's value (a */
    const float* dev_lr;          /*   step >= 1): a captured graph's step then follows them from replay to replay */
    const float* dev_grad_scale;  /*   (multiplied with grad_scale: a clipping factor) */
    uint64_t seed;                /* stochastic rounding's seed: another one for every step */
    int32_t stochastic;           /* 1: stochastic rounding of 8-bit states, seed + *dev_step where there is one */
    int32_t reserved[5];          /* must be 0 */
} ag_adamw_hyper_t;

/* 0 <= beta < 1, eps > 0, the rest finite.  One launch; nothing to do for zero elements. */
ag_status_t ag_adamw_step(const ag_adamw_t* optimizer, const ag_adamw_hyper_t* hyper, void* stream);

/* The values that 8-bit states stand for, as fp32 (checkpoints): exp_avg[i]
 * and exp_avg_sq[i] are host arrays of count device addresses of float[n].
 * AG_ERR_INVALID_ARG on a handle of 32-bit states. */
ag_status_t ag_adamw_read_states(const ag_adamw_t* optimizer, float* const* exp_avg, float* const* exp_avg_sq,
                                 void* stream);

/* ------------------------------------------------------------------------ */
const char* ag_status_string(ag_status_t status);  /* static string, never NULL */
const char* ag_last_error_message(void);           /* thread-local; "" after AG_OK */
const char* ag_version(void);                      /* static string */

#ifdef __cplusplus
}
#endif

#endif /* AG_H */
