/*
 * argreduce.h - row-wise ArgMax / ArgMin over the last axis on a GB300 GPU.
 *
 * C ABI of libargreduce.so. Every argument is a plain pointer or integer; no
 * C++ or framework type crosses this boundary. Device pointers are CUDA
 * device addresses in the caller's current context. The library never
 * allocates, frees or synchronises memory inside argreduce(); all work is
 * queued on the caller's stream.
 *
 * The operation is defined by two onnxruntime pull requests:
 *   - "[CUDA] Parallelize ArgMax/ArgMin over wide last axes" (#32092),
 *     sections Approach and Semantics: a [rows, cols] row-major tensor is
 *     reduced over its last axis to one int64 index per row; ties resolve to
 *     the lowest index; a leading NaN yields index 0; rows that are entirely
 *     -inf, +inf or NaN yield index 0; the result equals the sequential
 *     one-thread-per-row scan bit for bit for every input.
 *   - "[CUDA] Parallelize ArgMax/ArgMin over the reduction axis" (#31694),
 *     section Semantics: the sequential scan seeds with element 0 and a later
 *     element replaces the candidate only when strictly better.
 *
 * "Strictly better" is an IEEE comparison: greater (ArgMax) or less (ArgMin),
 * false when either operand is NaN. So a NaN after element 0 never wins, +0.0
 * and -0.0 tie (lowest index wins), and subnormals are compared exactly
 * (no flush to zero). binary16 and bfloat16 values are compared after an
 * exact widening to binary32.
 */
#ifndef ARGREDUCE_H
#define ARGREDUCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The same type as cudaStream_t. NULL is the legacy default stream. */
typedef struct CUstream_st* argr_stream;

/* Element type of x (and of out_val). argreduce() and argreduce_axis() take
 * the floating types; the integer types are for argreduce_cum(). */
typedef enum {
    ARGR_F32 = 0,  /* IEEE binary32 */
    ARGR_F16 = 1,  /* IEEE binary16 */
    ARGR_BF16 = 2, /* bfloat16 (upper half of binary32) */
    ARGR_F64 = 3,  /* IEEE binary64 */
    ARGR_I32 = 4,  /* int32: argreduce_cum() only */
    ARGR_I64 = 5   /* int64: argreduce_cum() only */
} argr_dtype;

/* ArgMax / ArgMin; ties resolve to the first index, or to the last index for
 * the *_LAST ops (ONNX select_last_index = 1: the same scan with a non-strict
 * comparison, still false on NaN, so NaN handling is unchanged). */
typedef enum { ARGR_MAX = 0, ARGR_MIN = 1, ARGR_MAX_LAST = 2, ARGR_MIN_LAST = 3 } argr_op;

typedef enum {
    ARGR_OK = 0,
    ARGR_EINVAL = 1,      /* bad pointer, size, enum or plan; nothing was launched */
    ARGR_ESCRATCH = 2,    /* scratch missing, too small or not 16-byte aligned; nothing launched */
    ARGR_EUNSUPPORTED = 3,/* valid request this build or device cannot run; nothing launched */
    ARGR_ECUDA = 4,       /* a CUDA runtime call failed (launch or device query) */
    ARGR_ETIMEOUT = 5     /* a bounded device-side wait expired (reported by argreduce_read_error) */
} argr_status;

/* Kernel paths the planner chooses between (#32092 Approach: thread per row
 * for narrow rows; a row spread over warps and blocks otherwise). */
typedef enum {
    ARGR_PATH_NONE = 0,    /* rows == 0: nothing to launch */
    ARGR_PATH_ROWS = 1,    /* `group` lanes per row (1 = thread per row, 32 = warp per row) */
    ARGR_PATH_SPLIT = 2,   /* `blocks_per_row` CTAs per row; >1 merges through scratch,
                              the last CTA to arrive for a row reduces the partials */
    ARGR_PATH_CLUSTER = 3, /* one thread-block cluster of `cluster` CTAs per row, merged
                              through distributed shared memory; no scratch. With a row
                              slot per row (grid_rows == rows) and at most 512 threads
                              per CTA every warp pushes its
                              candidate into CTA 0 (st.async on an mbarrier, a bounded
                              wait in CTA 0); with fewer slots CTAs loop over rows and
                              merge through a cluster barrier */
    ARGR_PATH_AXIS = 5,    /* non-last axis (argreduce_axis): a warp is `group` column lanes (each
                              V consecutive inner positions, `vec`: V-element vectors) by 32/group
                              lanes along R; the CTA's block/32 warps split R, and a cluster of
                              `cluster` CTAs (1 = none) splits it further. unroll 4 or 8 */
    ARGR_PATH_CUM = 6,     /* cummax / cummin (argreduce_cum): a row in `cluster` chunks, one CTA
                              each (1 = none), scanned in tiles of block * 7 elements */
    ARGR_PATH_CUM_SPLIT = 7, /* cummax / cummin: a row in `blocks_per_row` chunks, one CTA each,
                              any number of CTAs; chunk aggregates are exchanged through
                              scratch (rows * blocks_per_row <= 65536; above 1024 record
                              words the records need a scratch buffer of more than 1 MiB) */
    ARGR_PATH_CUM_STREAM = 8, /* cummax / cummin: tiles of block * 7 elements (`blocks_per_row` =
                              tiles per row) taken in ticket order by `grid_rows` CTAs, each
                              tile read once; carries by decoupled look-back through scratch
                              (rows * blocks_per_row <= 32768). Not chosen by the planner */
    ARGR_PATH_LOGITS = 9,  /* vocabulary rows, forward (argreduce_logprobs, argreduce_distill): `block`
                              threads per CTA, `cluster` CTAs per row (1 = none), `grid_rows`
                              row slots */
    ARGR_PATH_LOGITS_GRAD = 10, /* vocabulary rows, gradients: a row in `blocks_per_row` chunks, a
                              CTA of `block` threads each */
    ARGR_PATH_LOGITS_STEP = 11, /* argreduce_distill_step: as ARGR_PATH_LOGITS, the row held in the shared
                              memory of its CTAs (about 40 KB each, at most 108) */
    ARGR_PATH_LOGITS_STREAM = 12, /* vocabulary rows, forward: `grid_rows` persistent CTAs of `block` threads,
                              `group` (1 to 3) of their warps finish rows while the others read on */
    ARGR_PATH_STREAM = 4   /* every warp streams a contiguous range of rows through its own
                              `stages` shared-memory buffers of `stage_bytes`, filled by bulk
                              (TMA) copies; `group` lanes per row for rows that fit a buffer,
                              the whole warp otherwise. Needs 16-byte aligned rows. */
} argr_path;

/* Device properties the planner uses. */
typedef struct {
    int32_t sm_count;           /* streaming multiprocessors */
    int32_t max_threads_per_sm; /* resident threads per SM */
    int32_t max_cluster;        /* largest cluster size this device launches (1 = none) */
    int32_t cc_major, cc_minor; /* compute capability */
} argr_caps;

/* Plan flag: launch as a programmatic dependent of the previous grid in the
 * stream. The kernel still waits for that grid to complete before it touches
 * memory, so results are the same; only the launch latency overlaps. */
#define ARGR_PLAN_PDL 1
/* Plan flag (CLUSTER path): each CTA's share of the row is fetched into shared
 * memory by bulk (TMA) copies issued all at once, instead of by loads from
 * every thread. The share must be at most 128 KiB. */
#define ARGR_PLAN_BULK 2
/* Plan flag for tests of failure handling (STREAM, CLUSTER with a row slot
 * per row, CUM_SPLIT, CUM_STREAM and LOGITS_STEP paths only). STREAM: one bulk copy's
 * barrier is made to expect more bytes than arrive, so the kernel's bounded
 * wait (2 ms under this flag) expires; the kernel records the expiry, skips
 * its work and returns. CLUSTER (push merge only: grid_rows == rows, at
 * most 512 threads): CTA 0's barrier expects 16 bytes more than
 * the cluster's candidates, so its wait expires and it returns without
 * writing the row. CUM_SPLIT and
 * CUM_STREAM: the first chunk (tile) of each row never publishes its record,
 * so every wait for it expires after 2 ms. Either way argreduce_read_error()
 * then reports ARGR_ETIMEOUT and outputs are undefined. LOGITS_STEP: the last
 * stage of every CTA's part expects 16 bytes more than are copied, as STREAM
 * does. Never set in the planner's plans. */
#define ARGR_PLAN_TEST_EXPIRE 4
/* Plan flag (CUM_SPLIT path): each CTA copies its whole chunk (at most 80 KiB)
 * into shared memory with bulk (TMA) copies and scans it there, so the input
 * is read from memory once; without it, phase B reads the chunk again (from
 * L2 while the chunks in flight fit it). Measured slower on GB300 at every
 * size (two CTAs per SM alternate loading and scanning), so the planner does
 * not set it. */
#define ARGR_PLAN_STASH 8
/* Plan flag (CUM_SPLIT path, not with ARGR_PLAN_STASH): decoupled look-back.
 * Every chunk also publishes its inclusive prefix once known, and a CTA reads
 * back only to the nearest one, so chunks can be one tile each (read once,
 * from registers) at any chunk count; two record words per chunk. */
#define ARGR_PLAN_LOOKBACK 16
/* Plan flag (ROWS path with vec = 1 and group 16 or 32): software-pipelined
 * loads. Every lane issues the next batch of `unroll` 16-byte loads before it
 * compares the current batch, so its loads stay in flight while it compares;
 * twice the registers for loaded data, so at most 256 threads per CTA. */
#define ARGR_PLAN_PIPELINE 32
/* Plan flag (ROWS, SPLIT, CLUSTER and STREAM paths): before its dependency
 * wait, each CTA asks the L2 cache to fetch the part of x it reads first (bulk L2
 * prefetches of 16-byte aligned pieces). A prefetch changes no value (L2 is
 * where the GPU keeps memory coherent, so a line written by the previous
 * grid is read as written), so results are the same; when the CTA starts
 * while the previous grid in the stream is still running (ARGR_PLAN_PDL),
 * the read of x from HBM overlaps that grid instead of following it. */
#define ARGR_PLAN_PREFETCH 64
/* Plan flag (ROWS path, with ARGR_PLAN_PREFETCH): each CTA prefetches at most
 * 16 KiB (the head of its rows) instead of 128 KiB. For inputs above 32 MiB,
 * where two calls' inputs no longer share L2: only the first bytes each CTA
 * reads come early, covering the gap between the previous grid's last loads
 * and this grid's first, without evicting what the previous grid still needs. */
#define ARGR_PLAN_PREFETCH_HEAD 128

/* A launch plan. Produced by argreduce_plan(); tests may edit it to force a
 * path and pass it to argreduce_with_plan(), which re-validates it. */
typedef struct {
    int32_t path;           /* argr_path */
    int32_t block;          /* threads per CTA: multiple of 32, 32..1024 */
    int32_t group;          /* ROWS / STREAM: lanes per row; AXIS: column lanes per warp; power of two 1..32 */
    int32_t vec;            /* 1: 16-byte vector loads (ROWS needs every row 16-byte aligned) */
    int32_t unroll;         /* loads in flight per thread per step: ROWS 4 or 8; SPLIT/CLUSTER 1,2,4,8 */
    int32_t cluster;        /* CLUSTER: CTAs per cluster, 2..16 */
    int32_t flags;          /* ARGR_PLAN_* bits */
    int32_t stages;         /* STREAM: buffers per warp, 1..4 */
    int32_t stage_bytes;    /* STREAM: bytes per buffer, multiple of 16, 1 KiB..64 KiB */
    int32_t reserved;       /* 0 */
    int64_t blocks_per_row; /* SPLIT / CLUSTER / CUM: CTAs that share one row; CUM_SPLIT: chunks
                               per row; CUM_STREAM: tiles per row */
    int64_t grid_rows;      /* SPLIT / CLUSTER / CUM: row slots in the grid (rows loop over them;
                               CUM_SPLIT: the rows); ROWS / STREAM / CUM_STREAM: number of CTAs */
    uint64_t scratch_bytes; /* bytes of scratch this plan needs (0 = none) */
} argr_plan;

/*
 * Scratch bytes argreduce() needs for this problem on the current device
 * (0 when the chosen path needs none). The bound is small: a multi-CTA row
 * needs one 16-byte partial per CTA plus a 4-byte counter per row, and such
 * plans are only chosen while the whole grid fits one wave of the device
 * (#32092 Approach: scratch bounded by the device's thread capacity).
 * Returns 0 also when the device cannot be queried; argreduce() then reports
 * the error.
 */
size_t argreduce_scratch_bytes(int64_t rows, int64_t cols, argr_dtype dtype, argr_op op);

/*
 * Prepare a scratch buffer once after allocating it: zeroes the per-row
 * arrival counters and the error word (an asynchronous memset on `stream`).
 * After that the counters reset themselves at the end of every call, so no
 * per-call memset is needed and argreduce() can be captured in a CUDA graph
 * and replayed. The partial-result region may hold any bytes between calls.
 * `scratch` must be a device pointer, 16-byte aligned.
 */
argr_status argreduce_scratch_init(void* scratch, size_t scratch_bytes, argr_stream stream);

/*
 * Row-wise ArgMax (op = ARGR_MAX) or ArgMin (ARGR_MIN) of x[rows, cols]
 * (onnxruntime #32092, Approach: one int64 index per row of the last axis,
 * chosen by a planner among thread-per-row, block-per-row and multi-block
 * kernels; Semantics: the sequential first-occurrence scan, bit for bit).
 *
 *   x         device pointer to rows*cols elements of `dtype`, row-major and
 *             contiguous (row r starts at element r*cols). Any address that is
 *             a multiple of the element size; unaligned row starts are handled.
 *   rows      >= 0. rows == 0 returns ARGR_OK and launches nothing.
 *   cols      1 .. INT32_MAX (the index is computed in 32 bits within a row).
 *   out_idx   device pointer to rows int64 values (written).
 *   out_val   NULL, or a device pointer to rows elements of `dtype`, aligned to
 *             the element size; receives the raw bits of x[r, out_idx[r]]
 *             (NaN payloads and the sign of zero preserved).
 *   scratch   device pointer prepared by argreduce_scratch_init(), 16-byte
 *             aligned, at least argreduce_scratch_bytes() bytes; may be NULL
 *             when that is 0. Owned by the caller. Two calls that may run at
 *             the same time on the GPU must not share a scratch buffer.
 *   stream    CUDA stream the kernel is queued on.
 *
 * All validation happens before any launch: on an error status nothing was
 * queued. The call does not synchronise; kernel faults surface on the stream.
 * No per-call allocation, memset or host synchronisation, so the call can be
 * captured into a CUDA graph (as long as the same scratch stays alive).
 */
argr_status argreduce(const void* x, argr_dtype dtype, int64_t rows, int64_t cols, argr_op op,
                      int64_t* out_idx, void* out_val, void* scratch, size_t scratch_bytes,
                      argr_stream stream);

/*
 * Query the planner. caps == NULL uses the current device (one query per
 * device, cached); a non-NULL caps plans for those properties instead, which
 * lets tests force geometries of other device sizes (#32092 Testing: fuzz
 * repeated with several simulated device capacities). Pure host code when
 * caps is given: needs no GPU.
 */
argr_status argreduce_plan(int64_t rows, int64_t cols, argr_dtype dtype, argr_op op,
                           const argr_caps* caps, argr_plan* out);

/*
 * argreduce() with an explicit plan (tests and benchmarks force each path
 * with it). The plan is checked against the problem and the device: an
 * impossible plan returns ARGR_EINVAL (or ARGR_EUNSUPPORTED for a cluster the
 * device cannot launch) before anything is queued. Scratch must be at least
 * plan->scratch_bytes as recomputed for the problem.
 */
argr_status argreduce_with_plan(const argr_plan* plan, const void* x, argr_dtype dtype, int64_t rows,
                                int64_t cols, argr_op op, int64_t* out_idx, void* out_val, void* scratch,
                                size_t scratch_bytes, argr_stream stream);

/*
 * The checks argreduce_with_plan() applies to a plan, against the given device
 * properties instead of the current device's: path, CTA size, lanes per row,
 * loads in flight, flags (each only on the paths it applies to), grid limits
 * and the cluster size (ARGR_EUNSUPPORTED above caps->max_cluster). Covers the
 * last-axis paths (NONE, ROWS, SPLIT, CLUSTER, STREAM). rows_aligned != 0 says
 * every row of the input starts on a 16-byte boundary (vector loads allowed).
 * Returns ARGR_OK, ARGR_EINVAL or ARGR_EUNSUPPORTED as argreduce_with_plan()
 * would; pure host code (#32092 Testing: every dispatch path, simulated device
 * capacities), so forced plans can be checked without a GPU.
 */
argr_status argreduce_plan_check(const argr_plan* plan, int64_t rows, int64_t cols, argr_dtype dtype,
                                 const argr_caps* caps, int rows_aligned);

/*
 * ArgMax / ArgMin over a non-last axis: x is row-major [outer, reduce, inner]
 * and the result is out_idx[outer, inner] (int64, the position along the
 * reduced axis), out_val[outer, inner] optional. Element (o, r, i) is at
 * x[(o * reduce + r) * inner + i]; each output applies exactly the rules of
 * argreduce() to the `reduce` elements x[o, 0..reduce-1, i], which lie
 * `inner` elements apart. With inner == 1 this is argreduce() on
 * [outer, reduce]. Needs no scratch unless inner == 1 and the last-axis plan
 * does (pass scratch as for argreduce(); argreduce_scratch_bytes(outer,
 * reduce, ...) sizes it). Errors as for argreduce(); ARGR_EUNSUPPORTED if
 * inner needs more than 65535 column tiles of 32 lanes.
 */
argr_status argreduce_axis(const void* x, argr_dtype dtype, int64_t outer, int64_t reduce, int64_t inner,
                           argr_op op, int64_t* out_idx, void* out_val, void* scratch, size_t scratch_bytes,
                           argr_stream stream);

/* The planner for argreduce_axis() (a last-axis plan when inner == 1). */
argr_status argreduce_axis_plan(int64_t outer, int64_t reduce, int64_t inner, argr_dtype dtype, argr_op op,
                                const argr_caps* caps, argr_plan* out);

/* argreduce_axis() with an explicit plan (re-validated; an ARGR_PATH_AXIS
 * plan for any inner, a last-axis plan only for inner == 1). */
argr_status argreduce_axis_with_plan(const argr_plan* plan, const void* x, argr_dtype dtype, int64_t outer,
                                     int64_t reduce, int64_t inner, argr_op op, int64_t* out_idx, void* out_val,
                                     void* scratch, size_t scratch_bytes, argr_stream stream);

/*
 * cummax / cummin with indices along the last axis of x[rows, cols]
 * (op = ARGR_MAX or ARGR_MIN; the *_LAST ops return ARGR_EUNSUPPORTED).
 * For every position j of every row: out_idx[r * cols + j] is the row's
 * ArgMax (ArgMin) over x[r, 0..j] by the rules of argreduce() (ties keep the
 * earlier index; a NaN after x[r, 0] is never chosen; a leading NaN gives 0
 * everywhere), and out_val[r * cols + j] (optional) the raw bits of that
 * element. So out_idx[r * cols + cols - 1] equals argreduce()'s result.
 * Element types: the four floating types and ARGR_I32 / ARGR_I64 (compared
 * as integers). Paddle issue #79670 ("Possible fixes": a scan with argmax
 * semantics where ties take the earlier index, and a two-pass tiled scan when
 * the rows alone do not fill the GPU). out_idx holds rows * cols int64.
 * Scratch: argreduce_cum_scratch_bytes() bytes (0 when the plan needs none;
 * then scratch may be NULL), prepared once by argreduce_scratch_init(); the
 * same buffer may serve argreduce() calls that do not run at the same time.
 * Errors as for argreduce().
 */
argr_status argreduce_cum(const void* x, argr_dtype dtype, int64_t rows, int64_t cols, argr_op op, int64_t* out_idx,
                          void* out_val, void* scratch, size_t scratch_bytes, argr_stream stream);

/* Scratch bytes argreduce_cum() needs for this problem on the current device
 * (0 = none). */
size_t argreduce_cum_scratch_bytes(int64_t rows, int64_t cols, argr_dtype dtype, argr_op op);

/* The planner for argreduce_cum(). */
argr_status argreduce_cum_plan(int64_t rows, int64_t cols, argr_dtype dtype, argr_op op, const argr_caps* caps,
                               argr_plan* out);

/* argreduce_cum() with an explicit ARGR_PATH_CUM, ARGR_PATH_CUM_SPLIT or
 * ARGR_PATH_CUM_STREAM plan (re-validated). */
argr_status argreduce_cum_with_plan(const argr_plan* plan, const void* x, argr_dtype dtype, int64_t rows,
                                    int64_t cols, argr_op op, int64_t* out_idx, void* out_val, void* scratch,
                                    size_t scratch_bytes, argr_stream stream);

/* Scratch bytes a given plan needs for `rows` rows. */
size_t argreduce_plan_scratch_bytes(const argr_plan* plan, int64_t rows);

/*
 * Failure reporting for the bounded device-side waits (onnxruntime #32092,
 * Testing: forced dispatch paths must neither hang nor silently corrupt; the
 * scan's waits follow Paddle issue #79670, "Possible fixes", whose two-pass
 * scan hands chunk totals from one CTA to the next).
 * Synchronise `stream` and read the library's device error words (set by a
 * kernel whose bounded wait expired: for a bulk copy, after which the kernel
 * skips the rest of its work, or for another CTA's chunk record in the split
 * or streaming scan) and the one in `scratch` (may be NULL). Returns
 * ARGR_ESCRATCH if a split or streaming scan found counters or records its
 * launch did not write (a scratch buffer that argreduce_scratch_init() never
 * prepared), else ARGR_ETIMEOUT if
 * any word was set, ARGR_OK otherwise (the words are cleared), and ARGR_ECUDA
 * if the stream reports a fault. For tests and benchmarks; it blocks the host.
 */
argr_status argreduce_read_error(void* scratch, argr_stream stream);

/*
 * argreduce() for callers that cannot allocate device memory. The paper has
 * no counterpart to this entry point: it exists for code that runs where
 * cudaMalloc is not available to it, for example a plugin inside an inference
 * engine that owns every device allocation and hands it no allocator, a
 * real-time path that may not make a call that can synchronise the device or
 * block for an unbounded time, or code that must not grow its memory use
 * after start-up.
 *
 * It runs the split-row kernel (a row spread over CTAs of the whole device,
 * merged by the CTA that arrives last) with its scratch in a 32 KiB array
 * inside this library instead of caller memory. That array exists once per
 * GPU, on every GPU that loads the library, until the process exits. The
 * caller still passes x, out_idx and out_val exactly as for argreduce();
 * there is no scratch argument. The call allocates and frees nothing.
 *
 *   - The first call on each device (with that device current) finds the
 *     array's device address and zeroes it, synchronously. Make that first
 *     call before capturing any stream on the device. The address is kept
 *     for the device's primary context: after cudaDeviceReset(), or with a
 *     context other than the primary one current, it is stale, so do not
 *     call this entry point there.
 *   - Every call reuses the same array, which keeps what the last call left:
 *     two calls that can overlap on the GPU (other streams, other host
 *     threads) race on it and give wrong results; serialise them. No call
 *     clears it: each row's arrival counter is bumped with a wrapping
 *     increment that leaves it at zero when the row's last CTA arrives, and
 *     every partial is written before it is read.
 *   - A problem whose plan needs more than the array holds returns
 *     ARGR_ESCRATCH before anything is queued (on a GB300 every shape fits).
 *   - Other errors as for argreduce(), checked before anything is queued:
 *     ARGR_EUNSUPPORTED for the integer types, ARGR_EINVAL for the rest.
 */
argr_status argreduce_noalloc(const void* x, argr_dtype dtype, int64_t rows, int64_t cols, argr_op op,
                              int64_t* out_idx, void* out_val, argr_stream stream);

/*
 * Vocabulary rows: log probabilities, entropy and top alternatives of rows of
 * logits, a distillation loss from a teacher's top logits, and the gradients
 * of both with respect to the logits.
 *
 * x is [rows, cols] logits of type ARGR_F32, ARGR_F16 or ARGR_BF16 (other
 * types: ARGR_EUNSUPPORTED), row r at element r * row_stride (row_stride >= 0;
 * 0 reads the same row for every r). Element-aligned addresses suffice.
 * Exponentials, sums and statistics are binary32 throughout. With
 *     z = x / temperature,  m = max x,  s = sum_j exp((x_j - m) / temperature),
 *     lse = m / temperature + ln s,  p = exp(z - lse):
 *
 *   - A logit of -inf has p = 0 and adds nothing to any sum. A row of -inf
 *     alone is empty: lse = -inf, every log p = -inf, entropy 0, gradient 0.
 *   - A row with a NaN or +inf has NaN log probabilities, loss and gradients.
 *   - A token (slot id) < 0 names nothing: the position has no token (the
 *     slot is empty). One >= cols is a mistake that the host cannot see: the
 *     row's log probability (loss) and gradient become NaN, and nothing is
 *     read or written outside the row.
 *
 * temperature must be positive and finite, and so must log2(e) / temperature.
 * Results do not depend on timing: no floating-point atomics are used (but see
 * the distillation's ids).
 */

/* The operators, for argreduce_logits_plan(). */
typedef enum {
    ARGR_LOGITS_LOGPROBS = 0,
    ARGR_LOGITS_LOGPROBS_GRAD = 1,
    ARGR_LOGITS_DISTILL = 2,
    ARGR_LOGITS_DISTILL_GRAD = 3,
    ARGR_LOGITS_DISTILL_STEP = 4
} argr_logits_op;

#define ARGR_LOGITS_MAX_TOP 128    /* top alternatives of a row, at most */
#define ARGR_LOGITS_MAX_SLOTS 1024 /* distillation slots of a row, at most */

/*
 * For each row: logprob = log p of tokens[r] (0 where tokens[r] < 0), entropy =
 * -sum_j p_j log p_j, lse, and the top_k largest logits in descending order,
 * ties to the lowest index, NaNs after every number: their indices and their
 * log p. Any output may be NULL (top_ids and top_logprobs also separately);
 * tokens may be NULL when logprob is. stats receives 4 floats per row,
 * {m, ln s, entropy, 0}: what argreduce_logprobs_backward() needs (an empty
 * row: {-inf, -inf, 0, 0}). 0 <= top_k <= min(cols, ARGR_LOGITS_MAX_TOP).
 * plan: NULL for the planner's. Errors as for argreduce(); stats 16-byte
 * aligned.
 */
argr_status argreduce_logprobs(const void* x, argr_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                               float temperature, const int64_t* tokens, int32_t top_k, float* logprob,
                               float* entropy, float* lse, int64_t* top_ids, float* top_logprobs, float* stats,
                               const argr_plan* plan, argr_stream stream);

/*
 * The gradient of sum_r (g * logprob + h * entropy + c * lse) with respect to x:
 *     grad[r, j] = (g ([j == token] - p_j) - h p_j (log p_j + entropy) + c p_j) / temperature
 * g = grad_logprob[r] (0 where the row has no token), h = grad_entropy[r], c =
 * grad_lse[r]; each may be NULL (zeros). stats: as argreduce_logprobs() wrote
 * it for the same x and temperature. grad has x's type, rows grad_stride
 * elements apart (>= cols); rounded once from binary32. It may be x itself
 * (same pointer and stride) but must not overlap x otherwise: ARGR_EINVAL.
 */
argr_status argreduce_logprobs_backward(const void* x, argr_dtype dtype, int64_t rows, int64_t cols,
                                        int64_t row_stride, float temperature, const int64_t* tokens,
                                        const float* stats, const float* grad_logprob, const float* grad_entropy,
                                        const float* grad_lse, void* grad, int64_t grad_stride,
                                        const argr_plan* plan, argr_stream stream);

/*
 * Distillation of a student (x) from a teacher's top logits. ids[rows, slots]
 * name distinct indices of the row (negative: an empty slot; give places that
 * are left over a negative id, not an index with teacher -inf), teacher[rows,
 * slots] holds the teacher's value for each. An index that a row names several
 * times is a mistake that the host cannot see: with a tail the row's sum counts
 * it as often, and its gradient is that of one of its slots, which one is a
 * matter of timing. Nothing outside the row is read or written.
 *   tail == 0: q = softmax of teacher / temperature over the row's filled slots;
 *              loss = sum_i q_i (ln q_i - ln p_{id_i}).
 *   tail != 0: q_i = exp(teacher_i): teacher holds log probabilities (taken at
 *              the same temperature). What is left, rest = max(0, 1 - sum q),
 *              is one more outcome: loss = sum_i q_i (ln q_i - ln p_{id_i}) +
 *              rest (ln rest - ln p_rest), p_rest being the student's probability
 *              of every index no slot names, summed over those indices (not
 *              taken as a difference from 1) and kept as a logarithm. The last term
 *              is left out where p_rest = 0, that is below e^-745, as in binary64
 *              (a tail masked by the type's lowest value).
 * A slot with q = 0 adds nothing; one with q > 0 and p = 0 makes the loss
 * +inf. A row without a filled slot (tail == 0: or with teacher -inf in all of
 * them) has loss 0 and gradient 0. stats receives
 * 4 floats per row, {m, ln s, ln s_rest, 0}, s_rest = the part of s over the
 * indices that no slot names (ln s where tail == 0, -inf where p_rest = 0): what
 * argreduce_distill_backward() needs. 0 <= slots <= ARGR_LOGITS_MAX_SLOTS.
 */
argr_status argreduce_distill(const void* x, argr_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                              float temperature, const int64_t* ids, const float* teacher, int32_t slots, int tail,
                              float* loss, float* stats, const argr_plan* plan, argr_stream stream);

/*
 * The gradient of sum_r grad_loss[r] * loss[r] with respect to x:
 *     grad[r, j] = grad_loss / temperature * ((sum q + rest) p_j - q_j          where a slot names j,
 *                                             (sum q + rest) p_j - rest p_j / p_rest  elsewhere).
 * stats from argreduce_distill() with the same arguments; grad as in
 * argreduce_logprobs_backward().
 */
argr_status argreduce_distill_backward(const void* x, argr_dtype dtype, int64_t rows, int64_t cols,
                                       int64_t row_stride, float temperature, const int64_t* ids,
                                       const float* teacher, int32_t slots, int tail, const float* stats,
                                       const float* grad_loss, void* grad, int64_t grad_stride,
                                       const argr_plan* plan, argr_stream stream);

/*
 * Both in one call, for a training step that knows each row's weight
 * (grad_loss) before the loss: loss, stats and grad as the two calls above
 * would give them.
 */
argr_status argreduce_distill_step(const void* x, argr_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                   float temperature, const int64_t* ids, const float* teacher, int32_t slots,
                                   int tail, const float* grad_loss, float* loss, float* stats, void* grad,
                                   int64_t grad_stride, const argr_plan* plan, argr_stream stream);

/* The planner of these operators. k: top_k or slots. caps as for argreduce_plan(). */
argr_status argreduce_logits_plan(argr_logits_op what, int64_t rows, int64_t cols, argr_dtype dtype, int32_t k,
                                  const argr_caps* caps, argr_plan* out);

/*
 * Beam search: the step from the totals of an item's beams and their logits to
 * the best continuations, and the reordering of what the beams keep.
 *
 * x is [items * beams, cols] logits as above (row r of item r / beams), scores[items,
 * beams] the totals so far. A continuation (b, v) of an item has the total
 *     scores[b] + x_bv / temperature - lse_b
 * (lse_b as above), a beam with ended[b] != 0 only one, (b, end_token), with the
 * total scores[b]. The `count` continuations of the largest scale[b] * total come out, the
 * first of them first, ties to the lowest (b, v): tokens, parents (the beam b in
 * [0, beams)) and totals, [items, count] each. ended and scale may be NULL (none
 * has ended; 1).
 *   - Only totals above -inf count. Places that none is left for get token -1,
 *     parent -1 and total -inf.
 *   - A beam with the total -inf has not begun (or is over): it has no
 *     continuation. Its logits are not looked at, nor are those of ended beams.
 *   - An item with a total that is NaN or +inf, a scale (of a beam above -inf) that is
 *     not positive and finite, or a NaN or +inf among the logits it looks at
 *     gets tokens and parents -1 and totals NaN.
 * Totals are formed in binary64 and rounded once (one below binary32's range keeps its place by its
 * rank and comes out as -inf, with its token and parent); lse_b's sum is binary32, so
 * continuations of different beams whose totals differ by less than about 1e-6
 * may come in either order (and equal ones, where the beams' rows do not begin
 * at the same place between two 32-byte boundaries). Within a beam the order is exact.
 * 1 <= beams <= ARGR_BEAM_MAX_BEAMS, items < 2^25, 1 <= count <= ARGR_LOGITS_MAX_TOP. Steps of many
 * rows, and those whose clusters the device has no place for, need scratch
 * (argreduce_beam_scratch_bytes() for the current device, 0 for the others; 16-byte aligned, no
 * preparation), which belongs to the call until it has finished on the stream. Errors as
 * for argreduce_logprobs(); ARGR_ESCRATCH.
 */
#define ARGR_BEAM_MAX_BEAMS 64
argr_status argreduce_beam_select(const void* x, argr_dtype dtype, int64_t items, int32_t beams, int64_t cols,
                                  int64_t row_stride, float temperature, const float* scores, const uint8_t* ended,
                                  int64_t end_token, const float* scale, int32_t count, int64_t* tokens,
                                  int64_t* parents, float* out_scores, void* scratch, size_t scratch_bytes,
                                  argr_stream stream);
size_t argreduce_beam_scratch_bytes(int64_t items, int32_t beams, int64_t cols, argr_dtype dtype, int32_t count);

/*
 * Beam j of item i takes over what beam parents[i * beams + j] kept, in each of the
 * `n_states` states (an array in host memory of device pointers, read during the
 * call), in place. Beam j's part of item i's state lies at i * item_stride + j *
 * beam_stride (strides in bytes): `outer` segments, outer_stride apart, of `positions` *
 * position_bytes contiguous bytes. Only the first lengths[i] positions (NULL:
 * all; clamped to [0, positions]) of each segment change.
 *   - A parent outside [0, beams) names nothing: the beam keeps its own state.
 *   - Several beams may have the same parent, and beams may exchange places.
 * No state may overlap itself (its dimensions have to nest: no stride smaller than what lies within it),
 * another one, parents or lengths: ARGR_EINVAL. At most ARGR_REORDER_MAX_STATES of them.
 * argreduce_beam_reorder_check() makes these checks alone, before the first of several calls.
 */
#define ARGR_REORDER_MAX_STATES 1024
argr_status argreduce_beam_reorder(void* const* states, int32_t n_states, int64_t items, int32_t beams,
                                   int64_t item_stride, int64_t beam_stride, int64_t outer, int64_t outer_stride,
                                   int64_t positions, int64_t position_bytes, const int64_t* parents,
                                   const int64_t* lengths, argr_stream stream);
argr_status argreduce_beam_reorder_check(void* const* states, int32_t n_states, int64_t items, int32_t beams,
                                         int64_t item_stride, int64_t beam_stride, int64_t outer, int64_t outer_stride,
                                         int64_t positions, int64_t position_bytes, const int64_t* parents,
                                         const int64_t* lengths);

/*
 * A router's choice of experts. x is [rows, experts] logits (types, strides and
 * arithmetic as for the vocabulary rows, temperature 1). For each row: ids, the top_k
 * largest logits' indices in descending order, ties to the lowest index; their
 * weights, p at the ids, divided by their sum where normalize != 0; lse. What is not
 * above -inf is not chosen: id -1, weight 0. A row with valid[r] == 0 (valid may
 * be NULL) is padding: it is not looked at; it and a row of -inf alone get ids -1, weights 0,
 * lse -inf and take part in nothing below. A row with a NaN or +inf has NaN weights and
 * lse (NaNs are not chosen) and makes the loss NaN.
 *   counts[e]  how many rows chose expert e
 *   taken      N, how many rows take part (one value)
 *   balance    experts * sum_e (counts[e] / (top_k N)) * (sum of p_e over the rows / N);
 *              1 when all is even, 0 when N = 0 (one value)
 * counts and taken may be NULL together, balance always; balance needs counts. For many
 * rows they need scratch (argreduce_route_scratch_bytes(), 0 for the others; 16-byte aligned, no
 * preparation), which belongs to the call until it has finished on the stream.
 * 1 <= experts <= ARGR_ROUTE_MAX_EXPERTS, 1 <= top_k <= min(experts, ARGR_ROUTE_MAX_TOP).
 * Results do not depend on timing.
 */
#define ARGR_ROUTE_MAX_EXPERTS 1024
#define ARGR_ROUTE_MAX_TOP 32
size_t argreduce_route_scratch_bytes(int64_t rows, int64_t experts);
argr_status argreduce_route(const void* x, argr_dtype dtype, int64_t rows, int64_t experts, int64_t row_stride,
                            int32_t top_k, int normalize, const uint8_t* valid, float* weights, int64_t* ids,
                            float* lse, int64_t* counts, int64_t* taken, float* balance, void* scratch,
                            size_t scratch_bytes, argr_stream stream);

/*
 * The gradient of sum(grad_weights * weights) + sum(grad_lse * lse) + grad_balance *
 * balance with respect to x, choice and counts held fixed; each of the three may be NULL (zero). ids,
 * weights, lse, counts and taken as argreduce_route() wrote them for the same x
 * (ids and weights are needed with grad_weights, counts and taken with
 * grad_balance). Rows with lse -inf are not looked at and get 0; p is divided by the
 * row's own sum, so it is as exact far from zero as near it. grad as in
 * argreduce_logprobs_backward().
 */
argr_status argreduce_route_backward(const void* x, argr_dtype dtype, int64_t rows, int64_t experts,
                                     int64_t row_stride, int32_t top_k, int normalize, const float* weights,
                                     const int64_t* ids, const float* lse, const int64_t* counts,
                                     const int64_t* taken, const float* grad_weights, const float* grad_lse,
                                     const float* grad_balance, void* grad, int64_t grad_stride, argr_stream stream);

/* Properties of `device` as the planner sees them (queried once, cached). */
argr_status argreduce_device_caps(int device, argr_caps* out);

/* Static, human-readable name of a status code. */
const char* argreduce_status_string(argr_status status);

/* Build identification: "argreduce <version> sm_103a". */
const char* argreduce_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ARGREDUCE_H */
