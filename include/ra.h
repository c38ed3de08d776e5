/*
 * ra.h -- C ABI of the ring all-reduce library (libra.so) for one MI355X (gfx950).
 *
 * The library runs the ring all-reduce chunk schedule over p "virtual ranks"
 * whose buffers all live in the HBM of one GPU.  Sources, by page and section:
 *
 *   [InDepth]   "Ring All-Reduce, in depth: the chunk schedule step by step, a
 *               working implementation, pipelining, multi-ring and hierarchical
 *               variants" (aicassindra.com)
 *   [Derive]    "Derive the cost of a ring all-reduce" (aiinfrainterviews.com)
 *   [Deepinsea] "AllReduce 与 Ring 通信算法详解" (deepinsea.top)
 *
 * Conventions shared by the all-reduce entry points (the row operators at the end
 * of this file state their own)
 * ---------------------------------------
 *  bufs    host array of p device pointers, one buffer per rank.  The array is
 *          read during the call only and never retained.  Every buffer holds n
 *          contiguous elements of `dtype`, starts on a 16-byte boundary and
 *          must not overlap another.  The caller owns the buffers and keeps
 *          them alive until the stream work completes.
 *  n       elements per rank (int64; buffers beyond 2^32 elements are fine).
 *  dtype   RA_INT32, RA_FLOAT32, RA_BFLOAT16, RA_FLOAT16, RA_FLOAT64 or RA_INT64.
 *  op      RA_SUM, RA_MAX or RA_AVG ([Deepinsea] "AllReduce 语义": sum, average,
 *          maximum).  RA_AVG (floating-point types only) divides every rank's
 *          contribution by p, rounded to the element type, before it enters
 *          the sum ([InDepth] "Failure modes": pre-divide so that fp16 sums over
 *          many ranks do not overflow); the divided terms are then summed in
 *          exactly the order and rounding of RA_SUM.  RA_MAX is exact: a NaN
 *          operand gives the type's canonical quiet NaN and +0 counts as larger
 *          than -0 (IEEE 754-2019 maximum), so every algorithm gives the same bits.
 *  stream  HIP stream the work is enqueued on.  Calls return as soon as the
 *          work is enqueued.  Argument errors are reported synchronously by
 *          the return value, before anything is enqueued; errors that happen
 *          on the device (a wait that timed out) are sticky per stream and are
 *          reported by ra_stream_status().
 *  In place: results overwrite the inputs.  p == 1 or n == 0 is a no-op that
 *  returns RA_OK ([InDepth] "An implementation": a world of one returns at once).
 *  Rounding: every hop's sum is rounded to the buffer type (integers wrap
 *  modulo 2^32 or 2^64, floats round to nearest even), which is how an in-place
 *  add in the buffer's dtype accumulates ([InDepth] "An implementation";
 *  [Derive] "What interviewers probe next").  RA_FLAG_WIDE_ACCUM asks for the
 *  other remedy of [InDepth] "Failure modes": accumulate in a wider type.
 *  Concurrency: calls on different streams may overlap; calls on one stream
 *  are ordered by the stream.  The library keeps a small device workspace per
 *  (device, stream), allocated on first use and kept until process exit.  The
 *  flag-driven pipelined and channel algorithms, and the step algorithms when
 *  ra_options.grid or step_ts is set, run persistent grids: ordinary launches
 *  whose workgroups wait for each other, so all of them must be resident at
 *  once.  Such a grid is sized to what the GPU can hold of it (by default 3
 *  workgroups of 256 threads per compute unit -- or, for the step algorithms
 *  on 4 MiB to 256 MiB per rank, 2 of 512 or 1 of 1024 threads, so that fewer
 *  workgroups wait at each barrier -- and 4 for RING_PIPELINED_FLAGS, whose
 *  LDS stages allow no more), so overlapping such calls should each set
 *  ra_options.grid (in 256-thread workgroups) to their share; a call that
 *  cannot get all its workgroups resident times out (RA_ERR_TIMEOUT from
 *  ra_stream_status) instead of hanging.
 *
 *  HIP graphs.  The one-pass algorithms (FUSED, HIER_FUSED), the pipelined ring
 *  (RING_PIPELINED) and the step algorithms' default launches (one per step,
 *  or one workgroup) are grids with no device-side waits and no workspace, and
 *  can be captured on any stream.  Calls that run persistent grids can be
 *  captured on a stream that has made such a call before (its workspace is
 *  allocated then, and cannot be during capture: RA_ERR_UNSUPPORTED); their
 *  counters are reset by kernels that the graph holds, and a captured
 *  RING_PIPELINED_FLAGS call numbers its ready counters from 0 after zeroing
 *  them, so replays and eager calls may alternate on the stream.  A replay uses
 *  the capturing stream's workspace: it must not overlap other calls of that
 *  stream.
 *
 * Return codes are ra_status values; ra_status_string() names them and
 * ra_last_error() gives the calling thread's last error message.
 */
#ifndef RA_H
#define RA_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RA_MAX_RANKS 64

typedef enum ra_status {
  RA_OK = 0,
  RA_ERR_INVALID_ARG = 1,  /* p < 1, n < 0, NULL pointer (buffers may be NULL when n == 0),
                              unknown enum value */
  RA_ERR_UNSUPPORTED = 2,  /* p > RA_MAX_RANKS, unknown op, RA_AVG on an integer type, algo or
                              flag not valid for the call */
  RA_ERR_ALIAS = 3,        /* two rank buffers overlap */
  RA_ERR_MISALIGNED = 4,   /* a buffer does not start on a 16-byte boundary (row operators: on a
                              boundary of its elements) */
  RA_ERR_HIP = 5,          /* a HIP runtime call failed (see ra_last_error) */
  RA_ERR_TIMEOUT = 6       /* a device-side wait exceeded its time budget */
} ra_status;

typedef enum ra_dtype {
  RA_INT32 = 0, RA_FLOAT32 = 1, RA_BFLOAT16 = 2, RA_FLOAT16 = 3, RA_FLOAT64 = 4, RA_INT64 = 5,
  RA_FLOAT8_E4M3 = 6   /* outputs of ra_allreduce_rmsnorm only: 8 bits, 4 of exponent, no infinities */
} ra_dtype;

typedef enum ra_op { RA_SUM = 0, RA_MAX = 1, RA_AVG = 2 } ra_op;

/* Algorithms.  All ring variants give bit-identical results to the step-by-step
 * schedule; the tree sums in a different order. */
typedef enum ra_algo {
  RA_ALGO_DEFAULT = -1,       /* RA_ALGO_FUSED (all-reduce: overridable with the RA_ALGO
                                 environment variable, by name or number) */
  RA_ALGO_RING_STEP = 0,      /* the 2(p-1) steps one after another.  Steps that move at most
                                 256 16-byte vectors: one workgroup, its own barrier between
                                 steps.  Larger steps: one ordinary launch per step (the
                                 stream orders them), or, when ra_options.grid or step_ts is
                                 set, one persistent grid with a device-wide barrier between
                                 steps.  RING_BIDIR, TREE and HIER run their steps the same
                                 way. */
  RA_ALGO_RING_PIPELINED = 1, /* chunks cut into slices, each carried through all its hops by one
                                 workgroup: no barriers, no flags; the running partial stays in
                                 registers and every hop writes the receiver's partial, so the
                                 all-reduce moves (3p-2)S bytes (p reads, 2(p-1) writes per
                                 element position) and a reduce-scatter leaves the step-by-step
                                 partials */
  RA_ALGO_RING_BIDIR = 2,     /* two counter-rotating rings, each on half of the buffer */
  RA_ALGO_FUSED = 3,          /* one pass: each element folded in its ring order, written to all ranks */
  RA_ALGO_TREE = 4,           /* binomial tree: reduce to rank 0, broadcast back */
  RA_ALGO_RING_CHANNELS = 5,  /* RING_STEP split into independent channels: channel h takes
                                 part h of every chunk and synchronises only with itself */
  RA_ALGO_AUTO = 6,           /* chosen per call by ra_select_algo (all-reduce only) */
  RA_ALGO_HIER = 7,           /* two-level ring on g ranks per node (ra_options.group): in-node
                                 reduce-scatter, cross-node ring all-reduce of each 1/g shard,
                                 in-node all-gather; 2(g-1) + 2(p/g-1) steps */
  RA_ALGO_HIER_FUSED = 8,     /* one pass in the same two-level order (the same bits as HIER) */
  RA_ALGO_RING_PIPELINED_FLAGS = 9 /* chunks cut into slices; workgroups play ranks, and a rank
                                 forwards slice k as soon as its left neighbour's per-slice
                                 ready counter says it has finished slice k (the layout a
                                 ring of GPUs would run); 5(p-1)S bytes */
} ra_algo;

/* ra_options.flags bits */
#define RA_FLAG_FORCE_TIMEOUT 1u  /* test hook: the first device wait expects an
                                     arrival that never comes, so it times out
                                     after timeout_us and every workgroup exits */
#define RA_FLAG_STRESS 4u         /* test hook: every workgroup of the step-by-step and
                                     pipelined kernels sleeps a pseudo-random 0-25 us
                                     before each barrier arrival and each slice hop,
                                     shuffling arrival orders so that a missing fence
                                     or wait shows up as a wrong result */
#define RA_FLAG_RENEW_COUNTERS 8u /* test hook, RING_PIPELINED_FLAGS: before the call the
                                     stream's ready counters are reallocated (fresh zeros)
                                     and the call's counter numbering starts at 2^31, as
                                     after about 16.7 million calls and a larger one */
#define RA_FLAG_PHASES 16u        /* RA_ALGO_FUSED (all-reduce, reduce-scatter, all-gather):
                                     run the pass in read and write phases (see
                                     ra_allreduce_ex) whenever the GPU holds its grid, at
                                     any size and rank count (the result is the same
                                     either way) */
#define RA_FLAG_NO_PHASES 32u     /* RA_ALGO_FUSED: never use the phases (wins over
                                     RA_FLAG_PHASES) */
#define RA_FLAG_WIDE_ACCUM 2u     /* RA_ALGO_FUSED, bfloat16 / float16 / float32 only:
                                     every term is widened exactly to float32
                                     (float64 for float32 buffers), the ring order
                                     is folded there, rounding each hop to the wide
                                     type, and the result is rounded once to the
                                     element type.  RA_AVG divides the widened terms.
                                     Other algorithms or dtypes: RA_ERR_UNSUPPORTED. */

typedef struct ra_options {
  int64_t slice_elems;  /* RING_PIPELINED: elements of a chunk one workgroup carries, in
                           whole 256-vector tiles (rounded up); 0 = one tile (4 KiB).
                           RING_PIPELINED_FLAGS: slice length in elements; 0 = library
                           default (about four slices per worker per hop, at least
                           64 KiB, but at least eight slices per chunk when they can be
                           16 KiB or more), rounded up to whole 128-byte lines; every
                           slice after a chunk's first starts on a line (counted from
                           the buffer's start).  The result does not depend on it. */
  int64_t timeout_us;   /* budget of any single device-side wait; 0 = 10 s */
  int32_t grid;         /* step algorithms (RING_STEP, RING_BIDIR, TREE, HIER): 0 = the
                           library chooses (see RA_ALGO_RING_STEP).  1 with steps of at
                           most 256 vectors: the single workgroup.  Otherwise a value
                           above 0 runs one persistent grid of that many 256-thread
                           workgroups (at most as many as fit the GPU) with a
                           device-wide barrier between steps.  RING_PIPELINED_FLAGS,
                           RING_CHANNELS: an upper bound on the 256-thread workgroups
                           of their persistent grid (the flag ring uses the same number
                           per rank, rounded down to a multiple of 8 when 8 or more
                           fit); 0 = the library's choice (the flag ring 4 per compute
                           unit; channels 3 per compute unit, or 2 of 512 threads from
                           4 MiB per rank and 1 of 1024 threads from 16 MiB to 256 MiB,
                           64 MiB above 16 ranks).  Values above what fits the GPU are
                           cut to that.  Other algorithms ignore it. */
  uint32_t flags;       /* RA_FLAG_* */
  uint64_t* step_ts;    /* optional DEVICE array of (steps + 1) uint64: device wall-clock
                           ticks at kernel start and as each step's barrier releases
                           (RING_STEP, RING_BIDIR, TREE, HIER, RING_CHANNELS: channel 0).
                           Setting it keeps the steps in one launch (one workgroup or a
                           persistent grid).  NULL = not recorded. */
  int32_t channels;     /* RING_CHANNELS: number of channels, 1..64; 0 = automatic (8, one
                           per XCD, when every segment of a channel still gets a
                           workgroup, else 1).  Capped at the number of workgroups.
                           Counts that are multiples of 8 keep each channel on one XCD.
                           Other algorithms ignore it. */
  int32_t group;        /* HIER, HIER_FUSED: ranks per node g, dividing p; 0 = the largest
                           divisor of p that is at most 8.  Other algorithms ignore it. */
  double link_alpha_us; /* AUTO: per-step latency alpha of the link the schedule is priced
                           for, in microseconds; 0 = no link model (see ra_select_algo) */
  double link_GBps;     /* AUTO: per-direction link bandwidth B, in 10^9 bytes/s; 0 = none */
} ra_options;

/*
 * ra_chunk_bounds -- chunk partition of an n-element buffer into p chunks.
 * [InDepth] "An implementation": chunk i starts at i*floor(n/p) + min(i, n mod p),
 * so the first n mod p chunks hold one element more.
 *   starts  host array of p + 1 int64, written: chunk i is [starts[i], starts[i+1]).
 * Pure host code, no GPU needed.  RA_ERR_INVALID_ARG for p < 1, n < 0 or NULL;
 * RA_ERR_UNSUPPORTED for p > RA_MAX_RANKS.
 */
int ra_chunk_bounds(int64_t n, int p, int64_t* starts);

/*
 * ra_reduce_scatter -- the p - 1 reduce-scatter steps ([InDepth] "The schedule";
 * [Deepinsea] "Phase 1: Reduce-Scatter").  Step s: rank r's chunk (r - s) mod p is
 * added into rank r+1's copy of that chunk.  Afterwards rank r's chunk
 * (r + 1) mod p holds the full sum, accumulated in ring order.  What the other
 * chunks hold depends on the algorithm: RING_STEP, RING_PIPELINED,
 * RING_PIPELINED_FLAGS and RING_CHANNELS leave the ring's partial sum of chunk c
 * over ranks c, c+1, ..., r (the step-by-step states; RING_PIPELINED writes them
 * in (2p-1)*S bytes); FUSED (the default) leaves them as they were, and moves
 * (p+1)*S bytes instead of 3(p-1)*S ([InDepth] "Trade-offs": reduce-scatter
 * and all-gather are used on their own by sharded optimisers and FSDP).
 */
int ra_reduce_scatter(void* const* bufs, int p, int64_t n, int dtype, int op,
                      hipStream_t stream);

/*
 * ra_all_gather -- the p - 1 all-gather steps ([InDepth] "The schedule";
 * [Deepinsea] "Phase 2: All-Gather").  Expects the layout ra_reduce_scatter
 * leaves (rank r owns chunk (r + 1) mod p).  Step s: rank r's chunk
 * (r + 1 - s) mod p overwrites rank r+1's copy; afterwards every rank holds every
 * owned chunk.  Only the owned chunks are read, whatever the other chunks hold,
 * so ra_reduce_scatter followed by ra_all_gather equals ra_allreduce for every
 * pairing of the algorithms.  FUSED (the default) moves p*S bytes; calls of 8
 * ranks of at least 12 GiB each run it in read and write phases (see
 * ra_allreduce_ex), sized for 6.35 TB/s.  FUSED reduce-scatters take the phases
 * only when RA_FLAG_PHASES asks (they measured no faster).
 */
int ra_all_gather(void* const* bufs, int p, int64_t n, int dtype, hipStream_t stream);

/*
 * ra_allreduce -- reduce-scatter then all-gather ([InDepth] "The schedule";
 * [Derive] "A strong answer"): every rank ends with the element-wise sum,
 * accumulated in ring order (element i of chunk c summed over ranks
 * c, c+1, ..., c+p-1 mod p, rounding every hop).  Uses RA_ALGO_DEFAULT.
 */
int ra_allreduce(void* const* bufs, int p, int64_t n, int dtype, int op,
                 hipStream_t stream);

/*
 * ra_allreduce_ex -- ra_allreduce with an explicit algorithm and options.
 *   algo  an ra_algo value.  RING_BIDIR: [InDepth] "What real libraries add",
 *         bidirectional rings -- the first ceil(n/2) elements go round the
 *         forward ring, the rest round the mirrored ring (rank r sends to r - 1,
 *         reduce-scatter step s sends chunk (r + s) mod p).  RING_PIPELINED,
 *         RING_PIPELINED_FLAGS: [InDepth] "What real libraries add", pipelining
 *         (a chunk cut into pieces, so that a piece moves on while the next one
 *         is reduced).  TREE: [Derive]
 *         "Where it stops scaling", a binomial tree rooted at rank 0 (reduce
 *         level k adds rank r + 2^k into rank r for r a multiple of 2^(k+1)).
 *         RING_CHANNELS: [InDepth] "What real libraries add", multiple rings or
 *         channels -- the result is the same bits as RING_STEP for any channel count.
 *         HIER, HIER_FUSED: [InDepth] "What real libraries add", hierarchy;
 *         [Deepinsea] "Ring vs Hierarchical".  Rank r = q*g + l is local rank l of
 *         node q.  Element i of chunk c of the g-way partition, in piece d of that
 *         chunk cut p/g ways, is summed over local ranks c, c+1, ... of each node
 *         and those node sums over nodes d, d+1, ..., rounding every hop.  g = 1
 *         and g = p give the flat ring's bits.  A group that does not divide p:
 *         RA_ERR_INVALID_ARG.  RA_FLAG_WIDE_ACCUM is not available here.
 *         FUSED, read and write phases: sum and maximum all-reduces of 8
 *         ranks of at least 12 GiB each (other sizes, rank counts and averages
 *         only when forced) run the same fold on a
 *         resident grid of 8 workgroups per compute unit whose loads and stores
 *         take turns chip-wide, in windows timed by the device's constant clock
 *         and sized for the bytes one round moves at 6.42 TB/s.  The bits are
 *         those of the plain pass.  The windows assume the call has the GPU's
 *         memory to itself: work running beside it on other streams slows
 *         both (RA_FLAG_NO_PHASES turns them off; RA_FLAG_PHASES forces them
 *         for any size).
 *   opt   may be NULL (all defaults).
 */
int ra_allreduce_ex(void* const* bufs, int p, int64_t n, int dtype, int op, int algo,
                    const ra_options* opt, hipStream_t stream);

/* ra_reduce_scatter / ra_all_gather with algo RING_STEP, RING_PIPELINED,
 * RING_PIPELINED_FLAGS, RING_CHANNELS or FUSED and options; other algorithms return RA_ERR_UNSUPPORTED, a channel count
 * outside 0..64 RA_ERR_INVALID_ARG. */
int ra_reduce_scatter_ex(void* const* bufs, int p, int64_t n, int dtype, int op, int algo,
                         const ra_options* opt, hipStream_t stream);
int ra_all_gather_ex(void* const* bufs, int p, int64_t n, int dtype, int algo,
                     const ra_options* opt, hipStream_t stream);

/*
 * ra_stream_status -- waits for `stream`, then returns RA_ERR_TIMEOUT if a
 * device-side wait of an earlier call on it timed out ([InDepth] "Failure
 * modes": a dead or stalled rank must fail fast instead of hanging), else
 * RA_OK (or RA_ERR_HIP if synchronising failed).  A timed-out call leaves its
 * buffers in an unspecified state; calls enqueued after it on the same stream
 * do no work until this function has reported the error, which also clears it.
 */
int ra_stream_status(hipStream_t stream);

/*
 * ra_allreduce_noalloc -- ra_allreduce_ex for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc.  Same arguments, algorithms and results as
 * ra_allreduce_ex; the call allocates nothing.  The device workspace of the
 * persistent grids (barrier words, status word, the flag-driven pipelined
 * ring's ready counters) is a 1 MiB array in the library's own device data,
 * one per GPU, held until the process ends:
 *  - ready counters: at most 253,952 per call (p times the slices per chunk of
 *    RING_PIPELINED_FLAGS); a call that needs more returns RA_ERR_UNSUPPORTED
 *    before enqueueing anything (larger ra_options.slice_elems need fewer);
 *  - the array keeps what the last call left (counters are numbered per call
 *    and reset by a kernel on the calling stream when the numbering wraps);
 *  - every call on a GPU shares that GPU's array, so calls that overlap on one
 *    GPU (on different streams, or from different threads) race;
 *  - a device-side timeout is sticky in the array: later calls on that GPU do
 *    no work until ra_stream_status (on any stream of that GPU) reports it,
 *    which also clears it.
 * The placement probe that lets persistent grids synchronise per XCD needs an
 * allocation; until another call has run it on the device, these calls use
 * device-wide barriers instead (same results).
 */
int ra_allreduce_noalloc(void* const* bufs, int p, int64_t n, int dtype, int op, int algo,
                         const ra_options* opt, hipStream_t stream);

/*
 * ra_select_algo -- the algorithm RA_ALGO_AUTO runs for an all-reduce of p buffers
 * of n elements of `dtype` ([InDepth] "Trade-offs": libraries choose between
 * ring and tree for each call, by the size of the message and the number of
 * ranks; [Derive] "Where it stops scaling": the tree takes over when each
 * rank's share shrinks to some hundreds of kilobytes).
 *   With opt->link_alpha_us > 0 and opt->link_GBps > 0: the pages' cost model for
 *   S = n * element size bytes -- T_ring = 2(p-1) alpha + 2(p-1)/p * S/B
 *   ([Derive] "Where it stops scaling") against T_tree = 2 ceil(log2 p) (alpha + S/B),
 *   each tree step moving the whole buffer -- and RA_ALGO_TREE if the tree is
 *   strictly faster, else RA_ALGO_RING_STEP.  This prices the schedule for the
 *   given link; the chosen algorithm then runs over the p buffers in this GPU.
 *   Otherwise (no link model): RA_ALGO_FUSED.  Over buffers that share one GPU's
 *   memory it moves the least data (2pS bytes), and on MI355X it was the fastest
 *   all-reduce, or tied with the fastest, at every size from 1 KiB to 64 MiB per rank
 *   and every p from 2 to 64 measured: where another algorithm's median beat it (the
 *   slice-carrying pipelined ring, whose partial writes partly merge in the caches),
 *   it did so by 0.1-2 us, mostly at the launch floor (about 6 us per call), and the
 *   sizes where it happened changed from run to run.
 * Writes the ra_algo value to *algo_out.  Host only, no GPU needed.
 * RA_ERR_INVALID_ARG for p < 1, n < 0, an unknown dtype, NULL algo_out, or a
 * negative or non-finite link parameter; RA_ERR_UNSUPPORTED for p > RA_MAX_RANKS.
 */
int ra_select_algo(int p, int64_t n, int dtype, const ra_options* opt, int* algo_out);

/* Static name of a status code ("RA_OK", ...). */
const char* ra_status_string(int code);

/* Message of the calling thread's last failing call ("" if none).  Valid until
 * that thread's next call into the library. */
const char* ra_last_error(void);

/*
 * ra_wallclock_hz -- frequency of the device clock step_ts is stamped with.
 * Writes it to *hz; RA_ERR_HIP if the device cannot be queried.
 */
int ra_wallclock_hz(int64_t* hz);

/*
 * ra_stream_copy -- plain device copy of `bytes` bytes (16-byte aligned
 * pointers, bytes a multiple of 16), one read and one write per byte.  A
 * measurement helper: the streaming ceiling the all-reduce kernels are
 * compared with, and the known-size kernel that HBM byte counters are
 * calibrated against.  Not part of the all-reduce.
 */
int ra_stream_copy(void* dst, const void* src, int64_t bytes, hipStream_t stream);

/*
 * ra_stream_copy_resident -- the same copy on a resident grid of `grid`
 * workgroups (0 = the library's default persistent grid, 3 per compute unit)
 * that loop over 16 KiB tiles, the workgroups of each XCD taking a contiguous
 * range of tiles in order from a tile counter: the way the persistent step
 * kernels take a large step's tiles, and the streaming ceiling they are
 * compared with (on MI355X a resident grid streams slower than a grid that
 * covers the data once).  The counters live in the stream's workspace, which
 * the first call on a stream allocates, as the all-reduce calls do.  Same
 * argument rules as ra_stream_copy; grid < 0 is RA_ERR_INVALID_ARG.  Not part
 * of the all-reduce.
 */
int ra_stream_copy_resident(void* dst, const void* src, int64_t bytes, int grid,
                            hipStream_t stream);

/*
 * Row operators
 * -------------
 * What a transformer whose layers are cut over the p ranks ("tensor parallel")
 * does at the places where it folds the ranks' buffers: the sum of a sublayer's
 * partial outputs goes into the residual stream and its norm, the embedding and
 * the loss have a vocabulary cut over the ranks, and the gradients go the same
 * way back.  Shared by the calls below:
 *
 *  rows    an array of `tokens` x `hidden` is contiguous, one token after the
 *          other.  Arrays start on a boundary of their elements; calls whose
 *          arrays all start on 16-byte boundaries and whose rows have a multiple
 *          of 8 elements run faster kernels, with the same results.
 *  vocabulary  cut over the ranks as ra_chunk_bounds(vocab, p) says.  At most
 *          2^24 columns.  Pieces without a column may be NULL.
 *  dtype   RA_FLOAT32, RA_BFLOAT16 or RA_FLOAT16 (others: RA_ERR_UNSUPPORTED).
 *          Sums, norms and exponentials are computed in float32, and every
 *          output is rounded once, to nearest even.  The ranks' partials are
 *          added in rank order, 0 first, in float32 (not rounded every hop as
 *          ra_allreduce does).
 *  outs    a result that all ranks need: n pointers, each of which gets the whole
 *          result; n = 1 for ranks that share one copy.
 *  results do not depend on the stream, the GPU's load or the call's history:
 *          there are no floating-point atomics.
 *  overlap two arrays of a call may share memory only if neither is written, or
 *          where a call says that one may be exactly the other (RA_ERR_ALIAS).
 *  workspace  device memory of the caller's, 16-byte aligned, whose size the
 *          matching ..._workspace call gives (host only; 0 where none is needed,
 *          then NULL will do).  It is scratch: nothing is kept in it between
 *          calls, and calls that may overlap need one each.  So do HIP graphs
 *          whose replays may overlap.
 *  The calls wait for nothing, allocate nothing and can be captured into HIP
 *  graphs on any stream.  The current device has to be the stream's.
 *  tokens == 0 is RA_OK and writes nothing but what a call says.
 */

/*
 * ra_allreduce_rmsnorm -- the sum over the ranks, added to the residual stream and
 * normalised by its root mean square, to every rank:
 *     h = residual_in + sum_r bufs[r]
 *     y = h / sqrt(mean(h^2) + eps) * weight          (mean over the hidden columns)
 *   bufs          p arrays [tokens][hidden] of `dtype`, read.  p = 1 is a plain norm.
 *   residual_in   [tokens][hidden] of residual_dtype (`dtype` or RA_FLOAT32), or
 *                 NULL for zeros
 *   residual_out  h, rounded to residual_dtype, or NULL.  May be residual_in.  y is
 *                 computed from the unrounded h.
 *   weight        [hidden] of `dtype`
 *   outs          n_out (1..p) arrays for y, of out_dtype: `dtype`, where each may be
 *                 one of bufs (the sum in place, as ra_allreduce leaves it), or
 *                 RA_FLOAT8_E4M3
 *   scales        8-bit outputs: n_out arrays [tokens][ceil(hidden / group)] float32
 *                 (group = 0: [tokens]), else ignored.  y stands for q * scale with
 *                 scale = max(max |y|, 2^-110) / 448 over the group, q = y / scale to
 *                 nearest even.  A group that holds an infinity or a NaN gives NaN.
 *   group         0, 32, 64 or 128 columns to a scale
 *   rstd          1 / sqrt(mean(h^2) + eps), [tokens] float32, or NULL; the backward
 *                 call wants it
 *   eps           > 0 and finite, so that a row of zeros gives zeros
 * hidden is at most 32768.  The squares are float32: rows with |h| beyond 1e19 / sqrt(hidden)
 * overflow, and give zeros.
 */
int ra_allreduce_rmsnorm(void* const* bufs, int p, int64_t tokens, int64_t hidden, int dtype,
                         const void* residual_in, void* residual_out, int residual_dtype,
                         const void* weight, float eps, void* const* outs, int n_out,
                         int out_dtype, float* const* scales, int group, float* rstd,
                         hipStream_t stream);

/*
 * ra_allreduce_rmsnorm_backward -- the gradient of ra_allreduce_rmsnorm:
 *     g = sum_r dys[r],  x = h * rstd
 *     dh = dh_in + rstd * (weight g - x mean(weight g x)),   dweight = sum over tokens of g x
 *   dys      p arrays [tokens][hidden] of `dtype`: the gradients of y, of which each
 *            rank has a part (p = 1: the whole)
 *   h, rstd  what the forward call left in residual_out (h_dtype: `dtype` or
 *            RA_FLOAT32) and rstd
 *   dh_in    the gradient of residual_out that comes along the stream, h_dtype, or NULL
 *   dh       the gradient of residual_in, h_dtype.  May be dh_in.
 *   dxs      n_dx (0..p) arrays of `dtype`: the gradient of the ranks' partials, which
 *            is dh for each of them.  Each may be one of dys.
 *   dweight  [hidden] float32, or NULL.  With tokens == 0 it gets zeros.  Its sum over
 *            the tokens has a fixed order.
 *   workspace  ra_allreduce_rmsnorm_backward_workspace bytes where dweight is wanted
 */
int ra_allreduce_rmsnorm_backward(void* const* dys, int p, int64_t tokens, int64_t hidden,
                                  int dtype, const void* h, int h_dtype, const float* rstd,
                                  const void* weight, const void* dh_in, void* dh,
                                  void* const* dxs, int n_dx, float* dweight, void* workspace,
                                  int64_t workspace_bytes, hipStream_t stream);
int ra_allreduce_rmsnorm_backward_workspace(int64_t tokens, int64_t hidden, int64_t* bytes);

/*
 * ra_cross_entropy -- softmax cross entropy of logits whose vocabulary is cut over
 * the ranks, and its gradient in the same call:
 *     lse = ln sum_j exp(x_j),  loss = lse - x_target
 *     dx_j = grad_scale * dloss * (exp(x_j - lse) - [j = target])
 *   logits   p arrays; rank r's is [tokens][its columns] of `dtype`
 *   valid    1..vocab: columns from `valid` on are padding.  They are not read as
 *            logits, and their gradient is zero.
 *   targets  [tokens] of target_dtype (RA_INT32 or RA_INT64).  Below 0: a token
 *            without a loss (loss 0, gradient zeros whatever its logits hold).  From
 *            `valid` on: NaN for the token's loss and gradient.
 *   loss, lse  [tokens] float32; either may be NULL
 *   grads    p arrays like logits, or NULL for no gradient.  grads[r] may be
 *            logits[r]: then the gradient takes the logits' place and neither they
 *            nor the probabilities are kept.
 *   dloss    [tokens] float32: the gradient of each token's loss; NULL: ones
 * Logits of -inf are masked columns.  A token all of whose columns are -inf has
 * lse = -inf, loss = +inf and a gradient of zeros.  A logit of +inf or NaN makes
 * its token NaN.
 */
int ra_cross_entropy(void* const* logits, int p, int64_t tokens, int64_t vocab, int64_t valid,
                     int dtype, const void* targets, int target_dtype, float* loss, float* lse,
                     void* const* grads, const float* dloss, float grad_scale, void* workspace,
                     int64_t workspace_bytes, hipStream_t stream);
int ra_cross_entropy_workspace(int64_t tokens, int64_t vocab, int p, int64_t* bytes);

/*
 * ra_cross_entropy_backward -- the gradient alone, from the logits and the lse that an
 * earlier ra_cross_entropy gave: for a program that learns dloss only later.
 * Arguments as above; grads[r] may be logits[r].
 */
int ra_cross_entropy_backward(void* const* logits, int p, int64_t tokens, int64_t vocab,
                              int64_t valid, int dtype, const void* targets, int target_dtype,
                              const float* lse, void* const* grads, const float* dloss,
                              float grad_scale, hipStream_t stream);

/*
 * ra_embedding -- rows of a table whose vocabulary is cut over the ranks, to every
 * rank: y_t = scale * table[id_t].  (Each rank looking up its own rows, zeros for
 * the others, and an all-reduce give the same.)
 *   tables   p arrays; rank r's is [its rows][hidden] of `dtype`
 *   ids      [tokens] of id_dtype (RA_INT32 or RA_INT64).  Below 0: padding, a row of
 *            zeros.  From vocab on: a row of NaN.
 *   outs     n_out (1..p) arrays [tokens][hidden] of `dtype`
 * hidden is at most 2^20.
 */
int ra_embedding(const void* const* tables, int p, int64_t vocab, int64_t hidden, int dtype,
                 const void* ids, int id_dtype, int64_t tokens, float scale, void* const* outs,
                 int n_out, hipStream_t stream);

/*
 * ra_embedding_backward -- the gradient of the tables: dtable[v] = scale * the sum of dy
 * over the tokens with id v, added up in an order that the ids alone decide.
 *   dy       [tokens][hidden] of `dtype`
 *   dtables  p arrays like the tables, of dtable_dtype (`dtype` or RA_FLOAT32)
 *   accumulate  0: every row is written, zeros where no token has it (with tokens ==
 *            0 too).  1: the rows that tokens have are added to, others left alone.
 *   ids outside 0..vocab-1 have no row and are ignored
 *   workspace  ra_embedding_backward_workspace bytes
 * One call takes fewer than 2^31 - 4096 tokens, and at most
 *     ceil(tokens / 16) * ceil(hidden / 512) + ceil(vocab / 8)  <=  2^24 - 1
 * (else RA_ERR_UNSUPPORTED, from the workspace call too): some 200 million tokens of 512
 * columns, or 14 million of 8192.  Larger batches go in parts, with accumulate.
 */
int ra_embedding_backward(const void* dy, int64_t tokens, int64_t hidden, int dtype,
                          const void* ids, int id_dtype, float scale, void* const* dtables, int p,
                          int64_t vocab, int dtable_dtype, int accumulate, void* workspace,
                          int64_t workspace_bytes, hipStream_t stream);
int ra_embedding_backward_workspace(int64_t tokens, int64_t vocab, int64_t hidden, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* RA_H */
