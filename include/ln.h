/*
 * ln.h -- C ABI of libln.so: LayerNorm forward and analytical backward on an
 * NVIDIA B200 (sm_100a).
 *
 * The operation.  "llm.c's Origin and the Future of LLM Compilers" (CUDA MODE
 * talk page), chapter "Deconstructing PyTorch Abstractions and Setting
 * Reference Baselines", describes LayerNorm forward and backward written over
 * bare float arrays with no tensor abstraction; "llm.c: Large Language Model
 * Training in Pure C/CUDA Without Dependencies", features "Tensor Memory
 * Layout" (flat 1-D row-major arrays, explicit stride arithmetic) and "Exact
 * Analytical Backward Pass" (hand-derived LayerNorm gradients).  The pages do
 * not print the equations; this library computes the textbook definition:
 *
 *   mean[r] = (1/C) sum_c x[r,c]
 *   rstd[r] = 1 / sqrt((1/C) sum_c (x[r,c] - mean[r])^2 + eps)
 *   out     = (x - mean[r]) * rstd[r] * weight[c] + bias[c]
 *
 *   xhat    = (x - mean[r]) * rstd[r],   g = dout * weight[c]
 *   dinp    = rstd[r] * (g - (1/C) sum_c g - xhat * (1/C) sum_c g * xhat)
 *   dweight = sum over all N rows of dout * xhat
 *   dbias   = sum over all N rows of dout
 *
 * Layout.  Activations (inp, out, dout, dinp) are flat row-major [N * C]
 * arrays: row r starts at element r * C.  weight, bias, dweight and dbias hold
 * C elements, mean and rstd hold N.  All pointers are DEVICE pointers of the
 * current CUDA device, owned by the caller; the library never frees them.
 *
 * Types.  `dtype` (LN_F32, LN_BF16 or LN_F16) is the element type of inp,
 * out, dout, dinp, weight and bias.  mean, rstd, dweight and dbias are always
 * fp32.  Arithmetic is fp32 in registers; bf16 and fp16 results are rounded
 * to nearest-even (fp16 results beyond 65504 become infinite, as rounding
 * requires).  The pages this library follows name fp32 and bf16 kernels;
 * fp16 is the other 16-bit training format and takes the same paths.
 *
 * Semantics shared by every call.
 *   - Asynchronous on `stream` (NULL: the legacy default stream); no host
 *     synchronisation; the library creates no streams of its own.
 *   - Any number of host threads may call at once, each on its own stream:
 *     the library's per-device state and caches are guarded, and results do
 *     not depend on which thread called first (ln_backward_noalloc's shared
 *     array is the one exception; see there).
 *   - Outputs are overwritten, never accumulated into, except where
 *     ln_backward_ex is asked to accumulate.
 *   - Results are deterministic: the same inputs give bitwise-identical
 *     outputs on every call (no floating-point atomics).
 *   - No call works in place: an output must not share a byte with another
 *     output or with an array the call reads (LN_ERR_ALIAS, checked on the
 *     host before anything is launched).  Inputs may overlap one another.
 *     The accumulating backward reads the outputs it adds to; that is the
 *     same array, not an overlap.  One exception: dresid_out of
 *     ln_backward_dropout_residual may be dresid.
 *   - Any alignment is accepted (the dropout calls: of whole elements).  Fully
 *     16-byte-aligned arrays with C * size a multiple of 16 bytes take the
 *     vectorised path, others a scalar path; the dropout calls also take rows
 *     of other lengths on a vectorised path when the [N * C] arrays start on 16
 *     bytes.
 *   - Errors are returned as an ln_status value; nothing is launched when
 *     validation fails, and no kernel asserts or traps.
 *   - ln_forward, ln_forward_residual, ln_backward, ln_backward_ex and the
 *     dropout calls can be captured into a CUDA graph (the backward's workspace then
 *     becomes graph allocation nodes); make one uncaptured call of the same
 *     shape on the device first, so that one-time set-up (the device's memory
 *     pool, kernel attributes) happens outside the capture.
 *   - 1 <= C <= LN_MAX_C; 0 <= N <= LN_MAX_N; N * C <= LN_MAX_ELEMS.
 *     N == 0 launches nothing in the forward; in the backward it only
 *     zero-fills dweight and dbias (pointers other than dweight and dbias
 *     may then be NULL).
 */
#ifndef LN_H
#define LN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared here so that C callers need no CUDA
 * header. */
struct CUstream_st;
typedef struct CUstream_st *ln_stream_t;

#define LN_MAX_C ((int64_t)1 << 24)
#define LN_MAX_N ((int64_t)1 << 40)
#define LN_MAX_ELEMS ((int64_t)1 << 50)   /* bound on N * C */

typedef enum {
    LN_F32 = 0,   /* IEEE binary32 */
    LN_BF16 = 1,  /* bfloat16 (8 significant bits, binary32 exponent range) */
    LN_F16 = 2    /* IEEE binary16 (11 significant bits, largest finite 65504) */
} ln_dtype;

typedef enum {
    LN_OK = 0,
    LN_ERR_NULL = 1,       /* a required pointer is NULL */
    LN_ERR_SHAPE = 2,      /* N < 0, N > LN_MAX_N, C < 1, C > LN_MAX_C or
                              N * C > LN_MAX_ELEMS */
    LN_ERR_DTYPE = 3,      /* dtype is not LN_F32, LN_BF16 or LN_F16 */
    LN_ERR_EPS = 4,        /* eps is not finite, or not > 0 */
    LN_ERR_WORKSPACE = 5,  /* the backward's workspace could not be allocated */
    LN_ERR_CUDA = 6,       /* a CUDA runtime call or launch failed */
    LN_ERR_SCRATCH = 7,    /* ln_backward_noalloc: C > LN_NOALLOC_MAX_C */
    LN_ERR_FLAGS = 8,      /* ln_backward_ex: unknown bits in flags */
    LN_ERR_ALIAS = 9,      /* an output overlaps another output or an array
                              the call reads */
    LN_ERR_PROB = 10,      /* dropout calls: p is not in [0, 1] */
    LN_ERR_ALIGN = 11      /* dropout calls: an array does not lie on a
                              multiple of its element size (step: of 8) */
} ln_status;

/*
 * LayerNorm forward over N rows of C channels.
 *   out   [N*C] dtype, written      normalised, scaled and shifted rows
 *   mean  [N]   fp32,  written      per-row mean
 *   rstd  [N]   fp32,  written      per-row 1/sqrt(var + eps), var biased (1/C)
 *   inp   [N*C] dtype, read
 *   weight, bias [C] dtype, read
 *   eps   finite, > 0 (1e-5 in GPT-2)
 * out, mean and rstd must not overlap one another or inp, weight or bias
 * (LN_ERR_ALIAS).  Returns LN_OK or an ln_status error.
 */
int ln_forward(void *out, float *mean, float *rstd, const void *inp,
               const void *weight, const void *bias, int64_t N, int64_t C,
               float eps, int dtype, ln_stream_t stream);

/*
 * LayerNorm backward for the loss gradient dout, given the statistics that
 * ln_forward saved for the same inp.
 *   dinp    [N*C] dtype, written    gradient w.r.t. inp
 *   dweight [C]   fp32,  written    sum over rows of dout * xhat
 *   dbias   [C]   fp32,  written    sum over rows of dout
 *   dout    [N*C] dtype, read
 *   inp     [N*C] dtype, read
 *   weight  [C]   dtype, read
 *   mean, rstd [N] fp32, read
 * The column sums are formed in two stages with a fixed summation order:
 * per-block partial sums into a library-owned workspace drawn, stream-ordered,
 * from a per-device memory pool (returned to the pool on `stream` after use),
 * then one fixed-order sum of the partials.  dinp, dweight and dbias must
 * not overlap one another or dout, inp, weight, mean or rstd (LN_ERR_ALIAS).
 * Returns LN_OK or an ln_status error (LN_ERR_WORKSPACE when the pool cannot
 * supply the workspace).
 */
int ln_backward(void *dinp, float *dweight, float *dbias, const void *dout,
                const void *inp, const void *weight, const float *mean,
                const float *rstd, int64_t N, int64_t C, int dtype,
                ln_stream_t stream);

/*
 * LayerNorm forward of a residual sum, the step that precedes LayerNorm in a
 * GPT-2 block: "llm.c: Large Language Model Training in Pure C/CUDA Without
 * Dependencies" credits its speed to custom fused kernels (feature list, and
 * the question "Can llm.c achieve competitive training speeds with
 * PyTorch?").  Here the residual add is fused into the forward, so the sum is
 * read from registers instead of being written and read back:
 *   x         = resid + branch, rounded to dtype (each element rounded once,
 *               to nearest-even)
 *   resid_out = x
 *   out, mean, rstd = ln_forward(x)      (the rounded x, so that the saved
 *                                         residual and the statistics agree)
 *   resid_out [N*C] dtype, written       the residual stream after the add
 *   out, mean, rstd                      as in ln_forward
 *   resid, branch [N*C] dtype, read      the two summands
 *   weight, bias [C] dtype, read; eps as in ln_forward
 * resid_out, out, mean and rstd must not overlap one another or any input
 * (no in-place update; LN_ERR_ALIAS).  Bytes moved: 4*N*C*size (two reads, two writes) against 5*N*C*size
 * for a separate add and ln_forward.  Returns LN_OK or an ln_status error.
 */
int ln_forward_residual(void *resid_out, void *out, float *mean, float *rstd,
                        const void *resid, const void *branch, const void *weight,
                        const void *bias, int64_t N, int64_t C, float eps, int dtype,
                        ln_stream_t stream);

/* Flags of ln_backward_ex (bitwise or). */
/* dinp += the gradient: the previous dinp is read and each sum is rounded to
 * dtype once.  For a residual stream, whose gradient is the sum of the
 * branches' gradients ("llm.c: Large Language Model Training in Pure C/CUDA
 * Without Dependencies", question "How does llm.c handle distributed
 * multi-GPU training?": gradients are accumulated locally before they are
 * synchronised). */
#define LN_BWD_ACCUMULATE_DINP 1u
/* dweight += and dbias += the column sums (fp32), e.g. over micro-batches of
 * one optimiser step. */
#define LN_BWD_ACCUMULATE_DPARAMS 2u
/* mean and rstd are recomputed from inp (with eps, exactly as ln_forward
 * computes them) instead of being read; the mean and rstd arguments may then
 * be NULL.  Saves the 8*N bytes of the saved statistics, and lets a caller
 * drop them (activation recomputation). */
#define LN_BWD_RECOMPUTE_STATS 4u

/*
 * ln_backward with variants: flags == 0 is exactly ln_backward (eps is then
 * unused).  Arguments as in ln_backward, plus
 *   eps    finite, > 0; read only with LN_BWD_RECOMPUTE_STATS
 *   flags  a combination of LN_BWD_ACCUMULATE_DINP, LN_BWD_ACCUMULATE_DPARAMS
 *          and LN_BWD_RECOMPUTE_STATS; other bits give LN_ERR_FLAGS
 * With LN_BWD_ACCUMULATE_DINP, dinp is read as well as written (it must hold
 * the previous gradient); with LN_BWD_ACCUMULATE_DPARAMS, dweight and dbias
 * are read and N == 0 leaves them unchanged.  With LN_BWD_RECOMPUTE_STATS
 * mean and rstd are not read, so their overlaps are not checked.  The column
 * sums keep their fixed order, so results stay deterministic.
 */
int ln_backward_ex(void *dinp, float *dweight, float *dbias, const void *dout,
                   const void *inp, const void *weight, const float *mean,
                   const float *rstd, int64_t N, int64_t C, float eps, int dtype,
                   unsigned int flags, ln_stream_t stream);

/*
 * Dropout.  GPT-2 training drops out the embedding once and each sub-layer's
 * output before it joins the residual stream.  The mask is never stored: it
 * is a function of the call's keys and of the element's index, and forward
 * and backward each draw it again.
 *
 *   dropout(v)[e] = keep(e) ? v[e] * 65536 / (65536 - T) : 0
 *   T             = round(65536 p)       (p rounded to the nearest 2^-16)
 *   keep(e)       = the 16 bits of element e, as a number, are >= T
 *
 * Elements are numbered in memory order (e = r * C + c).  The bits of element
 * e are half e % 2 (0: low) of word (e % 8) / 2 of Philox4x32-10 (Salmon,
 * Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011)
 * with key (seed low word, seed high word) and counter (g low, g high, o low,
 * o high), g = e / 8, o = offset + *step (mod 2^64).  The mask is the same for
 * every dtype, shape of the same element numbering, alignment and device.
 *
 * Arguments common to the dropout calls:
 *   p       0 <= p <= 1 (LN_ERR_PROB; NaN too).  T = 0 keeps every element
 *           unscaled; T = 65536 drops every element.  Dropped elements are
 *           exactly zero, whatever value (infinity, NaN) they had.
 *   seed, offset   64-bit keys, any value (read as unsigned bit patterns).
 *           Two calls with the same seed and offset + *step draw the same
 *           mask: give every dropout of every step its own sum, and a backward
 *           the keys of its forward.
 *   step    device address of a 64-bit counter added to offset when the
 *           kernel runs, 8-byte aligned, or NULL (adds 0).  A captured CUDA
 *           graph keeps the offset it was captured with; a counter that the
 *           graph's owner advances gives every replay a new mask.  Dropouts
 *           that share a seed and a counter need offsets further apart than
 *           the counter ever runs, for example site << 32 with a counter
 *           advanced by 1 per step: with neighbouring offsets, site s at one
 *           step would have the mask of site s - 1 at the next.
 * These calls follow the semantics above (streams, determinism, aliasing,
 * graphs).  Every array must lie on a multiple of its element size
 * (LN_ERR_ALIGN).
 */

/*
 * out = dropout(inp) over n elements in a row.  The backward of this call is
 * the call itself on the gradient with the same keys.
 *   out [n] dtype, written;  inp [n] dtype, read;  0 <= n <= LN_MAX_ELEMS
 * Returns LN_OK or an ln_status error.
 */
int ln_dropout(void *out, const void *inp, int64_t n, float p, int64_t seed, int64_t offset,
               const void *step, int dtype, ln_stream_t stream);

/*
 * ln_forward_residual with a dropped-out branch, the boundary of two GPT-2
 * sub-layers in training:
 *   x         = resid + dropout(branch): the product with the scale rounded
 *               to fp32, the sum to fp32, then once to dtype
 *   resid_out = x
 *   out, mean, rstd = the forward of the rounded x, as ln_forward defines it
 * Arguments as in ln_forward_residual, then the dropout arguments.  mean
 * carries a correction that ln_forward does not make (it stays exact to fp32
 * where it is far smaller than the elements), and the rows' sums may be grouped
 * otherwise than in ln_forward.
 */
int ln_forward_dropout_residual(void *resid_out, void *out, float *mean, float *rstd,
                                const void *resid, const void *branch, const void *weight,
                                const void *bias, int64_t N, int64_t C, float eps, float p,
                                int64_t seed, int64_t offset, const void *step, int dtype,
                                ln_stream_t stream);

/*
 * The backward of ln_forward_dropout_residual.
 *   dx      = dresid_out + (the gradient ln_backward computes from dout), in
 *             fp32 (dresid_out NULL: nothing but the LayerNorm reads x)
 *   dresid  = dx, rounded to dtype             the gradient of resid
 *   dbranch = dropout(dx), rounded to dtype    the gradient of branch
 *   dweight, dbias as in ln_backward
 *   dresid, dbranch [N*C] dtype, written
 *   dresid_out [N*C] dtype, read, or NULL: the gradient that reaches
 *           resid_out other than through the LayerNorm.  May be dresid itself
 *           (a residual gradient updated in place); any other overlap with an
 *           output is LN_ERR_ALIAS.
 *   dout [N*C] dtype, read;  inp [N*C] dtype, read: the forward's resid_out
 *   weight, mean, rstd, eps as in ln_backward_ex
 *   p, seed, offset, step: the forward's, *step holding the forward's value
 *   flags   LN_BWD_ACCUMULATE_DPARAMS and LN_BWD_RECOMPUTE_STATS, as in
 *           ln_backward_ex; other bits give LN_ERR_FLAGS
 * The workspace is ln_backward's; a call of few rows runs as one launch without
 * any.  Returns LN_OK or an ln_status error.
 */
int ln_backward_dropout_residual(void *dresid, void *dbranch, float *dweight, float *dbias,
                                 const void *dresid_out, const void *dout, const void *inp,
                                 const void *weight, const float *mean, const float *rstd,
                                 int64_t N, int64_t C, float eps, float p, int64_t seed,
                                 int64_t offset, const void *step, int dtype,
                                 unsigned int flags, ln_stream_t stream);

/*
 * ln_backward_noalloc: the same computation and arguments as ln_backward, for
 * callers that cannot allocate device memory.  (No counterpart on the pages
 * this library follows: it exists for callers, not for the method.)  Who
 * needs it: programs that reserve all device memory in one arena at start-up
 * and forbid allocation afterwards, code running inside another allocator
 * (where an allocation would re-enter it), and hosts whose memory accounting
 * must not see a second pool.  ln_backward takes its partial sums from a
 * stream-ordered pool; this variant keeps them in a static device array of
 * LN_NOALLOC_SCRATCH_BYTES inside the library, which every GPU that loads the
 * library holds until the process exits.  It calls no cudaMalloc, cudaFree or
 * other allocating routine, and does not create the memory pool that
 * ln_backward uses (a process that only calls this entry point has none).
 *   - The first call on a device (made with that device current) looks up the
 *     array's device address once; make that call before any stream capture.
 *   - All calls share the one array.  Each call overwrites what it reads, so
 *     nothing needs clearing, but calls whose kernels overlap on the GPU
 *     (other streams, other host threads) race on it: serialise them.
 *   - C > LN_NOALLOC_MAX_C (one partial row of 2*C fp32 must fit) returns
 *     LN_ERR_SCRATCH without launching; wide rows run on fewer blocks than
 *     ln_backward would use, so they may be slower.
 * Results match ln_backward within the library's stated tolerances (the
 * column sums may be grouped differently when the array caps the grid).
 */
#define LN_NOALLOC_SCRATCH_BYTES ((int64_t)4 << 20)
#define LN_NOALLOC_MAX_C (LN_NOALLOC_SCRATCH_BYTES / 8)
int ln_backward_noalloc(void *dinp, float *dweight, float *dbias, const void *dout,
                        const void *inp, const void *weight, const float *mean,
                        const float *rstd, int64_t N, int64_t C, int dtype,
                        ln_stream_t stream);

/* Static description of an ln_status value (never NULL). */
const char *ln_status_string(int status);

/* Number of kernels this library has launched in this process (all devices,
 * all streams).  For accounting in benchmarks and tests. */
uint64_t ln_launch_count(void);

/* Diagnostics: the bits that kernels of this library set on the current
 * device when one of their bounded waits ran out (1: a consumer gave up on a
 * stage's data, 2: the producer gave up on a stage's release, 4: a bulk copy
 * in flight did not land in time).  0 means healthy; any other value means
 * the results of the calls since the last clear are not to be trusted.
 * Writes the bits to *bits and, when clear != 0, resets them.  Synchronises
 * the current device.  Returns LN_OK, LN_ERR_NULL or LN_ERR_CUDA. */
int ln_device_status(unsigned int *bits, int clear);

/*
 * Caps the workspace that one ln_backward, ln_backward_ex or
 * ln_backward_dropout_residual call on the current device may draw from the
 * pool, in bytes (0, the default: no cap; a dropout backward of few rows draws
 * none).
 * A call that needs more (G * 2 * C * 4 bytes, G the backward's grid, about
 * the SM count) returns LN_ERR_WORKSPACE before launching anything, exactly
 * as when the pool cannot supply it; the setting stays until changed, and
 * later calls that fit run normally.  For callers that budget device memory
 * per library, and for exercising the workspace-failure path without
 * exhausting a shared GPU.  ln_backward_noalloc is not affected.  Returns
 * LN_OK, LN_ERR_SHAPE for bytes < 0, or LN_ERR_CUDA.
 */
int ln_set_workspace_limit(int64_t bytes);

/*
 * The CUDA error behind the most recent LN_ERR_CUDA returned on the calling
 * host thread: its name, number and description, and the runtime call that
 * raised it (for example "cudaErrorInvalidValue (1: invalid argument) in
 * cudaLaunchKernelEx").  Never NULL; the text is owned by the library and
 * stays valid until the thread's next failing call.  Calls that succeed do
 * not reset it.
 */
const char *ln_last_cuda_error(void);

/* Library ABI version: 3 (2 plus ln_set_workspace_limit and
 * ln_last_cuda_error; 2 was 1 plus ln_forward_residual, ln_backward_ex and
 * LN_F16).  Version 3 libraries from the dropout calls on also export
 * ln_dropout, ln_forward_dropout_residual and ln_backward_dropout_residual;
 * nothing that version 3 had before changed. */
int ln_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LN_H */
