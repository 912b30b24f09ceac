/*
 * mxfp8_wgrad.h -- C ABI of the MI355X (gfx950) MXFP8 ragged weight-gradient
 * grouped GEMM.
 *
 * The operation (blog post "Ragged MXFP8 Weight Gradients: A FlyDSL Grouped
 * GEMM on MI355X", section 1): after expert-parallel dispatch the routed tokens
 * are sorted by expert, and offs[g] is where expert g's run of tokens ends.
 * For every expert g the weight gradient is
 *
 *     dW[g] = dY[g]^T * X[g]          (contraction over expert g's tokens)
 *
 * so the ragged axis is the contraction axis and the output [E, N, K] is
 * dense.  The operands are MXFP8 and quantised along tokens (same section):
 * FP8 E4M3 codes with one E8M0 scale per 32 tokens, passed as A = dY^T [N, M]
 * and B = X^T [K, M] with the token axis contiguous, plus row-major scale
 * planes [N, M/32] and [K, M/32].  Element by element:
 *
 *     dW[g][n][k] = sum_{m = start_g}^{end_g - 1}
 *                     e4m3(A[n][m]) 2^(sA[n][m/32] - 127) *
 *                     e4m3(B[k][m]) 2^(sB[k][m/32] - 127)
 *
 * with start_0 = 0, start_g = offs[g-1], end_g = offs[g] (the XLA blog
 * "Group-GEMM in XLA", section "Contracting": group start = exclusive prefix,
 * end = inclusive prefix).  E4M3 is the OCP E4M3FN flavour; E8M0 is 2^(s-127),
 * 0xFF = NaN.  Accumulation is FP32 on the block-scaled MFMA; the result is
 * rounded once to bfloat16, round-to-nearest-even (blog section 5.5).
 *
 * Every function is callable from C; no exception crosses the boundary.
 */
#ifndef MXFP8_WGRAD_H
#define MXFP8_WGRAD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define MXW_OK 0
#define MXW_ERR_NULL (-1)      /* a required pointer is NULL */
#define MXW_ERR_DIM (-2)       /* a size outside the supported range */
#define MXW_ERR_ALIGN (-3)     /* A, B or out not 16-byte aligned, or sA / sB
                                  not 4-byte aligned (or as the entry says) */
#define MXW_ERR_DEVICE (-4)    /* current device is not gfx950, or no device */
#define MXW_ERR_LAUNCH (-5)    /* a kernel launch failed (hipGetLastError) */
#define MXW_ERR_WORKSPACE (-6) /* workspace NULL, smaller than its size query,
                                  or not 256-byte aligned */
#define MXW_ERR_SCRATCH (-7)   /* the shape needs more workspace than
                                  MXW_SCRATCH_BYTES (no-allocation entry) */
#define MXW_ERR_OVERLAP (-8)   /* what the call writes overlaps itself or an
                                  input */

/* Size of the static device scratch of mxfp8_wgrad_grouped_noalloc. */
#define MXW_SCRATCH_BYTES (160u * 1024u * 1024u)

/* Supported ranges (checked on the host, no device access). */
#define MXW_MAX_EXPERTS 256
#define MXW_MAX_TOKENS (8 * 1024 * 1024)
#define MXW_MAX_ROWS (8 * 1024 * 1024)

/*
 * mxfp8_wgrad_grouped -- the weight-gradient grouped GEMM above.
 *
 * Arguments (every pointer is caller-owned DEVICE memory on the current HIP
 * device):
 *   A     uint8  [N, M]    E4M3 codes of dY^T, row stride M bytes.
 *   sA    uint8  [N, M/32] E8M0 scales of A, row stride M/32 bytes.
 *   B     uint8  [K, M]    E4M3 codes of X^T, row stride M bytes.
 *   sB    uint8  [K, M/32] E8M0 scales of B, row stride M/32 bytes.
 *   offs  int32  [E]       cumulative end of each expert's token run.
 *   E     number of experts, 1 <= E <= MXW_MAX_EXPERTS.
 *   M     token-axis length of A and B (routed tokens plus any padding),
 *         0 <= M <= MXW_MAX_TOKENS, M % 32 == 0.
 *   N, K  output dimensions, each >= 16 and a multiple of 16, <= 65536.
 *   out   bf16 bit patterns [E, N, K], row-major (k contiguous).
 *   stream  a hipStream_t (NULL = the default stream), passed as void*.
 *
 * Host-checked preconditions (violations return an error code and launch
 * nothing): non-NULL pointers; A, B and out 16-byte aligned, sA and sB
 * 4-byte aligned; the ranges above; the current device is gfx950.
 *
 * Device-data preconditions (not checked on the host, which never reads
 * offs): offs non-decreasing, every offs[g] a multiple of 32, offs[E-1] <= M.
 * Tokens in [offs[E-1], M) belong to no expert and may hold anything (NaN
 * codes, 0xFF scales): they never reach the result.  Malformed offs give
 * unspecified values but no out-of-bounds access: windows are clamped to
 * [0, M] and made monotone, every load is range-checked, and every store
 * lands inside out.
 *
 * Effects: enqueues one kernel on `stream` and returns without
 * synchronising.  It allocates nothing, keeps no state between calls, takes
 * no lock (the first call on a device reads its properties once, under a
 * host mutex) and never writes its inputs, so it may run concurrently on any
 * number of streams and be captured into a HIP graph at any time, the very
 * first call included.  `out` is completely overwritten; an expert with no
 * tokens gets exact +0.0.
 *
 * Scheduling and bits: one workgroup per (expert, 256 x 256 output tile)
 * (blog section 4), experts taken longest first (section 5.4), no atomics;
 * when N % 256 == 128 the last 384 rows of N are two tiles of 192 rows
 * instead of a whole one and one half past N (the same tile count); with
 * short experts and a partly filled last round, that round's tiles run
 * as two half-tile workgroups each (mxw_tail_split; such a launch keeps
 * whole 256-row tiles), computing every element exactly as the whole tile
 * does.
 * Each output element is one workgroup's sum over its expert's window in
 * token order, so the result depends only on that expert's window of A, sA,
 * B and sB: it is bitwise reproducible run to run, and unchanged by the
 * other experts' sizes, by the padding past offs[E-1] and by M.
 *
 * Returns MXW_OK or a negative MXW_ERR_* code.
 */
int mxfp8_wgrad_grouped(const uint8_t* A, const uint8_t* sA, const uint8_t* B, const uint8_t* sB,
                        const int32_t* offs, int E, int M, int N, int K, uint16_t* out, void* stream);

/*
 * mxfp8_wgrad_workspace_size -- bytes of device workspace that
 * mxfp8_wgrad_grouped_ws needs for (E, M, ld, N, K) on the current device (0
 * if it needs none), or a negative MXW_ERR_* code.  ld is the row stride
 * described there (0 = M).  Reads device properties only.  128 MiB of FP32
 * partial tiles on a 256-CU device when the launch runs in column mode
 * (mxw_columns() > 0), plus (ceil(N/256) + ceil(K/256)) * ceil(M/512) * 4 KiB
 * of shuffled scales when it pre-shuffles (M >= 4096 E):
 * 149 MiB at the 16B shape with 196,608 tokens, 88 MiB at 671B gate/up with
 * 262,144.
 */
int64_t mxfp8_wgrad_workspace_size(int E, int M, int ld, int N, int K);

/*
 * mxfp8_wgrad_grouped_ws -- the same weight gradient, given a caller-owned
 * device workspace, which lets the launch use two faster schedules where they
 * pay (the blog does not describe either):
 *  - column mode (few output tiles per compute unit, long experts): one
 *    workgroup per CU; 16 workgroups on one XCD form a column that streams
 *    regions of up to 16 tiles of one expert together through that XCD's L2.
 *    The K-step-weighted sequence of (expert, region) pieces is cut into one
 *    equal span per column, and a region cut between columns is summed in a
 *    fixed order through FP32 partial tiles in the workspace: the last of
 *    its pieces to finish (found with a device-scope counter) adds the
 *    others' partials.  No workgroup ever waits for another.
 *  - the scale pre-shuffle (M >= 4096 E): a short first
 *    kernel rewrites sA and sB into the workspace so that the main kernel's
 *    scale loads read consecutive bytes (the blog has a per-call pre-shuffle
 *    too, section 5.6).
 *
 * Arguments: as mxfp8_wgrad_grouped, plus
 *   ld               the row stride of A and B in bytes (tokens), M <= ld <=
 *                    MXW_MAX_TOKENS, ld % 32 == 0, or 0 for M; the scale
 *                    planes' rows are then ld / 32 bytes apart.  A is
 *                    [N, ld] storage holding the [N, M] matrix in its first M
 *                    columns (likewise sA, B, sB); columns [M, ld) are never
 *                    read.  Rows whose stride is a multiple of 64 KiB (the
 *                    16B shape's M = 3 * 2^16, the 671B shapes' 2^18) put the
 *                    lines a tile needs at once into few L2 sets; a stride
 *                    padded by an odd number of 128-token lines
 *                    (ld = M + 128) avoids that at long experts (16B shape,
 *                    196,608 tokens: 35% fewer HBM bytes, 3-4% faster;
 *                    671B: 13% fewer reads, 2-3% faster; within 2% of
 *                    contiguous rows at ~1,000 tokens per expert).
 *                    mxfp8_quantize_tokens writes such padded rows.
 *   workspace        caller-owned device memory, 256-byte aligned, of at
 *                    least mxfp8_wgrad_workspace_size(E, M, ld, N, K) bytes
 *                    (may be NULL when that size is 0).  Its contents are
 *                    undefined on entry and on exit: the call's first kernel
 *                    initialises what the others read.
 *   workspace_bytes  its size.
 *
 * Effects: enqueues one or two kernels on `stream`, returns without
 * synchronising, allocates nothing and keeps no state; graph-capturable at
 * any time.  The workspace is in use until the call's work on `stream` has
 * finished: calls that run concurrently (other streams, overlapping graph
 * replays) need workspaces of their own.  `out` is completely overwritten.
 *
 * Bits: bitwise reproducible run to run for the same (offs, M) on the same
 * device, but in column mode an output element is the sum of FP32 partials
 * whose cut points depend on the whole of offs, on M (through the mode
 * choice) and on the device's CU count: dW[g] may then differ, within the
 * tolerance of FP32 summation order, from mxfp8_wgrad_grouped's result and
 * from the result of a call whose other experts or padding differ.  Without
 * column mode the bits equal mxfp8_wgrad_grouped's.
 *
 * Returns MXW_OK or a negative MXW_ERR_* code (MXW_ERR_WORKSPACE for a
 * missing, short or misaligned workspace).
 */
int mxfp8_wgrad_grouped_ws(const uint8_t* A, const uint8_t* sA, const uint8_t* B, const uint8_t* sB,
                           const int32_t* offs, int E, int M, int ld, int N, int K, uint16_t* out, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * mxfp8_wgrad_grouped_noalloc -- for callers that cannot allocate device
 * memory (code under HIP-graph capture, tight serving loops, harnesses that
 * forbid allocation): mxfp8_wgrad_grouped_ws with its workspace taken from a
 * static device array of MXW_SCRATCH_BYTES (160 MiB) inside the library, which
 * every device the library runs on holds until the process ends.
 *
 * Arguments and results: as mxfp8_wgrad_grouped_ws (row stride ld included)
 * without the workspace arguments; the same plan, kernels and bits.  The
 * caller still passes the operands and out.  A shape whose workspace size
 * (mxfp8_wgrad_workspace_size) exceeds MXW_SCRATCH_BYTES returns
 * MXW_ERR_SCRATCH and launches nothing (the 16B shape with 196,608 tokens
 * needs 149 MiB, 671B gate/up with 262,144 tokens 88 MiB).  It calls no
 * allocating routine; the first call on a device looks up that device's
 * scratch address (hipGetSymbolAddress) once.
 *
 * Every call on a device shares that device's scratch: calls that overlap in
 * time on one device (other streams, overlapping graph replays) race on it
 * and give wrong results.  Each call initialises what it reads; the scratch
 * keeps the last call's contents.
 */
int mxfp8_wgrad_grouped_noalloc(const uint8_t* A, const uint8_t* sA, const uint8_t* B, const uint8_t* sB,
                                const int32_t* offs, int E, int M, int ld, int N, int K, uint16_t* out,
                                void* stream);

/*
 * bf16_wgrad_grouped -- the same weight gradient on plain bfloat16 operands:
 * the "contracting" ragged dot of the XLA blog ("Group-GEMM in XLA", Table 1,
 * and the bfloat16 wgrad_wi / wgrad_wo classes of its Table 7, which contract
 * the ragged token axis into one slab per expert).  For every expert g,
 * n < N, k < K:
 *
 *     out[g][n][k] = sum_{m = start_g}^{end_g - 1} bf16(A[n][m]) * bf16(B[k][m])
 *
 * accumulated in FP32 on the bf16 MFMA (every product is exact in FP32) and
 * rounded once to bf16, round-to-nearest-even.  Same windows as above.
 *
 * Arguments (caller-owned DEVICE memory on the current HIP device):
 *   A     bf16 bit patterns [N, M] (dY^T), token-contiguous, row stride M.
 *   B     bf16 bit patterns [K, M] (X^T), token-contiguous, row stride M.
 *   offs  int32 [E] cumulative ends.  E, N, K, out, stream: as above.
 *   M     0 <= M <= MXW_MAX_TOKENS / 2, M % 16 == 0.
 * The pages give the classes' dimension numbers, not a storage order; the
 * operands are taken with the contracted (token) axis innermost, as for the
 * MXFP8 path.  Device-data preconditions: offs non-decreasing, every offs[g]
 * a multiple of 16, offs[E-1] <= M (malformed offs: unspecified values, no
 * out-of-bounds access).  Tokens in [offs[E-1], M) may hold anything, NaN and
 * infinity included: they never reach the result.
 *
 * Effects, reproducibility and scheduling: as mxfp8_wgrad_grouped (one
 * kernel, allocates nothing, keeps no state; each output element one
 * workgroup's sum in token order).
 *
 * Returns MXW_OK or a negative MXW_ERR_* code.
 */
int bf16_wgrad_grouped(const uint16_t* A, const uint16_t* B, const int32_t* offs, int E, int M, int N, int K,
                       uint16_t* out, void* stream);

/*
 * bf16_wgrad_workspace_size -- bytes of device workspace bf16_wgrad_grouped_ws
 * needs for (E, M, N, K) on the current device (0 if none), or a negative
 * MXW_ERR_* code.  Planned on the token axis in bytes: column mode exactly
 * when mxw_columns(E, 2 M, N, K) > 0; there are no scales to shuffle.
 */
int64_t bf16_wgrad_workspace_size(int E, int M, int N, int K);

/*
 * bf16_wgrad_grouped_ws -- bf16_wgrad_grouped with a caller-owned workspace
 * for column mode, with the workspace contract, effects and bits of
 * mxfp8_wgrad_grouped_ws (a first one-workgroup kernel clears the counters).
 */
int bf16_wgrad_grouped_ws(const uint16_t* A, const uint16_t* B, const int32_t* offs, int E, int M, int N, int K,
                          uint16_t* out, void* workspace, size_t workspace_bytes, void* stream);

/*
 * mxw_grid_size -- the number of (expert, 256 x 256 output tile) work items
 * of (E, N, K), E * ceil(N/256) * ceil(K/256) (blog section 4: one block per
 * expert per output tile): the workgroups mxfp8_wgrad_grouped launches, and
 * mxfp8_wgrad_grouped_ws outside column mode.  Returns 0 for invalid sizes.
 */
int64_t mxw_grid_size(int E, int N, int K);

/*
 * mxw_columns -- the number of columns mxfp8_wgrad_grouped_ws uses for
 * (E, M, N, K) on the current device: 0 when it launches one workgroup per
 * work item, otherwise the column count of column mode (16 workgroups per
 * column, one per compute unit).  Column mode is chosen when the work items
 * fill the device at most 4 times over and M >= 8192 * E.  Reads device
 * properties only; returns MXW_ERR_DIM or MXW_ERR_DEVICE on invalid input or
 * no gfx950 device.
 */
int mxw_columns(int E, int M, int N, int K);

/*
 * mxw_tail_split -- how many output tiles mxfp8_wgrad_grouped runs as two
 * half tiles for (E, M, N, K) on the current device (0: none); the same
 * holds for mxfp8_wgrad_grouped_ws when it runs one workgroup per tile
 * without the scale pre-shuffle (mxw_columns() == 0, mxw_scale_shuffle() ==
 * 0), and for the bf16 entries with M tokens when they run one workgroup per
 * tile (mxw_columns(E, 2 M, N, K) == 0).  When the tiles fill the device only a few times over (more than once,
 * under 4 times) and experts are short (M <= 2048 E), the tiles of the last,
 * partly filled round (the last in longest-first order) each run as two
 * workgroups, one for the even and one for the odd 32-row blocks of the
 * tile's 256 rows of N, so that round has twice as many workgroups of a
 * little over half the length.  Each output element is computed exactly as
 * in the whole tile: the bits do not change.  Returns MXW_ERR_DIM or
 * MXW_ERR_DEVICE on invalid input or no gfx950 device.
 */
int mxw_tail_split(int E, int M, int N, int K);

/*
 * mxw_scale_shuffle -- 1 if mxfp8_wgrad_grouped_ws with (E, M) runs the scale
 * pre-shuffle kernel before the main kernel (M >= 4096 E),
 * 0 if it launches the main kernel alone, MXW_ERR_DIM for invalid sizes.
 * Host-only: no device access.
 */
int mxw_scale_shuffle(int E, int M);

/*
 * mxfp8_grouped_fwd -- the row-ragged MXFP8 grouped GEMM: the forward and
 * data-gradient GEMMs of the same MoE layer.  (Blog section 1: the weight
 * gradient is one of three grouped GEMMs per expert layer; the other two keep
 * the contraction over the fixed hidden dimension and carry the raggedness
 * in their rows.  XLA blog: the "non-contracting" ragged dot and its forward
 * and data-gradient classes.)  For every expert g, every row m in
 * [start_g, end_g) (start_0 = 0, start_g = offs[g-1], end_g = offs[g]) and
 * every n < N:
 *
 *   out[m][n] = sum over c in [0, C) of
 *               e4m3(A[m][c]) 2^(sA[m][c/32] - 127) * e4m3(B[g][n][c]) 2^(sB[g][n][c/32] - 127)
 *
 * accumulated in FP32 and rounded to bf16 (round to nearest even).  Forward:
 * A = the routed tokens' activations (C = the layer's input width), B = the
 * expert weights.  Data gradient: A = the output gradient, B = the weights
 * quantized along their other axis.  MXFP8 puts its 32-element blocks along
 * the contraction axis, so both operands are stored with C innermost.
 *
 * Arguments (caller-owned DEVICE memory on the current HIP device):
 *   A     uint8  [R, C]       E4M3 codes, row stride C bytes.
 *   sA    uint8  [R, C/32]    E8M0 scales of A.
 *   B     uint8  [E, N, C]    E4M3 codes of each expert's [N, C] operand.
 *   sB    uint8  [E, N, C/32] E8M0 scales of B.
 *   offs  int32  [E]          cumulative end of each expert's run of rows.
 *   E     1 <= E <= MXW_MAX_EXPERTS.
 *   R     rows of A and out, 0 <= R <= MXW_MAX_ROWS.
 *   C     contraction length, 32 <= C <= 65536, C % 32 == 0.
 *   N     output columns, 16 <= N <= 65536, N % 16 == 0.
 *   out   bf16 bit patterns [R, N], row-major.
 *   stream  a hipStream_t (NULL = the default stream), passed as void*.
 *
 * Host-checked preconditions return an error code and launch nothing:
 * non-NULL pointers; A, B and out 16-byte aligned, sA and sB 4-byte
 * aligned; the ranges above; a gfx950 device.  Device-data preconditions
 * (never read on the host): offs non-decreasing and offs[E-1] <= R; row boundaries need no alignment.
 * Rows in [offs[E-1], R) belong to no expert: they are neither read as
 * values nor written.  Malformed offs give unspecified values but no
 * out-of-bounds access (windows are clamped to [0, R], loads range-checked,
 * stores confined to the clamped windows).
 *
 * Effects: enqueues one kernel on `stream`; allocates nothing, keeps no
 * state, never writes its inputs.  Each output element is one workgroup's
 * fixed-order sum: bitwise reproducible run to run.
 *
 * Returns MXW_OK or a negative MXW_ERR_* code.
 */
int mxfp8_grouped_fwd(const uint8_t* A, const uint8_t* sA, const uint8_t* B, const uint8_t* sB,
                      const int32_t* offs, int E, int R, int C, int N, uint16_t* out, void* stream);

/*
 * mxw_fwd_grid_size -- the workgroups mxfp8_grouped_fwd launches for
 * (E, R, N): (R / 256 + E) * ceil(N / 256) work items at most (each expert
 * adds at most one partial 256-row tile), rounded up to a multiple of 8.
 * Workgroups past the actual number of work items exit at once.  Returns 0
 * for invalid sizes.
 */
int64_t mxw_fwd_grid_size(int E, int R, int N);

/*
 * mxfp8_quantize_tokens -- the token-axis MXFP8 quantiser that produces the
 * weight gradient's operands (blog section 1: both operands are quantised
 * along the token axis and handed over token-contiguous, with one E8M0
 * scale per 32 tokens; the blog times its operator without this step,
 * section 7).  From bf16 x [M, H] (tokens x hidden, hidden contiguous) to
 * E4M3 codes q [H, M] and E8M0 scales s [H, M/32]; for every hidden column
 * h and 32-token block b:
 *
 *   amax    = max |x[m][h]| over the block's tokens below `used`
 *   s[h][b] = clamp(floor(log2 amax) - 8 + 127, 0, 254), 127 if amax == 0
 *   q[h][m] = E4M3FN(x[m][h] / 2^(s[h][b] - 127)): round to nearest, ties to
 *             the even code, saturated to +-448, zero encoded as +0; 0 for
 *             m >= used
 *
 * (8 = floor(log2 448), the largest E4M3 binade: the OCP MX shared scale.)
 * Call it on dY for A and on X for B.  `used` is offs[E-1] read on the
 * device (tokens past the last expert become finite zeros, whatever x holds
 * there), or M when offs is NULL.
 *
 * Arguments (caller-owned DEVICE memory on the current HIP device):
 *   x     uint16 [M, H]    bf16 bit patterns.
 *   offs  int32  [E]       cumulative expert ends (may be NULL: all tokens).
 *   E     1 <= E <= MXW_MAX_EXPERTS when offs is not NULL.
 *   M     0 <= M <= MXW_MAX_TOKENS, M % 32 == 0.
 *   ld    row stride of q in bytes (tokens), M <= ld <= MXW_MAX_TOKENS,
 *         ld % 32 == 0, or 0 for M; s's rows are ld / 32 bytes apart.  A
 *         padded stride (ld = M + 128) is the layout mxfp8_wgrad_grouped_ws
 *         reads best (see there); columns [M, ld) of q and [M/32, ld/32) of
 *         s are not written.
 *   H     16 <= H <= 65536, H % 16 == 0.
 *   q     uint8  [H, ld]   codes (the first M bytes of each row).
 *   s     uint8  [H, ld/32] scales (the first M/32 bytes of each row); any
 *         alignment, but with s 8-byte aligned and ld % 256 == 0 every
 *         whole 256-token tile's scale bytes go out as one 8-byte store
 *         per row, and with s 4-byte aligned and ld % 128 == 0 as two
 *         4-byte stores (either way faster than byte stores).
 *   stream  a hipStream_t, passed as void*.
 *
 * Host-checked preconditions return an error code and launch nothing:
 * non-NULL x, q, s; x and q 16-byte aligned; the ranges above; a gfx950
 * device.  Effects: one kernel on `stream`; allocates nothing; the [H, M]
 * codes and [H, M/32] scales are fully overwritten; the result depends only
 * on x and `used`.
 *
 * Returns MXW_OK or a negative MXW_ERR_* code.
 */
int mxfp8_quantize_tokens(const uint16_t* x, const int32_t* offs, int E, int M, int ld, int H, uint8_t* q,
                          uint8_t* s, void* stream);

/* Element types of entries that take more than one. */
#define MXW_BF16 0
#define MXW_F32 1

/*
 * mxw_orthogonalize -- what an optimiser that orthogonalises its updates does
 * with the weight gradients (or a momentum of them): for every expert g, with
 * X = G[g] / (|G[g]|_F + eps), each step replaces
 *
 *     X <- a X + (b S + c S S) X,    S = X X^T
 *
 * with that step's (a, b, c) (for N > K the same on X^T), which drives the
 * singular values of X towards 1 and keeps its singular vectors; out[g] is X
 * after the last step.  The usual five steps of (3.4445, -4.7750, 2.0315) bring
 * every singular value above about 0.01 |G|_2 into 0.7 .. 1.2.
 *
 * Arguments (pointers other than coeffs are caller-owned DEVICE memory):
 *   G        [E, N, K] elements of `type` (MXW_BF16 or MXW_F32), the last axis
 *            contiguous; rows row_stride >= K elements apart, experts
 *            expert_stride >= 0 elements.
 *   E, N, K  1 <= E <= MXW_MAX_EXPERTS, 1 <= N, K <= 65536, and at most 2^20
 *            256 x 256 tiles in all; no multiples are asked for.
 *   coeffs   HOST memory, 3 * steps floats: (a, b, c) of each step, read
 *            during the call.
 *   steps    1 .. 32.
 *   eps      >= 0, added to the norm.
 *   out      bf16 [E, N, K], contiguous, fully overwritten; not overlapping G.
 *   workspace, workspace_bytes  256-byte aligned device memory of at least
 *            mxw_orthogonalize_workspace_size(E, N, K) bytes; contents
 *            undefined on entry and exit, in use until the call's work is done.
 *
 * The norm's sum is taken in 64 bits; X, S and P = a I + b S + c S S are held
 * in f16 times 2^10 between products, whose sums are FP32.  Against the same
 * formula in 64 bits the result is off by about 0.13% of its norm (its own
 * rounding to bf16: 0.17%).  An entry of X, S or P beyond +-63 (no published
 * coefficients come near) overflows to infinity and shows as NaN.  An expert
 * whose gradient is zero gets zeros, with eps = 0 too; one with a NaN or
 * infinity gets NaN, and no expert's result depends on another's values.  Their
 * number can: with few short matrices the sums over a long side are split by how many
 * there are, and a matrix's last bits differ between calls of another E.  Bitwise
 * reproducible run to run.
 *
 * Effects: enqueues one kernel (matrices that fit in LDS) or 2 + 3 * steps and
 * some more on `stream`, allocates nothing, keeps
 * no state, never writes G, does not synchronise; graph-capturable.
 * Returns MXW_OK or a negative MXW_ERR_* code.
 */
int mxw_orthogonalize(const void* G, int type, int64_t expert_stride, int64_t row_stride, int E, int N, int K,
                      const float* coeffs, int steps, float eps, uint16_t* out, void* workspace,
                      size_t workspace_bytes, void* stream);

/* mxw_orthogonalize_workspace_size -- bytes of workspace that mxw_orthogonalize
 * needs, or MXW_ERR_DIM.  Host-only. */
int64_t mxw_orthogonalize_workspace_size(int E, int N, int K);

/* Reductions of mxw_vocab_loss. */
#define MXW_NONE 0
#define MXW_MEAN 1
#define MXW_SUM 2

/*
 * mxw_vocab_loss -- softmax cross entropy of hidden states against a large
 * vocabulary, with its gradients, in bounded memory.  For every token t with
 * target y(t):
 *
 *     l_tv = sum_h x[t][h] w[v][h],  loss_t = log sum_v exp(l_tv) - l_t,y(t)
 *     g_tv = (exp(l_tv) / sum_u exp(l_tu) - [v = y(t)]) * s
 *     dx[t] = sum_v g_tv w[v],       dw[v] = sum_t g_tv x[t]
 *
 * Tokens whose target is ignore_index have loss 0 and no gradient, whatever
 * their x holds (NaN included).  MXW_NONE
 * gives the loss of every token, MXW_SUM their sum, MXW_MEAN the sum divided by
 * the number of tokens that are not ignored (0 if there is none).  s is
 * grad_scale, divided by that number for MXW_MEAN: dx and dw are the gradients
 * of grad_scale times the reduced loss (of the sum, for MXW_NONE).
 *
 * Arguments (caller-owned DEVICE memory):
 *   x, ldx   bf16 [T, H], rows ldx >= H elements apart.
 *   w, ldw   bf16 [V, H], rows ldw >= H elements apart.
 *   targets  [T] int32 (target_bytes 4) or int64 (8).  A target outside
 *            [0, V) that is not ignore_index makes that token's loss (and the
 *            reduced loss) NaN and gives no gradient either.
 *   T, H, V  1 <= T <= 131072, 1 <= H <= 65536, 1 <= V <= 1048576, no
 *            multiples asked for.  With H % 64 == 0, 16-byte aligned x and w
 *            and row strides of whole 16 bytes (up to 2^21 elements) the
 *            operands are read in place (x is copied, without the tokens that
 *            give no gradient, if dw is wanted); otherwise padded copies are
 *            made in the workspace, w's by pieces.
 *   loss     FP32, [T] for MXW_NONE, one value otherwise.
 *   dx, dw   bf16 [T, H] and [V, H], contiguous, fully overwritten; either may
 *            be NULL (not wanted).  They overlap no input.
 *   workspace, workspace_bytes  256-byte aligned device memory of at least
 *            mxw_vocab_loss_workspace_size(...) bytes; contents undefined on
 *            entry and exit, in use until the call's work is done.  If
 *            gradients are wanted it has room for the FP32 logits where they
 *            take at most 4 GiB (64 MiB for H < 1024); with a smaller one, of
 *            at least the size for MXW_LOSS_SMALL, they are made twice
 *            instead: up to a quarter more time, the same bits.
 *
 * Logits, statistics and sums are FP32; the g of a piece of the vocabulary is
 * rounded to bf16 before the two products that use it.  NaN in the x of a token
 * that counts reaches that token's loss and dx, and dw; a NaN or +infinite logit makes
 * its token's loss NaN.  A -infinite one is a word of probability 0: the loss stays
 * finite (infinite if it is the target).  The gradients are the formula's there too: a
 * g of 0 times an infinite value of w or x is NaN, in every dx that meets it or in dw.
 * Bitwise reproducible run to run on the same device.
 *
 * Effects: enqueues kernels on `stream`, allocates nothing, keeps no state,
 * never writes its inputs, does not synchronise; graph-capturable.
 * Returns MXW_OK or a negative MXW_ERR_* code.
 */
int mxw_vocab_loss(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, const void* targets,
                   int target_bytes, int64_t ignore_index, int T, int H, int V, int reduction, float grad_scale,
                   float* loss, uint16_t* dx, uint16_t* dw, void* workspace, size_t workspace_bytes, void* stream);

/* mxw_vocab_loss_workspace_size -- bytes of workspace that mxw_vocab_loss needs
 * on the current device, or a negative MXW_ERR_* code.  x and w are looked at
 * for their alignment alone; grads: 1 if dx is wanted, plus 2 if dw is, plus
 * MXW_LOSS_SMALL for the size without room for the logits. */
#define MXW_LOSS_SMALL 8
int64_t mxw_vocab_loss_workspace_size(const uint16_t* x, int64_t ldx, const uint16_t* w, int64_t ldw, int T, int H,
                                      int V, int grads);

/* Most tokens of a mxw_moe_layer call. */
#define MXW_MOE_MAX_TOKENS 64

/*
 * mxw_moe_layer -- a whole mixture-of-experts layer for a few tokens (single
 * tokens and small batches, as in generation; mxfp8_grouped_fwd is the form for
 * many).  For every token t:
 *
 *     r_e   = sum_h x[t][h] router[e][h]
 *     ids   = the k experts with the largest r, largest first (ties: the lower)
 *     weight_j = softmax(r) at ids[j], divided by the k values' sum if
 *             `normalize`, times `scale`
 *     h_j   = silu(x[t] Wg^T) * (x[t] Wu^T)  of expert ids[j]
 *     out[t] = sum_j weight_j h_j Wd^T
 *
 * Arguments (caller-owned DEVICE memory):
 *   x, ldx   bf16 [T, H], rows ldx >= H elements apart (a multiple of 8).
 *   router   bf16 [E, H], or NULL: then ids and weights are inputs (an id
 *            outside [0, E) is an empty slot; weights are used as they are).
 *   wgu, sgu E4M3 codes [E, 2 I, H] and E8M0 scales [E, 2 I, H/32]: each
 *            expert's I gate rows, then its I up rows, 32-element blocks along
 *            H (the layout mxfp8_grouped_fwd takes).
 *   wd, sd   E4M3 codes [E, H, I] and E8M0 scales [E, H, I/32].
 *   active   uint8 [T], 0 for a token that is not there (an unused slot of the
 *            batch): its out is zeros and x's row is not used; with a router
 *            its ids are -1 and its weights 0.  NULL: all are.
 *   T        1 .. MXW_MOE_MAX_TOKENS.   E  1 .. MXW_MAX_EXPERTS.
 *   k        1 .. 16, at most E.        H, I  multiples of 32, 32 .. 65536.
 *   ids, weights  int32 and FP32 [T, k]: outputs, inputs without a router.
 *   out      bf16 [T, H], contiguous, fully overwritten.
 *   x, router, wgu, wd 16-byte aligned; sgu, sd, ids, weights 4-byte aligned.
 *   workspace, workspace_bytes  256-byte aligned device memory of at least
 *            mxw_moe_workspace_size(T, E, k, H, I) bytes; contents undefined on
 *            entry and exit, in use until the call's work is done.
 *
 * Codes and scales become bf16 exactly where their product has a normal bf16
 * value (below 2^-126 it is 0, beyond bf16's range infinity; scale 0xFF: NaN);
 * all sums are FP32; weight_j h_j is rounded to bf16 between the two products.
 * A NaN or +infinite logit, or -infinite ones alone, make that token's weights and
 * out NaN; else an expert of -infinite logit is chosen last, with weight 0.  No token's
 * result depends on another's values.  Bitwise reproducible run to run.
 *
 * Effects: enqueues two to five kernels on `stream`, allocates nothing, keeps no
 * state, does not synchronise; graph-capturable.  Only the chosen experts'
 * weights are read.  Returns MXW_OK or a negative MXW_ERR_* code.
 */
int mxw_moe_layer(const uint16_t* x, int64_t ldx, const uint16_t* router, const uint8_t* wgu, const uint8_t* sgu,
                  const uint8_t* wd, const uint8_t* sd, const uint8_t* active, int T, int E, int k, int H, int I,
                  int normalize, float scale, int32_t* ids, float* weights, uint16_t* out, void* workspace,
                  size_t workspace_bytes, void* stream);

/* mxw_moe_workspace_size -- bytes of workspace that mxw_moe_layer needs, or
 * MXW_ERR_DIM.  Host-only. */
int64_t mxw_moe_workspace_size(int T, int E, int k, int H, int I);

/* Most choices (experts) of a token in the entries below. */
#define MXW_MAX_CHOICES 64

/*
 * mxw_sort_tokens -- which row every token goes to when tokens are grouped by
 * expert, as the grouped products above take them.  With e = ids[t][j], choices in the
 * order (t, j):
 *
 *     counts[e] = the number of choices of expert e
 *     offs[e]   = sum over e' <= e of counts[e'] rounded up to a multiple of `align`
 *     rows[t][j] = offs[e-1] + the number of earlier choices of e;  -1 for an id
 *                  outside [0, E) (an empty slot)
 *
 * offs is the cumulative ends that the grouped products read; the rows from an
 * expert's last choice to its end are padding.
 *
 * Arguments (caller-owned DEVICE memory):
 *   ids, id_bytes, ld  [T, k] int32 (4) or int64 (8), rows ld >= k elements apart.
 *   T, k     T >= 0, 1 <= k <= MXW_MAX_CHOICES, T k <= MXW_MAX_ROWS.  An expert may
 *            be named more than once by a token: each is a row of its own.
 *   E        1 .. MXW_MAX_EXPERTS.
 *   align    1 .. 1024 (32 is what mxfp8_wgrad_grouped needs, 16 bf16_wgrad_grouped).
 *   offs, counts  int32 [E];  rows  int32 [T, k]; fully overwritten.
 *   workspace, workspace_bytes  256-byte aligned device memory of at least
 *            mxw_sort_workspace_size(T, k, E) bytes (NULL if that is 0: up to 4,096
 *            choices); contents undefined on entry and exit, in use until the
 *            call's work is done.
 *
 * mxw_token_rows gives the rows that any ids of these sizes fit in, a multiple of
 * align: what to allocate without reading offs on the host.  MXW_ERR_DIM if that is
 * over MXW_MAX_ROWS.
 *
 * Effects: enqueues one or two kernels on `stream`, allocates nothing, keeps no state,
 * does not synchronise; graph-capturable.  Returns MXW_OK or a negative code.
 */
int mxw_sort_tokens(const void* ids, int id_bytes, int64_t ld, int T, int k, int E, int align, int32_t* offs,
                    int32_t* counts, int32_t* rows, void* workspace, size_t workspace_bytes, void* stream);
int64_t mxw_token_rows(int T, int k, int E, int align);
int64_t mxw_sort_workspace_size(int T, int k, int E);

/*
 * mxw_dispatch_tokens -- tokens copied to their rows, as they are, as MXFP8 or both:
 *
 *     xs[rows[t][j]] = x[t],   (q, s)[rows[t][j]] = MXFP8 of x[t]
 *
 * with blocks of 32 along H and the codes and scales of mxw_quantize_rows (bit for
 * bit): A and sA of mxfp8_grouped_fwd.  The padding rows of every expert (from
 * offs[e-1] + counts[e] to offs[e]) become zeros (codes 0, scales 127); rows from
 * offs[E-1] on are left as they were.  The gradient with respect to x is
 * mxw_combine_tokens of the rows' gradient, without weights.
 *
 * Arguments (caller-owned DEVICE memory):
 *   x, type, ldx  [T, H] MXW_BF16 or MXW_F32, rows ldx >= H elements apart.
 *   offs, counts, rows  as mxw_sort_tokens leaves them.  A row outside [0, R) is
 *            skipped (an empty slot, or rows that were cut); whatever they hold, no
 *            store leaves the outputs.
 *   T, k, E  as above.  H  1 .. 65536, a multiple of 32 with q.
 *   R        rows of the outputs, 0 .. MXW_MAX_ROWS.
 *   xs       [R, H] of `type`, contiguous, or NULL.
 *   q, s     uint8 [R, H] and [R, H/32], contiguous, or both NULL; q 8-byte aligned.
 * What is written overlaps neither itself nor an input (MXW_ERR_OVERLAP, as in
 * mxw_sort_tokens and the entries below; strided rows count with what lies between them).
 * Effects: one kernel on `stream`, allocates nothing, keeps no state, does not synchronise;
 * graph-capturable.
 */
int mxw_dispatch_tokens(const void* x, int type, int64_t ldx, const int32_t* offs, const int32_t* counts,
                        const int32_t* rows, int T, int k, int E, int H, int R, void* xs, uint8_t* q, uint8_t* s,
                        void* stream);

/*
 * mxw_combine_tokens -- the experts' rows joined to tokens again:
 *
 *     out[t] = sum_j weights[t][j] y[rows[t][j]] + residual[t]
 *
 * summed in FP32 in the order of j, the residual last, and rounded once.  Choices
 * whose row is outside [0, R) count nothing, whatever their weight holds.
 *
 *   y, type, ldy  [R, H] MXW_BF16 or MXW_F32, rows ldy >= H elements apart.
 *   weights  FP32 [T, k], contiguous, or NULL: 1.
 *   residual, ldr  [T, H] of `type`, rows ldr >= H elements apart, or NULL: none.
 *   out      [T, H] of `type`, contiguous; it may be residual itself (ldr == H).
 * Effects: as above.  A token's result depends on its own rows and weights alone.
 */
int mxw_combine_tokens(const void* y, int type, int64_t ldy, const int32_t* rows, const float* weights,
                       const void* residual, int64_t ldr, int T, int k, int H, int R, void* out, void* stream);

/*
 * mxw_combine_tokens_grad -- the gradients of mxw_combine_tokens from that of out:
 *
 *     dy[rows[t][j]] = weights[t][j] dout[t],   dweights[t][j] = <dout[t], y[rows[t][j]]>
 *
 * (that of the residual is dout).  dy in the type of dout, and/or as MXFP8 rows of what
 * dy would hold (q, s, as in mxw_dispatch_tokens: A and sA of the data gradient's
 * product); padding rows become zeros and rows from offs[E-1] on are left as they were.
 * dweights FP32 [T, k], 0 for empty slots; sums in FP32.  Any of the three outputs may
 * be NULL (not wanted), and offs and counts if dy and q are.  y is read only for
 * dweights; dy may be y itself (ldy == H).  Other sizes, checks and effects: as above.
 */
int mxw_combine_tokens_grad(const void* dout, int type, int64_t ldo, const void* y, int64_t ldy, const int32_t* offs,
                            const int32_t* counts, const int32_t* rows, const float* weights, int T, int k, int E, int H,
                            int R, void* dy, uint8_t* q, uint8_t* s, float* dweights, void* stream);

/* Formats of quantised rows and weights. */
#define MXW_MXFP8 0 /* E4M3 codes, an E8M0 scale for 32 */
#define MXW_MXFP4 1 /* E2M1 codes, two a byte, an E8M0 scale for 32 */
#define MXW_INT4 2  /* unsigned 4-bit codes, two a byte, a bf16 scale (and a zero) for a group */

/*
 * mxw_quantize_rows -- the row-wise MX quantiser: operands whose blocks of 32 lie
 * along the rows, as mxfp8_grouped_fwd takes them (MXFP8) and mxw_linear_4bit takes its
 * weights (MXFP4).  For every block, with amax = max |x|:
 *
 *     s = clamp(floor(log2 amax) - b + 127, 0, 254), 127 if amax == 0, and 255 (NaN) if
 *         the block holds an infinity or a NaN
 *     q = the format's number nearest to x / 2^(s - 127): ties to even, saturated at
 *         its largest, zeros as +0 (under a NaN scale: 0x7F in MXFP8, 0 in MXFP4)
 *
 * with b = 8 and the largest 448 (MXFP8, as mxfp8_quantize_tokens), b = 2 and 6 (MXFP4).
 *
 *   x, type, ldx  [R, C] MXW_BF16 or MXW_F32, rows ldx >= C elements apart.
 *   R        >= 0, at most 2^31 and 2^35 - 4096 elements in all.  C  a multiple of 32, 32 .. 65536.
 *   q        uint8 [R, C] (MXFP8) or [R, C/2] (MXFP4: element 2 i in the low half of byte
 *            i), contiguous, 8-byte aligned.  s  uint8 [R, C/32], contiguous.
 * Effects: one kernel on `stream`, allocates nothing, keeps no state, does not
 * synchronise; graph-capturable.
 */
int mxw_quantize_rows(const void* x, int type, int64_t ldx, int64_t R, int C, int format, uint8_t* q, uint8_t* s,
                      void* stream);

/* Norms of mxw_clip_grads, and its most tensors. */
#define MXW_NORM_2 2
#define MXW_NORM_MAX 0
#define MXW_MAX_TENSORS 65536

/*
 * mxw_clip_grads -- the norm of many gradients together, and the gradients clipped to
 * it:
 *
 *     n = (sum over all elements of g^2)^(1/2)   or   max |g|
 *     out[i] = g[i] min(1, max_norm / (n + eps))
 *
 * Arguments:
 *   grads, outs, sizes, types  HOST arrays of `count` entries, read during the call:
 *            device addresses, element counts (0 .. 2^40; a NULL address with 0) and
 *            MXW_BF16 or MXW_F32.  outs[i] may be grads[i] (in place); otherwise nothing
 *            that is written (norm and workspace too) may overlap (MXW_ERR_OVERLAP).  outs
 *            NULL: the norm alone.
 *   count    0 .. MXW_MAX_TENSORS (0: norm 0).
 *   norm_type  MXW_NORM_2 or MXW_NORM_MAX.   max_norm, eps  >= 0.
 *   norm     DEVICE memory, one FP32: n before clipping.
 *   workspace, workspace_bytes  256-byte aligned device memory of at least
 *            mxw_clip_workspace_size(count) bytes; contents undefined on entry and exit,
 *            in use until the call's work is done.
 *
 * Squares are summed in 64 bits: the norm neither overflows nor vanishes before FP32
 * does.  The product with the factor is FP32 (by 2^-126 first where the factor is below that),
 * rounded once more for bf16 outputs.  A NaN makes the norm and
 * all outputs NaN; an infinity makes the norm infinite and the factor 0 (its own element
 * NaN), unless max_norm is infinite too (NaN).  Where n + eps is 0 the factor is 1.  Bitwise
 * reproducible run to run.
 * Effects: enqueues two kernels for every 96 tensors (one more if there are more) on
 * `stream`, allocates nothing on the device, keeps no state, does not synchronise;
 * graph-capturable (the addresses are the kernels' arguments).
 */
int mxw_clip_grads(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* types, int count,
                   int norm_type, double max_norm, double eps, float* norm, void* workspace, size_t workspace_bytes,
                   void* stream);
int64_t mxw_clip_workspace_size(int count);

/*
 * mxw_linear_4bit -- a dense product of a few tokens with 4-bit weights (the
 * projections and the vocabulary around mxw_moe_layer in generation):
 *
 *     out[t][n] = sum_k x[t][k] v[n][k]
 *     MXW_MXFP4:  v = e2m1(code) 2^(scale - 127)        (scale 0xFF: NaN)
 *     MXW_INT4:   v = (code - zero) scale
 *
 * Arguments (caller-owned DEVICE memory):
 *   x, ldx   bf16 [T, K], rows ldx >= K elements apart (a multiple of 8, up to 2^23), 16-byte
 *            aligned.
 *   codes    uint8 [N, K/2], element 2 i of a row in the low half of byte i; contiguous,
 *            16-byte aligned.
 *   scales   [N, K/group]: E8M0 bytes (MXW_MXFP4) or bf16 (MXW_INT4), contiguous.
 *   zeros    uint8 [N, K/group], 0 .. 15, MXW_INT4 only, or NULL: 8.
 *   group    32 (MXW_MXFP4) or 32, 64, 128 (MXW_INT4).
 *   T        0 .. MXW_MOE_MAX_TOKENS.  N  1 .. 2^20.  K  a multiple of group, up to 65536.
 *   out, out_type  [T, N] MXW_BF16 or MXW_F32, contiguous, fully overwritten.
 *
 * The numbers that MXFP4 codes stand for enter as bf16, exactly, subnormals included (2^128
 * and beyond as infinity); integer codes and zeros enter as whole numbers, summed apart, and
 * each group's FP32 difference is scaled: an infinity in x then gives NaN where the formula may
 * give an infinity, and a group's sums of x times its codes must stay in FP32's range (x up to
 * 2^116 keeps them there).  All sums are FP32.  A token's result does not depend on the other
 * tokens' values; its last bits can depend on T and N, by which K is split.  Bitwise
 * reproducible run to run.
 * Effects: one kernel on `stream`, allocates nothing, keeps no state, does not
 * synchronise; graph-capturable.
 */
int mxw_linear_4bit(const uint16_t* x, int64_t ldx, const uint8_t* codes, const void* scales, const uint8_t* zeros,
                    int format, int group, int T, int K, int N, void* out, int out_type, void* stream);

/* mxw_strerror -- a static, human-readable message for a return code. */
const char* mxw_strerror(int code);

/* mxw_version -- library ABI version (major * 10000 + minor * 100 + patch). */
int mxw_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_WGRAD_H */
