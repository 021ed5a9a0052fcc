/*
 * pgemm.h -- persistent-tile-scheduled GEMM for AMD Instinct MI355X (gfx950).
 *
 * C-ABI boundary of the library: plain pointers and sizes, no C++ or torch
 * types. All matrix pointers are DEVICE pointers (hipMalloc'd or torch
 * tensors' data_ptr()); everything else is host memory.
 *
 * The operation (persistent-kernel forum thread, question): the GEMM
 *     C[i][j] = sum_k A[i][k] * B[k][j]
 * with A: M x K row-major (leading dimension K), B: K x N row-major
 * (leading dimension N) -- or, after pgemm_set_b_layout(h, PGEMM_B_NK),
 * N x K row-major (leading dimension K, i.e. B stored transposed, the layout
 * of a linear layer's weight) -- and C: M x N row-major (leading dimension
 * N), all contiguous, accumulated in fp32. The output is cut into macro tiles and
 * a tile scheduler hands tiles to workgroups (same question). Scheduling
 * never changes the value of C: modes NONPERSISTENT..CANCEL run the same
 * tile body, so C is bitwise identical across them and across reruns
 * (KernelWiki "Persistent Kernels with Cluster Launch Control", "Choosing
 * between static and CLC scheduling": neither scheduler adds work).
 * STREAMK adds work (split tiles' partial sums), so its C may differ from
 * theirs in the last bits; it is bitwise identical across its own reruns.
 *
 * Errors: every entry point returns a pgemm_status_t. No C++ exception
 * crosses this boundary. Launches are asynchronous on the handle's stream;
 * errors of the launch itself are returned as PGEMM_ERR_HIP, with detail
 * in pgemm_last_error(). A handle is not thread-safe: use one handle per
 * stream used concurrently (the dynamic scheduler's work counter is per
 * handle; DYNAMIC and CANCEL share it).
 */
#ifndef PGEMM_H
#define PGEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct pgemm_ctx* pgemm_handle_t;

typedef enum {
  PGEMM_OK = 0,
  PGEMM_ERR_INVALID_ARG = 1, /* null pointer with non-zero size, negative size, bad enum */
  PGEMM_ERR_UNSUPPORTED = 2, /* size beyond the 32-bit tile/offset limits */
  PGEMM_ERR_HIP = 3,         /* a HIP runtime call failed; see pgemm_last_error() */
  PGEMM_ERR_OOM = 4,         /* device or host allocation failed */
  PGEMM_ERR_TIMEOUT = 5      /* pgemm_wait: the stream's work did not finish in time */
} pgemm_status_t;

/* Element formats. The pages name fp16 and fp8 (Triton persistent-matmul
 * issue: "--prec fp16", and the fp8 example on H100); bf16 is the other
 * 16-bit format of the same MFMA family. fp8 is OCP E4M3 ("fn": bias 7,
 * max 448, no infinities) with a per-tensor scale for each of A and B: 1.0
 * by default, any finite value through pgemm_set_fp8_scales. */
typedef enum {
  PGEMM_F16 = 0,         /* A, B, C: IEEE binary16 */
  PGEMM_BF16 = 1,        /* A, B, C: bfloat16 */
  PGEMM_F8E4M3_BF16 = 2  /* A, B: OCP e4m3 (1 byte); C: bfloat16 */
} pgemm_dtype_t;

/* Tile scheduling modes.
 * NONPERSISTENT: one workgroup per output tile (forum thread, question:
 *   "a thread block for each tile"); grid = number of tiles T.
 * STATIC: a persistent grid of G workgroups (forum thread, question: block
 *   count set to the SM count; first answer: sized so all blocks stay
 *   resident); workgroup w computes tiles w, w+G, w+2G, ... of the tile
 *   order, a deterministic mapping (KernelWiki, "Choosing between static
 *   and CLC scheduling").
 * DYNAMIC: a persistent grid of G workgroups; workgroup w starts on tile
 *   w, then claims further tile ids from a device-wide atomic work counter
 *   until a claim fails, after which it never claims again -- the AMD
 *   analogue of cluster launch control's cancel-and-reuse (KernelWiki,
 *   intro), not a port of it. With G >= T there is nothing to claim and no
 *   claim is made.
 * CANCEL: the grid is one workgroup per tile (T), as in NONPERSISTENT, but
 *   every workgroup claims its tiles -- the first one too -- from the work
 *   counter and keeps claiming until a claim fails. Workgroups that run
 *   early take over the tiles of workgroups that have not started; those
 *   find no tile left when they start and exit at once. This is the closer
 *   analogue of cancel-and-reuse (a grid whose not-yet-launched members'
 *   ids are taken over, same page, intro) and needs no co-residency
 *   assumption; grid_multiple is ignored.
 * STREAMK: tail handling that creates work instead of idling CUs, for
 *   tile counts T that the grid G does not divide (the case the KernelWiki
 *   page's static-vs-CLC guidance leaves open: neither of its schedulers
 *   creates work at the tail). With T = W*G + R, the first W*G tiles of the
 *   tile order run whole, as in STATIC; the k-steps of the last R tiles are
 *   split evenly over the G workgroups (over fewer when pieces would drop
 *   below a minimum length), so every workgroup gets about W + R/G tiles
 *   of work. A workgroup whose piece covers only part of a tile's k-range
 *   writes an fp32 partial tile to a workspace the handle owns. A second
 *   launch on the same stream then adds each split tile's partials in k
 *   order, rounds the sum and stores the tile. G as in STATIC, without the
 *   clamp to T: with T < G (W = 0) the split spreads even a few tiles over
 *   the whole chip. The whole waves run as one STATIC launch over the first
 *   W*G tiles, the tail as a second launch on its own grid, then the fix-up:
 *   up to three launches per run, all on the handle's stream. R = 0 is
 *   exactly STATIC (one launch). Operands that take the generic kernel
 *   (below) run this mode as STATIC. */
typedef enum {
  PGEMM_SCHED_NONPERSISTENT = 0,
  PGEMM_SCHED_STATIC = 1,
  PGEMM_SCHED_DYNAMIC = 2,
  PGEMM_SCHED_CANCEL = 3,
  PGEMM_SCHED_STREAMK = 4
} pgemm_sched_t;

/* Macro-tile configurations of the fast kernel (the Triton persistent-
 * matmul issue tunes BLOCK_SIZE_M/N per problem, "What I've tried").
 * TILE_256: 256 x 256 tiles, 512 threads, one workgroup per CU: the fewest
 *   operand bytes per flop, for problems with many tiles.
 * TILE_128: 128 x 128 tiles, 256 threads, two workgroups per CU: four times
 *   the tiles, so small problems fill the chip and persistent workgroups
 *   get several tiles each.
 * AUTO (default): TILE_128 when 256 x 256 tiles would number fewer than the
 *   CUs (some CUs would idle), else TILE_256. The environment variable PGEMM_TILE (256 or 128)
 *   overrides the default at pgemm_create. */
typedef enum {
  PGEMM_TILE_AUTO = 0,
  PGEMM_TILE_256 = 1,
  PGEMM_TILE_128 = 2
} pgemm_tile_t;

/* Wave schedule of the 256-row fast tile (pgemm_set_mainloop). The value of
 * C does not depend on it: every schedule gives every accumulator the same
 * MFMAs on the same operands in the same order, so C is bitwise the same.
 * LOCKSTEP: all eight waves of a workgroup copy, read and multiply in step,
 *   one barrier per k-step; each step's global -> LDS copy is issued right
 *   after its barrier (the copy/compute overlap of the persistent-kernel
 *   forum thread's first answer, per workgroup).
 * PINGPONG: the two waves of each SIMD run opposite phases: while one issues
 *   copies and reads the next fragments from LDS, the other runs its MFMAs,
 *   and they swap at each barrier (the same overlap, per SIMD; the load role
 *   alternates between the waves instead of being given to a producer wave,
 *   KernelWiki "Persistent Kernels with Cluster Launch Control", tutorial
 *   note on warp specialization).
 * PRODUCER: a dedicated load role (the KernelWiki page's producer-side
 *   request pipeline and its warp-specialization note): waves 4-7 of the
 *   workgroup only copy operand tiles into a three-stage LDS ring and make
 *   the tile claims of the claiming modes, waves 0-3 only read fragments and
 *   run MFMAs. Every wave of a workgroup gets the same register budget on
 *   CDNA, so with four waves copying the tile shrinks to 256 x 128 (T is
 *   counted in those tiles). STREAMK keeps the lockstep 256 x 256 body.
 *   Offered for measurement; AUTO never picks it (measured slower).
 * AUTO (default): PINGPONG for tiles of at least 20 k-steps of 64 for
 *   fp16/bf16 (K >= 1217) and 8 k-steps of 128 for fp8 (K >= 897), LOCKSTEP
 *   below, where its cheaper tile prologue and epilogue win (measured).
 *   The 128 x 128 tile, the generic body and the split tail of STREAMK
 *   always run lockstep. The environment variable PGEMM_MAINLOOP (1, 2 or 3)
 *   overrides the default at pgemm_create. */
typedef enum {
  PGEMM_MAINLOOP_AUTO = 0,
  PGEMM_MAINLOOP_LOCKSTEP = 1,
  PGEMM_MAINLOOP_PINGPONG = 2,
  PGEMM_MAINLOOP_PRODUCER = 3
} pgemm_mainloop_t;

/* Storage of B (pgemm_set_b_layout). The value of C does not depend on it:
 * both layouts feed the MFMAs the same operands in the same order, so C is
 * bitwise the same. */
typedef enum {
  PGEMM_B_KN = 0, /* B[k][n] at B + k*N + n (default) */
  PGEMM_B_NK = 1  /* B[k][n] at B + n*K + k */
} pgemm_b_layout_t;

/* Create a handle on HIP device `device` (which becomes current). Allocates
 * the claiming modes' device work counter (zeroed) and caches the CU count.
 * The handle starts on the null stream. *out is NULL on failure.
 * pgemm_create, pgemm_run and pgemm_destroy are this library's stated
 * interface (the pages specify no API; they fix the operation: forum
 * thread, question); the other entry points complete it. PGEMM_ERR_INVALID_ARG
 * for a NULL out or a device outside [0, device count); PGEMM_ERR_OOM if the
 * handle or the counter cannot be allocated; PGEMM_ERR_HIP if the device
 * cannot be queried. */
int pgemm_create(pgemm_handle_t* out, int device);

/* Bind a hipStream_t (passed as void*; NULL = null stream). Later runs
 * enqueue on it; the caller keeps ownership of the stream, which must
 * outlive its use by the handle. Part of the stated interface's completion
 * (asynchronous runs on a caller's stream). PGEMM_ERR_INVALID_ARG for a
 * NULL handle. */
int pgemm_set_stream(pgemm_handle_t h, void* hip_stream);

/* Enqueue C = A * B on the handle's stream; returns without waiting.
 *   A, B, C: device pointers to contiguous row-major matrices (layouts
 *     above); they must not alias and must stay valid until the work is
 *     done. The caller owns them.
 *   M, N, K: sizes, each in [0, 2^31 - 1]. M == 0 or N == 0: no work, OK.
 *     K == 0: C is filled with zeros (an empty sum).
 *   dtype: pgemm_dtype_t.
 *   sched_mode: pgemm_sched_t.
 *   grid_multiple: persistent modes only (ignored for NONPERSISTENT and
 *     CANCEL).
 *     <= 0: G = occupancy x CU count (all workgroups co-resident, the
 *     sizing of the forum thread's first answer); > 0: G = grid_multiple x
 *     CU count (the NUM_SMS multiple of the Triton issue's follow-up
 *     comment), which may exceed co-residency -- no workgroup waits on
 *     another, so that stays correct. G is clamped to the tile count T
 *     (except in STREAMK, see above).
 * Operands whose K and N are multiples of 16 bytes of elements (8 for
 * fp16/bf16, 16 for fp8) with 16-byte-aligned A, B and C
 * take the fast kernel (256 x 256 or 128 x 128 tiles, pgemm_tile_t);
 * others take a generic 64 x 64 tile kernel with the same schedulers
 * (correct, slower).
 * STREAMK workspace: a run whose split needs more workspace than the handle
 * holds (pgemm_query_streamk) first waits for the handle's stream, frees
 * the old workspace and hipMallocs the new one (PGEMM_ERR_OOM if that
 * fails); later runs of the same or smaller need allocate nothing. Under
 * stream capture, make one such run before capturing. Two runs in flight
 * on one handle share the workspace, which the one-stream-per-handle rule
 * above already orders. */
int pgemm_run(pgemm_handle_t h, const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K,
              int dtype, int sched_mode, int grid_multiple);

/* Wait for the handle's stream, free the work counter, the stream-K
 * workspace and the handle (stated interface). NULL is accepted (no-op).
 * Returns PGEMM_ERR_HIP if the wait or a free failed; the handle is freed
 * either way and must not be used again. */
int pgemm_destroy(pgemm_handle_t h);

/* Size in bytes of the device scratch that pgemm_run_noalloc uses for
 * STREAMK partial tiles (one copy per device, held until the process ends). */
#define PGEMM_NOALLOC_SCRATCH_BYTES (96u << 20)

/* pgemm_run that allocates nothing, for callers that cannot call hipMalloc
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation). Same arguments, semantics, errors and results (bitwise) as
 * pgemm_run, except for where STREAMK keeps its fp32 partial tiles: in a
 * file-scope device array of PGEMM_NOALLOC_SCRATCH_BYTES per device (set up
 * by pgemm_create on the handle's device), not in the handle's workspace.
 * A STREAMK split that needs more (pgemm_query_streamk's workspace_bytes)
 * fails with PGEMM_ERR_UNSUPPORTED before any launch; no other mode needs
 * scratch. The partial tiles are fully written before they are read, so the
 * array needs no clearing between calls. All calls on one device share its
 * array: two STREAMK calls whose work overlaps on the device (on different
 * streams, or different handles) race on it; serialize them (one stream).
 * The call makes no hipMalloc, hipFree or stream synchronization. */
int pgemm_run_noalloc(pgemm_handle_t h, const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K,
                      int dtype, int sched_mode, int grid_multiple);

/* pgemm_run with leading dimensions, for operands that are row-major views
 * inside larger allocations: A[i][k] at A + i*lda + k, B[k][n] at
 * B + k*ldb + n (or, with PGEMM_B_NK, at B + n*ldb + k), C[i][j] at
 * C + i*ldc + j, all counted in elements. pgemm_run is this call with
 * lda = K, ldb = N (K for PGEMM_B_NK) and ldc = N. Requires ldc >= N and,
 * when K > 0, lda >= K and ldb >= the length of B's rows (N, or K for
 * PGEMM_B_NK); each below 2^31; else PGEMM_ERR_INVALID_ARG. Only the M x N
 * window of C is written. The fast kernel additionally needs lda and ldb
 * to be multiples of 16 bytes of elements and ldc a multiple of 8 (16-byte
 * rows of C); otherwise the generic kernel runs. Leading dimensions whose
 * tile spans exceed 32-bit buffer offsets give PGEMM_ERR_UNSUPPORTED.
 * Everything else is as for pgemm_run. */
int pgemm_run_ld(pgemm_handle_t h, const void* A, int64_t lda, const void* B, int64_t ldb, void* C, int64_t ldc,
                 int64_t M, int64_t N, int64_t K, int dtype, int sched_mode, int grid_multiple);

/* Watchdog wait: poll the handle's stream (hipStreamQuery, about every
 * 50 microseconds) until all work enqueued on it has finished, or until
 * timeout_ms milliseconds have passed. Returns PGEMM_OK when the stream is
 * idle, PGEMM_ERR_TIMEOUT when the deadline passed first (the work keeps
 * running; the caller may wait again), PGEMM_ERR_HIP if the stream reports
 * an error (e.g. a kernel fault), PGEMM_ERR_INVALID_ARG for a NULL handle
 * or a negative timeout. Lets a harness notice a kernel that never ends
 * instead of blocking in a synchronize. */
int pgemm_wait(pgemm_handle_t h, int timeout_ms);

/* Static text for a status code (never NULL; unknown codes give
 * "PGEMM_ERR_UNKNOWN"). Error reporting of the stated interface: every
 * entry point returns a status instead of raising. */
const char* pgemm_status_string(int status);

/* Detail of the last failure on this handle ("" if none; "invalid handle"
 * for NULL). Owned by the handle, valid until the next call on it. Error
 * reporting of the stated interface. */
const char* pgemm_last_error(pgemm_handle_t h);

/* ---- checking and reporting (not for timed runs) ---------------------- */

/* Attach a caller-owned device int32 array of n_tiles entries. Each run
 * then atomically adds 1 to visits[t] after tile t's C store, so after a
 * run from zeroed memory every entry must read exactly 1 (every tile
 * written exactly once). dev_visits == NULL detaches. Runs whose tile
 * count exceeds n_tiles fail with PGEMM_ERR_INVALID_ARG. */
int pgemm_set_tile_counter(pgemm_handle_t h, int32_t* dev_visits, int64_t n_tiles);

/* Attach a caller-owned device int32 array of n_tiles entries; each run
 * writes owner[t] = the id of the workgroup that computed tile t. NULL
 * detaches. Same size rule as the visit counter. In STREAMK the W*G
 * whole-wave tiles are logged by workgroup id of that launch (t mod G), a
 * tail tile computed whole by the id of its workgroup in the tail launch,
 * and a split tile, stored by the fix-up launch, as -1 - s (s = the tile's
 * index among the R tail tiles); the visit counter counts that store, so
 * every tile still reads 1. */
int pgemm_set_owner_log(pgemm_handle_t h, int32_t* dev_owner, int64_t n_tiles);

/* Attach a caller-owned device int64 array of 4 * n_tiles entries: the
 * tile trace, used to draw per-workgroup timelines of the tail effect
 * (KernelWiki "Persistent Kernels with Cluster Launch Control", "Choosing
 * between static and CLC scheduling": the last wave of tiles leaves part
 * of the chip idle). Each run writes, for every tile t,
 *   trace[4t+0]  id of the workgroup that stored tile t (the owner-log
 *                convention: -1 - s for a STREAMK split tile, which the
 *                fix-up launch stores),
 *   trace[4t+1]  id of the XCD (0..7) whose CU ran that workgroup,
 *   trace[4t+2]  start: when that workgroup began the tile (its k-loop),
 *   trace[4t+3]  end: after the tile's C store was issued,
 * the times in ticks of the device's constant-rate clock (see
 * pgemm_clock_khz). For a split tile, start and end bracket its fix-up.
 * The trace adds a clock read and a few stores per tile: leave it off in
 * timed runs. NULL detaches. Runs whose tile count exceeds n_tiles fail
 * with PGEMM_ERR_INVALID_ARG before launching. */
int pgemm_set_tile_trace(pgemm_handle_t h, int64_t* dev_trace, int64_t n_tiles);

/* Rate in kHz of the constant-rate clock that stamps the tile trace, for
 * device `device`. PGEMM_ERR_INVALID_ARG if khz is NULL, PGEMM_ERR_HIP if
 * the device cannot be queried. */
int pgemm_clock_khz(int device, int* khz);

/* Report how pgemm_run would launch this problem, without launching:
 * tile count, grid size, occupancy (workgroups per CU), macro tile
 * (bm x bn, k-step bk in elements), and the tile body of the launch that
 * computes the whole tiles: 0 = the generic kernel (unaligned sizes),
 * 1 = the fast kernel with lockstep waves, 2 = the fast kernel in ping-pong,
 * 3 = the fast kernel with producer waves (pgemm_mainloop_t). Output
 * pointers may be NULL. Alignment is judged from
 * the sizes only (pointers assumed 16-byte aligned). */
int pgemm_query_launch(pgemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int sched_mode,
                       int grid_multiple, int* tiles, int* grid, int* occupancy, int* bm, int* bn, int* bk,
                       int* body);

/* Report the STREAMK split pgemm_run would use for this problem, without
 * launching: whole_tiles = W*G tiles run whole, split_tiles = R tail
 * tiles whose k-steps are split, split_groups = workgroups sharing them,
 * pieces_split = tail tiles actually cut into two or more pieces (0: no
 * fix-up launch), workspace_bytes = the workspace the run needs (0 when
 * nothing is cut). Output pointers may be NULL. Operands that take the
 * generic kernel report split_tiles = 0. */
int pgemm_query_streamk(pgemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int grid_multiple,
                        int* whole_tiles, int* split_tiles, int* split_groups, int* pieces_split,
                        int64_t* workspace_bytes);

/* Tile-order knobs: GROUP_SIZE_M of the grouped order (default 4; the
 * Triton issue's setting is 8; 1 = row-major), and the XCD-aware remap
 * (1 = on; 0 = off; -1 = automatic, the default: on for launches with more
 * tiles than the device has CUs, off otherwise). Both apply identically to
 * all modes and never change C's bits, only which workgroup computes which
 * tile. The environment variables PGEMM_GROUP_M and PGEMM_XCD_REMAP override
 * the defaults at pgemm_create. */
int pgemm_set_tile_order(pgemm_handle_t h, int group_m, int xcd_remap);

/* Choose the fast kernel's macro tile for later runs on this handle
 * (pgemm_tile_t). Unaligned operands always take the generic 64 x 64 body.
 * Returns PGEMM_ERR_INVALID_ARG for an unknown value. */
int pgemm_set_tile_config(pgemm_handle_t h, int tile);

/* Per-tensor scales of e4m3 A and B for later PGEMM_F8E4M3_BF16 runs on this
 * handle: the stored codes represent scale_a * dec(a) and scale_b * dec(b),
 * so C[i][j] = scale_a * scale_b * sum_k dec(A[i][k]) * dec(B[k][j]). The
 * epilogue multiplies the fp32 sum by the fp32 product scale_a * scale_b and
 * rounds to bf16 (nearest-even); with power-of-two scales that product and
 * multiplication are exact. Default 1.0 and 1.0 (exact: C unchanged). Other
 * dtypes ignore the scales. PGEMM_ERR_INVALID_ARG for a NULL handle, a
 * non-finite scale or a non-finite product. */
int pgemm_set_fp8_scales(pgemm_handle_t h, float scale_a, float scale_b);

/* Choose the wave schedule of the 256-row tile for later runs on this
 * handle (pgemm_mainloop_t; C's bits do not depend on it). Returns
 * PGEMM_ERR_INVALID_ARG for a NULL handle or an unknown value. */
int pgemm_set_mainloop(pgemm_handle_t h, int mainloop);

/* Choose how B is stored for later runs on this handle (pgemm_b_layout_t;
 * default PGEMM_B_KN). With PGEMM_B_NK the fast kernel copies B's tile like
 * A's (rows of 128 bytes) and reads its fragments with plain 16-byte LDS
 * reads instead of LDS transpose reads. The fast-kernel size rule is the
 * same in both layouts (K and N multiples of 16 bytes of elements).
 * Returns PGEMM_ERR_INVALID_ARG for a NULL handle or an unknown value. */
int pgemm_set_b_layout(pgemm_handle_t h, int layout);

/* Host mirror of the device tile order: (pid_m, pid_n) of tile t for an
 * n_m x n_n tile grid, with the same knobs and CU-count chunking the
 * device uses (cu_chunk = CU count, or 0 for no XCD remap). Pure function,
 * no GPU needed. */
int pgemm_tile_coords(int64_t t, int64_t n_m, int64_t n_n, int group_m, int cu_chunk, int* pid_m,
                      int* pid_n);

/* Read the device work counter of the claiming modes (synchronizes the
 * handle's stream). It reads 0 between launches -- each launch's last claim
 * resets it -- so any other value means a launch was cut short. */
int pgemm_read_work_counter(pgemm_handle_t h, int32_t* value);

/* ---- token rows to their experts and back ------------------------------ */
/*
 * The steps around the per-expert products of a mixture-of-experts layer.
 * T tokens name k experts each; slot s = t*k + j is choice j of token t,
 * n = T*k. A slot whose id lies outside [0, E) is dropped: it has no row, no
 * share in any sum and no gradient, whatever its weight holds. Kept slots are
 * sorted by expert, slots of one expert in slot order (a stable sort, so
 * every result is the same on every run):
 *   offsets[e]  first sorted row of expert e, e = 0..E; offsets[E] = kept slots
 *   order[p]    slot of sorted row p, -1 for p >= offsets[E]
 *   pos[s]      sorted row of slot s, -1 for a dropped slot
 * All three are int32 device arrays. dtype is PGEMM_F16 or PGEMM_BF16; rows
 * are 16-bit elements, ld* is the distance of two rows in elements (0 repeats
 * one row; it may be smaller or larger than H), outputs are contiguous. Sums
 * are fp32, rounded once to nearest even. Rows of any length and any even
 * address are taken; those of a multiple of 8 elements at 16-byte addresses
 * are the fastest. All work is enqueued on the handle's stream; nothing is
 * allocated. Entries of pos outside [0, n) count as dropped.
 * PGEMM_ERR_INVALID_ARG for a NULL handle or needed pointer, a negative size,
 * k < 1, E < 1, an unknown type or too small a workspace;
 * PGEMM_ERR_UNSUPPORTED for n or H above 2^30, E above 1024, or more tokens than
 * one launch takes (2^26 of up to 1024 elements, 2^24 of more). */

/* Integer type of the expert ids. */
typedef enum { PGEMM_IDS_I32 = 0, PGEMM_IDS_I64 = 1 } pgemm_ids_t;

/* Bytes of device scratch that pgemm_moe_dispatch needs for these sizes (0
 * for few slots). A pure function. */
int pgemm_moe_dispatch_workspace(int64_t T, int64_t k, int64_t E, int64_t* bytes);

/* Sort the slots and move the rows: xs[p] = x[order[p] / k], zeros where
 * order[p] = -1. x: T rows of H; ids: [T, k] contiguous; xs: [n, H]. offsets
 * is written for T = 0 too. `work` is device memory of at least the bytes
 * above, free again once the call's work is done. */
int pgemm_moe_dispatch(pgemm_handle_t h, const void* x, int64_t ldx, const void* ids, int ids_type, int64_t T, int64_t k,
                       int64_t E, int64_t H, int dtype, int32_t* offsets, int32_t* order, int32_t* pos, void* xs,
                       void* work, int64_t work_bytes);

/* Gradient of the rows: dx[t] = sum of dxs[pos[t*k + j]] over the token's
 * kept slots, in the order of j. dxs: n rows of H; dx: [T, H]. */
int pgemm_moe_dispatch_backward(pgemm_handle_t h, const void* dxs, int64_t lddxs, const int32_t* pos, int64_t T,
                                int64_t k, int64_t H, int dtype, void* dx);

/* Back to the tokens: out[t] = sum of w[t*k + j] * ys[pos[t*k + j]] over the
 * token's kept slots. ys: n rows of H; w: [T, k] fp32; out: [T, H]. */
int pgemm_moe_combine(pgemm_handle_t h, const void* ys, int64_t ldys, const float* w, const int32_t* pos, int64_t T,
                      int64_t k, int64_t H, int dtype, void* out);

/* Its gradients: dys[pos[s]] = w[s] * dout[t] (zeros in the rows from
 * offsets[E] on) and dw[s] = <ys[pos[s]], dout[t]> in fp32 (0 for a dropped
 * slot), s = t*k + j. dout: T rows of H; dys: [n, H]; dw: [T, k]. For a plan as
 * the sort left it: rows below offsets[E] that no entry of pos names are not
 * written. */
int pgemm_moe_combine_backward(pgemm_handle_t h, const void* dout, int64_t lddout, const void* ys, int64_t ldys,
                               const float* w, const int32_t* offsets, const int32_t* pos, int64_t T, int64_t k,
                               int64_t E, int64_t H, int dtype, void* dys, float* dw);

/* The same for a plan from which slots were taken after the sort, by setting
 * their pos outside [0, n) (for instance where an expert has more rows than it
 * may take): zeros too in a row whose slot, by order, has no place any more. */
int pgemm_moe_combine_backward_plan(pgemm_handle_t h, const void* dout, int64_t lddout, const void* ys, int64_t ldys,
                                    const float* w, const int32_t* offsets, const int32_t* order, const int32_t* pos,
                                    int64_t T, int64_t k, int64_t E, int64_t H, int dtype, void* dys, float* dw);

/* ---- products of rows sorted by expert ---------------------------------- */
/*
 * offsets: E + 1 ascending row bounds on the device (those of
 * pgemm_moe_dispatch), rows offsets[e]..offsets[e+1]-1 belonging to expert e.
 * The host never reads them, so a call can be captured and replayed with
 * other bounds. dtype is PGEMM_F16 or PGEMM_BF16; ld* is the distance of two
 * rows in elements (0 repeats one row), w and the outputs are contiguous.
 * Sums are fp32, rounded once, and the same on every run. Sizes may be odd, and
 * addresses any that elements have; K and N of a multiple of 8 with rows at 16-byte
 * addresses are the fastest. Nothing is allocated.
 * PGEMM_ERR_INVALID_ARG for a NULL handle or needed pointer, a negative size,
 * E < 1, an unknown layout or type; PGEMM_ERR_UNSUPPORTED for sizes above
 * 2^30, E above 1024 or more output tiles than one launch takes (2^23). */

/* Enqueue y[r] = x[r] * w[e(r)]. x: R rows of K; w: [E, K, N] for PGEMM_B_KN,
 * [E, N, K] for PGEMM_B_NK; y: [R, N], zeros in rows of no expert (whatever x
 * holds there) and for K = 0. The gradient of x is the same call on y's
 * gradient with K and N exchanged and the other layout. */
int pgemm_grouped_run(pgemm_handle_t h, const void* x, int64_t ldx, const void* w, const int32_t* offsets, void* y,
                      int64_t R, int64_t E, int64_t K, int64_t N, int layout, int dtype);

/* Enqueue c[e] = sum over the rows r of expert e of a[r]^T * b[r], zeros for
 * an expert without rows. a: R rows of I; b: R rows of J; c: [E, I, J]. The
 * gradient of w: (a, b) = (x, dy) for PGEMM_B_KN, (dy, x) for PGEMM_B_NK.
 * With few output tiles the rows are cut into pieces whose fp32 sums meet in
 * `work` (at least the bytes below, free again once the call's work is done)
 * and are added in order. */
int pgemm_grouped_weight_grad(pgemm_handle_t h, const void* a, int64_t lda, const void* b, int64_t ldb,
                              const int32_t* offsets, void* c, int64_t R, int64_t E, int64_t I, int64_t J, int dtype,
                              void* work, int64_t work_bytes);

/* Bytes of device scratch that pgemm_grouped_weight_grad needs for these
 * sizes, at a multiple of 16 (0 where no expert's rows are cut into pieces).
 * A pure function. */
int pgemm_grouped_weight_grad_workspace(int64_t R, int64_t E, int64_t I, int64_t J, int64_t* bytes);

/* Body of a grouped product. ANY: 128 x 128 tiles, operands of any alignment;
 * PINGPONG: 256 x 256 tiles, persistent; FEW16, FEW16_WIDE, FEW32_WIDE: 16 or 32
 * rows at once (WIDE: two column blocks of N x K matrices); FEW_GRAD: the weight
 * gradient of few rows. */
typedef enum {
  PGEMM_GROUPED_ANY = 0,
  PGEMM_GROUPED_PINGPONG = 1,
  PGEMM_GROUPED_FEW16 = 2,
  PGEMM_GROUPED_FEW16_WIDE = 3,
  PGEMM_GROUPED_FEW32_WIDE = 4,
  PGEMM_GROUPED_FEW_GRAD = 5
} pgemm_grouped_body_t;

/* Report the body that pgemm_grouped_run would launch. `wide` tells whether
 * every operand's rows lie at 16-byte addresses (which PINGPONG needs, next to
 * K and N of a multiple of 8). A pure function. PGEMM_ERR_INVALID_ARG for a
 * NULL pointer, a size below 1 or an unknown layout. */
int pgemm_grouped_query(int64_t R, int64_t E, int64_t K, int64_t N, int layout, int wide, int* body);

/* The same for pgemm_grouped_weight_grad, and the pieces an expert's rows are
 * cut into. */
int pgemm_grouped_weight_grad_query(int64_t R, int64_t E, int64_t I, int64_t J, int wide, int* body, int* pieces);

/* ---- few rows times 4-bit weights -------------------------------------- */

/* Format of the 4-bit codes. INT4: whole numbers 0..15 less a zero point;
 * E2M1: sign, two exponent bits (bias 1), one mantissa bit: 0, 0.5, 1, 1.5,
 * 2, 3, 4, 6 and their negatives. */
typedef enum { PGEMM_W4_INT4 = 0, PGEMM_W4_E2M1 = 1 } pgemm_w4_format_t;

/* Enqueue y = x * dec(q)^T on the handle's stream, for the few rows of a
 * decoding batch (any number is computed; each 32 read the weights again).
 *   x: M rows of K elements, ldx apart (0 repeats one row); y: [M, N].
 *   q: [E, N, ceil(K / 2)] bytes, code k of a row in byte k / 2, the even one
 *     in the low nibble; a last half byte is ignored.
 *   scales: [E, N, ceil(K / group)] of x's type, one for each `group` (32, 64
 *     or 128) elements along K.
 *   zeros: int4 zero points, uint8 of the same shape, their low four bits;
 *     NULL: 8. E2M1 has none.
 *   offsets: NULL: one matrix for all rows (E = 1); else E + 1 ascending row
 *     bounds on the device, rows offsets[e]..offsets[e+1]-1 belonging to
 *     matrix e; rows of none give zeros.
 *   dtype: PGEMM_F16 or PGEMM_BF16, of x, scales and y.
 * Each weight is (code - zero) * scale or e2m1(code) * scale, never rounded:
 * the sum of a group is formed in fp32 from exact products, multiplied by its
 * scale in fp32, and y is rounded once. K = 0 gives zeros. Nothing is
 * allocated; pointers may have any alignment their elements have.
 * PGEMM_ERR_INVALID_ARG for a NULL handle or needed pointer, a negative size,
 * an unknown group, format or type, zeros with E2M1, or E > 1 without
 * offsets; PGEMM_ERR_UNSUPPORTED for sizes above 2^30, E above 65534 or N above
 * what one launch takes (2^27). */
int pgemm_w4_run(pgemm_handle_t h, const void* x, int64_t ldx, const void* q, const void* scales, const void* zeros,
                 const int32_t* offsets, void* y, int64_t M, int64_t N, int64_t K, int64_t E, int group, int fmt,
                 int dtype);

/* Report the form that pgemm_w4_run would launch on a device of `cus` CUs:
 * rows of x at once (4, 16 or 32) and blocks of 16 columns a wave takes (1 or
 * 2). `experts`: nonzero with offsets. A pure function. PGEMM_ERR_INVALID_ARG
 * for a NULL pointer or a size below 1. */
int pgemm_w4_query(int64_t M, int64_t N, int64_t E, int experts, int cus, int* rows, int* blocks);

/* ---- the linear layer -------------------------------------------------- */
/*
 * z = x W + bias, y = act(z) + residual; gated: W and bias have 2N columns,
 * the gate's first, and y = act(z[:, :N]) * z[:, N:] + residual. C below is the
 * number of W's columns, N or 2N.
 *   x: M rows of K; W: [K, C] for PGEMM_B_KN, [C, K] for PGEMM_B_NK, rows ldw
 *   apart; bias: [C]; residual: M rows of N; y: [M, N]; z: [M, C], contiguous.
 * dtype is PGEMM_F16 or PGEMM_BF16, of every matrix and vector. ld* is the
 * distance of two rows in elements (0 repeats one row). Sums, activations and
 * column sums are fp32; y, z and each gradient are rounded once (dz, the
 * gradient of z, too: it is an operand of the two products), the same on every
 * run. Sizes may be odd and addresses any that elements have; rows of a multiple
 * of 8 elements at 16-byte addresses are the fastest (others are moved to the
 * workspace first, but by the few-row bodies). `work` is device memory at a multiple of
 * 16, of at least the bytes that the workspace functions report, free again
 * once the call's work is done; nothing is allocated. Empty sums give the
 * epilogue of zero. An fp16 z beyond 65504 is stored as that (y is formed from
 * the fp32 sum all the same): without a gate its gradient is the true one, gated
 * the other half's is that of 65504. An infinite sum stays infinite, and has a
 * NaN gradient but for PGEMM_ACT_NONE and PGEMM_ACT_RELU. fp16 outputs, and dz,
 * are infinite where they exceed 65504, and so are the sums that read such a dz.
 * PGEMM_ERR_INVALID_ARG for a NULL handle or needed pointer, a negative size or
 * stride, an unknown layout, activation or type, or too small a workspace;
 * PGEMM_ERR_UNSUPPORTED for K or C above 2^21 or more tiles than one launch
 * takes (2^21 of 64 x 128, of any two of M, C, K). */

/* Activations. GELU: x Phi(x); GELU_TANH: its form with tanh; SILU: x / (1 + exp(-x)). */
typedef enum {
  PGEMM_ACT_NONE = 0,
  PGEMM_ACT_RELU = 1,
  PGEMM_ACT_GELU = 2,
  PGEMM_ACT_GELU_TANH = 3,
  PGEMM_ACT_SILU = 4
} pgemm_act_t;

/* Enqueue y, and z unless it is NULL. bias and residual may be NULL. */
int pgemm_dense_run(pgemm_handle_t h, const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                    const void* residual, int64_t ldr, void* y, void* z, int64_t M, int64_t N, int64_t K, int layout,
                    int act, int gated, int dtype, void* work, int64_t work_bytes);

/* Bytes of scratch that pgemm_dense_run needs. `wide` tells whether the rows of
 * x and W lie at 16-byte addresses, at most 2^21 elements apart. A pure function. */
int pgemm_dense_workspace(int64_t M, int64_t N, int64_t K, int layout, int gated, int wide, int64_t* bytes);

/* Enqueue the gradients from that of y: dx [M, K], dw like W (contiguous), db
 * [C], each unless it is NULL. z as pgemm_dense_run left it (NULL for
 * PGEMM_ACT_NONE without a gate). The residual's gradient is dy itself. */
int pgemm_dense_backward(pgemm_handle_t h, const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w,
                         int64_t ldw, const void* z, void* dx, void* dw, void* db, int64_t M, int64_t N, int64_t K,
                         int layout, int act, int gated, int dtype, void* work, int64_t work_bytes);

/* Gradients asked for, added up. */
typedef enum { PGEMM_DENSE_DX = 1, PGEMM_DENSE_DW = 2, PGEMM_DENSE_DB = 4 } pgemm_dense_needs_t;

/* Bytes of scratch that pgemm_dense_backward needs for these gradients; `wide`
 * as above, for dy, x and W. A pure function. */
int pgemm_dense_backward_workspace(int64_t M, int64_t N, int64_t K, int layout, int act, int gated, int needs, int wide,
                                   int64_t* bytes);

/* Body of a product of the linear layer. FEW8, FEW16, FEW32: so many rows at
 * once; TILE64, TILE128: tiles of 64 or 128 x 128; TILE128_PAIR: the same, two
 * to a CU; PINGPONG: 256 x 256 tiles, persistent. */
typedef enum {
  PGEMM_DENSE_FEW8 = 0,
  PGEMM_DENSE_FEW16 = 1,
  PGEMM_DENSE_FEW32 = 2,
  PGEMM_DENSE_TILE64 = 3,
  PGEMM_DENSE_TILE128 = 4,
  PGEMM_DENSE_TILE128_PAIR = 5,
  PGEMM_DENSE_PINGPONG = 6
} pgemm_dense_body_t;

/* Report the body that pgemm_dense_run would launch and the pieces it cuts the
 * sum into. (The gradient of x is the product of M, K, C with the other layout
 * and no gate.) Pure functions. PGEMM_ERR_INVALID_ARG for a NULL pointer or a
 * size below 1. */
int pgemm_dense_query(int64_t M, int64_t N, int64_t K, int layout, int gated, int* body, int* pieces);

/* The same for the gradient of W: [I, J] = a^T b over R rows. */
int pgemm_dense_weight_grad_query(int64_t R, int64_t I, int64_t J, int* body, int* pieces);

/* Whether the gradients of x and W, both asked for, go into one launch: its body
 * and each one's pieces (which each keeps where it alone is asked for, so that
 * its values stay the same); a body of -1 for two, as the queries above tell them. */
int pgemm_dense_gradients_query(int64_t M, int64_t C, int64_t K, int layout, int* body, int* pieces_dx, int* pieces_dw);

/* ---- the router, and a routed layer of few tokens ----------------------- */

/* Type of the router's logits. */
typedef enum { PGEMM_LOGITS_F16 = 0, PGEMM_LOGITS_BF16 = 1, PGEMM_LOGITS_F32 = 3 } pgemm_logits_t;

/* Scores: softmax over the experts, or each logit's sigmoid. */
typedef enum { PGEMM_SCORE_SOFTMAX = 0, PGEMM_SCORE_SIGMOID = 1 } pgemm_score_t;

/* Enqueue the choice of each token's k experts: ids[t] the k largest of the
 * token's E logits, largest first and the first of equal ones first, weights[t]
 * their scores, with `normalize` divided by the chosen scores' sum. Logits of
 * -inf or NaN are never chosen (their scores are 0); where a token has fewer
 * than k others, the places left get the id -1 and the weight 0, which
 * pgemm_moe_dispatch drops. A logit of +inf gives NaN weights.
 *   logits: T rows of E, ld apart; ids int32 and weights fp32: [T, k].
 * All sums and exponentials are fp32. PGEMM_ERR_INVALID_ARG for a NULL handle
 * or pointer, a negative size, E < 1, k outside [1, E], an unknown type or
 * score; PGEMM_ERR_UNSUPPORTED for T above 2^24, E above 1024 or k above 64. */
int pgemm_moe_route(pgemm_handle_t h, const void* logits, int64_t ld, int type, int64_t T, int64_t E, int64_t k, int score,
                    int normalize, int32_t* ids, float* weights);

/* Its gradient: dlogits [T, E], of the logits' type, from the gradient of the
 * weights [T, k], with the call's logits, ids and weights. Places with an id
 * outside [0, E) have none, whatever their dweights hold. */
int pgemm_moe_route_backward(pgemm_handle_t h, const float* dweights, const void* logits, int64_t ld, int type,
                             const int32_t* ids, const float* weights, int64_t T, int64_t E, int64_t k, int score,
                             int normalize, void* dlogits);

/* Enqueue a whole routed layer for few tokens, two launches for each 64:
 *   out[t] = sum over j of weights[t, j] * (a(x[t]) W_out[e]^T), e = ids[t, j],
 *   a(x) = act(x W_in[e]^T), gated: act of its first I columns times the others.
 *   x: T rows of H, ldx apart; ids: [T, k] contiguous (outside [0, E): dropped;
 *   an expert named twice counts twice); weights: fp32 [T, k]; w_in: [E, I, H],
 *   gated [E, 2I, H]; w_out: [E, H, I]; out: [T, H].
 * Only the experts that a token names are read: once for each 16, 32 or 64 of
 * the tokens that name one (the mean number of them decides which), so an expert
 * that all of 64 tokens name is read up to four times. Sums are fp32 in an order
 * that the ids of the pass's 64 tokens fix, so a token's last bits may depend on
 * the ids of those beside it; a(x) and out are rounded once (an fp16 a(x) beyond
 * 65504 is infinite, and so then is what it is summed into). `work` as for the
 * linear layer; nothing is allocated. dtype is PGEMM_F16 or PGEMM_BF16.
 * PGEMM_ERR_INVALID_ARG for a NULL handle or needed pointer, a negative size,
 * k < 1, E < 1, an unknown type or activation or too small a workspace;
 * PGEMM_ERR_UNSUPPORTED for T above 4096, k above 32, E above 1024, H above
 * 2^20 or I above 2^19. */
int pgemm_moe_layer(pgemm_handle_t h, const void* x, int64_t ldx, const void* ids, int ids_type, const float* weights,
                    const void* w_in, const void* w_out, void* out, int64_t T, int64_t k, int64_t E, int64_t H, int64_t I,
                    int act, int gated, int dtype, void* work, int64_t work_bytes);

/* Bytes of scratch that it needs. A pure function. */
int pgemm_moe_layer_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int64_t* bytes);

/* Benchmark aid, not part of the GEMM: make about `n_cus` CUs of device
 * `device` unavailable for about `microseconds`, asynchronously on the HIP
 * stream `hip_stream` (NULL = null stream). It launches n_cus workgroups
 * that each hold a whole CU's LDS (so no GEMM workgroup can share that CU)
 * and idle until the device's constant-rate clock has advanced by the
 * given time; the wait is also capped by a pass count, so the kernel ends
 * even if that clock stalled. Used to measure the schedulers when only part
 * of the GPU is available (KernelWiki "Persistent Kernels with Cluster
 * Launch Control", "Choosing between static and CLC scheduling"). n_cus in
 * [0, 65536], microseconds in [0, 10^6], else PGEMM_ERR_INVALID_ARG; 0 for
 * either launches nothing. */
int pgemm_hold_cus(void* hip_stream, int device, int n_cus, int microseconds);

#ifdef __cplusplus
}
#endif

#endif /* PGEMM_H */
