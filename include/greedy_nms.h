/*
 * greedy_nms.h -- C ABI of the MI355X (gfx950) greedy IoU non-maximum
 * suppression library (libgreedy_nms.so).
 *
 * What the library computes.  Greedy NMS as described on "LeetCUDA 14-nms"
 * (introduction and "algorithm and data flow"): visit the boxes by score,
 * highest first, with equal scores in ascending input order (stable sort);
 * keep a box unless an already-kept box of its group overlaps it with
 * IoU > iou_thresh (strictly); return the kept boxes as their original input
 * indices (that page's bug-3 fix), int64, in visiting order.  A group is the
 * pair (image, class): boxes of different images or classes never suppress
 * each other (the class check of "YOLOv5 post-processing GPU port",
 * section 2.2, extended to images).  With several groups the result is one
 * list over all boxes in global score order, with global indices.
 *
 * The IoU is this float32 expression, one IEEE binary32 operation per step,
 * no fused multiply-add (none of the pages prints its IoU routine; this
 * expression is the one the library fixes):
 *     area  = (x2 - x1) * (y2 - y1)
 *     w     = max(min(x2i, x2j) - max(x1i, x1j), 0)
 *     h     = max(min(y2i, y2j) - max(y1i, y1j), 0)
 *     inter = w * h
 *     union = (area_i + area_j) - inter
 *     suppress  iff  inter / union > iou_thresh      (correctly rounded)
 * No clipping or reordering of coordinates is applied.
 *
 * Memory.  Every pointer argument named "device" is HIP device memory on the
 * current device; the caller allocates and owns every buffer (inputs, output,
 * workspace).  The library allocates no device memory, keeps no pointer to a
 * caller's buffer after a call returns and holds no device state between
 * calls, so calls on different streams with distinct workspaces may run
 * concurrently.  What the library does allocate, and keeps:
 *   - pinned host buffers of 40 bytes (hipHostMalloc) into which a call's
 *     last kernel posts the kept count, the device-detected errors and the
 *     call's tag: a process-wide pool of at most 64, one per call running at
 *     that moment, allocated when every existing one is in use and kept
 *     until the process ends (past 64 concurrent calls the call copies the
 *     control block back into pageable memory instead);
 *   - per profiled call (the *_profiled variants), HIP events, created and
 *     destroyed inside the call;
 *   - for nms_f32_static, a statically sized device array in the library's
 *     code object (see there).
 * No library code runs at process exit (no static or thread-local object
 * has a destructor).
 *
 * Streams.  `stream` is a hipStream_t (NULL = the default stream).  All work
 * is enqueued on it.  The selection operators at the end of this header
 * return at once; each other nms_* compute call returns once its result is
 * complete: its last kernel posts the result into a pinned buffer of the
 * pool and the host spins on it (for up to 2 ms, then it blocks in
 * hipStreamSynchronize); the profiled variants, nms_f32_static and calls
 * past the pool copy the control block back and synchronise the stream
 * instead.  Either way, when the call returns *num_kept (a host pointer)
 * is valid and every write of the call to keep_out and the workspace has
 * completed (its last kernel may still be retiring; it writes nothing
 * more).  Inputs must not change until the call returns.
 *
 * Errors.  No exception crosses the ABI.  Every call returns an nms_status;
 * on any status other than NMS_OK, *num_kept (when given) is 0 and keep_out is
 * unspecified.  Device-detected errors (non-finite input, bad offsets) arrive
 * with the same read-back that carries the kept count.
 */
#ifndef GREEDY_NMS_H
#define GREEDY_NMS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum nms_status {
    NMS_OK = 0,
    /* A null pointer with n > 0, n < 0, iou_thresh NaN, num_images
     * inconsistent with batch_offsets, or a misaligned boxes pointer. */
    NMS_INVALID_ARG = 1,
    /* workspace_bytes is below what nms_workspace_size reports (one image:
     * below nms_workspace_size_lists, or below nms_workspace_size for an
     * input that needs the dense bitmask). */
    NMS_WORKSPACE_TOO_SMALL = 2,
    /* A NaN score or a non-finite box coordinate (detected on the device). */
    NMS_NONFINITE_INPUT = 3,
    /* batch_offsets not non-decreasing from 0 to n (detected on the device). */
    NMS_BAD_OFFSETS = 4,
    /* n above NMS_MAX_BOXES. */
    NMS_TOO_LARGE = 5,
    /* A HIP runtime call or kernel launch failed. */
    NMS_HIP_ERROR = 6,
    /* Matrix NMS: a box with x1 > x2 or y1 > y2 (detected on the device). */
    NMS_BAD_BOXES = 7
} nms_status;

/* Largest n accepted: one workgroup keeps the removed bitmap (n/8 bytes) in
 * at most 64 KiB of LDS during the sweep. */
#define NMS_MAX_BOXES 512000

/* Stages timed by nms_f32_profiled, in launch order. */
#define NMS_STAGE_SORT 0     /* score keys, stable LSD radix sort, grouping  */
#define NMS_STAGE_GATHER 1   /* sorted box gather + areas + input checks     */
#define NMS_STAGE_MASK 2     /* triangle-tiled IoU suppression bitmask; one  */
                             /* image of 32705 to 262144 boxes: mask and     */
                             /* sweep in one launch (sweep overlaps mask);   */
                             /* the one-launch path for small inputs: the    */
                             /* whole call, timed here                       */
#define NMS_STAGE_SWEEP 3    /* greedy sweep over the mask (+ compaction);   */
                             /* after the fused launch, only its completion  */
                             /* check (or the sweep, if a tile's list of     */
                             /* nonzero words overflowed)                    */
#define NMS_STAGE_COMPACT 4  /* score-order compaction (grouped input only)  */
#define NMS_NUM_STAGES 5

/*
 * nms_workspace_size -- device workspace needed by nms_f32 for n boxes.
 *   n            number of boxes (0 <= n <= NMS_MAX_BOXES)
 *   num_images   number of images in batch_offsets (0 or 1 when there are
 *                none); has_classes: nonzero when class_ids will be given.
 *   *bytes       receives the size; it is a bound computed from n alone
 *                (dominated by the n * ceil(n/64) * 8-byte suppression
 *                bitmask), so no device synchronisation is needed.
 * Returns NMS_OK, NMS_INVALID_ARG (bytes NULL, n < 0) or NMS_TOO_LARGE.
 * Why a bound from n alone: sizing a buffer from the data costs a device
 * round trip before the work can start ("LeetCUDA 12-histogram", its binding
 * section: the max() read back to size the histogram is a forced device
 * synchronisation, which a caller-chosen size avoids).  Our reading: the
 * caller sizes the workspace once from n and reuses it.
 */
nms_status nms_workspace_size(int64_t n, int64_t num_images, int has_classes, size_t *bytes);

/*
 * nms_workspace_size_lists -- a smaller workspace for one image of n boxes:
 * everything but the dense suppression bitmask: about 530 bytes per box,
 * most of it the lists of nonzero mask words (24 KiB per 64 boxes), against
 * n * ceil(n/64) * 8 more bytes for the bitmask (35 MB instead of 572 MB at
 * 65,536 boxes, 273 MB instead of 33 GB at 512,000).
 *   n       number of boxes (0 <= n <= NMS_MAX_BOXES); *bytes receives it.
 * Returns NMS_OK, NMS_INVALID_ARG (bytes NULL, n < 0) or NMS_TOO_LARGE.
 * For one image nms_f32 never writes the dense bitmask unless it must: the
 * sweep reads only the lists of nonzero words of each 64-row tile ("LeetCUDA
 * 14-nms", measured results: the blocked bitmask its authors name as the
 * next step to cut the mask's memory).  A tile with more nonzero words than
 * its list holds (2048: each of its boxes overlapping boxes in 32 or more
 * other tiles on average) needs the dense rows; nms_f32 then runs the call
 * again with them if its workspace holds nms_workspace_size() bytes, and
 * otherwise returns NMS_WORKSPACE_TOO_SMALL (nothing else changes; call
 * again with the larger workspace).  Grouped input always needs
 * nms_workspace_size() bytes.
 */
nms_status nms_workspace_size_lists(int64_t n, size_t *bytes);

/*
 * nms_f32 -- greedy IoU NMS (see the file comment for the exact result).
 *   boxes          device, n*4 floats, row k = (x1, y1, x2, y2) of box k;
 *                  16-byte aligned.
 *   scores         device, n floats.
 *   n              number of boxes; n = 0 returns NMS_OK with *num_kept = 0.
 *   iou_thresh     float32 threshold; any value but NaN (values < 0 remove
 *                  every later box of a group with a defined IoU).
 *   class_ids      device, n int32 class ids, or NULL (one class).
 *   batch_offsets  device, num_images+1 int64 offsets; image m holds boxes
 *                  [off[m], off[m+1]).  NULL = one image (num_images 0 or 1).
 *   keep_out       device, capacity n int64: receives the kept input indices
 *                  in descending score order (ties: ascending index).
 *   num_kept       host: receives the number of kept boxes.
 *   workspace      device scratch of at least nms_workspace_size() bytes
 *                  (one image: nms_workspace_size_lists() bytes will do
 *                  unless the input is dense, see there), 256-byte aligned;
 *                  its contents on entry do not matter.
 *   stream         hipStream_t or NULL.
 * Sorting follows "LeetCUDA 14-nms" step 1 (stable, descending); the
 * bitmask layout follows its Phase 1 (bit k of word w of row i means sorted
 * box 64w + k; only boxes after row i vote); the sweep follows its Phase 2
 * (removed bitmap in on-chip memory, kept rows ORed in in score order); the
 * map-back follows its host section.
 */
nms_status nms_f32(const float *boxes, const float *scores, int64_t n, float iou_thresh,
                   const int32_t *class_ids, const int64_t *batch_offsets, int64_t num_images,
                   int64_t *keep_out, int64_t *num_kept, void *workspace,
                   size_t workspace_bytes, void *stream);

/* Largest n nms_f32_static accepts, and the size of its static scratch. */
#define NMS_STATIC_MAX_BOXES 16384
#define NMS_STATIC_SCRATCH_BYTES (48u << 20)

/*
 * nms_f32_static -- nms_f32 without a workspace argument, for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc).  It runs the same kernels as
 * nms_f32 on a scratch array that the library holds in its code object: a
 * file-scope device array of NMS_STATIC_SCRATCH_BYTES, one per device the
 * library runs on, allocated by the HIP runtime when the library's code is
 * loaded on that device and held until the process ends.  The call itself
 * allocates nothing: no hipMalloc, no hipHostMalloc (the kept count is
 * copied into the caller's stack frame), no events.
 *   boxes, scores, n, iou_thresh, class_ids, batch_offsets, num_images,
 *   keep_out, num_kept, stream   as for nms_f32.
 * Returns as nms_f32, and NMS_TOO_LARGE for n > NMS_STATIC_MAX_BOXES.
 * Every call on one device shares that device's scratch, which keeps the
 * last call's contents (the kernels need no particular contents on entry):
 * calls that overlap on one device -- from two host threads, or on two
 * streams -- race and must be serialised by the caller.
 */
nms_status nms_f32_static(const float *boxes, const float *scores, int64_t n, float iou_thresh,
                          const int32_t *class_ids, const int64_t *batch_offsets,
                          int64_t num_images, int64_t *keep_out, int64_t *num_kept,
                          void *stream);

/* nms_f32_ex flags. */
#define NMS_FLAG_ONE_LAUNCH 1    /* one image of 1 to 4096 boxes: the whole  */
                                 /* call in a single launch                  */
#define NMS_FLAG_PASS_SORT 2     /* the radix sort as one launch per pass,   */
                                 /* as for inputs above 131072 boxes         */
#define NMS_FLAG_RADIX_SORT 4    /* one image: the radix sort in one launch  */
                                 /* instead of the sample sort               */

/*
 * nms_f32_ex -- nms_f32 with launch-plan flags; flags 0 is nms_f32.
 *   flags   0, or any of NMS_FLAG_ONE_LAUNCH, NMS_FLAG_PASS_SORT and
 *           NMS_FLAG_RADIX_SORT (other bits: NMS_INVALID_ARG).
 * NMS_FLAG_ONE_LAUNCH: one image of 1 to 4096 boxes runs sort, mask, sweep
 * and output in one launch, against the fixed per-launch cost that the
 * "LeetCUDA 14-nms" page (measured results) blames for its losses at 1024
 * and 2048 boxes.  Its workgroups hand over through device memory (a
 * bounded wait on the sort's workgroups, then per-row-tile counters as in
 * the fused launch); if a wait gives up, or a row tile's list of nonzero
 * mask words overflows, the call runs nms_f32's launches instead.  The
 * result is identical either way.  Other inputs ignore the flag.  Our
 * measurement: on MI355X a dependent launch on the same stream costs less
 * than those hand-overs (the three launches of a 1024-box call span 17 us
 * of GPU time, the one launch 25 us), so nms_f32 does not take it.
 * NMS_FLAG_PASS_SORT: grouped input, and one image of more than 16384 boxes,
 * is sorted with one launch per radix pass, the form inputs of more than
 * 131072 boxes always take, instead of by a team of workgroups that stay
 * resident through every pass (one launch).  The result is identical; the
 * flag exists to compare the two (our reading: the pages fix the sort's
 * result, a stable descending order, not its form).
 * NMS_FLAG_RADIX_SORT: one image of 16385 to 131072 boxes, which nms_f32
 * sorts by sample sort in one launch (256 buckets between sampled
 * splitters, each sorted in LDS by one workgroup; a call whose buckets
 * outgrow the LDS runs again with the radix passes), is sorted by the team's
 * radix passes instead.  Same result; the flag exists to compare the two.
 * Other arguments and returns as for nms_f32.
 */
nms_status nms_f32_ex(const float *boxes, const float *scores, int64_t n, float iou_thresh,
                      const int32_t *class_ids, const int64_t *batch_offsets, int64_t num_images,
                      int64_t *keep_out, int64_t *num_kept, void *workspace,
                      size_t workspace_bytes, void *stream, int flags);

/* nms_f32_profiled flags. */
#define NMS_PROFILE_NO_FUSION 1  /* run the mask and the sweep as separate */
                                 /* launches (to time the mask kernel alone) */
#define NMS_PROFILE_ONE_LAUNCH 2 /* as NMS_FLAG_ONE_LAUNCH (timed as the    */
                                 /* mask stage)                              */
#define NMS_PROFILE_PASS_SORT 4  /* as NMS_FLAG_PASS_SORT                    */
#define NMS_PROFILE_RADIX_SORT 8 /* as NMS_FLAG_RADIX_SORT                   */

/*
 * nms_f32_profiled -- nms_f32 with HIP events recorded on `stream` around
 * each stage.  stage_ms (host, NMS_NUM_STAGES floats) receives each stage's
 * elapsed GPU time in milliseconds (0 for a stage that did not run).  flags:
 * 0, NMS_PROFILE_NO_FUSION or NMS_PROFILE_ONE_LAUNCH, with any of
 * NMS_PROFILE_PASS_SORT and NMS_PROFILE_RADIX_SORT (other bits, or the
 * first two together: NMS_INVALID_ARG).  The result is identical to nms_f32's either way.
 */
nms_status nms_f32_profiled(const float *boxes, const float *scores, int64_t n,
                            float iou_thresh, const int32_t *class_ids,
                            const int64_t *batch_offsets, int64_t num_images,
                            int64_t *keep_out, int64_t *num_kept, void *workspace,
                            size_t workspace_bytes, void *stream, float *stage_ms,
                            int flags);

/* Human-readable name of a status ("NMS_OK", ...); never NULL; the
 * returned string is static.  Our reading: the pages' bindings raise
 * exceptions on bad arguments (the device and dtype checks of "LeetCUDA
 * 12-histogram"'s binding section), which cannot cross a C ABI, so every
 * failure is a status code with a name. */
const char *nms_status_string(nms_status status);

/* ---- test-only exports: copy out one stage's intermediate result ---- */

/*
 * nms_debug_order -- run the sort stage only ("LeetCUDA 14-nms", algorithm
 * step 1: a stable descending sort, equal scores in input order; the order is
 * what bug 3's map-back needs).
 *   order_out        device, n int32: input index at each sorted position
 *                    (grouped input: ascending image, then class, then
 *                    descending score, then ascending index).
 *   score_order_out  device, n int32 or NULL: the plain score order
 *                    (descending score, ascending index).
 * Other arguments as for nms_f32; returns as nms_f32 (NMS_NONFINITE_INPUT
 * for a NaN score, with order_out still a permutation).
 */
nms_status nms_debug_order(const float *scores, int64_t n, const int32_t *class_ids,
                           const int64_t *batch_offsets, int64_t num_images,
                           int32_t *order_out, int32_t *score_order_out, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * nms_debug_mask -- run sort, gather and the IoU-mask stage, then expand the
 * mask into a dense row-major array.  The layout is the suppression bitmask
 * of "LeetCUDA 14-nms", Phase 1 (its alignment rule 2: bit k of word w in
 * every row stands for sorted box w * width + k, and boxes at or before the
 * row vote 0), with 64-bit words instead of the page's 32-bit ones.
 *   mask_out   device, n * ceil(n/64) uint64, row stride ceil(n/64) words:
 *              word c of row p (sorted position p) has bit l set iff box
 *              q = 64c + l satisfies p < q < n, q in p's group and
 *              IoU > iou_thresh.  Words the kernel never computes (below
 *              the diagonal tile, beyond the group's last tile) read 0.
 *   order_out  device, n int32 or NULL: the sorted order the rows refer to.
 * Other arguments and returns as for nms_f32.
 */
nms_status nms_debug_mask(const float *boxes, const float *scores, int64_t n,
                          float iou_thresh, const int32_t *class_ids,
                          const int64_t *batch_offsets, int64_t num_images,
                          uint64_t *mask_out, int32_t *order_out, void *workspace,
                          size_t workspace_bytes, void *stream);

/* nms_debug_plan fields. */
#define NMS_PLAN_MASK_QSHIFT 0   /* log2 of the row groups a mask item of the   */
                                 /* separate mask launch is split into (0: the  */
                                 /* sign-test form of the overlap question)     */
#define NMS_PLAN_FUSED 1         /* 1: nms_f32 runs mask and sweep in one launch */
#define NMS_PLAN_FUSED_QSHIFT 2  /* the fused launch's split, -1 if not fused   */
#define NMS_PLAN_RANK_SORT 3     /* 1: the one-launch ranking sort, 0: radix    */
#define NMS_PLAN_SMALL 4         /* 1: the input may take the one-launch path */
                                 /* (one image of 1 to 4096 boxes)             */
#define NMS_PLAN_TEAM_SORT 5     /* 1: the radix sort runs in one launch (a team */
                                 /* of resident workgroups), 0: one launch per  */
                                 /* pass (or the ranking sort)                  */
#define NMS_PLAN_SAMPLE_SORT 6   /* 1: one image sorted by sample sort in one   */
                                 /* launch (before any fallback to the radix)   */
#define NMS_PLAN_FIELDS 8

/*
 * nms_debug_plan -- the launch plan nms_f32 and nms_debug_mask take for n
 * boxes on the current device, without running anything.
 *   plan   host, NMS_PLAN_FIELDS int32: the fields above (unused ones -1;
 *          all -1 for n = 0).
 * Returns NMS_OK, NMS_INVALID_ARG (plan NULL, n < 0, num_images < 0) or
 * NMS_TOO_LARGE.  Our reading: the pages time whole calls only; the plan is
 * exported so that tests can show which kernel form produced a result.
 */
nms_status nms_debug_plan(int64_t n, int64_t num_images, int has_classes, int32_t *plan);

/*
 * nms_debug_decide -- the IoU-mask kernel's threshold test alone: the strict
 * "IoU > threshold" of "LeetCUDA 14-nms" (introduction) on given
 * intersection and union values, decided as the mask kernel decides it (its
 * division-free form is this library's own and must agree with the float32
 * quotient bit for bit, which this export lets a test check).
 *   inter, uni  device, count floats each: an intersection and a union value.
 *   out         device, count bytes: 1 iff the test "inter / uni > t" holds
 *               as the mask kernel decides it.
 *   all_positive_areas  nonzero selects the division-free test the mask
 *               kernel uses when every box has a finite positive area (it
 *               presumes 0 <= inter <= union, union > 0); zero selects the
 *               literal float32 division.
 */
nms_status nms_debug_decide(const float *inter, const float *uni, int64_t count,
                            float iou_thresh, int all_positive_areas, uint8_t *out,
                            void *stream);

/* ------------------------------------------------------------------------
 * Matrix NMS (Gaussian decay), "Fastest Matrix NMS in the West (Part 2)":
 * "What do we need to compute?" and optimisation 4.
 *
 * With the boxes in descending score order (stable, as for nms_f32), the
 * overlap of a father p (earlier) and a child q (later) is the float32 IoU
 * expression above (0/0, two empty boxes, counted as 0); omax[q] is the
 * largest overlap of q with any of its fathers (0 for the first box).  Box q
 * is dropped iff its score is below score_thresh, or some father p gives
 *     exp((omax[p]^2 - O[p][q]^2) / sigma) * score_q  <  score_thresh
 * evaluated in binary64 from the float32 overlaps (the page's
 * s'_j = s_j min_i d_ij < t, with d_ij = exp((O_max,i^2 - O_ij^2) / sigma);
 * the page hard-codes sigma = 0.5).  Every other box is kept; the result is
 * the kept input indices, int64, in descending score order.  Boxes must have
 * x1 <= x2 and y1 <= y2.
 * ------------------------------------------------------------------------ */

/* Stages timed by nms_matrix_f32_profiled. */
#define NMS_MATRIX_STAGE_SORT 0     /* stable sort, gather, scores and checks */
#define NMS_MATRIX_STAGE_OVERLAP 1  /* largest overlap of each box with a father */
#define NMS_MATRIX_STAGE_DECAY 2    /* decay test, kept bitmap, compaction */
#define NMS_MATRIX_NUM_STAGES 3

/*
 * nms_matrix_workspace_size -- device workspace needed by nms_matrix_f32 for
 * n boxes (linear in n: no pairwise matrix is stored).  Returns NMS_OK,
 * NMS_INVALID_ARG (bytes NULL, n < 0) or NMS_TOO_LARGE.
 */
nms_status nms_matrix_workspace_size(int64_t n, size_t *bytes);

/*
 * nms_matrix_f32 -- Matrix NMS as described above.
 *   boxes, scores, n, keep_out, num_kept, workspace, stream  as for nms_f32
 *                  (workspace of at least nms_matrix_workspace_size() bytes).
 *   score_thresh   float32 threshold t on the decayed score; any value but
 *                  NaN.
 *   sigma          Gaussian decay width; finite and > 0 (0.5 on the page).
 * Returns NMS_OK, NMS_INVALID_ARG, NMS_WORKSPACE_TOO_SMALL, NMS_TOO_LARGE,
 * NMS_NONFINITE_INPUT, NMS_BAD_BOXES or NMS_HIP_ERROR.
 */
nms_status nms_matrix_f32(const float *boxes, const float *scores, int64_t n, float score_thresh,
                          double sigma, int64_t *keep_out, int64_t *num_kept, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * nms_matrix_f32_profiled -- nms_matrix_f32 with HIP events on the launch
 * stream around each stage; stage_ms (host, NMS_MATRIX_NUM_STAGES floats)
 * receives the stage times in milliseconds.
 */
nms_status nms_matrix_f32_profiled(const float *boxes, const float *scores, int64_t n,
                                   float score_thresh, double sigma, int64_t *keep_out,
                                   int64_t *num_kept, void *workspace, size_t workspace_bytes,
                                   void *stream, float *stage_ms);

/* ------------------------------------------------------------------------
 * Selection operators of language models: the same step as NMS, a model's
 * scores in and the selected indices out, by descending score with ties to
 * the lower index.  Routing of tokens to experts (with its gradient),
 * penalties, biases and grammar masks on logits, and the next token.
 *
 * These calls are asynchronous: they check their arguments, enqueue their
 * launches on `stream` and return, so they may be captured into a graph.
 * They allocate nothing, read nothing back and keep nothing; outputs and
 * workspace must stay as they are until the work on the stream is done.
 * Two calls that may run at the same time need workspaces of their own.
 * Device data cannot make them fail: what bad values do is stated below.
 * ------------------------------------------------------------------------ */

typedef enum nms_dtype { NMS_F32 = 0, NMS_F16 = 1, NMS_BF16 = 2 } nms_dtype;

#define NMS_ROUTE_SOFTMAX 0
#define NMS_ROUTE_SIGMOID 1
#define NMS_ROUTE_MAX_EXPERTS 1024
#define NMS_ROUTE_MAX_TOP_K 64
#define NMS_ROUTE_MAX_TOKENS (1 << 24)

typedef struct nms_route_options {
    int score;       /* NMS_ROUTE_SOFTMAX or NMS_ROUTE_SIGMOID */
    int top_k;       /* experts per token, 1 .. NMS_ROUTE_MAX_TOP_K, and at most
                        kept_groups * (experts / groups) */
    int renormalise; /* nonzero: the weights of a token sum to scale */
    float scale;     /* finite */
    int groups;      /* groups of neighbouring experts; divides experts; 1: none */
    int kept_groups; /* groups of a token that may be chosen from, 1 .. groups */
    int group_top;   /* a group's score: the sum of its best 1 or 2 experts */
} nms_route_options;

/*
 * nms_route_experts -- the experts of every token and their weights.
 *   logits      device, tokens rows of `experts` elements of `dtype`,
 *               row_stride elements apart.
 *   bias        device float[experts] or NULL: added to the scores for the
 *               choice only (balance), not for the weights.
 *   live        device byte[tokens] or NULL: 0 marks a padded row.
 *   ids         device int32[tokens * top_k]; weights: float, the same shape.
 *   counts      device int32[experts] or NULL: receives how many tokens chose
 *               each expert (written, not added to).
 * Per token, in binary64 from the logits z:
 *     s = exp(z - max z) / sum, or 1 / (1 + exp(-z));  c = s + bias.
 * An expert with z or c NaN or -infinity is never chosen.  With groups > 1
 * only the kept_groups groups with the largest sums of their best group_top c
 * stay (a group with fewer takes those it has; with none it never stays).
 * Then the first top_k experts by descending c (without bias by descending
 * z), every tie to the lower index.  Their weights are scale * s, divided by
 * the sum of the chosen s if renormalise is set (for softmax: the softmax of
 * the chosen logits; all 0 where that sum is 0), in float32, off by at most
 * 2^-21 of the value.
 * Places that no expert is left for, and all places of a padded row, hold id
 * -1 and weight 0.
 * Returns NMS_OK, NMS_INVALID_ARG, NMS_TOO_LARGE (experts or tokens above the
 * limits) or NMS_HIP_ERROR.
 */
nms_status nms_route_experts(const void *logits, nms_dtype dtype, int64_t tokens, int64_t experts,
                             int64_t row_stride, const float *bias, const uint8_t *live,
                             const nms_route_options *options, int32_t *ids, float *weights,
                             int32_t *counts, void *stream);

/*
 * nms_route_experts_backward -- the gradient of nms_route_experts' weights in
 * its logits (the choice itself has none, and neither has the bias).
 *   logits, dtype, tokens, experts, row_stride, options  as in the forward
 *                 call (of the options, the groups are not used).
 *   ids           device, the forward call's ids (one outside 0..experts-1
 *                 is an empty place).
 *   grad_weights  device float[tokens * top_k]: the gradient of the weights.
 *   grad_logits   device, tokens rows of `experts` elements of dtype,
 *                 grad_stride elements apart; every element is written
 *                 (0 in rows without a chosen expert); may be logits, with
 *                 the same stride, and must not overlap it otherwise.
 * Computed in float32, rounded once.  Returns as nms_route_experts.
 */
nms_status nms_route_experts_backward(const void *logits, nms_dtype dtype, int64_t tokens,
                                      int64_t experts, int64_t row_stride, const int32_t *ids,
                                      const float *grad_weights, const nms_route_options *options,
                                      void *grad_logits, int64_t grad_stride, void *stream);

#define NMS_MAX_ROWS 65536
#define NMS_MAX_VOCAB (1 << 22)
#define NMS_MAX_HISTORY 1048575
#define NMS_MAX_BIASES 2047
#define NMS_MAX_TOP_K 1024

/* What applies to a batch of rows of logits.  Every pointer is device memory
 * or NULL; per-row arrays have one entry per row. */
typedef struct nms_logit_rules {
    const int32_t *history;     /* the row's tokens so far: the prompt, then what
                                   was generated; rows history_stride apart */
    int64_t history_stride;
    int64_t history_capacity;   /* entries a row has, at most NMS_MAX_HISTORY */
    const int32_t *history_len; /* entries in use (clamped into 0..capacity) */
    const int32_t *prompt_len;  /* of them the prompt; NULL: none */
    const float *repetition;    /* r > 0; NULL: 1 */
    const float *presence;      /* NULL: 0 */
    const float *frequency;     /* NULL: 0 */
    const int32_t *bias_ids;    /* bias_count entries per row, bias_stride apart; */
    const float *bias_values;   /* entries outside the vocabulary are unused */
    int64_t bias_stride;
    int64_t bias_count;         /* at most NMS_MAX_BIASES */
    const uint64_t *allowed;    /* allowed_count masks, allowed_stride words apart: */
    int64_t allowed_stride;     /* bit v mod 64 of word v / 64 set: v is allowed */
    int64_t allowed_count;
    const int32_t *allowed_rows; /* the mask of each row: negative: none, every
                                    token is allowed; allowed_count or above: no
                                    token is.  NULL: row i has mask i */
} nms_logit_rules;

/*
 * nms_adjust_logits -- the rules applied to logits.
 *   logits, out  device, rows of `vocab` elements of dtype, row_stride and
 *                out_stride elements apart; out may be logits (with the same
 *                stride), and must not overlap it otherwise.
 * For token v of a row, with z its logit in float32, each step rounded to
 * float32 (no fused multiply-add):
 *     v is in the history:            z = z > 0 ? z / r : z * r
 *     v was generated c > 0 times:    z = z - frequency * c;  z = z - presence
 *     v is in the row's bias list:    z = z + value (of its last entry there)
 *     v is not allowed:               z = -infinity
 * and then once to dtype.  History entries outside the vocabulary are skipped.
 * Returns NMS_OK, NMS_INVALID_ARG, NMS_TOO_LARGE or NMS_HIP_ERROR.
 */
nms_status nms_adjust_logits(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                             int64_t row_stride, const nms_logit_rules *rules, void *out,
                             int64_t out_stride, void *stream);

/*
 * nms_pick_workspace_size -- device workspace needed by nms_pick_tokens.
 * Returns NMS_OK, NMS_INVALID_ARG or NMS_TOO_LARGE.
 */
nms_status nms_pick_workspace_size(int64_t rows, int64_t vocab, int max_top_k, size_t *bytes);

/*
 * nms_pick_tokens -- the next token of every row, from its logits under the
 * rules (which are applied on the way: adjusted logits are not written).
 *   rules        as for nms_adjust_logits, or NULL: none.
 *   uniform      device float[rows]: one number in [0, 1) per row (below: as
 *                0; above: the last token that stays).
 *   temperature  device float[rows] or NULL (1): t; 0 or below takes the first
 *                token; at +infinity all allowed tokens weigh alike.
 *   top_k        device int32[rows] or NULL (max_top_k): clamped into
 *                1..max_top_k (0 and below take the first token; there is no
 *                value for a draw from more than max_top_k tokens).
 *   top_p, min_p device float[rows] or NULL (1 and 0).  Where one of these
 *                four is not a number, the first token is taken.
 *   max_top_k    1 .. NMS_MAX_TOP_K.
 *   ids          device int32[rows]; logprobs: device float[rows].
 *   workspace    device, 256-byte aligned, nms_pick_workspace_size() bytes.
 * With z the adjusted logits in float32 (not rounded to dtype again), the
 * candidates of a row are its first top_k tokens by descending z, ties to the
 * lower token, without those at -infinity or NaN.  In binary64, with z0 the
 * first one's: w = exp((z - z0) / t).  Of the candidates stay the shortest
 * prefix whose sum reaches top_p times the sum of all, and of it those with
 * w >= min_p, at least the first.  The token is the first of them at which
 * the running sum passes uniform times their sum.  Its logprob is
 * log(exp(z / t) / sum over all tokens of exp(z / t)), with t = 1 where the
 * temperature is 0; the sum is made of float32 terms, which leaves the logprob
 * off by at most 7e-6 and its rounding.  A row without candidates gets id -1
 * and logprob -infinity.
 * Returns NMS_OK, NMS_INVALID_ARG, NMS_WORKSPACE_TOO_SMALL, NMS_TOO_LARGE or
 * NMS_HIP_ERROR.
 */
nms_status nms_pick_tokens(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                           int64_t row_stride, const nms_logit_rules *rules, const float *uniform,
                           const float *temperature, const int32_t *top_k, const float *top_p,
                           const float *min_p, int max_top_k, int32_t *ids, float *logprobs,
                           void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Losses of language models: what trains the models whose tokens and experts
 * the operators above select.  Log probabilities of given tokens, the clipped
 * policy loss and the preference loss that are made of them, and the balance
 * loss of routing, each with its gradient in the logits.
 *
 * As for the operators above: asynchronous, capturable, nothing is allocated,
 * read back or kept, device data cannot make a call fail, and two calls that
 * may run at the same time need workspaces of their own.  Results do not
 * depend on how the GPU schedules a call: the same input gives the same bits.
 *
 * Rows of logits: `rows` rows of `vocab` elements of dtype, row_stride
 * elements apart, with one token each.  A row counts where its token is in
 * 0..vocab-1 (and, for the policy loss, its weight is not 0); one that does
 * not has log probability, entropy and gradient 0 and is not read.  With t
 * the row's temperature, p = softmax(z / t) and a the token,
 *     log probability  log p_a;    entropy  H = -sum p log p.
 * A logit of -infinity, or further below the row's largest than float32 holds,
 * has probability 0.  NaN or +infinity in a row that counts makes its results
 * and its whole gradient NaN (nms_pick_tokens passes over a NaN; a loss does not
 * hide it); where all logits are -infinity, the log probability is -infinity and
 * entropy and gradient are 0.  A temperature of 0 or below, or NaN, counts as 1
 * (the log probability that nms_pick_tokens gives for it); at +infinity all
 * tokens but those of probability 0 weigh alike; below 4.2e-39 log2(e) / t
 * counts as float32's largest number in the probabilities.
 * Terms are computed in float32, sums over rows in binary64; a probability
 * below 2^-126 of the row's largest counts as 0.
 *
 * grad_logits: device, rows of elements of dtype, grad_stride elements apart,
 * every element is written (0 in rows that do not count); may be logits, with
 * the same stride, and must not overlap it otherwise.  Rounded once to dtype.
 * grad_loss: device float, the gradient of the loss, or NULL: 1.  (With
 * float16 logits a scaled loss keeps small gradients in range.)
 * ------------------------------------------------------------------------ */

#define NMS_MAX_PAIRS 32768
#define NMS_MAX_SEQUENCES 65536

/*
 * nms_loss_workspace_size -- device workspace needed by the calls on rows of
 * logits below.
 *   pairs  of nms_preference_loss and its gradient; 0 for the others.
 * Returns NMS_OK, NMS_INVALID_ARG or NMS_TOO_LARGE.
 */
nms_status nms_loss_workspace_size(int64_t rows, int64_t vocab, int64_t pairs, size_t *bytes);

/*
 * nms_token_logprobs -- log probabilities of given tokens.
 *   tokens       device int32[rows].
 *   temperature  device float[rows] or NULL: 1.
 *   logprobs     device float[rows].
 *   entropies    device float[rows] or NULL: not wanted.
 *   workspace    device, 256-byte aligned, nms_loss_workspace_size() bytes.
 * Returns NMS_OK, NMS_INVALID_ARG, NMS_WORKSPACE_TOO_SMALL, NMS_TOO_LARGE (as
 * for nms_pick_tokens) or NMS_HIP_ERROR.
 */
nms_status nms_token_logprobs(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                              int64_t row_stride, const int32_t *tokens, const float *temperature,
                              float *logprobs, float *entropies, void *workspace,
                              size_t workspace_bytes, void *stream);

/*
 * nms_token_logprobs_backward -- the gradient of these in the logits,
 *     dz_j = (g ([j = a] - p_j) - h p_j (log p_j + H)) / t
 *   grad_logprobs   device float[rows]: g.
 *   grad_entropies  device float[rows] or NULL: h, 0.
 * A row whose g and h are 0 has gradient 0, whatever it holds.
 * Returns as nms_token_logprobs.
 */
nms_status nms_token_logprobs_backward(const void *logits, nms_dtype dtype, int64_t rows,
                                       int64_t vocab, int64_t row_stride, const int32_t *tokens,
                                       const float *temperature, const float *grad_logprobs,
                                       const float *grad_entropies, void *grad_logits,
                                       int64_t grad_stride, void *workspace,
                                       size_t workspace_bytes, void *stream);

typedef struct nms_policy_options {
    float clip_low, clip_high; /* the ratio is held in 1 - clip_low .. 1 + clip_high;
                                  0 <= clip_low <= 1, 0 <= clip_high (finite) */
    float kl;                  /* weight of the divergence from the reference, >= 0 */
    float entropy;             /* weight of the entropy bonus, finite */
} nms_policy_options;

/*
 * nms_policy_loss -- the clipped policy loss over rows of logits, its gradient
 * or both at once (which reads the logits once where a row fits the registers
 * of a compute unit).  With l a row's log probability, r = exp(l - old),
 *     each = -min(r A, min(max(r, 1 - clip_low), 1 + clip_high) A)
 *            + kl (exp(ref - l) - (ref - l) - 1) - entropy H
 *     loss = sum over the rows that count of weight * each.
 * Where A is 0 the first term is 0.  The gradient is that of r A where it is
 * the smaller one or equal, and 0 where the ratio is held.
 *   old_logprobs   device float[rows]: of the policy that picked the tokens.
 *   advantages     device float[rows]: A.
 *   weights        device float[rows] or NULL: 1 / rows.  0 marks a row that
 *                  does not count.  Means over tokens, sequences, micro-batches
 *                  and ranks are made by these weights.
 *   ref_logprobs   device float[rows] or NULL: no divergence.
 *   options        kl without ref_logprobs must be 0.
 *   grad_loss      as above.
 *   loss           device float or NULL; logprobs, entropies: device
 *                  float[rows] or NULL; grad_logits: as above or NULL.  At
 *                  least one of the four.
 * Returns as nms_token_logprobs.
 */
nms_status nms_policy_loss(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                           int64_t row_stride, const int32_t *tokens, const float *old_logprobs,
                           const float *advantages, const float *weights,
                           const float *ref_logprobs, const float *temperature,
                           const nms_policy_options *options, const float *grad_loss, float *loss,
                           float *logprobs, float *entropies, void *grad_logits,
                           int64_t grad_stride, void *workspace, size_t workspace_bytes,
                           void *stream);

#define NMS_PREFERENCE_SIGMOID 0
#define NMS_PREFERENCE_HINGE 1
#define NMS_PREFERENCE_SQUARED 2

typedef struct nms_preference_options {
    int kind;        /* NMS_PREFERENCE_* */
    int average;     /* nonzero: a sequence's log probability is the mean over
                        its rows that count, not the sum */
    float beta;      /* finite, > 0 */
    float smoothing; /* of the sigmoid kind, 0 .. 0.5 */
    float margin;    /* finite */
} nms_preference_options;

/*
 * nms_preference_loss -- the loss of paired log ratios, and its gradient where
 * grad_logits is given.  Sequence i < pairs is the preferred one of pair i,
 * sequence pairs + i the other.  With l_q the sum (or mean) of the log
 * probabilities of sequence q's rows that count,
 *     h = beta ((l_i - ref_i) - (l_pairs+i - ref_pairs+i)) - margin
 *     sigmoid  (1 - smoothing) log(1 + exp(-h)) + smoothing log(1 + exp(h))
 *     hinge    max(0, 1 - h)
 *     squared  ((h - 1/2) / beta)^2
 *     loss = sum over pairs of weight * each.
 *   offsets       device int64[2 * pairs + 1]: sequence q is the rows from
 *                 offsets[q] to offsets[q + 1], from the largest offset so far
 *                 where they decrease, within the rows.  Rows of no sequence
 *                 have gradient 0.
 *   ref_logprobs  device float[2 * pairs] or NULL: 0.
 *   weights       device float[pairs] or NULL: 1 / pairs.  A pair of weight 0
 *                 has no part in the loss, whatever it holds.
 *   loss          device float; logprobs: device float[2 * pairs], l;
 *                 margins: device float[pairs], h.
 *   grad_logits   as above, or NULL: not wanted.
 *   workspace     nms_loss_workspace_size(rows, vocab, pairs) bytes.
 * Returns as nms_token_logprobs (NMS_TOO_LARGE: pairs above NMS_MAX_PAIRS).
 */
nms_status nms_preference_loss(const void *logits, nms_dtype dtype, int64_t rows, int64_t vocab,
                               int64_t row_stride, const int32_t *tokens, const int64_t *offsets,
                               int64_t pairs, const float *ref_logprobs, const float *weights,
                               const nms_preference_options *options, const float *grad_loss,
                               float *loss, float *logprobs, float *margins, void *grad_logits,
                               int64_t grad_stride, void *workspace, size_t workspace_bytes,
                               void *stream);

/*
 * nms_preference_loss_backward -- the gradient alone, from the margins of the
 * forward call.
 */
nms_status nms_preference_loss_backward(const void *logits, nms_dtype dtype, int64_t rows,
                                        int64_t vocab, int64_t row_stride, const int32_t *tokens,
                                        const int64_t *offsets, int64_t pairs,
                                        const float *weights,
                                        const nms_preference_options *options,
                                        const float *margins, const float *grad_loss,
                                        void *grad_logits, int64_t grad_stride, void *workspace,
                                        size_t workspace_bytes, void *stream);

typedef struct nms_balance_options {
    int score;     /* NMS_ROUTE_SOFTMAX or NMS_ROUTE_SIGMOID, as in the routing */
    int top_k;     /* places per token in ids, 0 .. NMS_ROUTE_MAX_TOP_K */
    float balance; /* finite */
    float z;       /* finite */
} nms_balance_options;

/*
 * nms_balance_loss -- the balance loss of routing, the loss on the size of the
 * logits and the counts they go by, and the gradient where grad_logits is
 * given.  Over the tokens of sequence q that count (live, in a sequence), n_q
 * many, with c_qe those that chose expert e, s the softmax of their logits or
 * their sigmoids divided by the sum of these,
 *     f_qe = experts c_qe / sum_e c_qe,    P_qe = sum of s_e / n_q
 *     loss = balance / sequences * sum_q sum_e f_qe P_qe
 *            + z * the mean over all tokens that count of log(sum exp z)^2.
 * The counts have no gradient.  A logit of -infinity has score 0; a token with
 * no other logits has no part in the loss but counts as a token.  NaN in a
 * token that counts makes the loss NaN, and so does +infinity (of sigmoid
 * scores with z = 0 it does not).
 *   logits, dtype, tokens, experts, row_stride  as for nms_route_experts.
 *   ids        device int32[tokens * top_k], as nms_route_experts gives them
 *              (one outside 0..experts-1 is an empty place), or NULL: counts
 *              are given, of all ranks for instance.  NULL has that meaning for
 *              an empty batch too: where its counts are wanted (they are 0), or
 *              neither is given, pass any other address, which is not read.
 *   live       device byte[tokens] or NULL: 0 marks a padded row.
 *   offsets    device int64[sequences + 1]: as for nms_preference_loss; NULL:
 *              one sequence.
 *   loss       device float or NULL.
 *   counts     device int32[sequences * experts]: written (NULL: not wanted),
 *              or read where ids is NULL (below 0: as 0).
 *   workspace  device, 256-byte aligned, nms_balance_workspace_size() bytes.
 * Returns as nms_route_experts, or NMS_WORKSPACE_TOO_SMALL.
 */
nms_status nms_balance_loss(const void *logits, nms_dtype dtype, int64_t tokens, int64_t experts,
                            int64_t row_stride, const int32_t *ids, const uint8_t *live,
                            const int64_t *offsets, int64_t sequences,
                            const nms_balance_options *options, const float *grad_loss,
                            float *loss, int32_t *counts, void *grad_logits, int64_t grad_stride,
                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * nms_balance_workspace_size -- device workspace needed by nms_balance_loss.
 * Returns NMS_OK, NMS_INVALID_ARG or NMS_TOO_LARGE.
 */
nms_status nms_balance_workspace_size(int64_t tokens, int64_t experts, int64_t sequences,
                                      int top_k, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* GREEDY_NMS_H */
