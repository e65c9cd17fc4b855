/*
 * moe_ep.h -- C ABI of the MoE expert-parallel dispatch/combine core, one
 * rank's share, for AMD Instinct MI355X (gfx950).
 *
 * The library performs the data-parallel steps around the two all-to-all
 * exchanges of an expert-parallel MoE layer: routing, the per-destination
 * counts and offsets, packing each destination's rows contiguously, and
 * the gate-weighted reduction when the expert outputs return. The R
 * destinations are logical partitions of one device buffer; the library
 * performs no inter-GPU transfer.
 *
 * Conventions for every entry point:
 *  - All array pointers are DEVICE pointers owned by the caller. The
 *    library never allocates, frees or keeps a pointer after returning.
 *  - Every call only enqueues work on `stream` (a hipStream_t passed as
 *    void*; NULL is the null stream). No call synchronises the device or
 *    reads device memory from the host, so routing results never make a
 *    round trip through the host.
 *  - bf16 tensors are passed as uint16_t bit patterns, row-major.
 *  - Every scalar, required pointer and alignment is validated on the host
 *    before anything is enqueued; on error nothing is enqueued, outputs are
 *    untouched and the status says why. After a launch, a HIP launch error
 *    is reported as MOE_ERR_LAUNCH. No exception crosses the ABI and there
 *    is no global error state.
 *  - T = 0 is legal: the call enqueues nothing, except moe_dispatch_layout,
 *    which still writes its (all-zero) counts and offsets.
 *  - Results are bitwise reproducible from run to run: no floating-point
 *    atomics, integer atomics only where their order cannot matter.
 *  - Limits: 1 <= k <= min(E, 32); 1 <= E <= 1024; E % R == 0; H % 8 == 0;
 *    0 < H <= 65536; T * k < 2^31.
 */
#ifndef MOE_EP_H
#define MOE_EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,  /* NULL/misaligned pointer, bad size or relation */
    MOE_ERR_UNSUPPORTED = 2,  /* outside the limits above */
    MOE_ERR_WORKSPACE = 3,    /* workspace missing or too small */
    MOE_ERR_LAUNCH = 4,       /* the HIP runtime rejected a kernel launch */
    /* not a status: gives the type the range of a 32-bit int, so that any
       int value passed as a moe_status_t (moe_status_string of an unknown
       code) is a valid value of the type in C++ as well as in C */
    MOE_STATUS_RANGE_MIN = -0x7FFFFFFF - 1,
    MOE_STATUS_RANGE_MAX = 0x7FFFFFFF
} moe_status_t;

/* moe_route_topk flags */
#define MOE_ROUTE_NORMALIZE 1u   /* weights renormalised over the k selected */

/* moe_combine_reduce flags */
#define MOE_COMBINE_OUT_FP32 1u  /* out is float[T][H] instead of bf16[T][H] */

/*
 * moe_route_topk -- pick k experts per token and their gate weights.
 *
 * Defined by: ai-from-scratch "19. All-to-all", intro (after attention every
 * token holds a list of expert ids; results are mixed on return) and "Why
 * the router can ruin your day" (a per-expert balancing bias takes part in
 * the top-k decision only, never in the mix weights); aicassindra
 * "gpu_moe_all_to_all", "Two collectives per layer, and what each one
 * moves" (outputs are scaled by the router's gate weights).
 *
 * For each token t:
 *   s[e] = logits[t][e] + bias[e]   (one float32 add; bias may be NULL)
 *   topk_idx[t][0..k-1] = the k experts with the largest s, in descending
 *     order; -0 equals +0; any NaN ranks below every number (including
 *     -inf); ties go to the smaller expert id.
 *   topk_w[t][j] from the UNBIASED logits l of the selected experts:
 *     flags & MOE_ROUTE_NORMALIZE: w_j = exp(l_j - m) / sum_i exp(l_i - m)
 *       over the k selected (m = their max); the weights sum to 1.
 *     otherwise: w_j = exp(l_j - M) / sum over all E of exp(l_e - M)
 *       (softmax over all experts, not renormalised).
 *   Weights are computed in float32; for NaN or infinite logits they are
 *   unspecified.
 *
 * Arguments:
 *   logits   [T][E] float32, 4-byte aligned.
 *   bias     [E] float32 or NULL (selection only).
 *   topk_idx [T][k] int32 out;  topk_w [T][k] float32 out.
 * Errors: MOE_ERR_INVALID_ARG for NULL/misaligned pointers or T < 0;
 *   MOE_ERR_UNSUPPORTED outside the limits.
 */
moe_status_t moe_route_topk(const float *logits, const float *bias,
                            int64_t T, int32_t E, int32_t k, uint32_t flags,
                            int32_t *topk_idx, float *topk_w, void *stream);

/*
 * moe_route_topk_grouped -- group-limited routing: each token may use at
 * most topk_groups of n_groups contiguous expert groups (destination groups
 * such as nodes), then picks its k experts inside them.
 *
 * Defined by: ai-from-scratch "19. All-to-all", "DeepSeek's numbers" (each
 * token limited to at most 4 nodes, so the slow hop stays bounded) and the
 * closing section (node-limited routing as an architectural constraint);
 * zenaique Q&A "moe-hide-alltoall-techniques" (node-limited routing caps
 * cross-node traffic). The pages do not define a group's score; this call
 * ranks groups by their best selection score s[e] (as moe_route_topk orders
 * experts, so ties go to the lower group), keeps the best topk_groups, and
 * selects the k best experts among them. Gate weights are computed exactly
 * as in moe_route_topk, from the selected experts' unbiased logits.
 *
 * Arguments: as moe_route_topk, plus
 *   n_groups    groups of E / n_groups experts each; E % n_groups == 0,
 *               1 <= n_groups <= 64.
 *   topk_groups 1 <= topk_groups <= n_groups and
 *               k <= topk_groups * (E / n_groups).
 *   topk_groups == n_groups is plain moe_route_topk.
 * Errors: MOE_ERR_INVALID_ARG for bad pointers or group sizes;
 *   MOE_ERR_UNSUPPORTED outside the limits (n_groups > 64 included).
 */
moe_status_t moe_route_topk_grouped(const float *logits, const float *bias,
                                    int64_t T, int32_t E, int32_t k,
                                    int32_t n_groups, int32_t topk_groups,
                                    uint32_t flags, int32_t *topk_idx,
                                    float *topk_w, void *stream);

/*
 * moe_layout_workspace_size -- bytes of device workspace that
 * moe_dispatch_layout needs for these sizes (written to *bytes). The
 * workspace needs no initialisation: the layout call clears what it uses,
 * on-stream.
 * Errors: as moe_dispatch_layout's size checks; *bytes untouched on error.
 */
moe_status_t moe_layout_workspace_size(int64_t T, int32_t E, int32_t k,
                                       int32_t R, size_t *bytes);

/*
 * moe_dispatch_layout -- per-expert and per-destination counts, the offset
 * table, capacity drops in token order, and every replica's send row.
 *
 * Defined by: aicassindra "gpu_moe_all_to_all", "Two collectives per layer"
 * (per-destination counts precede the payload so that receivers can size
 * their buffers) and "Bucketing: cut the message count, not the byte count"
 * (sort by destination and build an offset table so that each destination
 * is one contiguous segment; keep indices and counts on the device);
 * "MoE All-to-All Dispatch and Ragged Routing", "Fixed Capacity vs. Ragged
 * Routing" (per-sender-expert slots under a capacity factor, the excess
 * dropped; ragged routing is dropless); ai-from-scratch "19. All-to-all",
 * "Why the router can ruin your day" (a dropped token counts as having
 * skipped that expert).
 *
 * Expert e lives on destination e / (E / R). With a = t * k + j:
 *   expert_demand[e]  = #{a : topk_idx[a] == e}
 *   rank(a)           = #{a' < a : topk_idx[a'] == topk_idx[a]}
 *   kept(a)           = capacity < 0 || rank(a) < capacity
 *   expert_counts[e]  = kept replicas of e = min(demand, capacity)
 *   expert_offsets    = exclusive prefix sum of counts, E + 1 entries;
 *                       expert_offsets[E] = N, the kept total
 *   dest_counts[r]    = sum of counts of r's experts
 *   dest_offsets[r]   = expert_offsets[r * E / R]; dest_offsets[R] = N
 *   pos[a]            = expert_offsets[e] + rank(a) if kept, else -1
 *   send_src[pos[a]]  = t for every kept a (send_src may be NULL)
 * The send rows are thereby grouped by destination, then by expert, then
 * by token. N stays on the device (expert_offsets[E]).
 *
 * Arguments:
 *   topk_idx  [T][k] int32 expert ids. Precondition: every id in [0, E)
 *             and distinct within a row; ids outside [0, E) are ignored
 *             (not counted, pos = -1).
 *   capacity  < 0: dropless; >= 0: at most `capacity` rows per expert.
 *   outputs   int32 arrays of the sizes above; send_src, when given,
 *             holds at least N entries: T * k when dropless, else
 *             min(T * k, E * capacity) (entries >= N are not written).
 *   workspace device memory of at least moe_layout_workspace_size() bytes,
 *             16-byte aligned; its contents on entry do not matter.
 * Errors: MOE_ERR_INVALID_ARG for NULL/misaligned pointers, T < 0, R < 1 or
 *   E % R != 0; MOE_ERR_UNSUPPORTED outside the limits; MOE_ERR_WORKSPACE
 *   when the workspace is NULL or too small.
 */
moe_status_t moe_dispatch_layout(const int32_t *topk_idx, int64_t T,
                                 int32_t E, int32_t k, int32_t R,
                                 int32_t capacity, int32_t *expert_demand,
                                 int32_t *expert_counts,
                                 int32_t *expert_offsets, int32_t *dest_counts,
                                 int32_t *dest_offsets, int32_t *pos,
                                 int32_t *send_src, void *workspace,
                                 size_t workspace_bytes, void *stream);

/*
 * moe_route_dispatch_layout -- moe_route_topk followed by
 * moe_dispatch_layout (no group limit), in one call: the same outputs, bit
 * for bit, with fewer launches for small batches.
 *
 * Defined by: the two calls' passages above, and aicassindra
 * "gpu_moe_all_to_all", "Latency-bound at decode, bandwidth-bound at
 * prefill" (at decode sizes the exchange is bound by latency: cut the
 * independent steps and synchronisation points, not the bytes).
 *
 * When T * k <= 4096, E <= 512, E % 4 == 0 and logits and bias are 16-byte
 * aligned, one kernel launch does both: its blocks route their tokens, and
 * the last block to finish (an atomic ticket in the first 16 bytes of the
 * workspace; no block waits for another) builds the layout from the ids the
 * others wrote. Otherwise the call launches the routing and the layout
 * kernels as the two separate calls do.
 *
 * Arguments: those of moe_route_topk (logits, bias, flags, topk_idx,
 *   topk_w) and of moe_dispatch_layout (R, capacity and its outputs), plus
 *   workspace  device memory of at least
 *              moe_route_dispatch_layout_workspace_size() bytes (16 or
 *              more), 16-byte aligned. Its contents on entry do not
 *              matter, with one exception: a call on a workspace its
 *              predecessor did not leave ready counts arrivals with a
 *              slower, stamp-keyed protocol, and every call leaves it
 *              ready; the exception is a first 64-bit word whose upper
 *              half holds the ready pattern 0x6D6F6574 and whose lower
 *              half is not 0 (no call leaves it so), which the call would
 *              take as arrivals already counted. Calls that overlap in
 *              time must not share a workspace.
 * Errors: those of the two calls; MOE_ERR_WORKSPACE when the workspace is
 *   NULL, misaligned or too small.
 */
moe_status_t moe_route_dispatch_layout_workspace_size(int64_t T, int32_t E,
                                                      int32_t k, int32_t R,
                                                      size_t *bytes);
moe_status_t moe_route_dispatch_layout(const float *logits, const float *bias,
                                       int64_t T, int32_t E, int32_t k,
                                       uint32_t flags, int32_t R,
                                       int32_t capacity, int32_t *topk_idx,
                                       float *topk_w, int32_t *expert_demand,
                                       int32_t *expert_counts,
                                       int32_t *expert_offsets,
                                       int32_t *dest_counts,
                                       int32_t *dest_offsets, int32_t *pos,
                                       int32_t *send_src, void *workspace,
                                       size_t workspace_bytes, void *stream);

/*
 * moe_dispatch_layout_noalloc -- moe_dispatch_layout with no workspace
 * argument, for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation.
 * Same arguments (minus workspace), outputs and errors. The call allocates
 * nothing: the per-tile histograms live in a device array of
 * MOE_LAYOUT_SCRATCH_BYTES that the library holds on each GPU it runs on
 * until the process ends; every legal size fits (sizes whose
 * moe_layout_workspace_size() exceeds it would return MOE_ERR_WORKSPACE).
 * All calls on one GPU share that array, and every call rewrites what it
 * reads, so nothing carries over from the previous call; calls that overlap
 * on one GPU (different streams, host threads) race on it and must be
 * serialised by the caller. MOE_ERR_LAUNCH also covers a failure to look
 * up the array's device address (once per device, on the first call).
 */
#define MOE_LAYOUT_SCRATCH_BYTES (128u * 1024u * 4u)
moe_status_t moe_dispatch_layout_noalloc(const int32_t *topk_idx, int64_t T,
                                         int32_t E, int32_t k, int32_t R,
                                         int32_t capacity, int32_t *expert_demand,
                                         int32_t *expert_counts,
                                         int32_t *expert_offsets,
                                         int32_t *dest_counts,
                                         int32_t *dest_offsets, int32_t *pos,
                                         int32_t *send_src, void *stream);

/*
 * moe_dispatch_permute -- pack each kept replica of each token into its
 * send row: send[pos[t][j]][:] = x[t][:] (a bit copy of the bf16 row).
 *
 * Defined by: aicassindra "gpu_moe_all_to_all", "Bucketing" (permute so that
 * everything bound for one destination is contiguous, fused into the
 * staging kernel) and "Two collectives per layer" (each token goes out k
 * times); thecoregrid "Mixture-of-experts acceleration through overlap",
 * paragraph on the remote-owner-aligned layout (each block of rows belongs
 * to one destination, so it leaves as one contiguous write).
 *
 * Arguments:
 *   x         [T][H] bf16, 16-byte aligned.
 *   pos       [T][k] int32 from moe_dispatch_layout (-1 = dropped).
 *   E, capacity  the expert count and capacity given to moe_dispatch_layout;
 *             they fix the bound on the kept rows N: T * k when dropless
 *             (capacity < 0), min(T * k, E * capacity) otherwise.
 *   send      [send_rows][H] bf16 out, 16-byte aligned, send_rows >= that
 *             bound. Rows that no replica points at are not written.
 *             Positions >= send_rows (a broken precondition on pos) are
 *             skipped, never written out of bounds.
 * Errors: MOE_ERR_INVALID_ARG for NULL/misaligned pointers, T < 0, or
 *   send_rows below the bound; MOE_ERR_UNSUPPORTED outside the limits.
 */
moe_status_t moe_dispatch_permute(const uint16_t *x, const int32_t *pos,
                                  int64_t T, int32_t H, int32_t k, int32_t E,
                                  int32_t capacity, uint16_t *send,
                                  int64_t send_rows, void *stream);

/*
 * moe_combine_reduce -- bring each token's k expert outputs back along the
 * inverse permutation and reduce them at the origin:
 *   out[t][h] = round( sum_{j : pos[t][j] >= 0} topk_w[t][j] * y[pos[t][j]][h]
 *                      + shared[t][h] + residual[t][h] )
 * accumulated in float32 with one fused multiply-add per kept replica in
 * ascending j, then + shared, then + residual, and one final rounding to
 * bf16 (nearest, ties to even) unless MOE_COMBINE_OUT_FP32 is set. Dropped
 * replicas contribute nothing; the other weights are not renormalised.
 *
 * Defined by: aicassindra "gpu_moe_all_to_all", "Two collectives per layer"
 * (outputs return along the inverse permutation, k partial results per
 * token, scaled by the gate weights at the origin); "MoE All-to-All
 * Dispatch and Ragged Routing", "Returning Tokens to the Original GPU" (the
 * residual x + dx is formed at the origin); ai-from-scratch "19.
 * All-to-all", section on 512 experts (10 routed + 1 always-active shared
 * expert) and "Why the router can ruin your day" (drops).
 *
 * Arguments:
 *   y         [y_rows][H] bf16 expert outputs in send layout, 16-byte
 *             aligned (may alias the send buffer of moe_dispatch_permute).
 *   pos       [T][k] int32; positions >= y_rows are skipped (a broken
 *             precondition, never a read out of bounds).
 *   topk_w    [T][k] float32.
 *   shared    [T][H] bf16 shared-expert output or NULL (weight 1).
 *   residual  [T][H] bf16 or NULL.
 *   out       [T][H] bf16, or float32 with MOE_COMBINE_OUT_FP32; 16-byte
 *             aligned; must not alias any input.
 * Errors: MOE_ERR_INVALID_ARG for NULL/misaligned pointers, T < 0,
 *   y_rows < 0; MOE_ERR_UNSUPPORTED outside the limits.
 */
moe_status_t moe_combine_reduce(const uint16_t *y, int64_t y_rows,
                                const int32_t *pos, const float *topk_w,
                                const uint16_t *shared,
                                const uint16_t *residual, int64_t T,
                                int32_t H, int32_t k, uint32_t flags,
                                void *out, void *stream);

/*
 * FP8 dispatch payload: the permute quantises each row as it packs it, so
 * the send buffer holds about half the bytes of the bf16 one.
 *
 * Defined by: aicassindra "gpu_moe_all_to_all", "Latency-bound at decode,
 * bandwidth-bound at prefill" (send fewer bytes: a lower-precision dispatch
 * payload, because the expert matmul casts its input anyway) and
 * "Bucketing" (the permutation fused into the staging kernel); zenaique Q&A
 * "moe-hide-alltoall-techniques" (shrink the payload). The pages fix no
 * format; this library's reading:
 *   - codes: OCP FP8 E4M3 (bias 7, largest finite 448, no infinities);
 *   - scales: one power of two 2^e per 32 consecutive values of a row,
 *     stored as the byte e + 127 (E8M0); e is the smallest integer >= -127
 *     with max|x| <= 448 * 2^e, so no value saturates;
 *   - code = the E4M3 value nearest to x / 2^e, ties to even (x / 2^e is
 *     exact, so the code does not depend on arithmetic precision);
 *   - a send row: H code bytes, then one 128-byte line per 4096 values
 *     holding that slab's 128 scale bytes, zero-padded in the last slab:
 *     moe_fp8_row_bytes(H) = H + 128 * ceil(H / 4096). For H % 128 == 0
 *     rows start on 128-byte lines and are written in whole lines; a
 *     destination's segment is still one contiguous range of rows.
 * NaN or infinite inputs give unspecified codes and scales.
 */

/* Bytes of one FP8 send row (written to *bytes). Needs H % 32 == 0. */
moe_status_t moe_fp8_row_bytes(int32_t H, int64_t *bytes);

/*
 * moe_dispatch_permute_fp8 -- as moe_dispatch_permute, but row pos[t][j] of
 * send ([send_rows][moe_fp8_row_bytes(H)] bytes, 16-byte aligned) receives
 * the FP8 codes, scale bytes and zero padding of x[t]. Rows no kept
 * assignment points at are left as they were. send_rows must cover the
 * same bound as in moe_dispatch_permute.
 * Errors: as moe_dispatch_permute; MOE_ERR_UNSUPPORTED when H % 32 != 0.
 */
moe_status_t moe_dispatch_permute_fp8(const uint16_t *x, const int32_t *pos, int64_t T,
                                      int32_t H, int32_t k, int32_t E, int32_t capacity,
                                      uint8_t *send, int64_t send_rows, void *stream);

/*
 * moe_fp8_dequant -- decode FP8 rows to bf16 (for an expert that takes
 * bf16, or to check a payload):
 *   out[i][h] = bf16 nearest to value(code[i][h]) * 2^(scale[i][h/32] - 127)
 * (ties to even; exact unless below bf16's subnormal spacing) for
 * i < min(*n_rows, max_rows), or i < max_rows when n_rows is NULL (n_rows
 * is a device pointer, e.g. expert_offsets + E). rows: [max_rows]
 * [moe_fp8_row_bytes(H)] bytes; out: [max_rows][H] bf16; both 16-byte
 * aligned. NaN codes give unspecified values.
 * Errors: MOE_ERR_INVALID_ARG (pointers, alignment, max_rows < 0),
 *   MOE_ERR_UNSUPPORTED (H limits, H % 32 != 0, max_rows >= 2^31).
 */
moe_status_t moe_fp8_dequant(const uint8_t *rows, const int32_t *n_rows, int64_t max_rows,
                             int32_t H, uint16_t *out, void *stream);

/*
 * Receive side: regroup a destination's receive buffer into expert-major
 * rows for the expert computation, and back for the return path.
 *
 * Defined by: aicassindra "gpu_moe_all_to_all", "Two collectives per layer"
 * (per-destination counts arrive before the payload so that the receiver
 * can size and place it; outputs return along the inverse permutation) and
 * "Bucketing" (one contiguous message per peer); "MoE All-to-All Dispatch
 * and Ragged Routing", "Why MoE Token Dispatch is All-to-All" (a GPU holds a
 * few of the experts) and "Fixed Capacity vs. Ragged Routing" (variable-
 * length exchange, the receiver pooling its local experts).
 *
 * The receive buffer is the concatenation, in source order, of one segment
 * per source s; each segment holds recv_counts[s][l] rows of local expert l
 * (l ascending), i.e. rows dest_offsets[r]..dest_offsets[r+1] of that
 * source's send buffer and expert_counts[r*E_l + l] of its counts. With
 * N = sum of recv_counts:
 *   local_expert_offsets[l] = rows of local experts < l     (E_l + 1 entries)
 *   source_offsets[s]       = rows of sources < s           (S + 1 entries)
 *   recv_pos[i]             = expert-major row of received row i: the block
 *                             (s, l) holding row i starts at
 *                             local_expert_offsets[l] + sum_{s' < s} recv_counts[s'][l]
 * so each local expert's rows are contiguous, sources in order within it.
 * N stays on the device: local_expert_offsets[E_l] == source_offsets[S].
 */

/* Workspace bytes for moe_recv_regroup_layout (written to *bytes). */
moe_status_t moe_recv_regroup_workspace_size(int32_t S, int32_t E_l, size_t *bytes);

/*
 * moe_recv_regroup_layout -- the offsets and recv_pos above.
 *   recv_counts [S][E_l] int32 (device; negative entries count as 0).
 *   recv_pos    [max_rows] int32; entries past N are not written, and rows
 *               past max_rows are not placed (a broken precondition when
 *               N > max_rows).
 *   workspace   moe_recv_regroup_workspace_size() bytes, 16-byte aligned;
 *               contents on entry do not matter.
 * Limits: 1 <= S, E_l <= 1024 and S * E_l <= 4096; max_rows < 2^31.
 * Device-side precondition: the counts total less than 2^31.
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE.
 */
moe_status_t moe_recv_regroup_layout(const int32_t *recv_counts, int32_t S, int32_t E_l,
                                     int32_t *local_expert_offsets,
                                     int32_t *source_offsets, int32_t *recv_pos,
                                     int64_t max_rows, void *workspace,
                                     size_t workspace_bytes, void *stream);

/*
 * moe_recv_regroup -- grouped[recv_pos[i]][:] = recv[i][:] for i < N (bit
 * copies of bf16 rows). n_rows points at N on the device (for example
 * source_offsets + S); max_rows bounds the grid and both buffers' rows.
 * recv and grouped are [max_rows][H] bf16, 16-byte aligned, not aliased.
 * moe_recv_ungroup -- the inverse for the return path:
 *   out[i][:] = grouped[recv_pos[i]][:] for i < N,
 * after which out is in receive order again and segment s goes back to
 * source s, landing in exactly the rows that source's combine reads.
 * Positions outside [0, max_rows) are skipped, never accessed.
 * Errors: MOE_ERR_INVALID_ARG (pointers, alignment, max_rows < 0),
 *   MOE_ERR_UNSUPPORTED (H limits, max_rows >= 2^31).
 */
moe_status_t moe_recv_regroup(const uint16_t *recv, const int32_t *recv_pos,
                              const int32_t *n_rows, int64_t max_rows, int32_t H,
                              uint16_t *grouped, void *stream);
moe_status_t moe_recv_ungroup(const uint16_t *grouped, const int32_t *recv_pos,
                              const int32_t *n_rows, int64_t max_rows, int32_t H,
                              uint16_t *out, void *stream);

/*
 * Tile-signalled return: a stand-in expert computation on a destination's
 * receive buffer whose output tiles are returned to their sources as soon
 * as they are ready.
 *
 * Defined by: thecoregrid "Mixture-of-experts acceleration through
 * overlap" (a producer GEMM and a consumer synchronised per tile: the GEMM
 * epilogue publishes a readiness flag per tile, and the consumer starts a
 * transfer once enough row bands are ready, several bands per transfer;
 * each tile belongs to one destination, the remote-owner-aligned layout,
 * and remote tiles are computed first; compute units are split between the
 * roles); aicassindra "gpu_moe_all_to_all", "Overlapping dispatch with
 * expert compute" (dispatch, compute and combine form a strict chain).
 *
 * The receive buffer recv [max_rows][H] bf16 is laid out as in
 * moe_recv_regroup_layout: S source segments in order, each holding
 * recv_counts[s][l] rows of local expert l, l ascending. The stand-in
 * expert is one linear map per local expert, W [E_l][H_out][H] bf16
 * (output-major, as a linear layer's weight):
 *   y[i][o] = bf16( sum_h recv[i][h] * W[l][o][h] )
 * accumulated in fp32 (MFMA) and rounded once, to nearest even, for every
 * row i < N = sum of the counts (rows past N are not written). Tiles are
 * 128 rows of one (source, expert) block by 512 output columns (the last
 * narrower when H_out % 512 != 0), so every tile goes back to exactly one
 * source.
 *
 * Limits: as moe_recv_regroup_layout for S and E_l; H % 64 == 0,
 * H_out % 128 == 0, both <= 65536; max_rows < 2^31. Buffers 16-byte
 * aligned; recv, W, y and ret do not overlap. Device-side precondition:
 * N <= max_rows. If it fails, nothing is computed and the status word
 * (below) reads 2.
 *
 * Workspace: moe_expert_linear_workspace_size() bytes, 16-byte aligned.
 * Its first int32 is a status word, which the caller may read after the
 * call completes: 0 = done; 1 = a consumer wait exceeded its bound and
 * some rows of ret were not returned; 2 = counts total more than max_rows.
 */
moe_status_t moe_expert_linear_workspace_size(int32_t S, int32_t E_l, int64_t max_rows,
                                              size_t *bytes);

/* moe_expert_linear -- y only, as one grouped GEMM launch (the schedule
 * without overlap: the return starts after it completes). */
moe_status_t moe_expert_linear(const uint16_t *recv, const int32_t *recv_counts, int32_t S,
                               int32_t E_l, int32_t H, int32_t H_out, const uint16_t *W,
                               int64_t max_rows, uint16_t *y, void *workspace,
                               size_t workspace_bytes, void *stream);

/*
 * moe_expert_linear_return -- y as above, and ret [max_rows][H_out] bf16
 * with ret[i] = y[i] for i < N: the rows returned to their sources (on one
 * device the sources' return buffers are partitions of ret, in the same
 * row positions, so moe_combine_reduce reads ret unchanged).
 *
 * One cooperative launch of moe_expert_return_slots() blocks, all resident.
 *   - Work units (a band -- the 128-row tile of one (source, expert) block --
 *     by one 512-column tile) go in remote-first order: sources
 *     self_rank+1, self_rank+2, ... (mod S), self_rank last.
 *   - After each unit a producer release-adds one to the band's count of
 *     column tiles.
 *   - A task is up to band_group consecutive bands of one source: one
 *     contiguous copy of rows from y to ret.
 * consumer_blocks > 0: that many blocks only return rows. Each takes tasks
 *   in order, waits until every band of the task has all its column tiles,
 *   and copies it. Every wait is bounded; on expiry the status word reads 1
 *   and that task is skipped, so no call hangs.
 * consumer_blocks == 0: every block computes. The unit that completes a
 *   band counts it toward its task, and the block that completes a task's
 *   last band copies the task itself. Nothing waits.
 * Errors: as moe_expert_linear; MOE_ERR_INVALID_ARG for self_rank outside
 *   [0, S), consumer_blocks < 0 or band_group < 1; MOE_ERR_UNSUPPORTED when
 *   consumer_blocks >= moe_expert_return_slots().
 */
moe_status_t moe_expert_linear_return(const uint16_t *recv, const int32_t *recv_counts,
                                      int32_t S, int32_t E_l, int32_t H, int32_t H_out,
                                      const uint16_t *W, int64_t max_rows, int32_t self_rank,
                                      int32_t consumer_blocks, int32_t band_group, uint16_t *y,
                                      uint16_t *ret, void *workspace, size_t workspace_bytes,
                                      void *stream);

/* Blocks of one moe_expert_linear_return launch on the current device
 * (resident blocks per compute unit x compute units). */
moe_status_t moe_expert_return_slots(int32_t *slots);

/*
 * Scored routing, the combine's gradient and the experts' products, forward
 * and backward: the rest of a trained mixture-of-experts layer around the
 * dispatch path. A layer's forward pass is route -> layout -> permute ->
 * expert products -> combine; its backward pass is moe_combine_backward ->
 * the products' gradients -> moe_combine_reduce with every weight 1 (the
 * permute's gradient: the sum of a token's replica rows) ->
 * moe_route_scored_backward.
 */

/* moe_route_scored flags, beside MOE_ROUTE_NORMALIZE */
#define MOE_SCORE_SIGMOID 2u  /* scores are sigmoid(logit); else softmax over all E */
#define MOE_GROUP_TOP2 4u     /* a group's score is the sum of its two best, not its best */
#define MOE_LOGITS_BF16 8u    /* logits (and their gradient) are bf16, else float32 */

/*
 * moe_route_scored -- top-k routing on scores: the selection bias is added
 * to the score (moe_route_topk adds it to the logit), scores are a sigmoid
 * of each logit or the softmax of all, and groups may be ranked by their
 * two best.
 *
 * Defined by: ai-from-scratch "19. All-to-all", "Why the router can ruin
 * your day" (the balancing bias takes part in the selection only) and
 * "DeepSeek's numbers" (each token limited to a few groups of experts).
 *
 * For each token t:
 *   p[e] = 1 / (1 + exp(-l[e])) with MOE_SCORE_SIGMOID, else
 *          exp(l[e]) / sum over all E of exp(l)
 *   s[e] = p[e] + bias[e]  (bias may be NULL: s = p)
 *   A logit of -inf masks its expert: p = 0 and s = -inf, whatever the bias.
 *   Groups (n_groups > topk_groups): the E experts form n_groups contiguous
 *     groups; a group's score is its best s, or with MOE_GROUP_TOP2 the sum
 *     of its two best (its only s when it has one expert); the best
 *     topk_groups groups take part, ties to the lower group.
 *   topk_idx = the k experts with the largest s among those, descending,
 *     ties to the smaller id. A NaN s ranks below every other.
 *   The order is that of s in exact arithmetic: without a bias that of the
 *     logits, and with one to the resolution of 64-bit floating point (where
 *     two scores lie closer than float32 resolves, the token is ranked again
 *     in 64 bits).
 *   topk_w[j] = scale * p[e_j] / sum_i p[e_i] with MOE_ROUTE_NORMALIZE, else
 *     scale * p[e_j]; computed in float32. Normalised weights keep the ratios
 *     of scores below float32's range. Masked experts, which are selected only
 *     when too few others are left, get 0; a row whose selected experts are all
 *     masked gets zeros.
 *   For a row that holds NaN or +inf under softmax, ids are distinct and in
 *     range and nothing else is specified.
 *
 * Arguments:
 *   logits   [T][E] float32, or bf16 with MOE_LOGITS_BF16; aligned to their
 *            elements.
 *   bias     [E] float32 or NULL.
 *   n_groups, topk_groups  as moe_route_topk_grouped; 1, 1 for no groups.
 *   scale    finite factor of the weights.
 *   topk_idx [T][k] int32 out;  topk_w [T][k] float32 out.
 * Errors: as moe_route_topk_grouped; MOE_ERR_INVALID_ARG for a scale that is
 *   not finite.
 */
moe_status_t moe_route_scored(const void *logits, const float *bias, int64_t T, int32_t E,
                              int32_t k, int32_t n_groups, int32_t topk_groups, float scale,
                              uint32_t flags, int32_t *topk_idx, float *topk_w, void *stream);

/*
 * moe_route_scored_backward -- the gradient of moe_route_scored's weights
 * with respect to the logits, given grad_w = dL/dtopk_w. The selection is
 * not differentiated, so the bias gets no gradient. With g = grad_w, sums
 * over the k selected:
 *   softmax, normalised:  dl[e_j] = w_j (g_j - sum_i g_i w_i / scale)
 *   sigmoid, normalised:  dl[e_j] = w_j (1 - p_j) (g_j - sum_i g_i w_i / scale)
 *   sigmoid:              dl[e_j] = scale g_j p_j (1 - p_j)
 *   softmax:              dl[e] = scale p_e ((g_j if e = e_j, else 0) - sum_i g_i p_i)
 * and 0 for every other expert. Scores are recomputed from the logits.
 *
 * Arguments: logits, k, scale and flags as given to moe_route_scored
 *   (MOE_GROUP_TOP2 has no effect on the gradient and is not accepted).
 *   topk_idx  [T][k] int32, distinct within a row; ids outside [0, E) are
 *             left out of the sums.
 *   grad_w    [T][k] float32.
 *   grad_logits [T][E] out, every element written, in the logits' type; must
 *             not alias logits.
 * Errors: as moe_route_scored.
 */
moe_status_t moe_route_scored_backward(const void *logits, const int32_t *topk_idx,
                                       const float *grad_w, int64_t T, int32_t E, int32_t k,
                                       float scale, uint32_t flags, void *grad_logits,
                                       void *stream);

/*
 * moe_combine_backward -- the gradients of moe_combine_reduce's sum, given
 * grad_out = dL/dout: for every kept replica
 *   grad_y[pos[t][j]][h] = bf16( topk_w[t][j] * grad_out[t][h] )
 *   grad_w[t][j]         = sum_h grad_out[t][h] * y[pos[t][j]][h]   (float32)
 * and grad_w[t][j] = 0 for a dropped one. Rows of grad_y that no replica
 * points at are not written. The gradients of shared and residual are
 * grad_out itself.
 *
 * Defined by: as moe_combine_reduce, whose derivative this is.
 *
 * Arguments:
 *   grad_out  [T][H] bf16, or float32 with MOE_COMBINE_OUT_FP32; 16-byte
 *             aligned.
 *   y         [y_rows][H] bf16, 16-byte aligned; NULL when grad_w is NULL.
 *   pos       [T][k] int32, every row at most once; positions outside
 *             [0, y_rows) count as dropped.
 *   topk_w    [T][k] float32; NULL when grad_y is NULL.
 *   grad_y    [y_rows][H] bf16 out, 16-byte aligned, or NULL.
 *   grad_w    [T][k] float32 out, or NULL (not both NULL).
 *   No output may alias an input.
 * Errors: as moe_combine_reduce.
 */
moe_status_t moe_combine_backward(const void *grad_out, const uint16_t *y, int64_t y_rows,
                                  const int32_t *pos, const float *topk_w, int64_t T, int32_t H,
                                  int32_t k, uint32_t flags, uint16_t *grad_y, float *grad_w,
                                  void *stream);

/* activations of the experts' products */
typedef enum moe_act {
    MOE_ACT_NONE = 0,
    MOE_ACT_RELU = 1,
    MOE_ACT_SILU = 2,      /* z / (1 + exp(-z)) */
    MOE_ACT_GELU = 3,      /* z (1 + erf(z / sqrt(2))) / 2 */
    MOE_ACT_GELU_TANH = 4  /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */
} moe_act_t;

/* moe_expert_product and moe_expert_product_dgrad flags */
#define MOE_PRODUCT_GATED 1u  /* the activation of one half gates the other */

/*
 * moe_expert_product -- each local expert's linear map on its rows, with
 * bias, activation, gate and residual applied before the one rounding:
 *   z[i][o] = sum_h x[i][h] * W[l][o][h] + bias[l][o]     (row i of expert l)
 *   y[i][o] = bf16( act(z[i][o]) + residual[i][o] ), or with
 *             MOE_PRODUCT_GATED, where W and bias hold 2 O outputs per expert
 *             (gate first),  bf16( act(z[i][o]) * z[i][O + o] + residual[i][o] )
 *   pre[i]  = bf16(z[i]) where pre is given (what the backward pass reads).
 * Products accumulate in float32 (MFMA); z stays in float32 until the
 * result is rounded to nearest even.
 *
 * Rows are expert-major: expert l owns rows expert_offsets[l] to
 * expert_offsets[l + 1], as moe_dispatch_layout (all experts local) and
 * moe_recv_regroup_layout (local_expert_offsets) write them; an expert may
 * have none. Rows from expert_offsets[E_l] on are neither read nor written.
 * An always-active shared expert is E_l = 1 with offsets {0, T}.
 * Whether the kernel for few rows per expert runs follows from max_rows / E_l,
 * since the offsets are on the device: for decoding, a max_rows near the rows
 * there are is up to twice as fast as one for the worst case.
 *
 * Defined by: "MoE All-to-All Dispatch and Ragged Routing", "Why MoE Token
 * Dispatch is All-to-All" (a GPU computes its local experts on the rows it
 * received) and "Fixed Capacity vs. Ragged Routing" (variable lengths).
 *
 * Arguments:
 *   x         [max_rows][H] bf16.
 *   expert_offsets [E_l + 1] int32 on the device, not decreasing, in
 *             [0, max_rows]. Values outside are clamped and nothing is
 *             computed where they decrease, so a broken precondition
 *             accesses no row outside the buffers.
 *   W         [E_l][O][H] bf16 ([E_l][2 O][H] gated).
 *   bias      [E_l][O] ([E_l][2 O]) bf16 or NULL.
 *   residual  [max_rows][O] bf16 or NULL; may be y itself.
 *   act       a moe_act value.
 *   pre       [max_rows][O] ([max_rows][2 O]) bf16 out or NULL.
 *   y         [max_rows][O] bf16 out.
 *   Buffers are 16-byte aligned, expert_offsets 4-byte; outputs alias no
 *   input but residual.
 * Limits: 1 <= E_l <= 1024; H % 8 == 0, O % 8 == 0, both in [8, 65536];
 *   max_rows < 2^31.
 * Errors: MOE_ERR_INVALID_ARG (pointers, alignment, max_rows < 0, unknown act
 *   or flags), MOE_ERR_UNSUPPORTED (limits).
 */
moe_status_t moe_expert_product(const uint16_t *x, const int32_t *expert_offsets, int32_t E_l,
                                int64_t max_rows, int32_t H, int32_t O, const uint16_t *W,
                                const uint16_t *bias, const uint16_t *residual, int32_t act,
                                uint32_t flags, uint16_t *pre, uint16_t *y, void *stream);

/*
 * moe_expert_product_dgrad -- the gradient of a product with respect to its
 * input, through the activation that made that input:
 *   d[i][h] = sum_o grad_y[i][o] * W[l][o][h]              (row i of expert l)
 *   pre NULL:  grad_x[i][h] = bf16( d[i][h] )
 *   pre given: the input was act(pre); grad_x = bf16( d * act'(pre) )
 *   MOE_PRODUCT_GATED: the input was act(pre[:, :H]) * pre[:, H:];
 *     grad_x[i][h]     = bf16( d * pre[i][H + h] * act'(pre[i][h]) )
 *     grad_x[i][H + h] = bf16( d * act(pre[i][h]) )
 * With the pre of the product before it, grad_x is the gradient of that
 * product's z, from which its own weight and input gradients follow.
 *
 * Arguments: as moe_expert_product; grad_y [max_rows][O] bf16,
 *   W [E_l][O][H] bf16, pre [max_rows][H] ([max_rows][2 H] gated) bf16 or
 *   NULL, grad_x [max_rows][H] ([max_rows][2 H] gated) bf16 out, which may be
 *   pre itself. Rows from expert_offsets[E_l] on are neither read nor
 *   written. Without pre, act must be MOE_ACT_NONE and flags 0.
 * Errors: as moe_expert_product.
 */
moe_status_t moe_expert_product_dgrad(const uint16_t *grad_y, const int32_t *expert_offsets,
                                      int32_t E_l, int64_t max_rows, int32_t O, int32_t H,
                                      const uint16_t *W, const uint16_t *pre, int32_t act,
                                      uint32_t flags, uint16_t *grad_x, void *stream);

/* moe_expert_product_wgrad flags */
#define MOE_GRAD_FP32 1u        /* grad_W is float32, else bf16 */
#define MOE_GRAD_ACCUMULATE 2u  /* add to grad_W (float32 only) and grad_bias */

/*
 * moe_expert_product_wgrad -- the gradients of a product's weights and bias:
 *   grad_W[l][o][h] = sum over expert l's rows i of grad_y[i][o] * x[i][h]
 *   grad_bias[l][o] = sum over expert l's rows i of grad_y[i][o]
 * accumulated in float32. Every element is written: an expert without rows
 * gets zeros, or keeps what it had with MOE_GRAD_ACCUMULATE. For a gated
 * product O is the 2 O of its forward call.
 *
 * Arguments: as moe_expert_product; grad_y [max_rows][O], x [max_rows][H]
 *   bf16; grad_W [E_l][O][H] bf16 or float32 out; grad_bias [E_l][O] float32
 *   out or NULL; workspace of moe_expert_product_wgrad_workspace_size()
 *   bytes, 16-byte aligned, contents on entry do not matter (NULL when the
 *   size is 0). Calls that overlap in time must not share a workspace.
 * Errors: as moe_expert_product; MOE_ERR_INVALID_ARG for accumulation into
 *   bf16; MOE_ERR_WORKSPACE.
 */
moe_status_t moe_expert_product_wgrad_workspace_size(int32_t E_l, int64_t max_rows, int32_t O,
                                                     int32_t H, size_t *bytes);
moe_status_t moe_expert_product_wgrad(const uint16_t *grad_y, const uint16_t *x,
                                      const int32_t *expert_offsets, int32_t E_l,
                                      int64_t max_rows, int32_t O, int32_t H, uint32_t flags,
                                      void *grad_W, float *grad_bias, void *workspace,
                                      size_t workspace_bytes, void *stream);

/* moe_rms_norm and moe_rms_norm_backward flags */
#define MOE_NORM_FP32 1u         /* x, residual, total and their gradients are float32, else bf16 */
#define MOE_NORM_WEIGHT_FP32 2u  /* weight is float32, else bf16 */
#define MOE_NORM_ACCUMULATE 4u   /* backward: add to grad_weight */

/*
 * moe_rms_norm -- the norm in front of the layer, with the residual's
 * addition:
 *   total[t] = round(x[t] + residual[t])        (x[t] itself without residual)
 *   v[t][h]  = total[t][h] * rsqrt(mean over h of total[t][h]^2 + eps) * weight[h]
 *   y[t]     = bf16(v[t])                       where y is given
 *   y8[t]    = v[t] as an FP8 row               where y8 is given
 * The norm is of total as it is stored, so that the backward pass, which reads
 * it, differentiates the function that ran. Sums and v are float32; y and y8
 * are each one rounding of v. y is what the router reads, and y8 has the
 * format of moe_dispatch_permute_fp8's rows (codes, scale bytes, zero padding):
 * moe_dispatch_permute moves FP8 rows as bf16 rows of moe_fp8_row_bytes(H) / 2
 * columns, and moe_expert_product_fp8 multiplies them. A v that is NaN
 * becomes a NaN code. A row of total with a NaN gives NaN throughout, one with
 * an infinity NaN there and zeros elsewhere.
 *
 * Defined by: ai-from-scratch "19. All-to-all", intro (every token's vector
 * after attention enters the layer) and "MoE All-to-All Dispatch and Ragged
 * Routing", "Returning Tokens to the Original GPU" (the residual stream);
 * aicassindra "gpu_moe_all_to_all", "Latency-bound at decode, bandwidth-bound
 * at prefill" (a lower-precision payload). The pages name no norm; this is the
 * root-mean-square one.
 *
 * Arguments:
 *   x         [T][H] bf16, or float32 with MOE_NORM_FP32.
 *   residual  [T][H] as x, or NULL.
 *   weight    [H] bf16, or float32 with MOE_NORM_WEIGHT_FP32.
 *   eps       finite, >= 0.
 *   total     [T][H] as x out; needed with residual, not accepted without it;
 *             may be x or residual.
 *   y         [T][H] bf16 out or NULL;  y8 [T][moe_fp8_row_bytes(H)] bytes out
 *             or NULL; not both NULL. Neither may alias an input or total.
 *   Buffers are 16-byte aligned.
 * Limits: T < 2^31, H % 8 == 0 (H % 32 == 0 with y8), 0 < H <= 65536. A row's
 *   sum of squares must lie within float32's range.
 * Errors: MOE_ERR_INVALID_ARG (pointers, alignment, T < 0, eps, unknown flags),
 *   MOE_ERR_UNSUPPORTED (limits).
 */
moe_status_t moe_rms_norm(const void *x, const void *residual, const void *weight, int64_t T,
                          int32_t H, float eps, uint32_t flags, void *total, uint16_t *y,
                          uint8_t *y8, void *stream);

/*
 * moe_rms_norm_backward -- the gradients of moe_rms_norm's v. With
 * r = rsqrt(mean(total^2) + eps), recomputed from total, and g = grad_y * weight:
 *   grad_x[t][h]   = r (g[h] - total[t][h] r^2 mean(g * total[t])) + grad_total[t][h]
 *   grad_weight[h] = sum over t of grad_y[t][h] * total[t][h] * r
 * grad_x is the gradient of x and of residual alike; grad_total is what
 * reaches the residual stream from behind the layer. FP8 rows are
 * differentiated as the values that they round (straight through). Every
 * element of grad_weight is written (T = 0: zeros, or what it had with
 * MOE_NORM_ACCUMULATE); the sum's order depends on T and H only.
 *
 * Arguments:
 *   grad_y      [T][H] bf16.
 *   total       [T][H] as moe_rms_norm stored it (x where it had no residual).
 *   weight, eps, flags  as moe_rms_norm's, and MOE_NORM_ACCUMULATE.
 *   grad_total  [T][H] as x, or NULL (zero).
 *   grad_x      [T][H] as x out, or NULL; may be grad_total.
 *   grad_weight [H] float32 out, or NULL (not both NULL).
 *   workspace   moe_rms_norm_backward_workspace_size() bytes, 16-byte aligned,
 *               contents on entry do not matter (NULL when the size is 0).
 *               Without grad_weight 8 T bytes where H > 16384, else none (NULL).
 *               Calls that overlap in time must not share a workspace.
 * Errors: as moe_rms_norm; MOE_ERR_WORKSPACE.
 */
moe_status_t moe_rms_norm_backward_workspace_size(int64_t T, int32_t H, size_t *bytes);
moe_status_t moe_rms_norm_backward(const uint16_t *grad_y, const void *total, const void *weight,
                                   int64_t T, int32_t H, float eps, uint32_t flags,
                                   const void *grad_total, void *grad_x, float *grad_weight,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* moe_fp8_quantize_weights flags */
#define MOE_WEIGHTS_FP32 1u  /* W is float32, else bf16 */

/*
 * moe_fp8_quantize_weights -- the experts' weights in 8 bits, with a float32
 * scale for each block of 128 x 128 (smaller at the lower and right edges):
 *   scale[l][a][b] = max|W[l]| in rows 128 a.. and columns 128 b.., over 448
 *                    (1 for a block of zeros; at least 2^-126)
 *   codes[l][o][h] = E4M3 nearest to W[l][o][h] * (1 / scale), ties to even
 * and, where codes_t is given, both transposed, as the input gradient reads
 * them: codes_t[l][h][o] = codes[l][o][h], scale_t[l][b][a] = scale[l][a][b].
 * NaN and infinite weights get the NaN code; an infinity makes its block's
 * scale infinite.
 *
 * Defined by: aicassindra "gpu_moe_all_to_all", "Latency-bound at decode,
 * bandwidth-bound at prefill" (the expert matmul casts its input to a lower
 * precision); the blocks are this library's reading.
 *
 * Arguments: W [n][O][H] bf16, or float32 with MOE_WEIGHTS_FP32; codes
 *   [n][O][H] bytes, scale [n][ceil(O/128)][ceil(H/128)] float32 out; codes_t
 *   [n][H][O] bytes and scale_t [n][ceil(H/128)][ceil(O/128)] float32 out, or
 *   both NULL. W, codes and codes_t are 16-byte aligned. No output aliases W.
 * Limits: 0 <= n <= 1024; O and H multiples of 32 in [32, 65536] (131072 for O,
 *   the rows of a gated weight).
 * Errors: MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED.
 */
moe_status_t moe_fp8_quantize_weights(const void *W, int32_t n, int32_t O, int32_t H,
                                      uint32_t flags, uint8_t *codes, float *scale,
                                      uint8_t *codes_t, float *scale_t, void *stream);

/*
 * moe_expert_product_fp8 -- moe_expert_product on FP8 rows and 8-bit weights:
 *   z[i][o] = sum_h x[i][h] * W[l][o][h] + bias[l][o]
 *     x[i][h]    = value(code) * 2^(scale byte - 127)     (row i, moe_fp8_dequant's value)
 *     W[l][o][h] = value(W code[l][o][h]) * W_scale[l][o / 128][h / 128]
 * with the bias, activation, gate and residual of moe_expert_product, and the
 * result v to y (bf16), to y8 (FP8 rows of O values, the next product's input)
 * or to both, each one rounding of the float32 v. The matrix
 * units sum the products of 128 values, which are added up in float32 with the
 * weights' scale. They align the products of eight neighbouring h to the
 * largest one, and keep of the others what is not below 2^-13 of its power of
 * two: the eight's sum is off by less than 2^-10 of the largest product. Where
 * rows fill tiles of 256, the sum is kept in units of the scale over its power
 * of two, and changes units from one 128 to the next, which rounds it by less
 * than 2^-22 of itself each time.
 * A weights' scale below 2^-126 may count as 2^-127; one that is infinite or
 * NaN makes the results that it reaches infinite or NaN, and so does a NaN
 * code or a row's scale byte 255. A v that is NaN or infinite becomes a NaN
 * code in y8. The order of an element's sum depends on max_rows, E_l, H, O and
 * expert_offsets; equal calls give equal bits.
 *
 * Defined by: as moe_expert_product, and aicassindra "gpu_moe_all_to_all",
 * "Latency-bound at decode, bandwidth-bound at prefill" (the expert matmul in
 * the payload's precision).
 *
 * Arguments: as moe_expert_product, but
 *   x         [max_rows][moe_fp8_row_bytes(H)] bytes, as moe_dispatch_permute_fp8,
 *             moe_rms_norm and this call write them.
 *   W         [E_l][O][H] bytes ([E_l][2 O][H] gated), E4M3 codes.
 *   W_scale   [E_l][ceil(O/128)][ceil(H/128)] float32 (gated: ceil(2 O/128); its
 *             blocks run over all 2 O rows), 4-byte aligned.
 *   y         [max_rows][O] bf16 out or NULL;  y8 [max_rows]
 *             [moe_fp8_row_bytes(O)] bytes out or NULL; not both NULL. Rows
 *             from expert_offsets[E_l] on are neither read nor written.
 * Limits: as moe_expert_product, with H % 32 == 0 and O % 32 == 0. The rows'
 *   sums over 128 values, before the weights' scale, must lie within
 *   float32's range (rows below 2^100 do).
 * Errors: as moe_expert_product.
 */
moe_status_t moe_expert_product_fp8(const uint8_t *x, const int32_t *expert_offsets, int32_t E_l,
                                    int64_t max_rows, int32_t H, int32_t O, const uint8_t *W,
                                    const float *W_scale, const uint16_t *bias,
                                    const uint16_t *residual, int32_t act, uint32_t flags,
                                    uint16_t *pre, uint16_t *y, uint8_t *y8, void *stream);

/*
 * moe_expert_product_fp8_dgrad -- moe_expert_product_dgrad on FP8 rows and the
 * transposed 8-bit weights:
 *   d[i][h] = sum_o grad_y[i][o] * W[l][o][h]
 * through the activation as there, to grad_x (bf16, what the weights' gradient
 * reads), to grad_x8 (FP8 rows, what the gradient of the product before it
 * reads) or to both. The weights' gradient itself sums over rows, along which
 * FP8 rows share no scale: it is moe_expert_product_wgrad on bf16 rows.
 *
 * Arguments: as moe_expert_product_dgrad, but
 *   grad_y    [max_rows][moe_fp8_row_bytes(O)] bytes.
 *   W_t       [E_l][H][O] bytes and W_t_scale [E_l][ceil(H/128)][ceil(O/128)]
 *             float32: moe_fp8_quantize_weights' codes_t and scale_t (of a
 *             gated product: H, and O = its 2 O rows).
 *   grad_x    [max_rows][H] ([max_rows][2 H] gated) bf16 out or NULL; may be pre
 *             itself.
 *   grad_x8   [max_rows][moe_fp8_row_bytes(H)] (of 2 H gated) bytes out or NULL;
 *             not both NULL.
 * Limits: as moe_expert_product_fp8, and 2 H <= 65536 gated with grad_x8.
 * Errors: as moe_expert_product_dgrad.
 */
moe_status_t moe_expert_product_fp8_dgrad(const uint8_t *grad_y, const int32_t *expert_offsets,
                                          int32_t E_l, int64_t max_rows, int32_t O, int32_t H,
                                          const uint8_t *W_t, const float *W_t_scale,
                                          const uint16_t *pre, int32_t act, uint32_t flags,
                                          uint16_t *grad_x, uint8_t *grad_x8, void *stream);

/* moe_hbm_floor flags */
#define MOE_FLOOR_NT_STORE 1u  /* stores carry the non-temporal hint */

/*
 * moe_hbm_floor -- the synthetic floor: read read_bytes from src and write
 * write_bytes to dst, both contiguous, with the 16-byte lane accesses of
 * the row kernels and nothing else (no gather, scatter or index). Timed
 * beside a call of the path with that call's read and write volumes, it is
 * the rate the memory system reaches for the same bytes; the gap is
 * overhead the path owns.
 *
 * Defined by: aicassindra "gpu_moe_all_to_all", "How to tell whether the
 * all-to-all is your bottleneck" (time a synthetic transfer of the same
 * sizes and compare).
 *
 * Arguments: src [read_bytes], dst [write_bytes], 16-byte aligned, not
 *   overlapping; sizes multiples of 16. dst receives the first write_bytes
 *   of src (a constant pattern past read_bytes); the contents are not part
 *   of the contract.
 * Errors: MOE_ERR_INVALID_ARG for negative or unaligned sizes, NULL or
 *   misaligned pointers with a non-zero size, or unknown flags.
 */
moe_status_t moe_hbm_floor(const void *src, int64_t read_bytes, void *dst,
                           int64_t write_bytes, uint32_t flags, void *stream);

/* moe_status_string -- a static, human-readable name for a status. */
const char *moe_status_string(moe_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EP_H */
