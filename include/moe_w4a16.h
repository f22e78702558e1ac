/*
 * moe_w4a16.h - C ABI of libmoe_w4a16.so, a routed-expert mixture-of-experts
 * layer with W4A16 group-32 expert weights for AMD Instinct MI355X (gfx950).
 *
 * The layer is the one tuned across a 512-expert, top-10, hidden-2560 model on
 * the pages "[Model][SM70] Adapt Qwen3.8 Flash Next NVFP4" (section
 * "Implemented route": the (2560, 640, 512, top-10) routed-expert geometry) and
 * "[Perf][SM70] Narrow Qwen3.8 AWQ active grouped decode" (section "Purpose":
 * AWQ W4A16 with effective group size 32, a grouped operator over active
 * experts, multi-row active-expert segments with offsets-based scheduling, and
 * scratch buffers the operator mutates).  One layer call is, in order:
 *
 *   moe_route              softmax over expert logits, top-k, renormalise
 *   moe_permute            token->expert permutation: segments and offsets
 *   moe_w4a16_grouped_ffn  dequant-fused gate/up GEMM, SiLU(gate)*up, down GEMM
 *   moe_combine            router-weighted sum back to token order
 *
 * Around it (the MoE block): moe_router_gate makes the logits from the
 * activations, and a shared expert runs on every token beside the routed
 * ones (moe_route_shared, moe_block_forward).
 *
 * Conventions for every entry point
 *   - Pointers to tensors are DEVICE pointers unless stated otherwise; fp16
 *     tensors are passed as uint16_t bit patterns.  Every non-null tensor
 *     pointer must be 16-byte aligned.  All tensors are dense, row-major.
 *   - Ownership: the caller allocates and frees every buffer, including the
 *     workspaces.  The library never allocates or frees memory and never
 *     synchronises.  Its only state is a per-device cache of two device
 *     attributes (compute-unit count, LDS bytes per workgroup) read from the
 *     runtime on first use, the per-device scratch array of
 *     moe_layer_forward_noalloc with its address cache, and the per-device
 *     completion counts of the one-launch FFN plan (moe_plan.one_launch),
 *     which every such call leaves at zero.  Entry points other than
 *     moe_layer_forward_noalloc, and plans other than one_launch, may be
 *     called from several host threads at once.
 *   - Work is enqueued on `stream` (a hipStream_t passed as void*; NULL is the
 *     default stream) and runs asynchronously.  A call that returns MOE_OK has
 *     only enqueued its kernels.
 *   - Errors: arguments are validated on the host before anything is enqueued;
 *     on a non-OK return nothing was enqueued, except MOE_ERR_HIP, which
 *     reports a failed launch (the library reads and clears hipGetLastError,
 *     so a pending error left by earlier unrelated work is reported too).
 *   - T == 0 is valid: the call returns MOE_OK, enqueues nothing and writes
 *     nothing; tensor pointers may then be NULL.
 *   - Device-side preconditions that are documented but not checked: logits
 *     are finite; expert ids are in [0, E) and distinct within a token (what
 *     moe_route produces); routing tensors passed to a later call are the
 *     unmodified outputs of the earlier calls of the same layer.
 *   - Results are deterministic: no step depends on the order in which
 *     threads or workgroups run, so a repeated call gives identical bits.
 *
 * Shapes.  T tokens, E experts, top_k experts per token, S = T * top_k slots
 * (slot s = t * top_k + j is the j-th choice of token t), hidden size H,
 * intermediate size I, group size 32 along the reduction dim K.
 *
 * Weight layout (N = output rows, K = reduction dim, G = K / 32):
 *   qweight int32 [E, N, K/8]   nibble j (bits 4j..4j+3) of word w is k = 8w+j
 *   scales  fp16  [E, N, G]
 *   qzeros  int32 [E, N/8, G]   nibble j of word w is row n = 8w+j
 *   dequantised weight  W[e, n, k] = (q - z[e, n, k/32]) * scales[e, n, k/32]
 * w13 has N = 2I, K = H (rows [0, I) gate, [I, 2I) up); w2 has N = H, K = I.
 *
 * Limits: 1 <= E <= 4096; 1 <= top_k <= min(E, 64); S < 2^31; group_size == 32;
 * H and I multiples of 32 with 32 <= H, I <= 16384; T * H < 2^31 (x is
 * addressed with 32-bit byte offsets).
 */
#ifndef MOE_W4A16_H_
#define MOE_W4A16_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes of every entry point. */
#define MOE_OK 0
#define MOE_ERR_INVALID_ARG 1 /* null/misaligned pointer, bad shape or count   */
#define MOE_ERR_UNSUPPORTED 2 /* valid but outside the limits (group_size...)  */
#define MOE_ERR_WORKSPACE 3   /* workspace_bytes below the size query's result */
#define MOE_ERR_HIP 4         /* a kernel launch failed                        */

/* Static, NUL-terminated description of a return code (host only). */
const char* moe_status_string(int status);

/* Library ABI version, MAJOR * 100 + MINOR (1.02: moe_plan gained one_launch). */
int moe_abi_version(void);

/*
 * moe_route - router softmax, top-k and renormalisation.
 *
 * For every token t: p = softmax(logits[t, :]); the top_k experts with the
 * largest logits are chosen in rank order (equal logits: lower expert index
 * first); weights[t, j] = p[id_j] / sum_j' p[id_j'].  Ranking is done on the
 * fp32 logits themselves, so the ids are exact.  The full-softmax denominator
 * cancels in the renormalisation and is not formed.
 * Source: the routed-expert top-10 geometry on "[Model][SM70] Adapt Qwen3.8
 * Flash Next NVFP4", section "Implemented route".
 *
 *   logits        in   fp32  [T, E]
 *   topk_ids      out  int32 [T, top_k]   expert ids in rank order
 *   topk_weights  out  fp32  [T, top_k]   sum to 1 per token
 */
int moe_route(const float* logits, int64_t T, int32_t E, int32_t top_k,
              int32_t* topk_ids, float* topk_weights, void* stream);

/*
 * moe_router_gate - the router's gate projection in front of moe_route:
 * logits[t, e] = sum_h x[t, h] * gate_weight[e, h], fp16 inputs, products
 * exact, sums in fp32.  "[Perf][SM70] Narrow Qwen3.8 AWQ active grouped
 * decode", section "Capacity, startup, and remaining limit", names this
 * projection among the costs beside the routed experts; the pages give no
 * formula, so this is the plain linear map without bias, with an unquantised
 * fp16 weight.  T <= 16: one GEMV launch bound by reading gate_weight; more
 * tokens: a matrix-core GEMM.  The order of every sum is fixed.
 *
 *   x            in   fp16 [T, H]
 *   gate_weight  in   fp16 [E, H]
 *   logits       out  fp32 [T, E]
 *
 * Limits: 1 <= E <= 4096; H a multiple of 32, <= 16384; T * H < 2^31.
 */
int moe_router_gate(const uint16_t* x, int64_t T, int32_t H,
                    const uint16_t* gate_weight, int32_t E, float* logits,
                    void* stream);

/*
 * moe_route_shared - moe_route for a layer with a shared expert: row t of
 * the outputs holds top_k + 1 entries, the top_k routed choices exactly as
 * moe_route gives them, then the shared expert, id E, with weight 1.  The
 * shared expert runs on every token with weight 1 beside the routed ones
 * ("[Perf][SM70] Narrow Qwen3.8 AWQ active grouped decode", section
 * "New-base bounded integration acceptance (r2)", names the shared overlap);
 * with these rows the permutation, the FFN and the combine treat it as expert
 * E of E + 1 experts, whose weights follow the routed experts' in the weight
 * arrays.
 *
 *   logits        in   fp32  [T, E]
 *   topk_ids      out  int32 [T, top_k + 1]
 *   topk_weights  out  fp32  [T, top_k + 1]
 *
 * Limits: as moe_route with top_k + 1 <= 64 and E + 1 <= 4096.
 */
int moe_route_shared(const float* logits, int64_t T, int32_t E, int32_t top_k,
                     int32_t* topk_ids, float* topk_weights, void* stream);

/* Workspace bytes moe_permute needs for these sizes (0 when T <= 64). */
size_t moe_permute_workspace_bytes(int64_t T, int32_t top_k, int32_t E);

/*
 * moe_permute - stable token-to-expert permutation: active-expert segments and
 * their offsets ("multi-row active-expert segments and offsets-based
 * scheduling", "[Perf][SM70] Narrow Qwen3.8 AWQ active grouped decode",
 * section "Purpose").
 *
 * Sorted row r belongs to expert e iff expert_offsets[e] <= r <
 * expert_offsets[e+1]; the rows of one expert are its slots in ascending slot
 * order.
 *
 *   topk_ids        in   int32 [T, top_k]
 *   expert_offsets  out  int32 [E + 1]   offsets[0] = 0, offsets[E] = S
 *   sorted_slots    out  int32 [S]       slot held by sorted row r
 *   slot_rows       out  int32 [S]       sorted row of slot s (inverse)
 *   active_experts  out  int32 [E]       experts with >= 1 row, ascending,
 *                                        then -1 up to E
 *   num_active      out  int32 [1]       number of active experts
 *   workspace       scratch, device, >= moe_permute_workspace_bytes(...)
 *                   bytes (may be NULL when that size is 0); contents on
 *                   entry are ignored.
 */
int moe_permute(const int32_t* topk_ids, int64_t T, int32_t top_k, int32_t E,
                int32_t* expert_offsets, int32_t* sorted_slots,
                int32_t* slot_rows, int32_t* active_experts,
                int32_t* num_active, void* workspace, size_t workspace_bytes,
                void* stream);

/*
 * moe_route_permute - moe_route followed by moe_permute, in one call: the
 * outputs of both, bit for bit identical to calling them in turn (routing of
 * "[Model][SM70] Adapt Qwen3.8 Flash Next NVFP4", section "Implemented route";
 * segments and offsets of "[Perf][SM70] Narrow Qwen3.8 AWQ active grouped
 * decode", section "Purpose").  For T <= 64 and E <= 1024 it is one kernel
 * launch (the decode path); otherwise it issues the two calls' kernels.
 *
 *   logits                                   in   fp32 [T, E], as moe_route
 *   topk_ids, topk_weights                   out  as moe_route
 *   expert_offsets, sorted_slots, slot_rows,
 *   active_experts, num_active               out  as moe_permute
 *   workspace       scratch, device, >= moe_permute_workspace_bytes(T,
 *                   top_k, E) bytes (0 when T <= 64; may then be NULL);
 *                   contents on entry are ignored.
 *
 * Errors as moe_route and moe_permute; nothing is enqueued on an error.
 */
int moe_route_permute(const float* logits, int64_t T, int32_t E, int32_t top_k,
                      int32_t* topk_ids, float* topk_weights,
                      int32_t* expert_offsets, int32_t* sorted_slots,
                      int32_t* slot_rows, int32_t* active_experts,
                      int32_t* num_active, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Workspace bytes the expert FFN entry points need for these sizes. */
size_t moe_ffn_workspace_bytes(int64_t T, int32_t top_k, int32_t E, int32_t H,
                               int32_t I);

/*
 * moe_w4a16_grouped_ffn - dequant-fused grouped expert FFN over the active
 * experts (the AWQ "active-stage" grouped W4A16 operator of "[Perf][SM70]
 * Narrow Qwen3.8 AWQ active grouped decode", section "Purpose"; W4A16 group
 * size 32 per "[Model][SM70] Support Qwen3.8 Flash Next with PLE offload",
 * section "SM70 QSA prefill tuning").
 *
 * For every sorted row r of expert e, with token t = sorted_slots[r] / top_k:
 *   h = x[t, :] . W13[e]^T                (2I values)
 *   a = SiLU(h[0:I]) * h[I:2I]            (I values, SiLU(v) = v / (1 + e^-v))
 *   y_sorted[r, :] = a . W2[e]^T          (H values)
 * Weights are dequantised exactly as (q - z) and scaled per 32-wide group in
 * fp32; x . W is accumulated in fp32 and a is carried to the down product at
 * about 22 bits of precision.  The kernel variant (bandwidth-bound decode
 * GEMV for T <= 8, matrix-core grouped GEMM otherwise) is chosen from T.
 *
 *   x                 in   fp16  [T, H]
 *   expert_offsets, sorted_slots, active_experts, num_active: moe_permute's
 *                     outputs for the same routing
 *   w13_qweight/scales/qzeros   in  W13 [E, 2I, H] in the layout above
 *   w2_qweight/scales/qzeros    in  W2  [E, H, I]  in the layout above
 *   group_size        must be 32
 *   y_sorted          out  fp32  [S, H]  per-row expert outputs, sorted order
 *   workspace         scratch, device, >= moe_ffn_workspace_bytes(...) bytes;
 *                     contents on entry are ignored.  Two calls that overlap
 *                     in time must not share a workspace.
 */
int moe_w4a16_grouped_ffn(
    const uint16_t* x, int64_t T, int32_t top_k, const int32_t* expert_offsets,
    const int32_t* sorted_slots, const int32_t* active_experts,
    const int32_t* num_active, const int32_t* w13_qweight,
    const uint16_t* w13_scales, const int32_t* w13_qzeros,
    const int32_t* w2_qweight, const uint16_t* w2_scales,
    const int32_t* w2_qzeros, int32_t E, int32_t H, int32_t I,
    int32_t group_size, float* y_sorted, void* workspace,
    size_t workspace_bytes, void* stream);

/*
 * moe_w4a16_gate_up / moe_w4a16_down - the two halves of
 * moe_w4a16_grouped_ffn, for callers that schedule or time them apart.
 * moe_w4a16_gate_up computes a = SiLU(h[0:I]) * h[I:2I] for every sorted row
 * into the workspace; moe_w4a16_down reads it and writes y_sorted.  A down
 * call must follow a gate_up call with the same routing, sizes and workspace,
 * on the same stream.  Arguments are as for moe_w4a16_grouped_ffn.
 */
int moe_w4a16_gate_up(const uint16_t* x, int64_t T, int32_t top_k,
                      const int32_t* expert_offsets,
                      const int32_t* sorted_slots,
                      const int32_t* active_experts,
                      const int32_t* num_active, const int32_t* w13_qweight,
                      const uint16_t* w13_scales, const int32_t* w13_qzeros,
                      int32_t E, int32_t H, int32_t I, int32_t group_size,
                      void* workspace, size_t workspace_bytes, void* stream);

int moe_w4a16_down(int64_t T, int32_t top_k, const int32_t* expert_offsets,
                   const int32_t* active_experts, const int32_t* num_active,
                   const int32_t* w2_qweight, const uint16_t* w2_scales,
                   const int32_t* w2_qzeros, int32_t E, int32_t H, int32_t I,
                   int32_t group_size, float* y_sorted, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * moe_route_gate_up - the first launch of moe_layer_forward at decode sizes:
 * the router, the permutation and the gate/up half of the FFN as one kernel
 * (every workgroup routes the tokens itself, so none waits for another;
 * workgroup 0 writes the routing out).  Its outputs equal those of
 * moe_route_permute followed by moe_w4a16_gate_up, bit for bit, and feed
 * moe_w4a16_down and moe_combine.  "[Perf][SM70] Narrow Qwen3.8 AWQ active
 * grouped decode", section "Capacity, startup, and remaining limit", names
 * each format's MoE preparation among the remaining decode costs; this takes
 * the preparation's launch out of the step.
 *
 *   logits, x        in   as moe_layer_forward
 *   w13_*            in   as moe_w4a16_grouped_ffn
 *   topk_ids ... num_active   out  as moe_route_permute
 *   workspace        FFN workspace (moe_ffn_workspace_bytes); holds act for
 *                    moe_w4a16_down afterwards
 *
 * MOE_ERR_UNSUPPORTED unless T <= 64 and E <= 1024 (moe_layer_forward uses
 * it up to 8 tokens, the default plan); other errors as the calls it stands
 * for.
 */
int moe_route_gate_up(const float* logits, const uint16_t* x, int64_t T,
                      int32_t E, int32_t top_k, const int32_t* w13_qweight,
                      const uint16_t* w13_scales, const int32_t* w13_qzeros,
                      int32_t H, int32_t I, int32_t group_size,
                      int32_t* topk_ids, float* topk_weights,
                      int32_t* expert_offsets, int32_t* sorted_slots,
                      int32_t* slot_rows, int32_t* active_experts,
                      int32_t* num_active, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * moe_combine - router-weighted combine back to token order.
 *
 *   out[t, h] = fp16_rne( sum_{j = 0..top_k-1} topk_weights[t, j] *
 *                          y_sorted[slot_rows[t * top_k + j], h] )
 * summed in fp32 in ascending j, rounded to fp16 once (round to nearest
 * even).  A gather without atomics.
 *
 *   y_sorted      in   fp32  [S, H]
 *   topk_weights  in   fp32  [T, top_k]
 *   slot_rows     in   int32 [S]
 *   out           out  fp16  [T, H]
 */
int moe_combine(const float* y_sorted, const float* topk_weights,
                const int32_t* slot_rows, int64_t T, int32_t top_k, int32_t H,
                uint16_t* out, void* stream);

/* Workspace bytes moe_layer_forward needs for these sizes. */
size_t moe_layer_workspace_bytes(int64_t T, int32_t top_k, int32_t E, int32_t H,
                                 int32_t I);

/*
 * moe_layer_forward - the whole routed-expert layer in one call:
 * moe_route_permute, moe_w4a16_grouped_ffn and moe_combine on the same
 * arguments, with the routing, the FFN scratch and y_sorted kept in the
 * workspace; out is what the four calls produce, bit for bit (the sections
 * cited above for each step).  For T <= 8 and E <= 1024 (decode) the gate/up
 * kernel routes the tokens itself, every workgroup the same way, which saves
 * the router/permutation launch.
 *
 *   logits      in   fp32 [T, E]
 *   x           in   fp16 [T, H]
 *   w13_*, w2_* in   as moe_w4a16_grouped_ffn
 *   group_size  must be 32
 *   out         out  fp16 [T, H]
 *   workspace   scratch, device, >= moe_layer_workspace_bytes(...) bytes;
 *               contents on entry are ignored.  After the call it holds, in
 *               order and each 256-byte aligned: topk_ids [S], topk_weights
 *               [S], expert_offsets [E+1], sorted_slots [S], slot_rows [S],
 *               active_experts [E], num_active [1], the permutation
 *               workspace, the FFN workspace and y_sorted [S, H].
 *
 * Errors as the calls it stands for; nothing is enqueued on an error.
 */
int moe_layer_forward(const float* logits, const uint16_t* x, int64_t T,
                      int32_t E, int32_t top_k, const int32_t* w13_qweight,
                      const uint16_t* w13_scales, const int32_t* w13_qzeros,
                      const int32_t* w2_qweight, const uint16_t* w2_scales,
                      const int32_t* w2_qzeros, int32_t H, int32_t I,
                      int32_t group_size, uint16_t* out, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Workspace bytes moe_block_forward needs for these sizes (0: invalid sizes). */
size_t moe_block_workspace_bytes(int64_t T, int32_t top_k, int32_t E,
                                 int32_t shared, int32_t H, int32_t I);

/*
 * moe_block_forward - the MoE block: moe_router_gate, then the routed layer,
 * plus the shared expert when shared == 1.  With shared == 0 it is
 * moe_router_gate followed by moe_layer_forward; with shared == 1 it is
 * moe_router_gate, moe_route_shared, then moe_permute, moe_w4a16_grouped_ffn
 * and moe_combine over E + 1 experts and top_k + 1 slots per token, so the
 * shared expert's rows run in the same launches as the routed experts' rows
 * and its output (weight 1) joins the fp32 sum before the one rounding to
 * fp16.  out is what those calls produce, bit for bit, when the plan keeps
 * the shared expert in the FFN's kernels (shared_mfma = 0); the default at
 * GEMV sizes from 3 tokens runs its rows on the matrix cores in extra
 * workgroups of the same launches (shared_mfma = 1), which changes the order
 * of its fp32 sums only, and where those rows do not fit in LDS (23 to 32
 * tokens at H = 2560) takes the matrix-core FFN instead.  Sections as moe_router_gate and moe_route_shared.
 *
 *   x            in   fp16 [T, H]
 *   gate_weight  in   fp16 [E, H]
 *   shared       0 or 1
 *   w13_*, w2_*  in   as moe_w4a16_grouped_ffn, for E + shared experts
 *                     (the shared expert is expert E)
 *   group_size   must be 32
 *   logits       out  fp32 [T, E]
 *   out          out  fp16 [T, H]
 *   workspace    scratch, device, >= moe_block_workspace_bytes(...) bytes;
 *                contents on entry are ignored.  After the call it holds the
 *                layout of moe_layer_forward's workspace for top_k + shared
 *                slots per token and E + shared experts.
 *
 * Errors as the calls it stands for; nothing is enqueued on an error.
 */
int moe_block_forward(const uint16_t* x, int64_t T, const uint16_t* gate_weight,
                      int32_t E, int32_t top_k, int32_t shared,
                      const int32_t* w13_qweight, const uint16_t* w13_scales,
                      const int32_t* w13_qzeros, const int32_t* w2_qweight,
                      const uint16_t* w2_scales, const int32_t* w2_qzeros,
                      int32_t H, int32_t I, int32_t group_size, float* logits,
                      uint16_t* out, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * Kernel variant and tile profile of a layer call.  Every entry point takes
 * its choices from moe_plan_default for its sizes; the _plan entry points
 * below take an explicit one (for measuring the alternatives).  The defaults
 * were chosen from a sweep on MI355X ("[Perf][SM70] Narrow Qwen3.8 AWQ
 * active grouped decode", section "Additional existing-autotune benefit
 * (fresh-process pair)": the tuned tile per shape, there a W13 tile change
 * from M64 x 128 x 32 to M8 x 256 x 64 at 4-8 tokens).
 */
#define MOE_FFN_GEMV 0            /* one weight stream per expert, A rows from LDS  */
#define MOE_FFN_MFMA 1            /* matrix-core grouped GEMMs                      */
#define MOE_ROUTE_IN_GATE_UP 0    /* the gate/up GEMV routes the tokens itself      */
#define MOE_ROUTE_ONE_LAUNCH 1    /* router and permutation in one launch           */
#define MOE_ROUTE_SEPARATE 2      /* router kernel, then the permutation kernels    */
typedef struct moe_plan {
  int32_t ffn;            /* MOE_FFN_GEMV or MOE_FFN_MFMA                            */
  int32_t route;          /* MOE_ROUTE_*                                              */
  int32_t msub;           /* MFMA: 32-row subtiles per M-tile, 1 or 4                 */
  int32_t lanes_gate_up;  /* GEMV: lanes per w13 row, 1/2/4/8/16 dividing H/32        */
  int32_t lanes_down;     /* GEMV: lanes per w2 row, 1/2/4/8/16 dividing I/32         */
  int32_t rows_per_pass;  /* GEMV: A rows of an expert per weight pass, 1/2/4/8
                             (the down stage takes at most 4)                         */
  int32_t cost_split;     /* GEMV: 1 share work out by cost (rows per expert), 0 evenly */
  int32_t router_gemv;    /* gate projection: 1 GEMV, 0 matrix cores                  */
  int32_t shared_mfma;    /* GEMV with a shared expert: 1 its rows on the matrix cores
                             in extra workgroups of the same launches (T <= 32, with
                             T x H and 2 T x I fp16 A rows and their K-split partial
                             sums in one workgroup's LDS: T <= 22 at H = 2560),
                             0 in the GEMV with the routed experts                    */
  int32_t combine_in_down; /* layer and block calls with the GEMV, up to 2 tokens: 1
                             the down launch also writes out (each workgroup takes
                             one block of output rows of every active expert and
                             combines it; needs shared_mfma = 0, I/32/lanes_down
                             <= 8 and every act row's fragments in LDS), 0 a
                             separate combine launch; the output is the same bit
                             for bit                                                  */
  int32_t one_launch;     /* GEMV with routing in gate/up, no shared expert, even split
                             (cost_split = 0), combine_in_down = 0: 1 gate/up and down
                             in one persistent launch (one workgroup per compute unit;
                             a workgroup's down share waits, bounded, for the gate/up
                             units of its experts, on per-device completion counts),
                             0 two launches; the output is the same bit for bit.
                             Calls with it that overlap in time on one device share
                             those counts and must not be issued                      */
} moe_plan;

/*
 * moe_plan_default - the plan every entry point uses for these sizes (pure
 * host function; `plan` is a HOST pointer).  top_k and E count the routed
 * experts; shared = 1 for a layer with a shared expert (one more slot per
 * token, one more expert, which holds all T rows).  MOE_ERR_INVALID_ARG /
 * UNSUPPORTED for sizes the layer rejects.
 */
int moe_plan_default(int64_t T, int32_t top_k, int32_t E, int32_t shared, int32_t H,
                     int32_t I, moe_plan* plan);

/*
 * moe_layer_forward_plan / moe_block_forward_plan - moe_layer_forward and
 * moe_block_forward with an explicit plan (HOST pointer; NULL = the default).
 * Every plan computes the same sums and the same routing; the order of the
 * fp32 additions inside the FFN differs between GEMV and MFMA and with the
 * lanes per row, so outputs may differ in the last bits.  Limits of a plan:
 * GEMV and
 * routing in gate/up or in one launch need T <= 64; routing in gate/up needs
 * the GEMV and E (with the shared expert) <= 1024, and so does the one-launch
 * router; the projection GEMV needs T <= 16.
 * MOE_ERR_INVALID_ARG for a malformed plan, MOE_ERR_UNSUPPORTED for one these
 * sizes do not allow; nothing is enqueued then.
 */
int moe_layer_forward_plan(const float* logits, const uint16_t* x, int64_t T,
                           int32_t E, int32_t top_k, const int32_t* w13_qweight,
                           const uint16_t* w13_scales, const int32_t* w13_qzeros,
                           const int32_t* w2_qweight, const uint16_t* w2_scales,
                           const int32_t* w2_qzeros, int32_t H, int32_t I,
                           int32_t group_size, uint16_t* out, void* workspace,
                           size_t workspace_bytes, const moe_plan* plan,
                           void* stream);
int moe_block_forward_plan(const uint16_t* x, int64_t T, const uint16_t* gate_weight,
                           int32_t E, int32_t top_k, int32_t shared,
                           const int32_t* w13_qweight, const uint16_t* w13_scales,
                           const int32_t* w13_qzeros, const int32_t* w2_qweight,
                           const uint16_t* w2_scales, const int32_t* w2_qzeros,
                           int32_t H, int32_t I, int32_t group_size, float* logits,
                           uint16_t* out, void* workspace, size_t workspace_bytes,
                           const moe_plan* plan, void* stream);

/* Scratch bytes of moe_layer_forward_noalloc (per device). */
#define MOE_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * moe_layer_forward_noalloc - moe_layer_forward for callers that cannot
 * allocate device memory or pass a workspace (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation): the same layer on
 * the same kernels, with the workspace taken from a scratch array that the
 * library holds on every device it runs on (MOE_NOALLOC_SCRATCH_BYTES, from
 * module load to process end).  out is what moe_layer_forward returns, bit
 * for bit.  The call allocates nothing (no hipMalloc/hipFree, no allocating
 * library routine); on its first call on a device it looks up that device's
 * scratch address once.
 *
 *   arguments   as moe_layer_forward, without workspace / workspace_bytes
 *
 * Errors as moe_layer_forward; MOE_ERR_WORKSPACE when moe_layer_workspace_bytes
 * for these sizes exceeds MOE_NOALLOC_SCRATCH_BYTES (at the 512-expert,
 * top-10, H 2560, I 640 geometry that is above about 240 tokens), and
 * MOE_ERR_HIP when the scratch address cannot be looked up; nothing is
 * enqueued then.  Every call on one device shares that device's scratch:
 * calls that overlap in time on one device (other streams, other threads)
 * race and must not be issued.  The scratch keeps the last call's contents;
 * a call reads nothing from it that it did not write itself.
 */
int moe_layer_forward_noalloc(const float* logits, const uint16_t* x, int64_t T,
                              int32_t E, int32_t top_k,
                              const int32_t* w13_qweight,
                              const uint16_t* w13_scales,
                              const int32_t* w13_qzeros,
                              const int32_t* w2_qweight,
                              const uint16_t* w2_scales,
                              const int32_t* w2_qzeros, int32_t H, int32_t I,
                              int32_t group_size, uint16_t* out, void* stream);

/* ------------------------------------------------------------------------- *
 * MXFP4: microscaled 4-bit floating point, its products and the layer on it
 *
 * Layout of a matrix of R rows and K columns (K a multiple of 32, <= 65536):
 *   codes   int32 [R, K/8]   E2M1 codes; nibble j of word w is column 8w+j:
 *                            sign, 2 exponent bits (bias 1), 1 mantissa bit:
 *                            0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives
 *   scales  uint8 [R, B]     B = moe_mxfp4_scale_bytes(K) = 4 ceil(K / 128);
 *                            byte b is the E8M0 scale 2^(byte - 127) of
 *                            columns [32b, 32b + 32), 255 stands for NaN;
 *                            bytes from K/32 on are padding, written as 127
 *                            and ignored when read
 * Expert weights are [E, N, ...] of such matrices, N the output columns.
 *
 * Typed tensors: a dtype code says fp32, fp16 or bf16, a stride is the
 * distance of two rows in elements (>= the columns, <= 2^31); rows are
 * contiguous, and such a tensor's pointer needs its element's alignment only.
 * Functions below do not change the ABI version: they are found by name.
 * ------------------------------------------------------------------------- */
#define MOE_F32 0
#define MOE_F16 1
#define MOE_BF16 2

/* Bytes of one row's scales (0: K is not a valid length).  Host only. */
int moe_mxfp4_scale_bytes(int32_t K);

/*
 * moe_mxfp4_quantize - rows to MXFP4.  Per block of 32 columns, with m the
 * largest magnitude: e = clamp(floor(log2 m) - 2, -127, 127), scale byte
 * e + 127, codes the nearest E2M1 values of x 2^-e, ties to even, at most 6 in
 * size.  A zero block has scale byte 0.  A block that holds an infinity or a
 * NaN has scale byte 255 and zero codes: it reads back as NaN.
 * moe_mxfp4_dequantize - the values they stand for, rounded once to dtype.
 *
 *   x       in/out  dtype [rows, K], stride x_stride
 *   codes   out/in  int32 [rows, K/8]
 *   scales  out/in  uint8 [rows, moe_mxfp4_scale_bytes(K)]
 *
 * rows == 0 is valid (nothing is done); rows < 2^31.
 */
int moe_mxfp4_quantize(const void* x, int32_t dtype, int64_t rows, int32_t K,
                       int64_t x_stride, int32_t* codes, uint8_t* scales,
                       void* stream);
int moe_mxfp4_dequantize(const int32_t* codes, const uint8_t* scales,
                         int64_t rows, int32_t K, void* x, int32_t dtype,
                         int64_t x_stride, void* stream);

/*
 * moe_mxfp4_grouped_gemm - rows times their expert's weights, both MXFP4:
 *   out[r, n] = sum_k A[a(r), k] * W[e, n, k]
 *                                for expert_offsets[e] <= r < expert_offsets[e+1]
 * Products are exact, summed in fp32, rounded once to out_dtype.  a(r) = r, or
 * row_slots[r] / top_k when row_slots is given (moe_permute's sorted_slots:
 * the rows of the tokens, without a copy in expert order); the row of a slot
 * outside [0, a_rows * top_k) is zeros, whatever the weights hold.  Rows
 * outside [expert_offsets[0], expert_offsets[E]) are left as they were.  A NaN
 * scale makes every sum that it enters NaN.
 *
 *   a_codes, a_scales  in   MXFP4 [a_rows, K]
 *   row_slots          in   int32 [rows], or NULL (then rows <= a_rows)
 *   expert_offsets     in   int32 [E + 1], ascending, or NULL with E == 1:
 *                           every row belongs to the one expert
 *   w_codes, w_scales  in   MXFP4 [E, N, K]
 *   out                out  out_dtype [rows, N], stride out_stride
 *
 * Limits: 1 <= E <= 4096; 1 <= N <= 65536; N * K < 2^32; rows <= 2^27 and
 * (rows / 16 + min(E, rows)) * ceil(N / 64) < 2^24.
 */
int moe_mxfp4_grouped_gemm(const int32_t* a_codes, const uint8_t* a_scales,
                           int64_t a_rows, const int32_t* row_slots,
                           int32_t top_k, int64_t rows,
                           const int32_t* expert_offsets, int32_t E,
                           const int32_t* w_codes, const uint8_t* w_scales,
                           int32_t N, int32_t K, void* out, int32_t out_dtype,
                           int64_t out_stride, void* stream);

/*
 * moe_mxfp4_gate_up - the gate/up half of an expert FFN on MXFP4 weights:
 *   h = A[a(r), :] . W13[e]^T (2I values, fp32), a = SiLU(h[0:I]) * h[I:2I],
 * and a, as moe_mxfp4_quantize turns fp32 rows of I columns to MXFP4, is
 * stored: the operand of the down product (moe_mxfp4_grouped_gemm with
 * N = H, K = I).  Arguments and rows as there, with K = H and N = 2I.
 *
 *   act_codes   out  int32 [rows, I/8]
 *   act_scales  out  uint8 [rows, moe_mxfp4_scale_bytes(I)]
 *
 * Limits: as there; I a multiple of 32, <= 32768.
 */
int moe_mxfp4_gate_up(const int32_t* a_codes, const uint8_t* a_scales,
                      int64_t a_rows, const int32_t* row_slots, int32_t top_k,
                      int64_t rows, const int32_t* expert_offsets, int32_t E,
                      const int32_t* w13_codes, const uint8_t* w13_scales,
                      int32_t I, int32_t H, int32_t* act_codes,
                      uint8_t* act_scales, void* stream);

/* Workspace bytes moe_mxfp4_layer_forward needs (0: invalid sizes). */
size_t moe_mxfp4_layer_workspace_bytes(int64_t T, int32_t top_k, int32_t E,
                                       int32_t H, int32_t I);

/*
 * moe_mxfp4_layer_forward - moe_layer_forward on MXFP4 experts, activations
 * quantised too: moe_route_permute, moe_mxfp4_quantize of x, moe_mxfp4_gate_up
 * over its sorted_slots, moe_mxfp4_grouped_gemm into fp32 rows and
 * moe_combine_masked, in one call.  out is what those calls produce up to the
 * order of the products' fp32 sums.  Up to 6 tokens, 64 slots, 1024 experts
 * and H = 16384 two launches of the layer's own do all of it.  Otherwise the
 * calls' kernels run, with two differences: each token is quantised once and
 * stored straight to its rows in expert order, which gate/up then reads in
 * order, and past 64 tokens the permutation is moe_permute_masked's.
 *
 *   logits      in   fp32 [T, E]
 *   x, out      in, out  dtype [T, H], dense; out may be x
 *   w13_*       in   MXFP4 [E, 2I, H], rows [0, I) gate, [I, 2I) up
 *   w2_*        in   MXFP4 [E, H, I]
 *   workspace   scratch, device, >= moe_mxfp4_layer_workspace_bytes(...);
 *               contents on entry are ignored.  Two calls that overlap in time
 *               must not share it.
 *
 * Errors as the calls it stands for; nothing is enqueued on an error that the
 * arguments show.
 */
int moe_mxfp4_layer_forward(const float* logits, const void* x, int32_t dtype,
                            int64_t T, int32_t E, int32_t top_k,
                            const int32_t* w13_codes, const uint8_t* w13_scales,
                            const int32_t* w2_codes, const uint8_t* w2_scales,
                            int32_t H, int32_t I, void* out, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------- *
 * Token rows to expert order and back, with slots left out, and gradients
 * ------------------------------------------------------------------------- */

/* Workspace bytes moe_permute_masked needs (0 up to 1024 slots). */
size_t moe_permute_masked_workspace_bytes(int64_t T, int32_t top_k, int32_t E);

/*
 * moe_permute_masked - moe_permute for ids that may leave slots out: a slot
 * counts when first_expert <= id < first_expert + E, as expert id -
 * first_expert; any other id (padding tokens: -1; experts held elsewhere)
 * drops it.  A token may name an expert more than once.  With R slots kept:
 *
 *   expert_offsets  out  int32 [E + 1]   offsets[0] = 0, offsets[E] = R
 *   sorted_slots    out  int32 [S]       slot held by row r < R, by expert, then
 *                                        ascending; -1 from R on
 *   slot_rows       out  int32 [S]       row of slot s, -1 for a dropped one
 *   active_experts, num_active           as moe_permute
 *   workspace       scratch, device, >= moe_permute_masked_workspace_bytes(...)
 *
 * Limits: 1 <= E <= 4096; 1 <= top_k <= 64; S < 2^31; first_expert >= 0.
 */
int moe_permute_masked(const int32_t* topk_ids, int64_t T, int32_t top_k,
                       int32_t first_expert, int32_t E, int32_t* expert_offsets,
                       int32_t* sorted_slots, int32_t* slot_rows,
                       int32_t* active_experts, int32_t* num_active,
                       void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_dispatch - token rows to expert order: x_sorted[slot_rows[s], :] =
 * x[s / top_k, :] for every slot s whose row is in [0, rows); rows that no
 * slot points at are left as they were.  Rows of distinct slots are distinct
 * (moe_permute, moe_permute_masked).
 * moe_dispatch_backward - its gradient: grad_x[t, :] = sum_j
 * grad_sorted[slot_rows[t * top_k + j], :], j ascending, in fp32, rounded
 * once; a token without a slot gets zeros.  Rows that no slot points at are
 * not read.
 *
 *   x, grad_x              dtype [T, H], stride x_stride
 *   x_sorted, grad_sorted  dtype [rows, H], stride sorted_stride
 *   slot_rows              in  int32 [T * top_k]
 *
 * Limits: 1 <= H <= 65536 (any H); 1 <= top_k <= 64; T * top_k, rows < 2^31.
 */
int moe_dispatch(const void* x, int32_t dtype, int64_t T, int32_t top_k,
                 int32_t H, int64_t x_stride, const int32_t* slot_rows,
                 int64_t rows, void* x_sorted, int64_t sorted_stride,
                 void* stream);
int moe_dispatch_backward(const void* grad_sorted, int32_t dtype, int64_t T,
                          int32_t top_k, int32_t H, int64_t sorted_stride,
                          const int32_t* slot_rows, int64_t rows, void* grad_x,
                          int64_t x_stride, void* stream);

/*
 * moe_combine_masked - moe_combine for typed rows and slots left out:
 *   out[t, :] = sum_j topk_weights[t, j] * y_sorted[slot_rows[t * top_k + j], :]
 * over the slots whose row is in [0, rows), j ascending, in fp32, rounded
 * once; a token without one gets zeros, and a dropped slot's weight and row
 * are not used, whatever they hold.
 * moe_combine_backward - its gradients:
 *   grad_y[slot_rows[s], :] = topk_weights[s] * grad_out[s / top_k, :]
 *   grad_weights[s] = sum_h grad_out[s / top_k, h] * y_sorted[slot_rows[s], h]
 * with 0 for a dropped slot; rows of grad_y that no slot points at are left
 * as they were.  As for moe_dispatch, rows of distinct slots are distinct (a
 * row that two slots hold would keep one slot's gradient, not their sum).
 * grad_y must not overlap y_sorted or grad_out.
 *
 *   y_sorted      in   y_dtype [rows, H], stride y_stride
 *   topk_weights  in   fp32 [T, top_k]
 *   slot_rows     in   int32 [T * top_k]
 *   out           out  out_dtype [T, H], stride out_stride
 *   grad_out      in   grad_dtype [T, H], stride grad_stride
 *   grad_y        out  y_dtype [rows, H], stride grad_y_stride
 *   grad_weights  out  fp32 [T, top_k]
 *
 * Limits as moe_dispatch.
 */
int moe_combine_masked(const void* y_sorted, int32_t y_dtype, int64_t T,
                       int32_t top_k, int32_t H, int64_t y_stride,
                       const float* topk_weights, const int32_t* slot_rows,
                       int64_t rows, void* out, int32_t out_dtype,
                       int64_t out_stride, void* stream);
int moe_combine_backward(const void* grad_out, int32_t grad_dtype,
                         int64_t grad_stride, const void* y_sorted,
                         int32_t y_dtype, int64_t y_stride,
                         const float* topk_weights, const int32_t* slot_rows,
                         int64_t T, int32_t top_k, int32_t H, int64_t rows,
                         void* grad_y, int64_t grad_y_stride,
                         float* grad_weights, void* stream);

/* ------------------------------------------------------------------------- *
 * Training the experts: products of rows grouped by expert in 16 bits with
 * their gradients, the activation between them, the router's gradient, and
 * the step that updates the weights.  Typed tensors and dtype codes as above;
 * gradients are calls of their own.
 * ------------------------------------------------------------------------- */

/*
 * moe_grouped_gemm - rows times their expert's weights:
 *   out[r, n] = sum_k a[r, k] * w[e, n, k]
 *                               for expert_offsets[e] <= r < expert_offsets[e+1]
 * moe_grouped_gemm_backward - the gradient of the rows:
 *   grad_a[r, k] = sum_n grad[r, n] * w[e, n, k]
 * moe_grouped_gemm_backward_weights - the gradient of the weights:
 *   grad_w[e, n, k] = sum_r grad[r, n] * a[r, k]   over the rows r of expert e,
 * zeros for an expert without rows; accumulate == 1 adds the sums to what
 * grad_w holds.  Products are exact, summed in fp32 (with what grad_w holds,
 * too), rounded once to out_dtype.  Rows outside [expert_offsets[0],
 * expert_offsets[E]) are not read, and those of out and grad_a left as they
 * were.  Which kernel runs, and with it the order of a sum, goes by the sizes:
 * a repeated call gives identical bits, another number of rows may differ in
 * the last ones.
 *
 *   a               in   dtype [rows, K], stride a_stride; dtype fp16 or bf16
 *   grad            in   dtype [rows, N], stride grad_stride
 *   expert_offsets  in   int32 [E + 1], ascending, or NULL with E == 1: every
 *                        row belongs to the one expert
 *   w               in   dtype [E, N, K], dense
 *   out             out  out_dtype [rows, N], stride out_stride
 *   grad_a          out  out_dtype [rows, K], stride grad_a_stride
 *   grad_w          out  out_dtype [E, N, K], dense (accumulate: in and out)
 *   workspace       scratch, device, >= moe_grouped_gemm_backward_weights_
 *                   workspace_bytes(...) bytes (may be NULL when that is 0);
 *                   contents on entry are ignored.  Two calls that overlap in
 *                   time must not share it.
 *
 * Any N, K and strides; where N, K, the strides and the addresses of a and grad
 * are multiples of 8 elements the calls are 1.5 to 2 times as fast.  An output
 * must not overlap an input.  rows == 0 is valid;
 * moe_grouped_gemm_backward_weights then still writes grad_w.
 *
 * Limits: fp32 operands are MOE_ERR_UNSUPPORTED; 1 <= E <= 4096; 1 <= N, K <=
 * 65536; N * K < 2^30; rows <= 2^27 and (rows / 16 + min(E, rows)) *
 * ceil(max(N, K) / 64) < 2^24.
 */
int moe_grouped_gemm(const void* a, int32_t dtype, int64_t rows,
                     int64_t a_stride, const int32_t* expert_offsets, int32_t E,
                     const void* w, int32_t N, int32_t K, void* out,
                     int32_t out_dtype, int64_t out_stride, void* stream);
int moe_grouped_gemm_backward(const void* grad, int32_t dtype, int64_t rows,
                              int64_t grad_stride,
                              const int32_t* expert_offsets, int32_t E,
                              const void* w, int32_t N, int32_t K,
                              void* grad_a, int32_t out_dtype,
                              int64_t grad_a_stride, void* stream);
size_t moe_grouped_gemm_backward_weights_workspace_bytes(int64_t rows,
                                                         int32_t E, int32_t N,
                                                         int32_t K);
int moe_grouped_gemm_backward_weights(
    const void* grad, int32_t dtype, int64_t rows, int64_t grad_stride,
    const void* a, int64_t a_stride, const int32_t* expert_offsets, int32_t E,
    int32_t N, int32_t K, void* grad_w, int32_t out_dtype, int32_t accumulate,
    void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_silu_mul - the activation between an expert's two products:
 *   act[r, i] = SiLU(h[r, i]) * h[r, I + i],   SiLU(v) = v s, s = 1 / (1 + e^-v)
 * (the gate's columns first, as w13's rows).
 * moe_silu_mul_backward - its gradient:
 *   grad_h[r, i]     = grad_act[r, i] * up * s (1 + gate (1 - s))
 *   grad_h[r, I + i] = grad_act[r, i] * gate * s
 * In fp32, rounded once.  With expert_offsets, rows outside [expert_offsets[0],
 * expert_offsets[E]) are not read and left as they were.  grad_h may be h
 * itself (same address and stride); otherwise outputs must not overlap inputs.
 *
 *   h, grad_h       dtype [rows, 2I], strides h_stride, grad_h_stride
 *   act, grad_act   dtype [rows, I], strides act_stride, grad_stride
 *   expert_offsets  in  int32 [E + 1], or NULL: all rows (E is not read)
 *
 * Limits: 1 <= I <= 32768 (any I); rows < 2^31; rows * ceil(I / 8) < 2^32 - 256.
 */
int moe_silu_mul(const void* h, int32_t dtype, int64_t rows, int32_t I,
                 int64_t h_stride, const int32_t* expert_offsets, int32_t E,
                 void* act, int64_t act_stride, void* stream);
int moe_silu_mul_backward(const void* grad_act, int64_t grad_stride,
                          const void* h, int64_t h_stride, int32_t dtype,
                          int64_t rows, int32_t I,
                          const int32_t* expert_offsets, int32_t E,
                          void* grad_h, int64_t grad_h_stride, void* stream);

/*
 * moe_route_backward - moe_route's gradient: with w = topk_weights and g =
 * grad_weights (moe_combine_backward's),
 *   grad_logits[t, id_j] = w[t, j] * (g[t, j] - sum_i w[t, i] g[t, i])
 * and 0 for every expert that the token did not choose.  A choice outside
 * [0, E) has no logit and is not written; its weight counts in the sum.  An
 * expert chosen twice gets the sum of both.
 *
 *   topk_ids      in   int32 [T, top_k]
 *   topk_weights  in   fp32 [T, top_k]
 *   grad_weights  in   fp32 [T, top_k]
 *   grad_logits   out  out_dtype [T, E]; must not overlap an input
 *
 * Limits: 1 <= E <= 4096; 1 <= top_k <= 64; T <= 2^26 - 4; T * top_k < 2^31.
 */
int moe_route_backward(const int32_t* topk_ids, const float* topk_weights,
                       const float* grad_weights, int64_t T, int32_t E,
                       int32_t top_k, void* grad_logits, int32_t out_dtype,
                       void* stream);

/*
 * moe_adamw - one AdamW step over `count` tensors at once:
 *   g = grad * grad_scale[0]
 *   m = beta1 m + (1 - beta1) g;   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) * m / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32, beta and 1 - beta each rounded to it; p is rounded once to its type
 * (and once to copy's), and is updated from m and v before these are rounded to
 * their states.  With eps 0 an element whose v is 0 divides by 0.  A positive eps
 * may be as small as it likes (fp32 holds it as 2^-149 at least): an element
 * whose m and v are 0 then moves by its weight decay alone.
 *
 * States of 8 bits: elements in blocks of MOE_ADAMW_BLOCK (the last may be
 * short), per block one fp32 scale = largest magnitude / 1.875.  A code's
 * value is scale times a small float: m sign, 4 exponent bits (bias 15), 3
 * mantissa bits; v, which is not negative, 5 exponent bits (bias 31) and 3; an
 * exponent of 0 is subnormal.  Zero codes and scales are zero moments.  Codes
 * are rounded up with the probability of the part cut off, by 20 bits of noise
 * that are a function of the element's number and `seed`; pass another seed at
 * every step (the step's number will do), and another one per call where one
 * step takes several.  v > 0 is never rounded to 0.  A block whose largest
 * magnitude is under 2.2e-38 becomes zeros; one that holds an infinity or a
 * NaN does not stay finite.
 *
 *   tensors     in   HOST array of `count` descriptions, read during the call:
 *     n                elements (0: skipped)
 *     param            in, out  param_dtype [n]
 *     grad             in       grad_dtype [n]
 *     m, v             in, out  fp32 [n], or uint8 codes [n]
 *     m_scales,        in, out  fp32 [ceil(n / MOE_ADAMW_BLOCK)] with 8 bits;
 *     v_scales                  not read with 32
 *     copy             out      copy_dtype [n], the new param once more (16-bit
 *                               weights beside fp32 ones), or NULL
 *   state_bits  8 or 32, of every tensor of the call
 *   grad_scale  in   fp32 [1] on the device, or NULL: 1 (clipping and loss
 *                    scales without a synchronisation)
 *
 * A buffer that the call writes must not overlap another of the call; gradients
 * may share theirs among them.  The scalars are the call's: a captured graph
 * repeats its step number, rate and seed when it is replayed.
 *
 * MOE_ERR_INVALID_ARG for state_bits, betas outside [0, 1), negative or
 * non-finite lr, eps or weight_decay, lr weight_decay or lr / (1 - beta1^step)
 * past fp32's range, step < 1, buffers that overlap.  Limits: n <= 2^33.
 */
#define MOE_ADAMW_BLOCK 128
typedef struct moe_adamw_tensor {
  int64_t n;
  void* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scales;
  float* v_scales;
  void* copy;
  int32_t param_dtype;
  int32_t grad_dtype;
  int32_t copy_dtype;
  int32_t reserved; /* 0 */
} moe_adamw_tensor;
int moe_adamw(const moe_adamw_tensor* tensors, int32_t count,
              int32_t state_bits, double lr, double beta1, double beta2,
              double eps, double weight_decay, int64_t step, uint32_t seed,
              const float* grad_scale, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_W4A16_H_ */
