/*
 * moe.h -- C ABI of libmoe.so, the single-GPU MoE-layer hot path for AMD
 * Instinct MI355X (gfx950):
 *
 *   moe_route -> moe_layout -> moe_permute -> moe_grouped_swiglu -> moe_combine
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every pointer argument named *_d is DEVICE memory on the current HIP
 *   device; descriptors (moe_layout_desc) are HOST memory. The caller owns
 *   and allocates every buffer; the library allocates nothing, keeps no state
 *   between calls and never blocks the host (moe_validate_layout excepted).
 *   The one exception to the ownership rule is moe_layout_noalloc, whose
 *   workspace is a static device array of the library (one per GPU). The
 *   weight-gradient calls also use small library-held device counters, one
 *   pair per stream, which each call leaves at zero.
 * - `stream` is a hipStream_t (NULL = the default stream). Each call only
 *   enqueues kernels on it and returns; results are ready when the stream
 *   reaches that point. Calls on different streams may run concurrently as
 *   long as they do not share output buffers.
 * - bf16 buffers hold IEEE bfloat16 bit patterns (uint16); float is fp32;
 *   indices are int32. Matrices are row-major and densely packed.
 * - Return value: a moe_status. Argument checks run on the host before any
 *   launch: a call that returns anything but MOE_OK has enqueued nothing.
 *   MOE_ERR_HIP reports a failed launch (hipGetLastError after the launch).
 * - Data errors (an expert id out of [0, E), a row index past the end of a
 *   buffer) are not diagnosed on the fast path; the kernels skip such
 *   entries so every access stays in bounds. moe_validate_layout reports them.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moe_status {
  MOE_OK = 0,
  MOE_ERR_ARG = 1,          /* null pointer, size out of range, misaligned buffer,
                               workspace or m_cap too small */
  MOE_ERR_UNSUPPORTED = 2,  /* a shape the kernels do not implement (see each call) */
  MOE_ERR_HIP = 3,          /* a HIP runtime call or kernel launch failed */
  MOE_ERR_COVERAGE = 4,     /* validator: a (token, slot) is missing or covered twice */
  MOE_ERR_EXPERT_ID = 5,    /* validator: expert id out of range or repeated in a token */
  MOE_ERR_LAYOUT = 6,       /* validator: offsets / src_row / dst_row inconsistent */
  MOE_ERR_TOO_LARGE = 7     /* moe_layout_noalloc: the layout needs more scratch than the
                               library's static array holds */
} moe_status;

/* Types of row buffers, for the calls that take more than bf16. */
enum { MOE_ROWS_BF16 = 0, MOE_ROWS_F16 = 1, MOE_ROWS_F32 = 2 };

/* Static name of a status code ("MOE_OK", ...); never NULL. */
const char* moe_status_string(int32_t status);

/* ABI version of this header; bumped on any incompatible change. */
int32_t moe_abi_version(void);

/*
 * moe_route -- token-choice top-k routing.
 *
 * Follows the token-choice top-k router of the AutoEP runtime (DeepSpeed
 * AutoEP commit text, section "Attribution": ep_router.py after TorchTitan's
 * TokenChoiceTopKRouter; section "Design", runtime step 2), with distinct
 * experts per token (DeepSpeed PR #8847, section "Benchmark") and FP32
 * routing weights kept in the router dtype (same page, section "Change").
 * Per token t: the k experts with the largest logits[t, :], in descending
 * order, ties to the lower expert id (-0.0 equals +0.0); weights are the
 * softmax over all E experts renormalised over the k selected, computed as
 * exp(l_j - l_max) / sum_selected exp(l_i - l_max) in fp32.
 *
 *   logits_d    [T, E] float, finite values
 *   topk_idx_d  [T, k] int32 (out)
 *   topk_w_d    [T, k] float (out)
 * Limits: T >= 0, 1 <= E <= 1024, 1 <= k <= min(E, 16). T = 0 is a no-op.
 */
int32_t moe_route(const float* logits_d, int64_t num_tokens, int32_t num_experts,
                  int32_t top_k, int32_t* topk_idx_d, float* topk_w_d, void* stream);

/*
 * moe_route_scored -- routing by scores, with a selection bias, groups of
 * experts and a choice of normalisation. Per token:
 *
 *   s_e = sigmoid(l_e), or softmax(l)_e over all E experts
 *   v_e = s_e + bias[e]          (bias NULL: v = s; the bias steers the choice, not the weights)
 *   experts [g*E/G, (g+1)*E/G) form group g of G = num_groups; a group's rank is its largest
 *   v (MOE_GROUP_MAX) or the sum of its two largest (MOE_GROUP_TOP2; a group of one expert:
 *   its v); the top_groups groups of the highest rank stay
 *   the k experts of those groups with the largest v, in descending order
 *   w_j = scale * s_j, or with renormalise scale * s_j / (sum of s over the k selected)
 *
 * ties to the lower index. The choice is the one that fp64 scores, values and
 * ranks give: it does not depend on how an fp32 exponential rounds. The weights
 * are formed in fp64 and rounded once (softmax without renormalise: over a sum of fp32 terms). A NaN logit counts as
 * -inf, +inf as the largest finite fp32; an expert at -inf has score 0 and stays selectable. v = NaN (from the bias)
 * counts as -inf. Renormalised weights whose sum is 0 are all 0.
 *
 *   logits_d    [T, E] float
 *   bias_d      [E] float, or NULL
 *   topk_idx_d  [T, k] int32 (out);  topk_w_d [T, k] float (out)
 * Limits: 0 <= T < 2^26, 1 <= E <= 1024, 1 <= num_groups <= 64 dividing E,
 * 1 <= top_groups <= num_groups, 1 <= k <= min(16, top_groups * E / num_groups),
 * finite scale. T = 0 is a no-op.
 */
enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 };

typedef struct moe_route_desc {
  int64_t num_tokens;  /* T */
  int32_t num_experts; /* E */
  int32_t top_k;       /* k */
  int32_t score;       /* MOE_SCORE_* */
  int32_t num_groups;  /* 1: no groups */
  int32_t top_groups;
  int32_t group_rank;  /* MOE_GROUP_*; no effect when every group stays */
  int32_t renormalise; /* 0 or 1 */
  float scale;
} moe_route_desc;

int32_t moe_route_scored(const moe_route_desc* desc, const float* logits_d, const float* bias_d,
                         int32_t* topk_idx_d, float* topk_w_d, void* stream);

/*
 * moe_route_scored_backward -- the gradient of moe_route_scored's weights
 * with respect to the logits, the choice held fixed (the bias has none), from
 * g = grad_w[t, :]. desc as in the forward, within its limits; the groups change nothing.
 *
 *   sigmoid:              dl_j = scale * g_j s_j (1 - s_j)
 *   sigmoid, renormalise: dl_j = scale * (g_j - sum_i g_i s_i / S) / S * s_j (1 - s_j), S = sum_i s_i
 *   softmax:              dl_e = scale * s_e (g_e - sum_i g_i s_i), every e; g_e = 0 unselected
 *   softmax, renormalise: dl_j = scale * q_j (g_j - sum_i g_i q_i), q the renormalised weights / scale
 *
 * and 0 for the experts a formula does not name. A slot whose id is outside
 * [0, E) is skipped; a repeated id takes the sum of its slots.
 *   logits_d [T, E];  topk_idx_d, grad_w_d [T, k];  grad_logits_d [T, E] float (out)
 */
int32_t moe_route_scored_backward(const moe_route_desc* desc, const float* logits_d,
                                  const int32_t* topk_idx_d, const float* grad_w_d,
                                  float* grad_logits_d, void* stream);

/*
 * Layout of one GPU's share when `ep_size` virtual ranks split the work:
 * source rank s owns tokens [s*T/ep, (s+1)*T/ep); destination rank d owns
 * experts [d*E/ep, (d+1)*E/ep); this GPU is destination `local_rank`
 * (-1: every expert is local, E_loc = E; otherwise E_loc = E/ep).
 */
typedef struct moe_layout_desc {
  int64_t num_tokens;  /* T, a multiple of ep_size */
  int32_t num_experts; /* E, a multiple of ep_size, <= 1024 */
  int32_t top_k;       /* k, 1..min(E, 16) */
  int32_t ep_size;     /* >= 1, <= 64 */
  int32_t local_rank;  /* -1 or 0..ep_size-1 */
  int32_t align;       /* row alignment of each local expert's group, power of two <= 1024 */
} moe_layout_desc;

/* Worst-case local rows: T*min(k, E_loc) + E_loc*(align-1). Returns -1 for
 * an invalid descriptor. Size src_row_d, x_perm, h and y with it. */
int64_t moe_layout_m_cap(const moe_layout_desc* desc);

/* Bytes of device workspace moe_layout needs (0 for an invalid descriptor). */
size_t moe_layout_workspace_bytes(const moe_layout_desc* desc);

/*
 * moe_layout -- dispatch layout from topk_idx, with no host sync.
 *
 * The layout is computed from topk_idx and the expert count before any data
 * moves (DeepEP issue #272, the maintainer's dispatch example:
 * get_dispatch_layout, then dispatch), its histogram must not force a host
 * sync (xtuner PR #2056, review comments: histc kept over bincount), and the
 * split plan comes from the per-expert count matrix alone, its row sums being
 * the splits (DeepSpeed PR #8190 "Derive AutoEP rank splits from the
 * per-expert count exchange", sections "Redundancy" and "Fix"). Rows are
 * grouped by local expert and each group is padded to `align` for the
 * grouped GEMM (DeepSpeed AutoEP commit text, section "Attribution": token
 * group alignment / padding helpers). Rows are named by the flat index
 * token*top_k + slot (DeepSpeed PR #8847, section "Change").
 *
 * Outputs (all int32, device):
 *   expert_counts_d [E]            assignments per expert (all E)
 *   send_counts_d   [ep, E]        [s, e]: assignments of source s to expert e
 *   split_matrix_d  [ep, ep]       [s, d]: assignments of source s to destination d
 *                                  (row sums: input splits; column local_rank: output splits)
 *   recv_counts_d   [ep, E_loc]    [s, e]: assignments of source s to local expert e
 *   output_splits_d [ep]           recv_counts row sums
 *   offsets_d       [E_loc + 1]    offsets[0] = 0, offsets[e+1] = offsets[e] + ceil(c_e/align)*align
 *   dst_row_d       [T, k]         local row of (t, slot), or -1 if its expert is not local
 *   src_row_d       [m_cap]        flat index t*k+slot held by a row; -1 for padding and
 *                                  for every row from offsets[E_loc] to m_cap
 * Within an expert's group, rows follow ascending flat index (a stable
 * order, independent of thread scheduling).
 *   topk_idx_d      [T, k] int32 expert ids; ids outside [0, E) are skipped.
 *   m_cap           >= moe_layout_m_cap(desc)
 *   workspace_d     >= moe_layout_workspace_bytes(desc) bytes, 16-byte aligned;
 *                   contents on entry do not matter.
 * Any output pointer except offsets_d, dst_row_d and src_row_d may be NULL
 * to skip it.
 */
int32_t moe_layout(const moe_layout_desc* desc, const int32_t* topk_idx_d,
                   int32_t* expert_counts_d, int32_t* send_counts_d,
                   int32_t* split_matrix_d, int32_t* recv_counts_d,
                   int32_t* output_splits_d, int32_t* offsets_d, int32_t* dst_row_d,
                   int32_t* src_row_d, int64_t m_cap, void* workspace_d,
                   size_t workspace_bytes, void* stream);

/*
 * moe_layout_noalloc -- moe_layout for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): no workspace argument, and the call allocates nothing.
 * The workspace lives in a static device array of MOE_LAYOUT_SCRATCH_BYTES
 * (4 MiB) that each GPU the library runs on holds until the process ends;
 * its device address is looked up once per device, on the first call with
 * that device current. Outputs, arguments and results are those of
 * moe_layout (the same kernels), on the current device's stream `stream`.
 * Limit: moe_layout_workspace_bytes(desc) <= MOE_LAYOUT_SCRATCH_BYTES, else
 * MOE_ERR_TOO_LARGE and nothing is launched (the layout's tiles grow with the
 * assignment count, so every layout of up to 2^30 assignments T * top_k fits,
 * and every valid one with at most 512 experts). Every call on one GPU shares that GPU's array:
 * calls that overlap on one GPU (on two streams, or from two host threads
 * without ordering) race and must not be made. Nothing in the array needs to
 * start at zero; a call leaves its contents behind.
 */
#define MOE_LAYOUT_SCRATCH_BYTES (4u << 20)

int32_t moe_layout_noalloc(const moe_layout_desc* desc, const int32_t* topk_idx_d,
                           int32_t* expert_counts_d, int32_t* send_counts_d,
                           int32_t* split_matrix_d, int32_t* recv_counts_d,
                           int32_t* output_splits_d, int32_t* offsets_d, int32_t* dst_row_d,
                           int32_t* src_row_d, int64_t m_cap, void* stream);

/*
 * moe_dispatch_layout -- per-rank deduplicated dispatch layout.
 *
 * The counts and table DeepEP's dispatch consumes, computed from topk_idx
 * and the expert count before any data moves (DeepEP issue #272, the
 * maintainer's example: get_dispatch_layout returns num_tokens_per_rank,
 * num_tokens_per_expert and is_token_in_rank). A token is sent once to each
 * rank that holds at least one of its experts (rank r holds experts
 * [r*E/ep, (r+1)*E/ep)), however many of its slots land there:
 *   is_token_in_rank_d      [T, ep] uint8: 1 if some slot of t maps to rank r
 *   num_tokens_per_rank_d   [ep] int32: column sums of is_token_in_rank
 *   num_tokens_per_expert_d [E] int32: assignments per expert
 *   token_rank_pos_d        [T, ep] int32: position of t among the tokens rank r
 *                           receives, in token order; -1 where t is not sent to r
 * Expert ids outside [0, E) are skipped. No host sync; the result does not
 * depend on scheduling.
 *   workspace_d >= moe_dispatch_layout_workspace_bytes(...) bytes.
 * Limits: 1 <= ep <= 64, E a multiple of ep, E <= 1024, 1 <= k <= min(E, 16),
 * T < 2^25.
 */
size_t moe_dispatch_layout_workspace_bytes(int64_t num_tokens, int32_t num_experts,
                                           int32_t top_k, int32_t ep_size);

int32_t moe_dispatch_layout(const int32_t* topk_idx_d, int64_t num_tokens, int32_t num_experts,
                            int32_t top_k, int32_t ep_size, int32_t* num_tokens_per_rank_d,
                            int32_t* num_tokens_per_expert_d, uint8_t* is_token_in_rank_d,
                            int32_t* token_rank_pos_d, void* workspace_d,
                            size_t workspace_bytes, void* stream);

/*
 * moe_permute -- expert-major token gather (the local part of dispatch).
 *
 * The reorder-by-expert step of the AutoEP flow (DeepSpeed AutoEP commit
 * text, section "Design", runtime step 3) and the local half of DeepEP's
 * dispatch (DeepEP issue #272: x, topk_idx, topk_weights in; rows grouped per
 * expert out). For every (t, slot) with dst_row[t, slot] = r >= 0:
 * x_perm[r, :] = x[t, :], a bit copy (each token row read once); every row r
 * below offsets[E_loc] with src_row[r] < 0 (the alignment padding of the
 * expert groups) is set to zero. Rows from offsets[E_loc] to m_cap are not
 * written.
 *   x_d         [T, H] bf16, 16-byte aligned
 *   dst_row_d   [T, k] int32 (from moe_layout); rows >= m_cap are skipped
 *   src_row_d   [m_cap] int32 (from moe_layout)
 *   offsets_d   [E_loc + 1] int32 (from moe_layout)
 *   x_perm_d    [m_cap, H] bf16 (out), 16-byte aligned
 * Limits: H a multiple of 8, 8 <= H <= 16384; 1 <= k <= 16;
 * 1 <= E_loc <= 1024. T = 0 writes only the padding rows.
 */
int32_t moe_permute(const void* x_d, int64_t num_tokens, int32_t hidden, int32_t top_k,
                    const int32_t* dst_row_d, const int32_t* src_row_d,
                    const int32_t* offsets_d, int32_t num_local_experts, int64_t m_cap,
                    void* x_perm_d, void* stream);

/*
 * moe_permute_weighted -- the permute with the routing score applied before
 * the experts (AutoEP's score_apply="pre", DeepSpeed PR #8847, section
 * "Change", which the fused restore refuses): x_perm[dst_row[t, s], :] =
 * bf16(topk_w[t, s] * x[t, :]), an fp32 product rounded once. The experts
 * then see scaled rows and the restore is a plain sum (moe_combine_rows with
 * no weights). x_d, dst_row_d, x_perm_d and the limits as moe_permute, plus
 * topk_w_d [T, k]; padding rows are not written.
 */
int32_t moe_permute_weighted(const void* x_d, int64_t num_tokens, int32_t hidden, int32_t top_k,
                             const int32_t* dst_row_d, const float* topk_w_d, int64_t m_cap,
                             void* x_perm_d, void* stream);

/*
 * moe_pack_weights -- one-time repack of expert matrices into the packed
 * layout the forward grouped GEMMs read (moe_grouped_gate_up, _gate_up_save,
 * _down, _swiglu). This is the load-time conversion into the grouped expert
 * layout the runtime expects (DeepSpeed AutoEP commit text, section "Design":
 * ep_repack.py), done once per weight set, outside the per-step path; the
 * layout itself is this library's. Expert weights arrive in math orientation
 * w[m, k, n] (gate/up [E, H, I], down [E, I, H]; k the reduction index, n the
 * output index, K = rows, N = cols). The packed matrix is output-major with
 * the N rows cut into blocks of R = 256 rows if N % 256 == 0, else 128, and
 * each block stored as K/64 consecutive [R][64] slices:
 *   wt[m*N*K + (n/R)*K*R + (k/64)*R*64 + (n%R)*64 + k%64] = w[m, k, n]
 * (a bf16 bit copy; wt has the element count of w).
 *   w_d  [num_mats, rows, cols] bf16;  wt_d (out), num_mats * rows * cols bf16
 * rows and cols multiples of 128, else MOE_ERR_UNSUPPORTED; w_d and wt_d
 * distinct (MOE_ERR_ARG otherwise).
 */
int32_t moe_pack_weights(const void* w_d, int64_t num_mats, int32_t rows, int32_t cols,
                         void* wt_d, void* stream);

/*
 * Grouped SwiGLU expert MLPs over ragged expert groups (local grouped expert
 * compute of the AutoEP flow, DeepSpeed AutoEP commit text, sections
 * "Attribution" (ep_experts.py, grouped-GEMM execution) and "Design",
 * runtime step 5; bf16 grouped GEMM as in DeepSpeed PR #8847, section
 * "Tests"). For local expert e the rows [offsets[e], offsets[e] + counts[e])
 * of the input go through expert e:
 *
 *   moe_grouped_gate_up:  h = silu(x_perm W1[e]) * (x_perm W3[e])   (fp32 math, bf16 out)
 *   moe_grouped_down:     y = h W2[e]                               (fp32 accumulate, bf16 out)
 *   moe_grouped_swiglu:   both, in that order, through the caller's h buffer
 *
 * silu(a) = a / (1 + e^-a). Products are bf16 x bf16 on the matrix cores,
 * accumulated in fp32, rounded to bf16 (nearest even) once at the end.
 * Rows outside every [offsets[e], offsets[e] + counts[e]) are neither read
 * nor written.
 *   x_perm_d   [m_cap, H] bf16          h_d [m_cap, I] bf16        y_d [m_cap, H] bf16
 *   offsets_d  [E_loc + 1] int32        counts_d [E_loc] int32 (local expert counts,
 *                                       = expert_counts_d + first local expert)
 *   w1t_d, w3t_d: W1, W3 packed by moe_pack_weights (rows H, cols I), E_loc * I * H bf16
 *   w2t_d: W2 packed by moe_pack_weights (rows I, cols H), E_loc * H * I bf16
 * Limits: H and I multiples of 128; E_loc <= 1024; offsets[E_loc] <= m_cap.
 * All bf16 pointers 16-byte aligned. Unsupported shapes: MOE_ERR_UNSUPPORTED.
 */
int32_t moe_grouped_gate_up(const void* x_perm_d, const int32_t* offsets_d,
                            const int32_t* counts_d, int32_t num_local_experts,
                            int64_t m_cap, int32_t hidden, int32_t inter,
                            const void* w1t_d, const void* w3t_d, void* h_d, void* stream);

/*
 * moe_grouped_gate_up_gather -- moe_grouped_gate_up with the permute fused
 * into its operand loads: the rows of local expert e are read straight from
 * the token rows, row r of the grouped layout being x[src_row[r] / top_k]
 * (the expert-major gather of the dispatch, DeepEP issue #272: rows grouped
 * per expert; DeepSpeed AutoEP commit text, section "Design", runtime steps
 * 3 and 5, reorder then grouped expert compute). h is then bit-identical to
 * moe_permute followed by moe_grouped_gate_up, and the expert-major copy of x
 * is never written.
 *   x_d        [T, H] bf16 token rows, 16-byte aligned
 *   src_row_d  [m_cap] int32, moe_layout's src_row
 *   h_d        [m_cap, I] bf16 (out); other arguments as moe_grouped_gate_up
 * Limits as moe_grouped_gate_up, 1 <= top_k <= 16, and (T + 1) * H * 2 < 2^32
 * (MOE_ERR_UNSUPPORTED otherwise).
 */
int32_t moe_grouped_gate_up_gather(const void* x_d, int64_t num_tokens, int32_t top_k,
                                   const int32_t* src_row_d, const int32_t* offsets_d,
                                   const int32_t* counts_d, int32_t num_local_experts,
                                   int64_t m_cap, int32_t hidden, int32_t inter,
                                   const void* w1t_d, const void* w3t_d, void* h_d,
                                   void* stream);

int32_t moe_grouped_down(const void* h_d, const int32_t* offsets_d, const int32_t* counts_d,
                         int32_t num_local_experts, int64_t m_cap, int32_t inter,
                         int32_t hidden, const void* w2t_d, void* y_d, void* stream);

int32_t moe_grouped_swiglu(const void* x_perm_d, const int32_t* offsets_d,
                           const int32_t* counts_d, int32_t num_local_experts,
                           int64_t m_cap, int32_t hidden, int32_t inter,
                           const void* w1t_d, const void* w3t_d, const void* w2t_d,
                           void* h_d, void* y_d, void* stream);

/*
 * Training: the forward keeps the pre-activations, and the backward of the
 * grouped SwiGLU experts produces the data gradient of x_perm. Training runs
 * the grouped-GEMM path forward and backward and hands the expert gradients
 * back in BF16 (xtuner PR #2056 "Integrate MoonEP dispatcher ...", section
 * "Summary"). With g = x W1[e], u = x W3[e] (fp32 accumulators), for the rows
 * [offsets[e], offsets[e] + counts[e]) of local expert e:
 *
 *   moe_grouped_gate_up_save:     h as moe_grouped_gate_up, and gu = [g | u] rounded to
 *                                 bf16 (the two halves of each gu row)
 *   moe_grouped_down_backward:    dh = dy W2[e]^T (fp32), then with g, u read from gu
 *                                 dgu = [dh u silu'(g) | dh silu(g)] rounded to bf16,
 *                                 silu'(g) = s (1 + g (1 - s)), s = 1 / (1 + e^-g)
 *   moe_grouped_gate_up_backward: dx_perm = dg W1[e]^T + du W3[e]^T (one fp32 sum over
 *                                 the 2I products), rounded to bf16
 *
 *   x_perm_d, dy_d, dx_perm_d [m_cap, H] bf16;  h_d [m_cap, I];  gu_d, dgu_d [m_cap, 2I]
 *   w1t_d, w3t_d: W1, W3 packed by moe_pack_weights (forward only)
 *   w1_d, w3_d [E_loc, H, I], w2_d [E_loc, I, H]: the math-orientation weights, which
 *   are already output-major for the backward products
 * Rows outside the expert groups are neither read nor written. Limits as the
 * forward calls (H and I multiples of 128).
 */
int32_t moe_grouped_gate_up_save(const void* x_perm_d, const int32_t* offsets_d,
                                 const int32_t* counts_d, int32_t num_local_experts,
                                 int64_t m_cap, int32_t hidden, int32_t inter,
                                 const void* w1t_d, const void* w3t_d, void* h_d, void* gu_d,
                                 void* stream);

int32_t moe_grouped_down_backward(const void* dy_d, const void* gu_d, const int32_t* offsets_d,
                                  const int32_t* counts_d, int32_t num_local_experts,
                                  int64_t m_cap, int32_t inter, int32_t hidden,
                                  const void* w2_d, void* dgu_d, void* stream);

int32_t moe_grouped_gate_up_backward(const void* dgu_d, const int32_t* offsets_d,
                                     const int32_t* counts_d, int32_t num_local_experts,
                                     int64_t m_cap, int32_t hidden, int32_t inter,
                                     const void* w1_d, const void* w3_d, void* dx_perm_d,
                                     void* stream);

/*
 * Weight gradients of the grouped experts (BF16 out, fp32 accumulation over
 * the expert's rows; xtuner PR #2056, section "Summary", and its commit
 * "extend grouped GEMM for dynamic expert gradients"):
 *
 *   moe_grouped_gate_up_wgrad:  dW1[e] = x_perm_e^T dg_e,  dW3[e] = x_perm_e^T du_e
 *   moe_grouped_down_wgrad:     dW2[e] = h_e^T dy_e
 *
 * where _e is the expert's rows [offsets[e], offsets[e] + counts[e]) and
 * dgu = [dg | du] is moe_grouped_down_backward's output. An expert without
 * rows gets a zero gradient.
 *   dw1_d, dw3_d [E_loc, H, I] bf16 (out);  dw2_d [E_loc, I, H] bf16 (out)
 *   (the math orientation of the weights)
 * Limits as the forward calls.
 * When the experts' row counts are skewed (a fixed tile order would give some
 * workgroup 1/16 more work than the mean), tiles are handed out at run time
 * from a small counter pair in library-held device memory, one pair per
 * stream (the first 64 streams a GPU sees; later streams keep the fixed
 * order). Each tile is one workgroup's fixed-order sum either way, so the
 * result does not depend on the order. A launch leaves its pair at zero.
 * Calls on different streams may overlap. A captured graph holding one of
 * these calls uses the pair of the stream it was captured on: do not replay
 * it while other calls run on that stream.
 */
int32_t moe_grouped_gate_up_wgrad(const void* x_perm_d, const void* dgu_d,
                                  const int32_t* offsets_d, const int32_t* counts_d,
                                  int32_t num_local_experts, int64_t m_cap, int32_t hidden,
                                  int32_t inter, void* dw1_d, void* dw3_d, void* stream);

int32_t moe_grouped_down_wgrad(const void* h_d, const void* dy_d, const int32_t* offsets_d,
                               const int32_t* counts_d, int32_t num_local_experts,
                               int64_t m_cap, int32_t inter, int32_t hidden, void* dw2_d,
                               void* stream);

/*
 * moe_linear -- dense matrix product with bias, activation and residual.
 *
 *   z = x w^T + bias          fp32 sums of the 16-bit products, bias added in fp32
 *   y = act(z) + residual     fp32, rounded once to y's type
 *   pre = z, rounded to the rows' type (kept for moe_linear_backward; NULL: not stored)
 *
 * act: none, relu, silu z / (1 + e^-z), or gelu z Phi(z) (Phi the normal
 * distribution function), within 2^-21 (2 + |z|) and 2^-21 (1 + z^2 / 2) of itself where it is
 * above 2^-118 (and below that, within 2^-118). The router projection (fp32 logits from 16-bit
 * rows), a shared expert's products and dense layers.
 *   x_d         [rows, inner], row stride ldx;  w_d: MOE_W_NK [cols, inner] or MOE_W_KN
 *               [inner, cols], row stride ldw; both of `dtype`, 16-byte aligned
 *   bias_d      [cols] float, or NULL
 *   residual_d  [rows, cols] of `dtype`, row stride ldr, or NULL
 *   y_d         [rows, cols] of `dtype` or (y_f32) float, row stride ldy (out)
 *   pre_d       [rows, cols] of `dtype`, row stride ldp, or NULL (out)
 * y may be the residual itself (same address, stride and type); other buffers
 * must not overlap (an output that begins where another buffer does is refused). Strides
 * are in elements; ldr and ldp are read only where their buffer is given.
 * A masked row's values reach that row of y alone.
 * Limits: 0 <= rows < 2^31, 8 <= inner, 1 <= cols, both <= 2^20; dtype MOE_ROWS_BF16 or
 * MOE_ROWS_F16 and inner, ldx and ldw multiples of 8, with MOE_W_KN cols too (else
 * MOE_ERR_UNSUPPORTED); strides at least the row length and at most 2^21. A product of more
 * tiles of 256 x 256 outputs than one launch takes, about 2^23, is MOE_ERR_UNSUPPORTED.
 *   workspace_d >= moe_linear_workspace_bytes(desc) bytes, 16-byte aligned (NULL if that
 *   is 0); contents on entry do not matter. Calls that may overlap need workspaces of their own.
 */
enum { MOE_W_NK = 0, MOE_W_KN = 1 };
enum { MOE_ACT_NONE = 0, MOE_ACT_RELU = 1, MOE_ACT_SILU = 2, MOE_ACT_GELU = 3 };
enum { MOE_DZ_16BIT = 16 }; /* with act: moe_linear_backward's dz in one part (no effect on moe_linear) */

typedef struct moe_linear_desc {
  int64_t rows;    /* M */
  int32_t inner;   /* K */
  int32_t cols;    /* N */
  int32_t dtype;   /* MOE_ROWS_BF16 or MOE_ROWS_F16 */
  int32_t w_order; /* MOE_W_* */
  int32_t act;     /* MOE_ACT_*, or with MOE_DZ_16BIT */
  int32_t y_f32;   /* 0: y (backward: dy) of dtype, 1: float */
  int64_t ldx, ldw, ldy, ldr, ldp;
} moe_linear_desc;

/* Bytes of workspace of the two calls (0 for an invalid descriptor). */
size_t moe_linear_workspace_bytes(const moe_linear_desc* desc);
size_t moe_linear_backward_workspace_bytes(const moe_linear_desc* desc);

int32_t moe_linear(const moe_linear_desc* desc, const void* x_d, const void* w_d,
                   const float* bias_d, const void* residual_d, void* y_d, void* pre_d,
                   void* workspace_d, size_t workspace_bytes, void* stream);

/*
 * moe_linear_backward -- gradients of moe_linear from dy [rows, cols] (of
 * dtype, or float with y_f32; row stride ldy) and the pre-activation:
 *
 *   dz = dy act'(pre)   fp32; the matrix cores read 16-bit values, so the two products take
 *                       it as two parts of dtype, dz rounded and what that leaves rounded:
 *                       2^-16 of dz is lost in bf16, 2^-22 in fp16 (or 2^-25, if that is
 *                       more). With act | MOE_DZ_16BIT as its first part alone, 2^-8 or
 *                       2^-11 (nothing is lost of a dtype dy under act none or relu, which is
 *                       one part anyway): half the products, and a second rounding of
 *                       the size that dx and dw have themselves. act' of an infinite
 *                       pre (z past fp16's range) is its limit
 *   dx = dz w           [rows, inner] of dtype, dense
 *   dw = dz^T x         in w's order, of dtype, dense
 *   dbias = column sums of the unrounded dz, [cols] float
 *
 * fp32 sums, one rounding per output; the residual's gradient is dy. dx_d,
 * dw_d and dbias_d may each be NULL to skip it. pre_d is needed unless act is none, w_d
 * for dx, x_d for dw. An infinity in w or x makes what it reaches NaN where the second part's
 * product with it is NaN or of the other sign. With fp16 rows, dz below fp16's range is lost, and dz past 65504 is an
 * infinity, also from a finite float dy, as are (or NaN) the row of dx and the row or column of
 * dw that it reaches: scale the loss so that dz lies in between.
 * rows = 0 sets dw and dbias to zero. dx_d and dw_d 16-byte aligned; limits and
 * workspace as moe_linear, with moe_linear_backward_workspace_bytes.
 */
int32_t moe_linear_backward(const moe_linear_desc* desc, const void* dy_d, const void* x_d,
                            const void* w_d, const void* pre_d, void* dx_d, void* dw_d,
                            float* dbias_d, void* workspace_d, size_t workspace_bytes,
                            void* stream);

/*
 * moe_rms_norm -- the residual's addition and the root-mean-square norm.
 *
 *   total = x + residual      fp32, rounded to the rows' type (no residual: total = x)
 *   y = total rstd gain       rstd = 1 / sqrt(mean(total^2) + eps), of the rounded total
 *
 * fp32 sums; y goes out rounded once to the rows' type and/or, unrounded, into 8 bits as
 * moe_quantize_fp8 takes it. The norm in front of a layer: y for the router, q and its
 * scales for the experts, total for the residual stream.
 *   x_d         [rows, hidden] of `dtype`, row stride ldx
 *   residual_d  [rows, hidden] of `dtype`, row stride ldr, or NULL
 *   gain_d      [hidden] float, or NULL (ones)
 *   total_d     [rows, hidden] of `dtype`, row stride ldt, or NULL (out; needs residual_d)
 *   y_d         [rows, hidden] of `dtype`, row stride ldy, or NULL (out)
 *   q_d         [rows, hidden] e4m3, dense, or NULL (out); scale_d [rows, ceil(hidden / 128)]
 *               float, with q_d (out)
 * total and y may each be x or the residual (same address and stride), not both the same one; other
 * buffers must not overlap. A row whose sum of squares is past fp32's range gets rstd = 0, one whose squares
 * vanish (all below about 1e-23) with eps = 0 an infinite rstd; a NaN reaches its row alone. rows = 0 is a no-op.
 * Limits: 0 <= rows < 2^31, hidden a multiple of 8, 8 <= hidden <= 16384, eps >= 0 and finite,
 * dtype MOE_ROWS_*, strides multiples of 8 from hidden to 2^21, all buffers 16-byte aligned.
 */
typedef struct moe_norm_desc {
  int64_t rows;
  int32_t hidden;
  int32_t dtype; /* MOE_ROWS_* */
  float eps;
  int32_t reserved; /* 0 */
  int64_t ldx, ldr, ldt, ldy; /* elements; read only where their buffer is given */
} moe_norm_desc;

int32_t moe_rms_norm(const moe_norm_desc* desc, const void* x_d, const void* residual_d,
                     const float* gain_d, void* total_d, void* y_d, void* q_d, float* scale_d,
                     void* stream);

/*
 * moe_rms_norm_backward -- gradients of moe_rms_norm from those of y and total.
 *
 *   dx = rstd (gain dy - xhat mean(gain dy xhat)) + dtotal,   xhat = total rstd
 *   dgain = sum over rows of dy xhat
 *
 * dx is the gradient of x and of the residual alike. fp32 (the rows' workgroups' dgain
 * added in fp64, in order), one rounding per output.
 *   dy_d      [rows, hidden] of `dtype`, row stride ldy
 *   total_d   [rows, hidden] the forward's total (x, without a residual), row stride ldx
 *   dtotal_d  [rows, hidden] what reaches total past the norm, row stride ldt, or NULL
 *   dx_d      [rows, hidden], row stride ldr, or NULL (out); may be dy, total or dtotal
 *             (same address and stride)
 *   dgain_d   [hidden] float, or NULL (out); rows = 0 sets it to zero
 *   workspace_d >= moe_rms_norm_backward_workspace_bytes(desc) bytes, 16-byte aligned, where dgain_d
 *             is given; contents on entry do not matter
 * Limits as moe_rms_norm.
 */
size_t moe_rms_norm_backward_workspace_bytes(const moe_norm_desc* desc);

int32_t moe_rms_norm_backward(const moe_norm_desc* desc, const void* dy_d, const void* total_d,
                              const float* gain_d, const void* dtotal_d, void* dx_d,
                              float* dgain_d, void* workspace_d, size_t workspace_bytes,
                              void* stream);

/*
 * 8-bit values: e4m3 (1 sign, 4 exponent, 3 fraction bits, largest 448, no infinity), with
 * an fp32 scale s for each run of 128:
 *
 *   s = max(amax / 448, 2^-126),  q = e4m3(v (1 / s)),   v is held as q s
 *
 * amax is the largest magnitude among the run's finite values; a value that is not finite
 * becomes NaN. fp32 operations, each rounded once, then one rounding (nearest even) to e4m3.
 *
 * moe_quantize_fp8: rows, a scale for each 128 columns (the last run may be shorter).
 *   x_d [rows, hidden] of `dtype`, row stride ldx;  q_d [rows, hidden];
 *   scale_d [rows, ceil(hidden / 128)] float (out)
 * Limits: 0 <= rows, hidden a multiple of 8 from 8 to 2^20, rows * ceil(hidden / 128) < 2^31, ldx a
 * multiple of 8 from hidden to 2^21.
 *
 * moe_quantize_fp8_weights: matrices, a scale for each block of 128 x 128 (the last ones
 * may be smaller), stored output-major, as the products read them.
 *   w_d     MOE_W_NK: [num_mats, cols, inner], MOE_W_KN: [num_mats, inner, cols], of `dtype`
 *   q_d     [num_mats, cols, inner];  scale_d [num_mats, ceil(cols / 128), ceil(inner / 128)] (out)
 * Limits: 0 <= num_mats < 65536, inner a multiple of 16 (MOE_W_KN: cols a multiple of 8), both
 * from 1 to 2^20.
 * All buffers 16-byte aligned; outputs must not overlap an input.
 */
int32_t moe_quantize_fp8(int32_t dtype, const void* x_d, int64_t rows, int32_t hidden, int64_t ldx,
                         void* q_d, float* scale_d, void* stream);

int32_t moe_quantize_fp8_weights(int32_t dtype, const void* w_d, int32_t num_mats, int32_t inner,
                                 int32_t cols, int32_t w_order, void* q_d, float* scale_d,
                                 void* stream);

/*
 * moe_linear_fp8 -- moe_linear on 8-bit operands.
 *
 *   z[m, n] = sum over runs b of x_scale[m, b] w_scale[n / 128, b] (sum over k in run b of x[m, k] w[n, k])
 *             + bias[n]
 *   y = act(z) + residual      fp32, rounded once to y's type
 *
 * The products of a run are summed on the matrix cores, the runs in fp32, with 24 bits throughout.
 * With act | MOE_FP8_FAST, more than 64 rows are summed by the 8-bit matrix instruction, up to twice as
 * fast, which cuts each of 8 neighbouring products to a multiple of 2^-13 of the largest one's power of two
 * before it adds them: 1.4e-5 of y's norm on normal values, and more where large products
 * cancel. act as in moe_linear.
 * The gradient of x is the same product with the transposed weights: blocks of 128 x 128
 * keep their values when turned over (moe_quantize_fp8_weights with the other w_order).
 *   x_d         [rows, inner] e4m3, dense;  x_scale_d [rows, ceil(inner / 128)] float
 *   w_d         [cols, inner] e4m3, dense;  w_scale_d [ceil(cols / 128), ceil(inner / 128)] float
 *   bias_d      [cols] float, or NULL
 *   residual_d  [rows, cols] of `dtype`, row stride ldr, or NULL
 *   y_d         [rows, cols] of `dtype` or (y_f32) float, row stride ldy (out)
 * y may be the residual itself (same address, stride and type); other buffers must not overlap.
 * Limits: 0 <= rows < 2^31, inner a multiple of 16 from 16 to 2^20, 1 <= cols <= 2^20; dtype
 * MOE_ROWS_BF16 or MOE_ROWS_F16; ldy and (read only with its buffer) ldr from cols to 2^21; fewer than 2^26
 * tiles of 128 x 128 outputs and 2^32 - 64 pieces of 8 columns of a row (else MOE_ERR_UNSUPPORTED). x_d and w_d 16-byte aligned.
 *   workspace_d >= moe_linear_fp8_workspace_bytes(desc) bytes, 16-byte aligned (NULL if that
 *   is 0); contents on entry do not matter. Calls that may overlap need workspaces of their own.
 */
enum { MOE_FP8_FAST = 32 }; /* with act: moe_linear_fp8's sums by the 8-bit matrix instruction */

typedef struct moe_linear_fp8_desc {
  int64_t rows;  /* M */
  int32_t inner; /* K */
  int32_t cols;  /* N */
  int32_t dtype; /* MOE_ROWS_BF16 or MOE_ROWS_F16: of y (unless y_f32) and the residual */
  int32_t act;   /* MOE_ACT_*, or with MOE_FP8_FAST */
  int32_t y_f32; /* 0 or 1 */
  int32_t reserved; /* 0 */
  int64_t ldy, ldr;
} moe_linear_fp8_desc;

size_t moe_linear_fp8_workspace_bytes(const moe_linear_fp8_desc* desc);

int32_t moe_linear_fp8(const moe_linear_fp8_desc* desc, const void* x_d, const float* x_scale_d,
                       const void* w_d, const float* w_scale_d, const float* bias_d,
                       const void* residual_d, void* y_d, void* workspace_d,
                       size_t workspace_bytes, void* stream);

/*
 * Grouped SwiGLU expert MLPs on 8-bit operands: moe_grouped_gate_up (and, with src_row_d,
 * moe_grouped_gate_up_gather) and moe_grouped_down with e4m3 rows, e4m3 weights and their scales,
 * for serving. For local expert e the rows [offsets[e], offsets[e] + counts[e]):
 *
 *   moe_grouped_gate_up_fp8:  h = silu(x W1[e]) * (x W3[e]), fp32, then e4m3 with a scale for each
 *                             128 columns of a row, as moe_quantize_fp8 takes it
 *   moe_grouped_down_fp8:     y = h W2[e], rounded once to bf16
 *
 * Sums with 24 bits throughout; with `fast` by the 8-bit instruction (moe_linear_fp8), whatever the rows, up
 * to 1.8 times as fast with many rows to a group, gate_up's scales up to 2e-5 off (root mean square). Rows outside the groups are
 * neither read nor written.
 *   x_d        [m_cap, inner] e4m3, or with src_row_d [num_tokens, inner]: row r of the groups is then
 *              x[src_row[r] / top_k] (moe_layout's src_row); a row whose src_row is not of [0, num_tokens top_k)
 *              holds no defined values
 *   x_scale_d  [rows of x, inner / 128] float
 *   w1_d, w3_d, w2_d  [num_groups, cols, inner] e4m3, output-major (moe_quantize_fp8_weights with MOE_W_KN
 *              takes the math orientation); their scales [num_groups, cols / 128, inner / 128] float
 *   offsets_d  [num_groups + 1], counts_d [num_groups] int32, as in moe_grouped_gate_up
 *   h_d        [m_cap, cols] e4m3, h_scale_d [m_cap, cols / 128] float (out);  y_d [m_cap, cols] bf16 (out)
 *   max_rows   a group's rows from max_rows on are not computed (the token count, say: a token
 *              comes to an expert once)
 * gate_up: inner is the hidden size, cols the experts' inner size; down: the other way round.
 * Limits: inner and cols multiples of 128, at most 2^20; 1 <= num_groups <= 1024; m_cap < 2^31; with
 * src_row_d 1 <= top_k <= 16 and num_tokens * inner < 2^31; m_cap / 65 + num_groups tiles of 256 columns (gate_up:
 * 128) fewer than 2^30; else MOE_ERR_UNSUPPORTED. Device pointers 16-byte aligned (offsets_d, counts_d, src_row_d: 4).
 */
typedef struct moe_grouped_fp8_desc {
  int64_t m_cap;
  int64_t max_rows;
  int64_t num_tokens; /* with src_row_d */
  int32_t num_groups;
  int32_t inner;
  int32_t cols;
  int32_t top_k; /* with src_row_d */
  int32_t fast;  /* 0 or 1 */
  int32_t reserved; /* 0 */
} moe_grouped_fp8_desc;

int32_t moe_grouped_gate_up_fp8(const moe_grouped_fp8_desc* desc, const void* x_d,
                                const float* x_scale_d, const int32_t* src_row_d,
                                const int32_t* offsets_d, const int32_t* counts_d,
                                const void* w1_d, const float* w1_scale_d, const void* w3_d,
                                const float* w3_scale_d, void* h_d, float* h_scale_d,
                                void* stream);

int32_t moe_grouped_down_fp8(const moe_grouped_fp8_desc* desc, const void* h_d,
                             const float* h_scale_d, const int32_t* offsets_d,
                             const int32_t* counts_d, const void* w2_d, const float* w2_scale_d,
                             void* y_d, void* stream);

/*
 * moe_combine -- fused weighted-sum restore.
 *
 * The fused restore of DeepSpeed PR #8847 ("AutoEP: support
 * combine_impl=fused_weighted_sum ...", sections "Problem" and "Change"):
 * each row is addressed by the flat index token*top_k + slot, the routing
 * weights stay FP32 in a [tokens, top_k] layout, and weight x row products
 * are accumulated in FP32 (section "Benchmark": the error left is the bf16
 * output rounding). Per token t:
 *
 *   out[t, :] = bf16( sum over slots s = 0..k-1 with 0 <= dst_row[t, s] < y_rows
 *                     of topk_w[t, s] * y[dst_row[t, s], :] )
 *
 * summed in fp32 in slot order (each product rounded to fp32, then added:
 * no fused multiply-add), rounded once to bf16 (nearest even). A token with no local slot gets a zero row. The result
 * does not depend on where the rows sit in y.
 *   y_d       [y_rows, H] bf16, 16-byte aligned
 *   dst_row_d [T, k] int32;  topk_w_d [T, k] float
 *   out_d     [T, H] bf16 (out), 16-byte aligned
 * Limits: H a multiple of 8, 8 <= H <= 16384; 1 <= k <= 16.
 */
int32_t moe_combine(const void* y_d, int64_t y_rows, const int32_t* dst_row_d,
                    const float* topk_w_d, int64_t num_tokens, int32_t hidden,
                    int32_t top_k, void* out_d, void* stream);

/*
 * Backward of the combine, the permute and the routing weights.
 *
 * The fused restore back-propagates a row gradient and a score gradient, the
 * score (router) gradient in FP32 (DeepSpeed PR #8847, sections "Tests" and
 * "Benchmark"); the backward of a combine is a dispatch of the output
 * gradient and the backward of a dispatch is a combine (DeepEP issue #272,
 * the maintainer's answer). G is the gradient of the combine's output.
 *
 * moe_combine_backward: for every (t, s) with 0 <= r = dst_row[t, s] < y_rows
 *   grad_y[r, :]  = bf16(topk_w[t, s] * G[t, :])    (fp32 product, one rounding)
 *   grad_w[t, s]  = sum_h G[t, h] * y[r, h]          (fp32, tree-shaped sum)
 * and grad_w[t, s] = 0 for every other slot. Rows of grad_y that no slot
 * points at are not written.
 *   grad_out_d [T, H] bf16;  y_d [y_rows, H] bf16 (the forward's expert output)
 *   dst_row_d, topk_w_d [T, k] as in moe_combine
 *   grad_y_d   [y_rows, H] bf16 (out);  grad_w_d [T, k] float (out)
 * Limits as moe_combine; bf16 pointers 16-byte aligned.
 */
int32_t moe_combine_backward(const void* grad_out_d, const void* y_d, int64_t y_rows,
                             const int32_t* dst_row_d, const float* topk_w_d,
                             int64_t num_tokens, int32_t hidden, int32_t top_k,
                             void* grad_y_d, float* grad_w_d, void* stream);

/*
 * moe_permute_backward: grad_x[t, :] = bf16( sum over slots s with
 *   0 <= dst_row[t, s] < x_perm_rows of grad_x_perm[dst_row[t, s], :] ),
 * an fp32 sum in slot order rounded once (moe_combine with unit weights); a
 * token with no local slot gets a zero row.
 *   grad_x_perm_d [x_perm_rows, H] bf16;  grad_x_d [T, H] bf16 (out)
 * Limits as moe_combine.
 */
int32_t moe_permute_backward(const void* grad_x_perm_d, int64_t x_perm_rows,
                             const int32_t* dst_row_d, int64_t num_tokens, int32_t hidden,
                             int32_t top_k, void* grad_x_d, void* stream);

/*
 * moe_route_backward: the routing weights are the softmax of the k selected
 * logits (moe_route), so with g = grad_w[t, :] (the score gradient)
 *   grad_logits[t, topk_idx[t, j]] = topk_w[t, j] * (g_j - sum_i topk_w[t, i] * g_i)
 * (the sum in fp32, slot order) and 0 for every unselected expert.
 *   topk_idx_d, topk_w_d, grad_w_d [T, k];  grad_logits_d [T, E] float (out)
 * Limits as moe_route; T * E < 2^32 (else MOE_ERR_UNSUPPORTED).
 */
int32_t moe_route_backward(const int32_t* topk_idx_d, const float* topk_w_d,
                           const float* grad_w_d, int64_t num_tokens, int32_t num_experts,
                           int32_t top_k, float* grad_logits_d, void* stream);

/*
 * Norm of all gradients together, and clipping (what follows the weight
 * gradients in a training step).
 *
 *   moe_grad_sumsq:  sumsq = sum of g^2 over every element of every tensor, in fp64
 *   moe_grad_clip:   norm = sqrt(sumsq);  coef = min(1, max_norm / (norm + 1e-6));
 *                    out = g * coef (fp32 product, one rounding);  norm_d = norm
 *
 * Two calls, so that ranks holding different parameters (expert parallelism)
 * can add their sums in between. A norm that is not finite gives what the
 * formula gives: coef NaN for a NaN norm, 0 for an infinite one (1 if max_norm is
 * infinite too: no bound). The order of the sum is
 * fixed by the tensors' order and sizes. In place, with coef = 1, nothing is written.
 *   tensors      HOST array of num_tensors descriptors, read during the call: `data` (device, aligned to
 *                its elements; may be NULL if numel is 0), `out` (moe_grad_clip: where the scaled
 *                tensor goes, of the same type; NULL or `data`: in place), numel, dtype MOE_ROWS_*
 *   sumsq_d      [1] double (moe_grad_sumsq: out, moe_grad_clip: in)
 *   norm_d       [1] float (out), or NULL
 *   max_norm     >= 0 (infinity: no bound)
 *   workspace_d  >= moe_grad_sumsq_workspace_bytes(...) bytes, 8-byte aligned
 * A tensor may appear twice in moe_grad_sumsq (it counts twice); moe_grad_clip refuses
 * tensors of which one is written and shares memory with another (MOE_ERR_ARG).
 * Limits: 0 <= num_tensors <= 65536, 0 <= numel < 2^44. No tensors: the sum is 0.
 */
typedef struct moe_tensor_ref {
  const void* data;
  void* out;
  int64_t numel;
  int32_t dtype;
  int32_t reserved; /* 0 */
} moe_tensor_ref;

size_t moe_grad_sumsq_workspace_bytes(const moe_tensor_ref* tensors, int32_t num_tensors);

int32_t moe_grad_sumsq(const moe_tensor_ref* tensors, int32_t num_tensors, double* sumsq_d,
                       void* workspace_d, size_t workspace_bytes, void* stream);

int32_t moe_grad_clip(const moe_tensor_ref* tensors, int32_t num_tensors, const double* sumsq_d,
                      float max_norm, float* norm_d, void* stream);

/*
 * moe_combine_rows -- the fused restore on other row dtypes and variants.
 *
 * The fused restore runs on bf16 and on fp32 rows (DeepSpeed PR #8847,
 * section "Tests"); fp16 rows are the third activation dtype the page
 * discusses. Per token t:
 *
 *   out[t, :] = round( sum over local slots s, in slot order, of w[t, s] * y[dst_row[t, s], :]
 *                      + shared[t, :] )
 *
 * in fp32 (products, then sums, no fused multiply-add) and rounded once to the
 * row dtype (nearest even; fp32 rows are not rounded again). topk_w_d = NULL
 * gives w = 1, the plain sum used when the score was applied before the
 * experts (moe_permute_weighted). shared_d = NULL adds nothing; otherwise it
 * holds the output rows [T, H] of a shared expert, merged as the last step of
 * the AutoEP runtime (DeepSpeed AutoEP commit text, section "Design": merge
 * shared experts if the model has them). y_d, shared_d and out_d are all of
 * the row dtype; MOE_ROWS_BF16 with weights and no shared rows is moe_combine.
 * Limits as moe_combine.
 */
int32_t moe_combine_rows(const void* y_d, int32_t row_dtype, int64_t y_rows,
                         const int32_t* dst_row_d, const float* topk_w_d, const void* shared_d,
                         int64_t num_tokens, int32_t hidden, int32_t top_k, void* out_d,
                         void* stream);

/*
 * moe_validate_layout -- debug check of a layout (SYNCHRONISES the stream,
 * copies the buffers to the host and checks there). Mirrors the fused
 * restore's coverage check (DeepSpeed PR #8847, section "Change": a missing
 * (token, slot) raises instead of reading an unset row).
 * Returns MOE_OK, MOE_ERR_EXPERT_ID (id out of range or repeated in a token),
 * MOE_ERR_COVERAGE (a local (t, slot) without a row, or a row claimed twice) or
 * MOE_ERR_LAYOUT (offsets not aligned/monotone, src_row and dst_row not
 * inverse, padding or order wrong). `detail` (may be NULL) receives a
 * NUL-terminated message of at most detail_len bytes.
 */
int32_t moe_validate_layout(const moe_layout_desc* desc, const int32_t* topk_idx_d,
                            const int32_t* offsets_d, const int32_t* dst_row_d,
                            const int32_t* src_row_d, int64_t m_cap, void* stream,
                            char* detail, size_t detail_len);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
