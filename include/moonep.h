/*
 * moonep.h -- C ABI of the balanced expert-parallel hot path on one MI355X (gfx950).
 *
 * R expert-parallel ranks are simulated as partitions of one GPU's HBM.  One MoE layer
 * step runs four calls, in the order the pages give for a forward and backward pass
 * ("MoonshotAI/MoonEP 딥다이브" (fiv.co.kr), section 5: planning -> dispatch -> expert
 * compute -> combine -> grad_reduce):
 *
 *   moonep_plan        live top-K router output -> replica plan + token->row map
 *   moonep_dispatch    zero-copy scatter of bf16 token rows into static per-rank buffers
 *   moonep_combine     weighted gather of expert outputs back to token order
 *   moonep_reduce_grad replica gradients summed into their home experts
 *
 * Notation.  T = R*S tokens; token t comes from rank t / S.  Assignment i = t*K + k.
 * E_loc = E/R experts per rank; expert e is homed on rank e / E_loc.  C = S*K is every
 * rank's exact quota ("Moonshot AI Open-Sources MoonEP" (tldrocket.com), paragraph 3).
 * G = E_loc + slots groups per rank.  NvS = align16(C + G*15) rows per rank buffer
 * (S*K plus alignment padding: deep dive, section 4, design pattern 2).
 *
 * Conventions for every call:
 *   - Device pointers are plain HIP device addresses; the caller owns and allocates all
 *     memory.  The library never allocates, frees or synchronises (except
 *     moonep_plan_status, which waits on `stream`).  moonep_plan_noalloc alone uses
 *     library-owned device memory: a static per-GPU workspace array.
 *   - All GPU work is enqueued on `stream` (0 = the null stream) and is asynchronous.
 *   - Return value: MOONEP_OK (0) or a negative MOONEP_E* code.  Argument errors
 *     (EINVAL, ELIMIT, EALIGN, EPLAN) are found on the host and nothing is enqueued; an
 *     EHIP from a call that launches several kernels (moonep_plan, the staged calls, the
 *     experts' forward calls and rows' gradient, the norm's backward) can follow launches of
 *     that call that were already enqueued.  Each call clears the
 *     thread's earlier HIP error before launching, so an EHIP is its own.  Data errors
 *     found on the device (an expert id outside [0, E)) are never reported by a return
 *     code: they set the plan's status word, read with moonep_plan_status; such a plan
 *     maps nothing (every dst_row is -1), dispatch and the experts' forward calls and rows'
 *     gradient then write nothing, combine writes zero rows, reduce adds nothing, and the
 *     weights' gradient is that of no rows.
 *   - Calls are thread-safe; the library has no global mutable state apart from
 *     moonep_plan_noalloc's per-GPU workspace array (see there).
 */
#ifndef MOONEP_H_
#define MOONEP_H_

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOONEP_ROW_ALIGN 16      /* rows: each home/slot group starts on a multiple */
#define MOONEP_MAX_R 64          /* the planner keeps one wave64 lane per rank      */
#define MOONEP_MAX_E 1024
#define MOONEP_MAX_K 32
#define MOONEP_MAX_SLOTS 256
#define MOONEP_MAX_FFN 32768     /* hidden and intermediate sizes of an expert          */
#define MOONEP_MAX_NORM 32768    /* hidden size of a normed row                         */
#define MOONEP_ACT_SILU 0        /* z / (1 + e^-z)                                      */
#define MOONEP_ACT_GELU 1        /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2     */
#define MOONEP_F32 0             /* types of the router's logits                        */
#define MOONEP_BF16 1
#define MOONEP_SCORE_SOFTMAX 0   /* the router's scores of an expert's logit            */
#define MOONEP_SCORE_SIGMOID 1
#define MOONEP_MAX_GROUPS 64     /* the router's groups of experts                      */
/* the matrix products of the experts' calls (moonep_expert_tile)                      */
#define MOONEP_PRODUCT_GATE_UP 0   /* moonep_expert_ffn: gate and up, with the activation */
#define MOONEP_PRODUCT_DOWN 1      /* moonep_expert_ffn: y                                */
#define MOONEP_PRODUCT_G_GATE_UP 2 /* moonep_expert_ffn_bwd_data: g_gu                    */
#define MOONEP_PRODUCT_G_ROWS 3    /* moonep_expert_ffn_bwd_data: g_recv                  */
#define MOONEP_PRODUCT_G_WEIGHTS 4 /* moonep_expert_ffn_bwd_weight                        */
/* largest planning workspace moonep_plan_noalloc serves from its static device array */
#define MOONEP_NOALLOC_WORKSPACE_MAX (8 << 20)

enum {
  MOONEP_OK = 0,
  MOONEP_EINVAL = -1,   /* a size or pointer argument is invalid                       */
  MOONEP_ELIMIT = -2,   /* sizes beyond MOONEP_MAX_* or int32 row indexing              */
  MOONEP_EPLAN = -3,    /* the plan descriptor is not initialised or does not match     */
  MOONEP_EHIP = -4,     /* a HIP launch or copy failed                                  */
  MOONEP_EALIGN = -5    /* a data pointer is not 16-byte aligned                        */
};

/* Sizes of one (R, E, K, S, slots) problem; filled by moonep_query (host only). */
typedef struct moonep_sizes {
  int32_t R, E, K, S, slots;
  int32_t E_loc, C, G, NvS, P_max;
  int64_t T, A;
  int64_t recv_rows;        /* R * NvS: rows of the dispatch buffer [R, NvS, H]          */
  int64_t plan_bytes;       /* device bytes of the plan blob                             */
  int64_t workspace_bytes;  /* device bytes of the transient workspace of moonep_plan    */
  int32_t nblk, blk;        /* assignment blocks used by the plan kernels                */
  /* int32-element offsets of the plan blob's arrays (for inspection and tests):        */
  int64_t o_hdr, o_load, o_shed, o_keep, o_home_row, o_pfirst, o_pnum, o_pieces,
          o_slot_expert, o_off, o_red, o_xtab, o_ptab, o_dst_row, o_w;
} moonep_sizes;

/* Host-side handle of a plan: sizes plus the caller's device blob.  Filled by
 * moonep_plan; read by the other calls.  Copying the struct copies the handle. */
typedef struct moonep_plan_desc {
  uint32_t magic;
  moonep_sizes sz;
  void* dev;                /* device blob of sz.plan_bytes, 256-byte aligned            */
} moonep_plan_desc;

/* Plan statistics, copied from the device by moonep_plan_status. */
typedef struct moonep_plan_stats {
  int32_t status;           /* 0 = valid plan; 1 = an expert id was outside [0, E)       */
  int32_t bad_index;        /* smallest assignment index with a bad id, else -1          */
  int32_t n_pieces;         /* replica pieces (slot-backed + fallback)                   */
  int32_t n_replicas;       /* slot-backed pieces = prefetch slots in use                */
  int32_t n_fallback;       /* pieces served by cross-partition weight reads             */
  int32_t max_pieces_per_rank;
  int32_t n_red;            /* experts with at least one slot replica                    */
  int32_t n_shed;           /* experts that shed assignments                             */
  int32_t max_load;         /* largest per-expert load                                   */
} moonep_plan_stats;

/* Sizes for a problem, host only ("MoonshotAI/MoonEP 딥다이브", section 4, design
 * pattern 2: per-rank buffers have a static size, S*K rows plus alignment padding, fixed
 * before any routing is seen; section 2, point 3: so the host never waits for the device
 * to learn how much to allocate).  Every buffer the other calls take is sized from here.
 * EINVAL unless R>=1, E%R==0, 1<=K<=E, S>=1, slots>=0; ELIMIT beyond R<=64, E<=1024,
 * K<=32, slots<=256, or when R*NvS or T*K exceeds int32. */
int moonep_query(int R, int E, int K, int S, int slots, moonep_sizes* out);

/* Planning ("Moonshot AI Open-Sources MoonEP", paragraph 3: duplicate a few overloaded
 * experts, planned from live router output, so every rank receives exactly S*K; deep
 * dive, section 4, design pattern 1: plan once, reuse).
 *
 *   topk_ids   device int32 [T, K] row-major, ranks contiguous (token t from rank t/S)
 *   topk_w     device fp32  [T, K]; copied into the plan, so combine needs no weights
 *   plan_dev   device blob of moonep_sizes.plan_bytes, 256-byte aligned
 *   workspace  device scratch of moonep_sizes.workspace_bytes, 256-byte aligned,
 *              zero-filled before its first use: its first word counts the planning
 *              workgroups as they finish, and every call leaves it at zero again, so a
 *              workspace reused call after call (for any sizes) needs no clearing.  A
 *              workspace whose first word is not zero leaves the plan undefined; every
 *              kernel that reads a plan still keeps its accesses inside the plan and the
 *              buffers it was given, whatever the plan holds.  Free for other use
 *              once the plan's kernels have run on `stream`; two calls whose kernels
 *              overlap in time must not share a workspace
 *   desc       host handle, filled synchronously (sizes + plan_dev)
 *
 * Boundary note.  The plan is a device blob, as in a blob-only signature, but the call also
 * fills `desc`, a host copy of the problem's sizes plus the blob's address, and every
 * later call takes `desc` instead of the bare blob.  The sizes of every launch (grid,
 * rows, K) are then known on the host without reading the device, so no call ever waits
 * for the plan (the deep dive's section 2, point 3: no per-layer host synchronisation);
 * the blob itself stays on the device and is what the kernels read.
 *
 * Errors: EINVAL, ELIMIT and EALIGN are found on the host before anything is enqueued;
 * EHIP means a launch failed, in which case kernels launched before it by this call may
 * already be enqueued (the plan is then unusable until a later call succeeds).
 *
 * The plan rule: experts are taken by (load descending, id ascending); an expert on a
 * home whose load exceeds S*K sheds min(load, remaining excess); each shed assignment
 * goes to the lowest-id rank still short of S*K that has a free prefetch slot, else
 * (slots exhausted) to the lowest-id rank still short, as a fallback piece whose expert
 * weights are read across partitions ("Moonshot AI Open-Sources MoonEP", paragraph 5).
 * Within an expert, assignments are taken in increasing i: the home keeps the first
 * `keep`, replica pieces take the rest in creation order.  Each rank's buffer holds its
 * home experts, then its slots (each group 16-row aligned), then a fallback region.
 * Deterministic: the same ids give a bit-identical plan. */
int moonep_plan(const int32_t* topk_ids, const float* topk_w, int R, int E, int K, int S,
                int slots, void* plan_dev, void* workspace, moonep_plan_desc* desc,
                hipStream_t stream);

/* moonep_plan for callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  Same arguments, result
 * and errors as moonep_plan, without `workspace`: the planning kernels use a file-scope
 * device array of MOONEP_NOALLOC_WORKSPACE_MAX bytes (8 MiB; enough for every
 * (R, E, K, S, slots) whose moonep_sizes.workspace_bytes is at most that), one copy per GPU,
 * held until the process ends.  The call allocates and frees nothing; the caller still
 * provides topk_ids, topk_w and the plan blob.
 *   ELIMIT  when workspace_bytes exceeds MOONEP_NOALLOC_WORKSPACE_MAX (nothing enqueued)
 *   EINVAL  when `stream` does not belong to the current device (the array used is the
 *           current device's)
 * Every call on one GPU shares that GPU's array: two of these calls whose kernels overlap
 * in time on the same GPU (different streams, or different host threads without ordering)
 * race and may both produce wrong plans.  Calls ordered on one stream are safe.  The array
 * is zero when the library is loaded; every call leaves its first word (the planning
 * workgroups' arrival count) at zero again and the rest holding the last call's
 * contents. */
int moonep_plan_noalloc(const int32_t* topk_ids, const float* topk_w, int R, int E, int K, int S,
                        int slots, void* plan_dev, moonep_plan_desc* desc, hipStream_t stream);

/* Zero-copy dispatch ("MoonshotAI/MoonEP 딥다이브", section 2, point 2: each token row
 * is written straight into its final expert position; no permute, no staging copy):
 *   recv[dst_row[t, k], :] = x[t, :]  (bit copy) for every assignment.
 *   x     device bf16 [T, H] (raw 16-bit patterns)      recv  device bf16 [R*NvS, H]
 * H % 8 == 0; x and recv 16-byte aligned.  Padding rows of recv are not written. */
int moonep_dispatch(const moonep_plan_desc* plan, const uint16_t* x, int H, uint16_t* recv,
                    hipStream_t stream);

/* Weighted combine (deep dive, section 1: dispatch -> expert compute -> combine):
 *   out[t, :] = bf16_rne( sum_{k=0..K-1} w[t,k] * float(y[dst_row[t,k], :]) )
 * accumulated in fp32, k ascending, each product and sum rounded separately (no fused
 * multiply-add), one round-to-nearest-even to bf16 at the end.
 *   y     device bf16 [R*NvS, H] (expert outputs, laid out like recv)
 *   out   device bf16 [T, H]
 * H % 8 == 0; y and out 16-byte aligned; out must not overlap y. */
int moonep_combine(const moonep_plan_desc* plan, const uint16_t* y, int H, uint16_t* out,
                   hipStream_t stream);

/* Staged (non-zero-copy) dispatch, the A/B baseline for zero-copy ("MoonshotAI/MoonEP
 * 딥다이브", section 2, point 2: the conventional scheme receives tokens into a
 * communication buffer, then permutes and copies them into the user buffer; section 8,
 * exercise D measures that copy):
 *   stage[t*K + k, :] = x[t, :]                  (arrival order)
 *   recv[dst_row[t,k], :] = stage[t*K + k, :]    (the epilogue copy)
 * recv ends bit-identical to moonep_dispatch's.  stage: device bf16 [T*K, H]. */
int moonep_dispatch_staged(const moonep_plan_desc* plan, const uint16_t* x, int H,
                           uint16_t* stage, uint16_t* recv, hipStream_t stream);

/* Staged combine (same passage): the prologue copy stage[t*K + k, :] = y[dst_row[t,k], :],
 * then out[t] as in moonep_combine, read from the staging buffer.  out ends bit-identical
 * to moonep_combine's.  stage: device bf16 [T*K, H]. */
int moonep_combine_staged(const moonep_plan_desc* plan, const uint16_t* y, int H,
                          uint16_t* stage, uint16_t* out, hipStream_t stream);

/* Backward of dispatch, reusing the forward plan ("MoonshotAI/MoonEP 딥다이브", section 4,
 * design pattern 1: the plan serves both backward passes).  Dispatch copied x[t] into
 * its K rows, so
 *   gx[t, :] = bf16_rne( sum_{k=0..K-1} float(g_recv[dst_row[t,k], :]) )
 * summed in fp32, k ascending.
 *   g_recv  device bf16 [R*NvS, H] (gradient w.r.t. the dispatched rows)
 *   gx      device bf16 [T, H]
 * H % 8 == 0; both 16-byte aligned; gx must not overlap g_recv. */
int moonep_dispatch_bwd(const moonep_plan_desc* plan, const uint16_t* g_recv, int H,
                        uint16_t* gx, hipStream_t stream);

/* Backward of combine, reusing the forward plan (same passage).  For
 * out[t] = sum_k w[t,k] * y[dst_row[t,k]]:
 *   g_y[dst_row[t,k], :] = bf16_rne( w[t,k] * float(dout[t, :]) )   (fp32 product)
 *   dw[t, k]             = sum_h float(dout[t,h]) * float(y[dst_row[t,k], h])   (fp32, fused
 *                          multiply-add, summation order unspecified)
 *   dout  device bf16 [T, H];  y  device bf16 [R*NvS, H] (the forward expert outputs)
 *   g_y   device bf16 [R*NvS, H], may be y itself (in place); padding rows untouched
 *   dw    device fp32 [T, K]
 * H % 8 == 0; dout, y, g_y 16-byte aligned. */
int moonep_combine_bwd(const moonep_plan_desc* plan, const uint16_t* dout, const uint16_t* y,
                       int H, uint16_t* g_y, float* dw, hipStream_t stream);

/* Replica-gradient reduce (deep dive, section 4, design pattern 3: a replica's gradient
 * is kept apart and added to its home expert, so training equals no replication):
 *   for each expert e, for its slot pieces in creation order:
 *       home_grad[e, :] += rep_grad[rank, slot, :]      (fp32 adds, in that order)
 *   home_grad  device fp32 [E, G_el], updated in place
 *   rep_grad   device fp32 [R, slots, G_el]
 * G_el % 4 == 0; both 16-byte aligned.  Fallback pieces own no slot and add nothing. */
int moonep_reduce_grad(const moonep_plan_desc* plan, float* home_grad, const float* rep_grad,
                       int64_t G_el, hipStream_t stream);

/* Replica weight prefetch ("Moonshot AI Open-Sources MoonEP", paragraph 3: the duplicated
 * experts are prefetched before computation starts; "MoonshotAI/MoonEP 딥다이브", section 3:
 * Buffer.prefetch_weight):
 *   for every slot piece p of the plan:  slot_w[r_p, slot_p, :] = home_w[e_p, :]  (bit copy)
 *   home_w  device bf16 [E, W_el] (each expert's weights, any layout, W_el elements)
 *   slot_w  device bf16 [R, slots, W_el]; slots no piece uses are not written
 * W_el % 8 == 0; both 16-byte aligned; slot_w must not overlap home_w.  Fallback pieces
 * own no slot: their rank reads home_w directly (see moonep_expert_stub). */
int moonep_prefetch_weight(const moonep_plan_desc* plan, const uint16_t* home_w, int64_t W_el,
                           uint16_t* slot_w, hipStream_t stream);

/* A toy expert that checks which weights each buffer group reads ("Moonshot AI
 * Open-Sources MoonEP", paragraph 5: without a free slot the rank falls back to remote
 * reads of the home expert):
 *   y[row, h] = bf16_rne( float(recv[row, h]) * float(W[h]) ),  h < H,
 * for every mapped row, where W is home_w[e] for a home group, slot_w[r, slot] for a slot
 * group and home_w[e] (read across partitions) for a fallback piece.  The row's expert e
 * comes from the caller's topk_ids (the same array given to moonep_plan).
 *   topk_ids int32 [T, K];  recv, y  bf16 [R*NvS, H];  home_w bf16 [E, W_el];
 *   slot_w bf16 [R, slots, W_el]  (W_el >= H, W_el % 8 == 0, H % 8 == 0)
 * Padding rows of y are not written. */
int moonep_expert_stub(const moonep_plan_desc* plan, const int32_t* topk_ids,
                       const uint16_t* recv, const uint16_t* home_w, const uint16_t* slot_w,
                       int64_t W_el, int H, uint16_t* y, hipStream_t stream);

/* The gated feed-forward experts, the expert compute between dispatch and combine ("MoonshotAI/MoonEP
 * 딥다이브", section 1: dispatch -> expert compute -> combine; section 2, point 2: the
 * receive buffer is handed to expert compute as a view).  For every mapped row:
 *   gate = Wg x, up = Wu x, h = act(gate) * up        (one kernel; fp32 sums, h rounded to bf16 once)
 *   y = Wd h                                          (fp32 sums, rounded to bf16 once)
 * with the weights the row's group uses: home_w[e] for a home group, slot_w[r, slot] for a
 * slot group and home_w[e] (read across partitions) for a fallback piece.
 *   recv    device bf16 [R*NvS, H]
 *   home_w  device bf16 [E, W_el]: an expert's slab is its gate [I, H], up [I, H] and down
 *           [H, I] matrices, row-major, in this order; W_el >= 3*I*H is the slabs' pitch
 *   slot_w  device bf16 [R, slots, W_el] (moonep_prefetch_weight's)
 *   act     MOONEP_ACT_SILU or MOONEP_ACT_GELU
 *   gu      device bf16 [R*NvS, 2*I] or NULL: gate, then up, of every row, for the backward pass
 *   h       device bf16 [R*NvS, I]: scratch of an inference call; the weights' gradient reads it
 *   y       device bf16 [R*NvS, H]
 * H and I are multiples of 8, at most MOONEP_MAX_FFN, with (I + 256) * H < 2^30; W_el is a
 * multiple of 8; all pointers 16-byte aligned.  Padding rows of recv are not read and those
 * of gu, h and y not written.  No output may overlap an input, the plan or another output
 * (EINVAL).  EHIP can follow the first of the two launches.  Deterministic. */
int moonep_expert_ffn(const moonep_plan_desc* plan, const uint16_t* recv, int H, int I, int act,
                      const uint16_t* home_w, const uint16_t* slot_w, int64_t W_el, uint16_t* gu,
                      uint16_t* h, uint16_t* y, hipStream_t stream);

/* Gradient of moonep_expert_ffn with respect to the rows, reusing the forward plan (deep
 * dive, section 4, design pattern 1).  For every mapped row:
 *   g_h = Wd^T g_y;  g_gate = g_h * up * act'(gate),  g_up = g_h * act(gate)
 *   g_recv = Wg^T g_gate + Wu^T g_up
 * from the saved gate and up of `gu`; fp32 sums, g_gate and g_up rounded to bf16 (they are
 * an output, and the second product's input), g_recv rounded to bf16 once.
 *   g_y     device bf16 [R*NvS, H]      gu      device bf16 [R*NvS, 2*I]
 *   g_gu    device bf16 [R*NvS, 2*I], may be gu itself (in place)
 *   g_recv  device bf16 [R*NvS, H]
 * Weights, sizes, padding rows, overlaps (but g_gu == gu) and errors as in moonep_expert_ffn. */
int moonep_expert_ffn_bwd_data(const moonep_plan_desc* plan, const uint16_t* g_y,
                               const uint16_t* gu, int H, int I, int act, const uint16_t* home_w,
                               const uint16_t* slot_w, int64_t W_el, uint16_t* g_gu,
                               uint16_t* g_recv, hipStream_t stream);

/* Gradient of moonep_expert_ffn with respect to the weights, kept apart for each replica
 * until moonep_reduce_grad adds it to its home (deep dive, section 4, design pattern 3):
 *   gate, up: sum over rows of g_gu[row, :]^T recv[row, :];  down: of g_y[row, :]^T h[row, :]
 * in fp32, over the rows of the group.  home_grad[e] takes expert e's home group and its
 * fallback pieces, which own no slot; rep_grad[r, slot] takes a slot's group.
 *   recv, g_y  device bf16 [R*NvS, H]     h  device bf16 [R*NvS, I]
 *   g_gu       device bf16 [R*NvS, 2*I]   (moonep_expert_ffn_bwd_data's)
 *   home_grad  device fp32 [E, G_el], laid out as the slabs of home_w; G_el >= 3*I*H
 *   rep_grad   device fp32 [R, slots, G_el]; slots no piece uses are not written
 *   accumulate 0: home_grad is overwritten (with zeros for an expert without rows);
 *              1: the sums are added to it.  rep_grad is overwritten either way.
 * Of a slab, the first 3*I*H elements are written.  H and I multiples of 8, G_el of 4; all
 * pointers 16-byte aligned; overlaps as in moonep_expert_ffn.  Deterministic. */
int moonep_expert_ffn_bwd_weight(const moonep_plan_desc* plan, const uint16_t* recv,
                                 const uint16_t* g_y, const uint16_t* h, const uint16_t* g_gu,
                                 int H, int I, float* home_grad, float* rep_grad, int64_t G_el,
                                 int accumulate, hipStream_t stream);

/* The tile that a product of the experts' calls is computed in for these sizes, for
 * profiles and for tests that mean a certain one.  Host only.
 *   product  MOONEP_PRODUCT_*
 *   tile     host int32 [3]: results along an output row (of gate and up, half of them each),
 *            output rows, and 1 where results are written past the caches, else 0
 * Errors of plan, H and I as in moonep_expert_ffn; EINVAL for another product. */
int moonep_expert_tile(const moonep_plan_desc* plan, int H, int I, int product, int32_t tile[3]);

/* The root-mean-square norm in front of the experts, with the residual's addition, over T
 * rows (any T, also 0, when nothing is written):
 *   h = bf16_rne(x + res);  rstd = 1 / sqrt(mean(h^2) + eps);  out = bf16_rne(h * rstd * gamma)
 * The norm is that of h as it is stored; squares are summed in fp32.
 *   x, res  device bf16 [T, H]; res may be NULL (then h = x)
 *   gamma   device bf16 [H]
 *   out     device bf16 [T, H]
 *   h       device bf16 [T, H] or NULL: the residual stream after this addition; may be x or
 *           res itself
 *   rstd    device fp32 [T] or NULL: for the backward pass
 * H % 8 == 0, H <= MOONEP_MAX_NORM, eps >= 0; pointers 16-byte aligned (rstd 4).  Other overlaps
 * of an output with an input or another output are refused (EINVAL). */
int moonep_rmsnorm(const uint16_t* x, const uint16_t* res, const uint16_t* gamma, float eps,
                   int64_t T, int H, uint16_t* out, uint16_t* h, float* rstd, hipStream_t stream);

/* Bytes of a row of H elements in 8 bits: H codes (OCP e4m3), H/32 scales (e8m0: byte b is
 * 2^(b-127)), one for each 32 elements, and zeros up to a multiple of 16.  Host only.
 * EINVAL unless H % 32 == 0; ELIMIT beyond MOONEP_MAX_NORM. */
int64_t moonep_q8_row_bytes(int H);

/* moonep_rmsnorm with its output in 8 bits: rows [T, moonep_q8_row_bytes(H)].  A block's
 * scale is the smallest power of two that brings its largest magnitude to 448 or less, so
 * nothing saturates; an element is rounded once, to nearest even, from fp32.  NaN and
 * infinities become the code NaN in their place.  moonep_dispatch moves such rows as they
 * are: pass them as bf16 rows of moonep_q8_row_bytes(H) / 2 elements; about half of
 * the bytes of bf16 rows.  moonep_q8_unpack expands them on the other side. */
int moonep_rmsnorm_q8(const uint16_t* x, const uint16_t* res, const uint16_t* gamma, float eps,
                      int64_t T, int H, uint8_t* rows, uint16_t* h, float* rstd, hipStream_t stream);

/* Expands N rows in 8 bits (moonep_rmsnorm_q8's, dispatched or not) to bf16 [N, H]:
 * out = code * scale, exact wherever that is a normal bf16 number.  The bytes are taken as
 * they are, so every row may be expanded, mapped or not.  out must not overlap rows (EINVAL). */
int moonep_q8_unpack(const uint8_t* rows, int64_t N, int H, uint16_t* out, hipStream_t stream);

/* Bytes of moonep_rmsnorm_bwd's workspace.  Host only.  Errors as in moonep_rmsnorm. */
int64_t moonep_rmsnorm_bwd_workspace(int64_t T, int H);

/* Backward of the norm, from the h and rstd that the forward call stored:
 *   xhat = h * rstd,  gg = g_out * gamma
 *   g_x = bf16_rne(rstd * (gg - xhat * mean(gg * xhat)) + g_h)    (the gradient of x and of res)
 *   g_gamma = sum over rows of g_out * xhat                       (fp32)
 *   g_out, h   device bf16 [T, H]      gamma  device bf16 [H]     rstd  device fp32 [T]
 *   g_h        device bf16 [T, H] or NULL: the gradient that reaches h past the norm
 *   workspace  device scratch of moonep_rmsnorm_bwd_workspace(T, H) bytes, 256-byte aligned;
 *              calls whose kernels overlap in time must not share one
 *   g_x        device bf16 [T, H], may be g_out, h or g_h itself
 *   g_gamma    device fp32 [H], overwritten (zeros when T is 0)
 * H % 8 == 0, H <= MOONEP_MAX_NORM; pointers 16-byte aligned (rstd 4).  Other overlaps of an output
 * or the workspace with anything else are refused (EINVAL).  EHIP can follow the first of the two
 * launches.  Deterministic. */
int moonep_rmsnorm_bwd(const uint16_t* g_out, const uint16_t* h, const uint16_t* gamma,
                       const float* rstd, const uint16_t* g_h, int64_t T, int H, void* workspace,
                       uint16_t* g_x, float* g_gamma, hipStream_t stream);

/* Weights in 4 bits.  32 neighbours along a matrix row (the last group of a row may be shorter)
 * share a power of two, the smallest from 2^-126 on that brings their largest magnitude to 6
 * or less, and each is an OCP e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6, with a sign) times it,
 * rounded once, to nearest even.  Values that are of this form are kept exactly, so
 * weights that come in it may be packed from their bf16 expansion.  A group with an
 * infinity or a NaN is NaN as a whole.
 * The slab of an expert: its gate, up and down matrices, in an order of the library's own
 * (moonep_w4_unpack reads it back).  moonep_prefetch_weight moves such slabs as they are: pass
 * them as bf16 slabs of W_bytes / 2 elements; W_bytes must then be what both home_w4 and slot_w4
 * are strided by.
 *
 * Bytes of such a slab, a multiple of 256: 17/32 of a byte an element, and what fills up I
 * to 32 (128 in the down matrix) and H to 128.  Host only.  EINVAL unless H and I are positive
 * multiples of 8; ELIMIT beyond MOONEP_MAX_FFN. */
int64_t moonep_w4_slab_bytes(int H, int I);

/* Packs n slabs of bf16 weights, and expands packed ones (exactly).
 *   w    device bf16 [n, W_el]: gate [I, H], up [I, H] and down [H, I] matrices as in
 *        moonep_expert_ffn; W_el >= 3*I*H, a multiple of 8
 *   w4   device [n, W_bytes]; W_bytes >= moonep_w4_slab_bytes(H, I), a multiple of 16
 * What follows a slab up to its pitch is not written.  n may be 0 (then nothing is done).  Both
 * 16-byte aligned; they must not overlap (EINVAL).  Beyond the forward calls below, expanded
 * weights serve moonep_expert_ffn_bwd_data: the gradient of the rows through weights that are
 * kept in 4 bits. */
int moonep_w4_pack(const uint16_t* w, int64_t W_el, int64_t n, int H, int I, uint8_t* w4, int64_t W_bytes,
                   hipStream_t stream);
int moonep_w4_unpack(const uint8_t* w4, int64_t W_bytes, int64_t n, int H, int I, uint16_t* w, int64_t W_el,
                     hipStream_t stream);

/* moonep_expert_ffn with weights in 4 bits (moonep_w4_pack's).  Weights are expanded in registers,
 * exactly; rows, sums and roundings as there.
 *   home_w4  device [E, W_bytes]      slot_w4  device [R, slots, W_bytes]
 * The other arguments, padding rows, overlaps and errors as in moonep_expert_ffn, but for its
 * limit on (I + 256) * H, which does not apply; W_bytes as in moonep_w4_pack. */
int moonep_expert_ffn_w4(const moonep_plan_desc* plan, const uint16_t* recv, int H, int I, int act,
                         const uint8_t* home_w4, const uint8_t* slot_w4, int64_t W_bytes, uint16_t* gu,
                         uint16_t* h, uint16_t* y, hipStream_t stream);

/* moonep_expert_ffn with weights in 4 bits and rows in 8: both are multiplied as they are.
 *   rows  device [R*NvS, moonep_q8_row_bytes(H)]: moonep_rmsnorm_q8's rows, dispatched
 *   h     device [R*NvS, moonep_q8_row_bytes(I)]: scratch.  h = act(gate) * up is rounded from
 *         fp32 to 8 bits by moonep_rmsnorm_q8's rule, once
 *   y     device bf16 [R*NvS, H]
 * The matrix units multiply exactly and add each four neighbours along k with what lies 13 bits
 * below the largest one's power of two cut off, then in fp32: y and h are off by up to 3 * 2^-13 of
 * the sum of the products' magnitudes for it (1e-4 of y for products of either sign, a twentieth
 * of its rounding).  A scale byte of 255, and the code NaN, make NaN of what they are in.
 * H and I are multiples of 32 (EINVAL).  For serving: nothing is saved for a backward pass.  Other
 * arguments and errors as in moonep_expert_ffn_w4. */
int moonep_expert_ffn_w4q8(const moonep_plan_desc* plan, const uint8_t* rows, int H, int I, int act,
                           const uint8_t* home_w4, const uint8_t* slot_w4, int64_t W_bytes, uint8_t* h,
                           uint16_t* y, hipStream_t stream);

/* The tile that a product of these two calls is computed in for these sizes, for profiles and for tests that mean a
 * certain one.  Host only.
 *   rows_q8  0: moonep_expert_ffn_w4; 1: moonep_expert_ffn_w4q8
 *   product  MOONEP_PRODUCT_GATE_UP or MOONEP_PRODUCT_DOWN (EINVAL for others)
 *   tile     host int32 [2]: weight rows (of gate and up, half of them each), buffer rows
 * Errors of plan, H and I as in the calls. */
int moonep_expert_tile_w4(const moonep_plan_desc* plan, int H, int I, int rows_q8, int product, int32_t tile[2]);

/* The router in front of the plan, over T tokens (any T, also 0, when nothing is written): what it
 * writes is what moonep_plan takes.
 *   s = softmax(l) or sigmoid(l) of a token's E logits;  key = s + bias
 *   The experts are in `groups` groups of E / groups neighbours.  A group's score is the sum of its
 *   two largest keys; the top_groups best groups are kept (1 of 1: all experts).
 *   topk_ids  the K experts of these groups with the largest keys, largest first
 *   topk_w    scale * s of each (fp32, without the bias), divided by their sum if normalize is 1
 * Equal keys and equal group scores go to the lowest index.  Keys are compared in 64 bits; without a bias and groups
 * the logits are compared, which is their order.
 * A logit of -inf or NaN masks its expert: its score is 0, whatever its bias, and it is chosen only
 * where a token has fewer than K others, the lowest index first, with weight 0 (all weights are 0 for a
 * token without any); a group's score leaves it out, and is -inf if nothing else is there.  A bias of
 * -inf or NaN does the same to the choice, one of +inf puts its expert, and its group, first.  A logit of +inf counts as
 * the largest fp32 number.
 *   logits    device fp32 (dtype MOONEP_F32) or bf16 (MOONEP_BF16) [T, E]
 *   bias      device fp32 [E] or NULL: moves the choice, not the weights
 *   score     MOONEP_SCORE_*          scale  finite
 *   topk_ids  device int32 [T, K]     topk_w  device fp32 [T, K]
 * 1 <= K <= E, E % groups == 0, 1 <= top_groups <= groups, top_groups * (E / groups) >= K; E, K and groups at
 * most MOONEP_MAX_E, MOONEP_MAX_K and MOONEP_MAX_GROUPS; pointers aligned to their elements.  Outputs must not overlap
 * anything else (EINVAL).  Deterministic. */
int moonep_router(const void* logits, int dtype, const float* bias, int64_t T, int E, int K, int score, int groups,
                  int top_groups, int normalize, float scale, int32_t* topk_ids, float* topk_w, hipStream_t stream);

/* Backward of the router: the logits' gradient from that of the weights (moonep_combine_bwd's dw), with
 * the choice held fixed.  With g = scale * g_w and, over a token's K experts, p = s / sum(s):
 *   normalised   p (g - sum(g p)), for the sigmoid times 1 - s
 *   else         sigmoid: g s (1 - s);  softmax: s (g - sum(g s)), and -s sum(g s) of the logits not chosen
 * and zero for the other logits, all in fp32, rounded to the logits' type once.  Masked experts (logits of -inf or
 * NaN) have a gradient of zero; an id outside [0, E) brings nothing; one named twice brings both.
 *   g_w       device fp32 [T, K]      g_logits  device [T, E], of the logits' type
 * The other arguments, and errors, as in moonep_router.  Deterministic. */
int moonep_router_bwd(const void* logits, int dtype, const int32_t* topk_ids, const float* g_w, int64_t T, int E,
                      int K, int score, int normalize, float scale, void* g_logits, hipStream_t stream);

/* Waits for `stream`, then copies the plan's statistics to the host.  The only call
 * that synchronises: the hot path itself never reads the plan back ("MoonshotAI/MoonEP
 * 딥다이브", section 2, point 3: static buffers remove the per-layer host sync), so data
 * errors found on the device (status 1: an expert id outside [0, E); status 2: an
 * internal invariant of the plan failed) are reported here, when the caller asks, and
 * meanwhile make the plan map nothing. */
int moonep_plan_status(const moonep_plan_desc* plan, moonep_plan_stats* out,
                       hipStream_t stream);

const char* moonep_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif /* MOONEP_H_ */
