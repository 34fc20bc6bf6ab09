/*
 * psispec.h -- C ABI of the Psi-Spec verify step on MI355X (gfx950).
 *
 * The verify step of Uno's Psi-Spec sampler: a frozen AR model has scored a block of B drafted
 * tokens (plus the row after the block) in one pass; the verifier applies an acceptance test to the
 * drafts in order, keeps the longest accepted run from the start, draws a replacement token from a
 * corrected residual distribution at the first rejection and discards the rest, or draws one extra
 * token from the block-end row when every draft passes.  Sources, cited by page title and section:
 *
 *   [alphalab] "Uno Ψ-Spec 是什麼？Diffusion-Augmented LLM 如何保留 AR 分布、一次驗證多個 Token":
 *              §"Uno Ψ-Spec 怎麼運作？完整走一次四個 Token" (steps 1-4 and the full-accept paragraph),
 *              §"為什麼 lossless 不等於答案完全一樣？" (the output law equals the AR's),
 *              §"Linear 與 Tree sampler" (one candidate per position vs a pruned prefix tree).
 *   [lanes]    "Uno / Ψ-Spec — 같은 모델 안에서 초안 뽑고 AR로 도장 찍기":
 *              §"Ψ-Spec이 한 스텝에서 하는 일" (frozen AR verifies, longest prefix kept),
 *              §"어디서 왔나" (speculative sampling of Leviathan et al. 2023 as the lineage).
 *
 * The pages print no formula.  The rule implemented is the speculative-sampling rule of that
 * lineage: accept draft d at position i when u_i < min(1, p'_i(d) / q'_i(d)); at the first rejected
 * position k draw from max(0, p'_k - q'_k) renormalised; after a full accept draw from p'_B.  p' and
 * q' are softmax(logits / temperature), optionally truncated to the tie-inclusive nucleus of mass
 * top_p and renormalised.  Uniforms come from Philox4x32-10 (Salmon et al., SC'11) with key = seed
 * and counter = (request_base + request, position, purpose, step); u = top 53 bits of
 * (word0 << 32 | word1) times 2^-53.  Purposes: 0 = accept test, 1 = final draw, 2 = drafting.
 *
 * Conventions shared by every entry point:
 *   - Tensor pointers are DEVICE pointers owned by the caller; rows are contiguous with V elements.
 *     The library never allocates or frees: its scratch lives in the caller's `workspace`
 *     (device memory, >= the size returned by the matching *_workspace query, 256-byte aligned).
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = the default stream), never
 *     synchronise the host, and are reentrant.  Concurrent calls need distinct workspaces.
 *     Outputs are a pure function of the inputs and (seed, step, request_base): reruns are bitwise
 *     identical.
 *   - Host-detectable errors (null pointers, bad sizes, temperature <= 0 or not finite, top_p
 *     outside (0, 1], bad dtype, small workspace) return a negative code and launch nothing;
 *     a failed launch returns PSISPEC_EHIP.
 *   - Data errors found on the device never abort: they set bits in status[request] and leave that
 *     request's other outputs unspecified (but in bounds).  When an input error is flagged
 *     (NONFINITE, BAD_TOKEN, BAD_PARENT) the remaining status bits are unspecified as well.
 */
#ifndef PSISPEC_H
#define PSISPEC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PSISPEC_OK = 0,
  PSISPEC_EINVAL = -1,       /* bad pointer, size or sampling parameter */
  PSISPEC_EDTYPE = -2,       /* unsupported element type */
  PSISPEC_EWORKSPACE = -3,   /* workspace missing, too small or misaligned */
  PSISPEC_EHIP = -4,         /* a HIP call or kernel launch failed */
  PSISPEC_EUNSUPPORTED = -5, /* a mode that is not implemented */
  PSISPEC_ESCRATCH = -6      /* sizes beyond the fixed scratch of the no-allocation entry point */
} psispec_status;

/* Logits are F32 or BF16.  The paged-cache calls take queries, keys and values in BF16 or F16 and
   caches in their type or in F8E4M3 (8 bits: 4 exponent, 3 mantissa; no infinities, largest 448).
   E8M0 is a power of two as a scale: byte e stands for 2^(e - 127), 255 for NaN. */
typedef enum {
  PSISPEC_F32 = 0,
  PSISPEC_BF16 = 1,
  PSISPEC_F16 = 2,
  PSISPEC_F8E4M3 = 3,
  PSISPEC_E8M0 = 4
} psispec_dtype;

/* flags */
#define PSISPEC_FIRST_FROM_TARGET 1u /* Uno layout: position 0 is the AR's own sample and is always
                                        kept ([alphalab] walkthrough step 1); q row 0 is not read */
/* Tree verify with q_logits only: PSISPEC_MAX_CHILDREN(k), 1 <= k <= 8, says that no node has more
   than k children (the drafter's branching), so the residual chain is built for k children only
   and its passes for more are not launched.  A node with more than k children is then reported
   with PSISPEC_ST_BAD_PARENT.  0 (not given) means 8.  Every other call rejects these bits. */
#define PSISPEC_MAX_CHILDREN_SHIFT 4
#define PSISPEC_MAX_CHILDREN_MASK (0xfu << PSISPEC_MAX_CHILDREN_SHIFT)
#define PSISPEC_MAX_CHILDREN(k) ((uint32_t)(k) << PSISPEC_MAX_CHILDREN_SHIFT)

/* per-request status bits */
#define PSISPEC_ST_NONFINITE 1   /* a row read by the request holds NaN/+Inf or no finite logit */
#define PSISPEC_ST_BAD_TOKEN 2   /* a drafted / node token outside [0, V) */
#define PSISPEC_ST_Q_ZERO 4      /* the draft probability of a drafted token is 0 (ratio set to
                                    1 if the target probability is positive, else 0) */
#define PSISPEC_ST_RESID_ZERO 8  /* residual mass 0 at a rejection: drew from the target row */
#define PSISPEC_ST_BAD_PARENT 16 /* tree: parent[j] outside [-1, j-1] or depth beyond max_depth */
#define PSISPEC_ST_BAD_KEEP 32   /* KV commit: kept count, kept positions or length invalid */
#define PSISPEC_ST_BAD_PAGE 64   /* paged cache: length, row count, source line or a page that the
                                    call needs is invalid */
#define PSISPEC_ST_NO_PAGE 128   /* psispec_pages_reserve: not enough free pages for the line */

typedef struct {
  double temperature;    /* > 0 and finite: logits are divided by it */
  double top_p;          /* (0, 1]; 1 disables the nucleus truncation */
  uint64_t seed;         /* Philox key */
  uint32_t step;         /* Philox counter word 3 */
  uint32_t request_base; /* global id of request 0 (counter word 0 = request_base + request) */
  uint32_t flags;        /* PSISPEC_FIRST_FROM_TARGET, PSISPEC_MAX_CHILDREN(k) or 0 */
  uint32_t reserved;     /* must be 0 */
} psispec_sampling;

/*
 * Linear verify ([alphalab] §"Linear 與 Tree sampler": one candidate per position;
 * walkthrough steps 3-4 and the full-accept paragraph).
 *
 *   p_logits     [batch][B+1][V]  target (AR) logits; row i scores draft i, row B is the block end
 *   q_logits     [batch][B][V]    draft logits; row i is the distribution draft i was drawn from
 *   dtype        element type of p_logits and q_logits (PSISPEC_F32 or PSISPEC_BF16)
 *   draft_tokens [batch][B] int32 drafted tokens
 *   B            1..64;  V >= 1;  batch >= 0 (0 launches nothing)
 *   s            host pointer to the sampling parameters
 * Outputs (device):
 *   accept_len   [batch] int32    k = number of leading drafts kept, in [0, B]
 *   out_tokens   [batch][B+1]     d_0..d_{k-1}, then the correction (k < B) or bonus (k = B) token,
 *                                 then -1; k+1 tokens are committed
 *   ratios       [batch][B] f32   min(1, p'_i(d_i)/q'_i(d_i)) for every i (also past k); nullable
 *   accept_mask  [batch] u64      bit i set when u_i < ratio_i (every i); nullable
 *   status       [batch] int32    PSISPEC_ST_* bits; nullable
 */
size_t psispec_verify_linear_workspace(int32_t batch, int32_t B, int32_t V, psispec_dtype dtype);

psispec_status psispec_verify_linear(const void* p_logits, const void* q_logits, psispec_dtype dtype,
                                     const int32_t* draft_tokens, int32_t batch, int32_t B,
                                     int32_t V, const psispec_sampling* s, int32_t* accept_len,
                                     int32_t* out_tokens, float* ratios, uint64_t* accept_mask,
                                     int32_t* status, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * Linear verify for callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): psispec_verify_linear with the same
 * arguments, outputs, determinism and errors, but no workspace argument.  Its scratch is a fixed
 * 64 MiB array in device memory that the library holds on every GPU it runs on until the process
 * ends; the call allocates nothing.  Sizes whose workspace (psispec_verify_linear_workspace)
 * exceeds 64 MiB return PSISPEC_ESCRATCH and launch nothing (batch 256 fits at any B up to 64
 * and V up to 262,144; batch 512 at B = 8, V = 151,936 does not).  Every call on one GPU uses the
 * same array: calls that overlap on one GPU (two streams, two host threads) race and must be
 * ordered by the caller.  Nothing in the array needs to start at zero; it keeps the last call's
 * contents.  (While psispec_timing_enable is on, the library's timing hooks create HIP events.)
 */
psispec_status psispec_verify_linear_noalloc(const void* p_logits, const void* q_logits,
                                             psispec_dtype dtype, const int32_t* draft_tokens,
                                             int32_t batch, int32_t B, int32_t V,
                                             const psispec_sampling* s, int32_t* accept_len,
                                             int32_t* out_tokens, float* ratios,
                                             uint64_t* accept_mask, int32_t* status, void* stream);

/*
 * Tree verify ([alphalab] §"Linear 與 Tree sampler": several likely candidates per position,
 * pruned to a finite prefix tree verified at once).  The rule for candidates chosen
 * deterministically (e.g. top-k of the draft): at node v, children are tried in ascending node
 * index; child c is kept when u_c < res(tok_c) / R, where res is p'_v with the tokens of the
 * already rejected siblings removed and R = 1 - their mass; a rejected child's token is removed
 * from res; when no child is kept (or v is a leaf) one token is drawn from res.  Node ratios are
 * computed for every node as if all its earlier siblings were rejected.
 *
 * With q_logits (candidates drawn from the draft), the rule is recursive rejection: at node v the
 * children were drawn independently from q'_v, in ascending node index; child i is kept when
 * u < min(1, r_{i-1}(tok) / q'_v(tok)), r_0 = p'_v, and a rejection replaces the residual by
 * max(0, r_{i-1} - q'_v) renormalised; with no child kept one token is drawn from the last
 * residual.  At most 8 children per node (PSISPEC_ST_BAD_PARENT otherwise).
 *
 *   p_logits     [batch][N+1][V]  row 0 = root, row j+1 = node j
 *   q_logits     NULL (candidates chosen, e.g. top-k of the draft), or [batch][N+1][V] draft logits
 *                whose row v+1 (row 0: the root) is the distribution node v's children were drawn
 *                from (the tree's shape must not depend on the drawn tokens)
 *   parent       [batch][N] int32 parent node of node j, -1 = root, must be < j
 *   node_tokens  [batch][N] int32 token of node j
 *   N            1..1024 nodes per request;  V >= 1;  batch >= 0 (0 launches nothing)
 *   max_depth    bound on the depth of any node (1..64)
 * Uniforms: node c's test at (request, c+1, accept); the final draw at (request, row, draw) where
 * row is the stopping node's row.
 * Outputs (device):
 *   accept_len   [batch] int32            depth of the kept path
 *   accept_nodes [batch][max_depth]       the kept nodes in order, then -1
 *   out_tokens   [batch][max_depth+1]     their tokens, then the drawn token, then -1
 *   node_ratios  [batch][N] f32           nullable
 *   status       [batch] int32            nullable
 * The workspace query covers both rules.
 */
size_t psispec_verify_tree_workspace(int32_t batch, int32_t N, int32_t V, psispec_dtype dtype);

psispec_status psispec_verify_tree(const void* p_logits, const void* q_logits, psispec_dtype dtype,
                                   const int32_t* parent, const int32_t* node_tokens, int32_t batch,
                                   int32_t N, int32_t V, int32_t max_depth,
                                   const psispec_sampling* s, int32_t* accept_len,
                                   int32_t* accept_nodes, int32_t* out_tokens, float* node_ratios,
                                   int32_t* status, void* workspace, size_t workspace_bytes,
                                   void* stream);

/*
 * Drafting step ([alphalab] walkthrough steps 1-2: the AR path samples the first token of the
 * block, the diffusion path proposes the others in parallel).  Draws d_0..d_{B-1} of every request,
 * each from its row after the transform the verify applies (softmax(logits / temperature), then the
 * nucleus of mass top_p, renormalised): the verify is lossless only for drafts drawn from exactly
 * that q'.  Each draw is an inverse CDF by ascending token id with the Philox uniform of
 * (request_base + request, i, purpose 2 = draft, step), decided as in exact arithmetic: an fp32 pass
 * with a rigorous error bound settles a draw when the bound cannot change it, the others are drawn
 * in fp64 like the verify's final draw.
 *
 *   ar_logits    AR rows, read only with PSISPEC_FIRST_FROM_TARGET (may be NULL otherwise): the row
 *                of request r starts at element r * ar_stride; d_0 is drawn from it.  ar_stride >= V
 *                ((B+1)*V reads row 0 of the verify's p_logits [batch][B+1][V]; V reads packed
 *                [batch][V] rows)
 *   q_logits     [batch][B][V] draft rows; d_i is drawn from row i.  With PSISPEC_FIRST_FROM_TARGET
 *                row 0 is not read, and q_logits may be NULL when B = 1
 *   dtype        element type of ar_logits and q_logits (PSISPEC_F32 or PSISPEC_BF16)
 *   B            1..64;  V >= 1;  batch >= 0 (0 launches nothing)
 *   s            host pointer to the sampling parameters (the verify's temperature and top_p)
 * Outputs (device):
 *   draft_tokens [batch][B] int32   in [0, V)
 *   status       [batch][B] int32   PSISPEC_ST_NONFINITE when the row holds NaN/+Inf or no finite
 *                                   logit (that token is then unspecified); nullable
 * Rows that are 16-byte aligned with V * element size and ar_stride * element size multiples of 16
 * are read with 16-byte loads; any other layout is read element by element.
 */
size_t psispec_sample_drafts_workspace(int32_t batch, int32_t B, int32_t V, psispec_dtype dtype);

psispec_status psispec_sample_drafts(const void* ar_logits, int64_t ar_stride,
                                     const void* q_logits, psispec_dtype dtype, int32_t batch,
                                     int32_t B, int32_t V, const psispec_sampling* s,
                                     int32_t* draft_tokens, int32_t* status, void* workspace,
                                     size_t workspace_bytes, void* stream);

/*
 * KV commit after a verify ([lanes] §"헤드냐, LoRA냐": drafting and verifying share one KV line per
 * sequence, the AR verifies and appends; [alphalab] walkthrough step 4: the accepted prefix is kept,
 * the rest is discarded and drafted again).  The verify forward has written the KV rows of the
 * block's blk positions at positions len[r] .. len[r]+blk-1 of line r.  The kept rows, block
 * positions keep[r][0..n_keep[r]-1], move to len[r] .. len[r]+n_keep[r]-1 in that order and
 * len[r] grows by n_keep[r]; the rows past the new length are free (rolled back, untouched).
 *
 *   kv           device; line r starts at kv + r * line_stride bytes, position t at
 *                + t * row_bytes; rows are opaque bytes (any layout of layers, heads and K/V)
 *   line_stride  bytes, multiple of 16, >= Lmax * row_bytes
 *   row_bytes    bytes per position, a multiple of 16;  kv 16-byte aligned
 *   Lmax         positions per line;  blk: 1..min(Lmax, 1024) block positions
 *   keep         [batch][keep_stride] int32 kept block positions, strictly increasing in [0, blk)
 *                (the tree verify's accept_nodes as they are, keep_stride = max_depth), or NULL:
 *                the first n_keep positions (the linear verify: nothing moves)
 *   n_keep       [batch] int32 in [0, blk] (and <= keep_stride): the verify's accept_len
 *   len          [batch] int32, in/out, with len + blk <= Lmax
 *   status       [batch] int32, nullable: PSISPEC_ST_BAD_KEEP when n_keep, keep or len is invalid;
 *                that request's line and length are then left unchanged
 * Asynchronous on `stream`; no workspace.  Host-detectable errors return PSISPEC_EINVAL.
 */
psispec_status psispec_kv_commit(void* kv, int64_t line_stride, int64_t row_bytes, int32_t Lmax,
                                 int32_t blk, const int32_t* keep, int32_t keep_stride,
                                 const int32_t* n_keep, int32_t* len, int32_t* status,
                                 int32_t batch, void* stream);

/*
 * LM head + linear verify ([lanes] §"헤드냐, LoRA냐": the draft path is the frozen AR weights plus a
 * low-rank LoRA delta; [alphalab] walkthrough steps 2-3: the draft rows go through the LoRA path, the
 * AR path scores the block).  Computes, on the bf16 matrix cores with fp32 accumulation,
 *   p logits (AR rows)    = h_ar . W
 *   q logits (draft rows) = h_draft . W + lora_scale (h_draft . A) . B
 * and runs the linear verify on them (same sampling, outputs, statuses and Philox keys as
 * psispec_verify_linear on those fp32 logits).  The logits are not written to memory: the matrix
 * product's epilogue hands the verify each row's softmax statistics and the logit at each draft
 * token, and the one or two rows that the final draw reads (p_k and q_k at the first rejection k,
 * or the block-end row p_B) are recomputed, bit-identical, into the workspace.
 *
 *   h_ar      bf16 [batch][B+1][H]  final hidden states of the AR rows (row B = block end)
 *   h_draft   bf16 [batch][B][H]    final hidden states of the draft rows
 *   W         bf16 [H][V]           the LM-head weight (V contiguous)
 *   lora_A    bf16 [H][r]           the LoRA down-projection; NULL when r = 0
 *   lora_B    bf16 [r][V]           the LoRA up-projection (V contiguous); NULL when r = 0
 *   H         multiple of 64, at most 2^20;  V multiple of 8;  0 <= r <= 64;  B 1..64
 *   p_logits_dbg, q_logits_dbg
 *             fp32 [batch][B+1][V] and [batch][B][V], or both NULL (the logits are never
 *             materialised).  When given, the logits are also stored there and the final draw
 *             reads them instead of recomputing its rows.  With top_p < 1 both are required (the
 *             nucleus needs every row's values a second time): PSISPEC_EUNSUPPORTED otherwise.
 * h_ar, h_draft, W, lora_B and the logit buffers must be 16-byte aligned (PSISPEC_EINVAL
 * otherwise).  All inputs are read-only and caller-owned; the call is asynchronous on `stream`.
 * The product h_draft . A is formed in fp64 and enters the matrix product as a bf16 pair
 * (hi + lo, relative error 2^-17).
 */
size_t psispec_lmhead_verify_workspace(int32_t batch, int32_t B, int32_t H, int32_t V, int32_t r);

psispec_status psispec_lmhead_verify(const void* h_ar, const void* h_draft, const void* W,
                                     const void* lora_A, const void* lora_B, float lora_scale,
                                     int32_t batch, int32_t B, int32_t H, int32_t V, int32_t r,
                                     const int32_t* draft_tokens, const psispec_sampling* s,
                                     int32_t* accept_len, int32_t* out_tokens, float* ratios,
                                     uint64_t* accept_mask, int32_t* status, float* p_logits_dbg,
                                     float* q_logits_dbg, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * Paged KV cache.  Instead of one contiguous line per sequence (psispec_kv_commit), the lines of
 * all sequences share a pool of pages of page_size positions each; table[r][s] is the page that
 * holds positions s * page_size .. (s + 1) * page_size - 1 of line r, or -1.  The verify forward's
 * path over it: psispec_pages_reserve gives every line pages for its next block,
 * psispec_qkv_append writes the block's rows at positions len[r] .. len[r]+n-1,
 * psispec_paged_attention reads them, psispec_paged_commit keeps the accepted ones and advances
 * len, psispec_pages_assign forks, cuts and frees lines.  A status lies apart from the lengths, counts
 * and tables that its call reads (PSISPEC_EINVAL otherwise).
 *
 * One layer's keys and values as the append and the attention see them.  Element (page p, offset o,
 * head h, dimension d) of K is k[p * page_stride + o * row_stride + h * head_stride + d], of V the
 * same from v: any order of pages, positions and heads, for example views into a pool that holds
 * every layer.  Bases 16-byte aligned and strides multiples of 16 bytes.
 */
typedef struct {
  void* k;                /* device; the attention only reads both */
  void* v;
  const float* k_scale;   /* device [heads], F8E4M3 caches only: a stored number x stands for */
  const float* v_scale;   /* x * scale[head]; NULL means 1 */
  const int32_t* table;   /* device [batch][table_stride], the first `slots` entries of a row used */
  int64_t page_stride;    /* elements */
  int64_t row_stride;     /* elements */
  int64_t head_stride;    /* elements */
  int64_t table_stride;   /* entries, >= slots */
  int32_t num_pages;      /* >= 1: valid page ids are 0 .. num_pages-1 */
  int32_t page_size;      /* positions per page, 1..4096 */
  int32_t slots;          /* >= 1 and slots * page_size <= 2^30 */
  int32_t heads;          /* key/value heads, >= 1 */
  int32_t dim;            /* head dimension, a multiple of 16, 16..256 */
  int32_t dtype;          /* psispec_dtype: the calls' element type or PSISPEC_F8E4M3 */
} psispec_paged_cache;

/* Norm and position rotation of psispec_qkv_append. */
#define PSISPEC_ROPE_INTERLEAVED 1u /* pairs are dimensions (2j, 2j+1); else (j, j + rot/2) */
typedef struct {
  const void* q_weight;   /* device [dim] of the call's dtype: norm weight of the query heads, or
                             NULL: queries are not normalised */
  const void* k_weight;   /* the same for the key heads */
  const double* inv_freq; /* device [rot/2]: angle per position of pair j (the long-context scalings
                             are other frequencies, and rope_scale); NULL only when rot = 0 */
  double eps;             /* >= 0, finite in 32 bits: added to the mean square */
  double rope_scale;      /* finite in 32 bits: the rotated pairs are multiplied by it */
  int32_t rot;            /* leading dimensions that are rotated: a multiple of 16, 0..dim */
  uint32_t flags;         /* PSISPEC_ROPE_INTERLEAVED or 0 */
} psispec_qkv_prep;

/*
 * The block's queries, keys and values, normalised, rotated and written where the attention reads
 * them, in one pass:
 *   x = x / sqrt(mean(x^2) + eps) * weight              (query and key heads with a weight)
 *   (a, b) = rope_scale (a cos t - b sin t, b cos t + a sin t), t = position * inv_freq[j]
 *                                                       (pair j of the first rot dimensions)
 * in 32 bits with the angles formed and reduced in 64, rounded once to the output's type.  Queries
 * go to q_out, keys and values to the cache at positions len[r] .. len[r]+n-1 of line r, n =
 * n_new[r] (blk when NULL).  An 8-bit cache stores x / scale[head], clamped to +-448 and rounded to
 * the nearest (NaN stays NaN).
 *   c          host pointer; heads and dim are those of k and v
 *   p          host pointer
 *   q, k, v    row (r, i) at (r * blk + i) * stride elements: heads_q (q) or c->heads (k, v) heads of
 *              dim contiguous elements; dtype PSISPEC_BF16 or PSISPEC_F16.  Views into one packed
 *              projection are fine; pointers 16-byte aligned, strides multiples of 8 elements
 *   positions  [batch][blk] int32 rotation position of each row (a tree's len + depth; any value),
 *              or NULL: len[r] + i
 *   len        [batch] int32 rows that the line holds already
 *   n_new      [batch] int32 in [0, blk], or NULL: rows i >= n_new[r] have no effect and are not
 *              written
 *   q_out      row (r, i) at (r * blk + i) * q_out_stride; may be q itself with q_stride, and
 *              overlaps no input otherwise (PSISPEC_EINVAL when it lies over q, k, v or the cache)
 *   status     [batch] int32, nullable: PSISPEC_ST_BAD_PAGE when len < 0, n_new is outside [0, blk]
 *              or the rows do not fit the slots (nothing of the line is then written, q_out
 *              included), or when a page of the rows is not in 0..num_pages-1 (the rows on such a
 *              page are then not written, q_out included)
 *   blk 1..2^20;  batch >= 0 (0 launches nothing), batch * blk < 2^24;  heads_q 1..1024
 * No two (page, position, head) of the cache share an element, nor do K and V (PSISPEC_EINVAL).  The
 * pages written must be the line's own (psispec_pages_reserve sees to it): rows of two lines in one
 * page position race.  The inputs q, k and v lie outside the cache, but for rows of k or v that are
 * already in the very places that they go to, in a cache of their type.
 * Asynchronous on `stream`; no workspace.
 */
psispec_status psispec_qkv_append(const psispec_paged_cache* c, const psispec_qkv_prep* p,
                                  const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                  const void* v, int64_t v_stride, psispec_dtype dtype,
                                  int32_t batch, int32_t blk, int32_t heads_q,
                                  const int32_t* positions, const int32_t* len,
                                  const int32_t* n_new, void* q_out, int64_t q_out_stride,
                                  int32_t* status, void* stream);

/*
 * Attention of the block's queries over the paged cache: one new token per line (blk = 1) or the
 * drafted block of a verify forward.  Row i of line r sees the line's first len[r] positions and, of
 * the block's rows (which the cache already holds at len[r] ..), rows 0..i (parent NULL) or row i
 * and its ancestors in the tree:
 *   out = sum_t w_t v_t / sum_t w_t,   w_t = exp(scale * q . k_t)   over the positions t that it sees
 * Query heads share key/value heads in groups: head h reads key/value head h / (heads_q / heads).
 * Products of the matrix cores in the inputs' type with 32-bit sums; softmax statistics in 32 bits;
 * weights enter the second product as a pair of 16-bit numbers with a relative error of 2^-16, so out
 * is as exact as its own rounding.  What the pairs' range leaves out is at most 2^-26 of the largest
 * |v| for an F16 cache (half of F16's smallest number for values up to 2), 2^-96 of it otherwise.  A
 * position that a row does not see has no effect on it, whatever the cache holds there.  Infinities
 * among what it sees give infinities or NaN.
 *   q, out     row (r, i) at (r * blk + i) * stride elements: heads_q heads of c->dim contiguous
 *              elements; dtype PSISPEC_BF16 or PSISPEC_F16; 16-byte aligned, strides multiples of 8;
 *              out overlaps no input (PSISPEC_EINVAL when it lies over q or the cache)
 *   parent     [batch][blk] int32: the block row that row j follows, -1 = the line's last position;
 *              must be < j.  NULL: row j follows row j-1
 *   len, n_new as in psispec_qkv_append; rows i >= n_new[r] of out are left as they are
 *   scale      finite, in 32 bits and times log2 e
 *   status     [batch] int32, nullable: PSISPEC_ST_BAD_PAGE as in psispec_qkv_append, for every page
 *              of the line's first len + n_new positions; PSISPEC_ST_BAD_PARENT.  Out rows of such a
 *              line are unspecified, other lines are not affected
 *   blk 1..1024;  batch 0..2^24-1 (0 launches nothing);  heads_q a multiple of c->heads, at most 1024
 * The work is cut into equal shares over the whole batch by the lines' lengths, read on the device,
 * and rows cut by a share's border are joined in a fixed order: reruns are bitwise identical.
 */
size_t psispec_paged_attention_workspace(int32_t batch, int32_t blk, int32_t heads_q,
                                         int32_t heads_kv, int32_t dim);

psispec_status psispec_paged_attention(const psispec_paged_cache* c, const void* q, int64_t q_stride,
                                       psispec_dtype dtype, int32_t batch, int32_t blk,
                                       int32_t heads_q, const int32_t* parent, const int32_t* len,
                                       const int32_t* n_new, double scale, void* out,
                                       int64_t out_stride, int32_t* status, void* workspace,
                                       size_t workspace_bytes, void* stream);

/*
 * A pool of pages as the calls that move rows see it: `planes` planes (layers, K and V, or whatever
 * lies apart), each num_pages pages of page_size rows of row_bytes opaque bytes.  Row o of page p of
 * plane w starts at base + w * plane_stride + p * page_stride + o * row_bytes.
 */
typedef struct {
  void* base;             /* device, 16-byte aligned */
  int64_t plane_stride;   /* bytes, a multiple of 16; planes do not overlap */
  int64_t page_stride;    /* bytes, a multiple of 16, >= page_size * row_bytes */
  int64_t row_bytes;      /* a multiple of 16, >= 16 */
  int32_t planes;         /* >= 1 */
  int32_t num_pages;      /* >= 1 */
  int32_t page_size;      /* 1..4096 */
  int32_t reserved;       /* must be 0 */
} psispec_page_pool;

/*
 * psispec_kv_commit for lines in pages: the kept rows, block positions keep[r][0..n_keep[r]-1], move
 * to positions len[r] .. len[r]+n_keep[r]-1 of line r, in every plane, and new_len[r] becomes
 * len[r] + n_keep[r].  Pages that the block needed stay with the line for its next block.
 *   table      [batch][table_stride] int32, the first `slots` entries of a row used
 *   blk, keep, keep_stride, n_keep   as in psispec_kv_commit (blk 1..1024); of a line whose block was
 *              shorter (n_new) keep names rows of that block: which rows were written is not known here
 *   len        [batch] int32; the line's first len rows and the kept ones lie within slots * page_size
 *              positions (all blk rows need not: a short block may end where the table does)
 *   new_len    [batch] int32; len itself, or apart from every input (PSISPEC_EINVAL otherwise)
 *   status     [batch] int32, nullable: PSISPEC_ST_BAD_KEEP as in psispec_kv_commit,
 *              PSISPEC_ST_BAD_PAGE when a page of the rows that move is not in 0..num_pages-1;
 *              nothing of such a line moves and its length stays
 * Asynchronous on `stream`; no workspace.
 */
psispec_status psispec_paged_commit(const psispec_page_pool* pool, const int32_t* table,
                                    int64_t table_stride, int32_t slots, int32_t batch, int32_t blk,
                                    const int32_t* keep, int32_t keep_stride, const int32_t* n_keep,
                                    const int32_t* len, int32_t* new_len, int32_t* status,
                                    void* stream);

/*
 * Owners of pages.  refs[p] counts the table entries of all lines that name page p; a page with
 * count 0 is free.  All lines that share a pool are rows of one table.  An empty pool has refs all
 * 0, tables all -1 and lengths 0.
 *
 * psispec_pages_assign makes every line r a copy of the first new_len[r] positions of the line
 * src[r] as it was before the call, by sharing its pages (no row moves): src[r] = r and new_len[r] =
 * len[r] keeps a line, a smaller new_len cuts it, src[r] = -1 or new_len 0 frees it, another line
 * forks that line (any number of lines from one; a beam's reorder is one call).  Slots past
 * ceil(new_len / page_size) become -1, those reserved for a block included.  Pages that no line
 * holds any more are free from then on.
 *   table      [batch][table_stride] int32, in/out
 *   refs       [num_pages] int32, in/out
 *   len        [batch] int32, in/out
 *   src        [batch] int32 in [-1, batch)
 *   new_len    [batch] int32 in [0, len[src]] (ignored when src = -1)
 *   status     [batch] int32, nullable: PSISPEC_ST_BAD_PAGE when src, new_len or a page of the
 *              positions taken is invalid; that line then stays as it is
 */
size_t psispec_pages_workspace(int32_t batch, int32_t slots, int32_t num_pages, int32_t blk,
                               int32_t page_size);

psispec_status psispec_pages_assign(int32_t* table, int64_t table_stride, int32_t slots,
                                    int32_t* refs, int32_t num_pages, int32_t page_size,
                                    int32_t* len, const int32_t* src, const int32_t* new_len,
                                    int32_t* status, int32_t batch, void* workspace,
                                    size_t workspace_bytes, void* stream);

/*
 * psispec_pages_reserve gives every line pages of its own for positions len[r] .. len[r]+n-1, n =
 * n_new[r] (blk when NULL): slots without a page get the lowest-numbered free pages in the order
 * of lines and slots, and a page among them that other lines hold too is replaced by a free one, the
 * line's rows before len[r] in it copied in every plane (the copy on a first write after a fork).
 * Every page that holds the reserved positions then has count 1.
 *   status     [batch] int32, nullable: PSISPEC_ST_NO_PAGE when the free pages run out before this
 *              line is served (then neither it nor any later line that needs a page is),
 *              PSISPEC_ST_BAD_PAGE when len, n_new or a page of these slots is invalid; such a line
 *              stays as it is
 *   blk        1..2^20 (a whole prompt may be reserved at once)
 * Pages that become free in the call are given out by later calls only.  Workspace of both calls:
 * psispec_pages_workspace (blk of the reserve).
 */
psispec_status psispec_pages_reserve(const psispec_page_pool* pool, int32_t* table,
                                     int64_t table_stride, int32_t slots, int32_t* refs,
                                     const int32_t* len, const int32_t* n_new, int32_t blk,
                                     int32_t* status, int32_t batch, void* workspace,
                                     size_t workspace_bytes, void* stream);

/*
 * The layers around the paged attention: the norm of the residual stream and linear layers with frozen
 * weights of 4 bits, for the rows of a draft or verify forward (one token of one line up to a block of
 * every line; prompts too).
 *
 * psispec_add_rmsnorm, in one pass over the rows:
 *   h = x + residual;  residual_out = h;  y = h / sqrt(mean(h^2) + eps) * weight
 * in 32 bits; h is normalised as the 32-bit sum, y and residual_out are rounded once.  out holds y, or
 * 8-bit numbers q = y / s (clamped to +-448, to nearest) with
 *   scale_dtype F32   one s per row: the row's largest |y| / 448
 *   scale_dtype E8M0  one s per 32 columns: the smallest power of two (from 2^-127) with |y| <= 448 s in
 *                     the block; what psispec_w4_linear and psispec_w4_gated take
 * A row (block) of zeros gives zeros, with eps 0 too; one with an infinity or a NaN has an infinite or NaN scale,
 * its q are unspecified.
 *   x             rows of dim elements, x_stride elements apart; dtype PSISPEC_BF16 or PSISPEC_F16
 *   residual      rows of residual_dtype (dtype or PSISPEC_F32), or NULL: h = x
 *   residual_out  rows of residual_dtype, or NULL: h is not written
 *   weight        [dim] of dtype, or NULL: 1
 *   eps           >= 0, finite in 32 bits
 *   rows 0..2^24-1 (0 launches nothing);  dim 1..32768, a multiple of 32 with E8M0 scales
 *   out           rows of out_dtype: dtype or PSISPEC_F8E4M3
 *   scale         with F8E4M3 only (NULL otherwise): [rows] f32, or rows of dim / 32 bytes, scale_stride apart
 * Rows may start anywhere.  residual_out and
 * out may each be the rows of x or of residual themselves; every other overlap of an output with an input or
 * another output is refused (PSISPEC_EINVAL).  Asynchronous on `stream`; no workspace.
 */
psispec_status psispec_add_rmsnorm(const void* x, int64_t x_stride, psispec_dtype dtype,
                                   const void* residual, int64_t residual_stride,
                                   void* residual_out, int64_t residual_out_stride,
                                   psispec_dtype residual_dtype, const void* weight, double eps,
                                   int32_t rows, int32_t dim, void* out, int64_t out_stride,
                                   psispec_dtype out_dtype, void* scale, int64_t scale_stride,
                                   psispec_dtype scale_dtype, void* stream);

/*
 * Weights of 4 bits: w[n][k] = code[n][k] * scale[n][k / group], n outputs, k inputs.
 *   PSISPEC_W4_INT  codes are two's complement, -8..7; scales BF16 or F16, group 32, 64 or a multiple of 128
 *   PSISPEC_W4_MX   codes are floats of sign, 2 bits of exponent, 1 of mantissa (0, 0.5, 1, 1.5, 2, 3, 4,
 *                   6 and their negatives from code 8 on); scales E8M0, group 32
 * psispec_w4_pack writes a layer's codes and scales, as a checkpoint holds them, in the order in which the
 * products read them into `packed` (device, 256-byte aligned, psispec_w4_packed_bytes, the caller's for as long
 * as the layer is used).  Once per layer; the codes and scales are not needed afterwards.  packed_bytes gives 0 for
 * what is not supported.
 *   codes      row n at n * codes_stride bytes: k / 2 bytes, the even input's code in the low four bits
 *   scales     row n at n * scales_stride elements: ceil(k / group) of scale_dtype (a last group may be short)
 */
typedef enum { PSISPEC_W4_INT = 0, PSISPEC_W4_MX = 1 } psispec_w4_format;
typedef enum { PSISPEC_W4_SILU = 0, PSISPEC_W4_GELU = 1, PSISPEC_W4_GELU_TANH = 2 } psispec_w4_activation;
typedef struct {
  void* packed;        /* device; the products only read it */
  int32_t n;           /* outputs, 1..2^20 */
  int32_t k;           /* inputs, a multiple of 32, 32..2^20; ceil(n / 16) * ceil(k / 128) <= 2^26 - 4 */
  int32_t group;       /* inputs per scale */
  int32_t format;      /* psispec_w4_format */
  int32_t scale_dtype; /* PSISPEC_BF16 or PSISPEC_F16 (INT), PSISPEC_E8M0 (MX) */
  int32_t reserved;    /* must be 0 */
} psispec_w4_weight;

size_t psispec_w4_packed_bytes(int32_t n, int32_t k, int32_t group, int32_t format);

psispec_status psispec_w4_pack(const uint8_t* codes, int64_t codes_stride, const void* scales,
                               int64_t scales_stride, const psispec_w4_weight* w,
                               size_t packed_bytes, void* stream);

/*
 * A linear layer, and the two projections of a gated feed-forward block with their activation and product:
 *   psispec_w4_linear  out = x w^T + bias
 *   psispec_w4_gated   out = act(x gate^T) * (x up^T),  act(a) = a / (1 + exp(-a))   (PSISPEC_W4_SILU)
 *                      or a (1 + erf(a / sqrt 2)) / 2                                 (PSISPEC_W4_GELU)
 *                      or a (1 + tanh(sqrt(2 / pi) (a + 0.044715 a^3))) / 2           (PSISPEC_W4_GELU_TANH)
 * Codes and rows enter the matrix cores as they are, the sums are of 32 bits, INT scales are applied to the
 * sums of their groups in 32 bits, and out is rounded once: no weight is rounded.  Three exceptions:
 *   F16 rows, MX weights  exact for scales down to 2^-36 of the output's largest; smaller ones give weights off
 *                         by at most 2^-38 of that largest scale
 *   BF16 rows, MX weights an output whose largest scale is 2^126 takes 2^-127 as 2^-126, one with 2^127 takes
 *                         both as 2^-125
 *   8-bit rows            go through the scaled matrix instruction, at twice the 16-bit rate: among eight
 *                         neighbouring inputs each product is cut to a multiple of 2^-13 of the power of two
 *                         that the largest of them reaches
 * (INT weights: 31 times the sum of |x| over a group has to stay within 32 bits.)
 * An infinity or a NaN in a row, its scale or an output's scale gives infinities or NaN in that row, that
 * output, and nowhere else.
 *   x        rows of k elements, x_stride elements apart, 16-byte aligned, strides of 16-byte multiples up to 2^24
 *            bytes: dtype PSISPEC_BF16, PSISPEC_F16, or (MX weights) PSISPEC_F8E4M3 with x_scale: rows of k / 32
 *            E8M0 bytes, x_scale_stride apart (NULL for the other types)
 *   bias     [n] of out_dtype, or NULL
 *   out      rows of n elements, out_stride elements apart, of dtype (8-bit x: BF16 or F16); overlaps no input
 *            (PSISPEC_EINVAL)
 *   rows     0..2^24-1 (0 launches nothing), ceil(rows / 16) * ceil(n / 16) < 2^23
 *   gate, up of the same n, k, group, format and scale_dtype
 * The workspace is psispec_w4_weight_workspace(w, rows, 1) bytes, (.., 2) for a gated call; 0: none is needed and
 * NULL will do.  psispec_w4_workspace(rows, n, k, 1), (.., 2), is enough for either format: MX weights need no
 * sums of their rows, and mostly nothing.  What is needed of it overlaps no input and no output (PSISPEC_EINVAL).  Sums are taken in a fixed
 * order: reruns are bitwise identical.
 */
size_t psispec_w4_workspace(int32_t rows, int32_t n, int32_t k, int32_t mats);

size_t psispec_w4_weight_workspace(const psispec_w4_weight* w, int32_t rows, int32_t mats);

psispec_status psispec_w4_linear(const psispec_w4_weight* w, const void* x, int64_t x_stride,
                                 psispec_dtype dtype, const void* x_scale, int64_t x_scale_stride,
                                 int32_t rows, const void* bias, void* out, int64_t out_stride,
                                 psispec_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                 void* stream);

psispec_status psispec_w4_gated(const psispec_w4_weight* gate, const psispec_w4_weight* up,
                                int32_t activation, const void* x, int64_t x_stride,
                                psispec_dtype dtype, const void* x_scale, int64_t x_scale_stride,
                                int32_t rows, void* out, int64_t out_stride, psispec_dtype out_dtype,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Message for a return code (static string). */
const char* psispec_strerror(psispec_status code);

/*
 * Measured ceilings (for benchmarks; not steps of the verify).  psispec_peak_read reads every
 * 16-byte word of `buf` (device, 16-byte aligned, `bytes` long; make it larger than the 256 MB
 * last-level cache) once with nontemporal loads, each of `blocks` workgroups of 256 threads
 * streaming its own contiguous segment, and writes one word per block to out[blocks]:
 * bytes / kernel time is the sustained read bandwidth.  psispec_peak_mfma runs `iters` rounds of 16 independent v_mfma_f32_32x32x16_bf16 per
 * wave in `blocks` workgroups of four waves, with no memory traffic, and writes one float per
 * thread to out[blocks * 256]: blocks * 4 * iters * 16 * 32768 / kernel time is the bf16 matrix-core
 * issue rate at the clock the chip holds under that load.  Both are asynchronous on `stream`;
 * the kernels appear in the timing records as "peak_read" and "peak_mfma".
 */
psispec_status psispec_peak_read(const void* buf, size_t bytes, uint32_t* out, int32_t blocks,
                                 void* stream);
psispec_status psispec_peak_mfma(int64_t iters, float* out, int32_t blocks, void* stream);

/*
 * Kernel timing (for benchmarks).  While enabled, every kernel launch of the library records a
 * start and a stop event through its own dispatch (hipExtLaunchKernelGGL) on the call's stream:
 * the events measure the kernel itself, as a profiler's kernel trace does.  psispec_timing_read synchronises those events and
 * returns, per kernel name, the summed device milliseconds and the launch count since the last
 * enable; it returns the number of kernels written (at most max_kernels).  names receives
 * max_kernels fixed slots of 64 bytes (NUL-terminated).
 */
psispec_status psispec_timing_enable(int32_t on);
int32_t psispec_timing_read(char* names, float* total_ms, int32_t* launches, int32_t max_kernels);

#ifdef __cplusplus
}
#endif
#endif /* PSISPEC_H */
