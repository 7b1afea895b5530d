/*
 * ga_attn.h -- C ABI of the GB300 (sm_103a) gated grouped-query attention library
 * (libga_attn.so).
 *
 * The operation (pegainfer PR #1151, "feat(qwen4): add the QSA sparse-attention kernel
 * and its golden", §Semantics): split each fused q|gate row, apply (1+w) RMSNorm to q
 * and k (eps 1e-6), rotate dims 0..63 of q and k (rotate-half partial RoPE) from a
 * shared bf16 cos/sin table, score s = bf16(q.k) / 16 over GQA groups of 12 (query
 * head h reads KV head h / 12), softmax in fp32 over the visible keys with the weights
 * rounded to bf16 before the context reduction, reduce P.V, and multiply by
 * bf16(sigmoid(gate)). Output columns are head-major (h * 256 + d).
 *
 * Geometry is compiled in: 24 query heads, 2 KV heads, head_dim 256, 64 rotary dims,
 * eps 1e-6, RoPE base 1e7 (the same page, the commit that replaces the proxy geometry).
 *
 * Conventions for every entry point below:
 *  - Tensor pointers are DEVICE pointers owned by the caller, unless a comment says
 *    HOST. The library never allocates device memory on a call path, and keeps no
 *    pointer after the call returns. bf16 values are passed as their 16-bit patterns
 *    (ga_bf16). All tensors are dense, row-major, without padding unless a leading
 *    dimension argument says otherwise.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy default stream)
 *    and is asynchronous: the return value reports argument validation and launch
 *    errors, not the kernels' completion. Calls on different streams are re-entrant.
 *  - Every argument is validated BEFORE any CUDA call (system1-omni PR #99, "run
 *    prompts that share prefixes once per prefix": refusals happen before any
 *    allocation or CUDA call). A zero-row call returns GA_OK without touching the GPU
 *    (pegainfer PR #1151, §What changed: an empty launch is a no-op).
 *  - There is no fallback path: a launch failure is returned as GA_ERR_CUDA with the
 *    CUDA error kept for ga_last_cuda_error() (system1-omni PR #202, "cuda: widen the
 *    attention query tile on sm_89 and sm_120", review §Dispatch/guard: no silent
 *    fallback).
 *  - Kernels never trap. A bounded device-side wait that gives up records an error in
 *    the library's device status word (ga_device_status).
 *  - Pointers that the kernels read or write with 16-byte vector or TMA accesses must be
 *    16-byte aligned (GA_ERR_ALIGN otherwise).
 */
#ifndef GA_ATTN_H
#define GA_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GA_ABI_VERSION 1

#define GA_N_Q_HEADS 24
#define GA_N_KV_HEADS 2
#define GA_HEAD_DIM 256
#define GA_ROPE_DIMS 64
#define GA_MASKED_MAX_TOKENS 8192 /* pegainfer PR #1151, §Summary: the 8192-token cap */
#define GA_MAX_TOKENS (1 << 20)   /* index-arithmetic limit of the library */
/* Keys per indexer block (pegainfer PR #1151: a budget of 2048 tokens is 512 blocks). */
#define GA_INDEX_BLOCK_TOKENS 4

typedef uint16_t ga_bf16; /* bfloat16 bit pattern */
typedef void* ga_stream;  /* cudaStream_t */

enum ga_status {
  GA_OK = 0,
  GA_ERR_NULL = -1,      /* a required pointer is NULL */
  GA_ERR_SHAPE = -2,     /* a size is negative or zero where it must be positive */
  GA_ERR_ALIGN = -3,     /* a pointer or leading dimension breaks 16-byte alignment */
  GA_ERR_RANGE = -4,     /* a window, position or size is outside what the call allows */
  GA_ERR_TABLE = -5,     /* the cos/sin table is shorter than the largest position + 1 */
  GA_ERR_WORKSPACE = -6, /* workspace missing, misaligned or smaller than required */
  GA_ERR_DEVICE = -7,    /* current device is not sm_103 or refused the smem opt-in */
  GA_ERR_CUDA = -8,      /* a CUDA call failed; see ga_last_cuda_error() */
  GA_ERR_GEOMETRY = -9   /* ga_check_geometry: not the compiled geometry */
};

/* Geometry a caller expects; ga_check_geometry compares it with the compiled constants
 * (pegainfer PR #1151, §What changed: the wrapper validates its geometry against the
 * compiled constants before sizing any buffer). */
typedef struct ga_geometry {
  int n_q_heads;    /* 24 */
  int n_kv_heads;   /* 2 */
  int head_dim;     /* 256 */
  int rope_dims;    /* 64 */
  float eps;        /* 1e-6 */
  double rope_base; /* 1e7 */
} ga_geometry;

/* GA_ABI_VERSION of the loaded library. */
int ga_abi_version(void);

/* GA_OK if *g equals the compiled geometry, GA_ERR_GEOMETRY if not, GA_ERR_NULL for NULL. */
int ga_check_geometry(const ga_geometry* g);

/* Static English text for a status code (never NULL). */
const char* ga_status_string(int status);

/* The cudaError_t value behind the calling thread's last GA_ERR_CUDA (0 if none). */
int ga_last_cuda_error(void);

/* Number of CUDA runtime calls this library has made in this process (diagnostic: a
 * refused call must not change it). Makes no CUDA call itself. */
unsigned long long ga_debug_cuda_calls(void);

/* Reads the current device's status word, written by kernels whose bounded waits gave
 * up or whose inputs failed a device-side check (0 = no error, 1 = wait timeout, 2 = bad
 * launch configuration, 3 = a page-table entry or slot outside the page pool, see
 * ga_attn_verify_paged, ga_kv_quantize_q4 and the calls over pages, 4 = a rotary position outside the table or a
 * cached length outside the page table, see ga_qk_prologue_axes and ga_attn_verify_q4).
 * Synchronises the device. clear != 0 resets the word afterwards. */
int ga_device_status(int* status_out, int clear);

/* Test hook for failure detection (no counterpart in the pages): launches a one-thread
 * kernel that waits, bounded by limit_cycles SM clock cycles (1 .. 2e9), on an mbarrier
 * that nothing arrives on. The wait gives up, the kernel records the wait-timeout status
 * (1) in the device status word and returns: the same bounded wait and recording every
 * kernel of the library uses, without a fault, a trap or a hang. Read the result with
 * ga_device_status. Errors: RANGE, DEVICE, CUDA. */
int ga_debug_wait_timeout(long long limit_cycles, ga_stream stream);

/* Selects how the attention passes run (no counterpart in the pages; the results are the
 * same bits either way). mode 2: the causal, bidirectional, stored-mask and batched passes
 * as clusters of two CTAs that share each key and value tile, two query heads of one KV
 * group per pair item, whenever the call's heads come in such pairs (every call through the
 * ABI does: the KV-group entry points take whole groups of 12); the weights pass and the
 * verify passes on single CTAs. mode 1 (the default): the same, except that causal,
 * bidirectional and stored-mask calls over fewer than 2,048 keys run on single CTAs, which
 * are faster there. mode 0: every pass on single CTAs (one CTA per 128-row tile and head).
 * Process-wide; takes effect from the next call. Returns the previous mode (0, 1 or 2).
 * Errors: RANGE (mode outside 0 .. 2). Makes no CUDA call. */
int ga_debug_set_cta_pairs(int mode);

/* Test hook: the fp32 dot products the tensor cores form for the scores, before any
 * rounding. For each of n_tiles tiles, s[n][i][j] = q[n][i] . k[n][j] over 256 dims, computed
 * exactly as the attention kernel computes S = Q K^T (tcgen05.mma kind::f16, M128 N128,
 * sixteen K16 steps accumulating in fp32 in tensor memory, operands in shared memory in the
 * kernel's 128-byte-swizzled layout). The score is the bf16 rounding of this value (pegainfer
 * PR #1151, the commit that adds the attention reader: "the bf16 GEMM result"); the fp32
 * reduction order inside the tensor core is the hardware's, and the tests use this hook to
 * bound its distance from the exact dot product.
 *   q, k   [n_tiles][128][256] bf16, 16-byte aligned
 *   s      [n_tiles][128][128] fp32, 16-byte aligned
 * Rules: 0 <= n_tiles <= 65535 (0 is a no-op).
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_debug_qk_fp32(const ga_bf16* q, const ga_bf16* k, int n_tiles, float* s,
                     ga_stream stream);

/* HOST helper. Fills cos_out and sin_out (HOST arrays of n_pos * 32 values each,
 * [position][pair]) with cos and sin of p * 1e7^(-2i/64) for positions p < n_pos and
 * pairs i < 32, each computed in double and rounded once to bf16 (pegainfer PR #1151,
 * review F4: a double pow, rounded once; §What changed: one shared table, no device
 * trigonometry). Pair i rotates dims i and i + 32. Makes no CUDA call. */
int ga_rope_table_host(int n_pos, ga_bf16* cos_out, ga_bf16* sin_out);

/* K prologue (pegainfer PR #1151, §What changed: one key pass (1+w)-norms and partially
 * rotates every token's two key heads once, because all twelve query heads of a KV head
 * read the same prepared key).
 *   k_raw  [n_tok][2][256]  raw keys of tokens at positions pos_base .. pos_base+n_tok-1
 *   w_k    [256]            key norm weight w (applied as 1 + w)
 *   cos_tab, sin_tab [table_rows][32]; table_rows >= pos_base + n_tok
 *   k_prep [n_tok][2][256]  output: bf16(rope(norm(k))); may not alias k_raw
 * Errors: NULL, SHAPE (n_tok < 0), RANGE (pos_base < 0 or n_tok > GA_MAX_TOKENS), TABLE,
 * ALIGN (k_raw, k_prep, cos_tab, sin_tab, w_k), DEVICE, CUDA. */
int ga_k_prologue(const ga_bf16* k_raw, const ga_bf16* w_k, const ga_bf16* cos_tab,
                  const ga_bf16* sin_tab, int table_rows, int n_tok, int pos_base,
                  ga_bf16* k_prep, ga_stream stream);

/* Query prologue: the same (1+w) RMSNorm and partial RoPE for the q half of every fused
 * row and head (pegainfer PR #1151, §Semantics: q is split from the fused q|gate row,
 * normed and rotated at its own position). ga_attn_prefill runs it itself; it is exposed
 * so that a caller can time or reuse the prepared queries (ga_attn_prefill_prepared).
 *   qg      [rows][24][512]  fused rows of positions q_base .. q_base+rows-1
 *   w_q     [256]            query norm weight w (applied as 1 + w)
 *   cos_tab, sin_tab [table_rows][32]; table_rows >= q_base + rows
 *   q_prep  [rows][24][256]  output: bf16(rope(norm(q))); may not overlap qg
 * Errors: NULL, SHAPE (rows < 0), RANGE (q_base < 0 or rows > GA_MAX_TOKENS), TABLE,
 * ALIGN (qg, w_q, cos_tab, sin_tab, q_prep), DEVICE, CUDA. */
int ga_q_prologue(const ga_bf16* qg, const ga_bf16* w_q, const ga_bf16* cos_tab,
                  const ga_bf16* sin_tab, int table_rows, int rows, int q_base,
                  ga_bf16* q_prep, ga_stream stream);

/* Both prologues in one launch (pegainfer PR #1151, §What changed and §Semantics: the key
 * pass and the query pass take the same (1+w) norm and partial rotation):
 * ga_k_prologue over n_tok key tokens and ga_q_prologue over rows fused query rows, with
 * the same results bit for bit. One persistent grid walks the
 * key rows and then the query rows, so the two share every SM instead of competing as two
 * launches on two streams would.
 *   k_raw, w_k, n_tok, k_pos_base, k_prep: as ga_k_prologue's k_raw, w_k, n_tok, pos_base
 *                            and k_prep
 *   qg, w_q, rows, q_base, q_prep: as ga_q_prologue's; q_prep may not overlap qg, and no
 *                            output may overlap the other call's inputs or output
 *   cos_tab, sin_tab [table_rows][32]; table_rows >= k_pos_base + n_tok and
 *                            table_rows >= q_base + rows
 * Errors: NULL, SHAPE (n_tok < 0 or rows < 0), RANGE, TABLE, ALIGN (every pointer),
 * DEVICE, CUDA; all checked before anything is launched. */
int ga_qk_prologue(const ga_bf16* k_raw, const ga_bf16* w_k, int n_tok, int k_pos_base,
                   ga_bf16* k_prep, const ga_bf16* qg, const ga_bf16* w_q, int rows, int q_base,
                   ga_bf16* q_prep, const ga_bf16* cos_tab, const ga_bf16* sin_tab,
                   int table_rows, ga_stream stream);

/* Causal / prefix-window / bidirectional gated GQA attention (system1-omni PR #202,
 * §Scope: full pass, causal or bidirectional, and causal prefix windows at q_base).
 *   qg      [rows][24][512]  fused rows of query positions q_base .. q_base+rows-1; per
 *                            head the first 256 values are q, the last 256 the gate
 *   k_prep  [T][2][256]      prepared keys (ga_k_prologue) of positions 0 .. T-1
 *   v       [T][2][256]      values
 *   w_q     [256]            query norm weight w (applied as 1 + w)
 *   cos_tab, sin_tab [table_rows][32]; table_rows >= q_base + rows
 *   causal  1: row r sees keys j <= q_base + r;  0: bidirectional, every key j < T
 *           (q_base must then be 0)
 *   out     [rows][24 * 256] bf16, head-major columns. It may not overlap any input;
 *           the call also uses it as scratch (each (row, head) slot holds that row's
 *           prepared query before its output), so its contents are unspecified until
 *           the call has completed on the stream.
 *   row_stats NULL or [24][rows][2] float: per (head, row) the final running maximum M
 *           (an integer, base-2 units) and the sum l of the rounded weights relative to
 *           2^M, so that the row's weights are bf16(2^(t - M)) / l with t = s * log2(e).
 * Rules (review §Dispatch/guard of the same page): q_base % 64 == 0, q_base >= 0,
 * q_base + rows <= T <= GA_MAX_TOKENS.
 * Errors: NULL, SHAPE, RANGE, TABLE, ALIGN (qg, k_prep, v, out, w_q, tables, row_stats),
 * DEVICE, CUDA. */
int ga_attn_prefill(const ga_bf16* qg, const ga_bf16* k_prep, const ga_bf16* v,
                    const ga_bf16* w_q, const ga_bf16* cos_tab, const ga_bf16* sin_tab,
                    int table_rows, int rows, int T, int q_base, int causal, ga_bf16* out,
                    float* row_stats, ga_stream stream);

/* ga_attn_prefill for one group of KV heads: the query heads 12 * kv_first ..
 * 12 * (kv_first + kv_count) - 1 (each KV head with the 12 query heads that read it) and
 * nothing else. This is how the pass shards over GPUs with no exchange between them: GPU g
 * takes KV head g, reads only that head's keys and values and its query heads' halves of the
 * fused rows, and writes only their output columns h * 256 .. h * 256 + 255; the other
 * columns of out (and of row_stats) are left as they were. The results are the bits of
 * ga_attn_prefill in those columns.
 *   kv_first, kv_count: 0 <= kv_first, 1 <= kv_count, kv_first + kv_count <= 2
 *   every other argument as in ga_attn_prefill (out doubles as scratch only in the columns
 *   of the heads processed)
 * Errors: as ga_attn_prefill (RANGE also for the KV-head group). */
int ga_attn_prefill_kv(const ga_bf16* qg, const ga_bf16* k_prep, const ga_bf16* v,
                       const ga_bf16* w_q, const ga_bf16* cos_tab, const ga_bf16* sin_tab,
                       int table_rows, int rows, int T, int q_base, int causal, int kv_first,
                       int kv_count, ga_bf16* out, float* row_stats, ga_stream stream);

/* ga_attn_prefill from prepared queries (ga_q_prologue's output): the attention kernel
 * alone. qg still supplies the gates (its last 256 values per head).
 *   q_prep  [rows][24][256]  prepared queries; may be the same buffer as out (each
 *                            (row, head) slot is read before its output is written there)
 *   qg, k_prep, v, rows, T, q_base, causal, out, row_stats: as in ga_attn_prefill
 * Errors: NULL, SHAPE, RANGE, ALIGN (q_prep, qg, k_prep, v, out, row_stats), DEVICE, CUDA. */
int ga_attn_prefill_prepared(const ga_bf16* q_prep, const ga_bf16* qg, const ga_bf16* k_prep,
                             const ga_bf16* v, int rows, int T, int q_base, int causal,
                             ga_bf16* out, float* row_stats, ga_stream stream);

/* Bytes of workspace ga_attn_masked needs for (rows, T); 0 for invalid sizes. */
size_t ga_masked_workspace_bytes(int rows, int T);

/* Stored-mask gated GQA attention (pegainfer PR #1151, §Semantics: the kernel consumes
 * the selection mask as given, non-zero = visible; it is not ANDed with causality here).
 *   qg, k_prep, v, w_q, cos_tab, sin_tab, table_rows, q_base: as in ga_attn_prefill
 *   mask    [rows][ld_mask] uint8; row r is query position q_base + r, column j key j
 *   out     [rows][24 * 256] (scratch during the call, as in ga_attn_prefill)
 *   weights NULL or [24][rows][T] bf16: the normalised weights bf16(w_hat / L), exactly
 *           0 where a key is hidden
 *   hidden_rows NULL or one device int; receives the number of rows with no visible key
 *           (their outputs and weights are 0; the page leaves such rows outside its
 *           contract)
 *   workspace >= ga_masked_workspace_bytes(rows, T) bytes of device memory, 256-byte
 *           aligned, owned by the caller, not shared with a concurrent call
 * Rules: T <= GA_MASKED_MAX_TOKENS, ld_mask >= T, ld_mask % 16 == 0, q_base % 64 == 0,
 * q_base + rows <= T.
 * Errors: NULL, SHAPE, RANGE, TABLE, ALIGN (mask also), WORKSPACE, DEVICE, CUDA. */
int ga_attn_masked(const ga_bf16* qg, const ga_bf16* k_prep, const ga_bf16* v,
                   const ga_bf16* w_q, const ga_bf16* cos_tab, const ga_bf16* sin_tab,
                   int table_rows, int rows, int T, int q_base, const uint8_t* mask,
                   long long ld_mask, ga_bf16* out, ga_bf16* weights, int* hidden_rows,
                   void* workspace, size_t ws_bytes, ga_stream stream);

/* ga_attn_masked for one group of KV heads (see ga_attn_prefill_kv): the query heads
 * 12 * kv_first .. 12 * (kv_first + kv_count) - 1 only. Their output columns (and, when
 * weights is given, their [12 * kv_count][rows][T] slice of weights, zeroed first) are
 * written; everything else is left as it was. hidden_rows counts each hidden row once.
 *   kv_first, kv_count: 0 <= kv_first, 1 <= kv_count, kv_first + kv_count <= 2
 *   every other argument as in ga_attn_masked
 * Errors: as ga_attn_masked (RANGE also for the KV-head group). */
int ga_attn_masked_kv(const ga_bf16* qg, const ga_bf16* k_prep, const ga_bf16* v,
                      const ga_bf16* w_q, const ga_bf16* cos_tab, const ga_bf16* sin_tab,
                      int table_rows, int rows, int T, int q_base, const uint8_t* mask,
                      long long ld_mask, int kv_first, int kv_count, ga_bf16* out,
                      ga_bf16* weights, int* hidden_rows, void* workspace, size_t ws_bytes,
                      ga_stream stream);

/* ga_attn_masked from prepared queries (ga_q_prologue's output): the mask prepass and the
 * attention kernel (and the weights pass) without the query prologue, exposed so that a
 * caller can time or reuse the prepared queries, as ga_attn_prefill_prepared does for the
 * causal pass.
 *   q_prep  [rows][24][256]  prepared queries of positions q_base .. q_base+rows-1, 16-byte
 *                            aligned; may not overlap out
 *   qg, k_prep, v, rows, T, q_base, mask, ld_mask, out, weights, hidden_rows, workspace,
 *           ws_bytes: as in ga_attn_masked (the workspace's query area is not used)
 * Rules and errors: as ga_attn_masked (NULL also for q_prep), without the table checks. */
int ga_attn_masked_prepared(const ga_bf16* q_prep, const ga_bf16* qg, const ga_bf16* k_prep,
                            const ga_bf16* v, int rows, int T, int q_base, const uint8_t* mask,
                            long long ld_mask, ga_bf16* out, ga_bf16* weights,
                            int* hidden_rows, void* workspace, size_t ws_bytes,
                            ga_stream stream);

/* Allocation-free variant of ga_attn_masked. The pages have no counterpart: this is an
 * addition of the library for callers that may not allocate device memory at call time,
 * such as a server step that runs under a fixed memory budget, or a framework that
 * forbids allocation inside a step (an allocation can synchronise the device, and can
 * fail when memory is fragmented). The scratch that ga_attn_masked takes as `workspace`
 * comes instead from one static device array of GA_STATIC_SCRATCH_BYTES per device,
 * reserved when the library is loaded; nothing is allocated by the call.
 *   Arguments, layouts and results: as in ga_attn_masked, without workspace/ws_bytes.
 *   Limit: the call runs when ga_masked_workspace_bytes(rows, T) <=
 *           GA_STATIC_SCRATCH_BYTES: up to 1,239 rows at T = 8192, 1,286 at T = 4096,
 *           1,315 at T = 2048. Larger calls are refused with GA_ERR_WORKSPACE before any
 *           CUDA call.
 *   The first call on a device looks up the array's address (one CUDA runtime query,
 *           once per device, with that device current); make a first call before any
 *           stream capture. The address is kept per device index for the life of the
 *           process: the library assumes each device's primary context (the runtime's
 *           default) and no cudaDeviceReset between calls, the same assumption as its
 *           other per-device set-up.
 *   The scratch needs no initial contents (every call writes all of it that it reads).
 *   The array is shared by all calls on a device: calls that may overlap in time (other
 *           streams, other host threads) race on it and must be serialised by the caller.
 * Errors: as ga_attn_masked. */
#define GA_STATIC_SCRATCH_BYTES ((size_t)16 << 20)
int ga_attn_masked_static(const ga_bf16* qg, const ga_bf16* k_prep, const ga_bf16* v,
                          const ga_bf16* w_q, const ga_bf16* cos_tab, const ga_bf16* sin_tab,
                          int table_rows, int rows, int T, int q_base, const uint8_t* mask,
                          long long ld_mask, ga_bf16* out, ga_bf16* weights, int* hidden_rows,
                          ga_stream stream);

/* The widened rows of e4m3 cache rows: out = bf16(fp32(code * scale)) per element, the
 * values ga_attn_verify_e4m3 attends over (TensorFold PR #1080: e4m3 cache rows with an
 * fp32 scale each, widened to bf16).
 *   q      [n_tok][2][256] uint8 e4m3 codes, as ga_kv_quantize_e4m3 writes them, 8-byte aligned
 *   scale  [n_tok][2] fp32, 4-byte aligned
 *   out    [n_tok][2][256] bf16, 16-byte aligned
 * Rules: 0 <= n_tok <= 64 * GA_MAX_TOKENS; n_tok == 0 is a no-op.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_kv_dequantize_e4m3(const uint8_t* q, const float* scale, long long n_tok, ga_bf16* out,
                          ga_stream stream);

/* Bytes of workspace ga_attn_prefill_e4m3 needs for T keys (the widened K and V); 0 for
 * T outside 1 .. GA_MAX_TOKENS. */
size_t ga_prefill_e4m3_workspace_bytes(int T);

/* ga_attn_prefill over e4m3 caches of prepared keys and values (TensorFold PR #1080: e4m3
 * cache rows with an fp32 scale each, read by the prompt chain). Prefill reads every key
 * tile once per 128-row tile of queries, so the rows are widened once, into the workspace,
 * by ga_kv_dequantize_e4m3's kernel, and the bf16 pass then runs over them: the results
 * are the bits of ga_attn_prefill over the widened rows.
 *   k_codes, v_codes [T][2][256] uint8, 16-byte aligned; k_scale, v_scale [T][2] fp32
 *   qg, w_q, cos_tab, sin_tab, table_rows, rows, T, q_base, causal, out, row_stats: as in
 *           ga_attn_prefill
 *   workspace >= ga_prefill_e4m3_workspace_bytes(T) bytes, 256-byte aligned, owned by the
 *           caller and not shared with a concurrent call; it holds the widened K then V
 * Errors: NULL, SHAPE, RANGE, TABLE, ALIGN, WORKSPACE, DEVICE, CUDA. */
int ga_attn_prefill_e4m3(const ga_bf16* qg, const uint8_t* k_codes, const float* k_scale,
                         const uint8_t* v_codes, const float* v_scale, const ga_bf16* w_q,
                         const ga_bf16* cos_tab, const ga_bf16* sin_tab, int table_rows,
                         int rows, int T, int q_base, int causal, ga_bf16* out,
                         float* row_stats, void* workspace, size_t ws_bytes, ga_stream stream);

/* The selection mask ga_attn_masked reads, from the indexer's per-block scores (pegainfer
 * PR #1151, "feat(qwen4): add the QSA sparse-attention kernel and its golden": the mask is
 * the indexer's selection AND causality; a budget of 2048 tokens keeps 512 blocks of 4 keys,
 * a budget of 16 keeps 4). The scores themselves come from the indexer, which the pages
 * do not specify; this call does the selection and writes the mask.
 *   block_scores [rows][ld_scores] fp32, 4-byte aligned: row r scores block b (keys
 *           4b .. 4b+3) at r * ld_scores + b for b < ceil(T / 4). Scores may be +-inf
 *           and -0 equals +0; a NaN score gives an unspecified selection for its row.
 *   rows, T, q_base: row r is query position p = q_base + r; the keys are 0 .. T-1
 *   block_topk  blocks kept per row (budget / GA_INDEX_BLOCK_TOKENS)
 *   mask    [rows][ld_mask] uint8, written for columns 0 .. T-1 (later columns untouched):
 *           1 iff j <= p and block j / 4 is among the row's block_topk highest-scoring
 *           candidates (the blocks b <= p / 4), a tie going to the lower block index;
 *           every candidate when there are fewer. A row always sees at least one key.
 * Rules: T <= GA_MASKED_MAX_TOKENS, q_base + rows <= T, ld_scores >= ceil(T / 4),
 * ld_mask >= T, ld_mask % 16 == 0, mask 16-byte aligned, both leading dimensions <= 2^31.
 * Nothing is allocated; the call keeps no pointer. rows == 0 is a no-op.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_select_mask(const float* block_scores, long long ld_scores, int rows, int T, int q_base,
                   int block_topk, uint8_t* mask, long long ld_mask, ga_stream stream);

/* Bytes of workspace ga_attn_verify needs; max_len is the largest L over the sequences. */
size_t ga_verify_workspace_bytes(int n_seq, int rows, int max_len);

/* Few-row verify windows over long caches, split over key chunks with a log-sum-exp
 * combine (TensorFold PR #1080, "qwen CUDA: long-prompt prefill 5.4x faster", the
 * attn_partial commit: keys split into chunks, partial rows combined afterwards).
 *   qg       [n_seq][rows][24][512] fused rows; sequence b's row r is position L_b + r
 *   k_cache  [n_seq][cap][2][256] PREPARED keys of positions 0 .. L_b+rows-1 (the
 *            window's own keys included; fill with ga_k_prologue)
 *   v_cache  [n_seq][cap][2][256] values
 *   seq_len  HOST array of n_seq ints: L_b, with L_b >= 0 and L_b + rows <= cap
 *   out      [n_seq][rows][24 * 256] (scratch during the call, as in ga_attn_prefill)
 *   workspace >= ga_verify_workspace_bytes(n_seq, rows, max L_b), 256-byte aligned
 * Row r of sequence b sees keys 0 .. L_b + r. Cache positions from L_b + rows up to the
 * end of the 128-key tile that holds position L_b + rows - 1 are read and hidden, so they
 * must hold finite values (a hidden value still meets the tensor cores with weight 0).
 * Rules: 1 <= rows <= 16, cap <= GA_MAX_TOKENS, table_rows >= max L_b + rows.
 * Errors: NULL, SHAPE, RANGE, TABLE, ALIGN, WORKSPACE, DEVICE, CUDA. */
int ga_attn_verify(const ga_bf16* qg, const ga_bf16* k_cache, const ga_bf16* v_cache,
                   int cap, const int* seq_len, int n_seq, int rows, const ga_bf16* w_q,
                   const ga_bf16* cos_tab, const ga_bf16* sin_tab, int table_rows,
                   ga_bf16* out, void* workspace, size_t ws_bytes, ga_stream stream);

/* ga_attn_verify over e4m3 caches (TensorFold PR #1080, "qwen CUDA: long-prompt prefill 5.4x
 * faster": e4m3 cache rows with an fp32 scale each, staged a step ahead and widened to bf16
 * in the shared-memory slot). The caches hold what ga_kv_quantize_e4m3 writes:
 *   k_codes, v_codes  [n_seq][cap][2][256] uint8 e4m3 codes, 16-byte aligned
 *   k_scale, v_scale  [n_seq][cap][2] fp32 row scales, 4-byte aligned
 * Each row is widened to bf16(fp32(code * scale)) and the call then computes exactly what
 * ga_attn_verify computes over those bf16 rows: the same bits. It reads half the cache bytes.
 * Positions read but hidden (past L_b + rows inside the last 128-key tile, below cap) must
 * hold codes other than NaN (0x7F, 0xFF) and finite scales. Everything else, the rules and
 * the errors are those of ga_attn_verify, with the same workspace size. */
int ga_attn_verify_e4m3(const ga_bf16* qg, const uint8_t* k_codes, const float* k_scale,
                        const uint8_t* v_codes, const float* v_scale, int cap, const int* seq_len,
                        int n_seq, int rows, const ga_bf16* w_q, const ga_bf16* cos_tab,
                        const ga_bf16* sin_tab, int table_rows, ga_bf16* out, void* workspace,
                        size_t ws_bytes, ga_stream stream);

/* ga_attn_verify over PAGED caches, and decode (rows = 1). pegainfer PR #1151, "feat(qwen4):
 * add the QSA sparse-attention kernel and its golden", §Summary and §Limits name paged KV
 * and decode as the next steps after its contiguous key array; the layout is the plain
 * reading of a page table. Each sequence's positions live in fixed-size pages of two pools:
 *   k_pages   [n_pages][page_size][2][256] PREPARED keys (as ga_k_prologue writes them)
 *   v_pages   [n_pages][page_size][2][256] values
 *   page_table DEVICE int32 [n_seq][max_pages]: position t of sequence b lives on page
 *             page_table[b * max_pages + t / page_size], slot t % page_size. Only the
 *             entries that cover positions 0 .. L_b + rows - 1 are read; each must lie in
 *             [0, n_pages). An entry outside that range is not a fault: the kernel records
 *             status 3 in the device status word (ga_device_status) and reads zeros for
 *             that tile, so the call's outputs are then meaningless.
 *   page_size a multiple of 128 (one or more 128-key tiles per page)
 * Everything else (qg, seq_len on the HOST, rows, the tables, out, the workspace from
 * ga_verify_workspace_bytes, the finite-values rule for hidden positions) is as in
 * ga_attn_verify, and so are the results: the same sequence gives the same bits whether
 * its caches are contiguous or paged. Pages may be shared between sequences (a common
 * prefix) and need not be in any order. Nothing is allocated; the call keeps no pointer.
 * Rules: 1 <= rows <= 16, L_b + rows <= max_pages * page_size and <= GA_MAX_TOKENS,
 * table_rows >= max L_b + rows, page_table 4-byte aligned.
 * Errors: NULL, SHAPE, RANGE, TABLE, ALIGN, WORKSPACE, DEVICE, CUDA. */
int ga_attn_verify_paged(const ga_bf16* qg, const ga_bf16* k_pages, const ga_bf16* v_pages,
                         int n_pages, int page_size, const int* page_table, int max_pages,
                         const int* seq_len, int n_seq, int rows, const ga_bf16* w_q,
                         const ga_bf16* cos_tab, const ga_bf16* sin_tab, int table_rows,
                         ga_bf16* out, void* workspace, size_t ws_bytes, ga_stream stream);

/* e4m3 cache rows with one fp32 scale each (TensorFold PR #1080, "qwen CUDA: long-prompt
 * prefill 5.4x faster": its prompt chain reads e4m3 cache rows with an fp32 scale each and
 * widens them to bf16 in the shared-memory slot; its rope kernels compute the e4m3 scales by
 * reductions over the row). For every (token, head) row of 256 bf16 values x:
 *   scale = fp32(max|x| / 448),  q = e4m3(fp32(x / scale))
 * with IEEE divisions rounded to nearest and the OCP FP8 E4M3 conversion rounding to nearest
 * (ties to even) and saturating at +-448; a row of zeros gives scale 0 and q 0. The widened
 * row that ga_attn_verify_e4m3 attends over is bf16(fp32(q * scale)).
 *   x      [n_tok][2][256] bf16: prepared keys (as ga_k_prologue writes them) or values
 *   q      [n_tok][2][256] uint8 e4m3 codes (byte d of a row is dim d)
 *   scale  [n_tok][2] fp32
 * Rules: x 8-byte aligned, q 4-byte aligned, scale 4-byte aligned, 0 <= n_tok <= GA_MAX_TOKENS
 * x 64 (sequences laid end to end count as one long run). n_tok = 0 is a no-op.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_kv_quantize_e4m3(const ga_bf16* x, long long n_tok, uint8_t* q, float* scale,
                        ga_stream stream);

/* Several causal prefills in one call: sequences (or branches) of different lengths, each a
 * window of rows at its own q_base over its own paged cache. system1-omni PR #99, "run
 * prompts that share prefixes once per prefix", and PR #196, "perf(open-jev): optimize 9B
 * prefill while preserving native outputs" (its batched gated-attention entry points,
 * checked bit for bit against the one-sequence path): prompts that share a prefix run the
 * prefix once and continue each branch from it. Here a branch is a sequence whose page-table
 * row lists the prefix's pages (whole pages, shared) and then its own; its rows are its
 * positions after the prefix (q_base = the prefix length).
 *   qg          [total_rows][24][512] fused rows of all sequences, packed: sequence b's row r
 *               is packed row row_start[b] + r, at position q_base[b] + r
 *   row_start   HOST int[n_seq + 1], ascending, row_start[0] >= 0; sequence b has
 *               row_start[b + 1] - row_start[b] >= 0 rows
 *   q_base      HOST int[n_seq], multiples of 64
 *   k_pages, v_pages, n_pages, page_size, page_table, max_pages: as in ga_attn_verify_paged;
 *               sequence b's keys 0 .. q_base[b] + rows_b - 1 are read through page-table
 *               row b (they must be prepared and present, the window's own keys included)
 *   out         [total_rows][24 * 256] (scratch during the call, as in ga_attn_prefill)
 * Row r of sequence b sees keys 0 .. q_base[b] + r. Every sequence's rows come out with the
 * same bits as ga_attn_prefill gives for them over the same keys (causal, window q_base[b],
 * T = q_base[b] + rows_b). The kernels handle up to 64 sequences and 256 row tiles of 128
 * rows per launch and the call launches as many times as needed; nothing is allocated and
 * no pointer is kept. Hidden positions read inside a window's last key tile must be finite.
 * Rules: page_size a multiple of 128, q_base[b] + rows_b <= max_pages * page_size and
 * <= GA_MAX_TOKENS, row_start[n_seq] <= GA_MAX_TOKENS, table_rows >= max q_base[b] + rows_b,
 * page_table 4-byte aligned. A call with no rows returns GA_OK without a CUDA call.
 * Errors: NULL, SHAPE, RANGE, TABLE, ALIGN, DEVICE, CUDA. */
int ga_attn_prefill_batch(const ga_bf16* qg, const int* row_start, const int* q_base, int n_seq,
                          const ga_bf16* k_pages, const ga_bf16* v_pages, int n_pages,
                          int page_size, const int* page_table, int max_pages,
                          const ga_bf16* w_q, const ga_bf16* cos_tab, const ga_bf16* sin_tab,
                          int table_rows, ga_bf16* out, ga_stream stream);

/* ------------------------------------------------------------------------------------------
 * Serving over a 4-bit paged cache, with every length on the device. The pages have no
 * counterpart beyond paged caches and decode (pegainfer PR #1151, §Summary and §Limits); the
 * calls below are additions. One step of a server is
 *   ga_page_plan          pages, slots and positions of the step's tokens
 *   ga_qk_prologue_axes   their prepared keys and queries
 *   ga_kv_quantize_q4     their keys and values into the cache
 *   ga_attn_verify_q4     attention of every sequence's window over its cache
 * and reads no length on the host, so it can be captured once and replayed as they change.
 * The plan packs its tokens: a sequence that adds fewer moves the ones after it. They lie as the
 * attention's windows [n_seq][rows] do while every sequence in use adds `rows` tokens and idle
 * rows of the batch (length -1) stand at its end.
 * ------------------------------------------------------------------------------------------ */

#define GA_PLAN_MAX_SEQ 2048 /* sequences of one ga_page_plan call */
#define GA_Q4_PAGE_TOKENS 32 /* pages of a 4-bit cache hold a multiple of this many tokens */
#define GA_Q4_ROW_BYTES 128  /* code bytes of one (token, KV head) row of 256 values */
#define GA_Q4_SCALE_BYTES 16 /* scale bytes of one row */

/* Page tables, slot maps and positions of one step, from the sequences' lengths. Sequence b
 * holds held[b] pages (page_table row b, columns 0 .. held[b] - 1) and seq_len[b] cached
 * tokens, and adds new_len[b] tokens at positions seq_len[b] ..:
 *   new_len[b] >= 0, seq_len[b] >= 0: it needs ceil((seq_len + new_len) / page_size) pages; those
 *           it lacks are taken from the top of the stack of free pages, in order of sequence and
 *           then of page (the i-th is free_pages[count - 1 - i]), and appended to its row
 *   new_len[b] < 0:  it is finished: its held pages go back on the stack, on top of what the step
 *           left, in order of sequence and then of column, and it holds none. (Pages that other
 *           rows share must not be given back this way: ga_page_release.)
 *   seq_len[b] < 0 (and new_len[b] >= 0): the row is unused and left as it is
 * All arrays are DEVICE int32:
 *   seq_len, new_len, held [n_seq]; page_table [n_seq][max_pages], updated in place
 *   held_out [n_seq], may be held itself
 *   free_pages [n_free]: the stack, n_free the pages of the pool; free_count [1]: pages on it;
 *           free_count_out [1], may be free_count itself
 *   pos_delta NULL or [n_seq]: added to the positions of sequence b's tokens (text after images
 *           sits at other rotary positions than cache slots)
 *   row_start [n_seq + 1]: packed row of each sequence's first new token; the last is the total
 *   slot_map [max_tokens]: packed token t's cache slot, page * page_size + offset; -1 from the
 *           total on
 *   positions NULL or [max_tokens]: packed token t's position (seq_len + index + pos_delta); 0
 *           from the total on
 *   info    [4]: status, tokens, pages taken, pages given back. Status 0: done; 1: more than
 *           max_tokens tokens; 2: a sequence past max_pages * page_size or GA_MAX_TOKENS; 3: not
 *           enough free pages; 4: held or free_count out of range, or more pages given back than
 *           the stack has room for. Of several reasons the first of these counts: held or
 *           free_count (4), a sequence (2), the stack's room (4), tokens (1), free pages (3).
 *           When it is not 0 nothing is planned: page_table and
 *           free_pages keep their contents, held_out and free_count_out are copies, row_start
 *           and the totals are 0, every slot is -1.
 * Other than those pairs, no output may overlap an input or another output. The call takes one
 * launch up to 8,192 slots, two above.
 * With lengths of 0 and the cached lengths as new_len it lists the slots of cached tokens, for
 * ga_kv_dequantize_q4 to widen whole caches: no page is taken while the rows hold theirs.
 * Rules: 0 <= n_seq <= GA_PLAN_MAX_SEQ, page_size >= 1, 1 <= max_pages, max_pages * page_size
 * < 2^31, n_free * page_size < 2^31, 0 <= max_tokens < 2^30; every array 4-byte aligned. With
 * n_seq = 0, row_start, slot_map, positions and info are still written.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_page_plan(const int* seq_len, const int* new_len, int n_seq, int page_size,
                 int* page_table, int max_pages, const int* held, int* held_out, int* free_pages,
                 int n_free, const int* free_count, int* free_count_out, const int* pos_delta,
                 int max_tokens, int* row_start, int* slot_map, int* positions, int* info,
                 ga_stream stream);

/* ga_qk_prologue with positions from device memory, on up to four axes (time, height and width
 * of image and video tokens; all axes alike for text): rotary pair i (dims i and i + 32) of
 * token t turns by the angle of position positions[axis][t], axis = pair_axis[i]. The rounding
 * points are ga_qk_prologue's, and so are the bits where a token's positions are all the same.
 *   k_raw, w_k, k_prep  as in ga_qk_prologue, for n_tok tokens; or all three NULL
 *   qg, w_q, q_prep     as in ga_qk_prologue, for the same n_tok tokens; or all three NULL
 *   positions DEVICE int32 [n_axes][ld_pos], 4-byte aligned; ld_pos >= n_tok, or 0: one row
 *             [n_tok] for all axes. A position outside 0 .. table_rows - 1 is not a fault:
 *             status 4 is recorded (ga_device_status) and the pair turns by position 0.
 *   pair_axis HOST array of 32 bytes, each below n_axes (contiguous or interleaved sections)
 *   cos_tab, sin_tab [table_rows][32]
 * Rules: 1 <= n_axes <= 4, 0 <= n_tok <= GA_MAX_TOKENS, table_rows >= 1; no output may overlap an
 * input or the other output.
 * Errors: NULL, SHAPE, RANGE, TABLE (table_rows < 1), ALIGN, DEVICE, CUDA. */
int ga_qk_prologue_axes(const ga_bf16* k_raw, const ga_bf16* w_k, ga_bf16* k_prep,
                        const ga_bf16* qg, const ga_bf16* w_q, ga_bf16* q_prep, int n_tok,
                        const int* positions, long long ld_pos, int n_axes,
                        const uint8_t* pair_axis, const ga_bf16* cos_tab, const ga_bf16* sin_tab,
                        int table_rows, ga_stream stream);

/* 4-bit cache rows. A row of 256 values has 16 groups of 16; a group's scale is
 *   s = fp32(max|x| / 7), clamped to [2^-20, 3840] and rounded to 4 significant bits (ties to
 *       even), stored as the byte 8 E + m for s = 2^(E - 20) (1 + m / 8)
 * and a value's code is clamp(round(x / s), -8, 7) + 8 (ties to even), 4 bits. The widened value
 * (code - 8) * s is a bf16 value exactly. A NaN is stored as 0; values beyond the largest scale's
 * reach saturate. Any bytes are finite rows, so hidden positions need no initial contents.
 * Eight dims make a little-endian 32-bit word: bits 4p .. 4p+3 hold dim 2p for p < 4, dim
 * 2(p - 4) + 1 for p >= 4. Pools, per keys and values:
 *   codes   [n_pages][2][page_size][128] uint8, 16-byte aligned (head-major within a page)
 *   scales  [n_pages][2][page_size][16] uint8, 16-byte aligned
 * Slot x is position x % page_size of page x / page_size.
 * ga_kv_quantize_q4 stores token t's key and value rows at slots[t]:
 *   k, v    bf16 rows of two heads' 256 values, token t at t * ld_k (ld_v) values; 16-byte
 *           aligned, leading dimensions >= 512 and multiples of 8 (a slice of a fused projection)
 *   slots   DEVICE int32 [n_tok], 4-byte aligned, or NULL: token t goes to slot t. A negative
 *           slot stores nothing; one past the pool stores nothing and records status 3. Slots of
 *           one call must differ (two tokens of one slot leave an unspecified mixture).
 * Rules: page_size a multiple of 32, n_pages * page_size < 2^30, 0 <= n_tok <= 64 *
 * GA_MAX_TOKENS; with slots NULL, n_tok <= n_pages * page_size.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_kv_quantize_q4(const ga_bf16* k, long long ld_k, const ga_bf16* v, long long ld_v,
                      long long n_tok, const int* slots, uint8_t* k_codes, uint8_t* k_scales,
                      uint8_t* v_codes, uint8_t* v_scales, int n_pages, int page_size,
                      ga_stream stream);

/* The widened rows of the tokens at slots[0 .. n_tok - 1] (or slots 0 .. n_tok - 1 with NULL), as
 * the other entry points read them: a prefix of a 4-bit cache for ga_attn_prefill, say.
 *   k_out, v_out [n_tok][2][256] bf16, 16-byte aligned. Rows of negative or refused slots are
 *           left as they were. The same slot may appear more than once.
 * Everything else as in ga_kv_quantize_q4.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_kv_dequantize_q4(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                        const uint8_t* v_scales, int n_pages, int page_size, const int* slots,
                        long long n_tok, ga_bf16* k_out, ga_bf16* v_out, ga_stream stream);

/* Bytes of workspace ga_attn_verify_q4 needs, whatever the sequences and lengths. */
size_t ga_verify_q4_workspace_bytes(void);

/* Few-row verify windows, and decode (rows = 1), over 4-bit paged caches. Unlike the other
 * verify calls it takes prepared queries (their positions need not be their cache slots) and
 * lengths on the DEVICE, and it rounds the softmax weights and the output only: scores, O and
 * the gate stay in fp32. The same call gives the same bits; where a sequence's keys are cut
 * among the SMs, and so its last bits, depends on all the lengths of the call. A NaN query (or one
 * whose scores are infinite, or pass 2^29 in magnitude, which fp32 no longer tells apart) makes its
 * own head's row meaningless, mostly NaN, and no other.
 *   q_prep   [n_seq][rows][24][256] prepared queries (ga_qk_prologue_axes or ga_q_prologue)
 *   qg       [n_seq][rows][24][512] fused rows, read for their gate halves
 *   k_codes, k_scales, v_codes, v_scales, n_pages, page_size: the pools, as ga_kv_quantize_q4
 *            writes them (prepared keys); the window's own keys included
 *   page_table DEVICE int32 [n_seq][max_pages]: as in ga_attn_verify_paged; the entries that
 *            cover keys 0 .. L + rows - 1 are read, one outside the pool records status 3 and
 *            reads zero bytes
 *   seq_len  DEVICE int32 [n_seq]: L, the cached tokens before the window. Negative: an unused
 *            row, of which nothing is read and whose outputs are left as they were; L + rows
 *            past max_pages * page_size or GA_MAX_TOKENS records status 4 and is treated so too
 *   out      [n_seq][rows][24 * 256], row r over keys 0 .. L + r; may not overlap any input
 *   workspace >= ga_verify_q4_workspace_bytes() bytes, 256-byte aligned, not shared with a
 *            concurrent call (captured graphs that may run at once need one each); it needs no
 *            initial contents
 * Rules: 0 <= rows <= 16, page_size a multiple of 32 up to GA_MAX_TOKENS, n_pages * page_size
 * < 2^30. Nothing is allocated; the call keeps no pointer. n_seq = 0 or rows = 0 is a no-op.
 * Errors: NULL, SHAPE, RANGE, ALIGN, WORKSPACE, DEVICE, CUDA. */
int ga_attn_verify_q4(const ga_bf16* q_prep, const ga_bf16* qg, const uint8_t* k_codes,
                      const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                      int n_pages, int page_size, const int* page_table, int max_pages,
                      const int* seq_len, int n_seq, int rows, ga_bf16* out, void* workspace,
                      size_t ws_bytes, ga_stream stream);

/* ------------------------------------------------------------------------------------------
 * Serving over an 8-bit paged cache: ga_page_plan and ga_qk_prologue_axes as above, then
 *   ga_kv_quantize_q8     the step's keys and values into the cache
 *   ga_attn_verify_q8     attention of every sequence's window over its cache
 * (The e4m3 calls above take contiguous caches, a scale per row and lengths on the host.)
 * ------------------------------------------------------------------------------------------ */

#define GA_Q8_BLOCK_TOKENS 32 /* tokens of one head that share a scale; pages hold a multiple */
#define GA_Q8_ROW_BYTES 256   /* code bytes of one (token, KV head) row */

/* 8-bit cache rows: e4m3 codes with a power-of-two scale for each block of 32 tokens (slots 32 i ..
 * 32 i + 31) and head. A value's code is e4m3(x / 2^e), to nearest, ties to even, saturating; the
 * widened value code * 2^e is a bf16 value exactly. For the tokens that a call stores into a block,
 *   e = the least integer in [-32, 31] with max|x| <= 448 * 2^e over their rows (31 if none)
 * and, unless the block's first slot is among them, no less than the block's exponent was; where it
 * grows, the block's other codes become e4m3(code / 2^growth), so earlier rows keep their values
 * but for what falls under the smallest codes. A store of a block's first slot begins it anew: its
 * other codes are left as they are. So a block is filled from its first slot on, in any number of
 * calls; writing over its later slots (tokens taken back) is fine. A NaN is stored as 0; an
 * infinity saturates, and takes the block's exponent to 31. Pools, per keys and values:
 *   codes   [n_pages][2][page_size][256] uint8, 16-byte aligned (head-major within a page)
 *   scales  [n_pages][2][page_size / 32] uint8, any alignment: e + 32 in the low six bits (stores
 *           clear the others)
 * Slot x is position x % page_size of page x / page_size.
 * ga_kv_quantize_q8 stores token t's key and value rows at slots[t]:
 *   k, v    bf16 rows of two heads' 256 values, token t at t * ld_k (ld_v) values; 16-byte
 *           aligned, leading dimensions >= 512 and multiples of 8 (a slice of a fused projection)
 *   slots   DEVICE int32 [n_tok], 4-byte aligned, or NULL: token t goes to slot t. A negative
 *           slot stores nothing; one past the pool stores nothing and records status 3. Slots of
 *           one call must differ, and the tokens of one block follow one another in the call, with no
 *           other token and no skipped one between them, as ga_page_plan lists them (else that
 *           block's rows are unspecified).
 * Rules: page_size a multiple of 32, n_pages * page_size < 2^30, 0 <= n_tok <= 64 *
 * GA_MAX_TOKENS; with slots NULL, n_tok <= n_pages * page_size.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_kv_quantize_q8(const ga_bf16* k, long long ld_k, const ga_bf16* v, long long ld_v,
                      long long n_tok, const int* slots, uint8_t* k_codes, uint8_t* k_scales,
                      uint8_t* v_codes, uint8_t* v_scales, int n_pages, int page_size,
                      ga_stream stream);

/* The widened rows of the tokens at slots[0 .. n_tok - 1] (or slots 0 .. n_tok - 1 with NULL).
 *   k_out, v_out [n_tok][2][256] bf16, 16-byte aligned. Rows of negative or refused slots are
 *           left as they were. The same slot may appear more than once.
 * Codes 0x7F and 0xFF, which ga_kv_quantize_q8 never writes, widen to NaN. Everything else as in
 * ga_kv_quantize_q8.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_kv_dequantize_q8(const uint8_t* k_codes, const uint8_t* k_scales, const uint8_t* v_codes,
                        const uint8_t* v_scales, int n_pages, int page_size, const int* slots,
                        long long n_tok, ga_bf16* k_out, ga_bf16* v_out, ga_stream stream);

/* Bytes of workspace ga_attn_verify_q8 needs, whatever the sequences and lengths. */
size_t ga_verify_q8_workspace_bytes(void);

/* Few-row verify windows, and decode (rows = 1), over 8-bit paged caches: ga_attn_verify_q4's
 * arguments, rules, workspace rules and errors over the pools above (pages of a multiple of 32
 * tokens). Hidden positions need no initial contents: whatever their codes and scales, NaN codes
 * included, they do not reach a result. Queries and softmax weights meet the codes as sums of two
 * 8-bit parts: a query is within 2^-17 of its row's largest magnitude, a weight within 2^-9 of
 * itself or 2^-22 of the largest of its block of 32 keys (2^-15 where the scores pass 2^23); sums,
 * maxima and O are fp32, and the output is rounded once. Scores are fp32 too: large ones are known to
 * a few of their last steps (an eighth at 2^20), and their weights to match, but up to 2^29 a row's
 * weights are the same in its sum as in its output. A NaN query (or one whose scores are infinite, or
 * pass 2^29 in magnitude) makes its own head's row meaningless, and no other.
 * A page-table entry outside the pool records status 3 and its keys are read as zeros.
 * Errors: NULL, SHAPE, RANGE, ALIGN, WORKSPACE, DEVICE, CUDA. */
int ga_attn_verify_q8(const ga_bf16* q_prep, const ga_bf16* qg, const uint8_t* k_codes,
                      const uint8_t* k_scales, const uint8_t* v_codes, const uint8_t* v_scales,
                      int n_pages, int page_size, const int* page_table, int max_pages,
                      const int* seq_len, int n_seq, int rows, ga_bf16* out, void* workspace,
                      size_t ws_bytes, ga_stream stream);

/* ------------------------------------------------------------------------------------------
 * Pages that several sequences hold (branches over a shared prefix), beside ga_page_plan. Its
 * page_table, held, free_pages and free_count are these calls' too, with one count more:
 *   shared  DEVICE int32 [n_free]: the rows beyond the first that hold each page; 0 for a page of
 *           one row and for a free page, so pages that ga_page_plan takes need no entry
 * A row may append only to pages that it alone holds: ga_page_fork sees to that at the branch. A row
 * that is cut back (ga_page_release) into a page that others hold must not go on inside it; fork it
 * into an unused row and release it instead. ga_page_plan gives back a finished row's pages whoever
 * else holds them: rows that share pages are finished by ga_page_release.
 * All arrays are DEVICE int32, 4-byte aligned; an output may be the input of the same kind itself
 * (held_out held, and so on) and overlap nothing else. Each call reads every length on the device
 * and so can be captured once. A page-table entry outside the pool is not a fault: it records status
 * 3 (ga_device_status) and is passed over. info [4] begins with a status; when it is not 0 nothing
 * is done: tables, stacks and lists of free pages keep their contents, outputs are copies of their
 * inputs, copy and move lists are -1 throughout and info's other entries 0. Status 4: held or
 * free_count out of range.
 * ------------------------------------------------------------------------------------------ */

/* Forks: row child[i] becomes a branch of the first len[i] tokens of row parent[i]. It holds the
 * parent's whole pages of them with it (shared grows) and, where len[i] % page_size is not 0, a page
 * of its own, taken from the top of the stack in order of the forks, for the page begun, whose copy
 * is the caller's to make: ga_page_copy with the lists below, before either row is written to.
 *   parent, child, len [n_fork]; parent[i] < 0: an unused entry. A parent may appear any number of
 *           times. A child's row holds no page before (it need not be cleared)
 *   page_table [n_seq][max_pages], updated in place; held, held_out [n_seq]
 *   free_pages [n_free], read; free_count, free_count_out [1]; shared, shared_out [n_free]
 *   copy_src, copy_dst [n_fork]: the pages to copy, -1 for a fork without
 *   info    {status, forks made, pages taken, pages now held by one row more}. Status 1: a row
 *           outside 0 .. n_seq - 1, a parent as its own child, a child twice, or one that holds
 *           pages; 2: len[i] negative or past the pages that the parent holds; 3: not enough free
 *           pages. Of several reasons the first counts, in the order 4, 1, 2, 3.
 * The children's cached lengths (ga_page_plan's seq_len) are the caller's to set.
 * Rules: 0 <= n_fork, n_seq <= GA_PLAN_MAX_SEQ, page_size >= 1, max_pages >= 1, max_pages *
 * page_size < 2^31, n_seq * max_pages < 2^30, 0 <= n_free, n_free * page_size < 2^31.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_page_fork(const int* parent, const int* child, const int* len, int n_fork, int n_seq,
                 int page_size, int* page_table, int max_pages, const int* held, int* held_out,
                 const int* free_pages, int n_free, const int* free_count, int* free_count_out,
                 const int* shared, int* shared_out, int* copy_src, int* copy_dst, int* info,
                 ga_stream stream);

/* Pages given back: row b keeps the pages of its first keep[b] tokens and lets the others go (0: a
 * finished row, negative: a row left as it is). A page that other rows still hold loses a holder;
 * one that all its holders let go, in this call or before, goes on the stack, in order of row and
 * then of column (of several places of a page its first).
 *   keep [n_seq]; page_table [n_seq][max_pages], read; held, held_out [n_seq]
 *   free_pages [n_free]: entries from free_count on are written; free_count, free_count_out [1]
 *   shared, shared_out [n_free]
 *   info    {status, rows that let pages go, pages put on the stack, pages let go}. Status 4 also:
 *           more pages given back than the stack has room for; 5: a page let go more often than
 *           `shared` says that it is held. 4 for held or free_count counts first, then 5.
 * Rules: as ga_page_fork's.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_page_release(const int* keep, int n_seq, int page_size, const int* page_table,
                    int max_pages, const int* held, int* held_out, int* free_pages, int n_free,
                    const int* free_count, int* free_count_out, const int* shared,
                    int* shared_out, int* info, ga_stream stream);

/* Bytes of workspace ga_page_compact needs for a pool of n_free pages; 0 for a negative one. */
size_t ga_page_compact_workspace_bytes(int n_free);

/* Compaction: pages in use move down into free ones until they fill the front of the pool. With
 * n_live = n_free - free_count pages in use, move i takes the i-th highest page in use at or past
 * n_live to the i-th lowest free page below it, for the first max_moves of them (the budget of one
 * step). The pages' contents are the caller's to move: ga_page_copy with the lists below, before
 * either row is written to and before a page is taken from the new stack.
 *   page_table [n_seq][max_pages], its first held[b] columns; page_table_out of the same shape (its
 *           other columns are copies); held [n_seq], read
 *   free_pages [n_free], free_count [1]: the stack; its pages differ. free_pages_out [n_free]: the
 *           stack after, its lowest page on top (entries from free_count on are copies)
 *   shared, shared_out [n_free]: a page's count moves with it
 *   move_src, move_dst [max_moves]: the moves, then -1
 *   info    {status, moves, pages in use, moves left for another call}. Status 4 also: a free page
 *           outside the pool or twice on the stack.
 *   workspace >= ga_page_compact_workspace_bytes(n_free) bytes, 16-byte aligned, not shared with a
 *           concurrent call
 * Pages that are not on the stack are in use, whether or not a row holds them.
 * Rules: 0 <= n_seq <= GA_PLAN_MAX_SEQ, max_pages >= 1, n_seq * max_pages < 2^30, 0 <= n_free <
 * 2^30, 0 <= max_moves < 2^30.
 * Errors: NULL, SHAPE, RANGE, ALIGN, WORKSPACE, DEVICE, CUDA. */
int ga_page_compact(int n_seq, const int* page_table, int* page_table_out, int max_pages,
                    const int* held, const int* free_pages, int* free_pages_out, int n_free,
                    const int* free_count, const int* shared, int* shared_out, int max_moves,
                    int* move_src, int* move_dst, int* info, void* workspace, size_t ws_bytes,
                    ga_stream stream);

#define GA_PAGE_COPY_POOLS 16 /* pools of one ga_page_copy call */

/* Copies whole pages inside each of several pools: page src[i] to page dst[i], in all of them, one
 * launch. Any pools of pages do: bf16, 4-bit and 8-bit ones, codes and scales.
 *   pools      HOST array of n_pools DEVICE pointers; page p of pool j begins at byte p * page_bytes[j]
 *   page_bytes HOST array of n_pools sizes; any size and alignment is right, multiples of 16 at
 *              16-byte aligned addresses are fast
 *   src, dst   DEVICE int32 [n_copies], 4-byte aligned. An entry with either negative is passed
 *              over; one outside the pool is passed over and records status 3. No page is written
 *              twice, or read and written, in one call (else its contents are unspecified); a page
 *              may be read many times
 * Rules: 1 <= n_pools <= GA_PAGE_COPY_POOLS, n_pages >= 0, 1 <= page_bytes[j] <= 2^30, 0 <=
 * n_copies < 2^30. n_copies or n_pages = 0 is a no-op.
 * Errors: NULL, SHAPE, RANGE, ALIGN, DEVICE, CUDA. */
int ga_page_copy(void* const* pools, const size_t* page_bytes, int n_pools, int n_pages,
                 const int* src, const int* dst, int n_copies, ga_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* GA_ATTN_H */
