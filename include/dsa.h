/*
 * dsa.h - C ABI of libdsa.so: the DeepSeek Sparse Attention (DSA) layer hot
 * path on one NVIDIA GB300 (sm_103a).
 *
 * The path has three stages ("DeepSeek3.2: Onboard sparse attention",
 * Background): a lightning indexer that scores every causal (query, key)
 * pair, a per-query top-k that turns the scores into an index set, and
 * attention restricted to that set, forward and backward ("Support Ring
 * Attention with DeepSeek DSA Sparse Indexer", Forward Flow / Backward Flow).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - All pointers are DEVICE pointers owned by the caller, 16-byte aligned,
 *    to contiguous row-major tensors of the shapes given below. The library
 *    never allocates or frees device memory.
 *  - `stream` is a cudaStream_t (NULL = the legacy default stream). Every call
 *    only enqueues work on it and returns; nothing synchronises except
 *    dsa_get_last_device_error().
 *  - Every call returns a dsa_status. Arguments are validated on the host
 *    before anything is launched; an unsupported shape returns
 *    DSA_ERR_UNSUPPORTED and nothing runs (there is no fallback path).
 *  - Faults found on the device (an index outside [-1, S), a bounded wait that
 *    ran out) do not trap: the kernel records a code in a device error word,
 *    skips the bad access and finishes. Read it with
 *    dsa_get_last_device_error().
 *  - "Valid" pairs: key s is valid for query t when s <= t (the causal mask
 *    q_pos >= kv_pos, diagonal included; "Support Ring Attention with
 *    DeepSeek DSA Sparse Indexer", Forward Flow step 3) and, when segment ids
 *    are given, seg[b,s] == seg[b,t] (packed documents; same page, Tests:
 *    indexer mask with segment ids).
 *  - bf16 arguments are IEEE bfloat16 bit patterns; results are rounded to
 *    nearest even from fp32.
 */
#ifndef DSA_H_
#define DSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  DSA_OK = 0,
  DSA_ERR_INVALID_ARG = 1, /* null pointer, bad size, misaligned pointer */
  DSA_ERR_UNSUPPORTED = 2, /* well-formed but outside what the kernels implement */
  DSA_ERR_WORKSPACE = 3,   /* workspace pointer null or smaller than required */
  DSA_ERR_CUDA = 4,        /* a CUDA runtime / driver call failed */
  DSA_ERR_TIMEOUT = 5,     /* a bounded device-side wait ran out */
  DSA_ERR_DEVICE = 6       /* the device reported bad input (see the code) */
} dsa_status;

typedef enum { DSA_BF16 = 0, DSA_F32 = 1 } dsa_dtype;

/* Device error codes returned by dsa_get_last_device_error(). 0 = none. The
 * low byte is the kind, the next byte the stage that reported it. */
#define DSA_DEVERR_TIMEOUT 0x01   /* a bounded mbarrier wait ran out */
#define DSA_DEVERR_BAD_INDEX 0x02 /* an index outside [-1, S) was skipped */
#define DSA_DEVERR_MISALIGNED 0x03 /* shared memory not aligned as the kernel needs */
#define DSA_DEVERR_BAD_PAGE 0x04   /* a page or a length outside the cache was skipped */
#define DSA_STAGE_INDEXER 0x100
#define DSA_STAGE_TOPK 0x200
#define DSA_STAGE_FWD 0x300
#define DSA_STAGE_BWD 0x400
#define DSA_STAGE_LOSS 0x500
#define DSA_STAGE_LOSS_BWD 0x600
#define DSA_STAGE_CACHE 0x700
#define DSA_STAGE_LATENT 0x800
#define DSA_STAGE_EVICT 0x900

/* Human-readable name of a status. Never NULL. */
const char* dsa_status_string(int status);

/* Library version, e.g. 100 for 0.1.0. */
int dsa_version(void);

/*
 * Synchronise `stream`, then read and clear the device error word of the
 * current device. *code receives the first code recorded since the last read
 * (0 if none). Returns DSA_OK, or DSA_ERR_CUDA if the synchronisation failed.
 */
int dsa_get_last_device_error(void* stream, int32_t* code);

/*
 * dsa_index_scores - lightning-indexer scores.
 *
 * Defines ("DeepSeek3.2: Onboard sparse attention", Background: a per-head
 * q.k product gives the index score; "Implement QK attention head chunking
 * for CSA", Description: per-head products reduced over heads):
 *
 *     I[b,t,s] = sum_h w[b,t,h] * max(0, sum_d q_idx[b,t,h,d] * k_idx[b,s,d])
 *
 * for valid (t, s); -inf where s <= t but the document differs. Entries with
 * s > t are not written. Per-head products are never stored.
 *
 *   q_idx   bf16 [B, S, Hi, Di]
 *   k_idx   bf16 [B, S, Di]
 *   w       [B, S, Hi], fp32 (w_dtype = DSA_F32) or bf16 (DSA_BF16)
 *   seg     int32 [B, S] or NULL (NULL: one document per row)
 *   scores  fp32 [B, S, ld_scores], ld_scores >= S and a multiple of 4
 *
 * Supported: Hi in {1, 2, 4, ..., 128}, Di in {32, 64, 128}. Accumulation is
 * fp32 on the tensor cores; with inputs whose partial sums are all exact in
 * fp32 (e.g. small dyadic values) the result is exact.
 */
int dsa_index_scores(const void* q_idx, const void* k_idx, const void* w, int w_dtype,
                     const int32_t* seg, int B, int S, int Hi, int Di, float* scores,
                     int64_t ld_scores, void* stream);

/*
 * dsa_index_scores_fp8 - the same scores from 8-bit float inputs. The pages
 * note that the original indexer is an fp8 kernel over quantized activations
 * ("DeepSeek3.2: Onboard sparse attention", What this PR does, item 4). With a
 * positive scale c_s per key (k = c_s * k8):
 *
 *     I[b,t,s] = c_s * sum_h w[b,t,h] * max(0, sum_d q8[b,t,h,d] * k8[b,s,d])
 *
 * which equals the bf16 definition on the dequantized k, because ReLU is
 * positively homogeneous. A per-(query, head) scale of q belongs in w.
 *
 *   q_idx    e4m3 bytes [B, S, Hi, Di] (OCP FP8 E4M3: bias 7, no infinities)
 *   k_idx    e4m3 bytes [B, S, Di]
 *   k_scale  fp32 [B, S], every entry > 0, or NULL (all 1)
 *   w, seg, scores, ld_scores, stream: as for dsa_index_scores
 *
 * Supported: Hi in {1, 2, 4, ..., 128}, Di in {32, 64, 128}. The products run at
 * twice the bf16 tensor rate and accumulate in fp32; the scale is one fp32
 * multiply of the reduced score. Inputs that are small dyadic values (exact in
 * e4m3) with power-of-two scales give exact results, identical to
 * dsa_index_scores on the same values.
 */
int dsa_index_scores_fp8(const void* q_idx, const void* k_idx, const float* k_scale,
                         const void* w, int w_dtype, const int32_t* seg, int B, int S, int Hi,
                         int Di, float* scores, int64_t ld_scores, void* stream);

/*
 * dsa_topk - per-query top-k of the index scores ("DeepSeek3.2: Onboard
 * sparse attention", Background: non-parametric top-k token selection).
 *
 * For each (b, t) select m(t) = min(k, n(t)) valid keys (n(t) = number of
 * valid keys) with the largest score. Equal scores go to the lower key index;
 * -0.0 equals +0.0. Scores must not be NaN.
 *
 *   scores  fp32 [B, S, ld_scores]; only valid entries (s <= t) are read
 *   seg     int32 [B, S] or NULL
 *   idx     int32 [B, S, k] out: the selected keys in ascending order,
 *           slots m(t)..k-1 set to -1
 *   count   int32 [B, S] out, or NULL: m(t)
 *   vals    fp32 [B, S, k] out, or NULL: the score of the key in each slot of idx,
 *           -inf at slots holding -1. It is read back from the score row just after
 *           the row's selection (while the row is in L2), so that a consumer of the
 *           selected scores (dsa_indexer_loss with ld_scores = 0) reads k contiguous
 *           floats per row instead of gathering them from the row.
 *   ws      workspace of dsa_topk_workspace_size() bytes (may be NULL if 0)
 */
size_t dsa_topk_workspace_size(int B, int S, int k);
int dsa_topk(const float* scores, int64_t ld_scores, const int32_t* seg, int B, int S, int k,
             int32_t* idx, int32_t* count, float* vals, void* ws, size_t ws_bytes,
             void* stream);

/*
 * dsa_sparse_attn_fwd - attention over the selected keys ("Support Ring
 * Attention with DeepSeek DSA Sparse Indexer", Forward Flow step 5):
 *
 *     l_j = scale * Q[b,t,h] . K[b,s_j]      for the listed s_j with s_j <= t
 *     O[b,t,h] = sum_j softmax(l)_j V[b,s_j],   lse[b,t,h] = log sum_j exp(l_j)
 *
 * The selected set of query t is shared by all H heads. Entries of idx equal
 * to -1 and entries above the diagonal are ignored; a row with no key gets
 * O = 0 and lse = -inf. The entries of a row must be distinct.
 *
 *   Q    bf16 [B, S, H, Dqk]     K  bf16 [B, S, Hkv, Dqk]    V  bf16 [B, S, Hkv, Dv]
 *   idx  int32 [B, S, k]         O  bf16 [B, S, H, Dv] out   lse fp32 [B, S, H] out
 *
 * Supported: 1 <= H <= 128 and
 *  - Hkv = 1 (one K/V row shared by every head, the form the indexer's
 *    selection is built for): (Dqk, Dv) in {(32, 32), (64, 64), (128, 128),
 *    (192, 128)};
 *  - Hkv > 1 dividing H (per-head K/V, Hkv = H, or groups of H / Hkv heads;
 *    head h reads K/V head h / (H / Hkv)): the dense-tile kernel only, so
 *    (Dqk, Dv) in {(128, 128), (192, 128)}, S <= 65536 and a positive scale;
 *    DSA_ERR_UNSUPPORTED otherwise.
 *
 * Two tensor-core kernels compute it. One gathers each query's selected K/V
 * rows and puts the heads on the 128 lanes of a tile. The other evaluates dense
 * 128 x 128 (query, key) tiles of one head under a bitmap of the selection and
 * skips tiles without a selected key (see dsa_sparse_attn_fwd_dense). The call
 * takes the one with fewer tile products for the shape.
 *
 *   ws  workspace of dsa_sparse_attn_fwd_workspace_size() bytes, 16-byte aligned:
 *       the dense-tile kernel's selection bitmap and tile flags (overwritten). It
 *       is reserved whenever that kernel can take the shape, whichever kernel
 *       the call then picks; where the size is 0, ws may be NULL.
 *
 * DSA_ERR_WORKSPACE if ws is NULL, misaligned or smaller than the size (when the
 * size is not 0).
 */
size_t dsa_sparse_attn_fwd_workspace_size(int B, int S, int H, int Hkv, int Dqk, int Dv);
int dsa_sparse_attn_fwd(const void* Q, const void* K, const void* V, const int32_t* idx, int B,
                        int S, int H, int Hkv, int Dqk, int Dv, int k, float scale, void* O,
                        float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * dsa_sparse_attn_fwd_kernel - which kernel dsa_sparse_attn_fwd runs for a shape:
 * DSA_FWD_GATHER_TC (the gathered-key tensor-core kernel, one launch),
 * DSA_FWD_DENSE_TC (the dense-tile tensor-core kernel: a bitmap build and the
 * attention, two launches) or DSA_FWD_MMA_SYNC (one launch); the negated status
 * (-DSA_ERR_INVALID_ARG, -DSA_ERR_UNSUPPORTED) when the call would refuse the shape.
 * Launches nothing.
 */
#define DSA_FWD_GATHER_TC 0
#define DSA_FWD_DENSE_TC 1
#define DSA_FWD_MMA_SYNC 2
int dsa_sparse_attn_fwd_kernel(int B, int S, int H, int Hkv, int Dqk, int Dv, int k,
                               float scale);

/*
 * dsa_sparse_attn_fwd_dense - the same result from the dense-tile kernel only
 * (the pages' own design evaluates the masked logits as dense blocks with
 * partial mask blocks: "Support Ring Attention with DeepSeek DSA Sparse
 * Indexer", Forward Flow). Arguments, workspace included, as for
 * dsa_sparse_attn_fwd. Supported: any Hkv dividing H, 1 <= H <= 128, (Dqk, Dv)
 * in {(128, 128), (192, 128)}, S <= 65536, a positive scale; DSA_ERR_UNSUPPORTED
 * otherwise.
 */
int dsa_sparse_attn_fwd_dense(const void* Q, const void* K, const void* V, const int32_t* idx,
                              int B, int S, int H, int Hkv, int Dqk, int Dv, int k, float scale,
                              void* O, float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * dsa_sparse_attn_bwd - gradients of the sparse attention ("Support Ring
 * Attention with DeepSeek DSA Sparse Indexer", Backward Flow step 6:
 * dQ = dP.K, dK = dP^T.Q, dV = P^T.dO over the same mask, "dP" being the
 * gradient of the logits):
 *
 *     P_j recomputed from lse;  Delta = sum_c dO[c] O[c];  dS_j = P_j (dO.V[s_j] - Delta)
 *     dQ[t,h] = scale sum_j dS_j K[s_j];  dK[s] = scale sum dS Q;  dV[s] = sum P dO
 *
 *   Q, K, V, idx as for the forward; O, lse the forward's outputs;
 *   dO bf16 [B, S, H, Dv];  dQ bf16 [B, S, H, Dqk] out;
 *   dK bf16 [B, S, Hkv, Dqk] out;  dV bf16 [B, S, Hkv, Dv] out;
 *   ws  workspace of dsa_sparse_attn_bwd_workspace_size() bytes, 16-byte aligned
 *       (overwritten): the fp32 dK/dV accumulators [B*S*Hkv, Dqk + Dv] rounded up
 *       to 256 bytes, then, whenever the dense-tile kernels can take the shape,
 *       their selection bitmap, tile flags and Delta (fp32 [B, S, H]).
 *
 * Supported shapes as for the forward. dK/dV are summed with fp32 atomics, so
 * their rounding order is not fixed from run to run.
 */
size_t dsa_sparse_attn_bwd_workspace_size(int B, int S, int H, int Hkv, int Dqk, int Dv);
int dsa_sparse_attn_bwd(const void* Q, const void* K, const void* V, const int32_t* idx,
                        const void* O, const float* lse, const void* dO, int B, int S, int H,
                        int Hkv, int Dqk, int Dv, int k, float scale, void* dQ, void* dK, void* dV,
                        void* ws, size_t ws_bytes, void* stream);

/*
 * dsa_sparse_attn_bwd_dense - the same gradients from the dense-tile kernels only:
 * a dQ pass over (batch, head, query tile) items and a key-major dK / dV pass over
 * (batch, key tile, group of heads) items, both under the bitmap of the selection
 * (the pages' design: dense blocks with partial mask blocks and a key-major pass
 * for dK / dV, "Support Ring Attention with DeepSeek DSA Sparse Indexer",
 * Backward Flow). Arguments, workspace included, as for dsa_sparse_attn_bwd.
 * Supported: any Hkv dividing H, 1 <= H <= 128, (Dqk, Dv) in {(128, 128),
 * (192, 128)}, S <= 65536, a positive scale; DSA_ERR_UNSUPPORTED otherwise.
 * dsa_sparse_attn_bwd takes these kernels when they have fewer tile products for
 * the shape, and always for Hkv > 1; dsa_sparse_attn_bwd_noalloc never does (so
 * it takes Hkv = 1 only).
 */
int dsa_sparse_attn_bwd_dense(const void* Q, const void* K, const void* V, const int32_t* idx,
                              const void* O, const float* lse, const void* dO, int B, int S, int H,
                              int Hkv, int Dqk, int Dv, int k, float scale, void* dQ, void* dK, void* dV,
                              void* ws, size_t ws_bytes, void* stream);

/*
 * dsa_sparse_attn_bwd_kernel - which kernels dsa_sparse_attn_bwd runs for a shape:
 * DSA_BWD_GATHER_TC (gathered-key tensor-core kernel + finalize: 2 launches),
 * DSA_BWD_DENSE_TC (bitmap, dQ pass, dK / dV pass, finalize: 4 launches) or
 * DSA_BWD_MMA_SYNC (2 launches); the negated status when the call would refuse the
 * shape. Launches nothing.
 */
#define DSA_BWD_GATHER_TC 0
#define DSA_BWD_DENSE_TC 1
#define DSA_BWD_MMA_SYNC 2
int dsa_sparse_attn_bwd_kernel(int B, int S, int H, int Hkv, int Dqk, int Dv, int k,
                               float scale);

/*
 * dsa_sparse_attn_bwd_noalloc - dsa_sparse_attn_bwd for callers that cannot
 * allocate device memory. The pages have no counterpart: this is a
 * deployment variant of the same backward pass, not part of the method.
 *
 * Callers that are handed their input and output buffers by a host program
 * and cannot obtain more device memory (a plugin inside a runtime that owns
 * every allocation through its own pool, or code that must not call
 * cudaMalloc while it runs because an allocation there can fail or stall the
 * device) cannot pass the fp32 workspace of dsa_sparse_attn_bwd. This entry
 * point takes the same tensors without it and keeps the dK/dV accumulator in
 * a fixed array inside the library: DSA_NOALLOC_BWD_MAX_FLOATS floats
 * (32 MiB), held on every GPU that loads the library until the process exits.
 *
 *  - Limit: B * S * Hkv * (Dqk + Dv) must not exceed DSA_NOALLOC_BWD_MAX_FLOATS
 *    (e.g. 26214 tokens at Dqk + Dv = 320); larger calls return
 *    DSA_ERR_WORKSPACE and launch nothing.
 *  - Nothing is allocated or freed. The first call on a device looks up the
 *    array's device address (cudaGetSymbolAddress) with that device current;
 *    make that first call before any stream capture.
 *  - Every call shares the one array and zeroes the part it uses before
 *    accumulating, so calls whose work overlaps on the GPU (two streams, or
 *    two host threads) race and corrupt each other's dK/dV. Serialise them.
 *  - Arguments, supported shapes and results are those of dsa_sparse_attn_bwd
 *    with Hkv = 1 (per-head K/V needs the dense-tile kernels, whose scratch is
 *    part of dsa_sparse_attn_bwd's workspace).
 */
#define DSA_NOALLOC_BWD_MAX_FLOATS 8388608
int dsa_sparse_attn_bwd_noalloc(const void* Q, const void* K, const void* V, const int32_t* idx,
                                const void* O, const float* lse, const void* dO, int B, int S,
                                int H, int Hkv, int Dqk, int Dv, int k, float scale, void* dQ,
                                void* dK, void* dV, void* stream);

/*
 * dsa_index_topk - dsa_index_scores followed by dsa_topk, fused through blocks of
 * query rows: the [B, S, S] score matrix never exists. Each block of block_rows
 * query rows is scored into a [B, block_rows, ld] fp32 buffer in `ws` (ld = S
 * rounded up to a multiple of 4) and its top-k is taken before the next block
 * reuses the buffer, so the scores' memory is B * block_rows * ld * 4 bytes instead
 * of B * S * ld * 4 (at S = 131072 and block_rows = 2048: 1 GiB instead of 64 GiB),
 * and a small block keeps them in L2. "DeepSeek3.2: Onboard sparse attention"
 * (Background: the top-k of the index scores gives the index mask) and "Implement QK
 * attention head chunking for CSA" (the dense score products run out of memory at
 * long context).
 *
 *   q_idx, k_idx, w, w_dtype, seg, B, S, Hi, Di as for dsa_index_scores;
 *   k, idx [B, S, k], count [B, S] (or NULL), vals [B, S, k] (or NULL) as for dsa_topk
 *               (identical results);
 *   block_rows  query rows per block: a positive multiple of 256;
 *   ws          at least dsa_index_topk_workspace_size(B, S, block_rows) bytes.
 *
 * Supported as for dsa_index_scores (bf16 inputs). DSA_ERR_WORKSPACE if ws is too small.
 */
size_t dsa_index_topk_workspace_size(int B, int S, int block_rows);
int dsa_index_topk(const void* q_idx, const void* k_idx, const void* w, int w_dtype,
                   const int32_t* seg, int B, int S, int Hi, int Di, int k, int block_rows,
                   int32_t* idx, int32_t* count, float* vals, void* ws, size_t ws_bytes,
                   void* stream);

/*
 * dsa_index_topk_fp8 - dsa_index_topk on e4m3 q_idx / k_idx with an optional
 * per-key scale of k: dsa_index_scores_fp8 followed by dsa_topk, through blocks of
 * query rows. Arguments as for dsa_index_topk, plus k_scale as for
 * dsa_index_scores_fp8 (Di a multiple of 16).
 */
int dsa_index_topk_fp8(const void* q_idx, const void* k_idx, const float* k_scale, const void* w,
                       int w_dtype, const int32_t* seg, int B, int S, int Hi, int Di, int k,
                       int block_rows, int32_t* idx, int32_t* count, float* vals, void* ws,
                       size_t ws_bytes, void* stream);

/*
 * dsa_index_topk_stream - dsa_index_scores followed by dsa_topk, with no score row in
 * memory (the streaming form of the fused indexer + top-k; "Implement QK attention head
 * chunking for CSA", Description: the dense score products do not fit at long context).
 * Results are those of dsa_index_topk, bit for bit.
 *
 *  1. A sampled indexer pass scores evenly spaced 128-key tiles of each query group's
 *     causal range: a 16th of its tiles, at least 8 and at most 32 (all of them when
 *     there are fewer).
 *  2. From each row's sample, a window [L, U) around its k-th largest score: the sample's
 *     order statistics at rank k * (sampled) / (valid keys), +- 5 standard deviations.
 *  3. The full indexer pass keeps, per row, the keys scoring >= U (their indices, in the
 *     row's idx slots, and with vals their scores in the row's vals slots) and the keys in
 *     [L, U) (index and score, up to 4096), and stores no other score. Rows with at most
 *     k keys take every valid key this way (U = L = -inf).
 *  4. Each row is settled from these two lists: when at most k keys score >= U and the
 *     two lists together hold at least min(k, valid keys), the k-th largest score lies in
 *     the window and is found there; ties go to the lower key index as in dsa_topk.
 *  5. A row the lists cannot settle (the sample misplaced its window, or a list
 *     overflowed) marks its block of block_rows query rows; such blocks are redone by
 *     dsa_index_topk's memory form (indexer and top-k of the block's scores in `ws`),
 *     launches that a flag on the device switches on. On typical score distributions few
 *     or no blocks are redone.
 *
 *   q_idx, k_idx, w, w_dtype, seg, B, S, Hi, Di, k, idx, count, vals: as for
 *               dsa_index_topk; vals needs k <= 2048 (the scores of a row are staged by
 *               slot in shared memory), DSA_ERR_UNSUPPORTED otherwise;
 *   block_rows  rows per redone block: a positive multiple of 256;
 *   ws          at least dsa_index_topk_stream_workspace_size(B, S, block_rows) bytes:
 *               the samples (16 KB per query row), the window lists (32 KB per query row)
 *               and one block of fp32 scores (B * block_rows * S * 4 bytes).
 *
 * Supported as for dsa_index_scores, with S <= 131072; DSA_ERR_UNSUPPORTED otherwise.
 */
size_t dsa_index_topk_stream_workspace_size(int B, int S, int block_rows);
int dsa_index_topk_stream(const void* q_idx, const void* k_idx, const void* w, int w_dtype,
                          const int32_t* seg, int B, int S, int Hi, int Di, int k, int block_rows,
                          int32_t* idx, int32_t* count, float* vals, void* ws, size_t ws_bytes,
                          void* stream);

/*
 * dsa_index_topk_stream_fp8 - dsa_index_topk_stream on e4m3 q_idx / k_idx with an optional
 * per-key scale of k (as dsa_index_scores_fp8; Di a multiple of 16).
 */
int dsa_index_topk_stream_fp8(const void* q_idx, const void* k_idx, const float* k_scale,
                              const void* w, int w_dtype, const int32_t* seg, int B, int S, int Hi,
                              int Di, int k, int block_rows, int32_t* idx, int32_t* count,
                              float* vals, void* ws, size_t ws_bytes, void* stream);

/*
 * dsa_indexer_loss - the indexer's auxiliary loss and its gradient with respect
 * to the index scores.
 *
 * "Implement QK attention head chunking for CSA" gives the target: every head's
 * attention scores go through an fp32 softmax over the valid tokens, are zeroed
 * elsewhere, summed over the heads and held constant. "Support Ring Attention
 * with DeepSeek DSA Sparse Indexer" (Loss Harvesting & Objective Injection) adds
 * the loss to the objective so that its gradient trains the indexer. The pages
 * do not print the loss itself; this library reads it as the KL divergence
 * between the head-averaged target and the softmax of the index scores, both
 * over the query's selected keys (slots j with 0 <= s_j = idx[b,t,j] <= t):
 *
 *   pbar_j = (1/H) sum_h exp(scale Q[b,t,h].K[b,s_j] - lse[b,t,h])
 *   q_j    = softmax_j(scores[b,t,s_j])
 *   kl[b,t]   = sum_j pbar_j (log pbar_j - log q_j)          (0 log 0 = 0)
 *   dI[b,t,j] = grad_scale (q_j - pbar_j)   (0 at slots without a selected key)
 *
 * dI is the gradient of grad_scale * sum_{b,t} kl[b,t] with respect to the score
 * at each slot: pass it to dsa_indexer_loss_bwd.
 *
 *   Q      bf16 [B, S, H, Dqk]     K    bf16 [B, S, Hkv, Dqk]
 *   idx    int32 [B, S, k]          lse  fp32 [B, S, H] (from dsa_sparse_attn_fwd)
 *   scores fp32 [B, S, ld_scores]   only the selected entries are read; or, with
 *          ld_scores = 0, fp32 [B, S, k]: the selected keys' scores slot by slot (the
 *          `vals` of dsa_topk / dsa_index_topk / dsa_index_topk_stream), read contiguously
 *   kl     fp32 [B, S] out          dI   fp32 [B, S, k] out
 *
 * Hkv divides H (head h reads K head h / (H / Hkv)). The tensor-core kernel takes
 * Hkv = 1, 1 <= H <= 128, Dqk in {128, 192} and scale > 0; every other shape runs on
 * the CUDA cores (one CTA per query row, far slower). Rows with no selected key get
 * kl = 0 and dI = 0. An index outside [-1, S) is skipped and
 * recorded as DSA_STAGE_LOSS | DSA_DEVERR_BAD_INDEX. kl is accumulated with
 * atomics (summation order unspecified).
 */
int dsa_indexer_loss(const void* Q, const void* K, const int32_t* idx, const float* lse,
                     const float* scores, int64_t ld_scores, int B, int S, int H, int Hkv,
                     int Dqk, int k, float scale, float grad_scale, float* kl, float* dI,
                     void* stream);

/*
 * dsa_indexer_loss_bwd - the gradient of the indexer loss with respect to the
 * indexer's inputs, given dI from dsa_indexer_loss. With
 * I[t,s] = sum_h w[t,h] max(0, z_h), z_h = q_idx[t,h].k_idx[s] (the index score
 * of dsa_index_scores) and the derivative of max(0, z) at z = 0 taken as 0:
 *
 *   dw[b,t,h]     = sum_j dI[b,t,j] max(0, z_hj)
 *   dq_idx[b,t,h] = sum_j dI[b,t,j] w[b,t,h] [z_hj > 0] k_idx[b,s_j]
 *   dk_idx[b,s]   = sum over (t, j) with s_j = s of sum_h dI[b,t,j] w[b,t,h] [z_hj > 0] q_idx[b,t,h]
 *
 * over the selected slots (0 <= s_j <= t).
 *
 *   q_idx  bf16 [B, S, Hi, Di]   k_idx bf16 [B, S, Di]   w fp32 [B, S, Hi]
 *   idx    int32 [B, S, k]       dI    fp32 [B, S, k]
 *   dq_idx fp32 [B, S, Hi, Di] out   dk_idx fp32 [B, S, Di] out   dw fp32 [B, S, Hi] out
 *
 * Hi = 64, Di = 128 run on the tensor cores, with G = dI w [z > 0] rounded to bf16
 * and fp32 accumulation; other shapes on the CUDA cores in fp32 (one CTA per query
 * row, far slower), up to Hi * (Di + 1) <= 51200 (DSA_ERR_UNSUPPORTED above). dk_idx
 * is accumulated with fp32 atomics (summation order unspecified).
 */
int dsa_indexer_loss_bwd(const void* q_idx, const void* k_idx, const float* w,
                         const int32_t* idx, const float* dI, int B, int S, int Hi, int Di,
                         int k, float* dq_idx, float* dk_idx, float* dw, void* stream);

/*
 * ---------------------------------------------------------------- serving
 *
 * The layer of a model that answers token by token: rotary positions, a paged cache of
 * latent rows, and the attention of the newest tokens over it (the absorbed form of
 * multi-head latent attention, whose keys and values are one shared vector per token, so
 * that the selection of the indexer gathers one row per key: "DeepSeek3.2: Onboard sparse
 * attention", Background).
 */

/*
 * dsa_rope - rotary positions on dims [off, off + rot) of each head; the other dims are
 * copied. With i = 0 .. rot/2 - 1, t = pos[n] * inv_freq[i] and (a, b) the dims
 * (off + 2i, off + 2i + 1) in DSA_ROPE_INTERLEAVED or (off + i, off + rot/2 + i) in
 * DSA_ROPE_HALF:
 *
 *     y_a = mscale (x_a cos t - x_b sin t),   y_b = mscale (x_a sin t + x_b cos t)
 *
 * inverse != 0 takes -t. The map is linear in x and its transpose is the map at -t, so the
 * gradient of x is dsa_rope(dy) with inverse toggled and the same mscale.
 *
 *   x, y      [T, H, D], bf16 (dtype = DSA_BF16) or fp32 (DSA_F32); y = x rotates in place,
 *             any other overlap is refused (DSA_ERR_INVALID_ARG)
 *   pos       int32 [T], any value (the angle is reduced exactly: far positions lose nothing)
 *   inv_freq  fp32 [rot / 2], finite, radians per position
 *
 * Supported: D <= 1024 and off multiples of 8, rot a multiple of 16 with off + rot <= D. The
 * arithmetic is fp32, rounded once.
 */
#define DSA_ROPE_INTERLEAVED 0
#define DSA_ROPE_HALF 1
int dsa_rope(const void* x, void* y, int dtype, const int32_t* pos, const float* inv_freq, int T,
             int H, int D, int off, int rot, int layout, float mscale, int inverse, void* stream);

/*
 * The paged latent cache: rows of Dc latent and Dr positional dims, page_size rows to a page,
 * uint8 [num_pages, page_size, dsa_cache_row_bytes(fmt, Dc, Dr)]; slot s is row s % page_size
 * of page s / page_size.
 *
 *   DSA_CACHE_BF16  the Dc + Dr dims in bf16
 *   DSA_CACHE_E4M3  Dc e4m3 bytes; one fp32 scale per 128 of them (the scales padded with
 *                   zeros to a multiple of 16 bytes); the Dr dims in bf16. A scale is the
 *                   smallest power of two 2^k, k >= -120, with max|x| <= 448 * 2^k over its
 *                   128 dims (1 if they are all zero), and a byte is x / 2^k rounded to nearest
 *                   even: within half an e4m3 step (2^-4 of the value, 2^-10 * 2^k for the
 *                   smallest ones). A power of two keeps the read back exact in bf16 (a
 *                   magnitude above 1.9375 * 2^127 rounds up and reads back as an infinity).
 *                   A group with an infinity or a NaN reads back as NaN. The readers take rows as
 *                   dsa_cache_write makes them: of a scale that is no power of two, or a NaN byte
 *                   under a finite scale, dsa_cache_read and dsa_latent_attn may make different
 *                   values.
 *
 * Supported: Dc a multiple of 128, 128 <= Dc <= 1024; Dr a multiple of 8, 0 <= Dr <= 256.
 * dsa_cache_row_bytes returns 0 for anything else.
 */
#define DSA_CACHE_BF16 0
#define DSA_CACHE_E4M3 1
size_t dsa_cache_row_bytes(int fmt, int Dc, int Dr);

/*
 * dsa_cache_write - rows kv (bf16 [T, Dc + Dr]) into the slots slots[T] (int32) of the cache.
 * Slot -1 skips its row (padding); a slot outside [-1, num_slots) is skipped and recorded as
 * DSA_STAGE_CACHE | DSA_DEVERR_BAD_INDEX. The slots >= 0 must be distinct. Every other byte of
 * the cache is left as it was.
 */
int dsa_cache_write(const void* kv, const int32_t* slots, int T, int Dc, int Dr, int fmt,
                    void* cache, int64_t num_slots, void* stream);

/*
 * dsa_cache_read - the values of the rows at slots[N] (int32, repeats allowed) as bf16
 * kv [N, Dc + Dr]. Slot -1 gives a row of zeros; so does one outside [-1, num_slots), which
 * is recorded as DSA_STAGE_CACHE | DSA_DEVERR_BAD_INDEX.
 */
int dsa_cache_read(const void* cache, int64_t num_slots, int fmt, const int32_t* slots, int N,
                   int Dc, int Dr, void* kv, void* stream);

/*
 * dsa_latent_attn - attention of the Sq newest tokens of each sequence over its cached rows.
 * With len = lens[b] the cached tokens of sequence b, its Sq new ones among them (they are
 * written first), token i stands at position len - Sq + i and sees the positions up to its
 * own:
 *
 *     l_j = scale * Q[b,i,h] . row_j[0 : Dc+Dr]      0 <= j <= len - Sq + i
 *     O[b,i,h] = sum_j softmax(l)_j row_j[0 : Dc],   lse[b,i,h] = log sum_j exp(l_j)
 *
 * over every such j (idx = NULL), or over the listed ones (in a time that goes by k, however many of
 * its entries are -1): idx[b,i,:] as dsa_topk gives them
 * (-1 entries and entries above the token's position are ignored, entries must be distinct; an
 * entry below -1 or >= len is skipped and recorded as DSA_STAGE_LATENT |
 * DSA_DEVERR_BAD_INDEX). Position j of sequence b is row j % page_size of page
 * page_table[b, j / page_size]. A token with no key (len < Sq - i, or an empty list) gets O = 0
 * and lse = -inf; a sequence with len <= 0 is skipped that way (padding). A length below 0 or
 * above max_pages * page_size is taken as the nearest of the two, and a page outside
 * [0, num_pages) is skipped as if its keys were not there; both are recorded as
 * DSA_STAGE_LATENT | DSA_DEVERR_BAD_PAGE. Rows of the cache that no token sees are not read. A NaN
 * in a row, or an infinity that makes a logit +inf or NaN, reaches every token that sees the row
 * (O and lse are NaN) and no other; a logit of -inf is a weight of zero.
 *
 *   Q     bf16 [B, Sq, H, Dc + Dr]        cache      as above, num_pages * page_size slots
 *   lens  int32 [B]                       page_table int32 [B, max_pages]
 *   idx   int32 [B, Sq, k] or NULL (k = 0)
 *   O     bf16 [B, Sq, H, Dc] out         lse        fp32 [B, Sq, H] out
 *   ws    workspace of dsa_latent_attn_workspace_size() bytes (overwritten): the parts of
 *         rows whose keys are split over the GPU. Nothing is kept in it between calls.
 *
 * Supported: (Dc, Dr) = (512, 64), 1 <= H <= 128, 0 < scale <= 2e38, page_size >= 1,
 * num_pages * page_size < 2^31, max_pages * page_size < 2^31, B * Sq * H < 2^31. Q . row_j counts
 * as an infinity where it is past fp32 (its products with scale may be: O is right all the same,
 * and lse the nearest fp32, an infinity past its range). The weights are rounded to bf16 for
 * their product with the rows, sums are fp32 in a fixed order (the same bits every time).
 */
size_t dsa_latent_attn_workspace_size(int B, int Sq, int H, int Dc, int Dr, int k);
int dsa_latent_attn(const void* Q, const void* cache, int fmt, int64_t num_pages, int page_size,
                    const int32_t* page_table, int max_pages, const int32_t* lens,
                    const int32_t* idx, int k, int B, int Sq, int H, int Dc, int Dr, float scale,
                    void* O, float* lse, void* ws, size_t ws_bytes, void* stream);

/*
 * dsa_latent_attn_shared - dsa_latent_attn for sequences that share long prefixes, each stored once
 * in the cache: the prefix of group g is prefix_lens[g] positions in the pages prefix_table[g,:], and
 * the sequences starts[g] <= b < starts[g+1] are its group (G + 1 starts that go up; a sequence in
 * front of the first or behind the last has no prefix). Token i of sequence b sees every position of
 * its group's prefix, then its own positions 0 <= j <= lens[b] - Sq + i in the pages page_table[b,:];
 * lens counts the sequence's own positions, its Sq new ones among them:
 *
 *     O[b,i,h] = sum softmax(l) row[0 : Dc],   lse[b,i,h] = log sum exp(l),   l = scale * Q[b,i,h] . row
 *
 * over both. The rows of a group's prefix are read for up to 128 (token, head) pairs of the group at
 * once, whatever sequences they belong to; the two parts are joined in fp32. With fewer than 128 pairs a
 * sequence (Sq * H) that saves most of the time over the prefix; from 128 on, dsa_latent_attn with the
 * prefix's pages in front of each sequence's own (where the prefix ends with a page) is 1 to 9% quicker
 * over many sequences, and this call over a few. A token that has no
 * position of its own (len < Sq - i: padding) sees no prefix either: O = 0 and lse = -inf.
 *
 *   prefix_table int32 [G, max_prefix_pages]   prefix_lens int32 [G]   starts int32 [G + 1]
 *   Q, cache, page_table, lens, O, lse as for dsa_latent_attn
 *   ws    workspace of dsa_latent_attn_shared_workspace_size() bytes (overwritten). Nothing is kept in it
 *         between calls. It holds fp32 parts of 128 rows, 2056 bytes a row, whether rows are used or not:
 *             B * Sq * H / 128 + min(G, B)   for the rows of the groups (each group's rounded up),
 *             B * ceil(Sq * H / 128)         for those of the sequences,
 *             80                             for tiles that are split over the GPU
 *         (of B * Sq * H rows rounded up to 32 where those are fewer than 128). With few heads and many
 *         sequences that is a part of 263 KB a sequence: 40 MB for 64 sequences of 16 heads, 308 MB for
 *         1024 of 8, 1.1 GB for 4096 of one.
 *
 * Lengths, prefix lengths and pages outside their range are treated and recorded as by
 * dsa_latent_attn; a start below the one in front of it, below 0 or above B is taken as the nearest
 * that is not and recorded as DSA_STAGE_LATENT | DSA_DEVERR_BAD_INDEX. Infinities, NaNs, roundings and
 * the order of sums as for dsa_latent_attn.
 *
 * Supported: as for dsa_latent_attn, with 1 <= G <= 64, max_prefix_pages * page_size < 2^31 and
 * B * Sq * H < 2^30.
 */
size_t dsa_latent_attn_shared_workspace_size(int B, int Sq, int H, int G, int Dc, int Dr);
int dsa_latent_attn_shared(const void* Q, const void* cache, int fmt, int64_t num_pages,
                           int page_size, const int32_t* prefix_table, int max_prefix_pages,
                           const int32_t* prefix_lens, const int32_t* starts, int G,
                           const int32_t* page_table, int max_pages, const int32_t* lens, int B,
                           int Sq, int H, int Dc, int Dr, float scale, void* O, float* lse, void* ws,
                           size_t ws_bytes, void* stream);

/*
 * Eviction from the cache by accumulated attention weight: dsa_cache_mass adds up what weight each
 * cached position receives, dsa_cache_keep chooses the positions that stay within a budget, and
 * dsa_cache_compact moves their rows.
 */

/*
 * dsa_cache_mass - the attention weight that each cached position receives from the Sq newest tokens
 * of its sequence, summed over tokens and heads and added to that of earlier steps. With len = lens[b]
 * as for dsa_latent_attn (or the sequences' own positions, for dsa_latent_attn_shared) and lse the one
 * that the attention gave for the same Q:
 *
 *     mass[b,j] = decay * prev[b,j] + sum_{i,h} exp(scale * Q[b,i,h] . row_j - lse[b,i,h]),   j < len
 *
 * over the tokens i that see j (j <= len - Sq + i), or, with lists idx[b,i,:] as dsa_latent_attn takes
 * them, over those whose list names it. mass[b,j] = 0 for j >= len. prev NULL: no earlier weight.
 *
 *   Q, cache, page_table, lens, idx, k as for dsa_latent_attn     lse  fp32 [B, Sq, H]
 *   prev  fp32 [B, n] or NULL     mass fp32 [B, n] out; may be prev itself, any other overlap is refused
 *   ws    workspace of dsa_cache_mass_workspace_size() bytes (0: none needed), overwritten: the lists'
 *         weights, or the parts of sums that are split over the GPU
 *
 * A token whose lse is -inf adds nothing (it has no key); a NaN in lse, in Q or in a row reaches the
 * positions that it bears on. Q . row_j counts as an infinity where it is past fp32; where it is not, a
 * token whose lse is +inf (a logit of it is past fp32) adds nothing. Lengths, list entries
 * and pages outside their range are treated as by dsa_latent_attn and recorded with DSA_STAGE_EVICT;
 * positions n and behind are left out, and a length above n is recorded as DSA_DEVERR_BAD_PAGE. The
 * arithmetic is fp32: products of bf16 exact, sums in a fixed order (the same bits every time). Q . row_j is
 * added up by the tensor cores in two accumulators, and they cut off what lies behind an addition's last bit
 * instead of rounding it: with logits of ordinary size a weight is off by about 7e-7 of itself.
 *
 * Supported: as for dsa_latent_attn, with a finite decay, n <= 2^30 and, with lists, B * Sq * k and
 * B * (n / 8192 + 1) below 2^31.
 */
size_t dsa_cache_mass_workspace_size(int B, int Sq, int H, int Dc, int Dr, int k);
int dsa_cache_mass(const void* Q, const void* cache, int fmt, int64_t num_pages, int page_size,
                   const int32_t* page_table, int max_pages, const int32_t* lens,
                   const int32_t* idx, int k, const float* lse, int B, int Sq, int H, int Dc, int Dr,
                   float scale, const float* prev, float decay, float* mass, int n, void* ws,
                   size_t ws_bytes, void* stream);

/*
 * dsa_cache_keep - the positions of each sequence that stay when it is cut to `budget`: its first
 * `sink` ones, its `recent` newest ones, and of the others the budget - sink - recent heaviest by
 * mass (ties go to the lower position, -0 counts as +0, a NaN as heavier than any number). A
 * sequence of at most `budget` positions keeps all of them.
 *
 *   mass   fp32 [B, n]          lens   int32 [B]: the positions that a sequence has
 *   keep   int32 [B, budget] out: ascending, -1 behind the last
 *   count  int32 [B] out: min(lens[b], budget), the sequence's new length
 *
 * A length below 0 or above n is taken as the nearest of the two and recorded as
 * DSA_STAGE_EVICT | DSA_DEVERR_BAD_PAGE. Entries of mass at or behind a sequence's length are not
 * read. Supported: sink >= 0, recent >= 0, sink + recent <= budget, 1 <= budget <= 2^30,
 * 1 <= n <= 2^30, B <= 2^27.
 */
int dsa_cache_keep(const float* mass, int n, const int32_t* lens, int B, int budget, int sink,
                   int recent, int32_t* keep, int32_t* count, void* stream);

/*
 * dsa_cache_compact - moves rows of the cache: position j of sequence b becomes what its position
 * keep[b,j] was (bytes are copied, in either format). keep int32 [B, budget] as dsa_cache_keep gives
 * it: ascending, -1 behind the last; lens int32 [B], page_table int32 [B, max_pages]: the sequences
 * before the move.
 *
 *   new_table  int32 [B, new_max_pages]: the pages that the kept rows go to, none of them in use by
 *              any sequence (new_max_pages * page_size >= budget); or NULL: the rows go to the front
 *              of the sequence's own pages, which no other sequence may share
 *   mass       fp32 [B, n] or NULL: moved with the rows into new_mass fp32 [B, new_n]
 *              (new_n >= budget): new_mass[b,j] = mass[b, keep[b,j]], zero behind the last. new_mass
 *              may be mass itself (new_n = n); any other overlap is refused.
 *
 * An entry outside [-1, lens[b]) moves nothing and is recorded as DSA_STAGE_EVICT |
 * DSA_DEVERR_BAD_INDEX, and so is, in place, one below its own place j. Where the weights alone move in
 * place (new_mass = mass, new pages), an entry below its own place moves its row, its weight becomes 0 and
 * it is recorded the same way; so does, wherever the weights go, an entry at n or behind. A page outside
 * [0, num_pages) moves no row (the weight moves all the same); it and a length below 0 or above
 * max_pages * page_size (taken as the nearest of the two) are recorded as DSA_STAGE_EVICT |
 * DSA_DEVERR_BAD_PAGE. Every other byte of the cache stays as it was.
 *
 * Supported: Dc and Dr as for the cache, budget <= 2^30, n and new_n <= 2^30, page_size >= 1,
 * num_pages * page_size, max_pages * page_size and new_max_pages * page_size below 2^31; in place,
 * B <= 65535; to new pages, B * budget below 2^37.
 */
int dsa_cache_compact(void* cache, int fmt, int64_t num_pages, int page_size,
                      const int32_t* page_table, int max_pages, const int32_t* lens,
                      const int32_t* keep, int budget, const int32_t* new_table, int new_max_pages,
                      int B, int Dc, int Dr, const float* mass, int n, float* new_mass, int new_n,
                      void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_H_ */
