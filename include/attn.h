/*
 * attn.h - C ABI of libattn: chunked causal self-attention on GB300 (sm_103a).
 *
 * The operation: causal softmax attention computed subsequence by subsequence.
 * The query rows of chunk i attend to the resident keys/values of everything
 * before them (the chunk's context) and to themselves.
 *   - SPPO, "Efficient Long-sequence LLM Training via Adaptive Sequence Pipeline
 *     Parallel Offloading": §3.2 (FLOPs-based vs length-based partition), §4
 *     (multiplexing sequence partition: edge subsequences re-split, results
 *     combined), §5.1 (attention of subsequence i reads all K/V so far, which
 *     stay resident on the GPU).
 *   - InfiniPipe, "Elastic Pipeline Parallelism for Efficient Variable-Length
 *     Long-Context LLM Training": §II-A (a slice's queries see only preceding
 *     keys; K/V gradients depend on later slices), §II-B (packed [sum(S), D]
 *     layout), §III-A1 (chunk = {context C, slice lengths S}).
 *   - "Sequence Parallelism: Long Sequence Training from System Perspective"
 *     (blog summary), Deep Dive "Ring Self-Attention": a chunk's output is the
 *     accumulation of one partial per key/value block.
 *
 * Definition computed (one batch row b, head h; scale given by the caller):
 *   key j is visible to query t  iff  chunk(t).ctx_begin <= j <= t
 *   LSE_t = ln sum_{j visible} exp(scale * q_t . k_j)
 *   O_t   = sum_{j visible} exp(scale * q_t . k_j - LSE_t) v_j
 * and its gradient dQ, dK, dV for an upstream dO.
 *
 * Conventions shared by every entry point
 *   - Device pointers are CUDA device memory owned by the caller. The library
 *     never allocates, frees or retains device memory; the caller passes a
 *     workspace sized by attn_workspace_size().
 *   - q, k, v, o, dout, dq, dk, dv: bf16 (IEEE bfloat16), element (b, t, h, d)
 *     at  b*sb + t*st + h*sh + d  (strides in elements, d contiguous), the same
 *     strides for all eight tensors. Dense [B, H, L, D]: sb = H*L*D, sh = L*D,
 *     st = D. Packed [T, H, D] (B = 1): st = H*D, sh = D.
 *     Base pointers must be 16-byte aligned and sb, st, sh multiples of 8.
 *   - Head dim D: any multiple of 8 from 8 to 256 (InfiniPipe §III-A2 Eq. (3)
 *     carries D and D_kv as model dimensions). The tile kernels work on 64
 *     (D <= 64), 128 (D <= 128) or 256 dims; the dims past D are loaded as
 *     zeros, which leaves every score, output and gradient unchanged, and are
 *     never written. Throughput in FLOP of the true D is therefore D/64,
 *     D/128 or D/256 of that at the tile width. Above 128 dims the backward
 *     splits each 128-key tile into two work items, one per 128 output dims,
 *     which both compute the tile's scores and score gradients: it does 7/5
 *     of the backward's tensor work.
 *   - Grouped key/value heads (GQA/MQA): with Hkv > 0 in the shape, k, v, dk,
 *     dv (and the fp32 accumulators of attn_bwd_chunk) have Hkv heads and
 *     their own strides sb_kv, st_kv, sh_kv; query head h reads key/value head
 *     h / (H / Hkv), and the gradient of a key/value head is the sum over its
 *     H / Hkv query heads. Hkv = 0 means Hkv = H with the query strides.
 *   - lse: fp32, [B][H][T] contiguous, natural log.
 *   - stream: a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Compute calls only enqueue work and return before it completes.
 *   - chunks: a HOST array read during the call only. Each compute call lays
 *     out its work list on the host and writes it into the workspace with
 *     small copy kernels on `stream` that carry it in their launch
 *     parameters (up to 31 KB per launch), so nothing on the device refers to
 *     host memory after the call returns.
 *   - Every call returns an attn status code. Argument errors are detected on
 *     the host before anything is enqueued. Device-side errors are recorded in
 *     the workspace and read with attn_status(): ATTN_E_TIMEOUT (a bounded
 *     wait gave up) and ATTN_E_BOUNDS (a work descriptor in the workspace did
 *     not fit the shape or the workspace; every kernel checks each descriptor
 *     before it forms an address from it, and skips it). No entry point traps
 *     or aborts.
 */
#ifndef ATTN_H_
#define ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define ATTN_OK             0
#define ATTN_E_INVAL        1  /* bad shape, chunk table, mode or pointer      */
#define ATTN_E_ALIGN        2  /* pointer or stride not 16-byte aligned        */
#define ATTN_E_UNSUPPORTED  3  /* head dim not a multiple of 8 in [8, 256] */
#define ATTN_E_WORKSPACE    4  /* workspace NULL or smaller than required      */
#define ATTN_E_CUDA         5  /* a CUDA runtime call or kernel launch failed  */
#define ATTN_E_TIMEOUT      6  /* device: a bounded wait gave up               */
#define ATTN_E_BOUNDS       7  /* device: an index check failed                */
#define ATTN_E_CAPACITY     8  /* output array of attn_plan* too small; device: too few pages */

/* ---- plan modes (SPPO §3.2, §4) ---------------------------------------- */
#define ATTN_PLAN_UNIFORM              0  /* length-based: equal 128-multiples  */
#define ATTN_PLAN_FLOPS                1  /* FLOPs-based: b_k ~ L*sqrt(k/N)     */
#define ATTN_PLAN_FLOPS_RESPLIT_EDGES  2  /* FLOPS + first/last chunk re-split  */

/* One chunk (InfiniPipe §III-A1 split chunk {C, s}): query rows
 * [q_begin, q_end) with context C = q_begin - ctx_begin. ctx_begin is the
 * first visible key (the document start). kv_split = 0: no re-split; m with
 * ctx_begin < m < q_end: the chunk's key range is cut into [ctx_begin, m) and
 * [m, q_end); -P (2 <= P <= 64): the key range is cut into P parts carrying
 * equal numbers of visible (query, key) pairs of the chunk's queries, at the
 * multiples of 128 from ctx_begin nearest to the equal-pair points (ties up;
 * an error if they collapse). Each part is computed as a partial and the
 * parts are merged by log-sum-exp (SPPO §4 multiplexing, read as a key/value
 * split). */
typedef struct {
    int32_t q_begin, q_end;
    int32_t ctx_begin;
    int32_t kv_split;
} attn_chunk;

typedef struct {
    int64_t B, H, T, D;   /* batch rows, heads, tokens per row, head dim
                             (a multiple of 8, 8 <= D <= 256)               */
    int64_t sb, st, sh;   /* element strides of batch, token, head           */
    float   scale;        /* softmax scale; usually 1/sqrt(D)                */
    int64_t Hkv;          /* key/value heads (H % Hkv == 0); 0: Hkv = H     */
    int64_t sb_kv, st_kv, sh_kv;   /* strides of k, v, dk, dv when Hkv > 0  */
} attn_shape;

/* ---- planning (host only, integer-exact; never touches the GPU) -------- */

/* Chunk boundaries of one causal sequence of L tokens in N chunks.
 * UNIFORM: b_k = 128*floor(k*L/(128*N)). FLOPS: b_k = the multiple of 128
 * nearest to L*sqrt(k/N) (ties up), which equalises the quadratic attention
 * cost of InfiniPipe Eq. (1) (SPPO §3.2 FLOPs-based partition: long chunks
 * first, short later). b_0 = 0, b_N = L. RESPLIT_EDGES also sets kv_split of
 * the first and last chunk to q_begin + 128*floor((q_end-q_begin)/256 + 1/2)
 * when that falls strictly inside the chunk (SPPO §4).
 * out: host array of cap entries; *n_out = N on success.
 * Errors: ATTN_E_INVAL (L <= 0, N <= 0, unknown mode, boundaries not strictly
 * increasing), ATTN_E_CAPACITY (cap < N). */
int attn_plan(int64_t L, int32_t N, int32_t mode,
              attn_chunk* out, int32_t cap, int32_t* n_out);

/* FLOPS chunks of one sequence (as attn_plan) with the edge chunks re-split
 * as in SPPO's multiplexed sequence partition (§4, Table 3) for PP pipeline
 * stages: the SP range of an edge subsequence shrinks by one device per
 * subsequence away from each pipeline end, so chunk i and chunk N-1-i get
 * kv_split = -P with P the largest count from 2 up to PP - i that the chunk
 * can hold (none when PP - i < 2). Errors as attn_plan (PP <= 0 is
 * ATTN_E_INVAL). */
int attn_plan_multiplex(int64_t L, int32_t N, int32_t PP,
                        attn_chunk* out, int32_t cap, int32_t* n_out);

/* Chunks of a packed batch (InfiniPipe §II-B, §III-A1). cu_seqlens: host
 * array of ndocs+1 non-decreasing offsets, cu_seqlens[0] = 0. A document of
 * L_d tokens becomes ceil(L_d / max_chunk_tokens) chunks by the mode's rule
 * measured from the document start, all with ctx_begin = document start;
 * empty documents give no chunk. RESPLIT_EDGES re-splits the first and last
 * chunk of the whole plan. Errors as attn_plan. */
int attn_plan_varlen(const int64_t* cu_seqlens, int32_t ndocs, int32_t max_chunk_tokens,
                     int32_t mode, attn_chunk* out, int32_t cap, int32_t* n_out);

/* InfiniPipe's workload-balanced sequence chunking (Algorithm 1, §III-B),
 * on one GPU. Inputs: nseq sequence lengths (packed back to back in this
 * order, so sequence i starts at seq_lens[0] + ... + seq_lens[i-1]); K, the
 * number of slices of the longest sequence; token_cap, the most tokens one
 * chunk may hold (T_m); the cost model of Eq. (1) with N = d_p = 1: a chunk
 * {C, S} costs beta1 + alpha1((C+s0)^2 - C^2) + alpha2 s0 + the sum over its
 * other slices of alpha1 s^2 + alpha2 s.
 * Steps: the longest sequence is cut into K slices of equal cost (the mesh;
 * boundaries at the multiple of 128 nearest to each equal-cost point, ties
 * up); each sequence takes mesh slices in order while it is longer than the
 * next one (split chunks, one call each) and keeps the rest as its tail
 * slice; sequences no longer than the first mesh slice are short. Every tail
 * seeds a bucket (a hybrid chunk); short sequences, most expensive first, go
 * into the first bucket in order of increasing time per token whose time
 * stays within T_t (initially the costliest mesh slice) and whose tokens stay
 * within token_cap; a sequence that even the emptiest bucket cannot hold
 * opens a new bucket (a batched chunk); when no bucket fits, T_t is raised to
 * the least time among buckets with token room plus the sequence's time.
 * Output: the chunks of every call (chunk {C, S}), call after call, in out
 * (ctx_begin = the sequence start, kv_split = 0, sorted by q_begin within a
 * call); call c holds out[call_off[c] .. call_off[c+1]); *n_out chunks and
 * *n_calls calls. The order can be run one call at a time: forward with
 * attn_fwd in call order, backward with attn_bwd_chunk in reverse order.
 * Errors: ATTN_E_INVAL (no sequence, a negative length, more than INT32_MAX
 * tokens, K <= 0, costs negative or not finite or alpha1 = alpha2 = 0, a
 * mesh whose boundaries are not strictly increasing, token_cap below the
 * first mesh slice), ATTN_E_CAPACITY (cap < *n_out or call_cap < *n_calls + 1;
 * both counts are then set to what is needed). Host only. */
int attn_plan_infinipipe(const int64_t* seq_lens, int32_t nseq, int32_t K, int64_t token_cap,
                         double alpha1, double alpha2, double beta1,
                         attn_chunk* out, int32_t cap, int32_t* n_out,
                         int32_t* call_off, int32_t call_cap, int32_t* n_calls);

/* Workspace bytes for pass 0 (forward: attn_fwd and its stages), pass 1
 * (backward: attn_bwd and its stages), pass 2 (attn_bwd_chunk on exactly
 * these chunks) or pass 3 (attn_key_mass) of this shape and chunk table.
 * Validates like the compute calls. */
int attn_workspace_size(const attn_shape* shape, const attn_chunk* chunks, int32_t n,
                        int32_t pass, size_t* bytes);

/* ---- forward ----------------------------------------------------------- */

/* Forward of every chunk: o (bf16) and lse (fp32) for all rows of the
 * chunks. Chunks must be sorted by q_begin with disjoint query ranges and
 * 0 <= ctx_begin <= q_begin < q_end <= T. Rows outside every chunk are not
 * written. Equivalent to attn_fwd_tiles followed by attn_fwd_merge. */
int attn_fwd(const void* q, const void* k, const void* v,
             const attn_chunk* chunks, int32_t n, const attn_shape* shape,
             void* o, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Stage 1 of the forward: the tile kernel. Rows of unsplit chunks (and rows
 * of split chunks whose tile lies wholly before the first split point) get
 * their final o and lse; the key-range partials of the remaining rows (two
 * for a split at one point, P for kv_split = -P) go to the workspace as
 * fp32. */
int attn_fwd_tiles(const void* q, const void* k, const void* v,
                   const attn_chunk* chunks, int32_t n, const attn_shape* shape,
                   void* o, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Stage 2 of the forward: log-sum-exp merge of the partials of re-split
 * chunks (RSA accumulation over key/value blocks, made exact with LSE):
 * LSE = ln sum_p e^{LSE_p}; O = sum_p e^{LSE_p-LSE} O_p over the parts whose
 * key range starts at or before the row; a partial with LSE = -inf has
 * weight 0. A no-op when no chunk is split. */
int attn_fwd_merge(const attn_chunk* chunks, int32_t n, const attn_shape* shape,
                   void* o, float* lse, void* ws, size_t ws_bytes, void* stream);

/* ---- backward ---------------------------------------------------------- */

/* Gradients of the forward for upstream dout, given the forward's o and lse.
 * The chunk table must partition [0, T) (sorted, contiguous) with every
 * chunk of one document sharing ctx_begin = the document start; the result
 * depends on the documents only, not on where chunks are cut (InfiniPipe
 * §II-A: dK/dV of a token gather contributions of all later tokens).
 * dq, dk, dv are bf16 with the shared strides. Equivalent to
 * attn_bwd_prep, attn_bwd_tiles, attn_bwd_dq in that order. */
int attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
             const void* dout, const attn_chunk* chunks, int32_t n, const attn_shape* shape,
             void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, void* stream);

/* Stage 1: D_t = sum_d dO_td * O_td (fp32) into the workspace, and zero the
 * fp32 dQ accumulator. */
int attn_bwd_prep(const void* o, const void* dout, const attn_chunk* chunks, int32_t n,
                  const attn_shape* shape, void* ws, size_t ws_bytes, void* stream);

/* Stage 2: one key tile per work item: recompute P = exp(S - LSE), then
 * dV += P^T dO, dS = P o (dO V^T - D), dK += scale dS^T Q (owned, written as
 * bf16) and dQ += scale dS K (fp32 reduction into the workspace). */
int attn_bwd_tiles(const void* q, const void* k, const void* v, const float* lse,
                   const void* dout, const attn_chunk* chunks, int32_t n,
                   const attn_shape* shape, void* dk, void* dv,
                   void* ws, size_t ws_bytes, void* stream);

/* Stage 3: dq = bf16(fp32 dQ accumulator). */
int attn_bwd_dq(const attn_chunk* chunks, int32_t n, const attn_shape* shape,
                void* dq, void* ws, size_t ws_bytes, void* stream);

/* ---- chunk-streamed backward ------------------------------------------- */

/* Backward of the query rows of a set of chunks against their resident
 * contexts, for a caller that runs chunks one call at a time: the forward in
 * chunk order (attn_fwd on the same chunks: their rows attend to the keys
 * [ctx_begin, q_end) already in k, v; SPPO §5.1, the K/V of earlier
 * subsequences stay resident), the backward in reverse order (InfiniPipe
 * §II-A: the K/V gradients of a token gather contributions from every later
 * token, so a chunk's keys are complete once the chunks after it and the
 * chunk itself have run). One call may hold the slices of several documents,
 * such as an InfiniPipe batched or hybrid chunk {C, S} (§III-A1).
 * For each chunk, with query rows t in [q_begin, q_end) (kv_split ignored):
 *   dq rows [q_begin, q_end)                 = their gradient (bf16; complete:
 *                                              every key they see is in the
 *                                              context);
 *   dk_acc, dv_acc rows [ctx_begin, q_end)  += the rows' contributions (fp32,
 *                                              dK including the scale);
 *   dk, dv rows [q_begin, q_end)             = bf16 of the updated accumulators.
 * Other rows of dq, dk, dv, dk_acc, dv_acc are not touched. Chunks: sorted by
 * q_begin, 0 <= ctx_begin <= q_begin < q_end <= T, and key ranges disjoint
 * (each ctx_begin >= the previous chunk's q_end), so that no accumulator row
 * is updated twice by one call. Zero dk_acc and dv_acc over a document before
 * the call holding its last chunk; after the calls holding all of its chunks,
 * in reverse chunk order, dq, dk, dv equal attn_bwd's result for the document.
 * o, lse are the forward's; o and dout are read for the chunks' rows.
 * dk_acc, dv_acc: fp32 device arrays indexed like the bf16 tensors, element
 * (b, t, h, d) at b*sb + t*st + h*sh + d, 16-byte aligned. The workspace comes
 * from attn_workspace_size(pass 2) for the same chunks; calls that share
 * dk_acc/dv_acc rows must run one after another (one stream).
 * Errors: ATTN_E_INVAL (bad shape or chunks, overlapping key ranges, a NULL
 * pointer), ATTN_E_ALIGN, ATTN_E_UNSUPPORTED, ATTN_E_WORKSPACE, ATTN_E_CUDA;
 * device errors through attn_status(ws). */
int attn_bwd_chunk(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dout, const attn_chunk* chunks, int32_t n, const attn_shape* shape,
                   void* dq, void* dk, void* dv, float* dk_acc, float* dv_acc,
                   void* ws, size_t ws_bytes, void* stream);

/* ---- attention weight of each key --------------------------------------- */

/* The attention weight that each key received, summed over the query rows of
 * the chunks and over the query heads of its key/value head:
 *   mass_out[b][hk][j] = mass_in[b][hk][j]
 *       + sum_{h of hk} sum_{t in chunks, ctx_begin <= j <= t} exp(scale * q_t . k_j - LSE_t)
 * from the forward's q, k and lse (no V, no O). Chunks as attn_fwd (kv_split is
 * validated and ignored): all of a prompt's chunks give the weights of the whole
 * prompt, one chunk holding the last rows the weights as those rows see them, and
 * a caller that runs chunk by chunk accumulates with mass_in = mass_out. Rows
 * outside every chunk contribute nothing; every entry j in [0, T) of mass_out is
 * written. A row whose lse is -inf contributes nothing. Sums are fp32 in a fixed
 * order: the result does not change from run to run.
 * mass_in, mass_out: fp32 [B][Hkv][T] contiguous, 16-byte aligned; mass_in may be
 * NULL (zeros) or equal mass_out, and must not overlap it otherwise. Workspace:
 * attn_workspace_size(pass 3) for the same chunks. Errors as attn_fwd. */
int attn_key_mass(const void* q, const void* k, const float* lse, const attn_chunk* chunks, int32_t n,
                  const attn_shape* shape, const float* mass_in, float* mass_out,
                  void* ws, size_t ws_bytes, void* stream);

/* ---- key/value cache held in 4 bits -------------------------------------- */

/* A cache of cap slots for each of B sequences and Hkv key/value heads. The row
 * of slot t of head h of sequence b is row r = b*sb + h*sh + t of four arrays in
 * device memory:
 *   k_codes, v_codes    r * D/2 bytes on: D codes e2m1 (sign, two exponent bits,
 *                       one fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two a
 *                       byte, the even dim in the low four bits
 *   k_scales, v_scales  r * ceil(D/16) bytes on: one e4m3 scale for each 16
 *                       consecutive dims (the last block may have 8)
 * A value is code * block scale * k_scale (or v_scale). k_scale and v_scale are
 * powers of two in [2^-64, 2^64], so every value has at most six significant bits
 * and is exact in bf16. A block that held a NaN or an infinity has scale NaN.
 * D: a multiple of 8 from 8 to 256. cap, sb and sh: multiples of 16; sb and sh
 * (in slots) allow a view of some sequences, heads or slots of a larger cache, no
 * two of whose rows are the same (ATTN_E_INVAL: the heads of a sequence lie between
 * two sequences, or the other way round).
 * The arrays are 16-byte aligned. */
typedef struct {
    int64_t B, Hkv, cap, D;
    int64_t sb, sh;
    void *k_codes, *k_scales, *v_codes, *v_scales;
    float k_scale, v_scale;
} attn_kv4_cache;

/* Conventions of the attn_kv4_* calls
 *   - pos, lens and cu_seqlens are device arrays of int32, read when the call
 *     runs: a captured graph replays with whatever they hold then.
 *   - ws: at least attn_kv4_workspace_size() bytes, 256-byte aligned. Its first
 *     256 bytes are zeroed by the caller once, before its first use. The calls
 *     only ever set the status word there and attn_status() reads and clears it
 *     (ATTN_E_BOUNDS: a slot, length or offset outside the cache), so that a
 *     decode loop needs one look at the end. Calls that may overlap on the GPU
 *     take different workspaces.
 *   - Every call may be captured into a graph, and allocates nothing. */

/* Workspace bytes of one attn_kv4_* call: op ATTN_KV4_ROWS (attn_kv4_store,
 * attn_kv4_load, attn_kv4_evict; shape may be NULL), ATTN_KV4_ATTEND
 * (attn_kv4_attend without mass_out; shape is the queries') or
 * ATTN_KV4_ATTEND_MASS (with). A workspace that is large enough for one may
 * serve the others. With mass_out it holds fp32 scores: 4 B Hkv cap bytes for each
 * of the H / Hkv * T rows of a key/value head (their number rounded up to 2, 4 or
 * groups of 8, 16 or 32), at most 1 GiB, or one group's where that is more; calls of
 * more rows take them in several passes. */
#define ATTN_KV4_ROWS         0
#define ATTN_KV4_ATTEND       1
#define ATTN_KV4_ATTEND_MASS  2
int attn_kv4_workspace_size(const attn_kv4_cache* cache, const attn_shape* shape, int32_t op, size_t* bytes);

/* Store rows of K and V. Dense (cu_seqlens NULL): shape B = cache B, H = cache
 * Hkv, T rows each; row t of sequence b goes to slot pos[b] + t. Packed
 * (cu_seqlens: B + 1 offsets): shape B = 1, T tokens in all, and token
 * cu_seqlens[b] + t goes to slot pos[b] + t of sequence b. k and v are bf16 with
 * the shape's (query) strides. For each block of 16 dims, with ts the tensor scale:
 *   s = e4m3(max|x| / (6 ts)),  code = e2m1(x / (s ts))
 * both to nearest even, saturating at 448 and 6; s = 0 gives code 0 (with the
 * sign of x). A row whose slot is outside [0, cap), and a token of no sequence,
 * is skipped (ATTN_E_BOUNDS). Errors: ATTN_E_INVAL (NULL pointers, sizes that
 * do not fit each other, 2^31 rows or more, a tensor scale that is not a power
 * of two in range, D of cache and shape differ), ATTN_E_ALIGN, ATTN_E_UNSUPPORTED,
 * ATTN_E_WORKSPACE, ATTN_E_CUDA. */
int attn_kv4_store(const void* k, const void* v, const attn_shape* shape, const attn_kv4_cache* cache,
                   const int32_t* pos, const int32_t* cu_seqlens, void* ws, size_t ws_bytes, void* stream);

/* The reverse of attn_kv4_store: the rows' values in bf16 (exact unless a value
 * leaves bf16's range). Rows that attn_kv4_store would skip are left as they were
 * (ATTN_E_BOUNDS). Rows of k and v that share memory (strides under which they
 * overlap) are ATTN_E_INVAL. Errors as attn_kv4_store. */
int attn_kv4_load(const attn_kv4_cache* cache, const int32_t* pos, const int32_t* cu_seqlens,
                  const attn_shape* shape, void* k, void* v, void* ws, size_t ws_bytes, void* stream);

/* Attention of the newest T tokens of each sequence over its cache (their own
 * rows stored before the call). q, o: bf16 with the shape's (query) strides,
 * shape B = cache B, H a multiple of cache Hkv (query head h reads key/value head
 * h / (H / Hkv); the shape's own Hkv fields are ignored), T = 1 for single-token
 * decoding, D = cache D, no two rows in the same memory (o has the same strides). With n = lens[b] slots in use, query i sees
 * the slots j <= n - T + i:
 *   LSE_i = ln sum_j exp(scale * q_i . k_j),  O_i = sum_j exp(scale * q_i . k_j - LSE_i) v_j
 * A query that sees no slot (n - T + i < 0; n = 0) has O = 0 and LSE = -inf.
 * lse: fp32 [B][H][T] contiguous. mass_out (or NULL): the weight of each slot over
 * the call's queries and the heads of its key/value head is added,
 *   mass_out[b][hk][j] = mass_in[b][hk][j] + sum exp(scale * q_i . k_j - LSE_i)  for j < n,
 * with rows of mass_ld fp32 (mass_in NULL: zeros; it may equal mass_out and must
 * not overlap it otherwise); entries j >= n are left as they were. A slot that was
 * appended since the last call counts too: its entry of mass_in has to be 0 before
 * the first call that sees it, also where the buffer held another cache's weights.
 * A length outside
 * [0, cap] (with mass_out: or above mass_ld) is reported (ATTN_E_BOUNDS) and taken
 * as the nearest in range. The products are made in fp16 with fp32 sums: cache
 * values and queries (scaled by a power of two) are exact there, softmax weights
 * are rounded to 11 bits. Errors as attn_kv4_store. */
int attn_kv4_attend(const void* q, const attn_shape* shape, const attn_kv4_cache* cache, const int32_t* lens,
                    void* o, float* lse, const float* mass_in, float* mass_out, int64_t mass_ld,
                    void* ws, size_t ws_bytes, void* stream);

/* Cut every sequence to at most `keep` slots: of the n = lens[b] slots in use, the
 * last min(recent, keep) and those of the others with the highest mass (ties: the
 * lowest slot; NaN counts as the highest), m = min(n, keep) in all, move to slots
 * 0..m-1 of dst in their order, chosen for each key/value head on its own.
 *   lens_out[b] = m;  slots[b][h][i] = the source slot of row i, -1 for m <= i < keep
 *   mass_out[b][h][i] = mass[b][h][slots[b][h][i]]   (mass_out may be NULL)
 * Rows m and on of dst and mass_out are left as they were: clear mass_out before the
 * call if slots appended later are to be weighed in it. mass: rows of mass_ld
 * fp32; mass_out: rows of mass_out_ld >= keep; slots: int32 [B][Hkv][keep]
 * contiguous (fewer than 2^31). src and dst have the same B, Hkv, D and tensor scales, dst.cap >= keep >= 1,
 * 0 <= recent; src and dst, and mass and mass_out, must not overlap (but may be slots
 * of one allocation that lie between one another), and lens_out may equal lens. Lengths out of range as in attn_kv4_attend. Errors as
 * attn_kv4_store. */
int attn_kv4_evict(const attn_kv4_cache* src, const int32_t* lens, const float* mass, int64_t mass_ld,
                   int32_t keep, int32_t recent, const attn_kv4_cache* dst, int32_t* lens_out,
                   float* mass_out, int64_t mass_out_ld, int32_t* slots,
                   void* ws, size_t ws_bytes, void* stream);

/* ---- key/value cache in pages --------------------------------------------- */

/* A pool of pages of `page` slots each (a power of two from 16 to 1024), bf16, shared
 * by all sequences: slot i of page p of key/value head h is the row of D elements at
 *   p*sp + h*sh + i*st
 * of k and of v (element strides, multiples of 8; no two rows share memory; base
 * pointers 16-byte aligned). Slot j of sequence b is slot j % page of the page
 * table[b*table_ld + j / page], and a slot's number in the pool is its page's number
 * times `page` plus its place in the page; pages * page is below 2^31. */
typedef struct {
    int64_t pages, Hkv, page, D;
    int64_t sp, sh, st;
    void *k, *v;
} attn_paged_cache;

/* Conventions of the attn_paged_* calls
 *   - Tokens are packed, [T, heads, D] (shape B = 1): sequence b's new tokens are those
 *     from cu_seqlens[b] up to cu_seqlens[b + 1]; tokens behind the last sequence's are
 *     padding, so that a captured graph serves batches of different sizes.
 *   - add, lens, table, cu_seqlens, slots and n_free are device arrays of int32, read
 *     when the call runs. Whatever they hold, nothing outside the given arrays is read
 *     or written.
 *   - ws: at least attn_paged_workspace_size() bytes, 256-byte aligned, its first 256
 *     bytes zeroed by the caller once, before its first use. attn_status() reads and
 *     clears the status word there, which the calls only set: ATTN_E_BOUNDS (a length,
 *     offset, page or slot out of range), ATTN_E_CAPACITY (attn_paged_reserve: a
 *     sequence was refused), ATTN_E_TIMEOUT. Calls that may overlap on the GPU take
 *     different workspaces.
 *   - B is at most 2^20, a sequence has fewer than 2^31 - 2^12 slots.
 *   - Every call may be captured into a graph, and allocates nothing. */

/* Workspace bytes of one attn_paged_* call: op ATTN_PAGED_STORE (shape may be NULL),
 * ATTN_PAGED_RESERVE (cache and shape may be NULL) or ATTN_PAGED_ATTEND (shape is the
 * queries') for B sequences. A workspace that is large enough for one may serve the
 * others. Attention keeps at most 17 partials of 128 rows for each SM (171 MB at 128
 * dims; fewer rows where T tokens of H / Hkv heads are fewer). */
#define ATTN_PAGED_STORE    0
#define ATTN_PAGED_RESERVE  1
#define ATTN_PAGED_ATTEND   2
int attn_paged_workspace_size(const attn_paged_cache* cache, const attn_shape* shape, int64_t B, int32_t op,
                              size_t* bytes);

/* Reserve slots for the next tokens of B sequences. With add[b] >= 0, sequence b gets
 * add[b] slots behind the lens[b] that it uses; with add[b] < 0 it ends, its pages go
 * back and lens_out[b] = 0 (its row of the table stays as it was). Free pages are a
 * stack: free_pages[0 .. n_free - 1], of `pages` entries. In this order:
 *   pages of ended sequences are put on the stack, sequence by sequence, page by page;
 *   with held = ceil(lens / page) and need = ceil((lens + add) / page) - held, the
 *   sequences are served in their order: page held + j of sequence b is the
 *   (needs of the sequences before + j)-th from the top of the stack;
 *   one whose need the rest of the stack does not cover is refused, and so are those
 *   after it, but for the ones that need no page. One that would outgrow its table's
 *   max_pages entries is refused on its own, and takes nothing (ATTN_E_CAPACITY).
 *   lens_out[b] = lens[b] + add[b], or lens[b] if refused;
 *   n_free_out = what is left on the stack;
 *   cu_seqlens[b] = sum of max(add, 0) before b, for B + 1 entries, refused or not;
 *   slots[t] = the slot's number in the pool, for token t of [0, T); -1 for the tokens
 *   of refused sequences and those behind the last.
 * Sequences whose tokens pass T are refused too and cu_seqlens ends at T; lengths
 * outside [0, max_pages * page] are taken as the nearest; pages put back beyond the
 * stack's end are dropped; a token whose page is outside the pool gets slot -1 (all
 * ATTN_E_BOUNDS).
 * Every page has to be in one place, in use in one row of the table or on the stack: it
 * keeps no count of a page's owners. A page in use in two rows goes onto the stack with
 * each of them, after which two sequences get it and write over each other's rows; that
 * is not found out. A caller whose sequences share pages ends them without this call:
 * it sets their lengths to 0 and puts a page on the stack when its last owner ends, and
 * gives a sequence that goes on in a shared page a copy of it first (attn_paged_store).
 * lens_out may equal lens, and n_free_out n_free; otherwise no array that is written
 * may overlap another, the gaps between the table's rows included (ATTN_E_INVAL). T is
 * below 2^30. Errors: ATTN_E_INVAL (NULL pointers, sizes), ATTN_E_ALIGN,
 * ATTN_E_WORKSPACE, ATTN_E_CUDA. */
int attn_paged_reserve(const int32_t* add, const int32_t* lens, int64_t B, int64_t page, int64_t pages,
                       const int32_t* n_free, int32_t* free_pages, int32_t* table, int64_t table_ld,
                       int64_t max_pages, int32_t* lens_out, int32_t* n_free_out, int32_t* cu_seqlens,
                       int32_t* slots, int64_t T, void* ws, size_t ws_bytes, void* stream);

/* Store row t of k and v, bf16 [T, Hkv, D] with the shape's (query) strides, in slot
 * slots[t]; a row with slot -1 is skipped, as is one with any other slot outside the
 * pool (ATTN_E_BOUNDS). A slot that two rows name holds pieces of either. Rows may be
 * slots of the pool itself, a page that is copied, say; what the call reads from a slot
 * that it also writes are pieces of the old row or of the new one. Errors:
 * ATTN_E_INVAL (NULL pointers, sizes that do not fit each other, T * Hkv * D of 2^34
 * or more), ATTN_E_ALIGN, ATTN_E_UNSUPPORTED, ATTN_E_WORKSPACE, ATTN_E_CUDA. */
int attn_paged_store(const void* k, const void* v, const attn_shape* shape, const attn_paged_cache* cache,
                     const int32_t* slots, void* ws, size_t ws_bytes, void* stream);

/* Attention of the newest tokens of B sequences, one or a chunk of many each, over
 * their pages (the tokens' own rows stored before the call; sequences may have pages in
 * common). q, o: bf16 [T, H, D] with
 * the shape's (query) strides, H a multiple of the cache's Hkv (query head h reads
 * key/value head h / (H / Hkv)), o apart from q. cu_seqlens as above, or NULL: T / B
 * tokens each. With n = lens[b] slots in use and n_q tokens, query i sees the slots
 * j <= n - n_q + i:
 *   LSE_i = ln sum_j exp(scale * q_i . k_j),  O_i = sum_j exp(scale * q_i . k_j - LSE_i) v_j
 * A query that sees no slot has O = 0 and LSE = -inf. lse: fp32 [H][T] contiguous.
 * Rows of padding are left as they were. Slots that a query does not see do not reach
 * its output, whatever they hold. A length outside [0, max_pages * page] is taken as
 * the nearest in range, an offset outside [the one before it, T] (the first: [0, T])
 * likewise, and a page outside the pool reads as zeros (all ATTN_E_BOUNDS). Softmax weights are rounded to bf16 for
 * the product with V; sums are fp32, in an order that the lengths alone decide: the
 * result does not change from run to run. Errors as attn_paged_store. */
int attn_paged_attend(const void* q, const attn_shape* shape, const attn_paged_cache* cache, const int32_t* table,
                      int64_t table_ld, int64_t max_pages, const int32_t* lens, const int32_t* cu_seqlens, int64_t B,
                      void* o, float* lse, void* ws, size_t ws_bytes, void* stream);

/* ---- forward without a caller-provided workspace ----------------------- */

/* Bytes of the scratch area inside the library used by attn_fwd_noalloc. */
#define ATTN_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* The forward (as attn_fwd) for callers that cannot allocate device memory,
 * e.g. code hosted by a runtime that owns all device memory and offers no
 * allocator, or code that must not allocate once it is running. The pages
 * have no counterpart: this is a convenience of this library.
 * Instead of a workspace argument it uses a scratch area of
 * ATTN_NOALLOC_SCRATCH_BYTES that lives in the library and that every GPU
 * which loads the library holds until the process exits. The caller still
 * passes q, k, v, o and lse; arguments, layouts and errors are as attn_fwd.
 * Returns ATTN_E_WORKSPACE when this shape and chunk table need more forward
 * workspace than ATTN_NOALLOC_SCRATCH_BYTES (attn_workspace_size, pass 0);
 * re-split chunks need fp32 partials, so they reach the limit first.
 * Every call looks up the scratch address in the context current on the
 * calling thread (nothing is cached, so a device reset or another context on
 * the device gets its own address); the first call in a context loads the
 * library's kernels there, so make it before any stream capture. It
 * allocates nothing. All calls share the one scratch area and it keeps the
 * last call's contents (every call rewrites what it reads): calls that
 * overlap on the GPU race with each other, so issue them on one stream, or
 * otherwise one after the other. Device-side errors of this path are read
 * with attn_noalloc_status(). */
int attn_fwd_noalloc(const void* q, const void* k, const void* v,
                     const attn_chunk* chunks, int32_t n, const attn_shape* shape,
                     void* o, float* lse, void* stream);

/* Device error word of attn_fwd_noalloc (its status header lives in the
 * library's scratch area): synchronises `stream`, then reads and clears it,
 * like attn_status() does for a caller workspace. Returns ATTN_OK,
 * ATTN_E_TIMEOUT or ATTN_E_BOUNDS (ATTN_E_CUDA if the read fails). The word
 * is cleared by every attn_fwd_noalloc call when it starts, and is shared by
 * all of them, like the rest of the scratch area. No counterpart on the
 * pages. */
int attn_noalloc_status(void* stream);

/* ---- status ------------------------------------------------------------ */

/* Synchronises `stream`, then reads and clears the device error word in the
 * workspace header: ATTN_OK, ATTN_E_TIMEOUT, ATTN_E_BOUNDS or, after
 * attn_paged_reserve, ATTN_E_CAPACITY (or ATTN_E_CUDA if the read itself fails). The word lives in the first 256 bytes of the
 * workspace; attn_fwd / attn_fwd_tiles / attn_bwd / attn_bwd_prep / attn_bwd_chunk clear it
 * when they start, and a workspace no such call has used must be zeroed by
 * the caller before its status is read. */
int attn_status(void* ws, void* stream);

/* Static English text for a status code. */
const char* attn_strerror(int status);

/* Library version string, e.g. "libattn 0.1 sm_103a". */
const char* attn_version(void);

/* Number of kernels this library has enqueued, on any stream and device,
 * since it was loaded (a relaxed atomic counter; thread-safe). A compute
 * call enqueues its tile kernels plus one small copy kernel per 31 KB of
 * work list it writes into the workspace. No counterpart on the pages. */
uint64_t attn_kernel_launches(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H_ */
