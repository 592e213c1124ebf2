/*
 * usp.h — C ABI of the GB300 Ulysses sequence-parallel attention hot path.
 *
 * The library emulates P sequence-parallel ranks inside one GPU's memory.  The
 * calls follow the attention wrapper of huggingface/accelerate PR #4209
 * ("Add an FSDP2-native Ulysses sequence parallelism backend"):
 *
 *   1. usp_relayout_fwd   q, k, v: "gather sequence, scatter heads"
 *                         (_gather_seq_scatter_heads, the all-to-all comment)
 *   2. usp_cu_seqlens_from_position_ids
 *                         document boundaries rebuilt from the *gathered*
 *                         position_ids, never the collator's per-shard
 *                         cu_seq_lens_q/k (the stale-kwargs comment: 41.8% of
 *                         logits mismatched with the per-shard ones)
 *   3. usp_attn_fwd       varlen causal GQA attention over the gathered
 *                         sequence, optional sliding window, one sink logit per
 *                         head sliced to the rank's heads (the gpt-oss finding)
 *   4. usp_relayout_bwd   the output: "gather heads, scatter sequence"
 *                         (_gather_heads_scatter_seq)
 *   backward: usp_relayout_fwd(dO), usp_attn_bwd, usp_relayout_bwd(dQ, dK, dV):
 *   the exchanges swap scatter and gather (same comment).
 *
 * Conventions shared by every call
 *   - Every pointer is a DEVICE pointer owned by the caller.  The library never
 *     allocates or frees device memory; scratch space is passed in as a
 *     workspace whose size a *_workspace_bytes query returns.
 *   - Every call only enqueues work on `stream` and returns without
 *     synchronising.  Results are valid once the stream reaches that point.
 *   - The return value reports host-side argument checks and launch errors.
 *     Data errors found on the device (stale or malformed cu_seqlens, negative
 *     position ids) are written to *dev_status (device int32, may be NULL)
 *     as a usp_status code; a call never clears *dev_status, so zero it
 *     before the first call and read it after synchronising.
 *   - Pointers passed to the relayout and attention calls must be 16-byte
 *     aligned (USP_ERR_ALIGNMENT otherwise).
 *   - Layout names:  seq-layout  [P][B][S/P][H][D]  rank r holds positions
 *                                 [r*S/P, (r+1)*S/P) of every row, all heads;
 *                    head-layout [P][B][S][H/P][D]  rank r holds every position,
 *                                 heads [r*H/P, (r+1)*H/P).
 *     Sequence chunks are contiguous in rank order, heads go to ranks in
 *     contiguous blocks, so rank r's query heads r*hq..r*hq+hq-1 read its own
 *     key/value heads under GQA.
 *   - The library is thread-safe per stream and keeps no state beyond a
 *     per-device cache of the SM count.
 */
#ifndef USP_H_
#define USP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t / CUstream; NULL is the legacy default stream. */
typedef struct CUstream_st* usp_stream_t;

typedef enum {
  USP_OK = 0,
  USP_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, bad flag */
  USP_ERR_INDIVISIBLE = 2,   /* P does not divide S, Hq or Hkv, or Hkv does not divide Hq
                                (accelerate PR #4209: "sp_size not dividing the heads" is refused) */
  USP_ERR_UNSUPPORTED = 3,   /* head dim, element size or size outside what the kernels take */
  USP_ERR_ALIGNMENT = 4,     /* pointer or contiguous run not a multiple of 16 bytes */
  USP_ERR_BAD_SEQLENS = 5,   /* device: cu_seqlens[0] != 0, not increasing, or cu_seqlens[n] != B*S
                                (e.g. a shard's stale per-shard boundaries) */
  USP_ERR_BAD_POSITIONS = 6, /* device: a negative position id */
  USP_ERR_TIMEOUT = 7,       /* device: a bounded wait inside a kernel gave up */
  USP_ERR_CUDA = 8,          /* a CUDA runtime/driver call or launch failed */
  USP_ERR_WORKSPACE = 9,     /* workspace pointer null/misaligned or smaller than required */
  USP_ERR_BAD_MODS = 10,     /* device: a bucket id outside [0, n_buckets), a negative prefix length, or
                                fewer prefix lengths than documents */
  USP_ERR_BAD_ROPE = 11,     /* device: an axis outside [0, n_axes), or a frequency that is not finite or above 1024 */
  USP_ERR_BAD_PAGES = 12     /* device: a page outside the pool, a length outside the block table, or boundaries of
                                appended tokens that do not fit their number or their sequences' lengths */
} usp_status;

/* Static, human-readable name of a status code.  Never NULL. */
const char* usp_status_string(int status);

/* Library version as major*10000 + minor*100 + patch. */
int usp_version(void);

/* ------------------------------------------------------------------------
 * Relayout (the all-to-all of each rank, emulated as one permutation of the
 * P ranks' buffers).  accelerate PR #4209, the comment on the four
 * _SeqAllToAll.apply call sites: queries/keys/values go from the local
 * sequence chunk with all heads to the whole sequence with H/P heads, and the
 * output comes back per rank as its sequence chunk with the heads of every rank.
 *
 *   usp_relayout_fwd:  x_head[r][b][r'*S/P + s'][j][d] = x_seq[r'][b][s'][r*H/P + j][d]
 *   usp_relayout_bwd:  x_seq[r'][b][s'][r*H/P + j][d]  = x_head[r][b][r'*S/P + s'][j][d]
 *
 * x_seq:  [P][B][S/P][H][D] elements of elem_bytes bytes (input of fwd, output of bwd)
 * x_head: [P][B][S][H/P][D]                          (output of fwd, input of bwd)
 *
 * Fewer heads than ranks (H < P, P a multiple of H; kv-head replication, a
 * follow-up listed in PR #4209): every head is replicated on P/H ranks, rank r
 * holding head r / (P/H), so x_head is [P][B][S][1][D] and
 *   usp_relayout_fwd:  x_head[r][b][r'*S/P + s'][0][d] = x_seq[r'][b][s'][r / (P/H)][d]
 *   usp_relayout_bwd:  x_seq[r'][b][s'][h][d] = sum over the P/H ranks r with r / (P/H) == h of
 *                      x_head[r][b][r'*S/P + s'][0][d]
 * (the exchange back of a gradient is the adjoint of the copy: the replicas'
 * gradients add up).  The sum is taken in fp32 in rank order and rounded once;
 * it is defined for bf16 only (elem_bytes 2, else USP_ERR_UNSUPPORTED).
 *
 * The two buffers must not overlap.  Each contiguous run, (H/P)*D*elem_bytes
 * bytes (D*elem_bytes when replicated), must be a multiple of 16
 * (USP_ERR_ALIGNMENT otherwise).
 * Errors: USP_ERR_INVALID_ARG (null pointer, size <= 0, elem_bytes not 1/2/4/8),
 *         USP_ERR_INDIVISIBLE (S % P, or H % P when H >= P, or P % H when H < P),
 *         USP_ERR_ALIGNMENT, USP_ERR_UNSUPPORTED, USP_ERR_CUDA.
 * Apart from the replica sum the result is a bit-exact copy of every element.
 * ---------------------------------------------------------------------- */
int usp_relayout_fwd(const void* x_seq, void* x_head, int B, int S, int H, int D, int P,
                     int elem_bytes, usp_stream_t stream);
int usp_relayout_bwd(const void* x_head, void* x_seq, int B, int S, int H, int D, int P,
                     int elem_bytes, usp_stream_t stream);

/* Same permutation for three tensors in one launch: q (Hq heads) and k, v
 * (Hkv heads, replicated when Hkv < P), all with head dim D.  Equivalent to
 * three usp_relayout_fwd calls; meant for the q/k/v exchange of one attention
 * layer.  Hq % P != 0 is USP_ERR_INDIVISIBLE (query heads are never replicated). */
int usp_relayout_fwd_qkv(const void* q_seq, const void* k_seq, const void* v_seq,
                         void* q_head, void* k_head, void* v_head,
                         int B, int S, int Hq, int Hkv, int D, int P, int elem_bytes,
                         usp_stream_t stream);

/* ------------------------------------------------------------------------
 * One real rank's side of the exchanges, for P processes (one per GPU) that
 * run the all-to-all themselves (NCCL all_to_all_single, or any transport
 * that sends chunk p of a buffer to rank p and lays the received chunks out
 * in source-rank order).  accelerate PR #4209, the comment on the four
 * _SeqAllToAll.apply call sites: each rank sends every other rank that rank's
 * heads of its own sequence chunk and receives its own heads of every chunk;
 * the way back swaps scatter and gather.
 *
 * Shapes (Sl = S/P positions per rank, hpr = H/P heads per rank, or 1 with
 * H < P where each head is replicated on P/H ranks, rank p holding head
 * p / (P/H)):
 *   x_local [B][Sl][H][D]     the rank's sequence chunk, all heads
 *   x_head  [B][P*Sl][hpr][D] the whole sequence, the rank's heads (what
 *                             usp_attn_fwd/_bwd take with P = 1 and Hq/Hkv set
 *                             to the rank's head counts)
 *   send, recv [P][B][Sl][hpr][D]  chunk p goes to / came from rank p
 *
 *   usp_a2a_pack_seq_to_head:   send[p][b][s][j][d] = x_local[b][s][p*hpr + j][d]
 *                               (H < P: x_local[b][s][p / (P/H)][d])
 *   usp_a2a_unpack_seq_to_head: x_head[b][p*Sl + s][j][d] = recv[p][b][s][j][d]
 *   usp_a2a_pack_head_to_seq:   send[p][b][s][j][d] = x_head[b][p*Sl + s][j][d]
 *   usp_a2a_unpack_head_to_seq: x_local[b][s][p*hpr + j][d] = recv[p][b][s][j][d]
 *                               (H < P: x_local[b][s][h][d] = sum over the P/H ranks p
 *                               with p / (P/H) == h of recv[p][b][s][0][d], in fp32 in
 *                               rank order, rounded once; bf16 only)
 * With B == 1 the unpack after the seq->head exchange and the pack before the
 * head->seq exchange are plain copies (recv already is x_head, x_head already
 * is send), and a caller may skip them.  H is always the global head count.
 * Apart from the replica sum every result is a bit-exact copy.  Buffers must
 * not overlap; pointers and each contiguous run of hpr*D*elem_bytes bytes must
 * be 16-byte aligned.
 * Errors: USP_ERR_INVALID_ARG, USP_ERR_INDIVISIBLE (H and P), USP_ERR_ALIGNMENT,
 * USP_ERR_UNSUPPORTED, USP_ERR_CUDA.
 * ---------------------------------------------------------------------- */
int usp_a2a_pack_seq_to_head(const void* x_local, void* send, int B, int S_local, int H, int D, int P,
                             int elem_bytes, usp_stream_t stream);
int usp_a2a_unpack_seq_to_head(const void* recv, void* x_head, int B, int S_local, int H, int D, int P,
                               int elem_bytes, usp_stream_t stream);
int usp_a2a_pack_head_to_seq(const void* x_head, void* send, int B, int S_local, int H, int D, int P,
                             int elem_bytes, usp_stream_t stream);
int usp_a2a_unpack_head_to_seq(const void* recv, void* x_local, int B, int S_local, int H, int D, int P,
                               int elem_bytes, usp_stream_t stream);

/* ------------------------------------------------------------------------
 * Document boundaries from the gathered position_ids.  accelerate PR #4209:
 * position_ids are all-gathered once per forward in the model's pre-hook and
 * every layer reads them; the per-shard cu_seq_lens_q/k and max_length_q/k a
 * padding-free collator computed are dropped and rebuilt from the gathered
 * positions.
 *
 * pos:         int32 [P][B][S/P], each rank's shard.  The gathered sequence is
 *              gathered[b][r*S/P + s'] = pos[r][b][s'] (for B == 1 the buffer
 *              already *is* the gathered [S], byte for byte).
 * cu_seqlens:  int32, capacity B*S + 1 (output).  A document starts at every
 *              row start b*S and wherever the gathered position is 0.
 *              cu_seqlens[0] = 0, cu_seqlens[n_docs] = B*S, strictly increasing.
 * n_docs:      int32 device scalar (output): number of documents.
 * max_len:     int32 device scalar (output): longest document.
 * ws:          device workspace of at least usp_cu_seqlens_workspace_bytes(B, S)
 *              bytes, 16-byte aligned; its contents on entry do not matter.
 * dev_status:  device int32 (nullable): USP_ERR_BAD_POSITIONS if any position is
 *              negative (the outputs are then unspecified).
 * Output is bit-exact (integers).  Errors: USP_ERR_INVALID_ARG, USP_ERR_INDIVISIBLE
 * (S % P), USP_ERR_UNSUPPORTED (B*S >= 2^31 - 1), USP_ERR_WORKSPACE, USP_ERR_CUDA.
 * ---------------------------------------------------------------------- */
size_t usp_cu_seqlens_workspace_bytes(int B, int S);
int usp_cu_seqlens_from_position_ids(const int32_t* pos, int B, int S, int P,
                                     int32_t* cu_seqlens, int32_t* n_docs, int32_t* max_len,
                                     void* ws, size_t ws_bytes, int32_t* dev_status,
                                     usp_stream_t stream);

/* Same result as usp_cu_seqlens_from_position_ids, for callers that cannot
 * allocate device memory or hand over a workspace (for example code whose
 * device memory is entirely reserved by another allocator, or a plugin
 * interface that passes only input and output pointers).  It allocates
 * nothing: the scan's scratch lives in a fixed 64 KiB device array inside the
 * library, which every GPU that loads the library holds until the process
 * exits.  The pages have no counterpart of this call.
 *   - B*S may be at most 2^24 tokens; larger sizes return USP_ERR_UNSUPPORTED.
 *   - Every call looks up the array's device address on the current device
 *     (the first lookup on a device may load the library's device code
 *     there); make the first call on a device before any stream capture.
 *   - Every call shares the one array: calls whose kernels may overlap on the
 *     GPU (other streams, other host threads) race and must be ordered by the
 *     caller.  Leftover contents from an earlier call never matter.
 * Other arguments, outputs and errors are those of
 * usp_cu_seqlens_from_position_ids. */
int usp_cu_seqlens_from_position_ids_noalloc(const int32_t* pos, int B, int S, int P, int32_t* cu_seqlens,
                                             int32_t* n_docs, int32_t* max_len, int32_t* dev_status,
                                             usp_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention over the gathered sequence, all P emulated ranks in one launch.
 *
 * For rank r, local query head j (global head r*hq + j, hq = Hq/P), its key/
 * value head j / (Hq/Hkv), token t of document [a, b): visible keys u are
 * a <= u <= t (causal; without causal a <= u < b) and t - u <= window_left
 * when window_left >= 0.  With s = softmax_scale * q_t . k_u and the sink
 * logit z = sinks[r*hq + j] (not scaled; absent when sinks == NULL):
 *     LSE_t = ln( sum_u exp(s_tu) + exp(z) )
 *     O_t   = sum_u exp(s_tu - LSE_t) v_u
 * (softmax over the keys plus one value-less sink logit; accelerate PR #4209,
 * the gpt-oss finding: each head has a single sink logit, so after the exchange
 * a rank uses the slice of the sinks for the heads it holds).
 * ---------------------------------------------------------------------- */
typedef struct {
  int B, S, Hq, Hkv, D, P;   /* global sizes; D must be 64 or 128 */
  int causal;                /* 1: causal mask inside each document; 0: full document */
  int window_left;           /* -1: none; else t - u <= window_left ("window 128" = 127) */
  float softmax_scale;       /* 0: 1/sqrt(D) */
  const int32_t* cu_seqlens; /* device int32 [n_docs+1], from usp_cu_seqlens_from_position_ids */
  const int32_t* n_docs;     /* device int32 scalar */
  const float* sinks;        /* device fp32 [Hq] (global heads), or NULL */
  int io_layout;             /* USP_IO_HEAD (0): q, k, v, dO, o, dq, dk, dv in head-layout;
                                USP_IO_SEQ (1): the same tensors in seq-layout — the exchanges
                                are fused into the kernels' loads and stores; needs (S/P) % 128 == 0;
                                USP_IO_SEQ_KV_HEAD (2, usp_attn_fwd only): q and o in seq-layout,
                                k and v in head-layout (the forward re-reads every k/v tile many
                                times, which runs faster from head-layout rows than from rows
                                strided over all key/value heads; the backward entry points
                                return USP_ERR_UNSUPPORTED for it) */
  int ring;                  /* ring x Ulysses hybrid: ring degree R (0 or 1: no ring).  With R > 1,
                                P is the Ulysses degree and a call computes one ring step: rows of
                                super-chunk a (S/R positions each) see only the keys of super-chunk
                                (a - ring_step) mod R.  The tensors are the hybrid head-layout of
                                usp_hybrid_relayout_fwd (USP_IO_HEAD) or the P*R sequence shards
                                [P*R][B][S/(P*R)][H][D] (USP_IO_SEQ, needs (S/(P*R)) % 128 == 0).
                                Needs (S/R) % 256 == 0. */
  int ring_step;             /* 0 <= ring_step < R */
  int head_first, head_count; /* usp_attn_bwd_dkdv / usp_attn_bwd_dq with USP_IO_SEQ only: process the
                                key/value heads [head_first, head_first + head_count) and their query
                                heads (0, 0: all), so that the stored dS of a long sequence can be
                                produced and consumed a group of heads at a time; every other entry
                                point needs 0, 0 */
} usp_attn_params;

enum { USP_IO_HEAD = 0, USP_IO_SEQ = 1, USP_IO_SEQ_KV_HEAD = 2 };

/* q:   bf16 head-layout [P][B][S][Hq/P][D];  k, v: bf16 [P][B][S][Hkv/P][D]
 *      (with io_layout = USP_IO_SEQ: seq-layout [P][B][S/P][Hq][D] and [P][B][S/P][Hkv][D],
 *      i.e. the shards each rank holds before the exchange; o then comes back in
 *      seq-layout too, exactly what usp_relayout_bwd of the head-layout o gives)
 * o:   bf16 head-layout like q (output)
 * lse: fp32 [P][B][Hq/P][S] natural-log LSE (output; includes the sink)
 * dev_status: nullable device int32; USP_ERR_BAD_SEQLENS when cu_seqlens does
 *   not start at 0, is not strictly increasing, or does not end at B*S (the
 *   outputs are then left unwritten).
 * Errors: USP_ERR_INVALID_ARG (also an unknown io_layout), USP_ERR_INDIVISIBLE,
 * USP_ERR_UNSUPPORTED (D not 64/128, window_left < -1, B*S >= 2^30 or
 * B*S*Hq >= 2^31, Hq > 1024, USP_IO_SEQ with (S/P) % 128 != 0), USP_ERR_ALIGNMENT,
 * USP_ERR_CUDA. */
int usp_attn_fwd(const usp_attn_params* params, const void* q, const void* k, const void* v,
                 void* o, float* lse, int32_t* dev_status, usp_stream_t stream);

/* ------------------------------------------------------------------------
 * Ring x Ulysses hybrid (USP; feifeibear/long-context-attention issue #135,
 * the device-mesh script: ranks form a (ring, ulysses) mesh with the Ulysses
 * dimension innermost and contiguous ("basic") sequence chunks).
 *
 * P = ring * ulysses ranks; rank p = rho*ulysses + u holds positions
 * [p*S/P, (p+1)*S/P).  The Ulysses exchange runs inside each ring group
 * rho, after which rank (rho, w) holds super-chunk rho (positions
 * [rho*C, (rho+1)*C), C = S/ring) for heads [w*H/U, (w+1)*H/U), U = ulysses.
 * The hybrid head-layout [U][B][S][H/U][D] lays the ring ranks' super-chunks
 * end to end for each w:
 *   x_head[w][b][rho*C + u*S/P + s'][j][d] = x_seq[rho*U + u][b][s'][w*H/U + j][d]
 * (H < U: replicated heads as in usp_relayout_fwd; the bwd exchange sums them).
 * ring = 1 is usp_relayout_fwd/bwd with P = ulysses.  Errors as usp_relayout_fwd,
 * with S % (ring*ulysses) for USP_ERR_INDIVISIBLE.
 * ---------------------------------------------------------------------- */
int usp_hybrid_relayout_fwd(const void* x_seq, void* x_head, int B, int S, int H, int D, int ring, int ulysses,
                            int elem_bytes, usp_stream_t stream);
int usp_hybrid_relayout_bwd(const void* x_head, void* x_seq, int B, int S, int H, int D, int ring, int ulysses,
                            int elem_bytes, usp_stream_t stream);
int usp_hybrid_relayout_fwd_qkv(const void* q_seq, const void* k_seq, const void* v_seq,
                                void* q_head, void* k_head, void* v_head,
                                int B, int S, int Hq, int Hkv, int D, int ring, int ulysses, int elem_bytes,
                                usp_stream_t stream);

enum { USP_RING_FIRST = 1, USP_RING_LAST = 2 };

/* Forward of one ring step's result into the running output: with the step's
 * o_step (bf16, head layout like o) and lse_step (fp32 [P][B][hq][S], -inf for
 * rows that saw no key) from usp_attn_fwd with params->ring_step = s:
 *   L = ln(e^L_acc + e^L_step),  O = e^(L_acc - L) O_acc + e^(L_step - L) O_step
 * o_step, o_acc and o share the layout params->io_layout names (the hybrid
 * head layout, or the sequence shards with USP_IO_SEQ); lse_* are always
 * [P][B][hq][S].
 * flags USP_RING_FIRST: the running values start as the step's (o_acc/lse_acc
 * are not read).  USP_RING_LAST: the sink logit z = sinks[r*hq + j] (if
 * params->sinks) joins once, L' = ln(e^L + e^z), O' = e^(L - L') O, and the
 * result goes to o (bf16) and lse (fp32), o_acc/lse_acc are not written;
 * otherwise it goes to o_acc (fp32, shaped like o) and lse_acc.  params is the
 * step call's (ring and ring_step are not read; sinks are, at the last step).
 * Pointers 16-byte aligned.  Errors: as usp_attn_fwd. */
int usp_ring_fwd_merge(const usp_attn_params* params, const void* o_step, const float* lse_step,
                       float* o_acc, float* lse_acc, void* o, float* lse, int flags, usp_stream_t stream);

/* Backward of the ring: g_acc (fp32) += g_step (bf16), n elements (a multiple
 * of 8).  USP_RING_FIRST: g_acc starts at zero (not read).  USP_RING_LAST: the
 * sum is rounded once to bf16 into g_out and g_acc is not written.  Every
 * step's dQ (kept by its rank) and dK/dV (carried with their super-chunk) is
 * summed at the element's own address.  Pointers 16-byte aligned.
 * Errors: USP_ERR_INVALID_ARG, USP_ERR_ALIGNMENT, USP_ERR_UNSUPPORTED (n/8 >= 2^32), USP_ERR_CUDA. */
int usp_ring_grad_accumulate(const void* g_step, float* g_acc, void* g_out, size_t n, int flags,
                             usp_stream_t stream);

/* Workspace that enables the faster backward: the dK/dV pass also stores dS
 * (bf16 blocks of [128 keys][64 queries] for every (query head, row, key tile,
 * query slice) pair a causal mask can reach) and the dQ pass computes
 * dQ = scale * dS K from them instead of recomputing S and dP.  Returns the
 * whole workspace size (the statistics of usp_attn_bwd_workspace_bytes plus
 * the blocks), or 0 when the shape has no such path (causal == 0, or S not a
 * multiple of 128).  The blocks' count depends only on the shape (the longest
 * possible document), so it is known without reading cu_seqlens.  Any
 * backward call given ws_bytes >= this size takes the stored-dS path; the
 * dK/dV and dQ calls of one backward must get the same ws and ws_bytes, with
 * the dK/dV call first. */
size_t usp_attn_bwd_fast_workspace_bytes(const usp_attn_params* params);
/* (With params->head_count > 0 the blocks are those of that head group, and
 * the dK/dV and dQ calls of the group use that workspace; the statistics
 * part still covers every head, as the preprocess writes it for all.) */

/* Bytes of workspace usp_attn_bwd needs: the fp32 row statistic
 * D_t = sum_d dO_td O_td for every query row and head, 256-byte aligned. */
size_t usp_attn_bwd_workspace_bytes(const usp_attn_params* params);

/* Gradients of usp_attn_fwd for the loss sum(O * dO):
 *   P_tu = exp(s_tu - LSE_t), dS_tu = P_tu (dO_t . v_u - D_t)
 *   dQ_t = scale sum_u dS_tu k_u,   dK_u = scale sum_t dS_tu q_t,
 *   dV_u = sum_t P_tu dO_t,         dsink = -sum_t exp(z - LSE_t) D_t
 * (key/value gradients sum over the query heads of their GQA group).
 * q, k, v, o, lse: the forward's inputs and outputs; dO: bf16 like o.
 * dq, dk, dv: bf16 outputs shaped like q, k, v.  dsinks: fp32 [Hq] output or
 * NULL (ignored when params->sinks is NULL).  ws: at least
 * usp_attn_bwd_workspace_bytes(params) bytes, 256-byte aligned.
 * The result is deterministic: no floating-point atomics.
 * Errors: as usp_attn_fwd, plus USP_ERR_WORKSPACE. */
int usp_attn_bwd(const usp_attn_params* params, const void* q, const void* k, const void* v,
                 const void* o, const float* lse, const void* dO,
                 void* dq, void* dk, void* dv, float* dsinks,
                 void* ws, size_t ws_bytes, int32_t* dev_status, usp_stream_t stream);

/* The three phases usp_attn_bwd runs, in order, each one kernel launch (the
 * preprocess adds one small reduction when sinks are given).  They are exposed
 * so that a caller can time them or place the two gradient passes, which only
 * read what the preprocess wrote, on different streams.  `ws` is
 * usp_attn_bwd's workspace: the preprocess writes D_t there, the gradient
 * passes read it.  Arguments and errors are as in usp_attn_bwd.
 *   usp_attn_bwd_preprocess: D_t = sum_d dO_td O_td; dsinks (nullable).
 *   usp_attn_bwd_dkdv:       dK, dV (every query head of each GQA group).
 *   usp_attn_bwd_dq:         dQ. */
int usp_attn_bwd_preprocess(const usp_attn_params* params, const void* o, const float* lse, const void* dO,
                            float* dsinks, void* ws, size_t ws_bytes, int32_t* dev_status, usp_stream_t stream);
int usp_attn_bwd_dkdv(const usp_attn_params* params, const void* q, const void* k, const void* v,
                      const float* lse, const void* dO, void* dk, void* dv, const void* ws, size_t ws_bytes,
                      int32_t* dev_status, usp_stream_t stream);
int usp_attn_bwd_dq(const usp_attn_params* params, const void* q, const void* k, const void* v,
                    const float* lse, const void* dO, void* dq, const void* ws, size_t ws_bytes,
                    int32_t* dev_status, usp_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention with modified scores: usp_attn_fwd / usp_attn_bwd with a tanh cap,
 * a bias by distance and a prefix mask.  For global query head h, token t, key
 * u of t's document [a, b):
 *     x = softmax_scale q_t.k_u - slopes[h] |t - u|
 *         + rel_bias[h][buckets[clamp(t - u, -R, R) + R]]          R = max_distance
 *     z = softcap tanh(x / softcap)   (z = x without a cap: the cap bounds the biased score)
 * and the softmax runs over z and the head's sink logit (which is not capped).
 * Visible keys: those of usp_attn_fwd, and with prefix_lens also every key u of
 * the first prefix_lens[d] tokens of t's document d, whatever its order
 * (t - u <= window_left still holds with a window).
 * ---------------------------------------------------------------------- */
typedef struct {
  float softcap;               /* 0: none; else 2^-10 .. 2^10.  The absolute error of z is under
                                  2.5e-7 softcap and that of x. */
  const float* slopes;         /* device fp32 [Hq] (global heads), or NULL: no linear bias.  |slope| <= 2^10.
                                  The score of a key at distance d has fp32's error at the size of |slope| (d + 128):
                                  up to 5 2^-24 |slope| (d + 128) in an exponent.  Where slopes are >= 0 (and no
                                  table hides the near keys) a far key has no weight and only 128 slopes count;
                                  slopes below 0 put the weights on the farthest keys (-0.5 over 32768 tokens: up
                                  to 5e-3 of a weight) */
  const float* rel_bias;       /* device fp32 [Hq][n_buckets], or NULL: no learned bias.  At most 2^20; an entry
                                  below -2^20 (-inf, the lowest fp32 value) hides its keys (only without a cap):
                                  a row that then sees nothing has O = 0, LSE = -inf */
  const int32_t* buckets;      /* device int32 [2*max_distance + 1]: the bucket of distance t - u at index
                                  t - u + max_distance; farther distances take the ends' buckets */
  int n_buckets;               /* 1 .. 4097 */
  int max_distance;            /* 1 .. 2048 */
  int rel_bias_grad;           /* 1: the backward collects the gradient of rel_bias (a larger workspace) */
  const int32_t* prefix_lens;  /* device int32 [n_prefix], one per document in cu_seqlens order, or NULL; more
                                  than the document's length means all of it.  Needs causal = 1. */
  int n_prefix;                /* at least the number of documents */
} usp_score_mods;

/* Host helper: a bucket map for usp_score_mods.buckets, into HOST memory
 * int32 [2*max_distance + 1].  With n = |t - u| and K = n_buckets (half of them
 * when bidirectional): distances n < K/2 have a bucket each, farther ones
 *     K/2 + floor( (K - K/2) ln(n / (K/2)) / ln(max_distance / (K/2)) ),
 * at most K - 1.  bidirectional: keys after the query (t - u < 0) take the upper
 * half of the buckets; otherwise they take bucket 0 (they are masked in a causal
 * model; with a prefix use a bidirectional map).
 * Errors: USP_ERR_INVALID_ARG (null, K < 2, odd n_buckets when bidirectional,
 * max_distance <= K/2), USP_ERR_UNSUPPORTED (max_distance > 2048, n_buckets > 4097). */
int usp_rel_buckets_log(int n_buckets, int max_distance, int bidirectional, int32_t* buckets);

/* Forward.  q, k, v, o, lse, dev_status and params as usp_attn_fwd (every
 * io_layout; ring <= 1).
 * dev_status may also get USP_ERR_BAD_MODS: a bucket id outside the table, a bias or
 * a slope above its limit or NaN, a negative or missing prefix length (the outputs are
 * then unspecified).
 * Every element of q, k and v must be finite, hidden keys' too: a tile's products
 * take all its keys, hidden ones with weight 0.
 * Errors: as usp_attn_fwd, and USP_ERR_INVALID_ARG (mods NULL, a softcap that is
 * negative, infinite or NaN, fields of an absent rel_bias or prefix_lens that are
 * not zero, a prefix without causal order), USP_ERR_UNSUPPORTED (softcap,
 * max_distance or n_buckets outside their ranges, ring > 1). */
int usp_attn_mod_fwd(const usp_attn_params* params, const usp_score_mods* mods, const void* q, const void* k,
                     const void* v, void* o, float* lse, int32_t* dev_status, usp_stream_t stream);

/* Workspace of the backward: the statistics of usp_attn_bwd, with rel_bias the
 * bias rows by distance, and with rel_bias_grad partial sums of the scores'
 * gradient by distance (16 (2R + 1) bytes per head and 32 tokens).  The fast form
 * adds the stored dS blocks, as usp_attn_bwd_fast_workspace_bytes does; with a
 * prefix or without causal order they cover every pair of a key tile and a query
 * slice of a row.  0: invalid arguments, or (fast) S not a multiple of 128. */
size_t usp_attn_mod_bwd_workspace_bytes(const usp_attn_params* params, const usp_score_mods* mods);
size_t usp_attn_mod_bwd_fast_workspace_bytes(const usp_attn_params* params, const usp_score_mods* mods);

/* Gradients of usp_attn_mod_fwd for the loss sum(O * dO): with P_tu = exp(z_tu - LSE_t)
 *     dX_tu = P_tu (dO_t . v_u - D_t) (1 - tanh^2(x_tu / softcap))
 *     dQ_t = scale sum_u dX_tu k_u,  dK_u = scale sum_t dX_tu q_t,  dV_u = sum_t P_tu dO_t
 *     drel_bias[h][b] = sum of dX_tu over the pairs whose distance has bucket b
 * and dsinks as in usp_attn_bwd.  slopes get no gradient.  D_t = dO_t . O_t is
 * taken from the bf16 o, or, where a gradient in fp32 would show its rounding
 * (rel_bias_grad, or dsinks with sinks), as sum_u P_tu (dO_t . v_u) in fp32 by a
 * pass of its own over the scores.  drel_bias: fp32 [Hq][n_buckets], given exactly when mods->rel_bias_grad.
 * Every element of q, k, v and dO must be finite (see the forward).
 * Deterministic.  A workspace belongs to one call at a time: backward calls that
 * may overlap (other streams, graphs launched at once) need one each.
 * Errors: as usp_attn_mod_fwd and usp_attn_bwd. */
int usp_attn_mod_bwd(const usp_attn_params* params, const usp_score_mods* mods, const void* q, const void* k,
                     const void* v, const void* o, const float* lse, const void* dO, void* dq, void* dk, void* dv,
                     float* dsinks, float* drel_bias, void* ws, size_t ws_bytes, int32_t* dev_status,
                     usp_stream_t stream);

/* Its phases, as those of usp_attn_bwd: the preprocess first (statistics, bias
 * rows), then dK/dV, then dQ; head groups for the dK/dV
 * and dQ passes with USP_IO_SEQ as there.  usp_attn_mod_bwd_rel_bias reduces the partial
 * sums once the dK/dV passes of all heads are done. */
int usp_attn_mod_bwd_preprocess(const usp_attn_params* params, const usp_score_mods* mods, const void* q,
                                const void* k, const void* v, const void* o, const float* lse, const void* dO,
                                float* dsinks, void* ws, size_t ws_bytes, int32_t* dev_status, usp_stream_t stream);
int usp_attn_mod_bwd_dkdv(const usp_attn_params* params, const usp_score_mods* mods, const void* q, const void* k,
                          const void* v, const void* dO, void* dk, void* dv, const void* ws, size_t ws_bytes,
                          int32_t* dev_status, usp_stream_t stream);
int usp_attn_mod_bwd_dq(const usp_attn_params* params, const usp_score_mods* mods, const void* q, const void* k,
                        const void* v, const void* dO, void* dq, const void* ws, size_t ws_bytes, int32_t* dev_status,
                        usp_stream_t stream);
int usp_attn_mod_bwd_rel_bias(const usp_attn_params* params, const usp_score_mods* mods, float* drel_bias, void* ws,
                              size_t ws_bytes, usp_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions of one or several axes (a text's position; height and width;
 * time, height and width), for q and k in one launch.  Pair i of a head turns by
 * the angle w = positions[axes[i]][t] * freqs[i]:
 *     y1 = x1 cos w - x2 sin w,  y2 = x1 sin w + x2 cos w
 * with (x1, x2) = elements (i, i + n_pairs), or (2i, 2i + 1) when interleaved; the
 * elements behind the 2 n_pairs turned ones pass through.  The layer applies it
 * to the sequence shards before the exchange, a decoding step to the new tokens.
 * ---------------------------------------------------------------------- */
typedef struct {
  int tokens;               /* tokens of q and k, in any order: q is [tokens][Hq][D] */
  int Hq, Hkv, D;           /* D 64 or 128; Hkv 0: no k */
  int n_axes;               /* 1 .. 8 */
  int n_pos;                /* divides tokens: token t has the position t mod n_pos (the ranks of a head layout
                               hold the same tokens) */
  int n_pairs;              /* a multiple of 8, 8 .. D/2 */
  int interleaved;
  const int32_t* positions; /* device int32 [n_axes][n_pos]; negative ones turn backwards */
  const float* freqs;       /* device fp32 [n_pairs], radians per position, |f| <= 1024 */
  const int32_t* axes;      /* device int32 [n_pairs], or NULL: axis 0 */
} usp_rope_params;

/* q, q_out: bf16 [tokens][Hq][D]; k, k_out: bf16 [tokens][Hkv][D] (NULL with Hkv 0).  An output may be its input
 * (in place), else buffers must not overlap.  usp_rope_bwd takes the gradients of q_out and k_out to those of q
 * and k: it turns back by the same angles.  The angle is taken modulo a turn in 64-bit fixed point: it is within
 * 2e-7 (5e-7 for |f| > 1) at any int32 position.  The turned values are rounded once.
 * dev_status: USP_ERR_BAD_ROPE (such pairs turn by 0).
 * Errors: USP_ERR_INVALID_ARG, USP_ERR_INDIVISIBLE (tokens % n_pos), USP_ERR_UNSUPPORTED (D, n_pairs, n_axes > 8,
 * Hq + Hkv > 4096, tokens >= 2^30, tokens (Hq + Hkv) >= 2^34), USP_ERR_ALIGNMENT, USP_ERR_CUDA. */
int usp_rope_fwd(const usp_rope_params* params, const void* q, const void* k, void* q_out, void* k_out,
                 int32_t* dev_status, usp_stream_t stream);
int usp_rope_bwd(const usp_rope_params* params, const void* dq_out, const void* dk_out, void* dq, void* dk,
                 int32_t* dev_status, usp_stream_t stream);

/* ------------------------------------------------------------------------
 * A key/value cache in pages, per rank the heads that the rank holds.  Position t
 * of sequence s is token t % page_size of page block_table[s][t / page_size].  The
 * heads of a rank are those of the head layout: Hkv/P of them, or with Hkv < P the
 * one head r / (P/Hkv) on rank r.
 * With dtype USP_CACHE_E4M3 a token's head has a power of two 2^e, the smallest
 * with e >= -126 for which every |x| <= 448 2^e (an infinity counts as the largest
 * finite bf16), stored as the byte e + 127 (1 to 247), and its elements are x / 2^e rounded to
 * the nearest e4m3 value (ties to even; an infinity is held as 448 2^120).  NaN stays NaN.
 * ---------------------------------------------------------------------- */
typedef struct {
  int P, Hkv, D;              /* global key/value heads; D 64 or 128 */
  int n_pages, page_size;     /* page_size a multiple of 16 */
  int n_seqs, max_pages;      /* the block table's sides */
  int dtype;                  /* USP_CACHE_BF16 or USP_CACHE_E4M3 */
  void* k_pages;              /* [P][n_pages][hk][page_size][D], bf16 or e4m3 */
  void* v_pages;
  uint8_t* k_scales;          /* [P][n_pages][hk][page_size], e4m3 only (else NULL) */
  uint8_t* v_scales;
  const int32_t* block_table; /* device int32 [n_seqs][max_pages]; entries behind a sequence's last page are not read */
  const int32_t* lens;        /* device int32 [n_seqs]: tokens of each sequence, appended ones included */
} usp_paged_cache;

enum { USP_CACHE_BF16 = 0, USP_CACHE_E4M3 = 1 };

/* Writes `tokens` new tokens, k and v bf16 [P][tokens][hk][D] (the head layout), as the last ones of their
 * sequences: with cu_seqlens (device int32 [n_seqs+1], e.g. a packed prompt's document boundaries) tokens
 * [cu[s], cu[s+1]) end at position lens[s]; a sequence may have none, and tokens behind cu[n_seqs] are not
 * written.  cu_seqlens NULL: one token each (tokens <= n_seqs: sequence s gets token s; a sequence of length 0,
 * an empty place of a padded batch, is passed over).  Nothing else in the pool changes.  Pages that two
 * sequences share may be read by both but not written in one call.
 * usp_cache_read is the way back: the same tokens out of the cache into k and v, rounded to bf16 (exact for a
 * bf16 cache; e4m3 values times their power of two are rounded only below bf16's normal range, and infinite from
 * 2^128 on, where |x| >= 248 2^120 has gone).  Tokens that are not described
 * (behind cu[n_seqs], or of an empty place) are left as they were.
 * Either of k and v may be NULL, when it is not wanted.  Neither may overlap the cache's arrays, nor, when read, the
 * other or cu_seqlens.
 * dev_status: USP_ERR_BAD_PAGES; tokens without a place in the pool are passed over.
 * Errors: USP_ERR_INVALID_ARG, USP_ERR_INDIVISIBLE, USP_ERR_UNSUPPORTED (D, page_size, dtype; sizes past 2^30
 * tokens or 2^40 elements), USP_ERR_ALIGNMENT, USP_ERR_CUDA. */
int usp_cache_append(const usp_paged_cache* cache, const void* k, const void* v, int tokens,
                     const int32_t* cu_seqlens, int32_t* dev_status, usp_stream_t stream);
int usp_cache_read(const usp_paged_cache* cache, void* k, void* v, int tokens, const int32_t* cu_seqlens,
                   int32_t* dev_status, usp_stream_t stream);

/* Attention of one new token per sequence over the cache (which already holds it: the query is at position
 * lens[s] - 1).  Query head j of a rank reads its key/value head j / (Hq/P / hk):
 *     s_u = softmax_scale q.k_u for u < lens[s], and lens[s] - 1 - u <= window_left with a window
 *     LSE = ln( sum_u exp(s_u) + exp(sink) ),  O = sum_u exp(s_u - LSE) v_u
 * O = 0 where nothing is visible (LSE = -inf, or the sink).
 * q, o: bf16 [P][n_seqs][Hq/P][D]; lse: fp32 [P][n_seqs][Hq/P]; sinks: fp32 [Hq] or NULL.  What is written
 * (o, lse, ws) may overlap nothing else of the call.
 * Products, sums and partial results are fp32.  For the products with the values a weight is rounded to 16 bits over a
 * bf16 cache, to 11 over an e4m3 one (their sum in the LSE is of unrounded weights); over an e4m3 one q is scaled by a
 * power of two into f16, which takes elements below 2^-39 of a head's largest for 0.  A score of -inf has no weight, one
 * of +inf or NaN (also where q and k are so large that fp32 does not hold their product) leaves a head no finite output.
 * A visible value that is not finite leaves its element of O none (over a bf16 cache it may be NaN for an infinity).  Over a
 * bf16 cache values are summed before they are divided: |v| 2^8 lens[s] has to stay below 2^128.
 * The work of all sequences is dealt out evenly in pieces of 16 positions, whatever their lengths, and pieces
 * of one sequence are joined in the order of their positions: the result does not depend on timing (on the other
 * sequences' lengths it does, within its roundings).
 * ws: usp_attn_decode_workspace_bytes bytes, 256-byte aligned, all zero before its first call; a call leaves zero
 * what has to be.  It belongs to one call at a time (calls that may overlap need one each).
 * dev_status: USP_ERR_BAD_PAGES (the sequence's outputs are then unspecified; nothing outside the pool is read);
 * USP_ERR_UNSUPPORTED (2^31 pieces of all sequences, ranks, key/value heads and, of a head's group, 8 or 16 query
 * heads each; or 2^30 positions in one of every 32 sequences: no output is written).
 * Errors: USP_ERR_INVALID_ARG, USP_ERR_INDIVISIBLE, USP_ERR_UNSUPPORTED (as the cache; window_left < -1, Hq > 1024),
 * USP_ERR_ALIGNMENT, USP_ERR_WORKSPACE, USP_ERR_CUDA. */
size_t usp_attn_decode_workspace_bytes(const usp_paged_cache* cache, int Hq);
int usp_attn_decode(const usp_paged_cache* cache, int Hq, int window_left, float softmax_scale, const float* sinks,
                    const void* q, void* o, float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                    usp_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* USP_H_ */
