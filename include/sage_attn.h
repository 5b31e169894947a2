/*
 * sage_attn.h -- C ABI of the GB300 (sm_103a) low-bit attention library:
 * the SageBwd scheme's quantize pass, forward and backward for training.
 *
 * What the calls compute
 * ----------------------
 * "SageBwd: A Trainable Low-bit Attention" (euno.news summary), Methodology 1-2:
 * six of the seven matmuls of an attention block run in low precision -- QK^T and
 * PV in the forward, the S recompute, dV, dQ and dK in the backward -- while the
 * softmax-gradient matmul dP = dO V^T stays in high precision (bf16 here).
 * Methodology 4 and Results: QK-norm (each query and key scaled to unit L2 norm
 * before the dot product) and K-smoothing (read here as subtracting the per-head
 * channel mean of K over tokens, which leaves the softmax unchanged).
 * "Attn-QAT: 4-Bit Attention With Quantization-Aware Training" (gist.science
 * summary), Methodology, principle 1: the backward recomputes P from the saved
 * log-sum-exp in the forward's low precision.  "ThriftAttention" (gist.science
 * summary), Methodology step 2: the FlashAttention-2 online softmax over key tiles.
 *
 * Number formats (the pages give no formulas; these are the plainest reading):
 *   Q: INT8, one fp32 scale max|q'|/127 per 128-token block (all channels);
 *   K: INT8, one fp32 scale max|k''|/127 per 64-token block;
 *   V, dO: FP8 e4m3, one fp32 scale max|x|/448 per (head, channel);
 *   P: FP8 e4m3 with the static scale 1/448 (probabilities relative to the
 *      running row maximum are at most 1);
 *   dS: INT8, one scale max|dS|/127 per (128-query x 64-key) tile.
 * INT8 products accumulate exactly (the codes sit in bf16 containers and every
 * partial sum is an integer below 2^24, exact in the fp32 accumulator).
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Tensors Q, K, V, O, dO, dQ, dK, dV: bf16, contiguous [B, H, N, D] (D fastest),
 *    device memory owned by the caller, 16-byte aligned.  LSE: fp32 [B, H, N],
 *    natural log.  O32 (optional): fp32 [B, H, N, D].
 *  - Supported shapes: B, H >= 1; N >= 1 (any value; tiles are padded internally);
 *    D in {64, 128}; queries and keys share N.  Other shapes: SAGE_ERR_UNSUPPORTED.
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call is
 *    asynchronous on that stream, allocates nothing and never synchronises,
 *    except sage_attn_get_status.
 *  - Argument errors are returned synchronously before anything is launched.
 *  - Workspaces are device memory the caller allocates with at least the size the
 *    *_ws_bytes call reports; their contents are owned by the library between
 *    sage_attn_quantize and the last forward/backward that reads them.
 *  - Every device-side wait is bounded; a wait that runs out records
 *    SAGE_ERR_TIMEOUT in the workspace status word (read with
 *    sage_attn_get_status) and the kernel returns.
 *  - The forward is deterministic.  dQ is accumulated with fp32 additions in L2
 *    (TMA reductions) across key blocks, so its last bits depend on their order.
 */
#ifndef SAGE_ATTN_H
#define SAGE_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SAGE_OK = 0,
  SAGE_ERR_INVALID_ARG = 1, /* null or misaligned pointer, bad size, workspace too small */
  SAGE_ERR_UNSUPPORTED = 2, /* shape outside the supported set */
  SAGE_ERR_CUDA = 3,        /* a CUDA runtime call failed (launch, attribute, tensor map) */
  SAGE_ERR_TIMEOUT = 4,     /* a device-side wait ran out of its time budget */
  SAGE_ERR_NO_PAGES = 5     /* a cache pool has too few free pages (device status) */
} sage_status;

/* Pointers into a quantize workspace (for inspection and parity tests).
 * Np = N rounded up to a multiple of 128; rows past N hold zero codes. */
typedef struct sage_ws_views {
  void *qc;      /* bf16 [B*H, Np, D]: INT8 codes of q' (bf16 containers)           */
  void *kc;      /* bf16 [B*H, Np, D]: INT8 codes of k'' (smoothed, bf16 containers) */
  void *v8t;     /* e4m3 [B*H, D, Np]: FP8 codes of V, channel-major                 */
  float *sq;     /* [B*H, Np/128] Q block scales                                     */
  float *sk;     /* [B*H, Np/64]  K block scales                                     */
  float *sv;     /* [B*H, D]      V channel scales                                   */
  float *kmean;  /* [B*H, D]      channel mean of k' (0 without K-smoothing)         */
  float *qr;     /* [B*H, Np]     1/||q|| per token (1 without QK-norm)              */
  float *kr;     /* [B*H, Np]     1/||k|| per token (1 without QK-norm)              */
  int *status;   /* device status word                                               */
  int n_pad;     /* Np                                                               */
  float *qmean;  /* Q-smoothing: [B*H, Np/128, D] query block means (else NULL)      */
  float *dsb;    /* Q-smoothing: [B*H, Np/128, Np] logit terms (else NULL)           */
  float *vg;     /* NVFP4: [B*H] V's tensor scale max|V| / 2688 (else NULL)          */
  uint8_t *v4;   /* NVFP4: [B*H, D, Np/2] V's e2m1 codes, two per byte, the lower    */
                 /*        token in the low nibble (else NULL)                       */
  uint8_t *v4sf; /* NVFP4: [B*H, Np/64, 512] V's e4m3 block scales; in atom c (tokens */
                 /*        64c ..) byte (d % 32) * 16 + (d / 32) * 4 + 16-token block */
} sage_ws_views;

/* Bytes of the quantize workspace for this shape (0 if unsupported). It holds the
 * codes and scales the forward and backward read, plus the status word. */
size_t sage_attn_ws_bytes(int B, int H, int N, int D);

/* Bytes of the backward scratch for this shape (0 if unsupported): the row terms
 * D_i = rowsum(dO * O) and LSE*log2(e), the FP8 codes of dO, and the fp32 dQ
 * accumulator. */
size_t sage_attn_bwd_ws_bytes(int B, int H, int N, int D);

/*
 * Quantize pass (SageBwd summary, Methodology 1 and 4).
 * Reads Q, K, V; optionally L2-normalises q and k per token (qk_norm != 0);
 * optionally subtracts the per-(b,h) channel mean of k over the N tokens
 * (k_smooth != 0); writes the INT8 codes and scales of q' and k'' and the FP8
 * codes and scales of V into `ws`, and clears the status word.
 * Rounding: every scale and quotient is a correctly rounded fp32 operation;
 * codes round half to even; the norms and means are the fp32 rounding of the
 * exact sums.
 */
int sage_attn_quantize(const void *Q, const void *K, const void *V, int B, int H, int N, int D,
                       int qk_norm, int k_smooth, void *ws, size_t ws_bytes, void *stream);

/*
 * Forward (SageBwd summary, Methodology 1; ThriftAttention summary, Methodology 2).
 * S = (q8 k8^T) * sq * sk * sm_scale computed exactly in integers and scaled in
 * fp32; causal (causal != 0) masks keys j > i; online softmax over 128-key tiles
 * with the running maximum; P = 2^(S*log2e - m) rounded to e4m3 after scaling by
 * 448; O = (P8 V8) * sv / (448 l).  Writes O (bf16), LSE (fp32, natural log) and,
 * if O32 is not NULL, O in fp32 before the bf16 rounding.
 * sm_scale <= 0 selects 1/sqrt(D).  `ws` comes from sage_attn_quantize with the
 * same B, H, N, D.
 */
int sage_attn_fwd(const void *ws, void *O, float *LSE, float *O32, int B, int H, int N, int D,
                  int causal, float sm_scale, void *stream);

/*
 * Backward (SageBwd summary, Methodology 2; Attn-QAT summary, principle 1).
 * D_i = sum_d dO*O; P recomputed from LSE and rounded to e4m3 exactly as in the
 * forward; dP = dO V^T in bf16 with fp32 accumulation (the one unquantized
 * matmul); dS = P (dP - D_i); dV = P8^T dO8 (FP8); dS to INT8 per 128x64 tile;
 * dQ = dS8 k8 and dK = dS8^T q8 (exact integer sums, scaled per tile); then
 * dQ, dK times sm_scale and back through QK-norm when qk_norm != 0.  K-smoothing
 * passes dK through unchanged (the exact dS rows sum to zero).
 * Q, K, V, dO are the same inputs the forward saw; O and LSE the forward's outputs;
 * `ws` the quantize workspace; `bwd_ws` scratch of sage_attn_bwd_ws_bytes.
 * Writes dQ, dK, dV (bf16).
 */
int sage_attn_bwd(const void *Q, const void *K, const void *V, const void *O, const float *LSE,
                  const void *dO, void *dQ, void *dK, void *dV, const void *ws, void *bwd_ws,
                  size_t bwd_ws_bytes, int B, int H, int N, int D, int causal, int qk_norm,
                  int k_smooth, float sm_scale, void *stream);

/*
 * Backward with the high-precision auxiliary output ("Attn-QAT: 4-Bit Attention With
 * Quantization-Aware Training" (gist.science summary), Methodology, principle 2): the same
 * as sage_attn_bwd, except that the row terms D_i = sum_d dO_id O'_id take O' = O32, the
 * forward's fp32 output before its bf16 rounding (the O32 output of sage_attn_fwd), instead
 * of the bf16 O.  O32: fp32 [B, H, N, D], device memory, 16-byte aligned.  The bf16 O is
 * not read.  Errors as for sage_attn_bwd.
 */
int sage_attn_bwd_o32(const void *Q, const void *K, const void *V, const float *O32, const float *LSE,
                      const void *dO, void *dQ, void *dK, void *dV, const void *ws, void *bwd_ws,
                      size_t bwd_ws_bytes, int B, int H, int N, int D, int causal, int qk_norm,
                      int k_smooth, float sm_scale, void *stream);

/*
 * Grouped-query attention: Hkv key/value heads per batch entry, each shared by G = H / Hkv
 * consecutive query heads (query head h reads key/value head h / G; Hkv = 1 is multi-query
 * attention).  The pages leave grouped heads unvalidated ("SageBwd: A Trainable Low-bit
 * Attention" (euno.news summary), Limitations); these calls extend the scheme as follows.
 *  - K, V, dK, dV are bf16 [B, Hkv, N, D]; Q, O, dO, dQ bf16 [B, H, N, D]; LSE [B, H, N].
 *  - Quantize: Q per query head as above; K (smoothing mean, block scales) and V (channel
 *    scales) per key/value head.
 *  - Forward: each query head against its key/value head, exactly as above.
 *  - Backward: dK and dV of a key/value head sum over its G query heads.  The e4m3 channel
 *    scale of dO spans the G query heads' tokens (one scale per key/value head and channel),
 *    so dV stays one FP8 accumulation over all of them.
 * With Hkv = H every call equals its counterpart above.  Hkv must divide H
 * (else SAGE_ERR_UNSUPPORTED).
 */
size_t sage_attn_gqa_ws_bytes(int B, int H, int Hkv, int N, int D);
size_t sage_attn_gqa_bwd_ws_bytes(int B, int H, int Hkv, int N, int D);
int sage_attn_gqa_quantize(const void *Q, const void *K, const void *V, int B, int H, int Hkv, int N, int D,
                           int qk_norm, int k_smooth, void *ws, size_t ws_bytes, void *stream);
int sage_attn_gqa_fwd(const void *ws, void *O, float *LSE, float *O32, int B, int H, int Hkv, int N, int D,
                      int causal, float sm_scale, void *stream);
int sage_attn_gqa_bwd(const void *Q, const void *K, const void *V, const void *O, const float *LSE,
                      const void *dO, void *dQ, void *dK, void *dV, const void *ws, void *bwd_ws,
                      size_t bwd_ws_bytes, int B, int H, int Hkv, int N, int D, int causal, int qk_norm,
                      int k_smooth, float sm_scale, void *stream);
/* Workspace views for the grouped layout: qc, sq, qr hold B*H heads; kc, v8t, sk, sv,
 * kmean, kr hold B*Hkv. */
int sage_attn_gqa_ws_views(void *ws, int B, int H, int Hkv, int N, int D, sage_ws_views *views);

/*
 * Q-smoothing (the optional companion of K-smoothing that "SageBwd: A Trainable Low-bit
 * Attention" (euno.news summary), Methodology 4, names without a formula), with grouped
 * heads as the sage_attn_gqa_* calls (Hkv = H: one key/value head per query head).
 *  - Quantize: each 128-token query block I loses its channel mean before the INT8
 *    quantizer: qmean_I = RN32(sum of the block's q' / its token count) (the fp32 rounding of
 *    the exact mean), qs = RN32(q' - qmean_I), codes and block scale of qs.  The logit terms
 *    dsb[I][j] = qmean_I . k''_j (fp32 products and sums, k'' the smoothed keys of the query
 *    head's key/value head) are stored for every (query block, key).  Workspace:
 *    sage_attn_qs_ws_bytes; it adds 4*B*H*Np/128*(D + Np) bytes to the grouped layout.
 *  - Forward: the logit of query i (block I) and key j is u = RN32(acc * RN32(s_q s_k) +
 *    dsb[I][j]) in natural units; u * RN32(sm_scale log2 e) enters the online softmax.
 *  - Backward (scratch: sage_attn_gqa_bwd_ws_bytes): P is recomputed with the same u, and
 *    dK of each key gets, per (query block, 64-key block) tile, s_dS (sum over the tile's
 *    queries of the dS codes) qmean_I: the mean's share of S = qs k'' + qmean k''.
 * Arguments, layouts, ownership and errors as in the sage_attn_gqa_* calls; a workspace
 * quantized with Q-smoothing is read only by sage_attn_qs_fwd and sage_attn_qs_bwd.
 */
size_t sage_attn_qs_ws_bytes(int B, int H, int Hkv, int N, int D);
int sage_attn_qs_quantize(const void *Q, const void *K, const void *V, int B, int H, int Hkv, int N, int D,
                          int qk_norm, int k_smooth, void *ws, size_t ws_bytes, void *stream);
int sage_attn_qs_fwd(const void *ws, void *O, float *LSE, float *O32, int B, int H, int Hkv, int N, int D,
                     int causal, float sm_scale, void *stream);
int sage_attn_qs_bwd(const void *Q, const void *K, const void *V, const void *O, const float *LSE,
                     const void *dO, void *dQ, void *dK, void *dV, const void *ws, void *bwd_ws,
                     size_t bwd_ws_bytes, int B, int H, int Hkv, int N, int D, int causal, int qk_norm,
                     int k_smooth, float sm_scale, void *stream);
/* Workspace views of the Q-smoothing layout, qmean and dsb included. */
int sage_attn_qs_ws_views(void *ws, int B, int H, int Hkv, int N, int D, sage_ws_views *views);

/*
 * ThriftAttention's selective mixed precision, forward only ("ThriftAttention"
 * (gist.science summary), Methodology steps 1-2 and its implementation paragraph).
 *  - Selection: the importance of the pair (128-query block I, 128-key tile J) is
 *    qbar_I . kbar_J, the dot product of the blocks' channel means over the raw Q and K
 *    (fp64: each mean sums the block's tokens in order and divides by their count; the
 *    dot product adds the channel products in order).  Of the pairs the mask lets through
 *    (causal: J <= I) the n = ceil(budget * pairs - 1e-12) largest are promoted, ties in
 *    index order I * nb + J (nb = Np / 128), per head.
 *  - Promoted pairs run in high precision: S = q16 . k16 (fp16 copies of q' and of the
 *    smoothed keys k'' = RN32(k' - kmean), fp32 accumulation), P16 = fp16(p~), O += P16 v16
 *    (v16 = fp16(V)) in fp32.  The others take the low-bit path of sage_attn_fwd.  A row
 *    runs its low-bit tiles first and its promoted tiles after them, in one online softmax
 *    (shared running maximum and row sum).
 * sage_attn_thrift_ws_bytes: size of the scratch (device memory, caller-owned) that holds
 *   the selection, the fp16 operands and the low-bit pass's hand-over; 0 for an unsupported
 *   shape.
 * sage_attn_thrift_quantize: the quantize pass of sage_attn_quantize into `ws`, then the
 *   selection and the fp16 operands into `tws`; budget in [0, 1].
 * sage_attn_thrift_fwd: the forward on `ws` and `tws` from that call; outputs, sm_scale
 *   and errors as in sage_attn_fwd.
 * sage_attn_thrift_sel: device pointer to the promoted pairs, uint8 [B*H, nb, nb] (1 =
 *   promoted), inside `tws`; NULL for an unsupported shape.
 * Q-smoothing and grouped heads are not combined with this path.
 */
size_t sage_attn_thrift_ws_bytes(int B, int H, int N, int D);
int sage_attn_thrift_quantize(const void *Q, const void *K, const void *V, int B, int H, int N, int D,
                              int qk_norm, int k_smooth, int causal, double budget, void *ws, size_t ws_bytes,
                              void *tws, size_t tws_bytes, void *stream);
int sage_attn_thrift_fwd(const void *ws, const void *tws, void *O, float *LSE, float *O32, int B, int H, int N,
                         int D, int causal, float sm_scale, void *stream);
uint8_t *sage_attn_thrift_sel(void *tws, int B, int H, int N, int D);

/*
 * NVFP4 variant of the forward PV ("Attn-QAT: 4-Bit Attention With Quantization-Aware
 * Training" (gist.science summary), Methodology principle 1 and Implementation: attention
 * trained in FP4 on Blackwell's FP4 path; "ThriftAttention" (gist.science summary),
 * Methodology step 2: the NVFP4 format).  The pages print no recipe; this is NVFP4 for P and
 * V with the rest of the scheme unchanged:
 *  - e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6, signed; nearest, ties to the even code,
 *    saturating), one e4m3 scale per 16 consecutive values along the contracted axis (keys),
 *    one fp32 scale per tensor;
 *  - V, per head: g = RN32(max|V| / 2688); per channel and 16-token block
 *    s = e4m3(RN32(amax / RN32(6 g))), code = e2m1(RN32(v / RN32(s g)));
 *  - P, per row and 16-key block of the online softmax's p~ (relative to the running maximum):
 *    y = RN32(2688 p~), s = e4m3(RN32(max y / 6)), code = e2m1(RN32(y / s)); P^ = code s / 2688;
 *  - O = sum(P^ V^) / l with l the sum of the fp32 p~; QK^T stays INT8.
 * The tensor core multiplies the e2m1 codes and their block scales
 * (tcgen05.mma kind::mxf4nvf4.block_scale); the codes and scales equal the definition above
 * bit for bit.
 * sage_attn_fp4_ws_bytes: workspace size; sage_attn_fp4_quantize: the quantize pass plus V's
 * NVFP4 codes and scales; sage_attn_fp4_fwd: the forward on that workspace (outputs, sm_scale
 * and errors as in sage_attn_fwd); sage_attn_fp4_ws_views: the workspace's pointers, vg, v4
 * and v4sf included.  Plain heads (no grouped heads, no Q-smoothing).
 */
size_t sage_attn_fp4_ws_bytes(int B, int H, int N, int D);
int sage_attn_fp4_quantize(const void *Q, const void *K, const void *V, int B, int H, int N, int D, int qk_norm,
                           int k_smooth, void *ws, size_t ws_bytes, void *stream);
int sage_attn_fp4_fwd(const void *ws, void *O, float *LSE, float *O32, int B, int H, int N, int D, int causal,
                      float sm_scale, void *stream);
int sage_attn_fp4_ws_views(void *ws, int B, int H, int N, int D, sage_ws_views *views);
/* NVFP4 backward (Attn-QAT, principle 1: P recomputed at the forward's precision): P^ in
 * NVFP4 from the saved LSE with the forward's 16-key blocks, used in dS = P^ (dP - D_i) and
 * dV = P^T dO8; the rest as sage_attn_bwd.  dV runs on bf16 tensor cores with the exact
 * values code * s and dO's e4m3 codes (P^'s scales vary along the keys, which dV does not
 * contract).  Scratch: sage_attn_fp4_bwd_ws_bytes (it adds dO's codes as bf16).  `ws` comes
 * from sage_attn_fp4_quantize. */
size_t sage_attn_fp4_bwd_ws_bytes(int B, int H, int N, int D);
int sage_attn_fp4_bwd(const void *Q, const void *K, const void *V, const void *O, const float *LSE, const void *dO,
                      void *dQ, void *dK, void *dV, const void *ws, void *bwd_ws, size_t bwd_ws_bytes, int B, int H,
                      int N, int D, int causal, int qk_norm, int k_smooth, float sm_scale, void *stream);

/*
 * The 8-bit paged key/value cache: what a model trained with the calls above is served from.
 * The training scheme quantizes K to INT8 in 64-token blocks and V to e4m3 ("SageBwd: A Trainable
 * Low-bit Attention" (euno.news summary), Methodology 1); the cache holds K and V in either of the
 * two formats with one fp32 scale per block and head, a block being a page.
 *
 * State, all of it device memory of the caller (one cache per layer):
 *  - k, v: codes [n_pages, Hkv, page, D], one byte each, 16-byte aligned; k_scale, v_scale: fp32
 *    [n_pages, Hkv].  A key is k = code * k_scale.  A page is `page` tokens of every head.
 *  - table: int32 [n_slots, max_pages]; slot s (one sequence) holds lengths[s] tokens (int32) in the
 *    pages table[s][0 .. ceil(lengths[s] / page)), in order.  What a row holds behind them is not
 *    read and may be anything.
 *  - refs: int32 [n_pages], 16-byte aligned: how many slots list the page; 0: the page is free.
 *  - status: one int32, zero at the start: the device status word (sage_attn_get_status(status,
 *    stream)).  SAGE_ERR_NO_PAGES: a slot could not be served; SAGE_ERR_INVALID_ARG: a number on the
 *    device was out of its range (a slot, a length, a page), and what it asked for was left out.  Of
 *    both the word keeps SAGE_ERR_INVALID_ARG.
 *  An empty cache is lengths, refs and status zero.
 * page is 16, 32, 64 or 128; D 64 or 128; n_slots at most 8192; max_pages * page below 2^31.
 *
 * The order of a serving step: sage_attn_kv_extend (room for the new tokens), sage_attn_kv_append
 * (their keys and values), sage_attn_kv_attention (their queries).  All sizes that change from step to
 * step are read on the device, so a captured CUDA graph of the step can be replayed.  Calls that
 * change one cache, or use one workspace, must not overlap on the GPU; attention calls on one cache may.  Host
 * threads may call at the same time.
 */
typedef enum { SAGE_KV_INT8 = 0, SAGE_KV_E4M3 = 1 } sage_kv_kind;

typedef struct sage_kv_cache {
  void *k, *v;              /* [n_pages, Hkv, page, D] codes */
  float *k_scale, *v_scale; /* [n_pages, Hkv] */
  int *table;               /* [n_slots, max_pages] */
  int *lengths;             /* [n_slots] */
  int *refs;                /* [n_pages] */
  int *status;              /* [1] */
  int n_pages, Hkv, page, D, n_slots, max_pages;
  int kind;                 /* sage_kv_kind */
} sage_kv_cache;

/*
 * Quantize new tokens into their pages.  K, V: bf16 [B, Hkv, Nn, D]; batch row b belongs to slot
 * s = slots[b] (slots NULL: s = b); its first n_new[s] tokens become tokens pos[s] .. of the slot
 * (n_new, pos: int32 [n_slots]; what K and V hold behind them is not read).  A slot
 * with n_new[s] <= 0 or pos[s] < 0 (as sage_attn_kv_extend leaves a slot that it refused) is left alone.
 * k_shift (NULL: none): fp32 [Hkv, D], 16-byte aligned, subtracted from every key (in fp32): K-smoothing
 * with a fixed mean (SageBwd summary, Results).  A shift that is the same for every token of a head
 * leaves the softmax as it is and moves LSE by -sm_scale q . k_shift.
 * Per (page, head), with a = max|x| over the call's tokens in the page and r = RN32(1/127) (INT8) or
 * RN32(1/448) (e4m3): s = RN32(a r) if the page holds no earlier token, else max(its scale, RN32(a r));
 * code = rint(RN32(x / s)) or e4m3(RN32(x / s)), saturating.  Where s has grown, an earlier code c becomes
 * the code of RN32(c s_old) under s.  A block whose s is 0 has codes 0.  Values must be finite, which is not
 * checked: a block's scale passes a NaN over; its code is any in int8, and in e4m3 NaN, which attention answers with
 * NaN up to 32 query rows of a shared head and reads as +-480 beyond.
 * A slot's tokens are written in order: what a page holds behind the call's tokens counts as not written yet.
 * Not written, with SAGE_ERR_INVALID_ARG in the status word: tokens of a slot without room for all of them
 * (pos[s] + n_new[s] past lengths[s], to which sage_attn_kv_extend has raised it, or n_new[s] past Nn); a page
 * that another slot lists too (refs != 1); a batch row that names the slot of an earlier row again.
 */
int sage_attn_kv_append(const sage_kv_cache *cache, const void *K, const void *V, const float *k_shift,
                        const int *slots, const int *pos, const int *n_new, int B, int Nn, void *stream);

/*
 * Attention of queries over the cache.  Q: bf16 [B, H, Nq, D], query head h reads key/value head
 * h / (H / Hkv); O as Q, LSE fp32 [B, H, Nq], all apart in memory.  Batch row b reads slot slots[b] (NULL:
 * slot b; a slot may be named by several rows); its first q_len[b] queries count (q_len int32 [B], values
 * outside 0 .. Nq count as the nearest; NULL: Nq), rows behind them are neither read nor written.  With
 * len = lengths[slot]: causal (causal != 0) lets query i see keys j <= len - q_len + i, as for the newest q_len
 * tokens of the sequence; otherwise every query sees all len keys (an encoder's states of another length).
 * The keys of a page number out of range are left out, a slot or length out of range counts as no keys
 * (SAGE_ERR_INVALID_ARG in the status word).
 * S = sm_scale q . k, O = softmax(S) V, LSE = log sum e^S; a row that sees no key has O = 0 and
 * LSE = -infinity.  Codes and queries enter the products exactly (a query's elements below 2^-25 of its
 * largest are rounded); P is rounded to fp16 relative to the running maximum; everything else is fp32.
 * V scales below 2^-80 are read as 2^-80.  sm_scale <= 0 selects 1/sqrt(D).  A query row with a NaN is NaN.
 * ws: sage_attn_kv_ws_bytes(B, H, Hkv, D, Nq) bytes, 16-byte aligned, contents free before and after.
 * Deterministic: the same call on the same state gives the same bits (another batch may cut the keys
 * elsewhere and differ in the last ones).  B is at most 4096.
 */
size_t sage_attn_kv_ws_bytes(int B, int H, int Hkv, int D, int Nq);
int sage_attn_kv_attention(const sage_kv_cache *cache, const void *Q, const int *slots, const int *q_len, void *O,
                           float *LSE, void *ws, size_t ws_bytes, int B, int H, int Nq, int causal, float sm_scale,
                           void *stream);

/*
 * Pages.  Arrays are int32 [n_slots], one entry per slot; results do not depend on the order in which
 * the GPU works.
 *  - fork: slot s with src[s] >= 0 takes over slot src[s]: its pages (shared, refs + 1) and length.  Slot
 *    s must be empty and src[s] must not take over itself (else SAGE_ERR_INVALID_ARG in the status word,
 *    and slot s is left alone).  src[s] < 0: nothing.
 *  - extend: room for n_new[s] >= 0 more tokens: pos[s] = lengths[s], lengths[s] += n_new[s].  The pages
 *    it takes are the free pages with the lowest numbers, in slot order.  A last page that is partly
 *    filled and listed by another slot too is first copied to a page of the slot's own; cow[s] = the page
 *    it was copied from (else -1).  A slot is served if it needs no page, or if the needs of all slots up to it
 *    fit in the free pages; one that is not served has pos[s] = -1 and is otherwise left alone
 *    (SAGE_ERR_NO_PAGES; past max_pages pages: SAGE_ERR_INVALID_ARG).  n_new, pos and cow are apart.
 *  - truncate: slot s with keep[s] >= 0 keeps its first min(keep[s], lengths[s]) tokens and gives the
 *    pages behind them back (refs - 1); keep[s] = 0 frees the slot.
 *  - compact: the live pages of `cache` (refs > 0), in order, become pages 0, 1, ... of the pool `to`;
 *    tables, lengths and refs of `to` follow (its refs behind them 0).  The caches have equal page, Hkv,
 *    D, kind, n_slots and max_pages, may differ in n_pages, and share no memory but, if the caller
 *    likes, the status word; errors go to the one of `cache`.  More live pages than `to` has:
 *    SAGE_ERR_NO_PAGES, and `to` is left alone.
 *    A listed page that is out of range or free (refs 0) is -1 in the table of `to`, SAGE_ERR_INVALID_ARG.
 *    ws: sage_attn_kv_compact_ws_bytes(cache->n_pages) bytes, 16-byte aligned.
 */
int sage_attn_kv_fork(const sage_kv_cache *cache, const int *src, void *stream);
int sage_attn_kv_extend(const sage_kv_cache *cache, const int *n_new, int *pos, int *cow, void *stream);
int sage_attn_kv_truncate(const sage_kv_cache *cache, const int *keep, void *stream);
size_t sage_attn_kv_compact_ws_bytes(int n_pages);
int sage_attn_kv_compact(const sage_kv_cache *cache, const sage_kv_cache *to, void *ws, size_t ws_bytes,
                         void *stream);

/* Fill `views` with the device pointers inside a quantize workspace (qmean, dsb: NULL). */
int sage_attn_ws_views(void *ws, int B, int H, int N, int D, sage_ws_views *views);

/* Synchronise `stream`, read and clear the workspace status word.  Returns SAGE_OK
 * or SAGE_ERR_TIMEOUT (or SAGE_ERR_CUDA if the read itself failed); for the status word of
 * a cache also SAGE_ERR_NO_PAGES and SAGE_ERR_INVALID_ARG. */
int sage_attn_get_status(void *ws, void *stream);

/* Self-test of the bounded wait: launches one warp that waits on a barrier nothing
 * arrives at, with a budget of `budget_ns` nanoseconds (capped at 1 s); the kernel
 * gives up, records SAGE_ERR_TIMEOUT in the status word of `ws` and returns. */
int sage_attn_selftest_wait(void *ws, unsigned long long budget_ns, void *stream);

/* Self-test of what follows a wait of sage_attn_kv_attention that ran out: launches the join of its partial
 * results alone (no q_len: Nq queries each), over a workspace that the caller has filled.  ws: for each of the
 * B * tiles * Hkv units (tiles = ceil(H / Hkv * Nq / R); R query rows: 8 up to 8 of a shared head, 16 up to 32, else
 * 256) int32 first and last part, then from the next multiple of 256 bytes the parts, part k of a unit at place
 * 2 k + 1 if it is the first, else 2 k: fp32 [R, D] sums, [R] maxima (powers of two), [R] row sums.  The rows of
 * a unit whose parts are not two or more within the workspace are left. */
int sage_attn_selftest_kv_join(const sage_kv_cache *cache, void *O, float *LSE, void *ws, size_t ws_bytes, int B,
                               int H, int Nq, void *stream);

/* Size of the library-owned scratch array used by sage_attn_bwd_noalloc. */
#define SAGE_ATTN_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * Backward without a caller-supplied scratch buffer.  The pages have no
 * counterpart to this call; it exists for callers that cannot allocate device
 * memory: code running while a CUDA graph is being captured (where a fresh
 * allocation is not allowed), hosts whose memory pool owns every device byte and
 * forbids allocations from extensions, and real-time or embedded deployments
 * that allocate nothing after start-up.  They still pass the inputs, outputs and
 * the quantize workspace, exactly as for sage_attn_bwd, and get the same result.
 *
 * The scratch is one fixed array of SAGE_ATTN_NOALLOC_SCRATCH_BYTES inside the
 * library; every GPU that loads the library holds it until the process exits.
 * Shapes whose scratch (sage_attn_bwd_ws_bytes) exceeds it are rejected with
 * SAGE_ERR_UNSUPPORTED before anything is launched.  The call allocates nothing.
 * Its first call on a device looks up the array's device address with that
 * device current; make that first call before any stream capture.
 * Every call shares the one array and each call clears what must start at zero,
 * so calls are independent in sequence, but calls that overlap on the GPU (on
 * different streams, or from several threads) race on the array.
 */
int sage_attn_bwd_noalloc(const void *Q, const void *K, const void *V, const void *O, const float *LSE,
                          const void *dO, void *dQ, void *dK, void *dV, const void *ws, int B, int H,
                          int N, int D, int causal, int qk_norm, int k_smooth, float sm_scale,
                          void *stream);

/*
 * One training step of the attention block on HOST-resident tensors: the quantize
 * pass, the forward and the backward above, with the host<->device copies overlapped
 * with the computation.  Every pass of the scheme treats heads independently, so the
 * B*H heads are split into `groups` contiguous ranges (groups <= 0: automatic, 5 or
 * fewer; at most 64; with 3 ranges or more the first and last hold half the heads of the
 * others): the inputs of all ranges are copied in on one copy stream, range g
 * runs on `stream` once its inputs have landed, and its outputs are copied out on a
 * second copy stream while range g+1 runs.  The results equal those of the three calls
 * on device tensors.
 *  - Q, K, V, dO: host bf16 [B, H, N, D] (read).  O, dQ, dK, dV: host bf16 [B, H, N, D]
 *    and LSE: host fp32 [B, H, N] (written).  Page-locked host memory lets the copies
 *    run asynchronously; with pageable memory the call is correct but the copies do
 *    not overlap the computation.
 *  - dev: device scratch, 256-byte aligned, of sage_attn_step_host_bytes(B, H, N, D,
 *    groups) bytes (the same `groups`): device copies of the inputs and outputs and
 *    the workspaces of one head range.  It begins with a quantize workspace whose
 *    status word collects the errors of every range: read it with
 *    sage_attn_get_status(dev, stream).
 *  - Returns once everything is enqueued; the outputs are in host memory when work
 *    enqueued on `stream` before the next call completes (e.g. after
 *    cudaStreamSynchronize(stream)).  The library's two copy streams are shared by all
 *    calls of the process: calls from several host threads at once are not supported.
 */
size_t sage_attn_step_host_bytes(int B, int H, int N, int D, int groups);
int sage_attn_step_host(const void *Q, const void *K, const void *V, const void *dO, void *O, float *LSE,
                        void *dQ, void *dK, void *dV, void *dev, size_t dev_bytes, int B, int H, int N,
                        int D, int causal, int qk_norm, int k_smooth, float sm_scale, int groups,
                        void *stream);

/* Kernel timing for benchmarks.  While enabled (on != 0) the library brackets
 * each launch group with CUDA events recorded on the launching stream: "quantize"
 * (the two quantize kernels), "fwd", "bwd_pre" (D_i, LSE*log2e, dO codes),
 * "bwd_main" and "bwd_dq"; of the cache calls "kv_append", "kv_attention", "kv_pages" (fork,
 * extend, truncate) and "kv_compact".  Costs two event records per group; off by default. */
int sage_attn_timer_enable(int on);

/* Restrict the timing to the launch group `kernel` (one of the names above; NULL:
 * every group).  An event recorded between two launches orders the second after the
 * first's completion, so timing every group removes the overlap of each launch with
 * its predecessor's tail; timing one group keeps it everywhere else. */
int sage_attn_timer_only(const char *kernel);

/* Synchronise the events recorded for `kernel` since the last read, store their
 * summed duration (ms) and number of launches, and forget them.  Unknown names
 * give zero. */
int sage_attn_timer_read(const char *kernel, double *total_ms, int *launches);

/* Static description of a status code. */
const char *sage_attn_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* SAGE_ATTN_H */
