/*
 * mikv.h - C ABI of libmikv.so, the GB300 (sm_103a) hot path of MiKV, the
 * importance-aware mixed-precision KV cache ("No Token Left Behind: Reliable KV
 * Cache Compression via Importance-Aware Mixed Precision Quantization", arXiv
 * 2402.18096), with the optional CriticalKV two-stage selection (arXiv
 * 2502.03805).
 *
 * Sources cited below:
 *   [notes]      "No Token Left Behind" reading notes (velog.io), sections
 *                "Observation", "Key contributions 1)-3)", "3.4 Accelerating the
 *                Mixed-Precision KV Cache".
 *   [paperlayer] paperlayer.ai summary of arXiv 2402.18096v1, sections 3.1-3.4,
 *                4.1, 5, Appendix C.
 *   [criticalkv] gist.science summary of arXiv 2502.03805 (CriticalKV),
 *                "Theoretical framework" and "Algorithm: perturbation-constrained
 *                selection".
 *
 * Conventions shared by every call
 * --------------------------------
 * - Every array pointer is a DEVICE pointer owned by the caller.  The library
 *   never allocates device memory; scratch comes from a caller workspace whose
 *   size a *_workspace_bytes query returns.
 * - fp16 arrays are passed as uint16_t* holding IEEE binary16 bit patterns.
 * - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *   Calls are asynchronous on that stream; none synchronises the host.
 * - All shapes are row-major, innermost dimension last, contiguous.
 * - Return value: MIKV_OK (0) or a negative status.  On any error nothing is
 *   launched and nothing is written; mikv_last_error() returns a message
 *   (thread-local, valid until the next call on the same thread).
 * - Head dimension D must be 128 (the kernels are specialised for it); the
 *   quantisation group is gs = D/2 = 64 ([notes] "2) Outlier-aware": group size
 *   = half the attention head dimension, against RoPE artefacts).
 * - GQA: Hq query heads, Hkv key/value heads, rep = Hq/Hkv in 1..8; query head
 *   h reads key head h / rep.
 */
#ifndef MIKV_H_
#define MIKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define MIKV_OK 0
#define MIKV_EINVAL (-1)       /* null pointer where one is required, bad enum, bad scalar */
#define MIKV_ESHAPE (-2)       /* dimension, capacity or count out of range */
#define MIKV_EALIGN (-3)       /* a buffer is not 16-byte aligned */
#define MIKV_EUNSUPPORTED (-4) /* bit width or head dimension the kernels do not implement */
#define MIKV_ECUDA (-5)        /* a CUDA launch failed (message in mikv_last_error) */

/* mikv_score_update modes */
#define MIKV_PREFILL 0
#define MIKV_DECODE 1

/* mikv_select policies */
#define MIKV_H2O 0
#define MIKV_CRITICALKV 1
#define MIKV_DEMOTE 2

/* mikv_quantize_append tiers */
#define MIKV_TIER_HI 0
#define MIKV_TIER_LO 1
#define MIKV_TIER_DEMOTE 2

/* mikv_cache.key_mode: how the low tier stores keys */
#define MIKV_KEYS_PER_TOKEN 0   /* per-token asymmetric groups of 64 channels (MiKV) */
#define MIKV_KEYS_PER_CHANNEL 1 /* per-channel groups of 64 slots (the Appendix C alternative) */

/*
 * One layer's two-tier cache ([notes] "Key contributions 1)" and "3)": tokens
 * an eviction policy would drop are kept in low precision next to the important
 * tokens kept in FP16 or INT8; [notes] 3.4: after positional embedding
 * attention is permutation invariant, so each precision lives in its own
 * contiguous tier).  Counts are uniform over (batch, key head).
 *
 * Slot layouts (all per [B][Hkv][capacity]):
 *   hi_bits == 16: k_hi, v_hi fp16 [B][Hkv][cap_hi][D]; hi meta unused (NULL).
 *   hi_bits == 8 or 4: k_hi, v_hi uint8 codes [B][Hkv][cap_hi][D*hi_bits/8],
 *                  packed as the lo tier below; k_hi_meta, v_hi_meta
 *                  [B][Hkv][cap_hi][D/64][2] fp16 (scale, zero).  An INT4 important
 *                  tier with an INT2 low tier is the INT4/INT2 split of the pages'
 *                  precision sweeps ([notes] "3)", [paperlayer] 4.1).
 *   lo tier:       k_lo, v_lo uint8 [B][Hkv][cap_lo][D*lo_bits/8] packed codes:
 *                  channel c sits in bits [(c*lo_bits) % 8, +lo_bits) of byte
 *                  (c*lo_bits)/8, least significant bits first;
 *                  k_lo_meta, v_lo_meta [B][Hkv][cap_lo][D/64][2] fp16 (scale, zero).
 *   pos_hi, pos_lo int32: original sequence position of each slot.
 *   scores         fp32 [B][Hkv][cap_hi]: accumulated H2O importance of each hi slot.
 *   balancer       fp32 [B][Hkv][D] or NULL (identity).
 * lo_bits <= hi_bits.  Quantised keys (INT8/INT4 hi tier and the lo tier) hold I(k*b); the FP16 tier holds
 * the original k.  Values are never balanced.
 * Code and meta buffers must be 16-byte aligned.
 *
 * key_mode == MIKV_KEYS_PER_CHANNEL ([notes] Appendix C remarks: per-channel quantisation
 * isolates outlier channels, but a cache then has to hold KV pairs in a buffer until enough
 * have accumulated; [paperlayer] C: group size 64, keys per channel, 20 % FP16 / 80 % INTx):
 *   hi_bits must be 16 and lo_bits 2 or 4; cap_lo a multiple of 64; the balancer is not used.
 *   The low tier's slots [0, n_lo - n_lo % 64) form closed groups of 64 slots: k_lo holds
 *   per-token code rows as above, but their scale and zero are per (group, channel):
 *   k_lo_meta [B][Hkv][cap_lo/64][D][2] fp16 (scale, zero), the per-token quantizer's rule
 *   applied to each channel's 64 values; v_lo and v_lo_meta stay per token.
 *   The last n_lo % 64 retained pairs wait unquantised:
 *   k_pend, v_pend fp16 [B][Hkv][64][D], row p = slot n_lo - n_lo % 64 + p (pos_lo holds their
 *   positions).  The pair that brings them to 64 closes the group: its keys are quantised per
 *   channel and its values per token into the group's slots.  Attention reads closed groups
 *   and waiting pairs (as stored); waiting pairs are attended with the original q.
 * key_mode == MIKV_KEYS_PER_TOKEN (0): k_pend, v_pend unused (NULL).
 */
typedef struct mikv_cache {
  int32_t B, Hkv, Hq, D;
  int32_t hi_bits, lo_bits; /* hi in {16, 8, 4}; lo in {2, 4, 8}, lo <= hi */
  int32_t cap_hi, cap_lo;
  int32_t n_hi, n_lo; /* current counts; updated on the host by the calls that change them */
  void* k_hi;
  void* v_hi;
  void* k_hi_meta;
  void* v_hi_meta;
  void* k_lo;
  void* v_lo;
  void* k_lo_meta;
  void* v_lo_meta;
  int32_t* pos_hi;
  int32_t* pos_lo;
  const float* balancer;
  float* scores;
  int32_t key_mode; /* MIKV_KEYS_PER_TOKEN or MIKV_KEYS_PER_CHANNEL */
  void* k_pend;     /* per-channel keys: waiting pairs, fp16 [B][Hkv][64][D] */
  void* v_pend;
} mikv_cache;

/*
 * Channel balancer ([notes] "2) Outlier-aware", balancer equation; [paperlayer]
 * 3.2): b[b][g][c] = sqrt(Mq / Mk), Mq = max over the group's query heads and
 * the T prompt tokens of |q[b][h][t][c]|, Mk = max over t of |k[b][g][t][c]|;
 * b = 1 where Mq or Mk is 0.  The ratio and the square root are fp32,
 * round-to-nearest-even.  q, k are the post-RoPE prompt tensors.
 *   q    fp16 [B][Hq][T][D]      k fp16 [B][Hkv][T][D]
 *   b_out fp32 [B][Hkv][D]       (written)
 *   ws   >= mikv_balance_workspace_bytes(B, Hkv, D) bytes, 16-byte aligned
 * Errors: EINVAL (null), ESHAPE (T < 1, Hq % Hkv, rep > 8), EUNSUPPORTED (D != 128),
 * EALIGN, ECUDA.
 */
int mikv_balance_prefill(const uint16_t* q, const uint16_t* k, int B, int Hq, int Hkv, int T,
                         int D, float* b_out, void* ws, size_t ws_bytes, void* stream);
size_t mikv_balance_workspace_bytes(int B, int Hkv, int D);

/*
 * Allocation-free variant of mikv_balance_prefill (the paper has no counterpart:
 * this is a deployment convenience).  Same inputs, output and result, but no
 * workspace argument: the scratch lives in a static device array inside the
 * library.  It is meant for callers that cannot allocate device memory, such as
 * a plugin that its host framework hands only input and output buffers, or a
 * serving loop that must never enter the allocator (cudaMalloc/cudaFree
 * synchronise the device and may fail under memory pressure).
 *   Limit: B * Hkv <= 1024 (the array holds 2 x 1024 x 128 floats, 1 MiB, on
 *   every device that loads the library, until the process exits); larger
 *   shapes return MIKV_ESHAPE.
 *   Every call looks up that array's device address in the context current on
 *   the calling thread (a lookup, not an allocation), so the address stays right
 *   after cudaDeviceReset or under another context.  The first call on a device
 *   may load the library's device code there; make it before any stream capture.
 *   All calls share the one array and each clears it first: calls whose kernels
 *   can overlap on the GPU (different streams, without ordering) race and
 *   return wrong results.  Calls allocate nothing.
 * Errors: as mikv_balance_prefill, plus ESHAPE above the limit and ECUDA if the
 * array's address cannot be obtained.
 */
int mikv_balance_prefill_noalloc(const uint16_t* q, const uint16_t* k, int B, int Hq, int Hkv,
                                 int T, int D, float* b_out, void* stream);

/*
 * H2O importance ([notes] "Observation 1-4" and "Key contributions 1)": H2O,
 * accumulated attention; read as the plain H2O definition).
 * MIKV_PREFILL: column sums of the causal softmax over the T prompt rows,
 *   S^h[b][h][i] = sum_{t >= i} exp(q_t.k_i/sqrt(D) - lse_t), and the group sum
 *   S[b][g][i] = sum over the group's query heads, h ascending, fp32.
 *   Uses q fp16 [B][Hq][T][D], k fp16 [B][Hkv][T][D] and the dims of c
 *   (c->B, Hkv, Hq, D; no cache buffer is touched).
 *   scores_full fp32 [B][Hkv][T] (written); scores_head fp32 [B][Hq][T] (written if not NULL).
 *   ws >= mikv_score_workspace_bytes(B, Hq, T) bytes.
 * MIKV_DECODE: c->scores[b][g][j] += sum_h exp(hi_logits[b][h][j] - lse[b][h]) for
 *   every hi slot j < c->n_hi; hi_logits fp32 [B][Hq][cap_hi] and lse fp32 [B][Hq]
 *   as written by mikv_decode_attention.  q, k, T, scores_*, ws unused.
 * Errors: EINVAL, ESHAPE, EUNSUPPORTED, ECUDA.
 */
int mikv_score_update(int mode, const uint16_t* q, const uint16_t* k, int T,
                      const float* hi_logits, const float* lse, mikv_cache* c,
                      float* scores_full, float* scores_head, void* ws, size_t ws_bytes,
                      void* stream);
size_t mikv_score_workspace_bytes(int B, int Hq, int T);

/*
 * Selection.  Budget n_keep(L) = min(L, max(window, floor(budget_pct*L/100))):
 * the `window` most recent positions are always kept and count inside the
 * budget ([paperlayer] 5: local tokens and heavy hitters).  Ranking key
 * (score descending, position ascending); ties keep the lower position.
 * MIKV_H2O ([notes] "Key contributions 1)"): keep the window plus the top
 *   n_keep - window older tokens by scores [B][Hkv][L].
 * MIKV_CRITICALKV ([criticalkv] "Algorithm"): bud = n_keep - window,
 *   b' = floor(alpha*bud), b'' = bud - b'; stage 1 takes the top b' older tokens
 *   by scores; stage 2 takes the top b'' of the remaining older tokens by
 *   C_i = sum_h fl(S^h_i * N[b][h][i]) (fp32, h ascending over the group), with
 *   S^h = scores_head [B][Hq][L] and N the projected-value L1 norms
 *   ([criticalkv] "Theoretical framework": V W_O):
 *     N[b][h][i] = || v[b][h/rep][i][:] . w_o[h*D:(h+1)*D][:] ||_1.
 *   If w_o != NULL, N is computed from v fp16 [B][Hkv][L][D] and w_o fp16
 *   [Hq*D][hidden] (hidden % 128 == 0) and written to vwo_norm fp32 [B][Hq][L];
 *   if w_o == NULL, vwo_norm is read as given.
 * Outputs (H2O, CRITICALKV): keep_pos int32 [B][Hkv][n_keep] ascending,
 *   evict_pos int32 [B][Hkv][L - n_keep] ascending, keep_scores fp32
 *   [B][Hkv][n_keep] = scores at keep_pos (written if not NULL).
 * MIKV_DEMOTE: reads c->scores, c->pos_hi and c->n_hi; among hi slots with
 *   pos < L - window picks the minimum of (score ascending, position descending)
 *   and writes its slot index to evict_pos [B][Hkv]; L is the current length.
 *   Requires c->n_hi > window.
 * ws >= mikv_select_workspace_bytes(policy, B, Hkv, Hq, L, hidden), 16-byte aligned;
 *   CRITICALKV keeps the stage-2 keys there and, when w_o != NULL, a transposed copy of
 *   w_o ([hidden][Hq*D] fp16, so both tensor-core operands are channel-contiguous).
 * Errors: EINVAL (null, policy, alpha outside [0,1]), ESHAPE (L, budget, window,
 * hidden, B*Hkv*L >= 2^31), EALIGN (v, w_o, ws), EUNSUPPORTED, ECUDA.
 */
int mikv_select(int policy, const mikv_cache* c, int L, int budget_pct, int window, float alpha,
                const float* scores, const float* scores_head, const uint16_t* v,
                const uint16_t* w_o, int hidden, float* vwo_norm, int32_t* keep_pos,
                int32_t* evict_pos, float* keep_scores, void* ws, size_t ws_bytes, void* stream);
size_t mikv_select_workspace_bytes(int policy, int B, int Hkv, int Hq, int L, int hidden);

/*
 * Quantise-and-append ([notes] "Key contributions 1)": per-token asymmetric
 * quantisation (LLM-QAT) of the retained tokens; "2)": keys as I(k*b);
 * "3)": INT8 important tier).  Per token, key head and 64-channel group:
 *   x = fl(k*b) for keys of a quantised tier, x = v for values;
 *   s = fp16(fl(max-min)/qmax), z = fp16(min),
 *   code = clamp(rint_even(fl(fl(x - z)/s)), 0, qmax), code 0 where s == 0.
 * MIKV_TIER_HI: slots n_hi..n_hi+n_tokens-1 take source tokens src_pos
 *   [B][Hkv][n_tokens] (indices into k, v fp16 [B][Hkv][src_len][D]); FP16
 *   tier: copy; INT8 tier: quantise.  pos_hi = src_pos + pos_base;
 *   scores = src_scores [B][Hkv][n_tokens] if not NULL, else 0.  n_hi += n_tokens.
 * MIKV_TIER_LO: same into the lo tier (lo_bits); pos_lo = src_pos + pos_base.
 *   n_lo += n_tokens.
 * MIKV_TIER_DEMOTE: n_tokens must be 1; src_pos [B][Hkv] are hi slots.  Each is
 *   re-quantised into lo slot n_lo from what the hi tier holds (FP16: fl(k*b)
 *   and v; INT8: fl(fl(s*code)+z), already balanced); then the last hi slot
 *   (k, v, meta, pos, score) moves into the freed slot.  n_hi -= 1, n_lo += 1.
 *   k, v, src_len, pos_base, src_scores unused.
 * Per-channel keys (c->key_mode == MIKV_KEYS_PER_CHANNEL): MIKV_TIER_LO requires n_lo % 64 == 0;
 *   the first floor(n_tokens / 64) * 64 tokens close groups at once (keys per channel, values
 *   per token), the rest wait in k_pend / v_pend.  MIKV_TIER_DEMOTE moves the victim's FP16
 *   pair into the waiting buffer (no quantisation); when it is the 64th waiting pair, a second
 *   launch closes the group.  MIKV_TIER_HI is unchanged (FP16 copy).
 * Counts in *c are updated on the host after a successful launch.
 * Errors: EINVAL, ESHAPE (capacity overflow, src_len, a per-channel LO append off a group
 * boundary), EALIGN, EUNSUPPORTED, ECUDA.
 */
int mikv_quantize_append(int tier, const uint16_t* k, const uint16_t* v, int src_len,
                         const int32_t* src_pos, int n_tokens, int pos_base,
                         const float* src_scores, mikv_cache* c, void* stream);

/*
 * Decode attention over the two-tier cache ([notes] 3.4 and [paperlayer] 3.4:
 * tiers grouped by precision, K and V low precision, Q and the attention map
 * floating point; [notes] "2)": quantised keys are attended with q/b).
 * For query head h of key head g:
 *   FP16 hi tier:  logit = q_h . k / sqrt(D)        (original q and k)
 *   quantised tiers: logit = (q_h / b_g) . k~ / sqrt(D)   (k~ dequantised k*b)
 *   p = softmax over both tiers; out_h = sum p v~; lse_h = log sum exp(logit).
 *   q      fp16 [B][Hq][D]
 *   out    fp32 [B][Hq][D]; lse fp32 [B][Hq] (natural log)
 *   hi_logits fp32 [B][Hq][cap_hi] (slots < n_hi written) or NULL
 *   ws >= mikv_decode_workspace_bytes(c) bytes (split-K partial results and the
 *   per-(batch, key head) query fragments).
 * Per-channel keys: closed groups give logit = (q_h . (s (.) code + z)) / sqrt(D) with the
 *   group's per-channel scale s and zero z (no balancer); waiting pairs are attended as FP16
 *   with the original q, like the FP16 tier.  The workspace also holds the fp32 query.
 * Requires n_hi + n_lo >= 1.  Errors: EINVAL, ESHAPE, EALIGN, EUNSUPPORTED, ECUDA.
 */
int mikv_decode_attention(const uint16_t* q, const mikv_cache* c, float* out, float* lse,
                          float* hi_logits, void* ws, size_t ws_bytes, void* stream);
size_t mikv_decode_workspace_bytes(const mikv_cache* c);

/*
 * One whole decode step in four launches (the same arithmetic as the sequence
 * quantize_append(HI) -> decode_attention -> score_update(DECODE) ->
 * select(DEMOTE) -> quantize_append(DEMOTE), with identical results):
 *   1. the new token (k_new, v_new fp16 [B][Hkv][D], position `pos`) is appended
 *      to the important tier with score 0 (the same launch prepares the query);
 *   2. q fp16 [B][Hq][D] attends over both tiers (split-K partials);
 *   3. the partials are merged into out fp32 [B][Hq][D] and lse fp32 [B][Hq];
 *   4. the step's attention is added to the H2O score of every important slot,
 *      and, if policy == MIKV_H2O and the important tier now holds more than
 *      n_keep(pos + 1) tokens, the victim (see mikv_select(MIKV_DEMOTE)) is
 *      demoted.  MIKV_CRITICALKV never demotes.
 * The order follows H2O: evict after the step's attention ([notes] "Key
 * contributions 1)"; [paperlayer] 5).  Per-channel keys: the demoted pair joins the waiting
 * buffer, and a fifth launch closes its group when it is the 64th.  ws >= mikv_decode_step_workspace_bytes(c)
 * (partials, the important-tier logits, per-chunk victim candidates).  Counts in
 * *c are updated.  Two calls must not share a workspace concurrently.
 * Errors: EINVAL, ESHAPE (capacity, budget, workspace), EALIGN, EUNSUPPORTED
 * (cap_hi above 65535*1024), ECUDA.
 */
int mikv_decode_step(const uint16_t* q, const uint16_t* k_new, const uint16_t* v_new, int pos,
                     int budget_pct, int window, int policy, mikv_cache* c, float* out, float* lse,
                     void* ws, size_t ws_bytes, void* stream);
size_t mikv_decode_step_workspace_bytes(const mikv_cache* c);

/*
 * K9: the step after attention ([criticalkv] "Theoretical framework": the output
 * perturbation L = ||o - o^||_1 of replacing the full cache, bounded through the value
 * states projected by W_O; "Experimental results": reported per attention head).
 * Head h reaches the hidden state through rows h*D .. h*D + D - 1 of W_O:
 *   y[b][:]  = sum_h o[b][h][:] . W_O^(h)                      (the output projection)
 *   pert[b][h] = || (o[b][h][:] - o_hat[b][h][:]) . W_O^(h) ||_1  (sum over hidden)
 * o, o_hat fp32 [B][Hq][D] (D = 128): e.g. decode attention over the full cache and over
 * the mixed-precision (or evicted) cache.  w_o_t fp16 [hidden][Hq*D], row-major: W_O
 * transposed, the layout nn.Linear stores; hidden % 128 == 0; 16-byte aligned.
 * y fp32 [B][hidden] is written if not NULL; pert fp32 [B][Hq] if not
 * NULL (needs o_hat).  With w_o_t == NULL, pert[b][h] = || o - o_hat ||_1 over D (y must
 * be NULL).  Products are formed from fp16 (hi, lo) splits of o and o - o_hat with fp32
 * accumulation (relative error ~1e-6).
 * ws >= mikv_output_perturbation_workspace_bytes(B, Hq, hidden), 16-byte aligned
 * (operand tiles and per-column partial sums).  Stream-ordered; no synchronisation.
 * Errors: EINVAL (null o, pert without o_hat, y without w_o_t, null ws), EUNSUPPORTED (D),
 * ESHAPE (B < 1, Hq outside 1..128, hidden, workspace), EALIGN, ECUDA.
 */
int mikv_output_perturbation(const float* o, const float* o_hat, const uint16_t* w_o_t, int B, int Hq,
                             int D, int hidden, float* y, float* pert, void* ws, size_t ws_bytes,
                             void* stream);
size_t mikv_output_perturbation_workspace_bytes(int B, int Hq, int hidden);

/*
 * Post-attention top-k over the full cache ([notes] "1-4) Quantitative analysis": the
 * oracle-eviction simulation computes the attention map over the full cache first and
 * applies top-k sparsity after the attention, an upper-bound proxy for eviction).
 * c must hold the full cache in its FP16 tier (hi_bits 16, n_lo 0, n_hi = L >= 1 tokens,
 * e.g. a prefill at budget 100).  Per (batch, query head) the k = max(1, floor(p*L/100))
 * largest logits q.k/sqrt(D) are kept (ties to the lower slot) and
 *   out[b][h] = sum_{i kept} exp(l_i - m) v_i / sum_{i kept} exp(l_i - m),
 *   lse[b][h] = log sum_{i kept} exp(l_i)            (natural log; written if not NULL),
 *   keep_idx [B][Hq][k] int32 = the kept slots, ascending (written if not NULL).
 * q fp16 [B][Hq][D]; out fp32 [B][Hq][D].  Three stages, stream-ordered: the decode attention
 * of this cache (all logits), a radix select per head, attention over the kept slots.
 * ws >= mikv_topk_attention_workspace_bytes(c, budget_pct), 16-byte aligned.
 * Errors: EINVAL (null), EUNSUPPORTED (not a full FP16 cache), ESHAPE (budget, heads,
 * n_hi outside 1..131072, workspace), and those of mikv_decode_attention.
 */
int mikv_topk_attention(const uint16_t* q, const mikv_cache* c, int budget_pct, float* out, float* lse,
                        int32_t* keep_idx, void* ws, size_t ws_bytes, void* stream);
size_t mikv_topk_attention_workspace_bytes(const mikv_cache* c, int budget_pct);

/*
 * Per-channel group quantisation of retained-tier keys ([notes] Appendix C remarks;
 * [paperlayer] C: group size 64, keys quantised per channel), standalone: the arithmetic the
 * per-channel cache (mikv_cache.key_mode) applies when it closes a group.
 * k fp16 [units][n][D] (D = 128): each unit's keys in slot order.  The floor(n / 64) full
 * groups are quantised; the n mod 64 keys after them are left alone (they wait in FP16 until
 * a group is full).  Per (group, channel c), over the group's 64 values of channel c:
 *   s = fp16(fl(fl(mx - mn) / qmax)), z = fp16(mn),
 *   code = clamp(rint_even(fl(fl(x - z) / s)), 0, qmax), 0 where s == 0.
 * codes uint8 [units][n][D*bits/8]: per-token rows (channel c at bits (c*bits) mod 8 of byte
 * c*bits/8, LSB first), rows of full groups written; meta fp16 [units][n/64][D][2] =
 * (scale, zero).  bits in {2, 4, 8}.  Stream-ordered.
 * Errors: EINVAL (null), EUNSUPPORTED (D, bits), ESHAPE (units outside 1..65535, n < 0).
 */
int mikv_channel_quantize(const uint16_t* k, int units, int n, int D, int bits, uint8_t* codes,
                          uint16_t* meta, void* stream);

/*
 * The paged cache (no counterpart in the papers: they give one prompt's tiers; a serving loop
 * holds many sequences that differ in length, share prefixes and give memory back).
 *
 * One pool of pages for all layers, one table for all layers: slot j of sequence s lies, in
 * every layer and for every key head, in row j % page_size of page table[s][j / page_size].
 *   k, v    type FP16, BF16: 16-bit rows [layers][n_pages][Hkv][page_size][D]
 *           type INT8: uint8 codes of the same shape, and k_meta, v_meta fp16
 *           [layers][n_pages][Hkv][page_size][D/64][2] (scale, zero): the per-token quantiser
 *           of mikv_quantize_append at 8 bits, unbalanced; rows handed in or out are fp16.
 *   table   int32 [max_seqs][max_pages]; entries past a sequence's pages are not read
 *           (-1 where a call has cleared them)
 *   lens    int32 [max_seqs]: slots of each sequence, 0 for one that is not in use; the
 *           sequence owns the first ceil(len / page_size) entries of its row
 *   refs    int32 [n_pages]: how many sequences own the page; 0 = free.  A page whose count
 *           the caller raises itself is never handed out, and not appended to while the count
 *           is above 1.
 * table, lens and refs are device arrays: the calls below read and change them on the stream,
 * so a whole step can be captured into a CUDA graph.  A new cache has lens 0 and refs 0.
 * Calls that change the same cache must be ordered (one stream, or events), like writes to any
 * buffer.  page_size 1..4096; max_pages * page_size < 2^31 - 4096; n_pages * Hkv * page_size
 * < 2^32 - 1; Hkv <= 1024; buffers 16-byte aligned.
 *
 * Calls over several sequences take their numbers in `seqs` int32 [n] (device), or NULL for
 * 0 .. n - 1 (n <= max_seqs).  The calls that change tables report per request; a request is
 * refused, and changes nothing, where
 *   - a sequence number is outside 0 .. max_seqs - 1, or an earlier request of the same call
 *     names the same sequence,
 *   - its own rule below is broken, or
 *   - it needs pages, and the free ones do not suffice for it and all requests before it that
 *     keep the first two rules (served or not; a compaction's positions are checked later, so
 *     one that is refused for them alone counts too).  A request that needs no page is served.
 * New pages are the free pages of lowest number, in request order.  n is at most 4096 for
 * reserve, fork and compact, 65535 otherwise; n == 0 does nothing.
 */
#define MIKV_PAGES_FP16 0
#define MIKV_PAGES_BF16 1
#define MIKV_PAGES_INT8 2

typedef struct mikv_pages {
  int32_t layers, n_pages, page_size, Hkv, D, type;
  int32_t max_seqs, max_pages;
  void* k;
  void* v;
  void* k_meta; /* INT8 only, else NULL */
  void* v_meta;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
} mikv_pages;

/* A strided view of 16-bit rows [B][H][T][D], D contiguous: element (b, h, t, d) at
 * data[b * stride_b + h * stride_h + t * stride_t + d].  data and the strides are multiples
 * of 16 bytes (8 elements), the strides not negative. */
typedef struct mikv_rows {
  void* data;
  int64_t stride_b, stride_h, stride_t; /* in elements */
} mikv_rows;

/*
 * Reserve: makes room for add[i] >= 0 more tokens behind each sequence, and lengthens it.
 * start[i] (written) is the slot of the first new token, the length before the call, or -1
 * where the request was refused.  Refused too: a length above max_pages * page_size.
 * ws >= mikv_page_workspace_bytes(p, n) bytes, 16-byte aligned (here and below).
 * Errors (all page calls): EINVAL (null), ESHAPE (dimensions, n, workspace), EALIGN,
 * EUNSUPPORTED (D), ECUDA.
 */
int mikv_page_reserve(const mikv_pages* p, const int32_t* seqs, const int32_t* add, int n, int32_t* start, void* ws,
                      size_t ws_bytes, void* stream);

/*
 * Fork: child[i] becomes a copy of parent[i].  Full pages are shared; a partly filled last
 * page is copied in all layers (its filled rows), so either sequence can grow.  ok[i]
 * (written) is 1, or 0 where refused: also where the child's length is not 0, or where the
 * child is a parent of the same call.  One parent may have several children in one call.
 * Append the slots that a parent has reserved before it is forked: the pages they fill are
 * shared by then and no longer written.
 */
int mikv_page_fork(const mikv_pages* p, const int32_t* parent, const int32_t* child, int n, int32_t* ok, void* ws,
                   size_t ws_bytes, void* stream);

/*
 * Free: the sequences give their pages back and have length 0.  ok[i] (written): 1, or 0
 * where refused; freeing an empty sequence is fine.
 */
int mikv_page_free(const mikv_pages* p, const int32_t* seqs, int n, int32_t* ok, void* stream);

/*
 * Copy: page dst[i] takes what page src[i] holds, in all layers, whoever owns them.  ok[i]
 * (written): 1, or 0 where refused: a page outside the pool, a destination that an earlier
 * pair of the call names too, or one that another pair reads.  src[i] == dst[i] does nothing.
 */
int mikv_page_copy(const mikv_pages* p, const int32_t* src, const int32_t* dst, int n, int32_t* ok, void* stream);

/*
 * Compact: sequence i keeps keep_n[i] of its slots; slot j of key head h in layer l becomes
 * what slot keep_pos[l][i][h][j] was (keep_pos int32 [layers][n][Hkv][max_keep], e.g. in each
 * layer's part the keep_pos that mikv_select writes; any order, a slot may be kept twice).  The kept rows move
 * into new pages and the old ones are given back, so a sequence that shares pages may be
 * compacted; the new pages have to be free before the old ones are.  ok[i] (written): 1, or 0
 * where refused: also keep_n[i] outside 0 .. min(max_keep, length), or a position outside the
 * sequence among its keep_n[i].
 */
int mikv_page_compact(const mikv_pages* p, const int32_t* seqs, const int32_t* keep_pos, const int32_t* keep_n, int n,
                      int max_keep, int32_t* ok, void* ws, size_t ws_bytes, void* stream);
size_t mikv_page_workspace_bytes(const mikv_pages* p, int n);

/*
 * Append: tokens 0 .. counts[i] - 1 of row i of k and v ([n][Hkv][T][D], fp16; bf16 for BF16
 * pages) go to slots start[i] .. of its sequence in one layer.  counts NULL: T each (a count
 * above T is T, one below 1 writes nothing).  start: what mikv_page_reserve wrote, rows with
 * start < 0 are skipped; NULL: the sequence's last counts[i] slots.  Slots at or past the
 * sequence's length are not written, nor are rows whose sequence is out of range or named by
 * an earlier row.  Nor are slots on a page whose count is above 1, which a fork shares: they
 * are left as every owner reads them, and reported (mikv_wait_status, bit 128).  Slots that are
 * reserved behind a sequence's last fork never lie on one.  INT8: quantised as in
 * mikv_quantize_append; NaN does not count for a group's extremes, and a quotient that is no
 * number (NaN, infinity / infinity) gives code 0.
 */
int mikv_paged_append(const mikv_pages* p, int layer, const mikv_rows* k, const mikv_rows* v, int n, int T,
                      const int32_t* seqs, const int32_t* start, const int32_t* counts, void* stream);

/*
 * Gather: the first T slots of each sequence, as far as it reaches, as rows k_out and v_out
 * ([n][Hkv][T][D], fp16; bf16 for BF16 pages).  INT8: fp16(fl(fl(scale * code) + zero)).  Rows at
 * or past the sequence's length are left as they were; so are all rows of a sequence number
 * out of range.  The output rows must not overlap one another.
 */
int mikv_paged_gather(const mikv_pages* p, int layer, const int32_t* seqs, int n, int T, const mikv_rows* k_out,
                      const mikv_rows* v_out, void* stream);

/*
 * Attention of one new token per sequence over one layer of the paged cache.  Row i's query
 * stands at the last slot p = len - 1 of its sequence (append its key and value first) and
 * sees slot j where
 *   window == 0, or j > p - window, or j < sinks        (0 <= j <= p)
 * i.e. the `window` most recent slots and the first `sinks` ones.
 *   l_j = q_h . k~_j / sqrt(D), out_h = sum_j exp(l_j - lse) v~_j, lse_h = log sum_j exp(l_j)
 * q, out [n][Hq][D] fp16 (bf16 for BF16 pages), lse fp32 [n][Hq] (natural log; NULL: not
 * written).  A sequence of length 0, or a number out of range, gives out 0 and lse -inf.
 * Hq a multiple of Hkv, up to 1024 query heads per key head; slots that are not seen may
 * hold anything.  ws >= mikv_paged_attention_workspace_bytes(p, n, Hq, window, sinks), 16-byte
 * aligned; two calls must not share a workspace concurrently.
 * Errors: EINVAL (null, window < 0, sinks < 0), ESHAPE (layer, n outside 0..65535, Hq, workspace), EALIGN,
 * EUNSUPPORTED, ECUDA.
 */
int mikv_paged_attention(const void* q, const mikv_pages* p, int layer, const int32_t* seqs, int n, int Hq, int window,
                         int sinks, void* out, float* lse, void* ws, size_t ws_bytes, void* stream);
size_t mikv_paged_attention_workspace_bytes(const mikv_pages* p, int n, int Hq, int window, int sinks);

/*
 * Attention of a prompt, or of a chunk of one, over contiguous keys and values under a sliding
 * window with sinks.  q, out [B][Hq][Tq][D], k, v [B][Hkv][Tk][D], all fp16 (type
 * MIKV_PAGES_FP16) or bf16 (MIKV_PAGES_BF16), strided views.  q_lens, k_lens int32 [B]
 * (device; NULL: Tq, Tk each; held inside 0 .. Tq, 0 .. Tk): the first q_lens[b] query rows and
 * k_lens[b] key rows of batch row b count.  Query i stands at position
 * p = k_lens[b] - q_lens[b] + i, the last one at the last key, and sees key j as in
 * mikv_paged_attention.  A query that sees nothing (p < 0) gives out 0 and lse -inf.
 * lse fp32 [B][Hq][Tq], or NULL.  Query rows at or past q_lens[b] are not written and may hold
 * anything, like key and value rows that no query of the call sees (those at or past k_lens[b],
 * and those between the sinks and the first query's window); a value row that some query sees
 * must be finite, or it may reach the other queries of the same head.
 * Requires 1 <= Tq, Tk <= 2^30, Hq a multiple of Hkv; k and v may repeat one head or batch row
 * (stride 0), rows of q, k, v along T and all rows of out are apart; B == 0 does nothing.
 * The softmax weights are rounded to the inputs' type before they meet the values; sums and
 * statistics are fp32.
 * ws >= mikv_window_attention_workspace_bytes(B, Hq, Hkv, Tq, Tk, window, sinks), 32-byte
 * aligned: sums of calls whose rows would leave SMs idle, and whose keys are shared out (0 bytes, and
 * ws may be NULL, otherwise); two calls must not share a workspace concurrently.
 * Errors: EINVAL (null, type, window, sinks), ESHAPE, EALIGN, EUNSUPPORTED (D), ECUDA.
 */
int mikv_window_attention(const mikv_rows* q, const mikv_rows* k, const mikv_rows* v, int B, int Hq, int Hkv, int Tq, int Tk,
                          int D, int type, const int32_t* q_lens, const int32_t* k_lens, int window, int sinks,
                          const mikv_rows* out, float* lse, void* ws, size_t ws_bytes, void* stream);
size_t mikv_window_attention_workspace_bytes(int B, int Hq, int Hkv, int Tq, int Tk, int window, int sinks);

/*
 * Packed batches: the new tokens of many requests, one request after the other, as rows
 * [rows][H][D] (chunks of prompts beside single tokens).  A row's sequence, position and slot are
 * worked out once a step (mikv_batch_rows) and serve every layer.
 *
 * Request i < n concerns sequence seqs[i] (NULL: i) and has counts[i] rows (below 0: none); its
 * row t stands at position start[i] + t (start: what mikv_page_reserve wrote; NULL: the rows are the
 * sequence's last ones).  Written, with row arrays int32 [rows]:
 *   row_start int32 [n + 1]   rows before request i, at most `rows`; [n]: all of them
 *   row_seq, row_pos          sequence and position; -1, -1 where the request was refused (start < 0, a
 *                             sequence number out of range, more rows than slots with start NULL),
 *                             where an earlier request names its sequence too, and past the last row
 *   row_slot                  the slot of the pool, page * page_size + position % page_size; -1 also at or
 *                             past the sequence's length and on a page outside the pool (reported,
 *                             mikv_wait_status bit 64)
 * Rows of requests that were refused keep their places: a batch is laid out from its counts alone.  What
 * lies past `rows` is cut off: with start NULL the rows that are left of a request are its sequence's last ones.
 * n at most 4096, rows at most 2^30; n_pages * page_size < 2^31; n == 0 with rows == 0 does nothing.
 * Errors: EINVAL (null), ESHAPE, and the cache's (EALIGN, EUNSUPPORTED), ECUDA.
 */
int mikv_batch_rows(const mikv_pages* p, const int32_t* seqs, const int32_t* start, const int32_t* counts, int n, int rows,
                    int32_t* row_start, int32_t* row_seq, int32_t* row_pos, int32_t* row_slot, void* stream);

/*
 * Append by slot: row r of k and v ([rows][Hkv][D] by stride_t and stride_h, stride_b unused; fp16,
 * bf16 for BF16 pages) goes to slot slots[r] of one layer; rows with a slot below 0 are skipped.
 * Stored, quantised and kept off shared pages as by mikv_paged_append; a slot outside the pool is
 * skipped and reported (mikv_wait_status, bit 64).  The slots of a call differ (those of
 * mikv_batch_rows do, for pages of one owner): one that is named twice is left with parts of either row.
 * rows at most 2^30.
 */
int mikv_slot_append(const mikv_pages* p, int layer, const mikv_rows* k, const mikv_rows* v, int rows, const int32_t* slots,
                     void* stream);

/*
 * Bounds of the keys of pages, for mikv_block_select: per (layer, page, key head) the smallest and
 * largest value of every channel over the page's filled slots, in 8 bits.
 *   scale = fl(max_c max(|lo_c|, |hi_c|) / 127),  codes floor(fl(lo_c / scale)), ceil(fl(hi_c / scale)),
 * held inside -127 .. 127, all 0 where scale is 0.  The keys are the stored values (INT8: fl(fl(s *
 * code) + z)).  A page that holds a key that is no finite number has scale infinity and codes 0.
 *   bounds  int8 [layers][n_pages][Hkv][2][D] (lo, hi), 16-byte aligned
 *   scales  fp32 [layers][n_pages][Hkv]
 * The pages that hold the positions (row_seq[r], row_pos[r]), as mikv_batch_rows writes them, are
 * done anew from all that they hold: call it behind each append.  Pages that mikv_page_fork,
 * _copy or _compact have filled need it too: with rows for all their positions (mikv_batch_rows
 * with counts = lengths), in every layer.  Rows without a sequence, or at or past its length, are skipped.
 */
int mikv_page_bounds(const mikv_pages* p, int layer, const int32_t* row_seq, const int32_t* row_pos, int rows, int8_t* bounds,
                     float* scales, void* stream);

/*
 * Blocks to read: for each row and key head, the `keep` blocks (pages of its sequence, in table
 * order) that score highest among those with a position up to the row's own.  Rows as in
 * mikv_page_bounds; row_seq NULL: row r is sequence r; row_pos NULL: the sequence's last slot (a position
 * at or past the length counts as the last slot too).
 * With c = rint(fl(q_c / s_q)), s_q = fl(max_c |q_c| / 127) of each query head, the score of a block is
 *   max over the group's heads of fl(fl(u * scale) * s_q),  u = sum_c (c_c > 0 ? c_c hi_c : c_c lo_c),
 * u exact.  A score that is no number counts as +infinity, so that blocks which hold one are read.
 * Always among the blocks: the first `first` and the last `recent` ones (recent >= 1, first + recent <= keep);
 * equal scores go to the lower block.  A row with `keep` blocks or fewer reads them all.
 *   sel int32 [rows][Hkv][keep]: the blocks in ascending order, -1 behind them;  n_sel int32 [rows][Hkv]
 * q [rows][Hq][D] fp16 (bf16 for BF16 pages).  rows * Hkv <= 65535, Hq a multiple of Hkv, up to 1024 query heads
 * per key head.  ws >= mikv_block_select_workspace_bytes(p, rows, Hq), 16-byte aligned; two calls must
 * not share a workspace concurrently.
 * Errors: EINVAL (null, keep, first, recent), ESHAPE, EALIGN, EUNSUPPORTED, ECUDA.
 */
int mikv_block_select(const void* q, const mikv_pages* p, int layer, const int8_t* bounds, const float* scales,
                      const int32_t* row_seq, const int32_t* row_pos, int rows, int Hq, int keep, int first, int recent,
                      int32_t* sel, int32_t* n_sel, void* ws, size_t ws_bytes, void* stream);
size_t mikv_block_select_workspace_bytes(const mikv_pages* p, int rows, int Hq);

/*
 * Attention of each row over the blocks that sel and n_sel name (as mikv_block_select writes them, or
 * in any order; entries past n_sel, which is held inside 0 .. keep, are not read), as far as their
 * slots lie at or before the row's position.  A block named twice counts twice; one that is none of
 * the row's is not seen and reported (mikv_wait_status, bit 64).  Otherwise as mikv_paged_attention:
 * out [rows][Hq][D], lse fp32 [rows][Hq] or NULL, over the seen slots alone.
 * rows * Hkv <= 65535 (more rows: several calls, each with its part of every array), up to 1024 query heads per key head,
 * keep * page_size at most 2^31 - 4097.
 * ws >= mikv_block_attention_workspace_bytes(p, rows, Hq, keep), 16-byte aligned; two calls must not
 * share a workspace concurrently.
 */
int mikv_block_attention(const void* q, const mikv_pages* p, int layer, const int32_t* row_seq, const int32_t* row_pos,
                         const int32_t* sel, const int32_t* n_sel, int rows, int Hq, int keep, void* out, float* lse, void* ws,
                         size_t ws_bytes, void* stream);
size_t mikv_block_attention_workspace_bytes(const mikv_pages* p, int rows, int Hq, int keep);

/*
 * Attention of the rows of a packed batch over one layer of the paged cache.  Rows row_start[i] ..
 * row_start[i + 1] - 1 (held inside 0 .. rows; int32 [n + 1], ascending, as mikv_batch_rows writes
 * it) are request i's, of sequence seqs[i] (NULL: i); row t of a request stands at position start[i] + t
 * (NULL: the rows are the sequence's last ones) and sees slot j of its sequence (j below the
 * length) as in mikv_paged_attention.  Append the rows' keys and values first.
 * q, out [rows][Hq][D] by stride_t and stride_h (stride_b unused), fp16 (bf16 for BF16 pages); lse fp32
 * [rows][Hq], or NULL.  A row that sees nothing (its request has a start below 0, or without starts more rows than
 * slots, its sequence is empty or out of range) gives out 0 and lse -inf.  Rows of no request are not written.
 * Several requests may name one sequence: each is answered, also those that mikv_batch_rows gives no
 * place to, as an earlier one has it.  Slots that are not seen by any row of a request may
 * hold anything; a value row that one of them sees must be finite, or it may reach the request's
 * other rows.  Slots on a page outside the pool read as zeros (reported, mikv_wait_status bit 64).
 * start is held at 2^30.  The softmax weights are rounded once to 16 bits before they meet the values, single tokens' too
 * (mikv_paged_attention and mikv_block_attention keep two 16-bit parts of each); sums and statistics are fp32.
 * rows at most 2^20, max_pages * page_size at most 2^30, n at most 4096, Hq a multiple of Hkv, up to 1024 query heads per key head; n == 0 or rows == 0 does nothing.
 * ws >= mikv_chunk_attention_workspace_bytes(p, n, rows, Hq), 32-byte aligned; two calls must not share
 * a workspace concurrently.
 * Errors: EINVAL (null, window, sinks, rows of out that overlap), ESHAPE, EALIGN, EUNSUPPORTED, ECUDA.
 */
int mikv_chunk_attention(const mikv_rows* q, const mikv_pages* p, int layer, const int32_t* seqs, const int32_t* start,
                         const int32_t* row_start, int n, int rows, int Hq, int window, int sinks, const mikv_rows* out, float* lse,
                         void* ws, size_t ws_bytes, void* stream);
size_t mikv_chunk_attention_workspace_bytes(const mikv_pages* p, int n, int rows, int Hq);

/*
 * Measurement hook (no counterpart in the papers): while set, every
 * mikv_decode_attention and mikv_decode_step call made by this thread records
 * `begin` (a cudaEvent_t) on its stream just before the split-K attention
 * launch and `end` just after it, so that a caller can time that kernel alone
 * with cudaEventElapsedTime.  The events are owned by the caller and must stay
 * valid while set; (NULL, NULL) clears the hook.  Setting only one of the two
 * is EINVAL.  A failed record is reported as ECUDA by the call that made it.
 */
int mikv_set_attention_events(void* begin, void* end);

/*
 * Wait status of the tensor-core kernels (no counterpart in the papers; a failure report).
 * The tcgen05 kernels (K3's two prefill score passes in mikv_score_update(MIKV_PREFILL),
 * K6's V.W_O norms in mikv_select(MIKV_CRITICALKV) with w_o, K9 in
 * mikv_output_perturbation, mikv_window_attention and mikv_chunk_attention) hand tiles between a TMA/MMA thread and
 * their consumer warps through mbarriers, and every wait there gives up after ~4 million polls instead of
 * spinning for ever.  No wait is expected to run out; if one does, the thread that gave up
 * issues no further copy or MMA, its later waits poll only ~1000 times each (so a stuck
 * pipeline still ends in a bounded time, and what was issued before has that long to land),
 * the kernel writes NaN into the outputs of the affected CTA (prefill scores and -lse rows,
 * V.W_O norms, perturbation and y partial sums, the rows of windowed and packed rows' attention under way; rows that
 * its CTA had taken over and not begun are left as they were, or joined from what the workspace held) and sets a bit in a device-side
 * status word.
 * The call that launched it has already returned MIKV_OK (launches are asynchronous).
 * mikv_wait_status stores the OR of the bits set since the last clear in *bits:
 *   1 = K3 pass 1 (row log-sum-exp), 2 = K3 pass 2 (column sums), 4 = K6 (V.W_O norms),
 *   8 = K9 (output perturbation), 16 = mikv_wait_probe, 32 = mikv_window_attention,
 *   64 = no wait: an append, a gather, row maps, bounds, a choice of blocks or an attention over pages
 *   met a table entry, slot or block outside the pool (skipped, read as zeros, or not seen)
 *   256 = mikv_chunk_attention
 *   128 = no wait: an append met a page that several sequences own (its slots are skipped)
 * and clears them if `clear` is non-zero.  It copies synchronously: call it after the work
 * in question has completed (e.g. after synchronising its stream).
 * Errors: EINVAL (null bits), ECUDA (the copy failed).
 */
int mikv_wait_status(unsigned* bits, int clear);

/*
 * Self-check of the give-up path above (no counterpart in the papers): one thread waits, with
 * the same bounded wait as the tensor-core kernels, on an mbarrier of one arrival that it
 * makes itself only if `arrive` is non-zero.  Without the arrival the first wait gives up
 * after `polls` polls (1 .. 2^24), a second one after the short limit, and status bit 16 is
 * set; with it nothing is set.  No memory is read or written but that bit; the launch does
 * not disturb the context.  Stream-ordered.  Errors: EINVAL (polls), ECUDA (launch).
 */
int mikv_wait_probe(int64_t polls, int arrive, void* stream);

/* Message of the last failed call on this thread ("" if none). */
const char* mikv_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* MIKV_H_ */
