/*
 * replayssm.h - C ABI of the MI355X (gfx950) ReplaySSM decode library.
 *
 * One decode step of a Mamba2 selective state update for a batch of rows,
 * either the standard read+write update or the ReplaySSM output-only form
 * (a checkpoint S0 plus a per-slot ring of the last inputs, folded into the
 * state only on flush rows), plus the gated-delta-rule counterparts (GDN
 * with a scalar gate, KDA with a per-key-channel gate), GDN speculative
 * verify and commit from the ring, and host-side cursor helpers.
 *
 * Sources (page title, then section):
 *  - vLLM #48018 "[Kernel] ReplaySSM: cache SSM inputs for faster Mamba2
 *    standard decode": Motivation (state traffic; ring + periodic checkpoint;
 *    write-back once every L steps), Implementation items 1-3 (per-row
 *    is_flush branch; x/dt/B ring caches; per-row write_pos and is_flush
 *    from the metadata builder), key source snippet of mamba_mixer2.py (the
 *    argument lists of the replay op and of the baseline update).
 *  - sglang #28451 (GDN/KDA ReplaySSM decode): Motivation, Implementation
 *    items 1-3 (one ring decode kernel for the GDN and KDA gates, static
 *    cursor buffers, copy rules) and review notes (the KDA gate ring).
 *  - sglang #28695 "[GDN] Support ReplaySSM Ring Spec-Verify": memory-pool
 *    snippet (the GDN ring holds d [L,V], k [L,K], g [L] per slot) and
 *    Implementation items 2-4 (spec verify from the ring, exact fold).
 *  - vLLM #52506 "[Mamba] Add FlashInfer ReplaySSM backend": Implementation
 *    item 1 (ring cursors are reset when a slot is reused).
 *
 * Conventions shared by every entry point
 *  - Every pointer is a DEVICE pointer to memory the caller owns (except
 *    for the host-side metadata helpers at the end), allocated
 *    on the device that is current when the call is made.  The library never
 *    allocates, frees or synchronises, keeps no global mutable state, and is
 *    re-entrant: it validates the arguments, enqueues kernels on `stream`
 *    (0 = the null stream) and returns.
 *  - All tensors are dense, row-major (last index fastest), with no padding.
 *    Pointers accessed with 16-byte vector loads (marked [16B]) must be
 *    16-byte aligned.
 *  - Element types follow the *_dtype fields (RSSM_F32 = float, RSSM_BF16 =
 *    bfloat16 bit pattern).  A, D, dt_bias, dt_ring, the GDN/KDA d and g
 *    rings, g and beta are always float32.  bf16 stores round to nearest
 *    even from the fp32 value (or stochastically, where rssm_dims.rounding
 *    asks for it); all arithmetic is fp32.
 *  - Return value: RSSM_OK (0) or a negative RSSM_E* code (nothing is
 *    enqueued on an error other than RSSM_ELAUNCH).  No exception crosses
 *    the ABI.
 *  - Device-side metadata errors do not fail the call: the kernel ORs
 *    RSSM_ST_* bits into *status (if status != NULL) and handles the row
 *    safely; outputs of such rows are unspecified (y is NaN for bad slots).
 *  - Contract: slot indices within one call are distinct; the next_* cursor
 *    buffers do not alias write_pos / is_flush.  Calls that share a state
 *    pool or rings must be ordered by the caller (same stream or events).
 */
#ifndef REPLAYSSM_H
#define REPLAYSSM_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
enum { RSSM_F32 = 0, RSSM_BF16 = 1, RSSM_F8E4M3 = 2 /* rms_norm_forward's output only */ };

/* return codes */
enum {
  RSSM_OK = 0,
  RSSM_EINVAL = -1,      /* NULL required pointer, bad size, misalignment, aliasing */
  RSSM_EDTYPE = -2,      /* unsupported dtype combination */
  RSSM_ELAUNCH = -3,     /* the kernel launch reported an error */
  RSSM_ESHAPE = -4       /* headdim / dstate / ring length not supported */
};

/* device status bits (ORed into *status) */
enum {
  RSSM_ST_BAD_WRITE_POS = 1, /* write_pos outside [0, L): clamped, row flushed */
  RSSM_ST_RING_OVERFLOW = 2, /* write_pos == L-1 without is_flush: row flushed */
  RSSM_ST_BAD_SLOT = 4,      /* slot index outside [0, num_slots): row skipped */
  RSSM_ST_BAD_ROW = 8,       /* ring reset or row order: row index outside [0, batch) */
  RSSM_ST_BAD_SEQ = 16       /* cu_seqlens not 0 = first <= ... <= last = tokens: clamped */
};

/*
 * Rounding of the bf16 state write-back (vLLM #48018, review notes:
 * stochastic rounding was added for quantised models whose baseline relies
 * on it).  RSSM_ROUND_STOCHASTIC rounds each element of a written bf16
 * state tile up or down with probability given by the dropped 16 bits of its
 * fp32 value, using 16 random bits per element from Philox4x64-10 (Salmon
 * et al., SC 2011) with key (sr_seed, sr_offset) and counter
 * (tile * P*N/16 + e/16, 0, 0, 0), tile = slot * nheads + head, e = p*N + n:
 * element e takes bits 16*(e%4).. of output word (e%16)/4 and its bf16 bit
 * pattern is (fp32 bits + those 16 bits) >> 16 (Inf and NaN round to
 * nearest).  Applies to every state store of ssu_standard_decode and to the
 * flush write-back of replayssm_decode.  Other values: RSSM_EINVAL;
 * stochastic with an fp32 state: RSSM_EDTYPE.
 */
enum { RSSM_ROUND_NEAREST = 0, RSSM_ROUND_STOCHASTIC = 1 };

/*
 * Mamba2 dimensions.  Supported: headdim in {32, 64, 128}; dstate in {16,
 * 32, 64, 128, 256}; 1 <= ring_len <= 64 with the ring rows a workgroup
 * stages, about 4*ring_len*(P+N) bytes, within 64 KB (RSSM_ESHAPE otherwise);
 * ngroups divides nheads; state,
 * io and out dtypes each RSSM_F32 or RSSM_BF16.
 */
typedef struct rssm_dims {
  int32_t batch;       /* decode rows (0: return RSSM_OK, read nothing)     */
  int32_t nheads;      /* H                                                 */
  int32_t headdim;     /* P                                                 */
  int32_t dstate;      /* N                                                 */
  int32_t ngroups;     /* G: head h reads B/C group h / (H / G)             */
  int32_t ring_len;    /* L (ignored by ssu_standard_decode)                */
  int32_t num_slots;   /* first dimension of the state pool and the rings   */
  int32_t state_dtype; /* state pool                                        */
  int32_t io_dtype;    /* x, z, dt, B, C and the x / B rings                */
  int32_t out_dtype;   /* y                                                 */
  int32_t dt_softplus; /* nonzero: dt = softplus(dt + dt_bias)              */
  int32_t rounding;    /* state write-back: RSSM_ROUND_NEAREST or           */
                       /* RSSM_ROUND_STOCHASTIC (bf16 state only)           */
  uint64_t sr_seed;    /* stochastic rounding: Philox key word 0            */
  uint64_t sr_offset;  /* stochastic rounding: Philox key word 1; change it */
                       /* on every call so each write-back draws new bits   */
} rssm_dims;

/*
 * ssu_standard_decode - the standard selective state update (the baseline
 * the replay is measured against; vLLM #48018, Motivation and the baseline
 * call in the mamba_mixer2.py snippet).  For each row b, head h, with
 * s = slot_idx[b], g = h / (H/G):
 *     dt = softplus(dt[b,h] + dt_bias[h])      (no softplus if !dt_softplus)
 *     S  = exp(dt*A[h]) * state[s,h] + dt * outer(x[b,h,:], B[b,g,:])
 *     y[b,h,:] = S @ C[b,g,:] + D[h] * x[b,h,:];   y *= z * sigmoid(z)
 *     state[s,h] = S
 *
 *   state   [num_slots, H, P, N]  state_dtype   [16B] read and written
 *   slot_idx [batch] int32        pool slot of each row
 *   x, z    [batch, H, P]         io_dtype      [16B] z may be NULL (no gate)
 *   dt      [batch, H]            io_dtype      raw dt
 *   A       [H] float32; D [H] float32 or NULL; dt_bias [H] float32 or NULL
 *   B, C    [batch, G, N]         io_dtype      [16B]
 *   y       [batch, H, P]         out_dtype     written
 *   status  int32 or NULL         RSSM_ST_BAD_SLOT rows are skipped
 */
int ssu_standard_decode(const rssm_dims* dims, void* state,
                        const int32_t* slot_idx, const void* x, const void* dt,
                        const float* A, const void* B, const void* C,
                        const float* D, const void* z, const float* dt_bias,
                        void* y, int32_t* status, hipStream_t stream);

/*
 * replayssm_decode - one ReplaySSM output-only decode step (vLLM #48018,
 * Motivation and Implementation item 1).  Row b with s = slot_idx[b],
 * w = write_pos[b], f = is_flush[b] uses ring entries 0..w-1 of slot s and
 * the current step as entry w.  With T = sum_{j<=w} dt_j and
 * r_i = sum_{i<j<=w} dt_j (dt_j after softplus):
 *     cumdecay = exp(A[h]*T),  wt_i = dt_i * exp(A[h]*r_i)
 *     y = cumdecay*(S0 @ C) + sum_{i<=w} wt_i*(B_i . C)*x_i + D*x_w; gate
 *   f == 0: (x_w, dt_w, B_w) is written at ring position w; the state is not
 *           touched; next position w+1.
 *   f != 0: S_new = cumdecay*S0 + sum_{i<=w} wt_i*outer(x_i, B_i) is written
 *           to state[s,h]; y = S_new @ C + D*x_w (gated); next position 0.
 *   next_write_pos[b] = next position; next_is_flush[b] = (next == L-1).
 * A flush may be requested early (w < L-1).  write_pos == L-1 without
 * is_flush sets RSSM_ST_RING_OVERFLOW and the row is flushed.
 *
 *   state    [num_slots, H, P, N]  state_dtype  [16B] checkpoints S0
 *   x_ring   [num_slots, H, L, P]  io_dtype     [16B] stored x (bit copies)
 *   dt_ring  [num_slots, H, L]     float32      stored dt after softplus
 *   B_ring   [num_slots, G, L, N]  io_dtype     [16B] stored B (bit copies)
 *   slot_idx [batch] int32; write_pos [batch] int32; is_flush [batch] uint8
 *   next_write_pos [batch] int32 or NULL; next_is_flush [batch] uint8 or NULL
 *   x, dt, A, B, C, D, z, dt_bias, y: as for ssu_standard_decode
 *   status   int32 or NULL
 * Ring entries at positions >= write_pos are never read.  The order in
 * which rows are processed does not change any result; the kernel takes the
 * flush rows first, dealt evenly over the GPU's eight dies (XCDs) when the
 * batch has at most 512 rows and is_flush is 8-byte aligned, otherwise by
 * aligned groups of 64 rows.
 */
int replayssm_decode(const rssm_dims* dims, void* state, void* x_ring,
                     float* dt_ring, void* B_ring, const int32_t* slot_idx,
                     const int32_t* write_pos, const uint8_t* is_flush,
                     int32_t* next_write_pos, uint8_t* next_is_flush,
                     const void* x, const void* dt, const float* A,
                     const void* B, const void* C, const float* D,
                     const void* z, const float* dt_bias, void* y,
                     int32_t* status, hipStream_t stream);

/*
 * replayssm_decode_ordered - replayssm_decode with the batch rows handed in
 * flush-first order by the host (not on the pages: a scheduling hint for
 * this GPU).  row_order [batch] int32 (device pointer) must be a
 * permutation of 0..batch-1; replayssm_flush_first_order builds it from the
 * flush flags the host metadata path already has.  The results are those
 * of replayssm_decode for any permutation; the order only decides which
 * rows each of the GPU's eight dies (XCDs) takes: the positions of the list
 * are dealt to them in turn, so each takes an equal share of the flush rows,
 * first (replayssm_decode does the same dealing itself for batches of up
 * to 512 rows; a host list can also order the rows by slot).  An entry
 * outside [0, batch) sets
 * RSSM_ST_BAD_ROW and its position processes nothing: the row missing from
 * the list gets no y, no next cursors and no fold (its ring append, which
 * does not depend on the order, still happens); every other row is
 * processed as by replayssm_decode.  A list that repeats a row is a
 * contract violation: that row's y, cursors and (on a flush) checkpoint are
 * undefined, and another row is left unprocessed.  row_order == NULL:
 * RSSM_EINVAL.
 */
int replayssm_decode_ordered(const rssm_dims* dims, void* state, void* x_ring,
                             float* dt_ring, void* B_ring, const int32_t* slot_idx,
                             const int32_t* write_pos, const uint8_t* is_flush,
                             int32_t* next_write_pos, uint8_t* next_is_flush,
                             const void* x, const void* dt, const float* A, const void* B,
                             const void* C, const float* D, const void* z,
                             const float* dt_bias, void* y, const int32_t* row_order,
                             int32_t* status, hipStream_t stream);

/*
 * replayssm_ring_reset - rows whose slot just received a fresh checkpoint
 * restart with an empty ring (vLLM #52506, Implementation item 1; sglang
 * #28451, Implementation item 3): for r in rows[0..n_rows):
 *     write_pos[r] = 0;  is_flush[r] = (ring_len == 1)
 * Uses dims->batch (row bound) and dims->ring_len only.  The caller writes
 * the fresh state itself.  rows is a device array; rows outside [0, batch)
 * are skipped and set RSSM_ST_BAD_ROW in *status (if not NULL).
 */
int replayssm_ring_reset(const rssm_dims* dims, int32_t* write_pos,
                         uint8_t* is_flush, const int32_t* rows,
                         int32_t n_rows, int32_t* status, hipStream_t stream);

/*
 * GDN dimensions.  Supported: dk == dv == 128 (also 64); v_heads a multiple
 * of k_heads (value head hv reads key head hv / (v_heads / k_heads));
 * 1 <= ring_len <= 64 with the staged ring rows within 64 KB of LDS (about
 * ring_len*(2K + 4V) bytes for bf16 q/k/v, plus 4*ring_len*K for the KDA gate
 * rows; RSSM_ESHAPE otherwise); state_dtype RSSM_F32; io_dtype (q, k, v, k ring) and
 * out_dtype RSSM_F32 or RSSM_BF16.  scale <= 0 selects 1/sqrt(dk).
 */
typedef struct rssm_gdn_dims {
  int32_t batch;
  int32_t k_heads;
  int32_t v_heads;
  int32_t dk;          /* K */
  int32_t dv;          /* V */
  int32_t ring_len;
  int32_t num_slots;
  int32_t state_dtype;
  int32_t io_dtype;
  int32_t out_dtype;
  float scale;
} rssm_gdn_dims;

/*
 * gdn_standard_decode - the recurrent gated delta rule (sglang #28451,
 * Motivation: each step reads and writes the full [HV, V, K] state):
 *     S = g*S;  S += beta * outer(v - S@k, k);  o = scale * S@q
 *   state [num_slots, HV, V, K] float32 [16B]; slot_idx [batch] int32
 *   q, k [batch, HK, K] io_dtype [16B]; v [batch, HV, V] io_dtype [16B]
 *   g, beta [batch, HV] float32 (already activated); o [batch, HV, V] out_dtype
 */
int gdn_standard_decode(const rssm_gdn_dims* dims, void* state,
                        const int32_t* slot_idx, const void* q, const void* k,
                        const void* v, const float* g, const float* beta,
                        void* o, int32_t* status, hipStream_t stream);

/*
 * replayssm_gdn_decode - GDN ReplaySSM decode (sglang #28451, Implementation
 * item 1; ring contents per sglang #28695, memory-pool snippet).  With
 * Gamma = prod_{j<=w} g_j and gamma_i = prod_{i<j<=w} g_j:
 *     pred = Gamma*(S0@k_w) + sum_{i<w} gamma_i*d_i*(k_i . k_w)
 *     d_w  = beta_w*(v_w - pred)
 *     o    = scale*[Gamma*(S0@q) + sum_{i<=w} gamma_i*d_i*(k_i . q)]
 *   f == 0: (d_w, k_w, g_w) written at ring position w;
 *   f != 0: state = Gamma*S0 + sum_{i<=w} gamma_i*outer(d_i, k_i).
 *   d_ring [num_slots, HV, L, V] float32 [16B]; k_ring [num_slots, HK, L, K]
 *   io_dtype [16B] (bit copies of k); g_ring [num_slots, HV, L] float32.
 *   Cursor and status rules as for replayssm_decode.
 */
int replayssm_gdn_decode(const rssm_gdn_dims* dims, void* state, float* d_ring,
                         void* k_ring, float* g_ring, const int32_t* slot_idx,
                         const int32_t* write_pos, const uint8_t* is_flush,
                         int32_t* next_write_pos, uint8_t* next_is_flush,
                         const void* q, const void* k, const void* v,
                         const float* g, const float* beta, void* o,
                         int32_t* status, hipStream_t stream);

/*
 * KDA: the gated delta rule with a per-key-channel gate g in R^K (sglang
 * #28451: Implementation item 1 - one decode kernel serves the GDN scalar
 * gate and the KDA per-K gate; review notes - the KDA ring holds a gate row
 * per entry, g_cache [slots, HV, L, K]).  Same dims, layouts, cursor and
 * status rules as the GDN calls, except that g is [batch, HV, K] float32
 * [16B] and g_ring [num_slots, HV, L, K] float32 [16B].
 *
 * kda_standard_decode - the recurrence, per value head:
 *     S = S diag(g);  S += beta * outer(v - S@k, k);  o = scale * S@q
 *
 * replayssm_kda_decode - ReplaySSM decode.  With Gamma = prod_{j<=w} g_j and
 * gamma_i = prod_{i<j<=w} g_j taken per channel and kt_i = gamma_i * k_i:
 *     pred = S0@(Gamma*k_w) + sum_{i<w} d_i*(kt_i . k_w)
 *     d_w  = beta_w*(v_w - pred)
 *     o    = scale*[S0@(Gamma*q) + sum_{i<=w} d_i*(kt_i . q)]
 *   f == 0: (d_w, k_w, g_w) written at ring position w;
 *   f != 0: state = S0 diag(Gamma) + sum_{i<=w} outer(d_i, kt_i).
 */
int kda_standard_decode(const rssm_gdn_dims* dims, void* state,
                        const int32_t* slot_idx, const void* q, const void* k,
                        const void* v, const float* g, const float* beta,
                        void* o, int32_t* status, hipStream_t stream);

int replayssm_kda_decode(const rssm_gdn_dims* dims, void* state, float* d_ring,
                         void* k_ring, float* g_ring, const int32_t* slot_idx,
                         const int32_t* write_pos, const uint8_t* is_flush,
                         int32_t* next_write_pos, uint8_t* next_is_flush,
                         const void* q, const void* k, const void* v,
                         const float* g, const float* beta, void* o,
                         int32_t* status, hipStream_t stream);

/*
 * GDN speculative decoding from the ring (sglang #28695 "[GDN] Support
 * ReplaySSM Ring Spec-Verify": Implementation items 2-4 - a per-slot ring of
 * d, k, g plus the raw inputs v, k, beta; the verify rebuilds every draft's
 * output from the frozen checkpoint and the ring; the commit advances the
 * cursor and, on flush, replays the raw inputs in order through the
 * recurrent update ("exact fold"); linear draft chains only; the ring holds
 * at least twice the drafts).  Per slot the rings are those of
 * replayssm_gdn_decode plus v_ring [num_slots, HV, L, V] (io_dtype [16B]) and
 * beta_ring [num_slots, HV, L] float32.  1 <= n_draft (T) <= 8 and
 * 2*T <= ring_len <= 64 (RSSM_ESHAPE otherwise).
 *
 * replayssm_gdn_spec_verify - for row b at cursor w (entries 0..w-1
 * committed; w + T <= L, else RSSM_ST_RING_OVERFLOW and o = NaN for the
 * row), draft t is ring entry p = w + t and is formed exactly like a decode
 * step of replayssm_gdn_decode at position p (Gamma and gamma over entries
 * 0..p, pred, d_p, o).  Writes o [batch, T, HV, V] (out_dtype) and ring
 * entries w..w+T-1 (d, k, g, v, beta); the state and the cursor are not
 * modified.  q, k [batch, T, HK, K] and v [batch, T, HV, V] io_dtype [16B];
 * g, beta [batch, T, HV] float32.
 */
int replayssm_gdn_spec_verify(const rssm_gdn_dims* dims, int32_t n_draft,
                              const void* state, float* d_ring, void* k_ring,
                              float* g_ring, void* v_ring, float* beta_ring,
                              const int32_t* slot_idx, const int32_t* write_pos,
                              const void* q, const void* k, const void* v,
                              const float* g, const float* beta, void* o,
                              int32_t* status, hipStream_t stream);

/*
 * replayssm_gdn_spec_commit - keep accepted[b] (0..T) verified drafts:
 * w' = write_pos[b] + accepted[b].  If w' + T > ring_len (the next verify
 * would not fit) or force_flush[b] != 0 (force_flush may be NULL), the state
 * is rebuilt by the recurrence over entries 0..w'-1 from their raw inputs,
 *     S = g_i*S;  d = beta_i*(v_i - S@k_i);  S += outer(d, k_i),
 * stored, and w' = 0 (fp32 arithmetic; the decays are carried as one running
 * product and applied to the state at the end, or earlier when that product
 * leaves [2^-60, 2^60]: the same recurrence up to rounding).  Writes next_write_pos[b] = w' (must not alias
 * write_pos) and flushed[b] (may be NULL).  accepted outside [0, T] sets
 * RSSM_ST_RING_OVERFLOW and is clamped.
 */
int replayssm_gdn_spec_commit(const rssm_gdn_dims* dims, int32_t n_draft, void* state,
                              const void* k_ring, const float* g_ring,
                              const void* v_ring, const float* beta_ring,
                              const int32_t* slot_idx, const int32_t* write_pos,
                              const int32_t* accepted, const uint8_t* force_flush,
                              int32_t* next_write_pos, uint8_t* flushed,
                              int32_t* status, hipStream_t stream);

/*
 * Deferred-fold rounds (the same method with the fold moved into the next
 * verify, where it reuses that verify's read of the state tile: sglang
 * #28695 Implementation items 2-4 name a per-slot is_flush cursor next to
 * write_pos, and the exact fold runs on flush).  A round is
 * replayssm_gdn_spec_verify_flush then replayssm_gdn_spec_advance; between
 * rounds a row's logical state is its checkpoint folded with ring entries
 * 0..write_pos-1, and is_flush marks rows whose next verify folds first.
 * Cursors start at write_pos = 0, is_flush = 0.  A row keeps to one kind of
 * round (a pending fold is not visible to replayssm_gdn_spec_verify).  To
 * empty a row's ring at once (before copying its slot, say),
 * replayssm_gdn_spec_commit with accepted = 0 and force_flush set folds its
 * entries 0..write_pos-1 and returns write_pos 0; then clear its is_flush.
 * A row the verify refused (status bit) is left unspecified by the advance,
 * which cannot tell that no fold took place.
 *
 * replayssm_gdn_spec_verify_flush - rows with is_flush[b] != 0 (is_flush
 * [batch] uint8, required) first fold ring entries 0..write_pos[b]-1 into
 * the state exactly as replayssm_gdn_spec_commit does (0 <= write_pos[b] <=
 * L, else RSSM_ST_RING_OVERFLOW), store it, then verify their drafts at ring
 * entries 0..T-1 (w = 0); other rows verify at w = write_pos[b] as in
 * replayssm_gdn_spec_verify (w + T <= L).  Writes o and the drafts' d rows
 * at ring entries w..w+T-1 only: their v, k, g and beta rows are written by
 * replayssm_gdn_spec_advance for the drafts kept.  Arguments otherwise as
 * replayssm_gdn_spec_verify, with the state written.  A folding row stages
 * the k and v rows of the whole ring next to the verify's own rows:
 * RSSM_ESHAPE when they do not fit one workgroup's 64 KB of LDS (at K = V =
 * 128 the longest rings are 46 entries for T <= 4 and 42 for T = 8 with bf16
 * inputs, 27 and 24 with fp32 ones).
 *
 * replayssm_gdn_spec_advance - after the verify, with accepted[b] (0..T)
 * drafts kept: w = is_flush[b] ? 0 : write_pos[b]; w' = w + accepted[b];
 * next_write_pos[b] = w'; next_is_flush[b] = (w' + T > L) or
 * force_flush[b] (may be NULL).  The kept drafts' rows go from this round's
 * verify inputs (k [batch, T, HK, K], v [batch, T, HV, V] io_dtype [16B];
 * g, beta [batch, T, HV] float32) to ring entries w..w'-1 of k_ring (per key
 * head), v_ring, g_ring and beta_ring.  The next_* buffers must not alias
 * write_pos / is_flush.  dims as for the verify.  accepted outside [0, T]
 * sets RSSM_ST_RING_OVERFLOW and is clamped; a slot out of range sets
 * RSSM_ST_BAD_SLOT and its row is neither marked nor written.
 */
int replayssm_gdn_spec_verify_flush(const rssm_gdn_dims* dims, int32_t n_draft,
                                    float* state, float* d_ring, void* k_ring,
                                    float* g_ring, void* v_ring, float* beta_ring,
                                    const int32_t* slot_idx, const int32_t* write_pos,
                                    const uint8_t* is_flush, const void* q,
                                    const void* k, const void* v, const float* g,
                                    const float* beta, void* o, int32_t* status,
                                    hipStream_t stream);

int replayssm_gdn_spec_advance(const rssm_gdn_dims* dims, int32_t n_draft, void* k_ring,
                               float* g_ring, void* v_ring, float* beta_ring,
                               const void* k, const void* v, const float* g,
                               const float* beta, const int32_t* slot_idx,
                               const int32_t* write_pos, const uint8_t* is_flush,
                               const int32_t* accepted, const uint8_t* force_flush,
                               int32_t* next_write_pos, uint8_t* next_is_flush,
                               int32_t* status, hipStream_t stream);

/*
 * Host-side metadata (HOST pointers; plain CPU code, nothing is enqueued).
 *
 * replayssm_build_metadata - per-row cursors of one decode step from token
 * positions (vLLM #48018, Implementation item 3: write_pos and is_flush come
 * from a per-request decode base; align-mode re-anchoring; review notes on
 * the flush boundary, one-token prefills and preemption).  For row r:
 *     pos[r]          index of the token decoded in this step (tokens before it)
 *     decode_base[r]  number of tokens folded into the row's checkpoint S0;
 *                     set it to the prefill length for a fresh request, and
 *                     to the re-prefilled length when a preempted request
 *                     resumes (re-anchoring)
 *     w = pos - decode_base, which must lie in [0, ring_len)
 *     f = (w == ring_len-1) || force_flush[r] ||
 *         (align_block > 0 && (pos+1) % align_block == 0)
 * Writes write_pos[r] = w, is_flush[r] = f, and decode_base[r] = pos+1 when
 * f (the checkpoint will hold this token once the step has run).  With
 * align_block > 0 every checkpoint lands on a multiple of align_block or on
 * a ring-full boundary, so a prefix cache can snapshot block-aligned states.
 * force_flush may be NULL.  Returns RSSM_EINVAL, writing nothing, if any row
 * is out of range (w < 0, w >= ring_len, negative positions) or on bad
 * arguments.  For rows advancing one token per step this reproduces the
 * device-side cursor advance of replayssm_decode.
 */
int replayssm_build_metadata(int32_t n_rows, int32_t ring_len, int32_t align_block,
                             const int64_t* pos, int64_t* decode_base,
                             const uint8_t* force_flush, int32_t* write_pos,
                             uint8_t* is_flush);

/*
 * replayssm_check_copy_sources - the copy rule for slots (sglang #28451 and
 * #28695: a slot's state may be copied only when its ring is empty, else
 * the ring entries not yet folded would be lost).  src_write_pos [n] are the
 * current write positions of the source rows (HOST pointer).  RSSM_OK if
 * every one is 0, RSSM_EINVAL otherwise.  After copying a state into a new
 * slot, reset that row's cursors with replayssm_ring_reset.
 */
int replayssm_check_copy_sources(int32_t n, const int32_t* src_write_pos);

/*
 * replayssm_flush_first_order - the row order for replayssm_decode_ordered:
 * the rows with is_flush[r] != 0 in increasing r, then the others in
 * increasing r.  is_flush [n_rows] and row_order [n_rows] are HOST pointers.
 * RSSM_OK, or RSSM_EINVAL for n_rows < 0 or a NULL pointer with n_rows > 0.
 */
int replayssm_flush_first_order(int32_t n_rows, const uint8_t* is_flush, int32_t* row_order);

/*
 * ---------------------------------------------------------------------------
 * Sequence operators of the same Mamba2 layer: prefill and training.  They
 * fill the state pools the decode entry points read, and give the gradients.
 *
 * Conventions beside the ones above
 *  - Sequences are packed one after another along the token axis:
 *    cu_seqlens [seqs + 1] int32, cu_seqlens[0] = 0, non-decreasing, last =
 *    tokens.  Sequences may be empty.  NULL: one sequence of all tokens
 *    (seqs = 1).  A table that breaks the rule sets RSSM_ST_BAD_SEQ and is
 *    clamped; the results are then unspecified.
 *  - Token strides (*_stride, in elements between two tokens' rows) let an
 *    operand be a slice of a wider row, such as a projection's output; 0
 *    means dense.  Rows themselves are contiguous.  Outputs are dense.
 *  - A workspace is device memory of at least the size its *_workspace
 *    function returns, 16-byte aligned, written before it is read: no
 *    content is kept between calls, and calls on different streams need
 *    workspaces of their own.
 *  - Sums over tokens, rows and heads are added in a fixed order: the same
 *    call gives the same bits.
 *  - A call whose launches would hold 2^32 threads or more is refused
 *    (RSSM_ESHAPE): a norm forward from 2^22 rows on (above 8192 elements; 2^26
 *    up to 1024), a convolution's decode step from 2^28 rows of 512 channels, a
 *    scan from 2^34 / (nheads*headdim*dstate) sequences on (backward 2^32 / that).
 *  - Sequences of one call that write to a pool (final_state,
 *    dinitial_state by slot) take slots of their own.
 *  - An output may share memory with an input only where its description
 *    says so: workgroups read rows that others have work to do on.
 */
enum { RSSM_ACT_NONE = 0, RSSM_ACT_SILU = 1 };

/*
 * Causal convolution.  Supported: width 2, 3, 4; 1 to 2^24 channels;
 * pointers aligned to their element type.
 */
typedef struct rssm_conv_dims {
  int32_t tokens;     /* T (decode: batch rows)                             */
  int32_t seqs;       /* sequences (ignored by the decode step)             */
  int32_t channels;   /* C                                                  */
  int32_t width;      /* W                                                  */
  int32_t num_slots;  /* first dimension of the conv states                 */
  int32_t io_dtype;   /* x, y, conv states and their gradients              */
  int32_t activation; /* RSSM_ACT_*                                         */
  int32_t reserved;
  int64_t x_stride;
  int64_t dy_stride;
} rssm_conv_dims;

/*
 * causal_conv_forward - for each sequence i and channel c, with row p < 0
 * taken from the W-1 rows before the sequence (row -1 the latest):
 *     v_p = bias[c] + sum_{j<W} weight[c,j] * x[p - (W-1) + j, c]
 *     y[p,c] = v_p * sigmoid(v_p)       (v_p with RSSM_ACT_NONE)
 *   x [tokens, C] io_dtype; weight [C, W] float32; bias [C] float32 or NULL
 *   initial_state [num_slots, W-1, C] io_dtype or NULL (zeros), sequence i
 *     reads slot slot_idx[i] (NULL: i) where has_initial[i] (NULL: all)
 *   final_state [num_slots, W-1, C] or NULL: the last W-1 rows, same slots;
 *     may be initial_state itself
 *   y [tokens, C] io_dtype; sharing memory with x's rows is refused
 */
int causal_conv_forward(const rssm_conv_dims* dims, const void* x, const float* weight,
                        const float* bias, const int32_t* cu_seqlens,
                        const void* initial_state, const uint8_t* has_initial,
                        const int32_t* slot_idx, void* final_state, void* y,
                        int32_t* status, hipStream_t stream);

/*
 * causal_conv_backward - gradients of causal_conv_forward's y:
 *   dx [tokens, C] io_dtype (sharing memory with x's or dy's rows is
 *   refused); dweight [C, W], dbias [C] (or NULL) float32;
 *   dinitial_state [num_slots, W-1, C] io_dtype or NULL: written for every
 *   sequence's slot, zero where has_initial[i] is 0.
 */
size_t causal_conv_backward_workspace(const rssm_conv_dims* dims);
int causal_conv_backward(const rssm_conv_dims* dims, const void* dy, const void* x,
                         const float* weight, const float* bias,
                         const int32_t* cu_seqlens, const void* initial_state,
                         const uint8_t* has_initial, const int32_t* slot_idx,
                         void* dx, float* dweight, float* dbias,
                         void* dinitial_state, void* workspace,
                         size_t workspace_bytes, int32_t* status, hipStream_t stream);

/*
 * causal_conv_decode - one token of dims->tokens rows: row b's window is the
 * W-1 rows of slot slot_idx[b] (NULL: b) and x[b]; new_state's slot gets the
 * window's last W-1 rows (new_state may be conv_state).  A slot out of range
 * sets RSSM_ST_BAD_SLOT, its y is NaN and no state is written.
 */
int causal_conv_decode(const rssm_conv_dims* dims, const void* x,
                       const void* conv_state, const float* weight,
                       const float* bias, const int32_t* slot_idx,
                       void* new_state, void* y, int32_t* status, hipStream_t stream);

/*
 * Root-mean-square norm.  dim <= 32768 (counted with each group rounded up to
 * a multiple of 8); group_size divides dim; pointers aligned to their
 * element type.
 */
typedef struct rssm_norm_dims {
  int32_t rows;
  int32_t dim;
  int32_t group_size;     /* elements that share one mean square            */
  int32_t io_dtype;       /* x, z, and out unless it is 8-bit               */
  int32_t residual_dtype; /* RSSM_F32 or io_dtype                           */
  int32_t out_dtype;      /* io_dtype or RSSM_F8E4M3                        */
  int32_t scale_block;    /* 8-bit: 0 one scale a row, 128 one a block of   */
                          /* 128 elements (group_size a multiple of 128)    */
  float eps;
  int64_t x_stride;
  int64_t z_stride;
  int64_t dy_stride;
} rssm_norm_dims;

/*
 * rms_norm_forward -
 *     h = x + residual (residual_out = h in residual_dtype; the norm reads h
 *         as stored; residual NULL: h = x)
 *     u = h * z * sigmoid(z)    (z NULL: u = h)
 *     y = u * rsqrt(mean over the group of u^2 + eps) * weight
 *   out = y in io_dtype, or the e4m3 values of y / scale with scale =
 *   max|y| / 448 over the row or block (1 where that is 0 or NaN, whose e4m3
 *   values are NaN, and at least the smallest normal number): scale [rows] or [rows, dim/128] float32.
 *   residual_out may be residual.
 */
int rms_norm_forward(const rssm_norm_dims* dims, const void* x, const float* weight,
                     const void* z, const void* residual, void* residual_out,
                     void* out, float* scale, hipStream_t stream);

/*
 * rms_norm_backward - gradients of y (without residual): dx, dz (z given)
 * [rows, dim] io_dtype, dweight [dim] float32.
 */
size_t rms_norm_backward_workspace(const rssm_norm_dims* dims);
int rms_norm_backward(const rssm_norm_dims* dims, const void* dy, const void* x,
                      const float* weight, const void* z, void* dx,
                      float* dweight, void* dz, void* workspace,
                      size_t workspace_bytes, hipStream_t stream);

/*
 * Selective scan over whole sequences: the recurrence of ssu_standard_decode
 * applied to every token.  Supported: headdim in {32, 64, 128}, dstate in
 * {16, 32, 64, 128, 256}, ngroups divides nheads.  x, z, B, C and dy:
 * 16-byte aligned, with token strides that are multiples of 16 bytes.
 */
typedef struct rssm_scan_dims {
  int32_t tokens;
  int32_t seqs;
  int32_t nheads;
  int32_t headdim;
  int32_t dstate;
  int32_t ngroups;
  int32_t num_slots;   /* first dimension of initial_state / final_state    */
  int32_t io_dtype;    /* x, dt, B, C, z, y, dy and the gradients of x, dt, */
                       /* B, C                                              */
  int32_t state_dtype; /* initial_state, final_state                        */
  int32_t dt_softplus; /* nonzero: dt = softplus(dt + dt_bias)              */
  int64_t x_stride;    /* elements between two tokens of x [T, H, P]        */
  int64_t dt_stride;   /* dt [T, H]                                         */
  int64_t B_stride;    /* B [T, G, N]                                       */
  int64_t C_stride;
  int64_t z_stride;
  int64_t dy_stride;
} rssm_scan_dims;

/*
 * ssu_scan_forward - for every sequence i (slot s = slot_idx[i], NULL: i) and
 * head h, from S = initial_state[s, h] (zeros where initial_state is NULL or
 * has_initial[i] is 0), token by token
 *     S = exp(dt*A[h]) * S + dt * outer(x, B);  y = S @ C + D[h] * x
 *     y *= z * sigmoid(z)    (z not NULL)
 * and final_state[s, h] = S (final_state may be initial_state, or NULL).
 * y [tokens, H, P] io_dtype.  A slot out of range sets RSSM_ST_BAD_SLOT: its
 * sequence starts from zeros and stores no state.  Tokens are worked on in
 * chunks of 64 of one sequence: a NaN or infinity in a token's x may also show
 * in the up to 63 tokens of its sequence and chunk before it, and never in
 * another sequence.  Calls of up to 128 tokens need no workspace.
 */
size_t ssu_scan_forward_workspace(const rssm_scan_dims* dims);
int ssu_scan_forward(const rssm_scan_dims* dims, const void* x, const void* dt, const float* A,
                     const void* B, const void* C, const float* D, const void* z,
                     const float* dt_bias, const int32_t* cu_seqlens,
                     const void* initial_state, const uint8_t* has_initial,
                     const int32_t* slot_idx, void* final_state, void* y,
                     void* workspace, size_t workspace_bytes, int32_t* status,
                     hipStream_t stream);

/*
 * ssu_scan_backward - gradients of ssu_scan_forward without z, given dy and
 * dfinal_state [seqs, H, P, N] float32 (the gradient of each sequence's last
 * state, by sequence and not by slot; NULL: zeros):
 *   dx [T, H, P], ddt [T, H], dB, dC [T, G, N] io_dtype;
 *   dA, dD, ddt_bias [H] float32 (dD and ddt_bias may be NULL);
 *   dinitial_state [seqs, H, P, N] float32 by sequence, zeros where
 *   has_initial[i] is 0 (NULL: not computed).
 */
size_t ssu_scan_backward_workspace(const rssm_scan_dims* dims);
int ssu_scan_backward(const rssm_scan_dims* dims, const void* dy, const void* x, const void* dt,
                      const float* A, const void* B, const void* C, const float* D,
                      const float* dt_bias, const int32_t* cu_seqlens,
                      const void* initial_state, const uint8_t* has_initial,
                      const int32_t* slot_idx, const float* dfinal_state, void* dx,
                      void* ddt, void* dB, void* dC, float* dA, float* dD,
                      float* ddt_bias, float* dinitial_state, void* workspace,
                      size_t workspace_bytes, int32_t* status, hipStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Operators of linear-attention layers: linear attention with a decay for each
 * head, the gated delta rule over whole sequences (it fills the pools that the
 * GDN decode entry points read), and rotary positions.  The conventions of the
 * sequence operators hold (packed sequences, token strides, workspaces).
 *
 * Decays are given as natural logarithms, log g <= 0 as a rule; -infinity
 * forgets the state.  Value head hv reads key head hv / (v_heads / k_heads).
 * States are float32 [num_slots, v_heads, dv, dk], as in the GDN pools.
 */
enum { RSSM_DECAY_NONE = 0, RSSM_DECAY_HEAD = 1, RSSM_DECAY_TOKEN = 2 };

typedef struct rssm_mixer_dims {
  int32_t tokens;     /* T (decode: batch rows)                             */
  int32_t seqs;       /* sequences (ignored by the decode step)             */
  int32_t k_heads;
  int32_t v_heads;
  int32_t dk;         /* K: 64 or 128                                       */
  int32_t dv;         /* V: 64 or 128 (the gated delta rule: dv == dk)      */
  int32_t num_slots;  /* first dimension of the state pools                 */
  int32_t io_dtype;   /* q, k, v, o and their gradients                     */
  int32_t decay;      /* RSSM_DECAY_*: no decay, log g [v_heads], or        */
                      /* [tokens, v_heads] (the gated delta rule: the last) */
  float scale;        /* of the outputs; <= 0 selects 1/sqrt(dk)            */
  int64_t q_stride;   /* elements between two tokens of q, k [T, HK, K]     */
  int64_t k_stride;
  int64_t v_stride;   /* v, do [T, HV, V]                                   */
  int64_t do_stride;
} rssm_mixer_dims;

/*
 * linear_attention_forward - for every sequence i (slot s = slot_idx[i], NULL:
 * i) and value head, from S = initial_state[s] (zeros where initial_state is
 * NULL or has_initial[i] is 0), token by token
 *     S = g*S + outer(v, k);  o = scale * S @ q
 * and final_state[s] = S (may be initial_state, or NULL).  q, k, v, o [16B]
 * with token strides that are multiples of 16 bytes; o [tokens, HV, V] dense.
 * Results that share memory with rows of q, k or v (backward: or do), and pools
 * that share memory with each other, are refused; o may be v itself where v is
 * dense, and the pools may be one.
 * A slot out of range sets RSSM_ST_BAD_SLOT: its sequence starts from zeros and
 * stores no state.  Tokens are worked on in chunks of 64 of one sequence: a NaN
 * or infinity in a token's inputs may also show in the up to 63 tokens of its
 * sequence and chunk before it, and never in another sequence.
 */
size_t linear_attention_forward_workspace(const rssm_mixer_dims* dims);
int linear_attention_forward(const rssm_mixer_dims* dims, const void* q, const void* k,
                             const void* v, const float* log_decay,
                             const int32_t* cu_seqlens, const float* initial_state,
                             const uint8_t* has_initial, const int32_t* slot_idx,
                             float* final_state, void* o, void* workspace,
                             size_t workspace_bytes, int32_t* status,
                             hipStream_t stream);

/*
 * linear_attention_backward - gradients of linear_attention_forward, given do
 * [tokens, HV, V] and dfinal_state [seqs, HV, V, K] float32 (the gradient of
 * each sequence's last state, by sequence and not by slot; NULL: zeros):
 *   dq, dk [T, HK, K], dv [T, HV, V] io_dtype; dlog_decay float32 in the shape
 *   of log_decay (NULL without one); dinitial_state [seqs, HV, V, K] float32 by
 *   sequence, zeros where has_initial[i] is 0 (NULL: not computed).
 * Workspaces, for each value head.  A chunk is up to 64 tokens of one sequence: at
 * most tokens / 64 + seqs of them.  Backward, each: 8 dk dv bytes, and for the
 * delta rule 512 dv and 36 KB (fp32: 24 KB) more.  Delta rule forward, each: 18 KB
 * (fp32: 12 KB).  Calls of more than 512 tokens, for segments of long sequences, at
 * most 4 tokens / 512 of them: 4 dk dv bytes forward and 8 dk dv backward each, and
 * for the delta rule 6 dk dk forward and 12 dk dk backward (fp32: 4 and 8).
 */
size_t linear_attention_backward_workspace(const rssm_mixer_dims* dims);
int linear_attention_backward(const rssm_mixer_dims* dims, const void* dout, const void* q,
                              const void* k, const void* v, const float* log_decay,
                              const int32_t* cu_seqlens, const float* initial_state,
                              const uint8_t* has_initial, const int32_t* slot_idx,
                              const float* dfinal_state, void* dq, void* dk, void* dv,
                              float* dlog_decay, float* dinitial_state, void* workspace,
                              size_t workspace_bytes, int32_t* status, hipStream_t stream);

/*
 * linear_attention_decode - one token of dims->tokens rows: row b's state is
 * slot slot_idx[b] (NULL: b) of state; the moved-on state goes to the same slot
 * of new_state (may be state).  A slot out of range sets RSSM_ST_BAD_SLOT, its o
 * is NaN and no state is written.
 */
int linear_attention_decode(const rssm_mixer_dims* dims, const float* state,
                            const int32_t* slot_idx, const void* q, const void* k,
                            const void* v, const float* log_decay, float* new_state,
                            void* o, int32_t* status, hipStream_t stream);

/*
 * gdn_scan_forward - the recurrence of gdn_standard_decode applied to every
 * token of packed sequences, with g = exp(log_g):
 *     S = g*S;  S += beta * outer(v - S@k, k);  o = scale * S@q
 * log_g, beta [tokens, HV] float32; the rest as linear_attention_forward.  With
 * beta |k|^2 from 0 to 2 a token enlarges nothing, and neither do the kernels
 * enlarge a rounding; beyond that the recurrence itself grows.
 */
size_t gdn_scan_forward_workspace(const rssm_mixer_dims* dims);
int gdn_scan_forward(const rssm_mixer_dims* dims, const void* q, const void* k,
                     const void* v, const float* log_g, const float* beta,
                     const int32_t* cu_seqlens, const float* initial_state,
                     const uint8_t* has_initial, const int32_t* slot_idx,
                     float* final_state, void* o, void* workspace,
                     size_t workspace_bytes, int32_t* status, hipStream_t stream);

/*
 * gdn_scan_backward - its gradients: dq, dk, dv io_dtype; dlog_g, dbeta
 * [tokens, HV] float32; dfinal_state and dinitial_state as
 * linear_attention_backward.
 */
size_t gdn_scan_backward_workspace(const rssm_mixer_dims* dims);
int gdn_scan_backward(const rssm_mixer_dims* dims, const void* dout, const void* q,
                      const void* k, const void* v, const float* log_g,
                      const float* beta, const int32_t* cu_seqlens,
                      const float* initial_state, const uint8_t* has_initial,
                      const int32_t* slot_idx, const float* dfinal_state, void* dq,
                      void* dk, void* dv, float* dlog_g, float* dbeta,
                      float* dinitial_state, void* workspace, size_t workspace_bytes,
                      int32_t* status, hipStream_t stream);

/*
 * Rotary positions: the first rotary_dim elements of every head turn in pairs,
 * pair i by the angle position * freqs[i]; the others are copied.
 */
typedef struct rssm_rotary_dims {
  int32_t tokens;
  int32_t heads;        /* up to 2^30                                       */
  int32_t dim;          /* elements of a head, up to 1024                   */
  int32_t rotary_dim;   /* even, 2 to dim                                   */
  int32_t io_dtype;
  int32_t interleaved;  /* nonzero: pair i is elements (2i, 2i + 1);        */
                        /* 0: (i, i + rotary_dim / 2)                       */
  int32_t pos_int64;    /* nonzero: positions are int64, else int32         */
  float amplitude;      /* factor of the turned elements                    */
  int64_t x_stride;     /* elements between two tokens (0: dense)           */
  int64_t y_stride;
} rssm_rotary_dims;

/*
 * rotary_forward - x [tokens, heads, dim], positions [tokens], freqs
 * [rotary_dim / 2] float32 -> y, which may be x itself (with the same stride)
 * and otherwise shares no memory with it.  For a pair (a, b) and its angle t,
 *     (a', b') = amplitude * (a cos t - b sin t, a sin t + b cos t).
 * The angle and its sine and cosine are formed in 64 bits.
 *
 * rotary_backward - the gradient dx of x, given y's gradient dy: the turn back.
 */
int rotary_forward(const rssm_rotary_dims* dims, const void* x, const void* positions,
                   const float* freqs, void* y, hipStream_t stream);
int rotary_backward(const rssm_rotary_dims* dims, const void* dy, const void* positions,
                    const float* freqs, void* dx, hipStream_t stream);

/* Human-readable text of a return code (static storage). */
const char* replayssm_strerror(int code);

/* Library ABI version (major * 100 + minor). */
int replayssm_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* REPLAYSSM_H */
