/*
 * ssm_linattn.h -- linear attention with a decay for each head: the layer's
 * recurrence with a matrix state, h_t in R^{dk x dv} per head, instead of the
 * diagonal one of ssm_adjoint.h.  Built into the same library; the
 * conventions of ssm_adjoint.h hold (device pointers owned by the caller,
 * 16-byte aligned; nothing allocated or synchronised; complete validation
 * before anything is enqueued; outputs overwritten, except the state of
 * ssm_linattn_step; bitwise repeatable results; SSM_* status codes).
 *
 * Per head h (key head h / (Hv / Hk)), token t of a sequence:
 *   h_t = e^{g_t} h_{t-1} + k_t v_t^T,   y_t = scale q_t^T h_t,   h_{-1} = h0
 * with g_t = log_decay[t][h], or log_decay[h] for every token when
 * dims.decay_tokens is 0.  Loss seen by the gradient:
 *   L = sum_t <dy_t, y_t> + <dhT, h_T>.
 *
 * Packed sequences: the token arrays hold dims.T rows.  With seq_start NULL
 * they are S sequences of T / S tokens each (T a multiple of S).  Otherwise
 * seq_start is a device array of S + 1 offsets, 0 <= seq_start[0] <= ... <=
 * seq_start[S] <= T: sequence s is rows seq_start[s] .. seq_start[s + 1] - 1,
 * possibly none.  Rows outside every sequence are neither read nor written.
 * The offsets are read on the device; offsets that break this rule give
 * undefined results but no access outside the arrays.  They may change
 * between replays of a captured graph.
 *
 * Layouts (row-major, elements): q, k [T][Hk][dk], v, y, dy [T][Hv][dv] in the
 * io dtype, dq, dk, dv likewise; a row of q, k, v, y, dy starts ld elements
 * after the one before it (heads * d <= ld <= 2^22, ld a multiple of 16 bytes).
 * log_decay and its gradient [T][Hv] or [Hv], states [S][Hv][dk][dv], float32.
 *
 * Supported: dk and dv multiples of 8 up to 128, Hk divides Hv, Hv <= 4096,
 * S <= 65535, S * Hv <= 2^22, T < 2^31.  log_decay may be -inf (a reset) and positive; a NaN or an
 * infinity in one token's q, k, v or dy may reach every output of its
 * sequence and head.
 */
#ifndef SSM_LINATTN_H
#define SSM_LINATTN_H

#include "ssm_adjoint.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int64_t T;            /* rows of the token arrays */
  int32_t S;            /* sequences */
  int32_t Hk, Hv;       /* heads of q and k; heads of v, y, the decay and the state */
  int32_t dk, dv;       /* channels of a q / k head and of a v / y head */
  int32_t io;           /* ssm_dtype of q, k, v, y, dy, dq, dk, dv */
  int32_t decay_tokens; /* 1: log_decay [T][Hv]; 0: [Hv] */
  float scale;          /* finite */
} ssm_linattn_dims;

typedef struct {
  const void *q, *k, *v;    /* rows ldq, ldk, ldv elements apart */
  int64_t ldq, ldk, ldv;
  const float *log_decay;
  const int32_t *seq_start; /* [S + 1] or NULL */
  const float *h0;          /* [S][Hv][dk][dv] or NULL (zero) */
} ssm_linattn_in;

/* Gradient outputs; NULL = not computed, at least one set.  Contiguous
 * (rows of dq and dk Hk * dk elements apart, of dv Hv * dv). */
typedef struct {
  void *dq, *dk, *dv;
  float *dlog_decay;  /* shape of log_decay; the sum over all tokens when that is [Hv] */
  float *dh0;         /* [S][Hv][dk][dv] */
} ssm_linattn_grads;

/* Workspace bytes of ssm_linattn_forward (grads NULL) or of
 * ssm_linattn_grad for the outputs set in grads (only which pointers are
 * NULL counts).  A forward call may need none: *bytes is then 0.  Returns the
 * status of the dims. */
ssm_status ssm_linattn_workspace_bytes(const ssm_linattn_dims *dims, const ssm_linattn_grads *grads, size_t *bytes);

/* Forward pass over packed sequences: y (rows ldy elements apart; must not
 * overlap an input) and, unless hT is NULL, the state after the last token of
 * each sequence (h0 for an empty one).  hT may be h0. */
ssm_status ssm_linattn_forward(const ssm_linattn_dims *dims, const ssm_linattn_in *in, void *y, int64_t ldy, float *hT,
                               void *ws, size_t ws_bytes, void *stream);

/* Gradient of L, from the forward pass's inputs (no saved state: the states
 * are recomputed).  dhT NULL: no final-state term.  No output may overlap an
 * input or another output. */
ssm_status ssm_linattn_grad(const ssm_linattn_dims *dims, const ssm_linattn_in *in, const void *dy, int64_t lddy,
                            const float *dhT, const ssm_linattn_grads *grads, void *ws, size_t ws_bytes, void *stream);

/* One token for each of dims.T sequences (S is not read): row t is the next
 * token of the sequence whose state is state[t] ([T][Hv][dk][dv]), which is
 * updated in place.  in->seq_start and in->h0 must be NULL; y must not overlap
 * an input.  No workspace. */
ssm_status ssm_linattn_step(const ssm_linattn_dims *dims, const ssm_linattn_in *in, float *state, void *y, int64_t ldy,
                            void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_LINATTN_H */
