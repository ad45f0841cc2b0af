/*
 * ssm_train.h -- what a training step does around the layers: the residual
 * update with the RMS norm of the next layer's input, its gradient, and the
 * global norm and clipping of the gradients.  Built into the same library;
 * the conventions of ssm_adjoint.h hold (device pointers owned by the caller,
 * 16-byte aligned; nothing allocated or synchronised; complete validation
 * before anything is enqueued; outputs overwritten; bitwise repeatable
 * results; SSM_* status codes).  An output overlaps no input and no other
 * output except where it says so below.
 */
#ifndef SSM_TRAIN_H
#define SSM_TRAIN_H

#include "ssm_adjoint.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Residual update and RMS norm, the step ssm_stack_grad takes before a
 * normalising layer, per row t of P channels (1 <= P <= 16384):
 *   r_out = r + y,  rinv_t = 1 / sqrt(mean_p r_out[t][p]^2 + eps),
 *   x = io(norm_scale r_out rinv_t)
 *   r [T][P] float32; y [T][P] io or NULL (zero); norm_scale [P] float32
 *   r_out [T][P] float32, may be r; NULL only when y is NULL (r is r_out then)
 *   x [T][P] io; rinv [T] float32 or NULL
 * eps > 0.
 */
ssm_status ssm_add_norm(int64_t T, int64_t P, int32_t io, const float *r, const void *y, const float *norm_scale,
                        float eps, float *r_out, void *x, float *rinv, void *stream);

/* Workspace bytes of ssm_add_norm_grad; 0 if the sizes are invalid. */
size_t ssm_add_norm_grad_workspace_bytes(int64_t T, int64_t P);

/*
 * Its gradient, from r_out and rinv of ssm_add_norm.  dx [T][P] io is the
 * cotangent of x, dr_out [T][P] float32 that of r_out from elsewhere (NULL:
 * none).  dr [T][P] float32 is the cotangent of r and of y; it may be dr_out.
 * dnorm_scale [P] float32 or NULL.
 */
ssm_status ssm_add_norm_grad(int64_t T, int64_t P, int32_t io, const float *r_out, const float *rinv,
                             const float *norm_scale, const void *dx, const float *dr_out, float *dr,
                             float *dnorm_scale, void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes of ssm_clip_grads for these element counts; 0 if count or an n is invalid. */
size_t ssm_clip_grads_workspace_bytes(int32_t count, const int64_t *n);

/*
 * Global norm of `count` gradient tensors (1 .. 65536; host arrays of device
 * pointers and of element counts n >= 0, all of dtype io) and the tensors
 * scaled to it:
 *   norm = sqrt(sum of all squares), out_i = io(in_i min(1, max_norm / norm)).
 * norm: one float32 on the device.  out may be NULL (the norm alone); out[i]
 * may be in[i], and must not otherwise overlap any tensor.  The sum is formed
 * in float64.  If it is not finite, out_i = in_i: the caller sees it in norm.
 * max_norm > 0 (infinity allowed).
 */
ssm_status ssm_clip_grads(int32_t count, const void *const *in, void *const *out, const int64_t *n, int32_t io,
                          float max_norm, float *norm, void *ws, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SSM_TRAIN_H */
