/*
 * glr.h -- C ABI of the gated linear recurrence in libssmscan.so (sm_103a):
 * forward over a sequence, its backward pass, and the single-token step.
 *
 * The operation, per channel d of [B, L, D] (one real state a channel, the
 * two gates fused), with s = softplus(lam[d]) and a constant c > 0:
 *   r_t = sigmoid(rgate_t),  i_t = sigmoid(igate_t)
 *   log a_t = -c s r_t                                  (a_t in (0, 1])
 *   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,  y_t = h_t
 * h starts from h0 (zeros when NULL). sqrt(1 - a^2) keeps the state's
 * variance that of its input; it is evaluated as sqrt(w (2 - w)) from
 * w = 1 - a = -expm1(log a), so that it keeps its leading digits for decays
 * near 1, and a from the exponential itself where it is small.
 * Backward for loss = <dy, y> + <dh_last, h_last>, with g_t the whole
 * gradient of h_t:
 *   g_t = dy_t + a_{t+1} g_{t+1}  (g_{L-1} = dy_{L-1} + dh_last)
 *   dx = g sqrt(1-a^2) i;  digate = g sqrt(1-a^2) x i (1-i)
 *   dloga = g (a h_{t-1} - a^2/sqrt(1-a^2) i x)   (second term 0 where a = 1)
 *   drgate = -c s dloga r (1-r);  dlam = -c sigmoid(lam) sum_{b,t} dloga r
 *   dh0 = a_0 g_0
 *
 * Layout: token-major, channel-contiguous. x, rgate, igate [B, L, D] in the
 * I/O dtype (SSM_F32 or SSM_BF16), the rows of each evenly spaced: x_stride,
 * r_stride and i_stride elements from one token to the next (0 = D, dense),
 * so all three may be column slices of one projection's output. y, dy, dx,
 * drgate, digate [B, L, D] dense, I/O dtype. lam, dlam [D]; h0, h_last,
 * dh_last, dh0, state [B, D]; ckpt [B, ceil(L/32), D]: the state before
 * tokens 0, 32, 64, ...; all fp32. Arithmetic, the state, the carries and
 * the sums are fp32.
 *
 * D must be a multiple of 8, every pointer 16-byte aligned and every row
 * stride a multiple of 16 bytes (else SSM_ERR_ALIGNMENT); strides of at
 * least D, c finite and positive, sizes non-negative, required pointers
 * non-null (else SSM_ERR_INVALID_ARG); at most 2^31 - 65 token rows and 2^31 - 1
 * tiles of 32 tokens x 64 channels (else SSM_ERR_UNSUPPORTED). B, L or D may be 0; with L = 0
 * h_last is h0, dh0 is dh_last and dlam is zero. Outputs must not overlap
 * inputs, except that dx may be dy, h_last h0 and dh0 dh_last (the state is
 * then carried on in its place).
 *
 * workspace: >= ssm_glr_workspace_bytes(B, L, D) bytes, 16-byte aligned: the
 * status word (ssm_poll_status: non-finite outputs; SSM_ERR_TIMEOUT if a
 * wait for another tile's carry ran out) and the carries. The library
 * prepares everything in it but the status word. Calls that overlap on the
 * GPU need a workspace each. Results do not depend on the order in which
 * the GPU runs the tiles: the same inputs give the same bits.
 * Calls are asynchronous on `stream` and allocate nothing; argument errors
 * return a negative SSM_ code before anything is launched.
 */
#ifndef GLR_H
#define GLR_H

#include <stddef.h>
#include <stdint.h>

#include "ssm_scan.h" /* the SSM_ status codes and ssm_poll_status */

#ifdef __cplusplus
extern "C" {
#endif

/* Forward. y required; h_last (nullable) the state after the last token;
 * ckpt (nullable) ssm_glr_ckpt_elems(B, L, D) floats for the backward. */
typedef struct {
    int64_t B, L, D;
    int64_t x_stride, r_stride, i_stride;
    int32_t io_dtype; /* ssm_dtype */
    float c;
    const void* x;
    const void* rgate;
    const void* igate;
    const float* lam;
    const float* h0;
    void* y;
    float* h_last;
    float* ckpt;
    void* workspace;
    size_t workspace_bytes;
} ssm_glr_args;

/* Backward. f: the forward's arguments (x, rgate, igate, lam and f.ckpt as
 * the forward left it are read; f.h0, f.y and f.h_last are not touched: the
 * first checkpoint is h0). dh_last and dh0 are nullable. */
typedef struct {
    ssm_glr_args f;
    const void* dy;
    const float* dh_last;
    void* dx;
    void* drgate;
    void* digate;
    float* dlam;
    float* dh0;
} ssm_glr_bwd_args;

/* One token: x_t, rgate_t, igate_t [B, D] (row strides as above), state
 * [B, D] fp32 updated in place, y_t [B, D] dense. workspace: nullable status
 * word (>= 256 bytes). */
typedef struct {
    int64_t B, D;
    int64_t x_stride, r_stride, i_stride;
    int32_t io_dtype;
    float c;
    const void* x_t;
    const void* rgate_t;
    const void* igate_t;
    const float* lam;
    float* state;
    void* y_t;
    void* workspace;
} ssm_glr_step_args;

int ssm_glr_fwd(const ssm_glr_args* args, void* stream);
int ssm_glr_bwd(const ssm_glr_bwd_args* args, void* stream);
int ssm_glr_step(const ssm_glr_step_args* args, void* stream);

/* Bytes of workspace a forward or backward call of this shape needs. */
size_t ssm_glr_workspace_bytes(int64_t B, int64_t L, int64_t D);
/* fp32 elements of the checkpoint buffer: B * ceil(L/32) * D. */
int64_t ssm_glr_ckpt_elems(int64_t B, int64_t L, int64_t D);

/* Test hook: arms, for this thread's next ssm_glr_fwd or ssm_glr_bwd only, a missing carry:
 * the tiles of chunk `chunk` (64 tokens in bf16, 32 in fp32, counted from 0) withhold what they
 * would hand on, and every bounded wait of that call gives up after wait_ns
 * (0: one second). The tiles that come after it in the scan (in the backward the
 * earlier chunks) stop and ssm_poll_status returns SSM_ERR_TIMEOUT. chunk < 0 disarms. SSM_ERR_INVALID_ARG for wait_ns above
 * 10 s. */
int ssm_glr_debug_arm_wait_fault(int64_t chunk, uint64_t wait_ns);

#ifdef __cplusplus
}
#endif
#endif /* GLR_H */
