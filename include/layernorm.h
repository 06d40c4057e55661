/*
 * layernorm.h -- C ABI of layer norm in libssmscan.so (sm_103a): forward over
 * rows, and the backward pass with the sums for weight and bias.
 *
 *   mean = sum_d x / D,  var = sum_d (x - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
 *   xh = (x - mean) rstd,  y = xh w + b
 * Backward for loss = <dy, y>, with t = dy w:
 *   dx = rstd (t - sum_d t / D - xh sum_d (t xh) / D)
 *   dw = sum over rows of dy xh,  db = sum over rows of dy
 *
 * x [rows, D], rows x_stride elements apart (0 = D, dense); y, dy, dx
 * [rows, D] dense; all in the I/O dtype (SSM_F32 or SSM_BF16). w, b, dw, db
 * [D] and mean, rstd [rows] fp32. Any D >= 1. Pointers need the alignment of
 * their elements only (else SSM_ERR_ALIGNMENT); rows whose starts are not all
 * on 16 bytes are read one element at a time. Sums are fp32, the variance
 * from the centred values (no cancellation for rows with a large mean).
 * Summing orders are fixed: the same inputs give the same bits.
 *
 * rows or D may be 0 (dw, db are then zero; mean and rstd of rows without
 * elements are not written). eps finite and non-negative,
 * sizes non-negative, x_stride 0 or >= D (else SSM_ERR_INVALID_ARG). y may be
 * x, and dx may be dy or x, where those are dense; nothing else may overlap.
 * status: nullable, >= 256 bytes, 16-byte aligned: the status word
 * (ssm_poll_status: non-finite outputs). Calls are asynchronous on `stream`
 * and allocate nothing; argument errors return before anything is launched.
 */
#ifndef SSM_LAYERNORM_H
#define SSM_LAYERNORM_H

#include <stddef.h>
#include <stdint.h>

#include "ssm_scan.h" /* the SSM_ status codes and ssm_poll_status */

#ifdef __cplusplus
extern "C" {
#endif

/* w and b nullable (1 and 0); mean and rstd nullable (the backward needs
 * both). */
typedef struct {
    int64_t rows, D, x_stride;
    int32_t io_dtype;
    float eps;
    const void* x;
    const float* w;
    const float* b;
    void* y;
    float* mean;
    float* rstd;
    void* status;
} ssm_layernorm_args;

/* f: x, w, mean and rstd are read; f.b, f.y and f.eps are not. dw and db
 * nullable. workspace: >= ssm_layernorm_workspace_bytes(rows, D) bytes,
 * 16-byte aligned, needed when dw or db is given: partial sums (no status
 * word; that is f.status). */
typedef struct {
    ssm_layernorm_args f;
    const void* dy;
    void* dx;
    float* dw;
    float* db;
    void* workspace;
    size_t workspace_bytes;
} ssm_layernorm_bwd_args;

int ssm_layernorm_fwd(const ssm_layernorm_args* args, void* stream);
int ssm_layernorm_bwd(const ssm_layernorm_bwd_args* args, void* stream);
size_t ssm_layernorm_workspace_bytes(int64_t rows, int64_t D);

#ifdef __cplusplus
}
#endif
#endif /* SSM_LAYERNORM_H */
