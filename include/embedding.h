/*
 * embedding.h -- C ABI of the scaled embedding lookup and its gradient in
 * libssmscan.so (sm_103a).
 *
 *   forward:   out[t, :] = scale * W[id[t], :]
 *   backward:  dW[v, :]  = scale * sum over the tokens t with id[t] = v of dy[t, :]
 *              (0 for a row that no token names, and for padding_id)
 *
 * ids [tokens] int64 or int32; W [V, D] and out, dy [tokens, D] dense in the
 * I/O dtype (SSM_F32 or SSM_BF16); dW [V, D] fp32, every element written. The
 * sum is taken in fp32 over the tokens in their order, sorted by id first: no
 * atomics, the same inputs give the same bits.
 *
 * An id outside [0, V) reads nothing: its output row is zero, its gradient
 * row goes nowhere, and the status word says so (ssm_poll_status:
 * SSM_ERR_INDEX). padding_id takes part in the lookup like any id; its
 * gradient is zero. padding_id outside [0, V): none.
 *
 * Any D >= 1, any alignment of W, out, dy and dW that suits their elements
 * (else SSM_ERR_ALIGNMENT); rows whose starts are not all on 16 bytes are read
 * one element at a time. V and tokens below 2^30 and D at most 2^20
 * (else SSM_ERR_UNSUPPORTED).
 * tokens, V or D may be 0. status: nullable, >= 256 bytes, 16-byte aligned.
 * Calls are asynchronous on `stream` and allocate nothing; argument errors
 * return before anything is launched.
 */
#ifndef SSM_EMBEDDING_H
#define SSM_EMBEDDING_H

#include <stddef.h>
#include <stdint.h>

#include "ssm_scan.h" /* the SSM_ status codes and ssm_poll_status */

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int64_t tokens, V, D;
    int32_t io_dtype;
    int32_t ids64; /* 1: ids are int64; 0: int32 */
    float scale;
    int32_t pad_;
    const void* ids;
    const void* W;
    void* out;
    void* status;
} ssm_embed_args;

/* workspace: >= ssm_embed_workspace_bytes(tokens, V, D) bytes, 16-byte
 * aligned: the sorted tokens and the partial sums of long runs. */
typedef struct {
    int64_t tokens, V, D;
    int64_t padding_id;
    int32_t io_dtype;
    int32_t ids64;
    float scale;
    int32_t pad_;
    const void* ids;
    const void* dy;
    float* dW;
    void* workspace;
    size_t workspace_bytes;
    void* status;
} ssm_embed_bwd_args;

int ssm_embed_fwd(const ssm_embed_args* args, void* stream);
int ssm_embed_bwd(const ssm_embed_bwd_args* args, void* stream);
size_t ssm_embed_workspace_bytes(int64_t tokens, int64_t V, int64_t D);

#ifdef __cplusplus
}
#endif
#endif /* SSM_EMBEDDING_H */
