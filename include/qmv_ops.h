/*
 * qmv_ops.h -- C ABI of the operators that stand beside the quantized product
 * (qmv.h) in a decode or speculative-verify step on MI355X (gfx950):
 *
 *   qmv_affine_lora   the affine-quantized projection of many requests'
 *                     tokens, each with its own low-rank adapter or none
 *   qmv_route         a mixture-of-experts router: top-k experts and weights
 *   qmv_experts       the chosen affine-quantized experts' gated product
 *   qmv_moe           both: the whole layer
 *   qmv_verify        drafted tokens accepted or replaced by the target's
 *                     probabilities and given random numbers
 *
 * The conventions of qmv.h hold: packed codes with field 0 in the low bits,
 * scales and biases per group, dtypes (qmv_dtype) and status codes, device
 * pointers owned by the caller, calls asynchronous on `stream`, arguments
 * checked on the host before anything is enqueued (QMV_E_LAUNCH from the HIP
 * runtime refusing one of a call's launches is the exception: earlier ones may
 * have written).  The calls use scratch memory that the caller gives as
 * `workspace` (its size from the *_workspace function of the same arguments);
 * its content before the call does not matter and after it means nothing, and
 * two calls may share one only if they are ordered on one stream.  Nothing is
 * kept between calls.  The library never synchronizes; calls can be captured
 * into a HIP graph.
 *
 * Numerics.  Products run on matrix instructions that multiply bf16 values
 * exactly and add in fp32; wider operands (fp32 activations and hidden values,
 * fp16 adapters) are split into bf16 pieces that add up to the value.  The
 * order of every sum depends on the row length, bits and group size only,
 * never on how many tokens the call has, which of them share an adapter or an
 * expert, or the launch shape: each token's outputs are bit-identical to those
 * of a call with that token alone, and repeated calls are bit-identical.  (The
 * order is not qmv_affine's: the two agree to rounding.)  A token with a NaN
 * or an infinity has non-finite outputs; other tokens are not touched by it.
 * Sums within a group of 32 codes' products must stay inside fp32 at 16 times
 * their size.
 */
#ifndef QMV_OPS_H
#define QMV_OPS_H

#include <stdint.h>

#include "qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    QMV_E_RANK = 11,      /* adapter rank not in [1, QMV_MAX_RANK], or no adapters */
    QMV_E_EXPERTS = 12,   /* experts not in [1, QMV_MAX_EXPERTS], or top_k not in
                             [1, QMV_MAX_TOP_K], or above a router's experts */
    QMV_E_WORKSPACE = 13, /* the workspace is smaller than the call needs */
    QMV_E_VOCAB = 14,     /* vocabulary, draft length or batch outside the limits */
    QMV_E_STRIDE = 15     /* a stride is negative or above 2^40 */
};

#define QMV_MAX_RANK 512
#define QMV_MAX_ADAPTERS 65536
#define QMV_MAX_EXPERTS 1024
#define QMV_MAX_TOP_K 32
#define QMV_MAX_VOCAB (1 << 26)
#define QMV_MAX_DRAFT 255
#define QMV_MAX_BATCH 65535

/*
 * y[m] = W x[m] + c_a * B_a (A_a x[m]),  a = ids[m]
 *
 *   w, scales, biases, x, y, M, N, K, bits, group_size: as qmv_affine_ex
 *   lora_a  [n_adapters][rank][K], lora_b [n_adapters][N][rank] (fp16 or
 *           bf16: ad_dt)
 *   ids     int32 [M]; a value outside [0, n_adapters) means no adapter
 *   scaling fp32 [n_adapters], or NULL for 1
 * A_a x is held in fp32; W x, A_a x and B_a's product are added in fp32 and
 * rounded once to y's dtype.  lora_a, lora_b 16-byte aligned.
 */
long long qmv_affine_lora_workspace(int M, int K, int rank);
int qmv_affine_lora(const uint32_t* w, const void* scales, const void* biases, const void* x,
                    void* y, const void* lora_a, const void* lora_b, const int32_t* ids,
                    const float* scaling, void* workspace, long long workspace_bytes, int M, int N,
                    int K, int bits, int group_size, int n_adapters, int rank, int x_dt, int sb_dt,
                    int y_dt, int ad_dt, void* stream);

/*
 * Router: logits[t][e] = sum_d x[t][d] * router[e][d] in fp64; ids[t][0..k) the
 * top_k largest, in descending order, ties to the lowest index (a NaN counts
 * as the smallest); weights[t][j] their softmax, over the chosen ones if
 * `renormalize`, else over all experts.
 *   x [T][D], router [n_experts][D]: fp32 or bf16 (x_dt, r_dt); 16-byte aligned
 *   D a multiple of 8; weights fp32 [T][top_k]; ids int32 [T][top_k]
 */
long long qmv_route_workspace(int T, int D, int n_experts);
int qmv_route(const void* x, const void* router, float* weights, int32_t* ids, void* workspace,
              long long workspace_bytes, int T, int D, int n_experts, int top_k, int renormalize,
              int x_dt, int r_dt, void* stream);

/*
 * Experts: y[t] = sum_j weights[t][j] * Down_e ( silu(Gate_e x[t]) * Up_e x[t] ),
 * e = ids[t][j], summed in the order of j; a slot whose id is outside
 * [0, n_experts) adds nothing (its weight is not read), and a token with no
 * other slots gets zeros.  Gate_e x, Up_e x, the hidden values and the experts'
 * outputs are held in fp32, and y is rounded once.
 *   w13 [n_experts][2F][D*bits/32]: F gate rows, then F up rows; s13, b13
 *   [n_experts][2F][D/gs]; w2 [n_experts][D][F*bits/32]; s2, b2
 *   [n_experts][D][F/gs]; x [T][D]; y [T][D]
 *   D and F multiples of group_size
 */
long long qmv_experts_workspace(int T, int D, int F, int top_k);
int qmv_experts(const void* x, const float* weights, const int32_t* ids, const uint32_t* w13,
                const void* s13, const void* b13, const uint32_t* w2, const void* s2,
                const void* b2, void* y, void* workspace, long long workspace_bytes, int T, int D,
                int F, int n_experts, int top_k, int bits, int group_size, int x_dt, int sb_dt,
                int y_dt, void* stream);

/* The whole layer: qmv_route, then qmv_experts on its weights and ids (both
 * are outputs of the call). */
long long qmv_moe_workspace(int T, int D, int F, int n_experts, int top_k);
int qmv_moe(const void* x, const void* router, const uint32_t* w13, const void* s13,
            const void* b13, const uint32_t* w2, const void* s2, const void* b2, void* y,
            float* weights, int32_t* ids, void* workspace, long long workspace_bytes, int T, int D,
            int F, int n_experts, int top_k, int renormalize, int bits, int group_size, int x_dt,
            int r_dt, int sb_dt, int y_dt, void* stream);

/*
 * Verification of drafted tokens.  For request b with n = lengths[b] drafted
 * tokens (NULL: S; clamped to [0, S]) and p_j = softmax(logits[b][j] /
 * temperature[b]):
 *   position j < n is accepted while uniforms[b][j] * q_j(x_j) < p_j(x_j),
 *   x_j = draft[b][j] (a token outside the vocabulary is rejected);
 *   the first position r that is not is given a token sampled from
 *   max(p_r - q_r, 0) (from p_r where that is zero throughout); if all n are
 *   accepted, position n is given one sampled from p_n.
 * A sample is the lowest index whose inclusive prefix sum passes
 * uniforms[b][n] times the total (the last index of positive weight if none
 * does).  Probabilities, accept decisions and samples are those of fp64 sums of
 * the logits as they are given.  temperature[b] not above 0 is greedy: p_j is 1
 * at the largest logit (ties to the lowest index).  NaN and -inf logits have
 * probability 0; where the largest is +inf, the ones equal to it share 1.  A
 * row with no other logits rejects its position, and a token sampled from it
 * is -1.
 *   logits   fp32 or bf16 (l_dt): row j of request b at element
 *            b * l_batch + j * l_row, V contiguous; S + 1 rows
 *   draft    int32 [B][S]; uniforms fp32 [B][S + 1] in [0, 1)
 *   probs    q: fp32 or bf16 (q_dt), row j of request b at b * q_batch +
 *            j * q_row; NULL: q_j is 1 at x_j (a drafter that gives tokens only)
 *   temperature fp32 [B] (NULL: 1), lengths int32 [B] (NULL: S)
 *   tokens   int32 [B][S + 1]: the accepted tokens, the sampled one, then -1
 *   accepted int32 [B]: how many were accepted
 */
long long qmv_verify_workspace(int B, int S, int V);
int qmv_verify(const void* logits, const int32_t* draft, const float* uniforms, const void* probs,
               const float* temperature, const int32_t* lengths, int32_t* tokens,
               int32_t* accepted, void* workspace, long long workspace_bytes, int B, int S, int V,
               long long l_batch, long long l_row, long long q_batch, long long q_row, int l_dt,
               int q_dt, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMV_OPS_H */
