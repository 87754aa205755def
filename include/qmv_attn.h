/*
 * qmv_attn.h -- C ABI of what lies between the quantized projections of a
 * decode, verify or prompt step on MI355X (gfx950):
 *
 *   qmv_rotate   norms of queries and keys for each head, and their position
 *                rotation, in one pass
 *   qmv_append   the same, with keys and values written to the pages of a cache
 *   qmv_attend   attention of each sequence's new tokens over its pages
 *
 * The conventions of qmv.h and qmv_ops.h hold: dtypes and status codes, device
 * pointers owned by the caller, calls asynchronous on `stream`, arguments checked
 * on the host before anything is enqueued, scratch memory given by the caller,
 * nothing kept between calls, no synchronization, calls that can be captured.
 * The structs are read during the call only.  What they point to on the device
 * (pages, starts, lengths, positions, axes) is read by the kernels, which keep
 * every access inside the arrays whatever the values are.
 */
#ifndef QMV_ATTN_H
#define QMV_ATTN_H

#include <stdint.h>

#include "qmv.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    QMV_E_HEADS = 16, /* head size not a multiple of 8 in [8, QMV_MAX_HEAD_SIZE], heads not in
                         [1, QMV_MAX_HEADS], query heads not a multiple of the cache's, a rotated
                         part not a multiple of 8 in [0, head size], or axes not in
                         [1, QMV_MAX_AXES] */
    QMV_E_CACHE = 17  /* pages, page size, sequences, tokens, a bound on the lengths, window or
                         sinks outside the limits */
};

#define QMV_MAX_HEAD_SIZE 256
#define QMV_MAX_HEADS 1024
#define QMV_MAX_AXES 8
#define QMV_MAX_PAGE_SIZE 65536
#define QMV_MAX_SEQS 65535
#define QMV_MAX_LENGTH (1 << 30)   /* places of a sequence: max_pages * page_size at most */
#define QMV_MAX_TOKENS (1 << 22)   /* new tokens of a call */

/*
 * A cache in pages, and the batch of sequences that a call works on.
 *   k, v     [n_pages][page_size][heads][head_size] of dt (fp16 or bf16) in any order:
 *            value d of head h of slot s of page p at element p * k_page + s * k_slot +
 *            h * k_head + d (v the same); strides multiples of 8, k and v 16-byte aligned
 *   pages    int32, row b (at b * pages_row) the max_pages pages of sequence b: its place j
 *            is slot j % page_size of page pages[b][j / page_size].  A page outside
 *            [0, n_pages) holds nothing: its places are not seen, and not written
 *   starts   int32 [n_seqs + 1], ascending: the call's tokens starts[b] .. starts[b + 1] - 1
 *            are the new ones of sequence b (there may be none); tokens outside all sequences
 *            are left out, and their rows of outputs as they were
 *   lengths  int32 [n_seqs]: sequence b's places with its new tokens, which are the last of
 *            them (more than max_pages * page_size count as that many)
 * Sequences may share pages that are only read.
 */
typedef struct {
    void* k;
    void* v;
    long long k_page, k_slot, k_head, v_page, v_slot, v_head;
    const int32_t* pages;
    const int32_t* starts;
    const int32_t* lengths;
    long long pages_row;
    int n_pages, page_size, n_seqs, max_pages;
    int heads, head_size, dt;
} qmv_cache;

/*
 * Norms and rotation of a head x of D values:
 *   n = x * w / sqrt(mean(x^2) + eps)           (weight NULL: n = x)
 *   pair i < rot / 2 of n is turned by the angle positions[axes[i]][t] * freqs[i]:
 *   (a, b) -> (a cos - b sin, b cos + a sin); the pair's places are i and i + rot / 2, or
 *   2i and 2i + 1 if `interleaved`; the values from rot on stay
 * The norm is taken in fp32, of heads of any size that fp32 holds, the angle in fp64, and the
 * result rounded once.
 *   freqs     fp32 [rot / 2]
 *   positions int32, row a (at a * positions_row) the T positions of axis a
 *   axes      int32 [rot / 2] (NULL: all 0); outside [0, n_axes): not turned
 *   q_weight, k_weight: [head_size] of w_dt (fp32 or bf16), each may be NULL
 */
typedef struct {
    const float* freqs;
    const int32_t* positions;
    const int32_t* axes;
    const void* q_weight;
    const void* k_weight;
    long long positions_row;
    float eps;
    int rot, n_axes, interleaved, w_dt;
} qmv_rotation;

/*
 * q [T][q_heads][head_size], k [T][k_heads][head_size] of x_dt (fp32 or bf16): value d of
 * head h of token t at element t * q_token + h * q_head + d, strides multiples of 8;
 * q_out, k_out the same shapes of out_dt (fp16 or bf16), contiguous.  All 16-byte aligned.
 * Each head's outputs depend on that head and its token's positions alone.
 */
int qmv_rotate(const qmv_rotation* r, const void* q, const void* k, void* q_out, void* k_out,
               int T, int q_heads, int k_heads, int head_size, long long q_token,
               long long q_head, long long k_token, long long k_head, int x_dt, int out_dt,
               void* stream);

/*
 * The same for the new tokens of a cache's sequences: q_out (of the cache's dtype,
 * contiguous), keys and values (v: rounded only) to their places.  positions NULL: a token's
 * place in its sequence.  Places below 0 (more new tokens than the length says) or on a page that
 * holds nothing are not written.  A length above the table's counts as the table's, here too: the new
 * tokens are its last places then, and write over what is there.  The cache's strides must keep its
 * values apart (QMV_E_STRIDE), k and v must not share values, and no two new tokens a slot.
 */
int qmv_append(const qmv_rotation* r, const qmv_cache* c, const void* q, const void* k,
               const void* v, void* q_out, int T, int q_heads, long long q_token,
               long long q_head, long long k_token, long long k_head, long long v_token,
               long long v_head, int x_dt, void* stream);

/*
 * Attention: new token i of sequence b, at place p = lengths[b] - (its new tokens) + i, sees
 * place j if j <= p, and, if window > 0, j > p - window or j < sinks.  For every head h
 *   out = sum_j softmax_j(scale * q . k_j) v_j     over the places it sees,
 * k and v those of head h / (q_heads / heads); zeros if it sees none.  A place that a token
 * does not see does not touch its output, whatever is there.
 *   q    [T][q_heads][head_size] of the cache's dtype: at t * q_token + h * q_head + d,
 *        strides multiples of 8, 16-byte aligned
 *   out  [T][q_heads][head_size] of out_dt (fp32 or bf16), contiguous, 16-byte aligned
 *   max_new, max_length: bounds on the sequences' new tokens (those above are left out, and
 *        their rows as they were) and lengths (longer ones count as that long).  Launch and
 *        workspace go by the bounds: both grow with max_length where sequences are far shorter
 *   workspace: qmv_attend_workspace bytes, 16-byte aligned; NULL where those are 0.  It holds
 *        nothing between calls, and serves one call at a time
 * Products are exact, and sums, maxima and exponentials fp32; the weights are rounded to the
 * cache's dtype for the second product, or split into pieces that hold 22 bits or more of them if
 * out is fp32.  fp16 weights below 2^-25 of the row's largest (fp32 out: 2^-17) are held to 2^-36
 * (2^-39) of that instead.  A value of the cache that is infinite or NaN makes infinite or NaN
 * (either) what the rows that see it sum up with it; but a key whose score is -inf weighs nothing.
 * Sequences of up to 16 new tokens: a token's bits depend on its place, the keys and values that it
 * sees and the head size alone, so those of a block are those of a call for each token, whatever
 * else is in the call.  Of longer ones the order of sums goes with the call's sizes.  A
 * call repeated gives the same bits.  No atomics.
 */
long long qmv_attend_workspace(const qmv_cache* c, int T, int q_heads, int max_new,
                               int max_length, int window, int sinks);
int qmv_attend(const qmv_cache* c, const void* q, void* out, void* workspace,
               long long workspace_bytes, int T, int q_heads, long long q_token,
               long long q_head, int max_new, int max_length, int window, int sinks,
               float scale, int out_dt, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMV_ATTN_H */
