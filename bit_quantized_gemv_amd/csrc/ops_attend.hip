// ops_attend.hip -- qmv_attend: attention of each sequence's new tokens over the
// pages of a cache.
//
// One pass over the keys with the running maximum and sum of the softmax: a wave per query
// head of a token, whose lanes hold the head's values.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ops_cache.hpp"

namespace ops {
namespace {

struct AttendParams {
    const char* q;
    char* out;
    long long q_token, q_head;      // bytes
    int q_heads, heads, D, window, sinks, max_new, out_f32;
    float scale;
    Cache cache;
};

template <class X>
__global__ __launch_bounds__(64) void attend_kernel(AttendParams p)
{
    const int lane = threadIdx.x, h = blockIdx.x, t = blockIdx.y + blockIdx.z * 65535;
    if (t >= p.cache.T) return;
    const int b = sequence_of(p.cache, t, lane);
    if (b < 0) return;
    const Seq s = sequence(p.cache, b);
    const int at = t - s.start;
    if (at < 0 || at >= s.count || at >= p.max_new) return;
    const int place = s.length - s.count + at, kh = h / (p.q_heads / p.heads);
    constexpr int R = QMV_MAX_HEAD_SIZE / 64;
    float q[R], o[R];
    const X* qr = reinterpret_cast<const X*>(p.q + t * p.q_token + h * p.q_head);
    for (int i = 0; i < R; ++i) {
        q[i] = i * 64 + lane < p.D ? (float)qr[i * 64 + lane] * p.scale : 0.0f;
        o[i] = 0.0f;
    }
    float m = -__builtin_huge_valf(), l = 0.0f;
    for (int j = 0; j <= place; ++j) {
        if (p.window > 0 && j <= place - p.window && j >= p.sinks) j = place - p.window + 1;
        const int index = page_index(p.cache, j), page = page_of(p.cache, b, index);
        if (page < 0) continue;
        const int slot = j - index * p.cache.page_size;
        const X* k = reinterpret_cast<const X*>(p.cache.k + page * p.cache.k_page + slot * p.cache.k_slot + kh * p.cache.k_head);
        const X* v = reinterpret_cast<const X*>(p.cache.v + page * p.cache.v_page + slot * p.cache.v_slot + kh * p.cache.v_head);
        float x = 0.0f;
        for (int i = 0; i < R; ++i)
            if (i * 64 + lane < p.D) x = __builtin_fmaf(q[i], (float)k[i * 64 + lane], x);
        for (int i = 1; i < 64; i <<= 1) x += __shfl_xor(x, i);
        const float top = __builtin_fmaxf(m, x), a = __expf(m - top), e = __expf(x - top);
        m = top;
        l = l * a + e;
        for (int i = 0; i < R; ++i)
            if (i * 64 + lane < p.D) o[i] = o[i] * a + e * (float)v[i * 64 + lane];
    }
    const float r = l > 0.0f ? 1.0f / l : l;
    for (int i = 0; i < R; ++i) {
        const int d = i * 64 + lane;
        const long long to = ((long long)t * p.q_heads + h) * p.D + d;
        if (d >= p.D) continue;
        if (p.out_f32) reinterpret_cast<float*>(p.out)[to] = o[i] * r;
        else reinterpret_cast<__bf16*>(p.out)[to] = (__bf16)(o[i] * r);
    }
}

int check_sizes(const qmv_cache* c, int T, int q_heads, int max_new, int max_length, int window, int sinks)
{
    if (int e = check_cache_sizes(c, T, q_heads)) return e;
    return max_new < 1 || max_length < 0 || window < 0 || sinks < 0 ? QMV_E_CACHE : QMV_OK;
}

}  // namespace
}  // namespace ops

extern "C" {

long long qmv_attend_workspace(const qmv_cache* c, int T, int q_heads, int max_new, int max_length,
                               int window, int sinks)
{
    using namespace ops;
    if (!c || check_sizes(c, T, q_heads, max_new, max_length, window, sinks) != QMV_OK) return -1;
    return 0;
}

int qmv_attend(const qmv_cache* c, const void* q, void* out, void* workspace,
               long long workspace_bytes, int T, int q_heads, long long q_token, long long q_head,
               int max_new, int max_length, int window, int sinks, float scale, int out_dt,
               void* stream)
{
    using namespace ops;
    if (!c || !q || !out || !workspace) return QMV_E_NULL;
    if (int e = check_sizes(c, T, q_heads, max_new, max_length, window, sinks)) return e;
    CacheSpans cs;
    if (int e = check_cache(c, T, q_heads, &cs)) return e;
    if (!wide(out_dt)) return QMV_E_DTYPE;
    if (!stride_ok(q_token) || !stride_ok(q_head)) return QMV_E_STRIDE;
    if (q_token % 8 != 0 || q_head % 8 != 0 || !aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16)) return QMV_E_ALIGN;
    const long long size[] = {T, q_heads}, stride[] = {q_token, q_head}, nq = extent(size, stride, c->head_size);
    if (nq < 0) return QMV_E_STRIDE;
    const long long need = qmv_attend_workspace(c, T, q_heads, max_new, max_length, window, sinks);
    if (workspace_bytes < need) return QMV_E_WORKSPACE;
    const Span in[] = {{q, (size_t)nq * 2}, {c->k, cs.k}, {c->v, cs.v}, {c->pages, cs.pages}, {c->starts, (size_t)(c->n_seqs + 1) * 4},
                       {c->lengths, (size_t)c->n_seqs * 4}};
    const Span outs[] = {{out, (size_t)T * q_heads * c->head_size * size_of(out_dt)}, {workspace, (size_t)need}};
    if (!disjoint(in, outs)) return QMV_E_ALIAS;
    AttendParams p;
    p.q = static_cast<const char*>(q);
    p.out = static_cast<char*>(out);
    p.q_token = 2 * q_token;
    p.q_head = 2 * q_head;
    p.q_heads = q_heads;
    p.heads = c->heads;
    p.D = c->head_size;
    p.window = window;
    p.sinks = sinks;
    p.max_new = max_new;
    p.out_f32 = out_dt == QMV_DT_F32;
    p.scale = scale;
    p.cache = device_cache(c, T);
    p.cache.max_places = std::min(p.cache.max_places, max_length);
    const void* f = c->dt == QMV_DT_F16 ? (const void*)&attend_kernel<_Float16> : (const void*)&attend_kernel<__bf16>;
    void* args[] = {&p};
    if (hipLaunchKernel(f, dim3(q_heads, std::min(T, 65535), (T + 65534) / 65535), dim3(64), args, 0, static_cast<hipStream_t>(stream)) != hipSuccess)
        return QMV_E_LAUNCH;
    return QMV_OK;
}

}  // extern "C"
