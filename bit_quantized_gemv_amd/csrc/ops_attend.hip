// ops_attend.hip -- qmv_attend: attention of each sequence's new tokens over the
// pages of a cache.  What is launched for a call, and the join of what its workgroups found.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ops_attend.hpp"

namespace ops {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;      // slots of a row asked for at once

// The parts of a block's rows, joined: leaves to supers and supers to rows, in order.  2^lanes_log2
// lanes a row, four values each.
__global__ __launch_bounds__(kThreads) void join_blocks_kernel(AttendParams p, int leaf, int lanes_log2)
{
    const int b = blockIdx.y;
    const Seq s = sequence(p.cache, b);
    if (s.count > kBlockTokens) return;
    const int tokens = min(s.count, p.max_new);
    const int r = blockIdx.x * (kThreads >> lanes_log2) + (threadIdx.x >> lanes_log2), d = (threadIdx.x & ((1 << lanes_log2) - 1)) * 4;
    if (r >= tokens * p.q_heads || d >= p.D) return;
    const Visible vis = visible(s, tokens, p.window, p.sinks, leaf * p.per_unit);
    const long long row = (long long)s.start * p.q_heads + r;
    const f32x2* stat = p.stat + row * p.slots;
    const float* part = p.part + row * p.slots * p.D + d;
    float m = kGone, l = 0.0f, ms = kGone, ls = 0.0f;
    f32x4 o = {0, 0, 0, 0}, os = {0, 0, 0, 0};
    int super = -1;
    for (int u0 = 0; u0 < vis.units; u0 += kAhead) {
        f32x2 st[kAhead];
        f32x4 pa[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int u = min(u0 + i, vis.units - 1);
            st[i] = stat[u];
            pa[i] = *reinterpret_cast<const f32x4*>(part + (long long)u * p.D);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (u0 + i >= vis.units) break;
            const int now = vis.unit(u0 + i) * p.per_unit / kSuper;
            if (now != super) {
                const Factors f = join(m, l, ms, ls);
                o = joined(o, os, f);
                ms = kGone;
                ls = 0.0f;
                os = f32x4{0, 0, 0, 0};
                super = now;
            }
            const Factors f = join(ms, ls, st[i].x, st[i].y);
            os = joined(os, pa[i], f);
        }
    }
    const Factors f = join(m, l, ms, ls);
    o = joined(o, os, f);
    put_result(p, row, d, o, l);
}

template <class X>
__global__ __launch_bounds__(64) void attend_kernel(AttendParams p)
{
    const int lane = threadIdx.x, h = blockIdx.x, t = blockIdx.y + blockIdx.z * 65535;
    if (t >= p.cache.T) return;
    const int b = sequence_of(p.cache, t, lane);
    if (b < 0) return;
    const Seq s = sequence(p.cache, b);
    const int at = t - s.start;
    if (s.count <= kBlockTokens || at < 0 || at >= s.count || at >= p.max_new) return;
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
        const float top = __builtin_fmaxf(m, x), a = exp2_of(m - top), e = exp2_of(x - top);
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

int bound_of(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// How a call is cut up: by its sizes alone.
struct Plan {
    int max_new, length;                          // as far as they matter
    int window, sinks;
    int leaf, row_tiles, row_blocks, per_unit;
    long long units;                              // of a sequence, at most
    long long rows, part_bytes, stat_bytes;
};

// units of U places that a sequence's block can see
long long units_of(const Plan& p, int tokens, long long U)
{
    const long long all = std::max<long long>(1, (p.length + U - 1) / U);
    if (p.window == 0) return all;
    return std::min(all, (std::min(p.sinks, p.length) + U - 1) / U + ((long long)p.window + tokens - 1 + U - 1) / U + 1);
}

Plan plan_of(const qmv_cache* c, int T, int q_heads, int max_new, int max_length, int window, int sinks)
{
    Plan p;
    p.max_new = std::min(max_new, T);
    p.length = (int)std::min<long long>(max_length, (long long)c->max_pages * c->page_size);
    p.window = std::min(window, QMV_MAX_LENGTH);
    p.sinks = window > 0 ? std::min(sinks, QMV_MAX_LENGTH) : 0;
    const int group = q_heads / c->heads, tokens = std::min(p.max_new, kBlockTokens);
    const int rows = tokens * group;
    p.leaf = 32768 / bound_of(c->head_size);
    p.row_tiles = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    p.row_blocks = (rows + 16 * p.row_tiles - 1) / (16 * p.row_tiles);
    // leaf by leaf while that is few workgroups, else a super each
    const long long leaves = units_of(p, tokens, p.leaf);
    p.per_unit = leaves * c->heads * p.row_blocks * c->n_seqs > 2048 ? kSuper : 1;
    p.units = units_of(p, tokens, (long long)p.leaf * p.per_unit);
    p.rows = (long long)T * q_heads;
    p.part_bytes = p.units > 1 ? piece(p.rows * p.units * c->head_size * 4) : 0;
    p.stat_bytes = p.units > 1 ? piece(p.rows * p.units * 8) : 0;
    return p;
}

const void* block_kernel_of(int bound, bool f16, bool f32_out, int row_tiles, int* lds)
{
    return bound == 64 ? block_kernel_64(f16, f32_out, row_tiles, lds) : bound == 128 ? block_kernel_128(f16, f32_out, row_tiles, lds)
                                                                                     : block_kernel_256(f16, f32_out, row_tiles, lds);
}

}  // namespace
}  // namespace ops

extern "C" {

long long qmv_attend_workspace(const qmv_cache* c, int T, int q_heads, int max_new, int max_length,
                               int window, int sinks)
{
    using namespace ops;
    if (!c || check_sizes(c, T, q_heads, max_new, max_length, window, sinks) != QMV_OK) return -1;
    const Plan plan = plan_of(c, T, q_heads, max_new, max_length, window, sinks);
    return plan.part_bytes + plan.stat_bytes;
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
    const Plan plan = plan_of(c, T, q_heads, max_new, max_length, window, sinks);
    const long long need = plan.part_bytes + plan.stat_bytes;
    if (workspace_bytes < need) return QMV_E_WORKSPACE;
    const Span in[] = {{q, (size_t)nq * 2}, {c->k, cs.k}, {c->v, cs.v}, {c->pages, cs.pages}, {c->starts, (size_t)(c->n_seqs + 1) * 4},
                       {c->lengths, (size_t)c->n_seqs * 4}};
    const Span outs[] = {{out, (size_t)T * q_heads * c->head_size * size_of(out_dt)}, {workspace, (size_t)need}};
    if (!disjoint(in, outs)) return QMV_E_ALIAS;
    const long long groups = (plan.units * c->heads + 7) / 8 * 8 * plan.row_blocks;
    if (groups > (1 << 24) - 1) return QMV_E_CACHE;      // a launch's size in threads is a 32-bit number
    AttendParams p;
    p.q = static_cast<const char*>(q);
    p.out = static_cast<char*>(out);
    p.part = static_cast<float*>(workspace);
    p.stat = reinterpret_cast<f32x2*>(static_cast<char*>(workspace) + plan.part_bytes);
    p.q_token = 2 * q_token;
    p.q_head = 2 * q_head;
    p.q_heads = q_heads;
    p.heads = c->heads;
    p.group = q_heads / c->heads;
    p.D = c->head_size;
    p.window = plan.window;
    p.sinks = plan.sinks;
    p.max_new = plan.max_new;
    p.out_f32 = out_dt == QMV_DT_F32;
    p.slots = p.units = (int)plan.units;
    p.row_blocks = plan.row_blocks;
    p.per_unit = plan.per_unit;
    p.scale = scale * 1.44269504088896340736f;
    p.cache = device_cache(c, T);
    p.cache.max_places = plan.length;
    hipStream_t st = static_cast<hipStream_t>(stream);
    int lds;
    const void* f = block_kernel_of(bound_of(p.D), c->dt == QMV_DT_F16, p.out_f32, plan.row_tiles, &lds);
    void* args[] = {&p};
    if (hipLaunchKernel(f, dim3((unsigned)groups, c->n_seqs), dim3(kThreads), args, (size_t)lds, st) != hipSuccess) return QMV_E_LAUNCH;
    if (plan.units > 1) {
        int lanes_log2 = 1, leaf = plan.leaf;
        while (4 << lanes_log2 < p.D) ++lanes_log2;
        const int rows = std::min(plan.max_new, kBlockTokens) * q_heads, per = kThreads >> lanes_log2;
        void* more[] = {&p, &leaf, &lanes_log2};
        if (hipLaunchKernel((const void*)&join_blocks_kernel, dim3((rows + per - 1) / per, c->n_seqs), dim3(kThreads), more, 0, st) != hipSuccess)
            return QMV_E_LAUNCH;
    }
    if (plan.max_new > kBlockTokens) {
        const void* f = c->dt == QMV_DT_F16 ? (const void*)&attend_kernel<_Float16> : (const void*)&attend_kernel<__bf16>;
        if (hipLaunchKernel(f, dim3(q_heads, std::min(T, 65535), (T + 65534) / 65535), dim3(64), args, 0, st) != hipSuccess) return QMV_E_LAUNCH;
    }
    return QMV_OK;
}

}  // extern "C"
