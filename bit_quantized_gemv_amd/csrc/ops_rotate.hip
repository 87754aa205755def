// ops_rotate.hip -- qmv_rotate and qmv_append: norms of queries and keys for
// each head, their position rotation, and keys and values to a cache's pages.
//
// One launch and one pass.  A head of D values is held by the lanes of a group, eight
// values each: where it is rotated, lane i < rot / 8 holds the values 4i .. 4i + 3 of the
// pairs' first places and the same of their second ones, so that a pair is turned within a
// lane, whichever way pairs lie.  The sum of squares is taken over the group's lanes, in
// fp32.  A workgroup takes all heads of some tokens (or some heads of one, where there
// are few tokens), since the angles are those of the token: a thread computes one of them,
// with its sine and cosine, for all heads.
//
// Angles: positions * freqs in fp64, as turns; the fraction of a turn that is left has lost
// nothing that fp32 holds, also at positions of 2^31.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ops_cache.hpp"

namespace ops {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;

constexpr int kThreads = 256;
constexpr int kHold = 4;              // heads in flight per group of lanes
constexpr int kMostTokens = 8;        // per workgroup
constexpr int kMostHalf = QMV_MAX_HEAD_SIZE / 2;

struct RotateParams {
    const char *q, *k, *v;
    char *q_out, *k_out;
    const char *q_weight, *k_weight;
    const float* freqs;
    const int32_t *positions, *axes;
    long long q_token, q_head, k_token, k_head, v_token, v_head;   // bytes
    long long positions_row;
    float eps;
    int T, q_heads, k_heads, D, half, n_axes, interleaved, w_f32;
    int lanes_log2;                   // lanes of a group
    int tokens, heads;                // per workgroup
    Cache cache;
};

template <class T>
struct Four;
template <>
struct Four<float> {
    typedef f32x4 type;
};
template <>
struct Four<__bf16> {
    typedef bf16x4 type;
};
template <>
struct Four<_Float16> {
    typedef f16x4 type;
};

template <class T>
__device__ __forceinline__ f32x4 wide_of(T v)
{
    return __builtin_convertvector(v, f32x4);
}

// sine and cosine of a fraction of a turn: its nearest quarter, and Taylor's series of what is
// left (at most pi / 4: the first term left out is below 2^-28)
__device__ __forceinline__ void sine_cosine(double turns, float& s, float& c)
{
    const double q = __builtin_rint(turns * 4.0);
    const float x = (float)((turns - q * 0.25) * 6.283185307179586476925);
    const float x2 = x * x;
    float a = __builtin_fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
    a = __builtin_fmaf(x2, a, 8.3333333e-3f);
    a = __builtin_fmaf(x2, a, -0.16666667f);
    a = __builtin_fmaf(x2 * x, a, x);
    float b = __builtin_fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
    b = __builtin_fmaf(x2, b, -1.3888889e-3f);
    b = __builtin_fmaf(x2, b, 4.1666667e-2f);
    b = __builtin_fmaf(x2, b, -0.5f);
    b = __builtin_fmaf(x2, b, 1.0f);
    const int n = (int)q & 3;
    const float sa = n & 1 ? b : a, ca = n & 1 ? a : b;
    s = n & 2 ? -sa : sa;
    c = (n + 1) & 2 ? -ca : ca;
}

// Whose rows a head of the workgroup's list is, and where they are.
struct Head {
    const char* from;
    char* to;              // nullptr: not written
    int which;             // 0 queries, 1 keys, 2 values
};

template <class X, class Y, bool APPEND>
__global__ __launch_bounds__(kThreads) void rotate_kernel(RotateParams p)
{
    typedef typename Four<X>::type X4;
    typedef typename Four<Y>::type Y4;
    __shared__ __align__(16) float cosines[kMostTokens * kMostHalf], sines[kMostTokens * kMostHalf];
    __shared__ int places[kMostTokens];
    __shared__ long long key_at[kMostTokens], value_at[kMostTokens];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t0 = blockIdx.x * p.tokens, tokens = min(p.tokens, p.T - t0);
    const int all = p.q_heads + (APPEND ? 2 : 1) * p.k_heads;
    const int h0 = blockIdx.y * p.heads, heads = min(p.heads, all - h0);
    const int items = tokens * heads;
    const int group = tid >> p.lanes_log2, part = tid & ((1 << p.lanes_log2) - 1), groups = kThreads >> p.lanes_log2;
    const bool live = part < p.D >> 3;
    // the lane's two runs of four values
    const bool turned = part < p.half >> 2;
    const int first = turned && !p.interleaved ? 4 * part : 8 * part, second = turned && !p.interleaved ? p.half + 4 * part : 8 * part + 4;

    auto head_of = [&](int item, int& tok) {
        tok = item / heads;
        const int h = h0 + item - tok * heads, t = t0 + tok;
        Head r;
        if (h < p.q_heads) {
            r.from = p.q + t * p.q_token + h * p.q_head;
            r.to = p.q_out + ((long long)t * p.q_heads + h) * p.D * sizeof(Y);
            r.which = 0;
        } else if (h < p.q_heads + p.k_heads) {
            r.from = p.k + t * p.k_token + (h - p.q_heads) * p.k_head;
            r.to = APPEND ? nullptr : p.k_out + ((long long)t * p.k_heads + h - p.q_heads) * p.D * sizeof(Y);
            r.which = 1;
        } else {
            r.from = p.v + t * p.v_token + (h - p.q_heads - p.k_heads) * p.v_head;
            r.to = nullptr;
            r.which = 2;
        }
        return r;
    };

    X4 a[kHold], b[kHold];
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int item = base + i * groups + group;
            if (live && item < items) {
                int tok;
                const char* from = head_of(item, tok).from;
                a[i] = *reinterpret_cast<const X4*>(from + first * sizeof(X));
                b[i] = *reinterpret_cast<const X4*>(from + second * sizeof(X));
            }
        }
    };
    load(0);

    if (APPEND) {
        for (int i = wave; i < tokens; i += kThreads / 64) {
            const int seq = sequence_of(p.cache, t0 + i, lane);
            if (lane == 0) {
                int place = 0;
                long long ka = -1, va = -1;
                bool in = false;
                if (seq >= 0) {
                    const Seq s = sequence(p.cache, seq);
                    const int at = t0 + i - s.start;
                    if (at >= 0 && at < s.count) {
                        in = true;
                        place = s.length - s.count + at;
                        if (place >= 0 && place < p.cache.max_places) {
                            const int index = page_index(p.cache, place), page = page_of(p.cache, seq, index);
                            if (page >= 0) {
                                const int slot = place - index * p.cache.page_size;
                                ka = page * p.cache.k_page + slot * p.cache.k_slot;
                                va = page * p.cache.v_page + slot * p.cache.v_slot;
                            }
                        }
                    }
                }
                places[i] = place;
                key_at[i] = in ? ka : -2;         // -2: the token is in no sequence, its queries are not written
                value_at[i] = va;
            }
        }
        __syncthreads();
    }
    for (int i = tid; i < tokens * p.half; i += kThreads) {
        const int tok = i / p.half, j = i - tok * p.half;
        const int axis = p.axes ? p.axes[j] : 0;
        float s = 0.0f, c = 1.0f;
        if ((uint32_t)axis < (uint32_t)p.n_axes) {
            const int pos = p.positions ? p.positions[axis * p.positions_row + t0 + tok] : places[tok];
            const double turns = (double)pos * ((double)p.freqs[j] * 0.15915494309189533576888);
            sine_cosine(turns - __builtin_floor(turns), s, c);
        }
        cosines[tok * kMostHalf + j] = c;
        sines[tok * kMostHalf + j] = s;
    }
    __syncthreads();

    for (int base = 0; base < items; base += kHold * groups) {
        if (base > 0) load(base);
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int item = base + i * groups + group;
            if (base + i * groups >= items) break;          // the whole workgroup's
            int tok = 0;
            Head h{nullptr, nullptr, 2};
            const bool mine = item < items;
            if (mine) h = head_of(item, tok);
            f32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
            if (mine && live) {
                x = wide_of(a[i]);
                y = wide_of(b[i]);
            }
            const char* w = h.which == 0 ? p.q_weight : p.k_weight;
            const f32x4 sq = x * x + y * y;
            float sum = (sq.x + sq.y) + (sq.z + sq.w);
            for (int m = 1; m < 1 << p.lanes_log2; m <<= 1) sum += __shfl_xor(sum, m);
            if (!mine || !live) continue;
            if (h.which < 2) {
                if (w) {
                    const float r = __builtin_amdgcn_rsqf(sum / (float)p.D + p.eps);
                    f32x4 wa, wb;
                    if (p.w_f32) {
                        wa = *reinterpret_cast<const f32x4*>(w + first * 4);
                        wb = *reinterpret_cast<const f32x4*>(w + second * 4);
                    } else {
                        wa = wide_of(*reinterpret_cast<const bf16x4*>(w + first * 2));
                        wb = wide_of(*reinterpret_cast<const bf16x4*>(w + second * 2));
                    }
                    x = x * r * wa;
                    y = y * r * wb;
                }
                if (turned) {
                    const f32x4 c = *reinterpret_cast<const f32x4*>(cosines + tok * kMostHalf + 4 * part);
                    const f32x4 s = *reinterpret_cast<const f32x4*>(sines + tok * kMostHalf + 4 * part);
                    if (p.interleaved) {          // the pairs are (x0 x1) (x2 x3) (y0 y1) (y2 y3)
                        const f32x4 e = {x.x, x.z, y.x, y.z}, o = {x.y, x.w, y.y, y.w};
                        const f32x4 u = e * c - o * s, v = o * c + e * s;
                        x = f32x4{u.x, v.x, u.y, v.y};
                        y = f32x4{u.z, v.z, u.w, v.w};
                    } else {
                        const f32x4 u = x * c - y * s;
                        y = y * c + x * s;
                        x = u;
                    }
                }
            }
            char* to = h.to;
            if (APPEND) {
                const long long ka = key_at[tok], va = value_at[tok];
                const int kh = h0 + item - tok * heads - p.q_heads - (h.which == 2 ? p.k_heads : 0);
                if (h.which == 0) to = ka == -2 ? nullptr : to;
                else if (h.which == 1) to = ka < 0 ? nullptr : const_cast<char*>(p.cache.k) + ka + kh * p.cache.k_head;
                else to = va < 0 ? nullptr : const_cast<char*>(p.cache.v) + va + kh * p.cache.v_head;
            }
            if (to) {
                *reinterpret_cast<Y4*>(to + first * sizeof(Y)) = __builtin_convertvector(x, Y4);
                *reinterpret_cast<Y4*>(to + second * sizeof(Y)) = __builtin_convertvector(y, Y4);
            }
        }
    }
}

int check_rotation(const qmv_rotation* r, int D, int T, bool append)
{
    if (r->rot < 0 || r->rot > D || r->rot % 8 != 0 || r->n_axes < 1 || r->n_axes > QMV_MAX_AXES) return QMV_E_HEADS;
    if (r->rot > 0 && (!r->freqs || (!append && !r->positions))) return QMV_E_NULL;
    if ((r->q_weight || r->k_weight) && !wide(r->w_dt)) return QMV_E_DTYPE;
    if (!stride_ok(r->positions_row) || (r->n_axes > 1 && r->positions && r->positions_row < 0)) return QMV_E_STRIDE;
    if (!aligned(r->freqs, 4) || !aligned(r->positions, 4) || !aligned(r->axes, 4) || !aligned(r->q_weight, 16) || !aligned(r->k_weight, 16))
        return QMV_E_ALIGN;
    return QMV_OK;
}

// strides of an input [T][heads][D]: its bytes, or an error below 0
long long input_span(int T, int heads, int D, long long token, long long head, int dt, int* e)
{
    *e = QMV_OK;
    if (!stride_ok(token) || !stride_ok(head)) *e = QMV_E_STRIDE;
    else if (token % 8 != 0 || head % 8 != 0) *e = QMV_E_ALIGN;
    if (*e) return 0;
    const long long size[] = {T, heads}, stride[] = {token, head};
    const long long n = extent(size, stride, D);
    if (n < 0) *e = QMV_E_STRIDE;
    return n * (long long)size_of(dt);
}

int run(RotateParams& p, const qmv_rotation* r, int T, int x_dt, int y_dt, bool append, void* stream)
{
    p.q_weight = static_cast<const char*>(r->q_weight);
    p.k_weight = static_cast<const char*>(r->k_weight);
    p.freqs = r->freqs;
    p.positions = r->positions;
    p.axes = r->axes;
    p.positions_row = r->positions_row;
    p.eps = r->eps;
    p.T = T;
    p.half = r->rot / 2;
    p.n_axes = r->n_axes;
    p.interleaved = r->interleaved != 0;
    p.w_f32 = r->w_dt == QMV_DT_F32;
    p.lanes_log2 = 0;
    while (1 << p.lanes_log2 < p.D / 8) ++p.lanes_log2;
    const int all = p.q_heads + (append ? 2 : 1) * p.k_heads, groups = kThreads >> p.lanes_log2;
    // A head per group where that is few workgroups; else all heads of a token (as many as
    // are in flight at once), or of several tokens, so that angles are computed once.
    p.tokens = 1;
    p.heads = std::min(all, groups);
    if ((long long)T * ((all + p.heads - 1) / p.heads) > 1024) {
        p.heads = std::min(all, kHold * groups);
        p.tokens = std::max(1, std::min(kMostTokens, kHold * groups / p.heads));
    }
    const bool xf = x_dt == QMV_DT_F32, yh = y_dt == QMV_DT_F16;
    const void* f;
    if (append)
        f = xf ? (yh ? (const void*)&rotate_kernel<float, _Float16, true> : (const void*)&rotate_kernel<float, __bf16, true>)
               : (yh ? (const void*)&rotate_kernel<__bf16, _Float16, true> : (const void*)&rotate_kernel<__bf16, __bf16, true>);
    else
        f = xf ? (yh ? (const void*)&rotate_kernel<float, _Float16, false> : (const void*)&rotate_kernel<float, __bf16, false>)
               : (yh ? (const void*)&rotate_kernel<__bf16, _Float16, false> : (const void*)&rotate_kernel<__bf16, __bf16, false>);
    void* args[] = {&p};
    const dim3 grid((T + p.tokens - 1) / p.tokens, (all + p.heads - 1) / p.heads);
    return hipLaunchKernel(f, grid, dim3(kThreads), args, 0, static_cast<hipStream_t>(stream)) == hipSuccess ? QMV_OK : QMV_E_LAUNCH;
}

Span weight_span(const void* w, int D, int dt) { return Span{w, (size_t)D * size_of(dt)}; }

size_t positions_bytes(const qmv_rotation* r, int T) { return r->positions ? (size_t)((r->n_axes - 1) * r->positions_row + T) * 4 : 0; }

}  // namespace
}  // namespace ops

extern "C" {

int qmv_rotate(const qmv_rotation* r, const void* q, const void* k, void* q_out, void* k_out, int T,
               int q_heads, int k_heads, int head_size, long long q_token, long long q_head,
               long long k_token, long long k_head, int x_dt, int out_dt, void* stream)
{
    using namespace ops;
    if (!r || !q || !k || !q_out || !k_out) return QMV_E_NULL;
    if (check_heads(q_heads, head_size) != QMV_OK || check_heads(k_heads, head_size) != QMV_OK) return QMV_E_HEADS;
    if (T < 1 || T > QMV_MAX_TOKENS) return QMV_E_CACHE;
    if (!wide(x_dt) || !half(out_dt)) return QMV_E_DTYPE;
    if (int e = check_rotation(r, head_size, T, false)) return e;
    int eq, ek;
    const long long nq = input_span(T, q_heads, head_size, q_token, q_head, x_dt, &eq);
    const long long nk = input_span(T, k_heads, head_size, k_token, k_head, x_dt, &ek);
    if (eq || ek) return eq ? eq : ek;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16)) return QMV_E_ALIGN;
    const size_t oq = (size_t)T * q_heads * head_size * 2, ok = (size_t)T * k_heads * head_size * 2;
    const Span in[] = {{q, (size_t)nq}, {k, (size_t)nk}, weight_span(r->q_weight, head_size, r->w_dt),
                       weight_span(r->k_weight, head_size, r->w_dt), {r->freqs, (size_t)r->rot * 2}, {r->axes, (size_t)r->rot * 2},
                       {r->positions, positions_bytes(r, T)}};
    const Span out[] = {{q_out, oq}, {k_out, ok}};
    if (!disjoint(in, out)) return QMV_E_ALIAS;
    RotateParams p{};
    p.q = static_cast<const char*>(q);
    p.k = static_cast<const char*>(k);
    p.q_out = static_cast<char*>(q_out);
    p.k_out = static_cast<char*>(k_out);
    p.q_token = q_token * (long long)size_of(x_dt);
    p.q_head = q_head * (long long)size_of(x_dt);
    p.k_token = k_token * (long long)size_of(x_dt);
    p.k_head = k_head * (long long)size_of(x_dt);
    p.q_heads = q_heads;
    p.k_heads = k_heads;
    p.D = head_size;
    return run(p, r, T, x_dt, out_dt, false, stream);
}

int qmv_append(const qmv_rotation* r, const qmv_cache* c, const void* q, const void* k, const void* v,
               void* q_out, int T, int q_heads, long long q_token, long long q_head,
               long long k_token, long long k_head, long long v_token, long long v_head, int x_dt,
               void* stream)
{
    using namespace ops;
    if (!r || !c || !q || !k || !v || !q_out) return QMV_E_NULL;
    CacheSpans cs;
    if (int e = check_cache(c, T, q_heads, &cs)) return e;
    if (!wide(x_dt)) return QMV_E_DTYPE;
    if (int e = check_rotation(r, c->head_size, T, true)) return e;
    const int D = c->head_size, H = c->heads;
    int eq, ek, ev;
    const long long nq = input_span(T, q_heads, D, q_token, q_head, x_dt, &eq);
    const long long nk = input_span(T, H, D, k_token, k_head, x_dt, &ek);
    const long long nv = input_span(T, H, D, v_token, v_head, x_dt, &ev);
    if (eq || ek || ev) return eq ? eq : ek ? ek : ev;
    long long size[] = {c->n_pages, c->page_size, H}, ks[] = {c->k_page, c->k_slot, c->k_head};
    long long again[] = {c->n_pages, c->page_size, H}, vs[] = {c->v_page, c->v_slot, c->v_head};
    if (!apart(size, ks, D) || !apart(again, vs, D)) return QMV_E_STRIDE;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16)) return QMV_E_ALIGN;
    const Span in[] = {{q, (size_t)nq}, {k, (size_t)nk}, {v, (size_t)nv}, weight_span(r->q_weight, D, r->w_dt),
                       weight_span(r->k_weight, D, r->w_dt), {r->freqs, (size_t)r->rot * 2}, {r->axes, (size_t)r->rot * 2},
                       {r->positions, positions_bytes(r, T)}, {c->pages, cs.pages}, {c->starts, (size_t)(c->n_seqs + 1) * 4},
                       {c->lengths, (size_t)c->n_seqs * 4}};
    // keys and values may lie between each other in one array: each is held apart from the rest
    const Span out_k[] = {{q_out, (size_t)T * q_heads * D * 2}, {c->k, cs.k}}, out_v[] = {{q_out, (size_t)T * q_heads * D * 2}, {c->v, cs.v}};
    if (!disjoint(in, out_k) || !disjoint(in, out_v) || c->k == c->v) return QMV_E_ALIAS;
    RotateParams p{};
    p.q = static_cast<const char*>(q);
    p.k = static_cast<const char*>(k);
    p.v = static_cast<const char*>(v);
    p.q_out = static_cast<char*>(q_out);
    p.q_token = q_token * (long long)size_of(x_dt);
    p.q_head = q_head * (long long)size_of(x_dt);
    p.k_token = k_token * (long long)size_of(x_dt);
    p.k_head = k_head * (long long)size_of(x_dt);
    p.v_token = v_token * (long long)size_of(x_dt);
    p.v_head = v_head * (long long)size_of(x_dt);
    p.q_heads = q_heads;
    p.k_heads = H;
    p.D = D;
    p.cache = device_cache(c, T);
    return run(p, r, T, x_dt, c->dt, true, stream);
}

}  // extern "C"
