// ops_rotate.hip -- qmv_rotate and qmv_append: norms of queries and keys for
// each head, their position rotation, and keys and values to a cache's pages.
//
// One launch and one pass.  A wave takes some heads of a token: a head of D values is held by a
// group of lanes, 16 values each (eight where sizes do not go by 16: half the bytes a load and
// store), and the groups take heads side by side, some in flight.  Where a head is rotated,
// lane i of a group holds the values 8i .. 8i + 7 of the pairs' first places and the same of their
// second ones, so that a pair is turned within a lane, whichever way pairs lie, and the lane's
// sines, cosines and weights are the same for all heads.  A lane computes one angle, for the whole wave.  The sum of squares is taken over the
// group's lanes, in fp32.  There is no barrier.
//
// Bound by memory where tokens are many: 8192 of 48 heads of 128 (201 MB read and written) 43 us, 4.7 TB/s, where a
// copy reaches 4.9 (8 values a lane instead of 16: 52 to 57); by latency where they are few: one token 4.8.
//
// Angles: positions * freqs in fp64, as turns.  1 / (2 pi) and the two products are rounded, to 2^-53 each, so an angle
// is off by up to 2^-51 of itself: below what fp32 rounds of the fraction of a turn that is left (2^-25) up to 2^26,
// 5e-7 at positions of 2^31 times a frequency of 1 (a result of fp16 near 1 is rounded by 2e-4).
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
constexpr int kWaves = kThreads / 64;
constexpr float kInfinity = __builtin_huge_valf();
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
    int parts, heads;                 // waves that share a token, and the heads of each
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

// Q: values of a lane's run in fours; two runs, of 8 Q values of a head together.  Four waves on a SIMD: with a few registers more
// than they leave, fp32 inputs have three (rotate of 8192 tokens of 40 heads 48 us for 45, append of 48 heads 57 for 54.7).
template <class X, class Y, bool APPEND, int Q>
__global__ __launch_bounds__(kThreads, 4) void rotate_kernel(RotateParams p)
{
    typedef typename Four<X>::type X4;
    typedef typename Four<Y>::type Y4;
    struct XRun {
        X4 v[Q];
    };
    struct __attribute__((aligned(8 * Q))) YRun {
        Y4 v[Q];
    };
    constexpr int kHold = 4 / Q;          // heads in flight per group of lanes
    __shared__ __align__(16) float cosines[kWaves][kMostHalf], sines[kWaves][kMostHalf];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int job = blockIdx.x * kWaves + wave, t = job / p.parts;
    if (t >= p.T) return;
    const int all = p.q_heads + (APPEND ? 2 : 1) * p.k_heads;
    const int h0 = (job - t * p.parts) * p.heads, h1 = min(all, h0 + p.heads);
    const int groups = 64 >> p.lanes_log2, group = lane >> p.lanes_log2, part = lane & ((1 << p.lanes_log2) - 1);
    const bool live = part < p.D / (8 * Q);
    // the lane's two runs
    const bool turned = part < p.half / (4 * Q);
    const int first = turned && !p.interleaved ? 4 * Q * part : 8 * Q * part;
    const int second = turned && !p.interleaved ? p.half + 4 * Q * part : 8 * Q * part + 4 * Q;

    const char* const q_at = p.q + t * p.q_token;
    const char* const k_at = p.k + t * p.k_token;
    const char* const v_at = p.v + t * p.v_token;
    const int k_from = p.q_heads, v_from = p.q_heads + p.k_heads;
    XRun a[kHold], b[kHold];
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int h = base + i * groups + group;
            if (live && h < h1) {
                const char* from = h < k_from ? q_at + h * p.q_head : k_at + (h - k_from) * p.k_head;
                if (APPEND && h >= v_from) from = v_at + (h - v_from) * p.v_head;
                a[i] = *reinterpret_cast<const XRun*>(__builtin_assume_aligned(from + first * sizeof(X), Q * 8));
                b[i] = *reinterpret_cast<const XRun*>(__builtin_assume_aligned(from + second * sizeof(X), Q * 8));
            }
        }
    };
    load(h0);

    // weights of queries and keys
    f32x4 wq[2 * Q], wk[2 * Q];
#pragma unroll
    for (int i = 0; i < 2 * Q; ++i) {
        const int at = (i < Q ? first : second) + 4 * (i % Q);
        wq[i] = wk[i] = f32x4{1, 1, 1, 1};
        if (p.q_weight && live)
            wq[i] = p.w_f32 ? *reinterpret_cast<const f32x4*>(p.q_weight + at * 4) : wide_of(*reinterpret_cast<const bf16x4*>(p.q_weight + at * 2));
        if (p.k_weight && live)
            wk[i] = p.w_f32 ? *reinterpret_cast<const f32x4*>(p.k_weight + at * 4) : wide_of(*reinterpret_cast<const bf16x4*>(p.k_weight + at * 2));
    }

    // the token's place, and where its keys and values go
    int place = 0;
    char *key_to = nullptr, *value_to = nullptr;
    if (APPEND) {
        const int seq = __builtin_amdgcn_readfirstlane(sequence_of(p.cache, t, lane));
        if (seq < 0) return;
        const Seq s = sequence(p.cache, seq);
        const int at = t - s.start;
        if (at < 0 || at >= s.count) return;
        place = s.length - s.count + at;
        if (place >= 0) {          // below max_places, as the sequence's length is
            const int index = page_index(p.cache, place), page = page_of(p.cache, seq, index);
            if (page >= 0) {
                const int slot = place - index * p.cache.page_size;
                key_to = const_cast<char*>(p.cache.k) + page * p.cache.k_page + slot * p.cache.k_slot;
                value_to = const_cast<char*>(p.cache.v) + page * p.cache.v_page + slot * p.cache.v_slot;
            }
        }
    }
    for (int j = lane; j < p.half; j += 64) {
        const int axis = p.axes ? p.axes[j] : 0;
        float s = 0.0f, c = 1.0f;
        if ((uint32_t)axis < (uint32_t)p.n_axes) {
            const int pos = p.positions ? p.positions[axis * p.positions_row + t] : place;
            const double turns = (double)pos * ((double)p.freqs[j] * 0.15915494309189533576888);
            sine_cosine(turns - __builtin_floor(turns), s, c);
        }
        cosines[wave][j] = c;
        sines[wave][j] = s;
    }
    // what a lane has put there, others of its wave read
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    f32x4 c[Q], s[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        c[i] = f32x4{1, 1, 1, 1};
        s[i] = f32x4{0, 0, 0, 0};
        if (turned) {
            c[i] = *reinterpret_cast<const f32x4*>(&cosines[wave][4 * Q * part + 4 * i]);
            s[i] = *reinterpret_cast<const f32x4*>(&sines[wave][4 * Q * part + 4 * i]);
        }
    }
    const float per = 1.0f / (float)p.D;

    for (int base = h0; base < h1; base += kHold * groups) {
        if (base > h0) load(base);
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            if (base + i * groups >= h1) break;          // the whole wave's
            const int h = base + i * groups + group;
            const bool mine = live && h < h1, key = h >= k_from, value = APPEND && h >= v_from;
            f32x4 z[2 * Q];
#pragma unroll
            for (int j = 0; j < 2 * Q; ++j) z[j] = mine ? wide_of(j < Q ? a[i].v[j] : b[i].v[j - Q]) : f32x4{0, 0, 0, 0};
            char* to;
            if (value) to = value_to ? value_to + (h - v_from) * p.cache.v_head : nullptr;
            else if (!key) to = p.q_out + ((long long)t * p.q_heads + h) * p.D * sizeof(Y);
            else if (APPEND) to = key_to ? key_to + (h - k_from) * p.cache.k_head : nullptr;
            else to = p.k_out + ((long long)t * p.k_heads + h - k_from) * p.D * sizeof(Y);
            // the norm, of a group that has any; lanes of values take part in the sum alone
            f32x4 sq = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 2 * Q; ++j) sq += z[j] * z[j];
            float sum = (sq.x + sq.y) + (sq.z + sq.w);
            for (int m = 1; m < 1 << p.lanes_log2; m <<= 1) sum += __shfl_xor(sum, m);
            if (!value && (key ? p.k_weight : p.q_weight)) {
                float mean = sum * per + p.eps;
                // Squares that are too small or too large for fp32 are taken again of a head that is moved by 2^96: x / sqrt(mean + eps) is
                // the same of s x and s^2 eps.
                if (__builtin_expect(!(mean >= 0x1p-96f && mean < kInfinity), 0)) {
                    const float move = mean < 0x1p-96f ? 0x1p96f : 0x1p-96f;
                    sum = 0.0f;
#pragma unroll
                    for (int j = 0; j < 2 * Q; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            z[j][i] *= move;
                            sum = __builtin_fmaf(z[j][i], z[j][i], sum);
                        }
                    for (int m = 1; m < 1 << p.lanes_log2; m <<= 1) sum += __shfl_xor(sum, m);
                    mean = sum * per + p.eps * move * move;
                }
                const float r = __builtin_amdgcn_rsqf(mean);
#pragma unroll
                for (int j = 0; j < 2 * Q; ++j) z[j] = z[j] * r * (key ? wk[j] : wq[j]);
            }
            if (turned && !value) {
#pragma unroll
                for (int j = 0; j < Q; ++j) {
                    if (p.interleaved) {          // pairs side by side: (x0 x1) (x2 x3) (y0 y1) (y2 y3)
                        const f32x4 x = z[2 * j], y = z[2 * j + 1], e = {x.x, x.z, y.x, y.z}, o = {x.y, x.w, y.y, y.w};
                        const f32x4 u = e * c[j] - o * s[j], w = o * c[j] + e * s[j];
                        z[2 * j] = f32x4{u.x, w.x, u.y, w.y};
                        z[2 * j + 1] = f32x4{u.z, w.z, u.w, w.w};
                    } else {
                        const f32x4 x = z[j], y = z[Q + j];
                        z[j] = x * c[j] - y * s[j];
                        z[Q + j] = y * c[j] + x * s[j];
                    }
                }
            }
            if (mine && to) {
                YRun r[2];
#pragma unroll
                for (int j = 0; j < 2 * Q; ++j) r[j / Q].v[j % Q] = __builtin_convertvector(z[j], Y4);
                *reinterpret_cast<YRun*>(to + first * sizeof(Y)) = r[0];
                *reinterpret_cast<YRun*>(to + second * sizeof(Y)) = r[1];
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

template <class X, class Y, bool APPEND>
const void* kernel_of_types(bool sixteen)
{
    return sixteen ? (const void*)&rotate_kernel<X, Y, APPEND, 2> : (const void*)&rotate_kernel<X, Y, APPEND, 1>;
}
template <bool APPEND>
const void* kernel_of(bool x_f32, bool y_f16, bool sixteen)
{
    if (x_f32) return y_f16 ? kernel_of_types<float, _Float16, APPEND>(sixteen) : kernel_of_types<float, __bf16, APPEND>(sixteen);
    return y_f16 ? kernel_of_types<__bf16, _Float16, APPEND>(sixteen) : kernel_of_types<__bf16, __bf16, APPEND>(sixteen);
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
    const bool sixteen = p.D % 16 == 0 && p.half % 8 == 0;
    const int lanes = p.D / (sixteen ? 16 : 8);
    p.lanes_log2 = 0;
    while (1 << p.lanes_log2 < lanes) ++p.lanes_log2;
    // A wave takes one round of heads, or as many more as leave 4096 waves (four for every SIMD): angles and
    // places then serve several heads, and a token's memory is one wave's.  48 heads of 128, us, by rounds of 8:
    // 256 tokens 5.5 with one, 6.4 with two, 10.1 with all; 1024: 12.5, 10.0, 12.8; 2048: 19.1, 16.4, 14.0 with
    // three, 15.3; 8192: 71, 57, 50, 43.
    const int all = p.q_heads + (append ? 2 : 1) * p.k_heads, groups = 64 >> p.lanes_log2;
    p.heads = groups;
    while (p.heads < all && (long long)T * ((all + p.heads - 1) / p.heads) > 4096) p.heads += groups;
    p.heads = std::min(all, p.heads);
    p.parts = (all + p.heads - 1) / p.heads;
    const bool xf = x_dt == QMV_DT_F32, yh = y_dt == QMV_DT_F16;
    const void* f = append ? kernel_of<true>(xf, yh, sixteen) : kernel_of<false>(xf, yh, sixteen);
    void* args[] = {&p};
    const dim3 grid((unsigned)(((long long)T * p.parts + kWaves - 1) / kWaves));
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
