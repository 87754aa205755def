// ops_verify.hip -- qmv_verify: drafted tokens accepted or replaced by the
// target's probabilities and given random numbers.
//
// Two launches.  The first passes over all logits once; every wave takes a span
// of a row: the largest value and the sum of exp((l - largest) / T).  In the
// second, every workgroup of a request joins those of its rows, makes the same
// accept decisions, and adds up the weights of its chunk of the one row that is
// sampled; the last to finish turns the chunks' sums into the token.  Bound by
// the read of the logits where there are many, by the chain of dependent loads
// of the second launch where there are few.  One request of 5 rows of 131072: 3.6 and
// 11.4 us.  32 requests of 8 rows of 131072 in bf16: 15.2 us, 67 MB at 4.4 TB/s, nearly a
// large copy's rate, and 21.6.
//
// Precision.  An accept decision compares one number with one border.  The first
// pass takes fp32 exponentials, which is what lets it keep up with the read, and
// its sums are off by less than 2^-19: that decides all but one number in 2^18, and
// for that the row is summed in fp64.  A sampled token is where a prefix sum
// of up to 2^17 and more terms first passes a number: with fp32 exponentials
// every one of those borders moves, and over a vocabulary about one request in a
// thousand would get a neighbour of the token that the definition gives.  So the
// sampled row is summed again, in fp64.  Its total Z is known only when all of its
// chunks are summed, but the weights max(e_i - q_i Z, 0) are needed with it: each
// chunk adds up e_i and q_i where e_i > q_i Z0 for the first pass's Z0, and their
// sums give those of the weights for the true Z, up to the values so near the
// border that Z and Z0 disagree about them; where those could matter (a drafter whose
// probabilities are the target's, u = 0) the sums are taken once more, by the last
// workgroup alone: 1.6 us for every 2048 values, 115 us for a row of 131072 in place of 13.5.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ops_args.hpp"
#include "ops_check.hpp"

namespace ops {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef u32x4 __attribute__((aligned(2))) u32x4_any;      // rows may start anywhere

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kSpanPer = 32;                  // first launch: values per lane
constexpr int kSpan = 64 * kSpanPer;          // and per wave
constexpr int kPer = 8;                       // second launch: values per thread
constexpr int kChunk = kThreads * kPer;       // and per workgroup
constexpr float kNone = -__builtin_huge_valf();
constexpr int kNoIndex = 0x7fffffff;

struct Stat {          // of a wave's stretch of a row
    double sum;        // of exp((l - top) / T)
    float top;         // the largest value, -inf if none counts
    int at;            // greedy: its first index
};

struct Part {          // of a chunk of the sampled row
    double p;          // sum of e
    double e, q;       // sums of e and q over the values with e > q Z0
    double near;       // sum of e over those too near to say
};

struct VerifyParams {
    const char* logits;
    const int32_t* draft;
    const float* u;
    const char* probs;
    const float* temperature;
    const int32_t* lengths;
    int32_t* tokens;
    int32_t* accepted;
    Stat* stats;       // [B][S + 1][stretches]
    Part* part;        // [B][chunks]
    uint32_t* tickets; // [B]
    int B, S, V, chunks;
    int walk, stretches; // first launch: spans per wave, waves per row
    int groups;          // second launch: workgroups per request
    long long l_batch, l_row, q_batch, q_row;
};

__device__ __forceinline__ float bits_f32(uint32_t u) { return __builtin_bit_cast(float, u); }

template <bool F32>
__device__ __forceinline__ float load1(const char* row, long long i)
{
    if constexpr (F32) return reinterpret_cast<const float*>(row)[i];
    return bits_f32((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
}

// the values of one 16-byte piece
template <bool F32>
__device__ __forceinline__ void unpack(float* o, const u32x4& w)
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        if constexpr (F32) {
            o[d] = bits_f32(w[d]);
        } else {
            o[2 * d] = bits_f32(w[d] << 16);
            o[2 * d + 1] = bits_f32(w[d] & 0xffff0000u);
        }
    }
}

// NV 16-byte pieces of a row, piece v from i + v * step on; `none` past its end
template <bool F32, int NV>
__device__ __forceinline__ void load_raw(u32x4 (&w)[NV], const char* row, long long i, int step, int V, float none)
{
    constexpr int SZ = F32 ? 4 : 2, PER = 16 / SZ;
    if (i + (NV - 1) * step + PER <= V) {
#pragma unroll
        for (int v = 0; v < NV; ++v) w[v] = *reinterpret_cast<const u32x4_any*>(row + (i + v * step) * SZ);
        return;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const long long at = i + v * step + d * (PER / 4);
            const uint32_t a = __builtin_bit_cast(uint32_t, at < V ? load1<F32>(row, at) : none);
            if constexpr (F32) {
                w[v][d] = a;
            } else {
                const uint32_t b = __builtin_bit_cast(uint32_t, at + 1 < V ? load1<F32>(row, at + 1) : none);
                w[v][d] = (a >> 16) | (b & 0xffff0000u);
            }
        }
}

template <bool F32, int N>
__device__ __forceinline__ void load_row(float (&o)[N], const char* row, long long i, int step, int V, float none)
{
    constexpr int PER = F32 ? 4 : 8;
    u32x4 w[N / PER];
    load_raw<F32>(w, row, i, step, V, none);
#pragma unroll
    for (int v = 0; v < N / PER; ++v) unpack<F32>(o + v * PER, w[v]);
}

__device__ __forceinline__ float no_nan(float v) { return v != v ? kNone : v; }

// Reductions over a wave in one fixed order, the result in every lane: pairs and
// quads by dpp, halves of a row by its mirrors, rows by swaps.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}

template <class Op>
__device__ __forceinline__ uint32_t wave_fold(uint32_t v, Op op)
{
    v = op(v, dpp<0xB1>(v));
    v = op(v, dpp<0x4E>(v));
    v = op(v, dpp<0x141>(v));
    v = op(v, dpp<0x140>(v));
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return op(b[0], b[1]);
}

__device__ __forceinline__ float wave_max(float v)
{
    return bits_f32(wave_fold(__builtin_bit_cast(uint32_t, v), [](uint32_t a, uint32_t b) {
        return __builtin_bit_cast(uint32_t, __builtin_fmaxf(bits_f32(a), bits_f32(b)));
    }));
}

__device__ __forceinline__ int wave_min(int v)
{
    return (int)wave_fold((uint32_t)v, [](uint32_t a, uint32_t b) { return (uint32_t)min((int)a, (int)b); });
}

__device__ __forceinline__ double two(uint32_t lo, uint32_t hi)
{
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

template <int CTRL>
__device__ __forceinline__ double dpp(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return two(dpp<CTRL>((uint32_t)u), dpp<CTRL>((uint32_t)(u >> 32)));
}

__device__ __forceinline__ double wave_sum(double v)
{
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    uint64_t u = __builtin_bit_cast(uint64_t, v);
    const auto al = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
    const auto ah = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
    v = two(al[0], ah[0]) + two(al[1], ah[1]);
    u = __builtin_bit_cast(uint64_t, v);
    const auto bl = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
    const auto bh = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
    return two(bl[0], bh[0]) + two(bl[1], bh[1]);
}

// 2^t for t <= 0: 2^n by the exponent, 2^f for |f| <= 1/2 by the series of
// exp(f ln 2) up to the tenth power (2e-13 of the value); 0 below 2^-1000.
__device__ __forceinline__ double exp2_down(double t)
{
    if (!(t > -1000.0)) return 0.0;
    const double n = __builtin_rint(t), x = (t - n) * 0.69314718055994530942;
    double p = 1.0 / 3628800;
    p = __builtin_fma(p, x, 1.0 / 362880);
    p = __builtin_fma(p, x, 1.0 / 40320);
    p = __builtin_fma(p, x, 1.0 / 5040);
    p = __builtin_fma(p, x, 1.0 / 720);
    p = __builtin_fma(p, x, 1.0 / 120);
    p = __builtin_fma(p, x, 1.0 / 24);
    p = __builtin_fma(p, x, 1.0 / 6);
    p = __builtin_fma(p, x, 0.5);
    p = __builtin_fma(p, x, 1.0);
    p = __builtin_fma(p, x, 1.0);
    return __builtin_ldexp(p, (int)n);
}

// exp((l - top) / T), rate = log2(e) / T: 1 at the top (an infinite one too), 0 at -inf and NaN
__device__ __forceinline__ double weight(float l, float top, double rate)
{
    if (!(l > kNone)) return 0.0;
    return l == top ? 1.0 : exp2_down(((double)l - (double)top) * rate);
}

__device__ __forceinline__ double rate_of(float t) { return 1.4426950408889634074 / (double)t; }

__device__ __forceinline__ int length_of(const VerifyParams& p, int b)
{
    return p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S;
}

// A wave walks p.walk spans of one row, the next one's loads in flight.
//
// A lane takes e = 2^t, t = (l - largest) * hi, in fp32: hi is log2(e) / T rounded
// and `largest` the lane's own so far.  The two roundings of t are relative to t, so
// they matter as little for values of 1e10 (a mask, a temperature near zero) as for
// ones of 10, and t is 0 at the largest and never above.  (As l * hi - largest * hi
// it would be off by an ulp of largest * hi, and e infinite where that passes 128.)
// The rest of the rate would shift all terms one way; to first order it adds ln 2 *
// (rate / hi - 1) * sum(e t).  Whatever is below 2^-200 of the largest, masks among
// it, is 0 there, and finite: no term of a sum is infinite or NaN.
//
// How far a lane's sum of at most 256 values can be off, in units of 2^-20 of it: 0.42 for
// t's roundings (2^-23 |t| ln 2 of a term, and the terms' mean |t| is 4.8 at most), 0.67 for
// chains of 64 additions, 0.3 for the factors between spans, 0.13 for the exponentials.
// (Observed: 0.2.)
template <bool LF32>
__global__ __launch_bounds__(kThreads) void stats_kernel(VerifyParams p)
{
    constexpr int PER = LF32 ? 4 : 8, NV = kSpanPer / PER, SZ = LF32 ? 4 : 2;
    together(p.logits, p.temperature, p.lengths, p.stats, p.tickets, p.S, p.V, p.walk, p.stretches, p.l_batch, p.l_row);
    const int lane = threadIdx.x & 63, at_row = blockIdx.x * kWaves + (threadIdx.x >> 6);
    const int b = blockIdx.z, j = blockIdx.y, row = b * (p.S + 1) + j;
    if (j == 0 && at_row == 0 && lane == 0) p.tickets[b] = 0;
    if (at_row >= p.stretches || j > length_of(p, b)) return;
    const float T = p.temperature ? p.temperature[b] : 1.0f;
    const char* l = p.logits + (b * p.l_batch + j * p.l_row) * SZ;
    const int spans = min(p.walk, (p.V + kSpan - 1) / kSpan - at_row * p.walk);
    const long long i0 = (long long)at_row * p.walk * kSpan + lane * PER;
    float top = kNone;
    int at = kNoIndex;
    double sum = 0.0;
    u32x4 w[NV], next[NV];
    float v[kSpanPer];
    constexpr double kLn2 = 0.69314718055994530942;
    constexpr float kLeast = -200.0f;             // of a term's exponent: 0 in fp32
    bool strange = !(T < 1e18f) || T <= 1e-18f;
    if (T > 0.0f && !strange) {
        const double rate = rate_of(T);
        const float hi = (float)rate;
        load_raw<LF32>(next, l, i0, 64 * PER, p.V, kNone);
        float mine = -1e18f, s[4] = {0.f, 0.f, 0.f, 0.f}, c[4] = {0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < spans; ++i) {
#pragma unroll
            for (int d = 0; d < NV; ++d) w[d] = next[d];
            if (i + 1 < spans) load_raw<LF32>(next, l, i0 + (long long)(i + 1) * kSpan, 64 * PER, p.V, kNone);
#pragma unroll
            for (int d = 0; d < NV; ++d) unpack<LF32>(v + d * PER, w[d]);
            // a maximum passes quiet NaNs over, and would take a signalling one for its result
            const float old = mine;
            float t4[4] = {mine, mine, mine, mine};
#pragma unroll
            for (int d = 0; d < kSpanPer; d += 2) {
                float& t = t4[(d >> 1) & 3];
                t = __builtin_fmaxf(__builtin_fmaxf(t, __builtin_canonicalizef(v[d])), __builtin_canonicalizef(v[d + 1]));
            }
            mine = __builtin_fmaxf(__builtin_fmaxf(t4[0], t4[1]), __builtin_fmaxf(t4[2], t4[3]));
            if (i > 0) {
                const float up = __builtin_fmaxf((old - mine) * hi, kLeast), f = __builtin_amdgcn_exp2f(up);
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    c[d] = f * __builtin_fmaf(up, s[d], c[d]);
                    s[d] *= f;
                }
            }
#pragma unroll
            for (int d = 0; d < kSpanPer; ++d) {
                const float t = __builtin_fmaxf((v[d] - mine) * hi, kLeast);      // masked and NaN too
                const float e = __builtin_amdgcn_exp2f(t);
                s[d & 3] += e;
                c[d & 3] = __builtin_fmaf(e, t, c[d & 3]);
            }
        }
        top = wave_max(mine);
        strange = !(__builtin_fabsf(top) < 1e18f);
        if (!strange) {
            const double sa = (double)((s[0] + s[1]) + (s[2] + s[3])), ca = (double)((c[0] + c[1]) + (c[2] + c[3]));
            const double all = sa + kLn2 * (rate / (double)hi - 1.0) * ca;
            const double t = ((double)mine - (double)top) * rate;                  // from the lane's largest to the wave's
            const float near = __builtin_fmaxf((float)t, kLeast), e = __builtin_amdgcn_exp2f(near);
            sum = wave_sum(all * ((double)e + kLn2 * (double)e * __builtin_fmax(t - (double)near, -1.0)));
        }
    }
    if (strange || !(T > 0.0f)) {
        // greedy requests, and what the arithmetic above has no range for
        float mine = kNone;
        for (int i = 0; i < spans; ++i) {
            load_row<LF32>(v, l, i0 + (long long)i * kSpan, 64 * PER, p.V, kNone);
#pragma unroll
            for (int d = 0; d < kSpanPer; ++d)
                if (v[d] > mine) {
                    mine = v[d];
                    at = (int)i0 + i * kSpan + (d / PER) * 64 * PER + d % PER;
                }
        }
        top = wave_max(mine);
        at = wave_min(mine == top ? at : kNoIndex);
        if (T > 0.0f && top > kNone) {
            const double rate = rate_of(T);
            sum = 0.0;
            for (int i = 0; i < spans; ++i) {
                load_row<LF32>(v, l, i0 + (long long)i * kSpan, 64 * PER, p.V, kNone);
#pragma unroll
                for (int d = 0; d < kSpanPer; ++d) sum += weight(v[d], top, rate);
            }
            sum = wave_sum(sum);
        }
    }
    if (lane == 0) p.stats[(size_t)row * p.stretches + at_row] = Stat{sum, top, at};
}

// Sums of the lanes up to each, by dpp: within rows of 16, then from row to row.
template <int CTRL, int ROWS>
__device__ __forceinline__ double add_dpp(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xf, false);
    return v + two(lo, hi);
}

__device__ __forceinline__ double wave_scan(double v)
{
    v = add_dpp<0x111, 0xf>(v);      // from 1, 2, 4 and 8 lanes below, zero from outside the row
    v = add_dpp<0x112, 0xf>(v);
    v = add_dpp<0x114, 0xf>(v);
    v = add_dpp<0x118, 0xf>(v);
    v = add_dpp<0x142, 0xa>(v);      // lane 15 of the row below to rows 1 and 3
    return add_dpp<0x143, 0xc>(v);   // lane 31 to rows 2 and 3
}

// The LDS of one choice among what all threads hold.
struct PickSpace {
    double sums[kWaves];
    double before[kWaves][2];
    int index[kWaves][2];
};

// Every thread holds the values get(i), i0 <= i < i1, in the threads' order, and
// their sum: the lowest index whose prefix sum passes target(total), or the highest of a
// positive value if none does (-1 if there is no such value), and the sum before it.
struct Pick {
    int index;
    double before;
};

template <class Get, class Target>
__device__ __forceinline__ Pick block_pick(PickSpace& sp, int i0, int i1, double sum, Get get, Target target)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double to = wave_scan(sum);
    if (lane == 63) sp.sums[wave] = to;
    __syncthreads();
    double total = 0.0, below = 0.0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) below = total;
        total += sp.sums[w];
    }
    const double t = target(total);
    to += below;
    // Of a thread's positive values only: the target may be below zero, by the rounding of a border
    // that it lies on, and then every thread's sum is past it.
    const unsigned long long some = __ballot(sum > 0.0), over = __ballot(to > t) & some;
    if (lane < 2) sp.index[wave][lane] = -1;
    // the first thread past the number, and the last with anything, look through their values
    const bool first = over != 0 && lane == __builtin_ctzll(over), last = some != 0 && lane == 63 - __builtin_clzll(some);
    if (first || last) {
        double c = to - sum;
        Pick found{-1, 0.0}, end{-1, 0.0};
        for (int i = i0; i < i1; ++i) {
            const double v = get(i);
            if (v > 0.0) {
                end = Pick{i, c};
                if (found.index < 0 && c + v > t) found = end;
            }
            c += v;
        }
        if (found.index < 0) found = end;        // the sums were rounded otherwise
        if (first) {
            sp.index[wave][0] = found.index;
            sp.before[wave][0] = found.before;
        }
        if (last) {
            sp.index[wave][1] = end.index;
            sp.before[wave][1] = end.before;
        }
    }
    __syncthreads();
    Pick r{-1, 0.0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        if (sp.index[w][1] >= 0) r = Pick{sp.index[w][1], sp.before[w][1]};
#pragma unroll
    for (int w = kWaves - 1; w >= 0; --w)
        if (sp.index[w][0] >= 0) r = Pick{sp.index[w][0], sp.before[w][0]};
    return r;
}

__device__ __forceinline__ void put(double* p, double v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ double get(const double* p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <bool LF32, bool QF32>
__global__ __launch_bounds__(kThreads) void sample_kernel(VerifyParams p)
{
    constexpr int kMaxRows = QMV_MAX_DRAFT + 1, LSZ = LF32 ? 4 : 2, QSZ = QF32 ? 4 : 2;
    static_assert(QMV_MAX_DRAFT < kThreads, "a thread per position");
    __shared__ float tops[kMaxRows];
    __shared__ int ats[kMaxRows];
    __shared__ double sums[kMaxRows];
    __shared__ double space[2][4][kWaves];
    __shared__ PickSpace picks[2];
    __shared__ int first_bad, first_close;
    __shared__ bool am_last;
    together(p.logits, p.draft, p.u, p.probs, p.temperature, p.lengths, p.stats, p.part, p.tickets, p.S, p.V, p.chunks, p.stretches,
             p.groups, p.l_batch, p.l_row, p.q_batch, p.q_row);
    const int chunk = blockIdx.x, b = blockIdx.y, len = length_of(p, b), tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const float T = p.temperature ? p.temperature[b] : 1.0f;
    const bool greedy = !(T > 0.0f);
    const double rate = greedy ? 0.0 : rate_of(T);
    const char* lb = p.logits + b * p.l_batch * LSZ;
    const char* qb = p.probs ? p.probs + b * p.q_batch * QSZ : nullptr;
    const float* ub = p.u + (size_t)b * (p.S + 1);

    // what the decisions need, on its way while the rows' statistics are joined
    const float u_last = ub[len];
    int x = -1;
    float u_at = 0.0f, l_at = kNone, q_at = 1.0f;
    if (tid < p.S) {           // positions past the length are read, not used
        x = p.draft[(size_t)b * p.S + tid];
        u_at = ub[tid];
        if (x >= 0 && x < p.V) {
            l_at = no_nan(load1<LF32>(lb + (size_t)tid * p.l_row * LSZ, x));
            if (qb) q_at = load1<QF32>(qb + (size_t)tid * p.q_row * QSZ, x);
        }
    }
    if (tid == 0) {
        first_bad = len;
        first_close = kNoIndex;
    }
    const Stat* sb = p.stats + (size_t)b * (p.S + 1) * p.stretches;
    for (int j0 = wave; j0 <= len; j0 += 4 * kWaves) {
        Stat st[4];                                  // four rows' first spans at once
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + i * kWaves;
            st[i] = Stat{0.0, kNone, kNoIndex};
            if (j <= p.S && lane < p.stretches) st[i] = sb[(size_t)j * p.stretches + lane];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = j0 + i * kWaves;
            if (j > len) break;
            const Stat* row = sb + (size_t)j * p.stretches;
            float top = st[i].top;
            for (int c = lane + 64; c < p.stretches; c += 64) top = __builtin_fmaxf(top, row[c].top);
            top = wave_max(top);
            if (greedy) {
                int at = st[i].top == top ? st[i].at : kNoIndex;
                for (int c = lane + 64; c < p.stretches; c += 64)
                    if (row[c].top == top) at = min(at, row[c].at);
                at = wave_min(at);
                if (lane == 0) ats[j] = at;
            } else {
                double s = st[i].sum * weight(st[i].top, top, rate);
                for (int c = lane + 64; c < p.stretches; c += 64) s += row[c].sum * weight(row[c].top, top, rate);
                s = wave_sum(s);
                if (lane == 0) sums[j] = s;
            }
            if (lane == 0) tops[j] = top;
        }
    }
    __syncthreads();
    // The first position that is not accepted.  One that is too close to call by the first pass's
    // sum has its row summed in fp64 before it is called (one in 2^18; 64 chunks of 2048 values
    // take 60 us).
    bool called = false;
    int n;
    for (;;) {
        if (tid < len) {
            bool yes = false, close = false;
            if (x >= 0 && x < p.V) {
                const double uq = (double)u_at * (double)q_at;
                if (greedy) {
                    yes = x == ats[tid] && uq < 1.0;
                } else if (l_at > kNone) {
                    const double e = weight(l_at, tops[tid], rate), off = uq * sums[tid] - e;
                    yes = off < 0.0;
                    close = !called && __builtin_fabs(off) < 0x1p-19 * e;
                }
            }
            if (!yes) atomicMin(&first_bad, tid);
            if (close) atomicMin(&first_close, tid);
        }
        __syncthreads();
        const int j = first_close;
        n = first_bad;
        if (j > n) break;
        double s = 0.0;
        for (int c = 0; c < p.chunks; ++c) {
            float v[kPer];
            load_row<LF32>(v, lb + (size_t)j * p.l_row * LSZ, (long long)c * kChunk + tid * kPer, 16 / LSZ, p.V, kNone);
#pragma unroll
            for (int i = 0; i < kPer; ++i) s += weight(v[i], tops[j], rate);
        }
        s = wave_sum(s);
        if (lane == 0) space[0][0][wave] = s;
        __syncthreads();
        if (tid == j) {
            sums[j] = ((space[0][0][0] + space[0][0][1]) + space[0][0][2]) + space[0][0][3];
            called = true;
        }
        if (tid == 0) {
            first_bad = len;
            first_close = kNoIndex;
        }
        __syncthreads();
    }
    const float top = tops[n];
    const bool sampled = !greedy && top > kNone, rest = sampled && n < len;
    if (!sampled && chunk != 0) return;

    int token = -1;
    if (greedy) {
        token = ats[n] == kNoIndex ? -1 : ats[n];
    } else if (sampled) {
        const double Z0 = sums[n];
        const char* ln = lb + (size_t)n * p.l_row * LSZ;
        const char* qn = rest && qb ? qb + (size_t)n * p.q_row * QSZ : nullptr;
        const int xn = rest ? p.draft[(size_t)b * p.S + n] : -1;
        double e[kPer], q[kPer];
        auto load_chunk = [&](int c) {
            const long long i0 = (long long)c * kChunk + tid * kPer;
            float lf[kPer], qf[kPer];
            load_row<LF32>(lf, ln, i0, 16 / LSZ, p.V, kNone);
            if (qn) load_row<QF32>(qf, qn, i0, 16 / QSZ, p.V, 0.0f);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                e[i] = weight(lf[i], top, rate);
                q[i] = qn ? (double)qf[i] : i0 + i == xn ? 1.0 : 0.0;
            }
        };
        Part* parts = p.part + (size_t)b * p.chunks;
        for (int c = chunk; c < p.chunks; c += p.groups) {
            load_chunk(c);
            Part mine{0.0, 0.0, 0.0, 0.0};
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                mine.p += e[i];
                const double d = __builtin_fma(-q[i], Z0, e[i]);
                if (d > 0.0) {
                    mine.e += e[i];
                    mine.q += q[i];
                }
                if (__builtin_fabs(d) <= 0x1p-19 * e[i]) mine.near += e[i];
            }
            mine.p = wave_sum(mine.p);
            if (rest) {
                mine.e = wave_sum(mine.e);
                mine.q = wave_sum(mine.q);
                mine.near = wave_sum(mine.near);
            }
            __syncthreads();
            if (lane == 0) {
                space[0][0][wave] = mine.p;
                space[0][1][wave] = mine.e;
                space[0][2][wave] = mine.q;
                space[0][3][wave] = mine.near;
            }
            __syncthreads();
            if (tid < 4) {
                double s = space[0][tid][0];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) s += space[0][tid][w];
                put(reinterpret_cast<double*>(parts + c) + tid, s);
            }
        }
        // The parts are written through by the first wave and read past the
        // caches, so its count after they have arrived orders them; a release of
        // the whole cache (about 40 us with 2048 workgroups) is not needed.
        if (tid == 0) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            am_last = __hip_atomic_fetch_add(&p.tickets[b], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)p.groups - 1;
        }
        __syncthreads();
        if (!am_last) return;

        // The totals, then the chunk in which the prefix sum passes the number:
        // every thread holds some neighbouring chunks, the first of them in registers.
        const int per = (p.chunks + kThreads - 1) / kThreads, c0 = min(tid * per, p.chunks), c1 = min(c0 + per, p.chunks);
        auto part = [&](int c) { return Part{get(&parts[c].p), get(&parts[c].e), get(&parts[c].q), get(&parts[c].near)}; };
        Part first{0.0, 0.0, 0.0, 0.0};
        if (c0 < c1) first = part(c0);
        Part t = first;
        for (int c = c0 + 1; c < c1; ++c) {
            const Part x = part(c);
            t.p += x.p;
            t.e += x.e;
            t.q += x.q;
            t.near += x.near;
        }
        // sums over the workgroup of four numbers at once
        auto all_of = [&](Part v) {
            v = Part{wave_sum(v.p), wave_sum(v.e), wave_sum(v.q), wave_sum(v.near)};
            if (lane == 0) {
                space[1][0][wave] = v.p;
                space[1][1][wave] = v.e;
                space[1][2][wave] = v.q;
                space[1][3][wave] = v.near;
            }
            __syncthreads();
            double r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                r[k] = space[1][k][0];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) r[k] += space[1][k][w];
            }
            return Part{r[0], r[1], r[2], r[3]};
        };
        t = all_of(t);
        const double Z = t.p, left = t.e - Z * t.q;
        bool use = rest && left > 0.0;
        // the border's values could move the sums by 2^-32 of them, or are all that is left before a number this small
        if (rest && (t.near * 0x1p13 > left || t.near > (double)u_last * left)) {
            double all = 0.0;
            for (int c = 0; c < p.chunks; ++c) {
                load_chunk(c);
                double s = 0.0;
#pragma unroll
                for (int i = 0; i < kPer; ++i) s += __builtin_fmax(__builtin_fma(-q[i], Z, e[i]), 0.0);
                __syncthreads();
                s = all_of(Part{s, 0.0, 0.0, 0.0}).p;
                all += s;
                if (tid == 0) {
                    put(&parts[c].e, s);
                    put(&parts[c].q, 0.0);
                }
            }
            use = all > 0.0;
            __threadfence();
            __syncthreads();
            if (c0 < c1) first = part(c0);
        }
        // nothing left: sampled from the target itself
        auto weight_of = [&](int c) {
            const Part x = c == c0 ? first : part(c);
            return use ? __builtin_fmax(x.e - Z * x.q, 0.0) : x.p;
        };
        double s = 0.0, aim = 0.0;
        for (int c = c0; c < c1; ++c) s += weight_of(c);
        const Pick k = block_pick(picks[0], c0, c1, s, weight_of, [&](double total) { return aim = (double)u_last * total; });
        if (k.index >= 0) {
            load_chunk(k.index);
            double w[kPer], sum = 0.0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                w[i] = use ? __builtin_fmax(__builtin_fma(-q[i], Z, e[i]), 0.0) : e[i];
                sum += w[i];
            }
            const double rest_of_aim = aim - k.before;
            const Pick i = block_pick(picks[1], tid * kPer, tid * kPer + kPer, sum, [&](int i) {
                double v = w[0];
#pragma unroll
                for (int j = 1; j < kPer; ++j) v = i - tid * kPer == j ? w[j] : v;
                return v;
            }, [&](double) { return rest_of_aim; });
            token = i.index < 0 ? -1 : k.index * kChunk + i.index;
        }
    }
    for (int j = tid; j <= p.S; j += kThreads)
        p.tokens[(size_t)b * (p.S + 1) + j] = j < n ? p.draft[(size_t)b * p.S + j] : j == n ? token : -1;
    if (tid == 0) p.accepted[b] = n;
}

int spans_of(int V) { return (V + kSpan - 1) / kSpan; }

// Spans per wave of the first launch: one while that leaves up to 16 waves for
// every compute unit, then more, which spreads a wave's joins over more values.
int walk_of(int B, int S, int V) { return std::min(8, std::max(1, (int)((long long)B * (S + 1) * spans_of(V) / 4096))); }
int chunks_of(int V) { return (V + kChunk - 1) / kChunk; }

bool verify_sizes(int B, int S, int V)
{
    return B >= 1 && B <= QMV_MAX_BATCH && S >= 0 && S <= QMV_MAX_DRAFT && V >= 1 && V <= QMV_MAX_VOCAB;
}

}  // namespace
}  // namespace ops

extern "C" {

long long qmv_verify_workspace(int B, int S, int V)
{
    using namespace ops;
    if (!verify_sizes(B, S, V)) return -1;
    return piece((long long)sizeof(Stat) * B * (S + 1) * spans_of(V)) + piece((long long)sizeof(Part) * B * chunks_of(V)) +
           piece(4LL * B);
}

int qmv_verify(const void* logits, const int32_t* draft, const float* uniforms, const void* probs,
               const float* temperature, const int32_t* lengths, int32_t* tokens,
               int32_t* accepted, void* workspace, long long workspace_bytes, int B, int S, int V,
               long long l_batch, long long l_row, long long q_batch, long long q_row, int l_dt,
               int q_dt, void* stream)
{
    using namespace ops;
    if (!logits || !uniforms || !tokens || !accepted || !workspace || (S > 0 && !draft)) return QMV_E_NULL;
    if (!verify_sizes(B, S, V)) return QMV_E_VOCAB;
    if (S == 0) probs = nullptr;
    if (!wide(l_dt) || (probs && !wide(q_dt))) return QMV_E_DTYPE;
    // rows may lie in any order and share memory: they are read only
    constexpr long long kMost = 1LL << 40;
    if (l_row < 0 || l_batch < 0 || l_row > kMost || l_batch > kMost) return QMV_E_STRIDE;
    if (probs && (q_row < 0 || q_batch < 0 || q_row > kMost || q_batch > kMost)) return QMV_E_STRIDE;
    if (!aligned(logits, size_of(l_dt)) || (probs && !aligned(probs, size_of(q_dt))) || !aligned(draft, 4) ||
        !aligned(uniforms, 4) || !aligned(temperature, 4) || !aligned(lengths, 4) || !aligned(tokens, 4) ||
        !aligned(accepted, 4) || !aligned(workspace, 16))
        return QMV_E_ALIGN;
    const long long need = qmv_verify_workspace(B, S, V);
    if (workspace_bytes < need) return QMV_E_WORKSPACE;
    const size_t nl = (size_t)((B - 1) * l_batch + S * l_row + V) * size_of(l_dt);
    const size_t nq = probs ? (size_t)((B - 1) * q_batch + (S - 1) * q_row + V) * size_of(q_dt) : 0;
    const Span in[] = {{logits, nl}, {draft, (size_t)B * S * 4}, {uniforms, (size_t)B * (S + 1) * 4}, {probs, nq},
                       {temperature, (size_t)B * 4}, {lengths, (size_t)B * 4}};
    const Span out[] = {{tokens, (size_t)B * (S + 1) * 4}, {accepted, (size_t)B * 4}, {workspace, (size_t)need}};
    if (!disjoint(in, out)) return QMV_E_ALIAS;

    VerifyParams p;
    p.logits = static_cast<const char*>(logits);
    p.draft = draft;
    p.u = uniforms;
    p.probs = static_cast<const char*>(probs);
    p.temperature = temperature;
    p.lengths = lengths;
    p.tokens = tokens;
    p.accepted = accepted;
    p.B = B;
    p.S = S;
    p.V = V;
    p.walk = walk_of(B, S, V);
    p.stretches = (spans_of(V) + p.walk - 1) / p.walk;
    p.chunks = chunks_of(V);
    char* ws = static_cast<char*>(workspace);
    p.stats = reinterpret_cast<Stat*>(ws);
    ws += piece((long long)sizeof(Stat) * B * (S + 1) * spans_of(V));
    p.part = reinterpret_cast<Part*>(ws);
    ws += piece((long long)sizeof(Part) * B * p.chunks);
    p.tickets = reinterpret_cast<uint32_t*>(ws);
    p.l_batch = l_batch;
    p.l_row = l_row;
    p.q_batch = q_batch;
    p.q_row = q_row;
    const bool lf = l_dt == QMV_DT_F32, qf = probs && q_dt == QMV_DT_F32;
    const void* f1 = lf ? (const void*)&stats_kernel<true> : (const void*)&stats_kernel<false>;
    const void* f2 = lf ? (qf ? (const void*)&sample_kernel<true, true> : (const void*)&sample_kernel<true, false>)
                        : (qf ? (const void*)&sample_kernel<false, true> : (const void*)&sample_kernel<false, false>);
    void* args[] = {&p};
    hipStream_t st = static_cast<hipStream_t>(stream);
    // Workgroups per request of the second launch: each repeats the decisions, so
    // no more than are resident at once.
    p.groups = std::min(p.chunks, std::max(1, 1024 / B));
    if (hipLaunchKernel(f1, dim3((p.stretches + kWaves - 1) / kWaves, S + 1, B), dim3(kThreads), args, 0, st) != hipSuccess ||
        hipLaunchKernel(f2, dim3(p.groups, B), dim3(kThreads), args, 0, st) != hipSuccess)
        return QMV_E_LAUNCH;
    return QMV_OK;
}

}  // extern "C"
