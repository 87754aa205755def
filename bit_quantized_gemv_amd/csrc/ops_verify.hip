// ops_verify.hip -- qmv_verify: drafted tokens accepted or replaced by the
// target's probabilities and given random numbers.
//
// Two launches.  The first passes over all logits once, in chunks of a row: the
// largest value, its first index, and the sum of exp((l - largest) / T).  In the
// second, every workgroup of a request joins those of its rows, makes the same
// accept decisions, and adds up the weights of its chunk of the one row that is
// sampled; the last to finish turns the chunks' sums into the token.  Bound by
// the read of the logits.
//
// fp64 throughout.  A token is chosen where a prefix sum of up to 2^17 and more
// terms first passes a random number; with fp32 exponentials every one of those
// borders moves by 2^-24 of its term, and over a vocabulary about one request
// in a thousand would get a neighbour of the token that the definition gives.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ops_check.hpp"

namespace ops {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef u32x4 __attribute__((aligned(2))) u32x4_any;      // rows may start anywhere

constexpr int kThreads = 256;
constexpr int kPer = 16;                      // values per thread and chunk
constexpr int kChunk = kThreads * kPer;

struct Stat {          // of a chunk of a row
    double sum;        // of exp((l - top) / T)
    float top;         // the largest value, -inf if none counts
    int at;            // its first index
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
    Stat* stats;       // [B][S + 1][chunks]
    double* part;      // [B][chunks]
    uint32_t* tickets; // [B]
    int B, S, V, chunks;
    long long l_batch, l_row, q_batch, q_row;
};

__device__ __forceinline__ float bits_f32(uint32_t u) { return __builtin_bit_cast(float, u); }

// sixteen values of a row from i on; -inf (or zero) past its end
template <bool F32>
__device__ __forceinline__ void load16(float (&o)[kPer], const char* row, long long i, int V, float none)
{
    constexpr int SZ = F32 ? 4 : 2;
    if (i + kPer <= V) {
        const u32x4_any* p = reinterpret_cast<const u32x4_any*>(row + i * SZ);
#pragma unroll
        for (int v = 0; v < SZ; ++v) {
            const u32x4 w = p[v];
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                if constexpr (F32) {
                    o[4 * v + d] = bits_f32(w[d]);
                } else {
                    o[8 * v + 2 * d] = bits_f32(w[d] << 16);
                    o[8 * v + 2 * d + 1] = bits_f32(w[d] & 0xffff0000u);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        o[j] = none;
        if (i + j < V) {
            if constexpr (F32)
                o[j] = reinterpret_cast<const float*>(row)[i + j];
            else
                o[j] = bits_f32((uint32_t)reinterpret_cast<const uint16_t*>(row)[i + j] << 16);
        }
    }
}

template <bool F32>
__device__ __forceinline__ float load1(const char* row, long long i)
{
    if constexpr (F32) return reinterpret_cast<const float*>(row)[i];
    return bits_f32((uint32_t)reinterpret_cast<const uint16_t*>(row)[i] << 16);
}

__device__ __forceinline__ float no_nan(float v) { return v != v ? -__builtin_huge_valf() : v; }

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

// exp((l - top) / T), rate = log2(e) / T: 1 at the top (an infinite one too), 0 at -inf
__device__ __forceinline__ double weight(float l, float top, double rate)
{
    return l == top ? 1.0 : exp2_down(((double)l - (double)top) * rate);
}

__device__ __forceinline__ double rate_of(float t) { return 1.4426950408889634074 / (double)t; }

__device__ __forceinline__ void join(float& top, int& at, float top2, int at2)
{
    if (top2 > top || (top2 == top && at2 < at)) {
        top = top2;
        at = at2;
    }
}

__device__ __forceinline__ int length_of(const VerifyParams& p, int b)
{
    return p.lengths ? min(max(p.lengths[b], 0), p.S) : p.S;
}

template <bool LF32>
__global__ __launch_bounds__(kThreads) void stats_kernel(VerifyParams p)
{
    __shared__ float tops[kThreads / 64];
    __shared__ int ats[kThreads / 64];
    __shared__ double sums[kThreads / 64];
    const int chunk = blockIdx.x, row = blockIdx.y, b = row / (p.S + 1), j = row % (p.S + 1);
    if (chunk == 0 && j == 0 && threadIdx.x == 0) p.tickets[b] = 0;
    if (j > length_of(p, b)) return;
    const float T = p.temperature ? p.temperature[b] : 1.0f;
    const char* l = p.logits + (b * p.l_batch + j * p.l_row) * (LF32 ? 4 : 2);
    const long long i0 = (long long)chunk * kChunk + threadIdx.x * kPer;
    float v[kPer];
    load16<LF32>(v, l, i0, p.V, -__builtin_huge_valf());
    float top = -__builtin_huge_valf();
    int at = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        v[i] = no_nan(v[i]);
        if (v[i] > top) {
            top = v[i];
            at = (int)i0 + i;
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) join(top, at, __shfl_xor(top, o), __shfl_xor(at, o));
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
        tops[wave] = top;
        ats[wave] = at;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) join(top, at, tops[w], ats[w]);
    double s = 0.0;
    if (T > 0.0f && at != 0x7fffffff) {
        const double rate = rate_of(T);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (v[i] > -__builtin_huge_valf()) s += weight(v[i], top, rate);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
    if ((threadIdx.x & 63) == 0) sums[wave] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 64; ++w) s += sums[w];
        p.stats[(size_t)row * p.chunks + chunk] = Stat{s, top, at};
    }
}

// Which of the values get(0..n) a prefix sum first passes target(total) in, by
// all threads: its index, or the last positive value's if none does, or -1 if no
// value is positive.  before: the sum of the values before it.
struct Pick {
    int index;
    double before;
};

template <class Get, class Target>
__device__ __forceinline__ Pick pick(int n, Get get, Target target)
{
    __shared__ double sums[kThreads];
    __shared__ int found, last;
    __shared__ double found_before, last_before;
    const int per = (n + kThreads - 1) / kThreads, i0 = min((int)threadIdx.x * per, n), i1 = min(i0 + per, n);
    __syncthreads();
    double s = 0.0;
    for (int i = i0; i < i1; ++i) s += get(i);
    sums[threadIdx.x] = s;
    if (threadIdx.x == 0) {
        found = 0x7fffffff;
        last = -1;
    }
    __syncthreads();
    for (int o = 1; o < kThreads; o <<= 1) {
        const double add = (int)threadIdx.x >= o ? sums[threadIdx.x - o] : 0.0;
        __syncthreads();
        sums[threadIdx.x] += add;
        __syncthreads();
    }
    const double t = target(sums[kThreads - 1]);
    double c = threadIdx.x > 0 ? sums[threadIdx.x - 1] : 0.0;
    int mine = -1, mine_last = -1;
    double mine_before = 0.0, mine_last_before = 0.0;
    for (int i = i0; i < i1; ++i) {
        const double v = get(i);
        if (v > 0.0) {
            mine_last = i;
            mine_last_before = c;
            if (mine < 0 && c + v > t) {
                mine = i;
                mine_before = c;
            }
        }
        c += v;
    }
    if (mine >= 0) atomicMin(&found, mine);
    if (mine_last >= 0) atomicMax(&last, mine_last);
    __syncthreads();
    if (mine >= 0 && found == mine) found_before = mine_before;
    if (mine_last >= 0 && last == mine_last) last_before = mine_last_before;
    __syncthreads();
    if (found != 0x7fffffff) return Pick{found, found_before};
    return Pick{last, last_before};
}

template <bool LF32, bool QF32>
__global__ __launch_bounds__(kThreads) void sample_kernel(VerifyParams p)
{
    constexpr int kMaxRows = QMV_MAX_DRAFT + 1;
    __shared__ float tops[kMaxRows];
    __shared__ int ats[kMaxRows];
    __shared__ double sums[kMaxRows];
    __shared__ int first_bad;
    __shared__ double partial[kThreads / 64];
    __shared__ bool am_last;
    const int chunk = blockIdx.x, b = blockIdx.y, len = length_of(p, b);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float T = p.temperature ? p.temperature[b] : 1.0f;
    const bool greedy = !(T > 0.0f);
    const double rate = greedy ? 0.0 : rate_of(T);
    const float none = -__builtin_huge_valf();
    const char* lb = p.logits + b * p.l_batch * (LF32 ? 4 : 2);
    const char* qb = p.probs ? p.probs + b * p.q_batch * (QF32 ? 4 : 2) : nullptr;

    // the rows' largest values and sums
    if (threadIdx.x == 0) first_bad = len;
    for (int j = wave; j <= len; j += kThreads / 64) {
        const Stat* st = p.stats + ((size_t)b * (p.S + 1) + j) * p.chunks;
        float top = none;
        int at = 0x7fffffff;
        for (int c = lane; c < p.chunks; c += 64) join(top, at, st[c].top, st[c].at);
        for (int o = 32; o > 0; o >>= 1) join(top, at, __shfl_xor(top, o), __shfl_xor(at, o));
        double s = 0.0;
        if (!greedy)
            for (int c = lane; c < p.chunks; c += 64)
                if (st[c].top > none) s += st[c].sum * weight(st[c].top, top, rate);
        for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
        if (lane == 0) {
            tops[j] = top;
            ats[j] = at;
            sums[j] = s;
        }
    }
    __syncthreads();
    // the first position that is not accepted
    for (int j = threadIdx.x; j < len; j += kThreads) {
        const int x = p.draft[(size_t)b * p.S + j];
        bool yes = false;
        if (x >= 0 && x < p.V) {
            const float l = no_nan(load1<LF32>(lb + (size_t)j * p.l_row * (LF32 ? 4 : 2), x));
            const double q = qb ? (double)load1<QF32>(qb + (size_t)j * p.q_row * (QF32 ? 4 : 2), x) : 1.0;
            const double u = p.u[(size_t)b * (p.S + 1) + j];
            if (greedy)
                yes = x == ats[j] && u * q < 1.0;
            else
                yes = l > none && u * q * sums[j] < weight(l, tops[j], rate);
        }
        if (!yes) atomicMin(&first_bad, j);
    }
    __syncthreads();
    const int n = first_bad;
    const float top = tops[n];
    const double Z = sums[n];
    const char* ln = lb + (size_t)n * p.l_row * (LF32 ? 4 : 2);
    const char* qn = qb ? qb + (size_t)n * p.q_row * (QF32 ? 4 : 2) : nullptr;
    const int xn = n < len ? p.draft[(size_t)b * p.S + n] : -1;
    // Only a rejected position's rest needs another pass over its row: greedy
    // requests take the largest, and a position after the last draft has the sums.
    const bool rest = n < len && !greedy;
    if (!rest && chunk != 0) return;

    // probability left for value i of the row, by chunk-wise loads
    auto rest_of = [&](float l, float q, int i) {
        const double e = l > none ? weight(l, top, rate) / Z : 0.0;
        const double d = e - (qn ? (double)q : i == xn ? 1.0 : 0.0);
        return d > 0.0 ? d : 0.0;
    };
    if (rest) {
        const long long i0 = (long long)chunk * kChunk + threadIdx.x * kPer;
        float l[kPer], q[kPer];
        load16<LF32>(l, ln, i0, p.V, none);
        if (qn) load16<QF32>(q, qn, i0, p.V, 0.0f);
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += rest_of(no_nan(l[i]), qn ? q[i] : 0.0f, (int)i0 + i);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
        if (lane == 0) partial[wave] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kThreads / 64; ++w) s += partial[w];
            __hip_atomic_store(&p.part[(size_t)b * p.chunks + chunk], s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            am_last = __hip_atomic_fetch_add(&p.tickets[b], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                      (uint32_t)p.chunks - 1;
        }
        __syncthreads();
        if (!am_last) return;
    }

    int token = -1;
    if (greedy) {
        token = ats[n] == 0x7fffffff ? -1 : ats[n];
    } else if (top > none) {
        const double u = p.u[(size_t)b * (p.S + 1) + len];
        const Stat* st = p.stats + ((size_t)b * (p.S + 1) + n) * p.chunks;
        double target = 0.0;
        auto aim = [&](double total) { return target = u * total; };
        bool use = rest;
        Pick k{-1, 0.0};
        if (use) {
            k = pick(p.chunks, [&](int c) {
                return __hip_atomic_load(&p.part[(size_t)b * p.chunks + c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }, aim);
            use = k.index >= 0;     // nothing left: sampled from the target itself
        }
        if (!use)
            k = pick(p.chunks, [&](int c) { return st[c].top > none ? st[c].sum * weight(st[c].top, top, rate) : 0.0; }, aim);
        if (k.index >= 0) {
            const int c0 = k.index * kChunk, m = min(kChunk, p.V - c0);
            const double left = target - k.before;
            const Pick i = pick(m, [&](int i) {
                const float l = no_nan(load1<LF32>(ln, c0 + i));
                if (!use) return l > none ? weight(l, top, rate) : 0.0;
                return rest_of(l, qn ? load1<QF32>(qn, c0 + i) : 0.0f, c0 + i);
            }, [&](double) { return left; });
            token = c0 + i.index;
        }
    }
    for (int j = threadIdx.x; j <= p.S; j += kThreads)
        p.tokens[(size_t)b * (p.S + 1) + j] = j < n ? p.draft[(size_t)b * p.S + j] : j == n ? token : -1;
    if (threadIdx.x == 0) p.accepted[b] = n;
}

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
    const long long c = chunks_of(V);
    return piece((long long)sizeof(Stat) * B * (S + 1) * c) + piece(8LL * B * c) + piece(4LL * B);
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
    p.chunks = chunks_of(V);
    char* ws = static_cast<char*>(workspace);
    p.stats = reinterpret_cast<Stat*>(ws);
    ws += piece((long long)sizeof(Stat) * B * (S + 1) * p.chunks);
    p.part = reinterpret_cast<double*>(ws);
    ws += piece(8LL * B * p.chunks);
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
    // the grid's second dimension ends at 65535: batches in slices of whole requests
    const int step = std::max(1, 65535 / (S + 1));
    for (int b = 0; b < B; b += step) {
        VerifyParams s = p;
        const int n = std::min(step, B - b);
        s.B = n;
        s.logits += (size_t)(b * l_batch) * size_of(l_dt);
        if (S > 0) s.draft += (size_t)b * S;
        s.u += (size_t)b * (S + 1);
        if (probs) s.probs += (size_t)(b * q_batch) * size_of(q_dt);
        if (temperature) s.temperature += b;
        if (lengths) s.lengths += b;
        s.tokens += (size_t)b * (S + 1);
        s.accepted += b;
        s.stats += (size_t)b * (S + 1) * p.chunks;
        s.part += (size_t)b * p.chunks;
        s.tickets += b;
        args[0] = &s;
        if (hipLaunchKernel(f1, dim3(p.chunks, n * (S + 1)), dim3(kThreads), args, 0, st) != hipSuccess ||
            hipLaunchKernel(f2, dim3(p.chunks, n), dim3(kThreads), args, 0, st) != hipSuccess)
            return QMV_E_LAUNCH;
    }
    return QMV_OK;
}

}  // extern "C"
