// ops_moe.hip -- qmv_route, qmv_experts and qmv_moe: checks, the router's
// kernels, the weighted sum of the experts' outputs, and the launches.
#include "ops_moe.hpp"
#include "ops_moe_kernel.hpp"

#include <algorithm>

#include "ops_check.hpp"
#include "ops_tile.hpp"

namespace ops {
namespace {

typedef __attribute__((ext_vector_type(4))) double f64x4;

constexpr int kRouteWaves = 4;
constexpr int kRouteK = 512;                    // columns of D per workgroup
constexpr int kRouteSteps = kRouteK / kRouteWaves / 32;

int route_pieces(int D) { return (D + kRouteK - 1) / kRouteK; }

struct RouteParams {
    const char* x;
    const char* r;
    double* part;       // [pieces][T][E]
    float* weights;
    int32_t* ids;
    int T, D, E, k, pieces;
    bool renorm;
    char* xp;           // where not null: the activations packed for codes of `bits` in groups of `gs`
    int bits, gs;
};

// Eight values of a row at d.. as doubles; zero past the row's end.
template <bool F32>
__device__ __forceinline__ void load8d(double (&o)[8], const char* row, int d, int D)
{
    if (d >= D) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0.0;
        return;
    }
    if constexpr (F32) {
        const f32x4* p = reinterpret_cast<const f32x4*>(row + (size_t)d * 4);
        const f32x4 a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] = a[i];
            o[4 + i] = b[i];
        }
    } else {
        const u32x4 v = *reinterpret_cast<const u32x4*>(row + (size_t)d * 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = bits_f32(v[i] << 16);
            o[2 * i + 1] = bits_f32(v[i] & 0xffff0000u);
        }
    }
}

// Router products of 16 tokens and 16 experts over a piece of D, in fp64 on
// matrix instructions (v_mfma_f64_16x16x4_f64: rows and columns l & 15, k =
// l >> 4, results at row 4 i + (l >> 4)).  fp64, because the choice of experts
// hangs on the order of nearly equal logits: bf16 and fp32 products are exact
// there, and the sums off by 2^-53 of their terms.  Bound by one round of loads: 5.0
// us for one token over 64 experts of 3840 values, or 13 over 128 of 2048; cut into
// pieces of D, since 16 x 16 results alone would leave most compute units idle.
template <bool XF32, bool RF32>
__global__ __launch_bounds__(kRouteWaves* kWave) void logits_kernel(RouteParams p)
{
    __shared__ double join[kRouteWaves][4][64];
    together(p.x, p.r, p.part, p.xp, p.T, p.D, p.E, p.pieces, p.bits, p.gs);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane & 15, q = lane >> 4;
    const int etiles = (p.E + 15) / 16, ttiles = (p.T + 15) / 16;
    int at = blockIdx.x;
    if (at >= etiles * ttiles * p.pieces) {
        const Packed pk(p.D, p.bits, p.gs, false);
        pack(p.x, p.xp, p.T, p.D, pk, XF32, (size_t)(at - etiles * ttiles * p.pieces) * (kRouteWaves * kWave) + threadIdx.x);
        return;
    }
    const int e0 = at % etiles * 16, t0 = at / etiles % ttiles * 16, z = at / (etiles * ttiles);
    const char* xr = p.x + (size_t)min(t0 + c, p.T - 1) * p.D * (XF32 ? 4 : 2);
    const char* rr = p.r + (size_t)min(e0 + c, p.E - 1) * p.D * (RF32 ? 4 : 2);
    const int d0 = z * kRouteK + wave * (kRouteK / kRouteWaves) + 8 * q;
    f64x4 acc = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int s = 0; s < kRouteSteps; ++s) {
        double a[8], b[8];
        load8d<XF32>(a, xr, d0 + 32 * s, p.D);
        load8d<RF32>(b, rr, d0 + 32 * s, p.D);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc = __builtin_amdgcn_mfma_f64_16x16x4f64(a[i], b[i], acc, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) join[wave][i][lane] = acc[i];
    __syncthreads();
    const int i = threadIdx.x >> 6, t = t0 + 4 * i + q, e = e0 + c;    // one result per thread
    double v = join[0][i][lane];
#pragma unroll
    for (int w = 1; w < kRouteWaves; ++w) v += join[w][i][lane];
    if (t < p.T && e < p.E) p.part[((size_t)z * p.T + t) * p.E + e] = v;
}

__global__ __launch_bounds__(kRouteWaves* kWave) void pack_kernel(const char* x, char* xp, int T, int D, int bits, int gs, bool f32)
{
    const Packed pk(D, bits, gs, false);
    pack(x, xp, T, D, pk, f32, (size_t)blockIdx.x * (kRouteWaves * kWave) + threadIdx.x);
}

// The pairs sorted by expert: each expert's take whole tiles of 16 rows, in their
// order.  A workgroup per pair counts for itself where its row lies, and packs the
// token's activations there; the first one notes every expert's place and count.
// 512 pairs over 32 experts: 6.2 us, three barriers and one round of loads.
struct SortParams {
    const char* x;
    char* xp;
    const int32_t* ids;
    int* base;
    int* count;
    int* place;
    size_t plane;
    int P, k, D, E, bits, gs;
    bool f32;
};

__global__ __launch_bounds__(kRouteWaves* kWave) void sort_kernel(SortParams p)
{
    constexpr int THREADS = kRouteWaves * kWave, PER = QMV_MAX_EXPERTS / THREADS;
    __shared__ int counts[QMV_MAX_EXPERTS];
    __shared__ int sums[2][kRouteWaves];
    together(p.x, p.xp, p.ids, p.base, p.count, p.place, p.plane, p.P, p.k, p.D, p.E, p.bits, p.gs);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, pair = blockIdx.x;
    const int id = p.ids[pair];
    const bool valid = id >= 0 && id < p.E;
    if (!valid && pair != 0) {
        if (tid == 0) p.place[pair] = -1;
        return;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) counts[tid + THREADS * j] = 0;
    __syncthreads();
    int before = 0;                     // pairs before this one of its expert
    for (int i = tid; i < p.P; i += THREADS) {
        const int v = p.ids[i];
        if (v >= 0 && v < p.E) {
            atomicAdd(&counts[v], 1);
            if (i < pair && v == id) ++before;
        }
    }
    __syncthreads();
    // a thread's PER neighbouring experts; their tiles, and those of the threads before it
    int tiles[PER], own = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        tiles[j] = (counts[tid * PER + j] + 15) / 16;
        own += tiles[j];
    }
    int to = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int add = __shfl_up(to, o);
        if (lane >= o) to += add;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) before += __shfl_xor(before, o);
    if (lane == 63) sums[0][wave] = to;
    if (lane == 0) sums[1][wave] = before;
    __syncthreads();
    int at = to - own;
    before = 0;
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) {
        if (w < wave) at += sums[0][w];
        before += sums[1][w];
    }
    __shared__ int bases[QMV_MAX_EXPERTS];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = tid * PER + j;
        bases[e] = at;
        if (pair == 0 && e < p.E) {
            p.base[e] = at;
            p.count[e] = counts[e];
        }
        at += tiles[j];
    }
    __syncthreads();
    const int row = valid ? bases[id] * 16 + before : -1;
    if (tid == 0) p.place[pair] = row;
    if (!valid) return;
    const Packed pk(p.D, p.bits, p.gs, true);
    const int words = p.D * p.bits / 32, vpw = 32 / p.bits;
    for (int w = tid; w < words; w += THREADS) {
        const size_t k = (size_t)(pair / p.k) * p.D + (size_t)w * vpw;
        char* o = p.xp + pk.word(row, w);
        if (p.bits == 4) {
            if (p.f32)
                pack_word<4, true>(p.x + k * 4, o, p.plane, pk.op_step());
            else
                pack_word<4, false>(p.x + k * 2, o, p.plane, pk.op_step());
        } else {
            if (p.f32)
                pack_word<2, true>(p.x + k * 4, o, p.plane, pk.op_step());
            else
                pack_word<2, false>(p.x + k * 2, o, p.plane, pk.op_step());
        }
    }
}

// Top-k and softmax of one token's logits by a workgroup.  An expert's place is the
// number of experts before it (a larger logit, or an equal one of a lower index),
// counted against all of them from LDS; with few experts the threads share the
// counting of each.  3.1 us over 64 experts, 5.0 over 128: the chain of its steps.
__global__ __launch_bounds__(kRouteWaves* kWave) void topk_kernel(RouteParams p)
{
    constexpr int THREADS = kRouteWaves * kWave, PER = QMV_MAX_EXPERTS / THREADS;
    __shared__ double value[QMV_MAX_EXPERTS];
    __shared__ int place[QMV_MAX_EXPERTS];
    __shared__ double top_value[QMV_MAX_TOP_K];
    __shared__ int top_id[QMV_MAX_TOP_K];
    __shared__ double sums[kRouteWaves];
    together(p.part, p.weights, p.ids, p.T, p.E, p.k, p.pieces);
    const int tid = threadIdx.x, t = blockIdx.x;
    const double low = -__builtin_huge_val();
    double v[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = tid + THREADS * j;
        v[j] = low;
        if (THREADS * j < p.E && e < p.E) {
            double s = 0.0;
            for (int z0 = 0; z0 < p.pieces; z0 += 8) {
                double x[8];
#pragma unroll
                for (int z = 0; z < 8; ++z) x[z] = p.part[((size_t)min(z0 + z, p.pieces - 1) * p.T + t) * p.E + e];
#pragma unroll
                for (int z = 0; z < 8; ++z)
                    if (z0 + z < p.pieces) s += x[z];
            }
            v[j] = s != s ? low : s;
            value[e] = v[j];
            place[e] = 0;
        }
    }
    __syncthreads();
    const int share = p.E <= 64 ? 4 : p.E <= 128 ? 2 : 1, wide = THREADS / share;      // threads per expert; experts at a time
    for (int e = tid % wide; e < p.E; e += wide) {
        const int part = tid / wide, j0 = part * p.E / share, j1 = (part + 1) * p.E / share;
        const double mine = value[e];
        int n = 0;
#pragma unroll 8
        for (int j = j0; j < j1; ++j) {
            const double x = value[j];
            n += x > mine || (x == mine && j < e) ? 1 : 0;
        }
        if (share == 1)
            place[e] = n;
        else
            atomicAdd(&place[e], n);
    }
    __syncthreads();
    for (int e = tid; e < p.E; e += THREADS) {
        const int at = place[e];
        if (at < p.k) {
            top_value[at] = value[e];
            top_id[at] = e;
        }
    }
    __syncthreads();
    const double top = top_value[0];
    const double mine = tid < p.k ? exp(top_value[tid] - top) : 0.0;
    double all = 0.0;
    if (p.renorm) {
        if (tid < kWave) value[tid] = mine;         // read by the same wave
        __builtin_amdgcn_wave_barrier();
        for (int j = 0; j < p.k; ++j) all += value[j];
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (tid + THREADS * j < p.E) all += exp(v[j] - top);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o);
        if ((tid & 63) == 0) sums[tid >> 6] = all;
        __syncthreads();
        all = sums[0];
#pragma unroll
        for (int w = 1; w < kRouteWaves; ++w) all += sums[w];
    }
    if (tid < p.k) {
        p.weights[(size_t)t * p.k + tid] = (float)(mine / all);
        p.ids[(size_t)t * p.k + tid] = top_id[tid];
    }
}

// y[t] = sum of weight * expert output over the token's slots, in their order: 4.7 us
// for 13 tokens of 8 x 2048 values, mostly the launch and three dependent loads.
__global__ __launch_bounds__(256) void combine_kernel(const float* z, const float* weights, const int32_t* ids, const int* place,
                                                      void* y, int D, int E, int k, bool yf32)
{
    const int d = blockIdx.x * 256 + threadIdx.x, t = blockIdx.y;
    if (d >= D) return;
    float v = 0.0f;
    for (int j = 0; j < k; ++j) {
        const size_t pair = (size_t)t * k + j;
        const int e = ids[pair];
        if (e >= 0 && e < E) v = __builtin_fmaf(weights[pair], z[(place ? (size_t)place[pair] : pair) * D + d], v);
    }
    store_y(y, (size_t)t * D + d, v, yf32);
}

bool launch(const void* fn, dim3 grid, int threads, void** args, hipStream_t st)
{
    return hipLaunchKernel(fn, grid, dim3(threads), args, 0, st) == hipSuccess;
}

int check_route(int T, int D, int E, int k, int x_dt, int r_dt)
{
    if (T < 1 || T > QMV_MAX_M) return QMV_E_M_RANGE;
    if (D < 8 || D > QMV_MAX_K || D % 8 != 0) return QMV_E_SHAPE;
    if (E < 1 || E > QMV_MAX_EXPERTS || k < 1 || k > E || k > QMV_MAX_TOP_K) return QMV_E_EXPERTS;
    if (!wide(x_dt) || !wide(r_dt)) return QMV_E_DTYPE;
    return QMV_OK;
}

int check_experts(int T, int D, int F, int E, int k, int bits, int gs, int x_dt, int sb_dt, int y_dt)
{
    if (const int e = check_matrix(2LL * F, D, bits, gs)) return e;
    if (const int e = check_matrix(D, F, bits, gs)) return e;
    if (T < 1 || T > QMV_MAX_M) return QMV_E_M_RANGE;
    if (E < 1 || E > QMV_MAX_EXPERTS || k < 1 || k > QMV_MAX_TOP_K) return QMV_E_EXPERTS;
    if (!wide(x_dt) || !half(sb_dt) || !wide(y_dt)) return QMV_E_DTYPE;
    return QMV_OK;
}

// the router of n tokens; where xp is not null their activations are packed too
int run_route(const char* x, const void* router, float* weights, int32_t* ids, void* part, char* xp, int n, int D, int E, int k,
              bool renorm, int x_dt, int r_dt, int bits, int gs, hipStream_t st)
{
    const bool xf = x_dt == QMV_DT_F32, rf = r_dt == QMV_DT_F32;
    const void* fn = xf ? (rf ? (const void*)&logits_kernel<true, true> : (const void*)&logits_kernel<true, false>)
                        : (rf ? (const void*)&logits_kernel<false, true> : (const void*)&logits_kernel<false, false>);
    RouteParams p;
    p.x = x;
    p.r = static_cast<const char*>(router);
    p.part = static_cast<double*>(part);
    p.weights = weights;
    p.ids = ids;
    p.T = n;
    p.D = D;
    p.E = E;
    p.k = k;
    p.pieces = route_pieces(D);
    p.renorm = renorm;
    p.xp = xp;
    p.bits = bits;
    p.gs = gs;
    constexpr int threads = kRouteWaves * kWave;
    const int packs = xp ? (int)(((long long)n * (D * bits / 32) + threads - 1) / threads) : 0;
    void* args[] = {&p};
    return launch(fn, dim3((E + 15) / 16 * ((n + 15) / 16) * p.pieces + packs), threads, args, st) &&
                   launch((const void*)&topk_kernel, dim3(n), threads, args, st)
               ? QMV_OK
               : QMV_E_LAUNCH;
}

// Pairs are sorted by expert where an expert meets eight or more on average and the
// products are not small.  Below that a wave's 16 rows are mostly repeats of a few,
// which cost it little, and sorting is a launch of about 5 us (128 tokens over 32
// experts of 3840 x 1920, 16 pairs each: 157 us sorted against 247; 64 tokens over 4 of
// 512 x 512, 32 pairs each: 27.7 against 23.6; over 4 of 1024 x 512, 30.2, 31.2).
bool sorted(int n, int k, int E, int D, int F)
{
    return (long long)n * k >= 8LL * E && (k > kTokenSlots || (long long)n * k * D * F > 1 << 25);
}

// Scratch memory of the experts' products for n tokens.
struct ExpertPieces {
    long long h, z, plan, all;       // where the hidden values, the outputs and the plan start; the packed activations come first
    size_t x_plane, h_plane;
    ExpertPieces(int n, int D, int F, int k, int E, int bits, int gs)
    {
        const bool s = sorted(n, k, E, D, F);
        const int rows = s ? (n * k / 16 + std::min(E, n * k)) * 16 : n * k;
        x_plane = Packed(D, bits, gs, s).plane(s ? rows : n);
        h_plane = Packed(F, bits, gs, s).plane(rows);
        h = piece(3 * (long long)x_plane);
        z = h + piece(3 * (long long)h_plane);
        plan = z + piece(4LL * rows * D);
        all = plan + piece(4LL * (2 * E + n * k));
    }
};

// The same for any codes and experts: rows are rounded up to whole slabs of 256 or
// 128 codes, and sorted pairs, eight to an expert or more, take three rows each at most.
long long expert_bytes(int T, int D, int F, int k)
{
    const int n = std::min(T, kMoeTile), d = (D + 255) / 256 * 256, f = (F + 255) / 256 * 256;
    const ExpertPieces a(n, d, f, k, QMV_MAX_EXPERTS, 4, 64), b(n, d, f, k, std::max(1, n * k / 8), 4, 64);
    return std::max(a.all, b.all);
}

// Packs the activations of n tokens for experts whose ids are known: sorted, or as they come.
int run_pack(const char* x, const int32_t* ids, char* ws, int n, int D, int F, int E, int k, int bits, int gs, int x_dt, hipStream_t st)
{
    constexpr int threads = kRouteWaves * kWave;
    bool f32 = x_dt == QMV_DT_F32;
    if (!sorted(n, k, E, D, F)) {
        void* args[] = {&x, &ws, &n, &D, &bits, &gs, &f32};
        const int packs = (int)(((long long)n * (D * bits / 32) + threads - 1) / threads);
        return launch((const void*)&pack_kernel, dim3(packs), threads, args, st) ? QMV_OK : QMV_E_LAUNCH;
    }
    const ExpertPieces at(n, D, F, k, E, bits, gs);
    SortParams p;
    p.x = x;
    p.xp = ws;
    p.ids = ids;
    p.base = reinterpret_cast<int*>(ws + at.plan);
    p.count = p.base + E;
    p.place = p.count + E;
    p.plane = at.x_plane;
    p.P = n * k;
    p.k = k;
    p.D = D;
    p.E = E;
    p.bits = bits;
    p.gs = gs;
    p.f32 = f32;
    void* args[] = {&p};
    return launch((const void*)&sort_kernel, dim3(p.P), threads, args, st) ? QMV_OK : QMV_E_LAUNCH;
}

// the experts of n tokens, whose activations lie packed at the start of ws
int run_experts(const float* weights, const int32_t* ids, const uint32_t* w13, const void* s13, const void* b13,
                const uint32_t* w2, const void* s2, const void* b2, char* y, char* ws, int n, int D, int F, int E, int k, int bits,
                int gs, int x_dt, int sb_dt, int y_dt, hipStream_t st)
{
    const auto go = bits == 4 ? (gs == 64 ? expert_launch_b4_g64 : expert_launch_b4_g128)
                              : (gs == 64 ? expert_launch_b2_g64 : expert_launch_b2_g128);
    const bool xf32 = x_dt == QMV_DT_F32, sbf = sb_dt == QMV_DT_BF16, by_expert = sorted(n, k, E, D, F);
    bool yf32 = y_dt == QMV_DT_F32;
    const ExpertPieces at(n, D, F, k, E, bits, gs);
    ExpertParams p;
    p.xp = ws;
    p.ids = ids;
    p.w13 = w13;
    p.s13 = static_cast<const uint16_t*>(s13);
    p.b13 = static_cast<const uint16_t*>(b13);
    p.w2 = w2;
    p.s2 = static_cast<const uint16_t*>(s2);
    p.b2 = static_cast<const uint16_t*>(b2);
    p.h = ws + at.h;
    p.z = reinterpret_cast<float*>(ws + at.z);
    p.x_plane = at.x_plane;
    p.h_plane = at.h_plane;
    p.P = n * k;
    p.k = k;
    p.D = D;
    p.F = F;
    p.E = E;
    p.slots = by_expert ? E : std::min(p.P, E);
    p.base = by_expert ? reinterpret_cast<const int*>(ws + at.plan) : nullptr;
    p.count = by_expert ? p.base + E : nullptr;
    p.log_parts = 0;
    p.per_k = 1.0f / (float)k;
    p.weights = weights;
    p.y = y;
    p.yf32 = yf32;
    if (!by_expert && by_token(n, k, D, F, bits)) return go(0, p, xf32, sbf, st) || go(2, p, xf32, sbf, st) ? QMV_E_LAUNCH : QMV_OK;
    if (go(0, p, xf32, sbf, st) || go(1, p, xf32, sbf, st)) return QMV_E_LAUNCH;
    const float* z = p.z;
    const int* place = by_expert ? p.count + E : nullptr;
    void* args[] = {&z, &weights, &ids, &place, &y, &D, &E, &k, &yf32};
    return launch((const void*)&combine_kernel, dim3((D + 255) / 256, n), 256, args, st) ? QMV_OK : QMV_E_LAUNCH;
}

}  // namespace
}  // namespace ops

extern "C" {

long long qmv_route_workspace(int T, int D, int n_experts)
{
    if (T < 1 || T > QMV_MAX_M || D < 1 || D > QMV_MAX_K || n_experts < 1 || n_experts > QMV_MAX_EXPERTS) return -1;
    return ops::piece(8LL * ops::route_pieces(D) * std::min(T, ops::kMoeTile) * n_experts);
}

int qmv_route(const void* x, const void* router, float* weights, int32_t* ids, void* workspace,
              long long workspace_bytes, int T, int D, int n_experts, int top_k, int renormalize,
              int x_dt, int r_dt, void* stream)
{
    using namespace ops;
    if (!x || !router || !weights || !ids || !workspace) return QMV_E_NULL;
    if (const int e = check_route(T, D, n_experts, top_k, x_dt, r_dt)) return e;
    if (!aligned(x, 16) || !aligned(router, 16) || !aligned(weights, 4) || !aligned(ids, 4) || !aligned(workspace, 16))
        return QMV_E_ALIGN;
    const long long need = qmv_route_workspace(T, D, n_experts);
    if (workspace_bytes < need) return QMV_E_WORKSPACE;
    const Span in[] = {{x, (size_t)T * D * size_of(x_dt)}, {router, (size_t)n_experts * D * size_of(r_dt)}};
    const Span out[] = {{weights, (size_t)T * top_k * 4}, {ids, (size_t)T * top_k * 4}, {workspace, (size_t)need}};
    if (!disjoint(in, out)) return QMV_E_ALIAS;
    for (int t = 0; t < T; t += kMoeTile)
        if (const int e = run_route(static_cast<const char*>(x) + (size_t)t * D * size_of(x_dt), router, weights + (size_t)t * top_k,
                                    ids + (size_t)t * top_k, workspace, nullptr, std::min(kMoeTile, T - t), D, n_experts, top_k,
                                    renormalize != 0, x_dt, r_dt, 4, 64, static_cast<hipStream_t>(stream)))
            return e;
    return QMV_OK;
}

long long qmv_experts_workspace(int T, int D, int F, int top_k)
{
    if (T < 1 || T > QMV_MAX_M || D < 1 || D > QMV_MAX_K || F < 1 || F > QMV_MAX_K || top_k < 1 || top_k > QMV_MAX_TOP_K)
        return -1;
    return ops::expert_bytes(T, D, F, top_k);
}

int qmv_experts(const void* x, const float* weights, const int32_t* ids, const uint32_t* w13,
                const void* s13, const void* b13, const uint32_t* w2, const void* s2,
                const void* b2, void* y, void* workspace, long long workspace_bytes, int T, int D,
                int F, int n_experts, int top_k, int bits, int group_size, int x_dt, int sb_dt,
                int y_dt, void* stream)
{
    using namespace ops;
    if (!x || !weights || !ids || !w13 || !s13 || !b13 || !w2 || !s2 || !b2 || !y || !workspace) return QMV_E_NULL;
    if (const int e = check_experts(T, D, F, n_experts, top_k, bits, group_size, x_dt, sb_dt, y_dt)) return e;
    if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(s13, 16) || !aligned(b13, 16) || !aligned(w2, 16) ||
        !aligned(s2, 16) || !aligned(b2, 16) || !aligned(weights, 4) || !aligned(ids, 4) || !aligned(workspace, 16) ||
        !aligned(y, size_of(y_dt)))
        return QMV_E_ALIGN;
    const long long need = qmv_experts_workspace(T, D, F, top_k);
    if (workspace_bytes < need) return QMV_E_WORKSPACE;
    const size_t E = (size_t)n_experts, nw = E * D * F * bits / 8, ns = E * D * (F / group_size) * 2;
    const size_t ns13 = E * 2 * F * (D / group_size) * 2;
    const Span in[] = {{x, (size_t)T * D * size_of(x_dt)}, {weights, (size_t)T * top_k * 4}, {ids, (size_t)T * top_k * 4},
                       {w13, 2 * nw}, {s13, ns13}, {b13, ns13}, {w2, nw}, {s2, ns}, {b2, ns}};
    const Span out[] = {{y, (size_t)T * D * size_of(y_dt)}, {workspace, (size_t)need}};
    if (!disjoint(in, out)) return QMV_E_ALIAS;
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    for (int t = 0; t < T; t += kMoeTile) {
        const int n = std::min(kMoeTile, T - t);
        if (const int e = run_pack(static_cast<const char*>(x) + (size_t)t * D * size_of(x_dt), ids + (size_t)t * top_k, ws, n, D, F,
                                   n_experts, top_k, bits, group_size, x_dt, st))
            return e;
        if (const int e = run_experts(weights + (size_t)t * top_k, ids + (size_t)t * top_k, w13, s13, b13, w2, s2, b2,
                                      static_cast<char*>(y) + (size_t)t * D * size_of(y_dt), ws, n, D, F, n_experts, top_k, bits,
                                      group_size, x_dt, sb_dt, y_dt, st))
            return e;
    }
    return QMV_OK;
}

long long qmv_moe_workspace(int T, int D, int F, int n_experts, int top_k)
{
    const long long r = qmv_route_workspace(T, D, n_experts), e = qmv_experts_workspace(T, D, F, top_k);
    return r < 0 || e < 0 ? -1 : r + e;
}

int qmv_moe(const void* x, const void* router, const uint32_t* w13, const void* s13,
            const void* b13, const uint32_t* w2, const void* s2, const void* b2, void* y,
            float* weights, int32_t* ids, void* workspace, long long workspace_bytes, int T, int D,
            int F, int n_experts, int top_k, int renormalize, int bits, int group_size, int x_dt,
            int r_dt, int sb_dt, int y_dt, void* stream)
{
    using namespace ops;
    if (!x || !router || !weights || !ids || !w13 || !s13 || !b13 || !w2 || !s2 || !b2 || !y || !workspace)
        return QMV_E_NULL;
    if (const int e = check_experts(T, D, F, n_experts, top_k, bits, group_size, x_dt, sb_dt, y_dt)) return e;
    if (const int e = check_route(T, D, n_experts, top_k, x_dt, r_dt)) return e;
    if (!aligned(x, 16) || !aligned(router, 16) || !aligned(w13, 16) || !aligned(s13, 16) || !aligned(b13, 16) ||
        !aligned(w2, 16) || !aligned(s2, 16) || !aligned(b2, 16) || !aligned(weights, 4) || !aligned(ids, 4) ||
        !aligned(workspace, 16) || !aligned(y, size_of(y_dt)))
        return QMV_E_ALIGN;
    const long long need = qmv_moe_workspace(T, D, F, n_experts, top_k);
    if (workspace_bytes < need) return QMV_E_WORKSPACE;
    const size_t E = (size_t)n_experts, nw = E * D * F * bits / 8, ns = E * D * (F / group_size) * 2;
    const size_t ns13 = E * 2 * F * (D / group_size) * 2;
    const Span in[] = {{x, (size_t)T * D * size_of(x_dt)}, {router, E * D * size_of(r_dt)},
                       {w13, 2 * nw}, {s13, ns13}, {b13, ns13}, {w2, nw}, {s2, ns}, {b2, ns}};
    const Span out[] = {{y, (size_t)T * D * size_of(y_dt)}, {weights, (size_t)T * top_k * 4},
                        {ids, (size_t)T * top_k * 4}, {workspace, (size_t)need}};
    if (!disjoint(in, out)) return QMV_E_ALIAS;
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* const part = static_cast<char*>(workspace) + qmv_experts_workspace(T, D, F, top_k);
    for (int t = 0; t < T; t += kMoeTile) {
        const int n = std::min(kMoeTile, T - t);
        float* const wt = weights + (size_t)t * top_k;
        int32_t* const it = ids + (size_t)t * top_k;
        const char* const xt = static_cast<const char*>(x) + (size_t)t * D * size_of(x_dt);
        char* const ws = static_cast<char*>(workspace);
        const bool later = sorted(n, top_k, n_experts, D, F);         // packed when the ids are known
        if (const int e = run_route(xt, router, wt, it, part, later ? nullptr : ws, n, D, n_experts, top_k, renormalize != 0, x_dt,
                                    r_dt, bits, group_size, st))
            return e;
        if (later)
            if (const int e = run_pack(xt, it, ws, n, D, F, n_experts, top_k, bits, group_size, x_dt, st)) return e;
        if (const int e = run_experts(wt, it, w13, s13, b13, w2, s2, b2, static_cast<char*>(y) + (size_t)t * D * size_of(y_dt),
                                      ws, n, D, F, n_experts, top_k, bits, group_size, x_dt, sb_dt, y_dt, st))
            return e;
    }
    return QMV_OK;
}

}  // extern "C"
