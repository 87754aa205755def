// ops_lora.hip -- qmv_affine_lora: checks, the first kernel (the adapters' first
// product) and the launches.
#include "ops_lora.hpp"

#include <algorithm>

#include "ops_check.hpp"
#include "ops_lora_kernel.hpp"

namespace ops {
namespace {

// h[piece][m][r] = sum over a piece of K of A_a[r][k] x[m][k].
//
// One workgroup per 16 ranks, piece of K and token; it does the work of all
// tokens of its block of 16 that share the token's adapter, and leaves at once if an
// earlier one does.  Bound by the latency of one round of loads: every wave
// has its whole share (8 steps of 16 x 32 values) in flight at once.
template <bool XF32, bool ADF16>
__global__ __launch_bounds__(kMaxWaves* kWave) void shrink_kernel(LoraParams p)
{
    constexpr int NP = XF32 ? 3 : 1, XV = XF32 ? 2 : 1, STEPS = kShrinkK / kMaxWaves / 32;
    __shared__ float join[kMaxWaves * Join<1>::kWords];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int r0 = blockIdx.x * 16, z = blockIdx.y, m = blockIdx.z, m0 = m & ~15;
    const int tok = min(m0 + c, p.M - 1);
    const int mine = p.ids[tok], a = p.ids[m];
    if (a < 0 || a >= p.L) return;
    const uint32_t same = (uint32_t)__ballot(m0 + c < p.M && mine == a) & 0xffffu;
    if (__builtin_ctz(same) != m - m0) return;

    const int k0 = z * kShrinkK + wave * (kShrinkK / kMaxWaves);
    const uint16_t* ar = p.la + ((size_t)a * p.R + min(r0 + c, p.R - 1)) * p.K + 8 * q;
    const char* xr = p.x + ((size_t)tok * p.K + 8 * q) * (XF32 ? 4 : 2);
    u32x4 av[STEPS], xv[STEPS][XV];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int k = min(k0 + 32 * i, p.K - 32);       // past the end: read, not used
        av[i] = *reinterpret_cast<const u32x4*>(ar + k);
#pragma unroll
        for (int v = 0; v < XV; ++v)
            xv[i][v] = reinterpret_cast<const u32x4*>(xr + (size_t)k * (XF32 ? 4 : 2))[v];
    }
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        if (k0 + 32 * i >= p.K) break;
        u32x4 xo[3];
        if constexpr (XF32)
            split_f32(__builtin_bit_cast(f32x4, xv[i][0]), __builtin_bit_cast(f32x4, xv[i][XV - 1]), xo);
        else
            xo[0] = xv[i][0];
        if constexpr (ADF16) {
            u32x4 h, l;
            split_f16(av[i], h, l);
#pragma unroll
            for (int e = 0; e < NP; ++e) acc = mfma(xo[e], l, mfma(xo[e], h, acc));
        } else {
#pragma unroll
            for (int e = 0; e < NP; ++e) acc = mfma(xo[e], av[i], acc);
        }
    }
    Join<1>::write(join, wave, lane, 0, acc);
    __syncthreads();
    if (threadIdx.x < 256) {
        const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
        if ((same >> t) & 1)      // ranks past the last are zero: the second kernel's steps are of 32
            p.h[((size_t)z * p.M + m0 + t) * p.Rp + r0 + r] =
                r0 + r < p.R ? Join<1>::sum(join, kMaxWaves, Join<1>::at(r, t)) : 0.0f;
    }
}

int shrink_launch(const LoraParams& p, bool xf32, hipStream_t st)
{
    const void* fn = xf32 ? (p.adf16 ? (const void*)&shrink_kernel<true, true> : (const void*)&shrink_kernel<true, false>)
                          : (p.adf16 ? (const void*)&shrink_kernel<false, true> : (const void*)&shrink_kernel<false, false>);
    LoraParams q = p;
    void* args[] = {&q};
    return hipLaunchKernel(fn, dim3(p.Rp / 16, p.pieces, p.M), dim3(kMaxWaves * kWave), args, 0, st) == hipSuccess ? 0 : 1;
}

// Row tiles per workgroup: as many as leave a workgroup for about every
// compute unit, since a workgroup reads all activations once.
int row_tiles(int N)
{
    const int tiles = (N + 15) / 16;
    return tiles >= 4 * 200 ? 4 : tiles >= 2 * 200 ? 2 : 1;
}

}  // namespace
}  // namespace ops

extern "C" {

long long qmv_affine_lora_workspace(int M, int K, int rank)
{
    if (M < 1 || M > QMV_MAX_M || K < 1 || K > QMV_MAX_K || rank < 1 || rank > QMV_MAX_RANK) return -1;
    return ops::piece(4LL * ops::shrink_pieces(K) * std::min(M, ops::kLoraTile) * ops::pad_rank(rank));
}

int qmv_affine_lora(const uint32_t* w, const void* scales, const void* biases, const void* x,
                    void* y, const void* lora_a, const void* lora_b, const int32_t* ids,
                    const float* scaling, void* workspace, long long workspace_bytes, int M, int N,
                    int K, int bits, int group_size, int n_adapters, int rank, int x_dt, int sb_dt,
                    int y_dt, int ad_dt, void* stream)
{
    using namespace ops;
    if (!w || !scales || !biases || !x || !y || !lora_a || !lora_b || !ids || !workspace) return QMV_E_NULL;
    if (const int e = check_matrix(N, K, bits, group_size)) return e;
    if (M < 1 || M > QMV_MAX_M) return QMV_E_M_RANGE;
    if (rank < 1 || rank > QMV_MAX_RANK || n_adapters < 1 || n_adapters > QMV_MAX_ADAPTERS) return QMV_E_RANK;
    if (!wide(x_dt) || !half(sb_dt) || !wide(y_dt) || !half(ad_dt)) return QMV_E_DTYPE;
    if (!aligned(w, 16) || !aligned(scales, 16) || !aligned(biases, 16) || !aligned(x, 16) || !aligned(lora_a, 16) ||
        !aligned(lora_b, 16) || !aligned(ids, 4) || !aligned(scaling, 4) || !aligned(workspace, 16) ||
        !aligned(y, size_of(y_dt)))
        return QMV_E_ALIGN;
    const long long need = qmv_affine_lora_workspace(M, K, rank);
    if (workspace_bytes < need) return QMV_E_WORKSPACE;
    const size_t nsb = (size_t)N * (K / group_size) * 2;
    const Span in[] = {{w, (size_t)N * K * bits / 8}, {scales, nsb}, {biases, nsb}, {x, (size_t)M * K * size_of(x_dt)},
                       {lora_a, (size_t)n_adapters * rank * K * 2}, {lora_b, (size_t)n_adapters * N * rank * 2},
                       {ids, (size_t)M * 4}, {scaling, (size_t)n_adapters * 4}};
    const Span out[] = {{y, (size_t)M * N * size_of(y_dt)}, {workspace, (size_t)need}};
    if (!disjoint(in, out)) return QMV_E_ALIAS;

    hipStream_t st = static_cast<hipStream_t>(stream);
    const bool xf32 = x_dt == QMV_DT_F32, sbf = sb_dt == QMV_DT_BF16;
    for (int m = 0; m < M; m += kLoraTile) {
        LoraParams p;
        p.w = w;
        p.s = static_cast<const uint16_t*>(scales);
        p.b = static_cast<const uint16_t*>(biases);
        p.x = static_cast<const char*>(x) + (size_t)m * K * size_of(x_dt);
        p.y = static_cast<char*>(y) + (size_t)m * N * size_of(y_dt);
        p.la = static_cast<const uint16_t*>(lora_a);
        p.lb = static_cast<const uint16_t*>(lora_b);
        p.ids = ids + m;
        p.scaling = scaling;
        p.h = static_cast<float*>(workspace);
        p.M = std::min(kLoraTile, M - m);
        p.N = N;
        p.K = K;
        p.L = n_adapters;
        p.R = rank;
        p.Rp = pad_rank(rank);
        p.pieces = shrink_pieces(K);
        p.yf32 = y_dt == QMV_DT_F32;
        p.adf16 = ad_dt == QMV_DT_F16;
        if (shrink_launch(p, xf32, st)) return QMV_E_LAUNCH;
        const int rt = row_tiles(N), ct = p.M <= 16 ? 1 : p.M <= 32 ? 2 : 4;
        const int bad = bits == 4 ? (group_size == 64 ? lora_launch_b4_g64(p, rt, ct, xf32, sbf, st)
                                                      : lora_launch_b4_g128(p, rt, ct, xf32, sbf, st))
                                  : (group_size == 64 ? lora_launch_b2_g64(p, rt, ct, xf32, sbf, st)
                                                      : lora_launch_b2_g128(p, rt, ct, xf32, sbf, st));
        if (bad) return QMV_E_LAUNCH;
    }
    return QMV_OK;
}

}  // extern "C"
