// ops_lora.hip -- qmv_affine_lora: checks, the first kernel (the adapters' first
// product) and the launches.
#include "ops_lora.hpp"

#include <algorithm>

#include "ops_check.hpp"
#include "ops_lora_kernel.hpp"

namespace ops {
namespace {

constexpr int kPackWords = kMaxWaves * kWave;   // words of codes whose activations a workgroup of the first kernel packs

// h[piece][m][r] = sum over a piece of K of A_a[r][k] x[m][k].
//
// A workgroup takes 16 ranks, a piece of K and a token: it does the work of all
// tokens of its block of 64 that share the token's adapter, 16 at a time, and
// leaves at once if an earlier one does.  Bound by the latency of one round of
// loads: every wave has its whole share (8 steps of 16 x 32 values) in flight at
// once.  Workgroups past those list a block's adapters, or pack activations, for
// the second kernel.  One token, rank 16, K = 3840: 4.4 us; 64 tokens of 32 adapters,
// rank 64, K = 5120: 24 MB in 8.4 us.
template <bool XF32, bool ADF16>
__global__ __launch_bounds__(kMaxWaves* kWave) void shrink_kernel(LoraParams p, int bits, int gs)
{
    constexpr int NP = XF32 ? 3 : 1, XV = XF32 ? 2 : 1, STEPS = kShrinkK / kMaxWaves / 32;
    __shared__ float join[kMaxWaves * Join<1>::kWords];
    __shared__ uint8_t order[kMaxWaves][kBlock];
    __shared__ __attribute__((aligned(16))) char turns[kMaxWaves][1024 * (1 + XV)];
    together(p.x, p.la, p.ids, p.scaling, p.h, p.lists, p.xp, p.M, p.K, p.L, p.R, p.Rp, p.pieces, bits, gs);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int rtiles = p.Rp / 16, blocks = (p.M + kBlock - 1) / kBlock;
    char* const turn = turns[wave];
    int at = blockIdx.x;
    if (at < blocks) {
        if (wave > 0) return;
        const int m = at * kBlock + lane, id = p.ids[min(m, p.M - 1)];
        const bool has = m < p.M && id >= 0 && id < p.L;
        const float scaling = has && p.scaling ? p.scaling[id] : 1.0f;
        unsigned long long left = __ballot(has);
        AdapterList& list = p.lists[at];
        int n = 0;
        if (lane == 0) list.any = left;
        for (; left != 0; ++n) {
            const int lead = __builtin_ctzll(left), a = __builtin_amdgcn_readlane(id, lead);
            const unsigned long long same = __ballot(has && id == a);
            if (lane == lead) {
                list.scaling[n] = scaling;
                list.adapter[n] = a;
                list.tokens[n] = same;
            }
            left &= ~same;
        }
        if (lane == 0) list.count = n;
        return;
    }
    at -= blocks;
    if (at >= rtiles * p.pieces * p.M) {
        const Packed pk(p.K, bits, gs, true);
        pack(p.x, p.xp, p.M, p.K, pk, XF32, (size_t)(at - rtiles * p.pieces * p.M) * kPackWords + threadIdx.x);
        return;
    }
    const int r0 = at % rtiles * 16, z = at / rtiles % p.pieces, m = at / (rtiles * p.pieces), m0 = m & ~(kBlock - 1);
    const int tok = min(m0 + lane, p.M - 1);
    const int mine = p.ids[tok], a = p.ids[m];
    if (a < 0 || a >= p.L) return;
    const unsigned long long same = __ballot(m0 + lane < p.M && mine == a);
    if (__builtin_ctzll(same) != m - m0) return;
    const int n = __popcll(same);
    if ((same >> lane) & 1) order[wave][__popcll(same & ((1ull << lane) - 1))] = (uint8_t)lane;
    __builtin_amdgcn_wave_barrier();

    // Four (eight for fp32) neighbouring lanes load a row's pieces, and the wave
    // turns them over through LDS into the order of the matrix instruction.
    const int k0 = z * kShrinkK + wave * (kShrinkK / kMaxWaves);
    const int row = lane >> 2, pc = (lane & 3) ^ ((row >> 1) & 3);
    const uint16_t* ar = p.la + ((size_t)a * p.R + min(r0 + row, p.R - 1)) * p.K + 8 * pc;
    u32x4 av[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        av[i] = *reinterpret_cast<const u32x4*>(ar + min(k0 + 32 * i, p.K - 32));       // past the end: read, not used
    for (int t0 = 0; t0 < n; t0 += 16) {
        u32x4 xv[STEPS][XV];
#pragma unroll
        for (int v = 0; v < XV; ++v) {
            const int t = XF32 ? (lane >> 3) + 8 * v : row, piece = XF32 ? (lane & 7) ^ (t & 7) : 2 * pc;     // of four values
            const char* xr = p.x + ((size_t)(m0 + order[wave][min(t0 + t, n - 1)]) * p.K + 4 * piece) * (XF32 ? 4 : 2);
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
                xv[i][v] = *reinterpret_cast<const u32x4*>(xr + (size_t)min(k0 + 32 * i, p.K - 32) * (XF32 ? 4 : 2));
        }
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            if (k0 + 32 * i >= p.K) break;
            *reinterpret_cast<u32x4*>(turn + lane * 16) = av[i];
#pragma unroll
            for (int v = 0; v < XV; ++v) *reinterpret_cast<u32x4*>(turn + 1024 + v * 1024 + lane * 16) = xv[i][v];
            __builtin_amdgcn_wave_barrier();
            const char* at4 = turn + (4 * c + (q ^ ((c >> 1) & 3))) * 16;
            const u32x4 ao = *reinterpret_cast<const u32x4*>(at4);
            u32x4 xo[3];
            if constexpr (XF32) {
                const char* at8 = turn + 1024 + c * 128;
                split_f32(*reinterpret_cast<const f32x4*>(at8 + ((2 * q) ^ (c & 7)) * 16),
                          *reinterpret_cast<const f32x4*>(at8 + ((2 * q + 1) ^ (c & 7)) * 16), xo);
            } else {
                xo[0] = *reinterpret_cast<const u32x4*>(at4 + 1024);
            }
            __builtin_amdgcn_wave_barrier();
            if constexpr (ADF16) {
                u32x4 h, l;
                split_f16(ao, h, l);
#pragma unroll
                for (int e = 0; e < NP; ++e) acc = mfma(xo[e], l, mfma(xo[e], h, acc));
            } else {
#pragma unroll
                for (int e = 0; e < NP; ++e) acc = mfma(xo[e], ao, acc);
            }
        }
        if (t0 > 0) __syncthreads();
        Join<1>::write(join, wave, lane, 0, acc);
        __syncthreads();
        if (threadIdx.x < 256) {
            const int r = threadIdx.x & 15, t = threadIdx.x >> 4;
            if (t0 + t < n)      // ranks past the last are zero: the second kernel's steps are of 32
                p.h[((size_t)z * p.M + m0 + order[wave][t0 + t]) * p.Rp + r0 + r] =
                    r0 + r < p.R ? Join<1>::sum(join, 0, kMaxWaves, Join<1>::at(r, t)) : 0.0f;
        }
    }
}

int shrink_launch(const LoraParams& p, int bits, int gs, bool xf32, hipStream_t st)
{
    const void* fn = xf32 ? (p.adf16 ? (const void*)&shrink_kernel<true, true> : (const void*)&shrink_kernel<true, false>)
                          : (p.adf16 ? (const void*)&shrink_kernel<false, true> : (const void*)&shrink_kernel<false, false>);
    LoraParams q = p;
    void* args[] = {&q, &bits, &gs};
    const long long blocks = (p.M + kBlock - 1) / kBlock, packs = ((long long)p.M * (p.K * bits / 32) + kPackWords - 1) / kPackWords;
    const long long grid = blocks + (long long)p.Rp / 16 * p.pieces * p.M + packs;
    return hipLaunchKernel(fn, dim3((uint32_t)grid), dim3(kMaxWaves * kWave), args, 0, st) == hipSuccess ? 0 : 1;
}

struct LoraPieces {
    long long h, lists, all;
    LoraPieces(int M, int K, int R)       // M: tokens of one pair of launches
    {
        h = piece(4LL * shrink_pieces(K) * M * pad_rank(R));
        lists = h + piece((long long)sizeof(AdapterList) * ((M + kBlock - 1) / kBlock));
        all = lists + piece(6LL * ((M + 15) / 16 * 16) * ((K + 255) / 256 * 256));     // three planes of two bytes, for fp32, in whole slabs
    }
};

}  // namespace
}  // namespace ops

extern "C" {

long long qmv_affine_lora_workspace(int M, int K, int rank)
{
    if (M < 1 || M > QMV_MAX_M || K < 1 || K > QMV_MAX_K || rank < 1 || rank > QMV_MAX_RANK) return -1;
    return ops::LoraPieces(std::min(M, ops::kLoraTile), K, rank).all;
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
    const LoraPieces at(std::min(M, kLoraTile), K, rank);
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
        p.lists = reinterpret_cast<AdapterList*>(static_cast<char*>(workspace) + at.h);
        p.xp = static_cast<char*>(workspace) + at.lists;
        p.plane = Packed(K, bits, group_size, true).plane(std::min(kLoraTile, M - m));
        p.M = std::min(kLoraTile, M - m);
        p.N = N;
        p.K = K;
        p.L = n_adapters;
        p.R = rank;
        p.Rp = pad_rank(rank);
        p.pieces = shrink_pieces(K);
        p.log_parts = __builtin_ctz(parts_of(K * bits / 128));
        p.yf32 = y_dt == QMV_DT_F32;
        p.adf16 = ad_dt == QMV_DT_F16;
        if (shrink_launch(p, bits, group_size, xf32, st)) return QMV_E_LAUNCH;
        // Row and token tiles of a wave: the fewest whose waves all fit at once, two per
        // SIMD.  More tiles read codes and activations less often, but a second round of
        // waves costs more, and idle SIMDs most.  Cold, us, one, two and four token tiles
        // of two row tiles each (waves of one): 32 tokens, 3840 x 15360 (1920) 27.8, 35.5;
        // 15360 x 3840 (3840), two and four: 26.5, 30.1; 64 tokens, 2048 x 2048 (512)
        // 13.8, 22.1, 31.8; 3840 x 15360 (3840) 43.4, 35.1, 47.4; 15360 x 3840 (7680), two
        // and four: 42.3, 35.4.  One and two row tiles, 13 tokens: 4096 x 12288 (2048
        // waves of one) 19.3, 21.7; 4608 x 12288 (2304) 29.6, 22.0; 15360 x 3840
        // (3840) 22.5, 19.2.  The hidden values of
        // the tokens have to fit the shared memory (52 KB of them beside 90 of the rest
        // at most).  Rows that are not cut into parts, short ones, have a wave per row tile.
        constexpr int kFit = 2048;
        const bool whole = p.log_parts == 0;
        const int tiles = (p.M + 15) / 16, waves = (N + 31) / 32 << p.log_parts, most = p.Rp > 256 ? 1 : p.Rp > 128 ? 2 : 4;
        const int fewest = whole || tiles == 1 || waves * tiles <= kFit ? 1 : tiles == 2 || waves * ((tiles + 1) / 2) <= kFit ? 2 : 4;
        const int ct = std::min(fewest, most), rt = !whole && ((N + 15) / 16 << p.log_parts) * tiles > kFit ? 2 : 1;
        const int bad = bits == 4 ? (group_size == 64 ? lora_launch_b4_g64(p, rt, ct, xf32, sbf, st)
                                                      : lora_launch_b4_g128(p, rt, ct, xf32, sbf, st))
                                  : (group_size == 64 ? lora_launch_b2_g64(p, rt, ct, xf32, sbf, st)
                                                      : lora_launch_b2_g128(p, rt, ct, xf32, sbf, st));
        if (bad) return QMV_E_LAUNCH;
    }
    return QMV_OK;
}

}  // extern "C"
