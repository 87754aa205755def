// ops_moe_kernel.hpp -- the two products of the experts.
//
// A workgroup takes one expert and 16 gate rows with their 16 up rows (or 16
// rows of the down product), collects the (token, slot) pairs that chose the
// expert, and multiplies their activations 16 * CT at a time.  With few tokens
// every chosen expert's weights are read once and bound the time.
#pragma once
#include "ops_moe.hpp"
#include "ops_tile.hpp"

namespace ops {

constexpr int kMaxPairs = kMoeTile * 32;

// The expert of this workgroup and its pairs in ascending order, in `list`;
// their count, or 0 if another workgroup takes them.  All threads.
__device__ __forceinline__ int collect(const ExpertParams& p, int slot, int& e, uint16_t* list, int* count)
{
    e = p.slots == p.P ? p.ids[slot] : slot;
    if (e < 0 || e >= p.E) return 0;
    if (threadIdx.x < kWave) {
        const int lane = threadIdx.x;
        int n = 0;
        for (int base = 0; base < p.P; base += 4 * kWave) {
            int id[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = base + i * kWave + lane;
                id[i] = at < p.P ? p.ids[at] : -1;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned long long hit = __ballot(id[i] == e);
                const int before = __popcll(hit & ((1ull << lane) - 1));
                if (id[i] == e) list[n + before] = (uint16_t)(base + i * kWave + lane);
                n += __popcll(hit);
            }
        }
        if (lane == 0) *count = n;
    }
    __syncthreads();
    const int n = *count;
    return n > 0 && p.slots == p.P && list[0] != slot ? 0 : n;
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// GATE: T::RT = 2 row tiles, the gate rows and the up rows
template <class T, bool GATE>
__global__ __launch_bounds__(kMaxWaves* kWave) void expert_kernel(ExpertParams p)
{
    constexpr int RT = T::RT, CT = T::CT;
    using J = Join<RT>;
    __shared__ float join[kMaxWaves * J::kWords];
    __shared__ uint16_t list[kMaxPairs];
    __shared__ int count;

    int e;
    const int n = uniform(collect(p, blockIdx.y, e, list, &count));
    if (n == 0) return;

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int c = lane & 15, q = lane >> 4;
    const int K = GATE ? p.D : p.F, N = GATE ? p.F : p.D;   // N is a multiple of 64
    const int n0 = blockIdx.x * 16 * (GATE ? 1 : RT);
    typename T::Rows r;
    r.K = K;
    r.G = K / T::GS;
    r.chunks = K / (4 * T::VPW);
    r.meta_al = r.G % T::NG == 0;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const size_t row = GATE ? (size_t)e * 2 * N + (size_t)i * N + n0 + c : (size_t)e * N + n0 + 16 * i + c;
        r.w[i] = reinterpret_cast<const u32x4*>(GATE ? p.w13 : p.w2) + row * r.chunks;
        r.s[i] = (GATE ? p.s13 : p.s2) + row * r.G;
        r.b[i] = (GATE ? p.b13 : p.b2) + row * r.G;
    }
    const int slabs = slabs_of(r.chunks);
    for (int t0 = 0; t0 < n; t0 += 16 * CT) {
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int pair = list[min(t0 + 16 * j + c, n - 1)];
            r.x[j] = GATE ? p.x + (size_t)(pair / p.k) * K * (T::XF32 ? 4 : 2)
                          : reinterpret_cast<const char*>(p.h + (size_t)pair * K);
        }
        f32x4 acc[RT][CT];
        T::clear(acc);
        T::run(acc, r, wave * slabs / waves, (wave + 1) * slabs / waves, q);
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            if (t0 + 16 * j >= n) break;
#pragma unroll
            for (int i = 0; i < RT; ++i) J::write(join, wave, lane, i, acc[i][j]);
            __syncthreads();
            constexpr int ROWS = GATE ? 16 : 16 * RT;
            for (int i = threadIdx.x; i < 16 * ROWS; i += blockDim.x) {
                const int en = i % ROWS, et = i / ROWS;
                if (t0 + 16 * j + et < n) {
                    const size_t pair = list[t0 + 16 * j + et];
                    const float v = J::sum(join, waves, J::at(en, et));
                    if constexpr (GATE)
                        p.h[pair * N + n0 + en] = silu(v) * J::sum(join, waves, J::at(16 + en, et));
                    else
                        p.z[pair * N + n0 + en] = v;
                }
            }
            __syncthreads();
        }
    }
}

template <class T, bool GATE>
int expert_start(const ExpertParams& p, hipStream_t st)
{
    const int K = GATE ? p.D : p.F, rows = GATE ? p.F : p.D;
    ExpertParams q = p;
    void* args[] = {&q};
    return hipLaunchKernel(reinterpret_cast<const void*>(&expert_kernel<T, GATE>),
                           dim3(rows / (16 * (GATE ? 1 : T::RT)), p.slots), dim3(kWave * waves_of(K / (4 * T::VPW))),
                           args, 0, st) == hipSuccess
               ? 0
               : 1;
}

template <int BITS, int GS, bool SBF>
int expert_pick(int which, const ExpertParams& p, int ct, bool xf32, hipStream_t st)
{
    if (which == 1)
        return ct == 1 ? expert_start<Tile<BITS, GS, 2, 1, true, SBF>, false>(p, st)
                       : expert_start<Tile<BITS, GS, 2, 2, true, SBF>, false>(p, st);
    if (xf32)
        return ct == 1 ? expert_start<Tile<BITS, GS, 2, 1, true, SBF>, true>(p, st)
                       : expert_start<Tile<BITS, GS, 2, 2, true, SBF>, true>(p, st);
    return ct == 1 ? expert_start<Tile<BITS, GS, 2, 1, false, SBF>, true>(p, st)
                   : expert_start<Tile<BITS, GS, 2, 2, false, SBF>, true>(p, st);
}

}  // namespace ops
