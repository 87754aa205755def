// ops_lora_kernel.hpp -- the second kernel of the adapted projection: the
// quantized product and, in its epilogue, the adapters' second product.
#pragma once
#include "ops_lora.hpp"
#include "ops_tile.hpp"

namespace ops {

// Eight values of a row of B_a at r.. as bf16 operands: one piece, or two for
// fp16 (8 + 3 bits).  Ranks that are no multiple of 8 have unaligned rows and are read
// value by value.
__device__ __forceinline__ u32x4 load8(const uint16_t* row, int r, int R)
{
    if (r >= R) return u32x4{0, 0, 0, 0};
    if ((R & 7) == 0) return *reinterpret_cast<const u32x4*>(row + r);
    u32x4 v;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t a = r + 2 * d < R ? row[r + 2 * d] : 0, b = r + 2 * d + 1 < R ? row[r + 2 * d + 1] : 0;
        v[d] = a | (b << 16);
    }
    return v;
}

// eight fp16 values as two bf16 pieces
__device__ __forceinline__ void split_f16(const u32x4& v, u32x4& h, u32x4& l)
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const float a = half_bits(v[d] & 0xffffu), b = half_bits(v[d] >> 16);
        const uint32_t ah = f32_bits(a) & 0xffff0000u, bh = f32_bits(b) & 0xffff0000u;
        h[d] = hi16(ah, bh);
        l[d] = hi16(f32_bits(a - bits_f32(ah)), f32_bits(b - bits_f32(bh)));
    }
}

// eight fp32 values as three bf16 pieces
__device__ __forceinline__ void split_f32(const f32x4& lo, const f32x4& hi, u32x4 (&o)[3])
{
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const float a = d < 2 ? lo[2 * d] : hi[2 * d - 4], b = d < 2 ? lo[2 * d + 1] : hi[2 * d - 3];
        uint32_t ah, am, al, bh, bm, bl;
        split3(a, ah, am, al);
        split3(b, bh, bm, bl);
        o[0][d] = hi16(ah, bh);
        o[1][d] = hi16(am, bm);
        o[2][d] = hi16(al, bl);
    }
}

template <class T>
__global__ __launch_bounds__(kMaxWaves* kWave) void lora_kernel(LoraParams p)
{
    constexpr int RT = T::RT, CT = T::CT;
    using J = Join<RT>;
    __shared__ float join[kMaxWaves * J::kWords];
    __shared__ float delta[J::kWords];

    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int c = lane & 15, q = lane >> 4;
    const int n0 = blockIdx.x * 16 * RT, m0 = blockIdx.y * 16 * CT;

    typename T::Rows r;
    r.K = p.K;
    r.G = p.K / T::GS;
    r.chunks = p.K / (4 * T::VPW);
    r.meta_al = r.G % T::NG == 0;
    const uint16_t* lb_row[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const size_t n = min(n0 + 16 * i + c, p.N - 1);     // rows past the last repeat it and are not stored
        r.w[i] = reinterpret_cast<const u32x4*>(p.w) + n * r.chunks;
        r.s[i] = p.s + n * r.G;
        r.b[i] = p.b + n * r.G;
        lb_row[i] = p.lb + n * p.R;
    }
#pragma unroll
    for (int j = 0; j < CT; ++j)
        r.x[j] = p.x + (size_t)min(m0 + 16 * j + c, p.M - 1) * p.K * (T::XF32 ? 4 : 2);

    f32x4 acc[RT][CT];
    T::clear(acc);
    const int n = slabs_of(r.chunks);
    T::run(acc, r, wave * n / waves, (wave + 1) * n / waves, q);

    const size_t lb_adapter = (size_t)p.N * p.R;
#pragma unroll
    for (int j = 0; j < CT; ++j) {
        const int mj = m0 + 16 * j;
        if (mj >= p.M) break;
#pragma unroll
        for (int i = 0; i < RT; ++i) J::write(join, wave, lane, i, acc[i][j]);

        // The adapters of these 16 tokens, the waves taking them in turn.  An
        // adapter's product is computed on all 16 tokens with the others'
        // hidden values zero, and written for its own alone, so every token's
        // term has one writer and one order.
        const int mine = p.ids[min(mj + c, p.M - 1)];
        const bool has = mj + c < p.M && mine >= 0 && mine < p.L;
        uint32_t left = (uint32_t)__ballot(has) & 0xffffu;
        for (int d = 0; left != 0; ++d) {
            const int a = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
            const bool in = has && mine == a;
            const uint32_t same = (uint32_t)__ballot(in) & 0xffffu;
            left &= ~same;
            if (d % waves != wave) continue;
            f32x4 acc2[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) acc2[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            const float* hrow = p.h + (size_t)min(mj + c, p.M - 1) * p.Rp;
            for (int k = 8 * q; k < p.Rp; k += 32) {
                f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
                if (in)
                    for (int z = 0; z < p.pieces; ++z) {
                        const f32x4* hp = reinterpret_cast<const f32x4*>(hrow + (size_t)z * p.M * p.Rp + k);
                        const f32x4 l4 = hp[0], h4 = hp[1];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            lo[e] += l4[e];
                            hi[e] += h4[e];
                        }
                    }
                u32x4 ho[3];
                split_f32(lo, hi, ho);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const u32x4 v = load8(lb_row[i] + (size_t)a * lb_adapter, k, p.R);
                    if (p.adf16) {
                        u32x4 vh, vl;
                        split_f16(v, vh, vl);
#pragma unroll
                        for (int e = 0; e < 3; ++e) acc2[i] = mfma(ho[e], vl, mfma(ho[e], vh, acc2[i]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 3; ++e) acc2[i] = mfma(ho[e], v, acc2[i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if ((same >> (4 * q + e)) & 1) delta[i * J::kTile + e * 64 + lane] = acc2[i][e];
        }
        __syncthreads();
        for (int e = threadIdx.x; e < 256 * RT; e += blockDim.x) {
            const int en = e % (16 * RT), et = e / (16 * RT);
            if (n0 + en < p.N && mj + et < p.M) {
                float v = J::sum(join, waves, J::at(en, et));
                const int a = p.ids[mj + et];
                if (a >= 0 && a < p.L)
                    v = __builtin_fmaf(p.scaling ? p.scaling[a] : 1.0f, delta[J::at(en, et)], v);
                store_y(p.y, (size_t)(mj + et) * p.N + n0 + en, v, p.yf32);
            }
        }
        if (j + 1 < CT) __syncthreads();
    }
}

template <class T>
int lora_start(const LoraParams& p, hipStream_t st)
{
    const dim3 grid((p.N + 16 * T::RT - 1) / (16 * T::RT), (p.M + 16 * T::CT - 1) / (16 * T::CT));
    LoraParams q = p;
    void* args[] = {&q};
    return hipLaunchKernel(reinterpret_cast<const void*>(&lora_kernel<T>), grid,
                           dim3(kWave * waves_of(p.K / (4 * T::VPW))), args, 0, st) == hipSuccess
               ? 0
               : 1;
}

template <int BITS, int GS, int RT, int CT>
int lora_types(const LoraParams& p, bool xf32, bool sbf, hipStream_t st)
{
    if (xf32) {
        constexpr int C = CT > 2 ? 2 : CT;     // three pieces of four token tiles do not fit the registers
        return sbf ? lora_start<Tile<BITS, GS, RT, C, true, true>>(p, st)
                   : lora_start<Tile<BITS, GS, RT, C, true, false>>(p, st);
    }
    return sbf ? lora_start<Tile<BITS, GS, RT, CT, false, true>>(p, st)
               : lora_start<Tile<BITS, GS, RT, CT, false, false>>(p, st);
}

template <int BITS, int GS>
int lora_pick(const LoraParams& p, int rt, int ct, bool xf32, bool sbf, hipStream_t st)
{
    if (ct == 1) {
        if (rt == 1) return lora_types<BITS, GS, 1, 1>(p, xf32, sbf, st);
        if (rt == 2) return lora_types<BITS, GS, 2, 1>(p, xf32, sbf, st);
        return lora_types<BITS, GS, 4, 1>(p, xf32, sbf, st);
    }
    if (ct == 2) {
        if (rt == 1) return lora_types<BITS, GS, 1, 2>(p, xf32, sbf, st);
        if (rt == 2) return lora_types<BITS, GS, 2, 2>(p, xf32, sbf, st);
        return lora_types<BITS, GS, 4, 2>(p, xf32, sbf, st);
    }
    if (rt == 1) return lora_types<BITS, GS, 1, 4>(p, xf32, sbf, st);
    if (rt == 2) return lora_types<BITS, GS, 2, 4>(p, xf32, sbf, st);
    return lora_types<BITS, GS, 4, 4>(p, xf32, sbf, st);
}

}  // namespace ops
