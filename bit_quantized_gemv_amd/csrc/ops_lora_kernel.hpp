// ops_lora_kernel.hpp -- the second kernel of the adapted projection: the
// quantized product and, in its epilogue, the adapters' second product.
#pragma once
#include <type_traits>

#include "ops_lora.hpp"
#include "ops_tile.hpp"

namespace ops {

// Eight values of a row of B_a at r.., zero past the rank.  Ranks that are a
// multiple of 8 have aligned rows: raw8 is a load, and trim8 clears what is past
// the rank when it is used; others are read value by value.
__device__ __forceinline__ u32x4 raw8(const uint16_t* row, int r, int R)
{
    return *reinterpret_cast<const u32x4*>(row + min(r, R - 8));
}

__device__ __forceinline__ u32x4 trim8(u32x4 v, int r, int R)
{
#pragma unroll
    for (int d = 0; d < 4; ++d) v[d] = r < R ? v[d] : 0;
    return v;
}

__device__ __forceinline__ u32x4 slow8(const uint16_t* row, int r, int R)
{
    uint32_t x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = row[min(r + i, R - 1)];
    u32x4 v;
#pragma unroll
    for (int d = 0; d < 4; ++d)
        v[d] = (r + 2 * d < R ? x[2 * d] : 0) | (r + 2 * d + 1 < R ? x[2 * d + 1] << 16 : 0);
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

constexpr int kFactorTurn = 16 * 9 * 16;       // bytes of LDS per wave to turn a unit's factors over

// LDS of the kernel, in bytes: the scales and biases; the slabs being turned over,
// the factors being turned over and the hidden values in three bf16 planes, and in
// the place of all three, when they are done with, the waves' partial results; the
// adapters' terms of the workgroup's row tiles.
struct LoraSpace {
    int biases, turn, factors, hidden, delta, bytes;
    __host__ __device__ LoraSpace(const Meta& meta, int waves, int groups, int rt, int ct, int Rp)
    {
        const int tiles = groups * rt, tokens = 16 * ct;
        biases = meta.bytes(16 * tiles) / 2;
        turn = 2 * biases;
        factors = turn + waves * rt * 1024;
        hidden = factors + waves * kFactorTurn;
        const int join = turn + ct * waves * rt * Join<1>::kWords * 4, end = hidden + 3 * tokens * (Rp + 8) * 2;
        delta = join > end ? join : end;
        bytes = delta + tiles * tokens * 64;
    }
};

// One workgroup per groups of 16 * RT rows and 16 * CT tokens; the waves of a
// group each sum a part of K.  What does not depend on another load is asked for
// first: the first slabs of codes and activations, and by way of the list of
// adapters the first of their factors and the hidden values, which go to LDS.  The
// adapters' terms follow the product, their factors streaming through a ring of
// registers that the product has left.  15360 x 3840, one token, rank 16: 13.4 us,
// 34 MB at 2.5 TB/s: 1.6 us before a wave's first load, 3.0 until it is there, 5.0 of
// products, 2.0 of the adapters, join and store, and 2-3 between the first wave's start and
// the last one's.  (qmv_affine's kernel, without adapters, takes 8.2 over this matrix.)  17408 x 5120, 64 tokens
// of 32 adapters, rank 64: 81 us, 140 TFLOP/s, 134 MB, bound by the decoding of codes
// beside the matrix instructions, the 71 MB of factors, and a second round of 32
// workgroups behind the 512 that fit.
template <class T>
__global__ __launch_bounds__(kMaxWaves* kWave, T::WAVES) void lora_kernel(LoraParams p)
{
    constexpr int RT = T::RT, CT = T::CT, DEPTH = 4;
    using J = Join<RT>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    together(p.w, p.s, p.b, p.y, p.lb, p.h, p.lists, p.xp, p.plane, p.M, p.N, p.K, p.R, p.Rp, p.pieces, p.log_parts, p.meta.groups,
             p.meta.window, p.meta.windows);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 15, q = lane >> 4;
    const int lp = p.log_parts, parts = 1 << lp, waves = waves_of(parts), groups = waves >> lp, tiles = groups * RT;      // powers of two
    const int first = blockIdx.x * tiles * 16, m0 = blockIdx.y * 16 * CT, tokens = min(16 * CT, p.M - m0);
    const int n0 = first + (wave >> lp) * RT * 16, part = wave & (parts - 1), rows = min(16 * tiles, p.N - first);
    const Meta& meta = p.meta;
    const LoraSpace sp(meta, waves, groups, RT, CT, p.Rp);
    uint16_t* const scales = reinterpret_cast<uint16_t*>(lds);
    uint16_t* const biases = reinterpret_cast<uint16_t*>(lds + sp.biases);
    float* const join = reinterpret_cast<float*>(lds + sp.turn);
    float* const delta = reinterpret_cast<float*>(lds + sp.delta);
    char* const hidden = lds + sp.hidden;
    const int hrow = (p.Rp + 8) * 2, hplane = 16 * CT * hrow;

    typename T::Rows r;
    r.G = p.K / T::GS;
    r.chunks = p.K / (4 * T::VPW);
    r.plane = p.plane;
    r.turn = lds + sp.turn + wave * T::TURN;
    r.even = meta.groups % T::NG == 0;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int row = min(n0 + 16 * i, p.N - 1);          // rows past the last repeat it and are not stored
        T::set_codes(r, i, p.w, row, p.N - row);
        const int at = min(n0 - first + 16 * i + c, rows - 1) * meta.groups;
        r.s[i] = scales + at;
        r.b[i] = biases + at;
    }
#pragma unroll
    for (int j = 0; j < CT; ++j) T::set_token(r, j, p.xp, min(m0 + 16 * j + c, p.M - 1));
    const int slabs = slabs_of(r.chunks), s0 = part_start(slabs, lp, part), s1 = part_start(slabs, lp, part + 1);
    typename T::Ring ring;
    int a0 = s0, a1 = min(s0 + meta.window, s1);
    const bool active = n0 < p.N;
    MetaCopy<4> copy(p.s + (size_t)first * r.G, p.b + (size_t)first * r.G, rows, r.G, kWave * waves);
    if (meta.windows == 1) {
        copy.ask();
    } else {
        stage_window(scales, copy.s, rows, r.G, T::NG, slabs, parts, meta.window, 0, kWave * waves);
        stage_window(biases, copy.b, rows, r.G, T::NG, slabs, parts, meta.window, 0, kWave * waves);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            r.s[i] += (part * meta.window - a0) * T::NG;
            r.b[i] += (part * meta.window - a0) * T::NG;
        }
    }
    keep_order();
    T::begin(ring, r, a0, a1);

    // The adapters' terms.  A wave has one row tile, and takes every so many of the
    // block's adapters in turn.  An adapter's product is computed on whole tiles of 16
    // tokens and kept for its own tokens alone (other rows may hold anything), in
    // registers until the last, so every token's term has one writer and one order.
    // Lane l holds entry l of the list.
    const AdapterList& list = p.lists[m0 / kBlock];
    const int list_adapter = list.adapter[lane];
    const float list_scaling = list.scaling[lane];
    const unsigned long long list_tokens = list.tokens[lane] >> (m0 % kBlock), adapted = list.any >> (m0 % kBlock);
    const int entries = uniform(list.count), shift = __builtin_ctz(tiles), tile = wave & (tiles - 1), every = waves >> shift;
    const bool r8 = p.R % 8 == 0;
    u32x4 v[DEPTH][2];
    // A unit's factors up to rank 64 lie together: the lanes load them in order
    // and turn them over through LDS, a row's pieces at an odd stride of 16 bytes.
    const int pieces = min(p.R / 8, 8), stride = pieces | 1;
    const int tile_row = min(first + tile * 16, p.N - 1), tile_last = min(16, p.N - tile_row) - 1;   // past the last row: not stored
    const uint16_t* const tile_rows = p.lb + (size_t)tile_row * p.R;
    const size_t per_adapter = (size_t)p.N * p.R;
    int at_row[2];
    uint32_t from[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        at_row[s] = small_div(lane + 64 * s, 1.0f / (float)max(pieces, 1));
        const int piece = lane + 64 * s - at_row[s] * pieces;
        from[s] = (uint32_t)(min(at_row[s], tile_last) * p.R + piece * 8);
        at_row[s] = at_row[s] < 16 ? (at_row[s] * stride + piece) * 16 : -1;
    }
    auto entry_rows = [&](int d) { return tile_rows + __builtin_amdgcn_readlane(list_adapter, d) * per_adapter; };
    auto load_unit = [&](u32x4 (&to)[2], int d) {
        const uint16_t* rows = entry_rows(d);
#pragma unroll
        for (int s = 0; s < 2; ++s) to[s] = *reinterpret_cast<const u32x4*>(rows + from[s]);
    };
    char* const turn = lds + sp.factors + wave * kFactorTurn;
    const int d0 = wave >> shift;
    if (r8 && d0 < entries) load_unit(v[0], d0);
    if (meta.windows == 1) copy.put(scales, biases);
    if (entries > 0) {
        const int octs = p.Rp / 8;
        const float per_oct = 1.0f / (float)octs;
        for (int e = threadIdx.x; e < tokens * octs; e += kWave * waves) {
            const int t = small_div(e, per_oct), k = (e - t * octs) * 8;
            const char* hp = reinterpret_cast<const char*>(p.h + (size_t)(m0 + t) * p.Rp + k);
            const size_t piece = (size_t)p.M * p.Rp * 4;
            f32x4 lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
            for (int z0 = 0; z0 < p.pieces; z0 += 4) {
                f32x4 x[4][2];
#pragma unroll
                for (int z = 0; z < 4; ++z)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        x[z][i] = reinterpret_cast<const f32x4*>(hp + min(z0 + z, p.pieces - 1) * piece)[i];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (z0 + z < p.pieces)
#pragma unroll
                        for (int d = 0; d < 4; ++d) {
                            lo[d] += x[z][0][d];
                            hi[d] += x[z][1][d];
                        }
            }
            u32x4 o[3];
            split_f32(lo, hi, o);
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<u32x4*>(hidden + i * hplane + t * hrow + k * 2) = o[i];
        }
    }
    lds_barrier();

    f32x4 acc[RT][CT];
    T::clear(acc);
    for (int k = 1;; ++k) {
        if (active) T::run(acc, ring, r, a0, a1);
        if (k >= meta.windows) break;
        lds_barrier();
        stage_window(scales, copy.s, rows, r.G, T::NG, slabs, parts, meta.window, k, kWave * waves);
        stage_window(biases, copy.b, rows, r.G, T::NG, slabs, parts, meta.window, k, kWave * waves);
        lds_barrier();
        a0 = a1;             // a part may end a window early: nothing is left of it then
        a1 = min(a0 + meta.window, s1);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            r.s[i] -= meta.window * T::NG;
            r.b[i] -= meta.window * T::NG;
        }
        if (a0 < a1) T::begin(ring, r, a0, a1);
    }

    f32x4 term[CT];
#pragma unroll
    for (int j = 0; j < CT; ++j) term[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto unit = [&](auto aligned, const u32x4 (&raw)[2], int d) {
        constexpr bool R8 = decltype(aligned)::value;
        const uint32_t mine[2] = {(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)list_tokens, d),
                                  (uint32_t)__builtin_amdgcn_readlane((int)(list_tokens >> 32), d)};
        const float scale = bits_f32(__builtin_amdgcn_readlane(f32_bits(list_scaling), d));
        const uint16_t* const row = entry_rows(d) + (size_t)min(c, tile_last) * p.R;
        u32x4 b[2];
        if constexpr (R8) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (at_row[s] >= 0) *reinterpret_cast<u32x4*>(turn + at_row[s]) = raw[s];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int s = 0; s < 2; ++s) b[s] = *reinterpret_cast<const u32x4*>(turn + (c * stride + min(q + 4 * s, pieces - 1)) * 16);
            __builtin_amdgcn_wave_barrier();
            if (p.R < 64)
#pragma unroll
                for (int s = 0; s < 2; ++s) b[s] = trim8(b[s], 8 * q + 32 * s, p.R);
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) b[s] = slow8(row, 8 * q + 32 * s, p.R);
        }
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const uint32_t of_tile = (mine[j / 2] >> (16 * (j % 2))) & 0xffffu;
            if (of_tile == 0) continue;
            const char* hr = hidden + (16 * j + c) * hrow + 16 * q;
            f32x4 acc = {0.f, 0.f, 0.f, 0.f};
            auto step = [&](const u32x4& x, int k) {
                u32x4 xh = x, xl = x;
                if (p.adf16) split_f16(x, xh, xl);
#pragma unroll
                for (int e = 0; e < 3; ++e) {
                    const u32x4 ho = *reinterpret_cast<const u32x4*>(hr + e * hplane + 2 * k);
                    acc = mfma(ho, xh, acc);
                    if (p.adf16) acc = mfma(ho, xl, acc);
                }
            };
            step(b[0], 0);
            if (p.Rp > 32) step(b[1], 32);
            for (int k = 64; k < p.Rp; k += 32)
                step(R8 ? trim8(raw8(row, 8 * q + k, p.R), 8 * q + k, p.R) : slow8(row, 8 * q + k, p.R), k);
            const uint32_t of_lane = of_tile >> (4 * q);
#pragma unroll
            for (int e = 0; e < 4; ++e) term[j][e] = (of_lane >> e) & 1 ? scale * acc[e] : term[j][e];
        }
    };
    // Of the loop's loads none is behind a branch (a wait would then assume it was not
    // taken); the last rounds, which have fewer left to ask for, come after it.
    if (r8) {
        constexpr std::true_type aligned{};
#pragma unroll
        for (int i = 1; i < DEPTH; ++i)
            if (d0 + i * every < entries) load_unit(v[i], d0 + i * every);
        int d = d0;
        for (; d + (2 * DEPTH - 1) * every < entries; d += DEPTH * every) {
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                const u32x4 raw[2] = {v[i][0], v[i][1]};
                load_unit(v[i], d + (i + DEPTH) * every);
                keep_order();
                unit(aligned, raw, d + i * every);
            }
        }
        for (; d < entries; d += DEPTH * every) {
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                const int at = d + i * every, next = at + DEPTH * every;
                if (at < entries) {
                    const u32x4 raw[2] = {v[i][0], v[i][1]};
                    if (next < entries) load_unit(v[i], next);
                    unit(aligned, raw, at);
                }
            }
        }
    } else {
        for (int d = d0; d < entries; d += every) unit(std::false_type{}, v[0], d);
    }
    // tokens of this wave's adapters
    if (d0 < entries) {
        const unsigned long long of_wave = lane < entries && (lane & (every - 1)) == d0 ? list_tokens : 0;
        uint32_t lo = (uint32_t)of_wave, hi = (uint32_t)(of_wave >> 32);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            lo |= __shfl_xor((int)lo, o);
            hi |= __shfl_xor((int)hi, o);
        }
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const uint32_t of_lane = ((j < 2 ? lo : hi) >> (16 * (j % 2))) >> (4 * q);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if ((of_lane >> e) & 1) delta[(tile * 16 * CT + 16 * j + 4 * q + e) * 16 + c] = term[j][e];
        }
    }

    lds_barrier();        // from here the join has the place of what came before
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int i = 0; i < RT; ++i) J::write(join + j * waves * J::kWords, wave, lane, i, acc[i][j]);
    lds_barrier();
    const int log_rows = 4 + shift;
    for (int e = threadIdx.x; e < tokens << log_rows; e += kWave * waves) {
        const int en = e & (16 * tiles - 1), t = e >> log_rows, n = first + en;
        if (n < p.N) {
            const int group = en / (16 * RT);
            float y = J::sum(join + (t >> 4) * waves * J::kWords, group * parts, parts, J::at(en % (16 * RT), t & 15));
            if ((adapted >> t) & 1) y += delta[((en >> 4) * 16 * CT + t) * 16 + (en & 15)];
            store_y(p.y, (size_t)(m0 + t) * p.N + n, y, p.yf32);
        }
    }
}

template <class T>
int lora_start(const LoraParams& p, hipStream_t st)
{
    const int parts = 1 << p.log_parts, waves = waves_of(parts), groups = waves / parts, rows = groups * 16 * T::RT;
    const dim3 grid((p.N + rows - 1) / rows, (p.M + 16 * T::CT - 1) / (16 * T::CT));
    LoraParams q = p;
    q.meta = Meta(rows, p.K, T::BITS, T::GS, parts);
    const LoraSpace sp(q.meta, waves, groups, T::RT, T::CT, p.Rp);
    const void* fn = reinterpret_cast<const void*>(&lora_kernel<T>);
    if (sp.bytes > 64 * 1024 &&
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, sp.bytes) != hipSuccess)
        return 1;
    void* args[] = {&q};
    return hipLaunchKernel(fn, grid, dim3(kWave * waves), args, sp.bytes, st) == hipSuccess ? 0 : 1;
}

template <int BITS, int GS, int RT, int CT, int NP>
int lora_scales(const LoraParams& p, bool sbf, hipStream_t st)
{
    return sbf ? lora_start<Tile<BITS, GS, RT, CT, NP, true, true>>(p, st) : lora_start<Tile<BITS, GS, RT, CT, NP, false, true>>(p, st);
}

// Token tiles per wave: as many as asked for and the registers hold.  Some of the rarer
// instances spill: 67 registers of two row tiles of 2-bit codes in groups of 64 and fp32
// activations (64 tokens, 15360 x 3840: 79 us, 58 in groups of 128, which do not), 33 of two
// token tiles of such codes and bf16, 16 to 24 of two token tiles of 4-bit codes and fp32.
template <int BITS, int GS>
int lora_pick(const LoraParams& p, int rt, int ct, bool xf32, bool sbf, hipStream_t st)
{
    if (xf32) {
        if constexpr (BITS == 4)
            if (ct > 1) return lora_scales<BITS, GS, 2, 2, 3>(p, sbf, st);
        return rt == 1 ? lora_scales<BITS, GS, 1, 1, 3>(p, sbf, st) : lora_scales<BITS, GS, 2, 1, 3>(p, sbf, st);
    }
    if constexpr (BITS == 4)
        if (ct == 4) return lora_scales<BITS, GS, 2, 4, 1>(p, sbf, st);
    if (ct > 1) return lora_scales<BITS, GS, 2, 2, 1>(p, sbf, st);
    return rt == 1 ? lora_scales<BITS, GS, 1, 1, 1>(p, sbf, st) : lora_scales<BITS, GS, 2, 1, 1>(p, sbf, st);
}

}  // namespace ops
