// ops_moe_kernel.hpp -- the two products of the experts.
//
// A workgroup takes one expert and, for each group of its waves, 16 gate rows with
// their 16 up rows (or 32 rows of the down product), finds the (token, slot) pairs
// that chose the expert, and multiplies their activations 16 * CT at a time.  With
// few tokens every chosen expert's weights are read once and bound the time.  Where
// an expert meets many pairs, they have been sorted by expert, in tiles of 16 whose
// activations lie in the order of the lanes (FRAG): gathered row by row, each of a
// wave's activation loads would look up a cache line per lane.
//
// 13 tokens over 128 experts of 2048 x 1024, 8 each: gate and up 46 us, 159 MB at 3.5
// TB/s; down 42 us, 84 MB at 2.0, whose rows are eight slabs: a wave is mostly its
// start and end.  128 tokens over 32 experts of 3840 x 1920, 4 each, 2-bit: 69 us, 219
// TFLOP/s, and 75 us, 101 (three planes of hidden values: three times the matrix
// instructions), bound by the decoding of codes beside the matrix instructions.
#pragma once
#include <algorithm>

#include "ops_moe.hpp"
#include "ops_tile.hpp"

namespace ops {

constexpr int kMaxPairs = kMoeTile * 32;

// The pairs that chose expert e, in ascending order: their count, and whether the
// first of them is `slot`.  Every wave by itself; the first wave writes the list.
struct Found {
    int n;
    bool first;
};

__device__ __forceinline__ Found find_pairs(const int32_t* ids, int P, int e, int slot, uint16_t* list)
{
    const int lane = threadIdx.x & 63;
    const bool writes = threadIdx.x < kWave;
    int n = 0, lowest = -1;
    for (int base = 0; base < P; base += 4 * kWave) {
        int id[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = base + i * kWave + lane;
            const int v = ids[min(at, P - 1)];
            id[i] = at < P ? v : -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned long long hit = __ballot(id[i] == e);
            if (lowest < 0 && hit != 0) lowest = base + i * kWave + __builtin_ctzll(hit);
            if (writes && id[i] == e) list[n + __popcll(hit & ((1ull << lane) - 1))] = (uint16_t)(base + i * kWave + lane);
            n += __popcll(hit);
        }
    }
    return {uniform(n), uniform(lowest) == slot};
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

struct ExpertSpace {
    int biases, turn, list, bytes;
    __host__ __device__ ExpertSpace(const Meta& meta, int waves, int rows, int P)
    {
        biases = meta.bytes(rows) / 2;
        turn = 2 * biases;
        list = turn + waves * 2 * Join<1>::kWords * 4;
        bytes = list + (P * 2 + 15) / 16 * 16;
    }
};

// GATE: T::RT = 2 row tiles, the gate rows and the up rows
template <class T, bool GATE>
__global__ __launch_bounds__(kMaxWaves* kWave, T::WAVES) void expert_kernel(ExpertParams p)
{
    constexpr int RT = 2, CT = T::CT;
    static_assert(T::RT == RT, "");
    using J = Join<RT>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    together(p.ids, GATE ? p.w13 : p.w2, GATE ? p.s13 : p.s2, GATE ? p.b13 : p.b2, GATE ? p.xp : p.h, GATE ? p.x_plane : p.h_plane,
             p.P, p.D, p.F, p.E, p.slots, p.takers, p.log_parts, p.groups, p.meta.groups, p.meta.window, p.meta.windows, p.per_k);
    const int slot = blockIdx.y;
    const bool by_pair = p.slots == p.P;
    const int e = by_pair ? p.ids[slot] : slot;
    if (e < 0 || e >= p.E) return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int c = lane & 15, lp = p.log_parts, parts = 1 << lp, groups = p.groups, waves = groups << lp, threads = kWave * waves;
    const int group = wave >> lp, part = wave & (parts - 1);
    const int K = GATE ? p.D : p.F, N = GATE ? p.F : p.D;
    constexpr int ROWS = GATE ? 16 : 32;                             // outputs of a group
    const int left = ROWS * groups, first = blockIdx.x * left;       // N is a multiple of the workgroup's rows
    const Meta& meta = p.meta;
    const ExpertSpace sp(meta, waves, 32 * groups, p.P);
    uint16_t* const scales = reinterpret_cast<uint16_t*>(lds);
    uint16_t* const biases = reinterpret_cast<uint16_t*>(lds + sp.biases);
    float* const join = reinterpret_cast<float*>(lds + sp.turn);
    uint16_t* const list = reinterpret_cast<uint16_t*>(lds + sp.list);

    int n, base = 0;
    if constexpr (T::FRAG) {
        n = p.count[e];
        base = p.base[e] * 16;
    } else {
        const Found found = find_pairs(p.ids, p.P, e, slot, list);
        n = by_pair && !found.first ? 0 : found.n;
    }
    // the pairs 16 * CT at a time, in turn with the workgroups of the same rows
    const int mine = 16 * CT * blockIdx.z, next = 16 * CT * p.takers;
    if (mine >= n) return;
    // the row of the expert's pair number t
    auto row_of = [&](int t) { return T::FRAG ? base + t : (int)list[t]; };

    // LDS rows: GATE: the groups' gate rows, then their up rows
    typename T::Rows r;
    r.G = K / T::GS;
    r.chunks = K / (4 * T::VPW);
    r.plane = GATE ? p.x_plane : p.h_plane;
    r.turn = lds + sp.turn + wave * T::TURN;
    r.even = meta.groups % T::NG == 0;
    const size_t row0 = (size_t)e * (GATE ? 2 * N : N);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        T::set_codes(r, i, GATE ? p.w13 : p.w2, row0 + first + group * ROWS + (GATE ? (size_t)i * N : 16 * i), 16);
        const int at = (GATE ? i * left + group * 16 : group * 32 + 16 * i) + c;
        r.s[i] = scales + at * meta.groups;
        r.b[i] = biases + at * meta.groups;
    }
    const uint16_t* const ms = (GATE ? p.s13 : p.s2) + (row0 + first) * r.G;
    const uint16_t* const mb = (GATE ? p.b13 : p.b2) + (row0 + first) * r.G;
    const size_t up = (size_t)N * r.G;
    const int slabs = slabs_of(r.chunks), s0 = part_start(slabs, lp, part), s1 = part_start(slabs, lp, part + 1);
    MetaCopy<GATE ? 1 : 4> copy(ms, mb, left, r.G, threads), copy_up(ms + (GATE ? up : 0), mb + (GATE ? up : 0), left, r.G, threads);
    const int half = 16 * groups * meta.groups;       // the up rows' place
    auto stage = [&](int k) {
        stage_window(scales, ms, left, r.G, T::NG, slabs, parts, meta.window, k, threads);
        stage_window(biases, mb, left, r.G, T::NG, slabs, parts, meta.window, k, threads);
        if (GATE) {
            stage_window(scales + half, ms + up, left, r.G, T::NG, slabs, parts, meta.window, k, threads);
            stage_window(biases + half, mb + up, left, r.G, T::NG, slabs, parts, meta.window, k, threads);
        }
    };
    int shifted = 0;
    auto shift = [&](int to) {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            r.s[i] += (to - shifted) * T::NG;
            r.b[i] += (to - shifted) * T::NG;
        }
        shifted = to;
    };
    if (meta.windows == 1) {
        copy.ask();
        if (GATE) copy_up.ask();
        keep_order();
    }
    const Packed pk(p.F, T::BITS, T::GS, T::FRAG);
    typename T::Ring ring;
    auto begin = [&](int t0) {
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int row = row_of(min(t0 + 16 * j + c, n - 1));
            T::set_token(r, j, GATE ? p.xp : p.h, GATE && !T::FRAG ? small_div(row, p.per_k) : row);
        }
        if (meta.windows == 1) T::begin(ring, r, min(s0, s1 - 1), max(s1, s0 + 1));
    };
    if constexpr (!T::FRAG) lds_barrier();      // the list is there
    begin(mine);
    if (meta.windows == 1) {
        copy.put(scales, biases);
        if (GATE) copy_up.put(scales + half, biases + half);
    }
    lds_barrier();
    for (int t0 = mine; t0 < n; t0 += next) {
        f32x4 acc[RT][CT];
        T::clear(acc);
        for (int k = 0; k < meta.windows; ++k) {
            const int a0 = min(s0 + k * meta.window, s1), a1 = min(a0 + meta.window, s1);
            if (meta.windows > 1) {
                lds_barrier();
                stage(k);
                lds_barrier();
                shift((part - k) * meta.window - s0);
                T::begin(ring, r, min(a0, s1 - 1), max(a1, s0 + 1));
            }
            T::run(acc, ring, r, a0, a1);
        }
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            if (t0 + 16 * j >= n) break;
            lds_barrier();          // the turning space is the join's from here
#pragma unroll
            for (int i = 0; i < RT; ++i) J::write(join, wave, lane, i, acc[i][j]);
            lds_barrier();
            if constexpr (GATE) {
                // two hidden values at a time, those that a dword of codes meets
                constexpr int H = T::VPW / 2;
                for (int i = threadIdx.x; i < 128 * groups; i += threads) {
                    const int et = i & 15, d = (i >> 4) & 7, g = i >> 7;
                    if (t0 + 16 * j + et < n) {
                        const int word = d / H, ii = d % H, en = word * T::VPW + ii;
                        float v[2];
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            v[b] = silu(J::sum(join, g * parts, parts, J::at(en + b * H, et))) *
                                   J::sum(join, g * parts, parts, J::at(16 + en + b * H, et));
                        uint32_t ah, am, al, bh, bm, bl;
                        split3(v[0], ah, am, al);
                        split3(v[1], bh, bm, bl);
                        char* to = p.h + pk.word(row_of(t0 + 16 * j + et), (first + g * 16) / T::VPW + word) + (ii / 4) * pk.op_step() + (ii % 4) * 4;
                        *reinterpret_cast<uint32_t*>(to) = hi16(ah, bh);
                        *reinterpret_cast<uint32_t*>(to + p.h_plane) = hi16(am, bm);
                        *reinterpret_cast<uint32_t*>(to + 2 * p.h_plane) = hi16(al, bl);
                    }
                }
            } else {
                for (int i = threadIdx.x; i < 16 * 32 * groups; i += threads) {
                    const int en = i & 31, g = (i >> 5) & (groups - 1), et = small_div(i >> 5, 1.0f / (float)groups);
                    if (t0 + 16 * j + et < n)
                        p.z[(size_t)row_of(t0 + 16 * j + et) * N + first + g * 32 + en] = J::sum(join, g * parts, parts, J::at(en, et));
                }
            }
        }
        if (t0 + next < n) {
            begin(t0 + next);
            lds_barrier();          // the partial results are read
        }
    }
}

// Parts of a row's K: with many experts there are waves enough, and a wave of few slabs
// is mostly its start and end (13 tokens over 128 experts 106 us with two parts of 8
// and of 4 slabs, 104 with one).
inline int expert_parts(int chunks)
{
    const int n = slabs_of(chunks);
    return n >= 64 ? 8 : n >= 24 ? 4 : 1;
}

constexpr int kFit = 2048;      // waves that run at once, two per SIMD

// Waves of a product if every workgroup goes through all its expert's pairs.
inline int expert_waves(const ExpertParams& p, int chunks, int tiles) { return p.slots * tiles * expert_parts(chunks); }

template <class T, bool GATE>
int expert_start(const ExpertParams& p, hipStream_t st)
{
    const int K = GATE ? p.D : p.F, N = GATE ? p.F : p.D;
    ExpertParams q = p;
    constexpr int ROWS = GATE ? 16 : 32;
    const int parts = expert_parts(K / (4 * T::VPW));
    q.log_parts = __builtin_ctz(parts);
    q.groups = std::max(1, 4 / parts);
    while (N / ROWS % q.groups != 0) q.groups /= 2;
    q.meta = Meta(32 * q.groups, K, T::BITS, T::GS, parts);
    // Where the rows alone are fewer waves than fit at once, workgroups share an expert's
    // pairs (as many as twice the average asks for, since experts differ): 128 tokens
    // over 4 experts of 512 x 512, 2 each: 58.8 us without, 28.6 with; of 2048 x 1024,
    // 102.8, 48.9; over 16 of 1024 x 768, 4 each: 58.7, 45.0.
    q.takers = std::max(1, std::min(kFit / expert_waves(p, K / (4 * T::VPW), N / ROWS), (2 * p.P / p.E + 16 * T::CT - 1) / (16 * T::CT)));
    const ExpertSpace sp(q.meta, q.groups * parts, 32 * q.groups, p.P);
    const void* fn = reinterpret_cast<const void*>(&expert_kernel<T, GATE>);
    if (sp.bytes > 64 * 1024 &&
        hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, sp.bytes) != hipSuccess)
        return 1;
    void* args[] = {&q};
    const dim3 grid(N / (ROWS * q.groups), p.slots, q.takers);
    return hipLaunchKernel(fn, grid, dim3(kWave * q.groups * parts), args, sp.bytes, st) == hipSuccess ? 0 : 1;
}

// The down products of one token's experts and their weighted sum, a wave per slot
// and 32 rows per workgroup: neither the experts' outputs are written nor another
// launch adds them up, but an expert that two tokens chose is read for each.  The sums
// are those of the two launches, bit for bit.  One token, 6 experts of 3840 x 1024:
// 12.4 us for 13.3 MB, of which 3 are the launch and its arguments.
constexpr int kTokenSlots = kMaxWaves;

inline int token_bytes(const Meta& meta, int k) { return k * (2048 + 2 * Join<1>::kWords * 4 + meta.bytes(32)); }

template <class T>
__global__ __launch_bounds__(kTokenSlots* kWave, T::WAVES) void token_kernel(ExpertParams p)
{
    using J = Join<2>;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    together(p.ids, p.weights, p.w2, p.s2, p.b2, p.h, p.h_plane, p.y, p.k, p.D, p.F, p.E, p.meta.groups);
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane & 15;
    const int n0 = blockIdx.x * 32, t = blockIdx.y, pair = t * p.k + wave, K = p.F, N = p.D;
    float* const join = reinterpret_cast<float*>(lds + p.k * 2048);
    char* const own = lds + p.k * (2048 + 2 * Join<1>::kWords * 4) + wave * p.meta.bytes(32);
    uint16_t* const scales = reinterpret_cast<uint16_t*>(own);
    uint16_t* const biases = reinterpret_cast<uint16_t*>(own + p.meta.bytes(32) / 2);
    const int e = p.ids[pair];
    if (e >= 0 && e < p.E) {
        typename T::Rows r;
        r.G = K / T::GS;
        r.chunks = K / (4 * T::VPW);
        r.plane = p.h_plane;
        r.turn = lds + wave * 2048;
        r.even = p.meta.groups % T::NG == 0;
        const size_t row = (size_t)e * N + n0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            T::set_codes(r, i, p.w2, row + 16 * i, 16);
            r.s[i] = scales + (16 * i + c) * p.meta.groups;
            r.b[i] = biases + (16 * i + c) * p.meta.groups;
        }
        MetaCopy<2> copy(p.s2 + row * r.G, p.b2 + row * r.G, 32, r.G, kWave, lane);
        copy.ask();
        keep_order();
        T::set_token(r, 0, p.h, pair);
        const int slabs = slabs_of(r.chunks);
        typename T::Ring ring;
        T::begin(ring, r, 0, slabs);
        copy.put(scales, biases);
        __builtin_amdgcn_wave_barrier();
        f32x4 acc[2][1];
        T::clear(acc);
        T::run(acc, ring, r, 0, slabs);
#pragma unroll
        for (int i = 0; i < 2; ++i) J::write(join, wave, lane, i, acc[i][0]);
    }
    lds_barrier();
    if (threadIdx.x >= 32) return;
    float v = 0.0f;
    for (int j = 0; j < p.k; ++j) {
        const int id = p.ids[t * p.k + j];
        if (id >= 0 && id < p.E) v = __builtin_fmaf(p.weights[t * p.k + j], join[j * J::kWords + J::at(lane, 0)], v);
    }
    store_y(p.y, (size_t)t * N + n0 + lane, v, p.yf32);
}

// Whole tokens where their slots fit the waves, a row of w2 is one wave's, and what is
// read again for experts that tokens share costs less than a launch.  Whole layers, us,
// by expert and by token: 1 token over 64 experts of 3840 x 1024, 6 each: 36.1, 34.1;
// 2 tokens: 43.7, 38.1; 8: 92.5, 96.9.  4 experts of 4096 x 2048, 2 each: 1 token 37.7,
// 33.5; 4: 41.4, 42.4; 7: 42.5, 44.8.  16 experts of 512 x 512, 4 each, 16 tokens: 26.1,
// 21.1.  2-bit, 16 experts of 5120 x 768, 8 each: 2 tokens 66.8, 62.5; 6: 74.3, 85.5.
inline bool by_token(int n, int k, int D, int F, int bits)
{
    return k <= kTokenSlots && expert_parts(F * bits / 128) == 1 && (n == 1 || (long long)n * k * D * F <= 1 << 26);
}

template <class T>
int token_start(const ExpertParams& p, hipStream_t st)
{
    ExpertParams q = p;
    q.meta = Meta(32, p.F, T::BITS, T::GS, 1);
    const int bytes = token_bytes(q.meta, p.k);
    const void* fn = reinterpret_cast<const void*>(&token_kernel<T>);
    if (bytes > 64 * 1024 && hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess) return 1;
    void* args[] = {&q};
    return hipLaunchKernel(fn, dim3(p.D / 32, p.P / p.k), dim3(kWave * p.k), args, bytes, st) == hipSuccess ? 0 : 1;
}

template <int BITS, int GS, bool SBF>
int expert_pick(int which, const ExpertParams& p, bool xf32, hipStream_t st)
{
    // The down products take the hidden values in three planes, exactly as fp32 held them.  (In two, off by 2^-17, 2.5
    // of 1000 bf16 outputs were the neighbour of the right one; now 0.3, and 1 where products and sums are plain fp32.
    // Layers were faster by up to a tenth, and with 2-bit codes in groups of 64, whose instances of three planes spill,
    // by a fifth: 13 tokens over 128 experts of 2048 x 1024 93 us, now 99; 2-bit, 91, now 117.)
    if (which == 2) return token_start<Tile<BITS, GS, 2, 1, 3, SBF, false>>(p, st);
    if (which == 1)
        return p.base ? expert_start<Tile<BITS, GS, 2, 1, 3, SBF, true>, false>(p, st)
                      : expert_start<Tile<BITS, GS, 2, 1, 3, SBF, false>, false>(p, st);
    // Two token tiles per wave for sorted pairs of more than 12 per expert, where waves of
    // one each do not fit at once: 128 tokens over 32 experts of 3840 x 1920, 4 each, 2-bit,
    // whole layers: 156 us with two in the gate and up products, 172 with one; 4-bit 203, 199.
    const int waves = expert_waves(p, p.D * BITS / 128, p.F / 16);
    const int ct = p.P > 12 * p.E && waves * ((p.P / p.E + 15) / 16) > kFit ? 2 : 1;
    if (p.base) {
        if (xf32) return expert_start<Tile<BITS, GS, 2, 1, 3, SBF, true>, true>(p, st);
        return ct == 1 ? expert_start<Tile<BITS, GS, 2, 1, 1, SBF, true>, true>(p, st)
                       : expert_start<Tile<BITS, GS, 2, 2, 1, SBF, true>, true>(p, st);
    }
    if (xf32) return expert_start<Tile<BITS, GS, 2, 1, 3, SBF, false>, true>(p, st);
    return expert_start<Tile<BITS, GS, 2, 1, 1, SBF, false>, true>(p, st);
}

}  // namespace ops
