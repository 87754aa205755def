// ops_attend_block.hpp -- attention of up to 16 new tokens a sequence: decode and
// verify.
//
// Bound by the read of keys and values.  A workgroup of four waves takes a unit of a
// sequence's keys for one head of the cache and the 16 NR query rows (tokens times heads
// that share it) of a block.  It walks the unit in leaves of 32 KB of keys and as
// much of values: every wave asks for its quarter of the keys, which go straight to the registers that
// the matrix instructions read, and for the values, which go through LDS to be turned over;
// the next leaf's are asked for as soon as the registers are free.  Each wave scores its
// quarter of the keys, the waves agree on the rows' largest scores, put their weights into
// LDS, and each sums its quarter of the columns over all keys of the leaf.
//
// Measured: one token of 32 query heads on 8 of 128 over 131072 places (537 MB) 110 us and 6.5 of the
// join, 4.9 TB/s, which is a copy's rate; 64 sequences of up to 8192 places (1.07 GB) 222 and 6,
// 4.8 TB/s; 13 tokens of 16 heads on 8 of 256 over 16384 places (134 MB) 35 and 5.  Short calls are a
// chain of dependent loads: one token over 411 places 6.4 and 4.2.
//
// Why leaves of 32 KB: of 64 KB the registers hold no leaf in flight beside the one at work (13 tokens over
// 16384 places 86 us for 46, 64 sequences 346 for 257, both before later steps).
//
// Order of sums.  Leaves begin at multiples of their length, a leaf's sums begin at zero, and
// are joined in order to those of the super that the leaf is in (kSuper leaves), and supers
// in order to a row's; whether by this kernel or the next one.  Leaves that a row sees nothing
// of change no bit.  So a row's bits depend on its place, keys and head size alone: a
// verify block gives each token the bits that a call of that token alone gives it, whatever
// else is in the call.
#pragma once
#include "ops_attend.hpp"

namespace ops {

// queries of more than one tile of rows lie in LDS
template <int DP, int NP, int NR>
constexpr int block_lds = kLeafBytes + NP * leaf_keys(DP) * 32 + 2 * 4 * 16 * 4 + 16 + (NR > 1 ? NR * DP * 32 : 0);

// One of the launch's workgroups; SHARE: which may take several units.
template <int DP, class X, int NP, int NR, bool SHARE>
__device__ __forceinline__ void block_body(const AttendParams& p, int block, char* lds)
{
    constexpr int KT = leaf_keys(DP);      // keys of a leaf
    constexpr int WK = KT / 4;             // of which a wave scores
    constexpr int TILES = WK / 16;         // in tiles of 16
    constexpr int DS = DP / 32;            // steps of 32 values of a head
    constexpr int DT = DP / 64;            // tiles of 16 columns that a wave sums
    constexpr int US = KT / 32;            // steps of 32 keys
    constexpr float kLift = 1 << (int)lift_log2(X());      // of a leaf's weights, whose largest is 1: exact, so what fp16 holds without it has the same bits
    char* const values = lds;
    char* const weights = lds + kLeafBytes;
    float* const tops = reinterpret_cast<float*>(weights + NP * KT * 32);
    float* const sums = tops + 64;
    uint32_t* const odds = reinterpret_cast<uint32_t*>(sums + 64);       // whether a wave has met values that are no numbers
    char* const queries = reinterpret_cast<char*>(odds + 4);

    const Cache& c = p.cache;
    together(c.pages, c.pages_row, c.starts, c.lengths, c.by_page.magic, c.by_page.shift, c.max_pages, c.T, c.n_seqs, p.per_unit, p.window, p.heads, p.row_blocks, p.shares,
             p.rows_last, p.by_rows.magic, p.by_rows.shift, p.by_heads.magic, p.by_heads.shift, p.by_seqs.magic, p.by_seqs.shift);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    // Eight units side by side on the eight compute dies; on a die, all of a unit's heads and row blocks one
    // after the other, since heads lie next to each other in memory in most caches.  Beside chunks, where most
    // sequences have one tile of rows, the others come last: workgroups without work between the others
    // would leave compute units to themselves.  255 single tokens of 1000 places, 8 heads of 128, with as many
    // rows as 16 tokens have, us: 205, 488 side by side.
    const int turn = block >> 3;
    const int rows_turn = divide(turn, p.by_rows), rows_rest = turn - rows_turn * (p.rows_last > 0 ? p.rows_last : p.row_blocks);
    const int rb = p.rows_last > 0 ? rows_turn : rows_rest, over = p.rows_last > 0 ? rows_rest : rows_turn;
    const int eight = divide(over, p.by_heads), head = over - eight * p.heads;
    const Turn at_turn = turn_of(eight * 8 + (block & 7), p);
    const int u = at_turn.turn, b = at_turn.b;
    if (u >= p.shares || rb >= p.row_blocks) return;
    // pages of the lane's keys of a leaf, key n of every tile
    const int32_t* const table = p.cache.pages + b * p.cache.pages_row;
    int entry[TILES];
    auto ask_pages = [&](int leaf) {
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            const int j = leaf + wave * WK + t * 16 + n;
            entry[t] = table[min(page_index(p.cache, j), p.cache.max_pages - 1)];
        }
    };
    // Without a window the first leaf is known before the sequence is: its pages are asked for together
    // with what is known of the sequence.
    const int U = KT * p.per_unit, early = p.window == 0 ? u * U : -1;
    if (early >= 0) ask_pages(early);
    const Seq s = sequence(p.cache, b);
    const int tokens = min(s.count, p.max_new), place0 = s.length - s.count;
    if (tokens > kBlockTokens) return;
    const int r0 = rb * NR * 16;
    if (r0 >= tokens * p.group) return;
    const Visible vis = visible(place0, tokens, p.window, p.sinks, U);
    if (u >= vis.units && !(u == 0 && p.units == 1)) return;      // a lone unit writes zeros where nothing is seen

    // this lane's rows
    int high[NR], low[NR];
    bool mine[NR];
    long long row[NR];
    u32x4 q[DS];
#pragma unroll
    for (int rt = 0; rt < NR; ++rt) {
        const int r = r0 + rt * 16 + n, i = divide(r, p.by_group), h = head * p.group + r - i * p.group;
        mine[rt] = i < tokens;
        high[rt] = mine[rt] ? place0 + i : -1;
        low[rt] = p.window > 0 ? place0 + i - p.window : -0x7fffffff - 1;
        const int t = s.start + i;
        row[rt] = (long long)t * p.q_heads + h;
        if (NR == 1 || rt == wave) {
#pragma unroll
            for (int d = 0; d < DS; ++d) {
                const int c = 4 * d + g;
                q[d] = u32x4{0, 0, 0, 0};
                if (mine[rt] && c * 8 < p.D) q[d] = *reinterpret_cast<const u32x4*>(p.q + t * p.q_token + h * p.q_head + c * 16);
            }
        }
    }
    const int i_first = divide(r0, p.by_group), i_last = min(tokens - 1, divide(r0 + NR * 16 - 1, p.by_group));
    const bool whole = p.D == DP;
    const int last_tile = min(NR - 1, (tokens * p.group - r0 - 1) / 16);      // of rows that there are

    f32x4 o[NR][DT];
    float m[NR], l[NR];
    auto begin = [&] {
#pragma unroll
        for (int rt = 0; rt < NR; ++rt) {
            m[rt] = kGone;
            l[rt] = 0.0f;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[rt][d] = f32x4{0, 0, 0, 0};
        }
    };
    // what the rows have found in a unit
    auto finish = [&](int unit) {
        const long long moved = block_row(p, b, s.start) - (long long)s.start * p.q_heads;
#pragma unroll
        for (int rt = 0; rt < NR; ++rt) {
            if (!mine[rt]) continue;
            const long long at = (row[rt] + moved) * p.units + unit;
            if (p.units > 1 && wave == 0 && g == 0) p.stat[at] = f32x2{m[rt], l[rt]};
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const int c = (wave * DT + d) * 16 + 4 * g;
                if (c >= p.D) continue;
                if (p.units == 1) put_result(p, row[rt], c, o[rt][d], l[rt]);
                else *reinterpret_cast<f32x4*>(p.part + at * p.D + c) = o[rt][d];
            }
        }
    };
    begin();

    // several units only without a window, whose units are one after the other from place 0 on
    const int from = u < vis.units ? vis.unit(u) * U : 0, to = u < vis.units ? SHARE && p.window == 0 ? vis.high + 1 : min(from + U, vis.high + 1) : 0;
    auto next_leaf = [&](int at) {
        while (at < to && !vis.meets(at, at + KT)) at += KT;
        return at < to ? at : -1;
    };

    u32x4 kf[TILES][DS], vf[TILES][DS];
    long long v_at[TILES];
    uint32_t valid[TILES];
    long long k_at[TILES];
    // Addresses: keys that hold nothing get the cache's first slot's, and are hidden later.
    auto addresses = [&](int leaf, uint32_t (&ok)[TILES]) {
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            const int j = leaf + wave * WK + t * 16 + n;
            const bool fine = j < s.length && (uint32_t)entry[t] < (uint32_t)p.cache.n_pages;
            const int slot = fine ? j - page_index(p.cache, j) * p.cache.page_size : 0, page = fine ? entry[t] : 0;
            ok[t] = (uint32_t)__ballot(fine) & 0xffff;
            k_at[t] = page * p.cache.k_page + slot * p.cache.k_slot + head * p.cache.k_head;
            const int vpage = __shfl(page, lane >> 2), vslot = __shfl(slot, lane >> 2);
            v_at[t] = vpage * p.cache.v_page + vslot * p.cache.v_slot + head * p.cache.v_head;
        }
    };
    auto ask_keys = [&] {
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int d = 0; d < DS; ++d) {
                const int c = whole ? 4 * d + g : min(4 * d + g, (p.D >> 3) - 1);
                kf[t][d] = *reinterpret_cast<const u32x4*>(p.cache.k + k_at[t] + c * 16);
            }
    };
    auto ask_values = [&] {
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int d = 0; d < DS; ++d) {
                const int c = whole ? 4 * d + (lane & 3) : min(4 * d + (lane & 3), (p.D >> 3) - 1);
                vf[t][d] = *reinterpret_cast<const u32x4*>(p.cache.v + v_at[t] + c * 16);
            }
    };

    int leaf = next_leaf(from), now = u;
    if (leaf >= 0) {
        if (leaf != early) ask_pages(leaf);
        addresses(leaf, valid);
        ask_keys();
        ask_values();
    }
    if constexpr (NR > 1) {
        if (wave < NR) {
#pragma unroll
            for (int d = 0; d < DS; ++d) *reinterpret_cast<u32x4*>(queries + (wave * DS + d) * 1024 + lane * 16) = q[d];
        }
        lds_only_barrier();
    }
    while (leaf >= 0) {
        const bool last = SHARE && (leaf + KT) % U == 0;      // of its unit
        const int next = next_leaf(leaf + KT + (last ? (p.shares - 1) * U : 0));
        if (next >= 0) ask_pages(next);
        uint32_t ok[TILES];
#pragma unroll
        for (int t = 0; t < TILES; ++t) ok[t] = valid[t];
        // whether all rows see the same places of the leaf, and whether those of this wave are all there
        const bool even = leaf + KT - 1 <= place0 + i_first && (p.window == 0 || leaf > place0 + i_last - p.window || leaf + KT <= p.sinks);
        bool full = even;
#pragma unroll
        for (int t = 0; t < TILES; ++t) full = full && ok[t] == 0xffff;
#pragma unroll
        for (int rt = 0; rt < NR; ++rt) {
            if (rt > 0 && r0 + rt * 16 >= tokens * p.group) continue;      // the whole workgroup's
            // scores of the wave's keys
            if constexpr (NR > 1) {
#pragma unroll
                for (int d = 0; d < DS; ++d) q[d] = *reinterpret_cast<const u32x4*>(queries + (rt * DS + d) * 1024 + lane * 16);
            }
            f32x4 x[TILES];
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                f32x4 a = {0, 0, 0, 0};
#pragma unroll
                for (int d = 0; d < DS; ++d) {
                    u32x4 k = kf[t][d];
                    if (!whole && 8 * (4 * d + g) >= p.D) k = u32x4{0, 0, 0, 0};
                    a = mfma(k, q[d], a, X());
                }
                x[t] = a * p.scale;
            }
            if (!full) {
#pragma unroll
                for (int t = 0; t < TILES; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = leaf + wave * WK + t * 16 + 4 * g + i;
                        x[t][i] = sees(j, high[rt], low[rt], p.sinks, ok[t] >> (4 * g + i)) ? x[t][i] : kGone;
                    }
            }
            // the leaf's largest score of the row
            float top = kGone;
#pragma unroll
            for (int t = 0; t < TILES; ++t) top = __builtin_fmaxf(__builtin_fmaxf(top, __builtin_fmaxf(x[t].x, x[t].y)), __builtin_fmaxf(x[t].z, x[t].w));
            top = row_max(top);
            if (g == 0) tops[wave * 16 + n] = top;
            if (rt > 0 && rt == last_tile && next >= 0) ask_keys();
            lds_only_barrier();
            if (rt == 0) {
                if (!even) {
                    bool found = false;
#pragma unroll
                    for (int t = 0; t < TILES; ++t)
#pragma unroll
                        for (int d = 0; d < DS; ++d) found |= (ok[t] >> (lane >> 2) & 1) && odd<X>(vf[t][d]);
                    found = __any(found);
                    if (lane == 0) odds[wave] = found;
                }
#pragma unroll
                for (int t = 0; t < TILES; ++t)
#pragma unroll
                    for (int d = 0; d < DS; ++d) {
                        u32x4 v = vf[t][d];
                        if (!full && !(ok[t] >> (lane >> 2) & 1)) v = u32x4{0, 0, 0, 0};
                        *reinterpret_cast<u32x4*>(values + ((wave * TILES + t) * DS + d) * 1024 + (lane >> 2) * 64 + (((lane & 3) ^ swizzle(lane >> 4)) << 4)) = v;
                    }
                if (next >= 0) {
                    addresses(next, valid);
                    if (last_tile == 0) ask_keys();
                    ask_values();
                }
            }
            top = __builtin_fmaxf(__builtin_fmaxf(tops[n], tops[16 + n]), __builtin_fmaxf(tops[32 + n], tops[48 + n]));
            const float at = top == kGone ? 0.0f : top;
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                f32x4 w;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = exp2_of(x[t][i] - at);
                sum += (w.x + w.y) + (w.z + w.w);
                w *= kLift;
                const int block = wave * TILES + t;
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    const u32x2 h = {pack(w.x, w.y, X()), pack(w.z, w.w, X())};
                    *reinterpret_cast<u32x2*>(weights + c * KT * 32 + (block >> 1) * 1024 + lane * 16 + (block & 1) * 8) = h;
                    if (c + 1 < NP) {
                        const f32x2 lo = unpack(h.x, X()), hi = unpack(h.y, X());
                        w -= f32x4{lo.x, lo.y, hi.x, hi.y};
                    }
                }
            }
            sum = row_sum(sum);
            if (g == 0) sums[wave * 16 + n] = sum;
            lds_only_barrier();
            sum = (sums[n] + sums[16 + n]) + (sums[32 + n] + sums[48 + n]);
            const Factors by = join(m[rt], l[rt], top, sum);

            // the wave's columns over the leaf's keys
            f32x4 a[DT];
#pragma unroll
            for (int d = 0; d < DT; ++d) a[d] = f32x4{0, 0, 0, 0};
            auto value = [&](int d, int k) {
                const int tile = wave * DT + d;
                const char* const at = values + (tile >> 1) * 1024 + (4 * g + (n >> 2)) * 64 + ((((tile & 1) * 2 + ((n & 3) >> 1)) ^ swizzle(g)) << 4) + (n & 1) * 8;
                const u32x2 v0 = read_turned(at + 2 * k * DS * 1024), v1 = read_turned(at + (2 * k + 1) * DS * 1024);
                return u32x4{v0.x, v0.y, v1.x, v1.y};
            };
            if (even || __builtin_amdgcn_readfirstlane(odds[0] | odds[1] | odds[2] | odds[3]) == 0) {
#pragma unroll
                for (int k = 0; k < US; ++k) {
                    u32x4 w[NP];
#pragma unroll
                    for (int c = 0; c < NP; ++c) w[c] = *reinterpret_cast<const u32x4*>(weights + c * KT * 32 + k * 1024 + lane * 16);
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const u32x4 v = value(d, k);
#pragma unroll
                        for (int c = 0; c < NP; ++c) a[d] = mfma(v, w[c], a[d], X());
                    }
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < US; ++k)
#pragma unroll 1
                    for (int c = 0; c < NP; ++c) {
                        const u32x4 w = *reinterpret_cast<const u32x4*>(weights + c * KT * 32 + k * 1024 + lane * 16);
#pragma unroll
                        for (int d = 0; d < DT; ++d) a[d] = mfma(numbers4<X>(value(d, k)), w, a[d], X());
                    }
#pragma unroll 1
                for (int i = 0; i < 3; ++i) {
                    const Kind kind = kind_of<X>(i);
                    f32x4 count[DT];
#pragma unroll
                    for (int d = 0; d < DT; ++d) count[d] = f32x4{0, 0, 0, 0};
#pragma unroll 1
                    for (int k = 0; k < US; ++k) {
                        u32x4 seen;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = leaf + k * 32 + (i >> 1) * 16 + 4 * g + 2 * (i & 1);
                            seen[i] = (sees(j, high[rt], low[rt], p.sinks, 1) ? one(X()) : 0) | (sees(j + 1, high[rt], low[rt], p.sinks, 1) ? one(X()) << 16 : 0);
                        }
#pragma unroll
                        for (int d = 0; d < DT; ++d) count[d] = mfma(marks4<X>(value(d, k), kind), seen, count[d], X());
                    }
#pragma unroll
                    for (int d = 0; d < DT; ++d) a[d] = met(a[d], count[d], kind);
                }
            }
#pragma unroll
            for (int d = 0; d < DT; ++d) o[rt][d] = joined(o[rt][d], a[d], Factors{by.a, by.b / kLift});
        }
        if (last && next >= 0) {
            finish(now);
            begin();
            now = next / U;
        }
        leaf = next;
    }

    finish(now);
}

// Three workgroups on a compute unit where one tile of rows leaves the registers for it (of heads of 64, three pieces of weights fill the LDS
// of two; bounds of two there: one token over 16384 places 17.8 us for 17.6); two tiles of heads of up to 64
// would spill eight (64 sequences of 5 tokens over 1024 places 20.6 us with two workgroups, 23.3 with three).
// SHARE: a workgroup may take several units; what that holds in registers leaves room for two workgroups on a
// compute unit where there are three otherwise (64 ragged sequences of up to 8192 places: 235 us, 228 without).
template <int DP, class X, int NP, int NR, bool SHARE>
__global__ __launch_bounds__(256, !SHARE && NR == 1 && DP < 256 ? 3 : 2) void block_kernel(AttendParams p)
{
    extern __shared__ __align__(16) char lds[];
    block_body<DP, X, NP, NR, SHARE>(p, blockIdx.y * gridDim.x + blockIdx.x, lds);
}

// the kernels of a head size
template <int DP, class X, int NP, bool SHARE>
const void* block_kernel_rows(int row_tiles, int* lds)
{
    *lds = row_tiles == 1 ? block_lds<DP, NP, 1> : row_tiles == 2 ? block_lds<DP, NP, 2> : block_lds<DP, NP, 4>;
    return row_tiles == 1   ? (const void*)&block_kernel<DP, X, NP, 1, SHARE>
           : row_tiles == 2 ? (const void*)&block_kernel<DP, X, NP, 2, SHARE>
                            : (const void*)&block_kernel<DP, X, NP, 4, SHARE>;
}

template <int DP, class X, int NP>
const void* block_kernel_shares(bool share, int row_tiles, int* lds)
{
    return share ? block_kernel_rows<DP, X, NP, true>(row_tiles, lds) : block_kernel_rows<DP, X, NP, false>(row_tiles, lds);
}

// A weight in one piece for bf16 outputs; for fp32 ones in as many as hold 22 bits of it or more (fp16: down to 2^-18 of the leaf's
// largest, and below that to 2^-40 of it).
template <int DP>
const void* block_kernel_types(bool f16, bool f32_out, bool share, int row_tiles, int* lds)
{
    if (f16) return f32_out ? block_kernel_shares<DP, _Float16, 2>(share, row_tiles, lds) : block_kernel_shares<DP, _Float16, 1>(share, row_tiles, lds);
    return f32_out ? block_kernel_shares<DP, __bf16, 3>(share, row_tiles, lds) : block_kernel_shares<DP, __bf16, 1>(share, row_tiles, lds);
}

}  // namespace ops
