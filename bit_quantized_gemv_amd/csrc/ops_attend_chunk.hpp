// ops_attend_chunk.hpp -- attention of more than 16 new tokens a sequence: prompts,
// whole or in chunks.
//
// Bound by the matrix instructions and, beside them, the exponentials.  A workgroup takes
// 32 query rows a wave (tokens times the heads that share a head of the cache), kept in
// registers with their outputs, and walks the keys that they see in tiles through LDS, the
// next tile's on their way there meanwhile.  A wave scores 32 rows against the tile,
// takes the weights with the rows' running maxima, and adds the weighted values up; a maximum
// is followed only when it has grown by 2^8 (fp16: less), which weights and sums have room for, since moving it
// costs a pass over the outputs.  Where the rows alone are few workgroups, several share the
// keys of a tile of rows, and a second launch joins them.
//
// Measured, 2048 tokens over 16384 places, 32 heads on 8 of 128: 569 us in turn with others' calls, 905 TFLOP/s
// (659 us back to back, the clock falling), where a library's product of 8192 x 8192 x 8192 reaches 1239.  The
// matrix instructions are busy 44% of the time, the vector instructions half of it, reads of LDS (32 KB a
// wave and tile) 41%; two waves on a SIMD overlap them in part.  Over 8192 places, back to back, heads of 64:
// 562 TFLOP/s, 96: 727, 192: 695, 256: 678; fp32 outputs (three pieces of each weight) 517 at 128.
#pragma once
#include "ops_attend_block.hpp"

namespace ops {

// Tiles of 64 keys of up to 128 values, of 32 above: scores and the next tile fill registers and LDS.
// As many waves as the registers hold, in workgroups of four, or of eight where the outputs and
// queries of two waves fill a unit's.
template <int DP>
struct Chunk {
    static constexpr int kWaves = DP > 192 ? 8 : 4;
    static constexpr int kAtOnce = DP > 192 ? 1 : DP > 64 ? 2 : 3;     // workgroups on a unit, as far as registers go
    static constexpr int kKeys = DP > 128 ? 32 : 64;               // of a tile
    static constexpr int kRows = kWaves * 32;
    static constexpr int kTileBytes = kKeys * DP * 2;
    static constexpr int kLds = 4 * kTileBytes + 2 * 48;           // keys and values, twice, and what is known of them
};

// 0 would follow every maximum, which makes the largest weights exact ones: bf16 outputs are off by 1.8e-3 of their norm
// then instead of 2.2e-3 (their own rounding alone: 1.7e-3), and the 2048 tokens above take 602 us for 571.
// fp16 has less room: what a maximum may lag by is lost to the smallest weights, which keep all their bits down to 2^(room - 29) of
// the largest, and for fp32 outputs, in two pieces, down to 2^(room - 18).  2048 tokens over 16384 places: 657 us with 8 (as bf16), 671
// with 4, 675 with 2, 694 with 0; fp32 out 903 with 8, 936 with 1, 932 with 2.
constexpr float room(__bf16, int) { return 8.0f; }
constexpr float room(_Float16, int pieces) { return pieces == 1 ? 4.0f : 1.0f; }

// One of the launch's workgroups: a tile of rows and one of a head's shares of their keys.
template <int DP, class X, int NP>
__device__ __forceinline__ void chunk_body(const AttendParams& p, int group, int share, char* lds)
{
    typedef Chunk<DP> C;
    constexpr int NK = C::kKeys, KB = NK / 16, DS = DP / 32, DT = DP / 16, US = NK / 32;
    constexpr int BW = KB * DS / C::kWaves;       // blocks of 16 keys and 32 columns that a wave loads
    constexpr float kRoom = room(X(), NP), kUp = lift_log2(X()) > 0.0f ? lift_log2(X()) - kRoom : 0.0f;
    uint32_t* const masks = reinterpret_cast<uint32_t*>(lds + 4 * C::kTileBytes);      // which keys there are
    uint32_t* const odds = masks + 8;                                                   // whether a wave has met values that are no numbers

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, g = lane >> 4;
    // The sequence whose rows these are: the launch has about as many workgroups as all chunks have
    // tiles of rows, one after the other.  255 single tokens beside a chunk of 2048, 1000 places each, us:
    // 1048 when every sequence had as many workgroups as the longest.
    int left = divide(group, p.by_heads), b = -1, rb = 0;
    const int head = group - left * p.heads;
    Seq s;
    for (int i = 0; i < p.cache.n_seqs && b < 0; i += 64) {
        Seq of = {0, 0, 0};
        if (i + lane < p.cache.n_seqs) of = sequence(p.cache, i + lane);
        const int count = min(of.count, p.max_new), blocks = count > kBlockTokens ? (count * p.group + C::kRows - 1) / C::kRows : 0;
        for (uint64_t chunks = __ballot(blocks > 0); chunks; chunks &= chunks - 1) {
            const int at = __builtin_ctzll(chunks), n = __builtin_amdgcn_readlane(blocks, at);
            if (left < n) {
                b = i + at;
                rb = n - 1 - left;      // those that see most first
                s.start = __builtin_amdgcn_readlane(of.start, at);
                s.count = __builtin_amdgcn_readlane(of.count, at);
                s.length = __builtin_amdgcn_readlane(of.length, at);
                break;
            }
            left -= n;
        }
    }
    if (b < 0) return;
    const int tokens = min(s.count, p.max_new), place0 = s.length - s.count;
    const int rows = tokens * p.group;
    const int r0 = rb * C::kRows, i_first = divide(r0, p.by_group), i_last = min(tokens - 1, divide(r0 + C::kRows - 1, p.by_group));

    // the tiles of keys that the workgroup's rows see, and its share of them
    const Visible vis = visible(place0 + i_first, i_last - i_first + 1, p.window, p.sinks, NK);
    const int t_from = (int)((long long)vis.units * share / p.splits), t_to = (int)((long long)vis.units * (share + 1) / p.splits);

    // queries, negative scales turned into them
    const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0;
    const float scale = __builtin_fabsf(p.scale);
    const int w_first = divide(r0 + wave * 32, p.by_group), w_last = min(tokens - 1, divide(r0 + wave * 32 + 31, p.by_group));
    const bool idle = r0 + wave * 32 >= rows;
    u32x4 q[2][DS];
    int high[2], low[2];
    long long row[2];
    bool mine[2];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
        const int r = r0 + wave * 32 + rt * 16 + n, i = divide(r, p.by_group), h = head * p.group + r - i * p.group, t = s.start + i;
        mine[rt] = r < rows;
        high[rt] = mine[rt] ? place0 + i : -1;
        low[rt] = p.window > 0 ? place0 + i - p.window : -0x7fffffff - 1;
        row[rt] = (long long)t * p.q_heads + h;
#pragma unroll
        for (int d = 0; d < DS; ++d) {
            const int c = 4 * d + g;
            q[rt][d] = u32x4{0, 0, 0, 0};
            if (mine[rt] && c * 8 < p.D) q[rt][d] = *reinterpret_cast<const u32x4*>(p.q + t * p.q_token + h * p.q_head + c * 16) ^ flip;
        }
    }
    f32x4 o[2][DT];
    float m[2] = {kGone, kGone};
    f32x4 l[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};       // a row's sum of weights, four times
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
        for (int d = 0; d < DT; ++d) o[rt][d] = f32x4{0, 0, 0, 0};

    // what this wave loads of a tile: rows lane / 4 of tile kb, columns from 32 d0 on
    const int kb = wave * BW / DS, d0 = wave * BW % DS;
    const int key_row = kb * 16 + (lane >> 2), piece = (lane & 3) ^ swizzle(lane >> 4);
    const uint32_t lds_at = lds_address(lds) + (kb * DS + d0) * 1024;
    bool held = false;
    int entry = 0;
    auto place_of = [&](int t) { return vis.unit(t) * NK + key_row; };
    auto ask_page = [&](int t) {
        if (t < t_to) entry = p.cache.pages[b * p.cache.pages_row + page_index(p.cache, min(place_of(t), s.length - 1))];
    };
    auto ask_tile = [&](int buffer, int t) {
        if (t >= t_to) return;
        const int j = place_of(t);
        held = j < s.length && (uint32_t)entry < (uint32_t)p.cache.n_pages;
        const int slot = held ? j - page_index(p.cache, j) * p.cache.page_size : 0, page = held ? entry : 0;
        const char* k = p.cache.k + page * p.cache.k_page + slot * p.cache.k_slot + head * p.cache.k_head + (4 * d0 + piece) * 16;
        const char* v = p.cache.v + page * p.cache.v_page + slot * p.cache.v_slot + head * p.cache.v_head + (4 * d0 + piece) * 16;
        const uint32_t to = lds_at + buffer * 2 * C::kTileBytes;
#pragma unroll
        for (int d = 0; d < BW; ++d)
            if (8 * (4 * (d0 + d) + piece) < p.D) {       // columns above D stay the zeros that they are
                send_to_lds(k + d * 64, to + d * 1024);
                send_to_lds(v + d * 64, to + C::kTileBytes + d * 1024);
            }
    };
    // whether all of the workgroup's rows see the same places of a tile
    auto even = [&](int j0) {
        return j0 + NK - 1 <= place0 + i_first && (p.window == 0 || j0 > place0 + i_last - p.window || j0 + NK <= p.sinks);
    };
    auto land = [&](int buffer, int t) {
        landed();
        char* const mine_at = lds + (buffer * 2 + 1) * C::kTileBytes + (kb * DS + d0) * 1024 + lane * 16;
        const uint64_t there = __ballot(held);
        if (there != ~0ull && !held) {
#pragma unroll
            for (int d = 0; d < BW; ++d) *reinterpret_cast<u32x4*>(mine_at + d * 1024) = u32x4{0, 0, 0, 0};
        }
        if (!even(vis.unit(t) * NK)) {
            bool found = false;
#pragma unroll
            for (int d = 0; d < BW; ++d) found |= odd<X>(*reinterpret_cast<const u32x4*>(mine_at + d * 1024));
            const uint32_t any = __any(found) ? 1 : 0;
            if (lane == 0) odds[buffer * 8 + wave] = any;
        }
        // one bit a key
        if (d0 == 0) {
            const uint32_t bits = (uint32_t)__ballot(lane < 16 && (there >> (4 * (lane & 15)) & 1));
            if (lane == 0) masks[buffer * 4 + kb] = bits;
        }
    };

    // a tile of 16 columns and 32 keys, turned over
    auto value = [&](const char* values, int d, int u) {
        const char* const at = values + (d >> 1) * 1024 + (4 * g + (n >> 2)) * 64 + ((((d & 1) * 2 + ((n & 3) >> 1)) ^ swizzle(g)) << 4) + (n & 1) * 8;
        const u32x2 v0 = read_turned(at + 2 * u * DS * 1024), v1 = read_turned(at + (2 * u + 1) * DS * 1024);
        return u32x4{v0.x, v0.y, v1.x, v1.y};
    };
    // one tile of a wave; full: every row sees all of its keys
    auto tile = [&](bool full, const char* keys, int j0, const uint32_t (&ok)[KB]) {
        const char* const values = keys + C::kTileBytes;
        f32x4 x[2][KB];
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int k = 0; k < KB; ++k) {
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) x[rt][k] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int d = 0; d < DS; ++d) {
                const u32x4 f = *reinterpret_cast<const u32x4*>(keys + (k * DS + d) * 1024 + n * 64 + ((g ^ swizzle(n >> 2)) << 4));
#pragma unroll
                for (int rt = 0; rt < 2; ++rt) x[rt][k] = mfma(f, q[rt][d], x[rt][k], X());
            }
        }
        __builtin_amdgcn_s_setprio(0);
        if (!full) {
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + k * 16 + 4 * g + i;
                    const uint32_t held = ok[k] >> (4 * g + i);
#pragma unroll
                    for (int rt = 0; rt < 2; ++rt) x[rt][k][i] = sees(j, high[rt], low[rt], p.sinks, held) ? x[rt][k][i] : kGone;
                }
        }
        u32x4 w[2][NP][US];
        float by[2];
        bool moved = false;
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
            float top = x[rt][0][0];
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) top = k + i > 0 ? larger(top, x[rt][k][i]) : top;
            top = row_max(top);
            top *= scale;
            const bool move = top > m[rt] + kRoom;
            const float now = move ? top : m[rt];
            by[rt] = move ? exp2_of(m[rt] - now) : 1.0f;
            m[rt] = now;
            moved = moved || move;
            const float at = now == kGone ? 0.0f : now - kUp;
#pragma unroll
            for (int k = 0; k < KB; ++k) {
                f32x4 e;
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = exp2_of(__builtin_fmaf(x[rt][k][i], scale, -at));
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    const u32x2 h = {pack(e.x, e.y, X()), pack(e.z, e.w, X())};
                    w[rt][c][k >> 1][(k & 1) * 2] = h.x;
                    w[rt][c][k >> 1][(k & 1) * 2 + 1] = h.y;
                    if (c + 1 < NP) {
                        const f32x2 a = unpack(h.x, X()), z = unpack(h.y, X());
                        e -= f32x4{a.x, a.y, z.x, z.y};
                    }
                }
            }
        }
        if (__any(moved)) {
#pragma unroll
            for (int rt = 0; rt < 2; ++rt) {
                l[rt] *= by[rt];
#pragma unroll
                for (int d = 0; d < DT; ++d) o[rt][d] *= by[rt];
            }
        }
        // sums of the weights as they are multiplied, by the matrix product of ones
        const u32x4 ones = u32x4{0x10001, 0x10001, 0x10001, 0x10001} * one(X());
#pragma unroll
        for (int u = 0; u < US; ++u) {
#pragma unroll
            for (int rt = 0; rt < 2; ++rt)
#pragma unroll
                for (int c = 0; c < NP; ++c) l[rt] = mfma(ones, w[rt][c][u], l[rt], X());
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const u32x4 v = value(values, d, u);
#pragma unroll
                for (int rt = 0; rt < 2; ++rt)
#pragma unroll
                    for (int c = 0; c < NP; ++c) o[rt][d] = mfma(v, w[rt][c][u], o[rt][d], X());
            }
        }
    };

    // A tile of which the workgroup's rows see different places, and which holds values that are no
    // numbers: they go to the outputs of the rows that see them, and out of the tile.
    auto clean = [&](char* values, int j0, const uint32_t (&ok)[KB]) {
        u32x4 seen[2][US];
#pragma unroll
        for (int rt = 0; rt < 2; ++rt)
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = j0 + k * 16 + 4 * g + 2 * i;
                    const uint32_t held = ok[k] >> (4 * g + 2 * i);
                    seen[rt][k >> 1][(k & 1) * 2 + i] = (sees(j, high[rt], low[rt], p.sinks, held) ? one(X()) : 0) |
                                                        (sees(j + 1, high[rt], low[rt], p.sinks, held >> 1) ? one(X()) << 16 : 0);
                }
#pragma unroll 1
        for (int i = 0; i < 3; ++i) {
            const Kind kind = kind_of<X>(i);
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                asm volatile("" ::: "memory");       // read again for every kind: registers are short
                f32x4 count[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                for (int u = 0; u < US; ++u) {
                    const u32x4 v = marks4<X>(value(values, d, u), kind);
#pragma unroll
                    for (int rt = 0; rt < 2; ++rt) count[rt] = mfma(v, seen[rt][u], count[rt], X());
                }
#pragma unroll
                for (int rt = 0; rt < 2; ++rt) o[rt][d] = met(o[rt][d], count[rt], kind);
            }
        }
        lds_only_barrier();
        char* const at = values + (kb * DS + d0) * 1024 + lane * 16;
#pragma unroll
        for (int d = 0; d < BW; ++d) *reinterpret_cast<u32x4*>(at + d * 1024) = numbers4<X>(*reinterpret_cast<const u32x4*>(at + d * 1024));
        lds_only_barrier();
    };

    if (p.D < DP) {
        for (int i = threadIdx.x * 16; i < 4 * C::kTileBytes; i += C::kWaves * 1024) *reinterpret_cast<u32x4*>(lds + i) = u32x4{0, 0, 0, 0};
        lds_only_barrier();
    }
    if (t_from < t_to) {
        ask_page(t_from);
        ask_tile(0, t_from);
        ask_page(t_from + 1);
        land(0, t_from);
    }
    lds_only_barrier();
    ask_tile(1, t_from + 1);
    ask_page(t_from + 2);
    for (int t = t_from; t < t_to; ++t) {
        const int buffer = (t - t_from) & 1;
        char* const keys = lds + buffer * 2 * C::kTileBytes;
        const int j0 = vis.unit(t) * NK;
        uint32_t ok[KB];
#pragma unroll
        for (int k = 0; k < KB; ++k) ok[k] = __builtin_amdgcn_readfirstlane(masks[buffer * 4 + k]);
        if (!even(j0)) {
            uint32_t odd = 0;
#pragma unroll
            for (int w = 0; w < C::kWaves; ++w) odd |= odds[buffer * 8 + w];
            if (__builtin_expect(__builtin_amdgcn_readfirstlane(odd) != 0, 0)) clean(keys + C::kTileBytes, j0, ok);
        }
        const bool any = !idle && j0 <= place0 + w_last && (p.window == 0 || j0 + NK > place0 + w_first - p.window + 1 || j0 < p.sinks);
        if (any) {
            bool full = j0 + NK - 1 <= place0 + w_first && (p.window == 0 || j0 > place0 + w_last - p.window || j0 + NK <= p.sinks);
#pragma unroll
            for (int k = 0; k < KB; ++k) full = full && ok[k] == 0xffff;
            tile(full, keys, j0, ok);
        }
        if (t + 1 < t_to) land(buffer ^ 1, t + 1);
        lds_only_barrier();
        ask_tile(buffer, t + 2);
        ask_page(t + 3);
    }

#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
        if (!mine[rt]) continue;
        const long long at = row[rt] * p.splits + share;
        if (p.splits > 1 && g == 0) p.chunk_stat[at] = f32x2{m[rt], l[rt].x};
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const int c = d * 16 + 4 * g;
            if (c >= p.D) continue;
            if (p.splits == 1) put_result(p, row[rt], c, o[rt][d], l[rt].x);
            else *reinterpret_cast<f32x4*>(p.chunk_part + at * p.D + c) = o[rt][d];
        }
    }
}

// What a launch of chunks and blocks asks for.
template <int DP, int NP, int NR>
struct Both {
    static constexpr int kBlock = DP > 128 ? 256 : DP > 64 ? 128 : 64;       // the block's head size
    static constexpr int kLds = Chunk<DP>::kLds > block_lds<kBlock, NP, NR> ? Chunk<DP>::kLds : block_lds<kBlock, NP, NR>;
    // Of heads of 64 with fp32 outputs, the block's pieces of weights may leave room for two alone.  512 tokens over 4096 places, bf16
    // cache, us: 74 with two planned, 79 with three.
    static constexpr int kAtOnce = fit(kLds) < Chunk<DP>::kAtOnce ? fit(kLds) : Chunk<DP>::kAtOnce;
};

// A call's blocks in the same launch: they are bound by memory, chunks by the matrix instructions, and neither waits
// for the other's end.  63 single tokens of 1000 places beside a chunk of 512, 8 heads of 128, us: 98, in two launches 134;
// 255 beside one of 2048: 291, 305.  They take turns by rounds of a workgroup for every compute unit: parts of the chip
// would get all of one kind otherwise (a chunk of 2048 over 16384 places by eights in turn with blocks without work:
// 986 us, by rounds 659).
template <int DP, class X, int NP, int NR>
__global__ __launch_bounds__(Chunk<DP>::kWaves * 64, (Both<DP, NP, NR>::kAtOnce * Chunk<DP>::kWaves / 4)) void chunk_kernel(AttendParams p)
{
    extern __shared__ __align__(16) char lds[];
    together(p.both_rounds, p.chunk_rounds, p.block_groups, p.chunk_groups, p.by_chunk_groups.magic, p.by_chunk_groups.shift);
    const int i = blockIdx.y * gridDim.x + blockIdx.x, round = i / kUnits;
    const bool rest = round >= 2 * p.both_rounds, chunk = rest ? p.chunk_rounds > p.both_rounds : !(round & 1);
    const int at = (rest ? round - p.both_rounds : round >> 1) * kUnits + i % kUnits;
    if (chunk) {
        const int share = divide(at, p.by_chunk_groups);
        // the arguments read apart from those of blocks: read for both at the start, they are spilled over the loop (5%)
        typedef __attribute__((address_space(4))) const AttendParams* Args;
        Args args = (Args)__builtin_amdgcn_kernarg_segment_ptr();
        asm volatile("" : "+s"(args));
        if (share < p.splits) chunk_body<DP, X, NP>(*(const AttendParams*)args, at - share * p.chunk_groups, share, lds);
    } else {
        if (threadIdx.x < 256 && at < p.block_groups) block_body<Both<DP, NP, NR>::kBlock, X, NP, NR, true>(p, at, lds);
    }
}

template <int DP, class X, int NP, int NR>
const void* chunk_kernel_shape(ChunkShape* shape)
{
    typedef Both<DP, NP, NR> B;
    *shape = ChunkShape{Chunk<DP>::kRows, Chunk<DP>::kWaves * 64, B::kAtOnce, B::kLds};
    return (const void*)&chunk_kernel<DP, X, NP, NR>;
}
template <int DP, class X, int NP>
const void* chunk_kernel_rows(int row_tiles, ChunkShape* shape)
{
    return row_tiles == 1 ? chunk_kernel_shape<DP, X, NP, 1>(shape) : chunk_kernel_shape<DP, X, NP, 2>(shape);
}

template <int DP>
const void* chunk_kernel_types(bool f16, bool f32_out, int row_tiles, ChunkShape* shape)
{
    if (f16) return f32_out ? chunk_kernel_rows<DP, _Float16, 2>(row_tiles, shape) : chunk_kernel_rows<DP, _Float16, 1>(row_tiles, shape);
    return f32_out ? chunk_kernel_rows<DP, __bf16, 3>(row_tiles, shape) : chunk_kernel_rows<DP, __bf16, 1>(row_tiles, shape);
}

}  // namespace ops
