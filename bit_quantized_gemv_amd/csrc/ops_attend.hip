// ops_attend.hip -- qmv_attend: attention of each sequence's new tokens over the
// pages of a cache.  What is launched for a call, and the join of what its workgroups found.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ops_attend.hpp"

namespace ops {
namespace {

constexpr int kThreads = 256;
constexpr int kMostGroups = 16384;         // of blocks, before they take several units each
constexpr long long kManyGroups = 4096;    // beside chunks, of which most have nothing to do

constexpr int kLanes = 16;                 // of a row's 64 columns
constexpr int kChains = kThreads / kLanes;

// The parts of rows, joined: those of blocks, and those of chunks, which are `splits` supers each.  Leaves
// are joined to supers one after the other, as the block's kernel does it; a row is the sum of its
// supers, each with its weight against the row's largest score, in order: first eights of them,
// then those.  A workgroup takes 64 columns of 2^-chains_log2 of 16 rows of a sequence (kRows), of some times
// as many (kMoreRows: 20 registers more and 0.7 us), or of a token's rows (kTokens).  Bound by latency, of the arguments, the sequence and the parts: 4.2 us
// for 32 rows of 4 parts, 6.5 for 32 rows of 128; every group of 16 lanes asks for eight parts at once.
// 16384 rows of 4 parts of 128 values (33 MB): 11 us.
enum class Join { kRows, kMoreRows, kTokens };

template <Join HOW>
__global__ __launch_bounds__(kThreads) void join_kernel(AttendParams p, int leaf, int block_chains, int chunk_chains, int columns, Divisor by_columns, int turns, Divisor by_turns)
{
    __shared__ __align__(16) f32x4 sums[kThreads];
    __shared__ f32x2 stats[kChains];
    __shared__ float tops[kChains];
    const Cache& c = p.cache;
    together(p.part, p.stat, p.chunk_part, p.chunk_stat, p.out, c.starts, c.lengths, c.n_seqs, c.max_places, c.T, p.units, p.per_unit, p.splits, p.apart, p.q_heads, p.D,
             p.window, p.sinks, p.max_new, p.out_f32, p.by_seqs.magic, p.by_seqs.shift, leaf, block_chains, chunk_chains, columns, by_columns.magic, by_columns.shift, turns,
             by_turns.magic, by_turns.shift);
    int b, over = blockIdx.y * gridDim.x + blockIdx.x, token = 0;
    if constexpr (HOW == Join::kTokens) {
        const int all = divide(over, by_columns);
        token = divide(all, by_turns);
        over -= token * turns * columns;
        if (token >= c.T) return;
        b = __builtin_amdgcn_readfirstlane(sequence_of(c, token, threadIdx.x & 63));
        if (b < 0) return;
    } else {
        const Turn at_turn = turn_of(over, p);
        over = at_turn.turn;
        b = at_turn.b;
    }
    const int turn = divide(over, by_columns), column = over - turn * columns;
    if (turn >= turns) return;
    const Seq s = sequence(c, b);
    const int tokens = min(s.count, p.max_new), place0 = s.length - s.count;
    const bool chunk = tokens > kBlockTokens;
    const int slots = chunk ? p.splits : p.units;
    if (slots <= 1) return;      // written already
    const int tid = threadIdx.x, lane = tid & (kLanes - 1), group = tid / kLanes;
    const int chains_log2 = chunk ? chunk_chains : block_chains, chains = 1 << chains_log2;
    const int chain = group & (chains - 1), team = group >> chains_log2;
    const int d = column * 64 + lane * 4, rows = kChains >> chains_log2;
    const bool leaves = !chunk && p.per_unit == 1;
    // the row's parts, and their eights: supers of leaves, or eights of supers
    Visible vis = visible(place0, tokens, p.window, p.sinks, leaf * p.per_unit), eights = visible(place0, tokens, p.window, p.sinks, leaf * p.per_unit * kSuper);
    if (chunk) {
        vis = Visible{0, 0, 0, 0, 0, slots};
        eights = Visible{0, 0, 0, 0, 0, (slots + kSuper - 1) / kSuper};
    }
    const long long first = chunk ? (long long)s.start * p.q_heads : block_row(p, b, s.start);
    // the rows of the sequence, or of the token
    int r_from = 0, r_to = tokens * p.q_heads;
    if constexpr (HOW == Join::kTokens) {
        const int i = token - s.start;
        if (i < 0 || i >= tokens) return;
        r_from = i * p.q_heads;
        r_to = r_from + p.q_heads;
    }
    for (int r0 = r_from + turn * rows; r0 < r_to; r0 += turns * rows) {
        const int r = r0 + team;
        const bool mine = r < r_to, mine_d = mine && d < p.D;
        const long long row = (long long)s.start * p.q_heads + r;
        const f32x2* stat = (chunk ? p.chunk_stat : p.stat) + (first + r) * slots;
        const float* part = (chunk ? p.chunk_part : p.part) + (first + r) * slots * p.D + d;
        // the parts of the first round are on their way while the largest score is found
        f32x2 st[kSuper];
        f32x4 pa[kSuper];
        int at[kSuper];
        auto ask = [&](int e) {
            const int from = e < eights.units ? eights.unit(e) * kSuper : 0;
#pragma unroll
            for (int i = 0; i < kSuper; ++i) {
                const int u = from + i, last = vis.units - vis.front;
                at[i] = e >= eights.units ? -1 : u < vis.front ? u : u >= vis.start && u - vis.start < last ? u - vis.start + vis.front : -1;
                st[i] = f32x2{kGone, 0.0f};
                pa[i] = f32x4{0, 0, 0, 0};
                if (mine && at[i] >= 0) {
                    st[i] = stat[at[i]];
                    if (mine_d) pa[i] = *reinterpret_cast<const f32x4*>(part + (long long)at[i] * p.D);
                }
            }
        };
        ask(chain);
        float top = kGone;
        if (mine)
            for (int u = chain * kLanes + lane; u < vis.units; u += chains * kLanes) top = __builtin_fmaxf(top, stat[u].x);
#pragma unroll
        for (int i = 1; i < kLanes; i <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, i));
        if (lane == 0) tops[group] = top;
        lds_only_barrier();
        for (int i = 0; i < chains; ++i) top = __builtin_fmaxf(top, tops[(team << chains_log2) + i]);
        const float base = top == kGone ? 0.0f : top;

        // o, l: sums of whole eights; oe, le: of the eight that is being added up
        float l = 0.0f, le = 0.0f;
        f32x4 o = {0, 0, 0, 0}, oe = {0, 0, 0, 0};
        int eight = -1;
        for (int e0 = 0; e0 < eights.units; e0 += chains) {
            if (e0 > 0) {
                ask(e0 + chain);
                lds_only_barrier();
            }
            float ls = 0.0f;
            f32x4 os = {0, 0, 0, 0};
            if (leaves) {
                float ms = kGone;
#pragma unroll
                for (int i = 0; i < kSuper; ++i) {
                    if (at[i] < 0) continue;
                    const Factors f = join(ms, ls, st[i].x, st[i].y);
                    os = joined(os, pa[i], f);
                }
                stats[group] = f32x2{ls, exp2_of(ms - base)};
            } else {
#pragma unroll
                for (int i = 0; i < kSuper; ++i) {
                    const float w = exp2_of(st[i].x - base);
                    ls = __builtin_fmaf(st[i].y, w, ls);
#pragma unroll
                    for (int c = 0; c < 4; ++c) os[c] = __builtin_fmaf(pa[i][c], w, os[c]);
                }
                stats[group] = f32x2{ls, 0.0f};
            }
            sums[tid] = os;
            lds_only_barrier();
            if (chain == 0) {
                const int n = min(chains, eights.units - e0);
                for (int i = 0; i < n; ++i) {
                    const f32x2 t = stats[group + i];
                    const f32x4 v = sums[tid + i * kLanes];
                    if (leaves) {
                        const int now = eights.unit(e0 + i) / kSuper;
                        if (now != eight) {
                            l += le;
                            o += oe;
                            le = 0.0f;
                            oe = f32x4{0, 0, 0, 0};
                            eight = now;
                        }
                        le = __builtin_fmaf(t.x, t.y, le);
#pragma unroll
                        for (int c = 0; c < 4; ++c) oe[c] = __builtin_fmaf(v[c], t.y, oe[c]);
                    } else {
                        l += t.x;
                        o += v;
                    }
                }
            }
        }
        l += le;
        o += oe;
        if (mine_d && chain == 0) put_result(p, row, d, o, l);
        if constexpr (HOW == Join::kRows) return;
        lds_only_barrier();
    }
}

int check_sizes(const qmv_cache* c, int T, int q_heads, int max_new, int max_length, int window, int sinks)
{
    if (int e = check_cache_sizes(c, T, q_heads)) return e;
    return max_new < 1 || max_length < 0 || window < 0 || sinks < 0 ? QMV_E_CACHE : QMV_OK;
}

// How a call is cut up: by its sizes alone.
struct Plan {
    int max_new, length, window, sinks;           // as far as they matter
    int bound, leaf;
    int row_tiles, row_blocks, per_unit;          // blocks: a workgroup's tiles of rows, and a unit's leaves
    long long units;                              // of a sequence, at most
    long long share;                              // and those that a workgroup takes
    long long chunk_tiles;                        // chunks: tiles of rows of all of them, at most
    int splits;                                   // and the shares of their keys
    const void *block, *chunk;
    int block_lds;
    ChunkShape shape;
    int block_chains, chunk_chains, columns;      // the join: groups of lanes to a row, and blocks of 64 columns
    long long join_turns, join_groups;            // workgroups of 64 columns of a sequence or token, and all of them
    Join join;                                    // of a sequence's, or of a token's
    int apart;                                    // rows of a sequence among the parts of blocks; 0: as in q
    long long part_bytes, stat_bytes, chunk_part_bytes, chunk_stat_bytes;
    long long bytes() const { return part_bytes + stat_bytes + chunk_part_bytes + chunk_stat_bytes; }
};

// units of U places that `tokens` neighbouring ones see at most
long long units_of(const Plan& p, int tokens, long long U)
{
    const long long all = std::max<long long>(1, (p.length + U - 1) / U);
    if (p.window == 0) return all;
    return std::min(all, (std::min(p.sinks, p.length) + U - 1) / U + ((long long)p.window + tokens - 1 + U - 1) / U + 1);
}

// groups of lanes that share a row of so many parts
int chains_of(long long parts)
{
    int log2 = 0;
    while (1 << log2 < std::min<long long>(kChains, (parts + kSuper - 1) / kSuper)) ++log2;
    return log2;
}

Plan plan_of(const qmv_cache* c, int T, int q_heads, int max_new, int max_length, int window, int sinks, bool f32_out)
{
    Plan p;
    p.max_new = std::min(max_new, T);
    p.length = (int)std::min<long long>(max_length, (long long)c->max_pages * c->page_size);
    p.window = std::min(window, QMV_MAX_LENGTH);
    p.sinks = window > 0 ? std::min(sinks, QMV_MAX_LENGTH) : 0;
    p.bound = c->head_size <= 64 ? 64 : c->head_size <= 128 ? 128 : 256;
    const bool f16 = c->dt == QMV_DT_F16;
    const int group = q_heads / c->heads, tokens = std::min(p.max_new, kBlockTokens);
    // Beside chunks, blocks are taken to be single tokens (others are more tiles of rows, which read the
    // keys again): 9 sequences of 1 to 13 tokens of 5 query heads to a head, 10.0 us for 13.1.
    const int rows = tokens * group, usual = p.max_new > kBlockTokens ? group : rows;
    p.leaf = leaf_keys(p.bound);
    auto blocks = [&](int tiles) { return (rows + 16 * tiles - 1) / (16 * tiles); };
    p.row_tiles = usual <= 16 ? 1 : usual <= 32 || p.max_new > kBlockTokens ? 2 : 4;
    // Leaf by leaf while those are about as many workgroups as run at once, a further tile of rows
    // counted as a third of one.  One token, 8 heads of 128, us: 16384 places 22.6 by leaves and 29.0 by
    // supers, 32768 42.9 and 39.0; 26 rows of 8 heads of 256, 8192 places: 34.6 and 28.7.
    const long long lists = (long long)c->heads * std::min(c->n_seqs, T);
    p.per_unit = units_of(p, tokens, p.leaf) * lists * blocks(p.row_tiles) * (2 + p.row_tiles) / 3 > 1200 ? kSuper : 1;
    p.units = units_of(p, tokens, (long long)p.leaf * p.per_unit);
    // Supers are few: four tiles of rows a workgroup only where that leaves two workgroups for every
    // compute unit, two where it leaves three for four.  13 tokens, 64 query heads on 8 of 128, 8192 places, us: 47.6
    // with four, 33.2 with two, 39.8 with one; 32 sequences of half the query heads, 2048: 82, 99, 137;
    // 16 on 8 of 256, 8192: 33.7 with two, 28.7 with one, 12000: 35.7 and 43.9.
    if (p.per_unit > 1) {
        while (p.row_tiles > 1 && p.units * lists * blocks(p.row_tiles) < (p.row_tiles == 4 ? 8 : 3) * kUnits / 4) p.row_tiles /= 2;
    }
    // Beside chunks, a workgroup takes further tiles of rows where those would be many workgroups, most without work.
    // 127 sequences of 5 tokens of 1000 places beside a chunk of 512, us: 203 for 304; 255 single tokens: 303 for 311,
    // or, with a bound of eight times their places, 324 for 311.
    if (p.max_new > kBlockTokens && p.units * lists * (blocks(p.row_tiles) - 1) > kManyGroups) p.row_tiles = 2;
    p.row_blocks = blocks(p.row_tiles);
    // A workgroup takes several units, one after the other, where there would be more than kMostGroups: most
    // have nothing to do then, their bounds being wide.  256 single tokens of 1000 places, 8 heads of 128, us, with a
    // bound of 131072: 292, 699 with a workgroup a unit; 203 with a bound of 1024.
    p.share = p.window > 0 ? 1 : std::min(p.units, (p.units * lists * p.row_blocks + kMostGroups - 1) / kMostGroups);
    p.block = p.bound == 64    ? block_kernel_64(f16, f32_out, p.share > 1, p.row_tiles, &p.block_lds)
              : p.bound == 128 ? block_kernel_128(f16, f32_out, p.share > 1, p.row_tiles, &p.block_lds)
                               : block_kernel_256(f16, f32_out, p.share > 1, p.row_tiles, &p.block_lds);
    // a chunk's kernel multiplies all the columns that it is made for
    const auto chunk = c->head_size <= 64    ? chunk_kernel_64
                       : c->head_size <= 96  ? chunk_kernel_96
                       : c->head_size <= 128 ? chunk_kernel_128
                       : c->head_size <= 192 ? chunk_kernel_192
                                             : chunk_kernel_256;
    p.chunk = chunk(f16, f32_out, std::min(p.row_tiles, 2), &p.shape);
    p.chunk_tiles = 0;
    p.splits = 1;
    if (p.max_new > kBlockTokens) {
        // As many shares as there is room for on the compute units, of 256 keys at least; a chunk has more
        // tokens than a block, so T bounds how many there are.  512 tokens over 4096 places, 32 heads on 8 of
        // 128 (128 workgroups a share, room for four), us: 130 with one share, 81, 73, 62 with four, 77 with six;
        // 4096 over 4096: 180 with one, 239 with two.
        const long long chunks = std::min<long long>(c->n_seqs, T / (kBlockTokens + 1));
        p.chunk_tiles = std::min(chunks * (((long long)p.max_new * group + p.shape.rows - 1) / p.shape.rows), (long long)T * group / p.shape.rows + chunks);
        const long long room = kUnits * p.shape.at_once / std::max<long long>(1, p.chunk_tiles * c->heads);
        const long long most = (std::min<long long>(p.length, p.window ? (long long)p.window + p.sinks + p.shape.rows / group : p.length) + 255) / 256;
        p.splits = (int)std::max<long long>(1, std::min(room, most));
    }
    p.columns = (c->head_size + 63) / 64;
    p.block_chains = chains_of(p.units);
    p.chunk_chains = chains_of(p.splits);
    auto joins = [&](long long rows, long long parts, int chains) { return parts > 1 ? (rows + (kChains >> chains) - 1) / (kChains >> chains) : 0; };
    // A workgroup for every 16 rows (or fewer of many parts) of a sequence, as many for each as the longest may have.  Where
    // chunks have parts and that is twice what the tokens have, a token's instead: 15 single tokens of 4000 places beside
    // a chunk of 512 tokens in two shares, whole calls, us: 85, by sequences 96; the chunk alone 61.8 and 59.5.  Where only
    // blocks beside chunks have parts, kManyGroups if those are fewer than half, and one token's at least, of blocks and of
    // chunks, whichever have parts; they then take more rows: the join of 255 single tokens beside a chunk of 2048 11 for 31.
    p.join = Join::kRows;
    p.join_turns = std::max(joins((long long)tokens * q_heads, p.units, p.block_chains), joins((long long)p.max_new * q_heads, p.splits, p.chunk_chains));
    const long long of_token = joins(q_heads, p.splits, p.chunk_chains);
    const long long most = std::max({joins(q_heads, p.units, p.block_chains), of_token, kManyGroups / (p.columns * c->n_seqs)});
    if (p.splits > 1 && p.join_turns * c->n_seqs > 2 * of_token * T) {
        p.join = Join::kTokens;
        p.join_turns = of_token;
    } else if (p.max_new > kBlockTokens && p.join_turns > 2 * most) {
        p.join = Join::kMoreRows;
        p.join_turns = most;
    }
    p.join_groups = p.join_turns * p.columns * (p.join == Join::kTokens ? T : c->n_seqs);
    p.apart = (long long)c->n_seqs * tokens < T ? tokens : 0;
    const long long parts = p.units > 1 ? (long long)(p.apart > 0 ? c->n_seqs * tokens : T) * q_heads * p.units : 0;
    const long long chunk_parts = p.splits > 1 ? (long long)T * q_heads * p.splits : 0;
    p.part_bytes = piece(parts * c->head_size * 4);
    p.stat_bytes = piece(parts * 8);
    p.chunk_part_bytes = piece(chunk_parts * c->head_size * 4);
    p.chunk_stat_bytes = piece(chunk_parts * 8);
    return p;
}

// so many workgroups, as blockIdx.y * gridDim.x + blockIdx.x counts them (and some more)
dim3 grid_of(long long groups)
{
    const long long wide = std::min<long long>(groups, 1 << 19);
    return dim3((unsigned)wide, (unsigned)((groups + wide - 1) / wide));
}

int launch(const void* f, dim3 grid, int threads, void** args, int lds, void* stream)
{
    return hipLaunchKernel(f, grid, dim3(threads), args, (size_t)lds, static_cast<hipStream_t>(stream)) == hipSuccess ? QMV_OK : QMV_E_LAUNCH;
}

}  // namespace
}  // namespace ops

extern "C" {

long long qmv_attend_workspace(const qmv_cache* c, int T, int q_heads, int max_new, int max_length,
                               int window, int sinks)
{
    using namespace ops;
    if (!c || check_sizes(c, T, q_heads, max_new, max_length, window, sinks) != QMV_OK) return -1;
    const Plan plan = plan_of(c, T, q_heads, max_new, max_length, window, sinks, false);
    return plan.bytes();
}

int qmv_attend(const qmv_cache* c, const void* q, void* out, void* workspace,
               long long workspace_bytes, int T, int q_heads, long long q_token, long long q_head,
               int max_new, int max_length, int window, int sinks, float scale, int out_dt,
               void* stream)
{
    using namespace ops;
    if (!c || !q || !out) return QMV_E_NULL;
    if (int e = check_sizes(c, T, q_heads, max_new, max_length, window, sinks)) return e;
    CacheSpans cs;
    if (int e = check_cache(c, T, q_heads, &cs)) return e;
    if (!wide(out_dt)) return QMV_E_DTYPE;
    if (!stride_ok(q_token) || !stride_ok(q_head)) return QMV_E_STRIDE;
    if (q_token % 8 != 0 || q_head % 8 != 0 || !aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16)) return QMV_E_ALIGN;
    const long long size[] = {T, q_heads}, stride[] = {q_token, q_head}, nq = extent(size, stride, c->head_size);
    if (nq < 0) return QMV_E_STRIDE;
    const Plan plan = plan_of(c, T, q_heads, max_new, max_length, window, sinks, out_dt == QMV_DT_F32);
    const long long need = plan.bytes();
    if (need > 0 && !workspace) return QMV_E_NULL;
    if (workspace_bytes < need) return QMV_E_WORKSPACE;
    const Span in[] = {{q, (size_t)nq * 2}, {c->k, cs.k}, {c->v, cs.v}, {c->pages, cs.pages}, {c->starts, (size_t)(c->n_seqs + 1) * 4},
                       {c->lengths, (size_t)c->n_seqs * 4}};
    const Span outs[] = {{out, (size_t)T * q_heads * c->head_size * size_of(out_dt)}, {workspace, (size_t)need}};
    if (!disjoint(in, outs)) return QMV_E_ALIAS;
    // rows are counted, and a launch's threads, in 32 bits
    const long long shares = (plan.units + plan.share - 1) / plan.share, groups = (shares * c->n_seqs + 7) / 8 * 8 * c->heads * plan.row_blocks;
    const long long chunk_groups = plan.chunk_tiles * c->heads;
    if ((long long)plan.max_new * q_heads > 1 << 30 || groups >= 1LL << 30 || chunk_groups * plan.splits >= 1LL << 30 || plan.join_groups >= 1LL << 31) return QMV_E_CACHE;
    AttendParams p;
    p.q = static_cast<const char*>(q);
    p.out = static_cast<char*>(out);
    char* const scratch = static_cast<char*>(workspace);
    p.part = reinterpret_cast<float*>(scratch);
    p.stat = reinterpret_cast<f32x2*>(scratch + plan.part_bytes);
    p.chunk_part = reinterpret_cast<float*>(scratch + plan.part_bytes + plan.stat_bytes);
    p.chunk_stat = reinterpret_cast<f32x2*>(scratch + plan.part_bytes + plan.stat_bytes + plan.chunk_part_bytes);
    p.apart = plan.apart;
    p.q_token = 2 * q_token;
    p.q_head = 2 * q_head;
    p.q_heads = q_heads;
    p.heads = c->heads;
    p.group = q_heads / c->heads;
    p.D = c->head_size;
    p.window = plan.window;
    p.sinks = plan.sinks;
    p.max_new = plan.max_new;
    p.out_f32 = out_dt == QMV_DT_F32;
    p.units = (int)plan.units;
    p.shares = (int)shares;
    p.splits = plan.splits;
    p.row_blocks = plan.row_blocks;
    p.rows_last = plan.max_new > kBlockTokens ? (int)(groups / 8 / plan.row_blocks) : 0;
    p.per_unit = plan.per_unit;
    // A scale of zero weighs all places that are seen alike; the smallest number, by which no score is 2^-20, does so too, and
    // leaves the -inf of the others.
    p.scale = scale == 0.0f ? 0x1p-149f : scale * 1.44269504088896340736f;
    p.by_group = divisor(p.group);
    p.by_heads = divisor(p.heads);
    p.by_seqs = divisor(c->n_seqs);
    p.by_rows = divisor(p.rows_last > 0 ? p.rows_last : p.row_blocks);
    p.cache = device_cache(c, T);
    p.cache.max_places = plan.length;
    void* args[] = {&p};
    if (chunk_groups > 0) {
        p.chunk_groups = (int)chunk_groups;
        p.by_chunk_groups = divisor(p.chunk_groups);
        p.block_groups = (int)groups;
        p.chunk_rounds = (int)((chunk_groups * plan.splits + kUnits - 1) / kUnits);
        const int block_rounds = (int)((groups + kUnits - 1) / kUnits);
        p.both_rounds = std::min(p.chunk_rounds, block_rounds);
        if (int e = launch(plan.chunk, grid_of((p.chunk_rounds + (long long)block_rounds) * kUnits), plan.shape.threads, args, plan.shape.lds, stream)) return e;
    } else if (int e = launch(plan.block, grid_of(groups), kThreads, args, plan.block_lds, stream)) {
        return e;
    }
    if (p.units == 1 && p.splits == 1) return QMV_OK;
    int leaf = plan.leaf, block_chains = plan.block_chains, chunk_chains = plan.chunk_chains, columns = plan.columns;
    int turns = (int)plan.join_turns;
    Divisor by_columns = divisor(columns), by_turns = divisor(turns);
    void* join[] = {&p, &leaf, &block_chains, &chunk_chains, &columns, &by_columns, &turns, &by_turns};
    const void* const f = plan.join == Join::kRows       ? (const void*)&join_kernel<Join::kRows>
                          : plan.join == Join::kMoreRows ? (const void*)&join_kernel<Join::kMoreRows>
                                                         : (const void*)&join_kernel<Join::kTokens>;
    return launch(f, grid_of(plan.join_groups), kThreads, join, 0, stream);
}

}  // extern "C"
