// ops_tile.hpp -- the quantized tile product shared by the operators beside
// qmv: a wavefront multiplies 16*RT weight rows with 16*CT activation rows over
// a range of K on matrix instructions.
//
// The mathematics.  For one group g of a weight row n and a token m,
//     s * sum_k q x + b * sum_k x .
// A 4-bit code placed in the upper mantissa bits of a bf16 of exponent 4 is the
// number 16 + q, exactly, for one shift and one and-or per two codes (2 bits:
// 4 + q).  With C0 = sum_k (-16) x from one matrix instruction on a constant
// operand, D = C0 + sum_k (16 + q) x = sum_k q x, so the offset costs no vector
// arithmetic, and sum_k x = -C0/16.  The group's fold is two fmas:
//     acc += s * D;   acc += (-b/16) * C0 .
// Products of bf16 values are exact in the matrix instruction and add in fp32.
//
// The layout.  v_mfma_f32_16x16x32_bf16 with the tokens as the first operand's
// rows and the weight rows as the second's columns: lane l holds token (l & 15)
// and weight row (l & 15) at k = 8 * (l >> 4) + j, and the result of weight row
// (l & 15), tokens 4 * (l >> 4) + i.  So the lane that multiplies a row's codes also
// needs that row's scale and bias, and no exchange is needed for the fold.  A row's
// slab is four 16-byte pieces, one per lane that multiplies it; where those hold
// more than one group, permlane swaps turn the four lanes' words so that every
// matrix instruction's k lies in one group.
//
// Codes.  The vector memory unit takes a wave's addresses four lanes at a time,
// and lanes that multiply neighbouring rows would have it look up a cache line for
// every lane.  So four neighbouring lanes load the 64 bytes of one row, and the
// wave turns the pieces over through LDS (a write and a read of 16 bytes a lane,
// one slab ahead; which piece a lane loads is swizzled so that the reads meet
// distinct banks).  Without this, and with scales loaded by each lane for itself, a
// 17408 x 5120 product of 16 tokens took 51 us; with both, 29.  Codes are asked for by
// two slabs, the two halves of a cache line: one at a time, half of the lines were
// read from memory twice (128 experts, 13 tokens: 249 MB for 157; by two, 168).  Rows
// that start inside a line still meet lines twice, so the loads leave them in the
// caches: as nontemporal ones, 32 experts of 3840 x 1920 in 2 bits read 394 MB for 199
// and took 154 us, against 143.
//
// Scales and biases go to LDS before the product, whole rows at a time: a row's
// few bytes per slab would cost as many lookups as its codes.
//
// Activations come packed (packed_word): one bf16 plane, or three that add up to
// an fp32 value exactly, with the two values that a dword of codes meets next to
// each other and the pieces in the order of the lanes, so they are operands as
// loaded; 16 tokens together (FRAG), or each by itself where they are gathered.
//
// The pipeline.  A wave keeps PF slabs of codes and activations in flight in
// registers.  Loads come back in order, so the activations, though near, are asked
// for as early as the codes: an activation load waited for would otherwise wait for
// every code load before it.  The loop body has no branch around a load, which would
// make each wait assume the shorter path, and the loads keep their order (slab by slab,
// before the loop as in it): a wait counts the loads after the one it needs, and takes
// the smaller count of the two ways in.
//
// What bounds it: with one token, the read of the codes and the start and end of a
// workgroup (15360 x 3840 in 13.4 us, of which the codes and scales are 6.8 at the
// rate of a large copy); from about 32 tokens the vector instructions of decoding and
// folding beside the matrix instructions.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ops_args.hpp"

namespace ops {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr int kWave = 64;
constexpr int kMaxWaves = 8;        // of a workgroup

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float bits_f32(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t f32_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

// the high halves of two words: (hi(b) << 16) | hi(a); and the low halves
__device__ __forceinline__ uint32_t hi16(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }
__device__ __forceinline__ uint32_t lo16(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }

__device__ __forceinline__ float half_bits(uint32_t u)   // fp16 in the low 16 bits
{
    return (float)__builtin_bit_cast(_Float16, (uint16_t)u);
}

// An fp32 value as three bf16 values that add up to it exactly (8 bits each,
// truncated): returned as fp32 bit patterns whose low halves are zero.
__device__ __forceinline__ void split3(float v, uint32_t& h, uint32_t& m, uint32_t& l)
{
    h = f32_bits(v) & 0xffff0000u;
    const float r = v - bits_f32(h);
    m = f32_bits(r) & 0xffff0000u;
    l = f32_bits(r - bits_f32(m));
}

// round to nearest even; NaN stays NaN
__device__ __forceinline__ uint16_t to_bf16(float f)
{
    const uint32_t u = f32_bits(f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40u);
    return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
}

__device__ __forceinline__ void store_y(void* y, size_t at, float v, bool f32)
{
    if (f32)
        static_cast<float*>(y)[at] = v;
    else
        static_cast<uint16_t*>(y)[at] = to_bf16(v);
}

// nothing but loads and stores from memory stays on its side
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0x78F); }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Slabs of K a row of `chunks` 16-byte pieces is walked in, four pieces each.
__host__ __device__ inline int slabs_of(int chunks) { return (chunks + 3) / 4; }

// Parts that a row's K is cut into, a wave each: enough waves to keep loads in
// flight where rows are few, and enough slabs per wave to pay for its start
// and the join.  Depends on the row length alone, as the order of the join does.
__host__ __device__ inline int parts_of(int chunks)
{
    const int n = slabs_of(chunks);
    return n >= 64 ? 8 : n >= 24 ? 4 : n >= 4 ? 2 : 1;
}

// The slabs of a part: whole pairs, since two slabs of a row share a cache line.
__host__ __device__ inline int part_start(int slabs, int log_parts, int part)
{
    const int at = (part * ((slabs + 1) / 2) >> log_parts) * 2;
    return at < slabs ? at : slabs;
}

// Small quotients: a / b with inv = 1 / b, for a below 2^20.  (A division by a number
// that is not known when compiling is some forty instructions, and a kernel's start
// is a good part of its time.)
__device__ __forceinline__ int small_div(int a, float inv) { return (int)(((float)a + 0.5f) * inv); }

// Waves of a workgroup, and row tile groups: the parts of several groups of rows.
__host__ __device__ inline int waves_of(int parts) { return parts > 4 ? parts : 4; }

// Where a row's packed word lies among a slab's operands, 16 words to a slab: the
// group and word of the lane and the lane's quarter.
struct WordAt {
    int op, q;       // first operand of the word; (l >> 4) of the lane
};

__host__ __device__ inline WordAt word_at(int w, int bits, int gs)
{
    const int fpw = bits == 4 ? 1 : 2, ng = 16 * (32 / bits) / gs;
    if (ng == 1) return {(w & 3) * fpw, w >> 2};
    if (ng == 2) return {((w >> 3) * 2 + (w & 1)) * fpw, ((w >> 2) & 1) | (w & 2)};
    return {(w >> 2) * fpw, w & 3};
}

// Packed activations: planes of [tiles of 16 tokens][slabs][operands][64 lanes][16 bytes]
// (FRAG), or of [tokens][slabs][operands][4 quarters][16 bytes].
struct Packed {
    int bits, gs, slabs, ops;
    bool frag;
    __host__ __device__ Packed(int K, int bits_, int gs_, bool frag_)
        : bits(bits_), gs(gs_), slabs(slabs_of(K * bits_ / 128)), ops(bits_ == 4 ? 4 : 8), frag(frag_)
    {
    }
    __host__ __device__ size_t plane(int tokens) const { return (size_t)(frag ? (tokens + 15) / 16 * 16 : tokens) * slabs * ops * 64; }
    // byte offset of the first operand of word w (of a whole row) of a token; further ones are op_step() on
    __device__ __forceinline__ size_t word(int token, int w) const
    {
        const WordAt a = word_at(w & 15, bits, gs);
        if (frag) return (((size_t)(token >> 4) * slabs + (w >> 4)) * ops + a.op) * 1024 + a.q * 256 + (token & 15) * 16;
        return (((size_t)token * slabs + (w >> 4)) * ops + a.op) * 64 + a.q * 16;
    }
    __device__ __forceinline__ int op_step() const { return frag ? 1024 : 64; }
};

// One word's activations, VPW values at `from` (fp32 or bf16), to the planes at `to`.
template <int BITS, bool F32>
__device__ __forceinline__ void pack_word(const char* from, char* to, size_t plane, int step)
{
    constexpr int VPW = 32 / BITS, H = VPW / 2, NV = VPW * (F32 ? 4 : 2) / 16;
    u32x4 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = reinterpret_cast<const u32x4*>(from)[i];
    u32x4 o[F32 ? 3 : 1][H / 4];
#pragma unroll
    for (int i = 0; i < H; ++i) {       // dword i pairs values i and i + H
        if constexpr (F32) {
            uint32_t ah, am, al, bh, bm, bl;
            split3(bits_f32(v[i / 4][i % 4]), ah, am, al);
            split3(bits_f32(v[(i + H) / 4][(i + H) % 4]), bh, bm, bl);
            o[0][i / 4][i % 4] = hi16(ah, bh);
            o[1][i / 4][i % 4] = hi16(am, bm);
            o[2][i / 4][i % 4] = hi16(al, bl);
        } else {
            const uint32_t a = v[(i / 2) / 4][(i / 2) % 4], b = v[((i + H) / 2) / 4][((i + H) / 2) % 4];
            o[0][i / 4][i % 4] = (i & 1) ? hi16(a, b) : lo16(a, b);
        }
    }
#pragma unroll
    for (int p = 0; p < (F32 ? 3 : 1); ++p)
#pragma unroll
        for (int i = 0; i < H / 4; ++i) *reinterpret_cast<u32x4*>(to + p * plane + i * step) = o[p][i];
}

// Packs word number `at` of the tokens' rows of K values.
__device__ __forceinline__ void pack(const char* x, char* to, int tokens, int K, const Packed& pk, bool f32, size_t at)
{
    const int words = K * pk.bits / 32;
    if (at >= (size_t)tokens * words) return;
    const int t = (int)(at / words), w = (int)(at % words);
    const size_t k = (size_t)t * K + (size_t)w * (32 / pk.bits);
    char* o = to + pk.word(t, w);
    const size_t plane = pk.plane(tokens);
    if (pk.bits == 4) {
        if (f32)
            pack_word<4, true>(x + k * 4, o, plane, pk.op_step());
        else
            pack_word<4, false>(x + k * 2, o, plane, pk.op_step());
    } else {
        if (f32)
            pack_word<2, true>(x + k * 4, o, plane, pk.op_step());
        else
            pack_word<2, false>(x + k * 2, o, plane, pk.op_step());
    }
}

// Scales and biases of a workgroup's rows in LDS.  All groups of a row at once
// where they fit; else a window of each part's groups at a time.
struct Meta {
    Meta() = default;
    int groups;        // values per row in LDS: a row's and, where rows are whole 16-byte pieces, one piece
                       // more, which puts 16 rows on different banks
    int window;        // slabs of a part per window
    int windows;
    Meta(int rows, int K, int bits, int gs, int parts)       // on the host: a kernel argument
    {
        constexpr int kMost = 48 * 1024;
        const int G = K / gs, slabs = slabs_of(K * bits / 128), ng = 16 * (32 / bits) / gs;
        const int per = ((slabs + 1) / 2 + parts - 1) / parts * 2;
        if (rows * G * 4 <= kMost) {
            groups = G % 8 == 0 ? G + 8 : G;
            window = per;
            windows = 1;
        } else {
            window = kMost / (rows * 4 * parts * ng) & ~1;
            groups = parts * window * ng;
            windows = (per + window - 1) / window;
        }
    }
    __host__ __device__ int bytes(int rows) const { return rows * ((groups + 7) / 8 * 8) * 4; }     // both arrays, 16-byte pieces
};

template <int BITS_, int GS_, int RT_, int CT_, int NP_, bool SBF_, bool FRAG_>
struct Tile {
    static constexpr int BITS = BITS_, GS = GS_, RT = RT_, CT = CT_;
    static constexpr int NP = NP_;                    // planes of the activations
    static constexpr bool SBF = SBF_, FRAG = FRAG_;
    static constexpr int VPW = 32 / BITS;             // codes per word
    static constexpr int SLAB = 16 * VPW;             // codes of a row per slab
    static constexpr int NG = SLAB / GS;              // groups per slab
    static constexpr int WPG = 4 / NG;                // words of a lane per group
    static constexpr int FPW = VPW / 8;               // matrix instructions per word
    static constexpr int NF = WPG * FPW;              // and per group
    static constexpr int NM = (NG + 1) / 2;           // dwords of scales per slab
    static constexpr int XOP = FRAG ? 1024 : 64, XQ = FRAG ? 256 : 16;       // bytes from operand to operand, quarter to quarter
    static constexpr uint32_t MASK = BITS == 4 ? 0x00780078u : 0x00600060u;
    static constexpr uint32_t BASE = BITS == 4 ? 0x41804180u : 0x40804080u;  // 16, 4
    static constexpr uint32_t NEG = BITS == 4 ? 0xC180C180u : 0xC080C080u;   // -16, -4
    static constexpr float INV = BITS == 4 ? -1.0f / 16 : -1.0f / 4;
    // Slabs in flight: about 100 registers of them, four at most, or two.  The lightest
    // instances take two and a third wave per SIMD (one token, 15360 x 3840: 17.8 us against 18.8).  Codes go by two
    // slabs at once, the halves of a cache line, even where activations go one by one.
    static constexpr bool LIGHT = BITS_ == 4 && RT_ == 2 && CT_ == 1 && NP_ == 1;
    static constexpr int SLAB_REGS = 4 * NG * NF * NP * CT + RT * 4;
    static constexpr int PF = !LIGHT && SLAB_REGS * 4 <= 100 ? 4 : SLAB_REGS * 2 <= 100 ? 2 : 1;
    static constexpr int WPF = PF < 2 ? 2 : PF;
    // waves per SIMD that its kernels leave registers for
    static constexpr int WAVES = LIGHT ? 3 : 2;
    static constexpr int TURN = RT * 1024;            // bytes of LDS per wave to turn a slab over

    struct Rows {                  // what a wave multiplies
        const char* w[RT];         // the row tiles' codes (the same for all lanes)
        uint32_t wo[RT];           // the row whose piece the lane loads
        const uint16_t* s[RT];     // scales and biases of the lane's row in LDS, less the groups before the window
        const uint16_t* b[RT];
        const char* x[CT];         // the lane's token
        size_t plane;              // bytes between the activations' planes
        char* turn;
        int chunks, G;
        bool even;                 // LDS rows start at a multiple of a slab's groups
    };

    struct Ring {
        u32x4 w[WPF][RT];
        u32x4 x[PF][CT][NG][NF][NP];
    };

    static __device__ __forceinline__ int lane() { return threadIdx.x & 63; }

    // the piece that lane 4 r + i of a load has: of row r, and which of the four
    static __device__ __forceinline__ int piece() { return (lane() & 3) ^ ((lane() >> 3) & 3); }

    // codes of the tile i whose first row is `row`, of which `left` exist: lanes past them repeat the last
    static __device__ __forceinline__ void set_codes(Rows& r, int i, const void* w, size_t row, int left)
    {
        r.w[i] = static_cast<const char*>(w) + row * r.chunks * 16;
        r.wo[i] = (uint32_t)min(lane() >> 2, left - 1) * r.chunks * 16;
    }

    static __device__ __forceinline__ void set_token(Rows& r, int j, const char* x, int token)
    {
        const int q = lane() >> 4;
        r.x[j] = x + (FRAG ? (size_t)(token >> 4) * 16 : (size_t)token) * slabs_of(r.chunks) * (NG * NF * 64) + q * XQ + (FRAG ? (token & 15) * 16 : 0);
    }

    static __device__ __forceinline__ void load_w(Ring& t, int u, const Rows& r, int slab)
    {
        const uint32_t at = 16 * (uint32_t)min(4 * slab + piece(), r.chunks - 1);   // a part slab's pieces past the row repeat its last
#pragma unroll
        for (int i = 0; i < RT; ++i)
            t.w[u][i] = *reinterpret_cast<const u32x4*>(r.w[i] + (r.wo[i] + at));
    }

    static __device__ __forceinline__ void load_x(Ring& t, int u, int j, int g, const Rows& r, int slab)
    {
        const char* p = r.x[j] + (size_t)slab * (NG * NF * XOP);
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int e = 0; e < NP; ++e)
                t.x[u][j][g][f][e] = *reinterpret_cast<const u32x4*>(p + (g * NF + f) * XOP + e * r.plane);
    }

    // a slab's pieces from the lanes that loaded them to those that multiply them
    static __device__ __forceinline__ void turn(u32x4 (&w)[RT], const Ring& t, int u, const Rows& r)
    {
        const int c = lane() & 15, q = lane() >> 4;
        char* to = r.turn + lane() * 16;
        const char* from = r.turn + (4 * c + (q ^ ((c >> 1) & 3))) * 16;
#pragma unroll
        for (int i = 0; i < RT; ++i) *reinterpret_cast<u32x4*>(to + i * 1024) = t.w[u][i];
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < RT; ++i) w[i] = *reinterpret_cast<const u32x4*>(from + i * 1024);
        __builtin_amdgcn_wave_barrier();
    }

    static __device__ __forceinline__ void meta(uint32_t (&v)[NM], const uint16_t* p, bool even)
    {
        if constexpr (NG == 1) {
            v[0] = p[0];
        } else if (even) {
            if constexpr (NG == 2) {
                v[0] = *reinterpret_cast<const uint32_t*>(p);
            } else {
                const u32x2 t = *reinterpret_cast<const u32x2*>(p);
                v[0] = t[0];
                v[NM - 1] = t[1];
            }
        } else {
#pragma unroll
            for (int m = 0; m < NM; ++m) v[m] = p[2 * m] | ((uint32_t)p[2 * m + 1] << 16);
        }
    }

    static __device__ __forceinline__ float param(const uint32_t (&v)[NM], int g)
    {
        const uint32_t u = v[g / 2];
        if constexpr (SBF) return bits_f32((g & 1) ? (u & 0xffff0000u) : (u << 16));
        return half_bits((g & 1) ? (u >> 16) : (u & 0xffffu));
    }

    // the codes of matrix instruction f of a word, as 16 + q (4 + q)
    static __device__ __forceinline__ u32x4 w_operand(uint32_t w, int f)
    {
        u32x4 o;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int sh = BITS * (4 * f + d) - (BITS == 4 ? 3 : 5);
            o[d] = ((sh >= 0 ? w >> (sh & 31) : w << ((-sh) & 31)) & MASK) | BASE;
        }
        return o;
    }

    // acc += the slab whose codes are w and whose activations are slot u's; where
    // MORE, the activations of slab `next` go in flight in their place, piece by piece
    template <bool MORE, bool TAIL>
    static __device__ __forceinline__ void step(f32x4 (&acc)[RT][CT], u32x4 (&w)[RT], Ring& t, int u, const Rows& r, int slab, int next)
    {
        uint32_t s[RT][NM], b[RT][NM];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            meta(s[i], r.s[i] + slab * NG, r.even);
            meta(b[i], r.b[i] + slab * NG, r.even);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if constexpr (NG >= 2) {
                const auto p = __builtin_amdgcn_permlane32_swap(w[i][0], w[i][2], false, false);
                const auto v = __builtin_amdgcn_permlane32_swap(w[i][1], w[i][3], false, false);
                w[i] = u32x4{p[0], v[0], p[1], v[1]};
            }
            if constexpr (NG == 4) {
                const auto p = __builtin_amdgcn_permlane16_swap(w[i][0], w[i][1], false, false);
                const auto v = __builtin_amdgcn_permlane16_swap(w[i][2], w[i][3], false, false);
                w[i] = u32x4{p[0], p[1], v[0], v[1]};
            }
        }
        const u32x4 neg = {NEG, NEG, NEG, NEG};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (TAIL && g > 0 && slab * NG + g >= r.G) break;      // past the row's end, in its last slab
            if constexpr (BITS == 2) __builtin_amdgcn_sched_barrier(0);      // groups drawn together spill
            u32x4 wo[RT][NF];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int c = 0; c < WPG; ++c)
#pragma unroll
                    for (int f = 0; f < FPW; ++f) wo[i][c * FPW + f] = w_operand(w[i][g * WPG + c], f);
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                // The first plane and those below it add up apart: a sum passes through
                // 16 times its terms, and would be rounded there once more per plane.
                f32x4 c0 = {0.f, 0.f, 0.f, 0.f}, c1 = c0;
#pragma unroll
                for (int f = 0; f < NF; ++f)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        f32x4& to = p == 0 ? c0 : c1;
                        to = mfma(t.x[u][j][g][f][p], neg, to);
                    }
                f32x4 d[RT], d1[RT];
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    d[i] = c0;
                    d1[i] = c1;
                }
#pragma unroll
                for (int f = 0; f < NF; ++f)
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            f32x4& to = p == 0 ? d[i] : d1[i];
                            to = mfma(t.x[u][j][g][f][p], wo[i][f], to);
                        }
                if constexpr (MORE) {
                    keep_order();
                    load_x(t, u, j, g, r, next);
                    keep_order();
                }
                if constexpr (NP > 1) {
                    c0 += c1;
#pragma unroll
                    for (int i = 0; i < RT; ++i) d[i] += d1[i];
                }
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const float sc = param(s[i], g), nb = param(b[i], g) * INV;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][j][e] = __builtin_fmaf(nb, c0[e], __builtin_fmaf(sc, d[i][e], acc[i][j][e]));
                }
            }
        }
    }

    // slabs s0.. of [s0, s1) (s0 < s1, s0 even) go in flight
    static __device__ __forceinline__ void begin(Ring& t, const Rows& r, int s0, int s1)
    {
#pragma unroll
        for (int u = 0; u < WPF; ++u) {
            if (u % 2 == 0) {
                load_w(t, u, r, min(s0 + u, s1 - 1));
                load_w(t, u + 1, r, min(s0 + u + 1, s1 - 1));
                keep_order();
            }
            if (u < PF) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int j = 0; j < CT; ++j) load_x(t, u, j, g, r, min(s0 + u, s1 - 1));
                keep_order();
            }
        }
    }

    // acc += the products over slabs [s0, s1) (none if s0 >= s1), begun by begin.  A
    // slab's codes are turned over while the one before it is multiplied.
    static __device__ __forceinline__ void run(f32x4 (&acc)[RT][CT], Ring& t, const Rows& r, int s0, int s1)
    {
        if (s0 >= s1) return;
        u32x4 w[RT];
        turn(w, t, 0, r);
        int s = s0;
        for (; s + WPF < s1; s += WPF) {
#pragma unroll
            for (int u = 0; u < WPF; ++u) {
                __builtin_amdgcn_sched_barrier(0);
                u32x4 n[RT];
                turn(n, t, (u + 1) % WPF, r);
                if (u % 2 == 0) {                              // both slots' codes are in w and n
                    keep_order();
                    load_w(t, u, r, min(s + u + WPF, s1 - 1));
                    load_w(t, u + 1, r, min(s + u + 1 + WPF, s1 - 1));
                    keep_order();
                }
                step<true, false>(acc, w, t, u % PF, r, s + u, min(s + u + PF, s1 - 1));
#pragma unroll
                for (int i = 0; i < RT; ++i) w[i] = n[i];
            }
        }
#pragma unroll
        for (int u = 0; u < WPF; ++u)
            if (s + u < s1) {
                __builtin_amdgcn_sched_barrier(0);
                u32x4 n[RT];
                if (u + 1 < WPF) turn(n, t, (u + 1) % WPF, r);
                if (u + PF < WPF)
                    step<true, true>(acc, w, t, u % PF, r, s + u, min(s + u + PF, s1 - 1));
                else
                    step<false, true>(acc, w, t, u % PF, r, s + u, 0);
                if (u + 1 < WPF)
#pragma unroll
                    for (int i = 0; i < RT; ++i) w[i] = n[i];
            }
    }

    static __device__ __forceinline__ void clear(f32x4 (&acc)[RT][CT])
    {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
};

// Scales and biases of `rows` rows from memory to LDS, by all threads, in 16-byte
// pieces: the first ones wait in registers while other loads are asked for.
template <int HELD>
struct MetaCopy {
    u32x4 v[HELD];
    const uint16_t *s, *b;
    int count, whole;      // values, and whole pieces, of each
    float per_row;         // where LDS rows are padded: 1 / pieces per row, else 0
    int thread, threads;   // of the workgroup (blockDim is an argument of its own, and a round trip), or of a wave
    __device__ __forceinline__ MetaCopy(const uint16_t* s_, const uint16_t* b_, int rows, int G, int threads_, int thread_ = threadIdx.x)
        : s(s_), b(b_), count(rows * G), whole(rows * G / 8), per_row(G % 8 == 0 ? 8.0f / (float)G : 0.0f), thread(thread_), threads(threads_)
    {
    }
    __device__ __forceinline__ u32x4 load(int i) const
    {
        return i < whole ? reinterpret_cast<const u32x4*>(s)[i] : reinterpret_cast<const u32x4*>(b)[min(i - whole, whole - 1)];
    }
    __device__ __forceinline__ void ask()
    {
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            const int i = min(thread + k * threads, 2 * whole - 1);
            if (whole > 0) v[k] = load(i);
        }
    }
    __device__ __forceinline__ void put(uint16_t* ts, uint16_t* tb) const
    {
        auto store = [&](int i, const u32x4& x) {
            const int at = i < whole ? i : i - whole;
            if (i < 2 * whole) reinterpret_cast<u32x4*>(i < whole ? ts : tb)[at + small_div(at, per_row)] = x;      // (0.5 * 0 is no row)
        };
#pragma unroll
        for (int k = 0; k < HELD; ++k) store(thread + k * threads, v[k]);
        for (int i = thread + HELD * threads; i < 2 * whole; i += threads) store(i, load(i));
        int at = whole * 8 + thread;
        asm volatile("" : "+v"(at));        // these loads stay here, behind those in flight
        if (at < count) {
            ts[at] = s[at];
            tb[at] = b[at];
        }
    }
};

// A window of every part's groups, of `rows` rows: row-major, part by part.
__device__ __forceinline__ void stage_window(uint16_t* to, const uint16_t* from, int rows, int G, int ng, int slabs, int parts,
                                             int window, int number, int threads)
{
    const int log_parts = __builtin_ctz(parts);
    const int wg = window * ng, row = parts * wg;
    for (int i = threadIdx.x; i < rows * row; i += threads) {
        const int part = i % row / wg, g = (part_start(slabs, log_parts, part) + number * window) * ng + i % wg;
        if (g < G) to[i] = from[(size_t)(i / row) * G + g];
    }
}

// A barrier for LDS alone: loads from memory stay in flight over it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The waves' partial results of one 16-token column of tiles, joined in the
// order of the waves.  Write: wave, row tile and result register; read:
// element (row n of 16*RT, token t of 16).  16 words between row tiles keep
// the reads of consecutive rows on different banks.
template <int RT>
struct Join {
    static constexpr int kTile = 256 + 16;
    static constexpr int kWords = RT * kTile;     // per wave
    static __device__ __forceinline__ void write(float* lds, int wave, int lane, int i, const f32x4& v)
    {
        float* p = lds + wave * kWords + i * kTile + lane;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e * 64] = v[e];
    }
    static __device__ __forceinline__ int at(int n, int t)
    {
        return (n >> 4) * kTile + (t & 3) * 64 + (t >> 2) * 16 + (n & 15);
    }
    // of waves first.. in their order
    static __device__ __forceinline__ float sum(const float* lds, int first, int waves, int at)
    {
        float v = lds[first * kWords + at];
        for (int w = 1; w < waves; ++w) v += lds[(first + w) * kWords + at];
        return v;
    }
};

}  // namespace ops
