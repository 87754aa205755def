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
// (l & 15), tokens 4 * (l >> 4) + i.  So the lane that loads a row's codes also
// needs that row's scale and bias, and no exchange is needed for the fold.
// Each lane loads 16 bytes of its row (a slab of 4 x 16 bytes per row and wave
// step); where those hold more than one group, permlane swaps turn the four
// lanes' words so that every matrix instruction's k lies in one group.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace ops {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;

constexpr int kWave = 64;
constexpr int kMaxWaves = 8;

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

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Slabs of K a row of `chunks` 16-byte pieces is walked in, four pieces each.
__host__ __device__ inline int slabs_of(int chunks) { return (chunks + 3) / 4; }

// Wavefronts that share a row's K: two slabs each at least, so that a wave has
// a load in flight behind the one it computes on; depends on the row length
// alone, as the order of the join does.
inline int waves_of(int chunks)
{
    const int n = slabs_of(chunks);
    return n >= 16 ? 8 : n >= 6 ? 4 : n >= 2 ? 2 : 1;
}

template <int BITS_, int GS_, int RT_, int CT_, bool XF32_, bool SBF_>
struct Tile {
    static constexpr int BITS = BITS_, GS = GS_, RT = RT_, CT = CT_;
    static constexpr bool XF32 = XF32_, SBF = SBF_;
    static constexpr int VPW = 32 / BITS;             // codes per word
    static constexpr int SLAB = 16 * VPW;             // codes of a row per slab
    static constexpr int NG = SLAB / GS;              // groups per slab
    static constexpr int WPG = 4 / NG;                // words of a lane per group
    static constexpr int FPW = VPW / 8;               // matrix instructions per word
    static constexpr int NF = WPG * FPW;              // and per group
    static constexpr int NP = XF32 ? 3 : 1;           // bf16 pieces of an activation
    static constexpr int XV = VPW / (XF32 ? 4 : 8);   // 16-byte loads per word's activations
    static constexpr uint32_t MASK = BITS == 4 ? 0x00780078u : 0x00600060u;
    static constexpr uint32_t BASE = BITS == 4 ? 0x41804180u : 0x40804080u;  // 16, 4
    static constexpr uint32_t NEG = BITS == 4 ? 0xC180C180u : 0xC080C080u;   // -16, -4
    static constexpr float INV = BITS == 4 ? -1.0f / 16 : -1.0f / 4;
    // Slabs of codes in flight per wave, about 4 KB; the activations fly with
    // them where one token tile's fit the registers beside, and are loaded for
    // the slab at hand otherwise.
    static constexpr bool XAHEAD = !XF32 && CT == 1;
    static constexpr int PF = RT == 1 ? 4 : (RT == 2 || (CT == 1 && !XF32)) ? 2 : 1;

    struct Rows {                  // a lane's operands
        const u32x4* w[RT];        // codes of its weight row
        const uint16_t* s[RT];     // scales and biases of its weight row
        const uint16_t* b[RT];
        const char* x[CT];         // its token's activations
        int chunks, G, K;
        bool meta_al;              // rows of scales start at a multiple of NG of them
    };

    struct Slab {
        u32x4 w[RT];
        uint32_t s[RT][(NG + 1) / 2], b[RT][(NG + 1) / 2];
    };
    struct Acts {
        u32x4 x[CT][NG][WPG][XV];
    };

    static __device__ __forceinline__ void load_meta(uint32_t (&v)[(NG + 1) / 2], const uint16_t* p, int g0,
                                                     int G, bool al)
    {
        if constexpr (NG == 1) {
            v[0] = p[g0];
        } else if (al) {
            if constexpr (NG == 2) {
                v[0] = *reinterpret_cast<const uint32_t*>(p + g0);
            } else {
                const u32x2 t = *reinterpret_cast<const u32x2*>(p + g0);
                v[0] = t[0];
                v[1] = t[1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < NG; i += 2) {
                const uint32_t lo = p[min(g0 + i, G - 1)], hi = p[min(g0 + i + 1, G - 1)];
                v[i / 2] = lo | (hi << 16);
            }
        }
    }

    // where a lane's activations for word c of group g of a slab start
    static __device__ __forceinline__ int x_at(int g, int c, int q)
    {
        if constexpr (NG == 1) return (GS / 4) * q + VPW * c;
        if constexpr (NG == 2) return GS * g + (GS / 2) * (q & 1) + VPW * (2 * (q >> 1) + c);
        return GS * g + VPW * q;
    }

    static __device__ __forceinline__ void load(Slab& t, const Rows& r, int slab, int q)
    {
        const int chunk = min(4 * slab + q, r.chunks - 1);   // a part slab's lanes past the row read its last piece
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            t.w[i] = __builtin_nontemporal_load(r.w[i] + chunk);
            load_meta(t.s[i], r.s[i], slab * NG, r.G, r.meta_al);
            load_meta(t.b[i], r.b[i], slab * NG, r.G, r.meta_al);
        }
    }

    static __device__ __forceinline__ void load_x(Acts& t, const Rows& r, int slab, int q)
    {
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int c = 0; c < WPG; ++c) {
                    const int k = min(slab * SLAB + x_at(g, c, q), r.K - VPW);
                    const u32x4* p = reinterpret_cast<const u32x4*>(r.x[j] + (size_t)k * (XF32 ? 4 : 2));
#pragma unroll
                    for (int v = 0; v < XV; ++v) t.x[j][g][c][v] = p[v];
                }
    }

    static __device__ __forceinline__ float param(const uint32_t (&v)[(NG + 1) / 2], int g)
    {
        const uint32_t u = v[g / 2];
        if constexpr (SBF) return bits_f32((g & 1) ? (u & 0xffff0000u) : (u << 16));
        return half_bits((g & 1) ? (u >> 16) : (u & 0xffffu));
    }

    // The operand of matrix instruction f of a word's activations, whose dword d
    // pairs fields p = 4 f + d and p + VPW / 2, as the codes' does.
    static __device__ __forceinline__ void x_operand(const u32x4 (&x)[XV], int f, u32x4 (&o)[NP])
    {
        constexpr int H = VPW / 2;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int p = 4 * f + d;
            if constexpr (!XF32) {
                const uint32_t a = x[(p / 2) / 4][(p / 2) % 4], b = x[((p + H) / 2) / 4][((p + H) / 2) % 4];
                o[0][d] = (p & 1) ? hi16(a, b) : lo16(a, b);
            } else {
                uint32_t ah, am, al, bh, bm, bl;
                split3(bits_f32(x[p / 4][p % 4]), ah, am, al);
                split3(bits_f32(x[(p + H) / 4][(p + H) % 4]), bh, bm, bl);
                o[0][d] = hi16(ah, bh);
                o[1][d] = hi16(am, bm);
                o[2][d] = hi16(al, bl);
            }
        }
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

    static __device__ __forceinline__ void compute(f32x4 (&acc)[RT][CT], Slab& t, const Acts& a, const Rows& r, int slab)
    {
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            if constexpr (NG >= 2) {
                const auto u = __builtin_amdgcn_permlane32_swap(t.w[i][0], t.w[i][2], false, false);
                const auto v = __builtin_amdgcn_permlane32_swap(t.w[i][1], t.w[i][3], false, false);
                t.w[i] = u32x4{u[0], v[0], u[1], v[1]};
            }
            if constexpr (NG == 4) {
                const auto u = __builtin_amdgcn_permlane16_swap(t.w[i][0], t.w[i][1], false, false);
                const auto v = __builtin_amdgcn_permlane16_swap(t.w[i][2], t.w[i][3], false, false);
                t.w[i] = u32x4{u[0], u[1], v[0], v[1]};
            }
        }
        const u32x4 neg = {NEG, NEG, NEG, NEG};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g > 0 && slab * NG + g >= r.G) break;
            u32x4 xo[CT][NF][NP];
            f32x4 c0[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                c0[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < WPG; ++c)
#pragma unroll
                    for (int f = 0; f < FPW; ++f) {
                        x_operand(a.x[j][g][c], f, xo[j][c * FPW + f]);
#pragma unroll
                        for (int p = 0; p < NP; ++p) c0[j] = mfma(xo[j][c * FPW + f][p], neg, c0[j]);
                    }
            }
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const float s = param(t.s[i], g), nb = param(t.b[i], g) * INV;
                u32x4 wo[NF];
#pragma unroll
                for (int c = 0; c < WPG; ++c)
#pragma unroll
                    for (int f = 0; f < FPW; ++f) wo[c * FPW + f] = w_operand(t.w[i][g * WPG + c], f);
#pragma unroll
                for (int j = 0; j < CT; ++j) {
                    f32x4 d = c0[j];
#pragma unroll
                    for (int f = 0; f < NF; ++f)
#pragma unroll
                        for (int p = 0; p < NP; ++p) d = mfma(xo[j][f][p], wo[f], d);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][j][e] = __builtin_fmaf(nb, c0[j][e], __builtin_fmaf(s, d[e], acc[i][j][e]));
                }
            }
        }
    }

    // acc += the products over slabs [s0, s1), PF of them in flight
    static __device__ __forceinline__ void run(f32x4 (&acc)[RT][CT], const Rows& r, int s0, int s1, int q)
    {
        Slab t[PF];
        Acts x[XAHEAD ? PF : 1];
#pragma unroll
        for (int u = 0; u < PF; ++u)
            if (s0 + u < s1) {
                if constexpr (XAHEAD) load_x(x[u], r, s0 + u, q);
                load(t[u], r, s0 + u, q);
            }
        for (int s = s0; s < s1; s += PF) {
#pragma unroll
            for (int u = 0; u < PF; ++u) {
                if (s + u < s1) {
                    Acts& a = x[XAHEAD ? u : 0];
                    if constexpr (!XAHEAD) load_x(a, r, s + u, q);
                    Slab now = t[u];
                    const Acts an = a;
                    if (s + u + PF < s1) {
                        if constexpr (XAHEAD) load_x(a, r, s + u + PF, q);
                        load(t[u], r, s + u + PF, q);
                    }
                    compute(acc, now, an, r, s + u);
                }
            }
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
    static __device__ __forceinline__ float sum(const float* lds, int waves, int at)
    {
        float v = lds[at];
        for (int w = 1; w < waves; ++w) v += lds[w * kWords + at];
        return v;
    }
};

}  // namespace ops
