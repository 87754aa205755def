// ops_attend.hpp -- what the kernels of qmv_attend share.
//
// Layouts.  Scores are computed turned over, S^T = K Q^T, so that a lane of the 16 x 16
// result holds four keys of one query row n = lane % 16 (key 4 (lane / 16) + i of a tile of
// 16), and the outputs too, O^T = V^T P^T: four values of a head of the same row.  Maxima,
// sums and factors of a row are then a lane's own numbers.  A step of the second product
// takes 32 keys, two tiles of scores; in which order is free as long as both operands have the
// same, and the order "four of the first tile, four of the second" for every group of 16
// lanes is the one in which a lane holds its weights already.  The values of V^T that belong
// to it are four neighbouring keys of one column: what the transposing read of LDS gives.
//
// Keys and values in LDS: blocks of 16 keys and 32 columns, 64 bytes a key, the four 16-byte
// pieces of key j at piece ^ swizzle(j / 4).  The reads of 16 keys' pieces and the transposing
// reads of 16 x 16 values then meet every bank as often as their bytes need.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ops_args.hpp"
#include "ops_cache.hpp"

namespace ops {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;

constexpr int kUnits = 256;           // compute units
// workgroups of so much LDS on a compute unit, which hands out its 160 KB in pieces of 1280 bytes (768 workgroups of one
// length: 307 us with 53760 bytes each, 604 with 53776)
constexpr int fit(int lds) { return 128 / ((lds + 1279) / 1280); }
constexpr int kBlockTokens = 16;      // up to so many new tokens a sequence is a block, above a chunk
constexpr int kLeafBytes = 32768;     // of keys in a leaf, and of values
constexpr int leaf_keys(int head_size) { return kLeafBytes / 2 / head_size; }
constexpr int kSuper = 8;             // leaves of a super (the two steps in which blocks of keys are joined)
constexpr float kGone = -__builtin_huge_valf();

struct AttendParams {
    const char* q;
    char* out;
    float* part;                    // [token][head][unit][D]: a block's sums of weights * values
    f32x2* stat;                    // [token][head][unit]: their largest scores and sums of weights
    float* chunk_part;              // the same of chunks, a share of the keys for every unit
    f32x2* chunk_stat;
    long long q_token, q_head;      // bytes
    int q_heads, heads, group, D;
    int window, sinks, max_new, out_f32;
    int units, row_blocks, per_unit, splits;
    int shares;                     // blocks: workgroups of a sequence's units; each takes every so many-th
    int rows_last;                  // blocks: workgroups of the first tiles of rows, on a die, after which those of the next come (0: side by side)
    int apart;                      // a block's tokens in part and stat: by sequence, so many each (0: as in q)
    float scale;                    // times log2(e)
    Divisor by_group, by_heads, by_seqs, by_rows;      // the last: rows_last, or row_blocks
    // calls with chunks: workgroups of a share of the keys, and of blocks, and the rounds of kUnits workgroups of
    // chunks, and those in which both take turns
    int chunk_groups, block_groups, chunk_rounds, both_rounds;
    Divisor by_chunk_groups;
    Cache cache;
};

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c, __bf16)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c, _Float16)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pack(float a, float b, __bf16) { return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b}); }
__device__ __forceinline__ uint32_t pack(float a, float b, _Float16) { return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b}); }
__device__ __forceinline__ f32x2 unpack(uint32_t v, __bf16) { return __builtin_convertvector(__builtin_bit_cast(bf16x2, v), f32x2); }
__device__ __forceinline__ f32x2 unpack(uint32_t v, _Float16) { return __builtin_convertvector(__builtin_bit_cast(f16x2, v), f32x2); }

// Weights of fp16 caches are multiplied by a power of two that takes a row's largest towards 2^15 before they are rounded.  As
// they are, those below 2^-14 would be less than fp16's normal numbers and lose their bits one by one; but a first key that takes
// nearly all the weight and holds next to nothing is common, and leaves the output to the others.  4096 keys at 2^-20 of the first,
// whose value is 0: outputs were off by 6e-4 of theirs, at 2^-24 by 3%.  bf16 has the range as it is.
constexpr float lift_log2(__bf16) { return 0.0f; }
constexpr float lift_log2(_Float16) { return 15.0f; }

// Values that are no numbers.  As a factor of a matrix product, the infinity or NaN of one key
// would reach the rows that do not see the key too, by zero times infinity.  So where rows of a tile
// see different keys, the values are looked at in LDS first.  If there are any, they are
// taken out of the product, and products of marks count for every output the NaN, infinities
// and negative infinities that its row sees.
constexpr uint32_t no_number(__bf16) { return 0x7f80; }       // the exponent
constexpr uint32_t no_number(_Float16) { return 0x7c00; }
constexpr uint32_t one(__bf16) { return 0x3f80; }
constexpr uint32_t one(_Float16) { return 0x3c00; }

// the two values of a word, those that are no numbers as zeros
template <class X>
__device__ __forceinline__ uint32_t numbers(uint32_t w)
{
    constexpr uint32_t E = no_number(X());
    const uint32_t lo = (w & E) == E ? 0 : w & 0xffff, hi = (w >> 16 & E) == E ? 0 : w & 0xffff0000;
    return lo | hi;
}
template <class X>
__device__ __forceinline__ u32x4 numbers4(u32x4 w)
{
    return u32x4{numbers<X>(w.x), numbers<X>(w.y), numbers<X>(w.z), numbers<X>(w.w)};
}
// whether a value of the words is no number
template <class X>
__device__ __forceinline__ bool odd(u32x4 v)
{
    constexpr uint32_t E = no_number(X());
    bool r = false;
#pragma unroll
    for (int c = 0; c < 4; ++c) r |= (v[c] & E) == E || (v[c] >> 16 & E) == E;
    return r;
}

// Ones where a value is of a kind: the bits of `mask` from `low` on, `more` values.
struct Kind {
    uint32_t mask, low, more;
    float what;
};
template <class X>
__device__ __forceinline__ Kind kind_of(int i)
{
    constexpr uint32_t E = no_number(X());
    return Kind{i == 0 ? 0x7fffu : 0xffffu, i == 0 ? E + 1 : i == 1 ? E : 0x8000u | E, i == 0 ? 0x7ffe - E : 0u,
                i == 0 ? __builtin_nanf("") : i == 1 ? -kGone : kGone};
}
template <class X>
__device__ __forceinline__ uint32_t marks(uint32_t w, Kind k)
{
    const uint32_t lo = (w & k.mask) - k.low <= k.more ? one(X()) : 0, hi = ((w >> 16) & k.mask) - k.low <= k.more ? one(X()) : 0;
    return lo | hi << 16;
}
template <class X>
__device__ __forceinline__ u32x4 marks4(u32x4 w, Kind k)
{
    return u32x4{marks<X>(w.x, k), marks<X>(w.y, k), marks<X>(w.z, k), marks<X>(w.w, k)};
}
// the output that has met `count` of them
__device__ __forceinline__ f32x4 met(f32x4 o, f32x4 count, Kind k)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = count[i] > 0.0f ? o[i] + k.what : o[i];
    return o;
}

// A barrier for LDS alone: loads from memory stay in flight over it.
__device__ __forceinline__ void lds_only_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The larger of two scores.  fmax would first turn a signalling NaN, which a matrix product might
// leave, into a quiet one, at an instruction for each; the median of three does not.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, -kGone); }

// Over the four lanes that hold a row's numbers: 16 and 32 lanes apart.
__device__ __forceinline__ float row_max(float x)
{
    const auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    x = __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return __builtin_fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
__device__ __forceinline__ float row_sum(float x)
{
    const auto a = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    x = __builtin_bit_cast(float, (uint32_t)a[0]) + __builtin_bit_cast(float, (uint32_t)a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
    return __builtin_bit_cast(float, (uint32_t)b[0]) + __builtin_bit_cast(float, (uint32_t)b[1]);
}

// Whether a row sees a key: places up to `high`, above `low` or below `sinks`; without branches.
__device__ __forceinline__ bool sees(int j, int high, int low, int sinks, uint32_t held)
{
    return (int)(j <= high) & ((int)(j > low) | (int)(j < sinks)) & (int)held & 1;
}

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// 0, 2, 3, 1 for the keys 0-3, 4-7, 8-11, 12-15 of a block
__device__ __forceinline__ int swizzle(int quarter) { return (quarter & 1) << 1 ^ (quarter >> 1) * 3; }

// 16 bytes a lane from memory to LDS, the wave's 1024 one after the other from `to` on, without
// registers between.  Written out, since the compiler would wait for it before any read of
// LDS; whoever reads the bytes waits with landed(), then passes a barrier.
__device__ __forceinline__ void send_to_lds(const char* from, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "s"(to) : "memory", "m0");
}
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_address(const char* at)
{
    typedef __attribute__((address_space(3))) const char* At;
    return (uint32_t)(uintptr_t)(At)at;
}

__device__ __forceinline__ u32x2 read_turned(const char* lds)
{
    typedef __attribute__((address_space(3))) s16x4* At;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((At)(uintptr_t)(lds)));
}

// What some new tokens of a sequence see, between them: the places below `first` and those
// from low to high, in units of U places, listed one after the other.
struct Visible {
    int first, low, high;         // high < 0: nothing
    int front, start, units;      // units of the first places; the unit of `low` after them; all units
    __device__ __forceinline__ int unit(int i) const { return i < front ? i : start + i - front; }
    __device__ __forceinline__ bool meets(int from, int to) const { return from < first || (from <= high && to > low); }
};

// of new tokens at places from `place` on
__device__ __forceinline__ Visible visible(int place, int tokens, int window, int sinks, int U)
{
    Visible v;
    v.high = place + tokens - 1;
    v.low = window > 0 ? max(0, place - window + 1) : 0;
    v.first = window > 0 ? min(sinks, v.low) : 0;
    if (v.high < 0) {
        v.front = v.start = v.units = 0;
        return v;
    }
    v.front = (v.first + U - 1) / U;
    v.start = max(v.low / U, v.front);
    v.units = v.front + max(0, v.high / U - v.start + 1);
    return v;
}

// One join of a row: the sums so far (m, l, o) and those of the next keys.  Weights go with
// 2^(score - m); a side that has seen nothing (m = -inf) adds exact zeros.
struct Factors {
    float a, b;
};
__device__ __forceinline__ Factors join(float& m, float& l, float m2, float l2)
{
    const float top = __builtin_fmaxf(m, m2), at = top == kGone ? 0.0f : top;
    const Factors f{exp2_of(m - at), exp2_of(m2 - at)};
    m = top;
    l = __builtin_fmaf(l2, f.b, l * f.a);
    return f;
}
__device__ __forceinline__ f32x4 joined(f32x4 o, f32x4 o2, Factors f)
{
    return f32x4{__builtin_fmaf(o2.x, f.b, o.x * f.a), __builtin_fmaf(o2.y, f.b, o.y * f.a), __builtin_fmaf(o2.z, f.b, o.z * f.a),
                 __builtin_fmaf(o2.w, f.b, o.w * f.a)};
}

// Work of the sequences over the compute dies, to which workgroups go in turn: the first turn of all sequences,
// then the second, and each sequence's turns over all eight dies, since its next one is an odd number of workgroups
// on (n_seqs, or one beside it).
struct Turn {
    int turn, b;
};
__device__ __forceinline__ Turn turn_of(int i, const AttendParams& p)
{
    const int n = p.cache.n_seqs, turn = divide(i, p.by_seqs), b = i - turn * n + (n & 1 ? 0 : turn - divide(turn, p.by_seqs) * n);
    return Turn{turn, b < n ? b : b - n};
}

// The first row of a block's tokens in part and stat.
__device__ __forceinline__ long long block_row(const AttendParams& p, int b, int start)
{
    return (long long)(p.apart > 0 ? b * p.apart : start) * p.q_heads;
}

// four values of a row's result; l = 0: the row has seen nothing
__device__ __forceinline__ void put_result(const AttendParams& p, long long row, int d, f32x4 o, float l)
{
    const f32x4 y = l == 0.0f ? f32x4{0, 0, 0, 0} : o / l;
    if (p.out_f32) *reinterpret_cast<f32x4*>(p.out + (row * p.D + d) * 4) = y;
    else *reinterpret_cast<bf16x4*>(p.out + (row * p.D + d) * 2) = __builtin_convertvector(y, bf16x4);
}

// The kernel of a head size (64, 128, 256), cache type, output type, several units a workgroup and
// tiles of query rows, and its LDS.
const void* block_kernel_64(bool f16, bool f32_out, bool share, int row_tiles, int* lds);
const void* block_kernel_128(bool f16, bool f32_out, bool share, int row_tiles, int* lds);
const void* block_kernel_256(bool f16, bool f32_out, bool share, int row_tiles, int* lds);
struct ChunkShape {
    int rows, threads;       // of a workgroup
    int at_once, lds;        // workgroups on a compute unit
};
const void* chunk_kernel_64(bool f16, bool f32_out, int row_tiles, ChunkShape* shape);
const void* chunk_kernel_96(bool f16, bool f32_out, int row_tiles, ChunkShape* shape);
const void* chunk_kernel_128(bool f16, bool f32_out, int row_tiles, ChunkShape* shape);
const void* chunk_kernel_192(bool f16, bool f32_out, int row_tiles, ChunkShape* shape);
const void* chunk_kernel_256(bool f16, bool f32_out, int row_tiles, ChunkShape* shape);

}  // namespace ops
