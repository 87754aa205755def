// ops_lora.hpp -- parameters and launches of the adapted projection
// (qmv_affine_lora).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ops_tile.hpp"

namespace ops {

// Columns of K that one workgroup of the first kernel sums: 8 waves of 8 steps
// of 32.  The second kernel adds the pieces in order.
constexpr int kShrinkK = 2048;
constexpr int kLoraTile = 256;    // tokens per pair of launches
constexpr int kBlock = 64;        // tokens whose adapters are listed together

inline int shrink_pieces(int K) { return (K + kShrinkK - 1) / kShrinkK; }
inline int pad_rank(int R) { return (R + 31) / 32 * 32; }

// The adapters of a block of tokens, each once, in the order of their first token.
struct AdapterList {
    unsigned long long tokens[kBlock];   // bit t: the block's token t has it
    unsigned long long any;              // those that have one
    int adapter[kBlock];
    float scaling[kBlock];
    int count, pad;
};

struct LoraParams {
    const uint32_t* w;
    const uint16_t* s;
    const uint16_t* b;
    const char* x;
    void* y;
    const uint16_t* la;
    const uint16_t* lb;
    const int32_t* ids;
    const float* scaling;
    float* h;             // [pieces][M][pad_rank(R)]
    AdapterList* lists;   // [blocks of tokens]
    char* xp;             // packed activations
    size_t plane;         // bytes of one of their planes
    int M, N, K, L, R, Rp, pieces, log_parts;
    Meta meta;
    bool yf32, adf16;
};

// the projection with the adapters' second product; rt, ct: row and token tiles per wave
int lora_launch_b4_g64(const LoraParams& p, int rt, int ct, bool xf32, bool sbf, hipStream_t st);
int lora_launch_b4_g128(const LoraParams& p, int rt, int ct, bool xf32, bool sbf, hipStream_t st);
int lora_launch_b2_g64(const LoraParams& p, int rt, int ct, bool xf32, bool sbf, hipStream_t st);
int lora_launch_b2_g128(const LoraParams& p, int rt, int ct, bool xf32, bool sbf, hipStream_t st);

}  // namespace ops
