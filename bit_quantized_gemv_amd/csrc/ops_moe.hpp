// ops_moe.hpp -- parameters and launches of the expert products (qmv_experts).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ops_tile.hpp"

namespace ops {

constexpr int kMoeTile = 256;      // tokens per set of launches

struct ExpertParams {
    const char* xp;                // packed activations of the tokens
    const int32_t* ids;            // [P], P = T * k (token, slot) pairs
    const uint32_t* w13;
    const uint16_t* s13;
    const uint16_t* b13;
    const uint32_t* w2;
    const uint16_t* s2;
    const uint16_t* b2;
    char* h;                       // packed hidden values of the pairs, in planes
    float* z;                      // [rows][D]
    size_t x_plane, h_plane;       // bytes of a plane
    int P, k, D, F, E;
    int slots;                     // P: a workgroup per pair, its expert's first; E: one per expert
    const int* base;               // sorted pairs: an expert's first tile of 16, its pairs, and each
    const int* count;              // pair's place (a row of xp, h and z); null where pairs keep their order
    int takers;                    // workgroups that share an expert's pairs
    int log_parts;                 // of a row's K
    int groups;                    // of waves in a workgroup
    Meta meta;
    float per_k;                   // 1 / k
    const float* weights;          // [P]
    void* y;                       // [P / k][D]
    bool yf32;
};

// which = 0: gate and up products and the activation (xp -> h); 1: down product (h -> z);
// 2: down products and weighted sums of whole tokens (h -> y)
int expert_launch_b4_g64(int which, const ExpertParams& p, bool xf32, bool sbf, hipStream_t st);
int expert_launch_b4_g128(int which, const ExpertParams& p, bool xf32, bool sbf, hipStream_t st);
int expert_launch_b2_g64(int which, const ExpertParams& p, bool xf32, bool sbf, hipStream_t st);
int expert_launch_b2_g128(int which, const ExpertParams& p, bool xf32, bool sbf, hipStream_t st);

}  // namespace ops
