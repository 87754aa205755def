// ops_check.hpp -- host checks shared by the operators' entry points.
#pragma once
#include <cstddef>
#include <cstdint>

#include "qmv_ops.h"

namespace ops {

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return na != 0 && nb != 0 && a0 < b0 + nb && b0 < a0 + na;
}

struct Span {
    const void* p;
    size_t n;
};

// every output (and the workspace) apart from the inputs and from each other
template <int NI, int NO>
bool disjoint(const Span (&in)[NI], const Span (&out)[NO])
{
    for (int o = 0; o < NO; ++o) {
        for (int i = 0; i < NI; ++i)
            if (in[i].p && overlap(out[o].p, out[o].n, in[i].p, in[i].n)) return false;
        for (int i = 0; i < o; ++i)
            if (overlap(out[o].p, out[o].n, out[i].p, out[i].n)) return false;
    }
    return true;
}

inline size_t size_of(int dt) { return dt == QMV_DT_F32 ? 4 : 2; }
inline bool wide(int dt) { return dt == QMV_DT_F32 || dt == QMV_DT_BF16; }       // activations and outputs
inline bool half(int dt) { return dt == QMV_DT_F16 || dt == QMV_DT_BF16; }       // scales, biases, adapters

// a quantized matrix of N rows and K columns
inline int check_matrix(long long N, int K, int bits, int gs)
{
    if (bits != 2 && bits != 4) return QMV_E_BITS;
    if (gs != 64 && gs != 128) return QMV_E_GROUP;
    if (N < 1 || N > QMV_MAX_N || K < gs || K > QMV_MAX_K || K % gs != 0) return QMV_E_SHAPE;
    return QMV_OK;
}

// workspaces are cut into 256-byte aligned pieces
inline long long piece(long long bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace ops
