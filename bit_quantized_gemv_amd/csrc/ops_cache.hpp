// ops_cache.hpp -- a cache in pages: its sequences and places on the device, and
// the host checks that append and attend share.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ops_check.hpp"
#include "qmv_attn.h"

namespace ops {

// x / n for x < 2^31, by one product
struct Divisor {
    uint32_t magic;
    int shift;
};

__host__ __device__ __forceinline__ int divide(int x, Divisor d) { return (int)(((uint64_t)(uint32_t)x * d.magic) >> d.shift); }

struct Cache {
    const char *k, *v;
    long long k_page, k_slot, k_head, v_page, v_slot, v_head;    // bytes
    const int32_t *pages, *starts, *lengths;
    long long pages_row;
    Divisor by_page;            // the page size
    int n_pages, page_size, n_seqs, max_pages, max_places;
    int T;
};

struct Seq {
    int start, count, length;   // its new tokens, and its places with them
};

// Both starts are taken into 0 .. T before one is taken from the other: the difference of any two would not fit 32 bits.
__host__ __device__ __forceinline__ Seq sequence(const Cache& c, int b)
{
    const int s0 = c.starts[b], s1 = c.starts[b + 1], n = c.lengths[b];
    Seq s;
    s.start = max(0, min(s0, c.T));
    s.count = max(0, max(0, min(s1, c.T)) - s.start);
    s.length = max(0, min(n, c.max_places));
    return s;
}

__device__ __forceinline__ int page_index(const Cache& c, int j) { return divide(j, c.by_page); }

// the page of place j < max_places of sequence b; -1 if it holds nothing
__device__ __forceinline__ int page_of(const Cache& c, int b, int index)
{
    const int p = c.pages[b * c.pages_row + index];
    return (uint32_t)p < (uint32_t)c.n_pages ? p : -1;
}

// The sequence of token t, told by a whole wave: how many starts are at or below it, by steps of
// 4096, 64 and 1 of ascending starts.  -1 if it is in none.
__device__ __forceinline__ int sequence_of(const Cache& c, int t, int lane)
{
    int b = 0;
    for (int step = c.n_seqs > 4096 ? 4096 : c.n_seqs > 64 ? 64 : 1; step > 0; step >>= 6) {
        const int i = b + (lane + 1) * step;
        b += step * __popcll(__ballot(i <= c.n_seqs && c.starts[i] <= t));
    }
    return b < c.n_seqs ? b : -1;
}

// ---- host -----------------------------------------------------------------

constexpr long long kMostStride = 1LL << 40;

inline bool stride_ok(long long s) { return s >= 0 && s <= kMostStride; }

// the elements from the first to the last of an array of these sizes and strides; -1 if above 2^50
template <int N>
long long extent(const long long (&size)[N], const long long (&stride)[N], long long inner)
{
    __int128 e = inner;
    for (int i = 0; i < N; ++i) e += (__int128)(size[i] - 1) * stride[i];
    return e > ((__int128)1 << 50) ? -1 : (long long)e;
}

// whether no two values of such an array share a place, as far as nested strides tell
inline bool apart(long long (&size)[3], long long (&stride)[3], long long inner)
{
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (stride[j] < stride[i] || (stride[j] == stride[i] && size[j] < size[i])) {
                const long long a = size[i], b = stride[i];
                size[i] = size[j];
                stride[i] = stride[j];
                size[j] = a;
                stride[j] = b;
            }
    __int128 reach = inner;
    for (int i = 0; i < 3; ++i) {
        if (size[i] == 1) continue;
        if (stride[i] < reach) return false;
        reach += (__int128)(size[i] - 1) * stride[i];
    }
    return true;
}

inline int check_heads(int heads, int D)
{
    return heads < 1 || heads > QMV_MAX_HEADS || D < 8 || D > QMV_MAX_HEAD_SIZE || D % 8 != 0 ? QMV_E_HEADS : QMV_OK;
}

// sizes alone: what a workspace is asked for with
inline int check_cache_sizes(const qmv_cache* c, int T, int q_heads)
{
    if (check_heads(c->heads, c->head_size) != QMV_OK || check_heads(q_heads, c->head_size) != QMV_OK || q_heads % c->heads != 0)
        return QMV_E_HEADS;
    if (c->n_pages < 1 || c->page_size < 1 || c->page_size > QMV_MAX_PAGE_SIZE || c->n_seqs < 1 || c->n_seqs > QMV_MAX_SEQS ||
        c->max_pages < 1 || (long long)c->max_pages * c->page_size > QMV_MAX_LENGTH || T < 1 || T > QMV_MAX_TOKENS)
        return QMV_E_CACHE;
    return QMV_OK;
}

struct CacheSpans {
    size_t k, v, pages;      // bytes
};

inline int check_cache(const qmv_cache* c, int T, int q_heads, CacheSpans* spans)
{
    if (!c->k || !c->v || !c->pages || !c->starts || !c->lengths) return QMV_E_NULL;
    if (int e = check_cache_sizes(c, T, q_heads)) return e;
    if (!half(c->dt)) return QMV_E_DTYPE;
    const long long s[] = {c->k_page, c->k_slot, c->k_head, c->v_page, c->v_slot, c->v_head, c->pages_row};
    for (long long x : s)
        if (!stride_ok(x)) return QMV_E_STRIDE;
    const long long size[] = {c->n_pages, c->page_size, c->heads};
    const long long ks[] = {c->k_page, c->k_slot, c->k_head}, vs[] = {c->v_page, c->v_slot, c->v_head};
    const long long ps[] = {c->n_seqs}, pr[] = {c->pages_row};
    const long long nk = extent(size, ks, c->head_size), nv = extent(size, vs, c->head_size), np = extent(ps, pr, c->max_pages);
    if (nk < 0 || nv < 0 || np < 0) return QMV_E_STRIDE;
    for (int i = 0; i < 6; ++i)
        if (s[i] % 8 != 0) return QMV_E_ALIGN;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->pages, 4) || !aligned(c->starts, 4) || !aligned(c->lengths, 4))
        return QMV_E_ALIGN;
    *spans = CacheSpans{(size_t)nk * 2, (size_t)nv * 2, (size_t)np * 4};
    return QMV_OK;
}

// n <= 2^l; m = floor(2^(31+l) / n) + 1 is above 2^(31+l) / n by at most 1, so x m / 2^(31+l) is
// above x / n by less than 2^31 / 2^(31+l) <= 1 / n, which its floor does not see
inline Divisor divisor(int n)
{
    int l = 0;
    while ((1LL << l) < n) ++l;
    return Divisor{(uint32_t)((1ULL << (31 + l)) / (unsigned)n + 1), 31 + l};
}

inline Cache device_cache(const qmv_cache* c, int T)
{
    Cache d;
    d.k = static_cast<const char*>(c->k);
    d.v = static_cast<const char*>(c->v);
    d.k_page = 2 * c->k_page;
    d.k_slot = 2 * c->k_slot;
    d.k_head = 2 * c->k_head;
    d.v_page = 2 * c->v_page;
    d.v_slot = 2 * c->v_slot;
    d.v_head = 2 * c->v_head;
    d.pages = c->pages;
    d.starts = c->starts;
    d.lengths = c->lengths;
    d.pages_row = c->pages_row;
    d.by_page = divisor(c->page_size);
    d.n_pages = c->n_pages;
    d.page_size = c->page_size;
    d.n_seqs = c->n_seqs;
    d.max_pages = c->max_pages;
    d.max_places = c->max_pages * c->page_size;
    d.T = T;
    return d;
}

}  // namespace ops
