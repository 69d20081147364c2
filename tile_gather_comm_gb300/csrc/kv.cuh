// kv.cuh -- the paged cache's table: every read of it goes through KvTable, which turns whatever it
// holds into a page of the pool or none, so bad entries cost results, never an access outside.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/tgc.h"

namespace tgc {

struct KvTable {
    int num_pages, page_size, num_seqs, max_pages;
    int64_t ld;  // elements between the table's rows

    __host__ __device__ bool is_seq(int s) const { return s >= 0 && s < num_seqs; }
    __host__ __device__ bool is_page(int page) const { return page >= 0 && page < num_pages; }
    // What the table has at place `i` of sequence `s`, a page only where is_page says so; -1 outside.
    __host__ __device__ int entry_at(const int32_t *table, int s, int i) const {
        return is_seq(s) && i >= 0 && i < max_pages ? table[s * ld + i] : -1;
    }
    // The page that holds place `i` of sequence `s`, or -1.
    __host__ __device__ int page_at(const int32_t *table, int s, int i) const {
        const int page = entry_at(table, s, i);
        return is_page(page) ? page : -1;
    }
    // A length as the cache can hold it.
    __host__ __device__ int tokens(int len) const {
        const int most = max_pages * page_size;  // checked against TGC_MAX_SIZE
        return len < 0 ? 0 : len > most ? most : len;
    }
    __host__ __device__ int pages_of(int len) const { return (int)(((int64_t)len + page_size - 1) / page_size); }
};

// Sizes of a table; fills in its row stride.
inline int kv_table_check(int64_t num_pages, int64_t page_size, int64_t num_seqs, int64_t max_pages, int64_t *ld) {
    if (num_pages < 0 || num_pages > TGC_MAX_SIZE || page_size < 1 || page_size > TGC_MAX_SIZE || num_seqs < 0 ||
        num_seqs > TGC_MAX_SIZE || max_pages < 0 || max_pages > TGC_MAX_SIZE / page_size)
        return TGC_ERR_INVALID_ARG;
    if (num_seqs > 0 && max_pages > TGC_MAX_SIZE / num_seqs) return TGC_ERR_INVALID_ARG;
    if (*ld == 0) *ld = max_pages;
    if ((*ld < max_pages && num_seqs > 1) || *ld < 0 || *ld > (int64_t(1) << 40)) return TGC_ERR_INVALID_ARG;
    return TGC_OK;
}

// Whether vectors of D elements, n[i] of them stride[i] elements apart in each of up to 3 dimensions, lie apart from
// one another (each dimension steps over all that the smaller ones span) and end below 2^59 elements.
inline bool lie_apart(int64_t D, const int64_t *n, const int64_t *stride, int dims) {
    bool used[3] = {false, false, false};
    int64_t span = D;
    for (int step = 0; step < dims; ++step) {
        int at = -1;
        for (int i = 0; i < dims; ++i)
            if (!used[i] && n[i] > 1 && (at < 0 || stride[i] < stride[at])) at = i;
        if (at < 0) return true;
        used[at] = true;
        int64_t more = 0;
        if (stride[at] < span || __builtin_mul_overflow(stride[at], n[at] - 1, &more) || more >= (int64_t(1) << 58)) return false;
        span += more;
    }
    return span < (int64_t(1) << 59);
}

// Strides of a (num_pages, page_size, heads, D) pool, filled in where they are 0: dense in that order.
inline int kv_pages_check(int64_t num_pages, int64_t page_size, int64_t heads, int64_t D, int64_t *page_s, int64_t *token_s,
                          int64_t *head_s) {
    if (*head_s == 0) *head_s = D;
    if (*token_s == 0 && __builtin_mul_overflow(heads, *head_s, token_s)) return TGC_ERR_INVALID_ARG;
    if (*page_s == 0 && __builtin_mul_overflow(page_size, *token_s, page_s)) return TGC_ERR_INVALID_ARG;
    const int64_t n[3] = {num_pages, page_size, heads}, stride[3] = {*page_s, *token_s, *head_s};
    return lie_apart(D, n, stride, 3) ? TGC_OK : TGC_ERR_INVALID_ARG;
}

// Strides of a (T, heads, D) operand, the same way; nothing to say about one without entries.
inline int heads_check(int64_t T, int64_t heads, int64_t D, int64_t *st, int64_t *sh) {
    if (T == 0 || heads == 0) return TGC_OK;
    if (*sh == 0) *sh = D;
    if (*st == 0 && __builtin_mul_overflow(heads, *sh, st)) return TGC_ERR_INVALID_ARG;
    const int64_t n[2] = {T, heads}, stride[2] = {*st, *sh};
    return lie_apart(D, n, stride, 2) ? TGC_OK : TGC_ERR_INVALID_ARG;
}

}  // namespace tgc
