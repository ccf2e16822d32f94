// Pieces shared by the operators over paged caches (paged_rows.cu,
// paged_attention.cu, attention_weights.cu): checks of pools and tables, and the
// lookup of rows.
#pragma once

#include "views.cuh"

namespace statekv {

// A pool with its table, as a call names them.
struct Paging {
    const int32_t* table;
    int32_t stride, pages, num_pages, page_rows;
    // rows that a sequence can hold
    __host__ __device__ int64_t capacity() const { return table ? (int64_t)pages * page_rows : page_rows; }
};

template <class Args>
__host__ __device__ inline Paging paging_of(const Args& a) {
    return {a.table, a.table_stride, a.table_pages, a.num_pages, a.page_rows};
}

// rows of a sequence: rounded up to tiles they stay in 32 bits
constexpr int64_t kMaxRows = 0x7fffffffll - 256;

// Sizes of a pool and its table (STATEKV_OK or what to refuse them with).
inline int paging_ok(const Paging& p, int batch) {
    if (p.num_pages < 0 || p.page_rows < 0 || !ints_ok(p.table)) return STATEKV_E_INVALID_ARG;
    if (!p.table) {
        if (p.capacity() > kMaxRows) return STATEKV_E_UNSUPPORTED;
        return batch > p.num_pages ? STATEKV_E_CAPACITY : STATEKV_OK;
    }
    if (p.pages < 0 || p.stride < p.pages || p.page_rows < 16) return STATEKV_E_INVALID_ARG;
    if (p.page_rows % 16 != 0 || p.capacity() > kMaxRows) return STATEKV_E_UNSUPPORTED;
    return STATEKV_OK;
}

// Whether nothing can be in the cache (its memory is then not looked at).
inline bool paging_empty(const Paging& p) { return p.num_pages == 0 || p.capacity() == 0; }

#ifdef __CUDACC__
// The page that holds entry i of batch entry n's table row, or -1 (recorded).
__device__ __forceinline__ int page_at(const Paging& p, int n, int i, uint32_t* err) {
    if (!p.table) return n;
    const int page = p.table[(int64_t)n * p.stride + i];
    if ((uint32_t)page < (uint32_t)p.num_pages) return page;
    record_error(err, (uint32_t)STATEKV_E_DEVICE, kSitePage, (uint32_t)page);
    return -1;
}

// Rows of a sequence in the cache, and the new tokens among them.
struct Seq {
    int len, count;
};
// Of sequence s: the arrays' entries (both read at once) or the common values,
// recorded and clamped where they are out of range.
template <class Args>
__device__ __forceinline__ Seq sequence_of(const Args& a, int capacity, int s) {
    int len = a.lengths ? a.lengths[s] : a.length, count = a.counts ? a.counts[s] : a.tokens;
    const int len0 = len, count0 = count;
    len = min(max(len, 0), capacity);
    count = min(max(count, 0), min(a.tokens, len));
    if (len != len0 || count != count0)
        record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteLength, (uint32_t)(len != len0 ? len0 : count0));
    return {len, count};
}
#endif

}  // namespace statekv
