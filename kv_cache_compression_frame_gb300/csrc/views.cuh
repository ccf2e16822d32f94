// Pieces shared by the handle-free text operators (norm_rope.cu,
// cache_rows.cu, tree_attention.cu, sparse_attention.cu): checks of strided
// views and the lookup of a sequence's cache length.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "statekv_internal.cuh"

namespace statekv {

// Lets a kernel take `bytes` of dynamic shared memory on device dev, once per
// device (`done`: one bit each; devices past 63 ask every time).
inline cudaError_t allow_smem(const void* kernel, int bytes, int dev, std::atomic<uint64_t>& done) {
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

inline bool current_device(int* dev, int* sms) {
    return cudaGetDevice(dev) == cudaSuccess &&
           cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) == cudaSuccess;
}

// A failed CUDA call: clear the runtime's last-error state (a refused launch,
// for instance, would otherwise be reported again by the next call that
// checks it, in this library or the caller's code) and report E_CUDA.
inline int view_cuda_fail() {
    cudaGetLastError();
    return STATEKV_E_CUDA;
}

inline bool aligned16(const void* p) { return p && reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// An array of 32-bit entries, or none.
inline bool ints_ok(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// Whether two arrays of n and m 32-bit entries share memory.
inline bool overlap(const void* p, int64_t n, const void* q, int64_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
    return x < y + 4 * (uint64_t)m && y < x + 4 * (uint64_t)n;
}

// Rows of `len` entries `stride` apart, or one row (0) for all.
inline bool rows_ok(int32_t stride, int32_t len) { return stride == 0 || stride >= len; }

// Every row of the view [batch][heads][rows] starts on a 16-byte boundary (what
// 16-byte loads and TMA need), and no stride is negative.  The stride of a
// dimension of one entry leads nowhere and may be anything.
inline bool view_ok(const statekv_view& v, int esize, int64_t batch, int64_t heads, int64_t rows) {
    if (!aligned16(v.data)) return false;
    auto ok = [&](int64_t n, int64_t s) { return n < 2 || (s >= 0 && s * esize % 16 == 0); };
    return ok(batch, v.batch_stride) && ok(heads, v.head_stride) && ok(rows, v.token_stride);
}

// No two entries of the view start at the same place (what a TMA view needs).
inline bool spread(const statekv_view& v, int64_t batch, int64_t heads, int64_t rows) {
    return (batch < 2 || v.batch_stride > 0) && (heads < 2 || v.head_stride > 0) && (rows < 2 || v.token_stride > 0);
}

// No entries of the view of rows of d elements share memory: what an output
// needs.  Taken from the smallest stride up, each has to span all that the
// smaller ones reach, as in any slice or permutation of an ordinary tensor.
inline bool apart(const statekv_view& v, int64_t batch, int64_t heads, int64_t rows, int64_t d) {
    if (batch < 1 || heads < 1 || rows < 1) return true;
    struct Dim { int64_t n, stride; } dims[3] = {{rows, v.token_stride}, {heads, v.head_stride}, {batch, v.batch_stride}};
    std::sort(dims, dims + 3, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
    int64_t reach = d;
    for (const Dim& x : dims) {
        if (x.n < 2) continue;
        if (x.stride < reach) return false;
        if (x.stride > (INT64_MAX - reach) / (x.n - 1)) return false;
        reach += x.stride * (x.n - 1);
    }
    return true;
}

// A view's dimensions.
struct Extent {
    int64_t batch, heads, rows;
};

// Whether rows of two views share memory.  They do where the distance of their first
// entries is a sum of differences of indices times the strides; dimensions of
// another stride in either are taken as a range.  So K and V next to each other in
// one tensor, page by page or row by row, and two parts of one cache are told apart.
inline bool share(const statekv_view& x, const Extent& nx, const statekv_view& y, const Extent& ny, int64_t d, int es) {
    struct Dim { __int128 stride, before, after; } dims[3];      // indices of y past x's, of x past y's
    if (nx.batch < 1 || nx.heads < 1 || nx.rows < 1 || ny.batch < 1 || ny.heads < 1 || ny.rows < 1) return false;
    __int128 up0 = d - 1, down0 = d - 1;
    int count = 0;
    auto take = [&](int64_t n, int64_t s, int64_t m, int64_t t) {
        if (n < 2 && m < 2) return;
        if (n < 2) s = t;                                        // (a stride of one entry leads nowhere)
        if (m < 2) t = s;
        if (s == t) {
            if (s > 0) dims[count++] = {s, m - 1, n - 1};
        } else {
            up0 += (__int128)(n - 1) * s;
            down0 += (__int128)(m - 1) * t;
        }
    };
    take(nx.batch, x.batch_stride, ny.batch, y.batch_stride);
    take(nx.heads, x.head_stride, ny.heads, y.head_stride);
    take(nx.rows, x.token_stride, ny.rows, y.token_stride);
    std::sort(dims, dims + count, [](const Dim& p, const Dim& q) { return p.stride > q.stride; });
    // left = sum of k_i stride_i + e, -before_i <= k_i <= after_i, -down0 <= e <= up0: largest stride
    // first, what the smaller ones reach leaves two steps of it (where they reach further, as in
    // views that overlap in themselves, it is not looked into)
    auto meet = [&](auto& self, int i, __int128 left) -> bool {
        if (i == count) return left <= up0 && -left <= down0;
        __int128 up = up0, down = down0;
        for (int j = i + 1; j < count; ++j) up += dims[j].after * dims[j].stride, down += dims[j].before * dims[j].stride;
        const __int128 s = dims[i].stride;
        auto floor_div = [](__int128 p, __int128 q) { return p / q - (p % q < 0 ? 1 : 0); };
        const __int128 from = std::max(-dims[i].before, -floor_div(up - left, s));
        const __int128 to = std::min(dims[i].after, floor_div(left + down, s));
        if (to - from > 2) return true;
        for (__int128 k = from; k <= to; ++k)
            if (self(self, i + 1, left - k * s)) return true;
        return false;
    };
    // y's first entry from x's, in elements (both are on 16-byte boundaries)
    const __int128 x0 = reinterpret_cast<uintptr_t>(x.data), y0 = reinterpret_cast<uintptr_t>(y.data);
    return meet(meet, 0, (y0 - x0) / es);
}

#ifdef __CUDACC__
// Rounding to 8 bits with one scale multiplies by 127 / max |x|, which passes
// fp32's range for maxima below 2^-121 (zeros would become inf * 0).  Values
// and maximum times this power of two, exact, give the same codes without that.
__device__ __forceinline__ float code_range(float top) { return top < 0x1p-100f ? 0x1p64f : 1.f; }

// Rows of sequence s, from the array or the common value.  A negative length
// or one past `most` is recorded and clamped, so that every access that
// follows from it stays in bounds.
__device__ __forceinline__ int cache_length(const int32_t* lengths, int32_t length, int s, int most,
                                            uint32_t* err) {
    int n = lengths ? lengths[s] : length;
    if (n < 0 || n > most) {
        record_error(err, (uint32_t)STATEKV_E_DEVICE, kSiteLength, (uint32_t)n);
        n = n < 0 ? 0 : most;
    }
    return n;
}
#endif

}  // namespace statekv
