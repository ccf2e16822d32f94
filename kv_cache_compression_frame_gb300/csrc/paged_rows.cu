// Rows of a paged cache: new ones are appended, and those of least accumulated
// attention weight are evicted.
#include <algorithm>

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace statekv {
namespace {

// A row of 16-byte units, K and V.
__device__ __forceinline__ char* row_ptr(const statekv_view& v, int page, int h, int row, int es) {
    return static_cast<char*>(v.data) +
           ((int64_t)page * v.batch_stride + h * v.head_stride + (int64_t)row * v.token_stride) * es;
}

// ------------------------------------------------------------------- append
//   cache[len + i] = new[i], i < count
// A CTA takes kAppendRows rows of one (batch entry, KV head); every 16 bytes are
// read and written once, and a thread's loads are independent of each other.
// Bound by the launch for a few tokens, by HBM (reads and writes) for a prompt:
// 512 rows of 56 units, 15 MB in and 15 out, take 6.6 us in the kernel and 10.3
// from launch to launch.
constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 32;

__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const __grid_constant__ statekv_paged_append_args a,
                                                                      int chunks) {
    const int u = blockIdx.x / chunks, chunk = blockIdx.x - u * chunks;
    const int n = u / a.kv_heads, h = u - n * a.kv_heads, seq = n / a.layers;
    const Paging pg = paging_of(a);
    const int len = cache_length(a.lengths, a.length, seq, (int)pg.capacity(), a.status);
    int count = a.counts ? a.counts[seq] : a.tokens;
    if (count < 0 || count > a.tokens) {
        record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteLength, (uint32_t)count);
        count = count < 0 ? 0 : a.tokens;
    }
    if (count > pg.capacity() - len) {
        record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteLength, (uint32_t)count);
        count = 0;                                           // nothing of this sequence is appended
    }
    if (a.new_lengths && h == 0 && n == seq * a.layers && chunk == 0 && threadIdx.x == 0)
        a.new_lengths[seq] = len + count;
    const int es = a.dtype == STATEKV_BF16 ? 2 : 4;
    const int row_units = a.head_dim * es / 16;
    // (none in most chunks of a batch padded far past its counts: a negative number would
    // leave 32 bits as a number of units)
    const int r0 = chunk * kAppendRows, rows = min(max(count - r0, 0), kAppendRows);
    for (int i = threadIdx.x; i < rows * row_units; i += kAppendThreads) {
        const int r = r0 + i / row_units, x = i % row_units;
        const int row = len + r;
        const int page = page_at(pg, n, a.table ? row / a.page_rows : 0, a.status);
        if (page < 0) continue;
        const int in_page = a.table ? row % a.page_rows : row;
        const uint4 k = reinterpret_cast<const uint4*>(row_ptr(a.k_new, n, h, r, es))[x];
        const uint4 v = reinterpret_cast<const uint4*>(row_ptr(a.v_new, n, h, r, es))[x];
        reinterpret_cast<uint4*>(row_ptr(a.k_pages, page, h, in_page, es))[x] = k;
        reinterpret_cast<uint4*>(row_ptr(a.v_pages, page, h, in_page, es))[x] = v;
    }
}

// ----------------------------------------------------------------- eviction
// Which rows stay: a radix select of the `keep` largest weights (ordered bits,
// 11 + 11 + 10 of them, -0 = 0, NaN lowest; rows that stay anyway rank above
// all), ties by row.  One cluster per (batch entry, KV head), each CTA a
// contiguous run of rows, in shared memory where it fits (it does up to 40960
// rows a CTA).  Of the cluster's histograms each CTA sums a part of the bins
// through distributed shared memory; the part that holds the threshold names it
// to all.  (Every CTA summing every bin read 128 KB a pass in a cluster of 16, 4 to 11 us.)
// A warp owns a contiguous run of its CTA's rows, so that a row's place among
// the kept is a sum of the counts before it.  Bound by latency: 131072 rows of 8
// units in clusters of 8 take 24 us, 4429 rows of 56 units 14.
constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;
static_assert(kEvictWarps == 32, "one lane per warp in the scans");
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxStaged = 40960;            // rows of a CTA in shared memory
constexpr int kMaxEvictRows = 1 << 22;

struct EvictKernelArgs {
    statekv_evict_args a;
    int32_t cluster;
    int32_t staged;                          // rows that the shared memory holds
};

// 16 bytes of another CTA's shared memory
__device__ __forceinline__ uint4 ld_cluster(uint32_t addr) {
    uint4 x;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(addr));
    return x;
}

// fp32 -> uint32 in the same order, from 1 up; NaN 0
__device__ __forceinline__ uint32_t weight_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);             // -0 and 0 tie
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictKernelArgs ka) {
    const statekv_evict_args& a = ka.a;
    __shared__ __align__(16) uint32_t s_hist[kBins], s_part[kBins];
    __shared__ uint32_t s_rows[kMaxCluster], s_scan[kEvictWarps];
    __shared__ uint32_t s_pick[3];                           // bin, rows of it that stay, its rows
    __shared__ uint32_t s_count[kEvictWarps][2];             // rows above the threshold, rows on it
    __shared__ uint32_t s_cta[kMaxCluster][2];
    extern __shared__ float s_weights[];
    // The move, where there is one, may be launched now; it waits for this grid to end.
    // Otherwise the next kernel is not ours to release.
    if (a.keep > 0) ptx::dep_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = ka.cluster, rank = blockIdx.x % C, u = blockIdx.x / C;
    const int n = u / a.kv_heads, h = u - n * a.kv_heads, seq = n / a.layers;
    const Paging pg = paging_of(a);
    const int len = cache_length(a.lengths, a.length, seq, (int)pg.capacity(), a.status);
    const int keep = min(len, a.keep);
    const float* w = a.weights + (int64_t)u * a.weight_rows;
    float* w_out = a.weights_out + (int64_t)u * a.out_rows;
    int32_t* kept = a.kept + (int64_t)u * a.keep;
    if (a.new_lengths && h == 0 && n == seq * a.layers && rank == 0 && tid == 0) a.new_lengths[seq] = keep;
    for (int64_t i = (int64_t)keep + rank * kEvictThreads + tid; i < a.out_rows; i += C * kEvictThreads) {
        w_out[i] = 0.f;
        if (i < a.keep) kept[i] = -1;
    }
    if (a.keep == 0) return;
    if (len <= a.keep) {
        for (int i = rank * kEvictThreads + tid; i < len; i += C * kEvictThreads) {
            kept[i] = i;
            w_out[i] = w[i];
        }
        return;                                              // (every CTA of the cluster)
    }
    // this CTA's rows, and this warp's of them
    const int per_warp = ((len + C * kEvictWarps - 1) / (C * kEvictWarps) + 31) / 32 * 32;
    const int c0 = min(len, rank * per_warp * kEvictWarps), c1 = min(len, c0 + per_warp * kEvictWarps);
    const int w0 = min(c1, c0 + warp * per_warp), w1 = min(c1, w0 + per_warp);
    const bool staged = c1 - c0 <= ka.staged;
    const float* src = staged ? s_weights - c0 : w;
    auto key_of = [&](int i, float x) {
        return i < a.sinks || i >= len - a.recent ? 0xffffffffu : weight_key(x);
    };
    uint32_t need = (uint32_t)keep, prefix = 0, fixed = 0;   // of the rows whose `fixed` bits are `prefix`
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
        for (int i = tid; i < kBins; i += kEvictThreads) s_hist[i] = s_part[i] = 0;
        __syncthreads();
        if (pass == 0) {
            // the rows come in on the way, eight loads of a thread at a time
            for (int i0 = c0 + tid; i0 < c1; i0 += 8 * kEvictThreads) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = i0 + e * kEvictThreads < c1 ? w[i0 + e * kEvictThreads] : 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = i0 + e * kEvictThreads;
                    if (i >= c1) break;
                    if (staged) s_weights[i - c0] = x[e];
                    atomicAdd(&s_hist[key_of(i, x[e]) >> shift], 1u);
                }
            }
        } else {
#pragma unroll 4
            for (int i = c0 + tid; i < c1; i += kEvictThreads) {
                const uint32_t key = key_of(i, src[i]);
                if ((key & fixed) == prefix) atomicAdd(&s_hist[(key >> shift) & (uint32_t)(bins - 1)], 1u);
            }
        }
        ptx::cluster_sync();
        // CTA r sums the cluster's bins of its part, and tells how many rows they hold
        const int part = bins / C, groups = part / 4;
        if (tid < bins / 4) {
            const int g = tid % groups, r = tid / groups;
            const uint4 x = ld_cluster(ptx::cluster_map(ptx::smem_u32(&s_hist[rank * part + 4 * g]), (uint32_t)r));
            if (C == 1) {
                *reinterpret_cast<uint4*>(&s_part[4 * g]) = x;
            } else {
                if (x.x) atomicAdd(&s_part[4 * g], x.x);
                if (x.y) atomicAdd(&s_part[4 * g + 1], x.y);
                if (x.z) atomicAdd(&s_part[4 * g + 2], x.z);
                if (x.w) atomicAdd(&s_part[4 * g + 3], x.w);
            }
        }
        __syncthreads();
        // thread t has the t-th bin of the part from the top, or two
        const int two = part > kEvictThreads, top = part - 1 - (two ? 2 * tid : tid);
        const uint32_t hi = top >= 0 ? s_part[top] : 0u, lo = two ? s_part[top - 1] : 0u, mine = hi + lo;
        uint32_t upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += x;
        }
        if (lane == 31) s_scan[warp] = upto;
        __syncthreads();
        const uint32_t of_warp = s_scan[lane];
        uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0u) + upto - mine;
        if (warp == 0) {
            const uint32_t all = __reduce_add_sync(0xffffffffu, of_warp);
            if (lane < C) ptx::st_cluster_u32(ptx::cluster_map(ptx::smem_u32(&s_rows[rank]), (uint32_t)lane), all);
        }
        ptx::cluster_sync();
        for (int r = C - 1; r > rank; --r) before += s_rows[r];
        if (before < need && need <= before + mine) {
            // the part that the threshold is in names it to all
            const bool low = before + hi < need;
            if (low) before += hi;
            for (int r = 0; r < C; ++r) {
                const uint32_t to = ptx::cluster_map(ptx::smem_u32(&s_pick[0]), (uint32_t)r);
                ptx::st_cluster_u32(to, (uint32_t)(rank * part + top - (low ? 1 : 0)));
                ptx::st_cluster_u32(to + 4, need - before);
                ptx::st_cluster_u32(to + 8, low ? lo : hi);
            }
        }
        ptx::cluster_sync();
        prefix |= s_pick[0] << shift;
        fixed |= (uint32_t)(bins - 1) << shift;
        need = s_pick[1];
        if (need == s_pick[2]) break;                        // the whole bin stays
    }
    // rows above `prefix` (of the bits that were looked at) stay, and the first `need` that are equal to it
    uint32_t gt = 0, eq = 0;
#pragma unroll 4
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const uint32_t key = i0 + lane < w1 ? key_of(i0 + lane, src[i0 + lane]) & fixed : 0u;
        gt += __popc(__ballot_sync(0xffffffffu, i0 + lane < w1 && key > prefix));
        eq += __popc(__ballot_sync(0xffffffffu, i0 + lane < w1 && key == prefix));
    }
    if (lane == 0) {
        s_count[warp][0] = gt;
        s_count[warp][1] = eq;
    }
    __syncthreads();
    if (tid < C) {
        // this CTA's counts into every CTA's shared memory
        uint32_t above = 0, on = 0;
        for (int i = 0; i < kEvictWarps; ++i) {
            above += s_count[i][0];
            on += s_count[i][1];
        }
        const uint32_t at = ptx::cluster_map(ptx::smem_u32(&s_cta[rank][0]), (uint32_t)tid);
        ptx::st_cluster_u32(at, above);
        ptx::st_cluster_u32(at + 4, on);
    }
    ptx::cluster_sync();
    gt = eq = 0;
    for (int r = 0; r < rank; ++r) {
        gt += s_cta[r][0];
        eq += s_cta[r][1];
    }
    for (int i = 0; i < warp; ++i) {
        gt += s_count[i][0];
        eq += s_count[i][1];
    }
#pragma unroll 4
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t key = i < w1 ? key_of(i, src[i]) & fixed : 0u;
        const unsigned above = __ballot_sync(0xffffffffu, i < w1 && key > prefix);
        const unsigned on = __ballot_sync(0xffffffffu, i < w1 && key == prefix);
        const unsigned lower = (1u << lane) - 1u;
        const uint32_t g = gt + __popc(above & lower), e = eq + __popc(on & lower);
        if (i < w1 && (key > prefix || (key == prefix && e < need))) {
            const uint32_t at = g + min(e, need);
            kept[at] = i;
            w_out[at] = src[i];
        }
        gt += __popc(above);
        eq += __popc(on);
    }
}

// The kept rows move: a CTA takes kMoveRows of one (batch entry, KV head),
// finds where they lie and where they go, and copies K and V, 16 bytes at a time.
// Bound by HBM: 4096 rows of 56 units, 117 MB in and out, take 40 us = 5.9 TB/s.
// (16 or 64 rows a CTA: 46, 40.)
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ statekv_evict_args a,
                                                                  int chunks) {
    __shared__ int s_from[kMoveRows][2], s_to[kMoveRows][2];     // page, row
    const int u = blockIdx.x / chunks, chunk = blockIdx.x - u * chunks;
    const int n = u / a.kv_heads, h = u - n * a.kv_heads;
    ptx::dep_wait();
    const int r0 = chunk * kMoveRows, rows = min(kMoveRows, a.keep - r0);
    const Paging from = paging_of(a), to{a.out_table, a.out_table_stride, a.out_table_pages, a.out_num_pages, a.out_page_rows};
    if ((int)threadIdx.x < rows) {
        const int r = r0 + threadIdx.x, row = a.kept[(int64_t)u * a.keep + r];
        int* s = s_from[threadIdx.x];
        s[0] = -1;
        if (row >= 0) {
            s[0] = page_at(from, n, from.table ? row / a.page_rows : 0, a.status);
            s[1] = from.table ? row % a.page_rows : row;
            int* t = s_to[threadIdx.x];
            t[0] = page_at(to, n, to.table ? r / a.out_page_rows : 0, a.status);
            t[1] = to.table ? r % a.out_page_rows : r;
            if (t[0] < 0) s[0] = -1;
        }
    }
    __syncthreads();
    const int es = a.dtype == STATEKV_BF16 ? 2 : 4;
    const int row_units = a.head_dim * es / 16;
#pragma unroll 4
    for (int i = threadIdx.x; i < rows * row_units; i += kMoveThreads) {
        const int r = i / row_units, x = i % row_units;
        if (s_from[r][0] < 0) continue;
        const uint4 k = reinterpret_cast<const uint4*>(row_ptr(a.k_pages, s_from[r][0], h, s_from[r][1], es))[x];
        const uint4 v = reinterpret_cast<const uint4*>(row_ptr(a.v_pages, s_from[r][0], h, s_from[r][1], es))[x];
        reinterpret_cast<uint4*>(row_ptr(a.k_out, s_to[r][0], h, s_to[r][1], es))[x] = k;
        reinterpret_cast<uint4*>(row_ptr(a.v_out, s_to[r][0], h, s_to[r][1], es))[x] = v;
    }
}

cudaError_t launch_evict(const statekv_evict_args& a, int dev, int sms, cudaStream_t st) {
    EvictKernelArgs ka{};
    ka.a = a;
    const int64_t units = (int64_t)a.batch * a.kv_heads;
    const int64_t cap = paging_of(a).capacity();
    // CTAs of at most 4096 rows, as long as they all run at once (one per SM: its
    // 1024 threads take the registers)
    int c = 1;
    while (c < kMaxCluster && cap > (int64_t)c * 4096 && units * c * 2 <= sms) c *= 2;
    ka.cluster = c;
    const int64_t slice = ((cap + c * kEvictWarps - 1) / (c * kEvictWarps) + 31) / 32 * 32 * kEvictWarps;
    ka.staged = slice <= kMaxStaged ? (int)slice : 0;
    static std::atomic<uint64_t> done{0};
    const void* kernel = reinterpret_cast<const void*>(&evict_select_kernel);
    cudaError_t e = allow_smem(kernel, kMaxStaged * 4, dev, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * c));
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = (size_t)ka.staged * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, ka);
    if (e != cudaSuccess || a.keep == 0) return e;
    const int chunks = (a.keep + kMoveRows - 1) / kMoveRows;
    cudaLaunchConfig_t mv = {};
    mv.gridDim = dim3((unsigned)(units * chunks));
    mv.blockDim = dim3(kMoveThreads);
    mv.stream = st;
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    mv.attrs = early;
    mv.numAttrs = 1;
    return cudaLaunchKernelEx(&mv, evict_move_kernel, a, chunks);
}

}  // namespace
}  // namespace statekv

extern "C" int statekv_paged_append(const statekv_paged_append_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_paged_append_args& a = *args;
    if (a.dtype != STATEKV_BF16 && a.dtype != STATEKV_F32) return STATEKV_E_INVALID_ARG;
    const int es = a.dtype == STATEKV_BF16 ? 2 : 4;
    if (a.batch < 0 || a.layers < 1 || a.batch % a.layers != 0 || a.kv_heads < 1 || a.tokens < 0 || a.length < 0)
        return STATEKV_E_INVALID_ARG;
    if (a.head_dim < 8 || a.head_dim > 512 || a.head_dim * es % 16 != 0) return STATEKV_E_UNSUPPORTED;
    if (!a.status || !ints_ok(a.status) || !ints_ok(a.counts) || !ints_ok(a.lengths) || !ints_ok(a.new_lengths))
        return STATEKV_E_INVALID_ARG;
    const Paging pg = paging_of(a);
    int r = paging_ok(pg, a.batch);
    if (r != STATEKV_OK) return r;
    // the sequence's length is read by every head's CTAs while one writes the new one
    if (a.new_lengths && (a.new_lengths == a.lengths || a.new_lengths == a.counts)) return STATEKV_E_INVALID_ARG;
    if (!a.lengths && !a.counts && (int64_t)a.length + a.tokens > pg.capacity()) return STATEKV_E_CAPACITY;
    if (!a.lengths && a.length > pg.capacity()) return STATEKV_E_CAPACITY;
    if (a.batch == 0) return STATEKV_OK;
    if (a.tokens > 0 && (!view_ok(a.k_new, es, a.batch, a.kv_heads, a.tokens) ||
                         !view_ok(a.v_new, es, a.batch, a.kv_heads, a.tokens)))
        return STATEKV_E_INVALID_ARG;
    if (!paging_empty(pg))
        for (const statekv_view* v : {&a.k_pages, &a.v_pages})
            if (!view_ok(*v, es, a.num_pages, a.kv_heads, a.page_rows) ||
                !apart(*v, a.num_pages, a.kv_heads, a.page_rows, a.head_dim))
                return STATEKV_E_INVALID_ARG;
    const Extent pool{a.num_pages, a.kv_heads, a.page_rows};
    if (!paging_empty(pg) && share(a.k_pages, pool, a.v_pages, pool, a.head_dim, es)) return STATEKV_E_INVALID_ARG;
    const int64_t seqs = a.batch / a.layers;
    for (const int32_t* in : {a.lengths, a.counts})
        if (in && a.new_lengths && overlap(in, seqs, a.new_lengths, seqs)) return STATEKV_E_INVALID_ARG;
    const int64_t chunks = std::max<int64_t>(1, ((int64_t)a.tokens + kAppendRows - 1) / kAppendRows);
    const int64_t grid = (int64_t)a.batch * a.kv_heads * chunks;
    if (grid > 0x7fffffffll) return STATEKV_E_UNSUPPORTED;
    paged_append_kernel<<<(unsigned)grid, kAppendThreads, 0, reinterpret_cast<cudaStream_t>(cuda_stream)>>>(
        a, (int)chunks);
    return cudaGetLastError() == cudaSuccess ? STATEKV_OK : view_cuda_fail();
}

extern "C" int statekv_evict_rows(const statekv_evict_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_evict_args& a = *args;
    if (a.dtype != STATEKV_BF16 && a.dtype != STATEKV_F32) return STATEKV_E_INVALID_ARG;
    const int es = a.dtype == STATEKV_BF16 ? 2 : 4;
    if (a.batch < 0 || a.layers < 1 || a.batch % a.layers != 0 || a.kv_heads < 1 || a.length < 0 || a.keep < 0 ||
        a.sinks < 0 || a.recent < 0 || (int64_t)a.sinks + a.recent > a.keep || a.weight_rows < 0 || a.out_rows < 0)
        return STATEKV_E_INVALID_ARG;
    if (a.head_dim < 8 || a.head_dim > 512 || a.head_dim * es % 16 != 0) return STATEKV_E_UNSUPPORTED;
    if (!a.status || !ints_ok(a.status) || !ints_ok(a.lengths) || !ints_ok(a.new_lengths) || !ints_ok(a.weights) ||
        !ints_ok(a.weights_out) || !ints_ok(a.kept))
        return STATEKV_E_INVALID_ARG;
    const Paging pg = paging_of(a), to{a.out_table, a.out_table_stride, a.out_table_pages, a.out_num_pages, a.out_page_rows};
    int r = paging_ok(pg, a.batch);
    if (r == STATEKV_OK) r = paging_ok(to, a.batch);
    if (r != STATEKV_OK) return r;
    if (pg.capacity() > kMaxEvictRows) return STATEKV_E_UNSUPPORTED;
    if (a.weight_rows < pg.capacity() || a.out_rows < a.keep || to.capacity() < a.keep) return STATEKV_E_CAPACITY;
    if (!a.lengths && a.length > pg.capacity()) return STATEKV_E_CAPACITY;
    if (a.new_lengths && a.new_lengths == a.lengths) return STATEKV_E_INVALID_ARG;
    // without a table of its own an entry's rows would go over those of another,
    // or over its own
    const bool same = a.k_out.data == a.k_pages.data || a.v_out.data == a.v_pages.data ||
                      a.k_out.data == a.v_pages.data || a.v_out.data == a.k_pages.data;
    if (same && (!a.out_table || !a.table)) return STATEKV_E_INVALID_ARG;
    if (a.batch == 0) return STATEKV_OK;
    if ((a.weight_rows > 0 && !a.weights) || (a.out_rows > 0 && !a.weights_out) || (a.keep > 0 && !a.kept))
        return STATEKV_E_INVALID_ARG;
    if (!paging_empty(pg) && (!view_ok(a.k_pages, es, a.num_pages, a.kv_heads, a.page_rows) ||
                              !view_ok(a.v_pages, es, a.num_pages, a.kv_heads, a.page_rows)))
        return STATEKV_E_INVALID_ARG;
    if (!paging_empty(to))
        for (const statekv_view* v : {&a.k_out, &a.v_out})
            if (!view_ok(*v, es, a.out_num_pages, a.kv_heads, a.out_page_rows) ||
                !apart(*v, a.out_num_pages, a.kv_heads, a.out_page_rows, a.head_dim))
                return STATEKV_E_INVALID_ARG;
    const int64_t units = (int64_t)a.batch * a.kv_heads, seqs = a.batch / a.layers;
    // (outputs first: an output with each input and with the outputs behind it)
    struct { const void* p; int64_t n; } arrays[] = {
        {a.weights_out, units * a.out_rows}, {a.kept, units * a.keep}, {a.new_lengths, seqs},
        {a.weights, units * a.weight_rows}, {a.lengths, seqs},
        {a.table, (int64_t)(a.batch - 1) * a.table_stride + a.table_pages},
        {a.out_table, (int64_t)(a.batch - 1) * a.out_table_stride + a.out_table_pages}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 7; ++j)
            if (arrays[i].p && arrays[j].p && overlap(arrays[i].p, arrays[i].n, arrays[j].p, arrays[j].n))
                return STATEKV_E_INVALID_ARG;
    // K and V go to rows of their own; with both tables the pages that are read and
    // those that are written are the caller's to keep apart
    const Extent source{a.num_pages, a.kv_heads, a.page_rows}, target{a.out_num_pages, a.kv_heads, a.out_page_rows};
    if (!paging_empty(to) && share(a.k_out, target, a.v_out, target, a.head_dim, es)) return STATEKV_E_INVALID_ARG;
    if ((!a.table || !a.out_table) && !paging_empty(pg) && !paging_empty(to))
        for (const statekv_view* x : {&a.k_pages, &a.v_pages})
            for (const statekv_view* y : {&a.k_out, &a.v_out})
                if (share(*x, source, *y, target, a.head_dim, es)) return STATEKV_E_INVALID_ARG;
    if (units * 16 > 0x7fffffffll || units * ((a.keep + kMoveRows - 1) / kMoveRows) > 0x7fffffffll)
        return STATEKV_E_UNSUPPORTED;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return view_cuda_fail();
    return launch_evict(a, dev, sms, reinterpret_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? STATEKV_OK
                                                                                                : view_cuda_fail();
}
