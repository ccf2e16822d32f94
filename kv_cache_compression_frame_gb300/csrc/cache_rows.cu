// Rows of a cache of keys and values: the accepted path of a drafted tree
// joins the cache, and complete 64-row blocks get the summaries that
// sparse_attention.cu selects them by.
#include <algorithm>

#include "views.cuh"
#include "sm100_ptx.cuh"

namespace statekv {
namespace {

// ------------------------------------------------------------ accepted rows
//   cache[len + i] = new[path[i]], i < count
// One CTA per (batch entry, KV head); every 16 bytes are read and written
// once, and all of a thread's loads are independent.  Bound by the launch: 13
// rows of 512 units, 7 MB in and out, take 3.5 us.
constexpr int kAppendThreads = 256;

__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ statekv_append_args a) {
    const int n = blockIdx.x / a.kv_heads, h = blockIdx.x - n * a.kv_heads;
    const int seq = n / a.layers;
    const int len = cache_length(a.lengths, a.length, seq, a.cache_rows, a.status);
    int count = a.counts ? a.counts[seq] : a.path_len;
    if (count < 0 || count > a.path_len || count > a.cache_rows - len) {
        record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteLength, (uint32_t)count);
        count = 0;                                           // nothing of this sequence is appended
    }
    const int row_units = a.head_dim * (a.dtype == STATEKV_BF16 ? 2 : 4) / 16;
    const int es = a.dtype == STATEKV_BF16 ? 2 : 4;
    const int32_t* path = a.path + (int64_t)seq * a.path_stride;
    // thread i takes the i-th 16 bytes of every 256: unit x of row r, all K rows
    // and then all V rows (their number, and the units', may pass 32 bits)
    const int dr = kAppendThreads / row_units, dx = kAppendThreads % row_units;
    int x = threadIdx.x % row_units;
    for (int64_t r = threadIdx.x / row_units; r < 2 * (int64_t)count;) {
        const bool is_v = r >= count;
        const int step = (int)(is_v ? r - count : r);
        const int node = path[step];
        if (node < 0 || node >= a.tokens) {
            record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteNode, (uint32_t)node);
        } else {
            const statekv_view& s = is_v ? a.v_new : a.k_new;
            const statekv_view& d = is_v ? a.v_cache : a.k_cache;
            const char* src = static_cast<const char*>(s.data) +
                              (n * s.batch_stride + h * s.head_stride + node * s.token_stride) * es;
            char* dst = static_cast<char*>(d.data) +
                        (n * d.batch_stride + h * d.head_stride + (int64_t)(len + step) * d.token_stride) * es;
            reinterpret_cast<uint4*>(dst)[x] = reinterpret_cast<const uint4*>(src)[x];
        }
        r += dr;
        x += dx;
        if (x >= row_units) {
            x -= row_units;
            ++r;
        }
    }
    if (a.new_lengths && h == 0 && n == seq * a.layers && threadIdx.x == 0) a.new_lengths[seq] = len + count;
}

// ---------------------------------------------------------- block summaries
// For each complete block of 64 rows:
//   mean  = fp32(sum of the rows) / 64
//   scale = max |mean| / 127,  code = round_even(mean * (127 / max |mean|))
// The codes have to come out the same however the rows are summed (a block's
// rank among the scores hangs on them), so the sum is exact to well below
// half an fp32 ulp: two-term accumulation, s + b = fl(s + b) + e with e
// recovered by Knuth's two-sum, in packed fp32 pairs.  Bound by HBM (each key
// is read once): a warp per block, 16 bytes per lane and load, eight loads on
// their way while eight are summed, across blocks too: 131072 rows of 8 heads,
// 270 MB, in 50 us = 5.4 TB/s (62 us with a warp per block and no overlap).
constexpr int kSumThreads = 128;
constexpr int kSumCtas = 5;                                  // per SM: 96 registers a thread, 64 of them keys in flight

// a - b (a fused multiply-add by -1 is exact in the product; there is no
// packed subtraction, and negating takes an instruction per half)
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return ptx::fma2(b, make_float2(-1.f, -1.f), a); }

// hi + lo += b
__device__ __forceinline__ void two_add(float2& hi, float2& lo, float2 b) {
    const float2 s = ptx::add2(hi, b);
    const float2 bb = sub2(s, hi);
    const float2 ea = sub2(hi, sub2(s, bb));
    const float2 eb = sub2(b, bb);
    lo = ptx::add2(lo, ptx::add2(ea, eb));
    hi = s;
}

template <int D>
__global__ void __launch_bounds__(kSumThreads, kSumCtas) summary_kernel(const __grid_constant__ statekv_summary_args a,
                                                                        int window) {
    constexpr int LPR = D / 8;                               // lanes per row
    constexpr int RPI = 32 / LPR;                            // rows per load
    constexpr int GROUP = 8;                                 // loads of a lane per group
    constexpr int GROUPS = STATEKV_BLOCK / RPI / GROUP;      // of a block: 4 or 2
    static_assert(GROUPS % 2 == 0, "a block starts in buffer 0");
    const int lane = threadIdx.x & 31;
    const int64_t items = (int64_t)a.batch * a.kv_heads * window;
    const int64_t step = (int64_t)gridDim.x * (kSumThreads / 32);
    // the first block from item i on that the appended rows completed: its
    // output index, and this lane's first key
    int64_t i = (int64_t)blockIdx.x * (kSumThreads / 32) + (threadIdx.x >> 5);
    int64_t out = 0;
    const __nv_bfloat16* k = nullptr;
    auto seek = [&]() -> bool {
        for (; i < items; i += step) {
            const int64_t unit = i / window;
            const int n = (int)(unit / a.kv_heads), h = (int)(unit - (int64_t)n * a.kv_heads);
            const int len = cache_length(a.lengths, a.length, n / a.layers, a.cache_rows, a.status);
            const int first = a.appended < len ? (len - a.appended) / STATEKV_BLOCK : 0;
            const int b = first + (int)(i - unit * window);
            if (b >= len / STATEKV_BLOCK) continue;
            out = unit * a.blocks + b;
            k = static_cast<const __nv_bfloat16*>(a.k_cache.data) + n * a.k_cache.batch_stride +
                h * a.k_cache.head_stride + ((int64_t)b * STATEKV_BLOCK + lane / LPR) * a.k_cache.token_stride +
                (lane % LPR) * 8;
            i += step;
            return true;
        }
        return false;
    };
    uint4 u[2][GROUP];
    auto load = [&](uint4 (&x)[GROUP], int g) {
#pragma unroll
        for (int r = 0; r < GROUP; ++r)
            x[r] = *reinterpret_cast<const uint4*>(k + (int64_t)((g * GROUP + r) * RPI) * a.k_cache.token_stride);
    };
    bool have = seek();
    if (have) load(u[0], 0);
    while (have) {
        const int64_t at = out;
        float2 hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) hi[j] = lo[j] = make_float2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            // the next group, or the next block's first, is on its way
            // while this one is summed
            if (g + 1 < GROUPS) load(u[(g + 1) & 1], g + 1);
            else if ((have = seek())) load(u[0], 0);
#pragma unroll
            for (int r = 0; r < GROUP; ++r) {
                const uint4 x = u[g & 1][r];
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    two_add(hi[j], lo[j], make_float2(__uint_as_float(w[j] << 16),
                                                      __uint_as_float(w[j] & 0xffff0000u)));
            }
        }
#pragma unroll
        for (int off = LPR; off < 32; off <<= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 oh = make_float2(__shfl_xor_sync(0xffffffffu, hi[j].x, off),
                                              __shfl_xor_sync(0xffffffffu, hi[j].y, off));
                const float2 ol = make_float2(__shfl_xor_sync(0xffffffffu, lo[j].x, off),
                                              __shfl_xor_sync(0xffffffffu, lo[j].y, off));
                // symmetric in the two lanes, so that both hold the same bits
                float2 e = make_float2(0.f, 0.f);
                two_add(hi[j], e, oh);
                lo[j] = ptx::add2(ptx::add2(lo[j], ol), e);
            }
        float m[8], top = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m[2 * j] = (hi[j].x + lo[j].x) * (1.f / STATEKV_BLOCK);
            m[2 * j + 1] = (hi[j].y + lo[j].y) * (1.f / STATEKV_BLOCK);
            top = fmaxf(top, fmaxf(fabsf(m[2 * j]), fabsf(m[2 * j + 1])));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        const float up = code_range(top), inv = top > 0.f ? 127.f / (top * up) : 0.f;
        if (lane < LPR) {
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int code = (int)fminf(fmaxf(rintf(m[j] * up * inv), -127.f), 127.f);
                w[j >> 2] |= (uint32_t)(code & 0xff) << (8 * (j & 3));
            }
            *reinterpret_cast<uint2*>(a.codes + at * D + lane * 8) = make_uint2(w[0], w[1]);
        }
        if (lane == 0) a.scales[at] = top / 127.f;
    }
}

}  // namespace

cudaError_t launch_append(const statekv_append_args& a, cudaStream_t st) {
    append_kernel<<<(unsigned)(a.batch * a.kv_heads), kAppendThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_summary(const statekv_summary_args& a, cudaStream_t st) {
    // blocks that the appended rows can have completed
    const int window = a.appended / STATEKV_BLOCK + 1 < a.blocks ? a.appended / STATEKV_BLOCK + 1 : a.blocks;
    const int64_t items = (int64_t)a.batch * a.kv_heads * window;
    // one wave of CTAs, each warp walking the blocks
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    const int64_t grid =
        std::min<int64_t>((items + kSumThreads / 32 - 1) / (kSumThreads / 32), (int64_t)sms * kSumCtas);
    if (a.head_dim == 128) summary_kernel<128><<<(unsigned)grid, kSumThreads, 0, st>>>(a, window);
    else summary_kernel<64><<<(unsigned)grid, kSumThreads, 0, st>>>(a, window);
    return cudaGetLastError();
}

}  // namespace statekv

extern "C" int statekv_append_accepted(const statekv_append_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_append_args& a = *args;
    if (a.dtype != STATEKV_BF16 && a.dtype != STATEKV_F32) return STATEKV_E_INVALID_ARG;
    const int es = a.dtype == STATEKV_BF16 ? 2 : 4;
    if (a.batch < 0 || a.layers < 1 || a.batch % a.layers != 0 || a.kv_heads < 1 || a.tokens < 0 ||
        a.path_len < 0 || !rows_ok(a.path_stride, a.path_len) || a.cache_rows < 0 || a.length < 0)
        return STATEKV_E_INVALID_ARG;
    if (a.head_dim < 8 || a.head_dim > 512 || a.head_dim * es % 16 != 0) return STATEKV_E_UNSUPPORTED;
    if ((int64_t)a.batch * a.kv_heads > 0x7fffffffll) return STATEKV_E_UNSUPPORTED;
    if (!a.status || !ints_ok(a.status) || !ints_ok(a.path) || !ints_ok(a.counts) || !ints_ok(a.lengths) ||
        !ints_ok(a.new_lengths))
        return STATEKV_E_INVALID_ARG;
    if (a.batch == 0) return STATEKV_OK;
    if (a.path_len > 0 && (!a.path || !view_ok(a.k_new, es, a.batch, a.kv_heads, a.tokens) ||
                           !view_ok(a.v_new, es, a.batch, a.kv_heads, a.tokens)))
        return STATEKV_E_INVALID_ARG;
    if (a.cache_rows > 0 && (!view_ok(a.k_cache, es, a.batch, a.kv_heads, a.cache_rows) ||
                             !view_ok(a.v_cache, es, a.batch, a.kv_heads, a.cache_rows) ||
                             !apart(a.k_cache, a.batch, a.kv_heads, a.cache_rows, a.head_dim) ||
                             !apart(a.v_cache, a.batch, a.kv_heads, a.cache_rows, a.head_dim)))
        return STATEKV_E_INVALID_ARG;
    // the sequence's length is read by every head's CTA while one writes the new one
    if (a.new_lengths && (a.new_lengths == a.lengths || a.new_lengths == a.counts)) return STATEKV_E_INVALID_ARG;
    if (!a.lengths && !a.counts && (int64_t)a.length + a.path_len > a.cache_rows) return STATEKV_E_CAPACITY;
    if (launch_append(a, reinterpret_cast<cudaStream_t>(cuda_stream)) != cudaSuccess) return view_cuda_fail();
    return STATEKV_OK;
}

extern "C" int statekv_block_summaries(const statekv_summary_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_summary_args& a = *args;
    if (a.batch < 0 || a.layers < 1 || a.batch % a.layers != 0 || a.kv_heads < 1 || a.blocks < 0 ||
        a.cache_rows < 0 || a.length < 0 || a.appended < 0)
        return STATEKV_E_INVALID_ARG;
    if (a.head_dim != 64 && a.head_dim != 128) return STATEKV_E_UNSUPPORTED;
    if (!a.status || !ints_ok(a.status) || !ints_ok(a.lengths)) return STATEKV_E_INVALID_ARG;
    if (a.blocks < a.cache_rows / STATEKV_BLOCK) return STATEKV_E_CAPACITY;
    if (a.batch == 0 || a.cache_rows < STATEKV_BLOCK) return STATEKV_OK;
    if (!view_ok(a.k_cache, 2, a.batch, a.kv_heads, a.cache_rows) || !a.codes ||
        reinterpret_cast<uintptr_t>(a.codes) % 8 || !a.scales || reinterpret_cast<uintptr_t>(a.scales) % 4)
        return STATEKV_E_INVALID_ARG;
    if (launch_summary(a, reinterpret_cast<cudaStream_t>(cuda_stream)) != cudaSuccess) return view_cuda_fail();
    return STATEKV_OK;
}
