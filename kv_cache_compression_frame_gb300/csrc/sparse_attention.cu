// Block-sparse attention of text tokens over a long cache: 8-bit block scores,
// top blocks, attention over them and over the rows since the last complete
// block, in one launch.
//
//   score_b = float(max_g qi_g . code_b) * scale_b      (whole-number products)
//   o = softmax(scale * q K_S^T) V_S,  S = rows of the top blocks and the tail
//
// After a 512-frame video one token of the dense step reads 67 MB of keys and
// values per layer with 2 KV heads; here it reads 0.5 MB of codes and 2 MB of
// the 64 best blocks.  The bound is latency: a chain of four dependent loads
// (query, codes, keys, values) and a selection in between.
//
// One cluster of C CTAs serves one (batch entry, KV head, token):
//  1. each CTA rounds the group's query rows to 8 bits and scores every C-th
//     run of 256 blocks, a block per thread (dp4a on 16-byte loads), storing
//     each score in all C CTAs' shared memory;
//  2. after a cluster barrier every CTA selects for itself (radix select on the
//     ordered scores, 11 + 11 + 10 bits; ties by index in the compaction), so
//     no result has to travel;
//  3. the chosen blocks and the tail's pieces go to the C * 8 warps in turn.
//     A warp attends over 64 rows on its own: K and V come from global memory
//     straight into matrix fragments (the order of d inside a product is free,
//     so each lane's 16-byte loads are its fragments), the G <= 16 query rows
//     are the 16 rows of m16n8k16, (m, l, O) stay in registers;
//  4. the warps merge in shared memory, the CTAs through distributed shared
//     memory, each CTA writing its share of the output.
// m16n8k16 and not tcgen05: with at most 16 query rows a 128-row product would
// waste 7/8 of the tensor core, and the data would have to pass through shared
// memory first.
// Scores, softmax statistics and O are fp32; P is rounded to bf16 for the
// product, l sums the unrounded P.
#include <algorithm>

#include "views.cuh"
#include "sm100_ptx.cuh"

namespace statekv {
namespace {

constexpr int kSparseThreads = 256;
constexpr int kSparseWarps = kSparseThreads / 32;
constexpr int kMaxTop = 1024;
constexpr int kMaxBlocks = 32768;
constexpr int kBins = 2048;

struct SparseKernelArgs {
    statekv_sparse_args a;
    float scale_log2;
    int32_t G, cluster;
    int32_t region;                  // bytes of shared memory used first for scores, then for partials
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// fp32 -> uint32 in the same order
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);             // -0 and 0 tie
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Exclusive prefix sum of one value per thread over the CTA, and the total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* s_warp, uint32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSparseWarps; ++w) {
        if (w < warp) before += s_warp[w];
        all += s_warp[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

template <int D>
__global__ void __launch_bounds__(kSparseThreads, 1) sparse_kernel(const __grid_constant__ SparseKernelArgs ka) {
    constexpr int KI = D / 32;               // 16-byte chunks of a K row per lane
    constexpr int DJ = D / 8;                // output columns per lane of a fragment's n index
    const statekv_sparse_args& a = ka.a;
    const int G = ka.G, C = ka.cluster;
    extern __shared__ __align__(16) uint8_t smem[];
    // region: scores [blocks] + bins, later the warps' O [8][G][D]
    uint32_t* s_key = reinterpret_cast<uint32_t*>(smem);
    float* s_o = reinterpret_cast<float*>(smem);
    uint8_t* fixed = smem + ka.region;
    float* s_part = reinterpret_cast<float*>(fixed);                    // [G][D] this CTA's O
    float2* s_pml = reinterpret_cast<float2*>(s_part + 16 * D);         // [16] its (m, l)
    float2* s_wml = s_pml + 16;                                         // [8][16] the warps' (m, l)
    int* s_list = reinterpret_cast<int*>(s_wml + kSparseWarps * 16);    // [kMaxTop]
    uint32_t* s_bin = reinterpret_cast<uint32_t*>(s_list + kMaxTop);    // [kBins]
    int8_t* s_q = reinterpret_cast<int8_t*>(s_bin + kBins);             // [16][D] query codes
    uint32_t* s_scan = reinterpret_cast<uint32_t*>(s_q + 16 * D);       // [8]
    uint32_t* s_pick = s_scan + kSparseWarps;                           // [2] digit, keys above it

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = C > 1 ? (int)ptx::cluster_ctarank() : 0;
    const int64_t item = blockIdx.x / C;
    const int64_t unit = item / a.tokens;
    const int tok = (int)(item - unit * a.tokens);
    const int n = (int)(unit / a.kv_heads), h = (int)(unit - (int64_t)n * a.kv_heads);
    const int len = cache_length(a.lengths, a.length, n / a.layers, a.cache_rows, a.status);
    const int row = len - a.tokens + tok;                    // this token's cache row
    const int nb = len > a.tokens ? (len - a.tokens) / STATEKV_BLOCK : 0;
    const bool choose = nb > a.top;
    if (C > 1) ptx::cluster_arrive_relaxed();

    // ---- the group's query rows, 8 bits, one scale
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q.data) + n * a.q.batch_stride +
                             (int64_t)(h * G) * a.q.head_stride + (int64_t)tok * a.q.token_stride;
    if (choose) {
        float top = 0.f;
        for (int i = tid; i < G * D; i += kSparseThreads)
            top = fmaxf(top, fabsf(__bfloat162float(q[(i / D) * a.q.head_stride + i % D])));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        if (lane == 0) s_scan[warp] = __float_as_uint(top);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kSparseWarps; ++w) top = fmaxf(top, __uint_as_float(s_scan[w]));
        const float inv = top > 0.f ? 127.f / top : 0.f;
        for (int i = tid; i < G * D; i += kSparseThreads) {
            const float x = rintf(__bfloat162float(q[(i / D) * a.q.head_stride + i % D]) * inv);
            s_q[i] = (int8_t)(int)fminf(fmaxf(x, -127.f), 127.f);
        }
        __syncthreads();
    }
    if (C > 1) ptx::cluster_wait();                          // every CTA has started: its memory may be written
    int nsel = nb;
    if (choose) {
        // ---- scores
        for (int b = rank * kSparseThreads + tid; b < nb; b += C * kSparseThreads) {
            const int64_t at = unit * a.blocks + b;
            const uint4* code = reinterpret_cast<const uint4*>(a.codes + at * D);
            uint4 w[D / 16];
#pragma unroll
            for (int i = 0; i < D / 16; ++i) w[i] = code[i];
            const float scale = a.scales[at];
            int best = INT32_MIN;
            for (int g = 0; g < G; ++g) {
                const uint4* qc = reinterpret_cast<const uint4*>(s_q + g * D);
                int s = 0;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint4 x = qc[i];
                    s = __dp4a((int)w[i].x, (int)x.x, s);
                    s = __dp4a((int)w[i].y, (int)x.y, s);
                    s = __dp4a((int)w[i].z, (int)x.z, s);
                    s = __dp4a((int)w[i].w, (int)x.w, s);
                }
                best = max(best, s);
            }
            const uint32_t key = ordered((float)best * scale);
            if (C == 1) s_key[b] = key;
            else
                for (int r = 0; r < C; ++r)
                    ptx::st_cluster_u32(ptx::cluster_map(ptx::smem_u32(s_key + b), (uint32_t)r), key);
        }
        if (C > 1) ptx::cluster_sync();
        else __syncthreads();
        // ---- the top-th largest key: digits of 11, 11 and 10 bits
        uint32_t prefix = 0, mask = 0, need = (uint32_t)a.top;
#pragma unroll 1
        for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
            for (int i = tid; i < kBins; i += kSparseThreads) s_bin[i] = 0;
            __syncthreads();
            const uint32_t digits = shift == 0 ? 1023u : 2047u;
            for (int b = tid; b < nb; b += kSparseThreads) {
                const uint32_t key = s_key[b];
                if ((key & mask) == prefix) atomicAdd(&s_bin[(key >> shift) & digits], 1u);
            }
            __syncthreads();
            // thread t holds the bins 8 t' .. 8 t' + 7 of t' = 255 - t: larger digits first
            uint32_t c[kBins / kSparseThreads], sum = 0, total;
#pragma unroll
            for (int i = 0; i < kBins / kSparseThreads; ++i) {
                c[i] = s_bin[kBins - 1 - (tid * (kBins / kSparseThreads) + i)];
                sum += c[i];
            }
            uint32_t above = block_scan(sum, s_scan, &total);
#pragma unroll
            for (int i = 0; i < kBins / kSparseThreads; ++i) {
                if (above < need && need <= above + c[i]) {
                    s_pick[0] = (uint32_t)(kBins - 1 - (tid * (kBins / kSparseThreads) + i));
                    s_pick[1] = above;
                }
                above += c[i];
            }
            __syncthreads();
            prefix |= s_pick[0] << shift;
            mask |= digits << shift;
            need -= s_pick[1];
            __syncthreads();
        }
        // ---- in index order: keys above the threshold, and the first `need` equal to it
        const int per = (nb + kSparseThreads - 1) / kSparseThreads;
        const int b0 = min(nb, tid * per), b1 = min(nb, b0 + per);
        uint32_t gt = 0, eq = 0, total;
        for (int b = b0; b < b1; ++b) {
            gt += s_key[b] > prefix;
            eq += s_key[b] == prefix;
        }
        // (both counts are at most 32768)
        uint32_t gt_before = block_scan(gt, s_scan, &total);
        uint32_t eq_before = block_scan(eq, s_scan, &total);
        for (int b = b0; b < b1; ++b) {
            const uint32_t key = s_key[b];
            const bool take = key > prefix || (key == prefix && eq_before < need);
            if (take) s_list[gt_before + min(eq_before, need)] = b;
            gt_before += key > prefix;
            eq_before += key == prefix;
        }
        nsel = a.top;
        __syncthreads();                                     // the list is complete, the scores are read
    }
    if (a.selected && rank == 0)
        for (int i = tid; i < a.top; i += kSparseThreads)
            a.selected[item * a.top + i] = i >= nsel || row < 0 ? -1 : choose ? s_list[i] : i;

    // ---- attention: entries 0..nsel-1 are blocks, the rest pieces of the tail
    const int quad = lane & 3, g8 = lane >> 2;
    uint32_t qf[D / 16][4];
    {
        const __nv_bfloat16* q0 = q + (int64_t)g8 * a.q.head_stride + quad * 8;
        const __nv_bfloat16* q1 = q0 + 8 * a.q.head_stride;
#pragma unroll
        for (int i = 0; i < KI; ++i) {
            const uint4 u = g8 < G ? *reinterpret_cast<const uint4*>(q0 + i * 32) : make_uint4(0, 0, 0, 0);
            const uint4 v = g8 + 8 < G ? *reinterpret_cast<const uint4*>(q1 + i * 32) : make_uint4(0, 0, 0, 0);
            qf[2 * i][0] = u.x; qf[2 * i][1] = v.x; qf[2 * i][2] = u.y; qf[2 * i][3] = v.y;
            qf[2 * i + 1][0] = u.z; qf[2 * i + 1][1] = v.z; qf[2 * i + 1][2] = u.w; qf[2 * i + 1][3] = v.w;
        }
    }
    float o[DJ][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < DJ; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(a.k_cache.data) + n * a.k_cache.batch_stride +
                              h * a.k_cache.head_stride + quad * 8;
    const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(a.v_cache.data) + n * a.v_cache.batch_stride +
                              h * a.v_cache.head_stride + g8 * DJ;
    const int tail = row - nb * STATEKV_BLOCK + 1;           // rows since the last complete block
    const int entries = nsel + (tail > 0 ? (tail + STATEKV_BLOCK - 1) / STATEKV_BLOCK : 0);
    for (int e = row < 0 ? entries : warp * C + rank; e < entries; e += kSparseWarps * C) {
        const int r0 = STATEKV_BLOCK * (e < nsel ? (choose ? s_list[e] : e) : nb + e - nsel);
        const int valid = min(STATEKV_BLOCK, row + 1 - r0);  // 64 for a block
        float s[8][4];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
            // (rows past the token's own are not read: they may lie past the cache)
            const int64_t r = r0 + min(8 * t + g8, valid - 1);
            uint4 kf[KI];
#pragma unroll
            for (int i = 0; i < KI; ++i)
                kf[i] = *reinterpret_cast<const uint4*>(kb + r * a.k_cache.token_stride + i * 32);
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                mma16816(s[t], qf[2 * i], kf[i].x, kf[i].y);
                mma16816(s[t], qf[2 * i + 1], kf[i].z, kf[i].w);
            }
        }
        if (valid < STATEKV_BLOCK) {
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (8 * t + 2 * quad + (x & 1) >= valid) s[t][x] = -INFINITY;
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            top[0] = ptx::max3(top[0], s[t][0], s[t][1]);
            top[1] = ptx::max3(top[1], s[t][2], s[t][3]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
            const float mn = fmaxf(m[x], top[x] * ka.scale_log2);
            const float f = m[x] == -INFINITY ? 0.f : ptx::ex2_approx(m[x] - mn);
            m[x] = mn;
            l[x] *= f;
#pragma unroll
            for (int j = 0; j < DJ; ++j) {
                o[j][2 * x] *= f;
                o[j][2 * x + 1] *= f;
            }
        }
        const float nm0 = m[0] == -INFINITY ? 0.f : -m[0], nm1 = m[1] == -INFINITY ? 0.f : -m[1];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            // V of keys 16 ks + {2 quad, 2 quad + 1} and 8 further, columns g8 * DJ ..
            uint4 v[4][DJ / 8];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int key = 16 * ks + 2 * quad + (y & 1) + 8 * (y >> 1);
                const int64_t r = r0 + min(key, valid - 1);
#pragma unroll
                for (int i = 0; i < DJ / 8; ++i) {
                    v[y][i] = *reinterpret_cast<const uint4*>(vb + r * a.v_cache.token_stride + 8 * i);
                    if (key >= valid) v[y][i] = make_uint4(0, 0, 0, 0);
                }
            }
            uint32_t p[4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float* x = s[2 * ks + t];
                const float p0 = ptx::ex2_approx(fmaf(x[0], ka.scale_log2, nm0));
                const float p1 = ptx::ex2_approx(fmaf(x[1], ka.scale_log2, nm0));
                const float p2 = ptx::ex2_approx(fmaf(x[2], ka.scale_log2, nm1));
                const float p3 = ptx::ex2_approx(fmaf(x[3], ka.scale_log2, nm1));
                l[0] += p0 + p1;
                l[1] += p2 + p3;
                p[2 * t] = ptx::pack_bf16x2(p0, p1);
                p[2 * t + 1] = ptx::pack_bf16x2(p2, p3);
            }
#pragma unroll
            for (int i = 0; i < DJ / 8; ++i) {
                const uint32_t k0[4] = {v[0][i].x, v[0][i].y, v[0][i].z, v[0][i].w};
                const uint32_t k1[4] = {v[1][i].x, v[1][i].y, v[1][i].z, v[1][i].w};
                const uint32_t k2[4] = {v[2][i].x, v[2][i].y, v[2][i].z, v[2][i].w};
                const uint32_t k3[4] = {v[3][i].x, v[3][i].y, v[3][i].z, v[3][i].w};
#pragma unroll
                for (int wd = 0; wd < 4; ++wd) {
                    mma16816(o[8 * i + 2 * wd], p, __byte_perm(k0[wd], k1[wd], 0x5410),
                             __byte_perm(k2[wd], k3[wd], 0x5410));
                    mma16816(o[8 * i + 2 * wd + 1], p, __byte_perm(k0[wd], k1[wd], 0x7632),
                             __byte_perm(k2[wd], k3[wd], 0x7632));
                }
            }
        }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
        l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
        const int r = g8 + 8 * x;
        if (r < G) {
            if (quad == 0) s_wml[warp * 16 + r] = make_float2(m[x], l[x]);
            float* dst = s_o + (warp * G + r) * D + 2 * quad * DJ;
#pragma unroll
            for (int j = 0; j < DJ; j += 4) {
                *reinterpret_cast<float4*>(dst + j) =
                    make_float4(o[j][2 * x], o[j + 1][2 * x], o[j + 2][2 * x], o[j + 3][2 * x]);
                *reinterpret_cast<float4*>(dst + DJ + j) =
                    make_float4(o[j][2 * x + 1], o[j + 1][2 * x + 1], o[j + 2][2 * x + 1], o[j + 3][2 * x + 1]);
            }
        }
    }
    __syncthreads();
    // ---- the CTA's warps, in order
    for (int i = tid; i < G * D; i += kSparseThreads) {
        const int r = i / D;
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < kSparseWarps; ++w) mm = fmaxf(mm, s_wml[w * 16 + r].x);
        float acc = 0.f, ls = 0.f;
#pragma unroll
        for (int w = 0; w < kSparseWarps; ++w) {
            const float2 x = s_wml[w * 16 + r];
            const float f = x.x == -INFINITY ? 0.f : ptx::ex2_approx(x.x - mm);
            acc = fmaf(s_o[w * G * D + i], f, acc);
            ls = fmaf(x.y, f, ls);
        }
        s_part[i] = acc;
        if (i % D == 0) s_pml[r] = make_float2(mm, ls);
    }
    if (C > 1) ptx::cluster_sync();
    else __syncthreads();
    // ---- the CTAs, in rank order; each writes its share of the output
    for (int i = (rank * kSparseThreads + tid) * 2; i < G * D; i += C * kSparseThreads * 2) {
        const int r = i / D;
        float2 ml[8];
        float mm = -INFINITY;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < C) {
                const uint32_t at = ptx::cluster_map(ptx::smem_u32(s_pml + r), (uint32_t)c);
                ml[c] = C > 1 ? ptx::ld_cluster_f32x2(at) : s_pml[r];
                mm = fmaxf(mm, ml[c].x);
            }
        float2 acc = make_float2(0.f, 0.f);
        float ls = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < C) {
                const uint32_t at = ptx::cluster_map(ptx::smem_u32(s_part + i), (uint32_t)c);
                const float2 x = C > 1 ? ptx::ld_cluster_f32x2(at) : *reinterpret_cast<const float2*>(s_part + i);
                const float f = ml[c].x == -INFINITY ? 0.f : ptx::ex2_approx(ml[c].x - mm);
                acc.x = fmaf(x.x, f, acc.x);
                acc.y = fmaf(x.y, f, acc.y);
                ls = fmaf(ml[c].y, f, ls);
            }
        const float inv = ls > 0.f || ls != ls ? 1.f / ls : 0.f;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + n * a.out.batch_stride +
                             (int64_t)(h * G + r) * a.out.head_stride + (int64_t)tok * a.out.token_stride + i % D;
        *reinterpret_cast<uint32_t*>(out) = ptx::pack_bf16x2(acc.x * inv, acc.y * inv);
    }
    if (C > 1) ptx::cluster_sync();                          // nobody leaves while its memory is read
}

// CTAs per (batch entry, KV head, token): as many as keep the device in one
// wave, at most 8 (the portable cluster size).
int cluster_for(int64_t items, int sms) {
    int c = 8;
    while (c > 1 && items * c > sms) c /= 2;
    return c;
}

template <int D>
cudaError_t launch(const SparseKernelArgs& ka, int64_t items, cudaStream_t st) {
    const size_t smem = ka.region + 16 * D * 4 + 16 * 8 + kSparseWarps * 16 * 8 + kMaxTop * 4 + kBins * 4 + 16 * D +
                        (kSparseWarps + 2) * 4;
    cudaError_t e = cudaFuncSetAttribute(sparse_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * ka.cluster));
    cfg.blockDim = dim3(kSparseThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ka.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sparse_kernel<D>, ka);
}

}  // namespace
}  // namespace statekv

extern "C" int statekv_sparse_attention(const statekv_sparse_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_sparse_args& a = *args;
    if (a.batch < 0 || a.layers < 1 || a.batch % a.layers != 0 || a.kv_heads < 1 || a.q_heads < a.kv_heads ||
        a.q_heads % a.kv_heads != 0 || a.tokens < 0 || a.cache_rows < 0 || a.length < 0 || a.blocks < 0 || a.top < 1 ||
        !(a.scale > 0.0) || !(a.scale < 1e30))
        return STATEKV_E_INVALID_ARG;
    if ((a.head_dim != 64 && a.head_dim != 128) || a.q_heads / a.kv_heads > 16 || a.top > kMaxTop ||
        a.cache_rows / STATEKV_BLOCK > kMaxBlocks)
        return STATEKV_E_UNSUPPORTED;
    const int64_t items = (int64_t)a.batch * a.kv_heads * a.tokens;
    if (items > 0x7fffffffll / 8) return STATEKV_E_UNSUPPORTED;
    if (!a.status || reinterpret_cast<uintptr_t>(a.status) % 4) return STATEKV_E_INVALID_ARG;
    if (a.blocks < a.cache_rows / STATEKV_BLOCK || (!a.lengths && a.length > a.cache_rows)) return STATEKV_E_CAPACITY;
    if (items == 0) return STATEKV_OK;
    if (!view_ok(a.q, 2) || !view_ok(a.out, 2) || reinterpret_cast<uintptr_t>(a.selected) % 4)
        return STATEKV_E_INVALID_ARG;
    if (a.cache_rows > 0 && (!view_ok(a.k_cache, 2) || !view_ok(a.v_cache, 2))) return STATEKV_E_INVALID_ARG;
    // the summaries are read only where there is something to choose
    const int most = (a.lengths ? a.cache_rows : a.length) / STATEKV_BLOCK;
    if (most > a.top && (!aligned16(a.codes) || !a.scales || reinterpret_cast<uintptr_t>(a.scales) % 4))
        return STATEKV_E_INVALID_ARG;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return view_cuda_fail();
    SparseKernelArgs k{};
    k.a = a;
    k.G = a.q_heads / a.kv_heads;
    k.scale_log2 = (float)(a.scale * 1.4426950408889634074);
    k.cluster = cluster_for(items, sms);
    k.region = (std::max(most > a.top ? most * 4 : 0, kSparseWarps * k.G * a.head_dim * 4) + 15) / 16 * 16;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = a.head_dim == 128 ? launch<128>(k, items, st) : launch<64>(k, items, st);
    return e == cudaSuccess ? STATEKV_OK : view_cuda_fail();
}
