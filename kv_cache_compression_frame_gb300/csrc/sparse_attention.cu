// Block-sparse attention of text tokens over a long cache: 8-bit block scores,
// top blocks, attention over them and over the rows since the last complete
// block, in one launch.
//
//   score_b = float(max_g qi_g . code_b) * scale_b      (whole-number products)
//   o = softmax(scale * q K_S^T) V_S,  S = rows of the top blocks and the tail
//
// After a 512-frame video one token of the dense step reads 134 MB of keys and
// values per layer with 2 KV heads; here it reads 0.5 MB of codes and 4.2 MB of
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
//  3. the quarters of the chosen blocks and the tail's pieces go to the C * 8
//     warps in turn.  A warp attends over 16 rows on its own, while the next 32
//     are copied into its ring in shared memory; a lane's 16-byte loads are
//     matrix fragments as they are (the order of d inside a product is free),
//     the G <= 16 query rows are the 16 rows of m16n8k16, (m, l, O) stay in
//     registers;
//  4. the warps merge in shared memory and store each part of the result in
//     the CTA that writes it (distributed shared memory), which merges the CTAs.
// m16n8k16 and not tcgen05: with at most 16 query rows a 128-row product would
// waste 7/8 of the tensor core; it is busy for less than a fifth of the time.
// Scores, softmax statistics and O are fp32; P is rounded to bf16 for the
// product, l sums the unrounded P.
// Measured, 64 blocks a token: one token in one layer of 2 KV heads over 131072
// rows 14.7 us (initial loads 2.5, scores and exchange 1.7, selection 3,
// attention 4, merges 2); 16 ragged streams x 8 KV heads x 3 tokens, 0.82 GB of
// blocks counted per token, 114.5 us.  The rings are what counts there: with
// rows of 32 straight from global memory into registers, which leave no room
// for a second entry in flight, it was 147.
// One token in all 28 layers through a handle, rotation and summaries included:
// 43 us with 2 KV heads (56 items, clusters of 2), 127 us with 8 (224 items, no
// clusters); the bytes alone would take 20 and 79.
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
constexpr int kRows = 16;                // cache rows per entry of the attention
constexpr int kStages = 3;               // entries of a warp in shared memory

struct SparseKernelArgs {
    statekv_sparse_args a;
    float scale_log2;
    int32_t G, cluster;
    int32_t region;                  // bytes of shared memory used for the selection, the rows, the partials
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

// Exclusive prefix sum of one value per thread over the CTA.  One barrier; two
// scans in a row need scratch of their own.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (int w = 0; w < kSparseWarps - 1; ++w)
        if (w < warp) before += s_warp[w];
    return before + x - v;
}

// 8-bit codes of one block against the group's query codes: max over g.
template <int D>
__device__ __forceinline__ int best_dot(const uint4 (&w)[D / 16], const int8_t* s_q, int G) {
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
    return best;
}

template <int D>
__global__ void __launch_bounds__(kSparseThreads, 1) sparse_kernel(const __grid_constant__ SparseKernelArgs ka) {
    constexpr int KI = D / 32;               // 16-byte chunks of a K row per lane
    constexpr int DJ = D / 8;                // output columns per lane of a fragment's n index
    const statekv_sparse_args& a = ka.a;
    const int G = ka.G, C = ka.cluster;
    extern __shared__ __align__(16) uint8_t smem[];
    // region, one after the other: bins and scores; the warps' rows of K and V
    // [8][kStages][2][kRows][D]; the warps' O [8][G][D]
    uint32_t* s_bins = reinterpret_cast<uint32_t*>(smem);               // [2][kBins]
    uint32_t* s_key = s_bins + 2 * kBins;                               // [blocks]
    float* s_o = reinterpret_cast<float*>(smem);
    uint8_t* fixed = smem + ka.region;
    float* s_part = reinterpret_cast<float*>(fixed);                    // [C][slice] the CTAs' O of this CTA's slice
    float2* s_pml = reinterpret_cast<float2*>(s_part + 16 * D + 64);    // [16][16] the CTAs' (m, l)
    float2* s_wml = s_pml + 16 * 16;                                    // [8][16] the warps' (m, l)
    int* s_list = reinterpret_cast<int*>(s_wml + kSparseWarps * 16);    // [kMaxTop]
    int8_t* s_q = reinterpret_cast<int8_t*>(s_list + kMaxTop);          // [16][D] query codes
    uint32_t* s_scan = reinterpret_cast<uint32_t*>(s_q + 16 * D);       // [2][8]
    uint32_t* s_pick = s_scan + 2 * kSparseWarps;                       // [2][3] digit, keys above it, keys of it

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
    int nsel = nb;
    if (choose) {
        // the first block's codes are on their way while the query is rounded
        uint4 w[D / 16];
        float scale = 0.f;
        int b = rank * kSparseThreads + tid;
        auto load_codes = [&]() {
            const int64_t at = unit * a.blocks + b;
            const uint4* code = reinterpret_cast<const uint4*>(a.codes + at * D);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) w[i] = code[i];
            scale = a.scales[at];
        };
        if (b < a.blocks) load_codes();                      // (without waiting for the length)
        // G * D / 8 <= 256 threads have 8 values of the query each
        float x[8], top = 0.f;
        const bool has_q = tid < G * (D / 8);
        if (has_q) {
            const uint4 u = *reinterpret_cast<const uint4*>(q + (tid / (D / 8)) * a.q.head_stride + tid % (D / 8) * 8);
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(uw[i] << 16);
                x[2 * i + 1] = __uint_as_float(uw[i] & 0xffff0000u);
                top = fmaxf(top, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        if (lane == 0) s_scan[warp] = __float_as_uint(top);
        for (int i = tid; i < 2 * kBins; i += kSparseThreads) s_bins[i] = 0;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSparseWarps; ++i) top = fmaxf(top, __uint_as_float(s_scan[i]));
        const float up = code_range(top), inv = top > 0.f ? 127.f / (top * up) : 0.f;
        if (has_q) {
            uint32_t c[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int code = (int)fminf(fmaxf(rintf(x[i] * up * inv), -127.f), 127.f);
                c[i >> 2] |= (uint32_t)(code & 0xff) << (8 * (i & 3));
            }
            *reinterpret_cast<uint2*>(s_q + tid * 8) = make_uint2(c[0], c[1]);
        }
        __syncthreads();
        if (C > 1) ptx::cluster_wait();                      // every CTA has started: its memory may be written
        // ---- scores
        while (b < nb) {
            const uint32_t key = ordered((float)best_dot<D>(w, s_q, G) * scale);
            if (C == 1) s_key[b] = key;
            else
                for (int r = 0; r < C; ++r)
                    ptx::st_cluster_u32(ptx::cluster_map(ptx::smem_u32(s_key + b), (uint32_t)r), key);
            b += C * kSparseThreads;
            if (b < nb) load_codes();
        }
        if (C > 1) ptx::cluster_sync();
        else __syncthreads();
        // ---- the top-th largest key, digits of 11, 11 and 10 bits.  Often the
        // second digit's keys are all wanted: then no third pass is needed.
        uint32_t prefix = 0, mask = 0, need = (uint32_t)a.top;
        constexpr int PER = kBins / kSparseThreads;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t digits = pass == 2 ? 1023u : 2047u;
            uint32_t* bins = s_bins + (pass & 1) * kBins;
            for (int i = tid; i < nb; i += kSparseThreads) {
                const uint32_t key = s_key[i];
                if ((key & mask) == prefix) atomicAdd(&bins[(key >> shift) & digits], 1u);
            }
            __syncthreads();
            // thread t holds the 8 bins from 8 (255 - t) on: larger digits first
            static_assert(PER == 8, "two 16-byte loads");
            uint4* mine = reinterpret_cast<uint4*>(bins + (kSparseThreads - 1 - tid) * PER);
            const uint4 lo = mine[0], hi = mine[1];
            mine[0] = mine[1] = make_uint4(0, 0, 0, 0);      // for the pass after the next
            const uint32_t c[PER] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};
            const uint32_t sum = (c[0] + c[1]) + (c[2] + c[3]) + ((c[4] + c[5]) + (c[6] + c[7]));
            uint32_t above = block_scan(sum, s_scan + (pass & 1) * kSparseWarps);
            uint32_t* pick = s_pick + (pass & 1) * 3;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (above < need && need <= above + c[i]) {
                    pick[0] = (uint32_t)(kBins - 1 - (tid * PER + i));
                    pick[1] = above;
                    pick[2] = c[i];
                }
                above += c[i];
            }
            __syncthreads();
            prefix |= pick[0] << shift;
            mask |= digits << shift;
            need -= pick[1];
            if (pick[2] == need) break;                      // (the same in every thread)
        }
        // ---- in index order: keys above the threshold, and the first `need`
        // equal to it; a warp has consecutive blocks and counts by ballot
        const int per = (nb + 32 * kSparseWarps - 1) / (32 * kSparseWarps) * 32;
        const int b0 = min(nb, warp * per), b1 = min(nb, b0 + per);
        // both counts in one word: fewer than top <= 1024 keys are above, at
        // most 32768 equal
        uint32_t count = 0;
        for (int i = b0 + lane; i < b0 + per; i += 32) {
            const uint32_t key = i < b1 ? s_key[i] & mask : 0u;
            count += __popc(__ballot_sync(0xffffffffu, i < b1 && key > prefix)) << 16;
            count += __popc(__ballot_sync(0xffffffffu, i < b1 && key == prefix));
        }
        uint32_t* sums = s_scan + kSparseWarps;
        if (lane == 0) sums[warp] = count;
        __syncthreads();
        uint32_t at = 0;
#pragma unroll
        for (int w2 = 0; w2 < kSparseWarps - 1; ++w2)
            if (w2 < warp) at += sums[w2];
        for (int i = b0 + lane; i < b0 + per; i += 32) {
            const uint32_t key = i < b1 ? s_key[i] & mask : 0u;
            const unsigned gt = __ballot_sync(0xffffffffu, i < b1 && key > prefix);
            const unsigned eq = __ballot_sync(0xffffffffu, i < b1 && key == prefix);
            const unsigned below = (1u << lane) - 1u;
            const uint32_t n_gt = (at >> 16) + __popc(gt & below), n_eq = (at & 0xffffu) + __popc(eq & below);
            if (((gt >> lane) & 1u) || (((eq >> lane) & 1u) && n_eq < need)) s_list[n_gt + min(n_eq, need)] = i;
            at += (__popc(gt) << 16) + __popc(eq);
        }
        nsel = a.top;
        __syncthreads();                                     // the list is complete, the scores are read
    } else if (C > 1) {
        ptx::cluster_wait();
    }
    if (a.selected && rank == 0)
        for (int i = tid; i < a.top; i += kSparseThreads)
            a.selected[item * a.top + i] = i >= nsel || row < 0 ? -1 : choose ? s_list[i] : i;

    // ---- attention over entries of 16 rows: four of every block, then the tail's
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
    const int tail = row - nb * STATEKV_BLOCK + 1;           // rows since the last complete block
    constexpr int PER_BLOCK = STATEKV_BLOCK / kRows;
    const int of_blocks = PER_BLOCK * nsel, entries = row < 0 ? 0 : of_blocks + (max(tail, 0) + kRows - 1) / kRows;
    auto row_of = [&](int e) -> int {                        // first row of entry e
        return e < of_blocks
                   ? STATEKV_BLOCK * (choose ? s_list[e / PER_BLOCK] : e / PER_BLOCK) + kRows * (e % PER_BLOCK)
                   : STATEKV_BLOCK * nb + kRows * (e - of_blocks);
    };
    // Each warp has a ring of its own.  Its rows are copied asynchronously in
    // 16-byte units; a unit's place in its row is XOR-ed with bits of the row,
    // so that the 8 lanes of a quarter warp, which read units of 2 rows of K or
    // of 4 rows of V, meet no bank twice.
    constexpr int UPR = D / 8, TILE = kRows * D * 2;         // units of a row, bytes of K or V of an entry
    auto k_unit = [](int r, int u) { return u ^ ((r & 1) << 2); };
    auto v_unit = [](int r, int u) {
        const int y = (r >> 1) & 3;
        return u ^ (D == 128 ? (y & 1) | (y >> 1 << 2) : y << 1);
    };
    uint8_t* ring = smem + warp * (kStages * 2 * TILE);
    const uint32_t ring_u32 = ptx::smem_u32(ring);
    const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(a.k_cache.data) + n * a.k_cache.batch_stride +
                              h * a.k_cache.head_stride + lane % UPR * 8;
    const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(a.v_cache.data) + n * a.v_cache.batch_stride +
                              h * a.v_cache.head_stride + lane % UPR * 8;
    auto copy = [&](int e, int stage) {
        if (e < entries) {
            const int r0 = row_of(e), valid = row + 1 - r0;  // rows past the token's own may not exist: zeros
            const uint32_t at = ring_u32 + stage * 2 * TILE;
#pragma unroll
            for (int i = 0; i < kRows * UPR / 32; ++i) {
                const int r = (i * 32 + lane) / UPR, u = lane % UPR;
                const int64_t src = r0 + min(r, valid - 1);
                const uint32_t have = r < valid ? 16u : 0u;
                ptx::cp_async_16(at + r * (D * 2) + 16 * k_unit(r, u), kb + src * a.k_cache.token_stride, have);
                ptx::cp_async_16(at + TILE + r * (D * 2) + 16 * v_unit(r, u), vb + src * a.v_cache.token_stride, have);
            }
        }
        ptx::cp_async_commit();                              // (one group per entry, empty ones too)
    };
    const int step = kSparseWarps * C;
    int e = warp * C + rank, stage = 0;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) copy(e + i * step, i);
    for (; e < entries; e += step) {
        ptx::cp_async_wait_group<kStages - 2>();
        __syncwarp();                                        // every lane's copies; the stage before this one is read
        copy(e + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
        const uint8_t* kt = ring + stage * 2 * TILE;
        const uint8_t* vt = kt + TILE;
        stage = stage == kStages - 1 ? 0 : stage + 1;
        const int valid = row + 1 - row_of(e);               // at least kRows but in the tail
        float s[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
            const int r = 8 * t + g8;
#pragma unroll
            for (int i = 0; i < KI; ++i) {
                const uint4 kf = *reinterpret_cast<const uint4*>(kt + r * (D * 2) + 16 * k_unit(r, 4 * i + quad));
                mma16816(s[t], qf[2 * i], kf.x, kf.y);
                mma16816(s[t], qf[2 * i + 1], kf.z, kf.w);
            }
        }
        if (valid < kRows) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (8 * t + 2 * quad + (x & 1) >= valid) s[t][x] = -INFINITY;
        }
        float top[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            top[x] = fmaxf(fmaxf(s[0][2 * x], s[0][2 * x + 1]), fmaxf(s[1][2 * x], s[1][2 * x + 1]));
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
            top[x] = fmaxf(m[x], top[x] * ka.scale_log2);
        }
        if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const float f = m[x] == -INFINITY ? 0.f : ptx::ex2_approx(m[x] - top[x]);
                m[x] = top[x];
                l[x] *= f;
#pragma unroll
                for (int j = 0; j < DJ; ++j) {
                    o[j][2 * x] *= f;
                    o[j][2 * x + 1] *= f;
                }
            }
        }
        const float nm0 = m[0] == -INFINITY ? 0.f : -m[0], nm1 = m[1] == -INFINITY ? 0.f : -m[1];
        uint32_t p[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const float p0 = ptx::ex2_approx(fmaf(s[t][0], ka.scale_log2, nm0));
            const float p1 = ptx::ex2_approx(fmaf(s[t][1], ka.scale_log2, nm0));
            const float p2 = ptx::ex2_approx(fmaf(s[t][2], ka.scale_log2, nm1));
            const float p3 = ptx::ex2_approx(fmaf(s[t][3], ka.scale_log2, nm1));
            l[0] += p0 + p1;
            l[1] += p2 + p3;
            p[2 * t] = ptx::pack_bf16x2(p0, p1);
            p[2 * t + 1] = ptx::pack_bf16x2(p2, p3);
        }
        // V of keys {2 quad, 2 quad + 1} and 8 further, columns g8 * DJ ..
#pragma unroll
        for (int i = 0; i < DJ / 8; ++i) {
            uint32_t v[4][4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int r = 2 * quad + (y & 1) + 8 * (y >> 1);
                const uint4 x = *reinterpret_cast<const uint4*>(vt + r * (D * 2) + 16 * v_unit(r, g8 * (DJ / 8) + i));
                v[y][0] = x.x; v[y][1] = x.y; v[y][2] = x.z; v[y][3] = x.w;
            }
#pragma unroll
            for (int wd = 0; wd < 4; ++wd) {
                mma16816(o[8 * i + 2 * wd], p, __byte_perm(v[0][wd], v[1][wd], 0x5410),
                         __byte_perm(v[2][wd], v[3][wd], 0x5410));
                mma16816(o[8 * i + 2 * wd + 1], p, __byte_perm(v[0][wd], v[1][wd], 0x7632),
                         __byte_perm(v[2][wd], v[3][wd], 0x7632));
            }
        }
    }
    ptx::cp_async_wait_group<0>();
    __syncthreads();                                         // the rings become the warps' partials
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
    // ---- the CTA's warps, in order, 4 columns a thread; the result goes to
    // the CTA of the cluster that writes this part of the output
    const int slice = ((G * D + C - 1) / C + 3) / 4 * 4;
    for (int i = 4 * tid; i < G * D; i += 4 * kSparseThreads) {
        const int r = i / D;
        float mm = -INFINITY, ls = 0.f;
#pragma unroll
        for (int w = 0; w < kSparseWarps; ++w) mm = fmaxf(mm, s_wml[w * 16 + r].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kSparseWarps; ++w) {
            const float2 x = s_wml[w * 16 + r];
            const float4 y = *reinterpret_cast<const float4*>(s_o + w * G * D + i);
            const float f = x.x == -INFINITY ? 0.f : ptx::ex2_approx(x.x - mm);
            acc.x = fmaf(y.x, f, acc.x);
            acc.y = fmaf(y.y, f, acc.y);
            acc.z = fmaf(y.z, f, acc.z);
            acc.w = fmaf(y.w, f, acc.w);
            ls = fmaf(x.y, f, ls);
        }
        const int owner = i / slice;
        float* part = s_part + rank * slice + i - owner * slice;
        if (C == 1) *reinterpret_cast<float4*>(part) = acc;
        else ptx::st_cluster_f32x4(ptx::cluster_map(ptx::smem_u32(part), (uint32_t)owner), acc);
        if (i % D == 0) {
            if (C == 1) s_pml[r] = make_float2(mm, ls);
            else
                for (int c = 0; c < C; ++c)
                    ptx::st_cluster_f32x2(ptx::cluster_map(ptx::smem_u32(s_pml + rank * 16 + r), (uint32_t)c),
                                          make_float2(mm, ls));
        }
    }
    if (C > 1) ptx::cluster_sync();                          // the last access to another CTA's memory
    else __syncthreads();
    // ---- the CTAs, in rank order
    for (int i = 4 * tid; i < slice; i += 4 * kSparseThreads) {
        const int at = rank * slice + i, r = at / D;
        if (at >= G * D) break;
        float mm = -INFINITY, ls = 0.f;
        for (int c = 0; c < C; ++c) mm = fmaxf(mm, s_pml[c * 16 + r].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < C; ++c) {
            const float2 x = s_pml[c * 16 + r];
            const float4 y = *reinterpret_cast<const float4*>(s_part + c * slice + i);
            const float f = x.x == -INFINITY ? 0.f : ptx::ex2_approx(x.x - mm);
            acc.x = fmaf(y.x, f, acc.x);
            acc.y = fmaf(y.y, f, acc.y);
            acc.z = fmaf(y.z, f, acc.z);
            acc.w = fmaf(y.w, f, acc.w);
            ls = fmaf(x.y, f, ls);
        }
        const float inv = ls > 0.f || ls != ls ? 1.f / ls : 0.f;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + n * a.out.batch_stride +
                             (int64_t)(h * G + r) * a.out.head_stride + (int64_t)tok * a.out.token_stride + at % D;
        *reinterpret_cast<uint2*>(out) = make_uint2(ptx::pack_bf16x2(acc.x * inv, acc.y * inv),
                                                    ptx::pack_bf16x2(acc.z * inv, acc.w * inv));
    }
}

template <int D>
cudaLaunchConfig_t config(int64_t items, int cluster, size_t smem, cudaStream_t st, cudaLaunchAttribute (&attr)[1]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * cluster));
    cfg.blockDim = dim3(kSparseThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Clusters of 16 CTAs (more than the portable 8) that device dev holds at
// once, one CTA per SM; asked for once.
template <int D>
int clusters_of_16(int dev) {
    static std::atomic<int> cache[64];
    static std::atomic<uint64_t> known{0};
    if (dev < 0 || dev >= 64) return 0;
    if (known.load(std::memory_order_acquire) >> dev & 1ull) return cache[dev].load(std::memory_order_relaxed);
    int n = 0;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config<D>(1, 16, 227 * 1024, nullptr, attr);
    const void* f = reinterpret_cast<const void*>(&sparse_kernel<D>);
    if (cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, sparse_kernel<D>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
    }
    cache[dev].store(n, std::memory_order_relaxed);
    known.fetch_or(1ull << dev, std::memory_order_release);
    return n;
}

// CTAs per (batch entry, KV head, token): as many as keep the device in one
// wave, at most 16.  An SM takes in about 50 GB/s of scattered rows: the 4 MB
// of one token in one layer want as many SMs as there are.
template <int D>
int cluster_for(int64_t items, int sms, int dev) {
    if (items * 16 <= sms && items <= clusters_of_16<D>(dev)) return 16;
    int c = 8;
    while (c > 1 && items * c > sms) c /= 2;
    return c;
}

template <int D>
cudaError_t launch(SparseKernelArgs& ka, int64_t items, int dev, int sms, cudaStream_t st) {
    ka.cluster = cluster_for<D>(items, sms, dev);
    const size_t smem = ka.region + (16 * D + 64) * 4 + 16 * 16 * 8 + kSparseWarps * 16 * 8 + kMaxTop * 4 +
                        16 * D + (2 * kSparseWarps + 6) * 4;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&sparse_kernel<D>), 227 * 1024, dev, done);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config<D>(items, ka.cluster, smem, st, attr);
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
        !(a.scale > 1e-30) || !(a.scale < 1e30))
        return STATEKV_E_INVALID_ARG;
    if ((a.head_dim != 64 && a.head_dim != 128) || a.q_heads / a.kv_heads > 16 || a.top > kMaxTop ||
        a.cache_rows / STATEKV_BLOCK > kMaxBlocks)
        return STATEKV_E_UNSUPPORTED;
    const int64_t items = (int64_t)a.batch * a.kv_heads * a.tokens;
    if (items > 0x7fffffffll / 8) return STATEKV_E_UNSUPPORTED;
    if (!a.status || !ints_ok(a.status) || !ints_ok(a.lengths)) return STATEKV_E_INVALID_ARG;
    if (a.blocks < a.cache_rows / STATEKV_BLOCK || (!a.lengths && a.length > a.cache_rows)) return STATEKV_E_CAPACITY;
    if (items == 0) return STATEKV_OK;
    if (!view_ok(a.q, 2, a.batch, a.q_heads, a.tokens) || !view_ok(a.out, 2, a.batch, a.q_heads, a.tokens) ||
        !apart(a.out, a.batch, a.q_heads, a.tokens, a.head_dim) || reinterpret_cast<uintptr_t>(a.selected) % 4)
        return STATEKV_E_INVALID_ARG;
    if (a.cache_rows > 0 && (!view_ok(a.k_cache, 2, a.batch, a.kv_heads, a.cache_rows) ||
                             !view_ok(a.v_cache, 2, a.batch, a.kv_heads, a.cache_rows)))
        return STATEKV_E_INVALID_ARG;
    // the summaries are read only where there is something to choose
    const int most = (a.lengths ? a.cache_rows : a.length) / STATEKV_BLOCK;
    if (most > a.top && (!aligned16(a.codes) || !a.scales || reinterpret_cast<uintptr_t>(a.scales) % 4))
        return STATEKV_E_INVALID_ARG;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return view_cuda_fail();
    SparseKernelArgs k{};
    k.a = a;
    k.G = a.q_heads / a.kv_heads;
    k.scale_log2 = (float)(a.scale * 1.4426950408889634074);
    const int select = most > a.top ? 2 * kBins * 4 + (most * 4 + 15) / 16 * 16 : 0;
    const int rings = kSparseWarps * kStages * 2 * kRows * a.head_dim * 2;
    k.region = std::max({select, rings, kSparseWarps * k.G * a.head_dim * 4});
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = a.head_dim == 128 ? launch<128>(k, items, dev, sms, st) : launch<64>(k, items, dev, sms, st);
    return e == cudaSuccess ? STATEKV_OK : view_cuda_fail();
}
