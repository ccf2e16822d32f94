// What attention each cache row received from a chunk of tokens (tcgen05, TMA):
//
//   out[row] = before[row] + sum over the queries that see it of
//              exp(scale q . k - lse)
//
// The second half of an attention whose rows' log-sum-exps are known: scores
// again, but no product with V and, keys being the rows of the product
// S^T = K Q^T, no reduction across threads either.  Thread = key (TMEM lane): it
// adds its columns' exponentials in registers, block after block of queries, so
// each sum has a fixed order, and nothing is written but one number per row.
//
// Work: an item is 256 rows of one (batch entry, KV head), two 128-row tiles,
// each with a slot of four warps and two S buffers of its own.  Items are dealt
// to the CTAs in turn (one CTA per SM): ragged lengths and the causal triangle
// even out.  The item's queries stream through shared memory in blocks of
// floor(128 / G) tokens x G heads, one TMA box each, shared by both tiles.
//
// Bound: by HBM for a few tokens (K once, 256 bytes a row and 8 of weights), by
// the exponentials for a prompt (16384 per tile and block against 512 cycles of
// tensor work).
//
// Scores and sums in fp32.  Tokens behind the count, columns that no query has
// and queries that saw nothing are selected away, not added as zeros.
#include <algorithm>

#include "paged.cuh"
#include "pipeline.cuh"

namespace statekv {
namespace {

constexpr int kTile = 128;
constexpr int kItem = 2 * kTile;             // rows of an item
constexpr int kWeightThreads = 384;

struct WeightKernelArgs {
    statekv_attention_weights_args a;
    float scale_log2;
    int32_t G, tb;                           // query heads of a KV head, tokens of a query block
    int32_t cols, n;                         // queries of a block; columns of a product (a multiple of 16)
    int32_t box, page_boxes;                 // rows of a TMA box of K, boxes of a page
    int32_t capacity;
};

struct Seq {
    int len, count;                          // rows to weigh (0 where there is no token), new tokens
};
__device__ __forceinline__ Seq seq_of(const WeightKernelArgs& k, int s) {
    Seq q;
    q.len = cache_length(k.a.lengths, k.a.length, s, k.capacity, k.a.status);
    q.count = new_tokens(k.a.counts, k.a.tokens, s, q.len, k.a.status);
    if (q.count == 0) q.len = 0;
    return q;
}

// Walks the items of a CTA: blockIdx.x, + gridDim.x, ...
struct Walk {
    int64_t it, end;                         // the next item; items before the next sequence
    int s, per_head;                         // sequence, its items per KV head
    Seq q;
    int n, h, row0;                          // the current item
    int b0, blocks;                          // first query block that sees any row of it; their end
    __device__ void begin() {
        it = blockIdx.x;
        end = 0;
        s = -1;
        per_head = 0;
    }
    __device__ bool next(const WeightKernelArgs& k) {
        const int heads = k.a.layers * k.a.kv_heads;
        while (it >= end) {
            if (++s >= k.a.batch / k.a.layers) return false;
            q = seq_of(k, s);
            per_head = (q.len + kItem - 1) / kItem;
            end += (int64_t)per_head * heads;
        }
        const int local = (int)(it - (end - (int64_t)per_head * heads));
        const int nh = local / per_head;
        row0 = (local - nh * per_head) * kItem;
        n = s * k.a.layers + nh / k.a.kv_heads;
        h = nh % k.a.kv_heads;
        blocks = (q.count + k.tb - 1) / k.tb;
        b0 = max(0, row0 - (q.len - q.count)) / k.tb;
        it += gridDim.x;
        return true;
    }
};

template <int D>
struct WeightLayout {
    static constexpr int KCH = D / 64;
    static constexpr int CHUNK = 128 * 128;              // [128 rows][64 bf16], 128B-swizzled
    static constexpr int TILE = KCH * CHUNK;
    static constexpr int KS = D == 64 ? 6 : 4;           // tiles of K: two or three items
    static constexpr int QS = D == 64 ? 4 : 3;           // blocks of queries
    static constexpr int OFF_K = 0;
    static constexpr int OFF_Q = OFF_K + KS * TILE;
    static constexpr int OFF_LSE = OFF_Q + QS * TILE;    // [QS][128] log-sum-exps in log2 units
    static constexpr int OFF_TOK = OFF_LSE + QS * 512;   // [128] token of a column in its block (255: none)
    static constexpr int OFF_BAR = OFF_TOK + 128;
    static constexpr int B_K_FULL = 0;
    static constexpr int B_K_EMPTY = B_K_FULL + KS;
    static constexpr int B_Q_FULL = B_K_EMPTY + KS;
    static constexpr int B_L_FULL = B_Q_FULL + QS;       // log-sum-exps stored (1 warp)
    static constexpr int B_Q_EMPTY = B_L_FULL + QS;      // both products done, 8 warps done
    static constexpr int B_S_FULL = B_Q_EMPTY + QS;      // [2 slots][2 buffers]
    static constexpr int B_S_EMPTY = B_S_FULL + 4;       // (4 warps)
    static constexpr int B_DRAIN = B_S_EMPTY + 4;
    static constexpr int NBAR = B_DRAIN + 1;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // TMEM address, abort flag, [QS] a query saw nothing
    static constexpr int SMEM = OFF_MISC + 8 + QS * 4;
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
    static constexpr uint32_t TMEM_COLS = 512;
};

template <int D>
__global__ void __launch_bounds__(kWeightThreads, 1)
weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
               const __grid_constant__ WeightKernelArgs k) {
    using L = WeightLayout<D>;
    const statekv_attention_weights_args& a = k.a;
    extern __shared__ __align__(1024) uint8_t base[];
    const uint32_t sbase = ptx::smem_u32(base);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteDrain, sbase);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + L::OFF_MISC);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base + L::OFF_MISC + 4);
    uint32_t* blind = reinterpret_cast<uint32_t*>(base + L::OFF_MISC + 8);
    uint8_t* tok = base + L::OFF_TOK;
    Sync sy{sbase + (uint32_t)L::OFF_BAR, abort_flag, a.status};
    const uint32_t sK = sbase + L::OFF_K, sQ = sbase + L::OFF_Q;
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::KS; ++s) {
            ptx::mbar_init(sy.bar(L::B_K_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_K_EMPTY + s), 1);
        }
        for (int s = 0; s < L::QS; ++s) {
            ptx::mbar_init(sy.bar(L::B_Q_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_L_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_Q_EMPTY + s), 9);
        }
        for (int s = 0; s < 4; ++s) {
            ptx::mbar_init(sy.bar(L::B_S_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_S_EMPTY + s), 4);
        }
        ptx::mbar_init(sy.bar(L::B_DRAIN), 1);
        *abort_flag = 0u;
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), L::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    if (warp == 2)
        for (int i = lane; i < 128; i += 32) tok[i] = (uint8_t)(i < k.cols ? i % k.tb : 255);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Walk x;
    x.begin();
    if (warp == 0) {
        // ------------------------------------------------------------- K tiles
        // lane i holds the table entry of box i of the item (at most 16), and of
        // the item after it: read while this one's copies wait for room
        const int per_tile = kTile / k.box;
        auto entry = [&](const Walk& y) -> int {
            const int i = lane;
            if (i >= 2 * per_tile || y.row0 + i * k.box >= y.q.len) return -1;
            if (!a.table) return y.n;
            return a.table[(int64_t)y.n * a.table_stride + (y.row0 / k.box + i) / k.page_boxes];
        };
        int kt = 0;
        bool have = x.next(k);
        int e = have ? entry(x) : -1;
        for (bool ok = true; ok && have;) {
            const Walk cur = x;
            int page = e;
            if (lane < 2 * per_tile && cur.row0 + lane * k.box < cur.q.len && (uint32_t)page >= (uint32_t)a.num_pages) {
                record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSitePage, (uint32_t)page);
                page = -1;
            }
            have = x.next(k);
            if (have) e = entry(x);
            for (int t = 0; t < 2; ++t, ++kt) {
                const int s = kt % L::KS;
                if (!(ok = sy.wait(L::B_K_EMPTY + s, (uint32_t)((kt / L::KS) & 1) ^ 1u, kSiteKvEmpty))) break;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive_expect_tx(sy.bar(L::B_K_FULL + s), L::TILE);
                __syncwarp();
                const int i = lane / L::KCH, kc = lane % L::KCH;
                const int p = __shfl_sync(0xffffffffu, page, (t * per_tile + i) & 31);
                if (i < per_tile) {
                    const int bx = cur.row0 / k.box + t * per_tile + i;
                    const int row = p < 0 ? 0 : a.table ? (bx % k.page_boxes) * k.box : bx * k.box;
                    ptx::tma_load_4d(sK + s * L::TILE + kc * L::CHUNK + i * k.box * 128, &tm_k,
                                     sy.bar(L::B_K_FULL + s), kc * 64, row, cur.h, p);
                }
                __syncwarp();
            }
        }
        for (int s = 0; s < L::KS && s < kt; ++s)
            sy.drain(L::B_K_FULL + s, (uint32_t)(((kt - 1 - s) / L::KS) & 1));
    } else if (warp == 1) {
        // ----------------------------------------------------------- MMA issuer
        const uint32_t idesc = ptx::idesc_bf16_f32(128, 16, false, false) - (uint32_t)((16 >> 3) << 17) +
                               ((uint32_t)(k.n >> 3) << 17);
        const uint32_t hi = (uint32_t)(ptx::sdesc_sw128(0, 16, 1024) >> 32);
        const uint32_t kb0 = (uint32_t)ptx::sdesc_sw128(sK, 16, 1024);
        const uint32_t qb0 = (uint32_t)ptx::sdesc_sw128(sQ, 16, 1024);
        int kt = 0, qt = 0;
        bool ok = true;
        while (ok && x.next(k)) {
            for (int b = x.b0; ok && b < x.blocks; ++b, ++qt) {
                const int qs = qt % L::QS, buf = qt & 1;
                if (!(ok = sy.wait(L::B_Q_FULL + qs, (uint32_t)((qt / L::QS) & 1), kSiteQFull))) break;
                for (int slot = 0; ok && slot < 2; ++slot) {
                    const int ks = (kt + slot) % L::KS;
                    if (b == x.b0 &&
                        !(ok = sy.wait(L::B_K_FULL + ks, (uint32_t)(((kt + slot) / L::KS) & 1), kSiteKvFull)))
                        break;
                    if (!(ok = sy.wait(L::B_S_EMPTY + 2 * slot + buf, (uint32_t)((qt >> 1) & 1) ^ 1u, kSiteSEmpty)))
                        break;
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        const uint32_t kb = kb0 + (uint32_t)ks * (L::TILE >> 4), qb = qb0 + (uint32_t)qs * (L::TILE >> 4);
#pragma unroll
                        for (int kc = 0; kc < L::KCH; ++kc)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                ptx::umma_ss_lh(tmem + 256u * slot + 128u * buf, kb + kc * (L::CHUNK >> 4) + 2 * i, hi,
                                                qb + kc * (L::CHUNK >> 4) + 2 * i, hi, idesc, (kc | i) ? 1u : 0u);
                        ptx::umma_commit(sy.bar(L::B_S_FULL + 2 * slot + buf));
                        if (slot == 1) ptx::umma_commit(sy.bar(L::B_Q_EMPTY + qs));
                        if (b == x.blocks - 1) ptx::umma_commit(sy.bar(L::B_K_EMPTY + ks));
                    }
                    __syncwarp();
                }
            }
            kt += 2;
        }
        if (ptx::elect_one()) ptx::umma_commit(sy.bar(L::B_DRAIN));
        __syncwarp();
        sy.drain(L::B_DRAIN, 0);
    } else if (warp == 2) {
        // ----------------------------------------------- queries and their lse
        const uint32_t bytes = (uint32_t)k.cols * D * 2;
        int qt = 0;
        bool ok = true;
        while (ok && x.next(k)) {
            for (int b = x.b0; b < x.blocks; ++b, ++qt) {
                const int s = qt % L::QS;
                if (!(ok = sy.wait(L::B_Q_EMPTY + s, (uint32_t)((qt / L::QS) & 1) ^ 1u, kSiteKvEmpty))) break;
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive_expect_tx(sy.bar(L::B_Q_FULL + s), bytes);
#pragma unroll
                    for (int kc = 0; kc < L::KCH; ++kc)
                        ptx::tma_load_4d(sQ + s * L::TILE + kc * L::CHUNK, &tm_q, sy.bar(L::B_Q_FULL + s), kc * 64,
                                         b * k.tb, x.h * k.G, x.n);
                }
                float* lse2 = reinterpret_cast<float*>(base + L::OFF_LSE) + s * 128;
                bool none = false;
                for (int i = lane; i < k.cols; i += 32) {
                    const int g = i / k.tb, j = b * k.tb + tok[i];
                    float v = INFINITY;
                    if (j < x.q.count) {
                        v = a.lse[((int64_t)x.n * a.q_heads + x.h * k.G + g) * a.tokens + j] * 1.4426950408889634f;
                        if (v == -INFINITY) {
                            v = INFINITY;
                            none = true;
                        }
                    }
                    lse2[i] = v;
                }
                none = __any_sync(0xffffffffu, none);
                if (lane == 0) blind[s] = none;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sy.bar(L::B_L_FULL + s));
            }
        }
        for (int s = 0; s < L::QS && s < qt; ++s)
            sy.drain(L::B_Q_FULL + s, (uint32_t)(((qt - 1 - s) / L::QS) & 1));
    } else if (warp == 3) {
        // --------------------------------- rows that no query sees stay as before
        if (a.out != a.before) {
            const int units = a.batch * a.kv_heads;
            for (int u = blockIdx.x; u < units; u += gridDim.x) {
                const Seq q = seq_of(k, u / a.kv_heads / a.layers);
                const int64_t o = (int64_t)u * a.weight_rows;
#pragma unroll 8
                for (int i = q.len + lane; i < a.weight_rows; i += 32) a.out[o + i] = a.before ? a.before[o + i] : 0.f;
            }
        }
    } else {
        // --------------------------------------------------------- exponentials
        const int slot = (warp - 4) >> 2, q4 = warp & 3;
        const int lrow = q4 * 32 + lane;                         // key of the tile = TMEM lane
        const uint32_t t_s = tmem + 256u * slot + ((uint32_t)(q4 * 32) << 16);
        const float2 sc = make_float2(k.scale_log2, k.scale_log2);
        int qt = 0;
        bool ok = true;
        while (ok && x.next(k)) {
            const int row = x.row0 + slot * kTile + lrow;
            const int64_t at = ((int64_t)x.n * a.kv_heads + x.h) * a.weight_rows + row;
            const bool live = row < x.q.len;
            const float before = live && a.before ? a.before[at] : 0.f;
            const int first_new = x.q.len - x.q.count;
            float total = 0.f;
            for (int b = x.b0; b < x.blocks; ++b, ++qt) {
                const int s = qt % L::QS, buf = qt & 1;
                if (!(ok = sy.wait(L::B_L_FULL + s, (uint32_t)((qt / L::QS) & 1), kSiteQFull))) break;
                if (!(ok = sy.wait(L::B_S_FULL + 2 * slot + buf, (uint32_t)((qt >> 1) & 1), kSiteSFull))) break;
                __syncwarp();
                ptx::tc_fence_after();
                const float* lse2 = reinterpret_cast<const float*>(base + L::OFF_LSE) + s * 128;
                const int j0 = b * k.tb;
                // tokens of the block that see this row: from `from` to `upto`
                const int from = row - first_new - j0, upto = x.q.count - j0;
                const bool special = x.row0 + kItem > first_new + j0 + 1 || upto < k.tb || blind[s] != 0u;
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int c0 = 0; c0 < k.cols; c0 += 32) {
                    uint32_t v[32];
                    ptx::tmem_ld_32x32b_x32(t_s + 128u * buf + c0, v);
                    ptx::tmem_ld_wait();
                    if (special || c0 + 32 > k.cols) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int j = tok[c0 + e];
                            const float m = lse2[c0 + e];
                            const float y = ptx::ex2_approx(fmaf(__uint_as_float(v[e]), sc.x, -m));
                            if (c0 + e < k.cols && j >= from && j < upto && m != INFINITY) sum[e & 1].x += y;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 m = *reinterpret_cast<const float4*>(lse2 + c0 + e);
                            const float2 z0 = ptx::fma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sc,
                                                        make_float2(-m.x, -m.y));
                            const float2 z1 = ptx::fma2(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                                                        sc, make_float2(-m.z, -m.w));
                            sum[0] = ptx::add2(sum[0], make_float2(ptx::ex2_approx(z0.x), ptx::ex2_approx(z0.y)));
                            sum[1] = ptx::add2(sum[1], make_float2(ptx::ex2_approx(z1.x), ptx::ex2_approx(z1.y)));
                        }
                    }
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(sy.bar(L::B_S_EMPTY + 2 * slot + buf));
                    ptx::mbar_arrive(sy.bar(L::B_Q_EMPTY + s));
                }
                total += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            if (ok && live) a.out[at] = before + total;
        }
    }
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

template <int D>
cudaError_t launch_weights(const WeightKernelArgs& k, const CUtensorMap& mk, const CUtensorMap& mq, int dev, int grid,
                           cudaStream_t st) {
    using L = WeightLayout<D>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&weights_kernel<D>), L::SMEM, dev, done);
    if (e != cudaSuccess) return e;
    weights_kernel<D><<<(unsigned)grid, kWeightThreads, L::SMEM, st>>>(mk, mq, k);
    return cudaGetLastError();
}

}  // namespace
}  // namespace statekv

extern "C" int statekv_attention_weights(const statekv_attention_weights_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_attention_weights_args& a = *args;
    if (a.layers < 1 || a.batch < 0 || a.batch % a.layers != 0 || a.length < 0 || a.kv_heads < 1 ||
        a.q_heads < a.kv_heads || a.q_heads % a.kv_heads != 0 || a.tokens < 1 || a.weight_rows < 0 ||
        !(a.scale > 1e-30) || !(a.scale < 1e30))
        return STATEKV_E_INVALID_ARG;
    const int G = a.q_heads / a.kv_heads;
    if ((a.head_dim != 64 && a.head_dim != 128) || G > 64) return STATEKV_E_UNSUPPORTED;
    if (!a.status || !ints_ok(a.status) || !ints_ok(a.lengths) || !ints_ok(a.counts) || !ints_ok(a.lse) ||
        !ints_ok(a.before) || !ints_ok(a.out))
        return STATEKV_E_INVALID_ARG;
    const Paging pg = paging_of(a);
    int r = paging_ok(pg, a.batch);
    if (r != STATEKV_OK) return r;
    if (a.weight_rows < pg.capacity() || (!a.lengths && a.length > pg.capacity())) return STATEKV_E_CAPACITY;
    if (a.batch == 0 || a.weight_rows == 0) return STATEKV_OK;
    if (!a.lse || !a.out || !view_ok(a.q, 2, a.batch, a.q_heads, a.tokens) ||
        !spread(a.q, a.batch, a.q_heads, a.tokens))
        return STATEKV_E_INVALID_ARG;
    const bool cached = !paging_empty(pg);
    if (cached && (!view_ok(a.k_pages, 2, a.num_pages, a.kv_heads, a.page_rows) ||
                   !spread(a.k_pages, a.num_pages, a.kv_heads, a.page_rows)))
        return STATEKV_E_INVALID_ARG;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return view_cuda_fail();
    WeightKernelArgs k{};
    k.a = a;
    k.G = G;
    k.tb = std::min(kTile / G, a.tokens);
    k.cols = k.tb * G;
    k.n = (k.cols + 15) / 16 * 16;
    k.scale_log2 = (float)(a.scale * 1.4426950408889634074);
    k.capacity = cached ? (int)pg.capacity() : 0;
    k.box = kTile;
    if (a.table)
        while (a.page_rows % k.box != 0) k.box /= 2;
    k.page_boxes = a.table ? a.page_rows / k.box : 1;
    CUtensorMap mk{}, mq{};
    if (!encode_view4(&mq, a.q, a.head_dim, a.tokens, a.q_heads, a.batch, k.tb, G) ||
        (cached && !encode_view4(&mk, a.k_pages, a.head_dim, a.page_rows, a.kv_heads, a.num_pages, k.box)))
        return STATEKV_E_UNSUPPORTED;
    const int64_t most = a.lengths ? k.capacity : a.length;
    const int64_t items = (int64_t)a.batch * a.kv_heads * ((most + kItem - 1) / kItem);
    const int grid = (int)std::min<int64_t>(sms, std::max<int64_t>(items, (int64_t)a.batch * a.kv_heads));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = a.head_dim == 128 ? launch_weights<128>(k, mk, mq, dev, grid, st)
                                            : launch_weights<64>(k, mk, mq, dev, grid, st);
    return e == cudaSuccess ? STATEKV_OK : view_cuda_fail();
}
