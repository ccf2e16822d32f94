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
// each with a slot of warps, an issuer and two S buffers of its own.  Items are
// dealt to the CTAs in turn (one CTA per SM): ragged lengths and the causal
// triangle even out.  The item's queries stream through shared memory in blocks
// of floor(128 / G) tokens x G heads, one TMA box each, shared by both tiles.
//
// The log-sum-exp is part of the product: a ninth k-step multiplies a row of ones
// with -lse / scale in three bf16 terms (24 bits), so S comes out as q . k - lse /
// scale and a column costs one multiplication, one exponential and one addition.
// (Read from shared memory for each column a prompt took 246 us, and 212 after:
// the products take all of its bandwidth, 8 KB per 64 cycles.)
//
// Bound: by HBM for a few tokens (K once, 256 bytes a row and 8 of weights), by
// the exponentials (16384 per tile and block at 32 a cycle) and the tensor cores
// (576 cycles) for a prompt.
//
// Scores and sums in fp32.  In blocks with tokens behind the count, with queries
// that saw nothing, or over rows that not every token sees, columns are selected,
// by a mask of bits that each row makes once per block.
//
// Measured: one token for each of 16 ragged streams of up to 32768 rows, 8 KV
// heads, 0.545 GB: 100 us = 5.4 TB/s.  512 tokens over 131072 rows, 12 heads on 2:
// 185 us, 2000 cycles a block (the exponentials alone 1024, the products 1152
// beside them): the warps that add up take 1700 of them from scores to sums, and
// wait 200 for the next.
#include <algorithm>

#include "paged.cuh"
#include "pipeline.cuh"

namespace statekv {
namespace {

constexpr int kTile = 128;
constexpr int kItem = 2 * kTile;             // rows of an item
constexpr int kRest = 512;                   // rows of a piece of what is copied

struct WeightKernelArgs {
    statekv_attention_weights_args a;
    float scale_log2, minus_inv_scale;
    int32_t G, tb;                           // query heads of a KV head, tokens of a query block
    int32_t cols, n;                         // queries of a block; columns of a product (a multiple of 16)
    int32_t box, page_boxes;                 // rows of a TMA box of K, boxes of a page
    int32_t capacity;
};

// (no rows to weigh where there is no token)
__device__ __forceinline__ Seq seq_of(const WeightKernelArgs& k, int s) {
    Seq q = sequence_of(k.a, k.capacity, s);
    if (q.count == 0) q.len = 0;
    return q;
}

// Walks the items of a CTA: blockIdx.x, + gridDim.x, ...  Within a sequence the
// step is added as (entries, heads, items of a head), so that only a sequence's
// first item costs divisions (every role of the kernel takes every step).
struct Walk {
    int64_t it, end;                         // the next item; items before the next sequence
    int s, per_head;                         // sequence, its items per KV head
    int dn, dh, di;                          // the step
    Seq q;
    int n, h, i;                             // the current item: entry, head, place in the head
    int row0;
    int b0, blocks;                          // first query block that sees any row of it; their end
    __device__ void begin() {
        it = blockIdx.x;
        end = 0;
        s = -1;
    }
    __device__ bool next(const WeightKernelArgs& k) {
        if (it < end) {
            n += dn;
            h += dh;
            if ((i += di) >= per_head) {
                i -= per_head;
                ++h;
            }
            if (h >= k.a.kv_heads) {
                h -= k.a.kv_heads;
                ++n;
            }
        } else {
            const int heads = k.a.layers * k.a.kv_heads;
            do {
                if (++s >= k.a.batch / k.a.layers) return false;
                q = seq_of(k, s);
                per_head = (q.len + kItem - 1) / kItem;
                end += (int64_t)per_head * heads;
            } while (it >= end);
            const int local = (int)(it - (end - (int64_t)per_head * heads)), step = (int)gridDim.x;
            h = local / per_head;
            i = local - h * per_head;
            n = h / k.a.kv_heads;
            h -= n * k.a.kv_heads;
            n += s * k.a.layers;
            dh = step / per_head;
            di = step - dh * per_head;
            dn = dh / k.a.kv_heads;
            dh -= dn * k.a.kv_heads;
            blocks = (q.count + k.tb - 1) / k.tb;
        }
        row0 = i * kItem;
        const int past = row0 - (q.len - q.count);
        b0 = past > 0 ? past / k.tb : 0;
        it += gridDim.x;
        return true;
    }
};

// WIDE: more than 64 columns, in two halves of eight warps each.  Otherwise two
// warps copy the rows that no query sees while eight add up.
template <int D, bool WIDE>
struct WeightLayout {
    // warps: K of slot 0, issuer of slot 0, helper, issuer of slot 1; ADDERS that
    // add up; the copiers; then a second helper and K of slot 1
    static constexpr int ADDERS = WIDE ? 16 : 8;
    static constexpr int HELPER = 4 + ADDERS + (WIDE ? 0 : 2), LOADER = HELPER + 1;
    static constexpr int THREADS = (LOADER + 1) * 32;
    static constexpr int KCH = D / 64;
    static constexpr int CHUNK = 128 * 128;              // [128 rows][64 bf16], 128B-swizzled
    static constexpr int TILE = KCH * CHUNK;
    static constexpr int QCHUNK = WIDE ? CHUNK : CHUNK / 2;
    static constexpr int QTILE = KCH * QCHUNK;
    // Tiles of K (an item has two), and blocks of queries.  KS is even: each slot
    // has stages of its own.  Sharing them, an issuer two items ahead of the other
    // could wait for a phase after one that is not complete, and pass.
    static constexpr int KS = D == 64 ? 8 : 4;
    static constexpr int QS = 2;                         // a helper each
    static_assert(KS % 2 == 0, "stages per slot");
    static constexpr int OFF_K = 0;
    static constexpr int OFF_Q = OFF_K + KS * TILE;
    static constexpr int OFF_LSE = OFF_Q + QS * QTILE;   // [128 rows][4 slices of 16 bf16]: lse terms of QS blocks, 3 ones
    static constexpr int OFF_PART = OFF_LSE + CHUNK;     // [2 slots][128] sums of the second half of the columns
    static constexpr int OFF_BLIND = OFF_PART + (WIDE ? 1024 : 0);   // [8 blocks][4]: columns that saw nothing
    static constexpr int OFF_TOK = OFF_BLIND + 128;      // [128] token of a column in its block (255: none)
    static constexpr int OFF_BAR = OFF_TOK + 128;
    static constexpr int B_K_FULL = 0;
    static constexpr int B_K_EMPTY = B_K_FULL + KS;
    static constexpr int B_Q_FULL = B_K_EMPTY + KS;      // queries there, lse terms stored
    static constexpr int B_Q_EMPTY = B_Q_FULL + QS;      // products done (2 slots)
    static constexpr int B_S_FULL = B_Q_EMPTY + QS;      // [2 slots][2 buffers]
    static constexpr int B_S_EMPTY = B_S_FULL + 4;       // (the slot's warps)
    static constexpr int B_PART = B_S_EMPTY + 4;         // [2 slots] the second half's sums stored (4 warps)
    static constexpr int B_TAKEN = B_PART + 2;           // [2 slots] and taken (4 warps)
    static constexpr int B_DRAIN = B_TAKEN + 2;
    static constexpr int NBAR = B_DRAIN + 2;             // [2 slots]
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // TMEM address, abort flag, rest
    static constexpr int SMEM = OFF_MISC + 12;
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
    static constexpr uint32_t TMEM_COLS = 512;
};

template <int D, bool WIDE>
__global__ void __launch_bounds__((WeightLayout<D, WIDE>::THREADS), 1)
weights_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
               const __grid_constant__ WeightKernelArgs k) {
    using L = WeightLayout<D, WIDE>;
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
    uint32_t* rest = reinterpret_cast<uint32_t*>(base + L::OFF_MISC + 8);
    volatile uint32_t* blind = reinterpret_cast<volatile uint32_t*>(base + L::OFF_BLIND);
    uint8_t* tok = base + L::OFF_TOK;
    Sync sy{sbase + (uint32_t)L::OFF_BAR, abort_flag, a.status};
    const uint32_t sK = sbase + L::OFF_K, sQ = sbase + L::OFF_Q;
    constexpr bool split = WIDE;
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::KS; ++s) {
            ptx::mbar_init(sy.bar(L::B_K_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_K_EMPTY + s), 1);
        }
        for (int s = 0; s < L::QS; ++s) {
            ptx::mbar_init(sy.bar(L::B_Q_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_Q_EMPTY + s), 2);
        }
        for (int s = 0; s < 4; ++s) {
            ptx::mbar_init(sy.bar(L::B_S_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_S_EMPTY + s), WIDE ? 8 : 4);
            ptx::mbar_init(sy.bar(L::B_PART + s), 4);       // (and B_TAKEN)
        }
        ptx::mbar_init(sy.bar(L::B_DRAIN), 1);
        ptx::mbar_init(sy.bar(L::B_DRAIN + 1), 1);
        *abort_flag = 0u;
        *rest = 0u;
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), L::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    if (warp == 2)
        for (int i = lane; i < 128; i += 32) tok[i] = (uint8_t)(i < k.cols ? i % k.tb : 255);
    // Rows of Q that no query fills are zeros, columns that no query has get a
    // score of -2^127: both once and for all.
    for (int i = threadIdx.x; i < L::QS * L::QTILE / 16; i += L::THREADS)
        reinterpret_cast<uint4*>(base + L::OFF_Q)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = threadIdx.x; i < 128 * 8; i += L::THREADS) {
        const int r = i >> 3, e = i & 7;                         // 16-byte unit e of row r
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (e == 6) x = make_uint4(0x3f803f80u, 0x3f80u, 0u, 0u);            // 1, 1, 1
        else if (e % 2 == 0 && r >= k.cols) x.x = 0xff00u;                   // -2^127
        *reinterpret_cast<uint4*>(base + L::OFF_LSE + r * 128 + ((e ^ (r & 7)) << 4)) = x;
    }
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Walk x;
    x.begin();
    // Rows that no query sees stay as before.  One step copies the next kRest of
    // the CTA's; false: none left.  The copiers take them from the
    // start, the others what is left when they are done.
    const int pieces = a.out == a.before ? 0 : (int)(((int64_t)a.weight_rows + kRest - 1) / kRest);
    const int64_t all = (int64_t)a.batch * a.kv_heads * pieces;
    auto copy_step = [&]() -> bool {
        int64_t p = 0;
        if (lane == 0) p = (int64_t)atomicAdd(rest, 1u) * gridDim.x + blockIdx.x;
        p = __shfl_sync(0xffffffffu, p, 0);
        if (p >= all) return false;
        const int u = (int)(p / pieces), r0 = (int)(p - (int64_t)u * pieces) * kRest;
        const int r1 = a.weight_rows - r0 < kRest ? a.weight_rows : r0 + kRest;
        const int from = max(r0, seq_of(k, u / a.kv_heads / a.layers).len);
        const int64_t o = (int64_t)u * a.weight_rows;
        float v[kRest / 32];
#pragma unroll
        for (int e = 0; e < kRest / 32; ++e) {
            const int i = r0 + lane + 32 * e;
            v[e] = a.before && i >= from && i < r1 ? a.before[o + i] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < kRest / 32; ++e) {
            const int i = r0 + lane + 32 * e;
            if (i >= from && i < r1) a.out[o + i] = v[e];
        }
        return true;
    };
    if (warp == 0 || warp == L::LOADER) {
        // ------------------------------------------- K tiles of a slot (0, 1)
        // lane i / KCH copies 64 columns of box i / KCH of the tile; it holds the
        // box's table entry, and that of the next item's: read while this one's
        // copies wait for room
        const int slot = warp == 0 ? 0 : 1, per_tile = kTile / k.box, i = lane / L::KCH;
        const uint32_t dst = sK + (uint32_t)(lane % L::KCH) * L::CHUNK + (uint32_t)(i * k.box) * 128;
        auto entry = [&](const Walk& y) -> int {
            const int row = y.row0 + slot * kTile + i * k.box;
            if (i >= per_tile || row >= y.q.len) return -1;
            if (!a.table) return y.n;
            return a.table[(int64_t)y.n * a.table_stride + row / k.box / k.page_boxes];
        };
        int s = slot, loaded = 0;
        uint32_t par = 1;
        bool have = x.next(k);
        int e = have ? entry(x) : -1;
        while (have) {
            const int row = x.row0 + slot * kTile + i * k.box, h = x.h;
            int page = e;
            if (i < per_tile && row < x.q.len && (uint32_t)page >= (uint32_t)a.num_pages) {
                record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSitePage, (uint32_t)page);
                page = -1;
            }
            have = x.next(k);
            if (have) e = entry(x);
            if (!sy.wait(L::B_K_EMPTY + s, par, kSiteKvEmpty)) break;
            if (lane == 0) ptx::mbar_arrive_expect_tx(sy.bar(L::B_K_FULL + s), L::TILE);
            __syncwarp();
            if (i < per_tile)
                ptx::tma_load_4d(dst + s * L::TILE, &tm_k, sy.bar(L::B_K_FULL + s), lane % L::KCH * 64,
                                 page < 0 ? 0 : a.table ? row / k.box % k.page_boxes * k.box : row, h, page);
            __syncwarp();
            ++loaded;
            if ((s += 2) >= L::KS) {
                s = slot;
                par ^= 1u;
            }
        }
        // never leave a copy in flight into this CTA's shared memory
        constexpr int STAGES = L::KS / 2;
        for (int j = 0; j < STAGES && j < loaded; ++j)
            sy.drain(L::B_K_FULL + slot + 2 * j, (uint32_t)(((loaded - 1 - j) / STAGES) & 1));
    } else if (warp == 1 || warp == 3) {
        // ---------------------------------------------------------- MMA issuers
        // one per slot: an issuer shares its scheduler with five other warps and
        // takes about 800 cycles between two products, which is twice a product's time
        const int slot = warp >> 1;
        const uint32_t idesc = ptx::idesc_bf16_f32(128, 16, false, false) - (uint32_t)((16 >> 3) << 17) +
                               ((uint32_t)(k.n >> 3) << 17);
        const uint32_t hi = (uint32_t)(ptx::sdesc_sw128(0, 16, 1024) >> 32);
        const uint32_t kb0 = (uint32_t)ptx::sdesc_sw128(sK, 16, 1024);
        const uint32_t qb0 = (uint32_t)ptx::sdesc_sw128(sQ, 16, 1024);
        const uint32_t lb0 = (uint32_t)ptx::sdesc_sw128(sbase + L::OFF_LSE, 16, 1024);
        int ks = slot, qs = 0;
        uint32_t k_par = 0, q_par = 0, s_par = 1, buf = 0;
        bool ok = true;
        while (ok && x.next(k)) {
            if (!(ok = sy.wait(L::B_K_FULL + ks, k_par, kSiteKvFull))) break;
            const uint32_t kb = kb0 + (uint32_t)ks * (L::TILE >> 4);
            for (int left = x.blocks - x.b0; left > 0; --left) {
                if (!(ok = sy.wait(L::B_Q_FULL + qs, q_par, kSiteQFull))) break;
                if (!(ok = sy.wait(L::B_S_EMPTY + 2 * slot + (int)buf, s_par, kSiteSEmpty))) break;
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
                    const uint32_t qb = qb0 + (uint32_t)qs * (L::QTILE >> 4);
#pragma unroll
                    for (int kc = 0; kc < L::KCH; ++kc)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            ptx::umma_ss_lh(tmem + 256u * slot + 128u * buf, kb + kc * (L::CHUNK >> 4) + 2 * i, hi,
                                            qb + kc * (L::QCHUNK >> 4) + 2 * i, hi, idesc, (kc | i) ? 1u : 0u);
                    ptx::umma_ss_lh(tmem + 256u * slot + 128u * buf, lb0 + 6, hi, lb0 + 2 * qs, hi, idesc, 1u);
                    ptx::umma_commit(sy.bar(L::B_S_FULL + 2 * slot + (int)buf));
                    ptx::umma_commit(sy.bar(L::B_Q_EMPTY + qs));
                    if (left == 1) ptx::umma_commit(sy.bar(L::B_K_EMPTY + ks));
                }
                __syncwarp();
                s_par ^= buf;
                buf ^= 1u;
                if (++qs == L::QS) {
                    qs = 0;
                    q_par ^= 1u;
                }
            }
            if ((ks += 2) >= L::KS) {
                ks -= L::KS;
                k_par ^= 1u;
            }
        }
        if (ptx::elect_one()) ptx::umma_commit(sy.bar(L::B_DRAIN + slot));
        __syncwarp();
        sy.drain(L::B_DRAIN + slot, 0);
        while (copy_step()) {}
    } else if (warp == 2 || warp == L::HELPER) {
        // -------------------------------------------- queries and log-sum-exps
        // A block costs a warp 1700 cycles (the splitting, the stores, the latency
        // of the next block's values), so there are two, with a stage each.
        const int mine = warp == 2 ? 0 : 1;
        const uint32_t bytes = (uint32_t)k.cols * D * 2;
        int off[4];                                              // of this lane's columns in a block
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = lane + 32 * e;
            off[e] = i < k.cols ? i / k.tb * a.tokens + tok[i] : -1;
        }
        int b = 0, head = 0, n = 0, qt = 0;
        uint32_t q_par = 1;
        const float* src = nullptr;
        auto item = [&]() -> bool {
            if (!x.next(k)) return false;
            b = x.b0;
            head = x.h * k.G;
            n = x.n;
            src = a.lse + ((int64_t)n * a.q_heads + head) * a.tokens + b * k.tb;
            return true;
        };
        bool have = item();
        auto advance = [&](int count) {
            for (; have && count > 0; --count) {
                ++qt;
                src += k.tb;
                if (++b == x.blocks) have = item();
            }
        };
        advance(mine);
        auto read = [&](float (&v)[4]) {
            const int upto = x.q.count - b * k.tb;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = off[e] >= 0 && (upto >= k.tb || tok[lane + 32 * e] < upto) ? src[off[e]] : 0.f;
        };
        // one block: its log-sum-exps are in v, the next one's go to w
        auto step = [&](const float (&v)[4], float (&w)[4]) -> bool {
            const int at = qt, b_at = b, head_at = head, n_at = n;
            advance(L::QS);
            if (have) read(w);
            if (!sy.wait(L::B_Q_EMPTY + mine, q_par, kSiteKvEmpty)) return false;
            if (ptx::elect_one()) {
                ptx::mbar_expect_tx(sy.bar(L::B_Q_FULL + mine), bytes);
#pragma unroll
                for (int kc = 0; kc < L::KCH; ++kc)
                    ptx::tma_load_4d(sQ + mine * L::QTILE + kc * L::QCHUNK, &tm_q, sy.bar(L::B_Q_FULL + mine), kc * 64,
                                     b_at * k.tb, head_at, n_at);
            }
            __syncwarp();
            uint32_t none = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = lane + 32 * e;
                if (off[e] >= 0) {
                    // -lse / scale = hi + mid + lo
                    const float y = v[e] * k.minus_inv_scale;
                    const float hi = __bfloat162float(__float2bfloat16(y)), y1 = y - hi;
                    const float mid = __bfloat162float(__float2bfloat16(y1));
                    *reinterpret_cast<uint2*>(base + L::OFF_LSE + r * 128 + (((2 * mine) ^ (r & 7)) << 4)) =
                        make_uint2(ptx::pack_bf16x2(hi, mid), ptx::pack_bf16x2(y1 - mid, 0.f));
                }
                const uint32_t who = __ballot_sync(0xffffffffu, fabsf(v[e]) == INFINITY);
                if (lane == e) none = who;
            }
            if (lane < 4) blind[4 * (at & 7) + lane] = none;
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sy.bar(L::B_Q_FULL + mine));
            q_par ^= 1u;
            return have;
        };
        // (two sets by turns: moving one to the other would wait for its loads)
        float v[4], w[4];
        if (have) read(v);
        while (have && step(v, w) && step(w, v)) {}
        // never leave a copy in flight into this CTA's shared memory
        sy.drain(L::B_Q_FULL + mine, q_par);
        while (copy_step()) {}
    } else if (warp < 4 + L::ADDERS) {
        // --------------------------------------------------------- exponentials
        // slot and half of its columns
        const int slot = (warp >> 2) - 1 & 1, half = WIDE ? (warp - 4) >> 3 : 0, q4 = warp & 3;
        const int lrow = q4 * 32 + lane;                         // key of the tile = TMEM lane
        const uint32_t t_s = tmem + 256u * slot + ((uint32_t)(q4 * 32) << 16);
        const float sc = k.scale_log2;
        volatile float* part = reinterpret_cast<volatile float*>(base + L::OFF_PART) + slot * 128 + lrow;
        const int c_begin = 64 * half, c_end = split && half == 0 ? 64 : k.n;
        uint32_t s_par = 0, item = 0, buf = 0, qt = 0;
        bool ok = true;
        auto weight_at = [&](const Walk& y) -> int64_t {
            const int row = y.row0 + slot * kTile + lrow;
            return half == 0 && row < y.q.len ? ((int64_t)y.n * a.kv_heads + y.h) * a.weight_rows + row : -1;
        };
        // An item of few queries is a block or two: the next one's weights are on
        // their way while this one is added up.  (With many queries that costs more
        // registers than it saves: 225 us for a prompt where the kernel took 211 without.)
        Walk ahead = x;
        bool have = !WIDE && ok && ahead.next(k);
        int64_t at_next = have ? weight_at(ahead) : -1;
        float next = at_next >= 0 && a.before ? a.before[at_next] : 0.f;
        for (; ok && (WIDE ? x.next(k) : have); ++item) {
            int64_t at;
            float before;
            if constexpr (WIDE) {
                at = weight_at(x);
                before = at >= 0 && a.before ? a.before[at] : 0.f;
            } else {
                x = ahead;
                at = at_next;
                before = next;
                have = ahead.next(k);
                at_next = have ? weight_at(ahead) : -1;
                next = at_next >= 0 && a.before ? a.before[at_next] : 0.f;
            }
            const int row = x.row0 + slot * kTile + lrow;
            const int first_new = x.q.len - x.q.count;
            float total = 0.f;
            for (int b = x.b0; b < x.blocks; ++b) {
                if (!(ok = sy.wait(L::B_S_FULL + 2 * slot + (int)buf, s_par, kSiteSFull))) break;
                __syncwarp();
                ptx::tc_fence_after();
                const uint32_t t_b = t_s + 128u * buf;
                const int j0 = b * k.tb;
                // tokens of the block that see this row: from `from` to `upto`
                const int from = row - first_new - j0, upto = x.q.count - j0;
                volatile uint32_t* unseen = blind + 4 * (qt & 7);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                if (x.row0 + kItem > first_new + j0 + 1 || upto < k.tb ||
                    (unseen[0] | unseen[1] | unseen[2] | unseen[3]) != 0u) {
                    // the columns (from c_begin on) that count for this row
                    uint64_t seen = 0;
                    const int j_first = max(from, 0), count = min(upto, k.tb) - j_first;
                    for (int g = 0; g < k.G && count > 0; ++g) {
                        const int lo = max(g * k.tb + j_first - c_begin, 0);
                        const int hi = min(g * k.tb + j_first + count - c_begin, 64);
                        if (lo < hi) seen |= ~0ull >> (64 - (hi - lo)) << lo;
                    }
                    seen &= ~((uint64_t)unseen[2 * half + 1] << 32 | unseen[2 * half]);
#pragma unroll 1
                    for (int c = c_begin; c < c_end; c += 16, seen >>= 16) {
                        uint32_t v[16];
                        __syncwarp();
                        ptx::tmem_ld_32x32b_x16(t_b + c, v);
                        ptx::tmem_ld_wait();
                        const uint32_t now = (uint32_t)seen;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float y = ptx::ex2_approx(__uint_as_float(v[e]) * sc);
                            sum[e & 1].x += now & 1u << e ? y : 0.f;
                        }
                    }
                } else {
                    // the next 16 columns are on their way while these are added
                    uint32_t v[2][16];
                    ptx::tmem_ld_32x32b_x16(t_b + c_begin, v[0]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = c_begin + 16 * i;
                        if (c >= c_end) break;
                        ptx::tmem_ld_wait();
                        if (i < 3 && c + 16 < c_end) ptx::tmem_ld_32x32b_x16(t_b + c + 16, v[(i + 1) & 1]);
                        const uint32_t (&x16)[16] = v[i & 1];
#pragma unroll
                        for (int e = 0; e < 16; e += 2)
                            sum[(e >> 1) & 1] = ptx::add2(sum[(e >> 1) & 1],
                                                          make_float2(ptx::ex2_approx(__uint_as_float(x16[e]) * sc),
                                                                      ptx::ex2_approx(__uint_as_float(x16[e + 1]) * sc)));
                    }
                }
                total += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sy.bar(L::B_S_EMPTY + 2 * slot + (int)buf));
                s_par ^= buf;
                buf ^= 1u;
                ++qt;
            }
            if (ok && split) {
                // the second half's sum joins the first's
                if (half == 1) {
                    if (!(ok = sy.wait(L::B_TAKEN + slot, (item & 1u) ^ 1u, kSiteCol))) break;
                    *part = total;
                } else {
                    if (!(ok = sy.wait(L::B_PART + slot, item & 1u, kSiteCol))) break;
                    total += *part;
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sy.bar((half == 1 ? L::B_PART : L::B_TAKEN) + slot));
            }
            if (ok && at >= 0) a.out[at] = before + total;
        }
        while (copy_step()) {}
    } else {
        while (copy_step()) {}
    }
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

template <int D, bool WIDE>
cudaError_t launch_weights(const WeightKernelArgs& k, const CUtensorMap& mk, const CUtensorMap& mq, int dev, int grid,
                           cudaStream_t st) {
    using L = WeightLayout<D, WIDE>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(&weights_kernel<D, WIDE>), L::SMEM, dev, done);
    if (e != cudaSuccess) return e;
    weights_kernel<D, WIDE><<<(unsigned)grid, L::THREADS, L::SMEM, st>>>(mk, mq, k);
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
    // the attention's own limit (a group's log-sum-exps are counted in 32 bits)
    if ((int64_t)G * a.tokens >= 1 << 26) return STATEKV_E_UNSUPPORTED;
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
    const int64_t all = (int64_t)a.batch * a.kv_heads * a.weight_rows;
    if (a.before && a.before != a.out && overlap(a.before, all, a.out, all)) return STATEKV_E_INVALID_ARG;
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
    k.minus_inv_scale = (float)(-1.0 / a.scale);
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
    const bool wide = k.cols > 64;
    const cudaError_t e = a.head_dim == 128 ? wide ? launch_weights<128, true>(k, mk, mq, dev, grid, st)
                                                   : launch_weights<128, false>(k, mk, mq, dev, grid, st)
                          : wide            ? launch_weights<64, true>(k, mk, mq, dev, grid, st)
                                            : launch_weights<64, false>(k, mk, mq, dev, grid, st);
    return e == cudaSuccess ? STATEKV_OK : view_cuda_fail();
}
