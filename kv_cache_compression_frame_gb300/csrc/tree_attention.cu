// Attention of a tree of drafted tokens over a cache of keys and values
// (tcgen05, TMA): the verification step of speculative decoding.
//
//   o = softmax(scale * q [K_cache[:len]; K_new]^T, masked) [V_cache; V_new]
//
// Every drafted token sees the whole cache and, among the drafted ones, the
// nodes its mask names.  Per (batch entry, KV head) the R = G * tokens query
// rows share one pass over the cache, so the bound is HBM up to R ~ 256 (at
// 128 rows a 128-key tile is 64 KB of K and V, 2700 cycles of one SM's share
// of HBM, against ~1100 of tensor work and 1024 of exponentials).
//
// Work: a unit is one (batch entry, KV head, block of query rows); its key
// tiles are the cache's 128-row tiles and then one tile of drafted keys.  All
// units' tiles, end to end, are cut into equal contiguous shares, one per CTA
// (one CTA per SM), so ragged lengths balance by themselves and a CTA starts
// a new unit only a few times.  The piece of a unit in one CTA's share is a
// segment; with units in order, segment number = CTA + unit.  A segment that
// is the whole unit writes the output itself, the others leave (m, l, O) in
// the workspace and tree_combine_kernel merges them in CTA order (the same
// bits on every run).
//
// Inside a CTA two slots of four softmax warps each take turns: with at most
// 128 query rows a slot takes every second key tile of the one row tile
// (SPLIT_ROWS = false), otherwise each slot has its own 128-row tile and all
// key tiles.  A slot is one S buffer, one O accumulator and one running
// maximum and sum per row.  Thread = query row (TMEM lane): no reduction
// across threads.  A "job" is one S = Q K^T, softmax, O += P V of a slot; the
// issuer runs S two jobs ahead of P V, so one slot's exponentials overlap the
// other's products.  The next unit's first scores are computed while the last
// one's output is written; two otherwise idle warps copy its Q.
// P (bf16 pairs) overwrites its own S buffer: the products of one thread run
// in issue order, and S of a slot's next job is issued after P V of its last.
// That order also makes S(next) complete imply P V(last) complete, so a warp
// that raises its reference may rescale O right away.
//
// Precision: S, m, l and O in fp32; P is rounded to bf16 for the product (as
// the values V are), l sums the unrounded P.  A row's reference is raised
// only when a tile's maximum passes it by 2^8: P stays below 2^8 and keeps
// bf16's relative precision.
//
// Masked places may hold anything: scores are selected, not added to; V rows
// past the cache's end are zeroed in shared memory, and non-finite values of
// drafted V rows too (0 * NaN would reach rows that mask them) and put back
// at the end for the rows that see them.
//
// Measured: 16 ragged streams of up to 32768 rows, 64 query rows a unit, 1.15
// GB: 190 us = 6.0 TB/s (HBM).  28 layers x 131072 rows, 252 query rows a unit,
// 3.76 GB and 0.95 TFLOP: 690 us on a cool chip, 705-775 us under the power
// limit (1380 W, 1657 MHz), which is the bound there: variants that need fewer
// cycles per tile were not faster.
#include <algorithm>

#include "pipeline.cuh"
#include "views.cuh"

namespace statekv {
namespace {

constexpr int kTile = 128;                   // keys per tile, query rows per row tile
constexpr float kSlack = 8.f;                // raise the reference past 2^8
constexpr int kUnitCost = 6;                 // a unit's start and end in key tiles' time
constexpr int kWholeTiles = 8;               // key tiles up to which few units stay whole
constexpr int kMinShare = 4;                 // least share (in tiles' time) before more CTAs join
constexpr int kTreeThreads = 384;
// registers a thread after the split: 128 threads of the first warpgroup and
// 256 softmax threads, together the 168 x 384 of the launch
constexpr int kRegsIssue = 40, kRegsSoftmax = 232;
static_assert(kRegsIssue + 2 * kRegsSoftmax <= 3 * 168, "registers of the launch");

struct TreeKernelArgs {
    statekv_tree_args a;
    float* part_o;                           // [segments][d/4][rows][4]
    float2* part_ml;                         // [segments][rows] (reference, sum)
    float scale_log2;
    int32_t G, R, rb, rows;                  // rows: most rows of a unit
    uint32_t inv_tokens;                     // floor(2^32 / tokens) + 1
    int32_t grid;                            // CTAs of the main kernel
    int32_t whole;                           // a share is a unit: nothing to merge
    int32_t merge;                           // tree_combine_kernel follows
};

// r / tokens for a query row r < 65536: the high word of r * (2^32 / tokens,
// rounded up) is off by less than r / 2^32 < 1 / tokens, so exact
__device__ __forceinline__ int head_of(const TreeKernelArgs& k, int r) {
    return k.a.tokens == 1 ? r : (int)__umulhi((uint32_t)r, k.inv_tokens);
}

// The schedule, from the sequences' lengths.  A unit of nt key tiles counts as
// kUnitCost + nt tiles (it starts with kUnitCost of no content): without that
// a CTA whose share held many short units took 1.5 times as long as the rest.
struct Plan {
    uint32_t ctas, each, more;               // shares; tiles of a share, of the first `more` one more
    __device__ uint32_t start(uint32_t c) const { return each * c + min(c, more); }
    // the share that holds tile w
    __device__ uint32_t cta_of(uint32_t w) const {
        const uint32_t big = (each + 1) * more;
        return w < big ? w / (each + 1) : more + (w - big) / each;
    }
};

__device__ __forceinline__ int seq_length(const TreeKernelArgs& k, int s) {
    return cache_length(k.a.lengths, k.a.length, s, k.a.cache_rows, k.a.status);
}
// Key tiles of a unit: the cache's and the drafted one.
__device__ __forceinline__ int unit_tiles(int len) { return (len + kTile - 1) / kTile + 1; }
__device__ __forceinline__ int unit_cost(const TreeKernelArgs& k, int s) {
    return unit_tiles(seq_length(k, s)) + kUnitCost;
}

// Cost of one unit of every sequence before s, and of all sequences; a whole
// warp, the same result in every lane.  (Totals are below 2^31, see the entry
// point; 64-bit divisions by run-time values took 1 us of the prologue.)
__device__ __forceinline__ void sum_costs(const TreeKernelArgs& k, int s, uint32_t& before, uint32_t& all) {
    const int seqs = k.a.batch / k.a.layers;
    if (!k.a.lengths) {
        const uint32_t t = (uint32_t)unit_cost(k, 0);
        before = t * (uint32_t)s;
        all = t * (uint32_t)seqs;
        return;
    }
    before = all = 0;
    for (int i = threadIdx.x & 31; i < seqs; i += 32) {
        const uint32_t t = (uint32_t)unit_cost(k, i);
        all += t;
        if (i < s) before += t;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
}

__device__ __forceinline__ Plan make_plan(const TreeKernelArgs& k, uint32_t costs) {
    const uint32_t total = costs * (uint32_t)(k.a.layers * k.a.kv_heads * k.rb);
    Plan p;
    p.ctas = min((total + kMinShare - 1) / kMinShare, (uint32_t)k.grid);
    p.each = total / p.ctas;
    p.more = total - p.each * p.ctas;
    return p;
}

// Walks a share segment by segment.
struct Walk {
    int next_s, next_len, v;                 // the next segment's sequence, its length, place in the unit
    int next_u;
    int left;                                // of the share
    // the current segment: sequence, cache rows, key tiles of the unit, unit,
    // first key tile and number of them
    int s, len, nt, u, t, tiles;
    __device__ bool next(const TreeKernelArgs& k) {
        const int per_seq = k.a.layers * k.a.kv_heads * k.rb;
        while (left > 0) {
            s = next_s;
            len = next_len;
            nt = unit_tiles(len);
            u = next_u;
            const int take = min(nt + kUnitCost - v, left);
            t = max(v - kUnitCost, 0);
            tiles = max(v + take - kUnitCost, 0) - t;
            left -= take;
            v += take;
            if (v == nt + kUnitCost) {
                v = 0;
                ++next_u;
                if (next_u == (s + 1) * per_seq && s + 1 < k.a.batch / k.a.layers) next_len = seq_length(k, ++next_s);
            }
            if (tiles > 0) return true;
        }
        return false;
    }
};

// The walk of the share [w, w1) (a whole warp, the same result in every lane).
__device__ __forceinline__ Walk find(const TreeKernelArgs& k, uint32_t w, uint32_t w1) {
    const uint32_t per_seq = (uint32_t)(k.a.layers * k.a.kv_heads * k.rb);
    const int seqs = k.a.batch / k.a.layers;
    Walk c{};
    c.left = (int)(w1 - w);
    uint32_t cost;
    if (!k.a.lengths) {
        c.next_len = seq_length(k, 0);
        cost = (uint32_t)(unit_tiles(c.next_len) + kUnitCost);
        c.next_s = (int)(w / (cost * per_seq));
        w -= (uint32_t)c.next_s * (cost * per_seq);
    } else {
        const int lane = threadIdx.x & 31;
        uint32_t base = 0;
        for (int s0 = 0; s0 < seqs; s0 += 32) {
            const uint32_t mine = s0 + lane < seqs ? (uint32_t)unit_cost(k, s0 + lane) * per_seq : 0u;
            uint32_t upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + upto > w);
            if (hit) {
                const int l = __ffs((int)hit) - 1;
                c.next_s = s0 + l;
                base += __shfl_sync(0xffffffffu, upto - mine, l);
                break;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
        }
        w -= base;
        c.next_len = seq_length(k, c.next_s);
        cost = (uint32_t)(unit_tiles(c.next_len) + kUnitCost);
    }
    const uint32_t local = w / cost;
    c.next_u = (int)((uint32_t)c.next_s * per_seq + local);
    c.v = (int)(w - local * cost);
    return c;
}

template <int D, bool SPLIT_ROWS>
struct TreeLayout {
    static constexpr int KCH = D / 64;
    static constexpr int CHUNK = 128 * 128;              // [128 rows][64 bf16], 128B-swizzled
    static constexpr int TILE = KCH * CHUNK;
    static constexpr int RT = SPLIT_ROWS ? 2 : 1;        // row tiles
    // as many stages as fit beside Q
    static constexpr int KS = D == 64 ? 6 : 3;
    static constexpr int VS = D == 64 ? 5 : (SPLIT_ROWS ? 2 : 3);
    static constexpr int LEAD = SPLIT_ROWS ? 1 : 2;      // K tiles loaded ahead of V, as S runs ahead of P V
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = OFF_K + KS * TILE;
    static constexpr int OFF_Q = OFF_V + VS * TILE;      // [RT] row tiles
    static constexpr int OFF_BAR = OFF_Q + RT * TILE;
    static constexpr int B_K_FULL = 0;
    static constexpr int B_K_EMPTY = B_K_FULL + KS;
    static constexpr int B_V_FULL = B_K_EMPTY + KS;
    static constexpr int B_V_EMPTY = B_V_FULL + VS;
    static constexpr int B_Q_FULL = B_V_EMPTY + VS;      // Q of the segment stored (2 warps)
    static constexpr int B_Q_FREE = B_Q_FULL + 1;        // the segment's last S is done
    static constexpr int B_S_FULL = B_Q_FREE + 1;        // [2 slots]
    static constexpr int B_P_FULL = B_S_FULL + 2;        // [2 slots][2 halves of 64 keys] (4 warps)
    static constexpr int B_O_FULL = B_P_FULL + 4;        // the segment's products are done
    static constexpr int B_SYNC = B_O_FULL + 1;          // the 8 softmax warps
    static constexpr int B_DRAIN = B_SYNC + 1;
    static constexpr int NBAR = B_DRAIN + 1;
    static constexpr int OFF_ML = OFF_BAR + NBAR * 8;    // float2 [2 slots][128]: the slots' (m, l)
    static constexpr int OFF_MISC = OFF_ML + 2048;       // TMEM address, abort flag, odd nodes [2]
    static constexpr int SMEM = OFF_MISC + 24;
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
    static_assert(NBAR * 8 % 8 == 0 && OFF_MISC % 8 == 0, "the node mask is 8-byte aligned");
    static constexpr uint32_t TMEM_COLS = 512, TM_S = 0, TM_O = 256;
};

// bf16 pairs of a 32-bit word: a mask of the halves that are infinite or NaN
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
    return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <int D, bool SPLIT_ROWS>
__global__ void __launch_bounds__(kTreeThreads, 1)
tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
            const __grid_constant__ CUtensorMap tm_kn, const __grid_constant__ CUtensorMap tm_vn,
            const __grid_constant__ TreeKernelArgs k) {
    using L = TreeLayout<D, SPLIT_ROWS>;
    const statekv_tree_args& a = k.a;
    // the swizzled tiles need 1024-byte alignment; there is no room for slack
    extern __shared__ __align__(1024) uint8_t base[];
    const uint32_t sbase = ptx::smem_u32(base);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteDrain, sbase);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // every warp finds the CTA's share by itself
    const int c = (int)blockIdx.x;
    Walk first{};
    if (k.whole) {
        first.next_u = c;
        first.next_s = c / (a.layers * a.kv_heads * k.rb);
        first.next_len = seq_length(k, first.next_s);
        first.left = unit_tiles(first.next_len) + kUnitCost;
    } else {
        uint32_t none, costs;
        sum_costs(k, 0, none, costs);
        const Plan plan = make_plan(k, costs);
        if (c >= (int)plan.ctas) return;
        first = find(k, plan.start((uint32_t)c), plan.start((uint32_t)c + 1));
    }

    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + L::OFF_MISC);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base + L::OFF_MISC + 4);
    unsigned long long* odd_nodes = reinterpret_cast<unsigned long long*>(base + L::OFF_MISC + 8);
    Sync sy{sbase + (uint32_t)L::OFF_BAR, abort_flag, a.status};
    const uint32_t sK = sbase + L::OFF_K, sV = sbase + L::OFF_V, sQ = sbase + L::OFF_Q;
    // the next key tile of the share into its ring (thread 0); 1 loaded, 0 none
    // left, -1 gave up
    Walk wk = first, wv = first;
    int kt = 0, vt = 0;                                  // tiles loaded
    auto load = [&](bool is_v) -> int {
        Walk& x = is_v ? wv : wk;
        if (x.tiles == 0 && !x.next(k)) return 0;
        int& cnt = is_v ? vt : kt;
        const int ns = is_v ? L::VS : L::KS;
        const int s = cnt % ns, j = cnt / ns;
        if (!sy.wait((is_v ? L::B_V_EMPTY : L::B_K_EMPTY) + s, (uint32_t)(j & 1) ^ 1u, kSiteKvEmpty)) return -1;
        const uint32_t fb = sy.bar((is_v ? L::B_V_FULL : L::B_K_FULL) + s);
        ptx::mbar_arrive_expect_tx(fb, L::TILE);
        const uint32_t dst = (is_v ? sV : sK) + s * L::TILE;
        const bool drafted = x.t == x.nt - 1;
        const CUtensorMap* map = drafted ? (is_v ? &tm_vn : &tm_kn) : (is_v ? &tm_v : &tm_k);
        const int nh = x.u / k.rb, n = nh / a.kv_heads, h = nh - n * a.kv_heads;
#pragma unroll
        for (int kc = 0; kc < L::KCH; ++kc)
            ptx::tma_load_4d(dst + kc * L::CHUNK, map, fb, kc * 64, drafted ? 0 : x.t * kTile, h, n);
        ++cnt;
        ++x.t;
        --x.tiles;
        return 1;
    };
    // a unit's rows r = g * tokens + j of Q, zeros past the last, into shared
    // memory (warps 2 and 3, asynchronously)
    auto copy_q = [&](int u) {
        constexpr int UPR = D / 8;                       // 16-byte units per row
        constexpr int STEP = 64 / UPR;                   // rows at a time: 4 or 8
        const int qt = (int)threadIdx.x - 64, e = qt % UPR, r0 = qt / UPR;
        const int nh = u / k.rb, n = nh / a.kv_heads, h = nh - n * a.kv_heads;
        const int row_base = (u - nh * k.rb) * L::RT * kTile;
        int g = head_of(k, row_base + r0), j = row_base + r0 - g * a.tokens;
        const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.q.data) + n * a.q.batch_stride +
                                 (int64_t)(h * k.G + g) * a.q.head_stride + j * a.q.token_stride + 8 * e;
        const int64_t row = STEP * a.q.token_stride, wrap = a.q.head_stride - a.tokens * a.q.token_stride;
        const int left = k.R - row_base;
        const void* some = a.q.data;                     // (nothing is read for the zeros)
#pragma unroll 4
        for (int r = r0; r < L::RT * kTile; r += STEP) {
            ptx::cp_async_16(sQ + (r / kTile) * L::TILE + (e >> 3) * L::CHUNK + (r % kTile) * 128 +
                                 (((e & 7) ^ (r & 7)) << 4),
                             r < left ? static_cast<const void*>(p) : some, r < left ? 16u : 0u);
            p += row;
            for (j += STEP; j >= a.tokens; j -= a.tokens) p += wrap;
        }
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::KS; ++s) {
            ptx::mbar_init(sy.bar(L::B_K_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_K_EMPTY + s), 1);
        }
        for (int s = 0; s < L::VS; ++s) {
            ptx::mbar_init(sy.bar(L::B_V_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_V_EMPTY + s), 1);
        }
        ptx::mbar_init(sy.bar(L::B_Q_FULL), 2);
        ptx::mbar_init(sy.bar(L::B_Q_FREE), 1);
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(sy.bar(L::B_S_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_P_FULL + 2 * s), 4);
            ptx::mbar_init(sy.bar(L::B_P_FULL + 2 * s + 1), 4);
        }
        ptx::mbar_init(sy.bar(L::B_O_FULL), 1);
        ptx::mbar_init(sy.bar(L::B_SYNC), 8);
        ptx::mbar_init(sy.bar(L::B_DRAIN), 1);
        *abort_flag = 0u;
        odd_nodes[0] = odd_nodes[1] = 0ull;
        ptx::fence_barrier_init();
        // the first tiles are on their way while the rest is set up (the
        // stages are empty: no wait)
        static_assert(L::LEAD <= L::KS, "no wait before every barrier is visible");
        for (int t = 0; t < L::LEAD; ++t) load(false);
        load(true);
    }
    if (warp == 2 || warp == 3) {
        Walk x = first;
        if (x.next(k)) copy_q(x.u);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), L::TMEM_COLS);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The merge, where there is one, may be launched now; it waits for this
    // grid to end.  Otherwise the next kernel is not ours to release: it may
    // be one that starts early and relies on this grid's end (launch_rope
    // writes Q' and D rows at once), so it gets the implicit release there.
    if (k.merge) ptx::dep_trigger();
    if (warp < 4) {
        ptx::regs_dec<kRegsIssue>();
        if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            if (lane == 0) {
                for (int got = 1; got >= 0;) {
                    got = load(false);
                    if (got >= 0 && load(true) <= 0) break;
                }
                // never leave a copy in flight into this CTA's shared memory
                for (int s = 0; s < L::KS && s < kt; ++s)
                    sy.drain(L::B_K_FULL + s, (uint32_t)(((kt - 1 - s) / L::KS) & 1));
                for (int s = 0; s < L::VS && s < vt; ++s)
                    sy.drain(L::B_V_FULL + s, (uint32_t)(((vt - 1 - s) / L::VS) & 1));
            }
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issuer
            constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t idesc_o = ptx::idesc_bf16_f32(128, D, false, true);
            const uint32_t kmaj_hi = (uint32_t)(ptx::sdesc_sw128(0, 16, 1024) >> 32);
            const uint32_t v_hi = (uint32_t)(ptx::sdesc_sw128(0, L::CHUNK, 1024) >> 32);
            const uint32_t kb0 = (uint32_t)ptx::sdesc_sw128(sK, 16, 1024);
            const uint32_t qb0 = (uint32_t)ptx::sdesc_sw128(sQ, 16, 1024);
            const uint32_t vb0 = (uint32_t)ptx::sdesc_sw128(sV, L::CHUNK, 1024);
            Walk x = first;
            int g0 = 0, seg = 0;                             // tiles before this segment, segments done
            uint32_t p_par[2] = {0, 0};
            bool ok = true;
            auto issue_s = [&](int j, bool last) -> bool {
                const int slot = j & 1, g = g0 + (SPLIT_ROWS ? j >> 1 : j), s = g % L::KS;
                if (!sy.wait(L::B_K_FULL + s, (uint32_t)((g / L::KS) & 1), kSiteKvFull)) return false;
                ptx::tc_fence_after();
                if (ptx::elect_one()) {
                    const uint32_t kb = kb0 + (uint32_t)s * (L::TILE >> 4);
                    const uint32_t qb = qb0 + (SPLIT_ROWS ? (uint32_t)slot * (L::TILE >> 4) : 0u);
#pragma unroll
                    for (int kc = 0; kc < L::KCH; ++kc)
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            ptx::umma_ss_lh(tmem + L::TM_S + 128u * slot, qb + kc * (L::CHUNK >> 4) + 2 * ks, kmaj_hi,
                                            kb + kc * (L::CHUNK >> 4) + 2 * ks, kmaj_hi, idesc_s,
                                            (kc | ks) ? 1u : 0u);
                    ptx::umma_commit(sy.bar(L::B_S_FULL + slot));
                    if (!SPLIT_ROWS || slot == 1) ptx::umma_commit(sy.bar(L::B_K_EMPTY + s));
                    if (last) ptx::umma_commit(sy.bar(L::B_Q_FREE));
                }
                __syncwarp();
                return true;
            };
            auto issue_pv = [&](int j) -> bool {
                const int slot = j & 1, g = g0 + (SPLIT_ROWS ? j >> 1 : j), s = g % L::VS;
                if (!sy.wait(L::B_V_FULL + s, (uint32_t)((g / L::VS) & 1), kSiteKvFull)) return false;
                // the first 64 keys' products run while the other 64 are exponentiated
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    if (!sy.wait(L::B_P_FULL + 2 * slot + hf, p_par[slot], kSitePFull)) return false;
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        const uint32_t vb = vb0 + (uint32_t)s * (L::TILE >> 4);
#pragma unroll
                        for (int ks = 4 * hf; ks < 4 * hf + 4; ++ks)     // 16 keys per step
                            ptx::umma_ts_lh(tmem + L::TM_O + 128u * slot, tmem + L::TM_S + 128u * slot + 8u * ks,
                                            vb + 128u * ks, v_hi, idesc_o, (j > 1 || ks > 0) ? 1u : 0u);
                        if (hf == 1 && (!SPLIT_ROWS || slot == 1)) ptx::umma_commit(sy.bar(L::B_V_EMPTY + s));
                    }
                    __syncwarp();
                }
                p_par[slot] ^= 1u;
                return true;
            };
            for (; ok && x.next(k); ++seg) {
                const int jobs = SPLIT_ROWS ? 2 * x.tiles : x.tiles;
                if (!(ok = sy.wait(L::B_Q_FULL, (uint32_t)(seg & 1), kSiteQFull))) break;
                ptx::tc_fence_after();
                ok = issue_s(0, jobs == 1);
                if (ok && jobs > 1) ok = issue_s(1, jobs == 2);
                for (int j = 0; ok && j < jobs; ++j) {
                    ok = issue_pv(j);
                    if (ok && j + 2 < jobs) ok = issue_s(j + 2, j + 3 == jobs);
                }
                if (!ok) break;
                if (ptx::elect_one()) ptx::umma_commit(sy.bar(L::B_O_FULL));
                __syncwarp();
                g0 += x.tiles;
            }
            if (ptx::elect_one()) ptx::umma_commit(sy.bar(L::B_DRAIN));
            __syncwarp();
            sy.drain(L::B_DRAIN, 0);
        } else {
            // --------------------------------------------------------- Q copier
            // (warps 2 and 3) a unit's rows r = g * tokens + j, zeros past the
            // last, as soon as the unit before needs Q no more: its last softmax
            // and its output hide the copy
            Walk x = first;
            for (int seg = 0; x.next(k); ++seg) {
                if (seg > 0) {
                    if (!sy.wait(L::B_Q_FREE, (uint32_t)((seg - 1) & 1), kSiteQFull)) break;
                    copy_q(x.u);
                }
                ptx::cp_async_wait();
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sy.bar(L::B_Q_FULL));
            }
        }
    } else {
        // ------------------------------------------------ softmax / epilogue
        ptx::regs_inc<kRegsSoftmax>();
        const int tid = (int)threadIdx.x - 128;
        const int slot = tid >> 7, q4 = warp & 3;
        const int st = tid & 127;                                // thread of the slot
        const int lrow = q4 * 32 + lane;                         // row of the row tile = TMEM lane
        const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
        const uint32_t t_s = tmem + L::TM_S + 128u * slot + lane_base;
        const uint32_t t_o = tmem + L::TM_O + 128u * slot + lane_base;
        const float sc = k.scale_log2;
        int g0 = 0, seg = 0;
        uint32_t s_par = 0, sync_par = 0;
        bool ok = true;
        // barrier of the softmax warps (a bounded mbarrier wait: a warp that
        // gave up cannot leave the others blocked).  relaxed: it orders no
        // memory access.  An arrive with release semantics first waits for the
        // warp's global stores, 8 us behind the partials' stores while HBM was
        // saturated.
        auto sync_sm = [&](bool relaxed) -> bool {
            __syncwarp();
            if (lane == 0) {
                if (relaxed) ptx::mbar_arrive_relaxed(sy.bar(L::B_SYNC));
                else ptx::mbar_arrive(sy.bar(L::B_SYNC));
            }
            const bool r = sy.wait(L::B_SYNC, sync_par, kSiteCol);
            sync_par ^= 1u;
            return r;
        };
        Walk cu = first;
        for (; ok && cu.next(k); ++seg) {
            const int tiles = cu.tiles;
            const int nh = cu.u / k.rb, rblk = cu.u - nh * k.rb;
            const int n = nh / a.kv_heads, h = nh - n * a.kv_heads;
            const int row_base = rblk * L::RT * kTile;
            const int rows = min(L::RT * kTile, k.R - row_base); // rows of this unit
            // this thread's row of the unit (both slots' threads have the
            // same row where they share the row tile)
            const int r = (SPLIT_ROWS ? slot * kTile : 0) + lrow;
            const bool live = r < rows;
            const int gg = head_of(k, row_base + r);                 // of the head group
            const int node = live ? row_base + r - gg * a.tokens : 0;
            uint64_t sees = 0;
            if (live) sees = a.tree[(int64_t)cu.s * a.tree_stride + node];
            if (a.tokens < 64) sees &= (1ull << a.tokens) - 1ull;
            const bool idle = (SPLIT_ROWS ? slot * kTile : 0) + q4 * 32 >= rows;   // no row in this warp

            float m = -INFINITY, l = 0.f;                        // reference (log2 units) and sum
            const int jobs = SPLIT_ROWS ? tiles : (tiles - slot + 1) / 2;   // of this slot
            for (int i = 0; ok && i < jobs; ++i) {
                const int dt = SPLIT_ROWS ? i : 2 * i + slot;    // tile of the segment
                const int t = cu.t + dt;
                const bool drafted = t == cu.nt - 1;
                const int valid = drafted ? a.tokens : min(kTile, cu.len - t * kTile);
                if (!(ok = sy.wait(L::B_S_FULL + slot, s_par, kSiteSFull))) break;
                s_par ^= 1u;
                __syncwarp();
                ptx::tc_fence_after();
                const bool special = drafted || valid < kTile;
                if (special) {
                    // V rows whose products with P = 0 must be 0.  (After S
                    // full, which implies that the slot's last P V is done
                    // and with it the load before this one in V's stage: a
                    // wait for a phase before the last one ended would pass.)
                    const int g = g0 + dt, vs = g % L::VS;
                    if (!(ok = sy.wait(L::B_V_FULL + vs, (uint32_t)((g / L::VS) & 1), kSiteKvFull))) break;
                    uint8_t* vt = base + L::OFF_V + vs * L::TILE;
                    constexpr int UPR = D / 8;
                    if (drafted) {
                        // (rows past the drafted ones were filled with zeros)
                        for (int x = st; x < valid * UPR; x += 128) {
                            const int vr = x / UPR, e = x - vr * UPR;
                            uint4* p = reinterpret_cast<uint4*>(vt + (e >> 3) * L::CHUNK + vr * 128 +
                                                                (((e & 7) ^ (vr & 7)) << 4));
                            uint4 v = *p;
                            const uint32_t o0 = odd_halves(v.x), o1 = odd_halves(v.y), o2 = odd_halves(v.z),
                                           o3 = odd_halves(v.w);
                            if (o0 | o1 | o2 | o3) {
                                atomicOr(odd_nodes + (seg & 1), 1ull << vr);
                                __threadfence_block();
                                *p = make_uint4(v.x & ~o0, v.y & ~o1, v.z & ~o2, v.w & ~o3);
                            }
                        }
                    } else {
                        for (int x = valid * UPR + st; x < kTile * UPR; x += 128) {
                            const int vr = x / UPR, e = x - vr * UPR;
                            *reinterpret_cast<uint4*>(vt + (e >> 3) * L::CHUNK + vr * 128 +
                                                      (((e & 7) ^ (vr & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    ptx::fence_proxy_async_smem();
                }
                if (!idle) {
                    uint32_t x[2][64];
                    ptx::tmem_ld_32x32b_x64(t_s, x[0]);
                    ptx::tmem_ld_32x32b_x64(t_s + 64, x[1]);
                    ptx::tmem_ld_wait();
                    if (drafted) {
                        // node e of the tree is key e; no key past 63
#pragma unroll
                        for (int e = 0; e < 64; ++e) {
                            if (!((sees >> e) & 1ull)) x[0][e] = 0xff800000u;
                            x[1][e] = 0xff800000u;
                        }
                    } else if (valid < kTile) {
#pragma unroll
                        for (int e = 0; e < 64; ++e) {
                            if (e >= valid) x[0][e] = 0xff800000u;
                            if (64 + e >= valid) x[1][e] = 0xff800000u;
                        }
                    }
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 64; e += 2)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            mx[b] = ptx::max3(mx[b], __uint_as_float(x[b][e]), __uint_as_float(x[b][e + 1]));
                    const float top = fmaxf(mx[0], mx[1]) * sc;
                    const bool raise = top > m + kSlack;
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? ptx::ex2_approx(m - top) : 1.f;
                        if (raise) m = top;
                        l *= f;
                        __syncwarp();
                        // S full: every product into O so far is done
                        if (i > 0) {
#pragma unroll
                            for (int cc = 0; cc < D; cc += 32) {
                                uint32_t o[32];
                                ptx::tmem_ld_32x32b_x32(t_o + cc, o);
                                ptx::tmem_ld_wait();
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                ptx::tmem_st_32x32b_x32(t_o + cc, o);
                            }
                            ptx::tmem_st_wait();
                        }
                    }
                    const float nm = m == -INFINITY ? 0.f : -m;
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t p[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const float2 z = ptx::fma2(make_float2(__uint_as_float(x[hh][2 * e]),
                                                                   __uint_as_float(x[hh][2 * e + 1])),
                                                       make_float2(sc, sc), make_float2(nm, nm));
                            const float2 y = make_float2(ptx::ex2_approx(z.x), ptx::ex2_approx(z.y));
                            sum[e & 1] = ptx::add2(sum[e & 1], y);
                            p[e] = ptx::pack_bf16x2(y.x, y.y);
                        }
                        ptx::tmem_st_32x32b_x32(t_s + 32 * hh, p);
                        ptx::tmem_st_wait();
                        ptx::tc_fence_before();
                        __syncwarp();
                        // P itself is ordered by the tensor-memory wait and
                        // fence; only cleaned rows of V need a release
                        if (lane == 0) {
                            if (special) ptx::mbar_arrive(sy.bar(L::B_P_FULL + 2 * slot + hh));
                            else ptx::mbar_arrive_relaxed(sy.bar(L::B_P_FULL + 2 * slot + hh));
                        }
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                } else {
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(sy.bar(L::B_P_FULL + 2 * slot));
                        ptx::mbar_arrive(sy.bar(L::B_P_FULL + 2 * slot + 1));
                    }
                }
            }
            if (!ok) break;
            // ---- end of the segment
            if (!(ok = sy.wait(L::B_O_FULL, (uint32_t)(seg & 1), kSiteOFull))) break;
            ptx::tc_fence_after();
            // the slots that share a row tile tell each other (m, l)
            float2* ml = reinterpret_cast<float2*>(base + L::OFF_ML);
            if (!SPLIT_ROWS) ml[slot * kTile + lrow] = make_float2(m, l);
            // the next segment's mask (every read of it was before the last
            // segment's second sync, every write comes after the next one)
            if (tid == 0) odd_nodes[(seg + 1) & 1] = 0ull;
            ptx::tc_fence_before();
            if (!(ok = sync_sm(false))) break;
            const bool whole = cu.t == 0 && tiles == cu.nt;
            constexpr int COLS = SPLIT_ROWS ? D : D / 2;         // columns this thread merges
            const int c0 = SPLIT_ROWS ? 0 : slot * COLS;
            float f0 = 1.f, f1 = 0.f;
            bool use1 = false;
            uint32_t t_o0 = t_o;
            if (!SPLIT_ROWS) {
                const float2 x0 = ml[lrow], x1 = ml[kTile + lrow];
                use1 = tiles > 1;                                // slot 1 had a tile
                m = fmaxf(x0.x, use1 ? x1.x : -INFINITY);
                f0 = x0.x == -INFINITY ? 0.f : ptx::ex2_approx(x0.x - m);
                f1 = !use1 || x1.x == -INFINITY ? 0.f : ptx::ex2_approx(x1.x - m);
                l = x0.y * f0 + (use1 ? x1.y * f1 : 0.f);
                t_o0 = tmem + L::TM_O + lane_base + c0;
            }
            const uint64_t odd =
                live ? *reinterpret_cast<volatile unsigned long long*>(odd_nodes + (seg & 1)) & sees : 0ull;
            const int64_t sgm = (int64_t)c + cu.u;               // segment number
            const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
            if (!idle) {
#pragma unroll 1
                for (int cc = 0; cc < COLS; cc += 32) {
                    uint32_t o0[32], o1[32];
                    __syncwarp();
                    ptx::tmem_ld_32x32b_x32(t_o0 + cc, o0);
                    if (use1) ptx::tmem_ld_32x32b_x32(t_o0 + 128 + cc, o1);
                    ptx::tmem_ld_wait();
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        v[e] = __uint_as_float(o0[e]) * f0;
                        if (use1) v[e] = fmaf(__uint_as_float(o1[e]), f1, v[e]);
                    }
                    if (odd != 0ull) {
                        // infinities and NaN of the drafted rows that this row sees
                        for (uint64_t b = odd; b; b &= b - 1) {
                            const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(a.v_new.data) +
                                                      n * a.v_new.batch_stride + h * a.v_new.head_stride +
                                                      (int64_t)(__ffsll((long long)b) - 1) * a.v_new.token_stride;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float y = __bfloat162float(vr[c0 + cc + e]);
                                if (!(fabsf(y) < INFINITY)) v[e] += y;
                            }
                        }
                    }
                    if (live && whole) {
                        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + n * a.out.batch_stride +
                                             (int64_t)(h * k.G + gg) * a.out.head_stride +
                                             (int64_t)node * a.out.token_stride + c0 + cc;
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4*>(out + e) =
                                make_uint4(ptx::pack_bf16x2(v[e] * inv, v[e + 1] * inv),
                                           ptx::pack_bf16x2(v[e + 2] * inv, v[e + 3] * inv),
                                           ptx::pack_bf16x2(v[e + 4] * inv, v[e + 5] * inv),
                                           ptx::pack_bf16x2(v[e + 6] * inv, v[e + 7] * inv));
                    } else if (live) {
                        float4* po = reinterpret_cast<float4*>(k.part_o) +
                                     (sgm * (D / 4) + (c0 + cc) / 4) * k.rows + r;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            po[(int64_t)(e / 4) * k.rows] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                }
                if (live && !whole && c0 == 0) k.part_ml[sgm * k.rows + r] = make_float2(m, l);
            }
            ptx::tc_fence_before();
            // O and ml are read (the values are in registers): the next segment
            // may write them
            if (!(ok = sync_sm(true))) break;
            g0 += tiles;
        }
    }
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

// Merges the segments of a unit that several CTAs shared, in CTA order:
//   O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i
// Thread = 4 columns of a row, consecutive threads consecutive rows (how the
// partials lie).  Where a unit has many segments (one layer at 128 k rows: up
// to 76) kWays threads share an output, each taking every kWays-th segment;
// with up to kFew one thread takes them all and no barrier is needed.
constexpr int kMergeThreads = 256;
constexpr int kWays = 8, kFew = 8;

struct Merge {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // adds (m2, l2, o2)
    __device__ void add(float m2, float l2, float4 o2) {
        const float mn = fmaxf(m, m2);
        const float f = m == -INFINITY ? 0.f : ptx::ex2_approx(m - mn);
        const float g = m2 == -INFINITY ? 0.f : ptx::ex2_approx(m2 - mn);
        l = l * f + l2 * g;
        o.x = o.x * f + o2.x * g;
        o.y = o.y * f + o2.y * g;
        o.z = o.z * f + o2.z * g;
        o.w = o.w * f + o2.w * g;
        m = mn;
    }
};

template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_combine_kernel(const __grid_constant__ TreeKernelArgs k,
                                                                     int per_unit) {
    const statekv_tree_args& a = k.a;
    const int u = blockIdx.x / per_unit, part = blockIdx.x - u * per_unit;
    const int per_seq = a.layers * a.kv_heads * k.rb;
    const int s = u / per_seq;
    uint32_t before, all;
    sum_costs(k, s, before, all);
    const Plan plan = make_plan(k, all);
    const int nt = unit_tiles(seq_length(k, s));
    const uint32_t w = before * (uint32_t)per_seq + (uint32_t)((u - s * per_seq) * (nt + kUnitCost) + kUnitCost);
    const int ca = (int)plan.cta_of(w), segs = (int)plan.cta_of(w + (uint32_t)nt - 1) - ca + 1;
    // in every CTA, before it may leave: this grid must not end before the one
    // whose end it stands for, even where there is nothing to merge
    ptx::dep_wait();
    if (segs == 1) return;                   // written by the one CTA
    const int nh = u / k.rb, rblk = u - nh * k.rb;
    const int row_tile = k.R > kTile ? 2 * kTile : kTile;
    const int rows = min(row_tile, k.R - rblk * row_tile);
    const int n = nh / a.kv_heads, h = nh - n * a.kv_heads;
    const int outs = rows * (D / 4);
    const int ways = segs > kFew ? kWays : 1;
    const int per_step = kMergeThreads / ways, x = threadIdx.x % per_step, way = threadIdx.x / per_step;
    __shared__ Merge sh[kMergeThreads];
    const float2* ml0 = k.part_ml + ((int64_t)ca + u) * k.rows;
    const float4* po0 = reinterpret_cast<const float4*>(k.part_o) + ((int64_t)ca + u) * (D / 4) * k.rows;
    for (int out0 = part * per_step; out0 < outs; out0 += per_unit * per_step) {
        const int out = out0 + x, c4 = out / rows, r = out - c4 * rows;
        const bool live = out < outs;
        Merge acc;
        if (live) {
            constexpr int B = 4;
            for (int i0 = way; i0 < segs; i0 += B * ways) {
                float2 ml[B];
                float4 y[B];
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const int64_t i = i0 + b * ways;
                    ml[b] = make_float2(-INFINITY, 0.f);
                    y[b] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < segs) {
                        ml[b] = ml0[i * k.rows + r];
                        y[b] = po0[(i * (D / 4) + c4) * k.rows + r];
                    }
                }
#pragma unroll
                for (int b = 0; b < B; ++b) acc.add(ml[b].x, ml[b].y, y[b]);
            }
        }
        if (ways > 1) {
            __syncthreads();                 // the last step's entries are read
            sh[threadIdx.x] = acc;
            __syncthreads();
            if (way != 0) continue;
#pragma unroll 1
            for (int i = 1; i < kWays; ++i)
                acc.add(sh[i * per_step + x].m, sh[i * per_step + x].l, sh[i * per_step + x].o);
        }
        if (!live) continue;
        const float inv = acc.l > 0.f || acc.l != acc.l ? 1.f / acc.l : 0.f;
        const int row = rblk * row_tile + r, gg = head_of(k, row), j = row - gg * a.tokens;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out.data) + n * a.out.batch_stride +
                             (int64_t)(h * k.G + gg) * a.out.head_stride + (int64_t)j * a.out.token_stride + c4 * 4;
        *reinterpret_cast<uint2*>(dst) = make_uint2(ptx::pack_bf16x2(acc.o.x * inv, acc.o.y * inv),
                                                    ptx::pack_bf16x2(acc.o.z * inv, acc.o.w * inv));
    }
}

struct TreeMaps {
    CUtensorMap k, v, kn, vn;
};

template <int D, bool SPLIT_ROWS>
cudaError_t launch_main(const TreeKernelArgs& k, const TreeMaps& m, int dev, cudaStream_t st) {
    using L = TreeLayout<D, SPLIT_ROWS>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(reinterpret_cast<const void*>(&tree_kernel<D, SPLIT_ROWS>), L::SMEM, dev, done);
    if (e != cudaSuccess) return e;
    tree_kernel<D, SPLIT_ROWS><<<(unsigned)k.grid, kTreeThreads, L::SMEM, st>>>(m.k, m.v, m.kn, m.vn, k);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_combine(const TreeKernelArgs& k, int64_t units, int sms, cudaStream_t st) {
    // about eight CTAs per SM, but no more than there are steps of the
    // many-segment form
    const int64_t steps = (k.rows * (D / 4) + kMergeThreads / kWays - 1) / (kMergeThreads / kWays);
    const int64_t per_unit = std::min<int64_t>(steps, std::max<int64_t>(1, 8 * sms / units));
    if (units * per_unit > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * per_unit));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_combine_kernel<D>, k, (int)per_unit);
}

// Sizes that follow from the arguments; false where they are refused.
struct TreeSizes {
    int G, R, rb, rows;
    int64_t units;
};
int tree_sizes(int batch, int q_heads, int kv_heads, int tokens, int head_dim, TreeSizes* z) {
    if (batch < 0 || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0 || tokens < 1)
        return STATEKV_E_INVALID_ARG;
    if (tokens > 64 || (head_dim != 64 && head_dim != 128) || q_heads / kv_heads > 64) return STATEKV_E_UNSUPPORTED;
    z->G = q_heads / kv_heads;
    z->R = z->G * tokens;
    const int row_tile = z->R > kTile ? 2 * kTile : kTile;
    z->rb = (z->R + row_tile - 1) / row_tile;
    z->rows = std::min(z->R, row_tile);
    z->units = (int64_t)batch * kv_heads * z->rb;
    return z->units > 0x7fffffff / 1024 ? STATEKV_E_UNSUPPORTED : STATEKV_OK;
}

// A few short units are not cut: their 8 tiles one after the other take about
// as long as the second launch that would merge them (one layer, 300 rows:
// 12.1 us cut, 10.9 us whole, and one launch less on the host).
int64_t most_tiles(int64_t cache_rows) { return (cache_rows + kTile - 1) / kTile + 1; }
bool stays_whole(const TreeSizes& z, int64_t cache_rows, int sms) {
    return most_tiles(cache_rows) <= kWholeTiles && z.units <= sms;
}

int64_t workspace_for(const TreeSizes& z, int sms, int d) {
    // one segment per CTA and per unit; O, then (m, l)
    return ((int64_t)sms + z.units) * z.rows * (d * 4 + 8);
}

}  // namespace
}  // namespace statekv

extern "C" int64_t statekv_tree_attention_workspace(int32_t batch, int32_t q_heads, int32_t kv_heads,
                                                    int32_t tokens, int32_t head_dim, int32_t cache_rows) {
    using namespace statekv;
    TreeSizes z;
    if (cache_rows < 0) return -1;
    if (tree_sizes(batch, q_heads, kv_heads, tokens, head_dim, &z) != STATEKV_OK) return -1;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) {
        cudaGetLastError();
        return -1;
    }
    return stays_whole(z, cache_rows, sms) ? 0 : workspace_for(z, sms, head_dim);
}

extern "C" int statekv_tree_attention(const statekv_tree_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_tree_args& a = *args;
    if (a.layers < 1 || a.batch < 0 || a.batch % a.layers != 0 || a.cache_rows < 0 || a.length < 0 ||
        !rows_ok(a.tree_stride, a.tokens) || !(a.scale > 1e-30) || !(a.scale < 1e30))
        return STATEKV_E_INVALID_ARG;
    TreeSizes z;
    int r = tree_sizes(a.batch, a.q_heads, a.kv_heads, a.tokens, a.head_dim, &z);
    if (r != STATEKV_OK) return r;
    if (!a.status || !ints_ok(a.status) || !ints_ok(a.lengths)) return STATEKV_E_INVALID_ARG;
    if (!a.lengths && a.length > a.cache_rows) return STATEKV_E_CAPACITY;
    if (a.batch == 0) return STATEKV_OK;
    if (!a.tree || reinterpret_cast<uintptr_t>(a.tree) % 8 || !view_ok(a.q, 2, a.batch, a.q_heads, a.tokens) ||
        !view_ok(a.out, 2, a.batch, a.q_heads, a.tokens) || !view_ok(a.k_new, 2, a.batch, a.kv_heads, a.tokens) ||
        !view_ok(a.v_new, 2, a.batch, a.kv_heads, a.tokens))
        return STATEKV_E_INVALID_ARG;
    // an empty cache needs no memory: its maps are never read
    const bool cached = a.cache_rows > 0;
    if (cached && (!view_ok(a.k_cache, 2, a.batch, a.kv_heads, a.cache_rows) ||
                   !view_ok(a.v_cache, 2, a.batch, a.kv_heads, a.cache_rows)))
        return STATEKV_E_INVALID_ARG;
    // (entries of K and V that share their memory have no TMA view)
    if (!apart(a.out, a.batch, a.q_heads, a.tokens, a.head_dim) || !spread(a.k_new, a.batch, a.kv_heads, a.tokens) ||
        !spread(a.v_new, a.batch, a.kv_heads, a.tokens) ||
        (cached && (!spread(a.k_cache, a.batch, a.kv_heads, a.cache_rows) ||
                    !spread(a.v_cache, a.batch, a.kv_heads, a.cache_rows))))
        return STATEKV_E_INVALID_ARG;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return view_cuda_fail();
    const bool whole = stays_whole(z, a.cache_rows, sms);
    if (!whole && (!aligned16(a.workspace) || a.workspace_bytes < workspace_for(z, sms, a.head_dim)))
        return STATEKV_E_INVALID_ARG;
    TreeMaps m;
    if (!encode_view4(&m.kn, a.k_new, a.head_dim, a.tokens, a.kv_heads, a.batch) ||
        !encode_view4(&m.vn, a.v_new, a.head_dim, a.tokens, a.kv_heads, a.batch))
        return STATEKV_E_UNSUPPORTED;
    m.k = m.kn;
    m.v = m.vn;
    if (cached && (!encode_view4(&m.k, a.k_cache, a.head_dim, a.cache_rows, a.kv_heads, a.batch) ||
                   !encode_view4(&m.v, a.v_cache, a.head_dim, a.cache_rows, a.kv_heads, a.batch)))
        return STATEKV_E_UNSUPPORTED;
    TreeKernelArgs k{};
    k.a = a;
    k.G = z.G; k.R = z.R; k.rb = z.rb; k.rows = z.rows;
    k.inv_tokens = (uint32_t)((1ull << 32) / (uint32_t)a.tokens + 1);
    k.scale_log2 = (float)(a.scale * 1.4426950408889634074);
    // otherwise no more CTAs than the longest cache could use
    k.whole = whole;
    const int64_t cost = most_tiles(a.lengths ? a.cache_rows : a.length) + kUnitCost;
    if (z.units * cost > 0x7fffffff) return STATEKV_E_UNSUPPORTED;   // the schedule counts in 32 bits
    k.grid = whole ? (int)z.units : (int)std::min<int64_t>(sms, (z.units * cost + kMinShare - 1) / kMinShare);
    k.merge = !whole && k.grid > 1;          // one CTA holds whole units only
    const int64_t segments = (int64_t)sms + z.units;
    k.part_o = static_cast<float*>(a.workspace);
    k.part_ml = reinterpret_cast<float2*>(k.part_o + segments * z.rows * a.head_dim);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    const bool two = z.R > kTile;
    cudaError_t e = a.head_dim == 128 ? two ? launch_main<128, true>(k, m, dev, st) : launch_main<128, false>(k, m, dev, st)
                    : two             ? launch_main<64, true>(k, m, dev, st)
                                      : launch_main<64, false>(k, m, dev, st);
    if (e == cudaSuccess && k.merge)
        e = a.head_dim == 128 ? launch_combine<128>(k, z.units, sms, st) : launch_combine<64>(k, z.units, sms, st);
    return e == cudaSuccess ? STATEKV_OK : view_cuda_fail();
}
