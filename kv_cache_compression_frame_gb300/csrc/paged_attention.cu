// Attention of a chunk of new tokens over a paged cache (tcgen05, TMA): one
// token after a video, a text prompt, or a padded batch of either.
//
//   o = softmax(scale * q K^T, causal on the new rows) V,   lse = log sum exp
//
// Per (batch entry, KV head) the R = G * tokens query rows r = token * G + head
// of the group are cut into blocks of 128 or 256.  A block reads the rows up to
// its last token, so one token of any group and a prompt of up to 256 / G tokens
// read the cache once: the bound is HBM up to ~ 256 rows, the tensor cores (and
// the exponentials, which take as long) above.
//
// Work: a unit is one (batch entry, KV head, query block) with its 128-row key
// tiles.  All units' tiles, end to end, are cut into equal contiguous shares,
// one per CTA (one CTA per SM), so ragged lengths and the causal triangle
// balance by themselves.  The piece of a unit in one CTA's share is a segment.
// A segment that is the whole unit writes the output itself; a share's first
// and its last segment can be parts, which leave (m, l, O) in the CTA's two
// places of the workspace, and paged_combine_kernel merges them in CTA order
// (the same bits on every run).
//
// Inside a CTA two slots of four softmax warps each take turns: with at most
// 128 query rows a slot takes every second key tile of the one row tile
// (SPLIT_ROWS = false), otherwise each slot has its own 128-row tile and all
// key tiles.  A slot is one S buffer, one O accumulator and one running maximum
// and sum per row.  Thread = query row (TMEM lane): no reduction across threads.
// A "job" is one S = Q K^T, softmax, O += P V of a slot; the issuer runs S two
// jobs ahead of P V, so one slot's exponentials overlap the other's products.
// The next unit's first scores are computed while the last one's output is
// written; a warp copies its Q.  P (bf16 pairs) overwrites its own S buffer:
// the products of one thread run in issue order, and S of a slot's next job is
// issued after P V of its last.  That order also makes S(next) complete imply
// P V(last) complete, so a warp that raises its reference may rescale O right
// away.
//
// Pages: a tile is copied in boxes of the largest power of two of rows (16..128)
// that divides a page, so no box crosses a page's end.  K and V have a producer
// warp each (the same code, once in the instruction cache).  Each lane holds the
// page of one of the next 32 boxes and the table entry of one of the 32 after
// them: table reads are off the critical path but at a unit's start.  Boxes past
// the sequence's end are asked for at a page that does not exist, which TMA
// fills with zeros without reading anything.
//
// Precision: S, m, l and O in fp32; P is rounded to bf16 for the product (as
// the values V are), l sums the unrounded P.  A row's reference is raised only
// when a tile's maximum passes it by 2^8: P stays below 2^8 and keeps bf16's
// relative precision.
//
// Masked places may hold anything: scores are selected, not added to; V rows
// past the block's last visible row are zeroed in shared memory.  Values of new
// rows that some of the block's tokens do not see are zeroed where they are not
// finite (0 * NaN would reach the rows that mask them) and put back at the end
// for the rows that see them.
//
// Measured: one token for each of 16 ragged streams of up to 32768 rows, 8 KV
// heads, 1.06 GB: 169 us = 6.25 TB/s (HBM).  One token in one layer of 131073
// rows, 134 MB: 38.5 to 40 us, of which 8.5 pass before the first scores and 4 in
// the merge.  512 tokens over 131072 rows, 12 heads on 2, 0.41 TFLOP: 272 us = 1.52
// PFLOP/s, the tensor pipe 68 % busy: products alone keep it busy whatever
// their order, and beside all the copies and tensor-memory accesses of this
// kernel, but the warp that issues them does not get through its waits in time
// (each 85 to 130 cycles where nothing is left to wait for).
#include <algorithm>

#include "paged.cuh"
#include "pipeline.cuh"

namespace statekv {
namespace {

constexpr int kTile = 128;                   // keys per tile, query rows per row tile
constexpr float kSlack = 8.f;                // raise the reference past 2^8
constexpr int kUnitCost = 6;                 // a unit's start and end in key tiles' time
constexpr int kWholeTiles = 8;               // key tiles up to which few units stay whole
constexpr int kMinShare = 4;                 // least share (in tiles' time) before more CTAs join
constexpr int kPagedThreads = 384;

// new rows that not every token of a block sees: less than its tokens
constexpr int kOddWords = 2 * kTile / 32;

struct PagedKernelArgs {
    statekv_paged_attention_args a;
    float* part_o;                           // [2 * grid][d/4][rows][4]
    float2* part_ml;                         // [2 * grid][rows] (reference, sum)
    float scale_log2;
    int32_t G, R, rb, rows;                  // query rows, blocks of a KV head; most rows of a block
    int32_t block;                           // rows of a full block: 128 or 256
    uint32_t inv_group;                      // floor(2^32 / G) + 1
    int32_t box;                             // rows of a TMA box
    int32_t page_boxes;                      // boxes of a page
    int32_t capacity;                        // rows that a sequence can hold
    int32_t grid;                            // CTAs of the main kernel
    int32_t whole;                           // a share is a unit: nothing to merge
    int32_t merge;                           // paged_combine_kernel follows
};

// r / G for a row r < 2^26: the high word of r * (2^32 / G, rounded up) is off
// by less than r G / 2^32 / G < 1 / G, so exact
__device__ __forceinline__ int token_of(const PagedKernelArgs& k, int r) {
    return k.G == 1 ? r : (int)__umulhi((uint32_t)r, k.inv_group);
}

__device__ __forceinline__ Seq seq_of(const PagedKernelArgs& k, int s) { return sequence_of(k.a, k.capacity, s); }

// Cache rows that block b's last token sees (0: no token in it), and their tiles.
__device__ __forceinline__ int block_keys(const PagedKernelArgs& k, Seq q, int b) {
    if (token_of(k, b * k.block) >= q.count) return 0;
    const int last = token_of(k, min(k.R, (b + 1) * k.block) - 1);
    return q.len - q.count + min(q.count, last + 1);
}
__device__ __forceinline__ int block_tiles(const PagedKernelArgs& k, Seq q, int b) {
    return (block_keys(k, q, b) + kTile - 1) / kTile;
}

// The schedule.  A unit of nt key tiles counts as kUnitCost + nt tiles (it
// starts with kUnitCost of no content).  Units are ordered by sequence, then
// (layer, KV head), then block.
struct Plan {
    uint32_t ctas, each, more;               // shares; tiles of a share, of the first `more` one more
    __device__ uint32_t start(uint32_t c) const { return each * c + min(c, more); }
    // the share that holds tile w
    __device__ uint32_t cta_of(uint32_t w) const {
        const uint32_t big = (each + 1) * more;
        return w < big ? w / (each + 1) : more + (w - big) / each;
    }
};

__device__ __forceinline__ Plan plan_of(const PagedKernelArgs& k, uint32_t total) {
    Plan p;
    p.ctas = min((total + kMinShare - 1) / kMinShare, (uint32_t)k.grid);
    p.each = total / p.ctas;
    p.more = total - p.each * p.ctas;
    return p;
}

// Cost of one KV head's blocks in sequence s (a whole warp, the same result in
// every lane).
__device__ __forceinline__ uint32_t head_cost(const PagedKernelArgs& k, Seq q) {
    if (k.rb == 1) return (uint32_t)(block_tiles(k, q, 0) + kUnitCost);
    uint32_t sum = 0;
    for (int b = threadIdx.x & 31; b < k.rb; b += 32) sum += (uint32_t)(block_tiles(k, q, b) + kUnitCost);
    return __reduce_add_sync(0xffffffffu, sum);
}

__device__ __forceinline__ Plan make_plan(const PagedKernelArgs& k) {
    const int seqs = k.a.batch / k.a.layers;
    uint32_t total = 0;
    if (!k.a.lengths && !k.a.counts) {
        total = head_cost(k, seq_of(k, 0)) * (uint32_t)seqs;
    } else if (k.rb == 1) {
        for (int s = threadIdx.x & 31; s < seqs; s += 32)
            total += (uint32_t)(block_tiles(k, seq_of(k, s), 0) + kUnitCost);
        total = __reduce_add_sync(0xffffffffu, total);
    } else {
        for (int s = 0; s < seqs; ++s) total += head_cost(k, seq_of(k, s));
    }
    return plan_of(k, total * (uint32_t)(k.a.layers * k.a.kv_heads));
}

// A place in the schedule: unit (sequence s, batch entry n, KV head h, block b),
// and how far into its cost.
struct Place {
    int s, n, h, b, v;
    Seq q;
};

// The place of tile w (a whole warp, the same result in every lane).
__device__ __forceinline__ Place find(const PagedKernelArgs& k, uint32_t w) {
    const uint32_t heads = (uint32_t)(k.a.layers * k.a.kv_heads);
    const int seqs = k.a.batch / k.a.layers, lane = threadIdx.x & 31;
    Place p{};
    uint32_t cost;
    if (!k.a.lengths && !k.a.counts) {
        p.q = seq_of(k, 0);
        cost = head_cost(k, p.q);
        p.s = (int)(w / (cost * heads));
        w -= (uint32_t)p.s * (cost * heads);
    } else if (k.rb == 1) {
        uint32_t base = 0;
        for (int s0 = 0; s0 < seqs; s0 += 32) {
            const uint32_t mine =
                s0 + lane < seqs ? (uint32_t)(block_tiles(k, seq_of(k, s0 + lane), 0) + kUnitCost) * heads : 0u;
            uint32_t upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + upto > w);
            if (hit) {
                const int l = __ffs((int)hit) - 1;
                p.s = s0 + l;
                base += __shfl_sync(0xffffffffu, upto - mine, l);
                break;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
        }
        w -= base;
        p.q = seq_of(k, p.s);
        cost = (uint32_t)(block_tiles(k, p.q, 0) + kUnitCost);
    } else {
        for (;; ++p.s) {
            p.q = seq_of(k, p.s);
            cost = head_cost(k, p.q);
            if (w < cost * heads || p.s + 1 == seqs) break;
            w -= cost * heads;
        }
    }
    const int nh = (int)(w / cost);
    w -= (uint32_t)nh * cost;
    p.n = nh / k.a.kv_heads;
    p.h = nh - p.n * k.a.kv_heads;
    p.n += p.s * k.a.layers;
    if (k.rb > 1) {
        uint32_t base = 0;
        for (int b0 = 0; b0 < k.rb; b0 += 32) {
            const uint32_t mine = b0 + lane < k.rb ? (uint32_t)(block_tiles(k, p.q, b0 + lane) + kUnitCost) : 0u;
            uint32_t upto = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t x = __shfl_up_sync(0xffffffffu, upto, off);
                if (lane >= off) upto += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + upto > w);
            if (hit) {
                const int l = __ffs((int)hit) - 1;
                p.b = b0 + l;
                base += __shfl_sync(0xffffffffu, upto - mine, l);
                break;
            }
            base += __shfl_sync(0xffffffffu, upto, 31);
        }
        w -= base;
    }
    p.v = (int)w;
    return p;
}

// The schedule, and the place where CTA c's share starts (a whole warp, the same
// result in every lane).  The usual case, one block per head and up to 32
// sequences, takes one look at the lengths.
__device__ __forceinline__ Place schedule(const PagedKernelArgs& k, int c, Plan& plan) {
    const int seqs = k.a.batch / k.a.layers, lane = threadIdx.x & 31;
    Place p{};
    if (k.rb > 1 || seqs > 32) {
        plan = make_plan(k);
        if (c < (int)plan.ctas) p = find(k, plan.start((uint32_t)c));
        return p;
    }
    const uint32_t heads = (uint32_t)(k.a.layers * k.a.kv_heads);
    Seq q{0, 0};
    uint32_t cost = 0;
    if (lane < seqs) {
        q = seq_of(k, lane);
        cost = (uint32_t)(block_tiles(k, q, 0) + kUnitCost);
    }
    uint32_t upto = cost * heads;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += x;
    }
    plan = plan_of(k, __shfl_sync(0xffffffffu, upto, 31));
    if (c >= (int)plan.ctas) return p;
    uint32_t w = plan.start((uint32_t)c);
    p.s = __ffs((int)__ballot_sync(0xffffffffu, upto > w)) - 1;
    w -= __shfl_sync(0xffffffffu, upto - cost * heads, p.s);
    cost = __shfl_sync(0xffffffffu, cost, p.s);
    p.q.len = __shfl_sync(0xffffffffu, q.len, p.s);
    p.q.count = __shfl_sync(0xffffffffu, q.count, p.s);
    const int nh = (int)(w / cost);
    p.v = (int)(w - (uint32_t)nh * cost);
    p.n = nh / k.a.kv_heads;
    p.h = nh - p.n * k.a.kv_heads;
    p.n += p.s * k.a.layers;
    return p;
}

// Where the u-th unit starts in the schedule, and which it is.
__device__ __forceinline__ uint32_t unit_start(const PagedKernelArgs& k, int u, Place& p) {
    const int heads = k.a.layers * k.a.kv_heads, lane = threadIdx.x & 31;
    const int nh = u / k.rb;                 // over all sequences
    p.n = nh / k.a.kv_heads;
    p.h = nh - p.n * k.a.kv_heads;
    p.s = p.n / k.a.layers;
    p.b = u - nh * k.rb;
    p.q = seq_of(k, p.s);
    const uint32_t cost = head_cost(k, p.q);
    uint32_t w = (uint32_t)(nh - p.s * heads) * cost, before = 0;
    if (!k.a.lengths && !k.a.counts) {
        w += (uint32_t)(p.s * heads) * cost;
    } else if (k.rb == 1) {
        for (int s = lane; s < p.s; s += 32) before += (uint32_t)(block_tiles(k, seq_of(k, s), 0) + kUnitCost);
        w += __reduce_add_sync(0xffffffffu, before) * (uint32_t)heads;
    } else {
        for (int s = 0; s < p.s; ++s) before += head_cost(k, seq_of(k, s));
        w += before * (uint32_t)heads;
    }
    before = 0;
    for (int b = lane; b < p.b; b += 32) before += (uint32_t)(block_tiles(k, p.q, b) + kUnitCost);
    return w + __reduce_add_sync(0xffffffffu, before);
}

// Walks a share segment by segment.
struct Walk {
    Place at;                                // the next segment's
    int left;                                // of the share
    bool later;                              // a unit after the share's first
    // the current segment: batch entry, KV head, block, sequence's lengths, rows
    // its last token sees and their tiles, first key tile and number of them
    // (0: a block without tokens), place among the CTA's partial results
    int n, h, b, keys, nt, t, tiles, part;
    Seq q;
    __device__ bool next(const PagedKernelArgs& k) {
        while (left > 0) {
            n = at.n;
            h = at.h;
            b = at.b;
            q = at.q;
            keys = block_keys(k, q, b);
            nt = (keys + kTile - 1) / kTile;
            part = later ? 1 : 0;
            const bool begins = at.v == 0;
            const int take = min(nt + kUnitCost - at.v, left);
            t = max(at.v - kUnitCost, 0);
            tiles = max(at.v + take - kUnitCost, 0) - t;
            left -= take;
            at.v += take;
            if (at.v == nt + kUnitCost) {
                at.v = 0;
                later = true;
                if (++at.b == k.rb) {
                    at.b = 0;
                    if (++at.h == k.a.kv_heads) {
                        at.h = 0;
                        if (++at.n == (at.s + 1) * k.a.layers && at.n < k.a.batch) at.q = seq_of(k, ++at.s);
                    }
                }
            }
            if (tiles > 0 || (nt == 0 && begins)) return true;
        }
        return false;
    }
    // the next segment that has tiles
    __device__ bool next_tiles(const PagedKernelArgs& k) {
        while (next(k))
            if (tiles > 0) return true;
        return false;
    }
};

// Where the boxes of the walked tiles lie, 32 at a time, one per lane.
struct Boxes {
    int chunk, page, entry;                  // this lane's box of the chunk; its table entry of the next
    // this lane's box of a chunk: its entry in the table row, or -1 past the end
    static __device__ int raw(const PagedKernelArgs& k, const Walk& x, int chunk) {
        const int bx = chunk * 32 + (int)(threadIdx.x & 31);
        if ((int64_t)bx * k.box >= x.keys) return -1;
        if (!k.a.table) return x.n;
        return k.a.table[(int64_t)x.n * k.a.table_stride + bx / k.page_boxes];
    }
    static __device__ int checked(const PagedKernelArgs& k, const Walk& x, int chunk, int e) {
        const int bx = chunk * 32 + (int)(threadIdx.x & 31);
        if ((int64_t)bx * k.box >= x.keys) return -1;
        if ((uint32_t)e < (uint32_t)k.a.num_pages) return e;
        record_error(k.a.status, (uint32_t)STATEKV_E_DEVICE, kSitePage, (uint32_t)e);
        return -1;
    }
    __device__ void begin(const PagedKernelArgs& k, const Walk& x, int c) {
        chunk = c;
        page = checked(k, x, c, raw(k, x, c));
        entry = raw(k, x, c + 1);
    }
    __device__ void advance(const PagedKernelArgs& k, const Walk& x) {
        page = checked(k, x, ++chunk, entry);
        entry = raw(k, x, chunk + 1);
    }
};

template <int D, bool SPLIT_ROWS>
struct PagedLayout {
    // registers a thread after the split: 128 threads of the first warpgroup and
    // 256 softmax threads, together the 168 x 384 of the launch.  (Two row tiles'
    // softmax holds 128 scores.  Elsewhere 56 and 224 take 2 to 5 % longer.)
    static constexpr int REGS_ISSUE = SPLIT_ROWS ? 56 : 88, REGS_SOFTMAX = SPLIT_ROWS ? 224 : 208;
    static_assert(REGS_ISSUE + 2 * REGS_SOFTMAX <= 3 * 168, "registers of the launch");
    static constexpr int KCH = D / 64;
    static constexpr int CHUNK = 128 * 128;              // [128 rows][64 bf16], 128B-swizzled
    static constexpr int TILE = KCH * CHUNK;
    static constexpr int RT = SPLIT_ROWS ? 2 : 1;        // row tiles
    // as many stages as fit beside Q
    static constexpr int KS = D == 64 ? 6 : 3;
    static constexpr int VS = D == 64 ? 5 : (SPLIT_ROWS ? 2 : 3);
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = OFF_K + KS * TILE;
    static constexpr int OFF_Q = OFF_V + VS * TILE;      // [RT] row tiles
    static constexpr int OFF_BAR = OFF_Q + RT * TILE;
    static constexpr int B_K_FULL = 0;
    static constexpr int B_K_EMPTY = B_K_FULL + KS;
    static constexpr int B_V_FULL = B_K_EMPTY + KS;
    static constexpr int B_V_EMPTY = B_V_FULL + VS;
    static constexpr int B_Q_FULL = B_V_EMPTY + VS;      // Q of the segment stored
    static constexpr int B_Q_FREE = B_Q_FULL + 1;        // the segment's last S is done
    static constexpr int B_S_FULL = B_Q_FREE + 1;        // [2 slots]
    static constexpr int B_P_FULL = B_S_FULL + 2;        // [2 slots][2 halves of 64 keys] (4 warps)
    static constexpr int B_O_FULL = B_P_FULL + 4;        // the segment's products are done
    static constexpr int B_SYNC = B_O_FULL + 1;          // the 8 softmax warps
    static constexpr int B_DRAIN = B_SYNC + 1;
    static constexpr int NBAR = B_DRAIN + 1;
    static constexpr int OFF_ML = OFF_BAR + NBAR * 8;    // float2 [2 slots][128]: the slots' (m, l)
    static constexpr int OFF_MISC = OFF_ML + 2048;       // TMEM address, abort flag
    static constexpr int OFF_ODD = OFF_MISC + 8;         // [2][kOddWords]: new rows that are not finite
    static constexpr int SMEM = OFF_ODD + 2 * kOddWords * 4;
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
    static constexpr uint32_t TMEM_COLS = 512, TM_S = 0, TM_O = 256;
};

// bf16 pairs of a 32-bit word: a mask of the halves that are infinite or NaN
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
    return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

template <int D, bool SPLIT_ROWS>
__global__ void __launch_bounds__(kPagedThreads, 1)
paged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
             const __grid_constant__ PagedKernelArgs k) {
    using L = PagedLayout<D, SPLIT_ROWS>;
    const statekv_paged_attention_args& a = k.a;
    // the swizzled tiles need 1024-byte alignment; there is no room for slack
    extern __shared__ __align__(1024) uint8_t base[];
    const uint32_t sbase = ptx::smem_u32(base);
    if (sbase & 1023u) {
        if (threadIdx.x == 0) record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteDrain, sbase);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + L::OFF_MISC);
    volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(base + L::OFF_MISC + 4);
    uint32_t* odd_rows = reinterpret_cast<uint32_t*>(base + L::OFF_ODD);
    Sync sy{sbase + (uint32_t)L::OFF_BAR, abort_flag, a.status};
    const uint32_t sK = sbase + L::OFF_K, sV = sbase + L::OFF_V, sQ = sbase + L::OFF_Q;
    // Nothing but barriers and tensor memory is set up together; every warp then
    // finds the CTA's share by itself and starts, the producers with the first loads.
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::KS; ++s) {
            ptx::mbar_init(sy.bar(L::B_K_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_K_EMPTY + s), 1);
        }
        for (int s = 0; s < L::VS; ++s) {
            ptx::mbar_init(sy.bar(L::B_V_FULL + s), 1);
            ptx::mbar_init(sy.bar(L::B_V_EMPTY + s), 1);
        }
        ptx::mbar_init(sy.bar(L::B_Q_FULL), 1);
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
        for (int i = 0; i < 2 * kOddWords; ++i) odd_rows[i] = 0u;
        ptx::fence_barrier_init();
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
    // grid to end.  Otherwise the next kernel is not ours to release: it gets
    // the implicit release at this grid's end.
    if (k.merge) ptx::dep_trigger();
    const int c = (int)blockIdx.x;
    Walk first{};                            // (no share: nothing left)
    if (k.whole) {
        const int per_seq = a.layers * a.kv_heads * k.rb;
        first.at.s = c / per_seq;
        const int nh = c / k.rb;
        first.at.n = nh / a.kv_heads;
        first.at.h = nh - first.at.n * a.kv_heads;
        first.at.b = c - nh * k.rb;
        first.at.q = seq_of(k, first.at.s);
        first.left = block_tiles(k, first.at.q, first.at.b) + kUnitCost;
    } else {
        Plan plan;
        first.at = schedule(k, c, plan);
        if (c < (int)plan.ctas) first.left = (int)(plan.start((uint32_t)c + 1) - plan.start((uint32_t)c));
    }
    if (warp < 4) {
        ptx::regs_dec<L::REGS_ISSUE>();
        if (warp == 0 || warp == 3) {
            // ------------------------------------- TMA producers: K (0) and V (3)
            const bool is_v = warp == 3;
            const CUtensorMap* map = is_v ? &tm_v : &tm_k;
            const uint32_t dst = (is_v ? sV : sK) + (uint32_t)(lane % L::KCH) * L::CHUNK +
                                 (uint32_t)(lane / L::KCH * k.box) * 128;
            const int full = is_v ? L::B_V_FULL : L::B_K_FULL, empty = is_v ? L::B_V_EMPTY : L::B_K_EMPTY;
            const int stages = is_v ? L::VS : L::KS;
            const int per_tile = kTile / k.box, column = lane % L::KCH * 64, mine = lane / L::KCH;
            Walk x = first;
            Boxes bo{};
            int s = 0, loaded = 0;
            uint32_t par = 1;
            bool ok = true;
            while (ok && x.next_tiles(k)) {
                bo.begin(k, x, x.t * per_tile / 32);
                int bx = x.t * per_tile + mine;                  // this lane's box (lanes past the tile's: none)
                int in_page = a.table ? bx % k.page_boxes : bx;
                for (; x.tiles > 0; --x.tiles) {
                    if ((bx - mine) >> 5 != bo.chunk) bo.advance(k, x);
                    const int page = __shfl_sync(0xffffffffu, bo.page, bx & 31);
                    if (!(ok = sy.wait(empty + s, par, kSiteKvEmpty))) break;
                    if (lane == 0) ptx::mbar_arrive_expect_tx(sy.bar(full + s), L::TILE);
                    __syncwarp();
                    if (mine < per_tile)
                        ptx::tma_load_4d(dst + s * L::TILE, map, sy.bar(full + s), column, page < 0 ? 0 : in_page * k.box,
                                         x.h, page);
                    ++loaded;
                    if (++s == stages) {
                        s = 0;
                        par ^= 1u;
                    }
                    bx += per_tile;
                    in_page += per_tile;
                    if (a.table)
                        while (in_page >= k.page_boxes) in_page -= k.page_boxes;
                }
            }
            __syncwarp();
            // never leave a copy in flight into this CTA's shared memory
            for (int i = 0; i < stages && i < loaded; ++i)
                sy.drain(full + i, (uint32_t)(((loaded - 1 - i) / stages) & 1));
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
            int seg = 0;                                     // segments done
            uint32_t p_par = 0;                              // bit per slot
            bool ok = true;
            // S of a slot (K stage ks), and the products of 64 keys with V (stage vs).
            // Four steps of a loop: a CTA meets the code cold, and eight take 5 % longer
            // for 38 tokens over 59208 rows, one 6 % for the prompt.
            auto mma_s = [&](int slot, int ks) {
                const uint32_t kb = kb0 + (uint32_t)ks * (L::TILE >> 4);
                const uint32_t qb = qb0 + (SPLIT_ROWS ? (uint32_t)slot * (L::TILE >> 4) : 0u);
#pragma unroll 4
                for (int e = 0; e < 4 * L::KCH; ++e) {
                    const uint32_t o = (uint32_t)(e >> 2) * (L::CHUNK >> 4) + 2u * (e & 3);
                    ptx::umma_ss_lh(tmem + L::TM_S + 128u * slot, qb + o, kmaj_hi, kb + o, kmaj_hi, idesc_s, e ? 1u : 0u);
                }
                ptx::umma_commit(sy.bar(L::B_S_FULL + slot));
            };
            auto mma_pv = [&](int slot, int vs, int hf, bool more) {
                const uint32_t vb = vb0 + (uint32_t)vs * (L::TILE >> 4);
#pragma unroll 4
                for (int e = 4 * hf; e < 4 * hf + 4; ++e)        // 16 keys per step
                    ptx::umma_ts_lh(tmem + L::TM_O + 128u * slot, tmem + L::TM_S + 128u * slot + 8u * e,
                                    vb + 128u * e, v_hi, idesc_o, (more || e > 0) ? 1u : 0u);
            };
            // stages in turn (a division costs more than a product's time here)
            int ks = 0, vs = 0;
            uint32_t k_par = 0, v_par = 0;
            auto next_k = [&] { if (++ks == L::KS) ks = 0, k_par ^= 1u; };
            auto next_v = [&] { if (++vs == L::VS) vs = 0, v_par ^= 1u; };
            auto wait_k = [&] { return ok = sy.wait(L::B_K_FULL + ks, k_par, kSiteKvFull); };
            auto wait_v = [&] { return ok = sy.wait(L::B_V_FULL + vs, v_par, kSiteKvFull); };
            auto wait_p = [&](int slot, int hf) {
                return ok = sy.wait(L::B_P_FULL + 2 * slot + hf, p_par >> slot & 1u, kSitePFull);
            };
            for (; ok && x.next_tiles(k); ++seg) {
                if (!(ok = sy.wait(L::B_Q_FULL, (uint32_t)(seg & 1), kSiteQFull))) break;
                if constexpr (SPLIT_ROWS) {
                    // Both slots go through a key tile.  The issuer bounds it, so one
                    // wait for K and one for V serve both, and what belongs
                    // together is issued in one piece.  (One wait for all of P
                    // instead of two gains another 1 % here and costs 8 % over 512
                    // rows, where the first half's products hide the other's softmax.)
                    if (!wait_k()) break;
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        mma_s(0, ks);
                        mma_s(1, ks);
                        ptx::umma_commit(sy.bar(L::B_K_EMPTY + ks));
                        if (x.tiles == 1) ptx::umma_commit(sy.bar(L::B_Q_FREE));
                    }
                    __syncwarp();
                    next_k();
#pragma unroll 1
                    for (int t = 0; t < x.tiles; ++t) {
                        const bool next = t + 1 < x.tiles;
                        if (!wait_v() || (next && !wait_k())) break;
#pragma unroll
                        for (int slot = 0; slot < 2; ++slot) {
                            // the first 64 keys' products run while the other 64 are exponentiated
                            if (!wait_p(slot, 0)) break;
                            ptx::tc_fence_after();
                            if (ptx::elect_one()) mma_pv(slot, vs, 0, t > 0);
                            __syncwarp();
                            if (!wait_p(slot, 1)) break;
                            ptx::tc_fence_after();
                            if (ptx::elect_one()) {
                                mma_pv(slot, vs, 1, true);
                                if (slot == 1) ptx::umma_commit(sy.bar(L::B_V_EMPTY + vs));
                                if (next) {
                                    mma_s(slot, ks);
                                    if (slot == 1) {
                                        ptx::umma_commit(sy.bar(L::B_K_EMPTY + ks));
                                        if (t + 2 == x.tiles) ptx::umma_commit(sy.bar(L::B_Q_FREE));
                                    }
                                }
                            }
                            __syncwarp();
                            p_par ^= 1u << slot;
                        }
                        if (!ok) break;
                        next_v();
                        if (next) next_k();
                    }
                } else {
                    // The slots take key tiles in turn; S runs two ahead of P V.
                    const int jobs = x.tiles;
                    for (int j = -2; ok && j < jobs; ++j) {
                        const int slot = j & 1;
                        if (j >= 0) {
                            if (!wait_v()) break;
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                if (!wait_p(slot, hf)) break;
                                ptx::tc_fence_after();
                                if (ptx::elect_one()) {
                                    mma_pv(slot, vs, hf, j > 1 || hf > 0);
                                    if (hf == 1) ptx::umma_commit(sy.bar(L::B_V_EMPTY + vs));
                                }
                                __syncwarp();
                            }
                            if (!ok) break;
                            p_par ^= 1u << slot;
                            next_v();
                        }
                        if (j + 2 < jobs) {
                            if (!wait_k()) break;
                            ptx::tc_fence_after();
                            if (ptx::elect_one()) {
                                mma_s(slot, ks);
                                ptx::umma_commit(sy.bar(L::B_K_EMPTY + ks));
                                if (j + 3 == jobs) ptx::umma_commit(sy.bar(L::B_Q_FREE));
                            }
                            __syncwarp();
                            next_k();
                        }
                    }
                }
                if (!ok) break;
                if (ptx::elect_one()) ptx::umma_commit(sy.bar(L::B_O_FULL));
                __syncwarp();
            }
            if (ptx::elect_one()) ptx::umma_commit(sy.bar(L::B_DRAIN));
            __syncwarp();
            sy.drain(L::B_DRAIN, 0);
        } else {
            // --------------------------------------------------------- Q copier
            // A block's rows r = token * G + g, as soon as the unit before needs Q
            // no more: its last softmax and its output hide the copy.  Rows past
            // the sequence's tokens are not filled (a row's score reaches no other).
            constexpr int UPR = D / 8;                           // 16-byte units per row
            constexpr int STEP = 32 / UPR;                       // rows at a time: 2 or 4
            const int e = lane % UPR, r0 = lane / UPR;
            const int64_t row = STEP * a.q.head_stride, wrap = a.q.token_stride - k.G * a.q.head_stride;
            Walk x = first;
            for (int seg = 0; x.next_tiles(k); ++seg) {
                if (seg > 0 && !sy.wait(L::B_Q_FREE, (uint32_t)((seg - 1) & 1), kSiteQFull)) break;
                const int row_base = x.b * k.block, rows = min(L::RT * kTile, k.G * x.q.count - row_base);
                int j = token_of(k, row_base + r0), g = row_base + r0 - j * k.G;
                const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.q.data) + x.n * a.q.batch_stride +
                                         (int64_t)(x.h * k.G + g) * a.q.head_stride + (int64_t)j * a.q.token_stride + 8 * e;
                uint32_t dst = sQ + (e >> 3) * L::CHUNK;
#pragma unroll 4
                for (int r = r0; r < rows; r += STEP) {
                    ptx::cp_async_16(dst + (r / kTile) * L::TILE + (r % kTile) * 128 + (((e & 7) ^ (r & 7)) << 4), p, 16u);
                    p += row;
                    for (g += STEP; g >= k.G; g -= k.G) p += wrap;
                }
                ptx::cp_async_wait();
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sy.bar(L::B_Q_FULL));
            }
        }
    } else {
        // ------------------------------------------------ softmax / epilogue
        ptx::regs_inc<L::REGS_SOFTMAX>();
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
        // memory access (an arrive with release semantics first waits for the
        // warp's global stores).
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
        while (ok && cu.next(k)) {
            const int tiles = cu.tiles;
            const int n = cu.n, h = cu.h;
            const int row_base = cu.b * k.block;
            const int rows = min(L::RT * kTile, k.R - row_base); // rows of this unit
            const int first_new = cu.q.len - cu.q.count;
            // this thread's row of the unit (both slots' threads have the
            // same row where they share the row tile)
            const int r = (SPLIT_ROWS ? slot * kTile : 0) + lrow;
            const bool live = r < rows;
            const int j = live ? token_of(k, row_base + r) : 0, gg = live ? row_base + r - j * k.G : 0;
            const bool sees = live && j < cu.q.count;            // a token of the sequence
            const int limit = sees ? first_new + j + 1 : 0;      // rows it sees
            // the rows from here on are not seen by every token of the block
            const int common = first_new + token_of(k, row_base) + 1;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + n * a.out.batch_stride +
                                 (int64_t)(h * k.G + gg) * a.out.head_stride + (int64_t)j * a.out.token_stride;
            float* lse = a.lse ? a.lse + ((int64_t)n * a.q_heads + h * k.G + gg) * a.tokens + j : nullptr;
            constexpr int COLS = SPLIT_ROWS ? D : D / 2;         // columns this thread merges and writes
            const int c0 = SPLIT_ROWS ? 0 : slot * COLS;
            if (tiles == 0) {
                // no token in this block
                if (live) {
                    for (int cc = 0; cc < COLS; cc += 8)
                        *reinterpret_cast<uint4*>(out + c0 + cc) = make_uint4(0u, 0u, 0u, 0u);
                    if (lse && c0 == 0) *lse = -INFINITY;
                }
                continue;
            }
            const bool idle = (SPLIT_ROWS ? slot * kTile : 0) + q4 * 32 >= rows;   // no row in this warp

            float m = -INFINITY, l = 0.f;                        // reference (log2 units) and sum
            const int jobs = SPLIT_ROWS ? tiles : (tiles - slot + 1) / 2;   // of this slot
            for (int i = 0; ok && i < jobs; ++i) {
                const int dt = SPLIT_ROWS ? i : 2 * i + slot;    // tile of the segment
                const int t = cu.t + dt;
                // rows of the tile that the block's first token sees, and its last
                const int all = common - t * kTile, some = cu.keys - t * kTile;
                if (!(ok = sy.wait(L::B_S_FULL + slot, s_par, kSiteSFull))) break;
                s_par ^= 1u;
                __syncwarp();
                ptx::tc_fence_after();
                const bool special = all < kTile;
                if (special) {
                    // V rows whose products with P = 0 must be 0.  (After S
                    // full, which implies that the slot's last P V is done
                    // and with it the load before this one in V's stage: a
                    // wait for a phase before the last one ended would pass.)
                    const int g = g0 + dt, vs = g % L::VS;
                    if (!(ok = sy.wait(L::B_V_FULL + vs, (uint32_t)((g / L::VS) & 1), kSiteKvFull))) break;
                    uint8_t* vt = base + L::OFF_V + vs * L::TILE;
                    constexpr int UPR = D / 8;
                    for (int x = max(all, 0) * UPR + st; x < kTile * UPR; x += 128) {
                        const int vr = x / UPR, e = x - vr * UPR;
                        uint4* p = reinterpret_cast<uint4*>(vt + (e >> 3) * L::CHUNK + vr * 128 +
                                                            (((e & 7) ^ (vr & 7)) << 4));
                        if (vr >= some) {
                            *p = make_uint4(0u, 0u, 0u, 0u);
                            continue;
                        }
                        const uint4 v = *p;
                        const uint32_t o0 = odd_halves(v.x), o1 = odd_halves(v.y), o2 = odd_halves(v.z),
                                       o3 = odd_halves(v.w);
                        if (o0 | o1 | o2 | o3) {
                            const int at = vr - all;             // of the rows from `common` on
                            atomicOr(odd_rows + (seg & 1) * kOddWords + (at >> 5), 1u << (at & 31));
                            __threadfence_block();
                            *p = make_uint4(v.x & ~o0, v.y & ~o1, v.z & ~o2, v.w & ~o3);
                        }
                    }
                    ptx::fence_proxy_async_smem();
                }
                if (!idle) {
                    // With one row tile HBM is the bound, and what counts is that a
                    // CTA meets this code cold: 32 columns at a time, read twice,
                    // it is a quarter as long.  (All 128 at once, fetched while every
                    // SM asks for its first tiles, the first tile took 4 to 7 us.)
                    const int valid = limit - t * kTile;
                    uint32_t x[SPLIT_ROWS ? 2 : 1][64];
                    auto scores32 = [&](int cc) {
                        uint32_t (&y)[32] = reinterpret_cast<uint32_t (&)[32]>(x[0]);
                        ptx::tmem_ld_32x32b_x32(t_s + cc, y);
                        ptx::tmem_ld_wait();
                        if (special)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (cc + e >= valid) y[e] = 0xff800000u;
                    };
                    float mx[2] = {-INFINITY, -INFINITY};
                    if constexpr (SPLIT_ROWS) {
                        ptx::tmem_ld_32x32b_x64(t_s, x[0]);
                        ptx::tmem_ld_32x32b_x64(t_s + 64, x[1]);
                        ptx::tmem_ld_wait();
                        if (special) {
#pragma unroll
                            for (int e = 0; e < 64; ++e) {
                                if (e >= valid) x[0][e] = 0xff800000u;
                                if (64 + e >= valid) x[1][e] = 0xff800000u;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 64; e += 2)
#pragma unroll
                            for (int b = 0; b < 2; ++b)
                                mx[b] = ptx::max3(mx[b], __uint_as_float(x[b][e]), __uint_as_float(x[b][e + 1]));
                    } else {
#pragma unroll 1
                        for (int cc = 0; cc < kTile; cc += 32) {
                            scores32(cc);
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                mx[0] = ptx::max3(mx[0], __uint_as_float(x[0][e]), __uint_as_float(x[0][e + 1]));
                                mx[1] = ptx::max3(mx[1], __uint_as_float(x[0][e + 2]), __uint_as_float(x[0][e + 3]));
                            }
                            __syncwarp();
                        }
                    }
                    const float top = fmaxf(mx[0], mx[1]) * sc;
                    const bool raise = sees && top > m + kSlack;   // (other rows' queries are anything)
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? ptx::ex2_approx(m - top) : 1.f;
                        if (raise) m = top;
                        l *= f;
                        __syncwarp();
                        // S full: every product into O so far is done
                        if (i > 0) {
#pragma unroll (SPLIT_ROWS ? D / 32 : 1)
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
                    // N pairs of columns: exponentials, their sums, P
                    auto weigh = [&](const uint32_t* from, auto& p) {
                        constexpr int N = sizeof(p) / 4;
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            const float2 z = ptx::fma2(make_float2(__uint_as_float(from[2 * e]),
                                                                   __uint_as_float(from[2 * e + 1])),
                                                       make_float2(sc, sc), make_float2(nm, nm));
                            const float2 y = make_float2(ptx::ex2_approx(z.x), ptx::ex2_approx(z.y));
                            sum[e & 1] = ptx::add2(sum[e & 1], y);
                            p[e] = ptx::pack_bf16x2(y.x, y.y);
                        }
                    };
                    // P of a half of 64 keys is stored: itself it is ordered by the
                    // tensor-memory wait and fence; only cleaned rows of V need a release
                    auto half_done = [&](int hh) {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if (special) ptx::mbar_arrive(sy.bar(L::B_P_FULL + 2 * slot + hh));
                            else ptx::mbar_arrive_relaxed(sy.bar(L::B_P_FULL + 2 * slot + hh));
                        }
                    };
                    if constexpr (SPLIT_ROWS) {
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            uint32_t p[32];
                            weigh(x[hh], p);
                            ptx::tmem_st_32x32b_x32(t_s + 32 * hh, p);
                            ptx::tmem_st_wait();
                            half_done(hh);
                        }
                    } else {
#pragma unroll 1
                        for (int cc = 0; cc < kTile; cc += 32) {
                            uint32_t p[16];
                            scores32(cc);
                            weigh(x[0], p);
                            __syncwarp();
                            ptx::tmem_st_32x32b_x16(t_s + cc / 2, p);
                            ptx::tmem_st_wait();
                            if (cc & 32) half_done(cc >> 6);
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
            // the next segment's marks (every read of them was before the last
            // segment's second sync, every write comes after the next one)
            if (tid < kOddWords) odd_rows[((seg + 1) & 1) * kOddWords + tid] = 0u;
            ptx::tc_fence_before();
            if (!(ok = sync_sm(false))) break;
            const bool whole = cu.t == 0 && tiles == cu.nt;
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
            volatile uint32_t* odd = odd_rows + (seg & 1) * kOddWords;
            bool any_odd = false;
            if (cu.keys > common)
                for (int i = 0; i < kOddWords; ++i) any_odd |= odd[i] != 0u;
            const int64_t place = 2 * (int64_t)c + cu.part;
            const float inv = !whole ? 1.f : sees && (l > 0.f || l != l) ? 1.f / l : 0.f;
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
                    if (any_odd) {
                        // infinities and NaN of the rows that this token sees
                        for (int i = common; i < limit; ++i) {
                            if (!(odd[(i - common) >> 5] >> ((i - common) & 31) & 1u)) continue;
                            const Paging pg = paging_of(a);
                            const int page = page_at(pg, n, a.table ? i / a.page_rows : 0, a.status);
                            if (page < 0) continue;
                            const __nv_bfloat16* vr =
                                static_cast<const __nv_bfloat16*>(a.v_pages.data) + page * a.v_pages.batch_stride +
                                h * a.v_pages.head_stride +
                                (int64_t)(a.table ? i % a.page_rows : i) * a.v_pages.token_stride;
#pragma unroll
                            for (int e = 0; e < 32; ++e) {
                                const float y = __bfloat162float(vr[c0 + cc + e]);
                                if (!(fabsf(y) < INFINITY)) v[e] += y;
                            }
                        }
                    }
                    // (a padded row's scores are those of zeros, but V may hold anything)
                    if (!sees)
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = 0.f;
                    if (live && whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4*>(out + c0 + cc + e) =
                                make_uint4(ptx::pack_bf16x2(v[e] * inv, v[e + 1] * inv),
                                           ptx::pack_bf16x2(v[e + 2] * inv, v[e + 3] * inv),
                                           ptx::pack_bf16x2(v[e + 4] * inv, v[e + 5] * inv),
                                           ptx::pack_bf16x2(v[e + 6] * inv, v[e + 7] * inv));
                    } else if (live) {
                        float4* po = reinterpret_cast<float4*>(k.part_o) +
                                     (place * (D / 4) + (c0 + cc) / 4) * k.rows + r;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            po[(int64_t)(e / 4) * k.rows] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    }
                }
                if (live && c0 == 0) {
                    if (!sees) m = -INFINITY, l = 0.f;
                    if (!whole) k.part_ml[place * k.rows + r] = make_float2(m, l);
                    else if (lse) *lse = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
                }
            }
            ptx::tc_fence_before();
            // O and ml are read (the values are in registers): the next segment
            // may write them
            if (!(ok = sync_sm(true))) break;
            g0 += tiles;
            ++seg;
        }
    }
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, L::TMEM_COLS);
    }
}

// Merges the parts of a unit that several CTAs shared, in CTA order:
//   O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i
// Fewer units than shares (one layer at 128 k rows: up to 76 parts each): the
// grid has many CTAs per unit.  Else a unit is cut where a share starts inside of
// it, so the grid has a few CTAs per share start, and the first start inside a
// unit merges it.  Thread = 4 columns of a row, consecutive threads consecutive
// rows (how the parts lie).  Where a unit has many parts kWays threads share an
// output, each taking every kWays-th part; with up to kFew one thread takes them
// all and no barrier is needed.
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
__global__ void __launch_bounds__(kMergeThreads) paged_combine_kernel(const __grid_constant__ PagedKernelArgs k,
                                                                      int per, int by_unit) {
    const statekv_paged_attention_args& a = k.a;
    const int which = blockIdx.x / per, part = blockIdx.x - which * per;
    Plan plan;
    Place p = schedule(k, by_unit ? 0 : which + 1, plan);
    uint32_t w = 0;                          // where the unit starts
    bool mine = true;
    if (by_unit) {
        w = unit_start(k, which, p);
    } else if ((mine = which + 1 < (int)plan.ctas)) {
        const uint32_t cut = plan.start((uint32_t)which + 1);
        w = cut - (uint32_t)p.v;
        mine = p.v > 0 && plan.start((uint32_t)which) <= w;
    }
    const int nt = mine ? block_tiles(k, p.q, p.b) : 0;
    // in every CTA, before it may leave: this grid must not end before the one
    // whose end it stands for, even where there is nothing to merge
    ptx::dep_wait();
    if (nt == 0) return;
    const int ca = (int)plan.cta_of(w + kUnitCost), cb = (int)plan.cta_of(w + kUnitCost + (uint32_t)nt - 1);
    const int segs = cb - ca + 1;
    if (segs == 1) return;                   // written by the one CTA
    const int n = p.n, h = p.h;
    const int rows = min(k.block, k.R - p.b * k.block);
    const int outs = rows * (D / 4);
    const int ways = segs > kFew ? kWays : 1;
    const int per_step = kMergeThreads / ways, x = threadIdx.x % per_step, way = threadIdx.x / per_step;
    __shared__ Merge sh[kMergeThreads];
    // part i: the share's first unit's where the share starts in the unit, else its last's
    const int64_t head = 2 * (int64_t)ca + (plan.start((uint32_t)ca) >= w ? 0 : 1);
    for (int out0 = part * per_step; out0 < outs; out0 += per * per_step) {
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
                    const int i = i0 + b * ways;
                    ml[b] = make_float2(-INFINITY, 0.f);
                    y[b] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i < segs) {
                        const int64_t at = i == 0 ? head : 2 * (int64_t)(ca + i);
                        ml[b] = k.part_ml[at * k.rows + r];
                        y[b] = reinterpret_cast<const float4*>(k.part_o)[(at * (D / 4) + c4) * k.rows + r];
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
        const int row = p.b * k.block + r, j = token_of(k, row), gg = row - j * k.G;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out.data) + n * a.out.batch_stride +
                             (int64_t)(h * k.G + gg) * a.out.head_stride + (int64_t)j * a.out.token_stride + c4 * 4;
        *reinterpret_cast<uint2*>(dst) = make_uint2(ptx::pack_bf16x2(acc.o.x * inv, acc.o.y * inv),
                                                    ptx::pack_bf16x2(acc.o.z * inv, acc.o.w * inv));
        if (a.lse && c4 == 0)
            a.lse[((int64_t)n * a.q_heads + h * k.G + gg) * a.tokens + j] =
                acc.l != 0.f ? (acc.m + log2f(acc.l)) * 0.6931471805599453f : -INFINITY;
    }
}

template <int D, bool SPLIT_ROWS>
cudaError_t launch_main(const PagedKernelArgs& k, const CUtensorMap& mk, const CUtensorMap& mv, int dev,
                        cudaStream_t st) {
    using L = PagedLayout<D, SPLIT_ROWS>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e =
        allow_smem(reinterpret_cast<const void*>(&paged_kernel<D, SPLIT_ROWS>), L::SMEM, dev, done);
    if (e != cudaSuccess) return e;
    paged_kernel<D, SPLIT_ROWS><<<(unsigned)k.grid, kPagedThreads, L::SMEM, st>>>(mk, mv, k);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_combine(const PagedKernelArgs& k, int64_t units, int sms, cudaStream_t st) {
    // about eight CTAs per SM, but no more than there are steps of the many-part
    // form.  (Eight per cut for two units of 228 rows, 18 MB of parts: 100 us.)
    const int steps = (k.rows * (D / 4) + kMergeThreads / kWays - 1) / (kMergeThreads / kWays);
    const int by_unit = units < k.grid;
    const int groups = by_unit ? (int)units : k.grid - 1;
    const int per = std::max(1, std::min(steps, 8 * sms / groups));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups * per));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_combine_kernel<D>, k, per, by_unit);
}

// Sizes that follow from the arguments; what to refuse them with.
struct PagedSizes {
    int G, R, rb, rows, block;
    int64_t units;
};
int paged_sizes(int batch, int q_heads, int kv_heads, int tokens, int head_dim, PagedSizes* z) {
    if (batch < 0 || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0 || tokens < 1)
        return STATEKV_E_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || q_heads / kv_heads > 64) return STATEKV_E_UNSUPPORTED;
    z->G = q_heads / kv_heads;
    if ((int64_t)z->G * tokens >= 1 << 26) return STATEKV_E_UNSUPPORTED;     // token_of
    z->R = z->G * tokens;
    z->block = z->R > kTile ? 2 * kTile : kTile;
    z->rb = (z->R + z->block - 1) / z->block;
    z->rows = std::min(z->R, z->block);
    z->units = (int64_t)batch * kv_heads * z->rb;
    return z->units > 0x7fffffff / 1024 ? STATEKV_E_UNSUPPORTED : STATEKV_OK;
}

// A few short units are not cut: their 8 tiles one after the other take about
// as long as the second launch that would merge them.
int64_t most_tiles(int64_t cache_rows) { return (cache_rows + kTile - 1) / kTile; }
bool stays_whole(const PagedSizes& z, int64_t cache_rows, int sms) {
    return most_tiles(cache_rows) <= kWholeTiles && z.units <= sms;
}

int64_t workspace_for(const PagedSizes& z, int sms, int d) {
    // two parts per CTA; O, then (m, l)
    return 2 * (int64_t)sms * z.rows * (d * 4 + 8);
}

}  // namespace
}  // namespace statekv

extern "C" int64_t statekv_paged_attention_workspace(int32_t batch, int32_t q_heads, int32_t kv_heads,
                                                     int32_t tokens, int32_t head_dim, int32_t cache_rows) {
    using namespace statekv;
    PagedSizes z;
    if (cache_rows < 0) return -1;
    if (paged_sizes(batch, q_heads, kv_heads, tokens, head_dim, &z) != STATEKV_OK) return -1;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) {
        cudaGetLastError();
        return -1;
    }
    return stays_whole(z, cache_rows, sms) ? 0 : workspace_for(z, sms, head_dim);
}

extern "C" int statekv_paged_attention(const statekv_paged_attention_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_paged_attention_args& a = *args;
    if (a.layers < 1 || a.batch < 0 || a.batch % a.layers != 0 || a.length < 0 || !(a.scale > 1e-30) ||
        !(a.scale < 1e30))
        return STATEKV_E_INVALID_ARG;
    PagedSizes z;
    int r = paged_sizes(a.batch, a.q_heads, a.kv_heads, a.tokens, a.head_dim, &z);
    if (r != STATEKV_OK) return r;
    if (!a.status || !ints_ok(a.status) || !ints_ok(a.lengths) || !ints_ok(a.counts) || !ints_ok(a.lse))
        return STATEKV_E_INVALID_ARG;
    const Paging pg = paging_of(a);
    if ((r = paging_ok(pg, a.batch)) != STATEKV_OK) return r;
    if (!a.lengths && a.length > pg.capacity()) return STATEKV_E_CAPACITY;
    if (a.batch == 0) return STATEKV_OK;
    if (!view_ok(a.q, 2, a.batch, a.q_heads, a.tokens) || !view_ok(a.out, 2, a.batch, a.q_heads, a.tokens) ||
        !apart(a.out, a.batch, a.q_heads, a.tokens, a.head_dim))
        return STATEKV_E_INVALID_ARG;
    // an empty pool needs no memory: its maps are never read
    const bool cached = !paging_empty(pg);
    if (cached) {
        for (const statekv_view* v : {&a.k_pages, &a.v_pages})
            if (!view_ok(*v, 2, a.num_pages, a.kv_heads, a.page_rows) ||
                !spread(*v, a.num_pages, a.kv_heads, a.page_rows))
                return STATEKV_E_INVALID_ARG;
    }
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return view_cuda_fail();
    const int64_t most = a.lengths ? (cached ? pg.capacity() : 0) : a.length;
    const bool whole = stays_whole(z, cached ? pg.capacity() : 0, sms);
    if (!whole && (!aligned16(a.workspace) || a.workspace_bytes < workspace_for(z, sms, a.head_dim)))
        return STATEKV_E_INVALID_ARG;
    PagedKernelArgs k{};
    k.a = a;
    k.G = z.G; k.R = z.R; k.rb = z.rb; k.rows = z.rows; k.block = z.block;
    k.inv_group = (uint32_t)((1ull << 32) / (uint32_t)z.G + 1);
    k.scale_log2 = (float)(a.scale * 1.4426950408889634074);
    k.capacity = cached ? (int)pg.capacity() : 0;
    // the largest power of two of rows that divides a page; a plain cache is
    // read past its end (zeros) in whole tiles
    k.box = kTile;
    if (a.table)
        while (a.page_rows % k.box != 0) k.box /= 2;
    k.page_boxes = a.table ? a.page_rows / k.box : 1;
    CUtensorMap mk{}, mv{};
    if (cached && (!encode_view4(&mk, a.k_pages, a.head_dim, a.page_rows, a.kv_heads, a.num_pages, k.box) ||
                   !encode_view4(&mv, a.v_pages, a.head_dim, a.page_rows, a.kv_heads, a.num_pages, k.box)))
        return STATEKV_E_UNSUPPORTED;
    // otherwise no more CTAs than the longest cache could use
    k.whole = whole;
    const int64_t cost = most_tiles(most) + kUnitCost;
    if (z.units * cost > 0x7fffffff) return STATEKV_E_UNSUPPORTED;   // the schedule counts in 32 bits
    k.grid = whole ? (int)z.units : (int)std::min<int64_t>(sms, (z.units * cost + kMinShare - 1) / kMinShare);
    k.merge = !whole && k.grid > 1;          // one CTA holds whole units only
    k.part_o = static_cast<float*>(a.workspace);
    k.part_ml = reinterpret_cast<float2*>(k.part_o + 2 * (int64_t)sms * z.rows * a.head_dim);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(cuda_stream);
    const bool two = z.R > kTile;
    cudaError_t e = a.head_dim == 128 ? two ? launch_main<128, true>(k, mk, mv, dev, st) : launch_main<128, false>(k, mk, mv, dev, st)
                    : two             ? launch_main<64, true>(k, mk, mv, dev, st)
                                      : launch_main<64, false>(k, mk, mv, dev, st);
    if (e == cudaSuccess && k.merge) e = a.head_dim == 128 ? launch_combine<128>(k, z.units, sms, st) : launch_combine<64>(k, z.units, sms, st);
    return e == cudaSuccess ? STATEKV_OK : view_cuda_fail();
}
