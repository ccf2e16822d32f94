// Verification of a drafted tree against the target's probabilities: the path
// that stands and the token after it.
//
// The residual after k refused children of a node, max(... max(max(p - q, 0) -
// R1 q, 0) ... - R(k-1) q, 0), is max(p - c q, 0) with c = 1 + R1 + ... , for q is
// not negative: a refusal costs one pass over the two rows that sums it up, and
// one number of state.  An accepted node needs no pass at all, and what the
// children's own tests read (one p, one q each) is fetched for the whole tree at
// the start, in one latency.  The last pass serves the sampling too: its partial
// sums say which warp's run of the vocabulary holds the token, and that warp
// reads its run (a few hundred entries) once more.
//
// One cluster per sequence; warp 0 of every CTA does the same walk, and a warp
// sums a contiguous run of the vocabulary, brought to shared memory by bulk
// copies (and kept for the node's next refusal, where the run fits).  Bound by
// latency: the passes of one sequence follow each other, 5 to 6 us each (rows
// 1 to 1.6, their sum 2.8, the cluster's 0.9, the walk 1.2).  16 trees of 42
// nodes over 150001 entries, 4 to 5 passes for the slowest: 35.6 us.
//
// Sums decide which token comes out, so they do not depend on how a row is cut:
// p - c q is formed with its rounding error (two-term products and sums, off by
// at most 2^-47), each entry is rounded once to a whole number of 2^-60, and whole
// numbers are added.  The splitting needs fp32 additions only (add_units); fp64
// ones would run at a 64th of the rate.
#include <algorithm>

#include "views.cuh"
#include "sm100_ptx.cuh"

namespace statekv {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxNodes = 64;
constexpr int kMaxCluster = 16;
constexpr int kRoomAlone = 1664, kRoomShared = 768;  // entries of a warp: 213 and 98 KB of p and q a CTA
constexpr int kMostAdded = 128;              // entries that a lane adds up in 32 bits (Units)
static_assert(kRoomAlone / 32 < kMostAdded, "entries of a lane");

struct VerifyKernelArgs {
    statekv_verify_args a;
    int32_t cluster;
    int32_t run;                             // entries of a warp, a multiple of 32
    int32_t room;                            // entries of p, and of q, that a warp has room for, a multiple of 8
};

// a - b (a fused multiply-add by -1 is exact in the product)
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return ptx::fma2(b, make_float2(-1.f, -1.f), a); }

// max(p - c q, 0) of two entries as h + l, c = -(mch + mcl)
__device__ __forceinline__ void residual2(float2 p, float2 q, float2 mch, float2 mcl, float2& h, float2& l) {
    const float2 t = ptx::fma2(mch, q, make_float2(0.f, 0.f));       // rounded -ch q
    h = ptx::add2(p, t);
    const float2 bb = sub2(h, p);
    l = ptx::add2(sub2(p, sub2(h, bb)), sub2(t, bb));                // what that sum lost, exactly
    // what the product lost, and the rest of c
    l = ptx::add2(l, ptx::fma2(mch, q, make_float2(-t.x, -t.y)));
    l = ptx::fma2(mcl, q, l);
    if (!(h.x + l.x > 0.f)) h.x = l.x = 0.f;
    if (!(h.y + l.y > 0.f)) h.y = l.y = 0.f;
}

// A sum in whole numbers of 2^-21, 2^-44 and 2^-60.  x + A for a constant A of
// 1.5 times a power of two is x rounded to a multiple of A's last place, its bits
// count them, and x - ((x + A) - A) is the rest, exactly: what an entry adds is a
// function of the entry alone.  It adds at most 2^23 to the middle one: kMostAdded
// of them stay in 32 bits.
constexpr float kTop = 6.f, kMid = 0x1.8p-21f, kLow = 0x1.8p-37f;
struct Units {
    uint32_t top = 0u, mid = 0u, low = 0u;
    __device__ __forceinline__ long long whole() const {
        return ((long long)(int)top << 39) + ((long long)(int)mid << 16) + (long long)(int)low;
    }
};

// Adds two entries h + l, |h| <= 2 and |l| <= 2^-22 (others add some number).
template <bool WITH_L>
__device__ __forceinline__ void add_units(Units& u, float2 h, float2 l) {
    auto both = [](float2 x, float a) {
        return __float_as_uint(x.x) + __float_as_uint(x.y) - 2u * __float_as_uint(a);
    };
    const float2 top = make_float2(kTop, kTop), mid = make_float2(kMid, kMid), low = make_float2(kLow, kLow);
    float2 x = ptx::add2(h, top);
    u.top += both(x, kTop);
    h = sub2(h, sub2(x, top));
    x = ptx::add2(h, mid);
    u.mid += both(x, kMid);
    h = sub2(h, sub2(x, mid));
    if constexpr (WITH_L) {
        x = ptx::add2(l, mid);
        u.mid += both(x, kMid);
        h = ptx::add2(h, sub2(l, sub2(x, mid)));
    }
    u.low += both(ptx::add2(h, low), kLow);
}

// max(p - c q, 0), or p where `with_q` is not, in units of 2^-60
__device__ __forceinline__ long long units_of(float p, float q, bool with_q, float ch, float cl) {
    Units u;
    float2 h = make_float2(p, 0.f), l = make_float2(0.f, 0.f);
    if (with_q) residual2(h, make_float2(q, 0.f), make_float2(-ch, -ch), make_float2(-cl, -cl), h, l);
    add_units<true>(u, h, l);
    return u.whole();
}

// NaN and negative values count as 0
__device__ __forceinline__ float weight(const float* p) { return fmaxf(__ldg(p), 0.f); }

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const __grid_constant__ VerifyKernelArgs ka) {
    const statekv_verify_args& a = ka.a;
    __shared__ int s_parent[kMaxNodes], s_token[kMaxNodes];  // token -1: out of range
    __shared__ float s_p[kMaxNodes], s_q[kMaxNodes], s_u[kMaxNodes + 1];
    __shared__ struct {
        uint64_t refused;
        float ch, cl;
        int node, more;
    } s_pass;
    __shared__ long long s_warp[kVerifyWarps];
    __shared__ long long s_sums[2][kMaxCluster];
    __shared__ __align__(8) uint64_t s_bars[kVerifyWarps][4];
    extern __shared__ __align__(16) float s_rows[];          // [warps][2][room]: p, q
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = ka.cluster, rank = blockIdx.x % C, seq = blockIdx.x / C;
    const float* target = a.target + seq * a.target_stride;
    const float* draft = a.draft ? a.draft + seq * a.draft_stride : nullptr;
    if (tid < kVerifyWarps * 4) ptx::mbar_init(ptx::smem_u32(&s_bars[0][0]) + 8 * tid, 1);
    ptx::fence_barrier_init();
    if (tid < a.tokens) {
        const uint64_t mask = a.tree[(int64_t)seq * a.tree_stride + tid] & ((1ull << tid) - 1ull);
        const int parent = mask ? 63 - __clzll((long long)mask) : -1;
        int x = a.drafted[(int64_t)seq * a.tokens + tid];
        s_p[tid] = s_q[tid] = 0.f;
        if ((uint32_t)x < (uint32_t)a.vocab) {
            s_p[tid] = weight(target + (parent + 1) * a.target_row + x);
            if (draft) s_q[tid] = weight(draft + (parent + 1) * a.draft_row + x);
        } else {
            if (rank == 0) record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteNode, (uint32_t)x);
            x = -1;
        }
        s_parent[tid] = parent;
        s_token[tid] = x;
    }
    if (tid <= a.tokens) s_u[tid] = fminf(fmaxf(a.uniforms[(int64_t)seq * (a.tokens + 1) + tid], 0.f), 0x1.fffffep-1f);
    __syncthreads();

    // this warp's run of the vocabulary
    const int v0 = min((int64_t)a.vocab, (int64_t)(rank * kVerifyWarps + warp) * ka.run);
    const int v1 = min((int64_t)a.vocab, (int64_t)v0 + ka.run);
    // what the next pass sums, from warp 0's walk
    int cur = -1, passes = 0;
    float ch = 0.f, cl = 0.f;                                // c
    uint64_t refused = 0;                                    // nodes refused here (without a draft)
    const float* p_row = target;
    const float* q_row = draft;
    auto refused_token = [&](int v) -> bool {
        for (uint64_t b = refused; b; b &= b - 1)
            if (s_token[__ffsll((long long)b) - 1] == v) return true;
        return false;
    };
    // Entries [from, to) of one of the current rows into this warp's shared
    // memory at `buf` (16-byte aligned, 4 entries more than that): whole 16-byte
    // units by bulk copies, on which the warp's barrier `bar` counts, the up to
    // three entries before and behind them by plain loads, so that nothing
    // outside of the row is read.  Returns where the first entry lies.
    auto fetch = [&](const float* row, int from, int to, float* buf, uint32_t bar) -> int {
        const float* src = row + from;
        const int off = (int)(reinterpret_cast<uintptr_t>(src) / 4 % 4), n = to - from;
        const int head = min(n, (4 - off) % 4), body = (n - head) / 4 * 4;
        if (lane == 0 && body > 0) {
            ptx::mbar_arrive_expect_tx(bar, (uint32_t)body * 4);
            ptx::bulk_load(ptx::smem_u32(buf + off + head), src + head, (uint32_t)body * 4, bar);
        } else if (lane == 0) {
            ptx::mbar_arrive(bar);
        }
        if (lane >= 1 && lane <= head) buf[off + lane - 1] = __ldg(src + lane - 1);
        const int last = head + body + lane - 4;
        if (lane >= 4 && last < n) buf[off + last] = __ldg(src + last);
        return off;
    };
    // waits for the copies of one phase of a barrier (bounded)
    auto landed = [&](uint32_t bar, uint32_t parity) {
        const uint64_t t0 = globaltimer_ns();
        while (!ptx::mbar_wait_hint(bar, parity, 20000u))
            if (globaltimer_ns() - t0 > 1000000000ull) {
                record_error(a.status, (uint32_t)STATEKV_E_TIMEOUT, kSiteKvFull, (uint32_t)warp);
                break;
            }
        __syncwarp();
    };
    float* p_buf = s_rows + warp * 2 * ka.room;
    float* q_buf = p_buf + ka.room;
    const uint32_t bar = ptx::smem_u32(&s_bars[warp][0]);    // [2 halves][p, q]
    uint32_t parity = 0;                                     // bit 2 * half + (q)
    const bool fits = v1 - v0 <= ka.room - 4;
    int p_off = 0, q_off = 0;                                // where a run's first entries lie
    int p_node = -2, q_node = -2;                            // whose rows the shared memory holds
    // the residual's sum in units of 2^-60, its parts in s_warp and s_sums
    auto sum_up = [&]() -> long long {
        const bool with_q = ch > 0.f;
        const float2 mch = make_float2(-ch, -ch), mcl = make_float2(-cl, -cl);
        long long sum = 0;
        auto add_all = [&](const float* ps, const float* qs, int count) {
            Units u;
#pragma unroll 4
            for (int i = lane; i < count; i += 64) {
                const bool two = i + 32 < count;
                float2 h = make_float2(fmaxf(ps[i], 0.f), two ? fmaxf(ps[i + 32], 0.f) : 0.f), l;
                if (with_q) {
                    residual2(h, make_float2(fmaxf(qs[i], 0.f), two ? fmaxf(qs[i + 32], 0.f) : 0.f), mch, mcl, h, l);
                    add_units<true>(u, h, l);
                } else {
                    add_units<false>(u, h, h);
                }
            }
            sum += u.whole();
        };
        if (fits) {
            // rows that are there already are not read again
            const bool new_p = p_node != cur, new_q = with_q && q_node != cur;
            if (new_p || new_q) ptx::fence_proxy_async_smem();
            __syncwarp();
            if (new_p) p_off = fetch(p_row, v0, v1, p_buf, bar);
            if (new_q) q_off = fetch(q_row, v0, v1, q_buf, bar + 8);
            if (new_p) {
                landed(bar, parity & 1);
                parity ^= 1;
                p_node = cur;
            }
            if (new_q) {
                landed(bar + 8, parity >> 1 & 1);
                parity ^= 2;
                q_node = cur;
            }
            add_all(p_buf + p_off, q_buf + q_off, v1 - v0);
        } else {
            // in pieces of half the room, the next one on its way
            const int half = ka.room / 2, piece = half - 4;
            int offs[2][2];
            auto start = [&](int v, int i) {
                offs[i][0] = fetch(p_row, v, min(v1, v + piece), p_buf + i * half, bar + 16 * i);
                offs[i][1] = with_q ? fetch(q_row, v, min(v1, v + piece), q_buf + i * half, bar + 16 * i + 8) : 0;
            };
            ptx::fence_proxy_async_smem();
            __syncwarp();
            start(v0, 0);
            int v = v0;
#pragma unroll 1
            while (v < v1) {
#pragma unroll
                for (int i = 0; i < 2; ++i, v += piece) {
                    if (v >= v1) break;
                    if (v + piece < v1) start(v + piece, i ^ 1);
                    landed(bar + 16 * i, parity >> (2 * i) & 1);
                    parity ^= 1u << (2 * i);
                    if (with_q) {
                        landed(bar + 16 * i + 8, parity >> (2 * i + 1) & 1);
                        parity ^= 2u << (2 * i);
                    }
                    add_all(p_buf + i * half + offs[i][0], q_buf + i * half + offs[i][1], min(piece, v1 - v));
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) {
            // each refused token once: that of a node no other refused node below has
            for (uint64_t b = refused; b; b &= b - 1) {
                const int i = __ffsll((long long)b) - 1, x = s_token[i];
                bool again = false;
                for (uint64_t e = refused & ((1ull << i) - 1ull); e; e &= e - 1)
                    again |= s_token[__ffsll((long long)e) - 1] == x;
                if (!again && x >= v0 && x < v1) sum -= units_of(s_p[i], 0.f, false, 0.f, 0.f);
            }
            s_warp[warp] = sum > 0 ? sum : 0;
        }
        __syncthreads();
        long long* sums = s_sums[passes & 1];
        if (tid < C) {
            long long cta = 0;
            for (int i = 0; i < kVerifyWarps; ++i) cta += s_warp[i];
            const uint32_t at = ptx::cluster_map(ptx::smem_u32(&sums[rank]), (uint32_t)tid);
            ptx::st_cluster_u32(at, (uint32_t)cta);
            ptx::st_cluster_u32(at + 4, (uint32_t)((uint64_t)cta >> 32));
        }
        ptx::cluster_sync();
        ++passes;
        long long all = 0;
        for (int i = 0; i < C; ++i) all += sums[i];
        return all;
    };

    // Token 0 until a warp finds its own: where no sum is left, and where rows that
    // are no probabilities take the sums out of range.
    if (rank == 0 && tid == 0) a.next[seq] = 0;
    // "every CTA of the cluster has started", before its memory is written
    ptx::cluster_sync();
    // The walk, by warp 0 alone (a step takes a dozen fp64 operations, which 512
    // threads would wait 256 cycles each for).  It goes on until a pass is needed
    // and leaves what that sums in s_pass; false: no pass, the last one's sum stands.
    int at = -1, count = 0;                                  // current node, accepted ones
    double c = 0.0, R = 1.0;
    uint64_t children = 0, out = 0;                          // of `at` that are left, refused (without a draft)
    bool summed = false, empty = false;
    long long total = 0;
    auto children_of = [&](int node) -> uint64_t {
        const unsigned lo = __ballot_sync(0xffffffffu, lane < a.tokens && s_parent[lane] == node);
        const unsigned hi = __ballot_sync(0xffffffffu, lane + 32 < a.tokens && s_parent[(lane + 32) % kMaxNodes] == node);
        return (uint64_t)hi << 32 | lo;
    };
    auto walk = [&]() -> bool {
        while (children) {
            const int i = __ffsll((long long)children) - 1;
            children &= children - 1;
            const double p = s_p[i], q = s_q[i], u = s_u[i];
            bool again = false;
            for (uint64_t b = out; b; b &= b - 1) again |= s_token[__ffsll((long long)b) - 1] == s_token[i];
            const double r = draft ? fmax(p - c * q, 0.0) : again ? 0.0 : p;
            if (s_token[i] >= 0 && (draft ? u * q * R : u * R) < r) {
                if (rank == 0 && lane == 0) a.path[(int64_t)seq * a.tokens + count] = i;
                ++count;
                at = i;
                children = children_of(i);
                c = 0.0;
                R = 1.0;
                out = 0;
                summed = false;
            } else if (draft) {
                c += R;
                summed = true;
                return true;
            } else {
                R = fmax(R - r, 0.0);
                if (s_token[i] >= 0) out |= 1ull << i;
            }
        }
        if (!summed) return summed = true;
        if (total <= 0 && !empty && (c > 0.0 || out != 0)) {
            // nothing is left: the target's own row
            c = 0.0;
            out = 0;
            return empty = true;
        }
        return false;
    };
    if (warp == 0) children = children_of(-1);
    for (;;) {
        if (warp == 0) {
            const bool more = walk();
            if (lane == 0) {
                s_pass.more = more;
                s_pass.node = at;
                s_pass.ch = (float)c;
                s_pass.cl = (float)(c - (double)(float)c);
                s_pass.refused = out;
            }
        }
        __syncthreads();
        cur = s_pass.node;
        ch = s_pass.ch;
        cl = s_pass.cl;
        refused = s_pass.refused;
        p_row = target + (int64_t)(cur + 1) * a.target_row;
        if (draft) q_row = draft + (int64_t)(cur + 1) * a.draft_row;
        if (!s_pass.more) break;
        total = sum_up();
        if (warp == 0 && draft) R = (double)total * 0x1p-60;
    }
    if (rank == 0 && warp == 0) {
        for (int i = count + lane; i < a.tokens; i += 32) a.path[(int64_t)seq * a.tokens + i] = -1;
        if (lane == 0) a.counts[seq] = count;
    }
    if (total <= 0) return;
    // the lowest entry whose sum passes `past`
    const long long past = min(__double2ll_rd((double)s_u[a.tokens] * (double)total), total - 1);
    const long long* sums = s_sums[(passes - 1) & 1];
    long long before = 0;
    for (int i = 0; i < rank; ++i) before += sums[i];
    for (int i = 0; i < warp; ++i) before += s_warp[i];
    if (past < before || past >= before + s_warp[warp]) return;
    int last = v0;                                           // the last entry that is not 0
    for (int i0 = v0; i0 < v1; i0 += 32) {
        const int v = i0 + lane;
        long long upto = 0;
        if (v < v1 && !refused_token(v)) {
            const float p = fits ? fmaxf(p_buf[p_off + v - v0], 0.f) : weight(p_row + v);
            const float q = !(ch > 0.f) ? 0.f : fits ? fmaxf(q_buf[q_off + v - v0], 0.f) : weight(q_row + v);
            upto = units_of(p, q, ch > 0.f, ch, cl);
        }
        const unsigned some = __ballot_sync(0xffffffffu, upto > 0);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + upto > past);
        if (hit) {
            last = i0 + __ffs((int)hit) - 1;
            break;
        }
        if (some) last = i0 + 31 - __clz((int)some);
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    // (where the entries are no probabilities and their sums end below the warp's: the last)
    if (lane == 0) a.next[seq] = last;
}

cudaError_t launch_verify(const statekv_verify_args& a, int dev, int sms, cudaStream_t st) {
    VerifyKernelArgs ka{};
    ka.a = a;
    // as many CTAs per sequence as run at once (clusters of 16 do not fill the
    // device), with four entries a thread at least
    int c = 1;
    while (c < kMaxCluster && (int64_t)a.sequences * c * 2 <= (c < 8 ? sms : sms / 2) &&
           a.vocab > c * 2 * kVerifyThreads * 2)
        c *= 2;
    ka.cluster = c;
    ka.run = (int)(((int64_t)a.vocab + c * kVerifyWarps * 32 - 1) / (c * kVerifyWarps * 32) * 32);
    // room for the whole run where that leaves the device one CTA per SM, else
    // for two CTAs on each
    const int most = (int64_t)a.sequences * c <= sms ? kRoomAlone : kRoomShared;
    ka.room = std::min(ka.run + 8, most);                    // (a run is a multiple of 32)
    const int bytes = kVerifyWarps * 2 * ka.room * 4;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(&verify_kernel), kVerifyWarps * 2 * kRoomAlone * 4, dev, done);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> wide{0};
    if (c > 8) {
        const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
        if (!(wide.load(std::memory_order_relaxed) & bit)) {
            e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&verify_kernel),
                                                       cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            wide.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.sequences * c));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel, ka);
}

}  // namespace
}  // namespace statekv

extern "C" int statekv_verify_tree(const statekv_verify_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_verify_args& a = *args;
    if (a.sequences < 0 || a.tokens < 1 || a.vocab < 1 || !rows_ok(a.tree_stride, a.tokens))
        return STATEKV_E_INVALID_ARG;
    if (a.tokens > kMaxNodes || a.vocab >= 1 << 26 || a.sequences > 0x7fffffff / kMaxCluster)
        return STATEKV_E_UNSUPPORTED;
    if (!a.status || !ints_ok(a.status) || !ints_ok(a.target) || !ints_ok(a.draft) || !ints_ok(a.drafted) ||
        !ints_ok(a.uniforms) || !ints_ok(a.path) || !ints_ok(a.counts) || !ints_ok(a.next) ||
        reinterpret_cast<uintptr_t>(a.tree) % 8)
        return STATEKV_E_INVALID_ARG;
    if (a.target_stride < 0 || a.target_row < 0 || a.draft_stride < 0 || a.draft_row < 0) return STATEKV_E_INVALID_ARG;
    if (a.sequences == 0) return STATEKV_OK;
    if (!a.target || !a.drafted || !a.tree || !a.uniforms || !a.path || !a.counts || !a.next)
        return STATEKV_E_INVALID_ARG;
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return view_cuda_fail();
    return launch_verify(a, dev, sms, reinterpret_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? STATEKV_OK
                                                                                                 : view_cuda_fail();
}
