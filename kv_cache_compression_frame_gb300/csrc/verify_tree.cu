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
// One cluster per sequence, every thread of which follows the same walk; a
// warp sums a contiguous run of the vocabulary.  Bound by latency: a pass moves
// 8 bytes per entry (150001 of them: 1.2 MB, 0.6 us of L2 for a cluster of 8).
//
// Sums decide which token comes out, so they do not depend on how a row is cut:
// p - c q is formed with its rounding error (two-term products and sums), and
// terms are added in pairs of fp32 (to about 2^-48) and then in whole numbers of
// 2^-52.  fp64 adds would do as well at a 64th of the rate.
#include <algorithm>

#include "views.cuh"
#include "sm100_ptx.cuh"

namespace statekv {
namespace {

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxNodes = 64;
constexpr int kMaxCluster = 16;

struct VerifyKernelArgs {
    statekv_verify_args a;
    int32_t cluster;
    int32_t run;                             // entries of a warp, a multiple of 32
};

// a + b = s + e exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
    s = __fadd_rn(a, b);
    const float bb = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb));
}

// max(p - c q, 0) as hi + lo
__device__ __forceinline__ void residual(float p, float q, float ch, float cl, float& hi, float& lo) {
    const float t = __fmul_rn(ch, q), te = __fmaf_rn(ch, q, -t);
    two_sum(p, -t, hi, lo);
    lo = __fsub_rn(__fsub_rn(lo, te), __fmul_rn(cl, q));
    if (!(__fadd_rn(hi, lo) > 0.f)) hi = lo = 0.f;
}

// hi + lo in units of 2^-52
__device__ __forceinline__ long long units_of(float hi, float lo) {
    return __float2ll_rn(hi * 0x1p52f) + __float2ll_rn(lo * 0x1p52f);
}

// NaN and negative values count as 0
__device__ __forceinline__ float weight(const float* p) { return fmaxf(__ldg(p), 0.f); }

__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const __grid_constant__ VerifyKernelArgs ka) {
    const statekv_verify_args& a = ka.a;
    __shared__ int s_parent[kMaxNodes], s_token[kMaxNodes];  // token -1: out of range
    __shared__ float s_p[kMaxNodes], s_q[kMaxNodes], s_u[kMaxNodes + 1];
    __shared__ long long s_warp[kVerifyWarps];
    __shared__ long long s_sums[2][kMaxCluster];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = ka.cluster, rank = blockIdx.x % C, seq = blockIdx.x / C;
    const float* target = a.target + seq * a.target_stride;
    const float* draft = a.draft ? a.draft + seq * a.draft_stride : nullptr;
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
    int cur = -1, count = 0, passes = 0;
    double c = 0.0, R = 1.0;
    uint64_t refused = 0;                                    // nodes refused here (without a draft)
    const float* p_row = target;
    const float* q_row = draft;
    // entry v of the residual, without the refused tokens
    auto refused_token = [&](int v) -> bool {
        for (uint64_t b = refused; b; b &= b - 1)
            if (s_token[__ffsll((long long)b) - 1] == v) return true;
        return false;
    };
    auto entry = [&](int v, float ch, float cl, float& hi, float& lo) {
        hi = weight(p_row + v);
        lo = 0.f;
        if (ch > 0.f) residual(hi, weight(q_row + v), ch, cl, hi, lo);
    };
    // the residual's sum in units of 2^-52, its parts in s_warp and s_sums
    auto sum_up = [&]() -> long long {
        const float ch = (float)c, cl = (float)(c - (double)ch);
        float hi = 0.f, lo = 0.f;
        int v = v0 + lane;
        constexpr int UNROLL = 8;
        for (; v + 32 * (UNROLL - 1) < v1; v += 32 * UNROLL) {
            float p[UNROLL], q[UNROLL];
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                p[i] = weight(p_row + v + 32 * i);
                q[i] = ch > 0.f ? weight(q_row + v + 32 * i) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                float h = p[i], l = 0.f, e;
                if (ch > 0.f) residual(p[i], q[i], ch, cl, h, l);
                two_sum(hi, h, hi, e);
                lo = __fadd_rn(lo, __fadd_rn(l, e));
            }
        }
        for (; v < v1; v += 32) {
            float h, l, e;
            entry(v, ch, cl, h, l);
            two_sum(hi, h, hi, e);
            lo = __fadd_rn(lo, __fadd_rn(l, e));
        }
        long long sum = units_of(hi, lo);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) {
            // each refused token once: that of a node no other refused node below has
            for (uint64_t b = refused; b; b &= b - 1) {
                const int i = __ffsll((long long)b) - 1, x = s_token[i];
                bool again = false;
                for (uint64_t e = refused & ((1ull << i) - 1ull); e; e &= e - 1)
                    again |= s_token[__ffsll((long long)e) - 1] == x;
                if (!again && x >= v0 && x < v1) sum -= units_of(s_p[i], 0.f);
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

    // "every CTA of the cluster has started", before its memory is written
    ptx::cluster_sync();
    bool summed = false;
    long long total = 0;
    for (int i = 0; i < a.tokens; ++i) {
        if (s_parent[i] != cur) continue;
        const double p = s_p[i], q = s_q[i], u = s_u[i];
        double r;
        bool stands;
        if (draft) {
            r = fmax(p - c * q, 0.0);
            stands = u * q * R < r;
        } else {
            r = s_token[i] >= 0 && refused_token(s_token[i]) ? 0.0 : p;
            stands = u * R < r;
        }
        if (s_token[i] >= 0 && stands) {
            if (rank == 0 && tid == 0) a.path[(int64_t)seq * a.tokens + count] = i;
            ++count;
            cur = i;
            c = 0.0;
            R = 1.0;
            refused = 0;
            summed = false;
            p_row = target + (int64_t)(i + 1) * a.target_row;
            if (draft) q_row = draft + (int64_t)(i + 1) * a.draft_row;
        } else if (draft) {
            c += R;
            total = sum_up();
            R = (double)total * 0x1p-52;
            summed = true;
        } else {
            R = fmax(R - r, 0.0);
            if (s_token[i] >= 0) refused |= 1ull << i;
        }
    }
    if (!summed) total = sum_up();
    if (total <= 0 && (c > 0.0 || refused != 0)) {
        // nothing is left: the target's own row
        c = 0.0;
        refused = 0;
        total = sum_up();
    }
    if (rank == 0) {
        for (int i = count + tid; i < a.tokens; i += kVerifyThreads) a.path[(int64_t)seq * a.tokens + i] = -1;
        if (tid == 0) {
            a.counts[seq] = count;
            if (total <= 0) a.next[seq] = 0;
        }
    }
    if (total <= 0) return;
    // the lowest entry whose sum passes `past`
    const long long past = min((long long)((double)s_u[a.tokens] * (double)total), total - 1);
    const long long* sums = s_sums[(passes - 1) & 1];
    long long before = 0;
    for (int i = 0; i < rank; ++i) before += sums[i];
    for (int i = 0; i < warp; ++i) before += s_warp[i];
    if (past < before || past >= before + s_warp[warp]) return;
    const float ch = (float)c, cl = (float)(c - (double)ch);
    int last = v0;                                           // the last entry that is not 0
    for (int i0 = v0; i0 < v1; i0 += 32) {
        const int v = i0 + lane;
        float hi = 0.f, lo = 0.f;
        if (v < v1 && !refused_token(v)) entry(v, ch, cl, hi, lo);
        long long upto = units_of(hi, lo);
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
    // (where the entries' own sums end below the warp's, by units of 2^-52: the last)
    if (lane == 0) a.next[seq] = last;
}

cudaError_t launch_verify(const statekv_verify_args& a, int dev, int sms, cudaStream_t st) {
    VerifyKernelArgs ka{};
    ka.a = a;
    // as many CTAs per sequence as run at once (clusters of 16 do not fill the
    // device), with four entries a thread at least
    int c = 1;
    while (c < 16 && (int64_t)a.sequences * c * 2 <= (c < 8 ? sms : sms / 2) && a.vocab > c * 2 * kVerifyThreads * 2) c *= 2;
    ka.cluster = c;
    ka.run = (int)(((int64_t)a.vocab + c * kVerifyWarps * 32 - 1) / (c * kVerifyWarps * 32) * 32);
    static std::atomic<uint64_t> wide{0};
    if (c > 8) {
        const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
        if (!(wide.load(std::memory_order_relaxed) & bit)) {
            const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&verify_kernel),
                                                       cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            wide.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.sequences * c));
    cfg.blockDim = dim3(kVerifyThreads);
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
