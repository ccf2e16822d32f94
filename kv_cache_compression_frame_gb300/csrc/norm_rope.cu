// RMS norm of every query and key head, rotation at the token's virtual
// position and the store of Q, K and V where their readers want them, in one
// pass.  Qwen3-VL normalises the heads of Q and K before it rotates them;
// StateKV ("Linear Scaling Video VLMs for Long Video Understanding",
// 关键设计 3) rotates at the logical position in the stream.
//
//   y = x * w / sqrt(mean(x^2) + eps)             (fp32)
//   out_k        = y_k cos(a_k) - y_{k+d/2} sin(a_k)
//   out_{k+d/2}  = y_{k+d/2} cos(a_k) + y_k sin(a_k),  a_k = p * omega_k
//
// rounded once, at the store.  Every value is read once and written once: the
// kernel is bound by HBM, or by the launch for a token or two.
//
// The angle.  p * omega in fp32 is off by 1e-2 rad at p = 1.3e5, and fp64
// arithmetic runs at 1/64 of the fp32 rate here.  So omega_k becomes a
// fraction of a turn in 64-bit fixed point, f_k = omega_k / (2 pi) * 2^64 mod
// 2^64, and p * f_k mod 2^64 (one integer multiplication) is the angle's
// fraction of a turn, off by at most p * 2^-53 relative to omega's own
// rounding.  Its top 32 bits go to sincospif.
//
// A CTA has up to kTokens tokens of one batch entry with all their heads.
// It computes the tokens' cosines and sines and the layer's weights once into
// shared memory; then d/(2*VEC) lanes take a row (a head of a token) at a
// time, two rows of loads in flight.  (With the angles in the registers of
// the lanes that own a token, computed for 4 heads each, they were 40 % of the
// instructions, and 100 registers a thread left a quarter of the warps: 78 us
// for 16384 tokens of 32 heads of 128, now 49 us; the bytes take 40 us.)
#include "views.cuh"

namespace statekv {
namespace {

// omega / (2 pi) as a 64-bit fraction of a turn.  With omega = M * 2^(e-63),
// 2^63 <= M < 2^64, the fraction is M * 2^e / pi.
__device__ __forceinline__ uint64_t turn_fraction(double omega) {
    const uint64_t bits = (uint64_t)__double_as_longlong(omega);
    const int e = (int)((bits >> 52) & 0x7ff) - 1023;
    const uint64_t m = ((bits & 0xfffffffffffffull) | (1ull << 52)) << 11;
    uint64_t f = __umul64hi(m, 0x517cc1b727220a94ull);      // 2^64 / pi
    f = e > 63 || e < -63 ? 0ull : e >= 0 ? f << e : f >> -e;
    return (bits >> 63) ? 0ull - f : f;
}

template <typename E> struct Row;
template <> struct Row<__nv_bfloat16> {
    static constexpr int N = 8;                              // values per 16 bytes
    __device__ static void unpack(uint4 u, float (&x)[N]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    }
    __device__ static uint4 pack(const float (&x)[N]) {
        uint4 u;
        __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) h[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        return u;
    }
};
template <> struct Row<float> {
    static constexpr int N = 4;
    __device__ static void unpack(uint4 u, float (&x)[N]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    __device__ static uint4 pack(const float (&x)[N]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};

constexpr int kTokens = 8;           // most tokens of a CTA
constexpr int kThreads = 256;
constexpr int kCtas = 5;             // per SM (4: 50.5 us for the batch above, 6 with one row in flight: 52)
constexpr int kRowsInFlight = 2;     // of a row's lanes

struct NormRopeKernelArgs {
    statekv_norm_rope_args a;
    int32_t heads;                   // of Q, K and V together
    uint32_t inv_heads;              // floor(2^32 / heads) + 1
    int32_t tokens;                  // of a CTA
    int32_t blocks;                  // CTAs per batch entry
};

__device__ __forceinline__ float weight_at(const void* w, int dtype, int64_t k) {
    return dtype == STATEKV_F32 ? static_cast<const float*>(w)[k]
                                : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[k]);
}

// Where element k of a half row sits in the shared tables: lane j of a row has
// elements j * VEC ..; their 16-byte pieces of one index lie side by side for
// consecutive lanes, so that a load has no bank conflict.
template <int VEC, int HALF>
__device__ __forceinline__ int table_at(int k) {
    const int j = k / VEC, e = k % VEC;
    return e / 4 * (HALF / VEC * 4) + j * 4 + e % 4;
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, kCtas) norm_rope_kernel(const __grid_constant__ NormRopeKernelArgs ka) {
    constexpr int VEC = Row<E>::N, HALF = D / 2, TPR = HALF / VEC;
    constexpr int STEP = kThreads / TPR;                     // rows at a time
    const statekv_norm_rope_args& a = ka.a;
    // cosines and sines apart, so that a lane's VEC values of each are 16-byte loads
    __shared__ __align__(16) float s_cos[kTokens][HALF], s_sin[kTokens][HALF], s_w[2][2][HALF];
    const int64_t n = blockIdx.x / ka.blocks;
    const int t0 = (int)(blockIdx.x - n * ka.blocks) * ka.tokens;
    const int nt = min(ka.tokens, a.tokens - t0);
    const int seq = (int)(n / a.layers);
    for (int i = threadIdx.x; i < nt * HALF; i += kThreads) {
        const int t = i / HALF, k = i % HALF;
        const int64_t p = a.position0 +
                          (a.positions ? (int64_t)a.positions[n / a.position_layers * a.position_stride + t0 + t]
                                       : t0 + t);
        const uint64_t turn = (uint64_t)p * turn_fraction(a.omega[k]);
        // the signed top half: half turns in [-1, 1)
        const int at = table_at<VEC, HALF>(k);
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s_sin[t][at], &s_cos[t][at]);
    }
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        const void* w = i < D ? a.q_weight : a.k_weight;
        const int k = i % D;
        if (w)
            s_w[i / D][k / HALF][table_at<VEC, HALF>(k % HALF)] =
                weight_at(w, a.weight_dtype, n % a.weight_rows * D + k);
    }
    const int row0 = a.out_rows ? a.out_rows[seq] : 0;
    const bool fits = row0 >= 0 && row0 <= a.out_capacity - a.tokens;
    if (!fits && threadIdx.x == 0 && t0 == 0 && a.kv_heads > 0)
        record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteLength, (uint32_t)row0);
    __syncthreads();
    const int j = threadIdx.x % TPR, k0 = j * VEC;
    const unsigned group = (TPR == 32 ? 0xffffffffu : ((1u << TPR) - 1u)) << ((threadIdx.x & 31) / TPR * TPR);
    const int rows = nt * ka.heads;
    constexpr int U = kRowsInFlight;
    // (a row's lanes leave together: the shuffles below stay within them)
    for (int r0 = threadIdx.x / TPR; r0 < rows; r0 += U * STEP) {
        uint4 lo[U], hi[U];
        int kind[U], head[U], tok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = min(r0 + u * STEP, rows - 1);
            // r < 2^32 / heads: exact
            tok[u] = ka.heads == 1 ? r : (int)__umulhi((uint32_t)r, ka.inv_heads);
            const int h = r - tok[u] * ka.heads;
            kind[u] = h < a.q_heads ? 0 : h < a.q_heads + a.kv_heads ? 1 : 2;
            head[u] = kind[u] == 0 ? h : kind[u] == 1 ? h - a.q_heads : h - a.q_heads - a.kv_heads;
            const statekv_view& v = kind[u] == 0 ? a.q : kind[u] == 1 ? a.k : a.v;
            const E* src = static_cast<const E*>(v.data) + n * v.batch_stride + head[u] * v.head_stride +
                           (t0 + tok[u]) * v.token_stride;
            lo[u] = *reinterpret_cast<const uint4*>(src + k0);
            hi[u] = *reinterpret_cast<const uint4*>(src + HALF + k0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r0 + u * STEP >= rows) break;
            if (kind[u] != 2) {
                float x[VEC], y[VEC];
                Row<E>::unpack(lo[u], x);
                Row<E>::unpack(hi[u], y);
                if (kind[u] == 0 ? a.q_weight != nullptr : a.k_weight != nullptr) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
                    for (int off = TPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(group, ss, off);
                    const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int at = e / 4 * (TPR * 4) + j * 4 + e % 4;
                        x[e] *= r * s_w[kind[u]][0][at];
                        y[e] *= r * s_w[kind[u]][1][at];
                    }
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int at = e / 4 * (TPR * 4) + j * 4 + e % 4;
                    const float c = s_cos[tok[u]][at], s = s_sin[tok[u]][at];
                    const float xr = fmaf(x[e], c, -y[e] * s);
                    y[e] = fmaf(y[e], c, x[e] * s);
                    x[e] = xr;
                }
                lo[u] = Row<E>::pack(x);
                hi[u] = Row<E>::pack(y);
            }
            if (kind[u] != 0 && !fits) continue;             // no such row in K and V's destination
            const statekv_view& v = kind[u] == 0 ? a.q_out : kind[u] == 1 ? a.k_out : a.v_out;
            const int64_t row = (kind[u] == 0 ? 0 : row0) + t0 + tok[u];
            E* dst = static_cast<E*>(v.data) + n * v.batch_stride + head[u] * v.head_stride + row * v.token_stride;
            *reinterpret_cast<uint4*>(dst + k0) = lo[u];
            *reinterpret_cast<uint4*>(dst + HALF + k0) = hi[u];
        }
    }
}

template <typename E, int D>
cudaError_t launch(const NormRopeKernelArgs& ka, cudaStream_t st) {
    const int64_t grid = (int64_t)ka.a.batch * ka.blocks;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
    norm_rope_kernel<E, D><<<(unsigned)grid, kThreads, 0, st>>>(ka);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const statekv_norm_rope_args& a, cudaStream_t st) {
    NormRopeKernelArgs ka{};
    ka.a = a;
    ka.heads = a.q_heads + (a.v.data ? 2 : 1) * a.kv_heads;
    ka.inv_heads = (uint32_t)((1ull << 32) / (uint32_t)ka.heads + 1);
    // as many tokens as share a CTA's tables, as long as every SM has four CTAs
    int dev = 0, sms = 0;
    if (!current_device(&dev, &sms)) return cudaErrorInvalidDevice;
    const int64_t most = (int64_t)a.batch * a.tokens / (4 * sms);
    ka.tokens = (int)(most < 1 ? 1 : most > kTokens ? kTokens : most);
    ka.blocks = (a.tokens + ka.tokens - 1) / ka.tokens;
    if (a.dtype == STATEKV_BF16)
        return a.head_dim == 128 ? launch<__nv_bfloat16, 128>(ka, st) : launch<__nv_bfloat16, 64>(ka, st);
    return a.head_dim == 128 ? launch<float, 128>(ka, st) : launch<float, 64>(ka, st);
}

}  // namespace statekv

extern "C" int statekv_norm_rope(const statekv_norm_rope_args* args, void* cuda_stream) {
    using namespace statekv;
    if (!args) return STATEKV_E_INVALID_ARG;
    const statekv_norm_rope_args& a = *args;
    if (a.dtype != STATEKV_BF16 && a.dtype != STATEKV_F32) return STATEKV_E_INVALID_ARG;
    if (a.weight_dtype != STATEKV_BF16 && a.weight_dtype != STATEKV_F32) return STATEKV_E_INVALID_ARG;
    if (a.batch < 0 || a.layers < 1 || a.batch % a.layers != 0 || a.tokens < 0 || a.q_heads < 0 ||
        a.kv_heads < 0 || a.position_stride < 0 || (a.positions && !rows_ok(a.position_stride, a.tokens)) ||
        a.position_layers < 1 || a.weight_rows < 1 || a.out_capacity < 0 || !(a.eps >= 0.f))
        return STATEKV_E_INVALID_ARG;
    if (a.head_dim != 64 && a.head_dim != 128) return STATEKV_E_UNSUPPORTED;
    if (!a.status || reinterpret_cast<uintptr_t>(a.status) % 4 || !a.omega ||
        reinterpret_cast<uintptr_t>(a.omega) % 8 || !ints_ok(a.positions) || !ints_ok(a.out_rows))
        return STATEKV_E_INVALID_ARG;
    for (const void* w : {a.q_weight, a.k_weight})
        if (w && !aligned16(w)) return STATEKV_E_INVALID_ARG;
    const int64_t heads = (int64_t)a.q_heads + 2ll * a.kv_heads;
    if (heads > 16384) return STATEKV_E_UNSUPPORTED;         // rows of a CTA times heads below 2^32
    if (a.batch == 0 || a.tokens == 0 || heads == 0) return STATEKV_OK;
    const int es = a.dtype == STATEKV_BF16 ? 2 : 4;
    if (a.q_heads > 0 &&
        (!view_ok(a.q, es, a.batch, a.q_heads, a.tokens) || !view_ok(a.q_out, es, a.batch, a.q_heads, a.tokens)))
        return STATEKV_E_INVALID_ARG;
    if (a.kv_heads > 0) {
        if (!view_ok(a.k, es, a.batch, a.kv_heads, a.tokens) ||
            !view_ok(a.k_out, es, a.batch, a.kv_heads, a.out_capacity))
            return STATEKV_E_INVALID_ARG;
        if ((a.v.data != nullptr) != (a.v_out.data != nullptr)) return STATEKV_E_INVALID_ARG;
        if (a.v.data && (!view_ok(a.v, es, a.batch, a.kv_heads, a.tokens) ||
                         !view_ok(a.v_out, es, a.batch, a.kv_heads, a.out_capacity)))
            return STATEKV_E_INVALID_ARG;
        if (!a.out_rows && a.out_capacity < a.tokens) return STATEKV_E_CAPACITY;
    } else if (a.v.data || a.v_out.data) {
        return STATEKV_E_INVALID_ARG;
    }
    if (!apart(a.q_out, a.batch, a.q_heads, a.tokens, a.head_dim) ||
        !apart(a.k_out, a.batch, a.kv_heads, a.out_capacity, a.head_dim) ||
        (a.v.data && !apart(a.v_out, a.batch, a.kv_heads, a.out_capacity, a.head_dim)))
        return STATEKV_E_INVALID_ARG;
    if (launch_norm_rope(a, reinterpret_cast<cudaStream_t>(cuda_stream)) != cudaSuccess)
        return view_cuda_fail();
    return STATEKV_OK;
}
