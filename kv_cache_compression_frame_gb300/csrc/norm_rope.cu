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
// A group of d/(2*VEC) lanes owns one token and kHeads heads of it: cosine and
// sine are computed once per group and used for its heads, whose loads are
// all in flight together.
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

constexpr int kHeads = 4;            // heads of a token per lane group
constexpr int kThreads = 256;

struct NormRopeKernelArgs {
    statekv_norm_rope_args a;
    int32_t chunks;                  // lane groups per token
    int64_t items;                   // batch * tokens * chunks
};

// VEC weights from element `at` on (an aligned multiple of VEC)
template <int VEC>
__device__ __forceinline__ void load_weights(const void* w, int dtype, int64_t at, float (&x)[VEC]) {
    if (dtype == STATEKV_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + at);
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 f = p[i];
            x[4 * i] = f.x; x[4 * i + 1] = f.y; x[4 * i + 2] = f.z; x[4 * i + 3] = f.w;
        }
    } else {
        const uint2* p = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + at);
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const uint2 u = p[i];
            x[4 * i] = __uint_as_float(u.x << 16); x[4 * i + 1] = __uint_as_float(u.x & 0xffff0000u);
            x[4 * i + 2] = __uint_as_float(u.y << 16); x[4 * i + 3] = __uint_as_float(u.y & 0xffff0000u);
        }
    }
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormRopeKernelArgs ka) {
    constexpr int VEC = Row<E>::N, HALF = D / 2, TPR = HALF / VEC;
    const statekv_norm_rope_args& a = ka.a;
    const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / TPR;
    const int j = threadIdx.x % TPR;
    // whole groups leave together: the shuffles below stay within a group
    if (item >= ka.items) return;
    const unsigned group = (TPR == 32 ? 0xffffffffu : ((1u << TPR) - 1u)) << ((threadIdx.x & 31) / TPR * TPR);
    const int64_t token_id = item / ka.chunks;
    const int h0 = (int)(item - token_id * ka.chunks) * kHeads;
    const int64_t n = token_id / a.tokens;
    const int t = (int)(token_id - n * a.tokens);
    const int k0 = j * VEC;
    const int heads = a.q_heads + (a.v.data ? 2 : 1) * a.kv_heads;

    uint4 lo[kHeads], hi[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i;
        if (h < heads) {
            const bool isq = h < a.q_heads, isk = !isq && h < a.q_heads + a.kv_heads;
            const statekv_view& v = isq ? a.q : isk ? a.k : a.v;
            const int hh = isq ? h : isk ? h - a.q_heads : h - a.q_heads - a.kv_heads;
            const E* src = static_cast<const E*>(v.data) + n * v.batch_stride + hh * v.head_stride +
                           t * v.token_stride;
            lo[i] = *reinterpret_cast<const uint4*>(src + k0);
            hi[i] = *reinterpret_cast<const uint4*>(src + HALF + k0);
        }
    }
    const int seq = (int)(n / a.layers);
    const int64_t p = a.position0 +
                      (a.positions ? (int64_t)a.positions[n / a.position_layers * a.position_stride + t] : t);
    float c[VEC], s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const uint64_t turn = (uint64_t)p * turn_fraction(a.omega[k0 + e]);
        // the signed top half: half turns in [-1, 1)
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s[e], &c[e]);
    }
    const int row0 = a.out_rows ? a.out_rows[seq] : 0;
    const bool fits = row0 >= 0 && row0 <= a.out_capacity - a.tokens;
    if (!fits && j == 0 && h0 == 0)
        record_error(a.status, (uint32_t)STATEKV_E_DEVICE, kSiteLength, (uint32_t)row0);
    const int64_t w_row = n % a.weight_rows * D;             // weights of this entry's layer
    float wl[VEC], wh[VEC];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i;
        if (h >= heads) break;
        const bool isq = h < a.q_heads, isk = !isq && h < a.q_heads + a.kv_heads;
        if (isq || isk) {
            float x[VEC], y[VEC];
            Row<E>::unpack(lo[i], x);
            Row<E>::unpack(hi[i], y);
            const void* weight = isq ? a.q_weight : a.k_weight;
            if (weight) {
                if (i == 0 || h == a.q_heads) {              // the first of its kind here
                    load_weights<VEC>(weight, a.weight_dtype, w_row + k0, wl);
                    load_weights<VEC>(weight, a.weight_dtype, w_row + HALF + k0, wh);
                }
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss = fmaf(x[e], x[e], fmaf(y[e], y[e], ss));
#pragma unroll
                for (int off = TPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(group, ss, off);
                const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    x[e] *= r * wl[e];
                    y[e] *= r * wh[e];
                }
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float xr = fmaf(x[e], c[e], -y[e] * s[e]);
                y[e] = fmaf(y[e], c[e], x[e] * s[e]);
                x[e] = xr;
            }
            lo[i] = Row<E>::pack(x);
            hi[i] = Row<E>::pack(y);
        }
        if (!isq && !fits) continue;                         // no such row in K and V's destination
        const statekv_view& v = isq ? a.q_out : isk ? a.k_out : a.v_out;
        const int hh = isq ? h : isk ? h - a.q_heads : h - a.q_heads - a.kv_heads;
        const int64_t row = isq ? t : (int64_t)row0 + t;
        E* dst = static_cast<E*>(v.data) + n * v.batch_stride + hh * v.head_stride + row * v.token_stride;
        *reinterpret_cast<uint4*>(dst + k0) = lo[i];
        *reinterpret_cast<uint4*>(dst + HALF + k0) = hi[i];
    }
}

template <typename E, int D>
cudaError_t launch(const NormRopeKernelArgs& ka, cudaStream_t st) {
    constexpr int TPR = D / 2 / Row<E>::N;
    const int64_t blocks = (ka.items * TPR + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    norm_rope_kernel<E, D><<<(unsigned)blocks, kThreads, 0, st>>>(ka);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const statekv_norm_rope_args& a, cudaStream_t st) {
    NormRopeKernelArgs ka{a, 0, 0};
    const int heads = a.q_heads + (a.v.data ? 2 : 1) * a.kv_heads;
    ka.chunks = (heads + kHeads - 1) / kHeads;
    ka.items = (int64_t)a.batch * a.tokens * ka.chunks;
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
        a.kv_heads < 0 || a.position_stride < 0 || a.position_layers < 1 || a.weight_rows < 1 || a.out_capacity < 0 || !(a.eps >= 0.f))
        return STATEKV_E_INVALID_ARG;
    if (a.head_dim != 64 && a.head_dim != 128) return STATEKV_E_UNSUPPORTED;
    if (!a.status || reinterpret_cast<uintptr_t>(a.status) % 4 || !a.omega ||
        reinterpret_cast<uintptr_t>(a.omega) % 8)
        return STATEKV_E_INVALID_ARG;
    for (const void* w : {a.q_weight, a.k_weight})
        if (w && !aligned16(w)) return STATEKV_E_INVALID_ARG;
    const int es = a.dtype == STATEKV_BF16 ? 2 : 4;
    if (a.q_heads > 0 && (!view_ok(a.q, es) || !view_ok(a.q_out, es))) return STATEKV_E_INVALID_ARG;
    if (a.kv_heads > 0) {
        if (!view_ok(a.k, es) || !view_ok(a.k_out, es)) return STATEKV_E_INVALID_ARG;
        if ((a.v.data != nullptr) != (a.v_out.data != nullptr)) return STATEKV_E_INVALID_ARG;
        if (a.v.data && (!view_ok(a.v, es) || !view_ok(a.v_out, es))) return STATEKV_E_INVALID_ARG;
        if (!a.out_rows && a.out_capacity < a.tokens) return STATEKV_E_CAPACITY;
    } else if (a.v.data || a.v_out.data) {
        return STATEKV_E_INVALID_ARG;
    }
    const int64_t heads = (int64_t)a.q_heads + 2ll * a.kv_heads;
    if (heads > 65536) return STATEKV_E_UNSUPPORTED;
    if (a.batch == 0 || a.tokens == 0 || heads == 0) return STATEKV_OK;
    if (launch_norm_rope(a, reinterpret_cast<cudaStream_t>(cuda_stream)) != cudaSuccess)
        return view_cuda_fail();
    return STATEKV_OK;
}
