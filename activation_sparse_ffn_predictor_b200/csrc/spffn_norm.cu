// Residual addition, RMS norm and 8-bit rows (spffn_norm_quant), and 8-bit rows alone
// (spffn_quantize_rows).
//
//   u = x + y, x_out = round(u), w = u g, a = max|w|, rs = 1 / sqrt(mean u^2 + eps),
//   q = rint(w (127 / a)), scale = a rs / 127
// The norm's factor cancels in q, so q needs only the row's maximum: u, w, 127 / a and the
// product each round once in fp32 in a fixed order, and q is the same bits however the sum
// of squares is arranged.
//
// Bound by the bytes of x, y, x_out and q at many rows (8192 rows of 7168, bf16: 79 us, 5.2 TB/s of the 6.56 that a
// copy reaches; reading a row twice took 240), by latency at few (32 rows of 9216: 3.9 us, one block a row).
#include <cmath>
#include "spffn_block.cuh"

namespace spffn {
namespace {

struct NParams {
    const void *x, *y, *g;
    void* x_out;
    int8_t* q;
    float* scale;
    int64_t ldx, ldy, ldo, ldq;
    int T, d;
    float eps;
};

constexpr float kTiny = 1.504632769052528e-36f;   // 2^-119: below it 127 / a overflows fp32

// element i of a row in the storage type or fp32
template <typename T> __device__ __forceinline__ float elem(const T* p, int i) { return DT<T>::f(p[i]); }
template <> __device__ __forceinline__ float elem<float>(const float* p, int i) { return p[i]; }

// the row's sum of squares and maximum over `n` threads (a multiple of 32) of the CTA
__device__ __forceinline__ void row_reduce(float& ss, float& a, float2* red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(ss, a);
    __syncthreads();
    ss = 0.f;
    a = 0.f;
    for (int w = 0; w < warps; ++w) {
        ss += red[w].x;
        a = fmaxf(a, red[w].y);
    }
}

// the factor 127 / a of a row and its scale; a row of zeros or of numbers that are not finite has q = 0
template <bool NORM>
__device__ __forceinline__ float row_factor(float ss, float a, int d, float eps, float* scale) {
    const bool finite = ss < INFINITY && a < INFINITY;     // false for NaN too
    const float rs = NORM ? 1.f / sqrtf(ss / (float)d + eps) : 1.f;
    *scale = !finite ? __int_as_float(0x7fc00000) : a < kTiny ? 0.f : __fmul_rn(a, rs) / 127.f;
    return finite && a >= kTiny ? __fdiv_rn(127.f, a) : 0.f;
}
__device__ __forceinline__ int to_q(float w, float r) {
    return r == 0.f ? 0 : max(-127, min(127, __float2int_rn(__fmul_rn(w, r))));
}

// One CTA per row, any width, stride and alignment: two passes over the row.
template <typename X, typename Y, typename T, bool NORM>
__global__ void __launch_bounds__(256) k_norm_any(const NParams p) {
    __shared__ float2 red[8];
    const int64_t t = blockIdx.x;
    const X* x = static_cast<const X*>(p.x) + t * p.ldx;
    const Y* y = p.y ? static_cast<const Y*>(p.y) + t * p.ldy : nullptr;
    const T* g = static_cast<const T*>(p.g);
    T* xo = p.x_out ? static_cast<T*>(p.x_out) + t * p.ldo : nullptr;
    int8_t* q = p.q + t * p.ldq;
    float ss = 0.f, a = 0.f;
    for (int i = threadIdx.x; i < p.d; i += blockDim.x) {
        float u = elem(x, i);
        if (NORM && y) u = __fadd_rn(u, elem(y, i));
        const float w = NORM && g ? __fmul_rn(u, DT<T>::f(g[i])) : u;
        if (NORM) ss += u * u;
        if (!NORM || g) ss = fmaf(w, 0.f, ss);             // NaN where w is not finite: the maximum drops one
        a = fmaxf(a, fabsf(w));
    }
    row_reduce(ss, a, red);
    float scale;
    const float r = row_factor<NORM>(ss, a, p.d, p.eps, &scale);
    if (threadIdx.x == 0) p.scale[t] = scale;
    for (int i = threadIdx.x; i < p.d; i += blockDim.x) {
        float u = elem(x, i);
        if (NORM && y) u = __fadd_rn(u, elem(y, i));
        const float w = NORM && g ? __fmul_rn(u, DT<T>::f(g[i])) : u;
        q[i] = (int8_t)to_q(w, r);
        if (NORM && xo) xo[i] = DT<T>::r(u);               // each element is read again by this thread only
    }
}

// The wide path: rows in pieces of 8 elements (16-byte loads of the storage type), the row in registers
// between its two passes, so that memory sees every byte once.  NT threads a row, at most 4 pieces a
// thread; a row of up to 1024 elements is one warp's, eight rows a block.
template <typename X> __device__ __forceinline__ void load8(const X* p, float* f) {
    if constexpr (sizeof(X) == 4) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        unpack8<X>(*reinterpret_cast<const uint4*>(p), f);
    }
}

template <typename X, typename Y, typename T, bool NORM, int NT>
__global__ void __launch_bounds__(NT == 32 ? 256 : NT) k_norm_wide(const NParams p) {
    constexpr int V = 4;
    __shared__ float2 red[NT / 32];
    const int64_t t = NT == 32 ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    if (t >= p.T) return;                                  // whole warps, in the one-warp form only
    const int i0 = NT == 32 ? threadIdx.x & 31 : threadIdx.x, pieces = p.d >> 3;
    const X* x = static_cast<const X*>(p.x) + t * p.ldx;
    const Y* y = static_cast<const Y*>(p.y) + t * p.ldy;
    const T* g = static_cast<const T*>(p.g);
    float u[V][8], ss = 0.f, a = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = i0 + v * NT;
        if (i >= pieces) continue;
        load8(x + 8 * i, u[v]);
        if (NORM && p.y) {
            float o[8];
            load8(y + 8 * i, o);
#pragma unroll
            for (int k = 0; k < 8; ++k) u[v][k] = __fadd_rn(u[v][k], o[k]);
        }
    }
    if (NORM && p.x_out) {
        T* xo = static_cast<T*>(p.x_out) + t * p.ldo;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int i = i0 + v * NT;
            if (i >= pieces) continue;
            T o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = DT<T>::r(u[v][k]);
            *reinterpret_cast<uint4*>(xo + 8 * i) = *reinterpret_cast<const uint4*>(o);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = i0 + v * NT;
        if (i >= pieces) continue;
        if (NORM) {
#pragma unroll
            for (int k = 0; k < 8; ++k) ss += u[v][k] * u[v][k];
            if (g) {
                float gv[8];
                load8(g + 8 * i, gv);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    u[v][k] = __fmul_rn(u[v][k], gv[k]);
                    ss = fmaf(u[v][k], 0.f, ss);           // NaN where w is not finite: the maximum drops one
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) ss += u[v][k] * 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) a = fmaxf(a, fabsf(u[v][k]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    }
    if constexpr (NT > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(ss, a);
        __syncthreads();
        ss = 0.f;
        a = 0.f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            ss += red[w].x;
            a = fmaxf(a, red[w].y);
        }
    }
    float scale;
    const float r = row_factor<NORM>(ss, a, p.d, p.eps, &scale);
    if (i0 == 0) p.scale[t] = scale;
    int8_t* q = p.q + t * p.ldq;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int i = i0 + v * NT;
        if (i >= pieces) continue;
        uint32_t b[2] = {0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k) b[k >> 2] |= ((uint32_t)to_q(u[v][k], r) & 255u) << (8 * (k & 3));
        *reinterpret_cast<uint2*>(q + 8 * i) = make_uint2(b[0], b[1]);
    }
}

template <typename X, typename Y, typename T, bool NORM>
cudaError_t launch(const NParams& p, cudaStream_t st) {
    const bool wide = p.d % 8 == 0 && p.d <= 16384 && aligned_to(p.x, 16) && p.ldx % 8 == 0 && aligned_to(p.y, 16) && p.ldy % 8 == 0 &&
                      aligned_to(p.g, 16) && aligned_to(p.x_out, 16) && p.ldo % 8 == 0 && aligned_to(p.q, 8) && p.ldq % 8 == 0;
    if (!wide) k_norm_any<X, Y, T, NORM><<<p.T, 256, 0, st>>>(p);
    else if (p.d <= 1024) k_norm_wide<X, Y, T, NORM, 32><<<(p.T + 7) / 8, 256, 0, st>>>(p);
    else if (p.d <= 4096) k_norm_wide<X, Y, T, NORM, 128><<<p.T, 128, 0, st>>>(p);
    else if (p.d <= 8192) k_norm_wide<X, Y, T, NORM, 256><<<p.T, 256, 0, st>>>(p);
    else k_norm_wide<X, Y, T, NORM, 512><<<p.T, 512, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace spffn

using namespace spffn;

extern "C" {

spffn_status spffn_norm_quant(int32_t T, int32_t d, int32_t dtype, const void* x, int64_t ldx, const void* y,
                              int64_t ldy, int32_t y_f32, const void* g, float eps, void* x_out, int64_t ldo,
                              int8_t* q, int64_t ldq, float* scale, void* stream) {
    if (T < 0 || d < 1 || d > 16384 || (dtype != SPFFN_F16 && dtype != SPFFN_BF16)) return SPFFN_ERR_INVALID_ARG;
    if (!(eps > 0.f) || !(eps < INFINITY)) return SPFFN_ERR_INVALID_ARG;
    if (T == 0) return SPFFN_OK;
    if (!x || !q || !scale || ldx < d || ldq < d || (y && ldy < d) || (x_out && ldo < d)) return SPFFN_ERR_INVALID_ARG;
    if (!aligned_to(x, 2) || !aligned_to(g, 2) || !aligned_to(x_out, 2) || !aligned_to(scale, 4) ||
        !aligned_to(y, y_f32 ? 4 : 2))
        return SPFFN_ERR_INVALID_ARG;
    // in place only element on element: a row of another stride or type would be read after it is written
    if (x_out && x_out == x && ldo != ldx) return SPFFN_ERR_INVALID_ARG;
    if (x_out && x_out == y && (y_f32 || ldo != ldy)) return SPFFN_ERR_INVALID_ARG;
    const NParams p{x, y, g, x_out, q, scale, ldx, ldy, ldo, ldq, T, d, eps};
    cudaStream_t st = (cudaStream_t)stream;
    if (dtype == SPFFN_BF16)
        return record_cuda(y_f32 ? launch<__nv_bfloat16, float, __nv_bfloat16, true>(p, st)
                                 : launch<__nv_bfloat16, __nv_bfloat16, __nv_bfloat16, true>(p, st));
    return record_cuda(y_f32 ? launch<__half, float, __half, true>(p, st) : launch<__half, __half, __half, true>(p, st));
}

spffn_status spffn_quantize_rows(int32_t T, int32_t d, int32_t dtype, const void* x, int64_t ldx, int32_t x_f32,
                                 int8_t* q, int64_t ldq, float* scale, void* stream) {
    if (T < 0 || d < 1 || d > 131072 || (dtype != SPFFN_F16 && dtype != SPFFN_BF16)) return SPFFN_ERR_INVALID_ARG;
    if (T == 0) return SPFFN_OK;
    if (!x || !q || !scale || ldx < d || ldq < d) return SPFFN_ERR_INVALID_ARG;
    if (!aligned_to(x, x_f32 ? 4 : 2) || !aligned_to(scale, 4)) return SPFFN_ERR_INVALID_ARG;
    const NParams p{x, nullptr, nullptr, nullptr, q, scale, ldx, 0, 0, ldq, T, d, 1.f};
    cudaStream_t st = (cudaStream_t)stream;
    if (x_f32) return record_cuda(launch<float, float, __half, false>(p, st));
    return record_cuda(dtype == SPFFN_BF16 ? launch<__nv_bfloat16, float, __nv_bfloat16, false>(p, st)
                                           : launch<__half, float, __half, false>(p, st));
}

}  // extern "C"
