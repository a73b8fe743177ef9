// Product of 8-bit integer rows and weights with a scale per token and channel (spffn_mm8_forward):
//   y[t][n] = round( a_scale[t] w_scale[n] sum_k A[t][k] W[n][k] + bias[n] )
// The 32-bit integer sum is exact (K <= 131072 products of at most 2^14), so any split of K gives
// the same bits.
#include <new>
#include "spffn_internal.cuh"
#include "../../include/spffn_block.h"

namespace spffn {
namespace {

struct MParams {
    const int8_t *A, *W;
    const float *a_scale, *w_scale;
    const void* bias;
    void* y;
    int64_t lda, ldy;
    int T, K, N;
};

// 64 channels x 64 tokens a CTA, 16 K-words at a time in shared memory, 4 x 4 sums a thread.
template <typename D>
__global__ void __launch_bounds__(256) k_mm8_plain(const MParams p) {
    __shared__ int wa[16][65], ta[16][65];
    const int n0 = blockIdx.x * 64, t0 = blockIdx.y * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int acc[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += 64) {
        for (int i = threadIdx.x; i < 64 * 16; i += 256) {
            const int r = i >> 4, c = i & 15, k = k0 + 4 * c;
            wa[c][r] = n0 + r < p.N && k < p.K ? *reinterpret_cast<const int*>(p.W + (int64_t)(n0 + r) * p.K + k) : 0;
            ta[c][r] = t0 + r < p.T && k < p.K ? *reinterpret_cast<const int*>(p.A + (t0 + r) * p.lda + k) : 0;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 16; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(wa[c][tx + 16 * j], ta[c][ty + 16 * i], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (t >= p.T || n >= p.N) continue;
            float v = (float)acc[i][j] * (p.a_scale[t] * p.w_scale[n]);
            if (p.bias) v += DT<D>::f(static_cast<const D*>(p.bias)[n]);
            static_cast<D*>(p.y)[t * p.ldy + n] = DT<D>::r(v);
        }
}

bool valid(const spffn_mm8_config* c) {
    return c && c->K >= 16 && c->K <= 131072 && c->K % 16 == 0 && c->N >= 1 && c->N <= 262144 && c->max_tokens >= 1 &&
           c->max_tokens <= 1048576 && (c->dtype == SPFFN_F16 || c->dtype == SPFFN_BF16) && c->flags == 0;
}

}  // namespace
}  // namespace spffn

struct spffn_mm8_ctx {
    spffn_mm8_config cfg;
    spffn_mm8_weights w;
    char* ws;
    int device, sms;
};

using namespace spffn;

extern "C" {

size_t spffn_mm8_workspace_bytes(const spffn_mm8_config* cfg) { return valid(cfg) ? kCtlBytes : 0; }

spffn_status spffn_mm8_create(const spffn_mm8_config* cfg, const spffn_mm8_weights* w, void* workspace,
                              size_t workspace_bytes, spffn_mm8_ctx** out) {
    if (!out) return SPFFN_ERR_INVALID_ARG;
    *out = nullptr;
    if (!valid(cfg) || !w || !w->W || !w->w_scale) return SPFFN_ERR_INVALID_ARG;
    if (!aligned_to(w->W, 16) || !aligned_to(w->w_scale, 4) || !aligned_to(w->bias, 2)) return SPFFN_ERR_INVALID_ARG;
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < spffn_mm8_workspace_bytes(cfg))
        return SPFFN_ERR_WORKSPACE;
    spffn_mm8_ctx* c = new (std::nothrow) spffn_mm8_ctx();
    if (!c) return SPFFN_ERR_UNSUPPORTED;
    c->cfg = *cfg;
    c->w = *w;
    c->ws = static_cast<char*>(workspace);
    c->device = 0;
    cudaGetDevice(&c->device);
    cudaGetLastError();
    c->sms = current_sms();
    *out = c;
    return SPFFN_OK;
}

spffn_status spffn_mm8_destroy(spffn_mm8_ctx* ctx) {
    delete ctx;
    return SPFFN_OK;
}

spffn_status spffn_mm8_forward(spffn_mm8_ctx* ctx, const int8_t* A, int64_t lda, const float* a_scale, int32_t T,
                               void* y, int64_t ldy, void* stream) {
    if (!ctx || T < 0 || T > ctx->cfg.max_tokens) return SPFFN_ERR_INVALID_ARG;
    if (T == 0) return SPFFN_OK;
    if (!A || !a_scale || !y || lda < ctx->cfg.K || ldy < ctx->cfg.N || lda % 16) return SPFFN_ERR_INVALID_ARG;
    if (!aligned_to(A, 16) || !aligned_to(a_scale, 4) || !aligned_to(y, 2)) return SPFFN_ERR_INVALID_ARG;
    if (!on_device(ctx->device)) return SPFFN_ERR_INVALID_ARG;
    const MParams p{A, ctx->w.W, a_scale, ctx->w.w_scale, ctx->w.bias, y, lda, ldy, T, ctx->cfg.K, ctx->cfg.N};
    const dim3 grid((p.N + 63) / 64, (T + 63) / 64);
    if (ctx->cfg.dtype == SPFFN_BF16) k_mm8_plain<__nv_bfloat16><<<grid, 256, 0, (cudaStream_t)stream>>>(p);
    else k_mm8_plain<__half><<<grid, 256, 0, (cudaStream_t)stream>>>(p);
    return record_cuda(cudaGetLastError());
}

spffn_status spffn_mm8_last_device_error(spffn_mm8_ctx* ctx, uint32_t* code, void* stream) {
    if (!ctx) return SPFFN_ERR_INVALID_ARG;
    return take_device_error(reinterpret_cast<uint32_t*>(ctx->ws), code, stream);
}

}  // extern "C"
