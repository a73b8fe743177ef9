// Attention over the paged 4-bit cache (spffn_kv4_attend in include/spffn_block.h).
#include "spffn_kv4.cuh"

namespace spffn {
namespace kv4 {
namespace {

struct KParams {
    AttendArgs a;
    const uint8_t* pool;
    int nh, kvh;
};

// One warp per (row, query head): one pass over the row's positions with the running maximum and sum.
// Lane l holds dims l, l + 32, ...
template <typename T, int NG>
__global__ void __launch_bounds__(128) k_attend_plain(const KParams p) {
    using L = Blk<NG>;
    const Batch& b = p.a.b;
    const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    const int t = (int)(w / p.nh), h = (int)(w % p.nh);
    if (t >= b.T) return;
    const int s = seq_of_row(b, t);
    if (s < 0) return;
    const Seq sq = seq_of(b, s);
    if (t < sq.row0 || t >= sq.row0 + sq.n) return;
    const int keys = sq.ok ? sq.len - sq.n + (t - sq.row0) + 1 : 0;
    const int hk = h / (p.nh / p.kvh);
    const T* q = static_cast<const T*>(p.a.q) + t * p.a.ldq + (int64_t)h * (32 * NG);
    float qv[NG], o[NG], m = -INFINITY, sum = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        qv[g] = DT<T>::f(q[32 * g + lane]) * p.a.scale;
        o[g] = 0.f;
    }
    for (int j = 0; j < keys; ++j) {
        const int page = b.table[s * b.ldt + j / b.page];
        if (page < 0 || page >= b.pages) {
            if (lane == 0) latch(b.err, ERR_PAGE_RANGE);
            continue;
        }
        const int tok = j % b.page, lt = tok & 15;
        const uint8_t* rec = p.pool + (((int64_t)page * p.kvh + hk) * (b.page >> 4) + (tok >> 4)) * L::kBytes;
        auto half_at = [&](int off) { return __half2float(*reinterpret_cast<const __half*>(rec + off)); };
        float dot = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int code = (rec[L::k(lt, g, lane >> 3) + ((lane & 7) >> 1)] >> (4 * (lane & 1))) & 15;
            dot += qv[g] * fmaf((float)code, half_at(L::ks(lt, g)), half_at(L::kz(lt, g)));
        }
        dot = warp_sum(dot);
        const float mn = fmaxf(m, dot), f = m == -INFINITY ? 0.f : __expf(m - mn), pr = __expf(dot - mn);
        sum = sum * f + pr;
        m = mn;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int code = (rec[L::v(lt, g, lane >> 2) + ((lane & 3) >> 1)] >> (4 * (lane & 1))) & 15;
            o[g] = o[g] * f + pr * fmaf((float)code, half_at(L::vs(lt, g)), half_at(L::vz(lt, g)));
        }
    }
    T* out = static_cast<T*>(p.a.out) + t * p.a.ldo + (int64_t)h * (32 * NG);
#pragma unroll
    for (int g = 0; g < NG; ++g) out[32 * g + lane] = DT<T>::r(sum == 0.f ? 0.f : o[g] / sum);
}

}  // namespace

Layout layout(const spffn_kv4_config& c, int sms) {
    Layout l;
    l.ctl = 0;
    l.tickets = kCtlBytes;
    l.part = kCtlBytes;
    l.total = kCtlBytes;
    return l;
}

cudaError_t launch_attend(const spffn_kv4_ctx& c, const AttendArgs& a, cudaStream_t st) {
    const KParams p{a, c.pool, c.cfg.nh, c.cfg.kvh};
    const int64_t warps = (int64_t)a.b.T * c.cfg.nh;
    const unsigned grid = (unsigned)((warps + 3) / 4);
    auto go = [&](auto tag) {
        using T = decltype(tag);
        if (c.cfg.dh == 64) k_attend_plain<T, 2><<<grid, 128, 0, st>>>(p);
        else if (c.cfg.dh == 128) k_attend_plain<T, 4><<<grid, 128, 0, st>>>(p);
        else k_attend_plain<T, 8><<<grid, 128, 0, st>>>(p);
    };
    if (c.cfg.dtype == SPFFN_BF16) go(__nv_bfloat16());
    else go(__half());
    return cudaGetLastError();
}

}  // namespace kv4
}  // namespace spffn
