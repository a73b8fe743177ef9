// The paged 4-bit cache: contexts, appending with rotary positions, reading back
// (declarations and the block format in include/spffn_block.h).
#include <cmath>
#include <new>
#include "spffn_kv4.cuh"

namespace spffn {
namespace kv4 {
namespace {

struct AppendParams {
    const void *q, *k, *v;
    void* q_out;
    int64_t ldq, ldk, ldv, ldqo;
    uint8_t* pool;
    const double* freqs;
    double amp;
    int nh, kvh, rd, inter;
    Batch b;
};

// Codes of 8 dims as 4 bytes, low 4 bits first: rint((x - zero) / step) with the correctly rounded quotient.  The
// product with 1 / step is within 16 3 2^-24 = 2.9e-6 of it (numbers up to 16, three roundings of 2^-24), so it gives
// the same code unless it lies within 4e-6 of a half; only there the division is made.
__device__ __forceinline__ uint32_t pack8(const float* x, float step, float zero) {
    if (!(step > 0.f)) return 0;
    const float inv = __fdiv_rn(1.f, step);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = __fsub_rn(x[i], zero);
        float a = __fmul_rn(t, inv), c = rintf(a);
        if (fabsf(fabsf(a - c) - 0.5f) < 4e-6f) c = rintf(__fdiv_rn(t, step));
        w |= (uint32_t)(int)fminf(fmaxf(c, 0.f), 15.f) << (4 * i);
    }
    return w;
}

__device__ __forceinline__ float f16_value(float v) {      // rounded to fp16, kept finite
    return __half2float(__float2half_rn(fminf(fmaxf(v, -65504.f), 65504.f)));
}

// Cosine and sine of pos freq times the amplitude, in fp64 and rounded once to fp32: codes are decided by the rotated
// values, and an fp32 sine's last place moved a few of four million of them to the next code.
__device__ __forceinline__ void angle(int pos, double freq, double amp, float* co, float* si) {
    const double t = (double)pos * freq * 0.15915494309189535;    // turns: 1 / (2 pi)
    double s, c;
    sincospi(2.0 * (t - rint(t)), &s, &c);
    *co = (float)(amp * c);
    *si = (float)(amp * s);
}

// A block takes a row, or a slice of its heads where there are few rows; a thread 8 dims of a head, so a
// group of 32 dims is four neighbouring lanes and a head 4 NG.  VEC: rows in 16-byte pieces and rotated pairs
// in whole pieces; otherwise element by element.
// Bound by latency at few rows (32 rows of 216 heads: 3.6 us) and by instructions at many (4099 rows of 40 + 16
// heads, half of each rotated: 35 us, 3.0 TB/s, warps that issue 74 % of the time; 41 with a division for every code).  Two and four slices a row took 44
// and 56 us there, pieces read ahead of the angles 86 (registers).
// V codes go out as words put together from two groups' lanes: a head's V codes lie in 8 places, and single
// halfwords doubled the stores.
template <typename T, int NG, bool VEC>
__global__ void __launch_bounds__(256) k_append(const AppendParams p) {
    using L = Blk<NG>;
    constexpr int LH = 4 * NG, DH = 32 * NG;                      // lanes of a head
    __shared__ float cs[DH / 2], sn[DH / 2];
    const int t = blockIdx.x;
    if (t == p.b.T) {                    // one block past the rows looks the sequences over, those without a row too
        for (int s = blockIdx.y * blockDim.x + threadIdx.x; s < p.b.B; s += gridDim.y * blockDim.x) seq_of(p.b, s);
        return;
    }
    const int s = seq_of_row(p.b, t);
    if (s < 0) return;
    const Seq sq = seq_of(p.b, s);
    if (!sq.ok || t < sq.row0 || t >= sq.row0 + sq.n) return;
    const int pos = sq.len - sq.n + (t - sq.row0);
    const int page = p.b.table[(int64_t)s * p.b.ldt + (pos >> p.b.page_log)];
    const int hrd = p.rd >> 1;
    for (int i = threadIdx.x; i < hrd; i += blockDim.x) angle(pos, p.freqs[i], p.amp, &cs[i], &sn[i]);
    if (hrd) __syncthreads();
    const bool paged = (unsigned)page < (unsigned)p.b.pages;
    if (!paged && threadIdx.x == 0 && blockIdx.y == 0) latch(p.b.err, ERR_PAGE_RANGE);
    const int q_heads = p.q ? p.nh : 0, heads = q_heads + 2 * p.kvh;
    const int tok = pos & (p.b.page - 1), lt = tok & 15;
    uint8_t* rec0 = p.pool + ((int64_t)page * p.kvh * (p.b.page >> 4) + (tok >> 4)) * L::kBytes;
    const int64_t head_bytes = (int64_t)(p.b.page >> 4) * L::kBytes;
    const int items = heads * LH, lane = threadIdx.x & 31;
    // whole warps go round together: lanes past the end repeat the last item and store nothing
    for (int it0 = blockIdx.y * blockDim.x + (threadIdx.x & ~31); it0 < items; it0 += gridDim.y * blockDim.x) {
        const bool live = it0 + lane < items;
        const int it = live ? it0 + lane : items - 1;
        const int h = it / LH, j = it % LH, e0 = 8 * j;
        const int kind = h < q_heads ? 0 : h < q_heads + p.kvh ? 1 : 2;
        const int hh = kind == 0 ? h : kind == 1 ? h - q_heads : h - q_heads - p.kvh;
        const T* x = (kind == 0 ? static_cast<const T*>(p.q) + t * p.ldq
                                : kind == 1 ? static_cast<const T*>(p.k) + t * p.ldk : static_cast<const T*>(p.v) + t * p.ldv) + (int64_t)hh * DH;
        float v[8];
        if constexpr (VEC) {
            unpack8<T>(*reinterpret_cast<const uint4*>(x + e0), v);
            if (kind < 2 && e0 < p.rd) {
                if (p.inter) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const float co = cs[(e0 + i) >> 1], si = sn[(e0 + i) >> 1], a = v[i], b = v[i + 1];
                        v[i] = __fsub_rn(__fmul_rn(a, co), __fmul_rn(b, si));
                        v[i + 1] = __fadd_rn(__fmul_rn(b, co), __fmul_rn(a, si));
                    }
                } else {
                    const bool second = e0 >= hrd;
                    const int f0 = second ? e0 - hrd : e0;
                    float o[8];
                    unpack8<T>(*reinterpret_cast<const uint4*>(x + (second ? f0 : e0 + hrd)), o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float m = __fmul_rn(v[i], cs[f0 + i]), n = __fmul_rn(o[i], sn[f0 + i]);
                        v[i] = second ? __fadd_rn(m, n) : __fsub_rn(m, n);
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + i;
                float a = DT<T>::f(x[e]);
                if (kind < 2 && e < p.rd) {
                    const int f = p.inter ? e >> 1 : e < hrd ? e : e - hrd;
                    const bool second = p.inter ? e & 1 : e >= hrd;
                    const float o = DT<T>::f(x[p.inter ? e ^ 1 : second ? e - hrd : e + hrd]);
                    const float m = __fmul_rn(a, cs[f]), n = __fmul_rn(o, sn[f]);
                    a = second ? __fadd_rn(m, n) : __fsub_rn(m, n);
                }
                v[i] = a;
            }
        }
        __syncwarp();        // q_out may be q: the loads of a head's lanes (one warp) come before the stores
        if (kind == 0 && live) {
            T* o = static_cast<T*>(p.q_out) + t * p.ldqo + (int64_t)hh * DH + e0;
            T w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = DT<T>::r(v[i]);
            if constexpr (VEC) *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(w);
            else {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = w[i];
            }
        }
        if (__all_sync(0xffffffffu, kind == 0)) continue;
        float lo = v[0], hi = v[0], bad = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
            bad += v[i] * 0.f;
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
            bad += __shfl_xor_sync(0xffffffffu, bad, o);
        }
        const float zero = f16_value(lo), step = bad == 0.f ? f16_value(__fmul_rn(__fsub_rn(hi, lo), 1.f / 15.f)) : __int_as_float(0x7fc00000);
        const uint32_t w = pack8(v, step, zero);
        // lane j's word of the V codes: place r = j / (NG / 2), groups 2 (j % (NG / 2)) and the next
        const int r = j / (NG / 2), g2 = 2 * (j % (NG / 2)), from = (lane & ~(LH - 1)) + 4 * g2 + (r >> 1);
        const uint32_t va = __shfl_sync(0xffffffffu, w, from), vb = __shfl_sync(0xffffffffu, w, from + 4);
        if (!paged || !live || kind == 0) continue;
        const int g = j >> 2, c = j & 3;
        uint8_t* rec = rec0 + hh * head_bytes;
        if (kind == 1) *reinterpret_cast<uint32_t*>(rec + L::k(lt, g, c)) = w;
        else *reinterpret_cast<uint32_t*>(rec + L::v(lt, g2, r)) = __byte_perm(va, vb, r & 1 ? 0x7632 : 0x5410);
        if (c == 0) {
            *reinterpret_cast<__half*>(rec + (kind == 1 ? L::ks(lt, g) : L::vs(lt, g))) = __float2half_rn(step);
            *reinterpret_cast<__half*>(rec + (kind == 1 ? L::kz(lt, g) : L::vz(lt, g))) = __float2half_rn(zero);
        }
    }
}

// A warp takes a block of 16 tokens of one kv head: the block comes into shared memory as it lies, the values go
// out a head's row at a time.  Bound by the bytes written (16 bits a value for 5 read): 32 pages of 16 tokens of 72
// heads in 4.7 us, 5.3 TB/s.
template <typename T, int NG>
__global__ void __launch_bounds__(256) k_read(const uint8_t* pool, const int32_t* ids, int64_t blocks, int kvh, int page_log,
                                              int pages, T* K, T* V, uint32_t* err) {
    using L = Blk<NG>;
    constexpr int LH = 4 * NG, TW = 32 / LH;                      // lanes of a row, rows of a warp at a time
    __shared__ __align__(16) uint8_t buf[8][L::kBytes];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t it = (int64_t)blockIdx.x * 8 + warp;            // (entry of the list, block of the page, kv head)
    if (it >= blocks) return;
    const int h = (int)(it % kvh), blk = (int)(it / kvh) & ((1 << (page_log - 4)) - 1);
    const int64_t i = (it / kvh) >> (page_log - 4);
    const int id = ids[i];
    if ((unsigned)id >= (unsigned)pages) {
        if (lane == 0) latch(err, ERR_PAGE_RANGE);
        return;
    }
    const uint4* src = reinterpret_cast<const uint4*>(pool + ((((int64_t)id * kvh + h) << (page_log - 4)) + blk) * L::kBytes);
    uint8_t* rec = buf[warp];
#pragma unroll
    for (int k = 0; k < (L::kBytes / 16 + 31) / 32; ++k)
        if (k * 32 + lane < L::kBytes / 16) reinterpret_cast<uint4*>(rec)[k * 32 + lane] = __ldg(src + k * 32 + lane);
    __syncwarp();
    const int j = lane % LH, g = j >> 2, c = j & 3;
    auto half_at = [&](int o) { return __half2float(*reinterpret_cast<const __half*>(rec + o)); };
#pragma unroll 4
    for (int lt = lane / LH; lt < 16; lt += TW) {
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(rec + L::k(lt, g, c));
        const uint32_t vw = *reinterpret_cast<const uint16_t*>(rec + L::v(lt, g, 2 * c)) |
                            ((uint32_t)*reinterpret_cast<const uint16_t*>(rec + L::v(lt, g, 2 * c + 1)) << 16);
        const float ks = half_at(L::ks(lt, g)), kz = half_at(L::kz(lt, g)), vs = half_at(L::vs(lt, g)), vz = half_at(L::vz(lt, g));
        T ko[8], vo[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ko[e] = DT<T>::r(fmaf((float)((kw >> (4 * e)) & 15u), ks, kz));
            vo[e] = DT<T>::r(fmaf((float)((vw >> (4 * e)) & 15u), vs, vz));
        }
        const int64_t at = ((((i << page_log) + blk * 16 + lt) * kvh + h) * LH + j) * 8;
        *reinterpret_cast<uint4*>(K + at) = *reinterpret_cast<const uint4*>(ko);
        *reinterpret_cast<uint4*>(V + at) = *reinterpret_cast<const uint4*>(vo);
    }
}

bool valid(const spffn_kv4_config* c) {
    if (!c || c->flags != 0 || c->pages < 1 || c->pages > (1 << 24)) return false;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 && c->page_size != 256) return false;
    if (c->nh < 1 || c->nh > 1024 || c->kvh < 1 || c->nh % c->kvh || c->nh / c->kvh > 64) return false;
    if (c->dh != 64 && c->dh != 128 && c->dh != 256) return false;
    if (c->max_seqs < 1 || c->max_seqs > 4096 || c->max_tokens < 1 || c->max_tokens > 65536) return false;
    if (c->dtype != SPFFN_F16 && c->dtype != SPFFN_BF16) return false;
    if (c->rope_dim < 0 || c->rope_dim > c->dh || c->rope_dim % 2) return false;
    if (c->rope_dim && !(std::isfinite(c->rope_amplitude))) return false;
    return true;
}

bool valid_batch(const spffn_kv4_ctx* c, int T, const int32_t* table, int64_t ldt, int width, const int32_t* lens,
                 const int32_t* start, int B) {
    if (B < 0 || B > c->cfg.max_seqs || T < 0 || T > c->cfg.max_tokens || width < 0) return false;
    if (B == 0 || T == 0) return true;
    return lens && aligned_to(lens, 4) && aligned_to(start, 4) && aligned_to(table, 4) && table && width >= 1 && ldt >= width &&
           (start || T >= B);
}

Batch batch_of(const spffn_kv4_ctx* c, int T, const int32_t* table, int64_t ldt, int width, const int32_t* lens,
               const int32_t* start, int B) {
    Batch b;
    b.table = table;
    b.lens = lens;
    b.start = start;
    b.ldt = ldt;
    b.width = width;
    b.B = B;
    b.T = T;
    b.page = c->cfg.page_size;
    b.page_log = 0;
    while ((1 << b.page_log) < b.page) ++b.page_log;
    b.pages = c->cfg.pages;
    b.err = c->err();
    return b;
}

}  // namespace
}  // namespace kv4
}  // namespace spffn

using namespace spffn;
using namespace spffn::kv4;

extern "C" {

spffn_status spffn_rope_frequencies(int32_t rope_dim, double base, int32_t scaling, double factor, double original_len,
                                    double* out, double* amplitude) {
    if (rope_dim < 2 || rope_dim % 2 || !out || !(base > 0) || !std::isfinite(base)) return SPFFN_ERR_INVALID_ARG;
    if (scaling < SPFFN_ROPE_PLAIN || scaling > SPFFN_ROPE_PARTS) return SPFFN_ERR_INVALID_ARG;
    if (scaling != SPFFN_ROPE_PLAIN && !(factor >= 1 && std::isfinite(factor))) return SPFFN_ERR_INVALID_ARG;
    if (scaling == SPFFN_ROPE_NTK && rope_dim < 4) return SPFFN_ERR_INVALID_ARG;
    if (scaling == SPFFN_ROPE_PARTS && !(original_len >= 1 && std::isfinite(original_len))) return SPFFN_ERR_INVALID_ARG;
    if (scaling == SPFFN_ROPE_NTK) base *= std::pow(factor, (double)rope_dim / (rope_dim - 2));
    for (int i = 0; i < rope_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rope_dim);
        if (scaling == SPFFN_ROPE_LINEAR) f /= factor;
        if (scaling == SPFFN_ROPE_PARTS) {
            const double turns = original_len * f / (2 * 3.14159265358979323846);
            const double keep = std::min(1.0, std::max(0.0, (turns - 1.0) / 31.0));
            f = f / factor * (1 - keep) + f * keep;
        }
        out[i] = f;
    }
    if (amplitude) *amplitude = scaling == SPFFN_ROPE_PARTS ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return SPFFN_OK;
}

size_t spffn_kv4_pool_bytes(const spffn_kv4_config* c) {
    if (!valid(c)) return 0;
    return (size_t)c->pages * c->kvh * (c->page_size / 16) * (20 * c->dh);
}

size_t spffn_kv4_workspace_bytes(const spffn_kv4_config* c) { return valid(c) ? layout(*c, current_sms()).total : 0; }

spffn_status spffn_kv4_create(const spffn_kv4_config* cfg, void* pool, size_t pool_bytes, const double* rope_freqs,
                              void* workspace, size_t workspace_bytes, spffn_kv4_ctx** out) {
    if (!out) return SPFFN_ERR_INVALID_ARG;
    *out = nullptr;
    if (!valid(cfg) || !pool || !aligned_to(pool, 256) || pool_bytes < spffn_kv4_pool_bytes(cfg)) return SPFFN_ERR_INVALID_ARG;
    if (cfg->rope_dim && (!rope_freqs || !aligned_to(rope_freqs, 8))) return SPFFN_ERR_INVALID_ARG;
    const kv4::Layout lay = layout(*cfg, current_sms());
    if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < lay.total) return SPFFN_ERR_WORKSPACE;
    spffn_kv4_ctx* c = new (std::nothrow) spffn_kv4_ctx();
    if (!c) return SPFFN_ERR_UNSUPPORTED;
    c->cfg = *cfg;
    c->pool = static_cast<uint8_t*>(pool);
    c->freqs = rope_freqs;
    c->ws = static_cast<char*>(workspace);
    c->lay = lay;
    c->device = 0;
    cudaGetDevice(&c->device);
    cudaGetLastError();
    c->sms = current_sms();
    *out = c;
    return SPFFN_OK;
}

spffn_status spffn_kv4_destroy(spffn_kv4_ctx* ctx) {
    delete ctx;
    return SPFFN_OK;
}

spffn_status spffn_kv4_append(spffn_kv4_ctx* ctx, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                              int64_t ldv, int32_t T, const int32_t* table, int64_t ld_table, int32_t width,
                              const int32_t* lens, const int32_t* q_start, int32_t B, void* q_out, int64_t ldqo,
                              void* stream) {
    if (!ctx || !valid_batch(ctx, T, table, ld_table, width, lens, q_start, B)) return SPFFN_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return SPFFN_OK;
    const auto& c = ctx->cfg;
    const int64_t qw = (int64_t)c.nh * c.dh, kw = (int64_t)c.kvh * c.dh;
    if (!k || !v || (!q != !q_out) || ldk < kw || ldv < kw || (q && (ldq < qw || ldqo < qw))) return SPFFN_ERR_INVALID_ARG;
    if (!aligned_to(q, 2) || !aligned_to(k, 2) || !aligned_to(v, 2) || !aligned_to(q_out, 2)) return SPFFN_ERR_INVALID_ARG;
    if (q && q == q_out && ldq != ldqo) return SPFFN_ERR_INVALID_ARG;
    if (!on_device(ctx->device)) return SPFFN_ERR_INVALID_ARG;
    AppendParams p{q, k, v, q_out, ldq, ldk, ldv, ldqo, ctx->pool, ctx->freqs, c.rope_amplitude, c.nh, c.kvh,
                   c.rope_dim, c.rope_interleaved != 0, batch_of(ctx, T, table, ld_table, width, lens, q_start, B)};
    // slices of a row where the rows alone do not fill the device (8 blocks an SM, two rounds)
    const int items = ((q ? c.nh : 0) + 2 * c.kvh) * (c.dh / 8);
    const dim3 grid(T + 1, std::max(1, std::min((items + 255) / 256, 16 * ctx->sms / T)));
    auto row16 = [](const void* x, int64_t ld) { return aligned_to(x, 16) && ld % 8 == 0; };
    const bool vec = row16(q, ldq) && row16(q_out, ldqo) && row16(k, ldk) && row16(v, ldv) && c.rope_dim % (c.rope_interleaved ? 8 : 16) == 0;
    cudaStream_t st = (cudaStream_t)stream;
    auto go = [&](auto tag, auto ng) {
        using T_ = decltype(tag);
        if (vec) k_append<T_, decltype(ng)::value, true><<<grid, 256, 0, st>>>(p);
        else k_append<T_, decltype(ng)::value, false><<<grid, 256, 0, st>>>(p);
    };
    auto by_ng = [&](auto tag) {
        if (c.dh == 64) go(tag, std::integral_constant<int, 2>());
        else if (c.dh == 128) go(tag, std::integral_constant<int, 4>());
        else go(tag, std::integral_constant<int, 8>());
    };
    if (c.dtype == SPFFN_BF16) by_ng(__nv_bfloat16());
    else by_ng(__half());
    return record_cuda(cudaGetLastError());
}

spffn_status spffn_kv4_attend(spffn_kv4_ctx* ctx, const void* q, int64_t ldq, int32_t T, const int32_t* table,
                              int64_t ld_table, int32_t width, const int32_t* lens, const int32_t* q_start, int32_t B,
                              float scale, void* out, int64_t ldo, void* stream) {
    if (!ctx || !valid_batch(ctx, T, table, ld_table, width, lens, q_start, B)) return SPFFN_ERR_INVALID_ARG;
    if (!std::isfinite(scale)) return SPFFN_ERR_INVALID_ARG;
    if (T == 0 || B == 0) return SPFFN_OK;
    const int64_t qw = (int64_t)ctx->cfg.nh * ctx->cfg.dh;
    if (!q || !out || q == out || ldq < qw || ldo < qw || !aligned_to(q, 2) || !aligned_to(out, 2)) return SPFFN_ERR_INVALID_ARG;
    if (!on_device(ctx->device)) return SPFFN_ERR_INVALID_ARG;
    const AttendArgs a{q, out, ldq, ldo, scale, batch_of(ctx, T, table, ld_table, width, lens, q_start, B)};
    return record_cuda(launch_attend(*ctx, a, (cudaStream_t)stream));
}

spffn_status spffn_kv4_read(spffn_kv4_ctx* ctx, const int32_t* page_ids, int32_t n, void* K, void* V, void* stream) {
    if (!ctx || n < 0) return SPFFN_ERR_INVALID_ARG;
    if (n == 0) return SPFFN_OK;
    if (!page_ids || !K || !V || K == V || !aligned_to(page_ids, 4) || !aligned_to(K, 16) || !aligned_to(V, 16)) return SPFFN_ERR_INVALID_ARG;
    if (!on_device(ctx->device)) return SPFFN_ERR_INVALID_ARG;
    const auto& c = ctx->cfg;
    const int64_t blocks = (int64_t)n * (c.page_size / 16) * c.kvh;
    if ((blocks + 7) / 8 > 0x7fffffffLL) return SPFFN_ERR_INVALID_ARG;
    const unsigned grid = (unsigned)((blocks + 7) / 8);
    int page_log = 4;
    while ((1 << page_log) < c.page_size) ++page_log;
    cudaStream_t st = (cudaStream_t)stream;
    auto go = [&](auto tag, auto ng) {
        using T = decltype(tag);
        k_read<T, decltype(ng)::value><<<grid, 256, 0, st>>>(ctx->pool, page_ids, blocks, c.kvh, page_log, c.pages,
                                                             static_cast<T*>(K), static_cast<T*>(V), ctx->err());
    };
    auto by_ng = [&](auto tag) {
        if (c.dh == 64) go(tag, std::integral_constant<int, 2>());
        else if (c.dh == 128) go(tag, std::integral_constant<int, 4>());
        else go(tag, std::integral_constant<int, 8>());
    };
    if (c.dtype == SPFFN_BF16) by_ng(__nv_bfloat16());
    else by_ng(__half());
    return record_cuda(cudaGetLastError());
}

spffn_status spffn_kv4_last_device_error(spffn_kv4_ctx* ctx, uint32_t* code, void* stream) {
    if (!ctx || !on_device(ctx->device)) return SPFFN_ERR_INVALID_ARG;
    return take_device_error(ctx->err(), code, stream);
}

}  // extern "C"
