// Product of 8-bit integer rows and weights with a scale per token and channel (spffn_mm8_forward):
//   y[t][n] = round( a_scale[t] w_scale[n] sum_k A[t][k] W[n][k] + bias[n] )
// The 32-bit integer sum is exact (K <= 131072 products of at most 2^14; the one sum of 2^31 is put right at the
// end), so any split of K gives the same bits.
//
// k_mm8: persistent tcgen05 kernel, int8 x int8 into int32 in TMEM.  A tile is 128 channels (the
// MMA's M: lane = channel) x BN tokens (its N, any multiple of 16 up to 256), K in blocks of 128
// bytes: W and A arrive as 2-D TMA tiles of 128-byte rows, 128-byte swizzle, in a ring as deep as
// shared memory allows.  Channels are M at every batch size, so a decode call streams each weight
// once with only its tokens' columns as padding (16), and the output's 32-lane rows are whole sectors.
// Tiles are dealt whole while full waves of CTAs last, or in equal rounds; what is left (at most two waves) is
// one line of K blocks cut into equal shares.  A cut tile's CTAs leave their
// int32 partials in the workspace and count themselves in; the last to arrive adds them: integer sums,
// so the order does not matter, and nobody waits.
//
// PAIR: two CTAs of a cluster make one tile of 256 channels (cta_group::2): each holds 128 channels' rows and
// half of the tokens' rows, so a K block brings 32 KB an SM into shared memory in place of 48 KB (BN = 256),
// and the MMA reads as much less of it.  The even CTA issues for both.
//
// Measured on one B200 (weights and activations from HBM, calls back to back in a graph): 1 token, 12,288
// channels of 4096: 13.9 us; 32 tokens, 9216 of 9216: 20.5 us; 256 tokens, 21,504 of 7168: 43 us; 8192 tokens,
// 9216 of 9216: 515 to 525 us (2.6 to 2.7 P operations/s).  Bound by the weights' bytes up to about 128 tokens: from
// 12,288 to 73,728 channels of 4096 a token takes 6.6 TB/s more, and the line begins at 6 us (launch, first bytes,
// epilogue, the joining of cut tiles).  By the joining of cut tiles at 256 tokens (all of 84 tiles on 74 pairs are cut;
// tensor cores busy 52 % of the time), by the tensor cores (86 %) and the power limit above.
#include <climits>
#include <new>
#include "spffn_umma.cuh"
#include "spffn_block.cuh"

namespace spffn {
namespace {

using namespace um;

constexpr int kTM = 128, kBK = 128, kThreads = 320, kMaxSt = 12;
constexpr int kEpiThreads = 256;      // eight epilogue warps: two for each 32 lanes of TMEM, half the columns each
constexpr int kGroupN = 8;            // channel tiles that share a stretch of the tile order
// Tokens of a tile from which pairs of CTAs take it.  Pairs against single CTAs, us, at 128 / 160 / 176 / 192 / 224 / 256
// tokens: 18,944 channels of 8192 32.1/32.3 33.5/33.5 34.4/34.3 34.6/34.6 35.4/36.0 36.8/38.9; 9216 of 9216 25.0/24.6
// 26.2/25.5 26.9/26.5 26.9/26.6 28.2/28.0 29.7/30.8; 21,504 of 7168 35.4/34.8 37.3/36.4 38.4/37.8 38.8/38.8 40.6/40.8
// 42.7/45.4.  (A pair's launch and barriers cost about 1 us; its smaller traffic into shared memory pays above.)
constexpr int kPairMin = 192;
constexpr int kMinBlocks = 4;         // K blocks of a share, at least
constexpr size_t kSmem = 227 * 1024;

struct MParams {
    CUtensorMap mW, mA;
    const float *a_scale, *w_scale;
    const void* bias;
    void* y;
    int64_t ldy;
    int T, N;
    int two;                          // y in whole pairs of channels
    int kblocks, n_tiles, t_tiles, bn, stages;
    int units;                        // CTAs, or pairs of them
    int whole;                        // tiles per CTA that are dealt whole
    int cut_base, cut_tiles;          // the tiles that are cut, in line
    int4* partial;                    // [2 grid][bn / 4][128 rows] of 4 columns
    uint32_t *tickets, *err;
};

// The pieces of work of one CTA: whole tiles first, then its share of the line, the share's last tile
// before its first: the front part of a cut tile is then in the workspace long before the CTA with the
// tile's end looks for it.
struct Walk {
    long long pos, end;
    int w = 0, cur, stop;             // tiles of the line still to come, from the last to the first
    int tile, k0, k1, cut;            // cut: index of the tile in the line, -1 for a whole one
    int unit;
    __device__ __forceinline__ Walk(const MParams& p, int u) : unit(u) {
        const long long total = (long long)p.cut_tiles * p.kblocks;
        pos = total * u / p.units;
        end = total * (u + 1) / p.units;
        cur = pos < end ? (int)((end - 1) / p.kblocks) : -1;
        stop = pos < end ? (int)(pos / p.kblocks) : 0;
    }
    __device__ __forceinline__ bool next(const MParams& p) {
        if (w < p.whole) {
            tile = w++ * p.units + unit;
            if (tile >= p.n_tiles * p.t_tiles) return false;      // the last round may not be full; nothing is cut then
            k0 = 0;
            k1 = p.kblocks;
            cut = -1;
            return true;
        }
        if (cur < stop) return false;
        cut = cur--;
        tile = p.cut_base + cut;
        const long long lo = (long long)cut * p.kblocks;
        k0 = (int)max(0ll, pos - lo);
        k1 = (int)min((long long)p.kblocks, end - lo);
        if (k0 == 0 && k1 == p.kblocks) cut = -1;
        return true;
    }
};

__device__ __forceinline__ void tile_at(const MParams& p, int tile, int& nt, int& tt) {
    const int per = kGroupN * p.t_tiles, g = tile / per, r = tile % per;
    const int gn = min(kGroupN, p.n_tiles - g * kGroupN);
    nt = g * kGroupN + r % gn;
    tt = r / gn;
}

template <bool PAIR>
__device__ __forceinline__ void umma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
    if constexpr (PAIR) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accum));
        return;
    }
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accum), "r"(0u), "r"(0u), "r"(0u), "r"(0u));
}
__device__ __forceinline__ void tmem_ld16i(uint32_t taddr, int* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// a tile of this CTA's, its arrival counted at the even CTA's barrier
__device__ __forceinline__ void tma_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
        ::"r"(s32(dst)), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
// what was issued so far is done: tell this CTA's barrier, or both CTAs' at the same place
template <bool PAIR> __device__ __forceinline__ void mma_commit(uint64_t* bar) {
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(s32(bar)),
                     "h"((uint16_t)3) : "memory");
    else ucommit(bar);
}
__device__ __forceinline__ void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <bool PAIR> __device__ __forceinline__ void tmem_alloc(uint32_t* slot) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(slot)), "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s32(slot)), "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <bool PAIR> __device__ __forceinline__ void tmem_free(uint32_t tmem) {
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

// the epilogue warps' barrier, and whether all of them say so: they leave a wait together or not at all
__device__ __forceinline__ bool epi_all(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 2, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"((uint32_t)ok) : "memory");
    return r != 0;
}

template <typename D, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) k_mm8(const __grid_constant__ MParams p) {
    extern __shared__ __align__(1024) char smem[];
    char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem) + 1023) & ~uintptr_t(1023));
    const int S = p.stages, BN = p.bn;
    const int AR = PAIR ? BN / 2 : BN;     // token rows of this CTA
    const uint32_t stage_bytes = kTM * kBK + AR * kBK;
    uint64_t* full = reinterpret_cast<uint64_t*>(base + S * stage_bytes);
    uint64_t* empty = full + kMaxSt;
    uint64_t* tfull = empty + kMaxSt;      // [2]
    uint64_t* tempty = tfull + 2;          // [2]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tempty + 2);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 3);
    int* s_lasts = reinterpret_cast<int*>(tempty + 4);       // [2]
    uint64_t* done = tempty + 5;
    float* s_scale = reinterpret_cast<float*>(tempty + 6);   // [2][256]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, rank = PAIR ? blockIdx.x & 1 : 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) { ub_init(&full[i], 1); ub_init(&empty[i], 1); }
        for (int i = 0; i < 2; ++i) { ub_init(&tfull[i], 1); ub_init(&tempty[i], (PAIR ? 2 : 1) * kEpiThreads / 32); }
        ub_init(done, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<PAIR>(tmem_slot);
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();   // the other CTA's barriers are there
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // programmatic dependent launch: what comes before overlaps the previous kernel's end
    pdl_trigger();
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {                   // ------------------------------------ TMA producer
            int st = 0, ph = 0;
            uint32_t issued = 0, last_ph = 0;
            Walk w(p, unit);
            bool ok = true;
            while (ok && w.next(p)) {
                int nt, tt;
                tile_at(p, w.tile, nt, tt);
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    if (!ub_wait(&empty[st], ph ^ 1, abort_flag, p.err)) { ok = false; break; }
                    char* sw = base + st * stage_bytes;
                    if constexpr (PAIR) {
                        const uint32_t bar = cluster_map(s32(&full[st]), 0);
                        if (rank == 0) ub_expect(&full[st], 2 * stage_bytes);
                        tma_2d_pair(sw, &p.mW, kb * kBK, nt * 2 * kTM + rank * kTM, bar);
                        tma_2d_pair(sw + kTM * kBK, &p.mA, kb * kBK, tt * BN + rank * AR, bar);
                    } else {
                        ub_expect(&full[st], stage_bytes);
                        tma_2d(sw, &p.mW, kb * kBK, nt * kTM, &full[st]);
                        tma_2d(sw + kTM * kBK, &p.mA, kb * kBK, tt * BN, &full[st]);
                    }
                    issued |= 1u << st;
                    last_ph = (last_ph & ~(1u << st)) | ((uint32_t)ph << st);
                    if (++st == S) { st = 0; ph ^= 1; }
                }
            }
            // the last fill of every stage has been consumed (of a pair: no arrival from the even CTA is still on
            // its way), or, after an abort, has landed; of a pair the even CTA sees both CTAs' copies, and the
            // other one stays until the cluster's last barrier
            for (int i = 0; i < S; ++i) {
                if (!((issued >> i) & 1u)) continue;
                const uint32_t parity = (last_ph >> i) & 1u;
                if (ub_wait(&empty[i], parity, abort_flag, p.err) || rank) continue;
                const unsigned long long t0 = now_ns();
                while (!ub_try(&full[i], parity) && now_ns() - t0 < 20000000ull) {}
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {      // ------------------------------------ MMA
            const uint32_t idesc = (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)((PAIR ? 2 : 1) * kTM >> 4) << 24);
            int st = 0, ph = 0, ab = 0, aph = 0;
            Walk w(p, unit);
            bool ok = true;
            while (ok && w.next(p)) {
                if (!ub_wait(&tempty[ab], aph ^ 1, abort_flag, p.err)) break;
                tc_fence_after();
                const uint32_t d = tmem + (uint32_t)(ab * 256);
                for (int kb = w.k0; kb < w.k1; ++kb) {
                    if (!ub_wait(&full[st], ph, abort_flag, p.err)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sw = s32(base + st * stage_bytes), sa = sw + kTM * kBK;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_i8<PAIR>(d, sdesc(sw + k * 32u, 1u, 64u), sdesc(sa + k * 32u, 1u, 64u), idesc, kb > w.k0 || k > 0);
                    mma_commit<PAIR>(&empty[st]);
                    if (++st == S) { st = 0; ph ^= 1; }
                }
                if (!ok) break;
                mma_commit<PAIR>(&tfull[ab]);
                if (++ab == 2) { ab = 0; aph ^= 1; }
            }
            if (*abort_flag) {             // what was issued ends before the block does
                mma_commit<PAIR>(done);
                const unsigned long long t0 = now_ns();
                while (!ub_try(done, 0) && now_ns() - t0 < 20000000ull) {}
            }
        }
    } else {                               // ---------------------------------------- epilogue
        const int quad = warp & 3, row = quad * 32 + lane, side = (warp - 2) >> 2;
        int ab = 0, aph = 0;
        Walk w(p, unit);
        while (w.next(p)) {
            int nt, tt;
            tile_at(p, w.tile, nt, tt);
            const int n = (PAIR ? 2 * nt + rank : nt) * kTM + row;
            const bool in = n < p.N;
            const float ws = in ? __ldg(p.w_scale + n) : 0.f;
            const float bias = in && p.bias ? DT<D>::f(static_cast<const D*>(p.bias)[n]) : 0.f;
            const int t0 = tt * BN, cols = min(BN, p.T - t0);
            // the tokens' scales, read back four at a time; the barrier below makes them visible, and two buffers
            // keep the tile before
            float* as = s_scale + 256 * ab;
            // one warp's answer for all eight; a warp may still read it when that one is at the next tile, and the tile
            // between two uses of a word has a barrier of all of them
            int* s_last = s_lasts + ab;
            const int et = threadIdx.x - 64;
            as[et] = et < cols ? __ldg(p.a_scale + t0 + et) : 0.f;
            int c_first = 0, c_last = -1;  // the CTAs (or pairs) of a cut tile
            uint32_t others = 0;           // how many there are beside this one
            uint32_t* ticket = p.tickets + (w.cut < 0 ? 0 : PAIR ? 2 * w.cut + rank : w.cut);
            constexpr int kSides = PAIR ? 2 : 1;
            bool finish = true;
            // pieces of 16 columns, the two warps of a quadrant take turns; a warp finishes 32 columns at a time
            auto part_of = [&](int o, int c0) {      // its piece of this tile starts at 0 only if it is the first
                return p.partial + ((size_t)((2 * o + (o == c_first)) * kSides + rank) * (BN / 4) + c0 / 4) * kTM + row;
            };
            int4 u[8];                     // of the only other part, the next 32 columns ahead
            auto fetch = [&](int o, int c0) {
                const int4* from = part_of(o, c0);
                const bool two = c0 + 32 < cols;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    u[c] = c0 < cols ? __ldcg(from + c * kTM) : make_int4(0, 0, 0, 0);
                    u[c + 4] = two ? __ldcg(from + (c + 8) * kTM) : make_int4(0, 0, 0, 0);
                }
            };
            int other = -1;                // set where there is only one
            if (w.cut >= 0) {
                const long long total = (long long)p.cut_tiles * p.kblocks, lo = (long long)w.cut * p.kblocks;
                c_first = (int)(((lo + 1) * p.units - 1) / total);
                c_last = (int)(((lo + p.kblocks) * p.units - 1) / total);
                others = (uint32_t)(c_last - c_first);
                if (others == 1) other = c_first == unit ? c_last : c_first;
                // where all the others are in, this one's part need not leave TMEM, and theirs can be read meanwhile
                if (threadIdx.x == 64) *s_last = ld_acquire_u32(ticket) == others;
                epi_all(true);
                finish = *s_last;
                if (finish && other >= 0) fetch(other, 16 * side);
            }
            if (!epi_all(ub_wait(&tfull[ab], aph, abort_flag, p.err))) break;
            tc_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(ab * 256);
            if (!finish) {
                if (threadIdx.x == 64) *s_last = ld_acquire_u32(ticket) == others;
                epi_all(true);
                finish = *s_last;
                if (!finish) {
                    int4* mine = p.partial + (size_t)((2 * unit + (w.k0 == 0)) * kSides + rank) * (BN / 4) * kTM + row;
                    for (int c0 = 16 * side; c0 < cols; c0 += 32) {
                        int v[16];
                        __syncwarp();                            // tcgen05.ld is the whole warp's
                        tmem_ld16i(taddr + c0, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            __stcg(mine + (c0 / 4 + c) * kTM, make_int4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]));
                    }
                    epi_all(true);
                    if (threadIdx.x == 64) *s_last = atom_acq_rel_add_u32(ticket, 1u) == others;
                    epi_all(true);
                    finish = *s_last;
                }
                if (finish && other >= 0) fetch(other, 16 * side);
            }
            if (w.cut >= 0 && finish && threadIdx.x == 64) *ticket = 0;      // for the next call
            if (finish) {
                D* y = static_cast<D*>(p.y) + (int64_t)t0 * p.ldy + n;
                for (int c0 = 16 * side; c0 < cols; c0 += 64) {
                    int v[32];
                    const bool two = c0 + 32 < cols;
                    __syncwarp();
                    tmem_ld16i(taddr + c0, v);
                    if (two) tmem_ld16i(taddr + c0 + 32, v + 16);
                    tmem_wait_ld();
                    if (other >= 0) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            v[4 * c] += u[c].x;
                            v[4 * c + 1] += u[c].y;
                            v[4 * c + 2] += u[c].z;
                            v[4 * c + 3] += u[c].w;
                        }
                        fetch(other, c0 + 64);
                    } else {
                        // four parts' loads at a time, 16 columns at a time
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h && !two) break;
                            for (int o = c_first; o <= c_last; o += 4) {
                                int4 w[4][4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const bool there = o + k <= c_last && o + k != unit;
                                    const int4* from = part_of(there ? o + k : c_first, c0 + 32 * h);
#pragma unroll
                                    for (int c = 0; c < 4; ++c) w[k][c] = there ? __ldcg(from + c * kTM) : make_int4(0, 0, 0, 0);
                                }
#pragma unroll
                                for (int k = 0; k < 4; ++k)
#pragma unroll
                                    for (int c = 0; c < 4; ++c) {
                                        v[16 * h + 4 * c] += w[k][c].x;
                                        v[16 * h + 4 * c + 1] += w[k][c].y;
                                        v[16 * h + 4 * c + 2] += w[k][c].z;
                                        v[16 * h + 4 * c + 3] += w[k][c].w;
                                    }
                            }
                        }
                    }
                    // K = 131072 of -128 times -128 is 2^31, which came round to -2^31 (no sum is that low) and is 2^31 in
                    // fp32 again as 2^31 - 1
                    if (p.kblocks == 1024) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) v[c] = v[c] == INT_MIN ? INT_MAX : v[c];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h && !two) break;
                        const int b0 = c0 + 32 * h;
                        float f[16];
#pragma unroll
                        for (int c = 0; c < 16; c += 4) {
                            const float4 a = *reinterpret_cast<const float4*>(as + b0 + c);
                            f[c] = fmaf((float)v[16 * h + c], a.x * ws, bias);
                            f[c + 1] = fmaf((float)v[16 * h + c + 1], a.y * ws, bias);
                            f[c + 2] = fmaf((float)v[16 * h + c + 2], a.z * ws, bias);
                            f[c + 3] = fmaf((float)v[16 * h + c + 3], a.w * ws, bias);
                        }
                        D* to = y + (int64_t)b0 * p.ldy;
                        if (p.two) {
                            // a lane and its neighbour swap, so that each stores two channels of every other column
                            const int odd = lane & 1;
                            uint32_t* to2 = reinterpret_cast<uint32_t*>(to + (int64_t)odd * p.ldy - odd);
#pragma unroll
                            for (int c = 0; c < 16; c += 2) {
                                const float got = __shfl_xor_sync(0xffffffffu, odd ? f[c] : f[c + 1], 1);
                                const D pr[2] = {DT<D>::r(odd ? got : f[c]), DT<D>::r(odd ? f[c + 1] : got)};
                                if (in && b0 + c + odd < cols) *to2 = *reinterpret_cast<const uint32_t*>(pr);
                                to2 += p.ldy;             // two rows, in pairs of channels
                            }
                        } else {
#pragma unroll
                            for (int c = 0; c < 16; ++c) {
                                if (in && b0 + c < cols) *to = DT<D>::r(f[c]);
                                to += p.ldy;
                            }
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (rank == 0) ub_arrive(&tempty[ab]);
                else arrive_at(cluster_map(s32(&tempty[ab]), 0));
            }
            if (++ab == 2) { ab = 0; aph ^= 1; }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (PAIR) cluster_sync_all();   // nothing of the other CTA's is still on its way here
    if (warp == 1) tmem_free<PAIR>(tmem);
}

// [rows][cols] bytes of row stride `ld`, box {128, box_rows}, 128-byte swizzle
bool map_i8(CUtensorMap* m, const void* ptr, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    EncodeTiledFn enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows}, estr[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Layout8 {
    size_t tickets, partial, total;
};
Layout8 layout8(const spffn_mm8_config& c, int sms) {
    Layout8 l;
    l.tickets = kCtlBytes;
    l.partial = align_up(l.tickets + (size_t)2 * sms * sizeof(uint32_t), 256);   // pairs: two a tile of half as many
    l.total = l.partial + (size_t)2 * sms * std::min(256, (c.max_tokens + 31) / 32 * 32) * kTM * sizeof(int);
    return l;
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
    spffn::Layout8 lay;
    int device, sms;
};

using namespace spffn;

extern "C" {

size_t spffn_mm8_workspace_bytes(const spffn_mm8_config* cfg) { return valid(cfg) ? layout8(*cfg, current_sms()).total : 0; }

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
    c->lay = layout8(*cfg, c->sms);
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
    MParams p;
    const auto& c = ctx->cfg;
    p.a_scale = a_scale;
    p.w_scale = ctx->w.w_scale;
    p.bias = ctx->w.bias;
    p.y = y;
    p.ldy = ldy;
    p.T = T;
    p.N = c.N;
    p.two = c.N % 2 == 0 && ldy % 2 == 0 && aligned_to(y, 4);
    p.kblocks = (c.K + kBK - 1) / kBK;
    p.t_tiles = (T + 255) / 256;
    p.bn = round16((T + p.t_tiles - 1) / p.t_tiles);
    // pairs of CTAs where the MMA's reads of shared memory bound a tile
    const bool pair = p.bn >= kPairMin && c.N > kTM;
    if (pair) p.bn = (p.bn + 31) / 32 * 32;
    const int rows = pair ? p.bn / 2 : p.bn;         // token rows of a CTA
    p.n_tiles = (c.N + (pair ? 2 : 1) * kTM - 1) / ((pair ? 2 : 1) * kTM);
    const size_t stage = (size_t)(kTM + rows) * kBK, extra = 1024 + (2 * kMaxSt + 10) * 8 + 2 * 256 * sizeof(float);
    p.stages = (int)std::min<size_t>(kMaxSt, (kSmem - extra) / stage);
    // whole tiles while two full waves are left, the rest in equal shares
    const long long tiles = (long long)p.n_tiles * p.t_tiles, total = tiles * p.kblocks;
    p.units = (int)std::min<long long>(pair ? ctx->sms / 2 : ctx->sms, std::max<long long>(tiles, total / kMinBlocks));
    // Fewer tiles than SMs: every tile in the same number of parts, though up to half of the SMs stay idle (memory
    // is busy all the same, and joining uneven parts costs more: 12,288 channels of 4096, 1 token, 13.9 us on 96 SMs
    // against 16.4 on all; 256 tokens 18.7 against 26.7; 9216 of 9216, 32 tokens, 20.5 against 21.9).  More tiles than
    // SMs: equal rounds of whole tiles where three quarters of the SMs are in them (27,648 of 9216, 73 %: 48.0 us
    // against 46.8 at 64 tokens, 51.2 against 52.4 at 128; 21,504 of 7168, 57 %: 38.2 against 30.9 at 32).
    // The more columns a tile has, the fewer parts: the last CTA reads the others'.  12 / 6 / 4 parts, us: 256 channels of
    // 16,384 10.1/12.4/14.9 at 1 token, 13.7/14.9/16.7 at 64, 19.0/18.6/19.5 at 128, 30.7/26.3/25.2 at 256; 512 of 8192
    // 8.8/9.4/10.5, 12.5/11.9/12.2, 18.0/15.5/14.8, 29.5/23.3/21.3; 2048 of 8192 10.2/10.3/10.8, 13.9/12.9/12.9,
    // 19.3/16.8/15.7, 31.5/25.9/22.5; 1024 of 4096 7.8/8.1/8.1, 10.8/10.6/9.9, 15.0/14.5/12.5, 24.5/22.7/18.7.  (The
    // narrow matrix of a long K decides at 64 and 128 tokens, where the wide ones would take 6 and 4: 0.6 to 2 us.)
    const long long parts = p.bn <= 64 ? 12 : p.bn <= 128 ? 6 : 4;
    const long long most = pair ? ctx->sms / 2 : ctx->sms, rounds = (tiles + most - 1) / most;
    const long long even = tiles >= most ? (tiles + rounds - 1) / rounds : std::min<long long>(p.units / tiles, parts) * tiles;
    const bool equal = tiles < most || tiles * 4 >= rounds * most * 3;
    if (equal) p.units = (int)even;
    p.whole = tiles % p.units == 0 ? (int)(tiles / p.units) : equal && tiles >= most ? (int)rounds : (int)std::max<long long>(0, tiles / p.units - 1);
    p.cut_base = p.whole * p.units;
    p.cut_tiles = (int)std::max<long long>(0, tiles - p.cut_base);
    p.partial = reinterpret_cast<int4*>(ctx->ws + ctx->lay.partial);
    p.tickets = reinterpret_cast<uint32_t*>(ctx->ws + ctx->lay.tickets);
    p.err = reinterpret_cast<uint32_t*>(ctx->ws);
    if (!map_i8(&p.mW, ctx->w.W, c.N, c.K, c.K, kTM) || !map_i8(&p.mA, A, T, c.K, lda, rows)) return SPFFN_ERR_UNSUPPORTED;
    const size_t smem = p.stages * stage + extra;
    auto kern = c.dtype == SPFFN_BF16 ? (pair ? k_mm8<__nv_bfloat16, true> : k_mm8<__nv_bfloat16, false>)
                                      : (pair ? k_mm8<__half, true> : k_mm8<__half, false>);
    static std::atomic<uint64_t> ready[4];              // a bit a device, for each of the four
    const cudaError_t e = allow_smem(kern, kSmem, ctx->device, ready[(c.dtype == SPFFN_BF16 ? 2 : 0) + (pair ? 1 : 0)]);
    if (e != cudaSuccess) return record_cuda(e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pair ? 2 * p.units : p.units));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pair ? 2 : 1;
    return record_cuda(cudaLaunchKernelEx(&cfg, kern, p));
}

spffn_status spffn_mm8_last_device_error(spffn_mm8_ctx* ctx, uint32_t* code, void* stream) {
    if (!ctx || !on_device(ctx->device)) return SPFFN_ERR_INVALID_ARG;
    const spffn_status s = take_device_error(reinterpret_cast<uint32_t*>(ctx->ws), code, stream);
    // a call that gave up may have left tiles counted in part
    if (s == SPFFN_ERR_TIMEOUT &&
        cudaMemsetAsync(ctx->ws + ctx->lay.tickets, 0, ctx->lay.partial - ctx->lay.tickets, (cudaStream_t)stream) != cudaSuccess)
        return SPFFN_ERR_CUDA;
    return s;
}

}  // extern "C"
