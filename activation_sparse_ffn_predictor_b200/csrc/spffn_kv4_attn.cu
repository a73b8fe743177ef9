// Attention over the paged 4-bit cache (spffn_kv4_attend in include/spffn_block.h):
//   out = sum_j softmax_j(scale q . K_j) V_j,   K_j = code step + zero per group of 32 dims
//
// Mathematics.  With n the codes, s the steps and z the zeros of a position j and a group g,
//   q . K_j = sum_g s_jg (q_g . n_jg) + sum_g z_jg (sum of q_g)
//   sum_j p_j V_j = sum_j (p_j s_jg) n_jg + sum_j p_j z_jg
// so the codes enter the matrix instructions as they are and steps and zeros touch only scores and
// probabilities: 16 positions x 8 query rows instead of 16 positions x dh values.
//
// Matrix instructions: mma.m16n8k16 in fp16 with fp32 sums.  Positions (for scores) and dims (for
// the output) are the 16 rows, query rows the 8 columns, so a head group of up to 8 rows costs one
// instruction per 16 x 16 codes and no row of it is padding for long contexts.  A code n in the low
// bits of a halfword is the fp16 subnormal n 2^-24 and in bits 4..7 n 2^-20: two ANDs turn a word
// into operands, no conversion; the 2^-24 and the 16 are undone on scores, outputs and q.
// q is brought to [2^9, 2^10) by a power of two per row (exact), so a bf16 q fits fp16; the sums of
// q_g enter as a high and a low half.  Probabilities times steps are rounded to fp16.  Where the output
// is bf16 (its own rounding is 2^-8) the probability is rounded before as well, and the codes of V enter
// as 0..15, whose sum the zeros take back.  Where it is fp16 (2^-11) a second half carries what the first
// rounding lost, so that one is left, of p s; zeros and 8 steps meet both halves as they are, so values with a
// large mean keep it (one half, and z + 8 s rounded, lost up to 6e-4 of a mean over 4 keys; 138 us in place of 143
// for 256 new tokens over 8205 positions).  V's codes enter as n - 8 (one fp16 operation a pair): the matrix
// instructions cut their sums off rather than round them, and over 100,000 positions that showed as 5e-4 of the small
// difference of two large sums.  Measured against 64 bits: 2.6e-4 in fp16, of which the output's rounding is 2.1e-4
// (6e-4 with codes from 0 and two roundings, 4 us less at 100,003 positions); 1.75e-3 and 1.66e-3 in bf16.
// Range: both factors of p s are kept near the top of what fp16 holds.  The largest probability stands at 2^11
// to 2^15 (the reference moves where a score passes that), and the steps of each group of dims are brought to at
// most 1 by a power of two of their own (at least 1/4 when it was set; the sums of the group move with it, exactly).
// What the operand loses at its small end is at most 2^-25 a position, 2^-34 of the largest p s and less: over N
// positions N 2^-34 of 15 steps, however far one key stands out and whatever size the steps have down to 2^-15.
// Smaller ones (fp16 holds them with few bits) are lifted by 2^15 and no further.
//
// Work: a unit is 32 positions of one (sequence, kv head, tile of query rows).  The units of the
// batch are one line, cut into equal shares, one a warp, which finds it from the lengths on the device (a
// captured graph replays with other lengths) and streams its units through a ring of bulk copies of its
// own (a unit is one stretch of a page, two where pages have 16 tokens): no warp waits for another.
// A head that lies inside a share is written out at once; the parts of a cut one go to the workspace and
// k_join adds them in their order.  (Measured and not kept: half shares that warps take as they come,
// 137 us against 127 at 32 sequences of 1400 positions, 72 heads; blocks that go through a share together
// and join through shared memory, with the last block to arrive joining the cut heads, 156 us; for many
// query rows, blocks that unpack 64 positions into shared memory for 64 rows in the usual layout, rows as
// M, 132 us against 138 at 256 new tokens over 8205 positions, 32 heads of 64 over 8: unpacking is a small
// part there, arithmetic on scores and its latency the large one.)
//
// Measured on one B200: 32 sequences of about 1400 positions, 72 heads, bf16, 120 us (4.3 TB/s); one sequence of
// 100,003, 32 heads over 8, fp16, 45.4 us; 70 new tokens of 16 sequences of about 4000, 56 heads over 8, bf16, 67.4 us;
// 256 new tokens over 8205, 32 heads of 64 over 8, fp16, 145 us.  Longer contexts: 32 sequences add 5.1 TB/s in bf16 and
// 4.2 in fp16 from 700 to 2800 positions each, one sequence 4.6 from 100,003 to 400,000, and the lines through these
// times begin at 19 and 18 us; one sequence of 1000 positions takes 11.  Bound by instructions: about 680 for a unit of
// one tile of 8 rows, of which 176 unpack codes, on 12 warps an SM.  Many new tokens: 136 to 168 Tflop/s (bf16, 32 heads of
// 128 over 8, 1024 to 8192 tokens of 8192 positions), by the same arithmetic on scores and probabilities.  There every warp
// also walks the row tiles of the batch to find its share, a division each.
#include <type_traits>
#include "spffn_umma.cuh"
#include "spffn_kv4.cuh"

namespace spffn {
namespace kv4 {
namespace {

using um::now_ns;
using um::s32;
using um::ub_expect;
using um::ub_init;
using um::ub_try;

constexpr int kUnit = 32;             // positions of a unit
// What a head costs beside its units, in units: its q, its sums, its rows.  Counted in the line, so that shares with
// more heads get fewer units: 118.4 us against 120.9 without at 32 sequences of 1400 positions, 72 heads.  (Moving cuts
// near a head's end to that end, 2 units at most, took 119.2 against 117.5, and 25.6 against 21.1 at 32 sequences of 256.)
constexpr int kHead = 1;
constexpr float kLog2e = 1.4426950408889634f;
// Probabilities: 2^kTop where the reference is set, 2^kMost before it moves (fp16 ends at 2^16).
constexpr float kTop = 11.f, kMost = 15.f;

struct KParams {
    AttendArgs a;
    const uint8_t* pool;
    float* part;                      // [2 shares][R rows][dh], then [2 shares][R] exponents and sums
    uint2* meta;                      // [T][nh] the shares that a row is cut into (and its place in its tile)
    int nh, kvh, G;
    int many;                         // the most shares
    int qvec, ovec;                   // rows of q in 16-byte pieces, rows of out in 8-byte pieces
    uint32_t head_bytes, page_bytes;  // of one kv head of a page, and of a page
};

__device__ __forceinline__ void mma(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with nothing to add to
__device__ __forceinline__ void mma0(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {     // a in the low half
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t as_u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(s32(bar)) : "memory");
}
// N words of shared memory
template <int N> __device__ __forceinline__ void lds(uint32_t* w, const uint8_t* p) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
        }
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
        static_assert(N == 1, "");
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// 64-bit by 64-bit, in 32 bits where both fit (the usual case by far: a 64-bit division is some hundred cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// A place in the line of units: (sequence, kv head, row tile, unit of it).  Pairs that differ in
// the row tile alone are neighbours, so their positions come from L2 the second time.
template <int R> struct Place {
    int b, hk, rt, u;
    int row0, n, len, ok;             // of the sequence
    int nrt, units, keys;             // its row tiles; units and visible positions of this row tile
    __device__ __forceinline__ void load_seq(const KParams& p) {
        const Seq s = seq_of(p.a.b, b);
        row0 = s.row0; n = s.n; len = s.len; ok = s.ok;
        nrt = (n * p.G + R - 1) / R;
    }
    static __device__ __forceinline__ int keys_of(int rt, int n, int len, bool ok, int G) {
        if (!ok) return 0;
        return (rt + 1) * R >= n * G ? len : len - n + ((rt + 1) * R - 1) / G + 1;
    }
    // a sequence whose length was refused keeps one unit a tile, without positions: its rows become 0
    static __device__ __forceinline__ int units_of(int keys) { return max(1, (keys + kUnit - 1) / kUnit); }
    __device__ __forceinline__ void load_tile(const KParams& p) {
        keys = keys_of(rt, n, len, ok, p.G);
        units = units_of(keys);
    }
    __device__ __forceinline__ void next_pair(const KParams& p) {
        if (++rt == nrt) {
            rt = 0;
            if (++hk == p.kvh) {
                hk = 0;
                do {
                    ++b;
                    if (b >= p.a.b.B) return;
                    load_seq(p);
                } while (n == 0);
            }
        }
        load_tile(p);
    }
};

// The running state of a tile of 8 NT query rows: thread (r, c) = (lane / 4, lane % 4) holds query columns
// 2c, 2c + 1 of each 8; o[2g + i][.][0, 1] dim 32g + 4r + 2i and [2, 3] dim + 1 of them.  `off`: the
// exponent that probabilities are taken against, -inf before the first; the o of group g hold steps times lift[g].
template <int NG, int NT> struct State {
    float off[NT][2], l[NT][2], o[2 * NG][NT][4];
    __half2 lift[NG];                 // the power of two that V steps of a group are multiplied by, twice
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int g = 0; g < NG; ++g) lift[g] = __float2half2_rn(32768.f);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            off[t][0] = off[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int j = 0; j < 2 * NG; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][t][i] = 0.f;
        }
    }
};

__device__ __forceinline__ float4* part_rows(const KParams& p, int slot, int R, int DH) {
    return reinterpret_cast<float4*>(p.part + (size_t)slot * R * DH);
}
__device__ __forceinline__ float2* part_sums(const KParams& p, int slot, int R, int DH) {
    return reinterpret_cast<float2*>(p.part + (size_t)2 * p.many * R * DH) + (size_t)slot * R;
}

// A share: where it begins, and where it ends: the row tile there and the unit of it.
template <int R> struct Share {
    Place<R> at;
    int64_t line, line_end;           // where the row tiles of its begin and its end begin in the line
    int u_end;
    int64_t each;
    int longer, shares;
    // the first share that begins at `unit` of the line or later
    __device__ __forceinline__ int from(int64_t unit) const {
        const int64_t bend = (each + 1) * longer;
        return unit <= bend ? (int)quotient(unit + each, each + 1) : longer + (int)quotient(unit - bend + each - 1, each);
    }
};

// Share `id` of at most `most`, found by a whole warp; false where there is none.
template <int R>
__device__ __forceinline__ bool find_share(const KParams& p, int most, int id, int lane, Share<R>& out) {
    using P = Place<R>;
    const Batch& bt = p.a.b;
    auto units_of_head = [&](const Seq& q) -> int64_t {           // length in the line of each kv head of a sequence
        const int nrt = (q.n * p.G + R - 1) / R;
        int64_t sum = 0;
        for (int t = 0; t < nrt; ++t) sum += kHead + P::units_of(P::keys_of(t, q.n, q.len, q.ok, p.G));
        return sum;
    };
    // a lane a sequence, 32 at a time: the units before it and its own
    auto sequences = [&](int s0, int64_t& mine, int64_t& before) {
        mine = s0 + lane < bt.B ? units_of_head(seq_of(bt, s0 + lane)) * p.kvh : 0;
        before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += v;
        }
        const int64_t sum = __shfl_sync(0xffffffffu, before, 31);
        before -= mine;
        return sum;
    };
    int64_t mine, before, total = sequences(0, mine, before);
    for (int s0 = 32; s0 < bt.B; s0 += 32) {
        int64_t m, b;
        total += sequences(s0, m, b);
    }
    if (total == 0) return false;
    // Equal shares, the first of them one unit longer where they do not divide; no more shares than units.
    const int shares = (int)min((int64_t)most, total);
    if (id >= shares) return false;
    const int64_t each = quotient(total, shares);
    const int longer = (int)(total - each * shares);
    P& at = out.at;                                                 // where the share stands
    int64_t line, line_end;                                       // where its row tile begins in the line; the same of
    int u_end;                                                    // the share's end, and the unit there
    {
        // lane 0 keeps the share's begin, the other lanes its end
        const int k = id + (lane != 0);
        const int64_t raw = each * k + min(k, longer);
        int64_t bound = total, in = 0;                            // the row tile's begin
        at.b = at.hk = at.rt = at.u = 0;
        int64_t done = 0;
        for (int s0 = 0; s0 < bt.B; s0 += 32) {
            int64_t sum;
            if (s0 == 0) sum = __shfl_sync(0xffffffffu, before + mine, 31);
            else sum = sequences(s0, mine, before);
#pragma unroll
            for (int side = 0; side < 2; ++side) {
                const int64_t x = __shfl_sync(0xffffffffu, raw, side) - done;
                const uint32_t here = __ballot_sync(0xffffffffu, x >= before && x < before + mine);
                if (here) {
                    const int from = __ffs(here) - 1;
                    const int64_t b0 = __shfl_sync(0xffffffffu, before, from);
                    if ((lane != 0) == side) {
                        at.b = s0 + from;
                        in = x - b0;
                    }
                }
            }
            done += sum;
        }
        if (raw < total) {
            at.load_seq(p);
            const int64_t head = units_of_head(Seq{at.row0, at.n, at.len, at.ok != 0});
            at.hk = (int)quotient(in, head);
            in -= head * at.hk;
            for (;; ++at.rt) {
                at.load_tile(p);
                if (in < kHead + at.units) break;
                in -= kHead + at.units;
            }
            bound = raw - in;
            at.u = max(0, (int)in - kHead);
        }
        line = __shfl_sync(0xffffffffu, bound, 0);
        line_end = __shfl_sync(0xffffffffu, bound, 1);
        u_end = __shfl_sync(0xffffffffu, at.u, 1);
        at.b = __shfl_sync(0xffffffffu, at.b, 0);
        at.hk = __shfl_sync(0xffffffffu, at.hk, 0);
        at.rt = __shfl_sync(0xffffffffu, at.rt, 0);
        at.u = __shfl_sync(0xffffffffu, at.u, 0);
    }
    if (line > line_end || (line == line_end && at.u >= u_end)) return false;
    at.load_seq(p);
    at.load_tile(p);
    out.line = line;
    out.line_end = line_end;
    out.u_end = u_end;
    out.each = each;
    out.longer = longer;
    out.shares = shares;
    return true;
}

template <typename T, int NG, int NT, int W, int NS, int MB>
__global__ void __launch_bounds__(32 * W, MB) k_attend(const KParams p) {
    using L = Blk<NG>;
    constexpr int R = 8 * NT, DH = 32 * NG;
    constexpr bool kFine = std::is_same<T, __half>::value;
    constexpr uint32_t kTile = 2 * L::kBytes;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;                                         // [W][NS][kTile]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + W * NS * kTile);   // [W][NS]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    const Batch& bt = p.a.b;

    // ------------------------------------------------------------------ the line and its cuts
    if (lane < NS) ub_init(&bars[warp * NS + lane], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    um::pdl_trigger();
    um::pdl_wait();
    Share<R> sh;
    if (!find_share(p, gridDim.x * W, blockIdx.x * W + warp, lane, sh)) return;
    Place<R> at = sh.at;
    int64_t line = sh.line;
    const int64_t line_end = sh.line_end;
    const int u_end = sh.u_end, id = blockIdx.x * W + warp;
    int st = 0;
    uint32_t phase = 0;
    uint8_t* my_ring = ring + warp * NS * kTile;
    uint64_t* my_bar = bars + warp * NS;
    bool failed = false;
    at.load_seq(p);
    at.load_tile(p);

    // ------------------------------------------------------------ the warp's ring of copies
    Place<R> ahead = at;                                          // the next unit to ask for
    int64_t line_ahead = line;
    int stop = line_ahead == line_end ? u_end : ahead.units;      // of its row tile; 0 once the share is through
    int page0 = -1, page1 = -1;
    uint32_t lacks = 0;                                           // blocks that were not copied, 2 bits a stage
    auto look_up = [&]() {                                        // the pages of `ahead`, used one round later
        const int pos = ahead.u * kUnit;
        const int32_t* row = bt.table + ahead.b * bt.ldt + (pos >> bt.page_log);
        page0 = pos < ahead.keys ? __ldg(row) : -1;               // no positions: a refused sequence
        if (bt.page_log == 4) page1 = pos + 16 < ahead.keys ? __ldg(row + 1) : -1;
    };
    const bool small = bt.page_log == 4;                          // a unit is two pages
    auto source = [&](int page, int pp) {
        return p.pool + (uint64_t)(uint32_t)page * p.page_bytes +
               ((uint32_t)ahead.hk * p.head_bytes + (uint32_t)((pp & (bt.page - 1)) >> 4) * L::kBytes);
    };
    auto ask = [&](int st) {
        if (stop == 0) return;
        const int pos = ahead.u * kUnit;
        uint64_t* bar = &my_bar[st];
        const uint32_t dst = s32(my_ring + st * kTile);
        lacks &= ~(3u << (2 * st));
        if (!small && (unsigned)page0 < (unsigned)bt.pages) {
            // one stretch; where the row's positions end in its first block the second comes along unread
            if (lane == 0) {
                ub_expect(bar, kTile);
                bulk_copy(dst, source(page0, pos), kTile, bar);
            }
        } else {
            const bool in0 = (unsigned)page0 < (unsigned)bt.pages, in1 = small && (unsigned)page1 < (unsigned)bt.pages;
            if (((pos < ahead.keys && !in0) || (small && pos + 16 < ahead.keys && !in1)) && lane == 0) latch(bt.err, ERR_PAGE_RANGE);
            lacks |= ((in0 ? 0u : 1u) | (in1 ? 0u : 2u)) << (2 * st);
            if (lane == 0) {
                if (!in0 && !in1) um::ub_arrive(bar);
                else {
                    ub_expect(bar, (in0 ? L::kBytes : 0) + (in1 ? L::kBytes : 0));
                    if (in0) bulk_copy(dst, source(page0, pos), L::kBytes, bar);
                    if (in1) bulk_copy(dst + L::kBytes, source(page1, pos + 16), L::kBytes, bar);
                }
            }
        }
        if (++ahead.u == stop) {
            line_ahead += kHead + ahead.units;
            stop = 0;
            if (line_ahead > line_end || (line_ahead == line_end && u_end == 0)) return;
            ahead.u = 0;
            ahead.next_pair(p);
            stop = line_ahead == line_end ? u_end : ahead.units;
        }
        look_up();
    };
    look_up();
#pragma unroll
    for (int i = 0; i < NS; ++i) ask(i);

    // -------------------------------------------------------------------- the share's heads
    for (;;) {
        const int u0 = at.u, u1 = line == line_end ? u_end : at.units;
        State<NG, NT> s;
        s.clear();
        float oz[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) oz[t][i] = 0.f;
        // q of row r as the second operand, its group sums as halves, the factor of the columns' scores
        uint32_t qf[NT][NG][4], qs[NT][2];
        float fq[NT][2];
        int pos[NT][2];
        const int rows = at.n * p.G;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int row = at.rt * R + t * 8 + r;
            float q[8 * NG], big = 0.f, bad = 0.f;
            if (row < rows) {
                const T* src = static_cast<const T*>(p.a.q) + (int64_t)(at.row0 + row / p.G) * p.a.ldq +
                               (int64_t)(at.hk * p.G + row % p.G) * DH + 8 * c;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    if (p.qvec) unpack8<T>(*reinterpret_cast<const uint4*>(src + 32 * g), q + 8 * g);
                    else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) q[8 * g + i] = DT<T>::f(src[32 * g + i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8 * NG; ++i) {
                    big = fmaxf(big, fabsf(q[i]));
                    bad += q[i] * 0.f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8 * NG; ++i) q[i] = 0.f;
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                bad += __shfl_xor_sync(0xffffffffu, bad, o);
            }
            const int e = (int)(__float_as_uint(big) >> 23) - 127;
            const int k = big == 0.f ? 0 : min(126, 9 - e);
            const float up = bad == 0.f ? __uint_as_float((uint32_t)(127 + k) << 23) : __int_as_float(0x7fc00000);
            const float f = p.a.scale * kLog2e * __uint_as_float((uint32_t)(127 - k) << 23);
            fq[t][0] = __shfl_sync(0xffffffffu, f, 8 * c);        // of rows 2c and 2c + 1
            fq[t][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
            uint32_t hs = 0, ls = 0;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float h[8], sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    h[i] = __half2float(__float2half_rn(q[8 * g + i] * up));
                    sum += h[i];
                }
                // codes 0, 4 | 1, 5 (times 16) | 2, 6 | 3, 7 (times 16) of the word
                qf[t][g][0] = pack2(h[0], h[4]);
                qf[t][g][1] = pack2(h[1] * 0.0625f, h[5] * 0.0625f);
                qf[t][g][2] = pack2(h[2], h[6]);
                qf[t][g][3] = pack2(h[3] * 0.0625f, h[7] * 0.0625f);
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                if (g >> 1 == c) {
                    const __half hi16 = __float2half_rn(sum), lo16 = __float2half_rn(sum - __half2float(hi16));
                    hs |= (uint32_t)__half_as_ushort(hi16) << (16 * (g & 1));
                    ls |= (uint32_t)__half_as_ushort(lo16) << (16 * (g & 1));
                }
            }
            qs[t][0] = hs;
            qs[t][1] = ls;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int rw = at.rt * R + t * 8 + 2 * c + i;
                pos[t][i] = at.len - at.n + rw / p.G;             // of rows past the last: never written
            }
        }
        const int clear_to = at.len - at.n + at.rt * R / p.G + 1; // positions that every row sees

        for (int u = u0; u < u1 && !failed; ++u) {
            const uint8_t* tile = my_ring + st * kTile;
            const uint32_t have = 3u & ~(lacks >> (2 * st));
            // lanes may see the copies' arrival at different tries: they agree before they part
            if (!__all_sync(0xffffffffu, ub_try(&my_bar[st], phase))) {
                const unsigned long long t0 = now_ns();
                while (!ub_try(&my_bar[st], phase)) {
                    if (now_ns() - t0 > um::kUWaitNs) {
                        failed = true;
                        break;
                    }
                }
                failed = __any_sync(0xffffffffu, failed);
            }
            if (failed) {
                if (lane == 0) latch(bt.err, ERR_PIPE_TIMEOUT);
                break;
            }
            const int p0 = u * kUnit;
            if (have) {
                // V steps: the largest of each group, and what must not enter the products: positions past
                // the last, and steps and zeros that are not finite (rows that see them have it from their scores)
                uint32_t nan_tok = 0;                             // bit t: position p0 + t has such a step or zero
                __half2 top[NG];                                  // of this lane's positions: 2c, 2c + 1 of each 8
                __half2 zs = __float2half2_rn(0.f);               // 0 where zeros are finite, a group a lane of r
                auto tops = [&]() {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t v[NG];
                        const uint8_t* from = tile + (k >> 1) * L::kBytes + L::kVs + (k & 1) * 16 * NG + c * 4 * NG;
                        zs = __hfma2(as_h2(*reinterpret_cast<const uint32_t*>(from + 32 * NG + 4 * (r & (NG - 1)))), __float2half2_rn(0.f), zs);
                        lds<NG>(v, from);
#pragma unroll
                        for (int g = 0; g < NG; ++g) top[g] = k ? __hmax2_nan(top[g], __habs2(as_h2(v[g]))) : __habs2(as_h2(v[g]));
                    }
                };
                auto fits = [&]() {                               // false where one is not a number, too
                    __half2 m = zs;
#pragma unroll
                    for (int g = 0; g < NG; ++g) m = __hmax2_nan(m, __hmul2(top[g], s.lift[g]));
                    return __all_sync(0xffffffffu, __hble2(m, __float2half2_rn(1.f)));
                };
                const bool edge = p0 + kUnit > at.keys || have != 3u;
                if (!edge) tops();
                if (edge || !fits()) {
                    uint8_t* w = const_cast<uint8_t*>(tile);
                    uint8_t* blk = w + (lane >> 4) * L::kBytes;   // a lane a position
                    const int tok = lane & 15;
                    const bool here = (have >> (lane >> 4)) & 1u;
                    bool nan = false;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        nan |= (*reinterpret_cast<const uint16_t*>(blk + L::vs(tok, g)) & 0x7c00u) == 0x7c00u ||
                               (*reinterpret_cast<const uint16_t*>(blk + L::vz(tok, g)) & 0x7c00u) == 0x7c00u;
                    if (nan || !here || p0 + lane >= at.keys) {
#pragma unroll
                        for (int g = 0; g < NG; ++g) {
                            *reinterpret_cast<uint16_t*>(blk + L::vs(tok, g)) = 0;
                            *reinterpret_cast<uint16_t*>(blk + L::vz(tok, g)) = 0;
                        }
                    }
                    nan_tok = nan && here ? 1u << lane : 0u;
                    um::fence_async_smem();                       // the ring's next copy comes by another proxy
                    nan_tok = __reduce_or_sync(0xffffffffu, nan_tok);
                    __syncwarp();
                    tops();
                    // a step above what its group is lifted for: lifted to 1/4 .. 1/2 from here on
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        __half2 m = top[g];
#pragma unroll
                        for (int o = 1; o < 4; o <<= 1) m = __hmax2(m, as_h2(__shfl_xor_sync(0xffffffffu, as_u(m), o)));
                        const float v = fmaxf(__low2float(m), __high2float(m)), now = __low2float(s.lift[g]);
                        if (v * now > 1.f) {                      // v and now are normal in fp32
                            const float next = __uint_as_float((252u << 23) - (__float_as_uint(v) & 0x7f800000u));   // 2^-2 over v's power of two
                            const float f = next * __uint_as_float((254u << 23) - __float_as_uint(now));
#pragma unroll
                            for (int t = 0; t < NT; ++t)
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    s.o[2 * g][t][i] *= f;
                                    s.o[2 * g + 1][t][i] *= f;
                                }
                            s.lift[g] = __float2half2_rn(next);
                        }
                    }
                }

                // scores of the unit: position r (and r + 8) of each block of 16, columns 2c, 2c + 1
                float sc[2][NT][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint8_t* blk = tile + j * L::kBytes;
                    uint32_t w0[NG], w1[NG], st0[(NG + 1) / 2], st1[(NG + 1) / 2];
                    lds<NG>(w0, blk + r * 16 * NG + c * 4 * NG);
                    lds<NG>(w1, blk + (r + 8) * 16 * NG + c * 4 * NG);
                    lds<NG / 2>(st0, blk + L::kKs + r * 2 * NG);
                    lds<NG / 2>(st1, blk + L::kKs + (r + 8) * 2 * NG);
                    const int zc = NG == 8 ? 4 * c : 4 * (c & (NG / 2 - 1));          // groups 2c, 2c + 1
                    uint32_t z0 = *reinterpret_cast<const uint32_t*>(blk + L::kKz + r * 2 * NG + zc);
                    uint32_t z1 = *reinterpret_cast<const uint32_t*>(blk + L::kKz + (r + 8) * 2 * NG + zc);
                    if (NG < 8 && 2 * c >= NG) z0 = z1 = 0u;
                    float part[NT][4];
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma0(sc[j][t], z0, z1, z0, z1, qs[t][0], qs[t][1]);
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        const float2 s0 = __half22float2(as_h2(st0[g >> 1])), s1 = __half22float2(as_h2(st1[g >> 1]));
                        const float k0 = g & 1 ? s0.y : s0.x, k1 = g & 1 ? s1.y : s1.x;
                        const uint32_t a0 = w0[g] & 0x000f000fu, a2 = w0[g] & 0x00f000f0u, b0 = (w0[g] >> 8) & 0x000f000fu,
                                       b2 = (w0[g] >> 8) & 0x00f000f0u;
                        const uint32_t a1 = w1[g] & 0x000f000fu, a3 = w1[g] & 0x00f000f0u, b1 = (w1[g] >> 8) & 0x000f000fu,
                                       b3 = (w1[g] >> 8) & 0x00f000f0u;
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            float d[4];
                            mma0(d, a0, a1, a2, a3, qf[t][g][0], qf[t][g][1]);
                            mma(d, b0, b1, b2, b3, qf[t][g][2], qf[t][g][3]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) part[t][i] = g == 0 ? d[i] * (i < 2 ? k0 : k1) : fmaf(d[i], i < 2 ? k0 : k1, part[t][i]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sc[j][t][i] = fmaf(part[t][i], 16777216.f, sc[j][t][i]) * fq[t][i & 1];
                }
                if (p0 + kUnit > clear_to || have != 3u || nan_tok) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int tok = 16 * j + r + 8 * (i >> 1);
                                if (p0 + tok > pos[t][i & 1] || p0 + tok >= at.keys || !((have >> j) & 1u)) sc[j][t][i] = -INFINITY;
                                else if ((nan_tok >> tok) & 1u) sc[j][t][i] = __int_as_float(0x7fc00000);
                            }
                }
                // The reference exponent moves only where a score passes it by more than fp16 has room for.
                float top_s[NT][2];
                bool far = false;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top_s[t][i] = fmaxf(fmaxf(sc[0][t][i], sc[0][t][i + 2]), fmaxf(sc[1][t][i], sc[1][t][i + 2]));
                        far |= top_s[t][i] > s.off[t][i] + kMost;
                    }
                if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float m = top_s[t][i];
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                            const float off = fmaxf(m - kTop, s.off[t][i]);             // -inf stays
                            const float f = off == s.off[t][i] ? 1.f : ex2(s.off[t][i] - off);
                            s.off[t][i] = off;
                            s.l[t][i] *= f;
                            oz[t][i] *= f;
                            oz[t][i + 2] *= f;
#pragma unroll
                            for (int d = 0; d < 2 * NG; ++d) {
                                s.o[d][t][i] *= f;
                                s.o[d][t][i + 2] *= f;
                            }
                        }
                }
                // probabilities, turned into the second operand of the output's product
                uint32_t pb[2][NT][2], pl[kFine ? 2 : 1][NT][2];   // and what rounding them lost
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float pr[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            pr[i] = ex2(sc[j][t][i] - fmaxf(s.off[t][i & 1], -3e38f));
                            s.l[t][i & 1] += pr[i];
                        }
                        const uint32_t h0 = pack2(pr[0], pr[1]), h1 = pack2(pr[2], pr[3]);
                        pb[j][t][0] = transpose8(h0);
                        pb[j][t][1] = transpose8(h1);
                        if constexpr (kFine) {
                            const float2 f0 = __half22float2(as_h2(h0)), f1 = __half22float2(as_h2(h1));
                            pl[j][t][0] = transpose8(pack2(pr[0] - f0.x, pr[1] - f0.y));
                            pl[j][t][1] = transpose8(pack2(pr[2] - f1.x, pr[3] - f1.y));
                        }
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint8_t* blk = tile + j * L::kBytes;
                    uint32_t w0[NG], w1[NG], s0[NG], s1[NG];       // words of tokens 2c, 2c + 1 | 2c + 8, 2c + 9
                    lds<NG>(w0, blk + L::kV + r * 16 * NG + c * 4 * NG);
                    lds<NG>(w1, blk + L::kV + 128 * NG + r * 16 * NG + c * 4 * NG);
                    lds<NG>(s0, blk + L::kVs + c * 4 * NG);
                    lds<NG>(s1, blk + L::kVs + 16 * NG + c * 4 * NG);
                    uint32_t z0 = *reinterpret_cast<const uint32_t*>(blk + L::kVz + c * 4 * NG + 4 * (r & (NG - 1)));
                    uint32_t z1 = *reinterpret_cast<const uint32_t*>(blk + L::kVz + 16 * NG + c * 4 * NG + 4 * (r & (NG - 1)));
                    uint32_t e0 = 0u, e1 = 0u;                    // codes around 8: 8 steps go with the zeros, as rows of their own
                    if constexpr (kFine) {
                        const uint8_t* at_s = blk + L::kVs + c * 4 * NG + 4 * (r & (NG - 1));
                        e0 = *reinterpret_cast<const uint32_t*>(at_s);
                        e1 = *reinterpret_cast<const uint32_t*>(at_s + 16 * NG);
                    }
                    if (r >= NG) z0 = z1 = e0 = e1 = 0u;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        mma(oz[t], z0, e0, z1, e1, pb[j][t][0], pb[j][t][1]);
                        if constexpr (kFine) mma(oz[t], z0, e0, z1, e1, pl[j][t][0], pl[j][t][1]);
                    }
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        uint32_t b0[NT], b1[NT];
                        const __half2 l0 = __hmul2(as_h2(s0[g]), s.lift[g]), l1 = __hmul2(as_h2(s1[g]), s.lift[g]);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if constexpr (kFine) {
                                b0[t] = as_u(__hfma2(as_h2(pb[j][t][0]), l0, __hmul2(as_h2(pl[j][t][0]), l0)));
                                b1[t] = as_u(__hfma2(as_h2(pb[j][t][1]), l1, __hmul2(as_h2(pl[j][t][1]), l1)));
                            } else {
                                b0[t] = as_u(__hmul2(as_h2(pb[j][t][0]), l0));
                                b1[t] = as_u(__hmul2(as_h2(pb[j][t][1]), l1));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            // byte i of group g of the two tokens, one in each half
                            const int wd = g >> 1, by = 2 * (g & 1) + i;
                            const uint32_t sel = (uint32_t)(by | (by << 4) | ((4 + by) << 8) | ((4 + by) << 12));
                            const uint32_t a = __byte_perm(w0[wd], w0[NG / 2 + wd], sel), b = __byte_perm(w1[wd], w1[NG / 2 + wd], sel);
                            uint32_t a0 = a & 0x000f000fu, a1 = a & 0x00f000f0u, a2 = b & 0x000f000fu, a3 = b & 0x00f000f0u;
                            if constexpr (kFine) {                // 1024 + n and 1024 + 16 n, brought to n - 8
                                const __half2 m1032 = __float2half2_rn(-1032.f), m72 = __float2half2_rn(-72.f), sixteenth = __float2half2_rn(0.0625f);
                                a0 = as_u(__hadd2(as_h2(a0 | 0x64006400u), m1032));
                                a1 = as_u(__hfma2(as_h2(a1 | 0x64006400u), sixteenth, m72));
                                a2 = as_u(__hadd2(as_h2(a2 | 0x64006400u), m1032));
                                a3 = as_u(__hfma2(as_h2(a3 | 0x64006400u), sixteenth, m72));
                            }
#pragma unroll
                            for (int t = 0; t < NT; ++t) mma(s.o[2 * g + i][t], a0, a1, a2, a3, b0[t], b1[t]);
                        }
                    }
                }
            }
            __syncwarp();                                         // every lane has read the stage
            ask(st);
            if (++st == NS) {
                st = 0;
                phase ^= 1;
            }
        }

        // ------------------------------------------- the head's rows, or this share's part of them
        // the sums over r of l; codes' and zeros' parts together, in true units
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) s.l[t][i] += __shfl_xor_sync(0xffffffffu, s.l[t][i], o);
                if constexpr (kFine) oz[t][i] = fmaf(8.f, oz[t][i + 2], oz[t][i]);
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float z = __shfl_sync(0xffffffffu, oz[t][i], 4 * g + c);
                    const float back = __uint_as_float((254u << 23) - __float_as_uint(__low2float(s.lift[g])));
#pragma unroll
                    for (int d = 2 * g; d < 2 * g + 2; ++d) {
                        s.o[d][t][i] = fmaf(s.o[d][t][i], kFine ? back : 16777216.f * back, z);
                        s.o[d][t][i + 2] = fmaf(s.o[d][t][i + 2], kFine ? back : 1048576.f * back, z);
                    }
                }
            }
        const bool whole = u0 == 0 && u1 == at.units;
        Cuts cuts{0u, 0u, 0u};                                    // from this share on, how many more
        if (u0 == 0 && !whole) {
            // the shares whose cuts fall inside the head, as the plan cuts
            const int past = sh.from(line + kHead + at.units);
            cuts = Cuts{(uint32_t)id, (uint32_t)(past - 1 - id), 0u};
        }
        const int slot = 2 * id + (u0 == 0);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int in = t * 8 + 2 * c + i, row = at.rt * R + in;
                if (row >= rows) continue;
                const int token = at.row0 + row / p.G, head = at.hk * p.G + row % p.G;
                if (u0 == 0 && r == 0) p.meta[(int64_t)token * p.nh + head] = pack_cuts(Cuts{cuts.first, cuts.more, (uint32_t)in});
                if (whole) {
                    T* to = static_cast<T*>(p.a.out) + (int64_t)token * p.a.ldo + (int64_t)head * DH + 4 * r;
                    const float inv = s.l[t][i] == 0.f ? 0.f : 1.f / s.l[t][i];
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        T v[4] = {DT<T>::r(s.o[2 * g][t][i] * inv), DT<T>::r(s.o[2 * g][t][i + 2] * inv),
                                  DT<T>::r(s.o[2 * g + 1][t][i] * inv), DT<T>::r(s.o[2 * g + 1][t][i + 2] * inv)};
                        if (p.ovec) *reinterpret_cast<uint2*>(to + 32 * g) = *reinterpret_cast<const uint2*>(v);
                        else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) to[32 * g + k] = v[k];
                        }
                    }
                } else {
                    float4* to = part_rows(p, slot, R, DH) + in * (DH / 4) + r;
#pragma unroll
                    for (int g = 0; g < NG; ++g)
                        __stcg(to + 8 * g, make_float4(s.o[2 * g][t][i], s.o[2 * g][t][i + 2], s.o[2 * g + 1][t][i], s.o[2 * g + 1][t][i + 2]));
                    if (r == 0) __stcg(part_sums(p, slot, R, DH) + in, make_float2(s.off[t][i], s.l[t][i]));
                }
            }
        line += kHead + at.units;
        if (failed || line > line_end || (line == line_end && u_end == 0)) break;
        at.u = 0;
        at.next_pair(p);
    }
    // copies that were asked for and not used (a wait that ran out) land before the block ends: the stages from
    // st on are in the current phase, those before it one further
    if (failed) {
        for (int i = 0; i < NS; ++i) {
            const unsigned long long t0 = now_ns();
            while (!ub_try(&my_bar[i], i >= st ? phase : phase ^ 1u) && now_ns() - t0 < 20000000ull) {}
        }
    }
}

// The rows of cut heads: sums of the shares' parts in their order.  WPR warps a row: 1 where a head is cut into
// a few shares, 16 where a few heads fill the device (their loads then go out together: the time is their latency).
template <typename T, int NG, int R, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 256 : 32 * WPR) k_join(const KParams p) {
    constexpr int DH = 32 * NG, V = (NG + 3) / 4, LR = DH / 4 < 32 ? DH / 4 : 32;   // a row is LR lanes of V float4
    __shared__ float4 acc_s[WPR][V][32];
    __shared__ float2 ml_s[WPR];
    // no early start for what comes next: blocks of the next call that wait on an SM slowed these (141 -> 127 us at
    // 32 sequences of 1400 positions, 72 heads)
    um::pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = WPR == 1 ? (int64_t)blockIdx.x * 8 + warp : blockIdx.x;
    if (row >= (int64_t)p.a.b.T * p.nh) return;
    const int token = (int)(row / p.nh), head = (int)(row % p.nh);
    const int sq = seq_of_row(p.a.b, token);
    if (sq < 0) return;
    if (p.a.b.start) {                                            // a row that the plan skipped has no entry
        const Seq q = seq_of(p.a.b, sq);
        if (q.n == 0) return;
    }
    const Cuts cuts = unpack_cuts(p.meta[row]);
    if (cuts.more == 0 || !cuts_in(cuts, p.many, R)) return;
    const int first = (int)cuts.first, in = (int)cuts.in, n = (int)cuts.more + 1;
    float top = -INFINITY, l = 0.f;
    float4 acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
    // 32 parts at a time: their exponents and sums a lane each, then their values
    const int k1 = WPR == 1 ? n : n * (warp + 1) / WPR;           // the warp's stretch of the parts
    for (int k0 = WPR == 1 ? 0 : n * warp / WPR; k0 < k1; k0 += 32) {
        const int k = k0 + lane;
        const float2 ml = k < k1 ? __ldcg(part_sums(p, 2 * (first + k) + (k == 0), R, DH) + in) : make_float2(-INFINITY, 0.f);
        float mx = ml.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        mx = fmaxf(mx, top);
        const float base = mx == -INFINITY ? 0.f : mx, f = ex2(top - base), w = ex2(ml.x - base);
        top = mx;
        l = l * f + warp_sum(ml.y * w);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = make_float4(acc[v].x * f, acc[v].y * f, acc[v].z * f, acc[v].w * f);
        const int here = min(32, k1 - k0);
        // a warp reads 32 / LR parts at once; the lanes past them repeat the last with no weight
        constexpr int P = 32 / LR;
#pragma unroll (WPR == 1 ? 4 : 16 / P)
        for (int j = 0; j < here; j += P) {
            const int mine = j + (P == 1 ? 0 : lane / LR);
            const int at = min(mine, here - 1);
            const float wj = __shfl_sync(0xffffffffu, w, at) * (mine < here ? 1.f : 0.f);
            const float4* from = part_rows(p, 2 * (first + k0 + at) + (k0 + at == 0), R, DH) + in * (DH / 4) + lane % LR;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 x = __ldcg(from + 32 * v);
                if (mine < here) {
                    acc[v].x = fmaf(x.x, wj, acc[v].x);
                    acc[v].y = fmaf(x.y, wj, acc[v].y);
                    acc[v].z = fmaf(x.z, wj, acc[v].z);
                    acc[v].w = fmaf(x.w, wj, acc[v].w);
                }
            }
        }
    }
    if constexpr (WPR > 1) {
        if (lane == 0) ml_s[warp] = make_float2(top, l);
#pragma unroll
        for (int v = 0; v < V; ++v) acc_s[warp][v][lane] = acc[v];
        __syncthreads();
        if (warp > 0) return;
        float mx = -INFINITY;
        for (int w = 0; w < WPR; ++w) mx = fmaxf(mx, ml_s[w].x);
        const float base = mx == -INFINITY ? 0.f : mx;
        l = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            const float f = ex2(ml_s[w].x - base);
            l += ml_s[w].y * f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float4 x = acc_s[w][v][lane];
                acc[v].x = fmaf(x.x, f, acc[v].x);
                acc[v].y = fmaf(x.y, f, acc[v].y);
                acc[v].z = fmaf(x.z, f, acc[v].z);
                acc[v].w = fmaf(x.w, f, acc[v].w);
            }
        }
    }
    if constexpr (LR < 32) {
        acc[0].x += __shfl_xor_sync(0xffffffffu, acc[0].x, 16);
        acc[0].y += __shfl_xor_sync(0xffffffffu, acc[0].y, 16);
        acc[0].z += __shfl_xor_sync(0xffffffffu, acc[0].z, 16);
        acc[0].w += __shfl_xor_sync(0xffffffffu, acc[0].w, 16);
        if (lane >= LR) return;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* to = static_cast<T*>(p.a.out) + (int64_t)token * p.a.ldo + (int64_t)head * DH + 4 * lane;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        T o[4] = {DT<T>::r(acc[v].x * inv), DT<T>::r(acc[v].y * inv), DT<T>::r(acc[v].z * inv), DT<T>::r(acc[v].w * inv)};
        if (p.ovec) *reinterpret_cast<uint2*>(to + 128 * v) = *reinterpret_cast<const uint2*>(o);
        else {
#pragma unroll
            for (int k = 0; k < 4; ++k) to[128 * v + k] = o[k];
        }
    }
}

// The shapes of a launch: warps and blocks at once as registers and the rings allow.
template <int NG, int NT> struct Shape {
    static constexpr int W = 4;
    static constexpr int NS = NG == 2 ? 4 : NG == 4 && NT == 2 ? 3 : 2;
    static constexpr int MB = NG == 2 ? (NT == 1 ? 4 : 2) : NG == 4 && NT == 1 ? 3 : 2;
    static constexpr size_t smem = (size_t)W * NS * 1280 * NG + W * NS * 8;
    static_assert(smem <= 227 * 1024 / MB - 1024, "");
    static constexpr int shares = MB * W;                         // of an SM
    static constexpr size_t part_floats = (size_t)2 * shares * 8 * NT * (32 * NG + 2);
};
constexpr int most_rows(int ng) { return ng == 2 ? 4 : 2; }       // 8-row tiles that a warp's registers hold
template <int NG> constexpr size_t part_floats() {
    return std::max(std::max(Shape<NG, 1>::part_floats, Shape<NG, 2>::part_floats), NG == 2 ? Shape<NG, 4>::part_floats : (size_t)0);
}

template <typename K>
cudaError_t launch_chained(K kern, unsigned grid, unsigned threads, size_t smem, const KParams& p, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, int NG, int NT>
cudaError_t go(const spffn_kv4_ctx& c, KParams p, cudaStream_t st) {
    using S = Shape<NG, NT>;
    auto kern = k_attend<T, NG, NT, S::W, S::NS, S::MB>;
    static std::atomic<uint64_t> ready{0};                        // a bit a device
    cudaError_t e = allow_smem(kern, S::smem, c.device, ready);
    if (e != cudaSuccess) return e;
    p.many = c.sms * S::shares;
    e = launch_chained(kern, (unsigned)(c.sms * S::MB), 32 * S::W, S::smem, p, st);
    if (e != cudaSuccess) return e;
    // a row tile is cut into about as many parts as there are warps for it; 16 warps a row where that is 16 or more
    // (one sequence of 100,003 positions, 32 heads over 8: 43.5 us, 94.3 with one warp a row)
    const int64_t rows = (int64_t)p.a.b.T * p.nh, tiles = std::max<int64_t>(p.a.b.B, (int64_t)p.a.b.T * p.G / (8 * NT)) * p.kvh;
    if (tiles * 16 <= (int64_t)c.sms * S::MB * S::W)
        return launch_chained(k_join<T, NG, 8 * NT, 16>, (unsigned)rows, 512, 0, p, st);
    return launch_chained(k_join<T, NG, 8 * NT, 1>, (unsigned)((rows + 7) / 8), 256, 0, p, st);
}

template <typename T, int NG>
cudaError_t by_rows(const spffn_kv4_ctx& c, const KParams& p, int nt, cudaStream_t st) {
    if constexpr (most_rows(NG) == 4) {
        if (nt == 4) return go<T, NG, 4>(c, p, st);
    }
    return nt == 1 ? go<T, NG, 1>(c, p, st) : go<T, NG, 2>(c, p, st);
}

template <typename T>
cudaError_t by_width(const spffn_kv4_ctx& c, const KParams& p, int nt, cudaStream_t st) {
    switch (c.cfg.dh) {
        case 64: return by_rows<T, 2>(c, p, nt, st);
        case 128: return by_rows<T, 4>(c, p, nt, st);
        default: return by_rows<T, 8>(c, p, nt, st);
    }
}

}  // namespace

Layout layout(const spffn_kv4_config& c, int sms) {
    Layout l;
    const size_t part = c.dh == 64 ? part_floats<2>() : c.dh == 128 ? part_floats<4>() : part_floats<8>();
    l.ctl = 0;
    l.meta = kCtlBytes;
    l.part = align_up(l.meta + (size_t)c.max_tokens * c.nh * sizeof(uint2), 256);
    l.total = l.part + sms * part * sizeof(float);
    return l;
}

cudaError_t launch_attend(const spffn_kv4_ctx& c, const AttendArgs& a, cudaStream_t st) {
    KParams p;
    p.a = a;
    p.pool = c.pool;
    p.part = reinterpret_cast<float*>(c.ws + c.lay.part);
    p.meta = reinterpret_cast<uint2*>(c.ws + c.lay.meta);
    p.many = 0;
    p.nh = c.cfg.nh;
    p.kvh = c.cfg.kvh;
    p.G = c.cfg.nh / c.cfg.kvh;
    p.qvec = aligned_to(a.q, 16) && a.ldq % 8 == 0;
    p.ovec = aligned_to(a.out, 8) && a.ldo % 4 == 0;
    p.head_bytes = (uint32_t)(c.cfg.page_size / 16) * (20u * c.cfg.dh);
    p.page_bytes = p.head_bytes * (uint32_t)c.cfg.kvh;
    // 8, 16 or 32 query rows a tile, by the rows that a kv head has in the mean: more rows share the unpacking, fewer
    // leave less of a tile empty (256 new tokens, 32 heads of 64 over 8: 138 us with 32 rows a tile, 177 with 16)
    const int64_t rows = ((int64_t)a.b.T + a.b.B - 1) / a.b.B * p.G;
    const int nt = std::min(rows <= 8 ? 1 : rows <= 16 ? 2 : 4, most_rows(c.cfg.dh / 32));
    return c.cfg.dtype == SPFFN_BF16 ? by_width<__nv_bfloat16>(c, p, nt, st) : by_width<__half>(c, p, nt, st);
}

}  // namespace kv4
}  // namespace spffn
