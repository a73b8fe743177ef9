// Shared pieces of the paged 4-bit cache: its block format, the batch of a call, the context.
#pragma once
#include "spffn_block.cuh"

namespace spffn {
namespace kv4 {

// byte offsets inside a block of 16 tokens (NG groups of 32 dims)
template <int NG> struct Blk {
    static constexpr int kV = 256 * NG, kKs = 512 * NG, kKz = 544 * NG, kVs = 576 * NG, kVz = 608 * NG, kBytes = 640 * NG;
    // the 4 bytes of K dims 32 g + 8 c .. + 7 of a token
    static __device__ __forceinline__ int k(int tok, int g, int c) { return tok * 16 * NG + c * 4 * NG + g * 4; }
    // the 2 bytes of V dims 32 g + 4 r .. + 3 of a token
    static __device__ __forceinline__ int v(int tok, int g, int r) {
        return kV + (tok >> 3) * 128 * NG + r * 16 * NG + (tok & 7) * 2 * NG + g * 2;
    }
    static __device__ __forceinline__ int ks(int tok, int g) { return kKs + (tok * NG + g) * 2; }
    static __device__ __forceinline__ int kz(int tok, int g) { return kKz + (tok * NG + g) * 2; }
    static __device__ __forceinline__ int vs(int tok, int g) {
        return kVs + (tok >> 3) * 16 * NG + ((tok & 7) >> 1) * 4 * NG + g * 4 + (tok & 1) * 2;
    }
    static __device__ __forceinline__ int vz(int tok, int g) { return vs(tok, g) + 32 * NG; }
};

constexpr int kMaxLen = 1 << 30;      // positions stay well inside 32 bits, their sums too

// The sequences of a call.
struct Batch {
    const int32_t *table, *lens, *start;
    int64_t ldt;
    int width, B, T, page, page_log, pages;
    uint32_t* err;
};

struct Seq {
    int row0, n, len;     // first row, new tokens, total length; n = 0: no rows of this call
    bool ok;              // false: its length is out of range, it caches and attends to nothing
};

__device__ __forceinline__ Seq seq_of(const Batch& b, int s) {
    Seq q;
    q.row0 = b.start ? b.start[s] : s;
    const int row1 = b.start ? b.start[s + 1] : s + 1;
    q.len = b.lens[s];
    q.n = row1 - q.row0;
    q.ok = true;
    if (q.row0 < 0 || row1 < q.row0 || row1 > b.T) {
        latch(b.err, ERR_BATCH_ROWS);
        q.n = 0;
    }
    if (q.len < q.n || (int64_t)q.len > (int64_t)b.width * b.page || q.len > kMaxLen) {
        latch(b.err, ERR_BATCH_LEN);
        q.ok = false;
        q.len = 0;
    }
    return q;
}

// The sequence that row t belongs to, -1 for a row behind the last (or between broken starts).
__device__ __forceinline__ int seq_of_row(const Batch& b, int t) {
    if (!b.start) return t < b.B ? t : -1;
    int lo = 0, hi = b.B;                    // the last s with start[s] <= t
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (b.start[m] <= t) lo = m;
        else hi = m;
    }
    return b.start[lo] <= t && t < b.start[lo + 1] ? lo : -1;
}

// The shares that a row is cut into, as the first of them leaves it for the join: that share, how many more, and the
// row's place in its tile.
struct Cuts {
    uint32_t first, more, in;
};
inline __host__ __device__ uint2 pack_cuts(const Cuts& c) { return uint2{c.first | (c.in << 24), c.more}; }
inline __host__ __device__ Cuts unpack_cuts(uint2 m) { return Cuts{m.x & 0xffffffu, m.y, m.x >> 24}; }
// Whether they lie in a call of `many` shares of tiles of R rows: after a wait that ran out an entry may be an earlier
// call's, of another tile height, and its parts would lie behind the workspace.
inline __host__ __device__ bool cuts_in(const Cuts& c, int many, int R) {
    return c.first < (uint32_t)many && c.more < (uint32_t)many - c.first && c.in < (uint32_t)R;
}

struct Layout {
    size_t ctl, meta, part, total;
};

}  // namespace kv4
}  // namespace spffn

struct spffn_kv4_ctx {
    spffn_kv4_config cfg;
    uint8_t* pool;
    const double* freqs;
    char* ws;
    spffn::kv4::Layout lay;
    int device, sms;

    uint32_t* err() const { return reinterpret_cast<uint32_t*>(ws + lay.ctl); }
};

namespace spffn {
namespace kv4 {
struct AttendArgs {
    const void* q;
    void* out;
    int64_t ldq, ldo;
    float scale;
    Batch b;
};
Layout layout(const spffn_kv4_config& c, int sms);
cudaError_t launch_attend(const spffn_kv4_ctx& c, const AttendArgs& a, cudaStream_t st);
}  // namespace kv4
}  // namespace spffn
