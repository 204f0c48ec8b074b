// How the attention of drafted tokens over a paged cache divides its work, shared by the
// tensor-core kernel, the fp32 kernel and the kernel that joins their partial results.
//
// An item is (sequence b, KV head g, row tile rt): up to RT of the G * T query rows of the group
// against all keys of the sequence, tiles(b) = ceil((ctx_b + T) / KT) key tiles long.  Laid end to
// end (b outermost, then g, then rt), each behind `pad` empty places that stand for the cost of
// beginning an item, the items form one line of W places, and CTA c of n takes the places
// [W c / n, W (c + 1) / n): every CTA has about the same work, however ragged the contexts are, and
// no host-side knowledge of them is needed.  A CTA that has all tiles of an item writes the result;
// else it leaves a partial (row maximum, row sum, unnormalised output) in one of its two slots --
// slot 1 when it has the item's first tile, else slot 0 -- and the join kernel, which redoes the same
// arithmetic, adds up the partials in CTA order.
#pragma once

#include "common.cuh"

namespace sala {
namespace tree {

struct Shape {
    const int32_t* ctx;  // [B] context lengths
    int B, Hkv, G, T, max_ctx;
    int rows;            // G * T query rows per (b, g)
    int n_rt;            // row tiles per (b, g)
    int kt;              // keys per tile
    int pad;             // places in front of an item
};

__host__ __device__ __forceinline__ int row_tiles(int rows, int rt) { return (rows + rt - 1) / rt; }

// Context length of sequence b, clamped to [0, max_ctx] (a value outside is flagged by the caller
// that passes bad).
__device__ __forceinline__ int ctx_of(const Shape& s, int b, bool* bad = nullptr) {
    const int c = __ldg(s.ctx + b);
    if (c < 0 || c > s.max_ctx) {
        if (bad) *bad = true;
        return c < 0 ? 0 : s.max_ctx;
    }
    return c;
}
__device__ __forceinline__ int tiles_of(const Shape& s, int ctx) { return (ctx + s.T + s.kt - 1) / s.kt; }

// Places of an item of sequence b.
__device__ __forceinline__ int places_of(const Shape& s, int ctx) { return tiles_of(s, ctx) + s.pad; }

// W, by one converged warp (every lane gets it).
__device__ __forceinline__ long long total_places(const Shape& s, int lane, bool* bad) {
    long long w = 0;
    for (int b = lane; b < s.B; b += 32) w += places_of(s, ctx_of(s, b, bad));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    return w * s.Hkv * s.n_rt;
}

__device__ __forceinline__ long long run_start(long long w, int c, int n) { return w * c / n; }
// The CTA whose run holds place x (0 <= x < w).
__device__ __forceinline__ int run_of(long long w, long long x, int n) {
    return (int)(((x + 1) * n - 1) / w);  // the last c with floor(w c / n) <= x
}

// One item and the part of it that a run covers.
struct Cursor {
    int b, g, rt;
    int ctx, n_tiles;    // of sequence b
    int tile;            // first tile of the item inside the run (negative: that many places before it)
    long long left;      // places of the run from here on
};

// The cursor at place x of the line, by one converged warp; left is the run's length.
__device__ __forceinline__ Cursor find_place(const Shape& s, long long x, long long left, int lane) {
    Cursor c;
    c.left = left;
    const long long per = (long long)s.Hkv * s.n_rt;
    long long before = 0;
    for (int b0 = 0; b0 < s.B; b0 += 32) {
        const int b = b0 + lane;
        const int ctx = b < s.B ? ctx_of(s, b) : 0;
        long long n = b < s.B ? places_of(s, ctx) * per : 0, inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, b < s.B && before + inc > x);
        if (hit) {
            const int w = __ffs((int)hit) - 1;
            const long long start = __shfl_sync(0xffffffffu, before + inc - n, w);
            c.ctx = __shfl_sync(0xffffffffu, ctx, w);
            c.b = b0 + w;
            c.n_tiles = tiles_of(s, c.ctx);
            const long long r = x - start;
            const int len = c.n_tiles + s.pad;
            const int item = (int)(r / len);
            c.tile = (int)(r - (long long)item * len) - s.pad;
            c.g = item / s.n_rt;
            c.rt = item - c.g * s.n_rt;
            return c;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    c.b = s.B;  // past the end
    c.g = c.rt = c.ctx = c.tile = 0;
    c.n_tiles = 1;
    c.left = 0;
    return c;
}

// The cursor of a CTA that has item i whole and nothing else (i = (b * Hkv + g) * n_rt + rt).
__device__ __forceinline__ Cursor item_at(const Shape& s, int i, bool* bad) {
    Cursor c;
    c.rt = i % s.n_rt;
    c.g = i / s.n_rt % s.Hkv;
    c.b = i / s.n_rt / s.Hkv;
    c.tile = 0;
    c.ctx = ctx_of(s, c.b, bad);
    c.n_tiles = tiles_of(s, c.ctx);
    c.left = c.n_tiles;
    return c;
}

// Places of the cursor's item inside the run, and the tiles among them: [first_tile, first_tile + n).
__device__ __forceinline__ int run_places(const Cursor& c) {
    const long long n = c.n_tiles - c.tile;
    return (int)(n < c.left ? n : c.left);
}
__device__ __forceinline__ int first_tile(const Cursor& c) { return c.tile < 0 ? 0 : c.tile; }
__device__ __forceinline__ int run_tiles(const Cursor& c) {
    const int n = run_places(c) + (c.tile < 0 ? c.tile : 0);
    return n < 0 ? 0 : n;
}

__device__ __forceinline__ void next_item(const Shape& s, Cursor& c) {
    c.left -= run_places(c);
    c.tile = -s.pad;
    if (++c.rt == s.n_rt) {
        c.rt = 0;
        if (++c.g == s.Hkv) {
            c.g = 0;
            ++c.b;
            if (c.left > 0 && c.b < s.B) {
                c.ctx = ctx_of(s, c.b);
                c.n_tiles = tiles_of(s, c.ctx);
            } else {
                c.left = 0;
            }
        }
    }
}

// CTAs of the tensor-core and warp-tile kernels: at most one per SM, and where the tiles are few, `least` to
// four tiles each, so that an item has up to 32 partials (what the join reads in one pass).  In us, one
// sequence, 2 KV heads of 16 query heads, bf16: one token over 128 pages 14.9 (a tile per CTA: 24.7), two
// tokens 18.6 (29.2), over 48 pages 16.7 (18.7).
inline int run_ctas(const Shape& s, int tiles, int least, int sms) {
    const int by32 = (tiles + 31) / 32, run = by32 < least ? least : by32 < 4 ? by32 : 4;
    const long long n = ((long long)s.B * s.Hkv * s.n_rt * tiles + run - 1) / run;
    return n < sms ? (int)n : sms;
}

// Bits of the drafts that row t of sequence b attends to.
__device__ __forceinline__ uint64_t draft_bits(const uint64_t* masks, int b, int t, int T) {
    const uint64_t m = __ldg(reinterpret_cast<const unsigned long long*>(masks) + (int64_t)b * T + t);
    return T >= 64 ? m : m & ((1ull << T) - 1);
}

// Partials: per CTA and slot, rt rows of (maximum in scaled log2 units, sum), then rt rows of d.
__host__ __device__ __forceinline__ size_t partial_rows(int n_cta, int rt) { return (size_t)n_cta * 2 * rt; }
struct Partials {
    float2* ml;
    float* o;
};
__host__ __device__ __forceinline__ size_t partial_bytes(int n_cta, int rt, int d) {
    return partial_rows(n_cta, rt) * (sizeof(float2) + (size_t)d * sizeof(float));
}
inline Partials partials_at(void* ws, int n_cta, int rt) {
    Partials p;
    p.ml = static_cast<float2*>(ws);
    p.o = reinterpret_cast<float*>(p.ml + partial_rows(n_cta, rt));
    return p;
}

}  // namespace tree
}  // namespace sala
