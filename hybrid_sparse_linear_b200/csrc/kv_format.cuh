// The paged key/value cache of the dense serving path: its formats, page lookup and element
// conversions, and the row ranges of packed sequences.
#pragma once

#include <cuda_fp8.h>

#include "kernels.h"

namespace sala {

constexpr int kPage = 64;  // tokens per page

// Page of block j of sequence b, or -1 when the table has no such entry or names no page.
__device__ __forceinline__ int page_of(const KvPages& p, int b, int j) {
    if (j < 0 || j >= p.max_pages) return -1;
    const int id = __ldg(p.table + (int64_t)b * p.max_pages + j);
    return id >= 0 && id < p.n_pages ? id : -1;
}

// Quantisation of a row from its largest magnitude a (floored at 2^-100, so that scale and
// reciprocal stay normal numbers).
//   Int8: scale = a / 127, mul = 127 / a, code = the integer nearest to x * mul, ties to even.
//         The product is formed and rounded to an integer in one fused operation, so no second
//         rounding sits next to a border.
//   E4M3: scale = the smallest power of two with a / scale <= 448, mul = its inverse.  e4m3 has
//         its precision relative to each value, so a power of two costs none (down to the type's
//         subnormals) and x * mul and code * scale are exact.
struct RowScale {
    float scale, mul;
};
template <KvFormat F>
__device__ __forceinline__ RowScale row_scale(float a) {
    a = fmaxf(a, 7.8886090522101181e-31f);  // 2^-100
    if constexpr (F == KvFormat::Int8) {
        return {__fdiv_rn(a, 127.f), __fdiv_rn(127.f, a)};
    } else {
        // a = m 2^e with m in [1, 2): a / 2^k <= 448 = 1.75 * 2^8 takes k = e - 8, one more above 1.75
        const uint32_t u = __float_as_uint(a);
        const int k = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
        return {__uint_as_float((uint32_t)(127 + k) << 23), __uint_as_float((uint32_t)(127 - k) << 23)};
    }
}
// Codes of four values, in memory order.
template <KvFormat F>
__device__ __forceinline__ uint32_t encode4(float x0, float x1, float x2, float x3, float mul) {
    if constexpr (F == KvFormat::Int8) {
        constexpr float kShift = 12582912.f;  // 1.5 * 2^23: the integer lands in the low mantissa bits
        const uint32_t c0 = __float_as_uint(fmaf(x0, mul, kShift)), c1 = __float_as_uint(fmaf(x1, mul, kShift));
        const uint32_t c2 = __float_as_uint(fmaf(x2, mul, kShift)), c3 = __float_as_uint(fmaf(x3, mul, kShift));
        return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
    } else {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0 * mul, x1 * mul), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2 * mul, x3 * mul), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
}
// The four code values (without the scale).
template <KvFormat F>
__device__ __forceinline__ float4 decode4(uint32_t c) {
    if constexpr (F == KvFormat::Int8) {
        // code + 128 in the low mantissa byte of 2^23; the difference is the code, exactly
        const uint32_t u = c ^ 0x80808080u;
        constexpr uint32_t k = 0x4b000000u;  // 2^23
        auto f = [&](uint32_t sel) { return __uint_as_float(__byte_perm(u, k, sel)) - 8388736.f; };
        return make_float4(f(0x7440), f(0x7441), f(0x7442), f(0x7443));
    } else {
        const __half2 lo(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3));
        const __half2 hi(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3));
        const float2 a = __half22float2(lo), b = __half22float2(hi);
        return make_float4(a.x, a.y, b.x, b.y);
    }
}

// Two codes as a bf16 pair, exactly (a code has at most 8 significant bits).  u holds a code in each 16
// bits: in the low byte for Int8 (the other zero), in the high byte for E4M3 (the other ignored).
template <KvFormat F>
__device__ __forceinline__ uint32_t code_pair(uint32_t u) {
    if constexpr (F == KvFormat::Int8) {
        // For a byte b, 128 + (b & 127) and 128 or 256 (bit 7 is the last exponent bit of 0x4300 = 128)
        // are bf16 numbers, and their difference is the signed byte.
        const uint32_t x = (u & 0x007f007fu) | 0x43004300u, y = (u & 0x00800080u) | 0x43004300u;
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                         *reinterpret_cast<const __nv_bfloat162*>(&y));
        return *reinterpret_cast<const uint32_t*>(&d);
    } else {
        // s eeee mmm moved to bf16's places is the value times 2^-120 (the biases differ by 120, and
        // e4m3's subnormals become bf16's); the product with 2^120 is exact.
        const uint32_t x = ((u >> 4) & 0x07f007f0u) | (u & 0x80008000u), k = 0x7b807b80u;
        const __nv_bfloat162 d = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x),
                                         *reinterpret_cast<const __nv_bfloat162*>(&k));
        return *reinterpret_cast<const uint32_t*>(&d);
    }
}
// bf16 pairs of four codes in memory order.
template <KvFormat F>
__device__ __forceinline__ uint2 codes_to_bf16(uint32_t c) {
    if constexpr (F == KvFormat::Int8)
        return make_uint2(code_pair<F>(__byte_perm(c, 0u, 0x4140)), code_pair<F>(__byte_perm(c, 0u, 0x4342)));
    else
        return make_uint2(code_pair<F>(__byte_perm(c, 0u, 0x1404)), code_pair<F>(__byte_perm(c, 0u, 0x3424)));
}

// Two codes as an fp16 pair, exactly.  u holds a code in each low byte of 16 bits: for Int8 offset by 128
// (xor 0x80) below the byte 0x64, which makes 1024 + 128 + code; for E4M3 both codes are in the low 16 bits.
template <KvFormat F>
__device__ __forceinline__ uint32_t code_pair_f16(uint32_t u) {
    if constexpr (F == KvFormat::Int8) {
        const uint32_t k = 0x64806480u;  // 1152
        const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&k));
        return *reinterpret_cast<const uint32_t*>(&d);
    } else {
        const __half2 d(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(u & 0xffffu), __NV_E4M3));
        return *reinterpret_cast<const uint32_t*>(&d);
    }
}
// fp16 pairs of four codes in memory order.
template <KvFormat F>
__device__ __forceinline__ uint2 codes_to_f16(uint32_t c) {
    if constexpr (F == KvFormat::Int8) {
        c ^= 0x80808080u;
        return make_uint2(code_pair_f16<F>(__byte_perm(c, 0x64646464u, 0x4140)),
                          code_pair_f16<F>(__byte_perm(c, 0x64646464u, 0x4342)));
    } else {
        return make_uint2(code_pair_f16<F>(c), code_pair_f16<F>(c >> 16));
    }
}
// Codes of two rows a (bytes 0, 1) and b (bytes 2, 3), as a transposing load leaves them: fp16 pairs
// (byte 0, byte 2) and (byte 1, byte 3).
template <KvFormat F>
__device__ __forceinline__ uint2 crossed_to_f16(uint32_t c) {
    if constexpr (F == KvFormat::Int8) {
        c ^= 0x80808080u;
        return make_uint2(code_pair_f16<F>(__byte_perm(c, 0x64646464u, 0x4240)),
                          code_pair_f16<F>(__byte_perm(c, 0x64646464u, 0x4341)));
    } else {
        const uint32_t a = code_pair_f16<F>(c), b = code_pair_f16<F>(c >> 16);
        return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    }
}

// ---------------------------------------------------------------- packed sequences
// Rows cu[b] .. cu[b + 1] of a packed tensor belong to sequence b.  A pair of offsets that does not
// lie in order inside [0, total] counts as an empty sequence and sets *bad.
__device__ __forceinline__ int packed_len(const int32_t* cu, int b, int total, int* start, bool* bad) {
    const int s = __ldg(cu + b), e = __ldg(cu + b + 1);
    *start = s;
    if (s < 0 || e < s || e > total) {
        *bad = true;
        return 0;
    }
    return e - s;
}

// The i-th tile of `rows` rows over all sequences, each sequence's tiles from its end to its start
// (the longest causal rows first).  len = 0: there is no such tile.  By one converged warp.
struct PackedTile {
    int start, len, first;  // the sequence's rows, and the tile's first row inside it
};
__device__ __forceinline__ PackedTile find_packed_tile(const int32_t* cu, int B, int total, int64_t i,
                                                       int rows, int lane, const DevCtx& ctx,
                                                       bool report) {
    int64_t before = 0;
    bool bad = false;
    PackedTile t{0, 0, 0};
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int b = b0 + lane;
        int start = 0;
        const int len = b < B ? packed_len(cu, b, total, &start, &bad) : 0;
        const int n = (len + rows - 1) / rows;
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + inc > i);
        if (hit && t.len == 0) {
            const int w = __ffs((int)hit) - 1;
            t.start = __shfl_sync(0xffffffffu, start, w);
            t.len = __shfl_sync(0xffffffffu, len, w);
            const int64_t end = __shfl_sync(0xffffffffu, before + inc, w);
            t.first = (int)(end - 1 - i) * rows;
            if (!report) return t;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (report && __any_sync(0xffffffffu, bad) && lane == 0) flag(ctx, kStatusBounds);
    return t;
}

// The tiles of `rows` rows (a power of two up to 256) over all sequences, those that begin latest in
// their sequence -- whose causal rows are longest -- first: in levels of 256 rows from the longest
// sequence's last down, and inside a level sequence by sequence.  One converged warp walks them in
// ascending order.
struct PackedOrder {
    static constexpr int kLevel = 256;
    const int32_t* cu;
    int B, total, rows, lane;
    int level;        // the level that holds tiles [before, before + n)
    int64_t before, n;

    // Tiles of sequence b in a level.
    __device__ __forceinline__ int tiles_in(int len, int lv) const {
        const int left = min(len - lv * kLevel, kLevel);
        return left > 0 ? (left + rows - 1) / rows : 0;
    }
    __device__ __forceinline__ int len_of(int b, int* start) const {
        bool bad = false;
        return b < B ? packed_len(cu, b, total, start, &bad) : 0;
    }
    __device__ __forceinline__ int64_t count(int lv) const {
        int64_t s = 0;
        int start;
        for (int b = lane; b < B; b += 32) s += tiles_in(len_of(b, &start), lv);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    }
    // report: flag offsets that are out of order.
    __device__ __forceinline__ PackedOrder(const int32_t* cu, int B, int total, int rows, int lane,
                                           const DevCtx& ctx, bool report)
        : cu(cu), B(B), total(total), rows(rows), lane(lane), before(0) {
        int longest = 0, start;
        bool bad = false;
        for (int b = lane; b < B; b += 32) longest = max(longest, packed_len(cu, b, total, &start, &bad));
        if (report && bad) flag(ctx, kStatusBounds);
        longest = __reduce_max_sync(0xffffffffu, longest);
        level = longest > 0 ? (longest - 1) / kLevel : -1;
        n = level >= 0 ? count(level) : 0;
    }
    // Tile i (not below the i of the last call); len = 0 when there are no more.
    __device__ __forceinline__ PackedTile at(int64_t i) {
        while (level >= 0 && i >= before + n) {
            before += n;
            n = --level >= 0 ? count(level) : 0;
        }
        if (level < 0) return {0, 0, 0};
        int64_t from = before;
        for (int b0 = 0; b0 < B; b0 += 32) {
            int start = 0;
            const int len = len_of(b0 + lane, &start), k = tiles_in(len, level);
            int inc = k;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, from + inc > i);
            if (hit) {
                const int w = __ffs((int)hit) - 1;
                const int end = __shfl_sync(0xffffffffu, inc, w);
                return {__shfl_sync(0xffffffffu, start, w), __shfl_sync(0xffffffffu, len, w),
                        level * kLevel + (int)(from + end - 1 - i) * rows};
            }
            from += __shfl_sync(0xffffffffu, inc, 31);
        }
        return {0, 0, 0};
    }
};

}  // namespace sala
