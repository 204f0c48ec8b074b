// The softmax side of dense attention on the tensor cores: a thread owns one row of a tile of
// logits S (128 rows, 64 keys) in tensor memory (TMEM lane = row) and turns it into bf16 probabilities over
// S's own columns, keeping the row's running maximum and sum in registers.
//
// The maximum is kept stale until a row's new one exceeds it by more than 8 in log2 units: a
// probability then stays below 2^8, which cancels in O / l, and the accumulator is rescaled only
// in the rare step that passes the threshold.  All exponentials go to the multi-function unit: it is
// busy 54 % of the time (packed prompts, 12288 tokens), and a pair of FMA-pipe exponentials (fastexp.cuh) takes
// about ten issue slots of the same warps (one pair in four there: 4 % slower at 32768 tokens).
//
// A NaN or +infinity among a row's visible logits makes its sum NaN (the maximum passes NaN on); a
// hidden position is left out by selection.
#pragma once

#include "ptx.cuh"

namespace sala {
namespace smx {

using namespace ptx;

constexpr float kGrow = 8.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Maxima that pass NaN on.
__device__ __forceinline__ float max2n(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max3n(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// mbar_try_wait that may sleep for up to 20 us before it answers, so that waiting warps leave the issue
// slots to the working ones.
__device__ __forceinline__ bool mbar_try_wait_long(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
// A wait that ends early once the block winds down; a timeout starts the wind-down.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, const DevCtx& ctx,
                                              volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_long(bar, parity)) {
        if (*abort) return false;
        if (globaltimer_ns() - t0 > ctx.wait_limit_ns) {
            flag(ctx, kStatusTimeout);
            *abort = 1;
            return false;
        }
    }
    return true;
}
// The same for a warp that no other one waits for.
__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t parity, const DevCtx& ctx) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_long(bar, parity))
        if (globaltimer_ns() - t0 > ctx.wait_limit_ns) {
            flag(ctx, kStatusTimeout);
            return false;
        }
    return true;
}
// The same with one outcome for the whole (converged) warp.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const DevCtx& ctx,
                                          volatile int* abort) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, ctx, abort));
}

// Maximum of 32 logits; of those whose bit in seen is set (-inf when none is).
__device__ __forceinline__ float max32(const uint32_t* s) {
    float m[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t* x = s + 16 * h;
        float v = max2n(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
        for (int k = 2; k < 16; k += 2) v = max3n(v, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
        m[h] = v;
    }
    return max2n(m[0], m[1]);
}
__device__ __forceinline__ float max32_masked(const uint32_t* s, uint32_t seen) {
    float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < 32; ++k)
        m[k & 1] = max2n(m[k & 1], ((seen >> k) & 1u) ? __uint_as_float(s[k]) : -INFINITY);
    return max2n(m[0], m[1]);
}
// Bits 0 .. lim of 32.
__device__ __forceinline__ uint32_t bits_to(int lim) {
    return lim >= 31 ? 0xffffffffu : lim < 0 ? 0u : (2u << lim) - 1u;
}

// p = 2^(s * sl2 + nb) for 32 logits as 16 bf16 pairs; sums of the unrounded p in acc[0..3].
// kMasked: positions whose bit in seen is clear give exact zeros.  kScaled: the pairs hold p times
// the key's entry of vs (the scale of its row of V), rounded once.
template <bool kMasked, bool kScaled>
__device__ __forceinline__ void exp32(const uint32_t* s, float sl2, float nb, uint32_t seen, const float* vs,
                                      float (&acc)[4], uint32_t (&pk)[16]) {
    [[maybe_unused]] float4 v4;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        const int k = 2 * q;
        float y0, y1, p0, p1;
        fma2_bcast(y0, y1, __uint_as_float(s[k]), __uint_as_float(s[k + 1]), sl2, nb);
        p0 = ex2(y0);
        p1 = ex2(y1);
        if (kMasked) {
            p0 = ((seen >> k) & 1u) ? p0 : 0.f;
            p1 = ((seen >> (k + 1)) & 1u) ? p1 : 0.f;
        }
        if (q & 1) add2(acc[2], acc[3], p0, p1);
        else add2(acc[0], acc[1], p0, p1);
        if (kScaled) {
            if ((q & 1) == 0) v4 = *reinterpret_cast<const float4*>(vs + k);
            mul2(p0, p1, (q & 1) ? v4.z : v4.x, (q & 1) ? v4.w : v4.y);
            if (kMasked) {  // a hidden row's scale may be anything
                p0 = ((seen >> k) & 1u) ? p0 : 0.f;
                p1 = ((seen >> (k + 1)) & 1u) ? p1 : 0.f;
            }
        }
        pk[q] = pack_bf16x2(p0, p1);
    }
}

// A row's running maximum (scaled log2 units) and sum.
struct RowState {
    float m = -INFINITY, l = 0.f;
    // Takes a tile's maximum in; returns the factor for the accumulated output (1: leave it).
    __device__ __forceinline__ float raise(float mx) {
        float alpha = 1.f;
        if (mx > m + kGrow) {
            if (m != -INFINITY) alpha = ex2(m - mx);
            l *= m == -INFINITY ? 0.f : alpha;  // a NaN stays
            m = mx;
        }
        if (!(mx <= 3.402823466e38f)) l = __uint_as_float(0x7fffffffu);
        return alpha;
    }
    // What is added to the scaled logits before the exponential.
    __device__ __forceinline__ float shift() const { return m == -INFINITY ? 0.f : -m; }
};

// O *= alpha, n columns of this thread's row.
template <int N>
__device__ __forceinline__ void scale_row(uint32_t taddr, float alpha) {
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
        uint32_t o[32];
        tmem_ld32(taddr + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 32; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
        tmem_st32(taddr + c, o);
    }
    tmem_st_wait();
}

template <int N>
__device__ __forceinline__ void set_regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Whether any of 8 bf16 values is an infinity or a NaN.
__device__ __forceinline__ bool any_nonfinite8(const uint4& w) {
    constexpr uint32_t e = 0x7f807f80u;
    const uint32_t m = __vmaxu2(__vmaxu2(w.x & e, w.y & e), __vmaxu2(w.z & e, w.w & e));
    return __vcmpeq2(m, e) != 0u;
}

}  // namespace smx
}  // namespace sala
