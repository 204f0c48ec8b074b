// Joins the partial results of the attention over a paged cache (tree_plan.cuh): with the partials
// (m_i, l_i, o_i) of a row, m = max m_i, out = sum 2^(m_i - m) o_i / sum 2^(m_i - m) l_i, in
// 32 bits and in CTA order, so the result does not depend on which CTA finished first.
//
// A warp per row: it redoes the plan's arithmetic to find the CTAs that share the row's item
// (returning at once when one CTA had it whole), takes the maximum and the weights lane by lane
// and then adds the outputs, a lane per D / 32 columns.  Reads come from L2: the partials were
// written by the launch before.
#include "kernels.h"
#include "ptx.cuh"
#include "tree_plan.cuh"

namespace sala {
namespace {

constexpr int kWarps = 8;

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
tree_join_kernel(tree::Partials part, T* __restrict__ out, tree::Shape s, int rt, int n_cta) {
    const int lane = threadIdx.x & 31;
    const int item = blockIdx.y;  // b * Hkv + g
    const int b = item / s.Hkv, g = item % s.Hkv;
    cudaGridDependencySynchronize();
    // where the group's items start in the line of tiles
    long long w = 0, before = 0;
    for (int i = lane; i < s.B; i += 32) {
        const int n = tree::places_of(s, tree::ctx_of(s, i));
        w += n;
        if (i < b) before += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        w += __shfl_xor_sync(0xffffffffu, w, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    const long long per = (long long)s.Hkv * s.n_rt;
    w *= per;
    const int n_tiles = tree::tiles_of(s, tree::ctx_of(s, b));
    for (int row = blockIdx.x * kWarps + (threadIdx.x >> 5); row < s.rows; row += gridDim.x * kWarps) {
        const int r_tile = row / rt;
        const long long x0 = before * per + ((long long)g * s.n_rt + r_tile) * (n_tiles + s.pad) + s.pad;
        const long long x1 = x0 + n_tiles;  // the item's tiles
        const int c0 = tree::run_of(w, x0, n_cta), c1 = tree::run_of(w, x1 - 1, n_cta);
        if (c0 == c1) continue;  // one CTA had the item whole and wrote the row
        auto slot = [&](int c) { return ((size_t)c * 2 + (c == c0 ? 1 : 0)) * rt + row % rt; };
        // A CTA between the two whose run is empty (fewer tiles than CTAs) left nothing.
        auto empty = [&](int c) { return tree::run_start(w, c, n_cta) == tree::run_start(w, c + 1, n_cta); };
        float m = -INFINITY;
        bool nan = false;
        for (int c = c0 + lane; c <= c1; c += 32)
            if (!empty(c)) {
                const float mc = part.ml[slot(c)].x;
                nan = nan || mc != mc;
                m = fmaxf(m, mc);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        nan = __any_sync(0xffffffffu, nan);
        constexpr int kC = D / 32;
        float acc[kC] = {};
        float l = 0.f;
        for (int base = c0; base <= c1; base += 32) {
            const int c = base + lane;
            float wt = 0.f, lc = 0.f;
            bool seen = false;  // the row saw a key there
            if (c <= c1 && !empty(c)) {
                const float2 ml = part.ml[slot(c)];
                seen = ml.x != -INFINITY || ml.y != 0.f;
                if (seen) {
                    wt = exp2f(ml.x - m);
                    lc = ml.y * wt;
                }
            }
            // Eight at a time, so that their reads are on the way together.
            const unsigned who = __ballot_sync(0xffffffffu, seen);
            const int n = min(32, c1 - base + 1);
            for (int i0 = 0; i0 < n; i0 += 8) {
                float2 x[8][kC / 2];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool take = (who >> (i0 + i)) & 1u;
                    const float* src = part.o + slot(base + i0 + i) * D + lane * kC;
#pragma unroll
                    for (int e = 0; e < kC / 2; ++e)
                        x[i][e] = take ? reinterpret_cast<const float2*>(src)[e] : make_float2(0.f, 0.f);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float wi = __shfl_sync(0xffffffffu, wt, (i0 + i) & 31);
                    l += __shfl_sync(0xffffffffu, lc, (i0 + i) & 31);
#pragma unroll
                    for (int e = 0; e < kC / 2; ++e) {
                        acc[2 * e] += wi * x[i][e].x;
                        acc[2 * e + 1] += wi * x[i][e].y;
                    }
                }
            }
        }
        const float inv = nan ? __uint_as_float(0x7fffffffu) : l == 0.f ? 0.f : 1.f / l;
        T* dst = out + ((int64_t)item * s.rows + row) * D + lane * kC;
#pragma unroll
        for (int e = 0; e < kC; e += 2) {
            if constexpr (sizeof(T) == 2)
                *reinterpret_cast<uint32_t*>(dst + e) = ptx::pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
            else
                *reinterpret_cast<float2*>(dst + e) = make_float2(acc[e] * inv, acc[e + 1] * inv);
        }
    }
}

template <typename T, int D>
cudaError_t join(tree::Partials part, void* out, const tree::Shape& s, int rt, int n_cta, cudaStream_t st) {
    const int items = s.B * s.Hkv;
    int bx = (s.rows + kWarps - 1) / kWarps;
    const int most = 16 * device_sm_count() / items;  // enough blocks; each then takes several rows
    if (bx > most) bx = most < 1 ? 1 : most;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(bx, items);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<T, D>, part, static_cast<T*>(out), s, rt, n_cta);
}

}  // namespace

cudaError_t launch_tree_join(DType dt, const tree::Partials& part, void* out, const tree::Shape& s,
                             int rt, int d, int n_cta, cudaStream_t st) {
    if (dt == DType::F32)
        return d == 64 ? join<float, 64>(part, out, s, rt, n_cta, st) : join<float, 128>(part, out, s, rt, n_cta, st);
    return d == 64 ? join<__nv_bfloat16, 64>(part, out, s, rt, n_cta, st)
                   : join<__nv_bfloat16, 128>(part, out, s, rt, n_cta, st);
}

}  // namespace sala
