// Writing key and value rows into the paged cache, quantised on the way, and reading them back.
//
// HBM-bound: a write reads D elements per row once and stores D codes and one scale; a read is the
// reverse.  A row (one token of one KV head) spans D * sizeof(T) / 16 lanes of 16 bytes, so a warp
// instruction covers one to four whole rows and the largest magnitude is a butterfly inside the
// row's lanes; each lane keeps kU rows in flight.  Rows of one head and one page are contiguous on
// both sides, so the stores of a warp fall into whole sectors.
#include "kv_format.cuh"

namespace sala {
namespace {

constexpr int kThreads = 256;
constexpr int kU = 4;  // rows in flight per lane

// Where packed row r stands in the cache: page and slot, or page -1 (not in any sequence, or the
// table does not hold its page; the latter sets *bad).  One search per row over the offsets.
struct Place {
    int page, slot;
};
__device__ __forceinline__ Place place_of(const int32_t* __restrict__ cu, const int32_t* __restrict__ pos,
                                          const KvPages& p, int B, int r, bool* bad) {
    int lo = 0, hi = B;  // the last b with cu[b] <= r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(cu + mid) <= r) lo = mid;
        else hi = mid - 1;
    }
    const int c0 = __ldg(cu + lo);
    if (lo == B) return {-1, 0};             // behind the last sequence
    if (c0 > r || __ldg(cu + lo + 1) <= r) {  // offsets out of order, or rows before the first
        *bad = true;
        return {-1, 0};
    }
    const int64_t at = (int64_t)__ldg(pos + lo) + (r - c0);
    const int64_t j = at >> 6;
    const int page = __ldg(pos + lo) < 0 || j >= p.max_pages ? -1 : page_of(p, lo, (int)j);
    if (page < 0) *bad = true;
    return {page, (int)(at & (kPage - 1))};
}

template <typename T>
__device__ __forceinline__ void unpack16(const uint4& u, float (&f)[16 / sizeof(T)]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            f[i] = __uint_as_float(w[i]);
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&f)[16 / sizeof(T)]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[i] = __float_as_uint(f[i]);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows are numbered tensor (k, v) outermost, then head, then packed row.
template <typename T, int D, KvFormat F>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(const T* __restrict__ k, const T* __restrict__ v, const int32_t* __restrict__ cu,
                const int32_t* __restrict__ pos, KvPages p, int B, int Hkv, int total, DevCtx ctx) {
    constexpr int kE = 16 / (int)sizeof(T);  // elements per lane
    constexpr int kL = D / kE;               // lanes per row
    constexpr int kRPI = 32 / kL;            // rows per warp instruction
    const int lane = threadIdx.x & 31, sub = lane / kL, col = (lane % kL) * kE;
    const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int64_t n_warps = ((int64_t)gridDim.x * kThreads) >> 5;
    const int64_t per = (int64_t)Hkv * total, rows = 2 * per;
    bool bad = false;
    for (int64_t r0 = warp * (kRPI * kU); r0 < rows; r0 += n_warps * (kRPI * kU)) {
        uint4 x[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t r = r0 + u * kRPI + sub;
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) x[u] = __ldg(reinterpret_cast<const uint4*>((r < per ? k + r * D : v + (r - per) * D) + col));
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t r = r0 + u * kRPI + sub;
            float f[kE];
            unpack16<T>(x[u], f);
            float a = 0.f;
            bool finite = true;
#pragma unroll
            for (int e = 0; e < kE; ++e) {
                a = fmaxf(a, fabsf(f[e]));
                finite = finite && fabsf(f[e]) <= 3.402823466e38f;
            }
            int fin = finite;
#pragma unroll
            for (int o = kL / 2; o > 0; o >>= 1) {
                a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                fin &= __shfl_xor_sync(0xffffffffu, fin, o);
            }
            if (r >= rows) continue;
            const bool is_k = r < per;
            const int64_t rr = is_k ? r : r - per;
            const int head = (int)(rr / total);
            const Place at = place_of(cu, pos, p, B, (int)(rr - (int64_t)head * total), &bad);
            if (at.page < 0) continue;
            const int64_t row = ((int64_t)at.page * Hkv + head) * kPage + at.slot;
            char* dst = static_cast<char*>(const_cast<void*>(is_k ? p.k : p.v));
            if constexpr (F == KvFormat::Same) {
                *reinterpret_cast<uint4*>(dst + (row * D + col) * sizeof(T)) = x[u];
            } else {
                const RowScale s = row_scale<F>(a);
                uint32_t c[kE / 4];
#pragma unroll
                for (int e = 0; e < kE; e += 4)
                    c[e / 4] = fin ? encode4<F>(f[e], f[e + 1], f[e + 2], f[e + 3], s.mul) : 0u;
                if constexpr (kE == 8) *reinterpret_cast<uint2*>(dst + row * D + col) = make_uint2(c[0], c[1]);
                else *reinterpret_cast<uint32_t*>(dst + row * D + col) = c[0];
                if (col == 0)
                    const_cast<float*>(is_k ? p.k_scale : p.v_scale)[row] =
                        fin ? s.scale : __uint_as_float(0x7fffffffu);
            }
        }
    }
    if (bad) flag(ctx, kStatusBounds);
}

template <typename T, int D, KvFormat F>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(KvPages p, const int32_t* __restrict__ cu, const int32_t* __restrict__ pos,
               T* __restrict__ k, T* __restrict__ v, int B, int Hkv, int total, DevCtx ctx) {
    constexpr int kE = 16 / (int)sizeof(T);
    constexpr int kL = D / kE;
    constexpr int kRPI = 32 / kL;
    const int lane = threadIdx.x & 31, sub = lane / kL, col = (lane % kL) * kE;
    const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int64_t n_warps = ((int64_t)gridDim.x * kThreads) >> 5;
    const int64_t per = (int64_t)Hkv * total, rows = 2 * per;
    bool bad = false;
    for (int64_t r0 = warp * (kRPI * kU); r0 < rows; r0 += n_warps * (kRPI * kU)) {
        uint4 x[kU];
        uint32_t c[kU][kE / 4];
        float sc[kU];
        bool have[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t r = r0 + u * kRPI + sub;
            have[u] = false;
            if (r >= rows) continue;
            const bool is_k = r < per;
            const int64_t rr = is_k ? r : r - per;
            const int head = (int)(rr / total);
            const Place at = place_of(cu, pos, p, B, (int)(rr - (int64_t)head * total), &bad);
            if (at.page < 0) continue;
            have[u] = true;
            const int64_t row = ((int64_t)at.page * Hkv + head) * kPage + at.slot;
            const char* src = static_cast<const char*>(is_k ? p.k : p.v);
            if constexpr (F == KvFormat::Same) {
                x[u] = __ldg(reinterpret_cast<const uint4*>(src + (row * D + col) * sizeof(T)));
            } else {
#pragma unroll
                for (int e = 0; e < kE / 4; ++e)
                    c[u][e] = __ldg(reinterpret_cast<const uint32_t*>(src + row * D + col) + e);
                sc[u] = __ldg((is_k ? p.k_scale : p.v_scale) + row);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (!have[u]) continue;
            const int64_t r = r0 + u * kRPI + sub;
            if constexpr (F != KvFormat::Same) {
                float f[kE];
#pragma unroll
                for (int e = 0; e < kE; e += 4) {
                    const float4 y = decode4<F>(c[u][e / 4]);
                    f[e] = y.x * sc[u];
                    f[e + 1] = y.y * sc[u];
                    f[e + 2] = y.z * sc[u];
                    f[e + 3] = y.w * sc[u];
                }
                x[u] = pack16<T>(f);
            }
            *reinterpret_cast<uint4*>((r < per ? k + r * D : v + (r - per) * D) + col) = x[u];
        }
    }
    if (bad) flag(ctx, kStatusBounds);
}

int grid_for(int64_t rows, int rows_per_warp) {
    const int64_t blocks = (rows + rows_per_warp * 8 - 1) / (rows_per_warp * 8);
    const int64_t most = (int64_t)device_sm_count() * 8;
    return (int)(blocks < most ? blocks : most);
}

// Calls go(element type, head dim, format) for the runtime values.
template <class Go>
cudaError_t dispatch(DType dt, int d, KvFormat f, Go go) {
    auto with_format = [&](auto t, auto dd) {
        if (f == KvFormat::Int8) return go(t, dd, std::integral_constant<KvFormat, KvFormat::Int8>{});
        if (f == KvFormat::E4M3) return go(t, dd, std::integral_constant<KvFormat, KvFormat::E4M3>{});
        return go(t, dd, std::integral_constant<KvFormat, KvFormat::Same>{});
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (dt == DType::F32) return d == 64 ? with_format(float{}, D64{}) : with_format(float{}, D128{});
    return d == 64 ? with_format(__nv_bfloat16{}, D64{}) : with_format(__nv_bfloat16{}, D128{});
}

}  // namespace

cudaError_t launch_kv_write(DType dt, KvFormat f, const void* k, const void* v, const int32_t* cu,
                            const int32_t* pos, const KvPages& p, int B, int Hkv, int total, int d,
                            cudaStream_t st, DevCtx ctx) {
    return dispatch(dt, d, f, [&](auto t, auto dd, auto ff) {
        using T = decltype(t);
        constexpr int D = decltype(dd)::value;
        const int64_t rows = 2 * (int64_t)Hkv * total;
        kv_write_kernel<T, D, decltype(ff)::value>
            <<<grid_for(rows, 512 / (D * (int)sizeof(T)) * kU), kThreads, 0, st>>>(
                static_cast<const T*>(k), static_cast<const T*>(v), cu, pos, p, B, Hkv, total, ctx);
        return cudaGetLastError();
    });
}

cudaError_t launch_kv_read(DType dt, KvFormat f, const KvPages& p, const int32_t* cu, const int32_t* pos,
                           void* k, void* v, int B, int Hkv, int total, int d, cudaStream_t st,
                           DevCtx ctx) {
    return dispatch(dt, d, f, [&](auto t, auto dd, auto ff) {
        using T = decltype(t);
        constexpr int D = decltype(dd)::value;
        const int64_t rows = 2 * (int64_t)Hkv * total;
        kv_read_kernel<T, D, decltype(ff)::value>
            <<<grid_for(rows, 512 / (D * (int)sizeof(T)) * kU), kThreads, 0, st>>>(
                p, cu, pos, static_cast<T*>(k), static_cast<T*>(v), B, Hkv, total, ctx);
        return cudaGetLastError();
    });
}

}  // namespace sala
