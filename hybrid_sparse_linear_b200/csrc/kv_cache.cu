// Writing key and value rows into the paged cache, quantised on the way, and reading them back.
//
// HBM-bound: a write reads D elements per row once and stores D codes and one scale; a read is the
// reverse.  A block takes 64 consecutive packed rows: it finds their pages and slots once (a search
// over the offsets and a page lookup per row, one thread each), then moves the rows of its planes
// (keys or values of one head).  A row spans D * sizeof(T) / 16 lanes of 16 bytes, a plane's 64 rows
// are all in flight at once, and the largest magnitude is a butterfly inside the row's lanes on the
// bits of |x|, which order like the numbers.  Long inputs give a block every plane, which spreads
// the search; short ones, where the latency of the chain offsets -> page -> row is the time, give
// each plane a block of its own.  262144 tokens of two heads of 128, bf16 to int8 and back: 139 us, 5.9 TB/s,
// with a plane per block 140; 64 single tokens 3 us a call, with every plane in one block 6.
#include "kv_format.cuh"

namespace sala {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;          // packed rows per block
constexpr int kStaged = 1024;      // offsets kept in shared memory (a longer batch searches global memory)
constexpr unsigned kOffsetBlocks = 1024;  // blocks at most that look through the offsets

// Row of the cache ((page * Hkv + head) * 64 + slot, without the head's part), or -1: not in any
// sequence, or on a page the table does not hold (the latter sets *bad).
__device__ __forceinline__ int place_of(const int32_t* offsets, const int32_t* __restrict__ pos,
                                        const KvPages& p, int B, int Hkv, int r, bool* bad) {
    int lo = 0, hi = B;  // the last b with offsets[b] <= r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (offsets[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    if (lo == B) return -1;  // behind the last sequence
    const int c0 = offsets[lo];
    if (c0 > r || offsets[lo + 1] <= r) {  // offsets out of order, or rows before the first
        *bad = true;
        return -1;
    }
    const int first = __ldg(pos + lo);
    const int64_t at = (int64_t)first + (r - c0);
    const int page = first < 0 || (at >> 6) >= p.max_pages ? -1 : page_of(p, lo, (int)(at >> 6));
    if (page < 0) {
        *bad = true;
        return -1;
    }
    return page * Hkv * kPage + (int)(at & (kPage - 1));
}

// The places of the block's rows, in shared memory.
__device__ __forceinline__ void find_places(int (&place)[kRows], int32_t (&staged)[kStaged], const int32_t* cu,
                                            const int32_t* pos, const KvPages& p, int B, int Hkv, int r0,
                                            int total, const DevCtx& ctx) {
    const bool fits = B + 1 <= kStaged;
    if (fits) {
        for (int i = threadIdx.x; i <= B; i += kThreads) staged[i] = __ldg(cu + i);
        __syncthreads();
    }
    bool bad = false;
    if (threadIdx.x < kRows) {
        const int r = r0 + threadIdx.x;
        place[threadIdx.x] = r < total ? place_of(fits ? staged : cu, pos, p, B, Hkv, r, &bad) : -1;
    } else if (blockIdx.y == 0 && blockIdx.x < kOffsetBlocks) {
        // The other threads meanwhile look for offsets out of order or outside [0, total], which a row's search
        // need not meet.
        const int32_t* o = fits ? staged : cu;
        for (unsigned i = blockIdx.x * (kThreads - kRows) + threadIdx.x - kRows; i < (unsigned)B;
             i += min(gridDim.x, kOffsetBlocks) * (kThreads - kRows))
            bad = bad || o[i] > o[i + 1] || o[i] < 0 || o[i + 1] > total;
    }
    if (bad) flag(ctx, kStatusBounds);
    __syncthreads();
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

// Largest of the magnitudes |x| of 16 bytes, as the bits of an fp32 number.
template <typename T>
__device__ __forceinline__ uint32_t max_bits(const uint4& u) {
    if constexpr (sizeof(T) == 4) {
        constexpr uint32_t k = 0x7fffffffu;
        return max(max(u.x & k, u.y & k), max(u.z & k, u.w & k));
    } else {
        constexpr uint32_t k = 0x7fff7fffu;
        const uint32_t m = __vmaxu2(__vmaxu2(u.x & k, u.y & k), __vmaxu2(u.z & k, u.w & k));
        return max(m << 16, m & 0xffff0000u);
    }
}

// blockIdx.x: 64 packed rows; blockIdx.y: planes blockIdx.y, + gridDim.y, ... of the 2 * Hkv (the keys of
// every head, then the values).
template <typename T, int D, KvFormat F>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(const T* __restrict__ k, const T* __restrict__ v, const int32_t* __restrict__ cu,
                const int32_t* __restrict__ pos, KvPages p, int B, int Hkv, int total, DevCtx ctx) {
    constexpr int kE = 16 / (int)sizeof(T);    // elements per lane
    constexpr int kL = D / kE;                 // lanes per row
    constexpr int kStep = kThreads / kL;       // rows per pass of the block
    constexpr int kU = kRows / kStep;
    __shared__ int place[kRows];
    __shared__ int32_t staged[kStaged];
    const int sub = threadIdx.x / kL, col = (threadIdx.x % kL) * kE, r0 = blockIdx.x * kRows;
    uint4 x[kU];
    auto load = [&](int plane) {
        const T* src = (plane < Hkv ? k : v) + ((int64_t)(plane < Hkv ? plane : plane - Hkv) * total + r0) * D + col;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = u * kStep + sub;
            x[u] = r0 + r < total ? __ldg(reinterpret_cast<const uint4*>(src + (int64_t)r * D)) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load(blockIdx.y);  // on their way while the places are found
    find_places(place, staged, cu, pos, p, B, Hkv, r0, total, ctx);
    for (int plane = blockIdx.y; plane < 2 * Hkv; plane += gridDim.y) {
        const bool is_k = plane < Hkv;
        const int head = is_k ? plane : plane - Hkv;
        char* dst = static_cast<char*>(const_cast<void*>(is_k ? p.k : p.v));
        if (plane != (int)blockIdx.y) load(plane);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            uint32_t m = F == KvFormat::Same ? 0u : max_bits<T>(x[u]);
            if constexpr (F != KvFormat::Same) {
#pragma unroll
                for (int o = kL / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            }
            const int at = place[u * kStep + sub];
            if (at < 0) continue;
            const int64_t row = at + head * kPage;
            if constexpr (F == KvFormat::Same) {
                *reinterpret_cast<uint4*>(dst + (row * D + col) * sizeof(T)) = x[u];
            } else {
                const bool finite = m < 0x7f800000u;
                const RowScale s = row_scale<F>(finite ? __uint_as_float(m) : 1.f);
                float f[kE];
                unpack16<T>(x[u], f);
                uint32_t c[kE / 4];
#pragma unroll
                for (int e = 0; e < kE; e += 4)
                    c[e / 4] = finite ? encode4<F>(f[e], f[e + 1], f[e + 2], f[e + 3], s.mul) : 0u;
                if constexpr (kE == 8) *reinterpret_cast<uint2*>(dst + row * D + col) = make_uint2(c[0], c[1]);
                else *reinterpret_cast<uint32_t*>(dst + row * D + col) = c[0];
                if (col == 0)
                    const_cast<float*>(is_k ? p.k_scale : p.v_scale)[row] =
                        finite ? s.scale : __uint_as_float(0x7fffffffu);
            }
        }
    }
}

template <typename T, int D, KvFormat F>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(KvPages p, const int32_t* __restrict__ cu, const int32_t* __restrict__ pos,
               T* __restrict__ k, T* __restrict__ v, int B, int Hkv, int total, DevCtx ctx) {
    constexpr int kE = 16 / (int)sizeof(T);
    constexpr int kL = D / kE;
    constexpr int kStep = kThreads / kL;
    constexpr int kU = kRows / kStep;
    __shared__ int place[kRows];
    __shared__ int32_t staged[kStaged];
    const int sub = threadIdx.x / kL, col = (threadIdx.x % kL) * kE, r0 = blockIdx.x * kRows;
    find_places(place, staged, cu, pos, p, B, Hkv, r0, total, ctx);
    for (int plane = blockIdx.y; plane < 2 * Hkv; plane += gridDim.y) {
        const bool is_k = plane < Hkv;
        const int head = is_k ? plane : plane - Hkv;
        const char* src = static_cast<const char*>(is_k ? p.k : p.v);
        T* dst = (is_k ? k : v) + ((int64_t)head * total + r0) * D + col;
        uint4 x[kU];
        uint2 c[kU];
        float sc[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int at = place[u * kStep + sub];
            if (at < 0) continue;
            const int64_t row = at + head * kPage;
            if constexpr (F == KvFormat::Same) {
                x[u] = __ldg(reinterpret_cast<const uint4*>(src + (row * D + col) * sizeof(T)));
            } else {
                if constexpr (kE == 8) c[u] = __ldg(reinterpret_cast<const uint2*>(src + row * D + col));
                else c[u].x = __ldg(reinterpret_cast<const uint32_t*>(src + row * D + col));
                sc[u] = __ldg((is_k ? p.k_scale : p.v_scale) + row);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            if (place[u * kStep + sub] < 0) continue;
            if constexpr (F != KvFormat::Same) {
                float f[kE];
#pragma unroll
                for (int e = 0; e < kE; e += 4) {
                    const float4 y = decode4<F>(e == 0 ? c[u].x : c[u].y);
                    f[e] = y.x * sc[u];
                    f[e + 1] = y.y * sc[u];
                    f[e + 2] = y.z * sc[u];
                    f[e + 3] = y.w * sc[u];
                }
                x[u] = pack16<T>(f);
            }
            *reinterpret_cast<uint4*>(dst + (int64_t)(u * kStep + sub) * D) = x[u];
        }
    }
}

// Every plane in one block once the rows alone give each SM a few blocks.
dim3 grid_for(int total, int Hkv) {
    const int chunks = (total + kRows - 1) / kRows;
    int planes = chunks >= 4 * device_sm_count() ? 1 : 2 * Hkv;
    return dim3(chunks, planes < 65535 ? planes : 65535);
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
        kv_write_kernel<T, D, decltype(ff)::value><<<grid_for(total, Hkv), kThreads, 0, st>>>(
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
        kv_read_kernel<T, D, decltype(ff)::value><<<grid_for(total, Hkv), kThreads, 0, st>>>(
            p, cu, pos, static_cast<T*>(k), static_cast<T*>(v), B, Hkv, total, ctx);
        return cudaGetLastError();
    });
}

}  // namespace sala
