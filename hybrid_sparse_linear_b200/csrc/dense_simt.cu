// Dense softmax attention on the CUDA cores, for packed prompts and for drafted tokens over a
// paged cache: the fp32 form of both (the bf16 form runs on the tensor cores).
//
// One block takes 16 R query rows (R = 1, 2 or 4 per thread) and walks 64-key tiles with the running
// maximum and sum of the softmax in registers: S = Q K^T as R x 4 values per thread, P through shared
// memory, O += P V with R x D/16 sums per thread.  V's tile is on its way into registers while S is
// formed and the next K's while P V is (loads at the point of use: 150 against 139 us for 2049 ragged
// tokens of eight heads of 64, R = 4).
//
// Bound: shared-memory reads.  A 16-byte read takes a warp four cycles, and 4 + R of them feed 16 R
// multiply-adds per thread, which take 4 R cycles: 29 TFLOP/s at R = 4 on long prompts (32 heads of 128,
// 3000 tokens: 2.5 ms; R = 2: 3.2).  Smaller R is for rows that would be empty and for few blocks: one token
// of 16 heads per KV head over 16 int8 caches of 4000 takes 96 us at R = 1, 187 at R = 4, two tokens 112 at
// R = 2; the 2049 ragged tokens take 114 us at R = 2, 134 at R = 4, because the longest rows' blocks decide.
//
// Masked positions are left out by selection, never by adding a large negative number or by
// multiplying with zero: a hidden key or value may hold an infinity or a NaN without touching the
// rows that do not see it.  A row that sees no key gives zeros.
#include <type_traits>

#include "kernels.h"
#include "kv_format.cuh"
#include "ptx.cuh"
#include "tree_plan.cuh"

namespace sala {
namespace {

constexpr int kKeys = 64;   // keys per tile: one page of the paged cache
constexpr int kThreads = 256;
constexpr int kPad = 4;     // floats: 16-byte rows that start 4 banks apart
// Beginning an item costs about a tile: one token of 16 heads per KV head over 16 int8 contexts of up to 9000 tokens
// 82 us (0: 85, 3: 82).
constexpr int kPad0 = 1;
constexpr float kHidden = -1.f;  // P of a position its row does not see (probabilities are >= 0)

// R: query rows per thread; a block has 16 R.
template <int D, int R>
constexpr int smem_floats() { return (16 * R + 2 * kKeys) * (D + kPad) + 16 * R * (kKeys + kPad); }
// Blocks per SM that its shared memory and registers hold.
template <int D, int R>
constexpr int packed_blocks() { return D == 64 ? (R == 4 ? 2 : 3) : (R == 4 ? 1 : 2); }
template <int D, int R>
constexpr int tree_blocks() { return D == 64 || R < 4 ? 2 : 1; }

// The state of 16 R query rows in 256 threads: thread (ty, tx) = (tid / 16, tid % 16) holds rows
// R ty .. R ty + R - 1 and of each the output columns 64 j + 4 tx .. + 3.
template <int D, int R>
struct Rows {
    float m[R], l[R];        // running maximum (scaled log2 units), running sum
    float acc[R][D / 16];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[i][c] = 0.f;
        }
    }
};

// A tile's K or V on its way: 4 consecutive floats of row r per thread and step, by load(r, c).
template <int D>
struct Fetch {
    static constexpr int kN = kKeys * (D / 4) / kThreads;
    float4 x[kN];
    template <class Load>
    __device__ __forceinline__ void get(Load load) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = threadIdx.x + i * kThreads;
            x[i] = load(e / (D / 4), (e % (D / 4)) * 4);
        }
    }
    __device__ __forceinline__ void put(float* sm) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = threadIdx.x + i * kThreads;
            *reinterpret_cast<float4*>(sm + e / (D / 4) * (D + kPad) + (e % (D / 4)) * 4) = x[i];
        }
    }
};

// One key tile; k holds its K.  load_v loads its V, next_k the next tile's K into k; seen(row, key) says
// whether the row attends to the tile's key; masked: whether any position may be hidden.
template <int D, int R, class LoadV, class NextK, class Seen>
__device__ __forceinline__ void attend_tile(Rows<D, R>& st, float* sm, float sl2, bool masked, Fetch<D>& k,
                                            LoadV load_v, NextK next_k, Seen seen) {
    constexpr int kLd = D + kPad, kLp = kKeys + kPad;
    float* Q = sm;
    float* K = sm + 16 * R * kLd;
    float* V = K + kKeys * kLd;
    float* P = V + kKeys * kLd;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    k.put(K);  // (S of the tile before is done with it: a barrier lies between)
    __syncthreads();
    Fetch<D> v;
    v.get(load_v);
    float s[R][4] = {};
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 a[R], b[4];
#pragma unroll
        for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const float4*>(Q + (ty * R + i) * kLd + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(K + (tx + 16 * j) * kLd + c);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[i][j] = fmaf(a[i].w, b[j].w, fmaf(a[i].z, b[j].z, fmaf(a[i].y, b[j].y, fmaf(a[i].x, b[j].x, s[i][j]))));
    }
    // A NaN logit has to reach its row: fmaxf drops it from the maximum, exp2f passes it on.
#pragma unroll
    for (int i = 0; i < R; ++i) {
        bool vis[4];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            vis[j] = !masked || seen(ty * R + i, tx + 16 * j);
            s[i][j] *= sl2;
            if (vis[j]) mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float m_new = fmaxf(st.m[i], mx);
        const float alpha = st.m[i] == -INFINITY ? 0.f : exp2f(st.m[i] - m_new);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float p = vis[j] ? (s[i][j] == -INFINITY ? 0.f : exp2f(s[i][j] - m_new)) : kHidden;
            if (vis[j]) sum += p;
            P[(ty * R + i) * kLp + tx + 16 * j] = p;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        st.l[i] = st.l[i] * alpha + sum;
        st.m[i] = m_new;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) st.acc[i][c] *= alpha;
    }
    v.put(V);
    __syncthreads();
    next_k(k);
    auto pv = [&](auto hide) {
#pragma unroll 2
        for (int k = 0; k < kKeys; k += 4) {
            float4 p[R];
#pragma unroll
            for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty * R + i) * kLp + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const float4 v = *reinterpret_cast<const float4*>(V + (k + kk) * kLd + 64 * j + 4 * tx);
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                        if (decltype(hide)::value && w == kHidden) continue;
                        st.acc[i][4 * j] += w * v.x;
                        st.acc[i][4 * j + 1] += w * v.y;
                        st.acc[i][4 * j + 2] += w * v.z;
                        st.acc[i][4 * j + 3] += w * v.w;
                    }
                }
        }
    };
    if (masked) pv(std::true_type{});
    else pv(std::false_type{});
}

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }

// Four values of row `row` of the cache's keys or values.
template <KvFormat F>
__device__ __forceinline__ float4 kv_load4(const void* p, const float* scale, int64_t row, int d, int col) {
    if constexpr (F == KvFormat::Same) {
        return load4(static_cast<const float*>(p) + row * d + col);
    } else {
        const float4 x = decode4<F>(__ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p) + row * d + col)));
        const float s = __ldg(scale + row);
        return make_float4(x.x * s, x.y * s, x.z * s, x.w * s);
    }
}

// ---------------------------------------------------------------- packed prompts
// Block = (16 R consecutive tokens of one sequence, one query head); blockIdx.x counts the tiles of
// all sequences, an upper bound of which the host launches.
template <int D, int R>
__global__ void __launch_bounds__(kThreads, packed_blocks<D, R>())
packed_simt_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                   const int32_t* __restrict__ cu, float* __restrict__ out, int B, int H, int Hkv,
                   int total, float sl2, DevCtx ctx) {
    constexpr int kRows = 16 * R;
    extern __shared__ __align__(16) float sm[];
    __shared__ PackedTile tile;
    const int tid = threadIdx.x;
    if (tid < 32) {
        const PackedTile t = find_packed_tile(cu, B, total, blockIdx.x, kRows, tid, ctx,
                                              blockIdx.x == 0 && blockIdx.y == 0);
        if (tid == 0) tile = t;
    }
    __syncthreads();
    const PackedTile t = tile;
    if (t.len <= 0) return;
    const int h = blockIdx.y, kvh = h / (H / Hkv);
    const int64_t row0 = (int64_t)h * total + t.start + t.first;
    const float* kb = k + ((int64_t)kvh * total + t.start) * D;
    const float* vb = v + ((int64_t)kvh * total + t.start) * D;
    const int n_rows = min(kRows, t.len - t.first), last = t.first + n_rows - 1;
    constexpr int kLd = D + kPad;
    for (int e = tid; e < kRows * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        *reinterpret_cast<float4*>(sm + r * kLd + c) =
            r < n_rows ? load4(q + (row0 + r) * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    Rows<D, R> st;
    st.clear();
    auto load = [&](const float* base, int j, int c) {  // key or value j
        return j < t.len ? load4(base + (int64_t)j * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    Fetch<D> kf;
    kf.get([&](int r, int c) { return load(kb, r, c); });
    for (int k0 = 0; k0 <= last; k0 += kKeys) {
        attend_tile<D, R>(st, sm, sl2, k0 + kKeys > t.first, kf,
                       [&](int r, int c) { return load(vb, k0 + r, c); },
                       [&](Fetch<D>& f) {
                           if (k0 + kKeys <= last) f.get([&](int r, int c) { return load(kb, k0 + kKeys + r, c); });
                       },
                       [&](int row, int key) { return k0 + key <= t.first + row; });
    }
    const int ty = tid >> 4, tx = tid & 15;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = ty * R + i;
        if (r >= n_rows) continue;
        const float inv = 1.f / st.l[i];  // every row sees itself
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
            store4(out + (row0 + r) * D + 64 * j + 4 * tx,
                   make_float4(st.acc[i][4 * j] * inv, st.acc[i][4 * j + 1] * inv,
                               st.acc[i][4 * j + 2] * inv, st.acc[i][4 * j + 3] * inv));
    }
}

// ---------------------------------------------------------------- drafted tokens, paged cache
template <int D, KvFormat F, int R>
__global__ void __launch_bounds__(kThreads, tree_blocks<D, R>())
tree_simt_kernel(const float* __restrict__ q, KvPages pages, const uint64_t* __restrict__ masks,
                 float* __restrict__ out, tree::Shape s, tree::Partials part, float sl2, DevCtx ctx) {
    constexpr int kRows = 16 * R;
    extern __shared__ __align__(16) float sm[];
    __shared__ tree::Cursor cur0;
    __shared__ uint64_t bits[kRows];
    const int tid = threadIdx.x;
    if (tid < 32) {
        bool bad = false;
        const long long w = tree::total_places(s, tid, &bad);
        const long long x0 = tree::run_start(w, blockIdx.x, gridDim.x);
        const long long x1 = tree::run_start(w, blockIdx.x + 1, gridDim.x);
        const tree::Cursor c = tree::find_place(s, x0, x1 - x0, tid);
        if (bad && blockIdx.x == 0) flag(ctx, kStatusBounds);
        if (tid == 0) cur0 = c;
    }
    __syncthreads();
    tree::Cursor c = cur0;
    constexpr int kLd = D + kPad;
    const int ty = tid >> 4, tx = tid & 15;
    for (; c.left > 0; tree::next_item(s, c)) {
        const int r0 = c.rt * kRows, n_rows = min(kRows, s.rows - r0);
        const int n = tree::run_tiles(c), t0 = tree::first_tile(c);
        if (n == 0) continue;
        const int64_t row0 = ((int64_t)c.b * s.Hkv + c.g) * s.rows + r0;
        __syncthreads();  // the previous item is done with Q and bits
        for (int e = tid; e < kRows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), col = (e % (D / 4)) * 4;
            *reinterpret_cast<float4*>(sm + r * kLd + col) =
                r < n_rows ? load4(q + (row0 + r) * D + col) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (tid < kRows) bits[tid] = tid < n_rows ? tree::draft_bits(masks, c.b, (r0 + tid) % s.T, s.T) : 0ull;
        __syncthreads();
        Rows<D, R> st;
        st.clear();
        // A page the table does not hold: its keys are left out.
        auto page_at = [&](int tl) { return page_of(pages, c.b, tl); };
        auto load = [&](const void* p, const float* sc, int page, int tl, int r, int col) {
            const bool have = page >= 0 && tl * kKeys + r < c.ctx + s.T;
            return have ? kv_load4<F>(p, sc, ((int64_t)page * s.Hkv + c.g) * kKeys + r, D, col)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
        };
        int page = page_at(t0);
        Fetch<D> kf;
        kf.get([&](int r, int col) { return load(pages.k, pages.k_scale, page, t0, r, col); });
        for (int t = t0; t < t0 + n; ++t) {
            if (page < 0 && tid == 0) flag(ctx, kStatusBounds);
            const int next = t + 1 < t0 + n ? page_at(t + 1) : -1, k0 = t * kKeys;
            attend_tile<D, R>(st, sm, sl2, k0 + kKeys > c.ctx || page < 0, kf,
                           [&](int r, int col) { return load(pages.v, pages.v_scale, page, t, r, col); },
                           [&](Fetch<D>& f) {
                               f.get([&](int r, int col) { return load(pages.k, pages.k_scale, next, t + 1, r, col); });
                           },
                           [&](int row, int key) {
                               const int j = k0 + key - c.ctx;  // draft number
                               return page >= 0 && (j < 0 || (j < s.T && ((bits[row] >> j) & 1ull)));
                           });
            page = next;
        }
        const bool whole = n == c.n_tiles;
        const size_t slot = ((size_t)blockIdx.x * 2 + (t0 > 0 ? 0 : 1)) * min(s.rows, kRows);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = ty * R + i;
            if (r >= n_rows) continue;
            const float inv = !whole ? 1.f : st.m[i] == -INFINITY && st.l[i] == 0.f ? 0.f : 1.f / st.l[i];
            if (!whole && tx == 0) part.ml[slot + r] = make_float2(st.m[i], st.l[i]);
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const float4 x = make_float4(st.acc[i][4 * j] * inv, st.acc[i][4 * j + 1] * inv,
                                             st.acc[i][4 * j + 2] * inv, st.acc[i][4 * j + 3] * inv);
                if (whole) store4(out + (row0 + r) * D + 64 * j + 4 * tx, x);
                else store4(part.o + (slot + r) * D + 64 * j + 4 * tx, x);
            }
        }
    }
}

template <int D, int R>
cudaError_t packed_simt(const void* q, const void* k, const void* v, const int32_t* cu, void* o,
                        int B, int H, int Hkv, int total, float scale, cudaStream_t st, DevCtx ctx) {
    constexpr int bytes = smem_floats<D, R>() * 4;
    if (cudaError_t e = ensure_smem<packed_simt_kernel<D, R>>(bytes); e != cudaSuccess) return e;
    // every sequence has at most one tile that is not full
    const long long tiles = (long long)total / (16 * R) + (B < total ? B : total);
    packed_simt_kernel<D, R><<<dim3((unsigned)tiles, H), kThreads, bytes, st>>>(
        static_cast<const float*>(q), static_cast<const float*>(k), static_cast<const float*>(v), cu,
        static_cast<float*>(o), B, H, Hkv, total, scale * 1.4426950408889634f, ctx);
    return cudaGetLastError();
}

// Rows per thread for a group's rows (the smallest block that holds them), and the rows of a partial slot.
int rows_per_thread(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
int slot_rows(int rows) { return rows < 64 ? rows : 64; }
template <int D, int R>
int tree_ctas() { return tree_blocks<D, R>() * device_sm_count(); }
int tree_ctas(int rows, int d) {
    switch (rows_per_thread(rows)) {
        case 1: return d == 64 ? tree_ctas<64, 1>() : tree_ctas<128, 1>();
        case 2: return d == 64 ? tree_ctas<64, 2>() : tree_ctas<128, 2>();
        default: return d == 64 ? tree_ctas<64, 4>() : tree_ctas<128, 4>();
    }
}

template <int D, KvFormat F, int R>
cudaError_t tree_simt(const void* q, const KvPages& pages, const uint64_t* masks, void* o,
                      tree::Shape s, void* ws, float scale, cudaStream_t st, DevCtx ctx) {
    constexpr int bytes = smem_floats<D, R>() * 4;
    if (cudaError_t e = ensure_smem<tree_simt_kernel<D, F, R>>(bytes); e != cudaSuccess) return e;
    s.n_rt = tree::row_tiles(s.rows, 16 * R);
    // One block per SM until all that fit have three tiles each: the join pays for every partial (one
    // token of 32 heads of 128 over 8000: 30 us with 148 blocks, 39 with 296).
    const long long most = (long long)s.B * s.Hkv * s.n_rt * ((s.max_ctx + s.T + kKeys - 1) / kKeys);
    const int all = tree_ctas<D, R>(), sms = device_sm_count();
    const int n_cta = most >= 3 * all ? all : most < sms ? (int)most : sms;
    const tree::Partials part = tree::partials_at(ws, n_cta, slot_rows(s.rows));
    tree_simt_kernel<D, F, R><<<n_cta, kThreads, bytes, st>>>(
        static_cast<const float*>(q), pages, masks, static_cast<float*>(o), s, part,
        scale * 1.4426950408889634f, ctx);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    return launch_tree_join(DType::F32, part, o, s, slot_rows(s.rows), D, n_cta, st);
}

}  // namespace

size_t tree_simt_workspace(int rows, int d) { return tree::partial_bytes(tree_ctas(rows, d), slot_rows(rows), d); }

cudaError_t launch_packed_simt(const void* q, const void* k, const void* v, const int32_t* cu, void* o,
                               int B, int H, int Hkv, int total, int d, float scale, cudaStream_t st,
                               DevCtx ctx) {
    auto go = [&](auto dd) {
        constexpr int D = decltype(dd)::value;
        // R = 2 while all blocks of R = 4 run at once: the longest of them is then the time (2000 tokens,
        // 8 heads of 64: 233 against 281 us; 300 tokens: 25 against 33; 1000 tokens lose, 104 against 96).
        const long long blocks = ((long long)total / 64 + (B < total ? B : total)) * H;
        return blocks <= packed_blocks<D, 4>() * device_sm_count()
                   ? packed_simt<D, 2>(q, k, v, cu, o, B, H, Hkv, total, scale, st, ctx)
                   : packed_simt<D, 4>(q, k, v, cu, o, B, H, Hkv, total, scale, st, ctx);
    };
    return d == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

cudaError_t launch_tree_simt(KvFormat f, const void* q, const KvPages& pages, const uint64_t* masks, void* o,
                             const int32_t* ctx_len, int max_ctx, int B, int H, int Hkv, int T, int d,
                             float scale, void* ws, cudaStream_t st, DevCtx ctx) {
    const int rows = H / Hkv * T;
    const tree::Shape s{ctx_len, B, Hkv, H / Hkv, T, max_ctx, rows, 0, kKeys, kPad0};
    auto with_format = [&](auto dd, auto rr) {
        constexpr int D = decltype(dd)::value, R = decltype(rr)::value;
        if (f == KvFormat::Int8) return tree_simt<D, KvFormat::Int8, R>(q, pages, masks, o, s, ws, scale, st, ctx);
        if (f == KvFormat::E4M3) return tree_simt<D, KvFormat::E4M3, R>(q, pages, masks, o, s, ws, scale, st, ctx);
        return tree_simt<D, KvFormat::Same, R>(q, pages, masks, o, s, ws, scale, st, ctx);
    };
    auto go = [&](auto dd) {
        switch (rows_per_thread(rows)) {
            case 1: return with_format(dd, std::integral_constant<int, 1>{});
            case 2: return with_format(dd, std::integral_constant<int, 2>{});
            default: return with_format(dd, std::integral_constant<int, 4>{});
        }
    };
    return d == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace sala
