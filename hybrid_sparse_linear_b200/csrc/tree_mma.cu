// Attention of new tokens over a paged key/value cache for few query rows: at most 16 per KV head
// (one token of a group of 16 heads), bf16 queries, the cache in bf16 or 8-bit codes.
//
// With 16 rows the step is the read of the cache: 64 d operations per key against 2 (d + 4) bytes in
// 8 bits.  A 128-row tensor-core tile would be seven eighths empty, and its chain through shared
// memory and TMEM costs more than the work, so each warp takes whole pages on its own: K and V of a
// page land in the warp's own buffers by TMA (the next page's K is requested as soon as S is formed,
// its V after P V), the products are m16n8k16 tiles, and codes become fp16 fragments in registers.
// A page's K and V take 8, 16 or 32 KB (rows of 64, 128 or 256 bytes); twelve warps, six at 32 KB, keep up to
// 96, 192 and 192 KB per SM on their way.  Measured, 32 query heads of 128 over 2: one token over four int8
// caches of 790000 tokens together 85 to 90 us (4.8 TB/s; on the 128-row tiles 225), over one bf16 cache of
// 1000 10.5 to 11.1 us.  At 168 registers the instances for rows of 128 codes spill, 24 bytes for int8, 148
// for e4m3.
//
// Fragments.  The contraction over d may take its elements in any order as long as Q and K agree: a
// lane reads 16 bytes of a key's row and uses them for consecutive steps of four elements, and Q's
// fragments are laid out to match.  The keys of an 8-key tile are dealt to the fragment's columns in
// the order 0 4 1 5 2 6 3 7 where rows are 128 bytes, so that the lanes of a load phase fall into
// different banks under the 128-byte swizzle; P's columns meet V's rows in the same order.  V comes
// transposed (ldmatrix): of codes, two neighbouring columns at a time, split by byte.
//
// Codes are multiplied as fp16, which they are exactly and which takes two to three instructions a
// pair where bf16 takes five (the conversion is half of the kernel's instructions).  Q's rows are
// brought to it by a power of two that puts their largest value in [2^14, 2^15); what falls below fp16's
// smallest step then is 2^-39 of that value.  P has no such bound, as it carries the scales of V's
// rows: the weight of key j in O is 2^(y_j + log2 sv_j - M + 7) with a running maximum M of its own
// exponent, which is stale by at most 8, so that weights stay below 2^15 and vanish 2^-32 under the
// largest of the warp's keys; the weight in the row's sum is 2^(y_j - m) as ever, and O is brought to m at
// the item's end.  The accumulators hold 32 bits: in a column where the largest key's value is not small, what
// one product of 16 keys adds is lost from 2^-24 of the sum down, long before fp16's steps count; those
// show in columns where that value is 0 or nearly so.
//
// Hidden positions, infinities and NaN: as in the tensor-core kernel (tree_tc.cu).  The warps'
// accumulators are joined in shared memory at an item's end.
#include <type_traits>

#include "decode_common.cuh"
#include "kv_format.cuh"
#include "softmax_tile.cuh"
#include "tmap.cuh"
#include "tree_plan.cuh"

namespace sala {
namespace {

using namespace ptx;
using namespace smx;
using namespace dec;

constexpr int kRows = 16;
constexpr int kUpQ = 14;      // Q's largest value, and 2^kUpP the weight of a key at M, in fp16
constexpr float kUpP = 7.f;

template <int D, KvFormat F>
struct Layout {
    static constexpr bool kCodes = F != KvFormat::Same;
    static constexpr int kRowBytes = D * (kCodes ? 1 : 2);
    static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;  // of a row, per TMA box
    static constexpr int kBoxes = kRowBytes / kBoxBytes;
    static constexpr int kTile = kPage * kRowBytes;                      // K or V of a page
    static constexpr int kWarps = kRowBytes > 128 ? 6 : 12;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kStage = 2 * kTile;                             // a warp's K and V
    static constexpr int kOffScale = kWarps * kStage;                    // [warp][k, v, log2 v][64]
    static constexpr int kOffQ = kOffScale + (kCodes ? kWarps * 3 * kPage * 4 : 0);  // [step][lane], 16 bytes
    static constexpr int kOffNotes = kOffQ + (D / 16) * 512;
    static constexpr int kOffMl = kOffNotes + (kCodes ? 0 : 2 * D * 8);  // [warp][16] (maximum, sum)
    static constexpr int kOffBars = kOffMl + kWarps * kRows * 8;
    static constexpr int kBytes = kOffBars + kWarps * 2 * 8;
    static_assert(kRows * D * 4 <= kStage, "a warp's accumulator goes into its buffers");
};

// 16-byte piece c of row r of a tile whose boxes are swizzled.
template <class L>
__device__ __forceinline__ uint8_t* piece(uint8_t* tile, int r, int c) {
    if constexpr (L::kBoxBytes == 128)
        return tile + (c >> 3) * (kPage * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    else
        return tile + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
// Key of an 8-key tile in fragment column n.
template <class L>
__device__ __forceinline__ int key_of(int n) {
    return L::kBoxBytes == 128 ? (n & 1) * 4 + (n >> 1) : n;
}

template <int D, KvFormat F>
__global__ void __launch_bounds__(Layout<D, F>::kThreads, 1)
tree_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __nv_bfloat16* __restrict__ q, KvPages pages, const uint64_t* __restrict__ masks,
                __nv_bfloat16* __restrict__ out, tree::Shape s, tree::Partials part, bool by_item, float sl2,
                DevCtx ctx) {
    using L = Layout<D, F>;
    constexpr bool kCodes = L::kCodes;
    constexpr int kPer = kCodes ? 16 : 8;     // elements in 16 bytes
    constexpr int kPieces = D / kPer;         // per row
    constexpr int kSteps = D / 16;            // of the contraction over d
    extern __shared__ __align__(1024) uint8_t sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;    // fragment row (and row + 8), column pair
    uint8_t* K = sm + warp * L::kStage;
    uint8_t* V = K + L::kTile;
    float* ksc = reinterpret_cast<float*>(sm + L::kOffScale) + warp * 3 * kPage;
    float* vsc = ksc + kPage;
    float* vlg = vsc + kPage;
    unsigned long long* notes = reinterpret_cast<unsigned long long*>(sm + L::kOffNotes);
    float2* ml = reinterpret_cast<float2*>(sm + L::kOffMl);
    uint64_t* kbar = reinterpret_cast<uint64_t*>(sm + L::kOffBars) + warp * 2;
    uint64_t* vbar = kbar + 1;
    __shared__ tree::Cursor cur0;
    __shared__ int noted;

    cudaTriggerProgrammaticLaunchCompletion();  // the join may be set up; it waits for this grid's end
    if (lane == 0) {
        mbar_init(kbar, 1);
        mbar_init(vbar, 1);
        fence_mbar_init();
    }
    if (by_item) {
        if (tid == 0) {
            bool bad = false;
            cur0 = tree::item_at(s, blockIdx.x, &bad);
            if (bad) flag(ctx, kStatusBounds);
        }
    } else if (warp == 0) {
        bool bad = false;
        const long long w = tree::total_places(s, lane, &bad);
        if (bad && blockIdx.x == 0) flag(ctx, kStatusBounds);
        const long long x0 = tree::run_start(w, blockIdx.x, gridDim.x);
        const tree::Cursor c = tree::find_place(s, x0, tree::run_start(w, blockIdx.x + 1, gridDim.x) - x0, lane);
        if (lane == 0) cur0 = c;
    }
    __syncthreads();
    tree::Cursor c = cur0;
    uint32_t nk = 0, nv = 0;  // loads requested so far
    bool dead = false;        // a wait ran out: no more loads

    for (; c.left > 0; tree::next_item(s, c)) {
        const int n = tree::run_tiles(c), t0 = tree::first_tile(c), end = t0 + n;
        if (n == 0) continue;
        const int64_t row0 = ((int64_t)c.b * s.Hkv + c.g) * s.rows;
        // Q's fragments, on their way while the pages are found, and the rows' draft masks.
        uint64_t bits[2];
        uint32_t qa[kSteps][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = g + 8 * h;
            const bool real = r < s.rows;
            bits[h] = real ? tree::draft_bits(masks, c.b, r % s.T, s.T) : 0ull;
            const __nv_bfloat16* src = q + (row0 + r) * D + t * kPer;
#pragma unroll
            for (int st = 0; st < kSteps; ++st) {
                const uint2 u = real ? __ldg(reinterpret_cast<const uint2*>(
                                           src + (st / (kPer / 4)) * 4 * kPer + (st % (kPer / 4)) * 4))
                                     : make_uint2(0u, 0u);
                qa[st][h] = u.x;
                qa[st][2 + h] = u.y;
            }
        }
        // This warp takes the run's pages warp, warp + kWarps, ...; lane i knows the page of the next
        // 32 of them that is its own i-th.
        int ids = -1, ids_at = -32;
        auto page_at = [&](int i) {  // converged; -1: left out, or past the end
            if (i >= ids_at + 32) {
                ids_at = i;
                const int tl = t0 + warp + L::kWarps * (i + lane);
                ids = page_of(pages, c.b, tl);
                if (tl >= end) ids = -1;
                else if (ids < 0) flag(ctx, kStatusBounds);
            }
            return __shfl_sync(0xffffffffu, ids, i - ids_at);
        };
        auto load = [&](int id, bool is_k) {
            if (id < 0 || dead) return;
            if (lane == 0) {
                uint64_t* bar = is_k ? kbar : vbar;
                const int row = (id * s.Hkv + c.g) * kPage;
                mbar_arrive_expect_tx(bar, L::kTile + (kCodes ? kPage * 4 : 0));
                for (int x = 0; x < L::kBoxes; ++x)
                    tma_load_2d((is_k ? K : V) + x * kPage * L::kBoxBytes, is_k ? &tmK : &tmV, bar,
                                x * (L::kBoxBytes / (kCodes ? 1 : 2)), row);
                if constexpr (kCodes)
                    bulk_load_g2s(is_k ? ksc : vsc, (is_k ? pages.k_scale : pages.v_scale) + row, kPage * 4, bar);
            }
            if (is_k) ++nk;
            else ++nv;
        };
        const int n_my = (n - warp + L::kWarps - 1) / L::kWarps;  // may be <= 0
        int id = n_my > 0 ? page_at(0) : -1;
        load(id, true);
        load(id, false);

        [[maybe_unused]] float up[2];  // per row: takes Q's lift back
        uint4* qf = reinterpret_cast<uint4*>(sm + L::kOffQ) + lane;
        if constexpr (kCodes) {  // to fp16, the largest value in [2^kUpQ, 2^(kUpQ + 1))
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t m = 0u;
#pragma unroll
                for (int st = 0; st < kSteps; ++st)
                    m = __vmaxu2(m, __vmaxu2(qa[st][h] & 0x7fff7fffu, qa[st][2 + h] & 0x7fff7fffu));
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
                int ex = (int)(max(m & 0xffffu, m >> 16) >> 7);  // biased exponent
                if (ex == 255) ex = 127;                         // an infinity or a NaN stays what it is
                ex = max(ex, kUpQ + 1) - kUpQ;
                const float down = __uint_as_float((uint32_t)(254 - ex) << 23);
                up[h] = __uint_as_float((uint32_t)ex << 23);
                auto half2 = [&](uint32_t w) {
                    const __half2 v = __floats2half2_rn(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xffff0000u) * down);
                    return *reinterpret_cast<const uint32_t*>(&v);
                };
#pragma unroll
                for (int st = 0; st < kSteps; ++st) {
                    qa[st][h] = half2(qa[st][h]);
                    qa[st][2 + h] = half2(qa[st][2 + h]);
                }
            }
        }
#pragma unroll
        for (int st = 0; st < kSteps; ++st)  // every warp has them all; one puts them down
            if (st % L::kWarps == warp) qf[st * 32] = make_uint4(qa[st][0], qa[st][1], qa[st][2], qa[st][3]);
        if constexpr (!kCodes) {
            if (tid == 0) noted = 0;
            for (int e = tid; e < 2 * D; e += L::kThreads) notes[e] = 0ull;
        }
        __syncthreads();
        RowState st[2];
        float top_v[2] = {-INFINITY, -INFINITY};  // M
        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;

        for (int i = 0; i < n_my; ++i) {
            const int next = i + 1 < n_my ? page_at(i + 1) : -1;
            const int k0 = (t0 + warp + L::kWarps * i) * kPage;
            if (id < 0) {
                id = next;
                load(id, true);
                load(id, false);
                continue;
            }
            if (!dead && !__all_sync(0xffffffffu, wait_long(kbar, (nk - 1) & 1, ctx))) dead = true;
            if (dead) break;
            float sc[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
#pragma unroll
            for (int p = 0; p < kPieces / 4; ++p) {
                constexpr int kN = kPer / 4;  // steps that 16 bytes make
                uint32_t qa[kN][4];
#pragma unroll
                for (int x = 0; x < kN; ++x) {
                    const uint4 u = qf[(kN * p + x) * 32];
                    qa[x][0] = u.x;
                    qa[x][1] = u.y;
                    qa[x][2] = u.z;
                    qa[x][3] = u.w;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint4 u = ld16(piece<L>(K, 8 * j + key_of<L>(g), 4 * p + t));
                    if constexpr (kCodes) {
                        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint2 b = codes_to_f16<F>(w[x]);
                            mma16816_f16(sc[j], qa[x], {b.x, b.y});
                        }
                    } else {
                        mma16816(sc[j], qa[0], {u.x, u.y});
                        mma16816(sc[j], qa[1], {u.z, u.w});
                    }
                }
            }
            if constexpr (kCodes) {
                // From S to log2 units, before anything is hidden.  The factors are joined first, the key's scale
                // with what takes Q's lift back: alone the scale would bring S, which holds the lift, out of
                // fp32's range where keys are large and queries small, and the other could round to zero.
                // Together they leave the range only where q . k does.
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float a = ksc[8 * j + key_of<L>(2 * t)], b = ksc[8 * j + key_of<L>(2 * t + 1)];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        sc[j][2 * h] *= a * up[h] * sl2;
                        sc[j][2 * h + 1] *= b * up[h] * sl2;
                    }
                }
            }
            __syncwarp();
            load(next, true);
            // A page with drafts or with slots behind the last token: what a row does not see becomes -inf, whose
            // weight is zero, so that one code serves every page.
            const bool tail = k0 + kPage > c.ctx;
            if (tail) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int dr = k0 + 8 * j + key_of<L>(2 * t + x) - c.ctx;  // draft number
                            if (dr >= 0 && (dr >= 64 || !((bits[h] >> dr) & 1ull))) sc[j][2 * h + x] = -INFINITY;
                        }
            }
            // nb, nv_: added to the exponents of l's and of O's weights; alpha: O's factor
            [[maybe_unused]] float alpha[2], nb[2], nv_[2] = {0.f, 0.f};
            if constexpr (!kCodes) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 8; ++j) mx = max3n(mx, sc[j][2 * h], sc[j][2 * h + 1]);
                    mx = max2n(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = max2n(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    alpha[h] = st[h].raise(mx * sl2);
                    nb[h] = st[h].shift();
                }
            }
            if (!__all_sync(0xffffffffu, wait_long(vbar, (nv - 1) & 1, ctx))) {
                dead = true;
                break;
            }
            if constexpr (kCodes) {
                if (!tail) {
                    vlg[lane] = lg2(vsc[lane]);
                    vlg[lane + 32] = lg2(vsc[lane + 32]);
                } else {
                    // A scale that is no number must reach the rows that see its draft and no other.
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int r = lane + 32 * x, dr = k0 + r - c.ctx;
                        const float v = lg2(vsc[r]);
                        const bool odd = dr >= 0 && !(fabsf(v) < INFINITY) && vsc[r] != 0.f;
                        vlg[r] = odd ? 0.f : v;
                        const unsigned who = __ballot_sync(0xffffffffu, odd && dr < s.T);
                        const int d0 = k0 + 32 * x - c.ctx;  // draft number of lane 0's row
                        const uint64_t drafts = d0 >= 0 ? (d0 < 64 ? (uint64_t)who << d0 : 0ull) : who >> min(-d0, 31);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (bits[h] & drafts) st[h].l = __uint_as_float(0x7fffffffu);
                    }
                }
                __syncwarp();
                float mx[2] = {-INFINITY, -INFINITY}, mv[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float va = vlg[8 * j + key_of<L>(2 * t)], vb = vlg[8 * j + key_of<L>(2 * t + 1)];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float y0 = sc[j][2 * h], y1 = sc[j][2 * h + 1];
                        mx[h] = max3n(mx[h], y0, y1);
                        mv[h] = max3n(mv[h], y0 + va, y1 + vb);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) {
                        mx[h] = max2n(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], o));
                        mv[h] = max2n(mv[h], __shfl_xor_sync(0xffffffffu, mv[h], o));
                    }
                    (void)st[h].raise(mx[h]);
                    nb[h] = st[h].shift();
                    alpha[h] = 1.f;
                    if (mv[h] > top_v[h] + kGrow) {
                        if (top_v[h] != -INFINITY) alpha[h] = ex2(top_v[h] - mv[h]);
                        top_v[h] = mv[h];
                    }
                    if (!(mv[h] <= 3.402823466e38f)) st[h].l = __uint_as_float(0x7fffffffu);
                    nv_[h] = top_v[h] == -INFINITY ? 0.f : kUpP - top_v[h];
                }
            }
            if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int e = 0; e < D / 8; ++e) {
                    o[e][0] *= alpha[0];
                    o[e][1] *= alpha[0];
                    o[e][2] *= alpha[1];
                    o[e][3] *= alpha[1];
                }
            }
            if constexpr (!kCodes) {
                if (tail) {  // V's rows that not every row sees: see tree_tc.cu
                    constexpr int kC = D / 8;
#pragma unroll 4
                    for (int e = max(c.ctx - k0, 0) * kC + lane; e < kPage * kC; e += 32) {
                        const int r = e / kC, p = e % kC, dr = k0 + r - c.ctx;
                        uint4* u = reinterpret_cast<uint4*>(piece<L>(V, r, p));
                        if (dr >= s.T) {
                            *u = make_uint4(0u, 0u, 0u, 0u);
                        } else if (dr >= 0 && any_nonfinite8(*u)) {
                            uint16_t* w = reinterpret_cast<uint16_t*>(u);
                            for (int x = 0; x < 8; ++x) {
                                if ((w[x] & 0x7f80u) != 0x7f80u) continue;
                                const bool nan = (w[x] & 0x7fu) != 0u, neg = (w[x] & 0x8000u) != 0u;
                                if (nan || !neg) atomicOr(notes + p * 8 + x, 1ull << dr);
                                if (nan || neg) atomicOr(notes + D + p * 8 + x, 1ull << dr);
                                w[x] = 0;
                            }
                            noted = 1;
                        }
                    }
                    __syncwarp();
                }
            }
            if (F == KvFormat::E4M3 && tail) {
                // Slots behind the last token may hold anything, e4m3's NaN code too, which zero weights would
                // not hide: they become zero, and so does that code in a draft's row (no write makes it).
#pragma unroll 4
                for (int e = max(c.ctx - k0, 0) * kPieces + lane; e < kPage * kPieces; e += 32) {
                    const int r = e / kPieces, dr = k0 + r - c.ctx;
                    uint4* u = reinterpret_cast<uint4*>(piece<L>(V, r, e % kPieces));
                    auto clean = [&](uint32_t w) { return dr >= s.T ? 0u : w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); };
                    *u = make_uint4(clean(u->x), clean(u->y), clean(u->z), clean(u->w));
                }
                __syncwarp();
            }
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                uint32_t pa[4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int j = 2 * jj + y;
                    [[maybe_unused]] float va, vb;
                    if constexpr (kCodes) {
                        va = vlg[8 * j + key_of<L>(2 * t)];
                        vb = vlg[8 * j + key_of<L>(2 * t + 1)];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float x0 = sc[j][2 * h], x1 = sc[j][2 * h + 1];
                        if constexpr (kCodes) {
                            st[h].l += ex2(x0 + nb[h]) + ex2(x1 + nb[h]);
                            const __half2 w = __floats2half2_rn(ex2(x0 + (va + nv_[h])), ex2(x1 + (vb + nv_[h])));
                            pa[2 * y + h] = *reinterpret_cast<const uint32_t*>(&w);
                        } else {
                            const float p0 = ex2(fmaf(x0, sl2, nb[h])), p1 = ex2(fmaf(x1, sl2, nb[h]));
                            st[h].l += p0 + p1;
                            pa[2 * y + h] = pack_bf16x2(p0, p1);
                        }
                    }
                }
                // lanes 8 m .. 8 m + 7 address matrix m: 8 keys of tile 2 jj + (m & 1), piece p + (m >> 1)
                const int vr = 8 * (2 * jj + ((lane >> 3) & 1)) + key_of<L>(lane & 7);
#pragma unroll
                for (int p = 0; p < kPieces; p += 2) {
                    uint32_t u[4];
                    ldsm_x4_t(u, piece<L>(V, vr, p + (lane >> 4)));
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t a = u[2 * y], b = u[2 * y + 1];
                        if constexpr (kCodes) {
                            const uint2 fa = crossed_to_f16<F>(a), fb = crossed_to_f16<F>(b);
                            mma16816_f16(o[2 * (p + y)], pa, {fa.x, fb.x});
                            mma16816_f16(o[2 * (p + y) + 1], pa, {fa.y, fb.y});
                        } else {
                            mma16816(o[p + y], pa, {a, b});
                        }
                    }
                }
            }
            if (F != KvFormat::Int8 && tail) fence_proxy_async_smem();  // the next copy comes behind the zeros
            __syncwarp();
            id = next;
            load(id, false);
        }

        // The warp's partial into its own buffers (every load of the item has landed and is used).
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float l = st[h].l;
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            if (t == 0) ml[warp * kRows + g + 8 * h] = make_float2(st[h].m, l);
            float* dst = reinterpret_cast<float*>(K) + (g + 8 * h) * D;
            if constexpr (kCodes) {  // O from M to m
                const float f = top_v[h] == -INFINITY ? 0.f : ex2(top_v[h] - kUpP - (st[h].m == -INFINITY ? 0.f : st[h].m));
#pragma unroll
                for (int e = 0; e < D / 8; ++e) {
                    o[e][2 * h] *= f;
                    o[e][2 * h + 1] *= f;
                }
            }
            if (n_my > 0 && !dead) {
                if constexpr (kCodes) {  // tiles 2 p and 2 p + 1: columns 16 p + 4 t + 0, 2 and 1, 3
#pragma unroll
                    for (int p = 0; p < kPieces; ++p)
                        *reinterpret_cast<float4*>(dst + 16 * p + 4 * t) =
                            make_float4(o[2 * p][2 * h], o[2 * p + 1][2 * h], o[2 * p][2 * h + 1], o[2 * p + 1][2 * h + 1]);
                } else {
#pragma unroll
                    for (int p = 0; p < D / 8; ++p)
                        *reinterpret_cast<float2*>(dst + 8 * p + 2 * t) = make_float2(o[p][2 * h], o[p][2 * h + 1]);
                }
            }
        }
        const bool lost = __syncthreads_or(dead);
        if (lost) break;
        const bool whole = n == c.n_tiles;
        const size_t slot = ((size_t)blockIdx.x * 2 + (t0 > 0 ? 0 : 1)) * s.rows;
        for (int e = tid; e < s.rows * (D / 4); e += L::kThreads) {
            const int r = e / (D / 4), col = (e % (D / 4)) * 4;
            float top = -INFINITY;
            float2 p[L::kWarps];
#pragma unroll
            for (int w = 0; w < L::kWarps; ++w) {
                p[w] = ml[w * kRows + r];
                top = fmaxf(top, p[w].x);
            }
            float l = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < L::kWarps; ++w) {
                const bool saw = p[w].x != -INFINITY || p[w].y != 0.f;  // else the buffer holds no row
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                if (saw) y = *reinterpret_cast<const float4*>(sm + w * L::kStage + (r * D + col) * 4);
                const float wt = saw ? ex2(p[w].x - top) : 0.f;
                l += wt * p[w].y;
                x.x += wt * y.x;
                x.y += wt * y.y;
                x.z += wt * y.z;
                x.w += wt * y.w;
            }
            if constexpr (!kCodes) {
                if (noted) {  // rows that attend to a draft with an infinity or a NaN in V get it back
                    const uint64_t b = tree::draft_bits(masks, c.b, r % s.T, s.T);
                    float* f = &x.x;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (notes[col + j] & b) f[j] += INFINITY;
                        if (notes[D + col + j] & b) f[j] -= INFINITY;
                    }
                }
            }
            if (whole) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                *reinterpret_cast<uint2*>(out + (row0 + r) * D + col) =
                    make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
            } else {
                if (col == 0) part.ml[slot + r] = make_float2(top, l);
                *reinterpret_cast<float4*>(part.o + (slot + r) * D + col) = x;
            }
        }
        fence_proxy_async_smem();  // the next item's copies come behind what was written here
        __syncthreads();
    }
    // Copies that a wind-down left on their way land before the block exits.
    if (dead && lane == 0) {
        if (nk > 0) (void)mbar_wait(kbar, (nk - 1) & 1, ctx);
        if (nv > 0) (void)mbar_wait(vbar, (nv - 1) & 1, ctx);
    }
}

// Short contexts: a block per item, with no partials to join.  Few items leave SMs idle, which pays up
// to 16 pages (bf16 pages, one token, in us: 2 items of 16 pages 10.9 against 14.1 with equal runs and their
// join, of 24 pages 13.3 against 12.6), more items up to 24 (32 items of 24 pages 13.9 against 16.7, of 32
// pages even).  Where items nearly fill the SMs it pays up to 64 (128 items of 64 pages: bf16 47 against 55,
// int8 37 against 49; of 1 to 64 pages 32 and 33 against 38 and 35; 200 int8 items of 64 pages lose, 70
// against 66), and is even at 128.
int item_pages(int items, int sms) { return 4 * items >= 3 * sms ? 64 : 8 * items >= sms ? 24 : 16; }
// Beginning an item (a round of loads that nothing overlaps, the warps' join) costs about as much as
// this many pages, or some more.  In us, one token of 32 heads of 128 over 2: 40 int8 contexts of up to 16000
// tokens 52 (4 pages: 60, 24: 50), 200 of up to 8000 109 (119, 105), 16 bf16 contexts of up to 9000 19.1
// (22.0, 19.1).
constexpr int kPad = 12;

template <int D, KvFormat F>
cudaError_t tree_mma(const void* q, const KvPages& pages, const uint64_t* masks, void* o, tree::Shape s,
                     void* ws, float scale, cudaStream_t st, DevCtx ctx) {
    using L = Layout<D, F>;
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return cudaErrorNotSupported;
    CUtensorMap tmK{}, tmV{};
    auto map = [&](CUtensorMap* m, const void* base) {
        cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)pages.n_pages * s.Hkv * kPage};
        cuuint64_t strides[1] = {(cuuint64_t)L::kRowBytes};
        cuuint32_t box[2] = {(cuuint32_t)(L::kBoxBytes / (L::kCodes ? 1 : 2)), (cuuint32_t)kPage};
        cuuint32_t one[2] = {1, 1};
        return fn(m, L::kCodes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  L::kBoxBytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (pages.n_pages > 0 && (!map(&tmK, pages.k) || !map(&tmV, pages.v))) return cudaErrorInvalidValue;
    if (cudaError_t e = ensure_smem<tree_mma_kernel<D, F>>(L::kBytes); e != cudaSuccess) return e;
    const int tiles = (s.max_ctx + s.T + kPage - 1) / kPage, items = s.B * s.Hkv, sms = device_sm_count();
    const bool by_item = tiles <= item_pages(items, sms);
    const int n_cta = by_item ? items : tree::run_ctas(s, tiles, 2, sms);
    const tree::Partials part = tree::partials_at(ws, by_item ? 0 : n_cta, s.rows);
    tree_mma_kernel<D, F><<<n_cta, L::kThreads, L::kBytes, st>>>(
        tmK, tmV, static_cast<const __nv_bfloat16*>(q), pages, masks, static_cast<__nv_bfloat16*>(o), s,
        part, by_item, scale * 1.4426950408889634f, ctx);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    if (by_item) return cudaSuccess;
    return launch_tree_join(DType::BF16, part, o, s, s.rows, D, n_cta, st);
}

}  // namespace

bool tree_mma_supported(int rows) { return rows <= kRows; }

cudaError_t launch_tree_mma(KvFormat f, const void* q, const KvPages& pages, const uint64_t* masks, void* o,
                            const int32_t* ctx_len, int max_ctx, int B, int H, int Hkv, int T, int d,
                            float scale, void* ws, cudaStream_t st, DevCtx ctx) {
    const tree::Shape s{ctx_len, B, Hkv, H / Hkv, T, max_ctx, H / Hkv * T, 1, kPage, kPad};
    auto go = [&](auto dd) {
        constexpr int D = decltype(dd)::value;
        if (f == KvFormat::Int8) return tree_mma<D, KvFormat::Int8>(q, pages, masks, o, s, ws, scale, st, ctx);
        if (f == KvFormat::E4M3) return tree_mma<D, KvFormat::E4M3>(q, pages, masks, o, s, ws, scale, st, ctx);
        return tree_mma<D, KvFormat::Same>(q, pages, masks, o, s, ws, scale, st, ctx);
    };
    return d == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace sala
