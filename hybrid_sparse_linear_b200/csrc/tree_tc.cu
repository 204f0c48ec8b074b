// Attention of new (drafted) tokens over a paged key/value cache on the 5th-generation tensor cores:
// bf16 queries; the cache in bf16 or as 8-bit codes with one scale per row.
//
// The G * T query rows of a KV head are its M: rows (head g, token t) are contiguous in q.  Above 128
// rows (wide) an item takes 256, two tiles A and B that share every K and V tile.  Up to 128 rows
// (narrow) there is one tile of rows, and A takes the even, B the odd key tiles of the CTA's run, each
// with its own ring and accumulator, joined at the end.  Either way two chains of 64-key steps run
// beside each other, each with two S buffers, so that the next S does not wait for this one's PV.
// Work is divided by key tiles (tree_plan.cuh), so a single sequence uses every SM.
//
// Bound: HBM for few rows (a key and value row are read once per 256 query rows: 4 G T d flops
// against 4 d bytes, 2 (d + 4) in 8 bits), the tensor pipe from about T = 16 at G = 16.  Measured, 32 query
// heads of 128 over 2: 64 drafts over 131072 tokens, bf16, 140 us (980 TFLOP/s; 163 in a run of a second under
// the power cap, at 1.7 GHz); 8 drafts over 16 e4m3 caches of 94000 tokens together 45 us (in the wide form 50),
// where no unit is full -- issue slots 46 %, ALU 37 %, tensor pipe 14 % -- and a tile waits for the chain codes,
// bf16 tile, S, softmax, PV.  The 8-bit instances start with 96 registers and spill 80 to 88 bytes.
//
// 8-bit caches.  Codes are at most 8 bits wide, so each is a bf16 number exactly; eight warps turn
// the raw bytes of a tile into bf16 tiles in shared memory and the matrix products run as for bf16.
// The scales never touch the tiles: a key's scale multiplies its column of S, a value's scale its
// column of P (before P's one rounding to bf16, after the row sum), both in 32 bits.
//
// Hidden positions (drafts a row does not attend to, slots behind the last token, pages the table
// does not hold) are left out by selection.  In a bf16 cache a hidden row of V could still turn a
// probability of zero into NaN, so one warp looks through the V tiles that hold such rows: rows
// nobody sees become zero; an infinity or NaN in a draft's row becomes zero and is noted per column,
// and the epilogue gives it to the rows that attend to that draft.
//
// Roles: warps 0-3 softmax and epilogue of tile A, 4-7 of B; 8 walks the items and loads (TMA for
// bf16 tiles, bulk copies for codes and scales); 9 and 10 issue the MMAs of A and B; 11 looks through
// V (bf16); 12-19 (8-bit caches only) convert.  Every wait is bounded.
#include <type_traits>

#include "kv_format.cuh"
#include "softmax_tile.cuh"
#include "tmap.cuh"
#include "tree_plan.cuh"

namespace sala {
namespace {

using namespace ptx;
using namespace smx;

constexpr int kK = 64;              // keys per tile: a page
constexpr int kConvThreads = 256;
// Short contexts: a CTA per item, without partials and their join.  Up to 8 tiles it pays for any number of
// items, up to 16 (wide: 32) where they are three eighths of the SMs, up to 32 (wide: 64) at three quarters.
// In us, against equal runs, bf16 and 2 KV heads of 16 query heads: two tokens, 8 sequences of 8 pages 13.3
// against 16.3, of 16 pages 19.0 against 17.7; 32 sequences of 16 pages 19.8 against 22.2, of 32 pages 30
// against 26; 60 of 32 pages 32 against 41, of 1 to 32 pages 30 and 30, of 64 pages 54 against 60, of 1 to 64
// pages 53 against 44; 64 drafts (wide), 16 sequences of 2 pages 17 against 41, 8 of 32 pages 48 against
// 55, of 64 pages 79 against 69, 16 of 64 pages 80 against 118, 50 of 64 pages 236 against 287.
inline int item_tiles(bool wide, long long items, int sms) {
    return 8 * items < 3 * sms ? 8 : (4 * items < 3 * sms ? 16 : 32) << (wide ? 1 : 0);
}
// Beginning an item (Q, the first tiles' chain, the epilogue) costs at least four tiles.  In us, 16 contexts of up
// to 9000 tokens: 8 drafts, e4m3 34 (1 tile: 46, 8: 33.5); 64 drafts, bf16 128 (195, 102); 32 drafts, int8 75.5 (88,
// 75); 4 drafts over 40 bf16 contexts of up to 16000 80 (83, 75).
constexpr int kPad = 4;

template <int D, KvFormat F, bool kWide>
struct Layout {
    static constexpr bool kCodes = F != KvFormat::Same;
    static constexpr int kThreads = kCodes ? 640 : 384;
    static constexpr int kRegsSoft = kCodes ? 144 : 216, kRegsRest = kCodes ? 64 : 72;
    static constexpr int kRows = kWide ? 256 : 128;          // query rows per item
    static constexpr int kQBox = 128 * 128;                  // [128 rows x 64 columns] bf16, swizzled
    static constexpr int kQTile = (D / 64) * kQBox;
    static constexpr int kBox = kK * 128;                    // [kK rows x 64 columns]
    static constexpr int kTile = (D / 64) * kBox;            // a K or V tile
    static constexpr int kRaw = kK * D;                      // the codes of one
    // K and V tiles: one ring that both tiles of rows use, or one for each.
    static constexpr int kRing = (kWide ? (kCodes ? 6 : 8) : (kCodes ? 4 : 5)) * (128 / D);
    static constexpr int kSlots = kWide ? kRing : 2 * kRing;
    static constexpr int kRawSlots = kCodes ? 5 * (128 / D) : 0;
    // The tiles first (each 1024-byte aligned), then the small parts.
    static constexpr int kOffRing = (kWide ? 2 : 1) * kQTile;
    static constexpr int kOffRaw = kOffRing + kSlots * kTile;
    static constexpr int kOffRawScale = kOffRaw + kRawSlots * kRaw;
    static constexpr int kOffScale = kOffRawScale + kRawSlots * kK * 4;
    static constexpr int kOffNotes = kOffScale + (kCodes ? kSlots * kK * 4 : 0);
    static constexpr int kNoteBytes = kCodes ? 0 : 2 * D * 8;    // sign x column, a bit per draft
    static constexpr int kOffMerge = kOffNotes + kNoteBytes;     // narrow: both tiles' (maximum, sum) per row
    static constexpr int kOffStage = kOffMerge + (kWide ? 0 : 2 * 128 * 8);  // per softmax warp: 32 rows of 64 bytes
    static constexpr int kOffBars = kOffStage + 8 * 2048;
};

// An item's part in this CTA's run.
struct Item {
    int b, g, rt, ctx;
    int tile, n;      // key tiles [tile, tile + n) (n 0: no more)
    int whole;         // the run has all of them
};
// A V tile to look through.
struct Look {
    int slot;     // where it is
    int k0, ctx;  // its first key; the sequence's context length
    int have;     // whether the table holds its page
    int it, last;  // the item, and whether this is its last tile with drafts
};

template <class L>
struct Bars {
    uint64_t full[L::kSlots], empty[L::kSlots];
    uint64_t raw_full[L::kRawSlots + 1], raw_empty[L::kRawSlots + 1];
    uint64_t q_full[2], q_empty;
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // per tile and S buffer
    uint64_t v_landed[2], look_free[2];  // alternating over the looks
    uint64_t v_seen[2];                  // per item parity: its drafts' V is looked through
    uint64_t both_done, merged;          // narrow: both tiles' accumulators are complete; have been read
    uint64_t item_full[2], item_empty[2];
    uint64_t fin[2];
    Item item[2];
    Look look[2];
    int have[2][16];                     // as Look::have, per ring and key tile (a ring holds at most 10)
    int raw_have[L::kRawSlots + 1];
    int noted_it;                        // the item that the notes belong to
    uint32_t tmem_base;
    int abort;
};

template <int D, KvFormat F, bool kWide>
__global__ void __launch_bounds__(Layout<D, F, kWide>::kThreads, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
               const __grid_constant__ CUtensorMap tmV, KvPages pages, const uint64_t* __restrict__ masks,
               __nv_bfloat16* __restrict__ out, tree::Shape s, tree::Partials part, bool by_item, float sl2,
               DevCtx ctx) {
    using L = Layout<D, F, kWide>;
    static_assert(L::kOffBars + sizeof(Bars<L>) <= 227 * 1024, "shared memory");
    constexpr bool kCodes = L::kCodes;
    constexpr uint32_t kRing = L::kRing, kSlots = L::kSlots, kRawSlots = kCodes ? L::kRawSlots : 1;
    constexpr uint32_t kColO = 0, kColS = 256;
    extern __shared__ __align__(1024) uint8_t sm[];  // all of the block's shared memory
    Bars<L>& bars = *reinterpret_cast<Bars<L>*>(sm + L::kOffBars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &bars.abort;
    unsigned long long* notes = reinterpret_cast<unsigned long long*>(sm + L::kOffNotes);
    float2* merge = reinterpret_cast<float2*>(sm + L::kOffMerge);

    cudaTriggerProgrammaticLaunchCompletion();  // the join may be set up; it waits for this grid's end
    if (warp == 9) {
        tmem_alloc(&bars.tmem_base, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (uint32_t i = 0; i < kSlots; ++i) {
            mbar_init(&bars.full[i], kCodes ? kConvThreads / 32 : 1);
            // Handed back by the commit of the tile's MMAs that read it and, where it has scales, by the
            // softmax warps; by both tiles of rows where they share it.
            mbar_init(&bars.empty[i], (kWide ? 2 : 1) * (kCodes ? 5 : 1));
        }
        for (uint32_t i = 0; i < kRawSlots; ++i) {
            mbar_init(&bars.raw_full[i], 1);
            mbar_init(&bars.raw_empty[i], kConvThreads / 32);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars.q_full[x], 1);
            for (int j = 0; j < 2; ++j) {
                mbar_init(&bars.s_full[x][j], 1);
                mbar_init(&bars.p_full[x][j], 4);
                mbar_init(&bars.pv_done[x][j], 1);
            }
            mbar_init(&bars.v_landed[x], 1);
            mbar_init(&bars.look_free[x], 1);
            mbar_init(&bars.v_seen[x], 1);
            mbar_init(&bars.item_full[x], 1);
            mbar_init(&bars.item_empty[x], 10 + (kCodes ? 8 : 0));  // softmax, issuers, converters
            mbar_init(&bars.fin[x], 1);
        }
        mbar_init(&bars.q_empty, 2);
        mbar_init(&bars.both_done, 8);
        mbar_init(&bars.merged, 8);
        bars.noted_it = -1;
        bars.abort = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;

    // Entry e of a ring (K and V of its key tiles in turn) lives in its slot e % kRing, as that slot's
    // use number e / kRing.  Who waits for an entry has waited for all before it in that ring, so no
    // parity wait runs two uses ahead, and none falls two behind: an entry is not overwritten before
    // every tile that uses it has handed it back.
    auto ring_of = [](int x) { return kWide ? 0u : (uint32_t)x; };
    auto slot_of = [&](int x, uint32_t e) { return ring_of(x) * kRing + e % kRing; };
    auto use_of = [](uint32_t e) { return (e / kRing) & 1u; };
    auto slot_ptr = [&](uint32_t slot) { return sm + L::kOffRing + slot * L::kTile; };
    auto raw_of = [](uint32_t e) { return e % kRawSlots; };
    auto raw_use = [](uint32_t e) { return (e / kRawSlots) & 1u; };
    auto take_item = [&](int it, Item& m) -> bool {
        if (!wait_warp(&bars.item_full[it & 1], (it >> 1) & 1, ctx, abort)) return false;
        m = bars.item[it & 1];
        return m.n > 0;
    };
    auto leave_item = [&](int it) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.item_empty[it & 1]);
    };
    // Key tiles of tile x of an item with n of them: all, or every other one.
    auto my_tiles = [](int n, int x) { return kWide ? n : (n + 1 - x) / 2; };
    auto nth_tile = [](int k, int x) { return kWide ? k : 2 * k + x; };

    if (warp >= 8) {
        set_regs_down<L::kRegsRest>();
        if (warp == 8) {
            // ------------------------------------------------------------ items and loads
            bool bad = false;
            tree::Cursor c;
            if (by_item) {
                c = tree::item_at(s, blockIdx.x, &bad);
                if (bad) flag(ctx, kStatusBounds);
            } else {
                const long long w = tree::total_places(s, lane, &bad);
                if (bad && blockIdx.x == 0) flag(ctx, kStatusBounds);
                const long long x0 = tree::run_start(w, blockIdx.x, gridDim.x);
                c = tree::find_place(s, x0, tree::run_start(w, blockIdx.x + 1, gridDim.x) - x0, lane);
            }
            uint32_t rc[2] = {0, 0}, rr = 0, kq = 0, looks = 0;  // entries, raw tiles, Q tiles, looks
            uint32_t via = 0;  // slots whose last load went to v_landed
            bool ok = true;
            for (int it = 0; ok; ++it) {
                while (c.left > 0 && tree::run_tiles(c) == 0) tree::next_item(s, c);
                const int n = c.left > 0 ? tree::run_tiles(c) : 0, t0 = tree::first_tile(c);
                if (it >= 2 && !wait_warp(&bars.item_empty[it & 1], ((it - 2) >> 1) & 1, ctx, abort)) break;
                if (lane == 0) {
                    bars.item[it & 1] = Item{c.b, c.g, c.rt, c.ctx, t0, n, n == c.n_tiles};
                    mbar_arrive(&bars.item_full[it & 1]);
                }
                if (n == 0) break;
                if (kq >= 1 && !wait_warp(&bars.q_empty, (kq - 1) & 1, ctx, abort)) break;
                if (lane == 0) {
                    const int y = (c.b * s.Hkv + c.g) * s.rows + c.rt * L::kRows;
                    for (int x = 0; x < (kWide ? 2 : 1); ++x) {
                        mbar_arrive_expect_tx(&bars.q_full[x], L::kQTile);
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_2d(sm + x * L::kQTile + h * L::kQBox, &tmQ, &bars.q_full[x], 64 * h, y + 128 * x);
                    }
                }
                ++kq;
                int ids = -1;
                for (int i = 0; ok && i < n; ++i) {
                    const int t = t0 + i;
                    if ((i & 31) == 0) ids = page_of(pages, c.b, t + lane);
                    const int id = __shfl_sync(0xffffffffu, ids, i & 31);
                    const bool have = id >= 0;
                    if (!have && lane == 0) flag(ctx, kStatusBounds);  // left out
                    const int row = (id * s.Hkv + c.g) * kPage;
                    const bool drafts = (t + 1) * kK > c.ctx;  // keys that some row does not see
                    for (int j = 0; ok && j < 2; ++j) {  // K, V
                        if constexpr (kCodes) {
                            const uint32_t q = raw_of(rr);
                            if (rr >= kRawSlots && !(ok = wait_warp(&bars.raw_empty[q], raw_use(rr - kRawSlots), ctx, abort)))
                                break;
                            ++rr;
                            if (lane == 0) {
                                bars.raw_have[q] = have;
                                mbar_arrive_expect_tx(&bars.raw_full[q], have ? L::kRaw + kK * 4 : 0);
                                if (have) {
                                    bulk_load_g2s(sm + L::kOffRaw + q * L::kRaw,
                                                  static_cast<const uint8_t*>(j ? pages.v : pages.k) + (int64_t)row * D,
                                                  L::kRaw, &bars.raw_full[q]);
                                    bulk_load_g2s(sm + L::kOffRawScale + q * kK * 4,
                                                  (j ? pages.v_scale : pages.k_scale) + row, kK * 4, &bars.raw_full[q]);
                                }
                            }
                        } else {
                            const bool odd = !kWide && (i & 1);
                            const uint32_t e = odd ? rc[1] : rc[0], q = slot_of(odd, e);
                            if (e >= kRing && !(ok = wait_warp(&bars.empty[q], use_of(e - kRing), ctx, abort)))
                                break;
                            const bool look = j == 1 && (drafts || !have);
                            if (look && looks >= 2 &&
                                !(ok = wait_warp(&bars.look_free[looks & 1], ((looks - 2) >> 1) & 1, ctx, abort)))
                                break;
                            if (lane == 0) {
                                uint64_t* fb = look ? &bars.v_landed[looks & 1] : &bars.full[q];
                                if (j == 0) bars.have[odd][(e >> 1) & 15] = have;
                                if (look) bars.look[looks & 1] = Look{(int)q, t * kK, c.ctx, have, it, drafts && i == n - 1};
                                mbar_arrive_expect_tx(fb, have ? L::kTile : 0);
                                for (int p = 0; have && p < D / 64; ++p)
                                    tma_load_2d(slot_ptr(q) + p * L::kBox, j ? &tmV : &tmK, fb, 64 * p, row);
                            }
                            via = (via & ~(1u << q)) | ((look ? 1u : 0u) << q);
                            looks += look ? 1 : 0;
                            if (odd) ++rc[1];
                            else ++rc[0];
                        }
                    }
                }
                tree::next_item(s, c);
            }
            if constexpr (!kCodes) {  // no more looks: an entry that says so
                if (ok && looks >= 2) ok = wait_warp(&bars.look_free[looks & 1], ((looks - 2) >> 1) & 1, ctx, abort);
                if (ok && lane == 0) {
                    bars.look[looks & 1].it = -1;
                    mbar_arrive(&bars.v_landed[looks & 1]);
                }
            }
            if (lane == 0) {  // drain: every copy this warp started has landed before the block exits
                if (kq > 0)
                    for (int x = 0; x < (kWide ? 2 : 1); ++x) (void)mbar_wait(&bars.q_full[x], (kq - 1) & 1, ctx);
                if constexpr (kCodes) {
                    for (uint32_t e = rr > kRawSlots ? rr - kRawSlots : 0; e < rr; ++e)
                        (void)mbar_wait(&bars.raw_full[raw_of(e)], raw_use(e), ctx);
                } else {
                    for (uint32_t l = looks > 2 ? looks - 2 : 0; l < looks; ++l)
                        // (a barrier that went on to the closing entry has this use behind it)
                        if (!ok || l != looks - 2) (void)mbar_wait(&bars.v_landed[l & 1], (l >> 1) & 1, ctx);
                    for (int x = 0; x < (kWide ? 1 : 2); ++x)
                        for (uint32_t e = rc[x] > kRing ? rc[x] - kRing : 0; e < rc[x]; ++e)
                            if (!((via >> slot_of(x, e)) & 1u))
                                (void)mbar_wait(&bars.full[slot_of(x, e)], use_of(e), ctx);
                }
            }
        } else if (warp < 11) {
            // ------------------------------------------------------------ MMA issuers
            // Order per tile: PV of a key tile, then S of the one two further, which lies over the P
            // that this PV read; MMAs of one thread run in order.  The whole warp runs the loop and one
            // elected lane issues.
            const int x = warp - 9;
            auto wait_w = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, ctx, abort); };
            const uint32_t dO = tmem + kColO + x * 128, dS = tmem + kColS + x * 128;
            const uint64_t dhi = (uint64_t)sdesc_sw128_hi(1024) << 32;
            const uint64_t q_d = dhi | sdesc_sw128_lo(smem_u32(sm + (kWide ? x : 0) * L::kQTile), 16);
            const uint64_t k_d0 = dhi | sdesc_sw128_lo(smem_u32(sm + L::kOffRing), 16);
            const uint64_t v_d0 = dhi | sdesc_sw128_lo(smem_u32(sm + L::kOffRing), L::kBox);
            constexpr uint32_t idS = idesc_bf16_f32(128, kK, false, false);
            constexpr uint32_t idPV = idesc_bf16_f32(128, D, false, true);
            uint32_t rc = 0, a = 0;  // ring entries, key tiles of the items before
            bool ok = true;
            Item m;
            for (int it = 0; ok && take_item(it, m); ++it) {
                const int nx = my_tiles(m.n, x);
                auto issue_s = [&](int k) -> bool {
                    const uint32_t e = rc + 2 * k, q = slot_of(x, e), j = (a + k) & 1;
                    if (!wait_w(&bars.full[q], use_of(e))) return false;
                    tc_fence_after();
                    const uint64_t k_d = k_d0 + q * (L::kTile >> 4);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_ss_elect(dS + j * 64, q_d + (((ks >> 2) * L::kQBox + (ks & 3) * 32) >> 4),
                                     k_d + (((ks >> 2) * L::kBox + (ks & 3) * 32) >> 4), idS, ks > 0 ? 1u : 0u);
                    mma_commit_elect(&bars.s_full[x][j]);
                    mma_commit_elect(&bars.empty[q]);
                    return true;
                };
                ok = wait_w(&bars.q_full[kWide ? x : 0], it & 1);
                for (int k = 0; ok && k < 2 && k < nx; ++k) ok = issue_s(k);
                for (int k = 0; ok && k < nx; ++k) {
                    const uint32_t e = rc + 2 * k + 1, q = slot_of(x, e), j = (a + k) & 1;
                    ok = wait_w(&bars.p_full[x][j], ((a + k) / 2) & 1) && wait_w(&bars.full[q], use_of(e));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v_d = v_d0 + q * (L::kTile >> 4);
#pragma unroll
                    for (int ks = 0; ks < kK / 16; ++ks)
                        mma_ts_elect(dO, dS + j * 64 + ks * 8, v_d + ((ks * 16 * 128) >> 4), idPV,
                                     (k > 0 || ks > 0) ? 1u : 0u);
                    mma_commit_elect(&bars.pv_done[x][j]);
                    mma_commit_elect(&bars.empty[q]);
                    if (k + 2 < nx) ok = issue_s(k + 2);
                }
                rc += 2 * nx;
                a += nx;
                if (ok) mma_commit_elect(&bars.q_empty);  // every S that reads this item's Q is done
                leave_item(it);
            }
            mma_commit_elect(&bars.fin[x]);
            (void)mbar_wait(&bars.fin[x], 0, ctx);
            __syncwarp();
        } else if (warp == 11) {
            // ------------------------------------------------------------ V rows not every row sees
            if constexpr (!kCodes) {
                for (uint32_t l = 0;; ++l) {
                    if (!wait_warp(&bars.v_landed[l & 1], (l >> 1) & 1, ctx, abort)) break;
                    const Look v = bars.look[l & 1];
                    if (v.it < 0) break;
                    constexpr int kC = D / 8;  // 16-byte pieces per row
                    uint8_t* tile = slot_ptr(v.slot);
                    const int keys = v.ctx + s.T;
                    for (int c0 = 0; c0 < kK * kC; c0 += 32) {
                        const int r = (c0 + lane) / kC, c = (c0 + lane) % kC, j = v.k0 + r - v.ctx;
                        uint4* p = reinterpret_cast<uint4*>(tile + (c >> 3) * L::kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                        bool bad = false;
                        if (v.k0 + r >= keys || !v.have) *p = make_uint4(0u, 0u, 0u, 0u);
                        else if (j >= 0) bad = any_nonfinite8(*p);
                        unsigned todo = __ballot_sync(0xffffffffu, bad);
                        if (todo == 0u) continue;
                        if (*reinterpret_cast<volatile int*>(&bars.noted_it) != v.it) {
                            // The notes may still be read for the item before.
                            if (v.it >= 1) (void)wait_warp(&bars.item_empty[(v.it - 1) & 1], ((v.it - 1) >> 1) & 1, ctx, abort);
                            for (int e = lane; e < 2 * D; e += 32) notes[e] = 0ull;
                            __syncwarp();
                            if (lane == 0) *reinterpret_cast<volatile int*>(&bars.noted_it) = v.it;
                            __syncwarp();
                        }
                        for (; todo; todo &= todo - 1) {  // one lane after another: they share columns
                            if (lane == __ffs((int)todo) - 1) {
                                uint16_t* e = reinterpret_cast<uint16_t*>(p);
                                for (int q = 0; q < 8; ++q) {
                                    if ((e[q] & 0x7f80u) != 0x7f80u) continue;
                                    const bool nan = (e[q] & 0x7fu) != 0u, neg = (e[q] & 0x8000u) != 0u;
                                    if (nan || !neg) notes[c * 8 + q] |= 1ull << j;
                                    if (nan || neg) notes[D + c * 8 + q] |= 1ull << j;
                                    e[q] = 0;
                                }
                            }
                            __syncwarp();
                        }
                    }
                    fence_proxy_async_smem();  // the MMA reads what was just written
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bars.full[v.slot]);
                        if (v.last) mbar_arrive(&bars.v_seen[v.it & 1]);
                        mbar_arrive(&bars.look_free[l & 1]);
                    }
                    __syncwarp();
                }
            }
        } else {
            // ------------------------------------------------------------ codes to bf16 tiles
            if constexpr (kCodes) {
                const int ct = tid - 12 * 32;
                uint32_t rc[2] = {0, 0}, rr = 0;
                bool ok = true;
                Item m;
                for (int it = 0; ok && take_item(it, m); ++it) {
                    for (int i = 0; ok && i < 2 * m.n; ++i, ++rr) {
                        const bool odd = !kWide && ((i >> 1) & 1);
                        const uint32_t e2 = odd ? rc[1]++ : rc[0]++, q = slot_of(odd, e2);
                        ok = wait_warp(&bars.raw_full[raw_of(rr)], raw_use(rr), ctx, abort);
                        if (ok && e2 >= kRing) ok = wait_warp(&bars.empty[q], use_of(e2 - kRing), ctx, abort);
                        if (!ok) break;
                        const uint8_t* raw = sm + L::kOffRaw + raw_of(rr) * L::kRaw;
                        uint8_t* tile = slot_ptr(q);
                        // A lane takes 16 codes, four lanes 64 columns of a row, neighbouring rows the
                        // other 64: eight lanes then read and (through the swizzle) write all 32 banks.
                        constexpr int kN = kK * (D / 16) / kConvThreads;  // pieces of 16 codes per thread
                        constexpr int kB = kN < 4 ? kN : 4;
#pragma unroll
                        for (int b0 = 0; b0 < kN; b0 += kB) {
                            uint4 u[kB];  // read before the first write, which the compiler keeps in order
#pragma unroll
                            for (int b = 0; b < kB; ++b) {
                                const int e = ct + (b0 + b) * kConvThreads, r = (e >> 2) % kK;
                                const int box = D == 64 ? 0 : (r + e / (kK * 4)) & 1;
                                u[b] = *reinterpret_cast<const uint4*>(raw + r * D + box * 64 + (e & 3) * 16);
                            }
#pragma unroll
                            for (int b = 0; b < kB; ++b) {
                                const int e = ct + (b0 + b) * kConvThreads, r = (e >> 2) % kK, c = e & 3;
                                const int box = D == 64 ? 0 : (r + e / (kK * 4)) & 1;
                                uint8_t* row = tile + box * L::kBox + r * 128;
                                const uint2 a0 = codes_to_bf16<F>(u[b].x), a1 = codes_to_bf16<F>(u[b].y);
                                const uint2 a2 = codes_to_bf16<F>(u[b].z), a3 = codes_to_bf16<F>(u[b].w);
                                *reinterpret_cast<uint4*>(row + (((2 * c) ^ (r & 7)) << 4)) =
                                    make_uint4(a0.x, a0.y, a1.x, a1.y);
                                *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ (r & 7)) << 4)) =
                                    make_uint4(a2.x, a2.y, a3.x, a3.y);
                            }
                        }
                        if (ct < kK)
                            reinterpret_cast<float*>(sm + L::kOffScale)[q * kK + ct] =
                                reinterpret_cast<const float*>(sm + L::kOffRawScale)[raw_of(rr) * kK + ct] *
                                ((i & 1) ? 1.f : sl2);  // K's with the softmax scale
                        if (ct == 0 && !(i & 1)) bars.have[odd][(e2 >> 1) & 15] = bars.raw_have[raw_of(rr)];
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&bars.full[q]);
                            mbar_arrive(&bars.raw_empty[raw_of(rr)]);
                        }
                    }
                    leave_item(it);
                }
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax + epilogue
        set_regs_up<L::kRegsSoft>();
        const int x = warp >> 2;
        const int r = tid & 127;
        const uint32_t lane_base = tmem_lane_base(warp);
        const uint32_t colO = tmem + lane_base + kColO + x * 128;
        const uint32_t colS = tmem + lane_base + kColS + x * 128;
        uint32_t rc = 0, a = 0;  // ring entries, key tiles of the items before
        uint32_t nseen[2] = {0, 0};
        bool ok = true;
        auto give = [&](uint32_t slot) {  // this warp has read the scales there
            if (kCodes && lane == 0) mbar_arrive(&bars.empty[slot]);
        };
        Item m;
        for (int it = 0; ok && take_item(it, m); ++it) {
            const int nx = my_tiles(m.n, x);
            const int row = m.rt * L::kRows + (kWide ? r + 128 * x : r);  // of the group
            const bool real = row < s.rows;
            const uint64_t bits = real ? tree::draft_bits(masks, m.b, row % s.T, s.T) : 0ull;
            const bool any_real = __any_sync(0xffffffffu, real);  // else the warp only passes stages on
            RowState st;
            for (int k = 0; k < nx; ++k) {
                const int i = nth_tile(k, x), k0 = (m.tile + i) * kK;
                const uint32_t e = rc + 2 * k, qk = slot_of(x, e), qv = slot_of(x, e + 1), j = (a + k) & 1;
                const uint32_t col = colS + j * 64;
                ok = wait_warp(&bars.s_full[x][j], ((a + k) / 2) & 1, ctx, abort);
                if (kCodes && ok) ok = wait_warp(&bars.full[qk], use_of(e), ctx, abort);  // (done: for its scales)
                if (!ok) break;
                tc_fence_after();
                float alpha = 1.f;
                if (any_real) {
                    uint32_t sr[kK];  // logits; with codes in log2 units already
                    const float sl = kCodes ? 1.f : sl2;
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < kK / 32; ++c) tmem_ld32(col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(sr + 32 * c));
                    const bool have = bars.have[ring_of(x)][(e >> 1) & 15] != 0;
                    tmem_ld_wait();
                    if constexpr (kCodes) {
                        const float* ks = reinterpret_cast<const float*>(sm + L::kOffScale) + qk * kK;
#pragma unroll
                        for (int c = 0; c < kK; c += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(ks + c);
                            float* z = reinterpret_cast<float*>(sr) + c;
                            mul2(z[0], z[1], f.x, f.y);
                            mul2(z[2], z[3], f.z, f.w);
                        }
                        __syncwarp();
                        give(qk);
                    }
                    const float* vs = reinterpret_cast<const float*>(sm + L::kOffScale) + qv * kK;
                    if (k0 + kK <= m.ctx && have) {
                        float mx = max32(sr);
#pragma unroll
                        for (int c = 1; c < kK / 32; ++c) mx = max2n(mx, max32(sr + 32 * c));
                        alpha = st.raise(mx * sl);
                        const float nb = st.shift();
                        if (kCodes) ok = wait_warp(&bars.full[qv], use_of(e + 1), ctx, abort);  // V's scales
#pragma unroll
                        for (int c = 0; c < kK / 32; ++c) {
                            uint32_t pk[16];
                            exp32<false, kCodes>(sr + 32 * c, sl, nb, 0u, vs + 32 * c, acc, pk);
                            tmem_st16(col + 16 * c, pk);
                        }
                    } else {
                        uint32_t seen[kK / 32];
                        float mx = -INFINITY;
#pragma unroll
                        for (int c = 0; c < kK / 32; ++c) {
                            const int d0 = k0 + 32 * c - m.ctx;  // draft number of the chunk's first key
                            const uint32_t drafts = d0 >= 64 ? 0u : d0 >= 0 ? (uint32_t)(bits >> d0)
                                                  : d0 > -32 ? (uint32_t)(bits << -d0) : 0u;
                            seen[c] = have ? (bits_to(-d0 - 1) | drafts) : 0u;
                            mx = max2n(mx, max32_masked(sr + 32 * c, seen[c]));
                        }
                        alpha = st.raise(mx * sl);
                        const float nb = st.shift();
                        if (kCodes) ok = wait_warp(&bars.full[qv], use_of(e + 1), ctx, abort);
#pragma unroll
                        for (int c = 0; c < kK / 32; ++c) {
                            uint32_t pk[16];
                            exp32<true, kCodes>(sr + 32 * c, sl, nb, seen[c], vs + 32 * c, acc, pk);
                            tmem_st16(col + 16 * c, pk);
                        }
                    }
                    st.l += (acc[0] + acc[1]) + (acc[2] + acc[3]);
                } else {
                    give(qk);
                    if (kCodes) ok = wait_warp(&bars.full[qv], use_of(e + 1), ctx, abort);
                }
                __syncwarp();
                give(qv);
                if (!ok) break;
                // Narrow: both tiles read both accumulators at an item's end.  P, which lets the issuer
                // start on this one, comes only after that.
                if (!kWide && k == 0 && it > 0) ok = wait_warp(&bars.merged, (it - 1) & 1, ctx, abort);
                if (ok && k > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    const uint32_t b = a + k - 1;  // the PV before has to be done with O
                    ok = wait_warp(&bars.pv_done[x][b & 1], (b / 2) & 1, ctx, abort);
                    if (ok) {
                        tc_fence_after();
                        scale_row<D>(colO, alpha);
                    }
                }
                if (!ok) break;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[x][j]);
            }
            if (!ok) break;
            // The drafts' V of this item is looked through (its notes can be read).
            bool noted = false;
            if constexpr (!kCodes) {
                if ((m.tile + m.n) * kK > m.ctx) {
                    ok = wait_warp(&bars.v_seen[it & 1], nseen[it & 1]++ & 1, ctx, abort);
                    if (!ok) break;
                    noted = *reinterpret_cast<volatile int*>(&bars.noted_it) == it;
                }
            }
            rc += 2 * nx;
            a += nx;
            if (nx > 0) {
                ok = wait_warp(&bars.pv_done[x][(a - 1) & 1], ((a - 1) / 2) & 1, ctx, abort);
                if (!ok) break;
                tc_fence_after();
            }
            // Narrow: the two tiles' accumulators belong to the same rows; A writes the first half of the
            // columns of their join, B the second.
            float top = st.m, l = st.l, w_a = 1.f, w_b = 0.f;
            if constexpr (!kWide) {
                // (Nobody is still reading the item before: P of this one came behind it, or comes next.)
                if (nx == 0 && it > 0) ok = wait_warp(&bars.merged, (it - 1) & 1, ctx, abort);
                if (!ok) break;
                merge[x * 128 + r] = make_float2(st.m, st.l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.both_done);
                ok = wait_warp(&bars.both_done, it & 1, ctx, abort);
                if (!ok) break;
                tc_fence_after();
                const float2 o = merge[(1 - x) * 128 + r];
                const float m_a = x ? o.x : st.m, m_b = x ? st.m : o.x;
                top = fmaxf(m_a, m_b);
                w_a = m_a == -INFINITY ? 0.f : ex2(m_a - top);
                w_b = m_b == -INFINITY ? 0.f : ex2(m_b - top);
                l = x ? o.y * w_a + st.l * w_b : st.l * w_a + o.y * w_b;
            }
            const bool two = !kWide && m.n > 1;
            const float inv = !m.whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
            const int64_t orow = ((int64_t)m.b * s.Hkv + m.g) * s.rows;  // of the group's row 0
            const int rt = kWide ? L::kRows : s.rows;  // rows a partial slot holds
            const size_t slot = ((size_t)blockIdx.x * 2 + (m.tile > 0 ? 0 : 1)) * rt;
            const int r0 = row - lane, s0 = kWide ? r0 - m.rt * L::kRows : r0;  // the warp's first row; in its slot
            if (real && !m.whole && (kWide || x == 0)) part.ml[slot + s0 + lane] = make_float2(top, l);
            if (any_real) {
                const uint32_t colA = tmem + lane_base + kColO + (kWide ? x * 128 : 0), colB = colA + 128;
                const int c_first = kWide || x == 0 ? 0 : D / 2, c_end = kWide || x == 1 ? D : D / 2;
                uint8_t* stage = sm + L::kOffStage + warp * 2048;
                // 16 columns at a time, 64 bytes per row and pass (of bf16 every second time) through
                // shared memory: four lanes then store a row's 64 bytes, whole sectors.
#pragma unroll 1
                for (int c0 = c_first; c0 < c_end; c0 += 16) {
                    uint32_t o[16];
                    tmem_ld16(colA + c0, o);
                    if (two) {
                        uint32_t q[16];
                        tmem_ld16(colB + c0, q);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * w_a + __uint_as_float(q[e]) * w_b);
                    } else {
                        tmem_ld_wait();
                    }
                    if (noted) {  // rows that attend to a draft with an infinity or a NaN in V get it back
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float y = __uint_as_float(o[e]);
                            if (notes[c0 + e] & bits) y += INFINITY;
                            if (notes[D + c0 + e] & bits) y -= INFINITY;
                            o[e] = __float_as_uint(y);
                        }
                    }
                    auto spot = [&](int rr, int p) { return reinterpret_cast<uint4*>(stage + rr * 64 + ((p ^ ((rr >> 1) & 3)) << 4)); };
                    if (m.whole) {
                        uint32_t w[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            w[j] = pack_bf16x2(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                        const int p = (c0 & 16) >> 3;
                        *spot(lane, p) = make_uint4(w[0], w[1], w[2], w[3]);
                        *spot(lane, p + 1) = make_uint4(w[4], w[5], w[6], w[7]);
                        if (p == 0) continue;
                    } else {
#pragma unroll
                        for (int p = 0; p < 4; ++p) *spot(lane, p) = make_uint4(o[4 * p], o[4 * p + 1], o[4 * p + 2], o[4 * p + 3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int rr = 8 * p + (lane >> 2);
                        const uint4 v = *spot(rr, lane & 3);
                        if (r0 + rr < s.rows) {
                            if (m.whole)
                                *reinterpret_cast<uint4*>(out + (orow + r0 + rr) * D + (c0 - 16) + 8 * (lane & 3)) = v;
                            else
                                *reinterpret_cast<uint4*>(part.o + (slot + s0 + rr) * D + c0 + 4 * (lane & 3)) = v;
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (!kWide && lane == 0) mbar_arrive(&bars.merged);
            leave_item(it);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, KvFormat F, bool kWide>
cudaError_t tree_tc(const void* q, const KvPages& pages, const uint64_t* masks, void* o, tree::Shape s,
                    void* ws, float scale, cudaStream_t st, DevCtx ctx) {
    using L = Layout<D, F, kWide>;
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return cudaErrorNotSupported;
    auto map = [&](CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows) {
        return make_tmap_bf16_2d(m, base, D, rows, D, 64, box_rows);
    };
    CUtensorMap tmQ, tmK{}, tmV{};
    if (cudaError_t e = map(&tmQ, q, (uint64_t)s.B * s.Hkv * s.rows, 128); e != cudaSuccess) return e;
    if (F == KvFormat::Same && pages.n_pages > 0) {
        const uint64_t rows = (uint64_t)pages.n_pages * s.Hkv * kPage;
        if (cudaError_t e = map(&tmK, pages.k, rows, kPage); e != cudaSuccess) return e;
        if (cudaError_t e = map(&tmV, pages.v, rows, kPage); e != cudaSuccess) return e;
    }
    constexpr int bytes = L::kOffBars + (int)sizeof(Bars<L>);
    if (cudaError_t e = ensure_smem<tree_tc_kernel<D, F, kWide>>(bytes); e != cudaSuccess) return e;
    s.n_rt = kWide ? tree::row_tiles(s.rows, L::kRows) : 1;
    s.kt = kK;
    s.pad = kPad;
    const int tiles = (s.max_ctx + s.T + kK - 1) / kK;
    const long long items = (long long)s.B * s.Hkv * s.n_rt;  // below 2^31, as the query rows are
    const int sms = device_sm_count();
    const bool by_item = tiles <= item_tiles(kWide, items, sms);
    const int n_cta = by_item ? (int)items : tree::run_ctas(s, tiles, 1, sms);
    const int rt = kWide ? L::kRows : s.rows;
    const tree::Partials part = tree::partials_at(ws, n_cta, rt);
    tree_tc_kernel<D, F, kWide><<<n_cta, L::kThreads, bytes, st>>>(
        tmQ, tmK, tmV, pages, masks, static_cast<__nv_bfloat16*>(o), s, part,
        by_item, scale * 1.4426950408889634f, ctx);
    if (cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
    if (by_item) return cudaSuccess;
    return launch_tree_join(DType::BF16, part, o, s, rt, D, n_cta, st);
}

}  // namespace

size_t tree_tc_workspace(int rows, int d) {
    return tree::partial_bytes(device_sm_count(), rows > 128 ? 256 : rows, d);
}

cudaError_t launch_tree_tc(KvFormat f, const void* q, const KvPages& pages, const uint64_t* masks, void* o,
                           const int32_t* ctx_len, int max_ctx, int B, int H, int Hkv, int T, int d,
                           float scale, void* ws, cudaStream_t st, DevCtx ctx) {
    const tree::Shape s{ctx_len, B, Hkv, H / Hkv, T, max_ctx, H / Hkv * T, 0, 0, 0};
    auto go = [&](auto dd, auto ff) {
        constexpr int D = decltype(dd)::value;
        constexpr KvFormat F = decltype(ff)::value;
        return s.rows > 128 ? tree_tc<D, F, true>(q, pages, masks, o, s, ws, scale, st, ctx)
                            : tree_tc<D, F, false>(q, pages, masks, o, s, ws, scale, st, ctx);
    };
    auto with_format = [&](auto dd) {
        if (f == KvFormat::Int8) return go(dd, std::integral_constant<KvFormat, KvFormat::Int8>{});
        if (f == KvFormat::E4M3) return go(dd, std::integral_constant<KvFormat, KvFormat::E4M3>{});
        return go(dd, std::integral_constant<KvFormat, KvFormat::Same>{});
    };
    return d == 64 ? with_format(std::integral_constant<int, 64>{})
                   : with_format(std::integral_constant<int, 128>{});
}

}  // namespace sala
