// Causal softmax attention over packed prompts on the 5th-generation tensor cores (bf16).
//
// Work unit: two tiles A and B of 128 query rows that share one KV head.  A tile packs TG query
// heads of the head's group (the largest power of two dividing the group size, at most 16) by
// TQ = 128 / TG consecutive tokens, so with 16 heads per KV head a unit is 16 tokens and its
// causal edge wastes at most 15 keys per row.  A unit walks its sequence's keys in tiles of 64; K and
// V of a tile are loaded once for both.
//
// Per key tile and query tile X:  S_X = Q_X K^T (M128 N64),  P_X = online softmax (softmax_tile.cuh),
// O_X += P_X V (A = P_X from TMEM over S_X's columns).  TMEM: O_A, O_B (128 columns each) and two S
// buffers of 64 columns per tile: the S of the next key tile is formed while the softmax works on this
// one, so a tile's chain is its softmax alone, and the two tiles' chains run beside each other.  One
// S of 128 keys per tile instead would feed the tensor core better (an N = 64 step reads 6 KB of
// shared memory in the 32 cycles of its math, 48 at 128 B per cycle) but leaves S -> softmax -> PV in
// line: per 128 keys it took 3900 cycles of which the tensor core worked 2048 (1008 TFLOP/s at 32768
// tokens; two threads per row in that form, which have to meet for the row's maximum, 814).
//
// This form takes 8.0 ms there (1100 TFLOP/s), and 270 to 307 us for 16 prompts of 0 to 4096 tokens.
//
// Only the last key tile(s) hold keys that some row must not see.  There S and PV stop at the last
// 16-key step a row sees, rows mask by their own position, and, since a probability of zero still
// turns an infinity or NaN of V into NaN, one warp first looks through the V rows that not every
// row sees, replaces such values by zero and notes per column the first key that held one; the
// epilogue gives them back to the rows behind that key.
//
// Roles (384 threads, persistent, one CTA per SM): warps 0-3 softmax and epilogue of tile A, 4-7 of
// tile B (thread = row); warp 8 issues the TMA loads; warps 9 and 10 issue the MMAs of tiles A and B;
// warp 11 finds the units, two ahead, and looks through V.  Completions: the issuer commits once per round,
// after PV(k) and S(k + 2), so the commit of round k + 2 says that both are done; two more rounds
// without an S close a unit.  Those two have no P, by which the softmax tells the issuer that it has seen
// a round, so units of even and odd number have barriers of their own: a unit that begins cannot turn
// those on which a late softmax warp still waits for the end of the one before, and the unit after it,
// which uses them again, begins when every warp has left that one (one set for all units: a warp that is
// late by the next unit's first S waits into the time limit).  The softmax hands K and V stages back as it sees
// the commits.  Every wait is bounded; a timeout sets the status word and all roles wind down.
#include <climits>

#include "kv_format.cuh"
#include "softmax_tile.cuh"
#include "tmap.cuh"

namespace sala {
namespace {

using namespace ptx;
using namespace smx;

constexpr int kThreads = 384;
constexpr int kK = 64;   // keys per tile
constexpr int kWarps = kThreads / 32;

template <int D>
struct Layout {
    static constexpr int kQBox = 128 * 128;           // [128 rows x 64 columns] bf16, 128-byte swizzle
    static constexpr int kQTile = (D / 64) * kQBox;
    static constexpr int kBox = kK * 128;             // [kK rows x 64 columns]
    static constexpr int kTile = (D / 64) * kBox;     // a K or V tile
    static constexpr int kSlots = 9;                  // ring of K and V tiles
    static constexpr int kOffRing = 2 * kQTile;
    static constexpr int kOffStage = kOffRing + kSlots * kTile;  // per softmax warp: 32 rows x 32 columns
    static constexpr int kOffNotes = kOffStage + 8 * 2048;
    static constexpr int kNoteBytes = 2 * 2 * D * 2;  // unit parity x sign x column, uint16
    static constexpr int kBytes = kOffNotes + kNoteBytes + 1024;  // + alignment of the base
};

struct Unit {
    int start, len, first;  // the sequence's rows; the unit's first token inside it (len 0: no more)
    int hg;                 // group of TG query heads
};

template <int kSlots>
struct Bars {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2][2][2];  // per unit parity and tile, alternating over the unit's rounds
    uint64_t p_full[2][2];     // per tile, alternating over the rounds with P
    uint64_t v_landed[2][4];  // V tiles to look through, per unit parity (at most four a unit)
    uint64_t v_seen[2];       // per unit parity: warp 11 is through with the unit
    uint64_t unit_full[2], unit_empty[2];
    uint64_t fin[2];
    Unit unit[2];
    int noted[2];  // whether the unit's notes hold anything
    uint32_t tmem_base;
    int abort;
};

constexpr uint16_t kNoKey = 0xffff;

// Key tiles of tile x (0 when it has no row), and the keys of its last one rounded to 16.
__device__ __forceinline__ int key_tiles(const Unit& u, int x, int tq, int* last_keys) {
    const int t0 = u.first + x * tq;
    if (t0 >= u.len) {
        *last_keys = 0;
        return 0;
    }
    const int last = min(t0 + tq, u.len) - 1;  // last token, the last key its rows see
    *last_keys = ((last % kK) / 16 + 1) * 16;
    return last / kK + 1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
packed_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const int32_t* __restrict__ cu,
                 __nv_bfloat16* __restrict__ out, int B, int H, int Hkv, int total, int tg, float sl2,
                 DevCtx ctx) {
    using L = Layout<D>;
    constexpr int kSlots = L::kSlots;
    constexpr uint32_t kColO = 0, kColS = 256;
    extern __shared__ uint8_t smraw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smraw) + 1023) & ~uintptr_t(1023));
    __shared__ Bars<kSlots> bars;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &bars.abort;
    const int tq = 128 / tg, ut = 2 * tq, n_hg = H / tg;
    uint16_t* notes = reinterpret_cast<uint16_t*>(sm + L::kOffNotes);

    if (warp == 9) {
        tmem_alloc(&bars.tmem_base, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&bars.full[s], 1);
            mbar_init(&bars.empty[s], 2);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bars.q_full[x], 1);
            mbar_init(&bars.q_empty[x], 1);
            for (int j = 0; j < 2; ++j) {
                for (int i = 0; i < 2; ++i) mbar_init(&bars.s_full[i][x][j], 1);
                mbar_init(&bars.p_full[x][j], 4);
            }
            mbar_init(&bars.unit_full[x], 1);
            mbar_init(&bars.unit_empty[x], kWarps);
            mbar_init(&bars.fin[x], 1);
            bars.noted[x] = 0;
        }
        for (int j = 0; j < 2; ++j) {
            for (int i = 0; i < 4; ++i) mbar_init(&bars.v_landed[j][i], 1);
            mbar_init(&bars.v_seen[j], 1);
        }
        bars.abort = 0;
        fence_mbar_init();
    }
    for (int e = tid; e < 4 * D; e += kThreads) notes[e] = kNoKey;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars.tmem_base;

    // Ring entry e lives in slot e % kSlots and is that slot's use number e / kSlots.
    auto slot_of = [](uint32_t e) { return e % kSlots; };
    auto use_of = [](uint32_t e) { return (e / kSlots) & 1u; };
    auto slot_ptr = [&](uint32_t e) { return sm + L::kOffRing + slot_of(e) * L::kTile; };
    // Unit number it of this CTA, once the finder has it.
    auto take_unit = [&](int it, Unit& u) -> bool {
        if (!wait_warp(&bars.unit_full[it & 1], (it >> 1) & 1, ctx, abort)) return false;
        u = bars.unit[it & 1];
        return u.len > 0;
    };
    auto leave_unit = [&](int it) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.unit_empty[it & 1]);
    };

    if (warp >= 8) {
        set_regs_down<72>();
        if (warp == 8) {
            // ------------------------------------------------------------ loads
            uint32_t rc = 0, kq[2] = {0, 0};
            uint32_t nl[2][4] = {};  // uses of v_landed
            uint32_t via = 0;        // slots whose last load went to v_landed
            Unit u;
            for (int it = 0; take_unit(it, u); ++it) {
                int lk;
                const int nA = key_tiles(u, 0, tq, &lk), nB = key_tiles(u, 1, tq, &lk);
                const int n = max(nA, nB);
                int stop = 0;
                if (lane == 0) {
                    const int kvh = u.hg * tg / (H / Hkv);
                    auto load_q = [&](int x) {
                        if ((x ? nB : nA) == 0) return;
                        if (kq[x] >= 1 && !wait_or_abort(&bars.q_empty[x], (kq[x] - 1) & 1, ctx, abort)) {
                            stop = 1;
                            return;
                        }
                        mbar_arrive_expect_tx(&bars.q_full[x], L::kQTile);
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(sm + x * L::kQTile + h * L::kQBox, &tmQ, &bars.q_full[x], 64 * h,
                                        u.start + u.first + x * tq, u.hg * tg);
                        ++kq[x];
                    };
                    load_q(0);
                    for (int e = 0; e < 2 * n && !stop; ++e, ++rc) {
                        if (rc >= kSlots &&
                            !wait_or_abort(&bars.empty[slot_of(rc)], use_of(rc - kSlots), ctx, abort)) {
                            stop = 1;
                            break;
                        }
                        // A V tile that warp 11 looks through lands there; the warp then passes it on.
                        const int look = (e & 1) ? (e >> 1) - u.first / kK : -1;
                        uint64_t* fb = look >= 0 ? &bars.v_landed[it & 1][look] : &bars.full[slot_of(rc)];
                        if (look >= 0) ++nl[it & 1][look];
                        via = (via & ~(1u << slot_of(rc))) | ((look >= 0 ? 1u : 0u) << slot_of(rc));
                        mbar_arrive_expect_tx(fb, L::kTile);
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_3d(slot_ptr(rc) + h * L::kBox, (e & 1) ? &tmV : &tmK, fb, 64 * h,
                                        u.start + (e >> 1) * kK, kvh);
                        if (e == 0) load_q(1);
                    }
                }
                leave_unit(it);
                if (__shfl_sync(0xffffffffu, stop, 0)) break;
            }
            if (lane == 0) {  // drain: every copy this warp started has landed before the block exits
                for (int x = 0; x < 2; ++x)
                    if (kq[x] > 0) (void)mbar_wait(&bars.q_full[x], (kq[x] - 1) & 1, ctx);
                for (int j = 0; j < 8; ++j)
                    if (nl[j >> 2][j & 3] > 0)
                        (void)mbar_wait(&bars.v_landed[j >> 2][j & 3], (nl[j >> 2][j & 3] - 1) & 1, ctx);
                for (uint32_t e = rc > kSlots ? rc - kSlots : 0; e < rc; ++e)
                    if (!((via >> slot_of(e)) & 1u)) (void)mbar_wait(&bars.full[slot_of(e)], use_of(e), ctx);
            }
        } else if (warp < 11) {
            // ------------------------------------------------------------ MMA issuers
            // The whole warp runs the loop and one elected lane issues.  S of round k + 2 lies over the P
            // that PV of round k reads: MMAs of one thread run in order.
            const int x = warp - 9;
            auto wait_w = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, ctx, abort); };
            const uint32_t dO = tmem + kColO + x * 128, dS = tmem + kColS + x * 128;
            const uint64_t dhi = (uint64_t)sdesc_sw128_hi(1024) << 32;
            const uint64_t q_d = dhi | sdesc_sw128_lo(smem_u32(sm + x * L::kQTile), 16);
            const uint64_t k_d0 = dhi | sdesc_sw128_lo(smem_u32(sm + L::kOffRing), 16);
            const uint64_t v_d0 = dhi | sdesc_sw128_lo(smem_u32(sm + L::kOffRing), L::kBox);
            constexpr uint32_t idPV = idesc_bf16_f32(128, D, false, true);
            // Entries, Q tiles, rounds (of units of this one's parity; sr_next: of the other), rounds with P,
            // before the unit.
            uint32_t rc = 0, kq = 0, sr = 0, sr_next = 0, pr = 0;
            bool ok = true;
            Unit u;
            for (int it = 0; ok && take_unit(it, u); ++it) {
                int lkA, lkB;
                const int nA = key_tiles(u, 0, tq, &lkA), nB = key_tiles(u, 1, tq, &lkB);
                const int n = max(nA, nB), nx = x ? nB : nA, lk = x ? lkB : lkA;
                auto issue_s = [&](int b) -> bool {  // round b; without an S past the last key tile
                    const uint32_t j = (sr + b) & 1;
                    if (b < nx) {
                        const uint32_t e = rc + 2 * b;
                        if (!wait_w(&bars.full[slot_of(e)], use_of(e))) return false;
                        tc_fence_after();
                        const uint32_t id = idesc_bf16_f32(128, b == nx - 1 ? lk : kK, false, false);
                        const uint64_t k_d = k_d0 + slot_of(e) * (L::kTile >> 4);
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            mma_ss_elect(dS + j * 64, q_d + (((ks >> 2) * L::kQBox + (ks & 3) * 32) >> 4),
                                         k_d + (((ks >> 2) * L::kBox + (ks & 3) * 32) >> 4), id, ks > 0 ? 1u : 0u);
                    }
                    mma_commit_elect(&bars.s_full[it & 1][x][j]);
                    return true;
                };
                if (nx > 0) {
                    ok = wait_w(&bars.q_full[x], kq & 1) && issue_s(0) && issue_s(1);
                    ++kq;
                }
                for (int b = 0; ok && b < nx; ++b, ++pr) {
                    const uint32_t e = rc + 2 * b + 1, j = (sr + b) & 1;
                    ok = wait_w(&bars.full[slot_of(e)], use_of(e)) && wait_w(&bars.p_full[x][pr & 1], (pr >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t v_d = v_d0 + slot_of(e) * (L::kTile >> 4);
                    const int steps = (b == nx - 1 ? lk : kK) / 16;
                    auto pv = [&](int ks) {
                        mma_ts_elect(dO, dS + j * 64 + ks * 8, v_d + ((ks * 16 * 128) >> 4), idPV,
                                     (b > 0 || ks > 0) ? 1u : 0u);
                    };
                    if (steps == kK / 16) {
#pragma unroll
                        for (int ks = 0; ks < kK / 16; ++ks) pv(ks);
                    } else {
                        for (int ks = 0; ks < steps; ++ks) pv(ks);
                    }
                    ok = issue_s(b + 2);
                }
                const uint32_t rounds = nx > 0 ? sr + nx + 2 : sr;
                sr = sr_next;
                sr_next = rounds;
                // Key tiles that only the other tile has: seen in order and handed back.
                for (int b = nx; ok && b < n; ++b) {
                    for (int j = 0; ok && j < 2; ++j) {
                        const uint32_t e = rc + 2 * b + j;
                        ok = wait_w(&bars.full[slot_of(e)], use_of(e));
                        if (ok) mbar_arrive_elect(&bars.empty[slot_of(e)]);
                    }
                }
                rc += 2 * n;
                leave_unit(it);
            }
            mma_commit_elect(&bars.fin[x]);
            (void)mbar_wait(&bars.fin[x], 0, ctx);
            __syncwarp();
        } else {
            // ------------------------------------------------------------ units; V rows not every row sees
            PackedOrder order(cu, B, total, ut, lane, ctx, blockIdx.x == 0);
            auto publish = [&](int it) {
                // Every other round runs the CTAs backwards: units come longest first, and the turn evens
                // out what the CTAs get.
                const int c = (it & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
                const int64_t i = (int64_t)it * gridDim.x + c;
                const PackedTile t = order.at(i / n_hg);
                if (it >= 2 && !wait_warp(&bars.unit_empty[it & 1], ((it - 2) >> 1) & 1, ctx, abort)) return;
                if (lane == 0) {
                    bars.unit[it & 1] = Unit{t.start, t.len, t.first, (int)(i % n_hg)};
                    mbar_arrive(&bars.unit_full[it & 1]);
                }
            };
            publish(0);
            publish(1);
            uint32_t rc = 0;
            uint32_t nl[2][4] = {};
            Unit u;
            bool dirty[2] = {false, false};
            for (int it = 0; take_unit(it, u); ++it) {
                int lkA, lkB;
                const int nA = key_tiles(u, 0, tq, &lkA), nB = key_tiles(u, 1, tq, &lkB);
                const int n = max(nA, nB);
                const int last = min(u.first + ut, u.len) - 1;
                uint16_t* note = notes + (it & 1) * 2 * D;  // [sign][column]; keys from key base on
                const int base = (u.first / kK) * kK;
                // The unit that used these notes last is done (its softmax warps have left it).
                if (dirty[it & 1]) {
                    for (int e = lane; e < 2 * D; e += 32) note[e] = kNoKey;
                    if (lane == 0) bars.noted[it & 1] = 0;
                    dirty[it & 1] = false;
                    __syncwarp();
                }
                const int looked = u.first / kK;
                bool ok = true;
                for (int b = looked; ok && b < n; ++b) {
                    const uint32_t e = rc + 2 * b + 1;
                    ok = wait_warp(&bars.v_landed[it & 1][b - looked], nl[it & 1][b - looked]++ & 1, ctx, abort);
                    if (!ok) break;
                    const int k0 = b * kK;
                    const int r0 = max(u.first + 1 - k0, 0);
                    const int r1 = min(((last - k0) / 16 + 1) * 16, kK);  // what PV reads
                    constexpr int kC = D / 8;                                // 16-byte pieces per row
                    bool wrote = false;
                    for (int c0 = 0; c0 < (r1 - r0) * kC; c0 += 32) {
                        const int r = r0 + (c0 + lane) / kC, c = (c0 + lane) % kC;
                        bool bad = false;
                        uint4* p = nullptr;
                        if (r < r1) {
                            p = reinterpret_cast<uint4*>(slot_ptr(e) + (c >> 3) * L::kBox + r * 128 +
                                                         (((c & 7) ^ (r & 7)) << 4));
                            bad = any_nonfinite8(*p);
                        }
                        unsigned todo = __ballot_sync(0xffffffffu, bad);
                        if (todo == 0u) continue;
                        wrote = true;
                        for (; todo; todo &= todo - 1) {  // one lane after another: they share columns
                            if (lane == __ffs((int)todo) - 1) {
                                uint16_t* w = reinterpret_cast<uint16_t*>(p);
                                const uint16_t key = (uint16_t)(k0 + r - base);
                                for (int j = 0; j < 8; ++j) {
                                    if ((w[j] & 0x7f80u) != 0x7f80u) continue;
                                    const bool nan = (w[j] & 0x7fu) != 0u, neg = (w[j] & 0x8000u) != 0u;
                                    if (nan || !neg) note[c * 8 + j] = min(note[c * 8 + j], key);
                                    if (nan || neg) note[D + c * 8 + j] = min(note[D + c * 8 + j], key);
                                    w[j] = 0;
                                }
                            }
                            __syncwarp();
                        }
                    }
                    if (wrote) {
                        dirty[it & 1] = true;
                        if (lane == 0) bars.noted[it & 1] = 1;
                        fence_proxy_async_smem();  // the MMA reads what was just written
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.full[slot_of(e)]);
                    __syncwarp();
                }
                if (ok && lane == 0) mbar_arrive(&bars.v_seen[it & 1]);
                rc += 2 * n;
                leave_unit(it);
                if (!ok) break;
                publish(it + 2);
            }
        }
    } else {
        // ---------------------------------------------------------------- softmax + epilogue
        set_regs_up<216>();
        const int x = warp >> 2;
        const int r = tid & 127;
        const uint32_t lane_base = tmem_lane_base(warp);
        const uint32_t colO = tmem + lane_base + kColO + x * 128;
        const uint32_t colS = tmem + lane_base + kColS + x * 128;
        const bool lead = (tid & 127) == 0;  // hands stages and Q back for the tile
        uint32_t rc = 0, sr = 0, sr_next = 0, pr = 0;  // as the issuer's
        bool ok = true;
        Unit u;
        for (int it = 0; ok && take_unit(it, u); ++it) {
            int lkA, lkB;
            const int nA = key_tiles(u, 0, tq, &lkA), nB = key_tiles(u, 1, tq, &lkB);
            const int n = max(nA, nB), nx = x ? nB : nA;
            const int i = u.first + x * tq + r % tq;  // this row's token
            const int full_tiles = (u.first + x * tq + 1) / kK;  // key tiles that every row sees whole
            RowState st;
            auto round = [&](int b) { return wait_warp(&bars.s_full[it & 1][x][(sr + b) & 1], ((sr + b) >> 1) & 1, ctx, abort); };
            auto give = [&](int e) { mbar_arrive(&bars.empty[slot_of(rc + e)]); };
            for (int b = 0; b < nx; ++b, ++pr) {
                ok = round(b);
                if (!ok) break;
                tc_fence_after();
                if (lead) {  // S of this round is done with K, PV of the one before last with its V
                    give(2 * b);
                    if (b > 1) give(2 * b - 3);
                    if (b == nx - 1) mbar_arrive(&bars.q_empty[x]);
                }
                const uint32_t col = colS + ((sr + b) & 1) * 64;
                uint32_t s[kK];  // (columns that S left unwritten are hidden)
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                float alpha;
                tmem_ld32(col, *reinterpret_cast<uint32_t(*)[32]>(s));
                tmem_ld32(col + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
                tmem_ld_wait();
                if (b < full_tiles) {
                    alpha = st.raise(max2n(max32(s), max32(s + 32)) * sl2);
                    const float nb = st.shift();
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[16];
                        exp32<false, false>(s + 32 * c, sl2, nb, 0u, nullptr, acc, pk);
                        tmem_st16(col + 16 * c, pk);
                    }
                } else {
                    const int lim = i - b * kK;
                    const uint32_t s0 = bits_to(lim), s1 = bits_to(lim - 32);
                    alpha = st.raise(max2n(max32_masked(s, s0), max32_masked(s + 32, s1)) * sl2);
                    const float nb = st.shift();
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t pk[16];
                        exp32<true, false>(s + 32 * c, sl2, nb, c ? s1 : s0, nullptr, acc, pk);
                        tmem_st16(col + 16 * c, pk);
                    }
                }
                st.l += (acc[0] + acc[1]) + (acc[2] + acc[3]);
                if (b > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    ok = round(b + 1);  // committed behind PV of the round before: O is ours to scale
                    if (!ok) break;
                    tc_fence_after();
                    scale_row<D>(colO, alpha);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[x][pr & 1]);
            }
            if (!ok) break;
            ok = wait_warp(&bars.v_seen[it & 1], (it >> 1) & 1, ctx, abort);
            if (!ok) break;
            if (nx > 0) {
                ok = round(nx) && round(nx + 1);  // all of the unit's PV
                if (!ok) break;
                tc_fence_after();
                if (lead) {
                    if (nx > 1) give(2 * nx - 3);
                    give(2 * nx - 1);
                }
                sr += nx + 2;
                const float inv = 1.f / st.l;
                const uint16_t* note = notes + (it & 1) * 2 * D;
                const int key = i - (u.first / kK) * kK;  // as the notes count
                const bool noted = *reinterpret_cast<volatile int*>(&bars.noted[it & 1]) != 0;
                // 32 columns at a time through shared memory: a row's 64 bytes are then stored by four
                // neighbouring lanes, whole sectors, instead of 16 bytes of 32 rows at once.
                uint8_t* stage = sm + L::kOffStage + warp * 2048;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(colO + c0, o);
                    tmem_ld_wait();
                    if (noted) {  // rows behind an infinity or a NaN of V get it back
#pragma unroll
                        for (int q = 0; q < 32; ++q) {
                            const bool pos = note[c0 + q] <= key, neg = note[D + c0 + q] <= key;
                            float y = __uint_as_float(o[q]);
                            if (pos) y += INFINITY;
                            if (neg) y -= INFINITY;
                            o[q] = __float_as_uint(y);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * j]) * inv,
                                               __uint_as_float(o[8 * q + 2 * j + 1]) * inv);
                        *reinterpret_cast<uint4*>(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int sr_row = 8 * q + (lane >> 2);           // of the warp's 32 rows
                        const int rr = (warp & 3) * 32 + sr_row, token = u.first + x * tq + rr % tq;
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            stage + sr_row * 64 + (((lane & 3) ^ ((sr_row >> 1) & 3)) << 4));
                        if (token < u.len)
                            *reinterpret_cast<uint4*>(out + ((int64_t)(u.hg * tg + rr / tq) * total + u.start + token) * D +
                                                      c0 + 8 * (lane & 3)) = v;
                    }
                    __syncwarp();
                }
                tc_fence_before();
            }
            const uint32_t rounds = sr;
            sr = sr_next;
            sr_next = rounds;
            rc += 2 * n;
            leave_unit(it);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t packed_tc(const void* q, const void* k, const void* v, const int32_t* cu, void* o, int B,
                      int H, int Hkv, int total, float scale, cudaStream_t st, DevCtx ctx) {
    using L = Layout<D>;
    int tg = 1;
    while (tg < 16 && (H / Hkv) % (2 * tg) == 0) tg *= 2;
    const int tq = 128 / tg;
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return cudaErrorNotSupported;
    auto map = [&](CUtensorMap* m, const void* base, uint64_t heads, uint32_t rows, uint32_t planes) {
        cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)total, heads};
        cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * total};
        cuuint32_t box[3] = {64, rows, planes};
        cuuint32_t one[3] = {1, 1, 1};
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    CUtensorMap tmQ, tmK, tmV;
    if (!map(&tmQ, q, H, tq, tg) || !map(&tmK, k, Hkv, kK, 1) || !map(&tmV, v, Hkv, kK, 1))
        return cudaErrorInvalidValue;
    if (cudaError_t e = ensure_smem<packed_tc_kernel<D>>(L::kBytes); e != cudaSuccess) return e;
    // every sequence has at most one unit that is not full
    const long long units = ((long long)total / (2 * tq) + (B < total ? B : total)) * (H / tg);
    const int sms = device_sm_count();
    packed_tc_kernel<D><<<units < sms ? (int)units : sms, kThreads, L::kBytes, st>>>(
        tmQ, tmK, tmV, cu, static_cast<__nv_bfloat16*>(o), B, H, Hkv, total, tg,
        scale * 1.4426950408889634f, ctx);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_tc(const void* q, const void* k, const void* v, const int32_t* cu, void* o,
                             int B, int H, int Hkv, int total, int d, float scale, cudaStream_t st,
                             DevCtx ctx) {
    return d == 64 ? packed_tc<64>(q, k, v, cu, o, B, H, Hkv, total, scale, st, ctx)
                   : packed_tc<128>(q, k, v, cu, o, B, H, Hkv, total, scale, st, ctx);
}

}  // namespace sala
