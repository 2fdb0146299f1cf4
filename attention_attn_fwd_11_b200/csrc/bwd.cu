// bwd.cu -- gradients of the fused attention (fa_bwd) for sm_100a.
//
// With s_ij the (modified) score of query i and key j, the forward's
// log-sum-exp lse_i and its output O, the probabilities are recomputed, not
// kept:
//
//   P_ij   = exp(s_ij - lse_i)
//   D_i    = dO_i . O_i - dlse_i
//   dV_j   = sum_i P_ij dO_i
//   dS_ij  = P_ij (dO_i . V_j - D_i)         (times ds/dz = c (1 - tanh^2 z) under a softcap)
//   dQ_i   = scale sum_j dS_ij K_j,   dK_j = scale sum_i dS_ij Q_i
//   dsink_h = -sum_i exp(sink_h - lse_i) D_i
//
// Kernels on the caller's stream:
//   1. bwd_prep_kernel: D and the LSE of every row, one pass over O and dO.
//      Rows with no visible key (LSE -inf) and the padding up to a whole tile
//      get LSE +inf, which makes every P of the row exactly 0.
//   2. bwd_tile_kernel, persistent, in which every SM takes items from one
//      list until it is empty:
//      - 128 keys of one KV head, walking the query tiles of every head of its
//        group: dK and dV, whose sums over the group's heads stay in the
//        accumulators;
//      - 128 queries of one head, walking the key tiles: dQ.
//   3. bwd_join_kernel, where walks are so long beside the whole work that
//      they were cut into parts for several SMs (bwd_split): adds the parts up.
// Scores and dO V^T are formed in both walks: seven matrix products where five
// would do, but every sum has a fixed order: nothing is accumulated with
// atomics in HBM and the result does not depend on timing.
//
// Both walks are one code.  An item's 128 resident rows X1, X2 (K and V; or Q
// and dO) meet tiles of BN rows Y1, Y2 (Q and dO; or K and V):
//
//   S = X1 Y1^T,  T = X2 Y2^T       (128 x BN each, fp32 in TMEM)
//   A1 += dS Y1,  and for dK / dV A2 += P Y2
//
// so for dK and dV the tile is transposed: lanes are keys, columns queries.
//   warp 0      TMA producer: X1, X2 once, then rings of Y1 (with the LSE and
//               D of its rows) and Y2 tiles.
//   warp 1      MMA issuer (whole warp, one elected lane issues).
//   warp 2      the sinks' gradient, if asked for.
//   warps 4 ..  BN / 32 warpgroups, each 32 of the tile's columns: P from S,
//               then dS from P and T, both as bf16 A operands in TMEM, so that
//               those products read only Y from shared memory.
// BN is 128 where TMEM allows: a 128 x 64 product whose operands are both in
// shared memory reads 6 KB in its 32 cycles and takes 48 (measured), one of
// 128 x 128 8 KB in 64; and the issuer has half as many steps to take.
//
// Measured on one B200 (the floor: five products of the visible tiles at 1645
// TFLOP/s; this form's seven take 1.4 times as long):
//   causal, 2 x 16 heads x 2048 x 128:  124 us in bursts, 141 to 144 sustained (floor 52)
//   causal, 32 on 8 heads x 4096 x 128: 436 and 455 (209)
//   causal, 2 x 16 x 2048, 192 / 128:   175 and 184 to 190 (68)
//   mask, ALiBi, softcap and sinks, 2 x 8 x 1024 x 128: 66 to 67 (13)
// The first spends 131 us in the tile kernel under a profiler, its tensor pipe
// 51 % active, its exponentials' pipe 31 %.  Sustained, the power limit sets
// the pace: fewer cycles (a second issuing warp, 4 %) bought a lower clock and
// no time.
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "score_mods.cuh"
#include "sm100.cuh"

namespace fa {
namespace {

__device__ int g_bwd_err;

struct BwdGrad {  // an output [B, H, S, d]
    char *p;
    int64_t sb, sh, ss;
};

struct BwdArgs {
    int B, Hq, Hkv, Sq, Sk, causal;
    float scale, scale_log2;  // of dQ and dK (with what softcap4_slope leaves out); of the scores
    ScoreMods mods;
    // -LSE and -D of every row.  The row kernel may still be writing them when
    // the tile kernel starts: read behind its griddepcontrol.wait, with plain
    // loads (the read-only path promises nothing about data that changes under
    // a running kernel, and its loads may be moved ahead of the wait).
    const float *nlse, *ndelta;
    const uint4 *ext;            // the two of a row as the B side of the extra step (see BwdCfg)
    int64_t pitch;               // rows per (batch, head) of the three
    int kv_items, items;          // 128-key tiles of every KV head, then 128-query tiles of every head
    int *next;                    // first item that no CTA has taken
    int kv_len, kv_parts, q_len, q_parts;  // walks cut into parts (see bwd_split)
    float *kv_part, *q_part;               // and those parts' sums
    BwdGrad gq, gk, gv;
    int g_bf16;
    float *gsinks;  // NULL: not asked for
    float cap_scale;  // of the scores under a softcap
};

// (dS is ready on two barriers in turn: dQ's workers may finish a tile before
// the issuer has looked at the one before.)
enum { B_X1FULL, B_X2FULL, B_X1FREE, B_X2FREE, B_SFULL, B_TFULL, B_SREAD, B_TREAD, B_PREADY, B_DSREADY, B_SETEND = B_DSREADY + 2 };

// Shared and tensor memory of one walk.  TMEM holds the accumulators and one
// S and one T tile.  Where there is room P and dS get columns of their own, so
// that S and T are free as soon as they are read.
template <int DK, int DV, bool KV, bool MODS>
struct BwdCfg {
    static constexpr int BN = bwd_walk(DK);
    // dK / dV without modifiers: LSE and D enter the products as one more
    // step of 16 columns.
    static constexpr bool EXT = KV && !MODS;
    // Stages of Y1 and of Y2.  dQ needs the third of Y1 (K: the next tile's S
    // comes before this tile's product with it) more than the second of Y2;
    // with modifiers the room goes to the mask.
    static constexpr int NST1 = DK == 64 ? 4 : KV || MODS ? 2 : 3;
    static constexpr int NST2 = DK == 64 ? 4 : !KV && DK == 192 && !MODS ? 1 : 2;
    static constexpr int X_CHUNK = 128 * 128, Y_CHUNK = BN * 128;  // bytes of a 64-column chunk
    static constexpr int X1_BYTES = 128 * DK * 2, X2_BYTES = 128 * DV * 2;
    static constexpr int Y1_BYTES = BN * DK * 2, Y2_BYTES = BN * DV * 2;
    static constexpr int EXT_A = EXT ? 2 * 128 * 16 : 0;  // ones beside zeros, for S; then for T
    static constexpr int ROW_BYTES = EXT ? 2 * BN * 16 : KV ? 2 * BN * 4 : 0;  // LSE and D of a query tile
    static constexpr int OFF_ROW = 2 * EXT_A;
    static constexpr int OFF_X1 = (OFF_ROW + NST1 * ROW_BYTES + 1023) / 1024 * 1024;
    static constexpr int OFF_X2 = OFF_X1 + X1_BYTES;
    static constexpr int OFF_Y1 = OFF_X2 + X2_BYTES;
    static constexpr int OFF_Y2 = OFF_Y1 + NST1 * Y1_BYTES;
    static constexpr int END = OFF_Y2 + NST2 * Y2_BYTES;
    static constexpr int WARPS = BN / 8;  // of elementwise work: four for 32 columns
    static constexpr int TMEM_COLS = 512;
    static constexpr int ACC = DK + (KV ? DV : 0);
    // S and T lie behind dK and dV in both walks: dQ's first products may run
    // while the last dK and dV are read out.
    static constexpr int T_A1 = 0, T_A2 = DK, T_S = DK + DV, T_T = T_S + BN, T_END = T_T + BN;
    // P over S and dS over T (each warpgroup in its own columns), or apart
    static constexpr bool ALIAS = KV && T_END + BN > TMEM_COLS;
    static constexpr int WG_COLS = ALIAS ? 32 : 16;  // from one warpgroup's P or dS to the next
    static constexpr int T_P = ALIAS ? T_S : T_END;
    static constexpr int T_D = ALIAS ? T_T : KV ? T_END + BN / 2 : T_END + BN <= TMEM_COLS ? T_END : DK;
    // dQ has two dS tiles in turn: S and T of the next tile are issued before
    // this tile's product, so the next dS would wait for all three.
    static constexpr int D_COLS = KV ? 0 : BN / 2;  // from one dS to the next
    static_assert(T_END <= TMEM_COLS && T_D + (ALIAS ? BN : BN / 2 + D_COLS) <= TMEM_COLS, "TMEM budget");
    static_assert(T_D >= T_END || ALIAS || T_D + BN <= T_S, "dS apart from S");
    // Barriers of this walk (each kind of item has its own set).
    static constexpr int FULL1 = B_SETEND, EMPTY1 = FULL1 + NST1, FULL2 = EMPTY1 + NST1, EMPTY2 = FULL2 + NST2;
    static constexpr int BARS = EMPTY2 + NST2;
};


template <int DK, int DV, bool MODS>
struct BwdKernel {
    using CK = BwdCfg<DK, DV, true, MODS>;
    using CQ = BwdCfg<DK, DV, false, MODS>;
    static constexpr int THREADS = 128 + 32 * CK::WARPS;
    // A warp's 32 x 32 mask values (f16), apart from both walks' tiles.
    static constexpr int OFF_MASK = CK::END > CQ::END ? CK::END : CQ::END;
    static constexpr int OFF_BAR = OFF_MASK + (MODS ? CK::WARPS * 2048 : 0);
    // Barriers: the item ring (full, empty), the end of a walk's products, of
    // all of them, of the last dK / dV's, the workers' change from dK / dV to
    // dQ, then both kinds' sets.
    static constexpr int BAR_DONE = 4, BAR_END = 5, BAR_KVEND = 6, BAR_MOVED = 7, BAR_KV = 8, BAR_Q = BAR_KV + CK::BARS, BARS = BAR_Q + CQ::BARS;
    static constexpr int SMEM_BYTES = OFF_BAR + 8 * BARS + 32;  // item ring, TMEM address, flag
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// One item: a 128-row tile x0 of (b, h) and its walk over tiles y_first ..
// y_first + n_y - 1, for dK / dV once per head of the group.  Of the whole
// walk's tiles the item has n, from tile y of head h_first on.
struct BwdItem {
    int b, h, x0, y_first, n_y, whole, n, y, h_first;
};

// Items in the order in which they are taken: dK / dV, then dQ, each with the
// longest walks first (key tile 0 sees the most queries, the last query tile
// the most keys), so that what is taken last is short.
template <bool KV, int BN>
FA_DEV BwdItem bwd_tile(const BwdArgs &a, int turn, int bh) {  // a whole walk
    BwdItem it;
    const int H = KV ? a.Hkv : a.Hq;
    const int xt = KV ? turn : (a.Sq + 127) / 128 - 1 - turn;
    it.b = bh / H;
    it.h = bh % H;
    it.x0 = xt * 128;
    const int shift = a.Sk - a.Sq;  // causal: key j is visible to query i iff j <= i + shift
    it.y_first = 0;
    if (KV) {
        if (a.causal) it.y_first = max(0, it.x0 - shift) / BN;
        it.n_y = max(0, (a.Sq + BN - 1) / BN - it.y_first);
        it.whole = it.n_y * (a.Hq / a.Hkv);
    } else {
        int last = a.Sk;  // keys visible to the tile's last row
        if (a.causal) last = min(last, min(a.Sq, it.x0 + 128) + shift);
        it.n_y = last <= 0 ? 0 : (last + BN - 1) / BN;
        it.whole = it.n_y;
    }
    it.n = it.whole, it.y = 0, it.h_first = KV ? it.h * (a.Hq / a.Hkv) : it.h;
    return it;
}
template <bool KV, int BN>
FA_DEV BwdItem bwd_item(const BwdArgs &a, int i) {
    const unsigned per = (unsigned)(a.B * (KV ? a.Hkv : a.Hq)), idx = (unsigned)(KV ? i : i - a.kv_items);
    const int parts = KV ? a.kv_parts : a.q_parts, len = KV ? a.kv_len : a.q_len;
    int turn = (int)(idx / per), part = 0;
    if (len > 0) part = turn % parts, turn /= parts;
    BwdItem it = bwd_tile<KV, BN>(a, turn, (int)(idx % per));
    if (len > 0) {
        const int t0 = part * len;
        it.n = min(len, max(0, it.whole - t0));
        if (it.n > 0) it.y = t0 % it.n_y, it.h_first += t0 / it.n_y;
    }
    return it;
}

// A position in a ring of N stages: the stage and the parity of its use.
template <int N>
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    FA_DEV void next() {
        if (++s == N) s = 0, ph ^= 1u;
    }
};

// What every role of a CTA shares.
struct BwdCta {
    uint8_t *smem;
    uint32_t sbase, bar0, tmem, mask;
    volatile int *abort_flag;
    FA_DEV uint32_t bar(int i) const { return bar0 + 8u * (uint32_t)i; }
    FA_DEV bool wait(int i, uint32_t parity) const {
        return mbar_wait_warp(bar(i), parity, abort_flag, &g_bwd_err);
    }
    FA_DEV bool wait1(int i, uint32_t parity) const { return mbar_wait(bar(i), parity, abort_flag, &g_bwd_err); }
};

// ---- warp 0, one lane: TMA producer ----------------------------------------
template <class C>
struct BwdProducer {
    Ring<C::NST1> r1;
    Ring<C::NST2> r2;
    int issued1 = 0, issued2 = 0, walks = 0;  // tiles asked for; items whose X1 and X2 were
    bool x1_pending = false;                  // X1 of one more was

    template <int DK, int DV, bool KV>
    FA_DEV bool item(const BwdCta &c, const BwdArgs &a, const BwdItem &it, int bars, const CUtensorMap *tmX1,
                     const CUtensorMap *tmX2, const CUtensorMap *tmY1, const CUtensorMap *tmY2) {
        if (it.n == 0) return true;
        const int group = a.Hq / a.Hkv;
        const uint32_t sb = c.sbase;
        // X of the walk before is free when its last S, its last T is done.
        const uint32_t px = ((uint32_t)walks & 1u) ^ 1u;
        int y = it.y, hy = KV ? it.h_first : it.h / group;
        for (int t = 0; t < it.n; ++t) {
            const int y0 = (it.y_first + y) * C::BN;
            if (t == 0) {
                if (!c.wait1(bars + B_X1FREE, px)) return false;
                const uint32_t xf = c.bar(bars + B_X1FULL);
                mbar_arrive_expect_tx(xf, C::X1_BYTES);
                x1_pending = true;
                for (int i = 0; i < DK / 64; ++i)
                    tma_load_4d(sb + C::OFF_X1 + i * C::X_CHUNK, tmX1, xf, i * 64, it.x0, it.h, it.b);
            }
            if (!c.wait1(bars + C::EMPTY1 + r1.s, r1.ph ^ 1u)) return false;
            const uint32_t f1 = c.bar(bars + C::FULL1 + r1.s);
            mbar_arrive_expect_tx(f1, C::Y1_BYTES + (C::EXT ? C::ROW_BYTES / 2 : C::ROW_BYTES));
            for (int i = 0; i < DK / 64; ++i)
                tma_load_4d(sb + C::OFF_Y1 + r1.s * C::Y1_BYTES + i * C::Y_CHUNK, tmY1, f1, i * 64, y0, hy, it.b);
            if (KV) {
                const int64_t row = ((int64_t)it.b * a.Hq + hy) * a.pitch + y0;
                const uint32_t sr = sb + C::OFF_ROW + r1.s * C::ROW_BYTES;
                if (C::EXT) {
                    bulk_load(sr, a.ext + row, C::BN * 16, f1);
                } else {
                    bulk_load(sr, a.nlse + row, C::BN * 4, f1);
                    bulk_load(sr + C::BN * 4, a.ndelta + row, C::BN * 4, f1);
                }
            }
            r1.next();
            ++issued1;
            if (t == 0) {
                if (!c.wait1(bars + B_X2FREE, px)) return false;
                const uint32_t xf = c.bar(bars + B_X2FULL);
                mbar_arrive_expect_tx(xf, C::X2_BYTES);
                for (int i = 0; i < DV / 64; ++i)
                    tma_load_4d(sb + C::OFF_X2 + i * C::X_CHUNK, tmX2, xf, i * 64, it.x0, it.h, it.b);
                ++walks;
                x1_pending = false;
            }
            if (!c.wait1(bars + C::EMPTY2 + r2.s, r2.ph ^ 1u)) return false;
            const uint32_t f2 = c.bar(bars + C::FULL2 + r2.s);
            mbar_arrive_expect_tx(f2, C::Y2_BYTES);
            for (int i = 0; i < DV / 64; ++i)
                tma_load_4d(sb + C::OFF_Y2 + r2.s * C::Y2_BYTES + i * C::Y_CHUNK, tmY2, f2, i * 64, y0, hy, it.b);
            r2.next();
            ++issued2;
            if (++y == it.n_y) y = 0, ++hy;
        }
        return true;
    }
    // After an abort: lets the copies already in flight land.
    FA_DEV void drain(const BwdCta &c, int bars) const {
        for (int i = max(0, issued1 - C::NST1); i < issued1; ++i)
            mbar_wait_drain(c.bar(bars + C::FULL1 + i % C::NST1), (uint32_t)(i / C::NST1) & 1u);
        for (int i = max(0, issued2 - C::NST2); i < issued2; ++i)
            mbar_wait_drain(c.bar(bars + C::FULL2 + i % C::NST2), (uint32_t)(i / C::NST2) & 1u);
        for (int i = max(0, walks - 1); i < walks; ++i) {
            mbar_wait_drain(c.bar(bars + B_X1FULL), (uint32_t)i & 1u);
            mbar_wait_drain(c.bar(bars + B_X2FULL), (uint32_t)i & 1u);
        }
        if (x1_pending) mbar_wait_drain(c.bar(bars + B_X1FULL), (uint32_t)walks & 1u);
    }
};

// ---- warp 1: MMA issuer (the whole warp, one elected lane issues) ------------
template <int DK, int DV, bool KV, class C>
struct BwdIssuer {
    Ring<C::NST1> s1, a1;  // Y1 stages of the next S and of the next dS product
    Ring<C::NST2> s2, a2;  // Y2 stages of the next T and of the next P product
    Ring<C::NST1> e1;      // Y1 stage of the tile whose T comes next (its rows' D)
    uint32_t walks = 0, tiles_s = 0, tiles_t = 0, tiles = 0;

    // 128 x BN product over D columns of a resident operand and a tile, both
    // K-major.
    template <int D>
    FA_DEV static void product(uint32_t d, uint32_t xs, uint32_t ys) {
        constexpr uint32_t id = idesc_bf16_f32(128, C::BN, false, false);
        const uint64_t x = sdesc_sw128(xs, 16, 1024), y = sdesc_sw128(ys, 16, 1024);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
            mma_ss4_warp<2, 4, 6>(d, x + (uint64_t)((c * C::X_CHUNK) >> 4), y + (uint64_t)((c * C::Y_CHUNK) >> 4), id, c > 0);
    }
    // Accumulator += (P or dS) Y over the tile's BN rows.
    template <int D>
    FA_DEV static void accumulate(uint32_t d, uint32_t pa, uint32_t ys, bool first) {
        constexpr uint32_t id = idesc_bf16_f32(128, D, false, true);
        const uint64_t y = sdesc_sw128(ys, C::Y_CHUNK, 1024);
        mma_ts4at_warp<8, C::WG_COLS, C::WG_COLS + 8, 128>(d, pa, y, id, !first);
        if constexpr (C::BN == 128)
            mma_ts4at_warp<8, C::WG_COLS, C::WG_COLS + 8, 128>(d, pa + 2 * C::WG_COLS, y + 512, id, 1);
        else
            mma_ts2_warp<8, 128>(d, pa + 2 * C::WG_COLS, y + 512, id, 1);
    }
    // The step that adds -LSE to S (off 0) or -D to T (off EXT_A).
    FA_DEV static void extra(const BwdCta &c, uint32_t d, uint32_t off, int stage) {
        if (C::EXT)
            mma_ss_warp(d, sdesc_plain(c.sbase + off, 2048, 128),
                        sdesc_plain(c.sbase + C::OFF_ROW + stage * C::ROW_BYTES, C::BN * 16, 128),
                        idesc_bf16_f32(128, C::BN, false, false), 1);
    }
    FA_DEV bool issue_s(const BwdCta &c, int bars, bool first, bool last) {
        if (first && !c.wait(bars + B_X1FULL, walks & 1u)) return false;
        if (!c.wait(bars + C::FULL1 + s1.s, s1.ph)) return false;
        if (!C::ALIAS && tiles_s > 0 && !c.wait(bars + B_SREAD, (tiles_s - 1) & 1u)) return false;
        tc_fence_after();
        product<DK>(c.tmem + C::T_S, c.sbase + C::OFF_X1, c.sbase + C::OFF_Y1 + s1.s * C::Y1_BYTES);
        extra(c, c.tmem + C::T_S, 0, s1.s);
        mma_commit_warp(c.bar(bars + B_SFULL));
        if (last) mma_commit_warp(c.bar(bars + B_X1FREE));
        s1.next();
        ++tiles_s;
        return true;
    }
    FA_DEV bool issue_t(const BwdCta &c, int bars, bool first, bool last) {
        if (first && !c.wait(bars + B_X2FULL, walks & 1u)) return false;
        if (!c.wait(bars + C::FULL2 + s2.s, s2.ph)) return false;
        // (dK / dV: behind dS's product, so the T before has been read.)
        if (!KV && tiles_t > 0 && !c.wait(bars + B_TREAD, (tiles_t - 1) & 1u)) return false;
        tc_fence_after();
        product<DV>(c.tmem + C::T_T, c.sbase + C::OFF_X2, c.sbase + C::OFF_Y2 + s2.s * C::Y2_BYTES);
        extra(c, c.tmem + C::T_T, C::EXT_A, e1.s);
        mma_commit_warp(c.bar(bars + B_TFULL));
        if (!KV) mma_commit_warp(c.bar(bars + C::EMPTY2 + s2.s));
        if (last) mma_commit_warp(c.bar(bars + B_X2FREE));
        s2.next();
        e1.next();
        ++tiles_t;
        return true;
    }
    FA_DEV bool item(const BwdCta &c, int n, int bars, int done) {
        if (n == 0) return true;
        if (!issue_s(c, bars, true, n == 1) || !issue_t(c, bars, true, n == 1)) return false;
        ++walks;
        for (int t = 0; t < n; ++t) {
            const bool more = t + 1 < n, last = t + 2 == n;
            if (!C::ALIAS && more && !issue_s(c, bars, false, last)) return false;
            if (KV) {
                if (!c.wait(bars + B_PREADY, tiles & 1u)) return false;
                tc_fence_after();
                accumulate<DV>(c.tmem + C::T_A2, c.tmem + C::T_P, c.sbase + C::OFF_Y2 + a2.s * C::Y2_BYTES, t == 0);
                mma_commit_warp(c.bar(bars + C::EMPTY2 + a2.s));
                a2.next();
            }
            // In place of P and dS, or where nothing waits for them: behind the
            // products that read those.
            if (C::ALIAS && more && !issue_s(c, bars, false, last)) return false;
            if (!KV && more && !issue_t(c, bars, false, last)) return false;
            if (!c.wait(bars + B_DSREADY + (int)(tiles & 1u), (tiles >> 1) & 1u)) return false;
            tc_fence_after();
            accumulate<DK>(c.tmem + C::T_A1, c.tmem + C::T_D + (tiles & 1u) * C::D_COLS, c.sbase + C::OFF_Y1 + a1.s * C::Y1_BYTES, t == 0);
            mma_commit_warp(c.bar(bars + C::EMPTY1 + a1.s));
            a1.next();
            if (KV && more && !issue_t(c, bars, false, last)) return false;
            ++tiles;
        }
        mma_commit_warp(c.bar(done));
        return true;
    }
};

// ---- warps 4 ..: P, dS, epilogue -------------------------------------------------

// Four 16-byte units a lane (unit u of its own row) to: lane l of each group
// of four holds unit l % 4 of the group's rows 0 .. 3, so that four lanes write
// 64 contiguous bytes of one row.
FA_DEV void transpose4(uint4 (&u)[4], int lane) {
    const auto swap = [&](uint4 &x, uint4 &y, int d, bool up) {
        // the lane with the bit clear gives y and keeps x, the other the reverse
        const uint4 give = up ? x : y;
        const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, d), __shfl_xor_sync(0xffffffffu, give.y, d),
                                     __shfl_xor_sync(0xffffffffu, give.z, d), __shfl_xor_sync(0xffffffffu, give.w, d));
        if (up)
            x = got;
        else
            y = got;
    };
    const bool b0 = lane & 1, b1 = lane & 2;
    swap(u[0], u[1], 1, b0);
    swap(u[2], u[3], 1, b0);
    swap(u[0], u[2], 2, b1);
    swap(u[1], u[3], 2, b1);
}

// 32 columns (fp32 bits in r, times f) of 32 rows of a gradient: this lane's
// row is row0 + lane, rows at or past S are not stored.
FA_DEV void store_rows(const BwdGrad &g, int bf16, int b, int h, int row0, int S, int col, const uint32_t (&r)[32], float f,
                       int lane) {
    const int q = lane & 3, first = row0 + (lane & ~3);
    char *base = g.p + ((int64_t)b * g.sb + (int64_t)h * g.sh) * (bf16 ? 2 : 4);
    const int units = bf16 ? 1 : 2;  // of 64 bytes
    for (int v = 0; v < units; ++v) {
        uint4 u[4];
        if (bf16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = make_uint4(pack_bf16x2(__uint_as_float(r[8 * i]) * f, __uint_as_float(r[8 * i + 1]) * f),
                                  pack_bf16x2(__uint_as_float(r[8 * i + 2]) * f, __uint_as_float(r[8 * i + 3]) * f),
                                  pack_bf16x2(__uint_as_float(r[8 * i + 4]) * f, __uint_as_float(r[8 * i + 5]) * f),
                                  pack_bf16x2(__uint_as_float(r[8 * i + 6]) * f, __uint_as_float(r[8 * i + 7]) * f));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = __float_as_uint(__uint_as_float(v ? r[16 + 4 * i + j] : r[4 * i + j]) * f);
                u[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        transpose4(u, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (first + i < S)
                *reinterpret_cast<uint4 *>(base + ((int64_t)(first + i) * g.ss + col) * (bf16 ? 2 : 4) + 64 * v + 16 * q) =
                    u[i];
    }
}

template <int DK, int DV, bool KV, bool MODS, class C>
struct BwdWorker {
    Ring<C::NST1> r1, p1;  // Y1 stage of this tile, of the tile whose dS it replaces
    Ring<C::NST2> p2;      // Y2 stage of the tile before
    uint32_t tiles = 0;

    FA_DEV static void arrive(const BwdCta &c, int i, int lane) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(c.bar(i));
    }

    FA_DEV bool item(const BwdCta &c, const BwdArgs &a, int index, int bars, int done, uint32_t &dones) {
        const BwdItem it = bwd_item<KV, C::BN>(a, index);
        constexpr int BN = C::BN;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int wg = (warp >> 2) - 1;           // columns 32 wg .. 32 wg + 31 of each tile
        const int row = (warp & 3) * 32 + lane;   // resident row: key or query
        const uint32_t tl = c.tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = tl + C::T_S + wg * 32, tT = tl + C::T_T + wg * 32;
        const uint32_t tP = tl + C::T_P + wg * C::WG_COLS, tD = tl + C::T_D + wg * C::WG_COLS;
        const int x0 = it.x0, xr = x0 + row;
        const int shift = a.Sk - a.Sq;
        const bool capped = MODS && a.mods.softcap != 0.f;
        const bool masked = MODS && a.mods.mask != nullptr;
        float row_nlse = 0.f, row_ndelta = 0.f;
        if (!KV) {  // rows past Sq are padded in the workspace
            const int64_t r = ((int64_t)it.b * a.Hq + it.h) * a.pitch + xr;
            row_nlse = a.nlse[r] * (MODS ? 1.f : kLog2e);
            row_ndelta = a.ndelta[r];
        }
        // dQ: columns c >= lim_hi - y0 of this row are hidden; dK / dV:
        // columns c < lim_lo - y0 of this key.
        const int lim_hi = a.causal ? min(a.Sk, xr + shift + 1) : a.Sk;
        const int lim_lo = a.causal ? xr - shift : 0;
        const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
        int y = it.y, hq = it.h_first;
        // The warp's mask values of a tile, 32 queries x 32 keys, come to shared
        // memory a tile ahead.  A query has 64 bytes, its 16-byte quarters
        // turned so that neither eight rows' quarters nor one row's halves
        // meet in a bank.  What lies past the end is 0: its P is 0, or its
        // results are not stored.
        const uint8_t *mv = c.smem + c.mask + (warp - 4) * 2048;
        const uint32_t ms = smem_u32(mv);
        const auto ask_mask = [&](int head, int tile) {
            const int walked = (it.y_first + tile) * BN + wg * 32, mine = x0 + (warp & 3) * 32;
            const int q0 = KV ? walked : mine, key = (KV ? mine : walked) + 8 * (lane & 3);
            const __half *m = a.mods.mask + (int64_t)it.b * a.mods.m_sb + (int64_t)head * a.mods.m_sh;
            const int width = min(16, max(0, 2 * (a.Sk - key)));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 8 * j + (lane >> 2);
                const int bytes = q0 + r < a.Sq ? width : 0;
                cp_async16(ms + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4), bytes ? m + (int64_t)(q0 + r) * a.mods.m_ss + key : m,
                           bytes);
            }
            cp_async_commit();
        };
        if (MODS && masked && it.n > 0) ask_mask(hq, y);
        for (int t = 0; t < it.n; ++t) {
            const int y0 = (it.y_first + y) * BN + wg * 32;  // first column: query or key
            const float *sl = reinterpret_cast<const float *>(c.smem + C::OFF_ROW + r1.s * C::ROW_BYTES) + wg * 32;
            const float slope = MODS ? alibi_slope(a.mods, hq) : 0.f;
            if (KV && MODS && !c.wait(bars + C::FULL1 + r1.s, r1.ph)) return false;
            if (!c.wait(bars + B_SFULL, tiles & 1u)) return false;
            tc_fence_after();
            float x[32];
            {
                uint32_t r[32];
                tmem_ld32(tS, r);
                tmem_wait_ld();
                reg_fence(r);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
            }
            if (!C::ALIAS) arrive(c, bars + B_SREAD, lane);
            const bool edge = KV ? (a.causal && y0 < x0 + 127 - shift)
                                 : (y0 + 32 > min(a.Sk, a.causal ? x0 + shift + 1 : a.Sk));
            const auto hide = [&](float (&v)[4], int i) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (KV ? (y0 + i + j < lim_lo) : (y0 + i + j >= lim_hi)) v[j] = -INFINITY;
            };
            if (MODS && masked) {
                cp_async_wait<0>();
                __syncwarp();
            }
            // P (and under a softcap P ds/dz / (4 softcap) in its place in x)
            uint32_t pk[16];
            // (One form for each set of modifiers: branches inside would keep
            // the columns' chains from overlapping.)
            const auto probabilities = [&](auto capped_, auto masked_) {
                [[maybe_unused]] constexpr bool CAPPED = decltype(capped_)::value, MASKED = decltype(masked_)::value;
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    float v[4] = {x[i], x[i + 1], x[i + 2], x[i + 3]};
                    float cap[4] = {1.f, 1.f, 1.f, 1.f};
                    // -LSE of the four: natural with modifiers, where the mask is
                    // added to it first (both may be as large as the mask's lowest
                    // value, and their sum is what counts), else in base 2
                    uint64_t nl[2];
                    if (C::EXT) {
                        nl[0] = nl[1] = 0;
                    } else if (KV) {
                        const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(sl + i);
                        nl[0] = l.x, nl[1] = l.y;
                    } else {
                        nl[0] = nl[1] = f2_pack(row_nlse, row_nlse);
                    }
                    if constexpr (MODS) {
                        if constexpr (CAPPED) {
                            softcap4_slope(v, cap, a.cap_scale, a.mods.softcap);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[j] *= a.scale_log2;
                        }
                        if constexpr (MASKED) {
                            float m[4];
                            if (KV) {
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    m[j] = __half2float(*reinterpret_cast<const __half *>(
                                        mv + (i + j) * 64 + (((lane >> 3) ^ ((i + j) >> 1 & 3)) << 4) + 2 * (lane & 7)));
                            } else {
                                const uint2 w = *reinterpret_cast<const uint2 *>(
                                    mv + lane * 64 + (((i >> 3) ^ (lane >> 1 & 3)) << 4) + (i & 4) * 2);
                                const float2 lo = __half22float2(*reinterpret_cast<const __half2 *>(&w.x));
                                const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&w.y));
                                m[0] = lo.x, m[1] = lo.y, m[2] = hi.x, m[3] = hi.y;
                            }
#pragma unroll
                            for (int j = 0; j < 4; j += 2)
                                nl[j / 2] = f2_fma(f2_pack(m[j], m[j + 1]), f2_pack(slope, slope), nl[j / 2]);
                        }
                    }
                    if (edge) hide(v, i);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int k = i + 2 * j;
                        const uint64_t xx = f2_pack(v[2 * j], v[2 * j + 1]);
                        float e0, e1;
                        f2_unpack(C::EXT ? f2_mul(xx, sc2)
                                  : MODS ? f2_fma(nl[j], f2_pack(kLog2e, kLog2e), xx)
                                         : f2_fma(xx, sc2, nl[j]), e0, e1);
                        x[k] = ex2(e0);
                        x[k + 1] = ex2(e1);
                        pk[k / 2] = pack_bf16x2(x[k], x[k + 1]);
                        if constexpr (CAPPED) f2_unpack(f2_mul(f2_pack(x[k], x[k + 1]), f2_pack(cap[2 * j], cap[2 * j + 1])), x[k], x[k + 1]);
                    }
                }
            };
            constexpr std::true_type yes;
            constexpr std::false_type no;
            if (capped)
                masked ? probabilities(yes, yes) : probabilities(yes, no);
            else
                masked ? probabilities(no, yes) : probabilities(no, no);
            if (MODS && masked) {
                __syncwarp();
                if (t + 1 < it.n) {
                    const bool wrap = y + 1 == it.n_y;
                    ask_mask(wrap ? hq + 1 : hq, wrap ? 0 : y + 1);
                }
            }
            if (KV) {
                // With its own columns: the product over the P before is done.
                if (!C::ALIAS && tiles > 0) {
                    if (!c.wait(bars + C::EMPTY2 + p2.s, p2.ph)) return false;
                    p2.next();
                }
                tmem_st16(tP, pk);
                tmem_wait_st();
                arrive(c, bars + B_PREADY, lane);
            }
            // dS
            if (!c.wait(bars + B_TFULL, tiles & 1u)) return false;
            tc_fence_after();
            uint32_t r[32];
            tmem_ld32(tT, r);
            tmem_wait_ld();
            reg_fence(r);
            if (!KV) arrive(c, bars + B_TREAD, lane);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                uint64_t nd[2];
                if (C::EXT) {
                    nd[0] = nd[1] = 0;
                } else if (KV) {
                    const ulonglong2 d = *reinterpret_cast<const ulonglong2 *>(sl + BN + i);
                    nd[0] = d.x, nd[1] = d.y;
                } else {
                    nd[0] = nd[1] = f2_pack(row_ndelta, row_ndelta);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = i + 2 * j;
                    uint64_t tt = f2_pack(__uint_as_float(r[k]), __uint_as_float(r[k + 1]));
                    if (!C::EXT) tt = f2_add(tt, nd[j]);
                    float d0, d1;
                    f2_unpack(f2_mul(f2_pack(x[k], x[k + 1]), tt), d0, d1);
                    pk[k / 2] = pack_bf16x2(d0, d1);
                }
            }
            // The product over the dS that was in these columns is done.
            if (!C::ALIAS && tiles > (KV ? 0u : 1u)) {
                if (!c.wait(bars + C::EMPTY1 + p1.s, p1.ph)) return false;
                p1.next();
            }
            tmem_st16(tD + (tiles & 1u) * C::D_COLS, pk);
            tmem_wait_st();
            arrive(c, bars + B_DSREADY + (int)(tiles & 1u), lane);
            r1.next();
            ++tiles;
            if (++y == it.n_y) y = 0, ++hq;
        }
        if (it.n > 0) {
            if (!c.wait(done, dones & 1u)) return false;
            ++dones;
            tc_fence_after();
        }
        // 32 accumulator columns at a time, dealt to the warpgroups.  The next
        // item's products into the accumulators wait for this warp's next P
        // and dS, so they cannot come before these loads.
        const int row0 = x0 + (warp & 3) * 32, S = KV ? a.Sk : a.Sq;
        if ((KV ? a.kv_len : a.q_len) > 0) {
            if (it.n > 0) {
                float4 *to = reinterpret_cast<float4 *>(KV ? a.kv_part + (int64_t)index * (128 * C::ACC)
                                                           : a.q_part + (int64_t)(index - a.kv_items) * (128 * C::ACC)) + row;
                for (int col = wg * 32; col < C::ACC; col += BN) {
                    uint32_t r[32];
                    tmem_ld32(tl + (uint32_t)(C::T_A1 + col), r);
                    tmem_wait_ld();
                    reg_fence(r);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        to[(col / 4 + i) * 128] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                                                              __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
                }
            }
            return true;
        }
        for (int col = wg * 32; col < C::ACC; col += BN) {
            const bool second = col >= DK;
            uint32_t r[32];
            if (it.n > 0) {
                tmem_ld32(tl + (uint32_t)(C::T_A1 + col), r);
                tmem_wait_ld();
                reg_fence(r);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = 0u;
            }
            store_rows(KV ? (second ? a.gv : a.gk) : a.gq, a.g_bf16, it.b, it.h, row0, S, second ? col - DK : col, r,
                       second ? 1.f : a.scale, lane);
        }
        return true;
    }
};

// ---- warp 2: the sinks' gradient, a head at a time ---------------------------
// A double a lane, in the order of the rows, and then the lanes; each term is a
// product in fp32, whose factors have no more bits.
FA_DEV void sink_gradients(const BwdArgs &a, int lane) {
    for (int h = blockIdx.x; h < a.Hq; h += gridDim.x) {
        const float sk = __ldg(a.mods.sinks + h);
        double s = 0;
        for (int b = 0; b < a.B; ++b) {
            const int64_t r = ((int64_t)b * a.Hq + h) * a.pitch;
#pragma unroll 4
            for (int i = lane; i < a.Sq; i += 32) s += ex2((sk + a.nlse[r + i]) * kLog2e) * a.ndelta[r + i];
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
        if (lane == 0) a.gsinks[h] = (float)s;
    }
}

// Persistent: one CTA an SM takes items from a counter until none is left.
template <int DK, int DV, bool MODS>
__global__ void __launch_bounds__(BwdKernel<DK, DV, MODS>::THREADS, 1)
bwd_tile_kernel(const __grid_constant__ CUtensorMap tmQx, const __grid_constant__ CUtensorMap tmKx,
                const __grid_constant__ CUtensorMap tmVx, const __grid_constant__ CUtensorMap tmDOx,
                const __grid_constant__ CUtensorMap tmQy, const __grid_constant__ CUtensorMap tmKy,
                const __grid_constant__ CUtensorMap tmVy, const __grid_constant__ CUtensorMap tmDOy, const BwdArgs a) {
    using K = BwdKernel<DK, DV, MODS>;
    using CK = typename K::CK;
    using CQ = typename K::CQ;
    constexpr int BN = CK::BN, WARPS = CK::WARPS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    BwdCta c;
    c.smem = smem_raw;
    c.sbase = smem_u32(c.smem);
    c.mask = K::OFF_MASK;
    uint64_t *bars = reinterpret_cast<uint64_t *>(c.smem + K::OFF_BAR);
    c.bar0 = smem_u32(bars);
    volatile int *slot = reinterpret_cast<volatile int *>(bars + K::BARS);  // two items
    uint32_t *tmem_holder = const_cast<uint32_t *>(reinterpret_cast<volatile uint32_t *>(slot + 2));
    c.abort_flag = slot + 3;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < K::BARS; ++i) {
            int count = 1;
            if (i == 2 || i == 3) count = 1 + WARPS;  // an item is free once the issuer and the workers have it
            if (i == K::BAR_MOVED) count = WARPS;
            const int j = i >= K::BAR_Q ? i - K::BAR_Q : i - K::BAR_KV;
            if (i >= K::BAR_KV && j >= B_SREAD && j < B_SETEND) count = WARPS;
            mbar_init(c.bar(i), count);
        }
        *c.abort_flag = 0;
        fence_barrier_init();
    }
    if (CK::EXT) {
        // A side of the extra step: row = 1 in columns 0 .. 2 for S (the three
        // pieces of the LSE), 3 .. 5 for T (those of D); the second half of
        // its 16 columns, on both sides, is zeros.
        uint4 *e = reinterpret_cast<uint4 *>(c.smem);
        for (int i = threadIdx.x; i < 2 * CK::EXT_A / 16; i += K::THREADS)
            e[i] = (i & 128) ? make_uint4(0, 0, 0, 0)
                   : i < 256 ? make_uint4(0x3f803f80u, 0x3f80u, 0, 0)
                             : make_uint4(0, 0x3f800000u, 0x3f803f80u, 0);
        for (int i = threadIdx.x; i < CK::NST1 * BN; i += K::THREADS)
            reinterpret_cast<uint4 *>(c.smem + CK::OFF_ROW + (i / BN) * CK::ROW_BYTES)[BN + i % BN] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_holder), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    c.tmem = *tmem_holder;
    // What follows reads the row kernel's results, or writes memory that
    // earlier work on the stream may still read.
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Item k of this CTA, or -1: waits until the producer has put it there.
    auto take = [&](int k) -> int {
        if (!c.wait(k & 1, (uint32_t)(k >> 1) & 1u)) return -1;
        const int i = slot[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(c.bar(2 + (k & 1)));
        return i < a.items ? i : -1;
    };

    if (warp == 0) {
        if (lane == 0) {
            if (a.Sq > 0 && a.Sk > 0) {  // an empty side has no maps
                prefetch_tmap(&tmQx), prefetch_tmap(&tmKx), prefetch_tmap(&tmVx), prefetch_tmap(&tmDOx);
                prefetch_tmap(&tmQy), prefetch_tmap(&tmKy), prefetch_tmap(&tmVy), prefetch_tmap(&tmDOy);
            }
            BwdProducer<CK> pk;
            BwdProducer<CQ> pq;
            bool kv = false;
            for (int k = 0;; ++k) {
                // Taken when the loads of the item before are all under way: its
                // last tiles hide the counter's latency, and nothing is held
                // by an SM that will not come to it soon.
                const int i = atomicAdd(a.next, 1);
                if (!c.wait1(2 + (k & 1), ((uint32_t)(k >> 1) & 1u) ^ 1u)) break;
                slot[k & 1] = i;
                mbar_arrive(c.bar(k & 1));
                if (i >= a.items) break;
                if (i < a.kv_items) {
                    const BwdItem it = bwd_item<true, BN>(a, i);
                    kv = true;
                    if (!pk.template item<DK, DV, true>(c, a, it, K::BAR_KV, &tmKx, &tmVx, &tmQy, &tmDOy)) break;
                } else {
                    // dQ lays shared memory out anew: every product of dK and
                    // dV must be done with it.  (The end of the last walk
                    // would not do: this lane may be two walks ahead, which
                    // the parity of a wait cannot tell.)
                    if (kv && !c.wait1(K::BAR_KVEND, 0)) break;
                    kv = false;
                    const BwdItem it = bwd_item<false, BN>(a, i);
                    if (!pq.template item<DK, DV, false>(c, a, it, K::BAR_Q, &tmQx, &tmDOx, &tmKy, &tmVy)) break;
                }
            }
            if (*c.abort_flag) {
                pk.drain(c, K::BAR_KV);
                pq.drain(c, K::BAR_Q);
            }
        }
    } else if (warp == 1) {
        BwdIssuer<DK, DV, true, CK> ik;
        BwdIssuer<DK, DV, false, CQ> iq;
        bool kv = false;
        for (int k = 0, i; (i = take(k)) >= 0; ++k) {
            if (i < a.kv_items) {
                kv = true;
                if (!ik.item(c, bwd_item<true, BN>(a, i).n, K::BAR_KV, K::BAR_DONE)) break;
            } else {
                if (kv) mma_commit_warp(c.bar(K::BAR_KVEND));
                kv = false;
                if (!iq.item(c, bwd_item<false, BN>(a, i).n, K::BAR_Q, K::BAR_DONE)) break;
            }
        }
        // Nothing of ours may still run on the tensor core once TMEM is freed.
        mma_commit_warp(c.bar(K::BAR_END));
        mbar_wait_drain(c.bar(K::BAR_END), 0);
        __syncwarp();
    } else if (warp == 2) {
        if (a.gsinks) sink_gradients(a, lane);
    } else if (warp >= 4) {
        // All of dK / dV, then all of dQ (the list's order).
        uint32_t dones = 0;
        int k = 0, i = take(0);
        bool ok = true;
        if (i >= 0 && i < a.kv_items) {
            BwdWorker<DK, DV, true, MODS, CK> w;
            while (ok && i >= 0 && i < a.kv_items) {
                ok = w.item(c, a, i, K::BAR_KV, K::BAR_DONE, dones);
                if (ok) i = take(++k);
            }
            // dQ's dS may lie where dK and dV were: every warp must have read them.
            if (ok && i >= 0) {
                w.arrive(c, K::BAR_MOVED, lane);
                ok = c.wait(K::BAR_MOVED, 0);
            }
        }
        BwdWorker<DK, DV, false, MODS, CQ> w;
        while (ok && i >= 0) {
            ok = w.item(c, a, i, K::BAR_Q, K::BAR_DONE, dones);
            if (ok) i = take(++k);
        }
        if (MODS) cp_async_wait<0>();  // (after an abort)
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(c.tmem, 512);
    }
}

// Sums the parts of walks that were cut: a block takes 16 columns of 128 rows,
// first of dK and dV, then of dQ, in four groups of threads that share the
// parts out; the order of the additions is fixed.
template <int DK, int DV>
__global__ void __launch_bounds__(512) bwd_join_kernel(const BwdArgs a, int kv_blocks) {
    constexpr int BN = bwd_walk(DK);
    __shared__ float4 others[3][4][128];
    const int row = threadIdx.x & 127, group = threadIdx.x >> 7;
    const auto join = [&](auto kv, int block) {
        constexpr bool KV = decltype(kv)::value;
        constexpr int ACC = KV ? DK + DV : DK;
        const int tile = block / (ACC / 16), col = block % (ACC / 16) * 16;
        const unsigned per = (unsigned)(a.B * (KV ? a.Hkv : a.Hq));
        const int parts = KV ? a.kv_parts : a.q_parts, len = KV ? a.kv_len : a.q_len;
        // the tile's first part; the others follow `per` items apart (a tile
        // that sees nothing has none, and gets zeros)
        const unsigned first = (unsigned)tile / per * (unsigned)parts * per + (unsigned)tile % per;
        const BwdItem it = bwd_tile<KV, BN>(a, (int)((unsigned)tile / per), (int)((unsigned)tile % per));
        const int n = (it.whole + len - 1) / len;
        const float4 *from = reinterpret_cast<const float4 *>(KV ? a.kv_part : a.q_part) + col / 4 * 128 + row;
        float4 s[4] = {};
#pragma unroll 2
        for (int p = group; p < n; p += 4) {
            const float4 *f = from + (int64_t)(first + (unsigned)p * per) * (32 * ACC);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = __ldcg(f + i * 128);
                s[i].x += v.x, s[i].y += v.y, s[i].z += v.z, s[i].w += v.w;
            }
        }
        if (group > 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) others[group - 1][i][row] = s[i];
        __syncthreads();
        const int S = KV ? a.Sk : a.Sq;
        if (group > 0 || it.x0 + row >= S) return;
        const bool second = col >= DK;
        const float f = second ? 1.f : a.scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int g = 0; g < 3; ++g) {
                const float4 v = others[g][i][row];
                s[i].x += v.x, s[i].y += v.y, s[i].z += v.z, s[i].w += v.w;
            }
            s[i].x *= f, s[i].y *= f, s[i].z *= f, s[i].w *= f;
        }
        const BwdGrad &g = KV ? (second ? a.gv : a.gk) : a.gq;
        const int64_t at = (int64_t)it.b * g.sb + (int64_t)it.h * g.sh + (int64_t)(it.x0 + row) * g.ss + (second ? col - DK : col);
        if (a.g_bf16) {
            uint4 *to = reinterpret_cast<uint4 *>(g.p + 2 * at);
#pragma unroll
            for (int i = 0; i < 4; i += 2)
                to[i / 2] = make_uint4(pack_bf16x2(s[i].x, s[i].y), pack_bf16x2(s[i].z, s[i].w),
                                       pack_bf16x2(s[i + 1].x, s[i + 1].y), pack_bf16x2(s[i + 1].z, s[i + 1].w));
        } else {
            float4 *to = reinterpret_cast<float4 *>(g.p + 4 * at);
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = s[i];
        }
    };
    if ((int)blockIdx.x < kv_blocks)
        join(std::true_type{}, (int)blockIdx.x);
    else
        join(std::false_type{}, (int)blockIdx.x - kv_blocks);
}

// D and LSE of every row, DV / 8 lanes a row.  A block takes kPrepRows rows of
// one head: each thread has the loads of all its rows under way before the
// first is used.  (9.7 us for 2 x 16 x 2048 rows of 128 bf16 values, 3.5 TB/s:
// one wave of blocks, mostly its start and end.)
constexpr int kPrepRows = 64;
struct PrepArgs {
    const void *o;
    const __nv_bfloat16 *dout;
    const float *lse, *dlse;
    int64_t o_sb, o_sh, o_ss, do_sb, do_sh, do_ss;
    int Hq, Sq, o_bf16;
    int blocks;  // of kPrepRows rows, for each head
    float *nlse, *ndelta;
    uint4 *ext;  // NULL: not wanted
    float inv_scale;
    int *next;  // set to 0
};

// A value as three bf16 that add up to its 24 bits.
FA_DEV void split3(float v, uint16_t (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        p[i] = __bfloat16_as_ushort(h);
        v -= __bfloat162float(h);
    }
}

FA_DEV float dot8(const uint4 &w, const float (&o)[8]) {
    const uint32_t g[4] = {w.x, w.y, w.z, w.w};
    float d = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        d = fmaf(__uint_as_float(g[j] << 16), o[2 * j], d);
        d = fmaf(__uint_as_float(g[j] & 0xffff0000u), o[2 * j + 1], d);
    }
    return d;
}

template <int DV, bool O_BF16>
__global__ void __launch_bounds__(256) bwd_prep_kernel(const PrepArgs a) {
    constexpr int LPR = DV / 8;                    // lanes of a row
    constexpr int N = kPrepRows * LPR / 256;       // rows of a thread
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.next = 0;
    if (a.blocks == 0) return;
    const int bh = (int)(blockIdx.x / (unsigned)a.blocks), r0 = (int)(blockIdx.x % (unsigned)a.blocks) * kPrepRows;
    const int b = bh / a.Hq, h = bh % a.Hq;
    const int l = threadIdx.x % LPR, first = r0 + threadIdx.x / LPR;
    const __nv_bfloat16 *g = a.dout + b * a.do_sb + h * a.do_sh + 8 * l;
    const int64_t ob = b * a.o_sb + h * a.o_sh + 8 * l;
    uint4 w[N], u[N];
    [[maybe_unused]] uint4 v[O_BF16 ? 1 : N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int i = min(first + k * (256 / LPR), a.Sq - 1);
        w[k] = __ldg(reinterpret_cast<const uint4 *>(g + i * a.do_ss));
        if constexpr (O_BF16) {
            u[k] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.o) + ob + i * a.o_ss));
        } else {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(a.o) + ob + i * a.o_ss);
            u[k] = __ldg(p);
            v[k] = __ldg(p + 1);
        }
    }
    // Lane k of a row's lanes keeps the sum of the thread's k-th row.
    float d = 0.f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float o[8];
        if constexpr (O_BF16) {
            const uint32_t t[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[2 * j] = __uint_as_float(t[j] << 16), o[2 * j + 1] = __uint_as_float(t[j] & 0xffff0000u);
        } else {
            o[0] = __uint_as_float(u[k].x), o[1] = __uint_as_float(u[k].y);
            o[2] = __uint_as_float(u[k].z), o[3] = __uint_as_float(u[k].w);
            o[4] = __uint_as_float(v[k].x), o[5] = __uint_as_float(v[k].y);
            o[6] = __uint_as_float(v[k].z), o[7] = __uint_as_float(v[k].w);
        }
        float s = dot8(w[k], o);
#pragma unroll
        for (int x = LPR / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        if (l == k) d = s;
    }
    if (l < N) {
        const int i = first + l * (256 / LPR);
        const int64_t r = (int64_t)bh * a.blocks * kPrepRows + i;
        float lse = INFINITY;
        if (i < a.Sq) {
            const int64_t at = (int64_t)bh * a.Sq + i;
            lse = a.lse[at];
            if (a.dlse && lse != -INFINITY) d -= a.dlse[at];
            lse = lse == -INFINITY ? INFINITY : lse;
        } else {
            d = 0.f;
        }
        a.nlse[r] = -lse;
        a.ndelta[r] = -d;
        if (a.ext) {
            // In units of q.k; a row that sees nothing gets bf16's lowest
            // value, which takes any finite score far below the exponential's
            // range (an infinity would leave NaN in the split).
            uint16_t s[3] = {0xff7fu, 0, 0}, e[3];
            if (lse != INFINITY) split3(-lse * a.inv_scale, s);
            split3(-d, e);
            a.ext[r] = make_uint4(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)e[0] << 16, e[1] | (uint32_t)e[2] << 16, 0);
        }
    }
}

template <int DK, int DV, bool MODS>
cudaError_t launch_tiles(const BwdLaunch &L, const BwdArgs &a, int num_sms, cudaStream_t stream) {
    using K = BwdKernel<DK, DV, MODS>;
    auto kern = bwd_tile_kernel<DK, DV, MODS>;
    // The kernel's shared-memory limit, once a device (a call costs 1 us).
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(set.load(std::memory_order_relaxed) & bit) || !bit) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, K::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_relaxed);
    }
    int grid = a.items < num_sms ? a.items : num_sms;
    if (grid == 0 && a.gsinks) grid = 1;
    if (grid == 0) return cudaSuccess;
    // Starts under the row kernel's end and waits for it on the device.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(K::THREADS);
    cfg.dynamicSmemBytes = K::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, L.tmQx, L.tmKx, L.tmVx, L.tmDOx, L.tmQy, L.tmKy, L.tmVy, L.tmDOy, a);
    if (e != cudaSuccess || a.kv_len + a.q_len == 0) return e;
    const int kv = a.kv_len ? a.kv_items / a.kv_parts * ((DK + DV) / 16) : 0;
    const int q = a.q_len ? a.B * a.Hq * ((a.Sq + 127) / 128) * (DK / 16) : 0;
    bwd_join_kernel<DK, DV><<<kv + q, 512, 0, stream>>>(a, kv);
    return cudaGetLastError();
}

}  // namespace

// Estimates in units of a tile's time (1.3 to 2 us): an item's fill, drain and
// epilogue cost kItem tiles more, a launch of the join kernel kJoin.
constexpr double kSms = 148, kItem = 2, kJoin = 3.5;

// When the last SM is done with `nk` items of length `k` and then `nq` of
// length `q`, each taken by whoever is free.
double bwd_makespan(double nk, double k, double nq, double q) {
    const double rounds = floor(nk / kSms), more = nk - rounds * kSms;  // SMs with one item more
    const double t0 = rounds * k, t1 = t0 + k;
    double t = (nk * k + nq * q) / kSms;
    if (t < t0) t = t0;
    if (more > 0 && t < t1) t = t1;
    while (nq > 0 && more * floor(fmax(t - t1, 0) / q) + (kSms - more) * floor((t - t0) / q) < nq) t += 1;
    return t;
}

// A walk that is longer than an SM's even share of all tiles ends last, alone:
// few KV heads with many queries, few queries with many keys.  Such walks are
// cut into parts of the length with the least estimate, or left whole if that
// is less.  Measured, cut and whole: 7 heads on 1, 4000 queries, 40 keys, 128
// wide: 28.8 and 381 us; 8 on 1, 1024 x 1024, causal: 28.7 and 117; 8 heads,
// 16 x 4096: 24.6 and 57; 1 head, 4096 x 4096, causal: 38.6 and 63.5; but 8
// heads, 1024 x 1024, causal (walks of 8, a share of 3.5): 28.5 and 24.5, so
// left whole.
BwdSplit bwd_split(int B, int Hq, int Hkv, int Sq, int Sk, int dk, int dv, int causal) {
    BwdSplit s = {0, 1, 0, 1, 0, 0};
    if (B <= 0 || Sq <= 0 || Sk <= 0) return s;
    const int64_t BN = bwd_walk(dk), nk = (int64_t)B * Hkv * ((Sk + 127) / 128), nq = (int64_t)B * Hq * ((Sq + 127) / 128);
    const int64_t nq_live = causal && Sq > Sk ? nq - (int64_t)B * Hq * ((Sq - Sk) / 128) : nq;
    const double room = fmax(256e6, 4.0 * B * ((double)Hq * Sq * dk + (double)Hkv * Sk * (dk + dv)));
    // The longest walks, and how long the mean one is beside it.
    const int64_t kv = Hq / Hkv * ((Sq + BN - 1) / BN - (causal && Sq > Sk ? (Sq - Sk) / BN : 0));
    const int64_t q = (Sk + BN - 1) / BN;
    const double kv_mean = !causal ? 1 : Sk >= Sq ? 1 - 0.5 * Sq / Sk : 0.5;
    const double q_mean = !causal ? 1 : Sk >= Sq ? 1 - 0.5 * Sq / Sk : 0.5 * Sk / Sq;
    const double kv_tiles = kv_mean * (double)nk * (double)kv, q_tiles = q_mean * (double)nq * (double)q;
    const double share = (kv_tiles + q_tiles) / kSms;
    const int64_t longest = kv > q ? kv : q;
    if ((double)longest <= share + kJoin) return s;
    double best = fmax((double)longest + kItem, share + kItem * (double)(nk + nq) / kSms);
    for (int64_t len = 2; len < longest && (double)len < 2 * share + 8; len += len < 8 ? 1 : len / 4) {
        // parts of even length; under a causal mask the mean walk ends half a part early
        const int64_t pk = (kv + len - 1) / len, lk = (kv + pk - 1) / pk, pq = (q + len - 1) / len, lq = (q + pq - 1) / pq;
        if (512 * ((pk > 1 ? (double)(nk * pk) * (dk + dv) : 0) + (pq > 1 ? (double)(nq_live * pq) * dk : 0)) > room) continue;
        const double ck = pk == 1 ? nk : ceil(causal ? kv_tiles / (double)lk + 0.5 * nk : (double)(nk * pk));
        const double cq = pq == 1 ? nq : ceil(causal ? q_tiles / (double)lq + 0.5 * nq_live : (double)(nq * pq));
        if (kJoin + share + kItem * (ck + cq) / kSms >= best) continue;  // the even share alone
        const double t = kJoin + fmax((double)(lk > lq ? lk : lq) + kItem,
                                      bwd_makespan(ck, kv_tiles / ck + kItem, cq, q_tiles / cq + kItem));
        if (t >= best) continue;
        best = t;
        s.kv_len = pk == 1 ? 0 : (int)lk, s.kv_parts = (int)pk, s.kv_chunks = pk == 1 ? 0 : nk * pk;
        s.q_len = pq == 1 ? 0 : (int)lq, s.q_parts = (int)pq, s.q_chunks = pq == 1 ? 0 : nq_live * pq;
    }
    return s;
}

cudaError_t launch_bwd(const BwdLaunch &L, int num_sms, cudaStream_t stream) {
    const int64_t pitch = bwd_pitch(L.Sq);
    {
        PrepArgs p;
        p.o = L.o, p.dout = static_cast<const __nv_bfloat16 *>(L.dout), p.lse = L.lse, p.dlse = L.dlse;
        p.o_sb = L.o_sb, p.o_sh = L.o_sh, p.o_ss = L.o_ss;
        p.do_sb = L.do_sb, p.do_sh = L.do_sh, p.do_ss = L.do_ss;
        p.Hq = L.Hq, p.Sq = L.Sq;
        p.blocks = (int)(pitch / kPrepRows);
        p.nlse = L.nlse, p.ndelta = L.ndelta;
        p.ext = L.has_mods ? nullptr : static_cast<uint4 *>(L.ext), p.inv_scale = 1.f / L.scale;
        p.next = L.next;
        unsigned grid = (unsigned)(L.B * L.Hq) * (unsigned)p.blocks;
        if (grid == 0) grid = 1, p.blocks = 0;  // the counter alone
        if (L.dv == 64)
            L.o_bf16 ? bwd_prep_kernel<64, true><<<grid, 256, 0, stream>>>(p)
                     : bwd_prep_kernel<64, false><<<grid, 256, 0, stream>>>(p);
        else
            L.o_bf16 ? bwd_prep_kernel<128, true><<<grid, 256, 0, stream>>>(p)
                     : bwd_prep_kernel<128, false><<<grid, 256, 0, stream>>>(p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    BwdArgs a = {};
    a.B = L.B, a.Hq = L.Hq, a.Hkv = L.Hkv, a.Sq = L.Sq, a.Sk = L.Sk, a.causal = L.causal;
    a.scale_log2 = L.scale * kLog2e, a.cap_scale = L.scale;
    a.mods = L.mods;
    a.scale = L.mods.softcap > 0.f ? 4.f * (L.mods.softcap * L.scale) : L.scale;
    a.nlse = L.nlse, a.ndelta = L.ndelta, a.ext = static_cast<const uint4 *>(L.ext), a.pitch = pitch;
    const BwdSplit cut = bwd_split(L.B, L.Hq, L.Hkv, L.Sq, L.Sk, L.dk, L.dv, L.causal);
    a.kv_len = cut.kv_len, a.kv_parts = cut.kv_parts, a.q_len = cut.q_len, a.q_parts = cut.q_parts;
    a.kv_part = L.part, a.q_part = L.part + cut.kv_chunks * 128 * (L.dk + L.dv);
    a.kv_items = L.B * L.Hkv * ((L.Sk + 127) / 128) * cut.kv_parts;
    a.items = a.kv_items + (cut.q_len ? (int)cut.q_chunks : L.B * L.Hq * ((L.Sq + 127) / 128));
    a.next = L.next;
    a.gq = BwdGrad{static_cast<char *>(L.gq), L.gq_sb, L.gq_sh, L.gq_ss};
    a.gk = BwdGrad{static_cast<char *>(L.gk), L.gk_sb, L.gk_sh, L.gk_ss};
    a.gv = BwdGrad{static_cast<char *>(L.gv), L.gv_sb, L.gv_sh, L.gv_ss};
    a.g_bf16 = L.g_bf16;
    a.gsinks = L.gsinks;
#define FA_BWD_PAIR(DK_, DV_) \
    (L.has_mods ? launch_tiles<DK_, DV_, true>(L, a, num_sms, stream) : launch_tiles<DK_, DV_, false>(L, a, num_sms, stream))
    cudaError_t e = cudaErrorInvalidValue;
    if (L.dk == 64 && L.dv == 64) e = FA_BWD_PAIR(64, 64);
    if (L.dk == 128 && L.dv == 128) e = FA_BWD_PAIR(128, 128);
    if (L.dk == 192 && L.dv == 128) e = FA_BWD_PAIR(192, 128);
#undef FA_BWD_PAIR
    return e;
}

cudaError_t bwd_device_error(int clear, int *code) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_bwd_err, sizeof(int));
    if (e != cudaSuccess) return e;
    *code = v;
    if (clear && v) {
        v = 0;
        e = cudaMemcpyToSymbol(g_bwd_err, &v, sizeof(int));
    }
    return e;
}

}  // namespace fa
