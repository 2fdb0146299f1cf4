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
// Three kernels on the caller's stream:
//   1. bwd_prep_kernel: D and the LSE in base 2, one pass over O and dO.
//      Rows with no visible key (LSE -inf) and the padding up to a whole
//      128-row tile get LSE +inf, which makes every P of the row exactly 0.
//   2. bwd_tile_kernel<..., true>: dK and dV.  A CTA owns 128 keys of one KV
//      head and walks the query tiles of every head of its group, so the sum
//      over the group's heads stays in its accumulators.
//   3. bwd_tile_kernel<..., false>: dQ.  A CTA owns 128 queries of one head
//      and walks the key tiles.
// Scores and dO V^T are formed in both 2 and 3: seven matrix products where
// five would do, but no sum crosses CTAs, so nothing is accumulated with
// atomics in HBM and the result does not depend on timing.
//
// Both walks are one kernel.  Its 128 resident rows X1, X2 (K and V; or Q and
// dO) meet tiles of BN rows Y1, Y2 (Q and dO; or K and V):
//
//   S = X1 Y1^T,  T = X2 Y2^T       (128 x BN each, fp32 in TMEM)
//   A1 += dS Y1,  and for dK / dV A2 += P Y2
//
// so for dK and dV the tile is transposed: lanes are keys, columns queries.
//   warp 0      TMA producer: X1, X2 once, then rings of Y1 (with the LSE and
//               D of its rows) and Y2 tiles.
//   warp 1      MMA issuer (whole warp, one elected lane issues).
//   warps 4 ..  BN / 32 warpgroups, each 32 of the tile's columns: P from S,
//               then dS from P and T, both as bf16 A operands in TMEM, so that
//               those products read only Y from shared memory.
// BN is 128 where TMEM allows: a 128 x 64 product whose operands are both in
// shared memory reads 6 KB in its 32 cycles and takes 48 (measured), one of
// 128 x 128 8 KB in 64; and the issuer has half as many steps to take.
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "internal.h"
#include "score_mods.cuh"
#include "sm100.cuh"

namespace fa {
namespace {

__device__ int g_bwd_err;

struct BwdArgs {
    int Hq, Hkv, Sq, Sk, causal;
    float scale, scale_log2;
    ScoreMods mods;
    const float *nlse2, *ndelta;  // -LSE in base 2 and -D of every row
    const uint4 *ext;             // the two of a row as the B side of the extra step (see BwdCfg)
    int64_t pitch;                // rows per (batch, head) of the three
    int outer;      // 128-row tiles of the resident side
    char *g1, *g2;  // dK and dV, or dQ
    int64_t g1_sb, g1_sh, g1_ss, g2_sb, g2_sh, g2_ss;
    int g_bf16;
};

// Shared and tensor memory of one walk.  TMEM holds the accumulators and one
// S and one T tile.  Where there is room P and dS get columns of their own, so
// that S and T are free as soon as they are read, and after that the resident
// operands: an operand in TMEM saves its reads of shared memory, which at 8 KB
// a product of 64 cycles are all that memory gives.
template <int DK, int DV, bool KV, bool MODS>
struct BwdCfg {
    static constexpr int BN = bwd_walk(DK);
    // dK / dV without modifiers: LSE and D enter the products as one more
    // step of 16 columns.
    static constexpr bool EXT = KV && !MODS;
    static constexpr int NST1 = DK == 64 ? 4 : KV ? 2 : 3, NST2 = DK == 64 ? 4 : 2;  // stages of Y1 and of Y2
    static constexpr int X_CHUNK = 128 * 128, Y_CHUNK = BN * 128;  // bytes of a 64-column chunk
    static constexpr int X1_BYTES = 128 * DK * 2, X2_BYTES = 128 * DV * 2;
    static constexpr int Y1_BYTES = BN * DK * 2, Y2_BYTES = BN * DV * 2;
    static constexpr int EXT_A = EXT ? 2 * 128 * 16 : 0;  // ones beside zeros, for S; then for T
    static constexpr int ROW_BYTES = EXT ? 2 * BN * 16 : KV ? 2 * BN * 4 : 0;  // LSE and D of a query tile
    static constexpr int OFF_ROW = 2 * EXT_A;
    static constexpr int OFF_X1 = (OFF_ROW + NST1 * ROW_BYTES + 1023) / 1024 * 1024;
    static constexpr int OFF_X2 = OFF_X1 + X1_BYTES;
    // The last stage of Y1 may lie where the operand was that moved to TMEM.
    static constexpr bool REUSE = !KV && DK > 64;
    static constexpr int X2_ROOM = REUSE && DK == 192 ? Y1_BYTES : X2_BYTES;
    static constexpr int OFF_Y1 = OFF_X2 + X2_ROOM;
    static constexpr int OFF_Y2 = OFF_Y1 + (NST1 - REUSE) * Y1_BYTES;
    static constexpr int OFF_BAR = OFF_Y2 + NST2 * Y2_BYTES;
    static constexpr int SMEM_BYTES = OFF_BAR + 256 + 1024;  // barriers + alignment slack
    FA_DEV static uint32_t y1(int s) {  // offset of stage s
        return REUSE && s == NST1 - 1 ? (DK == 192 ? OFF_X2 : OFF_X1) : OFF_Y1 + s * Y1_BYTES;
    }
    static constexpr int WARPS = BN / 8;            // of elementwise work: four for 32 columns
    static constexpr int THREADS = 128 + 32 * WARPS;
    static constexpr int TMEM_COLS = 512;
    static constexpr int ACC = DK + (KV ? DV : 0);
    static constexpr int OWN = (KV ? BN : BN / 2);  // columns of separate P and dS
    static constexpr bool ALIAS = ACC + 2 * BN + OWN > TMEM_COLS;
    static constexpr int T_A1 = 0, T_A2 = DK, T_S = ACC, T_T = T_S + BN;
    // P over S and dS over T (each warpgroup in its own columns), or apart
    static constexpr int WG_COLS = ALIAS ? 32 : 16;  // from one warpgroup's P or dS to the next
    static constexpr int T_P = ALIAS ? T_S : T_T + BN;
    static constexpr int T_D = ALIAS ? T_T : T_T + BN + (KV ? BN / 2 : 0);
    static constexpr int T_X = ALIAS ? T_T + BN : T_D + BN / 2;
    static constexpr bool X1_TMEM = T_X + DK / 2 <= TMEM_COLS;
    static constexpr int T_X2 = T_X + (X1_TMEM ? DK / 2 : 0);
    static constexpr bool X2_TMEM = T_X2 + DV / 2 <= TMEM_COLS;
    static constexpr bool X_TMEM = X1_TMEM || X2_TMEM;
    static_assert(T_X <= TMEM_COLS, "TMEM budget");
    static_assert(!REUSE || (DK == 192 ? X2_TMEM : X1_TMEM && X1_BYTES >= Y1_BYTES), "the reused operand is in TMEM");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

enum { B_XFULL, B_XTMEM, B_SFULL, B_TFULL, B_SREAD, B_TREAD, B_PREADY, B_DSREADY, B_DONE, B_RING };

// 64 columns of this thread's row of a swizzled chunk (128-byte rows) to 32
// TMEM columns.
FA_DEV void chunk_to_tmem(const uint8_t *chunk, int row, uint32_t taddr) {
    uint32_t r[32];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint4 w = *reinterpret_cast<const uint4 *>(chunk + row * 128 + ((j ^ (row & 7)) << 4));
        r[4 * j] = w.x, r[4 * j + 1] = w.y, r[4 * j + 2] = w.z, r[4 * j + 3] = w.w;
    }
    tmem_st32(taddr, r);
}

// Of every eight exponentials, this many go to the FMA pipe (exp2_poly2).
constexpr int kPolyOf8 = 2;

template <int DK, int DV, bool KV, bool MODS>
__global__ void __launch_bounds__(BwdCfg<DK, DV, KV, MODS>::THREADS, 1)
bwd_tile_kernel(const __grid_constant__ CUtensorMap tmX1, const __grid_constant__ CUtensorMap tmX2,
                const __grid_constant__ CUtensorMap tmY1, const __grid_constant__ CUtensorMap tmY2, const BwdArgs a) {
    using C = BwdCfg<DK, DV, KV, MODS>;
    constexpr int BN = C::BN, NST1 = C::NST1, NST2 = C::NST2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem), sX1 = sbase + C::OFF_X1, sX2 = sbase + C::OFF_X2, sY2 = sbase + C::OFF_Y2;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    auto full1 = [&](int s) { return bar(B_RING + s); };
    auto empty1 = [&](int s) { return bar(B_RING + NST1 + s); };
    auto full2 = [&](int s) { return bar(B_RING + 2 * NST1 + s); };
    auto empty2 = [&](int s) { return bar(B_RING + 2 * NST1 + NST2 + s); };
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 28);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    static_assert(B_RING + 2 * (NST1 + NST2) <= 28, "barrier slots");

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int group = a.Hq / a.Hkv;
    const int H = KV ? a.Hkv : a.Hq;
    // The tiles with the longest walks first: key tile 0 sees the most
    // queries, the last query tile the most keys.
    const int bh = (int)(blockIdx.x % (unsigned)(gridDim.x / a.outer));
    const int xt = KV ? (int)(blockIdx.x / (gridDim.x / a.outer)) : a.outer - 1 - (int)(blockIdx.x / (gridDim.x / a.outer));
    const int b = bh / H, h = bh % H;
    const int x0 = xt * 128;
    const int shift = a.Sk - a.Sq;  // causal: key j is visible to query i iff j <= i + shift
    // Walk: tiles y_first .. y_first + n_y - 1, for dK / dV once per head of
    // the group.
    int y_first = 0, n_y;
    if (KV) {
        if (a.causal) y_first = max(0, x0 - shift) / BN;
        n_y = max(0, (a.Sq + BN - 1) / BN - y_first);
    } else {
        int last = a.Sk;  // keys visible to the tile's last row
        if (a.causal) last = min(last, min(a.Sq, x0 + 128) + shift);
        n_y = last <= 0 ? 0 : (last + BN - 1) / BN;
    }
    const int n = KV ? n_y * group : n_y;

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_RING + 2 * (NST1 + NST2); ++i)
            mbar_init(bar(i), i == B_XTMEM || (i >= B_SREAD && i <= B_DSREADY) ? C::WARPS : 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (C::EXT) {
        // A side of the extra step: row = 1 in columns 0 .. 2 for S (the three
        // pieces of the LSE), 3 .. 5 for T (those of D); the second half of
        // its 16 columns, on both sides, is zeros.
        uint4 *e = reinterpret_cast<uint4 *>(smem);
        for (int i = threadIdx.x; i < 2 * C::EXT_A / 16; i += C::THREADS)
            e[i] = (i & 128) ? make_uint4(0, 0, 0, 0)
                   : i < 256 ? make_uint4(0x3f803f80u, 0x3f80u, 0, 0)
                             : make_uint4(0, 0x3f800000u, 0x3f803f80u, 0);
        for (int i = threadIdx.x; i < NST1 * BN; i += C::THREADS)
            reinterpret_cast<uint4 *>(smem + C::OFF_ROW + (i / BN) * C::ROW_BYTES)[BN + i % BN] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer --
        if (lane == 0 && n > 0) {
            prefetch_tmap(&tmX1);
            prefetch_tmap(&tmX2);
            prefetch_tmap(&tmY1);
            prefetch_tmap(&tmY2);
            mbar_arrive_expect_tx(bar(B_XFULL), C::X1_BYTES + C::X2_BYTES);
            for (int c = 0; c < DK / 64; ++c) tma_load_4d(sX1 + c * C::X_CHUNK, &tmX1, bar(B_XFULL), c * 64, x0, h, b);
            for (int c = 0; c < DV / 64; ++c) tma_load_4d(sX2 + c * C::X_CHUNK, &tmX2, bar(B_XFULL), c * 64, x0, h, b);
            int issued1 = 0, issued2 = 0, y = 0, hy = KV ? h * group : h / group;
            for (int t = 0; t < n; ++t) {
                const int s1 = t % NST1, s2 = t % NST2;
                const int y0 = (y_first + y) * BN;
                if (!mbar_wait(empty1(s1), ((uint32_t)(t / NST1) & 1u) ^ 1u, abort_flag, &g_bwd_err)) break;
                if (C::REUSE && t == NST1 - 1 && !mbar_wait(bar(B_XTMEM), 0, abort_flag, &g_bwd_err)) break;
                mbar_arrive_expect_tx(full1(s1), C::Y1_BYTES + (C::EXT ? C::ROW_BYTES / 2 : C::ROW_BYTES));
                for (int c = 0; c < DK / 64; ++c)
                    tma_load_4d(sbase + C::y1(s1) + c * C::Y_CHUNK, &tmY1, full1(s1), c * 64, y0, hy, b);
                if (KV) {
                    const int64_t row = ((int64_t)b * a.Hq + hy) * a.pitch + y0;
                    const uint32_t sr = sbase + C::OFF_ROW + s1 * C::ROW_BYTES;
                    if (C::EXT) {
                        bulk_load(sr, a.ext + row, BN * 16, full1(s1));
                    } else {
                        bulk_load(sr, a.nlse2 + row, BN * 4, full1(s1));
                        bulk_load(sr + BN * 4, a.ndelta + row, BN * 4, full1(s1));
                    }
                }
                issued1 = t + 1;
                if (!mbar_wait(empty2(s2), ((uint32_t)(t / NST2) & 1u) ^ 1u, abort_flag, &g_bwd_err)) break;
                mbar_arrive_expect_tx(full2(s2), C::Y2_BYTES);
                for (int c = 0; c < DV / 64; ++c)
                    tma_load_4d(sY2 + s2 * C::Y2_BYTES + c * C::Y_CHUNK, &tmY2, full2(s2), c * 64, y0, hy, b);
                issued2 = t + 1;
                if (++y == n_y) y = 0, ++hy;
            }
            if (*abort_flag) {
                mbar_wait_drain(bar(B_XFULL), 0);
                for (int t = max(0, issued1 - NST1); t < issued1; ++t)
                    mbar_wait_drain(full1(t % NST1), (uint32_t)(t / NST1) & 1u);
                for (int t = max(0, issued2 - NST2); t < issued2; ++t)
                    mbar_wait_drain(full2(t % NST2), (uint32_t)(t / NST2) & 1u);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------- MMA issuer --
        if (n > 0) {
            constexpr uint32_t id_st = idesc_bf16_f32(128, BN, false, false);
            auto wait = [&](uint32_t br, uint32_t parity) { return mbar_wait_warp(br, parity, abort_flag, &g_bwd_err); };
            // 128 x BN product over D columns of a resident operand and a
            // tile, both K-major.
            auto product = [&](uint32_t d, auto in_tmem, uint32_t xt_, uint32_t xs, uint32_t ys, int D) {
                const uint64_t x = sdesc_sw128(xs, 16, 1024), yd = sdesc_sw128(ys, 16, 1024);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint64_t yc = yd + (uint64_t)((c * C::Y_CHUNK) >> 4);
                    if constexpr (decltype(in_tmem)::value)
                        mma_ts4_warp<8, 2>(d, xt_ + c * 32, yc, id_st, c > 0);
                    else
                        mma_ss4_warp<2, 4, 6>(d, x + (uint64_t)((c * C::X_CHUNK) >> 4), yc, id_st, c > 0);
                }
            };
            // Accumulator += (P or dS) Y over the tile's BN rows.
            auto accumulate = [&](uint32_t d, uint32_t pa, uint32_t ys, uint32_t id, bool first) {
                const uint64_t yd = sdesc_sw128(ys, C::Y_CHUNK, 1024);
                mma_ts4at_warp<8, C::WG_COLS, C::WG_COLS + 8, 128>(d, pa, yd, id, !first);
                if constexpr (BN == 128)
                    mma_ts4at_warp<8, C::WG_COLS, C::WG_COLS + 8, 128>(d, pa + 2 * C::WG_COLS, yd + 512, id, 1);
                else
                    mma_ts2_warp<8, 128>(d, pa + 2 * C::WG_COLS, yd + 512, id, 1);
            };
            // The step that adds -LSE to S, or -D to T (Y1's stage holds both).
            auto extra = [&](uint32_t d, uint32_t off, int t) {
                if (C::EXT)
                    mma_ss_warp(d, sdesc_plain(sbase + off, 2048, 128),
                                sdesc_plain(sbase + C::OFF_ROW + (t % NST1) * C::ROW_BYTES, BN * 16, 128), id_st, 1);
            };
            auto issue_s = [&](int t) -> bool {
                const int s = t % NST1;
                if (!wait(full1(s), (uint32_t)(t / NST1) & 1u)) return false;
                if (!C::ALIAS && t > 0 && !wait(bar(B_SREAD), (uint32_t)(t - 1) & 1u)) return false;
                tc_fence_after();
                product(tmem + C::T_S, std::integral_constant<bool, C::X1_TMEM>{}, tmem + C::T_X, sX1, sbase + C::y1(s), DK);
                extra(tmem + C::T_S, 0, t);
                mma_commit_warp(bar(B_SFULL));
                return true;
            };
            auto issue_t = [&](int t) -> bool {
                const int s = t % NST2;
                if (!wait(full2(s), (uint32_t)(t / NST2) & 1u)) return false;
                if (!C::ALIAS && t > 0 && !wait(bar(B_TREAD), (uint32_t)(t - 1) & 1u)) return false;
                tc_fence_after();
                product(tmem + C::T_T, std::integral_constant<bool, C::X2_TMEM>{}, tmem + C::T_X2, sX2, sY2 + s * C::Y2_BYTES, DV);
                extra(tmem + C::T_T, C::EXT_A, t);
                mma_commit_warp(bar(B_TFULL));
                if (!KV) mma_commit_warp(empty2(s));
                return true;
            };
            bool ok = wait(bar(B_XFULL), 0);
            if (ok && C::X_TMEM) ok = wait(bar(B_XTMEM), 0);
            ok = ok && issue_s(0) && issue_t(0);
            for (int t = 0; ok && t < n; ++t) {
                const int s1 = t % NST1, s2 = t % NST2;
                const bool more = t + 1 < n;
                if (!C::ALIAS && more && !issue_s(t + 1)) break;
                if (KV) {
                    if (!wait(bar(B_PREADY), (uint32_t)t & 1u)) break;
                    tc_fence_after();
                    accumulate(tmem + C::T_A2, tmem + C::T_P, sY2 + s2 * C::Y2_BYTES,
                               idesc_bf16_f32(128, DV, false, true), t == 0);
                    mma_commit_warp(empty2(s2));
                }
                // In place of P and dS: behind the products that read them.
                if (C::ALIAS && more && !issue_s(t + 1)) break;
                if (!C::ALIAS && more && !issue_t(t + 1)) break;
                if (!wait(bar(B_DSREADY), (uint32_t)t & 1u)) break;
                tc_fence_after();
                accumulate(tmem + C::T_A1, tmem + C::T_D, sbase + C::y1(s1), idesc_bf16_f32(128, DK, false, true),
                           t == 0);
                mma_commit_warp(empty1(s1));
                if (C::ALIAS && more && !issue_t(t + 1)) break;
            }
            // Nothing of ours may still run on the tensor core once TMEM is
            // read out or freed.
            mma_commit_warp(bar(B_DONE));
            mbar_wait_drain(bar(B_DONE), 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // --------------------------------------------- P, dS, epilogue --
        const int wg = (warp >> 2) - 1;           // columns 32 wg .. 32 wg + 31 of each tile
        const int row = (warp & 3) * 32 + lane;   // resident row: key or query
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t tS = tl + C::T_S + wg * 32, tT = tl + C::T_T + wg * 32;
        const uint32_t tP = tl + C::T_P + wg * C::WG_COLS, tD = tl + C::T_D + wg * C::WG_COLS;
        const int xr = x0 + row;
        auto wait = [&](uint32_t br, uint32_t parity) { return mbar_wait_warp(br, parity, abort_flag, &g_bwd_err); };
        auto arrive = [&](int i) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(i));
        };
        const bool capped = MODS && a.mods.softcap != 0.f;
        const bool masked = MODS && a.mods.mask != nullptr;
        float row_nlse = 0.f, row_ndelta = 0.f;
        if (!KV) {  // rows past Sq are padded in the workspace
            const int64_t r = ((int64_t)b * a.Hq + h) * a.pitch + xr;
            row_nlse = __ldg(a.nlse2 + r);
            row_ndelta = __ldg(a.ndelta + r);
        }
        // dQ: columns c >= lim_hi - y0 of this row are hidden; dK / dV:
        // columns c < lim_lo - y0 of this key.
        const int lim_hi = a.causal ? min(a.Sk, xr + shift + 1) : a.Sk;
        const int lim_lo = a.causal ? xr - shift : 0;
        const uint64_t sc2 = f2_pack(a.scale_log2, a.scale_log2);
        bool ok = true;
        if (C::X_TMEM && n > 0) {
            ok = wait(bar(B_XFULL), 0);
            if (ok) {
                constexpr int N1 = C::X1_TMEM ? DK / 64 : 0, NC = N1 + (C::X2_TMEM ? DV / 64 : 0);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    if (c % (BN / 32) == wg)
                        chunk_to_tmem(c < N1 ? smem + C::OFF_X1 + c * C::X_CHUNK : smem + C::OFF_X2 + (c - N1) * C::X_CHUNK, row,
                                      tl + (uint32_t)(C::T_X + c * 32));
                }
                tmem_wait_st();
                arrive(B_XTMEM);
            }
        }
        int y = 0, hq = KV ? h * group : h;
        for (int t = 0; ok && t < n; ++t) {
            ok = false;
            const int s1 = t % NST1;
            const int y0 = (y_first + y) * BN + wg * 32;  // first column: query or key
            const float *sl = reinterpret_cast<const float *>(smem + C::OFF_ROW + s1 * C::ROW_BYTES) + wg * 32;
            if (KV && MODS && !wait(full1(s1), (uint32_t)(t / NST1) & 1u)) break;
            if (!wait(bar(B_SFULL), (uint32_t)t & 1u)) break;
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
            if (!C::ALIAS) arrive(B_SREAD);
            float cap[MODS ? 32 : 1];  // ds/dz under a softcap
            if constexpr (MODS) {
                const float slope = alibi_slope(a.mods, hq) * kLog2e;
                if (capped) {
                    const float inv = 1.f / (a.mods.softcap * kLog2e);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) softcap4(x + i, a.scale, a.mods.softcap);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float th = x[i] * inv;
                        cap[i] = fmaf(-th, th, 1.f) * a.mods.softcap;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] *= a.scale_log2;
                }
                if (masked) {
                    // Rows and keys past the end read the last one's values:
                    // their P is 0, or their results are not stored.
                    const __half *m = a.mods.mask + (int64_t)b * a.mods.m_sb + (int64_t)hq * a.mods.m_sh;
                    if (KV) {
                        m += min(xr, a.Sk - 1);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            x[i] = fmaf(__half2float(m[(int64_t)min(y0 + i, a.Sq - 1) * a.mods.m_ss]), slope, x[i]);
                    } else {
                        m += (int64_t)min(xr, a.Sq - 1) * a.mods.m_ss;
                        if (y0 + 32 <= a.Sk) {
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(m + y0 + i));
                                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[j]));
                                    x[i + 2 * j] = fmaf(f.x, slope, x[i + 2 * j]);
                                    x[i + 2 * j + 1] = fmaf(f.y, slope, x[i + 2 * j + 1]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                x[i] = fmaf(__half2float(m[min(y0 + i, a.Sk - 1)]), slope, x[i]);
                        }
                    }
                }
            }
            const bool edge = KV ? (a.causal && y0 < x0 + 127 - shift)
                                 : (y0 + 32 > min(a.Sk, a.causal ? x0 + shift + 1 : a.Sk));
            if (edge) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (KV ? (y0 + i < lim_lo) : (y0 + i >= lim_hi)) x[i] = -INFINITY;
            }
            // P
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                uint64_t nl[2];
                if (C::EXT) {
                    nl[0] = nl[1] = 0;
                } else if (KV) {
                    const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(sl + i);
                    nl[0] = l.x, nl[1] = l.y;
                } else {
                    nl[0] = nl[1] = f2_pack(row_nlse, row_nlse);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int k = i + 2 * j;
                    const uint64_t xx = f2_pack(x[k], x[k + 1]);
                    float e0, e1;
                    f2_unpack(C::EXT ? f2_mul(xx, sc2) : MODS ? f2_add(xx, nl[j]) : f2_fma(xx, sc2, nl[j]), e0, e1);
                    if (k % 8 < kPolyOf8) {
                        exp2_poly2(e0, e1, x[k], x[k + 1]);
                    } else {
                        x[k] = ex2(e0);
                        x[k + 1] = ex2(e1);
                    }
                    pk[k / 2] = pack_bf16x2(x[k], x[k + 1]);
                }
            }
            if (KV) {
                // With its own columns: the product over the P before is done.
                if (!C::ALIAS && t > 0 && !wait(empty2((t - 1) % NST2), (uint32_t)((t - 1) / NST2) & 1u)) break;
                tmem_st16(tP, pk);
                tmem_wait_st();
                arrive(B_PREADY);
            }
            if (MODS && capped) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] *= cap[i];
            }
            // dS
            if (!wait(bar(B_TFULL), (uint32_t)t & 1u)) break;
            tc_fence_after();
            uint32_t r[32];
            tmem_ld32(tT, r);
            tmem_wait_ld();
            reg_fence(r);
            if (!C::ALIAS) arrive(B_TREAD);
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
            if (!C::ALIAS && t > 0 && !wait(empty1((t - 1) % NST1), (uint32_t)((t - 1) / NST1) & 1u)) break;
            tmem_st16(tD, pk);
            tmem_wait_st();
            arrive(B_DSREADY);
            if (++y == n_y) y = 0, ++hq;
            ok = true;
        }
        bool have = ok && n > 0;
        if (have) {
            have = wait(bar(B_DONE), 0);
            tc_fence_after();
        }
        // 32 accumulator columns at a time, dealt to the warpgroups.
        const bool store = xr < (KV ? a.Sk : a.Sq);
        const int64_t off1 = (int64_t)b * a.g1_sb + (int64_t)h * a.g1_sh + (int64_t)xr * a.g1_ss;
        const int64_t off2 = (int64_t)b * a.g2_sb + (int64_t)h * a.g2_sh + (int64_t)xr * a.g2_ss;
        for (int c = wg * 32; c < C::ACC; c += BN) {
            const bool second = c >= DK;
            uint32_t r[32];
            if (have) {
                tmem_ld32(tl + (uint32_t)(C::T_A1 + c), r);
                tmem_wait_ld();
                reg_fence(r);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = 0u;
            }
            if (!store) continue;
            const float f = second ? 1.f : a.scale;
            const int64_t at = second ? off2 + c - DK : off1 + c;
            char *base = second ? a.g2 : a.g1;
            if (a.g_bf16) {
                uint4 *dst = reinterpret_cast<uint4 *>(base + 2 * at);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dst[i] = make_uint4(pack_bf16x2(__uint_as_float(r[8 * i]) * f, __uint_as_float(r[8 * i + 1]) * f),
                                        pack_bf16x2(__uint_as_float(r[8 * i + 2]) * f, __uint_as_float(r[8 * i + 3]) * f),
                                        pack_bf16x2(__uint_as_float(r[8 * i + 4]) * f, __uint_as_float(r[8 * i + 5]) * f),
                                        pack_bf16x2(__uint_as_float(r[8 * i + 6]) * f, __uint_as_float(r[8 * i + 7]) * f));
            } else {
                float4 *dst = reinterpret_cast<float4 *>(base + 4 * at);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dst[i] = make_float4(__uint_as_float(r[4 * i]) * f, __uint_as_float(r[4 * i + 1]) * f,
                                         __uint_as_float(r[4 * i + 2]) * f, __uint_as_float(r[4 * i + 3]) * f);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// D and base-2 LSE of every row, DV / 8 lanes a row.
struct PrepArgs {
    const void *o;
    const __nv_bfloat16 *dout;
    const float *lse, *dlse;
    int64_t o_sb, o_sh, o_ss, do_sb, do_sh, do_ss;
    int Hq, Sq, o_bf16;
    int64_t pitch, rows;  // rows = B * Hq * pitch
    float *nlse2, *ndelta;
    uint4 *ext;  // NULL: not wanted
    float inv_scale;
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

template <int DV>
__global__ void __launch_bounds__(256) bwd_prep_kernel(const PrepArgs a) {
    constexpr int LPR = DV / 8;  // lanes of a row
    const int64_t r = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int l = threadIdx.x % LPR;
    const int64_t bh = r / a.pitch;
    const int i = (int)(r % a.pitch), b = (int)(bh / a.Hq), h = (int)(bh % a.Hq);
    float d = 0.f;
    const bool live = r < a.rows && i < a.Sq;
    if (live) {
        const uint4 w = *reinterpret_cast<const uint4 *>(a.dout + b * a.do_sb + h * a.do_sh + i * a.do_ss + 8 * l);
        const uint32_t g[4] = {w.x, w.y, w.z, w.w};
        const int64_t off = b * a.o_sb + h * a.o_sh + i * a.o_ss + 8 * l;
        float o[8];
        if (a.o_bf16) {
            const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.o) + off);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[2 * j] = __uint_as_float(u[j] << 16), o[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        } else {
            const float4 *v = reinterpret_cast<const float4 *>(static_cast<const float *>(a.o) + off);
            const float4 p = v[0], q = v[1];
            o[0] = p.x, o[1] = p.y, o[2] = p.z, o[3] = p.w, o[4] = q.x, o[5] = q.y, o[6] = q.z, o[7] = q.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            d = fmaf(__uint_as_float(g[j] << 16), o[2 * j], d);
            d = fmaf(__uint_as_float(g[j] & 0xffff0000u), o[2 * j + 1], d);
        }
    }
#pragma unroll
    for (int k = LPR / 2; k > 0; k >>= 1) d += __shfl_xor_sync(0xffffffffu, d, k);
    if (l == 0 && r < a.rows) {
        float lse = INFINITY;
        if (live) {
            const int64_t at = bh * a.Sq + i;
            lse = a.lse[at];
            if (a.dlse && lse != -INFINITY) d -= a.dlse[at];
            lse = lse == -INFINITY ? INFINITY : lse;
        }
        a.nlse2[r] = -lse * kLog2e;
        a.ndelta[r] = -d;
        if (a.ext) {
            // In units of q.k; a row that sees nothing gets bf16's lowest
            // value, which takes any finite score far below the exponential's
            // range (an infinity would leave NaN in the split).
            uint16_t l[3] = {0xff7fu, 0, 0}, e[3];
            if (lse != INFINITY) split3(-lse * a.inv_scale, l);
            split3(-d, e);
            a.ext[r] = make_uint4(l[0] | (uint32_t)l[1] << 16, l[2] | (uint32_t)e[0] << 16, e[1] | (uint32_t)e[2] << 16, 0);
        }
    }
}

// dsink_h: one block a head, rows in a fixed order.
__global__ void __launch_bounds__(512) bwd_sink_kernel(const float *nlse2, const float *ndelta, int64_t pitch, int B,
                                                       int Hq, int Sq, const float *sinks, float *out) {
    __shared__ float part[16];
    const int h = blockIdx.x;
    const float sk = sinks[h] * kLog2e;
    float acc = 0.f;
    for (int b = 0; b < B; ++b) {
        const int64_t r = ((int64_t)b * Hq + h) * pitch;
        for (int i = threadIdx.x; i < Sq; i += 512) acc += ex2(sk + nlse2[r + i]) * ndelta[r + i];
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, k);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        float s = 0.f;
        for (int w = 0; w < 16; ++w) s += part[w];
        out[h] = s;
    }
}

template <int DK, int DV, bool KV, bool MODS>
cudaError_t launch_tiles(const BwdLaunch &L, BwdArgs a, cudaStream_t stream) {
    using C = BwdCfg<DK, DV, KV, MODS>;
    auto kern = bwd_tile_kernel<DK, DV, KV, MODS>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    a.outer = ((KV ? L.Sk : L.Sq) + 127) / 128;
    if (KV) {
        a.g1 = static_cast<char *>(L.gk), a.g1_sb = L.gk_sb, a.g1_sh = L.gk_sh, a.g1_ss = L.gk_ss;
        a.g2 = static_cast<char *>(L.gv), a.g2_sb = L.gv_sb, a.g2_sh = L.gv_sh, a.g2_ss = L.gv_ss;
    } else {
        a.g1 = static_cast<char *>(L.gq), a.g1_sb = L.gq_sb, a.g1_sh = L.gq_sh, a.g1_ss = L.gq_ss;
    }
    const unsigned grid = (unsigned)(L.B * (KV ? L.Hkv : L.Hq)) * (unsigned)a.outer;
    if (grid == 0) return cudaSuccess;
    if (KV)
        kern<<<grid, C::THREADS, C::SMEM_BYTES, stream>>>(L.tmKx, L.tmVx, L.tmQy, L.tmDOy, a);
    else
        kern<<<grid, C::THREADS, C::SMEM_BYTES, stream>>>(L.tmQx, L.tmDOx, L.tmKy, L.tmVy, a);
    return cudaGetLastError();
}

template <int DK, int DV, bool MODS>
cudaError_t launch_pair(const BwdLaunch &L, const BwdArgs &a, cudaStream_t stream) {
    cudaError_t e = launch_tiles<DK, DV, true, MODS>(L, a, stream);
    if (e == cudaSuccess) e = launch_tiles<DK, DV, false, MODS>(L, a, stream);
    return e;
}

}  // namespace

cudaError_t launch_bwd(const BwdLaunch &L, cudaStream_t stream) {
    const int64_t pitch = bwd_pitch(L.Sq);
    if (L.Sq > 0 && L.B > 0) {
        PrepArgs p;
        p.o = L.o, p.dout = static_cast<const __nv_bfloat16 *>(L.dout), p.lse = L.lse, p.dlse = L.dlse;
        p.o_sb = L.o_sb, p.o_sh = L.o_sh, p.o_ss = L.o_ss;
        p.do_sb = L.do_sb, p.do_sh = L.do_sh, p.do_ss = L.do_ss;
        p.Hq = L.Hq, p.Sq = L.Sq, p.o_bf16 = L.o_bf16;
        p.pitch = pitch, p.rows = (int64_t)L.B * L.Hq * pitch;
        p.nlse2 = L.nlse2, p.ndelta = L.ndelta;
        p.ext = L.has_mods ? nullptr : static_cast<uint4 *>(L.ext), p.inv_scale = 1.f / L.scale;
        const int per = 256 / (L.dv / 8);
        const unsigned grid = (unsigned)((p.rows + per - 1) / per);
        if (L.dv == 64)
            bwd_prep_kernel<64><<<grid, 256, 0, stream>>>(p);
        else
            bwd_prep_kernel<128><<<grid, 256, 0, stream>>>(p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (L.gsinks) {
        bwd_sink_kernel<<<L.Hq, 512, 0, stream>>>(L.nlse2, L.ndelta, pitch, L.B, L.Hq, L.Sq, L.mods.sinks, L.gsinks);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    BwdArgs a = {};
    a.Hq = L.Hq, a.Hkv = L.Hkv, a.Sq = L.Sq, a.Sk = L.Sk, a.causal = L.causal;
    a.scale = L.scale, a.scale_log2 = L.scale * kLog2e;
    a.mods = L.mods;
    a.nlse2 = L.nlse2, a.ndelta = L.ndelta, a.ext = static_cast<const uint4 *>(L.ext), a.pitch = pitch;
    a.g_bf16 = L.g_bf16;
#define FA_BWD_PAIR(DK_, DV_) \
    (L.has_mods ? launch_pair<DK_, DV_, true>(L, a, stream) : launch_pair<DK_, DV_, false>(L, a, stream))
    if (L.dk == 64 && L.dv == 64) return FA_BWD_PAIR(64, 64);
    if (L.dk == 128 && L.dv == 128) return FA_BWD_PAIR(128, 128);
    if (L.dk == 192 && L.dv == 128) return FA_BWD_PAIR(192, 128);
#undef FA_BWD_PAIR
    return cudaErrorInvalidValue;
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
