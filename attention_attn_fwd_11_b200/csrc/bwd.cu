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
// dO) meet tiles of 64 rows Y1, Y2 (Q and dO; or K and V):
//
//   S = X1 Y1^T,  T = X2 Y2^T       (128 x 64 each, fp32 in TMEM)
//   A1 += dS Y1,  and for dK / dV A2 += P Y2
//
// so for dK and dV the tile is transposed: lanes are keys, columns queries.
//   warp 0      TMA producer: X1, X2 once, then a ring of Y1, Y2 tiles (and
//               the LSE and D of their rows).
//   warp 1      MMA issuer (whole warp, one elected lane issues).
//   warps 4-11  two warpgroups, each 32 of the tile's 64 columns: S and T from
//               TMEM, P and dS as bf16 back into the S slot they came from.
// TMEM: A1 | A2 | S0 | S1 | T.  Two S slots let the next tile's products run
// under this tile's exponentials; T is one slot, free again as soon as the
// warpgroups have read it.  P and dS are A operands from TMEM, so those
// products read only Y from shared memory.
#include <cuda_runtime.h>
#include <math.h>

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
    const float *lse2, *delta;
    int64_t pitch;  // of lse2 and delta
    int outer;      // 128-row tiles of the resident side
    char *g1, *g2;  // dK and dV, or dQ
    int64_t g1_sb, g1_sh, g1_ss, g2_sb, g2_sh, g2_ss;
    int g_bf16;
};

template <int DK, int DV, bool KV, int NST>
struct BwdCfg {
    static constexpr int X_CHUNK = 128 * 128, Y_CHUNK = 64 * 128;  // bytes of a 64-column chunk
    static constexpr int X1_BYTES = 128 * DK * 2, X2_BYTES = 128 * DV * 2;
    static constexpr int Y1_BYTES = 64 * DK * 2, Y2_BYTES = 64 * DV * 2;
    static constexpr int ROW_BYTES = KV ? 512 : 0;  // LSE and D of a query tile
    static constexpr int OFF_X2 = X1_BYTES;
    static constexpr int OFF_Y = X1_BYTES + X2_BYTES;
    static constexpr int STAGE = Y1_BYTES + Y2_BYTES;
    static constexpr int OFF_ROW = OFF_Y + NST * STAGE;
    static constexpr int OFF_BAR = OFF_ROW + NST * ROW_BYTES;
    static constexpr int SMEM_BYTES = OFF_BAR + 256 + 1024;  // barriers + alignment slack
    static constexpr int T_A1 = 0, T_A2 = DK, T_S = DK + (KV ? DV : 0), T_T = T_S + 128;
    static constexpr int TMEM_COLS = 512;
    static_assert(T_T + 64 <= TMEM_COLS, "TMEM budget");
    static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

enum { B_XFULL = 0, B_STFULL = 1, B_TREAD = 2, B_DSREADY = 3, B_DONE = 5, B_RING = 6 };

template <int DK, int DV, bool KV, int NST, bool MODS>
__global__ void __launch_bounds__(384, 1)
bwd_tile_kernel(const __grid_constant__ CUtensorMap tmX1, const __grid_constant__ CUtensorMap tmX2,
                const __grid_constant__ CUtensorMap tmY1, const __grid_constant__ CUtensorMap tmY2, const BwdArgs a) {
    using C = BwdCfg<DK, DV, KV, NST>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sX1 = smem_u32(smem), sX2 = sX1 + C::OFF_X2, sY = sX1 + C::OFF_Y;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [&](int i) -> uint32_t { return bar0 + 8u * (uint32_t)i; };
    auto full = [&](int s) { return bar(B_RING + s); };
    auto empty = [&](int s) { return bar(B_RING + NST + s); };
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(bars + 24);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    static_assert(B_RING + 2 * NST <= 24, "barrier slots");

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
        if (a.causal) y_first = max(0, x0 - shift) / 64;
        n_y = max(0, (a.Sq + 63) / 64 - y_first);
    } else {
        int last = a.Sk;  // keys visible to the tile's last row
        if (a.causal) last = min(last, min(a.Sq, x0 + 128) + shift);
        n_y = last <= 0 ? 0 : (last + 63) / 64;
    }
    const int n = KV ? n_y * group : n_y;

    if (threadIdx.x == 0) {
        mbar_init(bar(B_XFULL), 1);
        mbar_init(bar(B_STFULL), 1);
        mbar_init(bar(B_TREAD), 8);
        mbar_init(bar(B_DSREADY), 8);
        mbar_init(bar(B_DSREADY + 1), 8);
        mbar_init(bar(B_DONE), 1);
        for (int s = 0; s < NST; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        *abort_flag = 0;
        fence_barrier_init();
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
            int issued = 0;
            for (int t = 0; t < n; ++t) {
                const int s = t % NST;
                if (!mbar_wait(empty(s), ((uint32_t)(t / NST) & 1u) ^ 1u, abort_flag, &g_bwd_err)) break;
                const int y0 = (y_first + t % n_y) * 64;
                const int hy = KV ? h * group + t / n_y : h / group;
                const uint32_t sy = sY + s * C::STAGE;
                mbar_arrive_expect_tx(full(s), C::STAGE + C::ROW_BYTES);
                for (int c = 0; c < DK / 64; ++c) tma_load_4d(sy + c * C::Y_CHUNK, &tmY1, full(s), c * 64, y0, hy, b);
                for (int c = 0; c < DV / 64; ++c)
                    tma_load_4d(sy + C::Y1_BYTES + c * C::Y_CHUNK, &tmY2, full(s), c * 64, y0, hy, b);
                if (KV) {
                    const int64_t row = ((int64_t)b * a.Hq + hy) * a.pitch + y0;
                    const uint32_t sr = sX1 + C::OFF_ROW + s * C::ROW_BYTES;
                    bulk_load(sr, a.lse2 + row, 256, full(s));
                    bulk_load(sr + 256, a.delta + row, 256, full(s));
                }
                issued = t + 1;
            }
            if (*abort_flag) {
                mbar_wait_drain(bar(B_XFULL), 0);
                for (int t = max(0, issued - NST); t < issued; ++t)
                    mbar_wait_drain(full(t % NST), (uint32_t)(t / NST) & 1u);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------- MMA issuer --
        if (n > 0) {
            constexpr uint32_t id_st = idesc_bf16_f32(128, 64, false, false);
            constexpr uint32_t id_a1 = idesc_bf16_f32(128, DK, false, true);
            constexpr uint32_t id_a2 = idesc_bf16_f32(128, DV, false, true);
            const uint64_t x1 = sdesc_sw128(sX1, 16, 1024), x2 = sdesc_sw128(sX2, 16, 1024);
            // S and T of tile t
            auto issue_st = [&](int t) -> bool {
                const int s = t % NST;
                if (!mbar_wait_warp(full(s), (uint32_t)(t / NST) & 1u, abort_flag, &g_bwd_err)) return false;
                tc_fence_after();
                const uint64_t y1 = sdesc_sw128(sY + s * C::STAGE, 16, 1024);
                const uint64_t y2 = sdesc_sw128(sY + s * C::STAGE + C::Y1_BYTES, 16, 1024);
#pragma unroll
                for (int c = 0; c < DK / 64; ++c)
                    mma_ss4_warp<2, 4, 6>(tmem + C::T_S + (t & 1) * 64, x1 + (uint64_t)((c * C::X_CHUNK) >> 4),
                                          y1 + (uint64_t)((c * C::Y_CHUNK) >> 4), id_st, c > 0);
                // T of the tile before must have been read
                if (t > 0 && !mbar_wait_warp(bar(B_TREAD), (uint32_t)(t - 1) & 1u, abort_flag, &g_bwd_err)) return false;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < DV / 64; ++c)
                    mma_ss4_warp<2, 4, 6>(tmem + C::T_T, x2 + (uint64_t)((c * C::X_CHUNK) >> 4),
                                          y2 + (uint64_t)((c * C::Y_CHUNK) >> 4), id_st, c > 0);
                mma_commit_warp(bar(B_STFULL));
                return true;
            };
            bool ok = mbar_wait_warp(bar(B_XFULL), 0, abort_flag, &g_bwd_err) && issue_st(0);
            for (int t = 0; ok && t < n; ++t) {
                if (t + 1 < n && !issue_st(t + 1)) break;
                if (!mbar_wait_warp(bar(B_DSREADY + (t & 1)), (uint32_t)(t >> 1) & 1u, abort_flag, &g_bwd_err)) break;
                tc_fence_after();
                const int s = t % NST;
                const uint32_t tP = tmem + C::T_S + (t & 1) * 64;
                if (KV)
                    mma_ts4at_warp<8, 32, 40, 128>(tmem + C::T_A2, tP,
                                                   sdesc_sw128(sY + s * C::STAGE + C::Y1_BYTES, C::Y_CHUNK, 1024), id_a2,
                                                   t > 0);
                mma_ts4at_warp<8, 32, 40, 128>(tmem + C::T_A1, tP + 16, sdesc_sw128(sY + s * C::STAGE, C::Y_CHUNK, 1024),
                                               id_a1, t > 0);
                mma_commit_warp(empty(s));
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
        const int xr = x0 + row;
        const bool capped = MODS && a.mods.softcap != 0.f;
        const bool masked = MODS && a.mods.mask != nullptr;
        float row_lse = 0.f, row_delta = 0.f;
        if (!KV) {  // rows past Sq are padded in the workspace
            const int64_t r = ((int64_t)b * a.Hq + h) * a.pitch + xr;
            row_lse = __ldg(a.lse2 + r);
            row_delta = __ldg(a.delta + r);
        }
        // dQ: columns c >= lim_hi - y0 of this row are hidden; dK / dV:
        // columns c < lim_lo - y0 of this key.
        const int lim_hi = a.causal ? min(a.Sk, xr + shift + 1) : a.Sk;
        const int lim_lo = a.causal ? xr - shift : 0;
        bool ok = true;
        for (int t = 0; t < n; ++t) {
            const int s = t % NST;
            if (KV && !mbar_wait_warp(full(s), (uint32_t)(t / NST) & 1u, abort_flag, &g_bwd_err)) {
                ok = false;
                break;
            }
            if (!mbar_wait_warp(bar(B_STFULL), (uint32_t)t & 1u, abort_flag, &g_bwd_err)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t slot = tl + (uint32_t)(C::T_S + (t & 1) * 64 + wg * 32);
            uint32_t sr[32], tr[32];
            tmem_ld32(slot, sr);
            tmem_ld32(tl + (uint32_t)(C::T_T + wg * 32), tr);
            tmem_wait_ld();
            reg_fence(sr);
            reg_fence(tr);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_TREAD));
            const int y0 = (y_first + t % n_y) * 64 + wg * 32;  // first column: query or key
            const int hq = KV ? h * group + t / n_y : h;
            const float *sl = reinterpret_cast<const float *>(smem + C::OFF_ROW + s * C::ROW_BYTES) + wg * 32;
            const bool edge = KV ? (a.causal && y0 < x0 + 127 - shift) : (y0 + 32 > min(a.Sk, a.causal ? x0 + shift + 1 : a.Sk));
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(sr[i]);
            float cap[32];  // ds/dz / softcap under a softcap
            (void)cap;
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
                    const __half *m = a.mods.mask + (int64_t)b * a.mods.m_sb + (int64_t)hq * a.mods.m_sh;
                    if (KV) {
                        if (xr < a.Sk) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (y0 + i < a.Sq)
                                    x[i] = fmaf(__half2float(m[(int64_t)(y0 + i) * a.mods.m_ss + xr]), slope, x[i]);
                        }
                    } else if (xr < a.Sq) {
                        const __half *mr = m + (int64_t)xr * a.mods.m_ss + y0;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (y0 + i < a.Sk) x[i] = fmaf(__half2float(mr[i]), slope, x[i]);
                    }
                }
            }
            if (edge) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (KV ? (y0 + i < lim_lo) : (y0 + i >= lim_hi)) x[i] = -INFINITY;
            }
            uint32_t pp[16], dd[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                float4 l4, d4;
                if (KV) {
                    l4 = *reinterpret_cast<const float4 *>(sl + i);
                    d4 = *reinterpret_cast<const float4 *>(sl + 64 + i);
                } else {
                    l4 = make_float4(row_lse, row_lse, row_lse, row_lse);
                    d4 = make_float4(row_delta, row_delta, row_delta, row_delta);
                }
                const float lv[4] = {l4.x, l4.y, l4.z, l4.w}, dv[4] = {d4.x, d4.y, d4.z, d4.w};
                float p[4], ds[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = MODS ? x[i + j] - lv[j] : fmaf(x[i + j], a.scale_log2, -lv[j]);
                    p[j] = ex2(e);
                    ds[j] = p[j] * (__uint_as_float(tr[i + j]) - dv[j]);
                    if (capped) ds[j] *= cap[i + j];
                }
                pp[i / 2] = pack_bf16x2(p[0], p[1]);
                pp[i / 2 + 1] = pack_bf16x2(p[2], p[3]);
                dd[i / 2] = pack_bf16x2(ds[0], ds[1]);
                dd[i / 2 + 1] = pack_bf16x2(ds[2], ds[3]);
            }
            if (KV) tmem_st16(slot, pp);
            tmem_st16(slot + 16, dd);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DSREADY + (t & 1)));
        }
        bool have = ok && n > 0;
        if (have) {
            have = mbar_wait_warp(bar(B_DONE), 0, abort_flag, &g_bwd_err);
            tc_fence_after();
        }
        const bool store = xr < (KV ? a.Sk : a.Sq);
        // dK / dV: one warpgroup each; dQ: half the columns each.
        const bool second = KV && wg == 1;
        const int ncol = KV ? (wg == 0 ? DK : DV) : DK / 2;
        const int tcol = KV ? (wg == 0 ? C::T_A1 : C::T_A2) : C::T_A1 + wg * (DK / 2);
        char *base = second ? a.g2 : a.g1;
        const int64_t off = second ? (int64_t)b * a.g2_sb + (int64_t)h * a.g2_sh + (int64_t)xr * a.g2_ss
                                   : (int64_t)b * a.g1_sb + (int64_t)h * a.g1_sh + (int64_t)xr * a.g1_ss;
        const float f = second ? 1.f : a.scale;
        const int col0 = KV ? 0 : wg * (DK / 2);
        for (int c = 0; c < ncol; c += 32) {
            uint32_t r[32];
            if (have) {
                tmem_ld32(tl + (uint32_t)(tcol + c), r);
                tmem_wait_ld();
                reg_fence(r);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = 0u;
            }
            if (!store) continue;
            if (a.g_bf16) {
                uint4 *dst = reinterpret_cast<uint4 *>(base + 2 * (off + col0 + c));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dst[i] = make_uint4(pack_bf16x2(__uint_as_float(r[8 * i]) * f, __uint_as_float(r[8 * i + 1]) * f),
                                        pack_bf16x2(__uint_as_float(r[8 * i + 2]) * f, __uint_as_float(r[8 * i + 3]) * f),
                                        pack_bf16x2(__uint_as_float(r[8 * i + 4]) * f, __uint_as_float(r[8 * i + 5]) * f),
                                        pack_bf16x2(__uint_as_float(r[8 * i + 6]) * f, __uint_as_float(r[8 * i + 7]) * f));
            } else {
                float4 *dst = reinterpret_cast<float4 *>(base + 4 * (off + col0 + c));
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
    float *lse2, *delta;
};

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
            lse = lse == -INFINITY ? INFINITY : lse * kLog2e;
        }
        a.lse2[r] = lse;
        a.delta[r] = d;
    }
}

// dsink_h: one block a head, rows in a fixed order.
__global__ void __launch_bounds__(512) bwd_sink_kernel(const float *lse2, const float *delta, int64_t pitch, int B,
                                                       int Hq, int Sq, const float *sinks, float *out) {
    __shared__ float part[16];
    const int h = blockIdx.x;
    const float sk = sinks[h] * kLog2e;
    float acc = 0.f;
    for (int b = 0; b < B; ++b) {
        const int64_t r = ((int64_t)b * Hq + h) * pitch;
        for (int i = threadIdx.x; i < Sq; i += 512) acc -= ex2(sk - lse2[r + i]) * delta[r + i];
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

template <int DK, int DV, bool KV, int NST, bool MODS>
cudaError_t launch_tiles(const BwdLaunch &L, BwdArgs a, cudaStream_t stream) {
    using C = BwdCfg<DK, DV, KV, NST>;
    auto kern = bwd_tile_kernel<DK, DV, KV, NST, MODS>;
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
        kern<<<grid, 384, C::SMEM_BYTES, stream>>>(L.tmKx, L.tmVx, L.tmQy, L.tmDOy, a);
    else
        kern<<<grid, 384, C::SMEM_BYTES, stream>>>(L.tmQx, L.tmDOx, L.tmKy, L.tmVy, a);
    return cudaGetLastError();
}

template <int DK, int DV, int NST, bool MODS>
cudaError_t launch_pair(const BwdLaunch &L, const BwdArgs &a, cudaStream_t stream) {
    cudaError_t e = launch_tiles<DK, DV, true, NST, MODS>(L, a, stream);
    if (e == cudaSuccess) e = launch_tiles<DK, DV, false, NST, MODS>(L, a, stream);
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
        p.lse2 = L.lse2, p.delta = L.delta;
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
        bwd_sink_kernel<<<L.Hq, 512, 0, stream>>>(L.lse2, L.delta, pitch, L.B, L.Hq, L.Sq, L.mods.sinks, L.gsinks);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    BwdArgs a = {};
    a.Hq = L.Hq, a.Hkv = L.Hkv, a.Sq = L.Sq, a.Sk = L.Sk, a.causal = L.causal;
    a.scale = L.scale, a.scale_log2 = L.scale * kLog2e;
    a.mods = L.mods;
    a.lse2 = L.lse2, a.delta = L.delta, a.pitch = pitch;
    a.g_bf16 = L.g_bf16;
#define FA_BWD_PAIR(DK_, DV_, NST_) \
    (L.has_mods ? launch_pair<DK_, DV_, NST_, true>(L, a, stream) : launch_pair<DK_, DV_, NST_, false>(L, a, stream))
    if (L.dk == 64 && L.dv == 64) return FA_BWD_PAIR(64, 64, 4);
    if (L.dk == 128 && L.dv == 128) return FA_BWD_PAIR(128, 128, 4);
    if (L.dk == 192 && L.dv == 128) return FA_BWD_PAIR(192, 128, 3);
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
