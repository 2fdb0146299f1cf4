// score_mods.cuh -- optional score modifiers of the prefill kernels:
// additive f16 mask, ALiBi slopes, logit softcap and attention sinks.
//
// These follow the llama.cpp tensor kernel ("ggml-metal: FA tensor path",
// kernel_flash_attn_ext_tensor_impl), in the order its score loop applies
// them:
//
//   s  = scale * (q . k)
//   s  = softcap * tanh(s)                 if softcap != 0
//   s += slope_h * mask[b][h][i][j]        if a mask is given
//
// slope_h is 1 unless max_bias != 0.  Otherwise it is
// m0^(h+1) for h < n_head_log2 and m1^(2(h - n_head_log2) + 1) above (the
// page's ALiBi block); the host forms log2(m0) = -max_bias / n_head_log2 and
// log2(m1) = -max_bias / 2 / n_head_log2 with n_head_log2 the largest power
// of two <= Hq.  A sink (the page's "final: sinks" block) is one more logit
// per head in the softmax denominator, with no value row.
#pragma once

#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include "sm100.cuh"

namespace fa {

struct ScoreMods {
    const __half *mask;        // NULL: no mask
    int64_t m_sb, m_sh, m_ss;  // element strides (0 broadcasts); all multiples of 8
    float log2_m0, log2_m1;    // ALiBi bases as base-2 logarithms
    int n_head_log2;           // 0: ALiBi off (slope 1)
    float softcap;             // 0: off
    const float *sinks;        // NULL: no sinks; else [Hq], natural-log units
};

// What a prefill kernel's scores go through: nothing (MODS_SINKS: but a sink in
// the epilogue), a softcap, a mask, or both; sinks may come with each.  The
// kernels have one instantiation each: code that the others skip still cost
// them, by the instructions fetched and the registers laid out for it (a mask
// alone 25 to 30 % beside the softcap, sinks alone 3 to 10 %).
enum ModsKind { MODS_NONE, MODS_SINKS, MODS_CAP, MODS_MASK, MODS_CAP_MASK };

constexpr float kLog2e = 1.4426950408889634f;

FA_DEV float alibi_slope(const ScoreMods &m, int h) {
    if (m.n_head_log2 == 0) return 1.f;
    return h < m.n_head_log2 ? exp2f(m.log2_m0 * (float)(h + 1))
                             : exp2f(m.log2_m1 * (float)(2 * (h - m.n_head_log2) + 1));
}

// Row of the mask for (b, h, query row i), or NULL (no mask, or a row past
// the end of the queries).
FA_DEV const __half *mask_row(const ScoreMods &m, int b, int h, int i, int Sq) {
    if (!m.mask || i >= Sq) return nullptr;
    return m.mask + (int64_t)b * m.m_sb + (int64_t)h * m.m_sh + (int64_t)i * m.m_ss;
}

// 1/x from the approximate reciprocal instruction (one MUFU operation,
// within about an ulp; 1/inf = 0).
FA_DEV float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// softcap * tanh(scale * x) * log2(e) for four raw scores x[0..4), as
// tanh(u) = 1 - 2 / d with d = e^(2u) + 1, which is exact at both ends: d may
// be infinite.  A NaN stays one and touches no other score (a tile holds keys
// that a row does not see, and those may hold anything).
//
// With a reciprocal each: eight MUFU operations, few others.
FA_DEV void softcap4(float *x, float scale, float softcap) {
    const float k = 2.f * kLog2e * scale, c = softcap * kLog2e;
    const uint64_t k2 = f2_pack(k, k), one2 = f2_pack(1.f, 1.f), c2 = f2_pack(c, c), m2c = f2_pack(-2.f * c, -2.f * c);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        float a0, a1, d0, d1;
        f2_unpack(f2_mul(f2_pack(x[i], x[i + 1]), k2), a0, a1);
        f2_unpack(f2_add(f2_pack(ex2(a0), ex2(a1)), one2), d0, d1);
        f2_unpack(f2_fma(f2_pack(rcp_approx(d0), rcp_approx(d1)), m2c, c2), x[i], x[i + 1]);
    }
}

FA_DEV float within30(float x) {  // x limited to +-30, NaN kept
    float y;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(30.f));
    return y;
}

// The same with one reciprocal for the four, r = 1 / (d0 d1 d2 d3): five MUFU
// operations.  f / d of scores 0, 1 is r2 d23 and of scores 2, 3 r2 d01, with
// d01, d23 the pairs of d; c01, c23 are c, or NaN where the score is.  e^(2u)
// is clamped to 2^30 (tanh is 1 in fp32 from about 2^26 on), so the product
// stays below 2^121 and its reciprocal a normal number; each 1 / d carries a
// few ulp of rounding.  The clamp takes a NaN for a number, as in the product
// it would reach the other three; it comes back with 0 times the argument,
// limited so that infinities add nothing.
struct JointCap {
    uint64_t d01, d23, r2, c01, c23;
    FA_DEV JointCap(const float *x, float scale, float f, float c) {
        const float k = 2.f * kLog2e * scale;
        const uint64_t k2 = f2_pack(k, k), one2 = f2_pack(1.f, 1.f), c2 = f2_pack(c, c);
        float a0, a1, a2, a3, m0, m1;
        f2_unpack(f2_mul(f2_pack(x[0], x[1]), k2), a0, a1);
        f2_unpack(f2_mul(f2_pack(x[2], x[3]), k2), a2, a3);
        d01 = f2_add(f2_pack(ex2(fminf(a0, 30.f)), ex2(fminf(a1, 30.f))), one2);
        d23 = f2_add(f2_pack(ex2(fminf(a2, 30.f)), ex2(fminf(a3, 30.f))), one2);
        f2_unpack(f2_mul(d01, d23), m0, m1);  // d0 d2, d1 d3
        const float r = rcp_approx(m0 * m1) * f;
        r2 = f2_pack(r * m1, r * m0);
        c01 = f2_fma(f2_pack(within30(a0), within30(a1)), 0, c2);
        c23 = f2_fma(f2_pack(within30(a2), within30(a3)), 0, c2);
    }
};
FA_DEV void softcap4_joint(float *x, float scale, float softcap) {
    const float c = softcap * kLog2e;
    const JointCap j(x, scale, -2.f * c, c);
    f2_unpack(f2_fma(j.r2, j.d23, j.c01), x[0], x[1]);
    f2_unpack(f2_fma(j.r2, j.d01, j.c23), x[2], x[3]);
}

// And the factor of its derivative: with q = 1 / d, 1 - tanh^2 = 4 (q - q^2),
// here without the 4.
FA_DEV void softcap4_slope(float (&x)[4], float (&slope)[4], float scale, float softcap) {
    const float c = softcap * kLog2e;
    const JointCap j(x, scale, 1.f, c);
    const uint64_t m2c = f2_pack(-2.f * c, -2.f * c), minus = f2_pack(-1.f, -1.f);
    const uint64_t q01 = f2_mul(j.r2, j.d23), q23 = f2_mul(j.r2, j.d01);
    f2_unpack(f2_fma(q01, m2c, j.c01), x[0], x[1]);
    f2_unpack(f2_fma(q23, m2c, j.c23), x[2], x[3]);
    f2_unpack(f2_fma(f2_mul(q01, minus), q01, q01), slope[0], slope[1]);
    f2_unpack(f2_fma(f2_mul(q23, minus), q23, q23), slope[2], slope[3]);
}

// One 64-key chunk: raw scores x[0..64) (unscaled q.k) and the chunk's mask
// values w (64 f16 in key order; all zero without a mask) -> base-2 scores
// (modified score) * log2(e).  Capped jointly, or (MIXED) the two ways in turn,
// which in the two-tile kernel keeps the MUFU and the other pipes busy alike
// (both modifiers at 2 x 16 x 2048 x 128, causal: mixed 96.8 us, all jointly 102,
// all by softcap4 97.1; 2 x 8 x 1024, not causal: 43.7, 44.4 and 45.1); the
// one-tile kernel, with half the softmax warps an SM, waits less for them than
// for instructions (2 x 16 x 2048 x 192 / 128: mixed 304, jointly 255, softcap4
// 308).
template <ModsKind KIND, bool MIXED>
FA_DEV void modify_chunk(float *x, const uint4 (&w)[8], const ScoreMods &m, float scale, float slope) {
    const float cs = scale * kLog2e;   // raw score -> base-2 units, without softcap
    const float cm = slope * kLog2e;   // mask value -> base-2 units
    const uint64_t cs2 = f2_pack(cs, cs), cm2 = f2_pack(cm, cm);
    constexpr bool capped = KIND == MODS_CAP_MASK;
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        const uint32_t mw[4] = {w[g].x, w[g].y, w[g].z, w[g].w};  // four f16 pairs
        if (capped) {
            if (MIXED)
                softcap4(x + 8 * g, scale, m.softcap);
            else
                softcap4_joint(x + 8 * g, scale, m.softcap);
            softcap4_joint(x + 8 * g + 4, scale, m.softcap);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = 8 * g + 2 * j;
            const float2 mf = __half22float2(*reinterpret_cast<const __half2 *>(&mw[j]));
            uint64_t y;
            if (capped) {  // x holds the capped score in base-2 units already
                y = f2_fma(f2_pack(mf.x, mf.y), cm2, f2_pack(x[k], x[k + 1]));
            } else {
                y = f2_fma(f2_pack(x[k], x[k + 1]), cs2, f2_mul(f2_pack(mf.x, mf.y), cm2));
            }
            f2_unpack(y, x[k], x[k + 1]);
        }
    }
}

// Keys k >= lim of the tile are hidden (-inf).
template <int BN>
FA_DEV void hide_keys(float (&x)[BN], int lim) {
    if (lim < BN) {
#pragma unroll
        for (int k = 0; k < BN; ++k)
            if (k >= lim) x[k] = -INFINITY;
    }
}

// One-tile kernel: raw scores x[k] (unscaled q.k of keys key0 + k) -> base-2
// scores (modified score) * log2(e); keys k >= lim are hidden (-inf).  mrow: this
// row's mask in global memory or NULL; keys at or past Sk are never read
// from it.  The mask is read 64 keys at a time: a chunk wholly inside the row
// issues its eight 16-byte loads before the first is used.
template <int BN, ModsKind KIND>
FA_DEV void modify_scores(float (&x)[BN], const ScoreMods &m, float scale, float slope, const __half *mrow,
                          int key0, int Sk, int lim) {
    static_assert(BN % 64 == 0, "tile width");
    if constexpr (KIND == MODS_CAP) {
#pragma unroll
        for (int k = 0; k < BN; k += 4) softcap4_joint(x + k, scale, m.softcap);
    } else {
#pragma unroll
        for (int h = 0; h < BN / 64; ++h) {
            const int kc = key0 + 64 * h;
            uint4 w[8];
            if (mrow && kc + 64 <= Sk) {
#pragma unroll
                for (int g = 0; g < 8; ++g) w[g] = __ldg(reinterpret_cast<const uint4 *>(mrow + kc + 8 * g));
            } else {
                uint32_t mw[32];  // f16 pairs; zero: no mask value
#pragma unroll
                for (int j = 0; j < 32; ++j) mw[j] = 0u;
                if (mrow) {  // the row's last, partial chunk: element loads up to Sk
                    const uint16_t *mr = reinterpret_cast<const uint16_t *>(mrow);
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (kc + e < Sk) mw[e >> 1] |= (uint32_t)mr[kc + e] << (16 * (e & 1));
                }
#pragma unroll
                for (int g = 0; g < 8; ++g) w[g] = make_uint4(mw[4 * g], mw[4 * g + 1], mw[4 * g + 2], mw[4 * g + 3]);
            }
            modify_chunk<KIND, false>(&x[64 * h], w, m, scale, slope);
        }
    }
    hide_keys<BN>(x, lim);
}

// Epilogue with a sink: O was accumulated relative to m_run (base 2);
// l_run is the fp32 weight sum and l_o the sum of the bf16-rounded weights O
// was built from.  Returns the factor that normalises O and, in *lse2, the
// base-2 log-sum-exp including the sink.
FA_DEV float sink_normalise(float m_run, float l_run, float l_o, float sink_nat, float *lse2) {
    const float sk = sink_nat * kLog2e;
    const float mm = fmaxf(m_run, sk);
    if (mm == -INFINITY) {
        *lse2 = -INFINITY;
        return 0.f;
    }
    const float a_o = l_run > 0.f ? ex2(m_run - mm) : 0.f;
    const float e_s = ex2(sk - mm);
    *lse2 = mm + __log2f(l_run * a_o + e_s);
    return a_o / (l_o * a_o + e_s);
}

}  // namespace fa
