// rope.cu -- rotary positions (fa_rope) and the write of new K/V rows into a
// paged cache with the rotation fused in (fa_kv_append).
//
// Rotation of pair i of a row at position p by the angle a = p f_i:
//
//   y0 = m (x0 cos a - x1 sin a),   y1 = m (x1 cos a + x0 sin a)
//
// and its gradient (inverse), the same with a negated: the map is m times a
// rotation, so its transpose turns back.  The pair is (x[i], x[i + rot / 2])
// (half layout) or (x[2i], x[2i + 1]) (interleaved), inside columns
// [offset, offset + rot); the other columns pass through.
//
// Angles: p f_i in fp32 would be off by p f_i 2^-24 radians, which is 0.06 at
// a million tokens.  The host turns f_i into a 64-bit fraction of a turn,
// t_i = f_i / (2 pi) mod 1, so that p t_i mod 2^64 -- one integer product,
// whose overflow drops the whole turns -- is the exact fraction of the turn
// that the position has reached.  Its upper 32 bits (1.5e-9 radians) go to
// sincospif.
//
// Both kernels move each row once and are bound by HBM.  A thread owns an
// item of 16 columns: eight pairs, or two 8-column vectors that pass through.
// It computes its eight sines and cosines once and walks a group of heads
// with them; neighbouring threads own neighbouring vectors, so a warp's
// loads and stores are whole 128-byte lines.  A thread reads its item before
// it writes it and nobody else touches it, so a tensor may be turned in place.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "sm100.cuh"

namespace fa {
namespace {

__device__ int g_append_err;

constexpr int kThreads = 256;

// Sine and cosine (times mscale) of the eight pairs of item `i`.
FA_DEV void item_angles(const RopeMap &r, int i, int pos, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint64_t t = r.turns[8 * i + j] * (uint64_t)(int64_t)pos;
        const float half_turns = (float)(int32_t)(uint32_t)(t >> 32) * 0x1p-31f;  // in [-1, 1]
        sincospif(half_turns, &s[j], &c[j]);
        c[j] *= r.mscale;
        s[j] *= r.inverse ? -r.mscale : r.mscale;
    }
}

// Columns of the two 8-column vectors of item i of a row of width d: items
// below rot / 16 hold pairs, the others pass through.
FA_DEV void item_columns(const RopeMap &r, int i, int &c0, int &c1) {
    const int ni = r.rot >> 4;
    if (i < ni) {
        c0 = r.offset + (r.interleaved ? 16 * i : 8 * i);
        c1 = c0 + (r.interleaved ? 8 : r.rot >> 1);
    } else {
        const int col = 16 * (i - ni);
        c0 = col < r.offset ? col : col + r.rot;
        c1 = c0 + 8;
    }
}

FA_DEV void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        x[2 * j] = __uint_as_float(u[j] << 16);
        x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
}
FA_DEV void load8(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
FA_DEV void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                               pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
FA_DEV void store8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// The item's two vectors turned, in 32 bits.
FA_DEV void turn(bool interleaved, const float (&c)[8], const float (&s)[8], float (&x)[8], float (&y)[8]) {
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = x[2 * j], b = x[2 * j + 1], e = y[2 * j], f = y[2 * j + 1];
            x[2 * j] = a * c[j] - b * s[j];
            x[2 * j + 1] = b * c[j] + a * s[j];
            y[2 * j] = e * c[j + 4] - f * s[j + 4];
            y[2 * j + 1] = f * c[j + 4] + e * s[j + 4];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float a = x[j], b = y[j];
            x[j] = a * c[j] - b * s[j];
            y[j] = b * c[j] + a * s[j];
        }
    }
}

// ---------------------------------------------------------------- fa_rope --

template <typename T>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeLaunch L) {
    const int ni = L.map.rot >> 4;
    const int item = threadIdx.x % L.items, tok = threadIdx.x / L.items;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / L.items) + tok;
    if (tok >= kThreads / L.items || row >= (int64_t)L.B * L.S) return;
    const int b = (int)(row / L.S), s = (int)(row % L.S);
    int c0, c1;
    item_columns(L.map, item, c0, c1);
    float cs[8], sn[8];
    if (item < ni) {
        const int pos = L.pos ? __ldg(L.pos + b * L.pos_sb + s) : L.pos0 + s;
        item_angles(L.map, item, pos, cs, sn);
    }
    const int h1 = min(L.x[0].H + L.x[1].H, ((int)blockIdx.y + 1) * L.heads);
    for (int h = blockIdx.y * L.heads; h < h1; ++h) {
        const int which = h >= L.x[0].H;
        const RopeTensor &t = L.x[which];
        if (t.in_place && item >= ni) continue;  // nothing to move
        const int hh = h - (which ? L.x[0].H : 0);
        const T *src = static_cast<const T *>(t.src) + b * t.sb + hh * t.sh + s * t.ss;
        T *dst = static_cast<T *>(t.dst) + b * t.ob + hh * t.oh + s * t.os;
        float x[8], y[8];
        load8(src + c0, x);
        load8(src + c1, y);
        if (item < ni) turn(L.map.interleaved, cs, sn, x, y);
        store8(dst + c0, x);
        store8(dst + c1, y);
    }
}

// ----------------------------------------------------------- fa_kv_append --

// Largest of `v` over the lanes whose vectors share a 32-value block: in the
// half layout's pairs each of the two vectors lies in its own block, with
// those of the three neighbouring items; otherwise the item's two vectors
// and those of one neighbour make a block.  Every lane of the warp takes part.
template <typename K>
FA_DEV void block_max(bool split, K &k0, K &k1) {
    if (!split) k0 = k1 = k0 > k1 ? k0 : k1;
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
        const K o0 = __shfl_xor_sync(0xffffffffu, k0, d), o1 = __shfl_xor_sync(0xffffffffu, k1, d);
        if (d == 1 || split) {
            k0 = o0 > k0 ? o0 : k0;
            k1 = o1 > k1 ? o1 : k1;
        }
    }
}

// A NaN orders above every number here, so that a block that holds one gets
// a NaN scale.
FA_DEV uint32_t abs_key(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Scale of a block as the f16 that is stored; its magnitude is limited to
// the largest f16, so that finite values stay finite.
FA_DEV __half block_scale(float d) {
    return __float2half_rn(isfinite(d) ? fminf(fmaxf(d, -65504.f), 65504.f) : NAN);
}

// Nearest code (ties to even) of x at scale d, within [lo, hi]; 0 where the
// scale is zero or not a number.
FA_DEV int code_of(float x, float d, float lo, float hi) {
    return d != 0.f && !isnan(d) ? (int)fminf(fmaxf(rintf(x / d), lo), hi) : 0;
}

// Writes the two vectors x (columns c0 ..) and y (columns c1 ..) of a row to
// the cache row `dst`.  All lanes of a warp call it (it shuffles); `live`
// says whether this lane's row is written.
template <int KV>
FA_DEV void put(uint8_t *dst, int c0, int c1, bool split, float scale, const float (&x)[8], const float (&y)[8],
                bool live) {
    if constexpr (KV == 0) {
        if (live) {
            store8(reinterpret_cast<__nv_bfloat16 *>(dst) + c0, x);
            store8(reinterpret_cast<__nv_bfloat16 *>(dst) + c1, y);
        }
    } else if constexpr (KV == 2) {
        // e4m3 of x / scale: the quotient in fp32, then one rounding to the
        // nearest, limited to the type's largest value
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float(&v)[8] = j < 2 ? x : y;
            const int k = 4 * (j & 1);
            w[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[k] / scale, v[k + 1] / scale), __NV_SATFINITE,
                                                      __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[k + 2] / scale, v[k + 3] / scale),
                                                      __NV_SATFINITE, __NV_E4M3)
                       << 16;
        }
        if (live) {
            *reinterpret_cast<uint2 *>(dst + c0) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(dst + c1) = make_uint2(w[2], w[3]);
        }
    } else if constexpr (KV == 8) {
        uint32_t k0 = 0, k1 = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) k0 = max(k0, abs_key(x[j])), k1 = max(k1, abs_key(y[j]));
        block_max(split, k0, k1);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int c = v ? c1 : c0;
            const __half h = block_scale(__uint_as_float(v ? k1 : k0) / 127.f);
            const float d = __half2float(h);
            uint8_t *blk = dst + (c >> 5) * 34;
            const int part = (c >> 3) & 3;
            if (live && part == 0) *reinterpret_cast<__half *>(blk) = h;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int q0 = code_of(v ? y[2 * j] : x[2 * j], d, -127.f, 127.f);
                const int q1 = code_of(v ? y[2 * j + 1] : x[2 * j + 1], d, -127.f, 127.f);
                if (live)
                    reinterpret_cast<uint16_t *>(blk + 2 + 8 * part)[j] = (uint16_t)((q0 & 255) | ((q1 & 255) << 8));
            }
        }
    } else {
        // q4_0.  The key orders by magnitude, then the lowest index, and
        // carries the sign.
        unsigned long long k0 = 0, k1 = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const auto key = [](float v, int idx) {
                return (unsigned long long)abs_key(v) << 32 | (unsigned)(31 - idx) << 1 | (__float_as_uint(v) >> 31);
            };
            k0 = max(k0, key(x[j], (c0 & 31) + j));
            k1 = max(k1, key(y[j], (c1 & 31) + j));
        }
        block_max(split, k0, k1);
        uint32_t n[2];  // eight nibbles each
        __half h[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const unsigned long long k = v ? k1 : k0;
            const float m = __uint_as_float((uint32_t)(k >> 32) | (uint32_t)(k & 1) << 31);
            h[v] = block_scale(m / -8.f);
            const float d = __half2float(h[v]);
            n[v] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) n[v] |= (uint32_t)(code_of(v ? y[j] : x[j], d, -8.f, 7.f) + 8) << (4 * j);
        }
        // Byte j of a block holds values j (low) and j + 16 (high): vectors 0
        // and 2, or 1 and 3, of the block.  Split: lanes 0, 1 of four own the
        // low nibbles and lanes 2, 3 the high ones, so lanes 0 and 1 write
        // after a swap with the lane two up.  Otherwise the even lane owns
        // values 0..15, the odd one 16..31: each writes eight bytes after a
        // swap of one vector.
        const uint32_t s0 = __shfl_xor_sync(0xffffffffu, n[0], 2), s1 = __shfl_xor_sync(0xffffffffu, n[1], 2);
        const bool high = (c0 >> 4) & 1;  // this item's c0 lies in the block's upper half
        const uint32_t give = high ? n[0] : n[1];
        const uint32_t take = __shfl_xor_sync(0xffffffffu, give, 1);
        const auto spread = [](uint32_t lo, uint32_t hi, uint8_t *at) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t l = lo >> (8 * j), u = hi >> (8 * j);
                reinterpret_cast<uint16_t *>(at)[j] =
                    (uint16_t)((l & 15) | (u & 15) << 4 | (l >> 4 & 15) << 8 | (u >> 4 & 15) << 12);
            }
        };
        if (!live) return;
        if (split) {
            if (high) return;
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int c = v ? c1 : c0;
                uint8_t *blk = dst + (c >> 5) * 18;
                if (((c >> 3) & 3) == 0) *reinterpret_cast<__half *>(blk) = h[v];
                spread(n[v], v ? s1 : s0, blk + 2 + (c & 8));
            }
        } else {
            uint8_t *blk = dst + (c0 >> 5) * 18;
            if (!high) *reinterpret_cast<__half *>(blk) = h[0];
            if (high)
                spread(take, n[1], blk + 10);
            else
                spread(n[0], take, blk + 2);
        }
    }
}

// blockIdx.x: rows (sequence, new row); blockIdx.y: groups of `heads` heads,
// first those of q, then of k, then of v.
template <int KV>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendLaunch L) {
    const int ni = L.map.rot >> 4;
    const int rows_per_block = kThreads / L.items;
    const int item = threadIdx.x % L.items, tok = threadIdx.x / L.items;
    const int64_t row = (int64_t)blockIdx.x * rows_per_block + tok;
    bool live = tok < rows_per_block && row < (int64_t)L.B * L.Sq;
    const int b = live ? (int)(row / L.Sq) : 0, i = live ? (int)(row % L.Sq) : 0;
    int g = blockIdx.y, kind = 0;  // 0: q, 1: k, 2: v
    if (g >= L.q_groups) {
        g -= L.q_groups;
        kind = 1;
        if (g >= L.kv_groups) g -= L.kv_groups, kind = 2;
    }
    const int n = L.q_lens ? max(0, min(__ldg(L.q_lens + b), L.Sq)) : L.Sq;
    const int64_t at = (int64_t)__ldg(L.seq_lens + b) - n + i;  // the row's place in its sequence
    const bool turned = kind < 2 && item < ni;
    const int d = kind == 2 ? L.dv : L.dk;
    live = live && item < (d >> 4);
    int c0, c1;
    if (kind < 2)
        item_columns(L.map, item, c0, c1);
    else
        c0 = 16 * item, c1 = c0 + 8;
    if (!live) c0 = 0, c1 = 8;
    float cs[8], sn[8];
    if (turned && live && i < n) {
        const int pos = L.pos ? __ldg(L.pos + b * L.pos_sb + i) : (int)at;
        item_angles(L.map, item, pos, cs, sn);
    }
    if (kind == 0) {
        // q: turned rows; the rows past the sequence's new ones are zeros
        if (!live || (i < n && L.q.in_place && !turned)) return;
        const int h1 = min(L.q.H, (g + 1) * L.heads);
        for (int h = g * L.heads; h < h1; ++h) {
            const __nv_bfloat16 *src =
                static_cast<const __nv_bfloat16 *>(L.q.src) + b * L.q.sb + h * L.q.sh + i * L.q.ss;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(L.q.dst) + b * L.q.ob + h * L.q.oh + i * L.q.os;
            float x[8] = {}, y[8] = {};
            if (i < n) {
                load8(src + c0, x);
                load8(src + c1, y);
                if (turned) turn(L.map.interleaved, cs, sn, x, y);
            }
            store8(dst + c0, x);
            store8(dst + c1, y);
        }
        return;
    }
    // A row before its sequence's start has no slot; one past the table's
    // end, or in a block that does not exist, is an error of the caller.
    live = live && i < n && at >= 0;
    int64_t slot0 = 0;
    if (live) {
        int blk = -1;
        if (at < (int64_t)L.max_blocks * 64) blk = __ldg(L.block_table + (int64_t)b * L.max_blocks + at / 64);
        if (blk < 0 || blk >= L.num_blocks) {
            atomicCAS(&g_append_err, 0, 2 /* FA_DEVERR_BAD_BLOCK */);
            live = false;
        }
        slot0 = (int64_t)blk * L.Hkv * 64 + at % 64;
    }
    const RopeTensor &t = kind == 1 ? L.k : L.v;
    const int64_t row_bytes = KV == 8 ? d / 32 * 34 : KV == 4 ? d / 32 * 18 : KV == 2 ? d : 2 * d;
    const bool split = turned && !L.map.interleaved;
    const int h1 = min(L.Hkv, (g + 1) * L.heads);
    for (int h = g * L.heads; h < h1; ++h) {
        float x[8] = {}, y[8] = {};
        if (live) {
            const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(t.src) + b * t.sb + h * t.sh + i * t.ss;
            load8(src + c0, x);
            load8(src + c1, y);
            if (turned) turn(L.map.interleaved, cs, sn, x, y);
        }
        uint8_t *dst = static_cast<uint8_t *>(t.dst) + (slot0 + (int64_t)h * 64) * row_bytes;
        put<KV>(dst, c0, c1, split, kind == 1 ? L.k_scale : L.v_scale, x, y, live);
    }
}

// Heads that one thread walks with its sines: up to 8, fewer while that
// leaves the device's threads idle.
int head_group(int64_t units, int heads, int num_sms) {
    int g = 8;
    while (g > 1 && units * ((heads + g - 1) / g) < (int64_t)num_sms * 2048) g >>= 1;
    return g;
}

}  // namespace

cudaError_t launch_rope(RopeLaunch L, bool f32, int num_sms, cudaStream_t stream) {
    L.items = L.d / 16;
    const int H = L.x[0].H + L.x[1].H, per = kThreads / L.items;
    const int64_t rows = (int64_t)L.B * L.S;
    L.heads = head_group(rows * L.items, H, num_sms);
    const dim3 grid((unsigned)((rows + per - 1) / per), (unsigned)((H + L.heads - 1) / L.heads));
    if (f32)
        rope_kernel<float><<<grid, kThreads, 0, stream>>>(L);
    else
        rope_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(L);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(AppendLaunch L, int num_sms, cudaStream_t stream) {
    L.items = (L.dk > L.dv ? L.dk : L.dv) / 16;
    const int per = kThreads / L.items;
    const int64_t rows = (int64_t)L.B * L.Sq;
    L.heads = head_group(rows * L.items, L.q.H + 2 * L.Hkv, num_sms);
    L.q_groups = (L.q.H + L.heads - 1) / L.heads;
    L.kv_groups = (L.Hkv + L.heads - 1) / L.heads;
    const dim3 grid((unsigned)((rows + per - 1) / per), (unsigned)(L.q_groups + 2 * L.kv_groups));
    switch (L.kv_type) {
        case 0: append_kernel<0><<<grid, kThreads, 0, stream>>>(L); break;
        case 2: append_kernel<2><<<grid, kThreads, 0, stream>>>(L); break;
        case 8: append_kernel<8><<<grid, kThreads, 0, stream>>>(L); break;
        default: append_kernel<4><<<grid, kThreads, 0, stream>>>(L); break;
    }
    return cudaGetLastError();
}

cudaError_t append_device_error(int clear, int *code) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_append_err, sizeof(int));
    if (e != cudaSuccess) return e;
    *code = v;
    if (clear && v) {
        v = 0;
        e = cudaMemcpyToSymbol(g_append_err, &v, sizeof(int));
    }
    return e;
}

}  // namespace fa
