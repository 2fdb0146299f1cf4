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
// whose overflow drops the whole turns -- is the fraction of the turn that the
// position has reached: within 3 p 2^-64 turns for f_i up to 2 pi, 2.2e-9
// radians at p = 2^31.  Its upper 32 bits (1.5e-9 radians) go to sincospif,
// less the nearest quarter turn, as fp32 (2.4e-8): together within 2.8e-8
// radians.
//
// Both kernels move each row once and are bound by HBM.  A thread owns an
// item of two 16-byte vectors: their pairs, or columns that pass through.
// It computes its sines and cosines once and walks a group of heads
// with them; neighbouring threads own neighbouring vectors, so a warp's
// loads and stores are whole 128-byte lines, and has several heads' loads under
// way at once.  A thread reads its item before
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

constexpr int kThreads = 128;  // 29.6 us for 33.5 M bf16 values, 30.8 with 256: a shorter last wave

// An item is two 16-byte vectors of V values: V pairs, or 2 V columns that
// pass through.
template <typename T>
constexpr int kVec = 16 / sizeof(T);

// Sine and cosine (times mscale) of the pairs of item `i`.
template <int V>
FA_DEV void item_angles(const RopeMap &r, int i, int pos, float (&c)[V], float (&s)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const uint32_t t = (uint32_t)(r.turns[V * i + j] * (uint64_t)(int64_t)pos >> 32);
        // The nearest quarter turn comes off in whole numbers, so that fp32
        // holds what is left (an eighth of a turn at most) to 2.4e-8 radians;
        // the whole turn's fraction would be rounded by up to 9.4e-8.
        const uint32_t quarters = (t + 0x20000000u) >> 30;
        const float half_turns = (float)(int32_t)(t - (quarters << 30)) * 0x1p-31f;  // in [-1/4, 1/4]
        float sn, cn;
        sincospif(half_turns, &sn, &cn);
        s[j] = quarters & 1 ? cn : sn;
        c[j] = quarters & 1 ? sn : cn;
        if (quarters & 2) s[j] = -s[j];
        if ((quarters + 1) & 2) c[j] = -c[j];
        c[j] *= r.mscale;
        s[j] *= r.inverse ? -r.mscale : r.mscale;
    }
}

// First columns of the two vectors of item i of a row: items below rot / 2V
// hold pairs, the others pass through.
template <int V>
FA_DEV void item_columns(const RopeMap &r, int i, int &c0, int &c1) {
    const int ni = r.rot / (2 * V);
    if (i < ni) {
        c0 = r.offset + (r.interleaved ? 2 * V * i : V * i);
        c1 = c0 + (r.interleaved ? V : r.rot >> 1);
    } else {
        const int col = 2 * V * (i - ni);
        c0 = col < r.offset ? col : col + r.rot;
        c1 = c0 + V;
    }
}

// A vector as it lies in memory.  Every value is used once, so loads and
// stores are marked to leave the caches first.
template <typename T>
struct Raw {
    uint4 w;
    FA_DEV void load(const T *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    FA_DEV void get(float (&x)[kVec<T>]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 2) {
                x[2 * j] = __uint_as_float(u[j] << 16);
                x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
            } else {
                x[j] = __uint_as_float(u[j]);
            }
        }
    }
};
FA_DEV void store_vec(__nv_bfloat16 *p, const float (&x)[8]) {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                    pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
}
FA_DEV void store_vec(float *p, const float (&x)[4]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
}

// The item's two vectors turned, in 32 bits.
template <int V>
FA_DEV void turn(bool interleaved, const float (&c)[V], const float (&s)[V], float (&x)[V], float (&y)[V]) {
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const float a = x[2 * j], b = x[2 * j + 1], e = y[2 * j], f = y[2 * j + 1];
            x[2 * j] = a * c[j] - b * s[j];
            x[2 * j + 1] = b * c[j] + a * s[j];
            y[2 * j] = e * c[j + V / 2] - f * s[j + V / 2];
            y[2 * j + 1] = f * c[j + V / 2] + e * s[j + V / 2];
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float a = x[j], b = y[j];
            x[j] = a * c[j] - b * s[j];
            y[j] = b * c[j] + a * s[j];
        }
    }
}

// ---------------------------------------------------------------- fa_rope --

// Heads whose loads a thread has under way together: enough bytes for HBM
// (33.5 M bf16 values: 37 us with one head at a time, 29.6 with four).
constexpr int kBatch = 4;

// Walks heads h0 .. h1 - 1 of one row of t with this thread's item, N heads at
// a time.  angles: computes the sines, called once, under the first loads.
// done(h, x, y) takes each head's two vectors; `read` false gives zeros.
template <typename T, int N, typename Angles, typename Done>
FA_DEV void walk_heads(const T *src, int64_t sh, int h0, int h1, int c0, int c1, bool read, bool turned, bool interleaved,
                       const Angles &angles, const Done &done) {
    constexpr int V = kVec<T>;
    float cs[V], sn[V];
    src += (int64_t)h0 * sh;
    for (int h = h0; h < h1; h += N, src += N * sh) {
        Raw<T> u[N], w[N];
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (read && h + k < h1) {
                u[k].load(src + k * sh + c0);
                w[k].load(src + k * sh + c1);
            }
        if (turned && h == h0) angles(cs, sn);
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (h + k < h1) {
                float x[V] = {}, y[V] = {};
                if (read) {
                    u[k].get(x);
                    w[k].get(y);
                    if (turned) turn(interleaved, cs, sn, x, y);
                }
                done(h + k, x, y);
            }
    }
}

// blockIdx.x: rows; blockIdx.y: groups of `heads` heads, first those of x[0].
// Bound by HBM: 42 M bf16 values (2 x 40 heads x 4096 x 128) take 26 to 28 us, a
// copy's rate 25.6; 6.3 M fp32 values 9 (7.7).
template <typename T, int N>
__global__ void __launch_bounds__(kThreads, 5) rope_kernel(const __grid_constant__ RopeLaunch L) {
    constexpr int V = kVec<T>;
    const int ni = L.map.rot / (2 * V);
    const int item = threadIdx.x % L.items, tok = threadIdx.x / L.items;
    const int64_t row = (int64_t)blockIdx.x * (kThreads / L.items) + tok;
    if (tok >= kThreads / L.items || row >= (int64_t)L.B * L.S) return;
    const int b = (int)((uint32_t)row / (uint32_t)L.S), s = (int)((uint32_t)row % (uint32_t)L.S);
    const bool turned = item < ni, second = (int)blockIdx.y >= L.groups0;
    const RopeTensor &t = L.x[second];
    if (t.in_place && !turned) return;  // nothing moves
    int c0, c1;
    item_columns<V>(L.map, item, c0, c1);
    const int h0 = ((int)blockIdx.y - (second ? L.groups0 : 0)) * L.heads;
    const int pos = turned && L.pos ? __ldg(L.pos + b * L.pos_sb + s) : L.pos0 + s;
    T *dst = static_cast<T *>(t.dst) + b * t.ob + s * t.os;
    walk_heads<T, N>(
        static_cast<const T *>(t.src) + b * t.sb + s * t.ss, t.sh, h0, min(t.H, h0 + L.heads), c0, c1, true, turned,
        L.map.interleaved, [&](float(&c)[V], float(&n)[V]) { item_angles(L.map, item, pos, c, n); },
        [&](int h, const float(&x)[V], const float(&y)[V]) {
            store_vec(dst + h * t.oh + c0, x);
            store_vec(dst + h * t.oh + c1, y);
        });
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

// Codes of one block: x / d to the nearest, ties to even, within [lo, hi]; 0
// where d is zero or not a number.  The quotient is taken by a product with
// 1 / d and rounded by adding 1.5 * 2^23, whose low bits are then the code;
// the remainder x - n d, exact in an FMA, tells the few quotients next to a
// half that the product put on the wrong side.  (Sixteen divisions and
// conversions a thread cost more than the copy.)
struct Coder {
    float d, inv, half, lo, hi;
    bool ok;
    FA_DEV Coder(float d_, float lo_, float hi_) : d(d_), lo(lo_), hi(hi_) {
        ok = d != 0.f && !isnan(d);
        inv = ok ? 1.f / d : 0.f;
        half = 0.5f * fabsf(d);
    }
    // The codes of a vector, each in the low bits (two's complement).
    FA_DEV void operator()(const float (&x)[8], uint32_t (&q)[8]) const {
        constexpr float magic = 12582912.f;
        float r[8], e[8];
        bool near = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = fminf(fmaxf(x[j] * inv, lo), hi) + magic;
            e[j] = fmaf(magic - r[j], d, x[j]);
            near |= fabsf(e[j]) >= half;
        }
        if (near) {  // rare: a quotient next to a half, or beyond the codes
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float t = d < 0.f ? -e[j] : e[j];
                const bool odd = __float_as_uint(r[j]) & 1u;
                float n = r[j] - magic;
                if (t > half || (t == half && odd)) n += 1.f;
                if (t < -half || (t == -half && odd)) n -= 1.f;
                r[j] = fminf(fmaxf(n, lo), hi) + magic;
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = ok ? __float_as_uint(r[j]) : 0u;
    }
};

// Writes the two vectors x (columns c0 ..) and y (columns c1 ..) of a row to
// the cache row `dst`.  All lanes of a warp call it (it shuffles); `live`
// says whether this lane's row is written.
template <int KV>
FA_DEV void put(uint8_t *dst, int c0, int c1, bool split, float inv, const float (&x)[8], const float (&y)[8],
                bool live) {
    if constexpr (KV == 0) {
        if (live) {
            store_vec(reinterpret_cast<__nv_bfloat16 *>(dst) + c0, x);
            store_vec(reinterpret_cast<__nv_bfloat16 *>(dst) + c1, y);
        }
    } else if constexpr (KV == 2) {
        // e4m3 of x * (1 / scale): the product in fp32, then one rounding to
        // the nearest, limited to the type's largest value
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float(&v)[8] = j < 2 ? x : y;
            const int k = 4 * (j & 1);
            w[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[k] * inv, v[k + 1] * inv), __NV_SATFINITE,
                                                      __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[k + 2] * inv, v[k + 3] * inv),
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
            const Coder code(__half2float(h), -127.f, 127.f);
            uint8_t *blk = dst + (c >> 5) * 34;
            const int part = (c >> 3) & 3;
            if (live && part == 0) *reinterpret_cast<__half *>(blk) = h;
            uint32_t q[8];
            code(v ? y : x, q);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (live)
                    reinterpret_cast<uint16_t *>(blk + 2 + 8 * part)[j] =
                        (uint16_t)__byte_perm(q[2 * j], q[2 * j + 1], 0x0040);
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
            const Coder code(__half2float(h[v]), -8.f, 7.f);
            uint32_t q[8];
            code(v ? y : x, q);
            n[v] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) n[v] |= ((q[j] + 8u) & 15u) << (4 * j);
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
// Bound by HBM where there is enough to move: 16 x 512 bf16 rows of 8 KV heads
// and 32 of q, 128 wide (201 MB), take 35 to 37 us, a copy's rate 31.  Codes are
// bound by their instructions: 4 x 1024 rows of 8 heads to q8_0, 8.4 M values,
// take 15 us (4.3).  Few rows take one pass through memory: 64 tokens 3.2 us.
template <int KV, int N>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const __grid_constant__ AppendLaunch L) {
    const int ni = L.map.rot >> 4;
    const int rows_per_block = kThreads / L.items;
    const int item = threadIdx.x % L.items, tok = threadIdx.x / L.items;
    const int64_t row = (int64_t)blockIdx.x * rows_per_block + tok;
    bool live = tok < rows_per_block && row < (int64_t)L.B * L.Sq;
    const int b = live ? (int)((uint32_t)row / (uint32_t)L.Sq) : 0, i = live ? (int)((uint32_t)row % (uint32_t)L.Sq) : 0;
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
        item_columns<8>(L.map, item, c0, c1);
    else
        c0 = 16 * item, c1 = c0 + 8;
    if (!live) c0 = 0, c1 = 8;
    const int pos = turned && live && i < n && L.pos ? __ldg(L.pos + b * L.pos_sb + i) : (int)at;
    const auto angles = [&](float(&c)[8], float(&s)[8]) { item_angles(L.map, item, pos, c, s); };
    if (kind == 0) {
        // q: turned rows; the rows past the sequence's new ones are zeros
        if (!live || (i < n && L.q.in_place && !turned)) return;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(L.q.dst) + b * L.q.ob + i * L.q.os;
        walk_heads<__nv_bfloat16, N>(
            static_cast<const __nv_bfloat16 *>(L.q.src) + b * L.q.sb + i * L.q.ss, L.q.sh, g * L.heads,
            min(L.q.H, (g + 1) * L.heads), c0, c1, i < n, turned && i < n, L.map.interleaved, angles,
            [&](int h, const float(&x)[8], const float(&y)[8]) {
                store_vec(dst + h * L.q.oh + c0, x);
                store_vec(dst + h * L.q.oh + c1, y);
            });
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
    uint8_t *dst = static_cast<uint8_t *>(t.dst) + slot0 * row_bytes;
    walk_heads<__nv_bfloat16, N>(
        static_cast<const __nv_bfloat16 *>(t.src) + b * t.sb + i * t.ss, t.sh, g * L.heads,
        min(L.Hkv, (g + 1) * L.heads), c0, c1, live, turned && live, L.map.interleaved, angles,
        [&](int h, const float(&x)[8], const float(&y)[8]) {
            put<KV>(dst + h * 64 * row_bytes, c0, c1, split, kind == 1 ? L.k_inv : L.v_inv, x, y, live);
        });
}

// Heads that one thread walks with its sines: 8 or 4 (whole batches of loads)
// while that leaves every SM 512 threads, else one: the work is then too small
// to fill the device and the shortest thread is the fastest (64 single tokens
// appended in 4.8 us with one, 5.5 with four).
int head_group(int64_t units, int heads, int num_sms) {
    for (int g = 8; g > 2; g >>= 1)
        if (units * ((heads + g - 1) / g) >= (int64_t)num_sms * 512) return g;
    return 1;
}

template <int N>
void start_append(const AppendLaunch &L, dim3 grid, cudaStream_t stream) {
    switch (L.kv_type) {
        case 0: append_kernel<0, N><<<grid, kThreads, 0, stream>>>(L); break;
        case 2: append_kernel<2, N><<<grid, kThreads, 0, stream>>>(L); break;
        case 8: append_kernel<8, N><<<grid, kThreads, 0, stream>>>(L); break;
        default: append_kernel<4, N><<<grid, kThreads, 0, stream>>>(L); break;
    }
}

}  // namespace

cudaError_t launch_rope(RopeLaunch L, bool f32, int num_sms, cudaStream_t stream) {
    L.items = L.d / (f32 ? 2 * kVec<float> : 2 * kVec<__nv_bfloat16>);
    const int H = L.x[0].H + L.x[1].H, per = kThreads / L.items;
    const int64_t rows = (int64_t)L.B * L.S;
    L.heads = head_group(rows * L.items, H, num_sms);
    L.groups0 = (L.x[0].H + L.heads - 1) / L.heads;
    const dim3 grid((unsigned)((rows + per - 1) / per), (unsigned)(L.groups0 + (L.x[1].H + L.heads - 1) / L.heads));
    if (f32)
        L.heads == 1 ? rope_kernel<float, 1><<<grid, kThreads, 0, stream>>>(L)
                     : rope_kernel<float, kBatch><<<grid, kThreads, 0, stream>>>(L);
    else
        L.heads == 1 ? rope_kernel<__nv_bfloat16, 1><<<grid, kThreads, 0, stream>>>(L)
                     : rope_kernel<__nv_bfloat16, kBatch><<<grid, kThreads, 0, stream>>>(L);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(AppendLaunch L, int num_sms, cudaStream_t stream) {
    L.items = (L.dk > L.dv ? L.dk : L.dv) / 16;
    const int per = kThreads / L.items;
    const int64_t rows = (int64_t)L.B * L.Sq;
    L.heads = head_group(rows * L.items, L.q.H + 2 * L.Hkv, num_sms);
    L.q_groups = (L.q.H + L.heads - 1) / L.heads;
    L.kv_groups = (L.Hkv + L.heads - 1) / L.heads;
    L.k_inv = 1.f / L.k_scale;
    L.v_inv = 1.f / L.v_scale;
    const dim3 grid((unsigned)((rows + per - 1) / per), (unsigned)(L.q_groups + 2 * L.kv_groups));
    if (L.heads == 1)
        start_append<1>(L, grid, stream);
    else
        start_append<kBatch>(L, grid, stream);
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
