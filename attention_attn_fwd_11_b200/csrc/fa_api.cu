// fa_api.cu -- the exported C ABI (include/fa.h): argument validation, TMA
// tensor-map encoding, workspace sizing, and kernel launch on the caller's
// stream.  No allocation, no synchronisation, no CPU fallback.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <mutex>
#include <utility>

#include "../../include/fa.h"
#include "internal.h"
#include "overlap.h"

namespace {

thread_local char g_msg[512] = "";

fa_status fail(fa_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof g_msg, fmt, ap);
    va_end(ap);
    return st;
}

fa_status cuda_fail(cudaError_t e, const char *what) {
    return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// cuTensorMapEncodeTiled from the driver, looked up once at run time (no
// link-time dependency on libcuda).
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool get_encoder() {
    std::call_once(g_encode_once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode != nullptr;
}

// 4-D bf16 tensor (d, S, H, B) with 128-byte swizzle and a box of
// (64, box_rows, 1, 1).  Strides in elements.  Dimensions of extent 1 get a
// packed stride (their stride is never used).
fa_status encode_4d(CUtensorMap *m, const void *base, int d, int S, int H, int B, int64_t s_s, int64_t s_h,
                    int64_t s_b, int box_rows, const char *name, int elem_bytes = 2) {
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)(S > 0 ? S : 1), (cuuint64_t)H, (cuuint64_t)B};
    int64_t st[3] = {s_s, s_h, s_b};
    int64_t packed = d;
    for (int i = 0; i < 3; ++i) {
        if (dims[i + 1] == 1) st[i] = packed;
        packed = st[i] * (int64_t)dims[i + 1];
    }
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        const int64_t bytes = st[i] * elem_bytes;
        if (bytes <= 0 || bytes % 16 != 0 || bytes >= (int64_t(1) << 40))
            return fail(FA_ERR_INVALID_ARG, "%s: stride %d (%lld elements) must be a positive multiple of %d", name,
                        i, (long long)st[i], 16 / elem_bytes);
        strides[i] = (cuuint64_t)bytes;
    }
    // The box is 128 bytes wide (64 bf16 or 32 fp32 elements) and box_rows high.
    cuuint32_t box[4] = {(cuuint32_t)(128 / elem_bytes), (cuuint32_t)box_rows, 1u, 1u};
    cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    CUresult r = g_encode(m, elem_bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                          const_cast<void *>(base), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", name, (int)r);
    return FA_OK;
}

// 2-D bf16 tensor [rows, cols] (row pitch in elements), 128-byte swizzle,
// box (64, box_rows).
fa_status encode_2d(CUtensorMap *m, const void *base, int64_t cols, int64_t rows, int64_t pitch, int box_rows,
                    const char *name) {
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)(pitch * 2)};
    if ((pitch * 2) % 16 != 0) return fail(FA_ERR_INVALID_ARG, "%s: row pitch must be a multiple of 8", name);
    cuuint32_t box[2] = {64u, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1u, 1u};
    CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box,
                          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed (%d)", name, (int)r);
    return FA_OK;
}

bool finite_pos(float x) { return isfinite(x) && x > 0.f; }

// SM count of the current device, looked up once per device.
cudaError_t num_sms(int *out) {
    constexpr int kMaxDevices = 64;
    static int cache[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices && cache[dev] > 0) {
        *out = cache[dev];
        return cudaSuccess;
    }
    int n = 0;
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) cache[dev] = n;
    *out = n;
    return cudaSuccess;
}

// ---------------------------------------------------------------- paged --

// Split count of a paged decode: the caller's, clamped to the table width,
// or (num_splits == 0) enough (sequence, KV head, split) units to fill
// every SM of the current device several times over (one resident CTA an
// SM; 12 or 8 waves, below), with splits of at least 8 blocks.  The
// automatic count needs the device's SM count: FA_ERR_CUDA if it cannot be
// read.
fa_status paged_splits(const fa_decode_paged_params *p, int *out) {
    if (p->num_splits > 0) {
        *out = p->num_splits < p->max_blocks_per_seq ? p->num_splits : p->max_blocks_per_seq;
        return FA_OK;
    }
    int sms = 0;
    cudaError_t e = num_sms(&sms);
    if (e != cudaSuccess) return cuda_fail(e, "fa_decode_paged: SM count for the automatic split count");
    const long long units = (long long)p->B * p->Hkv;
    // CTAs wanted per SM: 12 for bf16 caches; 8 for quantised ones, whose
    // CTAs carry a longer fixed start (two rings to fill) and do more work
    // a block (measured on 64 sequences of 1 024-8 192 keys, 8 KV heads: 3
    // splits instead of 4 took the q8_0 decode from 0.2016 to 0.1971 ms,
    // while the bf16 one is best at 4).
    const long long per_sm = p->kv_type == FA_KV_BF16 ? 12 : 8;
    const long long want = (long long)sms * per_sm;
    long long s = (want + units - 1) / units;
    long long max_by_len = (p->max_blocks_per_seq + 7) / 8;
    if (s > max_by_len) s = max_by_len;
    if (s < 1) s = 1;
    *out = (int)s;
    return FA_OK;
}

fa_status check_paged(const fa_decode_paged_params *p) {
    if (!p) return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: params is NULL");
    if (p->B < 0 || p->Hq <= 0 || p->Hkv <= 0 || p->num_blocks <= 0 || p->max_blocks_per_seq <= 0)
        return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: B >= 0, Hq, Hkv, num_blocks, max_blocks_per_seq > 0");
    if (p->Hq % p->Hkv != 0) return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: Hq %% Hkv != 0");
    if (p->dk != 128 || p->dv != 128 || p->block_size != 64)
        return fail(FA_ERR_UNSUPPORTED, "fa_decode_paged: supported dk = dv = 128, block_size = 64 (got %d/%d/%d)",
                    p->dk, p->dv, p->block_size);
    const int g = p->Hq / p->Hkv;
    if (g != 1 && g != 2 && g != 4 && g != 8)
        return fail(FA_ERR_UNSUPPORTED, "fa_decode_paged: Hq / Hkv must be 1, 2, 4 or 8 (got %d)", g);
    if (!finite_pos(p->scale)) return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: scale must be finite and > 0");
    if (p->o_dtype != FA_F32 && p->o_dtype != FA_BF16) return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: o_dtype");
    if (p->kv_type != FA_KV_BF16 && p->kv_type != FA_KV_Q8_0 && p->kv_type != FA_KV_Q4_0 &&
        p->kv_type != FA_KV_FP8_E4M3)
        return fail(FA_ERR_UNSUPPORTED,
                    "fa_decode_paged: kv_type must be FA_KV_BF16, FA_KV_Q8_0, FA_KV_Q4_0 or FA_KV_FP8_E4M3 (got %d)",
                    p->kv_type);
    if (p->kv_type == FA_KV_FP8_E4M3 && (!isfinite(p->k_scale) || !isfinite(p->v_scale)))
        return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: k_scale and v_scale must be finite");
    return FA_OK;
}

// Shapes (above) plus the tensor pointers, for the compute call.
fa_status check_paged_ptrs(const fa_decode_paged_params *p) {
    fa_status st = check_paged(p);
    if (st != FA_OK || p->B == 0) return st;
    if (!p->q || !p->k_cache || !p->v_cache || !p->block_table || !p->seq_lens || !p->o)
        return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: NULL tensor pointer");
    if (!aligned16(p->q) || !aligned16(p->k_cache) || !aligned16(p->v_cache) || !aligned16(p->o))
        return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: q, caches and o must be 16-byte aligned");
    if (((uintptr_t)p->lse & 3u) || ((uintptr_t)p->block_table & 3u) || ((uintptr_t)p->seq_lens & 3u))
        return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: lse, block_table, seq_lens must be 4-byte aligned");
    return FA_OK;
}

// Both caches as 2-D [num_blocks * Hkv * 64 rows, 128] bf16 tensors for TMA
// (128-byte swizzle, 64 x 64 boxes).
fa_status encode_paged_caches(const fa_decode_paged_params *p, fa::PagedLaunch *L) {
    memset(L, 0, sizeof *L);
    if (p->kv_type != FA_KV_BF16) {  // bulk-copied raw tiles: no tensor maps
        L->kv_type = p->kv_type;
        L->k_scale = p->k_scale;
        L->v_scale = p->v_scale;
        return FA_OK;
    }
    if (!get_encoder()) return fail(FA_ERR_CUDA, "fa_decode_paged: cuTensorMapEncodeTiled is not available");
    const int64_t rows = (int64_t)p->num_blocks * p->Hkv * p->block_size;
    if (rows >= (int64_t(1) << 31))
        return fail(FA_ERR_INVALID_ARG, "fa_decode_paged: num_blocks * Hkv * block_size must be < 2^31");
    fa_status st = encode_2d(&L->tmK, p->k_cache, p->dk, rows, p->dk, 64, "fa_decode_paged k_cache");
    if (st != FA_OK) return st;
    return encode_2d(&L->tmV, p->v_cache, p->dv, rows, p->dv, 64, "fa_decode_paged v_cache");
}

// Everything a paged-decode launch needs except where its split partials
// go (shared by fa_decode_paged, fa_decode_paged_noalloc and the timeout
// test hook).
fa_status paged_launch_setup(const fa_decode_paged_params *p, int splits, fa::PagedLaunch *L) {
    fa_status st = encode_paged_caches(p, L);
    if (st != FA_OK) return st;
    L->q = p->q;
    L->k_cache = p->k_cache;
    L->v_cache = p->v_cache;
    L->block_table = p->block_table;
    L->seq_lens = p->seq_lens;
    L->max_blocks_per_seq = p->max_blocks_per_seq;
    L->B = p->B;
    L->Hq = p->Hq;
    L->Hkv = p->Hkv;
    L->num_blocks = p->num_blocks;
    L->scale = p->scale;
    L->num_splits = splits;
    L->blocks_per_split = (p->max_blocks_per_seq + splits - 1) / splits;
    L->o = p->o;
    L->lse = p->lse;
    L->o_bf16 = p->o_dtype == FA_BF16;
    L->part_o = nullptr;
    L->part_lse = nullptr;
    return FA_OK;
}

// Byte offset of the partial LSEs in a paged workspace of `splits` splits.
size_t paged_lse_offset(const fa_decode_paged_params *p, int splits) {
    const size_t rows = (size_t)p->B * p->Hq * (size_t)splits;
    return (rows * 128 * sizeof(float) + 255) & ~size_t(255);
}

size_t paged_ws_bytes(const fa_decode_paged_params *p, int splits) {
    const size_t rows = (size_t)p->B * p->Hq * (size_t)splits;
    size_t o = rows * 128 * sizeof(float);
    o = (o + 255) & ~size_t(255);
    return o + ((rows * sizeof(float) + 255) & ~size_t(255));
}

// --------------------------------------------------------------- gather --

// Split count of a latent decode: the caller's, clamped to one split per 64
// keys, or (num_splits == 0) one two-CTA cluster per (token, split) and at
// most one wave of clusters (half the device's SMs), with at least 128
// keys per split.
fa_status gather_splits(const fa_decode_gather_params *p, int *out) {
    const int max_s = (p->topk + 63) / 64 > 0 ? (p->topk + 63) / 64 : 1;
    if (p->num_splits > 0) {
        *out = p->num_splits < max_s ? p->num_splits : max_s;
        return FA_OK;
    }
    int sms = 0;
    cudaError_t e = num_sms(&sms);
    if (e != cudaSuccess) return cuda_fail(e, "fa_decode_gather: SM count for the automatic split count");
    const long long want = sms / 2 > 0 ? sms / 2 : 1;
    const long long T = p->T > 0 ? p->T : 1;
    long long s = want / T;
    long long max_by_len = (p->topk + 127) / 128;
    if (s > max_by_len) s = max_by_len;
    if (s < 1) s = 1;
    *out = (int)s;
    return FA_OK;
}

fa_status check_gather(const fa_decode_gather_params *p) {
    if (!p) return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: params is NULL");
    if (p->T < 0 || p->Hq <= 0 || p->topk < 0 || p->n_rows <= 0)
        return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: T >= 0, Hq > 0, topk >= 0, n_rows > 0");
    const bool lat576 = p->dk == 576 && p->dv == 512 && p->v_offset == 64;
    const bool lat512 = p->dk == 512 && p->dv == 512 && p->v_offset == 0;
    if (!(lat576 || lat512) || p->Hq != 128)
        return fail(FA_ERR_UNSUPPORTED,
                    "fa_decode_gather: supported (dk, dv, v_offset) = (576, 512, 64) or (512, 512, 0), Hq = 128");
    if (p->row_stride < p->dk || p->row_stride % 8 != 0)
        return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: row_stride must be >= dk and a multiple of 8");
    if (p->n_rows > 0x7fffffffLL) return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: n_rows must fit in int32");
    if (!finite_pos(p->scale)) return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: scale must be finite and > 0");
    if (p->o_dtype != FA_F32 && p->o_dtype != FA_BF16) return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: o_dtype");
    return FA_OK;
}

fa_status check_gather_ptrs(const fa_decode_gather_params *p) {
    fa_status st = check_gather(p);
    if (st != FA_OK || p->T == 0) return st;
    if (!p->q || !p->kv_rows || !p->o)
        return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: NULL tensor pointer");
    if (!p->idx && p->topk > p->n_rows)
        return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: with idx NULL, topk (%d) must be <= n_rows", p->topk);
    if (!aligned16(p->q) || !aligned16(p->kv_rows) || !aligned16(p->o))
        return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: q, kv_rows and o must be 16-byte aligned");
    if (((uintptr_t)p->lse & 3u) || ((uintptr_t)p->idx & 3u) || ((uintptr_t)p->key_pos & 3u) ||
        ((uintptr_t)p->q_pos & 3u))
        return fail(FA_ERR_INVALID_ARG, "fa_decode_gather: lse, idx, key_pos, q_pos must be 4-byte aligned");
    return FA_OK;
}

size_t gather_ws_bytes(const fa_decode_gather_params *p, int splits) {
    const size_t rows = (size_t)p->T * p->Hq * (size_t)splits;
    size_t o = rows * 512 * sizeof(float);
    o = (o + 255) & ~size_t(255);
    return o + ((rows * sizeof(float) + 255) & ~size_t(255));
}

fa_status check_tail(const fa_mla_tail_params *p) {
    if (!p) return fail(FA_ERR_INVALID_ARG, "fa_mla_tail: params is NULL");
    if (p->T < 0 || p->Hq <= 0 || p->R <= 0 || p->V <= 0 || p->Hd <= 0)
        return fail(FA_ERR_INVALID_ARG, "fa_mla_tail: need T >= 0 and Hq, R, V, Hd > 0");
    if (p->V != 128 || p->R % 64 != 0 || p->Hd % 128 != 0 || ((int64_t)p->Hq * p->V) % 64 != 0)
        return fail(FA_ERR_UNSUPPORTED, "fa_mla_tail: supported V = 128, R % 64 == 0, Hd % 128 == 0 (got V %d R %d Hd %d)",
                    p->V, p->R, p->Hd);
    if ((int64_t)p->T * p->Hq > 0x7fffffffLL) return fail(FA_ERR_INVALID_ARG, "fa_mla_tail: T * Hq out of range");
    if ((int64_t)p->Hq * p->V > (1 << 30) || p->R > (1 << 20) || p->Hd > (1 << 24))
        return fail(FA_ERR_INVALID_ARG, "fa_mla_tail: sizes out of range");
    if (p->y_dtype != FA_F32 && p->y_dtype != FA_BF16) return fail(FA_ERR_INVALID_ARG, "fa_mla_tail: y_dtype");
    if (p->num_splits < 0) return fail(FA_ERR_INVALID_ARG, "fa_mla_tail: num_splits must be >= 0");
    return FA_OK;
}

// ------------------------------------------------- rotary, cache append --

// The rotation of a call: frequencies to 64-bit fractions of a turn.
fa_status make_rope_map(const char *who, const double *inv_freq, int rot, int offset, int d, int interleaved,
                        int inverse, float mscale, fa::RopeMap *m) {
    if (rot <= 0 || rot % 16 != 0 || rot > fa::kMaxRot || offset < 0 || offset % 16 != 0 || offset > d - rot)
        return fail(FA_ERR_UNSUPPORTED,
                    "%s: rot_dim and rot_offset must be multiples of 16, rot_dim in (0, %d], rot_offset + rot_dim <= d "
                    "(got %d, %d)",
                    who, fa::kMaxRot, rot, offset);
    if (!isfinite(mscale)) return fail(FA_ERR_INVALID_ARG, "%s: mscale must be finite", who);
    for (int i = 0; i < rot / 2; ++i) {
        if (!isfinite(inv_freq[i])) return fail(FA_ERR_INVALID_ARG, "%s: inv_freq[%d] is not finite", who, i);
        // The fraction is below 1 and has at most 64 significant bits, so the
        // scaled value fits.
        long double x = (long double)inv_freq[i] * 0.159154943091895335768883763372514362L;  // 1 / (2 pi)
        if (!(x >= 0.0L && x < 1.0L)) x -= floorl(x);
        m->turns[i] = x < 1.0L ? (uint64_t)(x * 18446744073709551616.0L) : 0;
    }
    m->rot = rot;
    m->offset = offset;
    m->interleaved = interleaved != 0;
    m->inverse = inverse != 0;
    m->mscale = mscale;
    return FA_OK;
}

// A tensor [B, H, S, .] of a rotary call: pointers and strides in units of
// 16 bytes (`unit` elements).  Dimensions of extent 1 may have any stride.
fa_status check_rows(const char *who, const char *name, const void *src, int64_t sb, int64_t sh, int64_t ss, int B,
                     int H, int S, int unit) {
    if (!src) return fail(FA_ERR_INVALID_ARG, "%s: %s is NULL", who, name);
    if (!aligned16(src)) return fail(FA_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", who, name);
    if ((B > 1 && sb % unit) || (H > 1 && sh % unit) || (S > 1 && ss % unit))
        return fail(FA_ERR_INVALID_ARG, "%s: %s strides must be multiples of %d elements", who, name, unit);
    constexpr int64_t far = int64_t(1) << 40;
    if ((B > 1 && (sb > far || sb < -far)) || (H > 1 && (sh > far || sh < -far)) || (S > 1 && (ss > far || ss < -far)))
        return fail(FA_ERR_INVALID_ARG, "%s: %s strides out of range", who, name);
    return FA_OK;
}

// What such a tensor covers (strides in elements of `bytes` bytes).
fa::Rows byte_rows(const void *p, int64_t sb, int64_t sh, int64_t ss, int B, int H, int S, int d, int bytes) {
    return fa::Rows{p, (int64_t)d * bytes, {B, H, S}, {sb * bytes, sh * bytes, ss * bytes}};
}

fa_status rope_tensor(const char *who, const char *name, const void *src, void *dst, int64_t sb, int64_t sh,
                      int64_t ss, int64_t ob, int64_t oh, int64_t os, int B, int H, int S, int d, int unit,
                      fa::RopeTensor *t) {
    fa_status st = check_rows(who, name, src, sb, sh, ss, B, H, S, unit);
    if (st == FA_OK) st = check_rows(who, name, dst, ob, oh, os, B, H, S, unit);
    if (st != FA_OK) return st;
    const bool same = (B == 1 || sb == ob) && (H == 1 || sh == oh) && (S == 1 || ss == os);
    const int bytes = 16 / unit;
    const fa::Rows to = byte_rows(dst, ob, oh, os, B, H, S, d, bytes);
    if (fa::rows_meet_themselves(to)) return fail(FA_ERR_INVALID_ARG, "%s: the rows of %s's output overlap", who, name);
    if (src == dst && !same)
        return fail(FA_ERR_INVALID_ARG, "%s: %s turned in place needs equal strides", who, name);
    if (src != dst && fa::rows_meet(to, byte_rows(src, sb, sh, ss, B, H, S, d, bytes)))
        return fail(FA_ERR_INVALID_ARG, "%s: %s's output and its input overlap and are not the same rows", who, name);
    *t = fa::RopeTensor{src, dst, H, sb, sh, ss, ob, oh, os, src == dst};
    return FA_OK;
}

// -------------------------------------------------------------- backward --

fa_status check_bwd(const fa_bwd_params *p) {
    if (!p) return fail(FA_ERR_INVALID_ARG, "fa_bwd: params is NULL");
    if (p->B < 0 || p->Hq <= 0 || p->Hkv <= 0 || p->Sq < 0 || p->Sk < 0)
        return fail(FA_ERR_INVALID_ARG, "fa_bwd: need B >= 0, Hq > 0, Hkv > 0, Sq >= 0, Sk >= 0");
    if (p->Hq % p->Hkv != 0) return fail(FA_ERR_INVALID_ARG, "fa_bwd: Hq (%d) %% Hkv (%d) != 0", p->Hq, p->Hkv);
    if (!((p->dk == 64 && p->dv == 64) || (p->dk == 128 && p->dv == 128) || (p->dk == 192 && p->dv == 128)))
        return fail(FA_ERR_UNSUPPORTED, "fa_bwd: supported (dk, dv) = (64, 64), (128, 128), (192, 128); got (%d, %d)",
                    p->dk, p->dv);
    if (!finite_pos(p->scale)) return fail(FA_ERR_INVALID_ARG, "fa_bwd: scale must be finite and > 0");
    if ((p->o_dtype != FA_F32 && p->o_dtype != FA_BF16) || (p->g_dtype != FA_F32 && p->g_dtype != FA_BF16))
        return fail(FA_ERR_INVALID_ARG, "fa_bwd: o_dtype, g_dtype");
    if (p->Sq > (1 << 30) || p->Sk > (1 << 30) ||
        ((int64_t)p->Sq / 64 + 2) * (int64_t)p->B * p->Hq > 0x3fffffffLL ||
        ((int64_t)p->Sk / 64 + 2) * (int64_t)p->B * p->Hkv > 0x3fffffffLL)
        return fail(FA_ERR_INVALID_ARG, "fa_bwd: sizes out of range");
    if (!isfinite(p->max_bias) || p->max_bias < 0.f || !isfinite(p->softcap) || p->softcap < 0.f)
        return fail(FA_ERR_INVALID_ARG, "fa_bwd: max_bias and softcap must be finite and >= 0");
    return FA_OK;
}

size_t bwd_row_bytes(const fa_bwd_params *p) {  // of the row LSE, of D, and a quarter of both as bf16 pieces
    const size_t n = (size_t)p->B * p->Hq * (size_t)fa::bwd_pitch(p->Sq) * sizeof(float);
    return (n + 255) & ~size_t(255);
}

// The rows' LSE and D, the tile counter, and the parts of walks that are cut.
size_t bwd_bytes(const fa_bwd_params *p, bool causal) {
    return 6 * bwd_row_bytes(p) + 256 +
           fa::bwd_split(p->B, p->Hq, p->Hkv, p->Sq, p->Sk, p->dk, p->dv, causal).bytes(p->dk, p->dv);
}

// A gradient's strides: vector stores of 16 bytes, rows that do not overlap.
// Dimensions of extent 1 may have any stride.
fa_status check_grad(const char *name, const void *g, int64_t sb, int64_t sh, int64_t ss, int B, int H, int S, int d,
                     int unit) {
    if (!g || !aligned16(g)) return fail(FA_ERR_INVALID_ARG, "fa_bwd: %s is NULL or not 16-byte aligned", name);
    int64_t st[3] = {sb, sh, ss}, n[3] = {B, H, S};
    int64_t span = d;  // elements from the first to the last of the dimensions looked at
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)  // extents of 1 first, then by stride
            if (n[i] > 1 && (n[j] == 1 || st[j] < st[i])) {
                std::swap(st[i], st[j]);
                std::swap(n[i], n[j]);
            }
        if (n[i] == 1) continue;
        if (st[i] % unit)
            return fail(FA_ERR_INVALID_ARG, "fa_bwd: %s strides must be multiples of %d elements", name, unit);
        if (st[i] < span) return fail(FA_ERR_INVALID_ARG, "fa_bwd: the rows of %s overlap", name);
        if (st[i] > (int64_t(1) << 40)) return fail(FA_ERR_INVALID_ARG, "fa_bwd: %s strides out of range", name);
        span += (n[i] - 1) * st[i];
    }
    return FA_OK;
}

// What fa_bwd writes -- the gradients, the sinks' gradient, the workspace --
// against all that it reads and one another.
fa_status check_bwd_apart(const fa_bwd_params *p, bool rows, bool keys, size_t ws_bytes) {
    struct Named {
        const char *name;
        fa::Rows r;
    } x[15];
    int n = 0;
    const auto put = [&](const char *name, const void *t, int64_t sb, int64_t sh, int64_t ss, int H, int S, int d, int bytes) {
        if (t && p->B > 0 && S > 0) x[n++] = Named{name, byte_rows(t, sb, sh, ss, p->B, H, S, d, bytes)};
    };
    const auto flat = [&](const char *name, const void *t, int64_t bytes) {
        if (t && bytes > 0) x[n++] = Named{name, fa::Rows{t, bytes, {1, 1, 1}, {0, 0, 0}}};
    };
    const int gb = p->g_dtype == FA_F32 ? 4 : 2, Sq = rows ? p->Sq : 0, Sk = keys ? p->Sk : 0;
    put("gq", p->gq, p->gq_sb, p->gq_sh, p->gq_ss, p->Hq, Sq, p->dk, gb);
    put("gk", p->gk, p->gk_sb, p->gk_sh, p->gk_ss, p->Hkv, Sk, p->dk, gb);
    put("gv", p->gv, p->gv_sb, p->gv_sh, p->gv_ss, p->Hkv, Sk, p->dv, gb);
    flat("gsinks", p->gsinks, 4 * (int64_t)p->Hq);
    flat("the workspace", p->workspace, (int64_t)ws_bytes);
    const int written = n;
    put("q", p->q, p->q_sb, p->q_sh, p->q_ss, p->Hq, Sq, p->dk, 2);
    put("k", p->k, p->k_sb, p->k_sh, p->k_ss, p->Hkv, Sk, p->dk, 2);
    put("v", p->v, p->v_sb, p->v_sh, p->v_ss, p->Hkv, Sk, p->dv, 2);
    put("o", p->o, p->o_sb, p->o_sh, p->o_ss, p->Hq, Sq, p->dv, p->o_dtype == FA_F32 ? 4 : 2);
    put("dout", p->dout, p->do_sb, p->do_sh, p->do_ss, p->Hq, Sq, p->dv, 2);
    flat("lse", p->lse, 4 * (int64_t)p->B * p->Hq * Sq);
    flat("dlse", p->dlse, 4 * (int64_t)p->B * p->Hq * Sq);
    flat("sinks", p->sinks, 4 * (int64_t)p->Hq);
    if (Sk > 0) put("mask", p->mask, p->m_sb, p->m_sh, p->m_ss, p->Hq, Sq, Sk, 2);
    for (int i = 0; i < written; ++i)
        for (int j = i + 1; j < n; ++j)
            if (fa::rows_meet(x[i].r, x[j].r))
                return fail(FA_ERR_INVALID_ARG, "fa_bwd: %s must be apart from %s", x[i].name, x[j].name);
    return FA_OK;
}

}  // namespace

extern "C" {

int fa_version(void) { return 100; }

const char *fa_last_error(void) { return g_msg; }

fa_status fa_fwd(const fa_fwd_params *p, void *stream) {
    if (!p) return fail(FA_ERR_INVALID_ARG, "fa_fwd: params is NULL");
    if (p->B < 0 || p->Hq <= 0 || p->Hkv <= 0 || p->Sq < 0 || p->Sk < 0)
        return fail(FA_ERR_INVALID_ARG, "fa_fwd: need B >= 0, Hq > 0, Hkv > 0, Sq >= 0, Sk >= 0");
    if (p->Hq % p->Hkv != 0) return fail(FA_ERR_INVALID_ARG, "fa_fwd: Hq (%d) %% Hkv (%d) != 0", p->Hq, p->Hkv);
    const bool d512 = p->dv == 512 && (p->dk == 576 || p->dk == 512);
    const bool pair_ok = (p->dk == p->dv && (p->dk == 64 || p->dk == 128 || p->dk == 256)) ||
                         (p->dk == 192 && (p->dv == 128 || p->dv == 192)) || (p->dk == 320 && p->dv == 256) || d512;
    if (!pair_ok)
        return fail(FA_ERR_UNSUPPORTED,
                    "fa_fwd: supported (dk, dv) = (64, 64), (128, 128), (192, 192), (256, 256), (192, 128), (320, 256), "
                    "(576, 512), (512, 512); got (%d, %d)",
                    p->dk, p->dv);
    if (d512 && (p->mask || p->softcap != 0.f || p->sinks || p->max_bias != 0.f))
        return fail(FA_ERR_UNSUPPORTED, "fa_fwd: score modifiers are not supported with dv = 512");
    if (!finite_pos(p->scale)) return fail(FA_ERR_INVALID_ARG, "fa_fwd: scale must be finite and > 0");
    if (p->o_dtype != FA_F32 && p->o_dtype != FA_BF16) return fail(FA_ERR_INVALID_ARG, "fa_fwd: o_dtype");
    if ((long long)p->B * p->Hq > 0x7fffffffLL || p->Sq > (1 << 30) || p->Sk > (1 << 30))
        return fail(FA_ERR_INVALID_ARG, "fa_fwd: sizes out of range");
    if (p->B == 0 || p->Sq == 0) return FA_OK;
    // k and v are never read when Sk == 0 (they may then be NULL).
    if (!p->q || !p->o || (p->Sk > 0 && (!p->k || !p->v)))
        return fail(FA_ERR_INVALID_ARG, "fa_fwd: NULL tensor pointer");
    if (!aligned16(p->q) || !aligned16(p->o) || (p->Sk > 0 && (!aligned16(p->k) || !aligned16(p->v))))
        return fail(FA_ERR_INVALID_ARG, "fa_fwd: q, k, v, o must be 16-byte aligned");
    if ((uintptr_t)p->lse & 3u) return fail(FA_ERR_INVALID_ARG, "fa_fwd: lse must be 4-byte aligned");
    const int ovec = p->o_dtype == FA_F32 ? 4 : 8;
    if (p->o_ss % ovec || p->o_sh % ovec || p->o_sb % ovec || p->o_ss < p->dv)
        return fail(FA_ERR_INVALID_ARG, "fa_fwd: o strides must be multiples of %d elements and o_ss >= dv", ovec);
    if (!isfinite(p->max_bias) || p->max_bias < 0.f || !isfinite(p->softcap) || p->softcap < 0.f)
        return fail(FA_ERR_INVALID_ARG, "fa_fwd: max_bias and softcap must be finite and >= 0");
    if (p->mask && (!aligned16(p->mask) || p->m_ss % 8 || p->m_sh % 8 || p->m_sb % 8 || p->m_ss < p->Sk ||
                    p->m_sh < 0 || p->m_sb < 0))
        return fail(FA_ERR_INVALID_ARG,
                    "fa_fwd: mask must be 16-byte aligned, its strides multiples of 8 elements, m_ss >= Sk");
    if ((uintptr_t)p->sinks & 3u) return fail(FA_ERR_INVALID_ARG, "fa_fwd: sinks must be 4-byte aligned");
    if (!get_encoder()) return fail(FA_ERR_CUDA, "fa_fwd: cuTensorMapEncodeTiled is not available");

    if (d512) {
        // The latent kernel's CTA pair: each CTA keeps half of the 512-wide O
        // in TMEM and the pair splits the dk-wide score contraction by columns.
        fa::Dense512Launch D;
        memset(&D, 0, sizeof D);
        fa_status st = encode_4d(&D.tmQ, p->q, p->dk, p->Sq, p->Hq, p->B, p->q_ss, p->q_sh, p->q_sb, 128, "fa_fwd q");
        if (st != FA_OK) return st;
        const void *kb = p->Sk > 0 ? p->k : p->q;
        const void *vb = p->Sk > 0 ? p->v : p->q;
        st = encode_4d(&D.tmK, kb, p->dk, p->Sk, p->Hkv, p->B, p->k_ss, p->k_sh, p->k_sb, 32, "fa_fwd k");
        if (st != FA_OK) return st;
        st = encode_4d(&D.tmV, vb, p->dv, p->Sk, p->Hkv, p->B, p->v_ss, p->v_sh, p->v_sb, 32, "fa_fwd v");
        if (st != FA_OK) return st;
        st = encode_4d(&D.tmO, p->o, p->dv, p->Sq, p->Hq, p->B, p->o_ss, p->o_sh, p->o_sb, 32, "fa_fwd o",
                       p->o_dtype == FA_F32 ? 4 : 2);
        if (st != FA_OK) return st;
        if ((long long)p->B * p->Hq > 65535 || (p->Sq + 127) / 128 > 65535)
            return fail(FA_ERR_INVALID_ARG, "fa_fwd: B * Hq and ceil(Sq / 128) must be <= 65535 for dv = 512");
        D.B = p->B;
        D.Hq = p->Hq;
        D.Hkv = p->Hkv;
        D.Sq = p->Sq;
        D.Sk = p->Sk;
        D.dk = p->dk;
        D.scale = p->scale;
        D.causal = p->causal ? 1 : 0;
        D.o = p->o;
        D.o_sb = p->o_sb;
        D.o_sh = p->o_sh;
        D.o_ss = p->o_ss;
        D.o_bf16 = p->o_dtype == FA_BF16;
        D.lse = p->lse;
        cudaError_t e = fa::launch_prefill_d512(D, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return cuda_fail(e, "fa_fwd: launch");
        return FA_OK;
    }

    fa::PrefillLaunch L;
    memset(&L, 0, sizeof L);
    // The two-tile kernel takes dk = dv <= 128 (K/V tiles of 128 keys); the
    // one-tile kernel the rest (64-key tiles, except 128 for (192, 128)).
    const bool two_tile = p->dk == p->dv && p->dk <= 128;
    const int box_k = two_tile || (p->dk == 192 && p->dv == 128) ? 128 : 64;
    fa_status st;
    st = encode_4d(&L.tmQ, p->q, p->dk, p->Sq, p->Hq, p->B, p->q_ss, p->q_sh, p->q_sb, 128, "fa_fwd q");
    if (st != FA_OK) return st;
    // With Sk == 0 no K/V tile is ever loaded; any valid map will do.
    const void *kb = p->Sk > 0 ? p->k : p->q;
    const void *vb = p->Sk > 0 ? p->v : p->q;
    st = encode_4d(&L.tmK, kb, p->dk, p->Sk, p->Hkv, p->B, p->k_ss, p->k_sh, p->k_sb, box_k, "fa_fwd k");
    if (st != FA_OK) return st;
    st = encode_4d(&L.tmV, vb, p->dv, p->Sk, p->Hkv, p->B, p->v_ss, p->v_sh, p->v_sb, box_k, "fa_fwd v");
    if (st != FA_OK) return st;
    if (two_tile) {  // the two-tile kernel writes O with TMA stores
        st = encode_4d(&L.tmO, p->o, p->dv, p->Sq, p->Hq, p->B, p->o_ss, p->o_sh, p->o_sb, 128, "fa_fwd o",
                       p->o_dtype == FA_F32 ? 4 : 2);
        if (st != FA_OK) return st;
    }
    L.B = p->B;
    L.Hq = p->Hq;
    L.Hkv = p->Hkv;
    L.Sq = p->Sq;
    L.Sk = p->Sk;
    L.dk = p->dk;
    L.dv = p->dv;
    L.scale = p->scale;
    L.causal = p->causal ? 1 : 0;
    L.o = p->o;
    L.o_sb = p->o_sb;
    L.o_sh = p->o_sh;
    L.o_ss = p->o_ss;
    L.o_bf16 = p->o_dtype == FA_BF16;
    L.lse = p->lse;
    L.mods.mask = static_cast<const __half *>(p->mask);
    L.mods.m_sb = p->m_sb;
    L.mods.m_sh = p->m_sh;
    L.mods.m_ss = p->m_ss;
    L.mods.softcap = p->softcap;
    L.mods.sinks = p->sinks;
    if (p->max_bias > 0.f) {  // ALiBi bases, as read in score_mods.cuh
        int n2 = 1;
        while (n2 * 2 <= p->Hq) n2 *= 2;
        L.mods.n_head_log2 = n2;
        L.mods.log2_m0 = -p->max_bias / (float)n2;
        L.mods.log2_m1 = -p->max_bias / 2.f / (float)n2;
    }
    L.has_mods = p->mask || p->softcap > 0.f || p->sinks;
    if (two_tile && p->mask && p->Sk > 0) {
        // Head and batch dimensions of stride 0 are broadcast: size 1, coordinate 0.
        st = encode_4d(&L.tmM, p->mask, p->Sk, p->Sq, p->m_sh ? p->Hq : 1, p->m_sb ? p->B : 1, p->m_ss,
                       p->m_sh ? p->m_sh : p->m_ss * p->Sq, p->m_sb ? p->m_sb : p->m_ss * p->Sq, 128, "fa_fwd mask");
        if (st != FA_OK) return st;
        L.mask_staged = true;
    }
    cudaError_t e;
    if (two_tile) {
        int sms = 0;
        e = num_sms(&sms);
        if (e == cudaSuccess) e = fa::launch_prefill2(L, sms, static_cast<cudaStream_t>(stream));
    } else {
        e = fa::launch_prefill(L, static_cast<cudaStream_t>(stream));
    }
    if (e != cudaSuccess) return cuda_fail(e, "fa_fwd: launch");
    return FA_OK;
}

fa_status fa_prefill_paged(const fa_prefill_paged_params *p, void *stream) {
    if (!p) return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: params is NULL");
    if (p->B < 0 || p->Hq <= 0 || p->Hkv <= 0 || p->Sq < 0 || p->num_blocks <= 0 || p->max_blocks_per_seq <= 0)
        return fail(FA_ERR_INVALID_ARG,
                    "fa_prefill_paged: need B >= 0, Hq > 0, Hkv > 0, Sq >= 0, num_blocks > 0, max_blocks_per_seq > 0");
    if (p->Hq % p->Hkv != 0)
        return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: Hq (%d) %% Hkv (%d) != 0", p->Hq, p->Hkv);
    const bool pair_ok = (p->dk == p->dv && (p->dk == 64 || p->dk == 128 || p->dk == 256)) ||
                         (p->dk == 192 && (p->dv == 128 || p->dv == 192)) || (p->dk == 320 && p->dv == 256);
    if (!pair_ok || p->block_size != 64)
        return fail(FA_ERR_UNSUPPORTED,
                    "fa_prefill_paged: supported (dk, dv) as fa_fwd, block_size = 64 (got %d/%d/%d)", p->dk, p->dv,
                    p->block_size);
    const bool two_tile = p->dk == p->dv && p->dk <= 128;
    if (!finite_pos(p->scale)) return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: scale must be finite and > 0");
    if (p->o_dtype != FA_F32 && p->o_dtype != FA_BF16) return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: o_dtype");
    if ((long long)p->B * p->Hq > 0x7fffffffLL || p->Sq > (1 << 30) ||
        (long long)p->max_blocks_per_seq * p->block_size > (1 << 30) || (long long)p->B * p->max_blocks_per_seq > 0x7fffffffLL)
        return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: sizes out of range");
    if (p->B == 0 || p->Sq == 0) return FA_OK;
    if (!p->q || !p->o || !p->k_cache || !p->v_cache || !p->block_table || !p->seq_lens)
        return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: NULL tensor pointer");
    if (!aligned16(p->q) || !aligned16(p->o) || !aligned16(p->k_cache) || !aligned16(p->v_cache))
        return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: q, caches and o must be 16-byte aligned");
    if (((uintptr_t)p->lse | (uintptr_t)p->block_table | (uintptr_t)p->seq_lens | (uintptr_t)p->q_lens) & 3u)
        return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: lse, block_table, seq_lens, q_lens must be 4-byte aligned");
    const int ovec = p->o_dtype == FA_F32 ? 4 : 8;
    if (p->o_ss % ovec || p->o_sh % ovec || p->o_sb % ovec || p->o_ss < p->dv)
        return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: o strides must be multiples of %d elements and o_ss >= dv",
                    ovec);
    if (!get_encoder()) return fail(FA_ERR_CUDA, "fa_prefill_paged: cuTensorMapEncodeTiled is not available");

    fa::PrefillLaunch L;
    memset(&L, 0, sizeof L);
    fa_status st;
    st = encode_4d(&L.tmQ, p->q, p->dk, p->Sq, p->Hq, p->B, p->q_ss, p->q_sh, p->q_sb, 128, "fa_prefill_paged q");
    if (st != FA_OK) return st;
    // The caches as (d, 64 slots, Hkv, num_blocks), 64-row boxes.
    const int64_t bs = p->block_size;
    st = encode_4d(&L.tmK, p->k_cache, p->dk, p->block_size, p->Hkv, p->num_blocks, p->dk, bs * p->dk,
                   bs * p->dk * p->Hkv, 64, "fa_prefill_paged k_cache");
    if (st != FA_OK) return st;
    st = encode_4d(&L.tmV, p->v_cache, p->dv, p->block_size, p->Hkv, p->num_blocks, p->dv, bs * p->dv,
                   bs * p->dv * p->Hkv, 64, "fa_prefill_paged v_cache");
    if (st != FA_OK) return st;
    if (two_tile) {  // the two-tile kernel writes O with TMA stores
        st = encode_4d(&L.tmO, p->o, p->dv, p->Sq, p->Hq, p->B, p->o_ss, p->o_sh, p->o_sb, 128, "fa_prefill_paged o",
                       p->o_dtype == FA_F32 ? 4 : 2);
        if (st != FA_OK) return st;
    }
    L.B = p->B;
    L.Hq = p->Hq;
    L.Hkv = p->Hkv;
    L.Sq = p->Sq;
    L.Sk = 0;
    L.dk = p->dk;
    L.dv = p->dv;
    L.scale = p->scale;
    L.causal = p->causal ? 1 : 0;
    L.o = p->o;
    L.o_sb = p->o_sb;
    L.o_sh = p->o_sh;
    L.o_ss = p->o_ss;
    L.o_bf16 = p->o_dtype == FA_BF16;
    L.lse = p->lse;
    if (!isfinite(p->max_bias) || p->max_bias < 0.f || !isfinite(p->softcap) || p->softcap < 0.f)
        return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: max_bias and softcap must be finite and >= 0");
    if (p->mask && (!aligned16(p->mask) || p->m_ss % 8 || p->m_sh % 8 || p->m_sb % 8 || p->m_ss <= 0 ||
                    p->m_sh < 0 || p->m_sb < 0))
        return fail(FA_ERR_INVALID_ARG,
                    "fa_prefill_paged: mask must be 16-byte aligned, its strides multiples of 8 elements, m_ss > 0");
    if ((uintptr_t)p->sinks & 3u) return fail(FA_ERR_INVALID_ARG, "fa_prefill_paged: sinks must be 4-byte aligned");
    L.mods.mask = static_cast<const __half *>(p->mask);
    L.mods.m_sb = p->m_sb;
    L.mods.m_sh = p->m_sh;
    L.mods.m_ss = p->m_ss;
    L.mods.softcap = p->softcap;
    L.mods.sinks = p->sinks;
    if (p->max_bias > 0.f) {  // ALiBi bases, as read in score_mods.cuh
        int n2 = 1;
        while (n2 * 2 <= p->Hq) n2 *= 2;
        L.mods.n_head_log2 = n2;
        L.mods.log2_m0 = -p->max_bias / (float)n2;
        L.mods.log2_m1 = -p->max_bias / 2.f / (float)n2;
    }
    L.has_mods = p->mask || p->softcap > 0.f || p->sinks;
    if (p->mask && two_tile) {
        // (keys, new rows, heads, batch) with rows m_ss long; stride-0 dims broadcast
        st = encode_4d(&L.tmM, p->mask, (int)(p->m_ss < (1 << 30) ? p->m_ss : (1 << 30)), p->Sq,
                       p->m_sh ? p->Hq : 1, p->m_sb ? p->B : 1, p->m_ss, p->m_sh ? p->m_sh : p->m_ss * p->Sq,
                       p->m_sb ? p->m_sb : p->m_ss * p->Sq, 128, "fa_prefill_paged mask");
        if (st != FA_OK) return st;
        L.mask_staged = true;
    }
    L.block_table = p->block_table;
    L.seq_lens = p->seq_lens;
    L.q_lens = p->q_lens;
    L.max_blocks = p->max_blocks_per_seq;
    L.num_blocks = p->num_blocks;
    cudaError_t e;
    if (two_tile) {
        int sms = 0;
        e = num_sms(&sms);
        if (e == cudaSuccess) e = fa::launch_prefill2(L, sms, static_cast<cudaStream_t>(stream));
    } else {
        e = fa::launch_prefill(L, static_cast<cudaStream_t>(stream));
    }
    if (e != cudaSuccess) return cuda_fail(e, "fa_prefill_paged: launch");
    return FA_OK;
}

fa_status fa_decode_paged_workspace_size(const fa_decode_paged_params *p, size_t *bytes) {
    fa_status st = check_paged(p);
    if (st != FA_OK) return st;
    if (!bytes) return fail(FA_ERR_INVALID_ARG, "fa_decode_paged_workspace_size: bytes is NULL");
    int splits = 0;
    st = paged_splits(p, &splits);
    if (st != FA_OK) return st;
    *bytes = paged_ws_bytes(p, splits);
    return FA_OK;
}

fa_status fa_decode_paged(const fa_decode_paged_params *p, void *stream) {
    fa_status st = check_paged_ptrs(p);
    if (st != FA_OK) return st;
    if (p->B == 0) return FA_OK;
    int splits = 0;
    st = paged_splits(p, &splits);
    if (st != FA_OK) return st;
    const size_t need = paged_ws_bytes(p, splits);
    if (!p->workspace || p->workspace_bytes < need || ((uintptr_t)p->workspace & 255u))
        return fail(FA_ERR_WORKSPACE, "fa_decode_paged: workspace needs %zu bytes, 256-byte aligned", need);
    fa::PagedLaunch L;
    st = paged_launch_setup(p, splits, &L);
    if (st != FA_OK) return st;
    L.part_o = static_cast<float *>(p->workspace);
    L.part_lse = reinterpret_cast<float *>(static_cast<char *>(p->workspace) + paged_lse_offset(p, splits));
    cudaError_t e = fa::launch_decode_paged(L, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "fa_decode_paged: launch");
    return FA_OK;
}

fa_status fa_decode_paged_noalloc(const fa_decode_paged_params *p, void *stream) {
    fa_status st = check_paged_ptrs(p);
    if (st != FA_OK) return st;
    if (p->B == 0) return FA_OK;
    int splits = 0;
    st = paged_splits(p, &splits);
    if (st != FA_OK) return st;
    const size_t need = paged_ws_bytes(p, splits);
    const size_t have = fa::paged_static_scratch_bytes();
    if (need > have)
        return fail(FA_ERR_WORKSPACE,
                    "fa_decode_paged_noalloc: these shapes need %zu bytes of scratch but the library's fixed scratch "
                    "holds %zu; pass fewer num_splits or call fa_decode_paged with a workspace",
                    need, have);
    fa::PagedLaunch L;
    st = paged_launch_setup(p, splits, &L);
    if (st != FA_OK) return st;
    cudaError_t e = fa::launch_decode_paged_static(L, paged_lse_offset(p, splits), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "fa_decode_paged_noalloc: launch");
    return FA_OK;
}

fa_status fa_debug_decode_paged_stall(const fa_decode_paged_params *p, uint64_t wait_limit_ns, void *stream) {
    fa_status st = check_paged_ptrs(p);
    if (st != FA_OK) return st;
    if (wait_limit_ns < 1000 || wait_limit_ns > 2000000000ull)
        return fail(FA_ERR_INVALID_ARG, "fa_debug_decode_paged_stall: wait_limit_ns must be in [1e3, 2e9]");
    if (p->B == 0) return FA_OK;
    int splits = 0;
    st = paged_splits(p, &splits);
    if (st != FA_OK) return st;
    const size_t need = paged_ws_bytes(p, splits);
    if (!p->workspace || p->workspace_bytes < need || ((uintptr_t)p->workspace & 255u))
        return fail(FA_ERR_WORKSPACE, "fa_debug_decode_paged_stall: workspace needs %zu bytes, 256-byte aligned",
                    need);
    fa::PagedLaunch L;
    st = paged_launch_setup(p, splits, &L);
    if (st != FA_OK) return st;
    L.part_o = static_cast<float *>(p->workspace);
    L.part_lse = reinterpret_cast<float *>(static_cast<char *>(p->workspace) + paged_lse_offset(p, splits));
    L.wait_ns = wait_limit_ns;
    L.stall = 1;
    cudaError_t e = fa::launch_decode_paged(L, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "fa_debug_decode_paged_stall: launch");
    return FA_OK;
}

fa_status fa_decode_gather_workspace_size(const fa_decode_gather_params *p, size_t *bytes) {
    fa_status st = check_gather(p);
    if (st != FA_OK) return st;
    if (!bytes) return fail(FA_ERR_INVALID_ARG, "fa_decode_gather_workspace_size: bytes is NULL");
    int splits = 0;
    st = gather_splits(p, &splits);
    if (st != FA_OK) return st;
    *bytes = gather_ws_bytes(p, splits);
    return FA_OK;
}

fa_status fa_decode_gather(const fa_decode_gather_params *p, void *stream) {
    fa_status st = check_gather_ptrs(p);
    if (st != FA_OK) return st;
    if (p->T == 0) return FA_OK;
    int splits = 0;
    st = gather_splits(p, &splits);
    if (st != FA_OK) return st;
    const size_t need = gather_ws_bytes(p, splits);
    if (!p->workspace || p->workspace_bytes < need || ((uintptr_t)p->workspace & 255u))
        return fail(FA_ERR_WORKSPACE, "fa_decode_gather: workspace needs %zu bytes, 256-byte aligned", need);
    if (!get_encoder()) return fail(FA_ERR_CUDA, "fa_decode_gather: cuTensorMapEncodeTiled is not available");
    fa::GatherLaunch L;
    st = encode_2d(&L.tmQ, p->q, p->dk, (int64_t)p->T * p->Hq, p->dk, 128, "fa_decode_gather q");
    if (st != FA_OK) return st;
    L.q = p->q;
    L.rows = p->kv_rows;
    L.n_rows = p->n_rows;
    L.row_stride = p->row_stride;
    L.idx = p->idx;
    L.key_pos = p->key_pos;
    L.q_pos = p->q_pos;
    L.topk = p->topk;
    L.T = p->T;
    L.Hq = p->Hq;
    L.dk = p->dk;
    L.scale = p->scale;
    L.num_splits = splits;
    L.keys_per_split = ((p->topk + splits - 1) / splits + 63) / 64 * 64;
    L.o = p->o;
    L.lse = p->lse;
    L.o_bf16 = p->o_dtype == FA_BF16;
    const size_t rows = (size_t)p->T * p->Hq * splits;
    L.part_o = static_cast<float *>(p->workspace);
    L.part_lse = reinterpret_cast<float *>(static_cast<char *>(p->workspace) +
                                           ((rows * 512 * sizeof(float) + 255) & ~size_t(255)));
    // The kernel writes its partials with TMA stores: (512 values, T * Hq
    // rows, splits) fp32, 32 x 32 boxes.
    st = encode_4d(&L.tmPO, L.part_o, 512, p->T * p->Hq, splits, 1, (int64_t)splits * 512, 512,
                   (int64_t)splits * 512 * p->T * p->Hq, 32, "fa_decode_gather partials", 4);
    if (st != FA_OK) return st;
    cudaError_t e = fa::launch_decode_gather(L, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "fa_decode_gather: launch");
    return FA_OK;
}

fa_status fa_mla_tail_workspace_size(const fa_mla_tail_params *p, size_t *bytes) {
    fa_status st = check_tail(p);
    if (st != FA_OK) return st;
    if (!bytes) return fail(FA_ERR_INVALID_ARG, "fa_mla_tail_workspace_size: bytes is NULL");
    fa::TailLaunch L;
    memset(&L, 0, sizeof L);
    L.T = p->T;
    L.Hq = p->Hq;
    L.R = p->R;
    L.V = p->V;
    L.Hd = p->Hd;
    *bytes = fa::mla_tail_ws_bytes(L);
    return FA_OK;
}

fa_status fa_mla_tail(const fa_mla_tail_params *p, void *stream) {
    fa_status st = check_tail(p);
    if (st != FA_OK) return st;
    if (p->T == 0) return FA_OK;
    if (!p->o_lat || !p->w_abs || !p->w_o || !p->y) return fail(FA_ERR_INVALID_ARG, "fa_mla_tail: NULL pointer");
    if (!aligned16(p->o_lat) || !aligned16(p->w_abs) || !aligned16(p->w_o) || !aligned16(p->y))
        return fail(FA_ERR_INVALID_ARG, "fa_mla_tail: o_lat, w_abs, w_o and y must be 16-byte aligned");
    fa::TailLaunch L;
    memset(&L, 0, sizeof L);
    L.T = p->T;
    L.Hq = p->Hq;
    L.R = p->R;
    L.V = p->V;
    L.Hd = p->Hd;
    L.splits = p->num_splits;
    const size_t need = fa::mla_tail_ws_bytes(L);
    if (!p->workspace || p->workspace_bytes < need || ((uintptr_t)p->workspace & 255u))
        return fail(FA_ERR_WORKSPACE, "fa_mla_tail: workspace must be 256-byte aligned and >= %zu bytes", need);
    if (!get_encoder()) return fail(FA_ERR_CUDA, "fa_mla_tail: cuTensorMapEncodeTiled is not available");
    const int NP = p->T < 256 ? (p->T + 15) / 16 * 16 : 256;  // token rows per chunk load
    const int64_t K = (int64_t)p->Hq * p->V;
    // (inner, rows, batch, 1) views; element strides.
    st = encode_4d(&L.tmAbsA, p->w_abs, p->R, p->V, p->Hq, 1, p->R, (int64_t)p->V * p->R,
                   (int64_t)p->Hq * p->V * p->R, 128, "fa_mla_tail w_abs");
    if (st != FA_OK) return st;
    st = encode_4d(&L.tmAbsB, p->o_lat, p->R, p->T, p->Hq, 1, (int64_t)p->Hq * p->R, p->R,
                   (int64_t)p->T * p->Hq * p->R, NP, "fa_mla_tail o_lat");
    if (st != FA_OK) return st;
    st = encode_4d(&L.tmOA, p->w_o, (int)K, p->Hd, 1, 1, K, K * p->Hd, K * p->Hd, 128, "fa_mla_tail w_o");
    if (st != FA_OK) return st;
    st = encode_4d(&L.tmOB, p->workspace, (int)K, p->T, 1, 1, K, K * p->T, K * p->T, NP, "fa_mla_tail u");
    if (st != FA_OK) return st;
    L.y = p->y;
    L.y_bf16 = p->y_dtype == FA_BF16;
    L.workspace = p->workspace;
    int sms = 0;
    cudaError_t e = num_sms(&sms);
    if (e == cudaSuccess) e = fa::launch_mla_tail(L, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "fa_mla_tail: launch");
    return FA_OK;
}

fa_status fa_kv_dequant_n(const fa_kv_dequant_params *p, int n, void *stream) {
    if (!p) return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant: params is NULL");
    if (n < 1 || n > fa::kMaxDequantSegs)
        return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant_n: n must be in [1, %d]", fa::kMaxDequantSegs);
    fa::KvDequantLaunch L[fa::kMaxDequantSegs];
    bool any = false;
    for (int i = 0; i < n; ++i) {
        const fa_kv_dequant_params *q = p + i;
        if (q->type != FA_KV_Q8_0 && q->type != FA_KV_Q4_0 && q->type != FA_KV_FP8_E4M3)
            return fail(FA_ERR_UNSUPPORTED, "fa_kv_dequant: type %d (supported: FA_KV_Q8_0, FA_KV_Q4_0, FA_KV_FP8_E4M3)",
                        q->type);
        if (q->type == FA_KV_FP8_E4M3 && !isfinite(q->scale))
            return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant: the fp8 scale must be finite");
        if (q->type != p->type) return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant_n: every entry must have one type");
        if (q->n_rows < 0 || q->row_elems <= 0 || q->row_elems % 32 != 0)
            return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant: need n_rows >= 0 and row_elems a positive multiple of 32");
        const int64_t block_bytes = q->type == FA_KV_Q8_0 ? 34 : (q->type == FA_KV_Q4_0 ? 18 : 32);
        const int64_t src_align = q->type == FA_KV_FP8_E4M3 ? 8 : 2;
        if (q->src_row_bytes < q->row_elems / 32 * block_bytes || q->src_row_bytes % src_align != 0)
            return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant: src_row_bytes must be a multiple of %lld and >= %lld",
                        (long long)src_align, (long long)(q->row_elems / 32 * block_bytes));
        if (q->dst_row_stride < q->row_elems || q->dst_row_stride % 8 != 0)
            return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant: dst_row_stride must be a multiple of 8 and >= row_elems");
        if (q->n_rows > 0) {
            if (!q->src || !q->dst) return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant: NULL pointer");
            if (reinterpret_cast<uintptr_t>(q->src) % src_align != 0 || reinterpret_cast<uintptr_t>(q->dst) % 16 != 0)
                return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant: src must be %lld-byte and dst 16-byte aligned",
                            (long long)src_align);
            const int64_t pitch = q->src_row_bytes > 2 * q->dst_row_stride ? q->src_row_bytes : 2 * q->dst_row_stride;
            if (q->n_rows > (INT64_MAX / 4) / pitch)
                return fail(FA_ERR_INVALID_ARG, "fa_kv_dequant: rows * pitch overflows");
            any = true;
        }
        L[i] = fa::KvDequantLaunch{q->src,     q->type, q->n_rows,         q->row_elems,
                                   q->src_row_bytes, q->dst, q->dst_row_stride, q->scale};
    }
    if (!any) return FA_OK;
    int sms = 0;
    cudaError_t e = num_sms(&sms);
    if (e != cudaSuccess) return cuda_fail(e, "fa_kv_dequant");
    e = fa::launch_kv_dequant(L, n, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "fa_kv_dequant launch");
    return FA_OK;
}

fa_status fa_kv_dequant(const fa_kv_dequant_params *p, void *stream) { return fa_kv_dequant_n(p, 1, stream); }

fa_status fa_rope(const fa_rope_params *p, void *stream) {
    const char *who = "fa_rope";
    if (!p) return fail(FA_ERR_INVALID_ARG, "fa_rope: params is NULL");
    if (p->B < 0 || p->S < 0 || p->Hq <= 0 || p->Hk < 0 || p->d <= 0)
        return fail(FA_ERR_INVALID_ARG, "fa_rope: need B, S, Hk >= 0 and Hq, d > 0");
    if (p->d % 16 != 0 || p->d > 1024)
        return fail(FA_ERR_UNSUPPORTED, "fa_rope: d must be a multiple of 16 up to 1024 (got %d)", p->d);
    if ((int64_t)p->B * p->S >= (int64_t(1) << 31) || (int64_t)p->Hq + p->Hk > 65535)
        return fail(FA_ERR_INVALID_ARG, "fa_rope: B * S must be < 2^31 and Hq + Hk <= 65535");
    if (p->dtype != FA_F32 && p->dtype != FA_BF16) return fail(FA_ERR_INVALID_ARG, "fa_rope: dtype");
    if (!p->inv_freq) return fail(FA_ERR_INVALID_ARG, "fa_rope: inv_freq is NULL");
    if ((uintptr_t)p->pos & 3u) return fail(FA_ERR_INVALID_ARG, "fa_rope: pos must be 4-byte aligned");
    if (!p->pos && (int64_t)p->pos0 + p->S > 0x7fffffffLL)
        return fail(FA_ERR_INVALID_ARG, "fa_rope: pos0 + S must be < 2^31");
    if ((p->k || p->k_out) && p->Hk == 0) return fail(FA_ERR_INVALID_ARG, "fa_rope: k needs Hk > 0");
    fa::RopeLaunch L;
    memset(&L, 0, sizeof L);
    fa_status st = make_rope_map(who, p->inv_freq, p->rot_dim, p->rot_offset, p->d, p->interleaved, p->inverse,
                                 p->mscale, &L.map);
    if (st != FA_OK) return st;
    if (p->B == 0 || p->S == 0) return FA_OK;
    const int unit = p->dtype == FA_F32 ? 4 : 8;
    st = rope_tensor(who, "q", p->q, p->q_out, p->q_sb, p->q_sh, p->q_ss, p->qo_sb, p->qo_sh, p->qo_ss, p->B, p->Hq,
                     p->S, p->d, unit, &L.x[0]);
    if (st == FA_OK && p->Hk > 0)
        st = rope_tensor(who, "k", p->k, p->k_out, p->k_sb, p->k_sh, p->k_ss, p->ko_sb, p->ko_sh, p->ko_ss, p->B,
                         p->Hk, p->S, p->d, unit, &L.x[1]);
    if (st != FA_OK) return st;
    if (p->Hk > 0) {  // one launch reads and writes all four
        const int bytes = 16 / unit;
        const fa::Rows q = byte_rows(p->q, p->q_sb, p->q_sh, p->q_ss, p->B, p->Hq, p->S, p->d, bytes),
                       k = byte_rows(p->k, p->k_sb, p->k_sh, p->k_ss, p->B, p->Hk, p->S, p->d, bytes),
                       qo = byte_rows(p->q_out, p->qo_sb, p->qo_sh, p->qo_ss, p->B, p->Hq, p->S, p->d, bytes),
                       ko = byte_rows(p->k_out, p->ko_sb, p->ko_sh, p->ko_ss, p->B, p->Hk, p->S, p->d, bytes);
        if (fa::rows_meet(qo, ko) || fa::rows_meet(qo, k) || fa::rows_meet(ko, q))
            return fail(FA_ERR_INVALID_ARG, "fa_rope: each output must be apart from the other and from the other's input");
    }
    L.B = p->B;
    L.S = p->S;
    L.d = p->d;
    L.pos = p->pos;
    L.pos_sb = p->pos_sb;
    L.pos0 = p->pos0;
    int sms = 0;
    cudaError_t e = num_sms(&sms);
    if (e == cudaSuccess) e = fa::launch_rope(L, p->dtype == FA_F32, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "fa_rope: launch");
    return FA_OK;
}

fa_status fa_kv_append(const fa_kv_append_params *p, void *stream) {
    const char *who = "fa_kv_append";
    if (!p) return fail(FA_ERR_INVALID_ARG, "fa_kv_append: params is NULL");
    if (p->B < 0 || p->Sq < 0 || p->Hkv <= 0 || p->dk <= 0 || p->dv <= 0 || p->num_blocks <= 0 ||
        p->max_blocks_per_seq <= 0)
        return fail(FA_ERR_INVALID_ARG,
                    "fa_kv_append: need B, Sq >= 0 and Hkv, dk, dv, num_blocks, max_blocks_per_seq > 0");
    if (p->block_size != 64) return fail(FA_ERR_UNSUPPORTED, "fa_kv_append: block_size must be 64 (got %d)", p->block_size);
    const bool quant = p->kv_type != FA_KV_BF16;
    if (quant && p->kv_type != FA_KV_Q8_0 && p->kv_type != FA_KV_Q4_0 && p->kv_type != FA_KV_FP8_E4M3)
        return fail(FA_ERR_UNSUPPORTED, "fa_kv_append: kv_type %d", p->kv_type);
    if (p->dk % 16 != 0 || p->dv % 16 != 0 || p->dk > 1024 || p->dv > 1024 ||
        (quant && (p->dk != 128 || p->dv != 128)))
        return fail(FA_ERR_UNSUPPORTED,
                    "fa_kv_append: dk and dv must be multiples of 16 up to 1024, 128 for quantised caches (got %d/%d)",
                    p->dk, p->dv);
    if (p->kv_type == FA_KV_FP8_E4M3 && (!finite_pos(p->k_scale) || !finite_pos(p->v_scale) ||
                                         !isfinite(1.f / p->k_scale) || !isfinite(1.f / p->v_scale)))
        return fail(FA_ERR_INVALID_ARG, "fa_kv_append: k_scale, v_scale and their reciprocals must be finite and > 0");
    const int Hq = p->q || p->q_out ? p->Hq : 0;
    if ((p->q || p->q_out) && (p->Hq <= 0 || !p->inv_freq))
        return fail(FA_ERR_INVALID_ARG, "fa_kv_append: q needs Hq > 0 and inv_freq");
    if ((int64_t)p->B * p->Sq >= (int64_t(1) << 31) || (int64_t)Hq + 2 * (int64_t)p->Hkv > 65535)
        return fail(FA_ERR_INVALID_ARG, "fa_kv_append: B * Sq must be < 2^31 and Hq + 2 Hkv <= 65535");
    if ((uintptr_t)p->pos & 3u) return fail(FA_ERR_INVALID_ARG, "fa_kv_append: pos must be 4-byte aligned");
    fa::AppendLaunch L;
    memset(&L, 0, sizeof L);
    fa_status st = FA_OK;
    if (p->inv_freq) {
        st = make_rope_map(who, p->inv_freq, p->rot_dim, p->rot_offset, p->dk, p->interleaved, 0, p->mscale, &L.map);
        if (st != FA_OK) return st;
        if ((p->kv_type == FA_KV_Q8_0 || p->kv_type == FA_KV_Q4_0) &&
            (p->rot_offset % 32 != 0 || p->rot_dim % (p->interleaved ? 32 : 64) != 0))
            return fail(FA_ERR_UNSUPPORTED,
                        "fa_kv_append: q8_0 and q4_0 rows need rot_offset %% 32 == 0 and rot_dim %% 64 == 0 "
                        "(interleaved: 32)");
    }
    if (p->B == 0 || p->Sq == 0) return FA_OK;
    st = check_rows(who, "k", p->k, p->k_sb, p->k_sh, p->k_ss, p->B, p->Hkv, p->Sq, 8);
    if (st == FA_OK) st = check_rows(who, "v", p->v, p->v_sb, p->v_sh, p->v_ss, p->B, p->Hkv, p->Sq, 8);
    if (st == FA_OK && Hq > 0)
        st = rope_tensor(who, "q", p->q, p->q_out, p->q_sb, p->q_sh, p->q_ss, p->qo_sb, p->qo_sh, p->qo_ss, p->B, Hq,
                         p->Sq, p->dk, 8, &L.q);
    if (st != FA_OK) return st;
    if (!p->k_cache || !p->v_cache || !p->block_table || !p->seq_lens)
        return fail(FA_ERR_INVALID_ARG, "fa_kv_append: NULL cache, block_table or seq_lens");
    if (!aligned16(p->k_cache) || !aligned16(p->v_cache))
        return fail(FA_ERR_INVALID_ARG, "fa_kv_append: the caches must be 16-byte aligned");
    if (((uintptr_t)p->block_table & 3u) || ((uintptr_t)p->seq_lens & 3u) || ((uintptr_t)p->q_lens & 3u))
        return fail(FA_ERR_INVALID_ARG, "fa_kv_append: block_table, seq_lens and q_lens must be 4-byte aligned");
    {
        const auto cache = [&](const void *c, int d) {
            const int64_t row = p->kv_type == FA_KV_BF16   ? 2 * d
                                : p->kv_type == FA_KV_Q8_0 ? d / 32 * 34
                                : p->kv_type == FA_KV_Q4_0 ? d / 32 * 18
                                                           : d;
            return fa::Rows{c, (int64_t)p->Hkv * 64 * row, {p->num_blocks, 1, 1}, {(int64_t)p->Hkv * 64 * row, 0, 0}};
        };
        const fa::Rows kc = cache(p->k_cache, p->dk), vc = cache(p->v_cache, p->dv);
        if (fa::rows_meet(kc, vc)) return fail(FA_ERR_INVALID_ARG, "fa_kv_append: the caches overlap");
        if (Hq > 0) {
            const fa::Rows to = byte_rows(p->q_out, p->qo_sb, p->qo_sh, p->qo_ss, p->B, Hq, p->Sq, p->dk, 2);
            if (fa::rows_meet(to, kc) || fa::rows_meet(to, vc) ||
                fa::rows_meet(to, byte_rows(p->k, p->k_sb, p->k_sh, p->k_ss, p->B, p->Hkv, p->Sq, p->dk, 2)) ||
                fa::rows_meet(to, byte_rows(p->v, p->v_sb, p->v_sh, p->v_ss, p->B, p->Hkv, p->Sq, p->dv, 2)))
                return fail(FA_ERR_INVALID_ARG, "fa_kv_append: q_out must be apart from k, v and the caches");
        }
    }
    L.k = fa::RopeTensor{p->k, p->k_cache, p->Hkv, p->k_sb, p->k_sh, p->k_ss, 0, 0, 0, 0};
    L.v = fa::RopeTensor{p->v, p->v_cache, p->Hkv, p->v_sb, p->v_sh, p->v_ss, 0, 0, 0, 0};
    L.block_table = p->block_table;
    L.seq_lens = p->seq_lens;
    L.q_lens = p->q_lens;
    L.max_blocks = p->max_blocks_per_seq;
    L.num_blocks = p->num_blocks;
    L.B = p->B;
    L.Hkv = p->Hkv;
    L.Sq = p->Sq;
    L.dk = p->dk;
    L.dv = p->dv;
    L.pos = p->pos;
    L.pos_sb = p->pos_sb;
    L.kv_type = p->kv_type;
    L.k_scale = p->k_scale;
    L.v_scale = p->v_scale;
    int sms = 0;
    cudaError_t e = num_sms(&sms);
    if (e == cudaSuccess) e = fa::launch_kv_append(L, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "fa_kv_append: launch");
    return FA_OK;
}

fa_status fa_bwd_workspace_size(const fa_bwd_params *p, size_t *bytes) {
    fa_status st = check_bwd(p);
    if (st != FA_OK) return st;
    if (!bytes) return fail(FA_ERR_INVALID_ARG, "fa_bwd_workspace_size: bytes is NULL");
    const size_t full = bwd_bytes(p, false), causal = bwd_bytes(p, true);
    *bytes = full > causal ? full : causal;
    return FA_OK;
}

fa_status fa_bwd_workspace_need(const fa_bwd_params *p, size_t *bytes) {
    fa_status st = check_bwd(p);
    if (st != FA_OK) return st;
    if (!bytes) return fail(FA_ERR_INVALID_ARG, "fa_bwd_workspace_need: bytes is NULL");
    *bytes = bwd_bytes(p, p->causal != 0);
    return FA_OK;
}

fa_status fa_bwd(const fa_bwd_params *p, void *stream) {
    fa_status st = check_bwd(p);
    if (st != FA_OK) return st;
    if (p->gsinks && !p->sinks) return fail(FA_ERR_INVALID_ARG, "fa_bwd: gsinks needs sinks");
    if (((uintptr_t)p->sinks & 3u) || ((uintptr_t)p->gsinks & 3u) || ((uintptr_t)p->lse & 3u) ||
        ((uintptr_t)p->dlse & 3u))
        return fail(FA_ERR_INVALID_ARG, "fa_bwd: lse, dlse, sinks and gsinks must be 4-byte aligned");
    const bool rows = p->B > 0 && p->Sq > 0, keys = p->B > 0 && p->Sk > 0;
    if (!rows && !keys && !p->gsinks) return FA_OK;
    if (rows) {
        if (!p->q || !p->o || !p->dout || !p->lse || !aligned16(p->q) || !aligned16(p->o) || !aligned16(p->dout))
            return fail(FA_ERR_INVALID_ARG, "fa_bwd: q, o, dout, lse must be given, tensors 16-byte aligned");
        const int ovec = p->o_dtype == FA_F32 ? 4 : 8;
        if ((p->Sq > 1 && p->o_ss % ovec) || (p->Hq > 1 && p->o_sh % ovec) || (p->B > 1 && p->o_sb % ovec))
            return fail(FA_ERR_INVALID_ARG, "fa_bwd: o strides must be multiples of %d elements", ovec);
    }
    if (keys && (!p->k || !p->v || !aligned16(p->k) || !aligned16(p->v)))
        return fail(FA_ERR_INVALID_ARG, "fa_bwd: k and v must be given, 16-byte aligned");
    const int gvec = p->g_dtype == FA_F32 ? 4 : 8;
    if (rows) st = check_grad("gq", p->gq, p->gq_sb, p->gq_sh, p->gq_ss, p->B, p->Hq, p->Sq, p->dk, gvec);
    if (st == FA_OK && keys)
        st = check_grad("gk", p->gk, p->gk_sb, p->gk_sh, p->gk_ss, p->B, p->Hkv, p->Sk, p->dk, gvec);
    if (st == FA_OK && keys)
        st = check_grad("gv", p->gv, p->gv_sb, p->gv_sh, p->gv_ss, p->B, p->Hkv, p->Sk, p->dv, gvec);
    if (st != FA_OK) return st;
    // Every input is read until the last gradient is written.
    const void *in[5] = {p->q, p->o, p->dout, p->k, p->v}, *out[3] = {p->gq, p->gk, p->gv};
    for (int i = 0; i < 3; ++i) {
        if (!(i ? keys : rows)) continue;
        bool taken = false;
        for (int j = 0; j < 5; ++j) taken |= (j < 3 ? rows : keys) && out[i] == in[j];
        for (int j = 0; j < i; ++j) taken |= (j ? keys : rows) && out[i] == out[j];
        if (taken) return fail(FA_ERR_INVALID_ARG, "fa_bwd: gq, gk and gv must be apart from the inputs and each other");
    }
    if (p->mask && (((uintptr_t)p->mask & 15u) || p->m_ss % 8 || p->m_sh % 8 || p->m_sb % 8 || p->m_ss < p->Sk ||
                    p->m_sh < 0 || p->m_sb < 0))
        return fail(FA_ERR_INVALID_ARG,
                    "fa_bwd: mask must be 16-byte aligned, its strides multiples of 8 elements, m_ss >= Sk");
    const size_t each = bwd_row_bytes(p), need = bwd_bytes(p, p->causal != 0);
    if (!p->workspace || p->workspace_bytes < need || ((uintptr_t)p->workspace & 255u))
        return fail(FA_ERR_WORKSPACE, "fa_bwd: workspace needs %zu bytes, 256-byte aligned", need);
    st = check_bwd_apart(p, rows, keys, need);
    if (st != FA_OK) return st;
    if (!get_encoder()) return fail(FA_ERR_CUDA, "fa_bwd: cuTensorMapEncodeTiled is not available");
    fa::BwdLaunch L;
    memset(&L, 0, sizeof L);
    // A side without rows is never loaded; its maps stay empty.
    const auto both = [&](CUtensorMap *x, CUtensorMap *y, const void *t, int d, int S, int H, int64_t ss, int64_t sh,
                          int64_t sb, const char *name) {
        fa_status r = encode_4d(x, t, d, S, H, p->B, ss, sh, sb, 128, name);
        if (r != FA_OK) return r;
        *y = *x;
        return fa::bwd_walk(p->dk) == 128 ? FA_OK
                                          : encode_4d(y, t, d, S, H, p->B, ss, sh, sb, fa::bwd_walk(p->dk), name);
    };
    if (rows) {
        st = both(&L.tmQx, &L.tmQy, p->q, p->dk, p->Sq, p->Hq, p->q_ss, p->q_sh, p->q_sb, "fa_bwd q");
        if (st == FA_OK)
            st = both(&L.tmDOx, &L.tmDOy, p->dout, p->dv, p->Sq, p->Hq, p->do_ss, p->do_sh, p->do_sb, "fa_bwd dout");
    }
    if (st == FA_OK && keys) {
        st = both(&L.tmKx, &L.tmKy, p->k, p->dk, p->Sk, p->Hkv, p->k_ss, p->k_sh, p->k_sb, "fa_bwd k");
        if (st == FA_OK) st = both(&L.tmVx, &L.tmVy, p->v, p->dv, p->Sk, p->Hkv, p->v_ss, p->v_sh, p->v_sb, "fa_bwd v");
    }
    if (st != FA_OK) return st;
    L.B = p->B;
    L.Hq = p->Hq;
    L.Hkv = p->Hkv;
    L.Sq = p->Sq;
    L.Sk = p->Sk;
    L.dk = p->dk;
    L.dv = p->dv;
    L.scale = p->scale;
    L.causal = p->causal ? 1 : 0;
    L.o = p->o;
    L.dout = p->dout;
    L.o_sb = p->o_sb;
    L.o_sh = p->o_sh;
    L.o_ss = p->o_ss;
    L.do_sb = p->do_sb;
    L.do_sh = p->do_sh;
    L.do_ss = p->do_ss;
    L.o_bf16 = p->o_dtype == FA_BF16;
    L.lse = p->lse;
    L.dlse = p->dlse;
    L.gq = p->gq;
    L.gk = p->gk;
    L.gv = p->gv;
    L.gq_sb = p->gq_sb;
    L.gq_sh = p->gq_sh;
    L.gq_ss = p->gq_ss;
    L.gk_sb = p->gk_sb;
    L.gk_sh = p->gk_sh;
    L.gk_ss = p->gk_ss;
    L.gv_sb = p->gv_sb;
    L.gv_sh = p->gv_sh;
    L.gv_ss = p->gv_ss;
    L.g_bf16 = p->g_dtype == FA_BF16;
    L.mods.mask = static_cast<const __half *>(p->mask);
    L.mods.m_sb = p->m_sb;
    L.mods.m_sh = p->m_sh;
    L.mods.m_ss = p->m_ss;
    L.mods.softcap = p->softcap;
    L.mods.sinks = p->sinks;
    if (p->max_bias > 0.f) {  // ALiBi bases, as read in score_mods.cuh
        int n2 = 1;
        while (n2 * 2 <= p->Hq) n2 *= 2;
        L.mods.n_head_log2 = n2;
        L.mods.log2_m0 = -p->max_bias / (float)n2;
        L.mods.log2_m1 = -p->max_bias / 2.f / (float)n2;
    }
    L.has_mods = p->mask || p->softcap > 0.f || p->scale < 1e-30f;
    L.gsinks = p->gsinks;
    L.nlse = static_cast<float *>(p->workspace);
    L.ndelta = reinterpret_cast<float *>(static_cast<char *>(p->workspace) + each);
    L.ext = static_cast<char *>(p->workspace) + 2 * each;
    L.next = reinterpret_cast<int *>(static_cast<char *>(p->workspace) + 6 * each);
    L.part = reinterpret_cast<float *>(static_cast<char *>(p->workspace) + 6 * each + 256);
    int sms = 0;
    cudaError_t e = num_sms(&sms);
    if (e == cudaSuccess) e = fa::launch_bwd(L, sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "fa_bwd: launch");
    return FA_OK;
}

fa_status fa_device_error(int clear, int *code) {
    if (!code) return fail(FA_ERR_INVALID_ARG, "fa_device_error: code is NULL");
    int c1 = 0, c2 = 0, c3 = 0, c4 = 0, c5 = 0, c6 = 0, c7 = 0;
    cudaError_t e = fa::prefill_device_error(clear, &c1);
    if (e == cudaSuccess) e = fa::tail_device_error(clear, &c5);
    if (e == cudaSuccess) e = fa::prefill2_device_error(clear, &c4);
    if (e == cudaSuccess) e = fa::decode_device_error(clear, &c2);
    if (e == cudaSuccess) e = fa::gather_device_error(clear, &c3);
    if (e == cudaSuccess) e = fa::append_device_error(clear, &c6);
    if (e == cudaSuccess) e = fa::bwd_device_error(clear, &c7);
    if (e != cudaSuccess) return cuda_fail(e, "fa_device_error");
    *code = c1 ? c1 : (c4 ? c4 : (c2 ? c2 : (c3 ? c3 : (c5 ? c5 : (c6 ? c6 : c7)))));
    return FA_OK;
}

}  // extern "C"
