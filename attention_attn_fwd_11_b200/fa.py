"""ctypes binding over libfa.so (include/fa.h).  Argument marshalling only:
every step of the computation runs in the library's CUDA kernels.  PyTorch
supplies device memory and the current stream.  There is no CPU fallback:
if the library is missing or the tensors are not on a CUDA device, calls
raise.

A call works on the current stream, or on the one given as ``stream``: the
caller sees to it that the inputs are ready there, and waits for that stream
before going on with the results elsewhere.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(6)
FA_F32, FA_BF16 = 0, 1
STATUS_NAMES = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_WORKSPACE",
                4: "FA_ERR_CUDA", 5: "FA_ERR_TIMEOUT"}

_vp = ctypes.c_void_p
_i32 = ctypes.c_int
_i64 = ctypes.c_int64


class FwdParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("lse", _vp),
                ("B", _i32), ("Hq", _i32), ("Hkv", _i32), ("Sq", _i32), ("Sk", _i32), ("dk", _i32), ("dv", _i32),
                ("q_sb", _i64), ("q_sh", _i64), ("q_ss", _i64),
                ("k_sb", _i64), ("k_sh", _i64), ("k_ss", _i64),
                ("v_sb", _i64), ("v_sh", _i64), ("v_ss", _i64),
                ("o_sb", _i64), ("o_sh", _i64), ("o_ss", _i64),
                ("scale", ctypes.c_float), ("causal", _i32), ("o_dtype", _i32),
                ("mask", _vp), ("m_sb", _i64), ("m_sh", _i64), ("m_ss", _i64),
                ("max_bias", ctypes.c_float), ("softcap", ctypes.c_float), ("sinks", _vp)]


class PagedParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("k_cache", _vp), ("v_cache", _vp), ("block_table", _vp), ("seq_lens", _vp),
                ("max_blocks_per_seq", _i32), ("B", _i32), ("Hq", _i32), ("Hkv", _i32), ("dk", _i32),
                ("dv", _i32), ("block_size", _i32), ("num_blocks", _i32), ("scale", ctypes.c_float),
                ("num_splits", _i32), ("o", _vp), ("lse", _vp), ("o_dtype", _i32), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t), ("kv_type", _i32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class PrefillPagedParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("q_sb", _i64), ("q_sh", _i64), ("q_ss", _i64), ("k_cache", _vp), ("v_cache", _vp),
                ("block_table", _vp), ("seq_lens", _vp), ("max_blocks_per_seq", _i32), ("B", _i32), ("Hq", _i32),
                ("Hkv", _i32), ("Sq", _i32), ("dk", _i32), ("dv", _i32), ("block_size", _i32), ("num_blocks", _i32),
                ("scale", ctypes.c_float), ("causal", _i32), ("o", _vp), ("o_sb", _i64), ("o_sh", _i64),
                ("o_ss", _i64), ("lse", _vp), ("o_dtype", _i32), ("q_lens", _vp), ("mask", _vp),
                ("m_sb", _i64), ("m_sh", _i64), ("m_ss", _i64), ("max_bias", ctypes.c_float),
                ("softcap", ctypes.c_float), ("sinks", _vp)]


class GatherParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("kv_rows", _vp), ("n_rows", _i64), ("row_stride", _i64), ("dk", _i32), ("dv", _i32),
                ("v_offset", _i32), ("idx", _vp), ("topk", _i32), ("key_pos", _vp), ("q_pos", _vp), ("T", _i32),
                ("Hq", _i32), ("scale", ctypes.c_float), ("num_splits", _i32), ("o", _vp), ("lse", _vp),
                ("o_dtype", _i32), ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class MlaTailParams(ctypes.Structure):
    _fields_ = [("o_lat", _vp), ("w_abs", _vp), ("w_o", _vp), ("T", _i32), ("Hq", _i32), ("R", _i32), ("V", _i32),
                ("Hd", _i32), ("y", _vp), ("y_dtype", _i32), ("num_splits", _i32), ("workspace", _vp),
                ("workspace_bytes", ctypes.c_size_t)]


class KvDequantParams(ctypes.Structure):
    _fields_ = [("src", _vp), ("type", _i32), ("n_rows", _i64), ("row_elems", _i32), ("src_row_bytes", _i64),
                ("dst", _vp), ("dst_row_stride", _i64), ("scale", ctypes.c_float)]


_STRIDES = lambda *names: [(n + e, _i64) for n in names for e in ("_sb", "_sh", "_ss")]  # noqa: E731


class BwdParams(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("q", "k", "v", "o", "dout", "lse", "dlse", "gq", "gk", "gv")] + \
        [(n, _i32) for n in ("B", "Hq", "Hkv", "Sq", "Sk", "dk", "dv")] + \
        _STRIDES("q", "k", "v", "o", "do", "gq", "gk", "gv") + \
        [("scale", ctypes.c_float), ("causal", _i32), ("o_dtype", _i32), ("g_dtype", _i32), ("mask", _vp)] + \
        _STRIDES("m") + [("max_bias", ctypes.c_float), ("softcap", ctypes.c_float), ("sinks", _vp), ("gsinks", _vp),
                         ("workspace", _vp), ("workspace_bytes", ctypes.c_size_t)]


class RopeParams(ctypes.Structure):
    _fields_ = [("q", _vp), ("q_out", _vp), ("q_sb", _i64), ("q_sh", _i64), ("q_ss", _i64), ("qo_sb", _i64),
                ("qo_sh", _i64), ("qo_ss", _i64), ("k", _vp), ("k_out", _vp), ("k_sb", _i64), ("k_sh", _i64),
                ("k_ss", _i64), ("ko_sb", _i64), ("ko_sh", _i64), ("ko_ss", _i64), ("B", _i32), ("Hq", _i32),
                ("Hk", _i32), ("S", _i32), ("d", _i32), ("dtype", _i32), ("pos", _vp), ("pos_sb", _i64),
                ("pos0", _i32), ("inv_freq", _vp), ("rot_dim", _i32), ("rot_offset", _i32), ("interleaved", _i32),
                ("inverse", _i32), ("mscale", ctypes.c_float)]


class KvAppendParams(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_sb", _i64), ("k_sh", _i64), ("k_ss", _i64), ("v_sb", _i64),
                ("v_sh", _i64), ("v_ss", _i64), ("k_cache", _vp), ("v_cache", _vp), ("block_table", _vp),
                ("seq_lens", _vp), ("q_lens", _vp), ("max_blocks_per_seq", _i32), ("B", _i32), ("Hkv", _i32),
                ("Sq", _i32), ("dk", _i32), ("dv", _i32), ("block_size", _i32), ("num_blocks", _i32),
                ("kv_type", _i32), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float), ("inv_freq", _vp),
                ("rot_dim", _i32), ("rot_offset", _i32), ("interleaved", _i32), ("mscale", ctypes.c_float),
                ("pos", _vp), ("pos_sb", _i64), ("q", _vp), ("q_out", _vp), ("Hq", _i32), ("q_sb", _i64),
                ("q_sh", _i64), ("q_ss", _i64), ("qo_sb", _i64), ("qo_sh", _i64), ("qo_ss", _i64)]


def _packer(cls, n):
    """A function that makes a cls from its first n fields; the others are 0.
    (One struct.pack: ctypes sets fields one by one, 6 us for 45 of them
    where this takes 1.5.)"""
    codes = {_vp: "P", _i32: "i", _i64: "q", ctypes.c_float: "f", ctypes.c_size_t: "N"}
    fields = "@" + "".join(codes[t] for _, t in cls._fields_[:n])
    whole = struct.Struct("%s%dx" % (fields, ctypes.sizeof(cls) - struct.calcsize(fields)))

    def make(*values):
        try:
            return cls.from_buffer_copy(whole.pack(*values))
        except struct.error as e:
            raise ValueError("an argument is out of its type's range: %s" % e) from None

    return make


def _int(x):
    """x for an int field set by name: ctypes would keep its lowest 32 bits without a word."""
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError("an argument is out of its type's range: %d" % x)
    return x


_pack_bwd, _pack_rope, _pack_append = _packer(BwdParams, 45), _packer(RopeParams, 31), _packer(KvAppendParams, 22)

FA_KV_Q8_0, FA_KV_Q4_0, FA_KV_FP8_E4M3 = 8, 4, 2
KV_QUANT = {"q8_0": (FA_KV_Q8_0, 34), "q4_0": (FA_KV_Q4_0, 18),
            "fp8_e4m3": (FA_KV_FP8_E4M3, 32)}  # type code, bytes per 32 values

_lib = None


def load():
    """Load libfa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libfa.so is not built (run python -m attention_attn_fwd_11_b200.build)")
        lib = ctypes.CDLL(LIB_PATH)
        lib.fa_fwd.argtypes = [ctypes.POINTER(FwdParams), _vp]
        lib.fa_fwd.restype = _i32
        lib.fa_prefill_paged.argtypes = [ctypes.POINTER(PrefillPagedParams), _vp]
        lib.fa_prefill_paged.restype = _i32
        lib.fa_decode_paged_workspace_size.argtypes = [ctypes.POINTER(PagedParams), ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_decode_paged_workspace_size.restype = _i32
        lib.fa_decode_paged.argtypes = [ctypes.POINTER(PagedParams), _vp]
        lib.fa_decode_paged.restype = _i32
        lib.fa_decode_gather_workspace_size.argtypes = [ctypes.POINTER(GatherParams), ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_decode_gather_workspace_size.restype = _i32
        lib.fa_decode_gather.argtypes = [ctypes.POINTER(GatherParams), _vp]
        lib.fa_decode_gather.restype = _i32
        lib.fa_mla_tail_workspace_size.argtypes = [ctypes.POINTER(MlaTailParams), ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_mla_tail_workspace_size.restype = _i32
        lib.fa_mla_tail.argtypes = [ctypes.POINTER(MlaTailParams), _vp]
        lib.fa_mla_tail.restype = _i32
        lib.fa_kv_dequant.argtypes = [ctypes.POINTER(KvDequantParams), _vp]
        lib.fa_kv_dequant.restype = _i32
        lib.fa_kv_dequant_n.argtypes = [ctypes.POINTER(KvDequantParams), _i32, _vp]
        lib.fa_kv_dequant_n.restype = _i32
        lib.fa_bwd_workspace_size.argtypes = [ctypes.POINTER(BwdParams), ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_bwd_workspace_size.restype = _i32
        lib.fa_bwd_workspace_need.argtypes = [ctypes.POINTER(BwdParams), ctypes.POINTER(ctypes.c_size_t)]
        lib.fa_bwd_workspace_need.restype = _i32
        lib.fa_bwd.argtypes = [ctypes.POINTER(BwdParams), _vp]
        lib.fa_bwd.restype = _i32
        lib.fa_rope.argtypes = [ctypes.POINTER(RopeParams), _vp]
        lib.fa_rope.restype = _i32
        lib.fa_kv_append.argtypes = [ctypes.POINTER(KvAppendParams), _vp]
        lib.fa_kv_append.restype = _i32
        lib.fa_last_error.argtypes = []
        lib.fa_last_error.restype = ctypes.c_char_p
        lib.fa_device_error.argtypes = [_i32, ctypes.POINTER(_i32)]
        lib.fa_device_error.restype = _i32
        lib.fa_version.restype = _i32
        _lib = lib
    return _lib


class FAError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s: %s" % (STATUS_NAMES.get(status, status), msg))
        self.status = status


def _check(st):
    if st != FA_OK:
        raise FAError(st, load().fa_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    """The current stream's handle, without building a Stream object (3 us)."""
    return _vp(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def _on(stream, call, *args, **kwargs):
    """call(*args) with the given stream as the current one, so that what it
    makes -- outputs, workspaces, temporaries -- comes from that stream's own
    memory: a block that another stream has freed may still be in use by work
    queued there, which the given stream does not wait for.  The memory of
    every tensor given outlasts the kernels, and that of the results also
    what the caller queues on its own current stream."""
    before = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        got = call(*args, **kwargs)
    for t in _tensors((args, tuple(kwargs.values()))):
        t.record_stream(stream)
    for t in _tensors(got):
        t.record_stream(stream)
        t.record_stream(before)
    return got


def _tensors(x):
    """The CUDA tensors in x, a tensor or (nested) tuples and lists."""
    if isinstance(x, torch.Tensor):
        if x.is_cuda:
            yield x
    elif isinstance(x, (tuple, list)):
        for y in x:
            yield from _tensors(y)


def _workspace(ws):
    """(address, bytes) of a workspace tensor."""
    if ws is None:
        return None, 0
    if not ws.is_contiguous():  # its elements would not fill the bytes from its address on
        raise ValueError("the workspace must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libfa works on CUDA tensors only (no CPU fallback)")


def _need_current_device(*ts):
    """CUDA tensors of one device, the current one (the library launches there)."""
    current = None
    for t in ts:
        if t is not None and t.get_device() != current:
            _need_cuda(t)
            if current is not None or t.get_device() != torch.cuda.current_device():
                raise ValueError("every tensor must be on the current CUDA device (see torch.cuda.device)")
            current = t.get_device()


def _odt(dtype):
    if dtype == torch.bfloat16:
        return FA_BF16
    if dtype == torch.float32:
        return FA_F32
    raise ValueError("output dtype must be float32 or bfloat16")


# ------------------------------------------------------------------ prefill --

def fwd_params(q, k, v, o, lse, scale, causal, mask=None, max_bias=0.0, softcap=0.0, sinks=None):
    B, Hq, Sq, dk = q.shape
    _, Hkv, Sk, dv = v.shape
    p = FwdParams()
    p.q, p.k, p.v, p.o, p.lse = _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse)
    p.B, p.Hq, p.Hkv, p.Sq, p.Sk, p.dk, p.dv = B, Hq, Hkv, Sq, Sk, dk, dv
    p.q_sb, p.q_sh, p.q_ss = q.stride(0), q.stride(1), q.stride(2)
    p.k_sb, p.k_sh, p.k_ss = k.stride(0), k.stride(1), k.stride(2)
    p.v_sb, p.v_sh, p.v_ss = v.stride(0), v.stride(1), v.stride(2)
    p.o_sb, p.o_sh, p.o_ss = o.stride(0), o.stride(1), o.stride(2)
    p.scale = scale
    p.causal = 1 if causal else 0
    p.o_dtype = _odt(o.dtype)
    if mask is not None:  # [Bm, Hm, Sq, Sk] f16; a size-1 batch or head dim broadcasts
        p.mask = _ptr(mask)
        p.m_sb = 0 if mask.shape[0] == 1 else mask.stride(0)
        p.m_sh = 0 if mask.shape[1] == 1 else mask.stride(1)
        p.m_ss = mask.stride(2)
    p.max_bias = max_bias
    p.softcap = softcap
    p.sinks = _ptr(sinks)
    return p


def fwd(q, k, v, scale=None, causal=False, out=None, return_lse=True, out_dtype=torch.float32, stream=None,
        mask=None, max_bias=0.0, softcap=0.0, sinks=None, lse=None):
    """O = softmax(scale * Q K^T + mask) V.  q [B,Hq,Sq,dk], k [B,Hkv,Sk,dk],
    v [B,Hkv,Sk,dv] bf16 CUDA tensors (any strides, head dim contiguous).
    Score modifiers (see fa_fwd in include/fa.h): mask [1|B, 1|Hq, Sq, Sk]
    float16 CUDA tensor with a contiguous last dim, max_bias (ALiBi slopes
    applied to the mask), softcap, sinks [Hq] float32 CUDA tensor.  out and
    lse may be given preallocated (lse: contiguous float32 [B,Hq,Sq]).
    Returns (O [B,Hq,Sq,dv], LSE [B,Hq,Sq] fp32 or None)."""
    if stream is not None:
        return _on(stream, fwd, q, k, v, scale, causal, out, return_lse, out_dtype, None, mask, max_bias, softcap,
                   sinks, lse)
    _need_cuda(q, k, v)
    if mask is not None:
        _need_cuda(mask)
        if mask.dtype != torch.float16 or mask.dim() != 4 or mask.stride(3) != 1:
            raise ValueError("mask must be a 4-D float16 tensor with a contiguous last dim")
    if sinks is not None:
        _need_cuda(sinks)
        if sinks.dtype != torch.float32 or sinks.shape != (q.shape[1],) or not sinks.is_contiguous():
            raise ValueError("sinks must be a contiguous float32 tensor of shape [Hq]")
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or t.dim() != 4 or t.stride(3) != 1:
            raise ValueError("q, k, v must be 4-D bf16 with a contiguous last dim")
    B, Hq, Sq, dk = q.shape
    dv = v.shape[3]
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if out is None:
        out = torch.empty((B, Hq, Sq, dv), device=q.device, dtype=out_dtype)
    if lse is not None:
        if lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Sq) or not lse.is_contiguous() or not lse.is_cuda:
            raise ValueError("lse must be a contiguous float32 CUDA tensor [B, Hq, Sq]")
    elif return_lse:
        lse = torch.empty((B, Hq, Sq), device=q.device, dtype=torch.float32)
    params = fwd_params(q, k, v, out, lse, scale, causal, mask, max_bias, softcap, sinks)
    _check(load().fa_fwd(ctypes.byref(params), _stream()))
    return out, lse


# ---------------------------------------------------------------- backward --

def _bwd_sizes(q, k, v):
    p = BwdParams()
    p.B, p.Hq, p.Sq, p.dk = map(_int, q.shape)
    p.Hkv, p.Sk, p.dv = map(_int, v.shape[1:])
    p.scale = 1.0
    return p


def bwd_workspace_bytes(q, k, v, causal=None):
    """Workspace of bwd() for these shapes, causal or not, or (given causal)
    for that alone.  A smaller shape can need more than a larger one."""
    n = ctypes.c_size_t(0)
    p = _bwd_sizes(q, k, v)
    if causal is None:
        _check(load().fa_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    else:
        p.causal = 1 if causal else 0
        _check(load().fa_bwd_workspace_need(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def bwd(q, k, v, o, lse, do, scale=None, causal=False, mask=None, max_bias=0.0, softcap=0.0, sinks=None, dlse=None,
        dq=None, dk=None, dv=None, grad_dtype=torch.bfloat16, workspace=None, stream=None):
    """Gradients of fwd() (fa_bwd), from its inputs, its output o and lse and
    the output's gradient do [B,Hq,Sq,dv] (bf16); the same scale, causal and
    modifiers as fwd() had.  dlse: the gradient of the log-sum-exp, if it is
    used ([B,Hq,Sq] float32).  dq, dk, dv may be given (any strides, head dim
    contiguous), else they are made in grad_dtype (bf16 or float32).
    (dk, dv) head sizes: (64, 64), (128, 128), (192, 128).
    Returns (dq, dk, dv), and with sinks (dq, dk, dv, dsinks [Hq] float32)."""
    if stream is not None:
        return _on(stream, bwd, q, k, v, o, lse, do, scale, causal, mask, max_bias, softcap, sinks, dlse, dq, dk, dv,
                   grad_dtype, workspace)
    _need_current_device(q, k, v, o, lse, do, mask, sinks, dlse, dq, dk, dv, workspace)
    bf16 = torch.bfloat16
    if lse is None:
        raise ValueError("lse, the log-sum-exp that fwd() returns, must be given")
    if q.dtype != bf16 or k.dtype != bf16 or v.dtype != bf16 or do.dtype != bf16:
        raise ValueError("q, k, v and do must be bf16")
    qs, ks, vs, os = q.shape, k.shape, v.shape, o.shape
    if not len(qs) == len(ks) == len(vs) == len(os) == 4:
        raise ValueError("q, k, v, o and do must be 4-D")
    B, Hq, Sq, hd = qs
    _, Hkv, Sk, vd = vs
    if ks != (B, Hkv, Sk, hd) or vs[0] != B:
        raise ValueError("k must be [B, Hkv, Sk, dk] and v [B, Hkv, Sk, dv] with q's B and dk")
    if os != (B, Hq, Sq, vd) or os != do.shape:
        raise ValueError("o and do must be [B, Hq, Sq, dv]")
    for t in (lse, dlse):
        if t is not None and (t.dtype != torch.float32 or t.shape != (B, Hq, Sq) or not t.is_contiguous()):
            raise ValueError("lse and dlse must be contiguous float32 [B, Hq, Sq]")
    if dq is None:
        dq = torch.empty_like(q) if grad_dtype == bf16 else torch.empty_like(q, dtype=grad_dtype)
    if dk is None:
        dk = torch.empty_like(k) if grad_dtype == bf16 else torch.empty_like(k, dtype=grad_dtype)
    if dv is None:
        dv = torch.empty_like(v) if grad_dtype == bf16 else torch.empty_like(v, dtype=grad_dtype)
    if dq.shape != qs or dk.shape != ks or dv.shape != vs or dk.dtype != dq.dtype or dv.dtype != dq.dtype:
        raise ValueError("dq, dk and dv must have the shapes of q, k and v and one dtype")
    q0, q1, q2, q3 = q.stride()
    k0, k1, k2, k3 = k.stride()
    v0, v1, v2, v3 = v.stride()
    o0, o1, o2, o3 = o.stride()
    g0, g1, g2, g3 = do.stride()
    a0, a1, a2, a3 = dq.stride()
    b0, b1, b2, b3 = dk.stride()
    c0, c1, c2, c3 = dv.stride()
    if not q3 == k3 == v3 == o3 == g3 == a3 == b3 == c3 == 1:
        raise ValueError("the last dim of q, k, v, o, do and the gradients must be contiguous")
    p = _pack_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                  dlse.data_ptr() if dlse is not None else 0, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                  B, Hq, Hkv, Sq, Sk, hd, vd, q0, q1, q2, k0, k1, k2, v0, v1, v2, o0, o1, o2, g0, g1, g2, a0, a1, a2,
                  b0, b1, b2, c0, c1, c2, 1.0 / math.sqrt(hd) if scale is None else scale, 1 if causal else 0,
                  _odt(o.dtype), _odt(dq.dtype))
    if mask is not None:  # [Bm, Hm, Sq, Sk] f16; a size-1 batch or head dim broadcasts
        if (mask.dtype != torch.float16 or mask.dim() != 4 or mask.stride(3) != 1 or mask.shape[0] not in (1, B) or
                mask.shape[1] not in (1, Hq) or mask.shape[2:] != (Sq, Sk)):
            raise ValueError("mask must be [1|B, 1|Hq, Sq, Sk] float16 with a contiguous last dim")
        p.mask = mask.data_ptr()
        p.m_sb = 0 if mask.shape[0] == 1 else mask.stride(0)
        p.m_sh = 0 if mask.shape[1] == 1 else mask.stride(1)
        p.m_ss = mask.stride(2)
    p.max_bias, p.softcap = max_bias, softcap
    dsinks = None
    if sinks is not None:
        if sinks.dtype != torch.float32 or sinks.shape != (Hq,) or not sinks.is_contiguous():
            raise ValueError("sinks must be a contiguous float32 tensor of shape [Hq]")
        dsinks = torch.empty_like(sinks)
        p.sinks, p.gsinks = sinks.data_ptr(), dsinks.data_ptr()
    lib = load()
    ref = ctypes.byref(p)
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check(lib.fa_bwd_workspace_need(ref, ctypes.byref(n)))
        workspace = torch.empty(n.value, device=q.device, dtype=torch.uint8)
    p.workspace, p.workspace_bytes = _workspace(workspace)
    _check(lib.fa_bwd(ref, _stream()))
    return (dq, dk, dv) if sinks is None else (dq, dk, dv, dsinks)


# ------------------------------------------------------------- paged decode --

def _paged_kv(q, v_cache, kv_type):
    """(cache type, dv) of a paged cache: bf16 rows, or uint8 rows of q8_0
    (34 bytes per 32 values), q4_0 (18) or fp8 e4m3 (32) -- told apart by
    the row length against dk when kv_type is not given."""
    if v_cache.dtype != torch.uint8:
        return None, v_cache.shape[3]
    if kv_type is None:
        dk, r = q.shape[-1], v_cache.shape[3]
        kv_type = {dk // 32 * 34: "q8_0", dk // 32 * 18: "q4_0", dk: "fp8_e4m3"}.get(r)
        if kv_type is None:
            raise ValueError("cannot tell the cache type from a row of %d bytes; pass kv_type" % r)
    return kv_type, v_cache.shape[3] // KV_QUANT[kv_type][1] * 32


def paged_params(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale, num_splits, ws, kv_type=None,
                 k_scale=1.0, v_scale=1.0):
    B, Hq, dk = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    p = PagedParams()
    p.q, p.k_cache, p.v_cache = _ptr(q), _ptr(k_cache), _ptr(v_cache)
    p.block_table, p.seq_lens = _ptr(block_table), _ptr(seq_lens)
    p.max_blocks_per_seq = block_table.shape[1]
    kv_type, dv = _paged_kv(q, v_cache, kv_type)
    if kv_type is not None:  # quantised rows, converted inside the kernel
        p.kv_type = KV_QUANT[kv_type][0]
        p.k_scale, p.v_scale = k_scale, v_scale
    p.B, p.Hq, p.Hkv, p.dk, p.dv, p.block_size, p.num_blocks = B, Hq, Hkv, dk, dv, bs, nb
    p.scale = scale
    p.num_splits = num_splits
    p.o, p.lse = _ptr(o), _ptr(lse)
    p.o_dtype = _odt(o.dtype) if o is not None else FA_F32
    p.workspace, p.workspace_bytes = _workspace(ws)
    return p


def paged_workspace_bytes(q, k_cache, v_cache, block_table, seq_lens, num_splits=0):
    p = paged_params(q, k_cache, v_cache, block_table, seq_lens, None, None, 1.0, num_splits, None)
    n = ctypes.c_size_t(0)
    _check(load().fa_decode_paged_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def decode_paged(q, k_cache, v_cache, block_table, seq_lens, scale=None, num_splits=0, out=None,
                 return_lse=True, out_dtype=torch.float32, workspace=None, stream=None, kv_type=None, k_scale=1.0,
                 v_scale=1.0):
    """Split-KV decode over a paged cache.  q [B,Hq,dk]; caches
    [num_blocks,Hkv,block_size,d] bf16, or uint8 [...,136] of q8_0 rows,
    [...,72] of q4_0 rows, or [...,128] of fp8 e4m3 bytes read as
    e4m3 * k_scale / v_scale (dequantised in the kernel); block_table int32
    [B,max_blocks]; seq_lens int32 [B].  Returns (O [B,Hq,dv], LSE [B,Hq] or
    None)."""
    if stream is not None:
        return _on(stream, decode_paged, q, k_cache, v_cache, block_table, seq_lens, scale, num_splits, out, return_lse,
                   out_dtype, workspace, None, kv_type, k_scale, v_scale)
    _need_cuda(q, k_cache, v_cache, block_table, seq_lens, out, workspace)
    B, Hq, dk = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    kv_type, dv = _paged_kv(q, v_cache, kv_type)
    if out is None:
        out = torch.empty((B, Hq, dv), device=q.device, dtype=out_dtype)
    lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32) if return_lse else None
    if workspace is None:
        n = paged_workspace_bytes(q, k_cache, v_cache, block_table, seq_lens, num_splits)
        workspace = torch.empty(max(n, 256), device=q.device, dtype=torch.uint8)
    p = paged_params(q, k_cache, v_cache, block_table, seq_lens, out, lse, scale, num_splits, workspace, kv_type,
                     k_scale, v_scale)
    _check(load().fa_decode_paged(ctypes.byref(p), _stream()))
    return out, lse


# ----------------------------------------------------------- paged prefill --

def prefill_paged_params(q, k_cache, v_cache, block_table, seq_lens, o, lse, scale, causal, q_lens=None,
                         mask=None, max_bias=0.0, softcap=0.0, sinks=None):
    B, Hq, Sq, dk = q.shape
    nb, Hkv, bs, _ = k_cache.shape
    p = PrefillPagedParams()
    p.q, p.q_sb, p.q_sh, p.q_ss = _ptr(q), q.stride(0), q.stride(1), q.stride(2)
    p.k_cache, p.v_cache = _ptr(k_cache), _ptr(v_cache)
    p.block_table, p.seq_lens = _ptr(block_table), _ptr(seq_lens)
    p.max_blocks_per_seq = block_table.shape[1]
    p.B, p.Hq, p.Hkv, p.Sq, p.dk, p.dv = B, Hq, Hkv, Sq, dk, v_cache.shape[3]
    p.block_size, p.num_blocks = bs, nb
    p.scale, p.causal = scale, 1 if causal else 0
    p.o, p.o_sb, p.o_sh, p.o_ss = _ptr(o), o.stride(0), o.stride(1), o.stride(2)
    p.lse = _ptr(lse)
    p.o_dtype = _odt(o.dtype)
    p.q_lens = _ptr(q_lens)
    if mask is not None:
        p.mask = _ptr(mask)
        p.m_sb = mask.stride(0) if mask.shape[0] > 1 else 0
        p.m_sh = mask.stride(1) if mask.shape[1] > 1 else 0
        p.m_ss = mask.stride(2)
    p.max_bias, p.softcap, p.sinks = max_bias, softcap, _ptr(sinks)
    return p


def prefill_paged(q, k_cache, v_cache, block_table, seq_lens, scale=None, causal=True, out=None,
                  return_lse=True, out_dtype=torch.float32, stream=None, q_lens=None, mask=None, max_bias=0.0,
                  softcap=0.0, sinks=None):
    """Chunked prefill over a paged cache (fa_prefill_paged).  q [B,Hq,Sq,dk]
    bf16 (head dim contiguous); k_cache [num_blocks,Hkv,64,dk], v_cache
    [num_blocks,Hkv,64,dv] bf16 contiguous, (dk, dv) a pair fwd() takes; block_table int32 [B,max_blocks]; seq_lens int32 [B] (keys
    including the new ones); q_lens: None or int32 [B], new rows per
    sequence (rows past it come back as O = 0, LSE = -inf); mask [1|B, 1|Hq,
    Sq, >= max seq_len] float16 (last dim contiguous), max_bias, softcap,
    sinks [Hq] float32: the score modifiers of fwd().
    Returns (O [B,Hq,Sq,dv], LSE [B,Hq,Sq] or None)."""
    if stream is not None:
        return _on(stream, prefill_paged, q, k_cache, v_cache, block_table, seq_lens, scale, causal, out, return_lse,
                   out_dtype, None, q_lens, mask, max_bias, softcap, sinks)
    _need_cuda(mask, sinks)
    if mask is not None and (mask.dtype != torch.float16 or mask.dim() != 4 or mask.stride(3) != 1):
        raise ValueError("mask must be a 4-D float16 tensor with a contiguous last dim")
    if sinks is not None and (sinks.dtype != torch.float32 or not sinks.is_contiguous()):
        raise ValueError("sinks must be contiguous float32 [Hq]")
    _need_cuda(q, k_cache, v_cache, block_table, seq_lens, out, q_lens)
    if q_lens is not None and (q_lens.dtype != torch.int32 or not q_lens.is_contiguous()):
        raise ValueError("q_lens must be contiguous int32")
    for t in (q, k_cache, v_cache):
        if t.dtype != torch.bfloat16 or t.stride(-1) != 1:
            raise ValueError("q and the caches must be bf16 with a contiguous head dimension")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("the caches must be contiguous")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32 or not block_table.is_contiguous():
        raise ValueError("block_table and seq_lens must be contiguous int32")
    B, Hq, Sq, dk = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if out is None:
        out = torch.empty((B, Hq, Sq, v_cache.shape[3]), device=q.device, dtype=out_dtype)
    lse = torch.empty((B, Hq, Sq), device=q.device, dtype=torch.float32) if return_lse else None
    p = prefill_paged_params(q, k_cache, v_cache, block_table, seq_lens, out, lse, scale, causal, q_lens, mask,
                             max_bias, softcap, sinks)
    _check(load().fa_prefill_paged(ctypes.byref(p), _stream()))
    return out, lse


# ------------------------------------------------------------ gather decode --

def gather_params(q, rows, idx, key_pos, q_pos, o, lse, scale, num_splits, ws, dk=576, dv=512, v_offset=64,
                  topk=None):
    T, Hq, _ = q.shape
    p = GatherParams()
    p.q, p.kv_rows = _ptr(q), _ptr(rows)
    p.n_rows, p.row_stride = rows.shape[0], rows.stride(0)
    p.dk, p.dv, p.v_offset = dk, dv, v_offset
    p.idx, p.topk = _ptr(idx), (idx.shape[1] if idx is not None else int(topk))
    p.key_pos, p.q_pos = _ptr(key_pos), _ptr(q_pos)
    p.T, p.Hq = T, Hq
    p.scale = scale
    p.num_splits = num_splits
    p.o, p.lse = _ptr(o), _ptr(lse)
    p.o_dtype = _odt(o.dtype) if o is not None else FA_F32
    p.workspace, p.workspace_bytes = _workspace(ws)
    return p


def gather_workspace_bytes(q, rows, idx, num_splits=0, topk=None, dk=576):
    p = gather_params(q, rows, idx, None, None, None, None, 1.0, num_splits, None, topk=topk, dk=dk,
                      v_offset=64 if dk == 576 else 0)
    n = ctypes.c_size_t(0)
    _check(load().fa_decode_gather_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def decode_gather(q, rows, idx, key_pos=None, q_pos=None, scale=None, num_splits=0, out=None, return_lse=True,
                  out_dtype=torch.float32, workspace=None, stream=None, topk=None, dk=576):
    """Latent sparse decode.  q [T,Hq,576]; rows [n_rows, >=576] bf16 (row
    pitch = rows.stride(0)); idx int32 [T,topk] (-1 = empty), or None with
    ``topk`` given: every token reads rows 0 .. topk - 1; key_pos int32
    [T,topk] or None; q_pos int32 [T] or None.
    Returns (O [T,Hq,512], LSE [T,Hq] or None)."""
    if stream is not None:
        return _on(stream, decode_gather, q, rows, idx, key_pos, q_pos, scale, num_splits, out, return_lse, out_dtype,
                   workspace, None, topk, dk)
    _need_cuda(q, rows, idx, key_pos, q_pos, out, workspace)
    if rows.stride(1) != 1:
        raise ValueError("rows must have a contiguous last dim")
    T, Hq, dk = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(dk)
    if out is None:
        out = torch.empty((T, Hq, 512), device=q.device, dtype=out_dtype)
    lse = torch.empty((T, Hq), device=q.device, dtype=torch.float32) if return_lse else None
    if workspace is None:
        n = gather_workspace_bytes(q, rows, idx, num_splits, topk=topk, dk=dk)
        workspace = torch.empty(max(n, 256), device=q.device, dtype=torch.uint8)
    p = gather_params(q, rows, idx, key_pos, q_pos, out, lse, scale, num_splits, workspace, topk=topk,
                      dk=dk, v_offset=64 if dk == 576 else 0)
    _check(load().fa_decode_gather(ctypes.byref(p), _stream()))
    return out, lse


def prefill_latent(q, rows, causal=True, scale=None, num_splits=0, out=None, return_lse=True,
                   out_dtype=torch.float32, workspace=None, stream=None, dk=576):
    """Prefill in latent space (MLA with the absorbed query): Sq new tokens,
    each with Hq = 128 heads, against the Sk latent rows [k_pe | kv_latent]
    of the sequence, rows 0 .. Sk - 1 of ``rows`` -- the (dk, dv) = (576,
    512) attention of the llama.cpp tensor path's head-size table, all heads
    sharing one latent row per key.  q [Sq, 128, 576]; with causal, new
    token t sits at position Sk - Sq + t.  dk=512: the (512, 512) pair, rows
    of 512 that are both key and value (q [Sq, 128, 512]).  Runs
    fa_decode_gather with contiguous rows (idx NULL).
    Returns (O [Sq, 128, 512], LSE [Sq, 128])."""
    if stream is not None:
        return _on(stream, prefill_latent, q, rows, causal, scale, num_splits, out, return_lse, out_dtype, workspace,
                   None, dk)
    _need_cuda(q, rows)
    Sq, Sk = q.shape[0], rows.shape[0]
    q_pos = None
    if causal:
        q_pos = torch.arange(Sk - Sq, Sk, device=q.device, dtype=torch.int32)
    return decode_gather(q, rows, None, q_pos=q_pos, scale=scale, num_splits=num_splits, out=out,
                         return_lse=return_lse, out_dtype=out_dtype, workspace=workspace, topk=Sk, dk=dk)


def device_error(clear=True) -> int:
    """Device-side error word (FA_DEVERR_*); synchronises the device."""
    c = _i32(0)
    _check(load().fa_device_error(1 if clear else 0, ctypes.byref(c)))
    return c.value


# ------------------------------------------------------ quantised K/V rows --

def kv_dequant_params(src, qtype, row_elems, dst, kv_scale=1.0):
    """Marshal a fa_kv_dequant call: src uint8 [..., row_bytes] (rows of
    ggml blocks or fp8 bytes), dst bf16 [..., >= row_elems] with unit stride
    in the last dimension and the same leading shape, both contiguous over
    the rows; kv_scale: the fp8 tensor scale."""
    code, _ = KV_QUANT[qtype]
    p = KvDequantParams()
    p.src, p.type, p.row_elems, p.dst = _ptr(src), code, row_elems, _ptr(dst)
    p.scale = kv_scale
    p.n_rows = src.numel() // src.shape[-1] if src.dim() else 0
    p.src_row_bytes = src.stride(-2) if src.dim() > 1 else src.shape[-1]
    p.dst_row_stride = dst.stride(-2) if dst.dim() > 1 else dst.shape[-1]
    return p


def _dequant_entry(src, qtype, row_elems, out, kv_scale=1.0):
    _need_cuda(src, out)
    if src.dtype != torch.uint8:
        raise ValueError("src must be uint8 blocks")
    if src.stride(-1) != 1:
        raise ValueError("src rows must be contiguous")
    *lead, width = src.shape
    whole = src.is_contiguous()
    if out is None:
        out = torch.empty((*lead, row_elems), device=src.device, dtype=torch.bfloat16)
    else:
        shape = out.shape
        if out.dtype != torch.bfloat16 or [*shape[:-1]] != lead or shape[-1] < row_elems or out.stride(-1) != 1:
            raise ValueError("out must be bf16 [..., >= row_elems] with the rows of src")
        whole = whole and out.is_contiguous()
    if whole and lead and width > 0:
        # one row stride each, without building the 2-D views (6 us of host time for two tensors)
        return KvDequantParams(src.data_ptr(), KV_QUANT[qtype][0], src.numel() // width, row_elems, width,
                               out.data_ptr(), out.shape[-1], kv_scale), out
    s2, o2 = src.reshape(-1, src.shape[-1]), out.reshape(-1, out.shape[-1])
    if s2.data_ptr() != src.data_ptr() or o2.data_ptr() != out.data_ptr():
        raise ValueError("leading dimensions must collapse to one row stride")
    return kv_dequant_params(s2, qtype, row_elems, o2, kv_scale), out


def kv_dequant(src, qtype, row_elems, out=None, stream=None, kv_scale=1.0):
    """Quantised rows -> bf16 rows on the GPU (fa_kv_dequant).  src: uint8
    CUDA tensor [..., row_bytes] whose rows each hold row_elems values of
    ``qtype`` ('q8_0' or 'q4_0' ggml blocks, or 'fp8_e4m3' bytes read as
    e4m3 * kv_scale); the leading dimensions must collapse to one row index
    with a single stride.  Returns (or fills) a bf16 tensor [..., row_elems]."""
    if stream is not None:
        return _on(stream, kv_dequant, src, qtype, row_elems, out, None, kv_scale)
    p, out = _dequant_entry(src, qtype, row_elems, out, kv_scale)
    _check(load().fa_kv_dequant(ctypes.byref(p), _stream()))
    return out


def kv_dequant_many(entries, stream=None):
    """Several conversions in one launch (fa_kv_dequant_n).  entries: list of
    (src, qtype, row_elems, out-or-None[, kv_scale]), 1 to 4 of them, one
    qtype.  Returns the list of outputs."""
    if stream is not None:
        return _on(stream, kv_dequant_many, entries)
    made = [_dequant_entry(*e) for e in entries]
    arr = (KvDequantParams * len(made))(*[m[0] for m in made])
    _check(load().fa_kv_dequant_n(arr, len(made), _stream()))
    return [m[1] for m in made]


def fwd_quant(q, k_blocks, v_blocks, qtype, dk, dv, scale=None, causal=False, out=None, return_lse=True,
              out_dtype=torch.float32, k_buf=None, v_buf=None, stream=None, k_scale=1.0, v_scale=1.0, **mods):
    """Prefill over quantised K/V, the pages' way: dequantise K and V to bf16
    (one fa_kv_dequant_n launch for both) and run fa_fwd on them.  k_blocks /
    v_blocks: uint8 [B, Hkv, Sk, dk / 32 * block bytes] and [..., dv / 32 *
    block bytes]; k_buf / v_buf: optional bf16 [B, Hkv, Sk, dk / dv] buffers
    for the dequantised rows (allocated when absent); k_scale / v_scale: the
    fp8 tensor scales.  Other arguments as fwd()."""
    if stream is not None:
        return _on(stream, fwd_quant, q, k_blocks, v_blocks, qtype, dk, dv, scale, causal, out, return_lse, out_dtype,
                   k_buf, v_buf, None, k_scale, v_scale, **mods)
    k, v = kv_dequant_many([(k_blocks, qtype, dk, k_buf, k_scale), (v_blocks, qtype, dv, v_buf, v_scale)])
    return fwd(q, k, v, scale=scale, causal=causal, out=out, return_lse=return_lse, out_dtype=out_dtype, **mods)


# --------------------------------------------------------- MLA decode tail --

def mla_tail_params(o_lat, w_abs, w_o, y, num_splits=0, workspace=None):
    T, Hq, R = o_lat.shape
    p = MlaTailParams()
    p.o_lat, p.w_abs, p.w_o, p.y = _ptr(o_lat), _ptr(w_abs), _ptr(w_o), _ptr(y)
    p.T, p.Hq, p.R, p.V, p.Hd = T, Hq, R, w_abs.shape[1], w_o.shape[0]
    p.y_dtype = _odt(y.dtype)
    p.num_splits = num_splits
    p.workspace, p.workspace_bytes = _workspace(workspace)
    return p


def mla_tail_workspace_bytes(o_lat, w_abs, w_o, num_splits=0):
    p = MlaTailParams()
    p.T, p.Hq, p.R = o_lat.shape
    p.V, p.Hd = w_abs.shape[1], w_o.shape[0]
    p.y_dtype, p.num_splits = FA_F32, num_splits
    n = ctypes.c_size_t(0)
    _check(load().fa_mla_tail_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return n.value


def mla_tail(o_lat, w_abs, w_o, out=None, out_dtype=torch.float32, num_splits=0, workspace=None, stream=None):
    """MLA decode tail (fa_mla_tail): y [T, Hd] = o-projection of the
    per-head out-absorb of o_lat [T, Hq, R].  w_abs [Hq, V, R]; w_o
    [Hd, Hq*V] (row = output feature).  All bf16, contiguous."""
    if stream is not None:
        return _on(stream, mla_tail, o_lat, w_abs, w_o, out, out_dtype, num_splits, workspace)
    _need_cuda(o_lat, w_abs, w_o, out, workspace)
    for t in (o_lat, w_abs, w_o):
        if t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError("o_lat, w_abs and w_o must be contiguous bf16")
    T = o_lat.shape[0]
    if out is None:
        out = torch.empty((T, w_o.shape[0]), device=o_lat.device, dtype=out_dtype)
    if workspace is None:
        n = mla_tail_workspace_bytes(o_lat, w_abs, w_o, num_splits)
        workspace = torch.empty(max(n, 256), device=o_lat.device, dtype=torch.uint8)
    p = mla_tail_params(o_lat, w_abs, w_o, out, num_splits, workspace)
    _check(load().fa_mla_tail(ctypes.byref(p), _stream()))
    return out


# --------------------------------------------------------- rotary positions --

def rope_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original_len=None, beta_fast=32.0,
                     beta_slow=1.0):
    """Angular frequencies for rope() and kv_append(): base ** (-2 i / rot_dim)
    for i < rot_dim / 2, as a float64 CPU tensor, and the factor (mscale) on
    the rotated columns.  For contexts ``factor`` (>= 1) times as long as the
    trained ``original_len``, scaling is one of
      None      none;
      "linear"  every frequency / factor;
      "ntk"     a larger base, factor ** (rot_dim / (rot_dim - 2)) times: the
                slowest pair is slowed by factor, the fastest not at all;
      "yarn"    by parts: pairs that turn more than beta_fast times over
                original_len are kept, those below beta_slow turns are slowed
                by factor, with a ramp over the pair index between, and
                mscale = 0.1 ln(factor) + 1.
    Returns (inv_freq, mscale)."""
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be positive and even")
    if not base > 1.0 or not factor >= 1.0:
        raise ValueError("base must be > 1 and factor >= 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "ntk":
        if rot_dim == 2:
            raise ValueError('scaling "ntk" needs rot_dim > 2')
        base = base * factor ** (rot_dim / (rot_dim - 2))
    inv = base ** (-2.0 * i / rot_dim)
    if scaling is None or scaling == "ntk":
        return inv, 1.0
    if scaling == "linear":
        return inv / factor, 1.0
    if scaling != "yarn":
        raise ValueError('scaling must be None, "linear", "ntk" or "yarn"')
    if original_len is None or original_len <= 0 or not beta_fast > beta_slow > 0:
        raise ValueError('scaling "yarn" needs original_len > 0 and beta_fast > beta_slow > 0')

    def pair(turns):  # the (fractional) pair that turns this often over original_len
        return rot_dim * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

    low = max(0, math.floor(pair(beta_fast)))
    high = min(rot_dim - 1, math.ceil(pair(beta_slow)))
    ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
    return inv / factor * ramp + inv * (1 - ramp), 0.1 * math.log(factor) + 1.0


def _check_inv_freq(inv_freq):
    if inv_freq.dtype != torch.float64 or inv_freq.is_cuda or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a 1-D contiguous float64 CPU tensor (see rope_frequencies)")


def _check_pos(pos, B, S):
    """Pitch of pos over the batch (0 broadcasts)."""
    if pos.dtype != torch.int32 or pos.shape not in ((B, S), (S,), (1, S)) or (S > 1 and pos.stride(-1) != 1):
        raise ValueError("pos must be an int32 tensor [S], [1, S] or [B, S] with a contiguous last dim")
    return pos.stride(0) if pos.dim() == 2 and pos.shape[0] > 1 else 0


def rope(q, inv_freq, k=None, pos=None, pos0=0, interleaved=False, offset=0, inverse=False, mscale=1.0, out=None,
         k_out=None, stream=None):
    """Rotary positions (fa_rope): the pairs of columns [offset, offset + 2
    len(inv_freq)) of q [B,Hq,S,d] and, if given, k [B,Hk,S,d] turned by their
    row's position times inv_freq (float64 CPU tensor, see rope_frequencies),
    one launch for both.  bf16 or fp32, any strides with a contiguous last
    dim.  pos: int32 CUDA tensor [S], [1,S] or [B,S], or None: row s is at
    pos0 + s.  inverse=True turns back: the gradient.  out / k_out may be
    given, also as q / k themselves.  Returns (q turned, k turned or None)."""
    if stream is not None:
        return _on(stream, rope, q, inv_freq, k, pos, pos0, interleaved, offset, inverse, mscale, out, k_out)
    _need_current_device(q, k, pos, out, k_out)
    dtype, qs = q.dtype, q.shape
    if (dtype != torch.bfloat16 and dtype != torch.float32) or len(qs) != 4:
        raise ValueError("q and k must be 4-D tensors of one dtype, bf16 or fp32")
    B, Hq, S, d = qs
    _check_inv_freq(inv_freq)
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    q0, q1, q2, q3 = q.stride()
    o0, o1, o2, o3 = out.stride()
    if out.shape != qs or out.dtype != dtype or q3 != 1 or o3 != 1:
        raise ValueError("an output must have its input's shape and dtype, and all a contiguous last dim")
    k_in, k_made, Hk, k0, k1, k2, k3, r0, r1, r2, r3 = 0, 0, 0, 0, 0, 0, 1, 0, 0, 0, 1
    if k is not None:
        ks = k.shape
        if k.dtype != dtype or len(ks) != 4 or ks[0] != B or ks[2] != S or ks[3] != d:
            raise ValueError("k must be [B, Hk, S, d] with q's dtype, B, S and d")
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        k0, k1, k2, k3 = k.stride()
        r0, r1, r2, r3 = k_out.stride()
        if k_out.shape != ks or k_out.dtype != dtype or k3 != 1 or r3 != 1:
            raise ValueError("an output must have its input's shape and dtype, and all a contiguous last dim")
        k_in, k_made, Hk = k.data_ptr(), k_out.data_ptr(), ks[1]
    elif k_out is not None:
        raise ValueError("k_out without k")
    pos_sb, pos_in = (0, 0) if pos is None else (_check_pos(pos, B, S), pos.data_ptr())
    p = _pack_rope(q.data_ptr(), out.data_ptr(), q0, q1, q2, o0, o1, o2, k_in, k_made, k0, k1, k2, r0, r1, r2, B, Hq, Hk,
                   S, d, _odt(dtype), pos_in, pos_sb, pos0, inv_freq.data_ptr(), 2 * inv_freq.numel(), offset,
                   1 if interleaved else 0, 1 if inverse else 0, mscale)
    _check(load().fa_rope(ctypes.byref(p), _stream()))
    return out, k_out


# ------------------------------------------------------ paged cache append --

def kv_append(k, v, k_cache, v_cache, block_table, seq_lens, q_lens=None, inv_freq=None, mscale=1.0, pos=None,
              interleaved=False, offset=0, q=None, q_out=None, kv_type=None, k_scale=1.0, v_scale=1.0, stream=None):
    """New rows into a paged cache (fa_kv_append): k [B,Hkv,Sq,dk] and v
    [B,Hkv,Sq,dv] (bf16, any strides with a contiguous last dim) go to the
    last places of their sequences, whose lengths seq_lens [B] INCLUDE them
    (q_lens [B]: how many of the Sq rows each sequence has).  Caches,
    block_table and kv_type as in decode_paged().  With inv_freq the columns
    [offset, offset + 2 len(inv_freq)) of k are turned as by rope() first, at
    pos (int32 [B,Sq], [1,Sq] or [Sq]) or else the row's place in its
    sequence; q [B,Hq,Sq,dk], if given, is turned too.  Returns q turned (in
    q_out, which may be q; rows past q_lens are zeros), or None without q."""
    if stream is not None:
        return _on(stream, kv_append, k, v, k_cache, v_cache, block_table, seq_lens, q_lens, inv_freq, mscale, pos,
                   interleaved, offset, q, q_out, kv_type, k_scale, v_scale)
    _need_current_device(k, v, k_cache, v_cache, block_table, seq_lens, q_lens, q, q_out, pos)
    bf16, ks, vs, cs, cvs, ctype = torch.bfloat16, k.shape, v.shape, k_cache.shape, v_cache.shape, k_cache.dtype
    k0, k1, k2, k3 = k.stride() if len(ks) == 4 else (0, 0, 0, 0)
    v0, v1, v2, v3 = v.stride() if len(vs) == 4 else (0, 0, 0, 0)
    if k.dtype != bf16 or v.dtype != bf16 or k3 != 1 or v3 != 1:
        raise ValueError("k and v must be 4-D bf16 with a contiguous last dim")
    B, Hkv, Sq, dk = ks
    dv = vs[3]
    if vs != (B, Hkv, Sq, dv):
        raise ValueError("k and v must have one B, Hkv and Sq")
    if len(cs) != 4 or cvs != (*cs[:3], cvs[-1]) or cs[1] != Hkv or not (k_cache.is_contiguous() and
                                                                        v_cache.is_contiguous()):
        raise ValueError("the caches must be contiguous [num_blocks, Hkv, block_size, row] with k's Hkv")
    if v_cache.dtype != ctype or (ctype != bf16 and ctype != torch.uint8):
        raise ValueError("the caches must both be bf16, or both uint8 rows of a quantised type")
    for t, dim in ((block_table, 2), (seq_lens, 1), (q_lens, 1)):
        if t is not None and (t.dtype != torch.int32 or t.dim() != dim or t.shape[0] != B or not t.is_contiguous()):
            raise ValueError("block_table [B, max_blocks], seq_lens [B] and q_lens [B] must be contiguous int32")
    p = _pack_append(k.data_ptr(), v.data_ptr(), k0, k1, k2, v0, v1, v2, k_cache.data_ptr(), v_cache.data_ptr(),
                     block_table.data_ptr(), seq_lens.data_ptr(), q_lens.data_ptr() if q_lens is not None else 0,
                     block_table.shape[1], B, Hkv, Sq, dk, dv, cs[2], cs[0], 0)
    if ctype != bf16:
        kv_type, _ = _paged_kv(k, k_cache, kv_type)
        code, per = KV_QUANT[kv_type]
        if cs[3] != dk // 32 * per or cvs[3] != dv // 32 * per:
            raise ValueError("the cache rows do not hold k's and v's rows as " + kv_type)
        p.kv_type, p.k_scale, p.v_scale = code, k_scale, v_scale
    elif cs[3] != dk or cvs[3] != dv or kv_type is not None:
        raise ValueError("the rows of a bf16 cache must be as wide as those of k and v (and kv_type is for uint8 ones)")
    p.mscale = mscale
    if inv_freq is not None:
        _check_inv_freq(inv_freq)
        p.inv_freq, p.rot_dim, p.rot_offset = inv_freq.data_ptr(), _int(2 * inv_freq.numel()), _int(offset)
        p.interleaved = 1 if interleaved else 0
    if pos is not None:
        p.pos_sb, p.pos = _check_pos(pos, B, Sq), pos.data_ptr()
    if q is not None:
        if inv_freq is None:
            raise ValueError("q without inv_freq: there is nothing to turn it by")
        qs = q.shape
        if q.dtype != bf16 or len(qs) != 4 or qs[0] != B or qs[2] != Sq or qs[3] != dk:
            raise ValueError("q must be bf16 [B, Hq, Sq, dk] with k's B, Sq and dk")
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        q0, q1, q2, q3 = q.stride()
        o0, o1, o2, o3 = q_out.stride()
        if q_out.shape != qs or q_out.dtype != bf16 or q3 != 1 or o3 != 1:
            raise ValueError("q_out must have q's shape and dtype, and both a contiguous last dim")
        p.q, p.q_out, p.Hq = q.data_ptr(), q_out.data_ptr(), _int(qs[1])
        p.q_sb, p.q_sh, p.q_ss, p.qo_sb, p.qo_sh, p.qo_ss = q0, q1, q2, o0, o1, o2
    elif q_out is not None:
        raise ValueError("q_out without q")
    _check(load().fa_kv_append(ctypes.byref(p), _stream()))
    return q_out
