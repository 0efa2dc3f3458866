"""Thin ctypes binding over libtq (include/tq.h).  Argument marshalling only:
every step of the path runs in the library's CUDA kernels.  There is no
fallback: if libtq.so is missing the import of a compute function raises.

Functions keep the C names.  Device buffers are torch tensors (their data
pointers are passed); streams default to torch's current CUDA stream.
Every non-zero status raises ``TQError``.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

TQ_OK, TQ_ERR_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_ALIGN, TQ_ERR_WORKSPACE, TQ_ERR_CUDA, TQ_ERR_TIMEOUT = \
    0, -1, -2, -3, -4, -5, -6
TQ_F32, TQ_BF16, TQ_F16 = 0, 1, 2
_DT = {torch.float32: TQ_F32, torch.bfloat16: TQ_BF16, torch.float16: TQ_F16}


class tq_codebook(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("bits", ctypes.c_int), ("levels", ctypes.c_int),
                ("centroids", ctypes.c_float * 16), ("boundaries", ctypes.c_float * 15)]


class tq_signs(ctypes.Structure):
    _fields_ = [("w", ctypes.c_uint32 * 4)]


class tq_rope(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int), ("style", ctypes.c_int),
                ("axes", ctypes.c_int), ("axis", ctypes.c_uint8 * 64), ("turn", ctypes.c_uint64 * 64)]


class TQError(RuntimeError):
    def __init__(self, status, what):
        super().__init__("%s: %s (status %d)" % (what, tq_status_string(status), status))
        self.status = status


_lib = None


def lib():
    """Load libtq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libtq.so not built at %s; run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, c_int, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        cbp = ctypes.POINTER(tq_codebook)
        L.tq_codebook_load.argtypes = [c_int, c_int, cbp]
        L.tq_signs_from_seed.argtypes = [ctypes.c_uint64, c_int, ctypes.POINTER(tq_signs)]
        L.tq_block_bytes.argtypes = [c_int]
        L.tq_block_bytes.restype = sz
        L.tq_encode_kv.argtypes = [vp, c_int, i64, i64, cbp, tq_signs, vp, i64, vp, vp]
        L.tq_decode_kv.argtypes = [vp, i64, i64, cbp, tq_signs, vp, c_int, i64, vp]
        L.tq_qjl_encode.argtypes = [vp, c_int, i64, i64, vp, i64, cbp, tq_signs, vp, vp, vp, vp]
        L.tq_attn_workspace_bytes.argtypes = [c_int, c_int, c_int, c_int]
        L.tq_attn_workspace_bytes.restype = sz
        L.tq_attn_plan.argtypes = [c_int] * 8 + [ctypes.POINTER(i64)]
        L.tq_attn_plan_d.argtypes = [c_int] * 5 + [ctypes.POINTER(ctypes.c_int32)]
        L.tq_attn_decode.argtypes = [vp, c_int, vp, cbp, vp, cbp, vp, c_int, c_int, c_int, c_int, c_int,
                                     ctypes.c_float, tq_signs, vp, vp, vp, vp, vp, sz, vp]
        L.tq_serde_size.argtypes = [c_int] * 10
        L.tq_serde_size.restype = sz
        ser = [vp, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int, cbp, cbp, tq_signs, vp, vp]
        L.tq_serde_serialize.argtypes = ser
        L.tq_serde_deserialize.argtypes = ser
        L.tq_attn_prefill.argtypes = [vp, c_int, vp, cbp, vp, cbp, vp, c_int, c_int, c_int, c_int, c_int, c_int,
                                      ctypes.c_float, tq_signs, vp, vp]
        L.tq_block_bytes_ex.argtypes = [c_int, c_int]
        L.tq_block_bytes_ex.restype = sz
        L.tq_encode_kv_ex.argtypes = [vp, c_int, i64, i64, cbp, tq_signs, vp, i64, vp, c_int, vp]
        L.tq_decode_kv_ex.argtypes = [vp, i64, i64, cbp, tq_signs, vp, c_int, i64, c_int, vp]
        L.tq_attn_prefill_paged.argtypes = [vp, c_int, vp, cbp, vp, cbp, vp, c_int, c_int, vp, c_int, c_int, c_int,
                                            c_int, c_int, ctypes.c_float, tq_signs, vp, vp]
        L.tq_attn_decode_paged.argtypes = [vp, c_int, vp, cbp, vp, cbp, vp, c_int, c_int, vp, c_int, c_int, c_int,
                                           c_int, ctypes.c_float, tq_signs, vp, vp, sz, vp]
        L.tq_device_status.argtypes = [c_int, vp]
        L.tq_debug_drop_copies.argtypes = [c_int]
        L.tq_attn_workspace_bytes_sms.argtypes = [c_int] * 5
        L.tq_attn_workspace_bytes_sms.restype = sz
        L.tq_status_string.argtypes = [c_int]
        L.tq_status_string.restype = ctypes.c_char_p
        L.tq_block_bytes_d.argtypes = [c_int, c_int]
        L.tq_block_bytes_d.restype = sz
        L.tq_rotation_hadamard.argtypes = [c_int, tq_signs, vp]
        L.tq_encode_kv_d.argtypes = [vp, c_int, i64, c_int, cbp, vp, vp, vp]
        L.tq_decode_kv_d.argtypes = [vp, i64, c_int, cbp, vp, vp, c_int, vp]
        L.tq_attn_workspace_bytes_d.argtypes = [c_int] * 5
        L.tq_attn_workspace_bytes_d.restype = sz
        L.tq_attn_decode_d.argtypes = [vp, c_int, vp, cbp, vp, cbp, vp, c_int, c_int, c_int, c_int, c_int, c_int,
                                       ctypes.c_float, vp, vp, vp, sz, vp]
        rp = ctypes.POINTER(tq_rope)
        L.tq_rope_load.argtypes = [c_int, c_int, ctypes.c_double, c_int, c_int, ctypes.POINTER(c_int), c_int, rp]
        L.tq_rope_set_freqs.argtypes = [rp, ctypes.POINTER(ctypes.c_double)]
        L.tq_rope_apply.argtypes = [vp, c_int, i64, c_int, i64, i64, vp, i64, rp, vp, i64, i64, vp]
        L.tq_insert_kv.argtypes = [vp, i64, i64, vp, i64, i64, c_int, i64, c_int, vp, i64, rp, cbp, cbp, tq_signs, vp,
                                   vp, i64, vp, i64, vp]
        L.tq_attn_weights_workspace_bytes.argtypes = [c_int] * 4
        L.tq_attn_weights_workspace_bytes.restype = sz
        L.tq_attn_decode_weights.argtypes = [vp, c_int, vp, cbp, vp, cbp, vp, c_int, c_int, vp, c_int, c_int, c_int,
                                             c_int, c_int, ctypes.c_float, tq_signs, vp, i64, ctypes.c_float, vp,
                                             c_int, vp, sz, vp]
        L.tq_evict_select.argtypes = [vp, i64, vp, c_int, c_int, c_int, c_int, c_int, c_int, vp, vp, vp]
        L.tq_evict_compact.argtypes = [vp, c_int, vp, c_int, vp, i64, vp, c_int, vp, vp, c_int, c_int, c_int, c_int,
                                       c_int, c_int, c_int, vp]
        _lib = L
    return _lib


def _check(status, what):
    if status != TQ_OK:
        raise TQError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


# the current stream's handle without building a Stream object (3 us a call on the host)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dtype(t):
    if t.dtype not in _DT:
        raise TypeError("unsupported dtype %s" % t.dtype)
    return _DT[t.dtype]


def _row_stride(x):
    if x.dim() < 1 or x.shape[-1] != 128 or x.stride(-1) != 1:
        raise ValueError("rows of 128 contiguous elements expected")
    if x.dim() == 1:
        return 128
    # rows may be strided along one flattened leading axis
    return x.stride(-2)


def tq_status_string(status):
    return lib().tq_status_string(int(status)).decode()


def tq_codebook_load(head_dim=128, bits=4):
    cb = tq_codebook()
    _check(lib().tq_codebook_load(head_dim, bits, ctypes.byref(cb)), "tq_codebook_load")
    return cb


def tq_signs_from_seed(seed, head_dim=128):
    s = tq_signs()
    _check(lib().tq_signs_from_seed(ctypes.c_uint64(seed), head_dim, ctypes.byref(s)), "tq_signs_from_seed")
    return s


def tq_block_bytes(bits):
    return int(lib().tq_block_bytes(bits))


def _nvec_rows(x):
    """Number of 128-element rows of x and their stride (leading dims must
    flatten to one uniformly strided axis)."""
    if x.dim() == 1:
        return 1, 128
    n = x.numel()
    if n and x.is_contiguous():   # (a contiguous tensor's strides of size-1 dims can be anything)
        d = x.shape[-1]
        return n // d, d
    lead = x.shape[:-1]
    n = 1
    for s in lead:
        n *= s
    if n == 0:
        return 0, 128
    stride = x.stride(-2)
    expect = stride
    for i in range(x.dim() - 2, -1, -1):
        if x.shape[i] != 1 and x.stride(i) != expect:
            raise ValueError("leading dims of x must flatten to one strided axis")
        expect *= x.shape[i]
    return n, stride


def tq_encode_kv(x, cb, signs, blocks, block_stride_bytes=None, dst_index=None, block_offset=0, stream=None):
    """Encode the 128-element rows of ``x`` into ``blocks`` (uint8 tensor).

    Block of row i is written at byte ``block_offset + dst(i) * block_stride_bytes``
    of ``blocks``; dst(i) = i, or ``dst_index[i]`` (int64 device tensor)."""
    n, stride = _nvec_rows(x)
    bs = block_stride_bytes or tq_block_bytes(cb.bits)
    base = ctypes.c_void_p(blocks.data_ptr() + block_offset)
    _check(lib().tq_encode_kv(_ptr(x), _dtype(x), n, stride, ctypes.byref(cb), signs, base, bs,
                              _ptr(dst_index), _stream(stream)), "tq_encode_kv")
    return blocks


def tq_decode_kv(blocks, n_vec, cb, signs, out, block_stride_bytes=None, block_offset=0, stream=None):
    """Dequantise ``n_vec`` blocks into the 128-element rows of ``out``."""
    _, stride = _nvec_rows(out)
    bs = block_stride_bytes or tq_block_bytes(cb.bits)
    base = ctypes.c_void_p(blocks.data_ptr() + block_offset)
    _check(lib().tq_decode_kv(base, bs, n_vec, ctypes.byref(cb), signs, _ptr(out), _dtype(out), stride,
                              _stream(stream)), "tq_decode_kv")
    return out


def tq_qjl_encode(k, k_blocks, cb, signs, S, qjl_bits, res_norm_f16, block_stride_bytes=None, stream=None):
    n, stride = _nvec_rows(k)
    bs = block_stride_bytes or tq_block_bytes(cb.bits)
    _check(lib().tq_qjl_encode(_ptr(k), _dtype(k), n, stride, _ptr(k_blocks), bs, ctypes.byref(cb), signs,
                               _ptr(S), _ptr(qjl_bits), _ptr(res_norm_f16), _stream(stream)), "tq_qjl_encode")


def tq_attn_plan(B, Hq, Hkv, T, key_bits, value_bits, qjl=False, sms=0):
    """The tensor-core attention path's work partition for a shape, as a dict
    (C, Ctot, P, W, Smax, combine_groups, warps); raises TQError when the shape
    takes the split path or is invalid."""
    out = (ctypes.c_int64 * 7)()
    _check(lib().tq_attn_plan(B, Hq, Hkv, T, key_bits, value_bits, 1 if qjl else 0, sms, out), "tq_attn_plan")
    return dict(zip(("C", "Ctot", "P", "W", "Smax", "combine_groups", "warps"), (int(x) for x in out)))


def tq_attn_plan_d(B, Hkv, T, ctas_resident, warps_per_cta=4):
    """Host-only split plan of tq_attn_decode_d: (splits, tokens per split, most splits)."""
    out = (ctypes.c_int32 * 3)()
    _check(lib().tq_attn_plan_d(B, Hkv, T, ctas_resident, warps_per_cta, out), "tq_attn_plan_d")
    return int(out[0]), int(out[1]), int(out[2])


def tq_attn_workspace_bytes(B, Hq, Hkv, T_cap):
    return int(lib().tq_attn_workspace_bytes(B, Hq, Hkv, T_cap))


def tq_attn_decode(q, k_blocks, kcb, v, vcb, out, workspace, T, scale, signs, seq_lens=None,
                   qjl_bits=None, res_norm_f16=None, S=None, stream=None):
    """Decode attention.  q [B, Hq, 128]; k_blocks uint8 [B, Hkv, T_cap, kbytes];
    v uint8 blocks [B, Hkv, T_cap, vbytes] (vcb given) or fp16 [B, Hkv, T_cap, 128]
    (vcb None); out float32 [B, Hq, 128]; workspace uint8 device tensor."""
    B, Hq, _ = q.shape
    Hkv, T_cap = k_blocks.shape[1], k_blocks.shape[2]
    _check(lib().tq_attn_decode(_ptr(q), _dtype(q), _ptr(k_blocks), ctypes.byref(kcb), _ptr(v),
                                ctypes.byref(vcb) if vcb is not None else None, _ptr(seq_lens), B, Hq, Hkv,
                                T_cap, T, ctypes.c_float(scale), signs, _ptr(qjl_bits), _ptr(res_norm_f16),
                                _ptr(S), _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream)), "tq_attn_decode")
    return out


def tq_serde_size(num_layers, num_tokens, hidden_dim, block_size, skip_first, skip_last, key_bits,
                  value_bits, head_dim=128, elem_bytes=2):
    return int(lib().tq_serde_size(num_layers, num_tokens, hidden_dim, head_dim, block_size, skip_first,
                                   skip_last, key_bits, value_bits, elem_bytes))


def tq_serde_serialize(src, kcb, vcb, signs, dst, block_size=16, skip_first=2, skip_last=2, stream=None):
    """src: [2, L, T, hidden] bf16/fp16 device tensor; dst: uint8 device tensor."""
    _, L, T, hidden = src.shape
    _check(lib().tq_serde_serialize(_ptr(src), _dtype(src), L, T, hidden, 128, block_size, skip_first,
                                    skip_last, ctypes.byref(kcb), ctypes.byref(vcb), signs, _ptr(dst),
                                    _stream(stream)), "tq_serde_serialize")
    return dst


def tq_serde_deserialize(src, kcb, vcb, signs, dst, block_size=16, skip_first=2, skip_last=2, stream=None):
    """src: serialised uint8 device tensor; dst: [2, L, T, hidden] bf16/fp16 device tensor."""
    _, L, T, hidden = dst.shape
    _check(lib().tq_serde_deserialize(_ptr(src), _dtype(dst), L, T, hidden, 128, block_size, skip_first,
                                      skip_last, ctypes.byref(kcb), ctypes.byref(vcb), signs, _ptr(dst),
                                      _stream(stream)), "tq_serde_deserialize")
    return dst


def tq_device_status(clear=False, stream=None):
    """Sticky status of the kernels' bounded waits on the current device
    (TQ_OK or TQ_ERR_TIMEOUT; returned, not raised).  Synchronises the stream."""
    return int(lib().tq_device_status(1 if clear else 0, _stream(stream)))


def tq_debug_drop_copies(on):
    """Test hook: while on, kernels with bounded waits issue no copies, so
    their waits run out (include/tq.h)."""
    _check(lib().tq_debug_drop_copies(1 if on else 0), "tq_debug_drop_copies")


def tq_attn_workspace_bytes_sms(B, Hq, Hkv, T_cap, sms):
    return int(lib().tq_attn_workspace_bytes_sms(B, Hq, Hkv, T_cap, sms))


def tq_attn_prefill(q, k_blocks, kcb, v_blocks, vcb, out, T, scale, signs, seq_lens=None, stream=None):
    """Causal attention of M query tokens per sequence.  q [B, M, Hq, 128];
    k_blocks / v_blocks uint8 [B, Hkv, T_cap, bytes]; out float32 [B, M, Hq, 128]."""
    B, M, Hq, _ = q.shape
    Hkv, T_cap = k_blocks.shape[1], k_blocks.shape[2]
    _check(lib().tq_attn_prefill(_ptr(q), _dtype(q), _ptr(k_blocks), ctypes.byref(kcb), _ptr(v_blocks),
                                 ctypes.byref(vcb), _ptr(seq_lens), B, M, Hq, Hkv, T_cap, T, ctypes.c_float(scale),
                                 signs, _ptr(out), _stream(stream)), "tq_attn_prefill")
    return out


TQ_FMT_NORM_CORRECT, TQ_FMT_DENSE3 = 1, 2


def tq_block_bytes_ex(bits, flags=0):
    return int(lib().tq_block_bytes_ex(bits, flags))


def tq_encode_kv_ex(x, cb, signs, blocks, flags=0, block_stride_bytes=None, dst_index=None, block_offset=0,
                    stream=None):
    """tq_encode_kv with format flags (TQ_FMT_NORM_CORRECT, TQ_FMT_DENSE3); an
    8-bit codebook selects turboq8."""
    n, stride = _nvec_rows(x)
    bs = block_stride_bytes or tq_block_bytes_ex(cb.bits, flags)
    base = ctypes.c_void_p(blocks.data_ptr() + block_offset)
    _check(lib().tq_encode_kv_ex(_ptr(x), _dtype(x), n, stride, ctypes.byref(cb), signs, base, bs, _ptr(dst_index),
                                 flags, _stream(stream)), "tq_encode_kv_ex")


def tq_decode_kv_ex(blocks, n_vec, cb, signs, out, flags=0, block_stride_bytes=None, block_offset=0, stream=None):
    bs = block_stride_bytes or tq_block_bytes_ex(cb.bits, flags)
    n, stride = _nvec_rows(out)
    base = ctypes.c_void_p(blocks.data_ptr() + block_offset)
    _check(lib().tq_decode_kv_ex(base, bs, n_vec, ctypes.byref(cb), signs, _ptr(out), _dtype(out), stride, flags,
                                 _stream(stream)), "tq_decode_kv_ex")


def tq_attn_prefill_paged(q, k_pool, kcb, v_pool, vcb, block_table, page_tokens, out, T, scale, signs,
                          seq_lens=None, stream=None):
    """Causal attention over a paged cache: q [B, M, Hq, 128]; k_pool / v_pool
    uint8 [pages, Hkv, page_tokens, bytes]; block_table int32 [B, max_pages]."""
    B, M, Hq, _ = q.shape
    Hkv = k_pool.shape[1]
    _check(lib().tq_attn_prefill_paged(_ptr(q), _dtype(q), _ptr(k_pool), ctypes.byref(kcb), _ptr(v_pool),
                                       ctypes.byref(vcb), _ptr(block_table), block_table.shape[1], page_tokens,
                                       _ptr(seq_lens), B, M, Hq, Hkv, T, ctypes.c_float(scale), signs, _ptr(out),
                                       _stream(stream)), "tq_attn_prefill_paged")
    return out


def tq_attn_decode_paged(q, k_pool, kcb, v_pool, vcb, block_table, page_tokens, out, T, scale, signs,
                         seq_lens=None, workspace=None, stream=None):
    """Decode attention over a paged cache: q [B, Hq, 128], out [B, Hq, 128];
    with a workspace (uint8 device tensor) the split-K decode kernels run."""
    B, Hq, _ = q.shape
    Hkv = k_pool.shape[1]
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().tq_attn_decode_paged(_ptr(q), _dtype(q), _ptr(k_pool), ctypes.byref(kcb), _ptr(v_pool),
                                      ctypes.byref(vcb), _ptr(block_table), block_table.shape[1], page_tokens,
                                      _ptr(seq_lens), B, Hq, Hkv, T, ctypes.c_float(scale), signs, _ptr(out),
                                      _ptr(workspace), nbytes, _stream(stream)), "tq_attn_decode_paged")
    return out


# ---- head dims 64 / 96 / 128 / 160 (the rotation R is a device float32 [d, d] orthogonal matrix)

def tq_block_bytes_d(head_dim, bits):
    return int(lib().tq_block_bytes_d(head_dim, bits))


def tq_rotation_hadamard(head_dim, signs):
    """R = H D / sqrt(head_dim) (head_dim 64 or 128) as a CPU float32 tensor [d, d]."""
    R = torch.empty((head_dim, head_dim), dtype=torch.float32)
    _check(lib().tq_rotation_hadamard(head_dim, signs, ctypes.c_void_p(R.data_ptr())), "tq_rotation_hadamard")
    return R


def tq_encode_kv_d(x, cb, R, blocks, stream=None):
    """Encode contiguous rows x [n, d] into blocks [n, tq_block_bytes_d(d, bits)]."""
    d = x.shape[-1]
    n = x.numel() // d if d else 0
    _check(lib().tq_encode_kv_d(_ptr(x), _dtype(x), n, d, ctypes.byref(cb), _ptr(R), _ptr(blocks), _stream(stream)),
           "tq_encode_kv_d")
    return blocks


def tq_decode_kv_d(blocks, n_vec, cb, R, out, stream=None):
    """Decode n_vec blocks into contiguous rows out [n_vec, d]."""
    _check(lib().tq_decode_kv_d(_ptr(blocks), n_vec, out.shape[-1], ctypes.byref(cb), _ptr(R), _ptr(out),
                                _dtype(out), _stream(stream)), "tq_decode_kv_d")
    return out


def tq_attn_workspace_bytes_d(B, Hq, Hkv, T_cap, head_dim):
    return int(lib().tq_attn_workspace_bytes_d(B, Hq, Hkv, T_cap, head_dim))


def tq_attn_decode_d(q, k_blocks, kcb, v_blocks, vcb, R, out, workspace, T, scale, seq_lens=None, stream=None):
    """Decode attention at head dim d = q.shape[-1]: q [B, Hq, d]; k/v blocks
    [B, Hkv, T_cap, bytes]; out float32 [B, Hq, d]."""
    B, Hq, d = q.shape
    Hkv, T_cap = k_blocks.shape[1], k_blocks.shape[2]
    _check(lib().tq_attn_decode_d(_ptr(q), _dtype(q), _ptr(k_blocks), ctypes.byref(kcb), _ptr(v_blocks),
                                  ctypes.byref(vcb), _ptr(seq_lens), B, Hq, Hkv, T_cap, T, d, ctypes.c_float(scale),
                                  _ptr(R), _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream)), "tq_attn_decode_d")
    return out


# ---- rotary positions, quantise-on-insert of new tokens, eviction by attention weight

TQ_ROPE_HALF, TQ_ROPE_ADJACENT = 0, 1


class _On:
    """Makes the device of a call's tensors current while it runs."""

    def __init__(self, dev):
        self.guard = None if dev == torch.cuda.current_device() else torch.cuda.device(dev)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _on(what, *tensors):
    """The one CUDA device of the tensors (None skipped), made current."""
    dev = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d < 0:
                raise ValueError("%s: CUDA tensors expected" % what)
            if d != dev:
                if dev >= 0:
                    raise ValueError("%s: tensors on different devices" % what)
                dev = d
    return _On(dev)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def tq_rope_load(rot_dim=128, base=10000.0, style=TQ_ROPE_HALF, sections=None, interleaved=False, head_dim=128):
    """Rotary positions; ``sections``: pairs of each axis (default: one axis)."""
    sections = [rot_dim // 2] if sections is None else [int(n) for n in sections]
    r = tq_rope()
    _check(lib().tq_rope_load(head_dim, rot_dim, float(base), style, len(sections),
                              (ctypes.c_int * max(1, len(sections)))(*sections), 1 if interleaved else 0,
                              ctypes.byref(r)), "tq_rope_load")
    return r


def tq_rope_set_freqs(rope, freqs):
    """Replace the frequencies (radians per position) of the rope's pairs."""
    freqs = [float(f) for f in freqs]
    _need(len(freqs) == rope.rot_dim // 2, "tq_rope_set_freqs: one frequency per pair expected")
    _check(lib().tq_rope_set_freqs(ctypes.byref(rope), (ctypes.c_double * len(freqs))(*freqs)), "tq_rope_set_freqs")
    return rope


def _heads(x, what):
    """(tokens, heads, token stride, head stride) of rows [n, heads, 128]."""
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or shape[2] != 128 or stride[2] != 1:
        raise ValueError("%s: [tokens, heads, 128] expected" % what)
    return shape[0], shape[1], stride[0], stride[1]


def _axis_stride(pos, rope, n, what):
    """Axis stride of positions [n] or [axes, n]."""
    shape, stride = tuple(pos.shape), pos.stride()
    axes = rope.axes
    if pos.dtype != torch.int64 or not (shape == (axes, n) or (axes == 1 and shape == (n,))):
        raise ValueError("%s: int64 positions [axes, tokens] expected" % what)
    if n > 1 and stride[-1] != 1:
        raise ValueError("%s: positions of an axis must be contiguous" % what)
    return stride[0] if len(shape) == 2 else 0


def tq_rope_apply(x, pos, rope, out, stream=None):
    """Rotate heads x [n, heads, 128] into out (same shape and dtype; out may
    be x).  pos int64 [axes, n] (or [n] for one axis)."""
    n, heads, xt, xh = _heads(x, "tq_rope_apply")
    m, oheads, ot, oh = _heads(out, "tq_rope_apply")
    if m != n or oheads != heads or out.dtype != x.dtype:
        raise ValueError("tq_rope_apply: out must have the shape and dtype of x")
    pa = _axis_stride(pos, rope, n, "tq_rope_apply")
    with _on("tq_rope_apply", x, pos, out):
        _check(lib().tq_rope_apply(x.data_ptr(), _dtype(x), n, heads, xt, xh, pos.data_ptr(), pa, rope, out.data_ptr(),
                                   ot, oh, _stream(stream)), "tq_rope_apply")
    return out


def tq_insert_kv(k, v, pos, rope, kcb, vcb, signs, k_blocks, v_blocks, dst, dst_head_stride, stream=None):
    """Rotate keys k [n, Hkv, 128] (rope None: as they are), quantise keys and
    values v [n, Hkv, 128] and write them into the caches (uint8, last dim the
    block): the block of head h of token n is number dst[n] + h *
    dst_head_stride; tokens of negative dst are skipped.  k with k_blocks, or v
    with v_blocks, may be None."""
    what = "tq_insert_kv"
    x = k if k is not None else v
    _need(x is not None, "tq_insert_kv: no rows")
    n, heads, st, sh = _heads(x, what)
    if dst.dtype != torch.int64 or dst.shape != (n,) or not dst.is_contiguous():
        raise ValueError("tq_insert_kv: dst int64 [tokens] expected")
    strides, blocks = [], None
    for rows, cache, cb in ((k, k_blocks, kcb), (v, v_blocks, vcb)):
        if rows is None or cache is None or cb is None:
            if rows is not None or cache is not None:
                raise ValueError("tq_insert_kv: rows, their blocks and their codebook come together")
            strides += (0, 0)
            continue
        if rows is not x:
            m, hh, st, sh = _heads(rows, what)
            if m != n or hh != heads or rows.dtype != x.dtype:
                raise ValueError("tq_insert_kv: k and v of one shape and dtype expected")
        size = 2 + 16 * cb.bits
        if cache.dtype != torch.uint8 or not cache.is_contiguous() or cache.dim() == 0 or cache.shape[-1] != size:
            raise ValueError("tq_insert_kv: contiguous uint8 blocks of %d bytes expected" % size)
        count = cache.numel() // size
        if blocks is not None and count != blocks:
            raise ValueError("tq_insert_kv: caches of different sizes")
        blocks = count
        strides += (st, sh)
    turn = rope is not None and k is not None
    pa = _axis_stride(pos, rope, n, what) if turn else 0
    with _on(what, k, v, pos if turn else None, k_blocks, v_blocks, dst):
        _check(lib().tq_insert_kv(_ptr(k), strides[0], strides[1], _ptr(v), strides[2], strides[3], _dtype(x), n, heads,
                                  pos.data_ptr() if turn else None, pa, rope if turn else None, kcb, vcb, signs,
                                  _ptr(k_blocks), _ptr(v_blocks), blocks, dst.data_ptr(), dst_head_stride,
                                  _stream(stream)), what)


def tq_attn_weights_workspace_bytes(B, Hq, Hkv, T):
    """Workspace bytes of tq_attn_decode_weights on the current device: make the tensors' device current first where
    devices are not alike (a workspace too small for its device is refused)."""
    return int(lib().tq_attn_weights_workspace_bytes(B, Hq, Hkv, T))


def _pages(block_table, B, what):
    """Entries of a sequence in a block table int32 [B, max_pages] (0 without one)."""
    if block_table is None:
        return 0
    shape = block_table.shape
    if block_table.dtype != torch.int32 or len(shape) != 2 or shape[0] != B or not block_table.is_contiguous():
        raise ValueError("%s: block_table int32 [B, max_pages] expected" % what)
    return shape[1]


def _row_of(w, B, Hkv, T, what):
    """Row stride of accumulators [B, Hkv, >= T]."""
    if w.dtype == torch.float32 and w.dim() == 3:
        (b, h, n), (sb, sh, st) = w.shape, w.stride()
        if b == B and h == Hkv and n >= T and st == 1:
            if h == 1:   # (strides of size-1 dims can be anything)
                return sb if b > 1 else n
            if b == 1 or sb == h * sh:
                return sh
    raise ValueError("%s: weights float32 [B, Hkv, >= T] expected" % what)


def _lens(t, B, what):
    if t.dtype != torch.int32 or t.shape != (B,) or not t.is_contiguous():
        raise ValueError("%s: lengths int32 [B] expected" % what)


def _cache(t, size, first, what):
    """Shape of caches [B or pages, Hkv, tokens, bytes]; size and first checked unless None."""
    if t.dtype == torch.uint8 and t.dim() == 4 and t.is_contiguous():
        shape = tuple(t.shape)
        if (first is None or shape[0] == first) and (size is None or shape[3] == size):
            return shape
    raise ValueError("%s: contiguous packed blocks expected" % what)


def tq_attn_decode_weights(q, k_blocks, kcb, v_blocks, vcb, weights, out, workspace, T, scale, signs, seq_lens=None,
                           block_table=None, decay=1.0, stream=None):
    """Decode attention that adds each cached token's attention weight to
    weights float32 [B, Hkv, >= T].  q [B, Hq, 128]; caches [B, Hkv, T_cap,
    bytes], or with a block_table int32 [B, max_pages] pools [pages, Hkv,
    page, bytes]; out [B, Hq, 128] float32, bfloat16 or float16."""
    what = "tq_attn_decode_weights"
    shape = q.shape
    if len(shape) != 3 or shape[2] != 128 or not q.is_contiguous():
        raise ValueError("%s: contiguous q [B, Hq, 128] expected" % what)
    B, Hq = shape[0], shape[1]
    first = B if block_table is None else None
    ks = _cache(k_blocks, 2 + 16 * kcb.bits, first, what)
    vs = _cache(v_blocks, 2 + 16 * vcb.bits, first, what)
    Hkv, unit = ks[1], ks[2]
    if ks[:3] != vs[:3]:
        raise ValueError("%s: caches of one shape expected" % what)
    if out.shape != shape or not out.is_contiguous():
        raise ValueError("%s: contiguous out of q's shape expected" % what)
    if seq_lens is not None:
        _lens(seq_lens, B, what)
    stride = _row_of(weights, B, Hkv, T, what)
    pages = _pages(block_table, B, what)
    with _on(what, q, k_blocks, v_blocks, weights, out, workspace, seq_lens, block_table):
        _check(lib().tq_attn_decode_weights(q.data_ptr(), _dtype(q), k_blocks.data_ptr(), kcb, v_blocks.data_ptr(), vcb,
                                            _ptr(block_table), pages, unit, _ptr(seq_lens), B, Hq, Hkv, unit, T, scale,
                                            signs, weights.data_ptr(), stride, decay, out.data_ptr(), _dtype(out),
                                            workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                            _stream(stream)), what)
    return out


def _kept(kept, new_lens, what):
    shape = kept.shape
    if kept.dtype != torch.int32 or len(shape) != 3 or not kept.is_contiguous():
        raise ValueError("%s: kept int32 [B, Hkv, keep] expected" % what)
    if new_lens is None:
        raise ValueError("%s: new_lens expected" % what)
    _lens(new_lens, shape[0], what)
    return shape


def tq_evict_select(weights, kept, new_lens, T, first, last, seq_lens=None, stream=None):
    """The tokens that stay: kept int32 [B, Hkv, keep] (ascending, -1 past the
    last), new_lens int32 [B]."""
    what = "tq_evict_select"
    B, Hkv, keep = _kept(kept, new_lens, what)
    if seq_lens is not None:
        _lens(seq_lens, B, what)
    stride = _row_of(weights, B, Hkv, T, what)
    with _on(what, weights, kept, new_lens, seq_lens):
        _check(lib().tq_evict_select(weights.data_ptr(), stride, _ptr(seq_lens), B, Hkv, T, keep, first, last,
                                     kept.data_ptr(), new_lens.data_ptr(), _stream(stream)), what)
    return kept


def tq_evict_compact(k_blocks, v_blocks, kept, new_lens, T, weights=None, block_table=None, stream=None):
    """Move the kept tokens together in place: caches (and pools) as for
    tq_attn_decode_weights, of any block format; v_blocks may be None."""
    what = "tq_evict_compact"
    B, Hkv, keep = _kept(kept, new_lens, what)
    pages = _pages(block_table, B, what)
    first = B if block_table is None else None
    ks = _cache(k_blocks, None, first, what)
    vbytes = 0
    if v_blocks is not None:
        vs = _cache(v_blocks, None, first, what)
        if vs[:3] != ks[:3]:
            raise ValueError("%s: caches of one shape expected" % what)
        vbytes = vs[3]
    if ks[1] != Hkv:
        raise ValueError("%s: caches of kept's heads expected" % what)
    unit = ks[2]
    stride = 0 if weights is None else _row_of(weights, B, Hkv, T, what)
    with _on(what, k_blocks, v_blocks, kept, new_lens, weights, block_table):
        _check(lib().tq_evict_compact(k_blocks.data_ptr(), ks[3], _ptr(v_blocks), vbytes, _ptr(weights), stride,
                                      kept.data_ptr(), keep, new_lens.data_ptr(), _ptr(block_table), pages, unit, ks[0],
                                      B, Hkv, unit, T, _stream(stream)), what)
