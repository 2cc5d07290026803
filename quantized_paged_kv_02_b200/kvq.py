"""Python binding of the kvq C ABI (include/kvq.h): argument marshalling only.

Every call goes through ctypes into libkvq.so; no step of the cache or of attention runs
in Python.  Device memory comes from torch and work is enqueued on torch's current
stream (or the stream given).  If the library is missing, importing this module fails.

The functions keep the C names (kvq_write, kvq_decode_attention, kvq_dequant, ...).
``PagedKVCache`` is a convenience holder: it asks the library for the pool sizes,
allocates them with torch and fills a ``CacheDesc``.
"""

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvq.so")

DTYPE = {"bf16": 0, "fp16": 1, "fp32": 2, "int8": 3, "fp8": 4, "int4": 5, "int2": 6}
SCALE = {"none": 0, "per_token_head": 1, "per_head": 2, "per_tensor": 3, "kivi": 4,
         "per_channel": 5, "int4_per_token": 6, "kivi_float_zero": 7}
STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_UNSUPPORTED", 3: "KVQ_ERR_CUDA",
          4: "KVQ_ERR_DEVICE_FAULT"}
FAULT_BITS = {"slot": 1, "block": 2, "context": 4, "seq": 8, "int4_run": 16, "timeout": 32,
              "tree": 64}
ROPE_LAYOUT = {"half": 0, "interleaved": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "wavelength": 3, "yarn": 4}
EXPORTS = ("kvq_status_string", "kvq_version", "kvq_cache_layout", "kvq_write",
           "kvq_decode_workspace_size", "kvq_decode_attention", "kvq_dequant",
           "kvq_calibrate_fp8_scales", "kvq_read_device_fault", "kvq_decode_attention_noalloc",
           "kvq_append_decode_attention", "kvq_calibrate_channel_scales", "kvq_flush_ring",
           "kvq_prefill_attention", "kvq_decode_plan", "kvq_calibrate_head_scales",
           "kvq_rope_frequencies", "kvq_rope", "kvq_rope_write", "kvq_gather",
           "kvq_tree_workspace_size", "kvq_tree_attention", "kvq_tree_commit")


class CacheDesc(ctypes.Structure):
    _fields_ = [("cache_dtype", ctypes.c_int32), ("act_dtype", ctypes.c_int32),
                ("scale_mode", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("residual_len", ctypes.c_int32), ("residual_cap", ctypes.c_int32),
                ("max_seqs", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("pages", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("fault", ctypes.c_void_p)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("original_context", ctypes.c_int32), ("theta", ctypes.c_double),
                ("factor", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("attention_factor", ctypes.c_double)]


class KVQError(RuntimeError):
    def __init__(self, status, what):
        super().__init__("%s failed: %s" % (what, STATUS.get(status, status)))
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError("kvq CUDA library not built (%s missing); run "
                          "`python -m quantized_paged_kv_02_b200.build`" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I, Z, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    D, R, L = ctypes.POINTER(CacheDesc), ctypes.POINTER(RopeDesc), ctypes.c_int64
    sig = {
        "kvq_status_string": (ctypes.c_char_p, [I]),
        "kvq_version": (I, []),
        "kvq_cache_layout": (I, [D, ctypes.POINTER(Z), ctypes.POINTER(Z), ctypes.POINTER(Z),
                                 ctypes.POINTER(Z)]),
        "kvq_write": (I, [D, P, P, I, P, P, P, P]),
        "kvq_decode_workspace_size": (I, [D, I, I, I, ctypes.POINTER(Z)]),
        "kvq_decode_plan": (I, [D, I, I, I, ctypes.POINTER(I), ctypes.POINTER(I), ctypes.POINTER(I)]),
        "kvq_decode_attention": (I, [D, P, I, I, P, I, P, P, I, F, P, ctypes.c_int32, P, Z, P]),
        "kvq_dequant": (I, [D, P, I, P, P]),
        "kvq_calibrate_fp8_scales": (I, [P, I, I, I, ctypes.c_int32, P, P]),
        "kvq_read_device_fault": (I, [D, ctypes.POINTER(ctypes.c_int32), I, P]),
        "kvq_decode_attention_noalloc": (I, [D, P, I, I, P, I, P, P, I, F, P, ctypes.c_int32, P]),
        "kvq_append_decode_attention": (I, [D, P, P, P, I, I, P, I, P, I, F, P, ctypes.c_int32, P,
                                            Z, P]),
        "kvq_calibrate_channel_scales": (I, [P, I, I, I, ctypes.c_int32, F, P, P]),
        "kvq_calibrate_head_scales": (I, [P, I, I, I, ctypes.c_int32, F, P, P]),
        "kvq_flush_ring": (I, [D, P, P, P, I, P]),
        "kvq_prefill_attention": (I, [D, P, I, I, I, P, I, P, I, P, I, F, P, ctypes.c_int32, P]),
        "kvq_rope_frequencies": (I, [R, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]),
        "kvq_rope": (I, [R, P, ctypes.c_int32, I, P, I, P, L, I, P, L, P, L, I, P, L, P]),
        "kvq_rope_write": (I, [D, R, P, P, I, P, L, I, P, L, P, L, P, L, P, P]),
        "kvq_gather": (I, [D, P, I, P, P, P]),
        "kvq_tree_workspace_size": (I, [D, I, I, I, I, ctypes.POINTER(Z)]),
        "kvq_tree_attention": (I, [D, P, I, I, I, P, I, P, I, P, I, P, I, F, P, ctypes.c_int32, P, Z, P]),
        "kvq_tree_commit": (I, [D, P, I, P, I, P, P, I, P, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(st, what):
    if st != 0:
        raise KVQError(st, what)


def _act(t):
    if t.dtype == torch.bfloat16:
        return "bf16"
    if t.dtype == torch.float16:
        return "fp16"
    raise TypeError("activations must be bfloat16 or float16, got %s" % t.dtype)


def _i32(t):
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise TypeError("index tensors must be contiguous int32")
    return t


# ----------------------------------------------------------------------------- C names
def kvq_status_string(status):
    return lib.kvq_status_string(status).decode()


def kvq_version():
    return lib.kvq_version()


def kvq_cache_layout(desc):
    """(record bytes, pages pool bytes, static scale bytes, residual bytes)."""
    sizes = [ctypes.c_size_t(0) for _ in range(4)]
    _check(lib.kvq_cache_layout(ctypes.byref(desc), *[ctypes.byref(s) for s in sizes]),
           "kvq_cache_layout")
    return tuple(s.value for s in sizes)


def kvq_write(desc, k_new, v_new, slot_mapping, seq_ids=None, positions=None, stream=None):
    _check(lib.kvq_write(ctypes.byref(desc), _ptr(k_new), _ptr(v_new), int(k_new.shape[0]),
                         _ptr(_i32(slot_mapping)), _ptr(_i32(seq_ids)), _ptr(_i32(positions)),
                         _stream(stream)), "kvq_write")


def kvq_decode_workspace_size(desc, batch, num_q_heads, max_context):
    n = ctypes.c_size_t(0)
    _check(lib.kvq_decode_workspace_size(ctypes.byref(desc), batch, num_q_heads, max_context,
                                         ctypes.byref(n)), "kvq_decode_workspace_size")
    return n.value


def kvq_decode_plan(desc, batch, num_q_heads, max_context):
    """(kernel, launches per call, splits or CTAs) of kvq_decode_attention for this shape."""
    k, n, s = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib.kvq_decode_plan(ctypes.byref(desc), batch, num_q_heads, max_context,
                               ctypes.byref(k), ctypes.byref(n), ctypes.byref(s)), "kvq_decode_plan")
    return k.value, n.value, s.value


def kvq_decode_attention(desc, q, block_tables, context_lens, max_context, out, workspace=None,
                         seq_ids=None, softmax_scale=0.0, stream=None):
    B, Hq, _ = q.shape
    out_dt = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}[out.dtype]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.kvq_decode_attention(
        ctypes.byref(desc), _ptr(q), B, Hq, _ptr(_i32(block_tables)), int(block_tables.shape[1]),
        _ptr(_i32(context_lens)), _ptr(_i32(seq_ids)), int(max_context), float(softmax_scale),
        _ptr(out), DTYPE[out_dt], _ptr(workspace), ws_bytes, _stream(stream)),
        "kvq_decode_attention")
    return out


def kvq_append_decode_attention(desc, k_new, v_new, q, block_tables, context_lens, max_context,
                                out, workspace=None, softmax_scale=0.0, stream=None):
    """Store each sequence's new K/V row at position context_lens[b] - 1, then decode:
    kvq_write followed by kvq_decode_attention in one launch (dense caches)."""
    B, Hq, _ = q.shape
    out_dt = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}[out.dtype]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.kvq_append_decode_attention(
        ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(q), B, Hq, _ptr(_i32(block_tables)),
        int(block_tables.shape[1]), _ptr(_i32(context_lens)), int(max_context),
        float(softmax_scale), _ptr(out), DTYPE[out_dt], _ptr(workspace), ws_bytes,
        _stream(stream)), "kvq_append_decode_attention")
    return out


def kvq_decode_attention_noalloc(desc, q, block_tables, context_lens, max_context, out,
                                 seq_ids=None, softmax_scale=0.0, stream=None):
    """kvq_decode_attention with the library's own fixed device scratch instead of a
    caller workspace (for callers that cannot allocate device memory when they decode)."""
    B, Hq, _ = q.shape
    out_dt = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}[out.dtype]
    _check(lib.kvq_decode_attention_noalloc(
        ctypes.byref(desc), _ptr(q), B, Hq, _ptr(_i32(block_tables)), int(block_tables.shape[1]),
        _ptr(_i32(context_lens)), _ptr(_i32(seq_ids)), int(max_context), float(softmax_scale),
        _ptr(out), DTYPE[out_dt], _stream(stream)), "kvq_decode_attention_noalloc")
    return out


def kvq_dequant(desc, block_ids, out, stream=None):
    _check(lib.kvq_dequant(ctypes.byref(desc), _ptr(_i32(block_ids)), int(block_ids.numel()),
                           _ptr(out), _stream(stream)), "kvq_dequant")
    return out


def kvq_calibrate_fp8_scales(x, scale_out, stream=None):
    T, H, D = x.shape
    _check(lib.kvq_calibrate_fp8_scales(_ptr(x), T, H, D, DTYPE[_act(x)], _ptr(scale_out),
                                        _stream(stream)), "kvq_calibrate_fp8_scales")
    return scale_out


def kvq_prefill_attention(desc, q, q_start, max_q_len, block_tables, context_lens, max_context,
                          out, softmax_scale=0.0, stream=None):
    """Causal attention of each sequence's chunk of new queries (rows q_start[b] ..
    q_start[b+1]-1 of q) over the cache."""
    Tq, Hq, _ = q.shape
    B = int(q_start.numel()) - 1
    out_dt = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}[out.dtype]
    _check(lib.kvq_prefill_attention(
        ctypes.byref(desc), _ptr(q), Tq, B, Hq, _ptr(_i32(q_start)), int(max_q_len),
        _ptr(_i32(block_tables)), int(block_tables.shape[1]), _ptr(_i32(context_lens)),
        int(max_context), float(softmax_scale), _ptr(out), DTYPE[out_dt], _stream(stream)),
        "kvq_prefill_attention")
    return out


def kvq_flush_ring(desc, seq_ids, positions, block_ids, stream=None):
    """INT4: quantize ring rows [positions[i], positions[i] + 64) of sequence seq_ids[i]
    into block block_ids[i] (all kv heads)."""
    n = int(seq_ids.numel())
    _check(lib.kvq_flush_ring(ctypes.byref(desc), _ptr(_i32(seq_ids)), _ptr(_i32(positions)),
                              _ptr(_i32(block_ids)), n, _stream(stream)), "kvq_flush_ring")


def kvq_calibrate_head_scales(x, qmax, scale_out, stream=None):
    """scale_out[h] = max over tokens and channels |x[t][h][:]| / qmax (127 INT8, 448 FP8)."""
    T, H, D = x.shape
    _check(lib.kvq_calibrate_head_scales(_ptr(x), T, H, D, DTYPE[_act(x)], float(qmax),
                                         _ptr(scale_out), _stream(stream)),
           "kvq_calibrate_head_scales")
    return scale_out


def kvq_calibrate_channel_scales(x, qmax, scale_out, stream=None):
    """scale_out[h][d] = max over tokens |x[t][h][d]| / qmax (127 INT8, 448 FP8)."""
    T, H, D = x.shape
    _check(lib.kvq_calibrate_channel_scales(_ptr(x), T, H, D, DTYPE[_act(x)], float(qmax),
                                            _ptr(scale_out), _stream(stream)),
           "kvq_calibrate_channel_scales")
    return scale_out


def kvq_read_device_fault(desc, reset=True, stream=None):
    out = (ctypes.c_int32 * 2)()
    st = lib.kvq_read_device_fault(ctypes.byref(desc), out, 1 if reset else 0, _stream(stream))
    if st not in (0, 4):
        _check(st, "kvq_read_device_fault")
    return int(out[0]), int(out[1])


# The wrappers below run once per layer and step beside kernels of a few microseconds, so they
# look at each tensor once and hand the addresses over as plain integers.
def _here():
    """The current device, which the call runs on and every tensor has to be on."""
    return torch.cuda.current_device()


def _raw_stream(stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream.cuda_stream


def _at(t, dev, what):
    """Address of a tensor on device dev (a host address, or another device's, would fault)."""
    if t.get_device() != dev:
        raise ValueError("%s is on %s, not on the current device" % (what, t.device))
    return t.data_ptr()


def _like(x, stream, shape=None, dtype=None):
    """A dense tensor like x, allocated for the stream that writes it: memory of the current stream could
    still be in use there, and a released workspace of it would be handed out again too early."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return _like(x, None, shape, dtype)
    if shape is None:
        return torch.empty_like(x) if dtype is None else torch.empty_like(x, dtype=dtype)
    return x.new_empty(shape, dtype=dtype)


def _freqs(t, rope, dev):
    """Address of a rope's frequencies."""
    if t.dtype != torch.float64 or not t.is_contiguous() or 2 * t.numel() < rope.rot_dim:
        raise ValueError("freqs must be contiguous float64 and have rot_dim / 2 entries")
    return _at(t, dev, "freqs")


def _rows(t, what):
    """(tokens, heads, dim, token stride) of a [T][heads][dim] tensor whose rows are dense (a view into
    fused projection rows is fine)."""
    try:
        T, H, D = t.shape
    except ValueError:
        raise ValueError("%s must be [tokens, heads, dim], got %s" % (what, tuple(t.shape))) from None
    a, b, c = t.stride()
    if c != 1 or (H > 1 and b != D):
        raise ValueError("%s: the heads of a token must be contiguous" % what)
    # (the stride of a single token says nothing)
    return T, H, D, a if T > 1 else H * D


def _index(t, n, dev, what):
    """Address of an index tensor of n entries (contiguous int32)."""
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise TypeError("%s must be contiguous int32" % what)
    if t.numel() != n:
        raise ValueError("%s must have %d entries, got %d" % (what, n, t.numel()))
    return _at(t, dev, what)


_ACT_CODE = {torch.bfloat16: 0, torch.float16: 1}
_OUT_CODE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def kvq_rope_frequencies(rope):
    """(frequencies in radians per position, factor of cosine and sine) of a RopeDesc."""
    f = (ctypes.c_double * max(rope.rot_dim // 2, 1))()
    m = ctypes.c_double(0.0)
    _check(lib.kvq_rope_frequencies(ctypes.byref(rope), f, ctypes.byref(m)), "kvq_rope_frequencies")
    return list(f)[:rope.rot_dim // 2], m.value


def kvq_rope(rope, freqs, positions, q=None, k=None, q_out=None, k_out=None, stream=None):
    """Rotate q [T, Hq, D] and / or k [T, H, D] (token strides as they are) into q_out / k_out
    (given, or allocated dense); an output may be its input."""
    if q is None and k is None:
        raise ValueError("neither q nor k to rotate")
    act = q.dtype if q is not None else k.dtype
    if act not in _ACT_CODE:
        raise TypeError("activations must be bfloat16 or float16, got %s" % act)
    dev = _here()
    T = D = None
    args = []
    for x, out, what in ((q, q_out, "q"), (k, k_out, "k")):
        if x is None:
            args += (None, 0, 0, None, 0)
            continue
        Tx, H, Dx, xs = _rows(x, what)
        if T is None:
            T, D = Tx, Dx
        if Tx != T or Dx != D:
            raise ValueError("q and k must have the same tokens and head_dim")
        if out is None:
            out = torch.empty_like(x) if stream is None else _like(x, stream)
            os = H * D
        else:
            shape = _rows(out, what + "_out")
            if shape[:3] != (T, H, D):
                raise ValueError("%s_out must have the shape of %s" % (what, what))
            os = shape[3]
        if x.dtype != act or out.dtype != act:
            raise TypeError("q, k and their outputs must have one type")
        args += (_at(x, dev, what), xs, H, _at(out, dev, what), os)
        if what == "q":
            q_out = out
        else:
            k_out = out
    st = lib.kvq_rope(ctypes.byref(rope), _freqs(freqs, rope, dev), _ACT_CODE[act], D, _index(positions, T, dev, "positions"), T,
                      *args, _raw_stream(stream, dev))
    if st:
        _check(st, "kvq_rope")
    return (q_out if q is not None else None), (k_out if k is not None else None)


def kvq_rope_write(desc, rope, freqs, positions, q, k_new, v_new, slot_mapping, q_out=None, stream=None):
    """kvq_rope of q and k_new, then kvq_write of the rotated keys and of v_new, in one launch.
    Returns q_out (None without q)."""
    T, H, D, ks = _rows(k_new, "k_new")
    Tv, Hv, Dv, vs = _rows(v_new, "v_new")
    act = k_new.dtype
    if _ACT_CODE.get(act) != desc.act_dtype or v_new.dtype != act:
        raise TypeError("k_new and v_new must have the cache's activation type")
    if Tv != T or H != desc.num_kv_heads or Hv != H or D != desc.head_dim or Dv != D:
        raise ValueError("k_new and v_new must be [tokens, %d, %d]" % (desc.num_kv_heads, desc.head_dim))
    dev = _here()
    qp, qs, hq, qop, qos = None, 0, 0, None, 0
    if q is not None:
        Tq, hq, Dq, qs = _rows(q, "q")
        if Tq != T or Dq != D:
            raise ValueError("q must have the tokens and head_dim of k_new")
        if q_out is None:
            q_out = torch.empty_like(q) if stream is None else _like(q, stream)
            qos = hq * D
        else:
            To, ho, Do, qos = _rows(q_out, "q_out")
            if (To, ho, Do) != (T, hq, D):
                raise ValueError("q_out must have the shape of q")
        if q.dtype != act or q_out.dtype != act:
            raise TypeError("q and q_out must have the cache's activation type")
        qp, qop = _at(q, dev, "q"), _at(q_out, dev, "q_out")
    st = lib.kvq_rope_write(ctypes.byref(desc), ctypes.byref(rope), _freqs(freqs, rope, dev),
                            _index(positions, T, dev, "positions"), T, qp, qs, hq, qop, qos, _at(k_new, dev, "k_new"), ks,
                            _at(v_new, dev, "v_new"), vs, _index(slot_mapping, T, dev, "slot_mapping"),
                            _raw_stream(stream, dev))
    if st:
        _check(st, "kvq_rope_write")
    return q_out


def kvq_gather(desc, slots, k_out, v_out, stream=None):
    """K and V rows of the listed cache slots, dequantized to the activation type."""
    n = slots.numel()
    for t, what in ((k_out, "k_out"), (v_out, "v_out")):
        if t.shape != (n, desc.num_kv_heads, desc.head_dim) or not t.is_contiguous():
            raise ValueError("%s must be contiguous [%d, %d, %d]" % (what, n, desc.num_kv_heads, desc.head_dim))
        if _ACT_CODE.get(t.dtype) != desc.act_dtype:
            raise TypeError("%s must have the cache's activation type" % what)
    dev = _here()
    st = lib.kvq_gather(ctypes.byref(desc), _index(slots, n, dev, "slots"), n, _at(k_out, dev, "k_out"), _at(v_out, dev, "v_out"),
                        _raw_stream(stream, dev))
    if st:
        _check(st, "kvq_gather")
    return k_out, v_out


def kvq_tree_workspace_size(desc, batch, num_q_heads, max_tree, max_context):
    n = ctypes.c_size_t(0)
    _check(lib.kvq_tree_workspace_size(ctypes.byref(desc), batch, num_q_heads, max_tree, max_context,
                                       ctypes.byref(n)), "kvq_tree_workspace_size")
    return n.value


def kvq_tree_attention(desc, q, q_start, max_tree, tree_mask, block_tables, context_lens, max_context, out,
                       workspace=None, softmax_scale=0.0, stream=None):
    """Attention of each sequence's drafted tokens (rows q_start[b] .. q_start[b+1]-1 of q, the newest
    cached positions) over the cached prefix and the drafted tokens its mask row names.  tree_mask:
    int32 [tokens, words], the bits of the C ABI's uint32."""
    T, Hq, D, _ = _rows(q, "q")
    if D != desc.head_dim or _ACT_CODE.get(q.dtype) != desc.act_dtype or not q.is_contiguous():
        raise ValueError("q must be contiguous [tokens, heads, %d] of the cache's activation type" % desc.head_dim)
    if out.shape != (T, Hq, D) or not out.is_contiguous():
        raise ValueError("out must be contiguous and have the shape of q")
    if out.dtype not in _OUT_CODE:
        raise TypeError("out must be bfloat16, float16 or float32, got %s" % out.dtype)
    B = context_lens.numel()
    if tree_mask.dim() != 2 or block_tables.dim() != 2:
        raise ValueError("tree_mask must be [tokens, words] and block_tables [batch, blocks]")
    words, blocks = tree_mask.shape[1], block_tables.shape[1]
    dev = _here()
    ws, ws_bytes = None, 0
    if workspace is not None:
        ws, ws_bytes = _at(workspace, dev, "workspace"), workspace.numel() * workspace.element_size()
    st = lib.kvq_tree_attention(
        ctypes.byref(desc), _at(q, dev, "q"), T, B, Hq, _index(q_start, B + 1, dev, "q_start"), max_tree,
        _index(tree_mask, T * words, dev, "tree_mask"), words, _index(block_tables, B * blocks, dev, "block_tables"), blocks,
        _index(context_lens, B, dev, "context_lens"), max_context, softmax_scale, _at(out, dev, "out"), _OUT_CODE[out.dtype],
        ws, ws_bytes, _raw_stream(stream, dev))
    if st:
        _check(st, "kvq_tree_attention")
    return out


def kvq_tree_commit(desc, path, accepted, q_start, block_tables, context_lens, new_lens=None, stream=None):
    """Move the cache rows of each sequence's accepted path (drafted indexes path[b, :accepted[b]]) to the
    first drafted positions; new_lens receives the new context lengths."""
    B = accepted.numel()
    if path.dim() != 2 or block_tables.dim() != 2:
        raise ValueError("path must be [batch, accepted at most] and block_tables [batch, blocks]")
    most, blocks = path.shape[1], block_tables.shape[1]
    dev = _here()
    st = lib.kvq_tree_commit(
        ctypes.byref(desc), _index(path, B * most, dev, "path"), most, _index(accepted, B, dev, "accepted"), B,
        _index(q_start, B + 1, dev, "q_start"), _index(block_tables, B * blocks, dev, "block_tables"), blocks,
        _index(context_lens, B, dev, "context_lens"), None if new_lens is None else _index(new_lens, B, dev, "new_lens"),
        _raw_stream(stream, dev))
    if st:
        _check(st, "kvq_tree_commit")
    return new_lens


# ----------------------------------------------------------------------------- holder
class Rope:
    """A rotary embedding: its descriptor and its frequencies on the device.

    layout "half" or "interleaved"; scaling "none", "linear", "ntk", "wavelength" or "yarn" (include/kvq.h);
    freqs: frequencies of the caller's own (radians per position), instead of the descriptor's."""

    def __init__(self, head_dim, rot_dim=None, theta=10000.0, layout="half", scaling="none", factor=1.0,
                 original_context=0, low=1.0, high=4.0, attention_factor=0.0, freqs=None, device="cuda"):
        r = self.desc = RopeDesc()
        self.head_dim = head_dim
        r.layout, r.scaling = ROPE_LAYOUT[layout], ROPE_SCALING[scaling]
        r.rot_dim = head_dim if rot_dim is None else rot_dim
        r.original_context, r.theta, r.factor = original_context, theta, factor
        r.low, r.high, r.attention_factor = low, high, attention_factor
        own, self.attention_factor = kvq_rope_frequencies(r)
        f = torch.tensor(own, dtype=torch.float64) if freqs is None else freqs.to(torch.float64)
        if f.shape != (r.rot_dim // 2,):
            raise ValueError("freqs must have rot_dim / 2 entries")
        self.freqs = f.to(device).contiguous()

    def apply(self, positions, q=None, k=None, q_out=None, k_out=None, stream=None):
        """(rotated q, rotated k); None for one not given."""
        return kvq_rope(self.desc, self.freqs, positions, q, k, q_out, k_out, stream)


class PagedKVCache:
    """One layer's cache, allocated with torch in the layout of include/kvq.h: the page
    records pool, the static scale arrays (PER_HEAD / PER_TENSOR) and the INT4 ring."""

    def __init__(self, cache_dtype, act_dtype, scale_mode, num_blocks, block_size, num_kv_heads,
                 head_dim, device="cuda", group_size=64, residual_len=128, residual_cap=192,
                 max_seqs=0, static_k_scale=None, static_v_scale=None, fill=0x5A, fault=True,
                 pages=None):
        self.desc = CacheDesc()
        d = self.desc
        d.cache_dtype, d.act_dtype, d.scale_mode = DTYPE[cache_dtype], DTYPE[act_dtype], SCALE[scale_mode]
        d.num_blocks, d.block_size, d.num_kv_heads, d.head_dim = num_blocks, block_size, num_kv_heads, head_dim
        d.group_size, d.residual_len, d.residual_cap = group_size, residual_len, residual_cap
        d.max_seqs = max_seqs
        self.cache_dtype, self.act_dtype, self.scale_mode = cache_dtype, act_dtype, scale_mode
        self.num_blocks, self.block_size = num_blocks, block_size
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim
        self.device = torch.device(device)
        self.record, pages_b, ss_b, res_b = kvq_cache_layout(d)
        if pages is None:
            self.pages = torch.full((pages_b,), fill, dtype=torch.uint8, device=self.device)
        else:                                     # a pool the caller holds
            if pages.dtype != torch.uint8 or not pages.is_contiguous() or pages.numel() < pages_b:
                raise ValueError("pages must be a contiguous uint8 pool of at least %d bytes" % pages_b)
            self.pages, self.device = pages, pages.device
        self.k_scales = self.v_scales = self.residual = None
        if ss_b:
            n = ss_b // 4
            self.k_scales = torch.zeros(max(n, 4), dtype=torch.float32, device=self.device)
            self.v_scales = torch.zeros(max(n, 4), dtype=torch.float32, device=self.device)
            if static_k_scale is not None:
                self.k_scales[:n].copy_(static_k_scale.reshape(n).to(torch.float32))
            if static_v_scale is not None:
                self.v_scales[:n].copy_(static_v_scale.reshape(n).to(torch.float32))
        if res_b:
            self.residual = torch.full((res_b,), fill, dtype=torch.uint8, device=self.device)
        self.fault = torch.zeros(4, dtype=torch.int32, device=self.device) if fault else None
        d.pages = self.pages.data_ptr()
        d.k_scales = self.k_scales.data_ptr() if self.k_scales is not None else None
        d.v_scales = self.v_scales.data_ptr() if self.v_scales is not None else None
        d.residual = self.residual.data_ptr() if self.residual is not None else None
        d.fault = self.fault.data_ptr() if self.fault is not None else None
        self.sizes = (self.record, pages_b, ss_b, res_b)

    def records(self):
        """The pages pool as [NB][H][record] bytes."""
        return self.pages.view(self.num_blocks, self.num_kv_heads, self.record)

    def write(self, k_new, v_new, slot_mapping, seq_ids=None, positions=None, stream=None):
        kvq_write(self.desc, k_new, v_new, slot_mapping, seq_ids, positions, stream)

    def workspace_size(self, batch, num_q_heads, max_context):
        return kvq_decode_workspace_size(self.desc, batch, num_q_heads, max_context)

    def decode_plan(self, batch, num_q_heads, max_context):
        return kvq_decode_plan(self.desc, batch, num_q_heads, max_context)

    def decode(self, q, block_tables, context_lens, max_context, out=None, out_dtype=torch.float32,
               workspace=None, seq_ids=None, softmax_scale=0.0, stream=None):
        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
        if workspace is None:
            n = self.workspace_size(q.shape[0], q.shape[1], max_context)
            workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device) if n else None
        return kvq_decode_attention(self.desc, q, block_tables, context_lens, max_context, out,
                                    workspace, seq_ids, softmax_scale, stream)

    def append_decode(self, k_new, v_new, q, block_tables, context_lens, max_context, out=None,
                      out_dtype=torch.float32, workspace=None, softmax_scale=0.0, stream=None):
        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
        if workspace is None:
            n = self.workspace_size(q.shape[0], q.shape[1], max_context)
            workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device) if n else None
        return kvq_append_decode_attention(self.desc, k_new, v_new, q, block_tables, context_lens,
                                           max_context, out, workspace, softmax_scale, stream)

    def prefill(self, q, q_start, max_q_len, block_tables, context_lens, max_context, out=None,
                out_dtype=torch.float32, softmax_scale=0.0, stream=None):
        if out is None:
            out = torch.empty(q.shape, dtype=out_dtype, device=q.device)
        return kvq_prefill_attention(self.desc, q, q_start, max_q_len, block_tables, context_lens,
                                     max_context, out, softmax_scale, stream)

    def rope_write(self, rope, positions, q, k_new, v_new, slot_mapping, q_out=None, stream=None):
        """Rotate q and k_new, store the rotated keys and v_new; returns the rotated q."""
        _at(self.pages, _here(), "the cache")
        return kvq_rope_write(self.desc, rope.desc, rope.freqs, positions, q, k_new, v_new, slot_mapping, q_out,
                              stream)

    def gather(self, slots, k_out=None, v_out=None, stream=None):
        """(K, V) rows of the listed slots, [rows, H, D] of the activation type."""
        _at(self.pages, _here(), "the cache")
        shape = (slots.numel(), self.num_kv_heads, self.head_dim)
        dt = torch.bfloat16 if self.act_dtype == "bf16" else torch.float16
        if k_out is None:
            k_out = _like(self.pages, stream, shape, dt)
        if v_out is None:
            v_out = _like(self.pages, stream, shape, dt)
        return kvq_gather(self.desc, slots, k_out, v_out, stream)

    def tree_workspace_size(self, batch, num_q_heads, max_tree, max_context):
        return kvq_tree_workspace_size(self.desc, batch, num_q_heads, max_tree, max_context)

    def tree_attention(self, q, q_start, max_tree, tree_mask, block_tables, context_lens, max_context, out=None,
                       out_dtype=torch.float32, workspace=None, softmax_scale=0.0, stream=None):
        _at(self.pages, _here(), "the cache")
        if out is None:
            out = _like(q, stream, None, out_dtype)
        if workspace is None:
            n = self.tree_workspace_size(context_lens.numel(), q.shape[1], max_tree, max_context)
            workspace = _like(q, stream, (n,), torch.uint8) if n else None
        return kvq_tree_attention(self.desc, q, q_start, max_tree, tree_mask, block_tables, context_lens,
                                  max_context, out, workspace, softmax_scale, stream)

    def tree_commit(self, path, accepted, q_start, block_tables, context_lens, new_lens=None, stream=None):
        """Keep each sequence's accepted path; returns the new context lengths."""
        _at(self.pages, _here(), "the cache")
        if new_lens is None:
            new_lens = _like(context_lens, stream)
        return kvq_tree_commit(self.desc, path, accepted, q_start, block_tables, context_lens, new_lens, stream)

    def flush_ring(self, seq_ids, positions, block_ids, stream=None):
        kvq_flush_ring(self.desc, seq_ids, positions, block_ids, stream)

    def dequant(self, block_ids, stream=None):
        out = torch.empty((block_ids.numel(), 2, self.num_kv_heads, self.block_size, self.head_dim),
                          dtype=torch.float32, device=self.device)
        return kvq_dequant(self.desc, block_ids, out, stream)

    def read_fault(self, reset=True):
        return kvq_read_device_fault(self.desc, reset)
