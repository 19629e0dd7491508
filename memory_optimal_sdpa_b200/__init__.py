"""Python binding of libsdpa.so, the B200 exact-attention library (C ABI in include/sdpa.h).

Argument marshalling only: every step of attention runs in the library's CUDA
kernels.  PyTorch is used for device tensors and streams.  There is no CPU
fallback: if libsdpa.so is missing, importing this package fails.

    import memory_optimal_sdpa_b200 as sdpa
    O, LSE = sdpa.fwd(q, k, v, causal=True)                 # bf16, tcgen05 tensor cores
    O, LSE = sdpa.fwd_f32(q, k, v)                          # fp32 on CUDA cores
    O, LSE = sdpa.decode(q, k_cache, v_cache, kv_lens)      # one row per (batch, head)
    O, LSE = sdpa.decode_gqa(q, k_cache, v_cache, kv_lens)  # query heads sharing key/value heads
    dQ, dK, dV = sdpa.bwd(q, k, v, O, dO, LSE, causal=True) # gradients of fwd

The bounded decode cache (C ABI in include/sdpa_cache.h):

    cache = sdpa.kv4_cache(batch, heads, n_cap, d)          # keys and values in 4 bits
    sdpa.kv4_append(cache, k_new, v_new, kv_lens)           # quantise rows into it
    O, LSE = sdpa.decode_kv4(q, cache, kv_lens, acc=acc)    # attend; acc sums each key's weight
    O, LSE = sdpa.decode_acc(q, k_cache, v_cache, kv_lens, acc)  # the same over a bf16 cache
    sdpa.fwd_acc(q, k, LSE, acc, causal=True)               # the weights of a prompt
    keep, kv_lens = sdpa.kv4_evict(cache, acc, kv_lens, budget, recent=64)  # (evict: bf16) drop the others
    k, v = sdpa.kv4_load(cache, kv_lens)                    # the rows as bf16
"""
import collections
import ctypes
import functools
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsdpa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libsdpa.so is not built: run `python memory_optimal_sdpa_b200/build.py` "
                      "(nvcc, sm_100a).  There is no fallback implementation.")

lib = ctypes.CDLL(LIB_PATH)

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
lib.sdpa_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp]
lib.sdpa_fwd.restype = _i
lib.sdpa_fwd_window.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _i, _vp]
lib.sdpa_fwd_window.restype = _i
lib.sdpa_fwd_f32.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp]
lib.sdpa_fwd_f32.restype = _i
lib.sdpa_decode_workspace_size.argtypes = [_i, _i, _i, _i]
lib.sdpa_decode_workspace_size.restype = _sz
lib.sdpa_decode.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]
lib.sdpa_decode.restype = _i
lib.sdpa_decode_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _vp]
lib.sdpa_decode_noalloc.restype = _i
lib.sdpa_decode_gqa_workspace_size.argtypes = [_i, _i, _i, _i, _i]
lib.sdpa_decode_gqa_workspace_size.restype = _sz
lib.sdpa_decode_gqa.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _vp, _sz, _vp]
lib.sdpa_decode_gqa.restype = _i
lib.sdpa_bwd_workspace_size.argtypes = [_i, _i, _i]
lib.sdpa_bwd_workspace_size.restype = _sz
lib.sdpa_bwd.argtypes = [_vp] * 9 + [_i] * 6 + [_f, _i, _vp, _sz, _vp]
lib.sdpa_bwd.restype = _i
lib.sdpa_kv4_append.argtypes = [_vp] * 10 + [_i] * 5 + [_vp]
lib.sdpa_kv4_append.restype = _i
lib.sdpa_kv4_load.argtypes = [_vp] * 7 + [_i] * 5 + [_vp]
lib.sdpa_kv4_load.restype = _i
lib.sdpa_decode_kv4_workspace_size.argtypes = [_i] * 6
lib.sdpa_decode_kv4_workspace_size.restype = _sz
lib.sdpa_decode_kv4.argtypes = [_vp] * 10 + [_i] * 5 + [_f, _vp, _sz, _vp]
lib.sdpa_decode_kv4.restype = _i
lib.sdpa_decode_acc_workspace_size.argtypes = [_i] * 5
lib.sdpa_decode_acc_workspace_size.restype = _sz
lib.sdpa_decode_acc.argtypes = [_vp] * 8 + [_i] * 5 + [_f, _vp, _sz, _vp]
lib.sdpa_decode_acc.restype = _i
lib.sdpa_fwd_acc.argtypes = [_vp] * 5 + [_i] * 7 + [_f, _i, _vp]
lib.sdpa_fwd_acc.restype = _i
lib.sdpa_evict.argtypes = [_vp] * 9 + [_i] * 7 + [_vp]
lib.sdpa_evict.restype = _i
lib.sdpa_kv4_evict.argtypes = [_vp] * 13 + [_i] * 7 + [_vp]
lib.sdpa_kv4_evict.restype = _i
lib.sdpa_get_last_device_error.argtypes = [_vp]
lib.sdpa_get_last_device_error.restype = _i
lib.sdpa_status_string.argtypes = [_i]
lib.sdpa_status_string.restype = ctypes.c_char_p

SDPA_OK = 0
SDPA_ERR_INVALID_ARG = 1
SDPA_ERR_UNSUPPORTED = 2
SDPA_ERR_MISALIGNED = 3
SDPA_ERR_WORKSPACE = 4
SDPA_ERR_CUDA = 5
SDPA_ERR_DEVICE_TIMEOUT = 6
SDPA_ERR_DEVICE_BAD_LENGTH = 7
SDPA_ERR_DEVICE_CHECK = 8


class SdpaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s" % (where, status_string(status)))


def status_string(status):
    return lib.sdpa_status_string(status).decode()


def _check(status, where):
    if status != SDPA_OK:
        raise SdpaError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# ------------------------------------------------------------------------------ argument guards
# The C ABI sees raw pointers and sizes only, so it cannot tell a transposed view, a tensor of
# another dtype or a tensor on another device from a valid argument.  These guards reject such
# tensors before the call.  Order: type, dtype, shape, contiguity, then device (so everything
# but the device check can be exercised with host tensors).
def _tensor(t, name, dtype, shape):
    """t must be a torch tensor of `dtype` whose shape matches `shape` (None entries are free)."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor, got %s" % (name, type(t).__name__))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != len(shape) or any(want is not None and got != want for got, want in zip(t.shape, shape)):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape),
                                                           tuple("*" if x is None else x for x in shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (row-major); got strides %s -- pass .contiguous()"
                         % (name, tuple(t.stride())))
    return t


def _device(ref_name, ref, *others):
    """ref must be a CUDA tensor and every other (name, tensor) must live on the same device."""
    if ref.device.type != "cuda":
        raise ValueError("%s must be a CUDA tensor, got device %s" % (ref_name, ref.device))
    for name, t in others:
        if t is not None and t.device != ref.device:
            raise ValueError("%s is on %s but %s is on %s" % (name, t.device, ref_name, ref.device))
    return ref.device


def _stream(stream, device):
    import torch
    s = torch.cuda.current_stream(device) if stream is None else stream
    if s.device != device:
        raise ValueError("stream is on %s but the tensors are on %s" % (s.device, device))
    return ctypes.c_void_p(s.cuda_stream)


def _call(device, fn, *args):
    """Run a library call with `device` current (the C ABI works on the current device)."""
    import torch
    with torch.cuda.device(device):
        return fn(*args)


def _nbytes(t):
    return t.numel() * t.element_size()


def _prefill_args(q, k, v, o, lse, dtype, want_lse):
    """Shapes of a prefill call: q [B,H,n_q,d_k], k [B,H,n_kv,d_k], v [B,H,n_kv,d_v]."""
    import torch
    _tensor(q, "q", dtype, (None, None, None, None))
    B, H, n_q, d_k = q.shape
    _tensor(k, "k", dtype, (B, H, None, d_k))
    n_kv = k.shape[2]
    _tensor(v, "v", dtype, (B, H, n_kv, None))
    d_v = v.shape[3]
    if o is not None:
        _tensor(o, "o", dtype, (B, H, n_q, d_v))
    if lse is not None:
        _tensor(lse, "lse", torch.float32, (B, H, n_q))
    dev = _device("q", q, ("k", k), ("v", v), ("o", o), ("lse", lse))
    if o is None:
        o = torch.empty((B, H, n_q, d_v), dtype=dtype, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, H, n_q), dtype=torch.float32, device=dev)
    return B, H, n_q, n_kv, d_k, d_v, o, lse, dev


def fwd(q, k, v, causal=False, scale=None, o=None, lse=None, want_lse=True, stream=None):
    """bf16 prefill. q [B,H,n_q,d], k/v [B,H,n_kv,d] contiguous CUDA bf16; d in {64,128}."""
    import torch
    B, H, n_q, n_kv, d_k, d_v, o, lse, dev = _prefill_args(q, k, v, o, lse, torch.bfloat16, want_lse)
    scale = 1.0 / math.sqrt(d_k) if scale is None else scale
    _check(_call(dev, lib.sdpa_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, n_q, n_kv, d_k, d_v,
                 float(scale), int(bool(causal)), _stream(stream, dev)), "sdpa_fwd")
    return o, lse


def fwd_window(q, k, v, window_left, window_right, scale=None, o=None, lse=None, want_lse=True, stream=None):
    """bf16 prefill with a local window: row i (key position p = i + n_kv - n_q) sees keys
    p - window_left .. p + window_right; -1 leaves a side open."""
    import torch
    B, H, n_q, n_kv, d_k, d_v, o, lse, dev = _prefill_args(q, k, v, o, lse, torch.bfloat16, want_lse)
    scale = 1.0 / math.sqrt(d_k) if scale is None else scale
    _check(_call(dev, lib.sdpa_fwd_window, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, n_q, n_kv, d_k,
                 d_v, float(scale), int(window_left), int(window_right), _stream(stream, dev)), "sdpa_fwd_window")
    return o, lse


def fwd_f32(q, k, v, causal=False, scale=None, o=None, lse=None, want_lse=True, stream=None):
    """fp32 prefill on CUDA cores. Shapes as fwd; d_k, d_v <= 128."""
    import torch
    B, H, n_q, n_kv, d_k, d_v, o, lse, dev = _prefill_args(q, k, v, o, lse, torch.float32, want_lse)
    scale = 1.0 / math.sqrt(d_k) if scale is None else scale
    _check(_call(dev, lib.sdpa_fwd_f32, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, n_q, n_kv, d_k, d_v,
                 float(scale), int(bool(causal)), _stream(stream, dev)), "sdpa_fwd_f32")
    return o, lse
def _decode_args(q, k, v, kv_lens, o, lse, want_lse, grouped):
    """Shapes of a decode call: q [B,H_q,d_k], k [B,H_kv,n_cap,d_k], v [B,H_kv,n_cap,d_v], kv_lens [B]."""
    import torch
    _tensor(k, "k", torch.bfloat16, (None, None, None, None))
    B, H_kv, n_cap, d_k = k.shape
    _tensor(v, "v", torch.bfloat16, (B, H_kv, n_cap, None))
    d_v = v.shape[3]
    _tensor(q, "q", torch.bfloat16, (B, None if grouped else H_kv, d_k))
    H_q = q.shape[1]
    _tensor(kv_lens, "kv_lens", torch.int32, (B,))
    if o is not None:
        _tensor(o, "o", torch.bfloat16, (B, H_q, d_v))
    if lse is not None:
        _tensor(lse, "lse", torch.float32, (B, H_q))
    dev = _device("q", q, ("k", k), ("v", v), ("kv_lens", kv_lens), ("o", o), ("lse", lse))
    if o is None:
        o = torch.empty((B, H_q, d_v), dtype=torch.bfloat16, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((B, H_q), dtype=torch.float32, device=dev)
    return B, H_q, H_kv, n_cap, d_k, d_v, o, lse, dev


def _workspace(workspace, need, dev):
    import torch
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous torch.Tensor")
    _device("workspace", workspace)
    if workspace.device != dev:
        raise ValueError("workspace is on %s but the tensors are on %s" % (workspace.device, dev))
    return workspace


def decode_workspace_size(batch, heads, n_kv_cap, d_v):
    return int(lib.sdpa_decode_workspace_size(batch, heads, n_kv_cap, d_v))


def decode(q, k, v, kv_lens, scale=None, o=None, lse=None, want_lse=True, workspace=None, stream=None):
    """Decode. q [B,H,d], k/v [B,H,n_cap,d] bf16, kv_lens int32 [B] on the device."""
    B, H, _, n_cap, d_k, d_v, o, lse, dev = _decode_args(q, k, v, kv_lens, o, lse, want_lse, grouped=False)
    scale = 1.0 / math.sqrt(d_k) if scale is None else scale
    workspace = _workspace(workspace, decode_workspace_size(B, H, n_cap, d_v), dev)
    _check(_call(dev, lib.sdpa_decode, _ptr(q), _ptr(k), _ptr(v), _ptr(kv_lens), _ptr(o), _ptr(lse), B, H, n_cap,
                 d_k, d_v, float(scale), _ptr(workspace), _nbytes(workspace), _stream(stream, dev)), "sdpa_decode")
    return o, lse


def decode_noalloc(q, k, v, kv_lens, scale=None, o=None, lse=None, want_lse=True, stream=None):
    """Decode without a workspace: for callers that may not allocate device memory.

    Uses the library's fixed device scratch array (see sdpa_decode_noalloc in
    include/sdpa.h).  o and lse are allocated here only when not given.
    """
    B, H, _, n_cap, d_k, d_v, o, lse, dev = _decode_args(q, k, v, kv_lens, o, lse, want_lse, grouped=False)
    scale = 1.0 / math.sqrt(d_k) if scale is None else scale
    _check(_call(dev, lib.sdpa_decode_noalloc, _ptr(q), _ptr(k), _ptr(v), _ptr(kv_lens), _ptr(o), _ptr(lse), B, H,
                 n_cap, d_k, d_v, float(scale), _stream(stream, dev)), "sdpa_decode_noalloc")
    return o, lse


def decode_gqa_workspace_size(batch, heads_q, heads_kv, n_kv_cap, d_v):
    return int(lib.sdpa_decode_gqa_workspace_size(batch, heads_q, heads_kv, n_kv_cap, d_v))


def decode_gqa(q, k, v, kv_lens, scale=None, o=None, lse=None, want_lse=True, workspace=None, stream=None):
    """Grouped-query decode. q [B, H_q, d], k/v [B, H_kv, n_cap, d] bf16 (H_q a multiple of H_kv),
    kv_lens int32 [B] on the device; query head h reads key/value head h // (H_q // H_kv)."""
    B, H_q, H_kv, n_cap, d_k, d_v, o, lse, dev = _decode_args(q, k, v, kv_lens, o, lse, want_lse, grouped=True)
    scale = 1.0 / math.sqrt(d_k) if scale is None else scale
    workspace = _workspace(workspace, decode_gqa_workspace_size(B, H_q, H_kv, n_cap, d_v), dev)
    _check(_call(dev, lib.sdpa_decode_gqa, _ptr(q), _ptr(k), _ptr(v), _ptr(kv_lens), _ptr(o), _ptr(lse), B, H_q,
                 H_kv, n_cap, d_k, d_v, float(scale), _ptr(workspace), _nbytes(workspace), _stream(stream, dev)),
           "sdpa_decode_gqa")
    return o, lse


def bwd_workspace_size(batch, heads, n_q):
    return int(lib.sdpa_bwd_workspace_size(batch, heads, n_q))


def bwd(q, k, v, o, do, lse, causal=False, scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """Gradients of fwd: returns dQ, dK, dV (bf16, shapes of q, k, v) for loss gradient `do`,
    from the forward's inputs, output `o` and `lse`."""
    import torch
    bf = torch.bfloat16
    _tensor(q, "q", bf, (None, None, None, None))
    B, H, n_q, d_k = q.shape
    _tensor(k, "k", bf, (B, H, None, d_k))
    n_kv = k.shape[2]
    _tensor(v, "v", bf, (B, H, n_kv, None))
    d_v = v.shape[3]
    _tensor(o, "o", bf, (B, H, n_q, d_v))
    _tensor(do, "do", bf, (B, H, n_q, d_v))
    _tensor(lse, "lse", torch.float32, (B, H, n_q))
    for name, g, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if g is not None:
            _tensor(g, name, bf, tuple(like.shape))
    dev = _device("q", q, ("k", k), ("v", v), ("o", o), ("do", do), ("lse", lse), ("dq", dq), ("dk", dk),
                  ("dv", dv))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    scale = 1.0 / math.sqrt(d_k) if scale is None else scale
    workspace = _workspace(workspace, bwd_workspace_size(B, H, n_q), dev)
    _check(_call(dev, lib.sdpa_bwd, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
                 _ptr(dv), B, H, n_q, n_kv, d_k, d_v, float(scale), int(bool(causal)), _ptr(workspace),
                 _nbytes(workspace), _stream(stream, dev)), "sdpa_bwd")
    return dq, dk, dv


# ------------------------------------------------------------------------------ the bounded decode cache
# A decode step makes several of these calls, each a few microseconds on the GPU, so their checks take the short
# way where everything fits: one comparison per tensor, and no context managers on the current device and stream.
Kv4Cache = collections.namedtuple("Kv4Cache", "k_codes k_scales v_codes v_scales")
Kv4Cache.__doc__ = """Keys and values in 4 bits: codes uint8 [B,H,n_cap,d/2], scales bf16 [B,H,n_cap,d/32,2] (scale, minimum)."""


def kv4_cache(batch, heads, n_cap, d, device=None):
    """A zeroed 4-bit cache on `device` (default: the current CUDA device); d in {64,128}."""
    import torch
    if d not in (64, 128):
        raise ValueError("d must be 64 or 128, got %r" % (d,))
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return Kv4Cache(*(torch.zeros(shape, dtype=dtype, device=device) for _ in "kv" for shape, dtype in
                      (((batch, heads, n_cap, d // 2), torch.uint8),
                       ((batch, heads, n_cap, d // 32, 2), torch.bfloat16))))


def _fit(t, name, dtype, shape):
    """_tensor for a shape without free entries."""
    if getattr(t, "dtype", None) is dtype and t.shape == shape and t.is_contiguous():
        return t
    return _tensor(t, name, dtype, shape)


def _free(t, name, dtype, ndim):
    """_tensor for a shape that is free in every entry; returns it."""
    if getattr(t, "dtype", None) is dtype and t.dim() == ndim and t.is_contiguous():
        return t.shape
    return _tensor(t, name, dtype, (None,) * ndim).shape


_KV4_NAMES = {name: tuple("%s.%s" % (name, x) for x in Kv4Cache._fields) for name in ("cache", "out")}


def _kv4(cache, name="cache", B=None, H=None, d=None):
    """Check a Kv4Cache; returns B, H, n_cap, d."""
    import torch
    if not isinstance(cache, (tuple, list)) or len(cache) != 4:
        raise TypeError("%s must be a Kv4Cache, got %s" % (name, type(cache).__name__))
    kc, ks, vc, vs = cache
    names = _KV4_NAMES[name]
    codes = _free(kc, names[0], torch.uint8, 4)
    if B is not None and (codes[0], codes[1], 2 * codes[3]) != (B, H, d):
        _tensor(kc, names[0], torch.uint8, (B, H, None, d // 2))
    B, H, n_cap, half = codes
    scales = (B, H, n_cap, half // 16, 2)
    _fit(ks, names[1], torch.bfloat16, scales)
    _fit(vc, names[2], torch.uint8, codes)
    _fit(vs, names[3], torch.bfloat16, scales)
    return B, H, n_cap, 2 * half


def _here(names, *tensors):
    """_device for tensors named by `names`."""
    index = tensors[0].get_device()  # -1: on the host
    if index >= 0:
        for t in tensors:
            if t is not None and t.get_device() != index:
                break
        else:
            return tensors[0].device
    return _device(names[0], tensors[0], *zip(names[1:], tensors[1:]))


def _both(name, a, b):
    if (a is None) != (b is None):
        raise ValueError("give both of %s or neither" % name)


def _some_heads(name, heads):
    """Refuse calls without a head that would have to fill an output: the library writes nothing then."""
    if heads == 0:
        raise ValueError("%s must have at least one head" % name)


def _made(stream, make):
    """make() with its tensors made (and filled) on `stream` (None: the current one)."""
    import torch
    if stream is None:
        return make()
    with torch.cuda.stream(stream):
        return make()


def _at(t):
    return None if t is None else t.data_ptr()


def _launch(where, dev, stream, *args):
    """Call the library function `where` with these arguments and the stream, `dev` being current."""
    import torch
    index = dev.index
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        handle = raw(index) if raw else torch.cuda.current_stream(dev).cuda_stream
    else:
        handle = _stream(stream, dev)
    fn = getattr(lib, where)
    if torch.cuda.current_device() == index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != SDPA_OK:
        _check(status, where)


def kv4_append(cache, k, v, kv_lens, n_new=None, k_read=None, v_read=None, stream=None):
    """Quantise k, v [B,H,n_rows,d] bf16 into `cache`: row t of sequence b becomes cache row kv_lens[b] + t
    (t < n_new[b]; all rows without n_new).  kv_lens, n_new: int32 [B] on the device; kv_lens is not
    changed, nor are weights kept beside the cache (zero them where a slot starts again at length 0).  k_read, v_read (both or neither, shapes of k, v) receive the values the cache now stands for."""
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    B, H, n_cap, d = _kv4(cache)
    rows = _free(k, "k", bf, 4)
    _fit(k, "k", bf, (B, H, rows[2], d))
    _fit(v, "v", bf, rows)
    _fit(kv_lens, "kv_lens", i32, (B,))
    if n_new is not None:
        _fit(n_new, "n_new", i32, (B,))
    _both("k_read and v_read", k_read, v_read)
    if k_read is not None:
        _fit(k_read, "k_read", bf, rows)
        _fit(v_read, "v_read", bf, rows)
    kc, ks, vc, vs = cache
    dev = _here(("k", "v", "kv_lens", "n_new", "k_read", "v_read") + _KV4_NAMES["cache"], k, v, kv_lens, n_new, k_read, v_read,
                kc, ks, vc, vs)
    _launch("sdpa_kv4_append", dev, stream, k.data_ptr(), v.data_ptr(), kv_lens.data_ptr(), _at(n_new), kc.data_ptr(),
            ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), _at(k_read), _at(v_read), B, H, rows[2], n_cap, d)


def kv4_load(cache, kv_lens, n_rows=None, k=None, v=None, stream=None):
    """Cache rows 0 .. min(kv_lens[b], n_rows) - 1 as bf16 k, v [B,H,n_rows,d].  n_rows: that of k, v where they
    are given, else n_cap.  Rows past a sequence's length are left as they were (zero in tensors made here)."""
    import torch
    bf = torch.bfloat16
    B, H, n_cap, d = _kv4(cache)
    _both("k and v", k, v)
    if k is not None:
        n_rows = _free(k, "k", bf, 4)[2] if n_rows is None else n_rows
        _fit(k, "k", bf, (B, H, n_rows, d))
        _fit(v, "v", bf, (B, H, n_rows, d))
    _fit(kv_lens, "kv_lens", torch.int32, (B,))
    kc, ks, vc, vs = cache
    dev = _here(_KV4_NAMES["cache"] + ("kv_lens", "k", "v"), kc, ks, vc, vs, kv_lens, k, v)
    n_rows = n_cap if n_rows is None else n_rows
    if n_rows < 0:
        raise ValueError("n_rows must not be negative, got %d" % n_rows)
    if k is None:
        k, v = _made(stream, lambda: [torch.zeros((B, H, n_rows, d), dtype=bf, device=dev) for _ in "kv"])
    _launch("sdpa_kv4_load", dev, stream, kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), kv_lens.data_ptr(),
            k.data_ptr(), v.data_ptr(), B, H, n_rows, n_cap, d)
    return k, v


def _acc_args(acc, acc_out, shape):
    """acc, acc_out of a decode or of fwd_acc (whose last entry is free: None): acc_out defaults to acc (the running sum)."""
    import torch
    for name, t in (("acc", acc), ("acc_out", acc_out)):
        if t is not None:
            if shape[2] is None:
                shape = shape[:2] + tuple(_free(t, name, torch.float32, 3)[2:])
            _fit(t, name, torch.float32, shape)
    return acc if acc_out is None else acc_out


def _decode_made(q, o, lse, want_lse, workspace, need, dev):
    """The outputs and the workspace of a decode, those not given made on the current stream."""
    import torch
    if o is None:
        o = torch.empty_like(q)
    if lse is None and want_lse:
        lse = q.new_empty(q.shape[:2], dtype=torch.float32)
    if workspace is None:
        return o, lse, q.new_empty(max(need, 16), dtype=torch.uint8)
    return o, lse, _workspace(workspace, 0, dev)


def _decode_run(where, size, q, keys, names, kv_lens, B, H_kv, n_cap, d, scale, o, lse, want_lse, acc, acc_out, workspace,
                stream):
    """The part that decode_kv4 and decode_acc share: `keys` are the cache's arrays, `size` the function that gives the
    workspace's bytes."""
    import torch
    H_q = _free(q, "q", torch.bfloat16, 3)[1]
    _fit(q, "q", torch.bfloat16, (B, H_q, d))
    if acc_out is not None:
        _some_heads("q", H_q)
    _fit(kv_lens, "kv_lens", torch.int32, (B,))
    if o is not None:
        _fit(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _fit(lse, "lse", torch.float32, (B, H_q))
    dev = _here(("q", "kv_lens", "o", "lse", "acc", "acc_out") + names, q, kv_lens, o, lse, acc, acc_out, *keys)
    need = size(B, H_q, H_kv, n_cap, d, acc_out is not None) if workspace is None else 0
    if stream is None:
        o, lse, ws = _decode_made(q, o, lse, want_lse, workspace, need, dev)
    else:
        with torch.cuda.stream(stream):
            o, lse, ws = _decode_made(q, o, lse, want_lse, workspace, need, dev)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    _launch(where, dev, stream, q.data_ptr(), *[t.data_ptr() for t in keys], kv_lens.data_ptr(), o.data_ptr(), _at(lse),
            _at(acc), _at(acc_out), B, H_q, H_kv, n_cap, d, scale, ws.data_ptr(), _nbytes(ws))
    return o, lse


@functools.lru_cache(maxsize=256)
def decode_kv4_workspace_size(batch, heads_q, heads_kv, n_kv_cap, d, with_acc=False):
    return int(lib.sdpa_decode_kv4_workspace_size(batch, heads_q, heads_kv, n_kv_cap, d, int(bool(with_acc))))


def decode_kv4(q, cache, kv_lens, scale=None, o=None, lse=None, want_lse=True, acc=None, acc_out=None, workspace=None,
               stream=None):
    """Grouped-query decode over a 4-bit cache. q [B,H_q,d] bf16, cache of H_kv heads (H_q a multiple), kv_lens int32
    [B] on the device (0: an empty slot, O = 0 and LSE = -inf).  With acc [B,H_kv,n_cap] fp32, each cached key's
    weights, summed over the query heads that read it, are added: acc_out = acc + weights (in place without acc_out;
    acc_out alone starts from zero); entries past kv_lens are left as they were."""
    B, H_kv, n_cap, d = _kv4(cache)
    if acc is not None or acc_out is not None:
        acc_out = _acc_args(acc, acc_out, (B, H_kv, n_cap))
    return _decode_run("sdpa_decode_kv4", decode_kv4_workspace_size, q, cache, _KV4_NAMES["cache"], kv_lens, B, H_kv,
                       n_cap, d, scale, o, lse, want_lse, acc, acc_out, workspace, stream)


@functools.lru_cache(maxsize=256)
def decode_acc_workspace_size(batch, heads_q, heads_kv, n_kv_cap, d):
    return int(lib.sdpa_decode_acc_workspace_size(batch, heads_q, heads_kv, n_kv_cap, d))


def _decode_acc_size(batch, heads_q, heads_kv, n_kv_cap, d, with_acc):
    return decode_acc_workspace_size(batch, heads_q, heads_kv, n_kv_cap, d)


def decode_acc(q, k, v, kv_lens, acc=None, acc_out=None, scale=None, o=None, lse=None, want_lse=True, workspace=None,
               stream=None):
    """decode_gqa over a bf16 cache k, v [B,H_kv,n_cap,d] that also sums the keys' attention weights; acc, acc_out (one
    of them at least) and empty slots as in decode_kv4."""
    import torch
    B, H_kv, n_cap, d = _free(k, "k", torch.bfloat16, 4)
    _fit(v, "v", torch.bfloat16, k.shape)
    if acc is None and acc_out is None:
        raise ValueError("give acc, acc_out or both")
    acc_out = _acc_args(acc, acc_out, (B, H_kv, n_cap))
    return _decode_run("sdpa_decode_acc", _decode_acc_size, q, (k, v), ("k", "v"), kv_lens, B, H_kv, n_cap, d, scale, o,
                       lse, want_lse, acc, acc_out, workspace, stream)


def fwd_acc(q, k, lse, acc=None, causal=False, scale=None, acc_out=None, stream=None):
    """The attention weights of a prompt summed over its queries and the heads of each group. q [B,H_q,n_q,d],
    k [B,H_kv,n_kv,d] bf16, lse [B,H_q,n_q] as fwd returned it for the same mask and scale; the last n_q queries of a
    longer prompt may be given alone (causal is bottom-right aligned).  acc [B,H_kv,n_acc] fp32, n_acc >= n_kv:
    acc_out = acc + weights for the n_kv keys, in place without acc_out; without both a new [B,H_kv,n_kv] tensor.
    Returns acc_out."""
    import torch
    B, H_q, n_q, d = _free(q, "q", torch.bfloat16, 4)
    _some_heads("q", H_q)
    _, H_kv, n_kv, _ = _free(k, "k", torch.bfloat16, 4)
    _fit(k, "k", torch.bfloat16, (B, H_kv, n_kv, d))
    _fit(lse, "lse", torch.float32, (B, H_q, n_q))
    acc_out = _acc_args(acc, acc_out, (B, H_kv, None))
    dev = _here(("q", "k", "lse", "acc", "acc_out"), q, k, lse, acc, acc_out)
    if acc_out is None:
        acc_out = _made(stream, lambda: torch.empty((B, H_kv, n_kv), dtype=torch.float32, device=dev))
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    _launch("sdpa_fwd_acc", dev, stream, q.data_ptr(), k.data_ptr(), lse.data_ptr(), _at(acc), acc_out.data_ptr(),
            B, H_q, H_kv, n_q, n_kv, acc_out.shape[2], d, scale, int(bool(causal)))
    return acc_out


def _evict_run(where, arrays, outs, names, out_names, acc, kv_lens, budget, recent, acc_out, B, H, n_cap, n_out, d, stream):
    """The part that evict and kv4_evict share; outs None: in place."""
    import torch
    budget, recent = int(budget), int(recent)
    _some_heads(names[0], H)
    _fit(acc, "acc", torch.float32, (B, H, n_cap))
    _fit(kv_lens, "kv_lens", torch.int32, (B,))
    if (outs is None) != (acc_out is None):
        raise ValueError("give %s and acc_out together, or none of them (in place)" % ", ".join(out_names))
    if acc_out is not None:
        _fit(acc_out, "acc_out", torch.float32, (B, H, n_out))
        dev = _here(names + ("acc", "kv_lens", "acc_out") + out_names, *arrays, acc, kv_lens, acc_out, *outs)
    else:
        outs, acc_out = arrays, acc
        dev = _here(names + ("acc", "kv_lens"), *arrays, acc, kv_lens)
    if not 1 <= budget <= n_out:
        raise ValueError("budget must be between 1 and the output's capacity %d, got %d" % (n_out, budget))

    def results():
        return kv_lens.new_empty((B, H, budget)), torch.empty_like(kv_lens)
    keep, new_lens = results() if stream is None else _made(stream, results)
    _launch(where, dev, stream, *[t.data_ptr() for t in arrays], acc.data_ptr(), kv_lens.data_ptr(),
            *[t.data_ptr() for t in outs], acc_out.data_ptr(), keep.data_ptr(), new_lens.data_ptr(), B, H, n_cap, n_out, d,
            budget, recent)
    return keep, new_lens


def evict(k, v, acc, kv_lens, budget, recent=0, k_out=None, v_out=None, acc_out=None, stream=None):
    """Keep at most `budget` rows of each sequence and head of a bf16 cache k, v [B,H,n_cap,d]: the last `recent` and
    those with the largest acc [B,H,n_cap] (the lower row where equal), in order, as rows 0, 1, ...  In place, or into
    k_out, v_out [B,H,n_out,d] and acc_out [B,H,n_out].  acc becomes the kept rows' weights, 0 after them.  Returns
    keep int32 [B,H,budget] (the old rows, -1 past the new length) and the new lengths int32 [B]."""
    import torch
    bf = torch.bfloat16
    B, H, n_cap, d = _free(k, "k", bf, 4)
    _fit(v, "v", bf, k.shape)
    _both("k_out and v_out", k_out, v_out)
    n_out, outs = n_cap, None
    if k_out is not None:
        n_out, outs = _free(k_out, "k_out", bf, 4)[2], (k_out, v_out)
        _fit(k_out, "k_out", bf, (B, H, n_out, d))
        _fit(v_out, "v_out", bf, k_out.shape)
    return _evict_run("sdpa_evict", (k, v), outs, ("k", "v"), ("k_out", "v_out"), acc, kv_lens, budget, recent, acc_out, B, H,
                      n_cap, n_out, d, stream)


def kv4_evict(cache, acc, kv_lens, budget, recent=0, out=None, acc_out=None, stream=None):
    """evict for a 4-bit cache: in place, or into the cache `out` (any capacity >= budget) and acc_out."""
    B, H, n_cap, d = _kv4(cache)
    n_out = n_cap if out is None else _kv4(out, "out", B, H, d)[2]
    return _evict_run("sdpa_kv4_evict", cache, out, _KV4_NAMES["cache"], _KV4_NAMES["out"], acc, kv_lens, budget, recent,
                      acc_out, B, H, n_cap, n_out, d, stream)


def get_last_device_error(stream=None):
    """Synchronise `stream` (default: the current stream of the current device), then read and
    clear the current device's error word."""
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(lib.sdpa_get_last_device_error(ctypes.c_void_p(s.cuda_stream)))
