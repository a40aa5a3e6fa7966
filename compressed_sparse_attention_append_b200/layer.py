"""Binding of include/csa2_layer.h: the operators around the CSA2 core. Argument marshalling only, in the
manner of the package's other calls (same names as the C entry points, tensors for pointers, the
current CUDA stream, Csa2Error on a non-zero status, no CPU fallback). Every tensor of a call lies on the
current device. A call as it should be goes through csrc/marshal.cpp (3.2 us of host time with the launch,
against 6 to 8 through ctypes); whatever that does not take comes back and is done, or refused with its reason,
by the code below.

One decode step of a layer of the pages' own shape, `B` sequences (bf16 unless noted):

    rope = Rope.for_context(64, 10000.0, "yarn", 16.0, 65536, offset=448, interleaved=True)
    cache = PagedCache(n_pages, 64, B, max_pages)         # cache.table [B, max_pages] int32: the caller's
    csa2_fp8_quantize(hidden, xq, xs)                      # E4M3 rows, one scale per 128 channels
    csa2_fp8_gemm(xq, xs, wq, wq_scale, q.view(B, -1))     # ... one product per projection
    csa2_norm_rope(rope, pos, eps, q, q_weight, q)         # per-head norm and rotation, in place
    csa2_paged_append(cache, B, 1, pos, latent, idx_k, swa, rope=rope, idx_rope=idx_rope,
                      w_latent=w_l, w_idx_k=w_k, w_swa=w_s, eps=eps, ws=ws)
    csa2_paged_index_topk(cache, B, 1, pos, idx_q, 512, idx, index_ws)
    csa2_paged_attend(cache, B, 1, pos, q, idx, 512, out, ws=ws)
    csa2_rope(rope.inverted(), pos, out, out)              # K = V: the output turned back, mscale taken out
"""
from __future__ import annotations

import ctypes
import struct

import torch

CSA2_BF16 = 0
CSA2_F32 = 1
CSA2_DEV_BAD_PAGE = 0x10
CSA2_ROPE_HALF = 0
CSA2_ROPE_INTERLEAVED = 1
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "yarn": 3}

LAYER_EXPORTS = (
    "csa2_rope_frequencies", "csa2_rope", "csa2_norm_rope", "csa2_fp8_quantize", "csa2_fp8_quantize_weight",
    "csa2_fp8_gemm", "csa2_paged_append", "csa2_paged_gather", "csa2_paged_attend", "csa2_paged_index_topk",
)


class csa2_rope_spec(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot", ctypes.c_int), ("offset", ctypes.c_int),
                ("layout", ctypes.c_int), ("transposed", ctypes.c_int), ("mscale", ctypes.c_float)]


class csa2_heads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("x_token", ctypes.c_int64),
                ("x_head", ctypes.c_int64), ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("heads", ctypes.c_int)]


class csa2_append_row(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_batch", ctypes.c_int64), ("x_token", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("rope", ctypes.POINTER(csa2_rope_spec))]


class csa2_paged_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("l_data", "l_scale", "k_data", "k_scale", "swa", "table", "swa_slot")]
    _fields_ += [(n, ctypes.c_int64) for n in ("n_pages", "max_pages", "n_slots", "swa_cap")]
    _fields_ += [("page", ctypes.c_int)]


class _rope_on(ctypes.Structure):
    """A rotation and the device that its frequencies lie on, as csrc/marshal.cpp reads them."""
    _fields_ = [("spec", csa2_rope_spec), ("dev", ctypes.c_int)]


def declare(L):
    """The signatures of include/csa2_layer.h on the loaded library."""
    vp, i, i64, u32, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float, ctypes.c_size_t
    dbl, P = ctypes.c_double, ctypes.POINTER
    # structs travel as their bytes (packing them costs half of filling a ctypes structure)
    R, H, A, C = P(csa2_rope_spec), vp, vp, P(csa2_paged_cache)
    sig = {
        "csa2_rope_frequencies": [i, dbl, i, dbl, i64, dbl, dbl, vp, P(f)],
        "csa2_rope": [R, i, i64, i, vp, H, vp],
        "csa2_norm_rope": [R, i, i64, i, vp, f, H, H, vp],
        "csa2_fp8_quantize": [i64, i, vp, i64, vp, vp, vp],
        "csa2_fp8_quantize_weight": [i64, i, vp, vp, vp, vp],
        "csa2_fp8_gemm": [i64, i64, i, vp, vp, vp, vp, i, vp, i64, vp, sz, vp],
        "csa2_paged_append": [C, i, i, vp, vp, vp, f, A, A, A, vp, sz, vp],
        "csa2_paged_gather": [C, i, i, vp, vp, vp, vp, sz, vp],
        "csa2_paged_attend": [C, i, i, vp, vp, vp, i, vp, i, i, f, vp, vp, vp, vp, sz, vp],
        "csa2_paged_index_topk": [C, i, i, vp, vp, i, i, i, i64, u32, vp, vp, sz, vp],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.restype = i
        fn.argtypes = args


from . import Csa2Error, _check, lib  # noqa: E402  (the package imports this module last)

_TYPES = {torch.bfloat16: CSA2_BF16, torch.float32: CSA2_F32}
_I64, _I32, _F32, _BF16, _U8, _F64 = torch.int64, torch.int32, torch.float32, torch.bfloat16, torch.uint8, torch.float64
_E4M3 = torch.float8_e4m3fn  # (uint8 bytes are taken too)
_raw_device = None
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _device():
    """The current device (-2 without a GPU, which no tensor lies on)."""
    global _raw_device
    if _raw_device is None:
        if not torch.cuda.is_available():
            return -2
        torch.cuda.init()
        _raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _raw_device()


def _stream(stream, dev):
    """The stream's handle; the current one's through the short way (a decode step's calls are host time)."""
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _refuse(t, dtype, dev, shape, dense):
    """Names what is wrong with a tensor that _ptr did not take."""
    names = f"{dtype} or {_U8}" if dtype is _E4M3 else str(dtype)
    assert isinstance(t, torch.Tensor) and (t.dtype is dtype or (dtype is _E4M3 and t.dtype is _U8)), f"expected a {names} tensor"
    assert t.is_cuda, "expected a CUDA tensor"
    assert t.get_device() == dev, "expected a tensor of the current device"
    assert not dense or t.is_contiguous(), "expected a contiguous tensor"
    assert shape is None or t.shape == shape, f"expected the shape {tuple(shape)}, got {tuple(t.shape)}"
    return t.data_ptr()


def _ptr(t, dtype, dev, shape):
    """The pointer of a dense tensor after the checks that the library cannot make (None stays None)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return _refuse(t, dtype, dev, shape, True)


def _strided(t, dtype, dev, shape):
    """The same for a tensor whose strides travel with it."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape:
            return t.data_ptr()
    except AttributeError:
        pass
    return _refuse(t, dtype, dev, shape, False)


_heads_bytes = struct.Struct("@PPqqqqPi4x").pack    # csa2_heads
_row_bytes = struct.Struct("@PqqPP").pack           # csa2_append_row
assert struct.calcsize("@PPqqqqPi4x") == ctypes.sizeof(csa2_heads)
assert struct.calcsize("@PqqPP") == ctypes.sizeof(csa2_append_row)


_lib = None
_fast = None  # csrc/marshal.cpp: the checks and the call of the plain cases in native code, once the library is loaded


def _load():
    """The library, kept here after the first call."""
    global _lib, _fast
    _lib = lib()
    try:
        from . import _marshal
    except ImportError:  # not built here: the calls below are complete without it
        return _lib
    if torch.__version__.split("+")[0] == _marshal.torch_version:
        names = ("rope", "norm_rope", "fp8_quantize", "fp8_gemm", "paged_append", "paged_gather", "paged_attend")
        _marshal.bind(*(ctypes.cast(getattr(_lib, "csa2_" + n), ctypes.c_void_p).value for n in names))
        _fast = _marshal
    return _lib


def _status(ws):
    """Address and size of a workspace, which has to be the current device's."""
    if ws is None:
        return None, 0
    buf = getattr(ws, "buf", None)
    assert buf is None or buf.get_device() == _device(), "expected a workspace of the current device"
    return ws.ptr, ws.nbytes


class _Fixed:
    """The attributes that a C struct was made from are set once: the struct would not follow them."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError(f"{name} is fixed: fill its tensor in place, or make another {type(self).__name__}")
        super().__setattr__(name, value)


class Rope(_Fixed):
    """A rotation (csa2_rope_spec) and the tensor of its frequencies: inv_freq [rot / 2] float64, radians
    per position, on the device that it is used on; `offset` the first rotated channel; `inverse` turns the other way
    (times mscale as well)."""

    def __init__(self, inv_freq, offset=0, interleaved=False, mscale=1.0, inverse=False):
        self.inv_freq, self.offset, self.interleaved = inv_freq, int(offset), bool(interleaved)
        self.mscale, self.inverse = float(mscale), bool(inverse)
        self.rot = 2 * inv_freq.numel()
        dev = _device()
        self.c = _rope_on((_ptr(inv_freq, _F64, dev, (self.rot // 2,)), self.rot, self.offset, int(self.interleaved),
                           int(self.inverse), self.mscale), dev)
        self.ref = ctypes.pointer(self.c.spec)
        self.at = ctypes.addressof(self.c)

    def on(self, dev):
        """Itself, for a call on device `dev`."""
        assert self.c.dev == dev, "expected a rotation of the current device"
        return self

    @classmethod
    def for_context(cls, rot, base=10000.0, scaling="plain", factor=1.0, orig_ctx=0, beta_fast=32.0, beta_slow=1.0,
                    offset=0, interleaved=False, device="cuda"):
        """The frequencies of csa2_rope_frequencies (scaling: "plain", "linear", "ntk" or "yarn")."""
        f, mscale = csa2_rope_frequencies(rot, base, scaling, factor, orig_ctx, beta_fast, beta_slow)
        return cls(f.to(device), offset, interleaved, mscale)

    def transposed(self):
        """The transposed matrix (turned back, times mscale again): the rotation's gradient."""
        return Rope(self.inv_freq, self.offset, self.interleaved, self.mscale, not self.inverse)

    def inverted(self):
        """The inverse (turned back, divided by mscale): what undoes the rotation. With K = V the attention's output
        needs it. (A rotation made with mscale 1 keeps the scale out of the values; mscale^2 / sqrt(512) is then
        the sm_scale of a head that is rotated whole.)"""
        return Rope(self.inv_freq, self.offset, self.interleaved, 1.0 / (self.mscale or 1.0), not self.inverse)


def csa2_rope_frequencies(rot, base=10000.0, scaling="plain", factor=1.0, orig_ctx=0, beta_fast=32.0, beta_slow=1.0):
    """(inv_freq [rot / 2] float64 on the host, mscale)."""
    f = torch.zeros(max(rot, 0) // 2, dtype=torch.float64)
    m = ctypes.c_float(0.0)
    _check("csa2_rope_frequencies", lib().csa2_rope_frequencies(
        rot, base, ROPE_SCALINGS[scaling], factor, orig_ctx, beta_fast, beta_slow, f.data_ptr(), ctypes.byref(m)))
    return f, m.value


def _heads(x, out, weight, dtype, dev, tokens, d):
    shape = x.shape
    t, heads, ch = shape
    x0, x1, x2 = x.stride()
    o0, o1, o2 = out.stride()
    assert t == tokens and ch == d, "expected [tokens, heads, d]"
    assert x2 == 1 and o2 == 1, "expected dense heads (stride 1 along the channels)"
    return _heads_bytes(_strided(x, dtype, dev, shape), _strided(out, dtype, dev, shape), x0, x1, o0, o1,
                        0 if weight is None else _ptr(weight, dtype, dev, (d,)), heads)


def csa2_rope(rope: Rope, pos, x, out, stream=None):
    """x [tokens, heads, d] bf16 or fp32 (any strides, dense heads) -> out (may be x), pos [tokens] int64."""
    s = _fast and _fast.rope(rope.at, pos, x, out, stream)
    if s is None:
        s = _rope(rope, pos, x, out, stream)
    if s:
        raise Csa2Error("csa2_rope", s)


def _rope(rope, pos, x, out, stream):
    tokens, _, d = x.shape
    dtype, dev = x.dtype, _device()
    assert dtype in _TYPES, "expected a bf16 or fp32 tensor"
    h = _heads(x, out, None, dtype, dev, tokens, d)
    return (_lib or _load()).csa2_rope(
        rope.on(dev).ref, _TYPES[dtype], tokens, d, _ptr(pos, _I64, dev, (tokens,)), h, _stream(stream, dev))


def csa2_norm_rope(rope, pos, eps, q, wq, q_out, k=None, wk=None, k_out=None, stream=None):
    """q [tokens, hq, d] and k [tokens, hk, d] (or None) normed per head with weights wq, wk [d] (or None) and
    rotated (rope None: the norm alone) -> q_out, k_out (may be q, k)."""
    s = _fast and _fast.norm_rope(None if rope is None else rope.at, pos, eps, q, wq, q_out, k, wk, k_out, stream)
    if s is None:
        s = _norm_rope(rope, pos, eps, q, wq, q_out, k, wk, k_out, stream)
    if s:
        raise Csa2Error("csa2_norm_rope", s)


def _norm_rope(rope, pos, eps, q, wq, q_out, k, wk, k_out, stream):
    tokens, _, d = q.shape
    dtype, dev = q.dtype, _device()
    assert dtype in _TYPES, "expected a bf16 or fp32 tensor"
    hq = _heads(q, q_out, wq, dtype, dev, tokens, d)
    hk = None if k is None else _heads(k, k_out, wk, dtype, dev, tokens, d)
    return (_lib or _load()).csa2_norm_rope(
        None if rope is None else rope.on(dev).ref, _TYPES[dtype], tokens, d, _ptr(pos, _I64, dev, (tokens,)), eps, hq, hk,
        _stream(stream, dev))


def csa2_fp8_quantize(x, data, scale, stream=None):
    """x [rows, k] bf16 (dense rows) -> data [rows, k] E4M3 (or uint8), scale [ceil(k / 128), rows] fp32."""
    s = _fast and _fast.quantize(x, data, scale, stream)
    if s is None:
        s = _fp8_quantize(x, data, scale, stream)
    if s:
        raise Csa2Error("csa2_fp8_quantize", s)


def _fp8_quantize(x, data, scale, stream):
    rows, k = x.shape
    xs, one = x.stride()
    dev = _device()
    assert one == 1 or k == 1, "expected dense rows"
    return (_lib or _load()).csa2_fp8_quantize(
        rows, k, _strided(x, _BF16, dev, (rows, k)), xs, _ptr(data, _E4M3, dev, (rows, k)),
        _ptr(scale, _F32, dev, (-(-k // 128), rows)), _stream(stream, dev))


def csa2_fp8_quantize_weight(w, data, scale, stream=None):
    """w [n, k] bf16 -> data [n, k] E4M3 (or uint8), scale [ceil(n / 128), ceil(k / 128)] fp32."""
    n, k = w.shape
    dev = _device()
    _check("csa2_fp8_quantize_weight", lib().csa2_fp8_quantize_weight(
        n, k, _ptr(w, _BF16, dev, (n, k)), _ptr(data, _E4M3, dev, (n, k)),
        _ptr(scale, _F32, dev, (-(-n // 128), -(-k // 128))), _stream(stream, dev)))


def csa2_fp8_gemm(x, xs, w, ws, out, status=None, stream=None):
    """out [m, n] (bf16 or fp32, dense rows) = x [m, k] w [n, k]^T, E4M3 with the scales of csa2_fp8_quantize (xs)
    and csa2_fp8_quantize_weight (ws); status: a workspace for CSA2_DEV_TIMEOUT."""
    at, size = _status(status)
    s = _fast and _fast.gemm(x, xs, w, ws, out, at, size, stream)
    if s is None:
        s = _fp8_gemm(x, xs, w, ws, out, at, size, stream)
    if s:
        raise Csa2Error("csa2_fp8_gemm", s)


def _fp8_gemm(x, xs, w, ws, out, at, size, stream):
    m, k = x.shape
    n, nb, dev, dtype = w.shape[0], -(-k // 128), _device(), out.dtype
    o0, o1 = out.stride()
    assert dtype in _TYPES, "expected a bf16 or fp32 tensor"
    assert o1 == 1 or n == 1, "expected dense rows"
    return (_lib or _load()).csa2_fp8_gemm(
        m, n, k, _ptr(x, _E4M3, dev, (m, k)), _ptr(xs, _F32, dev, (nb, m)), _ptr(w, _E4M3, dev, (n, k)),
        _ptr(ws, _F32, dev, (-(-n // 128), nb)), _TYPES[dtype], _strided(out, dtype, dev, (m, n)),
        o0 if m > 1 else n, at, size, _stream(stream, dev))  # (a single row's stride means nothing)


class PagedCache(_Fixed):
    """Planes of csa2_paged_cache, allocated with torch unless given: n_pages pages of `page` entries, the page
    table of `batch` sequences ([batch, max_pages] int32, -1 = no page; the caller fills `table` in place) and
    n_slots window rings (default: one per sequence; swa_slot [batch] int32 names each sequence's)."""

    def __init__(self, n_pages, page, batch, max_pages, swa_cap=128, n_slots=None, swa_slot=None, device="cuda",
                 latent=True, indexer=True, page_table=None, l_data=None, l_scale=None, k_data=None, k_scale=None,
                 swa=None):
        n_slots = batch if n_slots is None else n_slots
        self.n_pages, self.page, self.batch, self.max_pages = n_pages, page, batch, max_pages
        self.n_slots, self.swa_cap, self.swa_slot = n_slots, swa_cap, swa_slot
        z = lambda t, *s: torch.zeros(*s, dtype=torch.uint8, device=device) if t is None else t
        self.l_data = z(l_data, n_pages, page, 256) if latent else None
        self.l_scale = z(l_scale, n_pages, page, 32) if latent else None
        self.k_data = z(k_data, n_pages, page, 64) if indexer else None
        self.k_scale = z(k_scale, n_pages, page, 4) if indexer else None
        self.swa = z(swa, n_slots, swa_cap, 512)
        self.table = page_table if page_table is not None else torch.full((batch, max_pages), -1, dtype=torch.int32,
                                                                          device=device)
        assert swa_slot is not None or n_slots >= batch, "expected a window ring per sequence"
        dev = _device()
        self.c = csa2_paged_cache(
            _ptr(self.l_data, _U8, dev, (n_pages, page, 256)), _ptr(self.l_scale, _U8, dev, (n_pages, page, 32)),
            _ptr(self.k_data, _U8, dev, (n_pages, page, 64)), _ptr(self.k_scale, _U8, dev, (n_pages, page, 4)),
            _ptr(self.swa, _U8, dev, (n_slots, swa_cap, 512)), _ptr(self.table, _I32, dev, (batch, max_pages)),
            _ptr(swa_slot, _I32, dev, (batch,)), n_pages, max_pages, n_slots, swa_cap, page)
        self.dev = dev
        self.ref = ctypes.byref(self.c)
        self.at = ctypes.addressof(self.c)

    def on(self, batch):
        """The current device, which has to be the cache's, for a call of `batch` sequences."""
        dev = _device()
        assert dev == self.dev, "expected the cache's device to be the current one"
        assert batch <= self.batch, "expected at most the page table's sequences"
        return dev


def _append_row(x, weight, rope, dev, batch, t, channels):
    if x is None:
        return None
    x0, x1, x2 = x.stride()
    assert x2 == 1, f"expected dense rows [{batch}, {t}, {channels}]"
    return _row_bytes(_strided(x, _BF16, dev, (batch, t, channels)), x0, x1,
                      0 if weight is None else _ptr(weight, _BF16, dev, (channels,)), 0 if rope is None else rope.on(dev).at)


def csa2_paged_append(cache: PagedCache, batch, t, pos, latent=None, idx_k=None, swa=None, rope=None, idx_rope=None,
                      swa_rope=None, w_latent=None, w_idx_k=None, w_swa=None, eps=1e-6, length=None, rpos=None,
                      ws=None, stream=None):
    """latent [B, t, 512], idx_k [B, t, 128], swa [B, t, 512] bf16 (any may be None; any strides, dense rows) at
    entries pos [B] int64, normed with the weights that are given and rotated (`rope` latent and window rows,
    unless swa_rope is given, `idx_rope` the key); length [B] int32: tokens of each sequence (None: t);
    rpos [B, t] int64: the tokens' positions for the rotation (None: those of the entries)."""
    at, size = _status(ws)
    if swa_rope is None:
        swa_rope = rope
    turn = None if rope is None else rope.at
    s = _fast and _fast.append(
        cache.at, cache.dev, cache.batch, batch, t, pos, length, rpos, eps, latent, w_latent, turn, idx_k, w_idx_k,
        None if idx_rope is None else idx_rope.at, swa, w_swa, turn if swa_rope is rope else swa_rope.at, at, size, stream)
    if s is None:
        s = _paged_append(cache, batch, t, pos, latent, idx_k, swa, rope, idx_rope, swa_rope, w_latent, w_idx_k, w_swa, eps,
                          length, rpos, at, size, stream)
    if s:
        raise Csa2Error("csa2_paged_append", s)


def _paged_append(cache, batch, t, pos, latent, idx_k, swa, rope, idx_rope, swa_rope, w_latent, w_idx_k, w_swa, eps,
                  length, rpos, at, size, stream):
    dev = cache.on(batch)
    return (_lib or _load()).csa2_paged_append(
        cache.ref, batch, t, _ptr(pos, _I64, dev, (batch,)), _ptr(length, _I32, dev, (batch,)),
        _ptr(rpos, _I64, dev, (batch, t)), eps, _append_row(latent, w_latent, rope, dev, batch, t, 512),
        _append_row(idx_k, w_idx_k, idx_rope, dev, batch, t, 128),
        _append_row(swa, w_swa, swa_rope, dev, batch, t, 512), at, size,
        _stream(stream, dev))


def csa2_paged_gather(cache: PagedCache, batch, idx, latent=None, key=None, ws=None, stream=None):
    """idx [B, n] int32 entries (-1: zeros) -> latent [B, n, 512] and key [B, n, 128] bf16 (either may be None)."""
    at, size = _status(ws)
    s = _fast and _fast.gather(cache.at, cache.dev, cache.batch, batch, idx, latent, key, at, size, stream)
    if s is None:
        s = _paged_gather(cache, batch, idx, latent, key, at, size, stream)
    if s:
        raise Csa2Error("csa2_paged_gather", s)


def _paged_gather(cache, batch, idx, latent, key, at, size, stream):
    dev, n = cache.on(batch), idx.shape[1]
    return (_lib or _load()).csa2_paged_gather(
        cache.ref, batch, n, _ptr(idx, _I32, dev, (batch, n)), _ptr(latent, _BF16, dev, (batch, n, 512)),
        _ptr(key, _BF16, dev, (batch, n, 128)), at, size, _stream(stream, dev))


def csa2_paged_attend(cache: PagedCache, batch, tq, qpos, q, idx, k, out, swa_begin=None, win=128, ratio=1,
                      sm_scale=0.0, out_f32=None, lse=None, ws=None, stream=None):
    """q [B*tq, 64, 512] bf16, idx [B*tq, k] int32 -> out [B*tq, 64, 512] bf16 (tensor cores)."""
    at, size = _status(ws)
    s = _fast and _fast.attend(cache.at, cache.dev, cache.batch, batch, tq, qpos, q, idx, k, swa_begin, win, ratio, sm_scale,
                               out, out_f32, lse, at, size, stream)
    if s is None:
        s = _paged_attend(cache, batch, tq, qpos, q, idx, k, out, swa_begin, win, ratio, sm_scale, out_f32, lse, at, size,
                          stream)
    if s:
        raise Csa2Error("csa2_paged_attend", s)


def _paged_attend(cache, batch, tq, qpos, q, idx, k, out, swa_begin, win, ratio, sm_scale, out_f32, lse, at, size,
                  stream):
    dev, rows = cache.on(batch), batch * tq
    return (_lib or _load()).csa2_paged_attend(
        cache.ref, batch, tq, _ptr(qpos, _I64, dev, (rows,)), _ptr(q, _BF16, dev, (rows, 64, 512)),
        _ptr(idx, _I32, dev, (rows, k)), k, _ptr(swa_begin, _I64, dev, (batch,)), win, ratio, sm_scale,
        _ptr(out, _BF16, dev, (rows, 64, 512)), _ptr(out_f32, _F32, dev, (rows, 64, 512)),
        _ptr(lse, _F32, dev, (rows, 64)), at, size, _stream(stream, dev))


def csa2_paged_index_topk(cache: PagedCache, batch, tq, qpos, idx_q, k, out_idx, ws, ratio=1, max_ctx=None, flags=0,
                          stream=None):
    """idx_q [B*tq, hi, 128] bf16 -> out_idx [B*tq, k] int32; ws: a LatentIndexWorkspace."""
    dev, rows, hi = cache.on(batch), batch * tq, idx_q.shape[-2]
    if max_ctx is None:
        max_ctx = cache.max_pages * cache.page
    at, size = _status(ws)
    s = (_lib or _load()).csa2_paged_index_topk(
        cache.ref, batch, tq, _ptr(qpos, _I64, dev, (rows,)), _ptr(idx_q, _BF16, dev, (rows, hi, 128)), hi, k, ratio,
        max_ctx, flags, _ptr(out_idx, _I32, dev, (rows, k)), at, size, _stream(stream, dev))
    if s:
        raise Csa2Error("csa2_paged_index_topk", s)
