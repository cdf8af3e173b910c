"""Python binding of libsvq (include/svq.h): argument marshalling only.

Every entry point takes torch CUDA tensors (device memory) and the current
torch stream, passes raw pointers to the C ABI and raises SvqError on a
non-zero status.  All computation happens in the CUDA kernels of libsvq.so;
there is no CPU or PyTorch fallback.  If the library is missing the import of
the binding functions fails loudly (call ``compile_library()`` or
``python -m bit_spherical_vector_b200.build``).
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "lib", "libsvq.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "svq.h")

SVQ_OK, SVQ_ERR_INVALID_ARG, SVQ_ERR_UNSUPPORTED_SHAPE, SVQ_ERR_WORKSPACE, SVQ_ERR_CUDA, SVQ_ERR_TIMEOUT = range(6)
SVQ_F16, SVQ_BF16, SVQ_F32 = 1, 2, 3


class SvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({status_string(status)})")
        self.status = status


class svq_matrix(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("b_d", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("packed", ctypes.c_void_p), ("codebook", ctypes.c_void_p),
                ("radius_scale", ctypes.c_void_p), ("radius_offset", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("radius_lut", ctypes.c_void_p)]


class svq_kv_cache(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class svq_rope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("factor", ctypes.c_float), ("reserved", ctypes.c_int32)]


_lib = None


def compile_library(force: bool = False) -> str:
    """Compile libsvq.so in-tree (see bit_spherical_vector_b200/build.py)."""
    import importlib
    return importlib.import_module(__name__ + ".build").build(force=force)


def lib():
    """The loaded libsvq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libsvq.so not found at {LIB_PATH}; build it with "
                          "`python -m bit_spherical_vector_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, SZ, L64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_int64
    MP = ctypes.POINTER(svq_matrix)
    sig = {
        "svq_status_string": ([I], ctypes.c_char_p),
        "svq_version": ([], I),
        "svq_packed_bytes": ([I, I], SZ),
        "svq_canonical_bytes": ([I, I], SZ),
        "svq_repack": ([P, I, I, I, P, P], I),
        "svq_unpack_fields": ([P, I, I, I, P, P, P, P], I),
        "svq_dequantize": ([MP, I, P, P], I),
        "svq_linear_gemv_workspace_size": ([MP, I, ctypes.POINTER(SZ)], I),
        "svq_workspace_init": ([P, SZ, P], I),
        "svq_linear_gemv": ([MP, P, I, P, I, P, SZ, P], I),
        "svq_linear_gemv_batched_workspace_size": ([MP, I, I, ctypes.POINTER(SZ)], I),
        "svq_linear_gemv_batched": ([MP, I, ctypes.POINTER(P), I, ctypes.POINTER(P), I, P, SZ, P], I),
        "svq_linear_gemv_batched_host": ([MP, I, P, P, I, P, P, I, P, SZ, P], I),
        "svq_linear_gemv_noalloc": ([MP, P, I, P, I, P], I),
        "svq_linear_gemm_workspace_size": ([MP, I, ctypes.POINTER(SZ)], I),
        "svq_linear_gemm": ([MP, P, I, I, P, I, P, SZ, P], I),
        "svq_moe_grouped_gemv_workspace_size": ([I, I, I, I, ctypes.POINTER(SZ)], I),
        "svq_debug_set_wait_polls": ([ctypes.c_uint], ctypes.c_uint),
        "svq_moe_grouped_gemv": ([P, I, I, I, I, P, I, I, P, I, I, P, I, I, P, SZ, P], I),
        "svq_rmsnorm_permute": ([P, I, P, ctypes.c_float, I, I, ctypes.POINTER(P), ctypes.POINTER(P), I, P], I),
        "svq_swiglu_permute": ([P, P, I, I, P, P, P], I),
        "svq_kv_assign": ([P, P, I, I, P, I, P, I, P, P, P, P, P, P, I, P], I),
        "svq_rope_frequencies": ([I, ctypes.c_double, I, ctypes.c_double, I, P, P], I),
        "svq_qk_norm_rope_cache": ([P, P, P, I, L64, L64, L64, I, I, P, P, ctypes.c_float, P, P, P, P, P, P], I),
        "svq_paged_attention_workspace_size": ([P, I, ctypes.POINTER(SZ)], I),
        "svq_paged_attention": ([P, I, I, P, P, P, I, P, I, ctypes.c_float, P, P, I, P, P, SZ, P], I),
        "svq_get_device_status": ([P], I),
        "svq_esg": ([P, I, I, ctypes.c_double, P, P, P, P], I),
        "svq_radius_grid": ([P, I, I, P, I, P, P, P], I),
        "svq_encode": ([P, I, I, I, P, P, P, P, P, P, P, P, P], I),
        "svq_abs_select": ([P, I, I, P, P, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def status_string(status: int) -> str:
    try:
        return lib().svq_status_string(int(status)).decode()
    except ImportError:
        return "library not loaded"


def _check(status: int, what: str):
    if status != SVQ_OK:
        raise SvqError(status, what)


def _stream(stream=None):
    """The handle of a torch stream, or of the current one (the raw handle: building a Stream object takes as
    long as a launch, 3.2 us against 0.1 us)."""
    import torch
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


_dtype_codes: dict = {}


def _dtype_code(dtype) -> int:
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.float16: SVQ_F16, torch.bfloat16: SVQ_BF16, torch.float32: SVQ_F32})
    return _dtype_codes[dtype]


# ----------------------------------------------------------------------------- format
def svq_packed_bytes(N: int, K: int) -> int:
    return int(lib().svq_packed_bytes(N, K))


def svq_canonical_bytes(N: int, K: int) -> int:
    return int(lib().svq_canonical_bytes(N, K))


def svq_repack(canonical, N: int, K: int, b_d: int, packed_out, stream=None):
    _check(lib().svq_repack(_ptr(canonical), N, K, b_d, _ptr(packed_out), _stream(stream)), "svq_repack")


def svq_unpack_fields(packed, N: int, K: int, b_d: int, signs, idx, code, stream=None):
    _check(lib().svq_unpack_fields(_ptr(packed), N, K, b_d, _ptr(signs), _ptr(idx), _ptr(code),
                                   _stream(stream)), "svq_unpack_fields")


class SvqWeight:
    """Device-resident SVQ matrix (packed codes, codebook, radius params, perm, optional per-row radius
    table) and its C descriptor.  Built from canonical host arrays by ``from_canonical``.  ``perm``
    None means x is supplied already in the stored column order; ``lut`` (fp16 [N][2^b_r]) replaces the
    affine radius when given."""

    def __init__(self, N, K, b_d, packed, codebook, scale, offset, perm, lut=None):
        self.N, self.K, self.b_d = N, K, b_d
        self.packed, self.codebook, self.scale, self.offset, self.perm = packed, codebook, scale, offset, perm
        self.lut = lut
        ptr = lambda t: 0 if t is None else t.data_ptr()
        self.desc = svq_matrix(N, K, b_d, 0, packed.data_ptr(), codebook.data_ptr(), ptr(scale), ptr(offset),
                               ptr(perm), ptr(lut))

    def without_perm(self):
        """The same device arrays with perm NULL: its calls take x in stored column order."""
        return SvqWeight(self.N, self.K, self.b_d, self.packed, self.codebook, self.scale, self.offset, None,
                         self.lut)

    @classmethod
    def from_canonical(cls, N, K, b_d, canonical, codebook, scale, offset, perm, device="cuda", stream=None,
                       lut=None):
        """canonical/codebook/scale/offset/perm/lut: numpy arrays (uint8 / uint16 bit patterns / int32)."""
        import numpy as np
        import torch
        dev = torch.device(device)
        canon_d = torch.from_numpy(np.ascontiguousarray(canonical, np.uint8)).to(dev)
        packed = torch.empty(svq_packed_bytes(N, K), dtype=torch.uint8, device=dev)
        svq_repack(canon_d, N, K, b_d, packed, stream)
        to16 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.uint16).view(np.int16)).to(dev)
        w = cls(N, K, b_d, packed, to16(codebook), to16(scale), to16(offset),
                torch.from_numpy(np.ascontiguousarray(perm, np.int32)).to(dev),
                None if lut is None else to16(lut))
        w._canon_d = canon_d   # keep alive until the repack has run
        return w

    @classmethod
    def from_synth(cls, m, device="cuda", stream=None):
        return cls.from_canonical(m.N, m.K, m.b_d, m.canonical, m.codebook, m.scale, m.offset, m.perm,
                                  device, stream, getattr(m, "lut", None))


def svq_dequantize(W: SvqWeight, out, stream=None):
    _check(lib().svq_dequantize(ctypes.byref(W.desc), _dtype_code(out.dtype), _ptr(out), _stream(stream)),
           "svq_dequantize")


def svq_linear_gemv_workspace_size(W: SvqWeight, M: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().svq_linear_gemv_workspace_size(ctypes.byref(W.desc), M, ctypes.byref(n)),
           "svq_linear_gemv_workspace_size")
    return int(n.value)


def svq_linear_gemv_batched_workspace_size(Ws, M: int) -> int:
    arr = (svq_matrix * len(Ws))(*[w.desc for w in Ws])
    n = ctypes.c_size_t(0)
    _check(lib().svq_linear_gemv_batched_workspace_size(arr, len(Ws), M, ctypes.byref(n)),
           "svq_linear_gemv_batched_workspace_size")
    return int(n.value)


def svq_workspace_init(ws, stream=None):
    if ws is None or ws.numel() == 0:
        return
    _check(lib().svq_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "svq_workspace_init")


def svq_linear_gemv(W: SvqWeight, x, y, ws=None, stream=None):
    """y[M][N] = W x[M][K]^T with x fp16; y fp16 or fp32."""
    M = x.shape[0]
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().svq_linear_gemv(ctypes.byref(W.desc), _ptr(x), M, _ptr(y), _dtype_code(y.dtype), _ptr(ws), nb,
                                 _stream(stream)), "svq_linear_gemv")


def svq_linear_gemv_batched(Ws, xs, ys, ws=None, stream=None):
    n = len(Ws)
    arr = (svq_matrix * n)(*[w.desc for w in Ws])
    xp = (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs])
    yp = (ctypes.c_void_p * n)(*[y.data_ptr() for y in ys])
    M = xs[0].shape[0]
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().svq_linear_gemv_batched(arr, n, xp, M, yp, _dtype_code(ys[0].dtype), _ptr(ws), nb,
                                         _stream(stream)), "svq_linear_gemv_batched")


class GemvBatchCall:
    """svq_linear_gemv_batched with its arguments marshalled once, for loops that call
    the same layers on the same buffers (one decode step after another)."""

    def __init__(self, Ws, xs, ys, ws=None):
        n = len(Ws)
        self._keep = (list(Ws), list(xs), list(ys), ws)           # the buffers must outlive the calls
        self._args = ((svq_matrix * n)(*[w.desc for w in Ws]), n,
                      (ctypes.c_void_p * n)(*[x.data_ptr() for x in xs]), xs[0].shape[0],
                      (ctypes.c_void_p * n)(*[y.data_ptr() for y in ys]), _dtype_code(ys[0].dtype), _ptr(ws),
                      0 if ws is None else ws.numel() * ws.element_size())
        self._fn = lib().svq_linear_gemv_batched

    def __call__(self, stream=None):
        _check(self._fn(*self._args, _stream(stream)), "svq_linear_gemv_batched")


class GemvBatchHostCall:
    """svq_linear_gemv_batched_host with its arguments marshalled once: each call copies the step's
    inputs x_host (pinned, the inputs back to back) into x_dev, runs the grouped launch and copies
    y_dev (the outputs back to back) into y_host (pinned), all enqueued on the stream."""

    def __init__(self, Ws, M, x_host, x_dev, y_host, y_dev, ws=None):
        n = len(Ws)
        self._keep = (list(Ws), x_host, x_dev, y_host, y_dev, ws)  # the buffers must outlive the calls
        self._args = ((svq_matrix * n)(*[w.desc for w in Ws]), n, _ptr(x_host), _ptr(x_dev), M,
                      _ptr(y_host), _ptr(y_dev), _dtype_code(y_dev.dtype), _ptr(ws),
                      0 if ws is None else ws.numel() * ws.element_size())
        self._fn = lib().svq_linear_gemv_batched_host

    def __call__(self, stream=None):
        _check(self._fn(*self._args, _stream(stream)), "svq_linear_gemv_batched_host")


def svq_linear_gemv_noalloc(W: SvqWeight, x, y, stream=None):
    """svq_linear_gemv with the library's fixed internal scratch (no workspace argument)."""
    M = x.shape[0]
    _check(lib().svq_linear_gemv_noalloc(ctypes.byref(W.desc), _ptr(x), M, _ptr(y), _dtype_code(y.dtype),
                                         _stream(stream)), "svq_linear_gemv_noalloc")


def svq_linear_gemm_workspace_size(W: SvqWeight, M: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().svq_linear_gemm_workspace_size(ctypes.byref(W.desc), M, ctypes.byref(n)),
           "svq_linear_gemm_workspace_size")
    return int(n.value)


def svq_linear_gemm(W: SvqWeight, x, y, ws, stream=None):
    """y[M][N] = W x[M][K]^T on the tensor cores; x bf16 or fp16, y fp32 or bf16."""
    M = x.shape[0]
    nb = ws.numel() * ws.element_size()
    _check(lib().svq_linear_gemm(ctypes.byref(W.desc), _ptr(x), _dtype_code(x.dtype), M, _ptr(y),
                                 _dtype_code(y.dtype), _ptr(ws), nb, _stream(stream)), "svq_linear_gemm")


class svq_group_item(ctypes.Structure):
    _fields_ = [("matrix", ctypes.c_int32), ("x_row", ctypes.c_int32), ("out_row", ctypes.c_int32),
                ("out_scale", ctypes.c_float)]


SVQ_X_F16, SVQ_X_SWIGLU_F32 = 0, 1


def descriptor_table(Ws, device="cuda"):
    """Device array of svq_matrix descriptors (the layout the MoE kernel reads)."""
    import numpy as np
    import torch
    arr = (svq_matrix * len(Ws))(*[w.desc for w in Ws])
    raw = np.frombuffer(bytes(arr), dtype=np.uint8).copy()
    return torch.from_numpy(raw).to(device)


def item_table(matrix, x_row, out_row, out_scale):
    """Device array of svq_group_item from four equal-length device tensors (int32, int32, int32, float32)."""
    import torch
    t = torch.stack([matrix.to(torch.int32), x_row.to(torch.int32), out_row.to(torch.int32),
                     out_scale.to(torch.float32).view(torch.int32)], dim=1).contiguous()
    return t


def svq_moe_grouped_gemv_workspace_size(n_mats: int, n_items: int, N: int, accumulate: bool) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().svq_moe_grouped_gemv_workspace_size(n_mats, n_items, N, int(accumulate), ctypes.byref(n)),
           "svq_moe_grouped_gemv_workspace_size")
    return int(n.value)


def svq_moe_grouped_gemv(mats_dev, n_mats, N, K, max_b_d, items_dev, n_items, max_items_per_matrix, x, x_mode,
                         y, n_out_rows, accumulate, ws, stream=None):
    n_x_rows = int(x.shape[0])                 # items' x_row must lie below (checked on the device)
    _check(lib().svq_moe_grouped_gemv(_ptr(mats_dev), n_mats, N, K, max_b_d, _ptr(items_dev), n_items,
                                      max_items_per_matrix, _ptr(x), x_mode, n_x_rows, _ptr(y), n_out_rows,
                                      int(accumulate), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "svq_moe_grouped_gemv")


# ----------------------------------------------------------------------------- decoder-layer producers
def svq_rmsnorm_permute(h, gamma, eps: float, perms, outs, stream=None):
    """outs[g][m][j] = fp16(rmsnorm(h)[m][perms[g][j]]) (perms[g] None: natural order).
    h: [M][K] fp16/bf16, gamma: fp16 [K], outs: list of fp16 [M][K]."""
    n = len(outs)
    M, K = h.shape
    pp = (ctypes.c_void_p * n)(*[0 if p is None else p.data_ptr() for p in perms])
    op = (ctypes.c_void_p * n)(*[o.data_ptr() for o in outs])
    _check(lib().svq_rmsnorm_permute(_ptr(h), _dtype_code(h.dtype), _ptr(gamma), float(eps), M, K, pp, op, n,
                                     _stream(stream)), "svq_rmsnorm_permute")


def svq_swiglu_permute(gate, up, perm, x, stream=None):
    """x[m][j] = fp16(silu(gate[m][s]) * up[m][s]), s = perm[j] (perm None: s = j); gate/up fp32 [M][I]."""
    M, I = gate.shape
    _check(lib().svq_swiglu_permute(_ptr(gate), _ptr(up), M, I, _ptr(perm), _ptr(x), _stream(stream)),
           "svq_swiglu_permute")


# ------------------------------------------------------------------ attention step (paged cache)
SVQ_ROPE_PLAIN, SVQ_ROPE_LINEAR, SVQ_ROPE_NTK, SVQ_ROPE_YARN = range(4)


def _need(ok: bool, what: str):
    """Shapes, types and devices that the C ABI cannot see behind a pointer."""
    if not ok:
        raise ValueError(what)


# The three calls below are made for every layer of every step, and a short one's kernel takes less time than
# the host does; so their checks are written out, without helpers that would format a message or pack arguments
# each time.
def _wrong(what: str, why: str):
    raise ValueError(f"{what}: {why}")


def _arrays(what: str, dtype, dev: int, tensors):
    """Contiguous arrays of one type on the current device (None: an optional one that is absent)."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous()):
            _wrong(what, f"an array of {dtype} must be contiguous and on the current CUDA device")


class KvCache:
    """A paged key/value cache and its C descriptor: k and v are views [n_pages][page_size][n_heads][head_dim]
    (fp16 or bf16) of the pools, in any order in memory with the head's entries contiguous."""

    def __init__(self, k, v):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.stride() == v.stride(),
              "KvCache: k and v must be alike, [n_pages][page_size][n_heads][head_dim]")
        _need(k.stride(3) == 1, "KvCache: the entries of a head must be contiguous")
        _need(k.get_device() == v.get_device(), "KvCache: k and v must be on one device")
        self.k, self.v, self.dtype, self.device = k, v, k.dtype, k.get_device()
        self.n_pages, self.page_size, self.n_heads, self.head_dim = (int(d) for d in k.shape)
        self.desc = svq_kv_cache(_dtype_code(k.dtype), self.n_pages, self.page_size, self.n_heads, self.head_dim, 0,
                                 k.stride(0), k.stride(1), k.stride(2), k.data_ptr(), v.data_ptr())
        self._ref = ctypes.addressof(self.desc)


class Rope:
    """Rotary positions and their C descriptor: inv_freq (fp64 [rot_dim / 2], radians per position, on the device),
    the pair layout and the factor on rotated entries."""

    def __init__(self, inv_freq, interleaved: bool = False, factor: float = 1.0):
        import torch
        _need(inv_freq.dtype is torch.float64 and inv_freq.dim() == 1 and inv_freq.is_contiguous() and inv_freq.is_cuda,
              "Rope: inv_freq must be a contiguous fp64 vector on the device")
        self.inv_freq, self.interleaved, self.factor = inv_freq, bool(interleaved), float(factor)
        self.rot_dim, self.device = 2 * inv_freq.numel(), inv_freq.get_device()
        self.desc = svq_rope(inv_freq.data_ptr(), self.rot_dim, int(self.interleaved), self.factor, 0)
        self._ref = ctypes.addressof(self.desc)

    @classmethod
    def make(cls, rot_dim: int, base: float, scaling: int = SVQ_ROPE_PLAIN, scale: float = 1.0, trained_len: int = 0,
             interleaved: bool = False, device="cuda"):
        """The frequencies of svq_rope_frequencies, on the device."""
        import torch
        freq, factor = svq_rope_frequencies(rot_dim, base, scaling, scale, trained_len)
        return cls(torch.from_numpy(freq).to(device), interleaved, factor)


def svq_rope_frequencies(rot_dim: int, base: float, scaling: int = SVQ_ROPE_PLAIN, scale: float = 1.0,
                         trained_len: int = 0):
    """Radians per position of each rotated pair (numpy fp64 [rot_dim / 2]) and the factor on rotated entries."""
    import numpy as np
    freq, factor = np.empty(max(rot_dim // 2, 1), np.float64), ctypes.c_float(0)
    _check(lib().svq_rope_frequencies(rot_dim, float(base), scaling, float(scale), trained_len, freq.ctypes.data,
                                      ctypes.addressof(factor)), "svq_rope_frequencies")
    return freq, float(factor.value)


def svq_kv_assign(lens, n_new, page_size: int, block_table, free_pages, n_free, lens_out, n_free_out, cu_rows,
                  positions, slots, stream=None):
    """Block table, positions and slots of one step from the requests' lengths: request b holds lens[b] tokens and
    gets n_new[b] (negative: it is done).  All int32 on the device; lens_out may be lens, n_free_out may be n_free."""
    import torch
    n, rows = lens.numel(), slots.numel()
    dev = torch._C._cuda_getDevice()
    _arrays("svq_kv_assign", torch.int32, dev, (lens, n_new, block_table, free_pages, n_free, lens_out, n_free_out,
                                                cu_rows, positions, slots))
    if block_table.dim() != 2:
        _wrong("svq_kv_assign", "block_table must be [n_seqs][max_pages]")
    n_table, width = block_table.shape
    if not (n_table == n == n_new.numel() == lens_out.numel() == cu_rows.numel() - 1 and positions.numel() == rows
            and n_free.numel() == 1 == n_free_out.numel()):
        _wrong("svq_kv_assign", "sizes do not agree")
    st = lib().svq_kv_assign(
        lens.data_ptr(), n_new.data_ptr(), n, page_size, block_table.data_ptr(), width, free_pages.data_ptr(),
        free_pages.numel(), n_free.data_ptr(), lens_out.data_ptr(), n_free_out.data_ptr(), cu_rows.data_ptr(),
        positions.data_ptr(), slots.data_ptr(), rows,
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise SvqError(st, "svq_kv_assign")


def svq_qk_norm_rope_cache(q, k, v, q_gamma, k_gamma, eps: float, rope: Rope, positions, slots, cache: KvCache, q_out,
                           stream=None):
    """q [M][n_q * D], k and v [M][n_heads * D] (fp32, fp16 or bf16, rows any multiple of 8 apart) -> q_out
    [M][n_q][D] and the cache's slots; gammas fp16 [D] or None; rows with a negative slot are left out."""
    import torch
    D, wk, x = cache.head_dim, cache.n_heads * cache.head_dim, q.dtype
    (M, wq), (Mk, wkk), (Mv, wkv), (Mo, heads, Do) = q.shape, k.shape, v.shape, q_out.shape
    if not (Mk == Mv == Mo == M == positions.numel() == slots.numel() and wq == heads * D and wkk == wkv == wk
            and Do == D and (q_gamma is None or q_gamma.numel() == D) and (k_gamma is None or k_gamma.numel() == D)):
        _wrong("svq_qk_norm_rope_cache", "sizes do not agree")
    (ldq, sq), (ldk, sk), (ldv, sv) = q.stride(), k.stride(), v.stride()
    if k.dtype is not x or v.dtype is not x or (M and not sq == sk == sv == 1):
        _wrong("svq_qk_norm_rope_cache", "types or strides do not agree")
    if M < 2:                                    # the distance between rows of one row says nothing
        ldq, ldk, ldv = wq, wk, wk
    dev = torch._C._cuda_getDevice()
    if not (q.get_device() == k.get_device() == v.get_device() == rope.device == cache.device == dev):
        _wrong("svq_qk_norm_rope_cache", "not on the current CUDA device")
    _arrays("svq_qk_norm_rope_cache", torch.int32, dev, (positions, slots))
    _arrays("svq_qk_norm_rope_cache", torch.float16, dev, (q_gamma, k_gamma))
    _arrays("svq_qk_norm_rope_cache", cache.dtype, dev, (q_out,))
    st = lib().svq_qk_norm_rope_cache(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(x), ldq, ldk, ldv, M, heads,
        None if q_gamma is None else q_gamma.data_ptr(), None if k_gamma is None else k_gamma.data_ptr(), eps, rope._ref,
        positions.data_ptr(), slots.data_ptr(), cache._ref, q_out.data_ptr(),
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise SvqError(st, "svq_qk_norm_rope_cache")


def svq_paged_attention_workspace_size(cache: KvCache, n_q_heads: int) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().svq_paged_attention_workspace_size(cache._ref, n_q_heads, ctypes.byref(n)),
           "svq_paged_attention_workspace_size")
    return int(n.value)


def svq_paged_attention(q, cache: KvCache, lens, block_table, scale: float, out, ws, cu_rows=None, order=None,
                        lse=None, stream=None):
    """out [rows][n_q * D] (fp16 or bf16) = attention of q [rows][n_q][D] over the first lens[b] tokens of request b
    (row b, or row cu_rows[b + 1] - 1).  order (int32 [n_q * D]): column of each entry, the inverse of the o
    matrix's perm for its stored order; lse: fp32 [rows][n_q] or None.  ws: zero-filled once by svq_workspace_init."""
    import torch
    rows, heads, D = q.shape
    n = lens.numel()
    if block_table.dim() != 2:
        _wrong("svq_paged_attention", "block_table must be [n_seqs][max_pages]")
    n_table, width = block_table.shape
    if not (D == cache.head_dim and out.shape == (rows, heads * D) and n_table == n
            and (cu_rows.numel() == n + 1 if cu_rows is not None else n <= rows)
            and (order is None or order.numel() == heads * D) and (lse is None or lse.shape == (rows, heads))):
        _wrong("svq_paged_attention", "sizes do not agree")
    dev = torch._C._cuda_getDevice()
    if cache.device != dev:
        _wrong("svq_paged_attention", "not on the current CUDA device")
    _arrays("svq_paged_attention", torch.int32, dev, (lens, block_table, cu_rows, order))
    _arrays("svq_paged_attention", cache.dtype, dev, (q,))
    _arrays("svq_paged_attention", out.dtype, dev, (out,))
    _arrays("svq_paged_attention", ws.dtype, dev, (ws,))
    if lse is not None:
        _arrays("svq_paged_attention", torch.float32, dev, (lse,))
    st = lib().svq_paged_attention(
        q.data_ptr(), rows, heads, cache._ref, lens.data_ptr(), None if cu_rows is None else cu_rows.data_ptr(), n,
        block_table.data_ptr(), width, scale, None if order is None else order.data_ptr(), out.data_ptr(),
        _dtype_code(out.dtype), None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.nbytes,
        torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise SvqError(st, "svq_paged_attention")


# ------------------------------------------------------------------ calibration (ESG, radius grid, encoder, ABS)
def svq_esg(x_cal, gamma, energy, perm, weights=None, stream=None):
    """Channel energies (fp64 [K]), the ESG permutation (int32 [K]) and fitting weights e^gamma (fp32 [K] or None)
    from calibration activations x_cal (fp32 [T][K])."""
    T, K = x_cal.shape
    _check(lib().svq_esg(_ptr(x_cal), T, K, float(gamma), _ptr(energy), _ptr(perm), _ptr(weights), _stream(stream)),
           "svq_esg")


def svq_radius_grid(W, perm, b_d, scale, offset, stream=None):
    """Per-row uniform radius grid (fp16 bit patterns scale/offset [N], as int16/uint16 tensors) of W (fp32 [N][K])."""
    N, K = W.shape
    _check(lib().svq_radius_grid(_ptr(W), N, K, _ptr(perm), int(b_d), _ptr(scale), _ptr(offset), _stream(stream)),
           "svq_radius_grid")


def svq_encode(W, b_d, perm, weights, codebook, scale, offset, canonical, row_err=None, stream=None, lut=None):
    """Activation-weighted SVQ encoding of W (fp32 [N][K], natural column order) into the canonical stream
    (uint8 [N][row_bytes]); row_err (fp64 [N]) receives each row's weighted reconstruction error.  lut
    (fp16 [N][2^b_r]) gives per-row radius levels in place of scale/offset."""
    N, K = W.shape
    _check(lib().svq_encode(_ptr(W), N, K, int(b_d), _ptr(perm), _ptr(weights), _ptr(codebook), _ptr(scale),
                            _ptr(offset), _ptr(lut), _ptr(canonical), _ptr(row_err), _stream(stream)), "svq_encode")


def svq_abs_select(row_err, totals, best, stream=None):
    """ABS: totals[k] = sum of row_err[k] (fp64 [n_cand][N]) and best[0] = the first least total (int32)."""
    n_cand, N = row_err.shape
    _check(lib().svq_abs_select(_ptr(row_err), n_cand, N, _ptr(totals), _ptr(best), _stream(stream)),
           "svq_abs_select")


def svq_get_device_status(stream=None) -> int:
    return int(lib().svq_get_device_status(_stream(stream)))


def svq_debug_set_wait_polls(polls: int) -> int:
    """Poll bound of the GEMM's bounded waits for later launches (tests); returns the previous bound."""
    return int(lib().svq_debug_set_wait_polls(int(polls)))


def header_functions() -> list[str]:
    """Names of the functions declared in include/svq.h."""
    import re
    with open(HEADER) as f:
        src = f.read()
    return sorted(set(re.findall(r"SVQ_API\s+[\w\s\*]+?\b(svq_\w+)\s*\(", src)))
