"""MI355X-native weight-only group-quantized decode GEMM.

Python binding of libwq.so (C ABI in include/wq.h).  This layer only turns
torch tensors and the current HIP stream into raw pointers; every step of the
computation runs in the HIP kernels, and there is no CPU fallback: if the
library is not built, the calls raise.

    codes, scales, zeros = quantize_pack(W, group=128, bits=4)   # W fp16 [N, K] on the GPU
    Y = gemm(X, codes, scales, zeros, N=N, K=K, group=128, bits=4)  # X fp16 [B, K]
"""

from __future__ import annotations

import math
from operator import attrgetter

from . import roofline  # noqa: F401  (pure arithmetic, no GPU)
from ._lib import (WQ_PATH_AUTO, WQ_PATH_GEMV, WQ_PATH_MFMA, WQError,  # noqa: F401
                   LIB_PATH, check, load)

__all__ = ["quantize_pack", "gemm", "gemm_grouped", "gemm_workspace_bytes", "codes_bytes", "num_groups",
           "gemv_max_batch",
           "gemm_nf4", "gemm_offset", "KVCache", "kv_quantize_block", "kv_attention",
           "rope", "rope_frequencies", "PagedKV", "kv_paged_append", "kv_paged_attention", "kv_paged_workspace",
           "kv_paged_copy", "kv_paged_fork", "kv_paged_compact", "kv_paged_compact_workspace",
           "WQError", "LIB_PATH", "load"]

_PATHS = {"auto": WQ_PATH_AUTO, "gemv": WQ_PATH_GEMV, "mfma": WQ_PATH_MFMA}


def _stream_handle(device):
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _size_t(query, *args, where=""):
    """Bytes from a wq_*_workspace_size query (raises on its error status)."""
    import ctypes
    n = ctypes.c_size_t(0)
    check(query(*args, ctypes.byref(n)), where)
    return int(n.value)


def _workspace(nbytes, device, workspace=None):
    """(pointer, bytes, tensor) of a caller workspace: the given uint8 tensor
    (checked against nbytes) or a fresh one from torch's allocator, (None, 0,
    None) when the call needs none.  A fresh tensor goes back to torch's stream-ordered cache
    when the caller drops it, so reuse by later work on the stream is safe."""
    import torch
    if nbytes == 0:
        return None, 0, None
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif (not isinstance(workspace, torch.Tensor) or workspace.device != torch.device(device)
          or workspace.dtype != torch.uint8 or not workspace.is_contiguous()
          or workspace.numel() < nbytes):
        raise ValueError(f"workspace must be a contiguous uint8 tensor of >= {nbytes} bytes on {device}")
    return workspace.data_ptr(), workspace.numel(), workspace


def _need(t, dtype, shape, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def codes_bytes(N: int, K: int, bits: int) -> int:
    return int(load().wq_codes_bytes(N, K, bits))


def num_groups(N: int, K: int, group: int) -> int:
    return int(load().wq_num_groups(N, K, group))


def gemv_max_batch() -> int:
    return int(load().wq_gemv_max_batch())


def gemm_workspace_bytes(B: int, K: int, N: int, group: int = 128, bits: int = 4, path: str = "auto") -> int:
    """Workspace bytes of a gemm() call of this shape on the current device."""
    return _size_t(load().wq_gemm_workspace_size, B, K, N, group, bits, _PATHS[path], where="wq_gemm")


SCHEMES = {"asym": 0, "sym": 1, "sym_tensor": 2, "nf4": 3, "offset": 4}


def quantize_pack(W, group: int = 128, bits: int = 4, out=None, scheme: str = "asym"):
    """W fp16 [N, K] (GPU) -> (codes u8 [N, K*bits//8], scales fp16 [N, K//group], zeros fp16).

    scheme "asym" (min/max, integer zero point), "sym" (absolute maximum per
    group; group = K for one scale per output channel), "sym_tensor" (one
    absolute maximum for the whole matrix), "nf4" (normal-quantile levels,
    bits = 4; multiply with gemm_nf4) or "offset" (the group minimum as a
    float offset in the third array; multiply with gemm_offset)."""
    import torch
    lib = load()
    if scheme not in SCHEMES:
        raise ValueError(f"unknown scheme {scheme!r}")
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N, K]")
    N, K = W.shape
    _need(W, torch.float16, (N, K), "W")
    if K % group or (K * bits) % 8:
        raise ValueError("K must be a multiple of group and of 8/bits")
    if out is None:
        codes = torch.empty((N, K * bits // 8), dtype=torch.uint8, device=W.device)
        scales = torch.empty((N, K // group), dtype=torch.float16, device=W.device)
        zeros = torch.empty((N, K // group), dtype=torch.float16, device=W.device)
    else:
        codes, scales, zeros = out
        _need(codes, torch.uint8, (N, K * bits // 8), "codes")
        _need(scales, torch.float16, (N, K // group), "scales")
        _need(zeros, torch.float16, (N, K // group), "zeros")
    with torch.cuda.device(W.device):
        need = _size_t(lib.wq_quantize_workspace_size, N, K, group, bits, SCHEMES[scheme],
                       where="wq_quantize_pack")
        ws, ws_bytes, _keep = _workspace(need, W.device)
        st = lib.wq_quantize_pack_ex(W.data_ptr(), N, K, group, bits, SCHEMES[scheme],
                                     codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                                     ws, ws_bytes, _stream_handle(W.device))
    check(st, "wq_quantize_pack")
    return codes, scales, zeros


def gemm_grouped(items, workspace=None, use_workspace=True):
    """Several products in one call: items is a sequence of
    (X, codes, scales, zeros, N, K, group, bits[, out]) tuples; returns the Y
    tensors in order (each what gemm() gives for its item, within the product
    tolerance).  The call's workspace comes from torch (or `workspace`, a
    uint8 tensor); use_workspace=False runs the plans that need none."""
    import ctypes
    import torch
    from ._lib import GemmItem
    lib = load()
    arr = (GemmItem * max(len(items), 1))()
    outs = []
    dev = None
    for i, it in enumerate(items):
        X, codes, scales, zeros, N, K, group, bits = it[:8]
        out = it[8] if len(it) > 8 else None
        if X.dim() != 2:
            raise ValueError("X must be 2-D [B, K]")
        B = X.shape[0]
        _need(X, torch.float16, (B, K), "X")
        _need(codes, torch.uint8, (N, K * bits // 8), "codes")
        _need(scales, torch.float16, (N, K // group), "scales")
        _need(zeros, torch.float16, (N, K // group), "zeros")
        if dev is None:
            dev = X.device
        elif X.device != dev:
            raise ValueError("all items must be on one device")
        if out is None:
            out = torch.empty((B, N), dtype=torch.float16, device=X.device)
        else:
            _need(out, torch.float16, (B, N), "out")
        outs.append(out)
        arr[i] = GemmItem(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                          out.data_ptr(), B, K, N, group, bits)
    if not items:
        return outs
    with torch.cuda.device(dev):
        need = _size_t(lib.wq_gemm_grouped_workspace_size, arr, len(items),
                       where="wq_gemm_grouped") if use_workspace else 0
        ws, ws_bytes, _keep = _workspace(need, dev, workspace)
        st = lib.wq_gemm_grouped(arr, len(items), ws, ws_bytes, _stream_handle(dev))
    check(st, "wq_gemm_grouped")
    return outs


def gemm(X, codes, scales, zeros, N: int, K: int, group: int = 128, bits: int = 4,
         path: str = "auto", out=None, workspace=None, use_workspace=True):
    """Y fp16 [B, N] = X fp16 [B, K] times the dequantized [N, K] matrix, transposed.

    The call's workspace (wq_gemm_workspace_size bytes) comes from torch, or
    from `workspace` (a uint8 tensor); use_workspace=False runs the plan that
    needs none (wq_gemm's)."""
    import torch
    lib = load()
    if X.dim() != 2:
        raise ValueError("X must be 2-D [B, K]")
    B = X.shape[0]
    _need(X, torch.float16, (B, K), "X")
    _need(codes, torch.uint8, (N, K * bits // 8), "codes")
    _need(scales, torch.float16, (N, K // group), "scales")
    _need(zeros, torch.float16, (N, K // group), "zeros")
    if out is None:
        out = torch.empty((B, N), dtype=torch.float16, device=X.device)
    else:
        _need(out, torch.float16, (B, N), "out")
    with torch.cuda.device(X.device):
        need = _size_t(lib.wq_gemm_workspace_size, B, K, N, group, bits, _PATHS[path],
                       where="wq_gemm") if use_workspace else 0
        ws, ws_bytes, _keep = _workspace(need, X.device, workspace)
        st = lib.wq_gemm_ex(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
                            out.data_ptr(), B, K, N, group, bits, _PATHS[path], ws, ws_bytes,
                            _stream_handle(X.device))
    check(st, "wq_gemm")
    return out


class KVCache:
    """Caller-owned buffers of an int4 KV cache (head dimension 128, blocks of
    128 tokens), as torch tensors on one GPU; layout as wq_kv_cache in wq.h."""

    D = 128
    G = 128

    def __init__(self, heads: int, max_blocks: int, device="cuda"):
        import torch
        u8, f16 = torch.uint8, torch.float16
        H, NB, D, G = heads, max_blocks, self.D, self.G
        self.heads, self.max_blocks = heads, max_blocks
        self.kcodes = torch.zeros((H, NB, G, D // 2), dtype=u8, device=device)
        self.kscales = torch.zeros((H, NB, D), dtype=f16, device=device)
        self.kzeros = torch.zeros((H, NB, D), dtype=f16, device=device)
        self.vcodes = torch.zeros((H, NB, D, G // 2), dtype=u8, device=device)
        self.vscales = torch.zeros((H, NB * G), dtype=f16, device=device)
        self.vzeros = torch.zeros((H, NB * G), dtype=f16, device=device)
        self.kres = torch.zeros((H, G, D), dtype=f16, device=device)
        self.vres = torch.zeros((H, G, D), dtype=f16, device=device)

    @property
    def device(self):
        return self.kcodes.device

    def descriptor(self):
        from ._lib import KvCache
        return KvCache(self.kcodes.data_ptr(), self.kscales.data_ptr(), self.kzeros.data_ptr(),
                       self.vcodes.data_ptr(), self.vscales.data_ptr(), self.vzeros.data_ptr(),
                       self.kres.data_ptr(), self.vres.data_ptr(), self.heads, self.max_blocks)


def kv_quantize_block(K, V, cache: KVCache, block: int):
    """K, V fp16 [heads, 128, 128] (token-major) -> block `block` of every head."""
    import ctypes
    import torch
    shape = (cache.heads, cache.G, cache.D)
    _need(K, torch.float16, shape, "K")
    _need(V, torch.float16, shape, "V")
    desc = cache.descriptor()
    with torch.cuda.device(cache.device):
        st = load().wq_kv_quantize_block(K.data_ptr(), V.data_ptr(), ctypes.byref(desc), block,
                                         _stream_handle(cache.device))
    check(st, "wq_kv_quantize_block")


def kv_attention(q, cache: KVCache, lens, out=None, workspace=None, use_workspace=True):
    """q fp16 [heads, 128], lens int32 [heads] (GPU) -> out fp16 [heads, 128].
    The call's workspace (context-split partials) comes from torch or from
    `workspace`; use_workspace=False runs one workgroup per head."""
    import ctypes
    import torch
    _need(q, torch.float16, (cache.heads, cache.D), "q")
    _need(lens, torch.int32, (cache.heads,), "lens")
    if out is None:
        out = torch.empty((cache.heads, cache.D), dtype=torch.float16, device=q.device)
    _need(out, torch.float16, (cache.heads, cache.D), "out")
    desc = cache.descriptor()
    lib = load()
    with torch.cuda.device(cache.device):
        need = _size_t(lib.wq_kv_workspace_size, ctypes.byref(desc), where="wq_kv_attention") \
            if use_workspace else 0
        ws, ws_bytes, _keep = _workspace(need, cache.device, workspace)
        st = lib.wq_kv_attention(q.data_ptr(), ctypes.byref(desc), lens.data_ptr(), out.data_ptr(),
                                 ws, ws_bytes, _stream_handle(cache.device))
    check(st, "wq_kv_attention")
    return out


def gemm_nf4(X, codes, scales, N: int, K: int, group: int = 64, out=None):
    """Y fp16 [B, N] = X [B, K] times the NF4 weights (codes, scales from
    quantize_pack(..., scheme="nf4"))."""
    import torch
    if X.dim() != 2:
        raise ValueError("X must be 2-D [B, K]")
    B = X.shape[0]
    _need(X, torch.float16, (B, K), "X")
    _need(codes, torch.uint8, (N, K // 2), "codes")
    _need(scales, torch.float16, (N, K // group), "scales")
    if out is None:
        out = torch.empty((B, N), dtype=torch.float16, device=X.device)
    _need(out, torch.float16, (B, N), "out")
    with torch.cuda.device(X.device):
        st = load().wq_gemm_nf4(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), out.data_ptr(),
                                B, K, N, group, _stream_handle(X.device))
    check(st, "wq_gemm_nf4")
    return out


def gemm_offset(X, codes, scales, mins, N: int, K: int, group: int = 128, bits: int = 4, out=None):
    """Y fp16 [B, N] for float-offset weights (quantize_pack(..., scheme="offset"))."""
    import torch
    if X.dim() != 2:
        raise ValueError("X must be 2-D [B, K]")
    B = X.shape[0]
    _need(X, torch.float16, (B, K), "X")
    _need(codes, torch.uint8, (N, K * bits // 8), "codes")
    _need(scales, torch.float16, (N, K // group), "scales")
    _need(mins, torch.float16, (N, K // group), "mins")
    if out is None:
        out = torch.empty((B, N), dtype=torch.float16, device=X.device)
    _need(out, torch.float16, (B, N), "out")
    with torch.cuda.device(X.device):
        st = load().wq_gemm_offset(X.data_ptr(), codes.data_ptr(), scales.data_ptr(), mins.data_ptr(),
                                   out.data_ptr(), B, K, N, group, bits, _stream_handle(X.device))
    check(st, "wq_gemm_offset")
    return out


def dequantize(codes, scales, zeros, N: int, K: int, group: int = 128, bits: int = 4,
               scheme: str = "asym", out=None):
    """fp32 [N, K] weights reconstructed from quantize_pack(..., scheme) output
    (a test aid: the products reconstruct in registers)."""
    import torch
    if scheme not in SCHEMES:
        raise ValueError(f"unknown scheme {scheme!r}")
    _need(codes, torch.uint8, (N, K * bits // 8), "codes")
    _need(scales, torch.float16, (N, K // group), "scales")
    _need(zeros, torch.float16, (N, K // group), "zeros")
    if out is None:
        out = torch.empty((N, K), dtype=torch.float32, device=codes.device)
    _need(out, torch.float32, (N, K), "out")
    with torch.cuda.device(codes.device):
        st = load().wq_dequantize(codes.data_ptr(), scales.data_ptr(), zeros.data_ptr(), N, K, group,
                                  bits, SCHEMES[scheme], out.data_ptr(), _stream_handle(codes.device))
    check(st, "wq_dequantize")
    return out


# ---- rotary positions -----------------------------------------------------------

ROPE_LAYOUTS = {"half": 0, "interleaved": 1}


def _raw_stream(index):
    """Handle of the current stream of GPU `index`.  (torch's own call for it
    costs 0.1 us, a Stream object 2.8 us: more than a launch.)"""
    import torch
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return get(index) if get is not None else torch.cuda.current_stream(index).cuda_stream


def _launch(where, device, fn, *args):
    """fn(*args, stream) on `device` and its current stream."""
    import torch
    index = device.index
    if torch.cuda.current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            st = fn(*args, _raw_stream(index))
    if st:
        check(st, where)


def _gpu(t, dtype, name, device=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _line(t, dtype, n, name, device):
    """A contiguous 1-D tensor of n values (n None: any number)."""
    _gpu(t, dtype, name, device)
    if t.dim() != 1 or (n is not None and t.shape[0] != n) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D tensor" + (f" of {n}" if n is not None else "")
                         + f", got shape {tuple(t.shape)}")


def _rows_meet(a, b):
    """Whether [T, H, D] tensors a and b (last stride 1) share memory, told from
    their extents: rows of one token stride that lie side by side are apart, and
    so are heads that lie side by side at every multiple of all strides' common
    divisor."""
    size = a.element_size()
    extent = lambda t: sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1  # noqa: E731
    ea, eb = extent(a), extent(b)
    d = (b.data_ptr() - a.data_ptr()) / size
    if d >= ea or -d >= eb:
        return False
    step = a.stride(0)
    if step == b.stride(0) and step > 0:
        ra, rb = (1 + (t.shape[1] - 1) * t.stride(1) + t.shape[2] - 1 for t in (a, b))
        if ra <= d % step <= step - rb:
            return False
    step = math.gcd(*(s for t in (a, b) for n, s in zip(t.shape[:2], t.stride()) if n > 1))
    return not (step > 0 and a.shape[2] <= d % step <= step - b.shape[2])


def rope_frequencies(rot: int, base: float = 10000.0, kind: str = "none", factor: float = 1.0, context: int = 4096,
                     low: float = 1.0, high: float = 32.0, device="cuda"):
    """float64 [rot / 2]: radians per token of each pair, base^(-2j / rot), for a
    context stretched by `factor`:
      "none"    as they are
      "linear"  all divided by factor
      "base"    base multiplied by factor^(rot / (rot - 2)), which divides the
                slowest pair by factor and leaves the fastest
      "parts"   pairs that turn less than `low` times within `context` tokens
                divided by factor, those of more than `high` turns left, those
                between going over linearly in their turns."""
    import torch
    if rot < 0 or rot % 2 or base <= 0 or factor <= 0 or kind not in ("none", "linear", "base", "parts"):
        raise ValueError(f"rope_frequencies: need even rot >= 0, base > 0, factor > 0 and a known kind (rot={rot} "
                         f"kind={kind!r})")
    if kind == "parts" and not (context > 0 and low < high):
        raise ValueError(f"rope_frequencies: need context > 0 and low < high (context={context} low={low} high={high})")
    if kind == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    if kind == "linear":
        f = f / factor
    elif kind == "parts":
        keep = ((context * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f.to(device)


def rope(x, positions, freqs, layout: str = "half", scale: float = 1.0, out=None):
    """Rotary positions: fp16 [tokens, heads, dim] x with every pair of the first
    2 * len(freqs) channels turned by positions[token] * freqs[pair] radians
    (int32 positions, float64 freqs) and multiplied by scale; further channels
    are copied.  layout "half" pairs channels j and j + rot / 2, "interleaved"
    2j and 2j + 1.  x may be a strided part of a packed row (last stride 1).
    out: a tensor of x's shape, x itself for in place, or None for a new one."""
    import torch
    f16 = torch.float16
    _gpu(x, f16, "x")
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"unknown layout {layout!r}")
    if x.dim() != 3 or (x.shape[2] > 1 and x.stride(2) != 1):
        raise ValueError("x must be [tokens, heads, dim] with contiguous channels")
    T, H, dim = x.shape
    dev = x.device
    _line(positions, torch.int32, T, "positions", dev)
    _line(freqs, torch.float64, None, "freqs", dev)
    if out is None:
        out = torch.empty((T, H, dim), dtype=f16, device=dev)
    elif out is not x:
        _gpu(out, f16, "out", dev)
        if out.shape != x.shape or (dim > 1 and out.stride(2) != 1):
            raise ValueError("out must have x's shape and contiguous channels")
        if x.numel() and not (out.data_ptr() == x.data_ptr() and out.stride() == x.stride()) and _rows_meet(x, out):
            raise ValueError("out overlaps x: only in place, with x's strides")
    xs, os_ = x.stride(), out.stride()
    _launch("wq_rope", dev, load().wq_rope, x.data_ptr(), T, H, dim, xs[0], xs[1], positions.data_ptr(),
            freqs.data_ptr(), 2 * freqs.shape[0], ROPE_LAYOUTS[layout], scale, out.data_ptr(), os_[0], os_[1])
    return out


# ---- paged KV cache ---------------------------------------------------------------

class PagedKV:
    """Caller-owned buffers of one layer's paged int4 KV cache, as torch tensors
    on one GPU; layout as wq_kv_paged in wq.h.  Either new, zeroed buffers of the
    given sizes, or existing ones: pages u8 [num_pages, heads, 17408], windows
    fp16 [slots, heads, 2, 128, 128], table int32 [slots, max_pages].  The three
    may be set anew (pages of any number, windows and table of the same slots);
    the sizes follow them and cannot be set.

        cache = PagedKV(heads=8, num_pages=4096, slots=64, max_pages=256)
        cache.table[slot, block] = page        # which page a block will get
        lens += 1                              # int32 [slots], after the append
        kv_paged_append(k, v, cache, lens)     # the step's k (rotated) and v
        out = kv_paged_attention(q, cache, lens)"""

    D = 128
    G = 128
    RECORD = 17408

    def __init__(self, heads=None, num_pages=None, slots=None, max_pages=None, device="cuda", *, pages=None,
                 windows=None, table=None):
        import torch
        if pages is None:
            pages = torch.zeros((num_pages, heads, self.RECORD), dtype=torch.uint8, device=device)
        if windows is None:
            windows = torch.zeros((slots, pages.shape[1], 2, self.G, self.D), dtype=torch.float16, device=pages.device)
        if table is None:
            table = torch.full((windows.shape[0], max_pages), -1, dtype=torch.int32, device=pages.device)
        _gpu(pages, torch.uint8, "pages")
        self._pages = self._windows = self._table = None
        self._device = pages.device
        self.pages = pages
        self.windows = windows
        self.table = table

    @property
    def pages(self):
        return self._pages

    @pages.setter
    def pages(self, pages):
        import torch
        _gpu(pages, torch.uint8, "pages", self._device)
        if pages.dim() != 3 or pages.shape[2] != self.RECORD or not pages.is_contiguous():
            raise ValueError(f"pages must be contiguous [num_pages, heads, {self.RECORD}], got {tuple(pages.shape)}")
        if self._windows is not None and pages.shape[1] != self.heads:
            raise ValueError(f"pages must be of {self.heads} heads, got {pages.shape[1]}")
        self._pages = pages
        self._num_pages, self._heads = pages.shape[:2]
        self._describe()

    @property
    def windows(self):
        return self._windows

    @windows.setter
    def windows(self, windows):
        import torch
        _gpu(windows, torch.float16, "windows", self._device)
        if (windows.dim() != 5 or tuple(windows.shape[1:]) != (self.heads, 2, self.G, self.D)
                or not windows.is_contiguous()):
            raise ValueError(f"windows must be contiguous [slots, {self.heads}, 2, {self.G}, {self.D}], "
                             f"got {tuple(windows.shape)}")
        if self._table is not None and windows.shape[0] != self.slots:
            raise ValueError(f"windows must be of {self.slots} slots, got {windows.shape[0]}")
        self._windows, self._slots = windows, windows.shape[0]
        self._describe()

    @property
    def table(self):
        return self._table

    @table.setter
    def table(self, table):
        import torch
        _gpu(table, torch.int32, "table", self._device)
        if table.dim() != 2 or table.shape[0] != self.slots or not table.is_contiguous():
            raise ValueError(f"table must be contiguous [{self.slots}, max_pages], got {tuple(table.shape)}")
        self._table, self._max_pages = table, table.shape[1]
        self._describe()

    # (attrgetter: a call of one token asks for these often enough to count)
    device = property(attrgetter("_device"))
    num_pages = property(attrgetter("_num_pages"))
    heads = property(attrgetter("_heads"))
    slots = property(attrgetter("_slots"))
    max_pages = property(attrgetter("_max_pages"))

    def _describe(self):
        import ctypes
        from ._lib import KvPaged
        if self._table is None:            # (still in __init__)
            return
        self._desc = KvPaged(self._pages.data_ptr(), self._windows.data_ptr(), self._table.data_ptr(), self.heads,
                             self.num_pages, self.slots, self.max_pages)
        self._ref = ctypes.byref(self._desc)

    def descriptor(self):
        return self._desc


def _batch(cache, lens, seqs, count):
    """Checks a call's lens and seqs; returns (seqs pointer, entries)."""
    import torch
    _line(lens, torch.int32, cache.slots, "lens", cache.device)
    if seqs is None:
        return None, count
    _line(seqs, torch.int32, count, "seqs", cache.device)
    return seqs.data_ptr(), seqs.shape[0]


def _heads_rows(t, heads, name, device):
    """Checks fp16 [rows, heads, 128] with a row's heads contiguous; returns its
    row stride (heads None: any number)."""
    import torch
    _gpu(t, torch.float16, name, device)
    if t.dim() != 3 or t.shape[2] != 128 or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [rows, {heads if heads is not None else 'heads'}, 128], got {tuple(t.shape)}")
    n, h, _ = t.shape
    st = t.stride()
    if t.numel() and (st[2] != 1 or (h > 1 and st[1] != 128)):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return st[0] if n > 1 else h * 128


def kv_paged_append(k, v, cache: PagedKV, lens, seqs=None, cu=None):
    """Append new tokens: k, v fp16 [tokens, heads, 128] (rows may be strided
    parts of a packed row).  lens int32 [slots]: tokens held AFTER the append.
    seqs int32 [entries]: the slots of the entries (None: 0, 1, ..); cu int32
    [entries + 1]: entry i brings tokens cu[i] .. cu[i + 1] - 1 (None: one
    token each).  Blocks that become whole are quantized into the pages that
    cache.table names; see wq_kv_paged_append in wq.h for what is left out."""
    import torch
    ks = _heads_rows(k, cache.heads, "k", cache.device)
    vs = _heads_rows(v, cache.heads, "v", cache.device)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError(f"k and v must have equally many tokens, got {T} and {v.shape[0]}")
    if cu is None:
        sp, n = _batch(cache, lens, seqs, T)
        cp = None
    else:
        _line(cu, torch.int32, None, "cu", cache.device)
        if cu.shape[0] < 1:
            raise ValueError("cu must hold one value more than there are entries")
        sp, n = _batch(cache, lens, seqs, cu.shape[0] - 1)
        cp = cu.data_ptr()
    _launch("wq_kv_paged_append", cache.device, load().wq_kv_paged_append, k.data_ptr(), v.data_ptr(), T, ks, vs,
            cache._ref, lens.data_ptr(), sp, cp, n)


def kv_paged_workspace(cache: PagedKV, count: int, q_heads: int):
    """A workspace tensor for kv_paged_attention calls of this shape that do not
    overlap (uint8, possibly empty)."""
    import torch
    with torch.cuda.device(cache.device):
        need = _size_t(load().wq_kv_paged_workspace_size, cache._ref, count, q_heads, where="wq_kv_paged_attention")
    return torch.empty(need, dtype=torch.uint8, device=cache.device)


def _given(workspace, device):
    """(pointer, bytes) of a caller's workspace tensor (its size is checked by the call)."""
    import torch
    if (not isinstance(workspace, torch.Tensor) or workspace.device != device or workspace.dtype != torch.uint8
            or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    n = workspace.numel()
    return (workspace.data_ptr(), n) if n else (None, 0)


def kv_paged_attention(q, cache: PagedKV, lens, seqs=None, window: int = 0, scale=None, out=None, workspace=None,
                       use_workspace=True):
    """Decode attention of one new token per entry: q fp16 [entries, q_heads, 128]
    (rows may be strided parts of a packed row), q_heads a multiple of
    cache.heads -> out fp16 of the same shape, softmax(scale K q) V over the
    tokens lens says each slot holds.  seqs as in kv_paged_append; window > 0
    keeps the last `window` tokens; scale defaults to 1 / sqrt(128); out must not
    overlap q (it may lie beside it in one packed row).  The workspace comes
    from torch or from `workspace` (kv_paged_workspace); use_workspace=False
    gives each sequence and KV head one workgroup."""
    import torch
    dev = cache.device
    qs = _heads_rows(q, None, "q", dev)
    S, Hq, _ = q.shape
    sp, n = _batch(cache, lens, seqs, S)
    if out is None:
        out = torch.empty((S, Hq, 128), dtype=torch.float16, device=dev)
        os_ = Hq * 128
    else:
        os_ = _heads_rows(out, Hq, "out", dev)
        if out.shape[0] != S:
            raise ValueError(f"out must have q's shape {tuple(q.shape)}, got {tuple(out.shape)}")
        if out.numel() and _rows_meet(q, out):
            raise ValueError("out overlaps q")
    if workspace is None and use_workspace:
        workspace = kv_paged_workspace(cache, S, Hq)
    wp, wn = _given(workspace, dev) if workspace is not None and use_workspace else (None, 0)
    _launch("wq_kv_paged_attention", dev, load().wq_kv_paged_attention, q.data_ptr(), qs, Hq, cache._ref,
            lens.data_ptr(), sp, n, window, 0.08838834764831845 if scale is None else scale, out.data_ptr(), os_, wp,
            wn)
    return out


def _pairs(pairs):
    """Host int32 [n, 2] of (source, destination) ids."""
    import numpy as np
    a = np.asarray(pairs)
    if a.size == 0:
        return np.zeros((0, 2), np.int32)
    if a.ndim != 2 or a.shape[1] != 2 or a.dtype.kind not in "iu":
        raise ValueError(f"pairs must be whole numbers [n, 2], got {a.dtype} {a.shape}")
    if a.dtype != np.int32 and (a.min() < -2 ** 31 or a.max() > 2 ** 31 - 1):
        raise ValueError("pairs: an id out of range")
    return np.ascontiguousarray(a, dtype=np.int32)


def kv_paged_copy(cache: PagedKV, pairs):
    """Copy whole pages: pairs, on the host, of (source, destination) page ids
    (an int32 array [n, 2], or a list); no destination twice, none a source."""
    a = _pairs(pairs)
    _launch("wq_kv_paged_copy", cache.device, load().wq_kv_paged_copy, cache._ref, a.ctypes.data, a.shape[0])


def kv_paged_fork(cache: PagedKV, lens, pairs):
    """Fork sequences: for each (source, destination) slot of the host pairs the
    destination becomes a second holder of the source's tokens (whole blocks
    shared through the table, the window's tokens copied, lens set)."""
    import torch
    a = _pairs(pairs)
    _line(lens, torch.int32, cache.slots, "lens", cache.device)
    _launch("wq_kv_paged_fork", cache.device, load().wq_kv_paged_fork, cache._ref, lens.data_ptr(), a.ctypes.data,
            a.shape[0])


def kv_paged_compact_workspace(cache: PagedKV):
    """A workspace tensor for kv_paged_compact of this cache."""
    import torch
    need = _size_t(load().wq_kv_paged_compact_workspace_size, cache._ref, where="wq_kv_paged_compact")
    return torch.empty(need, dtype=torch.uint8, device=cache.device)


def kv_paged_compact(cache: PagedKV, lens, out=None, workspace=None):
    """Move the pages in use (those the table names for the whole blocks of lens)
    to ids 0 .. used - 1.  Returns (table, used): the new int32 table, and int32
    [1] on the GPU.  cache.table is not changed: set cache.table = table to go
    on with the packed pool.  out: such a pair to write into."""
    import torch
    dev = cache.device
    _line(lens, torch.int32, cache.slots, "lens", dev)
    if out is None:
        table = torch.empty((cache.slots, cache.max_pages), dtype=torch.int32, device=dev)
        used = torch.empty(1, dtype=torch.int32, device=dev)
    else:
        table, used = out
        _need(table, torch.int32, (cache.slots, cache.max_pages), "table")
        _line(used, torch.int32, 1, "used", dev)
        if table.device != dev:
            raise ValueError(f"table must be on {dev}")
    wp, wn = _given(kv_paged_compact_workspace(cache) if workspace is None else workspace, dev)
    _launch("wq_kv_paged_compact", dev, load().wq_kv_paged_compact, cache._ref, lens.data_ptr(), table.data_ptr(),
            used.data_ptr(), wp, wn)
    return table, used
