"""MI355X (gfx950) submanifold 3x3x3 sparse convolution: Python binding.

A thin ctypes binding over the C ABI in include/submconv.h.  It only
marshals arguments (torch tensors -> device pointers, the current HIP stream,
status codes -> exceptions); every step of the computation runs in the HIP
library `_lib/libsubmconv.so`.  PyTorch provides device memory and streams.

If the library has not been built, every call raises: there is no CPU or
PyTorch fallback.

No call records anything for torch's autograd: results are detached, also of tensors that
require a gradient.  The backward passes are calls of their own.

Functions carry the C names:

    submconv_build_map(coords, res, batch)        -> Rulebook
    submconv_forward(feats, weight, bias, rb, ...) -> out
    submconv_subdivide(coords, feats=None)          -> (coords8, feats8)
    submconv_space_to_depth(coords, feats, res, batch) -> (coarse, feats8c, mask)
    submconv_depth_to_space(coarse, feats8c, mask=None) -> (coords, feats)
    submconv_upsample_masked(coords, feats, mask)   -> (coords, feats)
    submconv_downsample(coords, feats, res, batch, mode) -> (coarse, feats)
    classify_5d(shape, hint=None)                   -> "krsc" | "oidhw"
    weight_to_krsc(weight, layout=None, hint=None, flip=False) -> KRSC weight
    flip_ab(feats, weight, bias, rb)                -> {"corr": out, "conv": out} for an A/B
    submconv_layer_norm(x, weight, bias, eps)       -> y (and its row statistics)
    submconv_layer_norm_backward(grad, x, stats, weight) -> (dx, dweight, dbias)
    submconv_rotary(x, positions, freqs, sections)  -> rotated heads
    rotary_freqs(sections, theta, device)           -> one frequency ladder per axis
    submconv_attention(q, k, v, q_offsets, k_offsets) -> out (and its log-sum-exp)
    submconv_attention_backward(grad, q, k, v, out, lse, q_offsets, k_offsets) -> (dq, dk, dv)
    batch_offsets(coords, batch)                    -> offsets of a coordinate set's batch entries
    submconv_head_norm_rotary(x, weight, positions, freqs, sections) -> normed and rotated heads (and their 1/rms)
    submconv_head_norm_rotary_backward(grad, x, rstd, weight, positions, freqs, sections) -> (dx, dweight)
    submconv_route(logits, k)                       -> Route(experts, gates, offsets, rows, slots)
    submconv_route_backward(grad, logits, experts, gates) -> dlogits
    submconv_grouped_linear(x, weight, offsets, bias, rows) -> out
    submconv_grouped_linear_backward(grad, x, weight, offsets, rows) -> (dx, dweight, dbias)
    submconv_combine(y, slots, gates)               -> out
    submconv_combine_backward(grad, y, slots, rows, gates) -> (dy, dgates)

`RulebookCache` keeps one rulebook per coordinate set, keyed like the
upstream library's indice_key, so every convolution on a set reuses its map
(lato.2_mrp_mlx working notes, commit summary).
"""
from __future__ import annotations

import ctypes
import os
import weakref
from typing import NamedTuple, Optional

import torch

__all__ = [
    "SubmconvError", "Rulebook", "RulebookCache", "lib_path", "load_library",
    "submconv_build_map", "submconv_forward", "submconv_subdivide",
    "submconv_space_to_depth", "submconv_depth_to_space", "submconv_upsample_masked", "submconv_downsample",
    "POOL_MAX", "POOL_MEAN", "classify_5d", "weight_to_krsc", "flip_ab", "release_cache", "set_cache_limit",
    "submconv_layer_norm", "submconv_layer_norm_backward", "submconv_rotary", "rotary_freqs",
    "submconv_attention", "submconv_attention_backward", "batch_offsets",
    "submconv_head_norm_rotary", "submconv_head_norm_rotary_backward", "Route", "submconv_route", "submconv_route_backward",
    "submconv_grouped_linear", "submconv_grouped_linear_backward", "submconv_combine", "submconv_combine_backward",
    "KERNEL_AUTO", "KERNEL_GENERIC", "KERNEL_LOWC", "KERNEL_MFMA", "KERNEL_WINDOW", "KERNEL_PERSISTENT",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_lib", "libsubmconv.so")

F32, BF16 = 0, 1
OUT_F32 = 256  # added to the type code of an attention call whose out is fp32 (SUBMCONV_OUT_F32)
ROUTE_MAX_K = 16  # SUBMCONV_ROUTE_MAX_K
KERNEL_AUTO, KERNEL_GENERIC, KERNEL_LOWC, KERNEL_MFMA, KERNEL_WINDOW, KERNEL_PERSISTENT = 0, 1, 2, 3, 4, 5

_lib = None


class SubmconvError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__("%s failed: %s (%d): %s" % (where, _status_name(status), status, detail))


def lib_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libsubmconv.so (torch's HIP runtime is already loaded by `import torch`)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError("libsubmconv.so is not built (%s); run "
                           "`python -m submanifold_sparse_convolution_submconv3d_amd._build`" % _LIB_PATH)
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    i64p, i32p = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int32)
    sig = {
        "submconv_build_map": [vp, i64, i32, i32, vp, ctypes.POINTER(vp)],
        "submconv_rulebook_neighbors": [vp, vp, ctypes.POINTER(vp), i64p],
        "submconv_rulebook_copy_neighbors": [vp, vp, vp],
        "submconv_rulebook_info": [vp, i64p, i32p, i32p, i64p],
        "submconv_rulebook_free": [vp, vp],
        "submconv_forward": [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp],
        "submconv_forward_variant": [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp],
        "submconv_subdivide": [vp, vp, i64, i32, i32, vp, vp, vp],
        "submconv_space_to_depth": [vp, vp, i64, i32, i32, i32, i32, vp, vp, vp, i64p, vp],
        "submconv_depth_to_space": [vp, vp, vp, i64, i32, i32, vp, vp, i64p, vp],
        "submconv_upsample_masked": [vp, vp, vp, i64, i32, i32, vp, vp, i64p, vp],
        "submconv_upsample_masked_noalloc": [vp, vp, vp, i64, i32, i32, vp, vp, i64p, vp],
        "submconv_downsample": [vp, vp, i64, i32, i32, i32, i32, i32, vp, vp, i64p, vp],
        "submconv_classify_5d": [i64p, i32, i32p],
        "submconv_release_cache": [i32],
        "submconv_set_cache_limit": [i64],
        "submconv_weight_convert": [vp, i32, i32, i32, i32, i32, vp, vp],
        "submconv_layer_norm": [vp, i64, i64, i32, i32, vp, vp, i32, f32, vp, i64, vp, vp],
        "submconv_layer_norm_backward": [vp, i64, vp, i64, i64, i32, i32, vp, vp, i32, vp, i64, vp, vp, vp,
                                         ctypes.c_size_t, vp],
        "submconv_rotary": [vp, i64, i64, vp, i64, vp, i32p, i32, i64, i32, i32, i32, i32, i32, vp, i64, i64, vp],
        "submconv_attention": [vp, vp, vp, i64p, vp, vp, i32, i64, i64, i32, i32, i32, i32, f32, vp, vp, vp,
                               ctypes.c_size_t, vp],
        "submconv_attention_backward": [vp, vp, vp, vp, vp, vp, i64p, vp, vp, i32, i64, i64, i32, i32, i32, i32, f32,
                                        vp, vp, vp, vp, ctypes.c_size_t, vp],
        "submconv_head_norm_rotary": [vp, i64, i64, vp, i32, i32, i32, f32, vp, i64, vp, i32p, i32, i64, i32, i32, i32, i32,
                                      vp, i64, i64, vp, vp],
        "submconv_head_norm_rotary_backward": [vp, vp, vp, vp, i32, i32, i32, vp, i64, vp, i32p, i32, i64p, i64, i32, i32,
                                               i32, i32, vp, vp, vp, ctypes.c_size_t, vp],
        "submconv_route": [vp, i64, i64, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp],
        "submconv_route_backward": [vp, vp, i64, i64, i32, i32, i32, i32, vp, vp, vp, i64, vp],
        "submconv_grouped_linear": [vp, i64, i64, vp, vp, vp, vp, i32, i64, i32, i32, i32, vp, i64, vp],
        "submconv_grouped_linear_backward": [vp, i64, vp, i64, i64, vp, vp, vp, i32, i64, i32, i32, i32, vp, i64, vp, vp,
                                             vp, ctypes.c_size_t, vp],
        "submconv_combine": [vp, i64, i64, vp, vp, i64, i32, i32, i32, vp, i64, vp],
        "submconv_combine_backward": [vp, i64, vp, i64, i64, vp, vp, vp, i64, i32, i32, i32, vp, i64, vp, vp],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("submconv_attention_workspace", "submconv_attention_backward_workspace"):
        getattr(lib, name).argtypes = [i32, i64, i64, i32, i32, i32, i32]
        getattr(lib, name).restype = ctypes.c_size_t
    lib.submconv_head_norm_rotary_backward_workspace.argtypes = [i64, i32, i32, i32, i32, i32]
    lib.submconv_route_workspace.argtypes = [i64, i32, i32]
    lib.submconv_grouped_linear_backward_workspace.argtypes = [i32, i64, i32, i32, i32]
    for name in ("submconv_head_norm_rotary_backward_workspace", "submconv_route_workspace",
                 "submconv_grouped_linear_backward_workspace"):
        getattr(lib, name).restype = ctypes.c_size_t
    lib.submconv_layer_norm_backward_workspace.argtypes = [i64, i32, i32]
    lib.submconv_layer_norm_backward_workspace.restype = ctypes.c_size_t
    for name in ("submconv_status_string",):
        getattr(lib, name).argtypes = [ctypes.c_int]
        getattr(lib, name).restype = ctypes.c_char_p
    for name in ("submconv_last_error", "submconv_version"):
        getattr(lib, name).argtypes = []
        getattr(lib, name).restype = ctypes.c_char_p
    _lib = lib
    return lib


def _status_name(status: int) -> str:
    try:
        return load_library().submconv_status_string(status).decode()
    except Exception:  # pragma: no cover - library missing
        return "status"


def _check(status: int, where: str):
    if status != 0:
        raise SubmconvError(status, where, load_library().submconv_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError("feature tensors must be float32 or bfloat16, got %s" % t.dtype)


def _dev(t: torch.Tensor, name: str, dtype=None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _raw_stream(index: int) -> int:
    """The current HIP stream of device `index` as an integer handle."""
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if get is not None:
        return get(index)
    return torch.cuda.current_stream(index).cuda_stream


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(_raw_stream(torch.device(device).index))


class Rulebook:
    """A neighbour map built on the device for one coordinate set."""

    def __init__(self, handle: ctypes.c_void_p, device: torch.device, stream: int, n: int, res: int, batch: int):
        self._h = handle
        self.device = device
        self._stream = stream          # raw handle of the stream it was built on
        self.n, self.res, self.batch = n, res, batch
        self._taps = None

    @property
    def taps_present(self) -> int:
        """P, the number of entries of the neighbour table that are not -1."""
        if self._taps is None:
            taps = ctypes.c_int64()
            _check(load_library().submconv_rulebook_info(self.handle, None, None, None, ctypes.byref(taps)),
                   "submconv_rulebook_info")
            self._taps = taps.value
        return self._taps

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h is None:
            raise RuntimeError("rulebook already freed")
        return self._h

    def neighbors(self) -> torch.Tensor:
        """A copy of the int32 [n,27] neighbour table (row i, tap k -> row or -1)."""
        out = torch.empty((self.n, 27), dtype=torch.int32, device=self.device)
        with _on_device(self.device):
            _check(load_library().submconv_rulebook_copy_neighbors(self.handle, ctypes.c_void_p(out.data_ptr()),
                                                                   _stream(self.device)),
                   "submconv_rulebook_copy_neighbors")
        return out

    def free(self, stream: Optional[torch.cuda.Stream] = None):
        """Release the map, ordered on `stream` (default: the current stream of its
        device).  Work on other streams that still reads it must be ordered before
        that stream first, as for any stream-ordered free."""
        if self._h is not None and _lib is not None:
            with _on_device(self.device):
                s = stream.cuda_stream if stream is not None else _raw_stream(self.device.index)
                _lib.submconv_rulebook_free(self._h, ctypes.c_void_p(s))
        self._h = None

    def __del__(self):
        try:
            if self._h is not None and _lib is not None:
                # garbage collection: the release is ordered on the stream the map was built on
                _lib.submconv_rulebook_free(self._h, ctypes.c_void_p(self._stream))
                self._h = None
        except Exception:
            pass


class _on_device:
    """`with torch.cuda.device(d)` without its cost when d is already current."""

    __slots__ = ("_ctx",)

    def __init__(self, device: torch.device):
        idx = device.index
        self._ctx = None if idx is None or idx == torch.cuda.current_device() else torch.cuda.device(idx)

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)


def submconv_build_map(coords: torch.Tensor, res: int, batch: Optional[int] = None) -> Rulebook:
    """Build the rulebook of int32 coords [N,4] (b, z, y, x) on a res^3 grid.

    `batch` is the number of batch entries; None reads max(b)+1 from the device."""
    _dev(coords, "coords", torch.int32)
    if coords.dim() != 2 or coords.shape[1] != 4:
        raise ValueError("coords must be [N,4]")
    if batch is None:
        batch = int(coords[:, 0].max().item()) + 1 if coords.shape[0] else 1
    lib = _lib if _lib is not None else load_library()
    h = ctypes.c_void_p()
    dev = coords.device
    n, res, batch = coords.shape[0], int(res), int(batch)
    with _on_device(dev):
        stream = _raw_stream(dev.index)
        _check(lib.submconv_build_map(coords.data_ptr(), n, res, batch, stream, ctypes.byref(h)),
               "submconv_build_map")
        return Rulebook(h, dev, stream, n, res, batch)


def submconv_forward(feats: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], rb: Rulebook,
                     out: Optional[torch.Tensor] = None, flip: bool = False,
                     variant: int = KERNEL_AUTO) -> torch.Tensor:
    """out[i] = bias + sum_k W[k] . feats[nbr[i,k]]; feats [N,Cin], weight KRSC [Cout,3,3,3,Cin]."""
    _dev(feats, "feats")
    _dev(weight, "weight", feats.dtype)
    if feats.dim() != 2 or feats.shape[0] != rb.n:
        raise ValueError("feats must be [N,Cin] with N = %d" % rb.n)
    cin = feats.shape[1]
    if weight.dim() != 5 or tuple(weight.shape[1:]) != (3, 3, 3, cin):
        raise ValueError("weight must be KRSC [Cout,3,3,3,%d]" % cin)
    cout = weight.shape[0]
    if bias is not None:
        _dev(bias, "bias", torch.float32)
        if bias.shape != (cout,):
            raise ValueError("bias must be fp32 [Cout]")
    if out is None:
        out = torch.empty((rb.n, cout), dtype=feats.dtype, device=feats.device)
    else:
        _dev(out, "out", feats.dtype)
        if tuple(out.shape) != (rb.n, cout):
            raise ValueError("out must be [N,Cout]")
    with _on_device(feats.device):
        _check(load_library().submconv_forward_variant(
            ctypes.c_void_p(feats.data_ptr()), ctypes.c_void_p(weight.data_ptr()),
            ctypes.c_void_p(bias.data_ptr() if bias is not None else None), rb.handle,
            ctypes.c_void_p(out.data_ptr()), cin, cout, _dtype_code(feats), int(bool(flip)), int(variant),
            _stream(feats.device)), "submconv_forward")
    return out


def submconv_subdivide(coords: torch.Tensor, feats: Optional[torch.Tensor] = None):
    """Children of every voxel: (int32 [8N,4], feats [8N,C] or None), parent-major, C order."""
    _dev(coords, "coords", torch.int32)
    n = coords.shape[0]
    out_c = torch.empty((8 * n, 4), dtype=torch.int32, device=coords.device)
    out_f, fp, ofp, c, dt = None, None, None, 0, F32
    if feats is not None:
        _dev(feats, "feats")
        c, dt = feats.shape[1], _dtype_code(feats)
        out_f = torch.empty((8 * n, c), dtype=feats.dtype, device=feats.device)
        fp, ofp = feats.data_ptr(), out_f.data_ptr()
    with _on_device(coords.device):
        _check(load_library().submconv_subdivide(ctypes.c_void_p(coords.data_ptr()), ctypes.c_void_p(fp), n, c, dt,
                                                 ctypes.c_void_p(out_c.data_ptr()), ctypes.c_void_p(ofp),
                                                 _stream(coords.device)), "submconv_subdivide")
    return out_c, out_f


def submconv_space_to_depth(coords: torch.Tensor, feats: torch.Tensor, res: int, batch: int):
    """Factor-2 sparse space-to-depth: (coarse int32 [M,4], feats [M,8C], uint8 mask [M,8])."""
    _dev(coords, "coords", torch.int32)
    _dev(feats, "feats")
    n, c = feats.shape
    out_c = torch.empty((max(n, 1), 4), dtype=torch.int32, device=coords.device)
    out_f = torch.empty((max(n, 1), 8 * c), dtype=feats.dtype, device=feats.device)
    mask = torch.empty((max(n, 1), 8), dtype=torch.uint8, device=feats.device)
    m = ctypes.c_int64()
    with _on_device(coords.device):
        _check(load_library().submconv_space_to_depth(
            ctypes.c_void_p(coords.data_ptr()), ctypes.c_void_p(feats.data_ptr()), n, c, _dtype_code(feats),
            int(res), int(batch), ctypes.c_void_p(out_c.data_ptr()), ctypes.c_void_p(out_f.data_ptr()),
            ctypes.c_void_p(mask.data_ptr()), ctypes.byref(m), _stream(coords.device)), "submconv_space_to_depth")
    m = m.value
    return out_c[:m], out_f[:m], mask[:m]


def submconv_depth_to_space(coarse: torch.Tensor, coarse_feats: torch.Tensor, mask: Optional[torch.Tensor] = None):
    """Inverse of space-to-depth: every slot (mask None) or the masked ones -> (coords, feats)."""
    _dev(coarse, "coarse", torch.int32)
    _dev(coarse_feats, "coarse_feats")
    m, c8 = coarse_feats.shape
    if c8 % 8:
        raise ValueError("coarse_feats must be [M, 8C]")
    c = c8 // 8
    mp = None
    if mask is not None:
        _dev(mask, "mask", torch.uint8)
        if tuple(mask.shape) != (m, 8):
            raise ValueError("mask must be uint8 [M,8]")
        mp = mask.data_ptr()
    out_c = torch.empty((max(8 * m, 1), 4), dtype=torch.int32, device=coarse.device)
    out_f = torch.empty((max(8 * m, 1), c), dtype=coarse_feats.dtype, device=coarse.device)
    cnt = ctypes.c_int64()
    with _on_device(coarse.device):
        _check(load_library().submconv_depth_to_space(
            ctypes.c_void_p(coarse.data_ptr()), ctypes.c_void_p(coarse_feats.data_ptr()), ctypes.c_void_p(mp), m, c,
            _dtype_code(coarse_feats), ctypes.c_void_p(out_c.data_ptr()), ctypes.c_void_p(out_f.data_ptr()),
            ctypes.byref(cnt), _stream(coarse.device)), "submconv_depth_to_space")
    k = cnt.value
    return out_c[:k], out_f[:k]


class RulebookCache:
    """One rulebook per coordinate set, looked up by a caller-chosen key
    (the upstream library's indice_key), built on first use.

    A cached map is reused only for the very coordinate tensor it was built from
    (the same tensor object, not modified in place since: its version counter is
    unchanged) and the same grid and batch count.  Any other tensor under the key,
    even one of the same size, rebuilds the map and replaces the entry."""

    def __init__(self):
        self._maps = {}

    def get(self, key, coords: torch.Tensor, res: int, batch: Optional[int] = None) -> Rulebook:
        entry = self._maps.get(key)
        if entry is not None:
            rb, ref, version, r, b = entry
            if (ref() is coords and coords._version == version and r == int(res)
                    and (batch is None or b == int(batch))):
                return rb
            self.drop(key)
        rb = submconv_build_map(coords, res, batch)
        self._maps[key] = (rb, weakref.ref(coords), coords._version, int(res), rb.batch)
        return rb

    def drop(self, key):
        entry = self._maps.pop(key, None)
        if entry is not None:
            entry[0].free()

    def clear(self):
        for k in list(self._maps):
            self.drop(k)

    def __len__(self):
        return len(self._maps)


POOL_MAX, POOL_MEAN = 0, 1  # submconv_downsample modes (SUBMCONV_POOL_*)


def submconv_upsample_masked(coords: torch.Tensor, feats: torch.Tensor, mask: torch.Tensor):
    """Masked expansion: voxel i emits child s iff mask[i, s] (axis 0 fastest), feats copied -> (coords, feats)."""
    _dev(coords, "coords", torch.int32)
    _dev(feats, "feats")
    _dev(mask, "mask", torch.uint8)
    n, c = feats.shape
    if tuple(mask.shape) != (n, 8) or coords.shape[0] != n:
        raise ValueError("coords [N,4], feats [N,C] and mask uint8 [N,8] must agree")
    out_c = torch.empty((max(8 * n, 1), 4), dtype=torch.int32, device=coords.device)
    out_f = torch.empty((max(8 * n, 1), c), dtype=feats.dtype, device=feats.device)
    cnt = ctypes.c_int64()
    with _on_device(coords.device):
        _check(load_library().submconv_upsample_masked(
            ctypes.c_void_p(coords.data_ptr()), ctypes.c_void_p(feats.data_ptr()), ctypes.c_void_p(mask.data_ptr()),
            n, c, _dtype_code(feats), ctypes.c_void_p(out_c.data_ptr()), ctypes.c_void_p(out_f.data_ptr()),
            ctypes.byref(cnt), _stream(coords.device)), "submconv_upsample_masked")
    k = cnt.value
    return out_c[:k], out_f[:k]


def submconv_downsample(coords: torch.Tensor, feats: torch.Tensor, res: int, batch: int, mode: str):
    """Factor-2 pooling of each coarse voxel's children, mode 'max' or 'mean' -> (coarse int32 [M,4], feats [M,C])."""
    if mode not in ("max", "mean"):
        raise ValueError("mode must be 'max' or 'mean' (it differs between models, so it has no default)")
    _dev(coords, "coords", torch.int32)
    _dev(feats, "feats")
    n, c = feats.shape
    out_c = torch.empty((max(n, 1), 4), dtype=torch.int32, device=coords.device)
    out_f = torch.empty((max(n, 1), c), dtype=feats.dtype, device=feats.device)
    m = ctypes.c_int64()
    with _on_device(coords.device):
        _check(load_library().submconv_downsample(
            ctypes.c_void_p(coords.data_ptr()), ctypes.c_void_p(feats.data_ptr()), n, c, _dtype_code(feats),
            int(res), int(batch), POOL_MAX if mode == "max" else POOL_MEAN, ctypes.c_void_p(out_c.data_ptr()),
            ctypes.c_void_p(out_f.data_ptr()), ctypes.byref(m), _stream(coords.device)), "submconv_downsample")
    k = m.value
    return out_c[:k], out_f[:k]


_LAYOUTS = {"krsc": 0, "oidhw": 1}


def classify_5d(shape, hint: Optional[str] = None) -> str:
    """"krsc" ([O,kz,ky,kx,I], spconv) or "oidhw" ([O,I,kz,ky,kx], torch Conv3d) for a
    5-D 3x3x3 weight shape; `hint` is the layout the caller's module implies, needed
    when the shape fits both ([O,3,3,3,3])."""
    if len(shape) != 5:
        raise ValueError("a 5-D weight shape is expected")
    arr = (ctypes.c_int64 * 5)(*[int(d) for d in shape])
    out = ctypes.c_int32(-1)
    h = -1 if hint is None else _LAYOUTS[hint]
    _check(load_library().submconv_classify_5d(arr, h, ctypes.byref(out)), "submconv_classify_5d")
    return "krsc" if out.value == 0 else "oidhw"


def weight_to_krsc(weight: torch.Tensor, layout: Optional[str] = None, hint: Optional[str] = None,
                   flip: bool = False) -> torch.Tensor:
    """KRSC copy of a 3x3x3 weight in either layout (classified from its shape when
    `layout` is None), mirrored (tap k -> 26 - k) when `flip`."""
    _dev(weight, "weight")
    if weight.dim() != 5:
        raise ValueError("a 5-D weight is expected")
    layout = layout or classify_5d(tuple(weight.shape), hint)
    if layout == "krsc":
        cout, cin = weight.shape[0], weight.shape[4]
    else:
        cout, cin = weight.shape[0], weight.shape[1]
    out = torch.empty((cout, 3, 3, 3, cin), dtype=weight.dtype, device=weight.device)
    with _on_device(weight.device):
        _check(load_library().submconv_weight_convert(
            ctypes.c_void_p(weight.data_ptr()), _LAYOUTS[layout], cout, cin, _dtype_code(weight), int(bool(flip)),
            ctypes.c_void_p(out.data_ptr()), _stream(weight.device)), "submconv_weight_convert")
    return out


def flip_ab(feats: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor], rb: "Rulebook") -> dict:
    """Both kernel orientations on the same input, for an end-to-end A/B (the caller
    compares them downstream): "corr" reads feats[c + d] (flip 0), "conv" feats[c - d]
    (flip 1, the mirrored kernel)."""
    return {"corr": submconv_forward(feats, weight, bias, rb, flip=False),
            "conv": submconv_forward(feats, weight, bias, rb, flip=True)}


def _strided(t: torch.Tensor, name: str, dims: int, device=None, dtype=None) -> torch.Tensor:
    """A GPU tensor of `dims` dimensions whose innermost elements are next to each other."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    if t.dim() != dims:
        raise ValueError("%s must have %d dimensions, got %d" % (name, dims, t.dim()))
    if t.stride(dims - 1) != 1 and t.shape[dims - 1] > 1 and t.numel():
        raise ValueError("the last dimension of %s must be contiguous" % name)
    return t


def _row_stride(t: torch.Tensor) -> int:
    """Distance between rows; torch may report any for a single row."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _norm_params(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor]) -> int:
    """Type code of the parameter vectors (both fp32 or both bf16)."""
    code = None
    index, shape = x.get_device(), x.shape[1:]
    for name, p in (("weight", weight), ("bias", bias)):
        if p is None:
            continue
        if _dev(p, name).get_device() != index:
            raise ValueError("%s is on %s, not on %s" % (name, p.device, x.device))
        if p.shape != shape:
            raise ValueError("%s must be [%d]" % (name, x.shape[1]))
        kind = _dtype_code(p)
        if code is not None and code != kind:
            raise TypeError("weight and bias must have one type")
        code = kind
    return F32 if code is None else code


def submconv_layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        eps: float = 1e-5, out: Optional[torch.Tensor] = None, return_stats: bool = False):
    """Layer normalisation of the rows of x [N,C] (C <= 8192; rows may be strided) -> y, or (y, stats)
    with stats fp32 [N,2] = (mean, 1/std) for the backward pass.

    weight and bias [C] are fp32 or bf16 (None: 1 and 0); statistics are fp32.  `out` may be x.
    Not recorded by autograd: submconv_layer_norm_backward gives the gradients."""
    dev = _strided(x, "x", 2).device
    n, c = x.shape
    code = _norm_params(x, weight, bias)
    if out is None:
        out = torch.empty((n, c), dtype=x.dtype, device=dev)
    elif tuple(_strided(out, "out", 2, dev, x.dtype).shape) != (n, c):
        raise ValueError("out must be [N,C]")
    stats = torch.empty((n, 2), dtype=torch.float32, device=dev) if return_stats else None
    lib = _lib if _lib is not None else load_library()
    with _on_device(dev):
        _check(lib.submconv_layer_norm(
            x.data_ptr(), _row_stride(x), n, c, _dtype_code(x), None if weight is None else weight.data_ptr(),
            None if bias is None else bias.data_ptr(), code, eps, out.data_ptr(), _row_stride(out),
            None if stats is None else stats.data_ptr(), _raw_stream(dev.index)), "submconv_layer_norm")
    return (out, stats) if return_stats else out


def submconv_layer_norm_backward(grad: torch.Tensor, x: torch.Tensor, stats: torch.Tensor,
                                 weight: Optional[torch.Tensor] = None, param_dtype: Optional[torch.dtype] = None,
                                 need_params: bool = True):
    """Gradients of submconv_layer_norm -> (dx, dweight, dbias).

    `stats` is what the forward returned for x.  dweight and dbias have weight's type (param_dtype,
    or fp32, without a weight) and are None with need_params=False; they are summed in a fixed
    order, so equal calls give equal bits."""
    dev = _strided(x, "x", 2).device
    n, c = x.shape
    if tuple(_strided(grad, "grad", 2, dev, x.dtype).shape) != (n, c):
        raise ValueError("grad must be [N,C]")
    _dev(stats, "stats", torch.float32)
    if tuple(stats.shape) != (n, 2) or stats.device != dev:
        raise ValueError("stats must be fp32 [N,2] on x's device")
    kind = weight.dtype if weight is not None else (param_dtype or torch.float32)
    code = _norm_params(x, weight, None)
    if weight is None and kind not in (torch.float32, torch.bfloat16):
        raise TypeError("param_dtype must be float32 or bfloat16, got %s" % kind)
    code = code if weight is not None else (F32 if kind == torch.float32 else BF16)
    dx = torch.empty((n, c), dtype=x.dtype, device=dev)
    lib = _lib if _lib is not None else load_library()
    dw = db = ws = None
    nbytes = 0
    if need_params:
        dw, db = torch.empty((2, c), dtype=kind, device=dev).unbind(0)
        nbytes = lib.submconv_layer_norm_backward_workspace(n, c, _dtype_code(x))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    with _on_device(dev):
        _check(lib.submconv_layer_norm_backward(
            grad.data_ptr(), _row_stride(grad), x.data_ptr(), _row_stride(x), n, c, _dtype_code(x), stats.data_ptr(),
            None if weight is None else weight.data_ptr(), code, dx.data_ptr(), c,
            None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(),
            None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dev.index)), "submconv_layer_norm_backward")
    return dx, dw, db


def rotary_freqs(sections, theta: float = 10000.0, device="cuda") -> torch.Tensor:
    """One ladder per axis, theta^(-i/n) for i < n = its pairs: fp32 [sum(sections)], formed in fp64.
    sections (21, 21, 21) are the 63 frequencies of a 128-wide head on three axes."""
    parts = [torch.pow(float(theta), -torch.arange(int(n), dtype=torch.float64) / max(1, int(n))) for n in sections]
    return torch.cat(parts).float().to(device)


def _head_strides(t: torch.Tensor):
    """(row, head) distances of [N,H,D]; torch may report any for a dimension of one."""
    n, h, d = t.shape
    if not n:
        return h * d, d
    head = t.stride(1) if h > 1 else d
    return (t.stride(0) if n > 1 else (h - 1) * head + d), head


def submconv_rotary(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, sections, inverse: bool = False,
                    split: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotate the head vectors x [N,H,D] by integer positions on several axes.

    positions int32 [N,A] (the coords[:, 1:] columns of a voxel set), freqs fp32 [sum(sections)] in
    radians a step, sections = pairs of each axis (their sum <= D/2; the pairs left over are
    copied).  Pair p is elements (2p, 2p+1), or (p, p + D/2) with split.  inverse turns back,
    which is the gradient (autograd does not record this call).  x may be strided (the query and key part of a packed projection);
    `out` may be x itself."""
    dev = _strided(x, "x", 3).device
    _strided(positions, "positions", 2, dev, torch.int32)
    if _dev(freqs, "freqs", torch.float32).device != dev:
        raise ValueError("freqs is on %s, not on %s" % (freqs.device, dev))
    n, h, d = x.shape
    axes = len(sections)
    if tuple(positions.shape) != (n, axes):
        raise ValueError("positions must be [N,%d]" % axes)
    if freqs.dim() != 1 or freqs.shape[0] != sum(sections):
        raise ValueError("freqs must be [%d], one for each pair of the sections" % sum(sections))
    if out is None:
        out = torch.empty((n, h, d), dtype=x.dtype, device=dev)
    elif tuple(_strided(out, "out", 3, dev, x.dtype).shape) != (n, h, d):
        raise ValueError("out must be [N,H,D]")
    xs, os_ = _head_strides(x), _head_strides(out)
    lib = _lib if _lib is not None else load_library()
    with _on_device(dev):
        _check(lib.submconv_rotary(
            x.data_ptr(), xs[0], xs[1], positions.data_ptr(), _row_stride(positions), freqs.data_ptr(),
            (ctypes.c_int32 * max(1, axes))(*sections), axes, n, h, d, _dtype_code(x), int(bool(split)),
            int(bool(inverse)), out.data_ptr(), os_[0], os_[1], _raw_stream(dev.index)), "submconv_rotary")
    return out


def batch_offsets(coords: torch.Tensor, batch: int) -> torch.Tensor:
    """Offsets int32 [batch+1] of the batch entries of coords [N,4] whose rows are grouped by
    ascending b (as argwhere order and every call here that makes coordinates leave them)."""
    _dev(coords, "coords", torch.int32)
    edges = torch.arange(int(batch) + 1, dtype=torch.int32, device=coords.device)
    return torch.searchsorted(coords[:, 0].contiguous(), edges, out_int32=True)


def _attention_sizes(q, k, v, q_offsets, k_offsets):
    """Checks shared by both directions -> (device, nq, heads, dim, nk, kv_heads, entries)."""
    dev = _strided(q, "q", 3).device
    _strided(k, "k", 3, dev, q.dtype)
    _strided(v, "v", 3, dev, q.dtype)
    if k.shape != v.shape or k.shape[2] != q.shape[2]:
        raise ValueError("q [Nq,H,D], k and v [Nk,Hk,D] must agree")
    for name, o in (("q_offsets", q_offsets), ("k_offsets", k_offsets)):
        if _dev(o, name, torch.int32).device != dev:
            raise ValueError("%s is on %s, not on %s" % (name, o.device, dev))
    entries = q_offsets.numel() - 1
    if q_offsets.dim() != 1 or k_offsets.shape != q_offsets.shape or entries < 1:
        raise ValueError("q_offsets and k_offsets must be [entries+1]")
    return (dev,) + tuple(q.shape) + (k.shape[0], k.shape[1], entries)


def _attention_scale(scale: Optional[float], d: int) -> float:
    return scale if scale is not None else max(d, 1) ** -0.5


def _attention_code(q: torch.Tensor, out: torch.Tensor) -> int:
    """Type code of an attention call: out has q's type or is fp32."""
    if out.dtype == q.dtype:
        return _dtype_code(q)
    if out.dtype != torch.float32:
        raise TypeError("out must be %s or float32, got %s" % (q.dtype, out.dtype))
    return _dtype_code(q) | OUT_F32


def submconv_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: torch.Tensor,
                       k_offsets: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None, return_lse: bool = False,
                       out_dtype: Optional[torch.dtype] = None):
    """Softmax attention inside each entry of a ragged batch -> out [Nq,H,D], or (out, lse) with
    lse fp32 [Nq,H] for the backward pass.

    q [Nq,H,D], k and v [Nk,Hk,D] with H a multiple of Hk, D a multiple of 8 up to 128; strided
    views (parts of a packed projection) are taken as they are.  Offsets int32 [entries+1] on the
    device (batch_offsets); k_offsets None: those of the queries.  scale None: 1/sqrt(D).  Queries
    of an entry without keys, and rows outside every entry, give zeros (lse -inf).  out_dtype (or
    `out`) may be float32 beside bf16 tensors: the result without its last rounding, from which the
    backward pass takes more accurate gradients.  Not recorded by autograd:
    submconv_attention_backward gives the gradients."""
    k_offsets = q_offsets if k_offsets is None else k_offsets
    dev, nq, h, d, nk, hk, entries = _attention_sizes(q, k, v, q_offsets, k_offsets)
    if out is None:
        out = torch.empty((nq, h, d), dtype=out_dtype or q.dtype, device=dev)
    elif tuple(_strided(out, "out", 3, dev, out_dtype).shape) != (nq, h, d):
        raise ValueError("out must be [Nq,H,D]")
    lse = torch.empty((nq, h), dtype=torch.float32, device=dev) if return_lse else None
    lib = _lib if _lib is not None else load_library()
    code = _attention_code(q, out)
    nbytes = lib.submconv_attention_workspace(entries, nq, nk, h, hk, d, code)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    strides = (ctypes.c_int64 * 8)(*_head_strides(q), *_head_strides(k), *_head_strides(v), *_head_strides(out))
    with _on_device(dev):
        _check(lib.submconv_attention(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), strides, q_offsets.data_ptr(), k_offsets.data_ptr(), entries, nq,
            nk, h, hk, d, code, _attention_scale(scale, d), out.data_ptr(),
            None if lse is None else lse.data_ptr(), None if ws is None else ws.data_ptr(), nbytes,
            _raw_stream(dev.index)), "submconv_attention")
    return (out, lse) if return_lse else out


def submconv_attention_backward(grad: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                out: torch.Tensor, lse: torch.Tensor, q_offsets: torch.Tensor,
                                k_offsets: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                                dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                                dv: Optional[torch.Tensor] = None):
    """Gradients of submconv_attention -> (dq, dk, dv), from its out and lse.  A shared key head's
    gradient is summed over its query heads.  dq, dk, dv may be given (parts of a packed gradient).
    Sums run in a fixed order: equal calls give equal bits.  With bf16 tensors, `out` kept in float32
    (the forward's out_dtype) spares dq and dk the rounding of out, which is the largest part of
    their error where the softmax is peaked or v has a common offset."""
    k_offsets = q_offsets if k_offsets is None else k_offsets
    dev, nq, h, d, nk, hk, entries = _attention_sizes(q, k, v, q_offsets, k_offsets)
    for name, t, kind in (("grad", grad, q.dtype), ("out", out, None)):
        if tuple(_strided(t, name, 3, dev, kind).shape) != (nq, h, d):
            raise ValueError("%s must be [Nq,H,D]" % name)
    if tuple(_dev(lse, "lse", torch.float32).shape) != (nq, h) or lse.device != dev:
        raise ValueError("lse must be fp32 [Nq,H] on q's device")
    made = []
    for name, t, shape in (("dq", dq, (nq, h, d)), ("dk", dk, (nk, hk, d)), ("dv", dv, (nk, hk, d))):
        if t is None:
            t = torch.empty(shape, dtype=q.dtype, device=dev)
        elif tuple(_strided(t, name, 3, dev, q.dtype).shape) != shape:
            raise ValueError("%s must be %s" % (name, list(shape)))
        made.append(t)
    dq, dk, dv = made
    lib = _lib if _lib is not None else load_library()
    code = _attention_code(q, out)
    nbytes = lib.submconv_attention_backward_workspace(entries, nq, nk, h, hk, d, code)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    strides = (ctypes.c_int64 * 16)(*[s for t in (grad, q, k, v, out, dq, dk, dv) for s in _head_strides(t)])
    with _on_device(dev):
        _check(lib.submconv_attention_backward(
            grad.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(), strides,
            q_offsets.data_ptr(), k_offsets.data_ptr(), entries, nq, nk, h, hk, d, code,
            _attention_scale(scale, d), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), ws.data_ptr(), nbytes,
            _raw_stream(dev.index)), "submconv_attention_backward")
    return dq, dk, dv


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _same_device(t: Optional[torch.Tensor], name: str, dtype, device, shape) -> Optional[torch.Tensor]:
    """A contiguous tensor of this type, device and shape (None passes)."""
    if t is not None:
        if _dev(t, name, dtype).device != device:
            raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
        if tuple(t.shape) != tuple(shape):
            raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    return t


def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _head_norm_args(x, weight, positions, freqs, sections, q_heads):
    """Checks shared by both directions -> (device, weight's rows, its type code, sections)."""
    dev = _strided(x, "x", 3).device
    n, h, d = x.shape
    many, code = 1, F32
    if weight is not None:
        code = _dtype_code(weight)
        many = weight.shape[0] if weight.dim() == 2 else 1
        if (2 if q_heads else many) != many or many not in (1, 2 if q_heads else 1, h):
            raise ValueError("weight must be [D], [H,D], or [2,D] with q_heads")
        _same_device(weight, "weight", None, dev, (d,) if weight.dim() == 1 else (many, d))
    elif q_heads:
        raise ValueError("q_heads without a weight")
    sections = tuple(sections) if positions is not None else ()
    if positions is not None:
        _strided(positions, "positions", 2, dev, torch.int32)
        if tuple(positions.shape) != (n, len(sections)):
            raise ValueError("positions must be [N,%d]" % len(sections))
        if freqs is None:
            raise ValueError("positions without freqs")
        _same_device(freqs, "freqs", torch.float32, dev, (sum(sections),))
    return dev, many, code, sections


def submconv_head_norm_rotary(x: torch.Tensor, weight: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                              freqs: Optional[torch.Tensor] = None, sections=(), eps: float = 1e-6, q_heads: int = 0,
                              split: bool = False, out: Optional[torch.Tensor] = None, return_rstd: bool = False):
    """Root-mean-square norm of the head vectors x [N,H,D] and their rotation by integer positions, in one
    pass -> y, or (y, rstd) with rstd fp32 [N,H] for the backward pass.

    weight (fp32 or bf16; None: 1) is [H,D], one for each head, [D], one for all, or [2,D] with q_heads: heads
    below q_heads are queries (row 0), the others keys (row 1).  positions, freqs, sections and split are
    those of submconv_rotary; without positions nothing turns.  x may be strided (the query and key part
    of a packed projection); `out` may be x itself.  fp32, one rounding at the end.  Not recorded by
    autograd: submconv_head_norm_rotary_backward gives the gradients."""
    dev, many, code, sections = _head_norm_args(x, weight, positions, freqs, sections, q_heads)
    n, h, d = x.shape
    if out is None:
        out = torch.empty((n, h, d), dtype=x.dtype, device=dev)
    elif tuple(_strided(out, "out", 3, dev, x.dtype).shape) != (n, h, d):
        raise ValueError("out must be [N,H,D]")
    rstd = torch.empty((n, h), dtype=torch.float32, device=dev) if return_rstd else None
    xs, os_ = _head_strides(x), _head_strides(out)
    lib = _lib if _lib is not None else load_library()
    with _on_device(dev):
        _check(lib.submconv_head_norm_rotary(
            x.data_ptr(), xs[0], xs[1], _ptr(weight), many, q_heads, code, eps, _ptr(positions),
            0 if positions is None else _row_stride(positions), None if positions is None else freqs.data_ptr(),
            (ctypes.c_int32 * max(1, len(sections)))(*sections), len(sections), n, h, d, _dtype_code(x), int(bool(split)),
            out.data_ptr(), os_[0], os_[1], _ptr(rstd), _raw_stream(dev.index)), "submconv_head_norm_rotary")
    return (out, rstd) if return_rstd else out


def submconv_head_norm_rotary_backward(grad: torch.Tensor, x: torch.Tensor, rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                                       positions: Optional[torch.Tensor] = None, freqs: Optional[torch.Tensor] = None, sections=(),
                                       q_heads: int = 0, split: bool = False, dx: Optional[torch.Tensor] = None,
                                       need_weight: bool = True):
    """Gradients of submconv_head_norm_rotary -> (dx, dweight).

    `rstd` is what the forward returned for x.  dweight has weight's shape and type (None without a weight
    or with need_weight=False), summed in a fixed order, so equal calls give equal bits.  dx may be given
    (part of a packed gradient, or grad itself)."""
    dev, many, code, sections = _head_norm_args(x, weight, positions, freqs, sections, q_heads)
    n, h, d = x.shape
    if tuple(_strided(grad, "grad", 3, dev, x.dtype).shape) != (n, h, d):
        raise ValueError("grad must be [N,H,D]")
    _same_device(rstd, "rstd", torch.float32, dev, (n, h))
    if dx is None:
        dx = torch.empty((n, h, d), dtype=x.dtype, device=dev)
    elif tuple(_strided(dx, "dx", 3, dev, x.dtype).shape) != (n, h, d):
        raise ValueError("dx must be [N,H,D]")
    lib = _lib if _lib is not None else load_library()
    dw = ws = None
    nbytes = 0
    if weight is not None and need_weight:
        dw = torch.empty_like(weight)
        nbytes = lib.submconv_head_norm_rotary_backward_workspace(n, h, d, _dtype_code(x), many, q_heads)
        ws = _workspace(nbytes, dev)
    strides = (ctypes.c_int64 * 6)(*_head_strides(grad), *_head_strides(x), *_head_strides(dx))
    with _on_device(dev):
        _check(lib.submconv_head_norm_rotary_backward(
            grad.data_ptr(), x.data_ptr(), rstd.data_ptr(), _ptr(weight), many, q_heads, code, _ptr(positions),
            0 if positions is None else _row_stride(positions), None if positions is None else freqs.data_ptr(),
            (ctypes.c_int32 * max(1, len(sections)))(*sections), len(sections), strides, n, h, d, _dtype_code(x),
            int(bool(split)), dx.data_ptr(), _ptr(dw), _ptr(ws), nbytes, _raw_stream(dev.index)),
            "submconv_head_norm_rotary_backward")
    return dx, dw


class Route(NamedTuple):
    """The plan of submconv_route for [N,E] scores and k experts a row."""
    experts: torch.Tensor  # int32 [N,k], best first; -1 where fewer than k are open
    gates: torch.Tensor    # fp32 [N,k]; 0 beside a -1
    offsets: torch.Tensor  # int32 [E+1]: the positions of each expert; from the last on, pairs without an expert
    rows: torch.Tensor     # int32 [N*k]: the row of each position
    slots: torch.Tensor    # int32 [N,k]: the position of each pair


def submconv_route(logits: torch.Tensor, k: int, normalize: bool = True) -> Route:
    """The k best experts of each row of scores [N,E], their gates, and the rows grouped by expert.

    Equal scores go by number; -inf closes an expert to a row.  Gates are the softmax over the row's chosen
    experts (normalize), or their share of the softmax over all.  The plan feeds submconv_grouped_linear
    (offsets, rows) and submconv_combine (slots, gates); it is exact and formed on the device."""
    dev = _strided(logits, "logits", 2).device
    n, e = logits.shape
    k = max(-1, min(int(k), 2 ** 31 - 1))       # what the library refuses, it refuses whole,
    m = k if 0 < k <= ROUTE_MAX_K else 0        # and nothing is allocated for
    experts = torch.empty((n, m), dtype=torch.int32, device=dev)
    slots = torch.empty((n, m), dtype=torch.int32, device=dev)
    rows = torch.empty(n * m, dtype=torch.int32, device=dev)
    gates = torch.empty((n, m), dtype=torch.float32, device=dev)
    offsets = torch.empty(e + 1, dtype=torch.int32, device=dev)
    lib = _lib if _lib is not None else load_library()
    nbytes = lib.submconv_route_workspace(n, e, k)
    ws = _workspace(nbytes, dev)
    with _on_device(dev):
        _check(lib.submconv_route(
            logits.data_ptr(), _row_stride(logits), n, e, k, _dtype_code(logits), int(bool(normalize)), experts.data_ptr(),
            gates.data_ptr(), offsets.data_ptr(), rows.data_ptr(), slots.data_ptr(), _ptr(ws), nbytes, _raw_stream(dev.index)),
            "submconv_route")
    return Route(experts, gates, offsets, rows, slots)


def submconv_route_backward(grad: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, gates: torch.Tensor,
                            normalize: bool = True) -> torch.Tensor:
    """Gradient of the scores [N,E] from the gradient of submconv_route's gates, fp32 [N,k] -> dlogits, of
    logits' type.  experts and gates are the Route's, normalize as in its call.  What grad holds beside a -1 is not used."""
    dev = _strided(logits, "logits", 2).device
    n, e = logits.shape
    k = gates.shape[1] if gates.dim() == 2 else 0
    for name, t, kind in (("grad", grad, torch.float32), ("gates", gates, torch.float32), ("experts", experts, torch.int32)):
        _same_device(t, name, kind, dev, (n, k))
    out = torch.empty((n, e), dtype=logits.dtype, device=dev)
    lib = _lib if _lib is not None else load_library()
    with _on_device(dev):
        _check(lib.submconv_route_backward(
            grad.data_ptr(), logits.data_ptr(), _row_stride(logits), n, e, k, _dtype_code(logits), int(bool(normalize)),
            experts.data_ptr(), gates.data_ptr(), out.data_ptr(), e, _raw_stream(dev.index)), "submconv_route_backward")
    return out


def _linear_args(x, weight, offsets, rows):
    """Checks shared by both directions -> (device, positions, groups, cout)."""
    dev = _strided(x, "x", 2).device
    if weight.dim() != 3 or weight.shape[2] != x.shape[1]:
        raise ValueError("weight must be [G,Cout,Cin] for x [N,Cin]")
    _same_device(weight, "weight", x.dtype, dev, weight.shape)
    groups, cout = weight.shape[:2]
    _same_device(offsets, "offsets", torch.int32, dev, (groups + 1,))
    if rows is not None:
        if rows.dim() != 1:
            raise ValueError("rows must be [P]")
        _same_device(rows, "rows", torch.int32, dev, rows.shape)
    return dev, x.shape[0] if rows is None else rows.shape[0], groups, cout


def submconv_grouped_linear(x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor, bias: Optional[torch.Tensor] = None,
                            rows: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Matrix products of ragged groups of rows, each group with its own weight -> out [P,Cout]:
    out[i] = weight[g] x[rows[i]] + bias[g] for the positions i of group g.

    x [N,Cin] (rows may be strided), weight [G,Cout,Cin] of x's type, bias fp32 [G,Cout] or None, offsets int32
    [G+1] on the device (submconv_route's, or batch_offsets), rows int32 [P]: the row of x of each position
    (None: the position itself, P = N).  Positions outside every group get zeros.  Not recorded by
    autograd: submconv_grouped_linear_backward gives the gradients."""
    dev, many, groups, cout = _linear_args(x, weight, offsets, rows)
    nx, cin = x.shape
    _same_device(bias, "bias", torch.float32, dev, (groups, cout))
    if out is None:
        out = torch.empty((many, cout), dtype=x.dtype, device=dev)
    elif tuple(_strided(out, "out", 2, dev, x.dtype).shape) != (many, cout):
        raise ValueError("out must be [P,Cout]")
    lib = _lib if _lib is not None else load_library()
    with _on_device(dev):
        _check(lib.submconv_grouped_linear(
            x.data_ptr(), _row_stride(x), nx, _ptr(rows), weight.data_ptr(), _ptr(bias), offsets.data_ptr(), groups, many, cin,
            cout, _dtype_code(x), out.data_ptr(), _row_stride(out), _raw_stream(dev.index)), "submconv_grouped_linear")
    return out


def submconv_grouped_linear_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                                     rows: Optional[torch.Tensor] = None, need_x: bool = True, need_weight: bool = True,
                                     need_bias: bool = False):
    """Gradients of submconv_grouped_linear from grad [P,Cout] -> (dx, dweight, dbias), None for what is not needed.

    dx [P,Cin] is the gradient of the rows as they were taken: with `rows`, submconv_combine(dx, slots) sums it for
    each row of x.  dweight has weight's type, dbias is fp32; need_bias takes need_weight.  Sums run in a
    fixed order: equal calls give equal bits."""
    dev, many, groups, cout = _linear_args(x, weight, offsets, rows)
    nx, cin = x.shape
    if tuple(_strided(grad, "grad", 2, dev, x.dtype).shape) != (many, cout):
        raise ValueError("grad must be [P,Cout]")
    if need_bias and not need_weight:
        raise ValueError("need_bias takes need_weight")
    dx = torch.empty((many, cin), dtype=x.dtype, device=dev) if need_x else None
    dw = torch.empty_like(weight) if need_weight else None
    db = torch.empty((groups, cout), dtype=torch.float32, device=dev) if need_bias else None
    lib = _lib if _lib is not None else load_library()
    nbytes = lib.submconv_grouped_linear_backward_workspace(groups, many, cin, cout, _dtype_code(x)) if need_weight else 0
    ws = _workspace(nbytes, dev)
    with _on_device(dev):
        _check(lib.submconv_grouped_linear_backward(
            grad.data_ptr(), _row_stride(grad), x.data_ptr(), _row_stride(x), nx, _ptr(rows), weight.data_ptr(), offsets.data_ptr(),
            groups, many, cin, cout, _dtype_code(x), _ptr(dx), cin, _ptr(dw), _ptr(db), _ptr(ws), nbytes, _raw_stream(dev.index)),
            "submconv_grouped_linear_backward")
    return dx, dw, db


def submconv_combine(y: torch.Tensor, slots: torch.Tensor, gates: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The sum of each row's expert results, out[i] = sum_j gates[i,j] y[slots[i,j]] -> out [N,C].

    y [P,C] (rows may be strided), slots int32 [N,k] and gates fp32 [N,k] of a Route (gates None: 1, which makes it
    the gradient of the gather by Route.rows).  Slots outside [0, P) add nothing.  Not recorded by
    autograd: submconv_combine_backward gives the gradients."""
    dev = _strided(y, "y", 2).device
    np_, c = y.shape
    if slots.dim() != 2:
        raise ValueError("slots must be [N,k]")
    n, k = slots.shape
    _same_device(slots, "slots", torch.int32, dev, (n, k))
    _same_device(gates, "gates", torch.float32, dev, (n, k))
    if out is None:
        out = torch.empty((n, c), dtype=y.dtype, device=dev)
    elif tuple(_strided(out, "out", 2, dev, y.dtype).shape) != (n, c):
        raise ValueError("out must be [N,C]")
    lib = _lib if _lib is not None else load_library()
    with _on_device(dev):
        _check(lib.submconv_combine(y.data_ptr(), _row_stride(y), np_, slots.data_ptr(), _ptr(gates), n, k, c, _dtype_code(y),
                                    out.data_ptr(), _row_stride(out), _raw_stream(dev.index)), "submconv_combine")
    return out


def submconv_combine_backward(grad: torch.Tensor, y: torch.Tensor, slots: torch.Tensor, rows: torch.Tensor,
                              gates: Optional[torch.Tensor] = None, need_y: bool = True):
    """Gradients of submconv_combine from grad [N,C] -> (dy, dgates): dy[slots[i,j]] = gates[i,j] grad[i],
    dgates[i,j] = grad[i] . y[slots[i,j]] (None without gates).

    rows int32 [P] is the Route's: position p of dy belongs to row rows[p], and gets zeros if that row does not
    name it among its slots."""
    dev = _strided(y, "y", 2).device
    np_, c = y.shape
    if slots.dim() != 2:
        raise ValueError("slots must be [N,k]")
    n, k = slots.shape
    _same_device(slots, "slots", torch.int32, dev, (n, k))
    _same_device(rows, "rows", torch.int32, dev, (np_,))
    _same_device(gates, "gates", torch.float32, dev, (n, k))
    if tuple(_strided(grad, "grad", 2, dev, y.dtype).shape) != (n, c):
        raise ValueError("grad must be [N,C]")
    dy = torch.empty((np_, c), dtype=y.dtype, device=dev) if need_y else None
    dgates = torch.empty((n, k), dtype=torch.float32, device=dev) if gates is not None else None
    lib = _lib if _lib is not None else load_library()
    with _on_device(dev):
        _check(lib.submconv_combine_backward(
            grad.data_ptr(), _row_stride(grad), y.data_ptr(), _row_stride(y), np_, slots.data_ptr(), rows.data_ptr(), _ptr(gates), n,
            k, c, _dtype_code(y), _ptr(dy), c, _ptr(dgates), _raw_stream(dev.index)), "submconv_combine_backward")
    return dy, dgates


def release_cache(device: int = -1) -> None:
    """Return the device blocks the library keeps for reuse (all devices when -1)."""
    _check(load_library().submconv_release_cache(int(device)), "submconv_release_cache")


def set_cache_limit(nbytes: int) -> None:
    """Per-device limit of the library's block cache in bytes (0: no caching)."""
    _check(load_library().submconv_set_cache_limit(int(nbytes)), "submconv_set_cache_limit")
