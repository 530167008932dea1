"""Python binding of the C ABI in include/pulsar.h (argument marshalling only).

Every step of the rendering path runs in the CUDA kernels of libpulsar.so.
There is no CPU fallback: if the library is missing, loading raises.
PyTorch is used only for device memory and streams.

Functions mirror the C entry points:
    create, destroy, project, bin, forward, backward, status, strerror,
    debug_copy
and, for the learned parts around the renderer (codebook embedding, group
norm, orthogonalised updates), the Learner class and the *_workspace
functions.
Tensor arguments are CUDA torch tensors (float32, contiguous) or raw device
pointers (int); streams are torch.cuda.Stream objects, raw handles (int) or
None for the current torch stream.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpulsar.so")

OK, ERR_ARG, ERR_CUDA, ERR_CAPACITY, ERR_STATE, ERR_NOMEM, ERR_TIMEOUT = 0, -1, -2, -3, -4, -5, -6
ERR_INTERNAL = -7   # debug build: a device index check failed
ERR_WORKSPACE, ERR_INDEX = -8, -9
FLAG_GEOM_CUTOFF = 0x1
FLAG_COUNT_HITS = 0x2
FLAG_NORMALIZE_GRADS = 0x4
FLAG_GAUSSIAN = 0x8
DBG = dict(records=1, tile_offsets=5, tile_ids=6, mg=7, wsum=8, ids=9, nhits=10)

_lib = None


class PulsarError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


class Camera(ctypes.Structure):
    _fields_ = [("R", ctypes.c_float * 9), ("t", ctypes.c_float * 3),
                ("fx", ctypes.c_float), ("fy", ctypes.c_float), ("cx", ctypes.c_float),
                ("cy", ctypes.c_float), ("width", ctypes.c_int32), ("height", ctypes.c_int32),
                ("znear", ctypes.c_float), ("zfar", ctypes.c_float),
                ("orthographic", ctypes.c_int32)]


class Params(ctypes.Structure):
    _fields_ = [("gamma", ctypes.c_float), ("bg_eps", ctypes.c_float),
                ("stop_tau", ctypes.c_float), ("kappa", ctypes.c_float),
                ("geom_min_area", ctypes.c_float), ("n_track", ctypes.c_int32),
                ("channels", ctypes.c_int32), ("flags", ctypes.c_uint32)]


EXPORTS = ("pulsar_create", "pulsar_create_cams", "pulsar_destroy", "pulsar_project",
           "pulsar_project_cams", "pulsar_bin", "pulsar_shade_forward", "pulsar_shade_backward",
           "pulsar_forward", "pulsar_backward", "pulsar_status", "pulsar_strerror",
           "pulsar_debug_copy", "pulsar_debug_inject", "pulsar_render_noalloc",
           "pulsar_learn_create", "pulsar_learn_destroy", "pulsar_learn_status",
           "pulsar_embed_workspace", "pulsar_group_norm_workspace",
           "pulsar_orthogonalize_workspace", "pulsar_embed_forward", "pulsar_embed_backward",
           "pulsar_group_norm_forward", "pulsar_group_norm_backward", "pulsar_orthogonalize")


def load(path: str = LIB_PATH):
    """Load libpulsar.so and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m splat_rendering_gb300.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.pulsar_create.argtypes = [ctypes.POINTER(P), ctypes.c_int, I64, I64, I32, I32, I32, I32]
    lib.pulsar_create_cams.argtypes = [ctypes.POINTER(P), ctypes.c_int, I64, I64, I32, I32, I32,
                                       I32, I32]
    lib.pulsar_destroy.argtypes = [P]
    lib.pulsar_project.argtypes = [P, P, P, P, I64, ctypes.POINTER(Camera),
                                   ctypes.POINTER(Params), P]
    lib.pulsar_project_cams.argtypes = [P, P, P, P, I64, ctypes.POINTER(Camera), I32,
                                        ctypes.POINTER(Params), P]
    lib.pulsar_bin.argtypes = [P, P]
    lib.pulsar_shade_forward.argtypes = [P, P, P, P, P]
    lib.pulsar_shade_backward.argtypes = [P] * 7
    lib.pulsar_forward.argtypes = [P, P, P, P, P]
    lib.pulsar_backward.argtypes = [P] + [P] * 9 + [P]
    lib.pulsar_status.argtypes = [P, P, ctypes.POINTER(I64), ctypes.POINTER(I64)]
    lib.pulsar_strerror.argtypes = [ctypes.c_int]
    lib.pulsar_strerror.restype = ctypes.c_char_p
    lib.pulsar_debug_copy.argtypes = [P, ctypes.c_int, P, I64, P]
    lib.pulsar_debug_inject.argtypes = [P, ctypes.c_int, P]
    lib.pulsar_debug_copy.restype = I64
    lib.pulsar_render_noalloc.argtypes = [P, P, P, P, I64, ctypes.POINTER(Camera),
                                          ctypes.POINTER(Params), P, P, P]
    I, F = ctypes.c_int, ctypes.c_float
    lib.pulsar_learn_create.argtypes = [ctypes.POINTER(P), I, I64]
    lib.pulsar_learn_destroy.argtypes = [P]
    lib.pulsar_learn_status.argtypes = [P, P]
    lib.pulsar_embed_workspace.argtypes = [I64, I64, I64]
    lib.pulsar_group_norm_workspace.argtypes = [I64, I64, I32, I32]
    lib.pulsar_orthogonalize_workspace.argtypes = [I64, I64, I64, I]
    workspaces = ("pulsar_embed_workspace", "pulsar_group_norm_workspace",
                  "pulsar_orthogonalize_workspace")
    for name in workspaces:
        getattr(lib, name).restype = I64
    lib.pulsar_embed_forward.argtypes = [P, P, P, I64, I64, I64, F, I, I, P, P]
    lib.pulsar_embed_backward.argtypes = [P, P, P, I64, I64, I64, F, I, I, P, P]
    lib.pulsar_group_norm_forward.argtypes = [P, P, I64, I64, I32, I32, P, P, F, I, I, P, P, P]
    lib.pulsar_group_norm_backward.argtypes = [P, P, P, P, I64, I64, I32, I32, P, P, I, I, P, P, P,
                                               P]
    lib.pulsar_orthogonalize.argtypes = [P, P, I64, I64, I64, I, P, F, I, P, P]
    for name in EXPORTS:
        if name not in ("pulsar_strerror", "pulsar_debug_copy") + workspaces:
            getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


def strerror(code: int) -> str:
    return load().pulsar_strerror(int(code)).decode()


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if isinstance(x, np.ndarray):
        return x.ctypes.data
    raise TypeError(f"cannot pass {type(x)} as a pointer")


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _empty(shape, device: int, dtype, stream):
    """A new tensor for a call on `stream` (None: the current one).  It comes
    from that stream's own memory: a block of another stream may still be in
    use there, and would be handed out again without waiting for this call."""
    import torch
    if stream is None or _stream(stream) == torch.cuda.current_stream(device).cuda_stream:
        return torch.empty(shape, device=f"cuda:{device}", dtype=dtype)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else \
            torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, device=f"cuda:{device}", dtype=dtype)


def _check(code: int, what: str):
    if code != OK:
        raise PulsarError(code, what)


def camera(cam) -> Camera:
    """Camera struct from any object with R, t, fx, fy, cx, cy, width, height,
    znear, zfar attributes (and optionally orthographic)."""
    c = Camera()
    c.R[:] = [float(v) for v in np.asarray(cam.R, np.float32).reshape(9)]
    c.t[:] = [float(v) for v in np.asarray(cam.t, np.float32).reshape(3)]
    for k in ("fx", "fy", "cx", "cy", "znear", "zfar"):
        setattr(c, k, float(getattr(cam, k)))
    c.width, c.height = int(cam.width), int(cam.height)
    c.orthographic = 1 if getattr(cam, "orthographic", False) else 0
    return c


def params(p, count_hits: bool = False) -> Params:
    """Params struct from any object with gamma, bg_eps, stop_tau, kappa,
    geom_min_area, n_track, channels, geom_cutoff (and optionally
    normalize_grads, gaussian) attributes."""
    q = Params()
    q.gamma, q.bg_eps, q.stop_tau = float(p.gamma), float(p.bg_eps), float(p.stop_tau)
    q.kappa, q.geom_min_area = float(p.kappa), float(p.geom_min_area)
    q.n_track, q.channels = int(p.n_track), int(p.channels)
    q.flags = (FLAG_GEOM_CUTOFF if getattr(p, "geom_cutoff", True) else 0) | \
              (FLAG_COUNT_HITS if count_hits else 0) | \
              (FLAG_NORMALIZE_GRADS if getattr(p, "normalize_grads", False) else 0) | \
              (FLAG_GAUSSIAN if getattr(p, "gaussian", False) else 0)
    return q


# ------------------------------------------------------------ C entry points --
def create(device: int, max_spheres: int, max_pairs: int, max_width: int, max_height: int,
           max_channels: int, max_track: int, max_cams: int = 1) -> int:
    h = ctypes.c_void_p()
    if max_cams == 1:
        _check(load().pulsar_create(ctypes.byref(h), device, max_spheres, max_pairs, max_width,
                                    max_height, max_channels, max_track), "pulsar_create")
    else:
        _check(load().pulsar_create_cams(ctypes.byref(h), device, max_spheres, max_pairs,
                                         max_width, max_height, max_channels, max_track,
                                         max_cams), "pulsar_create_cams")
    return h.value


def destroy(ctx: int):
    _check(load().pulsar_destroy(ctx), "pulsar_destroy")


def project(ctx, pos, radius, opacity, n: int, cam: Camera, prm: Params, stream=None):
    _check(load().pulsar_project(ctx, _ptr(pos), _ptr(radius), _ptr(opacity), int(n),
                                 ctypes.byref(cam), ctypes.byref(prm), _stream(stream)),
           "pulsar_project")


def project_cams(ctx, pos, radius, opacity, n: int, cams, prm: Params, stream=None):
    """Project the spheres for a batch of cameras (list of Camera structs)."""
    arr = (Camera * len(cams))(*cams)
    _check(load().pulsar_project_cams(ctx, _ptr(pos), _ptr(radius), _ptr(opacity), int(n), arr,
                                      len(cams), ctypes.byref(prm), _stream(stream)),
           "pulsar_project_cams")


def shade_forward(ctx, features, params, rgb, stream=None):
    """Per-pixel shading MLP of the frame's feature images (see
    pulsar_shade_forward in include/pulsar.h)."""
    _check(load().pulsar_shade_forward(ctx, _ptr(features), _ptr(params), _ptr(rgb),
                                       _stream(stream)), "pulsar_shade_forward")


def shade_backward(ctx, features, params, grad_rgb, grad_features, grad_params, stream=None):
    """Gradients of the shading MLP (see pulsar_shade_backward in
    include/pulsar.h); grad_features may be None."""
    _check(load().pulsar_shade_backward(ctx, _ptr(features), _ptr(params), _ptr(grad_rgb),
                                        _ptr(grad_features), _ptr(grad_params),
                                        _stream(stream)), "pulsar_shade_backward")


def bin(ctx, stream=None):  # noqa: A001  (same name as the C entry point)
    _check(load().pulsar_bin(ctx, _stream(stream)), "pulsar_bin")


def forward(ctx, features, bg, image, stream=None):
    _check(load().pulsar_forward(ctx, _ptr(features), _ptr(bg), _ptr(image), _stream(stream)),
           "pulsar_forward")


def backward(ctx, features, bg, image, grad_image, grad_pos=None, grad_radius=None,
             grad_opacity=None, grad_features=None, grad_cam=None, stream=None):
    _check(load().pulsar_backward(ctx, _ptr(features), _ptr(bg), _ptr(image), _ptr(grad_image),
                                  _ptr(grad_pos), _ptr(grad_radius), _ptr(grad_opacity),
                                  _ptr(grad_features), _ptr(grad_cam), _stream(stream)),
           "pulsar_backward")


def status(ctx, stream=None, raise_on_error: bool = True):
    """(code, n_pairs, n_hits) after synchronising the stream."""
    m, h = ctypes.c_int64(), ctypes.c_int64()
    code = load().pulsar_status(ctx, _stream(stream), ctypes.byref(m), ctypes.byref(h))
    if raise_on_error:
        _check(code, "pulsar_status")
    return code, m.value, h.value


def render_noalloc(pos, radius, opacity, features, n: int, cam: Camera, prm: Params, bg, image,
                   stream=None):
    """Forward render of a small frame without any memory allocation (see
    pulsar_render_noalloc in include/pulsar.h for its limits).  For callers
    that cannot allocate device memory at render time; synchronises the stream."""
    _check(load().pulsar_render_noalloc(_ptr(pos), _ptr(radius), _ptr(opacity), _ptr(features),
                                        int(n), ctypes.byref(cam), ctypes.byref(prm), _ptr(bg),
                                        _ptr(image), _stream(stream)), "pulsar_render_noalloc")


def debug_copy(ctx, what: str, stream=None) -> np.ndarray:
    """Copy an internal array of the last frame to a numpy array (raw bytes)."""
    lib = load()
    size = lib.pulsar_debug_copy(ctx, DBG[what], None, 0, _stream(stream))
    if size < 0:
        raise PulsarError(int(size), "pulsar_debug_copy")
    buf = np.empty(max(size, 1), np.uint8)
    code = lib.pulsar_debug_copy(ctx, DBG[what], buf.ctypes.data_as(ctypes.c_void_p), size,
                                 _stream(stream))
    _check(int(code), "pulsar_debug_copy")
    return buf[:size]


# ---------------------------------------------------------------- helper --
class Renderer:
    """One context and its call sequence for torch tensors on one device.

        r = Renderer(max_spheres=..., max_pairs=..., max_width=..., max_height=...)
        image = r.render(pos, radius, opacity, features, cam, prm, bg)
        grads = r.backward(grad_image)
    """

    def __init__(self, max_spheres: int, max_pairs: int, max_width: int, max_height: int,
                 max_channels: int = 3, max_track: int = 8, device: int = 0,
                 max_cams: int = 1):
        self.device = device
        self.ctx = create(device, max_spheres, max_pairs, max_width, max_height, max_channels,
                          max_track, max_cams)
        self._frame = None

    def close(self):
        if self.ctx:
            destroy(self.ctx)
            self.ctx = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def render(self, pos, radius, opacity, features, cam, prm: Params, bg, image=None,
               stream=None):
        """Render one camera (a Camera struct; image [H,W,C]) or a batch (a list
        of Camera structs of equal size; image [K,H,W,C])."""
        import torch
        n = int(pos.shape[0])
        C = int(prm.channels)
        batch = isinstance(cam, (list, tuple))
        first = cam[0] if batch else cam
        shape = ((len(cam),) if batch else ()) + (first.height, first.width, C)
        if image is None:
            image = _empty(shape, self.device, torch.float32, stream)
        if batch:
            project_cams(self.ctx, pos, radius, opacity, n, list(cam), prm, stream)
        else:
            project(self.ctx, pos, radius, opacity, n, cam, prm, stream)
        bin(self.ctx, stream)
        forward(self.ctx, features, bg, image, stream)
        self._frame = (pos, features, bg, image, n, C, len(cam) if batch else 0)
        return image

    def backward(self, grad_image, want=("pos", "radius", "opacity", "features", "cam"),
                 out=None, stream=None):
        import torch
        pos, features, bg, image, n, C, K = self._frame
        if out is None:
            out = {}
            shapes = dict(pos=(n, 3), radius=(n,), opacity=(n,), features=(n, C),
                          cam=(K, 16) if K else (16,))
            for k in want:
                out[k] = _empty(shapes[k], self.device, torch.float32, stream)
        backward(self.ctx, features, bg, image, grad_image, out.get("pos"), out.get("radius"),
                 out.get("opacity"), out.get("features"), out.get("cam"), stream)
        return out

    def shade(self, features, params, rgb=None, stream=None):
        """RGB of the per-pixel shading MLP over feature images [..., H, W, 16]
        of the current frame's camera(s)."""
        import torch
        if rgb is None:
            rgb = _empty(tuple(features.shape[:-1]) + (3,), self.device, torch.float32, stream)
        shade_forward(self.ctx, features, params, rgb, stream)
        return rgb

    def shade_backward(self, features, params, grad_rgb, grad_features=None, grad_params=None,
                       stream=None):
        """(dL/dfeatures, dL/dparams) of the shading for dL/drgb."""
        if grad_features is None:
            grad_features = _empty(features.shape, self.device, features.dtype, stream)
        if grad_params is None:
            grad_params = _empty(params.shape, self.device, params.dtype, stream)
        shade_backward(self.ctx, features, params, grad_rgb, grad_features, grad_params, stream)
        return grad_features, grad_params

    def status(self, stream=None, raise_on_error: bool = True):
        return status(self.ctx, stream, raise_on_error)

    def debug(self, what: str, stream=None) -> np.ndarray:
        return debug_copy(self.ctx, what, stream)


INJECT_SHADE_TIMEOUT = 1


def debug_inject(ctx, what: int, stream=None):
    """Arm a test failure (see pulsar_debug_inject in include/pulsar.h)."""
    _check(load().pulsar_debug_inject(ctx, int(what), _stream(stream)), "pulsar_debug_inject")


# ---------------------------------------------------------- learned parts --
ACT = dict(none=0, silu=1, relu=2)


_CODES = {}   # torch's types by what they can be: filled on first use (torch is imported late)


def _code(dtype, kind: str) -> int:
    if not _CODES:
        import torch
        _CODES.update(value={torch.float32: 0, torch.bfloat16: 1},
                      index={torch.int32: 0, torch.int64: 1})
    code = _CODES[kind].get(dtype)
    if code is None:
        raise TypeError(f"{' or '.join(str(t) for t in _CODES[kind])} is wanted, got {dtype}")
    return code


def _dtype_code(dtype) -> int:
    return _code(dtype, "value")


def _index_code(dtype) -> int:
    return _code(dtype, "index")


def _bytes(code: int, what: str) -> int:
    if code < 0:
        raise PulsarError(int(code), what)
    return int(code)


@functools.lru_cache(maxsize=1024)   # a function of the sizes alone
def embed_workspace(n: int, rows: int, dim: int) -> int:
    """Bytes of workspace of Learner.embed_backward for n tokens."""
    return _bytes(load().pulsar_embed_workspace(n, rows, dim), "pulsar_embed_workspace")


@functools.lru_cache(maxsize=1024)   # a function of the sizes alone
def group_norm_workspace(images: int, pixels: int, channels: int, groups: int) -> int:
    """Bytes of workspace of Learner.group_norm and group_norm_backward."""
    return _bytes(load().pulsar_group_norm_workspace(images, pixels, channels, groups),
                  "pulsar_group_norm_workspace")


@functools.lru_cache(maxsize=1024)   # a function of the sizes alone
def orthogonalize_workspace(batch: int, m: int, n: int, dtype) -> int:
    """Bytes of workspace of Learner.orthogonalize for `batch` m x n matrices."""
    return _bytes(load().pulsar_orthogonalize_workspace(batch, m, n, _dtype_code(dtype)),
                  "pulsar_orthogonalize_workspace")


class Learner:
    """A handle for the learned parts around the renderer, and its calls on
    torch tensors of one device (see include/pulsar.h for what they compute).

        ops = Learner(workspace_bytes=embed_workspace(n, rows, dim))
        features = ops.embed(codebook, tokens)          # -> Renderer.render
        y, stats = ops.group_norm(image, groups, weight, bias, act="silu")
        grad_image, gw, gb = ops.group_norm_backward(grad_y, image, stats, groups, weight, bias)
        grad_codebook = ops.embed_backward(grad_features, tokens, rows)
        update = ops.orthogonalize(grad_matrix)

    Tensors are contiguous and on the handle's device; anything else raises
    before a kernel is launched.  Outputs are allocated unless given, from the
    memory of the stream that the call runs on."""

    def __init__(self, workspace_bytes: int, device: int = 0):
        import torch
        self.device, self.workspace_bytes = int(device), int(workspace_bytes)
        self.handle = 0
        self._lib = load()
        # a call costs a few microseconds of host time: keep what it looks up
        self._torch, self._dev = torch, torch.device("cuda", self.device)
        self._current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
        h = ctypes.c_void_p()
        _check(self._lib.pulsar_learn_create(ctypes.byref(h), self.device, self.workspace_bytes),
               "pulsar_learn_create")
        self.handle = h.value

    def close(self):
        if self.handle:
            _check(load().pulsar_learn_destroy(self.handle), "pulsar_learn_destroy")
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def status(self, stream=None, raise_on_error: bool = True) -> int:
        """Synchronise the stream and report the latched device error."""
        code = self._lib.pulsar_learn_status(self.handle, self._stream(stream))
        if raise_on_error:
            _check(code, "pulsar_learn_status")
        return code

    def _stream(self, s):
        return self._current_stream(self.device) if s is None else _stream(s)

    def _tensor(self, t, what: str, shape=None, dtype=None):
        """Checks a tensor argument and returns its pointer (None stays None)."""
        if t is None:
            return None
        if t.get_device() != self.device:   # (-1 on the host)
            raise ValueError(f"{what} is not on cuda:{self.device}")
        if not t.is_contiguous():
            raise ValueError(f"{what} is not contiguous")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{what} has shape {tuple(t.shape)}, wanted {tuple(shape)}")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{what} is {t.dtype}, wanted {dtype}")
        return t.data_ptr()

    def _out(self, t, what: str, shape, dtype, stream):
        """An output and its pointer: `t` checked, or where it is None a new one."""
        if t is None:
            t = self._torch.empty(shape, device=self._dev, dtype=dtype) if stream is None else \
                _empty(shape, self.device, dtype, stream)
            return t, t.data_ptr()
        return t, self._tensor(t, what, shape, dtype)

    @staticmethod
    def _product(shape):
        n = 1
        for d in shape:
            n *= d
        return n

    def embed(self, table, tokens, scale: float = 1.0, out=None, stream=None):
        """scale * table[tokens] ([*tokens.shape, dim]); zeros where a token is negative."""
        if table.dim() != 2:
            raise ValueError(f"table has shape {tuple(table.shape)}, wanted [rows, dim]")
        rows, dim = table.shape
        shape = (*tokens.shape, dim)
        dt, ix = _dtype_code(table.dtype), _index_code(tokens.dtype)
        out, p_out = self._out(out, "out", shape, table.dtype, stream)
        _check(self._lib.pulsar_embed_forward(
            self.handle, self._tensor(table, "table"), self._tensor(tokens, "tokens"),
            tokens.numel(), rows, dim, scale, dt, ix, p_out, self._stream(stream)),
            "pulsar_embed_forward")
        return out

    def embed_backward(self, grad_out, tokens, rows: int, scale: float = 1.0, grad_table=None,
                       stream=None):
        """Gradient [rows, dim] of `embed` for grad_out [*tokens.shape, dim]."""
        if grad_out.shape[:-1] != tokens.shape:
            raise ValueError(f"grad_out has shape {tuple(grad_out.shape)}, wanted "
                             f"{tuple(tokens.shape) + ('dim',)}")
        dim = grad_out.shape[-1]
        dt, ix = _dtype_code(grad_out.dtype), _index_code(tokens.dtype)
        grad_table, p_table = self._out(grad_table, "grad_table", (rows, dim), grad_out.dtype, stream)
        _check(self._lib.pulsar_embed_backward(
            self.handle, self._tensor(grad_out, "grad_out"), self._tensor(tokens, "tokens"),
            tokens.numel(), rows, dim, scale, dt, ix, p_table, self._stream(stream)),
            "pulsar_embed_backward")
        return grad_table

    def _image_shape(self, x, act):
        shape = x.shape
        if len(shape) < 2:
            raise ValueError(f"x has shape {tuple(shape)}, wanted [images, ..., channels]")
        a = ACT.get(act)
        if a is None:
            raise ValueError(f"act is one of {sorted(ACT)}, got {act!r}")
        return shape, shape[0], self._product(shape[1:-1]), shape[-1], a

    def group_norm(self, x, groups: int, weight=None, bias=None, eps: float = 1e-5,
                   act: str = "none", out=None, stats=None, stream=None):
        """(y, stats): act(group norm) of x [images, ..., channels], channels
        last, and the (mean, 1/std) [images, groups, 2] its backward needs."""
        shape, images, pixels, C, a = self._image_shape(x, act)
        dt, f32 = _dtype_code(x.dtype), self._torch.float32
        out, p_out = self._out(out, "out", shape, x.dtype, stream)
        stats, p_stats = self._out(stats, "stats", (images, groups, 2), f32, stream)
        _check(self._lib.pulsar_group_norm_forward(
            self.handle, self._tensor(x, "x"), images, pixels, C, groups,
            self._tensor(weight, "weight", (C,), f32), self._tensor(bias, "bias", (C,), f32),
            eps, a, dt, p_out, p_stats, self._stream(stream)), "pulsar_group_norm_forward")
        return out, stats

    def group_norm_backward(self, grad_y, x, stats, groups: int, weight=None, bias=None,
                            act: str = "none", grad_x=None, grad_weight=None, grad_bias=None,
                            want=("x", "weight", "bias"), stream=None):
        """(grad_x, grad_weight, grad_bias) of `group_norm`; those not in
        `want` (and not given) are None and not computed."""
        shape, images, pixels, C, a = self._image_shape(x, act)
        dt, f32 = _dtype_code(x.dtype), self._torch.float32
        p_x = p_weight = p_bias = None
        if grad_x is not None or "x" in want:
            grad_x, p_x = self._out(grad_x, "grad_x", shape, x.dtype, stream)
        if grad_weight is not None or "weight" in want:
            grad_weight, p_weight = self._out(grad_weight, "grad_weight", (C,), f32, stream)
        if grad_bias is not None or "bias" in want:
            grad_bias, p_bias = self._out(grad_bias, "grad_bias", (C,), f32, stream)
        _check(self._lib.pulsar_group_norm_backward(
            self.handle, self._tensor(grad_y, "grad_y", shape, x.dtype), self._tensor(x, "x"),
            self._tensor(stats, "stats", (images, groups, 2), f32), images, pixels, C, groups,
            self._tensor(weight, "weight", (C,), f32), self._tensor(bias, "bias", (C,), f32), a, dt,
            p_x, p_weight, p_bias, self._stream(stream)), "pulsar_group_norm_backward")
        return grad_x, grad_weight, grad_bias

    def orthogonalize(self, grad, steps: int = 5, coeffs=(3.4445, -4.775, 2.0315),
                      eps: float = 1e-7, out=None, stream=None):
        """`steps` Newton-Schulz products on each matrix of grad [..., m, n].
        In bfloat16 the iterates are rounded to 11 bits in every step, in
        float32 to 22 (include/pulsar.h says how far off that leaves the
        result); convert the matrix first where 16 bits want more."""
        shape = grad.shape
        if len(shape) < 2:
            raise ValueError(f"grad has shape {tuple(shape)}, wanted [..., m, n]")
        dt = _dtype_code(grad.dtype)
        out, p_out = self._out(out, "out", shape, grad.dtype, stream)
        if len(coeffs) != 3:
            raise ValueError(f"coeffs are (a, b, c), got {len(coeffs)} values")
        abc = (ctypes.c_float * 3)(*[float(v) for v in coeffs])
        _check(self._lib.pulsar_orthogonalize(
            self.handle, self._tensor(grad, "grad"), self._product(shape[:-2]), shape[-2], shape[-1],
            steps, abc, eps, dt, p_out, self._stream(stream)), "pulsar_orthogonalize")
        return out
