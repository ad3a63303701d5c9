"""ctypes binding of libgconv.so (the C ABI declared in include/gconv.h).

Argument marshalling only: tensors must already be float32, contiguous and on
the GPU (the sequence operators at the end also take bfloat16, and strides
where they say so); outputs and the workspace are allocated here with torch (device
memory is torch's), and every op is enqueued on torch's current HIP stream.
Nothing is computed in Python or by torch. When the library is missing the
first call raises; there is no fallback.

Names mirror the C entry points: gconv_fwd, gconv_bwd_data, gconv_bwd_filter,
gconv_bwd_bias, gconv_output_dims, gconv_workspace_size, gconv_select_path,
gconv_set_path_override; gconv_linattn_fwd, gconv_linattn_bwd,
gconv_linattn_step, gconv_normgate_fwd, gconv_normgate_bwd, gconv_orthogonalize,
gconv_shortconv_fwd, gconv_shortconv_bwd, gconv_shortconv_step, gconv_scan_fwd,
gconv_scan_bwd, gconv_scan_step, gconv_embed_fwd, gconv_embed_bwd,
gconv_xent_fwd, gconv_xent_bwd.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgconv.so")

OK = 0
STATUS = {0: "GCONV_OK", 1: "GCONV_ERR_NULL", 2: "GCONV_ERR_SHAPE", 3: "GCONV_ERR_GROUPS",
          4: "GCONV_ERR_WORKSPACE", 5: "GCONV_ERR_HIP", 6: "GCONV_ERR_UNSUPPORTED",
          7: "GCONV_ERR_ARG"}
OP_FWD, OP_BWD_DATA, OP_BWD_FILTER, OP_BWD_BIAS = 0, 1, 2, 3
PATH_AUTO, PATH_DIRECT, PATH_SMALLGROUP, PATH_IGEMM, PATH_FC, PATH_POINTWISE = 0, 1, 2, 3, 4, 5
EPILOGUE_NONE, EPILOGUE_RELU = 0, 1
LAYOUT_NCHW, LAYOUT_NHWC = 0, 1
F32, BF16 = 0, 1
LINATTN_FWD, LINATTN_BWD = 0, 1
SCAN_FWD, SCAN_BWD = 0, 1
XENT_FWD, XENT_BWD = 0, 1
I32, I64 = 0, 1
GATE_NONE, GATE_FULL, GATE_SEQUENCE = 0, 1, 2
ACTS = {"none": 0, "sigmoid": 1, "silu": 2}
PATH_NAMES = {PATH_AUTO: "auto", PATH_DIRECT: "direct", PATH_SMALLGROUP: "smallgroup",
              PATH_IGEMM: "igemm", PATH_FC: "fc", PATH_POINTWISE: "pointwise"}

# Every symbol include/gconv.h declares.
EXPORTS = ("gconv_output_dims", "gconv_workspace_size", "gconv_fwd", "gconv_fwd_ex", "gconv_bwd_data",
           "gconv_bwd_filter", "gconv_bwd_filter_static", "gconv_bwd_bias", "gconv_select_path",
           "gconv_set_path_override", "gconv_status_string", "gconv_last_error", "gconv_version",
           "gconv_linattn_workspace_size", "gconv_linattn_fwd", "gconv_linattn_bwd", "gconv_linattn_step",
           "gconv_normgate_workspace_size", "gconv_normgate_fwd", "gconv_normgate_bwd",
           "gconv_orthogonalize_workspace_size", "gconv_orthogonalize",
           "gconv_shortconv_workspace_size", "gconv_shortconv_fwd", "gconv_shortconv_bwd", "gconv_shortconv_step",
           "gconv_scan_workspace_size", "gconv_scan_fwd", "gconv_scan_bwd", "gconv_scan_step",
           "gconv_embed_workspace_size", "gconv_embed_fwd", "gconv_embed_bwd", "gconv_xent_workspace_size", "gconv_xent_fwd",
           "gconv_xent_bwd")


class GconvError(RuntimeError):
    def __init__(self, status: int, func: str, detail: str):
        self.status = status
        super().__init__("%s failed: %s (%s): %s" % (func, STATUS.get(status, status),
                                                     _status_string(status), detail))


class gconv_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "N", "C", "H", "W", "K", "kh", "kw", "stride_h", "stride_w", "pad_h", "pad_w",
        "dil_h", "dil_w", "groups", "pad_h_extra", "pad_w_extra", "layout")]


class gconv_linattn_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("dtype", "packed", "sequences", "tokens", "heads",
                                               "kv_heads", "dk", "dv")] +
                [(n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "v_stride", "do_stride")] +
                [("scale", ctypes.c_double)])


class gconv_normgate_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("dtype", "sequences", "tokens", "dim", "gate", "act")] +
                [(n, ctypes.c_int64 * 2) for n in ("x_stride", "b_stride", "gate_stride", "dy_stride", "dh_stride")] +
                [("eps", ctypes.c_double)])


class gconv_ortho_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("dtype", "filters", "inner", "groups", "steps")] +
                [("eps", ctypes.c_double)])


class gconv_shortconv_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("dtype", "packed", "sequences", "tokens", "dim", "taps", "act")] +
                [(n, ctypes.c_int64 * 2) for n in ("x_stride", "dy_stride")])


class gconv_scan_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("dtype", "packed", "sequences", "tokens", "dim", "states", "groups", "softplus")] +
                [(n, ctypes.c_int64 * 2) for n in ("u_stride", "dt_stride", "gate_stride")] +
                [(n, ctypes.c_int64 * 3) for n in ("b_stride", "c_stride")] + [("dy_stride", ctypes.c_int64 * 2)])


class gconv_embed_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("dtype", "index", "sequences", "tokens", "rows", "dim")] +
                [("dy_stride", ctypes.c_int64 * 2), ("scale", ctypes.c_double)])


class gconv_xent_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("dtype", "index", "sequences", "tokens", "vocab", "dim")] +
                [("h_stride", ctypes.c_int64 * 2), ("scale", ctypes.c_double)])


_lib = None


def load(path: str = LIB_PATH):
    """Load libgconv.so and declare its signatures (once per process)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libgconv.so is not built (expected at %s); run "
                           "`python -m grouped_convolution_amd.build`" % path)
    lib = ctypes.CDLL(path)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    D = ctypes.POINTER(gconv_desc)
    i64p = ctypes.POINTER(ctypes.c_int64)
    sig = {
        "gconv_output_dims": [D, i64p, i64p],
        "gconv_workspace_size": [D, I, ctypes.POINTER(ctypes.c_size_t)],
        "gconv_fwd": [D, P, P, P, P, P, S, P],
        "gconv_fwd_ex": [D, P, P, P, I, P, P, S, P],
        "gconv_bwd_data": [D, P, P, P, P, S, P],
        "gconv_bwd_filter": [D, P, P, P, P, S, P],
        "gconv_bwd_filter_static": [D, P, P, P, P],
        "gconv_bwd_bias": [D, P, P, P, S, P],
        "gconv_select_path": [D, I, ctypes.POINTER(ctypes.c_int)],
        "gconv_set_path_override": [I],
        "gconv_status_string": [I],
        "gconv_last_error": [],
        "gconv_version": [],
        "gconv_linattn_workspace_size": [ctypes.POINTER(gconv_linattn_desc), I, ctypes.POINTER(S)],
        "gconv_linattn_fwd": [ctypes.POINTER(gconv_linattn_desc)] + [P] * 9 + [S, P],
        "gconv_linattn_bwd": [ctypes.POINTER(gconv_linattn_desc)] + [P] * 13 + [S, P],
        "gconv_linattn_step": [ctypes.POINTER(gconv_linattn_desc)] + [P] * 6 + [ctypes.c_int64, P, P],
        "gconv_normgate_workspace_size": [ctypes.POINTER(gconv_normgate_desc), ctypes.POINTER(S)],
        "gconv_normgate_fwd": [ctypes.POINTER(gconv_normgate_desc)] + [P] * 9,
        "gconv_normgate_bwd": [ctypes.POINTER(gconv_normgate_desc)] + [P] * 15 + [S, P],
        "gconv_orthogonalize_workspace_size": [ctypes.POINTER(gconv_ortho_desc), ctypes.POINTER(S)],
        "gconv_orthogonalize": [ctypes.POINTER(gconv_ortho_desc), P, P, P, S, P],
        "gconv_shortconv_workspace_size": [ctypes.POINTER(gconv_shortconv_desc), ctypes.POINTER(S)],
        "gconv_shortconv_fwd": [ctypes.POINTER(gconv_shortconv_desc)] + [P] * 8,
        "gconv_shortconv_bwd": [ctypes.POINTER(gconv_shortconv_desc)] + [P] * 12 + [S, P],
        "gconv_shortconv_step": [ctypes.POINTER(gconv_shortconv_desc)] + [P] * 5 + [ctypes.c_int64, P, P],
        "gconv_scan_workspace_size": [ctypes.POINTER(gconv_scan_desc), I, ctypes.POINTER(S)],
        "gconv_scan_fwd": [ctypes.POINTER(gconv_scan_desc)] + [P] * 13 + [S, P],
        "gconv_scan_bwd": [ctypes.POINTER(gconv_scan_desc)] + [P] * 22 + [S, P],
        "gconv_scan_step": [ctypes.POINTER(gconv_scan_desc)] + [P] * 10 + [ctypes.c_int64, P, P],
        "gconv_embed_workspace_size": [ctypes.POINTER(gconv_embed_desc), ctypes.POINTER(S)],
        "gconv_embed_fwd": [ctypes.POINTER(gconv_embed_desc)] + [P] * 4,
        "gconv_embed_bwd": [ctypes.POINTER(gconv_embed_desc)] + [P] * 4 + [S, P],
        "gconv_xent_workspace_size": [ctypes.POINTER(gconv_xent_desc), I, ctypes.POINTER(S)],
        "gconv_xent_fwd": [ctypes.POINTER(gconv_xent_desc)] + [P] * 6 + [S, P],
        "gconv_xent_bwd": [ctypes.POINTER(gconv_xent_desc)] + [P] * 9 + [S, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.gconv_status_string.restype = ctypes.c_char_p
    lib.gconv_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _status_string(status: int) -> str:
    return load().gconv_status_string(status).decode()


def _check(status: int, func: str):
    if status != OK:
        raise GconvError(status, func, load().gconv_last_error().decode())


def _pair(v, name):
    if isinstance(v, (tuple, list)):
        if len(v) != 2:
            raise ValueError("%s must be an int or a pair" % name)
        return int(v[0]), int(v[1])
    return int(v), int(v)


def _padding(v):
    """int, (pad_h, pad_w) or (top, bottom, left, right) -> (top, left, bottom - top, right - left)."""
    if isinstance(v, (tuple, list)) and len(v) == 4:
        t, b, l, r = (int(e) for e in v)
        return t, l, b - t, r - l
    ph, pw = _pair(v, "padding")
    return ph, pw, 0, 0


def same_padding(H, W, kh, kw, stride=1, dilation=1):
    """TensorFlow's "same" padding as (top, bottom, left, right): Ho = ceil(H / stride), the
    total padding split with the odd row or column at the end."""
    out = []
    for n, k, s, d in zip((H, W), (kh, kw), _pair(stride, "stride"), _pair(dilation, "dilation")):
        total = max((-(-n // s) - 1) * s + (k - 1) * d + 1 - n, 0)
        out += [total // 2, total - total // 2]
    return tuple(out)


def _layout(v) -> int:
    """"nchw" / "nhwc" (or LAYOUT_NCHW / LAYOUT_NHWC) -> gconv_layout."""
    if isinstance(v, str):
        key = v.lower()
        if key not in ("nchw", "nhwc"):
            raise ValueError("layout must be 'nchw' or 'nhwc', got %r" % v)
        return LAYOUT_NHWC if key == "nhwc" else LAYOUT_NCHW
    if int(v) not in (LAYOUT_NCHW, LAYOUT_NHWC):
        raise ValueError("unknown layout %r" % (v,))
    return int(v)


def make_desc(N, C, H, W, K, kh, kw, stride=1, padding=0, dilation=1, groups=1,
              layout="nchw") -> gconv_desc:
    """`padding` is an int, a pair (pad_h, pad_w) or a 4-tuple (top, bottom, left, right);
    `layout` ("nchw" or "nhwc") is that of x, dx, y and dy."""
    sh, sw = _pair(stride, "stride")
    ph, pw, eh, ew = _padding(padding)
    dh, dw = _pair(dilation, "dilation")
    return gconv_desc(int(N), int(C), int(H), int(W), int(K), int(kh), int(kw), sh, sw, ph, pw,
                      dh, dw, int(groups), eh, ew, _layout(layout))


def _act_shape(N, C, H, W, layout):
    """The 4-D shape of an activation with N images, C channels, H x W pixels."""
    return (N, H, W, C) if _layout(layout) == LAYOUT_NHWC else (N, C, H, W)


def _act_dims(shape, layout):
    """(N, C, H, W) of an activation tensor shape in `layout`."""
    N, a, b, c = (int(v) for v in shape)
    return (N, c, a, b) if _layout(layout) == LAYOUT_NHWC else (N, a, b, c)


def gconv_output_dims(desc: gconv_desc):
    ho, wo = ctypes.c_int64(), ctypes.c_int64()
    _check(load().gconv_output_dims(ctypes.byref(desc), ctypes.byref(ho), ctypes.byref(wo)),
           "gconv_output_dims")
    return ho.value, wo.value


def gconv_workspace_size(desc: gconv_desc, op: int) -> int:
    n = ctypes.c_size_t()
    _check(load().gconv_workspace_size(ctypes.byref(desc), int(op), ctypes.byref(n)),
           "gconv_workspace_size")
    return n.value


def gconv_select_path(desc: gconv_desc, op: int) -> int:
    p = ctypes.c_int()
    _check(load().gconv_select_path(ctypes.byref(desc), int(op), ctypes.byref(p)),
           "gconv_select_path")
    return p.value


def gconv_set_path_override(path: int):
    _check(load().gconv_set_path_override(int(path)), "gconv_set_path_override")


def version() -> int:
    return int(load().gconv_version())


# ---------------------------------------------------------------- tensor level

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dev_f32(t, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    if t.dtype != torch.float32:
        raise ValueError("%s must be float32, got %s" % (name, t.dtype))
    if t.device.type != "cuda":
        raise ValueError("%s must be on the GPU, got %s" % (name, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (row-major in its layout)" % name)
    return t


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(device):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _addr(t):
    """_ptr as a plain number, which ctypes takes for a pointer at less cost."""
    return t.data_ptr() if t is not None else None


def _launch(name, device, *args):
    """Calls a C entry point on `device`'s current stream, with `device` current while it launches:
    a stream that is another device's default one would otherwise stand for the current one's.
    (torch's own short ways to both, as a call's cost counts.)"""
    torch = _torch()
    entry, index = getattr(load(), name), device.index
    if torch._C._cuda_getDevice() == index:
        status = entry(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = entry(*args, torch._C._cuda_getCurrentRawStream(index))
    _check(status, name)


def _given_workspace(nbytes, device, workspace):
    """A caller's workspace and its size: `nbytes` or more, on `device`, one after another."""
    if not isinstance(workspace, _torch().Tensor):
        raise ValueError("workspace must be a torch.Tensor")
    if workspace.device != device:
        raise ValueError("workspace must be on %s, got %s" % (device, workspace.device))
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    have = workspace.numel() * workspace.element_size()
    if have < nbytes:
        raise ValueError("workspace holds %d bytes, %d needed" % (have, nbytes))
    return workspace, have


def _workspace(desc, op, device, workspace):
    n = gconv_workspace_size(desc, op)
    if n == 0:
        return None, 0
    if workspace is not None:
        return _given_workspace(n, device, workspace)
    torch = _torch()
    return torch.empty(n, dtype=torch.uint8, device=device), n


def _out(out, shape, like, name):
    torch = _torch()
    if out is None:
        return torch.empty(shape, dtype=torch.float32, device=like.device)
    _dev_f32(out, name)
    if tuple(out.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(out.shape), tuple(shape)))
    return out


def gconv_fwd(x, w, bias=None, *, stride=1, padding=0, dilation=1, groups=1, out=None,
              workspace=None, relu=False, layout="nchw"):
    """y = conv(x, w) + bias; x [N,C,H,W] (or [N,H,W,C] with layout="nhwc", giving y
    [N,Ho,Wo,K]), w [K,C/groups,kh,kw], bias [K] or None.
    With relu=True the kernels store max(y, 0) (gconv_fwd_ex, GCONV_EPILOGUE_RELU)."""
    _dev_f32(x, "x")
    _dev_f32(w, "w")
    if x.dim() != 4 or w.dim() != 4:
        raise ValueError("x and w must be 4-D (NCHW or NHWC, and [K, C/groups, kh, kw])")
    N, C, H, W = _act_dims(x.shape, layout)
    K, Cg, kh, kw = w.shape
    if groups < 1 or C % groups or Cg * groups != C:
        raise ValueError("channels_in C=%d must equal w.shape[1]*groups = %d*%d"
                         % (C, Cg, groups))
    if bias is not None:
        _dev_f32(bias, "bias")
        if tuple(bias.shape) != (K,):
            raise ValueError("bias must have shape [K]=[%d]" % K)
    desc = make_desc(N, C, H, W, K, kh, kw, stride, padding, dilation, groups, layout)
    Ho, Wo = gconv_output_dims(desc)
    y = _out(out, _act_shape(N, K, Ho, Wo, layout), x, "out")
    ws, nws = _workspace(desc, OP_FWD, x.device, workspace)
    _check(load().gconv_fwd_ex(ctypes.byref(desc), _ptr(x), _ptr(w), _ptr(bias),
                               EPILOGUE_RELU if relu else EPILOGUE_NONE, _ptr(y), _ptr(ws), nws,
                               _stream(x.device)), "gconv_fwd_ex")
    return y


def gconv_bwd_data(dy, w, x_shape, *, stride=1, padding=0, dilation=1, groups=1, out=None,
                   workspace=None, layout="nchw"):
    """gradInput [N,C,H,W] from dy [N,K,Ho,Wo] and w [K,C/groups,kh,kw] (x_shape, dy and
    the result in `layout`)."""
    _dev_f32(dy, "dy")
    _dev_f32(w, "w")
    N, C, H, W = _act_dims(x_shape, layout)
    K, Cg, kh, kw = w.shape
    if groups < 1 or Cg * groups != C:
        raise ValueError("channels_in C=%d must equal w.shape[1]*groups = %d*%d"
                         % (C, Cg, groups))
    desc = make_desc(N, C, H, W, K, kh, kw, stride, padding, dilation, groups, layout)
    Ho, Wo = gconv_output_dims(desc)
    if tuple(dy.shape) != _act_shape(N, K, Ho, Wo, layout):
        raise ValueError("dy has shape %s, expected %s"
                         % (tuple(dy.shape), _act_shape(N, K, Ho, Wo, layout)))
    dx = _out(out, _act_shape(N, C, H, W, layout), dy, "out")
    ws, nws = _workspace(desc, OP_BWD_DATA, dy.device, workspace)
    _check(load().gconv_bwd_data(ctypes.byref(desc), _ptr(dy), _ptr(w), _ptr(dx), _ptr(ws), nws,
                                 _stream(dy.device)), "gconv_bwd_data")
    return dx


def gconv_bwd_filter(x, dy, w_shape, *, stride=1, padding=0, dilation=1, groups=1, out=None,
                     workspace=None, layout="nchw"):
    """gradWeight [K,C/groups,kh,kw] from x [N,C,H,W] and dy [N,K,Ho,Wo] (x and dy in
    `layout`; overwrites)."""
    _dev_f32(x, "x")
    _dev_f32(dy, "dy")
    N, C, H, W = _act_dims(x.shape, layout)
    K, Cg, kh, kw = (int(v) for v in w_shape)
    if groups < 1 or Cg * groups != C:
        raise ValueError("channels_in C=%d must equal w_shape[1]*groups = %d*%d"
                         % (C, Cg, groups))
    desc = make_desc(N, C, H, W, K, kh, kw, stride, padding, dilation, groups, layout)
    Ho, Wo = gconv_output_dims(desc)
    if tuple(dy.shape) != _act_shape(N, K, Ho, Wo, layout):
        raise ValueError("dy has shape %s, expected %s"
                         % (tuple(dy.shape), _act_shape(N, K, Ho, Wo, layout)))
    dw = _out(out, (K, Cg, kh, kw), x, "out")
    ws, nws = _workspace(desc, OP_BWD_FILTER, x.device, workspace)
    _check(load().gconv_bwd_filter(ctypes.byref(desc), _ptr(x), _ptr(dy), _ptr(dw), _ptr(ws),
                                   nws, _stream(x.device)), "gconv_bwd_filter")
    return dw


def gconv_bwd_bias(dy, *, out=None, workspace=None, layout="nchw"):
    """gradBias [K] = sum of dy [N,K,Ho,Wo] (or [N,Ho,Wo,K]) over (n, ho, wo) (overwrites)."""
    _dev_f32(dy, "dy")
    if dy.dim() != 4:
        raise ValueError("dy must be 4-D [N, K, Ho, Wo] or [N, Ho, Wo, K]")
    N, K, Ho, Wo = _act_dims(dy.shape, layout)
    # Only N, K, Ho, Wo matter: describe dy as the output of a 1x1 conv.
    desc = make_desc(N, K, Ho, Wo, K, 1, 1, layout=layout)
    db = _out(out, (K,), dy, "out")
    ws, nws = _workspace(desc, OP_BWD_BIAS, dy.device, workspace)
    _check(load().gconv_bwd_bias(ctypes.byref(desc), _ptr(dy), _ptr(db), _ptr(ws), nws,
                                 _stream(dy.device)), "gconv_bwd_bias")
    return db


class Plan:
    """One op with its arguments marshalled once, for repeated launches.

    ``Plan.fwd(x, w, bias, y, ...)`` etc. validate exactly like the functions
    above and keep the ctypes argument tuple; calling the plan enqueues the op
    on the stream it was built with and checks the status. The tensors must
    stay alive (and keep their storage) as long as the plan is used."""

    def __init__(self, fn_name, args, keep):
        self._fn = getattr(load(), fn_name)
        self._name = fn_name
        self._args = args
        self._keep = keep

    def __call__(self):
        st = self._fn(*self._args)
        if st != OK:
            _check(st, self._name)

    @staticmethod
    def _prep(desc, op, device, workspace):
        ws, nws = _workspace(desc, op, device, workspace)
        return ws, nws, _stream(device)

    @classmethod
    def fwd(cls, x, w, bias, y, *, stride=1, padding=0, dilation=1, groups=1, workspace=None,
            relu=False, layout="nchw"):
        gconv_fwd(x, w, bias, stride=stride, padding=padding, dilation=dilation, groups=groups,
                  out=y, workspace=workspace, relu=relu, layout=layout)  # validates (and runs) once
        N, C, H, W = _act_dims(x.shape, layout)
        K, _, kh, kw = w.shape
        desc = make_desc(N, C, H, W, K, kh, kw, stride, padding, dilation, groups, layout)
        ws, nws, st = cls._prep(desc, OP_FWD, x.device, workspace)
        act = EPILOGUE_RELU if relu else EPILOGUE_NONE
        return cls("gconv_fwd_ex", (ctypes.byref(desc), _ptr(x), _ptr(w), _ptr(bias), act, _ptr(y),
                                    _ptr(ws), nws, st), (desc, x, w, bias, y, ws))

    @classmethod
    def bwd_data(cls, dy, w, dx, *, stride=1, padding=0, dilation=1, groups=1, workspace=None,
                 layout="nchw"):
        gconv_bwd_data(dy, w, dx.shape, stride=stride, padding=padding, dilation=dilation,
                       groups=groups, out=dx, workspace=workspace, layout=layout)
        N, C, H, W = _act_dims(dx.shape, layout)
        K, _, kh, kw = w.shape
        desc = make_desc(N, C, H, W, K, kh, kw, stride, padding, dilation, groups, layout)
        ws, nws, st = cls._prep(desc, OP_BWD_DATA, dy.device, workspace)
        return cls("gconv_bwd_data", (ctypes.byref(desc), _ptr(dy), _ptr(w), _ptr(dx), _ptr(ws),
                                      nws, st), (desc, dy, w, dx, ws))

    @classmethod
    def bwd_filter(cls, x, dy, dw, *, stride=1, padding=0, dilation=1, groups=1,
                   workspace=None, layout="nchw"):
        gconv_bwd_filter(x, dy, dw.shape, stride=stride, padding=padding, dilation=dilation,
                         groups=groups, out=dw, workspace=workspace, layout=layout)
        N, C, H, W = _act_dims(x.shape, layout)
        K, _, kh, kw = dw.shape
        desc = make_desc(N, C, H, W, K, kh, kw, stride, padding, dilation, groups, layout)
        ws, nws, st = cls._prep(desc, OP_BWD_FILTER, x.device, workspace)
        return cls("gconv_bwd_filter", (ctypes.byref(desc), _ptr(x), _ptr(dy), _ptr(dw),
                                        _ptr(ws), nws, st), (desc, x, dy, dw, ws))

    @classmethod
    def bwd_bias(cls, dy, db, *, workspace=None, layout="nchw"):
        gconv_bwd_bias(dy, out=db, workspace=workspace, layout=layout)
        N, K, Ho, Wo = _act_dims(dy.shape, layout)
        desc = make_desc(N, K, Ho, Wo, K, 1, 1, layout=layout)
        ws, nws, st = cls._prep(desc, OP_BWD_BIAS, dy.device, workspace)
        return cls("gconv_bwd_bias", (ctypes.byref(desc), _ptr(dy), _ptr(db), _ptr(ws), nws, st),
                   (desc, dy, db, ws))


# ---------------------------------------------------------------- sequence operators

def _seq(t, name, dtype=None, device=None):
    """A GPU tensor of float32 or bfloat16 (of `dtype`, on `device`, if given)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU, got %s" % (name, t.device))
    if device is not None and t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    return t


def _dense(t, name, shape, dtype, device):
    """A contiguous GPU tensor of one shape and type."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.device != device or not t.is_cuda:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


# What a call's descriptor and checks come to depends on its tensors' shapes, strides, types and
# devices alone, so it is kept by those: a repeated call of a decoding loop costs the host a
# lookup in place of the checks (one token 14 -> 8 us a call).
_plans = {}


def _plan(kind, tensors, numbers, make):
    """make()'s answer, kept by the layout of `tensors` and by `numbers` (plain numbers, texts or None)."""
    try:
        key = (kind, numbers, tuple([None if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in tensors]))
        plan = _plans.get(key)
    except (AttributeError, TypeError):  # not tensors: make() says what is wrong
        return make()
    if plan is None:
        plan = make()
        if all(n is None or type(n) in (int, float, str) for n in numbers):
            if len(_plans) >= 4096:
                _plans.clear()
            _plans[key] = plan
    return plan


def _dtype_code(t):
    return BF16 if t.dtype == _torch().bfloat16 else F32


def _last_axis(t, name):
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("the last axis of %s must be contiguous" % name)


def _scratch(nbytes, device, workspace):
    if nbytes == 0:
        return None, 0
    if workspace is not None:
        return _given_workspace(nbytes, device, workspace)
    torch = _torch()
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def _linattn_desc(q, k, v, log_decay, scale, cu_seqlens, initial_state, do=None):
    """Checks that the forward and the backward pass share; the descriptor and (N, state shape)."""
    torch = _torch()
    _seq(q, "q")
    packed = cu_seqlens is not None
    lead = 1 if packed else 2
    for t, name in ((k, "k"), (v, "v")):
        _seq(t, name, q.dtype, q.device)
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.dim() != lead + 2:
            raise ValueError("%s must be %s" % (name, "[T, heads, d] with cu_seqlens" if packed else "[N, T, heads, d]"))
        _last_axis(t, name)
        if t.shape[:lead] != q.shape[:lead]:
            raise ValueError("%s has %s tokens, q %s" % (name, tuple(t.shape[:lead]), tuple(q.shape[:lead])))
    H, dk = q.shape[-2:]
    Hk, dv = v.shape[-2:]
    if k.shape[-2] != Hk or k.shape[-1] != dk:
        raise ValueError("k has heads and size %s, expected %s" % (tuple(k.shape[-2:]), (Hk, dk)))
    _dense(log_decay, "log_decay", (H,), torch.float32, q.device)
    if packed:
        if not isinstance(cu_seqlens, torch.Tensor):
            raise ValueError("cu_seqlens must be a torch.Tensor")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be [sequences + 1]")
        _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, q.device)
    N = cu_seqlens.numel() - 1 if packed else q.shape[0]
    states = (N, H, dk, dv)
    if initial_state is not None:
        _dense(initial_state, "initial_state", states, torch.float32, q.device)

    def stride(t):
        return (0,) + t.stride()[:2] if packed else t.stride()[:3]

    i3 = ctypes.c_int64 * 3
    if scale is None:
        scale = dk ** -0.5
    d = gconv_linattn_desc(_dtype_code(q), int(packed), N, q.shape[lead - 1], H, Hk, dk, dv, i3(*stride(q)), i3(*stride(k)),
                           i3(*stride(v)), i3(), float(scale))
    if do is not None:
        _seq(do, "do", q.dtype, q.device)
        if do.shape != q.shape[:-1] + (dv,):
            raise ValueError("do has shape %s, expected %s" % (tuple(do.shape), tuple(q.shape[:-1]) + (dv,)))
        _last_axis(do, "do")
        d.do_stride = i3(*stride(do))
    return d, states


def gconv_linattn_workspace_size(desc: gconv_linattn_desc, op: int) -> int:
    n = ctypes.c_size_t()
    _check(load().gconv_linattn_workspace_size(ctypes.byref(desc), int(op), ctypes.byref(n)),
           "gconv_linattn_workspace_size")
    return n.value


def gconv_linattn_fwd(q, k, v, log_decay, *, scale=None, cu_seqlens=None, initial_state=None, workspace=None):
    """Linear attention with a decay for each head: S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,
    o_t = scale q_t S_t. q [N, T, H, dk], k [N, T, Hk, dk], v [N, T, Hk, dv] (H a multiple of Hk;
    float32 or bfloat16, any strides with a contiguous last axis), or [T, heads, d] with
    cu_seqlens (int32 [N + 1]) where sequences are packed (tokens in none of them give 0).
    log_decay [H] float32; scale defaults to dk^-0.5; initial_state [N, H, dk, dv] float32 or None.
    Returns o (q's type) and the final state [N, H, dk, dv] float32."""
    def make():
        d, states = _linattn_desc(q, k, v, log_decay, scale, cu_seqlens, initial_state)
        return ctypes.byref(d), states, q.shape[:-1] + (states[3],), gconv_linattn_workspace_size(d, LINATTN_FWD)

    d, states, shape, need = _plan("linattn_fwd", (q, k, v, log_decay, cu_seqlens, initial_state), (scale,), make)
    o = q.new_empty(shape)
    final = log_decay.new_empty(states)
    ws, nws = _scratch(need, q.device, workspace)
    _launch("gconv_linattn_fwd", q.device, d, _addr(q), _addr(k), _addr(v), _addr(log_decay), _addr(cu_seqlens),
            _addr(initial_state), _addr(o), _addr(final), _addr(ws), nws)
    return o, final


def gconv_linattn_bwd(do, q, k, v, log_decay, *, scale=None, cu_seqlens=None, initial_state=None,
                      d_final_state=None, workspace=None):
    """Gradients of gconv_linattn_fwd for the gradient `do` of o and `d_final_state` of the final
    state (None: 0). Returns dq, dk, dv (inputs' type and shape, dense) and the gradient of
    initial_state (None if that is None)."""
    def make():
        d, states = _linattn_desc(q, k, v, log_decay, scale, cu_seqlens, initial_state, do)
        if d_final_state is not None:
            _dense(d_final_state, "d_final_state", states, _torch().float32, q.device)
        return ctypes.byref(d), states, gconv_linattn_workspace_size(d, LINATTN_BWD)

    d, states, need = _plan("linattn_bwd", (do, q, k, v, log_decay, cu_seqlens, initial_state, d_final_state), (scale,), make)
    dq, dk, dv = (t.new_empty(t.shape) for t in (q, k, v))
    ds = log_decay.new_empty(states) if initial_state is not None else None
    ws, nws = _scratch(need, q.device, workspace)
    _launch("gconv_linattn_bwd", q.device, d, _addr(do), _addr(q), _addr(k), _addr(v), _addr(log_decay), _addr(cu_seqlens),
            _addr(initial_state), _addr(d_final_state), _addr(dq), _addr(dk), _addr(dv), _addr(ds), _addr(ws), nws)
    return dq, dk, dv, ds


def _linattn_step_plan(q, k, v, log_decay, state, scale, slots, out):
    torch = _torch()
    _seq(q, "q")
    for t, name in ((k, "k"), (v, "v")):
        _seq(t, name, q.dtype, q.device)
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t.dim() != 3 or t.shape[0] != q.shape[0]:
            raise ValueError("%s must be [B, heads, d]" % name)
        _last_axis(t, name)
    B, H, dk = q.shape
    Hk, dv = v.shape[1:]
    if k.shape[1] != Hk or k.shape[2] != dk:
        raise ValueError("k has heads and size %s, expected %s" % (tuple(k.shape[1:]), (Hk, dk)))
    _dense(log_decay, "log_decay", (H,), torch.float32, q.device)
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be [slots, H, dk, dv]")
    _dense(state, "state", (state.shape[0], H, dk, dv), torch.float32, q.device)
    if slots is not None:
        _dense(slots, "slots", (B,), torch.int32, q.device)
    if out is not None:
        _dense(out, "out", (B, H, dv), q.dtype, q.device)
    i3 = ctypes.c_int64 * 3
    sq, sk, sv = q.stride(), k.stride(), v.stride()
    d = gconv_linattn_desc(_dtype_code(q), 0, B, 0, H, Hk, dk, dv, i3(sq[0], 0, sq[1]), i3(sk[0], 0, sk[1]),
                           i3(sv[0], 0, sv[1]), i3(), float(dk ** -0.5 if scale is None else scale))
    return ctypes.byref(d), (B, H, dv), state.shape[0]


def gconv_linattn_step(q, k, v, log_decay, state, *, scale=None, slots=None, out=None):
    """One token of each of B sequences, in place on `state`: q [B, H, dk], k [B, Hk, dk],
    v [B, Hk, dv] (float32 or bfloat16, any strides with a contiguous last axis), state
    [slots, H, dk, dv] float32, slots int32 [B] (different ones; one out of range gives o = 0
    and touches no state) or None for slot b. Returns o [B, H, dv]."""
    d, shape, num = _plan("linattn_step", (q, k, v, log_decay, state, slots, out), (scale,),
                          lambda: _linattn_step_plan(q, k, v, log_decay, state, scale, slots, out))
    if out is None:
        out = q.new_empty(shape)
    _launch("gconv_linattn_step", q.device, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
            state.data_ptr(), _addr(slots), num, out.data_ptr())
    return out


def _normgate_desc(x, b, gate, act, w_post, scale, w_pre, eps, dy=None, dh=None):
    """Checks that the forward and the backward pass share; the descriptor."""
    _seq(b, "b")
    if b.dim() < 2:
        raise ValueError("b must be [N, T, D] or [T, D]")
    if b.dim() > 3:
        raise ValueError("b has %d axes, at most 3 are taken" % b.dim())
    dim = b.shape[-1]
    N, T = (b.shape[0], b.shape[1]) if b.dim() == 3 else (1, b.shape[0])
    if act not in ACTS:
        raise ValueError("act must be one of %s, got %r" % (", ".join(sorted(ACTS)), act))
    kind = GATE_NONE
    i2 = ctypes.c_int64 * 2

    def stride(t, name, shape):
        if t is None:
            return i2()
        _seq(t, name, b.dtype, b.device)
        if t.shape != shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
        _last_axis(t, name)
        return i2(*(t.stride()[:2] if t.dim() == 3 else (0, t.stride(0))))

    gshape = b.shape
    if gate is not None:
        kind = GATE_FULL
        if isinstance(gate, _torch().Tensor) and gate.shape != b.shape:
            kind, gshape = GATE_SEQUENCE, b.shape[:-2] + (1, dim)
    for w, name in ((w_post, "w_post"), (scale, "scale"), (w_pre, "w_pre")):
        if w is not None or name == "w_post":
            _dense(w, name, (dim,), b.dtype, b.device)
    return gconv_normgate_desc(_dtype_code(b), N, T, dim, kind, ACTS[act], stride(x, "x", b.shape), stride(b, "b", b.shape),
                               stride(gate, "gate", gshape), stride(dy, "dy", b.shape), stride(dh, "dh", b.shape), float(eps))


def gconv_normgate_fwd(x, b, *, w_post, gate=None, act="silu", scale=None, w_pre=None, eps=1e-6):
    """The norms around a block: y = x + scale * act(gate) * rmsnorm(b) * w_post and
    h = rmsnorm(y) * w_pre, over the last axis. b [N, T, D] or [T, D] (float32 or bfloat16, any
    strides with a contiguous last axis); x like b or None; gate like b, or [N, 1, D] ([1, D])
    for one row a sequence, or None; act "none", "sigmoid" or "silu"; w_post, scale, w_pre [D],
    the last two may be None. Returns y and h (None without w_pre)."""
    d = _plan("normgate_fwd", (x, b, gate, w_post, scale, w_pre), (act, eps),
              lambda: ctypes.byref(_normgate_desc(x, b, gate, act, w_post, scale, w_pre, eps)))
    y = b.new_empty(b.shape)
    h = b.new_empty(b.shape) if w_pre is not None else None
    _launch("gconv_normgate_fwd", b.device, d, _addr(x), b.data_ptr(), _addr(gate), w_post.data_ptr(), _addr(scale),
            _addr(w_pre), y.data_ptr(), _addr(h))
    return y, h


def gconv_normgate_bwd(dy, dh, x, b, *, w_post, gate=None, act="silu", scale=None, w_pre=None, eps=1e-6, workspace=None):
    """Gradients of gconv_normgate_fwd for dy of y and dh of h (None without w_pre). Returns
    dx, db, dgate, dw_post, dscale, dw_pre, of the inputs' shapes and type (None for those that
    are None)."""
    def make():
        d = _normgate_desc(x, b, gate, act, w_post, scale, w_pre, eps, _seq(dy, "dy"), dh)
        if (dh is None) != (w_pre is None):
            raise ValueError("dh must be given exactly when w_pre is")
        n = ctypes.c_size_t()
        _check(load().gconv_normgate_workspace_size(ctypes.byref(d), ctypes.byref(n)), "gconv_normgate_workspace_size")
        return ctypes.byref(d), n.value

    d, need = _plan("normgate_bwd", (dy, dh, x, b, gate, w_post, scale, w_pre), (act, eps), make)
    out = [t.new_empty(t.shape) if t is not None else None for t in (x, b, gate, w_post, scale, w_pre)]
    ws, nws = _scratch(need, b.device, workspace)
    _launch("gconv_normgate_bwd", b.device, d, _addr(dy), _addr(dh), _addr(x), _addr(b), _addr(gate), _addr(w_post),
            _addr(scale), _addr(w_pre), *(_addr(t) for t in out), _addr(ws), nws)
    return tuple(out)


def gconv_orthogonalize(u, *, groups=1, steps=5, eps=1e-7, out=None, workspace=None):
    """The orthogonalised update of a weight gradient u [K, C/groups, kh, kw] (or [K, D]; float32 or
    bfloat16, contiguous): each group's [K/groups, C/groups kh kw] matrix, scaled to norm 1, after
    `steps` rounds of the Newton-Schulz iteration. Returns a bfloat16 tensor of u's shape."""
    def make():
        torch = _torch()
        _seq(u, "u")
        if u.dim() < 2:
            raise ValueError("u must be [K, ...] with at least two axes")
        if not u.is_contiguous():
            raise ValueError("u must be contiguous")
        if out is not None:
            _dense(out, "out", u.shape, torch.bfloat16, u.device)
        K = u.shape[0]
        d = gconv_ortho_desc(_dtype_code(u), K, u.numel() // K if K else 0, int(groups), int(steps), float(eps))
        n = ctypes.c_size_t()
        _check(load().gconv_orthogonalize_workspace_size(ctypes.byref(d), ctypes.byref(n)), "gconv_orthogonalize_workspace_size")
        return ctypes.byref(d), n.value

    d, need = _plan("orthogonalize", (u, out), (groups, steps, eps), make)
    if out is None:
        out = u.new_empty(u.shape, dtype=_torch().bfloat16)
    ws, nws = _scratch(need, u.device, workspace)
    _launch("gconv_orthogonalize", u.device, d, u.data_ptr(), out.data_ptr(), _addr(ws), nws)
    return out


def _token_shape(x, cu_seqlens, name):
    """(packed, sequences, tokens) of x: [N, T, ...], or [T, ...] with cu_seqlens (checked here)."""
    torch = _torch()
    if cu_seqlens is None:
        return 0, x.shape[0], x.shape[1]
    if not isinstance(cu_seqlens, torch.Tensor):
        raise ValueError("cu_seqlens must be a torch.Tensor")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [sequences + 1]")
    _dense(cu_seqlens, "cu_seqlens", cu_seqlens.shape, torch.int32, x.device)
    return 1, cu_seqlens.numel() - 1, x.shape[0]


def _strides(t, packed, count):
    """The first `count` strides of t as (between sequences, between tokens, ...)."""
    if t is None:
        return (ctypes.c_int64 * count)()
    s = ((0,) + t.stride() if packed else t.stride())[:count]
    return (ctypes.c_int64 * count)(*s)


def _like(t, name, ref, shape):
    """A tensor of ref's type and device, of one shape, with a contiguous last axis."""
    _seq(t, name, ref.dtype, ref.device)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    _last_axis(t, name)
    return t


def _shortconv_desc(x, w, bias, act, cu_seqlens, initial_state, dy=None, d_final_state=None):
    """Checks that the forward and the backward pass share; the descriptor and the states' shape."""
    _seq(x, "x")
    if x.dim() != (2 if cu_seqlens is not None else 3):
        raise ValueError("x must be %s" % ("[T, D] with cu_seqlens" if cu_seqlens is not None else "[N, T, D]"))
    _last_axis(x, "x")
    if act not in ACTS:
        raise ValueError("act must be one of %s, got %r" % (", ".join(sorted(ACTS)), act))
    dim = x.shape[-1]
    _seq(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be [D, taps]")
    _dense(w, "w", (dim, w.shape[1]), x.dtype, x.device)
    taps = w.shape[1]
    if taps < 1:
        raise ValueError("w must have at least one tap")
    if bias is not None:
        _dense(bias, "bias", (dim,), x.dtype, x.device)
    packed, N, T = _token_shape(x, cu_seqlens, "x")
    states = (N, taps - 1, dim)
    for t, name in ((initial_state, "initial_state"), (d_final_state, "d_final_state")):
        if t is not None:
            _dense(t, name, states, x.dtype, x.device)
    if dy is not None:
        _like(dy, "dy", x, x.shape)
    d = gconv_shortconv_desc(_dtype_code(x), packed, N, T, dim, taps, ACTS[act], _strides(x, packed, 2), _strides(dy, packed, 2))
    return d, states


def gconv_shortconv_fwd(x, w, bias=None, *, act="silu", cu_seqlens=None, initial_state=None):
    """The short causal convolution of each channel: y_t = act(bias + sum_j w[:, j] x_{t-taps+1+j}).
    x [N, T, D] (or [T, D] with cu_seqlens, int32 [N + 1], where sequences are packed; tokens in none
    of them give 0), float32 or bfloat16, any strides with a contiguous last axis; w [D, taps] (up to
    8), bias [D] or None; act "none", "sigmoid" or "silu"; initial_state [N, taps - 1, D], the inputs
    before the first, or None for 0. Returns y and the final state [N, taps - 1, D], of x's type."""
    def make():
        d, states = _shortconv_desc(x, w, bias, act, cu_seqlens, initial_state)
        return ctypes.byref(d), states

    d, states = _plan("shortconv_fwd", (x, w, bias, cu_seqlens, initial_state), (act,), make)
    y, final = x.new_empty(x.shape), x.new_empty(states)
    _launch("gconv_shortconv_fwd", x.device, d, _addr(x), _addr(w), _addr(bias), _addr(cu_seqlens), _addr(initial_state), _addr(y),
            _addr(final))
    return y, final


def gconv_shortconv_bwd(dy, x, w, bias=None, *, act="silu", cu_seqlens=None, initial_state=None, d_final_state=None, workspace=None):
    """Gradients of gconv_shortconv_fwd for dy of y and d_final_state of the final state (None: 0).
    Returns dx, dw, dbias (None without bias) and the gradient of initial_state (None without it)."""
    def make():
        d, states = _shortconv_desc(x, w, bias, act, cu_seqlens, initial_state, _seq(dy, "dy"), d_final_state)
        n = ctypes.c_size_t()
        _check(load().gconv_shortconv_workspace_size(ctypes.byref(d), ctypes.byref(n)), "gconv_shortconv_workspace_size")
        return ctypes.byref(d), n.value

    d, need = _plan("shortconv_bwd", (dy, x, w, bias, cu_seqlens, initial_state, d_final_state), (act,), make)
    dx, dw, dbias, ds = (t.new_empty(t.shape) if t is not None else None for t in (x, w, bias, initial_state))
    ws, nws = _scratch(need, x.device, workspace)
    _launch("gconv_shortconv_bwd", x.device, d, _addr(dy), _addr(x), _addr(w), _addr(bias), _addr(cu_seqlens), _addr(initial_state),
            _addr(d_final_state), _addr(dx), _addr(dw), _addr(dbias), _addr(ds), _addr(ws), nws)
    return dx, dw, dbias, ds


def _shortconv_step_plan(x, w, state, bias, act, slots, out):
    torch = _torch()
    _seq(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [B, D]")
    d, _ = _shortconv_desc(x[:, None], w, bias, act, None, None)
    B, dim = x.shape
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be [slots, taps - 1, D]")
    _dense(state, "state", (state.shape[0], w.shape[1] - 1, dim), x.dtype, x.device)
    if slots is not None:
        _dense(slots, "slots", (B,), torch.int32, x.device)
    if out is not None:
        _dense(out, "out", (B, dim), x.dtype, x.device)
    d.tokens = 0
    return ctypes.byref(d), state.shape[0]


def gconv_shortconv_step(x, w, state, bias=None, *, act="silu", slots=None, out=None):
    """One token x [B, D] of each of B sequences, in place on `state` [slots, taps - 1, D] (x's type);
    slots int32 [B] (different ones; one out of range gives y = 0 and touches no state) or None for
    slot b. Returns y [B, D]."""
    d, num = _plan("shortconv_step", (x, w, state, bias, slots, out), (act,),
                   lambda: _shortconv_step_plan(x, w, state, bias, act, slots, out))
    if out is None:
        out = x.new_empty(x.shape)
    _launch("gconv_shortconv_step", x.device, d, x.data_ptr(), w.data_ptr(), _addr(bias), state.data_ptr(), _addr(slots), num,
            out.data_ptr())
    return out


def _scan_desc(u, dt, a, b, c, skip, gate, dt_bias, softplus, cu_seqlens, initial_state, dy=None, d_final_state=None):
    """Checks that the forward and the backward pass share; the descriptor and the states' shape."""
    torch = _torch()
    _seq(u, "u")
    lead = 1 if cu_seqlens is not None else 2
    if u.dim() != lead + 1:
        raise ValueError("u must be %s" % ("[T, D] with cu_seqlens" if lead == 1 else "[N, T, D]"))
    _last_axis(u, "u")
    dim = u.shape[-1]
    _like(dt, "dt", u, u.shape)
    _seq(b, "b", u.dtype, u.device)
    if b.dim() != lead + 2 or b.shape[:lead] != u.shape[:lead]:
        raise ValueError("b must be %s" % ("[T, groups, states]" if lead == 1 else "[N, T, groups, states]"))
    _last_axis(b, "b")
    _like(c, "c", u, b.shape)
    groups, n = b.shape[-2:]
    _dense(a, "a", (dim, n), torch.float32, u.device)
    for t, name in ((skip, "skip"), (dt_bias, "dt_bias")):
        if t is not None:
            _dense(t, name, (dim,), torch.float32, u.device)
    for t, name in ((gate, "gate"), (dy, "dy")):
        if t is not None:
            _like(t, name, u, u.shape)
    packed, N, T = _token_shape(u, cu_seqlens, "u")
    states = (N, dim, n)
    for t, name in ((initial_state, "initial_state"), (d_final_state, "d_final_state")):
        if t is not None:
            _dense(t, name, states, torch.float32, u.device)
    d = gconv_scan_desc(_dtype_code(u), packed, N, T, dim, n, groups, int(bool(softplus)), _strides(u, packed, 2),
                        _strides(dt, packed, 2), _strides(gate, packed, 2), _strides(b, packed, 3), _strides(c, packed, 3),
                        _strides(dy, packed, 2))
    return d, states


def gconv_scan_workspace_size(desc: gconv_scan_desc, op: int) -> int:
    n = ctypes.c_size_t()
    _check(load().gconv_scan_workspace_size(ctypes.byref(desc), int(op), ctypes.byref(n)), "gconv_scan_workspace_size")
    return n.value


def gconv_scan_fwd(u, dt, a, b, c, *, skip=None, gate=None, dt_bias=None, softplus=True, cu_seqlens=None, initial_state=None,
                   workspace=None):
    """The selective state space scan: with s_t = softplus(dt_t + dt_bias) (or without the softplus),
    h_t = exp(s_t a) h_{t-1} + s_t u_t b_t and y_t = (c_t . h_t + skip u_t) silu(gate_t), for each channel.
    u, dt, gate (None: no gate) [N, T, D], b, c [N, T, G, S] (D a multiple of G, S up to 64), or [T, D] and
    [T, G, S] with cu_seqlens (int32 [N + 1]) where sequences are packed (tokens in none of them give 0);
    float32 or bfloat16, any strides with a contiguous last axis. a [D, S], skip and dt_bias [D] (or None)
    float32; initial_state [N, D, S] float32 or None. Returns y and the final state [N, D, S] float32."""
    def make():
        d, states = _scan_desc(u, dt, a, b, c, skip, gate, dt_bias, softplus, cu_seqlens, initial_state)
        return ctypes.byref(d), states, gconv_scan_workspace_size(d, SCAN_FWD)

    d, states, need = _plan("scan_fwd", (u, dt, a, b, c, skip, gate, dt_bias, cu_seqlens, initial_state), (int(bool(softplus)),), make)
    y, final = u.new_empty(u.shape), a.new_empty(states)
    ws, nws = _scratch(need, u.device, workspace)
    _launch("gconv_scan_fwd", u.device, d, _addr(u), _addr(dt), _addr(a), _addr(b), _addr(c), _addr(skip), _addr(gate), _addr(dt_bias),
            _addr(cu_seqlens), _addr(initial_state), _addr(y), _addr(final), _addr(ws), nws)
    return y, final


def gconv_scan_bwd(dy, u, dt, a, b, c, *, skip=None, gate=None, dt_bias=None, softplus=True, cu_seqlens=None, initial_state=None,
                   d_final_state=None, workspace=None):
    """Gradients of gconv_scan_fwd for dy of y and d_final_state of the final state (None: 0). Returns du,
    ddt, da, db, dc, dskip, dgate, ddt_bias and the gradient of initial_state, of the inputs' shapes and
    types (None for those that are None). The workspace takes about 0.76 bytes for each token, channel and
    state."""
    def make():
        d, _ = _scan_desc(u, dt, a, b, c, skip, gate, dt_bias, softplus, cu_seqlens, initial_state, _seq(dy, "dy"), d_final_state)
        return ctypes.byref(d), gconv_scan_workspace_size(d, SCAN_BWD)

    d, need = _plan("scan_bwd", (dy, u, dt, a, b, c, skip, gate, dt_bias, cu_seqlens, initial_state, d_final_state),
                    (int(bool(softplus)),), make)
    out = [t.new_empty(t.shape) if t is not None else None for t in (u, dt, a, b, c, skip, gate, dt_bias, initial_state)]
    ws, nws = _scratch(need, u.device, workspace)
    _launch("gconv_scan_bwd", u.device, d, _addr(dy), _addr(u), _addr(dt), _addr(a), _addr(b), _addr(c), _addr(skip), _addr(gate),
            _addr(dt_bias), _addr(cu_seqlens), _addr(initial_state), _addr(d_final_state), *(_addr(t) for t in out), _addr(ws), nws)
    return tuple(out)


def _scan_step_plan(u, dt, a, b, c, state, skip, gate, dt_bias, softplus, slots, out):
    torch = _torch()
    for t, name in ((u, "u"), (dt, "dt"), (gate, "gate")):
        if t is not None and _seq(t, name).dim() != 2:
            raise ValueError("%s must be [B, D]" % name)
    for t, name in ((b, "b"), (c, "c")):
        if _seq(t, name).dim() != 3:
            raise ValueError("%s must be [B, groups, states]" % name)
    one = [t[:, None] if t is not None else None for t in (u, dt, b, c, gate)]
    d, _ = _scan_desc(one[0], one[1], a, one[2], one[3], skip, one[4], dt_bias, softplus, None, None)
    B, dim = u.shape
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be [slots, D, states]")
    _dense(state, "state", (state.shape[0],) + tuple(a.shape), torch.float32, u.device)
    if slots is not None:
        _dense(slots, "slots", (B,), torch.int32, u.device)
    if out is not None:
        _dense(out, "out", (B, dim), u.dtype, u.device)
    d.tokens = 0
    return ctypes.byref(d), state.shape[0]


def gconv_scan_step(u, dt, a, b, c, state, *, skip=None, gate=None, dt_bias=None, softplus=True, slots=None, out=None):
    """One token of each of B sequences, in place on `state` [slots, D, S] float32: u, dt, gate [B, D],
    b, c [B, G, S]; slots int32 [B] (different ones; one out of range gives y = 0 and touches no state)
    or None for slot b. Returns y [B, D]."""
    d, num = _plan("scan_step", (u, dt, a, b, c, state, skip, gate, dt_bias, slots, out), (int(bool(softplus)),),
                   lambda: _scan_step_plan(u, dt, a, b, c, state, skip, gate, dt_bias, softplus, slots, out))
    if out is None:
        out = u.new_empty(u.shape)
    _launch("gconv_scan_step", u.device, d, u.data_ptr(), dt.data_ptr(), a.data_ptr(), b.data_ptr(), c.data_ptr(), _addr(skip),
            _addr(gate), _addr(dt_bias), state.data_ptr(), _addr(slots), num, out.data_ptr())
    return out


def _names(t, name, device):
    """A contiguous GPU tensor of whole numbers that name tokens; its gconv_index."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError("%s must be a torch.Tensor" % name)
    if t.dtype not in (torch.int32, torch.int64):
        raise ValueError("%s must be int32 or int64, got %s" % (name, t.dtype))
    if t.dim() not in (1, 2):
        raise ValueError("%s must be [T] or [N, T]" % name)
    if t.device != device or not t.is_cuda:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return I64 if t.dtype == torch.int64 else I32


def _rows_of(t, name, lead):
    """(sequences, tokens) of tokens [T] or [N, T], and the strides of t [T, D] or [N, T, D] between them."""
    if tuple(t.shape[:-1]) != tuple(lead):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(lead) + ("D",)))
    _last_axis(t, name)
    N, T = lead if len(lead) == 2 else (1, lead[0])
    return N, T, (ctypes.c_int64 * 2)(*((0,) + t.stride()[:1] if len(lead) == 1 else t.stride()[:2]))


def gconv_embed_fwd(table, ids, *, scale=1.0):
    """The embedding of tokens: scale * table[ids], 0 for an id outside the table. table [rows, D]
    (float32 or bfloat16, contiguous), ids int32 or int64 [T] or [N, T]. Returns ids' shape + [D]."""
    def make():
        _seq(table, "table")
        if table.dim() != 2:
            raise ValueError("table must be [rows, D]")
        _dense(table, "table", table.shape, table.dtype, table.device)
        index = _names(ids, "ids", table.device)
        N, T = ids.shape if ids.dim() == 2 else (1, ids.shape[0])
        return (ctypes.byref(gconv_embed_desc(_dtype_code(table), index, N, T, table.shape[0], table.shape[1], (ctypes.c_int64 * 2)(),
                                              float(scale))),)

    d, = _plan("embed_fwd", (table, ids), (scale,), make)
    y = table.new_empty(ids.shape + table.shape[1:])
    _launch("gconv_embed_fwd", table.device, d, _addr(table), _addr(ids), _addr(y))
    return y


def gconv_embed_bwd(dy, ids, rows, *, scale=1.0, workspace=None):
    """The gradient [rows, D] of gconv_embed_fwd's table for dy of its result (any strides with a
    contiguous last axis): each row the sum over its tokens, in a fixed order; rows without tokens are 0."""
    def make():
        _seq(dy, "dy")
        index = _names(ids, "ids", dy.device)
        N, T, stride = _rows_of(dy, "dy", ids.shape)
        d = gconv_embed_desc(_dtype_code(dy), index, N, T, int(rows), dy.shape[-1], stride, float(scale))
        n = ctypes.c_size_t()
        _check(load().gconv_embed_workspace_size(ctypes.byref(d), ctypes.byref(n)), "gconv_embed_workspace_size")
        return ctypes.byref(d), n.value

    d, need = _plan("embed_bwd", (dy, ids), (rows, scale), make)
    dtable = dy.new_empty((int(rows), dy.shape[-1]))
    ws, nws = _scratch(need, dy.device, workspace)
    _launch("gconv_embed_bwd", dy.device, d, _addr(dy), _addr(ids), _addr(dtable), _addr(ws), nws)
    return dtable


def _xent_desc(h, w, targets, scale):
    _seq(h, "h")
    _seq(w, "w")
    if w.dim() != 2:
        raise ValueError("w must be [vocab, D]")
    _dense(w, "w", (w.shape[0], h.shape[-1] if h.dim() else 0), h.dtype, h.device)
    index = _names(targets, "targets", h.device)
    N, T, stride = _rows_of(h, "h", targets.shape)
    return gconv_xent_desc(_dtype_code(h), index, N, T, w.shape[0], w.shape[1], stride, float(scale))


def gconv_xent_workspace_size(desc: gconv_xent_desc, op: int) -> int:
    n = ctypes.c_size_t()
    _check(load().gconv_xent_workspace_size(ctypes.byref(desc), int(op), ctypes.byref(n)), "gconv_xent_workspace_size")
    return n.value


def gconv_xent_fwd(h, w, targets, *, scale=1.0, workspace=None):
    """Softmax cross entropy of tokens against a vocabulary, whose logits scale * h w^T are not kept.
    h [T, D] or [N, T, D] (float32 or bfloat16, any strides with a contiguous last axis), w [vocab, D]
    of the same type (at a 16-byte boundary where it is bfloat16 and D a multiple of 64), targets int32 or int64 [T] or [N, T]; a target outside the vocabulary does not
    count. Returns loss (0 where it does not count) and lse, the logarithm of the sum of the logits'
    exponentials, of targets' shape in float32."""
    def make():
        d = _xent_desc(h, w, targets, scale)
        return ctypes.byref(d), gconv_xent_workspace_size(d, XENT_FWD)

    d, need = _plan("xent_fwd", (h, w, targets), (scale,), make)
    torch = _torch()
    loss, lse = (h.new_empty(targets.shape, dtype=torch.float32) for _ in range(2))
    ws, nws = _scratch(need, h.device, workspace)
    _launch("gconv_xent_fwd", h.device, d, _addr(h), _addr(w), _addr(targets), _addr(loss), _addr(lse), _addr(ws), nws)
    return loss, lse


def gconv_xent_bwd(dloss, h, w, targets, lse, *, dlse=None, scale=1.0, workspace=None):
    """Gradients of gconv_xent_fwd for dloss of loss and dlse of lse (None: 0), both of targets' shape in
    float32; lse as the forward pass gave it. Returns dh and dw, of h's and w's shapes and type."""
    def make():
        d = _xent_desc(h, w, targets, scale)
        for t, name in ((dloss, "dloss"), (lse, "lse"), (dlse, "dlse")):
            if t is not None or name != "dlse":
                _dense(t, name, targets.shape, _torch().float32, h.device)
        return ctypes.byref(d), gconv_xent_workspace_size(d, XENT_BWD)

    d, need = _plan("xent_bwd", (dloss, h, w, targets, lse, dlse), (scale,), make)
    dh, dw = h.new_empty(h.shape), w.new_empty(w.shape)
    ws, nws = _scratch(need, h.device, workspace)
    _launch("gconv_xent_bwd", h.device, d, _addr(dloss), _addr(dlse), _addr(h), _addr(w), _addr(targets), _addr(lse), _addr(dh), _addr(dw),
            _addr(ws), nws)
    return dh, dw
