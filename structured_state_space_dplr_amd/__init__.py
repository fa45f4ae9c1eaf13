"""Python binding of libs4dplr (S4 DPLR convolution-mode forward on MI355X).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libs4dplr.so``.  The functions carry the names of the C entry
points in ``include/s4dplr.h`` (without the ``s4dplr_`` prefix).  Tensors are
float32, contiguous, on the GPU and 8-byte aligned (a view that starts at an
odd element is refused with status 8); complex parameters are [H, N, 2]
(interleaved re, im).  PyTorch supplies device memory and the current stream.

There is no fallback: if the library is missing or fails to load, importing
this package raises.

Preconditions that the kernels do not test on the device -- Re(Lambda) < 0
(stable poles), dt > 0 and every value finite -- are checked on the host
before the call when the environment variable ``S4DPLR_VALIDATE`` is ``1``;
a violation raises ``S4DPLRPreconditionError``.  The check copies the
inputs to host memory and synchronizes, so it is for debugging, not for the
timed path.

The token-major operators (``layer_norm_fwd`` / ``layer_norm_bwd`` and, on a
``DeltaPlan``, ``delta_fwd`` / ``delta_bwd``) take float32, bfloat16 or float16
tensors of any size and alignment, launch on the device of their tensors, and
``stream=None`` is that device's current stream.  With ``S4DPLR_VALIDATE=1``
their inputs are checked to be finite, the log decays g to be <= 0 and offsets
to rise within the rows; rows outside every sequence may hold anything.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch  # loads the HIP runtime that libs4dplr then shares

__all__ = [
    "S4DPLRError", "S4DPLRPreconditionError", "check_preconditions", "validation_enabled",
    "DIAGONAL", "ZOH", "BLOCK", "abi_version", "status_string", "plan_create",
    "plan_workspace_bytes", "plan_init", "kernel_gen", "generating_function", "conv_fwd",
    "forward", "forward_noalloc",
    "conv_apply", "recurrent_prepare", "recurrent_scan", "conv_bwd", "kernel_gen_bwd",
    "block_forward", "layer_norm_fwd", "layer_norm_bwd", "layer_norm_workspace_bytes",
    "DeltaPlan", "delta_fwd", "delta_bwd",
    "plan_destroy", "Plan", "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libs4dplr.so")
DIAGONAL = 1
ZOH = 2
BLOCK = 4
RANK_SHIFT = 8

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python structured_state_space_dplr_amd/build.py` "
        "(or __graft_entry__.build()) first")

_lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_lib.s4dplr_abi_version.restype = ctypes.c_int
_lib.s4dplr_abi_version.argtypes = []
_lib.s4dplr_status_string.restype = ctypes.c_char_p
_lib.s4dplr_status_string.argtypes = [ctypes.c_int]
_lib.s4dplr_last_hip_error.restype = ctypes.c_int
_lib.s4dplr_last_hip_error.argtypes = []
_lib.s4dplr_plan_create.restype = ctypes.c_int
_lib.s4dplr_plan_create.argtypes = [ctypes.POINTER(_p), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                    ctypes.c_int, ctypes.c_uint]
_lib.s4dplr_plan_workspace_bytes.restype = ctypes.c_int
_lib.s4dplr_plan_workspace_bytes.argtypes = [_p, ctypes.POINTER(ctypes.c_size_t)]
_lib.s4dplr_plan_init.restype = ctypes.c_int
_lib.s4dplr_plan_init.argtypes = [_p, _p, _p]
_lib.s4dplr_kernel_gen.restype = ctypes.c_int
_lib.s4dplr_kernel_gen.argtypes = [_p] * 10
_lib.s4dplr_generating_function.restype = ctypes.c_int
_lib.s4dplr_generating_function.argtypes = [_p] * 10
_lib.s4dplr_conv_fwd.restype = ctypes.c_int
_lib.s4dplr_conv_fwd.argtypes = [_p] * 7
_lib.s4dplr_forward.restype = ctypes.c_int
_lib.s4dplr_forward.argtypes = [_p] * 13
_lib.s4dplr_forward_noalloc.restype = ctypes.c_int
_lib.s4dplr_forward_noalloc.argtypes = [_p] * 12
_lib.s4dplr_conv_apply.restype = ctypes.c_int
_lib.s4dplr_conv_apply.argtypes = [_p] * 5
_lib.s4dplr_recurrent_prepare.restype = ctypes.c_int
_lib.s4dplr_recurrent_prepare.argtypes = [_p] * 9
_lib.s4dplr_recurrent_scan.restype = ctypes.c_int
_lib.s4dplr_recurrent_scan.argtypes = [_p, _p, _p, ctypes.c_int, _p, _p, _p, _p]
_lib.s4dplr_conv_bwd.restype = ctypes.c_int
_lib.s4dplr_conv_bwd.argtypes = [_p] * 10
_lib.s4dplr_kernel_gen_bwd.restype = ctypes.c_int
_lib.s4dplr_kernel_gen_bwd.argtypes = [_p] * 16
_lib.s4dplr_block_forward.restype = ctypes.c_int
_lib.s4dplr_block_forward.argtypes = [_p] * 16
_l, _i = ctypes.c_long, ctypes.c_int
_lib.s4dplr_layer_norm_fwd.restype = _i
_lib.s4dplr_layer_norm_fwd.argtypes = [_p] * 6 + [_l] * 3 + [ctypes.c_float, _i, _p]
_lib.s4dplr_layer_norm_workspace_bytes.restype = _i
_lib.s4dplr_layer_norm_workspace_bytes.argtypes = [_l] * 3 + [ctypes.POINTER(ctypes.c_size_t)]
_lib.s4dplr_layer_norm_bwd.restype = _i
_lib.s4dplr_layer_norm_bwd.argtypes = [_p] * 8 + [_l] * 3 + [_i, _p, _p]
_lib.s4dplr_delta_plan_create.restype = _i
_lib.s4dplr_delta_plan_create.argtypes = [ctypes.POINTER(_p), _i, _l, _i, _i, _i, _i, _i,
                                          ctypes.c_uint]
_lib.s4dplr_delta_plan_bytes.restype = _i
_lib.s4dplr_delta_plan_bytes.argtypes = [_p] + [ctypes.POINTER(ctypes.c_size_t)] * 2
_lib.s4dplr_delta_fwd.restype = _i
_lib.s4dplr_delta_fwd.argtypes = ([_p, _p, _l, _p, _l, _p, _l] + [_p] * 3 + [ctypes.c_float]
                                  + [_p] * 6)
_lib.s4dplr_delta_bwd.restype = _i
_lib.s4dplr_delta_bwd.argtypes = ([_p, _p, _l, _p, _l, _p, _l] + [_p] * 3 + [ctypes.c_float]
                                  + [_p] * 11)
_lib.s4dplr_delta_plan_destroy.restype = None
_lib.s4dplr_delta_plan_destroy.argtypes = [_p]
_lib.s4dplr_plan_destroy.restype = None
_lib.s4dplr_plan_destroy.argtypes = [_p]


class S4DPLRError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = status_string(status)
        if status == 5:
            msg += f" (hipError_t {_lib.s4dplr_last_hip_error()})"
        super().__init__(f"{where}: status {status}: {msg}")
        self.status = status


def _check(status: int, where: str) -> None:
    if status != 0:
        raise S4DPLRError(status, where)


VALIDATE_ENV = "S4DPLR_VALIDATE"


class S4DPLRPreconditionError(ValueError):
    """An input violates a precondition the kernels do not check: Re(Lambda)
    < 0 ("The S4 kernel, from scratch", section 6 keeps the real parts of the
    poles negative; "ML//SSM//S4": a stable discrete system needs its
    eigenvalues inside the unit circle, which the bilinear map gives exactly
    for Re(Lambda) < 0), dt > 0, or finite values.  Raised only with
    S4DPLR_VALIDATE=1."""

    def __init__(self, where: str, what: str):
        super().__init__(f"{where}: {what}")
        self.where, self.what = where, what


def validation_enabled() -> bool:
    return os.environ.get(VALIDATE_ENV, "") == "1"


def _host(t):
    return torch.as_tensor(t).detach().to(device="cpu", dtype=torch.float64)


def check_preconditions(where: str = "check_preconditions", lam=None, dt=None, **tensors) -> None:
    """Raise S4DPLRPreconditionError for the first violated precondition:
    every given tensor finite, Re(lam[..., 0]) < 0 strictly, dt > 0 strictly.
    Tensors may live on any device (they are copied to host memory); None is
    skipped."""
    named = dict(tensors)
    named["lam"], named["dt"] = lam, dt
    for name, t in named.items():
        if t is None:
            continue
        h = _host(t)
        bad = ~torch.isfinite(h)
        if bool(bad.any()):
            idx = tuple(int(i) for i in bad.nonzero()[0])
            raise S4DPLRPreconditionError(where, f"{name} is not finite at index {idx}")
    if lam is not None:
        re = _host(lam)[..., 0]
        bad = re >= 0
        if bool(bad.any()):
            idx = tuple(int(i) for i in bad.nonzero()[0])
            raise S4DPLRPreconditionError(
                where, f"Re(lam) must be < 0 (stable pole); lam{list(idx)} has Re = "
                       f"{float(re[idx]):g}")
    if dt is not None:
        d = _host(dt)
        bad = d <= 0
        if bool(bad.any()):
            idx = int(bad.nonzero()[0][0])
            raise S4DPLRPreconditionError(where, f"dt must be > 0; dt[{idx}] = {float(d[idx]):g}")


def _validate(where: str, **kw) -> None:
    if validation_enabled():
        check_preconditions(where, **kw)


def abi_version() -> int:
    return _lib.s4dplr_abi_version()


def status_string(status: int) -> str:
    return _lib.s4dplr_status_string(status).decode()


def plan_create(H: int, N: int, L: int, batch: int, flags: int = 0) -> int:
    h = _p()
    _check(_lib.s4dplr_plan_create(ctypes.byref(h), H, N, L, batch, flags), "plan_create")
    return h.value


def plan_workspace_bytes(plan: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.s4dplr_plan_workspace_bytes(plan, ctypes.byref(n)), "plan_workspace_bytes")
    return n.value


def plan_destroy(plan: int) -> None:
    _lib.s4dplr_plan_destroy(plan)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t, name, shape=None):
    """Device pointer of a float32 contiguous GPU tensor (None -> NULL)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")
    if t.dtype != torch.float32:
        raise TypeError(f"{name}: must be float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _ws_ptr(ws) -> int:
    if isinstance(ws, torch.Tensor):
        return ws.data_ptr()
    return int(ws)


def plan_init(plan: int, ws, stream=None) -> None:
    _check(_lib.s4dplr_plan_init(plan, _ws_ptr(ws), _stream(stream)), "plan_init")


def kernel_gen(plan: "Plan | int", lam, P, Q, B, C, dt, K, ws, stream=None) -> None:
    _validate("kernel_gen", lam=lam, dt=dt, P=P, Q=Q, B=B, C=C)
    p, (H, N, L, _) = _dims(plan)
    cplx = (H, N, 2)
    lr = _lowrank_shape(plan)
    _check(_lib.s4dplr_kernel_gen(
        p, _ptr(lam, "lam", cplx), _ptr(P, "P", lr), _ptr(Q, "Q", lr), _ptr(B, "B", cplx),
        _ptr(C, "C", cplx), _ptr(dt, "dt", (H,)), _ptr(K, "K", (H, L)), _ws_ptr(ws),
        _stream(stream)), "kernel_gen")


def generating_function(plan: "Plan | int", lam, P, Q, B, C, dt, khat, ws, stream=None) -> None:
    """K-hat at the L roots of unity into ``khat`` ([H, L, 2] float32)."""
    _validate("generating_function", lam=lam, dt=dt, P=P, Q=Q, B=B, C=C)
    p, (H, N, L, _) = _dims(plan)
    cplx = (H, N, 2)
    lr = _lowrank_shape(plan)
    _check(_lib.s4dplr_generating_function(
        p, _ptr(lam, "lam", cplx), _ptr(P, "P", lr), _ptr(Q, "Q", lr), _ptr(B, "B", cplx),
        _ptr(C, "C", cplx), _ptr(dt, "dt", (H,)), _ptr(khat, "khat", (H, L, 2)), _ws_ptr(ws),
        _stream(stream)), "generating_function")


def conv_fwd(plan: "Plan | int", u, K, D, y, ws, stream=None) -> None:
    _validate("conv_fwd", u=u, K=K, D=D)
    p, (H, N, L, batch) = _dims(plan)
    _check(_lib.s4dplr_conv_fwd(
        p, _ptr(u, "u", (batch, H, L)), _ptr(K, "K", (H, L)), _ptr(D, "D", (H,)),
        _ptr(y, "y", (batch, H, L)), _ws_ptr(ws), _stream(stream)), "conv_fwd")


def forward(plan: "Plan | int", lam, P, Q, B, C, dt, D, u, K, y, ws, stream=None) -> None:
    _validate("forward", lam=lam, dt=dt, P=P, Q=Q, B=B, C=C, D=D, u=u)
    p, (H, N, L, batch) = _dims(plan)
    cplx = (H, N, 2)
    lr = _lowrank_shape(plan)
    _check(_lib.s4dplr_forward(
        p, _ptr(lam, "lam", cplx), _ptr(P, "P", lr), _ptr(Q, "Q", lr), _ptr(B, "B", cplx),
        _ptr(C, "C", cplx), _ptr(dt, "dt", (H,)), _ptr(D, "D", (H,)),
        _ptr(u, "u", (batch, H, L)), _ptr(K, "K", (H, L)), _ptr(y, "y", (batch, H, L)),
        _ws_ptr(ws), _stream(stream)), "forward")


def forward_noalloc(plan: "Plan | int", lam, P, Q, B, C, dt, D, u, K, y, stream=None) -> None:
    """``forward`` on the library's static device scratch (no workspace)."""
    _validate("forward_noalloc", lam=lam, dt=dt, P=P, Q=Q, B=B, C=C, D=D, u=u)
    p, (H, N, L, batch) = _dims(plan)
    cplx = (H, N, 2)
    lr = _lowrank_shape(plan)
    _check(_lib.s4dplr_forward_noalloc(
        p, _ptr(lam, "lam", cplx), _ptr(P, "P", lr), _ptr(Q, "Q", lr), _ptr(B, "B", cplx),
        _ptr(C, "C", cplx), _ptr(dt, "dt", (H,)), _ptr(D, "D", (H,)),
        _ptr(u, "u", (batch, H, L)), _ptr(K, "K", (H, L)), _ptr(y, "y", (batch, H, L)),
        _stream(stream)), "forward_noalloc")


def conv_apply(plan: "Plan | int", u, y, ws, stream=None) -> None:
    _validate("conv_apply", u=u)
    p, (H, N, L, batch) = _dims(plan)
    _check(_lib.s4dplr_conv_apply(
        p, _ptr(u, "u", (batch, H, L)), _ptr(y, "y", (batch, H, L)), _ws_ptr(ws),
        _stream(stream)), "conv_apply")


def recurrent_prepare(plan: "Plan | int", lam, P, Q, B, C, dt, ws, stream=None) -> None:
    _validate("recurrent_prepare", lam=lam, dt=dt, P=P, Q=Q, B=B, C=C)
    p, (H, N, L, _) = _dims(plan)
    cplx = (H, N, 2)
    lr = _lowrank_shape(plan)
    _check(_lib.s4dplr_recurrent_prepare(
        p, _ptr(lam, "lam", cplx), _ptr(P, "P", lr), _ptr(Q, "Q", lr), _ptr(B, "B", cplx),
        _ptr(C, "C", cplx), _ptr(dt, "dt", (H,)), _ws_ptr(ws), _stream(stream)),
        "recurrent_prepare")


def recurrent_scan(plan: "Plan | int", D, u, state, y, ws, stream=None) -> None:
    """T = u.shape[-1] steps from ``state`` ([batch, H, N, 2], updated in place)."""
    p, (H, N, L, batch) = _dims(plan)
    _validate("recurrent_scan", D=D, u=u, state=state)
    if u is None or u.dim() != 3:
        raise ValueError("u: expected a [batch, H, T] tensor")
    T = int(u.shape[-1])
    _check(_lib.s4dplr_recurrent_scan(
        p, _ptr(D, "D", (H,)), _ptr(u, "u", (batch, H, T)), T,
        _ptr(state, "state", (batch, H, N, 2)), _ptr(y, "y", (batch, H, T)), _ws_ptr(ws),
        _stream(stream)), "recurrent_scan")


def conv_bwd(plan: "Plan | int", u, K, D, dy, du, dK, dD, ws, stream=None) -> None:
    _validate("conv_bwd", u=u, K=K, D=D, dy=dy)
    p, (H, N, L, batch) = _dims(plan)
    _check(_lib.s4dplr_conv_bwd(
        p, _ptr(u, "u", (batch, H, L)), _ptr(K, "K", (H, L)), _ptr(D, "D", (H,)),
        _ptr(dy, "dy", (batch, H, L)), _ptr(du, "du", (batch, H, L)), _ptr(dK, "dK", (H, L)),
        _ptr(dD, "dD", (H,)), _ws_ptr(ws), _stream(stream)), "conv_bwd")


def kernel_gen_bwd(plan: "Plan | int", lam, P, Q, B, C, dt, dK, dlam, dP, dQ, dB, dC, ddt, ws,
                   stream=None) -> None:
    _validate("kernel_gen_bwd", lam=lam, dt=dt, P=P, Q=Q, B=B, C=C, dK=dK)
    p, (H, N, L, _) = _dims(plan)
    cplx = (H, N, 2)
    lr = _lowrank_shape(plan)
    _check(_lib.s4dplr_kernel_gen_bwd(
        p, _ptr(lam, "lam", cplx), _ptr(P, "P", lr), _ptr(Q, "Q", lr), _ptr(B, "B", cplx),
        _ptr(C, "C", cplx), _ptr(dt, "dt", (H,)), _ptr(dK, "dK", (H, L)),
        _ptr(dlam, "dlam", cplx), _ptr(dP, "dP", lr), _ptr(dQ, "dQ", lr),
        _ptr(dB, "dB", cplx), _ptr(dC, "dC", cplx), _ptr(ddt, "ddt", (H,)), _ws_ptr(ws),
        _stream(stream)), "kernel_gen_bwd")


def block_forward(plan: "Plan | int", x, gamma, beta, lam, P, Q, B, C, dt, D, W, bias, out, ws,
                  stream=None) -> None:
    _validate("block_forward", lam=lam, dt=dt, x=x, gamma=gamma, beta=beta, P=P, Q=Q, B=B, C=C,
              D=D, W=W, bias=bias)
    p, (H, N, L, batch) = _dims(plan)
    cplx = (H, N, 2)
    lr = _lowrank_shape(plan)
    _check(_lib.s4dplr_block_forward(
        p, _ptr(x, "x", (batch, H, L)), _ptr(gamma, "gamma", (H,)), _ptr(beta, "beta", (H,)),
        _ptr(lam, "lam", cplx), _ptr(P, "P", lr), _ptr(Q, "Q", lr), _ptr(B, "B", cplx),
        _ptr(C, "C", cplx), _ptr(dt, "dt", (H,)), _ptr(D, "D", (H,)), _ptr(W, "W", (2 * H, H)),
        _ptr(bias, "bias", (2 * H,)), _ptr(out, "out", (batch, H, L)), _ws_ptr(ws),
        _stream(stream)), "block_forward")


def _dims(plan):
    if isinstance(plan, Plan):
        return plan.handle, (plan.H, plan.N, plan.L, plan.batch)
    raise TypeError("pass a Plan (its sizes are needed to check tensor shapes)")


def _lowrank_shape(plan):
    """Shape of P and Q: [H, N, 2] at rank 1, [H, r, N, 2] at rank r > 1."""
    if plan.rank == 1:
        return (plan.H, plan.N, 2)
    return (plan.H, plan.rank, plan.N, 2)


class Plan:
    """Owns a plan handle and (optionally) a workspace tensor on one device."""

    def __init__(self, H: int, N: int, L: int, batch: int, diagonal: bool = False,
                 device=None, zoh: bool = False, block: bool = False, rank: int = 1):
        self.H, self.N, self.L, self.batch = H, N, L, batch
        self.diagonal, self.zoh, self.block, self.rank = diagonal, zoh, block, rank
        self.handle = plan_create(H, N, L, batch, (DIAGONAL if diagonal else 0)
                                  | (ZOH if zoh else 0) | (BLOCK if block else 0)
                                  | ((rank << RANK_SHIFT) if rank != 1 else 0))
        self.workspace_bytes = plan_workspace_bytes(self.handle)
        self.device = torch.device("cuda" if device is None else device)
        self._ws_store = None
        self._ws = None

    def workspace(self, stream=None):
        """A 256-byte aligned workspace tensor with the tables already written."""
        if self._ws is None:
            store = torch.empty(self.workspace_bytes + 256, dtype=torch.uint8, device=self.device)
            off = (-store.data_ptr()) % 256
            self._ws_store = store
            self._ws = store[off: off + self.workspace_bytes]
            plan_init(self.handle, self._ws, stream)
        return self._ws

    def close(self) -> None:
        if self.handle:
            plan_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------- token-major operators

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
DELTA_TRAINING = 1


def _tensor(t, name, dtype, shape, device=None, optional=False):
    """Device pointer of a contiguous GPU tensor of that dtype and shape."""
    if t is None and optional:
        return None
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and \
            t.is_contiguous() and t.is_cuda and (device is None or t.device == device):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    return t.data_ptr()


def _rows(t, name, dtype, shape, device):
    """Device pointer and row pitch of a [rows, heads, d] tensor whose rows are
    contiguous (a column range of a wider matrix will do)."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and \
            t.is_contiguous() and t.is_cuda and t.device == device:
        return t.data_ptr(), shape[1] * shape[2]
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a GPU tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    n, heads, d = shape
    sr, sh, sd = t.stride()
    if (d > 1 and sd != 1) or (heads > 1 and sh != d) or (n > 1 and sr < heads * d):
        raise ValueError(f"{name}: each row must be contiguous and apart from the others, "
                         f"got strides {tuple(t.stride())}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    return t.data_ptr(), sr if n > 1 else heads * d


def _launch(device, stream, fn, args):
    """``fn(*args, stream)`` with ``device`` current."""
    index = device.index
    # the raw handle of the device's current stream, without a Stream object
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)
    if index == torch.cuda.current_device():
        return fn(*args, raw)
    with torch.cuda.device(device):
        return fn(*args, raw)


def _workspace(ws, name, need, device):
    if type(ws) is torch.Tensor and ws.dtype is torch.uint8 and ws.device == device and \
            ws.is_contiguous() and ws.numel() >= need:
        return ws.data_ptr()
    if not isinstance(ws, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if ws.device != device:
        raise ValueError(f"{name}: on {ws.device}, expected {device}")
    if not ws.is_contiguous() or ws.numel() * ws.element_size() < need:
        raise ValueError(f"{name}: must be contiguous and at least {need} bytes")
    return ws.data_ptr()


def _aligned(nbytes: int, device):
    """A 256-byte aligned uint8 tensor."""
    store = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
    off = (-store.data_ptr()) % 256
    return store[off: off + nbytes]


def _norm_dims(x, axis):
    """(outer, D, inner) and the shape of the statistics."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x: expected a torch.Tensor")
    if x.dtype not in _DTYPES:
        raise TypeError(f"x: must be float32, bfloat16 or float16, got {x.dtype}")
    shape = x.shape
    axis = axis + len(shape) if axis < 0 else axis
    if axis == 1 and len(shape) == 2:
        return shape[0], shape[1], 1, shape[:1]
    if not 0 <= axis < len(shape):
        raise ValueError(f"axis: out of range for {len(shape)} dimensions")
    outer = inner = 1
    for n in shape[:axis]:
        outer *= n
    for n in shape[axis + 1:]:
        inner *= n
    if inner == 0:               # no vectors at all
        outer, inner = 0, 1
    return outer, shape[axis], inner, shape[:axis] + shape[axis + 1:]


def layer_norm_fwd(x, gamma, beta, y, mean=None, rstd=None, eps: float = 1e-5, axis: int = -1,
                   stream=None) -> None:
    """``y`` = the layer norm of ``x`` along ``axis``; ``mean`` and ``rstd``
    (float32, the shape of ``x`` without that axis) are what
    ``layer_norm_bwd`` reads.  gamma, beta: [D] float32 or None (1 and 0)."""
    outer, D, inner, stat = _norm_dims(x, axis)
    dev = x.device
    if validation_enabled():
        check_preconditions("layer_norm_fwd", x=x, gamma=gamma, beta=beta)
    f32 = torch.float32
    args = (_tensor(x, "x", x.dtype, x.shape),
            _tensor(gamma, "gamma", f32, (D,), dev, True),
            _tensor(beta, "beta", f32, (D,), dev, True),
            _tensor(y, "y", x.dtype, x.shape, dev),
            _tensor(mean, "mean", f32, stat, dev, True),
            _tensor(rstd, "rstd", f32, stat, dev, True), outer, D, inner, eps, _DTYPES[x.dtype])
    _check(_launch(dev, stream, _lib.s4dplr_layer_norm_fwd, args),
           "layer_norm_fwd")


@functools.lru_cache(maxsize=1024)      # a call through ctypes takes longer than this
def _norm_workspace(outer, D, inner, where):
    n = ctypes.c_size_t()
    _check(_lib.s4dplr_layer_norm_workspace_bytes(outer, D, inner, ctypes.byref(n)), where)
    return n.value


def layer_norm_workspace_bytes(x, axis: int = -1) -> int:
    """Bytes of workspace of ``layer_norm_bwd`` for this ``x``."""
    outer, D, inner, _ = _norm_dims(x, axis)
    return _norm_workspace(outer, D, inner, "layer_norm_workspace_bytes")


def layer_norm_bwd(x, gamma, mean, rstd, dy, dx, dgamma, dbeta, ws, axis: int = -1,
                   stream=None) -> None:
    """Gradients of ``layer_norm_fwd``; any of dx, dgamma, dbeta may be None.
    ``ws``: a 256-byte aligned GPU tensor of ``layer_norm_workspace_bytes``."""
    outer, D, inner, stat = _norm_dims(x, axis)
    dev = x.device
    if validation_enabled():
        check_preconditions("layer_norm_bwd", x=x, gamma=gamma, mean=mean, rstd=rstd, dy=dy)
    f32, full = torch.float32, x.shape
    need = _norm_workspace(outer, D, inner, "layer_norm_bwd")
    args = (_tensor(x, "x", x.dtype, full), _tensor(gamma, "gamma", f32, (D,), dev, True),
            _tensor(mean, "mean", f32, stat, dev), _tensor(rstd, "rstd", f32, stat, dev),
            _tensor(dy, "dy", x.dtype, full, dev), _tensor(dx, "dx", x.dtype, full, dev, True),
            _tensor(dgamma, "dgamma", f32, (D,), dev, True),
            _tensor(dbeta, "dbeta", f32, (D,), dev, True), outer, D, inner, _DTYPES[x.dtype],
            _workspace(ws, "ws", need, dev))
    _check(_launch(dev, stream, _lib.s4dplr_layer_norm_bwd, args),
           "layer_norm_bwd")


class DeltaPlan:
    """A plan of the gated delta rule: ``sequences`` sequences packed into
    ``tokens`` rows, Hk key heads of dk and Hv value heads of dv values.
    ``training`` reserves what ``delta_bwd`` needs."""

    def __init__(self, sequences: int, tokens: int, Hk: int, Hv: int, dk: int, dv: int,
                 dtype=torch.bfloat16, training: bool = False, device=None):
        if dtype not in _DTYPES:
            raise TypeError(f"dtype: must be float32, bfloat16 or float16, got {dtype}")
        self.handle = 0
        self.sequences, self.tokens, self.Hk, self.Hv = sequences, tokens, Hk, Hv
        self.dk, self.dv, self.dtype, self.training = dk, dv, dtype, training
        if not all(abs(n) < 1 << 31 for n in (sequences, tokens, Hk, Hv, dk, dv)):
            raise S4DPLRError(2, "delta_plan_create")      # ctypes would wrap them
        h = _p()
        _check(_lib.s4dplr_delta_plan_create(
            ctypes.byref(h), sequences, tokens, Hk, Hv, dk, dv, _DTYPES[dtype],
            DELTA_TRAINING if training else 0), "delta_plan_create")
        self.handle = h.value
        a, b = ctypes.c_size_t(), ctypes.c_size_t()
        _check(_lib.s4dplr_delta_plan_bytes(self.handle, ctypes.byref(a), ctypes.byref(b)),
               "delta_plan_bytes")
        self.workspace_bytes, self.saved_bytes = a.value, b.value
        self._keys, self._vals = (tokens, Hk, dk), (tokens, Hv, dv)
        self._heads, self._states = (tokens, Hv), (sequences, Hv, dk, dv)
        self._scale = dk ** -0.5
        self.device = torch.device("cuda" if device is None else device)
        self._ws = None

    def workspace(self):
        """A workspace tensor, one per plan object: calls that can overlap in
        time, and graphs that can replay together, need one each."""
        if self._ws is None:
            self._ws = _aligned(self.workspace_bytes, self.device)
        return self._ws

    def saved(self):
        """A new buffer for ``delta_fwd(saved=...)``, one per layer and step."""
        if not self.training:
            raise ValueError("saved: the plan was made without training=True")
        return _aligned(self.saved_bytes, self.device)

    def close(self) -> None:
        if self.handle:
            _lib.s4dplr_delta_plan_destroy(self.handle)
            self.handle = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _validate_delta(where, plan, offsets, rows, states):
    """The preconditions of ``delta_fwd`` and ``delta_bwd``: offsets that rise within the rows,
    finite values and g <= 0 in the sequences' rows (the others are not read)."""
    lo, hi = 0, plan.tokens
    at = [] if offsets is None else [int(i) for i in _host(offsets).flatten()]
    if len(at) == plan.sequences + 1:       # any other length is refused behind this
        for i, (a, b) in enumerate(zip([0, *at], [*at, plan.tokens])):
            if a > b:
                what = f"offsets[{i}] = {b} < {a}" if i < len(at) else f"offsets end at {a} > {b} rows"
                raise S4DPLRPreconditionError(where, what)
        lo, hi = at[0], at[-1]
    for name, t in {**rows, **states}.items():
        if t is None:
            continue
        h = _host(t)
        bad = ~(h <= 0) if name == "g" else ~torch.isfinite(h)      # g = -infinity is a reset
        if name in rows and h.dim() > 0:
            bad[:lo] = False
            bad[hi:] = False
        if bool(bad.any()):
            idx = tuple(int(i) for i in bad.nonzero()[0])
            raise S4DPLRPreconditionError(where, f"g must be <= 0, not so at index {idx}" if name == "g"
                                          else f"{name} is not finite at index {idx}")


def _delta_inputs(where, plan, q, k, v, g, beta, ws, scale, offsets, state=None, dout=None,
                  dstate_out=None):
    if not isinstance(plan, DeltaPlan):
        raise TypeError("pass a DeltaPlan")
    if not plan.handle:
        raise ValueError("the plan is closed")
    if not isinstance(v, torch.Tensor):
        raise TypeError("v: expected a torch.Tensor")
    if validation_enabled():
        _validate_delta(where, plan, offsets, dict(q=q, k=k, v=v, g=g, beta=beta, dout=dout),
                        dict(state=state, dstate_out=dstate_out))
    dev, dt, f32 = v.device, plan.dtype, torch.float32
    keys, heads = plan._keys, plan._heads
    off = None
    if offsets is not None:
        off = _tensor(offsets, "offsets", torch.int32, (plan.sequences + 1,), dev)
    return dev, (plan.handle, *_rows(q, "q", dt, keys, dev), *_rows(k, "k", dt, keys, dev),
                 *_rows(v, "v", dt, plan._vals, dev),
                 _tensor(g, "g", f32, heads, dev), _tensor(beta, "beta", f32, heads, dev), off,
                 plan._scale if scale is None else float(scale)), \
        _workspace(ws, "ws", plan.workspace_bytes, dev)


def delta_fwd(plan: "DeltaPlan", q, k, v, g, beta, state, o, state_out, ws, saved=None,
              scale=None, offsets=None, stream=None) -> None:
    """``o`` and the states behind the last rows, from ``state`` (None: zeros).

    q, k: [tokens, Hk, dk]; v, o: [tokens, Hv, dv]; g (log decay), beta:
    [tokens, Hv] float32; state, state_out: [sequences, Hv, dk, dv] float32, may
    be one tensor, state_out may be None.  q, k, v may be column ranges of wider
    matrices.  offsets: [sequences + 1] int32 on the GPU, or None for equal
    lengths.  scale: None is dk ** -0.5.  saved: ``plan.saved()`` for a later
    ``delta_bwd``."""
    dev, args, w = _delta_inputs("delta_fwd", plan, q, k, v, g, beta, ws, scale, offsets,
                                 state=state)
    st, f32 = plan._states, torch.float32
    args += (_tensor(state, "state", f32, st, dev, True),
             _tensor(o, "o", plan.dtype, plan._vals, dev),
             _tensor(state_out, "state_out", f32, st, dev, True),
             None if saved is None else _workspace(saved, "saved", plan.saved_bytes, dev), w)
    _check(_launch(dev, stream, _lib.s4dplr_delta_fwd, args), "delta_fwd")


def delta_bwd(plan: "DeltaPlan", q, k, v, g, beta, saved, dout, dstate_out, dq, dk, dv, dg, dbeta,
              dstate, ws, scale=None, offsets=None, stream=None) -> None:
    """Gradients of ``delta_fwd`` with the same inputs and the ``saved`` buffer
    it filled, from ``dout`` and ``dstate_out`` (None: zeros); any of dq, dk, dv,
    dg, dbeta, dstate may be None."""
    dev, args, w = _delta_inputs("delta_bwd", plan, q, k, v, g, beta, ws, scale, offsets,
                                 dout=dout, dstate_out=dstate_out)
    dt, f32 = plan.dtype, torch.float32
    st, keys, vals, heads = plan._states, plan._keys, plan._vals, plan._heads
    args += (_workspace(saved, "saved", plan.saved_bytes, dev),
             _tensor(dout, "dout", dt, vals, dev),
             _tensor(dstate_out, "dstate_out", f32, st, dev, True),
             _tensor(dq, "dq", dt, keys, dev, True), _tensor(dk, "dk", dt, keys, dev, True),
             _tensor(dv, "dv", dt, vals, dev, True), _tensor(dg, "dg", f32, heads, dev, True),
             _tensor(dbeta, "dbeta", f32, heads, dev, True),
             _tensor(dstate, "dstate", f32, st, dev, True), w)
    _check(_launch(dev, stream, _lib.s4dplr_delta_bwd, args), "delta_bwd")
