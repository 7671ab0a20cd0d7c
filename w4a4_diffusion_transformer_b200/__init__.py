"""SVDQuant W4A4 linear layer for NVIDIA B200 (sm_100a).

A thin ctypes binding over the C ABI in ``include/svdq.h`` (``libsvdq.so``,
built in-tree by ``w4a4_diffusion_transformer_b200.build``).  The binding only
marshals arguments: every step of the layer runs in the library (host C++ for
the offline preparation, CUDA kernels for the forward).  There is no fallback:
if the library is missing, importing ``lib`` raises.

Device memory and streams come from the caller (for example PyTorch tensors:
anything with ``data_ptr()``, or raw integer addresses).  PyTorch tensors and
NumPy arrays are checked before the call: a device operand must be a
contiguous CUDA tensor, a host operand host memory, and each must hold at
least the bytes the call reads or writes (``ValueError`` otherwise).  Raw
addresses and other objects are passed through unchecked.
"""
from __future__ import annotations

import ctypes
import os
import sys
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsvdq.so")

# status codes (svdq_status)
OK, EINVAL, EUNSUPPORTED, ENOMEM, ECUDA, ENOCONVERGE, ETIMEOUT, ESTATE = range(8)
# formats (svdq_format)
NVFP4, INT4, W4A16_INT4, W8A8_INT8 = 0, 1, 2, 3
FORMATS = {"nvfp4": NVFP4, "int4": INT4, "w4a16": W4A16_INT4, "w8a8": W8A8_INT8}
# forward flags
FWD_GELU, FWD_UNFUSED, FWD_NO_BRANCH, FWD_CHECK = 0x1, 0x2, 0x4, 0x8
# exportable tensors (svdq_tensor)
TENSORS = {
    "lambda": (0, np.float32), "inv_lambda": (1, np.float32), "L1": (2, np.float64), "L2": (3, np.float64),
    "L1d": (4, np.uint16), "L2b": (5, np.uint16), "R": (6, np.float32), "sigma": (7, np.float64),
    "w_codes": (8, np.uint8), "w_scales": (9, None), "bias": (10, np.float32), "gptq_U": (11, np.float64),
    "lora_A": (12, np.uint16), "lora_B": (13, np.uint16),
}
# preparation flags (svdq_config.flags)
PREP_GPTQ, PREP_KEEP_GPTQ_FACTOR = 0x1, 0x2
# normalisation flags (svdq_norm.flags)
NORM_CENTER = 0x1
# rotary position flags (svdq_rope.flags)
ROPE_HALF, ROPE_SPAN, ROPE_NORM = 0x1, 0x2, 0x4

EXPORTED = [
    "svdq_prepare", "svdq_destroy", "svdq_get_info", "svdq_tensor_bytes", "svdq_export",
    "svdq_status_string", "svdq_workspace_bytes", "svdq_linear_forward", "svdq_quantize_act",
    "svdq_gemm", "svdq_act_scale_bytes", "svdq_act_scales_to_logical", "svdq_check",
    "svdq_linear_forward_static", "svdq_act_code_bytes", "svdq_act_codes_to_logical",
    "svdq_selftest_wait_timeout", "svdq_mlp_workspace_bytes", "svdq_mlp_fc1", "svdq_mlp_forward",
    "svdq_set_lora", "svdq_serialized_bytes", "svdq_serialize", "svdq_deserialize",
    "svdq_norm_quantize_act", "svdq_norm_linear_forward", "svdq_rope_heads", "svdq_qkv_forward",
    "svdq_gemm_residual", "svdq_linear_forward_residual", "svdq_mlp_block_forward",
]
STATIC_WORKSPACE_BYTES = 16 << 20   # SVDQ_STATIC_WORKSPACE_BYTES


class SvdqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class Config(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int), ("rank", ctypes.c_int), ("alpha", ctypes.c_float),
                ("flags", ctypes.c_uint)]


class LayerInfo(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int), ("N", ctypes.c_int), ("rank", ctypes.c_int), ("format", ctypes.c_int),
                ("device", ctypes.c_int), ("g_x_exp", ctypes.c_int), ("g_w_exp", ctypes.c_int),
                ("svd_iterations", ctypes.c_int), ("svd_tail_energy", ctypes.c_double)]


class NormStruct(ctypes.Structure):
    _fields_ = [("residual", ctypes.c_void_p), ("sum", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("shift", ctypes.c_void_p), ("mod_stride", ctypes.c_int64),
                ("rows_per_mod", ctypes.c_int), ("eps", ctypes.c_float), ("flags", ctypes.c_uint)]


class ResidualStruct(ctypes.Structure):
    _fields_ = [("residual", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_int64),
                ("rows_per_gate", ctypes.c_int)]


class RopeStruct(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int), ("dim", ctypes.c_int * 4), ("head_dim", ctypes.c_int),
                ("theta", ctypes.c_double), ("eps", ctypes.c_float), ("flags", ctypes.c_uint)]


class HeadsStruct(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int),
                ("in_batch", ctypes.c_int64), ("in_token", ctypes.c_int64), ("in_head", ctypes.c_int64),
                ("out_batch", ctypes.c_int64), ("out_token", ctypes.c_int64), ("out_head", ctypes.c_int64),
                ("weight", ctypes.c_void_p)]


_lib: Optional[ctypes.CDLL] = None


def load() -> ctypes.CDLL:
    """Load libsvdq.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m w4a4_diffusion_transformer_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, SZ, U = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint
    sig = {
        "svdq_prepare": (I, [ctypes.POINTER(Config), I, I, P, P, P, I, I, ctypes.POINTER(P)]),
        "svdq_destroy": (None, [P]),
        "svdq_get_info": (I, [P, ctypes.POINTER(LayerInfo)]),
        "svdq_tensor_bytes": (SZ, [P, I]),
        "svdq_export": (I, [P, I, P, SZ]),
        "svdq_status_string": (ctypes.c_char_p, [I]),
        "svdq_workspace_bytes": (SZ, [P, I]),
        "svdq_linear_forward": (I, [P, P, I, P, P, SZ, P, U]),
        "svdq_quantize_act": (I, [P, P, I, P, P, P, P, I]),
        "svdq_gemm": (I, [P, P, P, P, I, P, P, U]),
        "svdq_act_scale_bytes": (SZ, [P, I]),
        "svdq_act_scales_to_logical": (I, [P, P, I, P]),
        "svdq_check": (I, [P, P]),
        "svdq_linear_forward_static": (I, [P, P, I, P, P, U]),
        "svdq_act_code_bytes": (SZ, [P, I]),
        "svdq_act_codes_to_logical": (I, [P, P, I, P]),
        "svdq_selftest_wait_timeout": (I, [P, U, P]),
        "svdq_mlp_workspace_bytes": (SZ, [P, P, I, U]),
        "svdq_mlp_fc1": (I, [P, P, P, I, P, P, P, P, SZ, P, U]),
        "svdq_mlp_forward": (I, [P, P, P, I, P, P, SZ, P, U]),
        "svdq_set_lora": (I, [P, I, P, P, ctypes.c_float]),
        "svdq_serialized_bytes": (SZ, [P]),
        "svdq_serialize": (I, [P, P, SZ]),
        "svdq_deserialize": (I, [P, SZ, I, ctypes.POINTER(P)]),
        "svdq_norm_quantize_act": (I, [P, P, P, I, P, P, P, P, P]),
        "svdq_norm_linear_forward": (I, [P, P, P, I, P, P, SZ, P, U]),
        "svdq_gemm_residual": (I, [P, P, P, P, I, P, P, P, U]),
        "svdq_linear_forward_residual": (I, [P, P, I, P, P, P, SZ, P, U]),
        "svdq_mlp_block_forward": (I, [P, P, P, P, I, P, P, P, SZ, P, U]),
        "svdq_rope_heads": (I, [P, P, P, I, I, P, ctypes.c_int64, P]),
        "svdq_qkv_forward": (I, [P, P, P, I, I, P, I, I, P, P, P, ctypes.c_int64, P, P, SZ, P, U]),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def status_string(s: int) -> str:
    return load().svdq_status_string(int(s)).decode()


def _ptr(x) -> Optional[int]:
    """Device/host address of a tensor-like object (data_ptr()), an int, or None."""
    if x is None:
        return None
    if x.__class__ is _torch_tensor:
        return x.data_ptr()
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return int(x.data_ptr())
    if isinstance(x, np.ndarray):
        return int(x.ctypes.data)
    raise TypeError(f"cannot take the address of {type(x)}")


def _held_bytes(x, what: str, device: bool) -> Optional[int]:
    """Bytes held by a tensor or array argument after checking where it lives
    and that it is contiguous; None for raw addresses and unknown objects."""
    if x is None or isinstance(x, int):
        return None
    if isinstance(x, np.ndarray):
        if device:
            raise ValueError(f"{what}: a NumPy array is host memory; this operand is a device buffer")
        if not x.flags.c_contiguous:
            raise ValueError(f"{what}: not contiguous")
        return int(x.nbytes)
    if hasattr(x, "is_cuda") and hasattr(x, "numel"):
        if bool(x.is_cuda) != device:
            raise ValueError(f"{what}: must be a {'CUDA' if device else 'host'} tensor")
        if not x.is_contiguous():
            raise ValueError(f"{what}: not contiguous")
        return int(x.numel()) * int(x.element_size())
    return None


_torch_tensor = None                                   # torch.Tensor, once one was passed


def _plain_tensor(x) -> bool:
    """Whether x is a torch.Tensor itself (torch need not be importable)."""
    global _torch_tensor
    if _torch_tensor is None:
        torch = sys.modules.get("torch")
        if torch is None:
            return False
        _torch_tensor = torch.Tensor
    return x.__class__ is _torch_tensor


def _need(x, nbytes: int, what: str, device: bool = True, on: int = -1):
    """x holds nbytes on a device (or the host); with on >= 0, on that device."""
    # the usual operand, a contiguous tensor in the right place, without detours
    if x.__class__ is _torch_tensor and x.is_contiguous() and x.nbytes >= nbytes and (
            x.is_cuda is device if on < 0 else x.get_device() == on):
        return
    _plain_tensor(x)                                    # (the first call: torch is known from now on)
    have = _held_bytes(x, what, device)
    if have is not None and have < nbytes:
        raise ValueError(f"{what}: holds {have} bytes, the call accesses {nbytes}")
    if on >= 0 and hasattr(x, "get_device") and x.get_device() != on:
        raise ValueError(f"{what}: on device {x.get_device()}, the layer is on device {on}")


def _stream(s) -> Optional[int]:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return int(getattr(s, "cuda_stream"))


def _check(status: int, what: str):
    if status != OK:
        raise SvdqError(status, what)


def _is_tensor(x) -> bool:
    return hasattr(x, "is_cuda") and hasattr(x, "stride")


def _bf16_tensor(x, what: str):
    if not x.is_cuda:
        raise ValueError(f"{what}: must be a CUDA tensor")
    if x.element_size() != 2 or not x.dtype.is_floating_point or str(x.dtype) != "torch.bfloat16":
        raise ValueError(f"{what}: must be BF16, got {x.dtype}")
    if hasattr(x, "untyped_storage") and x.numel() > 0:
        end = x.storage_offset() + sum((n - 1) * s for n, s in zip(x.shape, x.stride())) + 1
        if x.untyped_storage().nbytes() < 2 * end:
            raise ValueError(f"{what}: its storage has been released")


class _Described:
    """Operands that the library gets as one struct (_c).  The checks of placement
    and layout run when the struct is filled; a tensor can get another storage
    later (tensor.data = ..., a module moved between devices), so every call
    compares the addresses first, and fills the struct again where one changed.  An
    alias of each operand keeps its storage until then, so that the same address is
    the same memory, whatever happened to the tensor in between.  (Comparing sizes
    and types at each call too would cost 0.7 us more for a rotation's six operands;
    a tensor that shows the same memory in another shape keeps the layout it was
    described with.)"""

    def _hold(self, *operands):
        self._keep = operands
        self._fill()

    def _fill(self):
        self._seen = self._aliases = None              # a refused operand is looked at again
        self._describe()
        on = {x.get_device() for x in self._keep if hasattr(x, "get_device")}
        if len(on) > 1:
            raise ValueError(f"{type(self).__name__}: its tensors must be on one device, got {sorted(on)}")
        self.device = on.pop() if on else None
        self._ref_c = ctypes.byref(self._c)
        if not any(hasattr(x, "data_ptr") and not _is_tensor(x) for x in self._keep):   # (those: at every call)
            tensors = [x for x in self._keep if _is_tensor(x)]
            self._aliases = [x.detach() for x in tensors if hasattr(x, "detach")]
            self._seen = [(x, x.data_ptr()) for x in tensors]

    def _now(self):
        """The struct as a call's argument, with the operands as they are now."""
        seen = self._seen                              # one read: another thread may fill it anew
        if seen is None:
            self._fill()
        else:
            for x, ptr in seen:
                if x.data_ptr() != ptr:
                    self._fill()
                    break
        return self._ref_c

    _ref = property(_now)

    def _on(self, device: int):
        if self.device is not None and self.device != device and device >= 0:
            raise ValueError(f"{type(self).__name__}: its tensors are on device {self.device}, the layer is on "
                             f"device {device}")


class _Rows:
    """Rows of BF16 values shared by runs of tokens (modulation scale and
    shift, a gate): a 1D tensor is one row for all tokens, a 2D tensor -- a
    column range of a wider one too -- row m // per for token m (per 0: row 0).
    A raw address takes its stride from the caller and is not checked."""

    def __init__(self, x, what: str, stride: Optional[int], stride_name: str, per: int):
        self.what, self.x, self.rows, self.cols = what, x, None, None
        self.stride = stride
        if not _is_tensor(x) and per > 0 and stride is None:
            raise ValueError(f"{what}: an address says nothing of its rows' distance: give {stride_name}")
        if _is_tensor(x):
            _bf16_tensor(x, what)
            if x.dim() not in (1, 2) or x.stride(-1) != 1:
                raise ValueError(f"{what}: must be [columns] or [rows][columns] with contiguous columns")
            self.rows, self.cols = (1, x.shape[0]) if x.dim() == 1 else (x.shape[0], x.shape[1])
            # the stride of a single row says nothing
            if self.rows > 1:
                self.stride = x.stride(0)
            elif stride is None:
                self.stride = self.cols

    def need(self, M: int, cols: int, per: int):
        if self.rows is None:
            return
        if self.cols < cols:
            raise ValueError(f"{self.what}: {self.cols} columns, the call reads {cols}")
        need = 1 if per <= 0 else -(-M // per)
        if self.rows < need:
            raise ValueError(f"{self.what}: {self.rows} rows, the call reads {need}")


class Norm(_Described):
    """A normalisation in front of a layer (svdq_norm): optional residual
    addition (``sum`` receives it), RMS norm -- or layer norm with ``center`` --
    times ``weight`` and modulated by rows of ``scale`` and ``shift``, of which
    token m uses row m // rows_per_mod (0: row 0).  Holds references to its
    tensors; one object can be used for any number of calls."""

    def __init__(self, residual=None, sum=None, weight=None, scale=None, shift=None, rows_per_mod: int = 0,
                 mod_stride: Optional[int] = None, eps: float = 1e-6, center: bool = False):
        self._mod_stride, self._per, self._eps, self._center = mod_stride, int(rows_per_mod), float(eps), bool(center)
        self._hold(residual, sum, weight, scale, shift)

    def _describe(self):
        residual, sum, weight, scale, shift = self._keep
        mod_stride = self._mod_stride
        self._held = []
        for t, what in ((residual, "residual"), (sum, "sum"), (weight, "weight")):
            if _is_tensor(t):
                _bf16_tensor(t, what)
            held = _held_bytes(t, what, True)
            if held is not None:
                self._held.append((held, what == "weight", what))
        rows = [_Rows(t, what, mod_stride, "mod_stride", self._per) for t, what in ((scale, "scale"), (shift, "shift")) if t is not None]
        strides = {r.stride for r in rows if r.rows != 1 or mod_stride is not None}
        if len(strides) > 1:
            raise ValueError("scale and shift: their rows must be the same distance apart")
        stride = strides.pop() if strides else 0
        self._rows = rows
        self._c = NormStruct(_ptr(residual), _ptr(sum), _ptr(weight), _ptr(scale), _ptr(shift), int(stride or 0),
                             self._per, self._eps, NORM_CENTER if self._center else 0)

    def _args(self, device: int, M: int, K: int):
        """The struct for a layer's call over M tokens, sizes checked."""
        now = self._now()
        self._on(device)
        if M <= 0:
            return now                 # the library answers M <= 0 itself
        for held, one_row, what in self._held:
            need = K * 2 if one_row else M * K * 2
            if held < need:
                raise ValueError(f"{what}: holds {held} bytes, the call accesses {need}")
        for r in self._rows:
            r.need(M, K, self._per)
        return now


class Residual(_Described):
    """A residual in a GEMM's epilogue (svdq_residual): Y = residual + gate * y,
    token m gated by row m // rows_per_gate (0: row 0; no gate: 1).  Holds
    references to its tensors; one object can be used for any number of calls."""

    def __init__(self, residual, gate=None, rows_per_gate: int = 0, gate_stride: Optional[int] = None):
        self._gate_stride, self._per = gate_stride, int(rows_per_gate)
        self._hold(residual, gate)

    def _describe(self):
        residual, gate = self._keep
        if _is_tensor(residual):
            _bf16_tensor(residual, "residual")
        self._held = _held_bytes(residual, "residual", True)
        self._rows = None if gate is None else _Rows(gate, "gate", self._gate_stride, "gate_stride", self._per)
        stride = 0 if self._rows is None or self._rows.rows == 1 else self._rows.stride or 0
        self._c = ResidualStruct(_ptr(residual), _ptr(gate), int(stride), self._per)

    def _args(self, device: int, M: int, N: int):
        """The struct for a layer's call over M tokens, sizes checked."""
        now = self._now()
        self._on(device)
        if M <= 0:
            return now
        if self._held is not None and self._held < M * N * 2:
            raise ValueError(f"residual: holds {self._held} bytes, the call accesses {M * N * 2}")
        if self._rows is not None:
            self._rows.need(M, N, self._per)
        return now


class Rope:
    """Rotary positions with several axes (svdq_rope): dims[a] values of a head
    belong to axis a; ``half`` pairs values half the span apart instead of
    neighbours, ``span`` runs the frequencies over the whole span instead of
    each axis, ``norm`` puts the per-head RMS norm in front."""

    def __init__(self, head_dim: int, dims, theta: float = 10000.0, half: bool = False, span: bool = False,
                 norm: bool = False, eps: float = 1e-6):
        dims = tuple(int(d) for d in dims)
        if not 1 <= len(dims) <= 4:
            raise ValueError(f"1 to 4 axes, got {len(dims)}")
        self.head_dim, self.axes = int(head_dim), len(dims)
        self._c = RopeStruct(len(dims), (ctypes.c_int * 4)(*dims), int(head_dim), float(theta), float(eps),
                             (ROPE_HALF if half else 0) | (ROPE_SPAN if span else 0) | (ROPE_NORM if norm else 0))

    # a reference made at the call: a copied or unpickled object has a struct of its own
    _ref = property(lambda self: ctypes.byref(self._c))


class Heads(_Described):
    """The heads of queries or keys (svdq_heads): BF16 CUDA tensors
    [batch, token, head, head_dim] -- or [token, head, head_dim] -- of any
    strides over contiguous values; out None is in place.  Holds references to
    its tensors; one object can be used for any number of calls."""

    def __init__(self, x, out=None, weight=None):
        self._hold(x, x if out is None else out, weight)

    def _describe(self):
        x, out, weight = self._keep
        shapes = []
        for t, what in ((x, "x"), (out, "out")):
            _bf16_tensor(t, what)
            if t.dim() not in (3, 4) or t.stride(-1) != 1:
                raise ValueError(f"{what}: must be [batch, token, head, head_dim] with contiguous values")
            shapes.append(tuple(t.shape) if t.dim() == 4 else (1,) + tuple(t.shape))
        if shapes[0] != shapes[1]:
            raise ValueError(f"x and out differ in shape: {shapes[0]} and {shapes[1]}")
        self.batch, self.tokens, self.heads, self.head_dim = shapes[0]
        if weight is not None:
            if _is_tensor(weight):
                _bf16_tensor(weight, "weight")
            _need(weight, self.head_dim * 2, "weight")

        def strides(t):
            s = tuple(t.stride())[:-1]
            s = s if t.dim() == 4 else (0,) + s
            # the stride of an axis of one is not used
            return [v if n > 1 else 0 for v, n in zip(s, shapes[0])]
        self._c = HeadsStruct(_ptr(x), _ptr(out), self.heads, *strides(x), *strides(out), _ptr(weight))


_float32 = None                                        # torch.float32, once positions were passed


def _is_float32(dtype) -> bool:
    global _float32
    if dtype is not _float32 and str(dtype) == "torch.float32":
        _float32 = dtype
    return dtype is _float32


def _positions(rope: Rope, positions, batch: int, tokens: int, pos_batch: int) -> int:
    """Elements between the positions of two sequences (0: shared), which a raw
    address takes from the caller."""
    if not _is_tensor(positions):
        return pos_batch
    if pos_batch:
        raise ValueError("pos_batch: for positions given by address; a tensor has its own")
    if not positions.is_cuda or not _is_float32(positions.dtype) or not positions.is_contiguous():
        raise ValueError("positions: must be a contiguous float32 CUDA tensor")
    shape = tuple(positions.shape)
    if shape not in ((tokens, rope.axes), (1, tokens, rope.axes), (batch, tokens, rope.axes)):
        raise ValueError(f"positions: must be [{tokens}, {rope.axes}] or [{batch}, {tokens}, {rope.axes}], got {shape}")
    return tokens * rope.axes if len(shape) == 3 and shape[0] > 1 else 0


def rope_heads(rope: Rope, q: Heads, k: Optional[Heads], positions, stream=None, pos_batch: int = 0):
    """Normalise and rotate the heads of q and k (svdq_rope_heads); positions:
    float32 [token, axis], or [batch, token, axis], or an address with pos_batch
    elements between two sequences' (0: shared by all)."""
    q_now, k_now = q._now(), None if k is None else k._now()
    for t, what in ((q, "q"), (k, "k")):
        if t is not None and (t.head_dim != rope.head_dim or t.batch != q.batch or t.tokens != q.tokens):
            raise ValueError(f"{what}: [{t.batch}, {t.tokens}, heads, {t.head_dim}] does not fit the others")
    if (k is not None and k.device != q.device) or (_is_tensor(positions) and positions.get_device() != q.device):
        raise ValueError("q, k and the positions must be on one device")
    pos_batch = _positions(rope, positions, q.batch, q.tokens, pos_batch)
    _check(load().svdq_rope_heads(rope._ref, q_now, k_now, q.batch, q.tokens,
                                  _ptr(positions), pos_batch, _stream(stream)), "svdq_rope_heads")


class Layer:
    """A prepared SVDQuant layer (owns its device buffers)."""

    def __init__(self, handle: int):
        self._h = ctypes.c_void_p(handle)
        info = self.info
        self._K, self._N, self._device = info["K"], info["N"], info["device"]
        self._act_last = (0, 0, 0)
        self._xl_cols = self._xl_width()

    def _xl_width(self) -> int:
        # XL is [M][32] BF16 (zeros past the rank); [M][64] with a LoRA adapter
        return 64 if load().svdq_tensor_bytes(self._h, TENSORS["lora_A"][0]) else 32

    @classmethod
    def prepare(cls, W_bits: np.ndarray, bias_bits: Optional[np.ndarray], calib_bits: Optional[np.ndarray],
                fmt: str = "nvfp4", rank: int = 32, alpha: float = 0.5, device: int = 0,
                flags: int = 0) -> "Layer":
        """W_bits: uint16 [K][N] BF16 bit patterns (Y = X W + b); bias_bits: uint16 [N] or None;
        calib_bits: uint16 [M_calib][K] or None (W4A16); flags: PREP_* bits."""
        L = load()
        W = np.ascontiguousarray(W_bits, dtype=np.uint16)
        if W.ndim != 2:
            raise ValueError(f"W_bits must be [K][N], got shape {W.shape}")
        K, N = W.shape
        b = None if bias_bits is None else np.ascontiguousarray(bias_bits, dtype=np.uint16)
        c = None if calib_bits is None else np.ascontiguousarray(calib_bits, dtype=np.uint16)
        if b is not None and b.size != N:
            raise ValueError(f"bias_bits must hold N = {N} values, got shape {b.shape}")
        if c is not None and (c.ndim != 2 or c.shape[1] != K):
            raise ValueError(f"calib_bits must be [M_calib][K = {K}], got shape {c.shape}")
        cfg = Config(FORMATS[fmt], rank, alpha, flags)
        out = ctypes.c_void_p()
        st = L.svdq_prepare(ctypes.byref(cfg), K, N, _ptr(W), _ptr(b), _ptr(c),
                            0 if c is None else c.shape[0], device, ctypes.byref(out))
        _check(st, "svdq_prepare")
        return cls(out.value)

    def serialize(self) -> bytes:
        """The prepared layer as bytes (svdq_serialize)."""
        n = int(load().svdq_serialized_bytes(self._h))
        buf = np.empty(n, dtype=np.uint8)
        _check(load().svdq_serialize(self._h, _ptr(buf), n), "svdq_serialize")
        return buf.tobytes()

    @classmethod
    def deserialize(cls, data: bytes, device: int = 0) -> "Layer":
        """Rebuild a layer from serialize()'s bytes (svdq_deserialize)."""
        buf = np.frombuffer(data, dtype=np.uint8)
        out = ctypes.c_void_p()
        _check(load().svdq_deserialize(_ptr(buf), buf.size, device, ctypes.byref(out)), "svdq_deserialize")
        return cls(out.value)

    def close(self):
        if self._h is not None and self._h.value:
            load().svdq_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self) -> "Layer":
        return self

    def __exit__(self, *exc):
        self.close()
        return False

    @property
    def info(self) -> dict:
        i = LayerInfo()
        _check(load().svdq_get_info(self._h, ctypes.byref(i)), "svdq_get_info")
        return {f: getattr(i, f) for f, _ in LayerInfo._fields_}

    def export(self, name: str) -> np.ndarray:
        tid, dt = TENSORS[name]
        info = self.info
        K, N, r = info["K"], info["N"], info["rank"]
        if dt is None:
            dt = {NVFP4: np.uint8, W8A8_INT8: np.float32}.get(info["format"], np.uint16)
        nbytes = load().svdq_tensor_bytes(self._h, tid)
        buf = np.empty(nbytes // np.dtype(dt).itemsize, dtype=dt)
        _check(load().svdq_export(self._h, tid, _ptr(buf), nbytes), f"svdq_export({name})")
        w8 = info["format"] == W8A8_INT8
        shapes = {"lambda": (K,), "inv_lambda": (K,), "L1": (K, r), "L2": (r, N), "L1d": (K, r),
                  "L2b": (r, N), "R": (K, N), "sigma": (r,), "w_codes": (N, K if w8 else K // 2), "bias": (N,),
                  "w_scales": (N,) if w8 else (N, -1), "gptq_U": (K, K), "lora_A": (K, -1), "lora_B": (-1, N)}
        return buf.reshape(shapes[name])

    def set_lora(self, A_bits: Optional[np.ndarray], B_bits: Optional[np.ndarray], scale: float = 1.0):
        """Attach a LoRA adapter W -> W + scale A B (A_bits uint16 [K][r], B_bits
        uint16 [r][N], BF16 patterns) to the low-rank branch; None removes it."""
        if A_bits is None:
            try:
                _check(load().svdq_set_lora(self._h, 0, None, None, 0.0), "svdq_set_lora")
            finally:
                self._xl_cols = self._xl_width()
            return
        A = np.ascontiguousarray(A_bits, dtype=np.uint16)
        B = np.ascontiguousarray(B_bits, dtype=np.uint16)
        if A.ndim != 2 or B.ndim != 2 or A.shape[0] != self._K or B.shape != (A.shape[1], self._N):
            raise ValueError(f"A is [K = {self._K}][r] and B is [r][N = {self._N}]; got {A.shape} and {B.shape}")
        r = A.shape[1]
        try:
            _check(load().svdq_set_lora(self._h, r, _ptr(A), _ptr(B), float(scale)), "svdq_set_lora")
        finally:
            self._xl_cols = self._xl_width()

    def workspace_bytes(self, M: int) -> int:
        return int(load().svdq_workspace_bytes(self._h, M))

    def act_scale_bytes(self, M: int) -> int:
        return int(load().svdq_act_scale_bytes(self._h, M))

    def act_code_bytes(self, M: int) -> int:
        return int(load().svdq_act_code_bytes(self._h, M))

    def _act_bytes(self, M: int):
        # (code, scale) bytes for M tokens, which a caller tends to ask for again and again
        last = self._act_last              # one read: another thread may replace it
        if last[0] != M:
            self._act_last = last = (M, self.act_code_bytes(M), self.act_scale_bytes(M))
        return last[1:]

    def act_codes_to_logical(self, device_layout: np.ndarray, M: int) -> np.ndarray:
        """Activation codes in the GEMM's layout -> uint8 [M][K/2] (two codes per
        byte); W8A8: int8 [M][K]."""
        info = self.info
        if info["format"] == W8A8_INT8:
            out = np.empty((M, info["K"]), dtype=np.int8)
        else:
            out = np.empty((M, info["K"] // 2), dtype=np.uint8)
        src = np.ascontiguousarray(device_layout, dtype=np.uint8)
        _need(src, self.act_code_bytes(M), "device_layout", device=False)
        _check(load().svdq_act_codes_to_logical(self._h, _ptr(src), M, _ptr(out)), "svdq_act_codes_to_logical")
        return out

    def _need_act(self, M: int, X=None, Y=None, codes=None, scales=None, xl=None, on: int = -1):
        if M <= 0:
            return                     # the library answers M <= 0 itself
        if X is not None:
            _need(X, M * self._K * 2, "X", True, on)
        if Y is not None:
            _need(Y, M * self._N * 2, "Y", True, on)
        if codes is not None:
            _need(codes, self._act_bytes(M)[0], "codes", True, on)
        if scales is not None:
            _need(scales, self._act_bytes(M)[1], "scales", True, on)
        if xl is not None:
            _need(xl, M * self._xl_cols * 2, "xl", True, on)

    def forward(self, X, M: int, Y, workspace, workspace_bytes: int, stream=None, flags: int = 0):
        self._need_act(M, X=X, Y=Y)
        _need(workspace, workspace_bytes, "workspace")
        _check(load().svdq_linear_forward(self._h, _ptr(X), M, _ptr(Y), _ptr(workspace), workspace_bytes,
                                          _stream(stream), flags), "svdq_linear_forward")

    def forward_static(self, X, M: int, Y, stream=None, flags: int = 0):
        """Forward with the library's built-in device workspace (no caller workspace,
        no allocation); see svdq_linear_forward_static in include/svdq.h."""
        self._need_act(M, X=X, Y=Y)
        _check(load().svdq_linear_forward_static(self._h, _ptr(X), M, _ptr(Y), _stream(stream), flags),
               "svdq_linear_forward_static")

    def quantize_act(self, X, M: int, codes, scales, xl, stream=None, mode: int = 0):
        self._need_act(M, X=X, codes=codes, scales=scales, xl=xl)
        _check(load().svdq_quantize_act(self._h, _ptr(X), M, _ptr(codes), _ptr(scales), _ptr(xl),
                                        _stream(stream), mode), "svdq_quantize_act")

    def gemm(self, codes, scales, xl, M: int, Y, stream=None, flags: int = 0):
        self._need_act(M, Y=Y, codes=codes, scales=scales, xl=xl)
        _check(load().svdq_gemm(self._h, _ptr(codes), _ptr(scales), _ptr(xl), M, _ptr(Y), _stream(stream),
                                flags), "svdq_gemm")

    def norm_quantize_act(self, norm: Norm, X, M: int, codes, scales, xl, stream=None, Y=None):
        """Normalisation and the first kernel in one pass (svdq_norm_quantize_act);
        Y, if given, receives the normalised rows."""
        self._need_act(M, X=X, codes=codes, scales=scales, xl=xl, on=self._device)
        n = norm._args(self._device, M, self._K)
        if M > 0 and Y is not None:
            _need(Y, M * self._K * 2, "Y", True, self._device)
        _check(load().svdq_norm_quantize_act(self._h, n, _ptr(X), M, _ptr(codes), _ptr(scales), _ptr(xl),
                                             _ptr(Y), _stream(stream)), "svdq_norm_quantize_act")

    def norm_forward(self, norm: Norm, X, M: int, Y, workspace, workspace_bytes: int, stream=None, flags: int = 0):
        """Normalisation, then the layer (svdq_norm_linear_forward)."""
        self._need_act(M, X=X, Y=Y, on=self._device)
        n = norm._args(self._device, M, self._K)
        _need(workspace, workspace_bytes, "workspace", True, self._device)
        _check(load().svdq_norm_linear_forward(self._h, n, _ptr(X), M, _ptr(Y), _ptr(workspace),
                                               workspace_bytes, _stream(stream), flags), "svdq_norm_linear_forward")

    def qkv_forward(self, norm: Optional[Norm], X, batch: int, T: int, rope: Rope, q_heads: int, k_heads: int,
                    positions, Y, workspace, workspace_bytes: int, q_weight=None, k_weight=None, stream=None,
                    flags: int = 0, pos_batch: int = 0):
        """[norm ->] layer -> per-head norm and rotation of the first q_heads +
        k_heads heads of each row, in place (svdq_qkv_forward); positions and
        pos_batch as for rope_heads."""
        M = batch * T
        self._need_act(M, X=X, Y=Y, on=self._device)
        n = None if norm is None else norm._args(self._device, M, self._K)
        pos_batch = _positions(rope, positions, batch, T, pos_batch) if batch > 0 and T > 0 else 0
        _need(positions, 0, "positions", True, self._device)
        for w, what in ((q_weight, "q_weight"), (k_weight, "k_weight")):
            if w is not None:
                if _is_tensor(w):
                    _bf16_tensor(w, what)
                _need(w, rope.head_dim * 2, what, True, self._device)
        _need(workspace, workspace_bytes, "workspace", True, self._device)
        _check(load().svdq_qkv_forward(self._h, n, _ptr(X), batch, T, rope._ref,
                                       q_heads, k_heads, _ptr(q_weight), _ptr(k_weight), _ptr(positions), pos_batch,
                                       _ptr(Y), _ptr(workspace), workspace_bytes, _stream(stream), flags),
               "svdq_qkv_forward")

    def gemm_residual(self, codes, scales, xl, M: int, residual: Residual, Y, stream=None, flags: int = 0):
        """The second kernel with a residual in its epilogue (svdq_gemm_residual)."""
        self._need_act(M, Y=Y, codes=codes, scales=scales, xl=xl, on=self._device)
        r = residual._args(self._device, M, self._N)
        _check(load().svdq_gemm_residual(self._h, _ptr(codes), _ptr(scales), _ptr(xl), M, r, _ptr(Y),
                                         _stream(stream), flags), "svdq_gemm_residual")

    def forward_residual(self, X, M: int, residual: Residual, Y, workspace, workspace_bytes: int, stream=None,
                         flags: int = 0):
        """Forward with a residual in the GEMM's epilogue (svdq_linear_forward_residual)."""
        self._need_act(M, X=X, Y=Y, on=self._device)
        r = residual._args(self._device, M, self._N)
        _need(workspace, workspace_bytes, "workspace", True, self._device)
        _check(load().svdq_linear_forward_residual(self._h, _ptr(X), M, r, _ptr(Y), _ptr(workspace),
                                                   workspace_bytes, _stream(stream), flags),
               "svdq_linear_forward_residual")

    def act_scales_to_logical(self, device_layout: np.ndarray, M: int) -> np.ndarray:
        """NVFP4: uint8 [M][K/16] E4M3 bytes; INT4: uint16 [M][K/64] BF16 bits;
        W8A8: float32 [M] (one scale per token)."""
        info = self.info
        if info["format"] == INT4:
            out = np.empty((M, info["K"] // 64), dtype=np.uint16)
        elif info["format"] == W8A8_INT8:
            out = np.empty((M,), dtype=np.float32)
        else:
            out = np.empty((M, info["K"] // 16), dtype=np.uint8)
        src = np.ascontiguousarray(device_layout, dtype=np.uint8)
        _need(src, self.act_scale_bytes(M), "device_layout", device=False)
        _check(load().svdq_act_scales_to_logical(self._h, _ptr(src), M, _ptr(out)), "svdq_act_scales_to_logical")
        return out

    def check(self, stream=None):
        _check(load().svdq_check(self._h, _stream(stream)), "svdq_check")

    def selftest_wait_timeout(self, budget_us: int, stream=None):
        """Enqueue a kernel whose only wait never completes and gives up after
        budget_us; the next check() raises SvdqError with SVDQ_ETIMEOUT."""
        _check(load().svdq_selftest_wait_timeout(self._h, budget_us, _stream(stream)), "svdq_selftest_wait_timeout")


# ---------------------------------------------------------------- fc1 -> fc2 chain

def mlp_workspace_bytes(fc1: Layer, fc2: Layer, M: int, flags: int = 0) -> int:
    """Workspace of mlp_forward / mlp_fc1 for M tokens (svdq_mlp_workspace_bytes)."""
    return int(load().svdq_mlp_workspace_bytes(fc1._h, fc2._h, M, flags))


def mlp_fc1(fc1: Layer, fc2: Layer, X, M: int, codes2, scales2, xl2, workspace, workspace_bytes: int,
            stream=None, flags: int = 0):
    """fc1 with its output handed to fc2 already quantized (svdq_mlp_fc1)."""
    fc1._need_act(M, X=X)
    if M > 0 and xl2 is not None:
        _need(xl2, M * 32 * 2, "xl2")
    fc2._need_act(M, codes=codes2, scales=scales2)
    _need(workspace, workspace_bytes, "workspace")
    _check(load().svdq_mlp_fc1(fc1._h, fc2._h, _ptr(X), M, _ptr(codes2), _ptr(scales2), _ptr(xl2),
                               _ptr(workspace), workspace_bytes, _stream(stream), flags), "svdq_mlp_fc1")


def mlp_forward(fc1: Layer, fc2: Layer, X, M: int, Y, workspace, workspace_bytes: int, stream=None,
                flags: int = 0):
    """fc1 -> [GELU] -> fc2 (svdq_mlp_forward)."""
    fc1._need_act(M, X=X)
    fc2._need_act(M, Y=Y)
    _need(workspace, workspace_bytes, "workspace")
    _check(load().svdq_mlp_forward(fc1._h, fc2._h, _ptr(X), M, _ptr(Y), _ptr(workspace), workspace_bytes,
                                   _stream(stream), flags), "svdq_mlp_forward")


def mlp_block_forward(fc1: Layer, fc2: Layer, norm: Optional[Norm], X, M: int, residual: Optional[Residual], Y,
                      workspace, workspace_bytes: int, stream=None, flags: int = 0):
    """[norm ->] fc1 -> [GELU] -> fc2 [-> residual] (svdq_mlp_block_forward)."""
    fc1._need_act(M, X=X, on=fc1._device)
    fc2._need_act(M, Y=Y, on=fc2._device)
    n = None if norm is None else norm._args(fc1._device, M, fc1._K)
    r = None if residual is None else residual._args(fc2._device, M, fc2._N)
    _need(workspace, workspace_bytes, "workspace", True, fc1._device)
    _check(load().svdq_mlp_block_forward(fc1._h, fc2._h, n, _ptr(X), M, r, _ptr(Y), _ptr(workspace),
                                         workspace_bytes, _stream(stream), flags), "svdq_mlp_block_forward")
