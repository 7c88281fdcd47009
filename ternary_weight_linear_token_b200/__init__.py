"""Thin Python binding of ``libbitnet158.so``, the B200 (sm_100a) C-ABI
library for the BitNet b1.58 BitLinear forward (W1.58A8).

Argument marshalling only: every function below checks the torch tensors it
is given (device, dtype, contiguity, shape), passes their device pointers and
the current CUDA stream to the C entry point of the same name, and raises
``BitnetError`` on a non-OK status.  All arithmetic runs in the library's
CUDA kernels; there is no CPU fallback.  Importing this module fails loudly
if the library has not been built (``python -m
ternary_weight_linear_token_b200.build``).
"""

from __future__ import annotations

import ctypes as C
import functools
import os

import torch

from .build import LIB as LIB_PATH

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m ternary_weight_linear_token_b200.build`"
        " (the BitLinear forward has no CPU fallback)")

lib = C.CDLL(LIB_PATH)

# ---------------------------------------------------------------- constants
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_SHAPE, ERR_MISALIGNED, ERR_CUDA, ERR_TIMEOUT, ERR_RANGE, \
    ERR_WORKSPACE = range(8)
F32, BF16, I8, I32 = 0, 1, 2, 3
EPI_NONE, EPI_RELU2 = 0, 1
FLAG_WEIGHTS_STATIC = 1
FLAG_WEIGHTS_EXPANDED = 2
FLAG_TABLE_LOOKUP = 4
FLAG_PREP_IN_KERNEL = 8
PATH_NONE, PATH_ROWS, PATH_MMA_TOKENS, PATH_MMA_WEIGHTS, PATH_TENSOR_CORE, PATH_GENERIC = range(6)
PATH_NAMES = {PATH_NONE: "none", PATH_ROWS: "rows", PATH_MMA_TOKENS: "mma_tokens",
              PATH_MMA_WEIGHTS: "mma_weights", PATH_TENSOR_CORE: "tensor_core",
              PATH_GENERIC: "generic"}

_DTYPE = {torch.float32: F32, torch.bfloat16: BF16, torch.int8: I8, torch.int32: I32}

_P = C.c_void_p
_I64 = C.c_int64
_SZ = C.c_size_t
_ST = C.c_int

_SIGS = {
    "bitnet_version": ([], C.c_int),
    "bitnet_status_string": ([_ST], C.c_char_p),
    "bitnet_get_device_status": ([_P], _ST),
    "bitnet_quantize_weights_workspace_size": ([_I64, _I64], _SZ),
    "bitnet_quantize_weights": ([_P, _ST, _I64, _I64, _P, _P, _P, _SZ, _P], _ST),
    "bitnet_quantize_act": ([_P, _ST, _I64, _I64, _P, _P, _P], _ST),
    "bitnet_w158a8_matmul_workspace_size": ([_I64, _I64, _I64, _ST], _SZ),
    "bitnet_w158a8_matmul_path": ([_I64, _I64, _I64, _ST], _ST),
    "bitnet_w158a8_matmul_host": ([_P, _ST, _P, _P, _P, _I64, _I64, _I64, _ST, _P, _P, _ST, _P, _SZ,
                                   C.c_uint32, _P], _ST),
    "bitnet_w158a8_matmul": ([_P, _ST, _P, _P, _P, _I64, _I64, _I64, _ST, _P, _ST, _P, _SZ,
                              C.c_uint32, _P], _ST),
    "bitnet_rms_norm": ([_P, _ST, _I64, _I64, _P, _ST, _P], _ST),
    "bitnet_rms_norm_w158a8_matmul": ([_P, _ST, _P, _P, _P, _I64, _I64, _I64, _ST, _P, _ST, _P,
                                       _SZ, C.c_uint32, _P], _ST),
    "bitnet_w158a8_matmul_noalloc": ([_P, _ST, _P, _P, _P, _I64, _I64, _I64, _ST, _P, _ST,
                                      C.c_uint32, _P], _ST),
    "bitnet_host_plan_create": ([_P, _ST, _P, _P, _P, _I64, _I64, _I64, _ST, _P, _P, _ST, _P, _SZ,
                                 C.c_uint32, _P, C.POINTER(_P)], _ST),
    "bitnet_host_plan_run": ([_P], _ST),
    "bitnet_host_plan_destroy": ([_P], None),
}


class ChainStep(C.Structure):
    """``bitnet_chain_step`` of the C header."""
    _fields_ = [("packed", C.c_void_p), ("gamma", C.c_void_p), ("N", C.c_int64),
                ("K", C.c_int64), ("flags", C.c_uint32), ("Y", C.c_void_p),
                ("X_normed", C.c_void_p)]


STEP_RELU2, STEP_NORM_IN = 1, 2
CHAIN_MAX_STEPS = 256
_SIGS["bitnet_decode_chain_workspace_size"] = ([C.POINTER(ChainStep), C.c_int], _SZ)
_SIGS["bitnet_decode_chain"] = ([C.POINTER(ChainStep), C.c_int, _P, _P, _P, _SZ, _P], _ST)


class KVCacheStruct(C.Structure):
    """``bitnet_kv_cache`` of the C header."""
    _fields_ = [("k_codes", C.c_void_p), ("v_codes", C.c_void_p), ("k_scales", C.c_void_p),
                ("v_scales", C.c_void_p), ("num_pages", C.c_int64), ("heads", C.c_int32),
                ("page_tokens", C.c_int32), ("head_dim", C.c_int32)]


LOGPROBS_MAX_TOP = 32
_I32 = C.c_int32
_SIGS["bitnet_kv_append"] = ([_P, _P, _I64, _P, _I64, _ST, _I64, _P, _I64, _P, _P, _I64, _I64, _P], _ST)
_SIGS["bitnet_kv_attention_workspace_size"] = ([_P, _ST, _I64, _I32, _I64, _I64, _I64, _I64], _SZ)
_SIGS["bitnet_kv_attention"] = ([_P, _P, _P, _ST, _I64, _I32, _P, _I64, _P, _P, _I64, _I64, C.c_float, _I64,
                                 _P, _SZ, _P], _ST)
_SIGS["bitnet_quantize_weights_w4"] = ([_P, _ST, _I64, _I64, _I32, _P, _P, _P], _ST)
_SIGS["bitnet_w4a16_matmul"] = ([_P, _ST, _P, _P, _I64, _I64, _I64, _I32, _P, _ST, C.c_uint32, _P], _ST)
_SIGS["bitnet_token_logprobs"] = ([_P, _ST, _I64, _I64, _I64, _P, _I32, _P, _P, _P, _P, _P], _ST)

for _name, (_args, _res) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.argtypes = _args
    _f.restype = _res


class BitnetError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib.bitnet_status_string(status).decode()} (status {status})")


def _check(status: int, what: str):
    if status != OK:
        raise BitnetError(status, what)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _dev(t: torch.Tensor, name: str, dtypes=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the BitLinear path has no CPU fallback)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")


def version() -> int:
    return lib.bitnet_version()


def status_string(status: int) -> str:
    return lib.bitnet_status_string(status).decode()


def bitnet_get_device_status(stream=None) -> int:
    return lib.bitnet_get_device_status(_stream(stream))


# ---------------------------------------------------------------- weights
def bitnet_quantize_weights_workspace_size(N: int, K: int) -> int:
    return lib.bitnet_quantize_weights_workspace_size(N, K)


def bitnet_quantize_weights(W: torch.Tensor, packed: torch.Tensor | None = None,
                            gamma: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None):
    """W [N, K] fp32/bf16 -> (packed [N, K/4] uint8, gamma [1] fp32)."""
    _dev(W, "W", (torch.float32, torch.bfloat16))
    N, K = W.shape
    if packed is None:
        packed = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device)
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=W.device)
    need = bitnet_quantize_weights_workspace_size(N, K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=W.device)
    _dev(packed, "packed", (torch.uint8,))
    _dev(gamma, "gamma", (torch.float32,))
    st = lib.bitnet_quantize_weights(_ptr(W), _DTYPE[W.dtype], N, K, _ptr(packed), _ptr(gamma),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream))
    _check(st, "bitnet_quantize_weights")
    return packed, gamma


# ---------------------------------------------------------------- activations
def bitnet_quantize_act(X: torch.Tensor, xq: torch.Tensor | None = None,
                        s: torch.Tensor | None = None, stream=None):
    """X [M, K] fp32/bf16 -> (xq [M, K] int8, s [M] fp32)."""
    _dev(X, "X", (torch.float32, torch.bfloat16))
    M, K = X.shape
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=X.device)
    if s is None:
        s = torch.empty(M, dtype=torch.float32, device=X.device)
    _dev(xq, "xq", (torch.int8,))
    _dev(s, "s", (torch.float32,))
    st = lib.bitnet_quantize_act(_ptr(X), _DTYPE[X.dtype], M, K, _ptr(xq), _ptr(s),
                                 _stream(stream))
    _check(st, "bitnet_quantize_act")
    return xq, s


# ---------------------------------------------------------------- matmul
@functools.lru_cache(maxsize=256)
def _workspace_size(M: int, N: int, K: int, xd: int) -> int:
    return lib.bitnet_w158a8_matmul_workspace_size(M, N, K, xd)


def bitnet_w158a8_matmul_workspace_size(M: int, N: int, K: int, x_dtype) -> int:
    # a pure function of its arguments: remembered, so that a call per forward costs no
    # second trip through ctypes
    xd = _DTYPE[x_dtype] if isinstance(x_dtype, torch.dtype) else int(x_dtype)
    return _workspace_size(int(M), int(N), int(K), xd)


def bitnet_w158a8_matmul_path(M: int, N: int, K: int, x_dtype) -> int:
    """The kernel path a call of these sizes takes on the current device
    (one of the PATH_* constants)."""
    xd = _DTYPE[x_dtype] if isinstance(x_dtype, torch.dtype) else int(x_dtype)
    return lib.bitnet_w158a8_matmul_path(M, N, K, xd)


def bitnet_w158a8_matmul(X: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor,
                         s: torch.Tensor | None = None, relu2: bool = False,
                         out_dtype: torch.dtype = torch.bfloat16, Y: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, weights_static: bool = False,
                         weights_expanded: bool = False, table_lookup: bool = False,
                         prep_in_kernel: bool = False, stream=None) -> torch.Tensor:
    """Y = BitLinear(X).  X is fp32/bf16 [M, K] (quantised inside the call) or
    int8 xq [M, K] with its scales ``s`` [M].  out_dtype fp32/bf16, or int32
    for the raw accumulators (relu2 must then be False).  ``weights_expanded``
    promises that ``workspace`` still holds the int8 weight copy of an
    earlier tensor-core-path call with the same weights and input kind;
    ``table_lookup`` runs the table-lookup comparison kernel (M <= 8);
    ``prep_in_kernel`` the tensor-core kernel that prepares its own operands."""
    _dev(X, "X", (torch.float32, torch.bfloat16, torch.int8))
    _dev(packed, "packed", (torch.uint8,))
    _dev(gamma, "gamma", (torch.float32,))
    M, K = X.shape
    N = packed.shape[0]
    if packed.shape[1] * 4 != K:
        raise ValueError(f"packed has {packed.shape[1]} bytes per row, expected K/4 = {K // 4}")
    if s is not None:
        _dev(s, "s", (torch.float32,))
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=X.device)
    _dev(Y, "Y", (torch.float32, torch.bfloat16, torch.int32))
    need = 0 if table_lookup else bitnet_w158a8_matmul_workspace_size(M, N, K, X.dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.bitnet_w158a8_matmul(_ptr(X), _DTYPE[X.dtype], _ptr(s), _ptr(packed), _ptr(gamma),
                                  M, N, K, EPI_RELU2 if relu2 else EPI_NONE, _ptr(Y),
                                  _DTYPE[Y.dtype], _ptr(workspace), ws_bytes,
                                  (FLAG_WEIGHTS_STATIC if weights_static else 0)
                                  | (FLAG_WEIGHTS_EXPANDED if weights_expanded else 0)
                                  | (FLAG_TABLE_LOOKUP if table_lookup else 0)
                                  | (FLAG_PREP_IN_KERNEL if prep_in_kernel else 0),
                                  _stream(stream))
    _check(st, "bitnet_w158a8_matmul")
    return Y


def _host_call_args(X_host, packed, gamma, X_dev, Y_dev, Y_host, relu2, workspace,
                    weights_static, stream):
    """Checks the arguments of bitnet_w158a8_matmul_host and returns them as
    the C call takes them (plus the workspace tensor, kept alive by the caller)."""
    if X_host.is_cuda or Y_host.is_cuda:
        raise ValueError("X_host and Y_host must be host (CPU) tensors")
    if not (X_host.is_contiguous() and Y_host.is_contiguous()):
        raise ValueError("X_host and Y_host must be contiguous")
    _dev(X_dev, "X_dev", (X_host.dtype,))
    _dev(Y_dev, "Y_dev", (Y_host.dtype,))
    _dev(packed, "packed", (torch.uint8,))
    _dev(gamma, "gamma", (torch.float32,))
    M, K = X_host.shape
    N = packed.shape[0]
    if X_dev.shape != X_host.shape or Y_dev.shape != Y_host.shape or Y_host.shape != (M, N):
        raise ValueError("X_dev/Y_dev must match the shapes of X_host [M, K] and Y_host [M, N]")
    need = bitnet_w158a8_matmul_workspace_size(M, N, K, X_host.dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=X_dev.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(X_host), _DTYPE[X_host.dtype], _ptr(X_dev), _ptr(packed), _ptr(gamma), M, N, K,
            EPI_RELU2 if relu2 else EPI_NONE, _ptr(Y_dev), _ptr(Y_host), _DTYPE[Y_host.dtype],
            _ptr(workspace), ws_bytes, FLAG_WEIGHTS_STATIC if weights_static else 0, _stream(stream))
    return args, workspace


def bitnet_w158a8_matmul_host(X_host: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor,
                              X_dev: torch.Tensor, Y_dev: torch.Tensor, Y_host: torch.Tensor,
                              relu2: bool = False, workspace: torch.Tensor | None = None,
                              weights_static: bool = False, stream=None) -> torch.Tensor:
    """Y_host = BitLinear(X_host) in one C call: X_host (CPU, fp32/bf16, best
    pinned) is copied to X_dev, the product writes Y_dev, which is copied to
    Y_host (CPU, pinned); returns once Y_host holds the result."""
    args, _ws = _host_call_args(X_host, packed, gamma, X_dev, Y_dev, Y_host, relu2, workspace,
                                weights_static, stream)
    _check(lib.bitnet_w158a8_matmul_host(*args), "bitnet_w158a8_matmul_host")
    return Y_host


class HostMatmulPlan:
    """bitnet_w158a8_matmul_host over fixed buffers, for a projection that
    runs again and again (a decode loop): the arguments are checked once,
    here, and with page-locked X_host and Y_host the copy in, the product and
    the copy out are recorded once as a CUDA graph (bitnet_host_plan_create);
    each call then launches it and waits (bitnet_host_plan_run).  With
    pageable host buffers each call is the one bitnet_w158a8_matmul_host call.
    The caller refills X_host before a call and reads Y_host after it; the
    tensors must stay alive and in place as long as the plan is used."""

    def __init__(self, X_host: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor,
                 X_dev: torch.Tensor, Y_dev: torch.Tensor, Y_host: torch.Tensor,
                 relu2: bool = False, workspace: torch.Tensor | None = None,
                 weights_static: bool = False, stream=None):
        self._plan = None
        self._args, self._ws = _host_call_args(X_host, packed, gamma, X_dev, Y_dev, Y_host, relu2,
                                               workspace, weights_static, stream)
        self._keep = (X_host, packed, gamma, X_dev, Y_dev, Y_host)
        self.Y_host = Y_host
        self.graph = False
        if X_host.is_pinned() and Y_host.is_pinned():
            h = _P()
            st = lib.bitnet_host_plan_create(*self._args, C.byref(h))
            if st == OK:
                self._plan = h
                self.graph = True
            elif st != ERR_CUDA:  # argument errors raise; a graph that could not be
                _check(st, "bitnet_host_plan_create")  # made leaves the per-call path
        self._run = lib.bitnet_host_plan_run
        self._call = lib.bitnet_w158a8_matmul_host

    def __call__(self) -> torch.Tensor:
        st = self._run(self._plan) if self._plan is not None else self._call(*self._args)
        if st != OK:
            raise BitnetError(st, "bitnet_host_plan_run" if self._plan is not None
                              else "bitnet_w158a8_matmul_host")
        return self.Y_host

    def close(self) -> None:
        """Frees the CUDA graph (also done when the plan is collected)."""
        if self._plan is not None:
            lib.bitnet_host_plan_destroy(self._plan)
            self._plan = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def bitnet_rms_norm_w158a8_matmul(X: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor,
                                  X_normed: torch.Tensor | None = None, relu2: bool = False,
                                  out_dtype: torch.dtype = torch.bfloat16,
                                  Y: torch.Tensor | None = None,
                                  workspace: torch.Tensor | None = None,
                                  weights_static: bool = False, stream=None) -> torch.Tensor:
    """Y = BitLinear(rms_norm(X)) for fp32/bf16 X [M, K].  X_normed (same
    dtype and shape as X) receives the normalised input; it may be omitted
    for M <= 8 and is allocated here otherwise."""
    _dev(X, "X", (torch.float32, torch.bfloat16))
    _dev(packed, "packed", (torch.uint8,))
    _dev(gamma, "gamma", (torch.float32,))
    M, K = X.shape
    N = packed.shape[0]
    if packed.shape[1] * 4 != K:
        raise ValueError(f"packed has {packed.shape[1]} bytes per row, expected K/4 = {K // 4}")
    if X_normed is None and M > 8:
        X_normed = torch.empty_like(X)
    if X_normed is not None:
        _dev(X_normed, "X_normed", (X.dtype,))
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=X.device)
    _dev(Y, "Y", (torch.float32, torch.bfloat16, torch.int32))
    need = bitnet_w158a8_matmul_workspace_size(M, N, K, X.dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.bitnet_rms_norm_w158a8_matmul(_ptr(X), _DTYPE[X.dtype], _ptr(X_normed), _ptr(packed),
                                           _ptr(gamma), M, N, K,
                                           EPI_RELU2 if relu2 else EPI_NONE, _ptr(Y),
                                           _DTYPE[Y.dtype], _ptr(workspace), ws_bytes,
                                           FLAG_WEIGHTS_STATIC if weights_static else 0,
                                           _stream(stream))
    _check(st, "bitnet_rms_norm_w158a8_matmul")
    return Y


STATIC_SCRATCH_BYTES = 32 << 20


def bitnet_w158a8_matmul_noalloc(X: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor,
                                 s: torch.Tensor | None = None, relu2: bool = False,
                                 out_dtype: torch.dtype = torch.bfloat16,
                                 Y: torch.Tensor | None = None, weights_static: bool = False,
                                 stream=None) -> torch.Tensor:
    """bitnet_w158a8_matmul with the library's built-in scratch array instead
    of a workspace, for callers that cannot allocate device memory (the output
    Y is still the caller's)."""
    _dev(X, "X", (torch.float32, torch.bfloat16, torch.int8))
    _dev(packed, "packed", (torch.uint8,))
    _dev(gamma, "gamma", (torch.float32,))
    M, K = X.shape
    N = packed.shape[0]
    if packed.shape[1] * 4 != K:
        raise ValueError(f"packed has {packed.shape[1]} bytes per row, expected K/4 = {K // 4}")
    if s is not None:
        _dev(s, "s", (torch.float32,))
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=X.device)
    _dev(Y, "Y", (torch.float32, torch.bfloat16, torch.int32))
    st = lib.bitnet_w158a8_matmul_noalloc(_ptr(X), _DTYPE[X.dtype], _ptr(s), _ptr(packed),
                                          _ptr(gamma), M, N, K, EPI_RELU2 if relu2 else EPI_NONE,
                                          _ptr(Y), _DTYPE[Y.dtype],
                                          FLAG_WEIGHTS_STATIC if weights_static else 0,
                                          _stream(stream))
    _check(st, "bitnet_w158a8_matmul_noalloc")
    return Y


# ---------------------------------------------------------------- glue
def bitnet_rms_norm(X: torch.Tensor, Y: torch.Tensor | None = None,
                    out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """Weightless per-token RMS normalisation (decode-chain glue)."""
    _dev(X, "X", (torch.float32, torch.bfloat16))
    M, K = X.shape
    if Y is None:
        Y = torch.empty((M, K), dtype=out_dtype or X.dtype, device=X.device)
    _dev(Y, "Y", (torch.float32, torch.bfloat16))
    st = lib.bitnet_rms_norm(_ptr(X), _DTYPE[X.dtype], M, K, _ptr(Y), _DTYPE[Y.dtype],
                             _stream(stream))
    _check(st, "bitnet_rms_norm")
    return Y


# ---------------------------------------------------------------- decode chain
def bitnet_decode_chain_steps(steps) -> C.Array:
    """Descriptor array for ``bitnet_decode_chain``: one dict per step with
    ``packed`` [N, K/4] uint8, ``gamma`` [1] fp32, ``Y`` bf16 with N elements
    and optionally ``relu2``, ``norm_in`` and ``X_normed`` (bf16, K elements).
    The tensors must outlive every call that uses the array."""
    arr = (ChainStep * len(steps))()
    for i, d in enumerate(steps):
        packed, gamma, Y = d["packed"], d["gamma"], d["Y"]
        _dev(packed, f"steps[{i}].packed", (torch.uint8,))
        _dev(gamma, f"steps[{i}].gamma", (torch.float32,))
        _dev(Y, f"steps[{i}].Y", (torch.bfloat16,))
        N, K = packed.shape[0], packed.shape[1] * 4
        if Y.numel() != N:
            raise ValueError(f"steps[{i}].Y has {Y.numel()} elements, expected N = {N}")
        xn = d.get("X_normed")
        if xn is not None:
            _dev(xn, f"steps[{i}].X_normed", (torch.bfloat16,))
            if xn.numel() != K:
                raise ValueError(f"steps[{i}].X_normed has {xn.numel()} elements, expected K = {K}")
        flags = (STEP_RELU2 if d.get("relu2") else 0) | (STEP_NORM_IN if d.get("norm_in") else 0)
        arr[i] = ChainStep(packed.data_ptr(), gamma.data_ptr(), N, K, flags, Y.data_ptr(),
                           None if xn is None else xn.data_ptr())
    return arr


def bitnet_decode_chain_workspace_size(steps) -> int:
    arr = steps if isinstance(steps, C.Array) else bitnet_decode_chain_steps(steps)
    return lib.bitnet_decode_chain_workspace_size(arr, len(arr))


def bitnet_decode_chain(steps, x0: torch.Tensor, workspace: torch.Tensor,
                        y_norm: torch.Tensor | None = None, stream=None) -> None:
    """Runs a chain of M = 1 BitLinear projections in one launch.  ``steps``
    is a list of step dicts (see ``bitnet_decode_chain_steps``) or a prebuilt
    descriptor array; x0 is the bf16 input of the first step; ``workspace``
    is a uint8 tensor of ``bitnet_decode_chain_workspace_size`` bytes,
    zero-filled once and then kept for every call of this chain; y_norm
    (optional, bf16) receives the RMS normalisation of the last output."""
    arr = steps if isinstance(steps, C.Array) else bitnet_decode_chain_steps(steps)
    _dev(x0, "x0", (torch.bfloat16,))
    _dev(workspace, "workspace", (torch.uint8,))
    if x0.numel() != arr[0].K:
        raise ValueError(f"x0 has {x0.numel()} elements, expected K = {arr[0].K}")
    if y_norm is not None:
        _dev(y_norm, "y_norm", (torch.bfloat16,))
        if y_norm.numel() != arr[len(arr) - 1].N:
            raise ValueError("y_norm must have the last step's N elements")
    st = lib.bitnet_decode_chain(arr, len(arr), _ptr(x0), _ptr(y_norm), _ptr(workspace),
                                 workspace.numel(), _stream(stream))
    _check(st, "bitnet_decode_chain")


# ---------------------------------------------------------------- decode step: cache, attention, head
# These entry points run on the device of their tensors, whichever is current,
# and allocate on the stream that they run on.  A decode step calls them for
# every token, so each checks its tensors by the cheapest calls there are and
# takes the raw stream of the current device; another device or a given
# stream goes through _elsewhere.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_FLOAT = {torch.float32: F32, torch.bfloat16: BF16}


def _elsewhere(device: int, stream, call, *args, **kwargs):
    """call(*args, **kwargs) with the tensors' device, and `stream`, current."""
    if stream is None:
        with torch.cuda.device(device):
            return call(*args, **kwargs)
    if stream.device.index != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{device}")
    with torch.cuda.stream(stream):
        return call(*args, **kwargs)


def _same_device(device: int, **tensors):
    """Raises the fitting error: `device` (of the first tensor) is no CUDA
    device, or one of the tensors is on another one."""
    if device < 0:
        raise ValueError("tensors must be CUDA tensors (there is no CPU fallback)")
    for name, t in tensors.items():
        if t is not None and t.get_device() != device:
            raise ValueError(f"{name} must be on cuda:{device}, it is on {t.device}")


def _dense(t: torch.Tensor, name: str, *dtypes):
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class KVCache:
    """Key/value cache in 8 bits: ``num_pages`` pages of ``page_tokens``
    tokens (16, 32, 64 or 128), ``heads`` key/value heads of ``head_dim`` (64
    or 128); for each page and head int8 codes [page_tokens, head_dim] of the
    keys and of the values, and a scale of each: value = code * scale.  Which
    pages a sequence uses, in which order, is the caller's page table."""

    def __init__(self, num_pages: int, page_tokens: int, heads: int, head_dim: int, device="cuda:0"):
        shape = (num_pages, heads, page_tokens, head_dim)
        self._take(torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape[:2], dtype=torch.float32, device=device),
                   torch.zeros(shape[:2], dtype=torch.float32, device=device))

    @classmethod
    def from_tensors(cls, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scales: torch.Tensor,
                     v_scales: torch.Tensor) -> "KVCache":
        """A cache over existing tensors (not copied): codes [num_pages, heads,
        page_tokens, head_dim] int8, scales [num_pages, heads] fp32."""
        self = cls.__new__(cls)
        self._take(k_codes, v_codes, k_scales, v_scales)
        return self

    def _take(self, k_codes, v_codes, k_scales, v_scales):
        for t, name in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            _dev(t, name, (torch.int8,))
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _dev(t, name, (torch.float32,))
        if k_codes.dim() != 4 or v_codes.shape != k_codes.shape:
            raise ValueError("k_codes and v_codes must be [num_pages, heads, page_tokens, head_dim]")
        if k_scales.shape != k_codes.shape[:2] or v_scales.shape != k_codes.shape[:2]:
            raise ValueError("k_scales and v_scales must be [num_pages, heads]")
        self.device = k_codes.get_device()
        _same_device(self.device, v_codes=v_codes, k_scales=k_scales, v_scales=v_scales)
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.num_pages, self.heads, self.page_tokens, self.head_dim = k_codes.shape
        self._struct = KVCacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                                     v_scales.data_ptr(), *k_codes.shape)
        self._ref = C.addressof(self._struct)


def _batch(pages, lens, offsets, T, max_new):
    """Checks the arrays that describe a batch; (B, max_pages, max_new)."""
    _dense(pages, "pages", torch.int32)
    _dense(lens, "lens", torch.int32)
    B = lens.numel()
    if pages.dim() != 2 or pages.size(0) != B or lens.dim() != 1:
        raise ValueError("pages must be [B, max_pages] and lens [B]")
    if offsets is None:
        if T != B:
            raise ValueError(f"{T} rows for {B} sequences: without offsets every sequence has one")
        return B, pages.size(1), 1
    _dense(offsets, "offsets", torch.int32)
    if offsets.numel() != B + 1:
        raise ValueError(f"offsets has {offsets.numel()} elements, expected B + 1 = {B + 1}")
    return B, pages.size(1), T if max_new is None else int(max_new)


def bitnet_kv_append(cache: KVCache, K: torch.Tensor, V: torch.Tensor, pages: torch.Tensor,
                     lens: torch.Tensor, offsets: torch.Tensor | None = None,
                     max_new: int | None = None, stream=None) -> None:
    """Quantises the new tokens' keys and values K, V [T, heads, head_dim]
    (fp32/bf16; columns of a wider row are taken as they are) into the cache.
    pages [B, max_pages], lens [B] (the new tokens included) and offsets
    [B + 1] int32 say where: rows offsets[b] .. offsets[b + 1] - 1 are the
    last tokens of sequence b; without offsets each sequence has one row.
    ``max_new``: the most rows of a sequence (default: T; the launch is sized
    and, for attention, the kernel chosen by it: give it for several sequences
    of few rows)."""
    kind = _FLOAT.get(K.dtype)
    if kind is None or V.dtype != K.dtype:
        raise TypeError(f"K and V must both be fp32 or bf16, got {K.dtype} and {V.dtype}")
    H, D = cache.heads, cache.head_dim
    shape = K.shape
    if len(shape) != 3 or shape[1] != H or shape[2] != D or V.shape != shape:
        raise ValueError(f"K and V must be [T, {H}, {D}]")
    T = shape[0]
    ks, vs = K.stride(), V.stride()
    if T > 0 and not (ks[2] == vs[2] == 1 and (H == 1 or ks[1] == vs[1] == D)):
        raise ValueError("the heads of a token must lie one after the other in K and V")
    B, W, most = _batch(pages, lens, offsets, T, max_new)
    d = K.get_device()
    if d < 0 or not (d == cache.device == V.get_device() == pages.get_device() == lens.get_device()):
        _same_device(d, cache=cache.k_codes, V=V, pages=pages, lens=lens)
    if offsets is not None and offsets.get_device() != d:
        _same_device(d, offsets=offsets)
    if stream is not None or d != _current_device():
        return _elsewhere(d, stream, bitnet_kv_append, cache, K, V, pages, lens, offsets, max_new)
    st = lib.bitnet_kv_append(
        cache._ref, K.data_ptr(), ks[0], V.data_ptr(), vs[0], kind, T, pages.data_ptr(), W, lens.data_ptr(),
        None if offsets is None else offsets.data_ptr(), B, most, _raw_stream(d))
    if st:
        _check(st, "bitnet_kv_append")


@functools.lru_cache(maxsize=1024)
def _kv_workspace(num_pages, heads, page_tokens, head_dim, dtype, T, q_heads, B, W, most, window):
    some = KVCacheStruct(256, 256, 256, 256, num_pages, heads, page_tokens, head_dim)
    return lib.bitnet_kv_attention_workspace_size(C.addressof(some), dtype, T, q_heads, B, W, most, window)


def bitnet_kv_attention_workspace_size(cache: KVCache, dtype: torch.dtype, T: int, q_heads: int, B: int,
                                       max_pages: int, max_new: int = 1, window: int = 0) -> int:
    return _kv_workspace(cache.num_pages, cache.heads, cache.page_tokens, cache.head_dim, _FLOAT[dtype],
                         int(T), int(q_heads), int(B), int(max_pages), int(max_new), int(window))


def bitnet_kv_attention(cache: KVCache, Q: torch.Tensor, pages: torch.Tensor, lens: torch.Tensor,
                        offsets: torch.Tensor | None = None, max_new: int | None = None,
                        scale: float | None = None, window: int = 0, O: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of the new tokens' queries Q [T, q_heads, head_dim]
    (fp32/bf16) over the cache, which already holds the new tokens; returns O
    like Q.  pages, lens, offsets and max_new as in ``bitnet_kv_append``;
    ``scale`` defaults to head_dim ** -0.5; ``window`` > 0 lets a token see
    the last ``window`` positions only, its own among them.  Without a
    ``workspace`` (``bitnet_kv_attention_workspace_size`` bytes) one is
    allocated.  Rows of no sequence are left as O has them (a new O: as its
    memory was)."""
    kind = _FLOAT.get(Q.dtype)
    if kind is None:
        raise TypeError(f"Q must be fp32 or bf16, got {Q.dtype}")
    if not Q.is_contiguous():
        raise ValueError("Q must be contiguous")
    D = cache.head_dim
    if Q.dim() != 3 or Q.size(2) != D:
        raise ValueError(f"Q must be [T, q_heads, {D}]")
    T, q_heads = Q.size(0), Q.size(1)
    B, W, most = _batch(pages, lens, offsets, T, max_new)
    d = Q.get_device()
    if d < 0 or not (d == cache.device == pages.get_device() == lens.get_device()):
        _same_device(d, cache=cache.k_codes, pages=pages, lens=lens)
    if offsets is not None and offsets.get_device() != d:
        _same_device(d, offsets=offsets)
    if stream is not None or d != _current_device():
        return _elsewhere(d, stream, bitnet_kv_attention, cache, Q, pages, lens, offsets, max_new, scale,
                          window, O, workspace)
    if O is None:
        O = torch.empty_like(Q)
    else:
        _dense(O, "O", Q.dtype)
        _same_device(d, O=O)
        if O.shape != Q.shape:
            raise ValueError("O must have the shape of Q")
    ws, size = 0, 0
    if workspace is None:
        size = _kv_workspace(cache.num_pages, cache.heads, cache.page_tokens, D, kind, T, q_heads, B, W, most,
                             window)
        if size > 0:
            workspace = torch.empty(size, dtype=torch.uint8, device=Q.device)
            ws = workspace.data_ptr()
    else:
        _same_device(d, workspace=workspace)
        ws, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib.bitnet_kv_attention(
        cache._ref, Q.data_ptr(), O.data_ptr(), kind, T, q_heads, pages.data_ptr(), W, lens.data_ptr(),
        None if offsets is None else offsets.data_ptr(), B, most, D ** -0.5 if scale is None else scale, window,
        ws, size, _raw_stream(d))
    if st:
        _check(st, "bitnet_kv_attention")
    return O


def bitnet_quantize_weights_w4(W: torch.Tensor, group: int = 128, packed: torch.Tensor | None = None,
                               scales: torch.Tensor | None = None, stream=None):
    """W [N, K] fp32/bf16 -> (packed [N, K/2] uint8, scales [N, K/group]
    bf16): 4-bit codes with a scale per group of 32, 64 or 128 weights."""
    _dense(W, "W", torch.float32, torch.bfloat16)
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    N, K = W.shape
    d = W.get_device()
    _same_device(d, packed=packed, scales=scales)
    if stream is not None or d != _current_device():
        return _elsewhere(d, stream, bitnet_quantize_weights_w4, W, group, packed, scales)
    if packed is None:
        packed = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((N, K // group), dtype=torch.bfloat16, device=W.device)
    _dense(packed, "packed", torch.uint8)
    _dense(scales, "scales", torch.bfloat16)
    if packed.shape != (N, K // 2) or scales.shape != (N, K // group):
        raise ValueError("packed must be [N, K/2] and scales [N, K/group]")
    st = lib.bitnet_quantize_weights_w4(W.data_ptr(), _FLOAT[W.dtype], N, K, group, packed.data_ptr(),
                                        scales.data_ptr(), _raw_stream(d))
    _check(st, "bitnet_quantize_weights_w4")
    return packed, scales


def bitnet_w4a16_matmul(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                        out_dtype: torch.dtype = torch.bfloat16, Y: torch.Tensor | None = None,
                        weights_static: bool = False, stream=None) -> torch.Tensor:
    """Y [M, N] = X [M, K] (fp32/bf16) times the transpose of the 4-bit
    weights of ``bitnet_quantize_weights_w4``; Y fp32/bf16.  Made for few
    tokens (a decode step); more run in blocks."""
    kind = _FLOAT.get(X.dtype)
    if kind is None:
        raise TypeError(f"X must be fp32 or bf16, got {X.dtype}")
    if packed.dtype is not torch.uint8 or scales.dtype is not torch.bfloat16:
        raise TypeError(f"packed must be uint8 and scales bf16, got {packed.dtype} and {scales.dtype}")
    if not (X.is_contiguous() and packed.is_contiguous() and scales.is_contiguous()):
        raise ValueError("X, packed and scales must be contiguous")
    if not X.dim() == packed.dim() == scales.dim() == 2:
        raise ValueError("X must be [M, K], packed [N, K/2] and scales [N, K/group]")
    M, K, N, groups = X.size(0), X.size(1), packed.size(0), scales.size(1)
    if packed.size(1) * 2 != K:
        raise ValueError(f"packed has {packed.size(1)} bytes per row, expected K/2 = {K // 2}")
    if groups == 0 or scales.size(0) != N or K % groups != 0:
        raise ValueError("scales must be [N, K/group]")
    d = X.get_device()
    if d < 0 or not (d == packed.get_device() == scales.get_device()):
        _same_device(d, packed=packed, scales=scales)
    if stream is not None or d != _current_device():
        return _elsewhere(d, stream, bitnet_w4a16_matmul, X, packed, scales, out_dtype, Y,
                          weights_static)
    if Y is None:
        Y = X.new_empty((M, N)) if out_dtype is X.dtype else torch.empty((M, N), dtype=out_dtype, device=X.device)
    else:
        _same_device(d, Y=Y)
        if Y.shape != (M, N) or not Y.is_contiguous():
            raise ValueError(f"Y must be [{M}, {N}] and contiguous")
    y_kind = _FLOAT.get(Y.dtype)
    if y_kind is None:
        raise TypeError(f"Y must be fp32 or bf16, got {Y.dtype}")
    st = lib.bitnet_w4a16_matmul(X.data_ptr(), kind, packed.data_ptr(), scales.data_ptr(), M, N, K, K // groups,
                                 Y.data_ptr(), y_kind, FLAG_WEIGHTS_STATIC if weights_static else 0,
                                 _raw_stream(d))
    if st:
        _check(st, "bitnet_w4a16_matmul")
    return Y


def bitnet_token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, stream=None):
    """For each row of logits [M, V] (fp32/bf16; rows may be part of wider
    ones): (logprob [M] of tokens[m], entropy [M], top_ids [M, top] int64,
    top_logprobs [M, top]), all but the ids fp32.  tokens [M] int64; a
    negative one asks for no log probability (0).  ``top`` <= 32 alternatives
    come most probable first, equal ones by the lower id."""
    kind = _FLOAT.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be fp32 or bf16, got {logits.dtype}")
    if tokens.dtype is not torch.int64:
        raise TypeError(f"tokens must be int64, got {tokens.dtype}")
    if logits.dim() != 2:
        raise ValueError("logits must be [M, V]")
    M, V = logits.size(0), logits.size(1)
    if tokens.dim() != 1 or tokens.size(0) != M or not tokens.is_contiguous():
        raise ValueError(f"tokens must be [{M}] and contiguous")
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("the values of a row of logits must be contiguous")
    if top < 0:
        raise ValueError(f"top must not be negative, got {top}")
    d = logits.get_device()
    if d < 0 or tokens.get_device() != d:
        _same_device(d, tokens=tokens)
    if stream is not None or d != _current_device():
        return _elsewhere(d, stream, bitnet_token_logprobs, logits, tokens, top)
    dev = logits.device
    lp = torch.empty(M, dtype=torch.float32, device=dev)
    h = torch.empty_like(lp)
    ids = tokens.new_empty((M, top))
    tl = lp.new_empty((M, top))
    st = lib.bitnet_token_logprobs(logits.data_ptr(), kind, M, V, logits.stride(0), tokens.data_ptr(), top,
                                   lp.data_ptr(), h.data_ptr(), ids.data_ptr() if top else None,
                                   tl.data_ptr() if top else None, _raw_stream(d))
    if st:
        _check(st, "bitnet_token_logprobs")
    return lp, h, ids, tl
