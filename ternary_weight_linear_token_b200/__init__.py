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
_SIGS["bitnet_w4a16_matmul_workspace_size"] = ([_I64, _I64, _I64, _ST], _SZ)
_SIGS["bitnet_w4a16_matmul"] = ([_P, _ST, _P, _P, _I64, _I64, _I64, _I32, _P, _ST, _P, _SZ, C.c_uint32, _P],
                                _ST)
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
# and take `stream` (default: that device's current stream) for the tensors
# that they allocate as well.
def _on(stream, *tensors):
    """Checks that the tensors share a CUDA device; (context to run in or
    None, raw stream) for a call on them."""
    dev = tensors[0].device
    for t in tensors:
        if t.device != dev:
            if not t.is_cuda:
                raise ValueError("tensors must be CUDA tensors (there is no CPU fallback)")
            raise ValueError(f"tensors are on {dev} and on {t.device}")
    if not tensors[0].is_cuda:
        raise ValueError("tensors must be CUDA tensors (there is no CPU fallback)")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev.index)
        return (None if dev.index == torch._C._cuda_getDevice() else torch.cuda.device(dev)), raw
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream), stream.cuda_stream


def _within(context, call):
    if context is None:
        return call()
    with context:
        return call()


def _is(t: torch.Tensor, name: str, *dtypes):
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")


def _dense(t: torch.Tensor, name: str, *dtypes):
    _is(t, name, *dtypes)
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
        if len({t.device for t in (k_codes, v_codes, k_scales, v_scales)}) != 1:
            raise ValueError("a cache lies on one device")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.num_pages, self.heads, self.page_tokens, self.head_dim = k_codes.shape
        self._struct = KVCacheStruct(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                                     v_scales.data_ptr(), *(k_codes.shape[i] for i in (0, 1, 2, 3)))
        self._ref = C.addressof(self._struct)


def _batch(pages, lens, offsets, T, max_new):
    """Checks the arrays that describe a batch; (B, max_pages, max_new)."""
    _dense(pages, "pages", torch.int32)
    _dense(lens, "lens", torch.int32)
    B = lens.numel()
    if pages.dim() != 2 or pages.shape[0] != B or lens.dim() != 1:
        raise ValueError("pages must be [B, max_pages] and lens [B]")
    if offsets is None:
        if T != B:
            raise ValueError(f"{T} rows for {B} sequences: without offsets every sequence has one")
        return B, pages.shape[1], 1
    _dense(offsets, "offsets", torch.int32)
    if offsets.numel() != B + 1:
        raise ValueError(f"offsets has {offsets.numel()} elements, expected B + 1 = {B + 1}")
    return B, pages.shape[1], T if max_new is None else int(max_new)


def bitnet_kv_append(cache: KVCache, K: torch.Tensor, V: torch.Tensor, pages: torch.Tensor,
                     lens: torch.Tensor, offsets: torch.Tensor | None = None,
                     max_new: int | None = None, stream=None) -> None:
    """Quantises the new tokens' keys and values K, V [T, heads, head_dim]
    (fp32/bf16; columns of a wider row are taken as they are) into the cache.
    pages [B, max_pages], lens [B] (the new tokens included) and offsets
    [B + 1] int32 say where: rows offsets[b] .. offsets[b + 1] - 1 are the
    last tokens of sequence b; without offsets each sequence has one row.
    ``max_new``: the most rows of a sequence (default: T)."""
    T = K.shape[0]
    _is(K, "K", torch.float32, torch.bfloat16)
    _is(V, "V", K.dtype)
    H, D = cache.heads, cache.head_dim
    if K.shape != (T, H, D) or V.shape != (T, H, D):
        raise ValueError(f"K and V must be [T, {H}, {D}]")
    ks, vs = K.stride(), V.stride()
    if T > 0 and not (ks[2] == vs[2] == 1 and (H == 1 or ks[1] == vs[1] == D)):
        raise ValueError("the heads of a token must lie one after the other in K and V")
    B, W, most = _batch(pages, lens, offsets, T, max_new)
    ctx, raw = _on(stream, cache.k_codes, K, V, pages, lens, *(() if offsets is None else (offsets,)))
    st = _within(ctx, lambda: lib.bitnet_kv_append(
        cache._ref, K.data_ptr(), ks[0], V.data_ptr(), vs[0], _DTYPE[K.dtype], T, pages.data_ptr(), W,
        lens.data_ptr(), None if offsets is None else offsets.data_ptr(), B, most, raw))
    _check(st, "bitnet_kv_append")


@functools.lru_cache(maxsize=1024)
def _kv_workspace(num_pages, heads, page_tokens, head_dim, dtype, T, q_heads, B, W, most, window):
    some = KVCacheStruct(256, 256, 256, 256, num_pages, heads, page_tokens, head_dim)
    return lib.bitnet_kv_attention_workspace_size(C.addressof(some), dtype, T, q_heads, B, W, most, window)


def bitnet_kv_attention_workspace_size(cache: KVCache, dtype: torch.dtype, T: int, q_heads: int, B: int,
                                       max_pages: int, max_new: int = 1, window: int = 0) -> int:
    return _kv_workspace(cache.num_pages, cache.heads, cache.page_tokens, cache.head_dim, _DTYPE[dtype],
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
    _dense(Q, "Q", torch.float32, torch.bfloat16)
    if Q.dim() != 3 or Q.shape[2] != cache.head_dim:
        raise ValueError(f"Q must be [T, q_heads, {cache.head_dim}]")
    T, q_heads, D = Q.shape
    B, W, most = _batch(pages, lens, offsets, T, max_new)
    ctx, raw = _on(stream, cache.k_codes, Q, pages, lens, *(() if offsets is None else (offsets,)),
                   *(() if O is None else (O,)), *(() if workspace is None else (workspace,)))
    if O is not None:
        _dense(O, "O", Q.dtype)
        if O.shape != Q.shape:
            raise ValueError("O must have the shape of Q")
    need = _kv_workspace(cache.num_pages, cache.heads, cache.page_tokens, D, _DTYPE[Q.dtype], T, q_heads, B,
                         W, most, int(window))

    def call():
        out, ws = O, workspace
        if out is None:
            out = torch.empty_like(Q)
        if ws is None and need > 0:
            ws = torch.empty(need, dtype=torch.uint8, device=Q.device)
        return lib.bitnet_kv_attention(
            cache._ref, Q.data_ptr(), out.data_ptr(), _DTYPE[Q.dtype], T, q_heads, pages.data_ptr(), W,
            lens.data_ptr(), None if offsets is None else offsets.data_ptr(), B, most,
            D ** -0.5 if scale is None else scale, window, None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel() * ws.element_size(), raw), out
    st, out = _within(ctx, call)
    _check(st, "bitnet_kv_attention")
    return out


def bitnet_quantize_weights_w4(W: torch.Tensor, group: int = 128, packed: torch.Tensor | None = None,
                               scales: torch.Tensor | None = None, stream=None):
    """W [N, K] fp32/bf16 -> (packed [N, K/2] uint8, scales [N, K/group]
    bf16): 4-bit codes with a scale per group of 32, 64 or 128 weights."""
    _dense(W, "W", torch.float32, torch.bfloat16)
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    N, K = W.shape
    ctx, raw = _on(stream, W, *(t for t in (packed, scales) if t is not None))

    def call():
        p = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device) if packed is None else packed
        s = torch.empty((N, K // group), dtype=torch.bfloat16, device=W.device) if scales is None else scales
        _dense(p, "packed", torch.uint8)
        _dense(s, "scales", torch.bfloat16)
        if p.shape != (N, K // 2) or s.shape != (N, K // group):
            raise ValueError("packed must be [N, K/2] and scales [N, K/group]")
        return lib.bitnet_quantize_weights_w4(W.data_ptr(), _DTYPE[W.dtype], N, K, group, p.data_ptr(),
                                              s.data_ptr(), raw), p, s
    st, p, s = _within(ctx, call)
    _check(st, "bitnet_quantize_weights_w4")
    return p, s


def bitnet_w4a16_matmul_workspace_size(M: int, N: int, K: int, x_dtype: torch.dtype) -> int:
    return lib.bitnet_w4a16_matmul_workspace_size(M, N, K, _DTYPE[x_dtype])


def bitnet_w4a16_matmul(X: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                        out_dtype: torch.dtype = torch.bfloat16, Y: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, weights_static: bool = False,
                        stream=None) -> torch.Tensor:
    """Y [M, N] = X [M, K] (fp32/bf16) times the transpose of the 4-bit
    weights of ``bitnet_quantize_weights_w4``; Y fp32/bf16.  Made for few
    tokens (a decode step); more run in blocks."""
    _dense(X, "X", torch.float32, torch.bfloat16)
    _dense(packed, "packed", torch.uint8)
    _dense(scales, "scales", torch.bfloat16)
    M, K = X.shape
    N = packed.shape[0]
    if packed.shape[1] * 2 != K:
        raise ValueError(f"packed has {packed.shape[1]} bytes per row, expected K/2 = {K // 2}")
    groups = scales.shape[1] if scales.dim() == 2 else 0
    if groups == 0 or scales.shape[0] != N or K % groups != 0:
        raise ValueError("scales must be [N, K/group]")
    ctx, raw = _on(stream, X, packed, scales, *(t for t in (Y, workspace) if t is not None))
    if Y is not None:
        _dense(Y, "Y", torch.float32, torch.bfloat16)
        if Y.shape != (M, N):
            raise ValueError(f"Y must be [{M}, {N}]")

    def call():
        out, ws = Y, workspace
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=X.device)
            _is(out, "out_dtype", torch.float32, torch.bfloat16)
        if ws is None:
            need = lib.bitnet_w4a16_matmul_workspace_size(M, N, K, _DTYPE[X.dtype])
            if need > 0:
                ws = torch.empty(need, dtype=torch.uint8, device=X.device)
        return lib.bitnet_w4a16_matmul(
            X.data_ptr(), _DTYPE[X.dtype], packed.data_ptr(), scales.data_ptr(), M, N, K, K // groups,
            out.data_ptr(), _DTYPE[out.dtype], None if ws is None else ws.data_ptr(),
            0 if ws is None else ws.numel() * ws.element_size(),
            FLAG_WEIGHTS_STATIC if weights_static else 0, raw), out
    st, out = _within(ctx, call)
    _check(st, "bitnet_w4a16_matmul")
    return out


def bitnet_token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, stream=None):
    """For each row of logits [M, V] (fp32/bf16; rows may be part of wider
    ones): (logprob [M] of tokens[m], entropy [M], top_ids [M, top] int64,
    top_logprobs [M, top]), all but the ids fp32.  tokens [M] int64; a
    negative one asks for no log probability (0).  ``top`` <= 32 alternatives
    come most probable first, equal ones by the lower id."""
    _is(logits, "logits", torch.float32, torch.bfloat16)
    _dense(tokens, "tokens", torch.int64)
    M, V = logits.shape
    if tokens.shape != (M,):
        raise ValueError(f"tokens must be [{M}]")
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("the values of a row of logits must be contiguous")
    ctx, raw = _on(stream, logits, tokens)

    def call():
        dev = logits.device
        lp = torch.empty((2, M), dtype=torch.float32, device=dev)
        ids = torch.empty((M, max(top, 0)), dtype=torch.int64, device=dev)
        tl = torch.empty((M, max(top, 0)), dtype=torch.float32, device=dev)
        at = lp.data_ptr()
        return lib.bitnet_token_logprobs(
            logits.data_ptr(), _DTYPE[logits.dtype], M, V, logits.stride(0), tokens.data_ptr(), top, at,
            at + 4 * M, ids.data_ptr() if top > 0 else None, tl.data_ptr() if top > 0 else None,
            raw), (lp[0], lp[1], ids, tl)
    st, out = _within(ctx, call)
    _check(st, "bitnet_token_logprobs")
    return out
