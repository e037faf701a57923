"""Thin Python binding of libqmoe (C ABI in include/moe.h).

Argument marshalling only: every step of the layer runs in the HIP library.
Tensors are torch tensors on the GPU; PyTorch supplies device memory and the
current stream.  If the library is not built this module raises on load --
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqmoe.so")

MOE_ABI_VERSION = 3
MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_F32, MOE_BF16 = 0, 1
MOE_FMT_NONE, MOE_FMT_IQ2XXS_L, MOE_FMT_Q2K_L, MOE_FMT_Q8_0_L, MOE_FMT_Q4K_L = 0, 1, 2, 3, 4
MOE_FMT_MXFP4_L, MOE_FMT_VQ12_L, MOE_FMT_VQ13_L = 5, 6, 7
MOE_LAYOUT_CANONICAL, MOE_LAYOUT_DEVICE = 0, 1
MOE_OP_ROUTE, MOE_OP_DECODE, MOE_OP_PREFILL, MOE_OP_LAYER = 0, 1, 2, 3
MOE_PATH_AUTO, MOE_PATH_DECODE, MOE_PATH_PREFILL = 0, 1, 2
MOE_DECODE_MAX_T = 8
MOE_AUTO_DECODE_MAX_T = 24
MOE_REPACK_TO_DEVICE, MOE_REPACK_TO_CANONICAL = 0, 1
MOE_NOALLOC_SCRATCH_BYTES = 8 << 20
MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2_SUM = 0, 1


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


_STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED", -3: "MOE_ERR_WORKSPACE",
           -4: "MOE_ERR_HIP"}


class MoeLayer(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("n_experts", ctypes.c_int32),
        ("d_model", ctypes.c_int32),
        ("d_ff", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("fmt_gate_up", ctypes.c_int32),
        ("fmt_down", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("w_gate", ctypes.c_void_p),
        ("w_up", ctypes.c_void_p),
        ("w_down", ctypes.c_void_p),
        ("iq2_grid", ctypes.c_void_p),
        ("w_router", ctypes.c_void_p),
        ("has_shared", ctypes.c_int32),
        ("fmt_shared", ctypes.c_int32),
        ("s_gate", ctypes.c_void_p),
        ("s_up", ctypes.c_void_p),
        ("s_down", ctypes.c_void_p),
        ("router_bias", ctypes.c_void_p),
        ("down_gain", ctypes.c_void_p),
        ("vq_codebook", ctypes.c_void_p),
        ("vq_codes", ctypes.c_int32),
    ]


class MoeGate(ctypes.Structure):
    _fields_ = [
        ("abi_version", ctypes.c_uint32),
        ("n_experts", ctypes.c_int32),
        ("top_k", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("n_groups", ctypes.c_int32),
        ("top_groups", ctypes.c_int32),
        ("group_score", ctypes.c_int32),
        ("renormalize", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("bias", ctypes.c_void_p),
    ]


_lib = None
_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "moe_abi_version": ([], ctypes.c_int),
            "moe_last_error": ([], ctypes.c_char_p),
            "moe_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "moe_matrix_bytes": ([_I32, _I32, _I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
            "moe_workspace_bytes": ([ctypes.POINTER(MoeLayer), _I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
            "moe_repack": ([_I32, _I32, _I32, _I32, _P, _P, _I32, _P], ctypes.c_int),
            "moe_route_topk": ([_P, _P, _I32, _I32, _P, _I32, _I32, _I32, _P, _P, _P, _SZ, _P], ctypes.c_int),
            "moe_bucket": ([_P, _I32, _I32, _I32, _P, _P, _P, _P, _P], ctypes.c_int),
            "moe_expert_ffn_decode": ([ctypes.POINTER(MoeLayer), _P, _I32, _I32, _P, _P, _P, _P, _SZ, _P],
                                      ctypes.c_int),
            "moe_expert_ffn_prefill": ([ctypes.POINTER(MoeLayer), _P, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P],
                                       ctypes.c_int),
            "moe_layer_forward": ([ctypes.POINTER(MoeLayer), _P, _I32, _I32, _P, _P, _P, _I32, _P, _SZ, _P],
                                  ctypes.c_int),
            "moe_layer_forward_noalloc": ([ctypes.POINTER(MoeLayer), _P, _I32, _I32, _P, _P, _P, _I32, _P],
                                          ctypes.c_int),
            "moe_prepare_weights": ([ctypes.POINTER(MoeLayer), ctypes.POINTER(MoeLayer), _P], ctypes.c_int),
            "moe_router_logits": ([_P, _I32, _I32, _P, _I32, _I32, _P, _P], ctypes.c_int),
            "moe_gate_topk": ([ctypes.POINTER(MoeGate), _P, _I32, _I64, _I32, _P, _P, _P], ctypes.c_int),
            "moe_blockscale_quantize": ([_P, _I32, _I64, _I32, _I32, _P, _I64, _P, _P], ctypes.c_int),
            "moe_blockscale_matmul_workspace_bytes": ([_I32, _I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
            "moe_blockscale_matmul": ([_P, _I64, _P, _I32, _P, _P, _I32, _I32, _P, _I32, _I64, _P, _SZ, _P],
                                      ctypes.c_int),
            "moe_blockscale_gateup": ([_P, _P, _I32, _I32, _P, _P, _I32, _P, _P, _P, _P, _I32, _I32, _P, _P, _P],
                                      ctypes.c_int),
            "moe_blockscale_down_workspace_bytes": ([_I32, _I32, _I32, ctypes.POINTER(_SZ)], ctypes.c_int),
            "moe_blockscale_down": ([_P, _P, _I32, _I32, _P, _P, _P, _I32, _P, _P, _I32, _I32, _P, _P, _P, _SZ, _P],
                                    ctypes.c_int),
            "moe_profile_enable": ([_I32], ctypes.c_int),
            "moe_profile_reset": ([], ctypes.c_int),
            "moe_profile_collect": ([_I32, _P, _P, _P, _P], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _lib = L
    return _lib


def last_error() -> str:
    return lib().moe_last_error().decode()


def _check(rc: int) -> None:
    if rc != MOE_OK:
        raise MoeError(rc, last_error())


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream=None) -> int:
    if stream is None:
        # the raw handle: torch.cuda.current_stream() builds a Stream object,
        # 2.6 us on the host of a call that takes 4
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def x_dtype_of(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return MOE_F32
    if x.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"activations must be float32 or bfloat16, not {x.dtype}")


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI, minus the moe_ prefix)
# ---------------------------------------------------------------------------
def abi_version() -> int:
    return lib().moe_abi_version()


def matrix_bytes(fmt: int, n_experts: int, rows: int, K: int) -> int:
    out = _SZ()
    _check(lib().moe_matrix_bytes(fmt, n_experts, rows, K, ctypes.byref(out)))
    return out.value


def workspace_bytes(layer: MoeLayer, T: int, op: int) -> int:
    out = _SZ()
    _check(lib().moe_workspace_bytes(ctypes.byref(layer), T, op, ctypes.byref(out)))
    return out.value


def repack(fmt, n_experts, rows, K, src: torch.Tensor, dst: torch.Tensor, direction=MOE_REPACK_TO_DEVICE,
           stream=None) -> None:
    _check(lib().moe_repack(fmt, n_experts, rows, K, _ptr(src), _ptr(dst), direction, _stream(stream)))


def prepare_weights(canonical: MoeLayer, device_out: MoeLayer, stream=None) -> None:
    """Whole-layer canonical -> device conversion into device_out's weight
    buffers; device_out then describes the prepared layer."""
    _check(lib().moe_prepare_weights(ctypes.byref(canonical), ctypes.byref(device_out), _stream(stream)))


def route_topk(w_router, x, k, idx, wt, ws, stream=None, bias=None) -> None:
    E, d = w_router.shape
    _check(lib().moe_route_topk(_ptr(w_router), _ptr(bias), E, d, _ptr(x), x_dtype_of(x), x.shape[0], k, _ptr(idx),
                                _ptr(wt), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def bucket(idx, E, counts, offsets, perm, pos, stream=None) -> None:
    T, k = idx.shape
    for t, n, name in ((counts, E, "counts"), (offsets, E + 1, "offsets"), (perm, T * k, "perm"), (pos, T * k, "pos")):
        if t.numel() < n:
            raise ValueError(f"bucket: {name} holds {t.numel()} entries, needs {n}")
    _check(lib().moe_bucket(_ptr(idx), T, k, E, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(pos),
                            _stream(stream)))


def expert_ffn_decode(layer: MoeLayer, x, idx, wt, y, ws, stream=None) -> None:
    _check(lib().moe_expert_ffn_decode(ctypes.byref(layer), _ptr(x), x_dtype_of(x), x.shape[0], _ptr(idx), _ptr(wt),
                                       _ptr(y), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def expert_ffn_prefill(layer: MoeLayer, x, idx, wt, y, ws, bucket_out=None, stream=None) -> None:
    _check(lib().moe_expert_ffn_prefill(ctypes.byref(layer), _ptr(x), x_dtype_of(x), x.shape[0], _ptr(idx),
                                        _ptr(wt), _ptr(y), _ptr(bucket_out), _ptr(ws),
                                        ws.numel() * ws.element_size(), _stream(stream)))


def layer_forward(layer: MoeLayer, x, y, ws, idx_out=None, wt_out=None, path=MOE_PATH_AUTO, stream=None) -> None:
    _check(lib().moe_layer_forward(ctypes.byref(layer), _ptr(x), x_dtype_of(x), x.shape[0], _ptr(y), _ptr(idx_out),
                                   _ptr(wt_out), path, _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def layer_forward_noalloc(layer: MoeLayer, x, y, idx_out=None, wt_out=None, path=MOE_PATH_AUTO,
                          stream=None) -> None:
    """moe_layer_forward on the library's fixed per-device scratch array
    (MOE_NOALLOC_SCRATCH_BYTES; no workspace argument, nothing allocated)."""
    _check(lib().moe_layer_forward_noalloc(ctypes.byref(layer), _ptr(x), x_dtype_of(x), x.shape[0], _ptr(y),
                                           _ptr(idx_out), _ptr(wt_out), path, _stream(stream)))


# ---------------------------------------------------------------------------
# gate and block-scaled E4M3 operators
# ---------------------------------------------------------------------------
_SCORES = {"sigmoid": MOE_SCORE_SIGMOID, "softmax": MOE_SCORE_SOFTMAX}
_GROUP_SCORES = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2_SUM}


_calls = None


def _load_calls():
    """The compiled calls (csrc/calls.cpp): they check their tensors and give
    the status, or None if a tensor is not as the call needs it; the functions
    below then say which."""
    global _calls
    lib()
    if not os.path.exists(os.path.join(_HERE, "_calls.so")):
        raise RuntimeError(f"{_HERE}/_calls.so is not built; run __graft_entry__.build() first")
    from . import _calls as module
    _calls = module
    return module


def _not_here(fn: str, *tensors, workspace=None) -> None:
    """Raises for tensors whose shapes and dtypes are right, but not the place."""
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError(f"{fn}: the workspace must be contiguous")
    if not all(t.is_cuda for t in (*tensors, workspace) if t is not None):
        raise ValueError(f"{fn}: every tensor must be in GPU memory")
    raise ValueError(f"{fn}: every tensor and the stream must be of the current device, cuda:{torch.cuda.current_device()}")


def _check_here(fn: str, stream, *tensors) -> None:
    if not all(t.is_cuda for t in tensors):
        _not_here(fn, *tensors)
    here = torch.cuda.current_device()
    if any(t.get_device() != here for t in tensors) or getattr(stream, "device_index", here) != here:
        _not_here(fn, *tensors)


def _need(fn: str, **tensors) -> None:
    """Raises for the first (tensor, dtype, shape) whose storage is not as the C
    call takes it: the dtype (codes, uint8, may be float8_e4m3fn), the size, no gaps."""
    for name, (t, dtype, shape) in tensors.items():
        if t.dtype != dtype and not (dtype == torch.uint8 and t.dtype == torch.float8_e4m3fn):
            raise TypeError(f"{fn}: {name} must be {dtype}, not {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, needs {tuple(shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous")


def _rows_of(fn: str, name: str, t: torch.Tensor, dtypes) -> int:
    """Row stride (elements) of a 2-D tensor whose rows have no gaps."""
    if t.dtype not in dtypes:
        raise TypeError(f"{fn}: {name} must be one of {tuple(dtypes)}, not {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{fn}: {name} must be 2-D with contiguous rows")
    (rows, cols), (ld, step) = t.shape, t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{fn}: {name} must be 2-D with contiguous rows")
    return ld if rows > 1 else cols  # (a single row's stride is free; torch leaves any number there)


def scale_blocks(n: int) -> int:
    """Scales along n inputs or outputs: one per 128, the last block may be short."""
    return (n + 127) // 128


_F8 = (torch.float8_e4m3fn, torch.uint8)
_XDT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def gate(n_experts: int, top_k: int, score="sigmoid", n_groups=1, top_groups=1, group_score="max", renormalize=True,
         scale=1.0, bias=None) -> MoeGate:
    """A gate's description for gate_topk (it keeps the bias tensor alive)."""
    if bias is not None:
        _need("gate", bias=(bias, torch.float32, (n_experts,)))
        if not bias.is_cuda:
            _not_here("gate", bias)
    g = MoeGate(abi_version=MOE_ABI_VERSION, n_experts=n_experts, top_k=top_k, score=_SCORES[score],
                n_groups=n_groups, top_groups=top_groups, group_score=_GROUP_SCORES[group_score],
                renormalize=1 if renormalize else 0, scale=scale, bias=_ptr(bias))
    g.bias_tensor = bias
    return g


def router_logits(w_router, x, z, stream=None) -> None:
    E, d = w_router.shape
    T = x.shape[0]
    _need("router_logits", w_router=(w_router, torch.float32, (E, d)), x=(x, x.dtype, (T, d)),
          z=(z, torch.float32, (T, E)))
    _check_here("router_logits", stream, w_router, x, z)
    _check(lib().moe_router_logits(_ptr(w_router), E, d, _ptr(x), x_dtype_of(x), T, _ptr(z), _stream(stream)))


def gate_topk(gate: MoeGate, z, idx, wt, stream=None) -> None:
    rc = (_calls or _load_calls()).gate_topk(gate, z, idx, wt, stream)
    if rc is None:
        T, E = z.shape
        _rows_of("gate_topk", "z", z, _XDT)
        if E != gate.n_experts:
            raise ValueError(f"gate_topk: z has {E} logits per row, the gate {gate.n_experts} experts")
        _need("gate_topk", idx=(idx, torch.int32, (T, gate.top_k)), wt=(wt, torch.float32, (T, gate.top_k)))
        _not_here("gate_topk", z, idx, wt)
    if rc:
        _check(rc)


def blockscale_quantize(x, q, s, stream=None) -> None:
    """x [M][K] to q (float8_e4m3fn or uint8) [M][K] and s [M][ceil(K / 128)]."""
    rc = (_calls or _load_calls()).quantize(x, q, s, stream)
    if rc is None:
        fn = "blockscale_quantize"
        _rows_of(fn, "x", x, _XDT), _rows_of(fn, "q", q, _F8)
        M, K = x.shape
        if q.shape != x.shape:
            raise ValueError(f"{fn}: q has shape {tuple(q.shape)}, needs {tuple(x.shape)}")
        _need(fn, s=(s, torch.float32, (M, scale_blocks(K))))
        _not_here(fn, x, q, s)
    if rc:
        _check(rc)


def blockscale_matmul_workspace_bytes(M: int, N: int, K: int) -> int:
    out = _SZ()
    _check(lib().moe_blockscale_matmul_workspace_bytes(M, N, K, ctypes.byref(out)))
    return out.value


def blockscale_matmul(xq, xs, wq, ws, y, workspace=None, stream=None) -> None:
    """y [M][N] (float32 or bfloat16) = xq [M][K] times wq [N][K] transposed,
    with scales xs [M][ceil(K / 128)] and ws [ceil(N / 128)][ceil(K / 128)]."""
    rc = (_calls or _load_calls()).matmul(xq, xs, wq, ws, y, workspace, stream)
    if rc is None:
        fn = "blockscale_matmul"
        _rows_of(fn, "xq", xq, _F8), _rows_of(fn, "y", y, _XDT)
        (M, K), N = xq.shape, wq.shape[0]
        KB, NB = scale_blocks(K), scale_blocks(N)
        if y.shape != (M, N):
            raise ValueError(f"{fn}: y has shape {tuple(y.shape)}, needs {(M, N)}")
        _need(fn, xs=(xs, torch.float32, (M, KB)), wq=(wq, torch.uint8, (N, K)), ws=(ws, torch.float32, (NB, KB)))
        _not_here(fn, xq, xs, wq, ws, y, workspace=workspace)
    if rc:
        _check(rc)


def blockscale_gateup(xq, xs, k, offsets, perm, w_gate, s_gate, w_up, s_up, hq, hs, stream=None) -> None:
    """hq [T*k][f], hs [T*k][ceil(f / 128)]: the bucket rows' silu(gate) * up,
    requantised; offsets and perm as bucket() writes them."""
    rc = (_calls or _load_calls()).gateup(xq, xs, k, offsets, perm, w_gate, s_gate, w_up, s_up, hq, hs, stream)
    if rc is None:
        fn = "blockscale_gateup"
        (T, d), (E, f, _) = xq.shape, w_gate.shape
        R, DB, FB = T * k, scale_blocks(d), scale_blocks(f)
        _need(fn, xq=(xq, torch.uint8, (T, d)), xs=(xs, torch.float32, (T, DB)),
              offsets=(offsets, torch.int32, (E + 1,)), perm=(perm, torch.int32, (R,)),
              w_gate=(w_gate, torch.uint8, (E, f, d)), s_gate=(s_gate, torch.float32, (E, FB, DB)),
              w_up=(w_up, torch.uint8, (E, f, d)), s_up=(s_up, torch.float32, (E, FB, DB)),
              hq=(hq, torch.uint8, (R, f)), hs=(hs, torch.float32, (R, FB)))
        _not_here(fn, xq, xs, offsets, perm, w_gate, s_gate, w_up, s_up, hq, hs)
    if rc:
        _check(rc)


def blockscale_down_workspace_bytes(T: int, k: int, d: int) -> int:
    out = _SZ()
    _check(lib().moe_blockscale_down_workspace_bytes(T, k, d, ctypes.byref(out)))
    return out.value


def blockscale_down(hq, hs, wt, offsets, pos, w_down, s_down, y, workspace, add=None, stream=None) -> None:
    """y [T][d] = add + the weighted sum of each token's experts' down products."""
    rc = (_calls or _load_calls()).down(hq, hs, wt, offsets, pos, w_down, s_down, y, workspace, add, stream)
    if rc is None:
        fn = "blockscale_down"
        (T, k), (E, d, f) = wt.shape, w_down.shape
        R, DB, FB = T * k, scale_blocks(d), scale_blocks(f)
        _need(fn, hq=(hq, torch.uint8, (R, f)), hs=(hs, torch.float32, (R, FB)), wt=(wt, torch.float32, (T, k)),
              offsets=(offsets, torch.int32, (E + 1,)), pos=(pos, torch.int32, (R,)),
              w_down=(w_down, torch.uint8, (E, d, f)), s_down=(s_down, torch.float32, (E, DB, FB)),
              y=(y, torch.float32, (T, d)))
        if add is not None:
            _need(fn, add=(add, torch.float32, (T, d)))
        _not_here(fn, hq, hs, wt, offsets, pos, w_down, s_down, y, add, workspace=workspace)
    if rc:
        _check(rc)


def profile_enable(on: bool) -> None:
    _check(lib().moe_profile_enable(1 if on else 0))


def profile_reset() -> None:
    _check(lib().moe_profile_reset())


def profile_collect(max_kernels: int = 32) -> dict:
    """{kernel name: (launches, total ms)} of the launches recorded so far."""
    names = ctypes.create_string_buffer(48 * max_kernels)
    launches = (ctypes.c_int64 * max_kernels)()
    ms = (ctypes.c_double * max_kernels)()
    n = ctypes.c_int32()
    _check(lib().moe_profile_collect(max_kernels, ctypes.addressof(names), ctypes.addressof(launches),
                                     ctypes.addressof(ms), ctypes.addressof(n)))
    out = {}
    for i in range(n.value):
        name = names.raw[48 * i:48 * (i + 1)].split(b"\0", 1)[0].decode()
        out[name] = (launches[i], ms[i])
    return out


# ---------------------------------------------------------------------------
# device-resident layer (memory management for callers and tests)
# ---------------------------------------------------------------------------
def _to_device_bytes(a: np.ndarray, device) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a).view(np.uint8).reshape(-1)).to(device)


class DeviceLayer:
    """A layer whose weights live on the GPU in the device layout.

    Built from canonical bytes (host numpy arrays): the tensors are uploaded
    and the whole layer is converted with one moe_prepare_weights call.
    `.desc` is the moe_layer descriptor of the prepared layer.
    """

    def __init__(self, E, d, f, k, fmt_gate_up, fmt_down, w_gate, w_up, w_down, grid, w_router,
                 fmt_shared=MOE_FMT_NONE, s_gate=None, s_up=None, s_down=None, device="cuda",
                 router_bias=None, down_gain=None, vq_codebook=None):
        self.E, self.d, self.f, self.k = E, d, f, k
        self.device = torch.device(device)
        has_shared = s_gate is not None
        shapes = {"w_gate": (fmt_gate_up, E, f, d, w_gate), "w_up": (fmt_gate_up, E, f, d, w_up),
                  "w_down": (fmt_down, E, d, f, w_down)}
        if has_shared:
            shapes.update({"s_gate": (fmt_shared, 1, f, d, s_gate), "s_up": (fmt_shared, 1, f, d, s_up),
                           "s_down": (fmt_shared, 1, d, f, s_down)})
        canon, self.tensors = {}, {}
        for name, (fmt, n_e, rows, K, blob) in shapes.items():
            n = matrix_bytes(fmt, n_e, rows, K)
            if blob.size != n:
                raise ValueError(f"{name}: expected {n} bytes, got {blob.size}")
            canon[name] = _to_device_bytes(blob, self.device)
            self.tensors[name] = torch.empty(n, dtype=torch.uint8, device=self.device)
        self.tensors["grid"] = _to_device_bytes(np.asarray(grid, np.uint8), self.device)
        self.tensors["w_router"] = torch.from_numpy(np.ascontiguousarray(w_router, np.float32)).to(self.device)
        if router_bias is not None:
            self.tensors["router_bias"] = torch.from_numpy(np.ascontiguousarray(router_bias, np.float32)).to(self.device)
        if down_gain is not None:
            self.tensors["down_gain"] = torch.from_numpy(np.ascontiguousarray(down_gain, np.float32)).to(self.device)
        n_codes = 0
        if vq_codebook is not None:
            cb = np.ascontiguousarray(vq_codebook, np.uint8).reshape(-1, 8)
            n_codes = cb.shape[0]
            self.tensors["vq_codebook"] = _to_device_bytes(cb, self.device)
        t = self.tensors
        src = MoeLayer(
            abi_version=MOE_ABI_VERSION, n_experts=E, d_model=d, d_ff=f, top_k=k, fmt_gate_up=fmt_gate_up,
            fmt_down=fmt_down, layout=MOE_LAYOUT_CANONICAL, w_gate=_ptr(canon["w_gate"]),
            w_up=_ptr(canon["w_up"]), w_down=_ptr(canon["w_down"]), iq2_grid=_ptr(t["grid"]),
            w_router=_ptr(t["w_router"]), has_shared=1 if has_shared else 0,
            fmt_shared=fmt_shared if has_shared else 0, s_gate=_ptr(canon.get("s_gate")),
            s_up=_ptr(canon.get("s_up")), s_down=_ptr(canon.get("s_down")),
            router_bias=_ptr(t.get("router_bias")), down_gain=_ptr(t.get("down_gain")),
            vq_codebook=_ptr(t.get("vq_codebook")), vq_codes=n_codes)
        self.desc = MoeLayer(w_gate=_ptr(t["w_gate"]), w_up=_ptr(t["w_up"]), w_down=_ptr(t["w_down"]),
                             s_gate=_ptr(t.get("s_gate")), s_up=_ptr(t.get("s_up")), s_down=_ptr(t.get("s_down")))
        prepare_weights(src, self.desc)
        torch.cuda.synchronize(self.device)  # the canonical copies are freed on return

    @classmethod
    def from_synth(cls, L, device="cuda"):
        """From a quantized_moe_amd.synth.Layer (canonical bytes)."""
        s = L.spec
        return cls(s.E, s.d, s.f, s.k, s.fmt_gate_up, s.fmt_down, L.w_gate, L.w_up, L.w_down, L.grid, L.w_router,
                   fmt_shared=s.fmt_shared if s.has_shared else MOE_FMT_NONE, s_gate=L.s_gate, s_up=L.s_up,
                   s_down=L.s_down, device=device, router_bias=getattr(L, "router_bias", None),
                   down_gain=getattr(L, "down_gain", None), vq_codebook=getattr(L, "vq_codebook", None))

    def workspace(self, T: int, op: int = MOE_OP_LAYER) -> torch.Tensor:
        n = workspace_bytes(self.desc, T, op)
        return torch.empty(max(n, 256), dtype=torch.uint8, device=self.device)
