"""ctypes binding of libmmf.so (the C ABI in include/mmf.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and streams.  If the library has not
been built this module raises on first use; there is no fallback path.

Raw entry points (``lib()``) take integer device pointers; the tensor helpers
below check dtypes/devices, allocate outputs with torch when none are given,
and pass the current torch stream.
"""
from __future__ import annotations

import ctypes as C
import os
import struct
import threading
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmmf.so")

MMF_OK = 0
STATUS = {
    0: "MMF_OK", 1: "MMF_ERR_INVALID_ARG", 2: "MMF_ERR_UNSUPPORTED_SHAPE", 3: "MMF_ERR_MISALIGNED",
    4: "MMF_ERR_WORKSPACE", 5: "MMF_ERR_CUDA", 6: "MMF_ERR_TIMEOUT", 7: "MMF_ERR_NO_DEVICE",
}

_lock = threading.Lock()
_lib = None

_P, _I64, _F, _SZ, _INT = C.c_void_p, C.c_int64, C.c_float, C.c_size_t, C.c_int

# name -> (restype, argtypes); mirrors include/mmf.h
SIGNATURES = {
    "mmf_status_string": (C.c_char_p, [_INT]),
    "mmf_version": (C.c_char_p, []),
    "mmf_packed_bytes": (_SZ, [_I64, _I64]),
    "mmf_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "mmf_fwd_launches": (_INT, [_I64, _I64, _I64, _INT]),
    "mmf_pack_ternary": (_INT, [_P, _I64, _I64, _F, _P, _P, _P]),
    "mmf_quantize_act": (_INT, [_P, _P, _F, _I64, _I64, _P, _P, _P]),
    "mmf_ternary_acc": (_INT, [_P, _P, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "mmf_bitlinear_fwd": (_INT, [_P, _P, _F, _P, _P, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "mmf_bitlinear_fwd_glu": (_INT, [_P, _P, _P, _F, _P, _P, _I64, _I64, _I64, _P, _P, _SZ, C.c_uint, _P]),
    "mmf_mlgru_scan": (_INT, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P]),
    "mmf_bwd_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "mmf_bitlinear_bwd": (_INT, [_P, _P, _P, _F, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _SZ, _P]),
    "mmf_bitlinear_fwd_group": (_INT, [_P, _P, _F, _I64, _I64, _P, _INT, _P, _SZ, C.c_uint, _P]),
    "mmf_bitlinear_fwd_noalloc": (_INT, [_P, _P, _F, _P, _P, _I64, _I64, _I64, _P, _P]),
    "mmf_embed_fwd": (_INT, [_P, _P, _F, _I64, _I64, _I64, _P, C.c_uint, _P]),
    "mmf_embed_bwd_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "mmf_embed_bwd": (_INT, [_P, _P, _F, _I64, _I64, _I64, _P, _P, _SZ, C.c_uint, _P]),
    "mmf_mlgru_scan_bwd_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "mmf_mlgru_scan_bwd": (_INT, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "mmf_adamw_step": (_INT, [_P, _INT, _P, _P, _P]),
    "mmf_adamw_scalars_at": (_INT, [_P, _P]),
    "mmf_hbm_copy": (_INT, [_P, _P, _SZ, _P]),
    "mmf_selftest_timeout": (_INT, [C.c_uint64, _P, _P]),
    "mmf_check_async": (_INT, [_P]),
}


FWD_PDL = 1
NOALLOC_SCRATCH_BYTES = 64 << 20   # MMF_NOALLOC_SCRATCH_BYTES
MAX_GROUP = 8
EMBED_IDS64, EMBED_TABLE_BF16, EMBED_ACCUMULATE = 1, 2, 4
ADAMW_STATE8, ADAMW_GRAD_BF16 = 1, 2
ADAMW_BLOCK = 256   # MMF_ADAMW_BLOCK


class Projection(C.Structure):
    """mirror of mmf_projection"""
    _fields_ = [("packed", _P), ("scale", _P), ("y", _P), ("N", _I64)]


class AdamWHyper(C.Structure):
    """mirror of mmf_adamw_hyper"""
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double), ("eps", C.c_double),
                ("grad_scale", C.c_double), ("step", _I64), ("seed", C.c_uint64)]


class MMFError(RuntimeError):
    def __init__(self, what: str, status: int):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


def lib() -> C.CDLL:
    """Loads libmmf.so (once); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -m bitlinear_rmsnorm_quant_b200.build`")
            L = C.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def check(status: int, what: str) -> None:
    if status != MMF_OK:
        raise MMFError(what, status)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# -- sizes ----------------------------------------------------------------------

def packed_bytes(N: int, K: int) -> int:
    return int(lib().mmf_packed_bytes(N, K))


def workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().mmf_workspace_bytes(M, K, N))


def fwd_launches(M: int, K: int, N: int, count: int = 1) -> int:
    return int(lib().mmf_fwd_launches(M, K, N, count))


def version() -> str:
    return lib().mmf_version().decode()


# -- entry points ---------------------------------------------------------------

def pack_ternary(W: torch.Tensor, eps_w: float = 1e-5, packed: torch.Tensor | None = None,
                 scale: torch.Tensor | None = None, stream=None):
    """fp32 W[N, K] -> (packed int32[N, K/16] holding uint32 words, scale fp32[1])."""
    _dev(W, torch.float32, "W")
    N, K = W.shape
    if packed is None:
        packed = torch.empty((N, K // 16), dtype=torch.int32, device=W.device)
    if scale is None:
        scale = torch.empty(4, dtype=torch.float32, device=W.device)[:1]
    check(lib().mmf_pack_ternary(W.data_ptr(), N, K, eps_w, packed.data_ptr(), scale.data_ptr(), _stream(stream)),
          "mmf_pack_ternary")
    return packed, scale


def quantize_act(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, stream=None):
    """bf16 x[M, K] -> (q int8[M, K], absmax fp32[M])."""
    _dev(x, torch.bfloat16, "x")
    _dev(gamma, torch.float32, "gamma")
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    a = torch.empty(max(M, 4), dtype=torch.float32, device=x.device)[:M]
    check(lib().mmf_quantize_act(x.data_ptr(), gamma.data_ptr(), eps, M, K, q.data_ptr(), a.data_ptr(),
                                 _stream(stream)), "mmf_quantize_act")
    return q, a


def _workspace(M, K, N, device, workspace):
    need = workspace_bytes(M, K, N)
    if need == 0:
        return None, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace.numel() < need:
        raise ValueError(f"workspace needs {need} bytes")
    return workspace, workspace.numel()


def ternary_acc(q: torch.Tensor, packed: torch.Tensor, N: int, workspace=None, out=None, stream=None):
    """int8 q[M, K] x packed[N, K/16] -> int32 acc[M, N]."""
    _dev(q, torch.int8, "q")
    M, K = q.shape
    acc = out if out is not None else torch.empty((M, N), dtype=torch.int32, device=q.device)
    ws, ws_n = _workspace(M, K, N, q.device, workspace)
    check(lib().mmf_ternary_acc(q.data_ptr(), packed.data_ptr(), M, K, N, acc.data_ptr(),
                                ws.data_ptr() if ws is not None else None, ws_n, _stream(stream)),
          "mmf_ternary_acc")
    return acc


def bitlinear_fwd(x: torch.Tensor, gamma: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor, N: int,
                  eps: float = 1e-6, workspace=None, out=None, stream=None):
    """bf16 x[M, K] -> bf16 y[M, N]."""
    _dev(x, torch.bfloat16, "x")
    M, K = x.shape
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    ws, ws_n = _workspace(M, K, N, x.device, workspace)
    check(lib().mmf_bitlinear_fwd(x.data_ptr(), gamma.data_ptr(), eps, packed.data_ptr(), scale.data_ptr(), M, K, N,
                                  y.data_ptr(), ws.data_ptr() if ws is not None else None, ws_n, _stream(stream)),
          "mmf_bitlinear_fwd")
    return y


def projection_array(items):
    """[(packed, scale, y, N), ...] -> ctypes array of mmf_projection (keep it alive while used)."""
    arr = (Projection * len(items))()
    for i, (packed, scale, y, N) in enumerate(items):
        arr[i] = Projection(packed.data_ptr(), scale.data_ptr(), y.data_ptr() if y is not None else None, N)
    return arr


def bitlinear_fwd_glu(g: torch.Tensor, u: torch.Tensor, gamma: torch.Tensor, packed: torch.Tensor,
                      scale: torch.Tensor, N: int, eps: float = 1e-6, workspace=None, out=None, flags: int = 0,
                      stream=None):
    """GLU down projection: bf16 g[M, K], u[M, K] -> bf16 y[M, N] of BitLinear(bf16(SiLU(g) * u))."""
    _dev(g, torch.bfloat16, "g")
    _dev(u, torch.bfloat16, "u")
    M, K = g.shape
    assert u.shape == g.shape
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=g.device)
    ws, ws_n = _workspace(M, K, N, g.device, workspace)
    check(lib().mmf_bitlinear_fwd_glu(g.data_ptr(), u.data_ptr(), gamma.data_ptr(), eps, packed.data_ptr(),
                                      scale.data_ptr(), M, K, N, y.data_ptr(),
                                      ws.data_ptr() if ws is not None else None, ws_n, flags, _stream(stream)),
          "mmf_bitlinear_fwd_glu")
    return y


def mlgru_scan(f_pre: torch.Tensor, c_pre: torch.Tensor, g_pre: torch.Tensor, h0: torch.Tensor | None = None,
               out=None, h_last=None, stream=None):
    """MLGRU recurrence: bf16 [B, T, D] pre-activations -> (bf16 o [B, T, D], fp32 h_last [B, D])."""
    for name, t in (("f_pre", f_pre), ("c_pre", c_pre), ("g_pre", g_pre)):
        _dev(t, torch.bfloat16, name)
    B, T, D = f_pre.shape
    o = out if out is not None else torch.empty((B, T, D), dtype=torch.bfloat16, device=f_pre.device)
    hl = h_last if h_last is not None else torch.empty((B, D), dtype=torch.float32, device=f_pre.device)
    check(lib().mmf_mlgru_scan(f_pre.data_ptr(), c_pre.data_ptr(), g_pre.data_ptr(),
                               h0.data_ptr() if h0 is not None else None, B, T, D, o.data_ptr(), hl.data_ptr(),
                               _stream(stream)), "mmf_mlgru_scan")
    return o, hl


def bitlinear_bwd(dy: torch.Tensor, x: torch.Tensor, gamma: torch.Tensor, packed: torch.Tensor,
                  scale: torch.Tensor, eps: float = 1e-6, stream=None):
    """Straight-through backward: bf16 dy[M, N], x[M, K] -> (bf16 dx[M, K], fp32 dgamma[K], fp32 dW[N, K])."""
    _dev(dy, torch.bfloat16, "dy")
    _dev(x, torch.bfloat16, "x")
    M, K = x.shape
    N = dy.shape[1]
    dx = torch.empty((M, K), dtype=torch.bfloat16, device=x.device)
    dg = torch.empty(K, dtype=torch.float32, device=x.device)
    dW = torch.empty((N, K), dtype=torch.float32, device=x.device)
    n = int(lib().mmf_bwd_workspace_bytes(M, K, N))
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)
    check(lib().mmf_bitlinear_bwd(dy.data_ptr(), x.data_ptr(), gamma.data_ptr(), eps, packed.data_ptr(),
                                  scale.data_ptr(), M, K, N, dx.data_ptr(), dg.data_ptr(), dW.data_ptr(),
                                  ws.data_ptr(), ws.numel(), _stream(stream)), "mmf_bitlinear_bwd")
    return dx, dg, dW


def bitlinear_fwd_group(x: torch.Tensor, gamma: torch.Tensor, weights, eps: float = 1e-6, workspace=None,
                        outs=None, flags: int = 0, stream=None):
    """bf16 x[M, K] and [(packed, scale, N), ...] sharing x -> [bf16 y_i[M, N_i], ...]."""
    _dev(x, torch.bfloat16, "x")
    M, K = x.shape
    ys = outs if outs is not None else [torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
                                        for (_, _, N) in weights]
    arr = projection_array([(pk, sc, y, N) for (pk, sc, N), y in zip(weights, ys)])
    ws, ws_n = _workspace(M, K, sum(N for _, _, N in weights), x.device, workspace)
    check(lib().mmf_bitlinear_fwd_group(x.data_ptr(), gamma.data_ptr(), eps, M, K, arr, len(weights),
                                        ws.data_ptr() if ws is not None else None, ws_n, flags, _stream(stream)),
          "mmf_bitlinear_fwd_group")
    return ys


def bitlinear_fwd_noalloc(x: torch.Tensor, gamma: torch.Tensor, packed: torch.Tensor, scale: torch.Tensor, N: int,
                          eps: float = 1e-6, out: torch.Tensor | None = None, stream=None):
    """As bitlinear_fwd, but the library's static scratch replaces the workspace
    (for callers that cannot allocate device memory; pass `out` to allocate
    nothing here either)."""
    _dev(x, torch.bfloat16, "x")
    M, K = x.shape
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    check(lib().mmf_bitlinear_fwd_noalloc(x.data_ptr(), gamma.data_ptr(), eps, packed.data_ptr(), scale.data_ptr(),
                                          M, K, N, y.data_ptr(), _stream(stream)), "mmf_bitlinear_fwd_noalloc")
    return y


# The current stream's handle of a device by its index.  torch.cuda.current_stream builds a Stream object first
# (3.3 us a call on the host, as long as a kernel's launch; this takes 0.1 us).
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(index: int, stream, call):
    """call(stream handle) with the tensors' device (its index) current and, when a stream is given, with it as
    torch's current stream, so that what the call allocates belongs to the stream that uses it."""
    if stream is None and index == torch.cuda.current_device():
        return call(_current_raw_stream(index))
    with torch.cuda.device(index):
        if stream is None:
            return call(_current_raw_stream(index))
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(s):
            return call(s.cuda_stream)


def _like(t: torch.Tensor, dtype, shape, index: int, name: str):
    """As _dev, for an argument of a known shape on the CUDA device of a known index."""
    if t.dtype != dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        _dev(t, dtype, name)
        if t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _embed_ids(ids: torch.Tensor) -> int:
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be torch.int32 or torch.int64, got {ids.dtype}")
    _dev(ids, ids.dtype, "ids")
    return EMBED_IDS64 if ids.dtype == torch.int64 else 0


def embed_fwd(ids: torch.Tensor, table: torch.Tensor, scale: float = 1.0, out=None, stream=None):
    """int32/int64 ids[...] and fp32/bf16 table[V, K] -> bf16 x[..., K] = scale * table[ids]; an id outside
    [0, V) gives a row of zeros."""
    flags = _embed_ids(ids)
    index = ids.get_device()
    if table.dtype == torch.bfloat16:
        flags |= EMBED_TABLE_BF16
    elif table.dtype != torch.float32:
        raise TypeError(f"table must be torch.float32 or torch.bfloat16, got {table.dtype}")
    V, K = table.shape
    _like(table, table.dtype, (V, K), index, "table")
    shape = (*ids.shape, K)
    if out is not None:
        _like(out, torch.bfloat16, shape, index, "out")

    def call(s):
        x = out if out is not None else torch.empty(shape, dtype=torch.bfloat16, device=ids.device)
        check(lib().mmf_embed_fwd(ids.data_ptr(), table.data_ptr(), scale, V, ids.numel(), K, x.data_ptr(), flags, s),
              "mmf_embed_fwd")
        return x

    return _on(index, stream, call)


def embed_bwd_workspace_bytes(V: int, M: int, K: int) -> int:
    return int(lib().mmf_embed_bwd_workspace_bytes(V, M, K))


def embed_bwd(ids: torch.Tensor, dx: torch.Tensor, V: int, scale: float = 1.0, out=None, accumulate: bool = False,
              workspace=None, stream=None):
    """Gradient of embed_fwd for its table: int32/int64 ids[...] and bf16 dx[..., K] -> fp32 dtable[V, K];
    with accumulate the sums are added to `out`, and rows no id names stay as they are."""
    flags = _embed_ids(ids)
    index = ids.get_device()
    K = dx.shape[-1]
    _like(dx, torch.bfloat16, (*ids.shape, K), index, "dx")
    if out is not None:
        _like(out, torch.float32, (V, K), index, "out")
    if accumulate:
        if out is None:
            raise ValueError("accumulate adds to out: out is missing")
        flags |= EMBED_ACCUMULATE
    M = ids.numel()
    need = embed_bwd_workspace_bytes(V, M, K)
    if workspace is not None:
        _like(workspace, torch.uint8, workspace.shape, index, "workspace")
        if workspace.numel() < need:
            raise ValueError(f"workspace needs {need} bytes")

    def call(s):
        d = out if out is not None else torch.empty((V, K), dtype=torch.float32, device=ids.device)
        ws = workspace
        if ws is None and need:
            ws = torch.empty(need, dtype=torch.uint8, device=ids.device)
        check(lib().mmf_embed_bwd(ids.data_ptr(), dx.data_ptr(), scale, V, M, K, d.data_ptr(),
                                  ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
                                  flags, s), "mmf_embed_bwd")
        return d

    return _on(index, stream, call)


def mlgru_scan_bwd_workspace_bytes(B: int, T: int, D: int) -> int:
    return int(lib().mmf_mlgru_scan_bwd_workspace_bytes(B, T, D))


def mlgru_scan_bwd(f_pre: torch.Tensor, c_pre: torch.Tensor, g_pre: torch.Tensor, d_o: torch.Tensor,
                   h0: torch.Tensor | None = None, dh_last: torch.Tensor | None = None, outs=None, dh0=None,
                   workspace=None, stream=None):
    """Gradient of mlgru_scan: its bf16 [B, T, D] inputs and d_o, the gradient of o (and fp32 [B, D] h0 and
    dh_last) -> (bf16 df_pre, dc_pre, dg_pre [B, T, D], fp32 dh0 [B, D])."""
    _dev(f_pre, torch.bfloat16, "f_pre")
    shape = f_pre.shape
    B, T, D = shape
    dev = f_pre.get_device()
    _like(c_pre, torch.bfloat16, shape, dev, "c_pre")
    _like(g_pre, torch.bfloat16, shape, dev, "g_pre")
    _like(d_o, torch.bfloat16, shape, dev, "d_o")
    for name, t in (("h0", h0), ("dh_last", dh_last), ("dh0", dh0)):
        if t is not None:
            _like(t, torch.float32, (B, D), dev, name)
    if outs is not None:
        for name, t in zip(("df_pre", "dc_pre", "dg_pre"), outs, strict=True):
            _like(t, torch.bfloat16, shape, dev, name)
    need = mlgru_scan_bwd_workspace_bytes(B, T, D)
    if workspace is not None:
        _like(workspace, torch.uint8, workspace.shape, dev, "workspace")
        if workspace.numel() < need:
            raise ValueError(f"workspace needs {need} bytes")

    def call(s):
        df, dc, dg = outs if outs is not None else (torch.empty_like(f_pre), torch.empty_like(f_pre),
                                                    torch.empty_like(f_pre))
        dh = dh0 if dh0 is not None else torch.empty((B, D), dtype=torch.float32, device=f_pre.device)
        ws = workspace
        if ws is None and need:
            ws = torch.empty(need, dtype=torch.uint8, device=f_pre.device)
        check(lib().mmf_mlgru_scan_bwd(f_pre.data_ptr(), c_pre.data_ptr(), g_pre.data_ptr(), d_o.data_ptr(),
                                       h0.data_ptr() if h0 is not None else None,
                                       dh_last.data_ptr() if dh_last is not None else None, B, T, D, df.data_ptr(),
                                       dc.data_ptr(), dg.data_ptr(), dh.data_ptr(),
                                       ws.data_ptr() if ws is not None else None,
                                       ws.numel() if ws is not None else 0, s),
              "mmf_mlgru_scan_bwd")
        return df, dc, dg, dh

    return _on(dev, stream, call)


@dataclass(slots=True)
class AdamWTensor:
    """One tensor of an AdamW step: fp32 p, its fp32 or bf16 gradient g, and its moments m, v (adamw_state),
    fp32 or float8_e4m3fn / float8_e5m2 with their blocks' scales; p_bf16 receives a bf16 copy of the new p."""
    p: torch.Tensor
    g: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    m_scale: torch.Tensor | None = None
    v_scale: torch.Tensor | None = None
    p_bf16: torch.Tensor | None = None
    weight_decay: float = 0.0


def adamw_state(p: torch.Tensor, bits: int = 32) -> dict:
    """Fresh moments for p in 32 or 8 bits, as AdamWTensor's keyword arguments."""
    if bits == 32:
        return {"m": torch.zeros_like(p), "v": torch.zeros_like(p)}
    if bits != 8:
        raise ValueError(f"bits must be 32 or 8, got {bits}")
    blocks = -(-p.numel() // ADAMW_BLOCK)
    return {"m": torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(torch.float8_e4m3fn),
            "v": torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(torch.float8_e5m2),
            "m_scale": torch.zeros(blocks, dtype=torch.float32, device=p.device),
            "v_scale": torch.zeros(blocks, dtype=torch.float32, device=p.device)}


_ADAMW_DESC = struct.Struct("<7QqfI")   # mmf_adamw_tensor


# the checks of a step run once per tensor on the host: the names they use, looked up once
_F32, _BF16, _E4M3, _E5M2 = torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.float8_e5m2
_pack_adamw = _ADAMW_DESC.pack_into


def _adamw_describe(t: AdamWTensor, index: int, buf, at: int) -> None:
    p, g, m, v, ms, vs, pb = t.p, t.g, t.m, t.v, t.m_scale, t.v_scale, t.p_bf16
    n = p.numel()
    flags = 0
    if g.dtype is _BF16:
        flags = ADAMW_GRAD_BF16
    elif g.dtype is not _F32:
        raise TypeError(f"g must be torch.float32 or torch.bfloat16, got {g.dtype}")
    if p.dtype is not _F32:
        raise TypeError(f"p must be torch.float32, got {p.dtype}")
    msp = vsp = pbp = 0
    if m.dtype is _E4M3:
        flags |= ADAMW_STATE8
        if v.dtype is not _E5M2:
            raise TypeError(f"v must be torch.float8_e5m2 beside an 8-bit m, got {v.dtype}")
        if ms is None or vs is None:
            raise ValueError("m_scale and v_scale are missing: 8-bit moments need them")
        blocks = (-(-n // ADAMW_BLOCK),)
        _like(ms, _F32, blocks, index, "m_scale")
        _like(vs, _F32, blocks, index, "v_scale")
        msp, vsp = ms.data_ptr(), vs.data_ptr()
    elif m.dtype is not _F32 or v.dtype is not _F32 or ms is not None or vs is not None:
        raise TypeError("m and v must be torch.float32, or torch.float8_e4m3fn and torch.float8_e5m2 with their scales")
    if pb is not None:
        _like(pb, _BF16, p.shape, index, "p_bf16")
        pbp = pb.data_ptr()
    if not (p.get_device() == g.get_device() == m.get_device() == v.get_device() == index):
        raise ValueError(f"p, g, m and v must be on cuda:{index}, got {p.device}, {g.device}, {m.device}, {v.device}")
    if not (g.numel() == m.numel() == v.numel() == n and p.is_contiguous() and g.is_contiguous()
            and m.is_contiguous() and v.is_contiguous()):
        raise ValueError("p, g, m and v must be contiguous, with as many elements each")
    _pack_adamw(buf, at, p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), msp, vsp, pbp, n, t.weight_decay, flags)


def _adamw_hyper(step, lr, beta1, beta2, eps, grad_scale, seed) -> AdamWHyper:
    """seed None: the step.  The noise of 8-bit moments has to be new at every step; with one that stays, each
    element rounds at a threshold of its own for good and its moments are biased (v 3 times too large in the median
    after some hundred steps)."""
    if seed is None:
        seed = step
    elif not -(1 << 63) <= seed < 1 << 64:
        raise ValueError(f"seed must fit 64 bits, got {seed}")
    return AdamWHyper(lr, beta1, beta2, eps, grad_scale, step, seed)


def adamw_scalars(step: int, lr: float, beta1: float = 0.9, beta2: float = 0.95, eps: float = 1e-8,
                  grad_scale: float = 1.0, seed: int | None = None) -> torch.Tensor:
    """A step's scalars as 32 bytes on the host (pinned when there is a GPU): copy them into the device buffer
    that a captured adamw_step was given as `scalars` before each replay.  `seed` as for adamw_step."""
    out = torch.zeros(32, dtype=torch.uint8, pin_memory=torch.cuda.is_available())
    hyper = _adamw_hyper(step, lr, beta1, beta2, eps, grad_scale, seed)
    check(lib().mmf_adamw_scalars_at(C.byref(hyper), out.data_ptr()), "mmf_adamw_scalars_at")
    return out


def adamw_step(tensors, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.95, eps: float = 1e-8,
               grad_scale: float = 1.0, seed: int | None = None, scalars: torch.Tensor | None = None, stream=None) -> None:
    """One AdamW step over a sequence of AdamWTensor, in place; `step` counts from 1.  With `scalars` (uint8[32]
    on the device, see adamw_scalars) the kernel takes lr, the bias corrections, grad_scale and seed from there.
    A graph captured without them repeats its step's on every replay, the noise too.
    `seed` is that of the rounding noise of 8-bit moments (without any it changes nothing): the step when not given;
    a caller that gives one gives another at every step, or the moments are biased."""
    tensors = list(tensors)
    if not tensors:
        return
    index = tensors[0].p.get_device()
    if index < 0:
        raise ValueError("p must be a CUDA tensor")
    size = _ADAMW_DESC.size
    buf = bytearray(size * len(tensors))
    for i, t in enumerate(tensors):
        _adamw_describe(t, index, buf, i * size)
    if scalars is not None:
        _like(scalars, torch.uint8, (32,), index, "scalars")
    hyper = _adamw_hyper(step, lr, beta1, beta2, eps, grad_scale, seed)
    desc = (C.c_char * len(buf)).from_buffer(buf)

    def call(s):
        check(lib().mmf_adamw_step(C.addressof(desc), len(tensors), C.addressof(hyper),
                                   scalars.data_ptr() if scalars is not None else None, s), "mmf_adamw_step")

    _on(index, stream, call)


def hbm_copy(src: torch.Tensor, dst: torch.Tensor, stream=None):
    nbytes = src.numel() * src.element_size()
    check(lib().mmf_hbm_copy(src.data_ptr(), dst.data_ptr(), nbytes, _stream(stream)), "mmf_hbm_copy")


def selftest_timeout(limit_ns: int, waited_out: torch.Tensor | None = None, stream=None):
    check(lib().mmf_selftest_timeout(limit_ns, waited_out.data_ptr() if waited_out is not None else None,
                                     _stream(stream)), "mmf_selftest_timeout")


def check_async(stream=None):
    check(lib().mmf_check_async(_stream(stream)), "mmf_check_async")
