"""Python binding of ``liblowbit.so``, the gfx950 low-bit-weight GEMM library.

Argument marshalling only: every step runs in the HIP kernels of the library.
PyTorch supplies device memory (``torch.empty`` on the GPU) and the current
HIP stream. If the library is not built, or no gfx950 GPU is present, calls
raise; there is no fallback implementation.

    packed = pack_ternary(codes_int8_cuda)            # [N, K/4] uint8
    y = gemm(x_bf16_cuda, packed, scales_f16_cuda, "ternary", bias=None)
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "liblowbit.so")

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DTYPE, ERR_GROUP, ERR_WORKSPACE, ERR_DEVICE, ERR_HIP, ERR_OVERLAP = range(10)
F16, BF16, F32, NONE = 0, 1, 2, 3
BINARY, TERNARY, BASE3, INT4 = 1, 2, 3, 4
ACT_NONE, ACT_GELU = 0, 1
GROUP = 128

_FMT = {"ternary": TERNARY, "binary": BINARY, "base3": BASE3, "int4": INT4, TERNARY: TERNARY, BINARY: BINARY,
        BASE3: BASE3, INT4: INT4}
_DT = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
_ACT = {None: ACT_NONE, "none": ACT_NONE, "gelu": ACT_GELU, ACT_NONE: ACT_NONE, ACT_GELU: ACT_GELU}

_lib = None

# (name, restype, argtypes) for every entry point of include/lowbit.h
_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = [
    ("lowbit_abi_version", _I32, []),
    ("lowbit_status_string", ctypes.c_char_p, [_I32]),
    ("lowbit_init", _I32, []),
    ("lowbit_debug_force_variant", _I32, [ctypes.c_char_p]),
    ("lowbit_packed_bytes", _I64, [_I32, _I64, _I64]),
    ("lowbit_scale_count", _I64, [_I64, _I64, _I32]),
    ("pack_ternary", _I32, [_P, _I64, _I64, _P, _P, _P]),
    ("pack_binary", _I32, [_P, _I64, _I64, _P, _P, _P]),
    ("pack_base3", _I32, [_P, _I64, _I64, _P, _P, _P]),
    ("unpack_lowbit", _I32, [_I32, _P, _I64, _I64, _P, _P, _P]),
    ("base3_to_int2", _I32, [_P, _I64, _I64, _P, _P, _P]),
    ("lowbit_gemm_workspace_bytes", _SZ, [_I32, _I64, _I64, _I64]),
    ("lowbit_gemm", _I32, [_I32, _P, _I32, _I64, _I64, _I64, _P, _P, _I32, _I64,
                           _P, _I32, _P, _I32, _I64, _I32, _P, _SZ, _P]),
    ("lowbit_gelu", _I32, [_P, _P, _I32, _I64, _P]),
    ("lowbit_gemm_grouped", _I32, [_I32, _I32, _P, _I32, _I64, _I64, _I64, _P, _P, _I32, _I64,
                                   _P, _I32, _P, _I32, _I64, _I32, _P, _SZ, _P]),
    ("lowbit_gemm_grouped_workspace_bytes", _SZ, [_I32, _I32, _I64, _I64, _I64]),
    ("lowbit_gemm_noalloc", _I32, [_I32, _P, _I32, _I64, _I64, _I64, _P, _P, _I32, _I64,
                                   _P, _I32, _P, _I32, _I64, _I32, _P]),
    ("pack_int4", _I32, [_P, _I64, _I64, _P, _P, _P]),
    ("lowbit_gemm_int4_workspace_bytes", _SZ, [_I64, _I64, _I64]),
    ("lowbit_gemm_int4", _I32, [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _I32, _I64,
                                _P, _I32, _P, _I32, _I64, _I32, _P, _SZ, _P]),
    ("lowbit_gemv_int4", _I32, [_P, _I32, _I64, _I64, _I64, _P, _P, _P, _I32, _I64,
                                _P, _I32, _P, _I32, _I64, _I32, _P]),
    ("lowbit_kv_append", _I32, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _I32, _P, _I64, _I64, _P, _I64, _I64,
                                _P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _I64, _I32, _P, _P]),
    ("lowbit_kv_read", _I32, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _I32, _P, _I64, _I64, _P, _I64, _I64, _P]),
    ("lowbit_attention", _I32, [_P, _P, _I64, _P, _P, _I64, _I64, _I64, _I64, _I32, _P, _I64, _I64, _I64,
                                _P, _I64, _I64, _P, ctypes.c_float, _I32, _I64, _P, _SZ, _P]),
    ("lowbit_attention_workspace_bytes", _SZ, [_I64, _I64, _I64, _I64, _I64, _I64, _I64, _I64]),
    ("lowbit_quantize", _I32, [_I32, _P, _I64, _I64, _I64, _P, _P, _P, _P]),
]
MAX_GROUP = 8


class LowbitError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Load liblowbit.so (built in-tree); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m bit_weight_gemm_int2_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().lowbit_status_string(status).decode()


def _check(status: int, what: str):
    if status != OK:
        raise LowbitError(status, what)


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _cuda(t: torch.Tensor, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")


def packed_bytes(fmt, N: int, K: int) -> int:
    return int(lib().lowbit_packed_bytes(_FMT[fmt], N, K))


def workspace_bytes(fmt, M: int, N: int, K: int) -> int:
    return int(lib().lowbit_gemm_workspace_bytes(_FMT[fmt], M, N, K))


def force_variant(name=None):
    """Test hook: force one kernel family ("large", "small", "large-wide",
    "large-pair", "small-split"; for the ternary quantiser "quant-eighth",
    "quant-lane": eight or one lane per group) for every later call of the process, or restore the
    automatic choice with None / "auto"."""
    _check(lib().lowbit_debug_force_variant(None if name is None else name.encode()), "lowbit_debug_force_variant")


_WORKSPACES = {}


def new_workspace(nbytes: int, device=None, stream=None) -> torch.Tensor:
    """A workspace for lowbit_gemm: zeroed device bytes (the library returns
    its counters to zero after every call, so it stays reusable). The zeros
    are written on `stream` (default: the current stream), the stream the
    workspace is then used on."""
    dev = torch.device(device or "cuda")
    st = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.stream(st):
        ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=dev)
        ws.zero_()
    return ws


def _given_workspace(workspace: torch.Tensor, need: int, what: str) -> int:
    """The bytes of a workspace given by the caller: one dense block of GPU
    memory where one is needed (the elements of an expanded or strided tensor
    count more bytes than it owns, or others than those behind its address)."""
    if need and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if need:
        _cuda(workspace, "workspace")
    size = workspace.numel() * workspace.element_size()
    if size < need:
        raise ValueError(f"workspace holds {size} bytes, {what} needs {need}")
    return size


def _shared_workspace(device: torch.device, nbytes: int, stream) -> torch.Tensor:
    """A workspace per (device, stream), reused by every call on that stream
    that passes none: calls on one stream never overlap, and calls on two
    streams never share one. It is zeroed on the stream it serves, and grows
    when a larger problem needs more (the buffer it replaces is kept alive
    until the work queued on the stream so far is done); grow it before any
    HIP graph capture by running the largest problem once."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    st = stream if stream is not None else torch.cuda.current_stream(idx)
    key = (idx, st.cuda_stream)
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        if ws is not None:
            ws.record_stream(st)
        ws = new_workspace(max(nbytes, 1 << 20), torch.device("cuda", idx), st)
        _WORKSPACES[key] = ws
    return ws


def _row_bytes(fmt: int, K: int) -> int:
    if fmt == BASE3:
        return (K + 4) // 5
    return K // {TERNARY: 4, BINARY: 8, INT4: 2}[fmt]


def _counted(fn, src: torch.Tensor, N: int, K: int, out: torch.Tensor, check: bool, stream, what: str):
    cnt = torch.empty(1, dtype=torch.int32, device=src.device) if check else None
    _check(fn(src.data_ptr(), N, K, out.data_ptr(), _ptr(cnt), _stream(stream)), fn.__name__)
    if check:
        bad = int(cnt.item())
        if bad:
            raise ValueError(f"{bad} {what}")
    return out


def _pack(fn, codes: torch.Tensor, fmt: int, check: bool, stream) -> torch.Tensor:
    _cuda(codes, "codes")
    want = torch.uint8 if fmt == INT4 else torch.int8
    if codes.dtype != want or codes.dim() != 2:
        raise ValueError(f"codes must be a 2-D {want} tensor")
    codes = codes.contiguous()
    N, K = codes.shape
    out = torch.empty((N, _row_bytes(fmt, K)), dtype=torch.uint8, device=codes.device)
    return _counted(fn, codes, N, K, out, check, stream, "code(s) outside the allowed set")


def pack_ternary(codes: torch.Tensor, check: bool = True, stream=None) -> torch.Tensor:
    """int8 codes [N, K] in {-1,0,+1} -> packed uint8 [N, K/4] (K % 16 == 0)."""
    return _pack(lib().pack_ternary, codes, TERNARY, check, stream)


def pack_binary(codes: torch.Tensor, check: bool = True, stream=None) -> torch.Tensor:
    """int8 codes [N, K] in {-1,+1} -> packed uint8 [N, K/8] (K % 32 == 0)."""
    return _pack(lib().pack_binary, codes, BINARY, check, stream)


def pack_int4(codes: torch.Tensor, check: bool = True, stream=None) -> torch.Tensor:
    """uint8 codes [N, K] in 0..15 -> packed uint8 [N, K/2] (K % 8 == 0)."""
    return _pack(lib().pack_int4, codes, INT4, check, stream)


def gemm_int4(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
              bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, activation=None,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Y = act(X W^T + bias) with W = s * (q - z) from 4-bit codes (lowbit_gemm_int4).

    x: [M, K] fp16/bf16; packed: [N, K/2] uint8; scales, zeros: fp16 [N, K/128].
    A workspace for the row sums is allocated per call unless one is given."""
    for t, nm in ((x, "x"), (packed, "packed"), (scales, "scales"), (zeros, "zeros")):
        _cuda(t, nm)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride along K")
    M, K = x.shape
    N = packed.shape[0]
    packed, scales, zeros = packed.contiguous(), scales.contiguous(), zeros.contiguous()
    _check_packed(INT4, packed, N, K)
    for t, nm in ((scales, "scales"), (zeros, "zeros")):
        if t.dtype != torch.float16 or tuple(t.shape) != (N, K // GROUP):
            raise ValueError(f"{nm} must be float16 [{N}, {K // GROUP}]")
    if bias is not None:
        _cuda(bias, "bias")
        bias = bias.contiguous()
        if bias.numel() != N or bias.dtype not in _DT:
            raise ValueError(f"bias must hold {N} float16, bfloat16 or float32 values")
    odt = out_dtype or x.dtype
    if out is None:
        out = torch.empty((M, N), dtype=odt, device=x.device)
    elif tuple(out.shape) != (M, N) or out.stride(1) != 1 or out.dtype not in _DT:
        raise ValueError(f"out must be [{M}, {N}] with unit stride along N")
    need = int(lib().lowbit_gemm_int4_workspace_bytes(M, N, K))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    size = _given_workspace(workspace, need, "lowbit_gemm_int4")
    _check(lib().lowbit_gemm_int4(
        x.data_ptr(), _DT[x.dtype], M, K, x.stride(0), packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
        GROUP, N, _ptr(bias), NONE if bias is None else _DT[bias.dtype], out.data_ptr(), _DT[out.dtype],
        out.stride(0), _ACT[activation], workspace.data_ptr(), size,
        _stream(stream)), "lowbit_gemm_int4")
    return out


def quantize(w: torch.Tensor, fmt, check: bool = True, out=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Dense FP16 weights [N, K] (row stride may exceed K) -> (packed uint8
    [N, K/4] or [N, K/8], fp16 scales [N, K/128]) by lowbit_quantize, into
    `out` = (packed, scales) when given. With check, waits for the device and
    raises on NaN or infinite weights."""
    _cuda(w, "w")
    if w.dtype != torch.float16 or w.dim() != 2 or w.stride(1) != 1:
        raise ValueError("w must be a 2-D float16 tensor with unit stride along K")
    fmt = _FMT[fmt]
    N, K = w.shape
    if fmt not in (TERNARY, BINARY) or K % GROUP:
        raise ValueError("quantize makes ternary or binary codes; K must be a multiple of 128")
    if out is None:
        packed = torch.empty((N, _row_bytes(fmt, K)), dtype=torch.uint8, device=w.device)
        scales = torch.empty((N, K // GROUP), dtype=torch.float16, device=w.device)
    else:
        packed, scales = out
        if (packed.dtype != torch.uint8 or tuple(packed.shape) != (N, _row_bytes(fmt, K))
                or not packed.is_contiguous() or scales.dtype != torch.float16
                or tuple(scales.shape) != (N, K // GROUP) or not scales.is_contiguous()):
            raise ValueError("out must be contiguous (uint8 packed [N, row bytes], float16 scales [N, K/128])")
    cnt = torch.empty(1, dtype=torch.int32, device=w.device) if check else None
    _check(lib().lowbit_quantize(fmt, w.data_ptr(), N, K, w.stride(0), packed.data_ptr(), scales.data_ptr(),
                                 _ptr(cnt), _stream(stream)), "lowbit_quantize")
    if check:
        bad = int(cnt.item())
        if bad:
            raise ValueError(f"{bad} non-finite weight(s)")
    return packed, scales


def pack_base3(codes: torch.Tensor, check: bool = True, stream=None) -> torch.Tensor:
    """int8 codes [N, K] in {-1,0,+1} -> base-3 uint8 [N, ceil(K/5)] (any K >= 1)."""
    return _pack(lib().pack_base3, codes, BASE3, check, stream)


def base3_to_int2(packed: torch.Tensor, K: int, check: bool = True, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """base-3 uint8 [N, ceil(K/5)] -> INT2 uint8 [N, K/4] for gemm (K % 16 == 0).
    With check, waits for the device and raises on invalid base-3 bytes."""
    _cuda(packed, "packed")
    if packed.dtype != torch.uint8 or packed.dim() != 2 or packed.shape[1] != (K + 4) // 5:
        raise ValueError("packed must be a 2-D uint8 tensor of ceil(K/5) bytes per row")
    packed = packed.contiguous()
    N = packed.shape[0]
    if out is None:
        out = torch.empty((N, K // 4), dtype=torch.uint8, device=packed.device)
    elif out.dtype != torch.uint8 or tuple(out.shape) != (N, K // 4) or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint8 tensor [N, K/4]")
    return _counted(lib().base3_to_int2, packed, N, K, out, check, stream, "invalid base-3 value(s)")


def _check_packed(fmt, packed: torch.Tensor, N: int, K: int):
    """The library reads N x (bytes per row) packed bytes: check the tensor holds them."""
    if packed.dtype != torch.uint8 or packed.dim() != 2:
        raise ValueError("packed must be a 2-D uint8 tensor")
    row = _row_bytes(_FMT[fmt], K)
    if tuple(packed.shape) != (N, row):
        raise ValueError(f"packed must be [{N}, {row}] for K = {K}, got {list(packed.shape)}")


def unpack(fmt, packed: torch.Tensor, K: int, stream=None) -> Tuple[torch.Tensor, int]:
    """packed [N, K/4, K/8, ceil(K/5) or K/2] -> (codes [N, K], number of invalid codes);
    int8 codes, uint8 for the 4-bit format."""
    _cuda(packed, "packed")
    packed = packed.contiguous()
    N = packed.shape[0]
    _check_packed(fmt, packed, N, K)
    codes = torch.empty((N, K), dtype=torch.uint8 if _FMT[fmt] == INT4 else torch.int8, device=packed.device)
    cnt = torch.empty(1, dtype=torch.int32, device=packed.device)
    _check(lib().unpack_lowbit(_FMT[fmt], packed.data_ptr(), N, K, codes.data_ptr(), cnt.data_ptr(),
                               _stream(stream)), "unpack_lowbit")
    return codes, int(cnt.item())


def gemm(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, fmt, bias: Optional[torch.Tensor] = None,
         out_dtype: Optional[torch.dtype] = None, activation=None, out: Optional[torch.Tensor] = None,
         workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = act(X W^T + bias) with W = scale_g * t from packed codes.

    x: [M, K] fp16/bf16 (row stride may exceed K); packed: [N, K/4] (ternary) or
    [N, K/8] (binary) uint8; scales: fp16 [N, K/128]; bias: [N] or None.
    Output dtype defaults to x's dtype."""
    for t, nm in ((x, "x"), (packed, "packed"), (scales, "scales")):
        _cuda(t, nm)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride along K")
    M, K = x.shape
    N = packed.shape[0]
    packed = packed.contiguous()
    scales = scales.contiguous()
    if x.dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("x must be float16 or bfloat16")
    _check_packed(fmt, packed, N, K)
    if scales.dtype != torch.float16 or tuple(scales.shape) != (N, K // GROUP):
        raise ValueError(f"scales must be float16 [{N}, {K // GROUP}]")
    if bias is not None:
        _cuda(bias, "bias")
        bias = bias.contiguous()
        if bias.numel() != N or bias.dtype not in _DT:
            raise ValueError(f"bias must hold {N} float16, bfloat16 or float32 values")
    odt = out_dtype or x.dtype
    if out is None:
        out = torch.empty((M, N), dtype=odt, device=x.device)
    elif tuple(out.shape) != (M, N) or out.dim() != 2 or out.stride(1) != 1 or out.dtype not in _DT:
        raise ValueError(f"out must be [{M}, {N}] with unit stride along N")
    ws_need = workspace_bytes(fmt, M, N, K)
    if ws_need and workspace is None:
        workspace = _shared_workspace(x.device, ws_need, stream)
    size = 0 if workspace is None else _given_workspace(workspace, ws_need, "lowbit_gemm")
    st = lib().lowbit_gemm(
        _FMT[fmt], x.data_ptr(), _DT[x.dtype], M, K, x.stride(0),
        packed.data_ptr(), scales.data_ptr(), GROUP, N,
        _ptr(bias), NONE if bias is None else _DT[bias.dtype],
        out.data_ptr(), _DT[out.dtype], out.stride(0), _ACT[activation],
        _ptr(workspace), size, _stream(stream))
    _check(st, "lowbit_gemm")
    return out


def _ptr_array(ptrs):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


def gemm_grouped(xs, packeds, scales, fmt, biases=None, out_dtype: Optional[torch.dtype] = None,
                 activation=None, outs=None, workspace: Optional[torch.Tensor] = None,
                 stream=None):
    """Several independent linears of one shape in one launch (small M):
    ys[z] = act(xs[z] W[z]^T + biases[z]). Every x shares shape, dtype and row
    stride; every packed / scales pair shares shape. Returns the list of outputs."""
    count = len(xs)
    if not 1 <= count <= MAX_GROUP or len(packeds) != count or len(scales) != count:
        raise ValueError(f"1 .. {MAX_GROUP} problems, with one packed and one scales tensor each")
    if biases is not None and len(biases) != count:
        raise ValueError("one bias per problem")
    x0 = xs[0]
    for t in list(xs) + list(packeds) + list(scales):
        _cuda(t, "operand")
    if x0.dim() != 2 or any(x.shape != x0.shape or x.stride() != x0.stride() or x.dtype != x0.dtype for x in xs):
        raise ValueError("every x must have the shape, stride and dtype of the first")
    if x0.stride(1) != 1:
        raise ValueError("x must have unit stride along K")
    M, K = x0.shape
    packeds = [p.contiguous() for p in packeds]
    scales = [s_.contiguous() for s_ in scales]
    N = packeds[0].shape[0]
    for p in packeds:
        _check_packed(fmt, p, N, K)
    if any(s_.dtype != torch.float16 or tuple(s_.shape) != (N, K // GROUP) for s_ in scales):
        raise ValueError(f"scales must be float16 [{N}, {K // GROUP}]")
    odt = out_dtype or x0.dtype
    if outs is None:
        outs = [torch.empty((M, N), dtype=odt, device=x0.device) for _ in range(count)]
    elif len(outs) != count or any(tuple(y.shape) != (M, N) or y.stride(1) != 1 or y.dtype != outs[0].dtype
                                   or y.stride(0) != outs[0].stride(0) for y in outs):
        raise ValueError(f"outs: {count} tensors [{M}, {N}] of one dtype and row stride")
    bdt = NONE
    if biases is not None:
        biases = [b.contiguous() for b in biases]
        if any(b.numel() != N or b.dtype != biases[0].dtype for b in biases):
            raise ValueError(f"biases: {count} tensors of {N} values and one dtype")
        bdt = _DT[biases[0].dtype]
    need = int(lib().lowbit_gemm_grouped_workspace_bytes(count, _FMT[fmt], M, N, K))
    if need and workspace is None:
        workspace = _shared_workspace(x0.device, need, stream)
    size = 0 if workspace is None else _given_workspace(workspace, need, "lowbit_gemm_grouped")
    st = lib().lowbit_gemm_grouped(
        count, _FMT[fmt], _ptr_array([x.data_ptr() for x in xs]), _DT[x0.dtype], M, K, x0.stride(0),
        _ptr_array([p.data_ptr() for p in packeds]), _ptr_array([s_.data_ptr() for s_ in scales]), GROUP, N,
        None if biases is None else _ptr_array([b.data_ptr() for b in biases]), bdt,
        _ptr_array([y.data_ptr() for y in outs]), _DT[outs[0].dtype], outs[0].stride(0), _ACT[activation],
        _ptr(workspace), size, _stream(stream))
    _check(st, "lowbit_gemm_grouped")
    return outs


def gelu(x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Exact-erf GELU (x * Phi(x)) in FP32, stored in x's dtype."""
    _cuda(x, "x")
    x = x.contiguous()
    out = torch.empty_like(x) if out is None else out
    _check(lib().lowbit_gelu(x.data_ptr(), out.data_ptr(), _DT[x.dtype], x.numel(), _stream(stream)),
           "lowbit_gelu")
    return out


# ---------------------------------------------------------------------------
# Decoding: 4-bit products of a few rows, the 8-bit paged key/value cache and
# attention over it
# ---------------------------------------------------------------------------

def _queue(stream, device: int) -> int:
    """The HIP stream of a call: `stream`, or the current stream of the
    operands' device (taken as a number: a decoding step makes many short
    calls, and the stream object of torch.cuda.current_stream costs 2 us)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"the stream is of GPU {stream.device_index}, the operands are on GPU {device}")
    return stream.cuda_stream


def _same_device(device: int, **operands):
    """The error of operands that are not all GPU tensors of one device."""
    on = ", ".join(f"{n} on {t.device}" for n, t in operands.items() if t.get_device() != device)
    where = f"GPU {device} like the first operand" if device >= 0 else "a GPU"
    return ValueError(f"every operand must be on {where}" + (f"; {on}" if on else ""))


def _new(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """Uninitialised memory for a result written on `stream` (default: the
    current stream): taken from that stream's pool, so that no pending work
    of another stream still uses it."""
    if stream is None:
        return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _dense(t: torch.Tensor, stream) -> torch.Tensor:
    """t itself, or a contiguous copy made on the stream that reads it."""
    if t.is_contiguous():
        return t
    if stream is None:
        return t.contiguous()
    with torch.cuda.stream(stream):
        return t.contiguous()


def gemv_int4(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
              bias: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, activation=None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """gemm_int4 for 1 .. 16 rows of x (lowbit_gemv_int4): one launch that
    reads the codes once, no workspace.

    x: [M, K] fp16/bf16; packed: [N, K/2] uint8; scales, zeros: fp16 [N, K/128]."""
    dev = x.get_device()
    if not 0 <= dev == packed.get_device() == scales.get_device() == zeros.get_device():
        raise _same_device(dev, packed=packed, scales=scales, zeros=zeros)
    if torch._C._cuda_getDevice() != dev:     # the library plans and launches for the current device
        with torch.cuda.device(dev):
            return gemv_int4(x, packed, scales, zeros, bias, out_dtype, activation, out, stream)
    xdt = _DT.get(x.dtype)
    if x.dim() != 2 or (xdt != F16 and xdt != BF16):
        raise ValueError("x must be 2-D float16 or bfloat16 with unit stride along K")
    M, K = x.shape
    ldx, unit = x.stride()
    if unit != 1 and K > 1:
        raise ValueError("x must be 2-D float16 or bfloat16 with unit stride along K")
    N = packed.shape[0]
    packed, scales, zeros = _dense(packed, stream), _dense(scales, stream), _dense(zeros, stream)
    if packed.dtype != torch.uint8 or packed.shape != (N, K // 2):
        raise ValueError(f"packed must be uint8 [{N}, {K // 2}] for K = {K}, got {packed.dtype} {list(packed.shape)}")
    for t, nm in ((scales, "scales"), (zeros, "zeros")):
        if t.dtype != torch.float16 or t.shape != (N, K // GROUP):
            raise ValueError(f"{nm} must be float16 [{N}, {K // GROUP}]")
    bdt = NONE
    if bias is not None:
        if bias.get_device() != dev:
            raise _same_device(dev, bias=bias)
        bias = _dense(bias, stream)
        if bias.numel() != N or bias.dtype not in _DT:
            raise ValueError(f"bias must hold {N} float16, bfloat16 or float32 values")
        bdt = _DT[bias.dtype]
    if out is None:
        out, ldy = _new((M, N), x.dtype if out_dtype is None else out_dtype, x, stream), N
    else:
        if out.get_device() != dev:
            raise _same_device(dev, out=out)
        if out.shape != (M, N) or out.stride(1) != 1 or out.dtype not in _DT:
            raise ValueError(f"out must be [{M}, {N}] with unit stride along N")
        ldy = out.stride(0)
    _check(lib().lowbit_gemv_int4(
        x.data_ptr(), xdt, M, K, ldx if M > 1 else K, packed.data_ptr(), scales.data_ptr(), zeros.data_ptr(),
        GROUP, N, _ptr(bias), bdt, out.data_ptr(), _DT[out.dtype], ldy, _ACT[activation],
        _queue(stream, dev)), "lowbit_gemv_int4")
    return out


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("pages", _I64),
                ("kv_heads", _I32), ("page", _I32), ("head_dim", _I32)]


class KVCache:
    """A paged cache of keys and values in 8 bits (lowbit_kv_cache).

    k, v: uint8 [pages, kv_heads, page, head_dim], contiguous, in the block
    layout of include/lowbit.h; k_scale, v_scale: float32 [pages, kv_heads].
    Made by new_kv_cache, filled by kv_append, read by attention and kv_read.
    It keeps the addresses of its tensors, so these are not assigned anew: a
    larger cache is another KVCache. device: the number of their GPU."""

    __slots__ = ("_tensors", "kv_heads", "page", "head_dim", "device", "struct", "ref")

    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_scale = property(lambda self: self._tensors[2])
    v_scale = property(lambda self: self._tensors[3])

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        shape = k.shape
        if len(shape) != 4 or k.dtype != torch.uint8 or v.dtype != torch.uint8 or v.shape != shape:
            raise ValueError("k and v must be uint8 [pages, kv_heads, page, head_dim] of one shape")
        pages, heads, page, d = shape
        self.kv_heads, self.page, self.head_dim = heads, page, d
        shape = shape[:2]
        if (k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or k_scale.shape != shape
                or v_scale.shape != shape):
            raise ValueError(f"k_scale and v_scale must be float32 [{pages}, {heads}]")
        self.device = dev = k.get_device()
        if not 0 <= dev == v.get_device() == k_scale.get_device() == v_scale.get_device():
            raise _same_device(dev, v=v, k_scale=k_scale, v_scale=v_scale)
        for t in (k, v, k_scale, v_scale):
            if not t.is_contiguous():
                raise ValueError("k, v, k_scale and v_scale must be contiguous")
        self._tensors = (k, v, k_scale, v_scale)
        self.struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                   pages, heads, page, d)
        self.ref = ctypes.byref(self.struct)


def new_kv_cache(pages: int, kv_heads: int, page: int, head_dim: int, device=None) -> KVCache:
    """An empty cache: 2 (page * head_dim + 4) bytes a page and head."""
    dev = torch.device(device or "cuda")
    k, v = (torch.zeros((pages, kv_heads, page, head_dim), dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros((pages, kv_heads), dtype=torch.float32, device=dev) for _ in range(2))
    return KVCache(k, v, ks, vs)


def _table(dev: int, block_table: torch.Tensor, cu: torch.Tensor, start: torch.Tensor, what: str):
    """Arguments that every call on the cache begins with, checked; `dev` is the cache's GPU."""
    if not dev == block_table.get_device() == cu.get_device() == start.get_device():
        raise _same_device(dev, block_table=block_table, cu_tokens=cu, **{what: start})
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 tensor [batch, pages of a sequence]")
    batch, width = block_table.shape
    if cu.dtype != torch.int32 or cu.shape != (batch + 1,) or not cu.is_contiguous():
        raise ValueError(f"cu_tokens must be int32 [{batch + 1}]")
    if start.dtype != torch.int32 or start.shape != (batch,) or not start.is_contiguous():
        raise ValueError(f"{what} must be int32 [{batch}]")
    return block_table.data_ptr(), width, cu.data_ptr(), start.data_ptr(), batch


def _rows3(dev: int, t: torch.Tensor, shape, dtype, name: str):
    ts, hs, unit = t.stride() if t.dim() == 3 else (0, 0, 0)
    if t.get_device() != dev:
        raise _same_device(dev, **{name: t})
    if t.shape != shape or t.dtype != dtype or (unit != 1 and shape[0]):
        raise ValueError(f"{name} must be {dtype} {list(shape)} with unit stride along the last dimension")
    return t.data_ptr(), ts, hs


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, block_table: torch.Tensor, cu_tokens: torch.Tensor,
              starts: torch.Tensor, max_tokens: int, q: Optional[torch.Tensor] = None,
              cos: Optional[torch.Tensor] = None, sin: Optional[torch.Tensor] = None, interleaved: bool = False,
              q_out: Optional[torch.Tensor] = None, bad_count: Optional[torch.Tensor] = None, stream=None):
    """Append new keys and values to the cache, rotated by position on the
    way (lowbit_kv_append); returns the rotated queries when q is given.

    k, v: [T, kv_heads, head_dim] and q: [T, q_heads, head_dim] of one dtype
    (fp16, bf16, fp32), last dimension contiguous (slices of a fused
    projection's output do). Sequence b's rows are cu_tokens[b] ..
    cu_tokens[b+1] - 1 and go to positions starts[b], ...; max_tokens is a
    host bound on the rows of one sequence. cos, sin: float32 [positions,
    rot/2], both or none. bad_count: int32 [2], added to: non-finite values
    (stored as 0) and tokens left out (no page or no position; a query
    without a position comes back as zeros)."""
    if k.dim() != 3:
        raise ValueError("k must be [tokens, kv_heads, head_dim]")
    shape, dtype = k.shape, k.dtype
    T, H, D = shape
    if cache.kv_heads != H or cache.head_dim != D:
        raise ValueError(f"the cache holds {cache.kv_heads} heads of {cache.head_dim}, k has {H} of {D}")
    if dtype not in _DT:
        raise ValueError("k must be float16, bfloat16 or float32")
    dev = cache.device
    if torch._C._cuda_getDevice() != dev:     # the library plans and launches for the current device
        with torch.cuda.device(dev):
            return kv_append(k, v, cache, block_table, cu_tokens, starts, max_tokens, q, cos, sin, interleaved, q_out,
                             bad_count, stream)
    head = _table(dev, block_table, cu_tokens, starts, "starts")
    ka, va = _rows3(dev, k, shape, dtype, "k"), _rows3(dev, v, shape, dtype, "v")
    if q is not None:
        Hq = q.shape[1]
        qa = _rows3(dev, q, (T, Hq, D), dtype, "q")
        if q_out is None:
            q_out = _new((T, Hq, D), dtype, k, stream)
            qo = q_out.data_ptr(), Hq * D, D
        else:
            qo = _rows3(dev, q_out, (T, Hq, D), dtype, "q_out")
    else:
        if q_out is not None:
            raise ValueError("q_out without q")
        Hq, qa, qo = 0, (None, 0, 0), (None, 0, 0)
    rot = positions = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        if cos.dim() != 2 or sin.shape != cos.shape:
            raise ValueError("cos and sin must be [positions, rot/2]")
        for t in (cos, sin):
            if t.get_device() != dev:
                raise _same_device(dev, cos=cos, sin=sin)
            if t.dtype != torch.float32 or not t.is_contiguous():
                raise ValueError("cos and sin must be contiguous float32 tensors")
        positions, rot = cos.shape
        rot *= 2
    if bad_count is not None:
        if bad_count.get_device() != dev:
            raise _same_device(dev, bad_count=bad_count)
        if bad_count.dtype != torch.int32 or bad_count.numel() != 2 or not bad_count.is_contiguous():
            raise ValueError("bad_count must be int32 [2]")
    _check(lib().lowbit_kv_append(cache.ref, *head, T, max_tokens, _DT[dtype], *ka, *va, *qa, Hq, *qo, _ptr(cos),
                                  _ptr(sin), rot, positions, interleaved, _ptr(bad_count),
                                  _queue(stream, dev)), "lowbit_kv_append")
    return q_out


def kv_read(cache: KVCache, block_table: torch.Tensor, cu_tokens: torch.Tensor, starts: torch.Tensor, tokens: int,
            max_tokens: int, dtype: torch.dtype = torch.bfloat16, out=None,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The keys and values that the cache holds for a range of each sequence
    (lowbit_kv_read): rows cu_tokens[b] .. of the two results [tokens,
    kv_heads, head_dim] are sequence b's tokens starts[b], ... `out` = (k, v)
    to write into."""
    if dtype not in _DT:
        raise ValueError("dtype must be float16, bfloat16 or float32")
    H, D = cache.kv_heads, cache.head_dim
    shape = (tokens, H, D)
    dev = cache.device
    if torch._C._cuda_getDevice() != dev:     # the library plans and launches for the current device
        with torch.cuda.device(dev):
            return kv_read(cache, block_table, cu_tokens, starts, tokens, max_tokens, dtype, out, stream)
    head = _table(dev, block_table, cu_tokens, starts, "starts")
    if out is None:
        k, v = _new(shape, dtype, cache.k, stream), _new(shape, dtype, cache.k, stream)
        ka, va = (k.data_ptr(), H * D, D), (v.data_ptr(), H * D, D)
    else:
        k, v = out
        ka, va = _rows3(dev, k, shape, dtype, "k"), _rows3(dev, v, shape, dtype, "v")
    _check(lib().lowbit_kv_read(cache.ref, *head, tokens, max_tokens, _DT[dtype], *ka, *va,
                                _queue(stream, dev)), "lowbit_kv_read")
    return k, v


def attention(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, cu_tokens: torch.Tensor,
              lens: torch.Tensor, max_tokens: int, max_len: int, scale: Optional[float] = None, causal: bool = True,
              window: int = 0, out: Optional[torch.Tensor] = None, return_lse: bool = False,
              workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of new queries over the cache (lowbit_attention).

    q: [T, q_heads, head_dim] fp16/bf16, last dimension contiguous; q_heads a
    multiple of the cache's heads. Sequence b has lens[b] tokens in the cache
    and its queries are rows cu_tokens[b] .. cu_tokens[b+1] - 1, the last ones
    of it. max_tokens and max_len are host bounds on the queries and the length
    of one sequence. scale defaults to head_dim ** -0.5; window > 0 keeps the
    last `window` tokens of each query. Returns out, or (out, lse) with the
    float32 [T, q_heads] log of the softmax's sum."""
    dtype = q.dtype
    if q.dim() != 3 or (dtype != torch.bfloat16 and dtype != torch.float16):
        raise ValueError("q must be float16 or bfloat16 [tokens, q_heads, head_dim]")
    shape = q.shape
    T, Hq, D = shape
    H = cache.kv_heads
    if cache.head_dim != D or Hq % H:
        raise ValueError(f"the cache holds {H} heads of {cache.head_dim}, q has {Hq} of {D}")
    dev = cache.device
    if torch._C._cuda_getDevice() != dev:     # the library plans and launches for the current device
        with torch.cuda.device(dev):
            return attention(q, cache, block_table, cu_tokens, lens, max_tokens, max_len, scale, causal, window, out,
                             return_lse, workspace, stream)
    head = _table(dev, block_table, cu_tokens, lens, "lens")
    qa = _rows3(dev, q, shape, dtype, "q")
    if out is None:
        out = _new(shape, dtype, q, stream)
        oa = out.data_ptr(), Hq * D, D
    else:
        oa = _rows3(dev, out, shape, dtype, "out")
    lse = _new((T, Hq), torch.float32, q, stream) if return_lse else None
    L = lib()
    need = L.lowbit_attention_workspace_bytes(head[4], T, max_tokens, max_len, Hq, H, D, window)
    size = 0
    if workspace is not None:
        size = _given_workspace(workspace, need, "lowbit_attention")
        if workspace.get_device() != dev:
            raise _same_device(dev, workspace=workspace)
    elif need:
        workspace, size = _new(need, torch.uint8, q, stream), need
    _check(L.lowbit_attention(cache.ref, *head, T, max_tokens, max_len, _DT[dtype], *qa, Hq, *oa, _ptr(lse),
                              D ** -0.5 if scale is None else scale, causal, window, _ptr(workspace), size,
                              _queue(stream, dev)), "lowbit_attention")
    return (out, lse) if return_lse else out
