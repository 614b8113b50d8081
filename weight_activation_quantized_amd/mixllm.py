"""Thin Python binding of libmixllm.so (C ABI in include/mixllm.h).

Argument marshalling only: every step of the layer runs in the library (host packer in
C++, activation quantization and the mixed GEMM in HIP kernels).  PyTorch supplies
device memory and the HIP stream.  The functions carry the C names; a non-zero status
raises ``MixLLMError``.  Importing this module fails loudly when the library is missing.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

try:  # torch first: its HIP runtime must be the one the library binds to
    import torch
except ImportError:  # pragma: no cover - host-only use of the packer
    torch = None

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("MIXLLM_LIB") or os.path.join(HERE, "libmixllm.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "mixllm.h")
GROUP = 128

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m weight_activation_quantized_amd.build` "
        "(there is no fallback implementation)")

_lib = ctypes.CDLL(LIB_PATH, mode=ctypes.RTLD_GLOBAL)
_variants = {}


def hip_runtimes_loaded():
    """Distinct libamdhip64 files mapped into this process."""
    paths = set()
    with open("/proc/self/maps") as f:
        for line in f:
            parts = line.split()
            if len(parts) >= 6 and "libamdhip64" in parts[-1]:
                paths.add(os.path.realpath(parts[-1]))
    return paths


_runtimes = hip_runtimes_loaded()
if len(_runtimes) > 1:
    raise ImportError(f"two HIP runtimes are loaded into one process: {sorted(_runtimes)}")


class BlobInfo(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
                ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("group", ctypes.c_int32),
                ("n8", ctypes.c_int32), ("n4", ctypes.c_int32), ("G", ctypes.c_int32),
                ("nb", ctypes.c_int32), ("nb4", ctypes.c_int32), ("nb8", ctypes.c_int32),
                ("n4_promoted", ctypes.c_int32),
                ("off_w4", ctypes.c_uint64), ("off_s4", ctypes.c_uint64), ("off_z4", ctypes.c_uint64),
                ("off_w8", ctypes.c_uint64), ("off_s8", ctypes.c_uint64), ("off_zp", ctypes.c_uint64),
                ("off_idx", ctypes.c_uint64), ("total_bytes", ctypes.c_uint64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


_vp, _i32, _i64, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_SIGS = {
    "mixllm_status_str": ([ctypes.c_int], ctypes.c_char_p),
    "mixllm_packed_bytes": ([_i32, _i32, _i32, _i32], _sz),
    "mixllm_pack_weights": ([_vp, _i32, _i32, _i32, _vp, _i32, _vp, _sz], ctypes.c_int),
    "mixllm_blob_get_info": ([_vp, _sz, ctypes.POINTER(BlobInfo)], ctypes.c_int),
    "mixllm_unpack_weights": ([_vp, _sz, _vp, _vp, _vp, _vp], ctypes.c_int),
    "mixllm_channel_salience": ([_vp, _vp, _i32, _i32, _i32, _i32, _vp], ctypes.c_int),
    "mixllm_assign_channels": ([_vp, _vp, _i32, _i64, _vp, _vp], ctypes.c_int),
    "mixllm_quant_act": ([_vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "mixllm_silu_mul_quant": ([_vp, _vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
    "mixllm_gemm_workspace_bytes": ([_i32, _i32, _i32, _i32], _sz),
    "mixllm_gemm_w4w8a8": ([_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _sz, _vp, _i64, _vp, _sz,
                            _vp], ctypes.c_int),
    "mixllm_gemm_w4w8a8_partials": ([_vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _sz, _i32, _i32,
                                     _vp, _vp], ctypes.c_int),
    "mixllm_residual_norm": ([_vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _i32,
                              _i32, _i32, _i32, _i32, _f32, _f32, _f32, _vp], ctypes.c_int),
    "mixllm_kv4_page_bytes": ([_i32, _i32, _i32], _sz),
    "mixllm_kv_plan": ([_vp, _vp, _i32, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i32,
                        _vp], ctypes.c_int),
    "mixllm_kv4_append": ([_vp, _i64, _vp, _i64, _i32, _vp, _i32, _vp, _sz, _i32, _i32, _i32, _i32, _vp],
                          ctypes.c_int),
    "mixllm_kv4_read": ([_vp, _sz, _i32, _i32, _i32, _i32, _vp, _i32, _vp, _i64, _vp, _i64, _i32, _vp], ctypes.c_int),
    "mixllm_kv4_attention_workspace_bytes": ([_i32] * 8, _sz),
    "mixllm_kv4_attention": ([_vp, _i64, _i32, _i32, _i32, _vp, _sz, _i32, _i32, _i32, _i32, _vp, _i64, _i32, _vp, _vp,
                              _i32, _i32, _i32, _f32, _i32, _vp, _i64, _vp, _vp, _sz, _vp], ctypes.c_int),
}
def _bind(lib):
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_bind(_lib)


def load_variant(name: str):
    """A measured variant of the library (libmixllm_<name>.so, built by
    ``python -m weight_activation_quantized_amd.build --variants``), loaded beside the
    main one with its symbols kept local.  Pass it as ``lib=`` to the device calls."""
    if name not in _variants:
        path = os.path.join(HERE, f"libmixllm_{name}.so")
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: build it with "
                              "`python -m weight_activation_quantized_amd.build --variants`")
        _variants[name] = _bind(ctypes.CDLL(path, mode=ctypes.RTLD_LOCAL))
    return _variants[name]

STATUS = {0: "MIXLLM_OK", -1: "MIXLLM_E_NULL", -2: "MIXLLM_E_SHAPE", -3: "MIXLLM_E_GROUP",
          -4: "MIXLLM_E_INDEX", -5: "MIXLLM_E_SPACE", -6: "MIXLLM_E_FORMAT", -7: "MIXLLM_E_HIP"}


class MixLLMError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(mixllm_status_str(status))


def _check(status: int) -> None:
    if status != 0:
        raise MixLLMError(status)


def exported_symbols():
    """Function names declared in include/mixllm.h."""
    import re
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"\b(mixllm_[a-z0-9_]+)\s*\(", text)))


def library_handle():
    return _lib


# ---------------------------------------------------------------------------- host calls

def mixllm_status_str(status: int) -> str:
    return _lib.mixllm_status_str(int(status)).decode()


def mixllm_packed_bytes(n: int, k: int, group: int = GROUP, n8: int = 0) -> int:
    return int(_lib.mixllm_packed_bytes(n, k, group, n8))


def mixllm_pack_weights(w_fp16: np.ndarray, idx8, group: int = GROUP) -> np.ndarray:
    """Packs an fp16 [N, K] weight matrix; returns the blob as a uint8 numpy array."""
    w = np.ascontiguousarray(w_fp16, dtype=np.float16)
    n, k = w.shape
    idx = np.ascontiguousarray(np.asarray(idx8, dtype=np.int32).reshape(-1))
    size = mixllm_packed_bytes(n, k, group, int(idx.size))
    blob = np.zeros(max(size, 1), dtype=np.uint8)
    _check(_lib.mixllm_pack_weights(w.ctypes.data, n, k, group,
                                    idx.ctypes.data if idx.size else None, int(idx.size),
                                    blob.ctypes.data, blob.size if size else 0))
    return blob


def blob_header(blob: np.ndarray) -> BlobInfo:
    """The checked header of a host blob (mixllm_blob_get_info), as the C struct the GEMM
    calls take."""
    b = np.ascontiguousarray(blob, dtype=np.uint8)
    info = BlobInfo()
    _check(_lib.mixllm_blob_get_info(b.ctypes.data, b.size, ctypes.byref(info)))
    return info


def mixllm_blob_get_info(blob: np.ndarray) -> dict:
    return blob_header(blob).as_dict()


def mixllm_unpack_weights(blob: np.ndarray):
    """Returns (q uint8 [N, K], z uint8 [N, G], s fp16 [N, G], is8 bool [N])."""
    info = mixllm_blob_get_info(blob)
    n, k, g = info["N"], info["K"], info["G"]
    b = np.ascontiguousarray(blob, dtype=np.uint8)
    q = np.zeros((n, k), np.uint8)
    z = np.zeros((n, g), np.uint8)
    s = np.zeros((n, g), np.uint16)
    is8 = np.zeros(n, np.uint8)
    _check(_lib.mixllm_unpack_weights(b.ctypes.data, b.size, q.ctypes.data, z.ctypes.data,
                                      s.ctypes.data, is8.ctypes.data))
    return q, z, s.view(np.float16), is8.astype(bool)


def mixllm_channel_salience(w_fp16: np.ndarray, grads: np.ndarray, group: int = GROUP) -> np.ndarray:
    """w_fp16: [N, K] fp16; grads: [D, N, K] fp32.  Returns the fp64 salience of each channel."""
    w = np.ascontiguousarray(w_fp16, dtype=np.float16)
    g = np.ascontiguousarray(grads, dtype=np.float32)
    n, k = w.shape
    if g.ndim != 3 or g.shape[1:] != (n, k):
        raise ValueError("grads must be [D, N, K]")
    out = np.zeros(n, np.float64)
    _check(_lib.mixllm_channel_salience(w.ctypes.data, g.ctypes.data, n, k, group, g.shape[0], out.ctypes.data))
    return out


def mixllm_assign_channels(scores, total_8bit: int):
    """scores: list of per-layer fp64 arrays.  Returns the per-layer idx8 arrays (int32,
    ascending) of the global top-``total_8bit`` channels."""
    per = [np.ascontiguousarray(s, dtype=np.float64).reshape(-1) for s in scores]
    flat = np.ascontiguousarray(np.concatenate(per)) if per else np.zeros(0)
    sizes = np.array([len(s) for s in per], np.int32)
    idx = np.zeros(max(int(total_8bit), 1), np.int32)
    n8 = np.zeros(max(len(per), 1), np.int32)
    _check(_lib.mixllm_assign_channels(flat.ctypes.data, sizes.ctypes.data, len(per), int(total_8bit),
                                       idx.ctypes.data, n8.ctypes.data))
    out, o = [], 0
    for c in n8[:len(per)]:
        out.append(idx[o:o + c].copy())
        o += int(c)
    return out


# ---------------------------------------------------------------------------- device calls

def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def mixllm_quant_act(a, aq, sa, asum=None, rowop=None, stream=None, lib=None):
    """a: fp16 [M, K] CUDA tensor (rows may be strided); aq: int8 [M, K];
    sa: fp32 [G, M]; asum: int32 [G, M] or None; rowop: 32-bit [G, M, 8] or None."""
    m, k = a.shape
    if a.dtype != torch.float16 or a.stride(1) != 1 or not a.is_cuda:
        raise ValueError("a must be an fp16 CUDA tensor with unit column stride")
    if m:
        g = k // GROUP
        _need(aq, "aq", torch.int8, (m, k))
        _need(sa, "sa", torch.float32, (g, m))
        if asum is not None:
            _need(asum, "asum", torch.int32, (g, m))
        if rowop is not None:
            _need(rowop, "rowop", torch.int32, (g, m, 8))
    lda = a.stride(0) if m > 1 else k
    _check((lib or _lib).mixllm_quant_act(_ptr(a), lda, m, k, GROUP, _ptr(aq), _ptr(sa), _ptr(asum),
                                          _ptr(rowop), _stream(stream)))


def mixllm_silu_mul_quant(gate, up, aq, sa, asum=None, rowop=None, h=None, stream=None, lib=None):
    """gate, up: fp16 [M, I] CUDA views with the same row stride (e.g. the two halves of a
    [M, 2I] GEMM output); outputs as mixllm_quant_act with K = I; h: fp16 [M, I] or None."""
    m, inter = gate.shape
    if gate.dtype != torch.float16 or up.dtype != torch.float16 or gate.stride(1) != 1 or up.stride(1) != 1:
        raise ValueError("gate and up must be fp16 with unit column stride")
    if up.shape != gate.shape or (m > 1 and up.stride(0) != gate.stride(0)):
        raise ValueError("gate and up must have the same shape and row stride")
    if m:
        g = inter // GROUP
        _need(aq, "aq", torch.int8, (m, inter))
        _need(sa, "sa", torch.float32, (g, m))
        if asum is not None:
            _need(asum, "asum", torch.int32, (g, m))
        if rowop is not None:
            _need(rowop, "rowop", torch.int32, (g, m, 8))
        if h is not None:
            _need(h, "h", torch.float16, (m, inter))
    ld = gate.stride(0) if m > 1 else inter
    _check((lib or _lib).mixllm_silu_mul_quant(_ptr(gate), _ptr(up), ld, m, inter, GROUP, _ptr(aq), _ptr(sa),
                                               _ptr(asum), _ptr(rowop), _ptr(h), _stream(stream)))


def mixllm_gemm_workspace_bytes(m: int, n: int, k: int, n8: int) -> int:
    return int(_lib.mixllm_gemm_workspace_bytes(m, n, k, n8))


class DeviceBlob:
    """A packed blob on the GPU with the host copy of its header (the GEMM calls check
    the header against the layer they are asked to compute)."""

    def __init__(self, blob_host: np.ndarray, device="cuda"):
        self.info = blob_header(blob_host)
        self.dev = torch.from_numpy(np.ascontiguousarray(blob_host, dtype=np.uint8)).to(device)
        self.nbytes = int(self.dev.numel())


def _need(t, name, dtype, shape=None, what=""):
    """Argument checks before a device call: a CUDA tensor of this dtype whose shape
    covers `shape` and whose innermost stride is 1."""
    if t is None:
        raise ValueError(f"{name} is required{what}")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit innermost stride")
    if shape is not None:
        if t.dim() != len(shape) or any(a < b for a, b in zip(t.shape, shape)):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, needs at least {tuple(shape)}")
        if not t.is_contiguous() and name != "y":
            raise ValueError(f"{name} must be contiguous")


def _gemm_inputs(aq, sa, asum, rowop, m, k, nb4):
    g = k // GROUP
    _need(aq, "aq", torch.int8, (m, k))
    _need(sa, "sa", torch.float32, (g, m))
    if asum is not None or nb4 > 0:
        _need(asum, "asum", torch.int32, (g, m), " for layers with 4-bit blocks")
    _need(rowop, "rowop", torch.int32, (g, m, 8))
    for t, name, shape in ((aq, "aq", (m, k)), (sa, "sa", (g, m)), (asum, "asum", (g, m)),
                           (rowop, "rowop", (g, m, 8))):
        if t is not None and m and tuple(t.shape) != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _blob(blob):
    if not isinstance(blob, DeviceBlob):
        raise ValueError("blob must be a DeviceBlob (the device copy plus its host header)")
    return blob


def mixllm_gemm_w4w8a8(aq, sa, asum, rowop, m: int, n: int, k: int, n8: int, blob, y, workspace=None,
                       stream=None, lib=None):
    """aq, sa, asum, rowop: outputs of mixllm_quant_act; y: fp16 [M, ldy] CUDA tensor (ldy >= N);
    blob: DeviceBlob of the packed layer."""
    b = _blob(blob)
    if m:
        _gemm_inputs(aq, sa, asum, rowop, m, k, b.info.nb4)
        _need(y, "y", torch.float16, (m, n))
        if y.dim() != 2:
            raise ValueError("y must be 2-D")
    ldy = y.stride(0) if y is not None and y.dim() == 2 and m > 1 else n
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check((lib or _lib).mixllm_gemm_w4w8a8(_ptr(aq), _ptr(sa), _ptr(asum), _ptr(rowop), m, n, k, n8,
                                            ctypes.byref(b.info), _ptr(b.dev), b.nbytes, _ptr(y), ldy,
                                            _ptr(workspace), ws, _stream(stream)))


def mixllm_gemm_w4w8a8_partials(aq, sa, asum, rowop, m: int, n: int, k: int, n8: int, blob, n_begin: int,
                                n_count: int, part, stream=None, lib=None):
    """part: int32 [M, n_count, G] CUDA tensor."""
    b = _blob(blob)
    if m and n_count:
        _gemm_inputs(aq, sa, asum, rowop, m, k, b.info.nb4)
        _need(part, "part", torch.int32, (m, n_count, k // GROUP))
        if not part.is_contiguous():
            raise ValueError("part must be contiguous")
    _check((lib or _lib).mixllm_gemm_w4w8a8_partials(_ptr(aq), _ptr(sa), _ptr(asum), _ptr(rowop), m, n, k, n8,
                                                     ctypes.byref(b.info), _ptr(b.dev), b.nbytes, n_begin,
                                                     n_count, _ptr(part), _stream(stream)))


# ------------------------------------------------------------- between the packed layers

FP16, BF16, FP32 = 0, 1, 2  # MIXLLM_FP16, MIXLLM_BF16, MIXLLM_FP32


def _type16(t, name):
    """The library's number of a 16-bit element type."""
    if t.dtype is torch.float16:
        return FP16
    if t.dtype is torch.bfloat16:
        return BF16
    raise ValueError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")


def _rows(t, name, dtype, shape):
    """The row stride of a [M, N] (or [M, heads, dim]) CUDA tensor with contiguous rows."""
    if not t.is_cuda or t.dtype is not dtype:
        raise ValueError(f"{name} must be a CUDA tensor of {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    st = t.stride()
    if len(shape) == 2:
        width = shape[1]
        whole = st[1] == 1 or width == 1
    else:
        width = shape[1] * shape[2]
        whole = st[2] == 1 and (st[1] == shape[2] or shape[1] == 1)
    if not whole:
        raise ValueError(f"{name} must have contiguous rows")
    if shape[0] <= 1:
        return (width + 7) // 8 * 8
    if st[0] < width:
        raise ValueError(f"the rows of {name} overlap")
    return st[0]


def _ints(t, name, numel):
    """An int32 CUDA tensor, contiguous, of at least `numel` elements."""
    if not t.is_cuda or t.dtype is not torch.int32 or not t.is_contiguous() or t.numel() < numel:
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor of at least {numel} elements")
    return t


def _launch(fn, tensors, stream, *args):
    """Calls a device entry point with the stream last, on the device of its tensors."""
    dev = tensors[0].device
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError(f"the tensors are on different devices: {dev} and {t.device}")
    if dev.index == torch.cuda.current_device():
        _check(fn(*args, _stream(stream)))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, _stream(stream)))


def _at(t):
    return None if t is None else t.data_ptr()


def mixllm_residual_norm(x, res, pre_weight, res_out=None, y=None, aq=None, sa=None, asum=None, rowop=None,
                         post_weight=None, gate=None, alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-5,
                         stream=None):
    """h' = alpha res + beta gate * norm(x; post_weight), y = norm(h'; pre_weight).  x: [M, N]
    fp16 or bf16 (None: no block before); res, res_out: [M, N] of that type or fp32 (res_out
    may be res); gate: [N], [M, N] or None; y: [M, N] in 16 bits; aq, sa, asum, rowop as
    mixllm_quant_act's outputs for y."""
    lead = x if x is not None else pre_weight
    if lead is None:
        raise ValueError("x or pre_weight is required")
    dtype = _type16(lead, "x" if x is not None else "pre_weight")
    shape = res.shape
    if len(shape) != 2:
        raise ValueError("res must be 2-D")
    m, n = shape
    t16 = lead.dtype
    res_dtype = FP32 if res.dtype is torch.float32 else dtype
    ldr = _rows(res, "res", torch.float32 if res_dtype == FP32 else t16, shape)
    ldx = _rows(x, "x", t16, shape) if x is not None else 0
    ldro = _rows(res_out, "res_out", res.dtype, shape) if res_out is not None else 0
    ldy = _rows(y, "y", t16, shape) if y is not None else 0
    ldgate = 0
    if gate is not None:
        if gate.dim() == 2:
            ldgate = _rows(gate, "gate", t16, shape)
        else:
            _rows(gate.view(1, -1), "gate", t16, (1, n))
    for w, name in ((post_weight, "post_weight"), (pre_weight, "pre_weight")):
        if w is not None and (not w.is_cuda or w.dtype is not t16 or w.shape != (n,) or w.stride(0) != 1):
            raise ValueError(f"{name} must be a contiguous [{n}] CUDA tensor of {t16}")
    if aq is not None and m:
        g = n // GROUP
        _need(aq, "aq", torch.int8, (m, n))
        _need(sa, "sa", torch.float32, (g, m))
        if asum is not None:
            _need(asum, "asum", torch.int32, (g, m))
        if rowop is not None:
            _need(rowop, "rowop", torch.int32, (g, m, 8))
        if aq.shape != (m, n) or sa.shape != (g, m):
            raise ValueError(f"aq and sa must be [{m}, {n}] and [{g}, {m}]")
    _launch(_lib.mixllm_residual_norm, (res, x, res_out, pre_weight, post_weight, gate, y, aq, sa, asum, rowop), stream,
            _at(x), ldx, _at(post_weight), _at(gate), ldgate, _at(res), ldr, _at(res_out), ldro, _at(pre_weight),
            _at(y), ldy, _at(aq), _at(sa), _at(asum), _at(rowop), m, n, GROUP, dtype, res_dtype, eps, alpha, beta)


def mixllm_kv4_page_bytes(page: int, heads: int, dim: int) -> int:
    return int(_lib.mixllm_kv4_page_bytes(page, heads, dim))


def kv4_cache(pages: int, page: int, heads: int, dim: int, device="cuda"):
    """Storage of one layer's cache: uint8 [pages, heads, bytes of a (page, head) block]."""
    size = mixllm_kv4_page_bytes(page, heads, dim)
    if not size or pages <= 0:
        raise ValueError("pages and heads must be positive, page a power of two of 16 .. 1024, dim 64, 128 or 256")
    return torch.empty((pages, heads, size // heads), dtype=torch.uint8, device=device)


def _cache(cache, page, dim):
    """(bytes, pages, heads) of a cache tensor for pages of `page` tokens and heads of `dim` channels."""
    if not cache.is_cuda or cache.dtype is not torch.uint8 or cache.dim() != 3 or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous uint8 CUDA tensor [pages, heads, block bytes]")
    pages, heads, block = cache.shape
    if block * 8 != page * dim * 9:
        raise ValueError(f"cache has blocks of {block} bytes, page {page} and dim {dim} need {page * dim * 9 / 8:g}")
    return pages * heads * block, pages, heads


def mixllm_kv_plan(fresh, lens, table, pool, count, page: int, pages: int, lens_out, count_out, cu, slots, pos,
                   stream=None):
    """The page tables and slot maps of a step from request lengths, on the GPU: fresh, lens,
    lens_out: int32 [B]; table: int32 [B, width] (rows may be strided); pool: int32 [F]; count:
    int32 [1 or more]; count_out: int32 [2]; cu: int32 [B + 1]; slots, pos: int32 [tokens]."""
    b = fresh.shape[0]
    if table.dim() != 2 or table.shape[0] != b or not table.is_cuda or table.dtype is not torch.int32 or (
            table.numel() and table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"table must be an int32 CUDA tensor [{b}, width] with contiguous rows")
    width = table.shape[1]
    for t, name, size in ((fresh, "fresh", b), (lens, "lens", b), (count, "count", 1), (lens_out, "lens_out", b),
                          (count_out, "count_out", 2), (cu, "cu", b + 1), (pool, "pool", 0),
                          (pos, "pos", slots.shape[0]), (slots, "slots", 0)):
        _ints(t, name, size)
    if b > 1 and table.stride(0) < width:
        raise ValueError("the rows of table overlap")
    _launch(_lib.mixllm_kv_plan, (fresh, lens, table, pool, count, lens_out, count_out, cu, slots, pos), stream,
            fresh.data_ptr(), lens.data_ptr(), b, table.data_ptr(), table.stride(0) if b > 1 else width, width,
            pool.data_ptr(), pool.numel(), count.data_ptr(), page, pages, lens_out.data_ptr(), count_out.data_ptr(),
            cu.data_ptr(), slots.data_ptr(), pos.data_ptr(), slots.shape[0])


def mixllm_kv4_append(k, v, slots, cache, page: int, stream=None):
    """Writes k and v ([T, heads, dim] fp16 or bf16, rows may be strided) into the cache at
    slots (int32 [T], negative: skip the row)."""
    t, _, dim = k.shape
    size, pages, heads = _cache(cache, page, dim)
    dtype, shape = _type16(k, "k"), (t, heads, dim)
    ldk, ldv = _rows(k, "k", k.dtype, shape), _rows(v, "v", k.dtype, shape)
    _ints(slots, "slots", t)
    _launch(_lib.mixllm_kv4_append, (cache, k, v, slots), stream, k.data_ptr(), ldk, v.data_ptr(), ldv, dtype,
            slots.data_ptr(), t, cache.data_ptr(), size, pages, page, heads, dim)


def mixllm_kv4_read(cache, slots, k, v, page: int, stream=None):
    """The values of the tokens at slots (int32 [T]) into k and v ([T, heads, dim] fp16 or
    bf16); rows with a negative slot are left as they were."""
    t, _, dim = k.shape
    size, pages, heads = _cache(cache, page, dim)
    dtype, shape = _type16(k, "k"), (t, heads, dim)
    ldk, ldv = _rows(k, "k", k.dtype, shape), _rows(v, "v", k.dtype, shape)
    _ints(slots, "slots", t)
    _launch(_lib.mixllm_kv4_read, (cache, k, v, slots), stream, cache.data_ptr(), size, pages, page, heads, dim,
            slots.data_ptr(), t, k.data_ptr(), ldk, v.data_ptr(), ldv, dtype)


def mixllm_kv4_attention_workspace_bytes(t: int, b: int, q_heads: int, kv_heads: int, dim: int, max_rows: int,
                                         max_len: int, window: int = 0) -> int:
    return int(_lib.mixllm_kv4_attention_workspace_bytes(t, b, q_heads, kv_heads, dim, max_rows, max_len, window))


def mixllm_kv4_attention(q, cache, table, lens, cu, out, page: int, max_rows: int, max_len: int, scale=None,
                         window: int = 0, lse=None, workspace=None, stream=None):
    """Attention of the rows q ([T, q_heads, dim] fp16 or bf16) of B requests over the cache:
    table: int32 [B, width]; lens: int32 [B] tokens cached (these rows' among them); cu: int32
    [B + 1] first row of each request; out: as q; lse: fp32 [T, q_heads] or None; scale: 1 /
    sqrt(dim) by default; workspace: a uint8 tensor of mixllm_kv4_attention_workspace_bytes(T,
    B, ..) for the same arguments (None where that is 0)."""
    t, hq, dim = q.shape
    size, pages, heads = _cache(cache, page, dim)
    dtype = _type16(q, "q")
    ldq, ldo = _rows(q, "q", q.dtype, q.shape), _rows(out, "out", q.dtype, q.shape)
    b = lens.shape[0]
    if table.dim() != 2 or table.shape[0] < b or not table.is_cuda or table.dtype is not torch.int32 or (
            table.numel() and table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"table must be an int32 CUDA tensor [{b}, width] with contiguous rows")
    _ints(lens, "lens", b)
    _ints(cu, "cu", b + 1)
    width = table.shape[1]
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (t, hq) or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous fp32 tensor [{t}, {hq}]")
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _launch(_lib.mixllm_kv4_attention, (q, cache, table, lens, cu, out, lse, workspace), stream, q.data_ptr(), ldq,
            dtype, t, hq, cache.data_ptr(), size, pages, page, heads, dim, table.data_ptr(),
            table.stride(0) if table.shape[0] > 1 else width, width, lens.data_ptr(), cu.data_ptr(), b, max_rows,
            max_len, dim ** -0.5 if scale is None else scale, window, out.data_ptr(), ldo, _at(lse), _at(workspace), ws)


def rowop_buffer(m: int, k: int, device="cuda"):
    """Storage for mixllm_quant_act's row operands: 32-bit words [G, M, 8]."""
    return torch.empty((k // GROUP, m, 8), dtype=torch.int32, device=device)


# ---------------------------------------------------------------------------- convenience

class PackedLinear:
    """A packed layer resident on the GPU plus the buffers one forward pass needs.

    ``forward(a)`` runs the hot path: mixllm_quant_act then mixllm_gemm_w4w8a8.
    """

    def __init__(self, w_fp16: np.ndarray, idx8, device="cuda"):
        self.n, self.k = w_fp16.shape
        self.n8 = int(np.asarray(idx8).size)
        self.g = self.k // GROUP
        self.blob_host = mixllm_pack_weights(w_fp16, idx8)
        self.blob = DeviceBlob(self.blob_host, device)
        self.device = device

    def buffers(self, m: int):
        dev = self.device
        return dict(aq=torch.empty((m, self.k), dtype=torch.int8, device=dev),
                    sa=torch.empty((self.g, m), dtype=torch.float32, device=dev),
                    asum=torch.empty((self.g, m), dtype=torch.int32, device=dev),
                    rowop=rowop_buffer(m, self.k, dev),
                    y=torch.empty((m, self.n), dtype=torch.float16, device=dev),
                    ws=self._workspace(m))

    def _workspace(self, m):
        nbytes = mixllm_gemm_workspace_bytes(m, self.n, self.k, self.n8)
        return torch.zeros(nbytes, dtype=torch.uint8, device=self.device) if nbytes else None

    def forward(self, a, bufs=None, stream=None):
        m = a.shape[0]
        bufs = bufs or self.buffers(m)
        mixllm_quant_act(a, bufs["aq"], bufs["sa"], bufs["asum"], bufs["rowop"], stream)
        mixllm_gemm_w4w8a8(bufs["aq"], bufs["sa"], bufs["asum"], bufs["rowop"], m, self.n, self.k, self.n8,
                           self.blob, bufs["y"], bufs["ws"], stream)
        return bufs["y"]


def concat_layers(weights, idx8s):
    """Several layers over the same input as one: their fp16 weights stacked along the output
    channels, each layer's 8-bit channel indices shifted to its rows.  Returns (w, idx8,
    bounds), bounds[i] = the output columns (begin, end) of layer i."""
    ws = [np.asarray(w, np.float16) for w in weights]
    if len({w.shape[1] for w in ws}) != 1:
        raise ValueError("the layers must share the input width")
    offs = np.cumsum([0] + [w.shape[0] for w in ws])
    idx = np.concatenate([np.asarray(i, np.int32).reshape(-1) + np.int32(o) for i, o in zip(idx8s, offs[:-1])])
    return np.concatenate(ws), idx, [(int(offs[i]), int(offs[i + 1])) for i in range(len(ws))]


class QKVProjection:
    """The attention input projections of one hidden state: q, k and v packed together as
    one layer (their output channels concatenated, each keeping its own 8-bit channels),
    so one activation quantization and one GEMM launch produce all three.  ``forward``
    returns views of the one output.  Argument marshalling only."""

    def __init__(self, w_q, w_k, w_v, idx8_q, idx8_k, idx8_v, device="cuda"):
        w, idx, self.bounds = concat_layers((w_q, w_k, w_v), (idx8_q, idx8_k, idx8_v))
        self.layer = PackedLinear(w, idx, device)
        self.device = device

    def buffers(self, m: int):
        return self.layer.buffers(m)

    def split(self, y):
        return tuple(y[:, a:b] for a, b in self.bounds)

    def forward(self, x, bufs, stream=None):
        return self.split(self.layer.forward(x, bufs, stream))

    def capture(self, x, bufs):
        """A HIP graph of one forward pass on these buffers (torch.cuda.CUDAGraph)."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.forward(x, bufs, s)  # warm-up outside the capture
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            self.forward(x, bufs, s)
        return g


class MLPBlock:
    """The Llama MLP block on the packed layers: one activation quantization feeds one GEMM
    over the gate and up channels (packed together as one layer of 2I channels), the fused
    SiLU(gate) * up + quantization feeds the down projection.  Four launches on one stream;
    ``capture`` records them in a HIP graph.  Argument marshalling only."""

    def __init__(self, w_gate, w_up, w_down, idx8_gate, idx8_up, idx8_down, device="cuda"):
        self.inter, self.hidden = np.asarray(w_gate).shape
        w_gu, idx_gu, _ = concat_layers((w_gate, w_up), (idx8_gate, idx8_up))
        self.gu = PackedLinear(w_gu, idx_gu, device)
        self.down = PackedLinear(np.asarray(w_down, np.float16), idx8_down, device)
        self.device = device

    def buffers(self, m: int):
        dev = self.device
        return dict(x=self.gu.buffers(m), h=self.down.buffers(m),
                    h16=torch.empty((m, self.inter), dtype=torch.float16, device=dev))

    def forward(self, x, bufs, stream=None, keep_h=False):
        m = x.shape[0]
        bx, bh = bufs["x"], bufs["h"]
        self.gu.forward(x, bx, stream)
        gu = bx["y"]
        mixllm_silu_mul_quant(gu[:, :self.inter], gu[:, self.inter:], bh["aq"], bh["sa"], bh["asum"], bh["rowop"],
                              bufs["h16"] if keep_h else None, stream)
        mixllm_gemm_w4w8a8(bh["aq"], bh["sa"], bh["asum"], bh["rowop"], m, self.down.n, self.down.k,
                           self.down.n8, self.down.blob, bh["y"], bh["ws"], stream)
        return bh["y"]

    def capture(self, x, bufs, keep_h=False):
        """A HIP graph of one forward pass on these buffers (torch.cuda.CUDAGraph)."""
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            self.forward(x, bufs, s, keep_h)  # warm-up outside the capture
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            self.forward(x, bufs, s, keep_h)
        return g
