"""Thin Python binding of libmixllm.so (C ABI in include/mixllm.h).

Argument marshalling only: every step of the layer runs in the library (host packer in
C++, activation quantization and the mixed GEMM in HIP kernels).  PyTorch supplies
device memory and the HIP stream.  The functions carry the C names; a non-zero status
raises ``MixLLMError``.  Importing this module fails loudly when the library is missing.
"""
from __future__ import annotations

import contextlib
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
    "mixllm_kv_plan_fit": ([_vp, _vp, _i32, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i32,
                            _vp], ctypes.c_int),
    "mixllm_kv4_append": ([_vp, _i64, _vp, _i64, _i32, _vp, _i32, _vp, _sz, _i32, _i32, _i32, _i32, _vp],
                          ctypes.c_int),
    "mixllm_kv4_read": ([_vp, _sz, _i32, _i32, _i32, _i32, _vp, _i32, _vp, _i64, _vp, _i64, _i32, _vp], ctypes.c_int),
    "mixllm_kv4_attention_workspace_bytes": ([_i32] * 8, _sz),
    "mixllm_kv4_attention": ([_vp, _i64, _i32, _i32, _i32, _vp, _sz, _i32, _i32, _i32, _i32, _vp, _i64, _i32, _vp, _vp,
                              _i32, _i32, _i32, _f32, _i32, _vp, _i64, _vp, _vp, _sz, _vp], ctypes.c_int),
    "mixllm_head_norm_rotate": ([_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                 _i32, _i32, _i32, _f32, _vp], ctypes.c_int),
    "mixllm_quant_rows": ([_vp, _i64, _i32, _i32, _i32, _vp, _i64, _vp, _vp], ctypes.c_int),
    "mixllm_gemm_w8a8": ([_vp, _i64, _vp, _vp, _i64, _vp, _i32, _i32, _i32, _vp, _i64, _i32, _vp], ctypes.c_int),
}
for _call in ("page_bytes", "append", "read", "attention_workspace_bytes", "attention"):  # the caches' calls are alike
    _SIGS[f"mixllm_kv8_{_call}"] = _SIGS[f"mixllm_kv4_{_call}"]
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

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def mixllm_quant_act(a, aq, sa, asum=None, rowop=None, stream=None, lib=None):
    """a: fp16 [M, K] CUDA tensor (rows may be strided); aq: int8 [M, K];
    sa: fp32 [G, M]; asum: int32 [G, M] or None; rowop: 32-bit [G, M, 8] or None."""
    m, k = a.shape
    if a.dtype != torch.float16 or a.stride(1) != 1:
        raise ValueError("a must be an fp16 CUDA tensor with unit column stride")
    dev = _gpu(a, "a")
    if m:
        g = k // GROUP
        _need(aq, "aq", torch.int8, (m, k))
        _need(sa, "sa", torch.float32, (g, m))
        if asum is not None:
            _need(asum, "asum", torch.int32, (g, m))
        if rowop is not None:
            _need(rowop, "rowop", torch.int32, (g, m, 8))
    lda = a.stride(0) if m > 1 else k
    _on(dev, stream, (lib or _lib).mixllm_quant_act, _ptr(a), lda, m, k, GROUP, _ptr(aq), _ptr(sa), _ptr(asum),
        _ptr(rowop))


def mixllm_silu_mul_quant(gate, up, aq, sa, asum=None, rowop=None, h=None, stream=None, lib=None):
    """gate, up: fp16 [M, I] CUDA views with the same row stride (e.g. the two halves of a
    [M, 2I] GEMM output); outputs as mixllm_quant_act with K = I; h: fp16 [M, I] or None."""
    m, inter = gate.shape
    if gate.dtype != torch.float16 or up.dtype != torch.float16 or gate.stride(1) != 1 or up.stride(1) != 1:
        raise ValueError("gate and up must be fp16 with unit column stride")
    if up.shape != gate.shape or (m > 1 and up.stride(0) != gate.stride(0)):
        raise ValueError("gate and up must have the same shape and row stride")
    dev = _gpu(gate, "gate")
    if _gpu(up, "up") != dev:
        raise ValueError("gate and up must be on the same device")
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
    _on(dev, stream, (lib or _lib).mixllm_silu_mul_quant, _ptr(gate), _ptr(up), ld, m, inter, GROUP, _ptr(aq), _ptr(sa),
        _ptr(asum), _ptr(rowop), _ptr(h))


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
    _on(_gpu(b.dev, "blob"), stream, (lib or _lib).mixllm_gemm_w4w8a8, _ptr(aq), _ptr(sa), _ptr(asum), _ptr(rowop), m, n,
        k, n8, ctypes.byref(b.info), _ptr(b.dev), b.nbytes, _ptr(y), ldy, _ptr(workspace), ws)


def mixllm_gemm_w4w8a8_partials(aq, sa, asum, rowop, m: int, n: int, k: int, n8: int, blob, n_begin: int,
                                n_count: int, part, stream=None, lib=None):
    """part: int32 [M, n_count, G] CUDA tensor."""
    b = _blob(blob)
    if m and n_count:
        _gemm_inputs(aq, sa, asum, rowop, m, k, b.info.nb4)
        _need(part, "part", torch.int32, (m, n_count, k // GROUP))
        if not part.is_contiguous():
            raise ValueError("part must be contiguous")
    _on(_gpu(b.dev, "blob"), stream, (lib or _lib).mixllm_gemm_w4w8a8_partials, _ptr(aq), _ptr(sa), _ptr(asum),
        _ptr(rowop), m, n, k, n8, ctypes.byref(b.info), _ptr(b.dev), b.nbytes, n_begin, n_count, _ptr(part))


# ------------------------------------------------------------- between the packed layers

FP16, BF16, FP32 = 0, 1, 2  # MIXLLM_FP16, MIXLLM_BF16, MIXLLM_FP32
_f16, _bf16, _i32t, _u8t = ((torch.float16, torch.bfloat16, torch.int32, torch.uint8) if torch is not None
                            else (None,) * 4)

# These calls run once or more per layer and token: a call that needs no error costs one
# comparison chain per tensor (about 0.3 us), the library call 1.2 us and the launch 3 us;
# torch.cuda.current_stream() alone would add 2.7 us to that.
_raw_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None)
_device = getattr(getattr(torch, "_C", None), "_cuda_getDevice", None)


_HALF = 1 << 31  # (v + _HALF) >> 32 is 0 for what fits 32 bits with a sign


def _past32(*values):
    raise ValueError(f"a number does not fit 32 bits, the library's integers: one of {values}")


def _dtype16(t, name):
    """The library's number of a 16-bit element type."""
    d = t.dtype
    if d is _f16:
        return FP16
    if d is _bf16:
        return BF16
    raise ValueError(f"{name} must be torch.float16 or torch.bfloat16, got {d}")


def _gpu(t, name):
    """The index of the GPU a tensor is on."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _ld(t, name, dtype, dev, shape, width):
    """The row stride of a tensor of this type, place and shape whose rows are contiguous."""
    if t.dtype is dtype and t.get_device() == dev and t.shape == shape:
        if t.is_contiguous():
            return width
        st, rows = t.stride(), shape[0]
        whole = True
        step = 1
        for size, stride in zip(reversed(shape[1:]), reversed(st[1:])):
            whole = whole and (size == 1 or stride == step)
            step *= size
        if whole and rows <= 1:
            return width
        if whole and st[0] >= width:
            return st[0]
        raise ValueError(f"{name} must have contiguous rows that do not overlap, has strides {st}")
    raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on cuda:{dev}, is {t.dtype} of shape "
                     f"{tuple(t.shape)} on {t.device}")


def _flat(t, name, dtype, dev, numel):
    """The address of a contiguous tensor of at least `numel` elements."""
    if t.dtype is dtype and t.get_device() == dev and t.numel() >= numel and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {numel} elements on cuda:{dev}, is "
                     f"{t.dtype} of shape {tuple(t.shape)} on {t.device}")


def _channels(t, name, dtype, dev, n):
    """The address of a tensor of one number per channel."""
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} elements, one per channel, is of shape {tuple(t.shape)}")
    return _flat(t, name, dtype, dev, n)


def _table(t, b, dev):
    """(address, row stride, width) of a page table of at least b rows."""
    if t.dtype is _i32t and t.dim() == 2 and t.get_device() == dev:
        rows, width = t.shape
        if rows >= b:
            if t.is_contiguous():
                return t.data_ptr(), width, width
            ld, one = t.stride()
            if (width <= 1 or one == 1) and (rows <= 1 or ld >= width):
                return t.data_ptr(), ld if rows > 1 else width, width
    raise ValueError(f"table must be an int32 tensor [{b} or more, width] with contiguous rows on cuda:{dev}, is "
                     f"{t.dtype} of shape {tuple(t.shape)} on {t.device}")


def _on(dev, stream, fn, *args):
    """Calls a device entry point with the stream last, on the tensors' device: by default its
    current stream."""
    if stream is not None:
        stream = stream if isinstance(stream, int) else stream.cuda_stream
    elif _raw_stream is not None:
        stream = _raw_stream(dev)
    else:
        stream = torch.cuda.current_stream(dev).cuda_stream
    if (_device() if _device is not None else torch.cuda.current_device()) == dev:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        raise MixLLMError(status)


def _current(stream, dev):
    """A context in which a stream (a torch stream, a handle or None for the current one) is
    torch's current one."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


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
    dtype, t16 = _dtype16(lead, "x or pre_weight"), lead.dtype
    dev = _gpu(res, "res")
    shape = res.shape
    if len(shape) != 2:
        raise ValueError("res must be 2-D")
    m, n = shape
    tres, res_dtype = (t16, dtype) if res.dtype is t16 else (torch.float32, FP32)
    ldr = _ld(res, "res", tres, dev, shape, n)
    ldx = ldro = ldy = ldgate = 0
    px = pro = py = pgate = ppost = ppre = paq = psa = psum = pro4 = None
    if x is not None:
        ldx, px = _ld(x, "x", t16, dev, shape, n), x.data_ptr()
    if res_out is not None:
        ldro, pro = _ld(res_out, "res_out", tres, dev, shape, n), res_out.data_ptr()
    if y is not None:
        ldy, py = _ld(y, "y", t16, dev, shape, n), y.data_ptr()
    if post_weight is not None:
        ppost = _channels(post_weight, "post_weight", t16, dev, n)
    if pre_weight is not None:
        ppre = _channels(pre_weight, "pre_weight", t16, dev, n)
    if gate is not None:
        if gate.dim() != 1:
            ldgate, pgate = _ld(gate, "gate", t16, dev, shape, n), gate.data_ptr()
        else:
            pgate = _channels(gate, "gate", t16, dev, n)
    if aq is not None:
        g = n // GROUP
        paq = _flat(aq, "aq", torch.int8, dev, m * n)
        if sa is None or aq.shape != shape or sa.shape != (g, m):
            raise ValueError(f"aq and sa must be [{m}, {n}] and [{g}, {m}]")
        psa = _flat(sa, "sa", torch.float32, dev, g * m)
        psum = _flat(asum, "asum", _i32t, dev, g * m) if asum is not None else None
        pro4 = _flat(rowop, "rowop", _i32t, dev, g * m * 8) if rowop is not None else None
    elif sa is not None or asum is not None or rowop is not None:
        raise ValueError("sa, asum and rowop are outputs beside the codes: aq is required")
    _on(dev, stream, _lib.mixllm_residual_norm, px, ldx, ppost, pgate, ldgate, res.data_ptr(), ldr, pro, ldro, ppre, py,
        ldy, paq, psa, psum, pro4, m, n, GROUP, dtype, res_dtype, eps, alpha, beta)


def mixllm_kv4_page_bytes(page: int, heads: int, dim: int) -> int:
    if (page + _HALF | heads + _HALF | dim + _HALF) >> 32:
        _past32(page, heads, dim)
    return int(_lib.mixllm_kv4_page_bytes(page, heads, dim))


def kv4_cache(pages: int, page: int, heads: int, dim: int, device="cuda"):
    """Storage of one layer's cache: uint8 [pages, heads, bytes of a (page, head) block]."""
    size = mixllm_kv4_page_bytes(page, heads, dim)
    if not size or pages <= 0:
        raise ValueError("pages and heads must be positive, page a power of two of 16 .. 1024, dim 64, 128 or 256")
    return torch.empty((pages, heads, size // heads), dtype=torch.uint8, device=device)


def _cache(cache, page, dim):
    """(device, address, bytes, pages, heads) of a cache for pages of `page` tokens and heads of
    `dim` channels."""
    if cache.dtype is _u8t and cache.dim() == 3 and cache.is_contiguous():
        pages, heads, block = cache.shape
        if block * 8 == page * dim * 9:
            return _gpu(cache, "cache"), cache.data_ptr(), pages * heads * block, pages, heads
    raise ValueError(f"cache must be a contiguous uint8 tensor [pages, heads, {page * dim * 9 / 8:g}] for page {page} and "
                     f"dim {dim}, is {cache.dtype} of shape {tuple(cache.shape)}")


def mixllm_kv_plan(fresh, lens, table, pool, count, page: int, pages: int, lens_out, count_out, cu, slots, pos,
                   stream=None):
    """The page tables and slot maps of a step from request lengths, on the GPU: fresh, lens,
    lens_out: int32 [B] (B is fresh's size; give attention as many lengths); table: int32 [B,
    width] (rows may be strided); pool: int32 [F]; count: int32 [1 or more]; count_out: int32 [2];
    cu: int32 [B + 1]; slots, pos: int32 [tokens], tokens at least the sum of what is added."""
    _plan(_lib.mixllm_kv_plan, fresh, lens, table, pool, count, page, pages, lens_out, count_out, cu, slots, pos, stream)


def mixllm_kv_plan_fit(fresh, lens, table, pool, count, page: int, pages: int, lens_out, count_out, cu, slots, pos,
                       stream=None):
    """mixllm_kv_plan, which also refuses the requests whose rows do not fit slots and pos."""
    _plan(_lib.mixllm_kv_plan_fit, fresh, lens, table, pool, count, page, pages, lens_out, count_out, cu, slots, pos,
          stream)


def _plan(fn, fresh, lens, table, pool, count, page, pages, lens_out, count_out, cu, slots, pos, stream):
    b, tokens = fresh.numel(), slots.numel()
    if (page + _HALF | pages + _HALF | tokens + _HALF | pool.numel() + _HALF) >> 32:
        _past32(page, pages, tokens, pool.numel())
    dev = _gpu(fresh, "fresh")
    ptable, ldt, width = _table(table, b, dev)
    _on(dev, stream, fn, _flat(fresh, "fresh", _i32t, dev, 0), _flat(lens, "lens", _i32t, dev, b), b,
        ptable, ldt, width, _flat(pool, "pool", _i32t, dev, 0), pool.numel(), _flat(count, "count", _i32t, dev, 1), page,
        pages, _flat(lens_out, "lens_out", _i32t, dev, b), _flat(count_out, "count_out", _i32t, dev, 2),
        _flat(cu, "cu", _i32t, dev, b + 1), _flat(slots, "slots", _i32t, dev, 0), _flat(pos, "pos", _i32t, dev, tokens),
        tokens)


# The calls of both caches: `fn` is the library's, `shape_of` the check of its cache.

def _append(fn, shape_of, k, v, slots, cache, page, stream):
    t, _, dim = shape = k.shape
    dev, pcache, size, pages, heads = shape_of(cache, page, dim)
    dtype, t16, width = _dtype16(k, "k"), k.dtype, heads * dim
    if shape[1] != heads:
        raise ValueError(f"k has {shape[1]} heads, the cache {heads}")
    _on(dev, stream, fn, k.data_ptr(), _ld(k, "k", t16, dev, shape, width), v.data_ptr(),
        _ld(v, "v", t16, dev, shape, width), dtype, _flat(slots, "slots", _i32t, dev, t), t, pcache, size, pages, page,
        heads, dim)


def _read(fn, shape_of, cache, slots, k, v, page, stream):
    t, _, dim = shape = k.shape
    dev, pcache, size, pages, heads = shape_of(cache, page, dim)
    dtype, t16, width = _dtype16(k, "k"), k.dtype, heads * dim
    if shape[1] != heads:
        raise ValueError(f"k has {shape[1]} heads, the cache {heads}")
    _on(dev, stream, fn, pcache, size, pages, page, heads, dim, _flat(slots, "slots", _i32t, dev, t), t,
        k.data_ptr(), _ld(k, "k", t16, dev, shape, width), v.data_ptr(), _ld(v, "v", t16, dev, shape, width), dtype)


def _attention_bytes(fn, *sizes):
    for v in sizes:
        if (v + _HALF) >> 32:
            _past32(v)
    return int(fn(*sizes))


def _attention(fn, shape_of, q, cache, table, lens, cu, out, page, max_rows, max_len, scale, window, lse, workspace, stream):
    if (max_rows + _HALF | max_len + _HALF | window + _HALF) >> 32:
        _past32(max_rows, max_len, window)
    t, hq, dim = shape = q.shape
    dev, pcache, size, pages, heads = shape_of(cache, page, dim)
    dtype, t16, width = _dtype16(q, "q"), q.dtype, hq * dim
    b = lens.numel()
    ptable, ldt, tw = _table(table, b, dev)
    plse = pws = None
    ws = 0
    if lse is not None:
        plse = _flat(lse, "lse", torch.float32, dev, t * hq)
        if lse.shape != (t, hq):
            raise ValueError(f"lse must be [{t}, {hq}], is {tuple(lse.shape)}")
    if workspace is not None:
        ws = workspace.numel()
        pws = _flat(workspace, "workspace", _u8t, dev, 0)
    _on(dev, stream, fn, q.data_ptr(), _ld(q, "q", t16, dev, shape, width), dtype, t, hq, pcache,
        size, pages, page, heads, dim, ptable, ldt, tw, _flat(lens, "lens", _i32t, dev, 0),
        _flat(cu, "cu", _i32t, dev, b + 1), b, max_rows, max_len, dim ** -0.5 if scale is None else scale, window,
        out.data_ptr(), _ld(out, "out", t16, dev, shape, width), plse, pws, ws)


def mixllm_kv4_append(k, v, slots, cache, page: int, stream=None):
    """Writes k and v ([T, heads, dim] fp16 or bf16, rows may be strided) into the cache at
    slots (int32 [T], negative: skip the row)."""
    _append(_lib.mixllm_kv4_append, _cache, k, v, slots, cache, page, stream)


def mixllm_kv4_read(cache, slots, k, v, page: int, stream=None):
    """The values of the tokens at slots (int32 [T]) into k and v ([T, heads, dim] fp16 or
    bf16); rows with a negative slot are left as they were."""
    _read(_lib.mixllm_kv4_read, _cache, cache, slots, k, v, page, stream)


def mixllm_kv4_attention_workspace_bytes(t: int, b: int, q_heads: int, kv_heads: int, dim: int, max_rows: int,
                                         max_len: int, window: int = 0) -> int:
    return _attention_bytes(_lib.mixllm_kv4_attention_workspace_bytes, t, b, q_heads, kv_heads, dim, max_rows, max_len,
                            window)


def mixllm_kv4_attention(q, cache, table, lens, cu, out, page: int, max_rows: int, max_len: int, scale=None,
                         window: int = 0, lse=None, workspace=None, stream=None):
    """Attention of the rows q ([T, q_heads, dim] fp16 or bf16) of B requests over the cache:
    table: int32 [B, width]; lens: int32 [B] tokens cached (these rows' among them); cu: int32
    [B + 1] first row of each request; out: as q; lse: fp32 [T, q_heads] or None; scale: 1 /
    sqrt(dim) by default; workspace: a uint8 tensor of mixllm_kv4_attention_workspace_bytes(T,
    B, ..) for the same arguments (None where that is 0)."""
    _attention(_lib.mixllm_kv4_attention, _cache, q, cache, table, lens, cu, out, page, max_rows, max_len, scale, window,
               lse, workspace, stream)


def mixllm_head_norm_rotate(q, k, pos, inv_freq, q_out=None, k_out=None, q_norm=None, k_norm=None, eps: float = 1e-6,
                            neighbours: bool = False, stream=None):
    """The norms of queries and keys per head and the rotation by position.  q, k: [T, heads,
    dim] fp16 or bf16 (rows may be strided; one of them may be None); pos: int32 [T]; inv_freq:
    fp32 [rot / 2], the first rot channels are turned (None: none); q_out, k_out: by default q and
    k, in place; q_norm, k_norm: [dim] norm weights or None; neighbours: pairs (2i, 2i + 1)
    instead of (i, i + rot / 2)."""
    lead = q if q is not None else k
    if lead is None:
        raise ValueError("q or k is required")
    dtype, t16, dev = _dtype16(lead, "q or k"), lead.dtype, _gpu(lead, "q or k")
    if lead.dim() != 3:
        raise ValueError(f"q and k must be [T, heads, dim], got {tuple(lead.shape)}")
    t, _, dim = lead.shape
    pq = pqo = pqn = pk = pko = pkn = pfreq = ppos = None
    ldq = ldqo = ldk = ldko = hq = hk = rot = 0
    if q is not None:
        shape = q.shape
        hq = shape[1]
        pq, ldq = q.data_ptr(), _ld(q, "q", t16, dev, shape, hq * dim)
        pqo, ldqo = (pq, ldq) if q_out is None else (q_out.data_ptr(), _ld(q_out, "q_out", t16, dev, shape, hq * dim))
        pqn = None if q_norm is None else _channels(q_norm, "q_norm", t16, dev, dim)
    elif q_out is not None or q_norm is not None:
        raise ValueError("q_out and q_norm go with q, which is None")
    if k is not None:
        shape = k.shape
        if len(shape) != 3 or shape[0] != t or shape[2] != dim:
            raise ValueError(f"q and k must be [T, heads, dim] with one T and dim, k is {tuple(shape)}")
        hk = shape[1]
        pk, ldk = k.data_ptr(), _ld(k, "k", t16, dev, shape, hk * dim)
        pko, ldko = (pk, ldk) if k_out is None else (k_out.data_ptr(), _ld(k_out, "k_out", t16, dev, shape, hk * dim))
        pkn = None if k_norm is None else _channels(k_norm, "k_norm", t16, dev, dim)
    elif k_out is not None or k_norm is not None:
        raise ValueError("k_out and k_norm go with k, which is None")
    if inv_freq is not None and inv_freq.numel():
        if pos is None:
            raise ValueError("pos is required for a rotation")
        rot = 2 * inv_freq.numel()
        pfreq, ppos = _flat(inv_freq, "inv_freq", torch.float32, dev, 0), _flat(pos, "pos", _i32t, dev, t)
    _on(dev, stream, _lib.mixllm_head_norm_rotate, pq, ldq, pk, ldk, pqo, ldqo, pko, ldko, ppos, pfreq, pqn, pkn, t, hq, hk,
        dim, rot, 1 if neighbours else 0, dtype, eps)


def mixllm_kv8_page_bytes(page: int, heads: int, dim: int) -> int:
    if (page + _HALF | heads + _HALF | dim + _HALF) >> 32:
        _past32(page, heads, dim)
    return int(_lib.mixllm_kv8_page_bytes(page, heads, dim))


def kv8_cache(pages: int, page: int, heads: int, dim: int, device="cuda"):
    """Storage of one layer's cache in 8 bits: uint8 [pages, heads, bytes of a (page, head) block]."""
    size = mixllm_kv8_page_bytes(page, heads, dim)
    if not size or pages <= 0:
        raise ValueError("pages and heads must be positive, page a power of two of 16 .. 1024, dim 64, 128 or 256")
    return torch.empty((pages, heads, size // heads), dtype=torch.uint8, device=device)


def _cache8(cache, page, dim):
    """As _cache, of a cache in 8 bits."""
    block = 2 * page * dim + (page // 2 + 127) // 128 * 128
    if cache.dtype is _u8t and cache.dim() == 3 and cache.is_contiguous() and cache.shape[2] == block:
        pages, heads, _ = cache.shape
        return _gpu(cache, "cache"), cache.data_ptr(), pages * heads * block, pages, heads
    raise ValueError(f"cache must be a contiguous uint8 tensor [pages, heads, {block}] for page {page} and dim {dim}, is "
                     f"{cache.dtype} of shape {tuple(cache.shape)}")


def mixllm_kv8_append(k, v, slots, cache, page: int, stream=None):
    """Writes k and v ([T, heads, dim] fp16 or bf16, rows may be strided) into the cache in 8 bits
    at slots (int32 [T], negative: skip the row; rows of one run of 16 tokens follow one another
    in the order of their slots)."""
    _append(_lib.mixllm_kv8_append, _cache8, k, v, slots, cache, page, stream)


def mixllm_kv8_read(cache, slots, k, v, page: int, stream=None):
    """The values of the tokens at slots (int32 [T]) into k and v ([T, heads, dim] fp16 or
    bf16); rows with a negative slot are left as they were."""
    _read(_lib.mixllm_kv8_read, _cache8, cache, slots, k, v, page, stream)


def mixllm_kv8_attention_workspace_bytes(t: int, b: int, q_heads: int, kv_heads: int, dim: int, max_rows: int,
                                         max_len: int, window: int = 0) -> int:
    return _attention_bytes(_lib.mixllm_kv8_attention_workspace_bytes, t, b, q_heads, kv_heads, dim, max_rows, max_len,
                            window)


def mixllm_kv8_attention(q, cache, table, lens, cu, out, page: int, max_rows: int, max_len: int, scale=None,
                         window: int = 0, lse=None, workspace=None, stream=None):
    """mixllm_kv4_attention over a cache in 8 bits; workspace: a uint8 tensor of
    mixllm_kv8_attention_workspace_bytes(T, B, ..) for the same arguments (None where that is 0)."""
    _attention(_lib.mixllm_kv8_attention, _cache8, q, cache, table, lens, cu, out, page, max_rows, max_len, scale, window,
               lse, workspace, stream)


def mixllm_quant_rows(a, q, s, stream=None):
    """Quantizes the rows of a ([M, K] fp16 or bf16, rows may be strided) to q (int8 [M, K]) with
    one scale per row in s (fp32 [M]; NaN, with codes of 0, for a row with a NaN or an infinity)."""
    if a.dim() != 2:
        raise ValueError(f"a must be [M, K], is {tuple(a.shape)}")
    m, k = shape = a.shape
    dtype, t16, dev = _dtype16(a, "a"), a.dtype, _gpu(a, "a")
    _on(dev, stream, _lib.mixllm_quant_rows, a.data_ptr(), _ld(a, "a", t16, dev, shape, k), dtype, m, k, q.data_ptr(),
        _ld(q, "q", torch.int8, dev, shape, k), _flat(s, "s", torch.float32, dev, m))


def mixllm_gemm_w8a8(aq, sa, w, sw, y, stream=None):
    """y = (aq w^T) sa sw: aq: int8 [M, K], w: int8 [N, K] (rows may be strided), sa: fp32 [M], sw:
    fp32 [N], y: fp16 or bf16 [M, N] (rows may be strided)."""
    if aq.dim() != 2 or w.dim() != 2 or aq.shape[1] != w.shape[1]:
        raise ValueError(f"aq and w must be [M, K] and [N, K], are {tuple(aq.shape)} and {tuple(w.shape)}")
    (m, k), n = aq.shape, w.shape[0]
    dtype, dev = _dtype16(y, "y"), _gpu(aq, "aq")
    _on(dev, stream, _lib.mixllm_gemm_w8a8, aq.data_ptr(), _ld(aq, "aq", torch.int8, dev, aq.shape, k),
        _flat(sa, "sa", torch.float32, dev, m), w.data_ptr(), _ld(w, "w", torch.int8, dev, w.shape, k),
        _flat(sw, "sw", torch.float32, dev, n), m, n, k, y.data_ptr(), _ld(y, "y", y.dtype, dev, (m, n), n), dtype)


def rowop_buffer(m: int, k: int, device="cuda"):
    """Storage for mixllm_quant_act's row operands: 32-bit words [G, M, 8]."""
    return torch.empty((k // GROUP, m, 8), dtype=torch.int32, device=device)


# ---------------------------------------------------------------------------- convenience

def _same_rows(bufs, m):
    """The quantized operands are packed by the number of rows: buffers for another number would
    be written by one and read by the other.  No rows: nothing is read."""
    if m and bufs["aq"].shape[0] != m:
        raise ValueError(f"the buffers are for {bufs['aq'].shape[0]} rows, the input has {m} rows")


def _own_buffers(layer, a, stream):
    """A layer's buffers for one call on ``stream``, from that stream's memory: freed when the call
    returns they wait for its work, where those of another stream could be given away before."""
    with _current(stream, a.device):
        return layer.buffers(a.shape[0])


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
        bufs = bufs or _own_buffers(self, a, stream)
        _same_rows(bufs, m)
        mixllm_quant_act(a, bufs["aq"], bufs["sa"], bufs["asum"], bufs["rowop"], stream)
        return self.gemm(bufs, stream, m)

    def gemm(self, bufs, stream=None, rows=None):
        """The product alone, of activations that are quantized in ``bufs`` already (as many
        rows as the buffers have, unless ``rows`` is given)."""
        m = bufs["aq"].shape[0] if rows is None else rows
        mixllm_gemm_w4w8a8(bufs["aq"], bufs["sa"], bufs["asum"], bufs["rowop"], m, self.n, self.k, self.n8, self.blob,
                           bufs["y"], bufs["ws"], stream)
        return bufs["y"]


class RowLinear:
    """A layer wholly in 8 bits with one scale per output channel, its activations with one per
    token: ``forward(a)`` runs mixllm_quant_rows then mixllm_gemm_w8a8.  ``w``: [N, K] fp16 (or bf16,
    as a tensor), quantized once on the GPU, which the constructor waits for; ``dtype``: of the
    outputs, fp16 or bf16."""

    def __init__(self, w, device="cuda", dtype=None):
        w = torch.as_tensor(w).to(device)
        self.n, self.k = w.shape
        self.w = torch.empty((self.n, self.k), dtype=torch.int8, device=device)
        self.sw = torch.empty(self.n, dtype=torch.float32, device=device)
        self.device, self.dtype = device, dtype or torch.float16
        mixllm_quant_rows(w.contiguous(), self.w, self.sw)
        if self.w.is_cuda:  # forward runs on any stream: the weights are there for all of them
            torch.cuda.current_stream(self.w.device).synchronize()

    def buffers(self, m: int):
        dev = self.device
        return dict(aq=torch.empty((m, self.k), dtype=torch.int8, device=dev),
                    sa=torch.empty(m, dtype=torch.float32, device=dev),
                    y=torch.empty((m, self.n), dtype=self.dtype, device=dev))

    def forward(self, a, bufs=None, stream=None):
        m = a.shape[0]
        bufs = bufs or _own_buffers(self, a, stream)
        _same_rows(bufs, m)
        if m:
            mixllm_quant_rows(a, bufs["aq"], bufs["sa"], stream)
        return self.gemm(bufs, stream, m)

    def gemm(self, bufs, stream=None, rows=None):
        """The product alone, of activations that are quantized in ``bufs`` already (as many
        rows as the buffers have, unless ``rows`` is given)."""
        m = bufs["aq"].shape[0] if rows is None else rows
        if m:
            mixllm_gemm_w8a8(bufs["aq"], bufs["sa"], self.w, self.sw, bufs["y"], stream)
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
        bx, m = bufs["x"], x.shape[0]
        for b in (bx, bufs["h"]):
            _same_rows(b, m)
        mixllm_quant_act(x, bx["aq"], bx["sa"], bx["asum"], bx["rowop"], stream)
        return self.forward_quantized(bufs, stream, keep_h, m)

    def forward_quantized(self, bufs, stream=None, keep_h=False, rows=None):
        """The block from a hidden state that is quantized in ``bufs["x"]`` already (as many
        rows as the buffers have, unless ``rows`` is given)."""
        bx, bh = bufs["x"], bufs["h"]
        m = bx["aq"].shape[0] if rows is None else rows
        _same_rows(bh, m)
        gu = self.gu.gemm(bx, stream, m)
        mixllm_silu_mul_quant(gu[:, :self.inter], gu[:, self.inter:], bh["aq"], bh["sa"], bh["asum"], bh["rowop"],
                              bufs["h16"] if keep_h else None, stream)
        return self.down.gemm(bh, stream, m)

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


class RequestPages:
    """Which pages the requests of a batch hold: the page table, the free pages and the lengths
    of up to ``requests`` requests over caches of ``pages`` pages (every layer's cache uses the
    same).  ``plan(fresh)`` moves it on by one step on the GPU and returns the step's slots
    and row bounds; it can be captured.  A request that the pages, ``max_len`` or the ``tokens``
    rows of a step have no room for is refused: its length stays, its rows have slot -1, and
    ``count[1]`` counts it.  Argument marshalling only."""

    def __init__(self, requests: int, pages: int, page: int, max_len: int, tokens: int, device="cuda"):
        if pages <= 0 or max_len <= 0:
            raise ValueError("pages and max_len must be positive")
        self.page, self.pages = page, pages
        new = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        self.table = new(requests, -(-max_len // page))
        self.pool = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device)
        self.count = torch.tensor([pages, 0], dtype=torch.int32, device=device)  # free pages, requests refused last
        self.lens, self.cu = new(requests), new(requests + 1)
        self.slots, self.pos = new(tokens), new(tokens)

    def plan(self, fresh, stream=None):
        """fresh: int32 [requests] tokens to add to each request; negative: it ended."""
        if fresh.numel() != self.lens.numel():  # the row bounds of the others would stay the last step's
            raise ValueError(f"fresh must have a count for each of the {self.lens.numel()} requests, has {fresh.numel()}")
        mixllm_kv_plan_fit(fresh, self.lens, self.table, self.pool, self.count, self.page, self.pages, self.lens,
                           self.count, self.cu, self.slots, self.pos, stream)
        return self


class AttentionBlock:
    """The attention half of a decoder layer on packed layers and a cache in 4 bits: the residual
    sum and norm quantized for the q/k/v projections, one GEMM over q, k and v, the write into
    the cache, attention, and the quantization and GEMM of the output projection.  Six launches on
    one stream (seven where attention splits the tokens).  ``norm`` is the weight of the norm
    before the projections; ``post_norm``, for layers that norm what a block gives, is the one of
    the block *before* this one (its output x is normed as it is added).

    ``cache_bits`` 8 keeps the cache in 8 bits.  ``q_norm``, ``k_norm`` ([dim]) norm every head of
    queries and keys (with ``eps``), ``inv_freq`` (fp32 [rot / 2]) turns their first rot channels by
    the position, pairs (i, i + rot / 2) or with ``neighbours`` (2i, 2i + 1): one launch more, between
    the product and the write.  ``idx8_o`` None takes the output projection wholly in 8 bits with a
    scale per channel and token (RowLinear).  Argument marshalling only."""

    def __init__(self, w_q, w_k, w_v, w_o, idx8_q, idx8_k, idx8_v, idx8_o, norm, q_heads: int, kv_heads: int,
                 pages: int, page: int, post_norm=None, eps: float = 1e-5, window: int = 0, device="cuda",
                 cache_bits: int = 4, q_norm=None, k_norm=None, inv_freq=None, neighbours: bool = False):
        if cache_bits not in (4, 8):
            raise ValueError(f"cache_bits must be 4 or 8, is {cache_bits}")
        self.qkv = QKVProjection(w_q, w_k, w_v, idx8_q, idx8_k, idx8_v, device)
        w_o = np.asarray(w_o, np.float16)
        self.o = RowLinear(w_o, device) if idx8_o is None else PackedLinear(w_o, idx8_o, device)
        self.q_heads, self.kv_heads = q_heads, kv_heads
        self.dim = np.asarray(w_k).shape[0] // kv_heads
        if np.asarray(w_q).shape[0] != q_heads * self.dim or np.asarray(w_k).shape != np.asarray(w_v).shape or (
                self.o.k != q_heads * self.dim):
            raise ValueError("the projections' shapes do not fit the heads")
        for w, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if w is not None and w.numel() != self.dim:
                raise ValueError(f"{name} must have {self.dim} elements, one per channel of a head, has {w.numel()}")
        if inv_freq is not None and not 0 < inv_freq.numel() <= self.dim // 2:
            raise ValueError(f"inv_freq must have 1 to {self.dim // 2} elements, has {inv_freq.numel()}")
        self.cache = (kv4_cache if cache_bits == 4 else kv8_cache)(pages, page, kv_heads, self.dim, device)
        self.norm, self.post_norm, self.eps, self.window, self.page, self.device = norm, post_norm, eps, window, page, device
        self.cache_bits, self.q_norm, self.k_norm, self.inv_freq, self.neighbours = cache_bits, q_norm, k_norm, inv_freq, neighbours

    def buffers(self, m: int, requests: int, max_rows: int, max_len: int):
        size_of = mixllm_kv4_attention_workspace_bytes if self.cache_bits == 4 else mixllm_kv8_attention_workspace_bytes
        size = size_of(m, requests, self.q_heads, self.kv_heads, self.dim, max_rows, max_len, self.window)
        return dict(qkv=self.qkv.buffers(m), o=self.o.buffers(m), max_rows=max_rows, max_len=max_len,
                    attn=torch.zeros((m, self.q_heads, self.dim), dtype=torch.float16, device=self.device),
                    ws=torch.empty(size, dtype=torch.uint8, device=self.device) if size else None)

    def forward(self, x, h, bufs, req, rotate=None, stream=None):
        """h: [M, hidden] the residual stream (fp16 or fp32), updated in place by the block output
        x of the layer before (None for the first); M the rows that the plan counts or more (a
        token whose row is missing here is counted and never written); req: RequestPages after
        its plan(); rotate: called with the views q [M, heads, dim], k and the positions before
        the keys are written, for an embedding of positions of the caller's own (in place, on the
        stream that is current then, which is ``stream``; after the layer's own norms and rotation,
        if it has them).  Returns the output projection's [M, hidden]."""
        if req.page != self.page or req.pages > self.cache.shape[0]:
            raise ValueError(f"the requests have {req.pages} pages of {req.page} tokens, the cache has "
                             f"{self.cache.shape[0]} pages of {self.page}")
        b, bo = bufs["qkv"], bufs["o"]
        m = h.shape[0]
        mixllm_residual_norm(x, h, self.norm, h if x is not None else None, aq=b["aq"], sa=b["sa"], asum=b["asum"],
                             rowop=b["rowop"], post_weight=self.post_norm if x is not None else None, eps=self.eps,
                             stream=stream)
        q, k, v = self.qkv.split(self.qkv.layer.gemm(b, stream))
        q, k, v = q.unflatten(1, (self.q_heads, self.dim)), k.unflatten(1, (self.kv_heads, self.dim)), v.unflatten(
            1, (self.kv_heads, self.dim))
        if self.q_norm is not None or self.k_norm is not None or self.inv_freq is not None:
            mixllm_head_norm_rotate(q, k, req.pos[:m], self.inv_freq, q_norm=self.q_norm, k_norm=self.k_norm, eps=self.eps,
                                    neighbours=self.neighbours, stream=stream)
        if rotate is not None:
            with _current(stream, q.device):  # between the product and the write, on the same stream
                rotate(q, k, req.pos[:m])
        append, attention = ((mixllm_kv4_append, mixllm_kv4_attention) if self.cache_bits == 4 else
                             (mixllm_kv8_append, mixllm_kv8_attention))
        append(k, v, req.slots[:m], self.cache, self.page, stream)
        attention(q, self.cache, req.table, req.lens, req.cu, bufs["attn"], self.page, bufs["max_rows"],
                  bufs["max_len"], window=self.window, workspace=bufs["ws"], stream=stream)
        return self.o.forward(bufs["attn"].flatten(1), bo, stream)


class DecoderLayer:
    """A decoder layer: AttentionBlock, the norm between, MLPBlock.  The layer's output is left
    to the next layer's first norm (or a last mixllm_residual_norm) to add.  ``norm`` is the
    weight before the MLP block, ``post_norm`` that of the attention block's output; the MLP
    block's output is normed by the next layer's ``AttentionBlock.post_norm``.  The blocks are
    added as they are: gates and factors are mixllm_residual_norm's own.  Argument marshalling
    only."""

    def __init__(self, attention: AttentionBlock, mlp: MLPBlock, norm, post_norm=None):
        self.attention, self.mlp, self.norm, self.post_norm = attention, mlp, norm, post_norm

    def buffers(self, m: int, requests: int, max_rows: int, max_len: int):
        return dict(attention=self.attention.buffers(m, requests, max_rows, max_len), mlp=self.mlp.buffers(m))

    def forward(self, x, h, bufs, req, rotate=None, stream=None):
        """As AttentionBlock.forward; returns the MLP block's [M, hidden]."""
        a = self.attention.forward(x, h, bufs["attention"], req, rotate, stream)
        b = bufs["mlp"]["x"]
        mixllm_residual_norm(a, h, self.norm, h, aq=b["aq"], sa=b["sa"], asum=b["asum"], rowop=b["rowop"],
                             post_weight=self.post_norm, eps=self.attention.eps, stream=stream)
        return self.mlp.forward_quantized(bufs["mlp"], stream)
