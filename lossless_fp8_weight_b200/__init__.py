"""ECF8 lossless FP8 E4M3 weight codec: Python binding of libecf8.

Thin ctypes layer over the C ABI in ``include/ecf8.h``: it marshals arguments
and nothing else.  Encoding runs in the library's host code; every step of
decoding runs in its sm_100a kernels.  PyTorch is used only to hand over
device pointers and the current CUDA stream.  There is no CPU fallback: if
``libecf8.so`` is missing, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_SO = os.path.join(_HERE, "libecf8.so")



def _ensure_built() -> None:
    """Compile libecf8.so in place when it is missing or older than its
    sources (the build script is loaded by path, so this package's own import
    does not recurse)."""
    import importlib.util
    spec = importlib.util.spec_from_file_location("_ecf8_build", os.path.join(_HERE, "_build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    if mod.stale():
        try:
            mod.build()
        except Exception as e:  # no toolchain: the decoder has no CPU fallback
            raise ImportError(f"{_SO} is missing or stale and could not be built: {e}") from e


_ensure_built()
_lib = ctypes.CDLL(_SO)

OK = 0
ERRORS = {-1: "ARG", -2: "FORMAT", -3: "CAPACITY", -4: "CODEBOOK", -5: "ALIGN", -6: "UNSUPPORTED", -7: "CUDA",
          -8: "WORKSPACE", -9: "TOO_MANY", -10: "CAPTURE"}
STATUS_COUNT_MISMATCH = 1
STATUS_BAD_CODE = 2
STATUS_BAD_OFFSETS = 4
STATUS_BAD_REQUEST = 16
STATUS_NONFINITE = 32
STATUS_TIMEOUT = 64
BATCH_INLINE_MAX = 64
NOALLOC_MAX_TENSORS = 1024
DEFAULT_CHUNK_BYTES = 32
DEFAULT_GROUP_CHUNKS = 32


class Codebook(ctypes.Structure):
    _fields_ = [("len", ctypes.c_uint8 * 16), ("code", ctypes.c_uint16 * 16), ("max_len", ctypes.c_uint32),
                ("n_symbols", ctypes.c_uint32)]

    @property
    def lengths(self) -> np.ndarray:
        return np.frombuffer(bytes(self.len), dtype=np.uint8).copy()


class Info(ctypes.Structure):
    _fields_ = [("n", ctypes.c_uint64), ("code_bits", ctypes.c_uint64), ("blob_bytes", ctypes.c_uint64),
                ("gaps_off", ctypes.c_uint64), ("groups_off", ctypes.c_uint64),
                ("stream_off", ctypes.c_uint64), ("nibbles_off", ctypes.c_uint64),
                ("chunk_bytes", ctypes.c_uint32), ("group_chunks", ctypes.c_uint32), ("n_groups", ctypes.c_uint32),
                ("max_len", ctypes.c_uint32), ("len", ctypes.c_uint8 * 16)]

    @property
    def lengths(self) -> np.ndarray:
        return np.frombuffer(bytes(self.len), dtype=np.uint8).copy()

    @property
    def ratio(self) -> float:
        return self.n / self.blob_bytes if self.blob_bytes else 0.0


class Tensor(ctypes.Structure):
    _fields_ = [("info", ctypes.POINTER(Info)), ("d_blob", ctypes.c_void_p), ("blob_size", ctypes.c_size_t),
                ("d_out", ctypes.c_void_p)]


_p, _sz, _u32, _i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_int
_lib.ecf8_histogram.argtypes = [_p, _sz, _p]
_lib.ecf8_build_codebook.argtypes = [_p, _u32, ctypes.POINTER(Codebook)]
_lib.ecf8_encoded_size.argtypes = [_p, _sz, ctypes.POINTER(Codebook), _u32, _u32, ctypes.POINTER(_sz)]
_lib.ecf8_encoded_size_bound.argtypes = [_sz, _u32, _u32]
_lib.ecf8_encoded_size_bound.restype = _sz
_lib.ecf8_encode.argtypes = [_p, _sz, ctypes.POINTER(Codebook), _u32, _u32, _p, _sz, ctypes.POINTER(_sz)]
_lib.ecf8_blob_info.argtypes = [_p, _sz, ctypes.POINTER(Info)]
_lib.ecf8_layout_supported.argtypes = [_u32, _u32]
_lib.ecf8_decode.argtypes = [ctypes.POINTER(Info), _p, _sz, _p, _sz, _p, _p]
_lib.ecf8_batched_workspace_size.argtypes = [_i32]
_lib.ecf8_batched_workspace_size.restype = _sz
_lib.ecf8_decode_batched.argtypes = [ctypes.POINTER(Tensor), _i32, _p, _sz, _p, _p]
_lib.ecf8_decode_batched_noalloc.argtypes = [ctypes.POINTER(Tensor), _i32, _p, _p]
_lib.ecf8_decode_batched_ctas.argtypes = [ctypes.POINTER(Tensor), _i32, _p, _sz, _p, _p, _u32]
_lib.ecf8_histogram_device.argtypes = [_p, _sz, _p, _p]
_lib.ecf8_encode_device_workspace_size.argtypes = [_sz]
_lib.ecf8_encode_device_workspace_size.restype = _sz
_lib.ecf8_encode_device.argtypes = [_p, _sz, _p, ctypes.POINTER(Codebook), _u32, _u32, _p, _sz, ctypes.POINTER(_sz),
                                    _p, _sz, _p]


class Bf16Info(ctypes.Structure):
    _fields_ = [("n", ctypes.c_uint64), ("code_bits", ctypes.c_uint64), ("blob_bytes", ctypes.c_uint64),
                ("lens_off", ctypes.c_uint64), ("gaps_off", ctypes.c_uint64), ("groups_off", ctypes.c_uint64),
                ("stream_off", ctypes.c_uint64), ("kept_off", ctypes.c_uint64),
                ("chunk_bytes", ctypes.c_uint32), ("group_chunks", ctypes.c_uint32), ("n_groups", ctypes.c_uint32),
                ("max_len", ctypes.c_uint32), ("len", ctypes.c_uint8 * 256)]

    @property
    def lengths(self) -> np.ndarray:
        return np.frombuffer(bytes(self.len), dtype=np.uint8).copy()

    @property
    def ratio(self) -> float:
        return 2 * self.n / self.blob_bytes if self.blob_bytes else 0.0


_lib.ecf8_bf16_code_lengths.argtypes = [_p, _sz, _u32, _p]
_lib.ecf8_bf16_encoded_size.argtypes = [_p, _sz, _p, _u32, _u32, ctypes.POINTER(_sz)]
_lib.ecf8_bf16_encode.argtypes = [_p, _sz, _p, _u32, _u32, _p, _sz, ctypes.POINTER(_sz)]
_lib.ecf8_bf16_blob_info.argtypes = [_p, _sz, ctypes.POINTER(Bf16Info)]
_lib.ecf8_bf16_table_bytes.restype = _sz
_lib.ecf8_bf16_build_table.argtypes = [ctypes.POINTER(Bf16Info), _p]
_lib.ecf8_bf16_table_nodes.argtypes = [ctypes.POINTER(Bf16Info)]
_lib.ecf8_bf16_table_nodes.restype = _u32
_lib.ecf8_bf16_decode.argtypes = [ctypes.POINTER(Bf16Info), _p, _p, _p, _sz, _p, _p]
_lib.ecf8_bf16_decode_layout.argtypes = [ctypes.POINTER(Bf16Info), _p, _p, _p, _sz, _p, _p, _i32]
_lib.ecf8_bf16_auto_layout.argtypes = [ctypes.POINTER(Bf16Info)]
BF16_LAYOUTS = {"auto": -1, "wide": 0, "narrow": 1, "narrow_lane": 2, "byte": 3}
BF16_BATCH_MAX = 32


class Bf16Tensor(ctypes.Structure):
    _fields_ = [("info", ctypes.POINTER(Bf16Info)), ("d_blob", ctypes.c_void_p), ("d_table", ctypes.c_void_p),
                ("d_out", ctypes.c_void_p)]


_lib.ecf8_bf16_decode_batched.argtypes = [ctypes.POINTER(Bf16Tensor), _i32, _p, _p]


class LayerTensor(ctypes.Structure):
    _fields_ = [("info", ctypes.POINTER(Info)), ("d_blob", ctypes.c_void_p), ("blob_size", ctypes.c_size_t),
                ("out_offset", ctypes.c_size_t)]


class Layer(ctypes.Structure):
    _fields_ = [("tensors", ctypes.POINTER(LayerTensor)), ("count", ctypes.c_int)]


_lib.ecf8_pipeline_create.argtypes = [ctypes.POINTER(Layer), _i32, ctypes.POINTER(ctypes.c_void_p), _i32, _sz, _i32,
                                      _u32, _p, _sz, _p, _p, ctypes.POINTER(ctypes.c_void_p)]
_lib.ecf8_pipeline_acquire.argtypes = [_p, _i32, _p, ctypes.POINTER(ctypes.c_void_p)]
_lib.ecf8_pipeline_release.argtypes = [_p, _i32, _p]
_lib.ecf8_pipeline_destroy.argtypes = [_p]
_lib.ecf8_pipeline_destroy.restype = None
_lib.ecf8_launch_count.restype = ctypes.c_uint64
_lib.ecf8_strerror.restype = ctypes.c_char_p
_lib.ecf8_strerror.argtypes = [_i32]


class Ecf8Error(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {_lib.ecf8_strerror(code).decode()} ({ERRORS.get(code, code)})")
        self.code = code


def _check(rc: int, what: str) -> None:
    if rc != OK:
        raise Ecf8Error(rc, what)


def library_path() -> str:
    return _SO


def launch_count() -> int:
    """Decode kernels launched by this process so far."""
    return int(_lib.ecf8_launch_count())


def _host_u8(x) -> np.ndarray:
    if hasattr(x, "detach"):  # a CPU torch tensor
        x = x.detach().contiguous().view(-1).numpy()
    a = np.ascontiguousarray(np.asarray(x).reshape(-1))
    if a.dtype != np.uint8:
        a = a.view(np.uint8)
    return a


def histogram(fp8) -> np.ndarray:
    x = _host_u8(fp8)
    h = np.zeros(16, dtype=np.uint64)
    _check(_lib.ecf8_histogram(x.ctypes.data, x.size, h.ctypes.data), "ecf8_histogram")
    return h


def build_codebook(hist, max_len: int = 16) -> Codebook:
    h = np.ascontiguousarray(np.asarray(hist, dtype=np.uint64))
    cb = Codebook()
    _check(_lib.ecf8_build_codebook(h.ctypes.data, max_len, ctypes.byref(cb)), "ecf8_build_codebook")
    return cb


def encode(fp8, codebook: Optional[Codebook] = None, chunk_bytes: int = DEFAULT_CHUNK_BYTES,
           group_chunks: int = DEFAULT_GROUP_CHUNKS, max_len: int = 16) -> np.ndarray:
    """Compress E4M3 bytes (numpy uint8 / float8 view, or CPU tensor) into a blob."""
    x = _host_u8(fp8)
    h = histogram(x)
    cb = codebook if codebook is not None else build_codebook(h, max_len)
    size = ctypes.c_size_t(0)
    _check(_lib.ecf8_encoded_size(h.ctypes.data, x.size, ctypes.byref(cb), chunk_bytes, group_chunks,
                                  ctypes.byref(size)), "ecf8_encoded_size")
    blob = np.empty(size.value, dtype=np.uint8)
    got = ctypes.c_size_t(0)
    _check(_lib.ecf8_encode(x.ctypes.data, x.size, ctypes.byref(cb), chunk_bytes, group_chunks, blob.ctypes.data,
                            blob.size, ctypes.byref(got)), "ecf8_encode")
    assert got.value == blob.size
    return blob


def histogram_device(d_fp8, stream=None) -> np.ndarray:
    """Exponent histogram of a CUDA uint8 tensor, computed on the GPU (the
    call waits for it and returns a host array)."""
    import torch
    n = d_fp8.numel()
    with torch.cuda.stream(_torch_stream(stream, d_fp8.device)):  # the copy waits for the stream it is made on
        d_fp8 = d_fp8.contiguous()
        d_hist = torch.empty(16, dtype=torch.int64, device=d_fp8.device)
        _check(_lib.ecf8_histogram_device(_ptr(d_fp8), n, _ptr(d_hist), _stream(stream)), "ecf8_histogram_device")
        return d_hist.cpu().numpy().astype(np.uint64)


def encode_device(d_fp8, codebook: Optional[Codebook] = None, chunk_bytes: int = DEFAULT_CHUNK_BYTES,
                  group_chunks: int = DEFAULT_GROUP_CHUNKS, max_len: int = 16, stream=None, hist=None):
    """Compress a CUDA uint8 tensor of E4M3 bytes on the GPU; returns the blob
    as a CUDA uint8 tensor (the same bytes as ``encode`` of the same input).
    On a stream given by its number the blob has to live until it is written."""
    import torch
    with torch.cuda.stream(_torch_stream(stream, d_fp8.device)):  # where a tensor with gaps is copied
        x = d_fp8.contiguous().reshape(-1)
    if x.dtype != torch.uint8:
        x = x.view(torch.uint8)
    n = x.numel()
    h = histogram_device(x, stream) if hist is None else np.ascontiguousarray(np.asarray(hist, dtype=np.uint64))
    cb = codebook if codebook is not None else build_codebook(h, max_len)
    size = ctypes.c_size_t(0)
    _check(_lib.ecf8_encoded_size(h.ctypes.data, n, ctypes.byref(cb), chunk_bytes, group_chunks, ctypes.byref(size)),
           "ecf8_encoded_size")
    blob = torch.empty(size.value, dtype=torch.uint8, device=x.device)
    if isinstance(stream, torch.cuda.Stream):
        blob.record_stream(stream)
    with torch.cuda.stream(_torch_stream(stream, x.device)):  # the stream's own memory, reused after the call on it
        ws = torch.empty(max(16, _lib.ecf8_encode_device_workspace_size(n)), dtype=torch.uint8, device=x.device)
    got = ctypes.c_size_t(0)
    _check(_lib.ecf8_encode_device(_ptr(x), n, h.ctypes.data, ctypes.byref(cb), chunk_bytes, group_chunks, _ptr(blob),
                                   blob.numel(), ctypes.byref(got), _ptr(ws), ws.numel(), _stream(stream)),
           "ecf8_encode_device")
    assert got.value == blob.numel()
    return blob


def encoded_size_bound(n: int, chunk_bytes: int = DEFAULT_CHUNK_BYTES, group_chunks: int = DEFAULT_GROUP_CHUNKS) -> int:
    """Blob bytes that suffice for any n weights in this layout (no histogram needed)."""
    return int(_lib.ecf8_encoded_size_bound(n, chunk_bytes, group_chunks))


def blob_info(blob) -> Info:
    b = _host_u8(blob)
    info = Info()
    _check(_lib.ecf8_blob_info(b.ctypes.data, b.size, ctypes.byref(info)), "ecf8_blob_info")
    return info


def blob_info_device(d_blob) -> Info:
    """blob_info of a blob held in device memory (a CUDA uint8 tensor): only
    its 128-byte header is copied to the host, which is all the parser reads."""
    hdr = np.ascontiguousarray(d_blob[:128].cpu().numpy())
    if hdr.size < 128:
        raise Ecf8Error(-2, "ecf8_blob_info")
    info = Info()
    _check(_lib.ecf8_blob_info(hdr.ctypes.data, int(d_blob.numel() * d_blob.element_size()), ctypes.byref(info)),
           "ecf8_blob_info")
    return info


def layout_supported(chunk_bytes: int, group_chunks: int) -> bool:
    return bool(_lib.ecf8_layout_supported(chunk_bytes, group_chunks))


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    return int(t.data_ptr())


def _nbytes(t, default: int) -> int:
    """Bytes of a torch tensor argument; a raw pointer is taken to hold `default`."""
    if t is None or isinstance(t, int):
        return int(default)
    return int(t.numel() * t.element_size())


def _stream(stream) -> int:
    if stream is None:
        import torch
        return int(torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice()))
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _torch_stream(stream, device):
    """The same as a torch stream, for what torch allocates and copies on the library's behalf."""
    import torch
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.current_stream(device) if stream is None else torch.cuda.ExternalStream(_stream(stream), device)


def decode(info: Info, d_blob, d_out, status=None, stream=None, blob_size: Optional[int] = None) -> None:
    """Asynchronously decode one blob already in device memory into d_out
    (torch uint8 CUDA tensors or raw device pointers) on ``stream``.  The
    bytes readable at d_blob are the tensor's size, or ``blob_size`` (which a
    raw pointer needs; it defaults to the blob's own size)."""
    size = _nbytes(d_blob, info.blob_bytes) if blob_size is None else int(blob_size)
    _check(_lib.ecf8_decode(ctypes.byref(info), _ptr(d_blob), size, _ptr(d_out), info.n, _ptr(status),
                            _stream(stream)), "ecf8_decode")


def batched_workspace_size(count: int) -> int:
    return int(_lib.ecf8_batched_workspace_size(count))


@dataclass
class BatchItem:
    info: Info
    d_blob: object
    d_out: object


def make_batch(items: Sequence[BatchItem]):
    """The ctypes array a batched decode takes; keep it alive while reused."""
    arr = (Tensor * len(items))()
    keep = []
    for i, it in enumerate(items):
        keep.append(it.info)
        arr[i].info = ctypes.pointer(it.info)
        arr[i].d_blob = _ptr(it.d_blob)
        arr[i].blob_size = _nbytes(it.d_blob, it.info.blob_bytes)
        arr[i].d_out = _ptr(it.d_out)
    return arr, keep


def decode_batched(items, workspace=None, status=None, stream=None, max_ctas: int = 0) -> None:
    """Decode several blobs in one kernel launch.  ``items`` is a list of
    BatchItem or the pair returned by make_batch.  ``max_ctas`` > 0 caps the
    persistent grid (one CTA per SM otherwise), leaving SMs to other kernels."""
    if isinstance(items, tuple):
        arr = items[0]
    else:
        arr, _keep = make_batch(items)
    ws = _ptr(workspace)
    ws_bytes = int(workspace.numel() * workspace.element_size()) if workspace is not None and not isinstance(
        workspace, int) else 0
    if max_ctas:
        _check(_lib.ecf8_decode_batched_ctas(arr, len(arr), ws, ws_bytes, _ptr(status), _stream(stream),
                                             int(max_ctas)), "ecf8_decode_batched_ctas")
    else:
        _check(_lib.ecf8_decode_batched(arr, len(arr), ws, ws_bytes, _ptr(status), _stream(stream)),
               "ecf8_decode_batched")


def decode_batched_noalloc(items, status=None, stream=None) -> None:
    """Like decode_batched, but with no workspace: the descriptor table lives
    in device memory the library holds (ECF8_NOALLOC_MAX_TENSORS entries), for
    callers that cannot allocate device memory while they decode.  Calls that
    can overlap on the GPU share that table and race; order them on one
    stream."""
    if isinstance(items, tuple):
        arr = items[0]
    else:
        arr, _keep = make_batch(items)
    _check(_lib.ecf8_decode_batched_noalloc(arr, len(arr), _ptr(status), _stream(stream)),
           "ecf8_decode_batched_noalloc")


@dataclass
class PipelineTensor:
    """One tensor of a pipeline layer: its blob info, device blob, and the
    byte offset of its FP8 output inside a slot (multiple of 16)."""
    info: Info
    d_blob: object
    out_offset: int


class Pipeline:
    """Decode-on-use over a fixed pool of slots (ecf8_pipeline_* in the C
    ABI): layer m is decoded into slot m % len(slots) on ``decode_stream``,
    ``depth`` layers ahead; ``acquire(l, stream)`` makes ``stream`` wait for
    layer l and returns its slot, ``release(l, stream)`` lets the slot be
    reused once the work already on ``stream`` is done."""

    def __init__(self, layers, slots, slot_bytes: int, depth: int = 1, max_ctas: int = 0, workspace=None,
                 status=None, decode_stream=None):
        self._slots = list(slots)
        self._keep = []
        n = len(layers)
        larr = (Layer * n)()
        for l, tensors in enumerate(layers):
            tarr = (LayerTensor * max(1, len(tensors)))()
            for i, t in enumerate(tensors):
                self._keep.append(t.info)
                tarr[i].info = ctypes.pointer(t.info)
                tarr[i].d_blob = _ptr(t.d_blob)
                tarr[i].blob_size = _nbytes(t.d_blob, t.info.blob_bytes)
                tarr[i].out_offset = int(t.out_offset)
            self._keep.append(tarr)
            larr[l].tensors = tarr
            larr[l].count = len(tensors)
        sarr = (ctypes.c_void_p * len(self._slots))(*[_ptr(x) for x in self._slots])
        ws = _ptr(workspace)
        ws_bytes = int(workspace.numel() * workspace.element_size()) if workspace is not None else 0
        self._decode_stream = decode_stream
        h = ctypes.c_void_p()
        _check(_lib.ecf8_pipeline_create(larr, n, sarr, len(self._slots), int(slot_bytes), int(depth),
                                         int(max_ctas), ws, ws_bytes, _ptr(status), _stream(decode_stream),
                                         ctypes.byref(h)), "ecf8_pipeline_create")
        self._h = h

    def acquire(self, layer: int, stream=None) -> int:
        """Device address of layer's slot; ``stream`` waits for its decode."""
        w = ctypes.c_void_p()
        _check(_lib.ecf8_pipeline_acquire(self._h, int(layer), _stream(stream), ctypes.byref(w)),
               "ecf8_pipeline_acquire")
        return int(w.value or 0)

    def release(self, layer: int, stream=None) -> None:
        _check(_lib.ecf8_pipeline_release(self._h, int(layer), _stream(stream)), "ecf8_pipeline_release")

    def close(self) -> None:
        if getattr(self, "_h", None):
            _lib.ecf8_pipeline_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()


# ---- BF16 variant: 8-bit exponent field coded, sign + mantissa byte kept ----

def _host_u16(x) -> np.ndarray:
    if hasattr(x, "detach"):  # a CPU torch tensor (bfloat16 or int16)
        import torch
        t = x.detach().contiguous().view(-1)
        if t.dtype != torch.int16:
            t = t.view(torch.int16)
        x = t.numpy()
    a = np.ascontiguousarray(np.asarray(x).reshape(-1))
    if a.dtype != np.uint16:
        a = a.view(np.uint16)
    return a


def bf16_code_lengths(x, max_len: int = 16) -> np.ndarray:
    """Code lengths (256 entries) for the exponent fields of BF16 bit patterns."""
    a = _host_u16(x)
    ln = np.zeros(256, dtype=np.uint8)
    _check(_lib.ecf8_bf16_code_lengths(a.ctypes.data, a.size, max_len, ln.ctypes.data), "ecf8_bf16_code_lengths")
    return ln


def bf16_encode(x, lengths=None, chunk_bytes: int = DEFAULT_CHUNK_BYTES, group_chunks: int = DEFAULT_GROUP_CHUNKS,
                max_len: int = 16) -> np.ndarray:
    """Compress BF16 weights (bit patterns as uint16, or a CPU bfloat16 tensor) into a blob."""
    a = _host_u16(x)
    ln = bf16_code_lengths(a, max_len) if lengths is None else np.ascontiguousarray(np.asarray(lengths, np.uint8))
    size = ctypes.c_size_t(0)
    _check(_lib.ecf8_bf16_encoded_size(a.ctypes.data, a.size, ln.ctypes.data, chunk_bytes, group_chunks,
                                       ctypes.byref(size)), "ecf8_bf16_encoded_size")
    blob = np.empty(size.value, dtype=np.uint8)
    got = ctypes.c_size_t(0)
    _check(_lib.ecf8_bf16_encode(a.ctypes.data, a.size, ln.ctypes.data, chunk_bytes, group_chunks, blob.ctypes.data,
                                 blob.size, ctypes.byref(got)), "ecf8_bf16_encode")
    assert got.value == blob.size
    return blob


def bf16_blob_info(blob) -> Bf16Info:
    b = _host_u8(blob)
    info = Bf16Info()
    _check(_lib.ecf8_bf16_blob_info(b.ctypes.data, b.size, ctypes.byref(info)), "ecf8_bf16_blob_info")
    return info


def bf16_table(info: Bf16Info) -> np.ndarray:
    """The decode table of info's code (host uint8 array; copy it to the device once)."""
    t = np.zeros(int(_lib.ecf8_bf16_table_bytes()), dtype=np.uint8)
    _check(_lib.ecf8_bf16_build_table(ctypes.byref(info), t.ctypes.data), "ecf8_bf16_build_table")
    return t


def bf16_table_nodes(info: Bf16Info) -> int:
    """Tree nodes of info's code; the node with this index is the table's error node."""
    return int(_lib.ecf8_bf16_table_nodes(ctypes.byref(info)))


def bf16_auto_layout(info: Bf16Info) -> str:
    """The table layout ``bf16_decode`` picks for info's code."""
    rc = _lib.ecf8_bf16_auto_layout(ctypes.byref(info))
    if rc < 0:
        raise Ecf8Error(rc, "ecf8_bf16_auto_layout")
    return {v: k for k, v in BF16_LAYOUTS.items()}[rc]


def bf16_decode(info: Bf16Info, d_blob, d_table, d_out, status=None, stream=None, layout: str = "auto") -> None:
    """Asynchronously decode one BF16 blob in device memory into d_out (n
    uint16/bfloat16 elements) with the device copy of ``bf16_table(info)``;
    ``layout`` forces one of the decoder's table layouts (same output)."""
    _check(_lib.ecf8_bf16_decode_layout(ctypes.byref(info), _ptr(d_blob), _ptr(d_table), _ptr(d_out), info.n,
                                        _ptr(status), _stream(stream), BF16_LAYOUTS[layout]), "ecf8_bf16_decode")


def bf16_decode_batched(items, status=None, stream=None) -> None:
    """Asynchronously decode several BF16 blobs: ``items`` is a sequence of
    (info, d_blob, d_table, d_out); one launch per table layout present."""
    infos = [it[0] for it in items]
    arr = (Bf16Tensor * max(1, len(items)))()
    for k, (info, d_blob, d_table, d_out) in enumerate(items):
        arr[k] = Bf16Tensor(ctypes.pointer(infos[k]), _ptr(d_blob), _ptr(d_table), _ptr(d_out))
    _check(_lib.ecf8_bf16_decode_batched(arr, len(items), _ptr(status), _stream(stream)), "ecf8_bf16_decode_batched")


# ---- linear layers over decoded weights, with low-rank adapters ----

_DTYPES = {"torch.bfloat16": 0, "torch.float16": 1, "torch.float32": 2}


def _refuse(what: str, why: str):
    raise Ecf8Error(-1, f"{what}: {why}")


def _dtype_of(t, what: str) -> int:
    d = _DTYPES.get(str(t.dtype))
    if d is None:
        _refuse(what, f"{t.dtype} is not bfloat16, float16 or float32")
    return d


def _is(t, what: str, dtype, shape) -> None:
    """A contiguous tensor of this type and shape."""
    if t.dtype is not dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        _refuse(what, f"want a contiguous {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _rows(t, what: str, dtype, rows: int, cols: int) -> int:
    """The row stride of a rows x cols tensor whose rows are contiguous."""
    if t.dtype is not dtype or t.shape != (rows, cols):
        _refuse(what, f"want {dtype} of shape {(rows, cols)}, got {t.dtype} {tuple(t.shape)}")
    stride, inner = t.stride()
    if inner != 1 and cols > 1:
        _refuse(what, f"rows of {cols} values have to be contiguous, got a stride of {inner}")
    return stride if rows > 1 else max(stride, cols)


def _here(what: str, device, tensors) -> None:
    """Every tensor on this CUDA device, which is the current one: the kernels
    run there, and reach no other device's memory."""
    import torch
    if device.type != "cuda" or device.index != torch._C._cuda_getDevice():
        _refuse(what, f"tensors are on {device}, which is not the current CUDA device")
    for t in tensors:
        if t is not None and not isinstance(t, int) and t.device != device:
            _refuse(what, f"tensors on {device} and {t.device}")


@dataclass
class Adapters:
    """Low-rank adapters of one projection: a (count, rank, in), b (count,
    out, rank) in the activations' type, alpha (count) float32."""
    a: object
    b: object
    alpha: object


@dataclass
class Requests:
    """Runs of rows and the adapter of each: request i is rows offsets[i] to
    offsets[i+1]-1 and uses adapter ids[i] (negative: none).  CUDA int32
    tensors of count + 1 and count values."""
    offsets: object
    ids: object


class LinearDesc(ctypes.Structure):
    _fields_ = [("d_w", _p), ("n_out", ctypes.c_uint64), ("k_in", ctypes.c_uint64), ("w_stride", ctypes.c_uint64),
                ("d_scale", _p), ("n_scale", ctypes.c_uint64), ("d_a", _p), ("d_b", _p), ("d_alpha", _p),
                ("n_adapters", _u32), ("rank", _u32), ("dtype", ctypes.c_int32)]


class RequestsDesc(ctypes.Structure):
    _fields_ = [("d_offsets", _p), ("d_ids", _p), ("count", _u32)]


_u64 = ctypes.c_uint64
_lib.ecf8_linear_workspace_size.argtypes = [ctypes.POINTER(LinearDesc), _u64]
_lib.ecf8_linear_workspace_size.restype = _sz
_lib.ecf8_linear_tile_ctas.argtypes = [ctypes.POINTER(LinearDesc), _u64, _i32]
_lib.ecf8_linear_forward.argtypes = [ctypes.POINTER(LinearDesc), ctypes.POINTER(RequestsDesc), _p, _u64, _p, _u64, _u64,
                                     _p, _p, _sz, _p, _p]
_lib.ecf8_linear_backward.argtypes = [ctypes.POINTER(LinearDesc), ctypes.POINTER(RequestsDesc), _p, _u64, _p, _u64, _p,
                                      _p, _u64, _p, _p, _u64, _p, _sz, _p, _p]


class Linear:
    """y = scale * (x W^T) over decoded E4M3 weights, with the low-rank
    adapters of many requests added (ecf8_linear_* in the C ABI).

    ``weight`` is a CUDA uint8 or float8_e4m3fn tensor (out, in) with contiguous rows, or the
    address at which a decode writes it (as ``Pipeline.acquire`` returns, plus
    the tensor's offset) with ``shape`` given.  ``scale``: float32 CUDA tensor
    of 1 or ``out`` values, or None.  ``dtype``: torch.bfloat16 or
    torch.float16, the type of activations, adapters and gradients.  The
    object keeps references and addresses; it holds no copy."""

    def __init__(self, weight, shape=None, scale=None, adapters: Optional[Adapters] = None, dtype=None):
        import torch
        d = LinearDesc()
        dtype = torch.bfloat16 if dtype is None else dtype
        if str(dtype) not in ("torch.bfloat16", "torch.float16"):
            _refuse("Linear", f"dtype {dtype} is not bfloat16 or float16")
        if isinstance(weight, int):
            if shape is None:
                _refuse("Linear", "a weight address needs a shape")
            n, k = (int(v) for v in shape)
            d.w_stride = k
        else:
            if weight.dim() != 2 or (shape is not None and tuple(shape) != tuple(weight.shape)):
                _refuse("Linear", f"want a weight of 2 dimensions, got {tuple(weight.shape)}")
            n, k = weight.shape
            if weight.dtype not in (torch.uint8, torch.float8_e4m3fn):  # other bytes mean other values
                _refuse("Linear", f"weights are E4M3 bytes, got {weight.dtype}")
            d.w_stride = _rows(weight, "Linear weight", weight.dtype, n, k)
        d.d_w, d.n_out, d.k_in, d.dtype = _ptr(weight), n, k, _DTYPES[str(dtype)]
        if scale is not None:
            if str(scale.dtype) != "torch.float32" or scale.numel() not in (1, n) or not scale.is_contiguous():
                _refuse("Linear", f"scale: want 1 or {n} contiguous float32, got {scale.dtype} {tuple(scale.shape)}")
            d.d_scale, d.n_scale = _ptr(scale), scale.numel()
        self.rank = 0
        if adapters is not None and adapters.a.shape[0]:
            count, self.rank = (int(v) for v in adapters.a.shape[:2])
            _is(adapters.a, "Linear adapters a", dtype, (count, self.rank, k))
            _is(adapters.b, "Linear adapters b", dtype, (count, n, self.rank))
            _is(adapters.alpha, "Linear adapters alpha", torch.float32, (count,))
            d.d_a, d.d_b, d.d_alpha = _ptr(adapters.a), _ptr(adapters.b), _ptr(adapters.alpha)
            d.n_adapters, d.rank = count, self.rank
        self.n_out, self.k_in, self.dtype = int(n), int(k), dtype
        self._keep, self._d, self._ref = (weight, scale, adapters), d, ctypes.byref(d)
        self._f32, self._i32 = torch.float32, torch.int32
        self._own = [t for t in (weight, scale, *((adapters.a, adapters.b, adapters.alpha) if self.rank else ()))
                     if t is not None and not isinstance(t, int)]
        if any(t.device != self._own[0].device for t in self._own):
            _refuse("Linear", f"tensors on {[str(t.device) for t in self._own]}")

    def workspace_size(self, rows: int) -> int:
        """Bytes of device workspace forward and backward need for this many rows."""
        return int(_lib.ecf8_linear_workspace_size(self._ref, rows))

    def tile_ctas(self, rows: int, backward: bool = False) -> int:
        """CTAs that share a tile of the projection, or of its input gradient, in a call of this many rows."""
        return int(_lib.ecf8_linear_tile_ctas(self._ref, rows, int(backward)))

    def _requests(self, q):
        if q is None:
            return None
        ids, offsets = q.ids, q.offsets
        count = ids.numel()
        _is(ids, "Requests ids", self._i32, (count,))
        _is(offsets, "Requests offsets", self._i32, (count + 1,))
        return RequestsDesc(offsets.data_ptr(), ids.data_ptr(), count)

    def forward(self, x, y, requests: Optional[Requests] = None, u=None, workspace=None, status=None,
                stream=None) -> None:
        """Asynchronously writes y (rows, out) for x (rows, in).  ``u`` (rows,
        rank) float32 keeps A x for ``backward``."""
        rows = x.shape[0]
        xs = _rows(x, "Linear x", self.dtype, rows, self.k_in)
        ys = _rows(y, "Linear y", self.dtype, rows, self.n_out)
        if u is not None:
            _is(u, "Linear u", self._f32, (rows, self.rank))
        q = self._requests(requests)
        _here("Linear forward", x.device, (y, u, workspace, status, *self._own[:1]))
        if requests is not None:
            _here("Linear forward", x.device, (requests.offsets, requests.ids))
        _check(_lib.ecf8_linear_forward(self._ref, q, _ptr(x), xs, _ptr(y), ys, rows, _ptr(u),
                                        _ptr(workspace), _nbytes(workspace, 0), _ptr(status), _stream(stream)),
               "ecf8_linear_forward")

    def backward(self, x, dy, u, dx=None, da=None, db=None, requests: Optional[Requests] = None, workspace=None,
                 status=None, stream=None) -> None:
        """Asynchronously writes the gradients that are given a tensor: dx
        (rows, in), da and db (as the adapters' a and b), from dy (rows, out),
        the forward pass's x (for da) and u (for db)."""
        rows = dy.shape[0]
        ds = _rows(dy, "Linear dy", self.dtype, rows, self.n_out)
        xs = _rows(x, "Linear x", self.dtype, rows, self.k_in) if x is not None else self.k_in
        gs = _rows(dx, "Linear dx", self.dtype, rows, self.k_in) if dx is not None else self.k_in
        if u is not None:
            _is(u, "Linear u", self._f32, (rows, self.rank))
        for g, of, what in ((da, "a", "Linear da"), (db, "b", "Linear db")):
            if g is not None:
                if not self.rank:
                    _refuse(what, "there are no adapters")
                _is(g, what, self.dtype, getattr(self._keep[2], of).shape)
        q = self._requests(requests)
        _here("Linear backward", dy.device, (x, u, dx, da, db, workspace, status, *self._own[:1]))
        if requests is not None:
            _here("Linear backward", dy.device, (requests.offsets, requests.ids))
        _check(_lib.ecf8_linear_backward(self._ref, q, _ptr(x), xs, _ptr(dy), ds, _ptr(u),
                                         _ptr(dx), gs, _ptr(da), _ptr(db), rows, _ptr(workspace),
                                         _nbytes(workspace, 0), _ptr(status), _stream(stream)),
               "ecf8_linear_backward")


# ---- the global norm of a set of gradients, and clipping ----

class Grad(ctypes.Structure):
    _fields_ = [("d_in", _p), ("d_out", _p), ("n", _u64), ("dtype", ctypes.c_int32)]


_lib.ecf8_grad_table_bytes.argtypes = [_i32]
_lib.ecf8_grad_table_bytes.restype = _sz
_lib.ecf8_grad_build_table.argtypes = [ctypes.POINTER(Grad), _i32, _p]
_lib.ecf8_grad_workspace_size.restype = _sz
_lib.ecf8_grad_norm.argtypes = [_p, _p, _p, _p, _sz, _p, _p]
_lib.ecf8_grad_clip.argtypes = [_p, _p, ctypes.c_float, _p, _p, _sz, _p, _p]


class GradSet:
    """A set of gradient tensors (contiguous CUDA bfloat16, float16 or float32,
    mixed as they come) whose global L2 norm is taken, and which are clipped by
    it, in one call (ecf8_grad_* in the C ABI).  ``outs`` (same sizes and
    types) receives the clipped values; by default they are written in place.
    None in the place of an output: only the norm is wanted, and tensors may
    share memory.
    The descriptor table is laid out and copied to the device here, once, at
    some 2 us a tensor on the host (448 tensors: 0.8 ms, a call on them 32 us
    on the GPU): a set is for tensors that stay where they are.  Calls that can overlap on the GPU
    need sets of their own.  A set may be dropped once its calls are made; on a
    stream given by its number, or captured into a graph, it has to live as
    long as they can run."""

    def __init__(self, grads, outs=None):
        import torch
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if len(outs) != len(grads):
            _refuse("GradSet", f"{len(grads)} tensors, {len(outs)} outputs")
        arr = (Grad * max(1, len(grads)))()
        for i, (g, o) in enumerate(zip(grads, outs)):
            if not g.is_contiguous() or (o is not None and (not o.is_contiguous() or o.dtype != g.dtype
                                                            or o.numel() != g.numel())):
                _refuse("GradSet", f"tensor {i}: want contiguous tensors, the output of the same type and size")
            arr[i] = Grad(_ptr(g), _ptr(o), g.numel(), _dtype_of(g, f"GradSet tensor {i}"))
        self._h = np.zeros(int(_lib.ecf8_grad_table_bytes(len(grads))), dtype=np.uint8)
        _check(_lib.ecf8_grad_build_table(arr, len(grads), self._h.ctypes.data), "ecf8_grad_build_table")
        dev = grads[0].device if grads else torch.device("cuda", torch._C._cuda_getDevice())
        _here("GradSet", dev, (*grads, *outs))
        self._device = dev
        self._d = torch.from_numpy(self._h).to(dev)
        self._ws = torch.empty(int(_lib.ecf8_grad_workspace_size()), dtype=torch.uint8, device=dev)
        self._keep = (grads, outs)
        self._args = (self._h.ctypes.data, _ptr(self._d))
        self._ws_args = (_ptr(self._ws), self._ws.numel())
        self._streams = {_stream(None)}  # those that the table's and the workspace's memory is known to serve

    def _on(self, stream) -> int:
        """The stream's number; the set's memory is not given to another use before the stream is done with it."""
        number = _stream(stream)
        if number not in self._streams and not isinstance(stream, int):
            stream = _torch_stream(stream, self._device)
            self._d.record_stream(stream)
            self._ws.record_stream(stream)
            self._streams.add(number)
        return number

    def _one(self, norm, status) -> None:
        if str(norm.dtype) != "torch.float32" or norm.numel() != 1:
            _refuse("GradSet norm", f"want one float32, got {norm.dtype} {tuple(norm.shape)}")
        _here("GradSet", self._device, (norm, status))

    def norm(self, norm, status=None, stream=None) -> None:
        """Asynchronously writes the L2 norm of the whole set to ``norm`` (one float32)."""
        self._one(norm, status)
        _check(_lib.ecf8_grad_norm(*self._args, _ptr(norm), *self._ws_args, _ptr(status),
                                   self._on(stream)), "ecf8_grad_norm")

    def clip(self, max_norm: float, norm, status=None, stream=None) -> None:
        """``norm``, then every tensor times min(1, max_norm / (norm + 1e-6)).
        A norm that is not finite sets ECF8_STATUS_NONFINITE and changes no value."""
        self._one(norm, status)
        _check(_lib.ecf8_grad_clip(*self._args, float(max_norm), _ptr(norm), *self._ws_args, _ptr(status),
                                   self._on(stream)), "ecf8_grad_clip")
