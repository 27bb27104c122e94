"""Python binding of libmla_decode.so (include/mla_decode.h and include/mla_kv8.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  Tensors must already live on the current CUDA
device; outputs, metadata and scratch are torch allocations owned by the
caller.  There is no CPU path: if the library is missing or no GPU is present
the calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import math
import threading
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libmla_decode.so"
D_QK, D_V, BLOCK_SIZE = 576, 512, 64

_lib = None


class MLAError(RuntimeError):
    pass


def load_library():
    """Loads libmla_decode.so (built by mla_decode_attention_03_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not LIB_PATH.exists():
        raise MLAError(f"{LIB_PATH} is missing: build it with "
                       "`python -m mla_decode_attention_03_gb300.build` (needs nvcc for sm_103a)")
    lib = ctypes.CDLL(str(LIB_PATH))
    P, I, I64, SZ, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_status_string.argtypes = [ctypes.c_int32]
    lib.mla_num_parts.restype = I
    lib.mla_num_parts.argtypes = [I, I, I, I]
    lib.mla_metadata_ints.restype = SZ
    lib.mla_metadata_ints.argtypes = [I]
    lib.mla_workspace_bytes.restype = SZ
    lib.mla_workspace_bytes.argtypes = [I, I, I, I]
    lib.mla_get_metadata.restype = ctypes.c_int32
    lib.mla_get_metadata.argtypes = [P, I, I, P, P, P, P]
    for name in ("mla_decode_with_kvcache", "mla_decode_splitkv", "mla_selftest_wait_timeout"):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int32
        fn.argtypes = [P, I, I, I, I, P, I64, I, I, I, P, I, P, I, P, I, P, F, I, P, P, P, SZ, P, P]
    lib.mla_combine_splits.restype = ctypes.c_int32
    lib.mla_combine_splits.argtypes = [P, I, I, I, P, I, P, P, P]
    lib.mla_write_cache.restype = ctypes.c_int32
    lib.mla_write_cache.argtypes = [P, I64, P, I64, P, I64, P, I64, I, I, P, P]
    lib.mla_copy_blocks.restype = ctypes.c_int32
    lib.mla_copy_blocks.argtypes = [P, I, P, I64, I64, I, I, P, P]
    lib.mla_host_pipeline_create.restype = ctypes.c_int32
    lib.mla_host_pipeline_create.argtypes = [ctypes.POINTER(P)]
    lib.mla_host_pipeline_destroy.restype = ctypes.c_int32
    lib.mla_host_pipeline_destroy.argtypes = [P]
    lib.mla_host_chunks.restype = I
    lib.mla_host_chunks.argtypes = [P, I, I, P]
    lib.mla_host_scratch_bytes.restype = SZ
    lib.mla_host_scratch_bytes.argtypes = [I, I, I, I, I]
    lib.mla_decode_host.restype = ctypes.c_int32
    lib.mla_decode_host.argtypes = [P, P, I, I, I, I, P, I64, I, I, I, P, I, P, I, I, F, I, P, P, I, P, SZ, P, P]
    lib.mla_write_cache_kv8.restype = ctypes.c_int32
    lib.mla_write_cache_kv8.argtypes = [P, I64, P, I64, P, I64, P, P, I64, I, I, P, P]
    lib.mla_read_cache_kv8.restype = ctypes.c_int32
    lib.mla_read_cache_kv8.argtypes = [P, P, I64, I, I, P, I, P, P, I, P, I64, P, P]
    lib.mla_num_parts_kv8.restype = I
    lib.mla_num_parts_kv8.argtypes = [I, I, I, I]
    lib.mla_workspace_bytes_kv8.restype = SZ
    lib.mla_workspace_bytes_kv8.argtypes = [I, I, I, I, I]
    lib.mla_decode_kv8.restype = ctypes.c_int32
    lib.mla_decode_kv8.argtypes = [P, I, I, I, I, P, P, I64, I, I, I, P, I, P, I, P, I, P, F, I, P, P, P, SZ, P, P]
    lib.mla_rope.restype = ctypes.c_int32
    lib.mla_rope.argtypes = [P, I64, I64, P, I64, I64, I, P, I64, I64, P, I64, I64, I, I64, I, P, I, P, F, I, I, I, P]
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().mla_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != 0:
        raise MLAError(f"{what}: {status_string(code)} ({code})")


def _stream_handle() -> int:
    return torch.cuda.current_stream().cuda_stream


def num_parts(s_q: int, h_q: int, h_kv: int = 1, device=None) -> int:
    dev = torch.cuda.current_device() if device is None else torch.device(device).index or 0
    n = load_library().mla_num_parts(s_q, h_q, h_kv, dev)
    if n < 0:
        _check(n, "mla_num_parts")
    return n


def workspace_bytes(b: int, s_q: int, h_q: int, parts: int) -> int:
    return int(load_library().mla_workspace_bytes(b, s_q, h_q, parts))


def new_status(device=None) -> torch.Tensor:
    """A zeroed device status word for the calls below."""
    return torch.zeros(1, dtype=torch.int32, device=device or torch.cuda.current_device())


_shared_status: dict[int, torch.Tensor] = {}
_shared_status_lock = threading.Lock()


def _status_of_device(device: torch.device) -> torch.Tensor:
    """The word that calls on the 8-bit cache without one of their own report to: made once per device, so that they
    neither allocate nor fill.  (A first call inside a stream capture gets a word of the capture's own.)"""
    word = _shared_status.get(device.index)
    if word is None:
        with torch.cuda.device(device):
            if torch.cuda.is_current_stream_capturing():
                return new_status(device)
            with _shared_status_lock:
                word = _shared_status.get(device.index)
                if word is None:
                    word = new_status(device)
                    torch.cuda.current_stream().synchronize()  # zero before any stream's kernel may report
                    _shared_status[device.index] = word
    return word


def check_status(status: torch.Tensor | None = None):
    """Synchronises on the status word and raises if a kernel reported an error.  Without a word: waits for the current
    device and looks at what the calls on the 8-bit cache that were given none reported there, clearing it."""
    shared = status is None
    if shared:
        status = _shared_status.get(torch.cuda.current_device())
        if status is None:
            return
        torch.cuda.synchronize(status.device)
    code = int(status.item())
    if code != 0:
        if shared:
            status.zero_()
            torch.cuda.current_stream(status.device).synchronize()
        raise MLAError(f"device reported {status_string(code)} ({code})")


def get_mla_metadata(cache_seqlens: torch.Tensor, parts: int, status: torch.Tensor | None = None):
    """Split-KV schedule: returns (metadata int32[parts, 8], num_splits int32[b+1])."""
    assert cache_seqlens.is_cuda and cache_seqlens.dtype == torch.int32 and cache_seqlens.dim() == 1
    sl = cache_seqlens.contiguous()
    b = sl.shape[0]
    meta = torch.empty((parts, 8), dtype=torch.int32, device=sl.device)
    nsplit = torch.empty((b + 1,), dtype=torch.int32, device=sl.device)
    if status is None:
        status = new_status(sl.device)
    _check(load_library().mla_get_metadata(sl.data_ptr(), b, parts, meta.data_ptr(), nsplit.data_ptr(),
                                           status.data_ptr(), _stream_handle()), "mla_get_metadata")
    return meta, nsplit


def entry_stride(kcache: torch.Tensor) -> int:
    """Elements between consecutive entries of a [num_blocks, 64, h_kv, 576]
    cache view (576 when dense, 640 for the 256-byte aligned layout)."""
    nb, bs, h_kv, d = kcache.shape
    st = kcache.stride()
    es = st[2] if h_kv > 1 else st[1]
    if st[3] != 1 or st[1] != h_kv * es or st[0] != bs * st[1]:
        raise MLAError(f"kcache layout not supported: shape {tuple(kcache.shape)}, strides {st}")
    return es


def _check_io(q, block_table, cache_seqlens, out, lse, dv=D_V):
    """Shapes, types and layouts of the per-sequence arrays against q
    [b, s_q, h_q, d]: the library reads and writes exactly these extents, so a
    smaller tensor must be refused here, before its pointer is handed over."""
    if q.dim() != 4:
        raise MLAError(f"q must be [b, s_q, h_q, d], got shape {tuple(q.shape)}")
    b, s_q, h_q, _ = q.shape
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.shape[0] != b:
        raise MLAError(f"block_table must be int32 [{b}, max_blocks], got {block_table.dtype} "
                       f"{tuple(block_table.shape)}")
    if cache_seqlens.dtype != torch.int32 or tuple(cache_seqlens.shape) != (b,):
        raise MLAError(f"cache_seqlens must be int32 [{b}], got {cache_seqlens.dtype} {tuple(cache_seqlens.shape)}")
    for name, t, shape, dtype in (("out", out, (b, s_q, h_q, dv), torch.bfloat16),
                                  ("lse", lse, (b, h_q, s_q), torch.float32)):
        if t is None:
            continue
        if tuple(t.shape) != shape or t.dtype != dtype or not t.is_contiguous():
            raise MLAError(f"{name} must be a contiguous {dtype} tensor of shape {shape}, got {t.dtype} "
                           f"{tuple(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'}")
        if t.device != q.device:
            raise MLAError(f"{name} must be on {q.device}")


def mla_decode_with_kvcache(q: torch.Tensor, kcache: torch.Tensor, block_table: torch.Tensor,
                            cache_seqlens: torch.Tensor, metadata: torch.Tensor,
                            num_splits: torch.Tensor, softmax_scale: float, causal: bool = False,
                            dv: int = D_V, out: torch.Tensor | None = None,
                            lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                            status: torch.Tensor | None = None, combine: bool = True):
    """MLA decode: returns (out bf16[b, s_q, h_q, 512], lse fp32[b, h_q, s_q]).

    combine=False runs only the split-KV decode kernel (mla_decode_splitkv);
    combine_splits() must then follow on the same stream."""
    if not (q.is_cuda and kcache.is_cuda):
        raise MLAError("q and kcache must be CUDA tensors")
    if q.dtype != torch.bfloat16 or kcache.dtype != torch.bfloat16:
        raise MLAError("q and kcache must be bfloat16")
    if not q.is_contiguous():
        raise MLAError("q must be contiguous")
    _check_io(q, block_table, cache_seqlens, out, lse, dv)
    b, s_q, h_q, d = q.shape
    nb, bs, h_kv, dk = kcache.shape
    stride = entry_stride(kcache)
    bt = block_table.contiguous()
    sl = cache_seqlens.contiguous()
    if not (bt.device == sl.device == kcache.device == q.device):
        raise MLAError("q, kcache, block_table and cache_seqlens must be on one device")
    if tuple(num_splits.shape) != (b + 1,) or metadata.dim() != 2 or metadata.shape[1] != 8:
        raise MLAError("metadata / num_splits do not come from get_mla_metadata for this batch")
    parts = metadata.shape[0]
    dev = q.device
    if out is None:
        out = torch.empty((b, s_q, h_q, dv), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((b, h_q, s_q), dtype=torch.float32, device=dev)
    need = workspace_bytes(b, s_q, h_q, parts)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if status is None:
        status = new_status(dev)
    lib = load_library()
    fn = lib.mla_decode_with_kvcache if combine else lib.mla_decode_splitkv
    rc = fn(
        q.data_ptr(), b, s_q, h_q, d, kcache.data_ptr(), nb, bs, h_kv, stride, bt.data_ptr(),
        bt.shape[1], sl.data_ptr(), dv, metadata.data_ptr(), parts, num_splits.data_ptr(),
        float(softmax_scale), int(bool(causal)), out.data_ptr(), lse.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), status.data_ptr(),
        _stream_handle())
    _check(rc, "mla_decode_with_kvcache" if combine else "mla_decode_splitkv")
    return out, lse


def combine_splits(num_splits: torch.Tensor, workspace: torch.Tensor, parts: int, out: torch.Tensor,
                   lse: torch.Tensor):
    """The merge half of mla_decode_with_kvcache (mla_combine_splits)."""
    if out.dim() != 4 or out.shape[3] != D_V or out.dtype != torch.bfloat16 or not out.is_contiguous():
        raise MLAError(f"out must be a contiguous bfloat16 [b, s_q, h_q, {D_V}] tensor")
    b, s_q, h_q, _ = out.shape
    if (tuple(lse.shape) != (b, h_q, s_q) or lse.dtype != torch.float32 or not lse.is_contiguous()
            or lse.device != out.device):
        raise MLAError(f"lse must be a contiguous float32 [{b}, {h_q}, {s_q}] tensor on {out.device}")
    if tuple(num_splits.shape) != (b + 1,):
        raise MLAError(f"num_splits must have {b + 1} entries")
    if workspace.numel() * workspace.element_size() < workspace_bytes(b, s_q, h_q, parts):
        raise MLAError("workspace smaller than mla_workspace_bytes for this shape")
    _check(load_library().mla_combine_splits(num_splits.data_ptr(), b, s_q, h_q, workspace.data_ptr(),
                                             parts, out.data_ptr(), lse.data_ptr(), _stream_handle()),
           "mla_combine_splits")
    return out, lse


def write_cache(kv_c: torch.Tensor, k_pe: torch.Tensor, slot_mapping: torch.Tensor, kcache: torch.Tensor,
                status: torch.Tensor | None = None):
    """New tokens into the paged cache: entry slot_mapping[t] <- [kv_c[t], k_pe[t]]
    (mla_write_cache).  kcache is the [num_blocks, 64, 1, 576] view of the cache."""
    if kv_c.dtype != torch.bfloat16 or k_pe.dtype != torch.bfloat16 or kcache.dtype != torch.bfloat16:
        raise MLAError("kv_c, k_pe and kcache must be bfloat16")
    if kv_c.stride(-1) != 1 or k_pe.stride(-1) != 1:
        raise MLAError("kv_c and k_pe rows must be contiguous")
    if kv_c.shape[-1] != 512 or k_pe.shape[-1] != 64 or kv_c.dim() != 2 or k_pe.dim() != 2:
        raise MLAError("kv_c must be [T, 512] and k_pe [T, 64]")
    if kv_c.shape[0] != k_pe.shape[0] or slot_mapping.numel() != kv_c.shape[0]:
        raise MLAError("kv_c, k_pe and slot_mapping must have one row per token")
    if kv_c.device != kcache.device or k_pe.device != kcache.device:
        raise MLAError("kv_c, k_pe and kcache must be on one device")
    sm = slot_mapping.to(device=kcache.device, dtype=torch.int64).contiguous()
    nb, bs, h_kv, _ = kcache.shape
    if h_kv != 1:
        raise MLAError("MLA caches have one latent head")
    if status is None:
        status = new_status(kcache.device)
    _check(load_library().mla_write_cache(kv_c.data_ptr(), kv_c.stride(0), k_pe.data_ptr(), k_pe.stride(0),
                                          sm.data_ptr(), sm.numel(), kcache.data_ptr(), nb, bs,
                                          entry_stride(kcache), status.data_ptr(), _stream_handle()),
           "mla_write_cache")
    return kcache


def copy_blocks(kcaches: list, block_mapping: torch.Tensor, status: torch.Tensor | None = None):
    """copy_blocks_mla: for every layer cache and (src, dst) pair, page dst <- page src."""
    if not kcaches:
        return kcaches
    nb, bs, h_kv, _ = kcaches[0].shape
    stride = entry_stride(kcaches[0])
    for c in kcaches:
        if c.dtype != torch.bfloat16 or c.device != kcaches[0].device:
            raise MLAError("layer caches must be bfloat16 tensors on one device")
        if c.shape != kcaches[0].shape or entry_stride(c) != stride:
            raise MLAError("all layer caches must share one shape and entry stride")
    dev = kcaches[0].device
    ptrs = torch.tensor([c.data_ptr() for c in kcaches], dtype=torch.int64, device=dev)
    bm = block_mapping.to(device=dev, dtype=torch.int64).contiguous()
    if bm.dim() != 2 or bm.shape[1] != 2:
        raise MLAError(f"block_mapping must be [num_pairs, 2], got {tuple(bm.shape)}")
    if status is None:
        status = new_status(dev)
    _check(load_library().mla_copy_blocks(ptrs.data_ptr(), len(kcaches), bm.data_ptr(), bm.shape[0], nb, bs,
                                          stride, status.data_ptr(), _stream_handle()), "mla_copy_blocks")
    return kcaches


class MLADecoder:
    """Holds the per-step schedule, scratch and status word for one decode shape.

    plan(cache_seqlens) once per decode step (the schedule is shared by all
    layers), then __call__ once per layer."""

    def __init__(self, b: int, s_q: int, h_q: int, h_kv: int = 1, device=None, parts: int | None = None):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.b, self.s_q, self.h_q, self.h_kv = b, s_q, h_q, h_kv
        self.parts = parts if parts is not None else num_parts(s_q, h_q, h_kv, self.device)
        self.workspace = torch.empty((workspace_bytes(b, s_q, h_q, self.parts),), dtype=torch.uint8,
                                     device=self.device)
        self.status = new_status(self.device)
        self.metadata = None
        self.num_splits = None

    def plan(self, cache_seqlens: torch.Tensor):
        self.metadata, self.num_splits = get_mla_metadata(cache_seqlens, self.parts, self.status)
        return self

    def __call__(self, q, kcache, block_table, cache_seqlens, softmax_scale, causal=False, out=None, lse=None):
        return mla_decode_with_kvcache(q, kcache, block_table, cache_seqlens, self.metadata,
                                       self.num_splits, softmax_scale, causal, out=out, lse=lse,
                                       workspace=self.workspace, status=self.status)


HOST_MAX_CHUNKS = 8  # MLA_HOST_MAX_CHUNKS


def host_chunks(cache_seqlens: torch.Tensor, chunks: int = 0) -> list:
    """The cut of a batch into runs of consecutive sequences that the
    host-buffer decode makes (mla_host_chunks): sequence bounds [0, ..., b]."""
    sl = cache_seqlens.to(torch.int32).contiguous()
    assert sl.device.type == "cpu" and sl.dim() == 1
    bounds = (ctypes.c_int32 * (HOST_MAX_CHUNKS + 1))()
    n = load_library().mla_host_chunks(sl.data_ptr(), sl.shape[0], int(chunks), ctypes.addressof(bounds))
    if n < 0:
        _check(n, "mla_host_chunks")
    return list(bounds[: n + 1])


class HostDecoder:
    """Decode from host tensors (mla_decode_host): q, block_table and
    cache_seqlens are CPU tensors (pinned for the copies to overlap), out and
    lse come back in CPU tensors; the KV cache stays on the device.  The batch
    is cut into runs of sequences whose copies in and out overlap the decode
    of the neighbouring runs.  Holds the pipeline's streams and events and the
    device staging scratch for batches up to (b, s_q, h_q, max_blocks_per_seq).

    The call returns once the work is enqueued on the current stream: keep the
    host tensors alive and unchanged, and read out/lse only after
    torch.cuda.current_stream().synchronize() (or check_status(self.status))."""

    def __init__(self, b: int, s_q: int, h_q: int, max_blocks_per_seq: int, h_kv: int = 1, device=None,
                 parts: int | None = None):
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.b, self.s_q, self.h_q, self.h_kv, self.max_blocks = b, s_q, h_q, h_kv, max_blocks_per_seq
        self.parts = parts if parts is not None else num_parts(s_q, h_q, h_kv, self.device)
        lib = load_library()
        self._handle = None
        with torch.cuda.device(self.device):
            h = ctypes.c_void_p()
            _check(lib.mla_host_pipeline_create(ctypes.byref(h)), "mla_host_pipeline_create")
            self._handle = h
        n = lib.mla_host_scratch_bytes(b, s_q, h_q, max_blocks_per_seq, self.parts)
        if n == 0:
            raise MLAError("mla_host_scratch_bytes: invalid shape")
        # zeroed once: no run can ever see stale schedule words, whatever was in the memory before
        self.scratch = torch.zeros((n,), dtype=torch.uint8, device=self.device)
        self.status = new_status(self.device)

    def __call__(self, q, kcache, block_table, cache_seqlens, softmax_scale, causal=False, out=None, lse=None,
                 chunks: int = 0):
        if self._handle is None:
            raise MLAError("HostDecoder is closed")
        for name, t in (("q", q), ("block_table", block_table), ("cache_seqlens", cache_seqlens)):
            if t.device.type != "cpu" or not t.is_contiguous():
                raise MLAError(f"{name} must be a contiguous CPU tensor")
        if q.dtype != torch.bfloat16 or kcache.dtype != torch.bfloat16 or not kcache.is_cuda:
            raise MLAError("q must be bfloat16 on the host and kcache bfloat16 on the device")
        if block_table.dtype != torch.int32 or cache_seqlens.dtype != torch.int32:
            raise MLAError("block_table and cache_seqlens must be int32")
        _check_io(q, block_table, cache_seqlens, out, lse)
        b, s_q, h_q, d = q.shape
        if b > self.b or s_q != self.s_q or h_q != self.h_q or block_table.shape[1] > self.max_blocks:
            raise MLAError(f"shape {tuple(q.shape)} / max_blocks {block_table.shape[1]} outside the decoder's "
                           f"({self.b}, {self.s_q}, {self.h_q}) / {self.max_blocks}")
        nb, bs, h_kv, dk = kcache.shape
        stride = entry_stride(kcache)
        if out is None:
            out = torch.empty((b, s_q, h_q, D_V), dtype=torch.bfloat16, pin_memory=True)
        if lse is None:
            lse = torch.empty((b, h_q, s_q), dtype=torch.float32, pin_memory=True)
        if out.device.type != "cpu" or lse.device.type != "cpu" or not (out.is_contiguous() and lse.is_contiguous()):
            raise MLAError("out and lse must be contiguous CPU tensors")
        with torch.cuda.device(self.device):
            rc = load_library().mla_decode_host(
                self._handle, q.data_ptr(), b, s_q, h_q, d, kcache.data_ptr(), nb, bs, h_kv, stride,
                block_table.data_ptr(), block_table.shape[1], cache_seqlens.data_ptr(), D_V, self.parts,
                float(softmax_scale), int(bool(causal)), out.data_ptr(), lse.data_ptr(), int(chunks),
                self.scratch.data_ptr(), self.scratch.numel(), self.status.data_ptr(), _stream_handle())
        _check(rc, "mla_decode_host")
        return out, lse

    def close(self):
        if self._handle is not None:
            h, self._handle = self._handle, None
            _check(load_library().mla_host_pipeline_destroy(h), "mla_host_pipeline_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- 8-bit cache
# The cache of include/mla_kv8.h: float8_e4m3fn [num_blocks, 64, h_kv, 576] (dense, or a view of padded entries) and
# float32 scales [num_blocks, h_kv, 64], one per token and head.
FP8 = torch.float8_e4m3fn


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch.cuda.current_device


def _call(what: str, fn, device: torch.device, *args):
    """fn(*args, stream) on the current stream of `device`, with that device current; raises what it refuses."""
    index = device.index
    now = _current_device()
    if now == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc != 0:
        _check(rc, what)


def empty_cache_fp8(num_blocks: int, h_kv: int = 1, stride: int = D_QK, device=None):
    """A new 8-bit cache, zeroed: (cache float8_e4m3fn [num_blocks, 64, h_kv, 576], scales float32 [num_blocks, h_kv, 64]).
    `stride`: bytes per entry, 576 or more and a multiple of 16."""
    if num_blocks < 1 or h_kv < 1 or stride < D_QK or stride % 16:
        raise MLAError(f"empty_cache_fp8: invalid sizes ({num_blocks}, {h_kv}, {stride})")
    device = torch.device("cuda") if device is None else device
    alloc = torch.zeros((num_blocks, BLOCK_SIZE, h_kv, stride), dtype=torch.uint8, device=device)
    scales = torch.zeros((num_blocks, h_kv, BLOCK_SIZE), dtype=torch.float32, device=device)
    return alloc.view(FP8)[..., :D_QK], scales


def _check_cache_fp8(kcache, scales):
    """(num_blocks, h_kv, entry stride in bytes) of an 8-bit cache."""
    shape, st = kcache.shape, kcache.stride()
    if kcache.dtype is not FP8 or len(shape) != 4 or shape[1] != BLOCK_SIZE or shape[3] != D_QK:
        raise MLAError(f"the cache must be float8_e4m3fn [num_blocks, {BLOCK_SIZE}, h_kv, {D_QK}], got {kcache.dtype} "
                       f"{tuple(shape)}")
    nb, _, h_kv, _ = shape
    if scales.dtype is not torch.float32 or scales.shape != (nb, h_kv, BLOCK_SIZE) or not scales.is_contiguous():
        raise MLAError(f"scales must be contiguous float32 [{nb}, {h_kv}, {BLOCK_SIZE}], got {scales.dtype} "
                       f"{tuple(scales.shape)}")
    if not kcache.is_cuda or scales.device != kcache.device:
        raise MLAError("the cache and its scales must be on one CUDA device")
    entry = st[2] if h_kv > 1 else st[1]
    if st[3] != 1 or st[1] != h_kv * entry or (st[0] != BLOCK_SIZE * st[1] and nb > 1):
        raise MLAError(f"cache layout not supported: shape {tuple(shape)}, strides {st}")
    return nb, h_kv, entry


def _status_word(status, device):
    if status is None:
        return _status_of_device(device) if device.type == "cuda" else new_status(device)  # (refused by who asked)
    if status.dtype is not torch.int32 or status.device != device or status.numel() < 1:
        raise MLAError(f"status must be an int32 word on {device}")
    return status


def write_cache_fp8(kv_c: torch.Tensor, k_pe: torch.Tensor, slot_mapping: torch.Tensor, kcache: torch.Tensor,
                    scales: torch.Tensor, status: torch.Tensor | None = None):
    """New tokens into the 8-bit cache (mla_write_cache_kv8): entry slot_mapping[t] <- [kv_c[t], k_pe[t]] as e4m3 with one
    power-of-two scale.  Slots below 0 are skipped; the others must differ from one another.  What the device finds wrong
    goes to `status`, or without one to the device's word that check_status() looks at."""
    nb, h_kv, stride = _check_cache_fp8(kcache, scales)
    if h_kv != 1:
        raise MLAError("MLA caches have one latent head")
    dev, n = kcache.device, slot_mapping.shape[0] if slot_mapping.dim() == 1 else -1
    if kv_c.dtype is not torch.bfloat16 or k_pe.dtype is not torch.bfloat16:
        raise MLAError("kv_c and k_pe must be bfloat16")
    if kv_c.shape != (n, D_V) or k_pe.shape != (n, D_QK - D_V):
        raise MLAError(f"kv_c must be [T, 512], k_pe [T, 64] and slot_mapping [T], got {tuple(kv_c.shape)}, "
                       f"{tuple(k_pe.shape)}, {tuple(slot_mapping.shape)}")
    kv_row, kv_1 = kv_c.stride()
    pe_row, pe_1 = k_pe.stride()
    if kv_1 != 1 or pe_1 != 1:
        raise MLAError("kv_c and k_pe rows must be contiguous")
    if n <= 1:  # one row's stride says nothing
        kv_row, pe_row = D_V, D_QK - D_V
    if kv_c.device != dev or k_pe.device != dev:
        raise MLAError("kv_c, k_pe and the cache must be on one device")
    if slot_mapping.dtype is not torch.int64 or slot_mapping.device != dev or not slot_mapping.is_contiguous():
        if slot_mapping.dtype not in (torch.int64, torch.int32):
            raise MLAError("slot_mapping must be int64 or int32")
        slot_mapping = slot_mapping.to(device=dev, dtype=torch.int64).contiguous()
    status = _status_word(status, dev)
    _call("mla_write_cache_kv8", load_library().mla_write_cache_kv8, dev, kv_c.data_ptr(), kv_row, k_pe.data_ptr(), pe_row,
          slot_mapping.data_ptr(), n, kcache.data_ptr(), scales.data_ptr(), nb, BLOCK_SIZE, stride, status.data_ptr())
    return kcache, scales


def read_cache_fp8(kcache: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor, cu_tokens: torch.Tensor,
                   total: int, starts: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   status: torch.Tensor | None = None):
    """Entries of ragged token ranges back as bf16 rows (mla_read_cache_kv8): row cu_tokens[i] + n is token
    starts[i] + n (starts: 0 where None) of sequence i.  Returns out [total, 576]; a given `out` may have more rows.
    Rows from cu_tokens[-1] on are left as they were.  `status` as for write_cache_fp8."""
    nb, h_kv, stride = _check_cache_fp8(kcache, scales)
    if h_kv != 1:
        raise MLAError("MLA caches have one latent head")
    dev = kcache.device
    if block_table.dtype is not torch.int32 or block_table.dim() != 2 or block_table.shape[0] < 1:
        raise MLAError("block_table must be int32 [b, max_blocks]")
    b, width = block_table.shape
    if cu_tokens.dtype is not torch.int32 or cu_tokens.shape != (b + 1,):
        raise MLAError(f"cu_tokens must be int32 [{b + 1}]")
    if starts is not None and (starts.dtype is not torch.int32 or starts.shape != (b,)):
        raise MLAError(f"starts must be int32 [{b}]")
    if block_table.device != dev or cu_tokens.device != dev or (starts is not None and starts.device != dev):
        raise MLAError("the cache, block_table, cu_tokens and starts must be on one device")
    if total < 0:
        raise MLAError("total must be 0 or more")
    if out is None:
        out = torch.empty((total, D_QK), dtype=torch.bfloat16, device=dev)
    elif (out.dtype is not torch.bfloat16 or out.dim() != 2 or out.shape[0] < total or out.shape[1] != D_QK
          or not out.is_contiguous() or out.device != dev):
        raise MLAError(f"out must be contiguous bfloat16 [{total} or more, {D_QK}] on {dev}")
    block_table, cu_tokens = block_table.contiguous(), cu_tokens.contiguous()
    if starts is not None:
        starts = starts.contiguous()
    status = _status_word(status, dev)
    _call("mla_read_cache_kv8", load_library().mla_read_cache_kv8, dev, kcache.data_ptr(), scales.data_ptr(), nb, BLOCK_SIZE,
          stride, block_table.data_ptr(), width, cu_tokens.data_ptr(), None if starts is None else starts.data_ptr(), b,
          out.data_ptr(), total, status.data_ptr())
    return out


def num_parts_fp8(s_q: int, h_q: int, h_kv: int = 1, device=None) -> int:
    """Recommended schedule parts of the decode over an 8-bit cache (mla_num_parts_kv8)."""
    dev = torch.cuda.current_device() if device is None else torch.device(device).index or 0
    n = load_library().mla_num_parts_kv8(s_q, h_q, h_kv, dev)
    if n < 0:
        _check(n, "mla_num_parts_kv8")
    return n


def workspace_bytes_fp8(b: int, s_q: int, h_q: int, h_kv: int, parts: int) -> int:
    """Scratch bytes of the decode over an 8-bit cache (mla_workspace_bytes_kv8)."""
    return int(load_library().mla_workspace_bytes_kv8(b, s_q, h_q, h_kv, parts))


def mla_decode_fp8(q: torch.Tensor, kcache: torch.Tensor, scales: torch.Tensor, block_table: torch.Tensor,
                   cache_seqlens: torch.Tensor, metadata: torch.Tensor, num_splits: torch.Tensor,
                   softmax_scale: float, causal: bool = False, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   status: torch.Tensor | None = None):
    """MLA decode over the 8-bit cache (mla_decode_kv8): returns (out bf16[b, s_q, h_q, 512], lse fp32[b, h_q, s_q]).
    `status` as for write_cache_fp8."""
    if q.dim() != 4:
        raise MLAError(f"q must be [b, s_q, h_q, 576], got {tuple(q.shape)}")
    b, s_q, h_q, _ = q.shape
    dev = q.device
    if (num_splits.shape != (b + 1,) or metadata.dim() != 2 or metadata.shape[1] != 8
            or metadata.dtype is not torch.int32 or num_splits.dtype is not torch.int32
            or metadata.device != dev or num_splits.device != dev
            or not (metadata.is_contiguous() and num_splits.is_contiguous())):
        raise MLAError("metadata / num_splits do not come from get_mla_metadata for this batch")
    if workspace is None:
        h_kv = kcache.shape[2] if kcache.dim() == 4 else 1
        workspace = torch.empty((workspace_bytes_fp8(b, s_q, h_q, h_kv, metadata.shape[0]),), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise MLAError(f"workspace must be contiguous on {dev}")
    return _decode_fp8(q, kcache, scales, block_table, cache_seqlens, metadata, num_splits, softmax_scale, causal, out, lse,
                       workspace, workspace.numel() * workspace.element_size(), _status_word(status, dev))


def _decode_fp8(q, kcache, scales, block_table, cache_seqlens, metadata, num_splits, softmax_scale, causal, out, lse,
                workspace, workspace_size, status):
    """mla_decode_fp8 with a schedule, workspace and status word that are known to be right for q's shape and device."""
    nb, h_kv, stride = _check_cache_fp8(kcache, scales)
    if q.dtype is not torch.bfloat16 or not q.is_contiguous():
        raise MLAError("q must be contiguous bfloat16 [b, s_q, h_q, 576]")
    b, s_q, h_q, d = q.shape
    dev = q.device
    # the library reads and writes exactly these extents: see _check_io
    if (block_table.dtype is not torch.int32 or block_table.dim() != 2 or block_table.shape[0] != b
            or cache_seqlens.dtype is not torch.int32 or cache_seqlens.shape != (b,) or out is not None or lse is not None):
        _check_io(q, block_table, cache_seqlens, out, lse)
    if kcache.device != dev or block_table.device != dev or cache_seqlens.device != dev:
        raise MLAError("q, the cache, block_table, cache_seqlens and the schedule must be on one device")
    block_table, cache_seqlens = block_table.contiguous(), cache_seqlens.contiguous()
    if out is None:
        out = torch.empty((b, s_q, h_q, D_V), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((b, h_q, s_q), dtype=torch.float32, device=dev)
    _call("mla_decode_kv8", load_library().mla_decode_kv8, dev, q.data_ptr(), b, s_q, h_q, d, kcache.data_ptr(),
          scales.data_ptr(), nb, BLOCK_SIZE, h_kv, stride, block_table.data_ptr(), block_table.shape[1],
          cache_seqlens.data_ptr(), D_V, metadata.data_ptr(), metadata.shape[0], num_splits.data_ptr(), softmax_scale,
          1 if causal else 0, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace_size, status.data_ptr())
    return out, lse


class MLADecoderFP8:
    """MLADecoder for the 8-bit cache: plan(cache_seqlens) once per decode step, then one call per layer, with
    the layer's cache and scales.  The schedule, scratch and status word belong to the decoder: its calls must follow
    one another on one stream (or be ordered by events), captured ones included."""

    def __init__(self, b: int, s_q: int, h_q: int, h_kv: int = 1, device=None, parts: int | None = None):
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.b, self.s_q, self.h_q, self.h_kv = b, s_q, h_q, h_kv
        self.parts = parts if parts is not None else num_parts_fp8(s_q, h_q, h_kv, self.device)
        self.workspace = torch.empty((workspace_bytes_fp8(b, s_q, h_q, h_kv, self.parts),), dtype=torch.uint8,
                                     device=self.device)
        self.status = new_status(self.device)
        self.metadata = None
        self.num_splits = None

    def plan(self, cache_seqlens: torch.Tensor):
        if tuple(cache_seqlens.shape) != (self.b,) or cache_seqlens.device != self.device:
            raise MLAError(f"cache_seqlens must be int32 [{self.b}] on {self.device}")
        with torch.cuda.device(self.device):
            self.metadata, self.num_splits = get_mla_metadata(cache_seqlens, self.parts, self.status)
        return self

    def __call__(self, q, kcache, scales, block_table, cache_seqlens, softmax_scale, causal=False, out=None, lse=None):
        if self.metadata is None:
            raise MLAError("plan(cache_seqlens) comes before the first decode")
        if (q.shape != (self.b, self.s_q, self.h_q, D_QK) or q.device != self.device or kcache.dim() != 4
                or kcache.shape[2] != self.h_kv):
            raise MLAError(f"q {tuple(q.shape)} on {q.device} / cache {tuple(kcache.shape)} do not fit the decoder's "
                           f"({self.b}, {self.s_q}, {self.h_q}, {D_QK}) on {self.device} / h_kv {self.h_kv}")
        return _decode_fp8(q, kcache, scales, block_table, cache_seqlens, self.metadata, self.num_splits, softmax_scale,
                           causal, out, lse, self.workspace, self.workspace.numel(), self.status)


# ------------------------------------------------------------ rotary positions
_ROPE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # MLA_BF16, MLA_FP16, MLA_FP32


_PI_BITS = 1300  # 64 below a turn of the largest double, 2^1024, with some to spare


@functools.lru_cache(None)
def _pi() -> int:
    """pi * 2^_PI_BITS, by pi = 16 arctan(1/5) - 4 arctan(1/239)."""
    def arctan_of_inverse(x):
        term = (1 << (_PI_BITS + 32)) // x
        total, n = term, 1
        while term:
            term //= -x * x
            n += 2
            total += term // n
        return total
    return (16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239)) >> 32


def _turns(f: float) -> int:
    """f radians as turns in 64-bit fixed point, whole turns dropped, rounded once."""
    num, den = f.as_integer_ratio()
    den *= _pi()
    return ((num << (_PI_BITS + 64)) + den) // (2 * den) % (1 << 64)


class Rotary:
    """A model's rotary frequencies, on the device, for rope().

    Pair i of `dim` / 2 turns by base^(-2i/dim) radians per position.  With factor > 1 the context is scaled: pairs
    that turn more than beta_fast times within original_length keep their frequency, pairs that turn less than
    beta_slow times have theirs divided by `factor`, and those between are blended linearly in i.  `gain` multiplies
    the turned values.  `frequencies`, where given, holds dim / 2 radians per position in place of all that."""

    def __init__(self, dim: int = D_QK - D_V, base: float = 10000.0, interleaved: bool = True, factor: float = 1.0,
                 original_length: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, gain: float = 1.0,
                 frequencies=None, device=None):
        if dim < 2 or dim > 256 or dim % 2:
            raise MLAError(f"rotary dim must be even and 2 .. 256, got {dim}")
        if not math.isfinite(gain) or not (base > 1.0 and math.isfinite(base)) or not factor >= 1.0 \
                or not math.isfinite(factor) or original_length < 1 or not beta_fast > 0.0 or not beta_slow > 0.0:
            raise MLAError("rotary: base > 1, factor >= 1, original_length >= 1, betas > 0 and a finite gain are needed")
        n = dim // 2
        if frequencies is not None:
            freq = [float(f) for f in frequencies]
            if len(freq) != n or not all(math.isfinite(f) for f in freq):
                raise MLAError(f"frequencies must be {n} finite radians per position")
        else:
            freq = [base ** (-2.0 * i / dim) for i in range(n)]
            if factor > 1.0:
                def edge(turns):  # the pair that turns so often within original_length
                    return dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))
                low, high = max(math.floor(edge(beta_fast)), 0), min(math.ceil(edge(beta_slow)), dim - 1)
                for i in range(n):
                    ramp = min(max((i - low) / max(high - low, 0.001), 0.0), 1.0)
                    freq[i] = freq[i] / factor * ramp + freq[i] * (1.0 - ramp)
        self.dim, self.interleaved, self.gain, self.frequencies = dim, int(bool(interleaved)), float(gain), freq
        # turns per position in 64-bit fixed point (two's complement in an int64 tensor)
        turns = [_turns(f) for f in freq]
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        self.turns = torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device=device)


def _rope_rows(x, out, tokens, dim, what):
    """(out; ptr, token stride, head stride, out ptr, token stride, head stride, heads) of rows [T, dim] or [T, h, dim]."""
    shape, st = x.shape, x.stride()
    nd = len(shape)
    if (nd != 3 and nd != 2) or shape[0] != tokens or shape[-1] != dim or st[-1] != 1:
        raise MLAError(f"{what} must be [{tokens}, {dim}] or [{tokens}, heads, {dim}] with dense rows, got "
                       f"{tuple(shape)}, strides {st}")
    heads, xh = (shape[1], st[1]) if nd == 3 else (1, 0)
    if out is None:
        out = torch.empty(shape, dtype=x.dtype, device=x.device)
        ot, oh = heads * dim, dim
    else:
        so = out.stride()
        if out.shape != shape or out.dtype is not x.dtype or out.device != x.device or so[-1] != 1:
            raise MLAError(f"the output of {what} must have its shape, type and device, with dense rows")
        ot, oh = so[0], so[1] if nd == 3 else 0
    return out, (x.data_ptr(), st[0], xh, out.data_ptr(), ot, oh, heads)


def rope(x: torch.Tensor, positions: torch.Tensor, rotary: Rotary, out: torch.Tensor | None = None,
         k: torch.Tensor | None = None, k_out: torch.Tensor | None = None, inverse: bool = False):
    """Rotary positions (mla_rope): x [T, dim] or [T, heads, dim] (a view of part of the head: q[..., 512:]), positions
    int32 or int64 [T].  Writes `out` (new where None; x itself turns in place; one whose rows meet x's otherwise is
    refused) and returns it.  With `k`, rows of another head count turn in the same launch, and (out, k_out) is
    returned; the rows written must not meet those of the other pair either.  `inverse` turns the other way, with the
    same gain: the gradient of the forward turn."""
    dtype = _ROPE_DTYPES.get(x.dtype)
    if dtype is None:
        raise MLAError(f"rope works on bfloat16, float16 and float32, not {x.dtype}")
    dev, dim = x.device, rotary.dim
    if positions.dtype is torch.int64:
        width = 8
    elif positions.dtype is torch.int32:
        width = 4
    else:
        raise MLAError("positions must be a contiguous int32 or int64 vector")
    if positions.dim() != 1 or not positions.is_contiguous():
        raise MLAError("positions must be a contiguous int32 or int64 vector")
    if not x.is_cuda or positions.device != dev or rotary.turns.device != dev:
        raise MLAError("x, positions and the rotary must be on one CUDA device")
    n = positions.shape[0]
    out, xs = _rope_rows(x, out, n, dim, "x")
    if k is not None:
        if k.dtype is not x.dtype or k.device != dev:
            raise MLAError("k must have the type and device of x")
        k_out, ks = _rope_rows(k, k_out, n, dim, "k")
    elif k_out is not None:
        raise MLAError("k_out without k")
    else:
        ks = (None, 0, 0, None, 0, 0, 0)
    first, second = (xs, ks) if xs[6] > 0 else (ks, (None, 0, 0, None, 0, 0, 0))  # x may have no heads
    if n > 0 and first[6] > 0:
        _call("mla_rope", load_library().mla_rope, dev, *first, *second, n, dim, positions.data_ptr(), width,
              rotary.turns.data_ptr(), rotary.gain, rotary.interleaved, 1 if inverse else 0, dtype)
    return out if k is None else (out, k_out)
