"""Paged KV cache decode path for one GB300 GPU: Python binding.

Argument marshalling only. Every step runs in the CUDA library
``_build/libpkv.so`` (built from ``csrc/`` by ``build.build()``) behind the C
ABI of ``include/pkv.h``; the functions here have the same names, take torch
tensors (or raw device addresses as ints), pass their device pointers and
the stream, and raise ``PkvError`` on a non-OK status. There is no fallback:
if the library is missing, every call raises.
"""

import ctypes
import os

from . import build as _build

PAGE_SIZE = 16
NUM_Q_HEADS = 32
NUM_KV_HEADS = 8
HEAD_DIM = 64
MAX_SEQ_LEN = 2048

STATUS = {0: "PKV_OK", 1: "PKV_ERR_INVALID_ARG", 2: "PKV_ERR_OUT_OF_RANGE", 3: "PKV_ERR_CUDA",
          4: "PKV_ERR_UNSUPPORTED", 5: "PKV_ERR_DEVICE_TIMEOUT", 6: "PKV_ERR_STATIC_LIMIT",
          7: "PKV_ERR_REJECTED"}
PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_OUT_OF_RANGE, PKV_ERR_CUDA, PKV_ERR_UNSUPPORTED, \
    PKV_ERR_DEVICE_TIMEOUT, PKV_ERR_STATIC_LIMIT, PKV_ERR_REJECTED = range(8)

EXPORTED = ("pkv_pool_create", "pkv_pool_destroy", "pkv_append", "pkv_decode_attention",
            "pkv_append_attend", "pkv_append_rope", "pkv_decode_attention_rope",
            "pkv_append_attend_rope", "pkv_append_attend_layers", "pkv_test_layers_wait_timeout",
            "pkv_get_error", "pkv_decode_attention_noalloc",
            "pkv_sched_budget", "pkv_sched_create", "pkv_sched_destroy", "pkv_sched_submit",
            "pkv_sched_admit", "pkv_sched_extend", "pkv_sched_extend_batch", "pkv_sched_finish",
            "pkv_sched_decode_batch",
            "pkv_sched_block_tables", "pkv_sched_get_stats", "pkv_prefill_fill",
            "pkv_prefill_attention", "pkv_prefill", "pkv_plan_decode",
            "pkv_pool_device_figures", "pkv_window_attention", "pkv_window_append_attend",
            "pkv_window_prefill_attention", "pkv_prefill_fill_axes", "pkv_copy_pages",
            "pkv_compact_pages", "pkv_sched_fork", "pkv_sched_held", "pkv_sched_release",
            "pkv_sched_compact", "pkv_status_string")


class PkvError(RuntimeError):
    def __init__(self, status, call):
        self.status = status
        super().__init__(f"{call}: {STATUS.get(status, status)}")


class SchedConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_layers", "num_pages", "page_size", "max_seq_len", "static_batching")]


class SchedStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "pool_pages", "submitted", "rejected", "admitted", "finished", "peak_active",
        "largest_decode_batch", "peak_assigned_pages", "admission_waits", "free_pages",
        "free_credits", "active", "waiting")]


class PoolConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_layers", "num_pages", "page_size", "num_q_heads", "num_kv_heads", "head_dim",
        "max_seq_len", "max_batch", "max_splits", "flags")]


PKV_FLAG_PDL, PKV_FLAG_LONG_CONTEXT = 1, 2
PKV_MAX_LONG_CONTEXT = 1048576
PKV_MAX_AXES = 4


class AxesRopeConfig(ctypes.Structure):
    _fields_ = [("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("rows", ctypes.c_int),
                ("num_axes", ctypes.c_int), ("axis_of_pair", ctypes.c_uint8 * (HEAD_DIM // 2))]


class DeviceFigures(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "num_sms", "ticket_blocks_per_sm", "narrow_blocks_per_sm", "wide_blocks_per_sm",
        "max_cluster", "max_splits", "max_seq_len")]


class Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "shape", "cluster", "num_splits", "chunk_pages", "range_div", "grid_splits",
        "grid_units", "longest_first")]


PKV_SHAPE_TICKET, PKV_SHAPE_NARROW, PKV_SHAPE_WIDE = 0, 1, 2


_lib = None


def library_path() -> str:
    return _build.LIBRARY


def load(path: str = None):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or _build.LIBRARY
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library not built: {path} (run paged_kv_cache_210_gb300.build)")
    lib = ctypes.CDLL(path)
    P, i = ctypes.c_void_p, ctypes.c_int
    lib.pkv_pool_create.argtypes = [ctypes.POINTER(PoolConfig), ctypes.POINTER(ctypes.c_void_p)]
    lib.pkv_pool_destroy.argtypes = [P]
    lib.pkv_append.argtypes = [P, i, P, P, P, P, P, P, i, P]
    lib.pkv_decode_attention.argtypes = [P, i, P, P, P, P, P, P, i, i, P]
    lib.pkv_append_attend.argtypes = [P, i, P, P, P, P, P, P, P, P, i, i, P]
    lib.pkv_append_rope.argtypes = [P, i, P, P, P, P, P, P, P, P, i, P]
    lib.pkv_decode_attention_rope.argtypes = [P, i, P, P, P, P, P, P, P, P, i, i, P]
    lib.pkv_append_attend_rope.argtypes = [P, i, P, P, P, P, P, P, P, P, P, P, i, i, P]
    lib.pkv_append_attend_layers.argtypes = [P, i, i, P, P, P, P, P, P, P, P, i, P]
    lib.pkv_test_layers_wait_timeout.argtypes = [P, i, i, P, P, P, P, P, P, P, P, i, P]
    lib.pkv_get_error.argtypes = [P, P]
    lib.pkv_decode_attention_noalloc.argtypes = [i, P, P, P, P, P, P, i, i, i, i, i, i, P, P]
    SC, SP = ctypes.POINTER(SchedConfig), ctypes.POINTER(ctypes.c_int)
    lib.pkv_sched_budget.argtypes = [SC, i, i, SP, SP, ctypes.POINTER(ctypes.c_int64)]
    lib.pkv_sched_create.argtypes = [SC, ctypes.POINTER(ctypes.c_void_p)]
    lib.pkv_sched_destroy.argtypes = [P]
    lib.pkv_sched_submit.argtypes = [P, i, i, SP]
    lib.pkv_sched_admit.argtypes = [P, P, i, SP]
    lib.pkv_sched_extend.argtypes = [P, i, i]
    lib.pkv_sched_finish.argtypes = [P, i]
    lib.pkv_sched_decode_batch.argtypes = [P, P, i, SP]
    lib.pkv_sched_extend_batch.argtypes = [P, P, P, i]
    lib.pkv_sched_block_tables.argtypes = [P, P, i, P, i, i, i]
    lib.pkv_sched_get_stats.argtypes = [P, ctypes.POINTER(SchedStats)]
    lib.pkv_prefill_fill.argtypes = [P, i, P, P, P, P, P, P, P, i, i, i, P]
    lib.pkv_prefill_attention.argtypes = [P, i, P, P, P, P, P, P, P, i, i, i, P]
    lib.pkv_prefill.argtypes = [P, i, P, P, P, P, P, P, P, P, P, i, i, i, P]
    lib.pkv_plan_decode.argtypes = [ctypes.POINTER(DeviceFigures), i, i, ctypes.POINTER(Plan)]
    lib.pkv_pool_device_figures.argtypes = [P, ctypes.POINTER(DeviceFigures)]
    lib.pkv_window_attention.argtypes = [P, i, P, P, P, P, P, P, i, i, P, P, i, i, i, P]
    lib.pkv_window_append_attend.argtypes = [P, i, P, P, P, P, P, P, P, P, i, i, P, P, i, i, i, P]
    lib.pkv_window_prefill_attention.argtypes = [P, i, P, P, P, P, P, P, P, i, i, i, i, i, P]
    lib.pkv_prefill_fill_axes.argtypes = [P, i, P, P, P, P, P, P, P, P, P, P, P, i, i, i, i, P]
    lib.pkv_copy_pages.argtypes = [P, P, P, P, P, P, i, P]
    lib.pkv_compact_pages.argtypes = [P, P, P, P, P, P, i, P]
    lib.pkv_sched_fork.argtypes = [P, i, i, i, SP, P, P, i, SP, SP]
    lib.pkv_sched_held.argtypes = [P, i, SP, SP]
    lib.pkv_sched_release.argtypes = [P, i, i, i, SP]
    lib.pkv_sched_compact.argtypes = [P, P, P, i, SP]
    lib.pkv_status_string.argtypes = [i]
    lib.pkv_status_string.restype = ctypes.c_char_p
    for name in EXPORTED[:-1]:
        getattr(lib, name).restype = ctypes.c_int
    if path == _build.LIBRARY:
        _lib = lib
    return lib


_dtype_names = {}


def _dtype_name(dtype):
    name = _dtype_names.get(dtype)
    if name is None:
        name = _dtype_names[dtype] = str(dtype).removeprefix("torch.")
    return name


def _addr(x, dtype=None, what="tensor"):
    """Address of a tensor (or an int address, or None). A tensor must be
    contiguous and, when `dtype` is given ("bfloat16", "float32", "int32"),
    of that dtype: the library reads raw memory in the layouts include/*.h
    documents."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError(f"{what}: the library takes contiguous tensors")
    if dtype is not None and _dtype_name(x.dtype) != dtype:
        raise ValueError(f"{what}: expected {dtype}, got {x.dtype}")
    return x.data_ptr()


def _i32(x, what):
    return _addr(x, "int32", what)


# the dtype of each tensor argument of the CUDA entry points, by parameter name
_DTYPES = {"q": "bfloat16", "k": "bfloat16", "v": "bfloat16", "k_pool": "bfloat16",
           "v_pool": "bfloat16", "block_tables": "int32", "positions": "int32",
           "seq_lens": "int32", "cu_tokens": "int32", "start_pos": "int32", "out": "float32",
           "rope_cos": "float32", "rope_sin": "float32", "rope_positions": "int32",
           "q_out": "bfloat16", "src": "int32", "dst": "int32", "tokens": "int32"}


def _ptrs(**tensors):
    """Checked addresses of the named tensor arguments, in the order given."""
    return [_addr(t, _DTYPES[name], name) for name, t in tensors.items()]


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status, call):
    if status != PKV_OK:
        raise PkvError(status, call)


class Pool:
    """Owns a pkv_pool_t handle (the split workspace and the error flag)."""

    def __init__(self, handle, config, lib, device=None):
        self.handle = handle
        self.config = config
        self.device = device     # CUDA device index, where known
        # elements of a pool tensor and entries of the block tables
        self.elements = config.num_pages * NUM_KV_HEADS * PAGE_SIZE * HEAD_DIM if config else 0
        self.entries = config.num_layers * config.max_batch * \
            (config.max_seq_len // PAGE_SIZE) if config else 0
        self._lib = lib

    def close(self):
        if self.handle:
            _check(self._lib.pkv_pool_destroy(self.handle), "pkv_pool_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _current_device():
    """The current CUDA device's index, or None where torch does not have one."""
    try:
        import torch
        return torch.cuda.current_device()
    except (ImportError, AssertionError, RuntimeError):   # no torch, no CUDA in it, no device
        return None


def pkv_pool_create(num_layers, num_pages, max_batch, max_seq_len=MAX_SEQ_LEN, max_splits=0,
                    flags=0, lib=None) -> Pool:
    lib = lib or load()
    cfg = PoolConfig(num_layers, num_pages, PAGE_SIZE, NUM_Q_HEADS, NUM_KV_HEADS, HEAD_DIM,
                     max_seq_len, max_batch, max_splits, flags)
    device = _current_device()      # before the handle exists: nothing after it may fail
    handle = ctypes.c_void_p()
    _check(lib.pkv_pool_create(ctypes.byref(cfg), ctypes.byref(handle)), "pkv_pool_create")
    return Pool(handle.value, cfg, lib, device)


def pkv_pool_destroy(pool: Pool):
    pool.close()


def _batch(x, batch):
    return int(x.shape[0]) if batch is None else int(batch)


def pkv_append(pool: Pool, layer, k, v, k_pool, v_pool, block_tables, positions, batch=None,
               stream=None):
    """k, v: bf16 [B][8][64]; pools bf16 [P][8][16][64]; tables int32 [L][max_batch][pages]."""
    st = pool._lib.pkv_append(
        pool.handle, int(layer),
        *_ptrs(k=k, v=v, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
               positions=positions),
        _batch(positions, batch), _stream(stream))
    _check(st, "pkv_append")


def pkv_decode_attention(pool: Pool, layer, q, k_pool, v_pool, block_tables, seq_lens, out,
                         batch=None, num_splits=0, stream=None):
    """q: bf16 [B][32][64]; out: fp32 [B][32][64]; seq_lens: int32 [B] (after the append)."""
    st = pool._lib.pkv_decode_attention(
        pool.handle, int(layer),
        *_ptrs(q=q, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables, seq_lens=seq_lens,
               out=out),
        _batch(seq_lens, batch), int(num_splits), _stream(stream))
    _check(st, "pkv_decode_attention")


def pkv_append_attend(pool: Pool, layer, q, k, v, k_pool, v_pool, block_tables, seq_lens, out,
                      batch=None, num_splits=0, stream=None):
    """Fused append (at seq_lens - 1) and decode attention for one layer."""
    st = pool._lib.pkv_append_attend(
        pool.handle, int(layer),
        *_ptrs(q=q, k=k, v=v, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
               seq_lens=seq_lens, out=out),
        _batch(seq_lens, batch), int(num_splits), _stream(stream))
    _check(st, "pkv_append_attend")


def pkv_append_rope(pool: Pool, layer, k, v, k_pool, v_pool, block_tables, positions,
                    rope_cos, rope_sin, batch=None, stream=None):
    """pkv_append with each key rotated to its position; rope_cos/rope_sin:
    fp32 [max_seq_len][32] on the device."""
    st = pool._lib.pkv_append_rope(
        pool.handle, int(layer),
        *_ptrs(k=k, v=v, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
               positions=positions, rope_cos=rope_cos, rope_sin=rope_sin),
        _batch(positions, batch), _stream(stream))
    _check(st, "pkv_append_rope")


def pkv_decode_attention_rope(pool: Pool, layer, q, k_pool, v_pool, block_tables, seq_lens,
                              rope_cos, rope_sin, out, batch=None, num_splits=0, stream=None):
    """pkv_decode_attention with each query rotated to position seq_lens - 1."""
    st = pool._lib.pkv_decode_attention_rope(
        pool.handle, int(layer),
        *_ptrs(q=q, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables, seq_lens=seq_lens,
               rope_cos=rope_cos, rope_sin=rope_sin, out=out),
        _batch(seq_lens, batch), int(num_splits), _stream(stream))
    _check(st, "pkv_decode_attention_rope")


def pkv_append_attend_rope(pool: Pool, layer, q, k, v, k_pool, v_pool, block_tables, seq_lens,
                           rope_cos, rope_sin, out, batch=None, num_splits=0, stream=None):
    """pkv_append_attend with the key and the queries rotated to seq_lens - 1."""
    st = pool._lib.pkv_append_attend_rope(
        pool.handle, int(layer),
        *_ptrs(q=q, k=k, v=v, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
               seq_lens=seq_lens, rope_cos=rope_cos, rope_sin=rope_sin, out=out),
        _batch(seq_lens, batch), int(num_splits), _stream(stream))
    _check(st, "pkv_append_attend_rope")


def pkv_append_attend_layers(pool: Pool, layer_begin, q, k, v, k_pool, v_pool, block_tables,
                             seq_lens, out, num_layers=None, batch=None, stream=None):
    """Fused append + attend of layers layer_begin .. layer_begin + num_layers - 1
    in one persistent launch (several for long calls). q: bf16 [J][B][32][64];
    k, v: bf16 [J][B][8][64]; out: fp32 [J][B][32][64]; J = num_layers
    (default: q's first dimension)."""
    J = int(q.shape[0]) if num_layers is None else int(num_layers)
    st = pool._lib.pkv_append_attend_layers(
        pool.handle, int(layer_begin), J,
        *_ptrs(q=q, k=k, v=v, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
               seq_lens=seq_lens, out=out),
        _batch(seq_lens, batch), _stream(stream))
    _check(st, "pkv_append_attend_layers")


def pkv_test_layers_wait_timeout(pool: Pool, layer_begin, q, k, v, k_pool, v_pool,
                                 block_tables, seq_lens, out, num_layers=None, batch=None,
                                 stream=None):
    """Failure-detection test hook: pkv_append_attend_layers with every
    between-layer wait unreachable; the device flags a timeout."""
    J = int(q.shape[0]) if num_layers is None else int(num_layers)
    st = pool._lib.pkv_test_layers_wait_timeout(
        pool.handle, int(layer_begin), J,
        *_ptrs(q=q, k=k, v=v, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
               seq_lens=seq_lens, out=out),
        _batch(seq_lens, batch), _stream(stream))
    _check(st, "pkv_test_layers_wait_timeout")


def pkv_plan_decode(figures: DeviceFigures, batch, num_splits=0, lib=None) -> Plan:
    """The decode launch plan for a batch on a device (host arithmetic, no GPU)."""
    lib = lib or load()
    plan = Plan()
    _check(lib.pkv_plan_decode(ctypes.byref(figures), int(batch), int(num_splits),
                               ctypes.byref(plan)), "pkv_plan_decode")
    return plan


def pkv_pool_device_figures(pool: Pool) -> DeviceFigures:
    figures = DeviceFigures()
    _check(pool._lib.pkv_pool_device_figures(pool.handle, ctypes.byref(figures)),
           "pkv_pool_device_figures")
    return figures


def pkv_get_error(pool: Pool, stream=None) -> int:
    """Synchronises the stream; returns (and clears) the sticky device status."""
    return pool._lib.pkv_get_error(pool.handle, _stream(stream))


def pkv_decode_attention_noalloc(layer, q, k_pool, v_pool, block_tables, seq_lens, out,
                                 num_layers, num_pages, max_batch, max_seq_len=MAX_SEQ_LEN,
                                 batch=None, num_splits=1, error_bits=None, stream=None,
                                 lib=None):
    """Decode attention for callers that may not allocate device memory: no
    pool handle, scratch in the library's own static device array (limits and
    the one-time set-up on first use are described in include/pkv.h)."""
    lib = lib or load()
    st = lib.pkv_decode_attention_noalloc(
        int(layer),
        *_ptrs(q=q, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables, seq_lens=seq_lens,
               out=out),
        int(num_layers), int(num_pages), int(max_batch), int(max_seq_len),
        _batch(seq_lens, batch), int(num_splits), _i32(error_bits, "error_bits"),
        _stream(stream))
    _check(st, "pkv_decode_attention_noalloc")


# ---------------------------------------------------------------- prefill
def pkv_prefill_fill(pool: Pool, layer, k, v, k_pool, v_pool, block_tables, cu_tokens, start_pos,
                     max_chunk_tokens, batch=None, total_tokens=None, stream=None):
    """Writes chunk tokens' K/V (bf16 [T][8][64]) into their pages."""
    batch = int(start_pos.shape[0]) if batch is None else int(batch)
    total = int(k.shape[0]) if total_tokens is None else int(total_tokens)
    st = pool._lib.pkv_prefill_fill(
        pool.handle, int(layer),
        *_ptrs(k=k, v=v, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
               cu_tokens=cu_tokens, start_pos=start_pos),
        batch, total, int(max_chunk_tokens), _stream(stream))
    _check(st, "pkv_prefill_fill")


def pkv_prefill_attention(pool: Pool, layer, q, k_pool, v_pool, block_tables, cu_tokens, start_pos,
                          out, max_chunk_tokens, batch=None, total_tokens=None, stream=None):
    """Causal attention of chunk tokens (q bf16 [T][32][64]) over the pages; out fp32."""
    batch = int(start_pos.shape[0]) if batch is None else int(batch)
    total = int(q.shape[0]) if total_tokens is None else int(total_tokens)
    st = pool._lib.pkv_prefill_attention(
        pool.handle, int(layer),
        *_ptrs(q=q, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
               cu_tokens=cu_tokens, start_pos=start_pos, out=out),
        batch, total, int(max_chunk_tokens), _stream(stream))
    _check(st, "pkv_prefill_attention")


def pkv_prefill(pool: Pool, layer, q, k, v, k_pool, v_pool, block_tables, cu_tokens, start_pos,
                out, max_chunk_tokens, batch=None, total_tokens=None, stream=None):
    """pkv_prefill_fill then pkv_prefill_attention."""
    batch = int(start_pos.shape[0]) if batch is None else int(batch)
    total = int(q.shape[0]) if total_tokens is None else int(total_tokens)
    st = pool._lib.pkv_prefill(
        pool.handle, int(layer),
        *_ptrs(q=q, k=k, v=v, k_pool=k_pool, v_pool=v_pool, block_tables=block_tables,
               cu_tokens=cu_tokens, start_pos=start_pos, out=out),
        batch, total, int(max_chunk_tokens), _stream(stream))
    _check(st, "pkv_prefill")


# ---------------------------------------------------------------- window, axes, pages
_torch_dtypes = {}


def _arg(pool, name, x, count=0):
    """Address of a tensor argument: what _addr checks, and that the tensor lies
    on the handle's device and holds at least `count` elements."""
    try:      # the common case in as few steps as a small call's latency wants
        if x.dtype is _torch_dtypes[name] and x.get_device() == pool.device and \
                x.numel() >= count and x.is_contiguous():
            return x.data_ptr()
    except (AttributeError, KeyError):
        if x is None or isinstance(x, int):
            return x
    address = _addr(x, _DTYPES[name], name)
    if pool.device is not None and x.get_device() != pool.device:
        raise ValueError(f"{name}: expected a tensor on cuda:{pool.device}, got {x.device}")
    if x.numel() < count:
        raise ValueError(f"{name}: expected at least {count} elements, got {x.numel()}")
    _torch_dtypes[name] = x.dtype     # the one that _addr accepts
    return address


_INT_MAX = 2 ** 31 - 1


def _length(x):
    """A window or sink count as the C int it becomes: any beyond an int means
    the whole context, any negative one is refused."""
    return x if 0 <= x <= _INT_MAX else _INT_MAX if x > 0 else -1


def _int(x):
    """A C int; a value outside its range becomes one that every call refuses."""
    return x if -1 <= x <= _INT_MAX else -1


def _pool_stream(pool, stream):
    """The stream's handle; by default the current stream of the handle's device."""
    if stream is None and pool.device is not None:
        import torch
        return torch._C._cuda_getCurrentRawStream(pool.device)
    return _stream(stream)


class AxesRope:
    """Rotation by several position axes (include/pkv_axes.h): keeps the tables."""

    def __init__(self, cos, sin, axis_of_pair):
        pairs = HEAD_DIM // 2
        axes = [int(a) for a in axis_of_pair]
        if len(axes) != pairs or min(axes) < 0 or max(axes) >= PKV_MAX_AXES:
            raise ValueError(f"axis_of_pair: expected {pairs} axes in 0 .. {PKV_MAX_AXES - 1}")
        for name, t in (("rope_cos", cos), ("rope_sin", sin)):
            if t.dim() != 2 or t.shape[1] != pairs or t.shape[0] < 1 or t.shape != cos.shape:
                raise ValueError(f"{name}: expected [rows][{pairs}]")
        if sin.device != cos.device:
            raise ValueError(f"rope_sin: expected a tensor on {cos.device}, got {sin.device}")
        self.tables = (cos, sin)
        self.num_axes = max(axes) + 1
        self.device = cos.get_device()
        self.config = AxesRopeConfig(_addr(cos, "float32", "rope_cos"),
                                     _addr(sin, "float32", "rope_sin"), int(cos.shape[0]),
                                     self.num_axes, (ctypes.c_uint8 * pairs)(*axes))
        self.address = ctypes.addressof(self.config)


def pkv_axes_rope(cos, sin, axis_of_pair) -> AxesRope:
    """cos, sin: fp32 [rows][32] on the device; axis_of_pair: the position axis of
    each of the 32 rotary pairs. Keep it for as many calls as use the tables."""
    return AxesRope(cos, sin, axis_of_pair)


def _rope_args(pool, rope, positions, tokens):
    """(rope, positions, stride) as the entry points take them; positions: int32
    [axes][>= tokens], or the address of [axes][tokens]."""
    if rope is None:
        if positions is not None:
            raise ValueError("rope_positions without rope")
        return None, None, 0
    if positions is None:
        raise ValueError("rope_positions: missing")
    if pool.device is not None and rope.device != pool.device:
        raise ValueError(f"rope_cos: expected a tensor on cuda:{pool.device}")
    if isinstance(positions, int):       # a raw address: rows of `tokens` entries
        return rope.address, positions, tokens
    if positions.dim() != 2 or positions.shape[0] < rope.num_axes or positions.shape[1] < tokens:
        raise ValueError(f"rope_positions: expected [{rope.num_axes}][>= {tokens}], got "
                         f"{tuple(positions.shape)}")
    return rope.address, _arg(pool, "rope_positions", positions), int(positions.shape[1])


def pkv_window_attention(pool: Pool, layer, q, k_pool, v_pool, block_tables, seq_lens, out, window,
                         sinks=0, rope=None, rope_positions=None, batch=None, num_splits=0,
                         stream=None):
    """Decode attention over the last `window` tokens and the first `sinks` ones
    (q bf16 [B][32][64], out fp32). rope: an AxesRope, with rope_positions
    int32 [axes][B]: the queries are rotated first. seq_lens 0: a padding row."""
    batch = _int(_batch(seq_lens, batch))
    rows = batch * NUM_Q_HEADS * HEAD_DIM
    st = pool._lib.pkv_window_attention(
        pool.handle, _int(int(layer)), _arg(pool, "q", q, rows),
        _arg(pool, "k_pool", k_pool, pool.elements),
        _arg(pool, "v_pool", v_pool, pool.elements),
        _arg(pool, "block_tables", block_tables, pool.entries),
        _arg(pool, "seq_lens", seq_lens, batch), _arg(pool, "out", out, rows), _length(int(window)),
        _length(int(sinks)), *_rope_args(pool, rope, rope_positions, batch), batch,
        _int(int(num_splits)), _pool_stream(pool, stream))
    _check(st, "pkv_window_attention")


def pkv_window_append_attend(pool: Pool, layer, q, k, v, k_pool, v_pool, block_tables, seq_lens,
                             out, window, sinks=0, rope=None, rope_positions=None, batch=None,
                             num_splits=0, stream=None):
    """Append (at seq_lens - 1, the key rotated with rope) and pkv_window_attention
    in one launch; k, v bf16 [B][8][64]."""
    batch = _int(_batch(seq_lens, batch))
    rows, new = batch * NUM_Q_HEADS * HEAD_DIM, batch * NUM_KV_HEADS * HEAD_DIM
    st = pool._lib.pkv_window_append_attend(
        pool.handle, _int(int(layer)), _arg(pool, "q", q, rows), _arg(pool, "k", k, new),
        _arg(pool, "v", v, new), _arg(pool, "k_pool", k_pool, pool.elements),
        _arg(pool, "v_pool", v_pool, pool.elements),
        _arg(pool, "block_tables", block_tables, pool.entries),
        _arg(pool, "seq_lens", seq_lens, batch), _arg(pool, "out", out, rows), _length(int(window)),
        _length(int(sinks)), *_rope_args(pool, rope, rope_positions, batch), batch,
        _int(int(num_splits)), _pool_stream(pool, stream))
    _check(st, "pkv_window_append_attend")


def pkv_window_prefill_attention(pool: Pool, layer, q, k_pool, v_pool, block_tables, cu_tokens,
                                 start_pos, out, max_chunk_tokens, window, sinks=0, batch=None,
                                 total_tokens=None, stream=None):
    """pkv_prefill_attention behind a window: every chunk token attends to the last
    `window` tokens up to itself and to the first `sinks` ones."""
    batch = _int(_batch(start_pos, batch))
    total = int(q.shape[0]) if total_tokens is None else _int(int(total_tokens))
    rows = total * NUM_Q_HEADS * HEAD_DIM
    st = pool._lib.pkv_window_prefill_attention(
        pool.handle, _int(int(layer)), _arg(pool, "q", q, rows),
        _arg(pool, "k_pool", k_pool, pool.elements),
        _arg(pool, "v_pool", v_pool, pool.elements),
        _arg(pool, "block_tables", block_tables, pool.entries),
        _arg(pool, "cu_tokens", cu_tokens, batch + 1), _arg(pool, "start_pos", start_pos, batch),
        _arg(pool, "out", out, rows), _length(int(window)), _length(int(sinks)),
        batch, total, _int(int(max_chunk_tokens)), _pool_stream(pool, stream))
    _check(st, "pkv_window_prefill_attention")


def pkv_prefill_fill_axes(pool: Pool, layer, q, k, v, q_out, k_pool, v_pool, block_tables,
                          cu_tokens, start_pos, rope, rope_positions, max_chunk_tokens,
                          batch=None, total_tokens=None, stream=None):
    """Writes the chunk's rotated keys and its values into their pages and its
    rotated queries into q_out (bf16; q itself, or None with q None).
    rope_positions: int32 [axes][>= T]."""
    if rope is None:
        raise ValueError("rope: missing")
    batch = _int(_batch(start_pos, batch))
    total = int(k.shape[0]) if total_tokens is None else _int(int(total_tokens))
    rows, new = total * NUM_Q_HEADS * HEAD_DIM, total * NUM_KV_HEADS * HEAD_DIM
    st = pool._lib.pkv_prefill_fill_axes(
        pool.handle, _int(int(layer)), _arg(pool, "q", q, rows), _arg(pool, "k", k, new),
        _arg(pool, "v", v, new), _arg(pool, "q_out", q_out, rows),
        _arg(pool, "k_pool", k_pool, pool.elements),
        _arg(pool, "v_pool", v_pool, pool.elements),
        _arg(pool, "block_tables", block_tables, pool.entries),
        _arg(pool, "cu_tokens", cu_tokens, batch + 1), _arg(pool, "start_pos", start_pos, batch),
        *_rope_args(pool, rope, rope_positions, total), batch, total, _int(int(max_chunk_tokens)),
        _pool_stream(pool, stream))
    _check(st, "pkv_prefill_fill_axes")


def pkv_copy_pages(pool: Pool, src, dst, k_pool, v_pool, tokens=None, n=None, stream=None):
    """Copies page src[i] to page dst[i] in both pools: whole, or its first
    tokens[i] tokens (int32 tensors on the device)."""
    n = int(src.shape[0]) if n is None else _int(int(n))
    st = pool._lib.pkv_copy_pages(
        pool.handle, _arg(pool, "src", src, n), _arg(pool, "dst", dst, n),
        _arg(pool, "tokens", tokens, n), _arg(pool, "k_pool", k_pool, pool.elements),
        _arg(pool, "v_pool", v_pool, pool.elements), n, _pool_stream(pool, stream))
    _check(st, "pkv_copy_pages")


def pkv_compact_pages(pool: Pool, src, dst, k_pool, v_pool, block_tables, n=None, stream=None):
    """Moves page src[i] to page dst[i] in both pools and rewrites the block
    tables (all layers and rows) in place."""
    n = int(src.shape[0]) if n is None else _int(int(n))
    st = pool._lib.pkv_compact_pages(
        pool.handle, _arg(pool, "src", src, n), _arg(pool, "dst", dst, n),
        _arg(pool, "k_pool", k_pool, pool.elements),
        _arg(pool, "v_pool", v_pool, pool.elements),
        _arg(pool, "block_tables", block_tables, pool.entries), n, _pool_stream(pool, stream))
    _check(st, "pkv_compact_pages")


# ---------------------------------------------------------------- admission scheduler (host)
class Scheduler:
    """Owns a pkv_sched_t: admission credits and lazy page assignment for the
    shared pool (host only; see include/pkv_sched.h)."""

    def __init__(self, handle, config, lib):
        self.handle = handle
        self.config = config
        self._lib = lib

    def close(self):
        if self.handle:
            _check(self._lib.pkv_sched_destroy(self.handle), "pkv_sched_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _sched_config(num_pages, num_layers, page_size, max_seq_len, static_batching):
    return SchedConfig(int(num_layers), int(num_pages), int(page_size), int(max_seq_len),
                       1 if static_batching else 0)


def pkv_sched_budget(prompt_tokens, max_new_tokens, num_layers=16, page_size=PAGE_SIZE,
                     max_seq_len=MAX_SEQ_LEN, lib=None):
    """(allowed new tokens, largest processed prefix, budget in pages)."""
    lib = lib or load()
    cfg = _sched_config(1, num_layers, page_size, max_seq_len, False)
    allowed, prefix, budget = ctypes.c_int(), ctypes.c_int(), ctypes.c_int64()
    _check(lib.pkv_sched_budget(ctypes.byref(cfg), int(prompt_tokens), int(max_new_tokens),
                                ctypes.byref(allowed), ctypes.byref(prefix),
                                ctypes.byref(budget)), "pkv_sched_budget")
    return allowed.value, prefix.value, budget.value


def pkv_sched_create(num_pages, num_layers=16, page_size=PAGE_SIZE, max_seq_len=MAX_SEQ_LEN,
                     static_batching=False, lib=None) -> Scheduler:
    lib = lib or load()
    cfg = _sched_config(num_pages, num_layers, page_size, max_seq_len, static_batching)
    handle = ctypes.c_void_p()
    _check(lib.pkv_sched_create(ctypes.byref(cfg), ctypes.byref(handle)), "pkv_sched_create")
    return Scheduler(handle.value, cfg, lib)


def pkv_sched_destroy(sched: Scheduler):
    sched.close()


def pkv_sched_submit(sched: Scheduler, prompt_tokens, max_new_tokens) -> int:
    """Queues a request and returns its id; PkvError(PKV_ERR_REJECTED) when
    its budget exceeds the pool."""
    rid = ctypes.c_int(-1)
    _check(sched._lib.pkv_sched_submit(sched.handle, int(prompt_tokens), int(max_new_tokens),
                                       ctypes.byref(rid)), "pkv_sched_submit")
    return rid.value


def pkv_sched_get_stats(sched: Scheduler) -> dict:
    st = SchedStats()
    _check(sched._lib.pkv_sched_get_stats(sched.handle, ctypes.byref(st)), "pkv_sched_get_stats")
    return {name: getattr(st, name) for name, _ in SchedStats._fields_}


def _id_buffer(n):
    return (ctypes.c_int * max(1, n))()


def pkv_sched_admit(sched: Scheduler) -> list:
    """One admission pass; the admitted ids in order."""
    cap = pkv_sched_get_stats(sched)["waiting"]
    buf, count = _id_buffer(cap), ctypes.c_int()
    _check(sched._lib.pkv_sched_admit(sched.handle, buf, int(cap), ctypes.byref(count)),
           "pkv_sched_admit")
    return list(buf[:count.value])


def pkv_sched_extend(sched: Scheduler, request_id, length):
    _check(sched._lib.pkv_sched_extend(sched.handle, int(request_id), int(length)),
           "pkv_sched_extend")


def pkv_sched_extend_batch(sched: Scheduler, ids, lengths):
    """pkv_sched_extend for every (id, length) pair, in one call."""
    import numpy as np
    id_buf = np.ascontiguousarray(ids, dtype=np.intc)
    len_buf = np.ascontiguousarray(lengths, dtype=np.intc)
    if id_buf.shape != len_buf.shape or id_buf.ndim != 1:
        raise ValueError("ids and lengths must be 1-D and of one length")
    _check(sched._lib.pkv_sched_extend_batch(sched.handle, id_buf.ctypes.data, len_buf.ctypes.data,
                                             int(id_buf.shape[0])), "pkv_sched_extend_batch")


def pkv_sched_finish(sched: Scheduler, request_id):
    _check(sched._lib.pkv_sched_finish(sched.handle, int(request_id)), "pkv_sched_finish")


def pkv_sched_fork(sched: Scheduler, request_id, length, max_new_tokens):
    """Forks an active request after its first `length` tokens: (child id, src,
    dst, tokens): the page copies (one per layer, or none) that the child needs
    before it is used, the first `tokens` tokens of each; int32 arrays for
    pkv_copy_pages. PkvError(PKV_ERR_REJECTED) when the free credits do not
    cover the child. Pages that the parent gave back are missing from the child
    as well: pkv_sched_held tells which tokens it has."""
    import numpy as np
    layers = sched.config.num_layers
    src, dst = np.empty(layers, np.intc), np.empty(layers, np.intc)
    rid, count, tokens = ctypes.c_int(-1), ctypes.c_int(), ctypes.c_int()
    _check(sched._lib.pkv_sched_fork(sched.handle, _int(int(request_id)), _int(int(length)),
                                     _int(int(max_new_tokens)), ctypes.byref(rid),
                                     src.ctypes.data, dst.ctypes.data, layers,
                                     ctypes.byref(count), ctypes.byref(tokens)),
           "pkv_sched_fork")
    n = count.value
    return rid.value, src[:n], dst[:n], np.full(n, tokens.value, np.intc)


def pkv_sched_held(sched: Scheduler, request_id):
    """(head, tail): the pages of the request's first `head` positions and of those
    from `tail` on are there in every layer (a whole request: head is its length,
    tail 0). Attention behind a window that starts at or after `tail`, with at
    most `head` sinks, finds every token."""
    head, tail = ctypes.c_int(), ctypes.c_int()
    _check(sched._lib.pkv_sched_held(sched.handle, _int(int(request_id)), ctypes.byref(head),
                                     ctypes.byref(tail)), "pkv_sched_held")
    return head.value, tail.value


def pkv_sched_release(sched: Scheduler, request_id, first_visible, sinks=0) -> int:
    """Gives back the request's pages all of whose positions lie in
    [sinks, first_visible); returns how many (over all layers)."""
    count = ctypes.c_int()
    _check(sched._lib.pkv_sched_release(sched.handle, _int(int(request_id)),
                                        _int(int(first_visible)), _length(int(sinks)),
                                        ctypes.byref(count)), "pkv_sched_release")
    return count.value


def pkv_sched_compact(sched: Scheduler, max_moves=None):
    """Renumbers pages so that those in use come first (at most max_moves of
    them): (src, dst) int32 arrays for pkv_compact_pages, or for
    pkv_copy_pages before tables of pkv_sched_block_tables are used."""
    import numpy as np
    cap = sched.config.num_pages if max_moves is None else int(max_moves)
    cap = _int(min(cap, sched.config.num_pages))
    src, dst = np.empty(max(cap, 1), np.intc), np.empty(max(cap, 1), np.intc)
    count = ctypes.c_int()
    _check(sched._lib.pkv_sched_compact(sched.handle, src.ctypes.data, dst.ctypes.data, cap,
                                        ctypes.byref(count)), "pkv_sched_compact")
    return src[:count.value].copy(), dst[:count.value].copy()


def pkv_sched_decode_batch(sched: Scheduler) -> list:
    """The active requests in admission order (one decode step's batch)."""
    cap = pkv_sched_get_stats(sched)["active"]
    buf, count = _id_buffer(cap), ctypes.c_int()
    _check(sched._lib.pkv_sched_decode_batch(sched.handle, buf, int(cap), ctypes.byref(count)),
           "pkv_sched_decode_batch")
    return list(buf[:count.value])


def pkv_sched_block_tables(sched: Scheduler, ids, max_batch=None, max_pages=None, out=None,
                           clear_tail=True):
    """Host block tables int32 [num_layers][max_batch][max_pages] for the batch
    `ids` (numpy array; `out` may supply a C-contiguous one to fill; with
    clear_tail False, entries past each row's pages are left as they were)."""
    import numpy as np
    ids = np.ascontiguousarray(ids, dtype=np.intc).reshape(-1)
    max_batch = len(ids) if max_batch is None else int(max_batch)
    max_pages = sched.config.max_seq_len // sched.config.page_size if max_pages is None \
        else int(max_pages)
    shape = (sched.config.num_layers, max_batch, max_pages)
    if out is None:
        out = np.empty(shape, np.int32)
    elif out.shape != shape or out.dtype != np.int32 or not out.flags.c_contiguous:
        raise ValueError(f"out must be a C-contiguous int32 array of shape {shape}")
    _check(sched._lib.pkv_sched_block_tables(sched.handle, ids.ctypes.data, len(ids),
                                             out.ctypes.data_as(ctypes.c_void_p), max_batch,
                                             max_pages, 1 if clear_tail else 0),
           "pkv_sched_block_tables")
    return out
