"""Windowed, multi-axis and page entry points on the CPU: refusals that come
before any CUDA call, the long-context flag's limits, and argument marshalling."""

import ctypes
import sys

import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
from paged_kv_cache_210_gb300 import build as lib_build


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return pkv.load()


def test_null_handles_are_rejected(lib):
    assert lib.pkv_window_attention(None, 0, 16, 16, 16, 16, 16, 16, 8, 0, None, None, 0, 1, 0,
                                    None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_window_append_attend(None, 0, 16, 16, 16, 16, 16, 16, 16, 16, 8, 0, None, None,
                                        0, 1, 0, None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_window_prefill_attention(None, 0, 16, 16, 16, 16, 16, 16, 16, 8, 0, 1, 1, 1,
                                            None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_prefill_fill_axes(None, 0, 16, 16, 16, 16, 16, 16, 16, 16, 16, None, 16, 1, 1,
                                     1, 1, None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_copy_pages(None, 16, 16, None, 16, 16, 1, None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_compact_pages(None, 16, 16, 16, 16, 16, 1, None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_sched_release(None, 0, 0, 0, None) == pkv.PKV_ERR_INVALID_ARG
    n = ctypes.c_int()
    assert lib.pkv_sched_compact(None, None, None, 0, ctypes.byref(n)) == pkv.PKV_ERR_INVALID_ARG


def test_long_context_limits(lib):
    h = ctypes.c_void_p()
    for seq, flags in ((2064, 0), (2064, pkv.PKV_FLAG_PDL), (1048592, 2), (4100, 2), (0, 2)):
        cfg = pkv.PoolConfig(1, 16, 16, 32, 8, 64, seq, 1, 0, flags)
        assert lib.pkv_pool_create(ctypes.byref(cfg), ctypes.byref(h)) == pkv.PKV_ERR_INVALID_ARG


class _NoLibrary:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} reached the library")
        return call


POOL = pkv.Pool(handle=1, config=None, lib=_NoLibrary())


def _args():
    bf = dict(dtype=torch.bfloat16)
    return dict(q=torch.zeros(2, 32, 64, **bf), k=torch.zeros(2, 8, 64, **bf),
                v=torch.zeros(2, 8, 64, **bf), k_pool=torch.zeros(4, 8, 16, 64, **bf),
                v_pool=torch.zeros(4, 8, 16, 64, **bf),
                block_tables=torch.zeros(1, 2, 128, dtype=torch.int32),
                seq_lens=torch.ones(2, dtype=torch.int32), out=torch.zeros(2, 32, 64), window=8)


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(2, 32, 64)), ("k", torch.zeros(2, 8, 64, dtype=torch.float16)),
    ("v_pool", torch.zeros(4, 8, 16, 64)), ("block_tables", torch.zeros(1, 2, 128)),
    ("seq_lens", torch.ones(2, dtype=torch.int64)),
    ("out", torch.zeros(2, 64, 32).transpose(1, 2)), ("out", torch.zeros(1, 32, 64)),
    ("q", torch.zeros(1, 32, 64, dtype=torch.bfloat16))])
def test_wrong_tensors_raise_before_the_library(name, bad):
    a = _args()
    a[name] = bad
    with pytest.raises(ValueError, match=name):
        pkv.pkv_window_append_attend(POOL, 0, **a)


def test_rope_arguments():
    cos = torch.zeros(10, 32)
    rope = pkv.pkv_axes_rope(cos, cos, [0] * 16 + [1] * 16)
    assert rope.num_axes == 2 and rope.config.rows == 10
    for kw in (dict(rope=rope), dict(rope_positions=torch.zeros(2, 2, dtype=torch.int32)),
               dict(rope=rope, rope_positions=torch.zeros(1, 2, dtype=torch.int32)),
               dict(rope=rope, rope_positions=torch.zeros(2, 1, dtype=torch.int32)),
               dict(rope=rope, rope_positions=torch.zeros(2, 2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            pkv.pkv_window_append_attend(POOL, 0, **_args(), **kw)
    for c, s, axes in ((cos, cos, [0] * 33), (cos, cos, [4] * 32), (cos, cos[:5], [0] * 32),
                       (cos.double(), cos.double(), [0] * 32), (cos[:, :16], cos, [0] * 32)):
        with pytest.raises(ValueError):
            pkv.pkv_axes_rope(c, s, axes)


def test_page_lists():
    i = torch.zeros(3, dtype=torch.int32)
    p = torch.zeros(4, 8, 16, 64, dtype=torch.bfloat16)
    for kw in (dict(src=i.long(), dst=i), dict(src=i, dst=i[:2]), dict(src=i, dst=i, tokens=i[:1])):
        with pytest.raises(ValueError):
            pkv.pkv_copy_pages(POOL, k_pool=p, v_pool=p, **kw)


def test_rotary_tables_lie_on_one_device():
    """The kernels read both tables: one elsewhere is refused, not passed on."""
    here, elsewhere = torch.zeros(10, 32), torch.zeros(10, 32, device="meta")
    for cos, sin in ((here, elsewhere), (elsewhere, here)):
        with pytest.raises(ValueError, match="rope_sin"):
            pkv.pkv_axes_rope(cos, sin, [0] * 32)


class _Creates:
    """Stands in for the CUDA library: hands out handle 7 and takes it back."""

    def __init__(self):
        self.destroyed = []

    def pkv_pool_create(self, config, out):
        out._obj.value = 7
        return pkv.PKV_OK

    def pkv_pool_destroy(self, handle):
        self.destroyed.append(handle)
        return pkv.PKV_OK


def _no_torch(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)       # an import raises


def _no_device(monkeypatch):
    def current_device():
        raise RuntimeError("no CUDA device")
    monkeypatch.setattr(torch.cuda, "current_device", current_device)


@pytest.mark.parametrize("missing", [_no_torch, _no_device])
def test_a_handle_needs_no_torch(monkeypatch, missing):
    """Raw addresses do without torch: the handle is there, and owned, where torch
    or its CUDA device is not."""
    missing(monkeypatch)
    lib = _Creates()
    pool = pkv.pkv_pool_create(1, 16, 1, lib=lib)
    assert pool.handle == 7 and pool.device is None
    pool.close()
    assert lib.destroyed == [7]
