"""The 8-bit cache's and drafted trees' entry points on the CPU: refusals that come
before any CUDA call, and argument marshalling."""

import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
from paged_kv_cache_210_gb300 import build as lib_build


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return pkv.load()


def test_null_handles_are_rejected(lib):
    p = 16
    assert lib.pkv_quant_fill(None, 0, p, p, p, p, p, p, None, None, 0, 1, 1, 1,
                              None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_quant_read(None, 0, p, p, p, p, p, p, 1, 1, 1, None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_quant_attention(None, 0, p, p, p, p, p, 8, 0, None, None, 0, 1, 0,
                                   None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_quant_append_attend(None, 0, p, p, p, p, p, p, p, 8, 0, None, None, 0, 1, 0,
                                       None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_tree_attention(None, 0, p, p, p, p, p, p, p, p, 8, 0, 1, 1,
                                  None) == pkv.PKV_ERR_INVALID_ARG
    assert lib.pkv_tree_commit(None, p, p, p, p, p, p, 1, 1, None) == pkv.PKV_ERR_INVALID_ARG


class _NoLibrary:
    def __getattr__(self, name):
        def call(*args):
            raise AssertionError(f"{name} reached the library")
        return call


class _Records:
    def __getattr__(self, name):
        def call(*args):
            self.__dict__.setdefault("calls", []).append((name, args))
            return pkv.PKV_OK
        return call


def _pool(lib):
    return pkv.Pool(handle=1, config=None, lib=lib)


BF = dict(dtype=torch.bfloat16)
I32 = dict(dtype=torch.int32)


def _quant():
    return dict(q=torch.zeros(2, 32, 64, **BF), k=torch.zeros(2, 8, 64, **BF),
                v=torch.zeros(2, 8, 64, **BF),
                kv_pool=torch.zeros(4, 8, pkv.PKV_QUANT_TILE_BYTES, dtype=torch.uint8),
                block_tables=torch.zeros(1, 2, 128, **I32), seq_lens=torch.ones(2, **I32),
                out=torch.zeros(2, 32, 64), window=8, stream=0)


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(2, 32, 64)), ("q", torch.zeros(1, 32, 64, **BF)),
    ("k", torch.zeros(2, 8, 64, dtype=torch.float16)), ("v", torch.zeros(1, 8, 64, **BF)),
    ("kv_pool", torch.zeros(4, 8, 2080, dtype=torch.int8)),
    ("kv_pool", torch.zeros(4, 16, 2080, dtype=torch.uint8)[:, ::2]),
    ("block_tables", torch.zeros(1, 2, 128)), ("seq_lens", torch.ones(2, dtype=torch.int64)),
    ("out", torch.zeros(2, 64, 32).transpose(1, 2)), ("out", torch.zeros(1, 32, 64))])
def test_wrong_tensors_of_the_decode_raise_before_the_library(name, bad):
    a = _quant()
    a[name] = bad
    with pytest.raises(ValueError, match=name):
        pkv.pkv_quant_append_attend(_pool(_NoLibrary()), 0, **a)


def _rows():
    return dict(k=torch.zeros(5, 8, 64, **BF), v=torch.zeros(5, 8, 64, **BF),
                kv_pool=torch.zeros(4, 8, 2080, dtype=torch.uint8),
                block_tables=torch.zeros(1, 2, 128, **I32),
                cu_tokens=torch.tensor([0, 2, 5], **I32), start_pos=torch.zeros(2, **I32),
                max_chunk_tokens=3, stream=0)


@pytest.mark.parametrize("call", [pkv.pkv_quant_fill, pkv.pkv_quant_read])
@pytest.mark.parametrize("name,bad", [
    ("k", torch.zeros(5, 8, 64)), ("v", torch.zeros(4, 8, 64, **BF)),
    ("cu_tokens", torch.zeros(2, **I32)), ("start_pos", torch.zeros(2, dtype=torch.int64))])
def test_wrong_tensors_of_the_store_raise_before_the_library(call, name, bad):
    a = _rows()
    a[name] = bad
    with pytest.raises(ValueError, match=name):
        call(_pool(_NoLibrary()), 0, **a)


def test_rope_of_a_fill():
    cos = torch.zeros(10, 32)
    rope = pkv.pkv_axes_rope(cos, cos, [0] * 16 + [1] * 16)
    for kw in (dict(rope=rope), dict(rope_positions=torch.zeros(2, 5, **I32)),
               dict(rope=rope, rope_positions=torch.zeros(1, 5, **I32)),
               dict(rope=rope, rope_positions=torch.zeros(2, 4, **I32))):
        with pytest.raises(ValueError, match="rope"):
            pkv.pkv_quant_fill(_pool(_NoLibrary()), 0, **_rows(), **kw)


@pytest.mark.parametrize("name,bad", [
    ("q", torch.zeros(5, 32, 64)), ("tree", torch.zeros(5, **I32)),
    ("tree", torch.zeros(4, dtype=torch.int64)), ("out", torch.zeros(4, 32, 64)),
    ("cu_tokens", torch.zeros(2, **I32)), ("k_pool", torch.zeros(4, 8, 16, 64))])
def test_wrong_tensors_of_a_tree_raise_before_the_library(name, bad):
    a = dict(q=torch.zeros(5, 32, 64, **BF), k_pool=torch.zeros(4, 8, 16, 64, **BF),
             v_pool=torch.zeros(4, 8, 16, 64, **BF), block_tables=torch.zeros(1, 2, 128, **I32),
             cu_tokens=torch.tensor([0, 2, 5], **I32), start_pos=torch.zeros(2, **I32),
             tree=torch.zeros(5, dtype=torch.int64), out=torch.zeros(5, 32, 64), window=8, stream=0)
    a[name] = bad
    with pytest.raises(ValueError, match=name):
        pkv.pkv_tree_attention(_pool(_NoLibrary()), 0, **a)


def test_counts_that_no_c_int_holds_are_refused_ones():
    lib = _Records()
    pool = _pool(lib)
    a = _quant()
    a["window"] = 1 << 40
    pkv.pkv_quant_append_attend(pool, 1 << 40, **a, sinks=-(1 << 40), num_splits=1 << 33)
    (name, args), = lib.calls
    assert name == "pkv_quant_append_attend"
    assert args[1] == -1 and args[9] == 2 ** 31 - 1 and args[10] == -1 and args[15] == -1
    lib.calls.clear()
    acc = torch.zeros(2, 3, **I32)
    pkv.pkv_tree_commit(pool, torch.zeros(4, 8, 16, 64, **BF), torch.zeros(4, 8, 16, 64, **BF),
                        torch.zeros(1, 2, 128, **I32), torch.zeros(2, **I32), acc,
                        torch.zeros(2, **I32), stream=0)
    (name, args), = lib.calls
    assert name == "pkv_tree_commit" and args[7:9] == (2, 3)
