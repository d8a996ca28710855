"""Handles with contexts past 2,048 tokens: the calls without a context limit of
their own write where they say, bit for bit, and the others refuse before anything
is written."""

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
import window_helpers as W

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.int16)


def _handle(c):
    return pkv.pkv_pool_create(c.num_layers, c.num_pages, c.max_batch, max_seq_len=c.max_seq_len,
                               flags=pkv.PKV_FLAG_LONG_CONTEXT)


def test_whole_prefill_refuses_before_it_fills():
    c = W.Cache([40], max_seq_len=4096)
    kp, vp = c.pools(lambda b: np.zeros(40, bool), 3.0)
    was = kp.clone(), vp.clone()
    pool = _handle(c)
    q = torch.randn(40, 32, 64, device="cuda").bfloat16()
    k = torch.randn(40, 8, 64, device="cuda").bfloat16()
    out = torch.full((40, 32, 64), 7.5, device="cuda")
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    start = torch.zeros(4, dtype=torch.int32, device="cuda")[:1]
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_prefill(pool, 0, q, k, k, kp, vp, c.tables, cu, start, out, 40)
    assert e.value.status == pkv.PKV_ERR_UNSUPPORTED
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert torch.equal(_bits(kp), _bits(was[0])) and torch.equal(_bits(vp), _bits(was[1]))
    assert (out == 7.5).all()
    pool.close()
