"""Decode attention over the BF16 cache with scores of any size that FP32 holds."""

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
from window_helpers import DIM, HKV, HQ, U, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _library():
    from paged_kv_cache_210_gb300 import build as lib_build
    lib_build.build()


@pytest.mark.parametrize("splits", [1, 0, 3])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("bits", [20, 24, 31, 33, 40, 77, 116])
@pytest.mark.parametrize("windowed", [True, False])
def test_huge_scores(windowed, bits, sign, splits):
    # Keys of one dim whose scores are +-9/8 .. 15/8 2^bits: the largest are equal and share
    # the output equally, the others lie 2^(bits - 4) and more below. The products are exact
    # and equal scores get equal weights; their terms are off by 2^-17 (the full decode's two)
    # and the sums by 2 (n / 16 + 16) u.
    lens = [900, 33, 2048]
    rng = np.random.RandomState(bits)
    c = Cache(lens, seed=bits)
    codes = []
    for b, n in enumerate(lens):
        code = rng.randint(9, 16, n)
        codes.append(code)
        c.k[b] = torch.zeros(n, HKV, DIM)
        c.k[b][:, :, 11] = torch.from_numpy(sign * code / 8.0 * 2.0 ** bits)[:, None]
        c.k[b] = c.k[b].bfloat16().cuda()
    k_pool, v_pool = c.pools(lambda b: np.ones(lens[b], bool))
    q = torch.zeros(3, HQ, DIM, dtype=torch.bfloat16, device="cuda")
    q[:, :, 11] = 8.0
    out = torch.empty(3, HQ, DIM, device="cuda")
    pool = pkv.pkv_pool_create(1, c.num_pages, 3)
    if windowed:
        pkv.pkv_window_attention(pool, 0, q, k_pool, v_pool, c.tables, c.lens_tensor(), out, 2048,
                                 num_splits=splits)
    else:
        pkv.pkv_decode_attention(pool, 0, q, k_pool, v_pool, c.tables, c.lens_tensor(), out,
                                 num_splits=splits)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    for b, n in enumerate(lens):
        first = codes[b] == (codes[b].min() if sign < 0 else codes[b].max())
        x = c.v[b].double()[torch.from_numpy(first).cuda()]
        ref = x.mean(0).repeat_interleave(HQ // HKV, 0)
        tol = (2.0 ** -17 + 2.0 ** -20 + 2 * (n / 16 + 16) * U) * float(x.abs().amax())
        off = float((out[b].double() - ref).abs().max())
        assert off <= tol, (b, off, tol)
