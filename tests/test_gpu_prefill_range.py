"""Full-context prefill attention up to the largest scores that it is documented for."""

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


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("bits", [20, 24, 28, 29])
def test_large_scores(bits, sign):
    # Keys of one dim whose scores are +-9/8 .. 15/8 2^bits: the largest that a row sees are
    # equal and share its output equally, the others lie 2^(bits - 4) and more below. The
    # products are exact and equal scores get equal weights; two BF16 terms of them are off by
    # 2^-17 (the second's half step), and the sums by 2 (n / 16 + 16) u.
    starts, nodes = [900, 0, 300], [140, 33, 300]
    rng = np.random.RandomState(bits)
    c = Cache([s + n for s, n in zip(starts, nodes)], seed=bits)
    codes = []
    for b, n in enumerate(c.lens):
        code = rng.randint(9, 16, n)
        codes.append(code)
        c.k[b] = torch.zeros(n, HKV, DIM)
        c.k[b][:, :, 11] = torch.from_numpy(sign * code / 8.0 * 2.0 ** bits)[:, None]
        c.k[b] = c.k[b].bfloat16().cuda()
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    total = sum(nodes)
    q = torch.zeros(total, HQ, DIM, dtype=torch.bfloat16, device="cuda")
    q[:, :, 11] = 8.0
    out = torch.empty(total, HQ, DIM, device="cuda")
    pool = pkv.pkv_pool_create(1, c.num_pages, 3)
    cu = torch.tensor(np.cumsum([0] + nodes), dtype=torch.int32).cuda()
    pkv.pkv_prefill_attention(pool, 0, q, k_pool, v_pool, c.tables, cu,
                              torch.tensor(starts, dtype=torch.int32).cuda(), out, max(nodes))
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    row = 0
    for b, n in enumerate(nodes):
        v, code = c.v[b].double(), codes[b]
        for i in range(n):
            seen = code[:starts[b] + i + 1]
            first = torch.from_numpy(np.nonzero(seen == (seen.min() if sign < 0 else seen.max()))[0])
            x = v[first.cuda()]
            ref = x.mean(0).repeat_interleave(HQ // HKV, 0)
            tol = (2.0 ** -17 + 2.0 ** -20 + 2 * (c.lens[b] / 16 + 16) * U) * float(x.abs().amax())
            off = float((out[row].double() - ref).abs().max())
            assert off <= tol, (b, i, off, tol)
            row += 1
