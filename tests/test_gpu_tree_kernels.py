"""Attention of drafted trees through each of its kernels: clusters, the line of few
rows with its join, and the tile kernel with its join. Which one a call takes goes by
its drafted tokens per sequence and by the context that its sequences may see."""

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
from tree_helpers import pack
from window_helpers import DIM, HKV, HQ, U, Cache

pytestmark = pytest.mark.gpu

# max_seq_len, committed and drafted tokens: 8 and fewer tokens on average over short and
# long contexts, more of them over long ones
KERNELS = {"clusters": (2048, [900, 30], [8, 5]), "line": (16384, [900, 3000], [8, 5]),
           "tiles": (16384, [900, 3000], [40, 17])}


@pytest.fixture(autouse=True, scope="module")
def _library():
    from paged_kv_cache_210_gb300 import build as lib_build
    lib_build.build()


def int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def handle(c):
    return pkv.pkv_pool_create(c.num_layers, c.num_pages, c.max_batch, max_seq_len=c.max_seq_len,
                               flags=pkv.PKV_FLAG_LONG_CONTEXT if c.max_seq_len > 2048 else 0)


def chain(n):
    return [(1 << i + 1) - 1 for i in range(n)]


@pytest.mark.parametrize("kernel", [*KERNELS, "windowed prefill"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("bits", [20, 23, 24, 31, 33, 40, 77, 116])
def test_huge_scores(bits, sign, kernel):
    # Keys of one dim whose scores are +-9/8 .. 15/8 2^bits: the largest that a row sees are
    # equal and share its output equally, the others lie 2^(bits - 4) and more below. The
    # products are exact and equal scores get equal weights, so what is left of the
    # tolerance is the sums, three BF16 terms and the joins' exponentials (2^-22 each).
    max_seq_len, starts, nodes = KERNELS.get(kernel, KERNELS["tiles"])
    rng = np.random.RandomState(bits)
    c = Cache([s + n for s, n in zip(starts, nodes)], max_seq_len=max_seq_len, seed=bits)
    codes = []
    for b, n in enumerate(c.lens):
        code = rng.randint(9, 16, n)
        code[rng.permutation(n)[:3]] = 9 if sign < 0 else 15
        codes.append(code)
        c.k[b] = torch.zeros(n, HKV, DIM)
        c.k[b][:, :, 11] = torch.from_numpy(sign * code / 8.0 * 2.0 ** bits)[:, None]
        c.k[b] = c.k[b].bfloat16().cuda()
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    total = sum(nodes)
    q = torch.zeros(total, HQ, DIM, dtype=torch.bfloat16, device="cuda")
    q[:, :, 11] = 8.0
    out = torch.empty(total, HQ, DIM, device="cuda")
    pool, cu = handle(c), int32(np.cumsum([0] + nodes))
    if kernel in KERNELS:
        pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, int32(starts),
                               pack(sum([chain(n) for n in nodes], [])), out, max_seq_len)
    else:
        pkv.pkv_window_prefill_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, int32(starts), out,
                                         max(nodes), max_seq_len)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    row = 0
    for b, n in enumerate(nodes):
        v, code = c.v[b].double(), codes[b]
        for i in range(n):
            seen = code[:starts[b] + i + 1]
            first = torch.from_numpy(np.nonzero(seen == (seen.min() if sign < 0 else seen.max()))[0])
            x = v[first.cuda()]
            ref = x.mean(0).repeat_interleave(HQ // HKV, 0)
            tol = (2.0 ** -20 + 2 * (c.lens[b] / 16 + 16) * U) * float(x.abs().amax())
            off = float((out[row].double() - ref).abs().max())
            assert off <= tol, (b, i, off, tol)
            row += 1
