"""The 8-bit decode on the GPU over the range of scores and values that a cache may
hold, against a 64-bit restatement, with tolerances that go by what each token weighs."""

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
from quant_helpers import QuantCache, attend, quantise
from window_helpers import DIM, HKV, HQ, U, check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _library():
    from paged_kv_cache_210_gb300 import build as lib_build
    lib_build.build()


def int32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def run_scores_and_sizes(score, size, window=2048, sinks=0, splits=1, seed=0):
    """Token t has base-e score score[t] and V of size[t] times normal values; every
    head's query and keys have one dim, so products and scores are exact and the rest
    of the arithmetic can be held to what each token weighs. p the weights, V_t the
    largest |v| of a row, A = sum p V / sum p. A weight is off by e = 3 u (|s| + |s_max| +
    8) + 2^-21 (the exponent's argument; its base-2 exponential here and in the merge) and
    2^-22 (two FP16 terms), or by 2^-32 of the largest weighted row and code, 2^-31
    max p V; the sums by 2 (n / 16 + 16) u A."""
    n = len(score)
    c = QuantCache([n], seed=seed)
    pool, kv = pkv.pkv_pool_create(1, c.num_pages, 1), c.pool()
    g = torch.Generator().manual_seed(seed)
    ks = torch.zeros(n, HKV, DIM)
    ks[:, :, 5] = torch.as_tensor(score)[:, None]
    vs = torch.randn(n, HKV, DIM, generator=g) * torch.as_tensor(size)[:, None, None]
    ks, vs = ks.bfloat16(), vs.bfloat16()
    q = torch.zeros(1, HQ, DIM, dtype=torch.bfloat16, device="cuda")
    q[:, :, 5] = 8.0
    pkv.pkv_quant_fill(pool, 0, ks.cuda(), vs.cuda(), kv, c.tables, int32([0, n]), int32([0]), n)
    out = torch.empty(1, HQ, DIM, device="cuda")
    pkv.pkv_quant_attention(pool, 0, q, kv, c.tables, c.lens_tensor(), out, window, sinks=sinks,
                            num_splits=splits)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    t = torch.arange(n)
    seen = (t > n - 1 - window) | (t < sinks)
    s = quantise(ks.double())[2][seen][:, :, 5].T                    # [8][tokens]
    v = quantise(vs.double())[2][seen].permute(1, 0, 2)              # [8][tokens][64]
    w = torch.exp(s - s.amax(1, keepdim=True))
    total = w.sum(1, keepdim=True)
    ref = (w[:, None] @ v)[:, 0] / total
    most = v.abs().amax(2)
    a = (w * most).sum(1, keepdim=True) / total
    e = 3 * U * (s.abs() + s.abs().amax(1, keepdim=True) + 8) + 2.0 ** -21 + 2.0 ** -22
    tol = ((w * e * most).sum(1, keepdim=True) + (w * e).sum(1, keepdim=True) * a) / total + \
        2 * (seen.sum() / 16 + 16) * U * a + \
        seen.sum() * 2.0 ** -31 * (w * most).amax(1, keepdim=True) / total
    off = (out[0].double().cpu() - ref.repeat_interleave(HQ // HKV, 0)).abs()
    worst = float((off / tol.repeat_interleave(HQ // HKV, 0)).amax())
    assert worst <= 1, worst


@pytest.mark.parametrize("splits", [1, 0])
@pytest.mark.parametrize("bits,down", [(20, 72), (35, 72), (60, 72), (100, 72), (40, 16), (24, 16),
                                       (60, 40)])
@pytest.mark.parametrize("where", ["first", "sinks", "middle"])
def test_large_values_whose_weights_become_small(where, bits, down, splits):
    # every warp meets V of 2^bits with scores `down` below those that follow, whose V is
    # of ordinary size (or, in the middle, lies on both sides)
    n = 600
    rng = np.random.RandomState(bits)
    score, size = rng.randn(n), np.ones(n)
    rows = slice(128, 256) if where == "middle" else slice(0, 128)
    score[rows] -= down
    size[rows] = 2.0 ** bits
    kw = dict(window=300, sinks=100) if where == "sinks" else {}
    run_scores_and_sizes(score, size, splits=splits, seed=bits, **kw)


@pytest.mark.parametrize("step,bits", [(16, 20), (16, 26), (12, 30), (3, 5), (40, 20)])
def test_values_that_shrink_as_scores_rise(step, bits):
    # in every group of a warp again: V 2^-bits of the last one's, scores `step` above
    group = np.arange(640) // 128
    run_scores_and_sizes(group * step + np.random.RandomState(step).randn(640) / 4,
                         2.0 ** (bits * (2.0 - group)), seed=bits)


@pytest.mark.parametrize("splits", [1, 0, 3])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("bits", [20, 23, 24, 30, 31, 33, 40, 77, 120])
@pytest.mark.parametrize("least", [8, 9])      # as a largest score exact in base 2, or not
def test_huge_scores(least, bits, sign, splits):
    # Scores of 2^bits, all different values of a code apart and each taken by tokens of
    # several groups: those of the largest share the output equally, the others, 2^(bits -
    # 4) or more below it, have no part of it. Equal scores get equal weights, so what is
    # left of the tolerance above is the sums and the terms.
    n = 700
    rng = np.random.RandomState(bits)
    code = rng.randint(least, 16, n)
    code[rng.permutation(n)[:3]] = least if sign < 0 else 15
    c = QuantCache([n], seed=bits)
    pool, kv = pkv.pkv_pool_create(1, c.num_pages, 1), c.pool()
    ks = torch.zeros(n, HKV, DIM)
    ks[:, :, 7] = torch.from_numpy(sign * code / 8.0 * 2.0 ** bits)[:, None]
    vs = torch.randn(n, HKV, DIM, generator=torch.Generator().manual_seed(bits)).bfloat16()
    q = torch.zeros(1, HQ, DIM, dtype=torch.bfloat16, device="cuda")
    q[:, :, 7] = 8.0
    pkv.pkv_quant_fill(pool, 0, ks.bfloat16().cuda(), vs.cuda(), kv, c.tables, int32([0, n]),
                       int32([0]), n)
    out = torch.empty(1, HQ, DIM, device="cuda")
    pkv.pkv_quant_attention(pool, 0, q, kv, c.tables, c.lens_tensor(), out, 2048, num_splits=splits)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    first = torch.from_numpy(code == (code.min() if sign < 0 else code.max()))
    v = quantise(vs.double())[2][first]                              # [tokens][8][64]
    ref, most = v.mean(0), v.abs().amax((0, 2))[:, None]
    tol = (2.0 ** -21 + 2 * (n / 16 + 16) * U) * most
    off = (out[0].double().cpu() - ref.repeat_interleave(HQ // HKV, 0)).abs()
    worst = float((off / tol.repeat_interleave(HQ // HKV, 0)).amax())
    assert worst <= 1, worst


@pytest.mark.parametrize("below", [0, 20, 31])
def test_query_dims_far_below_the_largest(below):
    # down to 2^-31 of a head's largest dim, where no key is, a query's dims keep every
    # bit: the scores are the other dims' alone, with keys larger by as much
    n = 300
    c = QuantCache([n], seed=below)
    pool, kv = pkv.pkv_pool_create(1, c.num_pages, 1), c.pool()
    g = torch.Generator().manual_seed(below)
    ks = (torch.randn(n, HKV, DIM, generator=g) * 2.0 ** below).bfloat16()
    vs = torch.randn(n, HKV, DIM, generator=g).bfloat16()
    q = (torch.rand(1, HQ, DIM, generator=g) + 1.0) * 2.0 ** -below
    q[:, :, 0] = 1.99
    q = q.bfloat16()
    ks[:, :, 0] = 0
    pkv.pkv_quant_fill(pool, 0, ks.cuda(), vs.cuda(), kv, c.tables, int32([0, n]), int32([0]), n)
    out = torch.empty(1, HQ, DIM, device="cuda")
    pkv.pkv_quant_attention(pool, 0, q.cuda(), kv, c.tables, c.lens_tensor(), out, 2048)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    ref, tol = attend(q.double(), quantise(ks.double())[2], quantise(vs.double())[2],
                      torch.tensor([n - 1]), 2048, 0)
    check(out.cpu(), ref, tol)


def test_the_smallest_weights_that_count():
    # one token's score lies 115 base-2 units below the others', its V 2^110 above
    score, size = np.zeros(200), np.ones(200)
    score[150], size[150] = -80.0, 2.0 ** 110
    run_scores_and_sizes(score, size)


@pytest.mark.parametrize("splits", [0, 1, 4])
def test_pages_moved_by_rows_of_the_tensor(splits):
    # a page is row i of the tensor, whole: moved elsewhere, with the table's entries, the
    # same outputs come bit for bit; so do those of a fork that shares all pages but its
    # last, which was copied
    lens = [900, 40, 2048, 5]
    c = QuantCache(lens, seed=1, spare=9)
    kv = c.pool()
    pool = pkv.pkv_pool_create(1, c.num_pages, 4)
    q = torch.randn(4, HQ, DIM, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()

    def attend_with(kv, tables, lens):
        out = torch.empty(4, HQ, DIM, device="cuda")
        pkv.pkv_quant_attention(pool, 0, q, kv, tables, int32(lens), out, 1500, sinks=20,
                                num_splits=splits)
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK
        return out

    want = attend_with(kv, c.tables, lens)
    for seed in range(2):
        to = torch.randperm(c.num_pages, generator=torch.Generator().manual_seed(seed)).cuda()
        moved = torch.empty_like(kv)
        moved[to] = kv
        tables = torch.where(c.tables >= 0, to[c.tables.clamp(min=0).long()].int(), -1)
        assert torch.equal(attend_with(moved, tables, lens), want)
    spare = sorted(set(range(c.num_pages)) - set(c.table[c.table >= 0].tolist()))[0]
    forked, tables = kv.clone(), c.tables.clone()
    forked[spare] = forked[int(tables[0, 0, 56])]          # 900 tokens: the last page is 56
    tables[0, 1, :56], tables[0, 1, 56] = tables[0, 0, :56], spare
    q[1] = q[0]
    out = attend_with(forked, tables, [900, 900, 2048, 5])
    assert torch.equal(out[0], out[1]) and torch.equal(out[2], want[2])


def test_a_context_of_a_million_tokens():
    n = pkv.PKV_MAX_LONG_CONTEXT
    pages = n // 16 + 3
    pool = pkv.pkv_pool_create(1, pages, 1, max_seq_len=n, flags=pkv.PKV_FLAG_LONG_CONTEXT)
    g = torch.Generator(device="cuda").manual_seed(1)
    tables = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:n // 16]
    tables = tables.int().view(1, 1, -1).cuda()
    kv = torch.zeros(pages, HKV, pkv.PKV_QUANT_TILE_BYTES, dtype=torch.uint8, device="cuda")
    # V grows along the context, so that a part lost or taken twice shows (2^-9 of it and more);
    # of n / 16 additions no more than 512 come one after the other (those of a warp's pages
    # and of the parts)
    k = (torch.randn(n, HKV, DIM, generator=g, device="cuda") / 8).bfloat16()
    v = (torch.arange(n, device="cuda") / n).bfloat16()[:, None, None].expand(n, HKV, DIM).contiguous()
    q = torch.randn(1, HQ, DIM, generator=g, device="cuda").bfloat16()
    pkv.pkv_quant_fill(pool, 0, k, v, kv, tables, int32([0, n]), int32([0]), n)
    pkv.pkv_quant_read(pool, 0, kv, tables, int32([0, n]), int32([0]), k, v, n)
    out = torch.empty(1, HQ, DIM, device="cuda")
    for window, sinks in ((n, 0), (500000, 100)):
        pkv.pkv_quant_attention(pool, 0, q, kv, tables, int32([n]), out, window, sinks=sinks)
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK
        ref, tol = attend(q.double(), k.double(), v.double(), torch.tensor([n - 1], device="cuda"),
                          window, sinks)
        count = min(n, window + sinks)
        check(out, ref, tol - 2 * (count / 16 - 512) * U)


@pytest.mark.parametrize("batch,longest", [(3, 2048), (40, 1500), (200, 300)])
def test_programmatic_steps_of_several_layers(batch, longest):
    # prompts filled, then steps of three layers: the same bytes and outputs as with ordinary
    # launches, one by one and in a replayed graph
    layers, steps = 3, 4
    rng = np.random.RandomState(batch)
    prompt = [int(x) for x in rng.randint(1, longest - steps, batch)]
    needed = [-(-(n + steps) // 16) for n in prompt]
    pages = layers * sum(needed) + 5
    table = np.full((layers, batch, 128), -1, np.int32)
    ids = iter(rng.permutation(pages))
    for layer in range(layers):
        for b in range(batch):
            table[layer, b, :needed[b]] = [next(ids) for _ in range(needed[b])]
    tables = torch.from_numpy(table).cuda()
    cu, zeros = int32(np.cumsum([0] + prompt).tolist()), int32([0] * batch)
    lens = [int32([n + step + 1 for n in prompt]) for step in range(steps)]
    g = torch.Generator(device="cuda").manual_seed(2)

    def rows(n, heads):
        return torch.randn(n, heads, DIM, generator=g, device="cuda").bfloat16()

    ks = [rows(sum(prompt), HKV) for _ in range(layers)]
    new = [[rows(batch, h) for h in (HQ, HKV, HKV)] for _ in range(layers * steps)]

    def run(flags, replays):
        pool = pkv.pkv_pool_create(layers, pages, batch, flags=flags)
        kv = torch.zeros(pages, HKV, pkv.PKV_QUANT_TILE_BYTES, dtype=torch.uint8, device="cuda")
        outs = [torch.zeros(batch, HQ, DIM, device="cuda") for _ in new]

        def go():
            for layer, k in enumerate(ks):
                pkv.pkv_quant_fill(pool, layer, k, k, kv, tables, cu, zeros, max(prompt))
            for i, (q, k, v) in enumerate(new):
                pkv.pkv_quant_append_attend(pool, i % layers, q, k, v, kv, tables, lens[i // layers],
                                            outs[i], 2048)

        go()
        if replays:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.stream(s):
                with torch.cuda.graph(graph, stream=s):
                    go()
            for _ in range(replays):
                graph.replay()
        torch.cuda.synchronize()
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK
        return [kv, *outs]

    want = run(0, 0)
    for replays in (0, 10):
        assert all(torch.equal(a, b) for a, b in zip(run(pkv.PKV_FLAG_PDL, replays), want))
