"""Windowed decode and prefill attention with sinks against the 64-bit
restatement (window_helpers): every slot that no query sees holds NaN,
infinities or huge values, every page without a visible token is unassigned."""

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
import window_helpers as W

pytestmark = pytest.mark.gpu

SECTIONS = {1: [0] * 32, 2: [i % 2 for i in range(32)], 3: [0] * 8 + [1] * 12 + [2] * 12,
            4: [(5 * i) % 4 for i in range(32)]}


def _pool(c, flags=0, max_splits=0):
    if c.max_seq_len > 2048:
        flags |= pkv.PKV_FLAG_LONG_CONTEXT
    return pkv.pkv_pool_create(c.num_layers, c.num_pages, c.max_batch, max_seq_len=c.max_seq_len,
                               max_splits=max_splits, flags=flags)


def _decode(lens, window, sinks, fused=False, axes=0, num_splits=0, max_seq_len=2048, seed=1,
            junk="mixed", pool=None, k_scale=1.0, stream=None, **kw):
    """One call against the restatement; returns (worst error over tolerance, cache)."""
    w = min(window, 1 << 40)
    c = W.Cache(lens, max_seq_len, seed, k_scale=k_scale,
                evict=lambda b: W.unseen_pages(lens[b], lens[b] - 1, w, sinks), **kw)
    # fused: the slot of the new token holds junk as well before the call
    kp, vp = c.pools(lambda b: W.seen_by_last(lens[b], w, sinks) &
                     ~((np.arange(lens[b]) == lens[b] - 1) & fused), junk)
    before = kp.clone(), vp.clone()
    B = len(lens)
    q = torch.randn(B, 32, 64, generator=c.gen, device="cuda").bfloat16()
    new = [torch.stack([t[b][-1] if lens[b] else torch.zeros(8, 64, device="cuda").bfloat16()
                        for b in range(B)]) for t in (c.k, c.v)]
    rope = {}
    q64 = q.double()
    if axes:
        cos, sin = W.angles(4000)
        pos = torch.randint(0, 4000, (axes, B + 3), generator=c.gen, device="cuda").int()
        rope = dict(rope=pkv.pkv_axes_rope(cos, sin, SECTIONS[axes]), rope_positions=pos)
        q64 = W.rotate(q, cos, sin, pos[:, :B], SECTIONS[axes], torch.float64)
    own_pool = pool or _pool(c)
    out = torch.full((B, 32, 64), 7.5, device="cuda")
    torch.cuda.synchronize()
    args = (kp, vp, c.tables, c.lens_tensor(), out, window)
    if fused:
        pkv.pkv_window_append_attend(own_pool, c.layer, q, *new, *args, sinks=sinks,
                                     num_splits=num_splits, stream=stream, **rope)
    else:
        pkv.pkv_window_attention(own_pool, c.layer, q, *args, sinks=sinks, num_splits=num_splits,
                                 stream=stream, **rope)
    torch.cuda.synchronize()
    assert pkv.pkv_get_error(own_pool) == pkv.PKV_OK
    worst = 0.0
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 7.5).all()
            continue
        if fused:
            key = new[0][b]
            if axes:
                key = W.rotate(key[None], cos, sin, pos[:, b:b + 1], SECTIONS[axes],
                               torch.float32)[0].bfloat16()
            page, slot = int(c.table[c.layer, b, (n - 1) // 16]), (n - 1) % 16
            for pool_, was, row in ((kp, before[0], key), (vp, before[1], new[1][b])):
                assert torch.equal(pool_[page, :, slot].view(torch.int16), row.view(torch.int16))
                was[page, :, slot] = row
            c.k[b][-1] = key
        ref, tol = W.attend(q64[b:b + 1], c.k[b].double(), c.v[b].double(),
                            torch.tensor([n - 1], device="cuda"), w, sinks)
        worst = max(worst, W.check(out[b:b + 1], ref, tol, f"len {n} window {window} sinks {sinks}"))
    for pool_, was in ((kp, before[0]), (vp, before[1])):   # nothing else was written
        assert torch.equal(pool_.view(torch.int16), was.view(torch.int16))
    if pool is None:
        own_pool.close()
    return worst, c


LENS = [1, 2, 15, 16, 17, 31, 33, 64, 100, 257, 513, 1024, 2000, 2047, 2048]


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 512, 2048, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 16, 21, 2 ** 31 - 1])
def test_decode_lengths(window, sinks):
    _decode(LENS, window, sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (33, 17), (700, 4), (2048, 0)])
@pytest.mark.parametrize("axes", [0, 1, 3])
def test_append_attend_lengths(window, sinks, axes):
    _decode(LENS, window, sinks, fused=True, axes=axes, seed=3)


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_rotated_queries_without_append(axes):
    _decode([5, 100, 2048], 300, 4, axes=axes, seed=5)


@pytest.mark.parametrize("num_splits", [1, 2, 3, 5, 8, 13, 16, 17, 33, 64])
@pytest.mark.parametrize("fused", [False, True])
def test_explicit_splits(num_splits, fused):
    _decode([1, 40, 777, 2048], 1500, 4, fused=fused, num_splits=num_splits, seed=7)


@pytest.mark.parametrize("batch", [1, 2, 3, 7, 20, 80, 256])
def test_batches(batch):
    rng = np.random.RandomState(batch)
    lens = rng.randint(1, 700, batch).tolist()
    _decode(lens, 256, 4, fused=True, axes=3, seed=batch)


def test_padding_rows_are_left_alone():
    _decode([0, 5, 0, 300, 0], 64, 4, fused=True, axes=2)
    _decode([0], 64, 4)


def test_large_scores():
    """Keys 30 times larger: weights spread over hundreds of binades."""
    _decode([3, 200, 2048], 512, 4, k_scale=30.0)


@pytest.mark.parametrize("n,window,sinks,num_splits", [
    (70000, 2 ** 31 - 1, 0, 0), (70000, 4096, 4, 0), (70001, 40000, 100, 3), (65537, 65537, 0, 1),
    (69999, 1, 69999, 16)])
def test_long_context(n, window, sinks, num_splits):
    _decode([n, 17, n - 1], window, sinks, fused=True, axes=1, num_splits=num_splits,
            max_seq_len=81920)


def test_pages_past_four_gib():
    """Page ids whose byte offset passes 2^32 and element offset 2^31."""
    _decode([100, 2048], 256, 4, fused=True, junk=float("nan"), base_page=280000)


def test_second_layer_and_wider_tables():
    _decode([300, 40], 100, 4, fused=True, num_layers=3, layer=2, max_batch=5)


def test_lists_that_start_anywhere():
    """seq_lens, positions, cu_tokens and start_pos taken as slices."""
    c = W.Cache([40, 33])
    kp, vp = c.pools(lambda b: np.ones(c.lens[b], bool), 0.0)
    pool = _pool(c)
    q = torch.randn(2, 32, 64, device="cuda").bfloat16()
    lens = torch.tensor([7, 40, 33], dtype=torch.int32, device="cuda")[1:]
    flat = torch.zeros(5, dtype=torch.int32, device="cuda")[1:]
    cos, sin = W.angles(4)
    rope = pkv.pkv_axes_rope(cos, sin, SECTIONS[2])
    a, b = torch.zeros(2, 32, 64, device="cuda"), torch.zeros(2, 32, 64, device="cuda")
    pkv.pkv_window_attention(pool, 0, q, kp, vp, c.tables, lens, a, 16, rope=rope,
                             rope_positions=flat.view(2, 2))
    pkv.pkv_window_attention(pool, 0, q, kp, vp, c.tables, c.lens_tensor(), b, 16)
    assert torch.equal(a, b)            # angle 0 leaves the queries as they are
    cu = torch.tensor([9, 0, 1, 2], dtype=torch.int32, device="cuda")[1:]
    start = torch.tensor([9, 39, 32], dtype=torch.int32, device="cuda")[1:]
    pkv.pkv_window_prefill_attention(pool, 0, q, kp, vp, c.tables, cu, start, a, 1, 16)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert (a - b).abs().max().item() <= 2e-5 * b.abs().max().item()
    pool.close()


def test_other_stream():
    s = torch.cuda.Stream()
    _decode([300, 40, 2048], 100, 4, fused=True, stream=s)


def test_flags_bad_data_and_recovers():
    lens = [40, 40, 40, 40, 40]
    c = W.Cache(lens)
    kp, vp = c.pools(lambda b: np.ones(40, bool))
    pool = _pool(c)
    q = torch.randn(5, 32, 64, device="cuda").bfloat16()
    k = torch.randn(5, 8, 64, device="cuda").bfloat16()
    cos, sin = W.angles(100)
    rope = pkv.pkv_axes_rope(cos, sin, SECTIONS[2])
    pos = torch.full((2, 5), 39, dtype=torch.int32, device="cuda")

    def run(lens_, pos_=pos, tables=c.tables):
        out = torch.full((5, 32, 64), 7.5, device="cuda")
        pkv.pkv_window_append_attend(pool, 0, q, k, k, kp, vp, tables,
                                     torch.tensor(lens_, dtype=torch.int32, device="cuda"), out, 16,
                                     sinks=4, rope=rope, rope_positions=pos_)
        return out, pkv.pkv_get_error(pool)

    def right(out, rows, sinks=4):
        """The split of a sequence depends on the batch, so its last bits may."""
        keys = W.rotate(k, cos, sin, pos, SECTIONS[2], torch.float32).bfloat16()
        q64 = W.rotate(q, cos, sin, pos, SECTIONS[2], torch.float64)
        for b in rows:
            kk, vv = c.k[b].double().clone(), c.v[b].double().clone()
            kk[39], vv[39] = keys[b].double(), k[b].double()
            ref, tol = W.attend(q64[b:b + 1], kk, vv, torch.tensor([39], device="cuda"), 16, sinks)
            W.check(out[b:b + 1], ref, tol, f"sequence {b}")

    good, st = run(lens)
    assert st == pkv.PKV_OK
    right(good, range(5))
    for bad in (2049, -1, 2 ** 31 - 1, -2 ** 31):
        out, st = run([40, bad, 40, 40, 40])
        assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[1] == 7.5).all()
        right(out, [0, 2, 3, 4])
    for bad in (-1, 100, 2 ** 31 - 1):
        p = pos.clone()
        p[1, 3] = bad
        was = kp.clone()
        out, st = run(lens, p)
        assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[3] == 7.5).all()
        right(out, [0, 1, 2, 4])
        assert torch.equal(was.view(torch.int16), kp.view(torch.int16))
    for bad in (-1, c.num_pages, 2 ** 31 - 1):
        t = c.tables.clone()
        t[0, 2, 0] = bad                   # the sinks' page: its tokens are skipped
        out, st = run(lens, tables=t)
        assert st == pkv.PKV_ERR_OUT_OF_RANGE
        right(out, [2], sinks=0)
        right(out, [0, 1, 3, 4])
    t = c.tables.clone()
    t[0, 2] = -1
    out, st = run(lens, tables=t)
    assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[2] == 0).all()
    out, st = run(lens)
    assert st == pkv.PKV_OK and torch.equal(out, good)
    pool.close()


@pytest.mark.parametrize("batch", [90, 100, 400])
def test_bad_lengths_and_padding_inside_shares(batch):
    """Sequences that are skipped, padding rows and good ones packed into the
    same blocks; every good row right, every other left alone."""
    rng = np.random.RandomState(batch)
    lens = rng.randint(1, 400, batch)
    lens[rng.rand(batch) < 0.2] = 0
    bad = (rng.rand(batch) < 0.1) & (lens > 0)
    c = W.Cache(lens.tolist(), seed=batch)
    kp, vp = c.pools(lambda b: np.ones(lens[b], bool), float("nan"))
    pool = _pool(c)
    q = torch.randn(batch, 32, 64, generator=c.gen, device="cuda").bfloat16()
    given = torch.tensor(np.where(bad, 5000, lens), dtype=torch.int32, device="cuda")
    out = torch.full((batch, 32, 64), 7.5, device="cuda")
    pkv.pkv_window_attention(pool, 0, q, kp, vp, c.tables, given, out, 200, sinks=4)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    for b in range(batch):
        if bad[b] or lens[b] == 0:
            assert (out[b] == 7.5).all()
        else:
            ref, tol = W.attend(q[b:b + 1].double(), c.k[b].double(), c.v[b].double(),
                                torch.tensor([lens[b] - 1], device="cuda"), 200, 4)
            W.check(out[b:b + 1], ref, tol, f"sequence {b}")
    # the tickets are whole again: a clean call on the same handle is right
    given = c.lens_tensor()
    pkv.pkv_window_attention(pool, 0, q, kp, vp, c.tables, given, out, 200, sinks=4)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    for b in np.flatnonzero(lens):
        ref, tol = W.attend(q[b:b + 1].double(), c.k[b].double(), c.v[b].double(),
                            torch.tensor([lens[b] - 1], device="cuda"), 200, 4)
        W.check(out[b:b + 1], ref, tol, f"sequence {b} again")
    pool.close()


def test_few_splits_allowed():
    """max_splits of 1, 2 and 3 bound the ranges of a sequence."""
    for max_splits in (1, 2, 3):
        lens = [2048, 5, 1000, 700, 0, 2048] * 15
        c = W.Cache(lens, seed=max_splits)
        _decode(lens, 2048, 0, fused=True, seed=max_splits, pool=_pool(c, max_splits=max_splits))


def test_captured_and_replayed_with_changing_lengths():
    """One captured step over the layers of a programmatic-launch handle, replayed
    while lengths and pools change between replays; the same bits as eager calls."""
    L, B = 3, 4
    lens = [30, 700, 2000, 64]
    table = np.full((L, B, 128), -1, np.int32)
    ids = np.random.RandomState(0).permutation(L * B * 128).reshape(L, B, 128)
    table[:] = ids
    tables = torch.from_numpy(table).cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    kp = torch.randn(L * B * 128, 8, 16, 64, generator=g, device="cuda").bfloat16()
    vp = torch.randn(L * B * 128, 8, 16, 64, generator=g, device="cuda").bfloat16()
    q = torch.randn(L, B, 32, 64, generator=g, device="cuda").bfloat16()
    k = torch.randn(L, B, 8, 64, generator=g, device="cuda").bfloat16()
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    results = []
    for flags, captured in ((0, False), (pkv.PKV_FLAG_PDL, True)):
        pool = pkv.pkv_pool_create(L, L * B * 128, B, flags=flags)
        pk, pv = kp.clone(), vp.clone()
        n = lens_t.clone()
        out = torch.zeros(L, B, 32, 64, device="cuda")

        def step():
            for layer in range(L):
                pkv.pkv_window_append_attend(pool, layer, q[layer], k[layer], k[layer], pk, pv,
                                             tables, n, out[layer], 512, sinks=4)
        seen = []
        if captured:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        for i in range(4):
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            seen.append(out.clone())
            n += 1
            torch.cuda.synchronize()
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK
        results.append((torch.stack(seen), pk, pv))
        del step
        pool.close()
    assert torch.equal(results[0][0], results[1][0])
    assert torch.equal(results[0][1], results[1][1]) and torch.equal(results[0][2], results[1][2])


def test_full_window_agrees_with_the_full_attention():
    lens = [1, 33, 500, 2048]
    c = W.Cache(lens)
    kp, vp = c.pools(lambda b: np.ones(lens[b], bool), 0.0)
    pool = _pool(c)
    q = torch.randn(4, 32, 64, device="cuda").bfloat16()
    a, b = torch.zeros(4, 32, 64, device="cuda"), torch.zeros(4, 32, 64, device="cuda")
    pkv.pkv_decode_attention(pool, 0, q, kp, vp, c.tables, c.lens_tensor(), a)
    pkv.pkv_window_attention(pool, 0, q, kp, vp, c.tables, c.lens_tensor(), b, 2048)
    assert (a - b).abs().max().item() <= 5e-4
    pool.close()


def _relative(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


def test_outputs_are_those_of_fp32_arithmetic():
    """Relative 2-norm error below 3e-6. A score is off by some sqrt(64) 2^-24 of
    itself, weights by 2^-22, which leaves 3e-7; a value sum of the prefill takes
    4 steps x 12 products on the tensor cores, each of which drops half of
    2^-23 of the accumulator on average while it grows to its final size:
    48 x 2^-24 / 2 = 1.4e-6. Probabilities of two BF16 terms would be off by
    2^-16 / sqrt(12) = 4.4e-6."""
    n, window, sinks = 2048, 700, 4
    c = W.Cache([n, n])
    kp, vp = c.pools(lambda b: np.ones(n, bool), 0.0)
    pool = _pool(c)
    at = torch.arange(n - 300, n, device="cuda")
    q = torch.randn(600, 32, 64, generator=c.gen, device="cuda").bfloat16()
    ref = torch.cat([W.attend(q[300 * b:300 * b + 300].double(), c.k[b].double(),
                              c.v[b].double(), at, window, sinks)[0] for b in range(2)])
    out = torch.zeros(600, 32, 64, device="cuda")
    cu = torch.tensor([0, 300, 600], dtype=torch.int32, device="cuda")
    start = torch.tensor([n - 300] * 2, dtype=torch.int32, device="cuda")
    pkv.pkv_window_prefill_attention(pool, 0, q, kp, vp, c.tables, cu, start, out, 300, window,
                                     sinks=sinks)
    assert _relative(out, ref) < 3e-6
    last = q[[299, 599]].contiguous()
    one = torch.zeros(2, 32, 64, device="cuda")
    pkv.pkv_window_attention(pool, 0, last, kp, vp, c.tables, c.lens_tensor(), one, window,
                             sinks=sinks)
    assert _relative(one, ref[[299, 599]]) < 3e-6
    pool.close()


# Relative 2-norm errors of FP32-grade results, inputs N(0, 1). A score (64 products in
# FP32, the argument in base 2 up to 8, 2^x to 2^-22) leaves a weight some 2.7e-7 off,
# a rotated query (two products and a sum, each rounded) 5e-8 more, and sums in FP32
# over the pages of a warp less than that; weights and values average to the same
# relative error of the output. Limits are some three times that. What they hold: a
# rotated query without its third BF16 term is 2^-17 / sqrt(3) = 4.4e-6 off an element,
# 1e-5 in the output; sums kept in the tensor cores over 100,000 tokens 1.8e-6.
DECODE_LIMIT = 1e-6


@pytest.mark.parametrize("lens,window,sinks,max_seq_len", [
    ([2048, 1500, 700], 700, 4, 2048), ([900] * 64, 600, 4, 2048),
    ([120000, 100003], 2 ** 31 - 1, 0, 131072)])
@pytest.mark.parametrize("axes", [0, 1, 3])
@pytest.mark.parametrize("fused", [False, True])
def test_decode_is_fp32_arithmetic(lens, window, sinks, max_seq_len, axes, fused):
    c = W.Cache(lens, max_seq_len, seed=21)
    kp, vp = c.pools(lambda b: np.ones(lens[b], bool), 0.0)
    pool = _pool(c)
    B = len(lens)
    q = torch.randn(B, 32, 64, generator=c.gen, device="cuda").bfloat16()
    out = torch.zeros(B, 32, 64, device="cuda")
    rope, q64 = {}, q.double()
    new = [torch.stack([t[b][-1] for b in range(B)]) for t in (c.k, c.v)]
    if axes:
        cos, sin = W.angles(4000)
        pos = torch.randint(0, 4000, (axes, B), generator=c.gen, device="cuda").int()
        rope = dict(rope=pkv.pkv_axes_rope(cos, sin, SECTIONS[axes]), rope_positions=pos)
        q64 = W.rotate(q, cos, sin, pos, SECTIONS[axes], torch.float64)
        if fused:
            turned = W.rotate(new[0], cos, sin, pos, SECTIONS[axes], torch.float32).bfloat16()
            for b in range(B):
                c.k[b][-1] = turned[b]
    if fused:
        pkv.pkv_window_append_attend(pool, 0, q, *new, kp, vp, c.tables, c.lens_tensor(), out,
                                     window, sinks=sinks, **rope)
    else:
        pkv.pkv_window_attention(pool, 0, q, kp, vp, c.tables, c.lens_tensor(), out, window,
                                 sinks=sinks, **rope)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    pool.close()
    ref = torch.cat([W.attend(q64[b:b + 1], c.k[b].double(), c.v[b].double(),
                              torch.tensor([lens[b] - 1], device="cuda"), window, sinks)[0]
                     for b in range(B)])
    assert _relative(out, ref) < DECODE_LIMIT


def test_prefill_is_fp32_arithmetic_over_long_windows():
    """A 4,096-token window, where a tile's sums are longest. A tensor-core sum drops
    0.36 of 2^-23 of its accumulator on average at each product, towards zero, while
    the accumulator grows as the square root of the products done: over the 12 n
    products of n steps 2/3 x 12 n x 0.36 x 2^-23 of it, for n = 2 6.9e-7, with the
    2.7e-7 of the weights 7.4e-7 (measured: 6.4e-7); sums left in the tensor cores for
    four steps come to 1.4e-6 (measured: 1.1e-6)."""
    window, sinks, n, start_at = 4096, 16, 128, 8000
    lens = [start_at + n] * 2
    c = W.Cache(lens, 16384, seed=22)
    kp, vp = c.pools(lambda b: np.ones(lens[b], bool), 0.0)
    pool = _pool(c)
    q = torch.randn(2 * n, 32, 64, generator=c.gen, device="cuda").bfloat16()
    out = torch.zeros(2 * n, 32, 64, device="cuda")
    cu = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    start = torch.tensor([start_at] * 2, dtype=torch.int32, device="cuda")
    pkv.pkv_window_prefill_attention(pool, 0, q, kp, vp, c.tables, cu, start, out, n, window,
                                     sinks=sinks)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    pool.close()
    at = torch.arange(start_at, start_at + n, device="cuda")
    ref = torch.cat([W.attend(q[n * b:n * b + n].double(), c.k[b].double(), c.v[b].double(), at,
                              window, sinks)[0] for b in range(2)])
    assert _relative(out, ref) < 8.5e-7


# ---------------------------------------------------------------- prefill
def _prefill(chunks, starts, window, sinks, max_seq_len=2048, seed=11, junk="mixed", k_scale=1.0,
             max_chunk=None, **kw):
    lens = [s + n if n else 0 for s, n in zip(starts, chunks)]
    w = min(window, 1 << 40)
    c = W.Cache(lens, max_seq_len, seed, k_scale=k_scale,
                evict=lambda b: W.unseen_pages(lens[b], starts[b], w, sinks), **kw)

    def keep(b):
        t = np.arange(lens[b])
        return (t > starts[b] - w) | (t < sinks)
    kp, vp = c.pools(keep, junk)
    total = sum(chunks)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(chunks)]), dtype=torch.int32, device="cuda")
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    q = torch.randn(total, 32, 64, generator=c.gen, device="cuda").bfloat16()
    out = torch.full((total + 3, 32, 64), 7.5, device="cuda")
    pool = _pool(c)
    pkv.pkv_window_prefill_attention(pool, c.layer, q, kp, vp, c.tables, cu, start, out,
                                     max_chunk or max(chunks), window, sinks=sinks)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    pool.close()
    assert (out[total:] == 7.5).all()
    row = worst = 0
    for b, n in enumerate(chunks):
        if n:
            at = torch.arange(starts[b], lens[b], device="cuda")
            ref, tol = W.attend(q[row:row + n].double(), c.k[b].double(), c.v[b].double(), at, w,
                                sinks)
            worst = max(worst, W.check(out[row:row + n], ref, tol,
                                       f"chunk {n} at {starts[b]} window {window} sinks {sinks}"))
        row += n
    return worst


@pytest.mark.parametrize("window", [1, 2, 17, 64, 65, 200, 1024, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 16, 70, 2 ** 31 - 1])
def test_prefill_chunks(window, sinks):
    _prefill([1, 16, 63, 64, 65, 300, 0, 130], [0, 5, 1000, 0, 64, 0, 9, 700], window, sinks)


@pytest.mark.parametrize("window,sinks", [(128, 4), (500, 0), (2048, 0)])
def test_prefill_full_prompts(window, sinks):
    _prefill([2048, 1500], [0, 548], window, sinks)


@pytest.mark.parametrize("window,sinks", [(4096, 16), (300, 1000), (2 ** 31 - 1, 0)])
def test_prefill_long_context(window, sinks):
    _prefill([200, 129], [30000, 20011], window, sinks, max_seq_len=32768)


def test_prefill_large_scores():
    _prefill([300], [100], 128, 4, k_scale=30.0)


def test_prefill_launch_wider_than_the_chunks():
    _prefill([3, 70], [0, 0], 32, 4, max_chunk=2048, max_batch=4, num_layers=2, layer=1)


# groups of 32 sequences: on both sides of one, two and three, with whole groups
# empty, and equal, single and ragged numbers of tiles
@pytest.mark.parametrize("chunks", [
    [1] * 31, [40] * 32, [1] * 33, [0] * 70 + [100] + [0] * 29, [70] + [0] * 63 + [33],
    [(37 * i * i) % 140 for i in range(75)], [200] + [3] * 64 + [0, 0, 161],
    [32 * (i % 5) for i in range(100)]])
@pytest.mark.parametrize("max_chunk", [None, 2048])
def test_prefill_many_sequences(chunks, max_chunk):
    starts = [(53 * i) % 300 for i in range(len(chunks))]
    _prefill(chunks, starts, 60, 4, max_chunk=max_chunk, seed=len(chunks))


def test_prefill_without_tokens_in_its_sequences():
    """Rows that belong to no sequence stay as they were."""
    c = W.Cache([5, 5])
    kp, vp = c.pools(lambda b: np.ones(5, bool))
    pool = _pool(c)
    q = torch.randn(40, 32, 64, device="cuda").bfloat16()
    out = torch.full((40, 32, 64), 7.5, device="cuda")
    zeros = torch.zeros(3, dtype=torch.int32, device="cuda")
    for _ in range(2):
        pkv.pkv_window_prefill_attention(pool, 0, q, kp, vp, c.tables, zeros, zeros[:2], out, 2048, 8)
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK and (out == 7.5).all()
    pool.close()


@pytest.mark.parametrize("where", [0, 31, 32, 69])
def test_prefill_one_bad_sequence_among_many(where):
    """It is flagged and skipped; the others' results keep their bits."""
    chunks, starts = [50 + i % 20 for i in range(70)], [(11 * i) % 90 for i in range(70)]
    lens = [s + n for s, n in zip(starts, chunks)]
    c = W.Cache(lens)
    kp, vp = c.pools(lambda b: np.ones(lens[b], bool), 0.0)
    pool = _pool(c)
    cu = np.concatenate([[0], np.cumsum(chunks)])
    q = torch.randn(cu[-1], 32, 64, device="cuda", generator=c.gen).bfloat16()
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")

    def run(start_=start, cu_=cu_t):
        out = torch.full((cu[-1], 32, 64), 7.5, device="cuda")
        pkv.pkv_window_prefill_attention(pool, 0, q, kp, vp, c.tables, cu_, start_, out, 100, 64,
                                         sinks=4)
        return out, pkv.pkv_get_error(pool)

    good, st = run()
    assert st == pkv.PKV_OK
    mine = torch.zeros(cu[-1], dtype=torch.bool, device="cuda")
    mine[cu[where]:cu[where + 1]] = True
    for bad in (-1, 2040, 2 ** 31 - 1):
        s = start.clone()
        s[where] = bad
        out, st = run(start_=s)
        assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[mine] == 7.5).all()
        assert torch.equal(out[~mine], good[~mine])
    bad_cu = cu_t.clone()
    bad_cu[where + 1] = 2 ** 31 - 1              # this sequence and the next one have no rows
    skipped = mine.clone()
    if where < 69:
        skipped[cu[where + 1]:cu[where + 2]] = True
    out, st = run(cu_=bad_cu)
    assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[skipped] == 7.5).all()
    assert torch.equal(out[~skipped], good[~skipped])
    out, st = run()
    assert st == pkv.PKV_OK and torch.equal(out, good)
    pool.close()


@pytest.mark.parametrize("batch,bound", [(1, 131072), (16, 32768)])
def test_prefill_time_follows_the_chunks(batch, bound):
    """Chunks of 32 tokens take the same time under a launch bound far above them:
    what is drawn are the tiles there are, 8 a sequence. Were every tile below the
    bound drawn, each of 304 resident CTAs would draw 108 or 430 in vain one after the
    other, half a microsecond each at the least, on top of some 10."""
    c = W.Cache([32] * batch, max_seq_len=131072)
    kp, vp = c.pools(lambda b: np.ones(32, bool), 0.0)
    pool = _pool(c)
    n = 32 * batch
    q = torch.randn(n, 32, 64, device="cuda").bfloat16()
    out = torch.zeros(n, 32, 64, device="cuda")
    cu = torch.arange(0, n + 1, 32, dtype=torch.int32, device="cuda")
    start = torch.zeros(batch, dtype=torch.int32, device="cuda")
    times = {}
    for chunk in (32, bound):
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            for _ in range(20):
                pkv.pkv_window_prefill_attention(pool, 0, q, kp, vp, c.tables, cu, start, out, chunk,
                                                 64)
        ends = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        times[chunk] = []
        for _ in range(8):
            ends[0].record()
            graph.replay()
            ends[1].record()
            torch.cuda.synchronize()
            times[chunk].append(ends[0].elapsed_time(ends[1]))
        del graph
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert min(times[bound]) < 3 * min(times[32]), times
    pool.close()


def test_prefill_pages_past_four_gib():
    _prefill([100], [30], 64, 4, junk=float("nan"), base_page=280000)


@pytest.mark.parametrize("start,at", [(0, 0), (5, 40), (100, 131), (13, 111)])
def test_prefill_rows_that_do_not_see_a_bad_token(start, at):
    """A NaN key concerns the rows that see it, a NaN value the 32-token tiles that do."""
    n, window = 150, 9
    c = W.Cache([start + n])
    q = torch.randn(n, 32, 64, device="cuda", generator=c.gen).bfloat16()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    first = torch.tensor([start], dtype=torch.int32, device="cuda")
    pos = torch.arange(start, start + n, device="cuda")
    pool = _pool(c)
    page, slot = int(c.table[0, 0, at // 16]), at % 16
    seen = W.visible(pos, torch.tensor(at, device="cuda"), window, 0)
    for which in (0, 1):
        pools = c.pools(lambda b: np.ones(start + n, bool))
        pools[which][page, :, slot] = float("nan")
        out = torch.empty(n, 32, 64, device="cuda")
        pkv.pkv_window_prefill_attention(pool, 0, q, *pools, c.tables, cu, first, out, n, window)
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK
        hit = seen
        if which == 1:
            tiles = torch.arange(n, device="cuda") // 32
            hit = torch.isin(tiles, tiles[seen])
        assert bool(seen.any()) and not bool(hit.all())
        assert torch.isnan(out[seen]).all()
        ref, tol = W.attend(q[~hit].double(), c.k[0].double(), c.v[0].double(), pos[~hit], window,
                            0)
        W.check(out[~hit], ref, tol, f"start {start}, token {at}, pool {which}")


def test_prefill_flags_bad_data():
    chunks, starts = [100, 100, 100], [0, 50, 0]
    lens = [100, 150, 100]
    c = W.Cache(lens)
    kp, vp = c.pools(lambda b: np.ones(lens[b], bool), 0.0)
    pool = _pool(c)
    q = torch.randn(300, 32, 64, device="cuda").bfloat16()
    cu = torch.tensor([0, 100, 200, 300], dtype=torch.int32, device="cuda")
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")

    def run(cu_=cu, start_=start, tables=c.tables, max_chunk=100, window=64, sinks=4):
        out = torch.full((300, 32, 64), 7.5, device="cuda")
        pkv.pkv_window_prefill_attention(pool, 0, q, kp, vp, tables, cu_, start_, out, max_chunk,
                                         window, sinks=sinks)
        return out, pkv.pkv_get_error(pool)

    good, st = run()
    assert st == pkv.PKV_OK
    s = start.clone()
    for bad in (-1, 1949, 2 ** 31 - 1):
        s[1] = bad
        out, st = run(start_=s)
        assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[100:200] == 7.5).all()
        assert torch.equal(out[:100], good[:100]) and torch.equal(out[200:], good[200:])
    bad_cu = torch.tensor([0, 100, 99, 300], dtype=torch.int32, device="cuda")
    assert run(cu_=bad_cu, max_chunk=2048)[1] == pkv.PKV_ERR_OUT_OF_RANGE
    bad_cu = torch.tensor([0, 100, 200, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out, st = run(cu_=bad_cu)
    assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[200:] == 7.5).all()
    assert run(max_chunk=64)[1] == pkv.PKV_ERR_OUT_OF_RANGE      # a chunk longer than announced
    # tokens of an invalid page are skipped: the sinks of sequence 1
    for bad in (-1, c.num_pages):
        t = c.tables.clone()
        t[0, 1, 0] = bad
        out, st = run(tables=t, window=8)
        assert st == pkv.PKV_ERR_OUT_OF_RANGE
        ref, tol = W.attend(q[100:200].double(), c.k[1].double(), c.v[1].double(),
                            torch.arange(50, 150, device="cuda"), 8, 0)
        W.check(out[100:200], ref, tol, "without the sinks")
    t = c.tables.clone()
    t[0, 1] = -1
    out, st = run(tables=t)
    assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[100:200] == 0).all()
    out, st = run()
    assert st == pkv.PKV_OK and torch.equal(out, good)
    pool.close()


def test_refusals():
    c = W.Cache([40], max_seq_len=4096)
    kp, vp = c.pools(lambda b: np.ones(40, bool), 0.0)
    pool = _pool(c)
    q = torch.zeros(1, 32, 64, device="cuda").bfloat16()
    k = torch.zeros(1, 8, 64, device="cuda").bfloat16()
    out = torch.zeros(1, 32, 64, device="cuda")
    lens = c.lens_tensor()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")

    def status(f):
        with pytest.raises(pkv.PkvError) as e:
            f()
        return e.value.status

    # the calls limited to 2,048 tokens refuse a longer handle
    long_calls = [
        lambda: pkv.pkv_decode_attention(pool, 0, q, kp, vp, c.tables, lens, out),
        lambda: pkv.pkv_append_attend(pool, 0, q, k, k, kp, vp, c.tables, lens, out),
        lambda: pkv.pkv_append_attend_layers(pool, 0, q[None], k[None], k[None], kp, vp, c.tables,
                                             lens, out[None]),
        lambda: pkv.pkv_prefill_attention(pool, 0, q, kp, vp, c.tables, cu, zero, out, 1)]
    for f in long_calls:
        assert status(f) == pkv.PKV_ERR_UNSUPPORTED
    cos, sin = W.angles(50)
    rope = pkv.pkv_axes_rope(cos, sin, SECTIONS[2])
    pos = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    big = 2 ** 32      # wraps to small C ints: 2^32 + 5 must not become 5

    def call(window=8, sinks=0, layer=0, num_splits=0, batch=None, **kw):
        pkv.pkv_window_append_attend(pool, layer, q, k, k, kp, vp, c.tables, lens, out, window,
                                     sinks=sinks, num_splits=num_splits, batch=batch, **kw)
    call(rope=rope, rope_positions=pos)
    call(batch=0)
    whole, wide = torch.zeros_like(out), torch.zeros_like(out)
    for o, w in ((whole, 4096), (wide, big + 3)):
        pkv.pkv_window_attention(pool, 0, q, kp, vp, c.tables, lens, o, w)
    assert torch.equal(whole, wide)
    for kw in (dict(window=0), dict(window=-3), dict(sinks=-1), dict(layer=1), dict(layer=-1),
               dict(num_splits=-1), dict(num_splits=65), dict(batch=-1), dict(layer=big),
               dict(window=5 - big), dict(sinks=3 - big), dict(num_splits=big + 1),
               dict(batch=1 - big)):
        assert status(lambda: call(**kw)) == pkv.PKV_ERR_INVALID_ARG
    for kw in (dict(rope=rope), dict(rope_positions=pos), dict(batch=2),
               dict(rope=rope, rope_positions=pos[:1]),
               dict(rope=rope, rope_positions=pos.cpu()),
               dict(rope=rope, rope_positions=pos.long())):
        with pytest.raises(ValueError):
            call(**kw)
    for name in ("q", "kp", "tables", "out"):
        a = dict(q=q, kp=kp, tables=c.tables, out=out)
        a[name] = a[name].cpu()
        with pytest.raises(ValueError):
            pkv.pkv_window_attention(pool, 0, a["q"], a["kp"], vp, a["tables"], lens, a["out"], 8)
    for kw in (dict(window=0), dict(sinks=-1), dict(max_chunk_tokens=0),
               dict(max_chunk_tokens=4097)):
        args = dict(max_chunk_tokens=1, window=8, sinks=0)
        args.update(kw)
        assert status(lambda: pkv.pkv_window_prefill_attention(
            pool, 0, q, kp, vp, c.tables, cu, zero, out, args["max_chunk_tokens"], args["window"],
            sinks=args["sinks"])) == pkv.PKV_ERR_INVALID_ARG
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    pool.close()
