"""Attention of drafted trees and the commit of accepted paths on the GPU, against a
64-bit restatement and plain moves."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
from tree_helpers import attend, depth, pack, random_tree, seen_matrix
from window_helpers import DIM, HKV, HQ, PAGE, Cache, angles, check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _library():
    from paged_kv_cache_210_gb300 import build as lib_build
    lib_build.build()


def handle(c, flags=0):
    if c.max_seq_len > 2048:
        flags |= pkv.PKV_FLAG_LONG_CONTEXT
    return pkv.pkv_pool_create(c.num_layers, c.num_pages, c.max_batch, max_seq_len=c.max_seq_len,
                               flags=flags)


def int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def normal(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16().cuda()


def run_tree(starts, nodes, window=2048, sinks=0, masks=None, seed=0, max_seq_len=2048, junk="mixed",
             k_scale=1.0, q_scale=1.0, num_layers=1, layer=0, spare=4, after=3):
    """One call over sequences of starts[b] committed and nodes[b] drafted tokens; every
    token that nobody may see is junk, pages without a token that somebody sees are
    missing. Returns the outputs."""
    rng = np.random.RandomState(seed)
    masks = masks or [random_tree(rng, n) for n in nodes]
    seen = [seen_matrix(s, m, window, sinks) for s, m in zip(starts, masks)]

    def needed(b):                         # tokens that a row sees, and every drafted one
        if len(masks[b]) == 0:
            return np.zeros(starts[b], bool)
        keep = seen[b].any(0)
        keep[starts[b]:] = True
        return keep

    def evict(b):
        keep = needed(b)
        whole = np.zeros(-(-max(len(keep), 1) // PAGE) * PAGE, bool)
        whole[:len(keep)] = keep
        return ~whole.reshape(-1, PAGE).any(1)

    c = Cache([s + n for s, n in zip(starts, nodes)], max_seq_len=max_seq_len, seed=seed, evict=evict,
              k_scale=k_scale, num_layers=num_layers, layer=layer, spare=spare)
    k_pool, v_pool = c.pools(needed, junk)
    total = sum(nodes)
    q = normal(seed + 5, total + after, HQ, DIM, scale=q_scale)
    out = torch.full((total + after, HQ, DIM), 3.0, device="cuda")
    cu = int32(np.cumsum([0] + list(nodes)))
    pool = handle(c)
    tree = pack([m for ms in masks for m in ms] + [0] * after)
    for _ in range(2):                     # twice: counters and parts are left as they were found
        pkv.pkv_tree_attention(pool, layer, q, k_pool, v_pool, c.tables, cu, int32(starts), tree, out,
                               window, sinks=sinks)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert bool((out[total:] == 3.0).all())
    row = 0
    for b, n in enumerate(nodes):
        if n:
            ref, tol = attend(q[row:row + n].double(), c.k[b].double(), c.v[b].double(), seen[b])
            check(out[row:row + n], ref, tol, f"sequence {b}: {starts[b]} + {n}")
        row += n
    return out


@pytest.mark.parametrize("start", [0, 1, 15, 16, 17, 63, 64, 100, 1000, 1984])
@pytest.mark.parametrize("nodes", [1, 2, 8, 9, 32, 33, 64])
def test_sizes(start, nodes):
    run_tree([start], [nodes], seed=start + nodes)


@pytest.mark.parametrize("starts,nodes", [
    ([0, 500, 3], [5, 1, 64]), ([1500] * 5, [16] * 5), ([10, 0, 0, 900, 31, 2], [0, 3, 0, 40, 33, 7]),
    ([100 * i for i in range(20)], [(7 * i) % 30 + 1 for i in range(20)])])
def test_ragged_batches(starts, nodes):
    run_tree(starts, nodes, seed=len(starts))


@pytest.mark.parametrize("starts,nodes", [
    # few drafted tokens a sequence on average: one large tree among them, long contexts,
    # batches of more than 32 sequences
    ([700, 3, 0, 50] + [90] * 20, [64, 0, 5, 1] + [1] * 20), ([300 + i for i in range(45)], [3] * 45),
    ([2000, 1, 16], [4, 4, 4]), ([0] * 70, [i % 3 for i in range(70)])])
@pytest.mark.parametrize("window,sinks", [(2048, 0), (50, 5)])
def test_few_rows(starts, nodes, window, sinks):
    run_tree(starts, nodes, window=window, sinks=sinks, seed=len(starts))


@pytest.mark.parametrize("most", [1, 12])
def test_batches_past_1024_sequences(most):
    rng = np.random.RandomState(most)
    starts = [int(x) for x in rng.randint(0, 40, 1300)]
    starts[1290], starts[1100], starts[40] = 900, 0, 500
    nodes = [int(x) for x in rng.randint(0, most + 1, 1300)]
    nodes[1290] = nodes[1] = 20
    run_tree(starts, nodes, max_seq_len=1024, seed=most)


def test_few_rows_over_long_contexts():
    run_tree([60000, 33333], [4, 3], max_seq_len=65536)
    run_tree([60000, 33333], [4, 3], max_seq_len=65536, window=3000, sinks=20)


@pytest.mark.parametrize("starts,nodes,max_seq_len", [
    # parts of a tile in clusters of 16, 8 and 4; sequences without tokens, tiles that are
    # not there, more parts than steps
    ([1999], [8], 2048), ([0], [16], 2048), ([700], [41], 2048), ([1000, 3], [25, 3], 2048),
    ([1900, 0, 40, 7, 333], [1, 8, 9, 2, 5], 2048),
    ([50 * i for i in range(32)], [[0, 0, 5, 0, 1, 0, 0, 2][i % 8] // (1 + i // 8) for i in range(32)],
     2048),
    ([200 * i for i in range(8)], [3, 1, 9, 0, 1, 4, 3, 5], 2048), ([90, 2], [9, 7], 2048),
    ([0, 64, 1990], [0, 12, 0], 2048), ([8000], [5], 8192), ([4000, 100], [20, 7], 4096)])
@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (37, 4)])
def test_clusters(starts, nodes, max_seq_len, window, sinks):
    run_tree(starts, nodes, window=window, sinks=sinks, max_seq_len=max_seq_len, seed=sum(nodes))


@pytest.mark.parametrize("start", [0, 1, 15, 17, 63, 64, 1000, 8100])
@pytest.mark.parametrize("nodes", [17, 32, 33, 64])
def test_large_trees_of_one_sequence(start, nodes):
    # too long a context for clusters
    run_tree([start], [nodes], max_seq_len=8192, window=1 << 20, seed=start + nodes)
    run_tree([start], [nodes], max_seq_len=16384, window=5000, sinks=3, seed=start)


@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (90, 6)])
@pytest.mark.parametrize("max_seq_len", [2048, 4096])
def test_trees_of_eight_on_average(max_seq_len, window, sinks):
    starts = [121 * i for i in range(16)]
    run_tree(starts, [1 + i % 15 for i in range(16)], max_seq_len=max_seq_len, window=window,
             sinks=sinks, seed=sinks)


@pytest.mark.parametrize("start", [0, 5, 380])
def test_any_mask_of_a_long_context(start):
    n = 50
    rng = np.random.RandomState(start)
    every = (1 << 64) - 1
    masks = [0, every, 1 << 49, 2, every << 50 & every, 1] + \
        [int(rng.randint(0, 1 << 32)) << 32 | int(rng.randint(0, 1 << 32)) for _ in range(n - 6)]
    run_tree([start], [n], masks=[masks], max_seq_len=8192, window=45 if start > 5 else 1 << 20)


def test_a_window_makes_clusters_of_a_long_context():
    run_tree([60000], [8], max_seq_len=65536, window=3000, sinks=20)


@pytest.mark.parametrize("batch", [39, 65, 150])
def test_many_sequences(batch):
    rng = np.random.RandomState(batch)
    starts = [int(x) for x in rng.randint(0, 700, batch)]
    starts[batch // 2] = 1900                       # one that is worth splitting
    nodes = [int(x) for x in rng.randint(0, 40, batch)]
    nodes[batch // 2] = 50
    run_tree(starts, nodes, seed=batch)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 0), (17, 4), (64, 70), (100, 0),
                                          (512, 4), (300, 2000)])
@pytest.mark.parametrize("starts,nodes", [([200, 3, 1000], [20, 64, 33]), ([1980], [64])])
def test_windows(starts, nodes, window, sinks):
    run_tree(starts, nodes, window=window, sinks=sinks, seed=window)


@pytest.mark.parametrize("start", [0, 5, 80])
def test_any_mask(start):
    # nothing, itself alone, later tokens, everything, bits past the last token
    n = 40
    rng = np.random.RandomState(start)
    every = (1 << 64) - 1
    masks = [0, every, 1 << 39, 2, every << 40 & every, 1] + \
        [int(rng.randint(0, 1 << 32)) << 32 | int(rng.randint(0, 1 << 32)) for _ in range(n - 6)]
    run_tree([start], [n], masks=[masks])
    # windows go by the number of drafted tokens seen
    run_tree([start + 300], [n], masks=[masks], window=45, sinks=2)


def test_rows_that_see_nothing_are_zero():
    out = run_tree([0, 50], [3, 2], masks=[[0, 2, 0], [0, 0]], window=1, sinks=0)
    assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())
    # p = start - 1 with window 1: the last committed token alone
    assert not bool((out[3] == 0).all())


@pytest.mark.parametrize("k_scale,q_scale", [(6.0, 3.0), (1e-3, 1e-2)])
def test_scales(k_scale, q_scale):
    run_tree([700, 40], [30, 64], k_scale=k_scale, q_scale=q_scale)


def test_another_layer():
    run_tree([90, 300], [12, 40], num_layers=3, layer=2)


@pytest.mark.parametrize("window,sinks", [(65536, 0), (4096, 10)])
def test_long_contexts(window, sinks):
    run_tree([60000, 17, 30001], [64, 20, 5], window=window, sinks=sinks, max_seq_len=65536)


def test_outputs_are_fp32_grade():
    # relative 2-norm against 64 bits: three BF16 terms and FP32 sums, not two terms
    # (2^-17 each)
    rng = np.random.RandomState(0)
    starts, nodes = [3000, 4000], [64, 40]
    masks = [random_tree(rng, n) for n in nodes]
    c = Cache([s + n for s, n in zip(starts, nodes)], max_seq_len=8192, seed=3)
    k_pool, v_pool = c.pools(lambda b: np.ones(starts[b] + nodes[b], bool))
    q = normal(1, sum(nodes), HQ, DIM)
    out = torch.empty(sum(nodes), HQ, DIM, device="cuda")
    pkv.pkv_tree_attention(handle(c), 0, q, k_pool, v_pool, c.tables, int32([0, 64, 104]),
                           int32(starts), pack(sum(masks, [])), out, 8192)
    off = norm = 0.0
    for b, rows in enumerate((slice(0, 64), slice(64, 104))):
        ref, _ = attend(q[rows].double(), c.k[b].double(), c.v[b].double(),
                        seen_matrix(starts[b], masks[b], 8192, 0))
        off += float((out[rows].double() - ref).square().sum())
        norm += float(ref.square().sum())
    assert math.sqrt(off / norm) < 1.5e-6


def test_a_chain_is_prefill():
    # a chain of drafted tokens is a chunk of a prompt
    c = Cache([1000 + 50, 64], seed=4)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    q = normal(1, 100, HQ, DIM)
    cu, start = int32([0, 50, 100]), int32([1000, 14])
    pool = handle(c)
    a, b = torch.empty(100, HQ, DIM, device="cuda"), torch.empty(100, HQ, DIM, device="cuda")
    chain = pack([(1 << i + 1) - 1 for i in range(50)] * 2)
    for window, sinks in ((2048, 0), (100, 4)):
        pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, chain, a, window,
                               sinks=sinks)
        if window == 2048:
            pkv.pkv_prefill_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, b, 50)
            assert float((a - b).abs().max()) < 2e-5        # that one's P has 16 bits
        # behind a window drafted tokens stay visible whatever their distance: 50 < 100
        pkv.pkv_window_prefill_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, b, 50,
                                         window, sinks=sinks)
        assert float((a - b).abs().max()) < 5e-6
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK


def test_invalid_pages_are_left_out():
    c = Cache([400 + 20], seed=5)
    c.table[0, 0, 3], c.table[0, 0, 25] = c.num_pages + 9, -1      # committed and drafted tokens
    tables = torch.from_numpy(c.table).cuda()
    tables_all = c.tables
    k_pool, v_pool = c.pools(lambda b: np.ones(420, bool))
    del tables_all
    rng = np.random.RandomState(5)
    masks = random_tree(rng, 20)
    q = normal(1, 20, HQ, DIM)
    out = torch.empty(20, HQ, DIM, device="cuda")
    pool = handle(c)
    pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, tables, int32([0, 20]), int32([400]),
                           pack(masks), out, 2048)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    seen = seen_matrix(400, masks, 2048, 0)
    seen[:, 48:64] = False
    seen[:, 400:416] = False
    ref, tol = attend(q.double(), c.k[0].double(), c.v[0].double(), seen)
    check(out, ref, tol)


@pytest.mark.parametrize("cu,start,nodes", [
    ([0, 5, 4], [10, 10], 5), ([0, 65, 70], [10, 10], 70), ([0, 4, 8], [-1, 10], 8),
    ([0, 4, 8], [2045, 10], 8), ([0, 4, 12], [10, 10], 8), ([-2, 4, 8], [10, 10], 8)])
def test_bad_sequences_are_flagged_and_left_alone(cu, start, nodes):
    c = Cache([2048, 300], seed=6)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    q = normal(1, nodes, HQ, DIM)
    out = torch.full((nodes, HQ, DIM), 3.0, device="cuda")
    pool = handle(c)
    chain = pack([(1 << min(i, 62) + 1) - 1 for i in range(nodes)])
    pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, int32(cu), int32(start), chain, out,
                           2048)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    good = [b for b in range(2) if 0 <= cu[b] <= cu[b + 1] <= nodes and cu[b + 1] - cu[b] <= 64
            and start[b] >= 0 and start[b] + cu[b + 1] - cu[b] <= 2048]
    rows = np.zeros(nodes, bool)
    masks = [(1 << min(i, 62) + 1) - 1 for i in range(nodes)]
    for b in good:
        n = cu[b + 1] - cu[b]
        rows[cu[b]:cu[b + 1]] = True
        mine = [m & ((1 << n) - 1) for m in masks[cu[b]:cu[b + 1]]]
        ref, tol = attend(q[cu[b]:cu[b + 1]].double(), c.k[b][:start[b] + n].double(),
                          c.v[b][:start[b] + n].double(), seen_matrix(start[b], mine, 2048, 0))
        check(out[cu[b]:cu[b + 1]], ref, tol)
    assert bool((out[torch.from_numpy(~rows).cuda()] == 3.0).all())


def test_captured_with_changing_lengths():
    c = Cache([1900, 700, 64], seed=7)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    q = normal(1, 60, HQ, DIM)
    out = torch.zeros(60, HQ, DIM, device="cuda")
    pool = handle(c)
    rng = np.random.RandomState(7)
    cu, start = int32([0, 20, 40, 60]), int32([0, 0, 0])
    tree = torch.zeros(60, dtype=torch.int64, device="cuda")

    def call():
        pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, tree, out, 2048)

    call()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            call()
    for starts, nodes in (([1880, 680, 44], [20, 20, 20]), ([0, 3, 40], [7, 33, 20]),
                          ([1800, 1, 0], [58, 0, 2]), ([5, 600, 9], [1, 1, 1])):
        masks = [random_tree(rng, n) for n in nodes]
        cu.copy_(int32(np.cumsum([0] + nodes)))
        start.copy_(int32(starts))
        flat = pack(sum(masks, []))
        tree[:flat.numel()].copy_(flat)
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        row = 0
        for b, n in enumerate(nodes):
            if n:
                ref, tol = attend(q[row:row + n].double(), c.k[b][:starts[b] + n].double(),
                                  c.v[b][:starts[b] + n].double(),
                                  seen_matrix(starts[b], masks[b], 2048, 0))
                check(out[row:row + n], ref, tol)
            row += n
        assert bool((out[row:] == 3.0).all())
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK


def test_captured_clusters_with_changing_lengths():
    c = Cache([1900, 700, 64], seed=17)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    total = 24
    q = normal(2, total, HQ, DIM)
    out = torch.zeros(total, HQ, DIM, device="cuda")
    pool = handle(c)
    rng = np.random.RandomState(17)
    cu, start = int32([0, 8, 16, 24]), int32([0, 0, 0])
    tree = torch.zeros(total, dtype=torch.int64, device="cuda")

    def call():
        pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, tree, out, 2048)

    call()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            call()
    for starts, nodes in (([1880, 680, 44], [8, 8, 8]), ([0, 3, 40], [1, 23, 0]),
                          ([1800, 1, 0], [0, 0, 2]), ([5, 600, 9], [0, 0, 0]),
                          ([1892, 0, 0], [6, 9, 9])):
        masks = [random_tree(rng, n) for n in nodes]
        cu.copy_(int32(np.cumsum([0] + nodes)))
        start.copy_(int32(starts))
        flat = pack(sum(masks, []) + [0] * (total - sum(nodes)))
        tree.copy_(flat)
        out.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        row = 0
        for b, n in enumerate(nodes):
            if n:
                ref, tol = attend(q[row:row + n].double(), c.k[b][:starts[b] + n].double(),
                                  c.v[b][:starts[b] + n].double(),
                                  seen_matrix(starts[b], masks[b], 2048, 0))
                check(out[row:row + n], ref, tol)
            row += n
        assert bool((out[row:] == 3.0).all())
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK


def test_between_windowed_prefills():
    # both draw their tiles from the handle's counter
    c = Cache([600, 400], seed=8)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    q = normal(1, 128, HQ, DIM)
    cu, start = int32([0, 64, 128]), int32([536, 336])
    pool = handle(c)
    chain = pack([(1 << i + 1) - 1 for i in range(64)] * 2)
    outs = [torch.empty(128, HQ, DIM, device="cuda") for _ in range(4)]
    for i in (0, 2):
        pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, chain, outs[i], 2048)
        pkv.pkv_window_prefill_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, outs[i + 1],
                                         64, 2048)
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    assert float((outs[0] - outs[1]).abs().max()) < 5e-6
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK


# ---------------------------------------------------------------- commit
def plain_commit(table, pools, starts, accepted, counts):
    out = [p.clone() for p in pools]
    for layer in range(table.shape[0]):
        for b, s in enumerate(starts):
            for k in range(counts[b]):
                t, d = s + int(accepted[b][k]), s + k
                for src, dst in zip(pools, out):
                    dst[table[layer, b, d // PAGE], :, d % PAGE] = \
                        src[table[layer, b, t // PAGE], :, t % PAGE]
    return out


def commit_case(starts, most, layers=2, seed=0, max_seq_len=2048, count=None):
    rng = np.random.RandomState(seed)
    batch, stride = len(starts), max_seq_len // PAGE
    table = np.full((layers, batch, stride), -1, np.int32)
    used = [(b, p) for b, s in enumerate(starts)
            for p in range(s // PAGE, min((s + 63) // PAGE, stride - 1) + 1)]
    ids = iter(rng.permutation(layers * len(used) + 2))
    for layer in range(layers):
        for b, p in used:
            table[layer, b, p] = next(ids)
    pages = layers * len(used) + 2
    pools = [torch.randint(-2 ** 15, 2 ** 15, (pages, HKV, PAGE, DIM), dtype=torch.int16,
                           generator=torch.Generator().manual_seed(seed + i)).cuda() for i in range(2)]
    room = [min(64, max_seq_len - s) for s in starts]
    accepted = np.array([rng.randint(0, room[b], most) for b in range(batch)], np.int32)
    counts = rng.randint(0, most + 1, batch) if count is None else np.full(batch, count)
    counts = [min(int(x), room[b]) for b, x in enumerate(counts)]
    pool = pkv.pkv_pool_create(layers, pages, batch, max_seq_len=max_seq_len,
                               flags=pkv.PKV_FLAG_LONG_CONTEXT if max_seq_len > 2048 else 0)
    return pool, table, pools, accepted, counts


def commit(pool, table, pools, starts, accepted, counts):
    bf = [p.view(torch.bfloat16) for p in pools]
    pkv.pkv_tree_commit(pool, bf[0], bf[1], torch.from_numpy(table).cuda(), int32(starts),
                        torch.from_numpy(np.ascontiguousarray(accepted)).cuda(), int32(counts))


@pytest.mark.parametrize("most", [1, 4, 7, 8, 9, 16, 17, 33, 64])
@pytest.mark.parametrize("starts", [[0], [15, 16, 1], [2047, 1985, 0, 77, 300]])
def test_commit(starts, most):
    # any order, tokens named twice, sources that are destinations of others
    pool, table, pools, accepted, counts = commit_case(starts, most, seed=most)
    want = plain_commit(table, pools, starts, accepted, counts)
    commit(pool, table, pools, starts, accepted, counts)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    for got, ref in zip(pools, want):
        assert torch.equal(got, ref)


def test_commit_of_a_large_batch_and_many_layers():
    starts = [(37 * i) % 1900 for i in range(60)]
    pool, table, pools, accepted, counts = commit_case(starts, 5, layers=16, seed=1)
    want = plain_commit(table, pools, starts, accepted, counts)
    commit(pool, table, pools, starts, accepted, counts)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    for got, ref in zip(pools, want):
        assert torch.equal(got, ref)


def test_commit_skips_and_flags_bad_data():
    starts = [10, 20, 30, 40, -1, 2040, 50]
    pool, table, pools, accepted, counts = commit_case([10, 20, 30, 40, 0, 1980, 50], 6, seed=2, count=6)
    accepted[0][3], accepted[1][2] = 64, -1             # no such drafted tokens
    counts[2], counts[3] = 7, -1                        # more than the list, fewer than none
    table[0, 6, 50 // PAGE] = -1                        # missing in layer 0 alone
    table[:, 5, 126:] = 0
    accepted[5][:] = [0, 1, 2, 3, 4, 20]                # past max_seq_len
    accepted[6][:] = [0, 5, 4, 3, 2, 1]
    want = [p.clone() for p in pools]
    one = plain_commit(table[1:], pools, [0] * 6 + [50], accepted, [0] * 6 + [6])
    for i in range(2):
        want[i] = one[i]
    commit(pool, table, pools, starts, accepted, counts)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    for got, ref in zip(pools, want):
        assert torch.equal(got, ref)


# ---------------------------------------------------------------- together
def test_draft_verify_commit_draft_again():
    # two rounds of drafting: fill the tree's slots, attend, commit a path, and check the
    # second round (and a decode step) against the sequence as it should be
    layers, batch = 2, 2
    lens = [40, 7]
    c = Cache([300] * batch, seed=9, num_layers=layers)
    rng = np.random.RandomState(9)
    ids = rng.permutation(c.num_pages + 60)[:layers * batch * 19].reshape(layers, batch, 19)
    c.table[:, :, :19] = ids
    tables = torch.from_numpy(c.table).cuda()
    pages = c.num_pages + 60
    pool = pkv.pkv_pool_create(layers, pages, batch, flags=pkv.PKV_FLAG_PDL)
    pools = [torch.zeros(pages, HKV, PAGE, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cos, sin = angles(2048)
    rope = pkv.pkv_axes_rope(cos, sin, [0] * 32)
    from window_helpers import rotate

    kept = [[[], []] for _ in range(layers)]            # per layer: per sequence (k, v) rows
    for layer in range(layers):
        for b in range(batch):
            kept[layer][b] = (normal(50 + 10 * layer + b, lens[b], HKV, DIM),
                              normal(70 + 10 * layer + b, lens[b], HKV, DIM))
        k = torch.cat([kept[layer][b][0] for b in range(batch)])
        v = torch.cat([kept[layer][b][1] for b in range(batch)])
        pkv.pkv_prefill_fill(pool, layer, k, v, *pools, tables, int32([0, lens[0], sum(lens)]),
                             int32([0, 0]), max(lens))
    for turn in range(2):
        nodes = [12, 30] if turn == 0 else [33, 5]
        masks = [random_tree(rng, n) for n in nodes]
        total = sum(nodes)
        cu, start = int32(np.cumsum([0] + nodes)), int32(lens)
        place = [lens[b] + depth(m, nodes[b]) for b in range(batch) for m in masks[b]]
        pos = int32(place)[None].contiguous()
        tree = pack(sum(masks, []))
        fresh = []
        for layer in range(layers):
            seed = 1000 * turn + 100 * layer
            q, k, v = (normal(seed + i, total, h, DIM) for i, h in enumerate((HQ, HKV, HKV)))
            q_rot, out = torch.empty_like(q), torch.empty(total, HQ, DIM, device="cuda")
            pkv.pkv_prefill_fill_axes(pool, layer, q, k, v, q_rot, *pools, tables, cu, start, rope, pos,
                                      max(nodes))
            pkv.pkv_tree_attention(pool, layer, q_rot, *pools, tables, cu, start, tree, out, 2048)
            k_rot = rotate(k, cos, sin, pos, [0] * 32, torch.float32).bfloat16()
            fresh.append((k_rot, v))
            for b in range(batch):
                rows = slice(int(cu[b]), int(cu[b + 1]))
                ks = torch.cat([kept[layer][b][0], k_rot[rows]]).double()
                vs = torch.cat([kept[layer][b][1], v[rows]]).double()
                ref, tol = attend(q_rot[rows].double(), ks, vs,
                                  seen_matrix(lens[b], masks[b], 2048, 0))
                check(out[rows], ref, tol, f"turn {turn} layer {layer} sequence {b}")
        # the path of the deepest token is accepted
        paths = []
        for b in range(batch):
            deepest = max(masks[b], key=lambda m: depth(m, nodes[b]))
            paths.append([j for j in range(nodes[b]) if deepest >> j & 1])
        most = max(len(p) for p in paths)
        accepted = int32([p + [0] * (most - len(p)) for p in paths])
        pkv.pkv_tree_commit(pool, *pools, tables, start, accepted, int32([len(p) for p in paths]))
        for layer in range(layers):
            for b in range(batch):
                rows = [int(cu[b]) + j for j in paths[b]]
                kept[layer][b] = tuple(torch.cat([old, new[rows]])
                                       for old, new in zip(kept[layer][b], fresh[layer]))
        lens = [lens[b] + len(paths[b]) for b in range(batch)]
    # a decode step right after the commit, on the same (programmatic) handle
    q = normal(7, batch, HQ, DIM)
    out = torch.empty(batch, HQ, DIM, device="cuda")
    pkv.pkv_window_attention(pool, 1, q, *pools, tables, int32(lens), out, 2048)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    for b in range(batch):
        ks, vs = (x.double() for x in kept[1][b])
        ref, tol = attend(q[b:b + 1].double(), ks, vs, np.ones((1, lens[b]), bool))
        check(out[b:b + 1], ref, tol)


def test_refusals():
    c = Cache([100, 100], seed=10)
    k_pool, v_pool = c.pools(lambda b: np.ones(100, bool))
    q, out = normal(1, 4, HQ, DIM), torch.empty(4, HQ, DIM, device="cuda")
    cu, start, tree = int32([0, 2, 4]), int32([90, 90]), pack([1, 3, 1, 3])
    pool = handle(c)

    def call(layer=0, q=q, tree=tree, window=9, **kw):
        pkv.pkv_tree_attention(pool, layer, q, k_pool, v_pool, c.tables, cu, start, tree, out, window,
                               **kw)

    for kw in (dict(layer=1), dict(layer=-1), dict(window=0), dict(sinks=-1), dict(q=None, total_tokens=4),
               dict(tree=tree.data_ptr() + 4)):
        with pytest.raises(pkv.PkvError) as e:
            call(**kw)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    for bad in (tree.to(torch.int32), tree[:3], tree.cpu()):
        with pytest.raises(ValueError, match="tree"):
            call(tree=bad)
    call(batch=0)
    call(total_tokens=0)
    acc, counts = int32([[0, 1]] * 2), int32([1, 2])
    for a in (torch.zeros(2, 65, dtype=torch.int32, device="cuda"),
              torch.zeros(2, 0, dtype=torch.int32, device="cuda")):
        with pytest.raises(pkv.PkvError) as e:
            pkv.pkv_tree_commit(pool, k_pool, v_pool, c.tables, start, a, counts)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    with pytest.raises(ValueError, match="counts"):
        pkv.pkv_tree_commit(pool, k_pool, v_pool, c.tables, start, acc, counts[:1])
    pkv.pkv_tree_commit(pool, k_pool, v_pool, c.tables, start, acc, counts, batch=0)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
