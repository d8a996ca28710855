"""Attention of drafted trees through each of its kernels: clusters, the line of few
rows with its join, and the tile kernel with its join. Which one a call takes goes by
its drafted tokens per sequence and by the context that its sequences may see."""

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
from tree_helpers import attend, pack, random_tree, seen_matrix
from window_helpers import DIM, HKV, HQ, PAGE, U, Cache, check

pytestmark = pytest.mark.gpu

# max_seq_len, committed and drafted tokens: few tokens of few sequences over a short
# context; 8 and fewer a sequence on average, and more than that, too many for clusters
KERNELS = {"clusters": (2048, [900, 30], [8, 5]),
           "line": (16384, [900, 3000] + [37 * i for i in range(12)],
                    [8, 5] + [1 + 3 * i % 8 for i in range(12)]),
           "tiles": (16384, [900, 3000], [64, 40])}


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


def expect(c, q, out, starts, nodes, masks, window, sinks, hidden=None, first_row=0):
    """Checks the rows of every sequence; hidden[b]: tokens that no row sees."""
    row = first_row
    for b, n in enumerate(nodes):
        if n:
            seen = seen_matrix(starts[b], masks[b], window, sinks)
            if hidden is not None:
                seen[:, hidden[b]] = False
            end = starts[b] + n
            ref, tol = attend(q[row:row + n].double(), c.k[b][:end].double(), c.v[b][:end].double(), seen)
            check(out[row:row + n], ref, tol, f"sequence {b}: {starts[b]} + {n}")
        row += n


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (700, 40)])
def test_invalid_pages_are_left_out(window, sinks, kernel):
    # of committed and drafted tokens, sinks, a whole step and the last page; tiles are cut
    # at several of them on the line
    max_seq_len, starts, nodes = KERNELS[kernel]
    rng = np.random.RandomState(5)
    c = Cache([s + n for s, n in zip(starts, nodes)], max_seq_len=max_seq_len, seed=5)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    hidden = []
    for b, n in enumerate(c.lens):
        last = (n - 1) // PAGE
        gone = sorted({0, last} | {p for p in (1, 17, 20, 21, 22, 23, 33, 48, 120, 175) if p < last}
                      if b == 0 or starts[b] > 1000 else {1})
        bad = [c.num_pages, -1, -(1 << 31), (1 << 31) - 1]
        for i, p in enumerate(gone):
            c.table[0, b, p] = bad[i % 4]
        hidden.append(np.concatenate([np.arange(p * PAGE, min((p + 1) * PAGE, n)) for p in gone]))
    masks = [random_tree(rng, n) for n in nodes]
    q = torch.randn(sum(nodes), HQ, DIM, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = torch.empty(sum(nodes), HQ, DIM, device="cuda")
    pool = handle(c)
    pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, torch.from_numpy(c.table).cuda(),
                           int32(np.cumsum([0] + nodes)), int32(starts), pack(sum(masks, [])), out,
                           window, sinks=sinks)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    expect(c, q, out, starts, nodes, masks, window, sinks, hidden)
    # none that is valid: every row is 0
    pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, torch.full_like(c.tables, -1),
                           int32(np.cumsum([0] + nodes)), int32(starts), pack(sum(masks, [])), out,
                           window, sinks=sinks)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    assert bool((out == 0).all())


@pytest.mark.parametrize("kernel", KERNELS)
@pytest.mark.parametrize("what", ["rows", "too many", "start", "end", "negative row", "past the rows"])
def test_bad_sequences_are_flagged_and_left_alone(what, kernel):
    # the second of three sequences is bad, its neighbours are as ever
    max_seq_len, starts, nodes = KERNELS[kernel]
    starts, nodes = [starts[0], 20, starts[1]], [nodes[0], 5, nodes[1]]
    cu = np.cumsum([0] + nodes)
    total = int(cu[3])
    if what == "rows":                            # fewer than none, and the third from there on
        cu[2] = cu[1] - 1
    elif what == "too many":
        cu[2:] += 60
        total += 60
    elif what == "start":
        starts[1] = -1
    elif what == "end":
        starts[1] = max_seq_len - 4
    elif what == "negative row":                  # the first two
        cu[1] = -3
    else:                                         # the last two
        cu[2] = total + 1
    if kernel == "line":                          # and some that draft nothing
        cu, starts = np.append(cu, [cu[3]] * 8), starts + [5] * 8
    c = Cache([max(s, 0) % (max_seq_len - 4) + 64 for s in starts], max_seq_len=max_seq_len, seed=6)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    q = torch.randn(total, HQ, DIM, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = torch.full((total, HQ, DIM), 3.0, device="cuda")
    rng = np.random.RandomState(7)
    flat = [int(rng.randint(0, 1 << 32)) << 32 | int(rng.randint(0, 1 << 32)) for _ in range(total)]
    pool = handle(c)
    pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, int32(cu), int32(starts), pack(flat),
                           out, max_seq_len)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    rows = np.zeros(total, int)                   # sequences that have the row
    checks = []
    for b in range(len(starts)):
        n = int(cu[b + 1] - cu[b])
        if not (0 <= cu[b] and 0 < n <= 64 and cu[b + 1] <= total and
                0 <= starts[b] <= max_seq_len - n):
            continue
        rows[cu[b]:cu[b + 1]] += 1
        at = slice(int(cu[b]), int(cu[b + 1]))
        end = starts[b] + n
        checks.append((at, *attend(q[at].double(), c.k[b][:end].double(), c.v[b][:end].double(),
                                   seen_matrix(starts[b], flat[at], max_seq_len, 0))))
    for at, ref, tol in checks:                   # a row of two sequences is neither's
        alone = torch.from_numpy(rows[at] == 1).cuda()
        check(out[at][alone], ref[alone], tol[alone], f"rows {at}")
    assert rows.any() and bool((out[torch.from_numpy(rows == 0).cuda()] == 3.0).all())


@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_that_see_nothing(kernel):
    max_seq_len, starts, nodes = KERNELS[kernel]
    starts = [0] + starts[1:]
    masks = [[1 << i if i % 3 else 0 for i in range(n)] for n in nodes]
    c = Cache([s + n for s, n in zip(starts, nodes)], max_seq_len=max_seq_len, seed=8)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    q = torch.randn(sum(nodes), HQ, DIM, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = torch.empty(sum(nodes), HQ, DIM, device="cuda")
    pool = handle(c)
    for window in (1, 1 << 20):
        pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, int32(np.cumsum([0] + nodes)),
                               int32(starts), pack(sum(masks, [])), out, window)
        expect(c, q, out, starts, nodes, masks, window, 0)
        assert bool((out[:nodes[0]:3] == 0).all())
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK


@pytest.mark.parametrize("kernel", KERNELS)
def test_captured_with_changing_lengths(kernel):
    # replays whose lengths move the cuts from tile to tile, and away: one long sequence,
    # several, none worth a cut, none at all
    max_seq_len, total = KERNELS[kernel][0], {"clusters": 24, "line": 24, "tiles": 90}[kernel]
    long = 1900 if kernel == "clusters" else 9000
    c = Cache([long, long // 2, 300], max_seq_len=max_seq_len, seed=9)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    q = torch.randn(total, HQ, DIM, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = torch.zeros(total, HQ, DIM, device="cuda")
    pool = handle(c)
    rng = np.random.RandomState(9)
    cu, start = int32([0, 0, 0, 0]), int32([0, 0, 0])
    tree = torch.zeros(total, dtype=torch.int64, device="cuda")

    def call():
        pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, tree, out, max_seq_len)

    call()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            call()
    third = total // 3
    for starts, nodes in (([long - third, long // 2 - third, 300 - third], [third] * 3),
                          ([0, long // 2 - 1, 0], [3, 1, third]), ([long - 2, 0, 0], [2, 0, 0]),
                          ([0, 5, 9], [0, 0, 0]), ([7, 1, 0], [third, third + 2, 1]),
                          ([long - third, 0, 64], [third, total - third - 1, 1]),
                          ([1, long // 2 - third, 300 - third], [0, third, third])):
        nodes = [min(n, 64) for n in nodes]
        masks = [random_tree(rng, n) for n in nodes]
        cu.copy_(int32(np.cumsum([0] + nodes)))
        start.copy_(int32(starts))
        tree.copy_(pack(sum(masks, []) + [0] * (total - sum(nodes))))
        for _ in range(2):
            out.fill_(3.0)
            graph.replay()
        torch.cuda.synchronize()
        expect(c, q, out, starts, nodes, masks, max_seq_len, 0)
        assert bool((out[sum(nodes):] == 3.0).all())
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK


def test_a_handle_of_many_sequences_keeps_no_room_for_trees():
    # the decode's partials of 32 sequences x 64 splits (34.6 MB) are room enough, so a handle
    # takes that and what cudaMalloc rounds up; with 20 MB of its own it took 55
    def create():
        return pkv.pkv_pool_create(1, 64, 32, max_seq_len=2048)

    first = create()                               # loads the kernels
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    handles = [create() for _ in range(8)]
    taken = before - torch.cuda.mem_get_info()[0]
    partials = 2 * 32 * 32 * 64 * (64 + 2) * 4
    assert taken <= 8 * (partials + (8 << 20)), taken
    del handles, first


@pytest.mark.parametrize("pdl", [False, True])
@pytest.mark.parametrize("kernel", KERNELS)
def test_trees_between_decode_calls_that_keep_partials(kernel, pdl):
    # trees and the decode's tickets share the handle's scratch: the same outputs bit for
    # bit as on a handle of each, issued one right after the other and replayed
    max_seq_len, starts, nodes = KERNELS[kernel]
    batch, total = len(starts), sum(nodes)
    c = Cache([s + n for s, n in zip(starts, nodes)], max_seq_len=max_seq_len, seed=10)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    flags = (pkv.PKV_FLAG_PDL if pdl else 0) | (pkv.PKV_FLAG_LONG_CONTEXT if max_seq_len > 2048 else 0)

    def create():
        return pkv.pkv_pool_create(1, c.num_pages, batch, max_seq_len=max_seq_len, flags=flags)

    g = torch.Generator().manual_seed(3)
    q = torch.randn(total, HQ, DIM, generator=g).bfloat16().cuda()
    qd = torch.randn(batch, HQ, DIM, generator=g).bfloat16().cuda()
    rng = np.random.RandomState(10)
    tree = pack(sum([random_tree(rng, n) for n in nodes], []))
    cu, start, lens = int32(np.cumsum([0] + nodes)), int32(starts), c.lens_tensor()

    def trees(pool, out):
        pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, tree, out, max_seq_len)

    def decode(pool, out, splits):
        pkv.pkv_window_attention(pool, 0, qd, k_pool, v_pool, c.tables, lens, out, max_seq_len,
                                 num_splits=splits)

    def outputs():
        return [torch.empty(total if i % 2 else batch, HQ, DIM, device="cuda") for i in range(5)]

    want = outputs()
    for i, out in enumerate(want):
        trees(create(), out) if i % 2 else decode(create(), out, (64, 0, 40)[i // 2])
    pool, got = create(), outputs()

    def run():
        for i, out in enumerate(got):
            trees(pool, out) if i % 2 else decode(pool, out, (64, 0, 40)[i // 2])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    for _ in range(20):
        for out in got:
            out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK


@pytest.mark.parametrize("nodes", [4, 40])
def test_a_context_of_a_million_tokens(nodes):
    start = pkv.PKV_MAX_LONG_CONTEXT - 64
    n = start + nodes
    # V grows along the context, so that a part lost or taken twice shows (2^-8 of it and more);
    # of n / 16 additions no more than 512 come one after the other (those of a warp's pages
    # or a part's segments, and of the parts)
    c = Cache([n], max_seq_len=pkv.PKV_MAX_LONG_CONTEXT, seed=1, k_scale=0.125)
    c.v[0] = (torch.arange(n, device="cuda") / n).bfloat16()[:, None, None].repeat(1, HKV, DIM)
    k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))
    pool = handle(c)
    masks = random_tree(np.random.RandomState(1), nodes)
    q = torch.randn(nodes, HQ, DIM, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    out = torch.empty(nodes, HQ, DIM, device="cuda")
    for window, sinks in ((c.max_seq_len, 0), (500000, 100)):
        pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, int32([0, nodes]), int32([start]),
                               pack(masks), out, window, sinks=sinks)
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK
        seen = seen_matrix(start, masks, window, sinks)
        for i in (0, nodes // 2, nodes - 1):
            ref, tol = attend(q[i:i + 1].double(), c.k[0].double(), c.v[0].double(), seen[i:i + 1])
            check(out[i:i + 1], ref, tol - 2 * (int(seen[i].sum()) / 16 - 512) * U)


@pytest.mark.parametrize("kernel", KERNELS)
def test_two_handles_on_two_streams(kernel):
    max_seq_len, starts, nodes = KERNELS[kernel]
    total = sum(nodes)
    tree = pack(sum([random_tree(np.random.RandomState(3), n) for n in nodes], []))
    q = torch.randn(total, HQ, DIM, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    cu, start = int32(np.cumsum([0] + nodes)), int32(starts)
    calls, want = [], []
    for seed in range(2):
        c = Cache([s + n for s, n in zip(starts, nodes)], max_seq_len=max_seq_len, seed=seed)
        k_pool, v_pool = c.pools(lambda b: np.ones(c.lens[b], bool))

        def call(out, c=c, k_pool=k_pool, v_pool=v_pool, pool=handle(c)):
            pkv.pkv_tree_attention(pool, 0, q, k_pool, v_pool, c.tables, cu, start, tree, out,
                                   max_seq_len)

        calls.append(call)
        want.append(torch.empty(total, HQ, DIM, device="cuda"))
        call(want[-1])
    outs = [[torch.empty_like(want[0]) for _ in range(20)] for _ in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for i in range(20):
        for call, stream, out in zip(calls, streams, outs):
            with torch.cuda.stream(stream):
                call(out[i])
    torch.cuda.synchronize()
    for out, ref in zip(outs, want):
        assert all(torch.equal(o, ref) for o in out)
