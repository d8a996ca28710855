"""Handles with programmatic dependent launch: which launches may start under the
one before them (read off the captured graph's edges), and the same bits as without
the flag in every launch shape of the windowed decode."""

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
import window_helpers as W

pytestmark = pytest.mark.gpu

AXES = [0] * 8 + [1] * 12 + [2] * 12


def _edges(step):
    """Whether each launch of step(stream) may start under the one before it, in
    order: the edges of the chain that the captured launches form."""
    cuda = ctypes.CDLL("libcuda.so.1")
    P = ctypes.c_void_p

    def call(name, *args):
        assert getattr(cuda, name)(*args) == 0, name
    stream = torch.cuda.Stream()
    handle, graph, count = P(stream.cuda_stream), P(), ctypes.c_size_t()
    torch.cuda.synchronize()
    call("cuStreamBeginCapture_v2", handle, 1)                   # this thread's calls only
    try:
        step(stream)
    finally:
        call("cuStreamEndCapture", handle, ctypes.byref(graph))
    call("cuGraphGetEdges_v2", graph, None, None, None, ctypes.byref(count))
    n = count.value
    tail, head, data = (P * n)(), (P * n)(), (ctypes.c_uint8 * 8 * n)()
    call("cuGraphGetEdges_v2", graph, tail, head, data, ctypes.byref(count))
    call("cuGraphDestroy", graph)
    after = {tail[i]: (head[i], data[i][2] == 1) for i in range(n)}
    node, = set(after) - {h for h, _ in after.values()}
    kinds = []
    while node in after:
        node, programmatic = after[node]
        kinds.append(programmatic)
    assert len(kinds) == n
    return kinds


class Batch:
    """A batch of sequences over shuffled pages, its inputs, and one handle."""

    def __init__(self, lens, flags=pkv.PKV_FLAG_PDL, layers=2, window=300, sinks=4, seed=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.layers, self.window, self.sinks = lens, layers, window, sinks
        B = len(lens)
        need = [-(-(n + 8) // 16) for n in lens]
        table = np.full((layers, B, 128), -1, np.int32)
        ids = np.random.RandomState(seed).permutation(layers * sum(need) + 64).astype(np.int32)
        at = 0
        for layer in range(layers):
            for b, n in enumerate(need):
                table[layer, b, :n] = ids[at:at + n]
                at += n
        self.spare = ids[at:]
        self.num_pages = len(ids)
        self.table = table
        self.tables = torch.from_numpy(table).cuda()

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda").bfloat16()
        self.kp, self.vp = normal(self.num_pages, 8, 16, 64), normal(self.num_pages, 8, 16, 64)
        self.q, self.k = normal(layers, B, 32, 64), normal(layers, B, 8, 64)
        self.v = normal(layers, B, 8, 64)
        self.n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.none = torch.zeros_like(self.n)
        cos, sin = W.angles(3000)
        self.rope = dict(rope=pkv.pkv_axes_rope(cos, sin, AXES),
                         rope_positions=torch.randint(0, 3000, (3, B), generator=g,
                                                      device="cuda").int())
        self.out = torch.zeros(layers, B, 32, 64, device="cuda")
        self.again = torch.zeros(layers, B, 32, 64, device="cuda")
        self.pool = pkv.pkv_pool_create(layers, self.num_pages, B, flags=flags)

    def fused(self, layer=0, stream=None, rope=None, **kw):
        pkv.pkv_window_append_attend(self.pool, layer, self.q[layer], self.k[layer], self.v[layer],
                                     self.kp, self.vp, self.tables, self.n, self.out[layer],
                                     self.window, sinks=self.sinks, stream=stream,
                                     **(rope or {}), **kw)

    def unfused(self, layer=0, stream=None, lens=None, rope=None, **kw):
        pkv.pkv_window_attention(self.pool, layer, self.q[layer], self.kp, self.vp, self.tables,
                                 self.n if lens is None else lens, self.again[layer], self.window,
                                 sinks=self.sinks, stream=stream, **(rope or {}), **kw)


def _writers(x):
    """The calls that write pages or tables, each with the number of its launches."""
    src, dst = [torch.from_numpy(x.spare[s:s + 8].copy()).cuda() for s in (0, 8)]
    long = [torch.from_numpy(np.arange(s, s + 1030, dtype=np.int32)).cuda() for s in (0, 1030)]
    B = len(x.lens)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    start = x.n - 1
    out = torch.empty_like(x.q[0])
    x.keep = (src, dst, long, cu, start, out)
    return {
        "copy": (1, lambda s: pkv.pkv_copy_pages(x.pool, src, dst, x.kp, x.vp, stream=s)),
        "long copy": (3, lambda s: pkv.pkv_copy_pages(x.pool, *long, x.kp, x.vp, stream=s)),
        "compact": (2, lambda s: pkv.pkv_compact_pages(x.pool, src, dst, x.kp, x.vp, x.tables,
                                                       stream=s)),
        "fill": (1, lambda s: pkv.pkv_prefill_fill_axes(
            x.pool, 0, x.q[0], x.k[0], x.v[0], out, x.kp, x.vp, x.tables, cu, start,
            x.rope["rope"], x.rope["rope_positions"], 1, stream=s))}


@pytest.mark.parametrize("what", ["copy", "long copy", "compact", "fill"])
def test_a_decode_waits_for_what_wrote_pages(what):
    """Before its wait a programmatic launch reads tables and pages, so it may not start
    under the handle's own call that writes them; later ones start early again."""
    x = Batch([2000] * 9 + [700])                          # > 2,060 pages
    launches, write = _writers(x)[what]
    pool = x.pool
    full = pkv.pkv_decode_attention
    decodes = {
        "fused": lambda s: x.fused(stream=s),
        "unfused": lambda s: x.unfused(stream=s),
        "units": lambda s: x.fused(stream=s, num_splits=33),
        "full": lambda s: full(pool, 0, x.q[0], x.kp, x.vp, x.tables, x.n, x.again[0], stream=s)}
    for name, decode in decodes.items():
        def step(s):
            decode(s)
            write(s)
            decode(s)
            decode(s)
        assert _edges(step) == [False] * launches + [False, True], name
    # a list without pairs launches nothing and holds nothing up
    empty = torch.zeros(1, dtype=torch.int32, device="cuda")

    def idle(s):
        x.fused(stream=s)
        pkv.pkv_copy_pages(pool, empty, empty, x.kp, x.vp, n=0, stream=s)
        x.fused(stream=s)
    assert _edges(idle) == [True]
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    pool.close()


def test_handles_without_the_flag_have_plain_launches():
    x = Batch([40, 50], flags=0)
    copy = _writers(x)["copy"][1]

    def step(s):
        x.fused(stream=s)
        copy(s)
        x.fused(stream=s)
        x.unfused(stream=s)
    assert _edges(step) == [False] * 3
    x.pool.close()


# (batch, splits): one cluster, units found by one warp and by a block, tickets
@pytest.mark.parametrize("batch,num_splits", [(3, 0), (64, 0), (120, 0), (6, 33), (6, 5)])
@pytest.mark.parametrize("rotated", [False, True])
def test_the_same_bits_as_without_the_flag(batch, num_splits, rotated):
    """Steps of two layers: append and attend, a launch whose rows are all padding, and
    attention again over what was appended two launches before; called one by one and
    replayed from a graph, lengths changing in between."""
    lens = np.random.RandomState(batch).randint(1, 1500, batch).tolist()
    results = []
    for flags, captured in ((0, False), (pkv.PKV_FLAG_PDL, False), (pkv.PKV_FLAG_PDL, True)):
        x = Batch(lens, flags, window=600)
        rope = x.rope if rotated else None
        kw = dict(rope=rope, num_splits=num_splits)

        def step():
            for layer in range(x.layers):
                x.fused(layer, **kw)
                x.unfused(layer, lens=x.none, **kw)
                x.unfused(layer, **kw)
        if captured:
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                step()
        seen = []
        for _ in range(5):
            graph.replay() if captured else step()
            torch.cuda.synchronize()
            seen += [x.out.clone(), x.again.clone()]
            x.n += 1
            torch.cuda.synchronize()
        assert pkv.pkv_get_error(x.pool) == pkv.PKV_OK
        results.append((torch.stack(seen), x.kp.view(torch.int16), x.vp.view(torch.int16)))
        if captured:
            del graph
        del step
        x.pool.close()
    assert not torch.isnan(results[0][0]).any() and (results[0][0] != 0).any(-1).all()
    for other in results[1:]:
        for a, b in zip(results[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("batch", [3, 64])
def test_decode_right_after_a_compaction(batch):
    """Pages move, the tables follow, and what the pages held before is overwritten: the
    decode after them gives the bits it gave before them."""
    lens = np.random.RandomState(batch).randint(40, 1500, batch).tolist()
    x = Batch(lens, window=2048)
    want = None
    src = torch.from_numpy(x.table[0, :min(batch, 30), 0].copy()).cuda()
    dst = torch.from_numpy(x.spare[:len(src)].copy()).cuda()
    gone = torch.from_numpy(x.spare[30:30 + 1].copy()).cuda().expand(len(src)).contiguous()
    x.kp[x.spare[30]], x.vp[x.spare[30]] = float("nan"), float("nan")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x.unfused()
        pkv.pkv_compact_pages(x.pool, src, dst, x.kp, x.vp, x.tables)
        pkv.pkv_copy_pages(x.pool, gone, src, x.kp, x.vp)
        x.unfused(layer=1)
        x.unfused()
    x.unfused()
    want = x.again[0].clone()
    graph.replay()
    assert pkv.pkv_get_error(x.pool) == pkv.PKV_OK
    assert torch.equal(x.again[0], want)
    assert torch.isnan(x.kp[src.long()].float()).all()
    assert torch.equal(x.tables[0, :len(src), 0], dst)
    del graph
    x.pool.close()
