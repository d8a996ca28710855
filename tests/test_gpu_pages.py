"""Page copies and compaction on the device against plain indexing (every bit of
both pools and of the tables), their refusals, and the whole run together:
multi-axis fill, windowed prefill, forks, windowed decode, release, compaction."""

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
import window_helpers as W

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def _pools(num_pages, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randint(-32768, 32768, (num_pages, 8, 16, 64), generator=g, device="cuda",
                          dtype=torch.int16).view(torch.bfloat16) for _ in range(2)]


def _bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("n", [1, 2, 31, 256, 257, 1000, 1024, 1025, 5000])
@pytest.mark.parametrize("partial", [False, True])
def test_copies(n, partial):
    pages = 2 * n + 7
    kp, vp = _pools(pages, n)
    rng = np.random.RandomState(n)
    ids = rng.permutation(pages)
    src, dst = ids[rng.randint(0, n, n)], ids[n:2 * n]
    tokens = rng.randint(0, 17, n) if partial else None
    want = [p.clone() for p in (kp, vp)]
    for w, p in zip(want, (kp, vp)):
        moved = _bits(p)[torch.as_tensor(src).cuda()].clone()
        old = _bits(p)[torch.as_tensor(dst).cuda()]
        if partial:
            keep = torch.arange(16, device="cuda")[None] < torch.as_tensor(tokens).cuda()[:, None]
            moved = torch.where(keep[:, None, :, None], moved, old)
        _bits(w)[torch.as_tensor(dst).cuda()] = moved
    pool = pkv.pkv_pool_create(1, pages, 1)
    pkv.pkv_copy_pages(pool, _i32(src), _i32(dst), kp, vp,
                       tokens=_i32(tokens) if partial else None)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert torch.equal(_bits(kp), _bits(want[0])) and torch.equal(_bits(vp), _bits(want[1]))
    pool.close()


@pytest.mark.parametrize("filler", [0, 300, 1200])
def test_pairs_that_clash_or_leave_the_pool_are_skipped(filler):
    """The same outcome in the one-launch form and, with `filler` good pairs
    around, in the counted one."""
    pages = 64 + 2 * filler
    far = 2 ** 31 - 1
    src = [0, 1, 2, 3, 4, 5, 6, 7, 8, -1, pages, 9, far, 10]
    dst = [20, 21, 21, 22, 23, 3, 6, 24, 25, 26, 27, -1, 28, pages]
    tok = [16, 16, 16, 16, 0, 16, 16, 17, -1, 16, 16, 16, 16, 16]
    good = {20: 0, 22: 3}                       # 21 named twice, 3 a source, 6 -> 6, the rest bad
    src = src + [64 + i for i in range(filler)]
    dst = dst + [64 + filler + i for i in range(filler)]
    tok = tok + [16] * filler
    good.update({64 + filler + i: 64 + i for i in range(filler)})
    kp, vp = _pools(pages, 3)
    want = [kp.clone(), vp.clone()]
    for w in want:
        for d, s in good.items():
            _bits(w)[d] = _bits(w)[s]
    pool = pkv.pkv_pool_create(1, pages, 1)
    pkv.pkv_copy_pages(pool, _i32(src), _i32(dst), kp, vp, tokens=_i32(tok))
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    assert torch.equal(_bits(kp), _bits(want[0])) and torch.equal(_bits(vp), _bits(want[1]))
    # a following call is not affected
    pkv.pkv_copy_pages(pool, _i32([1]), _i32([2]), kp, vp)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert torch.equal(_bits(kp[1]), _bits(kp[2]))
    pool.close()


@pytest.mark.parametrize("layers,max_batch,max_seq_len", [(1, 1, 16), (3, 5, 48), (2, 7, 2048)])
@pytest.mark.parametrize("n", [1, 40, 700])
def test_compaction(layers, max_batch, max_seq_len, n):
    pages = 2 * n + 30
    kp, vp = _pools(pages, n)
    rng = np.random.RandomState(n + layers)
    ids = rng.permutation(pages)
    src, dst, rest = ids[:n], ids[n:2 * n], ids[2 * n:]
    table = rng.choice(np.concatenate([src, rest, [-1, -1, pages, 2 ** 31 - 1]]),
                       (layers, max_batch, max_seq_len // 16)).astype(np.int32)
    to = {int(s): int(d) for s, d in zip(src, dst)}
    want_t = np.vectorize(lambda p: to.get(int(p), int(p)))(table).astype(np.int32)
    want = [kp.clone(), vp.clone()]
    for w in want:
        _bits(w)[torch.as_tensor(dst).cuda()] = _bits(w)[torch.as_tensor(src).cuda()]
    pool = pkv.pkv_pool_create(layers, pages, max_batch, max_seq_len=max_seq_len)
    t = _i32(table)
    for _ in range(2):                          # the second call finds nothing left to rewrite
        pkv.pkv_compact_pages(pool, _i32(src), _i32(dst), kp, vp, t)
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK
        assert np.array_equal(t.cpu().numpy(), want_t)
        assert torch.equal(_bits(kp), _bits(want[0])) and torch.equal(_bits(vp), _bits(want[1]))
    pool.close()


def test_compaction_skips_clashes():
    pages = 32
    kp, vp = _pools(pages)
    want = [kp.clone(), vp.clone()]
    src, dst = [20, 21, 21, 22, 23, 24, -1], [0, 1, 2, 3, 3, 20, 5]
    for w in want:
        _bits(w)[0] = _bits(w)[20]              # 21 moves twice, 3 is named twice, 20 is a source
    table = torch.arange(16, 32, dtype=torch.int32, device="cuda").view(1, 1, 16)
    want_t = table.clone()
    want_t[0, 0, 4] = 0
    pool = pkv.pkv_pool_create(1, pages, 1, max_seq_len=256)
    pkv.pkv_compact_pages(pool, _i32(src), _i32(dst), kp, vp, table)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    assert torch.equal(table, want_t)
    assert torch.equal(_bits(kp), _bits(want[0])) and torch.equal(_bits(vp), _bits(want[1]))
    pool.close()


@pytest.mark.parametrize("n", [5, 60, 256, 257, 400, 1024, 1025])
def test_compactions_one_after_another(n):
    """Random lists with sources and destinations named twice, ids out of range and
    pages that are both, over one handle: what one list leaves behind does not
    reach the next."""
    pages = max(900, 2 * n + 50)
    kp, vp = _pools(pages, n)
    rng = np.random.RandomState(n)
    pool = pkv.pkv_pool_create(2, pages, 3, max_seq_len=512)
    table = rng.randint(-1, pages, (2, 3, 32)).astype(np.int32)
    t = _i32(table)
    for _ in range(6):
        ids = rng.permutation(pages)
        src, dst = ids[:n].copy(), ids[n:2 * n].copy()
        for _ in range(4):                     # several rules broken at once
            a, b = rng.randint(0, n, 2)
            rng.choice([lambda: src.__setitem__(a, src[b]), lambda: dst.__setitem__(a, dst[b]),
                        lambda: dst.__setitem__(a, src[b]), lambda: src.__setitem__(a, -1),
                        lambda: dst.__setitem__(a, pages)])()
        ok = [0 <= s < pages and 0 <= d < pages and (src == s).sum() == 1
              and (dst == d).sum() == 1 and not (src == d).any() for s, d in zip(src, dst)]
        good_s, good_d = src[ok], dst[ok]
        want = [kp.clone(), vp.clone()]
        for w in want:
            if len(good_s):
                _bits(w)[torch.as_tensor(good_d).cuda()] = _bits(w)[torch.as_tensor(good_s).cuda()]
        to = {int(s): int(d) for s, d in zip(good_s, good_d)}
        table = np.vectorize(lambda p: to.get(int(p), int(p)))(table).astype(np.int32)
        pkv.pkv_compact_pages(pool, _i32(src), _i32(dst), kp, vp, t)
        st = pkv.pkv_get_error(pool)
        assert st == (pkv.PKV_OK if all(ok) else pkv.PKV_ERR_OUT_OF_RANGE)
        assert np.array_equal(t.cpu().numpy(), table)
        assert torch.equal(_bits(kp), _bits(want[0])) and torch.equal(_bits(vp), _bits(want[1]))
    pool.close()


@pytest.mark.parametrize("pages,n", [(700, 300), (2300, 1100)])
def test_captured_and_replayed_with_other_lists(pages, n):
    """Replays take the lists' current content; nothing is left over from the last."""
    kp, vp = _pools(pages)
    want = [kp.clone(), vp.clone()]
    pool = pkv.pkv_pool_create(1, pages, 1, max_seq_len=256)
    src, dst = _i32(np.zeros(n)), _i32(np.zeros(n))
    table = torch.zeros(1, 1, 16, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pkv.pkv_compact_pages(pool, src, dst, kp, vp, table)
    for seed in range(3):
        ids = np.random.RandomState(seed).permutation(pages)
        src.copy_(_i32(ids[:n]))
        dst.copy_(_i32(ids[n:2 * n]))
        at = np.arange(n - 10, n + 6)
        table.copy_(_i32(ids[at]).view(1, 1, 16))
        want_t = np.where(at < n, ids[at + n], ids[at])
        for w in want:
            _bits(w)[torch.as_tensor(ids[n:2 * n]).cuda()] = \
                _bits(w)[torch.as_tensor(ids[:n]).cuda()]
        graph.replay()
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK
        assert np.array_equal(table.cpu().numpy().ravel(), want_t)
        assert torch.equal(_bits(kp), _bits(want[0])) and torch.equal(_bits(vp), _bits(want[1]))
    del graph
    pool.close()


def test_lists_that_start_anywhere():
    """Slices of a longer list: int32 alignment is enough."""
    kp, vp = _pools(64)
    want = kp.clone()
    ids = _i32(range(64))
    tok = _i32([16] * 64)
    pool = pkv.pkv_pool_create(1, 64, 1)
    _bits(want)[33:36] = _bits(want)[5:8]
    pkv.pkv_copy_pages(pool, ids[5:8], ids[33:36], kp, vp, tokens=tok[1:4])
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert torch.equal(_bits(kp), _bits(want))
    pool.close()


def test_refusals():
    kp, vp = _pools(10)
    pool = pkv.pkv_pool_create(1, 10, 1, max_seq_len=256)
    a, b = _i32([1]), _i32([2])
    table = torch.zeros(1, 1, 16, dtype=torch.int32, device="cuda")
    pkv.pkv_copy_pages(pool, a, b, kp, vp, n=0)
    for f in (lambda: pkv.pkv_copy_pages(pool, a, b, kp, vp, n=-1),
              lambda: pkv.pkv_copy_pages(pool, a, None, kp, vp),
              lambda: pkv.pkv_copy_pages(pool, _i32(range(11)), _i32(range(11)), kp, vp),
              lambda: pkv.pkv_compact_pages(pool, a, b, kp, vp, None)):
        with pytest.raises(pkv.PkvError) as e:
            f()
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    for f in (lambda: pkv.pkv_copy_pages(pool, a.cpu(), b, kp, vp),
              lambda: pkv.pkv_copy_pages(pool, a.long(), b, kp, vp),
              lambda: pkv.pkv_copy_pages(pool, a, b, kp[:9], vp),
              lambda: pkv.pkv_copy_pages(pool, a, b, kp, vp, tokens=b[:0]),
              lambda: pkv.pkv_compact_pages(pool, a, b, kp, vp, table[:, :, :8].contiguous())):
        with pytest.raises(ValueError):
            f()
    pool.close()


def test_serving_run_with_forks_window_and_compaction():
    """Prompts with image positions are filled and attended behind a window,
    forked, decoded on, their old pages released, the pool compacted, and
    decoded on: every step against the 64-bit restatement of each sequence's own
    token history."""
    L, WINDOW, SINKS, PAGES, B = 2, 100, 20, 160, 5
    axes_of = [0] * 8 + [1] * 12 + [2] * 12
    cos, sin = W.angles(4096)
    rope = pkv.pkv_axes_rope(cos, sin, axes_of)
    g = torch.Generator(device="cuda").manual_seed(9)
    sched = pkv.pkv_sched_create(PAGES, num_layers=L)
    pool = pkv.pkv_pool_create(L, PAGES, B)
    kp, vp = [torch.full((PAGES, 8, 16, 64), float("nan"), device="cuda").bfloat16() for _ in "kv"]
    prompts = [150, 37]
    ids = [pkv.pkv_sched_submit(sched, n, 60) for n in prompts]
    assert pkv.pkv_sched_admit(sched) == ids
    hist = {}                                   # id -> per layer [K rows], [V rows] as stored

    def tables(batch):
        return torch.from_numpy(pkv.pkv_sched_block_tables(sched, batch, max_batch=B)).cuda()

    def rotated(x, pos, dtype):
        return W.rotate(x, cos, sin, pos, axes_of, dtype)

    # prefill, layer by layer
    pkv.pkv_sched_extend_batch(sched, ids, prompts)
    t = tables(ids)
    cu = _i32(np.concatenate([[0], np.cumsum(prompts)]))
    start = _i32([0, 0])
    total = sum(prompts)
    pos = torch.randint(0, 4096, (3, total), generator=g, device="cuda").int()
    for b, i in enumerate(ids):
        hist[i] = [[], []]
    for layer in range(L):
        q = torch.randn(total, 32, 64, generator=g, device="cuda").bfloat16()
        k = torch.randn(total, 8, 64, generator=g, device="cuda").bfloat16()
        v = torch.randn(total, 8, 64, generator=g, device="cuda").bfloat16()
        stored, turned = rotated(k, pos, torch.float32).bfloat16(), rotated(q, pos, torch.float32).bfloat16()
        pkv.pkv_prefill_fill_axes(pool, layer, q, k, v, q, kp, vp, t, cu, start, rope, pos, 150)
        out = torch.zeros(total, 32, 64, device="cuda")
        pkv.pkv_window_prefill_attention(pool, layer, q, kp, vp, t, cu, start, out, 150, WINDOW,
                                         sinks=SINKS)
        assert torch.equal(_bits(q), _bits(turned))
        row = 0
        for i, n in zip(ids, prompts):
            hist[i][0].append(stored[row:row + n])
            hist[i][1].append(v[row:row + n])
            ref, tol = W.attend(turned[row:row + n].double(), stored[row:row + n].double(),
                                v[row:row + n].double(), torch.arange(n, device="cuda"), WINDOW,
                                SINKS)
            W.check(out[row:row + n], ref, tol, "prefill")
            row += n

    lens = dict(zip(ids, prompts))

    def decode(batch):
        for i in batch:
            lens[i] += 1
        pkv.pkv_sched_extend_batch(sched, batch, [lens[i] for i in batch])
        t = tables(batch)
        n = _i32([lens[i] for i in batch])
        at = torch.randint(0, 4096, (3, len(batch)), generator=g, device="cuda").int()
        for layer in range(L):
            q = torch.randn(len(batch), 32, 64, generator=g, device="cuda").bfloat16()
            k = torch.randn(len(batch), 8, 64, generator=g, device="cuda").bfloat16()
            v = torch.randn(len(batch), 8, 64, generator=g, device="cuda").bfloat16()
            out = torch.zeros(len(batch), 32, 64, device="cuda")
            pkv.pkv_window_append_attend(pool, layer, q, k, v, kp, vp, t, n, out, WINDOW,
                                         sinks=SINKS, rope=rope, rope_positions=at)
            key, turned = rotated(k, at, torch.float32).bfloat16(), rotated(q, at, torch.float64)
            for b, i in enumerate(batch):
                hist[i][0][layer] = torch.cat([hist[i][0][layer], key[b:b + 1]])
                hist[i][1][layer] = torch.cat([hist[i][1][layer], v[b:b + 1]])
                ref, tol = W.attend(turned[b:b + 1], hist[i][0][layer].double(),
                                    hist[i][1][layer].double(),
                                    torch.tensor([lens[i] - 1], device="cuda"), WINDOW, SINKS)
                W.check(out[b:b + 1], ref, tol, f"decode of {i} at {lens[i]}")
        assert pkv.pkv_get_error(pool) == pkv.PKV_OK

    def fork(parent, length, new):
        child, src, dst, tokens = pkv.pkv_sched_fork(sched, parent, length, new)
        assert len(src) == (L if length % 16 else 0)
        if len(src):
            pkv.pkv_copy_pages(pool, _i32(src), _i32(dst), kp, vp, tokens=_i32(tokens))
        hist[child] = [[x[:length] for x in part] for part in hist[parent]]
        lens[child] = length
        return child

    a = fork(ids[0], 150, 30)                   # a partial page is copied
    b = fork(ids[0], 144, 30)                   # whole pages only
    c = fork(a, 149, 20)                        # a fork of a fork
    batch = [ids[0], ids[1], a, b, c]
    for _ in range(12):
        decode(batch)
    free = pkv.pkv_sched_get_stats(sched)["free_pages"]
    for i in batch:                             # what the window left behind goes
        pkv.pkv_sched_release(sched, i, max(0, lens[i] + 1 - WINDOW), SINKS)
    assert pkv.pkv_sched_get_stats(sched)["free_pages"] > free
    decode(batch)
    pkv.pkv_sched_finish(sched, ids[0])         # its shared pages stay with the forks
    batch = batch[1:]
    t = tables(batch)
    used = PAGES - pkv.pkv_sched_get_stats(sched)["free_pages"]
    src, dst = pkv.pkv_sched_compact(sched)
    assert len(src) and max(dst) < used <= min(src)
    pkv.pkv_compact_pages(pool, _i32(src), _i32(dst), kp, vp, t)
    assert torch.equal(t, tables(batch))        # the device's tables are the scheduler's
    for p in (kp, vp):
        _bits(p)[torch.as_tensor(src).long().cuda()] = _bits(torch.full((1,), float("nan"),
                                                             device="cuda").bfloat16())
    for _ in range(5):
        decode(batch)
    for i in batch:
        pkv.pkv_sched_finish(sched, i)
    st = pkv.pkv_sched_get_stats(sched)
    assert st["free_pages"] == st["free_credits"] == PAGES
    pool.close()
