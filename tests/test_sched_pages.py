"""The scheduler's forks, releases behind a window and compaction, on the CPU:
against a plain model of owners and credits, under random operations."""

import numpy as np
import pytest

import paged_kv_cache_210_gb300 as pkv
from paged_kv_cache_210_gb300 import build as lib_build


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return pkv.load()


def _sched(lib, pages, layers=2, max_seq_len=256):
    return pkv.pkv_sched_create(pages, num_layers=layers, max_seq_len=max_seq_len, lib=lib)


def _table(s, i):
    return pkv.pkv_sched_block_tables(s, [i])[:, 0]


def _status(f):
    with pytest.raises(pkv.PkvError) as e:
        f()
    return e.value.status


def _start(s, prompt, new):
    i = pkv.pkv_sched_submit(s, prompt, new)
    assert pkv.pkv_sched_admit(s) == [i]
    pkv.pkv_sched_extend(s, i, prompt)
    return i


def test_fork_shares_whole_pages_and_copies_the_last(lib):
    s = _sched(lib, 64)
    a = _start(s, 37, 20)
    child, src, dst, tokens = pkv.pkv_sched_fork(s, a, 37, 10)
    ta, tc = _table(s, a), _table(s, child)
    assert (ta[:, :2] == tc[:, :2]).all() and (ta[:, 2] != tc[:, 2]).all()
    assert src.tolist() == ta[:, 2].tolist() and dst.tolist() == tc[:, 2].tolist()
    assert tokens.tolist() == [5, 5]
    st = pkv.pkv_sched_get_stats(s)
    assert st["free_pages"] == 64 - 6 - 2 and st["active"] == 2
    # budgets: ceil(56 / 16) and ceil(46 / 16) pages in each of 2 layers
    assert st["free_credits"] == 64 - 8 - 6
    pkv.pkv_sched_extend(s, child, 46)
    assert _status(lambda: pkv.pkv_sched_extend(s, child, 47)) == pkv.PKV_ERR_INVALID_ARG
    pkv.pkv_sched_finish(s, a)                       # the shared pages stay
    assert pkv.pkv_sched_get_stats(s)["free_pages"] == 64 - 6
    assert (_table(s, child)[:, :2] == ta[:, :2]).all()
    pkv.pkv_sched_finish(s, child)
    st = pkv.pkv_sched_get_stats(s)
    assert st["free_pages"] == st["free_credits"] == 64 and st["finished"] == 2


def test_fork_of_whole_pages_copies_nothing(lib):
    s = _sched(lib, 64)
    a = _start(s, 48, 20)
    child, src, dst, tokens = pkv.pkv_sched_fork(s, a, 32, 10)
    assert len(src) == len(dst) == len(tokens) == 0
    assert (_table(s, child)[:, :2] == _table(s, a)[:, :2]).all()
    assert (_table(s, child)[:, 2:] == -1).all()


def test_fork_refusals(lib):
    s = _sched(lib, 12)
    a = _start(s, 33, 16)                            # budget 6, holds 6
    before = pkv.pkv_sched_get_stats(s)
    assert _status(lambda: pkv.pkv_sched_fork(s, a, 33, 70)) == pkv.PKV_ERR_REJECTED
    # 34: beyond what the parent reached, though inside its last page, which it
    # will go on writing
    for args in ((a, 0, 5), (a, 34, 5), (a, 49, 5), (a, -1, 5), (a, 33, 0), (a + 1, 33, 5)):
        assert _status(lambda: pkv.pkv_sched_fork(s, *args)) == pkv.PKV_ERR_INVALID_ARG
    assert pkv.pkv_sched_get_stats(s) == before
    w = pkv.pkv_sched_submit(s, 60, 5)               # waits; not forkable
    assert _status(lambda: pkv.pkv_sched_fork(s, w, 10, 5)) in (pkv.PKV_ERR_INVALID_ARG,)
    child = pkv.pkv_sched_fork(s, a, 33, 1)[0]
    assert _table(s, child).shape == (2, 16)


def test_release_behind_a_window(lib):
    s = _sched(lib, 64)
    a = _start(s, 150, 20)
    t = _table(s, a)
    free = pkv.pkv_sched_get_stats(s)
    # window starts at 70, 20 sinks: pages 2 and 3 hold only positions 32 .. 63
    assert pkv.pkv_sched_release(s, a, 70, 20) == 4
    t2 = _table(s, a)
    assert (t2[:, 2:4] == -1).all() and (np.delete(t2, [2, 3], 1) == np.delete(t, [2, 3], 1)).all()
    st = pkv.pkv_sched_get_stats(s)
    assert st["free_pages"] == free["free_pages"] + 4
    assert st["free_credits"] == free["free_credits"] + 4
    assert pkv.pkv_sched_release(s, a, 70, 20) == 0
    assert pkv.pkv_sched_release(s, a, 3, 0) == 0
    assert pkv.pkv_sched_release(s, a, 150, 200) == 0
    assert pkv.pkv_sched_release(s, a, 0, 2 ** 31 - 1) == 0
    for args in ((a, 151, 0), (a, 2 ** 31 - 1, 0), (a, -1, 0), (a, 10, -1), (a + 1, 10, 0)):
        assert _status(lambda: pkv.pkv_sched_release(s, *args)) == pkv.PKV_ERR_INVALID_ARG
    pkv.pkv_sched_extend(s, a, 169)
    child = pkv.pkv_sched_fork(s, a, 100, 5)[0]      # shares the holes
    assert (_table(s, child)[:, 2:4] == -1).all()
    # a partial page that is gone cannot be copied
    assert _status(lambda: pkv.pkv_sched_fork(s, a, 40, 5)) == pkv.PKV_ERR_INVALID_ARG
    pkv.pkv_sched_finish(s, a)
    pkv.pkv_sched_finish(s, child)
    st = pkv.pkv_sched_get_stats(s)
    assert st["free_pages"] == st["free_credits"] == 64


def test_compaction_moves_high_pages_down(lib):
    s = _sched(lib, 64)
    a, b, c = (_start(s, 48, 1) for _ in range(3))   # pages 0-5, 6-11, 12-17
    child = pkv.pkv_sched_fork(s, c, 48, 1)[0]
    pkv.pkv_sched_finish(s, a)
    old = {i: _table(s, i) for i in (b, c, child)}
    src, dst = pkv.pkv_sched_compact(s, max_moves=2)
    assert src.tolist() == [17, 16] and dst.tolist() == [0, 1]
    src2, dst2 = pkv.pkv_sched_compact(s)
    assert src2.tolist() == [15, 14, 13, 12] and dst2.tolist() == [2, 3, 4, 5]
    to = dict(zip(np.concatenate([src, src2]).tolist(), np.concatenate([dst, dst2]).tolist()))
    for i in (b, c, child):
        assert _table(s, i).tolist() == [[to.get(p, p) for p in row] for row in old[i].tolist()]
    assert [len(x) for x in pkv.pkv_sched_compact(s)] == [0, 0]
    assert _status(lambda: pkv.pkv_sched_compact(s, max_moves=-1)) == pkv.PKV_ERR_INVALID_ARG
    i = _start(s, 16, 1)
    assert sorted(_table(s, i)[:, 0].tolist()) == [12, 13]


def test_random_operations_keep_owners_and_credits(lib):
    rng = np.random.RandomState(5)
    pages, layers = 90, 2
    s = _sched(lib, pages, layers)
    model = {}        # id -> dict(tab=[layers][...], len, prefix, budget)

    def check():
        owned = set()
        for i, r in model.items():
            t = _table(s, i)
            assert (t[:, :r["n"]] == r["tab"]).all() and (t[:, r["n"]:] == -1).all()
            owned |= set(t[t >= 0].tolist())
        st = pkv.pkv_sched_get_stats(s)
        assert st["free_pages"] == pages - len(owned)
        assert st["free_credits"] == pages - sum(r["budget"] for r in model.values()) >= 0
        for r in model.values():    # each can still get what it reserved
            assert (r["tab"] >= 0).sum() <= r["budget"]

    for step in range(600):
        op = rng.randint(6)
        if op == 0:
            p, n = rng.randint(1, 100), rng.randint(1, 60)
            allowed, prefix, budget = pkv.pkv_sched_budget(p, n, num_layers=layers, max_seq_len=256)
            if budget <= pkv.pkv_sched_get_stats(s)["free_credits"]:
                i = _start(s, p, n)
                k = -(-p // 16)
                model[i] = dict(tab=_table(s, i)[:, :k].copy(), n=k, len=p, prefix=prefix,
                                budget=budget)
        elif model:
            i = list(model)[rng.randint(len(model))]
            r = model[i]
            if op == 1:
                r["len"] = min(r["prefix"], r["len"] + rng.randint(1, 30))
                pkv.pkv_sched_extend(s, i, r["len"])
                k = max(r["n"], -(-r["len"] // 16))
                new = _table(s, i)[:, :k].copy()
                assert (new[:, :r["n"]] == r["tab"]).all() and (new[:, r["n"]:] >= 0).all()
                r["tab"], r["n"] = new, k
            elif op == 2:
                length, n = rng.randint(1, r["len"] + 1), rng.randint(1, 40)
                shared, part = length // 16, length % 16
                budget = pkv.pkv_sched_budget(length, n, num_layers=layers, max_seq_len=256)
                holes = int((r["tab"][:, :shared] < 0).sum())
                want = budget[2] - holes
                if part and (r["tab"][:, shared] < 0).any():
                    assert _status(lambda: pkv.pkv_sched_fork(s, i, length, n)) == 1
                elif want > pkv.pkv_sched_get_stats(s)["free_credits"]:
                    assert _status(lambda: pkv.pkv_sched_fork(s, i, length, n)) == 7
                else:
                    c, src, dst, tok = pkv.pkv_sched_fork(s, i, length, n)
                    k = shared + (1 if part else 0)
                    tab = _table(s, c)[:, :k].copy()
                    assert (tab[:, :shared] == r["tab"][:, :shared]).all()
                    if part:
                        assert dst.tolist() == tab[:, shared].tolist()
                        assert src.tolist() == r["tab"][:, shared].tolist()
                        assert not set(dst.tolist()) & {int(p) for m in model.values()
                                                        for p in m["tab"].ravel()}
                    model[c] = dict(tab=tab, n=k, len=length, prefix=budget[1], budget=want)
            elif op == 3:
                first, sinks = rng.randint(0, r["len"] + 1), rng.randint(0, 40)
                n = pkv.pkv_sched_release(s, i, first, sinks)
                lo, hi = -(-sinks // 16), first // 16
                gone = r["tab"][:, lo:hi] if hi > lo else r["tab"][:, :0]
                assert n == int((gone >= 0).sum())
                gone[:] = -1
                r["budget"] -= n
            elif op == 4:
                src, dst = pkv.pkv_sched_compact(s, max_moves=rng.randint(0, 20))
                to = dict(zip(src.tolist(), dst.tolist()))
                assert not set(src.tolist()) & set(dst.tolist())
                for m in model.values():
                    m["tab"] = np.array([[to.get(int(p), int(p)) for p in row]
                                         for row in m["tab"]], np.int32).reshape(m["tab"].shape)
            elif op == 5 and rng.rand() < 0.6:
                pkv.pkv_sched_finish(s, i)
                del model[i]
        check()


def test_values_beyond_a_c_int(lib):
    """A sink count beyond an int keeps every token, as attention reads it; ids,
    lengths and counts beyond one are refused, not wrapped."""
    s = _sched(lib, 64)
    a = _start(s, 150, 20)
    t, before = _table(s, a), pkv.pkv_sched_get_stats(s)
    big = 2 ** 32      # wraps to small C ints: 2^32 + 5 must not become 5
    for sinks in (2 ** 31 - 1, 2 ** 31, big, big + 20, 1 << 40):
        assert pkv.pkv_sched_release(s, a, 128, sinks) == 0
    for args in ((a, big + 128, 0), (a, 128 - big, 0), (a + big, 128, 0), (a - big, 128, 0),
                 (a, 128, 3 - big), (a, 2 ** 31, 0)):
        assert _status(lambda: pkv.pkv_sched_release(s, *args)) == pkv.PKV_ERR_INVALID_ARG
    for args in ((a, big + 144, 5), (a, 144 - big, 5), (a + big, 144, 5), (a, 144, big + 5),
                 (a, 144, 5 - big)):
        assert _status(lambda: pkv.pkv_sched_fork(s, *args)) == pkv.PKV_ERR_INVALID_ARG
    for moves in (-1, -big, 5 - big):
        assert _status(lambda: pkv.pkv_sched_compact(s, max_moves=moves)) == \
            pkv.PKV_ERR_INVALID_ARG
    assert [len(x) for x in pkv.pkv_sched_compact(s, max_moves=1 << 40)] == [0, 0]
    assert (_table(s, a) == t).all() and pkv.pkv_sched_get_stats(s) == before


def test_what_a_request_still_holds(lib):
    """A fork inherits its parent's holes; what it lacks can be asked for before the
    first step behind a window."""
    s = _sched(lib, 128)
    a = _start(s, 200, 5)
    assert pkv.pkv_sched_held(s, a) == (200, 0)
    whole = pkv.pkv_sched_fork(s, a, 37, 5)[0]
    assert pkv.pkv_sched_held(s, whole) == (37, 0)
    pkv.pkv_sched_release(s, a, 160, 20)              # pages 2 .. 9 go
    assert pkv.pkv_sched_held(s, a) == (32, 160)
    assert pkv.pkv_sched_held(s, pkv.pkv_sched_fork(s, a, 170, 5)[0]) == (32, 160)
    assert pkv.pkv_sched_held(s, pkv.pkv_sched_fork(s, a, 96, 5)[0]) == (32, 96)
    assert pkv.pkv_sched_held(s, pkv.pkv_sched_fork(s, a, 32, 5)[0]) == (32, 0)
    pkv.pkv_sched_release(s, a, 160, 0)
    none = pkv.pkv_sched_fork(s, a, 160, 5)[0]        # nothing of it is there
    assert pkv.pkv_sched_held(s, none) == (0, 160) and (_table(s, none) == -1).all()
    pkv.pkv_sched_extend(s, none, 164)
    assert pkv.pkv_sched_held(s, none) == (0, 160)
    assert pkv.pkv_sched_held(s, whole) == (37, 0)    # a release by the parent is not its
    b = pkv.pkv_sched_submit(s, 10, 5)
    for i in (b, b + 1, -1, 2 ** 32 + a):             # waiting, unknown, not wrapped
        assert _status(lambda: pkv.pkv_sched_held(s, i)) == pkv.PKV_ERR_INVALID_ARG
    assert pkv.pkv_sched_admit(s) == [b]
    assert pkv.pkv_sched_held(s, b) == (0, 0)         # no position reached yet


def test_held_positions_under_random_releases(lib):
    """Against the block table, entry by entry."""
    rng = np.random.RandomState(11)
    s = _sched(lib, 4000, 3)
    for _ in range(60):
        n = rng.randint(1, 250)
        a = _start(s, n, 5)
        for _ in range(rng.randint(0, 4)):
            pkv.pkv_sched_release(s, a, rng.randint(0, n + 1), rng.randint(0, 200))
        if rng.rand() < 0.5:
            length = rng.randint(1, n + 1)
            try:
                a, n = pkv.pkv_sched_fork(s, a, length, 5)[0], length
            except pkv.PkvError:                      # its partial page is gone
                pass
        there = (_table(s, a) >= 0).all(0).repeat(16)[:n]
        head, tail = pkv.pkv_sched_held(s, a)
        assert there[:head].all() and (head == n or not there[head])
        assert there[tail:].all() and (tail == 0 or not there[tail - 1])
