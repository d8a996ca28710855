"""Prefill fill with rotation by several position axes: queries and stored keys
bit for bit against FP32 with every product and sum rounded, values copied,
nothing else written."""

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
import window_helpers as W

pytestmark = pytest.mark.gpu

SECTIONS = {1: [0] * 32, 2: [0] * 16 + [1] * 16, 3: [0] * 8 + [1] * 12 + [2] * 12,
            4: [(5 * i) % 4 for i in range(32)]}


def _bits(t):
    return t.view(torch.int16)


def _fill(chunks, starts, axes=3, in_place=False, queries=True, max_seq_len=2048, seed=0,
          rows=3000, extra=0, max_chunk=None, **kw):
    lens = [s + n if n else 0 for s, n in zip(starts, chunks)]
    c = W.Cache(lens, max_seq_len, seed, evict=lambda b: np.arange(-(-lens[b] // 16)) < starts[b] // 16,
                **kw)
    kp, vp = c.pools(lambda b: np.zeros(lens[b], bool), 3.0)
    total = sum(chunks)
    g = c.gen
    q = torch.randn(total, 32, 64, generator=g, device="cuda").bfloat16()
    k = torch.randn(total, 8, 64, generator=g, device="cuda").bfloat16()
    v = torch.randn(total, 8, 64, generator=g, device="cuda").bfloat16()
    pos = torch.randint(0, rows, (axes, total + extra), generator=g, device="cuda").int()
    cos, sin = W.angles(rows)
    rope = pkv.pkv_axes_rope(cos, sin, SECTIONS[axes])
    cu = torch.tensor(np.concatenate([[0], np.cumsum(chunks)]), dtype=torch.int32, device="cuda")
    start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    want_k, want_v = kp.clone(), vp.clone()
    rk = W.rotate(k, cos, sin, pos[:, :total], SECTIONS[axes], torch.float32).bfloat16()
    rq = W.rotate(q, cos, sin, pos[:, :total], SECTIONS[axes], torch.float32).bfloat16()
    row = 0
    for b, n in enumerate(chunks):
        for i in range(n):
            p = starts[b] + i
            page = int(c.table[c.layer, b, p // 16])
            want_k[page, :, p % 16], want_v[page, :, p % 16] = rk[row], v[row]
            row += 1
    pool = pkv.pkv_pool_create(c.num_layers, c.num_pages, c.max_batch, max_seq_len=max_seq_len,
                               flags=pkv.PKV_FLAG_LONG_CONTEXT)
    out = None if not queries else q if in_place else torch.full_like(q, 7.5)
    pkv.pkv_prefill_fill_axes(pool, c.layer, q if queries else None, k, v, out, kp, vp, c.tables,
                              cu, start, rope, pos, max_chunk or max(chunks))
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    pool.close()
    if queries:
        assert torch.equal(_bits(out), _bits(rq))
    assert torch.equal(_bits(kp), _bits(want_k)) and torch.equal(_bits(vp), _bits(want_v))


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("in_place", [False, True])
def test_ragged_chunks(axes, in_place):
    _fill([1, 17, 0, 64, 100, 9], [0, 3, 0, 16, 1900, 31], axes, in_place, seed=axes)


def test_keys_and_values_only():
    _fill([40, 3], [0, 5], queries=False)


def test_wider_launch_position_rows_and_tables():
    _fill([5, 33], [100, 0], extra=7, max_chunk=2048, num_layers=3, layer=1, max_batch=4)


def test_long_context():
    _fill([50, 20], [65000, 40001], max_seq_len=65536)


def test_pages_past_four_gib():
    _fill([50], [0], base_page=280000)


def test_single_axis_agrees_with_the_decode_append():
    """One axis is the rotation of pkv_append_rope, bit for bit."""
    n = 33
    c = W.Cache([n])
    cos, sin = W.angles(2048)
    k = torch.randn(n, 8, 64, device="cuda").bfloat16()
    pool = pkv.pkv_pool_create(1, c.num_pages, 1)
    a = [torch.zeros(c.num_pages, 8, 16, 64, device="cuda").bfloat16() for _ in range(4)]
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")[None].contiguous()
    pkv.pkv_prefill_fill_axes(pool, 0, None, k, k, None, a[0], a[1], c.tables, cu, zero,
                              pkv.pkv_axes_rope(cos, sin, [0] * 32), pos, n)
    for i in range(n):
        at = torch.tensor([i], dtype=torch.int32, device="cuda")
        pkv.pkv_append_rope(pool, 0, k[i:i + 1], k[i:i + 1], a[2], a[3], c.tables, at, cos, sin)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert torch.equal(_bits(a[0]), _bits(a[2])) and torch.equal(_bits(a[1]), _bits(a[3]))
    pool.close()


def test_flags_bad_data_and_refusals():
    c = W.Cache([40, 40])
    kp, vp = c.pools(lambda b: np.zeros(40, bool), 3.0)
    was = kp.clone()
    pool = pkv.pkv_pool_create(1, c.num_pages, 2)
    q = torch.randn(80, 32, 64, device="cuda").bfloat16()
    k = torch.randn(80, 8, 64, device="cuda").bfloat16()
    cos, sin = W.angles(50)
    rope = pkv.pkv_axes_rope(cos, sin, SECTIONS[2])
    pos = torch.zeros(2, 80, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40, 80], dtype=torch.int32, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")

    def run(cu_=cu, start_=start, tables=c.tables, pos_=pos, chunk=40, rope_=rope, total=None,
            layer=0, batch=None):
        out = torch.full_like(q, 7.5)
        pkv.pkv_prefill_fill_axes(pool, layer, q, k, k, out, kp, vp, tables, cu_, start_, rope_,
                                  pos_, chunk, total_tokens=total, batch=batch)
        return out, pkv.pkv_get_error(pool)

    for bad in (-1, 50, 2 ** 31 - 1):
        p = pos.clone()
        p[1, 7] = bad
        out, st = run(pos_=p)
        assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[7] == 7.5).all()
        assert torch.equal(kp[int(c.table[0, 0, 0]), :, 7], was[int(c.table[0, 0, 0]), :, 7])
        assert not (out[8] == 7.5).any()
    for bad in (-1, 2030, 2 ** 31 - 1):
        s = start.clone()
        s[1] = bad
        out, st = run(start_=s)
        assert st == pkv.PKV_ERR_OUT_OF_RANGE and not (out[:40] == 7.5).all(-1).any()
    t = c.tables.clone()
    t[0, 1, 0] = c.num_pages
    out, st = run(tables=t)
    assert st == pkv.PKV_ERR_OUT_OF_RANGE and (out[40:56] == 7.5).all()
    assert run(cu_=torch.tensor([0, 40, 81], dtype=torch.int32, device="cuda"))[1] == \
        pkv.PKV_ERR_OUT_OF_RANGE
    assert run(chunk=16)[1] == pkv.PKV_ERR_OUT_OF_RANGE
    for kw in (dict(chunk=0), dict(chunk=2049), dict(layer=1), dict(batch=-1), dict(total=-1)):
        with pytest.raises(pkv.PkvError) as e:
            run(**kw)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    for kw in (dict(pos_=pos[:, :79].contiguous()), dict(pos_=pos[0]), dict(rope_=None),
               dict(total=81)):
        with pytest.raises(ValueError):
            run(**kw)
    for bad in ([0] * 31, [4] + [0] * 31, [-1] + [0] * 31):
        with pytest.raises(ValueError):
            pkv.pkv_axes_rope(cos, sin, bad)
    assert run()[1] == pkv.PKV_OK
    pool.close()
