"""Handles with contexts past 2,048 tokens: the calls without a context limit of
their own write where they say, bit for bit, and the others refuse before anything
is written."""

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
import window_helpers as W

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.int16)


def _handle(c):
    return pkv.pkv_pool_create(c.num_layers, c.num_pages, c.max_batch, max_seq_len=c.max_seq_len,
                               flags=pkv.PKV_FLAG_LONG_CONTEXT)


def test_whole_prefill_refuses_before_it_fills():
    c = W.Cache([40], max_seq_len=4096)
    kp, vp = c.pools(lambda b: np.zeros(40, bool), 3.0)
    was = kp.clone(), vp.clone()
    pool = _handle(c)
    q = torch.randn(40, 32, 64, device="cuda").bfloat16()
    k = torch.randn(40, 8, 64, device="cuda").bfloat16()
    out = torch.full((40, 32, 64), 7.5, device="cuda")
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    start = torch.zeros(4, dtype=torch.int32, device="cuda")[:1]
    with pytest.raises(pkv.PkvError) as e:
        pkv.pkv_prefill(pool, 0, q, k, k, kp, vp, c.tables, cu, start, out, 40)
    assert e.value.status == pkv.PKV_ERR_UNSUPPORTED
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert torch.equal(_bits(kp), _bits(was[0])) and torch.equal(_bits(vp), _bits(was[1]))
    assert (out == 7.5).all()
    pool.close()


# the last position of the short context, the ones around it, and the last one there is
POSITIONS = [0, 5, 2046, 2047, 2048, 2063, 2064, 40001, 65535]


def _far(positions, max_seq_len=65536):
    """A cache with only the pages of `positions`, one sequence each, in layer 1 of 2."""
    lens = [p + 1 for p in positions]
    c = W.Cache(lens, max_seq_len, evict=lambda b: np.arange(-(-lens[b] // 16)) <
                positions[b] // 16, num_layers=2, layer=1)
    kp, vp = c.pools(lambda b: np.zeros(lens[b], bool), 3.0)
    return c, kp, vp


@pytest.mark.parametrize("rotated", [False, True])
def test_append(rotated):
    c, kp, vp = _far(POSITIONS)
    n = len(POSITIONS)
    k = torch.randn(n, 8, 64, device="cuda").bfloat16()
    v = torch.randn(n, 8, 64, device="cuda").bfloat16()
    at = torch.zeros(12, dtype=torch.int32, device="cuda")[:n]
    at.copy_(torch.tensor(POSITIONS, dtype=torch.int32))
    cos, sin = W.angles(65536)
    stored = W.rotate(k, cos, sin, at[None], [0] * 32, torch.float32).bfloat16() if rotated else k
    want_k, want_v = kp.clone(), vp.clone()
    for b, p in enumerate(POSITIONS):
        page = int(c.table[1, b, p // 16])
        want_k[page, :, p % 16], want_v[page, :, p % 16] = stored[b], v[b]
    pool = _handle(c)

    def run(positions):
        if rotated:
            pkv.pkv_append_rope(pool, 1, k, v, kp, vp, c.tables, positions, cos, sin)
        else:
            pkv.pkv_append(pool, 1, k, v, kp, vp, c.tables, positions)
        return pkv.pkv_get_error(pool)
    assert run(at) == pkv.PKV_OK
    assert torch.equal(_bits(kp), _bits(want_k)) and torch.equal(_bits(vp), _bits(want_v))
    for bad in (65536, -1, 2 ** 31 - 1):             # skipped and flagged, the others as before
        wrong = at.clone()
        wrong[7] = bad
        assert run(wrong) == pkv.PKV_ERR_OUT_OF_RANGE
        assert torch.equal(_bits(kp), _bits(want_k)) and torch.equal(_bits(vp), _bits(want_v))
    pool.close()


def test_prefill_fill_and_the_windowed_calls_after_it():
    """Chunks that cross position 2,048 and that end the context, filled without rotation,
    attended to, and decoded on."""
    chunks, starts = [40, 33, 100], [2030, 60000, 65436]
    lens = [s + n for s, n in zip(starts, chunks)]
    window = 70
    c = W.Cache(lens, 65536, evict=lambda b: np.arange(-(-lens[b] // 16)) <
                max(0, starts[b] - window) // 16, num_layers=2, layer=1)
    kp, vp = c.pools(lambda b: np.arange(lens[b]) < 0, 0.0)
    total = sum(chunks)
    cu = np.concatenate([[0], np.cumsum(chunks)])
    cu_t = torch.zeros(8, dtype=torch.int32, device="cuda")[:4]
    cu_t.copy_(torch.tensor(cu, dtype=torch.int32))
    start = torch.zeros(4, dtype=torch.int32, device="cuda")[:3]
    start.copy_(torch.tensor(starts, dtype=torch.int32))
    k = torch.cat([c.k[b][starts[b]:] for b in range(3)])
    v = torch.cat([c.v[b][starts[b]:] for b in range(3)])
    want_k, want_v = kp.clone(), vp.clone()
    for b, n in enumerate(chunks):                   # tokens before the chunks hold zeros
        c.k[b][:starts[b]], c.v[b][:starts[b]] = 0, 0
        for i in range(n):
            p = starts[b] + i
            page = int(c.table[1, b, p // 16])
            want_k[page, :, p % 16], want_v[page, :, p % 16] = k[cu[b] + i], v[cu[b] + i]
    pool = _handle(c)
    pkv.pkv_prefill_fill(pool, 1, k, v, kp, vp, c.tables, cu_t, start, 100)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert torch.equal(_bits(kp), _bits(want_k)) and torch.equal(_bits(vp), _bits(want_v))
    q = torch.randn(total, 32, 64, device="cuda", generator=c.gen).bfloat16()
    out, one = torch.zeros(total, 32, 64, device="cuda"), torch.zeros(3, 32, 64, device="cuda")
    pkv.pkv_window_prefill_attention(pool, 1, q, kp, vp, c.tables, cu_t, start, out, 100, window)
    last = q[cu[1:] - 1].contiguous()
    pkv.pkv_window_attention(pool, 1, last, kp, vp, c.tables, c.lens_tensor(), one, window)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    for b in range(3):
        at = torch.arange(starts[b], lens[b], device="cuda")
        ref, tol = W.attend(q[cu[b]:cu[b + 1]].double(), c.k[b].double(), c.v[b].double(), at,
                            window, 0)
        W.check(out[cu[b]:cu[b + 1]], ref, tol, f"chunk {b}")
        W.check(one[b:b + 1], ref[-1:], tol[-1:], f"decode {b}")
    wrong = start.clone()
    wrong[2] = 65437                                 # its last token would lie past the context
    pkv.pkv_prefill_fill(pool, 1, k, v, kp, vp, c.tables, cu_t, wrong, 100)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    pool.close()
