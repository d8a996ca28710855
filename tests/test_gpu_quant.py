"""The 8-bit cache on the GPU: fill, read-back and decode attention against a
64-bit restatement of the documented tiles."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_210_gb300 as pkv
from quant_helpers import LARGEST, TILE, QuantCache, attend, grid, places, put, quantise
from window_helpers import DIM, HKV, HQ, PAGE, angles, check, rotate, unseen_pages

pytestmark = pytest.mark.gpu

AXES = {1: [0] * 32, 2: [0, 1] * 16, 3: [0] * 8 + [1] * 12 + [2] * 12}


@pytest.fixture(autouse=True, scope="module")
def _library():
    from paged_kv_cache_210_gb300 import build as lib_build
    lib_build.build()


def handle(c, flags=0, max_splits=0):
    if c.max_seq_len > 2048:
        flags |= pkv.PKV_FLAG_LONG_CONTEXT
    return pkv.pkv_pool_create(c.num_layers, c.num_pages, c.max_batch, max_seq_len=c.max_seq_len,
                               max_splits=max_splits, flags=flags)


def normal(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16().cuda()


def int32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


# ---------------------------------------------------------------- fill and read-back
def expected_fill(c, before, starts, counts, k, v, skip=()):
    """The pool's bytes after a fill of the packed rows k, v (float64 values on the CPU)."""
    out = before.copy()
    row = 0
    for b, (s, n) in enumerate(zip(starts, counts)):
        t = np.arange(s, s + n)
        keep = np.array([row + i not in skip for i in range(n)], bool) if n else np.zeros(0, bool)
        page = c.table[c.layer, b, t // PAGE] if n else t
        for which, x in enumerate((k, v)):
            codes, exps, _ = quantise(x[row:row + n])
            put(out, page[keep], t[keep] % PAGE, which, codes.numpy()[keep], exps.numpy()[keep])
        row += n
    return out


@pytest.mark.parametrize("starts,counts", [
    ([0], [1]), ([15], [1]), ([3], [77]), ([0, 5, 31], [16, 0, 33]), ([2047], [1]),
    ([7, 0, 100, 16], [9, 2048, 1, 48])])
def test_fill_writes_the_documented_bytes_and_nothing_else(starts, counts):
    c = QuantCache([s + n for s, n in zip(starts, counts)], seed=sum(counts), num_layers=2, layer=1)
    pool, kv = handle(c), c.pool()
    total = sum(counts)
    k, v = normal(1, total, HKV, DIM, scale=3.0), normal(2, total, HKV, DIM, scale=0.01)
    cu = int32(np.cumsum([0] + counts))
    pkv.pkv_quant_fill(pool, 1, k, v, kv, c.tables, cu, int32(starts), max(max(counts), 1))
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    want = expected_fill(c, c.bytes, starts, counts, k.double().cpu(), v.double().cpu())
    assert np.array_equal(kv.cpu().numpy(), want)
    # and back: what the codes stand for, rows past the last left alone
    kb = torch.full((total + 2, HKV, DIM), 7.0, dtype=torch.bfloat16, device="cuda")
    vb = kb.clone()
    pkv.pkv_quant_read(pool, 1, kv, c.tables, cu, int32(starts), kb, vb, max(max(counts), 1))
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    for got, x in ((kb, k), (vb, v)):
        assert torch.equal(got[:total].double().cpu(), quantise(x.double().cpu())[2])
        assert bool((got[total:] == 7.0).all())


@pytest.mark.parametrize("axes", [1, 2, 3])
def test_rotated_fill_quantises_the_fp32_rotation(axes):
    starts, counts = [5, 0, 30], [40, 16, 3]
    c = QuantCache([s + n for s, n in zip(starts, counts)], seed=axes)
    pool, kv = handle(c), c.pool()
    total = sum(counts)
    k, v = normal(1, total, HKV, DIM), normal(2, total, HKV, DIM)
    cos, sin = angles(500)
    pos = torch.randint(0, 500, (axes, total + 3), dtype=torch.int32, device="cuda")
    rope = pkv.pkv_axes_rope(cos, sin, AXES[axes])
    pkv.pkv_quant_fill(pool, 0, k, v, kv, c.tables, int32(np.cumsum([0] + counts)), int32(starts),
                       64, rope=rope, rope_positions=pos)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    turned = rotate(k, cos, sin, pos[:, :total], AXES[axes], torch.float32)
    want = expected_fill(c, c.bytes, starts, counts, turned.double().cpu(), v.double().cpu())
    assert np.array_equal(kv.cpu().numpy(), want)


@pytest.mark.parametrize("chunk", [16384, 4000, 1])
def test_rotated_codes_of_many_tokens(chunk):
    # products and sum each rounded in FP32: a fused multiply-add would change about one
    # code in a million (8 million here; the last case takes the fused append, 2 million)
    total = 16384 if chunk > 1 else 4096
    c = QuantCache([0] * (total if chunk == 1 else 1), max_seq_len=16 if chunk == 1 else 16384,
                   spare=total // (1 if chunk == 1 else PAGE))
    pages = c.table.shape[2]
    c.tables = torch.randperm(c.num_pages, dtype=torch.int32)[:c.table.size].view(c.table.shape).cuda()
    assert c.tables.numel() == c.num_pages and pages * PAGE == c.max_seq_len
    pool, kv = handle(c), c.pool()
    k = normal(1, total, HKV, DIM)
    cos, sin = angles(20000)
    pos = torch.randint(0, 20000, (3, total), dtype=torch.int32, device="cuda")
    rope = pkv.pkv_axes_rope(cos, sin, AXES[3])
    kb, vb = torch.empty_like(k), torch.empty_like(k)
    if chunk > 1:
        for at in range(0, total, chunk):
            n = min(chunk, total - at)
            pkv.pkv_quant_fill(pool, 0, k[at:at + n], k[at:at + n], kv, c.tables, int32([0, n]),
                               int32([at]), n, rope=rope, rope_positions=pos[:, at:at + n].contiguous())
        cu, start, most = int32([0, total]), int32([0]), total
    else:
        q, out = normal(2, total, HQ, DIM), torch.empty(total, HQ, DIM, device="cuda")
        pkv.pkv_quant_append_attend(pool, 0, q, k, k, kv, c.tables, int32([1] * total), out, 16,
                                    rope=rope, rope_positions=pos)
        cu, start, most = int32(np.arange(total + 1)), int32([0] * total), 1
    pkv.pkv_quant_read(pool, 0, kv, c.tables, cu, start, kb, vb, most)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    turned = rotate(k, cos, sin, pos, AXES[3], torch.float32).double().cpu()
    assert int((kb.double().cpu() != quantise(turned)[2]).sum()) == 0
    assert torch.equal(vb.double().cpu(), quantise(k.double().cpu())[2])


def special_rows():
    """Rows at the edges of the rule: zeros, powers of two, 448 and its neighbours
    times powers, ties, subnormals, the largest values, one large among small."""
    rows = [np.zeros(64)]
    for e in (-133, -126, -30, -1, 0, 9, 60, 119, 127):
        rows.append(np.full(64, 2.0 ** e))
    for s in (2.0 ** -140, 2.0 ** -10, 1.0, 2.0 ** 100):
        for m in (446.0, 448.0, 450.0, 447.0):
            rows.append(np.linspace(-m, m, 64) * s)
    ties = np.concatenate([np.arange(16) * 2.0 + 17, np.arange(16) / 1024, np.arange(32) * 8 + 132])
    rows += [ties, -ties, np.where(np.arange(64) == 5, 448.0, ties / 64)]
    top = torch.finfo(torch.bfloat16).max
    rows += [np.full(64, top), np.where(np.arange(64) % 2, top, -1.0), np.full(64, LARGEST)]
    rows += [np.where(np.arange(64) == 63, 1e30, 1e-30)]
    return torch.tensor(np.stack(rows)).to(torch.bfloat16)


def test_extreme_rows():
    x = special_rows()
    n = x.shape[0]
    c = QuantCache([n])
    pool, kv = handle(c), c.pool()
    k = x[:, None].repeat(1, HKV, 1).cuda().contiguous()
    v = k.flip(0).contiguous()
    cu, start = int32([0, n]), int32([0])
    pkv.pkv_quant_fill(pool, 0, k, v, kv, c.tables, cu, start, n)
    want = expected_fill(c, c.bytes, [0], [n], k.double().cpu(), v.double().cpu())
    assert np.array_equal(kv.cpu().numpy(), want)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    pkv.pkv_quant_read(pool, 0, kv, c.tables, cu, start, kb, vb, n)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert torch.equal(kb.double().cpu(), quantise(k.double().cpu())[2])
    assert bool(torch.isfinite(vb).all())
    # half a step: 2^-4 of the value, or 2^-10 of the row's power of two
    e = (quantise(k.double().cpu())[1].double() - 127)[..., None]
    clamped = k.double().cpu().clamp(-LARGEST, LARGEST)
    off = (kb.double().cpu() - clamped).abs()
    assert bool((off <= torch.maximum(clamped.abs() * 2.0 ** -4, 2.0 ** (e - 10))).all())


def test_nan_and_infinity():
    n = 3
    c = QuantCache([n])
    pool, kv = handle(c), c.pool()
    k = normal(1, n, HKV, DIM)
    k[0, 0, 3], k[1, 2, 5], k[2, :, :] = math.nan, math.inf, math.nan
    v = -k
    cu, start = int32([0, n]), int32([0])
    pkv.pkv_quant_fill(pool, 0, k, v, kv, c.tables, cu, start, n)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    pkv.pkv_quant_read(pool, 0, kv, c.tables, cu, start, kb, vb, n)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    for got, x in ((kb, k), (vb, v)):
        got, x = got.double().cpu(), x.double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(x))
        want = quantise(x)[2]
        assert torch.equal(got[~torch.isnan(x)], want[~torch.isnan(x)])


def test_every_code_and_exponent_reads_back_exactly():
    c = QuantCache([256], spare=0)
    pool = handle(c)
    at_k, at_v = places()
    raw = c.bytes.copy()
    codes = np.arange(256, dtype=np.uint8)
    for b in range(256):                     # token b: codes b, b + 1, ..; exponents over the range
        page, slot = c.table[0, 0, b // PAGE], b % PAGE
        for h in range(HKV):
            row = codes[(b + np.arange(64) * 4 + h) % 256]
            row = np.where(row % 128 == 127, 0, row)
            raw[page, h, at_k[slot]] = row
            raw[page, h, at_v[slot]] = row[::-1]
            raw[page, h, 2048 + slot] = 3 + (b * 8 + h) % 244
            raw[page, h, 2064 + slot] = 246 - (b * 8 + h) % 244
    kv = torch.from_numpy(raw).cuda()
    kb = torch.empty(256, HKV, DIM, dtype=torch.bfloat16, device="cuda")
    vb = torch.empty_like(kb)
    pkv.pkv_quant_read(pool, 0, kv, c.tables, int32([0, 256]), int32([0]), kb, vb, 256)
    g = grid().numpy()
    for b in range(0, 256, 5):
        page, slot = c.table[0, 0, b // PAGE], b % PAGE
        for h in range(HKV):
            for got, at, e in ((kb, at_k, 2048), (vb, at_v, 2064)):
                want = g[raw[page, h, at[slot]]] * 2.0 ** (int(raw[page, h, e + slot]) - 127.0)
                assert np.array_equal(got[b, h].double().cpu().numpy(), want)


def test_what_is_skipped_is_flagged_and_left_alone():
    starts, counts = [0, 2040, -1, 10, 40], [20, 16, 4, 30, 3]
    c = QuantCache([20, 2048, 4, 40, 43], seed=3)
    c.table[0, 0, 1] = c.num_pages                       # an id past the pool
    c.table[0, 3, 1] = -1                                # a missing page
    tables = torch.from_numpy(c.table).cuda()
    total = sum(counts)
    k, v = normal(1, total, HKV, DIM), normal(2, total, HKV, DIM)
    cu = int32(np.cumsum([0] + counts))
    # what is left: tokens 0..15 of the first, the 8 that fit of the second, none of the
    # third, 10..15 and 32..39 of the fourth, all of the fifth
    skip = set(range(16, 20)) | set(range(28, 36)) | set(range(36, 40)) | set(range(46, 62))
    pool, kv = handle(c), c.pool()
    pkv.pkv_quant_fill(pool, 0, k, v, kv, tables, cu, int32(starts), 40)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    want = c.bytes.copy()
    row = 0
    kc, vc = quantise(k.double().cpu()), quantise(v.double().cpu())
    for b, (s, n) in enumerate(zip(starts, counts)):
        for i in range(n):
            if row + i not in skip:
                t = s + i
                for which, x in enumerate((kc, vc)):
                    put(want, [c.table[0, b, t // PAGE]], [t % PAGE], which,
                        x[0].numpy()[row + i:row + i + 1], x[1].numpy()[row + i:row + i + 1])
        row += n
    assert np.array_equal(kv.cpu().numpy(), want)
    kb = torch.full((total, HKV, DIM), 9.0, dtype=torch.bfloat16, device="cuda")
    vb = kb.clone()
    pkv.pkv_quant_read(pool, 0, kv, tables, cu, int32(starts), kb, vb, 40)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    for r in range(total):
        for got, x in ((kb, kc), (vb, vc)):
            if r in skip:
                assert bool((got[r] == 9.0).all()), r
            else:
                assert torch.equal(got[r].double().cpu(), x[2][r]), r
    # rotary positions outside the tables: that token alone
    cos, sin = angles(100)
    pos = torch.zeros(1, total, dtype=torch.int32, device="cuda")
    pos[0, 2], pos[0, 5] = 100, -1
    kv2 = c.pool()
    pkv.pkv_quant_fill(pool, 0, k, v, kv2, tables, cu, int32(starts), 40,
                       rope=pkv.pkv_axes_rope(cos, sin, AXES[1]), rope_positions=pos)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    page = c.table[0, 0, 0]
    got, was = kv2.cpu().numpy(), c.bytes
    at_k, at_v = places()
    for t in range(16):
        same = np.array_equal(got[page][:, at_k[t]], was[page][:, at_k[t]]) and \
            np.array_equal(got[page][:, at_v[t]], was[page][:, at_v[t]])
        assert same == (t in (2, 5)), t


@pytest.mark.parametrize("cu,total,most", [([0, 5, 4], 5, 8), ([0, 3, 9], 8, 8), ([-1, 3, 8], 8, 8),
                                           ([0, 8, 8], 8, 5)])
def test_bad_row_lists_are_flagged(cu, total, most):
    c = QuantCache([16, 16])
    pool, kv = handle(c), c.pool()
    k = normal(1, total, HKV, DIM)
    pkv.pkv_quant_fill(pool, 0, k, k, kv, c.tables, int32(cu), int32([0, 0]), most)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    kb = torch.empty_like(k)
    pkv.pkv_quant_read(pool, 0, kv, c.tables, int32(cu), int32([0, 0]), kb, kb.clone(), most)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE


# ---------------------------------------------------------------- decode
def run_decode(c, window, sinks, axes=0, fused=False, splits=0, seed=0, flags=0, q_scale=1.0,
               pool=None, kv=None):
    batch = len(c.lens)
    pool = pool or handle(c, flags, max_splits=128 if splits > 64 else 0)
    kv = c.pool() if kv is None else kv
    q = normal(seed + 10, batch, HQ, DIM, scale=q_scale)
    k, v = normal(seed + 11, batch, HKV, DIM), normal(seed + 12, batch, HKV, DIM)
    kw, pos = {}, None
    qd, kd = q.double(), k.double()
    if axes:
        cos, sin = angles(max(c.max_seq_len, 64))
        pos = torch.randint(0, max(c.max_seq_len, 64), (axes, batch), dtype=torch.int32,
                            device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        kw = dict(rope=pkv.pkv_axes_rope(cos, sin, AXES[axes]), rope_positions=pos)
        qd = rotate(q, cos, sin, pos, AXES[axes], torch.float64)
        kd = rotate(k, cos, sin, pos, AXES[axes], torch.float32).double()
    out = torch.full((batch, HQ, DIM), 5.0, device="cuda")
    lens = c.lens_tensor()
    if fused:
        pkv.pkv_quant_append_attend(pool, c.layer, q, k, v, kv, c.tables, lens, out, window,
                                    sinks=sinks, num_splits=splits, **kw)
    else:
        pkv.pkv_quant_attention(pool, c.layer, q, kv, c.tables, lens, out, window, sinks=sinks,
                                num_splits=splits, **kw)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    want_bytes = c.bytes.copy()
    kq, vq = quantise(kd.cpu()), quantise(v.double().cpu())
    for b, n in enumerate(c.lens):
        if n == 0:
            assert bool((out[b] == 5.0).all())
            continue
        ks, vs = c.k[b], c.v[b]
        if fused:
            ks, vs = ks.clone(), vs.clone()
            ks[-1], vs[-1] = kq[2][b].cuda(), vq[2][b].cuda()
            t = n - 1
            page = c.table[c.layer, b, t // PAGE]
            put(want_bytes, [page], [t % PAGE], 0, kq[0].numpy()[b:b + 1], kq[1].numpy()[b:b + 1])
            put(want_bytes, [page], [t % PAGE], 1, vq[0].numpy()[b:b + 1], vq[1].numpy()[b:b + 1])
        ref, tol = attend(qd[b:b + 1], ks, vs, torch.tensor([n - 1], device="cuda"), window, sinks)
        check(out[b:b + 1], ref, tol, f"sequence {b} of length {n}")
    assert np.array_equal(kv.cpu().numpy(), want_bytes)
    return out


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("axes", [0, 3])
@pytest.mark.parametrize("lens,window,sinks", [
    ([1], 1, 0), ([17, 40], 2048, 0), ([2048], 2048, 0), ([0, 16, 1, 0, 15, 33], 7, 2),
    ([500, 2048, 64, 65], 64, 4), ([2048] * 3, 512, 40), ([31, 32, 33, 900], 1, 1)])
def test_decode(lens, window, sinks, axes, fused):
    c = QuantCache(lens, seed=len(lens) + window,
                   evict=lambda b: unseen_pages(lens[b], lens[b] - 1, window, sinks))
    run_decode(c, window, sinks, axes, fused, seed=window)


@pytest.mark.parametrize("splits", [1, 2, 5, 16, 64, 128])
def test_chosen_splits(splits):
    c = QuantCache([700, 3, 2048], seed=splits, num_layers=2, layer=1)
    run_decode(c, 2048, 0, 1, True, splits=splits)


@pytest.mark.parametrize("batch,longest,window", [(40, 1500, 2048), (130, 700, 300), (400, 90, 2048),
                                                  (97, 300, 2048)])
def test_batches(batch, longest, window):
    rng = np.random.RandomState(batch)
    lens = [int(n) for n in rng.randint(0, longest + 1, batch)]
    c = QuantCache(lens, seed=batch)
    run_decode(c, window, 4, 2, True)


@pytest.mark.parametrize("k_scale,q_scale", [(8.0, 4.0), (1e-4, 1e-3), (1e4, 1e-4), (1e-20, 1e18)])
def test_scales(k_scale, q_scale):
    c = QuantCache([300, 45], seed=2, k_scale=k_scale)
    run_decode(c, 2048, 0, 1, False, q_scale=q_scale)


@pytest.mark.parametrize("axes", [0, 1])
@pytest.mark.parametrize("k_scale", [1e34, 1e30, 1e-34])
def test_keys_near_the_ends_of_the_range(k_scale, axes):
    # scores of ordinary size from factors whose product with the other's scaling is not
    c = QuantCache([300, 45], seed=3, k_scale=k_scale)
    run_decode(c, 2048, 0, axes, False, q_scale=2 / k_scale)


@pytest.mark.parametrize("spread", [4, 18, 60])
def test_values_of_very_different_sizes(spread):
    # rows of V from 2^-spread to 2^spread, some zero, in any order
    def sizes(rng, n):
        x = 2.0 ** torch.from_numpy(rng.randint(-spread, spread + 1, n).astype(np.float64))
        return torch.where(torch.from_numpy(rng.rand(n) < 0.1), torch.zeros(n, dtype=torch.float64), x)
    c = QuantCache([800, 17, 2], seed=spread, v_scale=sizes)
    run_decode(c, 2048, 0)


def test_a_large_value_with_a_negligible_weight_costs_no_precision():
    # one token's V is 2^40 times the others', its weight about 2^-60: it enters the
    # output with 2^-20, so the tolerance is that of the other rows
    c = QuantCache([200], seed=9)
    q = torch.ones(1, HQ, DIM, dtype=torch.bfloat16, device="cuda")
    ks = torch.full((200, HKV, DIM), 0.25, dtype=torch.bfloat16)
    ks[20] = -5.0                                        # score -40 against 2
    vs = torch.randn(200, HKV, DIM, generator=torch.Generator().manual_seed(1)).bfloat16()
    vs[20] *= 2.0 ** 40
    pool, kv = handle(c), c.pool()
    pkv.pkv_quant_fill(pool, 0, ks.cuda(), vs.cuda(), kv, c.tables, int32([0, 200]), int32([0]), 200)
    out = torch.empty(1, HQ, DIM, device="cuda")
    pkv.pkv_quant_attention(pool, 0, q, kv, c.tables, c.lens_tensor(), out, 2048)
    k64, v64 = quantise(ks.double())[2].cuda(), quantise(vs.double())[2].cuda()
    ref, tol = attend(q.double(), k64, v64, torch.tensor([199], device="cuda"), 2048, 0)
    small = v64.clone()
    small[20] = 0
    tol = tol / v64.abs().amax() * (small.abs().amax() + 1.0)
    check(out, ref, tol)


def test_padded_batch_and_bad_lengths():
    c = QuantCache([50, 60, 70], seed=4)
    pool, kv = handle(c), c.pool()
    q = normal(1, 3, HQ, DIM)
    out = torch.full((3, HQ, DIM), 5.0, device="cuda")
    pkv.pkv_quant_attention(pool, 0, q, kv, c.tables, int32([50, 2049, -3]), out, 2048)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    assert bool((out[1:] == 5.0).all())
    ref, tol = attend(q[:1].double(), c.k[0], c.v[0], torch.tensor([49], device="cuda"), 2048, 0)
    check(out[:1], ref, tol)


def test_invalid_pages_are_left_out():
    c = QuantCache([100], seed=5)
    c.table[0, 0, 2], c.table[0, 0, 6] = c.num_pages + 5, -2
    c.tables = torch.from_numpy(c.table).cuda()
    pool, kv = handle(c), c.pool()
    q, k = normal(1, 1, HQ, DIM), normal(2, 1, HKV, DIM)
    out = torch.empty(1, HQ, DIM, device="cuda")
    pkv.pkv_quant_append_attend(pool, 0, q, k, k, kv, c.tables, c.lens_tensor(), out, 2048)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    keep = np.ones(100, bool)
    keep[32:48] = keep[96:] = False
    keep = torch.from_numpy(keep).cuda()
    ref, tol = attend(q.double(), c.k[0][keep], c.v[0][keep], torch.tensor([10 ** 6], device="cuda"),
                      10 ** 7, 0)
    check(out, ref, tol)
    assert np.array_equal(kv.cpu().numpy(), c.bytes)
    c.table[:] = -1
    out.fill_(3.0)
    pkv.pkv_quant_attention(pool, 0, q, kv, torch.from_numpy(c.table).cuda(), c.lens_tensor(), out, 5)
    assert pkv.pkv_get_error(pool) == pkv.PKV_ERR_OUT_OF_RANGE
    assert bool((out == 0).all())


def test_long_context():
    n = 60000
    c = QuantCache([n, 33000], max_seq_len=65536, seed=6)
    run_decode(c, 65536, 0, 1, True)
    run_decode(c, 5000, 20, 0, False)


def test_pool_offsets_past_2_to_the_31():
    # 130,000 pages of 16,640 bytes; the sequence's pages are the last ones
    pages = 130000
    lens = [100]
    c = QuantCache(lens, seed=8, spare=0)
    small = c.bytes
    c.table[c.table >= 0] += pages - c.num_pages
    c.tables = torch.from_numpy(c.table).cuda()
    kv = torch.zeros(pages, HKV, TILE, dtype=torch.uint8, device="cuda")
    kv[pages - c.num_pages:] = torch.from_numpy(small).cuda()
    pool = pkv.pkv_pool_create(1, pages, 1)
    q, k, v = normal(1, 1, HQ, DIM), normal(2, 1, HKV, DIM), normal(3, 1, HKV, DIM)
    out = torch.empty(1, HQ, DIM, device="cuda")
    pkv.pkv_quant_append_attend(pool, 0, q, k, v, kv, c.tables, c.lens_tensor(), out, 2048)
    kb, vb = torch.empty(100, HKV, DIM, dtype=torch.bfloat16, device="cuda"), \
        torch.empty(100, HKV, DIM, dtype=torch.bfloat16, device="cuda")
    pkv.pkv_quant_read(pool, 0, kv, c.tables, int32([0, 100]), int32([0]), kb, vb, 100)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    ks, vs = c.k[0].clone(), c.v[0].clone()
    ks[-1], vs[-1] = quantise(k.double().cpu())[2][0].cuda(), quantise(v.double().cpu())[2][0].cuda()
    assert torch.equal(kb.double(), ks) and torch.equal(vb.double(), vs)
    ref, tol = attend(q.double(), ks, vs, torch.tensor([99], device="cuda"), 2048, 0)
    check(out, ref, tol)


def test_results_do_not_depend_on_the_pages_or_the_run():
    outs = []
    for spare in (0, 11):
        c = QuantCache([900, 40, 2048, 5], seed=1, spare=spare)
        rng = np.random.RandomState(spare)
        outs.append(run_decode(c, 1000, 4, 1, False))
        outs.append(run_decode(c, 1000, 4, 1, False))
        del rng
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[2], outs[3])


def test_prefill_then_decode_steps_then_read_back():
    # a prompt stored in chunks, then steps that append and attend; each step's output
    # against the values that are read back
    prompt, steps, batch = [37, 5], 14, 2
    c = QuantCache([n + steps for n in prompt], seed=7)
    pool, kv = handle(c), c.pool()
    cos, sin = angles(2048)
    rope = pkv.pkv_axes_rope(cos, sin, AXES[1])
    ks = [normal(20 + b, prompt[b], HKV, DIM) for b in range(batch)]
    vs = [normal(30 + b, prompt[b], HKV, DIM) for b in range(batch)]
    for lo, hi in ((0, 20), (20, 37)):
        rows = [(max(min(n, hi) - lo, 0)) for n in prompt]
        k = torch.cat([x[lo:hi] for x in ks])
        v = torch.cat([x[lo:hi] for x in vs])
        pos = torch.cat([torch.arange(lo, lo + r) for r in rows]).to(torch.int32).cuda()[None]
        pkv.pkv_quant_fill(pool, 0, k, v, kv, c.tables, int32(np.cumsum([0] + rows)),
                           int32([lo] * batch), 20, rope=rope, rope_positions=pos.contiguous())
    for step in range(steps):
        lens = int32([n + step + 1 for n in prompt])
        q, k, v = (normal(100 * step + i, batch, h, DIM) for i, h in enumerate((HQ, HKV, HKV)))
        out = torch.empty(batch, HQ, DIM, device="cuda")
        pos = (lens - 1)[None].contiguous()
        pkv.pkv_quant_append_attend(pool, 0, q, k, v, kv, c.tables, lens, out, 32, sinks=4,
                                    rope=rope, rope_positions=pos)
        total = int(lens.sum())
        kb = torch.empty(total, HKV, DIM, dtype=torch.bfloat16, device="cuda")
        vb = torch.empty_like(kb)
        cu = int32(np.cumsum([0] + lens.tolist()))
        pkv.pkv_quant_read(pool, 0, kv, c.tables, cu, int32([0, 0]), kb, vb, int(lens.max()))
        qd = rotate(q, cos, sin, pos, AXES[1], torch.float64)
        for b in range(batch):
            rows = slice(int(cu[b]), int(cu[b + 1]))
            ref, tol = attend(qd[b:b + 1], kb[rows].double(), vb[rows].double(),
                              torch.tensor([int(lens[b]) - 1], device="cuda"), 32, 4)
            check(out[b:b + 1], ref, tol, f"step {step}")
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK


def test_captured_and_on_another_stream():
    c = QuantCache([300, 1000], seed=12)
    pool, kv = handle(c), c.pool()
    q, k, v = normal(1, 2, HQ, DIM), normal(2, 2, HKV, DIM), normal(3, 2, HKV, DIM)
    lens, out = c.lens_tensor(), torch.zeros(2, HQ, DIM, device="cuda")
    kb = torch.zeros(2, HKV, DIM, dtype=torch.bfloat16, device="cuda")
    vb = torch.zeros_like(kb)
    cu, last = int32([0, 1, 2]), (lens - 1).contiguous()

    def step():
        pkv.pkv_quant_append_attend(pool, 0, q, k, v, kv, c.tables, lens, out, 700)
        pkv.pkv_quant_read(pool, 0, kv, c.tables, cu, last, kb, vb, 1)

    step()
    want = out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    out.zero_()
    kb.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(kb.double().cpu(), quantise(k.double().cpu())[2])
    q.copy_(normal(5, 2, HQ, DIM))                       # new inputs, same graph
    graph.replay()
    torch.cuda.synchronize()
    ks, vs = c.k[0].clone(), c.v[0].clone()
    ks[-1], vs[-1] = quantise(k.double().cpu())[2][0].cuda(), quantise(v.double().cpu())[2][0].cuda()
    ref, tol = attend(q[:1].double(), ks, vs, torch.tensor([299], device="cuda"), 700, 0)
    check(out[:1], ref, tol)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK


def test_programmatic_launches_after_a_fill():
    # on a PDL handle a decode right after the fill that writes its pages waits for it
    c = QuantCache([400, 77], seed=13)
    pool, kv = handle(c, pkv.PKV_FLAG_PDL), torch.from_numpy(c.bytes).cuda()
    k = [normal(40 + b, n, HKV, DIM) for b, n in enumerate(c.lens)]
    rows = torch.cat(k)
    q = normal(1, 2, HQ, DIM)
    out = torch.empty(2, HQ, DIM, device="cuda")
    for _ in range(3):
        pkv.pkv_quant_fill(pool, 0, rows, rows, kv, c.tables, int32([0, 400, 477]), int32([0, 0]), 400)
        pkv.pkv_quant_attention(pool, 0, q, kv, c.tables, c.lens_tensor(), out, 2048)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    for b, n in enumerate(c.lens):
        x = quantise(k[b].double().cpu())[2].cuda()
        ref, tol = attend(q[b:b + 1].double(), x, x, torch.tensor([n - 1], device="cuda"), 2048, 0)
        check(out[b:b + 1], ref, tol)


def test_refusals():
    c = QuantCache([30, 20])
    pool, kv = handle(c), c.pool()
    q, k, v = normal(1, 2, HQ, DIM), normal(2, 2, HKV, DIM), normal(3, 2, HKV, DIM)
    out, lens = torch.empty(2, HQ, DIM, device="cuda"), c.lens_tensor()
    cu, start = int32([0, 1, 2]), int32([0, 0])

    def refused(call, *args, **kw):
        with pytest.raises(pkv.PkvError) as e:
            call(*args, **kw)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG

    def attend_with(layer=0, window=9, kv=kv, q=q, **kw):
        pkv.pkv_quant_attention(pool, layer, q, kv, c.tables, lens, out, window, **kw)

    for kw in (dict(layer=1), dict(layer=-1), dict(window=0), dict(sinks=-1), dict(batch=3, q=q),
               dict(num_splits=-1), dict(num_splits=65)):
        if "batch" in kw:
            with pytest.raises((pkv.PkvError, ValueError)):
                attend_with(**kw)
        else:
            refused(attend_with, **kw)
    refused(attend_with, q=None)
    refused(attend_with, kv=kv.data_ptr() + 4)
    for bad in (kv.to(torch.int8), kv[:, :, :-16].contiguous(), kv[:-1].contiguous(), kv[:, ::2]):
        with pytest.raises(ValueError, match="kv_pool"):
            attend_with(kv=bad)
    refused(pkv.pkv_quant_fill, pool, 0, k, v, kv, c.tables, cu, start, 0)
    refused(pkv.pkv_quant_fill, pool, 0, k, v, kv, c.tables, cu, start, 2049)
    refused(pkv.pkv_quant_fill, pool, 0, None, v, kv, c.tables, cu, start, 1, total_tokens=2)
    refused(pkv.pkv_quant_read, pool, 2, kv, c.tables, cu, start, k, v, 1)
    refused(pkv.pkv_quant_read, pool, 0, kv, c.tables, cu, start, k, None, 1)
    with pytest.raises(ValueError, match="v:"):
        pkv.pkv_quant_read(pool, 0, kv, c.tables, cu, start, k, v[:1], 1)
    # nothing to do
    pkv.pkv_quant_fill(pool, 0, k, v, kv, c.tables, cu, start, 1, batch=0)
    pkv.pkv_quant_read(pool, 0, kv, c.tables, cu, start, k, v, 1, total_tokens=0)
    assert pkv.pkv_get_error(pool) == pkv.PKV_OK
    assert np.array_equal(kv.cpu().numpy(), c.bytes)
