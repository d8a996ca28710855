"""Plain restatement of the 8-bit cache and inputs for its tests.

A row's 64 values are e4m3 codes times a power of two; the restatement works on
those values and on the documented bytes of a tile, in 64 bits.

Tolerance of an attention row, derived from the arithmetic: products of FP16
operands are exact in FP32. A rotated query is the sum of two FP16 terms, off by
2^-23 of it (and 2^-39 of its head's largest dim, at most 2^-24 of a = max_t sum
|q_i k_i| / 8 once the largest dims count), a score a sum of 64 products with at
most 64 roundings of a (u = 2^-23 each: a tensor-core sum may truncate, twice half
a step), its scaling exact, and the exponent's argument adds 3 roundings of its own
size and the base-2 exponential 2^-22 of its value: a weight is off by e_w = (64 a +
3 s) u + 2^-22 + 2^-23 a, s = max_t |score|. Two FP16 terms of p 2^ev keep it to
2^-22 of itself or 2^-32 of the head's largest weighted row; every sum of a page has
16 roundings and n / 16 pages are added in FP32. Off by at most, then,
(2 e_w + 2^-22 + 2 (n / 16 + 16) u) max |v| + n 2^-32 max |v|.
"""

import math

import numpy as np
import torch

from window_helpers import DIM, HKV, HQ, PAGE, U, visible

TILE = 2080
LARGEST = 1.875 * 2.0 ** 127


def grid():
    """The values of the 256 codes."""
    out = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        x = math.nan if code & 127 == 127 else m / 512 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out.append(-x if code & 128 else x)
    return torch.tensor(out, dtype=torch.float64)


def quantise(x):
    """x [..., 64] (float64): (codes, exponent bytes, what they stand for), each value
    taken to the nearest of the grid's, ties to the even code. On the CPU."""
    x = x.clamp(-LARGEST, LARGEST)
    most = x.abs().nan_to_num(0.0).amax(-1)
    e = torch.full(most.shape, -124.0, dtype=torch.float64)
    for _ in range(260):
        e = torch.where(most > 448.0 * 2.0 ** e, e + 1, e)
    y = x / (2.0 ** e)[..., None]
    codes = torch.from_numpy(nearest(y.numpy()))
    exps = (e + 127).to(torch.uint8)
    value = grid()[codes.long()] * (2.0 ** e)[..., None]
    return codes, exps, value


def nearest(y):
    """uint8 codes of the grid's values nearest to y, found by bisection."""
    up = grid()[:127].numpy()                         # 0 .. 448, codes 0 .. 126
    a = np.abs(np.nan_to_num(y, nan=0.0))
    hi = np.clip(np.searchsorted(up, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_hi, d_lo = up[hi] - a, a - up[lo]
    take_lo = (d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0))
    code = np.where(take_lo, lo, hi).astype(np.uint8)
    code = np.where(np.isnan(y), np.uint8(127), code)
    return np.where(np.signbit(y) & ~np.isnan(y), code | 128, code).astype(np.uint8)


def places():
    """Where a tile keeps (K code, V code) of [token][dim]."""
    t, d = np.meshgrid(np.arange(PAGE), np.arange(DIM), indexing="ij")
    return t * DIM + d, 1024 + d // 16 * 256 + t * 16 + d % 16


def put(pool, page, slot, which, codes, exps):
    """Codes [tokens][8][64] and exponents [tokens][8] into a pool of bytes (numpy
    [pages][8][2080]) at page[i], slot[i]."""
    page, slot = np.asarray(page), np.asarray(slot)
    if page.size == 0:
        return
    heads = np.arange(HKV)[None, :]
    pool[page[:, None, None], heads[..., None], places()[which][slot][:, None]] = codes
    pool[page[:, None], heads, 2048 + 16 * which + slot[:, None]] = exps


def attend(q, k, v, pos, window, sinks):
    """q [rows][32][64], k and v [tokens][8][64], float64: (out, tolerance [rows][32])."""
    n = k.shape[0]
    t = torch.arange(n, device=q.device)
    seen = visible(pos[:, None], t[None], window, sinks)
    keep = seen.any(0)
    t, seen, k, v = t[keep], seen[:, keep], k[keep], v[keep]
    k = k.repeat_interleave(HQ // HKV, 1).permute(1, 2, 0)
    v = v.repeat_interleave(HQ // HKV, 1).permute(1, 0, 2)
    qh = q.permute(1, 0, 2)
    score = (qh @ k) / 8.0
    a = ((qh.abs() @ k.abs()) / 8.0).amax(-1)
    top = score.abs().amax(-1)
    score = score.masked_fill(~seen[None], -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    out = (w @ v) / w.sum(-1, keepdim=True)
    e_w = (64 * a + 3 * top) * U + 2.0 ** -22 + 2.0 ** -23 * a
    count = seen.sum(-1)[None].double()
    tol = (2 * e_w + 2.0 ** -22 + 2 * (count / 16 + 16) * U + count * 2.0 ** -32) * v.abs().amax()
    return out.permute(1, 0, 2), tol.T


class QuantCache:
    """One layer's sequences in a shuffled 8-bit pool. Slots that hold no token are
    junk: NaN codes and exponent bytes of every kind. evict(b) -> bool [pages]:
    logical pages that are not assigned."""

    def __init__(self, lens, max_seq_len=2048, seed=0, spare=3, k_scale=1.0, v_scale=None,
                 evict=None, max_batch=None, num_layers=1, layer=0):
        rng = np.random.RandomState(seed)
        self.lens, self.max_seq_len, self.layer = list(lens), max_seq_len, layer
        self.num_layers, self.max_batch = num_layers, max_batch or max(1, len(lens))
        used = []
        for b, n in enumerate(lens):
            pages = np.arange(-(-n // PAGE))
            if evict is not None:
                pages = pages[~evict(b)[:len(pages)]]
            used += [(b, int(p)) for p in pages]
        self.num_pages = len(used) + spare
        ids = rng.permutation(self.num_pages)
        self.table = np.full((num_layers, self.max_batch, max_seq_len // PAGE), -1, np.int32)
        for (b, p), i in zip(used, ids):
            self.table[layer, b, p] = i
        self.bytes = rng.choice(np.array([127, 255, 0, 126, 8, 240], np.uint8),
                                (self.num_pages, HKV, TILE))
        self.k, self.v = [], []                       # float64 [tokens][8][64], as stored
        for b, n in enumerate(lens):
            for which, to in enumerate((self.k, self.v)):
                x = torch.from_numpy(rng.randn(n, HKV, DIM)) * (k_scale if which == 0 else 1.0)
                if which == 1 and v_scale is not None:
                    x = x * v_scale(rng, n)[:, None, None]
                codes, exps, value = quantise(x.to(torch.bfloat16).double())
                to.append(value.cuda())
                t = np.arange(n)
                page = self.table[layer, b, t // PAGE]
                keep = page >= 0
                put(self.bytes, page[keep], t[keep] % PAGE, which, codes.numpy()[keep],
                    exps.numpy()[keep])
        self.tables = torch.from_numpy(self.table).cuda()

    def pool(self):
        return torch.from_numpy(self.bytes).cuda()

    def lens_tensor(self):
        return torch.tensor(self.lens, dtype=torch.int32, device="cuda")
