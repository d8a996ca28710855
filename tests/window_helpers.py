"""Plain 64-bit restatement of attention behind a sliding window with sinks, and
inputs for its tests: shuffled pages, and NaN, infinities or huge values in every
slot that no query may read.

Tolerance of a row (one query and head), derived from the arithmetic: each score
is a sum of 64 exact BF16 products in FP32, off by at most 64 roundings of
sum |q_i k_i| / 8; the exponent's argument adds 3 roundings of its own size and the
base-2 exponential 2^-22 of its value, so a weight's relative error is at most
e_w = (64 a + 3 s) u + 2^-22 with a = max_t sum |q_i k_i| / 8, s = max_t |score| and
u = 2^-23 (a tensor-core sum may truncate: twice half a step). Weights of three BF16
terms add 2^-24. Both sums over n tokens add n / 16 + 16 roundings. The output, a
weighted mean of v, is then off by at most
(2 e_w + 2 (n / 16 + 16) u) max_t |v_t|.
"""

import math

import numpy as np
import torch

HQ, HKV, DIM, PAGE = 32, 8, 64, 16
U = 2.0 ** -23


def visible(p, t, window, sinks):
    return (t <= p) & ((p - t < window) | (t < sinks))


def attend(q, k, v, pos, window, sinks):
    """q [rows][32][64], k and v [tokens][8][64] (float64; every token of the
    sequence), pos [rows]: (out, tolerance [rows][32])."""
    rows, n = q.shape[0], k.shape[0]
    t = torch.arange(n, device=q.device)
    seen = visible(pos[:, None], t[None], window, sinks)
    keep = seen.any(0)                       # tokens no row sees may hold anything
    t, seen, k, v = t[keep], seen[:, keep], k[keep], v[keep]
    k = k.repeat_interleave(HQ // HKV, 1).permute(1, 2, 0)
    v = v.repeat_interleave(HQ // HKV, 1).permute(1, 0, 2)
    qh = q.permute(1, 0, 2)                  # [32][rows][64]
    score = (qh @ k) / 8.0
    a = ((qh.abs() @ k.abs()) / 8.0).amax(-1)
    top = score.abs().amax(-1)
    score = score.masked_fill(~seen[None], -math.inf)
    w = torch.exp(score - score.amax(-1, keepdim=True))
    out = (w @ v) / w.sum(-1, keepdim=True)
    e_w = (64 * a + 3 * top) * U + 2.0 ** -22 + 2.0 ** -24
    count = seen.sum(-1)[None].double()
    tol = (2 * e_w + 2 * (count / 16 + 16) * U) * v.abs().amax()
    return out.permute(1, 0, 2), tol.T


class Cache:
    """One layer's sequences over a shuffled pool on the GPU. lens: tokens of each
    (0 allowed); evict(b) -> bool [pages]: logical pages that are not assigned (-1)."""

    def __init__(self, lens, max_seq_len=2048, seed=0, num_layers=1, layer=0, spare=5, evict=None,
                 max_batch=None, k_scale=1.0, base_page=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.max_seq_len, self.layer, self.num_layers = list(lens), max_seq_len, layer, num_layers
        self.max_batch = max_batch or max(1, len(lens))
        stride = max_seq_len // PAGE
        used = []
        for b, n in enumerate(lens):
            pages = np.arange(-(-n // PAGE))
            if evict is not None:
                pages = pages[~evict(b)[:len(pages)]]
            used += [(b, int(p)) for p in pages]
        count = len(used) + spare
        self.num_pages = base_page + count
        ids = (torch.randperm(count, generator=g) + base_page).tolist()
        self.table = np.full((num_layers, self.max_batch, stride), -1, np.int32)
        for (b, p), i in zip(used, ids):
            self.table[layer, b, p] = i
        self.tables = torch.from_numpy(self.table).cuda()
        self.k, self.v = [], []              # per sequence [tokens][8][64] bf16, on the GPU
        gc = torch.Generator(device="cuda").manual_seed(seed + 1)
        for n in lens:
            self.k.append((torch.randn(n, HKV, DIM, generator=gc, device="cuda") * k_scale).bfloat16())
            self.v.append(torch.randn(n, HKV, DIM, generator=gc, device="cuda").bfloat16())
        self.gen = gc

    def pools(self, keep, junk=math.nan):
        """Pools holding the tokens for which keep(b) (bool [tokens]) is true; every
        other slot holds `junk` (or NaN, infinities and huge values in turn)."""
        out = []
        for src in (self.k, self.v):
            pool = torch.empty(self.num_pages, HKV, PAGE, DIM, dtype=torch.bfloat16, device="cuda")
            if junk == "mixed":
                pat = torch.tensor([math.nan, math.inf, -math.inf, 3e38, -3e38, 0.0, 1.0],
                                   device="cuda").bfloat16()
                idx = torch.randint(0, 7, (HKV * PAGE * DIM,), generator=self.gen, device="cuda")
                pool.copy_(pat[idx].view(1, HKV, PAGE, DIM))
            else:
                pool.fill_(junk)
            for b, n in enumerate(self.lens):
                t = torch.nonzero(torch.as_tensor(keep(b)[:n])).flatten().cuda()
                if t.numel() == 0:
                    continue
                page = self.tables[self.layer, b].long()[t // PAGE]
                assert int(page.min()) >= 0
                pool[page, :, t % PAGE] = src[b][t]
            out.append(pool)
        return out

    def lens_tensor(self):
        return torch.tensor(self.lens, dtype=torch.int32, device="cuda")


def seen_by_last(n, window, sinks):
    t = np.arange(n)
    return visible(n - 1, t, window, sinks)


def unseen_pages(n, first, window, sinks):
    """Logical pages of an n-token sequence with no token that a query at a
    position >= first sees."""
    t = np.arange(-(-n // PAGE) * PAGE)
    seen = (t < n) & ((t > first - window) | (t < sinks))
    return ~seen.reshape(-1, PAGE).any(1)


def angles(rows, base=10000.0):
    p = torch.arange(rows, dtype=torch.float64)[:, None]
    f = base ** (-torch.arange(32, dtype=torch.float64) / 32)
    return torch.cos(p * f).float().cuda(), torch.sin(p * f).float().cuda()


def rotate(x, cos, sin, positions, axis_of_pair, dtype):
    """x [tokens][heads][64] rotated in `dtype` (float64, or float32 with every
    product and sum rounded)."""
    axis = torch.tensor(axis_of_pair, device=x.device)
    at = positions.long()[axis].T
    pair = torch.arange(32, device=x.device)
    c, s = cos[at, pair][:, None].to(dtype), sin[at, pair][:, None].to(dtype)
    a, b = x[..., :32].to(dtype), x[..., 32:].to(dtype)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def check(got, ref, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    worst = ((got - ref).abs() / tol[..., None]).max().item()
    assert worst <= 1.0, f"{what}: {worst:.2f} times the tolerance"
    return worst
