"""Plain 64-bit restatement of attention of drafted trees, random trees, and inputs
for its tests. Tolerance of a row: that of window_helpers, whose arithmetic this
attention shares (BF16 products summed in FP32, weights as three BF16 terms)."""

import math

import numpy as np
import torch

from window_helpers import HKV, HQ, U


def random_tree(rng, n, depth_first=0.7):
    """Masks (python ints) of a random tree of n nodes, each after its parent."""
    masks = []
    for i in range(n):
        if i == 0:
            masks.append(1)
            continue
        parent = i - 1 if rng.rand() < depth_first else int(rng.randint(0, i))
        masks.append(masks[parent] | 1 << i)
    return masks


def depth(mask, n):
    return bin(mask & ((1 << n) - 1)).count("1") - 1


def pack(masks):
    """int64 tensor of masks given as python ints of up to 64 bits."""
    return torch.from_numpy(np.array([m & (1 << 64) - 1 for m in masks], np.uint64).view(np.int64)).cuda()


def seen_matrix(start, masks, window, sinks):
    """bool [rows][start + n]: what each row sees."""
    n = len(masks)
    t = np.arange(start)
    out = np.zeros((n, start + n), bool)
    for i, m in enumerate(masks):
        p = start + depth(m, n)
        out[i, :start] = (p - t < window) | (t < sinks)
        out[i, start:] = [m >> j & 1 for j in range(n)]
    return out


def attend(q, k, v, seen):
    """q [rows][32][64], k and v [tokens][8][64] (float64), seen bool [rows][tokens]
    (numpy): (out, tolerance [rows][32]); rows that see nothing are 0."""
    seen = torch.from_numpy(seen).to(q.device)
    keep = seen.any(0)
    seen, k, v = seen[:, keep], k[keep], v[keep]
    if seen.shape[1] == 0:
        return torch.zeros_like(q), torch.full(q.shape[:2], 1e-30, dtype=q.dtype, device=q.device)
    k = k.repeat_interleave(HQ // HKV, 1).permute(1, 2, 0)
    v = v.repeat_interleave(HQ // HKV, 1).permute(1, 0, 2)
    qh = q.permute(1, 0, 2)
    score = (qh @ k) / 8.0
    a = ((qh.abs() @ k.abs()) / 8.0).masked_fill(~seen[None], 0).amax(-1)
    top = score.abs().masked_fill(~seen[None], 0).amax(-1)
    score = score.masked_fill(~seen[None], -math.inf)
    empty = ~seen.any(1)
    most = score.amax(-1, keepdim=True).masked_fill(empty[None, :, None], 0)
    w = torch.exp(score - most)
    out = (w @ v) / w.sum(-1, keepdim=True).masked_fill(empty[None, :, None], 1)
    e_w = (64 * a + 3 * top) * U + 2.0 ** -22 + 2.0 ** -24
    count = seen.sum(-1)[None].double()
    tol = (2 * e_w + 2 * (count / 16 + 16) * U) * v.abs().amax()
    return out.permute(1, 0, 2), tol.T
