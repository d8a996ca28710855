"""Timed cases of the 8-bit cache and of drafted token trees.

Geometry of the library: 32 query heads over 8 KV heads, head_dim 64, 16-token
pages. Where ``own`` is false, ``run`` computes the operator with elementary
torch operations in FP32; where it is true, it makes the library's calls.

The 8-bit pool is uint8 [num_pages][8][2080]: a (page, KV head) tile holds the
codes of K as [16 tokens][64 dims], those of V as [4 chunks][16 tokens][16 dims]
and the 16 tokens' exponents of K and of V. A token's 64 values of one head are
e4m3 codes times 2^(exponent byte - 127), the smallest such power of two (at
least 2^-124) with which the largest of them stays within 448.

  decode  attention of one new token per sequence over an 8-bit cache, over the
          last `window` tokens and the first `sinks` ones (window 0: all);
          fused: the token is quantised and appended first, and read back;
          axes > 0: keys and queries are rotated by that many position axes
  store   a chunk of prompt tokens per sequence quantised into its pages, and
          the sequence so far read back
  tree    attention of drafted tokens (a tree per sequence) over a BF16 cache
  commit  the accepted path of each tree moved together, in every layer
"""

import functools
import math

import numpy as np
import torch

own = False

HQ, HKV, DIM, PAGE = 32, 8, 64, 16
GROUP = HQ // HKV
PAIRS = DIM // 2
SECTIONS = {1: (32,), 2: (16, 16), 3: (8, 12, 12)}   # rotary pairs of each axis
SHORT_CONTEXT = 2048                                 # longer handles carry the long-context flag
CODES = PAGE * DIM                                   # bytes of K (and of V) in a tile
TILE = 2 * CODES + 2 * PAGE
TOKEN_BF16 = 2 * HKV * DIM * 2                       # K and V of one token
TOKEN_8BIT = 2 * HKV * (DIM + 1)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's chat turn at the end of the context: latency of a small call
        dict(name="decode-1-2048", kind="decode", batch=1, lo=2048, hi=2048, max_seq_len=2048,
             window=0, sinks=0, fused=False, axes=0),
        # a mixed batch of chats of every length, queries rotated
        dict(name="decode-64-2048", kind="decode", batch=64, lo=16, hi=2048, max_seq_len=2048,
             window=0, sinks=0, fused=False, axes=1),
        # a full serving batch of long chats behind a window, one step with append
        dict(name="step-256-w4096", kind="decode", batch=256, lo=1, hi=32768, max_seq_len=32768,
             window=4096, sinks=4, fused=True, axes=3),
        # a few very long documents, everything visible
        dict(name="decode-4-128k", kind="decode", batch=4, lo=120001, hi=131072,
             max_seq_len=131072, window=0, sinks=0, fused=False, axes=0),
        # a short question stored and read back for its continuation
        dict(name="store-1x77", kind="store", batch=1, chunk_lo=77, chunk_hi=77, start=0,
             max_seq_len=2048, axes=1),
        # a batch of image and video prompts
        dict(name="store-8x2048", kind="store", batch=8, chunk_lo=1536, chunk_hi=2048, start=0,
             max_seq_len=2048, axes=3),
        # chunks that continue long documents, whose prefill takes the whole prefix
        dict(name="store-4x512-at-30000", kind="store", batch=4, chunk_lo=412, chunk_hi=512,
             start=30001, max_seq_len=32768, axes=0),
        # a few drafted tokens of one user: latency of a small call
        dict(name="tree-1x8", kind="tree", batch=1, nodes_lo=8, nodes_hi=8, lo=2000, hi=2000,
             max_seq_len=2048, window=0, sinks=0),
        # a batch of chats of every length, each with a tree of up to 16 drafted tokens
        dict(name="tree-32x16", kind="tree", batch=32, nodes_lo=9, nodes_hi=16, lo=16, hi=2000,
             max_seq_len=2048, window=0, sinks=0),
        # the largest trees over long documents
        dict(name="tree-8x64", kind="tree", batch=8, nodes_lo=49, nodes_hi=64, lo=20001, hi=32700,
             max_seq_len=32768, window=0, sinks=0),
        # one user's accepted tokens
        dict(name="commit-1", kind="commit", batch=1, accept=4, nodes=8, layers=16),
        # a batch's
        dict(name="commit-256", kind="commit", batch=256, accept=8, nodes=32, layers=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _rounded(tokens):
    return SHORT_CONTEXT if tokens <= SHORT_CONTEXT else -(-tokens // PAGE) * PAGE


def draw(rng):
    kind = rng.choice(["decode", "decode", "store", "tree", "tree", "commit"])
    if kind == "decode":
        longest = _log_int(rng, 40, 131072)
        window = 0 if rng.random() < 0.4 else _log_int(rng, 16, 8192)
        seen = min(longest, window or longest)
        batch = _log_int(rng, 1, max(1, min(256, (1 << 19) // seen)))
        return dict(kind=kind, batch=batch, lo=rng.randint(1, longest), hi=longest,
                    max_seq_len=_rounded(longest), window=window,
                    sinks=rng.choice([0, 1, 4, rng.randint(0, 70)]),
                    fused=rng.random() < 0.6, axes=rng.choice([0, 1, 2, 3]))
    if kind == "store":
        start = 0 if rng.random() < 0.5 else _log_int(rng, 1, 28000)
        chunk = _log_int(rng, 5, 2048)
        batch = _log_int(rng, 1, max(1, min(16, 120000 // (start + chunk))))
        return dict(kind=kind, batch=batch, chunk_lo=rng.randint(1, chunk), chunk_hi=chunk,
                    start=start, max_seq_len=_rounded(start + chunk), axes=rng.choice([0, 1, 2, 3]))
    if kind == "tree":
        longest = _log_int(rng, 20, 60000)
        nodes = _log_int(rng, 2, 64)
        batch = _log_int(rng, 1, max(1, min(64, (1 << 18) // longest, (1 << 23) // longest // nodes)))
        window = 0 if rng.random() < 0.6 else _log_int(rng, 16, 8192)
        return dict(kind=kind, batch=batch, nodes_lo=rng.randint(1, nodes), nodes_hi=nodes,
                    lo=rng.randint(0, longest), hi=longest, max_seq_len=_rounded(longest + nodes),
                    window=window, sinks=rng.choice([0, 1, 4, rng.randint(0, 70)]))
    nodes = _log_int(rng, 1, 64)
    return dict(kind=kind, batch=_log_int(rng, 1, 256), accept=rng.randint(1, min(nodes, 16)),
                nodes=nodes, layers=rng.randint(1, 16))


# ------------------------------------------------------------------ sizes that a case fixes
def _spread(lo, hi, n):
    """n whole numbers from lo to hi, even in the logarithm (the seed only orders them)."""
    if n == 1:
        return np.array([hi], np.int64)
    x = np.exp(np.linspace(math.log(lo + 1), math.log(hi + 1), n)) - 1
    return np.clip(np.rint(x).astype(np.int64), lo, hi)


def _window(case):
    return case["window"] or case["max_seq_len"]


def _trees(case):
    """(prefix length, drafted tokens) of each sequence."""
    return (_spread(case["lo"], case["hi"], case["batch"]),
            _spread(case["nodes_lo"], case["nodes_hi"], case["batch"])[::-1])


def _accepted(case):
    """How many tokens of each sequence's path are accepted."""
    return np.arange(case["batch"], dtype=np.int64) * 5 % case["accept"] + 1


def work(case):
    kind = case["kind"]
    if kind == "decode":
        lens = _spread(case["lo"], case["hi"], case["batch"])
        w, s = _window(case), case["sinks"]
        seen = int((np.minimum(lens, w) + np.clip(np.minimum(s, lens - w), 0, None)).sum())
        per_seq = HQ * DIM * (2 + 4) + 4 + (2 * 4 * PAIRS if case["axes"] else 0)
        if case["fused"]:                              # the new row in, stored, and read back
            per_seq += 2 * TOKEN_BF16 + TOKEN_8BIT
        return {"bytes": seen * TOKEN_8BIT + case["batch"] * per_seq,
                "flops": seen * HQ * DIM * 4}
    if kind == "store":
        n = _spread(case["chunk_lo"], case["chunk_hi"], case["batch"])
        new, back = int(n.sum()), int(n.sum()) + case["batch"] * case["start"]
        return {"bytes": new * (TOKEN_BF16 + TOKEN_8BIT + 4 * case["axes"])
                + back * (TOKEN_8BIT + TOKEN_BF16),
                "flops": new * HKV * DIM * (3 if case["axes"] else 1)}
    if kind == "tree":
        start, n = _trees(case)
        w, s = min(_window(case), 1 << 30), case["sinks"]
        prefix = np.minimum(start, w) + np.clip(np.minimum(s, start - w), 0, None)
        keys = int((prefix + n).sum())
        pairs = int((n * (prefix + (n + 1) / 4)).sum())
        return {"bytes": keys * TOKEN_BF16 + int(n.sum()) * (HQ * DIM * (2 + 4) + 8),
                "flops": pairs * HQ * DIM * 4}
    moved = int(_accepted(case).sum()) * case["layers"]
    return {"bytes": moved * 2 * TOKEN_BF16, "flops": 0}


# ------------------------------------------------------------------ the 8-bit pool
def _views(kv_pool):
    """Codes of K and V as [pages][8][16][64] (views; V's dims split in 4 chunks:
    [pages][8][16][4][16]) and the exponents [pages][8][2][16]."""
    k = kv_pool[..., :CODES].unflatten(-1, (PAGE, DIM))
    v = kv_pool[..., CODES:2 * CODES].unflatten(-1, (4, PAGE, 16)).permute(0, 1, 3, 2, 4)
    return k, v, kv_pool[..., 2 * CODES:].unflatten(-1, (2, PAGE))


def _power(e):
    """2^e in FP32, exact, for whole numbers e from -126 to 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """x [..., 64] in FP32: codes (uint8 bits of e4m3) and exponent bytes [...]."""
    most = x.abs().amax(-1)
    m, e = torch.frexp(most)                           # most = m 2^e; 448 = 0.875 x 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(most > 0, torch.clamp(e, min=-124), torch.full_like(e, -124))
    codes = (x * _power(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _store(kv_pool, page, slot, k, v):
    """Rows k, v [tokens][8][64] (FP32) quantised into the slots of their pages."""
    kc, vc, exps = _views(kv_pool)
    codes, e = _quantise(k)
    kc[page, :, slot] = codes
    exps[page, :, 0, slot] = e
    codes, e = _quantise(v)
    vc[page, :, slot] = codes.unflatten(-1, (4, 16))
    exps[page, :, 1, slot] = e


def _load(kv_pool, page, slot):
    """K and V [..., 8, 64] in FP32 of the tokens in those slots."""
    kc, vc, exps = _views(kv_pool)
    out = []
    for i, codes in enumerate((kc[page, :, slot], vc[page, :, slot].flatten(-2))):
        scale = _power(exps[page, :, i, slot].to(torch.int32) - 127)
        out.append(codes.contiguous().view(torch.float8_e4m3fn).float().mul_(scale[..., None]))
    return out


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _pool8(gen, num_pages):
    """An 8-bit pool holding N(0, 1) keys and values, made a part at a time."""
    pool = torch.empty(num_pages, HKV, TILE, dtype=torch.uint8, device="cuda")
    for i in range(0, num_pages, 8192):
        part = pool[i:i + 8192]
        views = _views(part)
        for which in range(2):
            x = torch.randn((part.shape[0], HKV, PAGE, DIM), generator=gen, device="cuda")
            codes, e = _quantise(x)
            views[which].copy_(codes if which == 0 else codes.unflatten(-1, (4, 16)))
            views[2][:, :, which].copy_(e)
    return pool


def _pools(gen, num_pages):
    out = []
    for _ in range(2):
        pool = torch.empty(num_pages, HKV, PAGE, DIM, dtype=torch.bfloat16, device="cuda")
        for i in range(0, num_pages, 8192):
            part = pool[i:i + 8192]
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
        out.append(pool)
    return out


def _angles(rows):
    """cos and sin of p * 10000^(-2 i / 64), computed in 64 bits."""
    p = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None]
    f = 10000.0 ** (-torch.arange(PAIRS, dtype=torch.float64, device="cuda") / PAIRS)
    return torch.cos(p * f).float(), torch.sin(p * f).float()


def _needed_pages(case, first, last):
    """Which logical pages of each sequence hold a token that some query at a position
    from `first` on sees, up to token `last`: bool [sequences][pages of a row]."""
    page = np.arange(case["max_seq_len"] // PAGE)[None, :]
    first, last = np.asarray(first)[:, None], np.asarray(last)[:, None]
    lo = np.maximum(first - _window(case) + 1, 0) // PAGE
    return (page <= last // PAGE) & ((page >= lo) | (page * PAGE < case["sinks"]))


def _tables(gen, needed, num_pages):
    """Block tables of one layer: shuffled ids for the pages a sequence needs, else -1."""
    ids = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    need = torch.from_numpy(needed).cuda()
    table = torch.full(need.shape, -1, dtype=torch.int32, device="cuda")
    table[need] = ids[: int(needed.sum())]
    return table


def _int32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _packed(s, counts, name=""):
    """Offsets of packed rows and, for each row, its sequence and place in it."""
    cu = np.concatenate([[0], np.cumsum(counts)])
    s["cu" + name] = _int32(cu)
    seq = torch.repeat_interleave(torch.arange(len(counts), device="cuda"),
                                  torch.from_numpy(np.ascontiguousarray(counts)).cuda())
    s["seq" + name] = seq
    s["index" + name] = torch.arange(int(cu[-1]), device="cuda") - s["cu" + name].long()[seq]
    return int(cu[-1])


def _rope_inputs(s, positions, rows):
    axes = s["case"]["axes"]
    s["cos"], s["sin"] = _angles(rows)
    s["axis_positions"] = positions.to(torch.int32).contiguous()
    s["axis_of_pair"] = [a for a, n in enumerate(SECTIONS[axes]) for _ in range(n)]
    s["axis_index"] = torch.tensor(s["axis_of_pair"], device="cuda")


def _grid_positions(axes, index):
    """Rotary positions of the tokens at `index` in a prompt of 9 words and then
    frames of 12 x 20 patches (time, height, width)."""
    i = torch.clamp(index - 9, min=0)
    text = index < 9
    t, h, w = i // 240, i % 240 // 20, i % 20
    rows = [index] if axes == 1 else [t + 9, h * 20 + w + 9] if axes == 2 \
        else [t + 9, h + 9, w + 9]
    return torch.stack([torch.where(text, index, r) for r in rows])


def _random_trees(order, nodes):
    """A tree per sequence: node 0 is the root, each other one hangs from an earlier
    one, mostly a late one (drafts are deeper than they are wide). Bit j of a node's
    mask: it sees node j, an ancestor or itself."""
    masks = []
    for n in nodes:
        own_masks = [1]
        for i in range(1, n):
            parent = i - 1 - int(order.randint(0, min(i, 4)))
            own_masks.append(own_masks[parent] | 1 << i)
        masks += own_masks
    return torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = np.random.RandomState(seed % (1 << 32))
    s = {"case": case}
    kind = case["kind"]
    if kind == "decode":
        batch = case["batch"]
        lens = np.maximum(order.permutation(_spread(case["lo"], case["hi"], batch)), 1)
        needed = _needed_pages(case, lens - 1, lens - 1)
        s["num_pages"] = int(needed.sum()) + 3
        s["tables"] = _tables(gen, needed, s["num_pages"])[None].contiguous()
        s["kv_pool"] = _pool8(gen, s["num_pages"])
        s["lens"] = _int32(lens)
        s["q"] = _normal(gen, batch, HQ, DIM)
        if case["fused"]:
            s["k"], s["v"] = _normal(gen, batch, HKV, DIM), _normal(gen, batch, HKV, DIM)
            s["cu"], s["last"] = _int32(np.arange(batch + 1)), _int32(lens - 1)
            s["k_back"], s["v_back"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        if case["axes"]:
            back = torch.randint(0, 300, (case["axes"], batch), generator=gen, device="cuda")
            _rope_inputs(s, torch.clamp(s["lens"][None, :] - 1 - back, min=0), case["max_seq_len"])
        s["out"] = torch.zeros(batch, HQ, DIM, device="cuda")
    elif kind == "store":
        n = order.permutation(_spread(case["chunk_lo"], case["chunk_hi"], case["batch"]))
        start, batch = case["start"], case["batch"]
        sizes = dict(case, window=0, sinks=0)
        needed = _needed_pages(sizes, np.full(batch, start), start + n - 1)
        s["num_pages"] = int(needed.sum()) + 3
        s["tables"] = _tables(gen, needed, s["num_pages"])[None].contiguous()
        s["kv_pool"] = _pool8(gen, s["num_pages"])
        total = _packed(s, n)
        whole = _packed(s, n + start, "_all")
        s["start"], s["zeros"] = _int32(np.full(batch, start)), _int32(np.zeros(batch))
        s["max_chunk"], s["max_all"] = int(n.max()), int(n.max()) + start
        s["k"], s["v"] = _normal(gen, total, HKV, DIM), _normal(gen, total, HKV, DIM)
        s["k_back"] = torch.empty(whole, HKV, DIM, dtype=torch.bfloat16, device="cuda")
        s["v_back"] = torch.empty_like(s["k_back"])
        if case["axes"]:
            _rope_inputs(s, _grid_positions(case["axes"], s["index"] + start),
                         max(case["max_seq_len"], 512))
    elif kind == "tree":
        at = order.permutation(case["batch"])
        start, n = (x[at] for x in _trees(case))
        needed = _needed_pages(case, start, start + n - 1)
        s["num_pages"] = int(needed.sum()) + 3
        s["tables"] = _tables(gen, needed, s["num_pages"])[None].contiguous()
        s["k_pool"], s["v_pool"] = _pools(gen, s["num_pages"])
        total = _packed(s, n)
        s["start"], s["nodes"] = _int32(start), _int32(n)
        s["longest"], s["most"] = int((start + n).max()), int(n.max())
        s["masks"] = _random_trees(order, n)
        s["q"] = _normal(gen, total, HQ, DIM)
        s["out"] = torch.zeros(total, HQ, DIM, device="cuda")
    else:
        batch, layers, nodes = case["batch"], case["layers"], case["nodes"]
        start = order.permutation(np.arange(batch) * 37 % (SHORT_CONTEXT - nodes + 1))
        page = np.arange(SHORT_CONTEXT // PAGE)[None]
        needed = (page >= start[:, None] // PAGE) & (page <= (start[:, None] + nodes - 1) // PAGE)
        needed = np.broadcast_to(needed[None], (layers,) + needed.shape).reshape(layers * batch, -1)
        s["num_pages"] = int(needed.sum()) + 3
        s["tables"] = _tables(gen, needed, s["num_pages"]).view(layers, batch, -1)
        s["k_pool"], s["v_pool"] = _pools(gen, s["num_pages"])
        count = order.permutation(_accepted(case))
        s["start"], s["counts"] = _int32(start), _int32(count)
        # a path through the tree: the k-th accepted token is its k-th drafted one or a later one
        s["accepted"] = _int32(np.sort(np.argsort(order.rand(batch, nodes), 1)[:, :case["accept"]], 1))
    return s


# ------------------------------------------------------------------ the library's calls
@functools.lru_cache(maxsize=None)
def _handle(layers, num_pages, max_batch, max_seq_len):
    """The pool handle that a program keeps for its pool."""
    import paged_kv_cache_210_gb300 as pkv
    return pkv.pkv_pool_create(layers, num_pages, max_batch, max_seq_len=max_seq_len,
                               flags=pkv.PKV_FLAG_LONG_CONTEXT if max_seq_len > SHORT_CONTEXT
                               else 0)


def _own(s):
    import paged_kv_cache_210_gb300 as pkv
    case = s["case"]
    kind = case["kind"]
    pool = _handle(case.get("layers", 1), s["num_pages"], case["batch"],
                   case.get("max_seq_len", SHORT_CONTEXT))
    rope = {}
    if case.get("axes"):
        if "rope" not in s:                           # kept beside the tables
            s["rope"] = pkv.pkv_axes_rope(s["cos"], s["sin"], s["axis_of_pair"])
        rope = dict(rope=s["rope"], rope_positions=s["axis_positions"])
    if kind == "decode":
        window, sinks = _window(case), case["sinks"]
        if not case["fused"]:
            pkv.pkv_quant_attention(pool, 0, s["q"], s["kv_pool"], s["tables"], s["lens"],
                                    s["out"], window, sinks=sinks, **rope)
            return s["out"]
        pkv.pkv_quant_append_attend(pool, 0, s["q"], s["k"], s["v"], s["kv_pool"], s["tables"],
                                    s["lens"], s["out"], window, sinks=sinks, **rope)
        pkv.pkv_quant_read(pool, 0, s["kv_pool"], s["tables"], s["cu"], s["last"], s["k_back"],
                           s["v_back"], 1)
        return s["out"], s["k_back"], s["v_back"]
    if kind == "store":
        pkv.pkv_quant_fill(pool, 0, s["k"], s["v"], s["kv_pool"], s["tables"], s["cu"],
                           s["start"], s["max_chunk"], **rope)
        pkv.pkv_quant_read(pool, 0, s["kv_pool"], s["tables"], s["cu_all"], s["zeros"],
                           s["k_back"], s["v_back"], s["max_all"])
        return s["k_back"], s["v_back"]
    if kind == "tree":
        pkv.pkv_tree_attention(pool, 0, s["q"], s["k_pool"], s["v_pool"], s["tables"], s["cu"],
                               s["start"], s["masks"], s["out"], _window(case),
                               sinks=case["sinks"])
        return s["out"]
    pkv.pkv_tree_commit(pool, s["k_pool"], s["v_pool"], s["tables"], s["start"], s["accepted"],
                        s["counts"])
    return s["k_pool"].view(torch.int16), s["v_pool"].view(torch.int16)


# ------------------------------------------------------------------ plain form
def _rotate(x, s):
    """x [tokens][heads][64] rotated in FP32, dim i with dim i + 32, pair i by
    the position on its axis."""
    at = s["axis_positions"].long()[s["axis_index"]].T          # [tokens][32]
    pair = torch.arange(PAIRS, device="cuda")
    c, sn = s["cos"][at, pair][:, None], s["sin"][at, pair][:, None]
    a, b = x[..., :PAIRS].float(), x[..., PAIRS:].float()
    return torch.cat([a * c - b * sn, b * c + a * sn], -1)


def _page_of(s, pos, layer=0):
    """Physical pages of the tokens at pos [sequences][tokens]."""
    return torch.clamp(torch.gather(s["tables"][layer].long(), 1, pos // PAGE), min=0)


def _softmax_products(q, k, v, seen):
    """softmax(q k / 8 over the seen keys) v: q [B][8][rows][64], k and v
    [B][keys][8][64], seen broadcast over [B][8][rows][keys]."""
    x = torch.matmul(q, k.permute(0, 2, 3, 1)) * 0.125
    x.masked_fill_(~seen, -math.inf)
    x -= x.max(-1, keepdim=True).values
    x.exp_()
    total = x.sum(-1, keepdim=True)
    return torch.matmul(x, v.permute(0, 2, 1, 3)) / total


def _plain_decode(s):
    case = s["case"]
    lens = s["lens"].long()
    q = _rotate(s["q"], s) if case["axes"] else s["q"].float()
    if case["fused"]:
        at = lens[:, None] - 1
        page, slot = _page_of(s, at)[:, 0], at[:, 0] % PAGE
        _store(s["kv_pool"], page, slot, _rotate(s["k"], s) if case["axes"] else s["k"].float(),
               s["v"].float())
    window = min(_window(case), case["hi"])
    sinks = min(case["sinks"], case["hi"])
    first = lens[:, None] - window                              # of the window
    head = torch.arange(sinks, device="cuda")[None].expand(lens.numel(), -1)
    tail = first + torch.arange(window, device="cuda")[None]
    pos = torch.cat([head, tail], 1)
    seen = torch.cat([head < first, tail >= 0], 1)
    pos = torch.clamp(torch.minimum(pos, lens[:, None] - 1), min=0)
    k, v = _load(s["kv_pool"], _page_of(s, pos), pos % PAGE)
    o = _softmax_products(q.view(-1, HKV, GROUP, DIM), k, v, seen[:, None, None])
    s["out"].copy_(o.reshape(-1, HQ, DIM))
    if not case["fused"]:
        return s["out"]
    for back, x in zip((s["k_back"], s["v_back"]), _load(s["kv_pool"], page, slot)):
        back.copy_(x)
    return s["out"], s["k_back"], s["v_back"]


def _plain_store(s):
    case = s["case"]
    at = case["start"] + s["index"]
    page = s["tables"][0].long()[s["seq"], at // PAGE]
    _store(s["kv_pool"], page, at % PAGE,
           _rotate(s["k"], s) if case["axes"] else s["k"].float(), s["v"].float())
    at = s["index_all"]
    page = s["tables"][0].long()[s["seq_all"], at // PAGE]
    for back, x in zip((s["k_back"], s["v_back"]), _load(s["kv_pool"], page, at % PAGE)):
        back.copy_(x)
    return s["k_back"], s["v_back"]


def _plain_tree(s):
    case = s["case"]
    batch, n, w = case["batch"], s["most"], _window(case)
    start = s["start"].long()[:, None]
    pos = torch.arange(s["longest"], device="cuda")[None].expand(batch, -1)
    pos = torch.minimum(pos, start + s["nodes"].long()[:, None] - 1)
    page = _page_of(s, pos)
    k, v = (p[page, :, pos % PAGE].float() for p in (s["k_pool"], s["v_pool"]))
    # rows past a sequence's last node see its first token and are dropped below
    masks = torch.ones(batch, n, dtype=torch.int64, device="cuda")
    masks[s["seq"], s["index"]] = s["masks"]
    bits = (masks[..., None] >> torch.arange(n, device="cuda")) & 1      # [B][rows][nodes]
    at = start + bits.sum(-1) - 1                                        # position of each row
    t = torch.arange(s["longest"], device="cuda")
    node = torch.clamp(t[None] - start, min=0, max=n - 1)                # [B][keys]
    drafted = torch.gather(bits, 2, node[:, None].expand(-1, n, -1)) == 1
    drafted &= (t < start + s["nodes"].long()[:, None])[:, None]
    prefix = (at[..., None] - t < w) | (t < case["sinks"])
    seen = torch.where((t < start)[:, None], prefix, drafted)            # [B][rows][keys]
    q = torch.zeros(batch, n, HQ, DIM, device="cuda")
    q[s["seq"], s["index"]] = s["q"].float()
    q = q.view(batch, n, HKV, GROUP, DIM).permute(0, 2, 3, 1, 4).reshape(batch, HKV, GROUP * n, DIM)
    o = _softmax_products(q, k, v, seen.repeat(1, GROUP, 1)[:, None])
    o = o.view(batch, HKV, GROUP, n, DIM).permute(0, 3, 1, 2, 4).reshape(batch, n, HQ, DIM)
    s["out"].copy_(o[s["seq"], s["index"]])
    return s["out"]


def _plain_commit(s):
    layers, batch, accept = s["tables"].shape[0], s["tables"].shape[1], s["accepted"].shape[1]
    step = torch.arange(accept, device="cuda")[None]
    take = (step < s["counts"][:, None])[None].expand(layers, -1, -1)
    start = s["start"].long()[:, None]
    places = []
    for pos in (start + s["accepted"].long(), (start + step).expand(batch, -1)):
        page = torch.gather(s["tables"].long(), 2, (pos // PAGE)[None].expand(layers, -1, -1))
        places.append((page[take], (pos % PAGE)[None].expand(layers, -1, -1)[take]))
    (from_page, from_slot), (to_page, to_slot) = places
    for pool in (s["k_pool"], s["v_pool"]):
        pool[to_page, :, to_slot] = pool[from_page, :, from_slot]
    return s["k_pool"].view(torch.int16), s["v_pool"].view(torch.int16)


_PLAIN = {"decode": _plain_decode, "store": _plain_store, "tree": _plain_tree,
          "commit": _plain_commit}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["kind"]](state)


# ------------------------------------------------------------------ 64 bits, from the definition
@functools.lru_cache(maxsize=None)
def _e4m3_values():
    """What the 256 codes stand for: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    x = []
    for code in range(256):
        e, m = code >> 3 & 15, code & 7
        size = math.nan if code & 127 == 127 else \
            m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        x.append(-size if code & 128 else size)
    return torch.tensor(x, dtype=torch.float64, device="cuda")


def _exact_power(e):
    """2^e in 64 bits for whole numbers e from -1022 to 1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_stored(x):
    """x [..., 64] in 64 bits as the cache holds it: each value rounded to the nearest
    multiple of its code's step, ties to the even multiple."""
    most = x.abs().amax(-1, keepdim=True)
    e = torch.frexp(most)[1] - 10                     # 448 2^e is below `most`, unless that is 0
    for _ in range(2):
        e = torch.where(most > 448.0 * _exact_power(e), e + 1, e)
    scale = _exact_power(torch.clamp(e, min=-124))
    y = x / scale
    step = _exact_power(torch.clamp(torch.frexp(y)[1] - 1, min=-6) - 3)
    return torch.round(y / step) * step * scale


def _exact_read(s, page, head, slot):
    """K and V [tokens][64] of one head, from the bytes of their tiles."""
    tiles = s["kv_pool"][page, head]
    at = slot[:, None]
    dim = torch.arange(DIM, device="cuda")[None]
    value = _e4m3_values()
    k = value[torch.gather(tiles, 1, at * DIM + dim).long()]
    v = value[torch.gather(tiles, 1, CODES + dim // 16 * 256 + at * 16 + dim % 16).long()]
    ke = torch.gather(tiles, 1, 2 * CODES + at).long()
    ve = torch.gather(tiles, 1, 2 * CODES + PAGE + at).long()
    return k * _exact_power(ke - 127), v * _exact_power(ve - 127)


def _exact_rotated(s, x):
    cos, sin = s["cos"].double(), s["sin"].double()
    y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for i, axis in enumerate(s["axis_of_pair"]):
        row = s["axis_positions"][axis].long()
        c, t = cos[row, i][:, None], sin[row, i][:, None]
        a, b = x[:, :, i].double(), x[:, :, i + PAIRS].double()
        y[:, :, i] = a * c - b * t
        y[:, :, i + PAIRS] = b * c + a * t
    return y


def _rotated_keys(s, x):
    """The keys that are quantised: each product and the sum rounded to FP32."""
    y = torch.empty(x.shape, device="cuda")
    for i, axis in enumerate(s["axis_of_pair"]):
        row = s["axis_positions"][axis].long()
        c, t = s["cos"][row, i][:, None], s["sin"][row, i][:, None]
        a, b = x[:, :, i].float(), x[:, :, i + PAIRS].float()
        y[:, :, i] = torch.sub(torch.mul(a, c), torch.mul(b, t))
        y[:, :, i + PAIRS] = torch.add(torch.mul(b, c), torch.mul(a, t))
    return y.double()


def _exact_attend(q, k, v, hidden):
    """q [rows][4][64], k and v [keys][64], hidden [rows][keys]: [rows][4][64]."""
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for g in range(GROUP):
        x = (q[:, g] @ k.T) / math.sqrt(DIM)
        x = x.masked_fill(hidden, -math.inf)
        p = torch.exp(x - x.amax(1, keepdim=True))
        out[:, g] = (p @ v) / p.sum(1, keepdim=True)
    return out


def exact(case, seed):
    kind = case["kind"]
    if kind == "commit":
        return None                                   # copies: compared as whole numbers
    s = prepare(case, seed)
    if kind == "store":
        new_k = _exact_stored(_rotated_keys(s, s["k"]) if case["axes"] else s["k"].double())
        new_v = _exact_stored(s["v"].double())
        page = s["tables"][0].long()[s["seq_all"], s["index_all"] // PAGE]
        slot, fresh = s["index_all"] % PAGE, s["index_all"] >= case["start"]
        k = torch.empty(page.numel(), HKV, DIM, dtype=torch.float64, device="cuda")
        v = torch.empty_like(k)
        for h in range(HKV):
            k[:, h], v[:, h] = _exact_read(s, page, h, slot)
        k[fresh], v[fresh] = new_k, new_v             # both in the order of the packed rows
        return k, v
    if kind == "decode":
        q = _exact_rotated(s, s["q"]) if case["axes"] else s["q"].double()
        if case["fused"]:
            new_k = _exact_stored(_rotated_keys(s, s["k"]) if case["axes"] else s["k"].double())
            new_v = _exact_stored(s["v"].double())
        out = torch.empty(case["batch"], HQ, DIM, dtype=torch.float64, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            low = max(n - _window(case), 0)
            t = torch.cat([torch.arange(min(case["sinks"], low), device="cuda"),
                           torch.arange(low, n, device="cuda")])
            page = s["tables"][0, b].long()[t // PAGE]
            none_hidden = torch.zeros(1, t.numel(), dtype=torch.bool, device="cuda")
            for h in range(HKV):
                k, v = _exact_read(s, page, h, t % PAGE)
                if case["fused"]:
                    k[-1], v[-1] = new_k[b, h], new_v[b, h]
                heads = slice(h * GROUP, (h + 1) * GROUP)
                out[b, heads] = _exact_attend(q[b:b + 1, heads], k, v, none_hidden)[0]
        return (out, new_k, new_v) if case["fused"] else out
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    cu, masks = s["cu"].tolist(), s["masks"].tolist()
    for b, start in enumerate(s["start"].tolist()):
        n = cu[b + 1] - cu[b]
        t = torch.arange(start + n, device="cuda")
        hidden = torch.ones(n, start + n, dtype=torch.bool, device="cuda")
        for i in range(n):
            sees = [j for j in range(n) if masks[cu[b] + i] >> j & 1]
            place = start + len(sees) - 1
            hidden[i, :start] = (place - t[:start] >= _window(case)) & (t[:start] >= case["sinks"])
            hidden[i, [start + j for j in sees]] = False
        keep = ~hidden.all(0)                         # pages that nobody sees may be missing
        t, hidden = t[keep], hidden[:, keep]
        page = s["tables"][0, b].long()[t // PAGE]
        rows = slice(cu[b], cu[b + 1])
        for h in range(HKV):
            k, v = (p[page, h, t % PAGE].double() for p in (s["k_pool"], s["v_pool"]))
            heads = slice(h * GROUP, (h + 1) * GROUP)
            out[rows, heads] = _exact_attend(s["q"][rows, heads].double(), k, v, hidden)
    return out
