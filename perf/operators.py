"""Timed cases of the windowed attention, multi-axis rotary and page operators.

Each case is one call (or one call per pass) of an operator over the shared
BF16 page pool: 32 query heads over 8 KV heads, head_dim 64, 16-token pages.
Where ``own`` is false, ``run`` computes the operator with elementary torch
operations in FP32; where it is true, it makes the library's call.

  decode   attention of one new token per sequence over the last `window`
           tokens and the first `sinks` ones; fused: the token is appended
           first; axes > 0: keys and queries are rotated by that many position
           axes; window 0 stands for a window as long as the context
  prefill  the same visibility for a chunk of prompt tokens per sequence
  fill     a chunk's queries and keys rotated by several position axes, the
           keys and values written into their pages
  fork     pages of forked sequences copied, the first tokens of each
  compact  pages moved to lower ids and the block tables rewritten
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
TOKEN_BYTES = 2 * HKV * DIM * 2                      # K and V of one token


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's chat turn at the end of the context: latency of a small call
        dict(name="decode-1-w512", kind="decode", batch=1, lo=2048, hi=2048, max_seq_len=2048,
             window=512, sinks=4, fused=False, axes=0),
        # a mixed batch of image and text chats, one step with append and rotation
        dict(name="step-64-w1024-axes", kind="decode", batch=64, lo=16, hi=2048,
             max_seq_len=2048, window=1024, sinks=4, fused=True, axes=3),
        # a full serving batch of long chats behind a window
        dict(name="step-256-w4096", kind="decode", batch=256, lo=1, hi=32768, max_seq_len=32768,
             window=4096, sinks=4, fused=True, axes=1),
        # a few very long documents, everything visible
        dict(name="decode-4-128k", kind="decode", batch=4, lo=120001, hi=131072,
             max_seq_len=131072, window=0, sinks=0, fused=False, axes=0),
        # a short question
        dict(name="prefill-1x300-w128", kind="prefill", batch=1, chunk_lo=300, chunk_hi=300,
             start=0, max_seq_len=2048, window=128, sinks=4),
        # a batch of full prompts, ragged
        dict(name="prefill-8x2048-w512", kind="prefill", batch=8, chunk_lo=1201, chunk_hi=2048,
             start=0, max_seq_len=2048, window=512, sinks=4),
        # chunks that continue long documents
        dict(name="prefill-2x4096-w4096", kind="prefill", batch=2, chunk_lo=4096, chunk_hi=4096,
             start=28600, max_seq_len=32768, window=4096, sinks=16),
        # a thumbnail and a caption
        dict(name="fill-1x77", kind="fill", batch=1, chunk_lo=77, chunk_hi=77, start=0,
             max_seq_len=2048, axes=3),
        # a batch of video prompts
        dict(name="fill-8x2048", kind="fill", batch=8, chunk_lo=1536, chunk_hi=2048, start=0,
             max_seq_len=2048, axes=3),
        # one prompt sampled several ways: the last page of each of 16 layers per sample
        dict(name="fork-8", kind="fork", pairs=128, num_pages=4096),
        # a quarter of a pool moved down after many sequences ended
        dict(name="compact-16384", kind="compact", pairs=16384, num_pages=65536, layers=16,
             max_batch=256),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "prefill", "prefill", "fill", "fork", "compact"])
    if kind == "decode":
        longest = _log_int(rng, 40, 131072)
        # the visible tokens of the largest listed cases bound the batch
        window = 0 if rng.random() < 0.2 else _log_int(rng, 16, 8192)
        seen = min(longest, window or longest)
        batch = _log_int(rng, 1, max(1, min(256, (1 << 20) // seen // 2)))
        return dict(kind=kind, batch=batch, lo=rng.randint(1, longest), hi=longest,
                    max_seq_len=SHORT_CONTEXT if longest <= SHORT_CONTEXT
                    else -(-longest // PAGE) * PAGE,
                    window=window, sinks=rng.choice([0, 1, 4, rng.randint(0, 70)]),
                    fused=rng.random() < 0.6, axes=rng.choice([0, 1, 2, 3]))
    if kind in ("prefill", "fill"):
        long = rng.random() < 0.4
        chunk = _log_int(rng, 5, 4096 if long else 2048)
        start = _log_int(rng, 1, 28000) if long else rng.randint(0, SHORT_CONTEXT - chunk)
        batch = _log_int(rng, 1, max(1, min(16, 12000 // chunk)))
        lo = rng.randint(1, chunk)
        total = start + chunk
        base = dict(kind=kind, batch=batch, chunk_lo=lo, chunk_hi=chunk, start=start,
                    max_seq_len=SHORT_CONTEXT if total <= SHORT_CONTEXT
                    else -(-total // PAGE) * PAGE)
        if kind == "fill":
            return dict(base, axes=rng.choice([1, 2, 3]))
        window = _log_int(rng, 1, 4096)
        return dict(base, window=window, sinks=rng.choice([0, 1, 4, rng.randint(0, 130)]))
    if kind == "fork":
        pairs = _log_int(rng, 1, 4096)
        return dict(kind=kind, pairs=pairs, num_pages=2 * pairs + rng.randint(1, 500))
    pairs = _log_int(rng, 20, 12000)
    return dict(kind=kind, pairs=pairs, num_pages=2 * pairs + rng.randint(1, 4000),
                layers=rng.randint(1, 16), max_batch=_log_int(rng, 1, 256))


# ------------------------------------------------------------------ sizes that a case fixes
def _spread(lo, hi, n):
    """n lengths from lo to hi, even in their logarithm (the seed only orders them)."""
    if n == 1:
        return np.array([hi], np.int64)
    x = np.exp(np.linspace(math.log(lo), math.log(hi), n))
    return np.clip(np.rint(x).astype(np.int64), lo, hi)


def _window(case):
    return case["window"] or case["max_seq_len"]


def _needed_pages(case, last, first):
    """Which logical pages of each sequence hold a token that a query at a
    position in [first, last] may see: bool [sequences][pages of a row]."""
    page = np.arange(case["max_seq_len"] // PAGE)[None, :]
    last, first = np.asarray(last)[:, None], np.asarray(first)[:, None]
    lo = np.maximum(first - _window(case) + 1, 0) // PAGE
    return (page <= last // PAGE) & ((page >= lo) | (page * PAGE < case["sinks"]))


def _chunks(case):
    return _spread(case["chunk_lo"], case["chunk_hi"], case["batch"])


def work(case):
    if case["kind"] == "decode":
        lens = _spread(case["lo"], case["hi"], case["batch"])
        w, s = _window(case), case["sinks"]
        seen = np.minimum(lens, w) + np.clip(np.minimum(s, lens - w), 0, None)
        per_seq = HQ * DIM * (2 + 4) + 4 + (TOKEN_BYTES if case["fused"] else 0)
        rope = 2 * 4 * PAIRS if case["axes"] else 0
        return {"bytes": int(seen.sum()) * TOKEN_BYTES + case["batch"] * (per_seq + rope),
                "flops": int(seen.sum()) * HQ * DIM * 4}
    if case["kind"] == "prefill":
        n, start, w, s = _chunks(case), case["start"], _window(case), case["sinks"]
        keys = np.minimum(start + n, w + n - 1) + np.clip(np.minimum(s, start - w + 1), 0, None)
        pairs = 0
        for m in n:
            p = np.arange(start, start + m)
            pairs += int((np.minimum(p + 1, w) + np.clip(np.minimum(s, p + 1 - w), 0, None)).sum())
        return {"bytes": int(n.sum()) * HQ * DIM * (2 + 4) + int(keys.sum()) * TOKEN_BYTES,
                "flops": pairs * HQ * DIM * 4}
    if case["kind"] == "fill":
        t = int(_chunks(case).sum())
        return {"bytes": t * (2 * (HQ * DIM * 2 + TOKEN_BYTES) + 4 * case["axes"]),
                "flops": t * (HQ + HKV) * DIM * 3}
    if case["kind"] == "fork":
        tokens = int(_tokens(case["pairs"]).sum())
        return {"bytes": 2 * tokens * TOKEN_BYTES + 12 * case["pairs"], "flops": 0}
    table = case["layers"] * case["max_batch"] * (SHORT_CONTEXT // PAGE) * 4
    return {"bytes": case["pairs"] * (2 * PAGE * TOKEN_BYTES + 8) + table, "flops": 0}


def _tokens(pairs):
    return np.arange(pairs, dtype=np.int64) * 7 % PAGE + 1


# ------------------------------------------------------------------ inputs
def _pools(gen, num_pages):
    """K and V pools of N(0, 1) values, drawn a part at a time."""
    out = []
    for _ in range(2):
        pool = torch.empty(num_pages, HKV, PAGE, DIM, dtype=torch.bfloat16, device="cuda")
        for i in range(0, num_pages, 8192):
            part = pool[i:i + 8192]
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
        out.append(pool)
    return out


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)


def _angles(rows):
    """cos and sin of p * 10000^(-2 i / 64), computed in 64 bits."""
    p = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None]
    f = 10000.0 ** (-torch.arange(PAIRS, dtype=torch.float64, device="cuda") / PAIRS)
    return torch.cos(p * f).float(), torch.sin(p * f).float()


def _tables(gen, needed, num_pages):
    """Block table [1][sequences][pages]: shuffled ids for the pages a sequence needs, else -1."""
    ids = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    need = torch.from_numpy(needed).cuda()
    table = torch.full(need.shape, -1, dtype=torch.int32, device="cuda")
    table[need] = ids[: int(needed.sum())]
    return table[None].contiguous()


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = np.random.RandomState(seed % (1 << 32))
    s = {"case": case}
    kind = case["kind"]
    if kind == "decode":
        lens = order.permutation(_spread(case["lo"], case["hi"], case["batch"]))
        needed = _needed_pages(case, lens - 1, lens - 1)
        s["num_pages"] = int(needed.sum()) + 3
        s["tables"] = _tables(gen, needed, s["num_pages"])
        s["k_pool"], s["v_pool"] = _pools(gen, s["num_pages"])
        s["lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
        s["q"] = _normal(gen, case["batch"], HQ, DIM)
        if case["fused"]:
            s["k"], s["v"] = _normal(gen, case["batch"], HKV, DIM), _normal(gen, case["batch"], HKV, DIM)
        if case["axes"]:
            back = torch.randint(0, 300, (case["axes"], case["batch"]), generator=gen, device="cuda")
            _rope_inputs(s, torch.clamp(s["lens"][None, :] - 1 - back, min=0), case["max_seq_len"])
        s["out"] = torch.zeros(case["batch"], HQ, DIM, device="cuda")
    elif kind in ("prefill", "fill"):
        n = order.permutation(_chunks(case))
        start = np.full(case["batch"], case["start"], np.int64)
        sizes = case if kind == "prefill" else dict(case, window=0, sinks=0)
        needed = _needed_pages(sizes, start + n - 1, start)
        if kind == "fill":   # only the pages that are written
            needed &= np.arange(needed.shape[1])[None, :] >= case["start"] // PAGE
        s["num_pages"] = int(needed.sum()) + 3
        s["tables"] = _tables(gen, needed, s["num_pages"])
        s["k_pool"], s["v_pool"] = _pools(gen, s["num_pages"])
        s["total"], s["max_chunk"] = int(n.sum()), int(n.max())
        cu = np.concatenate([[0], np.cumsum(n)])
        s["cu"] = torch.from_numpy(cu.astype(np.int32)).cuda()
        s["start"] = torch.from_numpy(start.astype(np.int32)).cuda()
        # row -> (sequence, index in its chunk)
        s["seq"] = torch.repeat_interleave(torch.arange(case["batch"], device="cuda"),
                                           torch.from_numpy(n).cuda())
        s["index"] = torch.arange(s["total"], device="cuda") - s["cu"].long()[s["seq"]]
        s["q"] = _normal(gen, s["total"], HQ, DIM)
        if kind == "fill":
            s["k"], s["v"] = _normal(gen, s["total"], HKV, DIM), _normal(gen, s["total"], HKV, DIM)
            _rope_inputs(s, _grid_positions(case["axes"], s["index"] + case["start"]),
                         max(case["max_seq_len"], 512))
            s["q_out"] = torch.empty_like(s["q"])
        else:
            s["out"] = torch.zeros(s["total"], HQ, DIM, device="cuda")
    else:
        m, pages = case["pairs"], case["num_pages"]
        s["num_pages"] = pages
        s["k_pool"], s["v_pool"] = _pools(gen, pages)
        if kind == "fork":
            ids = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
            # several samples of one prompt share a source page
            s["src"], s["dst"] = ids[:m][torch.arange(m, device="cuda") // 4].contiguous(), ids[m:2 * m].contiguous()
            s["tokens"] = torch.from_numpy(order.permutation(_tokens(m)).astype(np.int32)).cuda()
        else:
            used = pages - m     # pages in use at the end occupy [0, used)
            high = torch.randperm(m, generator=gen, device="cuda") + used
            low = torch.randperm(used, generator=gen, device="cuda")
            s["src"], s["dst"] = high.to(torch.int32), low[:m].to(torch.int32).contiguous()
            shape = (case["layers"], case["max_batch"], SHORT_CONTEXT // PAGE)
            held = torch.cat([high, low[m:]])      # the pages that the tables name
            pick = torch.randint(0, held.numel(), shape, generator=gen, device="cuda")
            table = held[pick].to(torch.int32)
            table[torch.rand(shape, generator=gen, device="cuda") < 0.3] = -1
            s["tables"] = table.contiguous()
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
    pool = _handle(case.get("layers", 1), s["num_pages"],
                   case.get("max_batch", case.get("batch", 1)),
                   case.get("max_seq_len", SHORT_CONTEXT))
    if case.get("axes") and "rope" not in s:      # kept beside the tables
        s["rope"] = pkv.pkv_axes_rope(s["cos"], s["sin"], s["axis_of_pair"])
    if kind == "decode":
        window = _window(case)
        rope = dict(rope=s["rope"], rope_positions=s["axis_positions"]) if case["axes"] else {}
        if case["fused"]:
            pkv.pkv_window_append_attend(pool, 0, s["q"], s["k"], s["v"], s["k_pool"],
                                         s["v_pool"], s["tables"], s["lens"], s["out"], window,
                                         sinks=case["sinks"], **rope)
            return s["out"], s["k_pool"], s["v_pool"]
        pkv.pkv_window_attention(pool, 0, s["q"], s["k_pool"], s["v_pool"], s["tables"],
                                 s["lens"], s["out"], window, sinks=case["sinks"], **rope)
        return s["out"]
    if kind == "prefill":
        pkv.pkv_window_prefill_attention(pool, 0, s["q"], s["k_pool"], s["v_pool"], s["tables"],
                                         s["cu"], s["start"], s["out"], s["max_chunk"],
                                         _window(case), sinks=case["sinks"])
        return s["out"]
    if kind == "fill":
        pkv.pkv_prefill_fill_axes(pool, 0, s["q"], s["k"], s["v"], s["q_out"], s["k_pool"],
                                  s["v_pool"], s["tables"], s["cu"], s["start"], s["rope"],
                                  s["axis_positions"], s["max_chunk"])
        return s["q_out"], s["k_pool"], s["v_pool"]
    if kind == "fork":
        pkv.pkv_copy_pages(pool, s["src"], s["dst"], s["k_pool"], s["v_pool"], tokens=s["tokens"])
        return _bits(s["k_pool"]), _bits(s["v_pool"])
    pkv.pkv_compact_pages(pool, s["src"], s["dst"], s["k_pool"], s["v_pool"], s["tables"])
    return _bits(s["k_pool"]), _bits(s["v_pool"]), s["tables"]


def _bits(pool):
    """A pool's bits as whole numbers: what is copied has to be equal."""
    return pool.view(torch.int16)


# ------------------------------------------------------------------ plain form
def _rotate(x, s):
    """x [tokens][heads][64] rotated in FP32, dim i with dim i + 32, pair i by
    the position on its axis."""
    at = s["axis_positions"].long()[s["axis_index"]].T          # [tokens][32]
    pair = torch.arange(PAIRS, device="cuda")
    c, sn = s["cos"][at, pair][:, None], s["sin"][at, pair][:, None]
    a, b = x[..., :PAIRS].float(), x[..., PAIRS:].float()
    return torch.cat([a * c - b * sn, b * c + a * sn], -1)


def _gather(s, pos):
    """K and V [sequences][keys][8][64] in FP32 of the tokens at pos [sequences][keys]."""
    page = torch.gather(s["tables"][0].long(), 1, pos // PAGE)
    page = torch.clamp(page, min=0)
    return s["k_pool"][page, :, pos % PAGE].float(), s["v_pool"][page, :, pos % PAGE].float()


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
    q = s["q"].float()
    lens = s["lens"].long()
    if case["axes"]:
        q = _rotate(s["q"], s)
    if case["fused"]:
        k = _rotate(s["k"], s).to(torch.bfloat16) if case["axes"] else s["k"]
        at = lens - 1
        page = torch.gather(s["tables"][0].long(), 1, (at // PAGE)[:, None])[:, 0]
        s["k_pool"][page, :, at % PAGE] = k
        s["v_pool"][page, :, at % PAGE] = s["v"]
    window = min(_window(case), case["hi"])
    sinks = min(case["sinks"], case["hi"])
    first = lens[:, None] - window                              # of the window
    head = torch.arange(sinks, device="cuda")[None].expand(lens.numel(), -1)
    tail = first + torch.arange(window, device="cuda")[None]
    pos = torch.cat([head, tail], 1)
    seen = torch.cat([head < first, tail >= 0], 1)
    k, v = _gather(s, torch.clamp(torch.minimum(pos, lens[:, None] - 1), min=0))
    o = _softmax_products(q.view(-1, HKV, GROUP, DIM), k, v, seen[:, None, None])
    s["out"].copy_(o.reshape(-1, HQ, DIM))
    return (s["out"], s["k_pool"], s["v_pool"]) if case["fused"] else s["out"]


def _plain_prefill(s):
    case = s["case"]
    batch, n, w = case["batch"], s["max_chunk"], _window(case)
    start, sinks = case["start"], min(case["sinks"], case["start"] + s["max_chunk"])
    count = (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    low = max(start - w + 1, 0)                                 # first windowed key of the chunk
    head = torch.arange(min(sinks, low), device="cuda")
    pos = torch.cat([head, torch.arange(low, start + n, device="cuda")])
    pos = pos[None].expand(batch, -1)
    k, v = _gather(s, torch.minimum(pos, start + count - 1))
    at = start + torch.arange(n, device="cuda")[:, None]
    seen = (pos[0] <= at) & ((pos[0] > at - w) | (pos[0] < sinks))     # [rows][keys]
    q = torch.zeros(batch, n, HQ, DIM, device="cuda")
    q[s["seq"], s["index"]] = s["q"].float()
    q = q.view(batch, n, HKV, GROUP, DIM).permute(0, 2, 3, 1, 4).reshape(batch, HKV, GROUP * n, DIM)
    o = _softmax_products(q, k, v, seen.repeat(GROUP, 1))
    o = o.view(batch, HKV, GROUP, n, DIM).permute(0, 3, 1, 2, 4).reshape(batch, n, HQ, DIM)
    s["out"].copy_(o[s["seq"], s["index"]])
    return s["out"]


def _plain_fill(s):
    case = s["case"]
    s["q_out"].copy_(_rotate(s["q"], s))
    at = case["start"] + s["index"]
    page = s["tables"][0].long()[s["seq"], at // PAGE]
    s["k_pool"][page, :, at % PAGE] = _rotate(s["k"], s).to(torch.bfloat16)
    s["v_pool"][page, :, at % PAGE] = s["v"]
    return s["q_out"], s["k_pool"], s["v_pool"]


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for pool in (s["k_pool"], s["v_pool"]):
        moved = pool[src]
        if "tokens" in s:
            keep = torch.arange(PAGE, device="cuda")[None] < s["tokens"][:, None]
            moved = torch.where(keep[:, None, :, None], moved, pool[dst])
        pool[dst] = moved
    if "tables" not in s:
        return _bits(s["k_pool"]), _bits(s["v_pool"])
    to = torch.arange(s["num_pages"], dtype=torch.int32, device="cuda")
    to[src] = s["dst"]
    table = s["tables"]
    table.copy_(torch.where(table >= 0, to[torch.clamp(table, min=0).long()], table))
    return _bits(s["k_pool"]), _bits(s["v_pool"]), table


_PLAIN = {"decode": _plain_decode, "prefill": _plain_prefill, "fill": _plain_fill,
          "fork": _plain_copy, "compact": _plain_copy}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["kind"]](state)


# ------------------------------------------------------------------ 64 bits, from the definition
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


def _stored_keys(s, x):
    """The keys as a page holds them: each product and the sum rounded to FP32,
    then to BF16."""
    cos, sin = s["cos"], s["sin"]
    y = torch.empty_like(x)
    for i, axis in enumerate(s["axis_of_pair"]):
        row = s["axis_positions"][axis].long()
        c, t = cos[row, i][:, None], sin[row, i][:, None]
        a, b = x[:, :, i].float(), x[:, :, i + PAIRS].float()
        y[:, :, i] = torch.sub(torch.mul(a, c), torch.mul(b, t))
        y[:, :, i + PAIRS] = torch.add(torch.mul(b, c), torch.mul(a, t))
    return y


def _exact_rows(s, b, q, at, keys):
    """Attention of the queries q [rows][32][64] at positions `at` over the
    tokens `keys` of sequence b, one KV head at a time."""
    case = s["case"]
    w, sinks = _window(case), case["sinks"]
    row = s["tables"][0, b].long()
    page, slot = row[keys // PAGE], keys % PAGE
    d = at[:, None] - keys[None, :]
    hidden = (d < 0) | ((d >= w) & (keys[None, :] >= sinks))
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for h in range(HKV):
        k, v = s["k_pool"][page, h, slot].double(), s["v_pool"][page, h, slot].double()
        for g in range(h * GROUP, (h + 1) * GROUP):
            x = (q[:, g].double() @ k.T) / math.sqrt(DIM)
            p = torch.exp(x.masked_fill(hidden, -math.inf)
                          - x.masked_fill(hidden, -math.inf).amax(1, keepdim=True))
            out[:, g] = (p @ v) / p.sum(1, keepdim=True)
    return out


def _visible(lo, hi, sinks):
    """Token positions below `sinks` or in [lo, hi)."""
    lo = max(lo, 0)
    return torch.cat([torch.arange(min(sinks, lo), device="cuda"),
                      torch.arange(lo, hi, device="cuda")])


def exact(case, seed):
    kind = case["kind"]
    if kind in ("fork", "compact"):
        return None                                   # copies: compared as whole numbers
    s = prepare(case, seed)
    if kind == "decode":
        q = _exact_rotated(s, s["q"]) if case["axes"] else s["q"].double()
        pools = (None, None)
        if case["fused"]:
            new = _exact_rotated(s, s["k"]) if case["axes"] else s["k"].double()
            stored = _stored_keys(s, s["k"]) if case["axes"] else s["k"]
            pools = (s["k_pool"].double(), s["v_pool"].double())
            for b in range(case["batch"]):
                p = int(s["lens"][b]) - 1
                page = int(s["tables"][0, b, p // PAGE])
                pools[0][page, :, p % PAGE] = new[b]
                pools[1][page, :, p % PAGE] = s["v"][b].double()
                # what attention reads is the stored key
                s["k_pool"][page, :, p % PAGE] = stored[b]
                s["v_pool"][page, :, p % PAGE] = s["v"][b]
        out = torch.empty(case["batch"], HQ, DIM, dtype=torch.float64, device="cuda")
        for b in range(case["batch"]):
            n = int(s["lens"][b])
            keys = _visible(n - _window(case), n, case["sinks"])
            out[b] = _exact_rows(s, b, q[b:b + 1], torch.tensor([n - 1], device="cuda"), keys)[0]
        return (out, *pools) if case["fused"] else out
    if kind == "prefill":
        out = torch.empty(s["total"], HQ, DIM, dtype=torch.float64, device="cuda")
        cu, start = s["cu"].tolist(), case["start"]
        for b in range(case["batch"]):
            for r in range(cu[b], cu[b + 1], 1024):   # a part of the rows at a time
                e = min(r + 1024, cu[b + 1])
                at = torch.arange(start + r - cu[b], start + e - cu[b], device="cuda")
                keys = _visible(int(at[0]) - _window(case) + 1, int(at[-1]) + 1, case["sinks"])
                out[r:e] = _exact_rows(s, b, s["q"][r:e], at, keys)
        return out
    q, k = _exact_rotated(s, s["q"]), _exact_rotated(s, s["k"])
    k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
    at = case["start"] + s["index"]
    page = s["tables"][0][s["seq"], at // PAGE].long()
    for h in range(HKV):
        k_pool[page, h, at % PAGE] = k[:, h]
        v_pool[page, h, at % PAGE] = s["v"][:, h].double()
    return q, k_pool, v_pool
