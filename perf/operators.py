"""Cases of the decoding operators: attention over a paged key-value cache,
the cache's upkeep, and guided logits.

A case is a dict of plain values; its ``op`` names what one pass runs:

  decode   one new token a row attends over its pages (paged_attention)
  prompt   ragged runs of new tokens attend over their pages, causally, with
           an optional sliding window and first tokens that stay visible
           (prompt_attention)
  append   new keys and values go into the pages (cache_append)
  turn     a scheduler's turn: finished rows give their pages back, take
           forks of other rows and room for one more token (cache_free,
           cache_fork, cache_extend)
  compact  live pages move to the front of the pool (cache_compact)
  copy     listed pages are copied to others (cache_copy)
  logits   the guided combine of two branches' logits, penalties of repeated
           tokens, biases, temperature and a grammar mask (guided_logits)

``run`` computes them with elementary torch operations in 32 bits, or with the
package's kernels where ``own`` is true.  Row lengths and page counts follow
from the case alone (a scheduler knows them on the host); all values, and
which page holds what, follow from the seed.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one sample's two branches, early in a sequence: latency
        dict(name="decode_pair", op="decode", rows=2, heads=32, kv_heads=8, dim=128, page=16, length=700,
             q="bf16", kv="bf16", window=0, sinks=0),
        # a serving batch of mixed ages on an 8-bit cache
        dict(name="decode_batch_e4m3", op="decode", rows=96, heads=32, kv_heads=8, dim=128, page=32, length=8192,
             q="bf16", kv="e4m3", window=0, sinks=0),
        # few rows with a very long past: the cache's length is what there is to split
        dict(name="decode_long", op="decode", rows=4, heads=64, kv_heads=8, dim=128, page=64, length=131072,
             q="bf16", kv="bf16", window=0, sinks=0),
        # short runs of tokens after a cached prefix, in full precision
        dict(name="prompt_chunk_f32", op="prompt", rows=3, heads=16, kv_heads=16, dim=64, page=16, new=61, length=1500,
             q="f32", kv="f32", window=0, sinks=0),
        # a batch of ragged prompts, nothing cached before
        dict(name="prompt_batch", op="prompt", rows=8, heads=32, kv_heads=8, dim=128, page=16, new=2048, length=0,
             q="bf16", kv="bf16", window=0, sinks=0),
        # one long prompt with a sliding window and four sinks
        dict(name="prompt_window", op="prompt", rows=1, heads=32, kv_heads=8, dim=128, page=64, new=8192, length=0,
             q="bf16", kv="bf16", window=1024, sinks=4),
        # one token a row into an 8-bit cache
        dict(name="append_token_e4m3", op="append", rows=96, kv_heads=8, dim=128, page=32, new=1, length=1024,
             q="bf16", kv="e4m3"),
        # prompts into a bf16 cache, from the slices of a fused projection
        dict(name="append_prompt", op="append", rows=8, kv_heads=8, dim=128, page=16, new=2048, length=77,
             q="bf16", kv="bf16"),
        # the upkeep of one step: an eighth of the rows end, the slots take forks
        dict(name="pages_turn", op="turn", rows=64, moved=8, planes=16, kv_heads=8, dim=128, page=16, length=500,
             kv="bf16"),
        # a pool with holes, two fifths of it free
        dict(name="pages_compact", op="compact", rows=128, planes=16, kv_heads=8, dim=128, page=16, length=400,
             free=40, kv="bf16"),
        # one guided sample over a small odd vocabulary: latency
        dict(name="logits_one", op="logits", n=1, vocab=32001, q="bf16", out="f32", guided=100, history=300,
             bias=8, mask=True),
        # a full batch, three quarters of it guided
        dict(name="logits_batch", op="logits", n=256, vocab=131136, q="bf16", out="f32", guided=75, history=2048,
             bias=64, mask=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "prompt", "prompt", "prompt", "append", "turn", "compact", "copy",
                     "logits", "logits"])
    kv_heads = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    page = rng.choice([16, 32, 48, 64, 128])
    q, kv = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f32", "f32")])
    window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 1, 4096), rng.choice([0, 1, 4, 16]))])
    if op == "decode":
        rows, length = _log(rng, 1, 256), _log(rng, 1, 131072)
        length = max(1, min(length, int(2 ** 31 // (rows * kv_heads * dim * 2 * SIZE[kv])), 2 ** 29 // (rows * kv_heads * dim)))
        return dict(op=op, rows=rows, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, length=length,
                    q=q, kv=kv, window=window, sinks=sinks)
    if op == "prompt":
        rows, new = _log(rng, 1, 32), _log(rng, 1, 4096)
        length = rng.choice([0, _log(rng, 1, 16384)])
        while rows * kv_heads * group * new * (new + length) > 2 ** 30 or rows * kv_heads * dim * (new + length) > 2 ** 28:
            rows, new, length = max(1, rows // 2), max(1, new * 2 // 3), length * 2 // 3
        return dict(op=op, rows=rows, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, page=page, new=new,
                    length=length, q=q, kv=kv, window=window, sinks=sinks)
    if op == "append":
        rows, new = rng.choice([(_log(rng, 1, 256), 1), (_log(rng, 1, 16), _log(rng, 1, 2048))])
        new = max(1, min(new, 2 ** 24 // (rows * kv_heads * dim)))
        return dict(op=op, rows=rows, kv_heads=kv_heads, dim=dim, page=page, new=new, length=rng.choice([0, _log(rng, 1, 500)]),
                    q=q, kv=kv)
    if op in ("turn", "compact"):
        rows, length, planes = _log(rng, 3, 128), _log(rng, 1, 2000), 2 * _log(rng, 1, 12)
        while rows * length * planes * kv_heads * dim * SIZE[kv] > 2 ** 29:
            rows, length = max(3, rows * 2 // 3), max(1, length * 2 // 3)
        case = dict(op=op, rows=rows, planes=planes, kv_heads=kv_heads, dim=dim, page=page, length=length, kv=kv)
        case.update({"moved": rng.randint(1, max(1, rows // 2))} if op == "turn" else {"free": rng.randint(0, 90)})
        return case
    if op == "copy":
        planes = 2 * _log(rng, 1, 12)
        pages = max(2, min(_log(rng, 2, 2048), 2 ** 29 // (planes * page * kv_heads * dim * SIZE[kv])))
        return dict(op=op, pages=pages, moved=rng.randint(1, max(1, pages // 2)), planes=planes, kv_heads=kv_heads, dim=dim,
                    page=page, kv=kv)
    n, vocab = _log(rng, 1, 256), _log(rng, 1000, 131136)
    return dict(op="logits", n=n, vocab=vocab, q=rng.choice(["bf16", "f32"]), out=rng.choice(["f32", "bf16"]),
                guided=rng.choice([0, 50, 75, 100]), history=rng.choice([0, _log(rng, 1, 8192)]),
                bias=rng.choice([0, 1, 30, 300]), mask=rng.choice([True, False]))


# ---- what follows from the case alone ------------------------------------------

def _host(case):
    """The host's random numbers of a case: its lengths, not its values."""
    return random.Random(",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))


def _spread(rng, n, top, low=1):
    """n lengths up to ``top``, the first one ``top`` itself."""
    return [top if i == 0 else rng.randint(min(low, top), top) for i in range(n)]


def _lengths(case):
    """(new tokens, tokens in the cache with them) of every row."""
    rng, op, rows = _host(case), case["op"], case["rows"]
    if op == "decode":  # a long past is nearly the same for all rows, others are of any age
        kv = _spread(rng, rows, case["length"], case["length"] * 3 // 4 if case["length"] > 16384 else 1)
        return [1] * rows, kv
    new = _spread(rng, rows, case["new"], case["new"] // 4) if case["new"] > 1 else [1] * rows
    past = [0] * rows if not case["length"] else _spread(rng, rows, case["length"], 0)
    return new, [a + b for a, b in zip(new, past)]


def _seen(case):
    """Pairs of a query and a token that it sees, over all rows."""
    w, s, total = case["window"], case["sinks"], 0
    for a, b in zip(*_lengths(case)):
        p = np.arange(b - a, b, dtype=np.int64)
        total += int((p + 1 if not w else np.minimum(w, p + 1) + np.minimum(s, np.maximum(p + 1 - w, 0))).sum())
    return total


def _touched(case):
    """Cached tokens that some query sees, over all rows."""
    w, s, total = case["window"], case["sinks"], 0
    for a, b in zip(*_lengths(case)):
        first = max(0, b - a + 1 - w) if w else 0
        total += b - first + min(s, first)
    return total


def _held(case):
    """Pages that each row holds in a turn or before a compaction, with room
    left in the pool: (row lengths, pages of each, pages of the pool)."""
    rng = _host(case)
    lengths = _spread(rng, case["rows"], case["length"])
    pages = [-(-n // case["page"]) for n in lengths]
    live = sum(pages)
    if case["op"] == "compact":
        return lengths, pages, live + max(1, live * case["free"] // (100 - case["free"]))
    return lengths, pages, live + 2 * case["moved"] + 1


def _page_bytes(case):
    return case["kv_heads"] * case["page"] * case["dim"] * SIZE[case["kv"]]


def work(case):
    op = case["op"]
    if op in ("decode", "prompt"):
        new, _ = _lengths(case)
        io = 2 * sum(new) * case["heads"] * case["dim"] * SIZE[case["q"]]
        return {"bytes": _touched(case) * case["kv_heads"] * case["dim"] * 2 * SIZE[case["kv"]] + io,
                "flops": 4 * _seen(case) * case["heads"] * case["dim"]}
    if op == "append":
        return {"bytes": 2 * sum(_lengths(case)[0]) * case["kv_heads"] * case["dim"] * (SIZE[case["q"]] + SIZE[case["kv"]])}
    if op == "turn":
        lengths, pages, total = _held(case)
        part = sum(1 for n in lengths[case["moved"]:][:case["moved"]] if n % case["page"])
        return {"bytes": 2 * part * case["planes"] * _page_bytes(case) + 4 * total + 8 * sum(pages[:2 * case["moved"]])}
    if op == "compact":
        # the share of live pages that lie behind as many live ones as there are, on average
        _, pages, total = _held(case)
        live = sum(pages)
        return {"bytes": int(2 * live * (total - live) / total * case["planes"] * _page_bytes(case)) + 8 * (total + live)}
    if op == "copy":
        return {"bytes": 2 * case["moved"] * case["planes"] * _page_bytes(case)}
    n, v = case["n"], case["vocab"]
    return {"bytes": n * v * SIZE[case["out"]] + (n + n * case["guided"] // 100) * v * SIZE[case["q"]]
            + 4 * n * (case["history"] + 2 * case["bias"]) + (n * v // 8 if case["mask"] else 0)}


# ---- inputs --------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    t = torch.empty(shape, device=DEV, dtype=torch.bfloat16 if dtype == torch.float8_e4m3fn else dtype)
    t.normal_(0.0, scale, generator=g)
    return t.to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _tables(g, pages, total, width):
    """A block table whose rows hold ``pages[r]`` pages of a pool of ``total``
    in shuffled order, -1 behind them."""
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(pages), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = order[at:at + n]
        at += n
    return table


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    s = {"case": dict(case)}
    if op == "logits":
        return _prepare_logits(s, case, g)
    kv = TYPES[case["kv"]]
    if op == "copy":
        pool = _normal(g, (case["planes"], case["pages"], case["kv_heads"], case["page"], case["dim"]), kv)
        pick = torch.randperm(case["pages"], generator=g, device=DEV).to(torch.int32)
        return dict(s, pool=pool, src=pick[:case["moved"]].clone(),
                    dst=pick[case["pages"] - case["moved"]:].clone())
    if op in ("turn", "compact"):
        lengths, pages, total = _held(case)
        pool = _normal(g, (case["planes"], total, case["kv_heads"], case["page"], case["dim"]), kv)
        table = _tables(g, pages, total, max(pages) + 1)
        refs = torch.zeros(total, dtype=torch.int32, device=DEV)
        held = table[table >= 0].long()
        refs[held] = 1
        s.update(pool=pool, table=table, length=_i32(lengths), refs=refs)
        if op == "turn":
            m = case["moved"]
            src = [m + i % (case["rows"] - m) for i in range(m)]
            s.update(done=_i32(list(range(m))), src=_i32(src), one=_i32([1] * m))
        else:
            s.update(table_out=torch.empty_like(table), refs_out=torch.empty_like(refs))
        return s
    new, lens = _lengths(case)
    pages = [-(-n // case["page"]) for n in lens]
    total = sum(pages) + 3
    pool = _normal(g, (2, total, case["kv_heads"], case["page"], case["dim"]), kv)
    s.update(pool=pool, table=_tables(g, pages, total, max(pages)), length=_i32(lens), max_len=max(lens), max_new=max(new))
    # 8-bit pages stand for value times a scale of their head, as a calibrated cache has it
    s["k_scale"] = s["v_scale"] = None
    if case["kv"] == "e4m3":
        s["k_scale"], s["v_scale"] = (torch.rand(case["kv_heads"], generator=g, device=DEV) * 0.5 + 0.5 for _ in range(2))
    s["offset"] = _i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    if op == "append":
        qkv = _normal(g, (sum(new), 3, case["kv_heads"], case["dim"]), TYPES[case["q"]], 2.0)
        s["k"], s["v"] = qkv[:, 1], qkv[:, 2]  # strided slices of one projection
        return s
    s["q"] = _normal(g, (sum(new), case["heads"], case["dim"]), TYPES[case["q"]], 1.5)
    s["scale"] = case["dim"] ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV) if op == "decode" else None
    return s


def _prepare_logits(s, case, g):
    n, v = case["n"], case["vocab"]
    m = n * case["guided"] // 100
    s["logits"] = _normal(g, (m + n, v), TYPES[case["q"]], 3.0)
    scale = torch.rand(n, generator=g, device=DEV) * 6.0 + 1.5
    urow = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    pick = torch.randperm(n, generator=g, device=DEV)[:m].sort()[0]
    urow[pick] = torch.arange(m, dtype=torch.int32, device=DEV)
    s.update(scale=torch.where(urow < 0, torch.ones_like(scale), scale), uncond_row=urow,
             cond_row=torch.arange(m, m + n, dtype=torch.int32, device=DEV))
    s["out"] = torch.empty((n, v), dtype=TYPES[case["out"]], device=DEV)
    s["temperature"] = torch.rand(n, generator=g, device=DEV) + 0.4
    rand = lambda lo, hi: torch.rand(n, generator=g, device=DEV) * (hi - lo) + lo  # noqa: E731
    s["repetition"], s["presence"], s["frequency"] = rand(1.0, 1.4), rand(0.0, 0.8), rand(0.0, 0.5)
    s["history"] = s["history_len"] = s["prompt_len"] = None
    if case["history"]:
        h = case["history"]
        # tokens as texts have them: few of them often, many seldom
        s["history"] = (torch.rand((n, h), generator=g, device=DEV) ** 3 * v).to(torch.int32).clamp_(max=v - 1)
        s["history_len"] = torch.randint(h // 2, h + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
        s["prompt_len"] = (s["history_len"] * torch.rand(n, generator=g, device=DEV)).to(torch.int32)
    s["bias_ids"] = s["bias"] = None
    if case["bias"]:
        step = max(1, v // case["bias"])  # distinct tokens, at any place
        at = torch.arange(case["bias"], device=DEV) * step
        s["bias_ids"] = ((at + torch.randint(0, v, (n, 1), generator=g, device=DEV)) % v).to(torch.int32).contiguous()
        s["bias"] = torch.randn((n, case["bias"]), generator=g, device=DEV) * 4.0
    s["mask"] = None
    if case["mask"]:
        words = torch.randint(-2 ** 31, 2 ** 31, (n, (v + 31) // 32), generator=g, device=DEV)
        s["mask"] = words.to(torch.int32)
    return s


# ---- the operators in their plain form -------------------------------------------

def _gathered(cache, table, scale):
    """The rows' pages one after another, in 32 bits: [rows, kv_heads, tokens, dim]."""
    t = cache[table.clamp(min=0).long()].float()
    if scale is not None:
        t = t * scale[:, None, None]
    rows, blocks, heads, page, dim = t.shape
    return t.transpose(1, 2).reshape(rows, heads, blocks * page, dim)


def _attend(s, q, pos):
    """Attention of q [rows, new, heads, dim] at positions pos [rows, new]
    (negative: no query): (out in 32 bits, log of the sum of exponentials)."""
    c = s["case"]
    k, v = _gathered(s["pool"][0], s["table"], s["k_scale"]), _gathered(s["pool"][1], s["table"], s["v_scale"])
    rows, new, heads, dim = q.shape
    kvh, tokens = k.shape[1], k.shape[2]
    t = torch.arange(tokens, device=q.device)
    there = (s["table"] >= 0).repeat_interleave(c["page"], 1)
    seen = (t <= pos[..., None]) & there[:, None]
    if c["window"]:
        seen &= (t > pos[..., None] - c["window"]) | (t < c["sinks"])
    v = torch.where((t < s["length"][:, None])[:, None, :, None], v, 0.0)
    x = q.float().reshape(rows, new, kvh, heads // kvh, dim).permute(0, 2, 3, 1, 4).reshape(rows, kvh, -1, dim)
    x = (x @ k.transpose(-1, -2)).mul_(s["scale"]).view(rows, kvh, heads // kvh, new, tokens)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(rows, kvh, -1, tokens) @ v).view(rows, kvh, heads // kvh, new, dim) / total.clamp(min=1e-37)
    o = o.permute(0, 3, 1, 2, 4).reshape(rows, new, heads, dim)
    lse = (total.log() + top).squeeze(-1).permute(0, 3, 1, 2).reshape(rows, new, heads)
    return o, lse


def _plain_decode(s):
    o, lse = _attend(s, s["q"][:, None], s["length"][:, None].long() - 1)
    return {"out": o[:, 0].to(s["q"].dtype), "lse": lse[:, 0]}


def _plain_prompt(s):
    off = s["offset"].long()
    n = off[1:] - off[:-1]
    i = torch.arange(s["max_new"], device=off.device)
    at = (off[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    pos = torch.where(i < n[:, None], s["length"][:, None].long() - n[:, None] + i, -1)
    o, _ = _attend(s, s["q"][at], pos)
    token = torch.arange(s["q"].shape[0], device=off.device)
    row = torch.searchsorted(off, token, right=True) - 1
    return {"out": o[row, token - off[row]].to(s["q"].dtype)}


def _plain_append(s):
    c, off = s["case"], s["offset"].long()
    token = torch.arange(s["k"].shape[0], device=off.device)
    row = torch.searchsorted(off, token, right=True) - 1
    pos = s["length"].long()[row] - (off[row + 1] - off[row]) + token - off[row]
    page = s["table"][row, pos // c["page"]].long()
    for cache, x, scale in ((s["pool"][0], s["k"], s["k_scale"]), (s["pool"][1], s["v"], s["v_scale"])):
        x = x.float()
        if scale is not None:
            x = (x / scale[:, None]).clamp(-448.0, 448.0)
        cache[page, :, pos % c["page"]] = x.to(cache.dtype)
    return {"pool": s["pool"]}


def _plain_free(s, rows):
    t = s["table"][rows].long().flatten()
    total = s["refs"].shape[0]
    gone = torch.zeros(total + 1, dtype=torch.int32, device=t.device)
    gone.index_add_(0, torch.where(t < 0, total, t), torch.ones_like(t, dtype=torch.int32))
    s["refs"] -= gone[:-1]
    s["table"][rows] = -1
    s["length"][rows] = 0


def _lowest_free(refs):
    page = torch.arange(refs.shape[0], device=refs.device)
    return torch.where(refs <= 0, page, refs.shape[0]).sort()[0]


def _plain_turn(s):
    page = s["case"]["page"]
    done, src = s["done"].long(), s["src"].long()
    _plain_free(s, done)
    # forks: whole pages are shared, a partly filled last one is copied to the lowest free pages, in order
    n = s["length"][src].long()
    full, part = n // page, n % page > 0
    need = part.cumsum(0)
    free = _lowest_free(s["refs"])
    room = (s["refs"] <= 0).sum()
    granted = ~part | (need <= room)
    block = torch.arange(s["table"].shape[1], device=n.device)
    rows = torch.where((block < full[:, None]) & granted[:, None], s["table"][src], -1)
    fresh = free[(need - 1).clamp(min=0)]
    first = s["table"][src, 0].long()  # a page that stays as it is stands for "no copy"
    old = torch.where(part & granted, s["table"][src].long().gather(1, full[:, None].clamp(max=len(block) - 1))[:, 0], first)
    fresh = torch.where(part & granted, fresh, first)
    s["pool"][:, fresh] = s["pool"].view(torch.uint8)[:, old].view(s["pool"].dtype) if s["pool"].dtype == torch.float8_e4m3fn \
        else s["pool"][:, old]
    rows = torch.where((block == full[:, None]) & (part & granted)[:, None], fresh[:, None].int(), rows)
    s["table"][done] = rows
    s["length"][done] = torch.where(granted, n, 0).int()
    held = rows.long().flatten()
    total = s["refs"].shape[0]
    more = torch.zeros(total + 1, dtype=torch.int32, device=n.device)
    more.index_add_(0, torch.where(held < 0, total, held), torch.ones_like(held, dtype=torch.int32))
    s["refs"] += more[:-1]
    # one more token each
    n = s["length"][done].long()
    part = n % page == 0
    need = part.cumsum(0)
    free = _lowest_free(s["refs"])
    room = (s["refs"] <= 0).sum()
    more = ~part | (need <= room)
    fresh = torch.where(part & more, free[(need - 1).clamp(min=0)], total)
    at = (n // page).clamp(max=s["table"].shape[1] - 1)
    s["table"][done, at] = torch.where(part & more, fresh.int(), s["table"][done, at])
    refs = torch.cat([s["refs"], s["refs"][:1]])
    refs[fresh] = 1
    s["refs"].copy_(refs[:-1])
    s["length"][done] = (n + more).int()
    return {"pool": s["pool"], "table": s["table"], "length": s["length"], "refs": s["refs"],
            "forked": granted.int(), "extended": more.int()}


def _plain_compact(s):
    refs = s["refs"]
    page = torch.arange(refs.shape[0], device=refs.device)
    live = refs > 0
    count = live.sum()
    hole, mover = (page < count) & ~live, (page >= count) & live
    to, frm = hole.nonzero()[:, 0], mover.nonzero()[:, 0]
    pool = s["pool"].view(torch.uint8) if s["pool"].dtype == torch.float8_e4m3fn else s["pool"]
    pool[:, to] = pool[:, frm]
    new = page.int()
    new[frm] = to.int()
    s["table_out"].copy_(torch.where(s["table"] < 0, -1, new[s["table"].clamp(min=0).long()]))
    out = torch.where(live, refs, 0)
    out[to] = refs[frm]
    s["refs_out"].copy_(torch.where(page < count, out, 0))
    return {"pool": s["pool"], "table": s["table_out"], "refs": s["refs_out"]}


def _plain_copy(s):
    pool = s["pool"].view(torch.uint8) if s["pool"].dtype == torch.float8_e4m3fn else s["pool"]
    pool[:, s["dst"].long()] = pool[:, s["src"].long()]
    return {"pool": s["pool"]}


def _plain_logits(s):
    c = s["logits"][s["cond_row"].long()].float()
    u = s["logits"][s["uncond_row"].clamp(min=0).long()].float()
    w = s["scale"][:, None]
    z = torch.where((w == 1) | (s["uncond_row"] < 0)[:, None] | (c == u), c, u + w * (c - u))
    n, v = z.shape
    if s["history"] is not None:
        j = torch.arange(s["history"].shape[1], device=z.device)
        there = j < s["history_len"][:, None]
        said = there & (j >= s["prompt_len"][:, None])
        ids = s["history"].long()
        seen = torch.zeros_like(z).scatter_add_(1, ids, there.float()) > 0
        count = torch.zeros_like(z).scatter_add_(1, ids, said.float())
        r = s["repetition"][:, None]
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        z = z - s["frequency"][:, None] * count
        z = z - torch.where(count > 0, s["presence"][:, None], 0.0)
    if s["bias"] is not None:
        z = z.scatter_add(1, s["bias_ids"].long(), s["bias"])
    z = z / s["temperature"][:, None]
    if s["mask"] is not None:
        i = torch.arange(v, device=z.device)
        z = torch.where((s["mask"][:, i // 32] >> (i % 32)) & 1 == 1, z, -math.inf)
    return {"out": z.to(s["out"].dtype)}


_PLAIN = {"decode": _plain_decode, "prompt": _plain_prompt, "append": _plain_append, "turn": _plain_turn,
          "compact": _plain_compact, "copy": _plain_copy, "logits": _plain_logits}


# ---- the framework's calls ---------------------------------------------------------

def _own(s):
    import bucketed_classifier_free_amd as bcg
    c, op = s["case"], s["case"]["op"]
    if op == "logits":
        bcg.guided_logits(s["logits"], s["out"], s["cond_row"], s["uncond_row"], s["scale"], history=s["history"],
                          history_len=s["history_len"], prompt_len=s["prompt_len"], repetition=s["repetition"],
                          presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"],
                          temperature=s["temperature"], mask=s["mask"])
        return {"out": s["out"]}
    if op in ("decode", "prompt"):
        if "workspace" not in s:  # kept from call to call, as a decoding loop keeps it
            s["workspace"] = bcg.attention_workspace(s["q"].shape[0], c["heads"], c["dim"])
        kw = dict(scale=s["scale"], window=c["window"], sinks=c["sinks"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                  max_len=s["max_len"], workspace=s["workspace"])
        if op == "decode":
            bcg.paged_attention(s["q"], s["pool"][0], s["pool"][1], s["table"], s["length"], s["out"], lse=s["lse"], **kw)
            return {"out": s["out"], "lse": s["lse"]}
        bcg.prompt_attention(s["q"], s["offset"], s["pool"][0], s["pool"][1], s["table"], s["length"], s["out"],
                             max_new=s["max_new"], **kw)
        return {"out": s["out"]}
    if op == "append":
        bcg.cache_append(s["k"], s["v"], s["pool"][0], s["pool"][1], s["table"], s["length"], offset=s["offset"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"pool": s["pool"]}
    if op == "copy":
        bcg.cache_copy(s["pool"], s["src"], s["dst"])
        return {"pool": s["pool"]}
    if "cache" not in s:
        s["cache"] = bcg.PagedCache(s["pool"], s["table"], s["length"], s["refs"])
    if op == "compact":
        bcg.cache_compact(s["cache"], table_out=s["table_out"], refs_out=s["refs_out"])
        return {"pool": s["pool"], "table": s["table_out"], "refs": s["refs_out"]}
    bcg.cache_free(s["cache"], s["done"])
    forked = bcg.cache_fork(s["cache"], s["src"], s["done"])
    extended = bcg.cache_extend(s["cache"], s["done"], s["one"])
    return {"pool": s["pool"], "table": s["table"], "length": s["length"], "refs": s["refs"], "forked": forked,
            "extended": extended}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---- the definitions in 64 bits ------------------------------------------------------

def _exact_attention(case, s):
    new, lens = _lengths(case)
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    at = 0
    for r, (a, b) in enumerate(zip(new, lens)):
        pages = s["table"][r, :-(-b // case["page"])].long()
        part = []
        for side, scale in ((0, s["k_scale"]), (1, s["v_scale"])):
            t = s["pool"][side][pages].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :b]
            part.append(t if scale is None else t * scale.double()[:, None, None])
        pos = torch.arange(b - a, b, device=DEV)[:, None]
        tok = torch.arange(b, device=DEV)[None]
        hidden = tok > pos
        if case["window"]:
            hidden |= (tok <= pos - case["window"]) & (tok >= case["sinks"])
        for h in range(case["kv_heads"]):
            x = s["q"][at:at + a, h * group:(h + 1) * group].double().transpose(0, 1)  # [group, a, dim]
            y = torch.matmul(x, part[0][h].t().contiguous()) * case["dim"] ** -0.5
            y = y.masked_fill(hidden, -math.inf)
            lse[at:at + a, h * group:(h + 1) * group] = torch.logsumexp(y, -1).t()
            out[at:at + a, h * group:(h + 1) * group] = torch.matmul(torch.softmax(y, -1), part[1][h]).transpose(0, 1)
        at += a
    return {"out": out, "lse": lse} if case["op"] == "decode" else {"out": out}


def _exact_logits(case, s):
    v = case["vocab"]
    rows = []
    for i in range(case["n"]):
        z = s["logits"][int(s["cond_row"][i])].double()
        w, ur = float(s["scale"][i]), int(s["uncond_row"][i])
        if w != 1.0 and ur >= 0:
            z = z * w + s["logits"][ur].double() * (1.0 - w)
        if case["history"]:
            n, p = int(s["history_len"][i]), int(s["prompt_len"][i])
            all_of = torch.bincount(s["history"][i, :n], minlength=v)
            answer = torch.bincount(s["history"][i, p:n], minlength=v).double()
            r = float(s["repetition"][i])
            z = torch.where(all_of > 0, z * torch.where(z > 0, 1.0 / r, r), z)
            z = z - float(s["frequency"][i]) * answer - float(s["presence"][i]) * answer.clamp(max=1.0)
        if case["bias"]:
            z = z.clone()
            z[s["bias_ids"][i].long()] += s["bias"][i].double()
        z = z / float(s["temperature"][i])
        if case["mask"]:
            bits = (s["mask"][i][:, None] >> torch.arange(32, device=DEV)) & 1
            z = z.masked_fill(bits.flatten()[:v] == 0, -math.inf)
        rows.append(z)
    return {"out": torch.stack(rows)}


def _exact_append(case, s):
    pool = s["pool"].double()
    new, lens = _lengths(case)
    at = 0
    for r, (a, b) in enumerate(zip(new, lens)):
        pos = torch.arange(b - a, b, device=DEV)
        page = s["table"][r].long()[pos // case["page"]]
        for side, x, scale in ((0, s["k"], s["k_scale"]), (1, s["v"], s["v_scale"])):
            y = x[at:at + a].double()
            if scale is not None:
                y = (y / scale.double()[:, None]).clamp(-448.0, 448.0)
            pool[side][page, :, pos % case["page"]] = y
        at += a
    return {"pool": pool}


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op in ("decode", "prompt"):
        return _exact_attention(case, s)
    if op == "logits":
        return _exact_logits(case, s)
    if op == "append":
        return _exact_append(case, s)
    return None  # pages and counts are moved, not computed
