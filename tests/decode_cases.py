"""Inputs of the decoding operators' GPU tests, and their bounds."""
import numpy as np
import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def half_step(t):
    """How far one rounding is off, relative to the value."""
    return float(torch.finfo(t).eps) / 2


def np64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def tables(rng, pages, total, width):
    """A table whose rows hold pages[r] pages in shuffled order, -1 behind."""
    order = rng.permutation(total)
    table = np.full((len(pages), width), -1, np.int32)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = order[at:at + n]
        at += n
    return table


def make_cache(lens, kv_heads, dim, page, kv="bf16", seed=0, spare=2, extra_blocks=1, layout="split", rot=float("nan")):
    """A layer's pages holding random tokens of ``lens`` tokens a row; every
    slot that no token has holds ``rot``.  layout: "split" (two pools) or
    "paired" (a page's keys and values next to each other)."""
    rng = np.random.default_rng(seed)
    pages = [-(-n // page) for n in lens]
    total = sum(pages) + spare
    width = max(pages + [0]) + extra_blocks
    table = tables(rng, pages, total, width)
    data = np.full((2, total, kv_heads, page, dim), rot, np.float32)
    for r, n in enumerate(lens):
        for b in range(pages[r]):
            m = min(page, n - b * page)
            data[:, table[r, b], :, :m] = rng.standard_normal((2, kv_heads, m, dim))
    t = torch.from_numpy(data).cuda()
    t = (t.to(torch.bfloat16) if kv == "e4m3" else t).to(TYPES[kv])
    if layout == "paired":
        t = t.view(torch.uint8) if kv == "e4m3" else t
        t = t.transpose(0, 1).contiguous()
        t = t.view(torch.float8_e4m3fn) if kv == "e4m3" else t
        k, v = t[:, 0], t[:, 1]
    else:
        k, v = t[0], t[1]
    scales = (None, None)
    if kv == "e4m3":
        scales = tuple(torch.from_numpy(rng.uniform(0.5, 1.5, kv_heads).astype(np.float32)).cuda() for _ in range(2))
    return dict(k=k, v=v, table=torch.from_numpy(table).cuda(), length=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                k_scale=scales[0], v_scale=scales[1])


def make_queries(tokens, heads, dim, q="bf16", seed=0, strided=True):
    """Queries as the first part of a wider projection's rows."""
    g = torch.Generator().manual_seed(seed + 77)
    wide = torch.randn((tokens, heads + (3 if strided else 0), dim), generator=g) * 1.5
    return wide.to(TYPES[q]).cuda()[:, :heads]


def attention_bounds(ref, dim, tokens, qt):
    """Bounds of |out - ref| and |lse - ref| (oracle.decode.attention's
    results): one rounding of out and one of every probability to the query's
    type (fp32 rounds neither of them further), fp32 scores off by the
    rounding of dim + 8 terms that reach `bound` (log2 units: 1.5 times it),
    sums of `tokens` terms, and a few roundings of the exponential."""
    out, lse, weight, bound = ref
    f = 2.0 ** -24
    score = 4 * (dim + 8) * f * (bound + 1.0)
    rel = score + (tokens + 16) * f
    h = half_step(qt) if qt != torch.float32 else f
    lse = np.where(np.isfinite(lse), np.abs(lse), 0.0)
    return (1.01 * h * (np.abs(out) + weight) + rel[..., None] * 2 * weight + 1e-30,
            rel + 4 * f * (lse + 1.0))
