"""paged_attention and prompt_attention against their definition in float64
(oracle/decode.py), within bounds that follow from the types.

Every storage slot that holds no token is NaN, pages are shuffled, and the
tables are wider than needed: what a kernel reads beyond a row shows up.
"""
import numpy as np
import pytest
import torch

from decode_cases import TYPES, attention_bounds, make_cache, make_queries, np64
from oracle import decode as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bucketed_classifier_free_amd
    bucketed_classifier_free_amd.load()  # fails loudly without libbcg.so


def reference(q, offset, c, scale, window, sinks):
    return O.attention(np64(q), offset, np64(c["k"]), np64(c["v"]), c["table"].cpu().numpy(), c["length"].cpu().numpy(),
                       scale, window, sinks, np64(c["k_scale"]), np64(c["v_scale"]))


def check(got, lse, ref, dim, tokens, qt):
    out_tol, lse_tol = attention_bounds(ref, dim, tokens, qt)
    got, lse = np64(got), np64(lse)
    assert np.isfinite(got).all()
    worst = np.abs(got - ref[0]) / out_tol
    assert worst.max() <= 1.0, f"out {worst.max():.3g} of its bound at {np.unravel_index(worst.argmax(), worst.shape)}"
    assert np.array_equal(np.isinf(lse), np.isinf(ref[1]))
    fin = np.isfinite(ref[1])
    assert (np.abs(lse - ref[1])[fin] <= lse_tol[fin]).all()


def decode(c, q, window=0, sinks=0, scale=None, max_len=None, workspace=None, out=None):
    import bucketed_classifier_free_amd as bcg
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    ws = bcg.attention_workspace(*q.shape) if workspace is None else workspace
    bcg.paged_attention(q, c["k"], c["v"], c["table"], c["length"], out, workspace=ws, scale=scale, window=window,
                        sinks=sinks, k_scale=c["k_scale"], v_scale=c["v_scale"], max_len=max_len, lse=lse)
    torch.cuda.synchronize()
    return out, lse


def prompt(c, q, offset, window=0, sinks=0, scale=None, max_len=None, max_new=None):
    import bucketed_classifier_free_amd as bcg
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], float("nan"), device="cuda")
    off = torch.tensor(offset, dtype=torch.int32, device="cuda")
    bcg.prompt_attention(q, off, c["k"], c["v"], c["table"], c["length"], out, workspace=bcg.attention_workspace(*q.shape),
                         scale=scale, window=window, sinks=sinks, k_scale=c["k_scale"], v_scale=c["v_scale"],
                         max_len=max_len, max_new=max_new, lse=lse)
    torch.cuda.synchronize()
    return out, lse


KINDS = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3")]


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(4, 4, 64, 16), (8, 2, 128, 16), (8, 1, 128, 48), (17, 1, 80, 32),
                                                     (3, 3, 256, 16), (6, 2, 208, 64), (40, 2, 96, 128), (2, 2, 16, 16)])
def test_decode_heads_and_pages(q, kv, heads, kv_heads, dim, page):
    lens = [1, 0, 15, 16, 17, 31, 33, 100, 257]
    c = make_cache(lens, kv_heads, dim, page, kv, seed=heads + dim)
    x = make_queries(len(lens), heads, dim, q, seed=dim)
    out, lse = decode(c, x)
    check(out, lse, reference(x, np.arange(len(lens) + 1), c, dim ** -0.5, 0, 0), dim, 257, TYPES[q])
    assert (np64(out)[1] == 0).all() and np.isneginf(np64(lse)[1]).all()


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (16, 0), (40, 3), (64, 16), (100, 33), (5000, 4), (7, 5000)])
def test_decode_window_and_sinks(q, kv, window, sinks):
    lens = [1, 3, 16, 40, 41, 97, 300, 1000]
    c = make_cache(lens, 2, 64, 16, kv, seed=window)
    x = make_queries(len(lens), 6, 64, q, seed=sinks)
    out, lse = decode(c, x, window, sinks)
    check(out, lse, reference(x, np.arange(len(lens) + 1), c, 64 ** -0.5, window, sinks), 64, 1000, TYPES[q])


@pytest.mark.parametrize("q,kv", KINDS)
def test_decode_hidden_tokens_take_no_part(q, kv):
    """Storage of hidden tokens is NaN: outside the window, and on pages that
    were given back."""
    lens = [200, 131, 64]
    c = make_cache(lens, 2, 128, 16, kv, seed=5)
    x = make_queries(3, 8, 128, q, seed=5)
    window, sinks = 37, 5
    ref = reference(x, np.arange(4), c, 128 ** -0.5, window, sinks)
    k, v, table = c["k"], c["v"], c["table"].cpu().numpy()
    for r, n in enumerate(lens):
        for t in range(n):
            if not O.visible(np.array([t]), n - 1, window, sinks)[0]:
                if c["k"].dtype == torch.float8_e4m3fn:
                    k.view(torch.uint8)[table[r, t // 16], :, t % 16] = 0x7f
                    v.view(torch.uint8)[table[r, t // 16], :, t % 16] = 0x7f
                else:
                    k[table[r, t // 16], :, t % 16] = float("nan")
                    v[table[r, t // 16], :, t % 16] = float("inf")
    check(*decode(c, x, window, sinks), ref, 128, 200, TYPES[q])
    # pages wholly hidden leave the table
    for r, n in enumerate(lens):
        for b in range(-(-n // 16)):
            if not O.visible(np.arange(b * 16, min(n, b * 16 + 16)), n - 1, window, sinks).any():
                table[r, b] = -1
    c["table"].copy_(torch.from_numpy(table))
    check(*decode(c, x, window, sinks), ref, 128, 200, TYPES[q])


def test_decode_missing_pages_and_bad_entries():
    """Entries outside the pool are tokens that are not there."""
    lens = [100, 70, 48, 33]
    c = make_cache(lens, 2, 64, 16, "bf16", seed=9)
    t = c["table"]
    t[0, 2] = -1
    t[1, 0] = c["k"].shape[0]      # one beyond the pool
    t[1, 3] = 2 ** 31 - 1
    t[2] = -1                      # nothing left
    t[3, 1] = -2 ** 31
    x = make_queries(4, 4, 64, "bf16", seed=9)
    out, lse = decode(c, x)
    check(out, lse, reference(x, np.arange(5), c, 0.125, 0, 0), 64, 100, torch.bfloat16)
    assert (np64(out)[2] == 0).all()


def test_decode_lengths_out_of_range():
    """A negative length is 0, one beyond the table its width."""
    c = make_cache([64, 64], 1, 64, 16, "f32", seed=2, extra_blocks=0)
    x = make_queries(2, 2, 64, "f32", seed=2)
    ref = reference(x, np.arange(3), c, 0.125, 0, 0)
    c["length"].copy_(torch.tensor([2 ** 31 - 1, -5], dtype=torch.int32))
    out, lse = decode(c, x)
    assert np.array_equal(np64(out)[0], np64(decode(dict(c, length=torch.full((2,), 64, dtype=torch.int32, device="cuda")), x)[0])[0])
    assert np.abs(np64(out)[0] - ref[0][0]).max() < 1e-5
    assert (np64(out)[1] == 0).all() and np.isneginf(np64(lse)[1]).all()


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("rows,length,page", [(1, 5000, 16), (1, 9001, 64), (3, 3333, 32)])
def test_decode_long_rows_are_split_and_joined(q, kv, rows, length, page):
    lens = [length] + [length // 2 + 7] * (rows - 1)
    c = make_cache(lens, 2, 128, page, kv, seed=length)
    x = make_queries(rows, 8, 128, q, seed=length)
    out, lse = decode(c, x)
    check(out, lse, reference(x, np.arange(rows + 1), c, 128 ** -0.5, 0, 0), 128, length, TYPES[q])


def test_decode_workspace_serves_calls_of_other_shapes_and_results_repeat():
    import bucketed_classifier_free_amd as bcg
    ws = bcg.attention_workspace(8, 16, 128)
    first = {}
    for _ in range(3):
        for rows, heads, dim, length in ((1, 16, 128, 4000), (8, 4, 64, 90), (2, 8, 128, 2000)):
            c = make_cache([length] * rows, 2, dim, 16, "bf16", seed=rows)
            x = make_queries(rows, heads, dim, "bf16", seed=rows)
            out, lse = decode(c, x, workspace=ws)
            if rows in first:
                assert torch.equal(out, first[rows][0]) and torch.equal(lse, first[rows][1])
            first[rows] = (out.clone(), lse.clone())


def test_decode_large_scores_and_moving_maximum():
    """Scores that grow along the row move the running maximum at every block."""
    n = 700
    c = make_cache([n], 1, 64, 16, "f32", seed=3)
    x = torch.ones((1, 1, 64), device="cuda")
    table = c["table"].cpu().numpy()
    for t in range(n):
        c["k"][table[0, t // 16], 0, t % 16] = t * 0.05
    ref = reference(x, [0, 1], c, 0.5, 0, 0)
    check(*decode(c, x, scale=0.5), ref, 64, n, torch.float32)


@pytest.mark.parametrize("layout", ["split", "paired"])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_page_strides(layout, kv):
    lens = [50, 77]
    c = make_cache(lens, 4, 64, 32, kv, seed=1, layout=layout)
    x = make_queries(2, 8, 64, "bf16", seed=1)
    check(*decode(c, x), reference(x, np.arange(3), c, 0.125, 0, 0), 64, 77, torch.bfloat16)
    off = [0, 20, 60]
    y = make_queries(60, 8, 64, "bf16", seed=2)
    check(*prompt(c, y, off), reference(y, off, c, 0.125, 0, 0), 64, 77, torch.bfloat16)


def test_offsets_beyond_32_bits():
    """Pages that lie more than 2^32 elements into the cache."""
    pages = 2 ** 32 // (8 * 64 * 256) + 3
    k = torch.empty((pages, 8, 64, 256), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator().manual_seed(4)
    table = torch.full((2, 3), -1, dtype=torch.int32)
    table[0, :2] = torch.tensor([pages - 1, 0])
    table[1, :2] = torch.tensor([pages - 2, pages - 3])
    for p in (0, pages - 1, pages - 2, pages - 3):
        for t in (k, v):
            t[p].copy_(torch.randn((8, 64, 256), generator=g).to(torch.bfloat16).to(torch.float8_e4m3fn))
    one = torch.ones(8, device="cuda")
    lens = [100, 128]
    x = make_queries(2, 16, 256, "bf16", seed=6)
    # the oracle sees the four pages alone
    used = [pages - 1, 0, pages - 2, pages - 3]
    small = torch.tensor([[0, 1, -1], [2, 3, -1]], dtype=torch.int32)
    ref = O.attention(np64(x), np.arange(3), np64(torch.stack([k[p].float() for p in used])),
                      np64(torch.stack([v[p].float() for p in used])), small.numpy(), np.array(lens), 1 / 16)
    c = dict(k=k, v=v, table=table.cuda(), length=torch.tensor(lens, dtype=torch.int32, device="cuda"), k_scale=one, v_scale=one)
    check(*decode(c, x), ref, 256, 128, torch.bfloat16)
    check(*prompt(c, x, [0, 1, 2]), ref, 256, 128, torch.bfloat16)


# ---- prompts ---------------------------------------------------------------------

@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(2, 2, 64, 16), (8, 2, 128, 16), (3, 1, 128, 48), (2, 1, 256, 32),
                                                     (10, 2, 80, 64), (4, 2, 208, 16), (17, 1, 16, 16)])
def test_prompt_heads_and_pages(q, kv, heads, kv_heads, dim, page):
    new, past = [1, 17, 0, 64, 90, 5], [0, 0, 9, 0, 13, 100]
    lens = [a + b for a, b in zip(new, past)]
    off = np.concatenate([[0], np.cumsum(new)]).tolist()
    c = make_cache(lens, kv_heads, dim, page, kv, seed=heads * dim)
    x = make_queries(off[-1], heads, dim, q, seed=dim)
    check(*prompt(c, x, off), reference(x, off, c, dim ** -0.5, 0, 0), dim, max(lens), TYPES[q])


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (50, 1), (64, 64), (130, 7), (4000, 2)])
def test_prompt_window_and_sinks(q, kv, window, sinks):
    new, past = [150, 33, 1], [60, 0, 299]
    lens = [a + b for a, b in zip(new, past)]
    off = np.concatenate([[0], np.cumsum(new)]).tolist()
    c = make_cache(lens, 1, 64, 16, kv, seed=window)
    x = make_queries(off[-1], 3, 64, q, seed=window)
    check(*prompt(c, x, off, window, sinks, max_new=150), reference(x, off, c, 0.125, window, sinks), 64, max(lens), TYPES[q])


@pytest.mark.parametrize("q,kv", KINDS)
def test_prompt_few_queries_over_a_long_past_are_split(q, kv):
    new, past = [3, 16], [4000, 2500]
    lens = [a + b for a, b in zip(new, past)]
    off = [0, 3, 19]
    c = make_cache(lens, 1, 128, 16, kv, seed=8)
    x = make_queries(19, 4, 128, q, seed=8)
    check(*prompt(c, x, off, max_new=16), reference(x, off, c, 128 ** -0.5, 0, 0), 128, max(lens), TYPES[q])


@pytest.mark.parametrize("q,kv", KINDS)
def test_prompt_hidden_values_that_are_not_finite(q, kv):
    """A token with infinite or NaN values reaches the queries that see it and no other."""
    n, window, sinks = 150, 60, 2
    c = make_cache([n], 2, 64, 16, kv, seed=12)
    x = make_queries(n, 4, 64, q, seed=12)
    ref = reference(x, [0, n], c, 0.125, window, sinks)
    table = c["table"].cpu().numpy()
    bad = [30, 77, 78, 149]
    for t in bad:
        if kv == "e4m3":
            c["v"].view(torch.uint8)[table[0, t // 16], :, t % 16] = 0x7f
        else:
            c["v"][table[0, t // 16], :, t % 16] = float("nan") if t % 2 else float("inf")
    out, _ = prompt(c, x, [0, n], window, sinks)
    out = np64(out)
    tol, _ = attention_bounds(ref, 64, n, TYPES[q])
    for i in range(n):
        if O.visible(np.array(bad), i, window, sinks).any():
            assert not np.isfinite(out[i]).any(), i
        else:
            assert (np.abs(out[i] - ref[0][i]) <= tol[i]).all(), i


def test_prompt_missing_pages_negative_positions_and_unused_queries():
    c = make_cache([100, 20, 64], 1, 64, 16, "bf16", seed=15)
    c["table"][0, 1] = -1
    c["table"][0, 4] = 10 ** 6
    # row 1 claims more new tokens than it has; row 2's run ends before the last queries
    off = [0, 40, 70, 80]
    x = make_queries(85, 2, 64, "bf16", seed=15)
    ref = reference(x[:80], off, c, 0.125, 0, 0)
    out, lse = prompt(c, x, off)
    check(out[:80], lse[:80], ref, 64, 100, torch.bfloat16)
    assert torch.isnan(out[80:].float()).all()  # nobody's queries are not written
    assert (np64(out)[40:50] == 0).all()


def test_prompt_and_decode_agree_with_one_query_a_row():
    lens = [5, 64, 200]
    c = make_cache(lens, 2, 128, 16, "bf16", seed=21)
    x = make_queries(3, 8, 128, "bf16", seed=21)
    ref = reference(x, np.arange(4), c, 128 ** -0.5, 0, 0)
    check(*prompt(c, x, [0, 1, 2, 3]), ref, 128, 200, torch.bfloat16)
    check(*decode(c, x), ref, 128, 200, torch.bfloat16)


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 3)])
@pytest.mark.parametrize("top", [130, 2500])
def test_prompt_with_at_most_one_query_a_row(q, kv, window, sinks, top):
    """max_new of 1: rows with a query, without one, with more than it (the
    first counts), without tokens, and with more queries than tokens."""
    lens = [top, 40, 0, 77, 1, 2, 200, 16]
    off = [0, 1, 1, 2, 5, 6, 10, 10, 11]
    c = make_cache(lens, 2, 64, 16, kv, seed=top)
    c["table"][0, 2] = -1
    x = make_queries(13, 6, 64, q, seed=window)
    ref = reference(x[:11], off, c, 0.125, window, sinks)
    out, lse = prompt(c, x, off, window, sinks, max_new=1)
    first = [0, 1, 2, 5, 6, 10]
    check(out[first], lse[first], tuple(r[first] if isinstance(r, np.ndarray) and r.ndim else r for r in ref), 64, top, TYPES[q])
    rest = [i for i in range(13) if i not in first]
    assert torch.isnan(out[rest].float()).all() and torch.isnan(lse[rest]).all()


def dense64(x, c, pos, scale, window=0):
    """Attention of x [rows, new, heads, dim] at pos [new], heads == kv_heads,
    in float64 on the GPU; (out, bounds as oracle.decode.attention)."""
    rows, page = x.shape[0], c["k"].shape[2]
    k, v = (c[n].double()[c["table"].long()].transpose(1, 2).flatten(2, 3) for n in ("k", "v"))  # [rows, heads, tokens, dim]
    t = torch.arange(k.shape[2], device="cuda")
    seen = (t <= pos[:, None]) & ((t > pos[:, None] - window) if window else True)
    q = x.double().transpose(1, 2)
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()) * scale
    s = s.masked_fill(~seen, -float("inf"))
    p, lse = torch.softmax(s, -1), torch.logsumexp(s, -1)
    v = torch.where((t <= int(pos.max()))[:, None], v, 0.0)
    out, weight = torch.matmul(p, v), torch.matmul(p, v.abs())
    reach = torch.matmul(q.abs(), torch.nan_to_num(k).abs().transpose(-1, -2).contiguous()).amax(-1) * scale
    back = lambda y: y.transpose(1, 2).flatten(0, 1).cpu().numpy()  # noqa: E731
    return back(out), back(lse), back(weight), back(reach)


@pytest.mark.parametrize("q,kv", KINDS[:2])
@pytest.mark.parametrize("window", [0, 700])
def test_prompt_long_runs_without_splits(q, kv, window):
    """More tiles in one workgroup than one read of the table covers."""
    new, heads, dim = 1300, 32, 16
    c = make_cache([new, new], heads, dim, 48, kv, seed=window, rot=0.0)
    x = make_queries(2 * new, heads, dim, q, seed=1, strided=False)
    ref = dense64(x.view(2, new, heads, dim), c, torch.arange(new, device="cuda"), 0.25, window)
    check(*prompt(c, x, [0, new, 2 * new], window, 0, scale=0.25, max_new=new), ref, dim, new, TYPES[q])


@pytest.mark.parametrize("q,kv", KINDS[:2])
def test_decode_many_rows_without_splits(q, kv):
    """A workgroup that walks a whole long row, more blocks than one read of
    the table covers; rows share pages."""
    rows, heads, dim, n = 520, 8, 16, 4500
    c = make_cache([n], heads, dim, 16, kv, seed=2, rot=0.0, extra_blocks=0)
    order = torch.stack([torch.randperm(282, generator=torch.Generator().manual_seed(r)) for r in range(rows)])
    # the partly filled page stays last
    full = c["table"][0, :281].cpu()
    order = torch.cat([full[order[order < 281].view(rows, 281)], c["table"][0, 281:].cpu().expand(rows, 1)], 1)
    c["table"] = order.int().contiguous().cuda()
    c["length"] = torch.full((rows,), n, dtype=torch.int32, device="cuda")
    x = make_queries(rows, heads, dim, q, seed=5)
    ref = dense64(x[:, None], c, torch.tensor([n - 1], device="cuda"), 0.25)
    check(*decode(c, x), ref, dim, n, TYPES[q])


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("dim,page", [(48, 16), (64, 32), (128, 16), (208, 48), (256, 16)])
@pytest.mark.parametrize("rows,top,window,sinks", [(3, 64, 0, 0), (40, 90, 0, 0), (40, 300, 20, 3), (100, 250, 0, 0), (190, 130, 0, 0)])
def test_decode_rows_whole_in_one_launch(q, kv, dim, page, rows, top, window, sinks):
    """Rows that are not split, over workgroups of one, two, four and eight waves."""
    kv_heads = 8
    lens = [top if i == 0 else (i * 37) % (top + 1) for i in range(rows)]
    c = make_cache(lens, kv_heads, dim, page, kv, seed=rows + dim)
    x = make_queries(rows, 16, dim, q, seed=rows)
    out, lse = decode(c, x, window, sinks)
    check(out, lse, reference(x, np.arange(rows + 1), c, dim ** -0.5, window, sinks), dim, top, TYPES[q])


@pytest.mark.parametrize("q,kv", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[40, 700], [0, 2100, 1], [4500, 33]])
def test_decode_few_and_many_splits_are_joined(q, kv, dim, lens):
    """Up to 64 splits, most of them empty for the short rows."""
    import bucketed_classifier_free_amd as bcg
    c = make_cache(lens, 2, dim, 32, kv, seed=dim)
    x = make_queries(len(lens), 6, dim, q, seed=dim)
    ws = torch.full_like(bcg.attention_workspace(*x.shape), 255)  # NaN throughout
    out, lse = decode(c, x, workspace=ws)
    check(out, lse, reference(x, np.arange(len(lens) + 1), c, dim ** -0.5, 0, 0), dim, max(lens), TYPES[q])


def test_decode_many_short_rows():
    rng = np.random.default_rng(1)
    lens = [int(n) for n in rng.integers(0, 50, 600)]
    c = make_cache(lens, 8, 64, 16, "bf16", seed=3)
    x = make_queries(600, 8, 64, "bf16", seed=3)
    check(*decode(c, x), reference(x, np.arange(601), c, 0.125, 0, 0), 64, 50, torch.bfloat16)


def test_on_another_stream_and_in_a_graph():
    import bucketed_classifier_free_amd as bcg
    lens = [900, 77]
    c = make_cache(lens, 2, 64, 16, "bf16", seed=30)
    x = make_queries(2, 8, 64, "bf16", seed=30)
    want, _ = decode(c, x)
    ws = bcg.attention_workspace(2, 8, 64)
    out = torch.zeros_like(want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bcg.paged_attention(x, c["k"], c["v"], c["table"], c["length"], out, workspace=ws)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bcg.paged_attention(x, c["k"], c["v"], c["table"], c["length"], out, workspace=ws)
    for n in (900, 33, 512, 1):  # the lengths are read by the kernels, not by the capture
        c["length"].copy_(torch.tensor([n, 77], dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, decode(c, x)[0]), n
