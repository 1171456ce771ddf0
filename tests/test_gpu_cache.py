"""cache_append and the page operators against oracle/decode.py: the moved
data bit for bit, the tables and counts exactly."""
import numpy as np
import pytest
import torch

from decode_cases import TYPES, make_cache
from oracle import decode as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bucketed_classifier_free_amd
    bucketed_classifier_free_amd.load()  # fails loudly without libbcg.so


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ---- append ------------------------------------------------------------------------

@pytest.mark.parametrize("q,kv", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "e4m3")])
@pytest.mark.parametrize("new,past", [([1, 1, 1], [0, 15, 16]), ([5, 0, 70, 33], [3, 8, 0, 500]), ([2, 40], [0, 30])])
@pytest.mark.parametrize("layout", ["split", "paired"])
def test_append(q, kv, new, past, layout):
    import bucketed_classifier_free_amd as bcg
    heads, dim, page = 3, 80, 16
    lens = [a + b for a, b in zip(new, past)]
    c = make_cache(lens, heads, dim, page, kv, seed=sum(lens), layout=layout, rot=1.0)
    g = torch.Generator().manual_seed(3)
    qkv = (torch.randn((sum(new), 3, heads, dim), generator=g) * 200).to(TYPES[q]).cuda()
    k, v = qkv[:, 1], qkv[:, 2]
    if k.shape[0] > 1:
        k[0, 0, 0], k[0, 0, 1], v[0, 0, 0], v[0, 0, 1] = float("nan"), float("inf"), -float("inf"), 1e30
    off = np.concatenate([[0], np.cumsum(new)])
    want_k, want_v = c["k"].clone(), c["v"].clone()
    if kv == "e4m3":
        want_k, want_v = want_k.view(torch.uint8), want_v.view(torch.uint8)
    table = c["table"].cpu().numpy()
    for r, n in enumerate(lens):
        for t in range(past[r], n):
            for x, w, s in ((k, want_k, c["k_scale"]), (v, want_v, c["v_scale"])):
                y = x[off[r] + t - past[r]]
                if kv == "e4m3":
                    y = (y.float() / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                w[table[r, t // page], :, t % page] = y
    offset = None if new == [1] * len(new) else i32(off.tolist())
    bcg.cache_append(k, v, c["k"], c["v"], c["table"], c["length"], offset=offset, k_scale=c["k_scale"], v_scale=c["v_scale"])
    torch.cuda.synchronize()
    assert np.array_equal(bits(c["k"]), bits(want_k)) and np.array_equal(bits(c["v"]), bits(want_v))


@pytest.mark.parametrize("heads,dim", [(1, 8), (1, 64), (8, 128)])
@pytest.mark.parametrize("rows", [1, 70, 300])
def test_append_finds_the_row_of_every_token(heads, dim, rows):
    """Runs of unlike lengths, many of them empty, in many rows."""
    import bucketed_classifier_free_amd as bcg
    rng = np.random.default_rng(rows)
    new = [int(n) for n in rng.integers(0, 9, rows) * (rng.random(rows) < 0.6)]
    new[rng.integers(rows)] += 33
    c = make_cache(new, heads, dim, 16, "f32", seed=rows, rot=0.0)
    k = torch.randn((sum(new), heads, dim), device="cuda")
    want = c["k"].clone()
    table, off = c["table"].cpu().numpy(), np.concatenate([[0], np.cumsum(new)])
    for r, n in enumerate(new):
        for t in range(n):
            want[table[r, t // 16], :, t % 16] = k[off[r] + t]
    bcg.cache_append(k, k, c["k"], c["v"], c["table"], c["length"], offset=i32(off.tolist()))
    torch.cuda.synchronize()
    assert torch.equal(c["k"], want)


def test_append_drops_tokens_without_a_place():
    import bucketed_classifier_free_amd as bcg
    c = make_cache([40, 20, 16], 2, 64, 16, "f32", seed=1, rot=0.0)
    c["table"][0, 1] = -1
    c["table"][1, 0] = 10 ** 7
    k = torch.randn((60, 2, 64), device="cuda")
    table = c["table"].cpu().numpy()
    off = [0, 20, 50, 55]  # row 1 claims 30 tokens of 20; tokens 55..59 are nobody's
    want = c["k"].clone()
    for r, n in enumerate([40, 20, 16]):
        for i in range(off[r], off[r + 1]):
            pos = n - (off[r + 1] - i)
            if pos >= 0 and 0 <= table[r, pos // 16] < c["k"].shape[0]:
                want[table[r, pos // 16], :, pos % 16] = k[i]
    bcg.cache_append(k, k, c["k"], c["v"], c["table"], c["length"], offset=i32(off))
    torch.cuda.synchronize()
    assert torch.equal(c["k"], want)


# ---- pages -----------------------------------------------------------------------------

class Both:
    """A cache on the GPU and the oracle's, which must stay equal."""

    def __init__(self, lens, page=16, spare=6, planes=4, heads=2, dim=64, dtype=torch.bfloat16, width=None, seed=0, page_gap=0):
        import bucketed_classifier_free_amd as bcg
        rng = np.random.default_rng(seed)
        pages = [-(-n // page) for n in lens]
        total = sum(pages) + spare
        width = max(pages + [1]) + 2 if width is None else width
        order = rng.permutation(total)
        table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for r, n in enumerate(pages):
            table[r, :n] = order[at:at + n]
            at += n
        refs = np.zeros(total, np.int32)
        refs[order[:at]] = 1
        wide = torch.from_numpy(rng.standard_normal((planes, total, 1 + page_gap, heads, page, dim)).astype(np.float32)).to(dtype).cuda()
        self.cache = bcg.PagedCache(wide[:, :, 0], i32(table.tolist()), i32(lens), i32(refs.tolist()))
        self.wide, self.gap = wide, bits(wide[:, :, 1:]) if page_gap else None
        self.o = O.Pages(self.pool_bits(), table, np.array(lens, np.int32), refs, page)

    def pool_bits(self):
        return bits(self.cache.pool)

    def same(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.cache.table.cpu().numpy(), self.o.table)
        assert np.array_equal(self.cache.length.cpu().numpy(), self.o.length)
        assert np.array_equal(self.cache.refs.cpu().numpy(), self.o.refs)
        assert np.array_equal(self.pool_bits(), self.o.pool)
        if self.gap is not None:
            assert np.array_equal(bits(self.wide[:, :, 1:]), self.gap)

    def extend(self, rows, count):
        import bucketed_classifier_free_amd as bcg
        got = bcg.cache_extend(self.cache, i32(rows), i32(count)).cpu().numpy()
        assert np.array_equal(got, self.o.extend(rows, count)), got
        self.same()
        return got

    def fork(self, src, dst):
        import bucketed_classifier_free_amd as bcg
        got = bcg.cache_fork(self.cache, i32(src), i32(dst)).cpu().numpy()
        assert np.array_equal(got, self.o.fork(src, dst)), got
        self.same()
        return got

    def free(self, rows, **kw):
        import bucketed_classifier_free_amd as bcg
        bcg.cache_free(self.cache, i32(rows), **kw)
        self.o.free(rows, **kw)
        self.same()

    def compact(self):
        import bucketed_classifier_free_amd as bcg
        moved = torch.zeros(1, dtype=torch.int32, device="cuda")
        bcg.cache_compact(self.cache, moved=moved)
        want = self.o.compact()
        self.same()
        assert int(moved) == want


@pytest.mark.parametrize("dtype,page,heads,dim", [(torch.bfloat16, 16, 2, 64), (torch.float32, 48, 1, 8),
                                                  (torch.float8_e4m3fn, 16, 1, 16), (torch.bfloat16, 128, 3, 128)])
@pytest.mark.parametrize("gap", [0, 1])
def test_a_life_of_pages(dtype, page, heads, dim, gap):
    b = Both([page, 0, 3 * page + 1, 0, 5, 2 * page - 1, 0], page=page, heads=heads, dim=dim, dtype=dtype, spare=9, page_gap=gap)
    b.extend([1, 4, 0], [page + 2, 0, 1])
    b.free([2])
    b.fork([1, 0, 5], [2, 3, 6])
    b.extend([2, 3, 1], [1, 1, page])
    b.free([1])
    b.compact()
    b.free([0, 5, 6])
    b.compact()
    b.compact()


def test_extend_refuses():
    b = Both([16, 10, 0, 31], spare=4, width=4)
    # outside the table; twice the same row; a negative count; beyond the width
    got = b.extend([0, -1, 4, 2 ** 31 - 1, 0, 1, 2, 3], [1, 1, 1, 1, 1, -1, 65, 2 ** 31 - 1])
    assert got.tolist() == [1, 0, 0, 0, 0, 0, 0, 0]
    # three pages are left: what does not fit is refused, and what comes behind it too
    assert b.extend([2, 1, 3], [49, 16, 33]).tolist() == [0, 0, 0]
    assert b.extend([1, 3], [6, 2]).tolist() == [1, 1]
    b.extend([2], [0])


def test_fork_refuses():
    b = Both([20, 0, 5, 0, 32, 0], spare=1)
    # not empty; itself; outside; named before
    assert b.fork([0, 1, 9, 0, 4, 0], [2, 1, 3, -1, 3, 3]).tolist() == [0, 0, 0, 0, 0, 0]
    # an entry that is refused names its row all the same; whole pages need none
    assert b.fork([4, 0, 2], [3, 5, 1]).tolist() == [1, 1, 0]
    assert b.fork([1], [1]).tolist() == [0]


def test_fork_of_an_empty_row_and_of_a_row_forked_into():
    b = Both([20, 0, 0, 0], spare=8)
    assert b.fork([1, 0], [2, 1]).tolist() == [1, 1]  # the first reads the state before the call
    assert b.o.length.tolist() == [20, 20, 0, 0]


def test_free_repeats_and_rows_outside():
    b = Both([40, 17, 90], spare=2)
    b.free([1, 1, -3, 7, 1])
    b.free([1])
    b.free([0, 2])
    assert (b.o.refs == 0).all()


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (17, 4), (40, 17), (1000, 1), (1, 1000)])
def test_free_behind_a_window(window, sinks):
    b = Both([100, 16, 0, 1, 64, 33], spare=6)
    b.free([0, 1, 2, 3, 4, 5], window=window, sinks=sinks)
    # the next token has a place, shared or not
    b.extend([0, 1, 2, 3, 4, 5], [1] * 6)
    b.free([0])
    b.fork([5, 4], [0, 2])
    b.compact()


def test_shared_pages_stay_until_their_last_row():
    b = Both([64, 0, 0, 0], spare=3)
    b.fork([0, 0, 0], [1, 2, 3])
    assert b.o.refs.max() == 4
    b.free([0, 2])
    b.free([1])
    assert b.o.refs.max() == 1
    b.free([3])


@pytest.mark.parametrize("rows,length,spare", [(200, 60, 40), (1500, 20, 700), (3, 6000, 5000), (5000, 30, 9000)])
def test_many_pages(rows, length, spare):
    rng = np.random.default_rng(rows)
    lens = [int(n) for n in rng.integers(0, length + 1, rows)]
    b = Both(lens, spare=spare, planes=2, heads=1, dim=8, dtype=torch.bfloat16, seed=rows)
    gone = [int(r) for r in rng.permutation(rows)[:rows // 3 + 1]]
    b.free(gone)
    left = [r for r in range(rows) if r not in set(gone)]
    b.fork([left[i % len(left)] for i in range(len(gone))], gone)
    b.extend(list(range(rows)), [int(x) for x in rng.integers(0, 20, rows)])
    b.compact()


def test_compact_into_other_tables():
    import bucketed_classifier_free_amd as bcg
    b = Both([50, 20, 70], spare=9, seed=4)
    b.free([1])
    table, refs = torch.zeros_like(b.cache.table), torch.zeros_like(b.cache.refs)
    before = (b.cache.table.clone(), b.cache.refs.clone())
    bcg.cache_compact(b.cache, table_out=table, refs_out=refs)
    assert torch.equal(b.cache.table, before[0]) and torch.equal(b.cache.refs, before[1])
    b.o.compact()
    b.cache.table.copy_(table)
    b.cache.refs.copy_(refs)
    b.same()


def test_copy_pages():
    import bucketed_classifier_free_amd as bcg
    b = Both([200], spare=20, planes=6)
    src, dst = [0, 5, -1, 7, 3], [1, 2, 4, 10 ** 6, 6]
    bcg.cache_copy(b.cache.pool, i32(src), i32(dst))
    for s, d in ((0, 1), (5, 2), (3, 6)):
        b.o.pool[:, d] = b.o.pool[:, s]
    b.same()


def test_step_captured_into_a_graph_and_replayed():
    """A scheduler's turn as one graph: free, fork, extend; every replay
    against the oracle, with eager work of the same kind between replays."""
    import bucketed_classifier_free_amd as bcg
    b = Both([40, 33, 90, 12], spare=12)
    done, src, one = i32([1, 3]), i32([0, 2]), i32([1, 1])
    ok1, ok2 = torch.zeros_like(done), torch.zeros_like(done)
    b.cache.reserve(4)  # the workspace is there before the capture
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        bcg.cache_free(b.cache, done)
        bcg.cache_fork(b.cache, src, done, granted=ok1)
        bcg.cache_extend(b.cache, done, one, granted=ok2)
    for _ in range(4):
        g.replay()
        torch.cuda.synchronize()
        b.o.free([1, 3])
        assert np.array_equal(ok1.cpu().numpy(), b.o.fork([0, 2], [1, 3]))
        assert np.array_equal(ok2.cpu().numpy(), b.o.extend([1, 3], [1, 1]))
        b.same()
        b.extend([0], [1])
