"""guided_logits against its definition in float64 (oracle/decode.py).

Bounds: every fp32 operation of the chain rounds a value of at most `reach`
(the oracle's second result) by 2^-24 of it; there are at most nine (the
difference, the fused multiply-add, the penalty, the product and the two
differences of the counts, the bias, the temperature and one to spare), then
one rounding to the output's type.
"""
import numpy as np
import pytest
import torch

from decode_cases import TYPES, half_step, np64
from oracle import decode as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bucketed_classifier_free_amd
    bucketed_classifier_free_amd.load()  # fails loudly without libbcg.so


def case(n, vocab, q, seed=0, hist=0, biases=0, mask=False, guided=True, pad=0):
    rng = np.random.default_rng(seed)
    m = n // 2 if guided else 0
    wide = torch.from_numpy(rng.standard_normal((m + n, vocab + pad)).astype(np.float32) * 3).to(TYPES[q]).cuda()
    kw = {}
    urow = np.full(n, -1, np.int32)
    urow[rng.permutation(n)[:m]] = np.arange(m)
    scale = np.where(urow < 0, 1.0, rng.uniform(1.2, 8, n)).astype(np.float32)
    kw.update(cond_row=np.arange(m, m + n, dtype=np.int32), uncond_row=urow, scale=scale)
    if hist:
        kw.update(history=(rng.random((n, hist)) ** 3 * vocab).astype(np.int32),
                  history_len=rng.integers(0, hist + 1, n).astype(np.int32))
        kw.update(prompt_len=(kw["history_len"] * rng.random(n)).astype(np.int32),
                  repetition=rng.uniform(0.8, 1.6, n).astype(np.float32), presence=rng.uniform(-1, 1, n).astype(np.float32),
                  frequency=rng.uniform(-0.3, 0.6, n).astype(np.float32))
    if biases:
        kw.update(bias_ids=rng.integers(0, vocab, (n, biases)).astype(np.int32),
                  bias=rng.standard_normal((n, biases)).astype(np.float32) * 4)
    kw["temperature"] = rng.uniform(0.3, 2, n).astype(np.float32)
    if mask:
        kw["mask"] = rng.integers(-2 ** 31, 2 ** 31, (n, (vocab + 31) // 32)).astype(np.int32)
    return wide[:, :vocab], kw


def run(logits, kw, out="f32", pad=0):
    import bucketed_classifier_free_amd as bcg
    n, vocab = len(kw["cond_row"]), logits.shape[1]
    wide = torch.full((n, vocab + pad), 7.0, dtype=TYPES[out], device="cuda")
    bcg.guided_logits(logits, wide[:, :vocab], **{k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in kw.items()})
    torch.cuda.synchronize()
    assert (wide[:, vocab:] == 7.0).all()
    return wide[:, :vocab]


def check(logits, kw, out="f32", pad=0):
    got = np64(run(logits, kw, out, pad))
    z, reach = O.guided_logits(np64(logits), **kw)
    off = z == -np.inf
    assert np.array_equal(got == -np.inf, off)
    tol = 9 * 2.0 ** -24 * reach + (half_step(TYPES[out]) * (np.abs(z) + 9 * 2.0 ** -24 * reach) if out != "f32" else 0)
    bad = (np.abs(got - z) > tol) & ~off
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], z[bad][:3])


@pytest.mark.parametrize("q", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab", [(1, 1), (1, 7), (3, 8), (2, 33), (5, 4097), (4, 4095), (2, 50001), (7, 12288)])
def test_combine_and_mask(q, out, n, vocab):
    check(*case(n, vocab, q, seed=vocab, mask=True), out=out)
    check(*case(n, vocab, q, seed=vocab + 1, guided=False), out=out)


@pytest.mark.parametrize("q", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,hist,biases", [(2, 1000, 50, 0), (3, 9001, 1, 3), (4, 4099, 5000, 100), (1, 30000, 0, 4096), (6, 70, 300, 40)])
def test_penalties_and_biases(q, n, vocab, hist, biases):
    check(*case(n, vocab, q, seed=hist, hist=hist, biases=biases, mask=True))


@pytest.mark.parametrize("pad_in,pad_out", [(1, 0), (0, 1), (3, 5), (8, 8)])
def test_row_strides(pad_in, pad_out):
    for q in ("bf16", "f32"):
        logits, kw = case(5, 4111, q, seed=pad_in, hist=20, biases=4, mask=True, pad=pad_in)
        check(logits, kw, pad=pad_out)


def test_values_that_are_not_finite():
    """A masked token is -infinity whatever its logits hold; equal infinities
    of both branches stay; a visible NaN stays."""
    logits, kw = case(4, 600, "f32", seed=3, mask=True)
    low = torch.finfo(torch.float32).min
    logits[:, 0:3] = float("nan")
    logits[:, 5] = float("inf")
    logits[:, 6] = -float("inf")
    logits[:, 7] = low
    kw["mask"][:, 0] = 0b11100000  # tokens 0..4 and 8.. of the first word are masked
    got = np64(run(logits, kw))
    assert np.isneginf(got[:, :5]).all()
    assert (got[:, 5] == np.inf).all() and (got[:, 6] == -np.inf).all()
    want = np.maximum(low / kw["temperature"].astype(np.float64), -np.inf)
    assert np.allclose(got[:, 7], np.where(want < low, -np.inf, want), rtol=1e-6)
    kw["mask"][1] = 0   # nothing is left of this row
    kw["mask"][2] = -1
    got = np64(run(logits, kw))
    assert np.isneginf(got[1]).all() and np.isnan(got[2, :3]).all() and np.isfinite(got[2, 8:]).all()


def test_ids_lengths_and_rows_out_of_range():
    logits, kw = case(6, 500, "f32", seed=5, hist=40, biases=10)
    kw["history"][0, ::3] = [-1, 500, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 500, -7, 501, 700, 502, -2, 503, 504, -9][:len(kw["history"][0, ::3])]
    kw["bias_ids"][1, :4] = [-1, 500, 2 ** 31 - 1, -2 ** 31]
    kw["history_len"][2], kw["history_len"][3] = -4, 10 ** 6
    kw["prompt_len"][4], kw["prompt_len"][5] = -3, 10 ** 6
    want_u = kw["uncond_row"].copy()
    check(logits, kw)
    kw["uncond_row"] = want_u.copy()
    i = int(np.argmax(want_u >= 0))
    kw["uncond_row"][i] = 10 ** 6      # counts as none
    kw["cond_row"] = kw["cond_row"].copy()
    check(logits, kw)
    kw["cond_row"][0], kw["cond_row"][1] = -1, 10 ** 6  # not written
    got = run(logits, kw)
    assert (got[:2] == 7.0).all()


def test_penalties_without_a_history_do_nothing():
    logits, kw = case(3, 300, "f32", seed=8, hist=5)
    want = run(logits, {k: v for k, v in kw.items() if k in ("cond_row", "uncond_row", "scale", "temperature")})
    got = run(logits, {k: v for k, v in kw.items() if k not in ("history", "history_len", "prompt_len")})
    assert torch.equal(got, want)


def test_the_last_bias_of_a_token_counts():
    logits, kw = case(1, 100, "f32", seed=6, guided=False)
    kw["bias_ids"] = np.array([[5, 9, 5, 9, 5]], np.int32)
    kw["bias"] = np.array([[1, 2, 3, 4, 50]], np.float32)
    check(logits, kw)


def test_one_row_serves_several_samples_and_the_plans_rows():
    """The rows of bcg_plan_build: [uncond (compacted) | cond]."""
    import bucketed_classifier_free_amd as bcg
    table = bcg.bucket_table("front_high", 3.0, 1.0, 0.5, 4)
    plan = bcg.bcg_plan_build([0, 7, 2, 5, 1], 8, table)
    rows = plan.n_uncond + 5
    g = torch.Generator().manual_seed(1)
    logits = torch.randn((rows, 777), generator=g).cuda()
    kw = dict(cond_row=np.asarray(plan.cond_row, np.int32), uncond_row=np.asarray(plan.uncond_row, np.int32),
              scale=np.asarray(plan.scale, np.float32))
    assert 0 < plan.n_uncond < 5
    check(logits, kw)
    kw["cond_row"][:] = rows - 1
    check(logits, kw)


def test_the_combine_is_that_of_the_guided_step():
    """Without a schedule's step the combine of guided_step_rows is
    fma(w, c - u, u), bit for bit (w == 1: c)."""
    logits, kw = case(8, 5000, "f32", seed=9)
    del kw["temperature"]
    got = run(logits, kw).cpu().numpy()
    x = logits.cpu().numpy()
    for i in range(8):
        c, w = x[kw["cond_row"][i]], kw["scale"][i]
        if kw["uncond_row"][i] < 0:
            want = c
        else:
            u = x[kw["uncond_row"][i]]
            d = (c - u).astype(np.float64)          # one fp32 rounding
            exact = d * np.float64(w)               # 24 x 24 bits: exact in float64
            want = (exact + u.astype(np.float64)).astype(np.float32)  # double rounding: one in 2^29
        assert (got[i] != want).mean() <= 1e-3
        assert np.abs(got[i] - want).max() <= 2.0 ** -22 * np.abs(want).max()
