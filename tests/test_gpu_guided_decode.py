"""examples/guided_decode.py: every step's guided logits against a plain model
without a cache (full attention under the same window, in float64), and the
pool empty at the end."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from decode_cases import np64
from oracle import decode as O

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bucketed_classifier_free_amd
    bucketed_classifier_free_amd.load()  # fails loudly without libbcg.so
    spec = importlib.util.spec_from_file_location("guided_decode", os.path.join(ROOT, "examples", "guided_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain_logits(ex, model, tokens):
    """The logits behind the last of ``tokens``, in float64 without a cache."""
    w = lambda t: t.double().cpu()  # noqa: E731
    norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    n, group = len(tokens), ex.HEADS // ex.KV_HEADS
    x = w(model.embed)[torch.tensor(tokens)]
    t = torch.arange(n)
    seen = (t <= t[:, None]) & ((t > t[:, None] - ex.WINDOW) | (t < ex.SINKS))
    for layer in range(ex.LAYERS):
        qkv = (norm(x) @ w(model.qkv[layer])).view(n, -1, ex.DIM)
        q, k, v = (y.transpose(0, 1) for y in qkv.split([ex.HEADS, ex.KV_HEADS, ex.KV_HEADS], 1))
        k, v = (y.repeat_interleave(group, 0) for y in (k, v))
        s = (q @ k.transpose(-1, -2)) * ex.DIM ** -0.5
        o = torch.softmax(s.masked_fill(~seen, -float("inf")), -1) @ v
        x = x + o.transpose(0, 1).reshape(n, -1) @ w(model.out[layer])
        x = x + torch.relu(norm(x) @ w(model.up[layer])) @ w(model.down[layer])
    return norm(x)[-1] @ w(model.head)


@pytest.mark.parametrize("samples,steps", [(1, 3), (3, 40)])
def test_every_step_is_that_of_the_model_without_a_cache(ex, samples, steps):
    """fp32: two layers of sums of at most 1024 products, each rounding 2^-24
    of values of order one to ten: logits within 1e-3 of the exact model's."""
    import bucketed_classifier_free_amd as bcg
    model = ex.Model(torch.float32, seed=samples)
    d = ex.Decoder(model, samples, steps, torch.float32, torch.float32, bcg.bucket_table("front_high", 3.0, 1.0, 0.6, 8))
    rng = np.random.default_rng(samples)
    uncond, cond = rng.integers(0, ex.VOCAB, 7).tolist(), rng.integers(0, ex.VOCAB, 75).tolist()
    allowed = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (samples, (ex.VOCAB + 31) // 32)).astype(np.int32)).cuda()
    seen = []

    def on_step(dec, step, logits, out, need, scale, kw):
        seen.append(step)
        if step % 7 and step < steps - 1:
            return
        said = dec.history.cpu().numpy()
        rows = []
        for i in range(samples):
            answer = said[i, len(cond):len(cond) + step].tolist()
            rows += [plain_logits(ex, model, uncond + answer) if need[i] else torch.zeros(ex.VOCAB, dtype=torch.float64),
                     plain_logits(ex, model, cond + answer)]
        rows = torch.stack(rows).numpy()
        z, _ = O.guided_logits(rows, np.arange(samples) * 2 + 1, [2 * i if need[i] else -1 for i in range(samples)], scale,
                               **{k: None if v is None else v.cpu().numpy() for k, v in kw.items()})
        got = np64(out)
        off = np.isneginf(z)
        assert np.array_equal(np.isneginf(got), off)
        assert np.abs(got - z)[~off].max() < 1e-3 * max(1.0, np.abs(z[~off]).max()), step

    tokens = d.run(uncond, cond, allowed=allowed, on_step=on_step)
    assert seen == list(range(steps)) and tokens.shape == (samples, steps)
    bits = np.unpackbits(allowed.cpu().numpy().view(np.uint8), axis=1, bitorder="little")
    assert all(bits[i, t] for i in range(samples) for t in tokens[i].tolist())
    assert int((d.cache.refs != 0).sum()) == 0 and int((d.cache.table >= 0).sum()) == 0


@pytest.mark.parametrize("dtype,cache", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float8_e4m3fn)])
def test_other_types_run_and_leave_the_pool_empty(ex, dtype, cache):
    import bucketed_classifier_free_amd as bcg
    d = ex.Decoder(ex.Model(dtype), 4, 20, dtype, cache, bcg.bucket_table("linear", 2.0, 1.0, 0.0, 4))
    a = d.run(list(range(5)), list(range(50)))
    b = d.run(list(range(5)), list(range(50)))
    assert torch.equal(a, b)  # the same request on a used pool
    assert int((d.cache.refs != 0).sum()) == 0
