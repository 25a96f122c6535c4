"""The example of the paged cache: its answers against the same model in
float64 on the CPU, with whole sequences and no cache."""
import importlib.util
import math
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import kvcache as ok  # noqa: E402

from gpu_util import require_native  # noqa: E402

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    spec = importlib.util.spec_from_file_location("paged_decode", os.path.join(ROOT, "examples", "paged_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def dense_logits(model, tokens):
    """Logits of every position of one sequence in float64."""
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    x, n = f(model.embed)[tokens], len(tokens)
    thetas = ok.rope_thetas(model.dim, 10000.0, "ramp", 4.0, 4096, 1.0, 32.0)
    pos = np.arange(n)
    for layer in range(model.layers):
        q, k, v = ((x @ f(w[layer])).reshape(n, -1, model.dim) for w in (model.wq, model.wk, model.wv))
        q, k = (ok.rope(t, pos, thetas)[0] for t in (q, k))
        o = np.zeros((n, model.heads, model.dim))
        for h in range(model.heads):
            g = h // (model.heads // model.kv)
            s = q[:, h] @ k[:, g].T / math.sqrt(model.dim)
            s[np.triu_indices(n, 1)] = -np.inf
            w = np.exp(s - s.max(-1, keepdims=True))
            o[:, h] = w @ v[:, g] / w.sum(-1, keepdims=True)
        x = x + o.reshape(n, -1) @ f(model.wo[layer])
    return x @ f(model.head), x


def test_paged_decode_example():
    require_native()
    history, model, prompt, cache = load_example().generate(steps=13, answers=4, prompt=37, every=5, slots=4)
    history = history.cpu().numpy()
    assert history.shape == (4, 13)
    assert cache.lens.cpu().tolist()[0] == 37 and cache.lens.cpu().tolist()[1:5] == [12] * 4
    for row in history:
        # Each token is the likeliest one up to what bf16 costs: a logit is a sum over the residual stream, whose
        # elements were rounded about a dozen times on their way (embedding, projections, rotation, weights, result,
        # residual), relative 12 * 2^-8 at most; the errors of the 512 elements are independent, so the sum is off by
        # their root sum square times the head's 1 / sqrt(512) elements; four of those for either of two logits.
        logits, x = dense_logits(model, np.concatenate((prompt.cpu().numpy(), row)))
        slack = 2 * 4 * 12 * 2.0 ** -8 * np.sqrt((x ** 2).mean(-1))
        for i in range(1, len(row)):
            at = logits[37 + i - 1]
            assert at[row[i]] >= at.max() - slack[37 + i - 1], i
