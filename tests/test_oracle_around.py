"""Pins of the float64 oracles of the operators around the layer (oracle.select, oracle.ckpt8,
oracle.norm): brute force, closed forms, central differences, torch autograd. CPU only."""

import itertools

import numpy as np
import pytest
import torch

from oracle import ckpt8, norm, select


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
def test_selection_is_the_best_set(score, bias):
    """The chosen set has the largest sum of keys of all sets inside the kept groups."""
    rng = np.random.default_rng(1)
    s = rng.normal(size=(20, 8))
    b = rng.normal(size=8) * 0.2 if bias else None
    ids, _ = select.forward(s, 3, score, b, groups=4, kept=2, group_top=2)
    for t in range(20):
        key = select.probabilities(s[t], score) + (b if bias else 0)
        scores = key.reshape(4, 2).sum(axis=1)
        best = max(itertools.combinations(range(4), 2), key=lambda c: scores[list(c)].sum())
        inside = [e for g in best for e in (2 * g, 2 * g + 1)]
        want = max(itertools.combinations(inside, 3), key=lambda c: key[list(c)].sum())
        assert set(want) == set(ids[t])
        assert np.all(np.diff(key[ids[t]]) <= 0)


def test_selection_ties_and_masked_scores():
    ids, w = select.forward([[1.0, 2.0, 2.0, 1.0]], 3)
    assert ids.tolist() == [[1, 2, 0]]
    ids, w = select.forward([[-np.inf, 0.5, np.nan, -np.inf], [-np.inf] * 4], 2)
    assert ids.tolist() == [[1, 0], [0, 1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]]
    # one expert left in the last group: that group is chosen
    s = np.full((1, 8), -np.inf)
    s[0, 7] = -3.0
    assert select.forward(s, 1, groups=4, kept=1, group_top=2)[0].tolist() == [[7]]
    assert select.forward(s, 1, bias=np.full(8, -5.0), groups=4, kept=1, group_top=2)[0].tolist() == [[7]]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_selection_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    s, g = rng.normal(size=(4, 7)), rng.normal(size=(4, 3))
    ids, _ = select.forward(s, 3, score, renorm=renorm, scale=2.5)

    def loss(z):
        out = 0.0
        for t in range(4):
            p = select.probabilities(z[t], score)[ids[t]]
            out += (g[t] * 2.5 * (p / p.sum() if renorm else p)).sum()
        return out

    grad = select.backward(s, ids, g, score, renorm, 2.5)
    num = np.zeros_like(s)
    for i in np.ndindex(*s.shape):
        d = np.zeros_like(s)
        d[i] = 1e-6
        num[i] = (loss(s + d) - loss(s - d)) / 2e-6
    np.testing.assert_allclose(grad, num, atol=1e-8)  # differences: 2.5 * 1e-16 / 1e-6 and a second-order term


def test_e4m3_table_and_rounding_match_torch():
    v = torch.tensor(np.arange(256), dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ckpt8.e4m3_values(), v)
    x = np.random.default_rng(3).normal(size=2000) * np.exp2(np.random.default_rng(4).integers(-12, 6, 2000))
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = np.array([ckpt8._code_e4m3(float(a)) for a in x])
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_checkpoint_error_is_half_a_step(fmt):
    rng = np.random.default_rng(5)
    x = (rng.normal(size=(6, 77)) * np.exp2(rng.integers(-20, 20, size=(6, 1)))).astype(np.float32).astype(np.float64)
    x[2, 32:64] = 0.0
    codes, scales = ckpt8.save(x, fmt)
    y = ckpt8.load(codes, scales, fmt)
    step = np.repeat(2.0 ** (scales.astype(float) - 127), 32, axis=1)[:, :77]
    if fmt == "e4m3":
        half = np.maximum(np.exp2(np.floor(np.log2(np.maximum(np.abs(x) / step, 2.0 ** -6)))) / 16, 2.0 ** -10)
    else:
        half = 0.5
    assert np.all(np.abs(x - y) <= half * step)
    assert scales[2, 1] == 1  # nothing to scale
    # the exponent is the smallest that fits
    for r, g in np.ndindex(*scales.shape):
        amax = np.abs(x[r, 32 * g:32 * g + 32]).max()
        e = int(scales[r, g]) - 127
        assert amax == 0 or (ckpt8._fits(amax, e, fmt) and not ckpt8._fits(amax, e - 1, fmt))


def test_checkpoint_not_finite():
    for fmt in ("e4m3", "int8"):
        codes, scales = ckpt8.save([[1.0, np.inf, -np.inf, np.nan, -2.0]], fmt)
        y = ckpt8.load(codes, scales, fmt)[0]
        assert y[0] == 1.0 and y[4] == -2.0 and np.isnan(y[1:4]).all()


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_against_differences_and_autograd(kind):
    rng = np.random.default_rng(6)
    x, w, b, g = rng.normal(size=(3, 9)) + 0.5, rng.normal(size=9), rng.normal(size=9), rng.normal(size=(3, 9))
    y, mean, rstd = norm.forward(x, w, b, kind, 1e-3)
    dx, dw, db = norm.backward(g, x, mean, rstd, w, kind)
    xt, wt, bt = (torch.tensor(v, requires_grad=True) for v in (x, w, b))
    if kind == "layer":
        yt = torch.nn.functional.layer_norm(xt, (9,), wt, bt, 1e-3)
    else:
        yt = xt * torch.rsqrt((xt * xt).mean(1, keepdim=True) + 1e-3) * wt + bt
    yt.backward(torch.tensor(g))
    for got, want in ((y, yt), (dx, xt.grad), (dw, wt.grad), (db, bt.grad)):
        np.testing.assert_allclose(got, want.detach().numpy(), rtol=1e-12, atol=1e-13)
    num = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        d = np.zeros_like(x)
        d[i] = 1e-6
        num[i] = (g * (norm.forward(x + d, w, b, kind, 1e-3)[0] - norm.forward(x - d, w, b, kind, 1e-3)[0])).sum() / 2e-6
    np.testing.assert_allclose(dx, num, atol=2e-8)
