"""The layer norm of rows that lie far from 0 for their spread: xh = (x - mean) rstd has no rounding of the
size of mean rstd in it, in either direction, from a tensor or from a checkpoint.

u = 2^-24 is half a step of fp32 relative to the value. A sum over a row runs over at most 32 terms a
thread and 10 levels of a tree and its products: 48 u of the sum of magnitudes, 64 u with the factors."""

import numpy as np
import pytest
import torch

from oracle import ckpt8 as ockpt
from oracle import norm as onorm
from tests.test_gpu_around import DTYPES, U, close, f64, half_step, pitched

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def B():
    from int4_quantised_moe_b200 import binding
    return binding


@pytest.mark.parametrize("source", ["tensor", "e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("width,pad", [(1, 0), (7, 2), (64, 0), (704, 0), (2816, 8), (2817, 0), (4104, 0), (7168, 0),
                                       (16383, 0), (16384, 0)])
def test_rows_of_one_value(B, source, dtype, width, pad):
    """Mean: the value itself. y: the bias. dw: 0. dx: rstd (w dy - mean(w dy))."""
    dt = DTYPES[dtype]
    values = torch.tensor([5.0, 1000.3, 0.1, -7.0 / 3, 60000.0, 1e-3, 0.0, -1.0], dtype=torch.double).to(dt)
    x = values[:, None].expand(8, width).contiguous()
    xc = pitched(x, pad)
    g = torch.Generator().manual_seed(width)
    w, b = 1 + 0.1 * torch.randn(width, generator=g), torch.randn(width, generator=g)
    gy = torch.randn((8, width), generator=g).to(dt)
    x_in = xc if source == "tensor" else B.ckpt8_save(xc, source)
    held = f64(x) if source == "tensor" else ockpt.load(f64(x_in.codes).astype(np.uint8), f64(x_in.scales), source)
    kw = {} if source == "tensor" else {"dtype": dt}
    y, mean, rstd, _ = B.norm_fwd(x_in, w.cuda(), b.cuda(), kind="layer", eps=EPS, **kw)
    assert np.array_equal(f64(mean), held[:, 0])
    assert torch.equal(y, b.to(dt).cuda().expand_as(y))
    # the first mean is off by at most 64 u of the value; its square cancels up to four roundings
    wrong = 4 * U * (64 * U * held[:, 0]) ** 2 / EPS
    close(rstd, np.full(8, EPS ** -0.5), EPS ** -0.5 * (8 * U + wrong))
    dx, dw, db = B.norm_bwd(pitched(gy, pad), x_in, rstd, w.cuda(), mean=mean, kind="layer", bias_grad=True)
    assert not dw.any()
    wg = f64(gy) * f64(w)
    want = f64(rstd)[:, None] * (wg - wg.mean(1, keepdims=True))
    close(dx, want, 64 * U * f64(rstd)[:, None] * (np.abs(wg) + np.abs(wg).mean(1, keepdims=True)) + half_step(want, dt))
    close(db, f64(gy).sum(0), 8 * U * np.abs(f64(gy)).sum(0))


@pytest.mark.parametrize("rows,width,dtype,centre,pad", [
    (300, 704, "fp32", 1e4, 0), (300, 704, "fp32", 1e4, 3), (9, 2817, "fp32", 3e3, 0), (40, 2816, "fp32", 1e5, 0),
    (33, 7168, "fp16", 1e3, 0), (33, 7168, "fp32", 1e3, 0), (700, 257, "fp32", -1e4, 0), (12, 16384, "fp32", 1e4, 0)])
def test_rows_far_from_zero(B, rows, width, dtype, centre, pad):
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(rows + width)
    x = (torch.randn((rows, width), generator=g) + centre).to(dt)
    w = 1 + 0.1 * torch.randn(width, generator=g)
    gy = torch.randn((rows, width), generator=g).to(dt)
    xc, gc = pitched(x, pad), pitched(gy, pad)
    y, mean, rstd, _ = B.norm_fwd(xc, w.cuda(), kind="layer", eps=EPS)
    oy, omean, orstd = onorm.forward(f64(x), f64(w), None, "layer", EPS)
    # the mean: its own rounding, and what the centred sum leaves: 64 u of the first mean's error and of the spread
    emean = U * np.abs(omean) + 64 * U * (64 * U * np.abs(omean) + np.abs(f64(x) - omean[:, None]).mean(1))
    close(mean, omean, emean, "mean")
    close(rstd, orstd, 64 * U * orstd, "rstd")
    xh = (f64(x) - omean[:, None]) * orstd[:, None]
    exh = 70 * U * np.abs(xh) + (orstd * emean)[:, None]
    close(y, oy, exh * f64(w) + 2 * U * np.abs(oy) + half_step(oy, dt), "y")

    # the backward, for the statistics that it is given
    m, r = f64(mean), f64(rstd)
    odx, odw, odb = onorm.backward(f64(gy), f64(x), m, r, f64(w), "layer")
    xh = (f64(x) - m[:, None]) * r[:, None]
    dx, dw, db = B.norm_bwd(gc, xc, rstd, w.cuda(), mean=mean, kind="layer", bias_grad=True)
    wg = np.abs(f64(gy) * f64(w))
    m2 = (wg * np.abs(xh)).mean(1, keepdims=True)
    tol = 70 * U * r[:, None] * (wg + wg.mean(1, keepdims=True) + 2 * np.abs(xh) * m2)
    close(dx, odx, tol + half_step(odx, dt), "dx")
    terms = (rows + 8) * U  # one by one at most, and the factors' roundings
    close(dw, odw, terms * (np.abs(f64(gy)) * np.abs(xh)).sum(0), "dw")
    close(db, odb, terms * np.abs(f64(gy)).sum(0), "db")
