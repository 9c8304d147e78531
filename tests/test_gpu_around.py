"""GPU parity of the operators around the layer with their float64 oracles: expert selection and its
backward, 8-bit checkpoints, the norm and its backward from a tensor or from a checkpoint.

u = 2^-24 is half a step of fp32 relative to the value. Whole numbers (ids, counts, codes, scale bytes)
match exactly. Each tolerance on a computed number is a sum of roundings, stated where it is built; a
result of type t adds torch.finfo(t).eps / 2 relative for its own rounding (and half the smallest
subnormal)."""

import numpy as np
import pytest
import torch

from oracle import ckpt8 as ockpt
from oracle import norm as onorm
from oracle import select as oselect

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
GUARD = 0x5A


@pytest.fixture(scope="module")
def B():
    from int4_quantised_moe_b200 import binding
    return binding


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(want, dtype):
    info = torch.finfo(dtype)
    return np.abs(want) * (info.eps / 2) + info.smallest_normal * info.eps / 2


def close(got, want, tol, what=""):
    got = f64(got)
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(err - tol)), np.argwhere(bad)[:3].tolist(),
                           got[bad][:3], np.asarray(want)[bad][:3])


def pitched(t, pad):
    if not pad:
        return t.cuda()
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t.cuda()
    return buf[:, :t.shape[1]]


# ------------------------------------------------------------------ selection

SELECT = [
    # Q, E, k, score, dtype, groups, kept, group_top, bias, renorm, pad
    (1, 384, 8, "sigmoid", "fp32", 1, 1, 1, True, True, 0),
    (257, 384, 8, "sigmoid", "fp32", 1, 1, 1, True, True, 0),
    (64, 256, 8, "sigmoid", "bf16", 8, 4, 2, True, True, 0),
    (65, 256, 8, "sigmoid", "fp16", 8, 3, 2, True, False, 5),
    (33, 128, 8, "softmax", "bf16", 1, 1, 1, False, False, 0),
    (33, 128, 8, "softmax", "fp32", 4, 2, 1, False, True, 3),
    (40, 60, 6, "softmax", "fp32", 5, 3, 2, True, True, 0),
    (40, 60, 6, "softmax", "fp32", 5, 3, 2, False, False, 0),
    (7, 1, 1, "sigmoid", "fp32", 1, 1, 1, False, False, 0),
    (9, 2, 2, "sigmoid", "bf16", 2, 2, 1, True, True, 1),
    (17, 33, 32, "sigmoid", "fp32", 1, 1, 1, True, True, 0),
    (5, 31, 3, "softmax", "fp16", 1, 1, 1, True, True, 0),
    (5, 512, 10, "sigmoid", "bf16", 32, 7, 1, False, True, 8),
    (5, 1000, 16, "sigmoid", "fp32", 20, 9, 2, True, True, 0),
    (3, 4096, 32, "softmax", "fp32", 1, 1, 1, True, False, 0),
    (3, 4096, 32, "sigmoid", "bf16", 32, 16, 2, True, True, 0),
    (300, 16, 4, "sigmoid", "fp32", 4, 2, 2, True, True, 0),
    (3, 1536, 8, "sigmoid", "fp32", 1, 1, 1, False, True, 0),
    (4, 96, 8, "sigmoid", "fp32", 3, 1, 2, True, True, 0),
]


def select_case(case, seed=0):
    Q, E, k, score, dtype, groups, kept, top, bias, renorm, pad = case
    g = torch.Generator().manual_seed(seed + Q + 31 * E + k)
    z = (torch.randn((Q, E), generator=g) * 1.5).to(DTYPES[dtype])
    b = torch.randn(E, generator=g) * 0.1 if bias else None
    gr = torch.randn((Q, k), generator=g)
    return z, b, gr


def run_select(B, case, z, b, gr, scale=2.5):
    Q, E, k, score, dtype, groups, kept, top, bias, renorm, pad = case
    cfg = B.make_select_cfg(E, k, score=score, groups=groups, groups_kept=kept, group_top=top, renormalise=renorm,
                            scale=scale)
    zc = pitched(z, pad)
    counts = torch.full((E,), -5, dtype=torch.int32, device="cuda")
    ids, w = B.router_select(zc, cfg, b.cuda() if b is not None else None, counts=counts)
    return cfg, zc, counts, ids, w, B.router_select_bwd(zc, cfg, ids, gr.cuda())


def share_tolerance(z, k):
    """Relative error of a probability or its share: the exponent's argument is a rounded difference of
    scores (their range times u), exp is good to 2 ulp (4 u), the sum of up to k or E/32 + 5 terms, a
    product, a quotient and the scale to u each; every one counted twice for numerator and sum."""
    zz = f64(z)
    zz = zz[np.isfinite(zz)]
    spread = float(zz.max() - zz.min()) if zz.size else 0.0
    return 2 * U * (spread + np.abs(zz).max(initial=0.0) + 4 + z.shape[1] / 32 + 5 + k + 8)


@pytest.mark.parametrize("case", SELECT, ids=[f"{c[0]}x{c[1]}k{c[2]}-{c[3]}-{c[4]}-g{c[5]}" for c in SELECT])
def test_select_and_gradient(B, case):
    Q, E, k, score, dtype, groups, kept, top, bias, renorm, pad = case
    z, b, gr = select_case(case)
    cfg, zc, counts, ids, w, grad = run_select(B, case, z, b, gr)
    o_ids, o_w = oselect.forward(f64(z), k, score, None if b is None else f64(b), groups, kept, top, renorm, 2.5)
    assert np.array_equal(ids.cpu().numpy(), o_ids)
    assert np.array_equal(counts.cpu().numpy(), np.bincount(o_ids.reshape(-1), minlength=E))
    rel = share_tolerance(z, k)
    close(w, o_w, rel * o_w, "weights")
    want = oselect.backward(f64(z), o_ids, f64(gr), score, renorm, 2.5)
    # a slot's gradient is share (g - mean) slope: the error of each factor times |g| + mean |g|
    size = np.abs(o_w) * (np.abs(f64(gr)) + (np.abs(f64(gr)) * np.abs(o_w)).sum(1, keepdims=True))
    slot = np.zeros((Q, E))
    np.put_along_axis(slot, o_ids, size, axis=1)
    if score == "softmax" and not renorm:
        p = np.stack([oselect.probabilities(row, score) for row in f64(z)])
        slot = slot + p * (np.abs(f64(gr)) * np.abs(o_w)).sum(1, keepdims=True)
    close(grad, want, 3 * rel * slot + half_step(want, grad.dtype), "grad_scores")
    if renorm or score == "sigmoid":
        mask = np.ones((Q, E), bool)
        np.put_along_axis(mask, o_ids, False, axis=1)
        assert not f64(grad)[mask].any()


MANY = [
    # E, k, score, dtype, bias, renorm, pad, Q
    (128, 8, "softmax", "bf16", False, False, 0, 32768),
    (128, 8, "sigmoid", "fp32", True, True, 0, 32769),
    (128, 8, "softmax", "fp32", True, False, 8, 32770),
    (64, 8, "sigmoid", "fp16", False, True, 0, 40003),
    (60, 6, "softmax", "fp32", False, True, 3, 32771),
    (8, 8, "sigmoid", "bf16", True, True, 0, 32768),
    (5, 3, "softmax", "fp16", True, True, 1, 33000),
    (1, 1, "sigmoid", "bf16", False, False, 0, 32768),
    (100, 1, "softmax", "bf16", False, True, 0, 32768),
]


@pytest.mark.parametrize("case", MANY, ids=[f"{c[0]}k{c[1]}-{c[2]}-{c[3]}" for c in MANY])
def test_select_many_tokens(B, case):
    """Batches of 32768 tokens and more take their own kernels: every token's selection is that of the
    same token in a batch of 4096, every 97th is the oracle's; weights and gradients agree as two fp32
    results of the same formulas do. Ties, masked experts, NaN and whole rows without a score included."""
    E, k, score, dtype, bias, renorm, pad, Q = case
    g = torch.Generator().manual_seed(E * 10 + k)
    z = torch.randn((Q, E), generator=g) * 1.5
    z[::5] = z[::5].round()  # ties
    z[torch.rand((Q, E), generator=g) < 0.02] = -np.inf
    z[3::211] = -np.inf
    z[7::301, 0] = float("nan")
    if E > 16:
        z[11::103, 16:] = -np.inf  # all that is left lies in one lane
        z[11::103, :16] = 9.0 + 1e-6 * torch.rand((len(range(11, Q, 103)), 16), generator=g)
    z = z.to(DTYPES[dtype])
    b = torch.randn(E, generator=g) * 0.1 if bias else None
    gr = torch.randn((Q, k), generator=g)
    zc, bc, gc = pitched(z, pad), None if b is None else b.cuda(), gr.cuda()
    cfg = B.make_select_cfg(E, k, score=score, renormalise=renorm, scale=1.5)
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    ids, w = B.router_select(zc, cfg, bc, counts=counts)
    grad = B.router_select_bwd(zc, cfg, ids, gc)
    for lo in range(0, Q, 4096):
        ids2, w2 = B.router_select(zc[lo:lo + 4096], cfg, bc)
        assert torch.equal(ids[lo:lo + 4096], ids2)
        torch.testing.assert_close(w[lo:lo + 4096], w2, rtol=64 * U, atol=0)
        grad2 = B.router_select_bwd(zc[lo:lo + 4096], cfg, ids2, gc[lo:lo + 4096])
        step = torch.finfo(z.dtype).eps  # two roundings of nearly the same value may differ by a step
        torch.testing.assert_close(grad[lo:lo + 4096], grad2, rtol=2 * step, atol=64 * U * 8)
    assert torch.equal(counts.cpu(), torch.bincount(ids.reshape(-1), minlength=E).int().cpu())
    pick = sorted(set(range(0, Q, 97)) | set(range(11, Q, 1030)) | {Q - 1})
    want, ow = oselect.forward(f64(z[pick]), k, score, None if b is None else f64(b), 1, 1, 1, renorm, 1.5)
    assert np.array_equal(ids.cpu().numpy()[pick], want)
    close(w[pick], ow, share_tolerance(z[pick], k) * ow, "weights")


def test_select_gradient_against_differences(B):
    """Weights of the device at s + d and s - d against the device's gradient. d = 2^-6 is exact; the
    third derivative is at most 1 in magnitude times the scale and sum of |g|: d^2 / 6 of it; the
    weights' roundings come in over 2 d."""
    case = (1, 24, 5, "sigmoid", "fp32", 1, 1, 1, False, True, 0)
    z, b, gr = select_case(case)
    z = (z * 64).round() / 64
    cfg, zc, _, ids, _, grad = run_select(B, case, z, b, gr, scale=1.0)
    d = 2.0 ** -6
    for j in range(24):
        lo, hi = zc.clone(), zc.clone()
        hi[0, j] += d
        lo[0, j] -= d
        out = []
        for s in (hi, lo):
            i2, w2 = B.router_select(s, cfg)
            full = torch.zeros(24, dtype=torch.double, device="cuda").index_put_((i2[0],), w2[0].double())
            if set(i2[0].tolist()) != set(ids[0].tolist()):
                break  # the step changed the choice
            out.append((full[ids[0]] * gr[0].double().cuda()).sum())
        if len(out) == 2:
            num = (out[0] - out[1]).item() / (2 * d)
            gsum = gr.abs().sum().item()
            assert abs(num - grad[0, j].item()) <= gsum * (d * d / 6 + 64 * U / d)


def test_select_ties_and_near_ties(B):
    """Few distinct bf16 scores (ties go to the lower index), and fp32 keys p + b that differ by far less
    than an fp32 rounding of them."""
    g = torch.Generator().manual_seed(5)
    for groups, kept, top, score in ((1, 1, 1, "sigmoid"), (8, 3, 1, "softmax"), (8, 3, 2, "softmax")):
        z = torch.randint(-3, 4, (200, 128), generator=g).to(torch.bfloat16)
        cfg = B.make_select_cfg(128, 8, score=score, groups=groups, groups_kept=kept, group_top=top)
        for b in (None, torch.zeros(128)):
            ids, _ = B.router_select(z.cuda(), cfg, None if b is None else b.cuda())
            want, _ = oselect.forward(f64(z), 8, score, None if b is None else f64(b), groups, kept, top)
            assert np.array_equal(ids.cpu().numpy(), want)
    # keys within a few 1e-9 of one another: p is flat at large scores, the bias differs in its last bits
    z = (9.0 + torch.rand((300, 64), generator=g) * 4e-3).float()
    b = (0.5 + torch.randint(0, 2, (64,), generator=g) * 2.0 ** -24).float()
    cfg = B.make_select_cfg(64, 6, groups=8, groups_kept=4, group_top=2)
    ids, _ = B.router_select(z.cuda(), cfg, b.cuda())
    want, _ = oselect.forward(f64(z), 6, "sigmoid", f64(b), 8, 4, 2)
    assert np.array_equal(ids.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_select_equal_scores(B, dtype):
    """A router at its start: every score the same, with and without groups and a bias of zeros."""
    z = torch.zeros((40, 96), dtype=DTYPES[dtype])
    z[20:] = -3.25
    z[30:, ::2] = -0.0
    for groups, kept, top in ((1, 1, 1), (8, 3, 2)):
        for b in (None, torch.zeros(96)):
            cfg = B.make_select_cfg(96, 8, groups=groups, groups_kept=kept, group_top=top)
            ids, w = B.router_select(z.cuda(), cfg, None if b is None else b.cuda())
            want, ow = oselect.forward(f64(z), 8, "sigmoid", None if b is None else f64(b), groups, kept, top)
            assert np.array_equal(ids.cpu().numpy(), want)
            close(w, ow, share_tolerance(z, 8) * ow)


def test_select_past_32_bit_offsets(B):
    """Rows 2^32 elements into a buffer of scores."""
    pitch, rows = 1 << 20, 4200
    buf = torch.empty((rows, pitch), dtype=torch.bfloat16, device="cuda")
    z = buf[:, :64]
    z.copy_(torch.randn((rows, 64), generator=torch.Generator().manual_seed(6)))
    dense = z.contiguous()
    gr = torch.randn((rows, 4), generator=torch.Generator().manual_seed(7)).cuda()
    for score, bias in (("softmax", None), ("sigmoid", torch.linspace(-0.1, 0.1, 64, device="cuda"))):
        cfg = B.make_select_cfg(64, 4, score=score, renormalise=False)
        ids, w = B.router_select(z, cfg, bias)
        ids2, w2 = B.router_select(dense, cfg, bias)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)
        assert torch.equal(B.router_select_bwd(z, cfg, ids, gr), B.router_select_bwd(dense, cfg, ids2, gr))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_select_masked_and_extreme_scores(B, score, renorm, groups):
    """Masked experts (-inf), the type's lowest value, NaN, whole rows without a score, scores whose
    probabilities leave fp32's range."""
    g = torch.Generator().manual_seed(11)
    z = torch.randn((12, 32), generator=g)
    low = torch.finfo(torch.float32).min
    z[0, :] = -np.inf
    z[1, 3:] = -np.inf
    z[2, 5] = float("nan")
    z[3, :] = float("nan")
    z[4, ::2] = low
    z[5, :] = low
    z[6, :] = -200.0 + z[6, :]
    z[7, :] = 90.0 + z[7, :]
    z[8, 31] = np.inf
    z[9, 10:] = -np.inf
    z[9, 30] = -120.0
    z[10, :] = -np.inf
    z[10, 29] = 0.25
    gr = torch.randn((12, 4), generator=g)
    kept = 2 if groups > 1 else 1
    cfg = B.make_select_cfg(32, 4, score=score, groups=groups, groups_kept=kept, group_top=2 if groups > 1 else 1,
                            renormalise=renorm)
    for b in (None, torch.randn(32, generator=g) * 0.1):
        ids, w = B.router_select(z.cuda(), cfg, None if b is None else b.cuda())
        want, ow = oselect.forward(f64(z), 4, score, None if b is None else f64(b), groups, kept,
                                   2 if groups > 1 else 1, renorm)
        if b is None:
            # row 7: in 64 bits the group sums of p near 1 are told apart exactly, as here
            assert np.array_equal(ids.cpu().numpy(), want)
        else:
            rows = [r for r in range(12) if r != 7]  # row 7 with a bias: p = 1 - 1e-39 rounds to 1 in 64 bits too
            assert np.array_equal(ids.cpu().numpy()[rows], want[rows])
        got = f64(w)
        keep = (ids.cpu().numpy() == want).all(axis=1)
        tol = 2 * U * (220 + 64) * np.abs(ow) + 2.0 ** -126
        assert np.all(np.abs(got - ow)[keep] <= tol[keep])
        assert not got[[0, 3]].any()
        grad = f64(B.router_select_bwd(z.cuda(), cfg, ids, gr.cuda()))
        og = oselect.backward(f64(z), ids.cpu().numpy(), f64(gr), score, renorm)
        assert np.isfinite(grad).all()
        assert np.all(np.abs(grad - og) <= 2 * U * 900 * np.abs(f64(gr)).sum(1, keepdims=True) + 2.0 ** -126)


def test_select_bias_of_infinity_ranks_last(B):
    z = torch.randn((6, 16), generator=torch.Generator().manual_seed(3))
    b = torch.zeros(16)
    b[::2] = -np.inf
    b[1] = float("nan")
    cfg = B.make_select_cfg(16, 9)
    ids, w = B.router_select(z.cuda(), cfg, b.cuda())
    want, ow = oselect.forward(f64(z), 9, "sigmoid", f64(b))
    assert np.array_equal(ids.cpu().numpy(), want)
    close(w, ow, share_tolerance(z, 9) * ow)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_select_bwd_bad_and_repeated_ids(B, score, renorm):
    g = torch.Generator().manual_seed(9)
    z, gr = torch.randn((5, 20), generator=g), torch.randn((5, 4), generator=g)
    ids = torch.tensor([[0, 1, 2, 3], [4, 4, 4, 4], [-1, 5, 5, 20], [-1, -1, 1 << 40, -(1 << 40)], [19, 0, 19, 7]])
    cfg = B.make_select_cfg(20, 4, score=score, renormalise=renorm, scale=1.5)
    grad = B.router_select_bwd(z.cuda(), cfg, ids.cuda(), gr.cuda())
    want = oselect.backward(f64(z), ids.numpy(), f64(gr), score, renorm, 1.5)
    tol = 3 * share_tolerance(z, 4) * 2 * 1.5 * np.abs(f64(gr)).sum(1, keepdims=True)
    close(grad, want, tol + half_step(want, torch.float32))


def test_select_empty_batch_clears_the_counts(B):
    cfg = B.make_select_cfg(16, 2)
    counts = torch.full((16,), 9, dtype=torch.int32, device="cuda")
    z = torch.zeros((0, 16), device="cuda")
    ids, w = B.router_select(z, cfg, counts=counts)
    assert ids.shape == (0, 2) and w.shape == (0, 2) and not counts.any()
    assert B.router_select_bwd(z, cfg, ids, w).shape == (0, 16)


# ---------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,width,pad", [(1, 1, 0), (3, 7, 0), (2, 31, 1), (5, 32, 0), (4, 33, 3), (3, 40, 0),
                                            (7, 256, 8), (2, 1000, 0), (3, 264, 5), (9, 8, 0), (1, 2817, 7)])
def test_ckpt8_codes_and_values(B, fmt, dtype, rows, width, pad):
    g = torch.Generator().manual_seed(rows * 1000 + width)
    x = torch.randn((rows, width), generator=g) * torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g).float())
    x[torch.rand((rows, width), generator=g) < 0.02] *= 50
    x = x.to(DTYPES[dtype])
    ck = B.ckpt8_save(pitched(x, pad), fmt)
    codes, scales = ockpt.save(f64(x), fmt)
    assert np.array_equal(ck.scales.cpu().numpy(), scales)
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    for out in (torch.float32, DTYPES[dtype]):
        y = B.ckpt8_load(ck, out)
        want = ockpt.load(codes, scales, fmt, torch.finfo(out).max)
        # a code has at most 7 significant bits: exact unless it falls among fp16's subnormals
        close(y, want, half_step(want, out) if out == torch.float16 else 0.0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("width", [64, 37])
def test_ckpt8_borders(B, fmt, dtype, width):
    """Largest magnitudes at and beside the borders of the exponent, the type's largest and smallest
    numbers, zeros, halfway codes, infinities and NaN."""
    dt = DTYPES[dtype]
    info = torch.finfo(dt)
    tops = [448.0, 449.0, 127.5, 127.0, 127.49, 255.0, 256.0, 1.75, 1.7500001, 1.9921875, 1.992, 1.0, info.max, info.tiny,
            info.smallest_normal * info.eps, 2.0 ** -14, 0.0, 300.0]
    rows = []
    for top in tops:
        r = torch.linspace(-1, 1, width, dtype=torch.double) * top
        rows.append(r)
    x = torch.stack(rows).to(dt)
    extra = torch.arange(width, dtype=torch.double).remainder(17) * 0.5 - 4.25  # halves between int8 codes at top 64..127
    extra[0] = 100.0
    bad = torch.linspace(-2, 2, width, dtype=torch.double)
    bad[3], bad[9], bad[20] = np.inf, -np.inf, np.nan
    allbad = torch.full((width,), np.nan, dtype=torch.double)
    x = torch.cat([x, torch.stack([extra, bad, allbad]).to(dt)])
    ck = B.ckpt8_save(x.cuda(), fmt)
    codes, scales = ockpt.save(f64(x), fmt)
    assert np.array_equal(ck.scales.cpu().numpy(), scales)
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    y = f64(B.ckpt8_load(ck, dt))
    want = ockpt.load(codes, scales, fmt, info.max)
    finite = np.isfinite(f64(x))
    assert np.isfinite(y[finite]).all() and np.isnan(y[~finite]).all()
    assert np.all(np.abs(y - want)[finite] <= half_step(want, torch.float16)[finite] * (dtype == "fp16"))


def test_ckpt8_past_32_bit_offsets(B):
    """More than 2^32 bytes of input and 2^31 codes: the last rows are coded from their own values."""
    rows, width = 8200, 1 << 18
    x = torch.zeros((rows, width), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((2, width), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[-2:] = tail.cuda()
    ck = B.ckpt8_save(x, "e4m3")
    small = B.ckpt8_save(tail.cuda(), "e4m3")
    assert torch.equal(ck.codes[-2:], small.codes) and torch.equal(ck.scales[-2:], small.scales)
    assert not ck.codes[:-2].any()
    del x
    y = B.ckpt8_load(ck, torch.bfloat16)
    assert torch.equal(y[-2:], B.ckpt8_load(small, torch.bfloat16)) and not y[:-2].any()


# ----------------------------------------------------------------------- norm

NORM = [
    # rows, width, kind, dtype, wdtype, weight, bias, pad
    (1, 7168, "rms", "bf16", "bf16", True, False, 0),
    (5, 7168, "rms", "bf16", "fp32", True, True, 0),
    (3, 16384, "layer", "bf16", "bf16", True, True, 0),
    (3, 16383, "layer", "fp32", "fp32", True, True, 0),
    (301, 704, "layer", "fp32", "fp32", True, True, 64),
    (37, 2816, "layer", "bf16", "bf16", True, True, 0),
    (37, 2817, "rms", "fp16", "fp32", True, False, 7),
    (700, 256, "rms", "fp16", "fp16", True, False, 0),
    (9, 1024, "layer", "bf16", "fp32", True, True, 8),
    (9, 1032, "layer", "bf16", "fp32", True, True, 0),
    (11, 257, "layer", "bf16", "bf16", True, True, 3),
    (13, 64, "rms", "fp32", "fp32", True, True, 0),
    (1000, 8, "layer", "fp32", "fp32", True, True, 0),
    (4, 1, "rms", "fp32", "fp32", True, True, 0),
    (6, 3, "layer", "fp16", "fp32", True, True, 2),
    (5, 512, "layer", "fp32", "fp32", False, False, 0),
    (5, 512, "rms", "bf16", "fp32", False, True, 0),
    (2000, 4096, "rms", "bf16", "bf16", True, True, 0),
    (450, 8192, "layer", "fp16", "fp16", True, True, 0),
    (300, 512, "layer", "fp32", "bf16", True, True, 0),
    (33, 96, "rms", "bf16", "fp16", True, True, 8),
    (700, 400, "rms", "bf16", "fp32", True, False, 0),
    (12, 12288, "layer", "bf16", "bf16", True, True, 0),
    (12, 12288, "rms", "fp32", "fp32", True, False, 0),
]


def norm_case(case):
    rows, width, kind, dtype, wdtype, has_w, has_b, pad = case
    g = torch.Generator().manual_seed(rows + 7 * width)
    x = (torch.randn((rows, width), generator=g) * torch.exp(0.5 * torch.randn(width, generator=g)) + 0.2).to(DTYPES[dtype])
    gy = (torch.randn((rows, width), generator=g) * 0.1).to(DTYPES[dtype])
    w = (1 + 0.1 * torch.randn(width, generator=g)).to(DTYPES[wdtype]) if has_w else None
    b = (0.1 * torch.randn(width, generator=g)).to(DTYPES[wdtype]) if has_b else None
    return x, gy, w, b


def check_norm(case, x64, gy, w, b, y, mean, rstd, dx, dw, db):
    """Tolerances without the results' own rounding. A sum over a row is at most 32 serial terms a thread
    and 10 levels of a tree: 48 u of the sum of magnitudes, and u each for scaling and the like: c = 64 u.
    mean: c mean|x|. xh: that over the deviation, c (|xh| + rstd mean|x|), with rstd's own error. The
    gradient's two sums run over terms with these errors. dw and db: `rows` terms added one by one at most."""
    rows, width, kind, dtype, wdtype, has_w, has_b, pad = case
    w64 = np.ones(width) if w is None else f64(w)
    oy, omean, orstd = onorm.forward(x64, w64, None if b is None else f64(b), kind, 1e-6)
    c = 64 * U
    absx = np.abs(x64).mean(1, keepdims=True)
    off = orstd[:, None] * absx if kind == "layer" else 0.0 * orstd[:, None]
    xh = (x64 - omean[:, None]) * orstd[:, None]
    # rstd: relative c for its own sum, and the mean's error against the spread
    close(rstd, orstd, orstd * c * (1 + (off[:, 0] if kind == "layer" else 0)) + 0.0, "rstd")
    if kind == "layer":
        close(mean, omean, c * absx[:, 0], "mean")
    exh = 2 * c * (np.abs(xh) * (1 + off) + off)
    close(y, oy, exh * np.abs(w64) + 4 * U * (np.abs(oy) + (0 if b is None else np.abs(f64(b)))) + half_step(oy, y.dtype), "y")
    if dx is None:
        return
    g64 = f64(gy)
    odx, odw, odb = onorm.backward(g64, x64, omean, orstd, w64, kind)
    wg = np.abs(g64 * w64)
    m2 = (wg * np.abs(xh)).mean(1, keepdims=True)
    tol = orstd[:, None] * (c * (wg + wg.mean(1, keepdims=True) + 2 * np.abs(xh) * m2) + exh * m2
                            + np.abs(xh) * (wg * exh).mean(1, keepdims=True)) + c * (1 + off) * np.abs(odx)
    close(dx, odx, tol + half_step(odx, dx.dtype), "dx")
    terms = (rows + 128) * U
    if dw is not None:
        close(dw, odw, (np.abs(g64) * (terms * np.abs(xh) + exh)).sum(0) + half_step(odw, dw.dtype), "dw")
    if db is not None:
        close(db, odb, terms * np.abs(g64).sum(0) + half_step(odb, db.dtype), "db")


@pytest.mark.parametrize("case", NORM, ids=[f"{c[0]}x{c[1]}-{c[2]}-{c[3]}-{c[4]}" for c in NORM])
def test_norm_forward_and_backward(B, case):
    rows, width, kind, dtype, wdtype, has_w, has_b, pad = case
    x, gy, w, b = norm_case(case)
    xc, gc = pitched(x, pad), pitched(gy, pad)
    wc, bc = (None if t is None else t.cuda() for t in (w, b))
    y, mean, rstd, ck = B.norm_fwd(xc, wc, bc, kind=kind)
    assert ck is None and (mean is None) == (kind == "rms")
    dx, dw, db = B.norm_bwd(gc, xc, rstd, wc, mean=mean, kind=kind, bias_grad=has_b)
    assert (dw is None) == (w is None) and (db is None) == (not has_b)
    check_norm(case, f64(x), gy, w, b, y, mean, rstd, dx, dw, db)
    again = B.norm_bwd(gc, xc, rstd, wc, mean=mean, kind=kind, bias_grad=has_b)
    for a, c in zip((dx, dw, db), again):
        assert (a is None and c is None) or torch.equal(a, c)  # the order of the sums is fixed


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("case", [NORM[i] for i in (0, 1, 3, 4, 5, 6, 7, 10, 13, 14, 17, 20, 21, 22)],
                         ids=lambda c: f"{c[0]}x{c[1]}-{c[2]}-{c[3]}")
def test_norm_from_a_checkpoint(B, case, fmt):
    """Saving in the forward's pass writes the codes of ckpt8_save; the recomputed forward and the
    backward from the checkpoint are those of its values."""
    rows, width, kind, dtype, wdtype, has_w, has_b, pad = case
    x, gy, w, b = norm_case(case)
    xc, gc = pitched(x, pad), pitched(gy, pad)
    wc, bc = (None if t is None else t.cuda() for t in (w, b))
    plain = B.norm_fwd(xc, wc, bc, kind=kind)
    y, mean, rstd, ck = B.norm_fwd(xc, wc, bc, kind=kind, save=fmt)
    assert torch.equal(y, plain[0]) and torch.equal(rstd, plain[2])
    ref = B.ckpt8_save(xc, fmt)
    assert torch.equal(ck.codes, ref.codes) and torch.equal(ck.scales, ref.scales) and ck.format == fmt
    held = ockpt.load(ck.codes.cpu().numpy(), ck.scales.cpu().numpy(), fmt)
    y2, mean2, rstd2, none = B.norm_fwd(ck, wc, bc, kind=kind, dtype=DTYPES[dtype])
    assert none is None
    dx, dw, db = B.norm_bwd(gc, ck, rstd2, wc, mean=mean2, kind=kind, bias_grad=has_b)
    check_norm(case, held, gy, w, b, y2, mean2, rstd2, dx, dw, db)


def test_norm_gradient_against_differences(B):
    """L = sum(g y) of the device at x + d and x - d. d = 2^-5; L's third derivative in one entry is at
    most 15 rstd^3 |g w| sqrt(width)-ish: bounded here by 64 sum|g w| / width^0.5 over d^2 / 6; the
    results' roundings come in over 2 d."""
    g = torch.Generator().manual_seed(8)
    x = torch.randn((1, 96), generator=g)
    gy, w = torch.randn((1, 96), generator=g), 1 + 0.1 * torch.randn(96, generator=g)
    for kind in ("layer", "rms"):
        y, mean, rstd, _ = B.norm_fwd(x.cuda(), w.cuda(), kind=kind)
        dx, _, _ = B.norm_bwd(gy.cuda(), x.cuda(), rstd, w.cuda(), mean=mean, kind=kind)
        total = (gy * w).abs().sum().item()
        d = 2.0 ** -5
        for j in (0, 1, 50, 95):
            hi, lo = x.clone(), x.clone()
            hi[0, j] += d
            lo[0, j] -= d
            f = [(B.norm_fwd(v.cuda(), w.cuda(), kind=kind)[0].double().cpu() * gy.double()).sum().item() for v in (hi, lo)]
            num = (f[0] - f[1]) / (2 * d)
            assert abs(num - dx[0, j].item()) <= 64 * total / 96 ** 0.5 * d * d / 6 + 16 * U * total / d


def test_norm_accumulates_into_buffers(B):
    case = (50, 704, "layer", "bf16", "bf16", True, True, 0)
    x, gy, w, b = norm_case(case)
    y, mean, rstd, _ = B.norm_fwd(x.cuda(), w.cuda(), b.cuda(), kind="layer")
    run = lambda **kw: B.norm_bwd(gy.cuda(), x.cuda(), rstd, w.float().cuda(), mean=mean, kind="layer", bias_grad=True, **kw)
    _, dw, db = run()
    gw, gb = torch.full_like(dw, 3.0), torch.full_like(db, -2.0)
    _, gw2, gb2 = run(grad_weight=gw, grad_bias=gb, accumulate=True)
    assert gw2 is gw and gb2 is gb
    # one fp32 addition more, in another place of the sum
    n = 50 + 296
    assert (gw - (dw + 3)).abs().max() <= n * U * (3 + (gy.float().abs().sum(0).max() * 8).item())
    assert (gb - (db - 2)).abs().max() <= n * U * (2 + gy.float().abs().sum(0).max().item())
    with pytest.raises(ValueError, match="accumulate"):
        run(accumulate=True)


def test_norm_without_rows(B):
    w = torch.ones(64, device="cuda")
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    y, mean, rstd, ck = B.norm_fwd(x, w, w, kind="layer", save="int8")
    assert y.shape == (0, 64) and ck.codes.shape == (0, 64) and ck.scales.shape == (0, 2)
    gw = torch.full((64,), 4.0, device="cuda")
    dx, dw, db = B.norm_bwd(x, x, rstd, w, mean=mean, kind="layer", bias_grad=True)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    _, dw, _ = B.norm_bwd(x, x, rstd, w, mean=mean, kind="layer", bias_grad=True, grad_weight=gw,
                          grad_bias=torch.zeros_like(gw), accumulate=True)
    assert (dw == 4).all()
    B.norm_bwd(x, ck, rstd, w, mean=mean, kind="layer")


def test_norm_bad_rows_stay_alone(B):
    """A row with an infinity or NaN gives NaN in its own row only; a row of zeros is finite."""
    x = torch.randn((6, 512), generator=torch.Generator().manual_seed(2))
    x[1, 7], x[3, 500], x[4] = np.inf, np.nan, 0.0
    clean = x.clone()
    clean[1, 7] = clean[3, 500] = 0.0
    for kind in ("layer", "rms"):
        y = B.norm_fwd(x.cuda(), kind=kind)[0]
        ref = B.norm_fwd(clean.cuda(), kind=kind)[0]
        for r in (0, 2, 4, 5):
            assert torch.equal(y[r], ref[r])
        assert torch.isnan(y[3]).all() and torch.isnan(y[1]).any()
        assert not y[4].any()


def test_norm_past_32_bit_offsets(B):
    """Rows 2^32 bytes into a buffer, and results past 2^31 elements."""
    pitch = 1 << 17
    rows = 16400
    buf = torch.empty((rows, pitch), dtype=torch.bfloat16, device="cuda")
    x = buf[:, :256]
    x.copy_(torch.randn((rows, 256), generator=torch.Generator().manual_seed(4)))
    y, _, rstd, ck = B.norm_fwd(x, save="e4m3")
    dense = x.contiguous()
    y2, _, rstd2, ck2 = B.norm_fwd(dense, save="e4m3")
    assert torch.equal(y, y2) and torch.equal(ck.codes, ck2.codes)
    w = torch.ones(256, device="cuda")
    a = B.norm_bwd(x, x, rstd, w)
    b = B.norm_bwd(dense, dense, rstd, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ----------------------------------------------------- streams, graphs, overlap

def _pass(B, z, cfg, bias, gr, x, w, gy):
    counts = torch.empty(128, dtype=torch.int32, device="cuda")
    ids, wt = B.router_select(z, cfg, bias, counts=counts)
    gz = B.router_select_bwd(z, cfg, ids, gr)
    y, mean, rstd, ck = B.norm_fwd(x, w, save="int8")
    dx, dw, _ = B.norm_bwd(gy, ck, rstd, w)
    return ids, wt, gz, y, ck.codes, dx, dw, B.ckpt8_load(ck), counts


def _operands(seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((300, 128), generator=g).cuda(), torch.randn(128, generator=g).cuda(),
            torch.randn((300, 8), generator=g).cuda(), torch.randn((300, 704), generator=g).to(torch.bfloat16).cuda(),
            torch.ones(704, device="cuda"), torch.randn((300, 704), generator=g).to(torch.bfloat16).cuda())


def test_two_graphs_replayed_at_once(B):
    """Two captured passes, each with its own scratch, replayed on two streams at the same time, with
    inputs changed in place between replays."""
    cfg = B.make_select_cfg(128, 8, groups=8, groups_kept=4, group_top=2)
    sets = [_operands(i) for i in range(2)]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for z, bias, gr, x, w, gy in sets:
        _pass(B, z, cfg, bias, gr, x, w, gy)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_pass(B, z, cfg, bias, gr, x, w, gy))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(3):
        fresh = [_operands(10 * turn + i) for i in range(2)]
        for mine, new in zip(sets, fresh):
            for a, b in zip(mine, new):
                a.copy_(b)
        torch.cuda.synchronize()
        for _ in range(4):
            for s, graph in zip(streams, graphs):
                with torch.cuda.stream(s):
                    graph.replay()
        torch.cuda.synchronize()
        for (z, bias, gr, x, w, gy), got in zip(fresh, outs):
            for a, b in zip(got, _pass(B, z, cfg, bias, gr, x, w, gy)):
                assert torch.equal(a, b)


def test_capture_behind_copies_fills_and_other_streams(B):
    """The kernels start early behind one another; behind a copy, a fill, a host-pinned upload or a join with
    another stream in the same capture they wait like any kernel."""
    cfg = B.make_select_cfg(128, 8)
    z, bias, gr, x, w, gy = _operands(21)
    pinned = x.cpu().pin_memory()
    z2, x2, x3 = torch.empty_like(z), torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z2.copy_(z)
        ids, wt = B.router_select(z2, cfg, bias)
        x3.zero_()
        x3.copy_(pinned, non_blocking=True)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            x2.copy_(x)
            ck = B.ckpt8_save(x2, "e4m3")
        y, _, rstd, _ = B.norm_fwd(x3, w)
        torch.cuda.current_stream().wait_stream(side)
        dx, dw, _ = B.norm_bwd(gy, ck, rstd, w)
        back = B.ckpt8_load(ck)
    for seed in (22, 23):
        fresh = _operands(seed)
        for a, b in zip((z, bias, gr, x, w, gy), fresh):
            a.copy_(b)
        pinned.copy_(fresh[3])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want_ck = B.ckpt8_save(x, "e4m3")
        want_y, _, want_rstd, _ = B.norm_fwd(x, w)
        want_ids, want_wt = B.router_select(z, cfg, bias)
        want_dx, want_dw, _ = B.norm_bwd(gy, want_ck, want_rstd, w)
        for a, b in ((ids, want_ids), (wt, want_wt), (y, want_y), (ck.codes, want_ck.codes), (dx, want_dx), (dw, want_dw),
                     (back, B.ckpt8_load(want_ck))):
            assert torch.equal(a, b)


def test_a_stream_of_ones_own(B):
    """The same pass on a side stream, given by object, by handle, or made current."""
    cfg = B.make_select_cfg(128, 8)
    z, bias, gr, x, w, gy = _operands(3)
    want = _pass(B, z, cfg, bias, gr, x, w, gy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        ids, wt = B.router_select(z, cfg, bias, stream=stream)
        gz = B.router_select_bwd(z, cfg, ids, gr, stream=stream)
        y, _, rstd, ck = B.norm_fwd(x, w, save="int8", stream=stream)
        dx, dw, _ = B.norm_bwd(gy, ck, rstd, w, stream=stream)
        back = B.ckpt8_load(ck, stream=stream)
        again = B.ckpt8_save(x, "int8", stream=stream)
        s.synchronize()
        for a, b in zip((ids, wt, gz, y, ck.codes, dx, dw, back), want):
            assert torch.equal(a, b)
        assert torch.equal(again.codes, ck.codes)
    with torch.cuda.stream(s):
        got = _pass(B, z, cfg, bias, gr, x, w, gy)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()  # captured on a stream that the calls name as well
    with torch.cuda.graph(graph, stream=s):
        held = B.norm_bwd(gy, B.ckpt8_save(x, "int8", stream=s), rstd, w, stream=s)[0]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, want[5])
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_outputs_stop_at_their_ends(B):
    """Codes, scales, rows and statistics written through the C entry into the middle of a filled buffer
    leave both sides of it as they were."""
    lib = B.library()
    for rows, width, kind in ((5, 77, 1), (5, 80, 0), (3, 2816, 1), (70, 24, 0)):
        x = torch.randn((rows, width), generator=torch.Generator().manual_seed(width)).cuda()
        n = -(-width // 32)
        sizes = {"y": rows * width * 4, "rstd": rows * 4, "mean": rows * 4, "codes": rows * width, "scales": rows * n,
                 "gx": rows * width * 4, "gw": width * 4, "gb": width * 4}
        bufs = {k: torch.full((v + 512,), GUARD, dtype=torch.uint8, device="cuda") for k, v in sizes.items()}
        p = {k: b.data_ptr() + 256 for k, b in bufs.items()}
        cfg = B.NormCfg(rows, width, kind, 0, 0, 1e-6)
        mean = None if kind == 1 else p["mean"]
        st = torch.cuda.current_stream().cuda_stream
        w = torch.ones(width, device="cuda")
        assert lib.rawint4_norm_fwd(cfg, x.data_ptr(), width, None, w.data_ptr(), None, p["y"], mean, p["rstd"], 1,
                                    p["codes"], p["scales"], st) == B.OK
        ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
        assert lib.rawint4_norm_bwd(cfg, x.data_ptr(), width, None, x.data_ptr(), width, w.data_ptr(), mean, p["rstd"],
                                    p["gx"], p["gw"], p["gb"], 0, ws.data_ptr(), ws.numel(), st) == B.OK
        torch.cuda.synchronize()
        for k, b in bufs.items():
            if k == "mean" and mean is None:
                assert (b == GUARD).all()
                continue
            assert (b[:256] == GUARD).all() and (b[256 + sizes[k]:] == GUARD).all(), k
