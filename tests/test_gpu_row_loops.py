"""The loops of the kernels around the layer where a thread group takes several rows or tokens: the norm's
backward in each of its layouts, and expert selection of large batches beside that of small ones."""

import numpy as np
import pytest
import torch

from oracle import ckpt8 as ockpt
from oracle import select as oselect
from tests.test_gpu_around import (DTYPES, GUARD, U, check_norm, close, f64, half_step, norm_case, pitched, share_tolerance)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from int4_quantised_moe_b200 import binding
    return binding


# Rows a thread group, at 148 blocks: from 3 to 18, more than the ring's four stages in most.
ROWS = [
    # rows, width, kind, dtype, wdtype, weight, bias, pad
    (1500, 2817, "rms", "bf16", "bf16", True, False, 0),     # scalar, one chunk a thread
    (1500, 2817, "layer", "bf16", "bf16", True, True, 0),
    (1500, 2817, "layer", "fp32", "fp32", True, True, 3),
    (1500, 2817, "layer", "fp16", "fp32", True, False, 0),
    (1400, 3583, "rms", "fp16", "fp32", True, True, 2),
    (4500, 257, "layer", "bf16", "fp32", True, True, 0),
    (9000, 33, "rms", "fp32", "bf16", True, True, 1),
    (20000, 7, "layer", "fp32", "fp32", True, True, 0),
    (900, 5001, "layer", "bf16", "bf16", True, True, 0),     # scalar, two chunks
    (900, 5001, "rms", "fp32", "fp32", True, False, 1),
    (700, 16383, "layer", "bf16", "bf16", True, True, 0),    # scalar, four chunks
    (700, 16383, "rms", "bf16", "bf16", True, False, 0),
    (3000, 2816, "layer", "bf16", "bf16", True, True, 0),    # vector: one chunk from a checkpoint, two from a tensor
    (2500, 2816, "rms", "fp32", "fp32", True, True, 8),
    (3000, 7168, "rms", "bf16", "bf16", True, False, 0),     # vector, four chunks
    (3000, 7168, "layer", "fp16", "fp16", True, False, 8),
    (1500, 7168, "layer", "bf16", "bf16", True, True, 0),
    (700, 12288, "layer", "bf16", "bf16", True, True, 0),
    (700, 12288, "layer", "fp32", "fp32", True, True, 0),
    (9000, 256, "rms", "fp16", "fp16", True, False, 0),      # several row groups a block
    (9000, 200, "layer", "bf16", "fp32", True, True, 0),
]


@pytest.mark.parametrize("source", ["tensor", "e4m3", "int8"])
@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"{c[0]}x{c[1]}-{c[2]}-{c[3]}")
def test_norm_over_many_rows(B, case, source):
    rows, width, kind, dtype, wdtype, has_w, has_b, pad = case
    x, gy, w, b = norm_case(case)
    wc, bc = (None if t is None else t.cuda() for t in (w, b))
    given = pitched(x, pad)
    held = f64(x)
    kw = {}
    if source != "tensor":
        given = B.ckpt8_save(given, source)
        held = ockpt.load(given.codes.cpu().numpy(), given.scales.cpu().numpy(), source)
        kw["dtype"] = DTYPES[dtype]
    y, mean, rstd, _ = B.norm_fwd(given, wc, bc, kind=kind, **kw)
    dx, dw, db = B.norm_bwd(pitched(gy, pad), given, rstd, wc, mean=mean, kind=kind, bias_grad=has_b)
    check_norm(case, held, gy, w, b, y, mean, rstd, dx, dw, db)


def test_norm_results_past_2_31_elements(B):
    """The last rows of a result of more than 2^31 elements are those of the same rows by themselves. (300
    rows: fewer than 297 have other thread counts in the forward, and other orders of their sums.)"""
    width, rows, tail = 8192, (1 << 18) + 700, 300
    g = torch.Generator().manual_seed(4)
    x = torch.zeros((rows, width), dtype=torch.bfloat16, device="cuda")
    gy = torch.zeros((rows, width), dtype=torch.bfloat16, device="cuda")
    x[-tail:] = torch.randn((tail, width), generator=g).to(torch.bfloat16).cuda()
    gy[-tail:] = torch.randn((tail, width), generator=g).to(torch.bfloat16).cuda()
    w = torch.ones(width, dtype=torch.bfloat16, device="cuda")
    last, last_gy = x[-tail:].clone(), gy[-tail:].clone()
    y, _, rstd, ck = B.norm_fwd(x, w, save="e4m3")
    y2, _, rstd2, ck2 = B.norm_fwd(last, w, save="e4m3")
    assert torch.equal(y[-tail:], y2) and torch.equal(rstd[-tail:], rstd2)
    assert torch.equal(ck.codes[-tail:], ck2.codes) and torch.equal(ck.scales[-tail:], ck2.scales)
    assert not y[:-tail].any() and not ck.codes[:-tail].any()
    for given, given2 in ((x, last), (ck, ck2)):
        dx, dw, _ = B.norm_bwd(gy, given, rstd, w)
        dx2, dw2, _ = B.norm_bwd(last_gy, given2, rstd2, w)
        assert torch.equal(dx[-tail:], dx2) and not dx[:-tail].any()
        # 300 terms in two orders, each result rounded to bf16
        size = (last_gy.float().abs() * 8).sum(0)
        assert ((dw.float() - dw2.float()).abs() <= 2 * tail * U * size + dw2.float().abs() * 2.0 ** -7).all()
        del dx


# ------------------------------------------------------------------ selection

MANY = [
    # Q, E, k, score, dtype, renorm, pad
    (2047, 128, 8, "softmax", "bf16", False, 0),
    (2048, 128, 8, "softmax", "bf16", False, 0),
    (2049, 128, 8, "softmax", "bf16", False, 3),
    (2049, 128, 8, "sigmoid", "fp16", True, 0),
    (4099, 127, 7, "softmax", "fp16", True, 5),
    (4099, 64, 8, "sigmoid", "bf16", False, 8),
    (2050, 8, 8, "softmax", "bf16", True, 0),
    (2051, 9, 1, "sigmoid", "fp16", True, 0),
    (2048, 1, 1, "softmax", "fp16", False, 1),
    (9001, 72, 5, "softmax", "fp16", False, 0),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{c[0]}x{c[1]}k{c[2]}-{c[3]}-{c[4]}")
def test_large_batches_select_as_small_ones(B, case):
    """From 2048 tokens on 16-bit scores without a bias have a kernel of their own: every token beside the
    same token in a batch of 1024, and the oracle's."""
    Q, E, k, score, dtype, renorm, pad = case
    dt = DTYPES[dtype]
    g = torch.Generator().manual_seed(Q * 10 + E)
    z = torch.randn((Q, E), generator=g) * 1.5
    z[::5] = z[::5].round()  # ties
    z[1::7] = 0.25           # all of them equal
    z[torch.rand((Q, E), generator=g) < 0.02] = -np.inf
    z[3::211] = -np.inf
    z[4::211, 1:] = -np.inf
    z[7::301, 0] = float("nan")
    z[8::301, -1] = np.inf
    z[9::301] = torch.finfo(dt).min
    if E > 72:  # every slot in one lane's experts, 8 l + j and 64 + 8 l + j
        for lane in range(8):
            mine = [e for e in (*range(8 * lane, 8 * lane + 8), *range(64 + 8 * lane, 72 + 8 * lane)) if e < E]
            z[20 + lane::97] -= 40
            for r in range(20 + lane, Q, 97):
                z[r, mine] += 50
    z = z.to(dt)
    gr = torch.randn((Q, k), generator=g)
    zc, gc = pitched(z, pad), gr.cuda()
    cfg = B.make_select_cfg(E, k, score=score, renormalise=renorm, scale=1.5)
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    ids, w = B.router_select(zc, cfg, counts=counts)
    grad = B.router_select_bwd(zc, cfg, ids, gc)
    for lo in range(0, Q, 1024):
        ids2, w2 = B.router_select(zc[lo:lo + 1024], cfg)
        assert torch.equal(ids[lo:lo + 1024], ids2)
        torch.testing.assert_close(w[lo:lo + 1024], w2, rtol=64 * U, atol=0)
    pick = sorted(set(range(0, Q, 5)) | {r for s in (3, 4, 7, 8, 9) for r in range(s, Q, 211)}
                  | {r for s in range(20, 28) for r in range(s, Q, 97)} | set(range(Q - 9, Q)))
    want, ow = oselect.forward(f64(z[pick]), k, score, None, 1, 1, 1, renorm, 1.5)
    assert np.array_equal(ids.cpu().numpy()[pick], want)
    # scores differ by up to 90 and reach 60 (the type's largest numbers and infinity give exact 0 and 1)
    near = 2 * U * (150 + 4 + E / 32 + 5 + k + 8)
    close(w[pick], ow, near * ow + 2.0 ** -126, "weights")
    assert torch.equal(counts.cpu(), torch.bincount(ids.reshape(-1), minlength=E).int().cpu())
    og = oselect.backward(f64(z[pick]), want, f64(gr[pick]), score, renorm, 1.5)
    size = 3 * near * 1.5 * np.abs(f64(gr[pick])).sum(1, keepdims=True)
    close(grad[pick], og, size + half_step(og, dt), "grad_scores")


# ---------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 32), (4, 33), (2, 255), (3, 264), (2, 2817), (7, 40)])
def test_checkpoints_stop_at_their_ends(B, rows, width, dtype, fmt):
    """Codes, scales and rows written into the middle of a filled buffer leave both sides of it as they were."""
    lib, dt = B.library(), DTYPES[dtype]
    size = dt.itemsize
    x = torch.randn((rows, width), generator=torch.Generator().manual_seed(width)).to(dt).cuda()
    sizes = {"codes": rows * width, "scales": rows * -(-width // 32), "x": rows * width * size}
    st = torch.cuda.current_stream().cuda_stream
    for shift in (0, size):  # on and off the alignment of vector accesses
        bufs = {k: torch.full((v + 512 + 16,), GUARD, dtype=torch.uint8, device="cuda") for k, v in sizes.items()}
        at = {k: 256 + (shift if k != "scales" else 0) for k in sizes}
        p = {k: b.data_ptr() + at[k] for k, b in bufs.items()}
        typ = B.TYPES[dt]
        assert lib.rawint4_ckpt8_save(fmt, typ, x.data_ptr(), width, rows, width, p["codes"], p["scales"], st) == B.OK
        assert lib.rawint4_ckpt8_load(fmt, p["codes"], p["scales"], rows, width, typ, p["x"], st) == B.OK
        torch.cuda.synchronize()
        for k, b in bufs.items():
            assert (b[:at[k]] == GUARD).all() and (b[at[k] + sizes[k]:] == GUARD).all(), (k, shift)
        name = {0: "e4m3", 1: "int8"}[fmt]
        want = B.ckpt8_load(B.ckpt8_save(x, name), dt)
        got = bufs["x"][at["x"]:at["x"] + sizes["x"]].clone().view(dt).view(rows, width)
        assert torch.equal(got, want)
