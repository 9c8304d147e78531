"""The operators around the layer run together, as a block uses them: norm, the caller's projection,
expert selection, layer and their backward, with the input kept in 8 bits or as it is.

Each step is compared with its float64 oracle on the device's own inputs to that step (the layer's
tolerances are those of its parity tests; the other steps' outputs are fp32 or bf16, so relative L2 of
2^-8, bf16's half step, bounds them with room)."""

import numpy as np
import pytest
import torch

from oracle import metrics, moe as omoe
from oracle import ckpt8 as ockpt
from oracle import norm as onorm
from oracle import select as oselect
from tests._gpu import TOL_DX, TOL_LORA, TOL_OUT, TOL_ROUTE, grad_buffers, make_layer
from tests._util import f64, oracle_layer
from workloads import LORA_NAMES, make_workload, small_config

HALF = 2.0 ** -8


def near(name, got, want, tol):
    rel, cos = metrics.relative_l2_and_cosine(f64(got), want)
    assert rel <= tol[0] and cos >= tol[1], (name, rel, cos)


class StubLayer:
    def forward(self, ids, weights, h, save_for_backward=True):
        raise AssertionError("not reached")


def test_calls_out_of_order_are_refused():
    from int4_quantised_moe_b200 import binding as B
    from int4_quantised_moe_b200.block import RoutedBlock
    block = RoutedBlock(StubLayer(), B.make_select_cfg(4, 2))
    for call in (lambda: block.forward(None, None), lambda: block.backward(None, {}), lambda: block.finish(None)):
        with pytest.raises(RuntimeError, match="normalise comes next"):
            call()
    with pytest.raises(ValueError, match="keep"):
        RoutedBlock(StubLayer(), B.make_select_cfg(4, 2), keep="e5m2")
    with pytest.raises(ValueError, match="kind"):
        RoutedBlock(StubLayer(), B.make_select_cfg(4, 2), kind="group")


@pytest.mark.gpu
@pytest.mark.parametrize("keep", ["e4m3", "int8", None])
@pytest.mark.parametrize("kind,bias", [("rms", False), ("layer", True)])
def test_block_training_pass(keep, kind, bias):
    from int4_quantised_moe_b200 import binding as B
    from int4_quantised_moe_b200.block import RoutedBlock
    cfg = small_config("block", experts=8, top_k=2, hidden=256, inter=128, rank=8, qlen=67)
    wl = make_workload(cfg)
    dev = wl.to("cuda")
    g = torch.Generator().manual_seed(17)
    H, E = cfg.hidden, cfg.experts
    nw = (1 + 0.1 * torch.randn(H, generator=g)).to(torch.bfloat16)
    nb = (0.1 * torch.randn(H, generator=g)).to(torch.bfloat16) if bias else None
    rb = 0.05 * torch.randn(E, generator=g)
    proj = (torch.randn((E, H), generator=g) / H ** 0.5)
    select = B.make_select_cfg(E, cfg.top_k, groups=4, groups_kept=2, group_top=2, scale=2.5)
    layer = make_layer(dev)
    block = RoutedBlock(layer, select, nw.cuda(), None if nb is None else nb.cuda(), kind=kind, route_bias=rb.cuda(), keep=keep)
    pc = proj.cuda()
    x = dev.x

    for turn in range(2):  # the second pass starts from what the first left
        h = block.normalise(x)
        oh, mean, rstd = onorm.forward(f64(wl.x), f64(nw), None if nb is None else f64(nb), kind, 1e-6)
        near("h", h, oh, (HALF, 0.9999))
        scores = h.float() @ pc.t()
        counts = torch.empty(E, dtype=torch.int32, device="cuda")
        out = block.forward(h, scores, counts=counts)
        ids, w = oselect.forward(f64(scores), cfg.top_k, "sigmoid", f64(rb), 4, 2, 2, True, 2.5)
        assert np.array_equal(counts.cpu().numpy(), np.bincount(ids.reshape(-1), minlength=E))
        ol = oracle_layer(wl)
        oout, _ = omoe.forward(ol, f64(h), ids, w)
        near("out", out, oout, TOL_OUT)

        grads = grad_buffers(wl)
        grad_h, grad_scores = block.backward(dev.grad_out, grads)
        # what the backward works from: the kept input, normed again
        if keep is None:
            kept, h2 = f64(wl.x), f64(h)
        else:
            kept = ockpt.load(*ockpt.save(f64(wl.x), keep), keep)
            kh, mean, rstd = onorm.forward(kept, f64(nw), None if nb is None else f64(nb), kind, 1e-6)
            h2 = f64(B.norm_fwd(B.ckpt8_save(x, keep), nw.cuda(), None if nb is None else nb.cuda(), kind=kind)[0])
            near("h again", torch.from_numpy(h2), kh, (HALF, 0.9999))
        _, ctx = omoe.forward(ol, h2, ids, w)
        ogin, ogroute, ogr = omoe.backward(ol, ctx, f64(wl.grad_out))
        near("grad_h", grad_h, ogin, TOL_DX)
        near("grad_scores", grad_scores, oselect.backward(f64(scores), ids, ogroute, "sigmoid", True, 2.5), TOL_ROUTE)
        for n in LORA_NAMES:
            near(n, grads[n], ogr[n], TOL_LORA)

        total = (grad_h.float() + grad_scores @ pc).to(torch.bfloat16)
        grad_x, gw, gb = block.finish(total)
        odx, odw, odb = onorm.backward(f64(total), kept, mean, rstd, f64(nw), kind)
        near("grad_x", grad_x, odx, (HALF, 0.9999))
        near("grad_weight", gw, odw, (HALF, 0.9999))
        assert (gb is None) == (nb is None)
        if gb is not None:
            near("grad_bias", gb, odb, (HALF, 0.9999))
    assert layer.status() == 0
    # inference: nothing is kept, the next pass begins anew
    h = block.normalise(x)
    again = block.forward(h, scores, train=False)
    assert torch.equal(again, out)
    with pytest.raises(RuntimeError, match="normalise comes next"):
        block.backward(dev.grad_out, grads)


@pytest.mark.gpu
def test_block_keeps_little():
    """Between forward and backward the block holds the checkpoint, not x: 33 / 32 bytes an element."""
    from int4_quantised_moe_b200 import binding as B
    from int4_quantised_moe_b200.block import RoutedBlock
    cfg = small_config("block", experts=4, top_k=2, hidden=256, inter=128, rank=8, qlen=64)
    dev = make_workload(cfg).to("cuda")
    block = RoutedBlock(make_layer(dev), B.make_select_cfg(4, 2), torch.ones(256, dtype=torch.bfloat16, device="cuda"))
    h = block.normalise(dev.x)
    block.forward(h, torch.randn((64, 4), device="cuda"))
    assert isinstance(block._x, B.Ckpt8) and block._x.nbytes == 64 * 256 * 33 // 32
