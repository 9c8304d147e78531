"""Blocks that share a layer: without an 8-bit copy of its input a block depends on the layer's saved
context, and its backward is refused once another pass has replaced that context."""

import pytest
import torch

from int4_quantised_moe_b200 import binding as B
from int4_quantised_moe_b200 import block as block_module
from int4_quantised_moe_b200.block import RoutedBlock
from int4_quantised_moe_b200.ep import ExpertParallelLayer
from workloads import lora_shapes, make_workload, small_config


class CountingLayer:
    def __init__(self):
        self.passes = 0

    def forward(self, ids, weights, h, save_for_backward=True):
        self.passes += 1
        return h

    def backward(self, grad_out, grads, **kw):
        self.passes += 1
        return grad_out


@pytest.fixture
def plain(monkeypatch):
    """The operators around the layer replaced by ones that pass their inputs on."""
    row = torch.zeros(2)
    monkeypatch.setattr(block_module.B, "norm_fwd", lambda x, *a, **kw: (x, None, row, x if kw.get("save") else None))
    monkeypatch.setattr(block_module.B, "router_select", lambda s, *a, **kw: (torch.zeros(2, 1).long(), torch.ones(2, 1)))
    monkeypatch.setattr(block_module.B, "router_select_bwd", lambda s, *a: s)
    monkeypatch.setattr(block_module.B, "norm_bwd", lambda g, *a, **kw: (g, None, None))


def begin(block):
    x = torch.zeros(2, 4)
    return block.forward(block.normalise(x), x)


def end(block):
    g, _ = block.backward(torch.zeros(2, 4), {})
    block.finish(g)


def blocks(layer, *keeps):
    return [RoutedBlock(layer, B.make_select_cfg(4, 1), keep=keep) for keep in keeps]


def test_one_after_another(plain):
    first, second = blocks(CountingLayer(), None, None)
    for block in (first, second, first):
        begin(block)
        end(block)


@pytest.mark.parametrize("other", ["forward", "evaluation", "direct", "recomputed"])
def test_a_replaced_context_is_refused(plain, other):
    layer = CountingLayer()
    first, second = blocks(layer, None, "e4m3" if other == "recomputed" else None)
    if other == "recomputed":
        begin(second)
    begin(first)
    if other == "forward":
        begin(second)
    elif other == "evaluation":
        second.forward(second.normalise(torch.zeros(2, 4)), torch.zeros(2, 4), train=False)
    elif other == "direct":
        layer.forward(None, None, None)
    else:
        end(second)  # goes forward again first
    with pytest.raises(RuntimeError, match="saved context"):
        first.backward(torch.zeros(2, 4), {})
    begin(first)  # a pass of its own again
    end(first)


def test_blocks_that_keep_their_input_share(plain):
    first, second = blocks(CountingLayer(), "e4m3", "int8")
    begin(first)
    begin(second)
    end(first)
    end(second)


def test_a_layer_that_does_not_count(plain):
    """A wrapper with forward and backward alone works as before; nothing is checked."""
    layer = CountingLayer()

    class Wrapper:
        def forward(self, *args, **kw):
            return layer.forward(*args, **kw)

        def backward(self, *args, **kw):
            return layer.backward(*args, **kw)

    block, = blocks(Wrapper(), None)
    begin(block)
    end(block)


def test_a_refused_call_does_not_count(monkeypatch):
    """The library refuses before it touches the workspace, so the saved context is still there."""
    wl = make_workload(small_config("block", experts=2, top_k=1, hidden=64, inter=64, rank=8, qlen=3))
    monkeypatch.setattr(B, "_expect", lambda *args: None)  # host tensors; the calls are replaced
    monkeypatch.setattr(B, "make_grads", lambda grads: None)
    layer = B.Layer(B.make_cfg(2, 1, 64, 64, 8, 16.0, 0.0, 3), None, None, torch.zeros(256, dtype=torch.uint8), ())

    def refuse(*args, **kw):
        raise B.RawInt4Error(B.INVALID_ARGUMENT, "refused")

    grads = {n: torch.zeros(s, dtype=torch.bfloat16) for n, s in lora_shapes(wl.cfg).items()}
    for fwd, bwd, counted in ((refuse, refuse, 0), (lambda *a, **k: None, refuse, 1), (lambda *a, **k: None, lambda *a, **k: None, 3)):
        monkeypatch.setattr(B, "rawint4_moe_lora_fwd", fwd)
        monkeypatch.setattr(B, "rawint4_moe_lora_bwd", bwd)
        for call in (lambda: layer.forward(wl.expert_ids, wl.route_weights, wl.x), lambda: layer.backward(wl.grad_out, grads)):
            try:
                call()
            except B.RawInt4Error:
                pass
        assert layer.passes == counted


def test_expert_parallel_layers_count_too():
    class Dist:
        get_world_size = get_rank = staticmethod(lambda: 1)
    assert ExpertParallelLayer(Dist, 4, 1, None, 8, ops=object()).passes == 0


@pytest.mark.gpu
def test_shared_layer_on_the_device():
    """Two blocks, one layer: with copies of their inputs each gets the gradients that it gets alone."""
    from tests._gpu import grad_buffers, make_layer
    cfg = small_config("block", experts=8, top_k=2, hidden=256, inter=128, rank=8, qlen=67)
    wl = make_workload(cfg)
    dev = wl.to("cuda")
    g = torch.Generator().manual_seed(3)
    inputs = [dev.x, (torch.randn((67, 256), generator=g)).to(torch.bfloat16).cuda()]
    scores = [torch.randn((67, 8), generator=g).cuda() for _ in range(2)]
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    layer = make_layer(dev)
    select = B.make_select_cfg(8, 2)

    def go_back(block):
        grads = grad_buffers(wl)
        gh, gs = block.backward(dev.grad_out, grads)
        return [gh, gs, *block.finish(gh)[:2], *grads.values()]

    for keep in ("e4m3", None):
        alone = []
        for x, s in zip(inputs, scores):
            block = RoutedBlock(layer, select, w, keep=keep)
            block.forward(block.normalise(x), s)
            alone.append(go_back(block))
        both = [RoutedBlock(layer, select, w, keep=keep) for _ in range(2)]
        for block, x, s in zip(both, inputs, scores):
            block.forward(block.normalise(x), s)
        if keep is None:
            with pytest.raises(RuntimeError, match="saved context"):
                go_back(both[0])
            results = [None, go_back(both[1])]
        else:
            results = [go_back(block) for block in both]
        for got, want in zip(results, alone):
            if got is not None:
                assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert layer.status() == 0


def test_gradient_of_a_bias_without_weight_has_its_type(plain, monkeypatch):
    """norm_bwd cannot see the bias; the block asks for the gradient in its type."""
    seen = {}
    monkeypatch.setattr(block_module.B, "norm_bwd", lambda g, *a, **kw: (seen.update(kw), (g, None, kw["grad_bias"]))[1])
    bias = torch.zeros(4, dtype=torch.float16)
    block = RoutedBlock(CountingLayer(), B.make_select_cfg(4, 1), norm_bias=bias, kind="layer", keep=None)
    begin(block)
    block.backward(torch.zeros(2, 4), {})
    _, _, grad_bias = block.finish(torch.zeros(2, 4))
    assert seen["bias_grad"] and grad_bias.dtype == torch.float16 and grad_bias.shape == (4,)


@pytest.mark.gpu
def test_gradient_of_a_bias_without_weight_on_the_device():
    from tests._gpu import grad_buffers, make_layer
    cfg = small_config("block", experts=8, top_k=2, hidden=256, inter=128, rank=8, qlen=67)
    wl = make_workload(cfg)
    dev = wl.to("cuda")
    block = RoutedBlock(make_layer(dev), B.make_select_cfg(8, 2), norm_bias=torch.zeros(256, device="cuda"), kind="layer")
    block.forward(block.normalise(dev.x), torch.randn((67, 8), generator=torch.Generator().manual_seed(4)).cuda())
    gh, _ = block.backward(dev.grad_out, grad_buffers(wl))
    _, grad_weight, grad_bias = block.finish(gh)
    assert grad_weight is None and grad_bias.dtype == torch.float32
    want = gh.double().sum(0)  # 67 terms and the fold, each addition rounded in fp32
    assert ((grad_bias.double() - want).abs() <= 256 * 2.0 ** -24 * gh.double().abs().sum(0)).all()
