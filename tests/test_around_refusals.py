"""What the operators around the layer (expert selection, 8-bit checkpoints, norm) refuse, on the CPU:
every case returns on the host before any CUDA call, so the placeholder pointers are never dereferenced."""

import ctypes

import pytest
import torch

FAKE = 1 << 20  # aligned, never dereferenced
FAR = 1 << 40   # a second one, far from it
MIB = 1 << 20


@pytest.fixture(scope="module")
def B():
    from int4_quantised_moe_b200 import build as b
    b.build()
    from int4_quantised_moe_b200 import binding
    return binding


def _cfg(B, **over):
    base = dict(experts=64, top_k=4, groups=1, groups_kept=1, group_top=1, score=1, renormalise=1, type=0, scale=1.0)
    base.update(over)
    return B.SelectCfg(*[base[n] for n, _ in B.SelectCfg._fields_])


@pytest.mark.parametrize("over", [
    {"experts": 0}, {"experts": 4097}, {"top_k": 0}, {"top_k": 33}, {"top_k": 65}, {"groups": 0}, {"groups": 64},
    {"groups": 5}, {"groups": 4, "groups_kept": 0}, {"groups": 4, "groups_kept": 5}, {"groups": 4, "group_top": 3},
    {"groups": 4, "group_top": 0}, {"experts": 8, "groups": 8, "groups_kept": 8, "group_top": 2},
    {"groups": 16, "groups_kept": 1, "top_k": 5}, {"score": 2}, {"type": 3}, {"type": -1},
    {"scale": float("nan")}, {"scale": float("inf")}])
def test_select_cfg(B, over):
    lib, cfg = B.library(), _cfg(B, **over)
    rc = lib.rawint4_moe_router_select(cfg, FAKE, max(cfg.experts, 1), 2, None, FAR, FAR + MIB, None, None)
    assert rc == B.INVALID_ARGUMENT
    rc = lib.rawint4_moe_router_select_bwd(cfg, FAKE, max(cfg.experts, 1), 2, FAR, FAR + MIB, FAR + 2 * MIB, None)
    assert rc == B.INVALID_ARGUMENT


def test_select_arguments(B):
    f = B.library().rawint4_moe_router_select
    g = B.library().rawint4_moe_router_select_bwd
    ok = _cfg(B)
    bad = B.INVALID_ARGUMENT
    assert f(None, FAKE, 64, 2, None, FAR, FAR + MIB, None, None) == bad
    assert f(ok, None, 64, 2, None, FAR, FAR + MIB, None, None) == bad
    assert f(ok, FAKE, 63, 2, None, FAR, FAR + MIB, None, None) == bad   # pitch below the width
    assert f(ok, FAKE + 2, 64, 2, None, FAR, FAR + MIB, None, None) == bad  # fp32 off its alignment
    assert f(ok, FAKE, 64, -1, None, FAR, FAR + MIB, None, None) == bad
    assert f(ok, FAKE, 64, 2, None, None, FAR, None, None) == bad
    assert f(ok, FAKE, 64, 2, None, FAR, None, None, None) == bad
    assert f(ok, FAKE, 64, 2, FAR + 2, FAR, FAR + MIB, None, None) == bad  # bias off its alignment
    assert f(ok, FAKE, 64, 2, None, FAR + 4, FAR + MIB, None, None) == bad  # ids off theirs
    assert g(ok, FAKE, 64, 2, None, FAR, FAR + MIB, None) == bad
    assert g(ok, FAKE, 64, 2, FAR, None, FAR + MIB, None) == bad
    assert g(ok, FAKE, 64, 2, FAR, FAR + MIB, None, None) == bad
    assert g(ok, FAKE, 64, 2, FAR, FAR + MIB, FAKE + 256, None) == bad   # the gradient over the scores
    assert g(ok, FAKE, 64, 0, None, None, None, None) == B.OK            # nothing to do


def test_ckpt8_arguments(B):
    save, load = B.library().rawint4_ckpt8_save, B.library().rawint4_ckpt8_load
    bad = B.INVALID_ARGUMENT
    args = dict(format=0, type=1, x=FAKE, ldx=64, rows=4, width=64, codes=FAR, scales=FAR + MIB)
    for over in ({"format": 2}, {"type": 3}, {"x": None}, {"ldx": 63}, {"rows": -1}, {"rows": 1 << 31}, {"width": 0},
                 {"width": MIB + 1, "ldx": MIB + 1}, {"codes": None}, {"scales": None}, {"x": FAKE + 1},
                 {"codes": FAKE + 256}, {"scales": FAKE + 500}, {"scales": FAR + 255}, {"ldx": (1 << 28) + 1}):
        a = dict(args, **over)
        assert save(a["format"], a["type"], a["x"], a["ldx"], a["rows"], a["width"], a["codes"], a["scales"], None) == bad
        if "ldx" not in over and over != {"scales": FAR + 255}:  # reading codes and scales out of one buffer is fine
            assert load(a["format"], a["codes"], a["scales"], a["rows"], a["width"], a["type"], a["x"], None) == bad, over
    assert save(0, 1, None, 64, 0, 64, None, None, None) == B.OK
    assert load(0, None, None, 0, 64, 1, None, None) == B.OK


def _norm_cfg(B, **over):
    base = dict(rows=4, width=64, kind=1, type=1, weight_type=1, eps=1e-6)
    base.update(over)
    return B.NormCfg(*[base[n] for n, _ in B.NormCfg._fields_])


@pytest.mark.parametrize("over", [{"rows": -1}, {"width": 0}, {"width": 16385}, {"kind": 2}, {"type": 3},
                                  {"weight_type": -1}, {"eps": 0.0}, {"eps": -1.0}, {"eps": float("nan")},
                                  {"eps": float("inf")}])
def test_norm_cfg(B, over):
    lib, cfg = B.library(), _norm_cfg(B, **over)
    n = ctypes.c_size_t(0)
    assert lib.rawint4_norm_bwd_workspace_size(cfg, n) == B.INVALID_ARGUMENT
    assert lib.rawint4_norm_fwd(cfg, FAKE, 16385, None, None, None, FAR, None, FAR + MIB, 0, None, None,
                                None) == B.INVALID_ARGUMENT
    assert lib.rawint4_norm_bwd(cfg, FAKE, 16385, None, FAR, 16385, None, None, FAKE, FAR + MIB, None, None, 0, None, 0,
                                None) == B.INVALID_ARGUMENT


def test_norm_fwd_arguments(B):
    lib = B.library()
    good = dict(x=FAKE, ldx=64, ck=None, w=None, b=None, y=FAR, mean=None, rstd=FAR + MIB, fmt=0, codes=None, scales=None)
    ck = B.Ckpt8Ptrs(FAKE, FAKE + MIB, 0)
    for kind, over in [(1, {"x": None}), (1, {"ck": ck}), (1, {"ldx": 63}), (1, {"y": None}), (1, {"rstd": None}),
                       (1, {"mean": FAR + 2 * MIB}), (0, {}), (1, {"y": FAKE + 128}), (1, {"x": FAKE + 1}),
                       (1, {"y": FAR + 1}), (1, {"w": FAR + 1}), (1, {"b": FAR + 1}), (1, {"codes": FAR + 2 * MIB}),
                       (1, {"scales": FAR + 2 * MIB}), (1, {"rstd": FAR + MIB + 2}), (1, {"rstd": FAR + 64}),
                       (1, {"fmt": 2, "codes": FAR + 2 * MIB, "scales": FAR + 3 * MIB}),
                       (1, {"codes": FAKE + 64, "scales": FAR + 3 * MIB}),
                       (1, {"codes": FAR + 2 * MIB, "scales": FAKE + 64}),
                       (1, {"codes": FAR + 2 * MIB, "scales": FAR + 2 * MIB + 64}),
                       (1, {"codes": FAR + 64, "scales": FAR + 3 * MIB}),
                       (1, {"x": None, "ck": B.Ckpt8Ptrs(None, FAKE, 0)}), (1, {"x": None, "ck": B.Ckpt8Ptrs(FAKE, None, 0)}),
                       (1, {"x": None, "ck": B.Ckpt8Ptrs(FAKE, FAKE + MIB, 2)}),
                       (1, {"x": None, "ck": ck, "codes": FAR + 2 * MIB, "scales": FAR + 3 * MIB}),
                       (1, {"x": None, "ck": ck, "y": FAKE + MIB + 2})]:
        a = dict(good, **over)
        rc = lib.rawint4_norm_fwd(_norm_cfg(B, kind=kind), a["x"], a["ldx"], a["ck"], a["w"], a["b"], a["y"], a["mean"],
                                  a["rstd"], a["fmt"], a["codes"], a["scales"], None)
        assert rc == B.INVALID_ARGUMENT, (kind, over)
    assert lib.rawint4_norm_fwd(_norm_cfg(B, rows=0), None, 64, None, None, None, None, None, None, 0, None, None,
                                None) == B.OK


def test_norm_bwd_arguments(B):
    lib = B.library()
    n = ctypes.c_size_t(0)
    assert lib.rawint4_norm_bwd_workspace_size(_norm_cfg(B), n) == B.OK and n.value >= 2 * 64 * 4
    good = dict(x=FAKE, ldx=64, ck=None, gy=FAKE + MIB, ldg=64, w=None, mean=None, rstd=FAR, gx=FAR + MIB,
                gw=FAR + 2 * MIB, gb=FAR + 3 * MIB, ws=FAR + 4 * MIB, nbytes=n.value)
    for kind, over in [(1, {"x": None}), (1, {"ck": B.Ckpt8Ptrs(FAKE, FAKE + MIB, 0)}), (1, {"gy": None}),
                       (1, {"ldg": 63}), (1, {"rstd": None}), (0, {}), (1, {"gx": None}), (1, {"ws": None}),
                       (1, {"nbytes": n.value - 1}), (1, {"ws": FAR + 4 * MIB + 8}), (1, {"gx": FAKE + 64}),
                       (1, {"gx": FAKE + MIB + 64}), (1, {"gw": FAR + 1}), (1, {"gb": FAR + 1}), (1, {"gx": FAR + MIB + 1}),
                       (1, {"gy": FAKE + MIB + 1}), (1, {"rstd": FAR + 2}), (1, {"ws": FAR + MIB})]:
        a = dict(good, **over)
        rc = lib.rawint4_norm_bwd(_norm_cfg(B, kind=kind), a["x"], a["ldx"], a["ck"], a["gy"], a["ldg"], a["w"], a["mean"],
                                  a["rstd"], a["gx"], a["gw"], a["gb"], 0, a["ws"], a["nbytes"], None)
        assert rc == B.INVALID_ARGUMENT, (kind, over)


def test_binding_refuses_wrong_tensors(B):
    x = torch.zeros((4, 64))
    cfg = B.make_select_cfg(64, 4)
    with pytest.raises(ValueError, match="score"):
        B.make_select_cfg(64, 4, score="linear")
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.router_select(x, cfg)
    with pytest.raises(TypeError, match="dtype"):
        B.router_select(x.double(), cfg)
    with pytest.raises(ValueError, match="shape"):
        B.router_select(x[:, :63], cfg)
    with pytest.raises(TypeError, match="Tensor"):
        B.ckpt8_save([1.0], "e4m3")
    with pytest.raises(ValueError, match="format"):
        B.ckpt8_save(x, "e5m2")
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.ckpt8_save(x)
    huge = torch.zeros((1, 64)).expand(1 << 31, 64)  # a size that int32 would wrap
    for call in (lambda: B.router_select(huge, cfg), lambda: B.ckpt8_save(huge), lambda: B.norm_fwd(huge),
                 lambda: B.norm_bwd(x, huge, x[:, 0])):
        with pytest.raises(ValueError, match="above 2147483647"):
            call()
    with pytest.raises(ValueError, match="above 2147483647"):
        B.ckpt8_load(B.Ckpt8(torch.zeros((1, 64), dtype=torch.uint8).expand(1 << 31, 64), x, "int8"))
    codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.ckpt8_load(B.Ckpt8(codes, scales, "int8"))
    with pytest.raises(ValueError, match="format"):
        B.ckpt8_load(B.Ckpt8(codes, scales, "fp8"))
    with pytest.raises(ValueError, match="codes"):
        B.ckpt8_load(B.Ckpt8(codes[0], scales, "int8"))
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.norm_fwd(x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.norm_bwd(x, x, x[:, 0])
