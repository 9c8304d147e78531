"""The extension that shortens the calls around the layer is a convenience: the package imports and every
call works without it, or beside one made for another torch or Python, and it is built by itself."""

import os
import shutil
import subprocess
import sys
from pathlib import Path

import pytest
import torch

PACKAGE = Path(__file__).resolve().parents[1] / "int4_quantised_moe_b200"

USE = """
import sys, torch, warnings
sys.path.insert(0, {root!r})
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    from int4_quantised_moe_b200 import binding as B, block, dp, ep
assert B.__file__.startswith({root!r})
assert B.Layer and B.rawint4_moe_lora_workspace_size(B.make_cfg(8, 2, 256, 128, 8, 16.0, 0.0, 64)) > 0
for call in (lambda: B.router_select(torch.zeros(2, 8), B.make_select_cfg(8, 2)), lambda: B.norm_fwd(torch.zeros(2, 8)),
             lambda: B.ckpt8_save(torch.zeros(2, 8))):
    try:
        call()
    except ValueError as e:
        assert "CUDA tensor" in str(e)
    else:
        raise AssertionError("not refused")
print("ctypes" if any("ctypes" in str(w.message) for w in seen) else "quick")
"""


@pytest.fixture
def copied(tmp_path):
    """A copy of the package with the library and without an extension."""
    from int4_quantised_moe_b200 import build as b
    b.build()
    to = tmp_path / "int4_quantised_moe_b200"
    to.mkdir()
    for f in PACKAGE.glob("*.py"):
        shutil.copy(f, to)
    os.symlink(PACKAGE / "librawint4_moe.so", to / "librawint4_moe.so")
    return to


def use(copied):
    run = subprocess.run([sys.executable, "-c", USE.format(root=str(copied.parent))], capture_output=True, text=True)
    assert run.returncode == 0, run.stderr[-2000:]
    return run.stdout.strip()


def test_import_without_the_extension(copied):
    assert use(copied) == "ctypes"


def test_import_beside_an_extension_that_does_not_load(copied):
    (copied / "_fastcall.so").write_bytes(b"of another torch")
    assert use(copied) == "ctypes"
    from int4_quantised_moe_b200 import build as b
    (copied / os.path.basename(b.fastcall_path())).write_bytes(b"broken")
    assert use(copied) == "ctypes"


def test_import_with_the_extension(copied):
    from int4_quantised_moe_b200 import build as b
    shutil.copy(b.fastcall_path(), copied)
    assert use(copied) == "quick"


@pytest.fixture
def recorded(copied, monkeypatch):
    """The build of a copy, its commands recorded instead of run (their outputs are made empty)."""
    from int4_quantised_moe_b200 import build as b
    csrc = copied / "csrc"
    csrc.mkdir()
    (copied.parent / "include").mkdir()
    for name in [*b.SOURCES, *b.HEADERS, "fastcall.cpp"]:
        (csrc / name).write_text("")
    (copied.parent / "include" / "rawint4_moe.h").write_text("")
    (copied / "librawint4_moe.so").unlink()
    for name, value in (("HERE", copied), ("ROOT", copied.parent), ("CSRC", csrc), ("LIB", copied / "librawint4_moe.so"),
                        ("FASTCALL_SOURCE", csrc / "fastcall.cpp")):
        monkeypatch.setattr(b, name, str(value))
    ran = []

    def run(cmd, check):
        ran.append(os.path.basename(cmd[0]))
        Path(cmd[cmd.index("-o") + 1]).write_bytes(b"")

    monkeypatch.setattr(b.subprocess, "run", run)

    def build():
        ran.clear()
        b.build()
        return set(ran)

    return b, build


def test_each_is_built_when_its_own_sources_change(recorded):
    b, build = recorded
    assert build() == {"nvcc", "g++"}
    assert build() == set()
    header = os.path.join(b.ROOT, "include", "rawint4_moe.h")
    for source, tools in ((b.FASTCALL_SOURCE, {"g++"}), (os.path.join(b.CSRC, "norm.cu"), {"nvcc"}),
                          (os.path.join(b.CSRC, "rows.cuh"), {"nvcc"}), (header, {"nvcc", "g++"})):
        built = os.path.getmtime(b.LIB)
        os.utime(source, (built + 100, built + 100))
        assert build() == tools, source
        os.utime(source, (0, 0))


def test_another_torch_gets_an_extension_of_its_own(recorded, monkeypatch):
    b, build = recorded
    build()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert build() == {"g++"}
    assert build() == set()


def test_no_host_compiler_leaves_the_library(recorded, monkeypatch):
    b, build = recorded
    ran = b.subprocess.run

    def run(cmd, check):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        ran(cmd, check)

    monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert build() == {"nvcc"}
    assert os.path.exists(b.LIB)


@pytest.mark.gpu
def test_calls_through_ctypes_agree_with_the_extension(monkeypatch):
    """Every operator with the extension and without it, bit for bit; and the extension is there."""
    from int4_quantised_moe_b200 import binding as B
    from tests.test_gpu_around import _operands, _pass
    assert B._fast is not B._NoFastcall
    cfg = B.make_select_cfg(128, 8, groups=8, groups_kept=4, group_top=2)
    operands = _operands(31)
    want = _pass(B, operands[0], cfg, *operands[1:])
    monkeypatch.setattr(B, "_fast", B._NoFastcall)
    for a, b in zip(_pass(B, operands[0], cfg, *operands[1:]), want):
        assert torch.equal(a, b)
    gw = torch.zeros(704, device="cuda")
    w, x, gy = operands[4], operands[3], operands[5]
    y, mean, rstd, _ = B.norm_fwd(x, w, w, kind="layer")
    dx, dw, db = B.norm_bwd(gy, x, rstd, w, mean=mean, kind="layer", bias_grad=True, grad_weight=gw, grad_bias=gw.clone(),
                            accumulate=True)
    monkeypatch.undo()
    y2, mean2, rstd2, _ = B.norm_fwd(x, w, w, kind="layer")
    dx2, dw2, db2 = B.norm_bwd(gy, x, rstd2, w, mean=mean2, kind="layer", bias_grad=True)
    for a, b in ((y, y2), (mean, mean2), (rstd, rstd2), (dx, dx2), (dw, dw2), (db, db2)):
        assert torch.equal(a, b)
