"""The rules of kernels that are launched while the one before them drains, checked on the sources.

Such a kernel may be resident while its inputs are still being written. It reads memory behind its wait
only, so it may not promise the compiler that its inputs never change (`__restrict__`, `__ldg`), which
would free the loads to move in front of the wait; and a kernel that is started this way has the wait."""

import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "int4_quantised_moe_b200" / "csrc"
WAIT = "begin_after_previous();"


def closing(text, at, pair):
    """Index behind the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == pair[0]) - (text[i] == pair[1])
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced")


def kernels():
    """(file, name, parameters, body) of every kernel."""
    for path in sorted([*CSRC.glob("*.cu"), *CSRC.glob("*.cuh")]):
        text = re.sub(r"//[^\n]*", "", path.read_text())
        for m in re.finditer(r"__global__\s+void\s+", text):
            at = m.end()
            while text.startswith("__launch_bounds__", at):
                at = closing(text, text.index("(", at), "()")
                at += len(text[at:]) - len(text[at:].lstrip())
            name = re.match(r"\w+", text[at:]).group()
            params = text.index("(", at)
            end = closing(text, params, "()")
            body = re.match(r"\s*\{", text[end:])
            if body:
                yield path.name, name, text[params:end], text[end:closing(text, end + body.end() - 1, "{}")]


EARLY = [k for k in kernels() if WAIT in k[3]]


def test_the_kernels_are_found():
    names = {k[1] for k in EARLY}
    assert {"norm_fold_kernel", "norm_fwd_kernel", "norm_bwd_kernel", "ckpt8_save_vec", "ckpt8_load_any", "select_kernel",
            "select_bwd_kernel", "clear_counts_kernel"} <= names


@pytest.mark.parametrize("file,name,params,body", EARLY, ids=[k[1] for k in EARLY])
def test_no_promise_that_inputs_stay(file, name, params, body):
    assert "__restrict__" not in params + body, (file, name)
    assert "__ldg" not in body and "ld.global.nc" not in body, (file, name)


def test_what_is_started_early_waits():
    waiting = {k[1] for k in EARLY}
    every = {k[1] for k in kernels()}
    started = set()
    for path in [*CSRC.glob("*.cu"), *CSRC.glob("*.cuh")]:
        for m in re.finditer(r"launch_early\(", path.read_text()):
            text = path.read_text()
            started |= set(re.findall(r"\w+", text[m.start():closing(text, m.end() - 1, "()")])) & every
    assert started and started <= waiting
