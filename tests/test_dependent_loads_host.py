"""Loads of kernels that may start before the kernel in front of them has ended (no GPU needed: the sources are read).

A kernel launched with the programmatic attribute overlaps the one that writes its inputs. ``ld.global.nc`` and
``__ldg`` are for data that nobody writes while the kernel runs, and the compiler may move ``__ldg`` (or a load through
a ``const __restrict__`` pointer, which it takes for one) above ``griddepcontrol.wait``. So in every file with such a
kernel they may read weights only; activations, codes, scales, ids and offsets are read by coherent loads."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_only_pack_b200", "csrc")

# what the non-coherent loads of each file may read: the weights
WEIGHTS = {
    "w8a8.cuh": {"row + (size_t)c * 16"},  # `row` is a row of wq
    "moe_rows.cuh": set(),
}


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def argument(text, at):
    """The text between the bracket at `at` and the one that closes it."""
    depth = 0
    for i in range(at, len(text)):
        depth += {"(": 1, ")": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError("unbalanced")


@pytest.mark.parametrize("name", sorted(WEIGHTS))
def test_noncoherent_loads_read_weights_only(name):
    text = code(name)
    assert "griddep" in text
    read = {argument(text, m.end() - 1) for m in re.finditer(r"\b(?:__ldg|ld_nc_v4|ld_stream_v4)\(", text)}
    assert read <= WEIGHTS[name], f"{name}: {sorted(read - WEIGHTS[name])}"


@pytest.mark.parametrize("name", sorted(WEIGHTS))
def test_kernels_that_wait_take_no_restrict_inputs(name):
    text = code(name)
    for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\(([^{;]*)\)\s*\{", text):
        body = text[m.end():text.find("\n}", m.end())]
        if "griddep" in body:
            assert not re.search(r"const [\w ]+\*\s*__restrict__", m.group(2)), f"{name}: {m.group(1)}"
