"""Loads of kernels that may start before the kernel in front of them has ended (no GPU needed: the sources are read).

A kernel launched with the programmatic attribute overlaps the one that writes its inputs. ``ld.global.nc`` and
``__ldg`` are for data that nobody writes while the kernel runs, and the compiler may move ``__ldg`` (or a load through
a ``const __restrict__`` pointer, which it takes for one) above ``griddepcontrol.wait``. So in every file with such a
kernel they may read weights only; activations, codes, scales, ids and offsets are read by coherent loads."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_only_pack_b200", "csrc")

# what the non-coherent loads of each file may read: the weights (codes, scales a.s, zero points a.z, tables)
WEIGHTS = {
    "w8a8.cuh": {"row + (size_t)c * 16"},  # `row` is a row of wq
    "moe_rows.cuh": set(),
    "affine.cuh": {"p + 16 * i",  # `p` is a row's chunk in the code stream
                   *(f"reinterpret_cast<const {t}*>(a.{f})" for f, ts in (("s", ("uint4", "uint2", "uint32_t")),
                                                                          ("z", ("uint2", "uint32_t", "uint16_t")))
                     for t in ts)},
    "gemv_direct.cuh": {"a.q[it] + (size_t)(r0 + i) * rowb + (size_t)c * 16", "a.s[it] + m0 * 2"},
    "gemv_m1.cuh": set(),
    "gemv_tmma.cuh": set(),
    "lut3_direct.cuh": {"base + 16 * v",  # `base` is a tile's indices
                        "a.t_region + ((size_t)kt * (a.N >> 3) + rb) * 16"},
    "lut3_gemv.cuh": set(),
    "lut3_tmma.cuh": set(),
    "lut3_tmma_batch.cuh": set(),
    "skinny.cuh": set(),
    "tc_gemv.cuh": set(),
    "w4a8.cuh": {"a.q + (size_t)(n0 + r) * rowb + (size_t)c * 16",
                 *(f"reinterpret_cast<const {t}*>(a.{f})" for f, ts in (("s", ("uint4", "uint2", "uint32_t")),
                                                                        ("z", ("uint2", "uint32_t", "uint16_t")))
                   for t in ts)},
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
    read = {re.sub(r" \+ mi / \d$", "", r) for r in read}
    assert read <= WEIGHTS[name], f"{name}: {sorted(read - WEIGHTS[name])}"


@pytest.mark.parametrize("name", sorted(WEIGHTS))
def test_kernels_that_wait_take_no_restrict_inputs(name):
    text = code(name)
    for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\(([^{;]*)\)\s*\{", text):
        body = text[m.end():text.find("\n}", m.end())]
        if "griddep" in body:
            assert not re.search(r"const [\w ]+\*\s*__restrict__", m.group(2)), f"{name}: {m.group(1)}"


def test_every_file_with_a_wait_is_listed():
    assert {f for f in os.listdir(CSRC) if re.search(r"griddep_wait\(\)|griddepcontrol\.wait", code(f))} == set(WEIGHTS)
