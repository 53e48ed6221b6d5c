"""Kernels that may start before their predecessor has ended (launch_after) wait
for it before they load anything, and load nothing through the non-coherent
path, which that wait does not order.  Shown on the sources: a read that comes
too early is a matter of timing, and seldom seen in a result."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_cross_entropy_gb300", "csrc")
FILES = ("norm.cuh", "grad_clip.cu")
# A load of global memory, or a function of the file that makes one.
LOADS = re.compile(r"\.load\w*\(|load_\w+[<(]|copy_async<|request\w*\(|gather_typed|scale_from|k\.part|a\.mean\[|a\.rstd\[")


def _source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def _body(text, at):
    """From the first brace behind `at` to its partner."""
    start = text.index("{", at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]


def _kernels(text):
    return {m.group(1): _body(text, m.end())
            for m in re.finditer(r"__global__ void (?:__launch_bounds__\([^)]*\) )?(\w+)\(", text)}


def _started_early(text, kernels):
    """Kernels handed to launch_after, by name or as the variable `kernel`."""
    names = set()
    for m in re.finditer(r"launch_after\((\w+)", text):
        if m.group(1) != "kernel":
            names.add(m.group(1))
            continue
        before = text[:m.start()]
        names.add(re.findall(r"auto kernel = (\w+)<", before)[-1])
    assert names and names <= set(kernels)
    return names


@pytest.mark.parametrize("name", FILES)
def test_early_kernels_wait_before_they_load(name):
    text = _source(name)
    kernels = _kernels(text)
    for k in _started_early(text, kernels):
        body = kernels[k]
        wait = re.search(r"wait_for_previous\(\)|total_norm\(", body)
        assert wait, k
        # functions that are only defined before the wait load nothing yet
        before = re.sub(r"auto \w+ = \[&\]\([^)]*\) \{", "LAMBDA {", body[:wait.start()])
        while "LAMBDA" in before:
            at = before.index("LAMBDA")
            before = before[:at] + before[at + len("LAMBDA "):].replace(_body(before, at), "", 1)
        assert not LOADS.search(before), k
    total = _body(text, text.index("float total_norm(")) if "float total_norm(" in text else None
    if total:
        assert total.index("wait_for_previous()") < LOADS.search(total).start()


@pytest.mark.parametrize("name", FILES)
def test_early_kernels_load_nothing_as_constant(name):
    text = _source(name)
    kernels = _kernels(text)
    assert "__ldg" not in text and ".nc" not in text
    early = _started_early(text, kernels)
    for k, body in kernels.items():
        if re.search(r"load_constant|, true>\(", body):
            assert k not in early and "wait_for_previous" not in body, k
            assert re.search(k + r"<[^;(]*>\s*<<<", text), k  # an ordinary launch


def test_the_only_constant_load_is_the_one_that_says_so():
    text = _source("elements.cuh")
    assert text.count("__ldg") == 1 and "ld.global.nc" not in text
    at = text.index("__ldg")
    assert "if constexpr (CONSTANT)" in text[at - 60:at]
    assert re.search(r"void load\(const T\* p\) \{ load_as<false>\(p\); \}", text)
