"""The tests' sizes of 8-bit products reach every kernel that the library's rule
(matmul in int8.hip) can choose: the rule is read from the source, so that a
changed threshold that drops one fails here."""

import os
import re

import test_gpu_int8
import test_gpu_int8_tiles
from quantized_recurrent_state_gdnq_amd import build


def rule():
    """[(condition or None, kernel)] of the rule, conditions as Python's."""
    with open(os.path.join(build.CSRC, "int8.hip")) as f:
        text = f.read()
    body = text[text.index("hipError_t matmul("):text.index("hipError_t quantize(")]
    assert "rows = count(32, 16);" in body
    steps = re.findall(r"(?:if \((.*)\) )?return ((?:rows|tile)_product<.*?>)", body)
    python = lambda c: c.replace("&&", "and").replace("||", "or").replace("L.K", "K")  # noqa: E731
    return [(python(c) if c else None, kernel) for c, kernel in steps]


def choice(steps, M, N, K):
    def count(m, n):
        return -(-M // m) * -(-N // n)

    for condition, kernel in steps:
        if condition is None or eval(condition, {"count": count, "rows": count(32, 16), "K": K}):
            return kernel


def test_every_choice_is_tested():
    steps = rule()
    assert len(steps) == 7 and steps[-1][0] is None and all(c for c, _ in steps[:-1])
    sizes = test_gpu_int8.SIZES + test_gpu_int8_tiles.SIZES
    assert {choice(steps, *s) for s in sizes} == {kernel for _, kernel in steps}
    assert {choice(steps, *s) for s in test_gpu_int8_tiles.SIZES} == {steps[-1][1]}
    assert choice(steps, 2048, 4096, 4096) == steps[-1][1] == "tile_product<128, 128, 2, 2, 128, E>"
