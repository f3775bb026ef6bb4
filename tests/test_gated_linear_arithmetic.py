"""The decay's polynomials as they stand in the kernels' source, against e^x - 1 in 64 bits: their errors are
what the comment beside them says, and below half a step of fp32."""
import os
import re

import numpy as np

from mamba_chunked_ssd_gb300 import build_lib


def source():
    text = open(os.path.join(build_lib.CSRC, "glr_math.cuh")).read()
    return text[text.index("// a = e^la and m"):text.index("// sqrt(m)")]


def forms():
    """The coefficients of both forms from the highest one on, as fp32 values: (narrow, wide)."""
    found = []
    for form in source()[source().index("decay2("):].split("} else {")[:2]:
        c = re.findall(r"f2\((-?\d+\.\d*)f\)", form[:form.index("= mul2(")])
        found.append([np.float64(np.float32(float(v))) for v in c if float(v) not in (-87.0, -0.693147180559945)])
    return found


def horner(coefficients, x):
    p = np.zeros_like(x)
    for c in coefficients:
        p = p * x + c
    return p * x


def worst(coefficients, lo, hi):
    x = np.linspace(lo, hi, 2_000_001)
    x = x[x != 0]
    return np.abs(horner(coefficients, x) / np.expm1(x) - 1).max()


def test_errors_are_those_of_the_comment():
    said = [float(v) for v in re.findall(r"\((\d\.\de-\d+)", source())]
    assert len(said) == 2
    narrow, wide = forms()
    assert len(narrow) == 7 and len(wide) == 6 and narrow[-1] == wide[-1] == 1.0
    half = np.log(2) / 2
    # (the wide form's ends lie a rounding of n ln 2 beyond half of it)
    for found, stated in ((worst(narrow, -1, 0), said[0]), (worst(wide, -half * 1.001, half * 1.001), said[1])):
        assert 0.9 * stated <= found <= 1.05 * stated, (found, stated)
        assert found < 2.0 ** -24
