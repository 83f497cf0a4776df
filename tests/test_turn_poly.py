"""CPU pin of the polynomials that the rotary tables evaluate: parsed from the
source, evaluated in float32 Horner arithmetic, against numpy and the fit."""
import os
import re

import numpy as np

from tests.test_poly_constants import CSRC, _fit_module, _horner


def test_turn_polynomials():
    """The rotary tables' sine and cosine of half turns: the sources' constants are
    the fit's, and within 9e-8 of numpy's in float32 steps."""
    txt = open(os.path.join(CSRC, "rope.cu")).read()
    k = [np.array([float(x.strip().rstrip("f")) for x in re.search(rf"{n}\[\d\]\s*=\s*\{{([^}}]*)\}}", txt).group(1).split(",")],
                  dtype=np.float32) for n in ("kTurnS", "kTurnC")]
    s, c, _, _ = _fit_module().fit_turn()
    assert np.array_equal(k[0], s) and np.array_equal(k[1], c)
    x = np.linspace(-0.25, 0.25, 200001).astype(np.float32)
    z = (x * x).astype(np.float32)
    for got, want in (((x * _horner(k[0], z)).astype(np.float32), np.sin(np.pi * x.astype(np.float64))),
                      (_horner(k[1], z), np.cos(np.pi * x.astype(np.float64)))):
        assert np.max(np.abs(got - want)) < 9e-8
