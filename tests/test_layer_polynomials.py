"""The polynomials that stand for functions in the selective scan, with the coefficients as they are in the source, against these functions
in 64 bits: that they are off by no more than their comments say, and off to both sides alike."""
import os
import re

import numpy as np

from orthogonal_update_recurrent_b200 import build

with open(os.path.join(build.CSRC, "selective.cuh")) as f:
    SOURCE = f.read()
NUMBER = r"f2\((-?[0-9.]+)f\)"


def coefficients(function):
    """the Horner scheme's in `function`, highest power first, as fp32"""
    body = SOURCE[SOURCE.index(function):]
    body = body[:body.index("\n}\n")]
    first = re.search(rf"fma2\({NUMBER}, t(?:\[i\])?, {NUMBER}\)", body)
    rest = re.findall(rf"fma2\(p(?:\[i\])?, t(?:\[i\])?, {NUMBER}\)", body)
    return [float(np.float32(v)) for v in (*first.groups(), *rest)]


def error(c, t, want):
    return (np.polyval(c, t) - want) / want


def test_softplus():
    t = np.linspace(1e-9, 1, 200001)
    c = coefficients("F2 softplus(")
    assert len(c) == 10 and c[-1] == 1.0
    e = error(c, t, np.log1p(t) / t)
    assert np.abs(e).max() <= 5.4e-9 and abs(e.mean()) <= 1e-10


def test_decay():
    near = float(np.float32(re.search(r"kNear = (-[0-9.]+)f", SOURCE).group(1)))
    t = np.linspace(near, 0, 200001)
    c = coefficients("void decay(")
    assert len(c) == 4 and c[-1] == 1.0
    e = error(c, t, np.exp2(t))
    assert np.abs(e).max() <= 6.7e-9 and abs(e.mean()) <= 1e-10
