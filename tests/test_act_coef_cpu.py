"""One table of the activations' coefficients serves every kernel."""

import glob
import os
import re

import pytest

from memory_efficient_activation_amd import _lib

CSRC = os.path.join(os.path.dirname(os.path.abspath(_lib.__file__)), "csrc")


def test_the_coefficients_stand_once():
    found = [(os.path.basename(f), m) for f in sorted(glob.glob(os.path.join(CSRC, "*.h*")))
             for m in re.findall(r"\bCoef make_coef\(|1\.442695040888963407\d*", open(f).read())]
    assert [f for f, _ in found] == ["act_math.h"] * 2


@pytest.mark.parametrize("alpha,ok", [(2.35e38, True), (2.37e38, False), (-2.35e38, True),
                                      (-2.37e38, False), (0.0, True)])
def test_both_entries_draw_the_same_line(alpha, ok):
    lib = _lib.library()
    want = _lib.OK if ok else _lib.EINVAL
    assert lib.meswish_act_fwd(0, None, None, 0, alpha, 0, None) == want
    # No tokens: nothing is launched.
    assert lib.gated_ffn_fwd(0, alpha, None, 8, 0x10000, 8, 0x20000, 8, 0, 8, 8, None, 8, None, 0,
                             0, None) == want
