"""The activations' coefficients stand in two host files (the activations' own and
the gated unit's): the same table, and the same limit of Swish's slope."""

import os
import re

import pytest

from memory_efficient_activation_amd import _lib

CSRC = os.path.join(os.path.dirname(os.path.abspath(_lib.__file__)), "csrc")
NAMES = {"MESWISH_ACT_SWISH": "kSwish", "MESWISH_ACT_SIGMOID": "kSigmoid",
         "MESWISH_ACT_TANH": "kTanh", "MESWISH_ACT_GELU_ERF": "kGeluErf",
         "MESWISH_ACT_GELU_TANH": "kGeluTanh"}


def table(name):
    text = open(os.path.join(CSRC, name)).read()
    body = re.search(r"static Coef make_coef\(int act, float p\)\n\{.*?\n\}\n", text, re.S).group(0)
    body = re.sub(r"//[^\n]*", "", body)
    for long, short in NAMES.items():
        body = body.replace(long, short)
    return body.split()


def test_both_tables_are_the_same():
    assert table("gated_ffn.hip") == table("meswish.hip")


@pytest.mark.parametrize("alpha,ok", [(2.35e38, True), (2.37e38, False), (-2.35e38, True),
                                      (-2.37e38, False), (0.0, True)])
def test_both_entries_draw_the_same_line(alpha, ok):
    lib = _lib.library()
    want = _lib.OK if ok else _lib.EINVAL
    assert lib.meswish_act_fwd(0, None, None, 0, alpha, 0, None) == want
    # No tokens: nothing is launched.
    assert lib.gated_ffn_fwd(0, alpha, None, 8, 0x10000, 8, 0x20000, 8, 0, 8, 8, None, 8, None, 0,
                             0, None) == want
