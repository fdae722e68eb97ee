"""Which rows the gated unit's binding copies before the library sees them."""

import os
import re

import torch

from memory_efficient_activation_amd import _lib, ffn, norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_limit_is_the_headers():
    text = open(os.path.join(ROOT, "include", "gated_ffn.h")).read()
    assert int(re.search(r"#define GATED_FFN_MAX_LD (\d+)", text).group(1)) == _lib.GATED_FFN_MAX_LD


def test_rows_far_apart_are_copied(monkeypatch):
    monkeypatch.setattr(norm, "_require_device", lambda t, name: None)
    far = torch.randn(2, _lib.GATED_FFN_MAX_LD // 8 + 1, 8)[:, -1]  # the last token of each
    got, ld = ffn._rows(far, "x")
    assert got is not far and torch.equal(got, far) and ld == 8
    near = torch.randn(2, _lib.GATED_FFN_MAX_LD // 8, 8)[:, -1]
    got, ld = ffn._rows(near, "x")
    assert got is near and ld == _lib.GATED_FFN_MAX_LD
    one = torch.randn(1, 40, 8)[:, -1]
    assert ffn._rows(one, "x") == (one, 8)
