"""The C boundary of layer_norm.h and gated_ffn.h on the CPU: exports, the
binding's tables, workspace sizes, and every refusal that is answered before
anything is launched."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

from memory_efficient_activation_amd import _lib, ffn, norm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", h) for h in ("layer_norm.h", "gated_ffn.h")]


def header_text():
    text = "".join(open(h).read() + "\n" for h in HEADERS)
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


@pytest.fixture(scope="module")
def lib():
    return _lib.library()


def test_exports_and_binding(lib):
    declared = set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\([^;{]*\)\s*;", header_text()))
    assert declared == set(_lib.BLOCK_EXPORTED) == set(_lib._block_signatures())
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIBRARY], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert declared <= exported
    # As many arguments as the declarations have.
    for name, (args, _) in _lib._block_signatures().items():
        decl = re.search(r"\b" + name + r"\s*\(([^;{]*)\)\s*;", header_text()).group(1)
        assert len(args) == decl.count(",") + 1, name


def test_headers_compile_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "layer_norm.h"\n#include "gated_ffn.h"\nint main(void){return 0;}\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only",
                    "-I" + os.path.join(ROOT, "include"), str(src)], check=True)


# Addresses that are only compared, never read: every call below is refused
# (or has nothing to do) before a launch.
X, DY, OUT, W, B, M, R, WS = (0x10000000 * k for k in range(1, 9))


def norm_fwd(lib, x=X, ldx=64, w=W, b=B, rows=4, n=64, eps=1e-5, y=OUT, ldy=64, mean=M, rstd=R,
             dtype=0, pdtype=0):
    return lib.layer_norm_fwd(x, ldx, w, b, rows, n, eps, y, ldy, mean, rstd, dtype, pdtype, None)


def test_norm_forward_refusals(lib):
    E, A = _lib.EINVAL, _lib.EALIAS
    assert norm_fwd(lib, dtype=2) == E and norm_fwd(lib, pdtype=-1) == E
    for eps in (float("nan"), float("inf"), -1e-5):
        assert norm_fwd(lib, eps=eps) == E
    assert norm_fwd(lib, x=None) == E and norm_fwd(lib, y=None) == E
    assert norm_fwd(lib, x=X + 2) == E and norm_fwd(lib, w=W + 2) == E
    assert norm_fwd(lib, mean=M + 1) == E
    assert norm_fwd(lib, ldx=63) == E and norm_fwd(lib, ldy=63) == E
    assert norm_fwd(lib, n=1 << 31, ldx=1 << 31, ldy=1 << 31) == E
    assert norm_fwd(lib, rows=1 << 58) == E
    assert norm_fwd(lib, y=X + 16) == A
    assert norm_fwd(lib, y=X, ldy=80) == A
    assert norm_fwd(lib, y=W) == A and norm_fwd(lib, mean=R) == A
    assert norm_fwd(lib, mean=OUT + 4 * 64 * 3) == A
    assert norm_fwd(lib, x=None, y=None, rows=0) == _lib.OK
    assert norm_fwd(lib, x=None, y=None, n=0) == _lib.OK


def norm_bwd(lib, x=X, ldx=64, dy=DY, lddy=64, mean=M, rstd=R, w=W, rows=4, n=64, dx=OUT, lddx=64,
             dw=B, db=B + 4096, ws=WS, wsb=None, dtype=0, pdtype=0):
    if wsb is None:
        wsb = lib.layer_norm_workspace_bytes(rows, n)
    return lib.layer_norm_bwd(x, ldx, dy, lddy, mean, rstd, w, rows, n, dx, lddx, dw, db, ws, wsb,
                              dtype, pdtype, None)


def test_norm_backward_refusals(lib):
    E, A = _lib.EINVAL, _lib.EALIAS
    assert norm_bwd(lib, dtype=5) == E and norm_bwd(lib, pdtype=5) == E
    for name in ("x", "dy", "mean", "rstd", "dx", "ws"):
        assert norm_bwd(lib, **{name: None}) == E, name
    assert norm_bwd(lib, wsb=lib.layer_norm_workspace_bytes(4, 64) - 1) == E
    assert norm_bwd(lib, ws=WS + 2) == E and norm_bwd(lib, dw=B + 2) == E
    assert norm_bwd(lib, lddx=10) == E
    assert norm_bwd(lib, n=1 << 31, wsb=1) == E
    assert norm_bwd(lib, dx=X + 4) == A and norm_bwd(lib, dw=W) == A
    assert norm_bwd(lib, db=B + 4) == A and norm_bwd(lib, ws=OUT) == A
    assert norm_bwd(lib, ws=M) == A
    assert norm_bwd(lib, n=0) == _lib.OK
    assert norm_bwd(lib, rows=0, dw=None, db=None, ws=None, wsb=0) == _lib.OK
    assert lib.layer_norm_workspace_bytes(10, 1 << 31) == 0
    assert lib.layer_norm_workspace_bytes(1, 100) >= 800


def ffn_fwd(lib, act=0, param=1.0, x=X, ldx=64, wg=W, ldwg=64, wu=B, ldwu=64, tokens=4, dim=64,
            hidden=32, h=OUT, ldh=32, ws=WS, wsb=1 << 27, dtype=1):
    return lib.gated_ffn_fwd(act, param, x, ldx, wg, ldwg, wu, ldwu, tokens, dim, hidden, h, ldh,
                             ws, wsb, dtype, None)


def test_unit_forward_refusals(lib):
    E, A = _lib.EINVAL, _lib.EALIAS
    assert ffn_fwd(lib, act=7) == E and ffn_fwd(lib, act=-1) == E
    assert ffn_fwd(lib, param=float("nan")) == E and ffn_fwd(lib, param=3e38) == E
    assert ffn_fwd(lib, dtype=2) == E
    for name in ("x", "wg", "wu", "h"):
        assert ffn_fwd(lib, **{name: None}) == E, name
        assert ffn_fwd(lib, **{name: 0x90000001}) == E, name
    for name in ("ldx", "ldwg", "ldwu", "ldh"):
        assert ffn_fwd(lib, **{name: 31}) == E, name
        assert ffn_fwd(lib, **{name: 2097153}) == E, name
    assert ffn_fwd(lib, tokens=1 << 30) == E
    assert ffn_fwd(lib, dim=2097153, ldx=2097152) == E
    assert ffn_fwd(lib, h=X) == A and ffn_fwd(lib, h=W + 64) == A and ffn_fwd(lib, h=B) == A
    assert ffn_fwd(lib, tokens=0, x=None, h=None) == _lib.OK
    assert ffn_fwd(lib, hidden=0, wg=None, wu=None, h=None, ldh=0) == _lib.OK


DX, DWG, DWU, H = (0x10000000 * k for k in range(16, 20))


def ffn_bwd(lib, act=0, param=1.0, x=X, ldx=64, wg=W, ldwg=64, wu=B, ldwu=64, dh=DY, lddh=32,
            tokens=4, dim=64, hidden=32, dx=DX, lddx=64, dwg=DWG, lddwg=64, dwu=DWU, lddwu=64,
            h=H, ldh=32, ws=WS, wsb=None, dtype=1):
    if wsb is None:
        wsb = lib.gated_ffn_workspace_bytes(tokens, dim, hidden, dtype, 1, 1)
    return lib.gated_ffn_bwd(act, param, x, ldx, wg, ldwg, wu, ldwu, dh, lddh, tokens, dim, hidden,
                             dx, lddx, dwg, lddwg, dwu, lddwu, h, ldh, ws, wsb, dtype, None)


def test_unit_backward_refusals(lib):
    E, A = _lib.EINVAL, _lib.EALIAS
    assert ffn_bwd(lib, act=9) == E and ffn_bwd(lib, param=float("inf")) == E
    assert ffn_bwd(lib, dtype=-1, wsb=1 << 20) == E
    for name in ("x", "wg", "wu", "dh", "ws"):
        assert ffn_bwd(lib, **{name: None}) == E, name
    assert ffn_bwd(lib, dwg=None) == E and ffn_bwd(lib, dwu=None) == E
    for name in ("lddh", "lddx", "lddwg", "lddwu", "ldh"):
        assert ffn_bwd(lib, **{name: 31}) == E, name
    assert ffn_bwd(lib, ws=WS + 8) == E
    assert ffn_bwd(lib, wsb=lib.gated_ffn_workspace_bytes(4, 64, 32, 1, 1, 1) - 1) == E
    for name in ("dx", "dwg", "dwu", "h", "ws"):
        assert ffn_bwd(lib, **{name: X}) == A, name
        assert ffn_bwd(lib, **{name: DY}) == A, name
    assert ffn_bwd(lib, dwu=DWG) == A and ffn_bwd(lib, h=DX) == A
    assert ffn_bwd(lib, tokens=0, dim=0, x=None, dh=None, ws=None) == _lib.OK


def test_workspace_sizes(lib):
    size = lib.gated_ffn_workspace_bytes
    for dtype, es in ((0, 4), (1, 2)):
        # dg and du at the least; the padded copies of x, wg and wu beside them
        # where rows are not aligned, or cannot be.
        assert size(10, 64, 100, dtype, 1, 1) >= 2 * 10 * 100 * es
        assert size(10, 64, 100, dtype, 1, 0) >= size(10, 64, 100, dtype, 1, 1) + 210 * 64 * es
        assert size(10, 63, 100, dtype, 1, 1) == size(10, 63, 100, dtype, 1, 0)
        assert size(10, 63, 100, dtype, 0, 0) == 0  # few tokens: any rows
        assert size(100, 63, 100, dtype, 0, 0) >= 300 * 63 * es
    assert size(1 << 30, 64, 64, 1, 1, 1) == 0
    assert size(4, 64, 64, 3, 1, 1) == 0


def test_unaligned_rows_need_the_larger_workspace(lib):
    small = lib.gated_ffn_workspace_bytes(100, 64, 32, 1, 1, 1)
    assert small < lib.gated_ffn_workspace_bytes(100, 64, 32, 1, 1, 0)
    for bad in ({"x": X + 2}, {"ldx": 65}, {"wg": W + 4}, {"ldwg": 72}, {"wu": B + 8}):
        assert ffn_bwd(lib, tokens=100, wsb=small, **bad) == _lib.EINVAL, bad


def test_cpu_tensors_are_refused():
    x, w = torch.randn(4, 8), torch.randn(16, 8)
    with pytest.raises(RuntimeError, match="no CPU path"):
        norm.layer_norm_fwd(x)
    with pytest.raises(RuntimeError, match="no CPU path"):
        norm.layer_norm_bwd(x, x, x[:, 0], x[:, 0])
    with pytest.raises(RuntimeError, match="no CPU path"):
        ffn.gated_ffn_fwd(x, w, w)
    with pytest.raises(RuntimeError, match="no CPU path"):
        ffn.gated_ffn_bwd(x, w, w, torch.randn(4, 16))
    with pytest.raises(RuntimeError, match="no CPU path"):
        ffn.PreNormGatedFeedForward(8, 16)(x)
    with pytest.raises(ValueError, match="unknown activation"):
        ffn.GatedUnit(8, 16, "softmax")


def test_rows_of_a_tensor(monkeypatch):
    """Which strides are read in place and which are copied."""
    monkeypatch.setattr(norm, "_require_device", lambda t, name: None)
    t = torch.randn(6, 5, 32)
    assert norm.as_rows(t, "t")[1:] == (30, 32, 32)
    part = t[..., 3:20]
    assert norm.as_rows(part, "t")[0] is part and norm.as_rows(part, "t")[1:] == (30, 17, 32)
    some = t[:, 1:3]
    got = norm.as_rows(some, "t")
    assert got[0] is not some and got[0].is_contiguous() and got[1:] == (12, 32, 32)
    flip = t.transpose(0, 1)
    assert norm.as_rows(flip, "t")[0].is_contiguous()
    wide = t[0].expand(4, 5, 32)
    assert norm.as_rows(wide, "t")[0].is_contiguous()
    one = t[:1, :, :4]
    assert norm.as_rows(one, "t")[0] is one and norm.as_rows(one, "t")[1:] == (5, 4, 32)
    col = t[:, 0, 0]
    assert norm.as_rows(col, "t")[0].is_contiguous()
    assert norm.as_rows(torch.randn(7, 1).t(), "t")[1:] == (1, 7, 7)
    assert norm.as_rows(torch.empty(0, 9), "t")[1:] == (0, 9, 9)
    assert norm.as_rows(torch.empty(3, 0), "t")[2:] == (0, 0)


def test_interleaved_column_ranges_do_not_overlap(lib):
    """Two column ranges of one matrix are apart; rows that reach into each
    other are not.  (Refused calls only: rows == 0 and n == 0 do nothing, so
    the accepted side is on the GPU.)"""
    ld = 200
    assert norm_fwd(lib, ldx=ld, y=X + 4 * 63, ldy=ld) == _lib.EALIAS
    assert norm_fwd(lib, ldx=ld, y=X + 4 * (ld - 63), ldy=ld) == _lib.EALIAS
    assert norm_fwd(lib, ldx=ld, y=X - 4 * (ld - 63), ldy=ld) == _lib.EALIAS
