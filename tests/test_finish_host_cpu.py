"""The C boundary of linear.h and residual_norm.h on the CPU: exports, the
binding's tables, workspace sizes, and every refusal that is answered before
anything is launched."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

from memory_efficient_activation_amd import _lib, linear, residual

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = [os.path.join(ROOT, "include", h) for h in ("linear.h", "residual_norm.h")]


def header_text():
    text = "".join(open(h).read() + "\n" for h in HEADERS)
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


@pytest.fixture(scope="module")
def lib():
    return _lib.library()


def test_exports_and_binding(lib):
    declared = set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\([^;{]*\)\s*;", header_text()))
    assert declared == set(_lib.FINISH_EXPORTED) == set(_lib._finish_signatures())
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIBRARY], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if " T " in line}
    assert declared <= exported
    for name, (args, _) in _lib._finish_signatures().items():
        decl = re.search(r"\b" + name + r"\s*\(([^;{]*)\)\s*;", header_text()).group(1)
        assert len(args) == decl.count(",") + 1, name
    for name in ("LINEAR_MAX_LD", "LINEAR_IDENTITY", "LINEAR_ALIGNED_XW", "LINEAR_ALIGNED_DY"):
        value = re.search(r"#define " + name + r" \(?(-?\d+)\)?", header_text()).group(1)
        assert getattr(_lib, name) == int(value)


def test_description_has_the_headers_layout(tmp_path):
    """Offsets and size of residual_norm_op, as a C compiler lays it out."""
    fields = [f for f, _ in _lib.ResidualNormOp._fields_]
    src = tmp_path / "t.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "linear.h"\n'
                   '#include "residual_norm.h"\nint main(void){'
                   + "".join(f'printf("%zu ", offsetof(residual_norm_op, {f}));' for f in fields)
                   + 'printf("%zu", sizeof(residual_norm_op));return 0;}\n')
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"),
                    str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    want = [getattr(_lib.ResidualNormOp, f).offset for f in fields]
    assert [int(v) for v in got] == want + [ctypes.sizeof(_lib.ResidualNormOp)]


# Addresses that are only compared, never read: every call below is refused
# (or has nothing to do) before a launch.
X, W, B, R, Y, DY, DX, DW, DB, WS = (0x10000000 * k for k in range(1, 11))


def lin_fwd(lib, act=-1, param=0.0, x=X, ldx=64, w=W, ldw=64, b=B, r=R, ldr=32, tokens=40, dim=64,
            units=32, y=Y, ldy=32, ws=WS, wsb=1 << 27, dtype=1):
    return lib.linear_fwd(act, param, x, ldx, w, ldw, b, r, ldr, tokens, dim, units, y, ldy, ws, wsb,
                          dtype, None)


def test_linear_forward_refusals(lib):
    E, A = _lib.EINVAL, _lib.EALIAS
    assert lin_fwd(lib, act=7) == E and lin_fwd(lib, act=-2) == E
    for act in (-1, 0):
        assert lin_fwd(lib, act=act, param=float("nan")) == E
    assert lin_fwd(lib, act=0, param=3e38) == E
    assert lin_fwd(lib, dtype=2) == E
    for name in ("x", "w", "y"):
        assert lin_fwd(lib, **{name: None}) == E, name
    for name in ("x", "w", "b", "r", "y"):
        assert lin_fwd(lib, **{name: 0xb0000001}) == E, name
    for name in ("ldx", "ldw", "ldr", "ldy"):
        assert lin_fwd(lib, **{name: 31}) == E, name
        assert lin_fwd(lib, **{name: 2097153}) == E, name
    assert lin_fwd(lib, tokens=1 << 30) == E
    assert lin_fwd(lib, dim=2097153, ldx=2097152) == E
    for at in (X, W + 64, B, R):
        assert lin_fwd(lib, y=at) == A, hex(at)
    # Rows off 16-byte boundaries need the workspace they are copied to.
    need = lib.linear_workspace_bytes(40, 64, 32, -1, 1, 0, 0)
    assert need > lib.linear_workspace_bytes(40, 64, 32, -1, 1, 0, 1)
    for bad in ({"x": X + 2}, {"ldx": 65}, {"w": W + 4}, {"ldw": 68}):
        assert lin_fwd(lib, wsb=need - 1, **bad) == E, bad
        assert lin_fwd(lib, ws=None, **bad) == E, bad
        assert lin_fwd(lib, ws=WS + 8, **bad) == E, bad
        assert lin_fwd(lib, ws=Y, **bad) == A, bad
    assert lin_fwd(lib, tokens=0, x=None, y=None, r=None) == _lib.OK
    assert lin_fwd(lib, units=0, w=None, y=None, ldy=0) == _lib.OK


def lin_bwd(lib, act=0, param=1.0, x=X, ldx=64, w=W, ldw=64, b=B, dy=DY, lddy=32, tokens=40, dim=64,
            units=32, dx=DX, lddx=64, dw=DW, lddw=64, db=DB, ws=WS, wsb=None, dtype=1):
    if wsb is None:
        wsb = lib.linear_workspace_bytes(tokens, dim, units, act, dtype, 1, 3)
    return lib.linear_bwd(act, param, x, ldx, w, ldw, b, dy, lddy, tokens, dim, units, dx, lddx, dw,
                          lddw, db, ws, wsb, dtype, None)


def test_linear_backward_refusals(lib):
    E, A = _lib.EINVAL, _lib.EALIAS
    assert lin_bwd(lib, act=9) == E and lin_bwd(lib, param=float("inf")) == E
    assert lin_bwd(lib, dtype=-1, wsb=1 << 20) == E
    for name in ("x", "w", "dy", "ws"):
        assert lin_bwd(lib, **{name: None}) == E, name
    for name in ("ldx", "ldw", "lddy", "lddx", "lddw"):
        assert lin_bwd(lib, **{name: 31}) == E, name
    for name in ("b", "db", "dx"):
        assert lin_bwd(lib, **{name: 0xb0000001}) == E, name
    assert lin_bwd(lib, ws=WS + 8) == E
    for act in (0, -1):
        assert lin_bwd(lib, act=act,
                       wsb=lib.linear_workspace_bytes(40, 64, 32, act, 1, 1, 3) - 1) == E
        for name in ("dx", "dw", "db", "ws"):
            for at in (X, W, B, DY):
                assert lin_bwd(lib, act=act, **{name: at}) == A, (act, name, hex(at))
    assert lin_bwd(lib, dw=DX) == A and lin_bwd(lib, db=DW + 2) == A
    # dy off 16-byte boundaries: copied, without an activation alone.
    small = lib.linear_workspace_bytes(40, 64, 32, -1, 1, 1, 3)
    assert lib.linear_workspace_bytes(40, 64, 32, -1, 1, 1, 1) > small
    assert lin_bwd(lib, act=-1, lddy=36, wsb=small) == E
    assert lin_bwd(lib, dx=None, dw=None, db=None) == _lib.OK


def test_linear_workspace_sizes(lib):
    size = lib.linear_workspace_bytes
    for dtype, es in ((0, 4), (1, 2)):
        assert size(10, 64, 100, 0, dtype, 1, 3) >= 10 * 100 * es  # dz
        assert size(10, 64, 100, 0, dtype, 1, 2) >= size(10, 64, 100, 0, dtype, 1, 3) + 110 * 64 * es
        assert size(10, 63, 100, 0, dtype, 1, 3) == size(10, 63, 100, 0, dtype, 1, 2)
        assert size(10, 64, 101, -1, dtype, 1, 3) == size(10, 64, 101, -1, dtype, 1, 1)
        assert size(100, 63, 100, -1, dtype, 0, 0) >= 200 * 63 * es
    assert size(1 << 30, 64, 64, 0, 1, 1, 3) == 0
    assert size(4, 64, 64, 0, 3, 1, 3) == 0
    assert size(4, 64, 64, 7, 1, 1, 3) == 0 and size(4, 64, 64, -2, 1, 1, 3) == 0


Z, O, GATE, QW, QB, NW, NB, S1, S2, S3, S4, DO, DZ, DG, P1, P2, P3, P4 = (
    0x10000000 * k for k in range(16, 34))


def op(**k):
    d = dict(rows=12, n=64, gates=3, gate=GATE, post_weight=QW, post_bias=QB, pre_weight=NW,
             pre_bias=NB, skip=1.0, scale=1.0, eps=1e-5, post=1, pre=1, center=1, stream_dtype=1,
             branch_dtype=1, param_dtype=0)
    d.update(k)
    packed = _lib.RESIDUAL_NORM_OP.pack(*d.values())
    assert packed == bytes(_lib.ResidualNormOp(**d))
    return packed


def rn_fwd(lib, x=X, ldx=64, z=Z, ldz=64, y=Y, ldy=64, o=O, ldo=64, s1=S1, s2=S2, s3=S3, s4=S4,
           **k):
    return lib.residual_norm_fwd(op(**k), x, ldx, z, ldz, y, ldy, o, ldo, s1, s2, s3, s4, None)


BAD = [dict(post=0, pre=0), dict(stream_dtype=2), dict(branch_dtype=-1), dict(param_dtype=3),
       dict(stream_dtype=1, branch_dtype=0), dict(skip=float("nan")), dict(scale=float("inf")),
       dict(eps=-1e-5), dict(eps=float("nan")), dict(gates=0), dict(gates=5), dict(gates=24),
       dict(n=1 << 31), dict(rows=1 << 59), dict(gate=GATE + 2), dict(post_weight=QW + 1),
       dict(pre_bias=NB + 2)]


@pytest.mark.parametrize("bad", BAD, ids=str)
def test_border_refuses_descriptions(lib, bad):
    assert rn_fwd(lib, **bad) == _lib.EINVAL
    assert rn_bwd(lib, **bad) == _lib.EINVAL


def test_border_forward_refusals(lib):
    E, A = _lib.EINVAL, _lib.EALIAS
    assert lib.residual_norm_fwd(None, X, 64, Z, 64, Y, 64, O, 64, S1, S2, S3, S4, None) == E
    for name in ("x", "z", "y", "o"):
        assert rn_fwd(lib, **{name: None}) == E, name
        assert rn_fwd(lib, **{name: 0xb0000001}) == E, name
        assert rn_fwd(lib, **{"ld" + name: 63}) == E, name
    for name in ("s1", "s2", "s3", "s4"):
        assert rn_fwd(lib, **{name: S1 + 2}) == E, name
    for name in ("y", "o", "s1", "s4"):
        for at in (X, Z, GATE + 64, QW, QB, NW, NB):
            assert rn_fwd(lib, **{name: at}) == A, (name, hex(at))
    assert rn_fwd(lib, o=Y + 2) == A and rn_fwd(lib, s2=S1) == A and rn_fwd(lib, s3=Y) == A
    assert rn_fwd(lib, rows=0, x=None) == _lib.OK and rn_fwd(lib, n=0, x=None) == _lib.OK


def rn_bwd(lib, y=Y, ldy=64, z=Z, ldz=64, dy=DY, lddy=64, do=DO, lddo=64, s1=S1, s2=S2, s3=S3,
           s4=S4, dx=DX, lddx=64, dz=DZ, lddz=64, dg=DG, p1=P1, p2=P2, p3=P3, p4=P4, ws=WS, wsb=None,
           **k):
    if wsb is None:
        wsb = lib.residual_norm_workspace_bytes(12, 64, 3)
    return lib.residual_norm_bwd(op(**k), y, ldy, z, ldz, dy, lddy, do, lddo, s1, s2, s3, s4, dx,
                                 lddx, dz, lddz, dg, p1, p2, p3, p4, ws, wsb, None)


def test_border_backward_refusals(lib):
    E, A = _lib.EINVAL, _lib.EALIAS
    for name in ("y", "z", "do", "dx", "dz", "s1", "s2", "s3", "s4", "ws"):
        assert rn_bwd(lib, **{name: None}) == E, name
    for name in ("y", "z", "dy", "do", "dx", "dz"):
        assert rn_bwd(lib, **{"ld" + name: 63}) == E, name
    for name in ("dg", "p1", "p4", "s2"):
        assert rn_bwd(lib, **{name: 0xb0000002}) == E, name
    assert rn_bwd(lib, ws=WS + 8) == E
    assert rn_bwd(lib, wsb=lib.residual_norm_workspace_bytes(12, 64, 3) - 1) == E
    for name in ("dx", "dz", "dg", "p1", "p2", "p3", "p4", "ws"):
        for at in (Y, Z, DY, DO, S1, S4, GATE, QW, NB):
            assert rn_bwd(lib, **{name: at}) == A, (name, hex(at))
    assert rn_bwd(lib, dz=DX) == A and rn_bwd(lib, p2=P1 + 4) == A and rn_bwd(lib, dg=WS) == A
    assert rn_bwd(lib, n=0) == _lib.OK
    assert rn_bwd(lib, rows=0, gates=1, dg=None, p1=None, p2=None, p3=None, p4=None) == _lib.OK


def test_border_workspace_sizes(lib):
    size = lib.residual_norm_workspace_bytes
    assert size(1000, 64, 3) == 0  # 3 does not divide 1000
    assert size(1000, 1 << 31, 1) == 0 and size(1000, 64, 0) == 0 and size(8, 64, 16) == 0
    assert size(1, 100, 1) >= 5 * 100 * 4
    assert size(100000, 64, 1) == size(200000, 64, 1)
    assert size(1000, 9000, 1) >= size(1000, 8192, 1) + 2 * 1000 * 4


def test_cpu_tensors_are_refused():
    x, w = torch.randn(4, 8), torch.randn(16, 8)
    for call in (lambda: linear.linear_fwd(x, w), lambda: linear.Linear(8, 16, "gelu")(x),
                 lambda: linear.linear_bwd(x, w, torch.randn(4, 16)),
                 lambda: residual.residual_norm_fwd(x, x, pre=(None, None)),
                 lambda: residual.ResidualNorm(8)(x, x),
                 lambda: residual.residual_norm_bwd(x, x, x, x, residual.RowStats(*[None] * 4),
                                                    pre=(None, None))):
        with pytest.raises(RuntimeError, match="no CPU path"):
            call()
    with pytest.raises(ValueError, match="unknown activation"):
        linear.Linear(8, 16, "softmax")
    with pytest.raises(ValueError, match="at least one"):
        residual.ResidualNorm(8, post=False, pre=False)
