"""CPU checks of the fused operators' host side: every refusal happens before any
device call, and the workspace sizes of invalid shapes are 0."""
import ctypes

import pytest

from weight_only_int4_w4_b200 import build

P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
MB = 1 << 20
# fake, 16-byte aligned "device" addresses, far apart: never dereferenced (rejected first)
X, W, S, Z0, B, R, ZP, Y, D, WS = (0x10000000 * (i + 1) for i in range(10))
OK_, BAD, UNSUP = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(build.build_library())
    lib.w4a16_linear.argtypes = [P, I, I64, I64, I64, I, P, P, P, P, P, I, P, P, P, I, P, SZ, P]
    lib.w4a16_gated.argtypes = [P, I, I64, I64, I64, I, P, P, P, P, P, I, P, P, I, P, SZ, P]
    lib.w4a16_linear_grad.argtypes = [P, I, I64, I64, I64, I, P, P, P, P, P, I, P, I, P, P, SZ, P]
    lib.w4a16_gated_grad.argtypes = lib.w4a16_linear_grad.argtypes
    for f in ("linear", "gated", "linear_grad", "gated_grad"):
        fn = getattr(lib, f"w4a16_{f}_workspace_size")
        fn.argtypes, fn.restype = [I64, I64, I64], SZ
    lib.w4_last_error.restype = ctypes.c_char_p
    return lib


def linear(lib, **k):
    g = k.get
    return lib.w4a16_linear(g("X", X), g("xd", 2), g("M", 4), g("N", 256), g("K", 256), g("G", 128), g("W", W), g("S", S),
                            g("Z0", Z0), g("awq"), g("bias", B), g("act", 1), g("res", R), g("Z", ZP), g("Y", Y),
                            g("yd", 2), g("ws", WS), g("wsb", 0), None)


def gated(lib, **k):
    g = k.get
    return lib.w4a16_gated(g("X", X), g("xd", 2), g("M", 4), g("F", 128), g("K", 256), g("G", 128), g("W", W), S, Z0, None,
                           g("bias", B), g("act", 2), g("Z", ZP), g("Y", Y), g("yd", 2), g("ws", WS), g("wsb", 0), None)


def grad(lib, f="linear_grad", **k):
    g = k.get
    return getattr(lib, "w4a16_" + f)(g("X", X), g("xd", 2), g("M", 4), g("N", 256), g("K", 256), g("G", 128), g("W", W), S,
                                      Z0, None, g("Z", ZP), g("act", 2), g("Y", Y), g("yd", 2), g("db", D), g("ws", WS),
                                      g("wsb", 0), None)


BIG = 1 << 40
SHAPE_CASES = [(dict(M=0), BAD), (dict(M=-1), BAD), (dict(K=0), BAD), (dict(K=200), BAD), (dict(G=48), UNSUP),
               (dict(G=32, K=96), UNSUP), (dict(M=BIG * 2), BAD), (dict(xd=0), UNSUP), (dict(xd=9), UNSUP),
               (dict(yd=3), UNSUP), (dict(act=5), UNSUP), (dict(act=-1), UNSUP), (dict(X=None), BAD), (dict(W=None), BAD),
               (dict(Y=None), BAD), (dict(X=X + 8), BAD), (dict(Y=Y + 4), BAD), (dict(Z=ZP + 2), BAD), (dict(ws=WS + 8), BAD)]


@pytest.mark.parametrize("kw,want", SHAPE_CASES)
def test_every_entry_refuses(lib, kw, want):
    assert linear(lib, **kw) == want, lib.w4_last_error()
    assert gated(lib, **kw) == want, lib.w4_last_error()
    assert grad(lib, **kw) == want, lib.w4_last_error()
    assert grad(lib, "gated_grad", **{"N": 128, **kw}) == want, lib.w4_last_error()


def test_own_refusals(lib):
    assert linear(lib, N=0) == BAD and gated(lib, F=0) == BAD and grad(lib, N=0) == BAD
    assert gated(lib, F=1 << 31) == BAD and grad(lib, "gated_grad", N=(1 << 31) - 1) == BAD
    assert grad(lib, Z=None) == BAD and b"pre-activations" in lib.w4_last_error()
    assert grad(lib, "gated_grad", N=128, Z=None, act=0) == BAD
    assert linear(lib, bias=B + 4) == BAD and linear(lib, res=R + 2) == BAD and linear(lib, awq=B + 8) == BAD
    assert grad(lib, db=D + 4) == BAD


def test_overlaps_are_refused(lib):
    for kw in (dict(Y=X), dict(Y=X + 1024), dict(Z=X), dict(Y=W + 4096), dict(Y=S), dict(Z=Y), dict(Y=R + 16), dict(Y=WS, wsb=MB),
               dict(X=WS + 4096, wsb=MB), dict(Z=R), dict(Y=B)):
        assert linear(lib, **kw) == BAD, kw
        assert b"overlap" in lib.w4_last_error(), kw
    for kw in (dict(Y=X), dict(Y=ZP), dict(db=ZP), dict(db=Y), dict(Y=W), dict(db=X + 512)):
        assert grad(lib, **kw) == BAD, kw
        assert b"overlap" in lib.w4_last_error(), kw


def test_workspace_refused_when_short(lib):
    for f in ("linear_grad", "gated_grad"):
        n = 256 if f == "linear_grad" else 128
        need = getattr(lib, f"w4a16_{f}_workspace_size")(4, n, 256)
        assert need > 0
        for kw in (dict(ws=None), dict(wsb=need - 1)):
            assert grad(lib, f, N=n, **kw) == BAD
            assert b"workspace" in lib.w4_last_error()


def test_workspace_sizes(lib):
    for f in ("linear", "gated", "linear_grad", "gated_grad"):
        fn = getattr(lib, f"w4a16_{f}_workspace_size")
        assert fn(0, 16, 128) == fn(1, 0, 128) == fn(1, 16, 100) == fn(1, 16, 0) == fn(-1, 16, 128) == 0
        assert fn(2048, 14336, 4096) < 2 << 30


def test_only_the_residual_itself_may_be_written_in_place(lib):
    """Y may be the residual.  Another input that lies at the same address is still read while
    Y is written: refused (a square layer's h += act(h . W^T) in place, for one)."""
    for kw in (dict(X=R), dict(W=R), dict(S=R), dict(Z0=R), dict(bias=R), dict(awq=R), dict(X=R + 16), dict(ws=R, wsb=MB)):
        for M in (1, 8, 9, 64, 65):
            assert linear(lib, **{"Y": R, "M": M, **kw}) == BAD, (kw, M)
            assert b"overlaps" in lib.w4_last_error(), (kw, M)
    need = lib.w4a16_linear_workspace_size(9, 256, 256)
    assert linear(lib, Y=R, M=9, wsb=need - 1) == BAD and b"workspace too small" in lib.w4_last_error()  # no overlap
