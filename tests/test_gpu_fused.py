"""GPU parity of the fused operators (w4a16_linear, w4a16_gated and their gradients)
against a plain implementation in 64 bits of the formulas in include/w4.h.

Tolerances, per element, are sums of the roundings that the header names.  With
S = sum_k |x_k w^_k| of an output and A = sum_k |x_k| * 15 * scale * s (the largest
that code times scale can be, since a kernel may sum q and z apart):
  u = 2^-11 for W^ in fp16, and 2^-11 for x * s in fp16 with AWQ      -> u S
  fp32 sums of K terms, at most one ulp (2^-23) each                  -> K 2^-23 A
  bias, activation and residual in fp32                               -> 2^-20 of their sizes
  the output's one rounding                                           -> eps / 2 |y|
An activation passes an error on with a slope of at most 1.2.  Those sums are worst
cases; the random inputs' errors in the 2-norm have no such growth with K, so the
relative 2-norm is held to the sum of the half-ulps alone (`rel`)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -11
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def w4():
    from weight_only_int4_w4_b200 import w4 as mod
    return mod


def act64(x, act):
    if act == "none":
        return x
    if act == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x / math.sqrt(2)))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


def dact64(x, act):
    if act == "none":
        return torch.ones_like(x)
    if act == "relu":
        return (x > 0).double()
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(x / math.sqrt(2))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x ** 3))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)


class Layer:
    """Quantized weights of a seeded random matrix, and W^ in 64 bits."""

    def __init__(self, w4, N, K, group=128, awq=False, seed=0, std=None, W=None):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(1000 * N + K + seed)
        if W is None:
            W = torch.randn((N, K), generator=gen, device="cuda") * (1.28 / math.sqrt(K) if std is None else std)
        self.gen, self.N, self.K, self.group = gen, N, K, group
        self.s = torch.exp(0.5 * torch.randn(K, generator=gen, device="cuda")) if awq else None
        self.w = w4.w4_quantize(W, self.s, group)
        p, sc, z = self.w
        q = torch.stack([p & 15, p >> 4], 2).view(N, K // group, group).double()
        s64 = self.s.double() if awq else torch.ones(K, device="cuda", dtype=torch.float64)
        self.What = ((q - z.double()[:, :, None]) * sc.double()[:, :, None]).view(N, K) * s64
        self.big = (15 * sc.double()).repeat_interleave(group, 1) * s64

    def randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda")

    def z64(self, X, bias):
        Z = X.double() @ self.What.t()
        return Z if bias is None else Z + bias.double()

    def z_tol(self, X, Z, awq):
        a = X.double().abs()
        return (U * (2 if awq else 1)) * (a @ self.What.abs().t()) + self.K * 2.0 ** -23 * (a @ self.big.t()) + \
            2.0 ** -20 * Z.abs()


def half_ulp(t):
    return torch.finfo(t).eps / 2


def check(got, ref, tol, rel, what):
    assert got.shape == ref.shape
    g = got.double()
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    tol = tol + half_ulp(got.dtype) * ref.abs() + torch.finfo(got.dtype).tiny * half_ulp(got.dtype) * 2 + 1e-37
    worst = float(((g - ref).abs() / tol).max())
    assert worst <= 1.0, f"{what}: worst error / tolerance {worst:.3g}"
    norm = float(ref.norm())
    if rel is not None and norm > 0:
        off = float((g - ref).norm()) / norm
        assert off <= rel + half_ulp(got.dtype), f"{what}: 2-norm error {off:.3g} over {rel + half_ulp(got.dtype):.3g}"


# (M, N, K, group): every token count at which a kernel could take another path, widths
# that end inside tiles, single rows, shallow and deep layers
SHAPES = [
    (1, 1, 128, 128), (1, 256, 256, 128), (1, 4096, 4096, 128), (1, 1001, 1152, 128), (1, 4096, 14336, 128),
    (2, 130, 384, 128), (3, 999, 4096, 128), (4, 512, 2048, 128), (5, 1000, 640, 32), (7, 33, 128, 64),
    (8, 2048, 4096, 128), (9, 264, 1024, 128), (16, 768, 14336, 128), (17, 48, 192, 64), (31, 515, 512, 128),
    (33, 128, 64, 32), (48, 2000, 4096, 128), (64, 1024, 1024, 128), (65, 640, 896, 128), (77, 1001, 1088, 64),
    (96, 16, 256, 128), (128, 384, 4096, 128), (129, 130, 640, 32), (200, 1002, 448, 64), (209, 256, 128, 128),
    (256, 1024, 2048, 128), (300, 70, 1152, 128), (513, 776, 512, 128), (1030, 1250, 384, 64), (2048, 2048, 1024, 128),
]
KIN = 0.2  # size of the biases


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_linear(w4, i, shape):
    M, N, K, group = shape
    awq, act, dt = i % 3 == 1, ACTS[i % 5], (torch.bfloat16, torch.float16)[i % 2]
    odt = (dt, torch.float32, torch.bfloat16, torch.float16)[(i // 2) % 4]
    L = Layer(w4, N, K, group, awq, i)
    X = L.randn(M, K).to(dt)
    bias = L.randn(N) * KIN if i % 4 != 2 else None
    res = (L.randn(M, N) * 3).to(odt) if i % 3 != 0 else None
    save = i % 2 == 0
    r = w4.w4a16_linear(X, *L.w, awq_s=L.s, bias=bias, act=act, residual=res, out_dtype=odt, save_preact=save, group=group)
    Y, Z = r if save else (r, None)
    assert Y.dtype == odt
    Zr = L.z64(X, bias)
    tz = L.z_tol(X, Zr, awq)
    if bias is not None:
        tz = tz + 2.0 ** -20 * bias.abs().double()
    Yr = act64(Zr, act)
    tol = 1.2 * tz + 2.0 ** -20 * Yr.abs()
    if res is not None:
        Yr = Yr + res.double()
        tol = tol + 2.0 ** -23 * res.double().abs()
    rel = 1.2 * U * (2 if awq else 1)
    check(Y, Yr, tol, rel, f"linear {shape} {act}")
    if save:
        assert Z.dtype == dt
        check(Z, Zr, tz, rel, f"preact {shape}")
    assert w4.w4_device_error() == 0


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_gated(w4, i, shape):
    M, F, K, group = shape
    awq, act, dt = i % 3 == 2, ACTS[(i + 2) % 5], (torch.bfloat16, torch.float16)[(i // 2) % 2]
    odt = (dt, torch.float32, dt, torch.bfloat16)[i % 4]
    L = Layer(w4, 2 * F, K, group, awq, i)
    X = L.randn(M, K).to(dt)
    bias = L.randn(2 * F) * KIN if i % 2 else None
    save = i % 3 == 0
    r = w4.w4a16_gated(X, *L.w, awq_s=L.s, bias=bias, act=act, out_dtype=odt, save_preact=save, group=group)
    H, Z = r if save else (r, None)
    Zr = L.z64(X, bias)
    tz = L.z_tol(X, Zr, awq)
    if bias is not None:
        tz = tz + 2.0 ** -20 * bias.abs().double()
    G, Up, tg, tu = Zr[:, :F], Zr[:, F:], tz[:, :F], tz[:, F:]
    Ar = act64(G, act)
    Hr = Ar * Up
    tol = Ar.abs() * tu + 1.2 * tg * Up.abs() + 1.2 * tg * tu + 2.0 ** -20 * Hr.abs()
    rel = 3 * U * (2 if awq else 1)
    check(H, Hr, tol, rel, f"gated {shape} {act}")
    if save:
        check(Z, Zr, tz, rel, f"gated preact {shape}")
    assert w4.w4_device_error() == 0


def grad_ref(L, dY, Z, act, gated):
    dY = dY.double()
    if not gated:
        dZ = dY if Z is None else dY * dact64(Z.double(), act)
        return dZ, dZ.abs() + 2.0 ** -7 * dY.abs()
    F = L.N // 2
    G, Up = Z[:, :F].double(), Z[:, F:].double()
    dZ = torch.cat([dY * Up * dact64(G, act), dY * act64(G, act)], 1)
    # an activation or its slope near a zero crossing is exact to an ulp of 1, not of itself
    return dZ, dZ.abs() + 2.0 ** -7 * torch.cat([dY * Up, dY], 1).abs()


def check_grad(w4, L, dY, Z, act, gated, group, dbias, odt, what, rel=True):
    M = dY.shape[0]
    if gated:
        r = w4.w4a16_gated_grad(dY, Z, *L.w, awq_s=L.s, act=act, dbias=dbias, out_dtype=odt, group=group)
    else:
        r = w4.w4a16_linear_grad(dY, *L.w, awq_s=L.s, preact=Z, act=act, dbias=dbias, out_dtype=odt, group=group)
    dX, db = r if dbias else (r, None)
    dZ, size = grad_ref(L, dY, Z, act, gated)
    # dZ and W^ to fp16, activations to 2^-13 of `size`, N fp32 sums
    tol = (2 * U + 2.0 ** -13 + L.N * 2.0 ** -23) * (size @ L.What.abs())
    check(dX, dZ @ L.What, tol, 2.2 * U if rel else None, what)
    if dbias:
        assert db.dtype == torch.float32 and db.shape == (L.N,)
        check(db, dZ.sum(0), (2.0 ** -13 + M * 2.0 ** -23) * size.sum(0), None, what + " dbias")
    assert w4.w4_device_error() == 0


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_linear_grad(w4, i, shape):
    M, N, K, group = shape
    act, dt = ACTS[(i + 1) % 5], (torch.bfloat16, torch.float16)[i % 2]
    L = Layer(w4, N, K, group, i % 3 == 0, i)
    size = torch.exp(L.randn(M, 1) - (4 if dt == torch.float16 else 9))
    dY = (L.randn(M, N) * size).to(dt)
    Z = (L.randn(M, N) * 1.4).to(dt) if act != "none" else None
    odt = (dt, torch.float32, torch.bfloat16)[i % 3]
    check_grad(w4, L, dY, Z, act, False, group, i % 2 == 0, odt, f"linear_grad {shape} {act}")


@pytest.mark.parametrize("i,shape", list(enumerate(SHAPES)))
def test_gated_grad(w4, i, shape):
    M, F, K, group = shape
    act, dt = ACTS[(i + 2) % 5], (torch.bfloat16, torch.float16)[(i // 2) % 2]
    L = Layer(w4, 2 * F, K, group, i % 3 == 1, i)
    size = torch.exp(L.randn(M, 1) - (4 if dt == torch.float16 else 9))
    dH = (L.randn(M, F) * size).to(dt)
    Z = (L.randn(M, 2 * F) * 1.4).to(dt)
    check_grad(w4, L, dH, Z, act, True, group, i % 2 == 1, (dt, torch.float32)[i % 2], f"gated_grad {shape} {act}")


@pytest.mark.parametrize("gated,N", [(False, 16392), (False, 33001), (True, 2 * 16400), (True, 2 * 20003), (False, 65600),
                                     (False, 65537), (True, 2 * 65543)])
def test_grad_of_wide_layers(w4, gated, N):
    """Widths of every staging path: clusters of CTAs with one and two vectors a thread, rows
    on 16 bytes or not, and rows longer than a cluster's slices."""
    M, K = 21, 64
    L = Layer(w4, N, K, group=64, seed=7)
    dY = (L.randn(M, N // 2 if gated else N) * 1e-3).to(torch.bfloat16)
    Z = (L.randn(M, N) * 1.4).to(torch.bfloat16)
    check_grad(w4, L, dY, Z, "silu", gated, 64, True, torch.bfloat16, f"wide gradient {gated} {N}")


@pytest.mark.parametrize("gated", [False, True])
def test_gradient_against_differences(w4, gated):
    """<dX, V> against the central difference of f(X) = <dY, layer(X)> along V, in 64 bits.
    The direction's derivative sums M K products of dX, each off by the gradient's own
    roundings: at most (2^-11 + 2^-11 + 2^-13) of |dX| in the 2-norm (fp32 output, random
    signs), and Z is the library's own, rounded to 16 bits (2^-11), which the second
    derivative of the activations (at most 1.2 of |z| <= 8 here) carries on."""
    M, F, K = 24, 160, 256
    N = 2 * F if gated else F
    L = Layer(w4, N, K, seed=5)
    X = L.randn(M, K).to(torch.float16)
    bias = L.randn(N) * KIN
    dY = L.randn(M, F).to(torch.float16)
    fwd, act = (w4.w4a16_gated, "silu") if gated else (w4.w4a16_linear, "gelu_tanh")
    _, Z = fwd(X, *L.w, bias=bias, act=act, save_preact=True)
    if gated:
        dX = w4.w4a16_gated_grad(dY, Z, *L.w, act=act, out_dtype=torch.float32)
    else:
        dX = w4.w4a16_linear_grad(dY, *L.w, preact=Z, act=act, out_dtype=torch.float32)

    def f(x):
        Zr = x @ L.What.t() + bias.double()
        Y = act64(Zr[:, :F], act) * Zr[:, F:] if gated else act64(Zr, act)
        return (dY.double() * Y).sum()

    for k in range(4):
        V = L.randn(M, K).double()
        h = 1e-5
        slope = float((f(X.double() + h * V) - f(X.double() - h * V)) / (2 * h))
        tol = float(dX.double().norm()) * float(V.norm()) / math.sqrt(M * K) * 4 * 3 * U * 2
        assert abs(float((dX.double() * V).sum()) - slope) <= tol


def test_block_as_used(w4):
    """A feed-forward block and its gradient, the operators one after another: gated, down
    projection into the residual stream, and back."""
    M, K, F = 130, 512, 704
    up, down = Layer(w4, 2 * F, K, seed=1), Layer(w4, K, F, group=64, seed=2)
    X = up.randn(M, K).to(torch.bfloat16)
    H, Z = w4.w4a16_gated(X, *up.w, save_preact=True)
    Y = w4.w4a16_linear(H, *down.w, residual=X, group=64)
    dY = (up.randn(M, K) * 1e-3).to(torch.bfloat16)
    dH = w4.w4a16_linear_grad(dY, *down.w, group=64)
    dX = w4.w4a16_gated_grad(dH, Z, *up.w)
    Zr = X.double() @ up.What.t()
    Hr = act64(Zr[:, :F], "silu") * Zr[:, F:]
    Yr = X.double() + Hr @ down.What.t()
    dHr = dY.double() @ down.What
    dZr = torch.cat([dHr * Zr[:, F:] * dact64(Zr[:, :F], "silu"), dHr * act64(Zr[:, :F], "silu")], 1)
    dXr = dZr @ up.What
    # every stage rounds to bf16 (2^-8 at most) and multiplies by fp16 weights; Z enters twice
    assert float((Y.double() - Yr).norm() / Yr.norm()) <= 2 * 2.0 ** -8 + 4 * U
    assert float((dX.double() - dXr).norm() / dXr.norm()) <= 4 * 2.0 ** -8 + 4 * U


@pytest.mark.parametrize("M", [1, 16, 40, 150])
def test_in_place_residual(w4, M):
    L = Layer(w4, 520, 1024)
    X = L.randn(M, 1024).to(torch.bfloat16)
    R = L.randn(M, 520).to(torch.bfloat16)
    want = w4.w4a16_linear(X, *L.w, residual=R)
    got = w4.w4a16_linear(X, *L.w, residual=R, out=R)
    assert got.data_ptr() == R.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("M", [1, 8, 33, 64, 100, 333])
def test_same_bits_again_and_rows_behind_left_alone(w4, M):
    """Repeated calls give the same bits (sums do not depend on which block ends last), and
    nothing is written before or behind an output."""
    F, K = 531, 2048
    L = Layer(w4, 2 * F, K, awq=True)
    X = L.randn(M, K).to(torch.bfloat16)
    dH = L.randn(M, F).to(torch.bfloat16)
    buf = torch.full((M * F + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    H = buf[256:256 + M * F].view(M, F)
    gbuf = torch.full((M * K + 512,), 7.0, dtype=torch.bfloat16, device="cuda")
    dX = gbuf[256:256 + M * K].view(M, K)
    runs = []
    for _ in range(3):
        _, Z = w4.w4a16_gated(X, *L.w, awq_s=L.s, out=H, save_preact=True)
        _, db = w4.w4a16_gated_grad(dH, Z, *L.w, awq_s=L.s, out=dX, dbias=True)
        runs.append((H.clone(), Z, dX.clone(), db))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))
    for b, n in ((buf, M * F), (gbuf, M * K)):
        assert (b[:256] == 7).all() and (b[256 + n:] == 7).all()


@pytest.mark.parametrize("op", ["linear", "gated", "linear_grad", "gated_grad"])
def test_same_bits_under_load(w4, op):
    """Many tiles per block, several runs with nothing between them: the same bits each time
    (a buffer handed on too early shows here), and the 2-norm of the error."""
    M, N, K = 1024, 8192, 4096
    L = Layer(w4, N, K, seed=9)
    if op in ("linear", "gated"):
        X = L.randn(M, K).to(torch.bfloat16)
        call = (lambda: w4.w4a16_linear(X, *L.w)) if op == "linear" else (lambda: w4.w4a16_gated(X, *L.w))
        Z = L.z64(X, None)
        ref = Z if op == "linear" else act64(Z[:, :N // 2], "silu") * Z[:, N // 2:]
    else:
        gated = op == "gated_grad"
        dY = L.randn(M, N // 2 if gated else N).to(torch.bfloat16)
        Z = L.randn(M, N).to(torch.bfloat16)
        call = (lambda: w4.w4a16_gated_grad(dY, Z, *L.w)) if gated else \
            (lambda: w4.w4a16_linear_grad(dY, *L.w, preact=Z, act="silu"))
        ref = grad_ref(L, dY, Z, "silu", gated)[0] @ L.What
    outs = [call() for _ in range(8)]
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    assert float((outs[0].double() - ref).norm() / ref.norm()) <= 3 * U + half_ulp(torch.bfloat16)


@pytest.mark.parametrize("M", [2, 20, 90])
def test_sizes_far_from_one(w4, M):
    """Weights from subnormal fp16 scales to the largest, groups of very different scale in
    one row, bf16 activations and gradients far outside fp16's range, zero tokens."""
    N, K = 192, 512
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    W = torch.randn((N, K), generator=gen, device="cuda")
    W *= torch.exp2(torch.randint(-12, 13, (N, 1), generator=gen, device="cuda").float())
    W *= torch.exp2(torch.randint(-4, 3, (N, K // 128), generator=gen, device="cuda").float()).repeat_interleave(128, 1)
    W[0] = 1e5 * torch.sign(W[0])
    W[1] = 2e-6 * torch.sign(W[1])
    W[2] = 0
    L = Layer(w4, N, K, W=W)
    X = L.randn(M, K) * torch.exp2(torch.randint(-60, 40, (M, 1), generator=gen, device="cuda").float())
    X[M - 1] = 0
    X = X.to(torch.bfloat16)
    Y = w4.w4a16_linear(X, *L.w, out_dtype=torch.float32)
    Zr = L.z64(X, None)
    check(Y, Zr, L.z_tol(X, Zr, False), None, "linear of far sizes")
    dY = L.randn(M, N) * torch.exp2(torch.randint(-60, 40, (M, 1), generator=gen, device="cuda").float())
    dY[0] = 0
    check_grad(w4, L, dY.to(torch.bfloat16), None, "none", False, 128, True, torch.float32, "gradient of far sizes", rel=False)


@pytest.mark.parametrize("M", [3, 12, 70])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_token_stays_alone(w4, M, bad):
    F, K = 200, 384
    L = Layer(w4, 2 * F, K)
    X = L.randn(M, K).to(torch.bfloat16)
    dH = L.randn(M, F).to(torch.bfloat16)
    H, Z = w4.w4a16_gated(X, *L.w, save_preact=True)
    dX = w4.w4a16_gated_grad(dH, Z, *L.w)
    X2, dH2 = X.clone(), dH.clone()
    X2[1, 5] = bad
    dH2[1, 7] = bad
    H2 = w4.w4a16_gated(X2, *L.w)
    dX2 = w4.w4a16_gated_grad(dH2, Z, *L.w)
    rest = [m for m in range(M) if m != 1]
    assert torch.equal(H2[rest], H[rest]) and torch.equal(dX2[rest], dX[rest])
    assert not torch.isfinite(H2[1]).any() and not torch.isfinite(dX2[1]).any()


def test_other_stream_shared_workspace_and_graph(w4):
    """One workspace for all four operators in turn, on a stream that is not the current one;
    then the sequence captured in two graphs and replayed, one after the other, on new inputs."""
    M, F, K = 40, 300, 1024
    L = Layer(w4, 2 * F, K)
    X = L.randn(M, K).to(torch.bfloat16)
    R = L.randn(M, 2 * F).to(torch.bfloat16)
    dH = L.randn(M, F).to(torch.bfloat16)

    def all_four(stream=None, ws=None):
        H, Z = w4.w4a16_gated(X, *L.w, save_preact=True, stream=stream, ws=ws)
        Y = w4.w4a16_linear(X, *L.w, residual=R, act="gelu", stream=stream, ws=ws)
        dX, db = w4.w4a16_gated_grad(dH, Z, *L.w, dbias=True, stream=stream, ws=ws)
        dX2 = w4.w4a16_linear_grad(R, *L.w, preact=Z, act="silu", stream=stream, ws=ws)
        return H, Z, Y, dX, db, dX2

    want = all_four()
    need = max(w4.w4a16_gated_workspace_size(M, F, K), w4.w4a16_linear_workspace_size(M, 2 * F, K),
               w4.w4a16_gated_grad_workspace_size(M, F, K), w4.w4a16_linear_grad_workspace_size(M, 2 * F, K))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for w in (ws, None):
        got = all_four(side, w)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert not ws[:128 * 1024].any()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = all_four()
        graphs.append((g, out))
    X.copy_(L.randn(M, K))
    dH.copy_(L.randn(M, F))
    want = all_four()
    for _ in range(2):
        for g, out in graphs:
            g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("M", [4, 32, 96])
def test_results_on_another_stream_are_not_written_over(w4, M):
    """Kernels still queued on the current stream write memory that they gave back: results on
    another stream do not lie there."""
    F = 256
    L = Layer(w4, 2 * F, 256)
    X = L.randn(M, 256).to(torch.bfloat16)
    dH = L.randn(M, F).to(torch.bfloat16)

    def call(stream):
        H, Z = w4.w4a16_gated(X, *L.w, save_preact=True, stream=stream)
        Y, Z2 = w4.w4a16_linear(X, *L.w, act="silu", save_preact=True, stream=stream)
        dX, db = w4.w4a16_gated_grad(dH, Z, *L.w, dbias=True, stream=stream)
        return H, Z, Y, Z2, dX, db

    want = call(None)
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    given_back = [torch.empty_like(t) for t in want]
    torch.cuda._sleep(40_000_000)  # some 20 ms
    for t in given_back:
        t.fill_(7)
    del given_back, t
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_offsets_past_32_bits(w4):
    """More than 2^31 output elements: the last tokens' outputs and gradients."""
    M, N, K = 75000, 28704, 64
    L = Layer(w4, N, K, group=64)
    X = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 74814, M - 1], device="cuda")
    X[rows] = L.randn(3, K).to(torch.bfloat16)
    Y = w4.w4a16_linear(X, *L.w, group=64)
    Zr = L.z64(X[rows], None)
    check(Y[rows], Zr, L.z_tol(X[rows], Zr, False), U, "linear past 32 bits")
    assert not Y[1].any() and not Y[M - 2].any()
    dX = w4.w4a16_linear_grad(Y, *L.w, group=64)
    ref = Y[rows].double() @ L.What
    check(dX[rows], ref, (2 * U + N * 2.0 ** -23) * (Y[rows].double().abs() @ L.What.abs()), 2 * U, "gradient past 32 bits")
    del X, Y, dX
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [3, 20, 90])
def test_negative_scales(w4, M):
    """Scales of either sign, and rows that have only negative ones: as precise as positive ones."""
    N, K = 264, 768
    L = Layer(w4, N, K)
    p, sc, z = L.w
    sign = torch.ones_like(sc)
    sign[::2] = -1
    sign[1::4, ::2] = -1
    L.w = (p, sc * sign, z)
    L.What = L.What * sign.double().repeat_interleave(128, 1)
    X = L.randn(M, K).to(torch.float16)
    Zr = L.z64(X, None)
    Y = w4.w4a16_linear(X, *L.w, out_dtype=torch.float32)
    check(Y, Zr, L.z_tol(X, Zr, False), U, f"negative scales M={M}")
    dY = L.randn(M, N).to(torch.float16)
    check_grad(w4, L, dY, None, "none", False, 128, True, torch.float32, f"negative scales, gradient M={M}")


def test_weights_past_32_bits(w4):
    """More than 2^31 bytes of codes (and 2^32 weights): outputs of the first and last rows, and
    the gradient that comes from them."""
    N, K = 150016, 32768
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    p = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    sc = (torch.rand((N, K // 128), generator=gen, device="cuda") * 0.01 + 0.001).half()
    z = torch.randint(0, 16, (N, K // 128), generator=gen, device="cuda").half()
    rows = torch.tensor([0, 1, N // 2 - 1, N // 2, 131071, 131072, N - 2, N - 1], device="cuda")
    q = torch.stack([p[rows] & 15, p[rows] >> 4], 2).view(len(rows), K // 128, 128).double()
    What = ((q - z[rows].double()[:, :, None]) * sc[rows].double()[:, :, None]).view(len(rows), K)
    big = (15 * sc[rows].double()).repeat_interleave(128, 1)
    for M in (2, 20, 70):
        X = torch.randn((M, K), generator=gen, device="cuda").to(torch.bfloat16)
        ref = X.double() @ What.t()
        tol = U * (X.double().abs() @ What.abs().t()) + K * 2.0 ** -23 * (X.double().abs() @ big.t())
        Y = w4.w4a16_linear(X, p, sc, z, out_dtype=torch.float32)
        check(Y[:, rows], ref, tol, U, f"weights past 32 bits M={M}")
        dY = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
        dY[:, rows] = torch.randn((M, len(rows)), generator=gen, device="cuda").to(torch.bfloat16)
        dref = dY[:, rows].double() @ What
        dX = w4.w4a16_linear_grad(dY, p, sc, z, out_dtype=torch.float32)
        check(dX, dref, (2 * U + N * 2.0 ** -23) * (dY[:, rows].double().abs() @ big), 2 * U,
              f"gradient of weights past 32 bits M={M}")
    H, Z = w4.w4a16_gated(X, p, sc, z, act="none", save_preact=True)
    f = torch.tensor([0, N // 2 - 1], device="cuda")
    (G, tG), (Up, tU) = [(ref[:, i], tol[:, i]) for i in ([0, 2], [3, 7])]
    check(Z[:, f], G, tG, U, "gate, weights past 32 bits")
    check(Z[:, N // 2 + f], Up, tU, U, "up, weights past 32 bits")
    check(H[:, f], G * Up, G.abs() * tU + Up.abs() * tG + tG * tU + 2.0 ** -23 * (G * Up).abs(), None,
          "gated, weights past 32 bits")
    del p, X, Y, H, Z, dY, dX
    torch.cuda.empty_cache()


def test_calls_from_two_threads_on_two_streams(w4):
    """Two host threads, a stream each, call every kernel at the same time on the same weights:
    the same bits as one call alone."""
    import threading
    F, K = 1000, 1024
    L = Layer(w4, 2 * F, K)
    Xs = [L.randn(M, K).to(torch.bfloat16) for M in (1, 5, 24, 64, 150, 400)]
    dHs = [L.randn(X.shape[0], F).to(torch.bfloat16) for X in Xs]

    def once(X, dH):
        H, Z = w4.w4a16_gated(X, *L.w, save_preact=True)
        Y = w4.w4a16_linear(X, *L.w, act="silu")
        dX, db = w4.w4a16_gated_grad(dH, Z, *L.w, dbias=True)
        return H, Z, Y, dX, db

    want = [once(X, dH) for X, dH in zip(Xs, dHs)]
    torch.cuda.synchronize()
    wrong = []

    def work(order):
        try:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                for _ in range(15):
                    got = [(i, once(Xs[i], dHs[i])) for i in order]
                    side.synchronize()
                    wrong.extend(i for i, g in got if not all(torch.equal(a, b) for a, b in zip(g, want[i])))
        except Exception as e:  # seen by the test
            wrong.append(e)

    ts = [threading.Thread(target=work, args=(o,)) for o in ([0, 1, 2, 3, 4, 5], [5, 3, 1, 4, 2, 0])]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong, wrong[:3]


def test_refusals(w4):
    L = Layer(w4, 256, 256)
    X = L.randn(4, 256).to(torch.bfloat16)
    Y = torch.empty((4, 256), dtype=torch.bfloat16, device="cuda")
    p, sc, z = L.w
    with pytest.raises(ValueError):
        w4.w4a16_linear(X.float(), *L.w)
    with pytest.raises(ValueError):
        w4.w4a16_linear(X[:, ::2], *L.w)
    with pytest.raises(ValueError):
        w4.w4a16_linear(X[:, :128].contiguous(), *L.w)
    with pytest.raises(ValueError):
        w4.w4a16_linear(X, *L.w, act="swish")
    with pytest.raises(ValueError):
        w4.w4a16_linear(X, *L.w, bias=torch.zeros(255, device="cuda"))
    with pytest.raises(ValueError):
        w4.w4a16_linear(X, *L.w, bias=torch.zeros(256))
    with pytest.raises(ValueError):
        w4.w4a16_linear(X, *L.w, residual=Y.float())
    with pytest.raises(ValueError):
        w4.w4a16_linear(X, *L.w, group=64)
    with pytest.raises(ValueError):
        w4.w4a16_linear(X, *L.w, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        w4.w4a16_gated(X, p[:255], sc[:255], z[:255])
    with pytest.raises(ValueError):
        w4.w4a16_gated_grad(X, Y, *L.w)  # dH has 256 channels, the block 128
    with pytest.raises(w4.W4Error) as e:
        w4.w4a16_linear_grad(Y, *L.w, act="silu")
    assert e.value.status == w4.W4_ERR_INVALID_ARG and "pre-activations" in str(e.value)
    with pytest.raises(w4.W4Error) as e:
        w4.w4a16_linear(X, *L.w, out=X)
    assert e.value.status == w4.W4_ERR_INVALID_ARG and "overlaps" in str(e.value)
    with pytest.raises(w4.W4Error) as e:
        w4.w4a16_linear_grad(X, *L.w, ws=torch.zeros(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == w4.W4_ERR_INVALID_ARG and "workspace" in str(e.value)
    with pytest.raises(w4.W4Error):
        w4.w4a16_linear(X[:0], *L.w)


@pytest.mark.parametrize("M", [1, 8, 9, 65])
def test_in_place_over_the_activations_is_refused(w4, M):
    """h += h . W^T written over h itself: h is read as X while it is written."""
    L = Layer(w4, 256, 256)
    h = L.randn(M, 256).to(torch.bfloat16)
    keep = h.clone()
    with pytest.raises(w4.W4Error) as e:
        w4.w4a16_linear(h, *L.w, residual=h, out=h)
    assert e.value.status == w4.W4_ERR_INVALID_ARG and "overlaps" in str(e.value)
    assert torch.equal(h, keep)


@pytest.mark.parametrize("M", [9, 12, 16, 17, 36, 40, 48, 49, 64])
@pytest.mark.parametrize("K,tiles,less", [(128, 2, 0), (128, 4, 0), (128, 7, 37), (128, 18, 5), (256, 4, 0), (256, 9, 11),
                                          (384, 5, 1), (640, 4, 0), (640, 6, 3), (1152, 3, 0)])
@pytest.mark.parametrize("gated", [False, True])
def test_small_batches_on_wide_shallow_layers(w4, gated, K, tiles, less, M):
    """Several tiles to a block's range of rows (148 blocks), each of few groups: the ring of
    codes goes on across tiles, the accumulators alternate, the places of row factors come
    round again.  Three runs with nothing between them give the same bits."""
    N = 148 * 128 * tiles - 2 * less
    L = Layer(w4, N, K, seed=M)
    X = L.randn(M, K).to(torch.bfloat16)
    bias = L.randn(N) * KIN if less else None
    if gated:
        runs = [w4.w4a16_gated(X, *L.w, bias=bias, out_dtype=torch.float32) for _ in range(3)]
    else:
        runs = [w4.w4a16_linear(X, *L.w, bias=bias, out_dtype=torch.float32) for _ in range(3)]
    assert w4.w4_device_error() == 0
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])
    Zr = L.z64(X, bias)
    tz = L.z_tol(X, Zr, False) + (0 if bias is None else 2.0 ** -20 * bias.abs().double())
    if not gated:
        return check(runs[0], Zr, tz, 1.2 * U, f"linear {M} x {K} -> {N}")
    F = N // 2
    A, Up, tg, tu = act64(Zr[:, :F], "silu"), Zr[:, F:], tz[:, :F], tz[:, F:]
    check(runs[0], A * Up, A.abs() * tu + 1.2 * tg * Up.abs() + 1.2 * tg * tu + 2.0 ** -20 * (A * Up).abs(), 3 * U,
          f"gated {M} x {K} -> 2 x {F}")


def test_calls_from_threads_on_one_stream(w4):
    """Three host threads call on the same stream, with the binding's own workspace: the same bits
    as one call alone."""
    import threading
    F, K = 1000, 1024
    L = Layer(w4, 2 * F, K)
    Xs = [L.randn(M, K).to(torch.bfloat16) for M in (24, 64, 150, 400)]
    dHs = [L.randn(X.shape[0], F).to(torch.bfloat16) for X in Xs]

    def once(i):
        H, Z = w4.w4a16_gated(Xs[i], *L.w, save_preact=True)
        Y = w4.w4a16_linear(Xs[i], *L.w, act="silu")
        dX, db = w4.w4a16_gated_grad(dHs[i], Z, *L.w, dbias=True)
        return H, Z, Y, dX, db

    want = [once(i) for i in range(4)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    wrong = []

    def work(order):
        try:
            with torch.cuda.stream(side):
                for _ in range(25):
                    got = [(i, once(i)) for i in order]
                    wrong.extend(i for i, g in got if not all(torch.equal(a, b) for a, b in zip(g, want[i])))
        except Exception as e:  # seen by the test
            wrong.append(e)

    ts = [threading.Thread(target=work, args=(o,)) for o in ([0, 1, 2, 3], [3, 2, 1, 0], [1, 3, 0, 2])]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not wrong, wrong[:3]


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [3, 20, 90])
def test_activations_of_far_pre_activations(w4, M, act):
    """Pre-activations up to 2^68, whose square is past fp32, forward, and up to 2^100 in the
    gradients: an activation is then z or 0 and its slope 1 or 0, never 0 times infinity."""
    N, K = 192, 256
    F = N // 2
    gen = torch.Generator(device="cuda")
    gen.manual_seed(11)
    W = torch.randn((N, K), generator=gen, device="cuda") * (1.28 / math.sqrt(K))
    W[F:] *= 2.0 ** -12  # so that act(G) U stays in range
    L = Layer(w4, N, K, W=W)
    X = (L.randn(M, K) * 2.0 ** 66).to(torch.bfloat16)
    Zr = L.z64(X, None)
    assert float(Zr[:, :F].abs().median()) > 2.0 ** 64
    tz = L.z_tol(X, Zr, False)
    Y = w4.w4a16_linear(X, *L.w, act=act, out_dtype=torch.float32)
    check(Y, act64(Zr, act), 1.2 * tz + 2.0 ** -20 * act64(Zr, act).abs(), 1.2 * U, f"linear {act}")
    H = w4.w4a16_gated(X, *L.w, act=act, out_dtype=torch.float32)
    A, Up, tg, tu = act64(Zr[:, :F], act), Zr[:, F:], tz[:, :F], tz[:, F:]
    check(H, A * Up, A.abs() * tu + 1.2 * tg * Up.abs() + 1.2 * tg * tu + 2.0 ** -20 * (A * Up).abs(), 3 * U, f"gated {act}")
    Z = L.randn(M, N) * torch.exp2(torch.randint(0, 101, (M, N), generator=gen, device="cuda").float())
    Z[:, F:] = L.randn(M, F)
    Z = Z.to(torch.bfloat16)
    dY = (L.randn(M, N) * 1e-3).to(torch.bfloat16)
    check_grad(w4, L, dY, Z, act, False, 128, True, torch.float32, f"linear gradient {act}", rel=False)
    check_grad(w4, L, dY[:, :F].contiguous(), Z, act, True, 128, True, torch.float32, f"gated gradient {act}", rel=False)


@pytest.mark.parametrize("gated,N", [(False, 65600), (False, 65537), (True, 2 * 65543)])
def test_far_pre_activations_of_the_widest_layers(w4, gated, N):
    """The same in the gradients of layers wider than a cluster's slices."""
    M, K = 5, 64
    L = Layer(w4, N, K, group=64, seed=8)
    Z = L.randn(M, N) * torch.exp2(torch.randint(0, 101, (M, N), generator=L.gen, device="cuda").float())
    if gated:
        Z[:, N // 2:] = L.randn(M, N // 2)
    dY = (L.randn(M, N // 2 if gated else N) * 1e-3).to(torch.bfloat16)
    for act in ("silu", "gelu_tanh"):
        check_grad(w4, L, dY, Z.to(torch.bfloat16), act, gated, 64, True, torch.float32, f"wide gradient {gated} {act}", rel=False)


@pytest.mark.parametrize("M", [1, 8, 9, 33, 64, 65])
@pytest.mark.parametrize("N,K,group", [(1, 128, 128), (2, 256, 128), (3, 64, 32), (7, 384, 128), (9, 128, 64), (17, 128, 128),
                                       (4096, 14336, 128)])
def test_narrow_and_deep_layers(w4, M, N, K, group):
    """A handful of outputs, or clusters that share a range of rows with several tiles: every
    operator, with residual in place, biases and saved pre-activations."""
    L = Layer(w4, 2 * N if N < 4096 else N, K, group, seed=M)
    F = L.N // 2
    X = L.randn(M, K).to(torch.bfloat16)
    bias = L.randn(L.N) * KIN
    Zr = L.z64(X, bias)
    tz = L.z_tol(X, Zr, False) + 2.0 ** -20 * bias.abs().double()
    R = L.randn(M, L.N)
    keep = R.double()
    Y, Z = w4.w4a16_linear(X, *L.w, bias=bias, act="gelu", residual=R, out=R, save_preact=True, group=group)
    Yr = act64(Zr, "gelu") + keep
    check(Y, Yr, 1.2 * tz + 2.0 ** -20 * act64(Zr, "gelu").abs() + 2.0 ** -23 * keep.abs(), None, "linear")
    check(Z, Zr, tz, None, "linear preact")
    H, Z = w4.w4a16_gated(X, *L.w, bias=bias, save_preact=True, group=group)
    A, Up, tg, tu = act64(Zr[:, :F], "silu"), Zr[:, F:], tz[:, :F], tz[:, F:]
    check(H, A * Up, A.abs() * tu + 1.2 * tg * Up.abs() + 1.2 * tg * tu + 2.0 ** -20 * (A * Up).abs(), None, "gated")
    check(Z, Zr, tz, None, "gated preact")
    dY = L.randn(M, L.N).to(torch.bfloat16)
    check_grad(w4, L, dY, Z, "gelu_tanh", False, group, True, torch.float32, "linear gradient")
    check_grad(w4, L, dY[:, :F].contiguous(), Z, "silu", True, group, True, torch.bfloat16, "gated gradient")


@pytest.mark.parametrize("M", [4, 40, 120])
def test_two_graphs_replayed_at_the_same_time(w4, M):
    """Graphs of the same calls on two streams, replayed together: each has a workspace of its own."""
    F, K = 1000, 2048
    L = Layer(w4, 2 * F, K)
    graphs = []
    for i in range(2):
        X = L.randn(M, K).to(torch.bfloat16)
        dH = L.randn(M, F).to(torch.bfloat16)

        def calls():
            H, Z = w4.w4a16_gated(X, *L.w, save_preact=True)
            Y = w4.w4a16_linear(X, *L.w, act="silu")
            dX, db = w4.w4a16_gated_grad(dH, Z, *L.w, dbias=True)
            return H, Z, Y, dX, db

        want = calls()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = calls()
        graphs.append((g, out, want, torch.cuda.Stream(), (X, dH)))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, _, _, s, _ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, out, want, _, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert w4.w4_device_error() == 0
