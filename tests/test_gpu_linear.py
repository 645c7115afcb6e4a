"""moe_linear and moe_linear_backward against the float64 oracle.

Bounds (elementwise, u = 2^-23 a step of an fp32 sum, h = half a step of the type): a product of
length n is off by (n + 8) u times the sum of its terms' sizes; an activation passes that on times
its steepest slope (below 1.13) and adds its own error, 2^-19 of 1 + |z| (exponential, reciprocal and
error function are a few steps of fp32 off, the exponential's argument by |z| 2^-24); storing
rounds by h.  In the backward dZ is rounded by h as an operand of the products, not in dbias."""
import numpy as np
import pytest
import torch

from block_util import DT, HALF, U32, assert_guards, assert_within, check_replays, f64, strided
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from oracle import block as ob

pytestmark = pytest.mark.gpu
ACT_ERR = 2.0 ** -19


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield


class Proj:
    def __init__(self, M, N, K, dtype, act, bias, residual, save, pad, seed=0):
        g = torch.Generator().manual_seed(seed * 7919 + M * 31 + N * 7 + K)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.M, self.N, self.K, self.dtype, self.act, self.pad = M, N, K, dtype, act, pad
        self.NW = 2 * N if act == "swiglu" else N
        dt = DT[dtype]
        self.X, _ = strided(M, K, pad, dtype, rn(M, K))
        self.W = (rn(self.NW, K) / max(K, 1) ** 0.5).cuda().to(dt)
        self.bias = rn(self.NW).cuda() if bias else None
        self.res = strided(M, N, pad, dtype, rn(M, N))[0] if residual else None
        self.out, self.out_base = strided(M, N, pad, dtype, extra_rows=2)
        self.Z = torch.full((M + 1, self.NW), 777.0, device="cuda", dtype=dt) if save else None
        self.dY, _ = strided(M, N, pad, dtype, rn(M, N))
        self.dX, self.dX_base = strided(M, K, pad, dtype, extra_rows=2)
        self.dW = torch.full((self.NW + 1, K), 777.0, device="cuda", dtype=dt)
        self.db = torch.full((self.NW + 8,), 777.0, device="cuda")
        ld = lambda n: (n + pad) if pad else 0  # noqa: E731
        self.dims = B.make_linear_dims(M, N, K, dtype, act, ld(K), ld(N), ld(N))
        self.wf, self.nf = B.linear_workspace(self.dims, B.LINEAR_FORWARD)
        self.wb, self.nbk = B.linear_workspace(self.dims, B.LINEAR_BACKWARD)
        self.wf.fill_(0xFF)
        self.wb.fill_(0xFF)

    def forward(self):
        B.moe_linear(self.dims, self.X, self.W, self.bias, self.res, self.Z, self.out, self.wf, self.nf)

    def z_parts(self):
        """The exact z and the bound of its fp32 error."""
        X, W = f64(self.X), f64(self.W)
        b = f64(self.bias) if self.bias is not None else np.zeros(self.NW)
        z = X @ W.T + b
        return z, (self.K + 8) * U32 * (np.abs(X) @ np.abs(W).T + np.abs(b))

    def check_forward(self):
        self.forward()
        torch.cuda.synchronize()
        z, ze = self.z_parts()
        h, N = HALF[self.dtype], self.N
        res = f64(self.res) if self.res is not None else np.zeros((self.M, N))
        a = ob.activation(z, self.act)
        if self.act == "swiglu":
            g, u, ge, ue = z[:, :N], z[:, N:], ze[:, :N], ze[:, N:]
            ae = (1.13 * ge + ACT_ERR * (1 + np.abs(g))) * (np.abs(u) + ue) + np.abs(ob.activation(g, "silu")) * ue
        elif self.act in ("gelu", "silu"):
            ae = 1.13 * ze + ACT_ERR * (1 + np.abs(z))
        else:
            ae = ze
        ref = a + res
        assert_within("out", f64(self.out), ref, h * (np.abs(ref) + ae) + ae + 2 * U32 * (np.abs(a) + np.abs(res)))
        assert_guards(self.out_base, self.M, N, "out")
        if self.Z is not None:
            assert_within("Z", f64(self.Z[:self.M]), z, h * (np.abs(z) + ze) + ze)
            assert bool((self.Z[self.M] == 777.0).all())

    def backward(self, dX=True, dW=True, db=True):
        B.moe_linear_backward(self.dims, self.dY, self.X, self.W, self.Zs, self.dX if dX else None,
                              self.dW if dW else None, self.db if db else None, self.wb, self.nbk)

    def check_backward(self):
        z, _ = self.z_parts()
        self.Zs = torch.from_numpy(z).cuda().to(DT[self.dtype]) if self.act != "none" else None
        zs = f64(self.Zs) if self.Zs is not None else z
        self.backward()
        torch.cuda.synchronize()
        dY, X, W = f64(self.dY), f64(self.X), f64(self.W)
        rX, rW, rb, dz = ob.linear_backward(dY, X, W, zs, self.act)
        h, N = HALF[self.dtype], self.N
        if self.act == "swiglu":
            g, u = np.abs(zs[:, :N]), np.abs(zs[:, N:])
            de = ACT_ERR * np.concatenate([np.abs(dY) * u * (1 + g) ** 2, np.abs(dY) * (1 + g) ** 2], 1)
        elif self.act in ("gelu", "silu"):
            de = ACT_ERR * np.abs(dY) * (1 + np.abs(zs)) ** 2
        else:
            de = np.zeros_like(dz)
        op = de + (h * (np.abs(dz) + de) if self.act != "none" else 0)  # the operand as stored
        size = np.abs(dz) + op
        tX = op @ np.abs(W) + (self.NW + 8) * U32 * (size @ np.abs(W))
        tW = op.T @ np.abs(X) + (self.M + 8) * U32 * (size.T @ np.abs(X))
        assert_within("dX", f64(self.dX), rX, tX + h * (np.abs(rX) + tX))
        assert_within("dW", f64(self.dW[:self.NW]), rW, tW + h * (np.abs(rW) + tW))
        tb = de.sum(0) + (self.M + 8) * U32 * (np.abs(dz) + de).sum(0)
        assert_within("dbias", f64(self.db[:self.NW]), rb, tb)
        assert_guards(self.dX_base, self.M, self.K, "dX")
        assert bool((self.dW[self.NW] == 777.0).all()) and bool((self.db[self.NW:] == 777.0).all())
        # each gradient alone has the same bits
        want = [t.clone() for t in (self.dX, self.dW, self.db)]
        for k, t in enumerate((self.dX, self.dW, self.db)):
            t.fill_(777.0) if k else self.dX_base.fill_(777.0)
            self.backward(*[j == k for j in range(3)])
            assert torch.equal(t, want[k]), ("dX", "dW", "dbias")[k]


SIZES = [(1, 8, 8), (1, 264, 40), (1, 2048, 712), (2, 16, 4096), (3, 64, 1032), (7, 1000, 64), (16, 256, 512), (17, 520, 96),
         (31, 24, 2000), (33, 128, 136), (48, 392, 264), (64, 128, 1544), (65, 256, 320), (130, 72, 200), (255, 256, 256),
         (257, 264, 264), (300, 1000, 328), (513, 136, 72), (1000, 640, 1032), (1, 40, 8192), (129, 8, 24)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward_sizes(M, N, K, dtype):
    """Every size with two activations, bias, residual, saved z and row strides in turn."""
    n = SIZES.index((M, N, K))
    for k, act in enumerate((ob.ACTS[n % 5], ob.ACTS[(n + 3) % 5])):
        Proj(M, N, K, dtype, act, bias=(n + k) % 3 != 0, residual=(n + k) % 2 == 0, save=(n // 2 + k) % 2 == 0,
             pad=(0, 8, 24)[(n + k) % 3], seed=k).check_forward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ob.ACTS)
@pytest.mark.parametrize("bias,residual,save", [(0, 0, 0), (1, 0, 1), (0, 1, 0), (1, 1, 1)])
def test_forward_epilogues(act, bias, residual, save, dtype):
    """One row, a few rows, a split reduction and a whole grid of tiles, with every epilogue."""
    for M, N, K in ((1, 136, 256), (5, 72, 328), (300, 264, 520), (4100, 1096, 40)):
        if dtype == "f32" and M > 4000:
            M, N = 2100, 2056
        Proj(M, N, K, dtype, act, bias, residual, save, pad=8 * bias).check_forward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_backward_sizes(M, N, K, dtype):
    n = SIZES.index((M, N, K))
    for k, act in enumerate((ob.ACTS[(n + 1) % 5], ob.ACTS[(n + 4) % 5])):
        Proj(M, N, K, dtype, act, bias=False, residual=False, save=False, pad=(8, 0, 24)[(n + k) % 3], seed=k).check_backward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ob.ACTS)
def test_backward_whole_grids(act, dtype):
    """Products with enough tiles to go straight to their outputs (dX: many rows; dW: wide)."""
    Proj(4100, 72, 1928, dtype, act, False, False, False, pad=0).check_backward()
    Proj(96, 1800 if act == "swiglu" else 3600, 2312, dtype, act, False, False, False, pad=8).check_backward()


@pytest.mark.parametrize("act", ob.ACTS)
def test_backward_against_differences(act):
    """<dY, out(X + h v) - out(X - h v)> / 2 h against <dX, v>, and the same for W and bias, in fp32:
    fp32 noise 2^-20 / h of the sizes, truncation h^2."""
    p = Proj(40, 48, 56, "f32", act, True, True, True, pad=0)
    p.forward()
    p.Zs = p.Z[:40].clone()
    p.backward()
    h = 2.0 ** -7
    for var, grad in ((p.X, p.dX), (p.W, p.dW[:p.NW]), (p.bias, p.db[:p.NW])):
        v = torch.randn(var.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
        v /= v.double().norm()
        x0, val = var.clone(), []
        for s in (1, -1):
            var.copy_(x0 + s * h * v)
            p.forward()
            val.append((p.out.double() * p.dY.double()).sum().item())
        var.copy_(x0)
        size = p.dY.double().norm().item() * 4 * (1 + p.out.double().norm().item() / 40)
        if act == "relu":
            size += 4 * h ** -1 * h  # kinks: at most a few of the 1920 elements cross zero, each by h |v|
        assert abs((val[0] - val[1]) / (2 * h) - (grad.double() * v.double()).sum().item()) <= size * (h * h + 2.0 ** -20 / h)


def test_residual_may_be_the_output():
    for M, N, K in ((3, 264, 512), (200, 264, 512), (4200, 2056, 64)):
        for dtype in ("bf16", "f32"):
            p = Proj(M, N, K, dtype, "silu", True, True, False, pad=0)
            p.forward()
            want = p.out.clone()
            alias = p.res.clone()
            B.moe_linear(p.dims, p.X, p.W, p.bias, alias, None, alias, p.wf, p.nf)
            assert torch.equal(alias, want)


def test_no_rows():
    for dtype in ("bf16", "f32"):
        p = Proj(0, 264, 40, dtype, "gelu", True, False, False, pad=0)
        p.forward()
        assert_guards(p.out_base, 0, 264, "out")
        p.Zs = torch.empty(0, 264, dtype=DT[dtype], device="cuda")
        p.backward()
        assert not p.dW[:264].any() and not p.db[:264].any()
        assert bool((p.dW[264] == 777.0).all()) and bool((p.dX_base == 777.0).all())


def test_infinities_and_nans_stay_in_their_rows():
    """A row of X that holds a NaN or an infinity leaves every other row as it was."""
    for M in (5, 300, 4100):
        p = Proj(M, 1096, 72, "bf16", "silu", True, True, False, pad=0)
        p.forward()
        want = p.out.clone()
        p.X[1, 3], p.X[2, 70] = float("nan"), float("inf")
        p.forward()
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[[1, 2]] = False
        assert torch.equal(p.out[keep], want[keep]) and p.out[1].isnan().all()


@pytest.mark.parametrize("M,N,K,act", [(1, 520, 1032, "swiglu"), (40, 264, 1032, "gelu"), (300, 264, 520, "silu"), (4100, 1096, 40, "relu")])
def test_graph_replays_and_streams(M, N, K, act):
    p = Proj(M, N, K, "bf16", act, True, True, True, pad=0)
    p.forward()
    p.Zs = p.Z[:M].clone()

    def step():
        p.forward()
        p.backward()

    check_replays(step, dict(out=p.out, Z=p.Z[:M], dX=p.dX, dW=p.dW[:p.NW], db=p.db[:p.NW]))
    want = [t.clone() for t in (p.out, p.dX, p.dW, p.db)]
    qs = [Proj(M, N, K, "bf16", act, True, True, True, pad=0) for _ in range(2)]
    for q in qs:
        q.Zs = p.Zs
    torch.cuda.synchronize()
    for q in qs:
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(4):
                q.forward()
                q.backward()
    torch.cuda.synchronize()
    for q in qs:
        assert all(torch.equal(a, b) for a, b in zip((q.out, q.dX, q.dW, q.db), want))


@pytest.mark.parametrize("M", [3, 40])
def test_gelu_at_infinities(M):
    """z Phi(z) tends to z and to 0, its derivative to 1 and to 0."""
    X = torch.zeros(M, 64, device="cuda")
    X[0], X[1] = float("inf"), -float("inf")
    W = torch.full((72, 64), 0.5, device="cuda")
    dims = B.make_linear_dims(M, 72, 64, "f32", "gelu")
    ws, nb = B.linear_workspace(dims, B.LINEAR_BACKWARD)
    out, Z, db = torch.empty(M, 72, device="cuda"), torch.empty(M, 72, device="cuda"), torch.empty(72, device="cuda")
    B.moe_linear(dims, X, W, None, None, Z, out, ws, nb)
    assert (out[0] == float("inf")).all() and (out[1:] == 0).all()
    dY = torch.zeros(M, 72, device="cuda")
    dY[0], dY[1] = 3.0, 5.0
    B.moe_linear_backward(dims, dY, X, W, Z, None, None, db, ws, nb)
    assert (db == 3.0).all()


# few rows with a long reduction for dX, many rows with one for dW: products of the pair cut apart
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K,act", [(25, 1152, 232, "swiglu"), (3011, 72, 104, "relu"), (1100, 24, 1720, "gelu"), (700, 520, 16, "none")])
def test_backward_of_unequal_reductions(M, N, K, act, dtype):
    p = Proj(M, N, K, dtype, act, bias=True, residual=False, save=True, pad=8)
    p.check_backward()


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 1096), (4090, 4096, 328), (4096, 1096, 4096), (1100, 4096, 4096), (4000, 2000, 4040)])
def test_large_tiles_with_partial_stages(M, N, K):
    """Small whole numbers: every product and sum is exact, so the results are the exact ones rounded."""
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float()  # noqa: E731
    X, W, dY = ints(M, K), ints(N, K), ints(M, N)
    Xb, Wb, dYb = X.bfloat16(), W.bfloat16(), dY.bfloat16()
    out, dX, dW = torch.empty_like(dYb), torch.empty_like(Xb), torch.empty_like(Wb)
    dims = B.make_linear_dims(M, N, K, "bf16")
    wf, nf = B.linear_workspace(dims, B.LINEAR_FORWARD)
    wb, nb = B.linear_workspace(dims, B.LINEAR_BACKWARD)
    B.moe_linear(dims, Xb, Wb, None, None, None, out, wf, nf)
    B.moe_linear_backward(dims, dYb, Xb, Wb, None, dX, dW, None, wb, nb)
    assert torch.equal(out, (X @ W.t()).bfloat16())
    assert torch.equal(dX, (dY @ W).bfloat16())
    assert torch.equal(dW, (dY.t() @ X).bfloat16())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(3, 72, 64), (300, 264, 136)])
def test_relu_gradient_of_units_that_are_off(M, N, K, dtype):
    """An infinite or NaN dY where z <= 0 adds nothing to any gradient: the same bits as with zeros there."""
    p = Proj(M, N, K, dtype, "relu", True, False, False, pad=8)
    p.Zs = torch.randn(M, N, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").to(DT[dtype])
    p.Zs[0, :8] = 0.0
    off = p.Zs <= 0
    p.dY[off] = 0.0
    p.backward()
    want = [t.clone() for t in (p.dX, p.dW[:p.NW], p.db[:p.NW])]
    bad = torch.tensor([float("inf"), float("nan"), -float("inf")], device="cuda").to(DT[dtype])
    p.dY[off] = bad[torch.arange(int(off.sum()), device="cuda") % 3]
    p.backward()
    for got, ref in zip((p.dX, p.dW[:p.NW], p.db[:p.NW]), want):
        assert ref.isfinite().all() and torch.equal(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [16, 4096])
def test_gelu_keeps_its_digits(M, dtype):
    """GELU and its derivative relative to the tail Q(|z|) = Phi(-|z|), which both are made of.  With one
    column of ones as W, z is X exactly.  The tail is a reciprocal, nine multiply-adds, an exponential
    and two products, 16 roundings of 2^-24 at most, and the exponential's argument z^2 / 2 has three of its
    own: Q is off by Q (2^-20 + z^2 2^-23), and where it goes into a bf16 result by 2^-17 more (its
    polynomial is then cut at 4.7e-6).  out = max(z, 0) - |z| Q adds a rounding of 2^-24 (and that of
    the type); the derivative's z exp(-z^2 / 2) / sqrt(2 pi) three products and the exponential, and the
    sum is rounded."""
    z = torch.linspace(-12, 12, M + 1)[:M].to(DT[dtype])
    X, W = torch.zeros(M, 8, dtype=DT[dtype], device="cuda"), torch.zeros(8, 8, dtype=DT[dtype], device="cuda")
    X[:, 0], W[:, 0] = z.cuda(), 1.0
    dims = B.make_linear_dims(M, 8, 8, dtype, "gelu")
    ws, nb = B.linear_workspace(dims, B.LINEAR_FORWARD)
    out = torch.empty(M, 8, dtype=DT[dtype], device="cuda")
    B.moe_linear(dims, X, W, None, None, None, out, ws, nb)
    v = f64(z)[:, None]
    q, a = ob._phi(-np.abs(v)), np.abs(v)
    rel = 2.0 ** -20 + v * v * 2.0 ** -23
    cut = rel + (2.0 ** -17 if dtype == "bf16" else 0.0)
    ref = ob.activation(v, "gelu")
    assert_within("out", f64(out), np.repeat(ref, 8, 1), (a * q * cut + (HALF[dtype] + U32) * np.abs(ref)) * np.ones(8) + 1e-36)
    # the derivative through the bias gradient of single rows (fp32 whatever the type)
    phi = np.exp(-0.5 * v * v) / np.sqrt(2 * np.pi)
    want = ob.activation_backward(np.ones_like(v), v, "gelu")
    tol = q * rel + a * phi * (2.0 ** -21 + v * v * 2.0 ** -23) + U32 * (np.where(v < 0, q, 1.0) + a * phi) + 1e-36
    one = B.make_linear_dims(1, M, 8, dtype, "gelu")
    wb, nbb = B.linear_workspace(one, B.LINEAR_BACKWARD)
    db, dY = torch.empty(M, device="cuda"), torch.ones(1, M, dtype=DT[dtype], device="cuda")
    B.moe_linear_backward(one, dY, X[:1], torch.zeros(M, 8, dtype=DT[dtype], device="cuda"), z.cuda()[None].contiguous(),
                          None, None, db, wb, nbb)
    assert_within("derivative", f64(db)[:, None], want, tol)


# ragged last tiles: 250 of 256 rows; 136, 8 (of the first half only) and all 256 columns; 4090 x 1992 SwiGLU: 72 of 128
@pytest.mark.parametrize("M,N,K,act,bias,residual,save,alias", [
    (4090, 3976, 328, "gelu", True, True, True, False), (4090, 4096, 328, "silu", True, True, False, True),
    (3850, 3848, 1096, "relu", False, True, True, False), (4090, 3976, 320, "none", True, False, True, False),
    (4090, 1992, 328, "swiglu", True, True, True, False), (4090, 1928, 1096, "swiglu", False, True, False, True),
    (4090, 2048, 320, "swiglu", True, False, True, False),
])
def test_large_tiles_with_every_epilogue(M, N, K, act, bias, residual, save, alias):
    """X, bias and residual small whole numbers, W sixteenths of them: z is exact in fp32 (at most 4 K + 4
    sixteenths), so out is off by the activation's own error, 2^-19 of 1 + |z| times what multiplies it,
    one sum and one rounding, and Z is z rounded."""
    NW = 2 * N if act == "swiglu" else N
    pad, dt = 8, torch.bfloat16
    dims = B.make_linear_dims(M, N, K, "bf16", act, K + pad, N + pad, N + pad)
    assert B.moe_linear_plan(dims, B.LINEAR_OUT)[:2] == (256, 1)
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float()  # noqa: E731
    X, _ = strided(M, K, pad, "bf16", ints(M, K))
    W = (ints(NW, K) / 16).to(dt)
    b = ints(NW) if bias else None
    out, base = strided(M, N, pad, "bf16", extra_rows=2)
    res = ints(M, N).to(dt) if residual else None
    keep = res
    if alias:
        out.copy_(res)
        res = out
    elif residual:
        res = strided(M, N, pad, "bf16", res)[0]
    Z = torch.full((M + 1, NW), 777.0, dtype=dt, device="cuda") if save else None
    ws, nb = B.linear_workspace(dims, B.LINEAR_FORWARD)
    B.moe_linear(dims, X, W, b, res, Z, out, ws, nb)
    z = X.float() @ W.float().t()
    z = (z + b if bias else z).double()
    if save:
        assert torch.equal(Z[:M], z.to(dt)) and bool((Z[M] == 777.0).all())
    if act == "swiglu":
        gate, up = z[:, :N], z[:, N:]
        a, ae = gate * torch.sigmoid(gate) * up, ACT_ERR * (1 + gate.abs()) * up.abs()
    elif act == "silu":
        a, ae = z * torch.sigmoid(z), ACT_ERR * (1 + z.abs())
    elif act == "gelu":
        a, ae = z * torch.special.ndtr(z), ACT_ERR * (1 + z.abs())
    else:
        a, ae = z.clamp(min=0) if act == "relu" else z, torch.zeros_like(z)
    r = keep.double() if residual else torch.zeros_like(a)
    ref = a + r
    tol = HALF["bf16"] * (ref.abs() + ae) + ae + 2 * U32 * (a.abs() + r.abs())
    off = (out.double() - ref).abs()
    assert bool((off <= tol).all()), "worst %.3g" % (off / tol.clamp(min=1e-30)).max().item()
    assert_guards(base, M, N, "out")


@pytest.mark.parametrize("M,N,K,product", [(4088, 1096, 4088, B.LINEAR_DX), (4000, 1096, 3848, B.LINEAR_DX), (1100, 4088, 3976, B.LINEAR_DW)])
def test_large_tiles_backward_with_an_activation(M, N, K, product):
    """ReLU with whole numbers: dZ, the products (below 2^24) and dbias are exact, rounded once."""
    dims = B.make_linear_dims(M, N, K, "bf16", "relu", K + 8, 0, N + 24)
    assert B.moe_linear_plan(dims, product)[0] == 256
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float()  # noqa: E731
    X, W, dY, Z = ints(M, K), ints(N, K), ints(M, N), ints(M, N)
    Xs, dYs = strided(M, K, 8, "bf16", X)[0], strided(M, N, 24, "bf16", dY)[0]
    dX, base = strided(M, K, 8, "bf16", extra_rows=1)
    dW, db = torch.full((N + 1, K), 777.0, dtype=torch.bfloat16, device="cuda"), torch.full((N + 8,), 777.0, device="cuda")
    ws, nb = B.linear_workspace(dims, B.LINEAR_BACKWARD)
    B.moe_linear_backward(dims, dYs, Xs, W.bfloat16(), Z.bfloat16(), dX, dW[:N], db[:N], ws, nb)
    dZ = torch.where(Z > 0, dY, torch.zeros_like(dY))
    assert torch.equal(dX, (dZ @ W).bfloat16()) and torch.equal(dW[:N], (dZ.t() @ X).bfloat16())
    assert torch.equal(db[:N], dZ.sum(0))
    assert_guards(base, M, K, "dX")
    assert bool((dW[N] == 777.0).all()) and bool((db[N:] == 777.0).all())


@pytest.mark.parametrize("dtype,M", [("bf16", 300), ("f32", 140), ("bf16", 9)])
def test_row_strides_at_the_limit(dtype, M):
    """Strides of 2^22 elements: a tile's row offsets pass 2^31 bytes.  Whole numbers, so every result is exact."""
    N, K, ld = 72, 136, 1 << 22
    g = torch.Generator(device="cuda").manual_seed(M)
    ints = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float()  # noqa: E731

    def far(rows, cols, fill=None):
        v = torch.empty(rows * ld, dtype=DT[dtype], device="cuda").view(rows, ld)[:, :cols]
        if fill is not None:
            v.copy_(fill)
        return v

    X, W, R, dY = ints(M, K), ints(N, K), ints(M, N), ints(M, N)
    dims = B.make_linear_dims(M, N, K, dtype, "none", ld, ld, ld)
    wf, nf = B.linear_workspace(dims, B.LINEAR_FORWARD)
    wb, nb = B.linear_workspace(dims, B.LINEAR_BACKWARD)
    x, w, out, dX = far(M, K, X), W.to(DT[dtype]), far(M, N), far(M, K)
    B.moe_linear(dims, x, w, None, far(M, N, R), None, out, wf, nf)
    assert torch.equal(out, (X @ W.t() + R).to(DT[dtype]))
    dW, db = torch.empty_like(w), torch.empty(N, device="cuda")
    B.moe_linear_backward(dims, far(M, N, dY), x, w, None, dX, dW, db, wb, nb)
    assert torch.equal(dX, (dY @ W).to(DT[dtype])) and torch.equal(dW, (dY.t() @ X).to(DT[dtype])) and torch.equal(db, dY.sum(0))


def test_more_outputs_than_32_bits_count():
    """2^31 outputs and more: the last rows, and the sums over all of them, of whole numbers."""
    M, N, K = (1 << 20) + 8, 2056, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    ints = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda").bfloat16()  # noqa: E731
    X, W = ints(M, K), ints(N, K)
    dims = B.make_linear_dims(M, N, K, "bf16", "relu")
    ws, nb = B.linear_workspace(dims, B.LINEAR_BACKWARD)
    out, Z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    B.moe_linear(dims, X, W, None, None, Z, out, *B.linear_workspace(dims, B.LINEAR_FORWARD))
    dY = torch.ones(1, N, dtype=torch.bfloat16, device="cuda").expand(M, N).contiguous()
    dX, dW, db = torch.empty_like(X), torch.empty_like(W), torch.empty(N, device="cuda")
    B.moe_linear_backward(dims, dY, X, W, Z, dX, dW, db, ws, nb)
    tW, tb = torch.zeros(N, K, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
    for a in range(0, M, 1 << 16):
        x = X[a:a + (1 << 16)].float()
        z = x @ W.float().t()
        assert torch.equal(Z[a:a + (1 << 16)].float(), z) and torch.equal(out[a:a + (1 << 16)].float(), z.clamp(min=0))
        on = (z > 0).float()
        assert torch.equal(dX[a:a + (1 << 16)], (on @ W.float()).bfloat16())
        tW += (on.t() @ x).double()
        tb += on.sum(0).double()
    # counts stay below 2^24: exact in fp32, then dW is rounded once
    assert torch.equal(db.double(), tb) and torch.equal(dW, tW.float().bfloat16())
