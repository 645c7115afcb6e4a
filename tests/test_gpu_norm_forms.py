"""moe_norm and moe_norm_backward in more of the forms that a call may take, against the float64 oracle."""
import numpy as np
import pytest
import torch

import test_gpu_norm as tn
from block_util import DT, HALF, U32, assert_guards, assert_within, f64, strided
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from oracle import block as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


# workgroups of two waves: 1024 of them, which take several rows each
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", [(4100, 2048, 0), (4500, 2049, 7)])
def test_many_rows_of_two_waves(rows, cols, pad, dtype, wtype, kind):
    tn.test_norm_matches_oracle(rows, cols, pad, dtype, wtype, kind)
    tn.test_norm_backward_matches_oracle(rows, cols, pad, dtype, wtype, kind)


# k_norm_long (over 16384 columns) reads x + residual again after it stored sum
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(3, 16400), (300, 16390), (1, 65536)])
def test_long_rows_in_place(rows, cols, dtype, kind):
    a = tn.make(rows, cols, 0, dtype, "f32", 3)
    dims = B.make_norm_dims(rows, cols, dtype, kind)
    y, s = torch.empty_like(a["x"]), torch.empty_like(a["x"])
    mean, rstd = torch.zeros(rows, device="cuda"), torch.empty(rows, device="cuda")

    def go(x, r, s_, y_):
        m, q = torch.zeros(rows, device="cuda"), torch.empty(rows, device="cuda")
        B.moe_norm(dims, x, r, a["weight"], a["bias"], s_, y_, m, q)
        return m, q

    mean, rstd = go(a["x"], a["residual"], s, y)
    S = f64(s)
    rm, rr = ob.norm_stats(S, 1e-5, kind)
    ref = ob.norm(S, f64(a["weight"]), f64(a["bias"]), 1e-5, kind)
    assert_within("y", f64(y), ref, tn.forward_bound(S, f64(a["weight"]), f64(a["bias"]), rm, rr, 1e-5, dtype, ref))
    places = {"sum over x, y over residual": lambda x, r: (x, r), "sum over residual, y over x": lambda x, r: (r, x), "no sum, y over x": lambda x, r: (None, x),
              "no sum, y over residual": lambda x, r: (None, r), "sum over x": lambda x, r: (x, torch.empty_like(x)), "sum over residual": lambda x, r: (r, torch.empty_like(x))}
    for name, place in places.items():
        x, r = a["x"].clone(), a["residual"].clone()
        s_, y_ = place(x, r)
        m, q = go(x, r, s_, y_)
        assert torch.equal(y_, y) and (s_ is None or torch.equal(s_, s)) and torch.equal(m, mean) and torch.equal(q, rstd), name
    # without a residual, over x
    x, y0 = a["x"].clone(), torch.empty_like(a["x"])
    go(a["x"], None, None, y0)
    go(x, None, None, x)
    assert torch.equal(x, y0)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pads", [(37, 264, (8, 16, 24, 40)), (260, 1003, (1, 2, 5, 12)), (5, 9000, (3, 8, 17, 1)), (3, 16390, (2, 5, 9, 14)), (2100, 72, (7, 1, 0, 8))])
def test_every_array_with_a_stride_of_its_own(rows, cols, pads, dtype, kind):
    px, pr, ps, py = pads
    a = tn.make(rows, cols, 0, dtype, "f32", cols)
    lay = lambda t, pad: strided(rows, cols, pad, dtype, t)[0]  # noqa: E731
    dims = B.make_norm_dims(rows, cols, dtype, kind, 1e-5, "f32", ldx=cols + px, ldr=cols + pr, lds=cols + ps, ldy=cols + py)
    s, sbase = strided(rows, cols, ps, dtype, extra_rows=1)
    y, ybase = strided(rows, cols, py, dtype, extra_rows=1)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.empty(rows, device="cuda")
    B.moe_norm(dims, lay(a["x"], px), lay(a["residual"], pr), a["weight"], a["bias"], s, y, mean, rstd)
    assert torch.equal(s, (a["x"].float() + a["residual"].float()).to(DT[dtype]))
    S, w, b = f64(s), f64(a["weight"]), f64(a["bias"])
    rm, rr = ob.norm_stats(S, 1e-5, kind)
    ref = ob.norm(S, w, b, 1e-5, kind)
    assert_within("y", f64(y), ref, tn.forward_bound(S, w, b, rm, rr, 1e-5, dtype, ref))
    assert_guards(sbase, rows, cols, "sum")
    assert_guards(ybase, rows, cols, "y")
    # backward: dy by ldy, s by lds, dsum by ldr, dx by ldx
    dx, base = strided(rows, cols, px, dtype, extra_rows=1)
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws, nb = B.norm_workspace(dims)
    B.moe_norm_backward(dims, lay(a["dy"], py), s, a["weight"], mean, rstd, lay(a["dsum"], pr), dx, dw, db, ws, nb)
    assert_guards(base, rows, cols, "dx")
    DY, DS, m, r = f64(a["dy"]), f64(a["dsum"]), f64(mean), f64(rstd)
    rdx, rdw, rdb = ob.norm_backward(DY, S, w, m, r, DS, kind)
    xh = np.abs((S - (m[:, None] if kind == "layer" else 0.0)) * r[:, None])
    G = np.abs(DY * w)
    err = r[:, None] * ((tn.CHAIN + 10) * U32 * (G.mean(axis=1)[:, None] * (kind == "layer") + xh * (G * xh).mean(axis=1)[:, None]) + 8 * U32 * G) + 2 * U32 * np.abs(DS)
    assert_within("dx", f64(dx), rdx, HALF[dtype] * (np.abs(rdx) + err) + err + 1e-37)
    # at least 256 workgroups share the rows (fewer rows: one each), then up to 32 row groups and the join
    chain = -(-rows // 256) + 32 + 8
    assert_within("dweight", f64(dw), rdw, chain * U32 * (np.abs(DY) * xh).sum(axis=0) + 1e-37)
    assert_within("dbias", f64(db), rdb, chain * U32 * np.abs(DY).sum(axis=0) + 1e-37)
    # the strides change no sum's order: dense arrays give the same, dx and the vectors' gradients alone too
    dense = B.make_norm_dims(rows, cols, dtype, kind)
    dx1, dw1, db1 = torch.empty(rows, cols, dtype=DT[dtype], device="cuda"), torch.empty_like(dw), torch.empty_like(db)
    s1 = s.contiguous()
    B.moe_norm_backward(dense, a["dy"], s1, a["weight"], mean, rstd, a["dsum"], dx1, None, None, None, 0)
    B.moe_norm_backward(dense, a["dy"], s1, a["weight"], mean, rstd, None, None, dw1, db1, ws, nb)
    assert torch.equal(dx1, dx) and torch.equal(dw1, dw) and torch.equal(db1, db)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [8, 1003, 7168, 16390])
@pytest.mark.parametrize("eps", [0.0, 1e-12, 0.1])
def test_eps(cols, eps, dtype, kind):
    """Rows of small and of large variance: eps counts by its own value."""
    rows = 6
    a = tn.make(rows, cols, 0, dtype, "f32", cols, mean=0.0)
    x = (a["x"].float() * torch.tensor([1e-3, 1e-2, 0.1, 1.0, 10.0, 1e-6], device="cuda")[:, None]).to(DT[dtype])
    dims = B.make_norm_dims(rows, cols, dtype, kind, eps)
    eps = float(np.float32(eps))
    y, mean, rstd = torch.empty_like(x), torch.zeros(rows, device="cuda"), torch.empty(rows, device="cuda")
    B.moe_norm(dims, x, None, a["weight"], a["bias"], None, y, mean, rstd)
    X, w, b = f64(x), f64(a["weight"]), f64(a["bias"])
    rm, rr = ob.norm_stats(X, eps, kind)
    bm, br = tn.stat_bounds(X, rm, rr, eps)
    assert_within("rstd", f64(rstd), rr, br * rr)
    ref = ob.norm(X, w, b, eps, kind)
    assert_within("y", f64(y), ref, tn.forward_bound(X, w, b, rm, rr, eps, dtype, ref))
    if eps == 0.0:  # rows of zeros have no direction
        B.moe_norm(dims, torch.zeros_like(x), None, None, None, None, y, None, None)
        assert bool(y.isnan().all())


# rows in 8 lanes, in waves, in workgroups, of two chunks a thread of 1024, re-read
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [5, 60, 100, 200, 264, 520, 1003, 1100, 7168, 9000, 16390])
def test_rows_of_any_finite_size(cols, dtype, kind):
    """Rows whose squares or sums leave fp32's range, up and down, beside rows that stay in it."""
    sizes = [1.0, 1e19, 1e25, 1e37, 1e-12, 1e-20, 1e-30, 3.0, 1e30, 1e-36, 1e-3]
    rows = 3 * len(sizes)
    g = torch.Generator().manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64).clamp_(-4, 4)
    x[::3] += 2.0  # (means far from zero: the sum of 16390 elements of 2e37 is beyond the range, their mean is not)
    x *= torch.tensor(sizes, dtype=torch.float64).repeat(3)[:, None]
    x = x.to(DT[dtype]).cuda()
    assert bool(x.isfinite().all())
    w, b = torch.linspace(0.5, 1.5, cols, device="cuda"), torch.linspace(-1, 1, cols, device="cuda")
    for eps in (0.0, 1e-30, 1e-5):
        dims = B.make_norm_dims(rows, cols, dtype, kind, eps)
        y, mean, rstd = torch.empty_like(x), torch.zeros(rows, device="cuda"), torch.empty(rows, device="cuda")
        B.moe_norm(dims, x, None, w, b, None, y, mean, rstd)
        X, e = f64(x), float(np.float32(eps))
        rm, rr = ob.norm_stats(X, e, kind)
        bm, br = tn.stat_bounds(X, rm, rr, e)
        assert_within("mean", f64(mean), rm, bm + U32 * np.abs(rm))
        # (below the normal range a step is 2^-149)
        assert_within("rstd", f64(rstd), rr, br * rr + 2.0 ** -149)
        ref = ob.norm(X, f64(w), f64(b), e, kind)
        tiny = 2.0 ** -149 / rr[:, None] * np.abs(ref - f64(b))  # (rstd's last step, relative, and its part of y)
        assert_within("y", f64(y), ref, tn.forward_bound(X, f64(w), f64(b), rm, rr, e, dtype, ref) + tiny)
        # every row alone is the same: none reaches another
        for r in range(0, rows, 7):
            one = B.make_norm_dims(1, cols, dtype, kind, eps)
            y1 = torch.empty(1, cols, dtype=DT[dtype], device="cuda")
            B.moe_norm(one, x[r:r + 1].clone(), None, w, b, None, y1, None, None)
            ok = tn.forward_bound(X[r:r + 1], f64(w), f64(b), rm[r:r + 1], rr[r:r + 1], e, dtype, ref[r:r + 1]) + tiny[r:r + 1]
            assert_within("row %d alone" % r, f64(y1), ref[r:r + 1], ok)
