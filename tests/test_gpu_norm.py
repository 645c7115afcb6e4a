"""moe_norm and moe_norm_backward against the float64 oracle."""
import numpy as np
import pytest
import torch

from block_util import DT, HALF, U32, assert_guards, assert_within, check_replays, f64, strided
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


# terms that follow one another in a row's fp32 sums: a thread's elements (up to 64), the lanes (6), the waves (16)
CHAIN = 64 + 6 + 16


def stat_bounds(s, mean, rstd, eps):
    """How far mean (absolute) and rstd (relative) may be off: every partial sum rounds once; the squares' sum
    about a mean that is off by m is off by n m^2 (the linear term vanishes)."""
    m = (CHAIN + 2) * U32 * np.abs(s).mean(axis=1)
    d2 = ((s - mean[:, None]) ** 2).mean(axis=1)
    var = (CHAIN + 6) * U32 * d2 + m ** 2
    return m, 0.5 * var / (d2 + eps) + 6 * U32


def forward_bound(s, w, b, mean, rstd, eps, dtype, y):
    m, rel = stat_bounds(s, mean, rstd, eps)
    xw = np.abs((s - mean[:, None]) * rstd[:, None] * w)
    err = xw * (rel[:, None] + 6 * U32) + (m * rstd)[:, None] * np.abs(w) * (1 + rel[:, None]) + 2 * U32 * np.abs(b)
    return HALF[dtype] * (np.abs(y) + err) + err + 1e-37


def make(rows, cols, pad, dtype, wtype, seed, mean=0.5):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    a = {}
    for k, std in (("x", 1.0), ("residual", 2.0), ("dy", 1.0), ("dsum", 1.0)):
        a[k], _ = strided(rows, cols, pad, dtype, rn(rows, cols) * std + (mean if k == "x" else 0.0))
    a["weight"] = (rn(cols) * 0.3 + 1.0).to(DT[wtype]).cuda()
    a["bias"] = (rn(cols) * 0.2).to(DT[wtype]).cuda()
    return a


# one row and many; a lane's worth of columns to rows over 1024 threads; odd widths and strides
SHAPES = [
    (1, 1, 0), (1, 8, 0), (3, 7, 0), (5, 9, 7), (2, 63, 1), (1, 7168, 0), (4, 64, 0), (33, 264, 8), (257, 1003, 5),
    (64, 1024, 0), (7, 4096, 0), (2, 8200, 0), (3, 16385, 3), (2, 65536, 0), (2, 65535, 0), (1030, 136, 0), (2100, 520, 8),
    (1100, 1536, 0), (1025, 2049, 0), (1024, 7168, 0), (1030, 40, 4), (5000, 3, 0),
    (600, 8200, 0), (300, 16390, 2),  # workgroups of 1024 threads that take several rows
]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_norm_matches_oracle(rows, cols, pad, dtype, wtype, kind):
    a = make(rows, cols, pad, dtype, wtype, rows * 7 + cols)
    eps = 1e-5
    ld = dict(ldx=cols + pad, ldr=cols + pad, lds=cols + pad, ldy=cols + pad)
    dims = B.make_norm_dims(rows, cols, dtype, kind, eps, wtype, **ld)
    y, ybase = strided(rows, cols, pad, dtype, extra_rows=2)
    s, sbase = strided(rows, cols, pad, dtype, extra_rows=2)
    mean, rstd = torch.full((rows + 1,), 7.0, device="cuda"), torch.full((rows + 1,), 7.0, device="cuda")
    B.moe_norm(dims, a["x"], a["residual"], a["weight"], a["bias"], s, y, mean, rstd)
    torch.cuda.synchronize()
    assert torch.equal(s, (a["x"].float() + a["residual"].float()).to(DT[dtype]))
    S, w, b = f64(s), f64(a["weight"]), f64(a["bias"])
    rm, rr = ob.norm_stats(S, eps, kind)
    bm, br = stat_bounds(S, rm, rr, eps)
    if kind == "layer":
        assert_within("mean", f64(mean)[:rows], rm, bm + U32 * np.abs(rm))
    else:
        assert bool((mean == 7.0).all())
    assert_within("rstd", f64(rstd)[:rows], rr, br * rr)
    assert float(rstd[rows]) == 7.0 and float(mean[rows]) == 7.0
    ref = ob.norm(S, w, b, eps, kind)
    assert_within("y", f64(y), ref, forward_bound(S, w, b, rm, rr, eps, dtype, ref))
    assert_guards(ybase, rows, cols, "y")
    assert_guards(sbase, rows, cols, "sum")
    # without a residual, a weight, a bias, statistics: the same x normalised plainly
    y0, base0 = strided(rows, cols, pad, dtype, extra_rows=1)
    B.moe_norm(dims, a["x"], None, None, None, None, y0, None, None)
    X, one, zero = f64(a["x"]), np.ones(cols), np.zeros(cols)
    rm, rr = ob.norm_stats(X, eps, kind)
    ref = ob.norm(X, None, None, eps, kind)
    assert_within("plain y", f64(y0), ref, forward_bound(X, one, zero, rm, rr, eps, dtype, ref))
    assert_guards(base0, rows, cols, "plain y")
    # the sum need not be kept
    y1, _ = strided(rows, cols, pad, dtype)
    B.moe_norm(dims, a["x"], a["residual"], a["weight"], a["bias"], None, y1, None, None)
    assert torch.equal(y1, y)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_norm_backward_matches_oracle(rows, cols, pad, dtype, wtype, kind):
    a = make(rows, cols, pad, dtype, wtype, rows * 13 + cols)
    ld = dict(ldx=cols + pad, ldr=cols + pad, lds=cols + pad, ldy=cols + pad)
    dims = B.make_norm_dims(rows, cols, dtype, kind, 1e-5, wtype, **ld)
    S, w, DY, DS = f64(a["x"]), f64(a["weight"]), f64(a["dy"]), f64(a["dsum"])
    m, r = ob.norm_stats(S, 1e-5, kind)
    mean, rstd = torch.from_numpy(m.astype(np.float32)).cuda(), torch.from_numpy(r.astype(np.float32)).cuda()
    m, r = f64(mean), f64(rstd)
    dx, base = strided(rows, cols, pad, dtype, extra_rows=2)
    dw, db = torch.full((cols + 1,), 7.0, device="cuda"), torch.full((cols + 1,), 7.0, device="cuda")
    ws, nb = B.norm_workspace(dims)
    st = (mean if kind == "layer" else None, rstd)
    B.moe_norm_backward(dims, a["dy"], a["x"], a["weight"], *st, a["dsum"], dx, dw, db, ws, nb)
    torch.cuda.synchronize()
    rdx, rdw, rdb = ob.norm_backward(DY, S, w, m, r, DS, kind)
    xh = np.abs((S - (m[:, None] if kind == "layer" else 0.0)) * r[:, None])
    G = np.abs(DY * w)
    mg, mgx = G.mean(axis=1)[:, None], (G * xh).mean(axis=1)[:, None]
    err = r[:, None] * ((CHAIN + 10) * U32 * (mg * (kind == "layer") + xh * mgx) + 8 * U32 * G) + 2 * U32 * np.abs(DS)
    assert_within("dx", f64(dx), rdx, HALF[dtype] * (np.abs(rdx) + err) + err + 1e-37)
    assert_guards(base, rows, cols, "dx")
    # a thread's rows one after another (1024 workgroups at least share many rows), then up to 32 row groups
    chain = -(-rows // 1024) + 32 + 8
    assert_within("dweight", f64(dw)[:cols], rdw, chain * U32 * (np.abs(DY) * xh).sum(axis=0) + 1e-37)
    assert_within("dbias", f64(db)[:cols], rdb, chain * U32 * np.abs(DY).sum(axis=0) + 1e-37)
    assert float(dw[cols]) == 7.0 and float(db[cols]) == 7.0
    # each output alone is the same
    alone = torch.empty_like(dx)
    d2 = B.make_norm_dims(rows, cols, dtype, kind, 1e-5, wtype, **dict(ld, ldx=cols))
    B.moe_norm_backward(d2, a["dy"], a["x"], a["weight"], *st, a["dsum"], alone, None, None, None, 0)
    if pad % 8 == 0:  # (other strides, another order of the sums)
        assert torch.equal(alone, dx)
    w1, b1 = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    B.moe_norm_backward(dims, a["dy"], a["x"], a["weight"], *st, None, None, w1, None, ws, nb)
    B.moe_norm_backward(dims, a["dy"], a["x"], a["weight"], *st, None, None, None, b1, ws, nb)
    assert torch.equal(w1, dw[:cols]) and torch.equal(b1, db[:cols])
    # without dsum and weight
    B.moe_norm_backward(d2, a["dy"], a["x"], None, *st, None, alone, None, None, None, 0)
    rdx = ob.norm_backward(DY, S, None, m, r, None, kind)[0]
    G = np.abs(DY)
    err = r[:, None] * ((CHAIN + 10) * U32 * (G.mean(axis=1)[:, None] * (kind == "layer") + xh * (G * xh).mean(axis=1)[:, None]) + 8 * U32 * G)
    assert_within("dx alone", f64(alone), rdx, HALF[dtype] * (np.abs(rdx) + err) + err + 1e-37)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(5, 1000), (1200, 264), (3, 9000)])
def test_in_place(rows, cols, dtype):
    a = make(rows, cols, 0, dtype, "f32", 3)
    dims = B.make_norm_dims(rows, cols, dtype)
    y, s = torch.empty_like(a["x"]), torch.empty_like(a["x"])
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    go = lambda x, r, s_, y_: B.moe_norm(dims, x, r, a["weight"], a["bias"], s_, y_, mean, rstd)  # noqa: E731
    go(a["x"], a["residual"], s, y)
    for over in ("x", "residual"):
        x, r = a["x"].clone(), a["residual"].clone()
        go(x, r, dict(x=x, residual=r)[over], dict(x=r, residual=x)[over])
        assert torch.equal(dict(x=x, residual=r)[over], s) and torch.equal(dict(x=r, residual=x)[over], y)
    ws, nb = B.norm_workspace(dims)
    dx, dw, db = torch.empty_like(s), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    B.moe_norm_backward(dims, a["dy"], s, a["weight"], mean, rstd, a["dsum"], dx, dw, db, ws, nb)
    for over in ("dy", "s", "dsum"):
        t = dict(dy=a["dy"].clone(), s=s.clone(), dsum=a["dsum"].clone())
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        B.moe_norm_backward(dims, t["dy"], t["s"], a["weight"], mean, rstd, t["dsum"], t[over], dw2, db2, ws, nb)
        assert torch.equal(t[over], dx) and torch.equal(dw2, dw) and torch.equal(db2, db), over


def test_no_rows():
    cols = 70
    dims = B.make_norm_dims(0, cols, "bf16")
    B.moe_norm(dims, None, None, None, None, None, None, None, None)
    dw, db = torch.full((cols,), 7.0, device="cuda"), torch.full((cols,), 7.0, device="cuda")
    ws, nb = B.norm_workspace(dims)
    B.moe_norm_backward(dims, None, None, None, None, None, None, None, dw, db, ws, nb)
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_means_and_constant_rows(dtype):
    """Rows whose mean is 1000 times their deviation keep the bound (which grows with it); constant rows give
    the bias exactly; subnormal and huge finite rows stay finite where their squares do."""
    rows, cols = 6, 520
    g = torch.Generator().manual_seed(4)
    x = torch.randn(rows, cols, generator=g)
    x[0] = x[0] + 1000.0
    x[1] = 3.0
    x[2] = 0.0
    x[3] *= 1e15
    x[4] *= 1e-30
    x = x.to(DT[dtype]).cuda()
    w, b = torch.full((cols,), 1.5, device="cuda"), torch.linspace(-1, 1, cols, device="cuda")
    y = torch.empty_like(x)
    B.moe_norm(B.make_norm_dims(rows, cols, dtype), x, None, w, b, None, y, None, None)
    X = f64(x)
    m, r = ob.norm_stats(X, 1e-5)
    ref = ob.norm(X, f64(w), f64(b))
    assert_within("y", f64(y), ref, forward_bound(X, f64(w), f64(b), m, r, 1e-5, dtype, ref))
    assert torch.equal(y[2], b.to(DT[dtype]))


def test_infinities_and_nans_stay_in_their_rows():
    rows, cols = 70, 264
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    dims = B.make_norm_dims(rows, cols, "f32")
    want, got = torch.empty_like(x), torch.empty_like(x)
    B.moe_norm(dims, x, None, None, None, None, want, None, None)
    x[3, 5], x[40, 263], x[64, 0] = float("nan"), float("inf"), float("-inf")
    B.moe_norm(dims, x, None, None, None, None, got, None, None)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[[3, 40, 64]] = True
    assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], want[~bad])


def test_element_offsets_past_32_bits():
    rows, cols, ld = 5, 64, 1 << 29
    base = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = base.view(rows, ld)[:, :cols]
    x.copy_(torch.randn(rows, cols))
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    B.moe_norm(B.make_norm_dims(rows, cols, ldx=ld), x, None, None, None, None, y, None, None)
    X = f64(x)
    m, r = ob.norm_stats(X, 1e-5)
    ref = ob.norm(X)
    assert_within("y", f64(y), ref, forward_bound(X, np.ones(cols), np.zeros(cols), m, r, 1e-5, "bf16", ref))
    dy = torch.randn(rows, cols, device="cuda").bfloat16()
    mean, rstd = torch.from_numpy(m.astype(np.float32)).cuda(), torch.from_numpy(r.astype(np.float32)).cuda()
    near, far = torch.empty_like(y), x.clone()
    d = B.make_norm_dims(rows, cols)
    B.moe_norm_backward(d, dy, far, None, mean, rstd, None, near, None, None, None, 0)
    d = B.make_norm_dims(rows, cols, lds=ld, ldx=ld)
    B.moe_norm_backward(d, dy, x, None, mean, rstd, None, x, None, None, None, 0)
    assert torch.equal(x, near)


@pytest.mark.parametrize("rows,cols", [(1, 7168), (1500, 520)])
def test_graph_replays_match_eager(rows, cols):
    a = make(rows, cols, 0, "bf16", "f32", 11)
    dims = B.make_norm_dims(rows, cols, "bf16")
    o = dict(s=torch.empty_like(a["x"]), y=torch.empty_like(a["x"]), mean=torch.empty(rows, device="cuda"),
             rstd=torch.empty(rows, device="cuda"), dx=torch.empty_like(a["x"]), dw=torch.empty(cols, device="cuda"),
             db=torch.empty(cols, device="cuda"))
    ws, nb = B.norm_workspace(dims)

    def step():
        B.moe_norm(dims, a["x"], a["residual"], a["weight"], a["bias"], o["s"], o["y"], o["mean"], o["rstd"])
        B.moe_norm_backward(dims, a["dy"], o["s"], a["weight"], o["mean"], o["rstd"], a["dsum"], o["dx"], o["dw"], o["db"], ws, nb)

    check_replays(step, o)


def test_calls_on_two_streams_with_their_own_workspaces():
    rows, cols = 3000, 1032
    ins = [make(rows, cols, 0, "bf16", "f32", k) for k in (1, 2)]
    dims = B.make_norm_dims(rows, cols, "bf16")

    def step(a, ws, nb):
        s, y, dx = (torch.empty_like(a["x"]) for _ in range(3))
        m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        B.moe_norm(dims, a["x"], a["residual"], a["weight"], a["bias"], s, y, m, r)
        B.moe_norm_backward(dims, a["dy"], s, a["weight"], m, r, a["dsum"], dx, dw, db, ws, nb)
        return y, dx, dw, db

    wss = [B.norm_workspace(dims) for _ in ins]
    want = [step(a, *w) for a, w in zip(ins, wss)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ins], []
    for a, w, st in zip(ins, wss, streams):
        with torch.cuda.stream(st):
            got.append(step(a, *w))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for x, y in zip(g, w):
            assert torch.equal(x, y)
