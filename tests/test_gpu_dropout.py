"""moe_dropout and moe_combine_dropout against the float64 oracle: the mask bit for bit, values to the
output's rounding."""
import numpy as np
import pytest
import torch

from block_util import DT, HALF, U32, assert_guards, assert_within, check_replays, f64, strided
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from mixture_experts_layer_lds_amd import workloads as wl
from oracle import block as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield


def words(seed, offset):
    a = np.array([seed, offset], np.uint64).view(np.int64)
    return torch.from_numpy(a.copy()).cuda()


def bound(x, y, res, dtype, scale):
    """One rounding of the output and two fp32 operations (the scaling, whose factor is rounded too,
    and the sum)."""
    return HALF[dtype] * np.abs(y) + 2 * U32 * (np.abs(x) * scale + (np.abs(res) if res is not None else 0)) + 1e-300


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad,residual,p", [
    (1, 1, 0, False, 0.5), (1, 8, 0, True, 0.1), (3, 7, 0, True, 0.25), (5, 9, 7, False, 0.9), (257, 1003, 5, True, 0.1),
    (64, 1024, 0, False, 0.1), (33, 264, 8, True, 0.3), (7, 4096, 0, True, 0.0), (7, 130, 6, True, 1.0), (1000, 16, 0, False, 0.5),
    (2, 65539, 5, True, 0.37),
])
def test_dropout_matches_oracle(rows, cols, pad, residual, p, dtype):
    g = torch.Generator().manual_seed(rows * 1000 + cols)
    seed, offset = 0x9E3779B97F4A7C15 ^ cols, (rows << 33) + 5
    x, _ = strided(rows, cols, pad, dtype, torch.randn(rows, cols, generator=g))
    res = strided(rows, cols, pad, dtype, torch.randn(rows, cols, generator=g))[0] if residual else None
    out, base = strided(rows, cols, pad, dtype, extra_rows=2)
    B.moe_dropout(x, res, p, words(seed, offset), out)
    torch.cuda.synchronize()
    rx, rr = f64(x), f64(res) if residual else None
    keep = ob.dropout_keep(rows, cols, p, seed, offset)
    ref = ob.dropout(rx, p, seed, offset, rr)
    if not residual:
        assert np.array_equal((f64(out) != 0)[rx != 0], keep[rx != 0])
    t = ob.dropout_threshold(p)
    assert_within("out", f64(out), ref, bound(np.where(keep, rx, 0), ref, rr, dtype, 65536 / max(65536 - t, 1)))
    assert_guards(base, rows, cols, "out")


def test_dropped_infinities_and_nans_add_nothing():
    rows, cols, p = 64, 200, 0.5
    x = torch.full((rows, cols), float("nan"), device="cuda")
    x[:, ::2] = float("inf")
    r = torch.ones(rows, cols, device="cuda")
    out = torch.empty_like(x)
    B.moe_dropout(x, r, p, words(3, 4), out)
    keep = ob.dropout_keep(rows, cols, p, 3, 4)
    got = out.cpu().numpy()
    assert np.all(got[~keep] == 1.0) and not np.isfinite(got[keep]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_dropout_in_place_and_gradient_by_differences(dtype):
    """out may be x or residual; the gradient is the same call on dout: <dout, f(x)> is linear in x, so
    its difference along any direction v is <dx, v> exactly (up to fp32 rounding)."""
    rows, cols, p = 37, 272, 0.3
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(DT[dtype])
    r = torch.randn(rows, cols, generator=g, device="cuda").to(DT[dtype])
    rng = words(11, 1 << 40)
    want = torch.empty_like(x)
    B.moe_dropout(x, r, p, rng, want)
    a, b = x.clone(), r.clone()
    B.moe_dropout(a, r, p, rng, a)
    B.moe_dropout(x, b, p, rng, b)
    assert torch.equal(a, want) and torch.equal(b, want)
    if dtype == "f32":
        dout, v = (torch.randn(rows, cols, generator=g, device="cuda") for _ in range(2))
        dx, y0, y1 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        B.moe_dropout(dout, None, p, rng, dx)
        B.moe_dropout(x, r, p, rng, y0)
        B.moe_dropout(x + v, r, p, rng, y1)
        diff = (dout.double() * (y1.double() - y0.double())).sum().item()
        # each y is off by at most 2^-22 of its terms' sizes: the sum of their products with dout
        size = (dout.abs().double() * (x.abs() * 2 + v.abs() + r.abs()).double() * 1.5).sum().item()
        assert abs(diff - (dx.double() * v.double()).sum().item()) <= 2.0 ** -20 * size


def test_element_offsets_past_32_bits():
    """Rows whose element offset passes 2^31 (a large row stride): the last rows match the oracle."""
    rows, cols, ld = 5, 64, 1 << 29
    base = torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = base.view(rows, ld)[:, :cols]
    x.copy_(torch.randn(rows, cols))
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    B.moe_dropout(x, None, 0.25, words(5, 6), out)
    ref = ob.dropout(f64(x), 0.25, 5, 6)
    assert_within("out", f64(out), ref, bound(f64(x), ref, None, "bf16", 4 / 3))


def test_dropout_graph_draws_new_masks_when_the_words_change():
    x = torch.randn(100, 136, device="cuda")
    out, rng = torch.empty_like(x), words(1, 0)
    check_replays(lambda: B.moe_dropout(x, None, 0.5, rng, out), dict(out=out))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_dropout(x, None, 0.5, rng, out)
    for off in (0, 1, 2):
        rng.copy_(words(1, off))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy() != 0, ob.dropout_keep(100, 136, 0.5, 1, off))


def routed(cfg):
    inp = wl.make_inputs(cfg, device="cuda")
    dims = B.make_dims(cfg.T, cfg.d, cfg.n, cfg.E, cfg.K, cfg.dtype, cfg.round_mode, cfg.tile_m)
    plan = B.Plan(dims)
    logits = torch.empty(cfg.T, cfg.E, device="cuda")
    ws, nb = B.workspace(dims, B.OP_ROUTE)
    B.moe_route(dims, inp["X"], inp["W_r"], inp["bias"], logits, plan, ws, nb)
    return dims, plan


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,E,K,round_mode,residual,weighted", [
    (1, 64, 4, 1, 0, True, True), (77, 320, 6, 2, 0, True, True), (130, 1088, 8, 3, 0, False, True),
    (300, 1536, 8, 2, 3, True, True), (65, 2112, 5, 5, 0, True, False),
])
def test_combine_dropout_matches_oracle(T, d, E, K, round_mode, residual, weighted, dtype):
    """Token rounding down leaves some tokens without rows: they get their residual alone."""
    cfg = wl.small_shape(T=T, d=d, E=E, K=K, n=64, dtype=dtype, backward=False, round_mode=round_mode, tile_m=64)
    dims, plan = routed(cfg)
    h = plan.to_host()
    g = torch.Generator(device="cuda").manual_seed(3)
    Y = torch.randn(plan.R_max, d, generator=g, device="cuda").to(DT[dtype])
    res = torch.randn(T, d, generator=g, device="cuda").to(DT[dtype]) if residual else None
    out = torch.empty(T, d, dtype=DT[dtype], device="cuda")
    p = 0.25
    B.moe_combine_dropout(dims, plan, Y, weighted, res, p, words(21, 22), out)
    y, r = f64(Y), f64(res) if residual else np.zeros((T, d))
    summed, size = np.zeros((T, d)), np.zeros((T, d))
    for t in range(T):
        for i in range(h["tok_off"][t], h["tok_off"][t + 1]):
            row = h["tok_row"][i]
            term = (h["row_w"][row] if weighted else 1.0) * y[row]
            summed[t] += term
            size[t] += np.abs(term)
    ref = ob.dropout(summed, p, 21, 22, r)
    # K products and sums in fp32, then scaling and residual, then one rounding
    tol = HALF[dtype] * np.abs(ref) + (2 * K + 4) * U32 * (size * 4 / 3 + np.abs(r)) + 1e-300
    if round_mode == 3:
        assert (np.diff(h["tok_off"]) == 0).any()
    assert_within("out", f64(out), ref, tol)
    if residual:
        alias = res.clone()
        B.moe_combine_dropout(dims, plan, Y, weighted, alias, p, words(21, 22), alias)
        assert torch.equal(alias, out)
    plain, zero_p = torch.empty_like(out), torch.empty_like(out)
    B.moe_combine(dims, plan, Y, weighted, plain)
    B.moe_combine_dropout(dims, plan, Y, weighted, None, 0.0, words(21, 22), zero_p)
    assert torch.equal(plain, zero_p)
