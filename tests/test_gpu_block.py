"""A training step of a whole block run through the library: residual dropout on the routed experts,
a shared expert beside them, the router losses and every gradient, against float64."""
import numpy as np
import pytest
import torch

import oracle
from block_util import check_replays, f64
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from mixture_experts_layer_lds_amd import workloads as wl
from oracle import block as ob
from parity import TOL, assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


class Block:
    """out = X + dropout(moe(X)) + down(swiglu(gate_up(X))); loss = <dOut, out> + dloss . (balance, z)."""

    def __init__(self, cfg, p=0.2):
        self.cfg, self.p = cfg, p
        T, d, E, n = cfg.T, cfg.d, cfg.E, cfg.n
        dev = dict(device="cuda")
        self.inp = inp = wl.make_inputs(cfg, device="cuda", with_grad_out=True)
        dt = cfg.torch_dtype
        g = torch.Generator(device="cuda").manual_seed(8)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.Wgu, self.bgu = (rn(2 * n, d) / d ** 0.5).to(dt), rn(2 * n) * 0.1
        self.Wd = (rn(d, n) / n ** 0.5).to(dt)
        self.rng = torch.tensor([1234, 5678], dtype=torch.int64, device="cuda")
        self.dloss = torch.tensor([40.0, 3.0], device="cuda")
        self.off, self.S = torch.tensor([0, T // 3, T - 5], dtype=torch.int32, device="cuda"), 2
        self.dims = B.make_dims(T, d, n, E, cfg.K, cfg.dtype, cfg.round_mode, cfg.tile_m)
        self.plan = B.Plan(self.dims)
        R = self.plan.R_max
        e = lambda *s, t=dt: torch.empty(*s, dtype=t, **dev)  # noqa: E731
        f = torch.float32
        self.logits, self.Y, self.H, self.y1, self.out = e(T, E, t=f), e(R, d), e(R, 2 * n), e(T, d), e(T, d)
        self.act, self.Zgu = e(T, n), e(T, 2 * n)
        self.tokens, self.counts = e(2, t=torch.int32), e(2, E, t=torch.int32)
        self.prob, self.lse, self.loss, self.aux = e(2, E, t=f), e(T, t=f), e(2, t=f), e(T, E, t=f)
        self.dYm, self.dX, self.dXs, self.dact = e(T, d), e(T, d), e(T, d), e(T, n)
        self.dWg, self.dWu, self.dWdn = (torch.empty_like(inp[k]) for k in ("W_gate", "W_up", "W_down"))
        self.dS, self.dL, self.dWr = e(R, t=f), e(T, E, t=f), torch.empty_like(inp["W_r"])
        self.dWgu, self.dbgu, self.dWd = torch.empty_like(self.Wgu), torch.empty_like(self.bgu), torch.empty_like(self.Wd)
        self.gu, self.dn = B.make_linear_dims(T, n, d, cfg.dtype, "swiglu"), B.make_linear_dims(T, d, n, cfg.dtype)
        self.ws = {op: B.workspace(self.dims, op) for op in (B.OP_ROUTE, B.OP_FFN, B.OP_BACKWARD)}
        self.wl = B.router_loss_workspace(self.dims, 2)
        self.lw = {(k, op): B.linear_workspace(dm, op) for k, dm in (("gu", self.gu), ("dn", self.dn))
                   for op in (B.LINEAR_FORWARD, B.LINEAR_BACKWARD)}

    def step(self):
        i, F, G = self.inp, B.LINEAR_FORWARD, B.LINEAR_BACKWARD
        B.moe_route(self.dims, i["X"], i["W_r"], i["bias"], self.logits, self.plan, *self.ws[B.OP_ROUTE])
        B.moe_router_loss(self.dims, self.logits, self.plan.topk_idx, self.S, self.off, None, self.tokens, self.counts,
                          self.prob, self.lse, self.loss, *self.wl)
        B.moe_grouped_ffn(self.dims, self.plan, i["X"], True, i["W_gate"], i["W_up"], i["W_down"], self.H, self.Y,
                          *self.ws[B.OP_FFN])
        B.moe_combine_dropout(self.dims, self.plan, self.Y, True, i["X"], self.p, self.rng, self.y1)
        B.moe_linear(self.gu, i["X"], self.Wgu, self.bgu, None, self.Zgu, self.act, *self.lw["gu", F])
        B.moe_linear(self.dn, self.act, self.Wd, None, self.y1, None, self.out, *self.lw["dn", F])
        # backward of dOut = dY
        B.moe_linear_backward(self.dn, i["dY"], self.act, self.Wd, None, self.dact, self.dWd, None, *self.lw["dn", G])
        B.moe_linear_backward(self.gu, self.dact, i["X"], self.Wgu, self.Zgu, self.dXs, self.dWgu, self.dbgu, *self.lw["gu", G])
        B.moe_dropout(i["dY"], None, self.p, self.rng, self.dYm)
        B.moe_router_loss_backward(self.dims, self.dloss, self.logits, self.S, self.off, None, self.tokens, self.counts,
                                   self.lse, self.aux)
        B.moe_backward_aux(self.dims, self.dYm, i["X"], i["W_r"], i["W_gate"], i["W_up"], i["W_down"], self.plan, self.H,
                           self.aux, self.dX, self.dWg, self.dWu, self.dWdn, self.dS, self.dL, self.dWr,
                           *self.ws[B.OP_BACKWARD])

    def outs(self):
        names = ("out", "loss", "counts", "dX", "dXs", "dWg", "dWu", "dWdn", "dL", "dWr", "dWgu", "dbgu", "dWd", "aux")
        return {k: getattr(self, k) for k in names}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,E,K,n,round_mode", [(300, 128, 12, 2, 64, 0), (700, 320, 6, 2, 192, 1), (129, 192, 40, 4, 128, 0)])
def test_block_step(T, d, E, K, n, round_mode, dtype):
    cfg = wl.small_shape(T=T, d=d, E=E, K=K, n=n, dtype=dtype, backward=True, seed=41, round_mode=round_mode, tile_m=64)
    b = Block(cfg)
    b.step()
    torch.cuda.synchronize()
    i = {k: f64(v) for k, v in b.inp.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    h = b.plan.to_host()
    plan = oracle.build_plan(f64(b.logits), K, round_mode, 64)
    assert np.array_equal(h["row_token"], plan["row_token"])
    X, tol = i["X"], TOL[dtype]
    fw = oracle.layer_forward(X, i["W_gate"], i["W_up"], i["W_down"], plan)
    idx = h["topk_idx"].reshape(T, K)
    rl = ob.router_losses(f64(b.logits), idx, 2, b.off.cpu().numpy())
    assert np.array_equal(b.counts.cpu().numpy(), rl["counts"])
    assert_close("loss", f64(b.loss), rl["loss"], 1e-5)
    shared, z = ob.linear_forward(X, f64(b.Wgu), f64(b.bgu), None, "swiglu")
    out = X + ob.dropout(fw["out"], b.p, 1234, 5678) + shared @ f64(b.Wd).T
    assert_close("out", f64(b.out), out, tol)
    # gradients
    dY = i["dY"]
    dact, dWd, _, _ = ob.linear_backward(dY, shared, f64(b.Wd), None)
    dXs, dWgu, dbgu, _ = ob.linear_backward(dact, X, f64(b.Wgu), z, "swiglu")
    aux = ob.router_losses_backward([40.0, 3.0], f64(b.logits), K, rl["counts"], rl["tokens"], 2, b.off.cpu().numpy())
    assert_close("aux", f64(b.aux), aux, 1e-4)
    bw = oracle.layer_backward(ob.dropout(dY, b.p, 1234, 5678), X, i["W_gate"], i["W_up"], i["W_down"], plan, W_r=i["W_r"])
    dL = bw["dLogits"] + aux
    stack = lambda k: np.stack([bw[k][e] for e in range(E)])  # noqa: E731
    for name, got, ref in (("dWd", b.dWd, dWd), ("dWgu", b.dWgu, dWgu), ("dbgu", b.dbgu, dbgu), ("dXs", b.dXs, dXs),
                           ("dLogits", b.dL, dL), ("dX", b.dX, bw["dX"] + aux @ i["W_r"]), ("dW_r", b.dWr, dL.T @ X),
                           ("dW_gate", b.dWg, stack("dW_gate")), ("dW_down", b.dWdn, stack("dW_down"))):
        assert_close(name, f64(got), ref, tol)


def test_backward_aux_without_router_weights_and_with_null_aux():
    """aux NULL is moe_backward bit for bit; without W_r only dLogits receives the sum."""
    cfg = wl.small_shape(T=200, d=128, E=10, K=2, n=64, dtype="bf16", backward=True, seed=5)
    b = Block(cfg)
    b.step()
    i = b.inp

    def run(aux, W_r, dWr, plain=False):
        o = [torch.empty_like(t) for t in (b.dX, b.dWg, b.dWu, b.dWdn, b.dS, b.dL, b.dWr)]
        a = (i["X"], W_r, i["W_gate"], i["W_up"], i["W_down"], b.plan, b.H)
        if plain:
            B.moe_backward(b.dims, b.dYm, *a, *o[:6], o[6] if dWr else None, *b.ws[B.OP_BACKWARD])
        else:
            B.moe_backward_aux(b.dims, b.dYm, *a, aux, *o[:6], o[6] if dWr else None, *b.ws[B.OP_BACKWARD])
        return o

    for x, y in zip(run(None, i["W_r"], True), run(None, i["W_r"], True, plain=True)):
        assert torch.equal(x, y)
    base, only = run(None, None, False), run(b.aux, None, False)
    assert torch.equal(base[0], only[0]) and torch.equal(only[5], base[5] + b.aux)
    # W_r without dW_r: the same dX as with it
    assert torch.equal(run(b.aux, i["W_r"], False)[0], run(b.aux, i["W_r"], True)[0])


def test_block_graph_replays_match_eager():
    b = Block(wl.small_shape(T=400, d=256, E=8, K=2, n=128, dtype="bf16", backward=True, seed=12))
    check_replays(b.step, b.outs())


# E a multiple of the stage's 64 (32) rows of W_r and not, one stage to sixteen; 4096 x 4096 in bf16 fills the
# chip with 256 x 256 tiles
@pytest.mark.parametrize("T,d,E,dtype", [
    (500, 256, 67, "f32"), (500, 256, 130, "f32"), (333, 320, 250, "f32"), (500, 256, 256, "f32"), (300, 192, 384, "f32"), (200, 128, 1001, "f32"),
    (500, 256, 67, "bf16"), (500, 256, 130, "bf16"), (333, 320, 250, "bf16"), (500, 256, 256, "bf16"), (300, 192, 384, "bf16"), (200, 128, 1001, "bf16"),
    (4096, 4096, 379, "bf16"), (4090, 4096, 384, "bf16"),
])
def test_backward_aux_of_many_experts(T, d, E, dtype):
    """dX is the expert path's (the call without W_r) plus dLogits W_r with dLogits rounded to the type: a
    product of E terms on top of a rounded value, rounded once more."""
    cfg = wl.small_shape(T=T, d=d, E=E, K=2, n=64, dtype=dtype, backward=True, seed=E)
    b = Block(cfg)
    b.step()
    i, aux = b.inp, torch.randn(T, E, generator=torch.Generator(device="cuda").manual_seed(E), device="cuda")

    def run(W_r, dWr):
        o = [torch.full_like(t, 7.0) for t in (b.dX, b.dWg, b.dWu, b.dWdn, b.dS, b.dL, b.dWr)]
        B.moe_backward_aux(b.dims, b.dYm, i["X"], W_r, i["W_gate"], i["W_up"], i["W_down"], b.plan, b.H, aux, *o[:6],
                           o[6] if dWr else None, *b.ws[B.OP_BACKWARD])
        return o

    only, full = run(None, False), run(i["W_r"], True)
    assert torch.equal(only[5], full[5])
    X = i["X"].double()
    L, W, base = full[5].to(cfg.torch_dtype).double(), i["W_r"].double(), only[0].double()
    h = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for name, got, first, A, C in (("dX", full[0], base, L, W), ("dW_r", full[6], 0 * W, L.t(), X)):
        ref = first + A @ C
        err = (A.shape[1] + 8) * 2.0 ** -23 * (first.abs() + A.abs() @ C.abs())
        off, tol = (got.double() - ref).abs(), h * (ref.abs() + err) + err
        assert bool((off <= tol).all()), "%s: worst %.3g" % (name, (off / tol.clamp(min=1e-30)).max().item())
        # the product is not lost among the rounding
        assert ((A @ C).abs() > tol).float().mean().item() > 0.5
