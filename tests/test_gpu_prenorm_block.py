"""The operators of a pre-norm block run together through the library: a training step (norm, layer, their
backward, clipping of every gradient) and a decoding step on 4-bit weights (norm, routed experts, shared expert, the
next norm), against float64."""
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
from test_gpu_w4 import random_w4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


class Training:
    """s = x + r, y = norm(s), out = s + moe(y); loss = <dOut, out>; then all gradients cut to max_norm."""

    def __init__(self, cfg, kind, max_norm):
        self.cfg, self.kind, self.max_norm = cfg, kind, max_norm
        T, d, E, n = cfg.T, cfg.d, cfg.E, cfg.n
        self.inp = wl.make_inputs(cfg, device="cuda", with_grad_out=True)
        dt, f = cfg.torch_dtype, torch.float32
        g = torch.Generator(device="cuda").manual_seed(8)
        self.r = torch.randn(T, d, generator=g, device="cuda").to(dt)
        self.w, self.b = torch.randn(d, generator=g, device="cuda") * 0.2 + 1, torch.randn(d, generator=g, device="cuda") * 0.1
        self.dims = B.make_dims(T, d, n, E, cfg.K, cfg.dtype)
        self.nd = B.make_norm_dims(T, d, cfg.dtype, kind)
        self.plan = B.Plan(self.dims)
        R = self.plan.R_max
        e = lambda *s, t=dt: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        self.s, self.y, self.mean, self.rstd = e(T, d), e(T, d), e(T, t=f), e(T, t=f)
        self.logits, self.H, self.m = e(T, E, t=f), e(R, 2 * n), e(T, d)
        self.dy, self.dx, self.dw, self.db = e(T, d), e(T, d), e(d, t=f), e(d, t=f)
        self.dWg, self.dWu, self.dWd, self.dWr = (torch.empty_like(self.inp[k]) for k in ("W_gate", "W_up", "W_down", "W_r"))
        self.dS, self.dL = e(R, t=f), e(T, E, t=f)
        self.norm = e(1, t=f)
        self.raw = [self.dWg, self.dWu, self.dWd, self.dWr, self.dw, self.db]
        self.cut = [torch.empty_like(t) for t in self.raw]
        self.grads = B.Gradients(self.raw, self.cut)
        self.ws = {op: B.workspace(self.dims, op) for op in (B.OP_FORWARD, B.OP_BACKWARD)}
        self.wn, self.wg = B.norm_workspace(self.nd), B.grad_workspace(self.grads)

    def step(self):
        i = self.inp
        B.moe_norm(self.nd, i["X"], self.r, self.w, self.b, self.s, self.y, self.mean, self.rstd)
        B.moe_forward(self.dims, self.y, i["W_r"], i["bias"], i["W_gate"], i["W_up"], i["W_down"], self.logits, self.plan, self.H,
                      self.m, *self.ws[B.OP_FORWARD])
        B.moe_backward(self.dims, i["dY"], self.y, i["W_r"], i["W_gate"], i["W_up"], i["W_down"], self.plan, self.H, self.dy, self.dWg,
                       self.dWu, self.dWd, self.dS, self.dL, self.dWr, *self.ws[B.OP_BACKWARD])
        mean = self.mean if self.kind == "layer" else None
        B.moe_norm_backward(self.nd, self.dy, self.s, self.w, mean, self.rstd, i["dY"], self.dx, self.dw, self.db, *self.wn)
        B.moe_grad_clip(self.grads, self.max_norm, None, self.norm, *self.wg)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,E,K,n", [(300, 128, 12, 2, 64), (1100, 320, 6, 2, 192)])
def test_training_step(T, d, E, K, n, dtype, kind):
    t = Training(wl.small_shape(T=T, d=d, E=E, K=K, n=n, dtype=dtype, backward=True, seed=41), kind, 1.5)
    t.step()
    torch.cuda.synchronize()
    tol, i = TOL[dtype], {k: f64(v) for k, v in t.inp.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    S = f64((t.inp["X"].float() + t.r.float()).to(t.cfg.torch_dtype))
    y = ob.norm(S, f64(t.w), f64(t.b), 1e-5, kind)
    assert_close("y", f64(t.y), y, tol)
    plan = oracle.build_plan(f64(t.logits), K)
    assert np.array_equal(t.plan.to_host()["row_token"], plan["row_token"])
    fw = oracle.layer_forward(y, i["W_gate"], i["W_up"], i["W_down"], plan)
    assert_close("moe", f64(t.m), fw["out"], tol)
    bw = oracle.layer_backward(i["dY"], y, i["W_gate"], i["W_up"], i["W_down"], plan, W_r=i["W_r"])
    mean, rstd = ob.norm_stats(S, 1e-5, kind)
    dx, dw, db = ob.norm_backward(bw["dX"], S, f64(t.w), mean, rstd, i["dY"], kind)
    stack = lambda k: np.stack([bw[k][e] for e in range(E)])  # noqa: E731
    ref = [stack("dW_gate"), stack("dW_up"), stack("dW_down"), bw["dW_r"], dw, db]
    assert_close("dx", f64(t.dx), dx, tol)
    for name, got, want in zip(("dW_gate", "dW_up", "dW_down", "dW_r", "dweight", "dbias"), t.raw, ref):
        assert_close(name, f64(got), want, tol)
    norm = np.sqrt(sum((r ** 2).sum() for r in ref))
    assert norm > 1.5 and abs(float(t.norm) - norm) <= tol * norm
    true = np.sqrt(sum((f64(g) ** 2).sum() for g in t.raw))
    assert abs(float(t.norm) - true) <= 2.0 ** -23 * true
    for got, raw in zip(t.cut, t.raw):
        assert_close("clipped", f64(got), f64(raw) * (1.5 / true), 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -21)


def test_training_graph_replays_match_eager():
    t = Training(wl.small_shape(T=400, d=256, E=8, K=2, n=128, dtype="bf16", backward=True, seed=12), "layer", 2.0)
    outs = dict(y=t.y, m=t.m, dx=t.dx, norm=t.norm)
    outs.update({"cut%d" % k: v for k, v in enumerate(t.cut)})
    check_replays(t.step, outs)


class Serving:
    """s = x + r, y = norm(s); out = moe(y) + down(swiglu(gate_up(y))); s2 = out + s, y2 = norm(s2)."""

    def __init__(self, T, d, n, E, K, fmt, group, kind="rms"):
        self.T, self.d, self.n, self.E, self.K, self.kind, self.fmt = T, d, n, E, K, kind, fmt
        g = torch.Generator().manual_seed(T + d)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x, self.r = rn(T, d).bfloat16().cuda(), rn(T, d).bfloat16().cuda()
        self.w, self.w2 = (rn(d) * 0.2 + 1).bfloat16().cuda(), (rn(d) * 0.2 + 1).bfloat16().cuda()
        self.W_r = (rn(E, d) * 0.05).bfloat16().cuda()
        self.gate, _, _, self.Vg = random_w4(E * n, d, fmt, group, 1)
        self.up, _, _, self.Vu = random_w4(E * n, d, fmt, group, 2)
        self.down, _, _, self.Vd = random_w4(E * d, n, fmt, group, 3)
        self.sgu, _, _, self.Vsgu = random_w4(2 * n, d, fmt, group, 4)
        self.sd, _, _, self.Vsd = random_w4(d, n, fmt, group, 5)
        self.nd = B.make_norm_dims(T, d, "bf16", kind, wtype="bf16")
        self.dims = B.make_dims(T, d, n, E, K)
        self.lgu, self.ld = B.make_linear_dims(T, n, d, "bf16", "swiglu"), B.make_linear_dims(T, d, n)
        e = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        self.s, self.y, self.m, self.h, self.out, self.s2, self.y2 = e(T, d), e(T, d), e(T, d), e(T, n), e(T, d), e(T, d), e(T, d)
        self.logits, self.idx, self.tw = e(T, E, t=torch.float32), e(T, K, t=torch.int32), e(T, K, t=torch.float32)
        self.wd, self.w1, self.w3 = B.workspace(self.dims, B.OP_DECODE), B.linear_w4_workspace(self.lgu), B.linear_w4_workspace(self.ld)

    def step(self):
        B.moe_norm(self.nd, self.x, self.r, self.w, None, self.s, self.y, None, None)
        B.moe_decode_w4(self.dims, self.y, self.W_r, None, self.gate, self.up, self.down, self.logits, self.idx, self.tw, self.m, *self.wd)
        B.moe_linear_w4(self.lgu, self.y, self.sgu, None, None, self.h, *self.w1)
        B.moe_linear_w4(self.ld, self.h, self.sd, None, self.m, self.out, *self.w3)
        B.moe_norm(self.nd, self.out, self.s, self.w2, None, self.s2, self.y2, None, None)


@pytest.mark.parametrize("T,d,n,E,K,fmt,group", [(1, 512, 256, 8, 2, "fp4", 32), (5, 256, 128, 6, 2, "int4", 128), (70, 192, 192, 4, 2, "int4", 32)])
def test_decoding_step(T, d, n, E, K, fmt, group):
    s = Serving(T, d, n, E, K, fmt, group)
    s.step()
    torch.cuda.synchronize()
    tol = TOL["bf16"]
    S = f64((s.x.float() + s.r.float()).bfloat16())
    y = ob.norm(S, f64(s.w), None, 1e-5, s.kind)
    assert_close("y", f64(s.y), y, tol)
    plan = oracle.build_plan(f64(s.logits), K)
    moe = oracle.layer_forward(y, s.Vg.reshape(E, n, d), s.Vu.reshape(E, n, d), s.Vd.reshape(E, d, n), plan)["out"]
    shared = ob.linear_forward(y, s.Vsgu, None, None, "swiglu")[0] @ s.Vsd.T
    assert_close("out", f64(s.out), moe + shared, tol)
    assert torch.equal(s.s2, (s.out.float() + s.s.float()).bfloat16())
    assert_close("y2", f64(s.y2), ob.norm(f64(s.s2), f64(s.w2), None, 1e-5, s.kind), tol)


def test_decoding_graph_replays_match_eager():
    s = Serving(3, 256, 128, 8, 2, "int4", 64)
    check_replays(s.step, dict(out=s.out, y2=s.y2, logits=s.logits, idx=s.idx))


def test_two_captured_graphs_share_workspaces():
    """Two steps captured apart with the same workspaces, replayed in turn on one stream."""
    a, b = Serving(3, 256, 128, 8, 2, "fp4", 32), Serving(3, 256, 128, 8, 2, "fp4", 32)
    b.x.copy_(-a.x)
    b.wd, b.w1, b.w3 = a.wd, a.w1, a.w3
    want = []
    for t in (a, b):
        t.step()
        torch.cuda.synchronize()
        want.append((t.out.clone(), t.y2.clone()))
    graphs = []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            t.step()
        graphs.append(g)
    for _ in range(3):
        for t in (a, b):
            t.out.zero_()
            t.y2.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for t, (o, y2) in zip((a, b), want):
            assert torch.equal(t.out, o) and torch.equal(t.y2, y2)
