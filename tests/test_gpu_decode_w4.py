"""moe_decode_w4 against the float64 oracle on the weights' values, and against moe_decode."""
import numpy as np
import pytest
import torch

import oracle
from block_util import check_replays, f64
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from oracle import w4 as ow
from parity import TOL, assert_close
from test_gpu_w4 import FORMATS, random_w4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


class Layer:
    def __init__(self, T, d, n, E, K, fmt, group, seed=0, bias=True, skew=0.0):
        self.dims = B.make_dims(T, d, n, E, K, "bf16")
        self.T, self.d, self.n, self.E, self.K = T, d, n, E, K
        self.gate, _, _, self.Vg = random_w4(E * n, d, fmt, group, seed + 1)
        self.up, _, _, self.Vu = random_w4(E * n, d, fmt, group, seed + 2)
        self.down, _, _, self.Vd = random_w4(E * d, n, fmt, group, seed + 3)
        g = torch.Generator().manual_seed(seed + T)
        self.X = torch.randn(T, d, generator=g).bfloat16().cuda()
        self.W_r = (torch.randn(E, d, generator=g) * 0.05).bfloat16().cuda()
        self.bias = (torch.randn(E, generator=g) - skew * torch.arange(E)).cuda() if bias else None
        self.logits, self.idx = torch.empty(T, E, device="cuda"), torch.empty(T, K, dtype=torch.int32, device="cuda")
        self.w, self.out = torch.empty(T, K, device="cuda"), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
        self.ws = B.workspace(self.dims, B.OP_DECODE)

    def step(self):
        B.moe_decode_w4(self.dims, self.X, self.W_r, self.bias, self.gate, self.up, self.down, self.logits, self.idx, self.w,
                        self.out, *self.ws)

    def values(self):
        return self.Vg.reshape(self.E, self.n, self.d), self.Vu.reshape(self.E, self.n, self.d), self.Vd.reshape(self.E, self.d, self.n)

    def check(self):
        self.step()
        torch.cuda.synchronize()
        X = f64(self.X)
        logits = X @ f64(self.W_r).T + (f64(self.bias) if self.bias is not None else 0.0)
        assert_close("logits", f64(self.logits), logits, 1e-5)
        plan = oracle.build_plan(f64(self.logits), self.K)
        idx = oracle.topk_select(f64(self.logits), self.K)
        assert np.array_equal(self.idx.cpu().numpy(), np.asarray(idx).reshape(self.T, self.K))
        Vg, Vu, Vd = self.values()
        fw = oracle.layer_forward(X, Vg, Vu, Vd, plan)
        assert_close("out", f64(self.out), fw["out"], TOL["bf16"])
        # a wrong group, row or code would show in some column: every token's error stays far below its size
        err = np.abs(f64(self.out) - fw["out"]).max(axis=1)
        assert np.all(err <= 0.03 * np.sqrt((fw["out"] ** 2).mean(axis=1)) + 1e-6), err


# reductions of whole blocks of 128 and of one half; one to many tokens an expert (over 16 and 32: several passes);
# by pairs (T = 1, 2 T K <= E, or small weights) and by experts (over 1024 pairs, or over 64 MB read again)
@pytest.mark.parametrize("T,d,n,E,K,skew", [
    (2, 256, 128, 8, 2, 0.0), (4, 320, 192, 40, 5, 0.0), (1, 128, 64, 16, 16, 0.0), (7, 1088, 448, 256, 8, 0.0), (1, 64, 2048, 1024, 3, 0.0), (1, 192, 128, 3, 2, 0.0),
    (49, 128, 64, 130, 2, 0.0), (300, 64, 64, 5, 4, 0.2), (1024, 128, 64, 40, 2, 0.0), (520, 192, 448, 3, 2, 0.0), (1, 40960, 64, 2, 1, 0.0), (1, 64, 40960, 2, 1, 0.0),
    (1, 64, 64, 4, 1, 0.0), (1, 1536, 256, 16, 8, 0.0), (8, 320, 192, 12, 2, 0.0), (3, 128, 64, 1, 1, 0.0), (40, 192, 128, 5, 2, 0.5),
    (100, 256, 320, 6, 3, 1.0), (17, 2048, 128, 8, 4, 0.0), (64, 448, 704, 8, 2, 0.3),
    (100, 256, 640, 6, 3, 1.0), (64, 1088, 704, 8, 2, 0.3), (33, 704, 1088, 5, 5, 0.0), (512, 128, 64, 3, 2, 0.0),
])
@pytest.mark.parametrize("fmt,group", FORMATS)
def test_decode_matches_oracle(T, d, n, E, K, skew, fmt, group):
    up = lambda v: -(-v // max(group, 64)) * max(group, 64)  # noqa: E731
    Layer(T, up(d), up(n), E, K, fmt, group, skew=skew).check()


def test_fp4_equals_the_expanded_weights():
    """FP4 values are exact in bf16: moe_decode on them differs by the order of fp32 sums only."""
    L = Layer(6, 512, 256, 8, 2, "fp4", 32, bias=False)
    L.step()
    Vg, Vu, Vd = (torch.from_numpy(v).bfloat16().cuda().contiguous() for v in L.values())
    out = torch.empty_like(L.out)
    logits, idx, w = torch.empty_like(L.logits), torch.empty_like(L.idx), torch.empty_like(L.w)
    B.moe_decode(L.dims, L.X, L.W_r, None, Vg, Vu, Vd, logits, idx, w, out, *B.workspace(L.dims, B.OP_DECODE))
    B.moe_decode_status()
    assert_close("logits", f64(L.logits), f64(logits), 1e-5)
    assert torch.equal(idx, L.idx)
    assert_close("topk_w", f64(L.w), f64(w), 1e-5)
    assert_close("out", f64(L.out), f64(out), TOL["bf16"] / 4)


@pytest.mark.parametrize("fmt,group", [("fp4", 32), ("int4", 128)])
def test_graph_replays_match_eager(fmt, group):
    L = Layer(9, 256, 128, 8, 2, fmt, group)
    check_replays(L.step, dict(out=L.out, logits=L.logits, idx=L.idx, w=L.w))
    torch.cuda.synchronize()


def test_results_repeat_bit_for_bit():
    L = Layer(33, 512, 256, 16, 4, "int4", 64)
    L.step()
    first = L.out.clone()
    for _ in range(3):
        L.out.zero_()
        L.step()
        assert torch.equal(L.out, first)
    torch.cuda.synchronize()


def test_quantised_layer_end_to_end():
    """bf16 expert weights quantised by the library, decoded: against the layer on the values that they took."""
    T, d, n, E, K = 5, 256, 128, 6, 2
    L = Layer(T, d, n, E, K, "int4", 32)
    g = torch.Generator().manual_seed(3)
    for name, rows, k in (("gate", E * n, d), ("up", E * n, d), ("down", E * d, n)):
        w = (torch.randn(rows, k, generator=g) / k ** 0.5).bfloat16().cuda()
        q = B.make_w4(rows, k, "int4", 32)
        B.moe_quantize_w4(w, q)
        v = torch.empty(rows, k, device="cuda")
        B.moe_dequantize_w4(q, v)
        setattr(L, name, q)
        setattr(L, "V" + name[0], f64(v))
        # the quantisation itself is worth half a step of a seventh of the largest of 32: about a tenth of the deviation
        assert float((v - w.float()).norm() / w.float().norm()) < 0.15
    L.check()
    assert ow.E2M1[7] == 6.0


@pytest.mark.parametrize("T,K,E", [(2, 2, 520), (600, 2, 520)])
def test_code_offsets_past_32_bits(T, K, E):
    """4.4e9 bytes of codes a matrix, every token on the last two experts, by pairs and by experts."""
    d = n = 4096
    g = torch.Generator(device="cuda").manual_seed(5)

    def weights(rows, k):
        codes = torch.randint(0, 256, (rows, k // 2), dtype=torch.uint8, device="cuda", generator=g)
        scales = torch.randint(118, 121, (k // 128, rows, 4), dtype=torch.uint8, device="cuda", generator=g)
        return B.W4(codes, scales, "fp4", 32)

    def values(w, rows):  # of the last two experts
        v = torch.empty(2, rows, w.K, device="cuda")
        B.moe_dequantize_w4(B.W4(w.codes[-2 * rows:].contiguous(), w.scales[:, -2 * rows:].contiguous(), "fp4", 32), v)
        return v.double()

    gate, up, down = weights(E * n, d), weights(E * n, d), weights(E * d, n)
    assert gate.codes.numel() > 1 << 32
    X = torch.randn(T, d, device="cuda", generator=g).bfloat16()
    W_r = torch.zeros(E, d, dtype=torch.bfloat16, device="cuda")
    bias = torch.zeros(E, device="cuda")
    bias[-2:] = torch.tensor([3.0, 3.5])
    dims = B.make_dims(T, d, n, E, K)
    logits, idx = torch.empty(T, E, device="cuda"), torch.empty(T, K, dtype=torch.int32, device="cuda")
    w, out = torch.empty(T, K, device="cuda"), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    B.moe_decode_w4(dims, X, W_r, bias, gate, up, down, logits, idx, w, out, *B.workspace(dims, B.OP_DECODE))
    assert torch.equal(idx, torch.tensor([E - 1, E - 2], dtype=torch.int32, device="cuda").expand(T, 2))
    x, Vg, Vu, Vd = X.double(), values(gate, n), values(up, n), values(down, d)
    ref = sum(w[:, 1 - e:2 - e].double() * ((torch.nn.functional.silu(x @ Vg[e].T) * (x @ Vu[e].T)) @ Vd[e].T) for e in range(2))
    assert_close("out", f64(out), f64(ref), TOL["bf16"])


@pytest.mark.parametrize("T", [3, 200])
def test_a_token_that_is_not_finite_stays_alone(T):
    L = Layer(T, 256, 640, 6, 3, "int4", 64)
    L.step()
    want = [t.clone() for t in (L.logits, L.idx, L.w, L.out)]
    L.X[1, 7] = float("nan")
    L.step()
    keep = [t for t in range(T) if t != 1]
    for got, ref in zip((L.logits, L.idx, L.w, L.out), want):
        assert torch.equal(got[keep], ref[keep])
    assert bool(L.logits[1].isnan().all()) and bool(L.out[1].isnan().all())
    assert sorted(set(L.idx[1].tolist())) == [0, 1, 2]  # (of equal keys the lowest ids)


@pytest.mark.parametrize("T", [2, 200])
def test_calls_on_two_streams_with_their_own_workspaces(T):
    layers = [Layer(T, 256, 640, 6, 3, "fp4", 32, seed=k) for k in (1, 2)]
    for L in layers:
        L.step()
    torch.cuda.synchronize()
    want = [L.out.clone() for L in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(5):
        for L in layers:
            L.out.zero_()
        torch.cuda.synchronize()
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                L.step()
        torch.cuda.synchronize()
        for L, o in zip(layers, want):
            assert torch.equal(L.out, o)
