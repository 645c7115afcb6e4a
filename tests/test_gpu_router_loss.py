"""moe_router_loss and its gradient against the float64 oracle."""
import numpy as np
import pytest
import torch

from block_util import U32, assert_within, check_replays, f64
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from oracle import block as ob

pytestmark = pytest.mark.gpu
# relative error allowed to exp and log of the hardware and the products before them: the argument
# of exp is rounded once after scaling, |x - max| (here below 64) times 2^-24, plus a few steps
EXP = 64 * 2.0 ** -24 + 4 * U32


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield


class Case:
    def __init__(self, T, E, K, n_seq=1, off=None, masked=0.0, seed=0, logits=None, idx=None):
        g = torch.Generator().manual_seed(seed)
        self.T, self.E, self.K, self.S = T, E, K, n_seq
        x = torch.randn(T, E, generator=g) * 1.5 if logits is None else logits
        self.logits = x.cuda()
        self.idx = (torch.topk(torch.nan_to_num(x, nan=-1e9), K).indices if idx is None else idx).to(torch.int32)
        self.off = torch.tensor(off, dtype=torch.int32) if off is not None else None
        self.mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8) if masked else None
        self.dims = B.make_dims(T, 64, 64, E, K, "f32")
        c = lambda t: t.cuda() if t is not None else None  # noqa: E731
        self.d_idx, self.d_off, self.d_mask = c(self.idx), c(self.off), c(self.mask)
        f = dict(device="cuda")
        self.tokens, self.counts = torch.full((n_seq,), -1, dtype=torch.int32, **f), torch.full((n_seq, E), -1, dtype=torch.int32, **f)
        self.prob, self.lse, self.loss = torch.empty(n_seq, E, **f), torch.empty(T, **f), torch.empty(2, **f)
        self.dlogits, self.dloss = torch.full((T, E), 5.0, **f), torch.tensor([3.0, 0.25], **f)
        self.ws, self.nb = B.router_loss_workspace(self.dims, n_seq)
        self.ws.fill_(0xFF)

    def forward(self):
        B.moe_router_loss(self.dims, self.logits, self.d_idx, self.S, self.d_off, self.d_mask, self.tokens, self.counts,
                          self.prob, self.lse, self.loss, self.ws, self.nb)

    def backward(self):
        B.moe_router_loss_backward(self.dims, self.dloss, self.logits, self.S, self.d_off, self.d_mask, self.tokens,
                                   self.counts, self.lse, self.dlogits)

    def outs(self):
        return dict(tokens=self.tokens, counts=self.counts, prob=self.prob, lse=self.lse, loss=self.loss, dlogits=self.dlogits)

    def oracle(self):
        m = self.mask.numpy() if self.mask is not None else None
        off = self.off.numpy() if self.off is not None else None
        r = ob.router_losses(f64(self.logits), self.idx.numpy(), self.S, off, m)
        r["dlogits"] = ob.router_losses_backward(f64(self.dloss), f64(self.logits), self.K, r["counts"], r["tokens"], self.S, off, m)
        return r

    def check(self):
        self.forward()
        self.backward()
        torch.cuda.synchronize()
        r = self.oracle()
        assert np.array_equal(self.tokens.cpu().numpy(), r["tokens"])
        assert np.array_equal(self.counts.cpu().numpy(), r["counts"])
        lse = np.where(np.isneginf(r["lse"]), 0.0, r["lse"])
        got_lse = f64(self.lse)
        assert np.array_equal(np.isneginf(got_lse), np.isneginf(r["lse"]))
        # log(sum): the sum's relative error (E additions) becomes absolute, plus the roundings of
        # the logarithm (|log sum| <= 7) and of the result
        lse_err = EXP + (self.E + 20) * U32 + 4 * U32 * np.abs(lse)
        assert_within("lse", np.where(np.isneginf(got_lse), 0.0, got_lse), lse, lse_err)
        p_rel = 2 * EXP + (self.E + 70) * U32  # exp over its sum, then at most 64 additions per chunk
        assert_within("prob", f64(self.prob), r["prob"], p_rel * r["prob"] + 1e-37)
        z_rel = (2 * lse_err / np.maximum(np.abs(lse), 1e-3)).max() if lse.size else 0
        assert_within("loss", f64(self.loss), r["loss"], np.array([p_rel, z_rel + 70 * U32]) * r["loss"] + 1e-30)
        # the gradient: p's error (its exponent x - lse carries lse's), and the inner sum's
        p, _ = ob._softmax(f64(self.logits))
        n, d = max(1, r["tokens"].sum()), f64(self.dloss)
        tol = np.full(r["dlogits"].shape, 1e-37)
        off = [0, self.T] if self.off is None else self.off.tolist()
        for s in range(self.S):
            a = slice(off[s], off[s + 1])
            ts = r["tokens"][s]
            if not ts:
                continue
            mean = self.K * ts / self.E
            ex = np.abs(r["counts"][s] - mean) + U32 * (r["counts"][s] + mean)
            w = d[0] * self.E / (self.K * ts * n)
            size = w * (ex + (p[a] @ ex)[:, None]) + (2 * d[1] / n * np.abs(lse[a]))[:, None]
            tol[a] += p[a] * size * (2 * EXP + (self.E + 20) * U32 + 2 * lse_err[a])[:, None]
        assert_within("dlogits", f64(self.dlogits), r["dlogits"], tol)
        return r


@pytest.mark.parametrize("E,K", [(1, 1), (2, 1), (3, 2), (8, 2), (12, 3), (16, 4), (30, 5), (64, 6), (100, 8), (128, 8), (190, 8),
                                 (256, 8), (257, 4), (384, 8), (511, 16), (512, 8), (770, 2), (1024, 16)])
def test_every_row_layout(E, K):
    Case(T=131, E=E, K=K, seed=E).check()


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 129, 1000])
def test_lengths(T):
    Case(T=T, E=20, K=3, seed=T).check()


@pytest.mark.parametrize("T,off,masked", [
    (200, [0, 200], 0.3), (200, [0, 50, 50, 64, 128, 200], 0.0), (200, [0, 1, 2, 3, 199, 200], 0.2), (300, [10, 20, 250], 0.1),
    (70, [0, 0, 0, 0], 0.0), (70, [70, 70], 0.0), (129, [0, 64, 128, 129], 0.0), (100, list(range(101)), 0.1),
    (400, [5, 5, 300, 300, 300, 390, 390], 0.5),
])
def test_sequences_padding_and_masks(T, off, masked):
    r = Case(T=T, E=24, K=4, n_seq=len(off) - 1, off=off, masked=masked, seed=T + len(off)).check()
    assert len(r["tokens"]) == len(off) - 1


def test_all_tokens_masked_gives_zeros():
    c = Case(T=90, E=16, K=2, masked=2.0)
    c.check()
    assert not c.loss.any() and not c.dlogits.any() and not c.prob.any()


def test_masked_experts_rows_without_any_and_non_finite_rows():
    x = torch.randn(150, 40)
    x[:, 7] = -float("inf")
    x[3:20, 10:] = -float("inf")
    x[64] = -float("inf")
    x[149] = -float("inf")
    x[100, 5] = torch.finfo(torch.float32).min
    c = Case(T=150, E=40, K=2, logits=x)
    c.check()
    assert not c.dlogits[64].any() and not c.dlogits[:, 7].any()
    # a NaN or +infinity makes the losses NaN, and its own row of the gradient only
    y = torch.randn(150, 40)
    y[70, 3], y[90, 4] = float("nan"), float("inf")
    c = Case(T=150, E=40, K=2, logits=y)
    c.forward()
    c.backward()
    assert c.loss.isnan().all() and c.lse[70].isnan() and c.lse[90].isnan()
    fine = torch.ones(150, dtype=torch.bool, device="cuda")
    fine[[70, 90]] = False
    assert c.dlogits[fine].isfinite().all() and c.dlogits[~fine].isnan().any(1).all()


def test_large_logits_and_lowest_values():
    """Rows at the ends of fp32's range: the exponentials of the others are zero, nothing overflows."""
    big = torch.finfo(torch.float32).max
    x = torch.full((66, 9), -big)
    x[:, 4] = big
    x[1] = -big  # all equal, at the lowest value
    c = Case(T=66, E=9, K=1, logits=x)
    c.forward()
    torch.cuda.synchronize()
    p = f64(c.prob)[0]
    assert np.allclose(p, [1 / 9] * 4 + [65 + 1 / 9] + [1 / 9] * 4, rtol=1e-6)
    assert np.array_equal(c.counts.cpu().numpy()[0].sum(), 66)


def test_repeated_and_invalid_choices_are_counted_as_given():
    idx = torch.zeros(80, 3, dtype=torch.int32)
    idx[:, 1] = 5
    idx[:, 2] = 5       # the same expert twice
    idx[7] = torch.tensor([-1, 6, 1 << 30])  # none of them an expert
    c = Case(T=80, E=6, K=3, idx=idx)
    r = c.check()
    assert r["counts"][0].tolist() == [79, 0, 0, 0, 0, 158]


def test_gradient_against_differences():
    """loss(x + h v) - loss(x - h v) over 2 h against <dlogits, v>, the choice held fixed.  The loss is
    smooth; with h = 2^-6 the cubic term is below h^2 |v|^3 and fp32 noise below 2^-20 / h."""
    c = Case(T=500, E=32, K=4, seed=4)
    c.forward()
    c.backward()
    v = torch.randn(500, 32, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x0, h, val = c.logits.clone(), 2.0 ** -6, []
    for s in (1, -1):
        c.logits.copy_(x0 + s * h * v)
        c.forward()
        val.append((c.loss.double() * c.dloss.double()).sum().item())
    size = (3.0 + 0.25 * 16)
    assert abs((val[0] - val[1]) / (2 * h) - (c.dlogits.double() * v.double()).sum().item()) <= size * (h * h + 2.0 ** -20 / h)


def test_determinism_streams_and_graph():
    c = Case(T=3000, E=48, K=4, n_seq=4, off=[0, 700, 701, 2000, 2990], masked=0.1)

    def step():
        c.forward()
        c.backward()

    check_replays(step, c.outs())
    ref = {k: v.clone() for k, v in c.outs().items()}
    others = [Case(T=3000, E=48, K=4, n_seq=4, off=[0, 700, 701, 2000, 2990], masked=0.1) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in others]
    for o, s in zip(others, streams):
        with torch.cuda.stream(s):
            for _ in range(5):
                o.forward()
                o.backward()
    torch.cuda.synchronize()
    for o in others:
        for k, v in o.outs().items():
            assert torch.equal(v, ref[k]), k


def _cuts(T, lengths):
    """A table whose sequences have these lengths (the last one ends where they do, at most at T)."""
    off = [0]
    for n in lengths:
        off.append(min(T, off[-1] + n))
    return off


# chunks of many short sequences beside long ones: waves take the short pieces, the workgroup the long
@pytest.mark.parametrize("E,K", [(5, 2), (24, 4), (128, 8), (250, 3), (379, 6), (1000, 8)])
@pytest.mark.parametrize("lengths", [
    [1] * 64, [0, 3, 0, 0, 2, 1, 0, 7, 20, 5, 0, 4], [1, 1, 1, 40, 1, 1, 2, 30, 1, 1, 1, 50, 1], [5] * 40, [2, 300, 1, 1, 1, 1, 250, 3, 3, 3, 3],
], ids=["ones", "gaps", "mixed", "fives", "long"])
def test_many_sequences_in_a_chunk(E, K, lengths):
    T = sum(lengths) + 9
    Case(T=T, E=E, K=K, n_seq=len(lengths), off=_cuts(T, lengths), masked=0.2, seed=E + len(lengths)).check()


@pytest.mark.parametrize("T,E", [(40, 16), (1300, 16), (700, 300)])
def test_more_sequences_than_the_table_in_shared_memory_holds(T, E):
    off = np.sort(np.random.default_rng(T).integers(0, T + 1, 1500)).tolist()
    Case(T=T, E=E, K=2, n_seq=1499, off=off, masked=0.1, seed=T).check()


@pytest.mark.parametrize("T,lengths", [(60, [2] * 25), (900, [1, 2, 70, 3] * 11)])
def test_many_sequences_replayed(T, lengths):
    c = Case(T=T, E=48, K=4, n_seq=len(lengths), off=_cuts(T, lengths), masked=0.2, seed=T)

    def step():
        c.forward()
        c.backward()

    check_replays(step, c.outs())


@pytest.mark.parametrize("E,n_seq", [(256, 1 << 20), (16, 1 << 20), (40, (1 << 16) + 1)])
def test_as_many_sequences_as_allowed(E, n_seq):
    """Nearly all of them empty: the others give what they give in a table without the empty ones."""
    T, K = 3000, 4
    at = [0, 5, (1 << 16) - 1, n_seq // 2 + 3 if n_seq > 1 << 17 else 1 << 15, n_seq - 1]
    at, cuts = sorted(at), [0, 10, 700, 701, 2000, 2990]
    small = Case(T=T, E=E, K=K, n_seq=5, off=cuts, masked=0.1, seed=3)
    small.check()
    off = np.zeros(n_seq + 1, np.int32)
    for s, cut in zip(at, cuts[1:]):
        off[s + 1:] = cut
    big = Case(T=T, E=E, K=K, n_seq=n_seq, off=off, masked=0.1, seed=3)
    big.forward()
    big.backward()
    torch.cuda.synchronize()
    rows = torch.tensor(at, device="cuda")
    assert torch.equal(big.tokens[rows], small.tokens) and big.tokens.sum() == small.tokens.sum() and (big.tokens >= 0).all()
    assert torch.equal(big.counts[rows], small.counts) and big.counts.sum() == small.counts.sum() and (big.counts >= 0).all()
    # the order of additions may differ: each sum of at most T terms twice within its bound
    for name in ("prob", "lse", "loss", "dlogits"):
        a, b = getattr(big, name), getattr(small, name)
        if name == "prob":
            assert ((a != 0).any(1).sum() == 5) and bool((a >= 0).all())
            a = a[rows]
        assert_within(name, f64(a), f64(b), (2 * EXP + 2 * (E + 70) * U32) * np.abs(f64(b)) + 1e-30)
