"""Pins of the block oracle (dense projection, router losses, dropout) that do not use its own
formulas: central differences, torch autograd in float64, published generator outputs, statistics."""
import numpy as np
import pytest
import torch

from oracle import block as ob

RNG = np.random.default_rng(5)


def numeric_grad(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + h
        a = f()
        x[i] = old - h
        b = f()
        x[i] = old
        g[i] = (a - b) / (2 * h)
    return g


@pytest.mark.parametrize("act", ob.ACTS)
def test_linear_gradients_match_central_differences(act):
    M, N, K = 3, 4, 5
    NW = 2 * N if act == "swiglu" else N
    X, W, b = RNG.normal(size=(M, K)), RNG.normal(size=(NW, K)), RNG.normal(size=NW)
    R, dY = RNG.normal(size=(M, N)), RNG.normal(size=(M, N))
    f = lambda: float(np.sum(dY * ob.linear_forward(X, W, b, R, act)[0]))  # noqa: E731
    _, z = ob.linear_forward(X, W, b, R, act)
    dX, dW, db, _ = ob.linear_backward(dY, X, W, z, act)
    # central differences: truncation ~ h^2, cancellation ~ 2^-52 / h
    for got, var in ((dX, X), (dW, W), (db, b), (dY, R)):
        assert np.allclose(got, numeric_grad(f, var), rtol=0, atol=2e-8)


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_activations_match_torch(act):
    z = np.linspace(-12, 12, 97)[None]
    ref = {"relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[act](torch.tensor(z))
    assert np.allclose(ob.activation(z, act), ref.numpy(), rtol=1e-13, atol=1e-15)


def test_relu_gradient_selects():
    """Where a unit is off its gradient is 0 for any dy, as torch's own."""
    z = np.array([[-1.0, 0.0, 2.0, -3.0, -0.0, 1.0]])
    dy = np.array([[np.inf, np.nan, np.inf, -np.inf, 5.0, -2.0]])
    x = torch.tensor(z, requires_grad=True)
    torch.relu(x).backward(torch.tensor(dy))
    got = ob.activation_backward(dy, z, "relu")
    assert np.array_equal(got, [[0.0, 0.0, np.inf, 0.0, 0.0, -2.0]]) and np.array_equal(got, x.grad.numpy())


def test_router_losses_even_load_is_one_and_matches_autograd():
    T, E, K = 24, 6, 2
    logits = torch.zeros(T, E, dtype=torch.float64)
    idx = np.array([[t % E, (t + 1) % E] for t in range(T)])
    r = ob.router_losses(logits.numpy(), idx)
    assert np.isclose(r["loss"][0], 1.0) and np.isclose(r["loss"][1], np.log(E) ** 2)
    x = torch.tensor(RNG.normal(size=(T, E)), requires_grad=True)
    idx = torch.topk(x, K).indices.numpy()
    off, mask = [0, 7, 7, 20], RNG.random(T) > 0.2
    r = ob.router_losses(x.detach().numpy(), idx, 3, off, mask)
    # the losses written with torch, token by token
    p, lse = torch.softmax(x, 1), torch.logsumexp(x, 1)
    n = sum(int(mask[t]) for t in range(20))
    bal, z = 0.0, 0.0
    for s in range(3):
        rows = [t for t in range(off[s], off[s + 1]) if mask[t]]
        for e in range(E):
            share = sum(int(e in idx[t]) for t in rows)
            if rows:
                bal = bal + E * share / (K * len(rows) * n) * sum(p[t, e] for t in rows)
        z = z + sum(lse[t] ** 2 for t in rows) / n
    assert np.isclose(float(bal), r["loss"][0], rtol=1e-12) and np.isclose(float(z), r["loss"][1], rtol=1e-12)
    (3.0 * bal + 0.5 * z).backward()
    g = ob.router_losses_backward([3.0, 0.5], x.detach().numpy(), K, r["counts"], r["tokens"], 3, off, mask)
    assert np.allclose(g, x.grad.numpy(), rtol=1e-10, atol=1e-14)


def test_router_losses_of_masked_and_empty_rows():
    x = np.array([[0.0, -np.inf, 1.0], [-np.inf] * 3, [1.0, 2.0, 3.0]])
    idx = np.array([[2], [0], [2]])
    r = ob.router_losses(x, idx)
    assert np.isneginf(r["lse"][1]) and np.all(np.isfinite(r["loss"])) and r["counts"].tolist() == [[1, 0, 2]]
    assert np.isclose(r["prob"].sum(), 2.0)
    g = ob.router_losses_backward([1.0, 1.0], x, 1, r["counts"], r["tokens"])
    assert np.all(g[1] == 0) and g[0, 1] == 0 and np.all(np.isfinite(g))
    none = ob.router_losses(x, idx, 1, None, np.zeros(3))
    assert none["loss"].tolist() == [0.0, 0.0] and none["tokens"].tolist() == [0]


@pytest.mark.parametrize("counter,key,want", [
    ([0, 0, 0, 0], [0, 0], [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_philox_published_outputs(counter, key, want):
    """The authors' known answers for ten rounds: zeros, ones, digits of pi."""
    assert [int(v) for v in ob.philox4x32(counter, key)] == want


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9, 1.0])
def test_dropout_rate_scale_and_independence(p):
    R, C = 500, 403
    keep = ob.dropout_keep(R, C, p, 1234567890123, 77)
    rate = 1 - ob.dropout_threshold(p) / 65536
    # binomial: within 5 standard deviations
    assert abs(keep.mean() - rate) <= 5 * np.sqrt(max(rate * (1 - rate), 0) / keep.size)
    assert np.abs(keep.mean(axis=0) - rate).max() <= 6 * np.sqrt(0.25 / R)
    x = np.full((R, C), np.inf)
    y = ob.dropout(np.ones((R, C)), p, 1234567890123, 77, residual=np.full((R, C), 2.0))
    assert np.allclose(np.unique(y), sorted({2.0} if rate == 0 else ({3.0} if rate == 1 else {2.0, 2.0 + 1 / rate})))
    if rate < 1:
        with np.errstate(invalid="ignore"):
            assert np.all(ob.dropout(x, p, 1234567890123, 77)[~keep] == 0)
        other = ob.dropout_keep(R, C, p, 1234567890123, 78)
        if rate > 0:
            assert abs((keep & other).mean() - rate * rate) <= 6 * np.sqrt(0.25 / keep.size)
