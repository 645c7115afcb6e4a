"""Float64 numpy statement of what stands beside the MoE layer in a block: the dense projection with
its epilogue, the router losses and counter-based dropout.  Test infrastructure only."""
import math

import numpy as np

ACTS = ("none", "relu", "gelu", "silu", "swiglu")


# ---- dense projection ----
def _phi(z):
    """Standard normal distribution function."""
    return 0.5 * np.array([math.erfc(-v / math.sqrt(2.0)) for v in z.ravel()]).reshape(z.shape)


def _sigmoid(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def activation(z, act):
    if act == "relu":
        return np.where(z < 0, 0.0, z)
    if act == "gelu":
        return z * _phi(z)
    if act == "silu":
        return z * _sigmoid(z)
    if act == "swiglu":
        n = z.shape[1] // 2
        return z[:, :n] * _sigmoid(z[:, :n]) * z[:, n:]
    return z


def activation_backward(dy, z, act):
    """dL/dz from dL/d act(z)."""
    if act == "relu":
        return np.where(z > 0, dy, 0.0)  # a unit that is off passes nothing on, whatever dy holds
    if act == "gelu":
        return dy * (_phi(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi))
    if act == "silu":
        s = _sigmoid(z)
        return dy * (s + z * s * (1.0 - s))
    if act == "swiglu":
        n = z.shape[1] // 2
        g, u = z[:, :n], z[:, n:]
        s = _sigmoid(g)
        return np.concatenate([dy * u * (s + g * s * (1.0 - s)), dy * g * s], axis=1)
    return dy


def linear_forward(X, W, bias=None, residual=None, act="none"):
    """(out, z)."""
    z = X @ W.T
    if bias is not None:
        z = z + bias
    out = activation(z, act)
    return (out if residual is None else residual + out), z


def linear_backward(dY, X, W, z, act="none"):
    """(dX, dW, dbias, dz)."""
    dz = activation_backward(dY, z, act)
    return dz @ W, dz.T @ X, dz.sum(axis=0), dz


# ---- router losses ----
def _members(T, n_seq, seq_off, mask):
    """Per sequence, the token ids that count."""
    off = [0, T] if seq_off is None else [int(v) for v in seq_off]
    on = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    return [np.array([t for t in range(off[s], off[s + 1]) if on[t]], dtype=int) for s in range(n_seq)]


def _softmax(logits):
    """(p, lse) per row; a row of -infinity only has p = 0 and lse = -infinity."""
    with np.errstate(invalid="ignore", divide="ignore"):
        top = logits.max(axis=1, keepdims=True)
        top = np.where(np.isneginf(top), 0.0, top)
        ex = np.exp(logits - top)
        total = ex.sum(axis=1, keepdims=True)
        return np.where(total == 0, 0.0, ex / total), (top + np.log(total))[:, 0]


def router_losses(logits, topk_idx, n_seq=1, seq_off=None, mask=None):
    """dict(tokens, counts, prob, lse, loss): see the formulas in include/moe.h."""
    T, E = logits.shape
    K = topk_idx.shape[1]
    p, lse = _softmax(logits)
    rows = _members(T, n_seq, seq_off, mask)
    tokens = np.array([len(r) for r in rows])
    counts = np.zeros((n_seq, E), int)
    for s, r in enumerate(rows):
        for e in topk_idx[r].ravel():
            if 0 <= e < E:
                counts[s, e] += 1
    prob = np.stack([p[r].sum(axis=0) for r in rows])
    n = tokens.sum()
    loss = np.zeros(2)
    if n:
        loss[0] = sum(tokens[s] / n * E * np.sum(counts[s] / (K * tokens[s]) * prob[s] / tokens[s])
                      for s in range(n_seq) if tokens[s])
        loss[1] = sum(np.sum(np.where(np.isneginf(lse[r]), 0.0, lse[r]) ** 2) for r in rows) / n
    return dict(tokens=tokens, counts=counts, prob=prob, lse=lse, loss=loss)


def router_losses_backward(dloss, logits, K, counts, tokens, n_seq=1, seq_off=None, mask=None):
    """d(dloss . loss) / d logits with the counts held fixed."""
    T, E = logits.shape
    p, lse = _softmax(logits)
    n = int(tokens.sum())
    out = np.zeros_like(logits)
    for s, r in enumerate(_members(T, n_seq, seq_off, mask)):
        if not len(r):
            continue
        c = counts[s].astype(np.float64)
        l = np.where(np.isneginf(lse[r]), 0.0, lse[r])
        out[r] = p[r] * (dloss[0] * E / (K * tokens[s] * n) * (c - (p[r] @ c)[:, None]) + (dloss[1] * 2.0 / n * l)[:, None])
    return out


# ---- dropout ----
def philox4x32(counter, key, rounds=10):
    """Philox4x32 of Salmon et al. (SC 2011): four counter words (arrays of uint32) and two key words."""
    c = [np.asarray(v, np.uint64) for v in counter]
    k = [int(v) for v in key]
    low = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return [v.astype(np.uint32) for v in c]


def dropout_threshold(p):
    return int(math.floor(65536.0 * p + 0.5))


def dropout_keep(rows, cols, p, seed, offset):
    """[rows, cols] bool: the elements dropout keeps."""
    g = (cols + 7) // 8
    c0, c1 = np.meshgrid(np.arange(g, dtype=np.uint64), np.arange(rows, dtype=np.uint64))
    off = [np.full_like(c0, offset & 0xFFFFFFFF), np.full_like(c0, offset >> 32)]
    w = philox4x32([c0, c1] + off, (seed & 0xFFFFFFFF, seed >> 32))
    half = np.stack([x for v in w for x in (v & np.uint32(0xFFFF), v >> np.uint32(16))], axis=2)
    return half.reshape(rows, 8 * g)[:, :cols] >= dropout_threshold(p)


def dropout(x, p, seed, offset, residual=None):
    keep = dropout_keep(x.shape[0], x.shape[1], p, seed, offset)
    t = dropout_threshold(p)
    y = np.where(keep, x, 0.0) * (65536.0 / (65536 - t) if t < 65536 else 0.0)
    return y if residual is None else residual + y
