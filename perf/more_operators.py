"""More operators of the block around the MoE layer, as cases to be timed and compared.

Five passes, named by a case's "op":

* ``norm_fwd``   s = x + residual, y = layer norm (or RMS norm) of s, with the rows' statistics;
* ``norm_bwd``   gradients of it: dx (plus what reaches s directly), dweight, dbias;
* ``clip``       the global norm of many gradient tensors, and the tensors scaled down to a largest
                 norm (or the norm alone);
* ``linear_w4``  out = residual + act(X W^T + bias) with 4-bit weights and group scales;
* ``decode_w4``  the whole MoE layer for a few tokens with 4-bit expert weights.

4-bit weights: a row of K codes lies in K / 2 bytes, the even element in the low half.  "int4": value
(code - 8) s, one bf16 scale s per group of 32, 64 or 128 elements, scales [K / group, rows].  "fp4":
E2M1 values times 2^(e - 127), one byte e per 32 elements, bytes [ceil(K / 128), rows, 4].

``run`` computes a pass either in plain torch operations (``own`` false) or through the package's
entry points (``own`` true).  ``exact`` states the same operators in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoding token's norm with the residual stream (DeepSeek-V3-shaped layer): latency
        dict(name="norm_token_rms", op="norm_fwd", rows=1, cols=7168, dtype="bf16", wtype="bf16", kind="rms",
             residual=True, stats=False, bias=False, pad=0),
        # training forward in front of the Kimi-K2-shaped layer
        dict(name="norm_train", op="norm_fwd", rows=32768, cols=7168, dtype="bf16", wtype="f32", kind="layer",
             residual=True, stats=True, bias=True, pad=0),
        # its backward in front of the fine-grained layer, with the residual stream's gradient
        dict(name="norm_bwd_fine", op="norm_bwd", rows=32768, cols=1536, dtype="bf16", wtype="f32", kind="layer",
             dsum=True, bias=True, pad=0),
        # a small fp32 activation of odd width with a row stride
        dict(name="norm_bwd_odd_f32", op="norm_bwd", rows=999, cols=1003, dtype="f32", wtype="f32", kind="layer",
             dsum=False, bias=True, pad=5),
        # the tiny fp32 layer's gradients (router, gate, up, down, two norms' vectors): latency
        dict(name="clip_tiny", op="clip", sizes="layer", d=128, n=256, E=8, dtype="f32", max_norm=1.0, scale=True),
        # the fine-grained layer's gradients
        dict(name="clip_fine", op="clip", sizes="layer", d=1536, n=256, E=128, dtype="bf16", max_norm=1.0, scale=True),
        # many small tensors of odd sizes and both types (a model's biases and norm vectors)
        dict(name="clip_many", op="clip", sizes="many", count=600, most=20000, dtype="mixed", max_norm=1.0, scale=True),
        # one decoding token through the gate/up projection of a shared expert (DeepSeek-V3-shaped layer)
        dict(name="w4_token_swiglu", op="linear_w4", M=1, N=2048, K=7168, act="swiglu", format="fp4", group=32,
             bias=False, residual=False, pad=0),
        # a few decoding requests through a large down projection (Mixtral-shaped sizes), residual stream
        dict(name="w4_batch_residual", op="linear_w4", M=13, N=4096, K=14336, act="none", format="int4", group=128,
             bias=True, residual=True, pad=0),
        # a prompt of some hundred tokens through the shared expert's down projection, small groups
        dict(name="w4_prompt", op="linear_w4", M=777, N=7168, K=2048, act="none", format="int4", group=32,
             bias=False, residual=True, pad=8),
        # one token through the DeepSeek-V3-shaped layer
        dict(name="decode_w4_token", op="decode_w4", T=1, d=7168, n=2048, E=256, K=8, format="fp4", group=32),
        # a few requests through the fine-grained layer
        dict(name="decode_w4_fine", op="decode_w4", T=8, d=1536, n=256, E=128, K=8, format="int4", group=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "clip", "linear_w4", "linear_w4", "decode_w4"])
    if op.startswith("norm"):
        while True:
            c = dict(op=op, rows=_log(rng, 1, 32768), cols=rng.choice([_log(rng, 1, 16384), 64 * _log(rng, 1, 256)]),
                     dtype=rng.choice(["bf16", "bf16", "f32"]), wtype=rng.choice(["f32", "bf16"]),
                     kind=rng.choice(["layer", "rms"]), bias=rng.random() < 0.6, pad=rng.choice([0, 0, 3, 8]))
            if c["rows"] * c["cols"] <= 50e6:
                break
        if op == "norm_fwd":
            c.update(residual=rng.random() < 0.6, stats=rng.random() < 0.6)
        else:
            c.update(dsum=rng.random() < 0.6)
        return c
    if op == "clip":
        c = dict(op=op, sizes=rng.choice(["layer", "many"]), dtype=rng.choice(["bf16", "f32", "mixed"]),
                 max_norm=rng.choice([0.1, 1.0, 1e6]), scale=rng.random() < 0.7)
        if c["sizes"] == "many":
            c.update(count=_log(rng, 1, 700), most=_log(rng, 1, 60000))
        else:
            c.update(d=64 * _log(rng, 1, 32), n=64 * _log(rng, 1, 8), E=_log(rng, 1, 48))
        return c
    fmt = rng.choice(["int4", "int4", "fp4"])
    group = 32 if fmt == "fp4" else rng.choice([32, 64, 128])
    if op == "linear_w4":
        while True:
            c = dict(op=op, M=_log(rng, 1, 1024), N=max(8, _log(rng, 8, 16384) // 8 * 8),
                     K=max(group, _log(rng, group, 16384) // group * group), act=rng.choice(["none", "relu", "gelu", "silu", "swiglu"]),
                     format=fmt, group=group, bias=rng.random() < 0.5, residual=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 24]))
            if _rows_of_w(c) * c["K"] <= 6e7 and c["M"] * _rows_of_w(c) * c["K"] <= 1.1e10:
                return c
    while True:
        c = dict(op=op, T=_log(rng, 1, 64), d=128 * _log(rng, 1, 56), n=128 * _log(rng, 1, 32), E=rng.choice([4, 8, 60, 128]),
                 K=rng.choice([1, 2, 4, 8]), format=fmt, group=group)
        c["K"] = min(c["K"], c["E"])
        if c["T"] * c["K"] * c["n"] * c["d"] <= 1.0e8 and c["E"] * c["n"] * c["d"] <= 1e9:
            return c


def _rows_of_w(case):
    return case["N"] * (2 if case["act"] == "swiglu" else 1)


def _w4_bytes(rows, K, case):
    return rows * K // 2 + (rows * K // case["group"] * 2 if case["format"] == "int4" else rows * -(-K // 128) * 4)


def _gradient_sizes(case):
    """(elements, dtype) of every gradient tensor."""
    kinds = {"bf16": ["bf16"], "f32": ["f32"], "mixed": ["bf16", "f32", "f32"]}[case["dtype"]]
    if case["sizes"] == "layer":
        d, n, E = case["d"], case["n"], case["E"]
        shapes = [E * d, E * n * d, E * n * d, E * d * n]
        return [(s, kinds[i % len(kinds)]) for i, s in enumerate(shapes)] + [(d, "f32")] * 4  # two norms' vectors
    out, a = [], 12345
    for i in range(case["count"]):  # sizes spread over their logarithm, whatever the seed of the values
        a = (a * 1103515245 + 12345) % 2 ** 31
        out.append((max(1, int(round(case["most"] ** (a / 2.0 ** 31)))), kinds[i % len(kinds)]))
    return out


def work(case):
    op = case["op"]
    s = 2 if case.get("dtype") == "bf16" else 4
    if op.startswith("norm"):
        n, w = case["rows"] * case["cols"], case["cols"] * (2 if case["wtype"] == "bf16" else 4)
        stats = case["rows"] * (8 if case["kind"] == "layer" else 4)
        if op == "norm_fwd":
            return {"bytes": n * s * (4 if case["residual"] else 2) + w * (2 if case["bias"] else 1) + (stats if case["stats"] else 0),
                    "flops": 8 * n}
        return {"bytes": n * s * (4 if case["dsum"] else 3) + w + stats + 4 * case["cols"] * (2 if case["bias"] else 1), "flops": 14 * n}
    if op == "clip":
        n = sum(k * (2 if t == "bf16" else 4) for k, t in _gradient_sizes(case))
        return {"bytes": n * (2 if case["scale"] else 1) + 4, "flops": sum((3 if case["scale"] else 2) * k for k, _ in _gradient_sizes(case))}
    if op == "linear_w4":
        M, N, K, NW = case["M"], case["N"], case["K"], _rows_of_w(case)
        return {"bytes": _w4_bytes(NW, K, case) + 2 * M * K + 2 * M * N * (2 if case["residual"] else 1) + (4 * NW if case["bias"] else 0),
                "flops": 2 * M * NW * K}
    T, d, n, E, K = case["T"], case["d"], case["n"], case["E"], case["K"]
    hit = E * (1.0 - (1.0 - K / E) ** T)  # experts that some token picks, on average
    return {"bytes": int(hit * (2 * _w4_bytes(n, d, case) + _w4_bytes(d, n, case))) + 2 * E * d + 4 * T * d + 4 * T * E + 8 * T * K,
            "flops": 2 * T * E * d + 6 * T * K * n * d}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def _strided(rows, cols, pad, dtype, step=1):
    """An empty rows x cols tensor whose rows lie cols + pad (rounded up to a multiple of step) apart."""
    if not pad:
        return torch.empty(rows, cols, dtype=dtype, device="cuda")
    ld = (cols + pad + step - 1) // step * step
    return torch.empty(rows, ld, dtype=dtype, device="cuda")[:, :cols]


def _normal(g, rows, cols, std, dtype, pad=0, step=1):
    t = _strided(rows, cols, pad, dtype, step)
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda").mul_(std))
    return t


def _quantised(g, rows, K, case):
    """Codes and scales of normal weights of deviation 1 / sqrt(K), a few million at a time."""
    fmt, group = case["format"], case["group"]
    codes = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    if fmt == "int4":
        scales = torch.empty(K // group, rows, dtype=torch.bfloat16, device="cuda")
    else:
        scales = torch.full((-(-K // 128), rows, 4), 127, dtype=torch.uint8, device="cuda")
        borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 26) // K)
    for lo in range(0, rows, step):
        hi = min(rows, lo + step)
        w = torch.randn(hi - lo, K // group, group, generator=g, device="cuda").mul_(1.0 / math.sqrt(K))
        top = w.abs().amax(2, keepdim=True)
        if fmt == "int4":
            s = (top / 7.0).to(torch.bfloat16)
            scales[:, lo:hi] = s[:, :, 0].t()
            q = torch.round(w.div_(s.float().clamp(min=1e-30))).clamp_(-7, 7).add_(8).to(torch.uint8)
        else:
            e = torch.ceil(torch.log2((top / 6.0).clamp(min=2.0 ** -100)))
            groups = torch.nn.functional.pad((e[:, :, 0] + 127).to(torch.uint8), (0, 4 * scales.shape[0] - K // 32), value=127)
            scales[:, lo:hi] = groups.reshape(hi - lo, -1, 4).transpose(0, 1)
            w.div_(torch.exp2(e))
            q = torch.bucketize(w.abs(), borders).to(torch.uint8) + (w < 0).to(torch.uint8) * 8
        q = q.reshape(hi - lo, K // 2, 2)
        codes[lo:hi] = q[:, :, 0] | (q[:, :, 1] << 4)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op.startswith("norm"):
        R, C, pad = case["rows"], case["cols"], case["pad"]
        dt, f32 = DTYPES[case["dtype"]], torch.float32
        layer = case["kind"] == "layer"
        st["weight"] = torch.randn(C, generator=g, device="cuda").mul_(0.2).add_(1.0).to(DTYPES[case["wtype"]])
        st["bias"] = torch.randn(C, generator=g, device="cuda").mul_(0.1).to(DTYPES[case["wtype"]]) if case["bias"] else None
        if op == "norm_fwd":
            st["x"] = _normal(g, R, C, 1.0, dt, pad)
            st["residual"] = _normal(g, R, C, 3.0, dt, pad) if case["residual"] else None
            st["sum"] = _strided(R, C, pad, dt) if case["residual"] else None
            st["y"] = _strided(R, C, pad, dt)
            st["mean"] = torch.empty(R, device="cuda") if case["stats"] and layer else None
            st["rstd"] = torch.empty(R, device="cuda") if case["stats"] else None
        else:
            st["s"] = _normal(g, R, C, 3.0, dt, pad)
            st["dy"] = _normal(g, R, C, 1.0, dt, pad)
            st["dsum"] = _normal(g, R, C, 1.0, dt, pad) if case["dsum"] else None
            mean, rstd = _statistics(st["s"].double(), layer)  # what the forward left
            st["mean"], st["rstd"] = mean.to(f32) if layer else None, rstd.to(f32)
            st["dx"] = _strided(R, C, pad, dt)
            st["dweight"] = torch.empty(C, device="cuda")
            st["dbias"] = torch.empty(C, device="cuda") if case["bias"] else None
    elif op == "clip":
        st["grads"] = [torch.randn(k, generator=g, device="cuda").mul_(0.01).to(DTYPES[t]) for k, t in _gradient_sizes(case)]
        # the clipped gradients lie in one buffer per type, as buckets for a reduction or an optimizer do
        st["buckets"], st["clipped"] = _buckets(st["grads"], None) if case["scale"] else (None, None)
        st["norm"] = torch.empty(1, device="cuda")
    elif op == "linear_w4":
        M, N, K, NW, pad = case["M"], case["N"], case["K"], _rows_of_w(case), case["pad"]
        bf16 = torch.bfloat16
        st["X"] = _normal(g, M, K, 1.0, bf16, pad, 8)
        st["W"] = _quantised(g, NW, K, case)
        st["bias"] = torch.randn(NW, generator=g, device="cuda").mul_(0.5) if case["bias"] else None
        st["residual"] = _normal(g, M, N, 1.0, bf16, pad, 8) if case["residual"] else None
        st["out"] = _strided(M, N, pad, bf16, 8)
    else:
        T, d, n, E, K = case["T"], case["d"], case["n"], case["E"], case["K"]
        st["X"] = _normal(g, T, d, 1.0, torch.bfloat16)
        st["W_r"] = _normal(g, E, d, 0.02, torch.bfloat16)
        st["bias"] = torch.randn(E, generator=g, device="cuda")
        st["gate"], st["up"], st["down"] = _quantised(g, E * n, d, case), _quantised(g, E * n, d, case), _quantised(g, E * d, n, case)
        st["logits"] = torch.empty(T, E, device="cuda")
        st["topk_idx"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
        st["topk_w"] = torch.empty(T, K, device="cuda")
        st["out"] = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    if own:
        st["handle"] = _handle(st)
    return st


def _buckets(tensors, dtype):
    """A zeroed buffer for all tensors of a type (kept as dtype where given), and the tensors' places in
    it, each on a 16-byte border."""
    flat, views = {}, []
    for name, t in DTYPES.items():
        n = sum(-(-g.numel() // 8) * 8 for g in tensors if g.dtype == t)
        if n:
            flat[name] = torch.zeros(n, dtype=dtype or t, device="cuda")
    used = dict.fromkeys(flat, 0)
    for g in tensors:
        name = "bf16" if g.dtype == torch.bfloat16 else "f32"
        views.append(flat[name][used[name]:used[name] + g.numel()])
        used[name] += -(-g.numel() // 8) * 8
    return flat, views


def _statistics(s, layer):
    mean = s.mean(1) if layer else torch.zeros_like(s[:, 0])
    return mean, 1.0 / torch.sqrt((s - mean[:, None]).square().mean(1) + 1e-5)


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------
def run(state):
    return _own(state) if own else _plain(state)


def _act(z, act, N):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "swiglu":
        return z[:, :N] / (1.0 + torch.exp(-z[:, :N])) * z[:, N:]
    return z


def _values(codes, scales, case):
    """The weights [..., rows, K] in 32 bits of codes [..., rows, K / 2] and scales [groups, ..., rows(, 4)]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    if case["format"] == "int4":
        s = scales.float().movedim(0, -1).repeat_interleave(case["group"], -1)
        return (c.float() - 8.0) * s
    table = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")
    s = torch.exp2(scales.float() - 127.0).movedim(0, -2).flatten(-2)
    return table[c.int()] * s[..., : c.shape[-1] // 32].repeat_interleave(32, -1)


def _of_experts(w, rows, experts, case):
    """The weights of the experts that the (token, choice) pairs picked, [pairs, rows, K]."""
    codes, scales = w
    picked = codes.reshape(-1, rows, codes.shape[1])[experts]
    by_expert = scales.reshape((scales.shape[0], -1, rows) + tuple(scales.shape[2:]))
    return _values(picked, by_expert[:, experts], case)


def _norm_plain(st):
    c = st["case"]
    dt, layer = DTYPES[c["dtype"]], c["kind"] == "layer"
    w = st["weight"].float()
    if c["op"] == "norm_fwd":
        r = {}
        s = st["x"].float()
        if st["residual"] is not None:
            r["sum"] = (s + st["residual"].float()).to(dt)
            s = r["sum"].float()
        mean, rstd = _statistics(s, layer)
        y = (s - mean[:, None]) * rstd[:, None] * w
        r["y"] = (y + st["bias"].float() if st["bias"] is not None else y).to(dt)
        if c["stats"]:
            r["rstd"] = rstd
            if layer:
                r["mean"] = mean
        return r
    s, dy = st["s"].float(), st["dy"].float()
    xh = (s - st["mean"][:, None] if layer else s) * st["rstd"][:, None]
    gw = dy * w
    d = gw - xh * (gw * xh).mean(1, keepdim=True)
    if layer:
        d = d - gw.mean(1, keepdim=True)
    d = d * st["rstd"][:, None]
    if st["dsum"] is not None:
        d = d + st["dsum"].float()
    r = {"dx": d.to(dt), "dweight": (dy * xh).sum(0)}
    if st["dbias"] is not None:
        r["dbias"] = dy.sum(0)
    return r


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op.startswith("norm"):
        return _norm_plain(st)
    if op == "clip":
        norm = torch.sqrt(sum(t.double().square().sum() for t in st["grads"]))  # long sums: 64 bits
        r = {"norm": norm.float().reshape(1)}
        if c["scale"]:
            f = torch.where(norm > c["max_norm"], c["max_norm"] / norm, torch.ones_like(norm)).float()
            for out, t in zip(st["clipped"], st["grads"]):
                out.copy_(t.float() * f)
            r.update(st["buckets"])
        return r
    if op == "linear_w4":
        z = st["X"].float() @ _values(*st["W"], c).t()
        if st["bias"] is not None:
            z = z + st["bias"]
        y = _act(z, c["act"], c["N"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return {"out": y.to(torch.bfloat16)}
    T, d, n, K = c["T"], c["d"], c["n"], c["K"]
    # (64 bits: scores next to one another decide the choice)
    logits = (st["X"].double() @ st["W_r"].double().t() + st["bias"]).float()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    idx, top = order.indices[:, :K], order.values[:, :K]
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    pair = idx.reshape(-1)
    x = st["X"].float().repeat_interleave(K, 0)[:, :, None].contiguous()
    zg = torch.bmm(_of_experts(st["gate"], n, pair, c), x)
    zu = torch.bmm(_of_experts(st["up"], n, pair, c), x)
    h = zg / (1.0 + torch.exp(-zg)) * zu
    y = torch.bmm(_of_experts(st["down"], d, pair, c), h).reshape(T, K, d)
    return {"logits": logits, "topk_idx": idx.to(torch.int32), "topk_w": w, "out": (y * w[:, :, None]).sum(1).to(torch.bfloat16)}


def _handle(st):
    """What a program keeps between calls: shape structs, tensor lists, weight descriptors, workspaces."""
    from mixture_experts_layer_lds_amd import binding as B
    c = st["case"]
    op = c["op"]
    ld = lambda k: st[k].stride(0) if st.get(k) is not None and st[k].shape[0] > 1 else 0  # noqa: E731
    if op == "norm_fwd":
        return B.make_norm_dims(c["rows"], c["cols"], c["dtype"], c["kind"], 1e-5, c["wtype"], ldx=ld("x"), ldr=ld("residual"),
                                lds=ld("sum"), ldy=ld("y"))
    if op == "norm_bwd":
        dims = B.make_norm_dims(c["rows"], c["cols"], c["dtype"], c["kind"], 1e-5, c["wtype"], ldx=ld("dx"), ldr=ld("dsum"),
                                lds=ld("s"), ldy=ld("dy"))
        return (dims,) + B.norm_workspace(dims)
    if op == "clip":
        grads = B.Gradients(st["grads"], st["clipped"])
        return (grads,) + B.grad_workspace(grads)
    w4 = lambda k: B.W4(st[k][0], st[k][1], c["format"], c["group"])  # noqa: E731
    if op == "linear_w4":
        dims = B.make_linear_dims(c["M"], c["N"], c["K"], "bf16", c["act"], ldx=ld("X"), ldr=ld("residual"), ldy=ld("out"))
        return (dims, w4("W")) + B.linear_w4_workspace(dims)
    dims = B.make_dims(c["T"], c["d"], c["n"], c["E"], c["K"], "bf16")
    return (dims, w4("gate"), w4("up"), w4("down")) + B.workspace(dims, B.OP_DECODE)


def _own(st):
    from mixture_experts_layer_lds_amd import binding as B
    c = st["case"]
    op = c["op"]
    if op == "norm_fwd":
        B.moe_norm(st["handle"], st["x"], st["residual"], st["weight"], st["bias"], st["sum"], st["y"], st["mean"], st["rstd"])
        return {k: st[k] for k in ("sum", "y", "rstd", "mean") if st[k] is not None}
    if op == "norm_bwd":
        dims, ws, nb = st["handle"]
        B.moe_norm_backward(dims, st["dy"], st["s"], st["weight"], st["mean"], st["rstd"], st["dsum"], st["dx"], st["dweight"],
                            st["dbias"], ws, nb)
        return {k: st[k] for k in ("dx", "dweight", "dbias") if st[k] is not None}
    if op == "clip":
        grads, ws, nb = st["handle"]
        if not c["scale"]:
            B.moe_grad_norm(grads, st["norm"], ws, nb)
            return {"norm": st["norm"]}
        B.moe_grad_clip(grads, c["max_norm"], None, st["norm"], ws, nb)
        return dict({"norm": st["norm"]}, **st["buckets"])
    if op == "linear_w4":
        dims, W, ws, nb = st["handle"]
        B.moe_linear_w4(dims, st["X"], W, st["bias"], st["residual"], st["out"], ws, nb)
        return {"out": st["out"]}
    dims, gate, up, down, ws, nb = st["handle"]
    B.moe_decode_w4(dims, st["X"], st["W_r"], st["bias"], gate, up, down, st["logits"], st["topk_idx"], st["topk_w"], st["out"], ws, nb)
    return {"logits": st["logits"], "topk_idx": st["topk_idx"], "topk_w": st["topk_w"], "out": st["out"]}


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _weights64(codes, scales, case):
    """Weights [rows, K] in 64 bits, group by group."""
    rows, K, G = codes.shape[0], codes.shape[1] * 2, case["group"]
    out = torch.empty(rows, K, dtype=torch.float64, device="cuda")
    levels = [q - 8.0 for q in range(16)] if case["format"] == "int4" else E2M1 + [-v for v in E2M1]
    table = torch.tensor(levels, dtype=torch.float64, device="cuda")
    for g in range(K // G):
        part = codes[:, g * G // 2:(g + 1) * G // 2].long()
        s = scales[g].double() if case["format"] == "int4" else torch.pow(2.0, scales[g // 4, :, g % 4].double() - 127.0)
        out[:, g * G:(g + 1) * G:2] = table[part % 16] * s[:, None]
        out[:, g * G + 1:(g + 1) * G:2] = table[torch.div(part, 16, rounding_mode="floor")] * s[:, None]
    return out


def exact(case, seed):
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    d64 = lambda t: t.to(torch.float64)  # noqa: E731
    op = case["op"]
    if op.startswith("norm"):
        dt, C, layer = DTYPES[case["dtype"]], case["cols"], case["kind"] == "layer"
        w = d64(st["weight"])
        one = torch.ones(C, 1, dtype=torch.float64, device="cuda")
        if op == "norm_fwd":
            r = {}
            s = d64(st["x"])
            if st["residual"] is not None:
                r["sum"] = s + d64(st["residual"])
                s = d64(r["sum"].to(dt))  # what is normalised is the stored sum
            mu = torch.mm(s, one) / C if layer else torch.zeros(case["rows"], 1, dtype=torch.float64, device="cuda")
            centred = s - mu
            inv = torch.rsqrt(torch.mm(centred * centred, one) / C + 1e-5)
            r["y"] = centred * inv * w + (d64(st["bias"]) if st["bias"] is not None else 0.0)
            if case["stats"]:
                r["rstd"] = inv[:, 0]
                if layer:
                    r["mean"] = mu[:, 0]
            return r
        inv, dy = d64(st["rstd"])[:, None], d64(st["dy"])
        xh = (d64(st["s"]) - (d64(st["mean"])[:, None] if layer else 0.0)) * inv
        gw = dy * w
        dx = inv * (gw - xh * (torch.mm(gw * xh, one) / C) - (torch.mm(gw, one) / C if layer else 0.0))
        rows = torch.ones(1, case["rows"], dtype=torch.float64, device="cuda")
        r = {"dx": dx if st["dsum"] is None else dx + d64(st["dsum"]), "dweight": torch.mm(rows, dy * xh)[0]}
        if st["dbias"] is not None:
            r["dbias"] = torch.mm(rows, dy)[0]
        return r
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for t in st["grads"]:
            total += torch.dot(d64(t), d64(t))
        norm = math.sqrt(float(total))
        r = {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda")}
        if case["scale"]:
            flat, views = _buckets(st["grads"], torch.float64)
            for v, t in zip(views, st["grads"]):
                v.copy_(d64(t) * min(1.0, case["max_norm"] / max(norm, 1e-300)))
            r.update(flat)
        return r

    def activated(z, act, N):
        if act == "relu":
            return torch.where(z > 0, z, 0.0)
        if act == "gelu":
            return z * torch.special.ndtr(z)
        if act in ("silu", "swiglu"):
            return z[:, :N] * torch.sigmoid(z[:, :N]) * (z[:, N:] if act == "swiglu" else 1.0)
        return z

    if op == "linear_w4":
        z = torch.mm(d64(st["X"]), _weights64(*st["W"], case).t())
        z = z + d64(st["bias"]) if st["bias"] is not None else z
        y = activated(z, case["act"], case["N"])
        return {"out": y if st["residual"] is None else d64(st["residual"]) + y}
    T, d, n, K = case["T"], case["d"], case["n"], case["K"]
    x = d64(st["X"])
    logits = torch.mm(x, d64(st["W_r"]).t()) + d64(st["bias"])
    idx = torch.argsort(-logits, dim=1, stable=True)[:, :K]
    w = torch.softmax(torch.gather(logits, 1, idx), 1)
    out = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for e in sorted(set(idx.flatten().tolist())):
        part = lambda k, rows: _weights64(st[k][0][e * rows:(e + 1) * rows], st[k][1][:, e * rows:(e + 1) * rows], case)  # noqa: E731
        hit = idx == e
        t = hit.any(1).nonzero()[:, 0]
        both = torch.cat([part("gate", n), part("up", n)])
        h = activated(torch.mm(x[t], both.t()), "swiglu", n)
        out[t] += torch.mm(h, part("down", d).t()) * (w * hit).sum(1)[t][:, None]
    return {"logits": logits, "topk_idx": idx.to(torch.int32), "topk_w": w, "out": out}
