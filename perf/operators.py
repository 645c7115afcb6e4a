"""The training-block operators beside the MoE layer, as cases to be timed and compared.

Six passes, named by a case's "op":

* ``linear_fwd``   out = residual + act(X W^T + bias), optionally with the pre-activation saved;
* ``linear_bwd``   dX, dW and dbias of it from dY and the saved pre-activation;
* ``loss_fwd``     router balance loss and z-loss of one batch of logits: per-sequence expert
                   counts, probability sums, log-sum-exps and the two losses;
* ``loss_bwd``     their gradient with respect to the logits;
* ``dropout``      out = residual + dropout(x) with a counter-based mask that is never stored
                   (without a residual: also the gradient of dropout);
* ``combine_dropout``  the MoE layer's combine with dropout and the residual sum in its epilogue.

``run`` computes a pass either in plain torch operations (``own`` false) or through the package's
entry points (``own`` true).  ``exact`` states the same operators in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoding token through the gate/up projection of a shared expert (DeepSeek-V3-shaped
        # layer: d = 7168, n = 2048): latency, bound by reading the weights
        dict(name="linear_token_swiglu", op="linear_fwd", M=1, N=2048, K=7168, dtype="bf16", act="swiglu",
             bias=False, residual=False, save=False, pad=0),
        # a few decoding requests through its down projection, added to the routed experts' output
        dict(name="linear_decode_residual", op="linear_fwd", M=13, N=7168, K=2048, dtype="bf16", act="none",
             bias=False, residual=True, save=False, pad=0),
        # training forward of a dense FFN's first projection at the Mixtral-shaped sizes
        dict(name="linear_train_gelu", op="linear_fwd", M=8192, N=14336, K=4096, dtype="bf16", act="gelu",
             bias=True, residual=False, save=True, pad=0),
        # a small fp32 layer: odd row count, ragged widths, rows with a stride
        dict(name="linear_ragged_f32", op="linear_fwd", M=1237, N=904, K=1544, dtype="f32", act="silu",
             bias=True, residual=True, save=True, pad=8),
        # training backward of the shared expert's gate/up projection (DeepSeek-V3-shaped layer)
        dict(name="linear_bwd_train_swiglu", op="linear_bwd", M=16384, N=2048, K=7168, dtype="bf16", act="swiglu",
             bias=False, pad=0),
        # backward of a small ragged projection with a bias
        dict(name="linear_bwd_ragged_relu", op="linear_bwd", M=999, N=1000, K=264, dtype="bf16", act="relu",
             bias=True, pad=8),
        # router losses of the tiny fp32 layer (a unit test's or a debugging run's batch): latency
        dict(name="loss_tiny", op="loss_fwd", T=256, E=8, K=2, n_seq=1, masked=0.0),
        # router losses per sequence of the DeepSeek-V3-shaped layer, ragged sequences with padding
        dict(name="loss_sequences", op="loss_fwd", T=16384, E=256, K=8, n_seq=7, masked=0.05),
        # gradient of the batch-wide losses on the Kimi-K2-shaped layer
        dict(name="loss_bwd_batch", op="loss_bwd", T=32768, E=384, K=8, n_seq=1, masked=0.0),
        # the fine-grained layer's combine with residual dropout in its epilogue
        dict(name="combine_dropout_fine", op="combine_dropout", T=32768, d=1536, E=128, K=8, dtype="bf16", p=0.1,
             residual=True),
        # gradient of residual dropout at the Kimi-K2-shaped layer's output size
        dict(name="dropout_bwd_large", op="dropout", rows=32768, cols=7168, dtype="bf16", p=0.1, residual=False, pad=0),
        # a small fp32 activation of odd width with a row stride
        dict(name="dropout_add_odd_f32", op="dropout", rows=257, cols=1003, dtype="f32", p=0.25, residual=True, pad=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult8(rng, lo, hi):
    return max(8, _log(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["linear_fwd", "linear_fwd", "linear_bwd", "loss_fwd", "loss_bwd", "dropout", "combine_dropout"])
    if op.startswith("linear"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        most = 4.0e11 if dtype == "bf16" else 4.0e10  # M N' K of one product
        while True:
            c = dict(op=op, M=_log(rng, 1, 16384), N=_mult8(rng, 8, 8192), K=_mult8(rng, 8, 8192), dtype=dtype,
                     act=rng.choice(["none", "relu", "gelu", "silu", "swiglu"]), bias=rng.random() < 0.6,
                     pad=rng.choice([0, 0, 8, 24]))
            if c["M"] * _rows_of_w(c) * c["K"] <= most / (2 if op == "linear_bwd" else 1):
                break
        if op == "linear_fwd":
            c["residual"] = rng.random() < 0.5
            c["save"] = rng.random() < 0.5
        return c
    if op.startswith("loss"):
        E = rng.choice([_log(rng, 2, 512), rng.choice([8, 64, 128, 256, 384])])
        T = _log(rng, 1, 32768)
        return dict(op=op, T=T, E=E, K=min(E, rng.choice([1, 2, 6, 8])), n_seq=_log(rng, 1, 64), masked=rng.choice([0.0, 0.0, 0.2]))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    p = rng.choice([0.0, 0.05, 0.1, 0.5, round(rng.uniform(0.01, 0.9), 4)])
    if op == "dropout":
        return dict(op=op, rows=_log(rng, 1, 16384), cols=_log(rng, 1, 8192), dtype=dtype, p=p,
                    residual=rng.random() < 0.5, pad=rng.choice([0, 0, 3, 8]))
    return dict(op=op, T=_log(rng, 1, 16384), d=64 * _log(rng, 1, 64), E=rng.choice([8, 64, 128]), K=rng.choice([1, 2, 6, 8]),
                dtype=dtype, p=p, residual=rng.random() < 0.7)


def _rows_of_w(case):
    return case["N"] * (2 if case["act"] == "swiglu" else 1)


def work(case):
    op = case["op"]
    s = 2 if case.get("dtype") == "bf16" else 4
    if op.startswith("linear"):
        M, N, K, NW = case["M"], case["N"], case["K"], _rows_of_w(case)
        if op == "linear_fwd":
            n = M * K + NW * K + M * N + (M * N if case["residual"] else 0) + (M * NW if case["save"] else 0)
            return {"bytes": n * s + (4 * NW if case["bias"] else 0), "flops": 2 * M * NW * K}
        n = M * N + 2 * M * K + 2 * NW * K + (M * NW if case["act"] != "none" else 0)
        return {"bytes": n * s + (4 * NW if case["bias"] else 0), "flops": 4 * M * NW * K}
    if op.startswith("loss"):
        T, E, S = case["T"], case["E"], case["n_seq"]
        if op == "loss_fwd":
            return {"bytes": 4 * T * E + 4 * T * case["K"] + T + 4 * T + 8 * S * E + 8 * S + 8, "flops": 6 * T * E}
        return {"bytes": 8 * T * E + T + 4 * T + 4 * S * E + 8 * S + 8, "flops": 6 * T * E}
    if op == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": n * s * (3 if case["residual"] else 2) + 16, "flops": 2 * n}
    T, d, K = case["T"], case["d"], case["K"]
    return {"bytes": (T * K + T * (2 if case["residual"] else 1)) * d * s + 8 * T * K + 4 * (T + 1) + 16, "flops": 2 * T * K * d}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------
def _strided(rows, cols, pad, dtype):
    """An empty rows x cols tensor whose rows lie cols + pad (rounded up to 16 bytes) apart where pad > 0."""
    if not pad:
        return torch.empty(rows, cols, dtype=dtype, device="cuda")
    step = 8
    ld = (cols + pad + step - 1) // step * step
    return torch.empty(rows, ld, dtype=dtype, device="cuda")[:, :cols]


def _normal(g, rows, cols, std, dtype, pad=0):
    t = _strided(rows, cols, pad, dtype)
    t.copy_(torch.randn(rows, cols, generator=g, device="cuda").mul_(std))
    return t


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op.startswith("linear"):
        M, N, K, NW, pad = case["M"], case["N"], case["K"], _rows_of_w(case), case["pad"]
        dt = DTYPES[case["dtype"]]
        st["X"] = _normal(g, M, K, 1.0, dt, pad)
        st["W"] = _normal(g, NW, K, 1.0 / math.sqrt(K), dt)
        st["bias"] = torch.randn(NW, generator=g, device="cuda").mul_(0.5) if case["bias"] else None
        if op == "linear_fwd":
            st["residual"] = _normal(g, M, N, 1.0, dt, pad) if case["residual"] else None
            st["out"] = _strided(M, N, pad, dt)
            st["Z"] = torch.empty(M, NW, dtype=dt, device="cuda") if case["save"] else None
        else:
            st["dY"] = _normal(g, M, N, 1.0, dt, pad)
            # the pre-activation that the forward saved
            st["Z"] = _pre_activation(st["X"], st["W"], st["bias"]).to(dt) if case["act"] != "none" else None
            st["dX"] = _strided(M, K, pad, dt)
            st["dW"] = torch.empty(NW, K, dtype=dt, device="cuda")
            st["dbias"] = torch.empty(NW, device="cuda") if case["bias"] else None
    elif op.startswith("loss"):
        T, E, K, S = case["T"], case["E"], case["K"], case["n_seq"]
        st["logits"] = torch.randn(T, E, generator=g, device="cuda") * 1.2 + torch.randn(E, generator=g, device="cuda") * 0.5
        st["topk_idx"] = torch.topk(st["logits"], K, dim=1).indices.to(torch.int32).contiguous()
        # sequences of random lengths (some may be empty); the last one may end before the last token
        cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda")).values if S > 1 else None
        zero, end = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.full((1,), T - (T // 50 if S > 1 else 0), dtype=torch.int64, device="cuda")
        st["seq_off"] = torch.minimum(torch.cat([zero, cuts, end]) if S > 1 else torch.cat([zero, end]), end).to(torch.int32)
        st["mask"] = (torch.rand(T, generator=g, device="cuda") >= case["masked"]).to(torch.uint8) if case["masked"] else None
        st["tokens"] = torch.empty(S, dtype=torch.int32, device="cuda")
        st["counts"] = torch.empty(S, E, dtype=torch.int32, device="cuda")
        st["lse"] = torch.empty(T, device="cuda")
        if op == "loss_fwd":
            st["prob"] = torch.empty(S, E, device="cuda")
            st["loss"] = torch.empty(2, device="cuda")
        else:
            # what the forward left, and the weights of the two losses times the loss scale
            tokens, counts = _token_counts(st)
            st["tokens"].copy_(tokens)
            st["counts"].copy_(counts)
            st["lse"].copy_(torch.logsumexp(st["logits"].double(), 1))
            st["dloss"] = torch.tensor([0.01 * 1024, 0.001 * 1024], device="cuda")
            st["dlogits"] = torch.empty(T, E, device="cuda")
    else:
        dt = DTYPES[case["dtype"]]
        st["rng"] = torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")  # seed, offset
        if op == "dropout":
            R, C = case["rows"], case["cols"]
            st["x"] = _normal(g, R, C, 1.0, dt, case["pad"])
            st["residual"] = _normal(g, R, C, 1.0, dt, case["pad"]) if case["residual"] else None
            st["out"] = _strided(R, C, case["pad"], dt)
        else:
            T, d, E, K = case["T"], case["d"], case["E"], case["K"]
            scores = torch.randn(T, E, generator=g, device="cuda")
            top = torch.topk(scores, K, dim=1)
            st["plan"] = _plan(top.indices, torch.softmax(top.values, 1), T, E, K)
            st["Y"] = _normal(g, T * K, d, 1.0, dt)
            st["residual"] = _normal(g, T, d, 1.0, dt) if case["residual"] else None
            st["out"] = torch.empty(T, d, dtype=dt, device="cuda")
    if own:
        st["handle"] = _handle(st)
    return st


def _plan(idx, w, T, E, K):
    """The routing plan's arrays (see include/moe.h) of a plain top-K choice."""
    order = torch.sort(idx, dim=1)
    idx, w = order.values, torch.gather(w, 1, order.indices)
    pair = torch.sort(idx.reshape(-1) * T + torch.arange(T, device="cuda").repeat_interleave(K)).indices  # rows: by expert, then token
    row_of_pair = torch.empty_like(pair)
    row_of_pair[pair] = torch.arange(T * K, device="cuda")
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    i32 = torch.int32
    return dict(topk_idx=idx.reshape(-1).to(i32), topk_w=w.reshape(-1).contiguous(), counts=counts.to(i32),
                expert_off=torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(i32),
                row_token=torch.div(pair, K, rounding_mode="floor").to(i32), row_w=w.reshape(-1)[pair].contiguous(),
                tok_off=(torch.arange(T + 1, device="cuda") * K).to(i32), tok_row=row_of_pair.to(i32),
                meta=torch.full((16,), T * K, dtype=i32, device="cuda"))


def _pre_activation(X, W, bias):
    z = X.float() @ W.float().t()
    return z + bias if bias is not None else z


def _sequence_of(st):
    """Each token's sequence, and whether it counts (inside a sequence and not masked)."""
    T, S = st["case"]["T"], st["case"]["n_seq"]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(st["seq_off"][1:].contiguous(), t, right=True)
    live = (t >= st["seq_off"][0]) & (seq < S)
    if st["mask"] is not None:
        live = live & (st["mask"] != 0)
    return seq.clamp(max=S - 1), live


def _per_sequence(st, values):
    """Sums of the rows of values over each sequence's counting tokens (whole numbers stay exact)."""
    seq, live = _sequence_of(st)
    member = (seq[None, :] == torch.arange(st["case"]["n_seq"], device="cuda")[:, None]) & live[None, :]
    return member.float() @ values


def _token_counts(st):
    T, E = st["case"]["T"], st["case"]["E"]
    picks = torch.zeros(T, E + 1, device="cuda").scatter_(1, st["topk_idx"].long(), 1.0)
    picks[:, E] = 1.0  # a last column that counts the tokens
    sums = _per_sequence(st, picks).to(torch.int32)
    return sums[:, E].contiguous(), sums[:, :E].contiguous()


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
        g = z[:, :N]
        return g / (1.0 + torch.exp(-g)) * z[:, N:]
    return z


def _act_grad(dy, z, act, N):
    if act == "relu":
        return dy * (z > 0)
    if act == "gelu":
        return dy * (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi)))
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return dy * s * (1.0 + z * (1.0 - s))
    if act == "swiglu":
        g, u = z[:, :N], z[:, N:]
        s = 1.0 / (1.0 + torch.exp(-g))
        return torch.cat([dy * u * s * (1.0 + g * (1.0 - s)), dy * g * s], 1)
    return dy


def _keep(rng, rows, cols, p):
    """Which elements dropout keeps.  Philox4x32-10 (Salmon et al., SC'11): key = seed, counter =
    (column / 8, row, offset); element i of a group of eight takes 16 bits of word i / 2, the low
    half first, and is kept where they are at least round(p 65536)."""
    low = 0xFFFFFFFF
    n8 = (cols + 7) // 8
    seed, offset = rng[0], rng[1]
    c0 = torch.arange(n8, device="cuda").expand(rows, n8)
    c1 = torch.arange(rows, device="cuda")[:, None].expand(rows, n8)
    c2, c3 = (offset & low).expand(rows, n8), ((offset >> 32) & low).expand(rows, n8)
    k0, k1 = seed & low, (seed >> 32) & low

    def halves(a, m):  # high and low 32 bits of a * m
        lo = (a & 0xFFFF) * m
        mid = (lo >> 16) + (a >> 16) * m
        return mid >> 16, ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)

    for _ in range(10):
        h0, l0 = halves(c0, 0xD2511F53)
        h1, l1 = halves(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0 & 0xFFFF, c0 >> 16, c1 & 0xFFFF, c1 >> 16, c2 & 0xFFFF, c2 >> 16, c3 & 0xFFFF, c3 >> 16], 2)
    return words.reshape(rows, n8 * 8)[:, :cols] >= _threshold(p)


def _threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def _scale(p):
    t = _threshold(p)
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "linear_fwd":
        z = _pre_activation(st["X"], st["W"], st["bias"])
        y = _act(z, c["act"], c["N"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        out = y.to(st["X"].dtype)
        return {"out": out, "Z": z.to(st["X"].dtype)} if c["save"] else {"out": out}
    if op == "linear_bwd":
        dt = st["X"].dtype
        dy = st["dY"].float()
        dz = _act_grad(dy, st["Z"].float(), c["act"], c["N"]) if st["Z"] is not None else dy
        r = {"dX": (dz @ st["W"].float()).to(dt), "dW": (dz.t() @ st["X"].float()).to(dt)}
        if st["dbias"] is not None:
            r["dbias"] = dz.sum(0)
        return r
    if op.startswith("loss"):
        T, E, K, S = c["T"], c["E"], c["K"], c["n_seq"]
        seq, live = _sequence_of(st)
        x = st["logits"]
        if op == "loss_fwd":
            top = x.max(1, keepdim=True).values
            ex = torch.exp(x - top)
            total = ex.sum(1, keepdim=True)
            prob = ex / total
            lse = (top + torch.log(total))[:, 0]
            tokens, counts = _token_counts(st)
            psum = _per_sequence(st, prob)
            n = live.sum().clamp(min=1).double()
            ts = tokens.clamp(min=1).double()
            balance = ((counts.double() * psum).sum(1) / ts).sum() * E / (K * n)
            z = (lse.double().square() * live).sum() / n
            return {"tokens": tokens, "counts": counts, "prob": psum.float(), "lse": lse,
                    "loss": torch.stack([balance, z]).float()}
        n = st["tokens"].sum().clamp(min=1).float()
        ts = st["tokens"].clamp(min=1).float()
        # counts less their mean: the probabilities sum to 1, so the mean drops out of the difference
        excess = (st["counts"] - st["tokens"][:, None].float() * K / E)[seq]
        p = torch.exp(x - st["lse"][:, None])
        a = (st["dloss"][0] * E / (K * n)) / ts
        b = st["dloss"][1] * 2.0 / n
        d = p * (a[seq][:, None] * (excess - (excess * p).sum(1, keepdim=True)) + (b * st["lse"])[:, None])
        return {"dlogits": torch.where(live[:, None], d, torch.zeros_like(d))}
    if op == "dropout":
        x = st["x"].float()
        keep = _keep(st["rng"], c["rows"], c["cols"], c["p"])
        y = torch.where(keep, x * _scale(c["p"]), torch.zeros_like(x))
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return {"out": y.to(st["x"].dtype)}
    T, d, K = c["T"], c["d"], c["K"]
    rows = st["plan"]["tok_row"].long()
    y = (st["Y"][rows].float() * st["plan"]["row_w"][rows][:, None]).reshape(T, K, d).sum(1)
    keep = _keep(st["rng"], T, d, c["p"])
    y = torch.where(keep, y * _scale(c["p"]), torch.zeros_like(y))
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return {"out": y.to(st["Y"].dtype)}


def _handle(st):
    """What a program keeps between calls: shape structs, the routing plan and workspaces."""
    from mixture_experts_layer_lds_amd import binding as B
    c = st["case"]
    op = c["op"]
    if op.startswith("linear"):
        dims = B.make_linear_dims(c["M"], c["N"], c["K"], c["dtype"], c["act"], ldx=st["X"].stride(0),
                                  ldr=st["residual"].stride(0) if st.get("residual") is not None else 0,
                                  ldy=st["out" if op == "linear_fwd" else "dY"].stride(0))
        return (dims,) + B.linear_workspace(dims, B.LINEAR_FORWARD if op == "linear_fwd" else B.LINEAR_BACKWARD)
    if op.startswith("loss"):
        dims = B.make_dims(c["T"], 64, 64, c["E"], c["K"], "f32")
        return (dims,) + (B.router_loss_workspace(dims, c["n_seq"]) if op == "loss_fwd" else ())
    if op == "dropout":
        return ()
    dims = B.make_dims(c["T"], c["d"], 64, c["E"], c["K"], c["dtype"])
    plan = B.Plan(dims)
    for k, v in st["plan"].items():
        getattr(plan, k).copy_(v)
    return (dims, plan)


def _own(st):
    from mixture_experts_layer_lds_amd import binding as B
    c = st["case"]
    op = c["op"]
    if op == "linear_fwd":
        dims, ws, nb = st["handle"]
        B.moe_linear(dims, st["X"], st["W"], st["bias"], st["residual"], st["Z"], st["out"], ws, nb)
        return {"out": st["out"], "Z": st["Z"]} if c["save"] else {"out": st["out"]}
    if op == "linear_bwd":
        dims, ws, nb = st["handle"]
        B.moe_linear_backward(dims, st["dY"], st["X"], st["W"], st["Z"], st["dX"], st["dW"], st["dbias"], ws, nb)
        r = {"dX": st["dX"], "dW": st["dW"]}
        if st["dbias"] is not None:
            r["dbias"] = st["dbias"]
        return r
    if op == "loss_fwd":
        dims, ws, nb = st["handle"]
        B.moe_router_loss(dims, st["logits"], st["topk_idx"], c["n_seq"], st["seq_off"], st["mask"], st["tokens"],
                          st["counts"], st["prob"], st["lse"], st["loss"], ws, nb)
        return {"tokens": st["tokens"], "counts": st["counts"], "prob": st["prob"], "lse": st["lse"], "loss": st["loss"]}
    if op == "loss_bwd":
        B.moe_router_loss_backward(st["handle"][0], st["dloss"], st["logits"], c["n_seq"], st["seq_off"], st["mask"],
                                   st["tokens"], st["counts"], st["lse"], st["dlogits"])
        return {"dlogits": st["dlogits"]}
    if op == "dropout":
        B.moe_dropout(st["x"], st["residual"], c["p"], st["rng"], st["out"])
        return {"out": st["out"]}
    dims, plan = st["handle"]
    B.moe_combine_dropout(dims, plan, st["Y"], True, st["residual"], c["p"], st["rng"], st["out"])
    return {"out": st["out"]}


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    d = lambda t: t.to(torch.float64)  # noqa: E731
    op = case["op"]
    if op.startswith("linear"):
        N = case["N"]
        if op == "linear_fwd":
            z = torch.mm(d(st["X"]), d(st["W"]).t())
            z = z + d(st["bias"]) if st["bias"] is not None else z
            y = z
            if case["act"] == "relu":
                y = torch.where(z > 0, z, 0.0)
            elif case["act"] == "gelu":
                y = z * torch.special.ndtr(z)
            elif case["act"] in ("silu", "swiglu"):
                y = z[:, :N] * torch.sigmoid(z[:, :N]) * (z[:, N:] if case["act"] == "swiglu" else 1.0)
            if st["residual"] is not None:
                y = d(st["residual"]) + y
            return {"out": y, "Z": z} if case["save"] else {"out": y}
        dz = d(st["dY"])
        if case["act"] == "relu":
            dz = torch.where(d(st["Z"]) > 0, dz, 0.0)
        elif case["act"] == "gelu":
            z = d(st["Z"])
            dz = dz * (torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi))
        elif case["act"] in ("silu", "swiglu"):
            g = d(st["Z"])[:, :N]
            s = torch.sigmoid(g)
            slope = s + g * s * torch.sigmoid(-g)
            dz = torch.cat([dz * d(st["Z"])[:, N:] * slope, dz * g * s], 1) if case["act"] == "swiglu" else dz * slope
        r = {"dX": torch.mm(dz, d(st["W"])), "dW": torch.mm(dz.t(), d(st["X"]))}
        if st["dbias"] is not None:
            r["dbias"] = torch.mm(torch.ones(1, case["M"], dtype=torch.float64, device="cuda"), dz)[0]
        return r
    if op.startswith("loss"):
        T, E, K, S = case["T"], case["E"], case["K"], case["n_seq"]
        x = d(st["logits"])
        off = st["seq_off"].tolist()
        on = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"] != 0
        picked = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_add_(
            1, st["topk_idx"].long(), torch.ones(T, K, dtype=torch.float64, device="cuda"))
        p = torch.softmax(x, 1)
        lse = torch.logsumexp(x, 1)
        spans = [(slice(off[s], off[s + 1]), on[off[s]:off[s + 1]]) for s in range(S)]
        tokens = torch.stack([m.sum() for _, m in spans])
        n = max(1, int(tokens.sum()))
        counts = torch.stack([picked[a][m].sum(0) for a, m in spans])
        if op == "loss_fwd":
            prob = torch.stack([p[a][m].sum(0) for a, m in spans])
            balance = sum((E / (K * max(1, int(tokens[s])) * n) * (counts[s] * prob[s]).sum() for s in range(S)))
            z = sum(lse[a][m].square().sum() for a, m in spans) / n
            return {"tokens": tokens.to(torch.int32), "counts": counts.to(torch.int32), "prob": prob, "lse": lse,
                    "loss": torch.stack([balance, z])}
        grad = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        wb, wz = (float(v) for v in st["dloss"])
        for s, (a, m) in enumerate(spans):
            if not int(tokens[s]):
                continue
            f = counts[s] * (wb * E / (K * int(tokens[s]) * n))
            gs = p[a] * (f - (p[a] @ f)[:, None] + (2 * wz / n) * lse[a][:, None])
            grad[a] = gs * m[:, None]
        return {"dlogits": grad}
    # dropout: the generator's products taken whole (64-bit words wrap, their bits are right)
    rows, cols = (case["rows"], case["cols"]) if op == "dropout" else (case["T"], case["d"])
    full = 0xFFFFFFFF
    seed_w, off_w = (int(v) for v in st["rng"])
    g = torch.arange(rows * ((cols + 7) // 8), dtype=torch.int64, device="cuda")
    n8 = (cols + 7) // 8
    ctr = [g % n8, torch.div(g, n8, rounding_mode="floor"), torch.full_like(g, off_w & full), torch.full_like(g, off_w >> 32)]
    key = [seed_w & full, seed_w >> 32]
    for _ in range(10):
        a, b = ctr[0] * 0xD2511F53, ctr[2] * 0xCD9E8D57
        ctr = [((b >> 32) & full) ^ ctr[1] ^ key[0], b & full, ((a >> 32) & full) ^ ctr[3] ^ key[1], a & full]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    t = int(case["p"] * 65536 + 0.5)
    kept = torch.zeros(rows * n8, 8, dtype=torch.bool, device="cuda")
    for j in range(4):
        kept[:, 2 * j] = (ctr[j] % 65536) >= t
        kept[:, 2 * j + 1] = torch.div(ctr[j], 65536, rounding_mode="floor") >= t
    kept = kept.reshape(rows, n8 * 8)[:, :cols]
    if op == "dropout":
        x = d(st["x"])
    else:
        K = case["K"]
        x = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
        r = st["plan"]["tok_row"].long().reshape(rows, K)
        for k in range(K):
            x += d(st["plan"]["row_w"])[r[:, k]][:, None] * d(st["Y"][r[:, k]])
    y = x * (kept.double() / (1 - t / 65536) if t < 65536 else 0.0)
    return {"out": y if st["residual"] is None else y + d(st["residual"])}
