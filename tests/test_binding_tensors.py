"""The binding's checks of the tensors that the norm, gradient and 4-bit calls take: each call below is refused before
anything reaches the library; no GPU needed."""
import pytest
import torch

from mixture_experts_layer_lds_amd import binding as B

BF, F, I = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    """CPU tensors count as on the current device, and a call that passes the checks raises Reached."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(B, "_stream_on", lambda dev, stream: None)
    real = B.lib()

    class Stub:
        def __getattr__(self, name):
            if name in ("moe_norm", "moe_norm_backward", "moe_grad_norm", "moe_grad_clip", "moe_linear_w4", "moe_decode_w4"):
                def reached(*a):
                    raise Reached(name)
                return reached
            return getattr(real, name)

    monkeypatch.setattr(B, "lib", lambda: Stub())


class Reached(Exception):
    pass


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def check(call, good, bad):
    """call(**good) passes; replacing one argument by each of its bad tensors does not."""
    with pytest.raises(Reached):
        call(**good)
    for name, tensors in bad.items():
        for t in tensors:
            with pytest.raises(B.MoEError, match="workspace" if name == "ws" else name):
                call(**dict(good, **{name: t}))


ROWS = [z(5, 9), z(4, 8), z(5, 8, dtype=F), z(8, 5).t(), z(5, 16)[:, ::2], z(5, 16)[:, :8], torch.zeros(5, 8, dtype=torch.float16)]
VEC = [z(7, dtype=F), z(8), z(8, dtype=torch.float64), z(16, dtype=F)[::2]]


def test_norm():
    d = B.make_norm_dims(5, 8, "bf16")
    good = dict(x=z(5, 8), residual=z(5, 8), weight=z(8, dtype=F), bias=z(9, dtype=F), sum=z(5, 8), y=z(5, 8), mean=z(5, dtype=F), rstd=z(6, dtype=F))
    stat = [z(4, dtype=F), z(5), z(10, dtype=F)[::2]]
    check(lambda **k: B.moe_norm(d, **k), good, dict(x=ROWS, residual=ROWS, sum=ROWS, y=ROWS, weight=VEC, bias=VEC, mean=stat, rstd=stat))
    with pytest.raises(B.MoEError, match="weight is torch.float32, torch.bfloat16 expected"):
        B.moe_norm(B.make_norm_dims(5, 8, "bf16", wtype="bf16"), **good)
    # a bf16 vector with the default wtype
    with pytest.raises(B.MoEError, match="weight is torch.bfloat16, torch.float32 expected"):
        B.moe_norm(d, **dict(good, weight=z(8)))
    f32 = {k: v.float() for k, v in good.items()}
    with pytest.raises(Reached):
        B.moe_norm(B.make_norm_dims(5, 8, "f32"), **f32)


def test_strides():
    d = B.make_norm_dims(5, 8, "bf16", ldx=12, ldy=12)
    wide = z(5, 12)
    go = lambda x, y: B.moe_norm(d, x, None, None, None, None, y, None, None)  # noqa: E731
    for x in (wide, wide[:, :8], wide[:, 4:], z(60), z(6, 12)[1:, :8], z(1, 5, 12)):
        with pytest.raises(Reached):
            go(x, wide)
    # (a flat buffer without the last row's gap; a view whose storage ends in the last row)
    with pytest.raises(Reached):
        go(z(56), wide)
    for x in (z(55), z(5, 8), z(5, 16)[:, :8], wide[:, 5:], wide[1:, :8], z(5, 24)[:, :12]):
        with pytest.raises(B.MoEError, match="x"):
            go(x, wide)
    # tensors of three dimensions: rows at one distance or not
    three = B.make_norm_dims(6, 8, "bf16", ldx=12)
    with pytest.raises(Reached):
        B.moe_norm(three, z(2, 3, 12)[:, :, :8], None, None, None, None, z(2, 3, 8), None, None)
    with pytest.raises(B.MoEError, match="one distance"):
        B.moe_norm(three, z(2, 4, 12)[:, :3, :8], None, None, None, None, z(2, 3, 8), None, None)
    # one row has no stride, no rows nothing at all
    with pytest.raises(Reached):
        B.moe_norm(B.make_norm_dims(1, 8, "bf16"), z(1, 12)[:, :8], None, None, None, None, z(8), None, None)
    with pytest.raises(Reached):
        B.moe_norm(B.make_norm_dims(0, 8, "bf16"), z(0, 8), None, None, None, None, z(0, 8), None, None)


def test_norm_backward():
    d = B.make_norm_dims(5, 8, "bf16")
    nb = B.lib().moe_norm_workspace_bytes(d)
    good = dict(dy=z(5, 8), s=z(5, 8), weight=z(8, dtype=F), mean=z(5, dtype=F), rstd=z(5, dtype=F), dsum=z(5, 8), dx=z(5, 8), dweight=z(8, dtype=F),
                dbias=z(8, dtype=F), ws=torch.zeros(nb, dtype=torch.uint8), ws_bytes=nb)
    stat = [z(4, dtype=F), z(5)]
    check(lambda **k: B.moe_norm_backward(d, **k), good,
          dict(dy=ROWS, s=ROWS, dsum=ROWS, dx=ROWS, weight=VEC, dweight=VEC, dbias=VEC, mean=stat, rstd=stat, ws=[torch.zeros(nb - 1, dtype=torch.uint8)]))


def test_gradients():
    g = B.Gradients([z(100, dtype=F)])
    ws, nb = B.grad_workspace(g, "cpu")
    one = [z(0, dtype=F), z(1), z(1, dtype=torch.float64)]
    check(lambda **k: B.moe_grad_norm(g, **k), dict(norm=z(1, dtype=F), ws=ws, ws_bytes=nb), dict(norm=one, ws=[ws[1:]]))
    check(lambda **k: B.moe_grad_clip(g, 1.0, **k), dict(norm_in=z(1, dtype=F), norm=z(1, dtype=F), ws=ws, ws_bytes=nb), dict(norm=one, norm_in=one, ws=[ws[1:]]))


def test_linear_w4():
    w = B.make_w4(16, 64, "int4", 32, device="cpu")
    rows = lambda c: [z(5, c + 8), z(4, c), z(5, c, dtype=F), z(c, 5).t(), z(5, 2 * c)[:, :c]]  # noqa: E731
    for act, N in (("none", 16), ("swiglu", 8)):
        d = B.make_linear_dims(5, N, 64, "bf16", act)
        good = dict(X=z(5, 64), bias=z(16, dtype=F), residual=z(5, N), out=z(5, N), ws=torch.zeros(64, dtype=torch.uint8), ws_bytes=64)
        check(lambda **k: B.moe_linear_w4(d, W=w, **k), good,
              dict(X=rows(64), residual=rows(N), out=rows(N), bias=[z(15, dtype=F), z(16), z(32, dtype=F)[::2]], ws=[torch.zeros(63, dtype=torch.uint8)]))


def test_decode_w4():
    T, d, n, E, K = 3, 64, 64, 4, 2
    w = [B.make_w4(rows, k, "fp4", 32, device="cpu") for rows, k in ((E * n, d), (E * n, d), (E * d, n))]
    dims = B.make_dims(T, d, n, E, K)
    good = dict(X=z(T, d), W_r=z(E, d), bias=z(E, dtype=F), logits=z(T, E, dtype=F), topk_idx=z(T, K, dtype=I), topk_w=z(T, K, dtype=F), out=z(T, d),
                ws=torch.zeros(999, dtype=torch.uint8), ws_bytes=999)
    bad = {k: [v[1:].clone(), v.double(), torch.zeros(*v.shape[:-1], 2 * v.shape[-1], dtype=v.dtype)[..., ::2]] for k, v in good.items() if k not in ("ws", "ws_bytes")}
    check(lambda **k: B.moe_decode_w4(dims, W_gate=w[0], W_up=w[1], W_down=w[2], **k), good, dict(bad, ws=[torch.zeros(998, dtype=torch.uint8)]))
