"""Refusals of the block operators (dense projection, router losses, dropout): every call below fails
validation on the host, so no kernel is launched; no GPU needed."""
import ctypes

import pytest
import torch

from mixture_experts_layer_lds_amd import binding as B

FAKE = 1 << 20  # a non-null, 16-byte aligned address that is never dereferenced
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def ldims(**kw):
    d = B.make_linear_dims(64, 128, 256)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def linear(lib, d, X=FAKE, W=FAKE, bias=None, res=None, Z=None, out=FAKE, ws=FAKE, nb=BIG):
    return lib.moe_linear(ctypes.byref(d), X, W, bias, res, Z, out, ws, nb, None)


def linear_bwd(lib, d, dY=FAKE, X=FAKE, W=FAKE, Z=FAKE, dX=FAKE, dW=FAKE, db=None, ws=FAKE, nb=BIG):
    return lib.moe_linear_backward(ctypes.byref(d), dY, X, W, Z, dX, dW, db, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), -1), (dict(M=(1 << 24) + 1), -1), (dict(N=0), -1), (dict(K=4), -1), (dict(N=65544), -1),
    (dict(K=65544), -1), (dict(N=100), -2), (dict(K=12), -2), (dict(dtype=5), -2), (dict(act=5), -1), (dict(act=-1), -1),
    (dict(flags=1), -1), (dict(ldx=248), -1), (dict(ldx=260), -2), (dict(ldr=120), -1), (dict(ldy=132), -2),
    (dict(ldy=-8), -1), (dict(ldx=1 << 41), -1),
])
def test_linear_refuses_bad_shapes(lib, kw, status):
    d = ldims(**kw)
    assert linear(lib, d) == status and lib.moe_last_error()
    assert linear_bwd(lib, d) == status
    assert B.moe_linear_workspace_bytes(d, B.LINEAR_FORWARD) == 0


def test_linear_refuses_bad_pointers_and_workspaces(lib):
    d = ldims(act=B.ACTS["gelu"])
    for kw in (dict(X=None), dict(W=None), dict(out=None), dict(X=FAKE + 2), dict(bias=FAKE + 4), dict(res=FAKE + 8), dict(Z=FAKE + 8)):
        assert linear(lib, d, **kw) == -1, kw
    need = B.moe_linear_workspace_bytes(d, B.LINEAR_FORWARD)
    if need:
        assert linear(lib, d, nb=need - 1) == -3 and linear(lib, d, ws=None) == -1
    for kw in (dict(dY=None), dict(X=None), dict(W=None), dict(Z=None), dict(dX=None, dW=None), dict(dX=FAKE + 4), dict(db=FAKE + 4)):
        assert linear_bwd(lib, d, **kw) == -1, kw
    need = B.moe_linear_workspace_bytes(d, B.LINEAR_BACKWARD)
    assert need >= 64 * 128 * 2 and linear_bwd(lib, d, nb=need - 1) == -3
    assert B.moe_linear_workspace_bytes(d, 7) == 0 and b"op" in lib.moe_last_error()
    assert lib.moe_linear(None, FAKE, FAKE, None, None, None, FAKE, FAKE, BIG, None) == -1
    assert linear(lib, ldims(M=0), X=None, W=None, out=None) == 0  # no rows: nothing to do


def test_router_loss_refusals(lib):
    d = B.make_dims(64, 64, 64, 8, 2, "f32")
    need = lib.moe_router_loss_workspace_bytes(ctypes.byref(d), 3)
    assert need > 0
    assert lib.moe_router_loss_workspace_bytes(ctypes.byref(d), 0) == 0
    names = ["logits", "topk", "n_seq", "off", "mask", "tokens", "counts", "prob", "lse", "loss", "ws", "nb"]

    def fwd(dm=d, **kw):
        a = dict(logits=FAKE, topk=FAKE, n_seq=3, off=FAKE, mask=None, tokens=FAKE, counts=FAKE, prob=FAKE, lse=FAKE,
                 loss=FAKE, ws=FAKE, nb=need)
        a.update(kw)
        return lib.moe_router_loss(ctypes.byref(dm), *[a[n] for n in names], None)

    for n in ("logits", "topk", "tokens", "counts", "prob", "lse", "loss", "ws"):
        assert fwd(**{n: None}) == -1, n
        assert fwd(**{n: FAKE + 4}) == -1, n
    assert fwd(off=None) == -1 and b"seq_off" in lib.moe_last_error()
    assert fwd(n_seq=0) == -1 and fwd(n_seq=(1 << 20) + 1) == -1
    assert fwd(off=FAKE + 4) == -1 and fwd(mask=FAKE + 1) == -1
    assert fwd(nb=need - 1) == -3
    assert fwd(dm=B.make_dims(64, 64, 64, 8, 9, "f32")) == -1

    def bwd(**kw):
        a = dict(dloss=FAKE, logits=FAKE, n_seq=3, off=FAKE, mask=None, tokens=FAKE, counts=FAKE, lse=FAKE, dl=FAKE)
        a.update(kw)
        return lib.moe_router_loss_backward(ctypes.byref(d), *[a[n] for n in ("dloss", "logits", "n_seq", "off", "mask", "tokens", "counts", "lse", "dl")], None)

    for n in ("dloss", "logits", "tokens", "counts", "lse", "dl"):
        assert bwd(**{n: None}) == -1, n
    assert bwd(off=None) == -1 and bwd(n_seq=0) == -1


def test_dropout_refusals(lib):
    def drop(rows=4, cols=16, dtype=1, x=FAKE, ldx=16, res=None, ldr=0, p=0.1, rng=FAKE, out=FAKE, ldo=16):
        return lib.moe_dropout(rows, cols, dtype, x, ldx, res, ldr, p, rng, out, ldo, None)

    assert drop(rows=-1) == -1 and drop(cols=0) == -1 and drop(cols=(1 << 30) + 1, ldx=1 << 31, ldo=1 << 31) == -1
    assert drop(rows=1 << 30, cols=32, ldx=32, ldo=32) == -2
    assert drop(dtype=3) == -2
    assert drop(ldx=15) == -1 and drop(ldo=8) == -1 and drop(res=FAKE, ldr=3) == -1
    for p in (-0.01, 1.01, float("nan")):
        assert drop(p=p) == -1 and b"probability" in lib.moe_last_error()
    assert drop(rng=None) == -1 and drop(x=None) == -1 and drop(out=None) == -1 and drop(x=FAKE + 2) == -1
    assert drop(rows=0, x=None, out=None) == 0
    d = B.make_dims(64, 64, 64, 8, 2)
    plan = B.PlanStruct(*([FAKE] * 9))
    comb = lambda Y=FAKE, res=None, p=0.5, rng=FAKE, out=FAKE: lib.moe_combine_dropout(  # noqa: E731
        ctypes.byref(d), ctypes.byref(plan), Y, 1, res, p, rng, out, None)
    assert comb(Y=None) == -1 and comb(res=FAKE + 2) == -1 and comb(p=2.0) == -1 and comb(rng=None) == -1 and comb(out=None) == -1


def test_dropout_binding_checks_tensors():
    x = torch.zeros(4, 16)
    rng = torch.zeros(2, dtype=torch.int64)
    bad = [dict(out=torch.zeros(4, 15)), dict(out=torch.zeros(16, 4).t()), dict(residual=torch.zeros(4, 16, dtype=torch.bfloat16)),
           dict(rng=torch.zeros(2, dtype=torch.int32)), dict(rng=torch.zeros(1, dtype=torch.int64)), dict(x=torch.zeros(4, 16).half())]
    for kw in bad:
        a = dict(x=x, residual=None, rng=rng, out=torch.zeros(4, 16))
        a.update(kw)
        with pytest.raises(B.MoEError):
            B.moe_dropout(a["x"], a["residual"], 0.1, a["rng"], a["out"])


def test_backward_aux_refuses_a_misaligned_gradient(lib):
    d = B.make_dims(64, 64, 64, 8, 2)
    plan = B.PlanStruct(*([FAKE] * 9))
    r = lib.moe_backward_aux(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(plan), None, FAKE + 4, FAKE,
                             FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None)
    assert r == -1 and b"dLogits_aux" in lib.moe_last_error()


def test_gradients_refuse_the_array_they_read(lib):
    d = B.make_dims(64, 64, 64, 8, 2)
    plan = B.PlanStruct(*([FAKE] * 9))
    r = lib.moe_backward_aux(ctypes.byref(d), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(plan), None, FAKE + 64, FAKE,
                             FAKE, FAKE, FAKE, FAKE, FAKE + 64, FAKE, FAKE, BIG, None)
    assert r == -1 and b"dLogits_aux" in lib.moe_last_error()
    r = lib.moe_router_loss_backward(ctypes.byref(d), FAKE, FAKE + 64, 1, None, None, FAKE, FAKE, FAKE, FAKE + 64, None)
    assert r == -1 and b"logits" in lib.moe_last_error()


def test_linear_plan_query(lib):
    d = ldims(M=1)
    assert B.moe_linear_plan(d, B.LINEAR_OUT) == (0, 1, False)
    assert B.moe_linear_plan(ldims(M=8192, N=8192, K=8192), B.LINEAR_OUT) == (256, 1, False)
    assert lib.moe_linear_plan(ctypes.byref(d), B.LINEAR_DW, None, None) in (64, 128, 256)
    assert lib.moe_linear_plan(ctypes.byref(d), 3, None, None) == -1 and lib.moe_linear_plan(None, 0, None, None) == -1
    assert lib.moe_linear_plan(ctypes.byref(ldims(N=100)), 0, None, None) == -2


@pytest.mark.parametrize("M,N,K", [(3000, 2000, 1000), (2904, 1800, 1000), (2504, 1496, 1496), (1500, 1000, 2000), (5000, 328, 1000)])
def test_pairs_off_the_lines_avoid_small_tiles(lib, M, N, K):
    """Rows that do not start on 128-byte lines cost small tiles as much in a pair of products as apart."""
    d = B.make_linear_dims(M, N, K)
    for product in (B.LINEAR_DX, B.LINEAR_DW):
        tile, _, paired = B.moe_linear_plan(d, product)
        assert not paired or tile == 128


def test_dropout_binding_refuses_generator_words_that_the_kernel_cannot_read():
    """The kernel dereferences rng: words in host memory (where seeds are made), on another device, apart
    from each other, or of another kind are refused before any launch."""
    x, words = torch.zeros(4, 16), torch.zeros(2, dtype=torch.int64)
    d = B.make_dims(64, 64, 64, 8, 2)

    class NoPlan:
        def ref(self):
            raise AssertionError("reached the library")

    for rng, where in ((words, "cpu"), (words.to("meta"), "meta"), (torch.zeros(4, dtype=torch.int64)[::2], "consecutive"),
                       (torch.zeros(2, dtype=torch.float64), "64-bit"), (torch.zeros(1, dtype=torch.int64), "64-bit")):
        with pytest.raises(B.MoEError, match=where):
            B.moe_dropout(x, None, 0.1, rng, torch.zeros(4, 16))
        with pytest.raises((B.MoEError, AssertionError), match=where):
            B.moe_combine_dropout(d, NoPlan(), x, True, None, 0.1, rng, torch.zeros(64, 64))
