"""Refusals of the norm and of gradient clipping: every call below fails validation on the host (or has
nothing to do), so no kernel is launched; no GPU needed."""
import ctypes

import pytest
import torch

from mixture_experts_layer_lds_amd import binding as B

FAKE = 1 << 20  # a non-null, 16-byte aligned address that is never dereferenced
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def ndims(**kw):
    d = B.make_norm_dims(64, 128)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def norm(lib, d, x=FAKE, res=None, w=FAKE, b=FAKE, s=None, y=FAKE * 2, mean=None, rstd=None):
    return lib.moe_norm(ctypes.byref(d), x, res, w, b, s, y, mean, rstd, None)


def norm_bwd(lib, d, dy=FAKE, s=FAKE * 2, w=FAKE, mean=FAKE, rstd=FAKE, dsum=None, dx=FAKE * 3, dw=FAKE * 4, db=FAKE * 5, ws=FAKE, nb=BIG):
    return lib.moe_norm_backward(ctypes.byref(d), dy, s, w, mean, rstd, dsum, dx, dw, db, ws, nb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -1), (dict(rows=1 << 31), -1), (dict(cols=0), -1), (dict(cols=65537), -1), (dict(dtype=2), -2), (dict(wtype=-1), -2),
    (dict(kind=2), -1), (dict(kind=-1), -1), (dict(eps=-1e-5), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1),
    (dict(flags=1), -1), (dict(ldx=127), -1), (dict(ldr=1), -1), (dict(lds=-128), -1), (dict(ldy=(1 << 40) + 1), -1),
])
def test_norm_refuses_bad_shapes(lib, kw, status):
    d = ndims(**kw)
    assert norm(lib, d) == status and lib.moe_last_error()
    assert norm_bwd(lib, d) == status
    assert lib.moe_norm_workspace_bytes(ctypes.byref(d)) == 0


def test_norm_refuses_bad_pointers(lib):
    d = ndims()
    for kw in (dict(x=None), dict(y=None), dict(x=FAKE + 2), dict(res=FAKE + 8), dict(w=FAKE + 4), dict(b=FAKE + 4), dict(y=FAKE + 2),
               dict(mean=FAKE + 4), dict(rstd=FAKE + 8), dict(s=FAKE * 3), dict(res=FAKE * 3, s=FAKE * 2)):
        assert norm(lib, d, **kw) == -1, kw
    assert b"same array" in lib.moe_last_error()
    assert lib.moe_norm(None, FAKE, None, None, None, None, FAKE, None, None, None) == -1
    # an output over an input with another stride
    assert norm(lib, ndims(ldx=136), y=FAKE) == -1 and b"stride" in lib.moe_last_error()
    assert norm(lib, ndims(ldr=136), res=FAKE * 2) == -1
    assert norm(lib, ndims(lds=136), res=FAKE * 3, s=FAKE) == -1 and norm(lib, ndims(lds=136), res=FAKE * 3, s=FAKE * 3) == -1
    assert norm(lib, ndims(rows=0), x=None, y=None) == 0


def test_norm_backward_refuses_bad_pointers_and_workspaces(lib):
    d = ndims()
    for kw in (dict(dy=None), dict(s=None), dict(mean=None), dict(rstd=None), dict(w=FAKE + 2), dict(dsum=FAKE + 2), dict(dx=FAKE + 2),
               dict(dw=FAKE + 4), dict(db=FAKE + 4), dict(dx=None, dw=None, db=None), dict(dw=FAKE * 4, db=FAKE * 4), dict(ws=None), dict(ws=FAKE + 8)):
        assert norm_bwd(lib, d, **kw) == -1, kw
    need = lib.moe_norm_workspace_bytes(ctypes.byref(d))
    assert need >= 2 * 128 * 4 and norm_bwd(lib, d, nb=need - 1) == -3
    for k in ("ldy", "lds", "ldr"):
        over = dict(ldy=FAKE, lds=FAKE * 2, ldr=FAKE * 6)[k]
        assert norm_bwd(lib, ndims(**{k: 136}), dsum=FAKE * 6, dx=over) == -1 and b"stride" in lib.moe_last_error()


def grads(*items):
    a = (B.GradStruct * max(len(items), 1))()
    for i, (src, dst, n, dtype) in enumerate(items):
        a[i] = B.GradStruct(src, dst, n, dtype, 0)
    return a


def test_gradient_table_refusals(lib):
    host = (ctypes.c_uint64 * 64)()
    at = (ctypes.addressof(host) + 15) // 16 * 16
    out = B.GradListStruct()
    tab = lambda g, count=1, table=at, nb=400, o=ctypes.byref(out): lib.moe_grad_table(g, count, table, nb, o)  # noqa: E731
    ok = grads((FAKE, None, 8193, 0))
    need = lib.moe_grad_table_bytes(ok, 1)
    assert need == 32 + 2 * 4 and tab(ok) == 0 and (out.table, out.count, out.chunks) == (None, 1, 2)
    assert tab(ok, nb=need) == 0 and tab(ok, nb=need - 1) == -3
    assert tab(ok, table=None) == -1 and tab(ok, table=at + 8) == -1 and tab(ok, o=None) == -1
    for count in (-1, (1 << 16) + 1):
        assert tab(ok, count=count) == -1 and lib.moe_grad_table_bytes(ok, count) == 0
    assert tab(None) == -1 and lib.moe_grad_table_bytes(None, 1) == 0
    for item, status in (((FAKE, FAKE, -1, 0), -1), ((FAKE, FAKE, (1 << 36) + 1, 0), -1), ((None, FAKE, 3, 0), -1), ((FAKE + 2, FAKE, 3, 0), -1),
                         ((FAKE, FAKE + 2, 3, 0), -1), ((FAKE + 1, FAKE, 3, 1), -1), ((FAKE, FAKE, 3, 2), -2)):
        assert tab(grads(item)) == status, item
        assert b"tensor 0" in lib.moe_last_error() and lib.moe_grad_table_bytes(grads(item), 1) == 0
    bad = grads((FAKE, FAKE, 10, 0))
    bad[0].reserved = 1
    assert tab(bad) == -1
    # shared memory: the same tensor twice, parts of one, a destination over another's source
    for two in (((FAKE, None, 10, 0), (FAKE, None, 10, 0)), ((FAKE, None, 10, 0), (FAKE + 36, None, 2, 0)), ((FAKE, FAKE * 2, 10, 0), (FAKE * 2 + 20, None, 4, 1)),
                ((FAKE, FAKE * 2, 10, 0), (FAKE * 3, FAKE * 2, 10, 0)), ((FAKE, FAKE + 4, 10, 0), (FAKE * 3, None, 1, 0))):
        assert tab(grads(*two), count=2) == -1 and b"share memory" in lib.moe_last_error()
    assert tab(grads((FAKE, None, 10, 0), (FAKE + 40, None, 10, 0)), count=2) == 0 and out.chunks == 2
    assert tab(grads(), count=0) == 0 and (out.count, out.chunks) == (0, 0) and lib.moe_grad_table_bytes(None, 0) > 0


def test_gradient_call_refusals(lib):
    need = lib.moe_grad_workspace_bytes()
    assert need > 0
    glist = lambda **kw: B.GradListStruct(**dict(dict(table=FAKE, count=1, chunks=1), **kw))  # noqa: E731
    nrm = lambda g=glist(), norm_=FAKE, ws=FAKE, nb=need: lib.moe_grad_norm(ctypes.byref(g), norm_, ws, nb, None)  # noqa: E731
    clp = lambda g=glist(), m=1.0, ni=None, norm_=FAKE, ws=FAKE, nb=need: lib.moe_grad_clip(ctypes.byref(g), m, ni, norm_, ws, nb, None)  # noqa: E731
    for f in (nrm, clp):
        for kw in (dict(table=None), dict(table=FAKE + 8), dict(count=-1), dict(count=(1 << 16) + 1), dict(chunks=-1)):
            assert f(g=glist(**kw)) == -1, kw
        assert f(norm_=None) == -1 and f(norm_=FAKE + 4) == -1 and f(ws=None) == -1 and f(ws=FAKE + 8) == -1 and f(nb=need - 1) == -3
    assert lib.moe_grad_norm(None, FAKE, FAKE, need, None) == -1 and lib.moe_grad_clip(None, 1.0, None, FAKE, FAKE, need, None) == -1
    for m in (-1.0, float("nan"), float("-inf")):
        assert clp(m=m) == -1 and b"max_norm" in lib.moe_last_error()
    assert clp(ni=FAKE + 4) == -1
    # with a norm given and nothing to scale there is nothing to do
    assert clp(g=glist(table=None, count=0, chunks=0), ni=FAKE, norm_=None, ws=None, nb=0) == 0


def test_gradient_list_checks_tensors():
    t = torch.zeros(64)
    for src, dst in (([t.half()], None), ([torch.zeros(8, 8).t()], None), ([t], [torch.zeros(63)]), ([t], [t.bfloat16()]), ([t], []),
                     ([t], [torch.zeros(128)[::2]]), ([t, t], None), ([t, t[10:20]], None), ([t], [torch.zeros(64, device="meta")])):
        with pytest.raises(B.MoEError):
            B.Gradients(src, dst)
    both = torch.zeros(100)
    with pytest.raises(B.MoEError, match="share memory"):
        B.Gradients([both[:60]], [both[40:100]])
    with pytest.raises(B.MoEError, match="share memory"):
        B.Gradients([both[:40], both[40:80]], [torch.zeros(40), both[:40]])
    g = B.Gradients([both[:40], both[40:80], both[80:80]])
    assert g.count == 3 and g.array[1].n == 40 and g.struct.chunks == 2
