"""Refusals of the calls on 4-bit weights: every call below fails validation on the host (or has nothing
to do), so no kernel is launched; no GPU needed."""
import ctypes

import pytest
import torch

from mixture_experts_layer_lds_amd import binding as B

FAKE = 1 << 20  # a non-null, 16-byte aligned address that is never dereferenced
BIG = 1 << 50
ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def w4(codes=FAKE, scales=FAKE, format=0, group=64):
    return B.W4Struct(codes, scales, format, group)


BAD_FORMATS = [(dict(format=2), -1), (dict(format=-1), -1), (dict(group=16), -2), (dict(group=0), -2), (dict(group=96), -2),
               (dict(format=1, group=64), -2), (dict(codes=None), -1), (dict(codes=FAKE + 8), -1), (dict(scales=None), -1), (dict(scales=FAKE + 2), -1)]


def test_scale_bytes(lib):
    assert lib.moe_w4_scale_bytes(10, 256, 0, 64) == 10 * 4 * 2 and lib.moe_w4_scale_bytes(10, 160, 1, 32) == 2 * 10 * 4
    for a in ((-1, 256, 0, 64), (10, 0, 0, 64), (10, 65600, 0, 64), (10, 96, 0, 64), (10, 256, 3, 64), (10, 256, 1, 64), ((1 << 31) + 1, 256, 0, 64)):
        assert lib.moe_w4_scale_bytes(*a) == 0 and lib.moe_last_error()


@pytest.mark.parametrize("kw,status", BAD_FORMATS)
def test_bad_descriptors(lib, kw, status):
    w, ok = w4(**kw), w4()
    d, m = B.make_linear_dims(4, 64, 256), B.make_dims(4, 256, 128, 8, 2)
    assert lib.moe_quantize_w4(8, 256, 1, FAKE, ref(w), None) == status
    assert lib.moe_dequantize_w4(8, 256, 1, ref(w), FAKE, None) == status
    assert lib.moe_linear_w4(ref(d), FAKE, ref(w), None, None, FAKE * 2, None, 0, None) == status
    for three in ((w, ok, ok), (ok, w, ok), (ok, ok, w)):
        assert lib.moe_decode_w4(ref(m), FAKE, FAKE, None, *[ref(x) for x in three], FAKE, FAKE, FAKE, FAKE, FAKE, BIG, None) == status


def test_quantise_refusals(lib):
    w = w4()
    for rows, K, dtype, status in ((-1, 256, 1, -1), (1 << 32, 256, 1, -1), (8, 0, 1, -1), (8, 100, 1, -2), (8, 65600, 1, -1), (8, 256, 2, -2)):
        assert lib.moe_quantize_w4(rows, K, dtype, FAKE, ref(w), None) == status
        assert lib.moe_dequantize_w4(rows, K, dtype, ref(w), FAKE, None) == status
    assert lib.moe_quantize_w4(8, 256, 1, None, ref(w), None) == -1 and lib.moe_quantize_w4(8, 256, 1, FAKE + 4, ref(w), None) == -1
    assert lib.moe_dequantize_w4(8, 256, 1, ref(w), None, None) == -1 and lib.moe_dequantize_w4(8, 256, 1, ref(w), FAKE + 2, None) == -1
    assert lib.moe_quantize_w4(8, 256, 1, FAKE, None, None) == -1 and lib.moe_dequantize_w4(8, 256, 1, None, FAKE, None) == -1
    assert lib.moe_quantize_w4(0, 256, 1, None, ref(w), None) == 0 and lib.moe_dequantize_w4(0, 256, 1, ref(w), None, None) == 0


def test_linear_refusals(lib):
    w = w4(group=32)

    def lin(d, X=FAKE, W=w, bias=None, res=None, out=FAKE * 2, ws=FAKE, nb=BIG):
        return lib.moe_linear_w4(ref(d), X, ref(W) if W else None, bias, res, out, ws, nb, None)

    def ldims(**kw):
        d = B.make_linear_dims(100, 64, 256)
        for k, v in kw.items():
            setattr(d, k, v)
        return d

    for kw, status in ((dict(M=-1), -1), (dict(N=100), -2), (dict(K=40), -2), (dict(dtype=0), -2), (dict(act=5), -1), (dict(flags=1), -1),
                       (dict(ldx=8), -1), (dict(ldx=260), -2)):
        d = ldims(**kw)
        assert lin(d) == status, kw
        assert lib.moe_linear_w4_workspace_bytes(ref(d)) == 0
    assert lin(ldims(K=96), W=w4(group=64)) == -2
    for kw in (dict(X=None), dict(out=None), dict(W=None), dict(X=FAKE + 2), dict(bias=FAKE + 4), dict(res=FAKE + 2), dict(out=FAKE)):
        assert lin(ldims(), **kw) == -1, kw
    assert lin(ldims(ldr=72), res=FAKE * 2) == -1 and b"stride" in lib.moe_last_error()
    many = ldims(M=1100)
    need = lib.moe_linear_w4_workspace_bytes(ref(many))
    assert need >= 64 * 256 * 2 and lin(many, nb=need - 1) == -3 and lin(many, ws=None) == -1
    assert B.moe_linear_w4_plan(many) == "expanded" and B.moe_linear_w4_plan(ldims(M=64)) == "streamed"
    assert lib.moe_linear_w4_plan(ref(ldims(N=100))) == -2 and lib.moe_linear_w4_plan(None) == -1
    assert lin(ldims(M=0), X=None, W=None, out=None, ws=None, nb=0) == 0


def test_decode_refusals(lib):
    m, w = B.make_dims(4, 256, 128, 8, 2), w4()
    need = B.moe_workspace_bytes(m, B.OP_DECODE)
    names = ["X", "W_r", "bias", "g", "u", "d", "logits", "idx", "w", "out", "ws", "nb"]

    def dec(dm=m, **kw):
        a = dict(X=FAKE, W_r=FAKE, bias=None, g=w, u=w, d=w, logits=FAKE, idx=FAKE, w=FAKE, out=FAKE, ws=FAKE, nb=need)
        a.update(kw)
        for k in "gud":
            a[k] = ref(a[k]) if a[k] else None
        return lib.moe_decode_w4(ref(dm), *[a[k] for k in names], None)

    for k in ("X", "W_r", "logits", "idx", "w", "out", "ws"):
        assert dec(**{k: None}) == -1, k
        assert dec(**{k: FAKE + 4}) == -1, k
    for k in "gud":
        assert dec(**{k: None}) == -1
    assert dec(bias=FAKE + 4) == -1 and dec(nb=need - 1) == -3
    assert dec(u=w4(group=32)) == -2 and dec(d=w4(format=1, group=32)) == -2 and b"one format" in lib.moe_last_error()
    assert dec(dm=B.make_dims(4, 256, 128, 8, 2, "f32")) == -2
    assert dec(dm=B.make_dims(4, 256, 128, 8, 2, round_mode=B.ROUND_UP)) == -2
    assert dec(dm=B.make_dims(1025, 256, 128, 8, 2)) == -2
    big = w4(group=128)
    assert dec(dm=B.make_dims(4, 192, 128, 8, 2), g=big, u=big, d=big) == -2  # d is not a multiple of the group
    assert dec(dm=B.make_dims(4, 128, 192, 8, 2), g=big, u=big, d=big) == -2


def test_binding_checks_tensors():
    codes, scales = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(2, 8, dtype=torch.bfloat16)
    w = B.W4(codes, scales, "int4", 64)
    assert (w.rows, w.K) == (8, 128)
    assert B.W4(codes.view(2, 4, 64), scales, "int4", 64).rows == 8
    for c, s, f, g in ((codes.int(), scales, "int4", 64), (codes.t(), scales, "int4", 64), (codes, scales.float(), "int4", 64), (codes, scales[:1], "int4", 64),
                       (codes, scales, "int4", 48), (codes, scales, "fp4", 32), (codes, torch.zeros(1, 8, 4, dtype=torch.uint8), "fp4", 64),
                       (codes, scales.to("meta"), "int4", 64)):
        with pytest.raises(B.MoEError):
            B.W4(c, s, f, g)
    with pytest.raises(B.MoEError, match="expected"):
        B.moe_linear_w4(B.make_linear_dims(1, 16, 128), None, w, None, None, None, None, 0)
    with pytest.raises(B.MoEError, match="expected"):
        B.moe_linear_w4(B.make_linear_dims(1, 8, 128, "bf16", "swiglu"), None, w, None, None, None, None, 0)
    with pytest.raises(B.MoEError, match="expected"):
        B.moe_decode_w4(B.make_dims(1, 128, 64, 1, 1), None, None, None, w, w, w, None, None, None, None, None, 0)
    with pytest.raises(B.MoEError, match="contiguous"):
        B.moe_quantize_w4(torch.zeros(8, 127), w)
