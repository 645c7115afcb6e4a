"""moe_quantize_w4, moe_dequantize_w4 and moe_linear_w4 against the float64 oracle."""
import numpy as np
import pytest
import torch

from block_util import DT, HALF, U32, assert_guards, assert_within, check_replays, f64, strided
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from oracle import block as ob
from oracle import w4 as ow

pytestmark = pytest.mark.gpu

FORMATS = [("fp4", 32), ("int4", 32), ("int4", 64), ("int4", 128)]


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


def random_w4(rows, K, fmt, group, seed):
    """Random codes (all sixteen) and scales around 1 / sqrt(K), on the GPU and as values."""
    r = np.random.default_rng(seed)
    codes = r.integers(0, 16, (rows, K)).astype(np.uint8)
    if fmt == "int4":
        s = ow.bf16(((0.5 + r.random((rows, K // group))) * r.choice([1, -1], (rows, K // group)) / (5 * K ** 0.5)).astype(np.float32))
        t = torch.from_numpy(ow.store_scales(s, fmt)).to(torch.bfloat16).cuda()
    else:
        s = (127 - int(np.log2(3 * K ** 0.5)) + r.integers(-2, 3, (rows, K // 32))).astype(np.uint8)
        st = ow.store_scales(s, fmt)
        st.reshape(st.shape[0], rows, 4)[-1, :, (K // 32 - 1) % 4 + 1:] = 255  # (bytes past the row are not used)
        t = torch.from_numpy(st).cuda()
    return B.W4(torch.from_numpy(ow.pack(codes)).cuda(), t, fmt, group), codes, s, ow.values(codes, s, fmt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("rows,K", [(1, 128), (3, 256), (17, 384), (5, 8320), (1000, 128), (2, 65536)])
def test_quantise_and_expand(rows, K, fmt, group, dtype):
    g = torch.Generator().manual_seed(rows + K)
    x = (torch.randn(rows, K, generator=g) * torch.exp(torch.randn(rows, K, generator=g))).to(DT[dtype]).cuda()
    x[0, :group] = 0
    w = B.make_w4(rows, K, fmt, group)
    B.moe_quantize_w4(x, w)
    torch.cuda.synchronize()
    X = f64(x)
    codes, s = ow.quantize(X, fmt, group)
    got = ow.unpack(w.codes.cpu().numpy())
    stored = ow.store_scales(s, fmt)
    assert np.array_equal(f64(w.scales) if fmt == "int4" else w.scales.cpu().numpy(), stored)
    if fmt == "int4" and dtype == "f32":
        # the quotient is rounded to fp32 before it is rounded to an integer: where the two differ, x / s lies
        # within an fp32 step of a half, and either neighbour is nearest to that precision
        q = X / np.repeat(s, group, axis=1)
        edge = np.abs(np.abs(q - np.floor(q)) - 0.5) <= 8 * 2.0 ** -23
        assert np.all((got == codes) | edge) and np.abs(got.astype(int) - codes).max() <= 1
    elif fmt == "fp4":  # the sign of a zero is free
        assert np.array_equal(np.where(got == 8, 0, got), np.where(codes == 8, 0, codes))
    else:
        assert np.array_equal(got, codes)
    for out_type in ("bf16", "f32"):
        out = torch.empty(rows, K, dtype=DT[out_type], device="cuda")
        B.moe_dequantize_w4(w, out)
        v = ow.values(got, s, fmt)
        assert np.array_equal(f64(out), ow.bf16(v.astype(np.float32)) if out_type == "bf16" else v)


def test_every_fp4_code_and_scale_byte():
    """All 16 codes under all 255 finite scale bytes, expanded and multiplied: 2^-127 .. 2^127 times 0 .. 6."""
    rows, K = 256, 32
    codes = np.tile(np.arange(32) % 16, (rows, 1)).astype(np.uint8)
    s = np.minimum(np.arange(rows), 254)[:, None].astype(np.uint8)
    w = B.W4(torch.from_numpy(ow.pack(codes)).cuda(), torch.from_numpy(ow.store_scales(s, "fp4")).cuda(), "fp4", 32)
    V = ow.values(codes, s, "fp4")
    out = torch.empty(rows, K, device="cuda")
    B.moe_dequantize_w4(w, out)
    with np.errstate(over="ignore"):
        ref = V.astype(np.float32)  # (exact but for 2^128 and beyond, which is infinity: 2, 3, 4, 6 times 2^127 and the like)
    assert np.array_equal(f64(out), ref)
    # a token that picks one element returns the weight (bf16's normal range: the conversion's own zeros below it)
    dims = B.make_linear_dims(16, rows, K)
    y = torch.empty(16, rows, dtype=torch.bfloat16, device="cuda")
    for k0 in (0, 16):
        x = torch.zeros(16, K, dtype=torch.bfloat16, device="cuda")
        x[torch.arange(16), k0 + torch.arange(16)] = 1.0
        B.moe_linear_w4(dims, x, w, None, None, y, *B.linear_w4_workspace(dims))
        got = f64(y).T
        ok = (np.abs(V) >= 2.0 ** -126) & (np.abs(V) < 3.3e38) | (V == 0)
        # (a row with weights beyond the range has infinities times zero)
        ok &= ~np.isinf(ref).any(axis=1)[:, None]
        assert ok.sum() > 200 * 32 and np.array_equal(got[ok[:, k0:k0 + 16]], V[:, k0:k0 + 16][ok[:, k0:k0 + 16]])


def linear_bounds(X, codes, s, V, fmt, group, streamed):
    """|z - exact z| of the streaming kernel: exact products, fp32 sums.  INT4: within a group 33 additions per
    32 elements of terms up to 16 s |x| (1 + c / 16 + 1.5), then one addition per group in each of at least 1
    (K < 2048) or 4 waves, 8 waves at most; FP4: one addition per element.  Expanded weights: one per element."""
    K = X.shape[1]
    ax = np.abs(X)
    if fmt == "fp4" or not streamed:
        chain = (K if K < 2048 else K // 4) + 16 if streamed else K + 64
        return chain * U32 * (ax @ np.abs(V).T)
    groups = K // group
    sg = np.abs(s)                                                       # [rows, groups]
    wide = np.repeat(sg, group, axis=1) * 16 * (1 + codes / 16.0 + 1.5)
    inner = 33 * (group // 32) * U32 * (ax @ wide.T)
    part = np.abs(np.einsum("mgk,ngk->mng", X.reshape(len(X), groups, group), V.reshape(len(V), groups, group))).sum(2)
    return inner + ((groups if K < 2048 else groups // 4 + 1) + 12) * U32 * part


def check_linear(M, N, K, fmt, group, act, bias, residual, pad, seed=0):
    NW = 2 * N if act == "swiglu" else N
    w, codes, s, V = random_w4(NW, K, fmt, group, seed + N + K)
    g = torch.Generator().manual_seed(M + 3 * N + 7 * K)
    x, _ = strided(M, K, pad, "bf16", torch.randn(M, K, generator=g))
    b = torch.randn(NW, generator=g).cuda() * 0.5 if bias else None
    res = strided(M, N, pad, "bf16", torch.randn(M, N, generator=g))[0] if residual else None
    out, base = strided(M, N, pad, "bf16", extra_rows=2)
    dims = B.make_linear_dims(M, N, K, "bf16", act, ldx=K + pad, ldr=N + pad, ldy=N + pad)
    ws, nb = B.linear_w4_workspace(dims)
    B.moe_linear_w4(dims, x, w, b, res, out, ws, nb)
    torch.cuda.synchronize()
    X = f64(x)
    streamed = B.moe_linear_w4_plan(dims) == "streamed"
    if not streamed:
        V = ow.bf16(V.astype(np.float32))  # (exact products of 4 and 8 bits, rounded once)
    z = X @ V.T + (f64(b) if bias else 0.0)
    ez = linear_bounds(X, codes, s, V, fmt, group, streamed) + 2 * U32 * np.abs(z)
    y = ob.activation(z, act)
    if act == "swiglu":
        a, u, ea, eu = z[:, :N], z[:, N:], ez[:, :N], ez[:, N:]
        ey = 1.1 * ea * (np.abs(u) + eu) + np.abs(ob.activation(a, "silu")) * eu
        size = np.abs(y)
    else:
        ey, size = 1.13 * ez, np.abs(y)
    # the activation's own arithmetic: exponentials off by a few steps times their argument
    ey = ey + size * U32 * (8 + 2 * np.abs(z[:, :N])) + 1e-30
    if act == "gelu":
        ey = ey + 4e-5 * np.abs(y)  # (degree 5: 4.7e-6 of the tail, half a bf16 step is 400 times that)
    r = f64(res) if residual else 0.0
    ref = y + r
    assert_within("out", f64(out), ref, HALF["bf16"] * (np.abs(ref) + ey) + ey + U32 * (np.abs(y) + np.abs(r)))
    assert_guards(base, M, N, "out")
    if residual:
        B.moe_linear_w4(dims, x, w, b, res, res, ws, nb)
        assert torch.equal(res, out)


# whole blocks of 128, parts of 32, 64 and 96, fewer than one; one to many waves; tiles of 16 and 8 left over
@pytest.mark.parametrize("M,N,K,act,bias,residual,pad", [
    (1, 8, 32, "none", False, False, 0), (1, 16, 64, "swiglu", True, False, 0), (2, 24, 96, "relu", True, True, 8), (5, 40, 128, "silu", False, True, 0),
    (1, 1000, 160, "gelu", True, False, 8), (16, 56, 2144, "swiglu", True, True, 24), (17, 72, 4192, "none", False, True, 0), (1, 264, 7168, "swiglu", False, False, 0),
    (13, 4096, 512, "none", True, True, 0), (31, 200, 1120, "gelu", False, True, 8), (33, 104, 864, "swiglu", True, True, 0), (64, 48, 352, "none", False, False, 8),
    (65, 136, 416, "none", True, True, 0), (200, 264, 1088, "swiglu", True, True, 8), (300, 512, 2048, "relu", False, False, 0), (3, 8, 16384, "none", False, False, 0),
    # tiles: one and two row tiles a wave, slices, ragged tokens, rows and blocks, SwiGLU on both
    (129, 4104, 2080, "none", True, True, 8), (255, 1992, 1056, "swiglu", True, False, 0), (700, 4104, 416, "gelu", False, True, 0), (1024, 2056, 288, "swiglu", False, True, 8),
    (129, 7168, 2048, "relu", True, True, 0), (100, 2048, 4096, "swiglu", True, False, 0), (1000, 4096, 160, "none", False, False, 0), (66, 3976, 4192, "silu", False, False, 0), (513, 8, 8192, "relu", True, True, 0),
    # expanded
    (1025, 136, 416, "none", True, True, 0), (1100, 72, 1088, "swiglu", True, True, 8), (1300, 264, 32, "relu", False, False, 0),
])
@pytest.mark.parametrize("fmt,group", FORMATS)
def test_linear_matches_oracle(M, N, K, act, bias, residual, pad, fmt, group):
    K = max(K // group, 1) * group
    check_linear(M, N, K, fmt, group, act, bias, residual, pad)


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_large_shapes(fmt, group):
    check_linear(1, 16384, 4096, fmt, group, "none", True, False, 0)
    check_linear(16, 2048, 7168, fmt, group, "swiglu", False, False, 0)


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_rows_are_independent(fmt, group):
    """A token's result does not depend on the others of its group, nor on infinities and NaN among them."""
    M, N, K = 16, 128, 512
    w = random_w4(N, K, fmt, group, 5)[0]
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    dims = B.make_linear_dims(M, N, K)
    y, y1 = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws, nb = B.linear_w4_workspace(dims)
    B.moe_linear_w4(dims, x, w, None, None, y, ws, nb)
    for t in (0, 7, 15):
        other = torch.randn(M, K, generator=torch.Generator().manual_seed(t + 2)).bfloat16().cuda()
        other[t] = x[t]
        B.moe_linear_w4(dims, other, w, None, None, y1, ws, nb)
        assert torch.equal(y1[t], y[t])
    bad = x.clone()
    bad[3, 5], bad[9, 500] = float("nan"), float("inf")
    z = torch.empty_like(y)
    B.moe_linear_w4(dims, bad, w, None, None, z, ws, nb)
    keep = [t for t in range(M) if t not in (3, 9)]
    assert torch.equal(z[keep], y[keep]) and bool(z[3].isnan().all()) and not bool(z[9].isfinite().any())


def test_no_rows_and_no_weights():
    w = B.make_w4(64, 128, "fp4", 32)
    B.moe_linear_w4(B.make_linear_dims(0, 64, 128), None, w, None, None, None, None, 0)
    empty = B.W4(torch.empty(0, 64, dtype=torch.uint8, device="cuda"), torch.empty(1, 0, dtype=torch.bfloat16, device="cuda"), "int4", 128)
    B.moe_quantize_w4(torch.empty(0, 128, device="cuda"), empty)
    B.moe_dequantize_w4(empty, torch.empty(0, 128, device="cuda"))


def test_every_way_is_taken():
    way = lambda M, N, K, act="none": B.moe_linear_w4_plan(B.make_linear_dims(M, N, K, "bf16", act))  # noqa: E731
    assert {way(M, 7168, 2048) for M in (1, 5, 16, 17, 64)} == {"streamed"} and way(200, 512, 512) == "streamed"
    assert {way(M, 7168, 2048) for M in (129, 256, 777, 1024)} == {"tiled"} and way(700, 4104, 416) == way(1024, 2056, 288, "swiglu") == "tiled"
    assert way(1025, 8, 32) == way(5000, 4096, 4096) == "expanded"


@pytest.mark.parametrize("fmt,group", FORMATS)
def test_tiles_hold_infinities_and_nans_in_their_rows(fmt, group):
    M, N, K = 300, 4096, 2048 + 128
    w = random_w4(N, K, fmt, group, 5)[0]
    dims = B.make_linear_dims(M, N, K)
    assert B.moe_linear_w4_plan(dims) == "tiled"
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    y, z = (torch.empty(M, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws, nb = B.linear_w4_workspace(dims)
    B.moe_linear_w4(dims, x, w, None, None, y, ws, nb)
    x[3, 5], x[140, 2100], x[299, K - 1] = float("nan"), float("inf"), float("-inf")
    B.moe_linear_w4(dims, x, w, None, None, z, ws, nb)
    keep = [t for t in range(M) if t not in (3, 140, 299)]
    assert torch.equal(z[keep], y[keep]) and bool(z[3].isnan().all()) and not bool(z[140].isfinite().any()) and not bool(z[299].isfinite().any())


@pytest.mark.parametrize("M", [1, 24, 300, 1100])
def test_graph_replays_match_eager(M):
    N, K = 1800, 2048
    w = random_w4(2 * N, K, "int4", 64, 2)[0]
    x = torch.randn(M, K, device="cuda").bfloat16()
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    dims = B.make_linear_dims(M, N, K, "bf16", "swiglu")
    ws, nb = B.linear_w4_workspace(dims)
    check_replays(lambda: B.moe_linear_w4(dims, x, w, None, None, out, ws, nb), dict(out=out))


def test_code_offsets_past_32_bits():
    """Codes of more than 2^32 bytes (W of 65536 x 65536 is 2^31; the experts' of one matrix are longer): the last rows'
    quantisation and expansion."""
    rows, K = 2 * 65536 + 64, 65536
    w = B.make_w4(rows, K, "int4", 128)
    w.codes.fill_(0x88)
    w.scales.fill_(1.0)
    w.codes[-1, -16:] = torch.arange(16, dtype=torch.uint8, device="cuda") * 17
    w.scales[-1, -1] = 0.5
    last = B.W4(w.codes[-64:].contiguous(), w.scales[:, -64:].contiguous(), "int4", 128)
    out = torch.empty(64, K, dtype=torch.bfloat16, device="cuda")
    B.moe_dequantize_w4(last, out)
    whole = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    B.moe_dequantize_w4(w, whole)
    assert torch.equal(whole[-64:], out) and float(whole[-1, -1]) == 3.5 and int(whole[:-1].count_nonzero()) == 0
    again = B.make_w4(rows, K, "int4", 128)
    B.moe_quantize_w4(whole, again)
    back = torch.empty_like(out)
    B.moe_dequantize_w4(B.W4(again.codes[-64:].contiguous(), again.scales[:, -64:].contiguous(), "int4", 128), back)
    # the last group's largest value is -4 = -8 x 0.5: s = bf16(4 / 7), its values are off by at most half of it
    assert torch.equal(back[:-1], out[:-1]) and bool(((back[-1].float() - out[-1].float()).abs() <= 2 / 7 * 1.01).all())


@pytest.mark.parametrize("M,N,K", [(1, 520, 1024), (16, 264, 14336), (130, 2056, 4096), (1100, 264, 512)])
def test_calls_on_two_streams_with_their_own_workspaces(M, N, K):
    w = random_w4(N, K, "int4", 128, 9)[0]
    dims = B.make_linear_dims(M, N, K)
    g = torch.Generator().manual_seed(M)
    runs = [dict(x=torch.randn(M, K, generator=g).bfloat16().cuda(), out=torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), ws=B.linear_w4_workspace(dims))
            for _ in range(2)]

    def step(r):
        B.moe_linear_w4(dims, r["x"], w, None, None, r["out"], *r["ws"])

    for r in runs:
        step(r)
    torch.cuda.synchronize()
    want = [r["out"].clone() for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(5):
        for r in runs:
            r["out"].zero_()
        torch.cuda.synchronize()
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                step(r)
        torch.cuda.synchronize()
        for r, o in zip(runs, want):
            assert torch.equal(r["out"], o)
