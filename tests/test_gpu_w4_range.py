"""4-bit products where large elements of X meet weights of zero, and over the types' whole finite range."""
import numpy as np
import pytest
import torch

from block_util import HALF, U32, assert_within, f64
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from oracle import w4 as ow
from test_gpu_w4 import FORMATS, random_w4

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


def with_zero_columns(rows, K, fmt, group, seed, columns):
    """Random weights whose given columns are zero."""
    _, codes, s, _ = random_w4(rows, K, fmt, group, seed)
    codes[:, columns] = 8 if fmt == "int4" else 0
    return pack(codes, s, fmt, group) + (codes, s, ow.values(codes, s, fmt))


def pack(codes, s, fmt, group):
    t = torch.from_numpy(ow.store_scales(s, fmt))
    return (B.W4(torch.from_numpy(ow.pack(codes)).cuda(), (t.to(torch.bfloat16) if fmt == "int4" else t).cuda(), fmt, group),)


def linear(x, w, N):
    M, K = x.shape
    dims = B.make_linear_dims(M, N, K)
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    B.moe_linear_w4(dims, x, w, None, None, out, *B.linear_w4_workspace(dims))
    return out, B.moe_linear_w4_plan(dims)


def sum_bound(X, V, codes, s, fmt, group):
    """fp32 sums of exact products, at most two per element (INT4: the digits 4 h and l of c - 8 = 4 h + l), one addition
    each and one per group, slice and wave: all within 2 K + K / group + 32 steps of their size."""
    K = X.shape[1]
    size = np.abs(V)
    if fmt == "int4":
        size = (np.abs(4.0 * ((codes >> 2).astype(int) - 2)) + (codes & 3)) * np.abs(np.repeat(s, group, axis=1))
    return (2 * K + K // group + 32) * U32 * (np.abs(X) @ size.T)


# one token and a few from LDS, groups of 16 in memory's lines, tiles, expanded
@pytest.mark.parametrize("M,N,K", [(1, 72, 512), (4, 72, 640), (13, 136, 1024), (40, 264, 512), (300, 4096, 2048), (1100, 136, 512)])
@pytest.mark.parametrize("fmt,group", FORMATS)
def test_a_large_element_on_weights_of_zero_adds_nothing(M, N, K, fmt, group):
    columns = [5, K // 2 + 3, K - 1]
    w, codes, s, V = with_zero_columns(N, K, fmt, group, M, columns)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(K)).bfloat16()
    x[:, columns] = 0.0
    plain, way = linear(x.cuda(), w, N)
    for big in (1e5, -1e7, 3e38):
        x[:, columns] = big
        X = f64(x)
        if way != "streamed":
            V = ow.bf16(V.astype(np.float32))
        ref = X @ V.T
        err = sum_bound(X, V, codes, s, fmt, group)
        got, _ = linear(x.cuda(), w, N)
        assert_within("x of %g" % big, f64(got), ref, HALF["bf16"] * (np.abs(ref) + err) + err)
    # (the large elements are nowhere in the bound)
    assert np.all(err <= 0.05)


@pytest.mark.parametrize("M,K", [(1, 256), (4, 256), (13, 256), (40, 256), (300, 2048), (1100, 256)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_products_over_the_finite_range(M, K, group):
    """The codes that quantisation gives times its largest scales with small tokens, the largest tokens under small scales
    and the smallest ones (subnormal digit products) under large scales: where (c - 8) s and its product with x are finite numbers, that is the result."""
    N = 4096
    codes = np.full((N, K), 8, np.uint8)
    row = np.arange(N)
    codes[row, row % K] = 1 + (row + row // K) % 15  # one element a row that counts, in every place of a block in turn
    for scale, x0 in ((4.8e37, 2.0 ** -40), (-4.8e37, 3.0 * 2.0 ** -50), (2.0 ** -10, 3.3e38), (-(2.0 ** -10), -3.3e38), (2.0 ** 60, 2.0 ** -126)):
        s = ow.bf16(np.full((N, K // group), scale, np.float32))
        (w,) = pack(codes, s, "int4", group)
        x = torch.full((M, K), x0).bfloat16()
        got, _ = linear(x.cuda(), w, N)
        ref = f64(x) @ ow.values(codes, s, "int4").T   # (one product that is not zero: exact)
        assert np.abs(ref).max() > 2.0 ** -70
        # (7 s and the like are rounded to bf16 beyond 64 rows)
        assert_within("scale %g, x %g" % (scale, x0), f64(got), ref, 2.01 * HALF["bf16"] * np.abs(ref))


@pytest.mark.parametrize("T", [2, 100])  # by pairs, by experts
@pytest.mark.parametrize("fmt,group", FORMATS)
def test_decode_with_a_large_element_on_weights_of_zero(T, fmt, group):
    d, n, E, K = 512, 256, 6, 3
    columns = [7, 300]
    gate, up = (with_zero_columns(E * n, d, fmt, group, seed, columns)[0] for seed in (1, 2))
    down = random_w4(E * d, n, fmt, group, 3)[0]
    g = torch.Generator().manual_seed(T)
    X, W_r = torch.randn(T, d, generator=g).bfloat16(), (torch.randn(E, d, generator=g) * 0.05).bfloat16()
    X[:, columns], W_r[:, columns] = 0.0, 0.0
    dims = B.make_dims(T, d, n, E, K)
    logits, idx = torch.empty(T, E, device="cuda"), torch.empty(T, K, dtype=torch.int32, device="cuda")
    tw, out = torch.empty(T, K, device="cuda"), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    W_r = W_r.cuda()

    def decode():
        B.moe_decode_w4(dims, X.cuda(), W_r, None, gate, up, down, logits, idx, tw, out, *B.workspace(dims, B.OP_DECODE))
        return out.clone(), idx.clone()

    want, picked = decode()
    for big in (1e5, -3e38):
        X[:, columns] = big
        got, again = decode()
        assert torch.equal(again, picked)
        # (products of zero: no sum changes, so neither does the order of their roundings)
        assert torch.equal(got, want)
