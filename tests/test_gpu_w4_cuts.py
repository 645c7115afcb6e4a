"""moe_linear_w4 in every way and cut that its plan takes (CUTS lists a product for each), against float64."""
import pytest
import torch

from block_util import HALF, U32, assert_guards, strided
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from test_gpu_w4 import FORMATS, random_w4

# (M, N, K, act): tokens, columns and blocks that fill their tiles and such that do not
CUTS = [
    # up to 4 tokens from LDS; groups of 16 with one, two and four row tiles, then slices of the last
    (3, 200, 1120, "relu"), (2, 72, 2144, "swiglu"), (9, 200, 480, "gelu"), (16, 136, 1120, "swiglu"), (7, 7176, 256, "none"), (5, 4104, 288, "swiglu"), (6, 14344, 288, "silu"),
    (13, 7176, 160, "swiglu"), (11, 8200, 16384, "none"), (15, 4104, 16384, "swiglu"), (13, 4096, 14336, "none"), (9, 1608, 14336, "swiglu"), (10, 1608, 28672, "relu"),
    (6, 808, 28672, "swiglu"),
    # 32 tokens a workgroup
    (31, 200, 1120, "none"), (33, 104, 864, "swiglu"), (40, 20488, 96, "gelu"), (50, 10248, 160, "swiglu"), (33, 65528, 64, "none"), (50, 20488, 160, "swiglu"),
    (770, 200, 32768, "none"), (777, 104, 32768, "swiglu"), (17, 72, 14336, "silu"), (20, 40, 14336, "swiglu"), (30, 264, 16384, "none"), (17, 72, 16384, "swiglu"),
    # tiles: one and two row tiles a wave, whole and in slices
    (70, 8, 160, "none"), (67, 8, 160, "swiglu"), (1020, 648, 2176, "none"), (511, 808, 2048, "swiglu"), (100, 2056, 2048, "gelu"), (101, 1032, 2048, "swiglu"),
    (129, 10248, 160, "none"), (131, 4104, 160, "swiglu"), (129, 7176, 2048, "relu"), (65, 7176, 2048, "swiglu"), (103, 4104, 2048, "none"), (100, 2056, 2048, "swiglu"),
    (129, 7176, 2016, "none"), (150, 72, 416, "swiglu"),
    # expanded
    (1030, 72, 416, "silu"), (1025, 136, 288, "swiglu"),
]


def depth(K, group):
    """K cut to whole groups."""
    return max(K // group, 1) * group


def cut(M, N, K, act):
    """How the product goes: the way, row tiles, token groups, slices, and whether its epilogue is SwiGLU's."""
    return B.moe_linear_w4_cut(B.make_linear_dims(M, N, K, "bf16", act)) + (act == "swiglu",)


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


def activation(z, act, N):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "swiglu":
        return z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:]
    return z


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,group", FORMATS)
@pytest.mark.parametrize("M,N,K,act", CUTS)
def test_every_cut_matches_float64(M, N, K, act, fmt, group):
    K, NW = depth(K, group), 2 * N if act == "swiglu" else N
    way, _, token_groups, slices, _ = cut(M, N, K, act)
    w, codes, s, V = random_w4(NW, K, fmt, group, M + N + K)
    g = torch.Generator().manual_seed(M + 3 * N + 7 * K)
    pad = 8 * (M % 3)
    x, _ = strided(M, K, pad, "bf16", torch.randn(M, K, generator=g))
    bias = (torch.randn(NW, generator=g) * 0.5).cuda() if N % 3 else None
    res = strided(M, N, pad, "bf16", torch.randn(M, N, generator=g))[0] if M % 2 else None
    out, base = strided(M, N, pad, "bf16", extra_rows=2)
    dims = B.make_linear_dims(M, N, K, "bf16", act, ldx=K + pad, ldr=N + pad, ldy=N + pad)
    B.moe_linear_w4(dims, x, w, bias, res, out, *B.linear_w4_workspace(dims))
    # the sizes that fp32 sums carry: INT4's digits 4 h and l of c - 8 = 4 h + l where the codes are streamed
    V = torch.from_numpy(V).cuda()
    size = V.abs()
    if fmt == "int4" and way == "streamed":
        c = torch.from_numpy(codes.astype("int64")).cuda()
        size = ((4 * ((c >> 2) - 2)).abs() + (c & 3)).double() * torch.from_numpy(s).cuda().abs().repeat_interleave(group, 1)
    elif way != "streamed":
        V = V.float().bfloat16().double()  # (exact products of 4 and 8 bits, rounded once)
        size = V.abs()
    X = x.double()
    z = X @ V.T + (bias.double() if bias is not None else 0.0)
    # a slice's elements one after another in a wave (8 waves share what is at least 16 blocks; two products an element),
    # the groups' sums, the waves' and slices' joins
    share = -(-K // slices) if slices else K
    if way == "streamed" and token_groups and share >= 16 * 128:
        share = share // 8 + 128
    chain = 2 * share + share // group + 32
    ez = chain * U32 * (X.abs() @ size.T) + 2 * U32 * z.abs()
    y = activation(z, act, N)
    if act == "swiglu":
        a, u, ea, eu = z[:, :N], z[:, N:], ez[:, :N], ez[:, N:]
        ey = 1.1 * ea * (u.abs() + eu) + (a * torch.sigmoid(a)).abs() * eu
    else:
        ey = 1.13 * ez
    # the activation's own arithmetic: exponentials off by a few steps times their argument; GELU's tail
    ey = ey + y.abs() * U32 * (8 + 2 * z[:, :N].abs()) + (4e-5 * y.abs() if act == "gelu" else 0.0) + 1e-30
    ref = y + (res.double() if res is not None else 0.0)
    tol = HALF["bf16"] * (ref.abs() + ey) + ey + U32 * (y.abs() + (res.double().abs() if res is not None else 0.0))
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), "worst %.3g of the bound" % float((err / tol).max())
    # roundings to bf16 are half a step each; those of long sums, as a random walk, far less: a group that is missing or
    # taken twice is not (one of 32 in 32768 is a thirtieth of the result)
    assert float(err.norm()) <= 1.05 * HALF["bf16"] * float(ref.norm())
    assert_guards(base, M, N, "out")
