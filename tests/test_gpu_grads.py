"""moe_grad_norm and moe_grad_clip against float64."""
import math

import numpy as np
import pytest
import torch

from block_util import DT, GUARD, HALF, check_replays
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


def true_norm(tensors):
    return math.sqrt(math.fsum(float((t.cpu().double() ** 2).sum()) for t in tensors))


def close_norm(got, want):
    # fp64 sums: what is left is one rounding to fp32 (and 2^-40 for orders of the sum)
    return abs(float(got) - want) <= (2.0 ** -24 + 2.0 ** -40) * want


def clip(src, dst, max_norm, norm_in=None):
    norm = torch.full((1,), -1.0, device="cuda")
    g = B.Gradients(src, dst)
    ws, nb = B.grad_workspace(g)
    B.moe_grad_clip(g, max_norm, norm_in, norm, ws, nb)
    torch.cuda.synchronize()
    return norm


def check_scaled(src, dst, factor):
    for i, (s, d) in enumerate(zip(src, dst)):
        h = HALF["bf16" if s.dtype == torch.bfloat16 else "f32"]
        ref = s.double() * factor
        # the factor in fp32, the product in fp32, the result's rounding; below the normal range steps are fixed
        tol = (h + 3 * 2.0 ** -24) * ref.abs() + 2.0 ** -133
        assert bool(((d.double() - ref).abs() <= tol).all()), "tensor %d of %d elements" % (i, s.numel())


def tensors(sizes, dtypes, seed=0, std=1.0, offset=0):
    """Views with `offset` elements before them and guards around, so that none lies on a 16-byte border for
    odd offsets."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out, bases = [], []
    for i, n in enumerate(sizes):
        base = torch.full((n + offset + 3,), GUARD, dtype=DT[dtypes[i % len(dtypes)]], device="cuda")
        v = base[offset:offset + n]
        v.copy_(torch.randn(n, generator=g, device="cuda") * std)
        out.append(v)
        bases.append(base)
    return out, bases


LISTS = [
    ([1], ["f32"]), ([1], ["bf16"]), ([7, 0, 9], ["bf16", "f32"]), ([8191, 8192, 8193], ["f32"]), ([8191, 8192, 8193, 1], ["bf16"]),
    ([100003], ["bf16", "f32"]), ([0, 0], ["f32"]), ([3, 5, 1000, 70001, 2], ["bf16", "f32", "f32"]),
    (list(range(1, 112)), ["f32"]), (list(range(1, 114)), ["bf16", "f32"]), ([17, 4097, 0, 250] * 150, ["f32", "bf16", "bf16"]),
    ([3000001, 20000000, 11], ["bf16", "f32"]), ([0] * 120 + [5] + [0] * 130 + [9], ["f32"]),
]


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("sizes,dtypes", LISTS)
def test_norm_and_clip_match_float64(sizes, dtypes, offset):
    src, _ = tensors(sizes, dtypes, len(sizes), offset=offset)
    keep = [t.clone() for t in src]
    want = true_norm(src)
    g = B.Gradients(src)
    norm = torch.full((2,), -1.0, device="cuda")
    ws, nb = B.grad_workspace(g)
    B.moe_grad_norm(g, norm, ws, nb)
    torch.cuda.synchronize()
    assert close_norm(norm[0], want) and float(norm[1]) == -1.0
    for max_norm in (want * 0.37, want * 2 + 1, float("inf"), 0.0):
        dst, bases = tensors(sizes, dtypes, 99, offset=offset)
        n = clip(src, dst, max_norm)
        assert torch.equal(n, norm[:1])
        cut = want > max_norm
        check_scaled(src, dst, max_norm / want if cut else 1.0)
        if not cut:
            assert all(torch.equal(a, b) for a, b in zip(src, dst))
        for b, s in zip(bases, src):  # nothing written around them
            assert bool((b[:offset] == GUARD).all()) and bool((b[offset + s.numel():] == GUARD).all())
        # in place: the same values
        mine = [t.clone() for t in keep]
        clip(mine, None, max_norm)
        assert all(torch.equal(a, b) for a, b in zip(mine, dst))
    assert all(torch.equal(a, b) for a, b in zip(src, keep))
    # a norm given: used as it is
    half = norm[:1] * 0.5
    dst, _ = tensors(sizes, dtypes, 99, offset=offset)
    n = clip(src, dst, want * 0.25, half)
    assert float(n) == -1.0
    check_scaled(src, dst, 0.5 if want > 0 else 1.0)


@pytest.mark.parametrize("std", [1e-40, 1e-30, 1e20, 1e37])
def test_norms_whose_squares_leave_the_fp32_range(std):
    src, _ = tensors([1000, 20001], ["f32", "bf16"], 3, std)
    want = true_norm(src)
    n = clip(src, [t.clone() for t in src], 1.0)
    if want > 2.0 ** 128:  # the nearest fp32 number is infinity, and nothing is scaled then
        assert float(n) == float("inf")
        dst = [torch.empty_like(t) for t in src]
        clip(src, dst, want / 4)
        assert all(torch.equal(a, b) for a, b in zip(src, dst))
        return
    # (a norm below the normal range has a fixed step of 2^-149)
    assert abs(float(n) - want) <= (2.0 ** -24 + 2.0 ** -40) * want + 2.0 ** -150
    dst = [torch.empty_like(t) for t in src]
    clip(src, dst, want / 4)
    check_scaled(src, dst, 0.25)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("where", [0, 1, 2])
def test_a_norm_that_is_not_finite_changes_nothing(bad, where):
    src, _ = tensors([70000, 3, 9000], ["f32", "bf16"], 5)
    src[where][src[where].numel() // 2] = bad
    dst = [torch.zeros_like(t) for t in src]
    n = clip(src, dst, 0.5)
    assert math.isnan(float(n)) if math.isnan(bad) else float(n) == float("inf")
    for s, d in zip(src, dst):
        assert torch.equal(s.view(torch.int16 if s.dtype == torch.bfloat16 else torch.int32), d.view(torch.int16 if s.dtype == torch.bfloat16 else torch.int32))
    mine = [t.clone() for t in src]
    clip(mine, None, 0.5, torch.full((1,), bad, device="cuda"))
    for s, d in zip(src, mine):
        assert torch.equal(s.nan_to_num(1e9), d.nan_to_num(1e9))


def test_no_tensors():
    n = clip([], [], 1.0)
    assert float(n) == 0.0
    norm = torch.full((1,), -1.0, device="cuda")
    g = B.Gradients([])
    ws, nb = B.grad_workspace(g)
    B.moe_grad_norm(g, norm, ws, nb)
    assert float(norm) == 0.0


def test_a_tensor_past_2_to_the_31_elements():
    n = (1 << 31) + 8192 * 3 + 5
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[-1], t[1 << 31], t[5] = 3.0, 4.0, 12.0
    norm = clip([t], None, 6.5)
    assert float(norm) == 13.0
    assert float(t[-1]) == 1.5 and float(t[1 << 31]) == 2.0 and float(t[5]) == 6.0 and int(t.count_nonzero()) == 3


def test_graph_replays_match_eager():
    src, _ = tensors([5, 70000, 123] * 60, ["f32", "bf16"], 8)
    dst = [torch.empty_like(t) for t in src]
    g = B.Gradients(src, dst)
    ws, nb = B.grad_workspace(g)
    norm = torch.empty(1, device="cuda")
    check_replays(lambda: B.moe_grad_clip(g, 2.0, None, norm, ws, nb), dict(norm=norm, a=dst[1], b=dst[178], c=dst[0]))
    # new values in the same tensors reach a replay
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_grad_clip(g, 2.0, None, norm, ws, nb)
    for t in src:
        t.mul_(2.0)
    want = true_norm(src)
    graph.replay()
    torch.cuda.synchronize()
    assert close_norm(norm[0], want)
    check_scaled(src, dst, 2.0 / want)


def test_norm_of_parts_joins_to_the_whole():
    """Two ranks' norms joined by the caller give each the clipping of the whole."""
    a, _ = tensors([5000, 17], ["f32", "bf16"], 1)
    b, _ = tensors([9000, 3], ["bf16", "f32"], 2)
    norms = []
    for part in (a, b):
        g = B.Gradients(part)
        ws, nb = B.grad_workspace(g)
        norms.append(torch.empty(1, device="cuda"))
        B.moe_grad_norm(g, norms[-1], ws, nb)
    whole = torch.sqrt(norms[0].double() ** 2 + norms[1].double() ** 2).float()
    da, db, dall = ([torch.empty_like(t) for t in p] for p in (a, b, a + b))
    clip(a, da, 1.0, whole)
    clip(b, db, 1.0, whole)
    clip(a + b, dall, 1.0)
    for x, y in zip(da + db, dall):
        h = HALF["bf16" if x.dtype == torch.bfloat16 else "f32"]
        assert bool(((x.double() - y.double()).abs() <= (2 * h + 2.0 ** -21) * y.double().abs() + 1e-37).all())


def test_stream_of_its_own():
    src, _ = tensors([300000, 11], ["bf16", "f32"], 4)
    want = [torch.empty_like(t) for t in src]
    n0 = clip(src, want, 1.0)
    st = torch.cuda.Stream()
    dst = [torch.empty_like(t) for t in src]
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        n1 = clip(src, dst, 1.0)
    torch.cuda.synchronize()
    assert torch.equal(n0, n1) and all(torch.equal(a, b) for a, b in zip(want, dst))
    assert np.isfinite(float(n1))
