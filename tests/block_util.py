"""Helpers of the block operators' GPU tests: strided tensors with guarded gaps, and graph replays."""
import numpy as np
import torch

from parity import f64  # noqa: F401

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # a rounding to the type: half a step, relative
# fp32 sums: each partial sum may round (or, in the matrix unit, truncate) by one step of 2^-23
U32 = 2.0 ** -23
GUARD = 777.0


def strided(rows, cols, pad, dtype, fill=None, extra_rows=0):
    """(view [rows, cols], base): base holds GUARD outside the view (the gaps between rows, extra rows)."""
    base = torch.full((rows + extra_rows, cols + pad), GUARD, dtype=DT[dtype], device="cuda")
    v = base[:rows, :cols]
    if fill is not None:
        v.copy_(fill)
    return v, base


def assert_guards(base, rows, cols, what):
    assert bool((base[:, cols:] == GUARD).all()) and bool((base[rows:] == GUARD).all()), "%s: written outside its rows" % what


def assert_within(name, got, ref, tol):
    """|got - ref| <= tol, all arrays."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d off, worst |got-ref|/tol = %.3g at %s" % (
        name, bad.sum(), bad.size, np.nanmax(np.abs(got - ref) / np.broadcast_to(tol, ref.shape)), np.argwhere(bad)[0])


def check_replays(step, outs, replays=3):
    """Capture step, replay it with the outputs cleared and eager work in between, compare with eager."""
    step()
    torch.cuda.synchronize()
    ref = {k: v.clone() for k, v in outs.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    for rep in range(replays):
        for v in outs.values():
            v.fill_(0)
        noise = torch.randn(1 << 18, device="cuda").mul_(2.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(noise).all()
        for k, v in outs.items():
            assert torch.equal(v, ref[k]), "replay %d: %s differs from the eager call" % (rep, k)
