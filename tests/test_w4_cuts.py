"""The products that tests/test_gpu_w4_cuts.py lists reach every way and cut that the plan of moe_linear_w4 takes; no GPU
needed."""
import itertools

import pytest

from mixture_experts_layer_lds_amd import binding as B
from test_gpu_w4 import FORMATS
from test_gpu_w4_cuts import CUTS, cut, depth

M_ALL = [1, 2, 3, 4, 5, 9, 16, 17, 24, 32, 33, 48, 64, 65, 80, 100, 128, 129, 200, 256, 257, 385, 512, 513, 700, 777, 900, 1024, 1025]
N_ALL = [8, 24, 72, 104, 136, 264, 400, 512, 648, 800, 1024, 1600, 2048, 2560, 4096, 4104, 7168, 8192, 10240, 14336, 20480, 32768, 65536]
K_ALL = [32, 128, 256, 384, 1024, 2048, 3584, 4096, 7168, 8192, 14336, 16384, 28672, 32768, 65536]


def test_the_cuts_that_a_plan_takes_are_all_tested():
    taken = {}
    for M, N, K, act in itertools.product(M_ALL, N_ALL, K_ALL, ("none", "swiglu")):
        taken.setdefault(cut(M, N, K, act), (M, N, K, act))
    assert len(taken) >= 30
    for fmt, group in FORMATS:
        tested = {cut(M, N, depth(K, group), act) for M, N, K, act in CUTS}
        missing = {k: v for k, v in taken.items() if k not in tested}
        assert not missing, (fmt, group, missing)


def test_the_query():
    lib = B.lib()
    d = B.make_linear_dims(100, 64, 256)
    assert lib.moe_linear_w4_cut(d, None, None, None) == lib.moe_linear_w4_plan(d) >= 0
    assert lib.moe_linear_w4_cut(None, None, None, None) == -1
    with pytest.raises(B.MoEError):
        B.moe_linear_w4_cut(B.make_linear_dims(100, 64, 40))
    assert B.moe_linear_w4_cut(B.make_linear_dims(0, 64, 256)) == ("streamed", 0, 0, 0)
    # slices need room for each one's sums
    for M, N, K, act in CUTS:
        d = B.make_linear_dims(M, N, K, "bf16", act)
        way, _, _, slices = B.moe_linear_w4_cut(d)
        nb = lib.moe_linear_w4_workspace_bytes(d)
        assert nb > 0 if way == "expanded" else nb == (slices * M * N * (2 if act == "swiglu" else 1) * 4 if slices > 1 else 0)
