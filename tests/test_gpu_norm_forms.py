"""moe_norm and moe_norm_backward in more of the forms that a call may take, against the float64 oracle."""
import numpy as np
import pytest
import torch

import test_gpu_norm as tn
from block_util import DT, HALF, U32, assert_guards, assert_within, f64, strided
from conftest import announce_case
from mixture_experts_layer_lds_amd import binding as B
from oracle import block as ob

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def announce(request):
    announce_case(request.node.nodeid)
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    yield
    torch.cuda.empty_cache()


# workgroups of two waves: 1024 of them, which take several rows each
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,cols,pad", [(4100, 2048, 0), (4500, 2049, 7)])
def test_many_rows_of_two_waves(rows, cols, pad, dtype, wtype, kind):
    tn.test_norm_matches_oracle(rows, cols, pad, dtype, wtype, kind)
    tn.test_norm_backward_matches_oracle(rows, cols, pad, dtype, wtype, kind)
