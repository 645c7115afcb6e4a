"""How many workgroups the norm's backward takes, by its workspace (a partial row of both gradients each); no GPU needed."""
import pytest

from mixture_experts_layer_lds_amd import binding as B


@pytest.mark.parametrize("rows,cols,dtype,groups", [
    (32768, 1536, "bf16", 512), (32768, 1600, "bf16", 1024), (32768, 2048, "bf16", 1024), (32768, 2560, "bf16", 1024), (4096, 2048, "bf16", 1024),
    # fp32 rows are twice the bytes; few rows a workgroup would leave a partial row for each
    (32768, 2048, "f32", 512), (4095, 2048, "bf16", 512), (32768, 4096, "bf16", 512), (32768, 7168, "bf16", 256), (32768, 8200, "bf16", 256), (100, 2048, "bf16", 100),
    (1, 8, "bf16", 1), (33, 8, "bf16", 2),
])
def test_workgroups_of_the_backward(rows, cols, dtype, groups):
    dims = B.make_norm_dims(rows, cols, dtype)
    assert B.lib().moe_norm_workspace_bytes(dims) == groups * 2 * -(-cols // 8) * 8 * 4
