"""The layer norm's workspace size by the public function (no GPU needed)."""
import torch

import prefix_sum_outer_gb300 as cp


def test_workspace_size():
    assert "causal_product_layer_norm_workspace_size" in cp.__all__
    lib = cp.load_library()
    for dtype, code in ((torch.float32, 0), (torch.bfloat16, 1), (torch.float16, 2)):
        for size in ((2, 4, 70, 64), (1, 1, 32768, 1024), (1, 1, 1, 1)):
            n = cp.causal_product_layer_norm_workspace_size(*size, dtype)
            assert n == lib.causal_product_layer_norm_workspace_size(*size, code) > 256
    assert cp.causal_product_layer_norm_workspace_size(2, 4, 70, 64) == \
        cp.causal_product_layer_norm_workspace_size(2, 4, 70, 64, torch.bfloat16)
    assert cp.causal_product_layer_norm_workspace_size(1, 1, 1, 40000) == 0  # a shape that is refused
