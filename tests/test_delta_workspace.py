"""The workspace a caller hands to the gated delta rule's and the q/k norm's
calls: the C side sees a pointer and a size, so the binding refuses one on
another device or with gaps, and counts bytes, whatever the elements."""
import pytest
import torch

import prefix_sum_outer_gb300 as cp


def test_workspace_on_the_cpu_is_refused():
    with pytest.raises(RuntimeError):
        cp._delta_workspace(torch.zeros(4096, dtype=torch.uint8), 1024, torch.device("cuda", 0))


def test_workspace_with_gaps_is_refused():
    with pytest.raises(ValueError):
        cp._delta_workspace(torch.zeros(8192, dtype=torch.uint8)[::2], 1024, torch.device("cpu"))


def calls():
    import test_qk_rope_gpu as rope
    from test_delta_gpu import args, make

    x = make(1, 2, 1, 70, 64, 64, torch.bfloat16, seed=51, carry=True)
    y = rope.make(1, 2, 1, 20, 64, 32, "bf16", seed=52)
    _, ckpt = cp.causal_product_fwd_delta(*args(x), save=True)
    rows = (y["xq"], y["xk"], y["wq"], y["wk"], y["gq"], y["gk"], y["cos"], y["sin"])
    B, H, Hk, N, D, M = 1, 2, 1, 70, 64, 64
    sizes = [cp.causal_product_delta_workspace_size(B, H, Hk, N, D, M, torch.bfloat16, b)
             for b in (False, True)]
    sizes.append(cp.load_library().causal_product_qk_rope_workspace_size(1, 2, 1, 20, 64, 1))
    return zip(sizes, (lambda ws: cp.causal_product_fwd_delta(*args(x), workspace=ws),
                       lambda ws: cp.causal_product_bwd_delta(*args(x), x["go"], ckpt, workspace=ws),
                       lambda ws: cp.causal_product_qk_rope_bwd(*rows, workspace=ws)))


@pytest.mark.gpu
def test_calls():
    for n, call in calls():
        want = call(None)
        for bad in (torch.zeros(n, dtype=torch.uint8), torch.zeros(n, dtype=torch.uint8).pin_memory()):
            with pytest.raises(RuntimeError):
                call(bad)
        with pytest.raises(ValueError):
            call(torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2])
        with pytest.raises(cp.CausalProductError):
            call(torch.zeros(n // 4 - 1, device="cuda"))
        got = call(torch.zeros((n + 3) // 4, device="cuda"))   # float32, n bytes
        torch.cuda.synchronize()
        if torch.is_tensor(want):
            want, got = (want,), (got,)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
